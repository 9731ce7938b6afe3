// grouped_linear_sm100.cu -- the grouped linear operators' products over the groups' rows
// on the tensor cores:
//   forward      out[r, f] = act(sum_c x[r, c] W_e[f, c] + b_e[f]) + residual[r, f]
//   transposed   out[r, f] = sum_c x[r, c] W_e[c, f]          (the backward's dx = dz W_e)
// for the rows r of each group e, with the pre-activation kept in 8 bits on request.
//
// The weights are the M operand and the tokens the N operand ("swapped"): a tile is 128
// features (256 on a pair of SMs) x up to 256 tokens, and the tensor core's time goes with
// the tokens' number in steps of 16 (32 on a pair), so a ragged group wastes less than one
// such step where token rows on the M side would waste up to 127.  The tokens of a group
// are cut into the fewest tiles of at most 256, all of nearly the same width.
//
// Layout: every CTA is persistent; warp 0 feeds a ring of TMA stages (64 of the reduction:
// 128 features, 16 KiB, over the tile's token rows), warp 1 issues
// tcgen05.mma (fp32 accumulator in TMEM, two of 256 columns), warps 2-17 drain the
// other accumulator.  The ring's stage size goes by the widest tile of this call, read from
// `offsets` on the device: 11 stages for 16 tokens, 6 on a pair for 256.  Forward weights
// are K-major; the transposed product reads the same weights MN-major (64 x 64 boxes).
//
// Epilogue: TMEM lanes are features and columns tokens, so a warp turns its 32 features x
// eight tokens at a time in shared memory of its own (neither side meets a bank twice) and
// comes back with eight consecutive features of one token per thread: bias, residual,
// activation and the output are 16-byte accesses, 64 bytes of a row together, and a
// checkpoint block of 32 features is four neighbouring lanes (two shuffles for its largest
// magnitude).  Sixteen warps, because the rounds are chains of latencies.
//
// Split reduction (single SMs): tiles are dealt out round by round.  Where the last round
// would leave SMs idle, its tiles are cut along the reduction instead (equal shares of all
// remaining 64-steps, at most two tiles each): every share's fp32 tile goes to the
// workspace, and the CTA that finishes a tile last adds the shares in the order of the
// reduction, whoever it is, so the result does not depend on the timing; nobody waits for
// anybody.  Pairs do not share: they run at the power limit, where an idle SM lets the others
// clock higher (4096 x 14336 x 4096: 1286 TFLOP/s unshared, 1232 shared).
//
// Measured, rows x K x N in TFLOP/s after a pause (cuBLAS in parentheses): 4096^3 1440 (1500),
// 4096 x 14336 x 4096 1419 (1527), 8192 x 4096 x 14336 1569 (1527), 4096 x 2048 x 7168 1403
// (1325), 8192 x 512 x 7168 956 (938); without pauses the power limit takes a fifth.  8 experts,
// 32 rows, 14336 -> 4096: 134 to 143 us, 98 to 106 % of a copy's bandwidth.
//
// Every wait is bounded (sm100_ptx.cuh).
#include <cuda.h>
#include <cuda_bf16.h>

#include "linear_device.cuh"
#include "moe_internal.h"
#include "sm100_ptx.cuh"

namespace moe {

// Defined in grouped_gemm_sm100.cu.
bool encode_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                    uint32_t box_rows);
bool encode_bf16_3d(CUtensorMap* map, const void* base, uint64_t batches, uint64_t rows,
                    uint64_t cols, uint32_t box_rows);

namespace {

constexpr int kBK = 64;                // reduction per stage
constexpr int kF = 128;                // features per CTA (TMEM lanes)
constexpr int kTokens = 256;           // token columns of an accumulator
constexpr int kABytes = kF * kBK * 2;  // 16 KiB
constexpr int kRingBytes = 204 * 1024;
constexpr int kMaxStages = 11;
constexpr int kEpiGroups = 4;          // of four warps, one for each quarter of the lanes;
constexpr int kEpiWarps = 4 * kEpiGroups;  // they take the rounds of columns in turn
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 64 + kEpiThreads;
constexpr int kRound = 8;              // token columns per epilogue round
constexpr int kPitch = 32 + 4;         // staged token row of a warp, floats
constexpr int kStagingBytes = kEpiWarps * kRound * kPitch * 4;
constexpr int kBookBytes = 1024;
constexpr int kSmemBytes = kRingBytes + kStagingBytes + kBookBytes + 1024 /*align*/;
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr int kVoteBarrier = 1;
constexpr int kJoinBarrier = 2;
constexpr uint16_t kBothCtas = 0x3;
constexpr int kMinShare = 4;           // 64-steps of a share, at least
constexpr int kPrefetchSteps = 20;     // 64-steps of a tile up to which its residual is prefetched

// What a CTA's work takes, in clocks; fitted to measurements, to choose among layouts.  A
// stage of 128 features x `width` tokens: the tensor core's time, two clocks a token (on a pair
// both halves), or what issuing it or loading its 128-byte rows takes.  Measured with rows on
// 128-byte boundaries:
//   width            32   64   96  128  160  192  224  256
//   pairs, clocks   270  280  302  333  369  399  461  517
//   single SMs      295  309  339  390  453  484  596  625
// Rows that lie across two lines take longer, most of all across 32-byte sectors (3 groups, 300
// rows, K -> 5000, us on pairs and on single SMs: K = 4992 31 and 29, 5024 31 and 38, 5008 32
// and 39, 5000 33 and 45).
struct RowClocks {
    float w, x;  // a row of weights, of tokens
};
inline float row_clocks(int length) {
    return length % 64 == 0 ? 1.6f : (length % 16 == 0 ? 2.4f : 4.1f);
}
__host__ __device__ inline float stage_clocks(int width, bool pair, RowClocks row) {
    const float w = static_cast<float>(width);
    const float tensor = 2.02f * w;
    const float issue = pair ? 230.f + 0.8f * w : 245.f + 1.15f * w;
    const float load = kF * row.w + (pair ? 0.5f : 1.f) * w * row.x;
    return fmaxf(fmaxf(tensor, issue), load);
}
// A tile's epilogue with its turn of the accumulators; 256 and 128 tokens measured: plain 6700
// and 4300, with a GELU 9600 and 5900; single SMs a tenth more.  (With the checkpoint 12000 and
// 7000, which does not count here: training and inference take the same layout and so give the
// same y to the bit.)
inline float epilogue_clocks(const LinearArgs& a, int width, bool pair) {
    const float token = 19.f + (a.act >= MOE_ACT_GELU ? 10.f : 0.f) +
                        (a.residual != nullptr ? 12.f : 0.f);
    return (pair ? 1.f : 1.1f) * (1900.f + token * static_cast<float>(width));
}
// Pairs: a cluster's launch and its two synchronisations, without programmatic launch (4
// groups, 1900 rows, 1472 -> 1504: 16.5 us on pairs, 13.5 on single SMs).  Shares: writing one,
// and the joins below.
constexpr float kJoinClocks = 2200.f, kShareClocks = 3000.f, kPairClocks = 6500.f;

// How many CTAs (0: none) share the reduction of the last `rem` tiles, and the clocks.  No
// integer division: every thread goes through this before its first piece of work.
constexpr int kMostSteps = 1 << 15;  // of a shared reduction: 160 x 160 of them fit 32 bits
struct Sharing {
    int ctas;
    float clocks;
    __host__ __device__ Sharing(int rem, int num_kb, int width, int G, RowClocks row) {
        const float stage = stage_clocks(width, false, row), whole = num_kb * stage;
        ctas = 0;
        clocks = whole;
        if (rem == 0 || num_kb < 2 * kMinShare || num_kb >= kMostSteps) return;
        const float join = static_cast<float>((width + 31) / 32) * kJoinClocks;
        // the number of shares a tile where more of them cost as much as they save
        const int best = static_cast<int>(sqrtf(4.f * whole / join));
        int most = rem * (best < 2 ? 2 : best);
        if (most > rem * num_kb / kMinShare) most = rem * num_kb / kMinShare;
        if (most > G) most = G;
        if (most <= rem) return;
        // .. all of them, or a whole number a tile, which none then crosses
        const float each = static_cast<float>(most) / static_cast<float>(rem);
        const float even = floorf(each);
        const float crossing = cost(each, ceilf(each) + 1.f, num_kb, stage, join) + join +
                               kShareClocks;  // its two pieces come after one another
        const float aligned = even < 2.f ? crossing : cost(even, even, num_kb, stage, join);
        const bool align = aligned <= crossing && even >= 2.f;
        const float shared = align ? aligned : crossing;
        if (shared >= whole) return;
        ctas = align ? static_cast<int>(even) * rem : most;
        clocks = shared;
    }
    // `each` shares a tile on average, `most` at most: the join adds four at a time
    __host__ __device__ static float cost(float each, float most, int num_kb, float stage,
                                          float join) {
        return (num_kb / each + 1.f) * stage + ceilf(most * 0.25f) * join + kShareClocks;
    }
};

struct Args {
    const int32_t* offsets;
    int E, rows;
    int F;                // output features
    int C;                // reduction length
    int width;            // most token columns of a tile
    int group;            // token tiles whose rows stay in L2 together
    int act;
    const __nv_bfloat16* bias;
    const __nv_bfloat16* residual;
    void* out;
    int out_f32;
    int8_t* codes;
    float* scales;
    uint32_t* counters;
    float* partials;
    int slot_tokens;
    RowClocks row;
    uint32_t* status;
};

// Token rows in boxes of 16, 32, .. 128, so that a tile's half (pair) or its one or two
// parts arrive with one TMA load each and nothing more is read.
constexpr int kBoxes = 8;
struct TokenMaps {
    CUtensorMap box[kBoxes];
};

struct Book {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int last;                         // this CTA joins the tile's shares
    int off[kMaxExperts + 1];
    int tile_start[kMaxExperts + 1];
    int stages, stage_bytes;
    int one_tile_each;                // no group has a second token tile
    int widest;                       // token columns of the widest tile
};
static_assert(sizeof(Book) <= kBookBytes, "bookkeeping reserve");

struct Tile {
    int e, f0, row0, n, nt;  // n tokens from output row row0 on, nt columns (n rounded up)
};

// `g`: a group at or before the tile's; left at the tile's, since a CTA's tiles come in
// ascending order.  STEP: granularity of a tile's token columns.
template <int STEP>
__device__ __forceinline__ Tile decode_tile(const Book& bk, const Args& a, int ftiles, int fwidth,
                                            int tile, int& g) {
    while (g + 1 < a.E && tile >= bk.tile_start[g + 1]) ++g;
    const int local = tile - bk.tile_start[g];
    const int row0 = bk.off[g], n = bk.off[g + 1] - row0;
    int rest;
    const int tt = divide(n + a.width - 1, a.width, rest);
    // token tiles in runs of `group`; inside a run feature tiles are outer and token tiles
    // inner, so that CTAs running together share the weights
    int r = local, first = 0, width = tt;
    if (tt > a.group) {
        first = divide(local, a.group * ftiles, r) * a.group;
        width = tt - first < a.group ? tt - first : a.group;
    }
    int i, more;
    const int ft = divide(r, width, i);
    i += first;
    const int base = divide((n + STEP - 1) / STEP, tt, more);
    const int start = (i * base + (i < more ? i : more)) * STEP;
    Tile t;
    t.e = g;
    t.f0 = ft * fwidth;
    t.row0 = row0 + start;
    t.nt = (base + (i < more ? 1 : 0)) * STEP;
    t.n = n - start < t.nt ? n - start : t.nt;
    return t;
}

// The work of CTA (or pair) c of G, in pieces: its share of the last `rem` tiles'
// reduction (up to two tiles; first, so that joining the shares overlaps the rest), then
// `rounds` whole tiles; or, without shares, rounds whole tiles and maybe one more.
struct Plan {
    int G, c, num_kb, rounds, rem, share_ctas;
    int pieces;             // of this CTA's share: 0, 1 or 2
    int first, from, to;    // the share: 64-steps from .. to, counted from its first tile
    __device__ __forceinline__ Plan(int G_, int c_, int total, int num_kb_, int widest, bool may_share,
                                    RowClocks row)
        : G(G_), c(c_), num_kb(num_kb_) {
        rounds = divide(total, G, rem);
        share_ctas = pieces = first = from = to = 0;
        if (rem > 0 && may_share) {
            share_ctas = Sharing(rem, num_kb, widest, G, row).ctas;
            if (c < share_ctas) {
                const int u0 = bound(c), u1 = bound(c + 1);
                first = divide(u0, num_kb, from);
                to = from + u1 - u0;
                pieces = to > num_kb ? 2 : 1;
            }
        }
    }
    __device__ __forceinline__ int bound(int i) const {  // first 64-step of share i
        int rest;
        return divide(i * rem * num_kb, share_ctas, rest);
    }
    // Piece i of this CTA's work; false when there is none.
    __device__ __forceinline__ bool get(int i, int& tile, int& kb0, int& kb1) const {
        if (i < pieces) {
            tile = rounds * G + first + i;
            kb0 = i == 0 ? from : 0;
            kb1 = i == 0 ? (to < num_kb ? to : num_kb) : to - num_kb;
            return true;
        }
        i -= pieces;
        kb0 = 0;
        kb1 = num_kb;
        tile = i * G + c;
        return i < rounds || (i == rounds && share_ctas == 0 && c < rem);
    }
    // The share that holds the remaining tiles' 64-step u.
    __device__ __forceinline__ int holder(int u) const {
        int rest, i = divide(u * share_ctas, rem * num_kb, rest);
        while (i + 1 < share_ctas && bound(i + 1) <= u) ++i;
        while (i > 0 && bound(i) > u) --i;
        return i;
    }
};

// The pieces of a CTA's work one after the other, decoded.
template <int STEP>
struct Pieces {
    int i = -1, g = 0;
    int tile, kb0, kb1;
    Tile t;
    __device__ __forceinline__ bool next(const Plan& plan, const Book& bk, const Args& a,
                                         int ftiles, int fwidth) {
        if (++i == plan.pieces) g = 0;  // from the shares back to the first whole tile
        if (!plan.get(i, tile, kb0, kb1)) return false;
        t = decode_tile<STEP>(bk, a, ftiles, fwidth, tile, g);
        return true;
    }
};

template <bool PAIR, bool TRANSPOSED>
__global__ void __launch_bounds__(kThreads, 1)
    linear_sm100_kernel(const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ TokenMaps tmX, const Args args) {
    constexpr int kCtas = PAIR ? 2 : 1;
    constexpr int kStep = PAIR ? 32 : 16;
    constexpr int kTileF = kF * kCtas;
    constexpr uint32_t kTmemCols = 2 * kTokens;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* staging = reinterpret_cast<float*>(smem + kRingBytes);
    Book& bk = *reinterpret_cast<Book*>(smem + kRingBytes + kStagingBytes);
    volatile int* abort_flag = &bk.abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int ftiles = (args.F + kTileF - 1) / kTileF;
    const int num_kb = (args.C + kBK - 1) / kBK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&bk.full[s], 1);
            mbar_init(&bk.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&bk.tmem_full[a], 1);
            mbar_init(&bk.tmem_empty[a], kCtas * kEpiWarps);
        }
        mbar_init(&bk.drain, 1);
        bk.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        if (PAIR)
            tmem_alloc_pair(&bk.tmem_base, kTmemCols);
        else
            tmem_alloc(&bk.tmem_base, kTmemCols);
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {
        load_group_bounds(args.offsets, args.E, args.rows, bk.off);
        // lane g: group g's token tiles; tile_start is their running sum
        const int n = lane < args.E ? bk.off[lane + 1] - bk.off[lane] : 0;
        const int tt = (n + args.width - 1) / args.width;
        int sum = tt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int below = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += below;
        }
        if (lane < args.E) bk.tile_start[lane + 1] = sum * ftiles;
        const int units = (n + kStep - 1) / kStep;
        const int width = tt > 0 ? (units + tt - 1) / tt * kStep : kStep;
        const int widest = __reduce_max_sync(0xffffffffu, width);
        const int most = __reduce_max_sync(0xffffffffu, tt);
        if (lane == 0) {
            bk.tile_start[0] = 0;
            bk.stage_bytes = kABytes + widest / kCtas * kBK * 2;
            const int fit = kRingBytes / bk.stage_bytes;
            bk.stages = fit < kMaxStages ? fit : kMaxStages;
            bk.one_tile_each = most <= 1;
            bk.widest = widest;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();

    const uint32_t tmem_base = bk.tmem_base;
    const int stages = bk.stages, stage_bytes = bk.stage_bytes;
    const Plan plan(gridDim.x / kCtas, blockIdx.x / kCtas, bk.tile_start[args.E], num_kb,
                    bk.widest, !PAIR, args.row);
    Pieces<kStep> cur;
    auto next_piece = [&]() { return cur.next(plan, bk, args, ftiles, kTileF); };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (elect_one()) {
            int stage = 0;
            uint32_t phase = 0, pending = 0, pending_phase = 0;
            bool ok = true, issued = false;
            // weights that no second token tile reads again leave L2 first
            const bool stream = bk.one_tile_each != 0;
            const uint64_t policy = l2_policy_evict_first();
            while (ok && next_piece()) {
                const Tile t = cur.t;
                const int kb0 = cur.kb0, kb1 = cur.kb1;
                const int half = t.nt / kCtas;
                const int n0 = half < 128 ? half : 128, n1 = half - n0;
                const CUtensorMap* map0 = &tmX.box[n0 / 16 - 1];
                const CUtensorMap* map1 = &tmX.box[n1 > 0 ? n1 / 16 - 1 : 0];
                const int x_row = t.row0 + static_cast<int>(rank) * half;
                const int f = t.f0 + static_cast<int>(rank) * kF;
                const uint32_t bytes = static_cast<uint32_t>(kABytes + half * kBK * 2);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait_asleep(&bk.empty[stage], phase ^ 1u, abort_flag,
                                           args.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t* w = smem + stage * stage_bytes;
                    uint8_t* x = w + kABytes;
                    const int c = kb * kBK;
                    if (PAIR) {
                        const uint32_t bar = map_to_cta(smem_u32(&bk.full[stage]), 0);
                        if (leader) mbar_arrive_expect_tx(&bk.full[stage], 2 * bytes);
                        auto load_w = [&](uint8_t* dst, int c0, int c1) {
                            if (stream)
                                tma_load_3d_pair_hint(&tmW, bar, dst, c0, c1, t.e, policy);
                            else
                                tma_load_3d_pair(&tmW, bar, dst, c0, c1, t.e);
                        };
                        if (TRANSPOSED) {
                            load_w(w, f, c);
                            load_w(w + kMnBoxBytes, f + 64, c);
                        } else {
                            load_w(w, c, f);
                        }
                        tma_load_2d_pair(map0, bar, x, c, x_row);
                    } else {
                        uint64_t* bar = &bk.full[stage];
                        mbar_arrive_expect_tx(bar, bytes);
                        auto load_w = [&](uint8_t* dst, int c0, int c1) {
                            if (stream)
                                tma_load_3d_hint(&tmW, bar, dst, c0, c1, t.e, policy);
                            else
                                tma_load_3d(&tmW, bar, dst, c0, c1, t.e);
                        };
                        if (TRANSPOSED) {
                            load_w(w, f, c);
                            load_w(w + kMnBoxBytes, f + 64, c);
                        } else {
                            load_w(w, c, f);
                        }
                        tma_load_2d(map0, bar, x, c, x_row);
                        if (n1 > 0) tma_load_2d(map1, bar, x + 128 * kBK * 2, c, x_row + 128);
                    }
                    issued = true;
                    pending |= 1u << stage;
                    pending_phase = (pending_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && issued) {
                if (leader) {
                    for (int s = 0; s < stages; ++s)
                        if (pending & (1u << s)) drain_wait(&bk.full[s], (pending_phase >> s) & 1u);
                } else {
                    // the peer's copies complete on the leader's barriers: time to land
                    // before this CTA's shared memory can be released
                    short_pause_ns(2000000ull);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (leader)
        if (leader && elect_one()) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, issued = false;
            while (ok && next_piece()) {
                const int kb0 = cur.kb0, kb1 = cur.kb1;
                const uint32_t idesc = idesc_bf16_f32_major(kTileF, cur.t.nt, TRANSPOSED, false);
                if (!mbar_wait_asleep(&bk.tmem_empty[acc], acc_phase ^ 1u, abort_flag,
                                       args.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kTokens);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait_asleep(&bk.full[stage], phase, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t w = smem_u32(smem + stage * stage_bytes);
                    const uint64_t wd = TRANSPOSED ? sw128_mn_desc(w) : sw128_kmajor_desc(w);
                    const uint64_t xd = sw128_kmajor_desc(w + kABytes);
                    constexpr uint64_t kWStep = TRANSPOSED ? kMnDescStep : kKDescStep;
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k) {
                        const uint32_t accumulate = (kb != kb0 || k != 0) ? 1u : 0u;
                        if (PAIR)
                            umma_bf16_pair(d_tmem, wd + kWStep * k, xd + kKDescStep * k, idesc,
                                           accumulate);
                        else
                            umma_bf16(d_tmem, wd + kWStep * k, xd + kKDescStep * k, idesc,
                                      accumulate);
                    }
                    if (PAIR)
                        umma_commit_pair(&bk.empty[stage], kBothCtas);
                    else
                        umma_commit(&bk.empty[stage]);
                    issued = true;
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (PAIR)
                    umma_commit_pair(&bk.tmem_full[acc], kBothCtas);
                else
                    umma_commit(&bk.tmem_full[acc]);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok && issued) {
                if (PAIR)
                    umma_commit_pair(&bk.drain, 0x1);
                else
                    umma_commit(&bk.drain);
                drain_wait(&bk.drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const int group = (warp - 2) >> 2;
        const int my_tok = lane >> 2;                 // this thread's token of a round
        const int my_f = q * 32 + (lane & 3) * 8;     // and the first of its eight features
        float* my_staging = staging + (warp - 2) * kRound * kPitch;
        const float* get = my_staging + my_tok * kPitch + (lane & 3) * 8;
        const int nb = ckpt_blocks(args.F);
        const uint32_t free0 = PAIR ? map_to_cta(smem_u32(&bk.tmem_empty[0]), 0) : 0u;
        const uint32_t free1 = PAIR ? map_to_cta(smem_u32(&bk.tmem_empty[1]), 0) : 0u;
        auto release = [&](int acc) {
            tc_fence_before();
            __syncwarp();
            if (lane != 0) return;
            if (PAIR)
                mbar_arrive_cluster_light(acc == 0 ? free0 : free1);
            else
                mbar_arrive(&bk.tmem_empty[acc]);
        };
        auto sync_epilogue = [&]() {
            asm volatile("bar.sync %0, %1;" ::"n"(kJoinBarrier), "n"(kEpiThreads) : "memory");
        };
        const size_t slot_floats = static_cast<size_t>(kF) * args.slot_tokens;
        int acc = 0;
        uint32_t acc_phase = 0;
        while (next_piece()) {
            const Tile t = cur.t;
            const int i = cur.i, tile = cur.tile, kb0 = cur.kb0, kb1 = cur.kb1;
            const int f = t.f0 + static_cast<int>(rank) * kF + my_f;
            const bool have_f = f < args.F;  // F is a multiple of 8: all eight or none
            float bias[8] = {};
            if (args.bias != nullptr && have_f)
                load8(args.bias + static_cast<size_t>(t.e) * args.F + f, bias);
            // Where the epilogue is the bound, the residual is fetched to L2 ahead of it: 9472 x
            // K -> 8192 with K = 512: 134 -> 101 us, 1024: 138 -> 109, 1280: 142 -> 122; longer
            // reductions leave it time, and there the burst only disturbs (2048: 161 -> 168).
            // A CTA's first tile gains nothing either (600 x 1024 -> 7168: 17.8 -> 19.0).
            if (args.residual != nullptr && have_f && num_kb <= kPrefetchSteps && i > 0) {
                const __nv_bfloat16* p =
                    args.residual + static_cast<size_t>(t.row0 + group * kRound + my_tok) * args.F + f;
                for (int tok = group * kRound + my_tok; tok < t.n; tok += kEpiGroups * kRound) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
                    p += static_cast<size_t>(kEpiGroups * kRound) * args.F;
                }
            }
            // A warp that gives up leaves alone; only shares, which come before all whole
            // tiles, have barriers among the warps, and there they leave together.
            bool ok = __all_sync(0xffffffffu,
                                 mbar_wait_asleep(&bk.tmem_full[acc], acc_phase, abort_flag,
                                                  args.status, reduction_limit_ns(kb1 - kb0)));
            const bool whole = kb1 - kb0 == num_kb;
            if (i < plan.pieces) ok = bar_all(ok, kVoteBarrier, kEpiThreads);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                   static_cast<uint32_t>(acc * kTokens);
            // the eight sums of token `tok` -> checkpoint, activation, residual, output; `at`:
            // where that token's row has feature f
            const size_t origin = static_cast<size_t>(t.row0) * args.F + f;
            auto residual = [&](int tok, size_t at) {
                return args.residual != nullptr && have_f && tok < t.n
                           ? *reinterpret_cast<const uint4*>(args.residual + at)
                           : make_uint4(0u, 0u, 0u, 0u);
            };
            auto finish = [&](int tok, size_t at, float (&v)[8], uint4 res) {
                const bool valid = have_f && tok < t.n;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += bias[k];
                if (args.codes != nullptr) {
                    const float s = ckpt_scale(ckpt_amax_block(have_f ? ckpt_amax8(v) : 0.f));
                    if (valid) {
                        // a ReLU's slope at zero is zero: the backward tells z > 0 by the code
                        *reinterpret_cast<uint2*>(args.codes + at) =
                            args.act == MOE_ACT_RELU ? ckpt_pack8_sums<true>(v, s)
                                                     : ckpt_pack8_sums<false>(v, s);
                        if ((lane & 3) == 0)
                            args.scales[static_cast<size_t>(t.row0 + tok) * nb + f / kCkptBlock] =
                                s;
                    }
                }
                if (!valid) return;
                act_value8(args.act, v);
                if (args.residual != nullptr) {
                    v[0] += bf16_lo(res.x), v[1] += bf16_hi(res.x);
                    v[2] += bf16_lo(res.y), v[3] += bf16_hi(res.y);
                    v[4] += bf16_lo(res.z), v[5] += bf16_hi(res.z);
                    v[6] += bf16_lo(res.w), v[7] += bf16_hi(res.w);
                }
                if (args.out_f32)
                    store8_global(static_cast<float*>(args.out) + at, v);
                else
                    store8(static_cast<__nv_bfloat16*>(args.out) + at, v);
            };
            const size_t F = static_cast<size_t>(args.F);

            if (whole) {
                // round by round of 8 tokens; the next one's accumulator columns and residual
                // are on their way while this one is finished (the residual's latency alone took
                // longer than the rest: 9472 x 512 -> 8192, 154 us with it and 75 without)
                const size_t step = kEpiGroups * kRound * F;
                size_t at = origin + (group * kRound + my_tok) * F;
                uint32_t r[kRound];
                int c0 = group * kRound;
                uint4 next = residual(c0 + my_tok, at);
                if (c0 < t.nt)
                    tmem_ld_8cols(tbase + c0, r);
                else
                    release(acc);  // no round for this group
                for (; c0 < t.nt; c0 += kEpiGroups * kRound) {
                    tmem_ld_wait();
                    const int c1 = c0 + kEpiGroups * kRound;
                    if (c1 >= t.nt) release(acc);
                    __syncwarp();  // the last round's values have been read
#pragma unroll
                    for (int k = 0; k < kRound; ++k) my_staging[k * kPitch + lane] = bits_f32(r[k]);
                    if (c1 < t.nt) tmem_ld_8cols(tbase + c1, r);
                    const uint4 res = next;
                    next = residual(c1 + my_tok, at + step);
                    __syncwarp();
                    float v[8];
                    load8(get, v);
                    finish(c0 + my_tok, at, v, res);
                    at += step;
                }
            } else if constexpr (!PAIR) {
                // a share: the fp32 tile to the workspace as [token][feature]
                const int rem_tile = tile - plan.rounds * plan.G;
                float* slot = args.partials +
                              static_cast<size_t>(plan.c * 2 + i) * slot_floats;
                if (group * kRound >= t.nt) release(acc);
                for (int c0 = group * kRound; c0 < t.nt; c0 += kEpiGroups * kRound) {
                    uint32_t r[kRound];
                    tmem_ld_8cols(tbase + c0, r);
                    tmem_ld_wait();
                    if (c0 + kEpiGroups * kRound >= t.nt) release(acc);
#pragma unroll
                    for (int k = 0; k < kRound; ++k)
                        __stcg(slot + (c0 + k) * kF + q * 32 + lane, bits_f32(r[k]));
                }
                const int u = rem_tile * num_kb;
                const int first = plan.holder(u), last = plan.holder(u + num_kb - 1);
                uint32_t* counter = args.counters + rem_tile;
                __threadfence();
                sync_epilogue();
                if (threadIdx.x == 64) {
                    const uint32_t before = atomicAdd(counter, 1u);
                    bk.last = before == static_cast<uint32_t>(last - first);
                    if (bk.last) *counter = 0;  // zero again for the next call
                }
                sync_epilogue();
                if (bk.last) {
                    __threadfence();
                    // a share that began in an earlier tile has this one as its second
                    const size_t stride = 2 * slot_floats;
                    const float* shares =
                        args.partials + static_cast<size_t>(first) * stride + my_f;
                    const size_t second = plan.bound(first) < u ? slot_floats : 0;
                    for (int tok = group * kRound + my_tok; tok < t.nt;
                         tok += kEpiGroups * kRound) {
                        float v[8] = {};
                        const float* src = shares + tok * kF;
#pragma unroll 4
                        for (int s = 0; s <= last - first; ++s) {
                            const float4* p = reinterpret_cast<const float4*>(
                                src + s * stride + (s == 0 ? second : 0));
                            const float4 lo = __ldcg(p), hi = __ldcg(p + 1);
                            v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w;
                            v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
                        }
                        finish(tok, origin + tok * F, v, residual(tok, origin + tok * F));
                    }
                }
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // the leader's MMAs into this CTA's TMEM are done
    if (warp == 1) {
        tc_fence_after();
        if (PAIR)
            tmem_dealloc_pair(tmem_base, kTmemCols);
        else
            tmem_dealloc(tmem_base, kTmemCols);
    }
}

constexpr int kMinWidth = 32;      // narrowest tile limit
constexpr int kPairsAtFloor = 64;  // rows of a group

int usable_sms() {
    const int sms = device_sm_count();
    return sms < kLinearMaxCtas ? sms : kLinearMaxCtas;
}

// Most tiles of `width` tokens x `features` features there can be.
long long most_tiles(const LinearArgs& a, int F, int width, int features) {
    const long long groups = a.rows < a.E ? a.rows : a.E;
    return (a.rows / width + groups) * ((F + features - 1) / features);
}

template <bool PAIR, bool TRANSPOSED>
cudaError_t launch_engine(const LinearArgs& a, int F, int C, int width, RowClocks row) {
    constexpr int kCtas = PAIR ? 2 : 1;
    auto kern = linear_sm100_kernel<PAIR, TRANSPOSED>;
    static PerDeviceOnce once;
    if (const cudaError_t err = opt_in_smem(once, kern, kSmemBytes); err != cudaSuccess) return err;
    Args g{};
    g.offsets = a.offsets;
    g.E = a.E;
    g.rows = a.rows;
    g.F = F;
    g.C = C;
    g.width = width;
    // Token tiles of a run: 32 MB of rows, eight at least, so that the tiles in flight cover
    // about as many features as tokens and few of either (8192 x 4096 x 14336, one group,
    // 32 tiles a run: 1263 TFLOP/s, 16: 1372).
    const long long run = (32LL << 20) / (static_cast<long long>(kTokens) * C * 2);
    g.group = static_cast<int>(run < 8 ? 8 : (run > 1024 ? 1024 : run));
    g.act = a.act;
    g.bias = static_cast<const __nv_bfloat16*>(a.bias);
    g.residual = static_cast<const __nv_bfloat16*>(a.residual);
    g.out = a.y;
    g.out_f32 = a.y_dt == MOE_F32;
    g.codes = a.codes;
    g.scales = a.scales;
    g.counters = a.counters;
    g.partials = a.partials;
    g.slot_tokens = linear_slot_tokens(a.rows);
    g.row = row;
    g.status = a.status;
    CUtensorMap w;
    TokenMaps x;
    if (!(TRANSPOSED ? encode_bf16_3d(&w, a.W, a.E, C, F, 64) : encode_bf16_3d(&w, a.W, a.E, F, C, kF)))
        return cudaErrorInvalidValue;
    for (int b = 0; b < kBoxes && (b == 0 || 16 * b < a.rows); ++b)  // the sizes tiles can have
        if (!encode_bf16_2d(&x.box[b], a.x, a.rows, C, 16 * (b + 1))) return cudaErrorInvalidValue;
    // A reduction long enough to be shared can use every SM.
    const long long shares = (C + kBK - 1) / kBK / kMinShare;
    const long long want = most_tiles(a, F, width, kF * kCtas) * (shares < 1 ? 1 : shares);
    const int most = usable_sms() / kCtas;
    const int units = static_cast<int>(want < most ? want : most);
    if (!PAIR) return launch_k(kern, units, kThreads, kSmemBytes, a.stream, w, x, g);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, w, x, g);
    return err != cudaSuccess ? err : cudaGetLastError();
}

struct Layout {
    bool pair;
    int width;  // token columns of a tile, at most
};

// The layout with the least clocks for groups of the average size; the weights' bytes from
// HBM (23 a clock and SM) are a floor for all, and of layouts at the floor the first wins: wide
// tiles on single SMs, or on pairs from 64 rows a group on (uniform groups take the same time
// there, a group that is larger than the average less: 8 skewed groups, 600 rows, 7168 -> 2048
// 48 us on pairs and 54 on single SMs).  Measured (us; pairs, then single SMs with tiles of up to 256, 128,
// 64 and 32 tokens):
//   8 groups, 256 rows, K 4096, N 14336       144  137  138  138  153
//   8 groups, 2048 rows, K 4096, N 14336      204  233  243  296  432
//   1 group, 256 rows, K 4096, N 14336         31   34   40   42   61
//   2 groups, 3968 rows, K 11512, N 136        78   48   50   58   84
//   1 group, 1496 rows, K 5144, N 192          40   31   23   18   25
//   1 group, 100 rows, K 8192, N 1024          27   17   17   15   13
//   1 group, 512 rows, K 4096, N 4096          28   27   19   25   37
//   1 group, 8192 rows, K 512, N 7168          60   66   75   99  181
Layout choose_layout(const LinearArgs& a, int F, int C, RowClocks row) {
    const int sms = usable_sms();
    const int groups = a.rows < a.E ? a.rows : a.E;
    const int n = (a.rows + groups - 1) / groups;
    const int num_kb = (C + kBK - 1) / kBK;
    const float floor = 2.f * groups * F * C / (23.f * sms);
    auto tiles = [&](int width, int features, int step, int& wide) {
        const int tt = (n + width - 1) / width;
        wide = ((n + tt - 1) / tt + step - 1) / step * step;
        return static_cast<long long>(groups) * tt * ((F + features - 1) / features);
    };
    Layout best{false, kTokens};
    float least = 0.f;
    auto offer = [&](bool pair, int width, float clocks) {
        if (clocks < floor) clocks = floor;
        if (least == 0.f || clocks < least) best = {pair, width}, least = clocks;
    };
    // `rounds` whole tiles after one another, the epilogues beside the next one's products,
    // the last one's behind them
    auto whole = [&](long long rounds, int wide, bool pair) {
        const float products = num_kb * stage_clocks(wide, pair, row);
        const float epilogue = epilogue_clocks(a, wide, pair);
        return rounds == 0 ? 0.f
                           : static_cast<float>(rounds) * fmaxf(products, epilogue) + epilogue;
    };
    auto offer_pairs = [&]() {
        if (!pair_gemm_enabled()) return;
        int wide;
        const long long all = tiles(kTokens, 2 * kF, 32, wide), pairs = sms / 2;
        offer(true, kTokens, whole((all + pairs - 1) / pairs, wide, true) + kPairClocks);
    };
    if (n >= kPairsAtFloor) offer_pairs();
    for (int width = kTokens; width >= kMinWidth; width /= 2) {
        int wide;
        const long long all = tiles(width, kF, 16, wide);
        const int rem = static_cast<int>(all % sms);
        const Sharing shared(rem, num_kb, wide, sms, row);
        offer(false, width,
              shared.ctas > 0 ? whole(all / sms, wide, false) + shared.clocks
                              : whole((all + sms - 1) / sms, wide, false));
    }
    if (n < kPairsAtFloor) offer_pairs();
    return best;
}

}  // namespace

cudaError_t launch_linear_bf16(const LinearArgs& a, bool transposed) {
    const int F = a.N, C = a.K;
    const RowClocks row = {row_clocks(transposed ? F : C), row_clocks(C)};
    const Layout l = choose_layout(a, F, C, row);
    if (l.pair) {
        const cudaError_t err = transposed ? launch_engine<true, true>(a, F, C, l.width, row)
                                           : launch_engine<true, false>(a, F, C, l.width, row);
        if (err == cudaSuccess || err == cudaErrorInvalidValue) return err;
        cudaGetLastError();  // no room for a pair of CTAs: single SMs
    }
    return transposed ? launch_engine<false, true>(a, F, C, l.width, row)
                      : launch_engine<false, false>(a, F, C, l.width, row);
}

}  // namespace moe
