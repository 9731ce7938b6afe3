// grouped_linear_wgrad_sm100.cu -- the grouped linear operators' weight gradient on the
// tensor cores:
//   dW[e, n, k] = sum over the rows r of group e of dz[r, n] x[r, k]
// Both operands are rows as they lie in memory (n and k contiguous), read as MN-major
// 64 x 64 boxes; nothing is transposed.  A tile is 128 features n (256 on a pair of SMs,
// 128 from each) x up to 256 inputs k, the reduction runs over the group's rows in blocks of 64.
//
// A group starts and ends anywhere.  Its whole blocks come straight from dz and x; the rest
// comes from the tail buffers (linear_rows.cu), where the group's last rows are followed
// by zeros up to a multiple of 16, and only that many 16-row steps are issued.  So no row
// outside the group is ever multiplied, not even by zero, and groups of up to 16 rows (decode
// batches) load a quarter of a stage.
//
// Bound: many rows, the tensor cores (pairs of SMs halve the bytes staged per product);
// few rows, the gradient's own bytes (E N K elements written once).  The epilogue's warps
// turn 32 rows x 128 bytes at a time in shared memory and store whole 128-byte lines with
// the evict-first policy (nobody reads them here again).
//
// Roles, accumulators and bounded waits as in grouped_linear_sm100.cu.
#include <cuda.h>
#include <cuda_bf16.h>

#include "linear_device.cuh"
#include "moe_internal.h"
#include "sm100_ptx.cuh"

namespace moe {

// Defined in grouped_gemm_sm100.cu.
bool encode_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                    uint32_t box_rows);

namespace {

constexpr int kM = 128;              // features per CTA (TMEM lanes)
constexpr int kN = 256;              // inputs per tile, at most
constexpr int kMaxStages = 8;
constexpr int kBlock = kTailRows;    // rows of a whole block; a stage holds one or two
constexpr int kChunk = 32 * 128;     // staged output: 32 rows x 128 bytes
constexpr uint16_t kBothCtas = 0x3;

struct Args {
    const int32_t* offsets;
    int E, rows;
    int M;         // features (dz columns)
    int N;         // inputs (x columns)
    int width;     // inputs of a tile: 64, 128 or 256
    int m_tiles, n_tiles;
    void* out;     // [E, M, N]
    uint32_t* status;
};

struct Book {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int off[kMaxExperts + 1];
};

// GROUPS: epilogue groups of four warps, one for each quarter of the lanes; the groups take
// the output's 128-byte columns in turn.
// ROWS: the reduction per stage (64 or 128): with 128, half as many loads of twice the size.
// STAGES: of tiles with 256 inputs; narrower ones have more of them.
template <bool PAIR, int ROWS, int STAGES, int GROUPS>
struct Shape {
    static constexpr int kBox = 128 * ROWS;  // 64 columns of a stage's rows
    static constexpr int kEpiWarps = 4 * GROUPS;
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kABytes = 2 * kBox;
    static constexpr int kBBoxes = PAIR ? 2 : 4;  // a pair's CTAs hold half of x's columns
    static constexpr int kStageBytes = kABytes + kBBoxes * kBox;
    static constexpr int kStaging = kEpiWarps * kChunk;
    static constexpr int kSmem = STAGES * kStageBytes + kStaging + 1024 /*book*/ + 1024 /*align*/;
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(sizeof(Book) <= 1024, "bookkeeping reserve");
};

template <bool PAIR, bool F32, int ROWS, int STAGES, int GROUPS>
__global__ void __launch_bounds__(Shape<PAIR, ROWS, STAGES, GROUPS>::kThreads, 1)
    linear_wgrad_kernel(const __grid_constant__ CUtensorMap tmZ,
                        const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmZ1,
                        const __grid_constant__ CUtensorMap tmX1,
                        const __grid_constant__ CUtensorMap tmZt,
                        const __grid_constant__ CUtensorMap tmXt,
                        const __grid_constant__ CUtensorMap tmZs,
                        const __grid_constant__ CUtensorMap tmXs, const Args args) {
    using S = Shape<PAIR, ROWS, STAGES, GROUPS>;
    constexpr int kCtas = PAIR ? 2 : 1;
    constexpr uint32_t kTmemCols = 2 * kN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* staging = smem + STAGES * S::kStageBytes;
    Book& bk = *reinterpret_cast<Book*>(staging + S::kStaging);
    const int boxes = args.width / (64 * kCtas);  // of x, in a stage of this CTA
    const int stage_bytes = S::kABytes + boxes * S::kBox;
    const int stages = min(STAGES * S::kStageBytes / stage_bytes, kMaxStages);
    volatile int* abort_flag = &bk.abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&bk.full[s], 1);
            mbar_init(&bk.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&bk.tmem_full[a], 1);
            mbar_init(&bk.tmem_empty[a], kCtas * S::kEpiWarps);
        }
        mbar_init(&bk.drain, 1);
        bk.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmZ);
        tma_prefetch_desc(&tmX);
        if (ROWS > kBlock) {
            tma_prefetch_desc(&tmZ1);
            tma_prefetch_desc(&tmX1);
        }
        tma_prefetch_desc(&tmZt);
        tma_prefetch_desc(&tmXt);
        tma_prefetch_desc(&tmZs);
        tma_prefetch_desc(&tmXs);
    }
    if (warp == 1) {
        if (PAIR)
            tmem_alloc_pair(&bk.tmem_base, kTmemCols);
        else
            tmem_alloc(&bk.tmem_base, kTmemCols);
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) load_group_bounds(args.offsets, args.E, args.rows, bk.off);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = bk.tmem_base;
    const int per_e = args.m_tiles * args.n_tiles;
    const int total = args.E * per_e;
    const int first = blockIdx.x / kCtas, step = gridDim.x / kCtas;
    // column tiles innermost: CTAs running together write neighbouring parts of the same
    // gradient rows
    auto tile_of = [&](int tile, int& e, int& m0, int& n0, int& row0, int& n) {
        int local, nt;
        e = divide(tile, per_e, local);
        m0 = divide(local, args.n_tiles, nt) * (kM * kCtas);
        n0 = nt * args.width;
        row0 = bk.off[e];
        n = bk.off[e + 1] - row0;
    };
    // inputs of the tile at n0 that are multiplied: whole steps of 16 on each CTA
    auto width_of = [&](int n0) {
        const int left = (args.N - n0 + 16 * kCtas - 1) / (16 * kCtas) * (16 * kCtas);
        return left < args.width ? left : args.width;
    };
    int e, m0, n0, row0, n;

    if (warp == 0) {
        if (elect_one()) {
            int stage = 0;
            uint32_t phase = 0, pending = 0, pending_phase = 0;
            bool ok = true, issued = false;
            for (int tile = first; ok && tile < total; tile += step) {
                tile_of(tile, e, m0, n0, row0, n);
                const int mc = m0 + rank * kM;
                const int half = width_of(n0) / kCtas;
                const int nc = n0 + rank * half, nb = (half + 63) / 64;
                for (int r = 0; r < n; r += ROWS) {
                    if (!mbar_wait_asleep(&bk.empty[stage], phase ^ 1u, abort_flag,
                                           args.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t* z = smem + stage * stage_bytes;
                    uint8_t* x = z + S::kABytes;
                    const int left = n - r < ROWS ? n - r : ROWS;
                    auto load = [&](const CUtensorMap* map, uint8_t* dst, int c, int row) {
                        if (PAIR)
                            tma_load_2d_pair(map, map_to_cta(smem_u32(&bk.full[stage]), 0), dst, c,
                                             row);
                        else
                            tma_load_2d(map, &bk.full[stage], dst, c, row);
                    };
                    // rows row .. of both operands, to the stage's row `at`
                    auto rows = [&](const CUtensorMap* mz, const CUtensorMap* mx, int at, int row) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            load(mz, z + b * S::kBox + at * 128, mc + 64 * b, row);
#pragma unroll
                        for (int b = 0; b < S::kBBoxes; ++b)
                            if (b < nb) load(mx, x + b * S::kBox + at * 128, nc + 64 * b, row);
                    };
                    // a partial block: its first 16 rows if that is all, else 64 at once
                    // (what lies behind the zeros is loaded and not multiplied)
                    const int part = left % kBlock;
                    const int loaded = left - part + (part == 0 ? 0 : part <= 16 ? 16 : kBlock);
                    if (leader)
                        mbar_arrive_expect_tx(
                            &bk.full[stage],
                            static_cast<uint32_t>(kCtas * (2 + nb) * 128 * loaded));
                    if (left == ROWS) {
                        rows(&tmZ, &tmX, 0, row0 + r);
                    } else {
                        if (ROWS > kBlock && left >= kBlock) rows(&tmZ1, &tmX1, 0, row0 + r);
                        if (part > 16)
                            rows(&tmZt, &tmXt, left - part, e * kTailRows);
                        else if (part > 0)
                            rows(&tmZs, &tmXs, left - part, e * kTailRows);
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
                    short_pause_ns(2000000ull);  // its copies complete on the leader's barriers
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader && elect_one()) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, issued = false;
            for (int tile = first; ok && tile < total; tile += step) {
                tile_of(tile, e, m0, n0, row0, n);
                if (n == 0) continue;  // zeros, written by the epilogue alone
                if (!mbar_wait_asleep(&bk.tmem_empty[acc], acc_phase ^ 1u, abort_flag,
                                       args.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kN);
                const uint32_t idesc = idesc_bf16_f32_major(kM * kCtas, width_of(n0), true, true);
                for (int r = 0; r < n; r += ROWS) {
                    if (!mbar_wait_asleep(&bk.full[stage], phase, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t z = smem_u32(smem + stage * stage_bytes);
                    const uint64_t zd = sw128_mn_desc(z, S::kBox);
                    const uint64_t xd = sw128_mn_desc(z + S::kABytes, S::kBox);
                    const int left = n - r;
                    const int steps = left >= ROWS ? ROWS / 16 : (left + 15) / 16;
                    for (int k = 0; k < steps; ++k) {
                        const uint32_t accumulate = (r != 0 || k != 0) ? 1u : 0u;
                        if (PAIR)
                            umma_bf16_pair(d_tmem, zd + kMnDescStep * k, xd + kMnDescStep * k,
                                           idesc, accumulate);
                        else
                            umma_bf16(d_tmem, zd + kMnDescStep * k, xd + kMnDescStep * k, idesc,
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
        const int q = warp & 3, group = (warp - 2) >> 2;
        uint8_t* st = staging + (warp - 2) * kChunk;
        const uint32_t free0 = PAIR ? map_to_cta(smem_u32(&bk.tmem_empty[0]), 0) : 0u;
        const uint32_t free1 = PAIR ? map_to_cta(smem_u32(&bk.tmem_empty[1]), 0) : 0u;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = first; tile < total; tile += step) {
            tile_of(tile, e, m0, n0, row0, n);
            if (n > 0) {
                if (!__all_sync(0xffffffffu,
                                mbar_wait_asleep(&bk.tmem_full[acc], acc_phase, abort_flag,
                                                 args.status, reduction_limit_ns(n / kBlock + 1))))
                    break;  // a warp that gives up leaves alone
                tc_fence_after();
            }
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                   static_cast<uint32_t>(acc * kN);
            const int mrow = m0 + rank * kM + q * 32;
            constexpr int kEl = F32 ? 4 : 2;
            constexpr int kCols = 128 / kEl;  // output columns per chunk
            const size_t row_bytes = static_cast<size_t>(args.N) * kEl;
#pragma unroll 1
            for (int c = group * kCols; c < args.width; c += GROUPS * kCols) {
                uint4 out[8];  // this lane's row of the chunk
                if (n == 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) out[i] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    uint32_t v[32];
                    tmem_ld_32cols(tbase + c, v);
                    if constexpr (F32) {
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            out[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    } else {
                        uint32_t w[32];
                        tmem_ld_32cols(tbase + c + 32, w);
                        tmem_ld_wait();
                        auto pack = [](const uint32_t* p) {
                            return pack_bf16x2(bits_f32(p[0]), bits_f32(p[1]));
                        };
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            out[i] = make_uint4(pack(v + 8 * i), pack(v + 8 * i + 2),
                                                pack(v + 8 * i + 4), pack(v + 8 * i + 6));
                            out[4 + i] = make_uint4(pack(w + 8 * i), pack(w + 8 * i + 2),
                                                    pack(w + 8 * i + 4), pack(w + 8 * i + 6));
                        }
                    }
                }
                if (n0 + c >= args.N || mrow >= args.M) continue;  // uniform in the warp
                __syncwarp();  // the last chunk has been read
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(st + lane * 128 + ((i ^ (lane & 7)) << 4)) = out[i];
                __syncwarp();
                // eight lanes a row: whole 128-byte lines, four rows at a time
                const int part = lane & 7;
                const bool have = n0 + c + part * (16 / kEl) < args.N;
                uint8_t* to = static_cast<uint8_t*>(args.out) +
                              static_cast<size_t>(e) * args.M * row_bytes +
                              static_cast<size_t>(n0 + c) * kEl + part * 16;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = i * 4 + (lane >> 3);
                    const uint4 v =
                        *reinterpret_cast<const uint4*>(st + r * 128 + ((part ^ (r & 7)) << 4));
                    if (have && mrow + r < args.M)
                        __stcs(reinterpret_cast<uint4*>(
                                   to + static_cast<size_t>(mrow + r) * row_bytes),
                               v);
                }
            }
            if (n == 0) continue;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR)
                    mbar_arrive_cluster_light(acc == 0 ? free0 : free1);
                else
                    mbar_arrive(&bk.tmem_empty[acc]);
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR)
            tmem_dealloc_pair(tmem_base, kTmemCols);
        else
            tmem_dealloc(tmem_base, kTmemCols);
    }
}

template <bool PAIR, bool F32, int ROWS, int STAGES, int GROUPS>
cudaError_t launch_wgrad(const LinearBwdArgs& a, int width) {
    constexpr int kCtas = PAIR ? 2 : 1;
    constexpr int kSmem = Shape<PAIR, ROWS, STAGES, GROUPS>::kSmem;
    constexpr int kThreads = Shape<PAIR, ROWS, STAGES, GROUPS>::kThreads;
    auto kern = linear_wgrad_kernel<PAIR, F32, ROWS, STAGES, GROUPS>;
    static PerDeviceOnce once;
    if (const cudaError_t err = opt_in_smem(once, kern, kSmem); err != cudaSuccess) return err;
    const void* dz = a.codes ? a.dz : a.dy;
    const uint64_t tails = static_cast<uint64_t>(a.E) * kTailRows;
    // a stage's rows, one block's; the tails' rows, their first 16
    CUtensorMap z, x, z1, x1, zt, xt, zs, xs;
    if (!encode_bf16_2d(&z, dz, a.rows, a.N, ROWS) || !encode_bf16_2d(&x, a.x, a.rows, a.K, ROWS) ||
        !encode_bf16_2d(&z1, dz, a.rows, a.N, kBlock) ||
        !encode_bf16_2d(&x1, a.x, a.rows, a.K, kBlock) ||
        !encode_bf16_2d(&zt, a.dz_tail, tails, a.N, kBlock) ||
        !encode_bf16_2d(&xt, a.x_tail, tails, a.K, kBlock) ||
        !encode_bf16_2d(&zs, a.dz_tail, tails, a.N, 16) ||
        !encode_bf16_2d(&xs, a.x_tail, tails, a.K, 16))
        return cudaErrorInvalidValue;
    Args g{};
    g.offsets = a.offsets;
    g.E = a.E;
    g.rows = a.rows;
    g.M = a.N;
    g.N = a.K;
    g.m_tiles = (a.N + kM * kCtas - 1) / (kM * kCtas);
    g.width = width;
    g.n_tiles = (a.K + width - 1) / width;
    g.out = a.dW;
    g.status = a.status;
    const long long tiles = static_cast<long long>(a.E) * g.m_tiles * g.n_tiles;
    const int most = device_sm_count() / kCtas;
    const int units = static_cast<int>(tiles < most ? tiles : most);
    if (!PAIR) return launch_k(kern, units, kThreads, kSmem, a.stream, z, x, z1, x1, zt, xt, zs, xs, g);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, z, x, z1, x1, zt, xt, zs, xs, g);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// Average rows per group below which a bf16 gradient is bound by its epilogue.
constexpr int kShortRows = 128;

struct Layout {
    bool pair;
    int width;
};

// The layout with the least clocks (as in grouped_linear_sm100.cu; fitted likewise) for groups of
// the average size, the gradient's bytes to HBM being a floor for all; of layouts at the floor the
// first wins.  Measured, zero data (us; pairs, then single SMs with 256, 128 and 64 inputs):
//   8 groups, 256 rows, K 4096, N 14336, bf16     181  168  257  459   (sixteen epilogue warps)
//   8 groups, 1024 rows, K 4096, N 14336, bf16    194  201  239  371
//   8 groups, 8192 rows, K 4096, N 14336, bf16    554  641  777 1140
//   8 groups, 512 rows, K 4096, N 14336, fp32     338  341  317  404
//   1 group, 2000 rows, K 1024, N 1024, bf16       19   16   13   14
//   2 groups, 5814 rows, K 104, N 2640, bf16       27   29   29   24
//   1 group, 8000 rows, K 256, N 256, bf16         45   42   27   25
Layout choose_layout(const LinearBwdArgs& a, int el) {
    const int sms = device_sm_count();
    const int n = a.rows < a.E ? 1 : a.rows / a.E;
    const float floor = static_cast<float>(a.E) * a.N * a.K * el / (23.f * sms);
    const float row_z = a.N % 64 == 0 ? 1.6f : 4.1f, row_x = a.K % 64 == 0 ? 1.6f : 4.1f;
    Layout best{false, kN};
    float least = 0.f;
    auto offer = [&](bool pair, int width) {
        const int ctas = pair ? 2 : 1;
        const long long tiles = static_cast<long long>(a.E) * ((a.N + kM * ctas - 1) / (kM * ctas)) *
                                ((a.K + width - 1) / width);
        const long long rounds = (tiles + sms / ctas - 1) / (sms / ctas);
        const int wide = a.K < width ? (a.K + 31) / 32 * 32 : width;
        const float boxes = static_cast<float>((wide / ctas + 63) / 64);
        const float load = 64.f * (2.f * row_z + boxes * row_x);
        const float block = fmaxf(fmaxf(2.02f * wide, 260.f + 1.1f * wide), load);
        const float products = static_cast<float>((n + 63) / 64) * block;
        const float epilogue =
            el == 2 ? 1200.f + 7.3f * wide : fmaxf(850.f + 17.1f * wide, 25.f * wide);
        float clocks = static_cast<float>(rounds) * fmaxf(products, epilogue) + epilogue;
        if (pair) clocks += 6500.f;
        if (clocks < floor) clocks = floor;
        if (least == 0.f || clocks < least) best = {pair, width}, least = clocks;
    };
    if (n >= kShortRows && pair_gemm_enabled()) offer(true, kN);
    if (el == 4) offer(false, 128);
    offer(false, kN);
    if (el == 2) offer(false, 128);
    offer(false, 64);
    return best;
}

template <bool F32>
cudaError_t launch_typed(const LinearBwdArgs& a) {
    const Layout l = choose_layout(a, F32 ? 4 : 2);
    if (l.pair) {
        const cudaError_t err = launch_wgrad<true, F32, 128, 3, 2>(a, l.width);
        if (err == cudaSuccess || err == cudaErrorInvalidValue) return err;
        cudaGetLastError();  // no room for a pair of CTAs: single SMs
    }
    // Short reductions in bf16 are bound by the epilogue: sixteen warps of it and three stages
    // (K 4096, N 14336, 8 groups: 256 rows 168 us against 182 with eight warps and four stages,
    // 512 rows 175 and 187, 1024 rows 206 and 198).  fp32 has half the values per byte and twice
    // the bytes, where more writers only scatter them (341 against 316 us).
    if constexpr (!F32)
        if (a.rows / a.E < kShortRows) return launch_wgrad<false, F32, 64, 3, 4>(a, l.width);
    return launch_wgrad<false, F32, 64, 4, 2>(a, l.width);
}

}  // namespace

cudaError_t launch_linear_wgrad(const LinearBwdArgs& a) {
    return a.dw_dt == MOE_F32 ? launch_typed<true>(a) : launch_typed<false>(a);
}

}  // namespace moe
