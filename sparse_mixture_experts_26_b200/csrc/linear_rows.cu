// linear_rows.cu -- the element-wise part of the grouped linear backward:
//   dz = dy act'(z)   with z the value of its 8-bit code; bf16, one rounding
//   db_e = sum of dz over the group's rows, from the unrounded fp32 values
// and, for the weight gradient's reduction over rows in blocks of 64, each group's last
// partial block of dz and of x copied to a buffer where zero rows follow up to the next
// multiple of 16.  The rows behind a group belong to the next one, or to nobody and may
// hold anything; this way they are never read as part of a sum.
//
// Bytes: dy 2, code 1.125, dz 2 per value; 25 instructions a value (GELU) weigh as much.  A
// block takes 256 columns of a chunk of 64 to 512 rows of one group: a warp reads 512 bytes of
// a row, eight columns a lane, and the eight warps take the rows in turn, two to four in
// flight a thread.  The warps' column sums are added in order in shared memory; the chunks' go
// to the workspace, and the block that brings a group's last chunk adds them in chunk order
// (whichever block that is, so db does not depend on the timing).  Without an activation dz
// is dy itself: only the tails and db are made.
// Measured at 8192 x 14336 with db (us; 600 MB): ReLU 115, SiLU 124, GELU 136 (with chunks of 64
// rows 131, 142 and 160, of earlier forms of the slopes).  Small calls: one warp finds all groups'
// chunks with a scan (a walk over the groups by every thread took 250 clocks a group: 32 groups,
// 150 x 144, 5.9 -> 2.4 us).
#include <cuda_bf16.h>

#include "linear_device.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 256;  // columns per block
constexpr int kBlocksPerSm = 4;

struct DzArgs {
    const __nv_bfloat16* dy;
    const __nv_bfloat16* x;
    const int32_t* offsets;
    const int8_t* codes;   // nullptr: dz = dy
    const float* scales;
    int rows, K, N, E, act;
    __nv_bfloat16* dz;
    __nv_bfloat16* dz_tail;  // nullptr: no tails wanted
    __nv_bfloat16* x_tail;
    float* db;             // nullptr: not wanted
    float* part;           // the chunk sums of groups with several
    uint32_t* counters;    // one for each group and strip, zero between calls
    int dz_items;          // chunks times column strips of dz
    int items;             // .. and groups times column strips of x (for the tails)
    int chunk_rows;        // a multiple of kTailRows
    int n_strips, x_strips;
};

struct Groups {
    int off[kMaxExperts + 1];
    int chunk[kMaxExperts + 1];  // groups' first chunks; an empty group has one too
};
// One warp fills them.
__device__ __forceinline__ void load_groups(const DzArgs& a, Groups& g) {
    const int lane = threadIdx.x & 31;
    load_group_bounds(a.offsets, a.E, a.rows, g.off);
    int rest, sum = 0;
    if (lane < a.E)
        sum = max(divide(g.off[lane + 1] - g.off[lane] + a.chunk_rows - 1, a.chunk_rows, rest), 1);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += below;
    }
    if (lane < a.E) g.chunk[lane + 1] = sum;
    if (lane == 0) g.chunk[0] = 0;
}

// The rows of group e from its last whole block of 64 on, and how many rows of the tail buffers
// they and the zeros behind them take.
struct Tail {
    int whole, rows;
    __device__ __forceinline__ explicit Tail(int of_group) {
        whole = of_group / kTailRows * kTailRows;
        rows = (of_group - whole + 15) / 16 * 16;
    }
};

// One strip of columns of the tail of group e's x.
__device__ __forceinline__ void x_item(const DzArgs& a, const Groups& groups, int e, int strip) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = strip * kCols + lane * 8;
    const int row0 = groups.off[e], of_group = groups.off[e + 1] - row0;
    const Tail t(of_group);
    if (c >= a.K) return;
#pragma unroll 4
    for (int r = warp; r < t.rows; r += kWarps) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (t.whole + r < of_group)
            v = *reinterpret_cast<const uint4*>(
                a.x + static_cast<size_t>(row0 + t.whole + r) * a.K + c);
        *reinterpret_cast<uint4*>(a.x_tail + (static_cast<size_t>(e) * kTailRows + r) * a.K + c) = v;
    }
}

// One chunk's strip of columns.  All threads of the block call this together.
template <int FLIGHT>
__device__ __forceinline__ void dz_item(const DzArgs& a, const Groups& groups,
                                        float (*s_sum)[kCols], int& s_last, int item) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int* off = groups.off;
    int strip;
    const int chunk = divide(item, a.n_strips, strip);
    const int e = __popc(__ballot_sync(0xffffffffu, lane < a.E && groups.chunk[lane + 1] <= chunk));
    if (e == a.E) return;
    const int i = chunk - groups.chunk[e];  // chunk i of the group's
    const int chunks = groups.chunk[e + 1] - groups.chunk[e];
    const int of_group = off[e + 1] - off[e];
    const int first = i * a.chunk_rows;             // this chunk's rows, counted in the group
    const int end = min(first + a.chunk_rows, of_group);
    const int row0 = off[e];
    // the group's last, partial block of 64 rows, if it is in this chunk
    const Tail t(of_group);
    const bool tail = a.dz_tail != nullptr && end == of_group && t.rows > 0;
    const int whole = t.whole, end16 = whole + t.rows;  // zero rows up to here
    const size_t trow = static_cast<size_t>(e) * kTailRows;
    const float zero[8] = {};

    const int c = strip * kCols + lane * 8;
    const bool have = c < a.N && (a.codes || a.db || tail);  // else nothing to do here
    const int nb = ckpt_blocks(a.N);
    float sum[8] = {};
    if (have) {
        for (int r0 = first + warp; r0 < end; r0 += FLIGHT * kWarps) {
            uint4 dy[FLIGHT];  // rows whose loads are in flight together
            uint2 q[FLIGHT];
            float s[FLIGHT];
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const int r = r0 + k * kWarps;
                if (r >= end) continue;
                const size_t row = static_cast<size_t>(row0 + r), at = row * a.N + c;
                dy[k] = *reinterpret_cast<const uint4*>(a.dy + at);
                if (a.codes) {
                    q[k] = *reinterpret_cast<const uint2*>(a.codes + at);
                    s[k] = a.scales[row * nb + c / kCkptBlock];
                }
            }
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const int r = r0 + k * kWarps;
                if (r >= end) continue;
                float g[8] = {bf16_lo(dy[k].x), bf16_hi(dy[k].x), bf16_lo(dy[k].y),
                              bf16_hi(dy[k].y), bf16_lo(dy[k].z), bf16_hi(dy[k].z),
                              bf16_lo(dy[k].w), bf16_hi(dy[k].w)};
                if (a.codes) {
                    float z[8];
                    ckpt_unpack8(q[k], s[k], z);
                    act_slope8(a.act, z, g);
                    store8(a.dz + static_cast<size_t>(row0 + r) * a.N + c, g);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) sum[u] += g[u];
                if (tail && r >= whole) store8(a.dz_tail + (trow + r - whole) * a.N + c, g);
            }
        }
        if (tail)
            for (int r = end + warp; r < end16; r += kWarps)
                store8(a.dz_tail + (trow + r - whole) * a.N + c, zero);
    }
    if (a.db == nullptr) return;
    const int col = strip * kCols + threadIdx.x;
    // the warps' sums of this thread's column, in order
    auto join = [&]() {
        __syncthreads();  // what was there before has been read
        store8(&s_sum[warp][lane * 8], sum);
        __syncthreads();
        float total = s_sum[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) total += s_sum[w][threadIdx.x];
        return total;
    };
    float total = join();
    float* db = a.db + static_cast<size_t>(e) * a.N + col;
    if (chunks == 1) {
        if (col < a.N) *db = total;
        return;
    }
    if (col < a.N) __stcg(a.part + static_cast<size_t>(chunk) * a.N + col, total);
    __syncthreads();
    if (threadIdx.x == 0) {
        // the barriers carry the block's stores to this fence, and what it sees to the block
        __threadfence();
        uint32_t* counter = a.counters + static_cast<size_t>(e) * a.n_strips + strip;
        s_last = atomicAdd(counter, 1u) == static_cast<uint32_t>(chunks - 1);
        if (s_last) *counter = 0;  // zero again for the next call
        __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    // warp w adds chunks w, w + 8, .. of the group, then the warps' sums are added
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = 0.f;
    if (c < a.N) {
        const float* part = a.part + static_cast<size_t>(chunk - i) * a.N + c;
#pragma unroll 4
        for (int k = warp; k < chunks; k += kWarps) {
            const float4* p = reinterpret_cast<const float4*>(part + static_cast<size_t>(k) * a.N);
            const float4 lo = __ldcg(p), hi = __ldcg(p + 1);
            sum[0] += lo.x, sum[1] += lo.y, sum[2] += lo.z, sum[3] += lo.w;
            sum[4] += hi.x, sum[5] += hi.y, sum[6] += hi.z, sum[7] += hi.w;
        }
    }
    total = join();
    if (col < a.N) *db = total;
}

template <int FLIGHT, int BLOCKS_PER_SM>
__global__ void __launch_bounds__(kThreads, BLOCKS_PER_SM) linear_dz_kernel(const DzArgs a) {
    __shared__ Groups groups;
    __shared__ int s_last;
    __shared__ __align__(16) float s_sum[kWarps][kCols];  // written 16 bytes at a time
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x < 32) load_groups(a, groups);
    __syncthreads();
    int item = blockIdx.x;
    for (; item < a.dz_items; item += gridDim.x) dz_item<FLIGHT>(a, groups, s_sum, s_last, item);
    for (; item < a.items; item += gridDim.x) {
        int strip;
        const int e = divide(item - a.dz_items, a.x_strips, strip);
        x_item(a, groups, e, strip);
    }
}

}  // namespace

cudaError_t launch_linear_dz(const LinearBwdArgs& a) {
    if (a.codes == nullptr && a.dW == nullptr && a.db == nullptr) return cudaSuccess;
    DzArgs d{};
    d.dy = static_cast<const __nv_bfloat16*>(a.dy);
    d.x = static_cast<const __nv_bfloat16*>(a.x);
    d.offsets = a.offsets;
    d.codes = a.codes;
    d.scales = a.scales;
    d.rows = a.rows;
    d.K = a.K;
    d.N = a.N;
    d.E = a.E;
    d.act = a.act;
    d.dz = static_cast<__nv_bfloat16*>(a.dz);
    d.dz_tail = a.dW ? static_cast<__nv_bfloat16*>(a.dz_tail) : nullptr;
    d.x_tail = static_cast<__nv_bfloat16*>(a.x_tail);
    d.db = a.db;
    d.part = a.db_part;
    d.counters = a.db_counters;
    d.n_strips = (a.N + kCols - 1) / kCols;
    d.x_strips = a.dW ? (a.K + kCols - 1) / kCols : 0;
    // Blocks stay for several items, because reading the group bounds takes a block as long
    // as one; and chunks grow while there are several items for every block.  Where the
    // counters are too few, a group is one chunk: its strips (more than 256) are work enough.
    const int blocks = device_sm_count() * kBlocksPerSm;
    long long chunks;
    if (static_cast<long long>(a.E) * d.n_strips > kLinearDbCounters) {
        d.chunk_rows = (a.rows + kTailRows - 1) / kTailRows * kTailRows;
        chunks = a.E;
    } else {
        for (d.chunk_rows = kTailRows;; d.chunk_rows *= 2) {
            chunks = a.rows / d.chunk_rows + a.E;  // at most linear_chunks
            if (d.chunk_rows >= 512 || chunks * d.n_strips < 6LL * blocks) break;
        }
    }
    d.dz_items = static_cast<int>(chunks * d.n_strips);  // rows * N < 2^40: below 2^31
    d.items = d.dz_items + a.E * d.x_strips;
    // Few items are chains of latencies: more rows in flight where two or three blocks an SM hold
    // them all (counting half a chunk for a group's last, partial one).  Us with 2 rows and four
    // blocks, 3 and three, 4 and two: 1958 x 1168, 16 groups (GELU) 9.1, 8.9, 8.6; 600 x 7168, 8
    // groups (SiLU) 12.0, 10.0, 11.7; 2048 x 4096 (SiLU) 12.5, 14.3, 14.7.
    const int sms = device_sm_count();
    if (d.items <= 2 * sms)
        return launch_k(linear_dz_kernel<4, 2>, d.items, kThreads, 0, a.stream, d);
    const long long full = (chunks - a.E + (a.E + 1) / 2) * d.n_strips + a.E * d.x_strips / 2;
    if (full <= 3LL * sms)
        return launch_k(linear_dz_kernel<3, 3>, d.items < 3 * sms ? d.items : 3 * sms, kThreads, 0,
                        a.stream, d);
    return launch_k(linear_dz_kernel<2, kBlocksPerSm>, d.items < blocks ? d.items : blocks, kThreads, 0, a.stream, d);
}

}  // namespace moe
