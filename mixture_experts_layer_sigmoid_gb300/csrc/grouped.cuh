// grouped.cuh -- segments of rows sorted by expert, as the products over them see
// them (grouped_simt.cu, grouped_tc.cuh, matmul_fp8.cu): the rows of each expert and
// the list of row tiles, read on the device, so that no call waits for the routing.
#pragma once
#include "internal.h"

namespace moe {

constexpr int kMaxGroups = 1024;       // experts, as the sort's index has them
// Rows: any of them plus a unit of tiles (256 rows and a quarter's 96 more) or a ring of blocks of
// the contraction (8 x 32) is a row number in 32 bits, here and in a TMA coordinate.
constexpr long long kMaxRows = (1ll << 31) - 1024;

// The segments of one call. offsets null: one segment of all rows.
struct Groups {
    int E;
    int rows;                          // rows of the row buffers
    const int* offsets;                // E + 1
    const int* counts;                 // E, or null: every row of a segment counts
};

struct Segment {
    int begin, end;                    // rows of the segment, padding included
    int valid;                         // rows from `begin` on that belong to the expert
};

// Whatever the index holds, a segment lies inside the row buffers.
__device__ __forceinline__ Segment segment_of(const Groups& g, int e)
{
    if (!g.offsets) return Segment{0, g.rows, g.rows};
    Segment s;
    s.begin = min(max(g.offsets[e], 0), g.rows);
    s.end = min(max(g.offsets[e + 1], s.begin), g.rows);
    s.valid = g.counts ? min(max(g.counts[e], 0), s.end - s.begin) : s.end - s.begin;
    return s;
}

// The segments in shared memory (a tile's place is looked up by every role of a block, and a
// look at the index in L2 costs more than a short tile's products).
struct SegmentTable {
    int pre[kMaxGroups + 4];           // row tiles before each segment
    int begin[kMaxGroups], end[kMaxGroups], valid[kMaxGroups];
    __device__ __forceinline__ Segment at(int e) const { return Segment{begin[e], end[e], valid[e]}; }
};

// Fills the table: pre[e] = row tiles of TM rows in the segments before e; pre[E] = all of
// them. Called by every thread of the block.
template <int TM>
__device__ __forceinline__ void read_segments(const Groups& g, SegmentTable* table)
{
    int* pre = table->pre;
    for (int e = threadIdx.x; e < g.E; e += blockDim.x) {
        const Segment s = segment_of(g, e);
        table->begin[e] = s.begin;
        table->end[e] = s.end;
        table->valid[e] = s.valid;
        pre[e + 1] = (s.end - s.begin + TM - 1) / TM;
    }
    if (threadIdx.x == 0) pre[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        int carry = 0;
        for (int base = 0; base < g.E; base += 32) {
            const int e = base + (int)threadIdx.x;
            int v = e < g.E ? pre[e + 1] : 0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, off);
                if ((int)threadIdx.x >= off) v += u;
            }
            // (segments of a valid index are no more tiles than an int counts; others may overlap)
            const int most = 0x7fffffff - carry;
            if (e < g.E) pre[e + 1] = carry + min(v, most);
            carry += min(__shfl_sync(0xffffffffu, v, 31), most);
        }
    }
    __syncthreads();
}

// The segment that row tile q belongs to: the last e with pre[e] <= q < pre[E].
__device__ __forceinline__ int segment_at(const int* pre, int E, int q)
{
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= q) lo = mid;
        else hi = mid;
    }
    return lo;
}

// An upper bound of the row tiles of any index over `rows` rows.
inline long long row_tiles_bound(long long rows, int E, int TM)
{
    return rows / TM + (rows < E ? rows : E);
}

// Operands of a grouped product, in elements. Rows: Y[r][n] = sum_k X[r][k] W[e][k][n]
// with W at e sw + k ldw + n, or e sw + n ldw + k (w_nk). Weight gradient: dW[e][m][n] =
// sum_r A[r][m] B[r][n] with dW at e sw + m ldw + n.
struct GroupedRows {
    Groups g;
    int K, N;
    const void* X; long long ldx;
    const void* W; long long ldw, sw; int w_nk;
    void* Y; long long ldy;
};
struct GroupedWgrad {
    Groups g;
    int M, N;
    const void* A; long long lda;
    const void* B; long long ldb;
    void* D; long long ldd, sd;
};

// moe_fp8_matmul's operands.
struct Fp8Rows {
    Groups g;
    int K, N, dtype;
    moe_fp8_matmul_args_t a;
};

// fp32
cudaError_t launch_grouped_rows_simt(const GroupedRows& p, int num_sms, cudaStream_t s);
cudaError_t launch_grouped_wgrad_simt(const GroupedWgrad& p, int num_sms, cudaStream_t s);
// bf16
cudaError_t launch_grouped_rows_tc(const GroupedRows& p, int num_sms, cudaStream_t s);
cudaError_t launch_grouped_wgrad_tc(const GroupedWgrad& p, int num_sms, cudaStream_t s);
cudaError_t launch_fp8_rows(const Fp8Rows& p, int num_sms, cudaStream_t s);

}  // namespace moe
