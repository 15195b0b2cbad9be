// grouped_simt.cu -- products grouped by expert on the CUDA cores: the fp32 type
// (fp32 FMA arithmetic throughout, as the fp32 layer has it; the tensor cores have no
// mode of full fp32 precision).
//
//   rows            Y[r][n] = sum_k X[r][k] W[e(r)][k][n]
//   weight gradient D[e][m][n] = sum over the expert's rows r of A[r][m] B[r][n]
//
// A block of 256 threads owns a TM x TN tile of outputs, a thread (TM/16) x (TN/16) of
// them as pairs of columns (fma.rn.f32x2). Chunks of 16 along the contraction go through
// shared memory, the next chunk's loads in flight in registers meanwhile. Each output is
// one thread's sum in ascending order. Blocks are persistent and read the segments on the
// device. Loads are single values, so any strides and widths take this path.
#include "grouped.cuh"
#include "epilogue.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, BK = 16;

__device__ __forceinline__ uint64_t dup2(float a)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
    return r;
}
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

// Operand strides: value (i, k) at i * s_i + k * s_k, one of them 1 (K_FIRST: s_k = 1).
// One chunk of T x 16 values into registers; out-of-range ones are zeros.
template <typename T, int TT, bool K_FIRST>
__device__ __forceinline__ void fetch(const T* p, long long ld, int n_i, int n_k, float (&v)[TT * BK / kThreads])
{
#pragma unroll
    for (int j = 0; j < TT * BK / kThreads; ++j) {
        const int idx = threadIdx.x + j * kThreads;
        const int i = K_FIRST ? idx / BK : idx % TT, k = K_FIRST ? idx % BK : idx / TT;
        v[j] = (i < n_i && k < n_k) ? as_f32(p[K_FIRST ? i * ld + k : k * ld + i]) : 0.f;
    }
}
template <int TT, bool K_FIRST>
__device__ __forceinline__ void put(float (&s)[BK][TT + 4], const float (&v)[TT * BK / kThreads])
{
#pragma unroll
    for (int j = 0; j < TT * BK / kThreads; ++j) {
        const int idx = threadIdx.x + j * kThreads;
        const int i = K_FIRST ? idx / BK : idx % TT, k = K_FIRST ? idx % BK : idx / TT;
        s[k][i] = v[j];
    }
}

// acc (+)= A B over n_k values: A is up to TT values of i by k at a, B at b likewise.
template <typename T, int TM, int TN, bool A_K, bool B_K>
__device__ __forceinline__ void tile_product(const T* a, long long lda, int n_m, const T* b, long long ldb, int n_n,
                                             int n_k, float (&As)[2][BK][TM + 4], float (&Bs)[2][BK][TN + 4],
                                             uint64_t (&acc)[TM / 16][TN / 32])
{
    constexpr int MT = TM / 16, NT = TN / 16;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float ra[TM * BK / kThreads], rb[TN * BK / kThreads];
    fetch<T, TM, A_K>(a, lda, n_m, n_k, ra);
    fetch<T, TN, B_K>(b, ldb, n_n, n_k, rb);
    int st = 0;
    for (int k0 = 0; k0 < n_k; k0 += BK, st ^= 1) {
        put<TM, A_K>(As[st], ra);
        put<TN, B_K>(Bs[st], rb);
        __syncthreads();
        if (k0 + BK < n_k) {
            const int k1 = k0 + BK;
            fetch<T, TM, A_K>(a + (A_K ? (long long)k1 : k1 * lda), lda, n_m, n_k - k1, ra);
            fetch<T, TN, B_K>(b + (B_K ? (long long)k1 : k1 * ldb), ldb, n_n, n_k - k1, rb);
        }
#pragma unroll
        for (int kk = 0; kk < BK; ++kk) {
            float av[MT];
            uint64_t bv[NT / 2];
            // rows ty*4.. and, in the larger tile, TM/2 + ty*4..; columns likewise: four
            // consecutive values per read, the lanes side by side in the banks
#pragma unroll
            for (int h = 0; h < MT / 4; ++h) {
                const float4 q = *reinterpret_cast<const float4*>(&As[st][kk][h * (TM / 2) + ty * 4]);
                av[4 * h] = q.x; av[4 * h + 1] = q.y; av[4 * h + 2] = q.z; av[4 * h + 3] = q.w;
            }
#pragma unroll
            for (int h = 0; h < NT / 4; ++h) {
                const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&Bs[st][kk][h * (TN / 2) + tx * 4]);
                bv[2 * h] = q.x; bv[2 * h + 1] = q.y;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint64_t d = dup2(av[i]);
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) fma2(acc[i][j], d, bv[j]);
            }
        }
    }
    __syncthreads();
}

template <typename T, int TM, int TN>
__device__ __forceinline__ void store_tile(T* out, long long ld, int n_m, int n_valid, int n_n,
                                           const uint64_t (&acc)[TM / 16][TN / 32])
{
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
    for (int i = 0; i < TM / 16; ++i) {
        const int m = (i / 4) * (TM / 2) + ty * 4 + i % 4;
        if (m >= n_m) continue;
#pragma unroll
        for (int j = 0; j < TN / 32; ++j) {
            const int n = (j / 2) * (TN / 2) + tx * 4 + 2 * (j % 2);
            float lo, hi;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(acc[i][j]));
            if (n < n_n) out[m * ld + n] = from_f32<T>(m < n_valid ? lo : 0.f);
            if (n + 1 < n_n) out[m * ld + n + 1] = from_f32<T>(m < n_valid ? hi : 0.f);
        }
    }
}

template <typename T, int TM, int TN, bool W_NK>
__global__ void __launch_bounds__(kThreads)
grouped_rows_kernel(const GroupedRows p)
{
    __shared__ __align__(16) float As[2][BK][TM + 4];
    __shared__ __align__(16) float Bs[2][BK][TN + 4];
    __shared__ SegmentTable table;
    read_segments<TM>(p.g, &table);
    const int* pre = table.pre;
    const int num_n = (p.N + TN - 1) / TN;
    const long long total = (long long)pre[p.g.E] * num_n;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        const int q = (int)(w / num_n), n0 = (int)(w % num_n) * TN;
        const int e = segment_at(pre, p.g.E, q);
        const Segment s = table.at(e);
        const int at = (q - pre[e]) * TM, row = s.begin + at, valid = s.valid - at;
        uint64_t acc[TM / 16][TN / 32] = {};
        if (valid > 0) {
            const T* x = static_cast<const T*>(p.X) + (long long)row * p.ldx;
            const T* wt = static_cast<const T*>(p.W) + e * p.sw + (W_NK ? (long long)n0 * p.ldw : (long long)n0);
            tile_product<T, TM, TN, true, W_NK>(x, p.ldx, valid, wt, p.ldw, p.N - n0, p.K, As, Bs, acc);
        }
        store_tile<T, TM, TN>(static_cast<T*>(p.Y) + (long long)row * p.ldy + n0, p.ldy, s.end - row, valid, p.N - n0, acc);
    }
}

template <typename T, int TM, int TN>
__global__ void __launch_bounds__(kThreads)
grouped_wgrad_kernel(const GroupedWgrad p)
{
    __shared__ __align__(16) float As[2][BK][TM + 4];
    __shared__ __align__(16) float Bs[2][BK][TN + 4];
    const int num_m = (p.M + TM - 1) / TM, num_n = (p.N + TN - 1) / TN;
    const long long per = (long long)num_m * num_n, total = per * p.g.E;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        const int e = (int)(w / per), r = (int)(w % per), m0 = r / num_n * TM, n0 = r % num_n * TN;
        const Segment s = segment_of(p.g, e);
        uint64_t acc[TM / 16][TN / 32] = {};
        if (s.valid > 0)
            tile_product<T, TM, TN, false, false>(static_cast<const T*>(p.A) + (long long)s.begin * p.lda + m0, p.lda,
                                                  p.M - m0, static_cast<const T*>(p.B) + (long long)s.begin * p.ldb + n0,
                                                  p.ldb, p.N - n0, s.valid, As, Bs, acc);
        store_tile<T, TM, TN>(static_cast<T*>(p.D) + e * p.sd + (long long)m0 * p.ldd + n0, p.ldd, p.M - m0, p.M - m0,
                              p.N - n0, acc);
    }
}

unsigned grid_of(long long tiles, int num_sms, int per_sm)
{
    const long long most = (long long)num_sms * per_sm;
    return (unsigned)(tiles < most ? (tiles > 0 ? tiles : 1) : most);
}

template <typename T, int TM, int TN>
cudaError_t rows_simt(const GroupedRows& p, int num_sms, cudaStream_t s)
{
    const long long tiles = row_tiles_bound(p.g.rows, p.g.E, TM) * ((p.N + TN - 1) / TN);
    const unsigned grid = grid_of(tiles, num_sms, TM == 128 ? 2 : 4);
    if (p.w_nk) grouped_rows_kernel<T, TM, TN, true><<<grid, kThreads, 0, s>>>(p);
    else grouped_rows_kernel<T, TM, TN, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int TM, int TN>
cudaError_t wgrad_simt(const GroupedWgrad& p, int num_sms, cudaStream_t s)
{
    const long long tiles = (long long)p.g.E * ((p.M + TM - 1) / TM) * ((p.N + TN - 1) / TN);
    grouped_wgrad_kernel<T, TM, TN><<<grid_of(tiles, num_sms, TM == 128 ? 2 : 4), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_rows_simt(const GroupedRows& p, int num_sms, cudaStream_t s)
{
    return rows_simt<float, 64, 64>(p, num_sms, s);
}
cudaError_t launch_grouped_wgrad_simt(const GroupedWgrad& p, int num_sms, cudaStream_t s)
{
    return wgrad_simt<float, 64, 64>(p, num_sms, s);
}

}  // namespace moe
