// grouped_simt.cu -- products grouped by expert on the CUDA cores: the fp32 type
// (fp32 FMA arithmetic throughout, as the fp32 layer has it; the tensor cores have no
// mode of full fp32 precision).
//
//   rows            Y[r][n] = sum_k X[r][k] W[e(r)][k][n]
//   weight gradient D[e][m][n] = sum over the expert's rows r of A[r][m] B[r][n]
//
// A block of 256 threads owns a TM x TN tile of outputs, a thread (TM/16) x (TN/16) of
// them as pairs of columns (fma.rn.f32x2; scalar FMAs 128 us where pairs take 105). Chunks of 16 along the contraction come through a
// ring of three stages of shared memory by cp.async, four bytes at a time, so that any strides
// and widths take this path and operands are transposed on the way; with the loads through
// registers and one chunk ahead, a chunk cost a round trip to L2 (2042 rows of 1024 x 640
// 120 us). Each output is one thread's sum in ascending order. Blocks are persistent and
// read the segments on the device. Tiles of 128 x 128 need half of the reads of shared
// memory, tiles of 64 x 64 are taken while the larger ones do not fill the SMs.
#include "grouped.cuh"
#include "epilogue.cuh"

#include <atomic>

namespace moe {
namespace {

constexpr int kThreads = 256, BK = 16, kStages = 3;

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

// A stage of one operand: TT values by 16 along the contraction.
template <int TT> using Stage = float[BK][TT + 4];

// What a thread copies of each chunk of one operand: value (i, k) stands at i ld + k (K_FIRST)
// or k ld + i; a thread's values of a chunk have one i and k in steps, or the other way round.
template <int TT, bool K_FIRST>
struct Loader {
    static constexpr int COUNT = TT * BK / kThreads;
    static constexpr int STEP = K_FIRST ? kThreads / BK : kThreads / TT;    // of i, or of k
    const float *p, *first;             // the next chunk's; a value that exists
    long long step, chunk;
    int i, k, n_i;
    __device__ __forceinline__ Loader(const float* base, long long ld, int n_i_) : first(base), n_i(n_i_)
    {
        i = K_FIRST ? threadIdx.x / BK : threadIdx.x % TT;
        k = K_FIRST ? threadIdx.x % BK : threadIdx.x / TT;
        p = base + (K_FIRST ? i * ld + k : k * ld + i);
        step = STEP * ld;
        chunk = K_FIRST ? (long long)BK : BK * ld;
    }
    // the next chunk, of which n_k values along the contraction exist; the others are zeros
    __device__ __forceinline__ void copy(Stage<TT>& s, int n_k)
    {
        uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(&s[k][i]));
        const float* src = p;
#pragma unroll
        for (int j = 0; j < COUNT; ++j) {
            const bool have = K_FIRST ? k < n_k && i + j * STEP < n_i : k + j * STEP < n_k && i < n_i;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(have ? src : first), "r"(have ? 4 : 0) : "memory");
            src += step;
            dst += (K_FIRST ? STEP : STEP * (TT + 4)) * 4;
        }
        p += chunk;
    }
};

// acc = A B over n_k > 0 values: A is n_m values of i by k at a, B n_n at b likewise.
template <int TM, int TN, bool A_K, bool B_K>
__device__ __forceinline__ void tile_product(const float* a, long long lda, int n_m, const float* b, long long ldb, int n_n,
                                             int n_k, Stage<TM>* As, Stage<TN>* Bs, uint64_t (&acc)[TM / 16][TN / 32])
{
    constexpr int MT = TM / 16, NT = TN / 16;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    Loader<TM, A_K> la(a, lda, n_m);
    Loader<TN, B_K> lb(b, ldb, n_n);
    auto load = [&](int st, int left) {
        if (left > 0) {
            la.copy(As[st], left);
            lb.copy(Bs[st], left);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load(i, n_k - i * BK);
    int st = 0;
    for (int k0 = 0; k0 < n_k; k0 += BK) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();                       // this chunk is there, and the stage before it is read
        load(st == 0 ? kStages - 1 : st - 1, n_k - k0 - (kStages - 1) * BK);
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
        st = st + 1 == kStages ? 0 : st + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
}

template <int TM, int TN>
__device__ __forceinline__ void store_tile(float* out, long long ld, int n_m, int n_valid, int n_n,
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
            if (n < n_n) out[m * ld + n] = m < n_valid ? lo : 0.f;
            if (n + 1 < n_n) out[m * ld + n + 1] = m < n_valid ? hi : 0.f;
        }
    }
}

template <int TM, int TN>
constexpr int kStageBytes = kStages * BK * (TM + TN + 8) * 4;

template <int TM, int TN, bool W_NK>
__global__ void __launch_bounds__(kThreads, TM == 128 ? 2 : 3)
grouped_rows_kernel(const GroupedRows p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Stage<TM>* As = reinterpret_cast<Stage<TM>*>(smem);
    Stage<TN>* Bs = reinterpret_cast<Stage<TN>*>(smem + kStages * sizeof(Stage<TM>));
    SegmentTable& table = *reinterpret_cast<SegmentTable*>(smem + kStageBytes<TM, TN>);
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
            const float* x = static_cast<const float*>(p.X) + (long long)row * p.ldx;
            const float* wt = static_cast<const float*>(p.W) + e * p.sw + (W_NK ? (long long)n0 * p.ldw : (long long)n0);
            tile_product<TM, TN, true, W_NK>(x, p.ldx, valid, wt, p.ldw, p.N - n0, p.K, As, Bs, acc);
        }
        store_tile<TM, TN>(static_cast<float*>(p.Y) + (long long)row * p.ldy + n0, p.ldy, s.end - row, valid, p.N - n0, acc);
    }
}

template <int TM, int TN>
__global__ void __launch_bounds__(kThreads, TM == 128 ? 2 : 3)
grouped_wgrad_kernel(const GroupedWgrad p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Stage<TM>* As = reinterpret_cast<Stage<TM>*>(smem);
    Stage<TN>* Bs = reinterpret_cast<Stage<TN>*>(smem + kStages * sizeof(Stage<TM>));
    const int num_m = (p.M + TM - 1) / TM, num_n = (p.N + TN - 1) / TN;
    const long long per = (long long)num_m * num_n, total = per * p.g.E;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        const int e = (int)(w / per), r = (int)(w % per), m0 = r / num_n * TM, n0 = r % num_n * TN;
        const Segment s = segment_of(p.g, e);
        uint64_t acc[TM / 16][TN / 32] = {};
        if (s.valid > 0)
            tile_product<TM, TN, false, false>(static_cast<const float*>(p.A) + (long long)s.begin * p.lda + m0, p.lda,
                                               p.M - m0, static_cast<const float*>(p.B) + (long long)s.begin * p.ldb + n0,
                                               p.ldb, p.N - n0, s.valid, As, Bs, acc);
        store_tile<TM, TN>(static_cast<float*>(p.D) + e * p.sd + (long long)m0 * p.ldd + n0, p.ldd, p.M - m0, p.M - m0,
                           p.N - n0, acc);
    }
}

// A persistent launch; the kernel's shared memory is set up on the first call of a device.
template <typename P>
cudaError_t launch(void (*k)(const P), const P& p, int smem, std::atomic<bool> (&ready)[64], long long tiles, int most,
                   cudaStream_t s)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev].store(true, std::memory_order_release);
    }
    k<<<(unsigned)(tiles < most ? (tiles > 0 ? tiles : 1) : most), kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

template <int TT, bool W_NK>
cudaError_t rows_simt(const GroupedRows& p, int num_sms, cudaStream_t s)
{
    static std::atomic<bool> ready[64];
    const long long tiles = row_tiles_bound(p.g.rows, p.g.E, TT) * ((p.N + TT - 1) / TT);
    return launch(grouped_rows_kernel<TT, TT, W_NK>, p, kStageBytes<TT, TT> + (int)sizeof(SegmentTable), ready, tiles,
                  num_sms * (TT == 128 ? 2 : 3), s);
}
template <int TT>
cudaError_t wgrad_simt(const GroupedWgrad& p, int num_sms, cudaStream_t s)
{
    static std::atomic<bool> ready[64];
    const long long tiles = (long long)p.g.E * ((p.M + TT - 1) / TT) * ((p.N + TT - 1) / TT);
    return launch(grouped_wgrad_kernel<TT, TT>, p, kStageBytes<TT, TT>, ready, tiles, num_sms * (TT == 128 ? 2 : 3), s);
}
// Whether tiles of 128 x 128 are at least four for each SM.
bool large_tiles(long long by_m, int n, int num_sms) { return by_m * ((n + 127) / 128) >= 4ll * num_sms; }

}  // namespace

cudaError_t launch_grouped_rows_simt(const GroupedRows& p, int num_sms, cudaStream_t s)
{
    if (large_tiles(p.g.rows / 128, p.N, num_sms))
        return p.w_nk ? rows_simt<128, true>(p, num_sms, s) : rows_simt<128, false>(p, num_sms, s);
    return p.w_nk ? rows_simt<64, true>(p, num_sms, s) : rows_simt<64, false>(p, num_sms, s);
}
cudaError_t launch_grouped_wgrad_simt(const GroupedWgrad& p, int num_sms, cudaStream_t s)
{
    return large_tiles((long long)p.g.E * ((p.M + 127) / 128), p.N, num_sms) ? wgrad_simt<128>(p, num_sms, s)
                                                                             : wgrad_simt<64>(p, num_sms, s);
}

}  // namespace moe
