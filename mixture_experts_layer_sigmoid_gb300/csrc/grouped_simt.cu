// grouped_simt.cu -- products grouped by expert on the CUDA cores: the fp32 type
// (fp32 FMA arithmetic throughout, as the fp32 layer has it; the tensor cores have no
// mode of full fp32 precision).
//
//   rows            Y[r][n] = sum_k X[r][k] W[e(r)][k][n]
//   weight gradient D[e][m][n] = sum over the expert's rows r of A[r][m] B[r][n]
//
// A block of 256 threads owns a tile of TT x TT outputs (16 x 64 for few rows), a thread
// (TT/16)^2 of them. Chunks of
// 32 along the contraction come through a ring of stages of shared memory by cp.async,
// each operand as it lies in memory: in 16-byte pieces where its rows are aligned (four-byte
// ones, transposed on the way, took 107 us for 2042 rows of 1024 x 640), else value by value.
// A thread reads four values along the contraction (or four neighbours at each of four
// steps) at a time; the layout in shared memory keeps both ways free of bank conflicts. Each
// output is one thread's sum in ascending order, in pieces of 256 terms that are added to a
// running sum (8192 products of unit normal values: rms error 2.8e-5, one chain 1.5e-4, for 1% of
// the time; the running sums in shared memory took 2% more). Blocks are persistent and read the segments
// on the device. Tiles of 128 need half of the reads of shared memory; tiles of 64 are taken
// while the larger ones are fewer than four for each SM.
#include "grouped.cuh"
#include "per_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256, BK = 32;
constexpr int kTerms = 256;                    // of a piece of a sum
// Stages of the ring: with few rows the time is the loads' (one row of 8192 x 8192 197 us with three).
template <int TM> constexpr int kStages = TM == 16 ? 8 : 3;

// One operand of a tile: TT values of i by the contraction, value (i, k) at p + i ld + k
// (K_FIRST) or p + k ld + i; n_i of the i exist. In shared memory a chunk lies the same way, in
// rows of BK + 4 or TT + 4.
template <int TT, bool K_FIRST>
struct Operand {
    static constexpr int ROWS = K_FIRST ? TT : BK, ROW = K_FIRST ? BK : TT, LD = ROW + 4;
    static constexpr int STAGE = ROWS * LD;    // values
    static constexpr int PER = TT / 16;        // of a thread
    const float* p;
    long long ld;
    int n_i;
    bool vec;                                  // rows in 16-byte pieces

    // Copies the chunk from k0 on, of which `left` along the contraction exist; the rest is zeros.
    __device__ __forceinline__ void copy(float* s, int k0, int left) const
    {
        const float* src = p + (K_FIRST ? (long long)k0 : k0 * ld);
        const int n_rows = K_FIRST ? n_i : left, n_row = K_FIRST ? left : n_i;
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(s));
        if (vec) {
#pragma unroll
            for (int j = 0; j < (ROWS * ROW / 4 + kThreads - 1) / kThreads; ++j) {
                const int c = threadIdx.x + j * kThreads, r = c / (ROW / 4), x = c % (ROW / 4) * 4;
                if (ROWS * ROW / 4 < kThreads && r >= ROWS) break;
                const int n = r < n_rows ? min(max(n_row - x, 0), 4) : 0;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (r * LD + x) * 4),
                             "l"(n > 0 ? src + r * ld + x : p), "r"(4 * n) : "memory");
            }
        } else {
#pragma unroll 4
            for (int j = 0; j < ROWS * ROW / kThreads; ++j) {
                const int c = threadIdx.x + j * kThreads, r = c / ROW, x = c % ROW;
                const bool have = r < n_rows && x < n_row;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + (r * LD + x) * 4),
                             "l"(have ? src + r * ld + x : p), "r"(have ? 4 : 0) : "memory");
            }
        }
    }
    // The i of a thread's j-th value: neighbours where they are read together, else sixteen apart.
    static __device__ __forceinline__ int index(int t, int j)
    {
        return K_FIRST ? t + 16 * j : (j / 4) * (TT / 2) + t * 4 + j % 4;
    }
    // v[j][q]: the thread's j-th value at step k + q
    __device__ __forceinline__ void read(const float* s, int t, int k, float (&v)[PER][4]) const
    {
        if constexpr (K_FIRST) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const float4 f = *reinterpret_cast<const float4*>(s + index(t, j) * LD + k);
                v[j][0] = f.x; v[j][1] = f.y; v[j][2] = f.z; v[j][3] = f.w;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int h = 0; h < PER / 4; ++h) {
                    const float4 f = *reinterpret_cast<const float4*>(s + (k + q) * LD + index(t, 4 * h));
                    v[4 * h][q] = f.x; v[4 * h + 1][q] = f.y; v[4 * h + 2][q] = f.z; v[4 * h + 3][q] = f.w;
                }
        }
    }
};

template <typename OA, typename OB>
constexpr int stage_values() { return OA::STAGE + OB::STAGE; }

// acc = A B over n_k > 0 values.
template <int S, typename OA, typename OB>
__device__ __forceinline__ void tile_product(const OA& a, const OB& b, int n_k, float* smem, float (&acc)[OA::PER][OB::PER])
{
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float sums[OA::PER][OB::PER] = {};
    auto load = [&](int st, int k0) {
        if (k0 < n_k) {
            a.copy(smem + st * stage_values<OA, OB>(), k0, n_k - k0);
            b.copy(smem + st * stage_values<OA, OB>() + OA::STAGE, k0, n_k - k0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) load(i, i * BK);
    int st = 0;
    for (int k0 = 0;;) {
        for (const int stop = min(n_k, k0 + kTerms); k0 < stop; k0 += BK) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncthreads();                   // this chunk is there, and the stage before it is read
            load(st == 0 ? S - 1 : st - 1, k0 + (S - 1) * BK);
            const float* sa = smem + st * stage_values<OA, OB>();
            const float* sb = sa + OA::STAGE;
#pragma unroll
            for (int k = 0; k < BK; k += 4) {
                float av[OA::PER][4], bv[OB::PER][4];
                a.read(sa, ty, k, av);
                b.read(sb, tx, k, bv);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < OA::PER; ++i)
#pragma unroll
                        for (int j = 0; j < OB::PER; ++j) acc[i][j] = fmaf(av[i][q], bv[j][q], acc[i][j]);
            }
            st = st + 1 == S ? 0 : st + 1;
        }
        if (k0 >= n_k) break;
        // a piece ends, and more follow
#pragma unroll
        for (int i = 0; i < OA::PER; ++i)
#pragma unroll
            for (int j = 0; j < OB::PER; ++j) {
                sums[i][j] += acc[i][j];
                acc[i][j] = 0.f;
            }
    }
    if (n_k > kTerms) {
#pragma unroll
        for (int i = 0; i < OA::PER; ++i)
#pragma unroll
            for (int j = 0; j < OB::PER; ++j) acc[i][j] += sums[i][j];
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
}

template <typename OA, typename OB>
__device__ __forceinline__ void store_tile(float* out, long long ld, int n_m, int n_valid, int n_n,
                                           const float (&acc)[OA::PER][OB::PER])
{
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
    for (int i = 0; i < OA::PER; ++i) {
        const int m = OA::index(ty, i);
        if (m >= n_m) continue;
#pragma unroll
        for (int j = 0; j < OB::PER; ++j) {
            const int n = OB::index(tx, j);
            if (n < n_n) out[m * ld + n] = m < n_valid ? acc[i][j] : 0.f;
        }
    }
}

// Whether matrices at p with these strides in values have rows on 16-byte boundaries.
bool vectors(const void* p, long long ld, long long stride)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 4 == 0 && stride % 4 == 0;
}

struct Vec { bool a, b; };

template <int TM, int TT, bool W_NK>
__global__ void __launch_bounds__(kThreads, TT == 128 ? 1 : 2)
grouped_rows_kernel(const GroupedRows p, const Vec vec)
{
    using OA = Operand<TM, true>;
    using OB = Operand<TT, W_NK>;
    extern __shared__ __align__(16) float smem[];
    SegmentTable& table = *reinterpret_cast<SegmentTable*>(smem + kStages<TM> * stage_values<OA, OB>());
    read_segments<TM>(p.g, &table);
    const int* pre = table.pre;
    const int num_n = (p.N + TT - 1) / TT;
    const long long total = (long long)pre[p.g.E] * num_n;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        const int q = (int)(w / num_n), n0 = (int)(w % num_n) * TT;
        const int e = segment_at(pre, p.g.E, q);
        const Segment s = table.at(e);
        const int at = (q - pre[e]) * TM, row = s.begin + at, valid = s.valid - at;
        float acc[OA::PER][OB::PER] = {};
        if (valid > 0) {
            const OA a{static_cast<const float*>(p.X) + (long long)row * p.ldx, p.ldx, valid, vec.a};
            const OB b{static_cast<const float*>(p.W) + e * p.sw + (W_NK ? (long long)n0 * p.ldw : (long long)n0), p.ldw,
                       p.N - n0, vec.b};
            tile_product<kStages<TM>>(a, b, p.K, smem, acc);
        }
        store_tile<OA, OB>(static_cast<float*>(p.Y) + (long long)row * p.ldy + n0, p.ldy, min(s.end - row, TM), valid,
                           p.N - n0, acc);
    }
}

template <int TT>
__global__ void __launch_bounds__(kThreads, TT == 128 ? 1 : 2)
grouped_wgrad_kernel(const GroupedWgrad p, const Vec vec)
{
    using O = Operand<TT, false>;
    extern __shared__ __align__(16) float smem[];
    const int num_m = (p.M + TT - 1) / TT, num_n = (p.N + TT - 1) / TT;
    const long long per = (long long)num_m * num_n, total = per * p.g.E;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        const int e = (int)(w / per), r = (int)(w % per), m0 = r / num_n * TT, n0 = r % num_n * TT;
        const Segment s = segment_of(p.g, e);
        float acc[O::PER][O::PER] = {};
        if (s.valid > 0) {
            const O a{static_cast<const float*>(p.A) + (long long)s.begin * p.lda + m0, p.lda, p.M - m0, vec.a};
            const O b{static_cast<const float*>(p.B) + (long long)s.begin * p.ldb + n0, p.ldb, p.N - n0, vec.b};
            tile_product<kStages<TT>>(a, b, s.valid, smem, acc);
        }
        store_tile<O, O>(static_cast<float*>(p.D) + e * p.sd + (long long)m0 * p.ldd + n0, p.ldd, p.M - m0, p.M - m0,
                             p.N - n0, acc);
    }
}

// A persistent launch; the kernel's shared memory is set up on the first call of a device.
template <typename P>
cudaError_t launch(void (*k)(const P, const Vec), const P& p, const Vec& vec, int smem, std::atomic<int> (&ready)[kMaxDevices],
                   long long tiles, int most, cudaStream_t s)
{
    int dev = 0, set = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = per_device<cudaError_t>(ready, dev, [&](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    }, &set);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)(tiles < most ? (tiles > 0 ? tiles : 1) : most), kThreads, smem, s>>>(p, vec);
    return cudaGetLastError();
}

template <int TM, int TT, bool W_NK>
cudaError_t rows_simt(const GroupedRows& p, int num_sms, cudaStream_t s)
{
    static std::atomic<int> ready[kMaxDevices];
    using OA = Operand<TM, true>;
    using OB = Operand<TT, W_NK>;
    constexpr int smem = kStages<TM> * stage_values<OA, OB>() * 4 + (int)sizeof(SegmentTable);
    const long long tiles = row_tiles_bound(p.g.rows, p.g.E, TM) * ((p.N + TT - 1) / TT);
    return launch(grouped_rows_kernel<TM, TT, W_NK>, p, Vec{vectors(p.X, p.ldx, 0), vectors(p.W, p.ldw, p.sw)}, smem, ready,
                  tiles, num_sms * (TT == 128 ? 1 : 2), s);
}
template <int TT>
cudaError_t wgrad_simt(const GroupedWgrad& p, int num_sms, cudaStream_t s)
{
    static std::atomic<int> ready[kMaxDevices];
    using O = Operand<TT, false>;
    constexpr int smem = kStages<TT> * stage_values<O, O>() * 4;
    const long long tiles = (long long)p.g.E * ((p.M + TT - 1) / TT) * ((p.N + TT - 1) / TT);
    return launch(grouped_wgrad_kernel<TT>, p, Vec{vectors(p.A, p.lda, 0), vectors(p.B, p.ldb, 0)}, smem, ready, tiles,
                  num_sms * (TT == 128 ? 1 : 2), s);
}
// Rows of the buffers (padding included) for each expert below which a tile has 16 of them (one
// row of 8192 x 8192: 289 us with 64).
constexpr long long kFewRows = 32;
// Whether tiles of 128 x 128 are at least four for each SM.
bool large_tiles(long long by_m, int n, int num_sms) { return by_m * ((n + 127) / 128) >= 4ll * num_sms; }

}  // namespace

cudaError_t launch_grouped_rows_simt(const GroupedRows& p, int num_sms, cudaStream_t s)
{
    if (p.g.rows / p.g.E < kFewRows)
        return p.w_nk ? rows_simt<16, 64, true>(p, num_sms, s) : rows_simt<16, 64, false>(p, num_sms, s);
    if (large_tiles(p.g.rows / 128, p.N, num_sms))
        return p.w_nk ? rows_simt<128, 128, true>(p, num_sms, s) : rows_simt<128, 128, false>(p, num_sms, s);
    return p.w_nk ? rows_simt<64, 64, true>(p, num_sms, s) : rows_simt<64, 64, false>(p, num_sms, s);
}
cudaError_t launch_grouped_wgrad_simt(const GroupedWgrad& p, int num_sms, cudaStream_t s)
{
    return large_tiles((long long)p.g.E * ((p.M + 127) / 128), p.N, num_sms) ? wgrad_simt<128>(p, num_sms, s)
                                                                             : wgrad_simt<64>(p, num_sms, s);
}

}  // namespace moe
