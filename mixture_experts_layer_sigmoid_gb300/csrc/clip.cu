// clip.cu -- global gradient norm over many tensors, and clipping by it.
//
//   norm = sqrt(sum of g^2 over all tensors),  out = g min(1, max_norm / norm)
//
// Two passes over the values (the norm has to be known before the first
// product): bound by HBM for large sets, by launches for small ones. 1.41 G bf16
// values: 411 us for the norm (6.9 TB/s, reads), 857 us for the product (6.6
// TB/s); twenty fp32 tensors of 6.3 MB together: 8.2 us. The tensors' table
// travels in the kernel's parameters, so a call copies nothing to the device and
// can be captured; blocks take chunks of any tensor, so neither one large tensor
// nor hundreds of small ones leave SMs idle.
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr int kClipThreads = 256;
// Chunk sizes: the largest that still gives every block one, so a small set is
// spread over the SMs and a large one keeps its pieces long.
constexpr int kAhead = 4;               // 16-byte pieces that a thread loads together
constexpr int kChunkMin = kClipThreads * kAhead * 16, kChunkMax = 1 << 16;
constexpr int kSmCount = 152;
constexpr int kClipBlocks = 8 * kSmCount;
// Tensors per launch: 32 bytes each, within the 32,764 of kernel parameters (a
// shorter table launches no faster).
constexpr int kClipBatch = 896;

struct Entry {
    const void* g;      // aligned down to 16 bytes
    void* out;          // matches g (the same number of values below the first), or null
    long long n;        // values, the ones below the first included
    int chunk;          // first chunk of this tensor in the batch
    int info;           // bit 0: bf16; bits 1-3: values below the first; bit 4: out is not 16-byte aligned as g is
};
struct Table {
    int count, chunks;
    int chunk_bytes;
    Entry e[kClipBatch];
};

__device__ __forceinline__ int find_entry(const Table& t, int chunk)
{
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].chunk <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ double shfl_xor_double(double v, int off)
{
    return __hiloint2double(__shfl_xor_sync(0xffffffffu, __double2hiint(v), off),
                            __shfl_xor_sync(0xffffffffu, __double2loint(v), off));
}

// Sum of v over the block, in a fixed order; valid in the first warp. 64-bit
// additions run at two a cycle and SM, so the block's values go through shared
// memory to one warp (13 instructions) and not through every warp's shuffles.
__device__ __forceinline__ double block_sum_double(double v, double* red)
{
    red[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    double s = red[threadIdx.x];
#pragma unroll
    for (int w = 1; w < kClipThreads / 32; ++w) s += red[threadIdx.x + 32 * w];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += shfl_xor_double(s, off);
    return s;
}

// One chunk of a tensor: `base` is 16-byte aligned, its values [lo, hi) belong
// to the tensor.
template <typename T>
struct Chunk {
    const T* base;
    T* out;
    int lo, hi;
    bool whole;      // all of the chunk's pieces are whole
    bool aligned;    // out is aligned as base is
};

template <typename T>
__device__ __forceinline__ Chunk<T> chunk_of(const Entry& e, int chunk, int chunk_bytes)
{
    const int values = chunk_bytes / (int)sizeof(T);
    const long long v0 = (long long)(chunk - e.chunk) * values;
    const long long left = e.n - v0;
    Chunk<T> c;
    c.base = static_cast<const T*>(e.g) + v0;
    c.out = static_cast<T*>(e.out) + v0;
    c.lo = chunk == e.chunk ? (e.info >> 1) & 7 : 0;
    c.hi = left < values ? (int)left : values;
    c.whole = c.lo == 0 && c.hi == values;
    c.aligned = !(e.info & 16);
    return c;
}

// Gives each piece of V values of a whole chunk to fn(index, raw), AHEAD pieces
// of the thread loaded before the first is used.
template <int AHEAD, typename T, typename FN>
__device__ __forceinline__ void whole_chunk(const Chunk<T>& c, FN&& fn)
{
    constexpr int V = 16 / (int)sizeof(T);
    constexpr int STEP = kClipThreads * V;
#pragma unroll 1
    for (int at = threadIdx.x * V; at < c.hi; at += AHEAD * STEP) {    // whole chunks are whole batches
        Raw<T, V> q[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) q[i] = load_raw<T, V>(c.base + at + i * STEP);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fn(at + i * STEP, q[i]);
    }
}

// The same for a tensor's first and last chunks: fn gets the whole pieces,
// fn1(index, raw) the single values of the others.
template <typename T, typename FN, typename FN1>
__device__ __forceinline__ void ragged_chunk(const Chunk<T>& c, FN&& fn, FN1&& fn1)
{
    constexpr int V = 16 / (int)sizeof(T);
    constexpr int STEP = kClipThreads * V;
    constexpr int AHEAD = 4;
#pragma unroll 1
    for (int p0 = threadIdx.x * V; p0 < c.hi; p0 += AHEAD * STEP) {
        Raw<T, V> q[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int p = p0 + i * STEP;
            if (p >= c.lo && p + V <= c.hi) q[i] = load_raw<T, V>(c.base + p);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int p = p0 + i * STEP;
            if (p >= c.lo && p + V <= c.hi) {
                fn(p, q[i]);
            } else {
#pragma unroll 1
                for (int j = p; j < p + V; ++j)
                    if (j >= c.lo && j < c.hi) fn1(j, load_raw<T, 1>(c.base + j));
            }
        }
    }
}

// Sum of squares of the thread's share in 64 bits.
template <typename T>
__device__ __noinline__ double squares_64(Chunk<T> c)
{
    constexpr int V = 16 / (int)sizeof(T);
    double d = 0.0;
#pragma unroll 1
    for (int p = threadIdx.x * V; p < c.hi; p += kClipThreads * V)
#pragma unroll 1
        for (int j = p; j < p + V; ++j)
            if (j >= c.lo && j < c.hi) {
                float v[1];
                unpack<T, 1>(load_raw<T, 1>(c.base + j), v);
                d += (double)v[0] * (double)v[0];
            }
    return d;
}

// A sum of squares as two fp32 values, s and what its roundings lost, e. Two such
// sums to a register pair, those of the even and of the odd values. `any`: some bit
// of the values is set.
struct Squares {
    uint64_t s = 0, e = 0;
    uint32_t any = 0;
};
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// s += x^2, and e += what the rounded sum t lost: with z = t - s it is x^2 - z where
// s >= x^2 (T. J. Dekker, "A floating-point technique for extending the available
// precision", Numer. Math. 18, 1971). Where a square is the larger one, as a thread's
// first ones are, z is rounded too, by 2^-25 of that square at most; EXACT keeps that
// by two more steps (D. Knuth, The Art of Computer Programming 2, 4.2.2).
template <typename T, int V, bool EXACT>
__device__ __forceinline__ void add_squares(const Raw<T, V>& q, Squares& a)
{
    float v[V];
    unpack<T, V>(q, v);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const uint64_t x = pair(v[i], V > 1 ? v[i + 1] : 0.f);
        const uint64_t t = fma2(x, x, a.s), nz = sub2(a.s, t);           // -z
        uint64_t d = fma2(x, x, nz);
        if constexpr (EXACT) d = add2(d, sub2(a.s, add2(t, nz)));
        a.e = add2(a.e, d);
        a.s = t;
    }
    if constexpr (V == 1) a.any |= q;
    else a.any |= q.x | q.y | q.z | q.w;
}

// The sum in 64 bits. At most 64 additions to a sum leave e below 2^-18 of it and
// e's own roundings below 2^-35 of it (2^-46 in the mean); what is lost where a square
// is the larger one comes to 2^-31 of a thread's sum in the mean and to less over the
// 256 threads of a whole chunk. The ends of tensors, the only chunks that few values
// have, are added exactly. Where squares or sums leave fp32's range (a sum that is not
// finite, or so small that squares may have lost bits) the share is summed again in 64
// bits, so the norm is right from the smallest values to the largest.
template <typename T>
__device__ __forceinline__ double checked(const Chunk<T>& c, const Squares& a)
{
    float s0, s1, e0, e1;
    unpair(a.s, s0, s1);
    unpair(a.e, e0, e1);
    const float s = s0 + s1;
    if (a.any && !(s > 0x1p-60f && s < 0x1p126f)) return squares_64(c);
    // s0 + s1 = s + r exactly, as above
    const float z = s - s0, r = (s0 - (s - z)) + (s1 - z);
    return (double)s + (double)(r + (e0 + e1));
}

template <typename T>
__device__ __noinline__ double ragged_squares(Chunk<T> c)
{
    constexpr int V = 16 / (int)sizeof(T);
    Squares a;
    ragged_chunk(c, [&](int, const Raw<T, V>& q) { add_squares<T, V, true>(q, a); },
                 [&](int, const Raw<T, 1>& q) { add_squares<T, 1, true>(q, a); });
    return checked(c, a);
}

// This thread's share of the sum of squares of one chunk.
template <typename T>
__device__ __forceinline__ double chunk_squares(const Chunk<T>& c)
{
    constexpr int V = 16 / (int)sizeof(T);
    if (!c.whole) return ragged_squares(c);
    Squares a;
    auto add = [&](int, const Raw<T, V>& q) { add_squares<T, V, false>(q, a); };
    // eight pieces ahead of the sums' work where a chunk has them (2.8 GB bf16: 411 us,
    // 420 with four)
    if (c.hi % (2 * kAhead * kClipThreads * V) == 0) whole_chunk<2 * kAhead>(c, add);
    else whole_chunk<kAhead>(c, add);
    return checked(c, a);
}

// Three blocks an SM for many chunks: at four the sums spill (2.8 GB bf16: 411 us, 419
// with four; 434 with three in two waves and a part). Four where that puts every chunk
// in the first wave (500 tensors of 101 values: 6.3 us, 8.4 with three).
template <int PER_SM>
__global__ void __launch_bounds__(kClipThreads, PER_SM)
norm_kernel(const __grid_constant__ Table t, double* __restrict__ part)
{
    __shared__ double red[kClipThreads];
    ptx::griddep_launch_dependents();
    double s = 0.0;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry& e = t.e[find_entry(t, c)];
        s += e.info & 1 ? chunk_squares(chunk_of<__nv_bfloat16>(e, c, t.chunk_bytes))
                        : chunk_squares(chunk_of<float>(e, c, t.chunk_bytes));
    }
    s = block_sum_double(s, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// sqrt(s) for any s >= 0: s = m 4^e with m in [1, 4), the root of m taken in fp32
// and corrected once by its residual (Newton's iteration) in 64 bits, to 2^-46 of
// it. The 64-bit root and quotient take a microsecond of a call that takes seven.
__device__ __forceinline__ double root(double s)
{
    const int hi = __double2hiint(s), lo = __double2loint(s);
    if (!(s > 0.0) || hi >= 0x7FF00000) return s;                    // zero, infinite or NaN
    if (hi < 0x00100000) return 0.0;                                // below 2^-1022: its root is below fp32's range
    const int e = ((hi >> 20) - 1023) >> 1;                         // floor
    const double m = __hiloint2double(hi - (e << 21), lo);
    const float r = __fsqrt_rn((float)m);
    const double n = fma(fma(-(double)r, (double)r, m), (double)(0.5f * rsqrtf((float)m)), (double)r);
    return __hiloint2double(__double2hiint(n) + (e << 20), __double2loint(n));
}

// The fp32 value nearest to min(1, limit / n): the quotient in fp32 with its
// remainder in 64 bits. A norm that is infinite in fp32 or NaN clips nothing.
__device__ __forceinline__ float coefficient(float limit, double n)
{
    const float nf = (float)n;
    if (!(n > (double)limit) || !(nf < __int_as_float(0x7F800000))) return 1.f;
    if (!(limit > 0x1p-60f && nf < 0x1p60f)) return (float)((double)limit / n);   // fp32 parts could leave its range
    const float inv = __fdividef(1.f, nf), q = limit * inv;
    return (float)fma(fma(-(double)q, n, (double)limit), (double)inv, (double)q);
}

// The norm from the parts' sum, and the coefficient for the limit; every block
// adds the parts in the same order.
struct Total { float norm, coef; };
__device__ __forceinline__ Total total_norm(const double* part, int nparts, float limit, double* red)
{
    __shared__ Total total;
    double s = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kClipThreads) s += __ldcg(part + i);
    s = block_sum_double(s, red);
    if (threadIdx.x == 0) {
        const double n = root(s);
        total = Total{(float)n, coefficient(limit, n)};
    }
    __syncthreads();
    return total;
}

__global__ void __launch_bounds__(kClipThreads)
norm_finish_kernel(const double* __restrict__ part, int nparts, float* __restrict__ norm)
{
    __shared__ double red[kClipThreads];
    ptx::griddep_wait();
    const Total t = total_norm(part, nparts, __int_as_float(0x7F800000), red);
    if (threadIdx.x == 0) *norm = t.norm;
}

// The bits of value i of a piece.
template <typename T, int V>
__device__ __forceinline__ Raw<T, 1> piece_value(const Raw<T, V>& q, int i)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) return w[i];
    else return (uint16_t)(w[i / 2] >> (16 * (i & 1)));
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> scaled(const Raw<T, V>& q, float f)
{
    float v[V];
    unpack<T, V>(q, v);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= f;
    return pack<T, V>(v);
}

template <typename T>
__device__ __noinline__ void ragged_scale(Chunk<T> c, bool clip, float f)
{
    constexpr int V = 16 / (int)sizeof(T);
    ragged_chunk(c,
        [&](int p, const Raw<T, V>& q) {
            const Raw<T, V> r = clip ? scaled<T, V>(q, f) : q;
            if (c.aligned) {
                store_raw<T, V>(c.out + p, r);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) store_raw<T, 1>(c.out + p + i, piece_value<T, V>(r, i));
            }
        },
        [&](int p, const Raw<T, 1>& q) { store_raw<T, 1>(c.out + p, clip ? scaled<T, 1>(q, f) : q); });
}

// One chunk of out = g f, or without clip a copy of its bits.
template <typename T>
__device__ __forceinline__ void clip_chunk(const Chunk<T>& c, bool clip, float f)
{
    constexpr int V = 16 / (int)sizeof(T);
    if (!c.whole || !c.aligned) ragged_scale(c, clip, f);
    else whole_chunk<kAhead>(c, [&](int p, const Raw<T, V>& q) { store_raw<T, V>(c.out + p, clip ? scaled<T, V>(q, f) : q); });
}

// out = g c with c from the norm; the last chunks first, since the norm's pass
// read them last and L2 still holds some: a 100 MB set takes 50.3 us, 52.3 in
// the other order (2.8 GB: 1251 us either way).
__global__ void __launch_bounds__(kClipThreads, 4)
clip_kernel(const __grid_constant__ Table t, const double* __restrict__ part, int nparts, float max_norm,
            float* __restrict__ norm)
{
    __shared__ double red[kClipThreads];
    ptx::griddep_wait();
    const Total total = total_norm(part, nparts, max_norm, red);
    if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = total.norm;
    const float f = total.coef;
    const bool clip = f < 1.f;
    for (int c = t.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        const Entry& e = t.e[find_entry(t, c)];
        if (!e.out || (!clip && e.out == e.g)) continue;
        if (e.info & 1) clip_chunk(chunk_of<__nv_bfloat16>(e, c, t.chunk_bytes), clip, f);
        else clip_chunk(chunk_of<float>(e, c, t.chunk_bytes), clip, f);
    }
}

int batches(int count) { return (count + kClipBatch - 1) / kClipBatch; }

// The table of tensors [first, first + count) of the list.
void fill_table(const moe_grad_t* list, int first, int count, int chunk_bytes, Table& t)
{
    t.count = count;
    t.chunk_bytes = chunk_bytes;
    long long chunks = 0;
    for (int i = 0; i < count; ++i) {
        const moe_grad_t& m = list[first + i];
        const int size = m.dtype == MOE_FP32 ? 4 : 2;
        const uintptr_t a = reinterpret_cast<uintptr_t>(m.g);
        const int lo = m.n > 0 ? (int)(a % 16 / size) : 0;
        Entry& e = t.e[i];
        e.chunk = (int)chunks;
        e.n = m.n > 0 ? m.n + lo : 0;
        e.g = m.n > 0 ? reinterpret_cast<const void*>(a - lo * size) : nullptr;
        e.out = m.n > 0 && m.out ? reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(m.out) - lo * size) : nullptr;
        e.info = (m.dtype == MOE_BF16 ? 1 : 0) | lo << 1 | (reinterpret_cast<uintptr_t>(e.out) % 16 ? 16 : 0);
        chunks += (e.n * size + chunk_bytes - 1) / chunk_bytes;
    }
    t.chunks = (int)chunks;
}

// The launches of one call, kClipBatch tensors at a time: every batch's sum of
// squares, then (writes) every batch's product, or the norm alone.
cudaError_t run_clip(int count, const moe_grad_t* list, int chunk_bytes, bool writes, float max_norm, float* norm,
                     double* part, cudaStream_t s)
{
    Table t;
    int nparts = 0;
    auto fill = [&](int first) {
        fill_table(list, first, count - first < kClipBatch ? count - first : kClipBatch, chunk_bytes, t);
        return (unsigned)(t.chunks < kClipBlocks ? (t.chunks > 0 ? t.chunks : 1) : kClipBlocks);
    };
    unsigned grid = 0;
    for (int first = 0; first < count || first == 0; first += kClipBatch) {
        grid = fill(first);
        const bool few = grid <= 4 * kSmCount;
        const unsigned blocks = few ? grid : 3 * kSmCount;           // one wave
        double* to = part + nparts;
        void* args[] = {&t, &to};
        const cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(few ? norm_kernel<4> : norm_kernel<3>), dim3(blocks),
                                               dim3(kClipThreads), args, 0, s);
        if (e != cudaSuccess) return e;
        count_launches();
        nparts += (int)blocks;
    }
    if (!writes) {
        count_launches();
        return launch_early(norm_finish_kernel, dim3(1), dim3(kClipThreads), s, (const double*)part, nparts, norm);
    }
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kClipThreads);
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    for (int first = 0; first < count; first += kClipBatch) {
        if (count > kClipBatch) grid = fill(first);
        cfg.gridDim = dim3(grid);
        float* to = first == 0 ? norm : nullptr;
        const double* from = part;
        void* args[] = {&t, &from, &nparts, &max_norm, &to};
        const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(clip_kernel), args);
        if (e != cudaSuccess) return e;
        count_launches();
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace moe

using namespace moe;

moe_status_t moe_clip_workspace_size(int count, size_t* ws_bytes)
{
    if (!ws_bytes || count < 0 || count > (1 << 20)) return MOE_ERR_INVALID_ARG;
    *ws_bytes = (size_t)(batches(count) > 0 ? batches(count) : 1) * kClipBlocks * sizeof(double);
    return MOE_OK;
}

moe_status_t moe_clip_grad_norm(int count, const moe_grad_t* list, float max_norm, float* norm,
                                void* ws, size_t ws_bytes, moe_stream_t stream)
{
    size_t need = 0;
    if (moe_clip_workspace_size(count, &need) != MOE_OK || (count > 0 && !list) || !norm || !ws || !(max_norm > 0.f))
        return MOE_ERR_INVALID_ARG;
    long long bytes = 0;
    bool writes = false;
    for (int i = 0; i < count; ++i) {
        const moe_grad_t& m = list[i];
        if (m.n < 0 || m.n > (1ll << 46) || (m.n > 0 && !m.g) || (m.dtype != MOE_FP32 && m.dtype != MOE_BF16) || m.reserved)
            return MOE_ERR_INVALID_ARG;
        const uintptr_t mask = m.dtype == MOE_FP32 ? 3 : 1;
        if (m.n > 0 && ((reinterpret_cast<uintptr_t>(m.g) | reinterpret_cast<uintptr_t>(m.out)) & mask))
            return MOE_ERR_MISALIGNED;
        bytes += m.n * (m.dtype == MOE_FP32 ? 4 : 2);
        if (bytes > (1ll << 46)) return MOE_ERR_INVALID_ARG;
        writes = writes || (m.n > 0 && m.out);
    }
    if (!is_aligned16(ws) || (reinterpret_cast<uintptr_t>(norm) & 3u)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;

    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    double* part = static_cast<double*>(ws);
    int chunk_bytes = kChunkMax;
    while (chunk_bytes > kChunkMin && bytes / chunk_bytes < kClipBlocks) chunk_bytes /= 2;
    const cudaError_t e = run_clip(count, list, chunk_bytes, writes, max_norm, norm, part, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
