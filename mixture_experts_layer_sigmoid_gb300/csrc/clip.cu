// clip.cu -- global gradient norm over many tensors, and clipping by it.
//
//   norm = sqrt(sum of g^2 over all tensors),  out = g min(1, max_norm / norm)
//
// Two passes over the values (the norm has to be known before the first
// product): bound by HBM for large sets, by launches for small ones. The
// tensors' table travels in the kernel's parameters, so a call copies nothing
// to the device and can be captured; blocks take 64 KiB chunks of any tensor,
// so neither one large tensor nor hundreds of small ones leave SMs idle.
#include "internal.h"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr int kClipThreads = 256;
constexpr int kChunkBytes = 1 << 16;
constexpr int kClipBlocks = 1216;       // eight per SM
constexpr int kClipBatch = 896;         // tensors per launch: 32 bytes each, within 32,764 of parameters

struct Entry {
    const void* g;      // aligned down to 16 bytes
    void* out;          // matches g (the same number of values below the first), or null
    long long n;        // values, the ones below the first included
    int chunk;          // first chunk of this tensor in the batch
    int info;           // bit 0: bf16; bits 1-3: values below the first; bit 4: out is not 16-byte aligned as g is
};
struct Table {
    int count, chunks;
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

__device__ __forceinline__ double block_sum_double(double v, double* red)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += shfl_xor_double(v, off);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    double s = lane < kClipThreads / 32 ? red[lane] : 0.0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += shfl_xor_double(s, off);
    return s;
}

// Values of the piece at index v0 that belong to the tensor: [lo, n).
template <typename T, int V>
__device__ __forceinline__ void load_piece(const T* g, long long v0, int lo, long long n, float (&v)[V])
{
    if (v0 >= lo && v0 + V <= n) {
        load_vec<T, V>(g + v0, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float u[1] = {0.f};
            if (v0 + i >= lo && v0 + i < n) load_vec<T, 1>(g + v0 + i, u);
            v[i] = u[0];
        }
    }
}

// This thread's share of the sum of squares of one chunk. The squares are
// added in fp32; where that leaves its range (a sum that is not finite, or so
// small that squares may have been flushed), the share is summed again in 64
// bits, so the norm is right from the smallest values to the largest.
template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, long long v0, int lo, long long n)
{
    constexpr int V = 16 / (int)sizeof(T);
    constexpr int VALUES = kChunkBytes / (int)sizeof(T);
    const long long end = v0 + VALUES < n ? v0 + VALUES : n;
    float s = 0.f;
    bool any = false;
    for (long long c = v0 + threadIdx.x * V; c < end; c += kClipThreads * V) {
        float v[V];
        load_piece<T, V>(g, c, lo, n, v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s = fmaf(v[i], v[i], s);
            any = any || v[i] != 0.f;
        }
    }
    if (!any || (s > 0x1p-60f && s < 0x1p126f)) return (double)s;
    double d = 0.0;
    for (long long c = v0 + threadIdx.x * V; c < end; c += kClipThreads * V) {
        float v[V];
        load_piece<T, V>(g, c, lo, n, v);
        for (int i = 0; i < V; ++i) d += (double)v[i] * (double)v[i];
    }
    return d;
}

__global__ void __launch_bounds__(kClipThreads)
norm_kernel(const __grid_constant__ Table t, double* __restrict__ part)
{
    __shared__ double red[kClipThreads / 32];
    double s = 0.0;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry& e = t.e[find_entry(t, c)];
        const int lo = (e.info >> 1) & 7;
        const long long at = (long long)(c - e.chunk) * kChunkBytes;
        s += e.info & 1 ? chunk_squares(static_cast<const __nv_bfloat16*>(e.g), at / 2, lo, e.n)
                        : chunk_squares(static_cast<const float*>(e.g), at / 4, lo, e.n);
    }
    s = block_sum_double(s, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// sqrt of the parts' sum: every block adds them in the same order.
__device__ __forceinline__ double total_norm(const double* part, int nparts, double* red)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kClipThreads) s += part[i];
    return sqrt(block_sum_double(s, red));
}

__global__ void __launch_bounds__(kClipThreads)
norm_finish_kernel(const double* __restrict__ part, int nparts, float* __restrict__ norm)
{
    __shared__ double red[kClipThreads / 32];
    const double n = total_norm(part, nparts, red);
    if (threadIdx.x == 0) *norm = (float)n;
}

// One chunk of out = g c, or without CLIP a copy of its bits.
template <typename T, bool CLIP>
__device__ __forceinline__ void scale_chunk(const T* g, T* out, long long v0, int lo, long long n, bool aligned, float c)
{
    constexpr int V = 16 / (int)sizeof(T);
    constexpr int VALUES = kChunkBytes / (int)sizeof(T);
    const long long end = v0 + VALUES < n ? v0 + VALUES : n;
    for (long long p = v0 + threadIdx.x * V; p < end; p += kClipThreads * V) {
        if (aligned && p >= lo && p + V <= n) {
            Raw<T, V> q = load_raw<T, V>(g + p);
            if constexpr (CLIP) {
                float v[V];
                unpack<T, V>(q, v);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] *= c;
                q = pack<T, V>(v);
            }
            store_raw<T, V>(out + p, q);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (p + i < lo || p + i >= n) continue;
                Raw<T, 1> q = load_raw<T, 1>(g + p + i);
                if constexpr (CLIP) {
                    float v[1];
                    unpack<T, 1>(q, v);
                    v[0] *= c;
                    q = pack<T, 1>(v);
                }
                store_raw<T, 1>(out + p + i, q);
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void clip_chunk(const Entry& e, int chunk, bool clip, float f)
{
    const T* g = static_cast<const T*>(e.g);
    T* out = static_cast<T*>(e.out);
    const long long v0 = (long long)(chunk - e.chunk) * (kChunkBytes / (int)sizeof(T));
    const int lo = (e.info >> 1) & 7;
    const bool aligned = !(e.info & 16);
    if (clip) scale_chunk<T, true>(g, out, v0, lo, e.n, aligned, f);
    else scale_chunk<T, false>(g, out, v0, lo, e.n, aligned, f);
}

// out = g c with c from the norm; the last chunks first, since the norm's
// pass read them last and L2 still holds them.
__global__ void __launch_bounds__(kClipThreads)
clip_kernel(const __grid_constant__ Table t, const double* __restrict__ part, int nparts, float max_norm,
            float* __restrict__ norm)
{
    __shared__ double red[kClipThreads / 32];
    const double n = total_norm(part, nparts, red);
    if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = (float)n;
    const bool clip = n > (double)max_norm && n - n == 0.0;
    const float f = clip ? (float)((double)max_norm / n) : 1.f;
    for (int c = t.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        const Entry& e = t.e[find_entry(t, c)];
        if (!e.out || (!clip && e.out == e.g)) continue;
        if (e.info & 1) clip_chunk<__nv_bfloat16>(e, c, clip, f);
        else clip_chunk<float>(e, c, clip, f);
    }
}

int batches(int count) { return (count + kClipBatch - 1) / kClipBatch; }

// The table of tensors [first, first + count) of the list.
void fill_table(const moe_grad_t* list, int first, int count, Table& t)
{
    t.count = count;
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
        chunks += (e.n * size + kChunkBytes - 1) / kChunkBytes;
    }
    t.chunks = (int)chunks;
}

unsigned clip_grid(const Table& t) { return t.chunks < kClipBlocks ? (t.chunks > 0 ? t.chunks : 1) : kClipBlocks; }

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
    Table t;
    int nparts = 0;
    for (int first = 0; first < count || first == 0; first += kClipBatch) {
        fill_table(list, first, count - first < kClipBatch ? count - first : kClipBatch, t);
        const unsigned grid = clip_grid(t);
        norm_kernel<<<grid, kClipThreads, 0, s>>>(t, part + nparts);
        count_launches();
        nparts += (int)grid;
    }
    if (writes) {
        for (int first = 0; first < count; first += kClipBatch) {
            fill_table(list, first, count - first < kClipBatch ? count - first : kClipBatch, t);
            clip_kernel<<<clip_grid(t), kClipThreads, 0, s>>>(t, part, nparts, max_norm, first == 0 ? norm : nullptr);
            count_launches();
        }
    } else {
        norm_finish_kernel<<<1, kClipThreads, 0, s>>>(part, nparts, norm);
        count_launches();
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
