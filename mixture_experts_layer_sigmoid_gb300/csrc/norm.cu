// norm.cu -- residual addition and root-mean-square norm, forward (act or
// 8-bit output) and backward, for the layer's pre-norm.
//
//   s = x + r,  rstd = (mean(s^2) + eps)^(-1/2),  y = s rstd w
//   n = h rstd, c = mean(w dy n):  dx = rstd (w dy - n c) + dh,
//                                  dw = sum over rows of dy n
//
// About ten operations per value against 2 to 16 bytes moved: every kernel
// here is bound by HBM (large inputs) or by latency (a few rows).
#include "internal.h"
#include "mx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 256;
// Row groups of the weight gradient's partial sums (blocks of the backward):
// two per SM.
constexpr int kNormParts = 304;

// Sum of v over the block's NT threads, the same order on every call; `red`
// holds NT / 32 floats and may be reused after the next __syncthreads.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (NT == 32) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = lane < NT / 32 ? red[lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}

template <typename T> struct FwdArgs {
    const T* x; const T* r; const float* w;
    T* h; T* y; float* rstd; uint8_t* codes; void* scales;
    long long ldx, ldr, ldh, ldy;
    int rows, H; float eps;
};

// The 8-bit output of one piece of V values at column c of a row. All lanes
// of a warp call it together; `act` is false past the row's end, and the
// lanes of one block are all active or all inactive (H is a multiple of 128).
template <int QUANT, int V>
__device__ __forceinline__ void quantise(const float (&v)[V], bool act, int row, int c, int H,
                                         uint8_t* codes, void* scales)
{
    constexpr int BLOCK = QUANT == MOE_NORM_MXFP8 ? 32 : 128;
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
    for (int off = BLOCK / V / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    if (!act) return;
    float q[V];
    if constexpr (QUANT == MOE_NORM_MXFP8) {
        const int e = mx_exp(a);
        const float s = mx_inv(e);                       // a power of two: exact
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = v[i] * s;
        if (c % BLOCK == 0)
            static_cast<uint8_t*>(scales)[((size_t)(row >> 7) * (H / 128) + c / 128) * 512 +
                                          atom_byte(row & 127, (c / 32) & 3)] = (uint8_t)(e + 127);
    } else {
        const float t = __fdiv_rn(a, 448.f);
        const float s = t == 0.f ? 1.f : t;              // zero, or too small for a scale
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = __fdiv_rn(v[i], s);
        if (c % BLOCK == 0) static_cast<float*>(scales)[(size_t)row * (H / 128) + c / 128] = s;
    }
    uint32_t* out = reinterpret_cast<uint32_t*>(codes + (size_t)row * H + c);
    if constexpr (V == 8)
        *reinterpret_cast<uint2*>(out) = make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
    else if constexpr (V == 4)
        *out = e4m3x4(q[0], q[1], q[2], q[3]);
}

// The scale bytes of rows past the last one in the last 128-row tile (their
// blocks run beside the rows' blocks).
__device__ __forceinline__ void zero_scale_row(uint8_t* scales, int row, int H)
{
    for (int kb = threadIdx.x; kb < H / 128; kb += blockDim.x)
        *reinterpret_cast<uint32_t*>(scales + ((size_t)(row >> 7) * (H / 128) + kb) * 512 +
                                     atom_byte(row & 127, 0)) = 0u;
}

// One block per row, any width: the row is read twice (the second time from
// L2), so h and y may overwrite x or the residual.
template <typename T, int V, int QUANT>
__global__ void __launch_bounds__(kNormThreads)
norm_fwd_loop_kernel(FwdArgs<T> a)
{
    __shared__ float red[kNormThreads / 32];
    const int row = blockIdx.x;
    if (QUANT == MOE_NORM_MXFP8 && row >= a.rows) {
        zero_scale_row(static_cast<uint8_t*>(a.scales), row, a.H);
        return;
    }
    const T* x = a.x + (size_t)row * a.ldx;
    const T* r = a.r ? a.r + (size_t)row * a.ldr : nullptr;
    float ss = 0.f;
    for (int c = threadIdx.x * V; c < a.H; c += kNormThreads * V) {
        float v[V], u[V];
        load_vec<T, V>(x + c, v);
        if (r) {
            load_vec<T, V>(r + c, u);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] += u[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(v[i], v[i], ss);
    }
    const float rstd = rsqrtf(block_sum<kNormThreads>(ss, red) / (float)a.H + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    for (int c0 = 0; c0 < a.H; c0 += kNormThreads * V) {
        const int c = c0 + threadIdx.x * V;
        const bool act = c < a.H;
        float v[V], u[V], w[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
        if (act) {
            load_vec<T, V>(x + c, v);
            if (r) {
                load_vec<T, V>(r + c, u);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] += u[i];
            }
            if (a.h) store_vec<T, V>(a.h + (size_t)row * a.ldh + c, v);
            load_f32<V>(a.w + c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = v[i] * rstd * w[i];
            if (a.y) store_vec<T, V>(a.y + (size_t)row * a.ldy + c, v);
        }
        if constexpr (QUANT != MOE_NORM_PLAIN) quantise<QUANT, V>(v, act, row, c, a.H, a.codes, a.scales);
    }
}

template <typename T> struct BwdArgs {
    const T* dy; const T* h; const float* rstd; const float* w; const T* dh;
    T* dx; float* part;   // part: gridDim.x x H partial sums of dw, or null
    long long lddy, ldh, lddh, lddx;
    int rows, H;
};

// Block b takes rows b, b + gridDim.x, ...; each thread always holds the same
// columns, so it adds its rows' dy n into part[b] alone.
template <typename T, int V>
__global__ void __launch_bounds__(kNormThreads)
norm_bwd_loop_kernel(BwdArgs<T> a)
{
    __shared__ float red[kNormThreads / 32];
    float* part = a.part ? a.part + (size_t)blockIdx.x * a.H : nullptr;
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* dy = a.dy + (size_t)row * a.lddy;
        const T* h = a.h + (size_t)row * a.ldh;
        const T* dh = a.dh ? a.dh + (size_t)row * a.lddh : nullptr;
        T* dx = a.dx + (size_t)row * a.lddx;
        const float rstd = a.rstd[row];
        float d = 0.f;
        for (int c = threadIdx.x * V; c < a.H; c += kNormThreads * V) {
            float g[V], v[V], w[V];
            load_vec<T, V>(dy + c, g);
            load_vec<T, V>(h + c, v);
            load_f32<V>(a.w + c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) d = fmaf(g[i] * w[i], v[i], d);
        }
        __syncthreads();                       // red of the previous row is read
        const float m = block_sum<kNormThreads>(d, red) * rstd / (float)a.H;
        for (int c = threadIdx.x * V; c < a.H; c += kNormThreads * V) {
            float g[V], v[V], w[V], o[V], p[V];
            load_vec<T, V>(dy + c, g);
            load_vec<T, V>(h + c, v);
            load_f32<V>(a.w + c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = v[i] * rstd;
                o[i] = rstd * fmaf(-n, m, g[i] * w[i]);
                p[i] = g[i] * n;
            }
            if (dh) {
                float u[V];
                load_vec<T, V>(dh + c, u);
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] += u[i];
            }
            if (part) {
                if (row != (int)blockIdx.x) {
                    float q[V];
                    load_f32<V>(part + c, q);
#pragma unroll
                    for (int i = 0; i < V; ++i) p[i] += q[i];
                }
                store_f32<V>(part + c, p);
            }
            store_vec<T, V>(dx + c, o);
        }
    }
}

// dw[c] = sum of the parts in ascending order within each of 8 phases, the
// phases then added in order.
__global__ void __launch_bounds__(256)
norm_dweight_kernel(const float* __restrict__ part, int nparts, int H, float* __restrict__ dw)
{
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, ph = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < H)
        for (int b = ph; b < nparts; b += 8) s += part[(size_t)b * H + c];
    red[ph][lane] = s;
    __syncthreads();
    if (ph == 0 && c < H) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += red[i][lane];
        dw[c] = t;
    }
}

int norm_parts(int rows) { return rows < kNormParts ? rows : kNormParts; }

template <typename T, int QUANT>
cudaError_t launch_fwd(const FwdArgs<T>& a, int bytes, cudaStream_t s)
{
    constexpr int V16 = 16 / (int)sizeof(T);
    const int grid = QUANT == MOE_NORM_MXFP8 ? (a.rows + 127) / 128 * 128 : a.rows;
    if (bytes == 16) norm_fwd_loop_kernel<T, V16, QUANT><<<grid, kNormThreads, 0, s>>>(a);
    if constexpr (QUANT == MOE_NORM_PLAIN) {
        if (bytes == 4) norm_fwd_loop_kernel<T, 4 / (int)sizeof(T), QUANT><<<grid, kNormThreads, 0, s>>>(a);
        else if (bytes == 2) norm_fwd_loop_kernel<T, 1, QUANT><<<grid, kNormThreads, 0, s>>>(a);
    }
    count_launches();
    return cudaGetLastError();
}

template <typename T>
moe_status_t fwd(int rows, int H, int quant, float eps, const moe_norm_fwd_args_t& g, cudaStream_t s)
{
    FwdArgs<T> a{static_cast<const T*>(g.x), static_cast<const T*>(g.residual), g.weight,
                 static_cast<T*>(g.h), static_cast<T*>(g.y), g.rstd, g.codes, g.scales,
                 g.ldx, g.ldr, g.ldh, g.ldy, rows, H, eps};
    long long st[4];
    int n = 0;
    st[n++] = g.ldx;
    if (g.residual) st[n++] = g.ldr;
    if (g.h) st[n++] = g.ldh;
    if (g.y) st[n++] = g.ldy;
    const int bytes = access_bytes(H, (int)sizeof(T), st, n);
    if (quant != MOE_NORM_PLAIN && bytes != 16) return MOE_ERR_MISALIGNED;
    if (rows == 0) return MOE_OK;
    cudaError_t e;
    if (quant == MOE_NORM_PLAIN) e = launch_fwd<T, MOE_NORM_PLAIN>(a, bytes, s);
    else if (quant == MOE_NORM_FP8_BLOCK) e = launch_fwd<T, MOE_NORM_FP8_BLOCK>(a, bytes, s);
    else e = launch_fwd<T, MOE_NORM_MXFP8>(a, bytes, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T>
moe_status_t bwd(int rows, int H, const moe_norm_bwd_args_t& g, float* part, cudaStream_t s)
{
    BwdArgs<T> a{static_cast<const T*>(g.dy), static_cast<const T*>(g.h), g.rstd, g.weight,
                 static_cast<const T*>(g.dh), static_cast<T*>(g.dx), g.dweight ? part : nullptr,
                 g.lddy, g.ldh, g.lddh, g.lddx, rows, H};
    long long st[4];
    int n = 0;
    st[n++] = g.lddy;
    st[n++] = g.ldh;
    if (g.dh) st[n++] = g.lddh;
    st[n++] = g.lddx;
    const int bytes = access_bytes(H, (int)sizeof(T), st, n);
    const int parts = norm_parts(rows);
    if (rows > 0) {
        if (bytes == 16) norm_bwd_loop_kernel<T, 16 / (int)sizeof(T)><<<parts, kNormThreads, 0, s>>>(a);
        else if (bytes == 4) norm_bwd_loop_kernel<T, 4 / (int)sizeof(T)><<<parts, kNormThreads, 0, s>>>(a);
        else norm_bwd_loop_kernel<T, 1><<<parts, kNormThreads, 0, s>>>(a);
        count_launches();
    }
    if (g.dweight) {
        norm_dweight_kernel<<<(H + 31) / 32, 256, 0, s>>>(part, parts, H, g.dweight);
        count_launches();
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool act_dtype(int dtype) { return dtype == MOE_FP32 || dtype == MOE_BF16; }
constexpr int kNormMaxH = 1 << 20;

}  // namespace
}  // namespace moe

using namespace moe;

moe_status_t moe_add_rms_norm(int rows, int H, int dtype, int quant, float eps,
                              const moe_norm_fwd_args_t* args, moe_stream_t stream)
{
    if (!args || rows < 0 || H < 1 || H > kNormMaxH || !act_dtype(dtype) || quant < MOE_NORM_PLAIN ||
        quant > MOE_NORM_MXFP8 || !(eps >= 0.f) || eps - eps != 0.f)
        return MOE_ERR_INVALID_ARG;
    const moe_norm_fwd_args_t& g = *args;
    const bool q = quant != MOE_NORM_PLAIN;
    if (!g.weight || (q && H % 128)) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!g.x || (!q && !g.y) || (q && (!g.codes || !g.scales)))) return MOE_ERR_INVALID_ARG;
    if ((!q && (g.codes || g.scales)) || (g.h && !g.residual && rows > 0)) return MOE_ERR_INVALID_ARG;
    if (g.ldx < H || (g.residual && g.ldr < H) || (g.h && g.ldh < H) || (g.y && g.ldy < H))
        return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {g.x, g.residual, g.weight, g.h, g.y, g.rstd, g.codes, g.scales};
    for (const void* p : ptrs)
        if (!is_aligned16(p)) return MOE_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == MOE_FP32 ? fwd<float>(rows, H, quant, eps, g, s)
                             : fwd<__nv_bfloat16>(rows, H, quant, eps, g, s);
}

moe_status_t moe_norm_workspace_size(int rows, int H, size_t* ws_bytes)
{
    if (!ws_bytes || rows < 0 || H < 1 || H > kNormMaxH) return MOE_ERR_INVALID_ARG;
    *ws_bytes = (size_t)norm_parts(rows) * H * sizeof(float);
    return MOE_OK;
}

moe_status_t moe_add_rms_norm_backward(int rows, int H, int dtype, const moe_norm_bwd_args_t* args,
                                       void* ws, size_t ws_bytes, moe_stream_t stream)
{
    if (!args || rows < 0 || H < 1 || H > kNormMaxH || !act_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const moe_norm_bwd_args_t& g = *args;
    if (!g.weight || (rows > 0 && (!g.dy || !g.h || !g.rstd || !g.dx))) return MOE_ERR_INVALID_ARG;
    if (g.lddy < H || g.ldh < H || g.lddx < H || (g.dh && g.lddh < H)) return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {g.dy, g.h, g.rstd, g.weight, g.dh, g.dx, g.dweight, ws};
    for (const void* p : ptrs)
        if (!is_aligned16(p)) return MOE_ERR_MISALIGNED;
    if (g.dweight && rows > 0) {
        if (!ws) return MOE_ERR_INVALID_ARG;
        if (ws_bytes < (size_t)norm_parts(rows) * H * sizeof(float)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    float* part = static_cast<float*>(ws);
    return dtype == MOE_FP32 ? bwd<float>(rows, H, g, part, s) : bwd<__nv_bfloat16>(rows, H, g, part, s);
}
