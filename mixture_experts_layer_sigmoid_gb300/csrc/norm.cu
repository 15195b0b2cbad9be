// norm.cu -- residual addition and root-mean-square norm, forward (act or
// 8-bit output) and backward, for the layer's pre-norm.
//
//   s = x + r,  rstd = (mean(s^2) + eps)^(-1/2),  y = s rstd w
//   n = h rstd, c = mean(w dy n):  dx = rstd (w dy - n c) + dh,
//                                  dw = sum over rows of dy n
//
// About ten operations per value against 2 to 16 bytes moved: every kernel
// here is bound by HBM (large inputs), by latency (a few rows), or, where only
// codes are written or rows start off the 16-byte boundaries, by instruction
// issue. Rates below are of the measured copy rate, 6.79 TB/s.
//
// Roundings: sums, means, rstd, the weight and its gradient are fp32; y is
// rounded once from fp32, h once from the fp32 sum, dx once; the 8-bit codes are
// taken from the fp32 y, not from its bf16 rounding, which would add 2^-9 to a
// code's error and flip about one in thirty.
#include "internal.h"
#include "mx.cuh"
#include "ptx.cuh"
#include "rowvec.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kNormThreads = 256;
// Row groups of the weight gradient's partial sums (blocks of the backward): two per
// SM where a block's ring leaves room for another, else half as many (Ring::kParts).
constexpr int kNormParts = 304;
// Up to one row per SM the forward gives a row more threads: 8 rows of 7168 bf16
// take 2.6 us with a thread per eight values and 3.1 with one per 32 (to blockwise
// codes 3.0 and 4.4).
constexpr int kFewRows = 152;

// Sum of v over the block's threads (at most NT; NT = 32: the warp's), the same
// order on every call; `red` holds NT / 32 floats and may be reused after the
// next __syncthreads.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (NT == 32) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = lane < (int)blockDim.x / 32 ? red[lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}

// m^(-1/2) with one correction of the approximate root by its residual 1 - m r^2
// (Newton's iteration, the residual formed with fused multiply-adds): rstd enters
// every value of its row, so its last bit is worth five instructions a row.
__device__ __forceinline__ float inv_root(float m)
{
    const float r = rsqrtf(m);
    if (!(r > 0.f && r < __int_as_float(0x7F800000))) return r;      // 0, infinite or NaN
    const float p = m * r;
    const float e = fmaf(-fmaf(m, r, -p), r, fmaf(-p, r, 1.f));
    return fmaf(0.5f * e, r, r);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// 16 bytes of which the first n come from src, the rest zeros
__device__ __forceinline__ void copy_async_part(void* dst, const void* src, int n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// Rows staged whole in shared memory, for rows that are too wide for registers
// or start each tensor in its own way (WINDOW: the 16-byte windows that cover the
// row are copied, so any alignment moves in full accesses; values are then taken
// one at a time at the row's place inside them).
template <typename T, bool WINDOW>
struct Staged {
    static constexpr int V = WINDOW ? 1 : 16 / (int)sizeof(T);
    // bytes of one staged row
    __host__ __device__ static int row_bytes(int H) { return (H * (int)sizeof(T) + (WINDOW ? 30 : 0)) / 16 * 16; }
    static __device__ __forceinline__ int phase(const T* p) { return WINDOW ? (int)(reinterpret_cast<uintptr_t>(p) & 15) : 0; }
    // this thread's part of the copy of a row (tid of NT threads)
    template <int NT>
    static __device__ __forceinline__ void fetch(unsigned char* dst, const T* p, int H, int tid)
    {
        const int ph = phase(p);
        const unsigned char* src = reinterpret_cast<const unsigned char*>(p) - ph;
        const int bytes = ph + H * (int)sizeof(T);
        for (int at = tid * 16; at < bytes; at += NT * 16) {
            if constexpr (WINDOW) copy_async_part(dst + at, src + at, bytes - at < 16 ? bytes - at : 16);
            else copy_async<16>(dst + at, src + at);
        }
    }
    // the V values at `at` bytes from buf
    static __device__ __forceinline__ void get(const unsigned char* buf, int at, float (&v)[V])
    {
        unpack<T, V>(*reinterpret_cast<const Raw<T, V>*>(buf + at), v);
    }
};

// The cut of row `row` of tensors whose rows start alike.
template <typename T>
__device__ __forceinline__ Cut cut_alike(const T* row, int H)
{
    constexpr int V = kPiece<T>;
    const int below = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    Cut c;
    c.head = below ? V - below : 0;
    if (c.head > H) c.head = H;
    c.n = (H - c.head) / V;
    c.edges = H - c.n * V;
    return c;
}

template <typename T> struct FwdArgs {
    const T* x; const T* r; const float* w;
    T* h; T* y; float* rstd; uint8_t* codes; void* scales;
    long long ldx, ldr, ldh, ldy;
    int rows, H; float eps;
};

// Scales from which divide_vec's codes are those of a division: the remainder v - s y
// has to keep the bits down to one step of s times one of y, 2^-23 s 2^-34 where y
// rounds to a code but zero (y >= 2^-11), and fp32 ends at 2^-149.
// tests/e4m3_quotient_fp32_check.c finds no difference from here on; from 2^-112,
// where bf16 values still show none, fp32 values of small blocks took wrong codes.
constexpr float kQuotientMin = 0x1p-92f;

// The 8-bit output of one piece of V values at column c of a row. All lanes
// of a warp call it together; `act` is false past the row's end, and the
// lanes of one block are all active or all inactive (H is a multiple of 128).
template <int QUANT, int V>
__device__ __forceinline__ void quantise(const float (&v)[V], bool act, int row, int c, int H,
                                         uint8_t* codes, void* scales)
{
    constexpr int BLOCK = QUANT == MOE_NORM_MXFP8 ? 32 : 128;
    float a = max_abs(v);
#pragma unroll
    for (int off = BLOCK / V / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    if (!act) return;
    float q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = v[i];
    if constexpr (QUANT == MOE_NORM_MXFP8) {
        const int e = mx_exp(a);
        scale_vec(q, mx_inv(e));                         // a power of two: exact
        if (c % BLOCK == 0)
            static_cast<uint8_t*>(scales)[((size_t)(row >> 7) * (H / 128) + c / 128) * 512 +
                                          atom_byte(row & 127, (c / 32) & 3)] = (uint8_t)(e + 127);
    } else {
        const float t = __fdiv_rn(a, 448.f);
        const float s = t == 0.f ? 1.f : t;              // zero, or too small for a scale
        if (s >= kQuotientMin && s < 0x1p100f) {
            // a division per value took half of the kernel's time; the bare product with
            // the reciprocal moved some codes next to ties
            divide_vec(q, s, __frcp_rn(s));
        } else {                                         // the remainder could underflow
#pragma unroll
            for (int i = 0; i < V; ++i) q[i] = __fdiv_rn(v[i], s);
        }
        if (c % BLOCK == 0) static_cast<float*>(scales)[(size_t)row * (H / 128) + c / 128] = s;
    }
    uint32_t* out = reinterpret_cast<uint32_t*>(codes + (size_t)row * H + c);
    if constexpr (V == 8)
        *reinterpret_cast<uint2*>(out) = make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
    else if constexpr (V == 4)
        *out = e4m3x4(q[0], q[1], q[2], q[3]);
}

// The scale bytes of a row past the last one in the last 128-row tile (those
// rows' groups run beside the others).
__device__ __forceinline__ void zero_scale_row(uint8_t* scales, long long row, int rows, int tid, int step, int H)
{
    if (row >= ((long long)rows + 127) / 128 * 128) return;
    for (int kb = tid; kb < H / 128; kb += step)
        *reinterpret_cast<uint32_t*>(scales + ((size_t)(row >> 7) * (H / 128) + kb) * 512 +
                                     atom_byte(row & 127, 0)) = 0u;
}

// One block per row, any width: the row is read twice (the second time from
// L2); h and y may overwrite x or the residual, since a thread writes only what
// it has read for the last time. For rows whose two stages do not fit shared
// memory; on 8192 x 7168 it takes 75.9 us where the held kernel takes 70.7.
template <typename T, int V, int QUANT>
__global__ void __launch_bounds__(kNormThreads)
norm_fwd_loop_kernel(FwdArgs<T> a)
{
    __shared__ float red[kNormThreads / 32];
    const int row = blockIdx.x;
    if (QUANT == MOE_NORM_MXFP8 && row >= a.rows) {
        zero_scale_row(static_cast<uint8_t*>(a.scales), row, a.rows, threadIdx.x, kNormThreads, a.H);
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
    const float rstd = inv_root(block_sum<kNormThreads>(ss, red) / (float)a.H + a.eps);
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

// One row per group (GROUP = 32: a warp; else the block, of at most GROUP
// threads), held in registers between the sum and the output: each value is
// read once. N pieces of V values per thread cover the row.
// 8192 x 7168 bf16 with residual: 70.5 us, 98%; 16384 x 4096 to MXFP8 codes and
// bf16: 89.8 us, 99%. At 48 registers five blocks of 224 threads fit an SM, and
// their loads cover one another's sums.
// AHEAD fetches the weights with the row, for launches of few rows, whose time
// is the chain of loads.
// SHIFT: rows start alike off the 16-byte boundaries. They are cut there; the
// weights are shifted into place and thread e < 2 V holds the e-th edge column.
// 4308 x 5259 bf16 (odd rows): 20.5 us, 65%, with residual 30.3 us, 88%.
template <typename T, bool SHIFT, int N, int GROUP, int QUANT, bool AHEAD = false>
__global__ void __launch_bounds__(GROUP == 32 ? kNormThreads : GROUP)
norm_fwd_kernel(FwdArgs<T> a)
{
    constexpr int V = kPiece<T>;
    constexpr int NT = GROUP == 32 ? kNormThreads : GROUP;
    __shared__ float red[NT / 32];
    const int tid = GROUP == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int step = GROUP == 32 ? 32 : blockDim.x;
    const long long row = GROUP == 32 ? (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.rows) {                     // whole groups leave together
        if constexpr (QUANT == MOE_NORM_MXFP8)
            zero_scale_row(static_cast<uint8_t*>(a.scales), row, a.rows, tid, step, a.H);
        return;
    }
    const T* x = a.x + row * a.ldx;
    const T* r = a.r ? a.r + row * a.ldr : nullptr;
    Cut cut{0, a.H / V, 0};
    if constexpr (SHIFT) cut = cut_alike(x, a.H);
    const bool edge = SHIFT && tid < cut.edges;
    const int ec = SHIFT ? edge_column<T>(cut, tid) : 0;
    auto load_w = [&](int c, float (&w)[V]) {
        if constexpr (SHIFT) load_f32_at<V>(a.w, c, a.H, w);
        else load_f32<V>(a.w + c, w);
    };
    Raw<T, V> qx[N], qr[N];                  // zeros past the row's end
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int p = tid + i * step, c = cut.head + p * V;
        qx[i] = Raw<T, V>{};
        qr[i] = Raw<T, V>{};
        if (p < cut.n) {
            qx[i] = load_raw<T, V>(x + c);
            if (r) qr[i] = load_raw<T, V>(r + c);
        }
    }
    float ev[1] = {0.f}, eu[1] = {0.f};
    if (edge) {
        load_vec<T, 1>(x + ec, ev);
        if (r) load_vec<T, 1>(r + ec, eu);
        ev[0] += eu[0];
    }
    float wa[AHEAD ? N : 1][V];
    if constexpr (AHEAD) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (tid + i * step < cut.n) load_w(cut.head + (tid + i * step) * V, wa[i]);
    }
    float v[N][V];
    float s0 = ev[0] * ev[0], s1 = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        unpack<T, V>(qx[i], v[i]);
        if (r) {
            float u[V];
            unpack<T, V>(qr[i], u);
            add_vec(v[i], u);
        }
        add_squares(v[i], s0, s1);
    }
    const float rstd = inv_root(block_sum<GROUP>(s0 + s1, red) / (float)a.H + a.eps);
    if (tid == 0 && a.rstd) a.rstd[row] = rstd;
    if (edge) {
        if (a.h) store_vec<T, 1>(a.h + row * a.ldh + ec, ev);
        ev[0] = ev[0] * rstd * a.w[ec];
        if (a.y) store_vec<T, 1>(a.y + row * a.ldy + ec, ev);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int p = tid + i * step, c = cut.head + p * V;
        const bool act = p < cut.n;
        if (act) {
            float w[V];
            if (a.h) store_vec<T, V>(a.h + row * a.ldh + c, v[i]);
            if constexpr (!AHEAD) load_w(c, w);
            scale_vec(v[i], rstd);
            mul_vec(v[i], AHEAD ? wa[AHEAD ? i : 0] : w);
            if (a.y) store_vec<T, V>(a.y + row * a.ldy + c, v[i]);
        }
        if constexpr (QUANT != MOE_NORM_PLAIN) quantise<QUANT, V>(v[i], act, (int)row, c, a.H, a.codes, a.scales);
    }
}

// One row per block at a time, the next rows' x and residual on their way into
// a ring of S staged rows. Without WINDOW a thread reads back only what it
// copied itself, so the row's sum is the only barrier. With WINDOW 4308 x 5259
// bf16 takes 32.7 us, 41%, bound by issue at about 35 instructions per 32 values
// (77 us held in registers one value at a time, whose loads were the wait).
constexpr int kWideThreads = 512;
template <typename T, bool WINDOW, bool RES, int QUANT, int S>
__global__ void __launch_bounds__(kWideThreads, 3)
norm_fwd_ring_kernel(FwdArgs<T> a)
{
    using R = Staged<T, WINDOW>;
    constexpr int V = R::V;
    constexpr int U = WINDOW ? 4 : 2;        // pieces together; more would spill at three blocks an SM
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float red[2][kWideThreads / 32];
    const int tid = threadIdx.x;
    const int rb = R::row_bytes(a.H), sb = RES ? 2 * rb : rb;
    auto fetch = [&](int stage, long long row) {
        if (row < a.rows) {
            R::template fetch<kWideThreads>(ring + stage * sb, a.x + row * a.ldx, a.H, tid);
            if constexpr (RES) R::template fetch<kWideThreads>(ring + stage * sb + rb, a.r + row * a.ldr, a.H, tid);
        }
        copy_commit();
    };
    for (int s = 0; s < S; ++s) fetch(s, (long long)blockIdx.x + (long long)s * gridDim.x);
    int stage = 0, parity = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        copy_wait<S - 1>();
        if constexpr (WINDOW) __syncthreads();
        constexpr int SIZE = (int)sizeof(T);
        const unsigned char* bx = ring + stage * sb;
        bx += R::phase(a.x + row * a.ldx) + tid * (V * SIZE);
        const unsigned char* br = bx;
        if constexpr (RES) br = ring + stage * sb + rb + R::phase(a.r + row * a.ldr) + tid * (V * SIZE);
        // values of the thread's i-th piece
        auto value = [&](int i, float (&v)[V]) {
            R::get(bx, i * (kWideThreads * V * SIZE), v);
            if constexpr (RES) {
                float u[V];
                R::get(br, i * (kWideThreads * V * SIZE), u);
                add_vec(v, u);
            }
        };
        const int own = (a.H - tid * V + kWideThreads * V - 1) / (kWideThreads * V);   // pieces of this thread
        float s0 = 0.f, s1 = 0.f;
#pragma unroll U
        for (int i = 0; i < own; ++i) {
            float v[V];
            value(i, v);
            add_squares(v, s0, s1);
        }
        const float rstd = inv_root(block_sum<kWideThreads>(s0 + s1, red[parity]) / (float)a.H + a.eps);
        parity ^= 1;
        if (tid == 0 && a.rstd) a.rstd[row] = rstd;
        const float* w = a.w + tid * V;
        T* h = a.h ? a.h + row * a.ldh + tid * V : nullptr;
        T* y = a.y ? a.y + row * a.ldy + tid * V : nullptr;
        // 8-bit blocks are shared by lanes: every thread takes part in each step
        const int steps = QUANT == MOE_NORM_PLAIN ? own : (a.H + kWideThreads * V - 1) / (kWideThreads * V);
#pragma unroll U
        for (int i = 0; i < steps; ++i) {
            const int at = i * (kWideThreads * V);
            const bool act = QUANT == MOE_NORM_PLAIN || i < own;
            float v[V], wv[V];
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = 0.f;
            if (act) {
                value(i, v);
                if (RES && h) store_vec<T, V>(h + at, v);
                load_f32<V>(w + at, wv);
                scale_vec(v, rstd);
                mul_vec(v, wv);
                if (QUANT == MOE_NORM_PLAIN || y) store_vec<T, V>(y + at, v);
            }
            if constexpr (QUANT != MOE_NORM_PLAIN) quantise<QUANT, V>(v, act, (int)row, at + tid * V, a.H, a.codes, a.scales);
        }
        if constexpr (WINDOW) __syncthreads();          // the stage is read
        fetch(stage, row + (long long)S * gridDim.x);
        stage = stage + 1 == S ? 0 : stage + 1;
    }
    copy_wait<0>();
    if constexpr (QUANT == MOE_NORM_MXFP8)
        for (long long row = (long long)a.rows + blockIdx.x; row < ((long long)a.rows + 127) / 128 * 128; row += gridDim.x)
            zero_scale_row(static_cast<uint8_t*>(a.scales), row, a.rows, tid, kWideThreads, a.H);
}

template <typename T> struct BwdArgs {
    const T* dy; const T* h; const float* rstd; const float* w; const T* dh;
    T* dx; float* part;   // part: gridDim.x x H partial sums of dw, or null
    long long lddy, ldh, lddh, lddx;
    int rows, H;
};

// Block b takes rows b, b + gridDim.x, ...; each thread always holds the same
// columns, so it adds its rows' dy n into part[b] alone. For rows wider than the
// kernels below take: 4308 x 12000 fp32 174 us, 70% (305 us with 256 threads): each
// row is read twice, the second time from L2, and dw read and written for every row.
constexpr int kLoopThreads = 1024;
template <typename T, int V>
__global__ void __launch_bounds__(kLoopThreads)
norm_bwd_loop_kernel(BwdArgs<T> a)
{
    __shared__ float red[kLoopThreads / 32];
    float* part = a.part ? a.part + (size_t)blockIdx.x * a.H : nullptr;
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* dy = a.dy + (size_t)row * a.lddy;
        const T* h = a.h + (size_t)row * a.ldh;
        const T* dh = a.dh ? a.dh + (size_t)row * a.lddh : nullptr;
        T* dx = a.dx + (size_t)row * a.lddx;
        const float rstd = a.rstd[row];
        float d = 0.f;
        for (int c = threadIdx.x * V; c < a.H; c += kLoopThreads * V) {
            float g[V], v[V], w[V];
            load_vec<T, V>(dy + c, g);
            load_vec<T, V>(h + c, v);
            load_f32<V>(a.w + c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) d = fmaf(g[i] * w[i], v[i], d);
        }
        __syncthreads();                       // red of the previous row is read
        const float m = block_sum<kLoopThreads>(d, red) * rstd / (float)a.H;
        for (int c = threadIdx.x * V; c < a.H; c += kLoopThreads * V) {
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

// The same with rows streamed through shared memory: each thread copies its own
// pieces of dy, h and dh of the next rows into a ring of S stages (cp.async) and
// later reads back nothing but what it copied, so the ring needs no barrier and
// S rows per group are in flight while one is worked on. w and the partial sums
// of dw stay in registers over all rows of the thread.
// GROUP threads take a row (a warp, or the block); H <= GROUP * N * V.
// 8192 x 7168 bf16 with dh: 75.4 us with the sum of the parts, 92% (197 us when
// each row was loaded, summed and read again); bound by HBM, 71 us of it here.
// SHIFT: rows start alike off the 16-byte boundaries. The number of groups is a
// multiple of eight where a group has more than one row, so all of its rows are
// cut in the same columns; thread e < 2 V holds the e-th edge column, fetched one
// row ahead. 4308 x 5259 bf16: 39 us, 68%.
template <int N, int NT>
struct Ring {
    static constexpr int kTensor = NT * N * 16;              // one tensor's rows of one stage
    static constexpr int kStage = 3 * kTensor;
    // as many stages as fit beside a second block on the SM, at most 4, and two at least
    static constexpr int kStages = kStage * 4 <= 104 * 1024 ? 4 : (kStage * 3 <= 104 * 1024 ? 3 : 2);
    static constexpr int kBytes = kStages * kStage;
    // Blocks: those that are resident together, so that no ring is filled and no w read
    // for a second wave. With 192 KB (N = 4 of 512 threads, N = 8 of 256) that is one
    // per SM: 4000 x 16384 bf16 85.3 us, 88.2 with 304 blocks, 300 x 16384 14.4 and 18.5.
    static constexpr int kParts = kBytes <= 104 * 1024 ? kNormParts : kNormParts / 2;
    static_assert(kParts % 8 == 0, "see SHIFT");
};

template <typename T, bool SHIFT, int N, int GROUP, int NT>
__global__ void __launch_bounds__(NT, NT <= 256 ? 2 : 1)
norm_bwd_kernel(BwdArgs<T> a)
{
    constexpr int V = kPiece<T>;
    using R = Ring<N, NT>;
    constexpr int S = R::kStages;
    constexpr int GROUPS = NT / GROUP;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float red[2][NT / 32];
    __shared__ float rs[S][NT / 32];
    __shared__ int heads[NT / 32];
    const int tid = GROUP == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long first = GROUP == 32 ? (long long)blockIdx.x * GROUPS + warp : blockIdx.x;
    const long long step = (long long)gridDim.x * GROUPS;
    Cut cut{0, a.H / V, 0};
    if constexpr (SHIFT) cut = cut_alike(a.h + first * a.ldh, a.H);
    const bool edge = SHIFT && tid < cut.edges;
    const int ec = SHIFT ? edge_column<T>(cut, tid) : 0;

    auto slot = [&](int stage, int tensor, int i) {
        return reinterpret_cast<Raw<T, V>*>(ring + stage * R::kStage + tensor * R::kTensor) + i * NT + threadIdx.x;
    };
    auto fetch = [&](int stage, long long row) {
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = cut.head + (tid + i * GROUP) * V;
                if (tid + i * GROUP < cut.n) {
                    copy_async<16>(slot(stage, 0, i), a.dy + row * a.lddy + c);
                    copy_async<16>(slot(stage, 1, i), a.h + row * a.ldh + c);
                    if (a.dh) copy_async<16>(slot(stage, 2, i), a.dh + row * a.lddh + c);
                }
            }
            if (lane == 0) copy_async<4>(&rs[stage][warp], a.rstd + row);
        }
        copy_commit();
    };
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(s, first + s * step);

    // the edge column's dy, h and dh of the next row, as loaded: nothing waits for
    // them before that row's turn
    Raw<T, 1> ng = 0, nh = 0, nd = 0;
    float ew = 0.f, edw = 0.f;
    auto fetch_edge = [&](long long row) {
        if (edge && row < a.rows) {
            ng = load_raw<T, 1>(a.dy + row * a.lddy + ec);
            nh = load_raw<T, 1>(a.h + row * a.ldh + ec);
            if (a.dh) nd = load_raw<T, 1>(a.dh + row * a.lddh + ec);
        }
    };
    auto value = [](Raw<T, 1> q) {
        float v[1];
        unpack<T, 1>(q, v);
        return v[0];
    };
    if constexpr (SHIFT) {
        fetch_edge(first);
        if (edge) ew = a.w[ec];
    }
    float w[N][V], dw[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int p = tid + i * GROUP, c = cut.head + p * V;
#pragma unroll
        for (int j = 0; j < V; ++j) { w[i][j] = 0.f; dw[i][j] = 0.f; }
        if (p < cut.n) {
            if constexpr (SHIFT) {
#pragma unroll
                for (int j = 0; j < V; ++j) w[i][j] = a.w[c + j];      // all of them in flight together
            } else {
                load_f32<V>(a.w + c, w[i]);
            }
        }
    }
    ptx::griddep_launch_dependents();
    int stage = 0, parity = 0;
    for (long long row = first; row < a.rows; row += step) {
        const float eg = value(ng), eh = value(nh), ed = value(nd);
        if constexpr (SHIFT) fetch_edge(row + step);
        copy_wait<S - 1>();
        __syncwarp();
        const float rstd = rs[stage][warp];
        float d = eg * ew * eh;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (tid + i * GROUP >= cut.n) break;
            float g[V], v[V];
            unpack<T, V>(*slot(stage, 0, i), g);
            unpack<T, V>(*slot(stage, 1, i), v);
#pragma unroll
            for (int j = 0; j < V; ++j) d = fmaf(g[j] * w[i][j], v[j], d);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        if constexpr (GROUP != 32) {
            // one barrier a row: the sums alternate between two arrays
            if (lane == 0) red[parity][warp] = d;
            __syncthreads();
            d = 0.f;
#pragma unroll
            for (int k = 0; k < NT / 32; ++k) d += red[parity][k];
            parity ^= 1;
        }
        const float m = d * rstd / (float)a.H;
        T* dx = a.dx + row * a.lddx;
        if (edge) {
            const float n = eh * rstd;
            const float o[1] = {rstd * fmaf(-n, m, eg * ew) + ed};
            edw = fmaf(eg, n, edw);
            store_vec<T, 1>(dx + ec, o);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = cut.head + (tid + i * GROUP) * V;
            if (tid + i * GROUP >= cut.n) break;
            float g[V], v[V], o[V];
            unpack<T, V>(*slot(stage, 0, i), g);
            unpack<T, V>(*slot(stage, 1, i), v);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = v[j] * rstd;
                o[j] = rstd * fmaf(-n, m, g[j] * w[i][j]);
                dw[i][j] = fmaf(g[j], n, dw[i][j]);
            }
            if (a.dh) {
                float u[V];
                unpack<T, V>(*slot(stage, 2, i), u);
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] += u[j];
            }
            store_vec<T, V>(dx + c, o);
        }
        __syncwarp();                         // rs is read
        fetch(stage, row + S * step);
        stage = stage + 1 == S ? 0 : stage + 1;
    }
    copy_wait<0>();
    if (!a.part) return;
    float* part = a.part + (size_t)blockIdx.x * a.H;
    auto put_dw = [&](float* to) {
        if (edge) to[ec] = edw;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int p = tid + i * GROUP, c = cut.head + p * V;
            if (p >= cut.n) break;
            if constexpr (SHIFT) {
#pragma unroll
                for (int j = 0; j < V; ++j) to[c + j] = dw[i][j];
            } else {
                store_f32<V>(to + c, dw[i]);
            }
        }
    };
    if constexpr (GROUP == 32) {
        // the warps' sums, added in warp order
        constexpr int W = GROUP * N * V;                     // at least H
        static_assert(GROUPS * W * 4 <= R::kBytes, "the sums fit the ring");
        float* sum = reinterpret_cast<float*>(ring);
        __syncthreads();
        if constexpr (!SHIFT) {
            put_dw(sum + warp * W);
            __syncthreads();
            for (int c = threadIdx.x; c < a.H; c += NT) {
                float t = 0.f;
#pragma unroll
                for (int k = 0; k < GROUPS; ++k) t += sum[k * W + c];
                part[c] = t;
            }
        } else {
            // the warps' rows are cut in different columns. Value j of a lane's pieces
            // goes to row j of the warp's table, whose stride keeps both the lanes'
            // stores and the columns' reads on different banks; the edges behind it
            constexpr int L = GROUP * N + 32 / V;
            static_assert(GROUPS * (V * L + 32) * 4 <= R::kBytes, "the tables fit the ring");
            float* mine = sum + warp * (V * L + 32);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) mine[j * L + tid + i * GROUP] = dw[i][j];
            mine[V * L + tid] = edw;
            if (lane == 0) heads[warp] = cut.head;
            __syncthreads();
            for (int c = threadIdx.x; c < a.H; c += NT) {
                float t = 0.f;
#pragma unroll
                for (int k = 0; k < GROUPS; ++k) {
                    const int head = heads[k], n = (a.H - head) / V * V, at = c - head;
                    const float* table = sum + k * (V * L + 32);
                    t += at < 0 ? table[V * L + c] : (at < n ? table[at % V * L + at / V] : table[V * L + c - n]);
                }
                part[c] = t;
            }
        }
    } else {
        put_dw(part);
    }
}

// The same for rows that start each tensor in its own way, staged whole (as in
// the forward's ring); dw is summed in shared memory, each column by one thread.
// 4308 x 5259 bf16 takes 68 us, 39%, bound by issue, where the ring takes 40.
template <typename T, bool DH, int S>
__global__ void __launch_bounds__(kWideThreads)
norm_bwd_window_kernel(BwdArgs<T> a)
{
    using R = Staged<T, true>;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float red[2][kWideThreads / 32];
    const int tid = threadIdx.x;
    const int rb = R::row_bytes(a.H), sb = (DH ? 3 : 2) * rb;
    float* dw = reinterpret_cast<float*>(ring + S * sb);
    auto fetch = [&](int stage, long long row) {
        if (row < a.rows) {
            unsigned char* to = ring + stage * sb;
            R::template fetch<kWideThreads>(to, a.dy + row * a.lddy, a.H, tid);
            R::template fetch<kWideThreads>(to + rb, a.h + row * a.ldh, a.H, tid);
            if constexpr (DH) R::template fetch<kWideThreads>(to + 2 * rb, a.dh + row * a.lddh, a.H, tid);
        }
        copy_commit();
    };
    for (int s = 0; s < S; ++s) fetch(s, (long long)blockIdx.x + (long long)s * gridDim.x);
    for (int c = tid; c < a.H; c += kWideThreads) dw[c] = 0.f;
    ptx::griddep_launch_dependents();
    int stage = 0, parity = 0;
    float rstd = blockIdx.x < (unsigned)a.rows ? a.rstd[blockIdx.x] : 0.f;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float next = row + gridDim.x < a.rows ? a.rstd[row + gridDim.x] : 0.f;
        copy_wait<S - 1>();
        __syncthreads();
        constexpr int STEP = kWideThreads * (int)sizeof(T);
        const unsigned char* at = ring + stage * sb + tid * (int)sizeof(T);
        const unsigned char* bg = at + R::phase(a.dy + row * a.lddy);
        const unsigned char* bh = at + rb + R::phase(a.h + row * a.ldh);
        const unsigned char* bd = DH ? at + 2 * rb + R::phase(a.dh + row * a.lddh) : at;
        const float* w = a.w + tid;
        const int own = (a.H - tid + kWideThreads - 1) / kWideThreads;     // values of this thread
        float d = 0.f;
#pragma unroll 4
        for (int i = 0; i < own; ++i) {
            float g[1], v[1];
            R::get(bg, i * STEP, g);
            R::get(bh, i * STEP, v);
            d = fmaf(g[0] * w[i * kWideThreads], v[0], d);
        }
        const float m = block_sum<kWideThreads>(d, red[parity]) * rstd / (float)a.H;
        parity ^= 1;
        T* dx = a.dx + row * a.lddx + tid;
        float* dwt = dw + tid;
#pragma unroll 4
        for (int i = 0; i < own; ++i) {
            float g[1], v[1], o[1];
            R::get(bg, i * STEP, g);
            R::get(bh, i * STEP, v);
            const float n = v[0] * rstd;
            o[0] = rstd * fmaf(-n, m, g[0] * w[i * kWideThreads]);
            dwt[i * kWideThreads] = fmaf(g[0], n, dwt[i * kWideThreads]);
            if constexpr (DH) {
                float u[1];
                R::get(bd, i * STEP, u);
                o[0] += u[0];
            }
            store_vec<T, 1>(dx + i * kWideThreads, o);
        }
        __syncthreads();                                  // the stage is read
        fetch(stage, row + (long long)S * gridDim.x);
        stage = stage + 1 == S ? 0 : stage + 1;
        rstd = next;
    }
    copy_wait<0>();
    if (a.part)
        for (int c = tid; c < a.H; c += kWideThreads) a.part[(size_t)blockIdx.x * a.H + c] = dw[c];
}

// dw[c] = sum of the parts: ascending order within each of 32 phases, the
// phases then added in order. Launched ahead of the parts' kernel's end: about 3
// us for 304 parts of 7168, from L2.
constexpr int kPhases = 32;
__global__ void __launch_bounds__(32 * kPhases)
norm_dweight_kernel(const float* __restrict__ part, int nparts, int H, float* __restrict__ dw)
{
    __shared__ float red[kPhases][33];
    const int lane = threadIdx.x & 31, ph = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    constexpr int PER = (kNormParts + kPhases - 1) / kPhases;        // parts of a phase, all read together
    float v[PER], s = 0.f;
    ptx::griddep_wait();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = ph + i * kPhases;
        v[i] = c < H && b < nparts ? __ldcg(part + (size_t)b * H + c) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) s += v[i];
    red[ph][lane] = s;
    __syncthreads();
    if (ph == 0 && c < H) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kPhases; ++i) t += red[i][lane];
        dw[c] = t;
    }
}

int norm_parts(int rows) { return rows < kNormParts ? rows : kNormParts; }

// Shared memory of an SM's blocks together, and of one.
constexpr int kSmemAll = 224 * 1024, kSmemOne = 220 * 1024;
constexpr int kSms = 152;

// The forward's ring, up to three blocks on an SM (their registers allow no
// more): four stages a block where twelve rows fit, else two; false if two do
// not fit one block.
template <typename T, bool WINDOW, int QUANT>
bool launch_fwd_ring(const FwdArgs<T>& a, cudaStream_t s)
{
    const int stage = Staged<T, WINDOW>::row_bytes(a.H) * (a.r ? 2 : 1);
    auto launch = [&](auto kernel, int smem) {
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
        const int fit = kSmemAll / (smem + 1280);
        const int blocks = kSms * (fit < 1 ? 1 : (fit > 3 ? 3 : fit));
        kernel<<<a.rows < blocks ? a.rows : blocks, kWideThreads, smem, s>>>(a);
    };
    auto staged = [&](auto res) {
        constexpr bool RES = decltype(res)::value;
        if constexpr (WINDOW)                // other rows come here only when they are wider than that
            if (12 * stage + 3 * 1280 <= kSmemAll) {
                launch(norm_fwd_ring_kernel<T, WINDOW, RES, QUANT, 4>, 4 * stage);
                return true;
            }
        if (2 * stage > kSmemOne) return false;
        launch(norm_fwd_ring_kernel<T, WINDOW, RES, QUANT, 2>, 2 * stage);
        return true;
    };
    return a.r ? staged(std::true_type{}) : staged(std::false_type{});
}

// The held kernel with N pieces per thread and as many threads as that takes.
template <typename T, bool SHIFT, int N, int GROUP, int QUANT, bool AHEAD = false>
void launch_held(const FwdArgs<T>& a, int rows, cudaStream_t s)
{
    if constexpr (GROUP == 32) {
        norm_fwd_kernel<T, SHIFT, N, 32, QUANT><<<(rows + kNormThreads / 32 - 1) / (kNormThreads / 32), kNormThreads, 0, s>>>(a);
    } else {
        const int pieces = (a.H + kPiece<T> - 1) / kPiece<T>, threads = (pieces + N - 1) / N;
        norm_fwd_kernel<T, SHIFT, N, GROUP, QUANT, AHEAD><<<rows, (threads + 31) / 32 * 32, 0, s>>>(a);
    }
}

// Rows that start whole, or alike (SHIFT).
template <typename T, bool SHIFT, int QUANT>
void launch_fwd_cut(const FwdArgs<T>& a, cudaStream_t s)
{
    constexpr int P = 32 / kPiece<T>;        // pieces of 32 values
    const int rows = QUANT == MOE_NORM_MXFP8 ? (a.rows + 127) / 128 * 128 : a.rows;
    if (a.H <= 256) return launch_held<T, SHIFT, P / 4, 32, QUANT>(a, rows, s);
    if (a.H <= 512) return launch_held<T, SHIFT, P / 2, 32, QUANT>(a, rows, s);
    // few rows: a thread per eight values shortens each row's own chain
    if (a.H <= 8192 && a.rows <= kFewRows) return launch_held<T, SHIFT, P / 4, 1024, QUANT, true>(a, rows, s);
    // many rows to 8-bit codes are bound by issue: more pieces per thread share what
    // a warp does once (16384 x 2048 bf16 to MXFP8 codes 25.0 us, 30.8 with a thread
    // per eight values; 300 x 4096 3.1 us, 4.3 with one per 32)
    if constexpr (QUANT != MOE_NORM_PLAIN && sizeof(T) == 2)
        if (a.rows >= 8 * kSms && a.H <= 4096) {
            if (a.H <= 2048) return launch_held<T, SHIFT, P / 2, 256, QUANT>(a, rows, s);
            return launch_held<T, SHIFT, P, 256, QUANT>(a, rows, s);
        }
    if (a.H <= 1024) return launch_held<T, SHIFT, P / 4, 128, QUANT>(a, rows, s);
    if (a.H <= 2048) return launch_held<T, SHIFT, P / 4, 256, QUANT>(a, rows, s);
    if (a.H <= 4096) return launch_held<T, SHIFT, P / 2, 256, QUANT>(a, rows, s);
    if (a.H <= 8192) {
        if constexpr (sizeof(T) == 2) return launch_held<T, SHIFT, P, 256, QUANT>(a, rows, s);
        else return launch_held<T, SHIFT, P / 2, 512, QUANT>(a, rows, s);
    }
    // 4000 x 13568 bf16 with residual: 65.0 us, 67.2 with 512 threads, 69.5 in the ring;
    // 4000 x 16384 to blockwise codes: 79 us with 512 threads, 108 with 1024, 106 in the ring
    if (a.H <= 16384) {
        if constexpr (QUANT == MOE_NORM_PLAIN) return launch_held<T, SHIFT, P / 2, 1024, QUANT>(a, rows, s);
        else return launch_held<T, SHIFT, P, 512, QUANT>(a, rows, s);
    }
    if (launch_fwd_ring<T, SHIFT, QUANT>(a, s)) return;
    norm_fwd_loop_kernel<T, SHIFT ? 1 : kPiece<T>, QUANT><<<rows, kNormThreads, 0, s>>>(a);
}

template <typename T, int QUANT>
cudaError_t launch_fwd(const FwdArgs<T>& a, Rows start, cudaStream_t s)
{
    if (start == Rows::kWhole) {
        launch_fwd_cut<T, false, QUANT>(a, s);
    } else if constexpr (QUANT == MOE_NORM_PLAIN) {
        if (start == Rows::kAlike) launch_fwd_cut<T, true, QUANT>(a, s);
        else if (!launch_fwd_ring<T, true, QUANT>(a, s)) norm_fwd_loop_kernel<T, 1, QUANT><<<a.rows, kNormThreads, 0, s>>>(a);
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
    const Rows start = rows_start<T>(H, {g.ldx, g.residual ? g.ldr : g.ldx, g.h ? g.ldh : g.ldx, g.y ? g.ldy : g.ldx});
    if (quant != MOE_NORM_PLAIN && start != Rows::kWhole) return MOE_ERR_MISALIGNED;
    if (rows == 0) return MOE_OK;
    cudaError_t e;
    if (quant == MOE_NORM_PLAIN) e = launch_fwd<T, MOE_NORM_PLAIN>(a, start, s);
    else if (quant == MOE_NORM_FP8_BLOCK) e = launch_fwd<T, MOE_NORM_FP8_BLOCK>(a, start, s);
    else e = launch_fwd<T, MOE_NORM_MXFP8>(a, start, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Widths of which the backward gives a row to a warp: 32768 x 512 bf16 takes 26
// us with a warp and 54 with a block per row, 400 x 512 4.3 and 4.8 us.
constexpr int kWarpH = 1024;

// The blocks launched, each with its part of dw.
template <typename T, bool SHIFT, int N, int GROUP, int NT>
int launch_ring(const BwdArgs<T>& a, cudaStream_t s)
{
    using R = Ring<N, NT>;
    constexpr int rows = NT / GROUP;         // of a block at a time
    const int wanted = (a.rows + rows - 1) / rows, parts = wanted < R::kParts ? wanted : R::kParts;
    if (R::kBytes > 40 * 1024)
        cudaFuncSetAttribute(norm_bwd_kernel<T, SHIFT, N, GROUP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kBytes);
    norm_bwd_kernel<T, SHIFT, N, GROUP, NT><<<parts, NT, R::kBytes, s>>>(a);
    return parts;
}

// Rows that start whole, or alike (SHIFT); 0 for wider ones than the ring takes.
template <typename T, bool SHIFT>
int launch_bwd_cut(const BwdArgs<T>& a, cudaStream_t s)
{
    constexpr int P = 32 / kPiece<T>;        // pieces of 32 values
    if (a.H <= 256) return launch_ring<T, SHIFT, P / 4, 32, 256>(a, s);
    if (a.H <= kWarpH) return launch_ring<T, SHIFT, P, 32, 256>(a, s);
    if (a.H <= 2048) return launch_ring<T, SHIFT, P / 4, 256, 256>(a, s);
    if (a.H <= 4096) return launch_ring<T, SHIFT, P / 2, 256, 256>(a, s);
    if constexpr (sizeof(T) == 2) {
        if (a.H <= 8192) return launch_ring<T, SHIFT, P, 256, 256>(a, s);
        if (a.H <= 16384) return launch_ring<T, SHIFT, P, 512, 512>(a, s);
    } else {
        if (a.H <= 8192) return launch_ring<T, SHIFT, P / 2, 512, 512>(a, s);
    }
    return 0;
}

// Rows that start each in their own way, as far as two stages and dw fit shared memory.
template <typename T>
bool launch_bwd_window(const BwdArgs<T>& a, int parts, cudaStream_t s)
{
    const int smem = 2 * Staged<T, true>::row_bytes(a.H) * (a.dh ? 3 : 2) + a.H * (int)sizeof(float);
    if (smem > kSmemOne) return false;
    auto kernel = a.dh ? norm_bwd_window_kernel<T, true, 2> : norm_bwd_window_kernel<T, false, 2>;
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
    kernel<<<parts, kWideThreads, smem, s>>>(a);
    return true;
}

template <typename T>
moe_status_t bwd(int rows, int H, const moe_norm_bwd_args_t& g, float* part, cudaStream_t s)
{
    BwdArgs<T> a{static_cast<const T*>(g.dy), static_cast<const T*>(g.h), g.rstd, g.weight,
                 static_cast<const T*>(g.dh), static_cast<T*>(g.dx), g.dweight ? part : nullptr,
                 g.lddy, g.ldh, g.lddh, g.lddx, rows, H};
    const Rows start = rows_start<T>(H, {g.lddy, g.ldh, g.dh ? g.lddh : g.lddy, g.lddx});
    int parts = 0;
    if (rows > 0) {
        if (start == Rows::kWhole) parts = launch_bwd_cut<T, false>(a, s);
        else if (start == Rows::kAlike) parts = launch_bwd_cut<T, true>(a, s);
        if (parts == 0) {
            parts = norm_parts(rows);
            if (start == Rows::kWhole) norm_bwd_loop_kernel<T, kPiece<T>><<<parts, kLoopThreads, 0, s>>>(a);
            else if (!launch_bwd_window<T>(a, parts, s)) norm_bwd_loop_kernel<T, 1><<<parts, kLoopThreads, 0, s>>>(a);
        }
        count_launches();
    }
    if (g.dweight) {
        if (launch_early(norm_dweight_kernel, dim3((H + 31) / 32), dim3(32 * kPhases), s, (const float*)part, parts, H,
                         g.dweight) != cudaSuccess)
            return MOE_ERR_CUDA;
        count_launches();
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool act_dtype(int dtype) { return dtype == MOE_FP32 || dtype == MOE_BF16; }
constexpr int kNormMaxH = 1 << 20;
constexpr int kNormMaxRows = 0x7FFFFF00;     // rounded up to a tile of 128 it is still an int

}  // namespace
}  // namespace moe

using namespace moe;

moe_status_t moe_add_rms_norm(int rows, int H, int dtype, int quant, float eps,
                              const moe_norm_fwd_args_t* args, moe_stream_t stream)
{
    if (!args || rows < 0 || rows > kNormMaxRows || H < 1 || H > kNormMaxH || !act_dtype(dtype) || quant < MOE_NORM_PLAIN ||
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
    if (!ws_bytes || rows < 0 || rows > kNormMaxRows || H < 1 || H > kNormMaxH) return MOE_ERR_INVALID_ARG;
    *ws_bytes = (size_t)norm_parts(rows) * H * sizeof(float);
    return MOE_OK;
}

moe_status_t moe_add_rms_norm_backward(int rows, int H, int dtype, const moe_norm_bwd_args_t* args,
                                       void* ws, size_t ws_bytes, moe_stream_t stream)
{
    if (!args || rows < 0 || rows > kNormMaxRows || H < 1 || H > kNormMaxH || !act_dtype(dtype)) return MOE_ERR_INVALID_ARG;
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
