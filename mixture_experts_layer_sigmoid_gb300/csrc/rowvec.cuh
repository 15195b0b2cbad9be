// rowvec.cuh -- loads and stores of row pieces for the operators around the
// layer (norm.cu, sort.cu, clip.cu): the 16 bytes of a piece, or one value, as one
// access, unpacked to fp32.
//
// Rows move in 16-byte pieces. Where rows do not start on 16-byte boundaries (or
// are not a whole number of pieces) they are cut at their boundaries, with a few
// edge columns that one lane each moves; sort.cu shifts sources that are cut
// elsewhere, norm.cu stages them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

namespace moe {

template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };
template <typename T, int V> using Raw = typename RawOf<V * (int)sizeof(T)>::type;

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& q, float (&v)[V])
{
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 4) {
            v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
            v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
        } else {
            v[0] = __uint_as_float(q);
        }
    } else if constexpr (V == 1) {
        v[0] = __uint_as_float((uint32_t)q << 16);
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// fp32 -> act, nearest even
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack(const float (&v)[V])
{
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 4)
            return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                              __float_as_uint(v[3]));
        else
            return __float_as_uint(v[0]);
    } else if constexpr (V == 1) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p)
{
    return *reinterpret_cast<const Raw<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, V>& q)
{
    *reinterpret_cast<Raw<T, V>*>(p) = q;
}
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V])
{
    unpack<T, V>(load_raw<T, V>(p), v);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V])
{
    store_raw<T, V>(p, pack<T, V>(v));
}

// Values of a piece.
template <typename T> constexpr int kPiece = 16 / (int)sizeof(T);

// How a row of H columns is cut at its own boundaries: whole pieces begin at
// columns head, head + V, ... (n of them), `edges` columns lie around them.
struct Cut { int head, n, edges; };
// Column of the e-th edge.
template <typename T>
__device__ __forceinline__ int edge_column(const Cut& c, int e) { return e < c.head ? e : e + c.n * kPiece<T>; }

// Element-wise fp32 operations on a piece, two values to an instruction.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
// v *= w
template <int V>
__device__ __forceinline__ void mul_vec(float (&v)[V], const float (&w)[V])
{
    if constexpr (V == 1) {
        v[0] *= w[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            uint64_t d;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(v[i], v[i + 1])), "l"(pair(w[i], w[i + 1])));
            unpair(d, v[i], v[i + 1]);
        }
    }
}
// v *= s
template <int V>
__device__ __forceinline__ void scale_vec(float (&v)[V], float s)
{
    float w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = s;
    mul_vec(v, w);
}
// v /= s, by the reciprocal r of s rounded to nearest and one correction of the
// product by its remainder (P. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990): within an
// ulp of the quotient and nearly always equal to it. The remainder must not
// underflow. The quotient is formed with the other sign, which keeps a zero's:
// v = -0 gives the remainder +0, and -0 + 0 would be +0.
template <int V>
__device__ __forceinline__ void divide_vec(float (&v)[V], float s, float r)
{
    static_assert(V % 2 == 0, "pairs");
    const uint64_t nr = pair(-r, -r), ss = pair(s, s);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const uint64_t x = pair(v[i], v[i + 1]);
        uint64_t y, e;
        float a, b;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(x), "l"(nr));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(ss), "l"(y), "l"(x));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(e), "l"(nr), "l"(y));
        unpair(y, a, b);
        v[i] = -a;
        v[i + 1] = -b;
    }
}
// v += u
template <int V>
__device__ __forceinline__ void add_vec(float (&v)[V], const float (&u)[V])
{
    if constexpr (V == 1) {
        v[0] += u[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            uint64_t d;
            asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(v[i], v[i + 1])), "l"(pair(u[i], u[i + 1])));
            unpair(d, v[i], v[i + 1]);
        }
    }
}
// (s0, s1) += sums of v^2 over the even and the odd values
template <int V>
__device__ __forceinline__ void add_squares(const float (&v)[V], float& s0, float& s1)
{
    if constexpr (V == 1) {
        s0 = fmaf(v[0], v[0], s0);
    } else {
        uint64_t s = pair(s0, s1);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const uint64_t p = pair(v[i], v[i + 1]);
            asm("fma.rn.f32x2 %0, %1, %1, %0;" : "+l"(s) : "l"(p));
        }
        unpair(s, s0, s1);
    }
}
// largest magnitude
template <int V>
__device__ __forceinline__ float max_abs(const float (&v)[V])
{
    float a = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i + 1 < V; i += 2) asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(v[i]), "f"(v[i + 1]));
    if constexpr (V % 2 == 0) a = fmaxf(a, fabsf(v[V - 1]));
    return a;
}

// V consecutive fp32 values that start on a V-value boundary of an aligned array
template <int V>
__device__ __forceinline__ void load_f32(const float* p, float (&v)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 q = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
        }
    } else {
        v[0] = p[0];
    }
}
template <int V>
__device__ __forceinline__ void store_f32(float* p, const float (&v)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        p[0] = v[0];
    }
}
// V fp32 values from column c on of an aligned array of H, c on no boundary: the
// aligned quads around them, shifted (by the same amount along a row).
template <int V>
__device__ __forceinline__ void load_f32_at(const float* p, int c, int H, float (&v)[V])
{
    const int sh = c & 3, a = c - sh;
    float w[V + 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(p + a + 4 * i);
        w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
    }
#pragma unroll
    for (int i = V; i < V + 4; ++i) w[i] = 0.f;
    if (a + V + 4 <= H) {
        const float4 q = *reinterpret_cast<const float4*>(p + a + V);
        w[V] = q.x; w[V + 1] = q.y; w[V + 2] = q.z;
    } else {
#pragma unroll
        for (int i = V; i < V + 3; ++i)
            if (a + i < H) w[i] = p[a + i];
    }
#pragma unroll
    for (int i = 0; i < V + 2; ++i) w[i] = sh & 1 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = sh & 2 ? w[i + 2] : w[i];
}

// How rows of H values of T with these strides (every base pointer 16-byte
// aligned) start: all on 16-byte boundaries and whole pieces; all equally far off
// them, row by row; or each tensor in its own way.
enum class Rows { kWhole, kAlike, kOwn };
template <typename T>
Rows rows_start(int H, std::initializer_list<long long> strides)
{
    bool whole = H % kPiece<T> == 0, alike = true;
    for (long long ld : strides) {
        whole = whole && ld % kPiece<T> == 0;
        alike = alike && (ld - *strides.begin()) % kPiece<T> == 0;
    }
    return whole ? Rows::kWhole : (alike ? Rows::kAlike : Rows::kOwn);
}

// Launches a kernel that begins with griddep_wait: its blocks may be set up
// while the kernel before it on the stream still runs.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args)
{
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace moe
