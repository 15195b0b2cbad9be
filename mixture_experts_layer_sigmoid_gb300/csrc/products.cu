// products.cu -- C ABI of the products over rows sorted by expert (moe.h): the
// checks of their arguments, and the codes of activation rows.
//
// Row codes: a thread holds sixteen consecutive values (32 or 64 bytes in, 16 out), eight
// neighbours share a block of 128 and its largest magnitude. Bound by HBM, with the
// instructions close behind: with eight values a thread, the block's division and shuffles
// came twice as often (139264 rows of 4096 bf16 349 us; 278 now). More pieces of a thread in
// flight cost blocks of an SM: two 311 us, four 475; 8 waves of blocks instead of 16 315.
#include "grouped_tc.cuh"
#include "mx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256, kPer = 16;
// Scales from which the corrected product's codes are those of a division (norm.cu has
// the reason, and the test that walks the pairs).
constexpr float kRowQuotientMin = 0x1p-92f;

// n / d for n below 2^31, as a product: floor(n m / 2^(32 + s)), m = ceil(2^(32 + s) / d),
// 2^s >= d / 2 (T. Granlund and P. L. Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994).
struct Divider {
    unsigned m, s, d;
    explicit Divider(unsigned d_) : s(0), d(d_)
    {
        while ((1ull << (s + 1)) < d) ++s;
        m = (unsigned)(((1ull << (32 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ unsigned operator()(unsigned n) const { return d == 1 ? n : __umulhi(n, m) >> s; }
};

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[kPer])
{
    constexpr int V = kPiece<T>;
#pragma unroll
    for (int i = 0; i < kPer / V; ++i) {
        float u[V];
        load_vec<T, V>(p + i * V, u);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i * V + j] = u[j];
    }
}

template <typename T>
__global__ void __launch_bounds__(kQThreads)
quantize_rows_kernel(const T* __restrict__ x, long long ldx, uint8_t* codes, long long ldc, float* scales, long long lds,
                     unsigned rows, Divider per_row, long long row0, const int* in_use)
{
    if (in_use) {
        const long long n = (long long)*in_use - row0;
        rows = n < 0 ? 0u : (unsigned)(n < (long long)rows ? n : (long long)rows);
    }
    const unsigned total = rows * per_row.d;               // below 2^31: the host cuts the rows
    for (unsigned at = blockIdx.x * kQThreads + threadIdx.x; at - threadIdx.x < total; at += gridDim.x * kQThreads) {
        const unsigned r = per_row(at), c = (at - r * per_row.d) * kPer;
        float v[kPer];
        if (at < total) {
            load16(x + (long long)r * ldx + c, v);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] = 0.f;
        }
        float a = max_abs(v);
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        if (at >= total) continue;                         // the eight lanes of a block alike
        const float t = __fdiv_rn(a, 448.f);
        const float s = t == 0.f ? 1.f : t;
        if (s >= kRowQuotientMin && s < 0x1p100f) {
            divide_vec(v, s, __frcp_rn(s));
        } else {                                           // the remainder could underflow
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] = __fdiv_rn(v[j], s);
        }
        if (c % 128 == 0) scales[(long long)r * lds + c / 128] = s;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = e4m3x4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        *reinterpret_cast<uint4*>(codes + (long long)r * ldc + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename T>
cudaError_t quantize_rows(long long rows, int K, const void* x, long long ldx, uint8_t* codes, long long ldc,
                          float* scales, long long lds, const int* in_use, int num_sms, cudaStream_t s)
{
    const Divider per_row((unsigned)K / kPer);
    const long long slab = (1ll << 30) / per_row.d;        // rows whose pieces 32 bits count
    for (long long r = 0; r < rows; r += slab) {
        const long long n = rows - r < slab ? rows - r : slab;
        const long long blocks = (n * per_row.d + kQThreads - 1) / kQThreads;
        const unsigned grid = (unsigned)(blocks < num_sms * 16ll ? blocks : num_sms * 16ll);
        quantize_rows_kernel<T><<<grid, kQThreads, 0, s>>>(static_cast<const T*>(x) + r * ldx, ldx, codes + r * ldc, ldc,
                                                           scales + r * lds, lds, (unsigned)n, per_row, r, in_use);
        count_launches();
    }
    return cudaGetLastError();
}

constexpr int kMaxWidth = 1 << 20;
constexpr long long kMaxStride = 1ll << 40;

bool width_ok(int n) { return n >= 1 && n <= kMaxWidth; }
// Row stride of `rows` rows of n values.
bool stride_ok(long long ld, int n) { return ld >= n && ld <= kMaxStride; }
// Stride between E matrices of n_out rows of n_in values.
bool block_ok(long long stride, int E, int n_out, long long ld, int n_in)
{
    return E == 1 || (stride >= (n_out - 1) * ld + n_in && stride <= kMaxStride);
}

// The segments of a call; a status other than MOE_OK refuses it.
moe_status_t check_groups(const moe_groups_t* in, Groups* g)
{
    if (!in || in->E < 1 || in->E > kMaxGroups || (in->dtype != MOE_FP32 && in->dtype != MOE_BF16) || in->rows < 0 ||
        in->rows > kMaxRows || (!in->offsets && (in->E != 1 || in->counts)))
        return MOE_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(in->offsets) | reinterpret_cast<uintptr_t>(in->counts)) & 3u)
        return MOE_ERR_MISALIGNED;
    *g = Groups{in->E, (int)in->rows, in->offsets, in->counts};
    return MOE_OK;
}

bool current_sms(int* n)
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
           cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

moe_status_t done(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace
}  // namespace moe

using namespace moe;

moe_status_t moe_grouped_matmul(const moe_groups_t* groups, int K, int N, const void* X, long long ldx, const void* W,
                                long long ldw, long long sw, int w_nk, void* Y, long long ldy, moe_stream_t stream)
{
    GroupedRows p{};
    const moe_status_t st = check_groups(groups, &p.g);
    if (st != MOE_OK) return st;
    if (!width_ok(K) || !width_ok(N) || w_nk < 0 || w_nk > 1 || (groups->rows > 0 && (!X || !W || !Y)) ||
        !stride_ok(ldx, K) || !stride_ok(ldy, N) || !stride_ok(ldw, w_nk ? K : N) ||
        !block_ok(sw, groups->E, w_nk ? N : K, ldw, w_nk ? K : N))
        return MOE_ERR_INVALID_ARG;
    if (!is_aligned16(X) || !is_aligned16(W) || !is_aligned16(Y)) return MOE_ERR_MISALIGNED;
    if (groups->rows == 0) return MOE_OK;
    if (Y == X || Y == W) return MOE_ERR_INVALID_ARG;
    p.K = K; p.N = N;
    p.X = X; p.ldx = ldx;
    p.W = W; p.ldw = ldw; p.sw = groups->E > 1 ? sw : 0; p.w_nk = w_nk;
    p.Y = Y; p.ldy = ldy;
    int sms = 0;
    if (!current_sms(&sms)) return MOE_ERR_CUDA;
    count_launches();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return done(groups->dtype == MOE_FP32 ? launch_grouped_rows_simt(p, sms, s) : launch_grouped_rows_tc(p, sms, s));
}

moe_status_t moe_grouped_wgrad(const moe_groups_t* groups, int M, int N, const void* A, long long lda, const void* B,
                               long long ldb, void* D, long long ldd, long long sd, moe_stream_t stream)
{
    GroupedWgrad p{};
    const moe_status_t st = check_groups(groups, &p.g);
    if (st != MOE_OK) return st;
    if (!width_ok(M) || !width_ok(N) || !D || (groups->rows > 0 && (!A || !B)) || !stride_ok(lda, M) ||
        !stride_ok(ldb, N) || !stride_ok(ldd, N) || !block_ok(sd, groups->E, M, ldd, N))
        return MOE_ERR_INVALID_ARG;
    if (!is_aligned16(A) || !is_aligned16(B) || !is_aligned16(D)) return MOE_ERR_MISALIGNED;
    if (D == A || D == B) return MOE_ERR_INVALID_ARG;
    p.M = M; p.N = N;
    p.A = A; p.lda = lda;
    p.B = B; p.ldb = ldb;
    p.D = D; p.ldd = ldd; p.sd = groups->E > 1 ? sd : 0;
    int sms = 0;
    if (!current_sms(&sms)) return MOE_ERR_CUDA;
    count_launches();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return done(groups->dtype == MOE_FP32 ? launch_grouped_wgrad_simt(p, sms, s) : launch_grouped_wgrad_tc(p, sms, s));
}

moe_status_t moe_fp8_matmul(const moe_groups_t* groups, int K, int N, const moe_fp8_matmul_args_t* args,
                            moe_stream_t stream)
{
    Fp8Rows p{};
    const moe_status_t st = check_groups(groups, &p.g);
    if (st != MOE_OK) return st;
    if (!args || !width_ok(K) || K % 128 || !width_ok(N)) return MOE_ERR_INVALID_ARG;
    const moe_fp8_matmul_args_t& a = *args;
    const int nk = a.b_nk, kb = K / 128, nb = (N + 127) / 128;
    if (nk < 0 || nk > 1 || (groups->rows > 0 && (!a.A || !a.SA || !a.B || !a.SB || !a.Y)) || !stride_ok(a.lda, K) ||
        !stride_ok(a.ldsa, kb) || !stride_ok(a.ldy, N) || !stride_ok(a.ldb, nk ? K : N) ||
        !stride_ok(a.ldsb, nk ? kb : nb) || !block_ok(a.sb, groups->E, nk ? N : K, a.ldb, nk ? K : N) ||
        !block_ok(a.ssb, groups->E, nk ? nb : kb, a.ldsb, nk ? kb : nb))
        return MOE_ERR_INVALID_ARG;
    if (!is_aligned16(a.A) || !is_aligned16(a.SA) || !is_aligned16(a.B) || !is_aligned16(a.SB) || !is_aligned16(a.Y) ||
        a.lda % 16 || a.ldb % 16 || (groups->E > 1 && a.sb % 16))
        return MOE_ERR_MISALIGNED;
    if (groups->rows == 0) return MOE_OK;
    if (a.Y == a.A || a.Y == a.SA || a.Y == a.B || a.Y == a.SB) return MOE_ERR_INVALID_ARG;
    p.K = K; p.N = N; p.dtype = groups->dtype;
    p.a = a;
    if (groups->E == 1) p.a.sb = p.a.ssb = 0;
    int sms = 0;
    if (!current_sms(&sms)) return MOE_ERR_CUDA;
    count_launches();
    return done(launch_fp8_rows(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_quantize_rows(long long rows, int K, int dtype, const void* x, long long ldx, uint8_t* codes,
                               long long ldc, float* scales, long long lds, const int32_t* in_use, moe_stream_t stream)
{
    if (rows < 0 || rows >= (1ll << 31) - 1 || !width_ok(K) || K % 128 || (dtype != MOE_FP32 && dtype != MOE_BF16) ||
        (rows > 0 && (!x || !codes || !scales)) || !stride_ok(ldx, K) || !stride_ok(ldc, K) || !stride_ok(lds, K / 128))
        return MOE_ERR_INVALID_ARG;
    const int per = dtype == MOE_FP32 ? 4 : 8;
    if (!is_aligned16(x) || !is_aligned16(codes) || !is_aligned16(scales) || ldx % per || ldc % 16 ||
        (reinterpret_cast<uintptr_t>(in_use) & 3u))
        return MOE_ERR_MISALIGNED;
    if (rows == 0) return MOE_OK;
    if (codes == x || static_cast<const void*>(scales) == x || reinterpret_cast<uint8_t*>(scales) == codes) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (!current_sms(&sms)) return MOE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return done(dtype == MOE_FP32 ? quantize_rows<float>(rows, K, x, ldx, codes, ldc, scales, lds, in_use, sms, s)
                                  : quantize_rows<__nv_bfloat16>(rows, K, x, ldx, codes, ldc, scales, lds, in_use, sms, s));
}

moe_status_t moe_products_status(moe_stream_t stream)
{
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int code = 0;
    for (auto take : {take_rows_status, take_wgrad_status, take_fp8_status})
        if (take(&code, s) != cudaSuccess) return MOE_ERR_CUDA;
    return code ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

moe_status_t moe_diag_products_wait(int which, moe_stream_t stream)
{
    if (which < 0 || which > 2) return MOE_ERR_INVALID_ARG;
    cudaError_t (*const stall[])(cudaStream_t) = {stall_rows, stall_wgrad, stall_fp8};
    count_launches();
    return done(stall[which](reinterpret_cast<cudaStream_t>(stream)));
}
