// matmul_fp8.cu -- products of E4M3 codes with a scale for each block of 128, rows
// grouped by expert or dense:
//   Y[r][n] = sum_kb SA[r][kb] SB[kb][n/128] sum_{k in block kb} A[r][k] B[k][n].
// A block of 256 threads owns 16 x 64 outputs, four to a thread.
#include "grouped.cuh"
#include "epilogue.cuh"
#include <cuda_fp8.h>

namespace moe {
namespace {

constexpr int TM = 16, TN = 64;

__device__ __forceinline__ float e4m3_value(uint8_t c)
{
    __nv_fp8_e4m3 q;
    q.__x = c;
    return (float)q;
}

template <typename T>
__global__ void __launch_bounds__(256)
fp8_rows_kernel(const Fp8Rows p)
{
    __shared__ float As[TM][129];
    __shared__ float Bs[128][TN + 1];
    __shared__ int pre[kMaxGroups + 1];
    count_row_tiles<TM>(p.g, pre);
    const moe_fp8_matmul_args_t& a = p.a;
    const int num_n = (p.N + TN - 1) / TN, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const long long total = (long long)pre[p.g.E] * num_n;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        const int q = (int)(w / num_n), n0 = (int)(w % num_n) * TN;
        const int e = segment_at(pre, p.g.E, q);
        const Segment s = segment_of(p.g, e);
        const int at = (q - pre[e]) * TM, row = s.begin + at, valid = s.valid - at;
        float acc[4] = {};
        if (valid > 0) {
            for (int kb = 0; kb < p.K / 128; ++kb) {
                __syncthreads();
                for (int i = threadIdx.x; i < TM * 128; i += 256)
                    As[i / 128][i % 128] = i / 128 < valid ? e4m3_value(a.A[(row + i / 128) * a.lda + kb * 128 + i % 128]) : 0.f;
                for (int i = threadIdx.x; i < TN * 128; i += 256) {
                    const int n = a.b_nk ? i / 128 : i % TN, k = a.b_nk ? i % 128 : i / TN;
                    const long long o = a.b_nk ? (n0 + n) * a.ldb + kb * 128 + k : (kb * 128 + k) * a.ldb + n0 + n;
                    Bs[k][n] = n0 + n < p.N ? e4m3_value(a.B[e * a.sb + o]) : 0.f;
                }
                __syncthreads();
                float part[4] = {};
                for (int k = 0; k < 128; ++k)
                    for (int j = 0; j < 4; ++j) part[j] = fmaf(As[ty][k], Bs[k][tx + 16 * j], part[j]);
                if (ty < valid) {
                    const int nb = n0 / 128;
                    const float sc = a.SA[(row + ty) * a.ldsa + kb] *
                                     a.SB[e * a.ssb + (a.b_nk ? nb * a.ldsb + kb : kb * a.ldsb + nb)];
                    for (int j = 0; j < 4; ++j) acc[j] = fmaf(part[j], sc, acc[j]);
                }
            }
        }
        if (row + ty < s.end)
            for (int j = 0; j < 4; ++j)
                if (n0 + tx + 16 * j < p.N)
                    static_cast<T*>(a.Y)[(row + ty) * a.ldy + n0 + tx + 16 * j] = from_f32<T>(ty < valid ? acc[j] : 0.f);
    }
}

}  // namespace

cudaError_t launch_fp8_rows(const Fp8Rows& p, int num_sms, cudaStream_t s)
{
    const long long tiles = row_tiles_bound(p.g.rows, p.g.E, TM) * ((p.N + TN - 1) / TN);
    const unsigned grid = (unsigned)(tiles < num_sms * 4 ? (tiles > 0 ? tiles : 1) : num_sms * 4);
    if (p.dtype == MOE_FP32) fp8_rows_kernel<float><<<grid, 256, 0, s>>>(p);
    else fp8_rows_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace moe
