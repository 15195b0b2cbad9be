// grouped_tc_wgrad.cu -- D_e = sum over the expert's rows of A[r]^T B[r] on the tensor
// cores (grouped_tc.cuh has the kernel): the gradient of the experts' weights.
#include "grouped_tc.cuh"

namespace moe {

using namespace gtc;

cudaError_t launch_grouped_wgrad_tc(const GroupedWgrad& p, int num_sms, cudaStream_t s)
{
    Args a{};
    a.g = p.g;
    a.M = p.M; a.N = p.N;
    a.out = p.D; a.ldo = p.ldd; a.so = p.sd;
    CUtensorMap mO{};
    a.vec = make_map(&mO, p.D, p.N, p.M, p.g.E, p.ldd, p.sd, 32, 2, 64);
    // one CTA's 128 rows hold a narrow M; wider ones go to pairs
    const bool pair = p.M > BM;
    const long long num_n = (p.N + BN - 1) / BN;
    auto units = [&](int tm) { return (long long)p.g.E * ((p.M + tm - 1) / tm) * num_n; };
    CUtensorMap mA, mB;
    if (p.g.rows > 0 && make_map(&mA, p.A, p.M, p.g.rows, 1, p.lda, 0, BK) && make_map(&mB, p.B, p.N, p.g.rows, 1, p.ldb, 0, BK))
        return pair ? launch<true, true, PAIRS, false>(mA, mB, mA, mO, a, units(2 * BM), num_sms, s)
                    : launch<true, true, SINGLE, false>(mA, mB, mA, mO, a, units(BM), num_sms, s);
    a.A = static_cast<const __nv_bfloat16*>(p.A); a.lda = p.lda;
    a.B = static_cast<const __nv_bfloat16*>(p.B); a.ldb = p.ldb;
    return launch<true, true, SINGLE, true>(CUtensorMap{}, CUtensorMap{}, CUtensorMap{}, mO, a, units(BM), num_sms, s);
}
cudaError_t take_wgrad_status(int* code, cudaStream_t s) { return take_status(code, s); }
cudaError_t stall_wgrad(cudaStream_t s) { return launch_stalled(s); }

}  // namespace moe
