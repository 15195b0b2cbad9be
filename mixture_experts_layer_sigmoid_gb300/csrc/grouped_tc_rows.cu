// grouped_tc_rows.cu -- Y[r] = X[r] W_e on the tensor cores (grouped_tc.cuh has the
// kernel): the forward product, and with the weights' other orientation the gradient of X.
#include "grouped_tc.cuh"

namespace moe {
namespace gtc {

bool make_map(CUtensorMap* m, const void* p, long long inner, long long rows, long long mats, long long ld,
              long long stride, int box_rows, int bytes, int width)
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> found{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 encode = found.load(std::memory_order_acquire);
    if (!encode) {                                     // (not found is asked again)
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            found.store(encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn), std::memory_order_release);
    }
    if (!encode || (reinterpret_cast<uintptr_t>(p) & 15u) || ld * bytes % 16 || (mats > 1 && stride * bytes % 16)) return false;
    if (mats == 1) stride = ld * rows;
    if (stride * bytes >= (1ll << 40) || ld * bytes >= (1ll << 40)) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)mats};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * bytes), (cuuint64_t)(stride * bytes)};
    const cuuint32_t box[3] = {(unsigned)(width / bytes), (cuuint32_t)box_rows, 1u}, es[3] = {1u, 1u, 1u};
    return encode(m, bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gtc

using namespace gtc;

namespace {

// Rows of the buffers for each expert from which tiles go to CTA pairs (64 experts of 256 rows,
// 7168 x 2048, the gradient of the rows: 451 us as single CTAs, 414 as pairs). The host knows the
// buffers' rows, padding and room included, and not the routing: a batch of few rows in segments
// padded to 128 of them counts as one of 128-row experts.
constexpr long long kPairRows = 128;

// ... and below which they are tiles of few rows.
constexpr long long kFewRows = 32;

template <bool B_MN, Mode MODE>
bool rows_mode(const GroupedRows& p, const Args& a, const CUtensorMap& mO, int num_sms, cudaStream_t s, cudaError_t* e)
{
    using C = Cfg<MODE>;
    CUtensorMap mA, mB, mH{};
    if (!make_map(&mA, p.X, p.K, p.g.rows, 1, p.ldx, 0, MODE == FEW ? FM : BM) ||
        (MODE == PAIRS && !make_map(&mH, p.X, p.K, p.g.rows, 1, p.ldx, 0, BM / 2)) ||
        !(B_MN ? make_map(&mB, p.W, p.N, p.K, p.g.E, p.ldw, p.sw, BK)
               : make_map(&mB, p.W, p.K, p.N, p.g.E, p.ldw, p.sw, C::B_COLS)))
        return false;
    const long long units = row_tiles_bound(p.g.rows, p.g.E, C::ROWS) * ((p.N + C::COLS - 1) / C::COLS);
    *e = launch<false, B_MN, MODE, false>(mA, mB, mH, mO, a, units, num_sms, s);
    return true;
}

template <bool B_MN>
cudaError_t rows_tc(const GroupedRows& p, int num_sms, cudaStream_t s)
{
    Args a{};
    a.g = p.g;
    a.K = p.K; a.N = p.N;
    a.out = p.Y; a.ldo = p.ldy;
    CUtensorMap mO{};
    a.vec = make_map(&mO, p.Y, p.N, p.g.rows, 1, p.ldy, 0, 32, 2, 64);
    const long long each = p.g.rows / p.g.E;
    cudaError_t e = cudaSuccess;
    if (each < kFewRows ? rows_mode<B_MN, FEW>(p, a, mO, num_sms, s, &e)
                        : (each >= kPairRows ? rows_mode<B_MN, PAIRS>(p, a, mO, num_sms, s, &e)
                                             : rows_mode<B_MN, SINGLE>(p, a, mO, num_sms, s, &e)))
        return e;
    a.A = static_cast<const __nv_bfloat16*>(p.X); a.lda = p.ldx;
    a.B = static_cast<const __nv_bfloat16*>(p.W); a.ldb = p.ldw; a.sb = p.sw;
    const long long units = row_tiles_bound(p.g.rows, p.g.E, BM) * ((p.N + BN - 1) / BN);
    return launch<false, B_MN, SINGLE, true>(CUtensorMap{}, CUtensorMap{}, CUtensorMap{}, mO, a, units, num_sms, s);
}

}  // namespace

cudaError_t launch_grouped_rows_tc(const GroupedRows& p, int num_sms, cudaStream_t s)
{
    return p.w_nk ? rows_tc<false>(p, num_sms, s) : rows_tc<true>(p, num_sms, s);
}
cudaError_t take_rows_status(int* code, cudaStream_t s) { return take_status(code, s); }
cudaError_t stall_rows(cudaStream_t s) { return launch_stalled(s); }

}  // namespace moe
