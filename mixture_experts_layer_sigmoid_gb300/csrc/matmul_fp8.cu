// matmul_fp8.cu -- products of E4M3 codes with a scale for each block of 128, rows grouped
// by expert or dense, on the sm_103a tensor cores:
//   Y[r][n] = sum_kb SA[r][kb] SB[kb][n/128] sum_{k in block kb} A[r][k] B[k][n].
//
// Persistent blocks of twelve warps, one block to an SM. Warp 0 loads 128-deep blocks of both
// operands by TMA (swizzled; B K-major or MN-major as stored) and warp 2 their scales by
// cp.async; warp 1 issues tcgen05.mma.kind::f8f6f4 (128 x 256) from an elected thread, each block
// into one of two partial buffers in tensor memory; warps 4-11 fold each finished buffer into
// fp32 registers with its scales, a row's 128 columns (one scale of B) to a thread.
//   - Tensor memory holds two blocks' MMAs (2 x 512 cycles), so a block costs half of MMAs, fold
//     and the signals between them. The fold returns a buffer as soon as its last columns are
//     in registers, before their FMAs, with a relaxed arrive (a release would wait for
//     outstanding loads), and has its scales before the MMAs' signal (read after it they cost 90
//     cycles a block).
//   - setmaxnreg moves the loading warps' registers to the folding ones (128 sums, 64 columns
//     in flight); loop bounds and addresses of the fold are made uniform by a shuffle, and its
//     waits are bare (spin_tries): each kept the compiler from copying sums in the loop.
#include "grouped_tc.cuh"

namespace moe {
namespace {

using namespace gtc;

constexpr int QK = 128;                        // depth of a block, and of a scale
constexpr int kThreads8 = 384;
constexpr int kRegs = (128 * 88 + 256 * 208) / kThreads8;   // a thread's at the launch
constexpr int kFirst = 4;                      // first folding warp
constexpr int kGroup = 4;                      // blocks whose scales are copied together
constexpr int kSlots = 6;                      // groups of them in shared memory
constexpr int kSlot = 130 * 4 * kGroup;        // 128 rows' and two column blocks' scales of a group

struct Args8 {
    Args a;                                    // K, N, segments, output
    const float *SA, *SB;
    long long ldsa, ldsb, ssb;
    int sa_vec, out32;                         // rows of SA in 16-byte pieces, outputs in 32-byte ones
};

constexpr int A8 = BM * QK, STAGE8 = A8 + BN * QK;
constexpr int S8 = (kSmemMax - 1024 - kSlots * kSlot - kTable - kBars) / STAGE8;
constexpr int SMEM8 = 1024 + S8 * STAGE8 + kSlots * kSlot + kTable + kBars;
static_assert(S8 + 2 <= kSlots && kSlot % 16 == 0, "a slot's last readers are done when its next group's first stage is free");

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t more)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(more) : "memory");
}

// acc (pairs of columns) += 32 columns in r times the scale
__device__ __forceinline__ void fold32(uint64_t* acc, const uint32_t (&r)[32], float scale)
{
    uint64_t s2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(scale));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint64_t v;
        asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(r[2 * i]), "r"(r[2 * i + 1]));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i]) : "l"(v), "l"(s2));
    }
}
// Four or sixteen bytes to shared memory, asynchronously; zeros past the first `have` of them.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool have)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(have ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const float* src, int have)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
}

template <typename T, bool B_MN>
__global__ void __launch_bounds__(kThreads8, 1)
fp8_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB, const Args8 p)
{
    const Args& a = p.a;
    DeviceStatus* const status = &wait_status;
    constexpr int S = S8;
    // E4M3 in, fp32 out; A K-major
    constexpr uint32_t IDESC = (1u << 4) | (B_MN ? (1u << 16) : 0u) | ((uint32_t)(BM >> 4) << 24);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring = ptx::smem_u32(smem);
    const uint32_t slots = ring + S * STAGE8;
    SegmentTable& table = *reinterpret_cast<SegmentTable*>(smem + S * STAGE8 + kSlots * kSlot);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * STAGE8 + kSlots * kSlot + kTable);
    static_assert((2 * S + 5 + kSlots) * 8 + 8 + 16 <= kBars && SMEM8 % 16 == 0, "barriers");
    const uint32_t bar0 = (ptx::smem_u32(bars) + 7u) & ~7u;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto pfull_bar = [&](int i) { return bar0 + 8u * (2 * S + i); };
    auto pempty_bar = [&](int i) { return bar0 + 8u * (2 * S + 2 + i); };
    auto scale_bar = [&](int i) { return bar0 + 8u * (2 * S + 5 + i); };
    const uint32_t final_bar = bar0 + 8u * (2 * S + 4);
    uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem + SMEM8 - 1024 - 16);
    volatile int& abort_flag = *reinterpret_cast<volatile int*>(smem + SMEM8 - 1024 - 8);
    const uint32_t flag = ring + SMEM8 - 1024 - 8;

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 33);       // the operands, and each lane of the scales' warp
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(pfull_bar(i), 1);
            ptx::mbar_init(pempty_bar(i), 8);
        }
        for (int i = 0; i < kSlots; ++i) ptx::mbar_init(scale_bar(i), 32);
        ptx::mbar_init(final_bar, 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && elect_one()) {
        ptx::prefetch_tmap(&mA);
        ptx::prefetch_tmap(&mB);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    read_segments<BM>(a.g, &table);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

    Work<false, SINGLE, QK> work;
    work.init(a, table.pre);
    work.total = __shfl_sync(0xffffffffu, work.total, 0);
    auto wait = [&](uint32_t bar, uint32_t parity, int where) {
        return ptx::wait_bounded(bar, parity, &abort_flag, status, where);
    };

    // 384 threads x 168 registers at the launch (the host looks) = 128 x 88 + 256 x 208
    if (warp < kFirst) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) {
            // --------------------------------------------------- TMA loads
            if (elect_one()) {
                int s = 0;
                uint32_t ph = 0, loaded = 0;           // bits of stages
                bool ok = true;
                for (long long w = blockIdx.x; ok && w < work.total; w += gridDim.x) {
                    const Tile t = work.at(a, table, w, 0);
                    const int stripes = (t.nt + 127) / 128;        // MN-major: 128 columns each
                    const uint32_t bytes = A8 + (B_MN ? stripes * 128 : BN) * QK;
                    for (int kb = 0; kb < t.kblocks; ++kb) {
                        if (!wait(empty_bar(s), ph ^ 1u, 21)) { ok = false; break; }
                        const uint32_t dst_a = ring + s * STAGE8, dst_b = dst_a + A8, bar = full_bar(s);
                        ptx::mbar_arrive_expect_tx(bar, bytes);
                        load_3d<false>(dst_a, &mA, bar, kb * QK, t.row, 0);
                        if constexpr (B_MN) {
                            for (int i = 0; i < stripes; ++i)
                                load_3d<false>(dst_b + i * 128 * QK, &mB, bar, t.n0 + 128 * i, kb * QK, t.e);
                        } else {
                            load_3d<false>(dst_b, &mB, bar, kb * QK, t.n0, t.e);
                        }
                        loaded |= 1u << s;
                        if (++s == S) { s = 0; ph ^= 1u; }
                    }
                }
                // what is on its way into the ring lands before the block ends, with a limit of its own
                // once the pipeline has given up
                volatile int never = 0;
                for (int i = 0; i < S; ++i) {
                    if (!(loaded >> i & 1u)) continue;
                    const uint32_t parity = i < s ? ph : ph ^ 1u;
                    ok = ok && wait(full_bar(i), parity, 27);
                    if (!ok) ptx::wait_bounded(full_bar(i), parity, &never, status, 27, kDrainNs);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (elect_one()) {
                // ------------------------------------------------------- MMAs
                int s = 0;
                uint32_t ph = 0, used = 0;
                bool ok = true;
                for (long long w = blockIdx.x; ok && w < work.total; w += gridDim.x) {
                    const Tile t = work.at(a, table, w, 0);
                    const uint32_t id = IDESC | ((uint32_t)(t.nt >> 3) << 17);
                    for (int kb = 0; kb < t.kblocks; ++kb, ++used) {
                        const int b = (int)(used & 1u);
                        if (!spin(full_bar(s), ph, flag) || !spin(pempty_bar(b), ((used >> 1) & 1u) ^ 1u, flag)) { ok = false; break; }
                        ptx::tc_fence_after();
                        const uint32_t d = tmem + (uint32_t)(b * 256);
                        const uint32_t pa = ring + s * STAGE8, pb = pa + A8;
#pragma unroll
                        for (int k = 0; k < QK / 32; ++k) {
                            const uint64_t da = ptx::smem_desc_sw128(pa + k * 32, 16, 1024);
                            const uint64_t db = B_MN ? ptx::smem_desc_sw128(pb + k * 4096, 128 * QK, 1024)
                                                     : ptx::smem_desc_sw128(pb + k * 32, 16, 1024);
                            mma_e4m3(d, da, db, id, k > 0 ? 1u : 0u);
                        }
                        ptx::tc_commit(pfull_bar(b));
                        ptx::tc_commit(empty_bar(s));
                        if (++s == S) { s = 0; ph ^= 1u; }
                    }
                }
                ptx::tc_commit(final_bar);
                if (!ok) {
                    abort_flag = 1;
                    report_timeout(status, 22);
                }
            }
            __syncwarp();
            if (lane == 0) {
                volatile int never = 0;
                ptx::wait_bounded(final_bar, 0, &never, status, 24);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ----------------------------------------------------- scales
            // The scales of up to four blocks go to the next of six slots together, once the first
            // block's stage is free. That is block i's: then the MMAs of block i - S have
            // completed, which were issued after the fold of block i - S - 2 had its columns (and
            // scales) in registers; and the slot's last group, six before, ended no later than
            // i - 6 (six groups of a block each, or more blocks); S is 4.
            int s = 0, slot = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (long long w = blockIdx.x; ok && w < work.total; w += gridDim.x) {
                const Tile t = work.at(a, table, w, 0);
                // four of the tile's 128 rows to a lane; the first two lanes also have the
                // scales of its one or two column blocks
                const float* src = p.SA + (long long)t.row * p.ldsa;
                const int nb = t.n0 / 128 + (lane & 1);
                const bool have_b = nb * 128 < a.N;
                const float* src_b = p.SB + t.e * p.ssb + (have_b ? (B_MN ? (long long)nb : nb * p.ldsb) : 0ll);
                const long long step_b = B_MN ? p.ldsb : 1;
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    if (!__all_sync(0xffffffffu, wait(empty_bar(s), ph ^ 1u, 26))) { ok = false; break; }
                    if (kb % kGroup == 0) {
                        const uint32_t at = slots + (uint32_t)(slot * kSlot);
                        const int n = min(t.kblocks - kb, kGroup);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = lane + 32 * j;
                            const bool have = r < t.valid;
                            const float* from = have ? src + r * p.ldsa + kb : p.SA;
                            if (p.sa_vec) {
                                copy16(at + 16 * r, from, have ? 4 * n : 0);
                            } else {
                                for (int i = 0; i < n; ++i) copy4(at + 16 * r + 4 * i, have ? from + i : from, have);
                            }
                        }
                        if (lane < 2)
                            for (int i = 0; i < n; ++i) copy4(at + 2048 + 16 * lane + 4 * i, src_b + (kb + i) * step_b, have_b);
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(scale_bar(slot)) : "memory");
                        slot = slot + 1 == kSlots ? 0 : slot + 1;
                    }
                    // with every block: a block's MMAs wait for this warp, so that it never falls
                    // a whole round of stages behind
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full_bar(s)) : "memory");
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ------------------------------------------------- fold and outputs
        const int q = warp & 3, h = (warp - kFirst) >> 2;      // lanes 32 q..; columns 128 h..
        uint32_t it = 0, slot = 0, sph = 0;                    // blocks; groups of scales
        bool ok = true;
        for (long long w = blockIdx.x; ok && w < work.total; w += gridDim.x) {
            Tile t = work.at(a, table, w, 0);
            t.kblocks = __shfl_sync(0xffffffffu, t.kblocks, 0);
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0ull;
#pragma unroll 1
            for (int kb = 0; kb < t.kblocks; ++kb, ++it) {
                const uint32_t off = (kb & 3) * 4;
                if (off == 0) ok = ok && spin_tries(scale_bar(slot), sph);
                float sa, sb;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sa) : "r"(slots + slot * kSlot + off + 16 * (q * 32 + lane)));
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sb) : "r"(slots + slot * kSlot + off + 2048 + 16 * h));
                sa *= sb;
                const uint32_t b = it & 1u;
                ok = ok && spin_tries(pfull_bar(b), (it >> 1) & 1u);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                ptx::tc_fence_after();
                const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + b * 256 + h * 128;
                uint32_t r0[32], r1[32];
                ptx::tmem_ld32(ta, r0);
                ptx::tmem_ld32(ta + 32, r1);
                ptx::tmem_ld_wait();
                fold32(acc, r0, sa);
                ptx::tmem_ld32(ta + 64, r0);
                fold32(acc + 16, r1, sa);
                ptx::tmem_ld32(ta + 96, r1);
                ptx::tmem_ld_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_relaxed(pempty_bar(b));
                fold32(acc + 32, r0, sa);
                fold32(acc + 48, r1, sa);
                if (off == 12 || kb + 1 == t.kblocks) {
                    if (++slot == kSlots) { slot = 0; sph ^= 1u; }
                }
            }
            if (!ok) {
                abort_flag = 1;
                report_timeout(status, 25);
                break;
            }
            // outputs straight from the registers, a thread's 256 or 512 bytes of a row in order, in
            // whole 32-byte sectors where they are aligned (through a staging buffer they would go
            // out in whole lines, but that code made the compiler copy the sums in the loop above)
            const int r = q * 32 + lane, c0 = t.n0 + 128 * h;
            const bool mine = r < t.valid;
            if (r < t.end) {
                T* o = static_cast<T*>(a.out) + (long long)(t.row + r) * a.ldo + c0;
                const int left = a.N - c0;
                constexpr int CV = 32 / (int)sizeof(T);
#pragma unroll
                for (int j = 0; j < 128 / CV; ++j) {
                    uint32_t x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float lo, hi;
                        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(acc[(j * CV + i * CV / 8) / 2]));
                        if constexpr (sizeof(T) == 2) {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
                            x[i] = mine ? *reinterpret_cast<const uint32_t*>(&v) : 0u;
                        } else {
                            x[i] = mine ? __float_as_uint(i & 1 ? hi : lo) : 0u;
                        }
                    }
                    if (p.out32 && j * CV + CV <= left) {
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + j * CV), "r"(x[0]), "r"(x[1]),
                                     "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]) : "memory");
                    } else {
#pragma unroll
                        for (int c = 0; c < CV; ++c)
                            if (j * CV + c < left) {
                                if constexpr (sizeof(T) == 2)
                                    reinterpret_cast<unsigned short*>(o + j * CV)[c] = (unsigned short)(x[c / 2] >> (16 * (c & 1)));
                                else
                                    reinterpret_cast<uint32_t*>(o + j * CV)[c] = x[c];
                            }
                    }
                }
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <typename T, bool B_MN>
cudaError_t fp8_rows(const Fp8Rows& in, int num_sms, cudaStream_t s)
{
    const moe_fp8_matmul_args_t& f = in.a;
    Args8 p{};
    p.a.g = in.g;
    p.a.K = in.K; p.a.N = in.N;
    p.a.out = f.Y; p.a.ldo = f.ldy;
    p.out32 = f.ldy * (long long)sizeof(T) % 32 == 0 && (reinterpret_cast<uintptr_t>(f.Y) & 31u) == 0;
    p.SA = f.SA; p.ldsa = f.ldsa; p.sa_vec = f.ldsa % 4 == 0;
    p.SB = f.SB; p.ldsb = f.ldsb; p.ssb = f.ssb;
    const long long units = row_tiles_bound(in.g.rows, in.g.E, BM) * ((in.N + BN - 1) / BN);
    CUtensorMap mA, mB;
    if (!make_map(&mA, f.A, in.K, in.g.rows, 1, f.lda, 0, BM, 1) ||
        !(B_MN ? make_map(&mB, f.B, in.N, in.K, in.g.E, f.ldb, f.sb, QK, 1)
               : make_map(&mB, f.B, in.K, in.N, in.g.E, f.ldb, f.sb, BN, 1)))
        return cudaErrorInvalidValue;
    auto k = fp8_kernel<T, B_MN>;
    static std::atomic<int> slots[kMaxDevices];
    int n = 0;
    // (a build with fewer registers would leave setmaxnreg waiting)
    const cudaError_t e = units_at_once(reinterpret_cast<const void*>(k), kThreads8, SMEM8, false, num_sms, slots, &n, kRegs);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)(units < n ? units : n), kThreads8, SMEM8, s>>>(mA, mB, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_rows(const Fp8Rows& p, int num_sms, cudaStream_t s)
{
    if (p.dtype == MOE_FP32) return p.a.b_nk ? fp8_rows<float, false>(p, num_sms, s) : fp8_rows<float, true>(p, num_sms, s);
    return p.a.b_nk ? fp8_rows<__nv_bfloat16, false>(p, num_sms, s) : fp8_rows<__nv_bfloat16, true>(p, num_sms, s);
}
cudaError_t take_fp8_status(int* code, cudaStream_t s) { return take_status(code, s); }
cudaError_t stall_fp8(cudaStream_t s) { return launch_stalled(s); }

}  // namespace moe
