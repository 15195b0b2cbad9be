// grouped_tc.cuh -- products grouped by expert on the sm_103a tensor cores (bf16
// operands, fp32 accumulation in tensor memory): one kernel template, instantiated for
// rows (grouped_tc_rows.cu) and weight gradients (grouped_tc_wgrad.cu).
//
//   rows            Y[r][n] = sum_k X[r][k] W[e(r)][k][n], tiles of 128 rows of one segment
//                   (256 in a CTA pair) by up to 256 columns
//   weight gradient D[e][m][n] = sum over the expert's rows r of A[r][m] B[r][n]
//
// Persistent blocks, one to an SM. Warp 0 loads 64-deep blocks of both operands into a
// ring of shared-memory stages by TMA (128-byte swizzle); warp 1 issues tcgen05.mma from
// one elected thread into one of two 256-column accumulators; warps 2-5 read the other
// one (tcgen05.ld, a row to a thread) and store it by TMA from swizzled staging buffers (a
// segment's last rows by the warp). Segments start at any row: a tile's A box simply runs into the next
// expert's rows, whose products are not stored.
//   - The issuing loops run in an elected thread (elect.sync): from a branch on the lane
//     number the compiler cannot use the uniform datapath, and a block of four MMAs, its
//     commit and its wait took 536 cycles instead of 293 (512 is the time of the MMAs).
//   - CTA pairs (cta_group::2, M = 256) halve what a block loads and reads of B: 64 bytes a
//     cycle of shared memory for operands and 64 for loads, where a single CTA needs 96 and 96.
//   - The columns of the last tile need no padding: the MMA's N is the tile's own. The last
//     unit of a segment in a pair that has at most 128 rows takes M = 128, 64 rows to a CTA.
//   - A weight gradient's contraction ends inside a 64-row block that also holds rows of
//     others (perhaps NaN). That block's loads complete on a barrier of their own; a fixing
//     warp zeroes the rows up to the next multiple of 16 in both operands and then signals
//     the block; the MMAs stop at that multiple.
//   - FEW: tiles of 32 rows by 64 columns for buffers of few rows an expert, whose weights are all there is
//     to read: 16 stages of 8 KB of them in flight, and enough tiles for every SM. (The MMAs
//     still take 128 rows, 250 cycles a block, less than HBM takes to bring it.)
//   - GUARD: operands that TMA cannot take (strides off the 16-byte boundaries) are loaded by
//     sixteen warps, as pairs of aligned 16-byte windows that are shifted, into the same layout
//     (1777 x 3 rows of 1001 x 771 74 us; ten warps that worked out each address took 113, the
//     second window as the neighbour's by a shuffle 78).
#pragma once
#include "grouped.cuh"
#include "per_device.h"
#include "ptx.cuh"

#include <atomic>
#include <cudaTypedefs.h>

namespace moe {
namespace gtc {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int STRIPE = 64 * 128;               // 64 columns of a 64-deep block, MN-major
constexpr int kSmemMax = 232448;               // 227 KB
constexpr int kStaging = 4 * 4096;             // per epilogue warp 32 rows of 128 bytes
constexpr int kTable = (int)sizeof(SegmentTable);
constexpr int kBars = 512;
constexpr int kGroupSpan = 16;                 // as the layer's engine: a weight tile's units run at
                                               // most this many tiles apart

struct Args {
    Groups g;
    int K;                    // rows: contraction; unused by weight gradients
    int M, N;                 // outputs of a weight gradient (M); columns (N)
    void* out;
    long long ldo, so;
    int vec;                  // outputs in 16-byte pieces (and by TMA)
    const __nv_bfloat16 *A, *B;   // GUARD
    long long lda, ldb, sb;
};

// Single CTAs, pairs, or single CTAs on tiles of few rows.
enum Mode { SINGLE, PAIRS, FEW };
constexpr int FM = 32, FN = 64;                // a FEW tile

template <Mode MODE>
struct Cfg {
    static constexpr bool PAIR = MODE == PAIRS;
    static constexpr int ROWS = MODE == FEW ? FM : (PAIR ? 2 * BM : BM);        // of a unit
    static constexpr int COLS = MODE == FEW ? FN : BN;
    static constexpr int A_BYTES = (MODE == FEW ? FM : BM) * BK * 2;
    static constexpr int B_COLS = PAIR ? BN / 2 : COLS;
    static constexpr int STAGE = A_BYTES + B_COLS * BK * 2;
    static constexpr int STAGES = (kSmemMax - 1024 - kStaging - kTable - kBars) / STAGE;
    static constexpr int SMEM = 1024 + STAGES * STAGE + kStaging + kTable + kBars;
    // the MMAs of a FEW tile read 128 rows of A: what lies behind its 32, whose products are not stored
    static_assert(BM * BK * 2 - STAGE <= kStaging, "inside the block's shared memory");
};

// Limit of the wait for a stage's loads once a pipeline has given up.
constexpr uint64_t kDrainNs = 10000000;

// Set by a wait that ran out (one word per translation unit and device).
static __device__ DeviceStatus wait_status;

constexpr int kLoaders = 512;                  // GUARD: loading threads, eight to a row of 64

template <bool WGRAD, bool GUARD>
constexpr int threads() { return GUARD ? 192 + kLoaders : (WGRAD ? 224 : 192); }

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
    return p != 0;
}
// Waits for the phase with this parity as ptx::wait_bounded does, for the threads that issue MMAs:
// gives up when another role of the block has raised the abort flag (at this address), or LIMIT_NS
// after its first look at the clock; the caller raises the flag and records it. The looks come
// between rounds of tries, and their outcome is voted on: a branch on it that the compiler cannot
// prove uniform would take the MMAs behind it off the uniform datapath (four decoded tokens 97
// instead of 62 us). CLUSTER: the peer's fixing warp may be the last to arrive.
template <uint64_t LIMIT_NS = kWaitLimitNs, bool CLUSTER = false>
__device__ __forceinline__ bool spin(uint32_t bar, uint32_t parity, uint32_t abort_flag)
{
    uint64_t t0 = 0;
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)) return true;
        uint32_t raised;
        asm volatile("ld.volatile.shared::cta.u32 %0, [%1];" : "=r"(raised) : "r"(abort_flag) : "memory");
        const uint64_t t = ptx::globaltimer();
        if (t0 == 0) t0 = t;
        if (__any_sync(__activemask(), raised != 0 || t - t0 > LIMIT_NS)) return false;
    }
}
// The same with nothing but tries, for matmul_fp8.cu's fold: one on a barrier that nothing signals
// takes 2.8 us here, all of them 3 s. With a look at the flag or the clock between them the
// compiler copied the fold's sums (8192 x 7168 x 4096 codes 216 to 221 us instead of 195).
template <int TRIES = 1 << 20>
__device__ __forceinline__ bool spin_tries(uint32_t bar, uint32_t parity)
{
    for (int i = 0; i < TRIES; ++i)
        if (ptx::mbar_try_wait(bar, parity)) return true;
    return false;
}
// Records a wait that ran out.
__device__ __forceinline__ void report_timeout(DeviceStatus* st, int where)
{
    if (atomicCAS(&st->code, 0, (int)MOE_ERR_DEVICE_TIMEOUT) == 0) st->where = where;
}
template <bool PAIR>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z)
{
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar),
                     "r"(x), "r"(y), "r"(z) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar),
                     "r"(x), "r"(y), "r"(z) : "memory");
}

__device__ __forceinline__ void store_3d(const CUtensorMap* m, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)), "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}

// The limit of a wait for tiles of this many blocks in all, each up to some twenty times as long as
// the slowest one takes (0.9 us): a weight gradient's only tile may hold 2^31 rows.
__device__ __forceinline__ uint64_t limit_of(long long blocks) { return kWaitLimitNs + (uint64_t)blocks * 20000u; }

// A tile of outputs, as every role of a block sees it.
struct Tile {
    int e;
    int row;                  // first row: of the output rows, or of the contraction
    int m0, n0, nt;           // first column (and output row of a weight gradient); the MMA's N
    int kblocks, tail;        // blocks of the contraction; values in the last one
    int end, valid;           // rows: stored rows of this CTA's 128; those that are not padding
    bool half;                // a pair's unit of 128 rows (M = 128), 64 to a CTA
};

template <bool WGRAD, Mode MODE, int DEPTH = BK>
struct Work {
    static constexpr bool PAIR = MODE == PAIRS;
    static constexpr int TN = Cfg<MODE>::COLS;
    int num_n, num_m;
    long long total;
    __device__ __forceinline__ void init(const Args& a, const int* pre)
    {
        num_n = (a.N + TN - 1) / TN;
        num_m = WGRAD ? (a.M + (PAIR ? 2 * BM : BM) - 1) / (PAIR ? 2 * BM : BM) : pre[a.g.E];
        total = WGRAD ? (long long)a.g.E * num_m * num_n : (long long)num_m * num_n;
    }
    __device__ __forceinline__ Tile at(const Args& a, const SegmentTable& table, long long w, int rank) const
    {
        const int* pre = table.pre;
        Tile t;
        if constexpr (WGRAD) {
            // the smaller of the two tile counts runs fastest, so that the blocks at work
            // cover all of that dimension and read each slice of the other once
            const int per = num_m * num_n;
            t.e = (int)(w / per);
            const int r = (int)(w - (long long)t.e * per);
            const int mu = num_n < num_m ? r / num_n : r % num_m;
            t.n0 = (num_n < num_m ? r % num_n : r / num_m) * TN;
            t.m0 = (PAIR ? 2 * mu + rank : mu) * BM;
            const Segment s = table.at(t.e);
            t.row = s.begin;
            t.kblocks = (s.valid + DEPTH - 1) / DEPTH;
            t.tail = s.valid - (t.kblocks - 1) * DEPTH;
            t.end = t.valid = a.M - t.m0;
            t.half = false;
        } else {
            // expert by expert; within one, groups of G column tiles walk its row units, so
            // that its rows and weights stay in L2 while they are used
            const int q = (int)(w / num_n);
            t.e = segment_at(pre, a.g.E, q);
            const int u0 = pre[t.e], nu = max(pre[t.e + 1] - u0, 1);
            const int r0 = (int)(w - (long long)u0 * num_n);
            const int G = nu <= kGroupSpan / 2 ? max(1, kGroupSpan / nu) : kGroupSpan;
            const int group = r0 / (nu * G), r = r0 - group * nu * G;
            const int gsz = min(G, num_n - group * G);
            const int mu = r / gsz;
            t.n0 = (group * G + r % gsz) * TN;
            const Segment s = table.at(t.e);
            const int first = mu * Cfg<MODE>::ROWS;       // row of the unit in its segment
            t.half = PAIR && s.end - s.begin - first <= BM;
            const int mine = first + (PAIR ? rank * (t.half ? BM / 2 : BM) : 0);
            t.row = s.begin + mine;
            t.m0 = 0;
            t.kblocks = first < s.valid ? (a.K + DEPTH - 1) / DEPTH : 0;
            t.tail = DEPTH;
            t.end = s.end - t.row;
            if (MODE == FEW) t.end = min(t.end, FM);
            t.valid = s.valid - mine;
        }
        // the MMA's N: a multiple of 16, of 32 in a pair
        constexpr int step = PAIR ? 32 : 16;
        t.nt = min(TN, (a.N - t.n0 + step - 1) / step * step);
        return t;
    }
};

// Eight bf16 values from an address `off` bytes behind a 16-byte boundary, of which `n` exist,
// in two steps: the aligned 16-byte windows that hold them, and the shift.
struct Windows { uint4 a, b; };
__device__ __forceinline__ Windows load_windows(const __nv_bfloat16* p, unsigned off, int n)
{
    Windows w{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    const uint4* base = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
    if (n > 0) w.a = base[0];                           // holds the first value
    if (n > 0 && off + 2 * min(n, 8) > 16) w.b = base[1];   // holds the last one
    return w;
}
__device__ __forceinline__ uint4 shift_windows(const Windows& q, unsigned off, int n)
{
    uint32_t w[8] = {q.a.x, q.a.y, q.a.z, q.a.w, q.b.x, q.b.y, q.b.z, q.b.w};
    if (off & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const unsigned sh = (off & 2u) * 8;
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __funnelshift_r(w[i], w[i + 1], sh);
    if (n > 0 && n < 8) {                               // (with none the windows are zeros)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * i + 2 > n) r[i] = 2 * i + 1 > n ? 0u : r[i] & 0xFFFFu;
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool WGRAD, bool B_MN, Mode MODE, bool GUARD>
__global__ void __launch_bounds__(threads<WGRAD, GUARD>(), 1)
kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
       const __grid_constant__ CUtensorMap mH, const __grid_constant__ CUtensorMap mO, const Args a)
{
    using C = Cfg<MODE>;
    constexpr bool PAIR = MODE == PAIRS;
    DeviceStatus* const status = &wait_status;
    constexpr int S = C::STAGES;
    constexpr uint32_t IDESC = ptx::idesc_bf16<0, WGRAD, B_MN, PAIR ? 2 * BM : BM>();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring = ptx::smem_u32(smem);
    const uint32_t staging = ring + S * C::STAGE;
    SegmentTable& table = *reinterpret_cast<SegmentTable*>(smem + S * C::STAGE + kStaging);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * C::STAGE + kStaging + kTable);
    static_assert((3 * S + 5) * 8 + 8 + 16 <= kBars && C::SMEM % 16 == 0, "barriers");
    const uint32_t bar0 = (ptx::smem_u32(bars) + 7u) & ~7u;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto land_bar = [&](int s) { return bar0 + 8u * (2 * S + s); };
    auto accf_bar = [&](int i) { return bar0 + 8u * (3 * S + i); };
    auto acce_bar = [&](int i) { return bar0 + 8u * (3 * S + 2 + i); };
    const uint32_t final_bar = bar0 + 8u * (3 * S + 4);
    uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem + C::SMEM - 1024 - 16);
    volatile int& abort_flag = *reinterpret_cast<volatile int*>(smem + C::SMEM - 1024 - 8);
    const uint32_t flag = ring + C::SMEM - 1024 - 8;

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)ptx::cluster_ctarank() : 0;
    const int unit0 = PAIR ? (int)ptx::cluster_id_x() : (int)blockIdx.x;
    const int nunits = PAIR ? (int)ptx::nclusters_x() : (int)gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            // a weight gradient's block is signalled once by each CTA (its producer or, for
            // the last block, its fixing warp); other blocks by the even CTA's producer
            ptx::mbar_init(full_bar(s), GUARD ? kLoaders : (WGRAD && PAIR ? 2 : 1));
            ptx::mbar_init(empty_bar(s), 1);
            ptx::mbar_init(land_bar(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(accf_bar(i), 1);
            ptx::mbar_init(acce_bar(i), PAIR ? 8 : 4);
        }
        ptx::mbar_init(final_bar, 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (!GUARD && warp == 0 && elect_one()) {
        ptx::prefetch_tmap(&mA);
        ptx::prefetch_tmap(&mB);
    }
    if (warp == 1) {
        if (PAIR) {
            ptx::tmem_alloc_pair(ptx::smem_u32(&tmem_slot), 2 * BN);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), 2 * BN);
            ptx::tmem_relinquish();
        }
    }
    read_segments<C::ROWS>(a.g, &table);
    ptx::tc_fence_before();
    if (PAIR) ptx::cluster_sync();             // the peer's barriers exist before any remote signal
    else __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

    Work<WGRAD, MODE> work;
    work.init(a, table.pre);
    work.total = __shfl_sync(0xffffffffu, work.total, 0);
    auto wait = [&](uint32_t bar, uint32_t parity, int where, uint64_t limit = kWaitLimitNs) {
        return ptx::wait_bounded(bar, parity, &abort_flag, status, where, limit);
    };

    if (warp == 0 && !GUARD) {
        // ------------------------------------------------------- TMA loads
        if (elect_one()) {
            int s = 0;
            uint32_t ph = 0, loaded = 0, fixed = 0, lands = 0;   // bits of stages
            bool ok = true;
            for (long long w = unit0; ok && w < work.total; w += nunits) {
                const Tile t = work.at(a, table, w, rank);
                const int bcols = PAIR ? t.nt / 2 : t.nt, b0 = t.n0 + (PAIR ? rank * bcols : 0);
                const int stripes = (bcols + 63) / 64;
                const uint32_t bytes = (t.half ? C::A_BYTES / 2 : C::A_BYTES) + (B_MN ? stripes * STRIPE : C::B_COLS * BK * 2);
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    if (!wait(empty_bar(s), ph ^ 1u, 1)) { ok = false; break; }
                    const uint32_t dst_a = ring + s * C::STAGE, dst_b = dst_a + C::A_BYTES;
                    const bool fix = WGRAD && kb == t.kblocks - 1 && t.tail < BK;
                    uint32_t bar;
                    loaded |= 1u << s;
                    if (fix) {
                        bar = land_bar(s);
                        ptx::mbar_arrive_expect_tx(bar, bytes);
                        fixed |= 1u << s;
                        lands ^= 1u << s;
                    } else {
                        if (WGRAD) fixed &= ~(1u << s);
                        bar = PAIR ? ptx::mapa_shared(full_bar(s), 0) : full_bar(s);
                        if (rank == 0) {
                            ptx::mbar_arrive_expect_tx(full_bar(s), (PAIR ? 2 : 1) * bytes);
                            if (WGRAD && PAIR) ptx::mbar_arrive(full_bar(s));
                        }
                    }
                    if constexpr (WGRAD) {
                        const int y = t.row + kb * BK;
#pragma unroll
                        for (int i = 0; i < BM / 64; ++i) load_3d<PAIR>(dst_a + i * STRIPE, &mA, bar, t.m0 + 64 * i, y, 0);
                        for (int i = 0; i < stripes; ++i) load_3d<PAIR>(dst_b + i * STRIPE, &mB, bar, b0 + 64 * i, y, 0);
                    } else {
                        load_3d<PAIR>(dst_a, t.half ? &mH : &mA, bar, kb * BK, t.row, 0);
                        if constexpr (B_MN) {
                            for (int i = 0; i < stripes; ++i)
                                load_3d<PAIR>(dst_b + i * STRIPE, &mB, bar, b0 + 64 * i, kb * BK, t.e);
                        } else {
                            load_3d<PAIR>(dst_b, &mB, bar, kb * BK, b0, t.e);
                        }
                    }
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            // what is on its way into the ring lands before the block ends, with a limit of its own once
            // the pipeline has given up. (The even CTA waits for both; loads of the odd one that it never
            // counted get a millisecond.)
            volatile int never = 0;
            auto land = [&](uint32_t bar, uint32_t parity) {
                ok = ok && wait(bar, parity, 9);
                if (!ok) ptx::wait_bounded(bar, parity, &never, status, 9, kDrainNs);
            };
            for (int i = 0; i < S; ++i) {
                if (!(loaded >> i & 1u)) continue;
                if (fixed >> i & 1u) land(land_bar(i), (lands >> i & 1u) ^ 1u);
                else if (rank == 0) land(full_bar(i), i < s ? ph : ph ^ 1u);
            }
            if (PAIR && !ok && rank != 0) ptx::wait_bounded(full_bar(0), 0, &never, status, 9, kDrainNs / 10);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            // ------------------------------------------------------- MMAs
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (long long w = unit0; ok && w < work.total; w += nunits) {
                const Tile t = work.at(a, table, w, rank);
                if (!spin(acce_bar(acc), aph ^ 1u, flag)) { ok = false; break; }
                ptx::tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * BN);
                // (256 rows less 128 in the M / 16 field)
                const uint32_t id = (IDESC | ((uint32_t)(t.nt >> 3) << 17)) - (t.half ? 8u << 24 : 0u);
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    if (!spin<kWaitLimitNs, WGRAD && PAIR>(full_bar(s), ph, flag)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t pa = ring + s * C::STAGE, pb = pa + C::A_BYTES;
                    const int steps = WGRAD && kb == t.kblocks - 1 ? (t.tail + 15) / 16 : BK / 16;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) {
                        if (WGRAD && k >= steps) break;
                        const uint64_t da = WGRAD ? ptx::smem_desc_sw128(pa + k * 2048, STRIPE, 1024)
                                                  : ptx::smem_desc_sw128(pa + k * 32, 16, 1024);
                        const uint64_t db = B_MN ? ptx::smem_desc_sw128(pb + k * 2048, STRIPE, 1024)
                                                 : ptx::smem_desc_sw128(pb + k * 32, 16, 1024);
                        const uint32_t more = (kb > 0 || k > 0) ? 1u : 0u;
                        if (PAIR) ptx::tc_mma_f16_pair(d, da, db, id, more);
                        else ptx::tc_mma_f16(d, da, db, id, more);
                    }
                    if (PAIR) ptx::tc_commit_pair(empty_bar(s), 3);
                    else ptx::tc_commit(empty_bar(s));
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                if (PAIR) ptx::tc_commit_pair(accf_bar(acc), 3);
                else ptx::tc_commit(accf_bar(acc));
                acc ^= 1;
                if (acc == 0) aph ^= 1u;
            }
            if (PAIR) ptx::tc_commit_pair(final_bar, 3);
            else ptx::tc_commit(final_bar);
            if (!ok) {
                abort_flag = 1;
                report_timeout(status, 2);
            }
        }
        __syncwarp();
        // every MMA has completed before tensor memory is freed
        if (rank == 0 && lane == 0) {
            volatile int never = 0;
            ptx::wait_bounded(final_bar, 0, &never, status, 4);
        }
        __syncwarp();
    } else if (warp >= 2 && warp < 6) {
        // ----------------------------------------------------------- outputs
        const int q = warp & 3;                 // this warp's quarter of the TMEM lanes
        const uint32_t stg = staging + (uint32_t)q * 4096u;
        int acc = 0, stores = 0;
        uint32_t aph = 0;
        for (long long w = unit0; w < work.total; w += nunits) {
            Tile t = work.at(a, table, w, rank);
            t.kblocks = __shfl_sync(0xffffffffu, t.kblocks, 0);
            if (!__all_sync(0xffffffffu, wait(accf_bar(acc), aph, 5, limit_of(t.kblocks)))) break;
            ptx::tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
            // this warp's rows and columns of the tile: with M = 256 (or 128 in one CTA) a lane is a
            // row; with M = 128 in a pair, lanes 64-127 hold the second half of the columns
            // of the rows in lanes 0-63
            const int r0 = (t.half ? q & 1 : q) * 32, c0 = t.half ? (q >> 1) * (t.nt / 2) : 0;
            const int rows = __shfl_sync(0xffffffffu, t.end - r0, 0);   // of this warp's 32 rows those stored
            const bool mine = lane + r0 < t.valid;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + t.n0 + c0 +
                               (WGRAD ? t.e * a.so + (long long)(t.m0 + r0) * a.ldo
                                      : (long long)(t.row + r0) * a.ldo);
            const int cols = __shfl_sync(0xffffffffu, min(a.N - t.n0 - c0, t.half ? t.nt / 2 : t.nt), 0);
            const bool whole = a.vec && (WGRAD || rows >= 32), last = t.n0 + c0 + cols == a.N && a.N % 8 == 0;
#pragma unroll 1
            for (int u = 0; u * 32 < cols && rows > 0; ++u) {
                uint32_t v[32];
                if (t.kblocks > 0) {
                    ptx::tmem_ld32(taddr + u * 32, v);
                    ptx::tmem_ld_wait();
                }
                if (t.kblocks == 0 || !mine) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0u;
                }
                // 32 rows of 64 bytes, swizzled over them, in turns with the other half's store; TMA
                // leaves out what lies past the tensor (not past this warp's columns), in columns by
                // whole 16 bytes: a row that ends inside them would have zeros behind it
                const int left = cols - u * 32;
                const bool by_tma = __shfl_sync(0xffffffffu, (int)(whole && (left >= 32 || last)), 0) != 0;
                const uint32_t buf = stg + (uint32_t)(stores & 1) * 2048u;
                if (lane == 0) {                // what still reads this half
                    if (by_tma) ptx::bulk_wait_read<1>();
                    else ptx::bulk_wait_read<0>();
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
                        p[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)),
                                 "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]) : "memory");
                }
                if (by_tma) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        store_3d(&mO, buf, t.n0 + c0 + u * 32, WGRAD ? t.m0 + r0 : t.row + r0, WGRAD ? t.e : 0);
                        ptx::bulk_commit();
                    }
                    ++stores;
                    continue;
                }
                // the last rows of a segment, or outputs off the 16-byte boundaries
                __syncwarp();
                if (a.vec && left >= 32) {
                    // four lanes to a row of 64 bytes, eight rows an instruction
                    for (int r = lane >> 2; r < min(rows, 32); r += 8) {
                        uint4 x;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                     : "r"(buf + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)) : "memory");
                        *reinterpret_cast<uint4*>(o + r * a.ldo + u * 32 + (lane & 3) * 8) = x;
                    }
                } else if (lane < left) {
                    for (int r = 0; r < min(rows, 32); ++r) {
                        unsigned short x;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(buf + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2) : "memory");
                        reinterpret_cast<unsigned short*>(o + r * a.ldo + u * 32)[lane] = x;
                    }
                }
                __syncwarp();
            }
            // relaxed: nothing in memory is published, and a release would wait for the stores
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(acce_bar(acc), 0));
                else ptx::mbar_arrive_relaxed(acce_bar(acc));
            }
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
        if (lane == 0) ptx::bulk_wait_all();   // the stores are done before the block ends
        __syncwarp();
    } else if (GUARD && warp >= 6) {
        // ------------------------------------------- loads off the boundaries
        // The stage as rows of 128 bytes, A's (rows, or two stripes of 64) and then B's (columns,
        // or stripes of 64), eight threads to a row. A thread's rows are 64 apart, in memory 64
        // rows or 64 values: a multiple of 16 bytes, as is the way to the next block, so that the
        // shift is the tile's. All six loads are under way before the stage is free.
        const int tid = (int)threadIdx.x - 192, ch = tid & 7, r = tid >> 3;
        const uint32_t place = (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4));
        const long long ja = WGRAD ? 64 : 64 * a.lda, jb = B_MN ? 64 : 64 * a.ldb;
        const long long ka = WGRAD ? 64 * a.lda : 64, kb_ = B_MN ? 64 * a.ldb : 64;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (long long w = unit0; ok && w < work.total; w += nunits) {
            const Tile t = work.at(a, table, w, rank);
            const int n_cols = a.N - t.n0, stripes = (t.nt + 63) / 64;
            const __nv_bfloat16* pa = a.A + (long long)(t.row + r) * a.lda + t.m0 + ch * 8;
            const __nv_bfloat16* pb = WGRAD ? a.B + (long long)(t.row + r) * a.ldb + t.n0 + ch * 8
                                            : a.B + t.e * a.sb + (B_MN ? r * a.ldb + t.n0 : (long long)(t.n0 + r) * a.ldb) + ch * 8;
            const unsigned offa = (unsigned)(reinterpret_cast<uintptr_t>(pa) & 15u);
            const unsigned offb = (unsigned)(reinterpret_cast<uintptr_t>(pb) & 15u);
            for (int kb = 0; kb < t.kblocks; ++kb, pa += ka, pb += kb_) {
                const int left = WGRAD ? (kb == t.kblocks - 1 ? t.tail : BK) : a.K - kb * BK;
                Windows q[6];
                int n[6];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    n[j] = WGRAD ? (r < left ? a.M - t.m0 - 64 * j - ch * 8 : 0) : (r + 64 * j < t.valid ? left - ch * 8 : 0);
                    q[j] = load_windows(pa + j * ja, offa, n[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int m = B_MN ? (r < left ? n_cols - 64 * j - ch * 8 : 0) : (r + 64 * j < n_cols ? left - ch * 8 : 0);
                    n[2 + j] = j < stripes ? m : 0;
                    q[2 + j] = load_windows(pb + j * jb, offb, n[2 + j]);
                }
                if (!__all_sync(0xffffffffu, wait(empty_bar(s), ph ^ 1u, 6))) { ok = false; break; }
                const uint32_t dst = ring + s * C::STAGE + place;
#pragma unroll
                for (int j = 0; j < 6; ++j) {
                    if (j - 2 >= stripes) break;
                    const uint4 x = shift_windows(q[j], j < 2 ? offa : offb, n[j]);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + j * STRIPE), "r"(x.x), "r"(x.y),
                                 "r"(x.z), "r"(x.w) : "memory");
                }
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(full_bar(s));
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
    } else if (WGRAD && !GUARD) {
        // ------------------------------- the contraction's last, partial block
        int s0 = 0;
        uint32_t phases = 0;
        long long blocks = 0;                  // since the last such block, outputs (64 a tile) among them
        for (long long w = unit0; w < work.total; w += nunits) {
            const Tile t = work.at(a, table, w, rank);
            blocks += t.kblocks + 64;
            if (t.kblocks == 0) continue;
            const int s = (s0 + t.kblocks - 1) % S;
            s0 = (s0 + t.kblocks) % S;
            if (t.tail == BK) continue;
            if (!__all_sync(0xffffffffu, wait(land_bar(s), (phases >> s) & 1u, 7, limit_of(blocks)))) break;
            phases ^= 1u << s;
            blocks = 0;
            // the rows up to the next multiple of 16, in A's two stripes and in B's
            const int n = ((t.tail + 15) / 16 * 16 - t.tail) * 8;
            const int bcols = PAIR ? t.nt / 2 : t.nt, stripes = BM / 64 + (bcols + 63) / 64;
            const uint32_t at = ring + s * C::STAGE + t.tail * 128;
            for (int st = 0; st < stripes; ++st)
                for (int i = lane; i < n; i += 32)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + st * STRIPE + i * 16), "r"(0) : "memory");
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) ptx::mbar_arrive_cluster(ptx::mapa_shared(full_bar(s), 0));
                else ptx::mbar_arrive(full_bar(s));
            }
        }
    }

    ptx::tc_fence_before();
    if (PAIR) ptx::cluster_sync();             // both CTAs are done with tensor memory and signals
    else __syncthreads();
    if (warp == 1) {
        // the odd CTA's tensor memory is written by its peer's MMAs, whose last signal is on its way
        // here too (only now: a wait from the start on would have the whole kernel's time for a limit)
        if (PAIR && rank == 1 && lane == 0) {
            volatile int never = 0;
            ptx::wait_bounded(final_bar, 0, &never, status, 8);
        }
        __syncwarp();
        ptx::tc_fence_after();
        if (PAIR) ptx::tmem_dealloc_pair(tmem, 2 * BN);
        else ptx::tmem_dealloc(tmem, 2 * BN);
    }
}

// ------------------------------------------------------------------ host
// 3-D tensor map of bf16 values (or bytes): inner x rows x mats, boxes of `width` bytes x
// box_rows x 1, swizzled over that width, zeros outside. False where the strides are none
// that TMA takes.
bool make_map(CUtensorMap* m, const void* p, long long inner, long long rows, long long mats, long long ld,
              long long stride, int box_rows, int bytes = 2, int width = 128);

// The units that run at once of a kernel with this much shared memory, set up on the first
// call of each device (slots: one per kernel, zeros). `regs`: the least registers a thread that the
// kernel may have been built with.
inline cudaError_t units_at_once(const void* k, int threads, int smem, bool pair, int num_sms, std::atomic<int> (&slots)[kMaxDevices],
                                 int* out, int regs = 0)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return per_device<cudaError_t>(slots, dev, [&](int* n) {
        cudaFuncAttributes built{};
        cudaError_t e = regs ? cudaFuncGetAttributes(&built, k) : cudaSuccess;
        if (e != cudaSuccess) return e;
        if (built.numRegs < regs) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        *n = num_sms;
        if (!pair) return cudaSuccess;
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int most = 0;
        e = cudaOccupancyMaxActiveClusters(&most, k, &cfg);
        *n = most > 0 ? most : 1;
        return e;
    }, out);
}
// Waits for the stream and takes this translation unit's word.
static inline cudaError_t take_status(int* code, cudaStream_t s)
{
    DeviceStatus h{};
    cudaError_t e = cudaMemcpyFromSymbolAsync(&h, wait_status, sizeof(h), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && h.code != 0) {
        *code = h.code;
        const DeviceStatus zero{};
        e = cudaMemcpyToSymbolAsync(wait_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

// A stalled pipeline in small, on a barrier that nothing signals: one thread's wait runs out after
// 10 ms, raises the flag and records it in this translation unit's word; another's, of 2 s, ends
// with the flag; a third's after 4000 tries.
static __global__ void stalled_kernel()
{
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    const uint32_t b = ptx::smem_u32(&bar), flag = ptx::smem_u32(&abort_flag);
    if (threadIdx.x == 0) {
        ptx::mbar_init(b, 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (!spin<10000000>(b, 0, flag)) {
            *static_cast<volatile int*>(&abort_flag) = 1;
            report_timeout(&wait_status, 98);
        }
    } else if (threadIdx.x == 32) {
        spin(b, 0, flag);
    } else if (threadIdx.x == 64) {
        spin_tries<4000>(b, 0);
    }
}
static inline cudaError_t launch_stalled(cudaStream_t s)
{
    stalled_kernel<<<1, 96, 0, s>>>();
    return cudaGetLastError();
}

template <bool WGRAD, bool B_MN, Mode MODE, bool GUARD>
cudaError_t launch(const CUtensorMap& mA, const CUtensorMap& mB, const CUtensorMap& mH, const CUtensorMap& mO, const Args& a, long long units, int num_sms, cudaStream_t s)
{
    using C = Cfg<MODE>;
    constexpr bool PAIR = MODE == PAIRS;
    auto k = kernel<WGRAD, B_MN, MODE, GUARD>;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    cfg.blockDim = dim3(threads<WGRAD, GUARD>());
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    if (PAIR) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    static std::atomic<int> slots[kMaxDevices];
    int n = 0;
    const cudaError_t e = units_at_once(reinterpret_cast<const void*>(k), threads<WGRAD, GUARD>(), C::SMEM, PAIR, num_sms, slots, &n);
    if (e != cudaSuccess) return e;
    const long long grid = units < n ? (units > 0 ? units : 1) : n;
    cfg.gridDim = dim3((unsigned)(PAIR ? 2 * grid : grid));
    return cudaLaunchKernelEx(&cfg, k, mA, mB, mH, mO, a);
}

}  // namespace gtc

// The code of a wait that ran out on the current device, if one did, cleared.
cudaError_t take_rows_status(int* code, cudaStream_t s);
cudaError_t take_wgrad_status(int* code, cudaStream_t s);
cudaError_t take_fp8_status(int* code, cudaStream_t s);
// Makes one run out (moe_diag_products_wait).
cudaError_t stall_rows(cudaStream_t s);
cudaError_t stall_wgrad(cudaStream_t s);
cudaError_t stall_fp8(cudaStream_t s);

}  // namespace moe
