// sort.cu -- tokens sorted by expert and back: the index (a stable counting
// sort of the T k slots), the rows' way out, their weighted way back, and the
// gradient of that.
//
// The movers do one or two operations per value moved: bound by HBM when the
// rows are many, by latency when they are few. They go token by token, so x,
// dY and the residual are read once and only the sorted rows k times; sums are
// fp32 in slot order, rounded once. A block per token and no loop over tokens:
// a persistent grid with the next token's index fetched ahead took 179 us where
// combining 8192 x 8 rows of 7168 takes 165. Rates below are of the measured
// copy rate, 6.79 TB/s.
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kSortMaxK = 32;
constexpr int kSortMaxE = 1024;
constexpr int kSortMaxAlign = 4096;
constexpr int kSortMaxH = 1 << 20;

// ------------------------------------------------------------------ index
constexpr int kIndexThreads = 1024;
constexpr int kIndexWarps = kIndexThreads / 32;

// Four groups of slots for a warp while there are few. One block for few slots
// and rows, where a cluster's barriers cost more than they save (1024 slots
// unpadded: 3.5 us, 4.8 in a cluster; of 128 experts in segments of 128, so that
// 17 k rows have to be marked: 6.2 and 5.5 us), else clusters of eight: one for
// each 16384 slots, at most 16 (131072 slots: 9.7 us in eight, 17.8 in one, 15.7
// in sixteen).
constexpr int kIndexOneBlock = 1024, kIndexOneBlockRows = 4096;
constexpr int kIndexCluster = 8;
constexpr int kIndexSmem = 148 * 1024;  // 16 warps' pairs of 1024 experts, or 32 of 512, and the rest

// What topk says for slot i < n, or -1 past the end. Dropped slots are told
// apart where the value is used, so that loads ahead of that stay in flight.
__device__ __forceinline__ int slot_expert(const int32_t* topk, int i, int n) { return i < n ? topk[i] : -1; }

// The blocks of a cluster. Each warp takes a run of consecutive slots: it
// counts its slots of each expert, the counts are summed over warps, blocks
// (through distributed shared memory) and experts, and it then goes over its
// slots again in order, 32 at a time: each lane sets its bit in its expert's
// word, so lanes with the same expert see one another there and a slot's rank
// follows the slots' own order (one ballot per bit of the expert's number, or a
// match instruction, took 3 to 8 times as long). With several clusters each counts everything, and a run's second
// part is done by one of them: the scattered stores of slot_of, about one a
// cycle and SM, are what takes longest. 9.6 us for 131072 slots of 128 experts
// in segments of 128, 3.5 us for 264 (a single block took 200 us and 6 us).
// Shared memory: `warps` x E counters
// with their lane words, the block's E totals, the E bases and padding ranges.
template <bool CLUSTER>
__global__ void __launch_bounds__(kIndexThreads)
sort_index_kernel(const int32_t* __restrict__ topk, int n, int per, int warps, int E, int align,
                  int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ row_of,
                  int32_t* __restrict__ slot_of, int rows)
{
    extern __shared__ int2 hist[];           // [warps][E] of (count, lanes), [E] int2, [E], [E]
    __shared__ int wsum[kIndexWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const int rank = CLUSTER ? (int)ptx::cluster_ctarank() : 0, cluster = CLUSTER ? (int)ptx::cluster_id_x() : 0;
    const int clusters = CLUSTER ? (int)ptx::nclusters_x() : 1;
    const long long lo = ((long long)rank * warps + warp) * per;      // slots [lo, lo + per) of this warp
    const long long left = n - lo;
    const int mine_n = warp < warps && left > 0 ? (left < per ? (int)left : per) : 0;
    int2* mine = hist + warp * E;
    int2* pad = hist + warps * E;
    int* tot = reinterpret_cast<int*>(pad + E);
    int* base = tot + E;
    ptx::griddep_launch_dependents();        // sort_rows may be set up meanwhile; it waits for the end
    for (int i = tid; i < warps * E; i += nt) hist[i] = make_int2(0, 0);
    __syncthreads();
    // U groups of 32 slots are loaded together; the second part's first groups
    // are its last here
    constexpr int U = 8;
    int next[U];
    auto load = [&](int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = slot_expert(topk + lo, i + 32 * u + lane, mine_n);
    };
    load(0);
    for (int i = 0; i < mine_n; i += 32 * U) {
        int ex[U];
#pragma unroll
        for (int u = 0; u < U; ++u) ex[u] = next[u];
        load(i + 32 * U < mine_n ? i + 32 * U : 0);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if ((unsigned)ex[u] < (unsigned)E) atomicAdd(&mine[ex[u]].x, 1);    // integers: the order does not matter
    }
    __syncthreads();
    // thread e: counts of expert e -> each warp's base among the block's slots
    int total = 0, below = 0;
    if (tid < E) {
        constexpr int B = 8;                 // counters read together
        for (int w0 = 0; w0 < warps; w0 += B) {
            int c[B];
#pragma unroll
            for (int i = 0; i < B; ++i) c[i] = w0 + i < warps ? hist[(w0 + i) * E + tid].x : 0;
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if (w0 + i < warps) hist[(w0 + i) * E + tid].x = total;
                total += c[i];
            }
        }
        if constexpr (CLUSTER) tot[tid] = total;
    }
    if constexpr (CLUSTER) {
        ptx::cluster_sync();
        if (tid < E) {
            const uint32_t at = ptx::smem_u32(tot + tid);
            total = 0;
#pragma unroll
            for (int r = 0; r < kIndexCluster; ++r) {
                int c;
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(ptx::mapa_shared(at, r)) : "memory");
                total += c;
                below += r < rank ? c : 0;
            }
        }
    }
    // exclusive scan of the padded counts over the experts
    const int padded = (total + align - 1) / align * align;
    int sum = padded;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += t;
    }
    if (lane == 31) wsum[warp] = sum;
    __syncthreads();
    // the warps' sums: those below this warp's, and all
    int used = lane < nt / 32 ? wsum[lane] : 0, before = lane < warp ? used : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        used += __shfl_xor_sync(0xffffffffu, used, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    const int off = before + sum - padded;
    if (tid < E) {
        base[tid] = off + below;
        if (blockIdx.x == 0) {
            counts[tid] = total;
            offsets[tid] = off;
        }
        pad[tid] = make_int2(off + total, off + padded);
    }
    if (blockIdx.x == 0 && tid == 0) offsets[E] = used;
    __syncthreads();
    for (int i = 0; i < mine_n && warp % clusters == cluster; i += 32 * U) {
        int ex[U];
#pragma unroll
        for (int u = 0; u < U; ++u) ex[u] = next[u];
        load(i + 32 * U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = i + 32 * u + lane;
            if (s - lane >= mine_n) break;
            const bool live = (unsigned)ex[u] < (unsigned)E;
            if (live) atomicOr(&mine[ex[u]].y, 1 << lane);
            __syncwarp();
            int row = -1;
            int2 m = make_int2(0, 0);
            if (live) {
                m = mine[ex[u]];
                row = base[ex[u]] + m.x + __popc(m.y & ((1u << lane) - 1));
            }
            __syncwarp();
            if (live && lane == __ffs(m.y) - 1) mine[ex[u]] = make_int2(m.x + __popc(m.y), 0);
            __syncwarp();
            if (s < mine_n) {
                row_of[lo + s] = row;
                if (live) slot_of[row] = (int)(lo + s);
            }
        }
    }
    // a warp per segment's padding, and the rows after the last segment
    for (int e = blockIdx.x * (nt / 32) + warp; e < E && align > 1; e += gridDim.x * (nt / 32))
        for (long long r = (long long)pad[e].x + lane; r < pad[e].y; r += 32) slot_of[r] = -1;
    for (long long r = used + (long long)blockIdx.x * nt + tid; r < rows; r += gridDim.x * nt) slot_of[r] = -1;
    if constexpr (CLUSTER) ptx::cluster_sync();          // no block leaves while another may read its totals
}

cudaError_t launch_index(int n, int E, int align, const int32_t* topk, int32_t* counts, int32_t* offsets,
                         int32_t* row_of, int32_t* slot_of, int rows, cudaStream_t s)
{
    const int blocks = n <= kIndexOneBlock && rows <= kIndexOneBlockRows ? 1 : kIndexCluster;
    const int groups = (int)((n + 31ll) / 32);             // n is up to 2^31 - 3: sums next to it in 64 bits
    const int most = E <= 512 ? kIndexWarps : kIndexWarps / 2;       // of (count, lanes) pairs in shared memory
    int warps = (groups + 4 * blocks - 1) / (4 * blocks);
    warps = warps < 1 ? 1 : (warps > most ? most : warps);
    const int per = (groups + blocks * warps - 1) / (blocks * warps) * 32;
    // threads for the experts, and for the padding
    const int threads = align > 1 || E > 512 ? kIndexThreads : (32 * warps > E ? 32 * warps : (E + 31) / 32 * 32);
    const size_t smem = (size_t)E * ((warps + 1) * sizeof(int2) + 2 * sizeof(int));
    auto kernel = blocks == 1 ? sort_index_kernel<false> : sort_index_kernel<true>;
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kIndexSmem);
        if (e != cudaSuccess) return e;
    }
    const int clusters = blocks == 1 || n < 32768 ? 1 : (n >= 16 * 16384 ? 16 : n / 16384);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = blocks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks * clusters);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = blocks == 1 ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, topk, n, per, warps, E, align, counts, offsets, row_of, slot_of, rows);
}

// ------------------------------------------------------------------ rows
constexpr int kMoveThreads = 128;
// A row of at most two pieces per lane goes to a warp, four tokens to a block:
// 12906 x 4 rows of 344 bf16 combine in 11.1 us, 13.6 with a block per token.
constexpr int kNarrowPieces = 2;
// Up to this many tokens a block per token leaves SMs idle: rows are then cut
// into column parts (or, for the gradient's dot products, blocks are larger): 33
// tokens x 8 rows of 7168 go out in 2.7 us, 4.6 uncut; with many tokens the cut
// costs (8192 tokens back: 197 us in two parts, 192 whole).
constexpr int kFewTokens = 1216;
// Rows that one block of the padding part looks at.
constexpr int kPadRows = 32;

struct IndexArgs {
    int T, k, H;
    long long rows;
    const int32_t* row_of; const int32_t* slot_of; const int32_t* in_use;
};

// Pieces of 16 bytes. When every row starts on a 16-byte boundary and is a whole
// number of them (SHIFT false) a piece moves as it lies. Else pieces are cut at
// the destination's boundaries, and a source is read as the two aligned pieces
// around each, shifted together. The shift is the same along a row, so it costs
// a few instructions and no divergence. The columns before the first such piece
// and after the last whose two source pieces lie in the row (at most three
// pieces' worth) are moved by one lane each. 8192 x 8 rows of 4095 bf16 combine
// in 111 us (89%; 192 in 2-byte accesses, of 4098 148 in 4-byte ones), their
// gradient takes 273 (415, 266), 8634 x 8 rows of 3033 go out in 97 with their
// index (145).
//
// The cut of a destination row: its pieces whose two source pieces lie in the row.
template <typename T>
__device__ __forceinline__ Cut cut_row(const T* row, int H)
{
    constexpr int V = kPiece<T>;
    const int below = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    Cut c;
    c.head = below ? V - below : 0;
    c.n = H - V >= c.head + V ? (H - V - c.head) / V : 0;    // the last one's second source piece ends in the row
    if (c.n == 0) c.head = 0;                                // a narrow row is all edges
    c.edges = H - c.n * V;
    return c;
}

// The aligned pieces that hold columns [c, c + V) of a source row.
struct Pair { uint4 lo, hi; };
template <typename T>
__device__ __forceinline__ Pair load_pair(const T* row, int c)
{
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row + c) & ~(uintptr_t)15);
    return Pair{p[0], p[1]};
}
// The 16 bytes at row + c out of its pair.
template <typename T>
__device__ __forceinline__ uint4 shifted(const Pair& q, const T* row, int c)
{
    const int sh = (int)(reinterpret_cast<uintptr_t>(row + c) & 15);
    uint32_t w[8] = {q.lo.x, q.lo.y, q.lo.z, q.lo.w, q.hi.x, q.hi.y, q.hi.z, q.hi.w};
#pragma unroll
    for (int i = 0; i < 7; ++i) w[i] = sh & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = sh & 8 ? w[i + 2] : w[i];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = sh & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Zeros in the padding rows among [r0, r0 + kPadRows): every warp looks at all of
// their slots at once.
template <typename T, bool SHIFT>
__device__ __forceinline__ void zero_padding(const IndexArgs& ix, T* buf, long long ld, long long r0)
{
    constexpr int V = kPiece<T>;
    const long long used = *ix.in_use < ix.rows ? *ix.in_use : ix.rows;
    const int lane = threadIdx.x & 31;
    const bool padding = lane < kPadRows && r0 + lane < ix.rows && ix.slot_of[r0 + lane] < 0 && r0 + lane < used;
    for (unsigned m = __ballot_sync(0xffffffffu, padding); m; m &= m - 1) {
        T* row = buf + (r0 + __ffs(m) - 1) * ld;
        Cut cut{0, ix.H / V, 0};
        if constexpr (SHIFT) cut = cut_row(row, ix.H);
        for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < cut.n; i += gridDim.y * blockDim.x)
            store_raw<T, V>(row + cut.head + i * V, make_uint4(0, 0, 0, 0));
        if (SHIFT && blockIdx.y == 0)
            for (int e = threadIdx.x; e < cut.edges; e += blockDim.x) store_raw<T, 1>(row + edge_column<T>(cut, e), 0);
    }
}

// Row of slot j of token t, -1 if dropped or past k.
__device__ __forceinline__ int slot_row(const IndexArgs& ix, int t, int j)
{
    const int r = j < ix.k ? ix.row_of[(size_t)t * ix.k + j] : -1;
    return r < ix.rows ? r : -1;
}

// 32 bytes as one access.
struct Wide { uint32_t w[8]; };
__device__ __forceinline__ Wide load_wide(const void* p)
{
    Wide q;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(q.w[0]), "=r"(q.w[1]), "=r"(q.w[2]), "=r"(q.w[3]), "=r"(q.w[4]), "=r"(q.w[5]), "=r"(q.w[6]),
                   "=r"(q.w[7])
                 : "l"(p));
    return q;
}
__device__ __forceinline__ void store_wide(void* p, const Wide& q)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(q.w[0]), "r"(q.w[1]),
                 "r"(q.w[2]), "r"(q.w[3]), "r"(q.w[4]), "r"(q.w[5]), "r"(q.w[6]), "r"(q.w[7])
                 : "memory");
}

// sort_rows is launched while the kernel before it on the stream still runs and
// waits for its end (2 us of 204 behind the index): it reads by plain loads only,
// which see that kernel's stores, and takes no pointer as read-only.
//
// sort_rows for many tokens whose rows lie on 32-byte boundaries, in 32-byte
// accesses and larger blocks: 16384 tokens x 8 rows of 4096 bf16 take 191 us, 195
// in 16-byte ones (213 with blocks of 512 threads); 33 tokens gain nothing.
constexpr int kWideMove = 256;
template <typename T, int KM>
__global__ void __launch_bounds__(kWideMove)
sort_rows_wide_kernel(IndexArgs ix, const T* x, long long ldx, T* Xp, long long ldp)
{
    constexpr int V = 32 / (int)sizeof(T);
    const int t = blockIdx.x;
    ptx::griddep_wait();
    if (t >= ix.T) {
        zero_padding<T, false>(ix, Xp, ldp, (long long)(t - ix.T) * kPadRows);
        return;
    }
    const T* src = x + (size_t)t * ldx;
    for (int j0 = 0; j0 < ix.k; j0 += KM) {
        int row[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) row[j] = slot_row(ix, t, j0 + j);
        for (int i = threadIdx.x; i < ix.H / V; i += kWideMove) {
            const Wide q = load_wide(src + i * V);
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (row[j] >= 0) store_wide(Xp + row[j] * ldp + i * V, q);
        }
    }
}

// Blocks of T tokens, `per` to a block (without a sum that passes 32 bits).
__host__ __device__ constexpr int blocks_of(int T, int per) { return T / per + (T % per != 0); }
// Blocks of the tokens with GROUP threads a token.
template <int GROUP>
__host__ __device__ constexpr int token_blocks(int T) { return blocks_of(T, kMoveThreads / GROUP); }

// The first blocks: a token's row to its k rows, GROUP threads a token. The
// blocks after them: padding rows. 16384 tokens x 8 rows of 4096 bf16 with 7.7k
// padding rows: 195 us, 96% (nine tenths of it stores), 191 us and 98% in the
// wide kernel above.
template <typename T, bool SHIFT, int KM, int GROUP>
__global__ void __launch_bounds__(kMoveThreads)
sort_rows_kernel(IndexArgs ix, const T* x, long long ldx, T* Xp, long long ldp)
{
    constexpr int V = kPiece<T>;
    ptx::griddep_wait();
    if (blockIdx.x >= (unsigned)token_blocks<GROUP>(ix.T)) {
        zero_padding<T, SHIFT>(ix, Xp, ldp, (long long)(blockIdx.x - token_blocks<GROUP>(ix.T)) * kPadRows);
        return;
    }
    const int t = GROUP == 32 ? blockIdx.x * (kMoveThreads / 32) + threadIdx.x / 32 : blockIdx.x;
    const int tid = threadIdx.x % GROUP;
    if (t >= ix.T) return;
    const T* src = x + (size_t)t * ldx;
    for (int j0 = 0; j0 < ix.k; j0 += KM) {
        int row[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) row[j] = slot_row(ix, t, j0 + j);
        if constexpr (!SHIFT) {
            for (int i = blockIdx.y * GROUP + tid; i < ix.H / V; i += gridDim.y * GROUP) {
                const uint4 q = load_raw<T, V>(src + i * V);
#pragma unroll
                for (int j = 0; j < KM; ++j)
                    if (row[j] >= 0) store_raw<T, V>(Xp + row[j] * ldp + i * V, q);
            }
        } else {
            for (int i = blockIdx.y * GROUP + tid; i <= ix.H / V; i += gridDim.y * GROUP) {
                constexpr int B = KM < 4 ? KM : 4;           // rows loaded together
#pragma unroll
                for (int h = 0; h < KM; h += B) {
                    Pair q[B];
#pragma unroll
                    for (int j = 0; j < B; ++j) {
                        const Cut cut = cut_row(Xp + row[h + j] * ldp, ix.H);
                        if (row[h + j] >= 0 && i < cut.n) q[j] = load_pair(src, cut.head + i * V);
                    }
#pragma unroll
                    for (int j = 0; j < B; ++j) {
                        T* dst = Xp + row[h + j] * ldp;
                        const Cut cut = cut_row(dst, ix.H);
                        const int c = cut.head + i * V;
                        if (row[h + j] >= 0 && i < cut.n) store_raw<T, V>(dst + c, shifted(q[j], src, c));
                    }
                }
            }
            // lane e of a warp: the e-th edge of each of its rows
            if (blockIdx.y == 0)
                for (int j = tid / 32; j < KM; j += GROUP / 32) {
                    const int r = slot_row(ix, t, j0 + j);
                    if (r < 0) continue;
                    T* dst = Xp + r * ldp;
                    const Cut cut = cut_row(dst, ix.H);
                    for (int e = tid % 32; e < cut.edges; e += 32) {
                        const int c = edge_column<T>(cut, e);
                        store_raw<T, 1>(dst + c, load_raw<T, 1>(src + c));
                    }
                }
        }
    }
}

// y[t] = residual[t] + sum over the slots in order of g Yp[row]. WHOLE: k <= KM,
// the index is read once per token. 8192 x 8 rows of 7168 bf16 with residual:
// 166 us, 104% of the copy rate (mostly reads); the row numbers in 32 bits leave
// 64 registers and eight blocks an SM (192 us with 88).
template <typename T, bool SHIFT, int KM, bool WHOLE, int GROUP>
__global__ void __launch_bounds__(kMoveThreads)
unsort_rows_kernel(IndexArgs ix, const T* __restrict__ Yp, long long ldp, const float* __restrict__ gates,
                   const T* residual, long long ldr, T* y, long long ldy)
{
    constexpr int V = kPiece<T>;
    const int t = GROUP == 32 ? blockIdx.x * (kMoveThreads / 32) + threadIdx.x / 32 : blockIdx.x;
    const int tid = threadIdx.x % GROUP;
    if (t >= ix.T) return;
    int row[KM];
    float g[KM];
    auto index = [&](int j0) {
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            row[j] = slot_row(ix, t, j0 + j);
            g[j] = gates && j0 + j < ix.k ? gates[(size_t)t * ix.k + j0 + j] : 1.f;
        }
    };
    if (WHOLE) index(0);
    T* out = y + (size_t)t * ldy;
    const T* res_row = residual ? residual + (size_t)t * ldr : nullptr;
    Cut cut{0, ix.H / V, 0};
    if constexpr (SHIFT) {
        cut = cut_row(out, ix.H);
        if (blockIdx.y == 0)
            for (int e = tid; e < cut.edges; e += GROUP) {
                const int c = edge_column<T>(cut, e);
                float v[1], acc[1] = {0.f};
                if (residual) load_vec<T, 1>(res_row + c, acc);
#pragma unroll 8
                for (int j = 0; j < ix.k; ++j) {
                    const int r = slot_row(ix, t, j);
                    if (r < 0) continue;
                    load_vec<T, 1>(Yp + r * ldp + c, v);
                    acc[0] = fmaf(gates ? gates[(size_t)t * ix.k + j] : 1.f, v[0], acc[0]);
                }
                store_vec<T, 1>(out + c, acc);
            }
    }
    for (int i = blockIdx.y * GROUP + tid; i < cut.n; i += gridDim.y * GROUP) {
        const int c = cut.head + i * V;
        float acc[V];
#pragma unroll
        for (int n = 0; n < V; ++n) acc[n] = 0.f;
        Pair res2;
        uint4 res;
        if (residual) {
            if constexpr (SHIFT) res2 = load_pair(res_row, c);
            else res = load_raw<T, V>(res_row + c);
        }
        for (int j0 = 0; j0 < (WHOLE ? 1 : ix.k); j0 += KM) {
            if (!WHOLE) index(j0);
            constexpr int B = SHIFT && KM > 4 ? 4 : KM;      // rows loaded together
#pragma unroll
            for (int h = 0; h < KM; h += B) {
                uint4 q[B];
                Pair q2[SHIFT ? B : 1];
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if (row[h + j] >= 0) {
                        if constexpr (SHIFT) q2[j] = load_pair(Yp + row[h + j] * ldp, c);
                        else q[j] = load_raw<T, V>(Yp + row[h + j] * ldp + c);
                    }
                if (j0 == 0 && h == 0 && residual) {
                    if constexpr (SHIFT) res = shifted(res2, res_row, c);
                    unpack<T, V>(res, acc);
                }
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    if (row[h + j] < 0) continue;
                    float v[V];
                    if constexpr (SHIFT) q[j] = shifted(q2[j], Yp + row[h + j] * ldp, c);
                    unpack<T, V>(q[j], v);
#pragma unroll
                    for (int n = 0; n < V; ++n) acc[n] = fmaf(g[h + j], v[n], acc[n]);
                }
            }
        }
        store_vec<T, V>(out + c, acc);
    }
}

// The first blocks: dYp[row_j] = g_j dY[t] and dg_j = <dY[t], Yp[row_j]>, GROUP
// (a warp, or NT) threads a token. The blocks after them: padding rows. 16384 x
// 8 rows of 4096 bf16: 335 us with the padding, 98%. Shifted rows of more than four
// slots do not fit the 80 registers that six blocks an SM leave (up to 252 bytes
// spilled): part of what 8192 x 8 rows of 4095 take, 271 us, 62%.
template <typename T, bool SHIFT, int KM, int NT, int GROUP, bool DG>
__global__ void __launch_bounds__(NT, NT == kMoveThreads ? 6 : 1)
unsort_bwd_kernel(IndexArgs ix, const T* __restrict__ dY, long long lddy, const T* Yp, long long ldp,
                  const float* __restrict__ gates, T* dYp, long long ldd, float* __restrict__ dgates)
{
    constexpr int V = kPiece<T>;
    constexpr int TOKENS = NT / GROUP;       // of a block
    const int tb = blocks_of(ix.T, TOKENS);
    if (blockIdx.x >= (unsigned)tb) {
        zero_padding<T, SHIFT>(ix, dYp, ldd, (long long)(blockIdx.x - tb) * kPadRows);
        return;
    }
    __shared__ float red[NT / 32][KM];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x % GROUP;
    const int t = blockIdx.x * TOKENS + threadIdx.x / GROUP;
    if (t >= ix.T) return;                   // a block, or whole warps that meet no barrier
    for (int j0 = 0; j0 < ix.k; j0 += KM) {
        int row[KM];
        float g[KM], dot[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            row[j] = slot_row(ix, t, j0 + j);
            g[j] = gates && j0 + j < ix.k ? gates[(size_t)t * ix.k + j0 + j] : 1.f;
            dot[j] = 0.f;
        }
        const T* dy = dY + (size_t)t * lddy;
        for (int i = tid; i < ix.H / V + (SHIFT ? 1 : 0); i += GROUP) {
            if constexpr (!SHIFT) {
                float d[V];
                load_vec<T, V>(dy + i * V, d);
                // four rows' loads at a time: with all eight in flight fewer blocks fit
                // (347 against 339 us when this was measured)
                constexpr int B = KM < 4 ? KM : 4;
#pragma unroll
                for (int h = 0; h < KM; h += B) {
                    uint4 q[B];
                    if constexpr (DG) {
#pragma unroll
                        for (int j = 0; j < B; ++j)
                            if (row[h + j] >= 0) q[j] = load_raw<T, V>(Yp + row[h + j] * ldp + i * V);
                    }
#pragma unroll
                    for (int j = 0; j < B; ++j) {
                        if (row[h + j] < 0) continue;
                        float o[V];
                        if constexpr (DG) {
                            float v[V];
                            unpack<T, V>(q[j], v);
#pragma unroll
                            for (int n = 0; n < V; ++n) dot[h + j] = fmaf(d[n], v[n], dot[h + j]);
                        }
#pragma unroll
                        for (int n = 0; n < V; ++n) o[n] = g[h + j] * d[n];
                        store_vec<T, V>(dYp + row[h + j] * ldd + i * V, o);
                    }
                }
            } else {
                constexpr int B = KM < 2 ? KM : 2;           // rows loaded together
#pragma unroll
                for (int h = 0; h < KM; h += B) {
                    Pair qd[B], qy[DG ? B : 1];
#pragma unroll
                    for (int j = 0; j < B; ++j) {
                        const Cut cut = cut_row(dYp + row[h + j] * ldd, ix.H);
                        if (row[h + j] >= 0 && i < cut.n) {
                            qd[j] = load_pair(dy, cut.head + i * V);
                            if constexpr (DG) qy[j] = load_pair(Yp + row[h + j] * ldp, cut.head + i * V);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < B; ++j) {
                        T* out = dYp + row[h + j] * ldd;
                        const Cut cut = cut_row(out, ix.H);
                        if (row[h + j] < 0 || i >= cut.n) continue;
                        const int c = cut.head + i * V;
                        float d[V];
                        unpack<T, V>(shifted(qd[j], dy, c), d);
                        if constexpr (DG) {
                            float v[V];
                            unpack<T, V>(shifted(qy[j], Yp + row[h + j] * ldp, c), v);
#pragma unroll
                            for (int n = 0; n < V; ++n) dot[h + j] = fmaf(d[n], v[n], dot[h + j]);
                        }
#pragma unroll
                        for (int n = 0; n < V; ++n) d[n] *= g[h + j];
                        store_vec<T, V>(out + c, d);
                    }
                }
            }
        }
        if constexpr (SHIFT) {
            // lane e of a warp: the e-th edge of each of its rows
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                if (row[j] < 0 || (GROUP != 32 && j % (GROUP / 32) != warp)) continue;
                T* out = dYp + row[j] * ldd;
                const Cut cut = cut_row(out, ix.H);
                for (int e = lane; e < cut.edges; e += 32) {
                    const int c = edge_column<T>(cut, e);
                    float d[1], v[1];
                    load_vec<T, 1>(dy + c, d);
                    if constexpr (DG) {
                        load_vec<T, 1>(Yp + row[j] * ldp + c, v);
                        dot[j] = fmaf(d[0], v[0], dot[j]);
                    }
                    d[0] *= g[j];
                    store_vec<T, 1>(out + c, d);
                }
            }
        }
        if constexpr (DG) {
            if constexpr (GROUP != 32) __syncthreads();      // red of the previous slots is read
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                float s = dot[j];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                if (GROUP != 32 && lane == 0) red[warp][j] = s;
                if (GROUP == 32 && lane == 0 && j0 + j < ix.k) dgates[(size_t)t * ix.k + j0 + j] = s;
            }
            if constexpr (GROUP != 32) {
                __syncthreads();
                if (threadIdx.x < KM && j0 + (int)threadIdx.x < ix.k) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < NT / 32; ++w) s += red[w][threadIdx.x];
                    dgates[(size_t)t * ix.k + j0 + threadIdx.x] = s;
                }
            }
        }
    }
}

// Calls F with the slot bound of k: 1, 2, 4 or 8 rows at a time.
constexpr int kMaxSlots = 8;
template <typename F>
void with_slots(int k, F&& f)
{
    if (k <= 1) f(std::integral_constant<int, 1>{});
    else if (k <= 2) f(std::integral_constant<int, 2>{});
    else if (k <= 4) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, kMaxSlots>{});
}
// Calls F with whether rows have to be shifted: some stride or the width is not
// a whole number of 16-byte pieces.
template <typename T, typename F>
void with_shift(const moe_sorted_t& ix, std::initializer_list<long long> strides, F&& f)
{
    if (rows_start<T>(ix.H, strides) == Rows::kWhole) f(std::false_type{});
    else f(std::true_type{});
}

IndexArgs index_args(const moe_sorted_t& s)
{
    return IndexArgs{s.T, s.k, s.H, s.rows, s.row_of, s.slot_of, s.in_use};
}
// Blocks of a launch with GROUP threads a token, padding included.
unsigned move_grid(const moe_sorted_t& s, int token_blocks)
{
    return (unsigned)(token_blocks + (s.slot_of ? (s.rows + kPadRows - 1) / kPadRows : 0));
}
// Whether a token's row goes to a warp: few pieces, and enough tokens that the
// larger blocks are not needed to fill the SMs.
template <typename T>
bool narrow(const moe_sorted_t& s) { return s.H <= 32 * kPiece<T> * kNarrowPieces && s.T >= kFewTokens; }

using One = std::integral_constant<int, 32>;
using Block = std::integral_constant<int, kMoveThreads>;

// Column parts of a launch.
template <typename T>
unsigned column_parts(const moe_sorted_t& s)
{
    const int part = kMoveThreads * kPiece<T>, most = (s.H + part - 1) / part;
    const int wanted = s.T > 0 ? (kFewTokens + s.T - 1) / s.T : 1;
    return (unsigned)(s.T >= kFewTokens ? 1 : (wanted < most ? wanted : most));
}

template <typename T>
cudaError_t sort_rows(const moe_sorted_t& ix, const void* x, long long ldx, void* Xp, long long ldp, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    with_shift<T>(ix, {ldx, ldp}, [&](auto shift) {
        with_slots(ix.k, [&](auto km) {
            auto launch = [&](auto group) {
                constexpr int G = decltype(group)::value;
                e = launch_early(sort_rows_kernel<T, decltype(shift)::value, decltype(km)::value, G>,
                                 dim3(move_grid(ix, token_blocks<G>(ix.T)), column_parts<T>(ix)), dim3(kMoveThreads), s,
                                 index_args(ix), static_cast<const T*>(x), ldx, static_cast<T*>(Xp), ldp);
            };
            if constexpr (!decltype(shift)::value) {
                const uintptr_t low = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(Xp);
                const long long off = (ix.H | ldx | ldp) * (long long)sizeof(T);
                if (ix.T >= kFewTokens && !narrow<T>(ix) && ((low | (uintptr_t)off) & 31) == 0) {
                    e = launch_early(sort_rows_wide_kernel<T, decltype(km)::value>, dim3(move_grid(ix, ix.T)),
                                     dim3(kWideMove), s, index_args(ix), static_cast<const T*>(x), ldx,
                                     static_cast<T*>(Xp), ldp);
                    return;
                }
            }
            if (narrow<T>(ix)) launch(One{});
            else launch(Block{});
        });
    });
    return e;
}

template <typename T>
void unsort_rows(const moe_sorted_t& ix, const void* Yp, long long ldp, const float* gates, const void* residual,
                 long long ldr, void* y, long long ldy, cudaStream_t s)
{
    with_shift<T>(ix, {ldp, ldy, residual ? ldr : ldy}, [&](auto shift) {
        with_slots(ix.k, [&](auto km) {
            constexpr int KM = decltype(km)::value;
            auto launch = [&](auto whole, auto group) {
                constexpr int G = decltype(group)::value;
                unsort_rows_kernel<T, decltype(shift)::value, KM, decltype(whole)::value, G>
                    <<<dim3(token_blocks<G>(ix.T), column_parts<T>(ix)), kMoveThreads, 0, s>>>(
                        index_args(ix), static_cast<const T*>(Yp), ldp, gates, static_cast<const T*>(residual), ldr,
                        static_cast<T*>(y), ldy);
            };
            if (ix.k > KM) {
                if constexpr (KM == kMaxSlots) launch(std::false_type{}, Block{});
            } else if (narrow<T>(ix)) {
                launch(std::true_type{}, One{});
            } else {
                launch(std::true_type{}, Block{});
            }
        });
    });
}

template <typename T>
void unsort_bwd(const moe_sorted_t& ix, const void* dY, long long lddy, const void* Yp, long long ldp,
                const float* gates, void* dYp, long long ldd, float* dgates, cudaStream_t s)
{
    with_shift<T>(ix, {lddy, ldd, dgates ? ldp : ldd}, [&](auto shift) {
        with_slots(ix.k, [&](auto km) {
            constexpr int KM = decltype(km)::value;
            auto launch = [&](auto nt, auto group, auto dg) {
                constexpr int NT = decltype(nt)::value, G = decltype(group)::value;
                unsort_bwd_kernel<T, decltype(shift)::value, KM, NT, G, decltype(dg)::value>
                    <<<move_grid(ix, blocks_of(ix.T, NT / G)), NT, 0, s>>>(
                        index_args(ix), static_cast<const T*>(dY), lddy, static_cast<const T*>(Yp), ldp, gates,
                        static_cast<T*>(dYp), ldd, dgates);
            };
            using Large = std::integral_constant<int, 512>;
            // narrow rows by warps here too: a block for each of 2^31 tokens, and the
            // padding's behind them, are more than a grid holds (32768 x 8 rows of 128
            // bf16 without gates' gradient: 18.1 us, 32.0 by blocks)
            if (!dgates && narrow<T>(ix)) launch(Block{}, One{}, std::false_type{});
            else if (!dgates) launch(Block{}, Block{}, std::false_type{});
            else if (narrow<T>(ix)) launch(Block{}, One{}, std::true_type{});
            else if (ix.T < kFewTokens / 2) launch(Large{}, Large{}, std::true_type{});
            else launch(Block{}, Block{}, std::true_type{});
        });
    });
}

long long rows_cap(int T, int k, int E, int align)
{
    const long long n = (long long)T * k;
    return (n + (n < E ? n : E) * (align - 1) + align - 1) / align * align;
}

bool sort_args_ok(int T, int k, int E, int align)
{
    return T >= 0 && k >= 1 && k <= kSortMaxK && E >= 1 && E <= kSortMaxE && align >= 1 &&
           align <= kSortMaxAlign && rows_cap(T, k, E, align) < (1ll << 31) - 1;
}

// The checks that the movers share; MOE_OK if the index can be used.
moe_status_t check_index(const moe_sorted_t* ix, bool writes_rows)
{
    if (!ix || ix->T < 0 || ix->k < 1 || ix->k > kSortMaxK || ix->H < 1 || ix->H > kSortMaxH || ix->rows < 0 ||
        ix->rows >= (1ll << 31) - 1 || (long long)ix->T * ix->k >= (1ll << 31) - 1 ||
        (ix->dtype != MOE_FP32 && ix->dtype != MOE_BF16))
        return MOE_ERR_INVALID_ARG;
    if (ix->T > 0 && !ix->row_of) return MOE_ERR_INVALID_ARG;
    if (writes_rows && ix->slot_of && !ix->in_use) return MOE_ERR_INVALID_ARG;
    if (!is_aligned16(ix->row_of) || !is_aligned16(ix->slot_of) ||
        (reinterpret_cast<uintptr_t>(ix->in_use) & 3u))
        return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

moe_status_t launched()
{
    count_launches();
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

moe_status_t moe_sort_rows_cap(int T, int k, int E, int align, long long* rows)
{
    if (!rows || !sort_args_ok(T, k, E, align)) return MOE_ERR_INVALID_ARG;
    *rows = rows_cap(T, k, E, align);
    return MOE_OK;
}

moe_status_t moe_sort_index(int T, int k, int E, int align, const int32_t* topk, int32_t* counts,
                            int32_t* offsets, int32_t* row_of, int32_t* slot_of, long long rows,
                            moe_stream_t stream)
{
    if (!sort_args_ok(T, k, E, align) || rows < rows_cap(T, k, E, align) || rows >= (1ll << 31) - 1 ||
        !counts || !offsets || (T > 0 && (!topk || !row_of)) || (rows > 0 && !slot_of))
        return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {topk, counts, offsets, row_of, slot_of};
    for (const void* p : ptrs)
        if (!is_aligned16(p)) return MOE_ERR_MISALIGNED;
    if (launch_index(T * k, E, align, topk, counts, offsets, row_of, slot_of, (int)rows,
                     reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return MOE_ERR_CUDA;
    return launched();
}

moe_status_t moe_sort_rows(const moe_sorted_t* index, const void* x, long long ldx, void* Xp,
                           long long ldp, moe_stream_t stream)
{
    const moe_status_t st = check_index(index, true);
    if (st != MOE_OK) return st;
    const moe_sorted_t& ix = *index;
    if (ix.T > 0 && !x) return MOE_ERR_INVALID_ARG;
    if ((ix.rows > 0 && !Xp) || ldx < ix.H || ldp < ix.H) return MOE_ERR_INVALID_ARG;
    if (!is_aligned16(x) || !is_aligned16(Xp)) return MOE_ERR_MISALIGNED;
    if (ix.rows == 0 || (ix.T == 0 && !ix.slot_of)) return MOE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = ix.dtype == MOE_FP32 ? sort_rows<float>(ix, x, ldx, Xp, ldp, s)
                                               : sort_rows<__nv_bfloat16>(ix, x, ldx, Xp, ldp, s);
    count_launches();
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_unsort_rows(const moe_sorted_t* index, const void* Yp, long long ldp,
                             const float* gates, const void* residual, long long ldr, void* y,
                             long long ldy, moe_stream_t stream)
{
    const moe_status_t st = check_index(index, false);
    if (st != MOE_OK) return st;
    const moe_sorted_t& ix = *index;
    if ((ix.rows > 0 && !Yp) || (ix.T > 0 && !y) || ldp < ix.H || ldy < ix.H || (residual && ldr < ix.H))
        return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {Yp, gates, residual, y};
    for (const void* p : ptrs)
        if (!is_aligned16(p)) return MOE_ERR_MISALIGNED;
    if (ix.T == 0) return MOE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (ix.dtype == MOE_FP32) unsort_rows<float>(ix, Yp, ldp, gates, residual, ldr, y, ldy, s);
    else unsort_rows<__nv_bfloat16>(ix, Yp, ldp, gates, residual, ldr, y, ldy, s);
    return launched();
}

moe_status_t moe_unsort_rows_backward(const moe_sorted_t* index, const void* dY, long long lddy,
                                      const void* Yp, long long ldp, const float* gates, void* dYp,
                                      long long ldd, float* dgates, moe_stream_t stream)
{
    const moe_status_t st = check_index(index, true);
    if (st != MOE_OK) return st;
    const moe_sorted_t& ix = *index;
    if ((ix.T > 0 && !dY) || (ix.rows > 0 && (!dYp || (dgates && !Yp))) || lddy < ix.H || ldd < ix.H ||
        (dgates && ldp < ix.H))
        return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {dY, Yp, gates, dYp, dgates};
    for (const void* p : ptrs)
        if (!is_aligned16(p)) return MOE_ERR_MISALIGNED;
    if (ix.T == 0 && (ix.rows == 0 || !ix.slot_of)) return MOE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (ix.dtype == MOE_FP32) unsort_bwd<float>(ix, dY, lddy, Yp, ldp, gates, dYp, ldd, dgates, s);
    else unsort_bwd<__nv_bfloat16>(ix, dY, lddy, Yp, ldp, gates, dYp, ldd, dgates, s);
    return launched();
}
