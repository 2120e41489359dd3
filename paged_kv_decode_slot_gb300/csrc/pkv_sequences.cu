// pkv_sequences.cu - the life of a paged cache's blocks on the device: sequences forked and freed, extended by new
// tokens (with copies on write), blocks compacted, and the copies that these ask for, in the pools of every layer at once.
//
// The state is a count per physical block of the table rows that hold it; a block with count 0 is free.  There is no free
// list to keep in order: a call that hands out blocks takes the free ones in ascending order, so that its result follows
// from its inputs alone, whatever ran before and however the work is split.  Everything is integers and exact.
//
// What bounds these: a scan of the counts (4 bytes a block: 0.4 MB for 100,000 blocks) and the table entries that change,
// both from L2; the rest is the latency of a launch, of dependent loads and of a few barriers.  Scans run as one CTA or, of many
// blocks, as one cluster of eight, whose totals meet in shared memory, rather than as a grid that would have to be launched
// twice or count itself.  Measured inside CUDA graphs: 64 rows extended over 21,797 blocks 6.4 us, 250 rows of up to 700 new
// tokens over 68,943 blocks 13.9; 64 beams forked 4.2 us, 250 rows of 1,001 to 2,033 blocks 8.0;
// the plan of 20 rows' moves among 10,898 blocks 10 us with the tables' entries; copies 6.5 TB/s, 96% of a plain copy's rate.
#include <limits.h>

#include "pkv_cluster.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_sequences.h"

namespace pkv {

// ---- forking --------------------------------------------------------------------------------------
constexpr int kForkThreads = 256;
constexpr int kForkEntries = kSequenceEntries;  // table entries of a CTA (250 rows of up to 2,033: 8.0 us with 512, 8.2 with 1,024, 10.1 with 2,048)
constexpr int kForkEach = kForkEntries / kForkThreads;

__device__ __forceinline__ int fork_blocks(const ForkParams &p, int row, bool report, int &ctx)
{
    ctx = p.context_lens[row];
    if (ctx < 0 || ctx > p.max_nb * kBlockSize) {
        if (report) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        ctx = 0;
    }
    return (ctx + kBlockSize - 1) / kBlockSize;
}

// CTA (x, y): entries [y * kForkEntries, ..) of new row x, or, from rows_out on, of old row x - rows_out, whose blocks gain
// as many holders as rows take it over and lose one.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const ForkParams p)
{
    const int tid = threadIdx.x, e0 = blockIdx.y * kForkEntries, e1 = min(p.max_nb, e0 + kForkEntries);
    pdl_wait_primary();
    pdl_launch_dependents();
    int ctx;
    if ((int)blockIdx.x < p.rows_out) {
        const int row = blockIdx.x;
        int from = p.parents[row];
        const bool report = tid == 0 && blockIdx.y == 0;
        if (from < -1 || from >= p.rows_in) {
            if (report) set_flag(p.err_flag, PKV_FLAG_SEQ_RANGE);
            from = -1;
        }
        int nb = 0;
        ctx = 0;
        if (from >= 0) nb = fork_blocks(p, from, false, ctx);
        const int32_t *src = p.block_tables + (int64_t)from * p.max_nb;
        int32_t *dst = p.tables_out + (int64_t)row * p.max_nb;
        int id[kForkEach];
#pragma unroll
        for (int k = 0; k < kForkEach; ++k) {
            const int e = e0 + tid + k * kForkThreads;
            id[k] = e < min(e1, nb) ? src[e] : -1;
        }
#pragma unroll
        for (int k = 0; k < kForkEach; ++k) {
            const int e = e0 + tid + k * kForkThreads;
            if (e < e1) dst[e] = id[k];
        }
        if (report) p.lens_out[row] = ctx;
        return;
    }
    const int row = blockIdx.x - p.rows_out;
    const int nb = min(e1, fork_blocks(p, row, tid == 0 && blockIdx.y == 0, ctx));
    if (nb <= e0) return;
    int mine = 0;
    for (int r = tid; r < p.rows_out; r += kForkThreads) mine += p.parents[r] == row;
    // heirs, a block-wide sum
    __shared__ int sums[kForkThreads / 32];
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    if ((tid & 31) == 0) sums[tid >> 5] = mine;
    __syncthreads();
    int change = -1;
#pragma unroll
    for (int w = 0; w < kForkThreads / 32; ++w) change += sums[w];
    if (change == 0) return;
    const int32_t *src = p.block_tables + (int64_t)row * p.max_nb;
    // all of a thread's entries, then all of its additions, under way at once
    int id[kForkEach], left[kForkEach];
#pragma unroll
    for (int k = 0; k < kForkEach; ++k) {
        const int e = e0 + tid + k * kForkThreads;
        id[k] = e < nb ? src[e] : INT_MIN;
    }
#pragma unroll
    for (int k = 0; k < kForkEach; ++k) left[k] = id[k] >= 0 && id[k] < p.num_blocks ? atomicAdd(p.ref_counts + id[k], change) + change : 0;
#pragma unroll
    for (int k = 0; k < kForkEach; ++k) {
        if (id[k] != INT_MIN && (id[k] < 0 || id[k] >= p.num_blocks)) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
        if (left[k] < 0) set_flag(p.err_flag, PKV_FLAG_REF_RANGE);
    }
}

cudaError_t launch_fork_sequences(const ForkParams &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.rows_out + p.rows_in), (unsigned)((p.max_nb + kForkEntries - 1) / kForkEntries));
    return launch_kernel(fork_kernel, grid, dim3(kForkThreads), 0, stream, true, p);
}

// A list of pairs of integers (4-byte aligned, as the caller's tensors are).
struct PairList {
    int32_t *at;
    __device__ __forceinline__ int2 get(int64_t i) const { return make_int2(__ldcg(at + 2 * i), __ldcg(at + 2 * i + 1)); }
    __device__ __forceinline__ void put(int64_t i, int2 v) const { at[2 * i] = v.x, at[2 * i + 1] = v.y; }
};

// ---- a cluster that scans the counts ----------------------------------------------------------------
constexpr int kScanThreads = 1024, kScanWarps = kScanThreads / 32;
constexpr int kScanCtas = 8;         // CTAs of the cluster ..
// .. or one CTA, whose barriers cost less, where it reads the counts as fast as it needs them: extensions of up to this many
// rows and blocks (64 rows over 21,797 blocks 9.9 -> 7.4 us; 250 over 68,943 15.8 -> 24.6), plans of moves, which read them
// twice, in small pools (10,898 blocks 10.1 -> 12.2)
constexpr int kOneCtaBlocks = 32768, kOneCtaRows = kScanThreads, kOneCtaPlan = 4096;

// Warp w of the kCtas * 32 takes the counts [w * per_warp, (w + 1) * per_warp), 128 a step.
struct ScanRange {
    int begin, end;
};
template <int kCtas>
__device__ __forceinline__ ScanRange scan_range(int num_blocks, int rank)
{
    const int warps = kCtas * kScanWarps, w = rank * kScanWarps + (threadIdx.x >> 5);
    const int steps = (num_blocks + 127) / 128, per = (steps + warps - 1) / warps;
    const int64_t b = (int64_t)w * per * 128, e = b + (int64_t)per * 128;
    return ScanRange{(int)min((int64_t)num_blocks, b), (int)min((int64_t)num_blocks, e)};
}

// Which of the 32 counts from each of at, at + 32, at + 64, at + 96 are zero (free); behind the end none.
__device__ __forceinline__ void scan_free(const int32_t *counts, int at, int end, unsigned (&free)[4])
{
    const int i = at + (threadIdx.x & 31);
    int v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + 32 * j < end ? __ldcg(counts + i + 32 * j) : 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) free[j] = __ballot_sync(0xFFFFFFFFu, v[j] == 0);
}

__device__ __forceinline__ unsigned lanes_below() { return (1u << (threadIdx.x & 31)) - 1u; }

// Exclusive sum over a warp's lanes.
__device__ __forceinline__ int warp_before(int v, int &all)
{
    int s = v;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += up;
    }
    all = __shfl_sync(0xFFFFFFFFu, s, 31);
    return s - v;
}

// Free counts of a warp's range.
__device__ __forceinline__ int count_free(const int32_t *counts, ScanRange r)
{
    int n = 0;
#pragma unroll 4
    for (int at = r.begin; at < r.end; at += 128) {
        unsigned free[4];
        scan_free(counts, at, r.end, free);
#pragma unroll
        for (int j = 0; j < 4; ++j) n += __popc(free[j]);
    }
    return n;
}

// Exclusive prefix, over the CTA's warps, of one value a warp (given by every lane); the CTA's total.  Every thread.
__device__ __forceinline__ int cta_warps_before(int v, int *sums, int &all)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    const int before = warp_before(sums[lane], all);
    return __shfl_sync(0xFFFFFFFFu, before, warp);
}

// A barrier of all CTAs: what they wrote before it, to global or their shared memory, is seen behind it.
template <int kCtas>
__device__ __forceinline__ void scan_sync()
{
    if constexpr (kCtas > 1) cluster_sync();
    else __syncthreads();
}

// The values that every CTA published in `words` before a barrier, each summed before this one and over all.  Whole warps; a
// word's CTAs are read by a lane each (one after the other they take 0.1 us a word), the words' reads are under way at once.
template <int kCtas, int kWords>
__device__ __forceinline__ void cluster_before(const long long *words, int rank, long long (&before)[kWords], long long (&all)[kWords])
{
    if constexpr (kCtas == 1) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) before[w] = 0, all[w] = words[w];
    } else {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int w = 0; w < kWords; ++w) all[w] = lane < kCtas ? load_cluster<long long>(smem_u32(words + w), lane) : 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            before[w] = lane < rank ? all[w] : 0;
#pragma unroll
            for (int o = kCtas / 2; o; o >>= 1) {
                all[w] += __shfl_xor_sync(0xFFFFFFFFu, all[w], o);
                before[w] += __shfl_xor_sync(0xFFFFFFFFu, before[w], o);
            }
            all[w] = __shfl_sync(0xFFFFFFFFu, all[w], 0);
            before[w] = __shfl_sync(0xFFFFFFFFu, before[w], 0);
        }
    }
}

template <int kCtas>
__device__ __forceinline__ int scan_rank()
{
    uint32_t r = 0;
    if constexpr (kCtas > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}

// ---- extending --------------------------------------------------------------------------------------
// Rows in order.  A row that grows into a partly filled block needs that block for itself: where other rows hold it too
// (count above 1) it takes a fresh one and a copy is asked for, unless all the other holders grow in this call as well and
// come before it.  To find that out without order, every such row first takes itself off the count; a count that reaches
// zero had no other holders, and its last row, found by an atomic minimum over -(row + 1) in the count itself, keeps the
// block.  Then a scan over what the rows need says who gets which of the free blocks.
//
// A thread keeps its row's state in registers (`per` is 1 up to 8,192 rows) or in the row's entry of `copies`, which also
// tells the warps of rows with many fresh blocks: (block to copy, or one of the marks below; first rank of its fresh blocks).
// The last barrier is the one behind which free blocks are known: threads and warps then hand them out side by side (with
// states in registers; 250 rows over 68,943 blocks 14.6 -> 13.9 us against one barrier more).
constexpr int kNoCopy = -1, kKeeps = -2, kIdle = -3;
constexpr int kWaits = INT_MIN;  // + 1 + the block to copy: a row whose fresh blocks a warp hands out
constexpr int kFewBlocks = 4;  // fresh blocks that a row's own thread writes; more are a warp's work

struct GrowRow {
    int ctx, now, then;   // tokens, blocks before and after
};
__device__ __forceinline__ GrowRow grow_row(const ExtendParams &p, int row)
{
    GrowRow g;
    g.ctx = p.context_lens[row];
    const int64_t to = (int64_t)g.ctx + p.num_new[row];
    g.now = (g.ctx + kBlockSize - 1) / kBlockSize;
    g.then = (int)((to + kBlockSize - 1) / kBlockSize);
    return g;
}

// Gives row `row` its fresh blocks k0, k0 + step, .. of n, which replace or follow those up to entry `at` of its table.
__device__ __forceinline__ void give_blocks(const ExtendParams &p, int row, int at, int n, int first, int k0, int step, int cow_of)
{
    int32_t *tbl = p.block_tables + (int64_t)row * p.max_nb + at;
    for (int k = k0; k < n; k += step) {
        const int id = __ldcg(p.free_ids + first + k);
        if (id < 0 || id >= p.num_blocks) {  // only where counts and tables disagree
            set_flag(p.err_flag, PKV_FLAG_REF_RANGE);
            continue;
        }
        tbl[k] = id;
        p.ref_counts[id] = 1;
        if (k == 0 && cow_of >= 0) PairList{p.copies}.put(row, make_int2(cow_of, id));
    }
}

template <int kCtas>
__global__ void __launch_bounds__(kScanThreads, 1) extend_kernel(const ExtendParams p)
{
    __shared__ int sums[kScanWarps];
    __shared__ long long here[3];  // free blocks of this CTA's range, blocks its rows need, whether one needs many
    __shared__ long long warp_need[kScanWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = scan_rank<kCtas>();
    const PairList state{p.copies};
    // this thread's rows
    const int threads = kCtas * kScanThreads, per = (p.rows + threads - 1) / threads;
    const int64_t r0 = (int64_t)(rank * kScanThreads + tid) * per;
    const int rb = (int)min((int64_t)p.rows, r0), re = (int)min((int64_t)p.rows, r0 + per);
    const bool one = per == 1;
    int2 mine_state = make_int2(kIdle, 0);
    GrowRow mine_row = {};
    auto get = [&](int row) { return one ? mine_state : state.get(row); };
    auto put = [&](int row, int2 s) { if (one) mine_state = s; else state.put(row, s); };
    auto grow = [&](int row) { return one ? mine_row : grow_row(p, row); };
    if (tid == 0) here[2] = 0;
    pdl_wait_primary();
    pdl_launch_dependents();

    // (of the first row whose blocks this warp may hand out, while there is time)
    const int row0 = rank * kScanWarps + warp;
    GrowRow first_row = {};
    if (row0 < p.rows) first_row = grow_row(p, row0);
    for (int row = rb; row < re; ++row) {
        const int t = p.num_new[row], ctx = p.context_lens[row];
        int2 s = make_int2(kIdle, 0);
        if (t < 0 || ctx < 0 || (int64_t)ctx + t > (int64_t)p.max_nb * kBlockSize) {
            set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        } else if (t > 0) {
            s.x = kNoCopy;
            mine_row = GrowRow{ctx, (ctx + kBlockSize - 1) / kBlockSize, (int)(((int64_t)ctx + t + kBlockSize - 1) / kBlockSize)};
            if (ctx % kBlockSize != 0) {
                const int id = p.block_tables[(int64_t)row * p.max_nb + ctx / kBlockSize];
                if (id < 0 || id >= p.num_blocks) {
                    set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
                    s.x = kIdle;
                } else {
                    s.x = id;
                    if (atomicSub(p.ref_counts + id, 1) <= 0) set_flag(p.err_flag, PKV_FLAG_REF_RANGE);
                }
            }
        }
        put(row, s);
    }
    scan_sync<kCtas>();
    for (int row = rb; row < re; ++row) {
        const int id = get(row).x;
        if (id >= 0 && __ldcg(p.ref_counts + id) <= 0) atomicMin(p.ref_counts + id, -(row + 1));
    }
    scan_sync<kCtas>();
    // every held block's count is above zero or, where all its holders grow, below: zero says free
    const ScanRange range = scan_range<kCtas>(p.num_blocks, rank);
    const int mine = count_free(p.ref_counts, range);
    long long need = 0;
    for (int row = rb; row < re; ++row) {
        const int id = get(row).x;
        if (id == kIdle) continue;
        const GrowRow g = grow(row);
        need += g.then - g.now;
        if (id >= 0) {
            if (__ldcg(p.ref_counts + id) == -(row + 1)) put(row, make_int2(kKeeps, id));
            else ++need;
        }
        if (g.then - g.now >= kFewBlocks) here[2] = 1;
    }
    int all;
    const int free_in_cta = cta_warps_before(mine, sums, all);
    if (tid == 0) here[0] = all;
    // rows' needs: exclusive over the threads, 64-bit
    long long upto = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += up;
    }
    if (lane == 31) warp_need[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        long long v = warp_need[lane], s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += up;
        }
        warp_need[lane] = s - v;
        if (lane == 31) here[1] = s;
    }
    scan_sync<kCtas>();  // (also this CTA's barrier) every row has decided; the totals are there
    long long before_here[3], all_of[3];
    cluster_before<kCtas>(here, rank, before_here, all_of);
    const long long free_all = all_of[0], need_all = all_of[1];
    long long at = before_here[1] + warp_need[warp] + upto - need;
    for (int row = rb; row < re; ++row) {
        const int2 s = get(row);
        int2 now = make_int2(kIdle, 0);
        if (s.x != kIdle) {
            const GrowRow g = grow(row);
            if (s.x == kKeeps) p.ref_counts[s.y] = 1;
            const int cow_of = s.x >= 0 ? s.x : kNoCopy;
            const long long n = g.then - g.now + (s.x >= 0);
            if (at + n <= free_all) {
                now = make_int2(n > kFewBlocks ? kWaits + 1 + cow_of : cow_of, (int)at);
            } else {
                set_flag(p.err_flag, PKV_FLAG_NO_BLOCKS);
                // its block, if it was to leave it, has its holder back (behind the barrier: the keeper sets it to 1 here)
                now = make_int2(s.x >= 0 ? s.x : kIdle, -1);
            }
            at += n;
            put(row, now);
        }
        if (one) state.put(row, now.x < kIdle ? now : make_int2(-1, -1));  // (what the warps look for)
    }
    // the free blocks that are needed, in order
    const long long wanted = need_all < free_all ? need_all : free_all;
    long long base = before_here[0] + free_in_cta;
    for (int b = range.begin; b < range.end && base < wanted; b += 128) {
        unsigned free[4];
        scan_free(p.ref_counts, b, range.end, free);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long k = base + __popc(free[j] & lanes_below());
            if (((free[j] >> lane) & 1u) && k < wanted) p.free_ids[k] = b + 32 * j + lane;
            base += __popc(free[j]);
        }
    }
    scan_sync<kCtas>();
    auto step_len = [&](int row, int len) { if (p.step_lens) p.step_lens[row] = len; };
    // hand them out: few a row by its own thread ..
    for (int row = rb; row < re; ++row) {
        const int2 s = get(row);
        if (s.x < kIdle) continue;
        if (s.x == kIdle || s.y < 0) {
            if (s.x >= 0) atomicAdd(p.ref_counts + s.x, 1);
            state.put(row, make_int2(-1, -1));
            step_len(row, 0);
            continue;
        }
        const GrowRow g = grow(row);
        const int cow = s.x >= 0, n = g.then - g.now + cow;
        if (!cow) state.put(row, make_int2(-1, -1));
        give_blocks(p, row, g.now - cow, n, s.y, 0, 1, s.x);
        step_len(row, p.context_lens[row] = g.ctx + p.num_new[row]);
    }
    if (all_of[2] == 0) return;
    if (!one) scan_sync<kCtas>();  // a row's own thread still reads its state where a warp leaves the pair to copy
    // .. many by a warp
    for (int row = row0; row < p.rows; row += kCtas * kScanWarps) {
        const int2 s = state.get(row);
        if (s.x >= kIdle) continue;
        const int cow_of = s.x - kWaits - 1, cow = cow_of >= 0;
        const GrowRow g = row == row0 ? first_row : grow_row(p, row);
        const int t = p.num_new[row];
        __syncwarp();
        if (lane == 0 && !cow) state.put(row, make_int2(-1, -1));
        give_blocks(p, row, g.now - cow, g.then - g.now + cow, s.y, lane, 32, cow_of);
        if (lane == 0) step_len(row, p.context_lens[row] = g.ctx + t);
    }
}

cudaError_t launch_extend_sequences(const ExtendParams &p, cudaStream_t stream)
{
    if (p.num_blocks <= kOneCtaBlocks && p.rows <= kOneCtaRows)
        return launch_kernel(extend_kernel<1>, dim3(1), dim3(kScanThreads), 0, stream, true, p);
    return launch_clusters(extend_kernel<kScanCtas>, dim3(kScanCtas), dim3(kScanThreads), dim3(kScanCtas, 1, 1), 0, stream, p);
}

// ---- compacting -------------------------------------------------------------------------------------
// With U blocks in use, those with ids from U on move to the free ids below U: the highest to the lowest.  A used block's
// place in the moves is the number of used blocks above it, a free one's the number of free blocks below it, so the scan
// writes both sides of the list directly.
template <int kCtas>
__global__ void __launch_bounds__(kScanThreads, 1) plan_moves_kernel(const CompactParams p)
{
    __shared__ int sums[kScanWarps];
    __shared__ long long used_here, above_here;
    const int tid = threadIdx.x, lane = tid & 31, rank = scan_rank<kCtas>();
    pdl_wait_primary();
    pdl_launch_dependents();
    const ScanRange range = scan_range<kCtas>(p.num_blocks, rank);
    const int mine = range.end - range.begin - count_free(p.ref_counts, range);
    int all;
    const int in_cta = cta_warps_before(mine, sums, all);
    if (tid == 0) used_here = all, above_here = 0;
    scan_sync<kCtas>();
    long long before[1], used_of[1];
    cluster_before<kCtas>(&used_here, rank, before, used_of);
    const long long used = used_of[0];
    long long base = before[0] + in_cta;  // used blocks below this warp's range
    int above = 0;                     // used blocks from U on
    for (int b = range.begin; b < range.end; b += 128) {
        unsigned free[4];
        scan_free(p.ref_counts, b, range.end, free);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int id = b + 32 * j + lane;
            const unsigned in_use = __ballot_sync(0xFFFFFFFFu, id < range.end) & ~free[j];
            const long long k = base + __popc(in_use & lanes_below());
            if ((in_use >> lane) & 1u) {
                const long long place = used - 1 - k;
                if (id >= used) {
                    ++above;
                    if (place < p.max_moves) p.moves[2 * place] = id, p.move_of[id] = (int)place;
                }
            } else if (id < used) {
                const long long place = id - k;
                if (id < range.end && place < p.max_moves) p.moves[2 * place + 1] = id;
            }
            base += __popc(in_use);
        }
    }
    above = __reduce_add_sync(0xFFFFFFFFu, above);
    if (lane == 0 && above) atomicAdd(reinterpret_cast<unsigned long long *>(&above_here), (unsigned long long)above);
    scan_sync<kCtas>();
    long long total[1];
    cluster_before<kCtas>(&above_here, rank, before, total);
    const int n = (int)min(total[0], (long long)p.max_moves);
    if (rank == 0 && tid == 0) *p.num_moves = n;
    for (int k = rank * kScanThreads + tid; k < p.max_moves; k += kCtas * kScanThreads) {
        if (k >= n) {
            PairList{p.moves}.put(k, make_int2(-1, -1));
            continue;
        }
        const int src = __ldcg(p.moves + 2 * k), dst = __ldcg(p.moves + 2 * k + 1);
        p.ref_counts[dst] = p.ref_counts[src];
        p.ref_counts[src] = 0;
    }
    scan_sync<kCtas>();  // no CTA leaves while its totals are read
}

// Entries [y * kForkEntries, ..) of row x: a moved block's new id.
__global__ void __launch_bounds__(kForkThreads) move_entries_kernel(const CompactParams p)
{
    const int tid = threadIdx.x, row = blockIdx.x, e0 = blockIdx.y * kForkEntries;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int ctx = p.context_lens[row];
    if (ctx < 0 || ctx > p.max_nb * kBlockSize) {
        if (tid == 0 && e0 == 0) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        return;
    }
    const int nb = min((ctx + kBlockSize - 1) / kBlockSize, e0 + kForkEntries);
    const int n = __ldcg(p.num_moves);
    if (n <= 0 || n > p.max_moves) return;
    const int lowest = __ldcg(p.moves + 2 * (n - 1));  // sources descend
    int32_t *tbl = p.block_tables + (int64_t)row * p.max_nb;
#pragma unroll 4
    for (int e = e0 + tid; e < nb; e += kForkThreads) {
        const int id = tbl[e];
        if (id < 0 || id >= p.num_blocks) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
        else if (id >= lowest) {
            const int k = __ldcg(p.move_of + id);
            if (k >= 0 && k < n && __ldcg(p.moves + 2 * k) == id) tbl[e] = __ldcg(p.moves + 2 * k + 1);
            else set_flag(p.err_flag, PKV_FLAG_REF_RANGE);  // a block that no count speaks of
        }
    }
}

cudaError_t launch_compact_blocks(const CompactParams &p, cudaStream_t stream)
{
    cudaError_t e = p.num_blocks <= kOneCtaPlan
                        ? launch_kernel(plan_moves_kernel<1>, dim3(1), dim3(kScanThreads), 0, stream, true, p)
                        : launch_clusters(plan_moves_kernel<kScanCtas>, dim3(kScanCtas), dim3(kScanThreads), dim3(kScanCtas, 1, 1), 0, stream, p);
    if (e != cudaSuccess || p.rows == 0) return e;
    return launch_kernel(move_entries_kernel, dim3((unsigned)p.rows, (unsigned)((p.max_nb + kForkEntries - 1) / kForkEntries)),
                         dim3(kForkThreads), 0, stream, true, p);
}

// ---- copies in many pools -----------------------------------------------------------------------------
// Item k of pairs x pools (pools fastest) copies one block; CTA c takes items c, c + grid, ..  A warp's lanes read the pairs
// of 32 of them at once, so that the many entries without a copy cost nothing.  Bound by memory: every copied block is read
// and written once, 18 KB (a latent cache's block) by one round of loads.  With more CTAs than run at once those that end
// make room for others' loads: compacting eight pools (780 MB) 145.5 us with 8 CTAs of 256 threads an SM and rounds of 16
// KB, 141.5 with rounds of 20, 137 with 16 CTAs, 134 with 64 of 128 threads, 152 with one for every block.
constexpr int kCopyThreads = 128, kCopyAtOnce = 9, kCopyCtas = 64;  // threads, their vectors a round, CTAs an SM

__global__ void __launch_bounds__(kCopyThreads) copy_pools_kernel(const __grid_constant__ CopyPoolsParams p)
{
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t items = (int64_t)p.pairs * p.num_pools;
    for (int64_t k0 = blockIdx.x; k0 < items; k0 += 32ll * gridDim.x) {
        const int64_t k = k0 + (int64_t)lane * gridDim.x;
        int src = -1, dst = -1, pool = 0;
        if (k < items) {
            const int pair = (int)(k / p.num_pools);
            pool = (int)(k - (int64_t)pair * p.num_pools);
            src = __ldcg(p.src_dst + 2 * (int64_t)pair), dst = __ldcg(p.src_dst + 2 * (int64_t)pair + 1);
            if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
                if (tid < 32 && (src != -1 || dst != -1)) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
                src = dst = -1;
            }
        }
        unsigned todo = __ballot_sync(0xFFFFFFFFu, src >= 0 && src != dst);
        for (; todo; todo &= todo - 1) {
            const int l = __ffs(todo) - 1;
            uint4 *const base = static_cast<uint4 *>(p.pools[__shfl_sync(0xFFFFFFFFu, pool, l)]);
            const uint4 *from = base + (int64_t)__shfl_sync(0xFFFFFFFFu, src, l) * p.vectors;
            uint4 *to = base + (int64_t)__shfl_sync(0xFFFFFFFFu, dst, l) * p.vectors;
            for (int64_t x = tid; x < p.vectors; x += kCopyAtOnce * kCopyThreads) {
                uint4 v[kCopyAtOnce];
#pragma unroll
                for (int j = 0; j < kCopyAtOnce; ++j)
                    if (x + j * kCopyThreads < p.vectors) v[j] = from[x + j * kCopyThreads];
#pragma unroll
                for (int j = 0; j < kCopyAtOnce; ++j)
                    if (x + j * kCopyThreads < p.vectors) to[x + j * kCopyThreads] = v[j];
            }
        }
    }
}

cudaError_t launch_copy_pools(const CopyPoolsParams &p, int sms, cudaStream_t stream)
{
    const int64_t items = (int64_t)p.pairs * p.num_pools, most = (int64_t)sms * kCopyCtas;
    return launch_kernel(copy_pools_kernel, dim3((unsigned)(items < most ? items : most)), dim3(kCopyThreads), 0, stream, true, p);
}

}  // namespace pkv
