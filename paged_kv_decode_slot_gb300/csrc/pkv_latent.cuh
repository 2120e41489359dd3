// pkv_latent.cuh - what the two kernels of attention over a latent cache share: how the tiles of a batch are dealt out,
// waits, and the like.
#pragma once

#include <float.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_latent.h"
#include "pkv_tcgen05.cuh"

namespace pkv {

constexpr int kLatChunks = (kLatentDim + kLatentRope) / 64;   // 64-element chunks of a row
constexpr float kLatRescale = 8.f;                            // log2 of how far a logit may exceed the running maximum

// ---- dealing out the tiles ----------------------------------------------------------------------
// A unit's share of the work: its tiles and, as much as this many, its queries, statistics and outputs (64 ragged sequences of
// 128 heads: 81 us with 1, 78.5 with 2, 77.6 with 3 and 4).
constexpr int kLatentUnitCost = 3;

__device__ __forceinline__ int latent_ctx(const LatentAttnParams &p, int b)
{
    const int ctx = p.context_lens[b];
    return ctx < 0 || ctx > p.max_nb * kBlockSize ? 0 : ctx;
}
template <int kTile>
__device__ __forceinline__ int latent_cost(int ctx)
{
    return ctx > 0 ? (ctx + kTile - 1) / kTile + kLatentUnitCost : 0;
}

// Tiles [t0, t1) of unit (b, chunk), which starts at `start` in the row of all units.
struct LatentSegment {
    int b, chunk, ctx, t0, t1, tiles;
    int64_t start;
    bool whole;
};

template <int kTile>
struct LatentWalk {
    int64_t lo, hi, start;
    int b, chunk;
    __device__ __forceinline__ bool next(const LatentAttnParams &p, LatentSegment &s)
    {
        while (start < hi && b < p.B) {
            const int ctx = latent_ctx(p, b), cost = latent_cost<kTile>(ctx);
            const int64_t at = start;
            const int ub = b, uc = chunk;
            start += cost;
            if (++chunk == p.chunks || cost == 0) chunk = 0, ++b;
            if (cost == 0) continue;
            const int x0 = (int)max((int64_t)0, lo - at), x1 = (int)min((int64_t)cost, hi - at);
            s.t0 = max(0, x0 - kLatentUnitCost), s.t1 = max(0, x1 - kLatentUnitCost);
            if (s.t0 >= s.t1) continue;
            s.b = ub, s.chunk = uc, s.ctx = ctx, s.tiles = cost - kLatentUnitCost, s.start = at;
            s.whole = s.t0 == 0 && s.t1 == s.tiles;
            return true;
        }
        return false;
    }
};

// x * n / d of work x in [0, ..] (64-bit divisions take as long as a load).
__device__ __forceinline__ int64_t latent_share(int64_t x, int n, int d)
{
    return x < (1 << 24) && n <= 152 ? (int64_t)((uint32_t)x * (uint32_t)n / (uint32_t)d) : x * n / d;
}

// Runs that the work is cut into: as many as there are CTAs, of two tiles' worth at least (5 sequences of up to 3,000 tokens and
// 128 heads 17.6 us, with runs of one 22.8, of four 17.8; one of 2,000 tokens and 16 heads 10.0, 10.5 and 11.9).
__device__ __forceinline__ int latent_runs(const LatentAttnParams &p, int64_t total) { return (int)min((int64_t)p.ctas, (total + 1) / 2); }

// This CTA's (or cluster's: `cta` of p.ctas) run of the work, the same in every thread; false: nothing to do.  `sums` holds kThreads + 4 64-bit
// words of shared memory.  Every thread calls it.
// Up to 128 sequences each warp finds it by itself, four sequences a lane; with the CTA's barriers, as more need them, it took
// 1.5 us of the prologue.
template <int kTile, int kThreads>
__device__ __forceinline__ bool latent_deal(const LatentAttnParams &p, int cta, int64_t *sums, LatentWalk<kTile> &w, int64_t &total,
                                            int &ctas)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const auto bad = [&](int ctx) { return ctx < 0 || ctx > p.max_nb * kBlockSize; };
    if (p.B <= 128) {
        const int per = (p.B + 31) / 32, b0 = lane * per;
        int ctx[4], costs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ctx[k] = k < per && b0 + k < p.B ? p.context_lens[b0 + k] : 0;
        int64_t cost = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (bad(ctx[k])) {
                if (cta == 0 && tid < 32) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
                ctx[k] = 0;
            }
            cost += costs[k] = latent_cost<kTile>(ctx[k]);
        }
        int64_t upto = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += up;
        }
        total = __shfl_sync(0xFFFFFFFFu, upto, 31) * p.chunks;
        ctas = latent_runs(p, total);
        if (cta >= ctas) return false;
        w.lo = latent_share(total, cta, ctas);
        w.hi = latent_share(total, cta + 1, ctas);
        // the lane whose sequences hold its start
        int64_t at = (upto - cost) * p.chunks;
        const bool here = at <= w.lo && w.lo < upto * p.chunks;
        int b = b0, c = 1;
        if (here) {
            bool found = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t all = (int64_t)costs[k] * p.chunks;
                if (!found && w.lo < at + all) found = true, b = b0 + k, c = costs[k];
                if (!found) at += all;
            }
        }
        const int from = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
        at = __shfl_sync(0xFFFFFFFFu, at, from);
        c = __shfl_sync(0xFFFFFFFFu, c, from);
        w.b = __shfl_sync(0xFFFFFFFFu, b, from);
        w.chunk = p.chunks == 1 ? 0 : (int)((w.lo - at) / c);
        w.start = at + (int64_t)w.chunk * c;
        return true;
    }
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int64_t cost = 0;
    for (int b = b0; b < b1; ++b) {
        const int ctx = p.context_lens[b];
        if (cta == 0 && bad(ctx)) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        cost += latent_cost<kTile>(latent_ctx(p, b));
    }
    sums[tid] = cost;
    __syncthreads();
    if (tid < 32) {  // exclusive scan by one warp, kThreads / 32 entries a lane
        constexpr int kPer = kThreads / 32;
        int64_t mine = 0;
        for (int k = 0; k < kPer; ++k) mine += sums[tid * kPer + k];
        int64_t before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, before, o);
            if (tid >= o) before += up;
        }
        if (tid == 31) sums[kThreads] = before;
        before -= mine;
        for (int k = 0; k < kPer; ++k) {
            const int64_t v = sums[tid * kPer + k];
            sums[tid * kPer + k] = before;
            before += v;
        }
    }
    __syncthreads();
    total = sums[kThreads] * p.chunks;
    ctas = latent_runs(p, total);
    if (cta >= ctas) return false;
    w.lo = latent_share(total, cta, ctas);
    w.hi = latent_share(total, cta + 1, ctas);
    int64_t at = sums[tid] * p.chunks;
    if (at <= w.lo && w.lo < (sums[tid] + cost) * p.chunks) {
        for (int b = b0; b < b1; ++b) {
            const int c = latent_cost<kTile>(latent_ctx(p, b));
            if (w.lo < at + (int64_t)c * p.chunks) {
                const int chunk = (int)((w.lo - at) / c);
                sums[kThreads + 1] = b;
                sums[kThreads + 2] = chunk;
                sums[kThreads + 3] = at + (int64_t)chunk * c;
                break;
            }
            at += (int64_t)c * p.chunks;
        }
    }
    __syncthreads();
    w.b = (int)sums[kThreads + 1];
    w.chunk = (int)sums[kThreads + 2];
    w.start = sums[kThreads + 3];
    // the sums' place is TMA's from here on: what threads read and wrote there comes before its writes
    fence_proxy_async_shared();
    __syncthreads();
    return true;
}

// mbar_wait_bounded in two parts.  What is met on every stage of a pipeline stays short: with the loop in line a wait for a
// barrier that was ready took 220 clocks, with the call behind the first try 50.  And %globaltimer takes 0.4 us to read, as
// long as a stage is in use, so the first tries (each suspends the thread for a while) go without it.
static __device__ __noinline__ bool latent_wait_on(uint32_t bar, uint32_t parity, const volatile int *abort, uint64_t limit_ns)
{
#pragma unroll 1
    for (int it = 0; it < 64; ++it)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait_bounded(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool latent_wait(uint32_t bar, uint32_t parity, const volatile int *abort, uint64_t limit_ns)
{
    return mbar_try_wait(bar, parity) || latent_wait_on(bar, parity, abort, limit_ns);
}

// ---- small pieces -------------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Barrier of four softmax warps that share rows (128 threads; `half` 0 or 1), and the same with a vote.
__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); }
__device__ __forceinline__ bool half_any(int half, bool v)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(1 + half), "r"((int)v)
        : "memory");
    return r != 0;
}

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

}  // namespace pkv
