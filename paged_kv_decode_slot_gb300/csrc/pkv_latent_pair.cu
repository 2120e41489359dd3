// pkv_latent_pair.cu - decode attention over a paged latent cache for sequences of more than 32 (token, head) rows; the
// mathematics is in pkv_latent_attn.cu.  Chunks of up to 128 rows, a cluster of two CTAs each.
//
// With 128 rows a cached row of 1,152 bytes takes 2 * 1088 * 128 operations, 242 a byte, about what the chip has for one
// byte of DRAM, and 128 queries and a 128-token tile are 147 KB each: neither one CTA's shared memory (227 KB) nor its tensor
// memory (128 x 512 sums fill it) holds the problem.  tcgen05.mma with cta_group::2 spreads it over two SMs, and no operand
// is held twice:
//     S[128 x 128 tokens]  = Q . C^T            a CTA: its 64 rows of Q; the keys of 64 of the tokens
//     O^T[512 x 128 rows] += C[:, :512]^T . P^T a CTA: all tokens' values of its 256 elements; its 64 rows of P
// S is split by rows: a row's first half of the columns lies in lane r, its second half in lane 64 + r, so softmax stays within
// a CTA, and its weights are, row by row, what the second product takes from this CTA.  O^T is split by elements, each CTA with
// all rows.  That way P V runs as M = 256 at the full rate (as O += P V, M = 128, an MMA of the pair takes as long for half as
// much); what it costs is that scaling a row's sums takes both CTAs.  They do so at the end, for 1 / sum, and where a logit
// exceeds its row's reference (the maximum of its first tile) by 2^32, which weights and sums in 32-bit exponents bear: the
// MMA thread then refuses that round of weights, both CTAs exchange factors, scale, and make the tile's weights again.
// One thread of the first CTA issues all MMAs.
//
// The cache streams through nine slots, four of 16 KB for a CTA's share of a tile as keys (64 tokens x 128 elements), half a
// one for its rotary keys and four for its values (32 tokens x 256 elements, from L2): every tile uses every slot once, so
// all addresses and parities of the MMA thread's code are known when it is compiled.  (Through a ring whose stages had to
// be computed, that thread was what bounded the kernel: 4,700 clocks a tile, whatever the MMAs' rate.)  A box is one block's
// share of a slot, in swizzle atoms of 8 rows, [half][chunk][8 rows][128 bytes].  Each CTA's loads are counted on the first
// CTA's barrier.  The next tile's blocks are fetched into L2 meanwhile: a slot of keys is free again only when the last tile's
// are multiplied (64 sequences of 512 to 8,192 tokens: 81 us, without 87, two tiles ahead 84).
//
// CTA = 12 warps: 0-7 softmax (warps w, w + 2, .. share rows 32 (w % 2) ..; of a tile's 128 tokens each thread has a row's 32:
// half of them by lane, half by w / 4) and outputs (each thread an element of all rows), 8 issues the MMAs (first CTA), 9 and 10
// load keys and queries, 11 loads values and zeroes what lies behind a sequence's end.  QK^T of tile i + 1 is issued before P V of
// tile i, so the tensor cores work through the softmax of tile i.
//
// Bound by how soon a slot of keys is filled again (the MMA thread's own work takes 2,600 clocks a tile, the tiles 2,600 to
// 3,700, with DRAM, L2 and the tensor pipe busy for half to two thirds of it) and by what a unit costs beside its tiles
// (prologue, exchange, outputs and join, about 20 us of the 77): 152 sequences of 4,096 tokens and 128 heads take 135 to 144 us, 5.2
// TB/s and 1.2 PFLOP/s; 64 of 512 to 8,192 tokens 77 us, with 64 heads 71; one of 131,072 tokens 43.  Tiles of 256 tokens with both
// products as M = 256 took 134 us for the 64 sequences: each CTA then needs half of the other's weights in every tile, and 72
// KB of queries leave 96 KB for 278 KB of loads a tile.
#include "pkv_cluster.cuh"
#include "pkv_latent.cuh"

namespace pkv {

struct PairLayout {
    static constexpr int kTile = 128, kBlocks = kTile / kBlockSize;
    static constexpr int kRows = 64;                                   // of a CTA
    static constexpr int kStages = 9, kStage = 16384, kRope = 8;       // slots: 4 of keys, 4 of values, the rotary keys (half a slot)
    static constexpr int kQChunk = kRows * 128, kQBytes = kLatChunks * kQChunk;
    static constexpr int kPChunk = kRows * 128, kPBytes = 2 * kPChunk;  // 64 tokens a chunk
    static constexpr int kQOffset = 0, kPOffset = kQBytes, kSlotsOffset = kPOffset + kPBytes;
    static constexpr int kBarOffset = kSlotsOffset + 8 * kStage + kStage / 2;
    // full[S], empty[S], q_full, q_free, s_full[2], p_ready, pv_done, exchange, tail[2], fin
    static constexpr int kBars = 2 * kStages + 10;
    static constexpr int kMiscOffset = (kBarOffset + kBars * 8 + 15) & ~15;
    static constexpr int kWords = 4 /* tile masks */ + 8 /* abort, tmem, query loads, raise, verdict, - */ + 3 * kStages + 1 /* sent, use, want, - */ +
                                  4 * kRows /* of four warps */ + 2 * kRows /* factors */;
    static constexpr int kBytes = kMiscOffset + kWords * 4;
    static constexpr int kAlloc = kBytes + 1024;                       // room to align the window
    static_assert(kPOffset % 1024 == 0 && kSlotsOffset % 1024 == 0, "swizzle atoms are aligned");
    static_assert(kAlloc <= 227 * 1024, "shared memory of a CTA");
    static constexpr uint32_t kCols = 512;                             // tensor memory: O^T 2 x 128, S 2 x 64
};
constexpr int kPairSoftmaxWarps = 8, kPairMmaWarp = 8, kPairLoadWarp = 9, kPairValueWarp = 11;
constexpr int kPairThreads = 384;
constexpr int kBlockBytes = kBlockSize * (kLatentDim + kLatentRope) * 2;
// A logit may exceed its row's reference by this much (log2) before the reference moves: weights and sums have 32-bit
// exponents, so that only the far ends of the range matter, and moving it takes both CTAs.
constexpr float kPairRescale = 32.f;

// ---- cta_group::2 -------------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc2(uint32_t dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2()
{
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_mma_ss2(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive, when the MMAs issued so far are done, at the barrier at this place of both CTAs, or of this one.
__device__ __forceinline__ void tc_commit2_both(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tc_commit2(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t pair_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address, for the whole cluster, of what lies at `at` in CTA `rank`.
__device__ __forceinline__ uint32_t pair_at(uint32_t at, int rank)
{
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    return there;
}
// (what the arrival speaks of was fenced for the asynchronous proxy, which is who reads it)
__device__ __forceinline__ void pair_arrive(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// TMA loads into this CTA's shared memory, counted on a barrier of the cluster.
__device__ __forceinline__ void pair_load_5d(uint32_t dst, const CUtensorMap *map, uint32_t cluster_bar, int c0, int c1, int c2, int c3,
                                             int c4)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t cluster_bar, int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void tmem_load32(uint32_t taddr, float (&x)[32])
{
    uint32_t r[2][16];
    tmem_ld16(taddr, r[0]);
    tmem_ld16(taddr + 16, r[1]);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(r[c / 16][c % 16]);
}

__device__ __forceinline__ int load_word(const volatile int *at, int rank)
{
    return __float_as_int(load_cluster<float>(smem_u32((const void *)at), rank));
}

__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_addr, uint32_t v)
{
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
// An arrival, at a barrier of the cluster, that what this thread wrote to either CTA's shared memory comes before.
__device__ __forceinline__ void pair_arrive_release(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *at, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}
// A barrier's phase that is complete: what was written before its arrivals is seen behind this.
__device__ __forceinline__ void pair_acquired(uint32_t bar, uint32_t parity)
{
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(bar), "r"(parity)
                 : "memory");
}
// (2,000 clocks: for a refused round alone, not in every tile)
__device__ __forceinline__ void pair_fence() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

__global__ void __launch_bounds__(kPairThreads, 1)
latent_pair_kernel(const __grid_constant__ LatentPairMaps maps, const LatentAttnParams p)
{
    using L = PairLayout;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const mem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)pair_rank(), pair = (int)blockIdx.x >> 1;

    const uint32_t q_u32 = base + L::kQOffset, p_u32 = base + L::kPOffset, slots = base + L::kSlotsOffset;
    const uint32_t bar_full = base + L::kBarOffset, bar_empty = bar_full + 8 * L::kStages, bar_qfull = bar_empty + 8 * L::kStages,
                   bar_qfree = bar_qfull + 8, bar_s = bar_qfree + 8, bar_p = bar_s + 16, bar_pv = bar_p + 8, bar_x = bar_pv + 8,
                   bar_tail = bar_x + 8, bar_fin = bar_tail + 16;
    volatile int *const tile_mask = reinterpret_cast<volatile int *>(mem + L::kMiscOffset);  // [4], by tile % 4: blocks there
    volatile int *const abort_flag = tile_mask + 4;
    volatile uint32_t *const tmem_slot = reinterpret_cast<volatile uint32_t *>(tile_mask + 5);
    volatile int *const q_asked = tile_mask + 6;
    // of a slot's last use: bytes this CTA asked for, the use's number + 1, bytes the barrier was told (first CTA)
    volatile int *const raise = tile_mask + 7;    // first CTA: a logit passed its reference by too much
    volatile int *const verdict = tile_mask + 8;  // the last round of weights that is to be made again with new references
    volatile int *const sent = tile_mask + 12, *const use = sent + L::kStages, *const want = use + L::kStages;
    float *const quarters = const_cast<float *>(reinterpret_cast<volatile float *>(want + L::kStages + 1));  // [4][64]
    float *const factor = quarters + 4 * L::kRows;                                              // [128] of both CTAs' rows

    // What needs nothing of the launch ahead comes before the wait for it.  (Tensor memory too: a CTA that still has to take its own
    // does not fit beside this one's shared memory, so none of that launch waits for what is held here.)
    if (threadIdx.x == 0) {
        *abort_flag = 0, *q_asked = 0, *raise = 0, *verdict = 0;
        for (int s = 0; s < L::kStages; ++s) sent[s] = use[s] = want[s] = 0;
        for (int k = 0; k < L::kBars; ++k) {
            const uint32_t bar = bar_full + 8 * k;
            // weights: the softmax warps of both CTAs; exchanges: two warps of the other CTA and, so that none can be a round
            // behind, all eight of this one; stages and zeroed rows: both CTAs
            mbar_init(bar, bar == bar_p ? 2 * kPairSoftmaxWarps : bar == bar_x ? 2 + kPairSoftmaxWarps : k < L::kStages || bar == bar_tail + 8 ? 2 : 1);
        }
        prefetch_tensormap(&maps.keys);
        prefetch_tensormap(&maps.rope);
        prefetch_tensormap(&maps.values);
        prefetch_tensormap(&maps.queries);
    }
    if (warp == kPairMmaWarp) {
        tmem_alloc2(smem_u32((const void *)tmem_slot), L::kCols);
        tmem_relinquish2();
    }
    if (threadIdx.x == 0) fence_barrier_init();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and tensor memory are there
    tc_fence_after();
    pdl_wait_primary();
    pdl_launch_dependents();
    LatentWalk<L::kTile> walk;
    int64_t total;
    int pairs;
    // (the sums lie where the queries will; both CTAs find the same)
    const bool work = latent_deal<L::kTile, kPairThreads>(p, pair, reinterpret_cast<int64_t *>(mem), walk, total, pairs);
    if (!work) {
        if (warp == kPairMmaWarp) tmem_dealloc2(*tmem_slot, L::kCols);
        return;
    }
    const uint32_t tm_o = *tmem_slot, tm_s = tm_o + 256;

    auto give_up = [&]() {
        if (lane == 0 && !*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
        *abort_flag = 1;
    };
    auto wait_one = [&](uint32_t bar, uint32_t parity) { return latent_wait(bar, parity, abort_flag, p.wait_ns); };
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait_one(bar, parity)); };
    auto give_up_one = [&]() {
        if (!*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
        *abort_flag = 1;
    };
    bool issuer = false;  // the thread that issues the MMAs (a commit speaks of its thread's)

    // Slot s for tile number gt, once it is free; the first CTA's barrier is told what both will send.  The second CTA arrives there
    // also where it has nothing to send: the MMAs could otherwise use and release the slot twice before this thread came to
    // wait for the first time (a barrier tells only neighbouring uses apart).
    auto open = [&](int s, uint32_t gt, int bytes_all, int bytes_own) {
        if (gt > 0 && !wait_one(bar_empty + 8 * s, (gt & 1) ^ 1)) return false;
        sent[s] = bytes_own, use[s] = (int)gt + 1;
        if (rank == 0) {
            want[s] = bytes_all;
            mbar_arrive_expect_tx(bar_full + 8 * s, (uint32_t)bytes_all);
        } else {
            pair_arrive(pair_at(bar_full + 8 * s, 0));
        }
        return true;
    };
    // The blocks of tile t of a segment (-1: none, or none of the pool).
    auto ids_of = [&](const LatentSegment &sg, int t, int (&ids)[L::kBlocks]) {
        const int nb = (sg.ctx + kBlockSize - 1) / kBlockSize;
        const int32_t *tbl = p.block_tables + (size_t)sg.b * p.max_nb;
#pragma unroll
        for (int k = 0; k < L::kBlocks; ++k) {
            const int j = t * L::kBlocks + k;
            ids[k] = t < sg.t1 && j < nb ? tbl[j] : -1;
        }
    };
    auto mask_of = [&](const int (&ids)[L::kBlocks]) {
        uint32_t mask = 0;
#pragma unroll
        for (int k = 0; k < L::kBlocks; ++k) mask |= (uint32_t)(ids[k] >= 0 && ids[k] < p.num_blocks) << k;
        return mask;
    };
    if (warp == kPairLoadWarp || warp == kPairLoadWarp + 1) {
        // ------------------------------ keys and queries: one thread of two warps ------------------------------
        if (elect_one()) {
            const int me = warp - kPairLoadWarp;
            const uint32_t full_there = pair_at(bar_full, 0), qfull_there = pair_at(bar_qfull, 0);
            uint32_t g = 0, q_loads = 0;
            bool ok = true, withheld = false;
            LatentSegment sg;
            while (ok && walk.next(p, sg)) {
                int next[L::kBlocks];
                ids_of(sg, sg.t0, next);
                if (me == 0) {
                    // the queries, once the last unit's are no longer needed
                    if (q_loads > 0) ok = wait_one(bar_qfree, (q_loads - 1) & 1);
                    if (!ok) break;
                    const int64_t row = (int64_t)sg.b * p.rows + (int64_t)sg.chunk * 128 + rank * L::kRows;
                    *q_asked = (int)++q_loads;
                    if (rank == 0) mbar_arrive_expect_tx(bar_qfull, 2 * L::kQBytes);
                    for (int c = 0; c < kLatChunks; ++c) pair_load_3d(q_u32 + c * L::kQChunk, &maps.queries, qfull_there, 0, (int)row, c);
                }
                for (int t = sg.t0; t < sg.t1 && ok; ++t, ++g) {
                    if (PKV_TILE_WITHHELD(p, t)) {  // test builds: nothing is loaded or signalled from here on
                        withheld = true, ok = false;
                        break;
                    }
                    const uint32_t mask = mask_of(next), own = (mask >> (4 * rank)) & 0xFu;
                    int mine[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) mine[k] = rank ? next[4 + k] : next[k];
                    ids_of(sg, t + 1, next);
                    if (me == 0 && rank == 0) {
                        const int nblk = min(L::kBlocks, (sg.ctx + kBlockSize - 1) / kBlockSize - t * L::kBlocks);
                        if (mask != (1u << nblk) - 1u) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
                    }
                    tile_mask[g & 3] = (int)mask;  // (both threads write it, each before it fills a slot of the tile)
#pragma unroll 1
                    for (int c = 2 * me; c < 2 + 3 * me; ++c) {
                        const bool rope = c == 4;
                        const int s = rope ? L::kRope : c, bytes = rope ? 2048 : 4096;
                        ok = open(s, g, __popc(mask) * bytes, __popc(own) * bytes);
                        if (!ok) break;
                        const CUtensorMap *const map = rope ? &maps.rope : &maps.keys;
                        const uint32_t dst = slots + s * L::kStage, bar = full_there + 8 * s;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if ((own >> k) & 1u) pair_load_5d(dst + k * bytes, map, bar, 0, 0, 2 * c, 0, mine[k]);
                    }
                    if (me == 0) {
                        // the next tile on its way into L2 meanwhile
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int id = rank ? next[4 + k] : next[k];
                            if (id >= 0 && id < p.num_blocks) prefetch_l2(p.cache + (int64_t)id * kBlockBytes, kBlockBytes);
                        }
                    }
                }
            }
            // the slots and the queries released: no arrival is on its way into this CTA any more
            for (int c = 2 * me; c < 2 + 3 * me && ok && g > 0; ++c) ok = wait_one(bar_empty + 8 * (c == 4 ? L::kRope : c), (g - 1) & 1);
            if (ok && q_loads > 0) ok = wait_one(bar_qfree, (q_loads - 1) & 1);
            if (!ok && !withheld) give_up_one();
        }
        __syncwarp();
    } else if (warp == kPairValueWarp) {
        // ------------------------------ values: one thread; rows behind a sequence's end: the warp ------------------------------
        // Those may hold anything, and 0 x NaN is NaN: both CTAs zero them before P V reads them, when the MMA thread asks for it
        // (asked and answered in turn, so that neither can be a use of the slot ahead of the other).
        const bool leads = elect_one();
        uint32_t g = 0, asked = 0;
        bool ok = true, withheld = false;
        LatentSegment sg;
        while (ok && walk.next(p, sg)) {
            if (leads) {
                int next[L::kBlocks];
                ids_of(sg, sg.t0, next);
                for (int t = sg.t0; t < sg.t1 && ok; ++t, ++g) {
                    if (PKV_TILE_WITHHELD(p, t)) {
                        withheld = true, ok = false;
                        break;
                    }
                    const uint32_t mask = mask_of(next);
                    int ids[L::kBlocks];
#pragma unroll
                    for (int k = 0; k < L::kBlocks; ++k) ids[k] = next[k];
                    ids_of(sg, t + 1, next);
                    // (slots past the last block pass empty, so that all have a tile's parity)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const uint32_t two = (mask >> (2 * v)) & 3u;
                        if (ok) ok = open(4 + v, g, 2 * __popc(two) * 8192, __popc(two) * 8192);
                        if (!ok) break;
                        const uint32_t dst = slots + (4 + v) * L::kStage, bar = pair_at(bar_full + 8 * (4 + v), 0);
                        if (two & 1u) pair_load_5d(dst, &maps.values, bar, 0, 0, 4 * rank, 0, ids[2 * v]);
                        if (two & 2u) pair_load_5d(dst + 8192, &maps.values, bar, 0, 0, 4 * rank, 0, ids[2 * v + 1]);
                    }
                }
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            const int tail = sg.ctx % kBlockSize;
            if (!ok || sg.t1 != sg.tiles || tail == 0) continue;
            ok = wait(bar_tail, asked++ & 1);
            if (!ok) break;
            const int j = sg.ctx / kBlockSize - (sg.tiles - 1) * L::kBlocks;
            const uint32_t blk = slots + (4 + (j >> 1)) * L::kStage + (j & 1) * 8192;
            for (int x = lane; x < (kBlockSize - tail) * 32; x += 32) {
                const int u = x & 31, row = tail + (x >> 5);
                st_shared_v4(blk + (row >> 3) * 4096 + (u >> 3) * 1024 + (row & 7) * 128 + (u & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) pair_arrive(pair_at(bar_tail + 8, 0));
        }
        if (leads)
            for (int v = 0; v < 4 && ok && g > 0; ++v) ok = wait_one(bar_empty + 8 * (4 + v), (g - 1) & 1);
        if (!__all_sync(0xFFFFFFFFu, ok || withheld) && !__any_sync(0xFFFFFFFFu, withheld)) give_up();
    } else if (warp == kPairMmaWarp) {
        // ------------------------------ MMAs: one thread of the first CTA ------------------------------
        issuer = elect_one() && rank == 0;
        if (issuer) {
            constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, 0, 0), kIdO = idesc_bf16_f32(256, 128, 1, 0);
            const uint64_t k_desc = smem_desc_sw128(slots, 16, 2048), r_desc = smem_desc_sw128(slots + L::kRope * L::kStage, 16, 1024);
            const uint64_t v_desc = smem_desc_sw128(slots + 4 * L::kStage, 1024, 4096);
            const uint64_t q_desc = smem_desc_sw128(q_u32, 16, 1024), p_desc = smem_desc_sw128(p_u32, 16, 1024);
            const uint32_t ask_other = pair_at(bar_tail, 1), pv_other = pair_at(bar_pv, 1);
            const uint32_t verdict_other = pair_at(smem_u32((const void *)verdict), 1);
            uint32_t g = 0, unit = 0, tails = 0, rounds = 0;
            bool ok = true, started = false;
            // P V of tile number gt; tail_of: the slot whose last block's end is zeroed first
            auto pv = [&](uint32_t gt, int tail_of) {
                for (;;) {
                    ok = wait_one(bar_p, rounds & 1);
                    pair_acquired(bar_p, rounds++ & 1);
                    if (!ok) return;
                    if (*raise == 0) break;
                    *raise = 0;
                    *verdict = (int)rounds;
                    st_cluster_u32(verdict_other, rounds);
                    pair_arrive_release(pv_other);
                    mbar_arrive(bar_pv);
                }
                const uint32_t mask = (uint32_t)tile_mask[gt & 3];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    ok = wait_one(bar_full + 8 * (4 + v), gt & 1);
                    if (ok && v == tail_of) {
                        mbar_arrive(bar_tail);
                        pair_arrive(ask_other);
                        ok = wait_one(bar_tail + 8, tails++ & 1);
                    }
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        constexpr int kQuad = L::kPChunk >> 4;
                        const int blk = 2 * v + j;
                        if ((mask >> blk) & 1u) {
                            const uint64_t a = v_desc + ((v * L::kStage + j * 8192) >> 4), b = p_desc + (blk >> 2) * kQuad + 2 * (blk & 3);
                            tc_mma_ss2(tm_o, a, b, kIdO, started);
                            tc_mma_ss2(tm_o + 128, a + (2048 >> 4), b, kIdO, started);
                            started = true;
                        }
                    }
                    tc_commit2_both(bar_empty + 8 * (4 + v));
                }
                tc_commit2_both(bar_pv);
            };
            LatentSegment sg;
            while (ok && walk.next(p, sg)) {
                ok = wait_one(bar_qfull, unit & 1);
                ++unit;
                for (int t = sg.t0; t < sg.t1 && ok; ++t, ++g) {
                    const uint32_t d = tm_s + 64 * (g & 1);
#pragma unroll
                    for (int c = 0; c < 4 && ok; ++c) {
                        ok = wait_one(bar_full + 8 * c, g & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int q = ((2 * c + (k >> 2)) * L::kQChunk >> 4) + 2 * (k & 3), at = ((c * L::kStage + (k >> 2) * 1024) >> 4) + 2 * (k & 3);
                            tc_mma_ss2(d, q_desc + q, k_desc + at, kIdS, c + k > 0);
                        }
                        tc_commit2_both(bar_empty + 8 * c);
                    }
                    if (ok) ok = wait_one(bar_full + 8 * L::kRope, g & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma_ss2(d, q_desc + (8 * L::kQChunk >> 4) + 2 * k, r_desc + 2 * k, kIdS, 1);
                    tc_commit2_both(bar_empty + 8 * L::kRope);
                    tc_commit2_both(bar_s + 8 * (g & 1));
                    if (t + 1 == sg.t1) tc_commit2_both(bar_qfree);
                    if (t > sg.t0) pv(g - 1, -1);
                    else started = false;
                }
                const int blk_in_tile = sg.ctx / kBlockSize - (sg.tiles - 1) * L::kBlocks;
                if (ok) pv(g - 1, sg.t1 == sg.tiles && sg.ctx % kBlockSize > 0 ? blk_in_tile >> 1 : -1);
            }
            if (!ok) give_up_one();
        }
        __syncwarp();
    } else {
        // ------------------------------ softmax and outputs ------------------------------
        const int quarter = warp & 3, h = warp >> 2, group = quarter & 1, side = quarter >> 1;
        const int r = 32 * group + lane;              // row of the CTA
        const int tok0 = 64 * side + 32 * h;          // this thread's tokens of a tile
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t ready = pair_at(bar_p, 0), raise_there = pair_at(smem_u32((const void *)raise), 0);
        const uint32_t x_there = pair_at(bar_x, rank ^ 1), factor_there = pair_at(smem_u32(factor), rank ^ 1);
        const uint32_t p_row = p_u32 + side * L::kPChunk + r * 128;
        float *const quarter_at = quarters + r;
        uint32_t g = 0, rounds = 0, swaps = 0;
        bool ok = true;
        auto wait_for = [&](uint32_t bar, uint32_t parity) {
            if (ok) ok = wait(bar, parity);
            if (!ok) give_up();
        };
        // A value for each row of this CTA into both CTAs' factors.
        auto exchange = [&](float v) {
            if (side + h == 0) {
                factor[64 * rank + r] = v;
                st_cluster_u32(factor_there + (64 * rank + r) * 4, __float_as_uint(v));
                __syncwarp();
                if (lane == 0) pair_arrive_release(x_there);
            }
            if (lane == 0) mbar_arrive(bar_x);
            wait_for(bar_x, swaps & 1);
            pair_acquired(bar_x, swaps++ & 1);
        };
        LatentSegment sg;
        while (ok && walk.next(p, sg)) {
            const int row0 = sg.chunk * 128 + rank * L::kRows;  // first row of this CTA within the sequence
            const bool real = row0 + r < p.rows;
            if (threadIdx.x == 0 && rank == 0 && sg.t0 == 0) {
                // for the joining launch: the first pair of the unit's parts, and how many there are
                const int64_t last = sg.start + sg.tiles + kLatentUnitCost - 1;
                const int parts = sg.whole ? 1 : (int)(((last + 1) * pairs - 1) / total) - pair + 1;
                p.unit_parts[(int64_t)sg.b * p.chunks + sg.chunk] = make_int2(pair, parts);
            }
            const int limit = real ? sg.ctx - p.T + (row0 + r) / p.N + 1 : 0;  // tokens the row sees
            // The first tile sets the rows' references.  Where a later one exceeds them by too much, the MMA thread refuses the
            // round of weights: both CTAs then scale the sums of the rows concerned and make the tile's weights again.  That is
            // learned with the wait for the product, so after the next tile's weights were made: those are dropped.
            // The warps of a group leave together: one that gives up goes to a vote, and the others meet it at their next.
            // l, norm: sums of the weights, as they are and as the product has them; _here, _before: ahead of this tile, and of the last
            float m = -FLT_MAX, l = 0.f, l_here = 0.f, l_before = 0.f, norm = 0.f, norm_here = 0.f, norm_before = 0.f;
            bool left = false, first = true, redo = false, clear = true;
            for (int t = sg.t0;;) {
                if (t < sg.t1) wait_for(bar_s + 8 * (g & 1), (g >> 1) & 1);
                if (first || redo || !ok) {
                    left = half_any(group, !ok);
                    if (left) break;
                }
                float hi = -INFINITY;
                uint32_t w[16];
                bool over = false;
                if (t < sg.t1) {
                    tc_fence_after();
                    float x[32];
                    tmem_load32(lanes + tm_s + 64 * (g & 1) + 32 * h, x);
                    const uint32_t mask = (uint32_t)tile_mask[g & 3];
                    if (mask == 0xFFu && sg.ctx - p.T + 1 >= (t + 1) * L::kTile) {  // every row sees the whole tile
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] *= p.scale_log2;
                    } else {
                        const int left_of = limit - (t * L::kTile + tok0);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            x[c] = c < left_of && ((mask >> ((tok0 + c) / kBlockSize)) & 1u) ? x[c] * p.scale_log2 : -INFINITY;
                    }
#pragma unroll
                    for (int c = 0; c < 32; ++c) hi = fmaxf(hi, x[c]);
                    if (first || redo) {
                        quarter_at[64 * (side + 2 * h)] = hi;
                        half_sync(group);
                        hi = fmaxf(fmaxf(quarter_at[0], quarter_at[64]), fmaxf(quarter_at[128], quarter_at[192]));
                        const bool up = hi - m > kPairRescale;  // as the weights ask, or a round could end where it began
                        const float f = up ? exp2_sfu(m - hi) : 1.f;
                        if (up) m = hi;
                        if (redo) {
                            l = l_before * f, norm = norm_before * f;
                            exchange(f);
                            left = half_any(group, !ok);
                            if (left) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < 128 && t > sg.t0; c += 16) {
                                uint32_t o[16];
                                const uint32_t at = lanes + tm_o + 128 * h + c;
                                tmem_ld16(at, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * factor[c + k]);
                                tmem_st16(at, o);
                            }
                            tmem_st_wait();
                        }
                        first = redo = false;
                    }
                    over = hi - m > kPairRescale;
                    // weights: bf16, as the product takes them.  Outputs are normalised by the sum of the rounded ones, or a token
                    // that counts for all would scale its row by its own rounding; lse is of the sum of the weights as they are
                    l_here = l, norm_here = norm;
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float a = exp2_sfu(x[c] - m), b = exp2_sfu(x[c + 1] - m);
                        w[c / 2] = pack_bf16x2(a, b);
                        l += a + b;
                        norm += bf16x2_lo(w[c / 2]) + bf16x2_hi(w[c / 2]);
                    }
                }
                if (!clear) {
                    // the product of the last tile, unless its weights were refused
                    wait_for(bar_pv, rounds & 1);
                    pair_acquired(bar_pv, rounds++ & 1);
                    if (!ok) {
                        half_any(group, true);
                        left = true;
                        break;
                    }
                    if ((uint32_t)*verdict == rounds) {
                        --t, --g;
                        redo = clear = true;
                        continue;
                    }
                }
                if (t == sg.t1) break;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    st_shared_v4(p_row + (((4 * h + u) ^ (r & 7)) << 4), make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]));
                fence_proxy_async_shared();
                tc_fence_before();
                __syncwarp();
                if (__any_sync(0xFFFFFFFFu, over) && lane == 0) {
                    st_cluster_u32(raise_there, 1u);
                    pair_fence();
                }
                if (lane == 0) pair_arrive(ready);
                l_before = l_here, norm_before = norm_here, clear = false;
                ++t, ++g;
            }
            if (!left) left = half_any(group, false);
            if (left) {
                ok = false;
                break;
            }
            tc_fence_after();
            const auto all_of = [&](float v) {
                quarter_at[64 * (side + 2 * h)] = v;
                half_sync(group);
                return (quarter_at[0] + quarter_at[64]) + (quarter_at[128] + quarter_at[192]);
            };
            const float all_n = all_of(norm);
            const bool seen = all_n != 0.f;  // (NaN is something)
            const int64_t part = (int64_t)(2 * pair + (sg.t0 == 0)) * 128;  // rows of the workspace
            const int64_t first_row = (int64_t)sg.b * p.rows + sg.chunk * 128;
            exchange(seen ? 1.f / all_n : 0.f);
            left = half_any(group, !ok);
            if (left) {
                ok = false;
                break;
            }
            const float all = all_of(l);  // (behind the vote: the first sums are read)
            if (side + h == 0 && real) {
                const float lse2 = seen ? m + log2f(all) : -INFINITY;
                if (!sg.whole) p.part_lse[part + rank * L::kRows + r] = lse2;
                else if (p.lse_out) p.lse_out[first_row + rank * L::kRows + r] = lse2 * 0.69314718055994530942f;
            }
            // Outputs.  A lane has an element of all rows: a part's row is one line of 32 elements a warp; bf16 outputs pair up, two
            // lanes for two rows.  (Through shared memory in 16-byte units: parts took as long, with all CTAs at it 19 MB in 2.6 us,
            // it is the writes that bound it; bf16 outputs longer, 200 short sequences of 128 heads 37.4 us for 34.4.)
            const int h0 = 256 * rank + 128 * h + 32 * quarter, nrows = min(128, p.rows - sg.chunk * 128);
#pragma unroll 1
            for (int c = 0; c < nrows; c += 16) {
                uint32_t o[16];
                tmem_ld16(lanes + tm_o + 128 * h + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(factor + c + k);
                    const float inv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[k + e] = inv[e] == 0.f ? 0u : __float_as_uint(__uint_as_float(o[k + e]) * inv[e]);
                }
                if (!sg.whole) {
                    float *const to = p.part_out + (part + c) * kLatentDim + h0 + lane;
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (c + k < nrows) to[k * kLatentDim] = __uint_as_float(o[k]);
                    continue;
                }
                // two lanes, two rows: each takes one row's two elements
                __nv_bfloat16 *const to = p.out + (first_row + c + (lane & 1)) * kLatentDim + h0 + (lane & ~1);
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? o[k] : o[k + 1], 1);
                    const float a = __uint_as_float(lane & 1 ? got : o[k]), b = __uint_as_float(lane & 1 ? o[k + 1] : got);
                    if (c + k + (lane & 1) < nrows) *reinterpret_cast<uint32_t *>(to + k * kLatentDim) = pack_bf16x2(a, b);
                }
            }
            tc_fence_before();
            half_sync(group);  // the sums are read
        }
        if (!ok) give_up();
    }

    // ------------------------------ teardown ------------------------------
    __syncthreads();
    cluster_sync();  // neither CTA issues anything any more
    const bool bad = *abort_flag != 0 || load_word(abort_flag, rank ^ 1) != 0;
    if (bad && rank == 0) {
        if (warp == kPairMmaWarp) {
            // every MMA completes before the tensor memories are released
            if (issuer) tc_commit2(bar_fin);
            __syncwarp();
            mbar_wait_bounded(bar_fin, 0u, nullptr, kDrainLimitNs);
        }
        if (warp == kPairLoadWarp && lane == 0) {
            // Every copy on its way, into either CTA, is counted here: it lands before they leave.  A barrier is told to
            // expect what was asked for, where one of the two stopped before the other.
            auto settle = [&](uint32_t bar, int number, int own, int other_number, int other, int told, bool both_arrive) {
                if (number == 0 && other_number == 0) return;
                const int last = max(number, other_number);
                const int coming = (number == last ? own : 0) + (other_number == last ? other : 0);
                if (number != last) {
                    mbar_arrive_expect_tx(bar, (uint32_t)coming);
                    return;
                }
                if (told != coming)
                    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"((uint32_t)(told - coming))
                                 : "memory");
                if (both_arrive && other_number != last) mbar_arrive(bar);
            };
            for (int s = 0; s < L::kStages; ++s) {
                const int mine = use[s], theirs = load_word(use + s, 1);
                settle(bar_full + 8 * s, mine, sent[s], theirs, load_word(sent + s, 1), want[s], true);
                const int last = max(mine, theirs);
                if (last > 0) mbar_wait_bounded(bar_full + 8 * s, (uint32_t)((last - 1) & 1), nullptr, kDrainLimitNs);
            }
            const int mine = *q_asked, theirs = load_word(q_asked, 1), last = max(mine, theirs);
            settle(bar_qfull, mine, L::kQBytes, theirs, L::kQBytes, 2 * L::kQBytes, false);
            if (last > 0) mbar_wait_bounded(bar_qfull, (uint32_t)((last - 1) & 1), nullptr, kDrainLimitNs);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == kPairMmaWarp) {
        tc_fence_after();
        tmem_dealloc2(tm_o, L::kCols);
    }
}

cudaError_t launch_latent_pair(const LatentPairMaps &maps, const LatentAttnParams &params, int sms, cudaStream_t stream)
{
    using L = PairLayout;
    LatentAttnParams p = params;
    static int most[64] = {};  // per device: pairs that run at once
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!most[dev]) {
        e = cudaFuncSetAttribute(latent_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * sms), cfg.blockDim = dim3(kPairThreads), cfg.dynamicSmemBytes = L::kAlloc;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {2, 1, 1};
        cfg.attrs = attr, cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, latent_pair_kernel, &cfg);
        if (e != cudaSuccess) return e;
        most[dev] = max(1, min(n, kLatentMaxCtas / 2));
    }
    // no more pairs than there can be tiles
    const int64_t tiles = (int64_t)p.B * p.chunks * (((int64_t)p.max_nb + L::kBlocks - 1) / L::kBlocks);
    p.ctas = (int)min((int64_t)most[dev], tiles);
    e = launch_clusters(latent_pair_kernel, dim3(2 * p.ctas), dim3(kPairThreads), dim3(2, 1, 1), L::kAlloc, stream, maps, p);
    return e != cudaSuccess ? e : launch_latent_join(p, 128, sms, stream);
}

}  // namespace pkv
