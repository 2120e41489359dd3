// pkv_latent_pair.cu - decode attention over a paged latent cache for sequences of more than 48 (token, head) rows; the
// mathematics is in pkv_latent_attn.cu.  Chunks of up to 128 rows, a cluster of two CTAs each.
//
// With 128 rows a cached row of 1,152 bytes takes 2 * 1088 * 128 operations, 242 a byte, about what the chip has for one
// byte of DRAM, and 128 queries and a 128-token tile are 147 KB each: neither one CTA's shared memory (227 KB) nor its tensor
// memory (128 x 512 sums fill it) holds the problem.  tcgen05.mma with cta_group::2 spreads it over two SMs, and no operand
// is held twice:
//     S[128 x 128 tokens] = Q . C^T        a CTA: its 64 rows of Q; the keys of 64 of the tokens
//     O[128 x 512]       += P . C[:, :512] a CTA: its 64 rows of P; all tokens' values of its 256 elements
// S and O lie in both tensor memories, each CTA's 64 rows: a row's first half of the columns in lane r, its second half in
// lane 64 + r.  One thread of the first CTA issues all MMAs.
//
// The cache streams through a ring of 16 KB stages, a CTA's share of a tile first as keys (64 tokens x 128 elements, four and
// a half stages), then, from L2, as values (32 tokens x 256 elements, four): 138 KB a tile and CTA, of which nothing waits
// for the softmax, so that nearly the whole ring is always under way.  A box is one block's share of a stage, in swizzle
// atoms of 8 rows, [half][chunk][8 rows][128 bytes].  Each CTA's loads are counted on the first CTA's barrier.
//
// CTA = 11 warps: 0-7 softmax (warps w, w + 2, .. share rows 32 (w % 2) ..; of a tile's 128 tokens each thread has a row's 32:
// half of them by lane, half by w / 4), 8 issues the MMAs (first CTA), 9 the loads, 10 zeroes what lies behind a sequence's
// end.  QK^T of tile i + 1 is issued before P V of tile i, so the tensor cores work through the softmax of tile i.
//
// Bound by the tensor cores at half their rate: with 64 rows a CTA an MMA of M = 128 over the pair takes as long as one of
// M = 256 would (61 clocks per N = 128, 122 per N = 256), 4,350 clocks a tile of which the period measured is 4,700.  152
// sequences of 4,096 tokens and 128 heads take 170 us, 1.02 PFLOP/s; 64 of 512 to 8,192 tokens 94 us; one of 131,072 tokens 53.
// The full rate needs the transposed products, M = 256 tokens or elements: built and measured at 134 us for the 64 sequences.
// Both CTAs then need all tokens' weights for half of the rows (16 KB to the other CTA each tile, and common maxima), which
// leaves six 16 KB stages, and a CTA's 278 KB a tile in loads of 2 KB boxes (100 clocks each to issue) come too slowly
// through them.  Fetching tiles ahead into L2 gave nothing (100 to 113 us for 102, one to four tiles ahead).
#include "pkv_cluster.cuh"
#include "pkv_latent.cuh"

namespace pkv {

struct PairLayout {
    static constexpr int kTile = 128, kBlocks = kTile / kBlockSize;
    static constexpr int kRows = 64;                                   // of a CTA
    static constexpr int kStages = 8, kStage = 16384;
    static constexpr int kQChunk = kRows * 128, kQBytes = kLatChunks * kQChunk;
    static constexpr int kPChunk = kRows * 128, kPBytes = 2 * kPChunk;  // 64 tokens a chunk
    static constexpr int kQOffset = 0, kPOffset = kQBytes, kRingOffset = kPOffset + kPBytes;
    static constexpr int kBarOffset = kRingOffset + kStages * kStage;
    // full[S], empty[S], q_full, q_free, s_full[2], p_ready, pv_done, tail[2], fin
    static constexpr int kBars = 2 * kStages + 9;
    static constexpr int kMiscOffset = (kBarOffset + kBars * 8 + 15) & ~15;
    static constexpr int kWords = 4 /* tile masks */ + 4 /* abort, tmem, query loads, - */ + 3 * kStages /* sent, use, want */ + 4 * kRows;
    static constexpr int kBytes = kMiscOffset + kWords * 4;
    static constexpr int kAlloc = kBytes + 1024;                       // room to align the window
    static_assert(kPOffset % 1024 == 0 && kRingOffset % 1024 == 0, "swizzle atoms are aligned");
    static_assert(kAlloc <= 227 * 1024, "shared memory of a CTA");
    static constexpr uint32_t kCols = 512;                             // tensor memory: O 256, S 2 x 64
};
constexpr int kPairSoftmaxWarps = 8, kPairMmaWarp = 8, kPairLoadWarp = 9, kPairTailWarp = 10;
constexpr int kPairThreads = 352;

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

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ int load_word(const volatile int *at, int rank)
{
    return __float_as_int(load_cluster<float>(smem_u32((const void *)at), rank));
}

__global__ void __launch_bounds__(kPairThreads, 1)
latent_pair_kernel(const __grid_constant__ LatentPairMaps maps, const LatentAttnParams p)
{
    using L = PairLayout;
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const mem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)pair_rank(), pair = (int)blockIdx.x >> 1;

    const uint32_t q_u32 = base + L::kQOffset, p_u32 = base + L::kPOffset, ring = base + L::kRingOffset;
    const uint32_t bar_full = base + L::kBarOffset, bar_empty = bar_full + 8 * S, bar_qfull = bar_empty + 8 * S,
                   bar_qfree = bar_qfull + 8, bar_s = bar_qfree + 8, bar_p = bar_s + 16, bar_pv = bar_p + 8, bar_tail = bar_pv + 8,
                   bar_fin = bar_tail + 16;
    volatile int *const tile_mask = reinterpret_cast<volatile int *>(mem + L::kMiscOffset);  // [4], by tile % 4: blocks there
    volatile int *const abort_flag = tile_mask + 4;
    volatile uint32_t *const tmem_slot = reinterpret_cast<volatile uint32_t *>(tile_mask + 5);
    volatile int *const q_asked = tile_mask + 6;
    // of a stage's last use: bytes this CTA asked for, the use's number + 1, bytes the barrier was told (first CTA)
    volatile int *const sent = tile_mask + 8, *const use = sent + S, *const want = use + S;
    float *const quarters = const_cast<float *>(reinterpret_cast<volatile float *>(want + S));  // [4][64]

    // what needs nothing of the launch ahead comes before the wait for it
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *q_asked = 0;
        for (int s = 0; s < S; ++s) sent[s] = use[s] = want[s] = 0;
        for (int k = 0; k < L::kBars; ++k) {
            const uint32_t bar = bar_full + 8 * k;
            // weights: the softmax warps of both CTAs; stages and zeroed rows: both CTAs
            mbar_init(bar, bar == bar_p ? 2 * kPairSoftmaxWarps : k < S || bar == bar_tail + 8 ? 2 : 1);
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
    pdl_wait_primary();
    pdl_launch_dependents();
    LatentWalk<L::kTile> walk;
    int64_t total;
    int pairs;
    // (the sums lie where the queries will; both CTAs find the same)
    const bool work = latent_deal<L::kTile, kPairThreads>(p, pair, reinterpret_cast<int64_t *>(mem), walk, total, pairs);
    if (threadIdx.x == 0) fence_barrier_init();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and tensor memory are there
    tc_fence_after();
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
    bool issuer = false;  // the thread that issues the MMAs (a commit speaks of its thread's)

    if (warp == kPairLoadWarp) {
        // ------------------------------ loads: one thread ------------------------------
        if (elect_one()) {
            const uint32_t full_there = pair_at(bar_full, 0), qfull_there = pair_at(bar_qfull, 0);
            int n = 0;           // stages so far
            uint32_t g = 0, q_loads = 0;
            bool ok = true, withheld = false;
            // Stage n, once it is free; the first CTA's barrier is told what both will send.  The second CTA arrives there for
            // every stage, also for one that it has nothing to send for: the MMAs could otherwise use and release the stage
            // twice before this thread came to wait for the first time (a barrier tells only neighbouring uses apart).
            auto open = [&](int bytes_all, int bytes_own) {
                const int s = n % S;
                if (n >= S) ok = wait_one(bar_empty + 8 * s, (uint32_t)(((n / S) & 1) ^ 1));
                if (!ok) return;
                sent[s] = bytes_own, use[s] = n + 1;
                if (rank == 0) {
                    want[s] = bytes_all;
                    mbar_arrive_expect_tx(bar_full + 8 * s, (uint32_t)bytes_all);
                } else {
                    pair_arrive(full_there + 8 * s);
                }
            };
            int prev[L::kBlocks];
            uint32_t prev_mask = 0;
            auto fill_v = [&](int nblk) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if (2 * v >= nblk) break;
                    const uint32_t two = (prev_mask >> (2 * v)) & 3u;
                    open(2 * __popc(two) * 8192, __popc(two) * 8192);
                    if (!ok) return;
                    const uint32_t dst = ring + (n % S) * L::kStage, bar = full_there + 8 * (n % S);
                    if (two & 1u) pair_load_5d(dst, &maps.values, bar, 0, 0, 4 * rank, 0, prev[2 * v]);
                    if (two & 2u) pair_load_5d(dst + 8192, &maps.values, bar, 0, 0, 4 * rank, 0, prev[2 * v + 1]);
                    ++n;
                }
            };
            LatentSegment sg;
            while (ok && walk.next(p, sg)) {
                // the queries, once the last unit's are no longer needed
                if (q_loads > 0) ok = wait_one(bar_qfree, (q_loads - 1) & 1);
                if (!ok) break;
                const int64_t row = (int64_t)sg.b * p.rows + (int64_t)sg.chunk * 128 + rank * L::kRows;
                *q_asked = (int)++q_loads;
                if (rank == 0) mbar_arrive_expect_tx(bar_qfull, 2 * L::kQBytes);
                for (int c = 0; c < kLatChunks; ++c) pair_load_3d(q_u32 + c * L::kQChunk, &maps.queries, qfull_there, 0, (int)row, c);
                const int nb = (sg.ctx + kBlockSize - 1) / kBlockSize;
                const int32_t *tbl = p.block_tables + (size_t)sg.b * p.max_nb;
                int next[L::kBlocks];
                auto ids_of = [&](int t) {
#pragma unroll
                    for (int k = 0; k < L::kBlocks; ++k) {
                        const int j = t * L::kBlocks + k;
                        next[k] = t < sg.t1 && j < nb ? tbl[j] : -1;
                    }
                };
                ids_of(sg.t0);
                for (int t = sg.t0; t < sg.t1 && ok; ++t, ++g) {
                    const int nblk = min(L::kBlocks, nb - t * L::kBlocks);
                    int ids[L::kBlocks];
                    uint32_t mask = 0;
#pragma unroll
                    for (int k = 0; k < L::kBlocks; ++k) {
                        ids[k] = next[k];
                        mask |= (uint32_t)(ids[k] >= 0 && ids[k] < p.num_blocks) << k;
                    }
                    ids_of(t + 1);
                    if (PKV_TILE_WITHHELD(p, t)) {  // test builds: nothing is loaded or signalled from here on
                        withheld = true, ok = false;
                        break;
                    }
                    if (mask != (1u << nblk) - 1u && rank == 0) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
                    tile_mask[g & 3] = (int)mask;
                    const uint32_t own = (mask >> (4 * rank)) & 0xFu;
                    int mine[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) mine[k] = rank ? ids[4 + k] : ids[k];
#pragma unroll 1
                    for (int c = 0; c < 5; ++c, ++n) {
                        const int bytes = c < 4 ? 4096 : 2048;
                        open(__popc(mask) * bytes, __popc(own) * bytes);
                        if (!ok) break;
                        const CUtensorMap *const map = c < 4 ? &maps.keys : &maps.rope;
                        const uint32_t dst = ring + (n % S) * L::kStage, bar = full_there + 8 * (n % S);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if ((own >> k) & 1u) pair_load_5d(dst + k * bytes, map, bar, 0, 0, 2 * c, 0, mine[k]);
                    }
                    if (t > sg.t0 && ok) fill_v(L::kBlocks);
                    prev_mask = mask;
#pragma unroll
                    for (int k = 0; k < L::kBlocks; ++k) prev[k] = ids[k];
                }
                if (ok) fill_v(min(L::kBlocks, nb - (sg.t1 - 1) * L::kBlocks));
            }
            // every stage and the queries released: no arrival is on its way into this CTA any more
            for (int k = max(0, n - S); k < n && ok; ++k) ok = wait_one(bar_empty + 8 * (k % S), (uint32_t)((k / S) & 1));
            if (ok && q_loads > 0) ok = wait_one(bar_qfree, (q_loads - 1) & 1);
            if (!ok && !withheld) {
                if (!*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
                *abort_flag = 1;
            }
        }
        __syncwarp();
    } else if (warp == kPairTailWarp) {
        // ---------------- rows behind a sequence's end ----------------
        // They may hold anything, and 0 x NaN is NaN: both CTAs zero them before P V reads them, when the MMA thread asks for it
        // (asked and answered in turn, so that neither can be a use of the stage ahead of the other).
        int n = 0;
        uint32_t asked = 0;
        bool ok = true;
        LatentSegment sg;
        while (ok && walk.next(p, sg)) {
            const int count = sg.t1 - sg.t0, tail = sg.ctx % kBlockSize;
            int last = 4;  // stages of the last tile's values
            if (sg.t1 == sg.tiles) {
                const int nblk = (sg.ctx + kBlockSize - 1) / kBlockSize - (sg.tiles - 1) * L::kBlocks;
                last = (nblk + 1) / 2;
                if (tail > 0) {
                    ok = wait(bar_tail, asked++ & 1);
                    if (!ok) break;
                    const int k = n + 5 * count + 4 * (count - 1) + last - 1;
                    const uint32_t blk = ring + (k % S) * L::kStage + ((nblk - 1) & 1) * 8192;
                    for (int x = lane; x < (kBlockSize - tail) * 32; x += 32) {
                        const int u = x & 31, row = tail + (x >> 5);
                        st_shared_v4(blk + (row >> 3) * 4096 + (u >> 3) * 1024 + (row & 7) * 128 + (u & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) pair_arrive(pair_at(bar_tail + 8, 0));
                }
            }
            n += 5 * count + 4 * (count - 1) + last;
        }
        if (!ok) give_up();
    } else if (warp == kPairMmaWarp) {
        // ------------------------------ MMAs: one thread of the first CTA ------------------------------
        issuer = elect_one() && rank == 0;
        if (issuer) {
            constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, 0, 0), kIdO = idesc_bf16_f32(128, 256, 0, 1);
            // descriptors: an address moves the low word alone
            const uint64_t k_desc = smem_desc_sw128(ring, 16, 2048), r_desc = smem_desc_sw128(ring, 16, 1024);
            const uint64_t v_desc = smem_desc_sw128(ring, 1024, 4096);
            const uint64_t q_desc = smem_desc_sw128(q_u32, 16, 1024), p_desc = smem_desc_sw128(p_u32, 16, 1024);
            const uint32_t ask_other = pair_at(bar_tail, 1);
            int n = 0;
            uint32_t g = 0, unit = 0, tails = 0;
            bool ok = true, started = false;
            // P V of tile number gt; has_tail: its last block's end is zeroed first
            auto pv = [&](uint32_t gt, int nblk, bool has_tail) {
                ok = wait_one(bar_p, gt & 1);
                if (!ok) return;
                const uint32_t mask = (uint32_t)tile_mask[gt & 3];
                const int stages = (nblk + 1) / 2;
#pragma unroll 1
                for (int v = 0; v < stages; ++v, ++n) {
                    const int s = n % S;
                    ok = wait_one(bar_full + 8 * s, (uint32_t)((n / S) & 1));
                    if (ok && has_tail && v == stages - 1) {
                        mbar_arrive(bar_tail);
                        pair_arrive(ask_other);
                        ok = wait_one(bar_tail + 8, tails++ & 1);
                    }
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int blk = 2 * v + j;
                        if ((mask >> blk) & 1u) {
                            const uint64_t a = p_desc + (uint32_t)((blk >> 2) * (L::kPChunk >> 4) + 2 * (blk & 3));
                            const uint64_t b = v_desc + (uint32_t)((s * L::kStage + j * 8192) >> 4);
                            tc_mma_ss2(tm_o, a, b, kIdO, started);
                            tc_mma_ss2(tm_o + 128, a, b + (2048 >> 4), kIdO, started);
                            started = true;
                        }
                    }
                    tc_commit2_both(bar_empty + 8 * s);
                }
                tc_commit2_both(bar_pv);
            };
            LatentSegment sg;
            while (ok && walk.next(p, sg)) {
                ok = wait_one(bar_qfull, unit & 1);
                ++unit;
                const int nb = (sg.ctx + kBlockSize - 1) / kBlockSize;
                for (int t = sg.t0; t < sg.t1 && ok; ++t, ++g) {
                    const uint32_t d = tm_s + 64 * (g & 1);
#pragma unroll 1
                    for (int c = 0; c < 5; ++c, ++n) {
                        const int s = n % S;
                        ok = wait_one(bar_full + 8 * s, (uint32_t)((n / S) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t at = (uint32_t)((s * L::kStage) >> 4);
                        const uint64_t a = q_desc + (uint32_t)(2 * c * (L::kQChunk >> 4));
                        if (c < 4) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                tc_mma_ss2(d, a + (k >> 2) * (L::kQChunk >> 4) + 2 * (k & 3), k_desc + at + (k >> 2) * (1024 >> 4) + 2 * (k & 3), kIdS,
                                           c + k > 0);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) tc_mma_ss2(d, a + 2 * k, r_desc + at + 2 * k, kIdS, 1);
                        }
                        tc_commit2_both(bar_empty + 8 * s);
                    }
                    if (!ok) break;
                    tc_commit2_both(bar_s + 8 * (g & 1));
                    if (t + 1 == sg.t1) tc_commit2_both(bar_qfree);
                    if (t > sg.t0) pv(g - 1, L::kBlocks, false);
                    else started = false;
                }
                if (ok) pv(g - 1, min(L::kBlocks, nb - (sg.t1 - 1) * L::kBlocks), sg.t1 == sg.tiles && sg.ctx % kBlockSize > 0);
            }
            if (!ok) {
                if (!*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
                *abort_flag = 1;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------ softmax and outputs ------------------------------
        const int quarter = warp & 3, h = warp >> 2, group = quarter & 1, side = quarter >> 1;
        const int r = 32 * group + lane;              // row of the CTA
        const int tok0 = 64 * side + 32 * h;          // this thread's tokens of a tile
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t ready = pair_at(bar_p, 0);
        const uint32_t p_row = p_u32 + side * L::kPChunk + r * 128;
        float *const quarter_at = quarters + r;
        uint32_t g = 0;
        bool ok = true;
        LatentSegment sg;
        while (ok && walk.next(p, sg)) {
            const int row0 = sg.chunk * 128 + rank * L::kRows;  // first row of this CTA within the sequence
            const bool real = row0 + r < p.rows;
            if (threadIdx.x == 0 && rank == 0 && sg.t0 == 0) {
                // for the joining launch: the first pair of the unit's parts, and how many there are
                const int64_t last = sg.start + sg.tiles + latent_unit_cost<L::kTile>() - 1;
                const int parts = sg.whole ? 1 : (int)(((last + 1) * pairs - 1) / total) - pair + 1;
                p.unit_parts[(int64_t)sg.b * p.chunks + sg.chunk] = make_int2(pair, parts);
            }
            const int limit = real ? sg.ctx - p.T + (row0 + r) / p.N + 1 : 0;  // tokens the row sees
            float m = -FLT_MAX, l = 0.f;
            // The barriers below count all four warps of a group, so a warp whose wait gave up leaves only where
            // all four agree on it, at the votes that open a tile and the outputs.
            bool left = false;
            for (int t = sg.t0; t < sg.t1; ++t, ++g) {
                if (ok) ok = wait(bar_s + 8 * (g & 1), (g >> 1) & 1);
                if (!ok) give_up();
                left = half_any(group, !ok);
                if (left) break;
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
                float hi = -INFINITY;
#pragma unroll
                for (int c = 0; c < 32; ++c) hi = fmaxf(hi, x[c]);
                if (half_any(group, hi - m > kLatRescale)) {
                    quarter_at[64 * (side + 2 * h)] = hi;
                    half_sync(group);
                    hi = fmaxf(fmaxf(quarter_at[0], quarter_at[64]), fmaxf(quarter_at[128], quarter_at[192]));
                    const bool up = hi - m > kLatRescale;
                    const float factor = up ? exp2_sfu(m - hi) : 1.f;
                    if (up) m = hi;
                    l *= factor;
                    if (t > sg.t0) {
                        ok = wait(bar_pv, (g - 1) & 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 128; c += 32) {
                            float o[32];
                            const uint32_t at = lanes + tm_o + 128 * h + c;
                            tmem_load32(at, o);
                            uint32_t w[2][16];
#pragma unroll
                            for (int k = 0; k < 32; ++k) w[k / 16][k % 16] = __float_as_uint(o[k] * factor);
                            tmem_st16(at, w[0]);
                            tmem_st16(at + 16, w[1]);
                        }
                        tmem_st_wait();
                    }
                }
                // weights: rounded to bf16 for the product, summed as they are
                uint32_t w[16];
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float a = exp2_sfu(x[c] - m), b = exp2_sfu(x[c + 1] - m);
                    w[c / 2] = pack_bf16x2(a, b);
                    l += a + b;
                }
                if (g > 0) ok = wait(bar_pv, (g - 1) & 1) && ok;  // the last tile's weights are no longer needed
                if (!ok) give_up();
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    st_shared_v4(p_row + (((4 * h + u) ^ (r & 7)) << 4), make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]));
                fence_proxy_async_shared();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) pair_arrive(ready);
            }
            if (!left) {
                if (ok) ok = wait(bar_pv, (g - 1) & 1);
                if (!ok) give_up();
                left = half_any(group, !ok);
            }
            if (left) {
                ok = false;
                break;
            }
            tc_fence_after();
            quarter_at[64 * (side + 2 * h)] = l;
            half_sync(group);
            const float all = (quarter_at[0] + quarter_at[64]) + (quarter_at[128] + quarter_at[192]);
            const bool seen = all != 0.f;  // (NaN is something)
            const float inv = seen ? 1.f / all : 0.f;
            const int64_t part = (int64_t)(2 * pair + (sg.t0 == 0)) * 128 + rank * L::kRows + r;  // row of the workspace
            const int64_t row = (int64_t)sg.b * p.rows + row0 + r;
            if (side + h == 0 && real) {
                const float lse2 = seen ? m + log2f(all) : -INFINITY;
                if (!sg.whole) p.part_lse[part] = lse2;
                else if (p.lse_out) p.lse_out[row] = lse2 * 0.69314718055994530942f;
            }
            // Outputs.  A thread has a row's elements, its lanes' rows lie 1 or 2 KB apart: 16 elements of 32 rows at a time go
            // through the group's part of P (2 KB a warp, 16-byte units swizzled by row), so that a store covers whole sectors of
            // eight rows (straight from the registers a unit's outputs took 10,500 clocks; a ragged batch of 64 with 128 heads 102 -> 99 us).
            const int h0 = 256 * side + 128 * h;
            const uint32_t stage = p_u32 + group * 4096 + side * L::kPChunk + h * 2048;
            const int64_t part0 = part - lane, row_first = row - lane;
            const int rows_here = min(32, p.rows - (row0 + 32 * group));
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
                uint32_t o[16];
                tmem_ld16(lanes + tm_o + 128 * h + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = seen ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    st_shared_v4(stage + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4), make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]));
                __syncwarp();
                if (sg.whole) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int rr = 16 * k + (lane >> 1), u = 2 * (lane & 1), x = (rr >> 1) & 3;
                        const float4 a = ld_shared_f4(stage + rr * 64 + ((u ^ x) << 4)), b = ld_shared_f4(stage + rr * 64 + (((u + 1) ^ x) << 4));
                        if (rr < rows_here)
                            *reinterpret_cast<uint4 *>(p.out + (row_first + rr) * kLatentDim + h0 + c + 4 * u) =
                                make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int rr = 8 * k + (lane >> 2), u = lane & 3;
                        const float4 v = ld_shared_f4(stage + rr * 64 + ((u ^ ((rr >> 1) & 3)) << 4));
                        if (rr < rows_here) *reinterpret_cast<float4 *>(p.part_out + (part0 + rr) * kLatentDim + h0 + c + 4 * u) = v;
                    }
                }
                __syncwarp();
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
            for (int s = 0; s < S; ++s) {
                const int mine = use[s], theirs = load_word(use + s, 1);
                settle(bar_full + 8 * s, mine, sent[s], theirs, load_word(sent + s, 1), want[s], true);
                const int last = max(mine, theirs);
                if (last > 0) mbar_wait_bounded(bar_full + 8 * s, (uint32_t)(((last - 1) / S) & 1), nullptr, kDrainLimitNs);
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
