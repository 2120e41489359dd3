// pkv_latent_attn.cu - decode attention over a paged latent cache: one row of 576 elements a token, of which all 576
// are every head's key and the first 512 every head's value (the heads' own key and value projections are absorbed into
// the queries before and applied to the outputs after).
//     s[r][j] = scale q[r] . c[j],  out[r] = sum_j softmax(s[r])_j c[j][:512],  r a (token, head) row of a sequence.
//
// This is the kernel for sequences of at most 32 rows (few heads, as one of several GPUs has them); more rows take
// pkv_latent_pair.cu.  All rows share the keys, so that even here the contraction is dense (30 operations a byte with 16 rows)
// and goes to the tcgen05 tensor cores, both products transposed:
//     S^T[64 tokens x R]  = C[64 x 576] . Q^T       A: the tile's rows as they lie (K-major), B: the queries
//     O^T[512 x R]       += C^T[512 x 64] . P^T     A: the same bytes read MN-major (four M = 128 products), B: P
// so that R = 16 or 32 query rows a CTA is the N of the products, not a padded M: the 512 x R accumulator takes 4 R
// of the 512 tensor-memory columns, and a tile is loaded once and read as keys and as values where it lies.
//
// Bound by memory, where there is enough of it: 152 sequences of 4,096 tokens and 16 rows take 117 to 119 us, 6.1 TB/s, 90% of
// a copy's rate; 64 sequences of 512 to 8,192 tokens (325 MB) 63 us with 16 rows and 66 with 32.  One sequence of 2,000 tokens
// takes 10 us: launches, and the dependent loads of lengths, tables and tiles.
//
// A block of 16 tokens is one TMA load of 18 KB, a box of (64 elements, 8 tokens, 9 chunks of elements, 2 halves): it
// lands as [half][chunk][8 rows][128 bytes], swizzle atoms of 8 rows, so that the 8-row groups of consecutive blocks lie
// 9,216 bytes apart throughout and a tile of several blocks is one operand in either reading.
//
// The work is dealt out evenly: the tiles of all (sequence, chunk of rows) units in a row, cut into as many equal runs as
// CTAs run at once.  A unit that one CTA holds whole is written out directly; of one that is cut each part goes to the
// workspace, at most two a CTA, and a second launch joins them by their log-sum-exp.
//
// CTA = 11 warps: 0-7 softmax (warp w: block w % 4 of the tile, a token a lane; half w / 4 of the rows), 8 issues the MMAs,
// 9 the loads, 10 zeroes what lies behind a sequence's end.  QK^T of tile i + 1 is issued before P V of tile i, so the tensor
// cores work through the softmax of tile i.  The running maxima move only when a logit exceeds them by 2^8 (found with one
// barrier vote a tile); the sums stay in the threads' registers, a part for each token lane, until the end.
//
// A weight is rounded to bf16, 2^-8 of it: an MMA has one type for both operands, and the other one is the cache.  (In two terms
// the second product would take twice the MMAs, and in the pair kernel room that there is not.)  Normalised by the sum of the
// rounded weights, outputs are 0.0017 to 0.0020 off in the mean square, bf16 itself 0.0017.  The second sum costs 0.3%: 64
// sequences of 128 heads 76.8 -> 77.1 us.
#include "pkv_latent.cuh"

namespace pkv {

constexpr int kLatGroup = kLatChunks * 1024;                  // bytes of eight tokens: an atom per chunk
constexpr int kLatBlock = 2 * kLatGroup;                      // and of a block
constexpr int kLatSoftmaxWarps = 8, kLatMmaWarp = 8, kLatLoadWarp = 9, kLatTailWarp = 10;
constexpr int kLatThreads = 352;

// R: query rows of a CTA.
template <int R>
struct LatentLayout {
    static_assert(R == 16 || R == 32, "rows of a CTA");
    static constexpr int kBlocks = 3;                    // blocks of a tile (M = 64: at most four)
    static constexpr int kSlots = 3;                     // tiles in shared memory
    static constexpr int kTile = kBlocks * kBlockSize;   // tokens of a tile
    static constexpr int kRing = kSlots * kBlocks;
    static constexpr int kQChunk = R * 128;              // 64 elements of R queries, K-major, 128-byte swizzle
    static constexpr int kQBytes = kLatChunks * kQChunk;
    static constexpr int kPLine = R * 2;                 // bytes of one token's weights: a swizzle atom's row
    static constexpr int kPBytes = kTile * kPLine;
    static constexpr int kRingOffset = 0;
    static constexpr int kQOffset = kRing * kLatBlock;
    static constexpr int kPOffset = kQOffset + kQBytes;
    static constexpr int kBarOffset = kPOffset + ((kPBytes + 1023) & ~1023);
    // full[slots], empty[ring], q_full, q_free, s_full[2], p_ready, pv_done, tail[2], fin
    static constexpr int kBars = kSlots + kRing + 9;
    static constexpr int kMiscOffset = (kBarOffset + kBars * 8 + 15) & ~15;
    static constexpr int kWords = 4 /* tile masks */ + 4 /* abort, tmem, tiles, - */ + 2 * 4 /* - */ + R /* limits */ +
                                  R /* maxima */ + R /* factors */ + 8 * R /* of four warps */;
    static constexpr int kBytes = kMiscOffset + kWords * 4;
    static constexpr int kAlloc = kBytes + 1024;  // room to align the window
    static_assert(kQOffset % 1024 == 0 && kPOffset % 1024 == 0 && kSlots <= 4, "swizzle atoms are aligned");
    static_assert((kSlots - 1) * kBlocks * kLatBlock + 8 * kLatGroup <= kBytes, "M = 64 rows from any slot on lie inside the window");
    static_assert(kAlloc <= 227 * 1024, "shared memory of a CTA");
    static constexpr uint32_t kCols = R == 32 ? 256 : 128;  // tensor memory: O^T 4 R, S^T 2 R
};

// ---- small pieces -------------------------------------------------------------------------------
// Descriptor of P^T as an MN-major operand of R elements a row: the swizzle is as wide as the row.
template <int R>
__device__ __forceinline__ uint64_t latent_p_desc(uint32_t addr)
{
    constexpr uint64_t kMode = R == 32 ? 4 : 6;
    constexpr uint32_t kGroup = 8 * R * 2;  // eight tokens
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(kGroup >> 4) << 16) | ((uint64_t)(kGroup >> 4) << 32) | (1ull << 46) |
           (kMode << 61);
}

// Where 16-byte unit u of token t's weights lies.
template <int R>
__device__ __forceinline__ uint32_t latent_p_at(int t, int u)
{
    const int x = R == 32 ? (t >> 1) & 3 : (t >> 2) & 1;
    return (uint32_t)(t * (R * 2) + ((u ^ x) << 4));
}

// C columns of a warp's 32 lanes (C = 8, 16 or 32).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
template <int C>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&x)[C])
{
    if constexpr (C == 8) {
        uint32_t r[8];
        tmem_ld8(taddr, r);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = __uint_as_float(r[c]);
    } else {
        uint32_t r[C / 16][16];
#pragma unroll
        for (int k = 0; k < C / 16; ++k) tmem_ld16(taddr + 16 * k, r[k]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = __uint_as_float(r[c / 16][c % 16]);
    }
}
template <int C>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const float (&x)[C])
{
    if constexpr (C == 8) {
        uint32_t r[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) r[c] = __float_as_uint(x[c]);
        tmem_st8(taddr, r);
    } else {
#pragma unroll
        for (int k = 0; k < C / 16; ++k) {
            uint32_t r[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(x[16 * k + c]);
            tmem_st16(taddr + 16 * k, r);
        }
    }
}

// Reduce column c of a warp's 32 lanes for C columns at once; lane l receives column l % C.  x is used up.
template <int C, typename Op>
__device__ __forceinline__ float reduce_columns(float (&x)[C], int lane, Op op)
{
#pragma unroll
    for (int o = C / 2; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float give = up ? x[j] : x[j + o], keep = up ? x[j + o] : x[j];
            x[j] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
        }
    }
    float v = x[0];
#pragma unroll
    for (int o = C; o < 32; o <<= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

template <int R>
__global__ void __launch_bounds__(kLatThreads, 1)
latent_attn_kernel(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_q, const LatentAttnParams p)
{
    using L = LatentLayout<R>;
    constexpr int NB = L::kBlocks, NS = L::kSlots, kRing = L::kRing;
    constexpr int CW = R / 2;  // rows (columns of S^T) of a softmax thread
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const mem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

    const uint32_t q_u32 = base + L::kQOffset, p_u32 = base + L::kPOffset, ring = base + L::kRingOffset;
    const uint32_t bar_full = base + L::kBarOffset, bar_empty = bar_full + 8 * NS, bar_qfull = bar_empty + 8 * kRing,
                   bar_qfree = bar_qfull + 8, bar_s = bar_qfree + 8, bar_p = bar_s + 16, bar_pv = bar_p + 8, bar_tail = bar_pv + 8,
                   bar_fin = bar_tail + 16;
    volatile int *const tile_mask = reinterpret_cast<volatile int *>(mem + L::kMiscOffset);  // [4], by tile % 4: blocks there
    volatile int *const abort_flag = tile_mask + 4;
    volatile uint32_t *const tmem_slot = reinterpret_cast<volatile uint32_t *>(tile_mask + 5);
    volatile int *const tiles_begun = tile_mask + 6;                             // by the MMA thread
    int *const limit = const_cast<int *>(tile_mask + 16);                        // [R] tokens a row sees
    float *const top = reinterpret_cast<float *>(limit + R);                     // [R] running maxima (log2)
    float *const factor = top + R;                                               // [R]
    float *const quarters = factor + R, *const quarters_n = quarters + 4 * R;    // [4][R]

    // What needs nothing of the launch ahead comes before the wait for it.  (Tensor memory too: a CTA that still has to take its own
    // does not fit beside this one's shared memory, so none of that launch waits for what is held here.)
    if (threadIdx.x == 0) {
        *abort_flag = 0, *tiles_begun = 0;
        for (int s = 0; s < NS + kRing + 9; ++s) mbar_init(bar_full + 8 * s, s == NS + kRing + 4 ? kLatSoftmaxWarps : 1);
        prefetch_tensormap(&tm_c);
        prefetch_tensormap(&tm_q);
    }
    if (warp == kLatMmaWarp) {
        tmem_alloc(smem_u32((const void *)tmem_slot), L::kCols);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) fence_barrier_init();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait_primary();
    pdl_launch_dependents();
    LatentWalk<L::kTile> walk;
    int64_t total;
    int ctas;
    // (the sums lie where the first tiles will)
    const bool work = latent_deal<L::kTile, kLatThreads>(p, cta, reinterpret_cast<int64_t *>(mem), walk, total, ctas);
    if (!work) {
        if (warp == kLatMmaWarp) tmem_dealloc(*tmem_slot, L::kCols);
        return;
    }
    const uint32_t tm_o = *tmem_slot, tm_s = tm_o + 4 * R;

    auto give_up = [&]() {
        if (lane == 0 && !*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
        *abort_flag = 1;
    };
    auto wait_one = [&](uint32_t bar, uint32_t parity) { return latent_wait(bar, parity, abort_flag, p.wait_ns); };
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait_one(bar, parity)); };

    bool issuer = false;  // of the loading and the MMA warp: the thread that issues
    // of the loading thread: tiles begun, bytes of the last one that were not asked for, segments whose queries were
    uint32_t g_loads = 0, missing = 0, q_loads = 0;
    if (warp == kLatLoadWarp) {
        // ------------------------------ loads: one thread ------------------------------
        issuer = elect_one();
        if (issuer) {
            bool ok = true, withheld = false;
            int slot = 0;
            uint32_t parity = 0;  // of the slot's uses
            LatentSegment sg;
            while (ok && walk.next(p, sg)) {
                const int nb = (sg.ctx + kBlockSize - 1) / kBlockSize;
                const int32_t *tbl = p.block_tables + (size_t)sg.b * p.max_nb;
                int next[NB];
                auto ids_of = [&](int t) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) next[k] = t < sg.t1 && t * NB + k < nb ? tbl[t * NB + k] : -1;
                };
                ids_of(sg.t0);
                // the queries, once the last unit's are no longer needed
                if (q_loads > 0) ok = wait_one(bar_qfree, (q_loads - 1) & 1);
                if (!ok) break;
                const int64_t row = (int64_t)sg.b * p.rows + (int64_t)sg.chunk * R;
                mbar_arrive_expect_tx(bar_qfull, L::kQBytes);
                for (int c = 0; c < kLatChunks; ++c) tma_load_3d(q_u32 + c * L::kQChunk, &tm_q, bar_qfull, 0, (int)row, c);
                ++q_loads;
                for (int t = sg.t0; t < sg.t1 && ok; ++t) {
                    const int nblk = min(NB, nb - t * NB);
                    int ids[NB];
                    uint32_t mask = 0;
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        ids[k] = next[k];
                        mask |= (uint32_t)(ids[k] >= 0 && ids[k] < p.num_blocks) << k;
                    }
                    ids_of(t + 1);
                    if (PKV_TILE_WITHHELD(p, t)) {  // test builds: nothing is loaded or signalled from here on
                        withheld = true, ok = false;
                        break;
                    }
                    if (mask != (1u << nblk) - 1u) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
                    const uint32_t bar = bar_full + 8 * slot;
                    const bool used = g_loads >= NS;
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        if (ok && used) ok = wait_one(bar_empty + 8 * (slot * NB + j), parity ^ 1u);
                        if (!ok) continue;
                        if (j == 0) {
                            missing = (uint32_t)__popc(mask) * kLatBlock;
                            tile_mask[g_loads++ & 3] = (int)mask;
                            mbar_arrive_expect_tx(bar, missing);
                        }
                        if ((mask >> j) & 1u) {
                            tma_load_5d(ring + (slot * NB + j) * kLatBlock, &tm_c, bar, 0, 0, 0, 0, ids[j]);
                            missing -= kLatBlock;
                        }
                    }
                    if (++slot == NS) slot = 0, parity ^= 1u;
                }
            }
            if (!ok && !withheld) {
                if (!*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
                *abort_flag = 1;
            }
        }
        __syncwarp();
    } else if (warp == kLatTailWarp) {
        // ---------------- rows behind a sequence's end ----------------
        // They may hold anything, and 0 x NaN is NaN: they are zeroed before P V reads them, when the MMA warp asks for it
        // (asked and answered in turn, so that neither can be a use of the slot ahead of the other).
        uint32_t g = 0, asked = 0;
        bool ok = true;
        LatentSegment sg;
        while (ok && walk.next(p, sg)) {
            g += sg.t1 - sg.t0;
            const int tail = sg.ctx % kBlockSize;
            if (sg.t1 != sg.tiles || tail == 0) continue;
            // (the limit is of a step of the pipeline, and this wait goes over all tiles of the run up to here: it begins
            // again while the MMA thread gets on)
            int begun;
            do {
                begun = *tiles_begun;
                ok = wait(bar_tail, asked & 1);
            } while (!ok && __any_sync(0xFFFFFFFFu, *tiles_begun != begun) && __all_sync(0xFFFFFFFFu, !*abort_flag));
            if (!ok) break;
            ++asked;
            const int j = (sg.ctx / kBlockSize) - (sg.tiles - 1) * NB;
            const uint32_t blk = ring + ((int)((g - 1) % NS) * NB + j) * kLatBlock;
            // 16-byte units of the values' eight chunks
            for (int x = lane; x < (kBlockSize - tail) * 64; x += 32) {
                const int u = x & 63, row = tail + (x >> 6);
                st_shared_v4(blk + (row >> 3) * kLatGroup + (u >> 3) * 1024 + (row & 7) * 128 + (u & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_tail + 8);
        }
        if (!ok) give_up();
    } else if (warp == kLatMmaWarp) {
        // ------------------------------ MMAs: one thread ------------------------------
        // (whole warps at these waits and issues took 700 clocks for what takes one thread 150)
        issuer = elect_one();
        if (issuer) {
            constexpr uint32_t kIdS = idesc_bf16_f32(64, R, 0, 0), kIdO = idesc_bf16_f32(128, R, 1, 1);
            // descriptors: an address moves the low word alone
            const uint64_t k_desc = smem_desc_sw128(ring, 16, kLatGroup), q_desc = smem_desc_sw128(q_u32, 16, 1024);
            const uint64_t v_desc = smem_desc_sw128(ring, 1024, kLatGroup), p_desc = latent_p_desc<R>(p_u32);
            uint32_t g = 0, unit = 0, tails = 0, parity = 0;
            int slot = 0, pv_slot = 0;
            bool ok = true, started = false;
            // P V of tile number gt; has_tail: its last block's end is zeroed first
            auto pv = [&](uint32_t gt, bool has_tail) {
                ok = wait_one(bar_p, gt & 1);
                if (ok && has_tail) {
                    mbar_arrive(bar_tail);
                    ok = wait_one(bar_tail + 8, tails++ & 1);
                }
                if (!ok) return;
                tc_fence_after();
                const uint32_t mask = (uint32_t)tile_mask[gt & 3];
#pragma unroll 1
                for (int j = 0; j < NB; ++j) {
                    const int blk = pv_slot * NB + j;
                    if ((mask >> j) & 1u) {
                        const uint64_t a = v_desc + (uint32_t)(blk * (kLatBlock >> 4)), b = p_desc + (uint32_t)(j * (kBlockSize * L::kPLine >> 4));
#pragma unroll
                        for (int m = 0; m < 4; ++m) tc_mma_ss(tm_o + m * R, a + m * (2048 >> 4), b, kIdO, started);
                        started = true;
                    }
                    tc_commit(bar_empty + 8 * blk);
                }
                tc_commit(bar_pv);
                if (++pv_slot == NS) pv_slot = 0;
            };
            LatentSegment sg;
            while (ok && walk.next(p, sg)) {
                ok = wait_one(bar_qfull, unit & 1);
                ++unit;
                for (int t = sg.t0; t < sg.t1 && ok; ++t, ++g) {
                    ok = wait_one(bar_full + 8 * slot, parity);
                    if (!ok) break;
                    tc_fence_after();
                    *tiles_begun = (int)g + 1;
                    const uint32_t d = tm_s + R * (g & 1);
                    const uint64_t a = k_desc + (uint32_t)(slot * NB * (kLatBlock >> 4));
#pragma unroll
                    for (int c = 0; c < kLatChunks; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_ss(d, a + c * (1024 >> 4) + 2 * k, q_desc + c * (L::kQChunk >> 4) + 2 * k, kIdS, c + k > 0);
                    tc_commit(bar_s + 8 * (g & 1));
                    if (++slot == NS) slot = 0, parity ^= 1u;
                    if (t + 1 == sg.t1) tc_commit(bar_qfree);
                    if (t > sg.t0) pv(g - 1, false);
                    else started = false;
                }
                if (ok) pv(g - 1, sg.t1 == sg.tiles && sg.ctx % kBlockSize > 0);
            }
            if (!ok) {
                if (!*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
                *abort_flag = 1;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------ softmax and outputs ------------------------------
        // S^T has M = 64: its rows 16 q .. lie in tensor-memory lanes 32 q .. 32 q + 15
        const int quarter = warp & 3, half = warp >> 2, tok = 16 * quarter + lane, c0 = half * CW;
        const bool token = lane < 16 && quarter < NB;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const int col = lane & (CW - 1);  // the column this lane holds after a reduction
        uint32_t g = 0;
        bool ok = true;
        LatentSegment sg;
        while (ok && walk.next(p, sg)) {
            const int row0 = sg.chunk * R;  // first row of this unit within the sequence
            const int nrows = min(R, p.rows - row0);
            if (threadIdx.x == 0 && sg.t0 == 0) {
                // for the joining launch: the first CTA of the unit's parts, and how many there are
                const int64_t last = sg.start + sg.tiles + kLatentUnitCost - 1;
                const int parts = sg.whole ? 1 : (int)(((last + 1) * ctas - 1) / total) - cta + 1;
                p.unit_parts[(int64_t)sg.b * p.chunks + sg.chunk] = make_int2(cta, parts);
            }
            if (quarter == 0 && lane < CW) {
                const int r = row0 + c0 + lane;
                limit[c0 + lane] = c0 + lane < nrows ? sg.ctx - p.T + r / p.N + 1 : 0;
                top[c0 + lane] = -FLT_MAX;
            }
            half_sync(half);
            float l[CW], norm[CW];  // sums of the weights, as they are and as the product has them
#pragma unroll
            for (int c = 0; c < CW; ++c) l[c] = norm[c] = 0.f;
            // The barriers below count all four warps of a half, so a warp whose wait gave up leaves only where
            // all four agree on it, at the votes that open a tile and the outputs.
            bool left = false;
            for (int t = sg.t0; t < sg.t1; ++t, ++g) {
                if (ok) ok = wait(bar_s + 8 * (g & 1), (g >> 1) & 1);
                if (!ok) give_up();
                left = half_any(half, !ok);
                if (left) break;
                tc_fence_after();
                float x[CW];
                tmem_load<CW>(lanes + tm_s + R * (g & 1) + c0, x);
                const int at = t * L::kTile + tok;
                const bool here = token && at < sg.ctx && (((uint32_t)tile_mask[g & 3] >> quarter) & 1u);
                if (sg.ctx - p.T + 1 >= (t + 1) * L::kTile) {  // every row sees the whole tile
#pragma unroll
                    for (int c = 0; c < CW; ++c) x[c] = here ? x[c] * p.scale_log2 : -INFINITY;
                } else {
#pragma unroll
                    for (int c = 0; c < CW; ++c) x[c] = here && at < limit[c0 + c] ? x[c] * p.scale_log2 : -INFINITY;
                }
                float m[CW];
                auto load_top = [&]() {
#pragma unroll
                    for (int c = 0; c < CW; c += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(top + c0 + c);
                        m[c] = v.x, m[c + 1] = v.y, m[c + 2] = v.z, m[c + 3] = v.w;
                    }
                };
                load_top();
                float over = -INFINITY;
#pragma unroll
                for (int c = 0; c < CW; ++c) over = fmaxf(over, x[c] - m[c]);
                const bool raise = half_any(half, over > kLatRescale);
                if (raise) {
                    float v[CW];
#pragma unroll
                    for (int c = 0; c < CW; ++c) v[c] = x[c];
                    const float w = reduce_columns<CW>(v, lane, [](float a, float b) { return fmaxf(a, b); });
                    if (lane < CW) quarters[quarter * R + c0 + lane] = w;
                    half_sync(half);
                    if (quarter == 0 && lane < CW) {
                        const float *f = quarters + c0 + lane;
                        const float hi = fmaxf(fmaxf(f[0], f[R]), fmaxf(f[2 * R], f[3 * R])), old = top[c0 + lane];
                        const bool up = hi > old + kLatRescale || (old == -FLT_MAX && hi > old);
                        factor[c0 + lane] = up ? exp2_sfu(old - hi) : 1.f;
                        if (up) top[c0 + lane] = hi;
                    }
                    half_sync(half);
                    if (g > 0) ok = wait(bar_pv, (g - 1) & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int mb = 0; mb < 4 && t > sg.t0; ++mb) {
                        tmem_load<CW>(lanes + tm_o + mb * R + c0, v);
#pragma unroll
                        for (int c = 0; c < CW; ++c) v[c] *= factor[c0 + c];
                        tmem_store<CW>(lanes + tm_o + mb * R + c0, v);
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int c = 0; c < CW; ++c) l[c] *= factor[c0 + c], norm[c] *= factor[c0 + c];
                }
                load_top();  // (again: held across the vote the maxima would not fit the registers of 32 rows)
                // weights: bf16, as the product takes them.  Outputs are normalised by the sum of the rounded ones, or a token
                // that counts for all would scale its row by its own rounding; lse is of the sum of the weights as they are
                uint32_t w[CW / 2];
#pragma unroll
                for (int c = 0; c < CW; c += 2) {
                    const float a = exp2_sfu(x[c] - m[c]), b = exp2_sfu(x[c + 1] - m[c + 1]);
                    w[c / 2] = pack_bf16x2(a, b);
                    l[c] += a;
                    l[c + 1] += b;
                    norm[c] += bf16x2_lo(w[c / 2]);
                    norm[c + 1] += bf16x2_hi(w[c / 2]);
                }
                if (g > 0) ok = wait(bar_pv, (g - 1) & 1) && ok;  // the last tile's weights are no longer needed
                if (!ok) give_up();
#pragma unroll
                for (int u = 0; u < CW / 8; ++u)
                    if (token) st_shared_v4(p_u32 + latent_p_at<R>(tok, c0 / 8 + u), make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]));
                fence_proxy_async_shared();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(bar_p);
            }
            if (!left) {
                if (ok) ok = wait(bar_pv, (g - 1) & 1);
                left = half_any(half, !ok);
            }
            if (left) {
                ok = false;
                break;
            }
            tc_fence_after();
            // sums over the tokens: of the warp, then of the four warps
            const auto add = [](float a, float b) { return a + b; };
            const float sum = reduce_columns<CW>(l, lane, add), sum_n = reduce_columns<CW>(norm, lane, add);
            if (lane < CW) quarters[quarter * R + c0 + lane] = sum, quarters_n[quarter * R + c0 + lane] = sum_n;
            half_sync(half);
            const float *f = quarters + c0 + col, *fn = quarters_n + c0 + col;
            const float all = (f[0] + f[R]) + (f[2 * R] + f[3 * R]), all_n = (fn[0] + fn[R]) + (fn[2 * R] + fn[3 * R]), hi = top[c0 + col];
            const bool seen = all != 0.f;  // (NaN is something)
            const int64_t part = (int64_t)(2 * cta + (sg.t0 == 0)) * R;  // rows of the workspace
            if (quarter == 0 && lane < CW && c0 + lane < nrows) {
                const float lse2 = seen ? hi + log2f(all) : -INFINITY;
                const int64_t row = (int64_t)sg.b * p.rows + row0 + c0 + lane;
                if (!sg.whole) p.part_lse[part + c0 + lane] = lse2;
                else if (p.lse_out) p.lse_out[row] = lse2 * 0.69314718055994530942f;
            }
            if (quarter == 0 && lane < CW) factor[c0 + lane] = seen ? 1.f / all_n : 0.f;
            half_sync(half);
            float inv[CW];
#pragma unroll
            for (int c = 0; c < CW; ++c) inv[c] = factor[c0 + c];
#pragma unroll 1
            for (int mb = 0; mb < 4; ++mb) {
                float o[CW];
                tmem_load<CW>(lanes + tm_o + mb * R + c0, o);
                const int h = mb * 128 + 32 * quarter + lane;
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    if (c0 + c >= nrows) break;
                    const float v = inv[c] == 0.f ? 0.f : o[c] * inv[c];
                    if (sg.whole) p.out[((int64_t)sg.b * p.rows + row0 + c0 + c) * kLatentDim + h] = __float2bfloat16_rn(v);
                    else p.part_out[(part + c0 + c) * kLatentDim + h] = v;
                }
            }
            tc_fence_before();
            half_sync(half);  // limits, maxima and factors are read
        }
        if (!ok) give_up();
    }

    // ------------------------------ teardown ------------------------------
    __syncthreads();
    if (*abort_flag) {
        if (warp == kLatMmaWarp) {
            // every MMA this CTA issued completes before its tensor memory is released
            if (issuer) tc_commit(bar_fin);
            __syncwarp();
            mbar_wait_bounded(bar_fin, 0u, nullptr, kDrainLimitNs);
        }
        if (warp == kLatLoadWarp && issuer) {
            // every copy on its way lands before this CTA leaves; what the last tile still expects was never asked for
            if (missing)
                asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar_full + 8 * ((g_loads - 1) % NS)), "r"(missing)
                             : "memory");
            for (uint32_t k = g_loads > NS ? g_loads - NS : 0; k < g_loads; ++k)
                mbar_wait_bounded(bar_full + 8 * (k % NS), (k / NS) & 1, nullptr, kDrainLimitNs);
            if (q_loads > 0) mbar_wait_bounded(bar_qfull, (q_loads - 1) & 1, nullptr, kDrainLimitNs);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kLatMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tm_o, L::kCols);
    }
}

// ---- joining the parts of units that were cut -----------------------------------------------------
// out = sum_p e^(lse_p - lse) out_p, as in the other merges of partial softmaxes.  A CTA takes kRows rows of a unit and leaves
// at once where the unit was not cut; it also writes the rows of sequences without tokens, which no CTA of the attention has.
// Warps compute the rows' weights, then 128 threads take a row's elements, four each, and kGroups such groups the rows, or
// the parts of the one row.  Few rows are cut into many parts (one sequence over the whole GPU into up to 152): one row a
// CTA, eight groups that take every eighth part (one sequence of 128K tokens: one group 63 us, four 45.9, eight 43.8).  Rows of
// larger batches are cut into two or three if at all: two rows a CTA while the CTAs run at once (5 short sequences of 128 heads
// 23.8 us, four rows 26.6, eight 29.8), then eight, the fewest CTAs (152 sequences of 4,096 tokens 133.7 us, four rows 136.3, two
// 141.8; 200 short ones 37.7, 41.0, 47.2).
template <int kRows, int kGroups>
__global__ void __launch_bounds__(kGroups * kLatentDim / 4) latent_join_kernel(const LatentAttnParams p, int chunk_rows)
{
    constexpr int kThreads = kGroups * kLatentDim / 4, kWarps = kThreads / 32;
    constexpr bool kSplitParts = kRows == 1;  // the groups share the parts, else the rows
    __shared__ float weight[kRows][kLatentMaxCtas];
    __shared__ float lse_of[kRows];
    __shared__ float4 sums[kSplitParts ? kGroups : 1][kLatentDim / 4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = tid / (kLatentDim / 4), e = tid % (kLatentDim / 4);
    pdl_wait_primary();
    pdl_launch_dependents();
    const int pieces = (chunk_rows + kRows - 1) / kRows;
    const int64_t unit = blockIdx.x / pieces;
    const int cr = (int)(blockIdx.x - unit * pieces) * kRows;  // first row within the chunk
    const int b = (int)(unit / p.chunks), r0 = (int)(unit - (int64_t)b * p.chunks) * chunk_rows + cr, rows = min(kRows, p.rows - r0);
    const int2 info = __ldcg(p.unit_parts + unit);
    const bool empty = latent_ctx(p, b) <= 0;
    const int first = max(0, min(info.x, p.ctas - 1)), parts = empty ? 0 : max(0, min(info.y, p.ctas - first));
    if (rows <= 0 || parts == 1) return;
    const int64_t row0 = (int64_t)b * p.rows + r0;
    // part k of the unit lies in the last part of the first CTA and in the first parts of those behind it
    auto place = [&](int k, int row) { return (int64_t)(2 * (first + k) + (k == 0)) * chunk_rows + cr + row; };
    for (int row = warp; row < rows; row += kWarps) {
        float hi = -INFINITY;
        for (int k = lane; k < parts; k += 32) hi = fmaxf(hi, weight[row][k] = __ldcg(p.part_lse + place(k, row)));
#pragma unroll
        for (int o = 16; o; o >>= 1) hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
        float sum = 0.f;
        const float m = hi == -INFINITY ? 0.f : hi;
        for (int k = lane; k < parts; k += 32) sum += weight[row][k] = exp2f(weight[row][k] - m);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float inv = sum > 0.f ? 1.f / sum : sum;  // no key seen: 0; NaN stays
        for (int k = lane; k < parts; k += 32) weight[row][k] *= inv;
        if (lane == 0) lse_of[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
    }
    auto part_at = [&](int k, int row) { return __ldcg(reinterpret_cast<const float4 *>(p.part_out + place(k, row) * kLatentDim) + e); };
    auto add = [](float4 &a, float w, const float4 &v) { a.x += w * v.x, a.y += w * v.y, a.z += w * v.z, a.w += w * v.w; };
    auto write = [&](int row, const float4 &a) {
        reinterpret_cast<uint2 *>(p.out + (row0 + row) * kLatentDim)[e] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
        if (e == 0 && p.lse_out) p.lse_out[row0 + row] = lse_of[row];
    };
    if constexpr (kSplitParts) {
        constexpr int kAtOnce = 6;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = group; k0 < parts; k0 += kAtOnce * kGroups) {
            float4 v[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                v[j] = k0 + j * kGroups < parts ? part_at(k0 + j * kGroups, 0) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 == group) __syncthreads();  // the first parts' loads go out before the weights are known
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                if (k0 + j * kGroups < parts) add(acc, weight[0][k0 + j * kGroups], v[j]);
        }
        if (group >= parts) __syncthreads();
        sums[group][e] = acc;
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int g = 1; g < kGroups; ++g) add(acc, 1.f, sums[g][e]);
            write(0, acc);
        }
    } else {
        constexpr int kMine = kRows / kGroups;
        float4 acc[kMine], v[2][kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        auto load = [&](int k, float4 (&to)[kMine]) {
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                to[i] = k < parts && group + i * kGroups < rows ? part_at(k, group + i * kGroups) : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        load(0, v[0]);
        load(1, v[1]);
        __syncthreads();
        for (int k = 0; k < parts; k += 2) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (k + j < parts && group + i * kGroups < rows) add(acc[i], weight[group + i * kGroups][k + j], v[j][i]);
                load(k + j + 2, v[j]);
            }
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (group + i * kGroups < rows) write(group + i * kGroups, acc[i]);
    }
}

cudaError_t launch_latent_join(const LatentAttnParams &p, int chunk_rows, int sms, cudaStream_t stream)
{
    const int64_t rows = (int64_t)p.B * p.chunks * chunk_rows;
    const auto launch = [&](auto kernel, int rows_a_cta, int groups) {
        return launch_kernel(kernel, dim3((unsigned)(rows / rows_a_cta)), dim3(groups * kLatentDim / 4), 0, stream, true, p, chunk_rows);
    };
    if (rows <= 4 * (int64_t)sms) return launch(latent_join_kernel<1, 8>, 1, 8);
    if (rows <= 32 * (int64_t)sms) return launch(latent_join_kernel<2, 2>, 2, 2);
    return launch(latent_join_kernel<8, 2>, 8, 2);
}

template <int R>
static cudaError_t latent_attn_t(const CUtensorMap &tc, const CUtensorMap &tq, LatentAttnParams p, int sms, cudaStream_t stream)
{
    using L = LatentLayout<R>;
    static int ready[64] = {};  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(latent_attn_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
        if (e != cudaSuccess) return e;
        ready[dev] = 1;
    }
    // no more CTAs than there can be tiles
    const int64_t tiles = (int64_t)p.B * p.chunks * (((int64_t)p.max_nb + L::kBlocks - 1) / L::kBlocks);
    p.ctas = (int)min((int64_t)min(sms, kLatentMaxCtas), tiles);
    e = launch_kernel(latent_attn_kernel<R>, dim3(p.ctas), dim3(kLatThreads), L::kAlloc, stream, true, tc, tq, p);
    return e != cudaSuccess ? e : launch_latent_join(p, R, sms, stream);
}

cudaError_t launch_latent_attn(const CUtensorMap &tc, const CUtensorMap &tq, const LatentAttnParams &p, int cta_rows, int sms,
                               cudaStream_t stream)
{
    return cta_rows == 32 ? latent_attn_t<32>(tc, tq, p, sms, stream) : latent_attn_t<16>(tc, tq, p, sms, stream);
}

}  // namespace pkv
