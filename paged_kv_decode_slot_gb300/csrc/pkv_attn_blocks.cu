// pkv_attn_blocks.cu - decode attention over selected blocks of a paged cache.
//
// Every (sequence, KV head) brings a list of logical blocks; its G query heads attend to the tokens of those
// blocks alone.  The work is that of the dense kernel on a list in place of the table's leading blocks: TMA
// loads of one (block, KV head) tile each, streamed by producer warps into a ring of shared-memory stages, and
// consumer warps that keep an online softmax over the tiles they take (see pkv_attn.cu).  What differs:
//  * a tile's block id takes two dependent loads (list entry, table entry), looked up 32 tiles ahead of use by
//    the producer's lanes; the list's first entries are fetched before the sequence's length is there;
//  * the tokens that count of a tile follow from its logical block, not from its place in the list: the
//    producer leaves that number with the stage (0 for an entry to skip);
//  * the weights enter the product P V as pairs of 16-bit numbers and the running sum takes them in fp32 (kPairs in
//    pkv_attn_common.cuh), so that neither the output nor lse carries a rounding of the weights to 16 bits: with one
//    16-bit weight each, 64 sequences took 86.1 us instead of 87.9 and the e4m3 batch below 44.6 instead of 46.7.
// One CTA per (KV head, sequence, partition of the list); a list's partitions are one cluster, which joins their partial
// results in its shared memory, or (many of them) the last to finish joins them from the workspace.
// Bound by memory: 32 H bytes of K and as many of V per tile and two bytes an element.  64 sequences of 512 to 8,192 tokens,
// up to 128 blocks for each of 8 KV heads, 498 MB: 88 us (5.7 TB/s, 83% of the measured copy bandwidth); 20 sequences of 250
// e4m3 blocks, 165 MB: 47 us, 320 CTAs on 152 SMs; one sequence of 128 blocks:
// 6.8 us, the chain of length, list, table, tiles and merge.
#include "pkv_attn_common.cuh"
#include "pkv_cluster.cuh"
#include "pkv_ops.h"

namespace pkv {

constexpr int kClusterMost = 16;  // partitions of a list that are one cluster, at most (beyond 8 by the device's leave)

// kFp8: e4m3 pools (H = 128).  Scales come per tile in both granularities (the producer fetches them with the
// block id): the K scale multiplies the tile's logits, the V scale its weights relative to the largest seen
// (VScaleRef, pkv_attn_common.cuh).
template <int H, bool kFp8, int W, bool kCluster>
__global__ void __launch_bounds__((W + kProducers) * 32, W > 4 ? 2 : PKV_CTAS_PER_SM)
attn_blocks_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const BlocksParams p)
{
    constexpr int P = kProducers, S = kFp8 ? kStagesFp8 : (W > 4 ? 2 * kStages : kStages), kThreads = (W + P) * 32;
    static_assert(S % W == 0, "a stage's tiles belong to one warp");
    constexpr int kBatch = S / P / 2;
    static_assert(S == 2 * P * kBatch, "a producer's stages are two batches");
    using L = AttnLayout<H, S, W, P, kFp8 ? 1 : 2>;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_u32 - raw_u32);

    const int kvh = blockIdx.x, b = blockIdx.y, part = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.G;
    const int begin = part * p.part_blocks;  // this CTA's entries of the list: [begin, end)
    const int32_t *sel = p.selected + ((size_t)b * p.K + kvh) * p.M + begin;
    const int pw = warp - W;  // producer warp

    const uint32_t bar_full = base_u32 + L::kBarOffset;
    const uint32_t bar_empty = bar_full + 8 * S;
    volatile int *valid_of = reinterpret_cast<volatile int *>(base + L::kMiscOffset);  // [S] tokens that count
    volatile int *abort_flag = valid_of + S;
    volatile int *issued_count = abort_flag + 1;  // [P]
    volatile float2 *stage_sc = reinterpret_cast<volatile float2 *>(base + L::kScaleOffset);
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        *abort_flag = 0;
        for (int q = 0; q < P; ++q) issued_count[q] = 0;
        init_ring<S>(bar_full, bar_empty);
    }
    pdl_wait_primary();  // launched early: nothing is read or written before the launch ahead is done
    pdl_launch_dependents();
    int first_sel = -1;  // the producers' first list entries do not depend on the length
    if (pw >= 0 && begin + pw + P * lane < min(p.M, begin + p.part_blocks)) first_sel = __ldg(sel + pw + P * lane);
    int ctx = p.context_lens[b];
    if (ctx < 0 || ctx > p.max_nb * kBlockSize) {
        if (threadIdx.x == 0 && kvh == 0 && part == 0) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        ctx = 0;
    }
    const int nb = (ctx + kBlockSize - 1) / kBlockSize;
    const int entries = min(nb, p.M);  // a sequence has no more blocks to list
    const int nparts = (entries + p.part_blocks - 1) / p.part_blocks;
    const int n = min(entries - begin, p.part_blocks);
    const size_t bn0 = (size_t)b * p.N + (size_t)kvh * G;
    if (n <= 0) {
        if (entries == 0 && part == 0) {
            for (int idx = threadIdx.x; idx < G * H; idx += kThreads) {
                const int g = idx / H, h = idx - g * H;
                p.out[(bn0 + g) * H + h] = __float2bfloat16_rn(0.f);
                if (h == 0 && p.lse_out) p.lse_out[bn0 + g] = -INFINITY;
            }
        }
        return;
    }

    __syncthreads();

    WarpAcc<H> acc;
    VScaleRef vr{0.f, 0.f};

    if (pw >= 0) {
        // ------------------------------ producer warps ------------------------------
        const int32_t *tbl = p.block_tables + (size_t)b * p.max_nb;
        const int mine = n > pw ? (n - pw + P - 1) / P : 0;
        // one tile per lane: its block id (-1: skipped), the tokens that count, its scales
        struct Tile {
            int bid, valid;
            float ks, vs;
        };
        auto look_up = [&](int j) {
            Tile t{-1, 0, 0.f, 0.f};
            if (j < 0 || j >= nb) {
                if (j != -1) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);  // -1: an entry left empty
                return t;
            }
            const int bid = __ldg(tbl + j);
            if (bid < 0 || bid >= p.num_blocks) {
                set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
                return t;
            }
            t.bid = bid;
            t.valid = min(kBlockSize, ctx - j * kBlockSize);
            if constexpr (kFp8) {
                const size_t si = (size_t)bid * p.scale_stride + kvh;
                t.ks = __ldg(p.k_scale + si);
                t.vs = __ldg(p.v_scale + si);
            }
            return t;
        };
        Tile cur{-1, 0, 0.f, 0.f};
        if (lane < mine) cur = look_up(first_sel);
        int issued = 0;
        bool aborted = false;
        for (int k0 = 0; k0 < mine && !aborted; k0 += 32) {
            Tile nxt{-1, 0, 0.f, 0.f};
            if (k0 + 32 + lane < mine) nxt = look_up(__ldg(sel + pw + P * (k0 + 32 + lane)));
            const int cnt = min(32, mine - k0);
            // kBatch tiles at a time, one per lane: half of this producer's stages, so that the other half stays in flight
            for (int k = 0; k < cnt; k += kBatch) {
                const int from = min(k + lane, 31);
                const int bid = __shfl_sync(0xFFFFFFFFu, cur.bid, from);
                const int valid = __shfl_sync(0xFFFFFFFFu, cur.valid, from);
                float2 sc = make_float2(0.f, 0.f);
                if constexpr (kFp8) sc = make_float2(__shfl_sync(0xFFFFFFFFu, cur.ks, from), __shfl_sync(0xFFFFFFFFu, cur.vs, from));
                bool ok = true;
                if (lane < kBatch && k + lane < cnt) {
                    const int i = pw + P * (k0 + k + lane), s = i % S;
                    const uint32_t bar = bar_full + 8 * s;
                    if (i >= S && !mbar_wait_bounded(bar_empty + 8 * s, ((i / S) & 1) ^ 1, abort_flag, p.wait_ns)) {
                        if (!*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
                        *abort_flag = 1;
                        ok = false;
                    } else {
                        valid_of[s] = valid;
                        if constexpr (kFp8) stage_sc[s].x = sc.x, stage_sc[s].y = sc.y;
                        if (PKV_TILE_WITHHELD(p, i)) {
                            // test builds: never loaded, never signalled
                        } else if (valid > 0) {
                            const uint32_t dst = base_u32 + s * L::kStageBytes;
                            mbar_arrive_expect_tx(bar, L::kStageBytes);
                            if constexpr (kFp8) {
                                tma_load_4d(dst, &tm_k, bar, 0, kvh, 0, bid);
                                tma_load_4d(dst + L::kTileBytes, &tm_v, bar, 0, kvh, 0, bid);
                            } else if (p.tok_major) {
                                tma_load_5d(dst, &tm_k, bar, 0, 0, kvh, 0, bid);
                                tma_load_5d(dst + L::kTileBytes, &tm_v, bar, 0, 0, kvh, 0, bid);
                            } else {
                                tma_load_5d(dst, &tm_k, bar, 0, 0, 0, kvh, bid);
                                tma_load_5d(dst + L::kTileBytes, &tm_v, bar, 0, 0, 0, kvh, bid);
                            }
                        } else {
                            mbar_arrive(bar);
                        }
                    }
                }
                if (__any_sync(0xFFFFFFFFu, !ok)) {
                    // A refused wait ends the producer.  Lanes before and behind it may have issued their tiles, so each of
                    // the producer's stages is waited for by a lane: for this batch's tile if it was issued, else for the
                    // tile that had the stage before.
                    if (lane < 2 * kBatch) {
                        const bool now = lane < kBatch && k + lane < cnt && ok;
                        const int last = k0 + k + lane - (now ? 0 : 2 * kBatch), i = pw + P * last;
                        if (last >= 0) mbar_wait_bounded(bar_full + 8 * (i % S), (i / S) & 1, nullptr, kDrainLimitNs);
                    }
                    __syncwarp();
                    issued = 0;  // nothing is left to drain
                    aborted = true;
                    break;
                }
                issued += min(kBatch, cnt - k);
            }
            cur = nxt;
        }
        if (lane == 0) issued_count[pw] = issued;
    } else {
        // ------------------------------ consumer warps ------------------------------
        uint32_t qf[H / 16][2];
        float2 back;
        if constexpr (kFp8) back = load_q_frags_fp8_scaled<H>(qf, p.q, p.N, b, kvh, G, lane);
        else load_q_frags<H>(qf, p.q, p.N, b, kvh, G, lane);
        acc_reset<H>(acc);
        for (int i = warp; i < n; i += W) {
            const int s = i % S;
            // lanes may differ at the deadline: the warp agrees before its collective work
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar_full + 8 * s, (i / S) & 1, abort_flag, p.wait_ns))) {
                if (!*abort_flag) set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
                *abort_flag = 1;
                break;
            }
            const int valid = valid_of[s];
            if (valid > 0) {
                const uint32_t kt = base_u32 + s * L::kStageBytes;
                if constexpr (kFp8)
                    tile_update_fp8<H, true, true>(acc, qf, kt, kt + L::kTileBytes, valid, p.scale_log2 * stage_sc[s].x, stage_sc[s].y, vr, lane, back);
                else
                    tile_update<H, true>(acc, qf, kt, kt + L::kTileBytes, valid, p.scale_log2, p.tok_major, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * s);
        }
    }

    __syncthreads();
    const bool aborted = *abort_flag != 0;
    if (aborted) {
        if (pw >= 0 && lane == 0) drain_ring<S, P>(bar_full, pw, issued_count[pw]);
        __syncthreads();
        if (nparts <= 1) return;  // the list's other partitions still count on this one: a void partial
    }

    // ------------------------- merge the consumer warps' states -------------------------
    float *mo = reinterpret_cast<float *>(base);
    float *mm = mo + W * 8 * H;
    float *ml = mm + W * 8;
    float *mine = ml + W * 8;  // kCluster: this partition's [G][H], lse [8]
    static_assert((W * 8 * (H + 2) + 8 * (H + 1)) * 4 <= L::kPipeBytes, "the drained ring holds the states and the partial");
    if (!aborted) {
        if (warp < W) {
            if constexpr (kFp8) acc_scale_o<H>(acc, vr.v);
            deposit<H, kFp8>(acc, mo, mm, ml, warp, lane);
        }
        __syncthreads();
    }
    for (int idx = threadIdx.x; idx < G * H; idx += kThreads) {
        const int g = idx / H, h = idx - g * H;
        float val = __int_as_float(0x7FC00000), lse = __int_as_float(0x7FC00000);  // NaN: void
        if (!aborted) combine<H, W>(mo, mm, ml, g, h, val, lse);
        const size_t bn = bn0 + g;
        if (kCluster && nparts > 1) {
            mine[idx] = val;
            if (h == 0) mine[8 * H + g] = lse;
        } else if (nparts > 1) {
            p.part_out[(bn * p.max_parts + part) * H + h] = val;
            if (h == 0) p.part_lse[bn * p.max_parts + part] = lse;
        } else {
            p.out[bn * H + h] = __float2bfloat16_rn(val);
            if (h == 0 && p.lse_out) p.lse_out[bn] = lse;
        }
    }
    if (nparts <= 1) return;
    if constexpr (kCluster) {
        // the list's partitions are one cluster: each reads all partials where they are and writes its part of the rows
        cluster_sync();
        const uint32_t at = smem_u32(mine);
        for (int idx = part * kThreads + threadIdx.x; idx < G * H; idx += nparts * kThreads) {
            const int g = idx / H;
            float lse[kClusterMost], v[kClusterMost], M = -INFINITY;
#pragma unroll
            for (int q = 0; q < kClusterMost; ++q) {
                if (q >= nparts) break;
                lse[q] = load_cluster<float>(at + (8 * H + g) * 4, q);
                v[q] = load_cluster<float>(at + idx * 4, q);
            }
            bool none = true;  // no keys at all
#pragma unroll
            for (int q = 0; q < kClusterMost; ++q) {
                if (q >= nparts) break;
                M = fmaxf(M, lse[q]);
                none &= lse[q] == -INFINITY;
            }
            float sum = 0.f, val = 0.f;
#pragma unroll
            for (int q = 0; q < kClusterMost; ++q) {
                if (q >= nparts) break;
                const float w = none ? 0.f : expf(lse[q] - M);  // (a void partial's NaN stays)
                sum += w;
                val += w * v[q];
            }
            p.out[bn0 * H + idx] = __float2bfloat16_rn(none ? 0.f : val / sum);
            if (idx == g * H && p.lse_out) p.lse_out[bn0 + g] = none ? -INFINITY : M + logf(sum);
        }
        cluster_sync();  // no partition leaves before all have been read
        return;
    }

    // ----------------- log-sum-exp merge by the unit's last partition -----------------
    __shared__ int last_one;
    __syncthreads();
    int32_t *count = p.counters + (size_t)b * p.K + kvh;
    if (threadIdx.x == 0) last_one = atomic_add_acq_rel_gpu(count, 1) == nparts - 1;
    __syncthreads();
    if (!last_one) return;
    float *wts = reinterpret_cast<float *>(base);                          // [G][nparts]
    float *red = reinterpret_cast<float *>(base) + kInKernelMergeWeights;  // [kMergeWarps][8][H]
    for (int idx = threadIdx.x; idx < G * nparts; idx += kThreads) {
        const int g = idx / nparts, q = idx - g * nparts;
        wts[idx] = __ldcg(p.part_lse + (bn0 + g) * p.max_parts + q);
    }
    __syncthreads();
    for (int g = warp; g < G; g += kThreads / 32) {
        const float lse = lse_merge_weights<true>(wts + g * nparts, nparts, wts + g * nparts, lane);
        if (lane == 0 && p.lse_out) p.lse_out[bn0 + g] = lse;
    }
    __syncthreads();
    merge_rows<H, 8>(wts, nparts, G, p.part_out + bn0 * p.max_parts * H, (size_t)p.max_parts * H, red, p.out + bn0 * H, H,
                     threadIdx.x, kThreads);
    if (threadIdx.x == 0) *count = 0;  // ready for the next call
}

template <int H, bool kFp8, int W, bool kCluster>
static cudaError_t launch_t(const CUtensorMap &tk, const CUtensorMap &tv, const BlocksParams &p, cudaStream_t stream)
{
    constexpr int S = kFp8 ? kStagesFp8 : (W > 4 ? 2 * kStages : kStages);
    constexpr int smem = AttnLayout<H, S, W, kProducers, kFp8 ? 1 : 2>::kAlloc;
    static int ready[64] = {};  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(attn_blocks_kernel<H, kFp8, W, kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (kCluster) e = allow_wide_clusters(attn_blocks_kernel<H, kFp8, W, kCluster>);
        if (e != cudaSuccess) return e;
        ready[dev] = 1;
    }
    return launch_clusters(attn_blocks_kernel<H, kFp8, W, kCluster>, dim3(p.K, p.B, p.max_parts), dim3((W + kProducers) * 32),
                           dim3(1, 1, kCluster ? p.max_parts : 1), smem, stream, tk, tv, p);
}

cudaError_t launch_attn_blocks(int H, bool fp8, const CUtensorMap &tk, const CUtensorMap &tv, const BlocksParams &p, int sms,
                               cudaStream_t stream)
{
    // Eight consumer warps and sixteen stages instead of four (and eight in bf16) where one CTA takes a whole list.  Tiles of
    // 4 KB (e4m3, H = 64) leave room for two such CTAs per SM, or three of four warps: four only where all lists then run at
    // once and otherwise would not (64 * 8 e4m3 lists of 128 blocks 74.1 -> 58.4 us, bf16 H = 64 63.4 -> 50.5; but 46 * 8 lists
    // 49.1 with eight, 46.1 with four, and 44.5 and 36.1).  Tiles of 8 KB leave room for one: while there is one list per SM
    // at most (16 * 8 lists of 128: 31.2 -> 25.6; 64 * 8 lists: 99.7 and 98.0).  CTAs of a cut list are short and many: four
    // warps (2 * 160 e4m3 parts of 125 blocks 46.1, with eight 51.9).
    const int64_t lists = (int64_t)p.B * p.K;
    const bool wide = p.max_parts == 1 && (fp8 || H == 64 ? lists <= 2 * sms || lists > 3 * sms : lists <= sms);
    // A list's partitions as one cluster, which joins their partials in shared memory, where they all run at once (8 lists of
    // 128 in 11-block partitions 6.7 us, through the workspace 8.4; 64 lists of 250 in 42-block ones 26.5 and 28.7) or are two
    // (512 lists of 128 94.3 and 96.8); larger clusters start late in a grid of several waves (512 lists in 16-block ones 122, not
    // as clusters 106).  A cluster's CTAs share a group of SMs, so not all of three CTAs per SM are to be had: of 456, 435 to 456
    // in clusters of up to 6, 396 to 432 in ones of up to 12, 336 to 390 in ones of up to 16.
    const int fit = p.max_parts <= 6 ? 95 : (p.max_parts <= 12 ? 86 : 73);  // per cent
    const bool cluster = p.max_parts > 1 && p.max_parts <= kClusterMost &&
                         (p.max_parts == 2 || lists * p.max_parts * 100 <= (int64_t)PKV_CTAS_PER_SM * sms * fit);
    if (cluster) {
        if (fp8) return launch_t<128, true, 4, true>(tk, tv, p, stream);
        return H == 128 ? launch_t<128, false, 4, true>(tk, tv, p, stream) : launch_t<64, false, 4, true>(tk, tv, p, stream);
    }
    if (fp8) return wide ? launch_t<128, true, 8, false>(tk, tv, p, stream) : launch_t<128, true, 4, false>(tk, tv, p, stream);
    if (H == 128) return wide ? launch_t<128, false, 8, false>(tk, tv, p, stream) : launch_t<128, false, 4, false>(tk, tv, p, stream);
    return wide ? launch_t<64, false, 8, false>(tk, tv, p, stream) : launch_t<64, false, 4, false>(tk, tv, p, stream);
}

}  // namespace pkv
