// pkv_latent_append.cu - new tokens' rows into a latent cache: the latent vector normed, the shared rotary key turned
// by its position's angles, and the rotary parts of the tokens' queries turned into the rows that attention takes.
//     c' = c w / sqrt(mean(c^2) + eps)  (512 elements; without w the latents are copied),
//     (a, b)' = (a cos - b sin, a sin + b cos)  for the 32 pairs of the key and of each head's query.
//
// The angle is the fraction of a turn position * inv_freq / 2 pi in 64-bit integers, as in pkv_rope.cu: off by 1e-10 of a
// turn at position 10^6.  Sums of squares, norms and rotations in fp32, one rounding to bf16 at the end.
//
// Bound by memory: a token reads and writes 1,152 + 128 N bytes.  From a cold L2 8,192 tokens of 16 heads take 11.8 us, 5,001 of
// 40 heads 12.8 (4.9 TB/s, launch and a first wave's loads included; with CTAs of eight warps and fewer of them at once 14.8 and
// 13.7), 64 of 128 heads 3.1, a launch and the chain of length, table and position.  One warp takes a token's row and up to 32 of its heads
// (the key counts as one), so that lane j computes pair j's angle once for all of them and nothing waits for other
// warps: loads (all of them before the slot, the position and the angles are known), two shuffles a pair of elements,
// stores.  A head is four lanes' work of two 16-byte vectors, half a head apart.
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_latent.h"

namespace pkv {

constexpr int kLatAppendWarps = 4;                           // seven CTAs an SM: 72 registers
constexpr int kLatAppendHeads = 32;                          // heads of a warp's job, the key among them
constexpr int kLatAppendRounds = kLatAppendHeads * 4 / 32;   // of 32 lanes
constexpr int kLatRow = kLatentDim + kLatentRope;
constexpr double kLatInv2Pi = 0.15915494309189533577;

__device__ __forceinline__ void latent_unpack(const uint4 v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16x2_lo(w[i]), x[2 * i + 1] = bf16x2_hi(w[i]);
}
__device__ __forceinline__ uint4 latent_pack(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

template <bool kInter>
__global__ void __launch_bounds__(kLatAppendWarps * 32, 7) latent_append_kernel(const LatentAppendParams p, int parts, int per)
{
    __shared__ float2 angles[kLatAppendWarps][kLatentRope / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t job = (int64_t)blockIdx.x * kLatAppendWarps + warp;
    const int i = (int)(job / parts), part = (int)(job - (int64_t)i * parts);
    if (i >= p.n) return;
    // heads [h0, h1) of 0 (the key) .. N
    const int h0 = part * per, h1 = min(p.N + 1, h0 + per), items = (h1 - h0) * 4;
    const uint16_t *row = p.kv_new + (int64_t)i * kLatRow;
    const uint16_t *queries = p.q_rope + (int64_t)i * p.q_rope_token;

    uint4 a[kLatAppendRounds], b[kLatAppendRounds], c[2], w[2];
#pragma unroll
    for (int r = 0; r < kLatAppendRounds; ++r) {
        const int x = lane + 32 * r;
        if (x < items) {
            const int head = h0 + x / 4;
            const uint16_t *src = (head == 0 ? row + kLatentDim : queries + (int64_t)(head - 1) * p.q_rope_head) + 8 * (x & 3);
            a[r] = *reinterpret_cast<const uint4 *>(src);
            b[r] = *reinterpret_cast<const uint4 *>(src + kLatentRope / 2);
        }
    }
    if (part == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            c[k] = *reinterpret_cast<const uint4 *>(row + 8 * (lane + 32 * k));
            if (p.norm_weight) w[k] = __ldg(reinterpret_cast<const uint4 *>(p.norm_weight + 8 * (lane + 32 * k)));
        }
    }
    const double t = __ldg(p.inv_freq + lane) * kLatInv2Pi;

    // slot and position
    int64_t slot = -1;
    int pos = 0;
    if (!p.block_tables) {
        slot = p.slots[i];
        pos = p.positions[i];
        if (slot >= (int64_t)p.num_blocks * kBlockSize) {
            if (part == 0 && lane == 0) set_flag(p.err_flag, PKV_FLAG_SLOT_RANGE);
            slot = -1;
        }
    } else {
        const int seq = i / p.T, k = i - seq * p.T, ctx = p.context_lens[seq];
        const bool report = part == 0 && lane == 0;
        if (ctx < 0 || ctx > p.max_nb * kBlockSize) {
            if (report) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        } else if (k >= p.T - ctx) {
            pos = ctx - p.T + k;
            const int blk = p.block_tables[(size_t)seq * p.max_nb + pos / kBlockSize];
            if (blk >= 0 && blk < p.num_blocks) slot = (int64_t)blk * kBlockSize + pos % kBlockSize;
            else if (report) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
        }
        if (report) p.slots_out[i] = slot;
    }
    if (slot < 0) return;

    {
        const unsigned long long freq = __double2ull_rn((t - floor(t)) * 18446744073709551616.0);  // turns in units of 2^-64
        const unsigned turns = (unsigned)((freq * (unsigned long long)(long long)pos) >> 32);
        float s, co;
        sincospif((float)(int)turns * 0x1p-31f, &s, &co);
        angles[warp][lane] = make_float2(co, s);
    }
    __syncwarp();

    uint16_t *to = p.cache + slot * kLatRow;
    if (part == 0) {
        if (p.norm_weight) {
            float x[2][8], ss = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                latent_unpack(c[k], x[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += x[k][e] * x[k][e];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            const float by = 1.f / sqrtf(ss * (1.f / kLatentDim) + p.eps);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float y[8];
                latent_unpack(w[k], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= x[k][e] * by;
                c[k] = latent_pack(y);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) *reinterpret_cast<uint4 *>(to + 8 * (lane + 32 * k)) = c[k];
    }
    uint16_t *q = p.q + (int64_t)i * p.N * kLatRow + kLatentDim;
#pragma unroll
    for (int r = 0; r < kLatAppendRounds; ++r) {
        const int x = lane + 32 * r;
        if (x >= items) break;
        const int head = h0 + x / 4, v = x & 3;
        float f[8], g[8];
        latent_unpack(a[r], f);
        latent_unpack(b[r], g);
        if constexpr (kInter) {
            // vector v holds pairs 4 v .., vector v + 4 pairs 16 + 4 v ..
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 s0 = angles[warp][4 * v + e], s1 = angles[warp][16 + 4 * v + e];
                const float f0 = f[2 * e], f1 = f[2 * e + 1], g0 = g[2 * e], g1 = g[2 * e + 1];
                f[2 * e] = f0 * s0.x - f1 * s0.y, f[2 * e + 1] = f0 * s0.y + f1 * s0.x;
                g[2 * e] = g0 * s1.x - g1 * s1.y, g[2 * e + 1] = g0 * s1.y + g1 * s1.x;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 s = angles[warp][8 * v + e];
                const float f0 = f[e], g0 = g[e];
                f[e] = f0 * s.x - g0 * s.y, g[e] = f0 * s.y + g0 * s.x;
            }
        }
        uint16_t *dst = (head == 0 ? to + kLatentDim : q + (int64_t)(head - 1) * kLatRow) + 8 * v;
        *reinterpret_cast<uint4 *>(dst) = latent_pack(f);
        *reinterpret_cast<uint4 *>(dst + kLatentRope / 2) = latent_pack(g);
    }
}

cudaError_t launch_latent_append(const LatentAppendParams &p, bool interleaved, cudaStream_t stream)
{
    // where there are few, half as many a warp: 64 tokens of 128 heads 3.2 -> 3.1 us (250 of 128 3.9 -> 4.4)
    const int heads = (int64_t)p.n * (p.N + 1) <= 16384 ? kLatAppendHeads / 2 : kLatAppendHeads;
    const int parts = (p.N + heads) / heads, per = (p.N + parts) / parts;
    const int64_t jobs = (int64_t)p.n * parts;
    const unsigned grid = (unsigned)((jobs + kLatAppendWarps - 1) / kLatAppendWarps);
    return launch_kernel(interleaved ? latent_append_kernel<true> : latent_append_kernel<false>, dim3(grid),
                         dim3(kLatAppendWarps * 32), 0, stream, true, p, parts, per);
}

}  // namespace pkv
