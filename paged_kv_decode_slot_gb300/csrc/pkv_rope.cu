// pkv_rope.cu - rotary position embedding of a step's queries and keys with the append of its keys
// and values into the paged pools, in one pass.
//
// Token i at position P turns element pair (a, b) of a head by the angle P * inv_freq[j]:
//     a' = a cos - b sin,   b' = a sin + b cos,   j < R / 2,
// pair j being elements (j, j + R/2) or, interleaved, (2j, 2j + 1); elements from R on are copied.
// q goes to q_out, k into its slot of the K pool, v unturned into its slot of the V pool: what the
// separate rotation would write and the append read back never leaves the chip.
//
// The angle.  P * inv_freq in 32 bits is off by whole radians for far positions, so turns =
// P * inv_freq / (2 pi) and its distance to the nearest integer are taken in 64 bits (absolute error
// below 2^-52 of the turns: 1e-7 of a turn at position 2^31), and only that distance is rounded to
// 32 bits for sincospif.  The R / 2 angles of a token are computed once and shared by its N + K heads.
//
// Bound by memory: a token moves (N + 2K) * H elements each way and computes 6 operations a pair.
// One CTA per token: a thread's loads (two 16-byte vectors an item, up to kItems items) are issued
// before the token's position, slot and angles are there, and need none of them.  A token whose slot
// is negative is left out: nothing of its rows is written.
#include "pkv_device.cuh"
#include "pkv_ops.h"

namespace pkv {

constexpr int kRopeThreads = 192;
constexpr int kRopeItems = 2;  // items a thread holds at a time
constexpr double kInv2Pi = 0.15915494309189533577;

__device__ __forceinline__ uint2 rope_quantize8(const float (&x)[8], float sc)
{
    // e4m3(x / scale), the division rounded to nearest, as the plain append quantizes; x is the
    // rotation's 32-bit result, so a rotated key is rounded once
    auto q2 = [&](int i) -> uint32_t { return f32x2_to_e4m3x2(__fdiv_rn(x[i], sc), __fdiv_rn(x[i + 1], sc)); };
    return make_uint2(q2(0) | (q2(2) << 16), q2(4) | (q2(6) << 16));
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8])
{
    x[0] = bf16x2_lo(v.x), x[1] = bf16x2_hi(v.x), x[2] = bf16x2_lo(v.y), x[3] = bf16x2_hi(v.y);
    x[4] = bf16x2_lo(v.z), x[5] = bf16x2_hi(v.z), x[6] = bf16x2_lo(v.w), x[7] = bf16x2_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Slot and position of token i; false: nothing is written for it.
__device__ __forceinline__ bool rope_slot(const RopeParams &p, int64_t i, bool report, int64_t &slot, int &pos)
{
    if (!p.block_tables) {
        slot = p.slots[i];
        pos = p.positions[i];
        if (slot >= (int64_t)p.num_blocks * kBlockSize) {
            if (report) set_flag(p.err_flag, PKV_FLAG_SLOT_RANGE);
            return false;
        }
        return slot >= 0;
    }
    const int b = (int)(i / p.T), t = (int)(i - (int64_t)b * p.T);
    const int ctx = p.context_lens[b];
    slot = -1;
    pos = ctx - p.T + t;
    if (ctx > p.max_nb * kBlockSize) {
        if (report) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        pos = 0;
    } else if (ctx > 0 && pos >= 0) {
        const int blk = p.block_tables[(size_t)b * p.max_nb + pos / kBlockSize];
        if (blk < 0 || blk >= p.num_blocks) {
            if (report) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
        } else {
            slot = (int64_t)blk * kBlockSize + pos % kBlockSize;
        }
    }
    if (report) p.slots_out[i] = slot;
    return slot >= 0;
}

template <bool kInter, bool kFp8>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p)
{
    extern __shared__ float2 cs[];  // [R / 2] (cos, sin)
    const int64_t i = blockIdx.x;
    const int per_head = p.H / 16, nq = p.N * per_head, nk = p.K * per_head;
    const int items = nq + 2 * nk;
    const int rot = p.R / 16;  // rotated items of a head; the others copy 16 neighbouring elements

    // The two vectors of item x: rows of q, then k_new, then v_new.
    auto offsets = [&](int x, int &o0, int &o1, bool &turned) {
        const int c = x % per_head, head = x / per_head;
        turned = x < nq + nk && c < rot;
        o0 = head * p.H + (turned && !kInter ? 8 * c : 16 * c);
        o1 = turned && !kInter ? o0 + p.R / 2 : o0 + 8;
    };
    auto source = [&](int x) {
        return x < nq ? p.q + i * p.N * p.H
                      : (x < nq + nk ? p.k_new + i * p.K * p.H - (int64_t)p.N * p.H
                                     : p.v_new + i * p.K * p.H - (int64_t)(p.N + p.K) * p.H);
    };
    uint4 a[kRopeItems], b[kRopeItems];
    auto load = [&](int x0) {
#pragma unroll
        for (int u = 0; u < kRopeItems; ++u) {
            const int x = x0 + u * kRopeThreads;
            if (x < items) {
                int o0, o1;
                bool turned;
                offsets(x, o0, o1, turned);
                const uint16_t *src = source(x);
                a[u] = *reinterpret_cast<const uint4 *>(src + o0);
                b[u] = *reinterpret_cast<const uint4 *>(src + o1);
            }
        }
    };
    load(threadIdx.x);

    int64_t slot;
    int pos;
    if (!rope_slot(p, i, threadIdx.x == 0, slot, pos)) return;
    for (int j = threadIdx.x; j < p.R / 2; j += kRopeThreads) {
        const double turns = (double)pos * p.inv_freq[j] * kInv2Pi;
        const float f = (float)(turns - rint(turns));
        float s, c;
        sincospif(2.f * f, &s, &c);
        cs[j] = make_float2(c, s);
    }
    __syncthreads();

    for (int x0 = threadIdx.x; x0 < items; x0 += kRopeItems * kRopeThreads) {
        if (x0 != (int)threadIdx.x) load(x0);
#pragma unroll
        for (int u = 0; u < kRopeItems; ++u) {
            const int x = x0 + u * kRopeThreads;
            if (x >= items) break;
            int o0, o1;
            bool turned;
            offsets(x, o0, o1, turned);
            float y0[8], y1[8];
            unpack8(a[u], y0);
            unpack8(b[u], y1);
            if (turned) {
                const float2 *w = cs + 8 * (x % per_head);
                if (kInter) {  // pairs (2e, 2e + 1): the first four in y0, the others in y1
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 w0 = w[e], w1 = w[e + 4];
                        const float p0 = y0[2 * e], p1 = y0[2 * e + 1], r0 = y1[2 * e], r1 = y1[2 * e + 1];
                        y0[2 * e] = p0 * w0.x - p1 * w0.y;
                        y0[2 * e + 1] = p0 * w0.y + p1 * w0.x;
                        y1[2 * e] = r0 * w1.x - r1 * w1.y;
                        y1[2 * e + 1] = r0 * w1.y + r1 * w1.x;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 w0 = w[e];
                        const float p0 = y0[e], p1 = y1[e];
                        y0[e] = p0 * w0.x - p1 * w0.y;
                        y1[e] = p0 * w0.y + p1 * w0.x;
                    }
                }
            }
            if (x < nq) {
                uint16_t *dst = p.q_out + i * p.N * p.H;
                *reinterpret_cast<uint4 *>(dst + o0) = turned ? pack8(y0) : a[u];
                *reinterpret_cast<uint4 *>(dst + o1) = turned ? pack8(y1) : b[u];
                continue;
            }
            const bool is_v = x >= nq + nk;
            const int64_t row = slot * p.K * p.H - (int64_t)(is_v ? p.N + p.K : p.N) * p.H;
            void *pool = is_v ? p.v_cache : p.k_cache;
            if (kFp8) {
                const int kvh = x / per_head - (is_v ? p.N + p.K : p.N);
                const float sc = (is_v ? p.v_scale : p.k_scale)[(slot / kBlockSize) * p.scale_stride + kvh];
                uint8_t *dst = static_cast<uint8_t *>(pool) + row;
                *reinterpret_cast<uint2 *>(dst + o0) = rope_quantize8(y0, sc);
                *reinterpret_cast<uint2 *>(dst + o1) = rope_quantize8(y1, sc);
            } else {
                uint16_t *dst = static_cast<uint16_t *>(pool) + row;
                *reinterpret_cast<uint4 *>(dst + o0) = turned ? pack8(y0) : a[u];
                *reinterpret_cast<uint4 *>(dst + o1) = turned ? pack8(y1) : b[u];
            }
        }
    }
}

cudaError_t launch_rope_append(const RopeParams &p, bool interleaved, bool fp8, cudaStream_t stream)
{
    const size_t smem = sizeof(float2) * (size_t)(p.R / 2);
    const unsigned grid = (unsigned)p.n;
    if (interleaved) {
        if (fp8) rope_append_kernel<true, true><<<grid, kRopeThreads, smem, stream>>>(p);
        else rope_append_kernel<true, false><<<grid, kRopeThreads, smem, stream>>>(p);
    } else {
        if (fp8) rope_append_kernel<false, true><<<grid, kRopeThreads, smem, stream>>>(p);
        else rope_append_kernel<false, false><<<grid, kRopeThreads, smem, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace pkv
