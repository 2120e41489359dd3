// pkv_rope.cu - rotary position embedding of a step's queries and keys with the append of its keys
// and values into the paged pools, in one pass.
//
// Token i at position P turns element pair (a, b) of a head by the angle P * inv_freq[j]:
//     a' = a cos - b sin,   b' = a sin + b cos,   j < R / 2,
// pair j being elements (j, j + R/2) or, interleaved, (2j, 2j + 1); elements from R on are copied.
// q goes to q_out, k into its slot of the K pool, v unturned into its slot of the V pool: what a
// separate rotation would write and an append read back never leaves the chip.
//
// The angle.  P * inv_freq in 32 bits is off by whole radians for far positions.  Only the fraction of
// a turn counts, so each frequency is taken once, in 64 bits, as a fraction of a turn per position in
// units of 2^-64; the product with the position then wraps around a turn by itself, in integers.  The
// fraction is off by 2^-54 turns (inv_freq's and 1/2pi's roundings) and the angle by P times that:
// 10^-10 of a turn at position 10^6, 10^-7 at 2^31.  Its upper 32 bits go to sincospif.
//
// Bound by memory: a token moves (N + 2K) H elements each way and computes 6 operations a pair.  The work is cut into
// units of kUnitHeads heads of one token (q's, then k's, then v's); a CTA takes every gridDim-th unit and streams
// the units' rows through a ring in shared memory with bulk copies, so that the loads under way need no
// registers and the arithmetic (the e4m3 form's quotients above all) has enough warps; results go straight to global
// memory.  A token whose slot is negative is left out: nothing of its rows is written.
//
// Measured: 8,192 tokens of 32 query and 8 KV heads of 128 in bf16, 201 MB, 33.6 us (6.0 TB/s, 88% of the measured
// copy bandwidth); 5,001 tokens of 40 and 40 into e4m3, interleaved, 256 MB, 50.7 us (5.0 TB/s, 74%): neither DRAM (50%
// in a cold run) nor the issue slots (67%) are full, warps wait most for the CTA's barrier at the end of each unit (the check
// of the quotients takes 7 us; 28 of 32 lanes are busy, and an order of the items that put turned and copied ones into
// warps of their own cost 3 us).  64 decode tokens: 2.8 us, a launch and four dependent loads.  A unit holds heads of one
// token only, so few heads leave most threads and most of a stage empty: 8,192 tokens of 4 and 1 heads, 25 MB, 17.6 us
// (21% of the copy bandwidth), of 8 and 2 21.4.
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_ops.h"

namespace pkv {

// Threads, heads of a unit, stages and CTAs per SM, measured on 8,192 tokens of 32 + 2 * 8 heads (bf16) and 5,001 of
// 40 + 2 * 40 (e4m3) with an earlier form of the arithmetic: 256 / 64 / 2 / 4 34.8 and 55.0 us; 192 / 48 / 3 / 5 34.6 and
// 60.1 (three units a token instead of two); 192 / 48 / 2 / 6 36.1 and 68.6; 128 / 32 / 3 / 8 46.2 and 64.2; 384 / 96 / 2 / 3
// 42.8 and 83.4.  (48 and 120 heads are what they were chosen on.)
constexpr int kRopeThreads = 256;
constexpr int kUnitHeads = 64;
constexpr int kRopeStages = 2;
constexpr int kRopeCtasPerSm = 4;
constexpr double kInv2Pi = 0.15915494309189533577;

// Two fp32 operations at a time (add, mul and fma on f32x2, sm_100 and later): with the
// quotients checked from both sides, they took the e4m3 form from 57.8 us to 53.9.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi)
{
    f32x2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ float2 halves(f32x2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

__device__ __forceinline__ uint32_t codes(f32x2 v)
{
    const float2 r = halves(v);
    return f32x2_to_e4m3x2(r.x, r.y);
}

// A scale's reciprocal, made smaller and made larger by 2^-21.
struct Reciprocal {
    f32x2 down, up;
    float scale;
    bool plain;  // the scale is in [2^-100, 2^100]
};

__device__ __forceinline__ Reciprocal reciprocal(float scale)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));  // off by 2^-23 at most
    const float r0 = r * (1.f - 0x1p-21f), r1 = r * (1.f + 0x1p-21f);
    return Reciprocal{pair(r0, r0), pair(r1, r1), scale, scale >= 0x1p-100f && scale <= 0x1p100f};
}

// Two times eight values as e4m3 codes of x / scale, the quotient rounded to nearest in fp32 as the plain append takes it (the
// input is the rotation's 32-bit result, so a turned key is rounded once to 8 bits).  x times a reciprocal made smaller,
// and made larger, by 2^-21 lie to both sides of that quotient (five units of 2^-24 between them: two for the reciprocal, one
// for each product and for the quotient's rounding): where their codes agree, they are the quotient's too (rounding is
// monotonic; zeros, infinities and NaN agree with themselves); only where they differ is x divided.  The reciprocal of a
// scale outside [2^-100, 2^100] may over- or underflow: there every x is divided.  (Correcting one product by its remainder,
// Markstein's way, measured 57.8 us against 53.9 on 5,001 tokens of 3 * 40 heads.)
__device__ __forceinline__ void rope_quantize(const f32x2 (&x)[4], const f32x2 (&y)[4], const Reciprocal &by, uint2 &cx, uint2 &cy)
{
    uint32_t c[8], differ = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const f32x2 v = i < 4 ? x[i % 4] : y[i % 4];
        c[i] = codes(mul2(v, by.down));
        differ |= c[i] ^ codes(mul2(v, by.up));
    }
    if (differ || !by.plain) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = halves(i < 4 ? x[i % 4] : y[i % 4]);
            c[i] = f32x2_to_e4m3x2(__fdiv_rn(v.x, by.scale), __fdiv_rn(v.y, by.scale));
        }
    }
    cx = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    cy = make_uint2(c[4] | (c[5] << 16), c[6] | (c[7] << 16));
}

// A vector's words, unpacked: neighbouring elements of a word as one pair, or (kSplit) the lower elements of two
// words as one pair and the upper ones as another, which is what interleaved pairs want.
template <bool kSplit>
__device__ __forceinline__ void unpack8(const uint4 v, f32x2 (&x)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kSplit) {
            const uint32_t a = w[i & 2], b = w[(i & 2) + 1];
            x[i] = i & 1 ? pair(bf16x2_hi(a), bf16x2_hi(b)) : pair(bf16x2_lo(a), bf16x2_lo(b));
        } else {
            x[i] = pair(bf16x2_lo(w[i]), bf16x2_hi(w[i]));
        }
    }
}

// From the split order back to neighbouring elements.
__device__ __forceinline__ void join8(f32x2 (&x)[4])
{
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 a = halves(x[i]), b = halves(x[i + 1]);
        x[i] = pair(a.x, b.x);
        x[i + 1] = pair(a.y, b.y);
    }
}

__device__ __forceinline__ uint4 pack8(const f32x2 (&x)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = halves(x[i]);
        w[i] = pack_bf16x2(v.x, v.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Slot and position of token i (slot < 0: nothing is written for it).
__device__ __forceinline__ void rope_slot(const RopeParams &p, int i, bool report, int64_t &slot, int &pos)
{
    if (!p.block_tables) {
        slot = p.slots[i];
        pos = p.positions[i];
        if (slot >= (int64_t)p.num_blocks * kBlockSize) {
            if (report) set_flag(p.err_flag, PKV_FLAG_SLOT_RANGE);
            slot = -1;
        }
        return;
    }
    const int b = i / p.T, t = i - b * p.T;
    const int ctx = p.context_lens[b];
    slot = -1;
    pos = 0;
    if (ctx > p.max_nb * kBlockSize) {
        if (report) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
    } else if (ctx > 0 && t >= p.T - ctx) {
        pos = ctx - p.T + t;
        const int blk = p.block_tables[(size_t)b * p.max_nb + pos / kBlockSize];
        if (blk >= 0 && blk < p.num_blocks) slot = (int64_t)blk * kBlockSize + pos % kBlockSize;
        else if (report) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
    }
    if (report) p.slots_out[i] = slot;
}

// 1-D bulk copy global -> this CTA's shared memory, counted on the mbarrier (16-byte addresses and size).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int H, bool kInter, bool kFp8>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtasPerSm) rope_append_kernel(const RopeParams p)
{
    constexpr int S = kRopeStages, kPerHead = H / 16;  // items (two 16-byte vectors) of a head
    constexpr int kStageBytes = kUnitHeads * H * 2;
    extern __shared__ __align__(128) uint8_t ring[];  // [S][kUnitHeads][H] bf16
    // Cosines and sines of this unit's token and of the next one's: vector (e / 2) * kGroups + g holds (cos, cos, sin, sin) of
    // pairs e, e + 1 of group g, so that neighbouring threads, who turn neighbouring groups, read neighbouring vectors.
    // A group is what one thread reads in a row: 8 pairs, interleaved 4.
    constexpr int kPairs = kInter ? 4 : 8, kGroups = H / 2 / kPairs;
    __shared__ float4 cs[2][H / 4];
    __shared__ int64_t slot_of[4];                    // of this unit and the two after it
    __shared__ int pos_of[4];
    __shared__ __align__(8) uint64_t full[S];
    __shared__ int aborted;
    const int tid = threadIdx.x;
    const int heads = p.N + 2 * p.K;
    const int rot = p.R / 16;  // turned items of a head; the others copy 16 neighbouring elements
    // Units are (token, chunk of heads) pairs; from one to the next of this CTA's, gridDim.x units on, without a division.
    const int chunks = (heads + kUnitHeads - 1) / kUnitHeads, per = (heads + chunks - 1) / chunks;
    const int step_i = gridDim.x / chunks, step_c = gridDim.x - step_i * chunks;
    struct Unit {
        int i, chunk;
    };
    auto advance = [&](Unit &t) {
        t.i += step_i;
        t.chunk += step_c;
        if (t.chunk >= chunks) t.chunk -= chunks, ++t.i;
    };

    // Rows of a unit: up to three runs of heads, of q, k_new and v_new.
    auto load = [&](const Unit &t, int stage) {
        const int h0 = t.chunk * per, h1 = min(heads, h0 + per);
        const uint32_t bar = smem_u32(full + stage), dst = smem_u32(ring) + stage * kStageBytes;
        mbar_arrive_expect_tx(bar, (uint32_t)(h1 - h0) * H * 2);
        auto part = [&](const uint16_t *src, int from, int to) {  // heads [from, to) of all, src at head `from`
            const int a = max(from, h0), b = min(to, h1);
            if (a < b) bulk_load(dst + (a - h0) * H * 2, src + (int64_t)(a - from) * H, (uint32_t)(b - a) * H * 2, bar);
        };
        part(p.q + (int64_t)t.i * p.N * H, 0, p.N);
        part(p.k_new + (int64_t)t.i * p.K * H, p.N, p.N + p.K);
        part(p.v_new + (int64_t)t.i * p.K * H, p.N + p.K, heads);
    };
    const int first = blockIdx.x / chunks;
    Unit now{first, (int)blockIdx.x - first * chunks}, ahead = now;  // ahead: the next unit to load
    int copied = 0;  // units whose loads were issued (thread 0)
    if (tid == 0) {
        aborted = 0;
        for (int s = 0; s < S; ++s) mbar_init(smem_u32(full + s), 1);
        fence_barrier_init();
    }
    pdl_wait_primary();
    pdl_launch_dependents();
    if (tid == 0) {
        for (; copied < S && ahead.i < p.n; ++copied, advance(ahead)) load(ahead, copied);
    }
    unsigned long long freq = 0;  // turns per position in units of 2^-64, of pair tid
    if (tid < p.R / 2) {
        const double t = p.inv_freq[tid] * kInv2Pi;
        freq = __double2ull_rn((t - floor(t)) * 18446744073709551616.0);  // 1.0 saturates: 2^-64 of a turn off
    }
    // Slots and positions are loaded three units ahead by one thread and handed on two units ahead, the angles are
    // computed one ahead, so that a unit's vectors wait for neither.
    Unit asked = now;
    int64_t slot = -1;
    int pos = 0;
    auto ask = [&]() {
        slot = -1;
        if (asked.i < p.n) rope_slot(p, asked.i, asked.chunk == 0, slot, pos);
        advance(asked);
    };
    auto tell = [&](int k) { slot_of[k & 3] = slot, pos_of[k & 3] = pos; };
    if (tid == 0) {
        ask(), tell(0), ask(), tell(1), ask();
    }
    __syncthreads();  // the barriers exist, the first two slots are there
    auto turn = [&](int k) {
        if (tid < p.R / 2) {
            const unsigned turns = (unsigned)((freq * (unsigned long long)(long long)pos_of[k & 3]) >> 32);
            float s, c;
            sincospif((float)(int)turns * 0x1p-31f, &s, &c);  // the nearer way round: within half a turn
            const int g = tid / kPairs, e = tid % kPairs;
            float *to = reinterpret_cast<float *>(cs[k & 1]) + 4 * ((e / 2) * kGroups + g) + (e & 1);
            to[0] = c;
            to[2] = s;
        }
    };
    // e4m3: the scales of this thread's items of a unit, loaded one unit ahead
    constexpr int kRounds = kFp8 ? (kUnitHeads * kPerHead + kRopeThreads - 1) / kRopeThreads : 1;
    float sc[kRounds], sc_next[kRounds];
    auto scales = [&](const Unit &t, int64_t slot, float (&to)[kRounds]) {
        if constexpr (kFp8) {
            if (t.i >= p.n || slot < 0) return;
#pragma unroll
            for (int r = 0; r < kRounds; ++r) {
                const int kvh = t.chunk * per + (tid + r * kRopeThreads) / kPerHead - p.N;
                if (kvh >= 0 && kvh < 2 * p.K)
                    to[r] = __ldg((kvh < p.K ? p.k_scale + kvh : p.v_scale + kvh - p.K) + (int64_t)((uint64_t)slot / kBlockSize) * p.scale_stride);
            }
        }
    };
    Unit next = now;
    advance(next);
    scales(now, slot_of[0], sc);
    turn(0);
    __syncthreads();  // the first angles are there

    for (int k = 0;; ++k) {
        if (tid == 0) tell(k + 2), ask();
        scales(next, slot_of[(k + 1) & 3], sc_next);
        turn(k + 1);
        const int64_t at_slot = slot_of[k & 3];
        const int h0 = now.chunk * per, items = (min(heads, h0 + per) - h0) * kPerHead;
        const int stage = k % S;
        const bool there = mbar_wait_bounded(smem_u32(full + stage), (uint32_t)(k / S) & 1, nullptr, p.wait_ns);
        if (!there) aborted = 1;
        if (there && at_slot >= 0) {
            const uint8_t *src = ring + stage * kStageBytes;
            const float4 *angles = cs[k & 1];
            uint16_t *q_row = p.q_out + (int64_t)now.i * p.N * H;
            const int64_t row_off = at_slot * p.K * H;
#pragma unroll
            for (int r = 0; r < (kUnitHeads * kPerHead + kRopeThreads - 1) / kRopeThreads; ++r) {
                const int x = tid + r * kRopeThreads;
                if (x >= items) break;
                const int c = x % kPerHead, head = h0 + x / kPerHead;
                const bool is_v = head >= p.N + p.K, turned = !is_v && c < rot;
                // an item's vectors lie half of the turned (or of the copied) elements apart, so that neighbouring
                // threads read and write neighbouring vectors
                const int from = turned || is_v ? 0 : p.R, width = turned ? p.R : H - from;
                const int o0 = from + 8 * (turned || is_v ? c : c - rot), o1 = o0 + width / 2;
                const uint4 a = *reinterpret_cast<const uint4 *>(src + ((x / kPerHead) * H + o0) * 2);
                const uint4 b = *reinterpret_cast<const uint4 *>(src + ((x / kPerHead) * H + o1) * 2);
                f32x2 y0[4], y1[4];
                if (turned) {
                    unpack8<kInter>(a, y0);
                    unpack8<kInter>(b, y1);
                    // group c, or interleaved, group c for one vector and R / 16 + c for the other
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // two pairs at a time
                        const float4 v = angles[(kInter ? e & 1 : e) * kGroups + (kInter && e >= 2 ? rot + c : c)];
                        const f32x2 co = pair(v.x, v.y), si = pair(v.z, v.w), minus = pair(-v.z, -v.w);
                        f32x2 &r0 = kInter ? (e < 2 ? y0[2 * (e & 1)] : y1[2 * (e & 1)]) : y0[e];
                        f32x2 &r1 = kInter ? (e < 2 ? y0[2 * (e & 1) + 1] : y1[2 * (e & 1) + 1]) : y1[e];
                        const f32x2 f0 = r0, f1 = r1;
                        r0 = fma2(f0, co, mul2(f1, minus));
                        r1 = fma2(f0, si, mul2(f1, co));
                    }
                    if constexpr (kInter) {
                        join8(y0);
                        join8(y1);
                    }
                } else if (kFp8 && head >= p.N) {
                    unpack8<false>(a, y0);
                    unpack8<false>(b, y1);
                }
                const int at = (head - p.N - (is_v ? p.K : 0)) * H;
                if (kFp8 && head >= p.N) {
                    uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + row_off + at;
                    uint2 c0, c1;
                    rope_quantize(y0, y1, reciprocal(sc[kFp8 ? r : 0]), c0, c1);
                    *reinterpret_cast<uint2 *>(dst + o0) = c0;
                    *reinterpret_cast<uint2 *>(dst + o1) = c1;
                } else {
                    uint16_t *dst = head < p.N ? q_row + head * H : static_cast<uint16_t *>(is_v ? p.v_cache : p.k_cache) + row_off + at;
                    *reinterpret_cast<uint4 *>(dst + o0) = turned ? pack8(y0) : a;
                    *reinterpret_cast<uint4 *>(dst + o1) = turned ? pack8(y1) : b;
                }
            }
        }
        __syncthreads();  // every thread is done with this unit's stage and the next unit's angles
        if (aborted) {
            if (tid == 0) {  // leave no copy in flight behind
                set_flag(p.err_flag, PKV_FLAG_TIMEOUT);
                for (int x = k; x < copied; ++x)
                    mbar_wait_bounded(smem_u32(full + x % S), (uint32_t)(x / S) & 1, nullptr, kDrainLimitNs);
            }
            __syncthreads();
            return;
        }
        if (tid == 0 && ahead.i < p.n) {
            load(ahead, stage);
            ++copied;
            advance(ahead);
        }
        if (next.i >= p.n) return;
        now = next;
        advance(next);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) sc[r] = sc_next[r];
    }
}

template <int H, bool kInter, bool kFp8>
static cudaError_t launch_k(const RopeParams &p, unsigned grid, cudaStream_t stream)
{
    constexpr int smem = kRopeStages * kUnitHeads * H * 2;
    static int ready[64] = {};  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(rope_append_kernel<H, kInter, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev] = 1;
    }
    return launch_kernel(rope_append_kernel<H, kInter, kFp8>, dim3(grid), dim3(kRopeThreads), smem, stream, true, p);
}

template <int H>
static cudaError_t launch_t(const RopeParams &p, bool interleaved, bool fp8, int sms, cudaStream_t stream)
{
    const int heads = p.N + 2 * p.K;
    const int64_t units = (int64_t)p.n * ((heads + kUnitHeads - 1) / kUnitHeads), most = (int64_t)sms * kRopeCtasPerSm;
    const unsigned grid = (unsigned)(units < most ? units : most);
    if (interleaved) return fp8 ? launch_k<H, true, true>(p, grid, stream) : launch_k<H, true, false>(p, grid, stream);
    return fp8 ? launch_k<H, false, true>(p, grid, stream) : launch_k<H, false, false>(p, grid, stream);
}

cudaError_t launch_rope_append(const RopeParams &p, bool interleaved, bool fp8, int sms, cudaStream_t stream)
{
    return p.H == 128 ? launch_t<128>(p, interleaved, fp8, sms, stream)
                      : launch_t<64>(p, interleaved, fp8, sms, stream);
}

}  // namespace pkv
