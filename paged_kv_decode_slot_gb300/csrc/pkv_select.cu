// pkv_select.cu - which blocks of a long context a decode step attends to: the bounds of a block's
// keys, and the selection of the blocks whose bounds promise the largest logits.
//
// Bounds.  lo[h] and hi[h] are the minimum and the maximum over a block's tokens of element h of its
// keys, one pair of rows per (physical block, KV head), so that blocks shared by sequences share them.
//
// Score.  For any key k of a block  q . k <= sum_h max(q_h lo_h, q_h hi_h); a block's score for a KV head is
// the largest of that bound over the G query heads that share it.  As max(q lo, q hi) is q hi where
// q > 0 and q lo elsewhere, the bounds of 16 blocks against 8 heads are one matrix product of depth 2H:
//     S[16 blocks x 8] = lo . min(q, 0)^T + hi . max(q, 0)^T        (mma.sync m16n8k16, bf16, fp32 sums)
// The operands need no rounding (min, max and the parts of q are bf16 numbers), so a score is off by the
// order of its fp32 sums alone.
//
// Two launches, the second started early (programmatic serialization): scores into the workspace, then one CTA per
// (sequence, KV head) chooses.  64 sequences of 8K to 32K tokens, 8 KV heads, 128 blocks each: 71 us, of which the scores,
// bound by memory, 57 for 336 MB (5.9 TB/s, 87% of the measured copy bandwidth); one sequence of 32K tokens: 9.1 us, the
// latency of a tile's loads (3.5) and of the choice's barriers and passes over shared memory (5.5).
//
// Selection.  The first F and the last L blocks, and the best of the rest, M in all, in ascending order:
// exactly those that the scores' real values choose, rounded once to 64 bits, ties to the lowest index.  With eps bounding the
// error of every score, t the k-th largest score: a block above t + 2 eps is in, one below t - 2 eps is out,
// and if those between do not all fit, their sums are taken again, as integers (exact_score), and ranked.  Operands whose
// magnitudes lie more than 2^50 apart within a group and a block take a longer sum (wide_score): if every block of one sequence
// of 32K tokens has to, the selection takes 0.7 ms, of 64 such sequences 2.4 ms.
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_ops.h"

namespace pkv {

// ------------------------------------- key bounds -----------------------------------------
// One CTA per block that holds new tokens, one thread per 16-byte column of its [K][H] rows: all 16 rows are
// loaded at once (independent loads), rows past the context are left out.  One pass over the keys,
// bound by memory: 16 prompts of 512 to 8,192 tokens (8 heads of 128, 161 MB) 27.2 us, 5.9 TB/s, 87% of the measured copy
// bandwidth; the newest block of 64 sequences in e4m3 2.4 us, a launch and two dependent loads.  Threads without a column
// idle: half of them in e4m3 (the same prompts 23.5 us, 56%), seven in eight for one head of 128 in bf16 (9.0 us for an eighth of
// the bytes, 33%; e4m3 10.3).
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t min_f16x2(uint32_t a, uint32_t b)
{
    const __half2 r = __hmin2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b)
{
    const __half2 r = __hmax2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

constexpr int kBoundsThreads = 128;

// The physical block and the number of valid rows of this CTA's block; false: nothing to do.
__device__ __forceinline__ bool bounds_block(const BoundsParams &p, int &blk, int &rows)
{
    const int b = blockIdx.y;
    const int ctx = p.context_lens[b];
    if (ctx < 0 || ctx > p.max_nb * kBlockSize) {
        if (threadIdx.x == 0 && blockIdx.x == 0) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        return false;
    }
    const int j = max(0, ctx - p.num_new) / kBlockSize + blockIdx.x;
    if (j >= (ctx + kBlockSize - 1) / kBlockSize) return false;
    blk = p.block_tables[(size_t)b * p.max_nb + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (threadIdx.x == 0) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
        return false;
    }
    rows = min(kBlockSize, ctx - j * kBlockSize);
    return true;
}

__global__ void __launch_bounds__(kBoundsThreads) key_bounds_kernel(const BoundsParams p)
{
    pdl_wait_primary();
    pdl_launch_dependents();
    int blk, rows;
    if (!bounds_block(p, blk, rows)) return;
    const int vecs = p.K * p.H / 8;  // 16-byte columns of a token row
    const uint4 *src = static_cast<const uint4 *>(p.k_cache) + (int64_t)blk * kBlockSize * vecs;
    uint4 *dst = reinterpret_cast<uint4 *>(p.bounds) + (int64_t)blk * 2 * vecs;
    const int hv = p.H / 8;
    for (int x = threadIdx.x; x < vecs; x += kBoundsThreads) {
        uint4 v[kBlockSize];
#pragma unroll
        for (int r = 0; r < kBlockSize; ++r) v[r] = __ldg(src + (int64_t)min(r, rows - 1) * vecs + x);
        uint4 lo = v[0], hi = v[0];
#pragma unroll
        for (int r = 1; r < kBlockSize; ++r) {  // rows past the last one repeat it
            lo = make_uint4(min_bf16x2(lo.x, v[r].x), min_bf16x2(lo.y, v[r].y), min_bf16x2(lo.z, v[r].z), min_bf16x2(lo.w, v[r].w));
            hi = make_uint4(max_bf16x2(hi.x, v[r].x), max_bf16x2(hi.y, v[r].y), max_bf16x2(hi.z, v[r].z), max_bf16x2(hi.w, v[r].w));
        }
        uint4 *row = dst + (x / hv) * 2 * hv + x % hv;
        row[0] = lo;
        row[hv] = hi;
    }
}

// e4m3: the codes widen exactly to f16, the order of the values is the order of the codes (scales are
// positive), and code * scale is rounded once to bf16 -- to nearest, so a bound may lie half a bf16
// step inside the key it bounds.
__global__ void __launch_bounds__(kBoundsThreads) key_bounds_fp8_kernel(const BoundsParams p)
{
    pdl_wait_primary();
    pdl_launch_dependents();
    int blk, rows;
    if (!bounds_block(p, blk, rows)) return;
    const int vecs = p.K * p.H / 16;
    const uint4 *src = static_cast<const uint4 *>(p.k_cache) + (int64_t)blk * kBlockSize * vecs;
    const int hv = p.H / 16;
    for (int x = threadIdx.x; x < vecs; x += kBoundsThreads) {
        uint4 v[kBlockSize];
#pragma unroll
        for (int r = 0; r < kBlockSize; ++r) v[r] = __ldg(src + (int64_t)min(r, rows - 1) * vecs + x);
        const int kvh = x / hv;
        const float sc = __ldg(p.k_scale + (int64_t)blk * p.scale_stride + kvh);
        uint32_t lo[8], hi[8];
#pragma unroll
        for (int r = 0; r < kBlockSize; ++r) {
            const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t c0, c1;
                e4m3x4_to_f16x2x2(w[e], c0, c1);
                lo[2 * e] = r ? min_f16x2(lo[2 * e], c0) : c0;
                lo[2 * e + 1] = r ? min_f16x2(lo[2 * e + 1], c1) : c1;
                hi[2 * e] = r ? max_f16x2(hi[2 * e], c0) : c0;
                hi[2 * e + 1] = r ? max_f16x2(hi[2 * e + 1], c1) : c1;
            }
        }
        uint16_t *row = p.bounds + ((int64_t)blk * p.K + kvh) * 2 * p.H + (x % hv) * 16;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t *s = e ? hi : lo;
            uint32_t o[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) o[y] = pack_bf16x2(f16x2_lo(s[y]) * sc, f16x2_hi(s[y]) * sc);
            uint4 *d = reinterpret_cast<uint4 *>(row + e * p.H);
            d[0] = make_uint4(o[0], o[1], o[2], o[3]);
            d[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

cudaError_t launch_key_bounds(const BoundsParams &p, bool fp8, int span, cudaStream_t stream)
{
    const dim3 grid(span, p.B);
    return launch_kernel(fp8 ? key_bounds_fp8_kernel : key_bounds_kernel, grid, dim3(kBoundsThreads), 0, stream, true, p);
}

// -------------------------------------- selection -------------------------------------------
constexpr int kMostWarps = 16;      // of a choosing CTA
constexpr int kBinBits = 9, kBins = 1 << kBinBits;  // bins of one narrowing pass
constexpr int kRankMost = 256;      // undecided blocks ranked pairwise; more go through narrowing passes
constexpr int kFew = 64;            // keys of one bin ranked pairwise
constexpr int kKeep = 8192;         // scores the choosing CTA keeps in shared memory (131,072 tokens); longer
                                    // contexts read them from L2 in every pass

// Order-preserving maps to unsigned integers; NaN counts as +inf (such a block is attended to, so the NaN
// shows in the output instead of being left out), and -0 as +0.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (x != x) x = INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ unsigned long long order_key(double x)
{
    if (x != x) x = __longlong_as_double(0x7FF0000000000000ll);
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

struct SelectShared {
    uint32_t hist[kBins];
    uint32_t warp_sum[2][kMostWarps];
    unsigned long long range[2][kMostWarps];
    unsigned long long lo, hi;  // range of a narrowing pass
    uint32_t above, inside;     // keys above the chosen bin, and in it
    uint32_t few_n;
    unsigned long long few[kFew];
    float bound[2][kMostWarps];  // |q|_1 and the largest |bound|, by warp
    double exact[kRankMost];
    int32_t list[kRankMost];
    uint32_t chosen[kRankMost];
};

// Sum and exclusive prefix sum over the CTA of one value per thread.
template <int NT>
__device__ __forceinline__ uint32_t block_exclusive(SelectShared &s, uint32_t v, uint32_t &total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
        if (lane >= off) inc += o;
    }
    __syncthreads();
    if (lane == 31) s.warp_sum[0][warp] = inc;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < (NT / 32); ++w) {
        const uint32_t x = s.warp_sum[0][w];
        before += w < warp ? x : 0u;
        sum += x;
    }
    total = sum;
    return before + inc - v;
}

template <typename Key>
__device__ __forceinline__ void warp_range(Key &mn, Key &mx)
{
    if constexpr (sizeof(Key) == 4) {
        mn = __reduce_min_sync(0xFFFFFFFFu, mn);
        mx = __reduce_max_sync(0xFFFFFFFFu, mx);
    } else {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            mn = min(mn, (Key)__shfl_xor_sync(0xFFFFFFFFu, mn, off));
            mx = max(mx, (Key)__shfl_xor_sync(0xFFFFFFFFu, mx, off));
        }
    }
}

// The k-th largest (k >= 1) of the n keys key(0 .. n-1), whose smallest and largest are mn and mx over this
// thread's share (any split over the CTA), and the number of keys above it.  Narrowing passes: the keys' range
// is cut into up to 512 bins and the bin that holds the k-th becomes the range; a bin is 2^shift keys
// wide, so a pass takes nine bits off the range whatever the keys are.  The first range is that of the keys
// themselves: the scores of one query lie within a few powers of two and spread over the bins, so shared-memory
// atomics seldom meet, and one pass nearly always leaves few enough keys to rank them pairwise.  A thread only asks for
// the keys i = tid mod NT; a barrier has to lie between this and whatever used s before.
// Keys that change on the way (another stream writing the workspace, against the rules) make the result meaningless, but
// the passes are counted, places are checked and the call ends.
template <int NT, typename Key, typename F>
__device__ __forceinline__ Key kth_largest(SelectShared &s, int n, uint32_t k, F key, Key mn, Key mx, uint32_t &above)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kMine = kBins >= NT ? kBins / NT : 1;  // bins of a thread, of the first kBins / kMine threads
    // from the top: thread t holds bins [kBins - kMine (t + 1), kBins - kMine t)
    const int b0 = kBins - kMine * (tid + 1);
    warp_range(mn, mx);
    if (lane == 0) s.range[0][warp] = mn, s.range[1][warp] = mx;
#pragma unroll
    for (int x = 0; x < kMine; ++x)
        if (b0 >= 0) s.hist[b0 + x] = 0u;
    if (tid == 0) s.few_n = 0u;
    __syncthreads();
    unsigned long long all_lo = s.range[0][0], all_hi = s.range[1][0];
#pragma unroll
    for (int w = 1; w < (NT / 32); ++w) {
        all_lo = min(all_lo, s.range[0][w]);
        all_hi = max(all_hi, s.range[1][w]);
    }
    Key lo = (Key)all_lo, hi = (Key)all_hi;
    uint32_t up = 0, inside = (uint32_t)n;  // keys above hi, keys in [lo, hi]
    constexpr int kPasses = (8 * (int)sizeof(Key) + kBinBits - 1) / kBinBits;
    for (int pass = 0; pass < kPasses && lo < hi && inside > kFew; ++pass) {
        const int bits = 64 - __clzll((long long)(unsigned long long)(hi - lo));
        const int shift = max(0, bits - kBinBits);
#pragma unroll 4
        for (int i = tid; i < n; i += NT) {
            const Key x = key(i);
            if (x >= lo && x <= hi) atomicAdd(&s.hist[(uint32_t)((x - lo) >> shift)], 1u);
        }
        __syncthreads();
        uint32_t mine[kMine], sum = 0;
#pragma unroll
        for (int x = 0; x < kMine; ++x) {
            mine[x] = b0 >= 0 ? s.hist[b0 + x] : 0u;
            sum += mine[x];
            if (b0 >= 0) s.hist[b0 + x] = 0u;  // for another pass
        }
        uint32_t inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) s.warp_sum[0][warp] = inc;
        __syncthreads();
        uint32_t before = up + inc - sum;
#pragma unroll
        for (int w = 0; w < (NT / 32); ++w) before += w < warp ? s.warp_sum[0][w] : 0u;
        if (before < k && before + sum >= k) {  // one thread: the k-th is in one of its bins
#pragma unroll
            for (int x = kMine - 1; x >= 0; --x) {
                if (before < k && before + mine[x] >= k) {
                    const unsigned long long from = (unsigned long long)lo + ((unsigned long long)(b0 + x) << shift);
                    s.lo = from;
                    s.hi = min((unsigned long long)hi, from + min((1ull << shift) - 1, ~from));  // no wrap at the top
                    s.above = before;
                    s.inside = mine[x];
                }
                before += mine[x];
            }
        }
        __syncthreads();  // (the next write of lo, hi, above and inside lies behind another barrier)
        lo = (Key)s.lo;
        hi = (Key)s.hi;
        up = s.above;
        inside = s.inside;
    }
    if (lo < hi) {
#pragma unroll 4
        for (int i = tid; i < n; i += NT) {
            const Key x = key(i);
            if (x >= lo && x <= hi) {
                const uint32_t at = atomicAdd(&s.few_n, 1u);
                if (at < kFew) s.few[at] = (unsigned long long)x;
            }
        }
        __syncthreads();
        inside = min(inside, (uint32_t)kFew);
        if (tid < (int)inside) {
            const Key x = (Key)s.few[tid];
            uint32_t more = up, same = 0;
#pragma unroll 4
            for (uint32_t o = 0; o < inside; ++o) {
                const Key y = (Key)s.few[o];
                more += y > x;
                same += y == x;
            }
            if (more < k && more + same >= k) {  // equal keys write equal values
                s.lo = (unsigned long long)x;
                s.above = more;
            }
        }
        __syncthreads();
        lo = (Key)s.lo;
        up = s.above;
    }
    above = up;
    return lo;
}

// The sum over a warp of m[e] 2^(at[e] - 266), |m| < 2^16, 0 <= at <= 506, rounded once to 64 bits (to nearest, ties to even).
// In digits of 16 bits from the lowest one that any term reaches: the terms' parts of a digit are added up as integers, what
// is beyond 16 bits is carried on, and the last 80 bits are kept with a note of what fell off below them.
template <int E>
__device__ __forceinline__ double exact_sum(const int (&m)[E], const int (&at)[E])
{
    int from = 512, to = 0, sign = 1;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (m[e]) from = min(from, at[e]), to = max(to, at[e]);
    from = __reduce_min_sync(0xFFFFFFFFu, from) >> 4;
    to = (__reduce_max_sync(0xFFFFFFFFu, to) >> 4) + 2;  // 16 bits of the terms, 7 of their number
    unsigned long long window = 0, best = 0;  // the last four digits; as they were at the highest digit that is not 0
    unsigned under = 0, best_under = 0;       // the digit below them
    bool lost, best_lost = false;             // anything below that one
    int top = -1;
    for (int turn = 0; turn < 2; ++turn) {
        int carry = 0;
        lost = false, window = 0, under = 0, top = -1;
        for (int i = from; i <= to; ++i) {
            int part = carry;
            int mine = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int v = sign * m[e] * (1 << (at[e] & 15)), w = at[e] >> 4;  // below 2^31
                mine += w == i ? v & 0xFFFF : (w + 1 == i ? v >> 16 : 0);
            }
            part += __reduce_add_sync(0xFFFFFFFFu, mine);
            const unsigned digit = part & 0xFFFF;
            carry = part >> 16;
            lost |= under != 0;
            under = (unsigned)window & 0xFFFFu;
            window = window >> 16 | (unsigned long long)digit << 48;
            if (digit) best = window, best_under = under, best_lost = lost, top = i;
        }
        if (carry >= 0) break;
        if (turn == 0) sign = -1;  // a negative sum: once more with the signs turned round
    }
    if (top < 0) return 0.0;
    const int lead = __clzll((long long)best);  // below 16
    const unsigned long long r =
        best << lead | best_under >> (16 - lead) | (unsigned long long)(best_lost || (best_under << lead & 0xFFFFu));
    const double unit = __longlong_as_double((long long)(1023 + 16 * (top - 3) - lead - 266) << 52);
    return (sign < 0 ? -unit : unit) * __ull2double_rn(r);
}

// A block's score, rounded once to 64 bits, whatever its operands: q [G][H] and the block's two rows of bounds, at this lane's
// elements.  Head by head; infinities and NaN go through 64-bit floating point, where nothing finite changes the outcome.
// Seldom needed, so a call of its own.
template <int H>
__device__ __noinline__ double wide_score(const uint16_t *q, const uint16_t *row, int G)
{
    constexpr int E = H / 32;
    double best = -__longlong_as_double(0x7FF0000000000000ll);
    bool nan = false;
    for (int g = 0; g < G; ++g) {
        int m[E], at[E];
        uint16_t x[E], b[E];
        bool odd = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = q[g * H + e];
            b[e] = row[(bf16_to_f32(x[e]) > 0.f ? H : 0) + e];
            const int ex = x[e] >> 7 & 255, eb = b[e] >> 7 & 255;
            odd |= ex == 255 || eb == 255;
            const int v = ((x[e] & 127) | (ex ? 128 : 0)) * ((b[e] & 127) | (eb ? 128 : 0));
            m[e] = (x[e] ^ b[e]) >> 15 ? -v : v;
            at[e] = max(ex, 1) + max(eb, 1) - 2;  // q is its mantissa times 2^(ex - 134), and so is the bound
        }
        double sum = 0.0;
        if (__any_sync(0xFFFFFFFFu, odd)) {
#pragma unroll
            for (int e = 0; e < E; ++e) sum += (double)bf16_to_f32(x[e]) * (double)bf16_to_f32(b[e]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        } else {
            sum = exact_sum<E>(m, at);
        }
        nan |= sum != sum;
        best = sum > best ? sum : best;
    }
    return nan ? __longlong_as_double(0x7FF8000000000000ll) : best;
}

// The score of block j, rounded once to 64 bits.  fp64 units are few on this chip (through them this step took
// 5 us of a choice, so it takes 1.5), so the products, scaled below 1 by powers of two, are added up as integers: adding 3
// rounds a number below 1 to a multiple of 2^-22 in the sum's bits, the rest goes the same way at 2^-44 and 2^-66.  A product
// has 16 bits, so nothing is lost where the smallest operands are within 2^50 of the largest, in the exponents of the group's
// queries and of the block's bounds together; other blocks take wide_score.  kHold: the queries are held in registers and on
// their way while the block is looked up (1.2 us less for a CTA that has registers to spare).
template <int H, bool kHold>
__device__ __forceinline__ double exact_score(const SelectParams &p, int b, int kvh, int j, int lane)
{
    constexpr int E = H / 32;  // neighbouring elements of a lane
    constexpr float kA = 3.f, kB = 3.f / (1 << 22), kC = kB / (1 << 22);
    const double kInf = __longlong_as_double(0x7FF0000000000000ll);
    const int blk = __ldg(p.block_tables + (size_t)b * p.max_nb + j);
    const uint16_t *q = p.q + ((size_t)b * p.N + (size_t)kvh * p.G) * H + lane * E;
    uint16_t held[kHold ? 8 : 1][E];
    unsigned top_b = 0, top_q = 0, low_b = ~0u, low_q = ~0u;  // largest, and smallest but 0 (less 1)
    auto range = [](unsigned x, unsigned &top, unsigned &low) {
        top = max(top, x & 0x7FFFu);
        low = min(low, (x & 0x7FFFu) - 1u);
    };
    if constexpr (kHold) {
#pragma unroll
        for (int g = 0; g < 8; ++g)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                held[g][e] = g < p.G ? q[g * H + e] : 0;
                range(held[g][e], top_q, low_q);
            }
    }
    if (blk < 0 || blk >= p.num_blocks) return -kInf;
    const uint16_t *row = p.bounds + ((int64_t)blk * p.K + kvh) * 2 * H + lane * E;
    float lo[E], hi[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const unsigned l = row[e], h = row[H + e];
        lo[e] = bf16_to_f32((uint16_t)l), hi[e] = bf16_to_f32((uint16_t)h);
        range(l, top_b, low_b);
        range(h, top_b, low_b);
    }
    if constexpr (!kHold) {
#pragma unroll 4
        for (int g = 0; g < p.G; ++g)
#pragma unroll
            for (int e = 0; e < E; ++e) range(q[g * H + e], top_q, low_q);
    }
    const int eb = (int)(__reduce_max_sync(0xFFFFFFFFu, top_b) >> 7), eq = (int)(__reduce_max_sync(0xFFFFFFFFu, top_q) >> 7);
    const int sb = (int)(__reduce_min_sync(0xFFFFFFFFu, low_b) + 1u >> 7), sq = (int)(__reduce_min_sync(0xFFFFFFFFu, low_q) + 1u >> 7);
    // infinities, NaN and numbers whose scale is out of range; products whose last bit lies below 2^-66
    if (eb >= 253 || eq >= 253 || (eb - max(sb, 1)) + (eq - max(sq, 1)) > 50) return wide_score<H>(q, row, p.G);
    const float fb = __uint_as_float((unsigned)(253 - eb) << 23), fq = __uint_as_float((unsigned)(253 - eq) << 23);
#pragma unroll
    for (int e = 0; e < E; ++e) lo[e] *= fb, hi[e] *= fb;
    unsigned mine[3] = {0, 0, 0};  // lane g keeps head g's sums
#pragma unroll(kHold ? 8 : 2)
    for (int g = 0; g < (kHold ? 8 : p.G); ++g) {
        if (g >= p.G) break;
        unsigned a = 0, s1 = 0, s2 = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float x = bf16_to_f32(kHold ? held[kHold ? g : 0][e] : q[g * H + e]), y = (x * fq) * (x > 0.f ? hi[e] : lo[e]);
            const float t = __fadd_rn(y, kA), r = __fsub_rn(y, __fsub_rn(t, kA));
            const float t1 = __fadd_rn(r, kB), r1 = __fsub_rn(r, __fsub_rn(t1, kB));
            a += __float_as_uint(t);
            s1 += __float_as_uint(t1);
            s2 += __float_as_uint(__fadd_rn(r1, kC));
        }
        a = __reduce_add_sync(0xFFFFFFFFu, a);
        s1 = __reduce_add_sync(0xFFFFFFFFu, s1);
        s2 = __reduce_add_sync(0xFFFFFFFFu, s2);
        if (lane == g) mine[0] = a, mine[1] = s1, mine[2] = s2;
    }
    // the constants' bits off again: counts of 2^-22, 2^-44 and 2^-66
    const int ua = (int)(mine[0] - H * __float_as_uint(kA)), ub = (int)(mine[1] - H * __float_as_uint(kB)),
              uc = (int)(mine[2] - H * __float_as_uint(kC));
    const double unit = __longlong_as_double((long long)(1023 + eb + eq - 252 - 44) << 52);  // 2^-44 of the scales' product
    double sum = fma((double)uc, unit * 0x1p-22, (double)(((long long)ua << 22) + ub) * unit);
    if (lane >= p.G) sum = -kInf;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
        const double o = __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        sum = o > sum ? o : sum;
    }
    return __shfl_sync(0xFFFFFFFFu, sum, 0);
}

// A warp's contiguous run of the blocks [0, nb): the runs in warp order are the blocks in ascending order.
template <int NT>
__device__ __forceinline__ void warp_run(int nb, int &begin, int &end)
{
    const int per = ((nb + (NT / 32) - 1) / (NT / 32) + 31) / 32 * 32;
    begin = min(nb, (int)(threadIdx.x >> 5) * per);
    end = min(nb, begin + per);
}

// Blocks [0, nb) by class(j), two bits: bit 0 and bit 1 are counted apart, in all and in the runs of earlier warps.
// Lane i keeps what the warp's i-th 32 blocks answered.
struct Counts {
    uint32_t all[2], before[2], mask[2];
};

template <int NT, typename Class>
__device__ __forceinline__ Counts count_runs(SelectShared &s, int nb, Class cls)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int begin, end;
    warp_run<NT>(nb, begin, end);
    Counts c{{0, 0}, {0, 0}, {0, 0}};
    uint32_t n0 = 0, n1 = 0;
#pragma unroll 4
    for (int j0 = begin; j0 < end; j0 += 32) {
        const int x = j0 + lane < end ? cls(j0 + lane) : 0;
        const uint32_t m0 = __ballot_sync(0xFFFFFFFFu, x & 1), m1 = __ballot_sync(0xFFFFFFFFu, x & 2);
        if (lane == (j0 - begin) / 32) c.mask[0] = m0, c.mask[1] = m1;
        n0 += __popc(m0);
        n1 += __popc(m1);
    }
    __syncthreads();
    if (lane == 0) s.warp_sum[0][warp] = n0, s.warp_sum[1][warp] = n1;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < (NT / 32); ++w) {
        const uint32_t x = s.warp_sum[0][w], y = s.warp_sum[1][w];
        c.all[0] += x;
        c.all[1] += y;
        c.before[0] += w < warp ? x : 0u;
        c.before[1] += w < warp ? y : 0u;
    }
    return c;
}

// Writes the blocks of [0, nb) whose class has `bit` to dst, ascending.  kMasks: there are at most 1,024 blocks a warp,
// and what count_runs saw is still right.
template <int NT, bool kMasks, typename Class>
__device__ __forceinline__ void write_run(int nb, Class cls, int bit, const Counts &c, int32_t *dst, uint32_t most)
{
    const int lane = threadIdx.x & 31;
    int begin, end;
    warp_run<NT>(nb, begin, end);
    uint32_t before = c.before[bit];
    for (int j0 = begin; j0 < end; j0 += 32) {
        const uint32_t m = kMasks ? __shfl_sync(0xFFFFFFFFu, c.mask[bit], (j0 - begin) / 32)
                                  : __ballot_sync(0xFFFFFFFFu, j0 + lane < end && (cls(j0 + lane) >> bit & 1));
        const uint32_t o = before + __popc(m & ((1u << lane) - 1u));
        if ((m >> lane & 1u) && o < most) dst[o] = j0 + lane;
        before += __popc(m);
    }
}

// The choice of one (sequence, KV head) from its scores.  q1: this warp's share of the largest |q|_1 over the
// group's heads; kKept: the candidates' keys fit in keep (shared memory).
template <int H, int NT, bool kKept>
__device__ __forceinline__ void choose(SelectShared &s, uint32_t *keep, const SelectParams &p, int b, int kvh, int nb,
                                       float q1)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t unit = (size_t)b * p.K + kvh;
    float *scores = p.scores + unit * p.max_nb;
    int32_t *sel = p.selected + unit * p.M;
    const int first = p.first, n = nb - p.first - p.last;  // candidates: blocks first .. first + n - 1
    const uint32_t k = (uint32_t)(p.M - p.first - p.last);  // 0 <= k < n
    auto middle = [&](int j) { return j >= first && j < first + n; };
    if (k == 0) {
        auto forced = [&](int j) { return middle(j) ? 0 : 1; };
        write_run<NT, kKept>(nb, forced, 0, count_runs<NT>(s, nb, forced), sel, (uint32_t)p.M);
        return;
    }

    // the scores, as keys; their range; |q|_1 and the largest |bound| (all loads on their way together)
    uint32_t mn = ~0u, mx = 0u, mb = 0u;
    for (int c = tid; c < (nb + 15) / 16; c += NT) mb = max(mb, __float_as_uint(__ldcg(p.tile_max + unit * p.tiles + c)));
    auto load = [&](int i) { return __ldcg(scores + first + i); };
    {
        constexpr int U = 8;  // loads in flight a thread
        for (int i0 = tid; i0 < n; i0 += U * NT) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * NT < n) x[u] = load(i0 + u * NT);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * NT;
                if (i < n) {
                    const uint32_t y = order_key(x[u]);
                    mn = min(mn, y);
                    mx = max(mx, y);
                    if constexpr (kKept) keep[first + i] = y;
                }
            }
        }
    }
    mb = __reduce_max_sync(0xFFFFFFFFu, mb);  // non-negative numbers order like their bits
    if (lane == 0) s.bound[0][warp] = q1, s.bound[1][warp] = __uint_as_float(mb);  // read behind the barriers that follow
    auto at = [&](int j) -> uint32_t {  // key of block j
        if constexpr (kKept) return keep[j];
        else return order_key(__ldcg(scores + j));
    };
    uint32_t above;
    const uint32_t kt = kth_largest<NT, uint32_t>(s, n, k, [&](int i) { return at(first + i); }, mn, mx, above);
    const float t = __uint_as_float(kt & 0x80000000u ? kt & 0x7FFFFFFFu : ~kt);
    // eps: 2^-18 |q|_1 max|bound| = 2^-18 S.  A score is the fp32 sum of sixteen mma of 16 products each.  No product exceeds
    // S and an mma's own sum its part S' of S; one that keeps 23 bits below its largest term loses at most 2^-23 S' for each
    // of its 16 terms and once more at its end, and every addition after it 2^-24 S: (17 + 7.5) 2^-23 S, and a third as
    // much again for slack in what the documentation leaves open about the rounding inside an mma.  Products and sums that
    // underflow are off by 2^-126 each at most, 2^-117 for all of a score's: 2^-111 has the same slack and changes nothing
    // for scores of ordinary size.  Where products may overflow, S does.
    float all_q = s.bound[0][0], all_b = s.bound[1][0];
#pragma unroll
    for (int w = 1; w < (NT / 32); ++w) {
        all_q = fmaxf(all_q, s.bound[0][w]);
        all_b = fmaxf(all_b, s.bound[1][w]);
    }
    const float eps2 = 2.f * (ldexpf(all_q * all_b, -18) + 0x1p-111f);
    // bounds of the undecided scores, rounded outwards; infinite bounds (0 times infinity in the products) leave every
    // score undecided
    const bool bounded = eps2 < INFINITY;
    const uint32_t kin = bounded ? max(kt, order_key(__fadd_ru(t, eps2))) : ~0u;
    const uint32_t kout = bounded ? min(kt, order_key(__fadd_rd(t, -eps2))) : 0u;
    // bit 0: forced or not below the undecided range; bit 1: undecided
    auto cls = [&](int j) {
        if (!middle(j)) return 1;
        const uint32_t x = at(j);
        return x < kout ? 0 : (x <= kin ? 3 : 1);
    };
    const Counts c = count_runs<NT>(s, nb, cls);
    if (c.all[0] == (uint32_t)p.M) {  // nothing left to decide
        write_run<NT, kKept>(nb, cls, 0, c, sel, (uint32_t)p.M);
        return;
    }
    // more undecided blocks than places: rank them by their sums in 64 bits
    const uint32_t need = (uint32_t)p.M - (c.all[0] - c.all[1]);
    const int m = (int)c.all[1];
    const bool few = kKept && m <= kRankMost;
    int32_t *list = few ? s.list : p.list + unit * p.max_nb;
    write_run<NT, kKept>(nb, cls, 1, c, list, c.all[1]);
    __syncthreads();
    double *exact = m <= kRankMost ? s.exact : p.exact + unit * p.max_nb;
    auto listed = [&](int a) { return min(max(list[a], 0), nb - 1); };  // (a list in the workspace is not taken on trust)
    for (int a = warp; a < m; a += (NT / 32)) {
        const double x = exact_score<H, (NT > 256)>(p, b, kvh, listed(a), lane);
        if (lane == 0) exact[a] = x;
    }
    __syncthreads();
    if (few) {
        for (int a = tid; a < m; a += NT) {
            const unsigned long long x = order_key(exact[a]);
            uint32_t rank = 0;  // the list ascends, so among equals the earlier one goes first
            for (int o = 0; o < m; ++o) {
                const unsigned long long y = order_key(exact[o]);
                rank += y > x || (y == x && o < a);
            }
            s.chosen[a] = rank < need;
        }
        __syncthreads();
        // the earlier warps' runs hold the list's first before[1] blocks
        uint32_t lost = 0;
        for (int a0 = 0; a0 < (int)c.before[1]; a0 += 32)
            lost += __popc(__ballot_sync(0xFFFFFFFFu, a0 + lane < (int)c.before[1] && !s.chosen[a0 + lane]));
        uint32_t at_list = c.before[1], before = c.before[0] - lost;
        int begin, end;
        warp_run<NT>(nb, begin, end);
        for (int j0 = begin; j0 < end; j0 += 32) {
            const uint32_t m0 = __shfl_sync(0xFFFFFFFFu, c.mask[0], (j0 - begin) / 32);
            const uint32_t m1 = __shfl_sync(0xFFFFFFFFu, c.mask[1], (j0 - begin) / 32), below = (1u << lane) - 1u;
            bool in = m0 >> lane & 1u;
            if (m1 >> lane & 1u) in = s.chosen[at_list + __popc(m1 & below)] != 0;
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, in);
            if (in) sel[before + __popc(mask & below)] = j0 + lane;
            before += __popc(mask);
            at_list += __popc(m1);
        }
        return;
    }
    // a decided block's key becomes the largest or the smallest there is
    auto decide = [&](int a, bool in) {
        if constexpr (kKept) keep[listed(a)] = in ? ~0u : 0u;
        else scores[listed(a)] = in ? INFINITY : -INFINITY;
    };
    if (m <= kRankMost) {
        for (int a = tid; a < m; a += NT) {
            const unsigned long long x = order_key(exact[a]);
            uint32_t rank = 0;  // the list ascends, so among equals the earlier one goes first
            for (int o = 0; o < m; ++o) {
                const unsigned long long y = order_key(exact[o]);
                rank += y > x || (y == x && o < a);
            }
            decide(a, rank < need);
        }
    } else {
        unsigned long long lo = ~0ull, hi = 0ull;
        for (int a = tid; a < m; a += NT) {
            lo = min(lo, order_key(exact[a]));
            hi = max(hi, order_key(exact[a]));
        }
        uint32_t over;
        const unsigned long long xt =
            kth_largest<NT, unsigned long long>(s, m, need, [&](int a) { return order_key(exact[a]); }, lo, hi, over);
        // of the sums equal to the need-th one, the first need - over in the list
        uint32_t run = 0;
        for (int a0 = 0; a0 < m; a0 += NT) {
            const int a = a0 + tid;
            const unsigned long long x = a < m ? order_key(exact[a]) : 0ull;
            const bool tie = a < m && x == xt;
            uint32_t total;
            const uint32_t before = run + block_exclusive<NT>(s, tie ? 1u : 0u, total);
            run += total;
            if (a < m) decide(a, x > xt || (tie && before < need - over));
        }
    }
    __syncthreads();
    // above the undecided ones, or decided in (+inf itself may be the top of the undecided range)
    auto in = [&](int j) {
        if (!middle(j)) return 1;
        const uint32_t x = at(j);
        return x > kin || x == (kKept ? ~0u : order_key(INFINITY)) ? 1 : 0;
    };
    write_run<NT, kKept>(nb, in, 0, count_runs<NT>(s, nb, in), sel, (uint32_t)p.M);
}

// ---------------------------------------- scores --------------------------------------------
constexpr int kScoreWarps = 8, kScoreThreads = 32 * kScoreWarps;
constexpr int kScoreStages = 2;  // three measured the same

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool there)
{
    // 16 bytes, or 16 zeros where there is nothing to load
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Tiles of 16 blocks that sequence b is scored in: none where all its blocks are selected anyway.
__device__ __forceinline__ int score_tiles(const SelectParams &p, int b)
{
    if (b >= p.B) return 0;
    const int ctx = __ldg(p.context_lens + b);
    if (ctx < 0 || ctx > p.max_nb * kBlockSize) return 0;
    const int nb = (ctx + kBlockSize - 1) / kBlockSize;
    return nb > p.M ? (nb + 15) / 16 : 0;
}

// Blocks of a sequence that the table has room for.
__device__ __forceinline__ int score_blocks(const SelectParams &p, int b)
{
    return min((__ldg(p.context_lens + b) + kBlockSize - 1) / kBlockSize, p.max_nb);
}

// A warp's place in the list of tiles, ordered (sequence, tile, KV head); b = p.B behind the last one.
struct TileAt {
    int b, tile, kvh, tiles;
    // kScoreWarps entries on, without a division: by_tile and by_kvh are kScoreWarps / K and the remainder
    __device__ __forceinline__ void next(const SelectParams &p, int by_tile, int by_kvh)
    {
        tile += by_tile;
        kvh += by_kvh;
        if (kvh >= p.K) kvh -= p.K, ++tile;
        wrap(p);
    }
    __device__ __forceinline__ void wrap(const SelectParams &p)
    {
        while (tile >= tiles && b < p.B) {
            tile -= tiles;
            tiles = score_tiles(p, ++b);
        }
    }
};

// Each CTA takes a contiguous share of all tiles (they are counted at the start from the lengths, so ragged
// batches and wide tables cost nothing), its warps in turn -- so that the heads of a block, next to each other
// in memory, are read at about the same time -- and each warp streams its tiles through a ring of its own in
// shared memory: a tile's bounds are 4 H bytes a block (8 KB at H = 128), copied asynchronously one tile ahead, the
// block ids one tile further ahead.  The product's depth may be taken in any order, so a lane's 16-byte vectors are its k indices:
// each lane copies exactly what it reads back as mma fragments, and the ring needs no barrier.  Bound by memory:
// eight warps with a tile or two each in flight are 64 to 128 KB per SM.  A warp whose tiles are all of one head (K divides 8)
// loads its queries once a sequence, others with every tile: 64 sequences of 8K to 32K tokens take 43 us with 4 heads, 50
// with 5, 71 with 8 and 86 with 10, 57, 62, 70 and 72% of the copy bandwidth.
template <int H>
__global__ void __launch_bounds__(kScoreThreads, 1) score_blocks_kernel(const SelectParams p)
{
    constexpr int V = H / 32;        // 16-byte vectors of a row that a lane holds
    constexpr int kVecs = 4 * V;     // of a tile: two rows, lo and hi
    constexpr int S = kScoreStages;
    extern __shared__ uint4 ring[];  // [warps][S][kVecs][32]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, m = lane & 3;
    pdl_wait_primary();
    pdl_launch_dependents();  // the choosing grid may take its place; it waits for this one before it reads scores

    int64_t total = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        int t = score_tiles(p, b0 + lane);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, off);
        total += (int64_t)t * p.K;
    }
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    const int64_t begin = blockIdx.x * share, end = min(total, begin + share);
    const int n = end - begin > warp ? (int)((end - begin - warp + kScoreWarps - 1) / kScoreWarps) : 0;
    if (n == 0) return;
    TileAt load_at{p.B, 0, 0, 0};
    const int by_tile = kScoreWarps / p.K, by_kvh = kScoreWarps - by_tile * p.K;
    {
        int64_t before = 0;  // the sequence that holds entry `begin`
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int t = score_tiles(p, b0 + lane);
            int64_t inc = (int64_t)t * p.K;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
                if (lane >= off) inc += o;
            }
            const unsigned past = __ballot_sync(0xFFFFFFFFu, before + inc > begin);
            if (past) {
                const int at = __ffs(past) - 1;
                load_at.b = b0 + at;
                load_at.tiles = __shfl_sync(0xFFFFFFFFu, t, at);
                const int64_t entry = begin + warp - (before + __shfl_sync(0xFFFFFFFFu, inc, at) - (int64_t)load_at.tiles * p.K);
                load_at.tile = (int)(entry / p.K);
                load_at.kvh = (int)(entry - (int64_t)load_at.tile * p.K);
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        load_at.wrap(p);
    }
    TileAt use_at = load_at;

    const uint32_t mine = smem_u32(ring + (warp * S * kVecs) * 32 + lane);
    int blk[2];        // ids of the next tile to copy, of the blocks that are scored
    bool scored[2];
    uint32_t bad = 0;  // of each stage's two rows: the id is outside the pool
    auto look_up = [&](const TileAt &at) {
        const int nb = at.b < p.B ? score_blocks(p, at.b) : 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j = at.tile * 16 + r + 8 * x;
            // forced blocks are selected without a score, and their bounds need not be up to date
            scored[x] = j >= p.first && j < nb - p.last;
            blk[x] = scored[x] ? __ldg(p.block_tables + (size_t)at.b * p.max_nb + j) : -1;
        }
    };
    auto copy = [&](const TileAt &at, int stage) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const bool there = blk[x] >= 0 && blk[x] < p.num_blocks;
            const uint32_t bit = 1u << (2 * stage + x);
            bad = there ? bad & ~bit : bad | bit;
            if (!there && scored[x] && m == 0) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
            const uint16_t *row = p.bounds + ((int64_t)(there ? blk[x] : 0) * p.K + at.kvh) * 2 * H + 8 * m;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    cp_async16(mine + ((stage * kVecs + (x * 2 + e) * V + i) * 32) * 16, row + e * H + 32 * i, there);
        }
    };
    int copied = 0;
    auto advance = [&]() {  // copy the next tile, look the one after it up
        if (copied < n) {
            copy(load_at, copied % S);
            if (++copied < n) {
                load_at.next(p, by_tile, by_kvh);
                look_up(load_at);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(load_at);
#pragma unroll
    for (int x = 0; x < S - 1; ++x) advance();

    int q_b = -1, q_kvh = -1, nb = 0;
    uint32_t qf[2][V][4];  // fragments of min(q, 0) and max(q, 0)
    for (int i = 0; i < n; ++i) {
        advance();
        if (use_at.b >= p.B) break;  // (lengths that changed since they were counted)
        const int tile = use_at.tile, kvh = use_at.kvh;
        if (use_at.b != q_b || kvh != q_kvh) {
            q_b = use_at.b, q_kvh = kvh;
            nb = score_blocks(p, q_b);
            const bool live = r < p.G;
            const uint16_t *qrow = p.q + ((size_t)q_b * p.N + (size_t)q_kvh * p.G + (live ? r : 0)) * H + 8 * m;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint4 x = live ? __ldg(reinterpret_cast<const uint4 *>(qrow + 32 * v)) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    qf[0][v][y] = min_bf16x2(xw[y], 0u);
                    qf[1][v][y] = max_bf16x2(xw[y], 0u);
                }
            }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        const int stage = i % S;
        const uint4 *src = ring + (size_t)((warp * S + stage) * kVecs) * 32 + lane;
        float c[4] = {};
        uint32_t big = 0u, small = 0u;  // packed largest upper and smallest lower bound: |bound| is at most the larger end
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint4 x = src[(e * V + v) * 32], y = src[((2 + e) * V + v) * 32];
                const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
                // every product's sum on its own, added up in fp32: the error bound of the scores stays small
                float c0[4] = {}, c1[4] = {};
                mma_bf16_16816(c0, a0, qf[e][v][0], qf[e][v][1]);
                mma_bf16_16816(c1, a1, qf[e][v][2], qf[e][v][3]);
#pragma unroll
                for (int y2 = 0; y2 < 4; ++y2) c[y2] += c0[y2] + c1[y2];
#pragma unroll
                for (int y2 = 0; y2 < 4; ++y2) {
                    if (e) big = max_bf16x2(max_bf16x2(big, a0[y2]), a1[y2]);
                    else small = min_bf16x2(min_bf16x2(small, a0[y2]), a1[y2]);
                }
            }
        }
        const size_t unit = (size_t)q_b * p.K + q_kvh;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            // this lane's columns are heads 2m and 2m + 1
            const float s0 = c[2 * x], s1 = c[2 * x + 1];
            float best = -INFINITY;
            bool nan = false;
            if (2 * m < p.G) best = s0, nan = s0 != s0;
            if (2 * m + 1 < p.G) best = fmaxf(best, s1), nan |= s1 != s1;
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, off));
            const unsigned nans = __ballot_sync(0xFFFFFFFFu, nan);
            if ((nans >> (lane & ~3)) & 15u) best = __int_as_float(0x7FC00000);
            if ((bad >> (2 * stage + x)) & 1u) best = -INFINITY;
            const int j = tile * 16 + r + 8 * x;
            if (m == 0 && j < nb) p.scores[unit * p.max_nb + j] = best;
        }
        big = max_bf16x2(big, small ^ 0x80008000u);  // NaN stays
        // non-negative numbers order like their bits, NaN above all: no bound on the error then, nor with infinities
        const uint32_t top = max(big & 0xFFFFu, big >> 16);
        const float mb = __uint_as_float(min(__reduce_max_sync(0xFFFFFFFFu, top & 0x7FFFu) << 16, 0x7F800000u));
        if (lane == 0) p.tile_max[unit * p.tiles + tile] = mb;
        if (i + 1 < n) use_at.next(p, by_tile, by_kvh);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int H, int NT>
__global__ void __launch_bounds__(NT, NT > 256 ? 1 : 4) choose_blocks_kernel(const SelectParams p)
{
    __shared__ SelectShared s;
    extern __shared__ uint32_t keep[];  // [min(max_nb, kKeep)]
    const int kvh = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ int blocks;
    if (tid == 0) {  // one thread's word for all, as the CTA's barriers depend on it
        int ctx = p.context_lens[b];
        if (ctx < 0 || ctx > p.max_nb * kBlockSize) {
            if (kvh == 0) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
            ctx = 0;
        }
        blocks = (ctx + kBlockSize - 1) / kBlockSize;
    }
    __syncthreads();
    const int nb = blocks;
    if (nb <= p.M) {  // every block is selected
        int32_t *sel = p.selected + ((size_t)b * p.K + kvh) * p.M;
        for (int x = tid; x < p.M; x += NT) sel[x] = x < nb ? x : -1;
        pdl_wait_primary();  // whatever runs next on the stream finds the scoring grid done, too
        return;
    }
    float q1 = 0.f;
    for (int g = warp; g < p.G; g += (NT / 32)) {
        const uint16_t *q = p.q + ((size_t)b * p.N + (size_t)kvh * p.G + g) * H;
        float x = 0.f;
#pragma unroll
        for (int h = 0; h < H; h += 32) x += fabsf(bf16_to_f32(q[h + lane]));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
        q1 = fmaxf(q1, x);
    }
    pdl_wait_primary();  // the scores
    pdl_launch_dependents();
    if (nb <= kKeep) choose<H, NT, true>(s, keep, p, b, kvh, nb, q1);
    else choose<H, NT, false>(s, keep, p, b, kvh, nb, q1);
}

template <int H>
static cudaError_t launch_select_t(const SelectParams &p, int sms, cudaStream_t stream)
{
    constexpr int smem = kScoreWarps * kScoreStages * (H / 8) * 32 * 16;
    static int ready[64] = {};  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(score_blocks_kernel<H>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev] = 1;
    }
    const int64_t most = ((int64_t)p.B * p.K * p.tiles + kScoreWarps - 1) / kScoreWarps;  // a tile per warp
    const unsigned grid = (unsigned)(most < sms ? most : sms);
    e = launch_kernel(score_blocks_kernel<H>, dim3(grid), dim3(kScoreThreads), smem, stream, true, p);
    if (e != cudaSuccess) return e;
    static_assert(sizeof(SelectShared) + sizeof(uint32_t) * kKeep <= 48 * 1024, "no opt-in to larger shared memory");
    const size_t keep = sizeof(uint32_t) * (size_t)(p.max_nb < kKeep ? p.max_nb : kKeep);
    const dim3 units(p.K, p.B);
    // Threads of a choosing CTA: 256 where the batch's CTAs share the SMs (64 * 8 units of up to 2,048 blocks: 70.2 us
    // for the whole selection, 82.4 with 512), 512 where there are fewer units than SMs (18 * 8 units of up to 2,048: 28.4,
    // 30.2 with 256; 8 * 8 of 2,048 23.3 and 25.6; 8 of 2,048 alike).
    if ((int64_t)p.K * p.B < sms) return launch_kernel(choose_blocks_kernel<H, 512>, units, dim3(512), keep, stream, true, p);
    return launch_kernel(choose_blocks_kernel<H, 256>, units, dim3(256), keep, stream, true, p);
}

cudaError_t launch_select_blocks(const SelectParams &p, int H, int sms, cudaStream_t stream)
{
    return H == 128 ? launch_select_t<128>(p, sms, stream) : launch_select_t<64>(p, sms, stream);
}

}  // namespace pkv
