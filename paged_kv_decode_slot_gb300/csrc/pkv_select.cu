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
// Selection.  The first F and the last L blocks, and the best of the rest, M in all, in ascending order:
// exactly those that the scores' real values choose, ties to the lowest index.  With eps bounding the
// error of every score, t the k-th largest score: a block above t + 2 eps is in, one below t - 2 eps is out,
// and if those between do not all fit, their sums are taken again in 64 bits and ranked.
#include "pkv_device.cuh"
#include "pkv_ops.h"

namespace pkv {

// ------------------------------------- key bounds -----------------------------------------
// One CTA per block that holds new tokens, one thread per 16-byte column of its [K][H] rows: all 16 rows are
// loaded at once (independent loads), rows past the context are left out.  One pass over the keys,
// bound by memory.
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
    if (j * kBlockSize >= ctx) return false;
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
    if (fp8) key_bounds_fp8_kernel<<<grid, kBoundsThreads, 0, stream>>>(p);
    else key_bounds_kernel<<<grid, kBoundsThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// -------------------------------------- selection -------------------------------------------
constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;         // bins of one narrowing pass
constexpr int kRankMost = 256;      // undecided blocks ranked pairwise; more go through narrowing passes
static_assert(kSelectChunk == 16 * kSelectWarps, "a warp scores 16 blocks");

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
    uint32_t warp_sum[kSelectWarps + 1];
    unsigned long long lo, hi;       // range of a narrowing pass
    uint32_t above;        // keys above the chosen bin
    uint32_t count;
    float eps, q1;
    double exact[kRankMost];
    int last_one;
};

// Exclusive prefix sum over the CTA of one value per thread; total gets the sum.
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
    if (lane == 31) s.warp_sum[warp] = inc;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kSelectWarps; ++w) {
        const uint32_t x = s.warp_sum[w];
        before += w < warp ? x : 0u;
        sum += x;
    }
    total = sum;
    return before + inc - v;
}

// The k-th largest (k >= 1) of the n keys key(0..n-1), and the number of keys above it.  Narrowing passes:
// the keys' range is cut into up to 2048 bins, the bin that holds the k-th becomes the range; a bin is
// 2^shift keys wide, so a pass takes eleven bits off the range, whatever the keys are.  The first range is
// that of the keys themselves: scores of one query lie within a few powers of two and spread over the
// bins, so the shared-memory atomics seldom meet.
template <typename Key, typename F>
__device__ __forceinline__ Key kth_largest(SelectShared &s, int n, uint32_t k, F key, uint32_t &above)
{
    const int tid = threadIdx.x;
    Key mn = ~Key(0), mx = 0;
    for (int i = tid; i < n; i += kSelectThreads) {
        const Key x = key(i);
        mn = min(mn, x);
        mx = max(mx, x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        mn = min(mn, (Key)__shfl_xor_sync(0xFFFFFFFFu, mn, off));
        mx = max(mx, (Key)__shfl_xor_sync(0xFFFFFFFFu, mx, off));
    }
    __syncthreads();
    if (tid == 0) s.lo = ~0ull, s.hi = 0ull, s.above = 0u;
    __syncthreads();
    if ((tid & 31) == 0) {
        atomicMin(&s.lo, (unsigned long long)mn);
        atomicMax(&s.hi, (unsigned long long)mx);
    }
    __syncthreads();
    Key lo = (Key)s.lo, hi = (Key)s.hi;
    uint32_t up = 0;  // keys above hi
    while (lo < hi) {
        const int bits = 64 - __clzll((long long)(unsigned long long)(hi - lo));
        const int shift = max(0, bits - 11);
        for (int x = tid; x < kBins; x += kSelectThreads) s.hist[x] = 0u;
        __syncthreads();
        for (int i = tid; i < n; i += kSelectThreads) {
            const Key x = key(i);
            if (x >= lo && x <= hi) atomicAdd(&s.hist[(uint32_t)((x - lo) >> shift)], 1u);
        }
        __syncthreads();
        // bins from the top: thread t holds bins [kBins - 8 (t + 1), kBins - 8 t)
        uint32_t mine[kBins / kSelectThreads], sum = 0, total;
        const int b0 = kBins - (kBins / kSelectThreads) * (tid + 1);
#pragma unroll
        for (int x = 0; x < kBins / kSelectThreads; ++x) {
            mine[x] = s.hist[b0 + x];
            sum += mine[x];
        }
        uint32_t before = up + block_exclusive(s, sum, total);
        if (before < k && before + sum >= k) {  // one thread: the k-th is in one of its bins
#pragma unroll
            for (int x = kBins / kSelectThreads - 1; x >= 0; --x) {
                if (before < k && before + mine[x] >= k) {
                    const unsigned long long from = (unsigned long long)lo + ((unsigned long long)(b0 + x) << shift);
                    s.lo = from;
                    s.hi = min((unsigned long long)hi, from + min((1ull << shift) - 1, ~from));  // no wrap at the top
                    s.above = before;
                }
                before += mine[x];
            }
        }
        __syncthreads();
        lo = (Key)s.lo;
        hi = (Key)s.hi;
        up = s.above;
        __syncthreads();
    }
    above = up;
    return lo;
}

// The sum over h of max(q lo, q hi) in 64 bits, the largest over the group's heads (products of two bf16
// numbers are exact in 32 bits), by one warp: every lane's order and the shuffles' are the same for
// every block, so equal blocks get equal sums.
template <int H>
__device__ __forceinline__ double exact_score(const SelectParams &p, int b, int kvh, int j, int lane)
{
    const int blk = __ldg(p.block_tables + (size_t)b * p.max_nb + j);
    if (blk < 0 || blk >= p.num_blocks) return -__longlong_as_double(0x7FF0000000000000ll);
    const uint16_t *lo = p.bounds + ((int64_t)blk * p.K + kvh) * 2 * H, *hi = lo + H;
    const uint16_t *q = p.q + ((size_t)b * p.N + (size_t)kvh * p.G) * H;
    double best = -__longlong_as_double(0x7FF0000000000000ll);
    bool nan = false;
    for (int g = 0; g < p.G; ++g) {
        double sum = 0.0;
        for (int h = lane; h < H; h += 32) {
            const float x = bf16_to_f32(q[g * H + h]);
            const float y = bf16_to_f32(x > 0.f ? hi[h] : lo[h]);
            sum += (double)(x * y);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        nan |= sum != sum;
        best = sum > best ? sum : best;
    }
    return nan ? __longlong_as_double(0x7FF8000000000000ll) : best;
}

// Writes the blocks j in [0, nb) with take(j) to dst in ascending order (at most `most`).  Each warp
// counts, then writes, a contiguous run of blocks; take is called twice for each j.
template <typename Take>
__device__ __forceinline__ uint32_t compact(SelectShared &s, int nb, Take take, int32_t *dst, uint32_t most)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = ((nb + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int begin = min(nb, warp * per), end = min(nb, begin + per);
    uint32_t n = 0;
    for (int j0 = begin; j0 < end; j0 += 32)
        n += __popc(__ballot_sync(0xFFFFFFFFu, j0 + lane < end && take(j0 + lane)));
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = n;
    __syncthreads();
    uint32_t at = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kSelectWarps; ++w) {
        at += w < warp ? s.warp_sum[w] : 0u;
        total += s.warp_sum[w];
    }
    for (int j0 = begin; j0 < end; j0 += 32) {
        const bool in = j0 + lane < end && take(j0 + lane);
        const unsigned m = __ballot_sync(0xFFFFFFFFu, in);
        const uint32_t o = at + __popc(m & ((1u << lane) - 1u));
        if (in && o < most) dst[o] = j0 + lane;
        at += __popc(m);
    }
    return min(total, most);
}

// The last CTA of a (sequence, KV head) chooses, from the scores that the chunks left.
template <int H>
__device__ __forceinline__ void choose(SelectShared &s, const SelectParams &p, int b, int kvh, int nb, int chunks)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t unit = (size_t)b * p.K + kvh;
    float *scores = p.scores + unit * p.max_nb;
    int32_t *sel = p.selected + unit * p.M;
    const int first = p.first, n = nb - p.first - p.last;  // candidates: blocks first .. first + n - 1
    const uint32_t k = (uint32_t)(p.M - p.first - p.last);  // 0 <= k < n

    // eps: 2^-14 |q|_1 max|bound|.  A product of depth 2H = 256 is 16 mma of 16 products each.  Each product is at
    // most its part of S = |q|_1 max|bound|, no partial sum exceeds S, and an mma that keeps 23 bits below its
    // largest term loses at most 2^-23 S for each of its 17 terms and once more at its end: 16 * 18 * 2^-23 S,
    // and as much again for slack in what the documentation leaves open about the sum's rounding.
    if (k > 0) {
        float q1 = 0.f, mb = 0.f;
        for (int g = warp; g < p.G; g += kSelectWarps) {
            float x = 0.f;
            for (int h = lane; h < H; h += 32) x += fabsf(bf16_to_f32(p.q[((size_t)b * p.N + (size_t)kvh * p.G + g) * H + h]));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
            q1 = fmaxf(q1, x);
        }
        for (int c = tid; c < chunks; c += kSelectThreads) mb = fmaxf(mb, __ldcg(p.chunk_max + unit * p.chunks + c));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, off));
        if (tid == 0) s.q1 = 0.f, s.eps = 0.f;
        __syncthreads();
        if (lane == 0) {  // non-negative floats order like their bits
            atomicMax(reinterpret_cast<int *>(&s.q1), __float_as_int(q1));
            atomicMax(reinterpret_cast<int *>(&s.eps), __float_as_int(mb));
        }
        __syncthreads();
        const float eps2 = 2.f * ldexpf(s.q1 * s.eps, -14);
        auto key = [&](int i) { return order_key(__ldcg(scores + first + i)); };
        uint32_t above;
        const uint32_t kt = kth_largest<uint32_t>(s, n, k, key, above);
        const float t = __uint_as_float(kt & 0x80000000u ? kt & 0x7FFFFFFFu : ~kt);
        // bounds of the undecided scores, rounded outwards; both ends at t where eps2 is no number
        const uint32_t kin = eps2 == eps2 ? max(kt, order_key(__fadd_ru(t, eps2))) : ~0u;
        const uint32_t kout = eps2 == eps2 ? min(kt, order_key(__fadd_rd(t, -eps2))) : 0u;
        auto score_key = [&](int j) { return order_key(__ldcg(scores + j)); };
        auto middle = [&](int j) { return j >= first && j < first + n; };
        uint32_t n_in = 0, n_amb = 0;
        for (int i = tid; i < n; i += kSelectThreads) {
            const uint32_t x = key(i);
            n_in += x > kin;
            n_amb += x <= kin && x >= kout;
        }
        uint32_t sum_in, sum_amb;
        block_exclusive(s, n_in, sum_in);
        block_exclusive(s, n_amb, sum_amb);
        const uint32_t need = k - sum_in;
        if (sum_amb > need) {
            // more undecided blocks than places: rank them by their sums in 64 bits
            int32_t *list = p.list + unit * p.max_nb;
            compact(s, nb, [&](int j) { return middle(j) && score_key(j) <= kin && score_key(j) >= kout; }, list, sum_amb);
            __syncthreads();
            const int m = (int)sum_amb;
            double *exact = m <= kRankMost ? s.exact : p.exact + unit * p.max_nb;
            for (int a = warp; a < m; a += kSelectWarps) {
                const double x = exact_score<H>(p, b, kvh, list[a], lane);
                if (lane == 0) exact[a] = x;
            }
            __syncthreads();
            if (m <= kRankMost) {
                for (int a = tid; a < m; a += kSelectThreads) {
                    const unsigned long long x = order_key(exact[a]);
                    uint32_t rank = 0;  // the list ascends, so among equals the earlier one goes first
                    for (int o = 0; o < m; ++o) {
                        const unsigned long long y = order_key(exact[o]);
                        rank += y > x || (y == x && o < a);
                    }
                    scores[list[a]] = rank < need ? INFINITY : -INFINITY;
                }
            } else {
                uint32_t over;
                const unsigned long long xt = kth_largest<unsigned long long>(s, m, need, [&](int a) { return order_key(exact[a]); }, over);
                // of the sums equal to the need-th one, the first need - over in the list
                uint32_t ties = need - over, run = 0;
                for (int a0 = 0; a0 < m; a0 += kSelectThreads) {
                    const int a = a0 + tid;
                    const unsigned long long x = a < m ? order_key(exact[a]) : 0ull;
                    const bool tie = a < m && x == xt;
                    uint32_t total;
                    const uint32_t before = run + block_exclusive(s, tie ? 1u : 0u, total);
                    run += total;
                    if (a < m) scores[list[a]] = x > xt || (tie && before < ties) ? INFINITY : -INFINITY;
                }
            }
            __syncthreads();
            // decided: above the band, or raised to +inf
            compact(s, nb, [&](int j) { return !middle(j) || score_key(j) > kin || __ldcg(scores + j) == INFINITY; }, sel, (uint32_t)p.M);
        } else {
            compact(s, nb, [&](int j) { return !middle(j) || score_key(j) >= kout; }, sel, (uint32_t)p.M);
        }
    } else {
        compact(s, nb, [&](int j) { return j < first || j >= first + n; }, sel, (uint32_t)p.M);
    }
}

// Grid (chunks, K, B): 128 blocks of a (sequence, KV head) a CTA, 16 a warp, whose bounds (4 H bytes a block)
// the warp loads straight into mma fragments -- the product's depth may be taken in any order, so a
// lane's 16-byte vectors are its k indices -- with all its loads (8 KB at H = 128) in flight at once.
template <int H>
__global__ void __launch_bounds__(kSelectThreads, 2) select_blocks_kernel(const SelectParams p)
{
    constexpr int V = H / 32;  // 16-byte vectors a lane holds of a row
    __shared__ SelectShared s;
    const int chunk = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int ctx = p.context_lens[b];
    if (ctx < 0 || ctx > p.max_nb * kBlockSize) {
        if (tid == 0 && kvh == 0 && chunk == 0) set_flag(p.err_flag, PKV_FLAG_CTX_RANGE);
        ctx = 0;
    }
    const int nb = (ctx + kBlockSize - 1) / kBlockSize;
    const size_t unit = (size_t)b * p.K + kvh;
    if (nb <= p.M) {  // every block is selected: no scores needed
        if (chunk == 0)
            for (int x = tid; x < p.M; x += kSelectThreads) p.selected[unit * p.M + x] = x < nb ? x : -1;
        return;
    }
    const int chunks = (nb + kSelectChunk - 1) / kSelectChunk;
    if (chunk >= chunks) return;

    const int r = lane >> 2, m = lane & 3;
    const int j0 = chunk * kSelectChunk + warp * 16 + r;
    const uint16_t *row[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int j = j0 + 8 * x;
        row[x] = nullptr;
        if (j >= p.first && j < nb - p.last) {  // the others are selected without a score
            const int blk = __ldg(p.block_tables + (size_t)b * p.max_nb + j);
            if (blk >= 0 && blk < p.num_blocks) row[x] = p.bounds + ((int64_t)blk * p.K + kvh) * 2 * H + 8 * m;
            else if (m == 0) set_flag(p.err_flag, PKV_FLAG_BLOCK_RANGE);
        }
    }
    uint4 av[2][2][V];  // [row][lo, hi][vector]
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < V; ++i)
                av[x][e][i] = row[x] ? __ldg(reinterpret_cast<const uint4 *>(row[x] + e * H + 32 * i)) : make_uint4(0u, 0u, 0u, 0u);
    const bool live = r < p.G;
    const uint16_t *qrow = p.q + ((size_t)b * p.N + (size_t)kvh * p.G + (live ? r : 0)) * H + 8 * m;
    uint4 qv[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        qv[i] = live ? __ldg(reinterpret_cast<const uint4 *>(qrow + 32 * i)) : make_uint4(0u, 0u, 0u, 0u);

    float c[2][4] = {};
    uint32_t big = 0u;  // packed max |bound|
    const uint32_t zero = 0u;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t qw[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
            uint32_t bq[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) bq[w] = e ? max_bf16x2(qw[w], zero) : min_bf16x2(qw[w], zero);
            const uint4 x = av[0][e][i], y = av[1][e][i];
            const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
            mma_bf16_16816(c[0], a0, bq[0], bq[1]);
            mma_bf16_16816(c[1], a1, bq[2], bq[3]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                big = max_bf16x2(big, a0[w] & 0x7FFF7FFFu);
                big = max_bf16x2(big, a1[w] & 0x7FFF7FFFu);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        // this lane's columns are heads 2m and 2m + 1
        const float s0 = c[0][2 * x] + c[1][2 * x], s1 = c[0][2 * x + 1] + c[1][2 * x + 1];
        float best = -INFINITY;
        bool nan = false;
        if (2 * m < p.G) best = s0, nan = s0 != s0;
        if (2 * m + 1 < p.G) best = fmaxf(best, s1), nan |= s1 != s1;
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, off));
        const unsigned nans = __ballot_sync(0xFFFFFFFFu, nan);
        const int j = j0 + 8 * x;
        if (m == 0 && j < nb)
            p.scores[unit * p.max_nb + j] = (nans >> (lane & ~3)) & 15u ? __int_as_float(0x7FC00000) : (row[x] ? best : -INFINITY);
    }
    float mb = fmaxf(bf16x2_lo(big), bf16x2_hi(big));
    const bool mb_nan = bf16x2_lo(big) != bf16x2_lo(big) || bf16x2_hi(big) != bf16x2_hi(big);
    if (mb_nan) mb = INFINITY;  // no bound on the error: every score is looked at in 64 bits
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, off));
    if (lane == 0) s.warp_sum[warp] = __float_as_uint(mb);
    __syncthreads();  // every score of this CTA is written
    if (tid == 0) {
        uint32_t top = 0u;
        for (int w = 0; w < kSelectWarps; ++w) top = max(top, s.warp_sum[w]);
        p.chunk_max[unit * p.chunks + chunk] = __uint_as_float(top);
        s.last_one = atomic_add_acq_rel_gpu(p.counters + unit, 1) == chunks - 1;
    }
    __syncthreads();
    if (!s.last_one) return;
    choose<H>(s, p, b, kvh, nb, chunks);
    if (tid == 0) p.counters[unit] = 0;  // ready for the next call
}

cudaError_t launch_select_blocks(const SelectParams &p, int H, cudaStream_t stream)
{
    const dim3 grid(p.chunks, p.K, p.B);
    if (H == 128) select_blocks_kernel<128><<<grid, kSelectThreads, 0, stream>>>(p);
    else select_blocks_kernel<64><<<grid, kSelectThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
