// pkv_verify.cu - verification of drafted tokens against the target model's probabilities, the random
// numbers given (speculative sampling).
//
// Drafted token x_t (t < gamma) stands while u_t q_t(x_t) < p_t(x_t), that is with probability min(1, p / q) for a
// uniform u_t.  At the first refusal the token is drawn from the residual max(p_t - q_t, 0), after gamma
// acceptances from p_gamma, by inversion: the first i whose running sum exceeds r times the total.  A draft
// without probabilities (q null) is one-hot at its token.
//
// Exact sums.  Which token a draw falls on is decided where two running sums over a vocabulary of 10^5
// entries differ by 10^-5 or less, and 32-bit sums, whose order depends on the split, would move those borders.
// So every weight is split into a multiple of 2^-22 and a multiple of 2^-44 of what is left (the difference
// p - q with its rounding error first), each summed exactly, as integers.  The sums do not depend on the order, and a
// weight is off by little more than 2^-45.  Where a row's weights add up to less than 2^-8 that may be much of them: the
// sequence's last CTA then scales the largest weight to [1/2, 1), sums the row once more and draws from that (draw_small).
//
// Bound by memory: one row of p, and where a token was refused one row of q.  A row is cut into one run of entries
// per warp, runs of at least 256 entries; the acceptance is decided by every CTA for itself (a few loads against a second
// launch).  A few sequences take one cluster each, whose first CTA reads the runs' sums in the others' shared memory; many
// take as many CTAs as are about four per SM over the whole batch (1,024 runs a row at most), and the last CTA of a
// sequence to finish takes the sums from the workspace.  It adds them up, finds the run that the draw falls into and the
// entry in it.
//
// Measured: one sequence (three drafted tokens, 32,000 bf16 entries) 5.7 us (5.6 to 5.8), a chain of dependent loads (length, token,
// probability, row, sums, entry); 64 sequences (four drafted tokens, 128,256 fp32 entries) 15.7 us, that chain around one
// pass over 55 MB in about 8 us.
#include "pkv_cluster.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_ops.h"

namespace pkv {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyRuns = 1024;  // runs of a row at most
constexpr int kClusterCtas = 16;   // of a cluster at most
constexpr int kClusterShare = 16384;  // entries of one of its CTAs at most

__device__ __forceinline__ float prob_at(const float *row, int64_t i) { return __ldg(row + i); }
__device__ __forceinline__ float prob_at(const uint16_t *row, int64_t i) { return bf16_to_f32(__ldg(row + i)); }

// Probabilities are numbers in [0, 1]: NaN and what is below count as 0, what is above as 1.
__device__ __forceinline__ float clean(float x) { return __saturatef(x); }

// Sums of weights max(p - q, 0) in two parts, multiples of 2^-22 and of 2^-44.  Adding 3 (1.5 * 2^-21) to a number below
// 1 (2^-22) rounds it to the last place there, 2^-22 (2^-44), and the sum's bit pattern counts those units: the patterns
// are added up as integers, the constants' taken off at the end.  Exact up to 256 weights (2^22 units each at most).
struct WeightSum {
    static constexpr float kA = 3.f, kB = 3.f / 4194304.f;
    unsigned a = 0, b = 0;
    // p cleaned; q only has to be cleaned from below: min(p, q) takes off what lies above p
    __device__ __forceinline__ void add(float p, float q) { add(p, q, [](float x) { return x; }); }
    template <typename Scale>
    __device__ __forceinline__ void add(float p, float q, Scale scale)
    {
        const float m = fminf(p, q);
        float d = __fsub_rn(p, m), e = __fsub_rn(__fsub_rn(p, d), m);  // p - m = d + e exactly (p >= m >= 0)
        d = scale(d), e = scale(e);
        const float ta = __fadd_rn(d, kA);
        const float r = __fadd_rn(__fsub_rn(d, __fsub_rn(ta, kA)), e);
        a += __float_as_uint(ta);
        b += __float_as_uint(__fadd_rn(r, kB));
    }
    // in units of 2^-44, after n additions (the counts wrap around and back)
    __device__ __forceinline__ long long units(int n) const
    {
        const int ua = (int)(a - n * __float_as_uint(kA));
        const int ub = (int)(b - n * __float_as_uint(kB));
        return ((long long)ua << 22) + ub;
    }
};

template <typename T>
struct VerifyRow {  // the row that a sequence's next token is drawn from
    const T *p, *q;  // q null: p alone
    int hot;         // one-hot draft refused: its token (else -1)
    int accepted, len;
    int token;       // lane t: drafted token t (t < 32)
};

// The acceptance of sequence b's drafted tokens.  Every CTA decides it for itself (gamma loads of each kind).
template <typename T>
__device__ __forceinline__ VerifyRow<T> decide(const VerifyParams &p, int b, bool report)
{
    const int lane = threadIdx.x & 31;
    // the first tokens and numbers do not depend on the draft's length: their loads go together with its
    int x_first = -1;
    float u_first = 0.f;
    if (lane < p.T) {
        x_first = p.tokens[(int64_t)b * p.T + lane];
        u_first = p.accept_u[(int64_t)b * p.T + lane];
    }
    int len = p.lens ? p.lens[b] : p.T;
    if (len < 0 || len > p.T) {
        if (report) set_flag(p.err_flag, PKV_FLAG_TOKEN_RANGE);
        len = min(max(len, 0), p.T);
    }
    const T *target = static_cast<const T *>(p.target) + (int64_t)b * (p.T + 1) * p.target_stride;
    const T *draft = p.draft ? static_cast<const T *>(p.draft) + (int64_t)b * p.T * p.draft_stride : nullptr;
    // lane t looks at token t (a warp's worth at a time): the first refusal of the warp's
    int n = len, hot = -1;
    for (int t0 = 0; t0 < len; t0 += 32) {
        const int t = t0 + lane;
        bool refuse = false;
        int x = -1;
        if (t < len) {
            x = t0 ? p.tokens[(int64_t)b * p.T + t] : x_first;
            const float u = t0 ? p.accept_u[(int64_t)b * p.T + t] : u_first;
            refuse = true;
            if (x < 0 || x >= p.V) {
                if (report) set_flag(p.err_flag, PKV_FLAG_TOKEN_RANGE);
            } else {
                const float pt = clean(prob_at(target + (int64_t)t * p.target_stride, x));
                const float qt = draft ? clean(prob_at(draft + (int64_t)t * p.draft_stride, x)) : 1.f;
                refuse = !((double)u * (double)qt < (double)pt);  // products of 24-bit numbers are exact in 64 bits
            }
        }
        const unsigned m = __ballot_sync(0xFFFFFFFFu, refuse);
        if (m) {
            const int at = __ffs(m) - 1;
            n = t0 + at;
            hot = __shfl_sync(0xFFFFFFFFu, x, at);
            break;
        }
    }
    VerifyRow<T> row;
    row.accepted = n;
    row.len = len;
    row.token = x_first;
    row.p = target + (int64_t)n * p.target_stride;
    row.q = draft && n < len ? draft + (int64_t)n * p.draft_stride : nullptr;
    row.hot = !draft && n < len ? hot : -1;
    return row;
}

// Two 16-byte vectors of each row that a thread holds: as loaded, so that the next ones can be on their way while
// these are summed.
template <typename T>
struct Pairs {
    static constexpr int E = 16 / sizeof(T), kEntries = 2 * E;
    uint4 p[2], q[2];

    __device__ static __forceinline__ float entry(const uint4 (&v)[2], int k)
    {
        const uint4 x = v[k / E];
        if constexpr (sizeof(T) == 4) {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            return __uint_as_float(w[k % E]);
        } else {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            return k & 1 ? bf16x2_hi(w[(k % E) / 2]) : bf16x2_lo(w[(k % E) / 2]);
        }
    }
    // kVec: vector k holds the entries from i0 + k * step on, and the rows start on 16 bytes; the part of a vector
    // behind `end` is left at zero.  Otherwise entry k of the thread is i0 + k * step (rows of an odd vocabulary
    // start anywhere: with step 32 and lanes next to each other a warp's loads are contiguous all the same).
    template <bool kVec>
    __device__ __forceinline__ void load(const VerifyRow<T> &row, int64_t i0, int step, int64_t end)
    {
        auto fetch = [&](const T *src, uint4 (&v)[2]) {
            if constexpr (kVec) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t i = i0 + k * (int64_t)step;
                    v[k] = i + E <= end ? __ldg(reinterpret_cast<const uint4 *>(src + i)) : make_uint4(0u, 0u, 0u, 0u);
                    if (i < end && i + E > end) v[k] = cut(src, i, 1, end);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) v[k] = cut(src, i0 + k * E * (int64_t)step, step, end);
            }
        };
        fetch(row.p, p);
        if (row.q) fetch(row.q, q);
        else q[0] = q[1] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ static __forceinline__ uint4 cut(const T *src, int64_t i, int step, int64_t end)
    {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (i + e * (int64_t)step < end) {
                if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(__ldg(src + i + e * (int64_t)step));
                else w[e / 2] |= (uint32_t)__ldg(src + i + e * (int64_t)step) << (16 * (e & 1));
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __forceinline__ float at_least_0(float x) { return fmaxf(x, 0.f); }  // NaN: 0
    // units of 2^-44 of all entries; a one-hot draft's token is entry `hot` of this thread's (-1: elsewhere)
    __device__ __forceinline__ long long units(int hot) const
    {
        WeightSum w;
        if (hot < 0) {
#pragma unroll
            for (int k = 0; k < kEntries; ++k) w.add(clean(entry(p, k)), at_least_0(entry(q, k)));
        } else {
#pragma unroll
            for (int k = 0; k < kEntries; ++k) w.add(clean(entry(p, k)), k == hot ? 1.f : 0.f);
        }
        return w.units(kEntries);
    }
};

// Which of the entries i0 + k of a thread (consecutive ones), or with vectors `step` apart, is the row's hot token.
template <typename T>
__device__ __forceinline__ int hot_entry(const VerifyRow<T> &row, int64_t i0, int step, bool vec)
{
    constexpr int E = Pairs<T>::E;
    if (row.hot < 0) return -1;
    const int64_t d = row.hot - i0;
    if (d < 0) return -1;
    if (!vec) return d % step == 0 && d / step < 2 * E ? (int)(d / step) : -1;
    const int64_t k = d / step;
    return k < 2 && d - k * step < E ? (int)(k * E + d - k * step) : -1;
}

// The sum of this warp's run of entries [begin, end), on every lane.
template <typename T, bool kVec>
__device__ __forceinline__ long long run_sum_t(const VerifyRow<T> &row, int64_t begin, int64_t end)
{
    constexpr int E = Pairs<T>::E, kStride = 64 * E;  // entries of a warp's round
    const int lane = threadIdx.x & 31;
    const int64_t off = kVec ? lane * E : lane;
    const int step = kVec ? 32 * E : 32;
    long long sum = 0;
    Pairs<T> next;
    next.template load<kVec>(row, begin + off, step, end);
    for (int64_t i = begin; i < end; i += kStride) {
        const Pairs<T> now = next;
        if (i + kStride < end) next.template load<kVec>(row, i + kStride + off, step, end);
        sum += now.units(hot_entry(row, i + off, step, kVec));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    return sum;
}

template <typename T>
__device__ __forceinline__ long long run_sum(const VerifyRow<T> &row, int64_t begin, int64_t end)
{
    const bool even = (reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) % 16 == 0;
    return even ? run_sum_t<T, true>(row, begin, end) : run_sum_t<T, false>(row, begin, end);
}

__device__ __forceinline__ long long warp_inclusive(long long v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

// The run that a draw falls into, from the runs' sums in shared memory, for every warp by itself (no barriers).
struct Place {
    long long total, bar;  // the row's weights; the draw falls on the first entry whose running sum exceeds bar
    long long base;        // sum of the runs before this one
    int run;
};

// least: no place is looked for where the total is below it (1 at least).
__device__ __forceinline__ Place find_run(const long long *sums, int runs, float sample, long long least)
{
    const int lane = threadIdx.x & 31;
    // lane's share: per consecutive runs
    const int per = (runs + 31) / 32;
    long long mine = 0;
    for (int x = lane * per; x < min(runs, (lane + 1) * per); ++x) mine += sums[x];
    const long long upto = warp_inclusive(mine);
    Place at{__shfl_sync(0xFFFFFFFFu, upto, 31), 0, 0, 0};
    if (at.total < least) return at;
    // the running sum has to exceed r * total, r < 1, so the last entry with weight always does; running sums are whole
    // numbers, so they exceed it where they exceed its floor (below 2^53 units, as those of probabilities are, exact)
    at.bar = (long long)floor(fmin(fmax((double)sample, 0.0), 1.0 - 0x1p-53) * (double)at.total);
    const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, upto > at.bar)) - 1;
    at.base = __shfl_sync(0xFFFFFFFFu, upto - mine, owner);
    at.run = owner * per;
    for (; at.base + sums[at.run] <= at.bar; ++at.run) at.base += sums[at.run];
    return at;
}

// Rows whose weights add up to less than 2^-8, where units of 2^-44 are too coarse (they lose a small weight, or all of
// them): the weights are scaled by a power of two that takes the largest to [1/2, 1) and summed again, run by run into sums
// and then entry by entry.  All threads call it; -1 where no entry has any weight.  A draw meets such a row about as often
// as its mass says, so the kernel's registers come first: a call of its own, one entry a thread at a time (a row of 128,256
// fp32 entries 157 us, 64 of them 215; 32,000 30 us).
template <typename T>
__device__ __noinline__ int draw_small(const VerifyRow<T> &row, const VerifyParams &p, int runs, float sample, long long *sums,
                                       long long *warp_sums, int *found)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto prob = [&](int64_t i) { return clean(prob_at(row.p, i)); };
    auto other = [&](int64_t i) { return row.q ? fmaxf(prob_at(row.q, i), 0.f) : (i == row.hot ? 1.f : 0.f); };
    float top = 0.f;
    for (int64_t i = tid; i < p.V; i += kVerifyThreads) {
        const float x = prob(i);
        top = fmaxf(top, __fsub_rn(x, fminf(x, other(i))));
    }
    const unsigned bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));  // non-negative numbers order like their bits
    __syncthreads();
    if (lane == 0) warp_sums[warp] = bits;
    __syncthreads();
    unsigned most = 0;
#pragma unroll
    for (int w = 0; w < kVerifyWarps; ++w) most = max(most, (unsigned)warp_sums[w]);
    if (most == 0) return -1;
    // 2^up takes the largest weight, 2^-149 at least, to [1/2, 1); in two factors, for it may be 2^148
    const int up = (most >> 23 ? 126 - (int)(most >> 23) : 117 + __clz((int)most));
    const float f0 = __uint_as_float((unsigned)(127 + min(up, 100)) << 23), f1 = __uint_as_float((unsigned)(127 + up - min(up, 100)) << 23);
    auto weight = [&](int64_t i, int64_t end) -> long long {
        if (i >= end) return 0;
        WeightSum one;
        one.add(prob(i), other(i), [&](float x) { return __fmul_rn(__fmul_rn(x, f0), f1); });
        return one.units(1);
    };
    for (int x = warp; x < runs; x += kVerifyWarps) {
        const int64_t begin = (int64_t)x * p.run, end = min((int64_t)p.V, begin + p.run);
        long long sum = 0;
        for (int64_t i = begin; i < end; i += 32) sum += weight(i + lane, end);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) sums[x] = sum;
    }
    __syncthreads();
    Place at = find_run(sums, runs, sample, 1);
    const int64_t begin = (int64_t)at.run * p.run, end = min((int64_t)p.V, begin + p.run);
    for (int64_t i0 = begin; i0 < end; i0 += kVerifyThreads) {
        const long long w = weight(i0 + tid, end), inc = warp_inclusive(w);
        if (lane == 31) warp_sums[warp] = inc;
        if (tid == 0) *found = -1;
        __syncthreads();
        long long after = at.base + inc, all = 0;
#pragma unroll
        for (int y = 0; y < kVerifyWarps; ++y) {
            after += y < warp ? warp_sums[y] : 0;
            all += warp_sums[y];
        }
        if (after > at.bar && after - w <= at.bar) *found = (int)(i0 + tid);  // one thread
        __syncthreads();
        const int token = *found;
        __syncthreads();
        if (token >= 0) return token;
        at.base += all;
    }
    return -1;
}

// A sequence's last CTA: the token drawn from the row, -1 where the row has no mass.  sums: the runs' sums in shared
// memory; all threads look together for the entry in the run.
template <typename T>
__device__ __forceinline__ int draw(const VerifyRow<T> &row, const VerifyParams &p, int runs, float sample, long long *sums,
                                    long long *warp_sums, int *found)
{
    constexpr int kMine = Pairs<T>::kEntries;
    constexpr long long kSmall = 1ll << 36;  // 2^-8
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place at_run = find_run(sums, runs, sample, kSmall);
    if (at_run.total < kSmall) return draw_small(row, p, runs, sample, sums, warp_sums, found);
    const long long bar = at_run.bar;
    long long base = at_run.base;
    const int run = at_run.run;
    // entries of the run, consecutive ones for each thread
    const int64_t begin = (int64_t)run * p.run, end = min((int64_t)p.V, begin + p.run);
    for (int64_t i0 = begin; i0 < end; i0 += kMine * kVerifyThreads) {
        const int each = (int)min((int64_t)kMine, (end - i0 + kVerifyThreads - 1) / kVerifyThreads);
        const int64_t i = i0 + (int64_t)tid * each, stop = min(end, i + each);
        Pairs<T> x;
        x.template load<false>(row, i, 1, stop);
        const int hot = hot_entry(row, i, 1, false);
        const long long w = x.units(hot < each ? hot : -1), inc = warp_inclusive(w);
        if (lane == 31) warp_sums[warp] = inc;
        if (tid == 0) *found = -1;
        __syncthreads();
        long long after = base + inc, all = 0;
#pragma unroll
        for (int y = 0; y < kVerifyWarps; ++y) {
            after += y < warp ? warp_sums[y] : 0;
            all += warp_sums[y];
        }
        if (after > bar && after - w <= bar) {  // one thread: its entries one by one
            long long at = after - w;
            int hit = -1;
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
                WeightSum one;
                one.add(clean(x.entry(x.p, k)), k == hot ? 1.f : x.at_least_0(x.entry(x.q, k)));
                at += one.units(1);
                if (hit < 0 && at > bar) hit = (int)(i + k);
            }
            *found = hit;
        }
        __syncthreads();
        const int token = *found;
        __syncthreads();
        if (token >= 0) return token;
        base += all;
    }
    return -1;
}

template <typename T, bool kCluster>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p)
{
    __shared__ long long all_sums[kCluster ? kClusterCtas * kVerifyWarps : kVerifyRuns];
    __shared__ long long my_sums[kVerifyWarps];
    __shared__ long long warp_sums[kVerifyWarps];
    __shared__ int found, last_one;
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    pdl_wait_primary();
    pdl_launch_dependents();
    VerifyRow<T> row = decide<T>(p, b, c == 0 && tid < 32);
    // what the last CTA needs besides the sums: loaded before it is known to be the last
    const float sample = p.sample_u[b];
    const int ctx = p.context_lens ? p.context_lens[b] : 0;
    const int runs = (p.V + p.run - 1) / p.run;
    long long *sums = p.sums + (int64_t)b * runs;
    const int r = c * kVerifyWarps + (tid >> 5);  // this warp's run
    long long mine = 0;
    if (r < runs) mine = run_sum(row, (int64_t)r * p.run, min((int64_t)p.V, (int64_t)(r + 1) * p.run));
    if constexpr (kCluster) {
        // a sequence's CTAs are one cluster: the first draws, and reads the others' sums where they are
        if ((tid & 31) == 0) my_sums[tid >> 5] = mine;
        cluster_sync();
        if (c == 0 && tid < runs) all_sums[tid] = load_cluster<long long>(smem_u32(my_sums + tid % kVerifyWarps), tid / kVerifyWarps);
        cluster_arrive();  // the others may leave
        if (c != 0) {
            cluster_wait();
            return;
        }
    } else {
        if ((tid & 31) == 0 && r < runs) sums[r] = mine;
        __syncthreads();
        if (tid == 0) last_one = atomic_add_acq_rel_gpu(p.counters + b, 1) == (int)gridDim.x - 1;
        __syncthreads();
        if (!last_one) return;
        for (int x = tid; x < runs; x += kVerifyThreads) all_sums[x] = __ldcg(sums + x);
    }
    __syncthreads();
    int token = draw(row, p, runs, sample, all_sums, warp_sums, &found);
    if (token < 0 && (row.q || row.hot >= 0)) {
        // no residual mass (p nowhere above q): the token is drawn from p itself
        row.q = nullptr;
        row.hot = -1;
        __syncthreads();
        for (int x = tid >> 5; x < runs; x += kVerifyWarps) {
            const long long v = run_sum(row, (int64_t)x * p.run, min((int64_t)p.V, (int64_t)(x + 1) * p.run));
            if ((tid & 31) == 0) all_sums[x] = v;
        }
        __syncthreads();
        token = draw(row, p, runs, sample, all_sums, warp_sums, &found);
    }
    if (token < 0 && tid == 0) set_flag(p.err_flag, PKV_FLAG_NO_MASS);
    const int n = row.accepted;
    for (int t = tid; t <= p.T; t += kVerifyThreads) {
        int x = token;
        if (t < n) x = t < 32 ? row.token : p.tokens[(int64_t)b * p.T + t];
        p.out[(int64_t)b * (p.T + 1) + t] = t <= n ? x : -1;
    }
    if (tid == 0) {
        p.accepted[b] = n;
        if (p.context_lens) p.context_lens_out[b] = ctx - row.len + n;
        if constexpr (!kCluster) p.counters[b] = 0;  // ready for the next call
    }
    if constexpr (kCluster) {
        __syncwarp();
        cluster_wait();
    }
}

cudaError_t launch_verify(VerifyParams p, bool bf16, int sms, cudaStream_t stream)
{
    // runs of at least kVerifyRun entries, at most kVerifyRuns of them, CTAs enough for about four per SM
    const int most = (p.V + kVerifyRun * kVerifyWarps - 1) / (kVerifyRun * kVerifyWarps);
    const int want = (4 * sms + p.B - 1) / p.B;
    int ctas = want < most ? want : most;
    if (ctas > kVerifyRuns / kVerifyWarps) ctas = kVerifyRuns / kVerifyWarps;
    // A cluster per sequence where that is one CTA per SM at most and 16,384 entries a CTA: 1 sequence of 128,256 entries 5.9 us,
    // through the workspace (63 CTAs) 7.5; 4: 6.3 and 9.1; 16: 8.6 and 9.4; 64 of 32,000: 7.9 and 9.5; but 32 of 128,256, 4
    // CTAs each, 15.4 and 11.1, 64, 2 CTAs each, 30.6 and 15.8.
    const int cap = sms / p.B < kClusterCtas ? sms / p.B : kClusterCtas;
    const bool clusters = cap > 0 && (p.V + cap - 1) / cap <= kClusterShare;
    if (clusters && ctas > cap) ctas = cap;
    const int per = (p.V + ctas * kVerifyWarps - 1) / (ctas * kVerifyWarps);
    p.run = (per + kVerifyRun - 1) / kVerifyRun * kVerifyRun;
    const int runs = (p.V + p.run - 1) / p.run;
    const dim3 grid((runs + kVerifyWarps - 1) / kVerifyWarps, p.B), one(1, 1, 1);
    if (clusters || grid.x == 1) {
        static bool ready[64] = {};  // per device
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!ready[dev]) {
            e = allow_wide_clusters(verify_kernel<uint16_t, true>);
            if (e == cudaSuccess) e = allow_wide_clusters(verify_kernel<float, true>);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
        return launch_clusters(bf16 ? verify_kernel<uint16_t, true> : verify_kernel<float, true>, grid, dim3(kVerifyThreads),
                               dim3(grid.x, 1, 1), 0, stream, p);
    }
    return launch_clusters(bf16 ? verify_kernel<uint16_t, false> : verify_kernel<float, false>, grid, dim3(kVerifyThreads), one, 0, stream, p);
}

}  // namespace pkv
