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
// p - q with its rounding error first), each summed exactly: four at a time in 32 bits, then as 64-bit integers
// in units of 2^-44.  The sums do not depend on the order, and a weight is off by little more than 2^-45.
//
// Bound by memory: one row of p, and where a token was refused one row of q.  A CTA sums a chunk of 4,096
// entries (whatever CTAs a sequence has, the rows are spread over the SMs); the last chunk to finish adds the
// chunks' sums up, finds the chunk that the draw falls into and then the entry in it.
#include "pkv_device.cuh"
#include "pkv_ops.h"

namespace pkv {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kPerThread = kVerifyChunk / kVerifyThreads;
static_assert(kPerThread == 16, "a thread's entries are four groups of four");

__device__ __forceinline__ float prob_at(const float *row, int64_t i) { return __ldg(row + i); }
__device__ __forceinline__ float prob_at(const uint16_t *row, int64_t i) { return bf16_to_f32(__ldg(row + i)); }

// Probabilities are numbers in [0, 1]: NaN and what is below count as 0, what is above as 1.
__device__ __forceinline__ float clean(float x) { return __saturatef(x); }

// Up to four weights, summed in their two parts, which fit the 24 bits of a float: a weight is at most 2^22
// units of 2^-22, and what is left of it at most 2^-23 + 2^-25, below 2^22 units of 2^-44.
struct WeightSum {
    float a, b;
    __device__ __forceinline__ void clear() { a = b = 0.f; }
    // max(p - q, 0) for cleaned p, q: d is the rounded difference, e what its rounding left (exact: p >= q)
    __device__ __forceinline__ void add(float p, float q)
    {
        const float d0 = __fsub_rn(p, q);
        const float e0 = __fsub_rn(__fsub_rn(p, d0), q);
        const bool pos = d0 > 0.f;
        const float d = pos ? d0 : 0.f, e = pos ? e0 : 0.f;
        constexpr float kA = 3.f, kB = 3.f / 4194304.f;  // 1.5 * 2^1 and 1.5 * 2^-21: units 2^-22 and 2^-44
        const float ha = __fsub_rn(__fadd_rn(d, kA), kA);
        const float r = __fadd_rn(__fsub_rn(d, ha), e);
        const float hb = __fsub_rn(__fadd_rn(r, kB), kB);
        a = __fadd_rn(a, ha);
        b = __fadd_rn(b, hb);
    }
    __device__ __forceinline__ long long units() const
    {
        return ((long long)(int)(a * 4194304.f) << 22) + (long long)(int)(b * 17592186044416.f);
    }
};

template <typename T>
struct VerifyRow {  // the row that a sequence's next token is drawn from
    const T *p, *q;  // q null: p alone
    int hot;         // one-hot draft refused: its token (else -1)
    int accepted;
};

// The acceptance of sequence b's drafted tokens.  Every CTA decides it for itself (gamma loads of each kind).
template <typename T>
__device__ __forceinline__ VerifyRow<T> decide(const VerifyParams &p, int b, bool report)
{
    int len = p.lens ? p.lens[b] : p.T;
    if (len < 0 || len > p.T) {
        if (report) set_flag(p.err_flag, PKV_FLAG_TOKEN_RANGE);
        len = min(max(len, 0), p.T);
    }
    const T *target = static_cast<const T *>(p.target) + (int64_t)b * (p.T + 1) * p.target_stride;
    const T *draft = p.draft ? static_cast<const T *>(p.draft) + (int64_t)b * p.T * p.draft_stride : nullptr;
    // lane t looks at token t (a warp's worth at a time): the first refusal of the warp's
    const int lane = threadIdx.x & 31;
    int n = len, hot = -1;
    for (int t0 = 0; t0 < len; t0 += 32) {
        const int t = t0 + lane;
        bool refuse = false;
        int x = -1;
        if (t < len) {
            x = p.tokens[(int64_t)b * p.T + t];
            refuse = true;
            if (x < 0 || x >= p.V) {
                if (report) set_flag(p.err_flag, PKV_FLAG_TOKEN_RANGE);
            } else {
                const float pt = clean(prob_at(target + (int64_t)t * p.target_stride, x));
                const float qt = draft ? clean(prob_at(draft + (int64_t)t * p.draft_stride, x)) : 1.f;
                // products of 24-bit numbers are exact in 64 bits
                refuse = !((double)p.accept_u[(int64_t)b * p.T + t] * (double)qt < (double)pt);
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
    row.p = target + (int64_t)n * p.target_stride;
    row.q = draft && n < len ? draft + (int64_t)n * p.draft_stride : nullptr;
    row.hot = !draft && n < len ? hot : -1;
    return row;
}

// A thread's 16 entries of chunk c as cleaned pairs.  kRuns: consecutive entries (running sums need the order);
// otherwise vectors a CTA's width apart, so that a warp's loads are contiguous.  16-byte loads where the rows
// allow them (a row of an odd vocabulary starts anywhere).
template <typename T, bool kRuns>
__device__ __forceinline__ int64_t entry_of(int c, int k)
{
    constexpr int E = 16 / sizeof(T);  // entries of a vector
    const int64_t i0 = (int64_t)c * kVerifyChunk;
    return kRuns ? i0 + threadIdx.x * kPerThread + k : i0 + ((k / E) * kVerifyThreads + (int)threadIdx.x) * E + k % E;
}

template <bool kRuns, typename T>
__device__ __forceinline__ void load16(const VerifyRow<T> &row, int c, int V, float (&p)[16], float (&q)[16])
{
    constexpr int E = 16 / sizeof(T);
    auto fetch = [&](const T *src, float (&x)[16]) {
        if ((c + 1) * (int64_t)kVerifyChunk <= V && reinterpret_cast<uintptr_t>(src) % 16 == 0) {
            uint4 v[16 / E];
#pragma unroll
            for (int k = 0; k < 16 / E; ++k) v[k] = __ldg(reinterpret_cast<const uint4 *>(src + entry_of<T, kRuns>(c, E * k)));
#pragma unroll
            for (int k = 0; k < 16 / E; ++k) {
                const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (sizeof(T) == 4) {
                        x[E * k + e] = clean(__uint_as_float(w[e]));
                    } else {
                        x[E * k + 2 * e] = clean(bf16x2_lo(w[e]));
                        x[E * k + 2 * e + 1] = clean(bf16x2_hi(w[e]));
                    }
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int64_t i = entry_of<T, kRuns>(c, k);
                x[k] = i < V ? clean(prob_at(src, i)) : 0.f;
            }
        }
    };
    fetch(row.p, p);
    if (row.q) {
        fetch(row.q, q);
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) q[k] = entry_of<T, kRuns>(c, k) == row.hot ? 1.f : 0.f;
    }
}

// The sum of a thread's 16 entries of chunk c.
template <bool kRuns, typename T>
__device__ __forceinline__ long long thread_sum(const VerifyRow<T> &row, int c, int V)
{
    float p[16], q[16];
    load16<kRuns>(row, c, V, p, q);
    long long sum = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        WeightSum w;
        w.clear();
#pragma unroll
        for (int k = 0; k < 4; ++k) w.add(p[4 * h + k], q[4 * h + k]);
        sum += w.units();
    }
    return sum;
}

__device__ __forceinline__ long long block_sum(long long v, long long *warp_sums)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
    __syncthreads();
    long long sum = 0;
#pragma unroll
    for (int w = 0; w < kVerifyWarps; ++w) sum += warp_sums[w];
    return sum;
}

// Inclusive prefix sums over the CTA.
__device__ __forceinline__ long long block_inclusive(long long v, long long *warp_sums)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, v, off);
        if (lane >= off) v += o;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kVerifyWarps; ++w) v += w < warp ? warp_sums[w] : 0;
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p)
{
    __shared__ long long warp_sums[kVerifyWarps];
    __shared__ long long found_before;
    __shared__ int found, last_one;
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    VerifyRow<T> row = decide<T>(p, b, c == 0 && tid < 32);
    long long *sums = p.sums + (int64_t)b * p.chunks;
    const long long mine = block_sum(thread_sum<false>(row, c, p.V), warp_sums);
    if (tid == 0) {
        sums[c] = mine;
        last_one = atomic_add_acq_rel_gpu(p.counters + b, 1) == p.chunks - 1;
    }
    __syncthreads();
    if (!last_one) return;

    // ---- the sequence's last CTA: total, chunk, entry ----
    int token = -1;
    for (int pass = 0; pass < 2 && token < 0; ++pass) {
        if (pass) {
            // no residual mass (p nowhere above q): the token is drawn from p itself
            if (!row.q && row.hot < 0) break;
            row.q = nullptr;
            row.hot = -1;
            for (int x = 0; x < p.chunks; ++x) {
                const long long v = block_sum(thread_sum<false>(row, x, p.V), warp_sums);
                if (tid == 0) sums[x] = v;
            }
            __syncthreads();
        }
        long long total = 0;
        for (int x = tid; x < p.chunks; x += kVerifyThreads) total += __ldcg(sums + x);
        total = block_sum(total, warp_sums);
        if (total <= 0) continue;
        // r in [0, 1): the running sum must exceed r * total, so the last entry with weight always does
        const double r = fmin(fmax((double)p.sample_u[b], 0.0), 1.0 - 0x1p-53);
        const double bar = r * (double)total;  // sums below 2^53 units are exact in 64 bits
        long long before = 0;
        for (int x0 = 0; x0 < p.chunks; x0 += kVerifyThreads) {
            const int x = x0 + tid;
            const long long v = x < p.chunks ? __ldcg(sums + x) : 0;
            const long long upto = before + block_inclusive(v, warp_sums);
            if (tid == 0) found = -1;
            __syncthreads();
            if ((double)upto > bar && (double)(upto - v) <= bar) {
                found = x;
                found_before = upto - v;
            }
            __syncthreads();
            if (found >= 0) break;
            before += block_sum(v, warp_sums);
        }
        const int at = found;
        const long long base = found_before;
        const long long w = thread_sum<true>(row, at, p.V);
        const long long upto = base + block_inclusive(w, warp_sums);
        if (tid == 0) found = -1;
        __syncthreads();
        if ((double)upto > bar && (double)(upto - w) <= bar) {
            // this thread's entries, one by one
            float pv[16], qv[16];
            load16<true>(row, at, p.V, pv, qv);
            long long run = upto - w;
            int hit = -1;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                WeightSum one;
                one.clear();
                one.add(pv[k], qv[k]);
                run += one.units();
                if (hit < 0 && (double)run > bar) hit = (int)entry_of<T, true>(at, k);
            }
            found = hit;
        }
        __syncthreads();
        token = found;
        __syncthreads();
    }
    if (token < 0 && tid == 0) set_flag(p.err_flag, PKV_FLAG_NO_MASS);
    const int n = row.accepted;
    for (int t = tid; t <= p.T; t += kVerifyThreads)
        p.out[(int64_t)b * (p.T + 1) + t] = t < n ? p.tokens[(int64_t)b * p.T + t] : (t == n ? token : -1);
    if (tid == 0) {
        p.accepted[b] = n;
        if (p.context_lens) {
            const int len = p.lens ? min(max(p.lens[b], 0), p.T) : p.T;
            p.context_lens_out[b] = p.context_lens[b] - len + n;
        }
        p.counters[b] = 0;  // ready for the next call
    }
}

cudaError_t launch_verify(const VerifyParams &p, bool bf16, cudaStream_t stream)
{
    const dim3 grid(p.chunks, p.B);
    if (bf16) verify_kernel<uint16_t><<<grid, kVerifyThreads, 0, stream>>>(p);
    else verify_kernel<float><<<grid, kVerifyThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
