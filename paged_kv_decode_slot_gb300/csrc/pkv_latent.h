// pkv_latent.h - kernel parameter blocks and launchers of the latent cache: its append and its decode attention (not part
// of the public C ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

constexpr int kLatentDim = 512;   // the latent vector of a token
constexpr int kLatentRope = 64;   // its rotary key
constexpr int kLatentMaxCtas = 152;

// How the (token, head) rows of a sequence are dealt out: chunks of chunk_rows rows, to a CTA (16 or 32) or to a pair of
// CTAs (128, 64 each).
struct LatentPlan {
    int chunk_rows;
    int64_t chunks;
    int ctas() const { return chunk_rows == 128 ? 2 : 1; }
};
// The narrowest that holds a sequence's rows (64 sequences of 512 to 8,192 tokens: 63 us with 16 rows, 66 with 32, by pairs 69
// with 48 and 71 with 64).  48 rows by one CTA were no faster than by a pair (three new tokens of 16 heads over 20 sequences of
// up to 32,520 tokens 82 us for 76, 5 short sequences 17 for 15).
inline LatentPlan latent_plan(int64_t rows)
{
    LatentPlan p;
    p.chunk_rows = rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
    p.chunks = (rows + p.chunk_rows - 1) / p.chunk_rows;
    return p;
}

struct LatentAttnParams {
    const char *cache;             // [num_blocks][16][576] bf16
    const int32_t *block_tables;   // [B][max_nb]
    const int32_t *context_lens;   // [B]
    int32_t max_nb, B, N, T, num_blocks;
    int32_t rows;                  // T * N
    int32_t chunks;                // chunks of rows a sequence
    int32_t ctas;                  // CTAs, or pairs of them, of the grid (set by the launcher)
    float scale_log2;
    __nv_bfloat16 *out;            // [B][T][N][512]
    float *lse_out;                // [B][T][N], nullable
    // workspace: two parts a CTA (or pair), and of each (sequence, chunk) its first CTA and how many there are
    float *part_out;               // [2 ctas][chunk_rows][512]
    float *part_lse;               // [2 ctas][chunk_rows], log2
    int2 *unit_parts;              // [B][chunks]
    int32_t *err_flag;
    uint64_t wait_ns;
#ifdef PKV_TEST_HOOKS
    int64_t withhold_tile;         // pkv_debug_withhold_tile: -1, or a tile no CTA loads
#endif
};

cudaError_t launch_latent_attn(const CUtensorMap &tc, const CUtensorMap &tq, const LatentAttnParams &p, int cta_rows, int sms,
                               cudaStream_t stream);
// Maps of the cache with boxes of a block's two chunks (keys), one chunk (the rotary key) and four chunks (values).
struct LatentPairMaps {
    CUtensorMap keys, rope, values, queries;
};
cudaError_t launch_latent_pair(const LatentPairMaps &maps, const LatentAttnParams &p, int sms, cudaStream_t stream);
cudaError_t launch_latent_join(const LatentAttnParams &p, int chunk_rows, int sms, cudaStream_t stream);

// Norm and rotation of new tokens' rows with their append, and rotation of their queries (pkv_latent_append.cu).
struct LatentAppendParams {
    const uint16_t *kv_new;        // [n][576]
    const uint16_t *q_rope;        // [n][N][64], strides below
    int64_t q_rope_token, q_rope_head;
    uint16_t *q;                   // [n][N][576]: elements 512 .. of a head are written
    const uint16_t *norm_weight;   // [512], nullable: latents are copied
    float eps;
    const double *inv_freq;        // [32] radians per position
    const int32_t *positions;      // [n]
    const int64_t *slots;          // [n]
    const int32_t *block_tables;   // [B][max_nb], else
    const int32_t *context_lens;   // [B]
    int64_t *slots_out;            // [B][T]
    int32_t max_nb, T;
    int32_t n, N, num_blocks;
    uint16_t *cache;               // [num_blocks][16][576]
    int32_t *err_flag;
};

cudaError_t launch_latent_append(const LatentAppendParams &p, bool interleaved, cudaStream_t stream);

}  // namespace pkv
