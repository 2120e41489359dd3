// pkv_ops.h - kernel parameter blocks and launchers of the operators around the attention of a
// decode step: the rotating append, key bounds, block selection, attention over selected blocks and
// the verification of drafted tokens (not part of the public C ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

// Rotary position embedding of q and k_new with the append of k_new and v_new (pkv_rope.cu).  The
// slot and the position of a token are given (slots, positions), or follow from the block tables and
// context lengths (block_tables != nullptr: token i is token i % T of sequence i / T, slots_out
// receives its slot).
struct RopeParams {
    const uint16_t *q;             // [n][N][H] bf16
    const uint16_t *k_new;         // [n][K][H]
    const uint16_t *v_new;
    uint16_t *q_out;               // [n][N][H], may be q itself
    void *k_cache;                 // the pools, bf16 or e4m3
    void *v_cache;
    const float *k_scale;          // e4m3: [K] or [num_blocks][K]
    const float *v_scale;
    int32_t scale_stride;          // e4m3: 0 per head, K per (block, head)
    const double *inv_freq;        // [R / 2] radians per position
    int32_t R;                     // rotated elements of a head
    const int32_t *positions;      // [n]
    const int64_t *slots;          // [n]
    const int32_t *block_tables;   // [B][max_nb]
    const int32_t *context_lens;   // [B]
    int64_t *slots_out;            // [B][T]
    int32_t max_nb, T;
    int32_t n;                     // tokens
    int32_t N, K, H;
    int32_t num_blocks;
    int32_t *err_flag;
    uint64_t wait_ns;
};

cudaError_t launch_rope_append(const RopeParams &p, bool interleaved, bool fp8, int sms, cudaStream_t stream);

// Element-wise minimum and maximum of the keys of every block that holds one of a sequence's last
// num_new tokens (pkv_select.cu): bounds [num_blocks][K][2][H].  span: blocks per sequence at most.
struct BoundsParams {
    const void *k_cache;
    const float *k_scale;
    int32_t scale_stride;
    const int32_t *block_tables;
    const int32_t *context_lens;
    int32_t max_nb, B, K, H, num_blocks, num_new;
    uint16_t *bounds;
    int32_t *err_flag;
};

cudaError_t launch_key_bounds(const BoundsParams &p, bool fp8, int span, cudaStream_t stream);

// Selection of M blocks per (sequence, KV head) by the upper bound of q . k over a block.
struct SelectParams {
    const uint16_t *q;             // [B][N][H] bf16
    const uint16_t *bounds;        // [num_blocks][K][2][H] bf16
    const int32_t *block_tables;
    const int32_t *context_lens;
    int32_t max_nb, B, N, K, G, num_blocks;
    int32_t first, last, M;
    int32_t *selected;             // [B][K][M]
    // workspace: scores by logical block; sums in 64 bits and the list of the blocks whose scores cannot be
    // told apart in 32 bits; the largest |bound| of each tile of 16 blocks
    float *scores;                 // [B][K][max_nb]
    double *exact;                 // [B][K][max_nb]
    int32_t *list;                 // [B][K][max_nb]
    float *tile_max;               // [B][K][tiles]
    int32_t tiles;                 // tiles that cover max_nb blocks
    int32_t *err_flag;
};

cudaError_t launch_select_blocks(const SelectParams &p, int H, int sms, cudaStream_t stream);

// Decode attention over selected blocks (pkv_attn_blocks.cu).
struct BlocksParams {
    const uint16_t *q;             // [B][N][H] bf16
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *selected;       // [B][K][M] logical blocks (-1: none)
    int32_t max_nb, B, N, K, G, M, num_blocks;
    float scale_log2;
    int32_t tok_major;
    int32_t part_blocks;           // list entries per partition
    int32_t max_parts;
    const float *k_scale;          // e4m3
    const float *v_scale;
    int32_t scale_stride;
    __nv_bfloat16 *out;            // [B][N][H]
    float *lse_out;                // nullable
    float *part_out;               // [B][N][max_parts][H]
    float *part_lse;               // [B][N][max_parts]
    int32_t *counters;             // [B][K], zero between calls
    int32_t *err_flag;
    uint64_t wait_ns;
#ifdef PKV_TEST_HOOKS
    int64_t withhold_tile;         // pkv_debug_withhold_tile: -1, or a tile no CTA loads
#endif
};

cudaError_t launch_attn_blocks(int H, bool fp8, const CUtensorMap &tk, const CUtensorMap &tv,
                               const BlocksParams &p, int sms, cudaStream_t stream);

// Verification of drafted tokens (pkv_verify.cu).
struct VerifyParams {
    const void *target;            // [B][T + 1] rows of target_stride elements
    const void *draft;             // [B][T] rows of draft_stride elements, nullable: one-hot drafts
    int64_t target_stride, draft_stride;
    const int32_t *tokens;         // [B][T]
    const int32_t *lens;           // [B], nullable: T everywhere
    const float *accept_u;         // [B][T]
    const float *sample_u;         // [B]
    int32_t B, T, V;
    int32_t *accepted;             // [B]
    int32_t *out;                  // [B][T + 1]
    const int32_t *context_lens;   // [B], nullable
    int32_t *context_lens_out;     // [B]
    long long *sums;               // workspace [B][runs]
    int32_t *counters;             // [B], zero between calls
    int32_t run;                   // entries of a warp's run (set by the launcher)
    int32_t *err_flag;
};

constexpr int kVerifyRun = 256;  // a run of the vocabulary summed by one warp is a multiple of this

cudaError_t launch_verify(VerifyParams p, bool bf16, int sms, cudaStream_t stream);

}  // namespace pkv
