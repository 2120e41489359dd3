// pkv_sequences.h - kernel parameter blocks and launchers of the operators on the blocks that sequences hold: forking,
// extending and compacting them, copies of blocks in many pools (not part of the public C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

constexpr int kMaxCopyPools = 256;
constexpr int kSequenceEntries = 512;  // table entries of a CTA (forks, moved blocks); a row takes up to 65,535 CTAs

struct ForkParams {
    const int32_t *block_tables;   // [rows_in][max_nb]
    const int32_t *context_lens;   // [rows_in]
    const int32_t *parents;        // [rows_out]
    int32_t max_nb, rows_in, rows_out, num_blocks;
    int32_t *ref_counts;           // [num_blocks]
    int32_t *tables_out;           // [rows_out][max_nb]
    int32_t *lens_out;             // [rows_out]
    int32_t *err_flag;
};

struct ExtendParams {
    int32_t *block_tables;         // [rows][max_nb]
    int32_t *context_lens;         // [rows]
    const int32_t *num_new;        // [rows]
    int32_t max_nb, rows, num_blocks;
    int32_t *ref_counts;           // [num_blocks]
    int32_t *copies;               // [rows][2]
    int32_t *step_lens;            // [rows], nullable: new lengths of the rows that grew, else 0
    int32_t *free_ids;             // workspace [num_blocks]
    int32_t *err_flag;
};

struct CompactParams {
    int32_t *block_tables;         // [rows][max_nb]
    const int32_t *context_lens;   // [rows]
    int32_t max_nb, rows, num_blocks;
    int32_t *ref_counts;           // [num_blocks]
    int32_t *moves;                // [max_moves][2]
    int32_t max_moves;
    int32_t *num_moves;            // [1]
    int32_t *move_of;              // workspace [num_blocks]: a moved block's place in moves
    int32_t *err_flag;
};

struct CopyPoolsParams {
    void *pools[kMaxCopyPools];
    const int32_t *src_dst;        // [pairs][2], -1: no copy
    int32_t num_pools, pairs, num_blocks;
    int64_t vectors;               // 16-byte vectors of a block
    int32_t *err_flag;
};

cudaError_t launch_fork_sequences(const ForkParams &p, cudaStream_t stream);
cudaError_t launch_extend_sequences(const ExtendParams &p, cudaStream_t stream);
cudaError_t launch_compact_blocks(const CompactParams &p, cudaStream_t stream);
cudaError_t launch_copy_pools(const CopyPoolsParams &p, int sms, cudaStream_t stream);

}  // namespace pkv
