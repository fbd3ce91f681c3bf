// Declarations of block-sparse attention (h3_blocks.cu, h3_block_attention.cu).
#pragma once
#include "h3_internal.cuh"

namespace h3 {

size_t block_scores_workspace_bytes(int nq, int nk, int H, int Hkv);
h3_status launch_block_scores(const void* q, int64_t ld_q, const void* k, int64_t ld_k,
                              float* scores, int Lq, int Lk, int H, int Hkv, int k_block,
                              float scale, void* workspace, cudaStream_t s);
h3_status launch_block_select(const float* scores, int32_t* ids, int32_t* counts, int rows,
                              int nk, int max_blocks, int keep_first, int keep_last,
                              cudaStream_t s);
h3_status launch_attention_blocks(const void* q, int64_t ld_q, const void* k, int64_t ld_k,
                                  const void* v, int64_t ld_v, void* o, int64_t ld_o,
                                  const int32_t* ids, const int32_t* counts, int max_blocks, int Lq,
                                  int Lk, int H, int Hkv, int k_block, float scale,
                                  cudaStream_t s);

}  // namespace h3
