// The tensor-core kernel of tq_b8_continue: chunks of queries against the
// 8-bit cache with block scales. Internal, not ABI.
#ifndef TQ_B8_CHUNK_CUH_
#define TQ_B8_CHUNK_CUH_

#include "tq_b8.cuh"

namespace tq {

struct B8ChunkArgs {
  B8Cache c;
  const void* q;
  long long q_stride;
  const int *block_table, *seq_lens, *query_start;
  unsigned int* status;
  void* out;
  float *rec_o, *rec_lse;   // [total_q][n_q][splits][d], [total_q][n_q][splits] (log2 units), for splits > 1
  int batch, total_q, max_q_len, n_q, group, max_seq_len, cap, splits, split_tiles;
  float qscale;             // softmax scale * log2(e)
};

// How the history is split over CTAs, and the workspace that takes.
struct B8ChunkPlan {
  long long q_tiles;   // at most
  int splits, split_tiles;
  size_t workspace;
};
B8ChunkPlan b8_chunk_plan(const tq_config* cfg, int batch, int total_q, int max_q_len, int max_seq_len);
cudaError_t b8_chunk_launch(B8ChunkArgs a, const B8ChunkPlan& p, bool is_int8, int q_dtype, int out_dtype,
                            void* workspace, cudaStream_t s);

}  // namespace tq

#endif  // TQ_B8_CHUNK_CUH_
