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
  // for units that are split: how many there are and in how many parts, then each one's
  // first row, rows and first head; a part's records, [parts][part_rows][d] and
  // [parts][part_rows] (log2 units)
  int4* split_units;
  float *rec_o, *rec_lse;
  int batch, total_q, max_q_len, n_q, group, max_seq_len, cap, may_split, part_rows;
  float qscale;             // softmax scale * log2(e)
};

// The grid, and the workspace that split histories take.
struct B8ChunkPlan {
  long long units;   // (tile of queries, KV head), at most
  int may_split, part_rows;
  size_t workspace;
};
B8ChunkPlan b8_chunk_plan(const tq_config* cfg, int batch, int total_q, int max_q_len, int max_seq_len);
cudaError_t b8_chunk_launch(B8ChunkArgs a, const B8ChunkPlan& p, bool is_int8, int q_dtype, int out_dtype,
                            void* workspace, cudaStream_t s);

}  // namespace tq

#endif  // TQ_B8_CHUNK_CUH_
