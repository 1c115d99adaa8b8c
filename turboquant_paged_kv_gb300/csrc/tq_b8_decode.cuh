// Split attention over the 8-bit cache, one query row at a time: the kernels
// behind tq_b8_decode, and behind tq_b8_continue where a chunk is too short to
// fill the tensor-core kernel's rows. Internal, not ABI.
#ifndef TQ_B8_DECODE_CUH_
#define TQ_B8_DECODE_CUH_

#include "tq_b8.cuh"

namespace tq {

// A line of work: `rows` query rows, row i attending to `len(i)` positions of
// sequence seq(i). For a decode step row i is sequence i; for chunks
// (query_start set) the row's sequence and length follow from query_start.
struct B8SplitArgs {
  const uint8_t* cache;
  long long num_blocks, block_bytes;
  int scale_off, n_kv, log2_bs, bt_stride;
  const void* q;
  long long q_stride;
  const int *block_table, *seq_lens, *query_start;
  unsigned int* status;
  void* out;
  float *rec_o, *rec_lse;   // [records][group][d], [records][group] (log2 units)
  int rows, batch, n_q, group, max_seq_len, cap, max_q_len, warps;   // warps: of the whole split grid
  int early_indices;
  float qscale;             // softmax scale * log2(e)
};

// Bytes of workspace for `rows` query rows.
size_t b8_split_workspace(const tq_config* cfg, long long rows);
// Launches the split and the merge; every argument but `warps`, rec_o and rec_lse is set.
cudaError_t b8_split_launch(B8SplitArgs a, bool is_int8, int q_dtype, int out_dtype, void* workspace, cudaStream_t s);

}  // namespace tq

#endif  // TQ_B8_DECODE_CUH_
