// tq_b8_continue: causal attention of chunks of queries over the 8-bit cache
// with block scales.
#include <climits>

#include "tq_b8_chunk.cuh"

extern "C" {

size_t tq_b8_continue_workspace_size(const tq_config* cfg, int batch, int total_q, int max_q_len, int max_seq_len) {
  using namespace tq;
  tq_b8_layout L;
  if (make_b8_layout(cfg, &L) != TQ_OK || batch < 0 || total_q < 0 || max_q_len < 0 || max_seq_len < 0) return 0;
  if (b8_heads(cfg) != TQ_OK) return 0;
  return b8_chunk_plan(cfg, batch, total_q, max_q_len, max_seq_len).workspace;
}

tq_status tq_b8_continue(const tq_config* cfg, const void* q, long long q_stride, int q_dtype, const int* query_start,
                         int batch, int total_q, int max_q_len, const void* cache, long long num_blocks,
                         const int* block_table, int bt_stride, const int* seq_lens, int max_seq_len, float scale,
                         void* out, int out_dtype, void* workspace, size_t workspace_bytes,
                         unsigned int* dev_status, tq_stream_t stream) {
  using namespace tq;
  tq_b8_layout L;
  tq_status st = make_b8_layout(cfg, &L);
  if (st != TQ_OK) return st;
  if (batch < 0 || total_q < 0 || max_q_len < 0 || max_seq_len < 0 || !b8_dtype16(q_dtype) || !b8_dtype(out_dtype))
    return TQ_ERR_INVALID_ARG;
  if ((st = b8_heads(cfg)) != TQ_OK) return st;
  if (batch == 0 || total_q == 0 || max_q_len == 0) return TQ_OK;
  if (!q || !query_start || !out || !workspace) return TQ_ERR_INVALID_ARG;
  if ((st = b8_check(cache, num_blocks, block_table, bt_stride, seq_lens, dev_status)) != TQ_OK) return st;
  if (!b8_aligned(q, 16) || !b8_aligned(out, 16) || !b8_aligned(workspace, 16) || !b8_aligned(query_start, 4))
    return TQ_ERR_MISALIGNED;
  if ((st = b8_stride(&q_stride, static_cast<long long>(cfg->num_q_heads) * kB8D)) != TQ_OK) return st;
  if (workspace_bytes < tq_b8_continue_workspace_size(cfg, batch, total_q, max_q_len, max_seq_len))
    return TQ_ERR_WORKSPACE_TOO_SMALL;
  if (static_cast<long long>(total_q) * cfg->num_q_heads > INT_MAX) return TQ_ERR_UNSUPPORTED;
  const B8ChunkPlan p = b8_chunk_plan(cfg, batch, total_q, max_q_len, max_seq_len);
  if (p.units > INT_MAX - 4096) return TQ_ERR_UNSUPPORTED;
  B8ChunkArgs a = {};
  a.c = b8_cache(cfg, L, cache, num_blocks, bt_stride);
  a.q = q;
  a.q_stride = q_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.status = dev_status;
  a.out = out;
  a.batch = batch;
  a.total_q = total_q;
  a.max_q_len = max_q_len;
  a.n_q = cfg->num_q_heads;
  a.group = cfg->num_q_heads / cfg->num_kv_heads;
  a.max_seq_len = max_seq_len;
  a.cap = b8_cap(cfg, bt_stride);
  a.qscale = b8_qscale(scale);
  const cudaError_t err = b8_chunk_launch(a, p, L.is_int8, q_dtype, out_dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
