// tq_kv16_continue: causal attention of chunks of queries over the 16-bit cache.
//
// A CTA per (query row, query head): 4 warps take every fourth tile of 16
// positions, a position at a time, 4 coordinates a lane, with the running maximum
// and sum of a softmax; the warps' results are joined in shared memory.
#include <climits>

#include "tq_attn.cuh"
#include "tq_kv16.cuh"

namespace tq {
namespace {

constexpr int kWarps = 4;

struct AttnArgs {
  Kv16Cache c;
  const void* q;
  long long q_stride;
  const int *block_table, *seq_lens, *query_start;   // query_start null: a row a sequence
  unsigned int* status;
  void* out;
  int batch, rows, max_q_len, n_q, group, limit;
  float qscale;
};

template <typename T>
__device__ __forceinline__ void four(const void* p, float out[4]) { u2_to_f4<T>(ld_dep_u32x2(p), out); }

template <typename T, typename TO>
__global__ void __launch_bounds__(kWarps * 32) kv16_attn_kernel(const AttnArgs a) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kKvD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / a.n_q, head = blockIdx.x - row * a.n_q;
  grid_dep_wait();
  grid_dep_launch();
  int b = row, seen;
  if (a.query_start) {
    if (row >= ld_dep_s32(a.query_start + a.batch)) return;
    for (b = a.batch - 1; b > 0 && ld_dep_s32(a.query_start + b) > row; --b) {}
    const int q0 = ld_dep_s32(a.query_start + b), q1 = ld_dep_s32(a.query_start + b + 1);
    if (row < q0 || row >= q1) return;
    const int len = ld_dep_s32(a.seq_lens + b);
    const bool served = row - q0 < a.max_q_len;
    if (threadIdx.x == 0 && (!served || len > a.limit)) b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
    seen = served ? static_cast<int>(max(min(static_cast<long long>(len) - q1 + row + 1, static_cast<long long>(a.limit)), 0ll)) : 0;
  } else {
    const int len = ld_dep_s32(a.seq_lens + b);
    if (threadIdx.x == 0 && len > a.limit) b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
    seen = min(max(len, 0), a.limit);
  }
  const int h = head / a.group;
  float q[4], m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  four<T>(static_cast<const T*>(a.q) + row * a.q_stride + head * kKvD + 4 * lane, q);
  for (int p0 = warp * kKvRows; p0 < seen; p0 += kWarps * kKvRows) {
    const int blk = ld_dep_s32(a.block_table + static_cast<long long>(b) * a.c.bt_stride + (p0 >> a.c.log2_bs));
    if (!a.c.good(blk)) {
      if (lane == 0) b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
      continue;
    }
    const uint8_t* tile = a.c.tile(blk, h, p0 >> 4);
    for (int r = 0; r < min(kKvRows, seen - p0); ++r) {
      const uint8_t* at = tile + kv16_at(r, lane >> 1) + 8 * (lane & 1);
      float k[4], v[4];
      four<T>(at, k);
      four<T>(at + kKvHalfBytes, v);
      float x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= a.qscale;
      const float u = fmaxf(m, x), e = exp2f(m - u), f = exp2f(x - u);
      m = u;
      l = l * e + f;
      for (int j = 0; j < 4; ++j) o[j] = o[j] * e + f * v[j];
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int j = 0; j < 4; ++j) s_o[warp][4 * lane + j] = o[j];
  __syncthreads();
  float top = s_m[0], sum = 0.f, y = 0.f;
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  for (int w = 0; w < kWarps; ++w) {
    if (s_l[w] == 0.f) continue;
    const float f = exp2f(s_m[w] - top);
    sum += s_l[w] * f;
    y += s_o[w][threadIdx.x] * f;
  }
  y = sum == 0.f ? 0.f : y / sum;
  static_cast<TO*>(a.out)[(static_cast<long long>(row) * a.n_q + head) * kKvD + threadIdx.x] = static_cast<TO>(y);
}

template <typename T>
cudaError_t launch(const AttnArgs& a, int out_dtype, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.rows) * static_cast<unsigned>(a.n_q));
  if (out_dtype == TQ_DTYPE_F32) return launch_pdl(kv16_attn_kernel<T, float>, grid, dim3(kWarps * 32), 0, s, a);
  if (out_dtype == TQ_DTYPE_F16) return launch_pdl(kv16_attn_kernel<T, __half>, grid, dim3(kWarps * 32), 0, s, a);
  return launch_pdl(kv16_attn_kernel<T, __nv_bfloat16>, grid, dim3(kWarps * 32), 0, s, a);
}

AttnArgs arguments(const tq_config* cfg, const tq_kv16_layout& L, const void* q, long long q_stride, const void* cache,
                   long long num_blocks, const int* block_table, int bt_stride, const int* seq_lens, int max_seq_len,
                   float scale, void* out, unsigned int* status) {
  AttnArgs a = {};
  a.c = kv16_cache(cfg, L, cache, num_blocks, bt_stride);
  a.q = q;
  a.q_stride = q_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.status = status;
  a.out = out;
  a.n_q = cfg->num_q_heads;
  a.group = cfg->num_q_heads / cfg->num_kv_heads;
  const int cap = b8_cap(cfg, bt_stride);
  a.limit = max_seq_len < cap ? max_seq_len : cap;
  a.qscale = b8_qscale(scale);
  return a;
}

}  // namespace
}  // namespace tq

extern "C" {

size_t tq_kv16_continue_workspace_size(const tq_config* cfg, int batch, int total_q, int max_q_len, int max_seq_len) {
  using namespace tq;
  tq_kv16_layout L;
  if (make_kv16_layout(cfg, &L) != TQ_OK || batch < 0 || total_q < 0 || max_q_len < 0 || max_seq_len < 0) return 0;
  if (b8_heads(cfg) != TQ_OK) return 0;
  return 16;
}

tq_status tq_kv16_continue(const tq_config* cfg, const void* q, long long q_stride, const int* query_start, int batch,
                           int total_q, int max_q_len, const void* cache, long long num_blocks, const int* block_table,
                           int bt_stride, const int* seq_lens, int max_seq_len, float scale, void* out, int out_dtype,
                           void* workspace, size_t workspace_bytes, unsigned int* dev_status, tq_stream_t stream) {
  using namespace tq;
  tq_kv16_layout L;
  tq_status st = make_kv16_layout(cfg, &L);
  if (st != TQ_OK) return st;
  if (batch < 0 || total_q < 0 || max_q_len < 0 || max_seq_len < 0 || !b8_dtype(out_dtype)) return TQ_ERR_INVALID_ARG;
  if ((st = b8_heads(cfg)) != TQ_OK) return st;
  if (batch == 0 || total_q == 0 || max_q_len == 0) return TQ_OK;
  if (!q || !query_start || !out || !workspace) return TQ_ERR_INVALID_ARG;
  if ((st = b8_check(cache, num_blocks, block_table, bt_stride, seq_lens, dev_status)) != TQ_OK) return st;
  if (!b8_aligned(q, 16) || !b8_aligned(out, 16) || !b8_aligned(workspace, 16) || !b8_aligned(query_start, 4))
    return TQ_ERR_MISALIGNED;
  if ((st = b8_stride(&q_stride, static_cast<long long>(cfg->num_q_heads) * kKvD)) != TQ_OK) return st;
  if (workspace_bytes < tq_kv16_continue_workspace_size(cfg, batch, total_q, max_q_len, max_seq_len))
    return TQ_ERR_WORKSPACE_TOO_SMALL;
  if (static_cast<long long>(total_q) * cfg->num_q_heads > INT_MAX) return TQ_ERR_UNSUPPORTED;
  AttnArgs a = arguments(cfg, L, q, q_stride, cache, num_blocks, block_table, bt_stride, seq_lens, max_seq_len, scale, out, dev_status);
  a.query_start = query_start;
  a.batch = batch;
  a.rows = total_q;
  a.max_q_len = max_q_len;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = L.is_bf16 ? launch<__nv_bfloat16>(a, out_dtype, s) : launch<__half>(a, out_dtype, s);
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
