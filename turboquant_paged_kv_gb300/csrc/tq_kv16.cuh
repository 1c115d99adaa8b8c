// Shared by the kernels of the 16-bit cache: addressing and argument checks
// (those that are not about codes and scales are the 8-bit cache's). Internal,
// not ABI.
//
// Cache block: [n_kv][block_size / 16] tiles of 8192 bytes, 16 key rows then 16
// value rows of 256 bytes, each as [2 groups of 8 rows][2 halves][8 rows][128
// bytes] with the 16-byte group c of row r at group c ^ (r & 7).
#ifndef TQ_KV16_CUH_
#define TQ_KV16_CUH_

#include "tq_b8.cuh"

namespace tq {
namespace {

constexpr int kKvD = 128;
constexpr int kKvRows = 16;          // positions per tile
constexpr int kKvTileBytes = 8192;
constexpr int kKvHalfBytes = 4096;   // the key rows, or the value rows, of a tile

// Where a (block, head) lies.
struct Kv16Cache {
  const uint8_t* base;
  long long num_blocks, block_bytes;
  int n_kv, log2_bs, bt_stride;
  __device__ __forceinline__ bool good(int blk) const { return blk >= 0 && blk < num_blocks; }
  // tile `t` of a sequence, whose block id is blk
  __device__ __forceinline__ const uint8_t* tile(int blk, int h, int t) const {
    const int tpb = 1 << (log2_bs - 4);
    return base + blk * block_bytes + (static_cast<long long>(h * tpb + (t & (tpb - 1))) << 13);
  }
};

// Byte of the 16-byte group c8 (0 .. 15) of row r (0 .. 15) in the key or the value rows of a tile.
__device__ __forceinline__ int kv16_at(int r, int c8) {
  return ((r >> 3) << 11) + ((c8 >> 3) << 10) + ((r & 7) << 7) + (((c8 ^ r) & 7) << 4);
}

// Two numbers of the cache's type in a word.
template <typename T>
__device__ __forceinline__ float2 to_floats(uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  else return half2_to_float2(w);
}
template <typename T>
__device__ __forceinline__ uint32_t to_pair(float x, float y) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
// The pair rounded, and what that leaves of x and y.
template <typename T>
__device__ __forceinline__ uint32_t take_pair(float& x, float& y) {
  const uint32_t w = to_pair<T>(x, y);
  const float2 f = to_floats<T>(w);
  x -= f.x;
  y -= f.y;
  return w;
}

inline Kv16Cache kv16_cache(const tq_config* cfg, const tq_kv16_layout& L, const void* cache, long long num_blocks, int bt_stride) {
  return {static_cast<const uint8_t*>(cache), num_blocks, L.block_bytes, cfg->num_kv_heads, b8_log2(cfg->block_size), bt_stride};
}

}  // namespace

// Rows of queries, each over positions of its own (tq_kv16_decode.cu).
struct Kv16RowsArgs {
  Kv16Cache c;
  const void* q;
  long long q_stride;
  const int *block_table, *seq_lens;
  const int* query_start;   // rows of chunks; null: a row a sequence
  unsigned int* status;
  void* out;
  float *rec_o, *rec_lse;   // [records][group][d], [records][group] (log2 units)
  int rows, n_kv, n_q, group, max_seq_len, cap;
  int batch, max_q_len;     // with query_start
  int warps;                // of the whole split grid
  int early_indices;
  float qscale;             // softmax scale * log2(e)
};
// How so many rows over so many positions are served by one launch: a cluster of `ctas` CTAs of 8 warps a (row, KV head),
// one an SM; where there are more of these than SMs, a CTA of 4 warps each, two an SM, or of 2, four an SM. False: there are
// more than are resident at once (unless `more`), or more than `most` (`most_small`: of 4 or 2, if resident) tiles a warp, 64 at
// most.
struct Kv16Short {
  int ctas;
  int warps;
};
bool kv16_short(long long rows, int n_kv, int max_len, int sms, int most, int most_small, bool more, Kv16Short* how);
cudaError_t kv16_short_launch(const Kv16RowsArgs& a, bool is_bf16, int out_dtype, const Kv16Short& how, int dev, cudaStream_t s);

}  // namespace tq

#endif  // TQ_KV16_CUH_
