// The line of work of the decodes over the 8-bit and the 16-bit cache, and the
// merge of what its parts leave. Internal, not ABI.
//
// The 16-position tiles of all (sequence, KV head) pairs form one line, cut evenly
// over the warps of the split kernel's grid; a warp writes one partial record (its
// normalised output and log-sum-exp for the pair's query heads) for every pair that
// it touches, at index pair + warp, unique as both run upwards. Args: seq_lens,
// rows, n_kv, n_q, group, max_seq_len, cap, warps, rec_o, rec_lse, out.
#ifndef TQ_LINE_CUH_
#define TQ_LINE_CUH_

#include "tq_attn.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kLineD = 128;

// How many positions sequence i sees.
template <typename Args>
__device__ __forceinline__ int length_of(const Args& a, int i, bool* too_long) {
  const int limit = min(a.max_seq_len, a.cap), raw = ld_dep_s32(a.seq_lens + i);
  *too_long = raw > limit;
  return min(max(raw, 0), limit);
}

// A place in the line.
struct Place {
  int row, h, t, tiles, len;
};
template <typename Args>
__device__ __forceinline__ void next_tile(const Args& a, Place& p) {
  if (++p.t < p.tiles) return;
  p.t = 0;
  if (++p.h < a.n_kv) return;
  p.h = 0;
  bool too_long;
  do {
    if (++p.row >= a.rows) return;
    p.len = length_of(a, p.row, &too_long);
    p.tiles = (p.len + kTileTokens - 1) / kTileTokens;
  } while (p.tiles == 0);
}

// The rows of a group of 32, one a lane.
struct Rows {
  int len, tiles;
  bool too_long;
};
template <typename Args>
__device__ __forceinline__ Rows rows_of(const Args& a, int i) {
  Rows r = {0, 0, false};
  if (i < a.rows) r.len = length_of(a, i, &r.too_long);
  r.tiles = (r.len + kTileTokens - 1) / kTileTokens;
  return r;
}

// Tiles of all rows, and before row `upto`, times n_kv (a warp's lanes
// together); `first` keeps the first 32 rows.
template <typename Args>
__device__ __forceinline__ void count_tiles(const Args& a, int upto, int lane, long long* total, long long* before,
                                            bool* too_long, Rows* first) {
  long long all = 0, bf = 0;
  bool tl = false;
  for (int i0 = 0; i0 < a.rows; i0 += 32) {
    const Rows r = rows_of(a, i0 + lane);
    if (i0 == 0) *first = r;
    tl |= r.too_long;
    all += __reduce_add_sync(0xffffffffu, r.tiles);
    bf += __reduce_add_sync(0xffffffffu, i0 + lane < upto ? r.tiles : 0);
  }
  *total = all * a.n_kv;
  *before = bf * a.n_kv;
  *too_long = __any_sync(0xffffffffu, tl);
}

// The place of tile x of the line (x < total).
template <typename Args>
__device__ __forceinline__ Place find_tile(const Args& a, long long x, int lane, const Rows& first) {
  Place p = {};
  long long before = 0;
  for (int i0 = 0; i0 < a.rows; i0 += 32) {
    const Rows r = i0 == 0 ? first : rows_of(a, i0 + lane);
    int inc = r.tiles;   // a group of 32 rows holds less than 2^32 tiles
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned m = __ballot_sync(0xffffffffu, x < (before + static_cast<unsigned>(inc)) * a.n_kv);
    if (m) {
      const int src = __ffs(m) - 1;
      const long long rest = x - (before + static_cast<unsigned>(__shfl_sync(0xffffffffu, inc - r.tiles, src))) * a.n_kv;
      p.row = i0 + src;
      p.tiles = __shfl_sync(0xffffffffu, r.tiles, src);
      p.len = __shfl_sync(0xffffffffu, r.len, src);
      p.h = static_cast<int>(divide(rest, p.tiles));
      p.t = static_cast<int>(rest - static_cast<long long>(p.h) * p.tiles);
      return p;
    }
    before += static_cast<unsigned>(__shfl_sync(0xffffffffu, inc, 31));
  }
  return p;
}

// WARPS warps per (sequence, query head), HEADS of these a CTA (several: of one warp
// each): the records of the pair are those of the warps whose parts of the line meet it;
// warp k takes every WARPS-th one, four at a time, a lane 4 coordinates.
template <typename TO, int WARPS, int HEADS, typename Args>
__global__ void __launch_bounds__(WARPS * HEADS * 32) line_merge_kernel(const Args a) {
  static_assert(WARPS == 1 || HEADS == 1, "warps of one head meet at the CTA's barrier");
  __shared__ float s_m[WARPS], s_l[WARPS];
  __shared__ float4 s_o[WARPS][32];
  const int warp = HEADS > 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int index = HEADS > 1 ? blockIdx.x * HEADS + (threadIdx.x >> 5) : blockIdx.x;
  const int row = index / a.n_q, qh = index - row * a.n_q;
  if (HEADS > 1 && row >= a.rows) return;
  const int h = qh / a.group, gg = qh - h * a.group;
  // lengths and starts are not written by the split kernel, which let this
  // launch go only after its own wait: they may be read before this one's
  long long total, before;
  bool too_long;
  Rows first;
  count_tiles(a, row, lane, &total, &before, &too_long, &first);
  int len;
  if (row < 32) {
    len = __shfl_sync(0xffffffffu, first.len, row & 31);
  } else {
    len = length_of(a, row, &too_long);
  }
  const int tiles = (len + kTileTokens - 1) / kTileTokens;
  const long long x0 = before + static_cast<long long>(h) * tiles;
  TO* out = static_cast<TO*>(a.out) + (static_cast<long long>(row) * a.n_q + qh) * kLineD + 4 * lane;
  grid_dep_wait();
  grid_dep_launch();
  if (tiles == 0) {
    if (warp == 0) write4<TO>(out, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  // owners of the pair's first and last tile: warp w owns [total w / nw, total (w + 1) / nw)
  const long long nw = min(static_cast<long long>(a.warps), total);
  const long long w0 = divide((x0 + 1) * nw - 1, total), w1 = divide((x0 + tiles) * nw - 1, total);
  const long long pair = static_cast<long long>(row) * a.n_kv + h;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (long long w = w0 + warp; w <= w1; w += 4 * WARPS) {
    float lse[4];
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long v = w + i * WARPS;
      const bool ok = v <= w1;
      const long long rec = (pair + v) * a.group + gg;
      lse[i] = ok ? ld_dep_f32(a.rec_lse + rec) : -INFINITY;
      x[i] = ok ? ld_dep_f32x4(reinterpret_cast<const float4*>(a.rec_o + rec * kLineD) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (lse[i] == -INFINITY) continue;
      const float u = fmaxf(m, lse[i]);
      const float e = m == -INFINITY ? 0.f : exp2f(m - u), f = exp2f(lse[i] - u);
      m = u;
      l = l * e + f;
      o.x = o.x * e + x[i].x * f;
      o.y = o.y * e + x[i].y * f;
      o.z = o.z * e + x[i].z * f;
      o.w = o.w * e + x[i].w * f;
    }
  }
  if constexpr (WARPS > 1) {
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
    s_o[warp][lane] = o;
    __syncthreads();
    if (warp) return;
  }
#pragma unroll
  for (int k = 1; k < WARPS; ++k) {
    const float mk = s_m[k];
    if (mk == -INFINITY) continue;
    const float u = fmaxf(m, mk);
    const float e = m == -INFINITY ? 0.f : exp2f(m - u), f = exp2f(mk - u);
    const float4 x = s_o[k][lane];
    m = u;
    l = l * e + s_l[k] * f;
    o.x = o.x * e + x.x * f;
    o.y = o.y * e + x.y * f;
    o.z = o.z * e + x.z * f;
    o.w = o.w * e + x.w * f;
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  write4<TO>(out, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
}

template <typename TO, int WARPS, int HEADS = 1, typename Args>
cudaError_t launch_merge_of(const Args& a, cudaStream_t s) {
  const unsigned heads = static_cast<unsigned>(a.rows) * static_cast<unsigned>(a.n_q);
  return launch_pdl(line_merge_kernel<TO, WARPS, HEADS, Args>, dim3((heads + HEADS - 1) / HEADS), dim3(WARPS * HEADS * 32), 0, s, a);
}
template <typename TO, typename Args>
cudaError_t launch_merge(const Args& a, long long records_each, cudaStream_t s) {
  // the whole decode of the 8-bit cache: 4 x 131072 (59 records) 170.3 us with 4 warps, 166.7 with 16; one sequence
  // of 301 (19 records) 6.39 with 4, 6.15 with 8; 32 x 4096 (9 records) 50.0 with 4, 51.5 with 8,
  // 57.3 with 16
  if (records_each > 32) return launch_merge_of<TO, 16>(a, s);
  if (records_each > 16) return launch_merge_of<TO, 8>(a, s);
  return launch_merge_of<TO, 4>(a, s);
}

}  // namespace
}  // namespace tq

#endif  // TQ_LINE_CUH_
