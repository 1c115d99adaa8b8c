// tq_b8_store and tq_b8_dequant: writing chunks of new tokens into the 8-bit
// cache with block scales, and reading the cache back.
//
// Store. A unit of work is one (cache block, KV head, keys or values) of a
// sequence; it has one scale, so whoever owns the unit sees everything that
// the scale depends on: the new rows, and the old scale when the block already
// held rows. No atomics, no order of execution. block_size / 16 warps own a
// unit, 16 rows each: a warp reads its rows once (8 x 16 bytes a lane, two
// whole rows per load), takes the largest magnitude on the packed 16-bit
// patterns (a magnitude's bit pattern orders like its value), and quantises
// from its registers. Old rows are read only where the block holds some, and
// written only where the scale grew. The rows are asked for before the block id
// is looked at; 64 registers a thread, since twice the warps (4 CTAs an SM
// instead of 2) took 4 x 8192 tokens of 8 heads from 45.0 to 35.5 us; warps
// whose rows are all new take a path without a look at each row (32.6 us).
// Bound: HBM, 512 bytes read and 256 written per (token, head): 201 MB there,
// 6.18 TB/s, 0.92 of a measured copy. One token each of 32 sequences: 2.6 us, a
// launch.
//
// Dequant. A warp per (sequence, 16 positions, KV head): 4 KB of codes in
// (8 bytes a lane and row), 16 rows of keys and of values out.
// Bound: HBM, 256 bytes read and 512 (16-bit) or 1024 (f32) written: 32 x 4096
// positions of 8 heads to bf16, 805 MB, 121.5 us, 6.63 TB/s, 0.99 of a measured
// copy.

#include "tq_b8.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;

struct StoreArgs {
  B8Cache c;
  const void *key, *value;
  long long key_stride, value_stride;
  const int *query_start, *block_table, *seq_lens;
  unsigned int* status;
  int batch, total_q, max_q_len, cap, cells;   // cells: CTAs per sequence
};

template <typename T>
__device__ __forceinline__ float2 pair_to_floats(uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  else return half2_to_float2(w);
}

// NaN to 0 and infinities to the largest code; nothing else changes.
__device__ __forceinline__ float tame(float y, float limit) { return isnan(y) ? 0.f : fminf(fmaxf(y, -limit), limit); }

template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads, 4) b8_store_kernel(const StoreArgs a) {
  constexpr float kLimit = INT8 ? 127.f : 448.f;
  constexpr uint32_t kInf = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  __shared__ uint32_t s_max[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int log2_wpu = a.c.log2_bs - 4, wpu = 1 << log2_wpu;   // warps per unit
  const int b = blockIdx.x / a.cells, cell = blockIdx.x - b * a.cells;
  grid_dep_wait();
  grid_dep_launch();

  const int raw0 = ld_dep_s32(a.query_start + b), raw1 = ld_dep_s32(a.query_start + b + 1);
  const int len = ld_dep_s32(a.seq_lens + b);
  const int q0 = min(max(raw0, 0), a.total_q);
  const int n = min(max(raw1, q0), a.total_q) - q0;
  const long long start = static_cast<long long>(len) - n;   // position of row q0
  const int lo = static_cast<int>(max(start, 0ll));
  const int end = static_cast<int>(min(min(static_cast<long long>(len), start + a.max_q_len), static_cast<long long>(a.cap)));
  if (cell == 0 && threadIdx.x == 0 &&
      (raw0 < 0 || raw1 < raw0 || raw1 > a.total_q || n > a.max_q_len || start < 0 || (n > 0 && len > a.cap)))
    b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
  if (n == 0 || lo >= end) return;

  const int u = (cell << (3 - log2_wpu)) + (warp >> log2_wpu);   // unit: (block, head, keys or values), the last fastest
  const int kv = u & 1, uh = u >> 1;
  const int jj = uh / a.c.n_kv, h = uh - jj * a.c.n_kv;
  const int j = (lo >> a.c.log2_bs) + jj;
  const long long p0 = static_cast<long long>(j) << a.c.log2_bs;   // position of the block's row 0
  bool active = p0 < end;
  int blk = -1;   // asked for now, looked at after the rows have been asked for
  if (active) blk = ld_dep_s32(a.block_table + static_cast<long long>(b) * a.c.bt_stride + j);
  const int first = static_cast<int>(max(static_cast<long long>(lo) - p0, 0ll));   // rows [first, last) are new
  const int last = static_cast<int>(min(max(static_cast<long long>(end) - p0, 0ll), 1ll << a.c.log2_bs));

  // this warp's rows: 16 (warp's place in the unit) .. + 15, lane: row parity and 8 coordinates
  const int c8 = lane & 15;
  const int r0 = ((warp & (wpu - 1)) << 4) + (lane >> 4);
  const T* src = static_cast<const T*>(kv ? a.value : a.key);
  const long long stride = kv ? a.value_stride : a.key_stride;
  src += (q0 + (p0 - start)) * stride + h * kB8D + 8 * c8;   // row 0 of the block (dereferenced from row `first` on)
  uint4 x[8];
  uint32_t m2 = 0;   // largest magnitudes of the low and of the high halves
  const int w0 = r0 & ~15;
  const bool full = w0 >= first && w0 + 16 <= last;   // all of this warp's rows are new: no row needs a look
  const T* at = src + r0 * stride;
  if (full) {
#pragma unroll
    for (int i = 0; i < 8; ++i, at += 2 * stride) x[i] = ld_dep_u32x4(at);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i, at += 2 * stride) x[i] = ld_or_zero4(at, r0 + 2 * i >= first && r0 + 2 * i < last);
  }
  if (active && !a.c.good(blk)) {
    active = false;
    if (lane == 0) b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
  }
  const bool held = active && first > 0;
  uint8_t* base = const_cast<uint8_t*>(a.c.base);
  float* scale_at = nullptr;
  float s_old = 0.f;
  if (held) s_old = ld_dep_f32(reinterpret_cast<const float*>(a.c.scales(blk, h)) + kv);
  if (active) scale_at = reinterpret_cast<float*>(base + (a.c.scales(blk, h) - a.c.base)) + kv;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m2 = __vmaxu2(m2, x[i].x & 0x7fff7fffu);
    m2 = __vmaxu2(m2, x[i].y & 0x7fff7fffu);
    m2 = __vmaxu2(m2, x[i].z & 0x7fff7fffu);
    m2 = __vmaxu2(m2, x[i].w & 0x7fff7fffu);
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
  const bool wild = m >= kInf;   // this warp's rows hold an infinity or a NaN
  if (wild) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t p = w[k] & 0x7fffu, q = (w[k] >> 16) & 0x7fffu;
        m = max(m, max(p < kInf ? p : 0u, q < kInf ? q : 0u));
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) b8_flag(a.status, TQ_DEV_NOT_FINITE);
  }
  if (wpu > 1) {   // the unit's other warps (all warps of the CTA come here)
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    for (int k = 0; k < wpu; ++k) m = max(m, s_max[(warp & ~(wpu - 1)) + k]);
  }
  if (!active) return;
  const float amax = pair_to_floats<T>(m).x;
  float s = fmaxf(__fdiv_rn(amax, kLimit), kB8Floor);
  if (held) s = fmaxf(s, s_old);
  const float inv = __frcp_rn(s);
  // this lane's 8 codes of row r0 + 2 i: group c8 / 2 at c8 / 2 ^ (r & 7), r odd with r0
  uint8_t* tile = base + (a.c.tile(blk, h, warp & (wpu - 1)) - a.c.base) + kv * kB8HalfBytes + (r0 & 1) * kB8D + ((c8 & 1) << 3);
  const int group = ((c8 >> 1) ^ (r0 & 1)) << 4;
  auto place = [&](int i) { return reinterpret_cast<uint2*>(tile + 2 * i * kB8D + (group ^ ((2 * i & 6) << 4))); };
  auto codes = [&](const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float y[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = pair_to_floats<T>(w[k]);
      y[2 * k] = __fmul_rn(f.x, inv);
      y[2 * k + 1] = __fmul_rn(f.y, inv);
    }
    if (wild) {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = tame(y[k], kLimit);
    }
    return make_uint2(floats_to_codes<INT8>(y[0], y[1], y[2], y[3]), floats_to_codes<INT8>(y[4], y[5], y[6], y[7]));
  };
  if (full) {
#pragma unroll
    for (int i = 0; i < 8; ++i) *place(i) = codes(x[i]);
  } else {
    const bool grew = held && s > s_old;
    const float ratio = grew ? __fdiv_rn(s_old, s) : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 2 * i;
      if (r >= first && r < last) {
        *place(i) = codes(x[i]);
      } else if (grew && r < first) {
        const uint2 old = ld_dep_u32x2(place(i));
        float y[8];
        codes_to_float4<INT8>(old.x, y);
        codes_to_float4<INT8>(old.y, y + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = __fmul_rn(y[k], ratio);
        *place(i) = make_uint2(floats_to_codes<INT8>(y[0], y[1], y[2], y[3]), floats_to_codes<INT8>(y[4], y[5], y[6], y[7]));
      }
    }
  }
  if (lane == 0 && (warp & (wpu - 1)) == 0 && !(held && s == s_old)) *scale_at = s;
}

struct DequantArgs {
  B8Cache c;
  const int *block_table, *seq_lens;
  void *key, *value;
  unsigned int* status;
  int max_seq_len, cap, tiles;   // tiles: 16-position tiles of an output sequence
  long long units;
};

template <typename TO>
__device__ __forceinline__ void write8(TO* dst, const float y[8]) {
  if constexpr (std::is_same<TO, float>::value) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    uint4 o;
    uint32_t* w = &o.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (std::is_same<TO, __half>::value) {
        const __half2 v = __floats2half2_rn(y[2 * k], y[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    *reinterpret_cast<uint4*>(dst) = o;
  }
}

template <typename TO, bool INT8>
__global__ void __launch_bounds__(kThreads) b8_dequant_kernel(const DequantArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long u = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;   // (sequence, tile, head), the last fastest
  grid_dep_wait();
  grid_dep_launch();
  if (u >= a.units) return;
  const long long bt = u / a.c.n_kv;
  const int h = static_cast<int>(u - bt * a.c.n_kv);
  const int b = static_cast<int>(bt / a.tiles), t = static_cast<int>(bt - static_cast<long long>(b) * a.tiles);
  const int raw = ld_dep_s32(a.seq_lens + b);
  const int limit = min(a.max_seq_len, a.cap);
  if (t == 0 && h == 0 && lane == 0 && raw > limit) b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
  int live = min(max(raw, 0), limit) - kB8Rows * t;   // rows of this tile that hold something
  const int rows = min(kB8Rows, a.max_seq_len - kB8Rows * t);
  int blk = -1;
  if (live > 0) {
    blk = ld_dep_s32(a.block_table + static_cast<long long>(b) * a.c.bt_stride + (t >> (a.c.log2_bs - 4)));
    if (!a.c.good(blk)) {
      live = 0;
      if (lane == 0) b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
    }
  }
  const int c8 = lane & 15, r0 = lane >> 4;
  const long long row = static_cast<long long>(a.c.n_kv) * kB8D;
  const long long at = (static_cast<long long>(b) * a.max_seq_len + kB8Rows * t) * row + h * kB8D + 8 * c8;
  uint2 codes[2][8];
  float2 s = make_float2(0.f, 0.f);
  if (live > 0) {
    const uint8_t* tile = a.c.tile(blk, h, t);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + 2 * i;
        codes[kv][i] = ld_dep_u32x2(tile + kv * kB8HalfBytes + r * kB8D + (((c8 >> 1) ^ (r & 7)) << 4) + ((c8 & 1) << 3));
      }
    const uint2 sw = ld_dep_u32x2(a.c.scales(blk, h));
    s = make_float2(__uint_as_float(sw.x), __uint_as_float(sw.y));
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    TO* out = static_cast<TO*>(kv ? a.value : a.key) + at;
    const float f = kv ? s.y : s.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 2 * i;
      if (r >= rows) continue;
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (r < live) {
        codes_to_float4<INT8>(codes[kv][i].x, y);
        codes_to_float4<INT8>(codes[kv][i].y, y + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] *= f;
      }
      write8<TO>(out + r * row, y);
    }
  }
}

template <bool INT8>
cudaError_t launch_dequant(const DequantArgs& a, int out_dtype, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.units + kThreads / 32 - 1) / (kThreads / 32)));
  if (out_dtype == TQ_DTYPE_F32) return launch_pdl(b8_dequant_kernel<float, INT8>, grid, dim3(kThreads), 0, s, a);
  if (out_dtype == TQ_DTYPE_F16) return launch_pdl(b8_dequant_kernel<__half, INT8>, grid, dim3(kThreads), 0, s, a);
  return launch_pdl(b8_dequant_kernel<__nv_bfloat16, INT8>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace
}  // namespace tq

extern "C" {

tq_status tq_b8_store(const tq_config* cfg, const void* key, long long key_stride, const void* value,
                      long long value_stride, int in_dtype, const int* query_start, int batch, int total_q,
                      int max_q_len, void* cache, long long num_blocks, const int* block_table, int bt_stride,
                      const int* seq_lens, unsigned int* dev_status, tq_stream_t stream) {
  using namespace tq;
  tq_b8_layout L;
  tq_status st = make_b8_layout(cfg, &L);
  if (st != TQ_OK) return st;
  if (batch < 0 || total_q < 0 || max_q_len < 0 || !b8_dtype16(in_dtype)) return TQ_ERR_INVALID_ARG;
  if (batch == 0 || total_q == 0 || max_q_len == 0) return TQ_OK;
  if (!key || !value || !query_start) return TQ_ERR_INVALID_ARG;
  if ((st = b8_check(cache, num_blocks, block_table, bt_stride, seq_lens, dev_status)) != TQ_OK) return st;
  if (!b8_aligned(key, 16) || !b8_aligned(value, 16) || !b8_aligned(query_start, 4)) return TQ_ERR_MISALIGNED;
  const long long row = static_cast<long long>(cfg->num_kv_heads) * kB8D;
  if ((st = b8_stride(&key_stride, row)) != TQ_OK || (st = b8_stride(&value_stride, row)) != TQ_OK) return st;
  StoreArgs a;
  a.c = b8_cache(cfg, L, cache, num_blocks, bt_stride);
  a.key = key;
  a.value = value;
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.query_start = query_start;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.status = dev_status;
  a.batch = batch;
  a.total_q = total_q;
  a.max_q_len = max_q_len < total_q ? max_q_len : total_q;
  a.cap = b8_cap(cfg, bt_stride);
  // blocks that a chunk of max_q_len tokens can touch, and 8 warps a CTA
  const int bs = cfg->block_size;
  const long long touched = (static_cast<long long>(a.max_q_len) + 2 * bs - 2) / bs;
  const long long cells = (touched * cfg->num_kv_heads * 2 * (bs / 16) + 7) / 8;
  if (cells * batch > 0x7fffffffll) return TQ_ERR_UNSUPPORTED;
  a.cells = static_cast<int>(cells);
  const dim3 grid(static_cast<unsigned>(cells * batch));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (in_dtype == TQ_DTYPE_BF16)
    err = L.is_int8 ? launch_pdl(b8_store_kernel<__nv_bfloat16, true>, grid, dim3(kThreads), 0, s, a)
                    : launch_pdl(b8_store_kernel<__nv_bfloat16, false>, grid, dim3(kThreads), 0, s, a);
  else
    err = L.is_int8 ? launch_pdl(b8_store_kernel<__half, true>, grid, dim3(kThreads), 0, s, a)
                    : launch_pdl(b8_store_kernel<__half, false>, grid, dim3(kThreads), 0, s, a);
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

tq_status tq_b8_dequant(const tq_config* cfg, const void* cache, long long num_blocks, const int* block_table,
                        int bt_stride, const int* seq_lens, int batch, int max_seq_len, void* key_out,
                        void* value_out, int out_dtype, unsigned int* dev_status, tq_stream_t stream) {
  using namespace tq;
  tq_b8_layout L;
  tq_status st = make_b8_layout(cfg, &L);
  if (st != TQ_OK) return st;
  if (batch < 0 || max_seq_len < 0 || !b8_dtype(out_dtype)) return TQ_ERR_INVALID_ARG;
  if (batch == 0 || max_seq_len == 0) return TQ_OK;
  if (!key_out || !value_out) return TQ_ERR_INVALID_ARG;
  if ((st = b8_check(cache, num_blocks, block_table, bt_stride, seq_lens, dev_status)) != TQ_OK) return st;
  if (!b8_aligned(key_out, 16) || !b8_aligned(value_out, 16)) return TQ_ERR_MISALIGNED;
  DequantArgs a;
  a.c = b8_cache(cfg, L, cache, num_blocks, bt_stride);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.key = key_out;
  a.value = value_out;
  a.status = dev_status;
  a.max_seq_len = max_seq_len;
  a.cap = b8_cap(cfg, bt_stride);
  a.tiles = static_cast<int>((static_cast<long long>(max_seq_len) + 15) / 16);
  a.units = static_cast<long long>(batch) * a.tiles * cfg->num_kv_heads;
  if (a.units > 0x7fffffffll * (kThreads / 32)) return TQ_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = L.is_int8 ? launch_dequant<true>(a, out_dtype, s) : launch_dequant<false>(a, out_dtype, s);
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
