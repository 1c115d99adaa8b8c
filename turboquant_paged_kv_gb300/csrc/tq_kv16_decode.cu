// tq_kv16_decode: attention of one query per sequence over the 16-bit cache.
//
//   out = sum_p softmax_p(scale q . k_p) v_p
//
// Work split: the line of all (sequence, KV head) pairs' tiles (tq_line.cuh), cut
// evenly over the warps of a grid of one CTA per SM, and a merge of the warps'
// records. A warp copies its own tiles, one bulk copy of 8192 bytes each into a
// ring of its own, and waits on that copy's barrier.
//
// Math, per tile of 16 positions x 128 coordinates, on mma.sync.m16n8k16 in the
// cache's type with fp32 sums:
//   S[16 positions, 8 heads] = K . Q^T: exact products
//   O^T[128, 8 heads] += V^T . P^T, P = 8 p in two parts of the type (hi + lo:
//     bf16 2^-16 of the weight, fp16 2^-22 and 2^-25 at least), or three for bf16
//     with f32 output (2^-24): the loads leave the tensor cores idle anyway. p
//     stays below 2^8 (see the softmax), so P fits in fp16.
//   With at most 4 heads a pair, columns 4 .. 7 repeat the heads and carry the lo
//   parts; else the lo parts take a second mma.
// Both operands come by ldmatrix (the values transposed); the cache's swizzle keeps
// its rows in different banks. Softmax in log2 units, the running maximum moving
// only when a score passes it by 2^8 (one warp vote a tile).
#include <climits>

#include "tq_attn.cuh"
#include "tq_kv16.cuh"
#include "tq_line.cuh"

namespace tq {
namespace {

struct Kv16SplitArgs {
  Kv16Cache c;
  const void* q;
  long long q_stride;
  const int *block_table, *seq_lens;
  unsigned int* status;
  void* out;
  float *rec_o, *rec_lse;   // [records][group][d], [records][group] (log2 units)
  int rows, n_kv, n_q, group, max_seq_len, cap, warps;   // rows: sequences; warps: of the whole split grid
  int early_indices;
  float qscale;             // softmax scale * log2(e)
};

constexpr int kWarps = 9;          // a CTA
constexpr int kStages = 3;         // tiles in a warp's ring
constexpr int kMaxCtas = 256;      // grid cap: sizes the workspace without a device query
constexpr int kMaxWarps = 4096;    // partial records beside one per pair
constexpr int kSmem = kWarps * kStages * (kKvTileBytes + 8) + 128;   // and room to align to 128
constexpr float kStep = 8.f;       // the running maximum moves in steps of at least this, log2 units
static_assert(kMaxCtas * kWarps <= kMaxWarps, "workspace");

template <typename T>
__device__ __forceinline__ void mma(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    mma16816(d, a[0], a[1], a[2], a[3], b0, b1);
  }
}
__device__ __forceinline__ void ldmatrix(uint32_t at, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t at, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

template <typename T, bool WIDE, int PARTS>
__global__ void __launch_bounds__(kWarps * 32, 1) kv16_split_kernel(const Kv16SplitArgs a) {
  extern __shared__ uint8_t s_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t smem = (static_cast<uint32_t>(__cvta_generic_to_shared(s_raw)) + 127u) & ~127u;
  const uint32_t ring = smem + warp * kStages * kKvTileBytes;
  const uint32_t bars = smem + kWarps * kStages * kKvTileBytes + warp * kStages * 8;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  __syncwarp();
  if (!a.early_indices) grid_dep_wait();

  const long long wid = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  long long total, before;
  bool too_long;
  Rows first;
  count_tiles(a, 0, lane, &total, &before, &too_long, &first);
  const long long nw = min(static_cast<long long>(a.warps), total);   // warps with work
  const long long x0 = wid < nw ? divide(total * wid, nw) : 0, x1 = wid < nw ? divide(total * (wid + 1), nw) : 0;
  int todo = static_cast<int>(x1 - x0);
  Place put = {}, get = {};   // next tile to load, next tile to use
  if (todo > 0) put = find_tile(a, x0, lane, first);
  get = put;
  if (a.early_indices) grid_dep_wait();
  grid_dep_launch();
  if (wid == 0 && lane == 0 && too_long) b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
  if (todo <= 0) return;

  const uint64_t policy = evict_first_policy();   // read once: the tiles leave L2 to the tables, queries and records
  int to_put = todo, put_stage = 0;
  unsigned bad = 0, phases = 0;   // a bit a stage: its block id is bad; its barrier's parity
  auto table_at = [&](const Place& p) {
    return a.block_table + static_cast<long long>(p.row) * a.c.bt_stride + (p.t >> (a.c.log2_bs - 4));
  };
  int blk = ld_dep_s32(table_at(put));
  auto put_one = [&]() {
    if (to_put <= 0) return;
    const uint32_t bar = bars + 8 * put_stage;
    if (a.c.good(blk)) {
      bad &= ~(1u << put_stage);
      if (lane == 0) {
        mbar_expect(bar, kKvTileBytes);
        bulk_g2s(ring + put_stage * kKvTileBytes, a.c.tile(blk, put.h, put.t), kKvTileBytes, bar, policy);
      }
    } else {
      bad |= 1u << put_stage;
      if (lane == 0) {
        mbar_arrive(bar);
        b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
      }
    }
    if (--to_put > 0) {
      next_tile(a, put);
      blk = ld_dep_s32(table_at(put));
    }
    put_stage = put_stage + 1 == kStages ? 0 : put_stage + 1;
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) put_one();

  // where this lane's rows of the operands are: K, rows lane & 15 and the k-step's group
  // lane / 16; V, rows (lane & 7) + 8 (lane / 16) and the coordinates' group lane / 8 & 1.
  // Step j's groups (2 j, 2 j + 1) lie at ^ 32 j, the second four steps' 1024 behind.
  const uint32_t r8 = lane & 7;
  const uint32_t k_at = ((lane >> 3 & 1) << 11) + (r8 << 7) + (((lane >> 4) ^ r8) << 4);
  const uint32_t v_at = kKvHalfBytes + ((lane >> 4) << 11) + (r8 << 7) + (((lane >> 3 & 1) ^ r8) << 4);
  uint32_t qf[16];           // the query heads as the B operand: coordinates 16 s + 2 t (+ 8) of head g (or g & 3)
  float acc[8][4];           // O^T: coordinates 16 j + g, + 8 (rows) x heads 2 t, 2 t + 1
  float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;
  bool fresh = true;
  int stage = 0;
  for (; todo > 0; --todo) {
    if (fresh) {   // a new (row, head) pair: its query heads
      fresh = false;
      const int head = WIDE ? g : g & 3;
      const T* src = static_cast<const T*>(a.q) + get.row * a.q_stride + (get.h * a.group + head) * kKvD + 2 * t;
#pragma unroll
      for (int i = 0; i < 16; ++i) qf[i] = static_cast<uint32_t>(ldg_or(reinterpret_cast<const int*>(src + 8 * i), head < a.group, 0));
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
      m0 = m1 = -1e30f;
      l0 = l1 = 0.f;
    }

    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, phases >> stage & 1))) {
      // gave up: the other copies in flight end, or have their time, before this warp does
      b8_flag(a.status, TQ_DEV_TIMEOUT);
      for (int i = 0; i < kStages; ++i) mbar_wait(bars + 8 * i, phases >> i & 1);
      return;
    }
    phases ^= 1u << stage;
    const uint32_t kt = ring + stage * kKvTileBytes;

    if (!(bad >> stage & 1)) {
      // S = K . Q^T
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t x[4], y[4];
        const uint32_t at = (kt + k_at) ^ (s << 5);
        ldmatrix(at, x);
        ldmatrix(at + 1024, y);
        mma<T>(sa, x, qf[2 * s], qf[2 * s + 1]);
        mma<T>(sb, y, qf[8 + 2 * s], qf[9 + 2 * s]);
      }
      float x00 = (sa[0] + sb[0]) * a.qscale, x01 = (sa[1] + sb[1]) * a.qscale;
      float x10 = (sa[2] + sb[2]) * a.qscale, x11 = (sa[3] + sb[3]) * a.qscale;
      const int left = get.len - kKvRows * get.t;   // positions from this tile on
      if (left < kKvRows) {
        if (g >= left) x00 = x01 = -INFINITY;
        if (g + 8 >= left) x10 = x11 = -INFINITY;
      }
      const float t0 = fmaxf(x00, x10), t1 = fmaxf(x01, x11);
      if (__any_sync(0xffffffffu, t0 > m0 + kStep || t1 > m1 + kStep)) {
        float u0 = fmaxf(m0, t0), u1 = fmaxf(m1, t1);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, o));
          u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, o));
        }
        const float f0 = ex2(m0 - u0), f1 = ex2(m1 - u1);
        m0 = u0;
        m1 = u1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[j][0] *= f0;
          acc[j][1] *= f1;
          acc[j][2] *= f0;
          acc[j][3] *= f1;
        }
      }
      float p00 = ex2(x00 - m0), p01 = ex2(x01 - m1), p10 = ex2(x10 - m0), p11 = ex2(x11 - m1);
      l0 += p00 + p10;
      l1 += p01 + p11;
      p00 *= 8.f;
      p01 *= 8.f;
      p10 *= 8.f;
      p11 *= 8.f;
      uint32_t h0 = take_pair<T>(p00, p01), h1 = take_pair<T>(p10, p11);
      const uint32_t e0 = take_pair<T>(p00, p01), e1 = take_pair<T>(p10, p11);
      uint32_t b0, b1, c0 = 0, c1 = 0, d0 = 0, d1 = 0;   // parts hi (and lo in columns 4 .. 7), then the other parts
      if constexpr (WIDE) {
        b0 = movmatrix_trans(h0);
        b1 = movmatrix_trans(h1);
        c0 = movmatrix_trans(e0);
        c1 = movmatrix_trans(e1);
      } else {
        b0 = movmatrix_trans(t < 2 ? h0 : e0);
        b1 = movmatrix_trans(t < 2 ? h1 : e1);
      }
      if constexpr (PARTS == 3) {
        h0 = to_pair<T>(p00, p01);
        h1 = to_pair<T>(p10, p11);
        d0 = movmatrix_trans(WIDE || t < 2 ? h0 : 0u);
        d1 = movmatrix_trans(WIDE || t < 2 ? h1 : 0u);
      }
      // O^T += V^T . P^T
      uint32_t live01 = 0xffffffffu, live23 = 0xffffffffu;   // rows behind the end may hold anything, infinities too
      if (left < kKvRows) {
        live01 = (2 * t < left ? 0xffffu : 0u) | (2 * t + 1 < left ? 0xffff0000u : 0u);
        live23 = (2 * t + 8 < left ? 0xffffu : 0u) | (2 * t + 9 < left ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t v[4];
        ldmatrix_trans(((kt + v_at) ^ ((j & 3) << 5)) + (j >> 2) * 1024, v);
        v[0] &= live01;
        v[1] &= live01;
        v[2] &= live23;
        v[3] &= live23;
        mma<T>(acc[j], v, b0, b1);
        if constexpr (WIDE) mma<T>(acc[j], v, c0, c1);
        if constexpr (PARTS == 3) mma<T>(acc[j], v, d0, d1);
      }
    }
    __syncwarp();   // the stage is read: its next tile
    put_one();
    stage = stage + 1 == kStages ? 0 : stage + 1;

    // the end of the pair, or of this warp's part of it
    if (get.t + 1 == get.tiles || todo == 1) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      }
      if constexpr (!WIDE) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[j][k] += __shfl_xor_sync(0xffffffffu, acc[j][k], 2);
      }
      const long long rec = (static_cast<long long>(get.row) * a.n_kv + get.h + wid) * a.group;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int head = 2 * t + k;
        const float l = k ? l1 : l0, m = k ? m1 : m0;
        if (head < a.group) {
          const float f = l > 0.f ? 0.125f / l : (l == 0.f ? 0.f : l);   // NaN stays
          float* o = a.rec_o + (rec + head) * kKvD + g;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[16 * j] = acc[j][k] * f;
            o[16 * j + 8] = acc[j][k + 2] * f;
          }
          if (g == 0) a.rec_lse[rec + head] = l == 0.f ? -INFINITY : m + __log2f(l);
        }
      }
      fresh = true;
    }
    if (todo > 1) next_tile(a, get);
  }
}

template <typename T, bool WIDE, int PARTS>
cudaError_t launch_split(const Kv16SplitArgs& a, int ctas, int dev, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t err = b8_allow_smem(kv16_split_kernel<T, WIDE, PARTS>, kSmem, dev, &done);
  if (err != cudaSuccess) return err;
  return launch_pdl(kv16_split_kernel<T, WIDE, PARTS>, dim3(ctas), dim3(kWarps * 32), kSmem, s, a);
}
template <typename T, int PARTS>
cudaError_t launch_split(const Kv16SplitArgs& a, int ctas, int dev, cudaStream_t s) {
  return a.group > 4 ? launch_split<T, true, PARTS>(a, ctas, dev, s) : launch_split<T, false, PARTS>(a, ctas, dev, s);
}

size_t split_workspace(const tq_config* cfg, long long rows) {
  const int group = cfg->num_q_heads / cfg->num_kv_heads;
  const size_t records = static_cast<size_t>(rows) * cfg->num_kv_heads + kMaxWarps;
  return (records * group * (kKvD + 1) * sizeof(float) + 15) / 16 * 16;
}

cudaError_t split_launch(Kv16SplitArgs a, bool is_bf16, int out_dtype, void* workspace, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t err = b8_current_device(&dev, &sms);
  if (err != cudaSuccess) return err;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  a.warps = ctas * kWarps;
  const size_t records = static_cast<size_t>(a.rows) * a.n_kv + kMaxWarps;
  a.rec_o = static_cast<float*>(workspace);
  a.rec_lse = a.rec_o + records * a.group * kKvD;
  if (!is_bf16) err = launch_split<__half, 2>(a, ctas, dev, s);
  else if (out_dtype == TQ_DTYPE_F32) err = launch_split<__nv_bfloat16, 3>(a, ctas, dev, s);
  else err = launch_split<__nv_bfloat16, 2>(a, ctas, dev, s);
  if (err != cudaSuccess) return err;
  // records of a pair, if the lengths are alike: all of them in one round of loads
  const long long tiles = (static_cast<long long>(a.max_seq_len) + kKvRows - 1) / kKvRows;
  long long records_each = a.warps / (static_cast<long long>(a.rows) * a.n_kv) + 2;
  if (records_each > tiles) records_each = tiles;
  if (out_dtype == TQ_DTYPE_F32) return launch_merge<float>(a, records_each, s);
  if (out_dtype == TQ_DTYPE_F16) return launch_merge<__half>(a, records_each, s);
  return launch_merge<__nv_bfloat16>(a, records_each, s);
}

}  // namespace
}  // namespace tq

extern "C" {

size_t tq_kv16_decode_workspace_size(const tq_config* cfg, int batch, int max_seq_len) {
  using namespace tq;
  tq_kv16_layout L;
  if (make_kv16_layout(cfg, &L) != TQ_OK || batch < 0 || max_seq_len < 0 || b8_heads(cfg) != TQ_OK) return 0;
  return split_workspace(cfg, batch);
}

tq_status tq_kv16_decode(const tq_config* cfg, const void* q, long long q_stride, const void* cache, long long num_blocks,
                         const int* block_table, int bt_stride, const int* seq_lens, int batch, int max_seq_len,
                         float scale, void* out, int out_dtype, void* workspace, size_t workspace_bytes,
                         unsigned int* dev_status, tq_stream_t stream) {
  using namespace tq;
  tq_kv16_layout L;
  tq_status st = make_kv16_layout(cfg, &L);
  if (st != TQ_OK) return st;
  if (batch < 0 || max_seq_len < 0 || !b8_dtype(out_dtype)) return TQ_ERR_INVALID_ARG;
  if ((st = b8_heads(cfg)) != TQ_OK) return st;
  if (batch == 0) return TQ_OK;
  if (!q || !out || !workspace) return TQ_ERR_INVALID_ARG;
  if ((st = b8_check(cache, num_blocks, block_table, bt_stride, seq_lens, dev_status)) != TQ_OK) return st;
  if (!b8_aligned(q, 16) || !b8_aligned(out, 16) || !b8_aligned(workspace, 16)) return TQ_ERR_MISALIGNED;
  if ((st = b8_stride(&q_stride, static_cast<long long>(cfg->num_q_heads) * kKvD)) != TQ_OK) return st;
  if (workspace_bytes < split_workspace(cfg, batch)) return TQ_ERR_WORKSPACE_TOO_SMALL;
  if (static_cast<long long>(batch) * cfg->num_q_heads > INT_MAX) return TQ_ERR_UNSUPPORTED;
  Kv16SplitArgs a = {};
  a.c = kv16_cache(cfg, L, cache, num_blocks, bt_stride);
  a.q = q;
  a.q_stride = q_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.status = dev_status;
  a.out = out;
  a.rows = batch;
  a.n_kv = cfg->num_kv_heads;
  a.n_q = cfg->num_q_heads;
  a.group = cfg->num_q_heads / cfg->num_kv_heads;
  a.max_seq_len = max_seq_len;
  a.cap = b8_cap(cfg, bt_stride);
  a.early_indices = (cfg->flags & TQ_FLAG_INDICES_READY) != 0;
  a.qscale = b8_qscale(scale);
  const cudaError_t err = split_launch(a, L.is_bf16, out_dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
