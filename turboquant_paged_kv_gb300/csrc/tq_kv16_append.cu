// tq_kv16_append: chunks of new tokens rotated by their positions and written
// into the 16-bit cache.
//
// A warp takes 8 head rows (queries, then keys, then values) of one token, a half
// warp a row, 16 bytes a lane; all 4 loads of a lane are asked for before the
// token's sequence, position, table row and block are known, three loads one
// after another. A token's cosines and sines are read once for the warp's 8 rows.
// A pair's two coordinates are in one lane (pairs) or in two of a half warp
// (halves: one exchange of the packed 16-bit words). In fp32 from the 16-bit input
// to the one rounding of the output.
//
// Bound: memory. Every row is read and written once: 4 x 8192 tokens of 32 + 2 x 8
// heads 124 us, 6.5 TB/s of 810 MB (0.96 of a measured copy; 80 % of DRAM's cycles,
// 72 registers a thread). 24 chunks of 0-700 tokens, 28 + 2 x 4 heads: 28 us of 21.7,
// one wave with its start, its three loads in a row and its end; 32 sequences' one
// token: 4.1 us, the three loads. A round's loads (kEach = 4 a lane) are asked
// for before the round before is turned and stored. Steps, in that order: one round a
// warp 187 us and 40, more rounds 128 and 28, CTAs of 128 threads 124.
#include <climits>

#include "tq_attn.cuh"
#include "tq_kv16.cuh"

namespace tq {
namespace {

constexpr int kThreads = 128;   // 4 x 8192 tokens, 24 chunks of 0-700: 124 and 28.0 us, 256: 128 and 28.0, 512: 152 and 28.6
constexpr int kEach = 4;   // loads a lane and round: 8 head rows a warp
// Warps from which on they take more rounds of a token rather than being more: its angles are then read, its sequence and
// block found, once for more rows. (The same two, with 256 threads: never 186.6 and 40.1 us, from 152 x 256 on 158.9 and
// 40.1, 152 x 48 127.9 and 28.0, 152 x 16 127.9 and 28.0.) Below, few tokens need all warps: they wait for the three loads.
constexpr int kEnough = 152 * 48;

struct AppendArgs {
  Kv16Cache c;
  const void *q, *key, *value;
  void* q_out;
  long long q_stride, key_stride, value_stride, q_out_stride;
  const float* cos_sin;
  const int *query_start, *block_table, *seq_lens;
  unsigned int* status;
  long long units;
  int batch, total_q, n_q, heads, parts, rounds, rot, num_pos, cap;   // heads: rows of a token; parts: warps a token; rounds of loads each
};

enum Style { kNone, kHalves, kPairs };

// Infinities to the largest number of their sign, NaN to 0; true if there were any.
template <typename T>
__device__ __forceinline__ bool tame(uint32_t& w) {
  constexpr uint32_t kExp = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  const bool lo = (w & kExp) == kExp, hi = (w >> 16 & kExp) == kExp;
  if (__builtin_expect(!(lo || hi), 1)) return false;
  auto one = [&](uint32_t x) { return (x & 0x7fffu) > kExp ? 0u : ((x & 0x8000u) | (kExp - 1)); };
  w = (lo ? one(w & 0xffffu) : (w & 0xffffu)) | (hi ? one(w >> 16) : w >> 16) << 16;
  return true;
}

// The sequence of a row: query_start[b] <= row < query_start[b + 1], with its
// starts and its length; none: false. The warp's lanes together: 32 sequences at
// once, or every n-th first where there are more.
struct Sequence {
  int b, q0, q1, len;
};
__device__ __forceinline__ bool find_sequence(const AppendArgs& a, int row, int lane, Sequence* s) {
  int lo = 0, n = a.batch;   // the answer is in [lo, lo + n) if there is one
  while (n > 32) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, ldg_or(a.query_start + at, lane * step < n, INT_MAX) <= row);
    const int k = m ? 31 - __clz(m) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  const int q0 = ldg_or(a.query_start + lo + lane, lane < n, INT_MAX), q1 = ldg_or(a.query_start + lo + lane + 1, lane < n, 0);
  const int len = ldg_or(a.seq_lens + lo + lane, lane < n, 0);
  const unsigned m = __ballot_sync(0xffffffffu, q0 <= row);
  if (!m) return false;
  const int k = 31 - __clz(m);
  s->b = lo + k;
  s->q0 = __shfl_sync(0xffffffffu, q0, k);
  s->q1 = __shfl_sync(0xffffffffu, q1, k);
  s->len = __shfl_sync(0xffffffffu, len, k);
  return row < s->q1;   // (and starts that go backwards)
}

template <typename T, int STYLE>
__global__ void __launch_bounds__(kThreads) kv16_append_kernel(const AppendArgs a) {
  const int lane = threadIdx.x & 31, c8 = lane & 15;
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  grid_dep_wait();
  grid_dep_launch();
  if (unit >= a.units) return;
  const int row = static_cast<int>(unit / a.parts), part = static_cast<int>(unit - static_cast<long long>(row) * a.parts);
  // this lane's rows: heads head0, head0 + 2, .. of the token's line of queries, keys, values
  int head0 = part * a.rounds * 2 * kEach + (lane >> 4);
  const int n_kv = a.c.n_kv;
  auto load = [&](uint4 (&x)[kEach], int head) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int u = head + 2 * i;
      const T* src = static_cast<const T*>(a.q) + row * a.q_stride + u * kKvD;
      if (u >= a.n_q) src = static_cast<const T*>(a.key) + row * a.key_stride + (u - a.n_q) * kKvD;
      if (u >= a.n_q + n_kv) src = static_cast<const T*>(a.value) + row * a.value_stride + (u - a.n_q - n_kv) * kKvD;
      x[i] = ld_or_zero4(src + 8 * c8, u < a.heads);
    }
  };
  uint4 x[kEach];
  load(x, head0);
  Sequence seq;
  if (!find_sequence(a, row, lane, &seq)) return;
  const long long pos = static_cast<long long>(seq.len) - seq.q1 + row;
  const bool turned = pos >= 0 && (STYLE == kNone || pos < a.num_pos);   // has its angles
  bool stored = turned && pos < a.cap;
  if (part == 0 && lane == 0 && !stored) b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
  if (!turned) return;
  int blk = -1;
  if (stored) blk = ld_dep_s32(a.block_table + static_cast<long long>(seq.b) * a.c.bt_stride + (pos >> a.c.log2_bs));

  float cs[8], sn[8];   // what this lane's coordinates and their partners take
  int from = lane;      // who holds the partners
  if constexpr (STYLE != kNone) {
    const int half = a.rot >> 1;
    const float* angles = a.cos_sin + pos * a.rot;
    const bool in = 8 * c8 < a.rot;
    if constexpr (STYLE == kHalves) {
      const bool second = 8 * c8 >= half;
      const float* at = angles + 8 * c8 - (second ? half : 0);
      if (in) from = second ? lane - (half >> 3) : lane + (half >> 3);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 c4 = in ? ld_dep_f32x4(reinterpret_cast<const float4*>(at) + k) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 s4 = in ? ld_dep_f32x4(reinterpret_cast<const float4*>(at + half) + k) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float f = second ? 1.f : -1.f;
        cs[4 * k] = c4.x; cs[4 * k + 1] = c4.y; cs[4 * k + 2] = c4.z; cs[4 * k + 3] = c4.w;
        sn[4 * k] = f * s4.x; sn[4 * k + 1] = f * s4.y; sn[4 * k + 2] = f * s4.z; sn[4 * k + 3] = f * s4.w;
      }
    } else {
      const float4 c4 = in ? ld_dep_f32x4(reinterpret_cast<const float4*>(angles) + c8) : make_float4(1.f, 1.f, 1.f, 1.f);
      const float4 s4 = in ? ld_dep_f32x4(reinterpret_cast<const float4*>(angles + half) + c8) : make_float4(0.f, 0.f, 0.f, 0.f);
      cs[0] = cs[1] = c4.x; cs[2] = cs[3] = c4.y; cs[4] = cs[5] = c4.z; cs[6] = cs[7] = c4.w;
      sn[0] = -s4.x; sn[1] = s4.x; sn[2] = -s4.y; sn[3] = s4.y; sn[4] = -s4.z; sn[5] = s4.z; sn[6] = -s4.w; sn[7] = s4.w;
    }
  }
  if (stored && !a.c.good(blk)) {
    stored = false;
    if (part == 0 && lane == 0) b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
  }
  const int r = static_cast<int>(pos) & (kKvRows - 1), t = static_cast<int>(pos >> 4);
  bool wild = false;
  for (int round = 1;; ++round, head0 += 2 * kEach) {
    const bool more = round < a.rounds;
    uint4 next[kEach];
    if (more) load(next, head0 + 2 * kEach);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int u = head0 + 2 * i;
      uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      if constexpr (STYLE != kNone) {
        uint32_t p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = STYLE == kHalves ? __shfl_sync(0xffffffffu, w[k], from) : __byte_perm(w[k], 0, 0x1032);
        if (u < a.n_q + n_kv && 8 * c8 < a.rot) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = to_floats<T>(w[k]), o = to_floats<T>(p[k]);
            w[k] = to_pair<T>(fmaf(v.x, cs[2 * k], o.x * sn[2 * k]), fmaf(v.y, cs[2 * k + 1], o.y * sn[2 * k + 1]));
          }
        }
      }
      if (u < a.n_q) {
        *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + row * a.q_out_stride + u * kKvD + 8 * c8) = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (u < a.heads && stored) {
#pragma unroll
        for (int k = 0; k < 4; ++k) wild |= tame<T>(w[k]);
        const int kv = u >= a.n_q + n_kv, h = u - a.n_q - (kv ? n_kv : 0);
        uint8_t* dst = const_cast<uint8_t*>(a.c.tile(blk, h, t)) + kv * kKvHalfBytes + kv16_at(r, c8);
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (!more) break;
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = next[i];
  }
  if (__builtin_expect(wild, 0)) b8_flag(a.status, TQ_DEV_NOT_FINITE);
}

template <typename T>
cudaError_t launch(const AppendArgs& a, int style, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.units + kThreads / 32 - 1) / (kThreads / 32)));
  if (a.rot == 0) return launch_pdl(kv16_append_kernel<T, kNone>, grid, dim3(kThreads), 0, s, a);
  if (style == TQ_ROPE_HALVES) return launch_pdl(kv16_append_kernel<T, kHalves>, grid, dim3(kThreads), 0, s, a);
  return launch_pdl(kv16_append_kernel<T, kPairs>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace
}  // namespace tq

extern "C" {

tq_status tq_kv16_append(const tq_config* cfg, const void* key, long long key_stride, const void* value,
                         long long value_stride, const void* q, long long q_stride, void* q_out,
                         long long q_out_stride, const float* cos_sin, int rot_dim, int num_positions, int rope_style,
                         const int* query_start, int batch, int total_q, void* cache, long long num_blocks,
                         const int* block_table, int bt_stride, const int* seq_lens, unsigned int* dev_status,
                         tq_stream_t stream) {
  using namespace tq;
  tq_kv16_layout L;
  tq_status st = make_kv16_layout(cfg, &L);
  if (st != TQ_OK) return st;
  if (batch < 0 || total_q < 0 || rot_dim < 0 || num_positions < 0) return TQ_ERR_INVALID_ARG;
  if (rot_dim > kKvD || rot_dim % 16) return TQ_ERR_UNSUPPORTED;
  if (rot_dim && rope_style != TQ_ROPE_HALVES && rope_style != TQ_ROPE_PAIRS) return TQ_ERR_INVALID_ARG;
  if ((st = b8_heads(cfg)) != TQ_OK) return st;
  if (batch == 0 || total_q == 0) return TQ_OK;
  if (!key || !value || !query_start || !q != !q_out || !cos_sin != (rot_dim == 0)) return TQ_ERR_INVALID_ARG;
  if ((st = b8_check(cache, num_blocks, block_table, bt_stride, seq_lens, dev_status)) != TQ_OK) return st;
  if (!b8_aligned(key, 16) || !b8_aligned(value, 16) || !b8_aligned(q, 16) || !b8_aligned(q_out, 16) ||
      !b8_aligned(cos_sin, 16) || !b8_aligned(query_start, 4))
    return TQ_ERR_MISALIGNED;
  const long long kv_row = static_cast<long long>(cfg->num_kv_heads) * kKvD, q_row = static_cast<long long>(cfg->num_q_heads) * kKvD;
  if ((st = b8_stride(&key_stride, kv_row)) != TQ_OK || (st = b8_stride(&value_stride, kv_row)) != TQ_OK) return st;
  if (q && ((st = b8_stride(&q_stride, q_row)) != TQ_OK || (st = b8_stride(&q_out_stride, q_row)) != TQ_OK)) return st;
  if (q && q == q_out && q_stride != q_out_stride) return TQ_ERR_INVALID_ARG;
  AppendArgs a = {};
  a.c = kv16_cache(cfg, L, cache, num_blocks, bt_stride);
  a.q = q;
  a.key = key;
  a.value = value;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.q_out_stride = q_out_stride;
  a.cos_sin = cos_sin;
  a.query_start = query_start;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.status = dev_status;
  a.batch = batch;
  a.total_q = total_q;
  a.n_q = q ? cfg->num_q_heads : 0;
  a.heads = a.n_q + 2 * cfg->num_kv_heads;
  const int most = (a.heads + 2 * kEach - 1) / (2 * kEach);
  const long long warps = static_cast<long long>(total_q) * most / kEnough;
  a.rounds = warps < 1 ? 1 : (warps < most ? static_cast<int>(warps) : most);
  a.parts = (most + a.rounds - 1) / a.rounds;
  a.rot = rot_dim;
  a.num_pos = num_positions;
  a.cap = b8_cap(cfg, bt_stride);
  a.units = static_cast<long long>(total_q) * a.parts;
  if (a.units > static_cast<long long>(INT_MAX) * (kThreads / 32)) return TQ_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = L.is_bf16 ? launch<__nv_bfloat16>(a, rope_style, s) : launch<__half>(a, rope_style, s);
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
