// tq_b8_decode: attention of one query per sequence over the 8-bit cache with
// block scales.
//
//   out = sum_p softmax_p(scale s_k(p) q . k_p) s_v(p) v_p
//
// Work split. The 16-position tiles of all (sequence, KV head) pairs form one
// line, cut evenly over the warps of a grid of one CTA per SM (neighbouring
// parts to different SMs; with fewer tiles than warps, a tile each). A warp writes,
// for every pair that it touches, one partial record (its normalised output
// and log-sum-exp for the pair's query heads) at index pair + warp, unique as
// both run upwards; a second kernel merges a pair's records by their
// log-sum-exp.
//
// Math, per tile of 16 positions x 128 coordinates, on mma.sync.m16n8k16 (f16
// in, f32 out), with every operand but p exact in fp16:
//   S[16 positions, 8 heads] = K . Q^T: codes are exact in fp16; the query row
//     is scaled by a power of two that brings its largest magnitude to 2^14,
//     so a bf16 or fp16 query is exact but for coordinates 2^-28 of the
//     largest. The scales multiply S, 4 numbers a lane and tile.
//   O^T[128, 8 heads] += V^T . P^T with P = 8 p s_v / sigma in two fp16 parts
//     (hi + lo, 2^-22 relative, and never more than 2^-25 off: the weight of a
//     position errs by at most 2^-28 sigma / s_v of the largest). sigma, the
//     reference of a head's accumulators, is a block scale met before: it moves
//     (and the accumulators are rescaled) when a block's s_v leaves [sigma / 16,
//     16 sigma], so P keeps its bits whatever the blocks' scales are (see
//     `reference` for scales very far apart). P stays below 8 * 2^8 * 16 = 2^15
//     (2^8: see the softmax).
//   With at most 4 heads a pair, columns 4 .. 7 repeat the heads and carry the
//   lo parts; else the lo parts take a second mma.
// Softmax in log2 units, the running maximum moving only when a score passes
// it by 2^8 (one warp vote a tile).
//
// Bound: HBM, 256 bytes a (position, head). 4 x 131072 positions of 8 heads, 64
// query heads: 166.5 us, 6.45 TB/s, 0.96 of a measured copy; 64 sequences of 512
// to 16384: 192 us, 6.23 TB/s; 32 x 4096: 49.7 us, 5.4 TB/s, where a warp has 36
// tiles only and the start (lengths, block ids, first tiles, one after another)
// and the merge (3.4 us) show. A warp copies its own tiles (cp.async, 4 in a
// ring): 12 warps with 4 tiles each took 49.3 us there, 10 with 5 52.1, 8 with 6
// 55.6, 14 with 3 48.7 (but 191 and 170 us on the other two): what counts is
// warps, not bytes in flight.
#include <climits>

#include "tq_attn.cuh"
#include "tq_b8.cuh"
#include "tq_line.cuh"

namespace tq {
namespace {

struct B8SplitArgs {
  const uint8_t* cache;
  long long num_blocks, block_bytes;
  int scale_off, n_kv, log2_bs, bt_stride;
  const void* q;
  long long q_stride;
  const int *block_table, *seq_lens;
  unsigned int* status;
  void* out;
  float *rec_o, *rec_lse;   // [records][group][d], [records][group] (log2 units)
  int rows, n_q, group, max_seq_len, cap, warps;   // rows: sequences; warps: of the whole split grid
  int early_indices;
  float qscale;             // softmax scale * log2(e)
};

constexpr int kWarps = 12;         // a CTA
constexpr int kStages = 4;         // tiles in a warp's ring
constexpr int kB8MaxCtas = 256;    // grid cap: sizes the workspace without a device query
constexpr int kMaxWarps = 4096;    // partial records beside one per pair
constexpr int kSmem = kWarps * kStages * (kB8TileBytes + 16);
constexpr float kStep = 8.f;       // the running maximum moves in steps of at least this, log2 units
static_assert(kB8MaxCtas * kWarps <= kMaxWarps, "workspace");

// (codes are read once: they leave L2 to the tables, queries and records)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// The log2 of a head's reference, a whole number: that of the block's value scale,
// lv, as long as neither side is lost. `had` is the log2 of what the accumulators
// hold, `comes` that of the block's largest weight times its scale: the
// accumulators stay below 2^100 and P below 2^15, and P keeps its bits unless it is
// 2^-16 of what is there. Both in units of the output, so 2^-120 is low enough.
__device__ __forceinline__ float reference(float lv, float had, float comes) {
  const float least = fmaxf(had - 100.f, comes - 12.f), most = fmaxf(comes + 6.f, had - 10.f);
  return fmaxf(rintf(fminf(fmaxf(lv, least), most)), -120.f);
}
// 2^x, x whole, -126 <= x <= 127
__device__ __forceinline__ float power_of_2(float x) { return __int_as_float((static_cast<int>(x) + 127) << 23); }

template <typename TQ, bool INT8, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32, 1) b8_split_kernel(const B8SplitArgs a) {
  extern __shared__ __align__(128) uint8_t s_ring[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
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

  const B8Cache c = {a.cache, a.num_blocks, a.block_bytes, a.scale_off, a.n_kv, a.log2_bs, a.bt_stride};
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(s_ring)) + warp * kStages * kB8TileBytes;
  const uint32_t tail = static_cast<uint32_t>(__cvta_generic_to_shared(s_ring)) + kWarps * kStages * kB8TileBytes +
                        warp * kStages * 16;   // a stage's scales: key, value of two heads (negative: bad block)
  const uint64_t policy = evict_first_policy();
  int to_put = todo, put_stage = 0;
  auto table_at = [&](const Place& p) {
    return a.block_table + static_cast<long long>(p.row) * a.bt_stride + (p.t >> (a.log2_bs - 4));
  };
  int blk = ld_dep_s32(table_at(put));
  auto put_one = [&]() {
    if (to_put > 0) {
      const uint32_t dst = ring + put_stage * kB8TileBytes + lane * 16, sdst = tail + put_stage * 16;
      if (c.good(blk)) {
        const uint8_t* src = c.tile(blk, put.h, put.t) + lane * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) cp_async16(dst + i * 512, src + i * 512, policy);
        // the scales of heads h & ~1, h | 1: 16 bytes, since only those go past L1, which may
        // hold what stood there before the kernel in front of this one
        if (lane == 0) cp_async16(sdst, c.scales(blk, put.h & ~1), policy);
      } else if (lane == 0) {
        sts64(sdst, make_uint2(0xbf800000u, 0xbf800000u));
        sts64(sdst + 8, make_uint2(0xbf800000u, 0xbf800000u));
        b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
      }
      if (--to_put > 0) {
        next_tile(a, put);
        blk = ld_dep_s32(table_at(put));
      }
      put_stage = put_stage + 1 == kStages ? 0 : put_stage + 1;
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) put_one();

  uint32_t qf[16];           // the query heads as the B operand: k-step s, coordinates 32 t + 4 s .. + 3 of head g (or g & 3)
  float qs0 = 0.f, qs1 = 0.f;  // scale of heads 2 t, 2 t + 1 (mod 4 unless WIDE)
  float acc[8][4];           // O^T: coordinates 16 g + 2 j, + 1 (rows) x heads 2 t, 2 t + 1
  float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f, sigma0 = 0.f, sigma1 = 0.f, inv0 = 0.f, inv1 = 0.f;   // sigma: log2 of the reference, a whole number; inv: 8 / 2^sigma
  bool fresh = true;
  int stage = 0;
  for (; todo > 0; --todo) {
    if (fresh) {   // a new (row, head) pair: its query heads
      fresh = false;
      const int head = WIDE ? g : g & 3;
      float amax = 0.f;
      float x[32];
      if (head < a.group) {
        const TQ* src = static_cast<const TQ*>(a.q) + get.row * a.q_stride + (get.h * a.group + head) * kB8D + 32 * t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = ld_dep_u32x4(src + 8 * i);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 f;
            if constexpr (std::is_same<TQ, __nv_bfloat16>::value) f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ws[k]));
            else f = half2_to_float2(ws[k]);
            x[8 * i + 2 * k] = f.x;
            x[8 * i + 2 * k + 1] = f.y;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(x[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^k with amax 2^k in [2^14, 2^15)
      const int k = min(max(14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23), -112), 112);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
      const float down = a.qscale * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i) qf[i] = pack_half2(x[2 * i] * up, x[2 * i + 1] * up);
      const int col = WIDE ? 2 * t : (2 * t) & 3;
      qs0 = __shfl_sync(0xffffffffu, down, 4 * col);
      qs1 = __shfl_sync(0xffffffffu, down, 4 * col + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
      m0 = m1 = -1e30f;
      l0 = l1 = 0.f;
      sigma0 = sigma1 = inv0 = inv1 = 0.f;   // no reference yet
    }

    cp_wait<kStages - 2>();
    __syncwarp();
    put_one();
    const uint32_t kt = ring + stage * kB8TileBytes;
    const uint2 sw = lds64(tail + stage * 16 + 8 * (get.h & 1));
    const float s_k = __uint_as_float(sw.x), s_v = __uint_as_float(sw.y);
    stage = stage + 1 == kStages ? 0 : stage + 1;

    if (s_k > 0.f) {   // a good block
      // S = K . Q^T
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t at = kt + g * kB8D + (((2 * t + half) ^ g) << 4);
        const uint4 r0 = lds128(at), r1 = lds128(at + 8 * kB8D);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          codes_to_half2<INT8>(word_of(r0, w), a0, a2);
          codes_to_half2<INT8>(word_of(r1, w), a1, a3);
          mma16816(half ? sb : sa, a0, a1, a2, a3, qf[8 * half + 2 * w], qf[8 * half + 2 * w + 1]);
        }
      }
      const float f0 = qs0 * s_k, f1 = qs1 * s_k;
      float x00 = (sa[0] + sb[0]) * f0, x01 = (sa[1] + sb[1]) * f1;
      float x10 = (sa[2] + sb[2]) * f0, x11 = (sa[3] + sb[3]) * f1;
      const int left = get.len - kB8Rows * get.t;   // positions from this tile on
      if (left < kB8Rows) {
        if (g >= left) x00 = x01 = -INFINITY;
        if (g + 8 >= left) x10 = x11 = -INFINITY;
      }
      const float t0 = fmaxf(x00, x10), t1 = fmaxf(x01, x11);
      float rv0 = s_v * inv0, rv1 = s_v * inv1, far0 = 0.f, far1 = 0.f;
      bool far = false;
      const bool grow = t0 > m0 + kStep || t1 > m1 + kStep;
      const bool move = !(fmaxf(rv0, rv1) <= 8.f * 16.f && fminf(rv0, rv1) >= 8.f * 0.0625f);
      if (__any_sync(0xffffffffu, grow || move)) {
        float u0 = fmaxf(m0, t0), u1 = fmaxf(m1, t1);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, o));
          u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, o));
        }
        const float by0 = m0 - u0, by1 = m1 - u1;
        m0 = u0;
        m1 = u1;
        l0 *= ex2(by0);
        l1 *= ex2(by1);
        float n0 = sigma0, n1 = sigma1;
        if (__any_sync(0xffffffffu, move)) {
          float a0 = 0.f, a1 = 0.f, v0 = t0, v1 = t1;   // a head's largest accumulator and its largest score here
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a0 = fmaxf(a0, fmaxf(fabsf(acc[j][0]), fabsf(acc[j][2])));
            a1 = fmaxf(a1, fmaxf(fabsf(acc[j][1]), fabsf(acc[j][3])));
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
            a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
            v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, v0, o));
            v1 = fmaxf(v1, __shfl_xor_sync(0xffffffffu, v1, o));
          }
          if constexpr (!WIDE) {
            a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 2));
            a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 2));
          }
          const float lv = __log2f(s_v);
          n0 = reference(lv, __log2f(a0) + sigma0 + by0, v0 - u0 + lv);
          n1 = reference(lv, __log2f(a1) + sigma1 + by1, v1 - u1 + lv);
          inv0 = power_of_2(3.f - n0);
          inv1 = power_of_2(3.f - n1);
          far0 = fmaxf(rintf(lv) - n0 - 60.f, 0.f);
          far1 = fmaxf(rintf(lv) - n1 - 60.f, 0.f);
          far = __any_sync(0xffffffffu, far0 + far1 > 0.f);
          rv0 = s_v * power_of_2(3.f - n0 - far0);
          rv1 = s_v * power_of_2(3.f - n1 - far1);
        }
        // 2^(by + sigma - n) in two factors: either alone may pass what fp32 holds
        const float d0 = sigma0 - n0, d1 = sigma1 - n1, h0 = floorf(0.5f * d0), h1 = floorf(0.5f * d1);
        const float f0a = ex2(0.5f * by0 + h0), f0b = ex2(0.5f * by0 + (d0 - h0));
        const float f1a = ex2(0.5f * by1 + h1), f1b = ex2(0.5f * by1 + (d1 - h1));
        sigma0 = n0;
        sigma1 = n1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[j][0] = acc[j][0] * f0a * f0b;
          acc[j][1] = acc[j][1] * f1a * f1b;
          acc[j][2] = acc[j][2] * f0a * f0b;
          acc[j][3] = acc[j][3] * f1a * f1b;
        }
      }
      float p00 = ex2(x00 - m0), p01 = ex2(x01 - m1), p10 = ex2(x10 - m0), p11 = ex2(x11 - m1);
      l0 += p00 + p10;
      l1 += p01 + p11;
      if (__builtin_expect(far, 0)) {   // small weights of large values: p alone may vanish
        p00 = ex2((x00 - m0) + far0);
        p10 = ex2((x10 - m0) + far0);
        p01 = ex2((x01 - m1) + far1);
        p11 = ex2((x11 - m1) + far1);
      }
      p00 *= rv0;
      p01 *= rv1;
      p10 *= rv0;
      p11 *= rv1;
      uint32_t h0, h1, e0, e1;
      split_half2(p00, p01, h0, e0);
      split_half2(p10, p11, h1, e1);
      uint32_t b0, b1, b2 = 0, b3 = 0;
      if constexpr (WIDE) {
        b0 = movmatrix_trans(h0);
        b1 = movmatrix_trans(h1);
        b2 = movmatrix_trans(e0);
        b3 = movmatrix_trans(e1);
      } else {
        b0 = movmatrix_trans(t < 2 ? h0 : e0);
        b1 = movmatrix_trans(t < 2 ? h1 : e1);
      }
      // O^T += V^T . P^T: this lane's four positions at 16 coordinates
      const uint32_t vt = kt + kB8HalfBytes + 2 * t * kB8D;
      uint4 v0 = lds128(vt + ((g ^ (2 * t)) << 4)), v1 = lds128(vt + kB8D + ((g ^ (2 * t + 1)) << 4));
      uint4 v2 = lds128(vt + 8 * kB8D + ((g ^ (2 * t)) << 4)), v3 = lds128(vt + 9 * kB8D + ((g ^ (2 * t + 1)) << 4));
      if (left < kB8Rows) {   // rows behind the end may hold anything, NaN codes too
        const uint4 z = make_uint4(0, 0, 0, 0);
        if (2 * t >= left) v0 = z;
        if (2 * t + 1 >= left) v1 = z;
        if (2 * t + 8 >= left) v2 = z;
        if (2 * t + 9 >= left) v3 = z;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int sel = half ? 0x7362 : 0x5140;
          uint32_t a0, a1, a2, a3;
          codes_to_half2<INT8>(__byte_perm(word_of(v0, w), word_of(v1, w), sel), a0, a1);
          codes_to_half2<INT8>(__byte_perm(word_of(v2, w), word_of(v3, w), sel), a2, a3);
          mma16816(acc[2 * w + half], a0, a1, a2, a3, b0, b1);
          if constexpr (WIDE) mma16816(acc[2 * w + half], a0, a1, a2, a3, b2, b3);
        }
      }
    }

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
        const float l = k ? l1 : l0, m = k ? m1 : m0, sigma = k ? sigma1 : sigma0;
        if (head < a.group) {
          const float f = l > 0.f ? power_of_2(sigma - 3.f) / l : (l == 0.f ? 0.f : l);   // NaN stays
          float4* o = reinterpret_cast<float4*>(a.rec_o + (rec + head) * kB8D + 16 * g);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = make_float4(acc[2 * j][k] * f, acc[2 * j][k + 2] * f, acc[2 * j + 1][k] * f, acc[2 * j + 1][k + 2] * f);
          if (g == 0) a.rec_lse[rec + head] = l == 0.f ? -INFINITY : m + __log2f(l);
        }
      }
      fresh = true;
    }
    if (todo > 1) next_tile(a, get);
  }
}

template <typename TQ, bool INT8, bool WIDE>
cudaError_t launch_split(const B8SplitArgs& a, int ctas, int dev, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t err = b8_allow_smem(b8_split_kernel<TQ, INT8, WIDE>, kSmem, dev, &done);
  if (err != cudaSuccess) return err;
  return launch_pdl(b8_split_kernel<TQ, INT8, WIDE>, dim3(ctas), dim3(kWarps * 32), kSmem, s, a);
}
template <typename TQ>
cudaError_t launch_split(const B8SplitArgs& a, bool is_int8, int ctas, int dev, cudaStream_t s) {
  if (a.group > 4) return is_int8 ? launch_split<TQ, true, true>(a, ctas, dev, s) : launch_split<TQ, false, true>(a, ctas, dev, s);
  return is_int8 ? launch_split<TQ, true, false>(a, ctas, dev, s) : launch_split<TQ, false, false>(a, ctas, dev, s);
}

size_t b8_split_workspace(const tq_config* cfg, long long rows) {
  const int group = cfg->num_q_heads / cfg->num_kv_heads;
  const size_t records = static_cast<size_t>(rows) * cfg->num_kv_heads + kMaxWarps;
  return (records * group * (kB8D + 1) * sizeof(float) + 15) / 16 * 16;
}

cudaError_t b8_split_launch(B8SplitArgs a, bool is_int8, int q_dtype, int out_dtype, void* workspace, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t err = b8_current_device(&dev, &sms);
  if (err != cudaSuccess) return err;
  const int ctas = sms < kB8MaxCtas ? sms : kB8MaxCtas;
  a.warps = ctas * kWarps;
  const size_t records = static_cast<size_t>(a.rows) * a.n_kv + kMaxWarps;
  a.rec_o = static_cast<float*>(workspace);
  a.rec_lse = a.rec_o + records * a.group * kB8D;
  err = q_dtype == TQ_DTYPE_BF16 ? launch_split<__nv_bfloat16>(a, is_int8, ctas, dev, s) : launch_split<__half>(a, is_int8, ctas, dev, s);
  if (err != cudaSuccess) return err;
  // records of a pair, if the lengths are alike: all of them in one round of loads
  const long long tiles = (static_cast<long long>(a.max_seq_len) + kB8Rows - 1) / kB8Rows;
  long long records_each = a.warps / (static_cast<long long>(a.rows) * a.n_kv) + 2;
  if (records_each > tiles) records_each = tiles;
  if (out_dtype == TQ_DTYPE_F32) return launch_merge<float>(a, records_each, s);
  if (out_dtype == TQ_DTYPE_F16) return launch_merge<__half>(a, records_each, s);
  return launch_merge<__nv_bfloat16>(a, records_each, s);
}

}  // namespace
}  // namespace tq

extern "C" {

size_t tq_b8_decode_workspace_size(const tq_config* cfg, int batch, int max_seq_len) {
  using namespace tq;
  tq_b8_layout L;
  if (make_b8_layout(cfg, &L) != TQ_OK || batch < 0 || max_seq_len < 0) return 0;
  if (b8_heads(cfg) != TQ_OK) return 0;
  return b8_split_workspace(cfg, batch);
}

tq_status tq_b8_decode(const tq_config* cfg, const void* q, long long q_stride, int q_dtype, const void* cache,
                       long long num_blocks, const int* block_table, int bt_stride, const int* seq_lens, int batch,
                       int max_seq_len, float scale, void* out, int out_dtype, void* workspace,
                       size_t workspace_bytes, unsigned int* dev_status, tq_stream_t stream) {
  using namespace tq;
  tq_b8_layout L;
  tq_status st = make_b8_layout(cfg, &L);
  if (st != TQ_OK) return st;
  if (batch < 0 || max_seq_len < 0 || !b8_dtype16(q_dtype) || !b8_dtype(out_dtype)) return TQ_ERR_INVALID_ARG;
  if ((st = b8_heads(cfg)) != TQ_OK) return st;
  if (batch == 0) return TQ_OK;
  if (!q || !out || !workspace) return TQ_ERR_INVALID_ARG;
  if ((st = b8_check(cache, num_blocks, block_table, bt_stride, seq_lens, dev_status)) != TQ_OK) return st;
  if (!b8_aligned(q, 16) || !b8_aligned(out, 16) || !b8_aligned(workspace, 16)) return TQ_ERR_MISALIGNED;
  if ((st = b8_stride(&q_stride, static_cast<long long>(cfg->num_q_heads) * kB8D)) != TQ_OK) return st;
  if (workspace_bytes < b8_split_workspace(cfg, batch)) return TQ_ERR_WORKSPACE_TOO_SMALL;
  if (static_cast<long long>(batch) * cfg->num_q_heads > INT_MAX) return TQ_ERR_UNSUPPORTED;
  B8SplitArgs a = {};
  a.cache = static_cast<const uint8_t*>(cache);
  a.num_blocks = num_blocks;
  a.block_bytes = L.block_bytes;
  a.scale_off = L.scale_off;
  a.n_kv = cfg->num_kv_heads;
  a.log2_bs = b8_log2(cfg->block_size);
  a.bt_stride = bt_stride;
  a.q = q;
  a.q_stride = q_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.status = dev_status;
  a.out = out;
  a.rows = batch;
  a.n_q = cfg->num_q_heads;
  a.group = cfg->num_q_heads / cfg->num_kv_heads;
  a.max_seq_len = max_seq_len;
  a.cap = b8_cap(cfg, bt_stride);
  a.early_indices = (cfg->flags & TQ_FLAG_INDICES_READY) != 0;
  a.qscale = b8_qscale(scale);
  const cudaError_t err = b8_split_launch(a, L.is_int8, q_dtype, out_dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
