// tq_kv16_decode: attention of one query per sequence over the 16-bit cache.
//
//   out = sum_p softmax_p(scale q . k_p) v_p
//
// Work split: the line of all (sequence, KV head) pairs' tiles (tq_line.cuh), cut
// evenly over the warps of a grid of one CTA per SM, and a merge of the warps'
// records. A warp copies its own tiles, one bulk copy of 8192 bytes each into a
// ring of its own, and waits on that copy's barrier. Short work takes one launch
// instead (kv16_short_kernel), a CTA or a cluster a pair, and so do few queries of chunks.
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
//
// Bound: memory, the cache being read once. 64 x 512-16384, 8 KV heads: 357-369 us, 6.5-6.7 TB/s
// of 2.39 GB (0.96-0.99 of a measured copy); 4 x 131072, 4 KV heads: 336, 6.4. (32 x 4096 by the
// line: 90 us, 5.96 TB/s, 77 % of DRAM's cycles, tensor cores busy for 9 %, of which 4 to 5
// us are the start, lengths, table and first tiles one after another, and 3 the merge; in
// one launch 82, 6.5 TB/s.) 1 x 301 5.7, a chain of those loads, the tiles and the
// cluster's merge.
#include <climits>

#include "tq_attn.cuh"
#include "tq_kv16.cuh"
#include "tq_line.cuh"
#include "tq_tc.cuh"

namespace tq {
namespace {

// Warps a CTA and tiles in a warp's ring; 32 x 4096, 64 x 512-16384, 4 x 131072: 13 x 2 91.0, 361, 338 us; 9 x 3 92.5, 381,
// 337; 8 x 3 93.6, 378, 340; 7 x 4 94.7, 393, 364; 6 x 4 96, 386, 358. All of shared memory in each, so nearly as much asked
// for at once: more warps share the products, which come between a tile and the next one's request.
constexpr int kWarps = 13;
constexpr int kStages = 2;
constexpr int kMaxCtas = 256;      // grid cap: sizes the workspace without a device query
constexpr int kMaxWarps = 4096;    // partial records beside one per pair
constexpr int kSmem = kWarps * kStages * (kKvTileBytes + 8) + 128;   // and room to align to 128
constexpr int kShortStages = 3;    // of kv16_short_kernel, a warp
constexpr int short_smem(int warps) { return warps * kShortStages * (kKvTileBytes + 8) + 128; }
// Up to which tiles a warp the short kernel is used in place of the split and the merge. By CTAs of 8 warps, and of 2 where
// there are more than are resident at once: 16 x 1024 of 8 heads (8 tiles) 13.4 us for 17.4, 1 x 16000 (16) 16.6 for 20.9;
// 80 x 1000 (640 CTAs of 608) 59.1 for 56.4, 80 x 0-1000 30.4 for 35.8, 256 x 100-600 62 for 73, 1000 x 300 of 2 heads 50 for
// 64. By CTAs of 4 and 2, all resident (64 at most: two ids a lane): 20 x 1000 13.1 for 15.9, 32 x 4096 79 for 88, 32 x 0-4096
// 44.2 for 45.2, 20 x 0-4096 37.7 for 36.5, 64 x 300 10.6 for 16.3, 64 x 2000 75 for 83, 75 x 0-2000 50 for 53, 26 x 0-3000
// 30.1 for 28.7. What a line cut evenly gains where lengths differ, its records and their merge cost.
constexpr int kShortMost = 32, kShortMostSmall = 64;
// From more query heads than kManyHeads on, of at most kFewRecords records each, a warp merges one rather than a CTA:
// 128 x 1000-3000 of 64 heads (1024 pairs, 3 records) 178 us for 195, 100 x 500-5000 of 32 (6 records) 99.9 for 105.7;
// 100 x 500-5000 of 8 heads 182.5 for 181, 26 x 1000-9000 of 48 (14 records) 73.7 for 68.9
constexpr int kManyHeads = 152 * 8, kFewRecords = 8;
// Tiles that are summed in one go. The tensor cores cut what they add off rather than round it, about 2^-25 of the sum each
// time; with f32 output a warp that walks a long history joins the sums of its runs in fp32, in its record (against 64 bits,
// 128 x 16384 of 8 heads, bf16: 4.0e-6, else 1.3e-5). Beside a 16-bit output's rounding that is nothing, and it takes 2 % of
// 4 x 131072 to look for the ends of runs.
constexpr int kRun = 128;
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

__device__ __forceinline__ float ld_cluster(uint32_t at, uint32_t rank) {   // what CTA `rank` of the cluster has at this address
  float v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}\n" : "=f"(v) : "r"(at), "r"(rank) : "memory");
  return v;
}

// What a warp holds of a (sequence, KV head) pair: the query heads, their output so
// far and the softmax's running maximum and sum.
template <typename T, bool WIDE, int PARTS>
struct Heads {
  uint32_t qf[16];   // the B operand: coordinates 16 s + 2 t (+ 8) of head g (or g & 3)
  float acc[8][4];   // O^T: coordinates 16 j + g, + 8 (rows) x heads 2 t, 2 t + 1; 8 times the sum of p v
  float m0, m1, l0, l1;

  __device__ __forceinline__ void begin(const T* q, int group, int lane) {
    const int g = lane >> 2, t = lane & 3, head = WIDE ? g : g & 3;
    const T* src = q + head * kKvD + 2 * t;
#pragma unroll
    for (int i = 0; i < 16; ++i) qf[i] = static_cast<uint32_t>(ldg_or(reinterpret_cast<const int*>(src + 8 * i), head < group, 0));
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    m0 = m1 = -1e30f;
    l0 = l1 = 0.f;
  }

  // The tile at kt in shared memory, of which the first `left` positions count.
  __device__ __forceinline__ void tile(uint32_t kt, int left, float qscale, int lane) {
    const int g = lane >> 2, t = lane & 3;
    // where this lane's rows of the operands are: K, rows lane & 15 and the k-step's group
    // lane / 16; V, rows (lane & 7) + 8 (lane / 16) and the coordinates' group lane / 8 & 1.
    // Step j's groups (2 j, 2 j + 1) lie at ^ 32 j, the second four steps' 1024 behind.
    const uint32_t r8 = lane & 7;
    const uint32_t k_at = ((lane >> 3 & 1) << 11) + (r8 << 7) + (((lane >> 4) ^ r8) << 4);
    const uint32_t v_at = kKvHalfBytes + ((lane >> 4) << 11) + (r8 << 7) + (((lane >> 3 & 1) ^ r8) << 4);
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
    float x00 = (sa[0] + sb[0]) * qscale, x01 = (sa[1] + sb[1]) * qscale;
    float x10 = (sa[2] + sb[2]) * qscale, x11 = (sa[3] + sb[3]) * qscale;
    if (left < kKvRows) {
      if (g >= left) x00 = x01 = -INFINITY;
      if (g + 8 >= left) x10 = x11 = -INFINITY;
    }
    const float t0 = fmaxf(x00, x10), t1 = fmaxf(x01, x11);
    // (the difference and not the sum, which rounds by as much as kStep where scores are 2^27: a weight of 2^16 fits in no fp16)
    if (__any_sync(0xffffffffu, t0 - m0 > kStep || t1 - m1 > kStep)) {
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

  // The whole pair's sums in every lane that has the head (l0, l1 of heads 2 t, 2 t + 1).
  __device__ __forceinline__ void end() {
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
  }
};

// RUNS: sums of no more than kRun tiles, joined in the record.
template <typename T, bool WIDE, int PARTS, bool RUNS>
__global__ void __launch_bounds__(kWarps * 32, 1) kv16_split_kernel(const Kv16RowsArgs a) {
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

  Heads<T, WIDE, PARTS> heads;
  bool fresh = true, again = false;   // begin anew; with the same pair
  float seen[2] = {0.f, 0.f};         // if again, the log2-sums of heads 2 t and 2 t + 1 so far
  int stage = 0, run = 0;             // run: tiles since the beginning
  for (; todo > 0; --todo) {
    if (fresh) {   // a new (row, head) pair, or a new run of one: its query heads
      fresh = false;
      run = 0;
      heads.begin(static_cast<const T*>(a.q) + get.row * a.q_stride + get.h * a.group * kKvD, a.group, lane);
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
      heads.tile(kt, get.len - kKvRows * get.t, a.qscale, lane);
    }
    __syncwarp();   // the stage is read: its next tile
    put_one();
    stage = stage + 1 == kStages ? 0 : stage + 1;

    // the end of the pair, of this warp's part of it, or of a run
    const bool ends = get.t + 1 == get.tiles || todo == 1;
    if (ends || (RUNS && ++run == kRun)) {
      heads.end();
      const long long rec = (static_cast<long long>(get.row) * a.n_kv + get.h + wid) * a.group;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int head = 2 * t + k;
        const float l = k ? heads.l1 : heads.l0, m = k ? heads.m1 : heads.m0;
        if (head < a.group) {
          float f = l > 0.f ? 0.125f / l : (l == 0.f ? 0.f : l);   // NaN stays
          float sum = l == 0.f ? -INFINITY : m + __log2f(l);
          float* o = a.rec_o + (rec + head) * kKvD + g;
          if (RUNS && again) {   // what the runs before left, this lane's own
            const float top = fmaxf(seen[k], sum);
            const float e = seen[k] == -INFINITY ? 0.f : exp2f(seen[k] - top), w = sum == -INFINITY ? 0.f : exp2f(sum - top);
            const float all = e + w == 0.f ? 0.f : 1.f / (e + w);
            sum = e + w == 0.f ? -INFINITY : top + __log2f(e + w);
            f *= w * all;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[16 * j] = fmaf(ld_dep_f32(o + 16 * j), e * all, heads.acc[j][k] * f);
              o[16 * j + 8] = fmaf(ld_dep_f32(o + 16 * j + 8), e * all, heads.acc[j][k + 2] * f);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[16 * j] = heads.acc[j][k] * f;
              o[16 * j + 8] = heads.acc[j][k + 2] * f;
            }
          }
          if (RUNS) seen[k] = sum;
          if (g == 0) a.rec_lse[rec + head] = sum;
        }
      }
      fresh = true;
      again = !ends;
    }
    if (todo > 1) next_tile(a, get);
  }
}

// What row `row` of chunks sees, as tq_kv16_continue has it: positions of sequence `seq`.
__device__ __forceinline__ int row_of_chunk(const Kv16RowsArgs& a, int row, int lane, int* seq, bool* too_long, bool* ours) {
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const bool in = b0 + lane < a.batch;
    const int q0 = max(ldg_or(a.query_start + b0 + lane, in, INT_MAX), 0), q1 = ldg_or(a.query_start + b0 + lane + 1, in, 0);
    const int len = max(ldg_or(a.seq_lens + b0 + lane, in, 0), 0);
    const unsigned m = __ballot_sync(0xffffffffu, q0 <= row && row < q1);
    if (m) {
      const int k = __ffs(m) - 1, limit = min(a.max_seq_len, a.cap);
      const int first = __shfl_sync(0xffffffffu, q0, k), last = __shfl_sync(0xffffffffu, q1, k), all = __shfl_sync(0xffffffffu, len, k);
      const bool served = row - first < a.max_q_len;
      *seq = b0 + k;
      *too_long = !served || all > limit;
      *ours = true;
      // the chunk ends at the end of the rows, should its start say otherwise
      return served ? max(min(all - min(last, a.rows) + row + 1, limit), 0) : 0;
    }
  }
  *ours = *too_long = false;
  return 0;
}

// Work in one launch: a CTA, or a cluster of up to 8, per (sequence, KV head) pair, its
// tiles dealt to their warps in turn; what the warps hold is merged in shared memory,
// then what the CTAs hold, each CTA a part of the output. Measured against the split
// and the merge, or the chunks' kernel: see kShortMost here and in tq_kv16_continue.cu.
template <typename T, typename TO, bool WIDE, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 8 / WARPS) kv16_short_kernel(const Kv16RowsArgs a) {
  constexpr int kParts = std::is_same<T, __nv_bfloat16>::value && std::is_same<TO, float>::value ? 3 : 2;
  extern __shared__ uint8_t s_raw[];
  __shared__ float s_m[WARPS][kB8MaxGroup], s_l[WARPS][kB8MaxGroup];
  __shared__ float s_o[kB8MaxGroup * kKvD], s_om[kB8MaxGroup], s_ol[kB8MaxGroup];   // the CTA's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t smem = (static_cast<uint32_t>(__cvta_generic_to_shared(s_raw)) + 127u) & ~127u;
  const uint32_t ring = smem + warp * kShortStages * kKvTileBytes;
  const uint32_t bars = smem + WARPS * kShortStages * kKvTileBytes + warp * kShortStages * 8;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kShortStages; ++i) mbar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  __syncwarp();
  const int ctas = a.warps, rank = blockIdx.x % ctas, pair = blockIdx.x / ctas;   // CTAs of a pair
  const int row = pair / a.n_kv, h = pair - row * a.n_kv;
  const int first = rank * WARPS + warp, step = ctas * WARPS;   // of the pair's tiles
  if (!a.early_indices) grid_dep_wait();
  bool too_long, ours = true;   // ours: the row is somebody's
  int len, seq = row;
  if (a.query_start) {
    len = row_of_chunk(a, row, lane, &seq, &too_long, &ours);
  } else {
    len = length_of(a, row, &too_long);
  }
  const int tiles = (len + kKvRows - 1) / kKvRows;
  const int todo = tiles > first ? (tiles - first + step - 1) / step : 0;
  // two block ids a lane: this warp's tiles number `lane` and lane + 32 (no more than 64: see the launch)
  const int* table = a.block_table + static_cast<long long>(seq) * a.c.bt_stride;
  const int ids = ldg_or(table + ((first + lane * step) >> (a.c.log2_bs - 4)), lane < todo, -1);
  const int ids2 = ldg_or(table + ((first + (lane + 32) * step) >> (a.c.log2_bs - 4)), lane + 32 < todo, -1);
  if (a.early_indices) grid_dep_wait();
  grid_dep_launch();
  if (too_long && h == 0 && rank == 0 && threadIdx.x == 0) b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
  const uint64_t policy = evict_first_policy();
  const unsigned long long bad = __ballot_sync(0xffffffffu, lane < todo && !a.c.good(ids)) |   // tiles that are left out
                                 static_cast<unsigned long long>(__ballot_sync(0xffffffffu, lane + 32 < todo && !a.c.good(ids2))) << 32;
  if (bad && lane == 0) b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
  auto put = [&](int i) {   // tile i of this warp's to stage i % kShortStages
    const int blk = __shfl_sync(0xffffffffu, i < 32 ? ids : ids2, i & 31);
    const uint32_t bar = bars + 8 * (i % kShortStages);
    if (lane == 0 && !(bad >> i & 1)) {
      mbar_expect(bar, kKvTileBytes);
      bulk_g2s(ring + (i % kShortStages) * kKvTileBytes, a.c.tile(blk, h, first + i * step), kKvTileBytes, bar, policy);
    }
  };
  for (int i = 0; i < kShortStages && i < todo; ++i) put(i);
  Heads<T, WIDE, kParts> heads;
  heads.begin(static_cast<const T*>(a.q) + row * a.q_stride + h * a.group * kKvD, ours ? a.group : 0, lane);
  unsigned phases = 0;   // a barrier's parity
  bool ok = true;
  for (int i = 0; i < todo; ++i) {
    const int stage = i % kShortStages;
    if (!(bad >> i & 1) && ok) {
      ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, phases >> stage & 1)) != 0;
      if (!ok) {   // gave up: the other copies in flight end, or have their time, and no more are asked for
        b8_flag(a.status, TQ_DEV_TIMEOUT);
        for (int k = 0; k < kShortStages; ++k) mbar_wait(bars + 8 * k, phases >> k & 1);
        break;
      }
      phases ^= 1u << stage;
      heads.tile(ring + stage * kKvTileBytes, len - kKvRows * (first + i * step), a.qscale, lane);
    }
    __syncwarp();
    if (i + kShortStages < todo) put(i + kShortStages);
  }
  heads.end();
  // the warp's heads to its own ring, [head][d], and their sums
  float* mine = reinterpret_cast<float*>(s_raw + (ring - static_cast<uint32_t>(__cvta_generic_to_shared(s_raw))));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int head = 2 * t + k;
    if (head < a.group && ok) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mine[head * kKvD + 16 * j + g] = heads.acc[j][k] * 0.125f;
        mine[head * kKvD + 16 * j + g + 8] = heads.acc[j][k + 2] * 0.125f;
      }
    }
    if (head < a.group && g == 0) {
      s_m[warp][head] = k ? heads.m1 : heads.m0;
      s_l[warp][head] = ok ? (k ? heads.l1 : heads.l0) : 0.f;
    }
  }
  __syncthreads();
  const int all = a.group * kKvD;
  const float* rings = reinterpret_cast<const float*>(s_raw + (smem - static_cast<uint32_t>(__cvta_generic_to_shared(s_raw))));
  TO* out = static_cast<TO*>(a.out) + (static_cast<long long>(row) * a.n_q + h * a.group) * kKvD;
  if (!ours && ctas == 1) return;
  for (int e = threadIdx.x; e < all; e += WARPS * 32) {
    const int head = e >> 7;
    float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = fmaxf(m, s_m[w][head]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float lw = s_l[w][head];
      if (lw == 0.f) continue;   // nothing seen, and nothing in the ring
      const float f = exp2f(s_m[w][head] - m);
      l += lw * f;
      o += rings[w * (kShortStages * kKvTileBytes / 4) + e] * f;
    }
    if (ctas == 1) {
      out[e] = static_cast<TO>(l == 0.f ? 0.f : o / l);
    } else {
      s_o[e] = o;
      if ((e & (kKvD - 1)) == 0) {
        s_om[head] = m;
        s_ol[head] = l;
      }
    }
  }
  if (ctas == 1) return;
  cluster_sync();
  const uint32_t at_o = static_cast<uint32_t>(__cvta_generic_to_shared(s_o)), at_m = static_cast<uint32_t>(__cvta_generic_to_shared(s_om)),
                 at_l = static_cast<uint32_t>(__cvta_generic_to_shared(s_ol));
  for (int e = rank * (WARPS * 32) + threadIdx.x; e < all; e += ctas * WARPS * 32) {
    const int head = e >> 7;
    float mk[8], lk[8], ok_[8], m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t from = k < ctas ? k : 0;
      mk[k] = ld_cluster(at_m + 4 * head, from);
      lk[k] = k < ctas ? ld_cluster(at_l + 4 * head, from) : 0.f;
      ok_[k] = ld_cluster(at_o + 4 * e, from);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, mk[k]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (lk[k] == 0.f) continue;
      const float f = exp2f(mk[k] - m);
      l += lk[k] * f;
      o += ok_[k] * f;
    }
    if (ours) out[e] = static_cast<TO>(l == 0.f ? 0.f : o / l);
  }
  cluster_sync();   // nobody goes while its sums are read
}

template <typename T, bool WIDE, int PARTS, bool RUNS>
cudaError_t launch_split(const Kv16RowsArgs& a, int ctas, int dev, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t err = b8_allow_smem(kv16_split_kernel<T, WIDE, PARTS, RUNS>, kSmem, dev, &done);
  if (err != cudaSuccess) return err;
  return launch_pdl(kv16_split_kernel<T, WIDE, PARTS, RUNS>, dim3(ctas), dim3(kWarps * 32), kSmem, s, a);
}
template <typename T, int PARTS, bool RUNS>
cudaError_t launch_split(const Kv16RowsArgs& a, int ctas, int dev, cudaStream_t s) {
  return a.group > 4 ? launch_split<T, true, PARTS, RUNS>(a, ctas, dev, s) : launch_split<T, false, PARTS, RUNS>(a, ctas, dev, s);
}

template <typename T, typename TO, bool WIDE, int WARPS>
cudaError_t launch_short(const Kv16RowsArgs& a, int dev, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t err = b8_allow_smem(kv16_short_kernel<T, TO, WIDE, WARPS>, short_smem(WARPS), dev, &done);
  if (err != cudaSuccess) return err;
  const dim3 grid(static_cast<unsigned>(a.rows) * a.n_kv * a.warps);
  return launch_pdl_cluster(kv16_short_kernel<T, TO, WIDE, WARPS>, grid, dim3(WARPS * 32), a.warps, short_smem(WARPS), s, a);
}
template <typename T, typename TO>
cudaError_t launch_short(Kv16RowsArgs a, const Kv16Short& how, int dev, cudaStream_t s) {
  a.warps = how.ctas;
  if (how.warps == 2) return a.group > 4 ? launch_short<T, TO, true, 2>(a, dev, s) : launch_short<T, TO, false, 2>(a, dev, s);
  if (how.warps == 4) return a.group > 4 ? launch_short<T, TO, true, 4>(a, dev, s) : launch_short<T, TO, false, 4>(a, dev, s);
  return a.group > 4 ? launch_short<T, TO, true, 8>(a, dev, s) : launch_short<T, TO, false, 8>(a, dev, s);
}
template <typename T>
cudaError_t launch_short(const Kv16RowsArgs& a, int out_dtype, const Kv16Short& how, int dev, cudaStream_t s) {
  if (out_dtype == TQ_DTYPE_F32) return launch_short<T, float>(a, how, dev, s);
  if (out_dtype == TQ_DTYPE_F16) return launch_short<T, __half>(a, how, dev, s);
  return launch_short<T, __nv_bfloat16>(a, how, dev, s);
}

template <typename TO>
cudaError_t merge(const Kv16RowsArgs& a, long long records_each, cudaStream_t s) {
  const bool many = static_cast<long long>(a.rows) * a.n_q > kManyHeads && records_each <= kFewRecords;
  return many ? launch_merge_of<TO, 1, 8>(a, s) : launch_merge<TO>(a, records_each, s);
}

size_t split_workspace(const tq_config* cfg, long long rows) {
  const int group = cfg->num_q_heads / cfg->num_kv_heads;
  const size_t records = static_cast<size_t>(rows) * cfg->num_kv_heads + kMaxWarps;
  return (records * group * (kKvD + 1) * sizeof(float) + 15) / 16 * 16;
}

cudaError_t split_launch(Kv16RowsArgs a, bool is_bf16, int out_dtype, void* workspace, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t err = b8_current_device(&dev, &sms);
  if (err != cudaSuccess) return err;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  const long long tiles = (static_cast<long long>(a.max_seq_len) + kKvRows - 1) / kKvRows;
  const long long pairs = static_cast<long long>(a.rows) * a.n_kv;
  Kv16Short how;
  if (kv16_short(a.rows, a.n_kv, a.max_seq_len < a.cap ? a.max_seq_len : a.cap, ctas, kShortMost, kShortMostSmall, true, &how))
    return kv16_short_launch(a, is_bf16, out_dtype, how, dev, s);
  a.warps = ctas * kWarps;
  const size_t records = static_cast<size_t>(a.rows) * a.n_kv + kMaxWarps;
  a.rec_o = static_cast<float*>(workspace);
  a.rec_lse = a.rec_o + records * a.group * kKvD;
  if (out_dtype == TQ_DTYPE_F32) err = is_bf16 ? launch_split<__nv_bfloat16, 3, true>(a, ctas, dev, s) : launch_split<__half, 2, true>(a, ctas, dev, s);
  else err = is_bf16 ? launch_split<__nv_bfloat16, 2, false>(a, ctas, dev, s) : launch_split<__half, 2, false>(a, ctas, dev, s);
  if (err != cudaSuccess) return err;
  // records of a pair, if the lengths are alike: all of them in one round of loads
  long long records_each = a.warps / pairs + 2;
  if (records_each > tiles) records_each = tiles;
  if (out_dtype == TQ_DTYPE_F32) return merge<float>(a, records_each, s);
  if (out_dtype == TQ_DTYPE_F16) return merge<__half>(a, records_each, s);
  return merge<__nv_bfloat16>(a, records_each, s);
}

}  // namespace

bool kv16_short(long long rows, int n_kv, int max_len, int sms, int most, int most_small, bool more, Kv16Short* how) {
  const long long pairs = rows * n_kv, tiles = (static_cast<long long>(max_len) + kKvRows - 1) / kKvRows;
  how->warps = pairs > 2 * sms ? 2 : pairs > sms ? 4 : 8;
  how->ctas = 1;
  if (how->warps < 8) return (more || pairs <= 4 * sms) && tiles <= how->warps * static_cast<long long>(pairs > 4 * sms ? most : most_small);
  how->ctas = 8;   // as many as have an SM each, and a tile a warp
  while (how->ctas > 1 && (pairs * how->ctas > sms || tiles <= how->ctas / 2 * 8ll)) how->ctas /= 2;
  return tiles <= how->ctas * 8ll * most;
}

cudaError_t kv16_short_launch(const Kv16RowsArgs& a, bool is_bf16, int out_dtype, const Kv16Short& how, int dev, cudaStream_t s) {
  return is_bf16 ? launch_short<__nv_bfloat16>(a, out_dtype, how, dev, s) : launch_short<__half>(a, out_dtype, how, dev, s);
}

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
  Kv16RowsArgs a = {};
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
