// tq_kv16_continue: causal attention of chunks of queries over the 16-bit cache,
// on tcgen05 tensor cores.
//
//   out_i = sum_p softmax_p(scale q_i . k_p) v_p, p <= position of i
//
// A unit of work is 256 rows (the query heads of one KV head of 256 / group
// consecutive queries, in two tiles of 128 rows) against all positions that they
// see, 128 at a time:
//   S_t = Q_t K^T      tcgen05.mma, A and B from shared memory
//   P_t = 8 p          a row a thread, S read from tensor memory
//   O_t += P_t V       A = P_t from tensor memory (it takes S_t's place), B = V
// The steps of all units form one line, cut evenly over a grid of one CTA per SM,
// whatever the lengths are; a unit that a cut goes through leaves records, which a
// second kernel merges. A CTA walks its part of the line with one pipeline: the
// loads of a unit's first steps and its queries come while the last steps of the
// unit before are worked on.
//
// p = 2^(score - m): no maximum is sought in the common case. The weights are taken
// with the maximum so far, and a row of which some P would not fit in fp16 shows in
// its sums; only then the row's new m is found, and what was accumulated (by the
// softmax warps, in tensor memory) and the step's earlier P are rescaled. m is the
// row's own, at most its largest score so far, so the largest P of a row is 8 or
// more, and no position behind the row's own changes a bit of it. P is rounded to
// the cache's type (bf16: by 2^-8, fp16: by 2^-11 and no finer than 2^-25), which is
// what a 16-bit output is rounded to as well; with f32 output it is held in two
// parts (bf16 2^-16, fp16 2^-22).
//
// Warps: 0-3 and 4-7 the softmax of tile 0 and 1, 8 issues the products (of the two
// tiles in turn, so that one tile's products run while the other's softmax does), 9
// finds the work and loads keys and values, 10 and 11 load queries. Keys and values
// come by bulk copies, 4096 bytes a tile of 16 positions: they lie in the cache as
// the tensor cores read them (128-byte swizzle; K a K-major operand, V an MN-major
// one). Every wait is bounded; one that runs out sets TQ_DEV_TIMEOUT and ends the
// CTA, after its products and copies in flight.
#include <climits>

#include "tq_kv16.cuh"
#include "tq_tc.cuh"

namespace tq {
namespace {

constexpr int kRows = 256;             // of a unit: two tiles of 128
constexpr int kCols = 128;             // positions a step
constexpr int kThreads = 640;
constexpr int kCtas = 152;             // grid, one an SM: sizes the workspace without a device query
constexpr float kMost = 60000.f;       // sums of P up to this: every P fits in fp16
constexpr uint32_t kTileOp = 32768;    // a 128 x 128 operand
constexpr uint32_t kHalfQ = 16384;     // Q: two halves of 64 columns, 128 bytes a row
constexpr uint32_t kOffK = 2 * kTileOp, kOffV = 4 * kTileOp, kOffBar = 6 * kTileOp;
constexpr uint32_t kSmem = kOffBar + 256 + 1024;   // and room to align to 1024
constexpr uint32_t kColS = 0, kColO = 256;         // tensor memory columns
constexpr unsigned long long kStepNs = 100000;     // what a step may take, where a wait is for many

struct ChunkArgs {
  Kv16Cache c;
  const void* q;
  long long q_stride;
  const int *block_table, *seq_lens, *query_start;
  unsigned int* status;
  void* out;
  // CTA i's unit that others go on with: first row, rows, first head, parts (0: none);
  // record 2 i is what it adds to a unit that others began, 2 i + 1 the first part of
  // one that others go on with: [part_rows][d] and [part_rows] (log2 units)
  int4* split_units;
  float *rec_o, *rec_lse;
  int batch, total_q, max_q_len, n_q, group, limit, may_split, part_rows;   // limit: positions at most
  float qscale;                        // softmax scale * log2(e)
};

// barriers, 8 bytes each from kOffBar
enum {
  kWFull0, kWFull1, kWEmpty0, kWEmpty1, kQFull, kQEmpty, kKFull0, kKFull1, kVFull0, kVFull1, kKEmpty0, kKEmpty1, kVEmpty0, kVEmpty1,
  kSFull0, kSFull1, kPFull0, kPFull1, kODone0, kODone1, kEnd, kBars
};
static_assert(kBars * 8 <= 256, "barriers");

// shared-memory operand descriptors, 128-byte swizzle. Q: 8-row groups 1024 bytes
// apart; K: 2048 (its halves lie 1024 behind); V: halves 1024 apart, groups 2048.
__device__ __forceinline__ uint64_t desc_q(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1ull << 16) | (128ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_v(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (64ull << 16) | (128ull << 32) | (1ull << 46) | (2ull << 61);
}
// f16 x f16 or bf16 x bf16 -> f32, M = 128, N = 128
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc_qk() {
  return (1u << 4) | (std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u) | ((128u / 8) << 17) | ((128u / 16) << 24);
}
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc_pv() { return idesc_qk<T>() | (1u << 16); }   // B is MN-major

// Waits for the loads from tensor memory; what they brought is not used before.
__device__ __forceinline__ void wait_ld(float (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]),
                 "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])::"memory");
}
__device__ __forceinline__ void wait_ld(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]),
                 "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]),
                 "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]),
                 "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])::"memory");
}
__device__ __forceinline__ void load16(uint32_t addr, float (&r)[16]) { tmem_ld16(addr, reinterpret_cast<uint32_t*>(r)); }
__device__ __forceinline__ void load32(uint32_t addr, float (&r)[32]) { tmem_ld32(addr, reinterpret_cast<uint32_t*>(r)); }

// Waits for the other warp of the pair; true if `x` is true in any lane of either.
__device__ __forceinline__ bool pair_any(int id, bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(r)
               : "r"(id), "r"(static_cast<uint32_t>(x))
               : "memory");
  return r != 0;
}

// A part of a unit, as a CTA works on it.
struct Work {
  int seq, h;          // sequence (-1: the end), KV head
  int slot;            // its record (-1: the whole unit)
  int q0, rows;        // row of its first query in q and out; rows of A, its queries' heads
  int pos0;            // position of that query (may be negative)
  int limit;           // positions that its last query sees: what stands behind them need not have been stored
  int tile0, tiles;    // steps: [tile0, tile0 + tiles); none: zeros are written
  int zero0, zeros;    // queries that nobody serves
  unsigned step0;      // steps of the CTA before
};

// A sequence's chunk: its first row, queries, length and tiles of queries.
struct Chunk {
  int q0, n, len, tiles;
};
__device__ __forceinline__ Chunk chunk_of(const ChunkArgs& a, int b, int per) {
  Chunk c;
  c.q0 = min(max(ldg_or(a.query_start + b, b < a.batch, 0), 0), a.total_q);
  c.n = min(max(ldg_or(a.query_start + b + 1, b < a.batch, 0), c.q0), a.total_q) - c.q0;
  c.len = max(ldg_or(a.seq_lens + b, b < a.batch, 0), 0);
  c.tiles = (min(c.n, a.max_q_len) + per - 1) / per;
  return c;
}
// Positions that the last query of tile j sees, and the unit's steps: one at least, though it may see nothing.
__device__ __forceinline__ int limit_of(const ChunkArgs& a, const Chunk& c, int j, int per) {
  return max(min(c.len - c.n + min((j + 1) * per, min(c.n, a.max_q_len)), a.limit), 0);
}
__device__ __forceinline__ int steps_of(const ChunkArgs& a, const Chunk& c, int j, int per) {
  return j < c.tiles ? max((limit_of(a, c, j, per) + kCols - 1) / kCols, 1) : 0;
}
__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The line: for each tile index j, each sequence that has such a tile, each KV head,
// its steps. (Units that read the same keys and values, tiles of one chunk, are then a
// fixed part of the line apart, so that CTAs meet them at the same time where chunks
// are alike.) A warp walks it, the lanes together.
struct Line {
  const ChunkArgs& a;
  int per, lane, tiles_most = 0;
  long long total = 0;
  int b0 = -1;
  Chunk ch = {};       // lane's chunk of the 32 from b0 on
  // a place: tile, sequence, head; the unit's steps, the step in it
  struct Place {
    int j, b, h, steps, off;
    // A cut one step from a unit's end is not worth a record: it moves there.
    __device__ int shift() const { return off == 1 ? -1 : (off > 0 && off == steps - 1 ? 1 : 0); }
  } at = {};

  __device__ Line(const ChunkArgs& args, int per_, int lane_) : a(args), per(per_), lane(lane_) {
    for (int i = 0; i < a.batch; i += 32) {
      group(i);
      for (int k = 0; k < ch.tiles; ++k) total += steps_of(a, ch, k, per);
      tiles_most = max(tiles_most, __reduce_max_sync(0xffffffffu, ch.tiles));
    }
    total = warp_sum(total) * a.c.n_kv;
  }
  __device__ void group(int first) {
    if (first == b0) return;
    b0 = first;
    ch = chunk_of(a, first + lane, per);
  }
  // Step x of the units of tile index j_ of the 32 sequences: `s` their steps, a lane each.
  __device__ Place locate(long long x, int j, int s) {
    int inc = s;   // below 32 * 2^24
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, x < static_cast<long long>(inc) * a.c.n_kv)) - 1;
    const int steps = __shfl_sync(0xffffffffu, s, src);
    x -= static_cast<long long>(__shfl_sync(0xffffffffu, inc, src) - steps) * a.c.n_kv;
    const int h = static_cast<int>(x / steps);
    return {j, b0 + src, h, steps, static_cast<int>(x - static_cast<long long>(h) * steps)};
  }
  // Goes to step x0 of the line, where its cut moves; x1, the next cut, moves too (x0 < x1 <= total).
  __device__ void go(long long& x0, long long& x1) {
    long long before = 0, end = x1;
    bool found = false, last = x1 >= total;
    for (int j = 0; j < tiles_most && !(found && last); ++j) {
      for (int i = 0; i < a.batch; i += 32) {
        group(i);
        const int s = steps_of(a, ch, j, per);
        const long long behind = before + static_cast<long long>(__reduce_add_sync(0xffffffffu, s)) * a.c.n_kv;
        if (!found && x0 < behind) {
          found = true;
          at = locate(x0 - before, j, s);
        }
        if (!last && x1 < behind) {
          last = true;
          end = x1 + locate(x1 - before, j, s).shift();
        }
        before = behind;
      }
    }
    x1 = end;
    const int by = at.shift();
    x0 += by;
    group(at.b & ~31);
    if (by < 0) at.off = 0;
    if (by > 0 && x0 < x1) next();
  }
  __device__ void next() {   // the next unit, from its first step (there is one)
    at.off = 0;
    if (++at.h < a.c.n_kv) return;
    at.h = 0;
    ++at.b;
    while (at.j < tiles_most) {
      for (int i = at.b & ~31; i < a.batch; i += 32) {
        group(i);
        const unsigned more = __ballot_sync(0xffffffffu, i + lane >= at.b && ch.tiles > at.j);
        if (more) {
          at.b = i + __ffs(more) - 1;
          at.steps = __shfl_sync(0xffffffffu, steps_of(a, ch, at.j, per), at.b & 31);
          return;
        }
      }
      at.b = 0;
      ++at.j;
    }
  }
};

template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads, 1) kv16_chunk_kernel(const ChunkArgs a) {
  constexpr bool kTwo = std::is_same<TO, float>::value;   // P in two parts
  extern __shared__ uint8_t s_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ Work s_work[2];
  __shared__ unsigned s_bad[4];   // a step's groups of 16 positions whose block id is bad
  __shared__ float2 s_pair[2][kRows];   // what the two threads of a row tell one another
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t base = (static_cast<uint32_t>(__cvta_generic_to_shared(s_raw)) + 1023u) & ~1023u;
  const uint32_t bars = base + kOffBar;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  if (threadIdx.x == 32) {
    for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i == kWEmpty0 || i == kWEmpty1 ? 19 : (i == kPFull0 || i == kPFull1 ? 8 : (i == kQFull ? 2 : 1)));
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(&s_tmem))) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  const int per = kRows / a.group;   // queries of a unit
  grid_dep_wait();
  grid_dep_launch();

  auto wait = [&](int b, uint32_t parity) {   // false: give up
    if (mbar_wait(bar(b), parity)) return true;
    b8_flag(a.status, TQ_DEV_TIMEOUT);
    return false;
  };
  auto warp_wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };   // one answer for the warp
  // A wait for a whole part of `steps` steps.
  auto long_wait = [&](int b, uint32_t parity, int steps) {
    const uint64_t t0 = global_ns(), most = kWaitNs + kStepNs * static_cast<uint64_t>(steps);
    bool ok;
    do {
      ok = mbar_try(bar(b), parity);
    } while (!ok && global_ns() - t0 < most);
    if (!ok) b8_flag(a.status, TQ_DEV_TIMEOUT);
    return __all_sync(0xffffffffu, ok) != 0;
  };

  if (warp < 16) {
    // ---- softmax: of tile warp / 8, two threads a row, for the left and the right 64 columns
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");   // 4 x 104 + 64 = 5 x 96 registers a thread
    const int t = warp >> 3, half = warp >> 2 & 1;
    const int pair = 1 + (t << 2 | (warp & 3));   // the barrier of this warp and the one of the other half
    const unsigned by_group = (65536u + a.group - 1) / a.group;   // row / group for rows below 256, group <= 8
    const int r = t * 128 + (warp & 3) * 32 + lane;   // this thread's row, 0 .. 255
    const int qi = static_cast<int>(r * by_group >> 16), head = r - qi * a.group;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + kColS + t * 128 + half * 64, t_o = tmem + lanes + kColO + t * 128 + half * 64;
    const float f = fmaxf(a.qscale, 0x1p-126f);   // never 0, which would make NaN of a masked place
    unsigned steps = 0, served = 0;   // of this tile so far
    int before = 0;
    bool ok = true;   // the same for both warps of a pair, so that neither waits for one that gave up
    for (unsigned part = 0; ok; ++part) {
      if (pair_any(pair, !long_wait(kWFull0 + (part & 1), part >> 1 & 1, before))) break;
      const Work w = s_work[part & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWEmpty0 + (part & 1)));
      if (w.seq < 0) break;
      before = w.tiles;
      auto zero_rows = [&](int q0, int count) {   // `count` queries from q0 on, this KV head's part
        const long long all = static_cast<long long>(count) * a.group * (kKvD / 4);
        for (long long i = threadIdx.x; i < all; i += 512) {
          const long long x = i / (kKvD / 4);
          write4<TO>(static_cast<TO*>(a.out) + ((q0 + x / a.group) * a.n_q + w.h * a.group + x % a.group) * kKvD + 4 * (i % (kKvD / 4)),
                     make_float4(0.f, 0.f, 0.f, 0.f));
        }
      };
      if (w.zeros) zero_rows(w.zero0, w.zeros);
      if (w.tiles == 0) {
        zero_rows(w.q0, w.rows / a.group);
        continue;
      }
      if (t * 128 >= w.rows) continue;
      const bool live = r < w.rows;
      const int vis = live ? max(min(w.pos0 + qi + 1, w.limit), 0) : 0;   // positions that this row sees
      const int vis_least = __reduce_min_sync(0xffffffffu, live ? vis : 0x7fffffff);
      float m = -1e30f, l = 0.f;   // l: sum of this thread's P
      for (int i = 0; i < w.tiles; ++i, ++steps) {
        const bool there = warp_wait(kSFull0 + t, steps & 1);
        fence_after();
        const int at = (w.tile0 + i) * kCols + half * 64;
        const unsigned bad = s_bad[(w.step0 + i) & 3] >> 4 * half & 15;
        const bool masked = bad || at + 64 > vis_least;
        auto mask = [&](float (&s)[16], int c) {
          if (__builtin_expect(masked, 0)) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (at + 16 * c + j >= vis || (bad >> c & 1)) s[j] = -INFINITY;
          }
        };
        uint32_t p[kTwo ? 64 : 32];   // 64 positions; in two parts: of each 32 the hi parts, then the lo parts
        float2 x0, x1;
        auto weigh = [&](const float (&s)[16], int c) {   // the P of 16 positions, added to the sums
          const float a0 = 3.f - m;
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            float2 y0 = fma2(make_float2(s[j], s[j + 1]), make_float2(f, f), make_float2(a0, a0));
            float2 y1 = fma2(make_float2(s[j + 2], s[j + 3]), make_float2(f, f), make_float2(a0, a0));
            y0.x = ex2(y0.x);
            y0.y = ex2(y0.y);
            y1.x = ex2(y1.x);
            y1.y = ex2(y1.y);
            x0 = add2(x0, y0);
            x1 = add2(x1, y1);
            if constexpr (kTwo) {
              const int k = 32 * (c >> 1) + 8 * (c & 1) + j / 2;
              p[k] = take_pair<T>(y0.x, y0.y);
              p[k + 1] = take_pair<T>(y1.x, y1.y);
              p[k + 16] = to_pair<T>(y0.x, y0.y);
              p[k + 17] = to_pair<T>(y1.x, y1.y);
            } else {
              p[8 * c + j / 2] = to_pair<T>(y0.x, y0.y);
              p[8 * c + j / 2 + 1] = to_pair<T>(y1.x, y1.y);
            }
          }
        };
        auto weigh_all = [&]() {
          x0 = x1 = make_float2(0.f, 0.f);
          float s[16], z[16];
          load16(t_s, s);
          wait_ld(s);
          load16(t_s + 16, z);
          mask(s, 0);
          weigh(s, 0);
          wait_ld(z);
          load16(t_s + 32, s);
          mask(z, 1);
          weigh(z, 1);
          wait_ld(s);
          load16(t_s + 48, z);
          mask(s, 2);
          weigh(s, 2);
          wait_ld(z);
          mask(z, 3);
          weigh(z, 3);
          x0 = add2(x0, x1);
          return x0.x + x0.y;
        };
        float sum;
        for (int go = 0;; ++go) {   // once, but for rows that outgrow their m
          sum = weigh_all();
          if (go) break;
          const bool over = !(sum <= kMost);   // NaN too
          if (__builtin_expect(!pair_any(pair, over || !there), 1)) break;
          if (pair_any(pair, !there)) {
            ok = false;
            break;
          }
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float s[16];
            load16(t_s + 16 * c, s);
            wait_ld(s);
            mask(s, c);
#pragma unroll
            for (int j = 0; j < 16; ++j) top = fmaxf(top, s[j]);
          }
          s_pair[half][r] = make_float2(top * f, over ? 1.f : 0.f);
          pair_any(pair, false);
          const float2 other = s_pair[half ^ 1][r];
          const float u = over || other.y != 0.f ? fmaxf(m, fmaxf(top * f, other.x)) : m, e = ex2(m - u);
          m = u;
          l *= e;
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float o[16];
              load16(t_o + 16 * c, o);
              wait_ld(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= e;
              tmem_st16(t_o + 16 * c, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
        if (!ok) break;
        l += sum;
        // where these columns of S stood
        tmem_st32(t_s, p);
        if constexpr (kTwo) tmem_st32(t_s + 32, p + 32);
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull0 + t));
      }
      if (!ok) break;
      const bool there = warp_wait(kODone0 + t, served++ & 1);
      fence_after();
      s_pair[half][r].x = l;
      if (pair_any(pair, !there)) break;
      l += s_pair[half ^ 1][r].x;
      pair_any(pair, false);   // read before it is written again
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays
      const bool whole = w.slot < 0;
      const bool wide = ((whole ? reinterpret_cast<uintptr_t>(a.out) : reinterpret_cast<uintptr_t>(a.rec_o)) & 31) == 0;
      const long long orow = static_cast<long long>(w.q0 + qi) * a.n_q + w.h * a.group + head;
      const long long rec = static_cast<long long>(w.slot) * a.part_rows + r;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {   // 32 bytes a store: whole sectors, though a row a thread
        float o[32];
        load32(t_o + 32 * c, o);
        wait_ld(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = l == 0.f ? 0.f : o[j] * inv;
        if (live) {
          if (whole) write32<TO>(static_cast<TO*>(a.out) + orow * kKvD + half * 64 + 32 * c, o, wide);
          else write32<float>(a.rec_o + rec * kKvD + half * 64 + 32 * c, o, wide);
        }
      }
      if (live && !whole && half == 0) a.rec_lse[rec] = l == 0.f ? -INFINITY : m - 3.f + __log2f(l);
    }
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
  if (warp == 16) {
    // ---- products. The whole warp walks the steps, so that descriptors and addresses
    // stay in uniform registers; one lane, always the same, issues.
    const bool leader = elect_one();
    auto qk = [&](int t, int st) {
      const uint64_t q_at = desc_q(base + t * kTileOp), k_at = desc_k(base + kOffK + st * kTileOp);
      const uint32_t d = tmem + kColS + t * 128;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ss(d, q_at + (((k >> 2) * kHalfQ + (k & 3) * 32) >> 4), k_at + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), idesc_qk<T>(), k > 0);
      mma_commit(bar(kSFull0 + t));
    };
    unsigned step = 0, filled = 0;   // steps and loaded queries so far
    unsigned weighed[2] = {0, 0};    // steps of each tile
    int before = 0;
    bool ok = true;
    for (unsigned part = 0; ok; ++part) {
      if (!(ok = long_wait(kWFull0 + (part & 1), part >> 1 & 1, before))) break;
      const int seq = s_work[part & 1].seq, tiles = s_work[part & 1].tiles, halves = s_work[part & 1].rows > 128 ? 2 : 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWEmpty0 + (part & 1)));
      if (seq < 0) break;
      before = tiles;
      if (tiles == 0) continue;
      if (!(ok = warp_wait(kQFull, filled++ & 1) && warp_wait(kKFull0 + (step & 1), step >> 1 & 1))) break;
      fence_after();
      if (leader) {
        for (int t = 0; t < halves; ++t) qk(t, step & 1);
        mma_commit(bar(kKEmpty0 + (step & 1)));
        if (tiles == 1) mma_commit(bar(kQEmpty));
      }
      __syncwarp();
      for (int i = 0; i < tiles && ok; ++i, ++step) {
        const int st = step & 1, nst = st ^ 1;
        const bool more = i + 1 < tiles;
        for (int t = 0; t < halves; ++t) {
          if (!(ok = warp_wait(kPFull0 + t, weighed[t]++ & 1))) break;
          if (t == 0 && !(ok = warp_wait(kVFull0 + st, step >> 1 & 1))) break;
          fence_after();
          if (leader) {
            const uint64_t v_at = desc_v(base + kOffV + st * kTileOp);
            const uint32_t d = tmem + kColO + t * 128, p = tmem + kColS + t * 128;
            mma_ts(d, p, v_at, idesc_pv<T>(), i > 0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {   // 16 positions: 8 columns
              const uint64_t vk = v_at + (4096 >> 4) * k;
              if constexpr (kTwo) {
                const uint32_t pk = p + 32 * (k >> 1) + 8 * (k & 1);
                if (k > 0) mma_ts(d, pk, vk, idesc_pv<T>(), true);
                mma_ts(d, pk + 16, vk, idesc_pv<T>(), true);
              } else {
                if (k > 0) mma_ts(d, p + 64 * (k >> 2) + 8 * (k & 3), vk, idesc_pv<T>(), true);
              }
            }
            if (!more) mma_commit(bar(kODone0 + t));
            if (t + 1 == halves) mma_commit(bar(kVEmpty0 + st));
          }
          __syncwarp();
          if (more) {
            if (t == 0 && !(ok = warp_wait(kKFull0 + nst, (step + 1) >> 1 & 1))) break;
            fence_after();
            if (leader) {
              qk(t, nst);
              if (t + 1 == halves) {
                mma_commit(bar(kKEmpty0 + nst));
                if (i + 2 == tiles) mma_commit(bar(kQEmpty));
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (!ok) {   // gave up: the products in flight come to rest before their memory goes
      if (leader) mma_commit(bar(kEnd));
      warp_wait(kEnd, 0);
    }
    __syncwarp();
  } else if (warp == 17) {
    // ---- the work, keys and values
    Line line(a, per, lane);
    const long long cut = line.total / 2;   // two steps a CTA at least
    const long long ctas = cut < 1 ? 1 : (cut < gridDim.x ? cut : gridDim.x);
    long long x = 0, end = 0;
    if (blockIdx.x < ctas && line.total > 0) {
      x = line.total * blockIdx.x / ctas;
      end = line.total * (blockIdx.x + 1) / ctas;
      line.go(x, end);
    }
    if (a.may_split && lane == 0) a.split_units[blockIdx.x] = make_int4(0, 0, 0, 0);
    const unsigned group16 = lane & 7;
    unsigned step = 0;
    int before = 0, before2 = 0;   // steps of the parts that the slot's last reader may be at
    bool ok = true;
    for (unsigned part = 0;; ++part) {
      if (!(ok = long_wait(kWEmpty0 + (part & 1), (part >> 1 & 1) ^ 1, before + before2))) break;
      Work w = {};
      w.seq = -1;
      if (x < end) {
        const int src = line.at.b & 31;
        Chunk ch;
        ch.q0 = __shfl_sync(0xffffffffu, line.ch.q0, src);
        ch.n = __shfl_sync(0xffffffffu, line.ch.n, src);
        ch.len = __shfl_sync(0xffffffffu, line.ch.len, src);
        const int served = min(ch.n, a.max_q_len), first = line.at.j * per;
        const long long left = end - x;
        const int steps = left < line.at.steps - line.at.off ? static_cast<int>(left) : line.at.steps - line.at.off;
        w.seq = line.at.b;
        w.h = line.at.h;
        w.q0 = ch.q0 + first;
        w.rows = min(per, served - first) * a.group;
        w.pos0 = ch.len - ch.n + first;
        w.limit = limit_of(a, ch, line.at.j, per);
        w.tile0 = line.at.off;
        w.tiles = w.limit == 0 ? 0 : steps;
        w.slot = line.at.off > 0 ? 2 * static_cast<int>(blockIdx.x) : (steps < line.at.steps ? 2 * static_cast<int>(blockIdx.x) + 1 : -1);
        w.zero0 = ch.q0 + served;
        w.zeros = line.at.j == 0 && line.at.off == 0 ? ch.n - served : 0;   // queries past max_q_len
        w.step0 = step;
        if (line.at.j == 0 && line.at.off == 0 && line.at.h == 0 && lane == 0 && (ch.n > a.max_q_len || ch.len > a.limit))
          b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
        if (line.at.off == 0 && steps < line.at.steps && lane == 0) {
          // who has the unit's last step, unless the cut before that one moved behind it
          const long long last = x + line.at.steps;
          long long owner = (last * ctas - 1) / line.total;
          if (last - line.total * owner / ctas < 2) --owner;
          a.split_units[blockIdx.x] = make_int4(w.q0, w.rows, w.h * a.group, static_cast<int>(owner) - blockIdx.x + 1);
        }
        x += steps;
      }
      if (lane == 0) s_work[part & 1] = w;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWFull0 + (part & 1)));
      if (w.seq < 0) break;
      before2 = before;
      before = w.tiles;
      // the block of this lane's group of 16 positions of step i (-1: behind the end)
      const int* table = a.block_table + static_cast<long long>(w.seq) * a.c.bt_stride;
      auto block_of = [&](int i) {
        const int g16 = (w.tile0 + i) * 8 + group16;
        return ldg_or(table + (g16 >> (a.c.log2_bs - 4)), i < w.tiles && g16 * 16 < w.limit, -1);
      };
      int blk = block_of(0);
      for (int i = 0; i < w.tiles; ++i, ++step) {
        const int st = step & 1;
        const uint32_t free_phase = (step >> 1 & 1) ^ 1;
        const int blk_next = block_of(i + 1);
        const int g16 = (w.tile0 + i) * 8 + group16;
        const bool inside = g16 * 16 < w.limit, good = inside && a.c.good(blk);
        const uint8_t* src = a.c.tile(good ? blk : 0, w.h, g16);
        const int rows = good ? min(w.limit - g16 * 16, kKvRows) : 0;   // of values: rows behind the end may hold anything
        const unsigned all = __ballot_sync(0xffffffffu, good) & 0xffu, bad = __ballot_sync(0xffffffffu, inside && !good) & 0xffu;
        const unsigned ragged = __ballot_sync(0xffffffffu, rows < kKvRows) & 0xffu;
        if (bad && lane == 0) b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
        if (!(ok = warp_wait(kKEmpty0 + st, free_phase))) break;
        const uint32_t k_to = base + kOffK + st * kTileOp + group16 * kKvHalfBytes, v_to = base + kOffV + st * kTileOp;
        if (lane == 0) {
          s_bad[step & 3] = bad;
          mbar_expect(bar(kKFull0 + st), __popc(all) * kKvHalfBytes);
        }
        __syncwarp();
        if (lane < 8 && good) bulk_g2s_plain(k_to, src, kKvHalfBytes, bar(kKFull0 + st));
        if (!(ok = warp_wait(kVEmpty0 + st, free_phase))) break;
        uint32_t bytes = __popc(all) * kKvHalfBytes;
        if (__builtin_expect(ragged, 0)) {   // their rows that are not loaded are 0: no weight takes NaN along
          bytes = 0;
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const int have = __shfl_sync(0xffffffffu, rows, g);
            bytes += have * 256;
            for (int k = lane; k < 256 && have < kKvRows; k += 32)
              if ((k >> 7) * 8 + (k >> 3 & 7) >= have)
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(v_to + g * kKvHalfBytes + 16 * k), "r"(0u) : "memory");
          }
          fence_smem_async();
          __syncwarp();
        }
        if (lane == 0) mbar_expect(bar(kVFull0 + st), bytes);
        __syncwarp();
        if (lane < 8 && rows > 0) {
          const uint32_t to = v_to + group16 * kKvHalfBytes;
          const uint8_t* from = src + kKvHalfBytes;
          if (rows == kKvRows) {
            bulk_g2s_plain(to, from, kKvHalfBytes, bar(kVFull0 + st));
          } else {   // whole groups of 8 rows, then the rows of one group, half by half
            const int whole = rows >> 3 << 11, rest = (rows & 7) * 128;
            if (whole) bulk_g2s_plain(to, from, whole, bar(kVFull0 + st));
            if (rest) {
              bulk_g2s_plain(to + whole, from + whole, rest, bar(kVFull0 + st));
              bulk_g2s_plain(to + whole + 1024, from + whole + 1024, rest, bar(kVFull0 + st));
            }
          }
        }
        __syncwarp();
        blk = blk_next;
      }
      if (!ok) break;
      if (x < end) line.next();
    }
    // the copies in flight end before their memory goes
    for (unsigned k = step > 2 ? step - 2 : 0; k < step; ++k) {
      warp_wait(kKFull0 + (k & 1), k >> 1 & 1);
      warp_wait(kVFull0 + (k & 1), k >> 1 & 1);
    }
  } else {
    // ---- queries: half a warp a row, as they are
    unsigned filled = 0;
    const unsigned by_group = (65536u + a.group - 1) / a.group;
    int before = 0;
    bool ok = true;
    for (unsigned part = 0; ok; ++part) {
      if (!(ok = long_wait(kWFull0 + (part & 1), part >> 1 & 1, before))) break;
      const int seq = s_work[part & 1].seq, tiles = s_work[part & 1].tiles, rows = s_work[part & 1].rows, q0 = s_work[part & 1].q0;
      const int head0 = s_work[part & 1].h * a.group;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWEmpty0 + (part & 1)));
      if (seq < 0) break;
      const int wait_for = before;
      before = tiles;
      if (tiles == 0) continue;
      if (!(ok = long_wait(kQEmpty, (filled++ & 1) ^ 1, wait_for))) break;
      const int c = lane & 15, last = rows > 128 ? kRows : 128;
#pragma unroll 8
      for (int r = 2 * (warp - 18) + (lane >> 4); r < last; r += 4) {
        const int qi = static_cast<int>(r * by_group >> 16), head = head0 + r - qi * a.group;
        const T* src = static_cast<const T*>(a.q) + (r < rows ? (q0 + qi) * a.q_stride + static_cast<long long>(head) * kKvD + 8 * c : 0);
        const uint32_t to = base + (r >> 7) * kTileOp + (c >> 3) * kHalfQ + (r & 127) * 128 + (((c ^ r) & 7) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(src), "r"(r < rows ? 16 : 0) : "memory");
      }
      asm volatile("cp.async.wait_all;\n" ::: "memory");
      fence_smem_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull));
    }
  }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
}

// Merges the parts of split units: a warp a row, 8 rows of a unit a CTA.
template <typename TO>
__global__ void __launch_bounds__(256) kv16_chunk_merge_kernel(const ChunkArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_unit = (a.part_rows + 7) / 8;
  const int u = blockIdx.x / per_unit, r = (blockIdx.x - u * per_unit) * 8 + warp;
  grid_dep_wait();
  grid_dep_launch();
  const uint4 unit = ld_dep_u32x4(a.split_units + u);   // first row, rows, first head, parts
  const int parts = unit.w;
  if (r >= static_cast<int>(unit.y) || parts == 0) return;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int z0 = 0; z0 < parts; z0 += 8) {   // eight parts' records on their way at once
    float lse[8];
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int z = z0 + k;
      const long long rec = static_cast<long long>(z == 0 ? 2 * u + 1 : 2 * (u + z)) * a.part_rows + r;
      lse[k] = z < parts ? ld_dep_f32(a.rec_lse + rec) : -INFINITY;
      x[k] = z < parts ? ld_dep_f32x4(reinterpret_cast<const float4*>(a.rec_o + rec * kKvD) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (lse[k] == -INFINITY) continue;   // nothing seen there
      const float top = fmaxf(m, lse[k]);
      const float e = m == -INFINITY ? 0.f : exp2f(m - top), f = exp2f(lse[k] - top);
      m = top;
      l = l * e + f;
      o.x = o.x * e + x[k].x * f;
      o.y = o.y * e + x[k].y * f;
      o.z = o.z * e + x[k].z * f;
      o.w = o.w * e + x[k].w * f;
    }
  }
  const float s = l == 0.f ? 0.f : 1.f / l;
  const long long orow = (static_cast<long long>(unit.x) + r / a.group) * a.n_q + unit.z + r % a.group;
  write4<TO>(static_cast<TO*>(a.out) + orow * kKvD + 4 * lane, make_float4(o.x * s, o.y * s, o.z * s, o.w * s));
}

// The grid, and the workspace that split units take.
struct Plan {
  long long units;   // (tile of queries, KV head), at most
  int may_split, part_rows;
  size_t workspace;
};
Plan plan_for(const tq_config* cfg, int batch, int total_q, int max_q_len, int max_seq_len) {
  Plan p;
  const int group = cfg->num_q_heads / cfg->num_kv_heads, per = kRows / group;
  const int longest = max_q_len < total_q ? max_q_len : total_q;
  // tiles of queries: a full one for every `per` rows at most, and one more for every
  // chunk; as many for every sequence as the longest chunk has at most
  const long long most = static_cast<long long>(batch) * ((longest + per - 1) / per);
  long long tiles = static_cast<long long>(total_q) / per + (batch < total_q ? batch : total_q);
  if (tiles > most) tiles = most;
  p.units = tiles * cfg->num_kv_heads;
  p.may_split = p.units > 0 && max_seq_len > 3 * kCols;   // a unit of three steps has no cut that stays where it is
  p.part_rows = longest < per ? longest * group : per * group;
  const size_t records = static_cast<size_t>(2 * kCtas) * p.part_rows;
  p.workspace = p.may_split ? (kCtas * sizeof(int4) + records * (kKvD + 1) * sizeof(float) + 15) / 16 * 16 : 16;
  return p;
}

template <typename T, typename TO>
cudaError_t launch(const ChunkArgs& a, const Plan& p, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0, sms = 0;
  cudaError_t err = b8_current_device(&dev, &sms);
  if (err == cudaSuccess) err = b8_allow_smem(kv16_chunk_kernel<T, TO>, kSmem, dev, &done);
  if (err != cudaSuccess) return err;
  const int ctas = sms < kCtas ? sms : kCtas;
  // starts that go backwards may name more units than these: they are served all the same
  const long long steps = p.units * ((static_cast<long long>(a.limit) + kCols - 1) / kCols + 1);
  const int grid = steps / 2 + 1 < ctas ? static_cast<int>(steps / 2 + 1) : ctas;
  err = launch_pdl(kv16_chunk_kernel<T, TO>, dim3(grid), dim3(kThreads), kSmem, s, a);
  if (err != cudaSuccess || !p.may_split) return err;
  return launch_pdl(kv16_chunk_merge_kernel<TO>, dim3(grid * ((p.part_rows + 7) / 8)), dim3(256), 0, s, a);
}
template <typename T>
cudaError_t launch(const ChunkArgs& a, const Plan& p, int out_dtype, cudaStream_t s) {
  if (out_dtype == TQ_DTYPE_F32) return launch<T, float>(a, p, s);
  if (out_dtype == TQ_DTYPE_F16) return launch<T, __half>(a, p, s);
  return launch<T, __nv_bfloat16>(a, p, s);
}

}  // namespace
}  // namespace tq

extern "C" {

size_t tq_kv16_continue_workspace_size(const tq_config* cfg, int batch, int total_q, int max_q_len, int max_seq_len) {
  using namespace tq;
  tq_kv16_layout L;
  if (make_kv16_layout(cfg, &L) != TQ_OK || batch < 0 || total_q < 0 || max_q_len < 0 || max_seq_len < 0) return 0;
  if (b8_heads(cfg) != TQ_OK) return 0;
  return plan_for(cfg, batch, total_q, max_q_len, max_seq_len).workspace;
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
  const Plan p = plan_for(cfg, batch, total_q, max_q_len, max_seq_len);
  if (workspace_bytes < p.workspace) return TQ_ERR_WORKSPACE_TOO_SMALL;
  if (static_cast<long long>(total_q) * cfg->num_q_heads > INT_MAX) return TQ_ERR_UNSUPPORTED;
  const int cap = b8_cap(cfg, bt_stride);
  ChunkArgs a = {};
  a.c = kv16_cache(cfg, L, cache, num_blocks, bt_stride);
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
  a.limit = max_seq_len < cap ? max_seq_len : cap;
  a.may_split = p.may_split;
  a.part_rows = p.part_rows;
  a.qscale = b8_qscale(scale);
  a.split_units = static_cast<int4*>(workspace);
  a.rec_o = reinterpret_cast<float*>(a.split_units + kCtas);
  a.rec_lse = a.rec_o + static_cast<size_t>(2 * kCtas) * p.part_rows * kKvD;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = L.is_bf16 ? launch<__nv_bfloat16>(a, p, out_dtype, s) : launch<__half>(a, p, out_dtype, s);
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
