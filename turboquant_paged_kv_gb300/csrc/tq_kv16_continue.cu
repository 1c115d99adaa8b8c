// tq_kv16_continue: causal attention of chunks of queries over the 16-bit cache,
// on tcgen05 tensor cores.
//
//   out_i = sum_p softmax_p(scale q_i . k_p) v_p, p <= position of i
//
// Work. A unit is 512 rows (the query heads of one KV head of 512 / group consecutive
// queries) of a pair of CTAs, or 256 of one, in two tiles of 128 rows a CTA, against
// all positions that they see, in steps of 128. The steps of all units form one line,
// cut by their cost into as many parts as there are teams of CTAs on the GPU, whatever
// the lengths are; a unit that a cut goes through leaves records, which a second
// kernel merges. A team walks its part of the line with one pipeline: the loads of a
// unit's first steps and its queries come while the last of the unit before are
// worked on. Few queries are not worth that: they run as rows of their own on the
// decode's short kernel.
//
// Math, per tile t and half a step (64 positions):
//   S_t = Q_t K^T      tcgen05.mma, A and B from shared memory
//   P_t = 8 p          a row a thread, S read from tensor memory
//   O_t += P_t V       A = P_t from tensor memory (it takes S_t's place), B = V
// S is double: the scores are issued two halves ahead, behind the product that frees
// their place, so the softmax finds the next ones there.
// p = 2^(score - m): no maximum is sought but in a part's first half. The weights are
// taken with the maximum so far, and a row of which some P would not fit in fp16 shows
// in its sum; only then the row's new m is found and what was accumulated (by the
// softmax warps, in tensor memory) rescaled. m is the row's own, at most its largest
// score so far, so the largest P of a row is 8 or more, and no position behind the
// row's own changes a bit of it. P is rounded to the cache's type (bf16: by 2^-8, fp16:
// by 2^-11 and no finer than 2^-25), as a 16-bit output is: against 64 bits, 2.3e-3
// instead of the output's own 1.7e-3 in bf16, 2.9e-4 instead of 2.1e-4 in fp16. With
// f32 output it is held in two parts (bf16 2^-16, fp16 2^-22), for twice the products
// of P V. The tensor cores cut what they add to O off rather than round it, about 2^-25 of
// O each time: with f32 output no more than kPiece steps are summed there, and the pieces
// of a unit joined in fp32 (against 64 bits, over 16384 positions: 6.5e-6, else 3.6e-5).
//
// A pair of CTAs shares one tile of keys and values (cta_group::2: each loads half of
// the keys' positions and half of the values' coordinates). A CTA alone needs all of
// shared memory's rate for it: of a step's 2048 cycles of products, 1024 go to reading
// Q and K, 512 to V, 512 to loading both.
//
// Warps: 0-3 and 4-7 the softmax of tile 0 and 1; 8 and 9 issue the products of tile 0
// and 1 (of both CTAs of a pair, in its first), in turn, so that the two tiles stay half
// a round apart; 10 finds the work and loads keys and values; 11, in the second CTA of
// a pair, tells the first what has come, and in the first writes the zeros of queries past
// max_q_len; 12-15 load queries. Keys and values come by bulk copies: they lie in the cache
// as the tensor cores read them (128-byte swizzle; K a K-major operand, V an MN-major one).
// Every wait is bounded; one that runs out sets TQ_DEV_TIMEOUT and ends the CTA, after its
// products and copies in flight.
//
// Bound: tensor cores by its operations. 4 chunks of 2001-2048 queries over 0-6144, 32
// query heads, fp16: 540 us, 1570 TFLOP/s, 0.83 of a measured bf16 GEMM (592 us, 1432,
// over seconds, where the power limit takes the clock to 1.7 GHz); 32 chunks of 128 over
// 4096, bf16: 197 us, 1417 (212 us); 12 of 1-500 over 0-16384, 64 heads: 405 us, 1325.
// A step of two tiles takes about 2800 cycles, 2304 of them products (64 a product,
// 40 instead of 32 where only 64 positions stand against Q). Steps that led here, on the
// second case: one CTA, a warp that issues for both tiles, S single 237 us; two threads a
// row 236; pairs of CTAs 249, with S double 237; an issuing warp a tile 214; in turn, with
// one barrier a load, 211; a line cut by cost, two-part merges 209; rows by way of shared
// memory 202; queries asked for early 199; the merge dealt evenly 197. Tried and left out: S of the next half loaded
// into registers before P is handed over (222 for 214), the turn given before the last
// products are issued (202 for 199), 5 stages for a pair (223 for 222 over seconds).
#include <climits>

#include "tq_attn.cuh"
#include "tq_chunk_cost.h"
#include "tq_kv16.cuh"
#include "tq_tc.cuh"

namespace tq {
namespace {

constexpr int kRows = 256;             // of a unit, a CTA: two tiles of 128
constexpr int kCols = kChunkCols;      // positions a step, in two halves
constexpr int kThreads = 512;
constexpr int kCtas = 152;             // grid, one an SM: sizes the workspace without a device query
constexpr float kMost = 60000.f;       // sums of P up to this: every P fits in fp16
constexpr uint32_t kTileOp = 32768;    // a 128 x 128 operand
constexpr uint32_t kHalfQ = 16384;     // Q: two halves of 64 columns, 128 bytes a row
constexpr uint32_t kStage = 32768;     // what is loaded at once: 16 KB of keys, then 16 KB of values
// behind Q and the stages: room for a pair's output, or one more stage for one CTA, whose few rows wait for loads (32 x 5
// queries over 4096: 102 us with 5 stages, 120 with 4; f32 output, which is read again by the next piece, has the room)
constexpr uint32_t kOffLoads = 2 * kTileOp, kOffOut = kOffLoads + 4 * kStage, kOffBar = kOffOut + kStage;
constexpr uint32_t kSmem = kOffBar + 512 + 1024;   // and room to align to 1024
constexpr int kBad = 16;               // loads whose bad blocks are remembered (more than are between the loads and the softmax)
constexpr uint32_t kColS = 0, kColO = 256;         // tensor memory columns: two halves' S of each tile, O of each tile
// Rows a chunk, on average, above which pairs of CTAs are used: 16 x 96 queries of 32 heads over 8192 (384 rows) 193 us for
// 217, 16 x 64 (256) 150 for 135, where a pair's units are half empty
constexpr int kPairRows = 256;
// Up to which tiles a warp (tq_kv16.cuh) queries are rows of their own, by CTAs of 8 warps, and of 4 or 2: 1 x 64 over
// 2000 of 2 heads (16 tiles a warp of 8) 12.4 us for 19.3, 1 x 16 over 4000 (31) 20.9 for 17.9; 3 x 7 over 400 of 8 (7 of 4)
// 8.4 for 13.6, over 1000 (16) 13.2 for 20.0, over 1400 (22) 16.5 for 15.8; 6 x 12 over 300
// of 8 (10 of 2) 10.6 for 12.3, over 600 (19) 15.9 for 16.1
constexpr int kShortMost = 19, kShortMostSmall = 20;
// Steps of the longest history up to which units are not cut: so many are done while records are written and merged. (One
// chunk of 416 over 445, 3 heads: 16.4 us whole, 19.7 cut; 4 of 50-150 over 97-391, 6 heads of 8: 19.7 and 26.2; 7 of 40-120
// over 218-872, one head: 18.0 and 19.5; with 12: 2 of 364-1093 over few, 4 heads: 25.6, with 8 22.1.)
constexpr int kNoSplit = 8;
constexpr int kMergeThreads = 256, kMergeCtas = 3;   // an SM, of the merge: with 8 (2.7 waves of what fits) 32 x 128 takes 208 us for 197
constexpr int kPiece = 20;                         // steps; 32 x 128 over 4096, f32: 294 us, with 16 311, with 24 294, in one piece 276
constexpr unsigned long long kStepNs = 100000;     // what a step may take, where a wait is for many; and the search for work among 32 sequences or 512 tile indexes

struct ChunkArgs {
  Kv16Cache c;
  const void* q;
  long long q_stride;
  const int *block_table, *seq_lens, *query_start;
  unsigned int* status;
  void* out;
  // team i's unit that others go on with: first row, rows, first head, parts (0: none);
  // record 2 i is what it adds to a unit that others began, 2 i + 1 the first part of
  // one that others go on with: [part_rows][d] and [part_rows] (log2 units)
  int4* split_units;
  float *rec_o, *rec_lse;
  int batch, total_q, max_q_len, n_q, group, limit, may_split, part_rows;   // limit: positions at most
  float qscale;                        // softmax scale * log2(e)
  unsigned long long search_ns;        // a wait's, with the search for work
};

// barriers, 8 bytes each from kOffBar
enum {
  kWFull0, kWFull1, kWEmpty0, kWEmpty1, kQFull, kQEmpty, kODone0, kODone1, kEnd0, kEnd1, kTurn0, kTurn1, kSFull0, kPFull0 = kSFull0 + 4,
  kFull0 = kPFull0 + 4, kEmpty0 = kFull0 + 5, kBars = kEmpty0 + 5
};
static_assert(kBars * 8 <= 512, "barriers");

// The stage of a load and its round through the stages.
template <int kStages>
struct Turn {
  int stage = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      round ^= 1;
    }
  }
};

// shared-memory operand descriptors, 128-byte swizzle. Q: 8-row groups 1024 bytes
// apart; K: 2048 (its halves lie 1024 behind); V: halves 1024 apart, groups 2048 (a pair:
// one half, groups 1024 apart).
__device__ __forceinline__ uint64_t desc_q(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1ull << 16) | (128ull << 32) | (1ull << 46) | (2ull << 61);
}
template <int CTAS>
__device__ __forceinline__ uint64_t desc_v(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (64ull << 16) | ((CTAS == 2 ? 64ull : 128ull) << 32) | (1ull << 46) | (2ull << 61);
}
// f16 x f16 or bf16 x bf16 -> f32, M = 128 a CTA, N = 64 positions or 128 coordinates
template <typename T, int CTAS>
__device__ __forceinline__ constexpr uint32_t idesc_qk() {
  return (1u << 4) | (std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u) | ((64u / 8) << 17) | ((CTAS * 128u / 16) << 24);
}
template <typename T, int CTAS>
__device__ __forceinline__ constexpr uint32_t idesc_pv() { return idesc_qk<T, CTAS>() + ((64u / 8) << 17) + (1u << 16); }   // B is MN-major

// Waits for the loads from tensor memory; what they brought is not used before.
__device__ __forceinline__ void wait_ld(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]),
                 "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]),
                 "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]),
                 "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])::"memory");
}
__device__ __forceinline__ void load32(uint32_t addr, float (&r)[32]) { tmem_ld32(addr, reinterpret_cast<uint32_t*>(r)); }

// mbar_try without a wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}

// A part of a unit, as a CTA works on it.
struct Work {
  int seq, h;          // sequence (-1: the end), KV head
  int slot;            // its record (-1: the whole unit)
  int q0, rows;        // row of its first query in q and out; rows of A, its queries' heads
  int pos0;            // position of that query (may be negative)
  int limit;           // positions that its last query sees: what stands behind them need not have been stored
  int tile0, tiles;    // steps: [tile0, tile0 + tiles); none: zeros are written
  int halves;          // of them, those that anybody sees
  int loads;           // that bring them: CTAS halves each
  int more, keep;      // this team's steps of the unit before tile0 are there already, where these come to be; the queries stay for the next part
  unsigned load0;      // loads of the CTA before
};

// A sequence's chunk: its first row, queries and length.
struct Chunk {
  int q0, n, len;
};
__device__ __forceinline__ Chunk chunk_of(const ChunkArgs& a, int q0, int q1, int len) {
  Chunk c;
  c.q0 = min(max(q0, 0), a.total_q);
  c.n = min(max(q1, c.q0), a.total_q) - c.q0;
  c.len = max(len, 0);
  return c;
}
__device__ __forceinline__ ChunkSize size_of(const ChunkArgs& a, const Chunk& c) { return {c.len - c.n, min(c.n, a.max_q_len)}; }
__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The line: for each tile index j, each sequence that has such a tile, each KV head,
// the cost of the unit (tq_chunk_cost.h). (Units that read the same keys and values, tiles of one chunk,
// are then a fixed part of the line apart, so that teams of CTAs meet them at the same
// time where chunks are alike.) A warp finds its places, the lanes together, a sequence a lane.
// MANY: more than 32 sequences. These are read once, into shared memory that no load has
// come to yet (up to kKept; behind these they are read anew whenever they are asked for). Where there
// are more than kClose tile indexes, a place's is found by bisection, from what all sequences cost up
// to one, and a walk over the last few; groups of 32 without a chunk of so many tiles are passed
// over. (4095 sequences of one query and one of 131072, 8 heads: at most 17 sums over 128
// groups. A walk over tile indexes and groups, each a round trip to L2, took 2048 x 128 of
// these, 45 ms at the least, which outlasts the other warps' waits; 512 with one of 16384, one KV head: 507 us for
// 2089, 256 with one of 8192, 8 KV heads: 1768 for 2026.) With up to 32 a walk over tile indexes alone is soon over,
// and a kernel without the rest starts sooner: 7 chunks of one query and one of 300, 13.0 us for 14.3.
template <bool MANY>
struct Line {
  static constexpr int kKept = 4 * kStage / 8;
  static constexpr int kClose = 8;   // tile indexes that are walked: a sum for one takes several times as long as going on by one
  const ChunkArgs& a;
  const ChunkCall call;
  int lane, tiles_most = 0;
  uint32_t kept;       // shared memory: (first position, queries served) of the first kKept sequences
  int span = 0;        // 2^span groups of 32 sequences a lane: the most tiles of a chunk there
  int most = 0;
  long long total = 0;
  int b0 = -1;
  Chunk ch = {};       // lane's chunk of the 32 from b0 on
  // a unit's tile, sequence and head, steps, what each costs, and where on the line it begins
  struct Unit {
    int j, b, h, steps, each;
    long long base;
    __device__ long long behind() const { return base + static_cast<long long>(steps) * each + kChunkUnit; }
    // The step where a cut at x (within the unit) comes to be. Fewer than `least` steps from an end are not worth a record:
    // the cut moves there.
    __device__ int step_of(long long x, int least) const {
      const int s = static_cast<int>(static_cast<unsigned>(x - base) / static_cast<unsigned>(each));   // x - base: at most a unit's cost
      return s < min(least, steps) ? 0 : s > steps - least ? steps : s;
    }
  } at = {};
  int least = 1;

  __device__ Line(const ChunkArgs& args, const ChunkCall& call_, uint32_t room, int lane_) : a(args), call(call_), lane(lane_), kept(room) {
    if constexpr (MANY) {
      while ((a.batch - 1) >> 5 >> span >= 32) ++span;
      for (int i = 0; i < min(a.batch, kKept); i += 128) {   // four round trips in one
        int q0[4], q1[4], len[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) read(i + 32 * k, q0[k], q1[k], len[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const ChunkSize z = size_of(a, chunk_of(a, q0[k], q1[k], len[k]));
          if (i + 32 * k < kKept) sts64(kept + 8 * (i + 32 * k + lane), make_uint2(z.first, z.served));
        }
      }
    } else {
      group(0);
    }
    for (int i = 0; i < end(); i += 32) {
      const ChunkSize z = size(i);
      const int tiles = chunk_tiles(z, call.per), tiles_here = __reduce_max_sync(0xffffffffu, tiles);
      if (MANY && tiles_here > kClose) {
        total += chunk_cost_before(z, call, INT_MAX);
      } else {
        for (int j = 0; j < tiles; ++j) total += chunk_cost(z, call, j);
      }
      if (MANY && i >> 5 >> span == lane) most = max(most, tiles_here);
      tiles_most = max(tiles_most, tiles_here);
    }
    total = warp_sum(total) * a.c.n_kv;
  }
  __device__ __forceinline__ int end() const { return MANY ? a.batch : 32; }   // (of a group of 32, lanes behind the last sequence have none)
  __device__ __forceinline__ void read(int first, int& q0, int& q1, int& len) const {
    const int b = first + lane;
    q0 = ldg_or(a.query_start + b, b < a.batch, 0);
    q1 = ldg_or(a.query_start + b + 1, b < a.batch, 0);
    len = ldg_or(a.seq_lens + b, b < a.batch, 0);
  }
  __device__ void group(int first) {
    if (first == b0) return;
    b0 = first;
    int q0, q1, len;
    read(first, q0, q1, len);
    ch = chunk_of(a, q0, q1, len);
  }
  // Sequence i + lane, i a multiple of 32 (each lane reads what it kept itself).
  __device__ ChunkSize size(int i) const {
    if constexpr (!MANY) return size_of(a, ch);
    if (i < kKept) {
      const uint2 z = lds64(kept + 8 * (i + lane));
      return {static_cast<int>(z.x), static_cast<int>(z.y)};
    }
    int q0, q1, len;
    read(i, q0, q1, len);
    return size_of(a, chunk_of(a, q0, q1, len));
  }
  // Which spans have a sequence with a tile j, and whether that of the 32 sequences from i on has none.
  __device__ unsigned tiles_past(int j) const { return MANY ? __ballot_sync(0xffffffffu, most > j) : 1u; }
  __device__ bool passes(unsigned live, int i) const { return MANY && !(live >> (i >> 5 >> span) & 1); }
  // What all sequences cost before tile index j.
  __device__ long long before_tile(int j) const {
    long long sum = 0;
    for (int i = 0; i < a.batch; i += 32) sum += chunk_cost_before(size(i), call, j);
    return warp_sum(sum) * a.c.n_kv;
  }
  // The unit of tile index j that place x is in, one of the 32 sequences from i on; these, `z`, begin at `base`, and cost
  // `c` each, `inc` up to and with their own.
  __device__ Unit locate(long long x, int j, int i, const ChunkSize& z, long long base, unsigned c, unsigned inc) const {
    const int src = __ffs(__ballot_sync(0xffffffffu, x - base < static_cast<long long>(inc) * a.c.n_kv)) - 1;
    const unsigned here = __shfl_sync(0xffffffffu, c, src);
    base += static_cast<long long>(__shfl_sync(0xffffffffu, inc, src) - here) * a.c.n_kv;
    const int h = static_cast<int>(divide(x - base, here));
    return {j, i + src, h, __shfl_sync(0xffffffffu, chunk_steps(z, call, j), src), __shfl_sync(0xffffffffu, chunk_each(z, call, j), src),
            base + static_cast<long long>(h) * here};
  }
  // Goes to the unit of place x0, whose step `step` the cut there comes to be; last, last_step: the unit where x1 is, and
  // the step up to which to go there (x0 < x1 <= total).
  __device__ void go(long long x0, long long x1, int& step, long long& last, int& last_step) {
    long long before = 0;
    bool found = false, ended = x1 >= total;
    last = total;
    last_step = 0;
    [[maybe_unused]] int walk = tiles_most > kClose ? 0 : kClose;   // tile indexes to go on by before the next one is searched for
    for (int j = 0; j < tiles_most && !(found && ended); ++j) {
      if constexpr (MANY) {
        if (walk == 0) {
          chunk_seek(found ? x1 : x0, tiles_most, kClose, found, j, before, [&](int to) { return before_tile(to); });
          walk = kClose;
        }
        --walk;
      }
      const unsigned live = tiles_past(j);
      for (int i = 0; i < end(); i += 32) {
        if (passes(live, i)) continue;
        const ChunkSize z = size(i);
        const unsigned c = chunk_cost(z, call, j);
        const long long behind = before + static_cast<long long>(__reduce_add_sync(0xffffffffu, c)) * a.c.n_kv;
        const bool first = !found && x0 < behind, final = !ended && x1 < behind;
        if (first || final) {
          unsigned inc = c;   // at most 32 * (4 * 2^24 + 10)
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
          }
          found |= first;
          ended |= final;
#pragma unroll 1   // (not unrolled: fetching the code is what takes time here)
          for (int k = first ? 0 : 1; k < (final ? 2 : 1); ++k) {
            const Unit u = locate(k ? x1 : x0, j, i, z, before, c, inc);
            if (k) {
              last = u.base;
              last_step = u.step_of(x1, least);
            } else {
              at = u;
            }
          }
        }
        before = behind;
      }
    }
    step = at.step_of(x0, least);
    group(at.b & ~31);
  }
  __device__ void next() {   // the next unit (the place behind the last one is the line's end)
    at.base = at.behind();
    if (++at.h < a.c.n_kv) return;
    at.h = 0;
    ++at.b;
    while (at.j < tiles_most) {
      const unsigned live = tiles_past(at.j);
      for (int i = at.b & ~31; i < end(); i += 32) {
        if (passes(live, i)) continue;
        group(i);
        const ChunkSize z = size_of(a, ch);
        const unsigned more = __ballot_sync(0xffffffffu, i + lane >= at.b && chunk_steps(z, call, at.j) > 0);
        if (more) {
          at.b = i + __ffs(more) - 1;
          at.steps = __shfl_sync(0xffffffffu, chunk_steps(z, call, at.j), at.b & 31);
          at.each = __shfl_sync(0xffffffffu, chunk_each(z, call, at.j), at.b & 31);
          return;
        }
      }
      at.b = 0;
      ++at.j;
    }
  }
};

template <typename T, typename TO, int CTAS, bool MANY>
__global__ void __launch_bounds__(kThreads, 1) kv16_chunk_kernel(const ChunkArgs a) {
  constexpr bool kTwo = std::is_same<TO, float>::value;   // P in two parts
  constexpr bool kStaged = CTAS == 2 || kTwo;   // output by way of shared memory
  constexpr int kStages = kStaged ? 4 : 5;
  extern __shared__ uint8_t s_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ Work s_work[2];
  __shared__ unsigned s_bad[kBad];   // a load's groups of 16 positions whose block id is bad
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t base = (static_cast<uint32_t>(__cvta_generic_to_shared(s_raw)) + 1023u) & ~1023u;
  const uint32_t bars = base + kOffBar;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const int rank = CTAS == 2 ? static_cast<int>(cluster_rank()) : 0;   // 0 issues the products
  const int team = blockIdx.x / CTAS, teams = gridDim.x / CTAS;
  if (threadIdx.x == 32) {
    for (int i = 0; i < kBars; ++i)
      mbar_init(bar(i), i == kWEmpty0 || i == kWEmpty1 ? 15
                        : (i >= kPFull0 && i < kPFull0 + 4) || i == kQFull ? 4 * CTAS
                        : i == kQEmpty || i >= kEmpty0 ? 2 : i >= kFull0 && rank == 0 ? CTAS : 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 8) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&s_tmem));
    if constexpr (CTAS == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(to) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(to) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
  }
  fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();   // the other CTA's barriers are there
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  const int per = CTAS * kRows / a.group;   // queries of a unit
  grid_dep_wait();
  grid_dep_launch();

  auto wait = [&](int b, uint32_t parity) {   // false: give up
    if (mbar_wait(bar(b), parity)) return true;
    b8_flag(a.status, TQ_DEV_TIMEOUT);
    return false;
  };
  auto warp_wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };   // one answer for the warp
  auto arrive_first = [&](int b) {   // at the barrier of the CTA that issues
    if (rank == 0) mbar_arrive(bar(b));
    else mbar_arrive_at(bar(b), 0);
  };
  auto commit = [&](int b) {
    if constexpr (CTAS == 2) mma_commit2(bar(b));
    else mma_commit(bar(b));
  };
  // A wait for a whole part of `steps` steps, and for the search for the next one.
  auto long_wait = [&](int b, uint32_t parity, int steps) {
    bool ok = mbar_try(bar(b), parity);
    if (!ok) {
      const uint64_t t0 = global_ns(), most = kWaitNs + kStepNs * static_cast<uint64_t>(steps);
      do {
        ok = mbar_try(bar(b), parity);
      } while (!ok && global_ns() - t0 < most);
    }
    if (!ok) b8_flag(a.status, TQ_DEV_TIMEOUT);
    return __all_sync(0xffffffffu, ok) != 0;
  };

  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
  if (warp < 8) {
    // ---- softmax: of tile warp / 4, a thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;\n");   // 2 x 192 + 2 x 64 = 4 x 128 registers a thread
    const int t = warp >> 2;
    const unsigned by_group = (65536u + a.group - 1) / a.group;   // row / group for rows below 512, group <= 8
    const int r = (CTAS * t + rank) * 128 + (warp & 3) * 32 + lane;   // this thread's row of the unit
    const int qi = static_cast<int>(r * by_group >> 16), head = r - qi * a.group;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lanes + kColO + t * 128;
    const float f = fmaxf(a.qscale, 0x1p-126f);   // never 0, which would make NaN of a masked place
    float seen = -INFINITY;       // the log2-sum of the row's pieces before
    unsigned n = 0, served = 0;   // halves of this tile so far (their S comes in that order), and parts
    int before = 0;
    bool ok = true;
    for (unsigned part = 0; ok; ++part) {
      if (!(ok = long_wait(kWFull0 + (part & 1), part >> 1 & 1, before))) break;
      const Work w = s_work[part & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWEmpty0 + (part & 1)));
      if (w.seq < 0) break;
      before = w.tiles;
      auto zero_rows = [&](int q0, int count) {   // `count` queries from q0 on, this KV head's part
        const long long all = static_cast<long long>(count) * a.group * (kKvD / 4);
        for (long long i = threadIdx.x; i < all; i += 256) {
          const long long x = i / (kKvD / 4);
          write4<TO>(static_cast<TO*>(a.out) + ((q0 + x / a.group) * a.n_q + w.h * a.group + x % a.group) * kKvD + 4 * (i % (kKvD / 4)),
                     make_float4(0.f, 0.f, 0.f, 0.f));
        }
      };
      if (w.tiles == 0) {
        if (rank == 0) zero_rows(w.q0, w.rows / a.group);
        continue;
      }
      if (t * CTAS * 128 >= w.rows) continue;
      const bool live = r < w.rows;
      const int vis = live ? max(min(w.pos0 + qi + 1, w.limit), 0) : 0;   // positions that this row sees
      const int vis_least = __reduce_min_sync(0xffffffffu, live ? vis : 0x7fffffff);
      auto scores_there = [&](unsigned i) { return warp_wait(kSFull0 + 2 * t + (i & 1), i >> 1 & 1); };
      float m = -1e30f, l = 0.f;   // l: sum of P
      for (int i = 0; i < w.halves; ++i, ++n) {
        if (!(ok = scores_there(n))) break;
        fence_after();
        const uint32_t t_s = tmem + lanes + kColS + t * 128 + (n & 1) * 64;
        const int at = w.tile0 * kCols + i * 64;
        const unsigned bad = s_bad[(w.load0 + i / CTAS) % kBad] >> 4 * (i % CTAS) & 15;
        const bool masked = bad || at + 64 > vis_least;
        auto mask = [&](float (&s)[32], int c) {
          if (__builtin_expect(masked, 0)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (at + 32 * c + j >= vis || (bad >> (2 * c + (j >> 4)) & 1)) s[j] = -INFINITY;
          }
        };
        uint32_t p[kTwo ? 64 : 32];   // 64 positions; in two parts: of each 32 the hi parts, then the lo parts
        auto weigh = [&](const float (&s)[32], int c) {   // the P of 32 positions, and their sum
          const float a0 = 3.f - m;
          float2 x0 = make_float2(0.f, 0.f), x1 = x0;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float2 y0 = fma2(make_float2(s[j], s[j + 1]), make_float2(f, f), make_float2(a0, a0));
            float2 y1 = fma2(make_float2(s[j + 2], s[j + 3]), make_float2(f, f), make_float2(a0, a0));
            y0.x = ex2(y0.x);
            y0.y = ex2(y0.y);
            y1.x = ex2(y1.x);
            y1.y = ex2(y1.y);
            x0 = add2(x0, y0);
            x1 = add2(x1, y1);
            if constexpr (kTwo) {
              const int k = 32 * c + j / 2;
              p[k] = take_pair<T>(y0.x, y0.y);
              p[k + 1] = take_pair<T>(y1.x, y1.y);
              p[k + 16] = to_pair<T>(y0.x, y0.y);
              p[k + 17] = to_pair<T>(y1.x, y1.y);
            } else {
              p[16 * c + j / 2] = to_pair<T>(y0.x, y0.y);
              p[16 * c + j / 2 + 1] = to_pair<T>(y1.x, y1.y);
            }
          }
          x0 = add2(x0, x1);
          return x0.x + x0.y;
        };
        float x[32], y[32];
        load32(t_s, x);
        wait_ld(x);
        load32(t_s + 32, y);
        mask(x, 0);
        if (i == 0) {   // a maximum to begin with
          wait_ld(y);
          mask(y, 1);
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; ++j) top = fmaxf(top, fmaxf(x[j], y[j]));
          m = fmaxf(m, top * f);
        }
        float sum = weigh(x, 0);
        wait_ld(y);
        mask(y, 1);
        sum += weigh(y, 1);
        const bool over = !(sum <= kMost);   // NaN too
        if (__builtin_expect(__any_sync(0xffffffffu, over), 0)) {
          float s[32], top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            load32(t_s + 32 * c, s);
            wait_ld(s);
            mask(s, c);
#pragma unroll
            for (int j = 0; j < 32; ++j) top = fmaxf(top, s[j]);
          }
          const float u = over ? fmaxf(m, top * f) : m, e = ex2(m - u);
          m = u;
          l *= e;
          if (i > 0) {
            // the next half's scores are issued after the product before this one's: once they are there, the accumulators rest
            if (!(ok = scores_there(n + 1))) break;
            fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              load32(t_o + 32 * c, s);
              wait_ld(s);
#pragma unroll
              for (int j = 0; j < 32; ++j) s[j] *= e;
              tmem_st32(t_o + 32 * c, reinterpret_cast<const uint32_t*>(s));
            }
          }
          load32(t_s, s);
          wait_ld(s);
          mask(s, 0);
          sum = weigh(s, 0);
          load32(t_s + 32, s);
          wait_ld(s);
          mask(s, 1);
          sum += weigh(s, 1);
        }
        l += sum;
        // where these columns of S stood
        tmem_st32(t_s, p);
        if constexpr (kTwo) tmem_st32(t_s + 32, p + 32);
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(kPFull0 + 2 * t + (n & 1));
      }
      if (ok && w.halves > 1) {   // the products' sign to the last half, answered so that the barriers' phases stay alike
        ok = scores_there(n);
        if (lane == 0) arrive_first(kPFull0 + 2 * t + (n & 1));
        ++n;
      }
      if (!ok || !(ok = warp_wait(kODone0 + t, served++ & 1))) break;
      fence_after();
      float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays
      const bool whole = w.slot < 0;
      const long long rec = static_cast<long long>(w.slot) * a.part_rows + r;
      auto row_of = [&](int q, int hd) { return (static_cast<long long>(w.q0 + q) * a.n_q + w.h * a.group + hd) * kKvD; };
      float sum = l == 0.f ? -INFINITY : m - 3.f + __log2f(l), of_old = 0.f;   // the row's log2-sum; what its pieces before count
      if constexpr (kTwo) {
        if (w.more) {
          const float top = fmaxf(seen, sum);
          const float e = seen == -INFINITY ? 0.f : exp2f(seen - top), g = sum == -INFINITY ? 0.f : exp2f(sum - top);
          const float all = e + g == 0.f ? 0.f : 1.f / (e + g);
          sum = e + g == 0.f ? -INFINITY : top + __log2f(e + g);
          inv *= g * all;
          of_old = e * all;
        }
        seen = sum;
      }
      auto read = [&](float (&o)[32], int col) {
        load32(t_o + col, o);
        wait_ld(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = l == 0.f ? 0.f : o[j] * inv;
      };
      if constexpr (kStaged) {
        // by way of shared memory, 128 bytes a row: a store then covers whole lines of 4 rows (a row a thread, it took a
        // line for every lane: 1.9 us a unit instead of 0.9)
        const uint32_t room = base + kOffOut + warp * 4096;
        auto pass = [&](auto* out, int col, auto&& at) {   // 128 bytes from column `col` on; at: where a row of the unit begins
          using E = typename std::remove_pointer<decltype(out)>::type;
          constexpr int kEach = 16 / sizeof(E);
          float o[32];
          [[maybe_unused]] float4 old[kTwo ? 8 : 1];   // the pieces before, as they are stored
          if constexpr (kTwo) {
            if (w.more) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int row = r - lane + 4 * k + (lane >> 3);
                old[k] = row < w.rows ? ld_dep_f32x4(reinterpret_cast<const float4*>(out + at(row) + col) + (lane & 7)) : make_float4(0.f, 0.f, 0.f, 0.f);
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 4 / static_cast<int>(sizeof(E)); ++c) {
            read(o, col + 32 * c);
#pragma unroll
            for (int k = 0; k < 2 * static_cast<int>(sizeof(E)); ++k) {
              uint32_t v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(E) == 4) v[j] = __float_as_uint(o[4 * k + j]);
                else v[j] = to_pair<E>(o[8 * k + 2 * j], o[8 * k + 2 * j + 1]);
              }
              const int unit = 2 * static_cast<int>(sizeof(E)) * c + k;
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(room + lane * 128 + ((unit ^ (lane & 7)) << 4)), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
            }
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int mine = 4 * k + (lane >> 3), unit = lane & 7, row = r - lane + mine;
            uint4 v = lds128(room + mine * 128 + ((unit ^ (mine & 7)) << 4));
            if constexpr (kTwo) {
              if (w.more) {
                const float e = __shfl_sync(0xffffffffu, of_old, mine);
                v.x = __float_as_uint(fmaf(old[k].x, e, __uint_as_float(v.x)));
                v.y = __float_as_uint(fmaf(old[k].y, e, __uint_as_float(v.y)));
                v.z = __float_as_uint(fmaf(old[k].z, e, __uint_as_float(v.z)));
                v.w = __float_as_uint(fmaf(old[k].w, e, __uint_as_float(v.w)));
              }
            }
            if (row < w.rows) *reinterpret_cast<uint4*>(out + at(row) + col + kEach * unit) = v;
          }
          __syncwarp();
        };
        if (whole) {
#pragma unroll 1
          for (int col = 0; col < kKvD; col += 128 / static_cast<int>(sizeof(TO)))
            pass(static_cast<TO*>(a.out), col, [&](int row) {
              const int q = static_cast<int>(row * by_group >> 16);
              return row_of(q, row - q * a.group);
            });
        } else {
#pragma unroll 1
          for (int col = 0; col < kKvD; col += 32) pass(a.rec_o, col, [&](int row) { return (rec - r + row) * kKvD; });
        }
      } else {
        const bool wide = ((whole ? reinterpret_cast<uintptr_t>(a.out) : reinterpret_cast<uintptr_t>(a.rec_o)) & 31) == 0;
#pragma unroll 1
        for (int col = 0; col < kKvD; col += 32) {   // 32 bytes a store: whole sectors, though a row a thread
          float o[32];
          read(o, col);
          if (live) {
            if (whole) write32<TO>(static_cast<TO*>(a.out) + row_of(qi, head) + col, o, wide);
            else write32<float>(a.rec_o + rec * kKvD + col, o, wide);
          }
        }
      }
      if (live && !whole) a.rec_lse[rec] = sum;
    }
  } else if (warp < 10 && rank == 0) {
    // ---- products, of tile warp - 8. The whole warp walks the halves of steps, so that
    // descriptors and addresses stay in uniform registers; one lane, always the same,
    // issues. Scores are issued two halves ahead: the softmax finds the next ones there.
    const bool leader = elect_one();
    const int t = warp - 8;
    const uint64_t q_at = desc_q(base + t * kTileOp);
    const uint32_t o = tmem + kColO + t * 128;
    Turn<kStages> scored, weighed;            // the next load whose scores are issued, whose values are
    unsigned filled = 0;             // loaded queries so far
    unsigned n = 0;                  // halves of the tile so far, as the softmax counts them
    unsigned turns = 0;              // where both tiles are at work, their products go in turn: what one needs next is not held up by the other's
    int before = 0;
    bool ok = true;
    for (unsigned part = 0; ok; ++part) {
      if (!(ok = long_wait(kWFull0 + (part & 1), part >> 1 & 1, before))) break;
      const int seq = s_work[part & 1].seq, halves = s_work[part & 1].tiles ? s_work[part & 1].halves : 0;
      const int rows = s_work[part & 1].rows, more = s_work[part & 1].more, keep = s_work[part & 1].keep;
      const bool mine = rows > t * CTAS * 128;   // else this warp only says that it is done with what is loaded
      const bool both = rows > CTAS * 128;
      before = s_work[part & 1].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWEmpty0 + (part & 1)));
      if (seq < 0) break;
      if (halves == 0) continue;
      // S of half i, of what is loaded in `stage` (by the leader)
      auto qk = [&](int i, int stage) {
        const uint64_t k_at = desc_k(base + kOffLoads + stage * kStage + (CTAS == 2 ? (i & 1) * 8192 : 0));
        const uint32_t d = tmem + kColS + t * 128 + ((n + i) & 1) * 64;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t qq = q_at + (((k >> 2) * kHalfQ + (k & 3) * 32) >> 4), kk = k_at + (((k >> 2) * 1024 + (k & 3) * 32) >> 4);
          if constexpr (CTAS == 2) mma_ss2(d, qq, kk, idesc_qk<T, CTAS>(), k > 0);
          else mma_ss(d, qq, kk, idesc_qk<T, CTAS>(), k > 0);
        }
      };
      auto pv = [&](uint32_t p, uint64_t v, bool acc) {
        if constexpr (CTAS == 2) mma_ts2(o, p, v, idesc_pv<T, CTAS>(), acc);
        else mma_ts(o, p, v, idesc_pv<T, CTAS>(), acc);
      };
      auto your_turn = [&]() {
        if (both && lane == 0) mbar_arrive(bar(kTurn0 + (t ^ 1)));
      };
      // Half i - 2's weights times values, half i's scores, when both are there.
      if (!more && !(ok = warp_wait(kQFull, filled++ & 1))) break;
      for (int i = 0; i < halves + 2; ++i) {
        const bool load = i < halves && i % CTAS == 0, weights = i >= 2;
        const unsigned count = n + i - 2;
        const uint32_t turn = (turns & 1) ^ (t ? 0 : 1);
        // most often all is there; else one after the other
        bool there = true;
        if (load) there = mbar_test(bar(kFull0 + scored.stage), scored.round);
        if (weights && mine) there = mbar_test(bar(kPFull0 + 2 * t + (count & 1)), count >> 1 & 1) && there;
        if (both) there = mbar_test(bar(kTurn0 + t), turn) && there;
        if (!__all_sync(0xffffffffu, there)) {
          if (load && !(ok = warp_wait(kFull0 + scored.stage, scored.round))) break;
          if (weights && mine && !(ok = warp_wait(kPFull0 + 2 * t + (count & 1), count >> 1 & 1))) break;
          if (both && !(ok = warp_wait(kTurn0 + t, turn))) break;
        }
        ++turns;
        fence_after();
        const bool frees = weights && ((i - 2) % CTAS == CTAS - 1 || i == halves + 1);   // the last half of a load
        if (leader) {
          if (mine) {
            if (weights) {
              const uint64_t v_at = desc_v<CTAS>(base + kOffLoads + 16384 + weighed.stage * kStage + (CTAS == 2 ? (i & 1) * 8192 : 0));
              const uint32_t p = tmem + kColS + t * 128 + (count & 1) * 64;
#pragma unroll
              for (int k = 0; k < 4; ++k) {   // 16 positions: 8 columns
                const uint64_t vk = v_at + (4096 / CTAS >> 4) * k;
                if constexpr (kTwo) {
                  const uint32_t pk = p + 32 * (k >> 1) + 8 * (k & 1);
                  pv(pk, vk, i > 2 || k > 0);
                  pv(pk + 16, vk, true);
                } else {
                  pv(p + 8 * k, vk, i > 2 || k > 0);
                }
              }
            }
            if (i < halves) qk(i, scored.stage);
            if (i <= halves && (i < halves || i >= 2)) commit(kSFull0 + 2 * t + ((n + i) & 1));   // of half `halves` there are none: the product before the last one's sign
            if (i == halves + 1) commit(kODone0 + t);
          }
          if (frees) commit(kEmpty0 + weighed.stage);
          if (i + 1 == halves && !keep) commit(kQEmpty);
        }
        __syncwarp();
        your_turn();
        if (i < halves && (i % CTAS == CTAS - 1 || i + 1 == halves)) scored.next();
        if (frees) weighed.next();
      }
      if (mine) n += halves + (halves > 1);
    }
    if (!ok) {   // gave up: the products in flight come to rest before their memory goes
      if (leader) commit(kEnd0 + t);
      warp_wait(kEnd0 + t, 0);
    }
    __syncwarp();
  } else if (warp < 10 || warp == 11) {
    // ---- the second CTA of a pair tells the first what it has loaded (and the other warps here only pass).
    // In the first one warp 11 writes zeros where queries are past max_q_len, row by row with the other
    // teams' and after all else: nobody waits for these, however many they are. (100000 of 8 heads 0.15 ms; by
    // the softmax warps of one CTA 13.6, and the waits for these give up after 20.)
    auto unserved = [&](int i) {   // of sequence i + lane: its chunk, if it has such
      const int b = i + lane;
      const bool in = b < a.batch;
      return chunk_of(a, ldg_or(a.query_start + b, in, 0), ldg_or(a.query_start + b + 1, in, 0), 0);
    };
    unsigned any = 0;
    for (int i = 0; i < a.batch && warp == 11 && rank == 0 && a.max_q_len < a.total_q; i += 32) any |= __ballot_sync(0xffffffffu, unserved(i).n > a.max_q_len);
    Turn<kStages> loaded;
    int before = 0;
    bool ok = true;
    for (unsigned part = 0; ok; ++part) {
      if (!(ok = long_wait(kWFull0 + (part & 1), part >> 1 & 1, before))) break;
      const int seq = s_work[part & 1].seq, loads = s_work[part & 1].loads;
      before = s_work[part & 1].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWEmpty0 + (part & 1)));
      if (seq < 0) break;
      for (int i = 0; i < loads && warp == 11 && rank == 1; ++i, loaded.next()) {
        if (!(ok = warp_wait(kFull0 + loaded.stage, loaded.round))) break;
        if (lane == 0) arrive_first(kFull0 + loaded.stage);
      }
    }
    for (int i = 0; i < a.batch && any; i += 32) {
      const Chunk c = unserved(i);
      for (unsigned m = __ballot_sync(0xffffffffu, c.n > a.max_q_len); m; m &= m - 1) {
        const int q0 = __shfl_sync(0xffffffffu, c.q0, __ffs(m) - 1), n = __shfl_sync(0xffffffffu, c.n, __ffs(m) - 1);
        for (int q = a.max_q_len + team; q < n; q += teams) {
          uint4* row = reinterpret_cast<uint4*>(static_cast<TO*>(a.out) + static_cast<long long>(q0 + q) * a.n_q * kKvD);
          for (int k = lane; k < a.n_q * kKvD * static_cast<int>(sizeof(TO)) / 16; k += 32) row[k] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
  } else if (warp == 10) {
    // ---- the work, keys and values
    Line<MANY> line(a, {per, a.limit, a.group, CTAS * 128}, base + kOffLoads, lane);
    const long long cut = line.total / 5;   // one step and more a team
    const long long ctas = cut < 1 ? 1 : (cut < teams ? cut : teams);
    line.least = !a.may_split ? INT_MAX : line.total < 16ll * teams ? 1 : 2;
    auto cut_of = [&](long long team_) { return divide(line.total * team_, ctas); };
    int from = 0, last_step = 0;   // steps of the unit at hand that are others'; and those up to which to go in the last unit
    long long last = 0;            // where that begins
    const bool works = team < ctas && line.total > 0;
    if (works) {
      line.go(cut_of(team), cut_of(team + 1), from, last, last_step);
      if (from == line.at.steps) {   // the cut moved to the next unit
        line.next();
        from = 0;
      }
    }
    if constexpr (MANY) {   // chunks that were kept, before loads come to their place
      fence_smem_async();
      __syncwarp();
    }
    const bool speaks = rank == 0 && lane == 0;
    if (a.may_split && speaks) a.split_units[team] = make_int4(0, 0, 0, 0);
    constexpr int kGroups = 4 * CTAS;   // of 16 positions a load
    const int group16 = lane & (kGroups - 1);
    Turn<kStages> load;
    unsigned loads = 0;
    int done = from;               // steps of the unit at hand that are done, or others'
    int before = 0, before2 = 0;   // steps of the parts that the slot's last reader may be at
    bool ok = true;
    for (unsigned part = 0;; ++part) {
      if (!(ok = long_wait(kWEmpty0 + (part & 1), (part >> 1 & 1) ^ 1, before + before2))) break;
      Work w = {};
      w.seq = -1;
      const auto& u = line.at;
      const int to = u.base < last ? u.steps : last_step;
      // in one piece, or in several of about a size
      const int pieces = kTwo ? max((to - done + kPiece - 1) / kPiece, 1) : 1;
      const int upto = done + (to - done + pieces - 1) / pieces;
      if (works && u.base <= last && from < to) {
        const int src = u.b & 31;
        Chunk ch;
        ch.q0 = __shfl_sync(0xffffffffu, line.ch.q0, src);
        ch.n = __shfl_sync(0xffffffffu, line.ch.n, src);
        ch.len = __shfl_sync(0xffffffffu, line.ch.len, src);
        const int served = min(ch.n, a.max_q_len), first = u.j * per;
        w.seq = u.b;
        w.h = u.h;
        w.q0 = ch.q0 + first;
        w.rows = min(per, served - first) * a.group;
        w.pos0 = ch.len - ch.n + first;
        w.limit = chunk_limit(size_of(a, ch), line.call, u.j);
        w.tile0 = done;
        w.tiles = w.limit == 0 ? 0 : upto - done;
        w.more = done > from;
        w.keep = upto < to;
        w.halves = min((w.limit + 63) / 64 - 2 * w.tile0, 2 * w.tiles);
        w.loads = w.tiles ? (w.halves + CTAS - 1) / CTAS : 0;
        w.slot = from > 0 ? 2 * team : (to < u.steps ? 2 * team + 1 : -1);
        w.load0 = loads;
        if (u.j == 0 && done == 0 && u.h == 0 && speaks && (ch.n > a.max_q_len || ch.len > a.limit))
          b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
        if (done == 0 && to < u.steps && speaks) {
          // the last team whose cut is in the unit, and stays there
          long long owner = divide(u.behind() * ctas - 1, line.total);
          while (owner > team && u.step_of(cut_of(owner), line.least) == u.steps) --owner;
          a.split_units[team] = make_int4(w.q0, w.rows, w.h * a.group, static_cast<int>(owner) - team + 1);
        }
      }
      if (lane == 0) s_work[part & 1] = w;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWFull0 + (part & 1)));
      if (w.seq < 0) break;
      before2 = before;
      before = w.tiles;
      // the block of this lane's group of 16 positions of load i (-1: behind the end)
      const int* table = a.block_table + static_cast<long long>(w.seq) * a.c.bt_stride;
      auto block_of = [&](int i) {
        const int g16 = w.tile0 * 8 + i * kGroups + group16;
        return ldg_or(table + (g16 >> (a.c.log2_bs - 4)), i < w.loads && g16 * 16 < w.limit, -1);
      };
      int blk = block_of(0);
      for (int i = 0; i < w.loads; ++i, ++loads, load.next()) {
        const int blk_next = block_of(i + 1);
        const int g16 = w.tile0 * 8 + i * kGroups + group16;
        const bool inside = g16 * 16 < w.limit, good = inside && a.c.good(blk);
        const uint8_t* src = a.c.tile(good ? blk : 0, w.h, g16);
        const int rows = good ? min(w.limit - g16 * 16, kKvRows) : 0;   // of values: rows behind the end may hold anything
        constexpr unsigned kAll = (1u << kGroups) - 1;
        const unsigned all = __ballot_sync(0xffffffffu, good) & kAll, bad = __ballot_sync(0xffffffffu, inside && !good) & kAll;
        const unsigned ragged = __ballot_sync(0xffffffffu, rows < kKvRows) & kAll;
        if (bad && speaks) b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
        // keys: all, or this CTA's 32 positions of each half; values: all coordinates, or this CTA's 64
        constexpr int kRowBytes = 256 / CTAS, kTileV = kKvHalfBytes / CTAS;   // of values, here
        const unsigned keys = CTAS == 2 ? all & 0x33u << 2 * rank : all;
        const uint32_t full = bar(kFull0 + load.stage), k_to = base + kOffLoads + load.stage * kStage, v_to = k_to + 16384;
        if (!(ok = warp_wait(kEmpty0 + load.stage, load.round ^ 1))) break;
        uint32_t bytes = __popc(keys) * kKvHalfBytes + __popc(all) * kTileV;
        if (__builtin_expect(ragged, 0)) {   // their rows that are not loaded are 0: no weight takes NaN along
          bytes = __popc(keys) * kKvHalfBytes;
#pragma unroll 1
          for (int g = 0; g < kGroups; ++g) {
            const int have = __shfl_sync(0xffffffffu, rows, g);
            bytes += have * kRowBytes;
            for (int k = lane; k < kTileV / 16 && have < kKvRows; k += 32)
              if (k / (kTileV / 32) * 8 + (k >> 3 & 7) >= have)
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(v_to + g * kTileV + 16 * k), "r"(0u) : "memory");
          }
          fence_smem_async();
          __syncwarp();
        }
        if (lane == 0) {
          s_bad[loads % kBad] = bad;
          mbar_expect(full, bytes);
        }
        __syncwarp();
        if (lane < kGroups && rows > 0) {
          if (keys >> lane & 1) bulk_g2s_plain(k_to + (CTAS == 2 ? (group16 & 1) + (group16 >> 2) * 2 : group16) * kKvHalfBytes, src, kKvHalfBytes, full);
          const uint32_t to = v_to + group16 * kTileV;
          const uint8_t* from = src + kKvHalfBytes + (CTAS == 2 ? rank * 1024 : 0);
          if (CTAS == 1 && rows == kKvRows) {
            bulk_g2s_plain(to, from, kKvHalfBytes, full);
          } else if constexpr (CTAS == 1) {   // whole groups of 8 rows, then the rows of one group, half by half
            const int whole = rows >> 3 << 11, rest = (rows & 7) * 128;
            if (whole) bulk_g2s_plain(to, from, whole, full);
            if (rest) {
              bulk_g2s_plain(to + whole, from + whole, rest, full);
              bulk_g2s_plain(to + whole + 1024, from + whole + 1024, rest, full);
            }
          } else {   // the two groups of 8 rows
            bulk_g2s_plain(to, from, min(rows, 8) * 128, full);
            if (rows > 8) bulk_g2s_plain(to + 1024, from + 2048, (rows - 8) * 128, full);
          }
        }
        __syncwarp();
        blk = blk_next;
      }
      if (!ok) break;
      if (kTwo && upto < to) {
        done = upto;
      } else {
        line.next();
        from = done = 0;
      }
    }
    // the copies in flight end before their memory goes (in the first CTA of a pair, the second one's too), and so do the
    // products that read them and what these signal to either CTA
    for (int k = 0; k < kStages; ++k) {   // the last load of each stage, the oldest first
      if (loads + k >= kStages) {
        warp_wait(kFull0 + load.stage, load.round ^ 1);
        if (ok) warp_wait(kEmpty0 + load.stage, load.round ^ 1);
      }
      load.next();
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
      const int head0 = s_work[part & 1].h * a.group, more = s_work[part & 1].more;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kWEmpty0 + (part & 1)));
      if (seq < 0) break;
      if (more) {   // they are there
        before += tiles;
        continue;
      }
      const int wait_for = before;
      before = tiles;
      if (tiles == 0) continue;
      const int c = lane & 15, last = rows > CTAS * 128 ? kRows : 128;
      auto unit_row = [&](int here) { return CTAS == 2 ? here + (here & 128) + 128 * rank : here; };
      auto row_at = [&](int r) {
        const int qi = static_cast<int>(r * by_group >> 16);
        return static_cast<const T*>(a.q) + (q0 + qi) * a.q_stride + static_cast<long long>(head0 + r - qi * a.group) * kKvD;
      };
      for (int k = threadIdx.x & 127; k < 2 * last && filled; k += 128) {   // to L2, while the queries before are still in use
        const int r = unit_row(k >> 1);
        if (r < rows) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(row_at(r) + 64 * (k & 1)));
      }
      if (!(ok = long_wait(kQEmpty, (filled++ & 1) ^ 1, wait_for))) break;
#pragma unroll 8
      for (int here = 2 * (warp - 12) + (lane >> 4); here < last; here += 8) {
        const int r = unit_row(here);
        const T* src = r < rows ? row_at(r) + 8 * c : static_cast<const T*>(a.q);
        const uint32_t to = base + (here >> 7) * kTileOp + (c >> 3) * kHalfQ + (here & 127) * 128 + (((c ^ here) & 7) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(src), "r"(r < rows ? 16 : 0) : "memory");
      }
      asm volatile("cp.async.wait_all;\n" ::: "memory");
      fence_smem_async();
      __syncwarp();
      if (lane == 0) arrive_first(kQFull);
    }
  }
  fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();   // the other CTA is done with this one's barriers and memory
  fence_after();
  if (warp == 8) {
    if constexpr (CTAS == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

// Merges the parts of split units. A warp takes a row, two or four at a time, by 8 loads
// of records at once: four rows of two parts, two of up to four, one of eight. What there
// is of that is dealt evenly to the warps of a grid of kMergeCtas CTAs an SM, which are
// resident at once. (CTAs for 8 rows of every team's unit, split or whole, 4864 of them
// that mostly found nothing to do, took 10 us: 4 chunks of 190-572 queries and few heads
// 34.6 us for 30.0, 2 of 430-1291 23.0 for 21.6. CTAs for 32 rows were slow where there
// are many parts: the latter 26.8.)
template <typename TO>
struct Merge {
  const ChunkArgs& a;
  int u, lane;
  int4 unit;   // first row, rows, first head, parts
  template <int ROWS, int PARTS>
  __device__ __forceinline__ void rows(int row0) const {
    static_assert(ROWS * PARTS == 8, "loads");
    const int end = unit.y, parts = unit.w;
    float m[ROWS], l[ROWS];
    float4 o[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int z0 = 0; z0 < parts; z0 += PARTS) {
      float lse[ROWS][PARTS];
      float4 x[ROWS][PARTS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
          const int z = z0 + k;
          const bool in = z < parts && row0 + r < end;
          const long long rec = static_cast<long long>(z == 0 ? 2 * u + 1 : 2 * (u + z)) * a.part_rows + row0 + r;
          lse[r][k] = in ? ld_dep_f32(a.rec_lse + rec) : -INFINITY;
          x[r][k] = in ? ld_dep_f32x4(reinterpret_cast<const float4*>(a.rec_o + rec * kKvD) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
          if (lse[r][k] == -INFINITY) continue;   // nothing seen there
          const float top = fmaxf(m[r], lse[r][k]);
          const float e = m[r] == -INFINITY ? 0.f : exp2f(m[r] - top), f = exp2f(lse[r][k] - top);
          m[r] = top;
          l[r] = l[r] * e + f;
          o[r].x = o[r].x * e + x[r][k].x * f;
          o[r].y = o[r].y * e + x[r][k].y * f;
          o[r].z = o[r].z * e + x[r][k].z * f;
          o[r].w = o[r].w * e + x[r][k].w * f;
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int row = row0 + r;
      if (row >= end) break;
      const float s = l[r] == 0.f ? 0.f : 1.f / l[r];
      const long long orow = (static_cast<long long>(unit.x) + row / a.group) * a.n_q + unit.z + row % a.group;
      write4<TO>(static_cast<TO*>(a.out) + orow * kKvD + 4 * lane, make_float4(o[r].x * s, o[r].y * s, o[r].z * s, o[r].w * s));
    }
  }
};
// Rows that a warp takes at once of a unit of so many parts.
__device__ __forceinline__ int rows_at_once(int parts) { return parts == 2 ? 4 : parts <= 4 ? 2 : 1; }
template <typename TO>
__global__ void __launch_bounds__(kMergeThreads, kMergeCtas) kv16_chunk_merge_kernel(const ChunkArgs a, int teams) {
  constexpr int kGroups = (kCtas + 31) / 32;
  static_assert(kGroups <= kMergeThreads / 32, "a warp a group of units");
  __shared__ int4 s_unit[kGroups * 32];
  __shared__ int s_end[kGroups * 32];   // pieces of work up to the unit's end, of its group of 32
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  if (warp < kGroups) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (static_cast<int>(threadIdx.x) < teams) x = ld_dep_u32x4(a.split_units + threadIdx.x);
    const int4 unit = make_int4(x.x, x.y, x.z, x.w);
    const int each = rows_at_once(unit.w);
    int inc = unit.w ? (unit.y + each - 1) / each : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    s_unit[threadIdx.x] = unit;
    s_end[threadIdx.x] = inc;
  }
  __syncthreads();
  int end[kGroups], total = 0;   // of this lane's unit of each group
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    end[k] = total + s_end[32 * k + lane];
    total += s_end[32 * k + 31];
  }
  for (int i = warp * gridDim.x + blockIdx.x; i < total; i += gridDim.x * (kMergeThreads / 32)) {
    int u = 0;   // units that end before piece i
#pragma unroll
    for (int k = 0; k < kGroups; ++k) u += __popc(__ballot_sync(0xffffffffu, end[k] <= i));
    int before = 0;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int all = __shfl_sync(0xffffffffu, end[k], (u - 1) & 31);
      if ((u - 1) >> 5 == k) before = all;
    }
    const int4 unit = s_unit[u];
    const int row = (i - before) * rows_at_once(unit.w);
    const Merge<TO> merge = {a, u, lane, unit};
    if (unit.w == 2) merge.template rows<4, 2>(row);
    else if (unit.w <= 4) merge.template rows<2, 4>(row);
    else merge.template rows<1, 8>(row);
  }
}

// The grid, and the workspace that split units take.
struct Plan {
  long long units;   // (tile of queries, KV head), at most
  int ctas;          // that work on a unit together
  int may_split, part_rows;
  size_t workspace;
};
Plan plan_for(const tq_config* cfg, int batch, int total_q, int max_q_len, int max_seq_len) {
  Plan p;
  const int group = cfg->num_q_heads / cfg->num_kv_heads;
  p.ctas = batch > 0 && static_cast<long long>(total_q) * group > static_cast<long long>(kPairRows) * batch ? 2 : 1;
  const int per = p.ctas * kRows / group;
  const int longest = max_q_len < total_q ? max_q_len : total_q;
  // tiles of queries: a full one for every `per` rows at most, and one more for every
  // chunk; as many for every sequence as the longest chunk has at most
  const long long most = static_cast<long long>(batch) * ((longest + per - 1) / per);
  long long tiles = static_cast<long long>(total_q) / per + (batch < total_q ? batch : total_q);
  if (tiles > most) tiles = most;
  p.units = tiles * cfg->num_kv_heads;
  p.may_split = p.units > 0 && max_seq_len > kNoSplit * kCols;
  p.part_rows = longest < per ? longest * group : per * group;
  // as many rows as either shape of units has, so that a workspace serves all smaller calls too
  const size_t records = static_cast<size_t>(2 * kCtas) * (longest * static_cast<long long>(group) < kRows ? longest * group : kRows);
  p.workspace = p.may_split ? (kCtas * sizeof(int4) + records * (kKvD + 1) * sizeof(float) + 15) / 16 * 16 : 16;
  return p;
}

template <typename T, typename TO, int CTAS, bool MANY>
cudaError_t launch(const ChunkArgs& a, const Plan& p, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0, sms = 0;
  cudaError_t err = b8_current_device(&dev, &sms);
  if (err == cudaSuccess) err = b8_allow_smem(kv16_chunk_kernel<T, TO, CTAS, MANY>, kSmem, dev, &done);
  if (err != cudaSuccess) return err;
  const int most = (sms < kCtas ? sms : kCtas) / CTAS;
  // starts that go backwards may name more units than these: they are served all the same
  const long long steps = p.units * ((static_cast<long long>(a.limit) + kCols - 1) / kCols + 1);
  const int teams = steps < most ? static_cast<int>(steps) : most;
  if (CTAS == 2) err = launch_pdl_cluster(kv16_chunk_kernel<T, TO, CTAS, MANY>, dim3(2 * teams), dim3(kThreads), 2, kSmem, s, a);
  else err = launch_pdl(kv16_chunk_kernel<T, TO, CTAS, MANY>, dim3(teams), dim3(kThreads), kSmem, s, a);
  if (err != cudaSuccess || !p.may_split) return err;
  return launch_pdl(kv16_chunk_merge_kernel<TO>, dim3(kMergeCtas * most * CTAS), dim3(kMergeThreads), 0, s, a, teams);
}
template <typename T, typename TO>
cudaError_t launch(const ChunkArgs& a, const Plan& p, cudaStream_t s) {
  if (a.batch > 32) return p.ctas == 2 ? launch<T, TO, 2, true>(a, p, s) : launch<T, TO, 1, true>(a, p, s);
  return p.ctas == 2 ? launch<T, TO, 2, false>(a, p, s) : launch<T, TO, 1, false>(a, p, s);
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // A few queries: each a row of its own over the cache, in one launch (one that this kernel's start and merge outlast).
  int dev = 0, sms = 0;
  Kv16Short how;
  if (b8_current_device(&dev, &sms) != cudaSuccess) return TQ_ERR_CUDA;
  if (kv16_short(total_q, cfg->num_kv_heads, max_seq_len < cap ? max_seq_len : cap, sms < kCtas ? sms : kCtas, kShortMost, kShortMostSmall, false, &how)) {
    Kv16RowsArgs r = {};
    r.c = kv16_cache(cfg, L, cache, num_blocks, bt_stride);
    r.q = q;
    r.q_stride = q_stride;
    r.block_table = block_table;
    r.seq_lens = seq_lens;
    r.query_start = query_start;
    r.status = dev_status;
    r.out = out;
    r.rows = total_q;
    r.n_kv = cfg->num_kv_heads;
    r.n_q = cfg->num_q_heads;
    r.group = cfg->num_q_heads / cfg->num_kv_heads;
    r.max_seq_len = max_seq_len;
    r.cap = cap;
    r.batch = batch;
    r.max_q_len = max_q_len;
    r.qscale = b8_qscale(scale);
    return kv16_short_launch(r, L.is_bf16, out_dtype, how, dev, s) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
  }
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
  a.search_ns = kWaitNs + kStepNs * (batch / 32 + p.units / cfg->num_kv_heads / 512);
  a.split_units = static_cast<int4*>(workspace);
  a.rec_o = reinterpret_cast<float*>(a.split_units + kCtas);
  a.rec_lse = a.rec_o + static_cast<size_t>(2 * kCtas / p.ctas) * p.part_rows * kKvD;
  const cudaError_t err = L.is_bf16 ? launch<__nv_bfloat16>(a, p, out_dtype, s) : launch<__half>(a, p, out_dtype, s);
  return err == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
