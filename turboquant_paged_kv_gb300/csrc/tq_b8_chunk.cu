// Chunks of queries against the 8-bit cache with block scales, on tcgen05
// tensor cores.
//
//   out_i = sum_p softmax_p(scale s_k(p) q_i . k_p) s_v(p) v_p, p <= position of i
//
// One CTA serves 256 rows, the query heads of one KV head of 256 / group
// consecutive queries, in two tiles of 128 rows, against 128 positions at a
// time:
//   S_t = Q_t K^T        tcgen05.mma, A and B from shared memory
//   P_t = 8 p s_v / 2^sigma   one row per thread, S read from tensor memory
//   O_t += P_t V         A = P_t from tensor memory (it takes S_t's place), B = V
// The codes are exact in fp16; a query row is scaled by a power of two that
// brings its largest magnitude to 2^14, so the scores are sums of exact
// products. The block scales enter with the softmax: s_k multiplies a group of
// 16 columns, log2(s_v) is added to the exponent, and the denominator takes
// each group's sum times 2^sigma / s_v. p = 2^(score - m), and m and sigma are
// the row's own: m at most its largest score so far, m + sigma at most its
// largest score + log2(s_v), over the positions that it sees. So the largest P
// of a row is 8 or more whatever the scales of the blocks are that it does not
// see or gives no weight (one sigma for a step, from its largest s_v, took 0 for
// rows whose own values were 2^-28 of that), and no later position changes a bit
// of a row. P is rounded to fp16: half a step is 2^-11, and no step below 2^-24
// errs by up to 2^-28 of the row's largest p s_v, for each code. With f32 output P
// is held in two fp16 parts (hi + lo, 2^-22), as in the decode, and its product
// takes twice the instructions: the two cases below with f32 output 259 -> 302 and
// 695 -> 815 us, their errors against 64 bits 2.1e-4 -> 0.9e-5 and 1.4e-5 (what is
// left is the tensor cores' sum over the positions). With fp16 output the one part
// adds 2.1e-4 to the output's own rounding of 2.1e-4 (together 2.9e-4), with bf16
// nothing to its 1.7e-3.
//
// Warps: 0-3 and 4-7 the softmax of tile 0 and 1 (a thread a row, no
// shuffles), 8-11 expand codes from global memory into the two-stage fp16
// operand buffers (128-byte swizzle, the same image for K, read as a K-major
// operand, and V, read as an MN-major one), 12 issues the products: of the two
// tiles in turn, so one tile's products run while the other's softmax does.
// No maximum is sought in the common case: the weights are taken with the
// maximum so far, and a row of which some P would not fit in fp16, or whose m has
// fallen far behind, shows in its sums; only then the row's new m and sigma are
// found, and what was accumulated (by the softmax warps, in tensor memory) and
// the step's earlier P are rescaled. S_t(i + 1) is issued after O_t += P_t(i) V,
// so a complete S_t(i + 1) also says that the accumulators of step i are at rest.
// Every wait is bounded; one that runs out sets TQ_DEV_TIMEOUT and ends the CTA,
// after its products in flight.
//
// Bound: tensor cores by its operations; measured, the softmax's latency beside
// them. A step of 256 rows x 128 positions is 32 products of 64 cycles (2240
// cycles with their commits) and takes about 3600: 7500 warp instructions, and
// the shared-memory pipe four fifths busy or more (operands, codes,
// tensor-memory traffic). 4 chunks of about 2000 queries over up to 8192
// positions, 32 query heads: 695 us, 1219 TFLOP/s, 0.63 of a measured bf16 GEMM;
// 32 chunks of 128 over 4096: 259 us, 1078 TFLOP/s. What moved it: products issued
// from uniform registers (from a branch that one lane takes, each cost 75 to 200
// cycles), no search for the maximum, and code small enough for the instruction
// cache (the step's softmax rolled, the prologue and the epilogue short: 823 to
// 695 us). A reference for each row costs nothing beside one for the step (691 to
// 696 us against 703): its arithmetic runs while the scores are on their way.
// Tried and slower: S in halves of 64 positions one half ahead, P handed over in
// halves, an issuing warp for each tile (both tiles then fall into step), two
// threads a row, eight expanding warps.
#include "tq_attn.cuh"
#include "tq_b8_chunk.cuh"

namespace tq {
namespace {

constexpr int kRows = 256;             // of a CTA: two tiles of 128
constexpr int kCols = 128;             // positions a step
constexpr int kThreads = 512;
constexpr int kParts = 152;            // CTAs of a wave, one an SM
constexpr float kMost = 60000.f;       // sums of 16 P up to this: every P fits in fp16
constexpr float kMostSum = 0x1p24f;    // sums of a step's 8 p up to this: the scores are below m + 21
constexpr float kLeast = -103.f;       // log2(s_v / 2^sigma) from below: a group's values vanish, its weights still count
constexpr uint32_t kTileOp = 32768;    // a 128 x 128 fp16 operand: two halves of 64 columns, 128 bytes a row
constexpr uint32_t kHalfOp = 16384;
constexpr uint32_t kOffK = 2 * kTileOp, kOffV = 4 * kTileOp, kOffBar = 6 * kTileOp;
constexpr uint32_t kSmem = kOffBar + 256 + 1024;   // and room to align to 1024
// tensor memory columns
constexpr uint32_t kColS = 0, kColO = 256;

// barriers, 8 bytes each from kOffBar
enum { kQFull, kKFull0, kKFull1, kVFull0, kVFull1, kKEmpty0, kKEmpty1, kVEmpty0, kVEmpty1, kSFull0, kSFull1, kPFull0, kPFull1, kODone0, kODone1, kEnd, kBars };

// shared-memory operand descriptors: 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t addr) {   // the halves of 64 columns kHalfOp apart
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (static_cast<uint64_t>(kHalfOp >> 4) << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}
// f16 x f16 -> f32, M = 128, N = 128
constexpr uint32_t kIdescQK = (1u << 4) | ((128u / 8) << 17) | ((128u / 16) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);   // B is MN-major

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
// two fp32 operations at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_smem_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// 32 columns of this warp's 32 rows, one row a lane
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) { tmem_ld16(addr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) { tmem_ld32(addr, r); }
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[16]) { tmem_st16(addr, r); }
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[32]) { tmem_st32(addr, r); }

template <typename TO>
__device__ __forceinline__ void write4(TO* dst, float4 v) {
  if constexpr (std::is_same<TO, float>::value) {
    *reinterpret_cast<float4*>(dst) = v;
  } else if constexpr (std::is_same<TO, __half>::value) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// 32 bytes, at once where the address allows it (one answer for the grid).
__device__ __forceinline__ void store32(void* dst, const uint32_t* v, bool wide) {
  if (!wide) {
    static_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}
// 32 numbers of a row.
template <typename TO>
__device__ __forceinline__ void write32(TO* dst, const float* y, bool wide) {
  if constexpr (std::is_same<TO, float>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(y[8 * i + j]);
      store32(dst + 8 * i, v, wide);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (std::is_same<TO, __half>::value) {
          v[j] = pack_half2(y[16 * i + 2 * j], y[16 * i + 2 * j + 1]);
        } else {
          const __nv_bfloat162 x = __floats2bfloat162_rn(y[16 * i + 2 * j], y[16 * i + 2 * j + 1]);
          v[j] = *reinterpret_cast<const uint32_t*>(&x);
        }
      }
      store32(dst + 16 * i, v, wide);
    }
  }
}

// What a CTA does.
struct Work {
  int seq, h;           // sequence (-1: nothing), KV head
  int slot;             // where the records of this part of a split unit go (-1: whole)
  int q0, rows;         // row of its first query in q and out; rows of A, its queries' heads
  int pos0;             // position of that query (may be negative)
  int limit;            // positions that its last query sees: what stands behind them need not have been stored
  int tile0, tiles;     // steps of 128 positions: [tile0, tile0 + tiles)
  int zero0, zeros;     // queries that nobody serves
};

// A sequence's chunk: its first row, queries, length and tiles of queries.
struct Chunk {
  int q0, n, len, tiles;
};
__device__ __forceinline__ Chunk tiles_of(const B8ChunkArgs& a, int b, int per) {
  Chunk c;
  c.q0 = min(max(ldg_or(a.query_start + b, b < a.batch, 0), 0), a.total_q);
  c.n = min(max(ldg_or(a.query_start + b + 1, b < a.batch, 0), c.q0), a.total_q) - c.q0;
  c.len = ldg_or(a.seq_lens + b, b < a.batch, 0);
  c.tiles = (min(c.n, a.max_q_len) + per - 1) / per;
  return c;
}

template <bool INT8>
__device__ __forceinline__ void expand_rows(const uint4 x, uint32_t row_at, int c, int r7) {
  // 16 codes of group c of a row -> 32 bytes: two 16-byte groups of the operand's half c / 4
  uint4 lo, hi;
  codes_to_half2<INT8>(x.x, lo.x, lo.y);
  codes_to_half2<INT8>(x.y, lo.z, lo.w);
  codes_to_half2<INT8>(x.z, hi.x, hi.y);
  codes_to_half2<INT8>(x.w, hi.z, hi.w);
  const uint32_t at = row_at + (c >> 2) * kHalfOp;
  const int g = 2 * (c & 3);
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(at + ((g ^ r7) << 4)), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w) : "memory");
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(at + (((g + 1) ^ r7) << 4)), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w) : "memory");
}

template <typename TQ, typename TO, bool INT8>
__global__ void __launch_bounds__(kThreads, 1) b8_chunk_kernel(const B8ChunkArgs a) {
  constexpr bool kTwo = std::is_same<TO, float>::value;   // P in two fp16 parts
  extern __shared__ uint8_t s_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ Work s_work;
  __shared__ float2 s_groups[8][8];   // each softmax warp's: s_k and log2(s_v) of the step's groups of 16 positions
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t base = (static_cast<uint32_t>(__cvta_generic_to_shared(s_raw)) + 1023u) & ~1023u;
  const uint32_t bars = base + kOffBar;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  // Barriers and tensor memory need nothing of the kernel before; one warp finds the
  // work meanwhile. Units of work: (tile of a chunk's queries, KV head), the last
  // fastest; sequence by sequence, and the latest queries of a chunk, which see the
  // most, first. Where there are few, those beyond a multiple of kParts (all, if they
  // are fewer) are split over the history, so that the last wave fills the GPU.
  if (threadIdx.x == 32) {
    mbar_init(bar(kQFull), 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kKFull0 + i), 4);
      mbar_init(bar(kVFull0 + i), 4);
      mbar_init(bar(kKEmpty0 + i), 1);
      mbar_init(bar(kVEmpty0 + i), 1);
      mbar_init(bar(kSFull0 + i), 1);
      mbar_init(bar(kPFull0 + i), 4);
      mbar_init(bar(kODone0 + i), 1);
    }
    mbar_init(bar(kEnd), 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(&s_tmem))) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  const int per = kRows / a.group;   // queries of a CTA
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 0) {
    int unit = blockIdx.x, part = 0, parts = 1, full = 0;
    if (a.may_split) {
      int tiles = 0;
      for (int b0 = 0; b0 < a.batch; b0 += 32) tiles += __reduce_add_sync(0xffffffffu, tiles_of(a, b0 + lane, per).tiles);
      const int units = tiles * a.c.n_kv, rem = units % kParts;
      full = units - rem;
      // starts that go backwards may name more units than the grid has CTAs for: no records then
      parts = rem && units <= static_cast<int>(gridDim.x) - kParts ? kParts / rem : 1;
      if (blockIdx.x == 0 && lane == 0) a.split_units[0] = make_int4(parts > 1 ? rem : 0, parts, 0, 0);
      if (parts > 1 && unit >= full) {
        part = (unit - full) % parts;
        unit = full + (unit - full) / parts;
      } else {
        parts = 1;
      }
    }
    int x = unit / a.c.n_kv;
    const int h = unit - x * a.c.n_kv;
    int seq = -1, qs = 0, n = 0, tile_q = 0, raw_len = 0;
    for (int b0 = 0; b0 < a.batch && seq < 0; b0 += 32) {   // 32 sequences at a time
      const Chunk ch = tiles_of(a, b0 + lane, per);
      int inc = ch.tiles;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned here = __ballot_sync(0xffffffffu, x < inc);
      if (here) {
        const int src = __ffs(here) - 1;
        seq = b0 + src;
        qs = __shfl_sync(0xffffffffu, ch.q0, src);
        n = __shfl_sync(0xffffffffu, ch.n, src);
        raw_len = max(__shfl_sync(0xffffffffu, ch.len, src), 0);
        tile_q = __shfl_sync(0xffffffffu, inc, src) - 1 - x;
      }
      x -= __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      Work w;
      w.seq = seq;
      w.h = h;
      w.slot = parts > 1 ? (unit - full) * parts + part : -1;
      const int served = min(n, a.max_q_len);
      w.zero0 = qs + served;
      w.zeros = tile_q == 0 && part == 0 ? n - served : 0;   // queries past max_q_len
      if (tile_q == 0 && part == 0 && h == 0 && n > 0 && (n > a.max_q_len || raw_len > min(a.max_seq_len, a.cap)))
        b8_flag(a.status, TQ_DEV_SEQ_TOO_LONG);
      w.q0 = qs + tile_q * per;
      w.rows = min(per, served - tile_q * per) * a.group;
      w.pos0 = raw_len - n + tile_q * per;
      w.limit = max(min(w.pos0 + min(per, served - tile_q * per), min(a.max_seq_len, a.cap)), 0);
      const int all_tiles = (w.limit + kCols - 1) / kCols;
      const int each = parts > 1 ? max((all_tiles + parts - 1) / parts, 2) : all_tiles;   // steps of a part
      w.tile0 = min(part * each, all_tiles);
      w.tiles = min(each, all_tiles - w.tile0);
      if (parts > 1 && part == 0 && seq >= 0) a.split_units[1 + unit - full] = make_int4(w.q0, w.rows, h * a.group, 0);
      s_work = w;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  const Work w = s_work;
  auto leave = [&]() {   // all of the CTA
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  };
  if (w.seq < 0) return leave();
  const int heads0 = w.h * a.group, rows = w.rows;
  const int halves = rows > 128 ? 2 : 1;   // row tiles at work
  const unsigned by_group = (65536u + a.group - 1) / a.group;   // row / group for rows below 256, group <= 8
  auto query_of = [&](int row) { return static_cast<int>(row * by_group >> 16); };
  auto zero_rows = [&](int q0, int count) {   // `count` queries from q0 on, this KV head's part
    const long long all = static_cast<long long>(count) * a.group * (kB8D / 4);
    for (long long i = threadIdx.x; i < all; i += kThreads) {
      const long long r = i / (kB8D / 4);
      write4<TO>(static_cast<TO*>(a.out) + ((q0 + r / a.group) * a.n_q + heads0 + r % a.group) * kB8D + 4 * (i % (kB8D / 4)),
                 make_float4(0.f, 0.f, 0.f, 0.f));
    }
  };
  if (w.zeros) zero_rows(w.zero0, w.zeros);
  if (w.tiles == 0) {   // nothing to see here
    if (w.slot < 0) zero_rows(w.q0, rows / a.group);
    else if (threadIdx.x < rows) a.rec_lse[w.slot * a.part_rows + threadIdx.x] = -INFINITY;
    return leave();
  }
  auto wait = [&](int b, uint32_t parity) {   // false: give up
    if (mbar_wait(bar(b), parity)) return true;
    b8_flag(a.status, TQ_DEV_TIMEOUT);
    return false;
  };
  auto warp_wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };   // one answer for the warp
  const int tiles = w.tiles;
  const int* table = a.block_table + static_cast<long long>(w.seq) * a.c.bt_stride;
  const int shift = a.c.log2_bs - 4;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;\n");
    const int t = warp >> 2;
    if (t >= halves) {
      if (lane == 0) mbar_arrive(bar(kQFull));
    } else {
      // The queries of 32 rows (a row: a query head) go to their places in A as they
      // are, half a warp a row; then each row is scaled and rounded to fp16 in place, a
      // thread a row.
      const uint32_t a_at = base + t * kTileOp;
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int r = t * 128 + (warp & 3) * 32 + 2 * i + (lane >> 4), c = lane & 15;
        const int qi = query_of(r), head = heads0 + r - qi * a.group;
        const TQ* src = static_cast<const TQ*>(a.q) + (r < rows ? (w.q0 + qi) * a.q_stride + static_cast<long long>(head) * kB8D + 8 * c : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(a_at + (r & 127) * 128 + (c >> 3) * kHalfOp + (((c & 7) ^ (r & 7)) << 4)), "l"(src), "r"(r < rows ? 16 : 0) : "memory");
      }
      asm volatile("cp.async.wait_all;\n" ::: "memory");
      __syncwarp();
      const int r = threadIdx.x;   // this thread's row, 0 .. 255
      const bool live = r < rows;
      const int qi = query_of(r), head = heads0 + r - qi * a.group;
      float down;
      {
        const uint32_t row_at = a_at + (r & 127) * 128;
        uint32_t m = 0;
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
          const uint4 v = lds128(row_at + (c >> 3) * kHalfOp + (((c & 7) ^ (r & 7)) << 4));
          m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
        m = max(m & 0xffffu, m >> 16);
        float amax;
        if constexpr (std::is_same<TQ, __nv_bfloat16>::value) amax = __uint_as_float(m << 16);
        else amax = half2_to_float2(m).x;
        // 2^k with amax 2^k in [2^14, 2^15)
        const int k = min(max(14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23), -112), 112);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
        down = a.qscale * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
          const uint32_t at = row_at + (c >> 3) * kHalfOp + (((c & 7) ^ (r & 7)) << 4);
          const uint4 v = lds128(at);
          const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 f;
            if constexpr (std::is_same<TQ, __nv_bfloat16>::value) f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ws[j]));
            else f = half2_to_float2(ws[j]);
            o[j] = pack_half2(f.x * up, f.y * up);
          }
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
        }
      }
      fence_smem_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull));
      const int vis = live ? max(min(w.pos0 + qi + 1, w.limit), 0) : 0;   // positions that this row sees
      const int vis_least = __reduce_min_sync(0xffffffffu, live ? vis : 0x7fffffff);
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t t_s = tmem + lanes + kColS + t * 128, t_o = tmem + lanes + kColO + t * 128;

      // lanes 0-7 hold the scales of the step's 8 groups of 16 positions; the
      // next step's are on their way meanwhile
      auto group_block = [&](int i) {   // block id of this lane's group of step i; -2: behind the end
        const int g16 = (w.tile0 + i) * 8 + (lane & 7);
        return ldg_or(table + (g16 >> shift), i < tiles && g16 * 16 < w.limit, -2);
      };
      auto group_scales = [&](int blk) {
        const bool good = a.c.good(blk);
        return ld_or_zero2(a.c.scales(good ? blk : 0, w.h), good);
      };
      int blk = group_block(0);
      uint2 sc = group_scales(blk);
      int blk_next = group_block(1);
      float m = -1e30f, sigma = 0.f, l = 0.f;   // l: sum of 8 p
      bool ok = true;
      for (int i = 0; i < tiles; ++i) {
        const bool bad = sc.x == 0u;   // a scale that was stored is never 0
        if (bad && blk != -2 && t == 0 && warp == 0 && !a.c.good(blk)) b8_flag(a.status, TQ_DEV_BLOCK_OUT_OF_RANGE);
        const unsigned bad_groups = __ballot_sync(0xffffffffu, bad) & 0xffu;
        if (lane < 8) s_groups[warp][lane] = bad ? make_float2(1.f, 0.f) : make_float2(__uint_as_float(sc.x), __log2f(__uint_as_float(sc.y)));
        float by_o = 1.f;   // what the accumulators take
        __syncwarp();
        blk = blk_next;
        sc = group_scales(blk);
        blk_next = group_block(i + 2);

        if (!(ok = warp_wait(kSFull0 + t, i & 1))) break;
        fence_after();
        const int at = (w.tile0 + i) * kCols;
        const bool masked = bad_groups || at + kCols > vis_least;
        float sums = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {   // rolled: unrolled, the code does not stay in the instruction cache
          float s[32];
          tmem_ld32(t_s + 32 * c, reinterpret_cast<uint32_t*>(s));
          wait_ld();
          if (__builtin_expect(masked, 0)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (at + 32 * c + j >= vis || (bad_groups >> (2 * c + (j >> 4)) & 1)) s[j] = -INFINITY;
          }
          const float2 g0 = s_groups[warp][2 * c], g1 = s_groups[warp][2 * c + 1];
          // never 0, which would make NaN of a masked place; below 2^-126 the scores vanish anyway (|s| < 2^31)
          const float f0 = fmaxf(g0.x * down, 0x1p-126f), f1 = fmaxf(g1.x * down, 0x1p-126f);
          uint32_t p[kTwo ? 32 : 16];   // the hi parts, then the lo parts
          float next;   // `sums` with these columns
          for (int go = 0;; ++go) {
            const float d0 = fmaxf(g0.y - sigma, kLeast), d1 = fmaxf(g1.y - sigma, kLeast);
            const float a0 = d0 + (3.f - m), a1 = d1 + (3.f - m);
            float2 x0 = make_float2(0.f, 0.f), x1 = x0;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float2 y0 = fma2(make_float2(s[j], s[j + 1]), make_float2(f0, f0), make_float2(a0, a0));
              float2 y1 = fma2(make_float2(s[16 + j], s[17 + j]), make_float2(f1, f1), make_float2(a1, a1));
              y0.x = ex2(y0.x);
              y0.y = ex2(y0.y);
              y1.x = ex2(y1.x);
              y1.y = ex2(y1.y);
              x0 = add2(x0, y0);
              x1 = add2(x1, y1);
              if constexpr (kTwo) {
                split_half2(y0.x, y0.y, p[j / 2], p[16 + j / 2]);
                split_half2(y1.x, y1.y, p[8 + j / 2], p[24 + j / 2]);
              } else {
                p[j / 2] = pack_half2(y0.x, y0.y);
                p[8 + j / 2] = pack_half2(y1.x, y1.y);
              }
            }
            const float sum0 = x0.x + x0.y, sum1 = x1.x + x1.y;
            next = fmaf(sum1, ex2(-d1), fmaf(sum0, ex2(-d0), sums));
            const bool over = !(fmaxf(sum0, sum1) <= kMost && next <= kMostSum);   // NaN too
            if (__builtin_expect(go || !__any_sync(0xffffffffu, over), 1)) break;
            float mx = -INFINITY, my = -INFINITY;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              mx = fmaxf(mx, s[j]);
              my = fmaxf(my, s[16 + j]);
            }
            mx *= f0;
            my *= f1;
            const float u = over ? fmaxf(m, fmaxf(mx, my)) : m, down_by = m - u;
            const float r = over ? fmaxf(sigma + down_by, fmaxf(g0.y + (mx - u), g1.y + (my - u))) : sigma;
            const float e = ex2(down_by + (sigma - r)), e_l = ex2(down_by);
            m = u;
            sigma = r;
            l *= e_l;
            sums *= e_l;
            by_o *= e;
            wait_st();
#pragma unroll 1
            for (int d = 0; d < c; ++d) {   // the P of this step that are there already
              uint32_t q[kTwo ? 32 : 16];
              tmem_ld(t_s + 32 * d, q);
              wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float2 y = half2_to_float2(q[j]);
                if constexpr (kTwo) {
                  const float2 lo = half2_to_float2(q[16 + j]);
                  y.x += lo.x;
                  y.y += lo.y;
                  split_half2(y.x * e, y.y * e, q[j], q[16 + j]);
                } else {
                  q[j] = pack_half2(y.x * e, y.y * e);
                }
              }
              tmem_st(t_s + 32 * d, q);
            }
          }
          sums = next;
          tmem_st(t_s + 32 * c, p);   // where these columns of S stood
        }
        l += sums;
        if (__builtin_expect(i > 0 && __any_sync(0xffffffffu, by_o != 1.f), 0)) {
          uint32_t o[32];
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            tmem_ld32(t_o + 32 * c, o);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * by_o);
            tmem_st32(t_o + 32 * c, o);
          }
        }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull0 + t));
      }
      if (ok && warp_wait(kODone0 + t, 0)) {
        fence_after();
        const float scale = l > 0.f ? ex2(sigma) / l : (l == 0.f ? 0.f : l);   // NaN stays
        const bool whole = w.slot < 0;
        const bool wide = ((whole ? reinterpret_cast<uintptr_t>(a.out) : reinterpret_cast<uintptr_t>(a.rec_o)) & 31) == 0;
        const long long orow = static_cast<long long>(w.q0 + qi) * a.n_q + head;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {   // 32 bytes a store: whole sectors, though a row a thread
          uint32_t o[32];
          tmem_ld32(t_o + 32 * c, o);
          wait_ld();
          float y[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = l == 0.f ? 0.f : __uint_as_float(o[j]) * scale;
          if (live) {
            if (whole) write32<TO>(static_cast<TO*>(a.out) + orow * kB8D + 32 * c, y, wide);
            else write32<float>(a.rec_o + static_cast<long long>(w.slot * a.part_rows + r) * kB8D + 32 * c, y, wide);
          }
        }
        if (live && !whole) a.rec_lse[w.slot * a.part_rows + r] = l == 0.f ? -INFINITY : m - 3.f + __log2f(l);
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;\n");
    // 32 positions a warp and step: 8 loads of 16 codes a lane for the keys, 8 for the values
    const int cw = warp - 8, rs = lane >> 2, cc = lane & 3;
    // block ids of the warp's two groups of 16 positions (-1: behind the end)
    auto blocks = [&](int i) {
      const int g16 = (w.tile0 + i) * 8 + 2 * cw;
      return make_int2(ldg_or(table + (g16 >> shift), i < tiles && g16 * 16 < w.limit, -1),
                       ldg_or(table + ((g16 + 1) >> shift), i < tiles && g16 * 16 + 16 < w.limit, -1));
    };
    auto load = [&](int i, int2 id, int kv, uint4* x) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int g16 = (w.tile0 + i) * 8 + 2 * cw + half;
        const int blk = half ? id.y : id.x;
        const bool good = a.c.good(blk);
        const uint8_t* src = a.c.tile(good ? blk : 0, w.h, g16) + kv * kB8HalfBytes;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 8 * (k >> 1) + rs, c = 4 * (k & 1) + cc;
          x[4 * half + k] = ld_or_zero4(src + row * kB8D + ((c ^ (row & 7)) << 4), good && g16 * 16 + row < w.limit);
        }
      }
    };
    auto store = [&](uint32_t op, const uint4* x) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int row = 32 * cw + 8 * (k >> 1) + rs;
        expand_rows<INT8>(x[k], op + row * 128, 4 * (k & 1) + cc, row & 7);
      }
    };
    uint4 x[8], y[8];
    int2 id = blocks(0), id_next = blocks(1);   // a step's ids are there before its codes are asked for
    load(0, id, 0, x);
    load(0, id, 1, y);
    bool ok = true;
    for (int i = 0; i < tiles && ok; ++i) {
      const int st = i & 1;
      const uint32_t free_phase = ((i >> 1) & 1) ^ 1;
      if (!(ok = warp_wait(kKEmpty0 + st, free_phase))) break;
      store(base + kOffK + st * kTileOp, x);
      fence_smem_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull0 + st));
      id = id_next;
      id_next = blocks(i + 2);
      load(i + 1, id, 0, x);
      if (!(ok = warp_wait(kVEmpty0 + st, free_phase))) break;
      store(base + kOffV + st * kTileOp, y);
      fence_smem_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kVFull0 + st));
      load(i + 1, id, 1, y);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    if (warp == 12) {
      // The whole warp walks the steps, so that descriptors and addresses stay in
      // uniform registers (issued from a branch that one lane takes, a product cost
      // 75 to 200 cycles of moves); one lane, always the same, issues.
      const bool leader = elect_one();
      auto qk = [&](int t, int st) {
        const uint64_t q_at = desc_k_major(base + t * kTileOp), k_at = desc_k_major(base + kOffK + st * kTileOp);
        const uint32_t d = tmem + kColS + t * 128;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t off = ((k >> 2) * kHalfOp + (k & 3) * 32) >> 4;
          mma_ss(d, q_at + off, k_at + off, kIdescQK, k > 0);
        }
        mma_commit(bar(kSFull0 + t));
      };
      bool ok = warp_wait(kQFull, 0) && warp_wait(kKFull0, 0);
      if (ok) {
        fence_after();
        if (leader) {
          for (int t = 0; t < halves; ++t) qk(t, 0);
          mma_commit(bar(kKEmpty0));
        }
        __syncwarp();
      }
      for (int i = 0; i < tiles && ok; ++i) {
        const int st = i & 1, nst = st ^ 1;
        const bool more = i + 1 < tiles;
        for (int t = 0; t < halves; ++t) {
          if (!(ok = warp_wait(kPFull0 + t, i & 1))) break;
          if (t == 0 && !(ok = warp_wait(kVFull0 + st, (i >> 1) & 1))) break;
          fence_after();
          if (leader) {
            const uint64_t v_at = desc_mn_major(base + kOffV + st * kTileOp);
            const uint32_t d = tmem + kColO + t * 128, p = tmem + kColS + t * 128;
            mma_ts(d, p, v_at, kIdescPV, i > 0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {   // 16 positions: 8 columns, 32 apart for each 32 positions
              const uint32_t at = p + 32 * (k >> 1) + 8 * (k & 1);
              if (k > 0) mma_ts(d, at, v_at + (2048 >> 4) * k, kIdescPV, true);
              if constexpr (kTwo) mma_ts(d, at + 16, v_at + (2048 >> 4) * k, kIdescPV, true);
            }
            if (!more) mma_commit(bar(kODone0 + t));
          }
          __syncwarp();
          if (more) {
            if (t == 0 && !(ok = warp_wait(kKFull0 + nst, ((i + 1) >> 1) & 1))) break;
            fence_after();
            if (leader) {
              qk(t, nst);
              if (t + 1 == halves) {
                mma_commit(bar(kVEmpty0 + st));
                mma_commit(bar(kKEmpty0 + nst));
              }
            }
            __syncwarp();
          }
        }
      }
      if (!ok) {   // gave up: the products in flight come to rest before their memory goes
        if (leader) mma_commit(bar(kEnd));
        warp_wait(kEnd, 0);
      }
    }
    __syncwarp();
  }
  leave();
}

// Merges the parts of split units: a warp a row, 8 rows of a unit a CTA.
template <typename TO>
__global__ void __launch_bounds__(256) b8_chunk_merge_kernel(const B8ChunkArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_unit = (a.part_rows + 7) / 8;
  const int u = blockIdx.x / per_unit, r = (blockIdx.x - u * per_unit) * 8 + warp;
  grid_dep_wait();
  grid_dep_launch();
  const uint2 head = ld_dep_u32x2(a.split_units);
  const int parts = head.y;
  if (u >= static_cast<int>(head.x)) return;
  const uint4 unit = ld_dep_u32x4(a.split_units + 1 + u);   // first row, rows, first head
  if (r >= static_cast<int>(unit.y)) return;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int z0 = 0; z0 < parts; z0 += 8) {   // eight parts' records on their way at once
    float lse[8];
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const long long rec = static_cast<long long>(u * parts + z0 + k) * a.part_rows + r;
      lse[k] = z0 + k < parts ? ld_dep_f32(a.rec_lse + rec) : -INFINITY;
      x[k] = z0 + k < parts ? ld_dep_f32x4(reinterpret_cast<const float4*>(a.rec_o + rec * kB8D) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (lse[k] == -INFINITY) continue;   // nothing seen there, and nothing written but this
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
  write4<TO>(static_cast<TO*>(a.out) + orow * kB8D + 4 * lane, make_float4(o.x * s, o.y * s, o.z * s, o.w * s));
}

template <typename TQ, typename TO, bool INT8>
cudaError_t launch(const B8ChunkArgs& a, const B8ChunkPlan& p, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = b8_allow_smem(b8_chunk_kernel<TQ, TO, INT8>, kSmem, dev, &done);
  if (err != cudaSuccess) return err;
  const long long ctas = p.units + (p.may_split ? kParts : 0);
  err = launch_pdl(b8_chunk_kernel<TQ, TO, INT8>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), kSmem, s, a);
  if (err != cudaSuccess || !p.may_split) return err;
  return launch_pdl(b8_chunk_merge_kernel<TO>, dim3(kParts / 2 * ((p.part_rows + 7) / 8)), dim3(256), 0, s, a);
}

template <typename TQ, typename TO>
cudaError_t launch_format(const B8ChunkArgs& a, const B8ChunkPlan& p, bool is_int8, cudaStream_t s) {
  return is_int8 ? launch<TQ, TO, true>(a, p, s) : launch<TQ, TO, false>(a, p, s);
}

template <typename TQ>
cudaError_t launch_out(const B8ChunkArgs& a, const B8ChunkPlan& p, bool is_int8, int out_dtype, cudaStream_t s) {
  if (out_dtype == TQ_DTYPE_F32) return launch_format<TQ, float>(a, p, is_int8, s);
  if (out_dtype == TQ_DTYPE_F16) return launch_format<TQ, __half>(a, p, is_int8, s);
  return launch_format<TQ, __nv_bfloat16>(a, p, is_int8, s);
}

}  // namespace

B8ChunkPlan b8_chunk_plan(const tq_config* cfg, int batch, int total_q, int max_q_len, int max_seq_len) {
  B8ChunkPlan p;
  const int group = cfg->num_q_heads / cfg->num_kv_heads, per = kRows / group;
  const int longest = max_q_len < total_q ? max_q_len : total_q;
  // tiles of queries: a full one for every `per` rows at most, and one more for every
  // chunk; as many for every sequence as the longest chunk has at most
  const long long most = static_cast<long long>(batch) * ((longest + per - 1) / per);
  long long tiles = static_cast<long long>(total_q) / per + (batch < total_q ? batch : total_q);
  if (tiles > most) tiles = most;
  p.units = tiles * cfg->num_kv_heads;
  // Splitting pays while the last wave is a good part of all (at most 6 waves), and
  // where the history has steps to split. Measured at 512 units of 33 steps (3.4
  // waves): 279 us whole, 257 us with the last 56 units in 2 parts. The rule counts
  // units and not their steps: one history of 131072 among 31 of 500, 5 queries each,
  // takes 1.77 ms, since the units of the long one are walked by one CTA each.
  p.may_split = p.units > 0 && p.units <= 6 * kParts && max_seq_len > 3 * kCols;
  p.part_rows = longest < per ? longest * group : per * group;
  const size_t records = static_cast<size_t>(kParts) * p.part_rows;
  p.workspace = p.may_split ? ((kParts / 2 + 2) * sizeof(int4) + records * (kB8D + 1) * sizeof(float) + 15) / 16 * 16 : 16;
  return p;
}

cudaError_t b8_chunk_launch(B8ChunkArgs a, const B8ChunkPlan& p, bool is_int8, int q_dtype, int out_dtype,
                            void* workspace, cudaStream_t s) {
  if (p.units == 0) return cudaSuccess;
  a.may_split = p.may_split;
  a.part_rows = p.part_rows;
  a.split_units = static_cast<int4*>(workspace);
  a.rec_o = reinterpret_cast<float*>(a.split_units + kParts / 2 + 2);
  a.rec_lse = a.rec_o + static_cast<size_t>(kParts) * p.part_rows * kB8D;
  return q_dtype == TQ_DTYPE_BF16 ? launch_out<__nv_bfloat16>(a, p, is_int8, out_dtype, s)
                                  : launch_out<__half>(a, p, is_int8, out_dtype, s);
}

}  // namespace tq
