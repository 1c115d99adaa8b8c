// Shared by the kernels of the 8-bit cache with block scales: addressing, code
// conversions and argument checks. Internal, not ABI.
//
// Cache block: [n_kv][block_size / 16] tiles of 4096 bytes (16 key rows of 128
// codes, then 16 value rows, the 16-byte group c of row r stored at group
// c ^ (r & 7)), then [n_kv] pairs of fp32 scales.
#ifndef TQ_B8_CUH_
#define TQ_B8_CUH_

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "tq_internal.h"
#include "tq_launch.cuh"

namespace tq {
namespace {

constexpr int kB8D = 128;
constexpr int kB8Rows = 16;           // positions per tile
constexpr int kB8HalfBytes = 2048;    // the key rows, or the value rows, of a tile
constexpr int kB8TileBytes = 4096;
constexpr float kB8Floor = 0x1p-100f; // smallest scale: its reciprocal and its quotients stay normal
constexpr int kB8MaxGroup = 8;        // query heads per KV head

// Where a (block, head) lies.
struct B8Cache {
  const uint8_t* base;
  long long num_blocks, block_bytes;
  int scale_off, n_kv, log2_bs, bt_stride;
  __device__ __forceinline__ int tiles_per_block() const { return 1 << (log2_bs - 4); }
  __device__ __forceinline__ bool good(int blk) const { return blk >= 0 && blk < num_blocks; }
  // tile `t` of a sequence, whose block id is blk
  __device__ __forceinline__ const uint8_t* tile(int blk, int h, int t) const {
    const int tpb = tiles_per_block();
    return base + blk * block_bytes + (static_cast<long long>(h * tpb + (t & (tpb - 1))) << 12);
  }
  __device__ __forceinline__ const uint8_t* scales(int blk, int h) const {
    return base + blk * block_bytes + scale_off + 8 * h;
  }
};

// Two codes in the low (or four in all) bytes of w as fp16 pairs. Both formats
// are exact in fp16.
template <bool INT8>
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (INT8) {
    // code + 128 in the low bits of 1024.0 (one unit there is 1), less 1152
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Four codes as floats.
template <bool INT8>
__device__ __forceinline__ void codes_to_float4(uint32_t w, float out[4]) {
  uint32_t lo, hi;
  codes_to_half2<INT8>(w, lo, hi);
  const float2 a = half2_to_float2(lo), b = half2_to_float2(hi);
  out[0] = a.x; out[1] = a.y; out[2] = b.x; out[3] = b.y;
}

// Four scaled values, |y| <= Q (1 + 2^-22) or infinite, to codes: to nearest,
// ties to even. int8: adding 1.5 * 2^23 rounds to an integer that then stands
// in the low bits of the sum.
template <bool INT8>
__device__ __forceinline__ uint32_t floats_to_codes(float a, float b, float c, float d) {
  if constexpr (INT8) {
    const float k = 12582912.0f;
    const uint32_t x = __float_as_uint(__fadd_rn(a, k)), y = __float_as_uint(__fadd_rn(b, k));
    const uint32_t z = __float_as_uint(__fadd_rn(c, k)), w = __float_as_uint(__fadd_rn(d, k));
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  } else {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        " mov.b32 %0, {lo, hi};\n}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  }
}

// *p where pred, else zeros: loads into preset registers, so that nothing waits
// for the value here (a select on what was loaded would).
__device__ __forceinline__ uint2 ld_or_zero2(const void* p, bool pred) {
  uint2 v = make_uint2(0u, 0u);
  asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %3, 0;\n @q ld.global.cg.v2.b32 {%0, %1}, [%2];\n}\n"
               : "+r"(v.x), "+r"(v.y)
               : "l"(p), "r"(static_cast<unsigned>(pred)));
  return v;
}
__device__ __forceinline__ uint4 ld_or_zero4(const void* p, bool pred) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %5, 0;\n @q ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];\n}\n"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
               : "l"(p), "r"(static_cast<unsigned>(pred)));
  return v;
}

__device__ __forceinline__ void b8_flag(unsigned int* status, unsigned int bit) {
  if (status) atomicOr(status, bit);
}

inline bool b8_dtype16(int t) { return t == TQ_DTYPE_F16 || t == TQ_DTYPE_BF16; }
inline bool b8_dtype(int t) { return b8_dtype16(t) || t == TQ_DTYPE_F32; }
inline bool b8_aligned(const void* p, unsigned n) { return (reinterpret_cast<unsigned long long>(p) & (n - 1)) == 0; }
inline int b8_log2(int x) { return x == 16 ? 4 : x == 32 ? 5 : x == 64 ? 6 : 7; }
inline B8Cache b8_cache(const tq_config* cfg, const tq_b8_layout& L, const void* cache, long long num_blocks, int bt_stride) {
  return {static_cast<const uint8_t*>(cache), num_blocks, L.block_bytes, L.scale_off, cfg->num_kv_heads,
          b8_log2(cfg->block_size), bt_stride};
}
// positions that a block-table row can name
inline int b8_cap(const tq_config* cfg, int bt_stride) {
  const long long cap = static_cast<long long>(bt_stride) * cfg->block_size;
  return cap > 0x7fffff00ll ? 0x7fffff00 : static_cast<int>(cap);
}
// Row strides in elements: 0 stands for contiguous rows.
inline tq_status b8_stride(long long* stride, long long row) {
  if (*stride == 0) *stride = row;
  return *stride < row || *stride % 8 ? TQ_ERR_INVALID_ARG : TQ_OK;
}
// What a device is asked for once: its SM count, and that a kernel may take `smem`
// bytes of dynamic shared memory (`done`: a bit a device, one word a kernel). The
// runtime keeps the latter for the device, through a reset and for every context.
inline cudaError_t b8_current_device(int* dev, int* sms) {
  static std::atomic<int> known[64];
  cudaError_t err = cudaGetDevice(dev);
  if (err != cudaSuccess) return err;
  int n = *dev < 64 ? known[*dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev);
    if (err != cudaSuccess) return err;
    if (*dev < 64) known[*dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return cudaSuccess;
}
template <typename Kernel>
cudaError_t b8_allow_smem(Kernel* kernel, int smem, int dev, std::atomic<unsigned long long>* done) {
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return err;
}

// Softmax scale in log2 units.
inline float b8_qscale(float scale) {
  const float s = scale > 0.f ? scale : 0.08838834764831845f;   // 1 / sqrt(128)
  return s * 1.4426950408889634f;
}
// Query heads against KV heads.
inline tq_status b8_heads(const tq_config* cfg) {
  if (cfg->num_q_heads <= 0 || cfg->num_q_heads % cfg->num_kv_heads) return TQ_ERR_INVALID_ARG;
  return cfg->num_q_heads / cfg->num_kv_heads > kB8MaxGroup ? TQ_ERR_UNSUPPORTED : TQ_OK;
}
// The checks that every device entry point shares.
inline tq_status b8_check(const void* cache, long long num_blocks, const int* block_table, int bt_stride,
                          const int* seq_lens, const unsigned int* status) {
  if (!cache || !block_table || !seq_lens || num_blocks < 0 || bt_stride <= 0) return TQ_ERR_INVALID_ARG;
  if (!b8_aligned(cache, 16) || !b8_aligned(block_table, 4) || !b8_aligned(seq_lens, 4) || !b8_aligned(status, 4))
    return TQ_ERR_MISALIGNED;
  return TQ_OK;
}

}  // namespace
}  // namespace tq

#endif  // TQ_B8_CUH_
