// Argument blocks and small device helpers of the streaming entry points
// (norm and rotation, 8-bit block cache, block selection, cache attention).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"

namespace svsa {

// Allow `Kernel` that much dynamic shared memory on the current device; the
// driver is asked once per device (an attribute of the loaded kernel).
template <auto Kernel>
inline cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// More status bits (see common.cuh): bit 3 = an index (position, map entry,
// page, length or list entry) out of range, bit 4 = a value that is not finite
// given to an 8-bit conversion.
constexpr unsigned int kFlagIndex = 8u, kFlagNotFinite = 16u;

struct NormRopeArgs {
  const void* x[2];                // q, k
  const void* dy[2];               // backward: gradients [B, heads, rows, d]
  void* out[2];                    // forward: [B, heads, rows, d]; backward: dx, strided
  const float* w[2];               // nullable
  const float* cos;                // nullable: no rotation
  const float* sin;
  const int32_t* pos;
  const int32_t* map;              // nullable; forward: output row -> token, backward: token -> output row
  float* part;                     // backward: partial dw rows [CTA][d]
  long long stride[2][3];          // x: batch, head, token
  long long out_stride[2][3];      // dx
  long long pos_stride;
  int heads[2];
  int B, N, rows, axes, split1, split2, table_rows, halves;
  float eps;
};

// The cache: [page][head][64 tokens][d] codes with a scale per (page, head),
// and per sequence a row of the table of pages and a length.
struct CacheArgs {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int8_t* mean;                  // nullable: [page][head][d] key means and their scales
  float* mean_scale;
  const int32_t* table;          // [B][max_blocks]
  const int32_t* len;            // [B]
  int B, heads, d, i8, n_pages, max_blocks;
};

// The smallest power of two s with amax / s <= top, top = 127 (int8) or 448
// (e4m3); 0 for amax = 0.  In binary, amax = f * 2^e with f in [1, 2), and top
// = t * 2^b with t = 127/64 (b = 6) or 1.75 (b = 8): s = 2^(e - b), one more
// where f > t.  Powers of two make x / s exact, so the codes do not depend on
// how the division is done, and a block whose scale grows keeps what its codes
// stand for up to one more rounding.
__device__ __forceinline__ float pow2_scale(float amax, bool i8) {
  if (!(amax > 0.f)) return 0.f;
  uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127;
  if (e == -127) {                                  // a subnormal: shift it up first
    u = __float_as_uint(amax * 16777216.f);
    e = (int)(u >> 23) - 127 - 24;
  }
  const uint32_t frac = u & 0x7fffffu;
  const uint32_t top = i8 ? 0x7e0000u : 0x600000u;  // 127/64 - 1 and 1.75 - 1 in 23 bits
  e -= i8 ? 6 : 8;
  if (frac > top) e += 1;
  if (e < -126) e = -126;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two fp32 lanes in one instruction (sm_100), each rounded as its scalar form.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2(F2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float sum2(F2 x) {
  float a, b;
  split2(x, a, b);
  return a + b;
}

}  // namespace svsa
