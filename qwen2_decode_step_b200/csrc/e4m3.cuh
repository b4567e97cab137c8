// e4m3.cuh -- what the 8-bit (e4m3) operators share: conversions, their error
// bit, tensor maps of bytes, TMA stores.
//
// e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; largest value 448,
// smallest 2^-9, NaN 0x7f / 0xff, no infinities.  Every e4m3 value is exact in
// fp16, bf16 and fp32.  A value v is stored with a scale s as the code of v / s.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"
#include "tma.h"

namespace q2 {

// Value 4 of the operators' device error word (op_error_flag): a device-side
// length past the capacity of an 8-bit cache.
constexpr int kErrCapacity = 4;

// Whether this is the first call on the current device for `done` (one bit per
// device; a kernel's attributes are set once).  Devices past 63 always set them.
inline bool first_on_device(std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return true;
  return (done.load(std::memory_order_acquire) >> dev & 1) == 0;
}
inline void done_on_device(std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev <= 63)
    done.fetch_or(1ull << dev, std::memory_order_release);
}

// Tensor maps as make_tmap_2d_bf16's, of bytes (box_cols bytes wide; x of a load
// a multiple of 16) and of fp32.
q2_status make_tmap_2d_u8(CUtensorMap* out, const void* base, uint64_t rows, uint64_t cols, uint64_t pitch_bytes,
                          uint32_t box_rows, uint32_t box_cols, int swizzle_bytes);
q2_status make_tmap_2d_f32(CUtensorMap* out, const void* base, uint64_t rows, uint64_t cols, uint64_t pitch_bytes,
                           uint32_t box_rows, uint32_t box_cols, int swizzle_bytes);

// Tiled 2-D TMA store of one box of shared memory to (x = column, y = row), in
// the issuing thread's current bulk group; elements outside the tensor are not
// written.  x and y must not be negative, x as for tma_load_2d.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, const void* smem_src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(smem_u32(smem_src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Every bulk group of this thread has read its shared memory / is complete.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Generic writes to shared memory before this are seen by later async-proxy reads.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

constexpr float kE4m3Max = 448.f;

// Two fp32 values to two codes, lo in the low byte: nearest, ties to even, held
// to +-448 (infinities too); NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Two codes to a pair of fp16 values (exact), the low byte in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// Four codes to fp32 (exact).
__device__ __forceinline__ void e4m3x4_to_f(uint32_t v, float* f) {
  const uint32_t lo = e4m3x2_to_f16x2((uint16_t)(v & 0xffffu)), hi = e4m3x2_to_f16x2((uint16_t)(v >> 16));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(f[0]), "=f"(f[1])
      : "r"(lo));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(f[2]), "=f"(f[3])
      : "r"(hi));
}

// |x| where x is finite, else 0: what counts towards a scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

}  // namespace q2
