// q8_quant.cu -- the operands of the 8-bit linear: rows (activations) or 128 x
// 128 blocks (weights) quantised to e4m3 with an fp32 scale per group.
//
//   a = max(largest finite |x| of the group, 2^-100)
//   scale = a / 448,  code = e4m3(x * (448 / a))
// 448 / a is kept as hi + lo to some 45 bits, hi an approximate quotient and lo
// its remainder over a, and x * hi + x * lo is one rounding from the definition's
// product, where x times a rounded quotient alone would fall on the other side of
// a code's border about three times as often.  The lower bound on a keeps 448 / a
// finite; a group of zeros gets codes of 0.
//
// Bound by HBM: the input once, a byte per element out, 4 bytes per group; next
// to that by instruction issue (with two IEEE divisions a lane and a test for
// infinities per element 4096 x 8960 bf16 took 26 us, and the warps' commonest
// stall was a ready instruction not selected).
#include "common.cuh"
#include "e4m3.cuh"

namespace q2 {

namespace {

constexpr int kGroup = Q2_Q8_GROUP;

struct Quant {
  const void* x;
  long long stride;  // elements between rows of x
  uint8_t* codes;    // [rows][cols]
  float* scales;     // rows: [groups][rows]; blocks: [row blocks][groups]
  int rows, cols, groups;
};

// A lane's share of a row of a group: vectors of 16 bytes (kV elements, so that
// a warp's loads and stores are whole lines), or, where rows do not start on 16
// bytes, elements 32 apart (a warp's loads are neighbours again).
template <typename T, bool VEC>
struct Share {
  static constexpr int kV = VEC ? Storage<T>::kVec : 4;   // elements of a lane
  static constexpr int kLanes = kGroup / kV;              // lanes of a row: 32, or 16 (bf16 vectors)
  static constexpr int kRows = 32 / kLanes;               // rows of a warp's step
  uint4 raw;                                              // as stored (VEC), or four fp32 values
  __device__ __forceinline__ void load(const T* row, int c0, int cols) {
    const int l = threadIdx.x % kLanes;
    if constexpr (VEC) {
      const int c = c0 + l * kV;
      raw = c < cols ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
    } else {
      uint32_t* w = &raw.x;
#pragma unroll
      for (int j = 0; j < kV; ++j) w[j] = __float_as_uint(c0 + l + 32 * j < cols ? to_f(row[c0 + l + 32 * j]) : 0.f);
    }
  }
  __device__ __forceinline__ void values(float* f) const {
    if constexpr (VEC)
      unpack16<T>(raw, f);
    else
      unpack16<float>(raw, f);
  }
  // The largest magnitude, infinities among them (the maxima pass over NaN; NaN
  // if there is nothing else).  bf16 pairs are compared as they are: half the
  // instructions.
  __device__ __forceinline__ float amax() const {
    if constexpr (VEC && sizeof(T) == 2) {
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      __nv_bfloat162 a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = w[i] & 0x7fff7fffu;
        a[i] = *reinterpret_cast<const __nv_bfloat162*>(&v);
      }
      const __nv_bfloat162 x = __hmax2(__hmax2(a[0], a[1]), __hmax2(a[2], a[3]));
      return fmaxf(__low2float(x), __high2float(x));
    } else {
      float f[kV];
      values(f);
      float m = fabsf(f[0]);
#pragma unroll
      for (int j = 1; j < kV; ++j) m = fmaxf(m, fabsf(f[j]));
      return m;
    }
  }
  __device__ __forceinline__ float amax_finite() const {
    float f[kV], m = 0.f;
    values(f);
#pragma unroll
    for (int j = 0; j < kV; ++j) m = fmaxf(m, finite_abs(f[j]));
    return m;
  }
  static __device__ __forceinline__ void store(uint8_t* row, int c0, int cols, const float* f) {
    const int l = threadIdx.x % kLanes;
    if constexpr (VEC) {
      const int c = c0 + l * kV;
      if (c < cols) {
        const uint32_t w = e4m3x4(f[0], f[1], f[2], f[3]);
        if constexpr (kV == 8)
          *reinterpret_cast<uint2*>(row + c) = make_uint2(w, e4m3x4(f[4], f[5], f[6], f[7]));
        else
          *reinterpret_cast<uint32_t*>(row + c) = w;
      }
    } else {
      const uint32_t w = e4m3x4(f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (c0 + l + 32 * j < cols) row[c0 + l + 32 * j] = (uint8_t)(w >> (8 * j));
    }
  }
};

// 448 / a as hi + lo (2^-100 <= a).  a / 256 keeps the reciprocal's argument and
// result inside the normal range.
__device__ __forceinline__ void quotient(float a, float* hi, float* lo) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * 0x1p-8f));
  *hi = 1.75f * r;
  *lo = fmaf(-*hi, a, kE4m3Max) * (r * 0x1p-8f);
}
// x * (448 / a) of N elements, in place; infinities, if there may be any, become
// +-448 (times lo they would become NaN).
template <int N>
__device__ __forceinline__ void to_code_range(float* f, float a, float hi, float lo, bool inf) {
  if (inf) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (fabsf(f[j]) == INFINITY) f[j] = copysignf(a, f[j]);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) f[j] = fmaf(f[j], hi, f[j] * lo);
}

// Rows: a CTA takes 16 (fp32 and unaligned rows: 8) rows x kRowGroups groups, a
// warp two rows (one).  CTAs go along a row first, so that the machine reads
// whole pages; all of a thread's loads are issued before the first is used.
constexpr int kRowGroups = 4;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quant_rows_kernel(const Quant a) {
  using S = Share<T, VEC>;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = (a.groups + kRowGroups - 1) / kRowGroups;
  const int rc = blockIdx.x / chunks, g0 = (blockIdx.x - rc * chunks) * kRowGroups;
  const int row = (rc * 8 + warp) * S::kRows + lane / S::kLanes;
  const int cols = row < a.rows ? a.cols : 0;
  S in[kRowGroups];
#pragma unroll
  for (int i = 0; i < kRowGroups; ++i)
    in[i].load(reinterpret_cast<const T*>(a.x) + (long long)row * a.stride, (g0 + i) * kGroup, cols);
#pragma unroll
  for (int i = 0; i < kRowGroups; ++i) {
    float m = in[i].amax();
#pragma unroll
    for (int o = 1; o < S::kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool inf = __any_sync(0xffffffffu, m == INFINITY);
    if (inf) {  // rare: once more over the finite ones
      m = in[i].amax_finite();
#pragma unroll
      for (int o = 1; o < S::kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    m = fmaxf(m, 0x1p-100f);
    float hi, lo;
    quotient(m, &hi, &lo);
    float f[S::kV];
    in[i].values(f);
    to_code_range<S::kV>(f, m, hi, lo, inf);
    S::store(a.codes + (size_t)row * a.cols, (g0 + i) * kGroup, cols, f);
    if (lane % S::kLanes == 0 && row < a.rows && g0 + i < a.groups)
      a.scales[(size_t)(g0 + i) * a.rows + row] = __fdiv_rn(m, kE4m3Max);
  }
}

// Blocks: one CTA of 16 warps per 128 x 128 block, held in registers between
// the maximum and the conversion (32 elements per thread).
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) quant_blocks_kernel(const Quant a) {
  using S = Share<T, VEC>;
  constexpr int kSteps = 128 / (16 * S::kRows);
  __shared__ float wmax[16];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = blockIdx.x, rb = blockIdx.y;
  const int row0 = rb * 128 + warp * S::kRows + lane / S::kLanes;
  S in[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int row = row0 + 16 * S::kRows * i;
    in[i].load(reinterpret_cast<const T*>(a.x) + (long long)row * a.stride, g * kGroup, row < a.rows ? a.cols : 0);
  }
  float m = 0.f;
  auto block_max = [&]() {
    m = warp_max(m);
    if (lane == 0) wmax[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) m = fmaxf(m, wmax[w]);
  };
#pragma unroll
  for (int i = 0; i < kSteps; ++i) m = fmaxf(m, in[i].amax());
  block_max();
  const bool any_inf = m == INFINITY;
  if (any_inf) {  // rare: once more over the finite ones
    m = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) m = fmaxf(m, in[i].amax_finite());
    __syncthreads();
    block_max();
  }
  m = fmaxf(m, 0x1p-100f);
  float hi, lo;
  quotient(m, &hi, &lo);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int row = row0 + 16 * S::kRows * i;
    float f[S::kV];
    in[i].values(f);
    to_code_range<S::kV>(f, m, hi, lo, any_inf);
    S::store(a.codes + (size_t)row * a.cols, g * kGroup, row < a.rows ? a.cols : 0, f);
  }
  if (threadIdx.x == 0) a.scales[(size_t)rb * a.groups + g] = __fdiv_rn(m, kE4m3Max);
}

template <typename T>
q2_status quant_t(const Quant& a, int block_rows, bool vec, cudaStream_t st) {
  if (block_rows == 1) {
    const int per = 8 * (vec ? Share<T, true>::kRows : Share<T, false>::kRows);
    const long long ctas = (long long)((a.rows + per - 1) / per) * ((a.groups + kRowGroups - 1) / kRowGroups);
    if (ctas >= (1ll << 31)) {
      set_error("quantize_q8: too many rows and columns for one call");
      return Q2_ERR_SHAPE;
    }
    const dim3 grid((unsigned)ctas);
    Q2_LAUNCH(vec ? quant_rows_kernel<T, true> : quant_rows_kernel<T, false>, grid, dim3(256), 0, st, true, a);
  } else {
    const dim3 grid(a.groups, (a.rows + 127) / 128);
    Q2_LAUNCH(vec ? quant_blocks_kernel<T, true> : quant_blocks_kernel<T, false>, grid, dim3(512), 0, st, true, a);
  }
  return Q2_OK;
}

}  // namespace

}  // namespace q2

using namespace q2;

extern "C" q2_status q2_quantize_q8(void* codes, float* scales, const void* in, size_t rows, size_t cols,
                                    size_t in_stride, int block_rows, int dtype, void* stream) {
  clear_error();
  Q2_CHECK_ARG(dtype == Q2_F32 || dtype == Q2_BF16, Q2_ERR_DTYPE, "quantize_q8: dtype must be Q2_F32 or Q2_BF16");
  Q2_CHECK_ARG(block_rows == 1 || block_rows == 128, Q2_ERR_INVALID_ARG, "quantize_q8: block_rows must be 1 or 128");
  Q2_CHECK_ARG(rows < (1u << 30) && cols < (1u << 22), Q2_ERR_SHAPE,
               "quantize_q8: need rows < 2^30 and cols < 2^22");
  Q2_CHECK_ARG(block_rows == 1 || rows <= 65535u * 128, Q2_ERR_SHAPE, "quantize_q8: too many row blocks");
  if (rows == 0 || cols == 0) return Q2_OK;
  Q2_CHECK_ARG(codes && scales && in, Q2_ERR_INVALID_ARG, "quantize_q8: NULL pointer");
  Q2_CHECK_ARG(in_stride >= cols || rows == 1, Q2_ERR_SHAPE, "quantize_q8: in_stride is below cols");
  const size_t es = dtype == Q2_BF16 ? 2 : 4;
  Quant a;
  a.x = in;
  a.stride = (long long)in_stride;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.rows = (int)rows;
  a.cols = (int)cols;
  a.groups = (int)((cols + kGroup - 1) / kGroup);
  const bool vec = cols % 16 == 0 && ((reinterpret_cast<uintptr_t>(in) | (in_stride * es) |
                                       reinterpret_cast<uintptr_t>(codes)) & 15) == 0;
  return dtype == Q2_BF16 ? quant_t<__nv_bfloat16>(a, block_rows, vec, as_stream(stream))
                          : quant_t<float>(a, block_rows, vec, as_stream(stream));
}
