// q8_quant.cu -- the operands of the 8-bit linear: rows (activations) or 128 x
// 128 blocks (weights) quantised to e4m3 with an fp32 scale per group.
//
//   a = max(largest finite |x| of the group, 2^-100)
//   scale = a / 448,  code = e4m3(x * (448 / a))
// Two divisions per group and none per element (an IEEE division each would
// cost more issue slots than the loads leave): 448 / a is kept as hi + lo, lo
// the remainder of the rounded quotient, and x * hi + x * lo is one fused
// rounding from the quotient of the definition, where x * hi alone would fall
// on the other side of a code's border about three times as often.  The lower
// bound on a keeps 448 / a finite; a group of zeros gets codes of 0.
//
// Bound by HBM: the input once, a byte per element out, 4 bytes per group.
#include "common.cuh"
#include "e4m3.cuh"

namespace q2 {

namespace {

constexpr int kGroup = Q2_Q8_GROUP;
constexpr int kItemsGroup = kGroup / 16;  // eight lanes hold a row of a group

struct Quant {
  const void* x;
  long long stride;  // elements between rows of x
  uint8_t* codes;    // [rows][cols]
  float* scales;     // rows: [groups][rows]; blocks: [row blocks][groups]
  int rows, cols, groups;
};

// The largest finite magnitude of sixteen elements (fmaxf passes over NaN);
// `inf` says whether an infinity was among them, which is rare and settled out
// of the way of the others.
__device__ __forceinline__ float thread_amax(const float* f, bool* inf) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int j = 1; j < 16; ++j) m = fmaxf(m, fabsf(f[j]));
  *inf = m == INFINITY;
  if (*inf) {
    m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, finite_abs(f[j]));
  }
  return m;
}

// x * (448 / a) of sixteen elements, in place (infinities go to +-448 here:
// times lo they would become NaN).
__device__ __forceinline__ void to_code_range(float* f, float a, bool inf) {
  if (inf) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (fabsf(f[j]) == INFINITY) f[j] = copysignf(a, f[j]);
  }
  const float hi = __fdiv_rn(kE4m3Max, a);
  const float lo = __fdiv_rn(fmaf(-hi, a, kE4m3Max), a);
#pragma unroll
  for (int j = 0; j < 16; ++j) f[j] = fmaf(f[j], hi, f[j] * lo);
}

// Rows: a CTA takes 32 rows x kRowGroups groups.  A warp takes one group of
// four rows (eight lanes each), so the CTA's scales of a group are 32
// consecutive floats of the [groups][rows] array and every row segment it
// reads is 256 bytes of bf16; all of a thread's loads are issued before the
// first is used.
constexpr int kRowGroups = 4;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quant_rows_kernel(const Quant a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + warp * 4 + (lane >> 3);
  const int g0 = blockIdx.y * kRowGroups;
  const bool in = row < a.rows;
  const T* x = reinterpret_cast<const T*>(a.x) + (long long)row * a.stride;
  float f[kRowGroups][16];
#pragma unroll
  for (int i = 0; i < kRowGroups; ++i) {
    const int c = (g0 + i) * kGroup + (lane & 7) * 16;
    const int n = in ? min(16, a.cols - c) : 0;
    if (n > 0) {
      load16<T, VEC>(x + c, n, f[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kRowGroups; ++i) {
    bool inf;
    float m = thread_amax(f[i], &inf);
#pragma unroll
    for (int o = 1; o < kItemsGroup; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(m, 0x1p-100f);
    const int c = (g0 + i) * kGroup + (lane & 7) * 16;
    const int n = in ? min(16, a.cols - c) : 0;
    to_code_range(f[i], m, inf);
    if (n > 0) store16_e4m3<VEC>(a.codes + (size_t)row * a.cols + c, n, f[i]);
    if (in && (lane & 7) == 0 && g0 + i < a.groups)
      a.scales[(size_t)(g0 + i) * a.rows + row] = __fdiv_rn(m, kE4m3Max);
  }
}

// Blocks: one CTA per 128 x 128 block, held in registers between the maximum
// and the conversion (32 elements per thread).
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) quant_blocks_kernel(const Quant a) {
  __shared__ float wmax[16];
  pdl_launch_dependents();
  pdl_wait();
  const int g = blockIdx.x, rb = blockIdx.y;
  const int c = g * kGroup + (threadIdx.x & 7) * 16, r0 = rb * 128 + (threadIdx.x >> 3);
  const int n = min(16, a.cols - c);
  float f[2][16];
  bool inf[2];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = r0 + 64 * i;
    if (row < a.rows && n > 0) {
      load16<T, VEC>(reinterpret_cast<const T*>(a.x) + (long long)row * a.stride + c, n, f[i]);
      m = fmaxf(m, thread_amax(f[i], &inf[i]));
    }
  }
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) m = fmaxf(m, wmax[w]);
  m = fmaxf(m, 0x1p-100f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = r0 + 64 * i;
    if (row < a.rows && n > 0) {
      to_code_range(f[i], m, inf[i]);
      store16_e4m3<VEC>(a.codes + (size_t)row * a.cols + c, n, f[i]);
    }
  }
  if (threadIdx.x == 0) a.scales[(size_t)rb * a.groups + g] = __fdiv_rn(m, kE4m3Max);
}

template <typename T>
q2_status quant_t(const Quant& a, int block_rows, bool vec, cudaStream_t st) {
  if (block_rows == 1) {
    const dim3 grid((a.rows + 31) / 32, (a.groups + kRowGroups - 1) / kRowGroups);
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
