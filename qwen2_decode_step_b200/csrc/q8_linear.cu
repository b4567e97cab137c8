// q8_linear.cu -- the 8-bit linear: e4m3 activations times e4m3 weights with an
// fp32 scale per group of 128 along the reduction.
//
//   out[m, n] = sum_g xs[g][m] * ws[n / 128][g] * sum_{k in group g} x[m, k] w[n, k]  (+ bias[n])
//
// One thread per output, fp32 sums.
#include "common.cuh"
#include "e4m3.cuh"

namespace q2 {

namespace {

constexpr int kGroup = Q2_Q8_GROUP;

struct Q8Lin {
  const uint8_t* x;   // [M][K]
  const float* xs;    // [groups][M]
  const uint8_t* w;   // [N][K]
  const float* ws;    // [N / 128][groups]
  const void* bias;   // [N] or null
  void* out;          // [M][N]
  int M, N, K, groups;
};

template <typename T>
__global__ void __launch_bounds__(128) q8_linear_simple_kernel(const Q8Lin a) {
  const int n = blockIdx.x * 128 + threadIdx.x, m = blockIdx.y;
  if (n >= a.N) return;
  const uint8_t* x = a.x + (size_t)m * a.K;
  const uint8_t* w = a.w + (size_t)n * a.K;
  float y = 0.f;
  for (int g = 0; g < a.groups; ++g) {
    float s = 0.f;
    for (int k = g * kGroup; k < min(a.K, (g + 1) * kGroup); k += 4) {
      float f[4], h[4];
      e4m3x4_to_f(*reinterpret_cast<const uint32_t*>(x + k), f);
      e4m3x4_to_f(*reinterpret_cast<const uint32_t*>(w + k), h);
      for (int j = 0; j < 4; ++j) s = fmaf(f[j], h[j], s);
    }
    y = fmaf(s, a.xs[(size_t)g * a.M + m] * a.ws[(size_t)(n / 128) * a.groups + g], y);
  }
  if (a.bias) y += to_f(reinterpret_cast<const T*>(a.bias)[n]);
  reinterpret_cast<T*>(a.out)[(size_t)m * a.N + n] = from_f<T>(y);
}

}  // namespace

}  // namespace q2

using namespace q2;

extern "C" q2_status q2_linear_q8(void* out, const void* xq, const float* xs, const void* wq, const float* ws,
                                  const void* bias, size_t M, size_t N, size_t K, int dtype, void* stream) {
  clear_error();
  Q2_CHECK_ARG(dtype == Q2_F32 || dtype == Q2_BF16, Q2_ERR_DTYPE, "linear_q8: dtype must be Q2_F32 or Q2_BF16");
  Q2_CHECK_ARG(K > 0 && K % 16 == 0 && K < (1u << 22), Q2_ERR_SHAPE,
               "linear_q8: K must be a positive multiple of 16 below 2^22");
  Q2_CHECK_ARG(M < (1u << 30) && N < (1u << 30), Q2_ERR_SHAPE, "linear_q8: size too large");
  if (M == 0 || N == 0) return Q2_OK;
  Q2_CHECK_ARG(out && xq && xs && wq && ws, Q2_ERR_INVALID_ARG, "linear_q8: NULL pointer");
  Q2_CHECK_ARG(((reinterpret_cast<uintptr_t>(xq) | reinterpret_cast<uintptr_t>(wq)) & 15) == 0, Q2_ERR_INVALID_ARG,
               "linear_q8: the codes must be 16-byte aligned");
  Q8Lin a;
  a.x = static_cast<const uint8_t*>(xq);
  a.xs = xs;
  a.w = static_cast<const uint8_t*>(wq);
  a.ws = ws;
  a.bias = bias;
  a.out = out;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.groups = (int)((K + kGroup - 1) / kGroup);
  const dim3 grid((a.N + 127) / 128, a.M);
  Q2_CHECK_ARG(M < 65536, Q2_ERR_SHAPE, "linear_q8: too many rows");
  cudaStream_t st = as_stream(stream);
  if (dtype == Q2_BF16)
    Q2_LAUNCH(q8_linear_simple_kernel<__nv_bfloat16>, grid, dim3(128), 0, st, false, a);
  else
    Q2_LAUNCH(q8_linear_simple_kernel<float>, grid, dim3(128), 0, st, false, a);
  return Q2_OK;
}
