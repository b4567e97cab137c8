// kv8.cu -- the 8-bit KV cache: keys and values quantised to e4m3 as they are
// written, and read back.
//
// Layout: codes [batch][nkv][max_seq][hd], scales [batch][nkv][ceil(max_seq /
// 64)] in fp32, one per block of 64 positions of one kv head.  The scale is a
// power of two, s = 2^k with the least k in [-60, 119] for which the block's
// largest finite magnitude is at most 448 s.  A power of two costs e4m3 none of
// its relative precision (the codes only sit up to one binade lower), it makes
// v / s and code * s exact, and when a later token raises a block's scale the
// earlier codes change by a shift of the exponent: they are rounded again only
// where they fall into e4m3's subnormals.  The bounds on k keep the products
// of any two scales, and code * s in bf16, inside the normal range.
#include "common.cuh"
#include "e4m3.cuh"
#include "kv8.h"

namespace q2 {

namespace {

constexpr int kBlk = Q2_KV8_BLOCK;
constexpr int kThreads = 256;
constexpr int kKMin = -60, kKMax = 119;

// 2^k of the block scale for a largest finite magnitude amax (>= 0).  448 is
// 1.75 * 2^8: with amax = 1.f * 2^e, k = e - 8, one more where 1.f > 1.75.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int k = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = min(max(k, kKMin), kKMax);
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

struct Kv8Append {
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  const void* k;
  const void* v;
  long long k_seq_stride, k_tok_stride, v_seq_stride, v_tok_stride;  // of k and v, in elements
  const int32_t* start;
  int batch, ntok, nkv, max_seq, nblk;
  int* err;
};

// One CTA writes one block of 64 positions (those of its rows that are new) of
// one kv head of K or of V: it owns the block's codes and scale, so nothing
// races.  Bound by HBM for long prompts (bf16 in, a byte out) and by launch
// latency for one token.  An item is 16 bytes of a new row, so a warp's loads
// are whole lines; a thread keeps its items (at most eight, fp32 and hd 128) in
// registers between the maximum and the conversion: the rows are read once.
template <typename T, int HD, bool VEC>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const Kv8Append a) {
  constexpr int kV = Storage<T>::kVec;
  constexpr int kItemsRow = HD / kV;
  constexpr int kPer = (kBlk * kItemsRow + kThreads - 1) / kThreads;
  __shared__ float wmax[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const bool isv = blockIdx.y & 1;
  const int g = blockIdx.y >> 1, b = blockIdx.z, tid = threadIdx.x;
  const int start = a.start[b];
  if (start < 0) return;  // an inactive sequence
  if (a.ntok > a.max_seq - start) {
    if (tid == 0) atomicOr(a.err, kErrCapacity);
    return;
  }
  const int blk = start / kBlk + blockIdx.x;
  const int p0 = blk * kBlk;                              // the block's first position
  const int lo = max(start, p0), hi = min(start + a.ntok, p0 + kBlk);  // the new ones
  if (lo >= hi) return;
  const size_t head = (size_t)b * a.nkv + g;
  uint8_t* codes = (isv ? a.vc : a.kc) + (head * a.max_seq + p0) * HD;
  float* scale = (isv ? a.vs : a.ks) + head * a.nblk + blk;
  const long long tok_stride = isv ? a.v_tok_stride : a.k_tok_stride;
  const T* x = reinterpret_cast<const T*>(isv ? a.v : a.k) + (long long)b * (isv ? a.v_seq_stride : a.k_seq_stride) +
               (long long)(lo - start) * tok_stride + (long long)g * HD;

  float f[kPer][kV];
  const int n = (hi - lo) * kItemsRow;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int it = tid + i * kThreads;
    const T* p = x + (long long)(it / kItemsRow) * tok_stride + (it % kItemsRow) * kV;
    if (it < n) {
      if constexpr (VEC) {
        unpack16<T>(*reinterpret_cast<const uint4*>(p), f[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) f[i][j] = to_f(p[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) f[i][j] = 0.f;
    }
  }
  const float before = lo > p0 ? *scale : 0.f;
  float m = 0.f;
  auto block_max = [&]() {
    m = warp_max(m);
    if ((tid & 31) == 0) wmax[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, wmax[w]);
  };
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < kV; ++j) m = fmaxf(m, fabsf(f[i][j]));  // (passes over NaN)
  block_max();
  if (m == INFINITY) {  // rare: once more over the finite ones
    m = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int j = 0; j < kV; ++j) m = fmaxf(m, finite_abs(f[i][j]));
    __syncthreads();
    block_max();
  }
  const float s = fmaxf(block_scale(m), before);
  const float inv = 1.f / s;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int it = tid + i * kThreads;
    if (it >= n) break;
    uint32_t w[kV / 4];
#pragma unroll
    for (int j = 0; j < kV / 4; ++j)
      w[j] = e4m3x4(f[i][4 * j] * inv, f[i][4 * j + 1] * inv, f[i][4 * j + 2] * inv, f[i][4 * j + 3] * inv);
    uint8_t* o = codes + (size_t)(lo - p0) * HD + (size_t)it * kV;
    if constexpr (kV == 8)
      *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(o) = w[0];
  }
  if (lo > p0 && s != before) {  // the earlier codes of the block move to the new scale
    const float ratio = before * inv;
    for (int it = tid; it < (lo - p0) * (HD / 4); it += kThreads) {
      uint32_t* p = reinterpret_cast<uint32_t*>(codes) + it;
      float o[4];
      e4m3x4_to_f(*p, o);
      *p = e4m3x4(o[0] * ratio, o[1] * ratio, o[2] * ratio, o[3] * ratio);
    }
  }
  if (tid == 0) *scale = s;  // every thread has read it: the barrier above
}

// One CTA reads 64 consecutive positions of one sequence and kv head of K or of
// V.  Bound by HBM: a byte in, two or four out per element.  A thread's
// item is 16 bytes of output, so a warp's stores are whole lines (with 16 codes
// an item they were 64 bytes apart: 22 us instead of 15 for 32768 positions
// of two heads to fp32); its loads are issued before the first store.
template <typename T, int HD, bool VEC>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const Kv8Read a, int nblk, int* err) {
  constexpr int kV = Storage<T>::kVec;   // 4 or 8 elements
  constexpr int kItemsRow = HD / kV;
  constexpr int kItems = kBlk * kItemsRow;
  constexpr int kPer = (kItems + kThreads - 1) / kThreads;
  pdl_launch_dependents();
  pdl_wait();
  const bool isv = blockIdx.y & 1;
  const int b = blockIdx.y >> 1, t0 = blockIdx.x * kBlk;
  const int start = a.start ? a.start[b] : 0;
  if (start < 0 || a.ntok > a.max_seq - start) {
    if (start >= 0 && threadIdx.x == 0) atomicOr(err, kErrCapacity);
    return;
  }
  const int n = min(kBlk, a.ntok - t0) * kItemsRow;
  const int g = blockIdx.z;
  const size_t head = (size_t)b * a.nkv + g;
  const uint8_t* codes = (isv ? a.vc : a.kc) + (head * a.max_seq + start + t0) * HD;
  const float* scale = (isv ? a.vs : a.ks) + head * nblk;
  T* out = reinterpret_cast<T*>(isv ? a.v : a.k) + (long long)b * a.seq_stride + (long long)g * a.head_stride;
  uint2 w[kPer];
  // the tile's 64 positions lie in two blocks at most
  const int b0 = (start + t0) / kBlk, split = (b0 + 1) * kBlk - start - t0;  // rows of the tile in the first
  const float by = isv && a.vnan ? kKv8VFactor : 1.f;
  const float s0 = __ldg(scale + b0) * by, s1 = __ldg(scale + min(b0 + 1, nblk - 1)) * by;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int it = threadIdx.x + i * kThreads;
    w[i] = make_uint2(0u, 0u);
    if (it < n) {
      if constexpr (kV == 8)
        w[i] = __ldg(reinterpret_cast<const uint2*>(codes) + it);
      else
        w[i].x = __ldg(reinterpret_cast<const uint32_t*>(codes) + it);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int it = threadIdx.x + i * kThreads;
    if (it >= n) break;
    const int t = t0 + it / kItemsRow, d = (it % kItemsRow) * kV;
    float f[kV];
    e4m3x4_to_f(w[i].x, f);
    if constexpr (kV == 8) e4m3x4_to_f(w[i].y, f + 4);
    if (isv && a.vnan) {
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (isnan(f[j])) {
          f[j] = 0.f;
          atomicMax(a.vnan + g * HD + d + j, INT32_MAX - (start + t));
        }
    }
    T* o = out + (long long)t * a.tok_stride + d;
#pragma unroll
    for (int j = 0; j < kV; ++j) f[j] *= it / kItemsRow < split ? s0 : s1;
    if constexpr (VEC) {
      *reinterpret_cast<uint4*>(o) = pack16<T>(f);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) o[j] = from_f<T>(f[j]);
    }
  }
}

template <typename T, int HD>
q2_status append_t(const Kv8Append& a, bool vec, cudaStream_t st) {
  const dim3 grid((a.ntok + kBlk - 2) / kBlk + 1, 2 * a.nkv, a.batch);
  Q2_LAUNCH(vec ? kv8_append_kernel<T, HD, true> : kv8_append_kernel<T, HD, false>, grid, dim3(kThreads), 0, st,
            true, a);
  return Q2_OK;
}

template <typename T, int HD>
q2_status read_t(const Kv8Read& a, bool vec, int* err, cudaStream_t st) {
  const dim3 grid((a.ntok + kBlk - 1) / kBlk, 2 * a.batch, a.nkv);
  Q2_LAUNCH(vec ? kv8_read_kernel<T, HD, true> : kv8_read_kernel<T, HD, false>, grid, dim3(kThreads), 0, st, true,
            a, (a.max_seq + kBlk - 1) / kBlk, err);
  return Q2_OK;
}

// Whether rows of `es`-byte elements at p with these strides start on 16 bytes.
bool rows_aligned(const void* p, long long s0, long long s1, size_t es) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(s0 * (long long)es) | (uintptr_t)(s1 * (long long)es)) & 15) == 0;
}

}  // namespace

q2_status launch_kv8_read(const Kv8Read& a, int dtype, int* err, cudaStream_t st) {
  const size_t es = dtype == Q2_BF16 ? 2 : 4;
  const bool vec = rows_aligned(a.k, a.seq_stride, a.tok_stride, es) && rows_aligned(a.v, a.head_stride, 0, es);
  const bool bf = dtype == Q2_BF16;
  switch (a.hd) {
    case 32: return bf ? read_t<__nv_bfloat16, 32>(a, vec, err, st) : read_t<float, 32>(a, vec, err, st);
    case 64: return bf ? read_t<__nv_bfloat16, 64>(a, vec, err, st) : read_t<float, 64>(a, vec, err, st);
    default: return bf ? read_t<__nv_bfloat16, 128>(a, vec, err, st) : read_t<float, 128>(a, vec, err, st);
  }
}

}  // namespace q2

using namespace q2;

extern "C" {

// The checks that every call on the cache shares.
#define Q2_KV8_CHECK(who)                                                                                        \
  Q2_CHECK_ARG(dtype == Q2_F32 || dtype == Q2_BF16, Q2_ERR_DTYPE, who ": dtype must be Q2_F32 or Q2_BF16");     \
  Q2_CHECK_ARG(hd == 32 || hd == 64 || hd == 128, Q2_ERR_SHAPE, who ": hd must be 32, 64 or 128");               \
  Q2_CHECK_ARG(nkv > 0 && nkv < 16384 && max_seq > 0 && batch < 32768, Q2_ERR_SHAPE,                             \
               who ": need 0 < nkv < 16384, max_seq > 0 and batch < 32768");                                     \
  Q2_CHECK_ARG(max_seq < (1u << 30) && ntok < (1u << 30), Q2_ERR_SHAPE, who ": size too large");                 \
  Q2_CHECK_ARG(ntok <= max_seq, Q2_ERR_CAPACITY, who ": ntok is past max_seq");                                  \
  if (batch == 0 || ntok == 0) return Q2_OK;                                                                     \
  Q2_CHECK_ARG(kc && vc && ks && vs && k && v && start, Q2_ERR_INVALID_ARG, who ": NULL pointer");               \
  Q2_CHECK_ARG(((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15) == 0,                  \
               Q2_ERR_INVALID_ARG, who ": the codes must be 16-byte aligned")

q2_status q2_kv8_append(void* kc, void* vc, float* ks, float* vs, const void* k, const void* v,
                        const int64_t* k_strides, const int64_t* v_strides, const int32_t* start, size_t batch,
                        size_t ntok, size_t nkv, size_t hd, size_t max_seq, int dtype, void* stream) {
  clear_error();
  Q2_KV8_CHECK("kv8_append");
  int* flag = op_error_flag();
  Q2_CHECK_ARG(flag, Q2_ERR_CUDA, "cannot resolve the device error flag");
  Kv8Append a;
  a.kc = static_cast<uint8_t*>(kc);
  a.vc = static_cast<uint8_t*>(vc);
  a.ks = ks;
  a.vs = vs;
  a.k = k;
  a.v = v;
  a.k_seq_stride = k_strides ? k_strides[0] : (long long)(ntok * nkv * hd);
  a.k_tok_stride = k_strides ? k_strides[1] : (long long)(nkv * hd);
  a.v_seq_stride = v_strides ? v_strides[0] : (long long)(ntok * nkv * hd);
  a.v_tok_stride = v_strides ? v_strides[1] : (long long)(nkv * hd);
  a.start = start;
  a.batch = (int)batch;
  a.ntok = (int)ntok;
  a.nkv = (int)nkv;
  a.max_seq = (int)max_seq;
  a.nblk = (int)((max_seq + kBlk - 1) / kBlk);
  a.err = flag;
  const size_t es = dtype == Q2_BF16 ? 2 : 4;
  const bool vec = rows_aligned(k, a.k_seq_stride, a.k_tok_stride, es) &&
                   rows_aligned(v, a.v_seq_stride, a.v_tok_stride, es);
  const bool bf = dtype == Q2_BF16;
  cudaStream_t st = as_stream(stream);
  switch (hd) {
    case 32: return bf ? append_t<__nv_bfloat16, 32>(a, vec, st) : append_t<float, 32>(a, vec, st);
    case 64: return bf ? append_t<__nv_bfloat16, 64>(a, vec, st) : append_t<float, 64>(a, vec, st);
    default: return bf ? append_t<__nv_bfloat16, 128>(a, vec, st) : append_t<float, 128>(a, vec, st);
  }
}

q2_status q2_kv8_read(void* k, void* v, const void* kc, const void* vc, const float* ks, const float* vs,
                      const int32_t* start, size_t batch, size_t ntok, size_t nkv, size_t hd, size_t max_seq,
                      int dtype, void* stream) {
  clear_error();
  Q2_KV8_CHECK("kv8_read");
  int* flag = op_error_flag();
  Q2_CHECK_ARG(flag, Q2_ERR_CUDA, "cannot resolve the device error flag");
  Kv8Read a;
  a.k = k;
  a.v = v;
  a.kc = static_cast<const uint8_t*>(kc);
  a.vc = static_cast<const uint8_t*>(vc);
  a.ks = ks;
  a.vs = vs;
  a.start = start;
  a.seq_stride = (long long)(ntok * nkv * hd);
  a.tok_stride = (long long)(nkv * hd);
  a.head_stride = (long long)hd;
  a.batch = (int)batch;
  a.ntok = (int)ntok;
  a.nkv = (int)nkv;
  a.hd = (int)hd;
  a.max_seq = (int)max_seq;
  a.vnan = nullptr;
  return launch_kv8_read(a, dtype, flag, as_stream(stream));
}

}  // extern "C"
