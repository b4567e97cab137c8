// kv8_attn.cu -- attention over the 8-bit KV cache.
//
// One CTA per (query head, query row, sequence): online softmax in fp32 over
// tiles of 128 keys, one key per thread for the scores, one dimension per
// thread for the output.
#include "common.cuh"
#include "e4m3.cuh"
#include "kv8.h"

namespace q2 {

namespace {

constexpr int kBlk = Q2_KV8_BLOCK;
constexpr float kLog2e = 1.4426950408889634f;

struct Kv8Attn {
  const void* q;
  long long q_seq_stride, q_tok_stride;
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  const int32_t* lens;  // [batch] keys of each sequence; null: fixed_len
  int fixed_len;
  int batch, ntok, nh, nkv, max_seq, nblk;
  float scale;
  void* out;  // [batch][ntok][nh][hd]
  int* err;
};

template <typename T, int HD>
__global__ void __launch_bounds__(128) kv8_attn_simple_kernel(const Kv8Attn a) {
  __shared__ float qs[HD], p[128], red[4];
  const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int g = h / (a.nh / a.nkv);
  int len = a.lens ? a.lens[b] : a.fixed_len;
  if (len > a.max_seq) {
    if (tid == 0) atomicOr(a.err, kErrCapacity);
    len = 0;
  }
  const int n = max(0, len - a.ntok + 1 + t);  // keys that this row sees
  const T* q = reinterpret_cast<const T*>(a.q) + (long long)b * a.q_seq_stride + (long long)t * a.q_tok_stride +
               (long long)h * HD;
  if (tid < HD) qs[tid] = to_f(q[tid]);
  const size_t head = (size_t)b * a.nkv + g;
  const uint8_t* kc = a.kc + head * a.max_seq * HD;
  const uint8_t* vc = a.vc + head * a.max_seq * HD;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int k0 = 0; k0 < n; k0 += 128) {
    __syncthreads();
    float s = -INFINITY;
    if (k0 + tid < n) {
      s = 0.f;
      const uint32_t* row = reinterpret_cast<const uint32_t*>(kc + (size_t)(k0 + tid) * HD);
      for (int d = 0; d < HD / 4; ++d) {
        float f[4];
        e4m3x4_to_f(row[d], f);
        for (int j = 0; j < 4; ++j) s = fmaf(f[j], qs[4 * d + j], s);
      }
      s *= a.scale * kLog2e * a.ks[head * a.nblk + (k0 + tid) / kBlk];
    }
    float w = warp_max(s);
    if ((tid & 31) == 0) red[tid >> 5] = w;
    __syncthreads();
    const float mn = fmaxf(fmaxf(m, fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
    const float ms = mn == -INFINITY ? 0.f : mn;
    const float e = exp2f(s - ms);
    p[tid] = e;
    w = warp_sum(e);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = w;
    __syncthreads();
    const float alpha = exp2f(m - ms);
    l = l * alpha + ((red[0] + red[1]) + (red[2] + red[3]));
    o *= alpha;
    m = mn;
    if (tid < HD)
      for (int j = 0; j < min(128, n - k0); ++j) {
        float f[4];
        e4m3x4_to_f(vc[(size_t)(k0 + j) * HD + tid], f);
        o = fmaf(p[j], f[0] * a.vs[head * a.nblk + (k0 + j) / kBlk], o);
      }
  }
  if (tid < HD)
    reinterpret_cast<T*>(a.out)[(((size_t)b * a.ntok + t) * a.nh + h) * HD + tid] =
        from_f<T>(l == 0.f ? 0.f : o / l);
}

template <typename T>
q2_status simple_t(const Kv8Attn& a, int hd, cudaStream_t st) {
  const dim3 grid(a.nh, a.ntok, a.batch);
  switch (hd) {
    case 32: Q2_LAUNCH(kv8_attn_simple_kernel<T, 32>, grid, dim3(128), 0, st, false, a); break;
    case 64: Q2_LAUNCH(kv8_attn_simple_kernel<T, 64>, grid, dim3(128), 0, st, false, a); break;
    default: Q2_LAUNCH(kv8_attn_simple_kernel<T, 128>, grid, dim3(128), 0, st, false, a); break;
  }
  return Q2_OK;
}

q2_status attn(const Kv8Attn& a, int hd, int dtype, cudaStream_t st) {
  return dtype == Q2_BF16 ? simple_t<__nv_bfloat16>(a, hd, st) : simple_t<float>(a, hd, st);
}

}  // namespace

}  // namespace q2

using namespace q2;

// The checks that both calls share.
#define Q2_KV8_ATTN_CHECK(who)                                                                                   \
  Q2_CHECK_ARG(dtype == Q2_F32 || dtype == Q2_BF16, Q2_ERR_DTYPE, who ": dtype must be Q2_F32 or Q2_BF16");     \
  Q2_CHECK_ARG(hd == 32 || hd == 64 || hd == 128, Q2_ERR_SHAPE, who ": hd must be 32, 64 or 128");               \
  Q2_CHECK_ARG(nkv > 0 && nh > 0 && nh % nkv == 0 && nh / nkv <= 8, Q2_ERR_SHAPE,                                \
               who ": need nh % nkv == 0 and nh / nkv <= 8");                                                    \
  Q2_CHECK_ARG(max_seq > 0 && max_seq < (1u << 30) && nh < 16384, Q2_ERR_SHAPE, who ": size out of range")
#define Q2_KV8_ATTN_PTRS(who)                                                                                    \
  Q2_CHECK_ARG(out && q && kc && vc && ks && vs, Q2_ERR_INVALID_ARG, who ": NULL pointer");                      \
  Q2_CHECK_ARG(((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15) == 0,                  \
               Q2_ERR_INVALID_ARG, who ": the codes must be 16-byte aligned")

extern "C" {

q2_status q2_kv8_attention(void* out, const void* q, const int64_t* q_strides, const void* kc, const void* vc,
                           const float* ks, const float* vs, const int32_t* lens, size_t batch, size_t ntok,
                           size_t nh, size_t nkv, size_t hd, size_t max_seq, float scale, int dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  Q2_KV8_ATTN_CHECK("kv8_attention");
  Q2_CHECK_ARG(batch < 32768, Q2_ERR_SHAPE, "kv8_attention: need batch < 32768");
  Q2_CHECK_ARG(ntok <= max_seq && ntok < 65536, Q2_ERR_CAPACITY, "kv8_attention: ntok is past max_seq or 65535");
  if (batch == 0 || ntok == 0) return Q2_OK;
  Q2_KV8_ATTN_PTRS("kv8_attention");
  Q2_CHECK_ARG(lens, Q2_ERR_INVALID_ARG, "kv8_attention: NULL lens");
  int* flag = op_error_flag();
  Q2_CHECK_ARG(flag, Q2_ERR_CUDA, "cannot resolve the device error flag");
  Q2_CHECK_ARG(workspace && workspace_bytes >= 256, Q2_ERR_INVALID_ARG, "kv8_attention: the workspace is too small");
  Kv8Attn a;
  a.q = q;
  a.q_seq_stride = q_strides ? q_strides[0] : (long long)(ntok * nh * hd);
  a.q_tok_stride = q_strides ? q_strides[1] : (long long)(nh * hd);
  a.kc = static_cast<const uint8_t*>(kc);
  a.vc = static_cast<const uint8_t*>(vc);
  a.ks = ks;
  a.vs = vs;
  a.lens = lens;
  a.fixed_len = 0;
  a.batch = (int)batch;
  a.ntok = (int)ntok;
  a.nh = (int)nh;
  a.nkv = (int)nkv;
  a.max_seq = (int)max_seq;
  a.nblk = (int)((max_seq + kBlk - 1) / kBlk);
  a.scale = scale;
  a.out = out;
  a.err = flag;
  return attn(a, (int)hd, dtype, as_stream(stream));
}

q2_status q2_kv8_self_attention(void* out, const void* q, const void* kc, const void* vc, const float* ks,
                                const float* vs, size_t seqlen, size_t total_len, size_t nh, size_t nkv, size_t hd,
                                size_t max_seq, float scale, int dtype, void* workspace, size_t workspace_bytes,
                                void* stream) {
  clear_error();
  Q2_KV8_ATTN_CHECK("kv8_self_attention");
  Q2_CHECK_ARG(seqlen <= total_len, Q2_ERR_SHAPE, "kv8_self_attention: seqlen > total_len");
  Q2_CHECK_ARG(total_len <= max_seq, Q2_ERR_CAPACITY, "kv8_self_attention: total_len is past max_seq");
  Q2_CHECK_ARG(seqlen < 65536, Q2_ERR_SHAPE, "kv8_self_attention: need seqlen < 65536");
  if (seqlen == 0) return Q2_OK;
  Q2_KV8_ATTN_PTRS("kv8_self_attention");
  int* flag = op_error_flag();
  Q2_CHECK_ARG(flag, Q2_ERR_CUDA, "cannot resolve the device error flag");
  Q2_CHECK_ARG(workspace && workspace_bytes >= 256, Q2_ERR_INVALID_ARG,
               "kv8_self_attention: the workspace is too small");
  Kv8Attn a;
  a.q = q;
  a.q_seq_stride = 0;
  a.q_tok_stride = (long long)(nh * hd);
  a.kc = static_cast<const uint8_t*>(kc);
  a.vc = static_cast<const uint8_t*>(vc);
  a.ks = ks;
  a.vs = vs;
  a.lens = nullptr;
  a.fixed_len = (int)total_len;
  a.batch = 1;
  a.ntok = (int)seqlen;
  a.nh = (int)nh;
  a.nkv = (int)nkv;
  a.max_seq = (int)max_seq;
  a.nblk = (int)((max_seq + kBlk - 1) / kBlk);
  a.scale = scale;
  a.out = out;
  a.err = flag;
  return attn(a, (int)hd, dtype, as_stream(stream));
}

q2_status q2_kv8_attention_workspace(size_t batch, size_t ntok, size_t total_len, size_t nh, size_t nkv, size_t hd,
                                     int dtype, size_t* bytes) {
  clear_error();
  const size_t max_seq = 1;
  Q2_KV8_ATTN_CHECK("kv8_attention_workspace");
  Q2_CHECK_ARG(bytes, Q2_ERR_INVALID_ARG, "kv8_attention_workspace: NULL bytes");
  (void)batch;
  (void)ntok;
  (void)total_len;
  *bytes = 256;
  return Q2_OK;
}

}  // extern "C"
