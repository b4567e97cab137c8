// kv8.h -- internal launchers of the 8-bit KV cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/q2.h"
#include "kernels.h"

namespace q2 {

// Dequantised K and V rows of positions [start, start + ntok) of each sequence.
struct Kv8Read {
  void* k;
  void* v;
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  const int32_t* start;  // [batch], or null: every sequence from position 0
  long long seq_stride, tok_stride, head_stride;  // of k and v, in elements
  int batch, ntok, nkv, hd, max_seq;
  // With vnan (int [nkv][hd], zero): a NaN of V reads as 0 and vnan[g][d]
  // becomes the largest INT32_MAX - position over the NaNs of that dimension, and V
  // reads times kKv8VFactor.
  int* vnan;
};
// The prompt attention's copy of V is scaled by this, and its result back: sums of
// values near the largest, 448 * 2^119, stay in fp32's range, and the smallest,
// 2^-69, in bf16's normal range.
constexpr float kKv8VFactor = 0x1p-40f;
q2_status launch_kv8_read(const Kv8Read& a, int dtype, int* err, cudaStream_t st);

// launch_attn_tc with V's NaN kept apart: vnan is null, or int [nkv][hd] with
// INT32_MAX - p for a V with its first NaN of that dim at position p (taken out
// of V), 0 for none; rows from p on get NaN there.  V is the cache's times
// kKv8VFactor then.
q2_status launch_attn_tc_nan(const AttnRows& a, void* ws, int* err, cudaStream_t st, const int* vnan);
// What one call of this size needs of its scratch (counters, then its slots).
size_t attn_tc_ws_need(int rows, int pos0, int nh);

}  // namespace q2
