// q8_linear.cu -- the 8-bit linear on the sm_100a tensor cores: e4m3 activations
// times e4m3 weights, an fp32 scale per group of 128 along the reduction.
//
//   out[m, n] = sum_g xs[g][m] * ws[n / 128][g] * P_g[m, n]  (+ bias[n]),
//   P_g[m, n] = sum over the 128 k of group g of x[m, k] w[n, k]
//
// P_g is one 128-byte-wide step of tcgen05.mma (kind::f8f6f4, four
// instructions of 32) into a fresh accumulator in tensor memory; the epilogue
// warps read it back, multiply by the group's two scales and add it in fp32
// registers, while the MMA fills the next of kAcc accumulators.  So the tensor
// core's own sums are never longer than 128 and every scale is applied in fp32.
//
// Two forms, by which operand sits on the 128 TMEM lanes:
//   tall  (M <= 64)  the weight rows on the lanes, BN = 16, 32 or 64 tokens on
//         the columns: bound by the weight bytes (HBM).  A lane's weight scale
//         is the tile's; the tokens' scales are one per lane and reach the
//         others by shuffle.
//   wide  (M > 64)   128 tokens on the lanes, BN features on the columns: bound
//         by the tensor core.  A thread owns a token, so its scale is one
//         register and one weight scale serves its 32 columns: one packed
//         two-lane FMA per two products and no operand but registers (with the
//         weights on the lanes every column would need its own scale from
//         shared memory).
// Warp roles (320 threads, one CTA per SM, persistent over the tiles): warp 0
// TMA (a 128 x 128-byte and a BN x 128-byte box per group, 128-byte swizzle, a
// ring of STAGES), warp 1 tensor memory and MMA, warps 2-9 epilogue: two per
// TMEM lane quarter, each half of the columns.
// When the tiles alone leave SMs idle, a cluster of up to 8 CTAs splits the
// groups of one tile: each leaves its fp32 partial tile in its shared memory
// and every CTA adds one share of it over the cluster in rank order
// (distributed shared memory; no workspace, no second launch, the same sum
// every time).
// Every wait is bounded: one that runs out sets value 2 in the device error
// word and the kernel carries on to its end.
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "e4m3.cuh"
#include "tcgen05.cuh"
#include "tma.h"

namespace q2 {

using bf16 = __nv_bfloat16;

namespace {

constexpr int kGroup = Q2_Q8_GROUP;
constexpr int kLanes = 128;                 // rows of the lane-side operand per tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kClusterMax = 8;

struct Q8Lin {
  const float* xs;    // [groups][M]
  const float* ws;    // [ceil(N / 128)][groups]
  const void* bias;   // [N] or null
  void* out;          // [M][N]
  int M, N, groups;
  int out_f32;
  int lane_tiles, tiles;  // of the lane-side operand; of the output
  int csize;          // CTAs that share a tile
  int g_per;          // groups per CTA of a cluster
  int vec;            // rows of out start on 16 bytes
  int* err;
};

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, e4m3 A and B, both
// K-major, N = bn, M = 128.
__host__ __device__ constexpr uint32_t idesc_e4m3(int bn) {
  return (1u << 4) | ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(kLanes >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// NC consecutive fp32 columns (8, 16 or 32) of this thread's TMEM lane.
template <int NC>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
  if constexpr (NC == 32) {
    tmem_ld32(taddr, v);
  } else if constexpr (NC == 16) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  } else {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
  }
}

template <int BN, int STAGES>
struct Q8Smem {
  static constexpr size_t kA = (size_t)kLanes * kGroup;
  static constexpr size_t kB = (size_t)BN * kGroup;
  static constexpr size_t kStage = kA + kB;
  // accumulators in tensor memory: as many as fit 512 columns, at most four
  static constexpr int kAcc = BN > 128 ? 2 : 4;
  static constexpr int kCols = kAcc * BN <= 64 ? 64 : kAcc * BN <= 128 ? 128 : kAcc * BN <= 256 ? 256 : 512;
  static constexpr size_t kBars = (2 * STAGES + 2 * kAcc) * 8 + 16;
  static constexpr size_t kTotal = STAGES * kStage + kBars + 1024;  // + alignment slack
  // a cluster's partial tile, [column][lane], lanes padded to an odd stride so
  // that it can be walked along either axis
  static constexpr int kPartStride = kLanes + 1;
  static constexpr bool kFits = (size_t)BN * kPartStride * 4 <= STAGES * kStage;
};

__device__ __forceinline__ void store_out(const Q8Lin& a, int m, int n, float y) {
  const size_t i = (size_t)m * a.N + n;
  if (a.out_f32) {
    if (a.bias) y += reinterpret_cast<const float*>(a.bias)[n];
    reinterpret_cast<float*>(a.out)[i] = y;
  } else {
    if (a.bias) y += to_f(reinterpret_cast<const bf16*>(a.bias)[n]);
    reinterpret_cast<bf16*>(a.out)[i] = from_f<bf16>(y);
  }
}

// ta: the lane-side operand's map, tb: the column-side one's.
template <bool WIDE, int BN, int STAGES>
__global__ void __launch_bounds__(kThreads, 1)
    q8_linear_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const Q8Lin a) {
  using SM = Q8Smem<BN, STAGES>;
  static_assert(SM::kFits && SM::kAcc * BN <= 512, "the partial tile fits the ring, the accumulators tensor memory");
  extern __shared__ __align__(1024) uint8_t q8_smem_raw[];
  uint8_t* smem = q8_smem_raw + ((1024u - (smem_u32(q8_smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * SM::kStage);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + SM::kAcc;
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(acc_empty + SM::kAcc);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % a.csize;  // of the cluster (csize consecutive CTAs)
  const int first = blockIdx.x / a.csize, step = gridDim.x / a.csize;
  const int g0 = rank * a.g_per, g1 = min(a.groups, g0 + a.g_per);

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < SM::kAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_base_s)),
                 "r"((uint32_t)SM::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_base_s);
  pdl_launch_dependents();
  pdl_wait();  // codes and scales may be the kernel before's

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      for (int t = first; t < a.tiles; t += step) {
        const int r0 = (t % a.lane_tiles) * kLanes, c0 = (t / a.lane_tiles) * BN;
        for (int g = g0; g < g1; ++g) {
          uint8_t* st = smem + s * SM::kStage;
          if (!tc_wait(&empty[s], ph ^ 1u)) atomicOr(a.err, kErrTimeout);
          mbar_arrive_expect_tx(&full[s], (uint32_t)SM::kStage);
          tma_load_2d(st, &ta, g * kGroup, r0, &full[s]);
          tma_load_2d(st + SM::kA, &tb, g * kGroup, c0, &full[s]);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(BN);
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      for (int t = first; t < a.tiles; t += step) {
        for (int g = g0; g < g1; ++g) {
          if (!tc_wait(&acc_empty[acc], aph ^ 1u)) atomicOr(a.err, kErrTimeout);
          if (!tc_wait(&full[s], ph)) atomicOr(a.err, kErrTimeout);
          tc_fence_after();
          const uint8_t* st = smem + s * SM::kStage;
          const uint64_t da = sw128_desc(st), db = sw128_desc(st + SM::kA);
          const uint32_t d = tmem + (uint32_t)(acc * BN);
#pragma unroll
          for (int k = 0; k < kGroup / 32; ++k)  // 32 bytes along the swizzle atom
            mma_e4m3(d, da + (uint64_t)(2 * k), db + (uint64_t)(2 * k), idesc, k != 0);
          tc_commit(&empty[s]);
          tc_commit(&acc_full[acc]);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
          if (++acc == SM::kAcc) {
            acc = 0;
            aph ^= 1u;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int kHalf = BN / 2;                      // columns of this warp
    constexpr int kCh = kHalf < 32 ? kHalf : 32;       // columns per TMEM load
    constexpr int kNCh = kHalf / kCh;
    constexpr int kWs = WIDE ? (BN == 192 ? 3 : 1) : 1;  // weight scales of the warp's columns: 96 may straddle a block
    const int q = warp & 3, half = (warp - 2) / 4;
    const int l = 32 * q + lane;                       // this thread's TMEM lane
    const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * kHalf);
    int acc = 0;
    uint32_t aph = 0;
    for (int t = first; t < a.tiles; t += step) {
      const int r0 = (t % a.lane_tiles) * kLanes, c0 = (t / a.lane_tiles) * BN + half * kHalf;
      // this thread's share of a group's scales: its token's (wide: the lane's;
      // tall: column c0 + lane's) and the weight blocks'
      const int mtok = WIDE ? r0 + l : c0 + lane;
      const bool has_tok = WIDE ? mtok < a.M : (lane < kHalf && mtok < a.M);
      auto load_x = [&](int g) { return has_tok && g < g1 ? __ldg(a.xs + (size_t)g * a.M + mtok) : 0.f; };
      auto load_w = [&](int g, int j) {
        const int n = WIDE ? c0 + 32 * j : r0;
        return g < g1 && n < a.N ? __ldg(a.ws + (size_t)(n >> 7) * a.groups + g) : 0.f;
      };
      float x0 = load_x(g0), x1 = load_x(g0 + 1);
      float w0[kWs], w1[kWs];
#pragma unroll
      for (int j = 0; j < kWs; ++j) {
        w0[j] = load_w(g0, j);
        w1[j] = load_w(g0 + 1, j);
      }
      float2 sum[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) sum[i] = make_float2(0.f, 0.f);
      for (int g = g0; g < g1; ++g) {
        const float x2 = load_x(g + 2);
        float w2[kWs];
#pragma unroll
        for (int j = 0; j < kWs; ++j) w2[j] = load_w(g + 2, j);
        if (lane == 0 && !tc_wait(&acc_full[acc], aph)) atomicOr(a.err, kErrTimeout);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kNCh; ++c) {
          float v[kCh];
          tmem_ld<kCh>(tbase + (uint32_t)(acc * BN + c * kCh), v);
          if (c == kNCh - 1) {  // the accumulator is read: the MMA may fill it again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
          }
          if constexpr (WIDE) {
            const float f = x0 * w0[kWs > 1 ? c : 0];
#pragma unroll
            for (int i = 0; i < kCh / 2; ++i)
              sum[c * kCh / 2 + i] =
                  __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(f, f), sum[c * kCh / 2 + i]);
          } else {
            const float f = x0 * w0[0];
#pragma unroll
            for (int i = 0; i < kCh / 2; ++i) {
              const float2 s2 = make_float2(__shfl_sync(0xffffffffu, f, c * kCh + 2 * i),
                                            __shfl_sync(0xffffffffu, f, c * kCh + 2 * i + 1));
              sum[c * kCh / 2 + i] = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), s2, sum[c * kCh / 2 + i]);
            }
          }
        }
        x0 = x1;
        x1 = x2;
#pragma unroll
        for (int j = 0; j < kWs; ++j) {
          w0[j] = w1[j];
          w1[j] = w2[j];
        }
        if (++acc == SM::kAcc) {
          acc = 0;
          aph ^= 1u;
        }
      }
      if (a.csize > 1) {
        // every load of the ring has been consumed by a completed MMA
        float* part = reinterpret_cast<float*>(smem) + (size_t)(half * kHalf) * SM::kPartStride + l;
#pragma unroll
        for (int i = 0; i < kHalf / 2; ++i) {
          part[(2 * i) * SM::kPartStride] = sum[i].x;
          part[(2 * i + 1) * SM::kPartStride] = sum[i].y;
        }
      } else if constexpr (WIDE) {
        const int m = r0 + l;
        if (m < a.M) {
          if (a.vec && c0 + kHalf <= a.N) {
            if (a.out_f32) {
              float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + (size_t)m * a.N + c0);
              const float4* b = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.bias) + c0);
#pragma unroll
              for (int i = 0; i < kHalf / 4; ++i) {
                float4 y = make_float4(sum[2 * i].x, sum[2 * i].y, sum[2 * i + 1].x, sum[2 * i + 1].y);
                if (a.bias) {
                  const float4 bb = __ldg(b + i);
                  y = make_float4(y.x + bb.x, y.y + bb.y, y.z + bb.z, y.w + bb.w);
                }
                o[i] = y;
              }
            } else {
              uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.out) + (size_t)m * a.N + c0);
              const uint4* b = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(a.bias) + c0);
#pragma unroll
              for (int i = 0; i < kHalf / 8; ++i) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  y[2 * j] = sum[4 * i + j].x;
                  y[2 * j + 1] = sum[4 * i + j].y;
                }
                if (a.bias) {
                  float bb[8];
                  unpack16<bf16>(__ldg(b + i), bb);
#pragma unroll
                  for (int j = 0; j < 8; ++j) y[j] += bb[j];
                }
                o[i] = pack16<bf16>(y);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < kHalf / 2; ++i) {
              if (c0 + 2 * i < a.N) store_out(a, m, c0 + 2 * i, sum[i].x);
              if (c0 + 2 * i + 1 < a.N) store_out(a, m, c0 + 2 * i + 1, sum[i].y);
            }
          }
        }
      } else {
        const int n = r0 + l;
        if (n < a.N) {
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) {
            if (c0 + 2 * i < a.M) store_out(a, c0 + 2 * i, n, sum[i].x);
            if (c0 + 2 * i + 1 < a.M) store_out(a, c0 + 2 * i + 1, n, sum[i].y);
          }
        }
      }
    }
  }

  if (a.csize > 1) {
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    __syncwarp();
    cl.sync();  // the partial tiles are written
    const int t = first;
    const int r0 = (t % a.lane_tiles) * kLanes, c0 = (t / a.lane_tiles) * BN;
    const float* part = reinterpret_cast<const float*>(smem);
    const float* peer[kClusterMax];
#pragma unroll
    for (int r = 0; r < kClusterMax; ++r)
      peer[r] = r < a.csize ? cl.map_shared_rank(part, r) : part;
    // wide: this CTA takes the token rows l % csize == rank, threads along the
    // features; tall: the token columns c % csize == rank, threads along the
    // features again (the lanes): either way a warp stores a row's neighbours
    constexpr int kAlong = WIDE ? BN : kLanes, kOther = WIDE ? kLanes : BN;
    for (int i = threadIdx.x; i < (kOther - rank + a.csize - 1) / a.csize * kAlong; i += kThreads) {
      const int f = i % kAlong, o = i / kAlong * a.csize + rank;
      const int m = (WIDE ? r0 : c0) + o, n = (WIDE ? c0 : r0) + f;
      if (m >= a.M || n >= a.N) continue;
      const size_t at = WIDE ? (size_t)f * SM::kPartStride + o : (size_t)o * SM::kPartStride + f;
      float y = 0.f;
#pragma unroll
      for (int r = 0; r < kClusterMax; ++r)
        if (r < a.csize) y += peer[r][at];
      store_out(a, m, n, y);
    }
    cl.sync();  // no CTA leaves while another reads its tile
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)SM::kCols)
                 : "memory");
  }
}

template <bool WIDE, int BN, int STAGES>
q2_status launch_q8(const void* xq, const void* wq, int K, Q8Lin a, cudaStream_t st) {
  using SM = Q8Smem<BN, STAGES>;
  auto* kernel = q8_linear_kernel<WIDE, BN, STAGES>;
  Q2_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SM::kTotal));
  a.lane_tiles = ((WIDE ? a.M : a.N) + kLanes - 1) / kLanes;
  const long long tiles = (long long)a.lane_tiles * (((WIDE ? a.N : a.M) + BN - 1) / BN);
  if (tiles >= (1ll << 30)) {
    set_error("linear_q8: too many tiles");
    return Q2_ERR_SHAPE;
  }
  a.tiles = (int)tiles;
  const int sms = num_sms();
  // CTAs per tile: as many as leave no SM without work, each with a group
  int cs = tiles < sms ? (int)(sms / tiles) : 1;
  cs = cs > kClusterMax ? kClusterMax : cs;
  cs = cs > a.groups ? a.groups : cs;
  a.g_per = (a.groups + cs - 1) / cs;
  a.csize = (a.groups + a.g_per - 1) / a.g_per;  // every CTA has a group
  CUtensorMap tx, tw;
  Q2_TRY(make_tmap_2d_u8(&tx, xq, (uint64_t)a.M, (uint64_t)K, (uint64_t)K, WIDE ? kLanes : BN, kGroup, 128));
  Q2_TRY(make_tmap_2d_u8(&tw, wq, (uint64_t)a.N, (uint64_t)K, (uint64_t)K, WIDE ? BN : kLanes, kGroup, 128));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.csize > 1 ? tiles * a.csize : tiles < sms ? tiles : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = SM::kTotal;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.csize;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  Q2_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, WIDE ? tx : tw, WIDE ? tw : tx, a));
  return Q2_OK;
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
  int* flag = op_error_flag();
  Q2_CHECK_ARG(flag, Q2_ERR_CUDA, "cannot resolve the device error flag");
  const size_t es = dtype == Q2_BF16 ? 2 : 4;
  Q8Lin a = {};
  a.xs = xs;
  a.ws = ws;
  a.bias = bias;
  a.out = out;
  a.M = (int)M;
  a.N = (int)N;
  a.groups = (int)((K + kGroup - 1) / kGroup);
  a.out_f32 = dtype == Q2_F32;
  a.vec = ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(bias) | (N * es)) & 15) == 0;
  a.err = flag;
  cudaStream_t st = as_stream(stream);
  if (M <= 16) return launch_q8<false, 16, 11>(xq, wq, (int)K, a, st);
  if (M <= 32) return launch_q8<false, 32, 10>(xq, wq, (int)K, a, st);
  if (M <= 64) return launch_q8<false, 64, 8>(xq, wq, (int)K, a, st);
  const int sms = num_sms();
  const long long lt = (a.M + kLanes - 1) / kLanes;
  auto cost = [&](int bn) { return (lt * ((a.N + bn - 1) / bn) + sms - 1) / sms * bn; };
  if (lt * ((a.N + 255) / 256) < sms) return launch_q8<true, 128, 6>(xq, wq, (int)K, a, st);
  if (10 * cost(192) <= 9 * cost(256)) return launch_q8<true, 192, 5>(xq, wq, (int)K, a, st);
  return launch_q8<true, 256, 4>(xq, wq, (int)K, a, st);
}
