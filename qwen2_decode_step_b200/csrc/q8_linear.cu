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
// Warp roles (384 threads, one CTA per SM, persistent over the tiles): warp 0
// TMA (a 128 x 128-byte and a BN x 128-byte box per group, 128-byte swizzle, a
// ring of STAGES), warp 1 tensor memory and MMA, warps 4-11 epilogue: two per
// TMEM lane quarter, each half of the columns.  The first four warps give most
// of their registers to the epilogue's: a wide thread keeps 128 sums and takes
// 64 products of a group per TMEM load (32 at a time left the loads' latency
// bare: 1470 cycles per group instead of the MMA's 512).
// When the tiles alone leave SMs idle, a cluster of up to 8 CTAs splits the
// groups of one tile: each leaves its fp32 partial tile in its shared memory
// and every CTA adds one share of it over the cluster in rank order
// (distributed shared memory; no workspace, no second launch, the same sum
// every time).
// Every wait is bounded: one that runs out sets value 2 in the device error
// word and the kernel carries on to its end.
#include <cooperative_groups.h>

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
constexpr int kEpiWarp0 = 4;                // warps 2 and 3 only fill their warpgroup
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
// registers: launched with 168 a thread (64512 / 384); the first warpgroup
// drops to 40, the two of the epilogue rise to 232: 128 * 40 + 256 * 232 = 64512
constexpr int kRegsLow = 40, kRegsHigh = 232;
constexpr int kClusterMax = 8;

struct Q8Lin {
  const float* xs;    // [groups][M]
  const float* ws;    // [ceil(N / 128)][groups]
  const void* bias;   // [N] or null
  void* out;          // [M][N]
  int M, N, groups;
  int lane_tiles, tiles;  // of the lane-side operand; of the output
  int csize;          // CTAs that share a tile
  int g_per;          // groups per CTA of a cluster
  int tma_out;        // wide: the output's tensor map is valid
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

// NC consecutive columns (8, 16 or 32) of this thread's TMEM lane, as bits; the
// values may be used after tmem_wait.
template <int NC>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  if constexpr (NC == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  } else if constexpr (NC == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr));
  }
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// The factor of a group's sum: the product of its two scales, held to fp32's
// largest value (an infinity would make NaN of a sum of 0; NaN stays).  Taking the
// two apart where their product leaves the normal range would bring results of
// sums below 1 back that this loses; any test for it in the loop cost wide tiles
// more than it is worth (a vote at each load 4096 x 17920 x 1536 141 -> 161 us, one
// a group 230).
__device__ __forceinline__ float scale_product(float x, float w) {
  float f;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(f) : "f"(x * w), "f"(3.402823466e38f));
  return f;
}

template <bool WIDE, int BN, int STAGES>
struct Q8Smem {
  static constexpr size_t kA = (size_t)kLanes * kGroup;
  static constexpr size_t kB = (size_t)BN * kGroup;
  static constexpr size_t kStage = kA + kB;
  // accumulators in tensor memory: as many as fit 512 columns, at most four
  static constexpr int kAcc = BN > 128 ? 2 : 4;
  static constexpr int kCols = kAcc * BN <= 64 ? 64 : kAcc * BN <= 128 ? 128 : kAcc * BN <= 256 ? 256 : 512;
  static constexpr size_t kBars = (2 * STAGES + 2 * kAcc) * 8 + 16;
  // wide: 32 rows x 128 bytes of output per epilogue warp, to turn them
  static constexpr size_t kTurn = STAGES * kStage;
  static constexpr size_t kBarOff = kTurn + (WIDE ? kEpiWarps * 4096 : 0);
  static constexpr size_t kTotal = kBarOff + kBars + 1024;  // + alignment slack
  // a cluster's partial tile, features contiguous (distributed shared memory
  // moves neighbouring words together): wide [token lane][BN], rows 16 bytes
  // longer against bank conflicts of the writes; tall [token column][lane]
  static_assert(kTotal <= 232448, "shared memory of one CTA");
  static constexpr int kPartStride = WIDE ? BN + 4 : kLanes;
  static constexpr bool kFits = (size_t)(WIDE ? kLanes : BN) * kPartStride * 4 <= STAGES * kStage;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T>
__device__ __forceinline__ void store_out(const Q8Lin& a, int m, int n, float y) {
  if (a.bias) y += to_f(reinterpret_cast<const T*>(a.bias)[n]);
  reinterpret_cast<T*>(a.out)[(size_t)m * a.N + n] = from_f<T>(y);
}

// A CTA's tiles in order (first, first + step, ...): lane-side tile lt fastest.
struct TileWalk {
  int t, lt, ct, step, dl, dc, lane_tiles;
  __device__ __forceinline__ TileWalk(int first, int step_, int lane_tiles_)
      : t(first), lt(first % lane_tiles_), ct(first / lane_tiles_), step(step_), dl(step_ % lane_tiles_),
        dc(step_ / lane_tiles_), lane_tiles(lane_tiles_) {}
  __device__ __forceinline__ void next() {
    t += step;
    lt += dl;
    ct += dc;
    if (lt >= lane_tiles) {
      lt -= lane_tiles;
      ++ct;
    }
  }
};

// ta: the lane-side operand's map, tb: the column-side one's, to: the output's
// (wide, boxes of 32 tokens x 128 bytes).
template <typename T, bool WIDE, int BN, int STAGES>
__global__ void __launch_bounds__(kThreads, 1)
    q8_linear_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                     const __grid_constant__ CUtensorMap to, const Q8Lin a) {
  using SM = Q8Smem<WIDE, BN, STAGES>;
  static_assert(SM::kFits && SM::kAcc * BN <= 512, "the partial tile fits the ring, the accumulators tensor memory");
  extern __shared__ __align__(1024) uint8_t q8_smem_raw[];
  uint8_t* smem = q8_smem_raw + ((1024u - (smem_u32(q8_smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBarOff);
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

  // (setmaxnreg inside each branch: the compiler allots a joint path the lower
  // count)
  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        int s = 0;
        uint32_t ph = 0;
        for (TileWalk w(first, step, a.lane_tiles); w.t < a.tiles; w.next()) {
          const int r0 = w.lt * kLanes, c0 = w.ct * BN;
          for (int g = g0; g < g1; ++g) {
            uint8_t* st = smem + s * SM::kStage;
            if (!tc_wait_asleep(&empty[s], ph ^ 1u)) atomicOr(a.err, kErrTimeout);
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
      // The whole warp walks the loop and one elected lane issues, so that the
      // descriptors stay in uniform registers (from one lane's own registers a
      // group's six instructions took 400 cycles to issue).  It polls: asleep it
      // woke so late that 61 tokens x 151936 features took 65 us, not 46.
      constexpr uint32_t idesc = idesc_e4m3(BN);
      const uint64_t da0 = sw128_desc(smem), db0 = sw128_desc(smem + SM::kA);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      for (int t = first; t < a.tiles; t += step) {
        for (int g = g0; g < g1; ++g) {
          if (!tc_wait_poll(&acc_empty[acc], aph ^ 1u) && lane == 0) atomicOr(a.err, kErrTimeout);
          if (!tc_wait_poll(&full[s], ph) && lane == 0) atomicOr(a.err, kErrTimeout);
          tc_fence_after();
          if (elect_one()) {
            const uint64_t at = (uint64_t)((uint32_t)s * (uint32_t)(SM::kStage >> 4));
            const uint32_t d = tm + (uint32_t)(acc * BN);
#pragma unroll
            for (int k = 0; k < kGroup / 32; ++k)  // 32 bytes along the swizzle atom
              mma_e4m3(d, da0 + at + (uint64_t)(2 * k), db0 + at + (uint64_t)(2 * k), idesc, k != 0);
            tc_commit(&empty[s]);
            tc_commit(&acc_full[acc]);
          }
          __syncwarp();
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
    if (a.csize > 1) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    // ------------------------------------------------------------ epilogue
    constexpr int kHalf = BN / 2;                      // columns of this warp
    constexpr int kCh = kHalf < 32 ? kHalf : 32;       // columns per TMEM load
    constexpr int kNCh = kHalf / kCh;
    constexpr int kTwo = kNCh > 1 ? 2 : 1;             // TMEM loads in flight
    constexpr int kWs = WIDE && BN == 192 ? 3 : 1;     // weight scales of the warp's columns: 96 may straddle a block
    constexpr int kV = Storage<T>::kVec;
    // Weight scales: of 256 columns by lane (32 groups' lie next to each other, a
    // lane reads one and hands it to the others at its group), and the loop in steps
    // of one group; 4096 x 17920 x 1536 131 -> 118 us (short runs; 139 in steady
    // calls, under the power limit), x 4096 308 -> 292.  Of fewer
    // columns by every lane at each group, in steps of two: by lane 192 columns
    // took 74-80 us instead of 65-72 (4096 x 1536 x 8960), 128 columns 32 instead
    // of 30 (1000 x 4096 x 4096 fp32), 64 tokens the same.
    constexpr bool kShare = WIDE && BN == 256;
    constexpr int kAhead = kShare ? 1 : 2;             // groups of a step; the next step's scales are read ahead
    const int q = warp & 3, half = (warp - kEpiWarp0) / 4;
    const int l = 32 * q + lane;                       // this thread's TMEM lane
    const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * kHalf);
    int acc = 0;
    uint32_t aph = 0;
    // A thread's share of a group's scales: its token's (wide: the lane's; tall:
    // column lane's) and the weight blocks'.  kAhead groups are read while the
    // kAhead before are used, the next tile's first ones before this tile is
    // stored.  Rows and groups outside are held to the last one (their products
    // are not stored or not formed), so that the loads need no predicate.
    float xs[kAhead], ws[kAhead][kWs];
    [[maybe_unused]] float wl = 0.f, wl_next = 0.f;  // kShare: of this lane's group of 32, of the next 32
    const float* xp;
    const float* wp[kWs];
    auto seek = [&](const TileWalk& w) {
      const int m = WIDE ? w.lt * kLanes + l : w.ct * BN + half * kHalf + (lane < kHalf ? lane : 0);
      xp = a.xs + min(m, a.M - 1);
#pragma unroll
      for (int j = 0; j < kWs; ++j) {
        const int n = WIDE ? w.ct * BN + half * kHalf + 32 * j : w.lt * kLanes;
        wp[j] = a.ws + (size_t)(min(n, a.N - 1) >> 7) * a.groups;
      }
    };
    auto load_scales = [&](float* x, float (*w)[kWs], int g) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int at = min(g + u, g1 - 1);
        x[u] = __ldg(xp + (size_t)at * a.M);
#pragma unroll
        for (int j = 0; j < kWs; ++j) w[u][j] = kShare ? 0.f : __ldg(wp[j] + at);
      }
    };
    auto load_lanes = [&](int g) { return __ldg(wp[0] + min(g + lane, g1 - 1)); };
    TileWalk w(first, step, a.lane_tiles);
    if (w.t < a.tiles) {
      seek(w);
      load_scales(xs, ws, g0);
      if constexpr (kShare) wl = load_lanes(g0);
    }
    while (w.t < a.tiles) {
      const int r0 = w.lt * kLanes, c0 = w.ct * BN + half * kHalf;
      float2 sum[kHalf / 2];
      // wide, 16-byte output rows: the sums begin at the bias (added at the end,
      // its loads lay bare in the store: 20 of 151 us)
      const bool bias_in = WIDE && a.tma_out && a.bias;
#pragma unroll
      for (int i = 0; i < kHalf / kV; ++i) {
        float y[kV];
        if (bias_in && c0 + i * kV < a.N) {
          unpack16<T>(__ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.bias) + c0) + i), y);
        } else {
#pragma unroll
          for (int j = 0; j < kV; ++j) y[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kV / 2; ++j) sum[i * kV / 2 + j] = make_float2(y[2 * j], y[2 * j + 1]);
      }
      for (int gg = g0; gg < g1; gg += kAhead) {
        float xn[kAhead], wn[kAhead][kWs];
        load_scales(xn, wn, gg + kAhead);
        if constexpr (kShare)
          if (((gg - g0) & 31) == 0 && gg + 32 < g1) wl_next = load_lanes(gg + 32);
#pragma unroll
        for (int ahead = 0; ahead < kAhead; ++ahead) {
          if (gg + ahead >= g1) break;
          if (!tc_wait_asleep(&acc_full[acc], aph) && lane == 0) atomicOr(a.err, kErrTimeout);
          __syncwarp();  // (each lane waited for itself: the loads below take whole warps)
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kNCh; c += kTwo) {
            uint32_t v[kTwo][kCh];
#pragma unroll
            for (int u = 0; u < kTwo; ++u)
              if (c + u < kNCh) tmem_ld<kCh>(tbase + (uint32_t)(acc * BN + (c + u) * kCh), v[u]);
            tmem_wait();
            if (c + kTwo >= kNCh) {  // the accumulator is read: the MMA may fill it again
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&acc_empty[acc]);
            }
#pragma unroll
            for (int u = 0; u < kTwo; ++u) {
              if (c + u >= kNCh) continue;
              const float f = scale_product(xs[ahead], kShare ? __shfl_sync(0xffffffffu, wl, (gg - g0) & 31)
                                                              : ws[ahead][kWs > 1 ? c + u : 0]);
#pragma unroll
              for (int i = 0; i < kCh / 2; ++i) {
                const int at = (c + u) * kCh / 2 + i;
                const float2 s2 = WIDE ? make_float2(f, f)
                                       : make_float2(__shfl_sync(0xffffffffu, f, (c + u) * kCh + 2 * i),
                                                     __shfl_sync(0xffffffffu, f, (c + u) * kCh + 2 * i + 1));
                sum[at] = __ffma2_rn(make_float2(__uint_as_float(v[u][2 * i]), __uint_as_float(v[u][2 * i + 1])),
                                     s2, sum[at]);
              }
            }
          }
          if (++acc == SM::kAcc) {
            acc = 0;
            aph ^= 1u;
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          xs[u] = xn[u];
#pragma unroll
          for (int j = 0; j < kWs; ++j) ws[u][j] = wn[u][j];
        }
        if constexpr (kShare)
          if (((gg + 1 - g0) & 31) == 0) wl = wl_next;
      }
      w.next();
      if (w.t < a.tiles) {
        seek(w);
        load_scales(xs, ws, g0);
        if constexpr (kShare) wl = load_lanes(g0);
      }
      if (a.csize > 1) {
        // every load of the ring has been consumed by a completed MMA
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < kHalf / 2; ++i) {
          if constexpr (WIDE) {
            if (i % 2 == 0)
              *reinterpret_cast<float4*>(part + (size_t)l * SM::kPartStride + half * kHalf + 2 * i) =
                  make_float4(sum[i].x, sum[i].y, sum[i + 1].x, sum[i + 1].y);
          } else {
            part[(half * kHalf + 2 * i) * SM::kPartStride + l] = sum[i].x;
            part[(half * kHalf + 2 * i + 1) * SM::kPartStride + l] = sum[i].y;
          }
        }
      } else if constexpr (WIDE) {
        if (a.tma_out) {
          // 32 tokens x 128 bytes at a time go to shared memory (16-byte chunk j
          // of row r at j ^ (r % 8), the tensor map's swizzle: no bank conflicts)
          // and leave by TMA, which also drops what lies outside the output.
          // (Stored by the threads, a row per lane, a tile's 64 KB took 13000
          // cycles against its 12 groups' 6100.)
          constexpr int kPer = 128 / (int)sizeof(T);     // columns of a part
          uint8_t* turn = smem + SM::kTurn + (size_t)(warp - kEpiWarp0) * 4096;
#pragma unroll
          for (int p = 0; p < (kHalf + kPer - 1) / kPer; ++p) {
            if (lane == 0) bulk_wait_read();  // the part before has left
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (p * kPer + j * kV >= kHalf) continue;
              float y[kV];
#pragma unroll
              for (int e = 0; e < kV / 2; ++e) {
                y[2 * e] = sum[(p * kPer + j * kV) / 2 + e].x;
                y[2 * e + 1] = sum[(p * kPer + j * kV) / 2 + e].y;
              }
              *reinterpret_cast<uint4*>(turn + lane * 128 + ((j ^ (lane & 7)) << 4)) = pack16<T>(y);
            }
            fence_async_smem();
            __syncwarp();
            // (a half part, 96 bf16 columns' last, ends inside its 64-column box:
            // its stale second half would land on the next warp's columns)
            const bool whole = (p + 1) * kPer <= kHalf;
            if (whole) {
              if (lane == 0 && c0 + p * kPer < a.N && r0 + 32 * q < a.M) {
                tma_store_2d(&to, c0 + p * kPer, r0 + 32 * q, turn);
                bulk_commit();
              }
            } else {
              const int r = lane, m = r0 + 32 * q + r;
              if (m < a.M)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int n = c0 + p * kPer + j * kV;
                  if (n < a.N)
                    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + (size_t)m * a.N + n) =
                        *reinterpret_cast<const uint4*>(turn + r * 128 + ((j ^ (r & 7)) << 4));
                }
            }
          }
        } else {
          // rows that do not start on 16 bytes: 32 x 32 values at a time are turned
          // (value c of row r at (c + r) % 32: no bank conflicts), a warp stores 32
          // neighbours of a row (a row per lane stored 32 lines at a time: 2416 x
          // 7093 x 1104 205 us instead of 42.6)
          float* turn = reinterpret_cast<float*>(smem + SM::kTurn + (size_t)(warp - kEpiWarp0) * 4096);
          const int m0 = r0 + 32 * q;
#pragma unroll
          for (int p = 0; p < kHalf / 32; ++p) {
            const int n = c0 + 32 * p + lane;
            const float b = a.bias && n < a.N ? to_f(reinterpret_cast<const T*>(a.bias)[n]) : 0.f;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              turn[lane * 32 + ((c + lane) & 31)] = c % 2 ? sum[16 * p + c / 2].y : sum[16 * p + c / 2].x;
            __syncwarp();
            if (n < a.N) {
              T* o = reinterpret_cast<T*>(a.out) + (size_t)m0 * a.N + n;
              const int rows = min(32, a.M - m0);
              for (int r = 0; r < rows; ++r, o += a.N) *o = from_f<T>(turn[r * 32 + ((lane + r) & 31)] + b);
            }
            __syncwarp();
          }
        }
      } else {
        const int n = r0 + l, left = a.M - c0;
        if (n < a.N) {
          const float b = a.bias ? to_f(reinterpret_cast<const T*>(a.bias)[n]) : 0.f;
          T* o = reinterpret_cast<T*>(a.out) + (size_t)c0 * a.N + n;
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) {
            if (2 * i < left) o[0] = from_f<T>(sum[i].x + b);
            if (2 * i + 1 < left) o[a.N] = from_f<T>(sum[i].y + b);
            o += 2 * (size_t)a.N;
          }
        }
      }
    }
    if (WIDE && lane == 0) bulk_wait_all();
    if (a.csize > 1) {
      namespace cg = cooperative_groups;
      cg::cluster_group cl = cg::this_cluster();
      __syncwarp();
      cluster_sync();  // the partial tiles are written
      const int t = first;
      const int r0 = (t % a.lane_tiles) * kLanes, c0 = (t / a.lane_tiles) * BN;
      const float* part = reinterpret_cast<const float*>(smem);
      // this CTA adds the tokens o % csize == rank, four features per thread
      constexpr int kFeat = WIDE ? BN : kLanes, kTok = WIDE ? kLanes : BN;
      for (int i = threadIdx.x - kEpiWarp0 * 32; i < (kTok - rank + a.csize - 1) / a.csize * (kFeat / 4); i += kEpiWarps * 32) {
        const int f = i % (kFeat / 4) * 4, o = i / (kFeat / 4) * a.csize + rank;
        const int m = (WIDE ? r0 : c0) + o, n = (WIDE ? c0 : r0) + f;
        if (m >= a.M || n >= a.N) continue;
        float4 v[kClusterMax];
#pragma unroll
        for (int r = 0; r < kClusterMax; ++r)
          if (r < a.csize)
            v[r] = *reinterpret_cast<const float4*>(cl.map_shared_rank(part, r) + (size_t)o * SM::kPartStride + f);
        float4 y = v[0];
#pragma unroll
        for (int r = 1; r < kClusterMax; ++r)
          if (r < a.csize) y = make_float4(y.x + v[r].x, y.y + v[r].y, y.z + v[r].z, y.w + v[r].w);
        store_out<T>(a, m, n, y.x);
        if (n + 1 < a.N) store_out<T>(a, m, n + 1, y.y);
        if (n + 2 < a.N) store_out<T>(a, m, n + 2, y.z);
        if (n + 3 < a.N) store_out<T>(a, m, n + 3, y.w);
      }
      __syncwarp();    // (lanes skip what lies outside the output: the barrier takes whole warps)
      cluster_sync();  // no CTA leaves while another reads its tile
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)SM::kCols)
                 : "memory");
  }
}

// How many clusters of cs CTAs of `kernel` the current device runs at once; asked
// once per device and size and kept in `known` (+ 1; 0: not asked yet).
constexpr int kDevs = 64;
using Known = std::atomic<int>[kDevs][kClusterMax + 1];
q2_status active_clusters(const void* kernel, int cs, size_t smem, Known& known, int* n) {
  int dev = 0;
  Q2_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < kDevs)
    if (const int k = known[dev][cs].load(std::memory_order_relaxed)) {
      *n = k - 1;
      return Q2_OK;
    }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  Q2_CUDA_TRY(cudaOccupancyMaxActiveClusters(n, kernel, &cfg));
  if (dev < kDevs) known[dev][cs].store(*n + 1, std::memory_order_relaxed);
  return Q2_OK;
}

template <typename T, bool WIDE, int BN, int STAGES>
q2_status launch_q8(const void* xq, const void* wq, int K, Q8Lin a, cudaStream_t st) {
  using SM = Q8Smem<WIDE, BN, STAGES>;
  auto* kernel = q8_linear_kernel<T, WIDE, BN, STAGES>;
  static std::atomic<uint64_t> done{0};
  static Known known;  // (zero)
  if (first_on_device(done)) {
    Q2_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SM::kTotal));
    // the register split draws on what the kernel is launched with: fewer would
    // leave setmaxnreg.inc waiting
    cudaFuncAttributes fa;
    Q2_CUDA_TRY(cudaFuncGetAttributes(&fa, kernel));
    if (fa.numRegs * kThreads < kRegsLow * kEpiWarp0 * 32 + kRegsHigh * kEpiWarps * 32) {
      set_error("linear_q8: the kernel was built with too few registers for its split");
      return Q2_ERR_CUDA;
    }
    done_on_device(done);
  }
  a.lane_tiles = ((WIDE ? a.M : a.N) + kLanes - 1) / kLanes;
  const long long tiles = (long long)a.lane_tiles * (((WIDE ? a.N : a.M) + BN - 1) / BN);
  if (tiles >= (1ll << 30)) {
    set_error("linear_q8: too many tiles");
    return Q2_ERR_SHAPE;
  }
  a.tiles = (int)tiles;
  // CTAs per tile.  Time in groups: a wave of tiles takes its groups and about
  // kFixed more (start, last store); joining a split tile about kJoin.  Clusters
  // pack badly (3 CTAs each: 48 clusters of 144 CTAs did not fit 148 SMs at once
  // and 512 x 1536 x 8960 took two waves, 26 us), so the driver is asked how many
  // are resident together.
  constexpr int kFixed = 4, kJoin = 3;
  const int sms = num_sms();
  int best = 1;
  long long best_cost = (tiles + sms - 1) / sms * (a.groups + kFixed);
  for (int cs = 2; cs <= kClusterMax && cs <= a.groups && tiles * cs <= sms; ++cs) {
    int active = 0;
    Q2_TRY(active_clusters(reinterpret_cast<const void*>(kernel), cs, SM::kTotal, known, &active));
    if (active < 1) continue;
    const long long cost = (tiles + active - 1) / active * ((a.groups + cs - 1) / cs + kFixed) + kJoin;
    if (cost < best_cost) {
      best_cost = cost;
      best = cs;
    }
  }
  a.g_per = (a.groups + best - 1) / best;
  a.csize = (a.groups + a.g_per - 1) / a.g_per;  // every CTA has a group
  CUtensorMap tx, tw;
  Q2_TRY(make_tmap_2d_u8(&tx, xq, (uint64_t)a.M, (uint64_t)K, (uint64_t)K, WIDE ? kLanes : BN, kGroup, 128));
  Q2_TRY(make_tmap_2d_u8(&tw, wq, (uint64_t)a.N, (uint64_t)K, (uint64_t)K, WIDE ? BN : kLanes, kGroup, 128));
  // the output by TMA where its rows start on 16 bytes
  CUtensorMap to = {};
  a.tma_out = WIDE && a.csize == 1 &&
              ((reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.bias) | (a.N * sizeof(T))) & 15) == 0;
  if (a.tma_out) {
    const uint64_t pitch = (uint64_t)a.N * sizeof(T);
    if (sizeof(T) == 2)
      Q2_TRY(make_tmap_2d_bf16(&to, a.out, (uint64_t)a.M, (uint64_t)a.N, pitch, 32, 64, 128));
    else
      Q2_TRY(make_tmap_2d_f32(&to, a.out, (uint64_t)a.M, (uint64_t)a.N, pitch, 32, 32, 128));
  }
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
  Q2_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, WIDE ? tx : tw, WIDE ? tw : tx, to, a));
  return Q2_OK;
}

template <typename T>
q2_status linear_t(const void* xq, const void* wq, int K, const Q8Lin& a, cudaStream_t st) {
  if (a.M <= 16) return launch_q8<T, false, 16, 11>(xq, wq, K, a, st);
  if (a.M <= 32) return launch_q8<T, false, 32, 10>(xq, wq, K, a, st);
  if (a.M <= 64) return launch_q8<T, false, 64, 8>(xq, wq, K, a, st);
  const int sms = num_sms();
  const long long lt = (a.M + kLanes - 1) / kLanes;
  auto cost = [&](int bn) { return (lt * ((a.N + bn - 1) / bn) + sms - 1) / sms * bn; };
  if (lt * ((a.N + 255) / 256) < sms) return launch_q8<T, true, 128, 6>(xq, wq, K, a, st);
  if (10 * cost(192) <= 9 * cost(256)) return launch_q8<T, true, 192, 4>(xq, wq, K, a, st);
  return launch_q8<T, true, 256, 4>(xq, wq, K, a, st);
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
  Q8Lin a = {};
  a.xs = xs;
  a.ws = ws;
  a.bias = bias;
  a.out = out;
  a.M = (int)M;
  a.N = (int)N;
  a.groups = (int)((K + kGroup - 1) / kGroup);
  a.err = flag;
  cudaStream_t st = as_stream(stream);
  return dtype == Q2_BF16 ? linear_t<bf16>(xq, wq, (int)K, a, st) : linear_t<float>(xq, wq, (int)K, a, st);
}
