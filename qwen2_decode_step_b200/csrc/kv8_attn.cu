// kv8_attn.cu -- attention over the 8-bit KV cache.
//
// Split kernel (any head dim, fp32 or bf16, one to many query rows).  Keys go on
// the M side of mma.sync m16n8k16 for the scores and head dims for the output,
// the query rows of a kv head (ntok rows x nh / nkv heads) on N, eight a tile:
// S^T = K q^T, O^T = V^T P^T.  A decode step's at most eight rows fill one
// tile; with the rows on M half of every MMA and of the accumulators stood
// empty.  A warp takes NT row tiles (one, two from nine rows on, in bf16 four from
// 65 on), up to four warps the rows of a work item (sequence, row group, kv head);
// its unit of work is 32 keys, half a block.  All items' units, in order, are dealt
// to a grid of resident CTAs in equal runs (lengths are read on the device), so
// ragged batches and a single long sequence load every SM alike; an item cut by a
// run's end leaves partial results that a second kernel joins in order (the same
// result every time).  Short items, and items in plenty, go to a CTA each instead:
// one launch, nothing to join (split_plan).
//
// Bound by HBM (a byte per cached element): a unit's K and V rows arrive by TMA
// (swizzled to the head's row length) in slots of their own for each group of
// warps that shares units, which fill them themselves.  e4m3 values are exact in
// fp16 and Blackwell converts two per instruction, so the products run in fp16
// with fp32 accumulation:
//   scores  a lane's 32 contiguous bytes of a key row (16-byte loads, no bank
//           conflicts under the swizzle) feed eight MMAs: the order of the dims
//           inside a dot product is free, the query's fragments take the same;
//   output  ldmatrix.trans on byte pairs gives a lane two keys x two dims; one
//           byte permute splits them into rows g (even dims) and g + 8 (odd) of
//           the A operand.  P turns from the scores' layout by movmatrix.
// The query rows are scaled by a power of two so that their largest element lies in
// [256, 512): a bf16 element is then exact in fp16 from 2^-25 of the largest on and
// within 2^-33 of the largest below that; an fp32 element is a high and a low fp16
// part (two MMAs) to 2^-22 of itself, and so is an fp32 row's probability (see kLow).
// Softmax in fp32, online, with p = 2^(s - m + 6), m the row's reference: the
// largest score when it was last taken.  It is taken again (shuffles over the eight
// lanes that hold a row's keys, the output rescaled) only when a score passes it by
// 8, so that most units need one vote; the common factor cancels.  p stays below
// 2^14.  A bf16 row's p is one fp16, as the output keeps 8 bits and its sums average
// the roundings: 11 bits down to 2^-20 of the largest, then to within 2^-31 of it (a
// second part would double the output's MMAs; over the decode batch the error
// against 64 bits is 0.0017, as a plain fp32 computation's: the output's rounding).
// The scale of K multiplies
// the scores; the output is accumulated in units of the current block's V scale and
// moved to the next block's where that differs (a power of two: exact).
//
// Prompt rows (bf16, head dim 128, 512 rows of a kv head or more): the cache's K and
// V are read back to bf16 (exact) in the workspace and the prompt attention on
// tcgen05 runs over them.  That product is bound by the tensor core: the copy
// moves 6 bytes per cached element once, against 4 rows x heads operations per
// element (4096 rows over 32768 keys, 12 / 2 heads: 1003 us in steady calls, 771
// TFLOP/s, 11 of them the copy).  A NaN of V, which the zero probabilities of rows
// that do not see it would spread, is taken out of the copy and put into the rows
// that do see it at the end.
#include "common.cuh"
#include "e4m3.cuh"
#include "kernels.h"
#include "kv8.h"
#include "tcgen05.cuh"
#include "tma.h"

namespace q2 {

namespace {

constexpr int kBlk = Q2_KV8_BLOCK;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKeys = 32;                       // keys per unit
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasMax = 512;
constexpr float kPBias = 6.f, kGrow = 8.f;      // p <= 2^(6 + 8) in fp16, see softmax
// References above this (in powers of two) may lie a sixteenth and more off their
// own exact product: from here on every score is rounded before the reference is taken
// from it, so that the difference is exact and the bound on p holds (below it one
// rounding of the difference, small where p is large).
constexpr float kCoarse = 0x1p20f;
// A part's sum is up to 2^14 for each of its keys: times this (it cancels) its
// product with outputs near fp32's largest value stays in range in the join.
constexpr float kPartScale = 0x1p-44f;
// fp32: the low fp16 part of a query element or probability is kept times kLow, in
// sums of its own, so that fp16's smallest step, 2^-24, costs 2^-37 and not 2^-25
// (a key holding nearly all weight over 32767 others of 2^-31 each: they were lost
// from the products and stayed in the sum).  The high part's error is at most 2^2
// (p below 2^14), times kLow 2^14.
constexpr float kLow = 0x1p12f;

struct Kv8Attn {
  const void* q;
  long long q_seq_stride, q_tok_stride;
  const float* ks;
  const float* vs;
  const int32_t* lens;  // [batch] keys of each sequence; null: fixed_len
  int fixed_len;
  int batch, ntok, nh, nkv, max_seq, nblk;
  int group;      // nh / nkv
  unsigned magic; // ceil(2^32 / group): r / group = umulhi(r, magic) for group > 1
  int nt;       // 8-row tiles of a warp: 1, 2 or 4
  int nm;       // warps that share an item's rows: 1, 2 or 4
  int irows;    // rows of an item: 8 nt nm
  int mgroups;  // items of a (sequence, kv head)
  float scale;
  void* out;    // [batch][ntok][nh][hd]
  float* part;  // [2 * CTAs][irows][hd + 2]: rows of partial items, then m and l 2^-44 of each row
  int4* cut;    // [items]: how the runs cut each item
  int ctas;     // of the split kernel
  int whole;    // a CTA per item, nothing is cut (see split_plan)
  int* err;
};

// --------------------------------------------------------------- work division

__device__ __forceinline__ int seq_len(const Kv8Attn& a, int b) {
  const int n = a.lens ? a.lens[b] : a.fixed_len;
  if (n > a.max_seq) atomicOr(a.err, kErrCapacity);
  return n > a.max_seq || n < 0 ? 0 : n;
}
// Query token of row r of a kv head's rows (r < 2^20: the rounding of the magic
// number adds less than r / 2^29 < 1 / group).
__device__ __forceinline__ int row_tok(const Kv8Attn& a, int r) {
  return a.group == 1 ? r : (int)__umulhi((unsigned)r, a.magic);
}
// Units that an item's rows see (the last row sees the most).
__device__ __forceinline__ int item_units(const Kv8Attn& a, int len, int mg) {
  const int last = min(a.ntok * a.group, (mg + 1) * a.irows) - 1;
  const int keys = max(0, len - a.ntok + 1 + row_tok(a, last));
  return (keys + kKeys - 1) / kKeys;
}

// Entries e = (sequence, m-group), e = b * mgroups + mg, hold nkv items of
// item_units() units each.
__device__ __forceinline__ int entry_units(const Kv8Attn& a, int e) {
  const int b = a.mgroups == 1 ? e : e / a.mgroups;
  return a.nkv * item_units(a, seq_len(a, b), e - b * a.mgroups);
}
// Every thread of the CTA (128) takes entries [*e0, *e1) and gets the units
// before them; returns all entries' units.
__device__ __forceinline__ int scan_entries(const Kv8Attn& a, int tid, int* s_warp, int* before, int* e0, int* e1) {
  const int entries = a.batch * a.mgroups, per = (entries + kThreads - 1) / kThreads;
  *e0 = min(entries, tid * per);
  *e1 = min(entries, *e0 + per);
  int sum = 0;
  for (int e = *e0; e < *e1; ++e) sum += entry_units(a, e);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if ((tid & 31) >= o) inc += v;
  }
  if ((tid & 31) == 31) s_warp[tid >> 5] = inc;
  __syncthreads();
  int base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < (tid >> 5)) base += s_warp[w];
    total += s_warp[w];
  }
  *before = base + inc - sum;
  return total;
}
// Units per CTA: equal runs, at least one unit per key-splitting warp.
__device__ __forceinline__ int run_units(const Kv8Attn& a, int total) {
  return max((total + a.ctas - 1) / a.ctas, kWarps / a.nm);
}

// What the join kernel needs of item i = (b * mgroups + mg) * nkv + g: how many
// CTAs hold a part of it (one: it is written already; 0: it has no units), the
// first of them, and whether its part there is that CTA's first (0) or last (1)
// partial.  Written by the CTA that begins the item.
__device__ __forceinline__ int4 make_cut(int parts, int cta, int slot) { return make_int4(parts, cta, slot, 0); }

// ------------------------------------------------------------------- fragments

// Byte offset of 16-byte chunk c of row r in a tile of rows of HD bytes laid
// down by TMA with an HD-byte swizzle.
template <int HD>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  constexpr int kShift = HD == 128 ? 0 : HD == 64 ? 1 : 2, kMask = HD / 16 - 1;
  return (uint32_t)(r * HD + ((c ^ ((r >> kShift) & kMask)) << 4));
}

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* x, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t turn8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <int BYTES>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* w) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
  float2 f;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(v));
  return f;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The CTA's barrier inside the item loop: it takes whole warps, whose lanes may
// just have done unequal work.
__device__ __forceinline__ void cta_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}
// What a row's raw scores over a block are multiplied by: its own factor (>= 0)
// times the scale of K, held to 2^120 (an infinity would make NaN of a score of 0;
// NaN stays).
__device__ __forceinline__ float score_factor(float row, float ksc) {
  float f;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(row * ksc), "f"(0x1p120f));
  return f;
}
// Which of the four codes of a word are NaN, as 0xff bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) {
  return __vcmpeq4(v & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

__device__ __forceinline__ void store_row4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store_row4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

template <int HD, int NT>
struct SplitSmem {
  // slots per warp: with one row tile three CTAs fit an SM, with two (twice the
  // accumulators) two
  static constexpr int kDepth = NT == 2 ? 3 : 2;
  static constexpr int kCtas = NT == 1 ? 3 : 2;
  // with four the query fragments stay in shared memory, each lane its own: [tile][word][lane][2]
  static constexpr bool kQShared = NT == 4;
  static constexpr size_t kQWarp = kQShared ? (size_t)NT * (HD / 16) * 32 * 8 : 0;
  static constexpr size_t kTile = (size_t)kKeys * HD;
  static constexpr size_t kSlot = 2 * kTile;
  // a warp's rows at an item's end, over its share of the slots (free then);
  // rows 4 floats longer against conflicts
  static constexpr int kRows = 8 * NT, kRowF = HD + 4;
  static constexpr size_t kShare = kDepth * kSlot > (size_t)kRows * kRowF * 4 ? kDepth * kSlot : (kRows * kRowF * 4 + 1023) / 1024 * 1024;
  static constexpr size_t kQ = kWarps * kShare;
  static constexpr size_t kML = kQ + kWarps * kQWarp;
  static constexpr size_t kNan = kML + (size_t)kWarps * kRows * 2 * 4;  // per warp: first NaN position of each dim
  static constexpr size_t kBars = kNan + (size_t)kWarps * HD * 4;
  static constexpr size_t kInts = kBars + 2 * kWarps * kDepth * 8;
  static constexpr size_t kTotal = kInts + 16 * 4 + 1024;
};

// Walks a CTA's units: item by item.
struct UnitWalk {
  int e, b, mg, g, len, nu, at;  // entry, its sequence and m-group, kv head, keys, units of an item, next unit
  __device__ __forceinline__ void entry_of(const Kv8Attn& a) {
    b = a.mgroups == 1 ? e : e / a.mgroups;
    mg = e - b * a.mgroups;
    len = seq_len(a, b);
    nu = item_units(a, len, mg);
  }
  __device__ __forceinline__ void seek(const Kv8Attn& a, int entry, int rem) {
    e = entry;
    entry_of(a);
    g = rem / nu;
    at = rem - g * nu;
  }
  // to the first unit of the next item (there is one)
  __device__ __forceinline__ void next_item(const Kv8Attn& a) {
    at = 0;
    if (++g == a.nkv) {
      g = 0;
      do {
        ++e;
        entry_of(a);
      } while (nu == 0);
    }
  }
};

// The V rows [row0, row1) of a 32-row tile in shared memory: rows from `stale`
// on are zeroed (they lie past the sequence and may hold anything; 0 x NaN would
// reach every query row); in the others the NaN codes are looked for.  first[d]
// becomes the lowest position of a NaN in dim d (pos0: the tile's first
// position).  Returns whether there was one.
template <int HD>
__device__ __noinline__ bool prepare_edge(uint8_t* vt, int stale, bool look, int pos0, int* first, int lane) {
  bool any = false;
  for (int i = lane; i < kKeys * HD / 16; i += 32) {
    const int r = i / (HD / 16), c = i % (HD / 16);
    uint4* p = reinterpret_cast<uint4*>(vt + tile_off<HD>(r, c));
    if (r >= stale) {
      *p = make_uint4(0u, 0u, 0u, 0u);
    } else if (look) {
      const uint4 v = *p;
      const uint32_t w[4] = {nan_bytes(v.x), nan_bytes(v.y), nan_bytes(v.z), nan_bytes(v.w)};
      if (w[0] | w[1] | w[2] | w[3]) {
        any = true;
        for (int j = 0; j < 16; ++j)
          if ((w[j >> 2] >> (8 * (j & 3))) & 1u) atomicMin(first + 16 * c + j, pos0 + r);
      }
    }
  }
  return __any_sync(0xffffffffu, any);
}

// Zeroes an m-group's rows of kv heads [g0, g1).
template <typename T, int HD>
__device__ __forceinline__ void zero_rows(const Kv8Attn& a, int b, int mg, int g0, int g1, int tid) {
  const int r0 = mg * a.irows, n = min(a.irows, a.ntok * a.group - r0) * (HD / 4);
  for (int i = tid; i < (g1 - g0) * n; i += kThreads) {
    const int g = g0 + i / n, r = r0 + i % n / (HD / 4), t = row_tok(a, r);
    store_row4(reinterpret_cast<T*>(a.out) +
                   (((size_t)b * a.ntok + t) * a.nh + g * a.group + (r - t * a.group)) * HD + i % (HD / 4) * 4,
               make_float4(0.f, 0.f, 0.f, 0.f));
  }
}

template <typename T, int HD, int NT>
__global__ void __launch_bounds__(kThreads, SplitSmem<HD, NT>::kCtas)
    kv8_split_kernel(const Kv8Attn a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using SM = SplitSmem<HD, NT>;
  constexpr bool kWide = sizeof(T) == 4;  // fp32: two fp16 parts of q and of p
  constexpr int kTerms = kWide ? 2 : 1;
  static_assert(kKeys == 32, "two key tiles a unit");
  constexpr int kMt = kKeys / 16, kC = HD / 16, kW = HD / 16;  // 16-key tiles; 16-dim chunks; words of a lane's key row
  constexpr int kDepth = SM::kDepth, kRows = SM::kRows;
  extern __shared__ __align__(1024) uint8_t kv8_smem_raw[];
  uint8_t* smem = kv8_smem_raw + ((1024u - (smem_u32(kv8_smem_raw) & 1023u)) & 1023u);
  float* MLw = reinterpret_cast<float*>(smem + SM::kML);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars);
  uint64_t* empty = full + kWarps * kDepth;
  int* s_int = reinterpret_cast<int*>(smem + SM::kInts);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kWarps * kDepth) {
    mbar_init(&full[tid], 1);
    mbar_init(&empty[tid], a.nm);
    fence_mbar_init();
  }
  // (no early launch of the join kernel: its CTAs took slots of the next call's)
  pdl_wait();

  // this CTA's run of units
  UnitWalk w;
  int u0 = 0, u1 = 0, run = 1;
  if (a.whole) {
    const int e = blockIdx.x / a.nkv;
    w.e = e;
    w.entry_of(a);
    w.g = blockIdx.x - e * a.nkv;
    w.at = 0;
    u1 = w.nu;
    if (w.nu == 0) zero_rows<T, HD>(a, w.b, w.mg, w.g, w.g + 1, tid);
    __syncthreads();  // the barriers are set up
    if (w.nu == 0) return;
  } else {
    int before, e0, e1;
    const int total = scan_entries(a, tid, s_int + 4, &before, &e0, &e1);
    run = run_units(a, total);
    u0 = (int)min((long long)blockIdx.x * run, (long long)total);
    u1 = min(total, u0 + run);
    if (u0 < u1)
      for (int e = e0; e < e1; ++e) {
        const int n = entry_units(a, e);
        if (before <= u0 && u0 < before + n) {
          s_int[0] = e;
          s_int[1] = u0 - before;
        }
        before += n;
      }
    // rows of items without a visible key are nobody's run: the CTAs share them out
    for (int e = blockIdx.x; e < a.batch * a.mgroups; e += gridDim.x)
      if (entry_units(a, e) == 0) {
        const int b = e / a.mgroups;
        zero_rows<T, HD>(a, b, e - b * a.mgroups, 0, a.nkv, tid);
        for (int g = tid; g < a.nkv; g += kThreads) a.cut[e * a.nkv + g] = make_cut(0, 0, 0);
      }
    __syncthreads();
    if (u0 >= u1) return;
    w.seek(a, s_int[0], s_int[1]);
  }

  const int kw = kWarps / a.nm;            // warps that split an item's keys
  const int mt = warp % a.nm, kg = warp / a.nm;
  const int gq = lane >> 2, tq = lane & 3;
  const int G = a.group, rows = a.ntok * G;
  const int mi = lane >> 3, mr = lane & 7;
  const float sl2 = fabsf(a.scale) * kLog2e;  // (its sign goes to the query rows)
  // the slots of this warp's group (the nm warps of one kg), a ring; its first
  // warp fills them
  const int slots = kDepth * a.nm, slot0 = kg * slots;
  uint8_t* ring = smem + (size_t)kg * a.nm * SM::kShare;
  int fill_s = 0, use_s = 0;
  uint32_t fill_ph = 0, use_ph = 0;
  int* first_nan = reinterpret_cast<int*>(smem + SM::kNan) + warp * HD;

  for (int u = u0; u < u1;) {
    const int n = min(w.nu - w.at, u1 - u);        // units of this item here
    const bool whole = n == w.nu;
    const int m0 = w.mg * a.irows + mt * kRows;    // this warp's first row
    const size_t head = (size_t)w.b * a.nkv + w.g;
    const float* ksp = a.ks + head * a.nblk;
    const float* vsp = a.vs + head * a.nblk;
    const int tile_row = (int)head * a.max_seq;

    // the query rows' and first scales' loads go out before the tiles' (behind
    // them they took 6900 cycles): row gq of each tile, the lane's HD / 4 dims
    constexpr int kV = Storage<T>::kVec, kQ = HD / 4 / kV;
    uint4 raw[NT][kQ];
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      const int r = m0 + gq + 8 * h, t = row_tok(a, r);
#pragma unroll
      for (int j = 0; j < kQ; ++j) raw[h][j] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const T* src = reinterpret_cast<const T*>(a.q) + (long long)w.b * a.q_seq_stride +
                       (long long)t * a.q_tok_stride + (long long)(w.g * G + r - t * G) * HD + tq * (HD / 4);
        if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
#pragma unroll
          for (int j = 0; j < kQ; ++j) raw[h][j] = __ldg(reinterpret_cast<const uint4*>(src) + j);
        } else {
#pragma unroll
          for (int j = 0; j < kQ; ++j) {
            float f[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) f[i] = to_f(src[j * kV + i]);
            raw[h][j] = pack16<T>(f);
          }
        }
      }
    }
    float ks_n = 0.f, vs_n = 0.f;
    if (kg < n) {
      ks_n = __ldg(ksp + (w.at + kg) * kKeys / kBlk);
      vs_n = __ldg(vsp + (w.at + kg) * kKeys / kBlk);
    }
    // units kg, kg + kw, ... of the n are this group's.  At an item's start every
    // slot is free: a lane each fills them
    auto copy_unit = [&](int unit, int slot) {
      uint64_t* bar = &full[slot0 + slot];
      uint8_t* st = ring + (size_t)slot * SM::kSlot;
      const int row = tile_row + (w.at + unit) * kKeys;
      mbar_arrive_expect_tx(bar, (uint32_t)SM::kSlot);
      tma_load_2d(st, &kmap, 0, row, bar);
      tma_load_2d(st + SM::kTile, &vmap, 0, row, bar);
    };
    const int mine = (n - kg + kw - 1) / kw;       // this group's units
    const int early = min(slots, mine);
    if (mt == 0 && lane < early) {
      int slot = fill_s + lane;
      if (slot >= slots) slot -= slots;
      copy_unit(kg + lane * kw, slot);
    }
    fill_s += early;
    if (fill_s >= slots) {
      fill_s -= slots;
      fill_ph ^= 1u;
    }
    int fill = kg + early * kw;

    // query fragments (the B operand: row gq, the lane's dims in words of four)
    uint32_t qb[kTerms][SM::kQShared ? 1 : NT][kW][2];
    uint2* qsh = reinterpret_cast<uint2*>(smem + SM::kQ + warp * SM::kQWarp) + lane;  // [NT][kW][32]
    float sc[NT][2];   // of rows 2 tq and 2 tq + 1 of each tile, as the scores sit
    int lim[NT][2];
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      float f[HD / 4];
#pragma unroll
      for (int j = 0; j < kQ; ++j) unpack16<T>(raw[h][j], f + j * kV);
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < HD / 4; ++j) m = fmaxf(m, fabsf(f[j]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // 2^k brings the row's largest magnitude to [256, 512)
      const int k = m > 0.f ? min(126, 127 + 8 - (int)(__float_as_uint(m) >> 23)) : 0;
      // (an infinite query leaves nothing but infinite and NaN scores: NaN, also
      // where all of them are -inf and no weight would be left)
      const float up = m < INFINITY ? copysignf(__uint_as_float((uint32_t)(127 + k) << 23), a.scale) : NAN;
      const float down = sl2 * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        const float x0 = f[4 * j] * up, x1 = f[4 * j + 1] * up, x2 = f[4 * j + 2] * up, x3 = f[4 * j + 3] * up;
        const uint32_t q0 = pack_f16x2(x0, x1), q1 = pack_f16x2(x2, x3);
        if constexpr (SM::kQShared) {
          static_assert(!SM::kQShared || !kWide, "four row tiles: one term");
          qsh[(h * kW + j) * 32] = make_uint2(q0, q1);
        } else {
          qb[0][h][j][0] = q0;
          qb[0][h][j][1] = q1;
          if constexpr (kWide) {
            const float2 y0 = unpack_f16x2(q0), y1 = unpack_f16x2(q1);
            qb[1][h][j][0] = pack_f16x2((x0 - y0.x) * kLow, (x1 - y0.y) * kLow);
            qb[1][h][j][1] = pack_f16x2((x2 - y1.x) * kLow, (x3 - y1.y) * kLow);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sc[h][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * tq + j));
        const int r = m0 + 8 * h + 2 * tq + j;
        lim[h][j] = r < rows ? w.len - a.ntok + 1 + row_tok(a, r) : 0;
      }
    }
    // keys below every row's limit need no mask
    const int clear = w.len - a.ntok + 1 + row_tok(a, min(m0, rows - 1));
    bool some_nan = false;  // first_nan is in use

    float o[NT][kC][4];  // (dim 16 c + 2 gq, row 2 tq), (same, + 1), (dim + 1, row), (dim + 1, row + 1)
    float m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int h = 0; h < NT; ++h) {
#pragma unroll
      for (int c = 0; c < kC; ++c) o[h][c][0] = o[h][c][1] = o[h][c][2] = o[h][c][3] = 0.f;
      m_run[h][0] = m_run[h][1] = -INFINITY;
      l_run[h][0] = l_run[h][1] = 0.f;
    }
    float unit = 0.f, unit_max = 0.f;
    bool coarse = false;  // a row's reference is large (the same in every lane)

    for (int x = kg; x < n; x += kw) {
      const int key0 = (w.at + x) * kKeys;
      const float ksc = ks_n, vsc = vs_n;
      if (x + kw < n) {
        ks_n = __ldg(ksp + (key0 + kw * kKeys) / kBlk);
        vs_n = __ldg(vsp + (key0 + kw * kKeys) / kBlk);
      }
      if (!tc_wait_asleep(&full[slot0 + use_s], use_ph) && lane == 0) atomicOr(a.err, kErrTimeout);
      __syncwarp();  // (each lane waited for itself: the MMAs take whole warps)
      uint8_t* tile = ring + (size_t)use_s * SM::kSlot;
      const uint32_t kt = smem_u32(tile), vt = kt + (uint32_t)SM::kTile;
      if (m0 < rows) {  // (three warps' rows of four: the last has none)
        // ---- scores: the key tiles side by side, so that no MMA waits for the last
        float s[NT][kMt][4];
        auto load_keys = [&](int m, uint32_t (*kb)[kW]) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 16 * m + 8 * i + gq;
            if constexpr (HD == 128) {
              lds_words<16>(kt + tile_off<HD>(r, 2 * tq), kb[i]);
              lds_words<16>(kt + tile_off<HD>(r, 2 * tq + 1), kb[i] + 4);
            } else if constexpr (HD == 64) {
              lds_words<16>(kt + tile_off<HD>(r, tq), kb[i]);
            } else {
              lds_words<8>(kt + tile_off<HD>(r, tq >> 1) + 8 * (tq & 1), kb[i]);
            }
          }
        };
        auto convert = [](const uint32_t (*kb)[kW], int j, uint32_t* ka) {
          ka[0] = e4m3x2_to_f16x2((uint16_t)(kb[0][j] & 0xffffu));
          ka[1] = e4m3x2_to_f16x2((uint16_t)(kb[1][j] & 0xffffu));
          ka[2] = e4m3x2_to_f16x2((uint16_t)(kb[0][j] >> 16));
          ka[3] = e4m3x2_to_f16x2((uint16_t)(kb[1][j] >> 16));
        };
        if constexpr (kWide) {
          // fp32: the tensor core cuts each sum's last bit off, so no chain is longer
          // than two MMAs (and the low terms have one of their own); they are added
          // with rounding.  One chain of sixteen left 1.3e-6 on outputs where fp32
          // products leave 0.7e-6.
          constexpr int kChains = kW < 4 ? kW : 4;
#pragma unroll
          for (int m = 0; m < kMt; ++m) {
            float t[kChains + 1][NT][4];
#pragma unroll
            for (int x2 = 0; x2 <= kChains; ++x2)
#pragma unroll
              for (int h = 0; h < NT; ++h) t[x2][h][0] = t[x2][h][1] = t[x2][h][2] = t[x2][h][3] = 0.f;
            uint32_t kb[2][kW];
            load_keys(m, kb);
#pragma unroll
            for (int j = 0; j < kW; ++j) {
              uint32_t ka[4];
              convert(kb, j, ka);
#pragma unroll
              for (int h = 0; h < NT; ++h) {
                mma_f16(t[j % kChains][h], ka, qb[0][h][j][0], qb[0][h][j][1]);
                mma_f16(t[kChains][h], ka, qb[kTerms - 1][h][j][0], qb[kTerms - 1][h][j][1]);
              }
            }
#pragma unroll
            for (int h = 0; h < NT; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float sum = t[0][h][i];
#pragma unroll
                for (int x2 = 1; x2 < kChains; ++x2) sum += t[x2][h][i];
                s[h][m][i] = fmaf(t[kChains][h][i], 1.f / kLow, sum);
              }
          }
        } else if constexpr (SM::kQShared) {  // the row tiles are side by side: one key tile at a time
#pragma unroll
          for (int m = 0; m < kMt; ++m) {
            uint32_t kb[2][kW];
            load_keys(m, kb);
#pragma unroll
            for (int h = 0; h < NT; ++h) s[h][m][0] = s[h][m][1] = s[h][m][2] = s[h][m][3] = 0.f;
#pragma unroll
            for (int j = 0; j < kW; ++j) {
              uint32_t ka[4];
              convert(kb, j, ka);
#pragma unroll
              for (int h = 0; h < NT; ++h) {
                const uint2 q = qsh[(h * kW + j) * 32];
                mma_f16(s[h][m], ka, q.x, q.y);
              }
            }
          }
        } else {
          // with one row tile two chains of sums per key tile, added at the end: a
          // chain of eight MMAs waits for itself
          constexpr int kChains = NT == 1 ? 2 : 1;
          float s2[kMt][4];
          uint32_t kb[kMt][2][kW];
#pragma unroll
          for (int m = 0; m < kMt; ++m) {
            load_keys(m, kb[m]);
            s2[m][0] = s2[m][1] = s2[m][2] = s2[m][3] = 0.f;
#pragma unroll
            for (int h = 0; h < NT; ++h) s[h][m][0] = s[h][m][1] = s[h][m][2] = s[h][m][3] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < kW; ++j)
#pragma unroll
            for (int m = 0; m < kMt; ++m) {
              uint32_t ka[4];
              convert(kb[m], j, ka);
#pragma unroll
              for (int h = 0; h < NT; ++h)
                mma_f16(kChains == 2 && j % 2 ? s2[m] : s[h][m], ka, qb[0][h][j][0], qb[0][h][j][1]);
            }
          if constexpr (kChains == 2) {
#pragma unroll
            for (int m = 0; m < kMt; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[0][m][i] += s2[m][i];
          }
        }
        // ---- the unit of the output from this block on: its V scale, within what
        // keeps all that was added in other units in range.  A block whose scale lies
        // outside adds its products times `apart`: fp32 to the sums, any scales; bf16
        // by way of the probabilities, where it loses bits from 2^-20 on (products of
        // their own took the registers of four row tiles: 336 bytes spilled).
        unit_max = fmaxf(unit_max, vsc);
        const float unit_new = kWide ? fminf(fmaxf(fmaxf(vsc, unit_max * 0x1p-60f), 0x1p-60f), 0x1p50f)
                                     : fmaxf(fmaxf(vsc, unit_max * 0x1p-80f), 0x1p-60f);
        const float ratio = unit_new == unit ? 1.f : unit / unit_new;
        const float apart = vsc == unit_new ? 1.f : vsc / unit_new;
        unit = unit_new;
        const bool edge = key0 + kKeys > clear;
        // ---- rows past the sequence, NaN that not every row sees
        bool drop_nan = false;
        if (edge && (a.ntok > 1 || key0 + kKeys > w.len)) {
          if (!some_nan) {
            for (int d = lane; d < HD; d += 32) first_nan[d] = INT32_MAX;
            __syncwarp();
          }
          drop_nan = prepare_edge<HD>(tile + SM::kTile, w.len - key0, a.ntok > 1, key0, first_nan, lane);
          some_nan |= drop_nan;
          __syncwarp();
        }
        // ---- V of the first 16 keys, on its way while the softmax runs
        auto load_values = [&](int kk, uint32_t (*r)[4]) {
#pragma unroll
          for (int c2 = 0; c2 < kC / 2; ++c2)
            ldsm4_t(vt + tile_off<HD>(16 * kk + (mi & 1) * 8 + mr, 2 * c2 + (mi >> 1)), r[c2]);
          if (drop_nan) {
#pragma unroll
            for (int c2 = 0; c2 < kC / 2; ++c2)
#pragma unroll
              for (int z = 0; z < 4; ++z) r[c2][z] &= ~nan_bytes(r[c2][z]);
          }
        };
        uint32_t r[kC / 2][4];
        load_values(0, r);
        // ---- softmax: value 2 i + j of tile m is key 16 m + 8 i + gq, row 2 tq + j
        bool grow = false;
        float top[NT][2];
        auto hidden = [&](int h, int j, int m, int i) { return key0 + 16 * m + 8 * i + gq >= lim[h][j]; };
#pragma unroll
        for (int h = 0; h < NT; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = score_factor(sc[h][j], ksc);
            float v[kMt][2];
#pragma unroll
            for (int m = 0; m < kMt; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i) v[m][i] = s[h][m][2 * i + j] * f;
            if (edge) {
#pragma unroll
              for (int m = 0; m < kMt; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (hidden(h, j, m, i)) v[m][i] = -INFINITY;
            }
            top[h][j] = fmaxf(fmaxf(v[0][0], v[0][1]), fmaxf(v[1][0], v[1][1]));
            grow |= top[h][j] - m_run[h][j] > kGrow;
          }
        if (__any_sync(0xffffffffu, grow)) {
          float move[NT][2];  // of the output: to the new reference and unit
          bool large = false;
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 <<= 1)
#pragma unroll
            for (int h = 0; h < NT; ++h)
#pragma unroll
              for (int j = 0; j < 2; ++j) top[h][j] = fmaxf(top[h][j], __shfl_xor_sync(0xffffffffu, top[h][j], o2));
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float mn = fmaxf(m_run[h][j], top[h][j]);
              const float alpha = ex2(m_run[h][j] - (mn == -INFINITY ? 0.f : mn));
              move[h][j] = ratio * alpha;
              l_run[h][j] *= alpha;
              m_run[h][j] = mn;
              large |= mn != -INFINITY && fabsf(mn) > kCoarse;
            }
          coarse = __any_sync(0xffffffffu, large);
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[h][c][j] *= move[h][j & 1];
        } else if (ratio != 1.f) {
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[h][c][j] *= ratio;
        }
        if (coarse) {  // (in one place: a branch at each row cost four row tiles 3 %)
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int m = 0; m < kMt; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[h][m][i] = __fmul_rn(s[h][m][i], score_factor(sc[h][i & 1], ksc));
        }
        uint32_t pb[kTerms][NT][kMt][2];
#pragma unroll
        for (int h = 0; h < NT; ++h) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = coarse ? 1.f : score_factor(sc[h][j], ksc);
            // (rounded up: never below the reference less the bias, nor above the reference)
            const float ms = __fadd_ru(m_run[h][j] == -INFINITY ? 0.f : m_run[h][j], -kPBias);
#pragma unroll
            for (int m = 0; m < kMt; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i) s[h][m][2 * i + j] = ex2(fmaf(s[h][m][2 * i + j], f, -ms));
            if (edge) {
#pragma unroll
              for (int m = 0; m < kMt; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (hidden(h, j, m, i)) s[h][m][2 * i + j] = 0.f;
            }
            const float sum = (s[h][0][j] + s[h][0][2 + j]) + (s[h][1][j] + s[h][1][2 + j]);
            l_run[h][j] += sum;
          }
          if (!kWide && apart != 1.f) {
#pragma unroll
            for (int m = 0; m < kMt; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[h][m][i] *= apart;
          }
#pragma unroll
          for (int m = 0; m < kMt; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p0 = s[h][m][2 * i], p1 = s[h][m][2 * i + 1];
              const uint32_t hi = pack_f16x2(p0, p1);
              pb[0][h][m][i] = turn8x8(hi);
              if constexpr (kWide) {
                const float2 y = unpack_f16x2(hi);
                pb[1][h][m][i] = turn8x8(pack_f16x2((p0 - y.x) * kLow, (p1 - y.y) * kLow));
              }
            }
        }
        // ---- output
#pragma unroll
        for (int kk = 0; kk < kMt; ++kk) {
          if (kk > 0) load_values(kk, r);
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            // bytes (key, dim): (0, even), (0, odd), (1, even), (1, odd)
            const uint32_t y0 = __byte_perm(r[c / 2][2 * (c & 1)], 0u, 0x3120);
            const uint32_t y1 = __byte_perm(r[c / 2][2 * (c & 1) + 1], 0u, 0x3120);
            const uint32_t va[4] = {e4m3x2_to_f16x2((uint16_t)(y0 & 0xffffu)), e4m3x2_to_f16x2((uint16_t)(y0 >> 16)),
                                    e4m3x2_to_f16x2((uint16_t)(y1 & 0xffffu)), e4m3x2_to_f16x2((uint16_t)(y1 >> 16))};
#pragma unroll
            for (int h = 0; h < NT; ++h) {
              if constexpr (kWide) {  // sums of their own, added with rounding (as the scores)
                float t[4] = {0.f, 0.f, 0.f, 0.f}, low[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(low, va, pb[kTerms - 1][h][kk][0], pb[kTerms - 1][h][kk][1]);
                mma_f16(t, va, pb[0][h][kk][0], pb[0][h][kk][1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[h][c][j] = fmaf(fmaf(low[j], 1.f / kLow, t[j]), apart, o[h][c][j]);
              } else {
                mma_f16(o[h][c], va, pb[0][h][kk][0], pb[0][h][kk][1]);
              }
            }
          }
        }
        if (edge) fence_async_smem();  // zeroed rows before the slot's next copy
      }
      __syncwarp();
      if (lane == 0) {
        if (a.nm > 1) mbar_arrive(&empty[slot0 + use_s]);
        if (mt == 0 && fill < n) {
          // (a warp with slots of its own has just read this one)
          if (a.nm > 1 && !tc_wait_asleep(&empty[slot0 + fill_s], fill_ph ^ 1u)) atomicOr(a.err, kErrTimeout);
          copy_unit(fill, fill_s);
        }
      }
      __syncwarp();
      if (fill < n) {
        fill += kw;
        if (++fill_s == slots) {
          fill_s = 0;
          fill_ph ^= 1u;
        }
      }
      if (++use_s == slots) {
        use_s = 0;
        use_ph ^= 1u;
      }
    }

    // ---- the item's rows: each warp's normalised output, maximum and sum, over
    // its share of the slots (all consumed, once every warp is here)
    cta_sync();
    float* Ow = reinterpret_cast<float*>(smem + (size_t)warp * SM::kShare);
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float l = l_run[h][j];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int r = 8 * h + 2 * tq + j;
        if (some_nan) {
#pragma unroll
          for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int d = 0; d < 2; ++d)
              if (first_nan[16 * c + 2 * gq + d] < lim[h][j]) o[h][c][2 * d + j] = NAN;
        }
#pragma unroll
        for (int c = 0; c < kC; ++c)
          *reinterpret_cast<float2*>(Ow + r * SM::kRowF + 16 * c + 2 * gq) =
              make_float2(o[h][c][j] * inv * unit, o[h][c][2 + j] * inv * unit);
        if (gq == 0) {
          MLw[2 * (kRows * warp + r)] = m_run[h][j];
          MLw[2 * (kRows * warp + r) + 1] = l;
        }
      }
    cta_sync();
    // ---- joined over the key-splitting warps: to the output, or to this CTA's
    // first (slot 0: the item began at or before the run) or last partial.  First
    // each row's weights, over its m and l
    const int part = 2 * blockIdx.x + (u != u0 ? 1 : 0);
    const int here = min(a.irows, rows - w.mg * a.irows);
    if (tid < here) {
      // row tid % kRows of warp tid / kRows; the next key part is nm warps on
      float2 ml[kWarps];
      float M = -INFINITY, W = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        if (k < kw) {
          ml[k] = *reinterpret_cast<const float2*>(MLw + 2 * (tid + kRows * a.nm * k));
          M = fmaxf(M, ml[k].x);
        }
      const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        if (k < kw) {
          ml[k].y = ml[k].y == 0.f ? 0.f : ml[k].y * ex2(ml[k].x - ms);
          W += ml[k].y;
        }
      const float inv = W == 0.f ? 0.f : 1.f / W;
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        if (k < kw) MLw[2 * (tid + kRows * a.nm * k)] = ml[k].y * inv;
      if (!whole)
        *reinterpret_cast<float2*>(a.part + (size_t)2 * a.ctas * a.irows * HD + 2 * ((size_t)part * a.irows + tid)) =
            make_float2(M, W * kPartScale);
    }
    if (tid == 0 && w.at == 0 && !a.whole)
      a.cut[w.e * a.nkv + w.g] = make_cut((u + w.nu - 1) / run - (int)blockIdx.x + 1, blockIdx.x, u != u0 ? 1 : 0);
    cta_sync();
#pragma unroll 2
    for (int i = tid; i < here * (HD / 4); i += kThreads) {
      const int rr = i / (HD / 4), d = i % (HD / 4) * 4;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        if (k < kw) {
          const int wp = rr / kRows + k * a.nm, lr = rr % kRows;
          const float e = MLw[2 * (kRows * wp + lr)];
          const float4 v = *reinterpret_cast<const float4*>(smem + (size_t)wp * SM::kShare + (lr * SM::kRowF + d) * 4);
          // (no weight is skipped: a part that saw no key has outputs of 0, and a NaN
          // of V counts also where the part's weight underflows)
          y.x = fmaf(e, v.x, y.x);
          y.y = fmaf(e, v.y, y.y);
          y.z = fmaf(e, v.z, y.z);
          y.w = fmaf(e, v.w, y.w);
        }
      if (whole) {
        const int r = w.mg * a.irows + rr, t = row_tok(a, r);
        store_row4(reinterpret_cast<T*>(a.out) +
                       (((size_t)w.b * a.ntok + t) * a.nh + w.g * G + (r - t * G)) * HD + d,
                   y);
      } else {
        *reinterpret_cast<float4*>(a.part + ((size_t)part * a.irows + rr) * HD + d) = y;
      }
    }
    u += n;
    w.at += n;
    if (u < u1) {
      fence_async_smem();  // the rows before the slots' next copies
      cta_sync();
      w.next_item(a);
    }
  }
}

// Joins the partial rows of the items that a run's end cut, in the runs' order:
// CTA (i, y) takes item i's rows y, y + gridDim.y, ...
// A row is read by pg groups of lanes, eight loads in flight each: by all of the
// CTA's groups where a few long sequences leave hundreds of parts (then the rows
// are spread over gridDim.y), by one where a batch's items have two or three.
constexpr int kJoinThreads = 256;
template <typename T, int HD>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const Kv8Attn a) {
  constexpr int kLanes = HD / 4, kGroups = kJoinThreads / kLanes, kBatch = 8;
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float2 s_ml[kGroups];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid % kLanes, grp = tid / kLanes;
  const int4 cut = a.cut[blockIdx.x];
  const int n = cut.x, c = cut.y;
  if (n < 2) return;
  const int e = blockIdx.x / a.nkv, g = blockIdx.x - e * a.nkv, b = e / a.mgroups, mg = e - b * a.mgroups;
  const int irows = a.irows;
  const int here = min(irows, a.ntok * a.group - mg * irows);
  int pg = kGroups;
  if (gridDim.y == 1)
    while (pg > 1 && (kGroups / pg < here || pg > n)) pg >>= 1;
  const int per = kGroups / pg;              // rows of a pass
  const int sub = grp % pg, row = grp / pg;  // this group's share of the parts, its row of the pass
  const float* ml = a.part + (size_t)2 * a.ctas * irows * HD;
  for (int base = blockIdx.y; base < here; base += gridDim.y == 1 ? per : (int)gridDim.y) {
    const int rr = gridDim.y == 1 ? base + row : base;
    const bool in = rr < here;
    // part i: of CTA c + i, its first partial (CTA c's as the cut says)
    const size_t at0 = ((size_t)2 * c + cut.z) * irows + rr;
    const size_t at1 = (size_t)2 * c * irows + rr, step = (size_t)2 * irows;
    float M = -INFINITY, W = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = sub; in && i0 < n; i0 += kBatch * pg) {
      float4 v[kBatch];
      float2 w[kBatch];
      float mb = M;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * pg;
        const size_t at = i == 0 ? at0 : at1 + i * step;
        if (i < n) {
          w[k] = *reinterpret_cast<const float2*>(ml + 2 * at);
          v[k] = *reinterpret_cast<const float4*>(a.part + at * HD + 4 * lane);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i0 + k * pg < n) mb = fmaxf(mb, w[k].x);
      const float ms = mb == -INFINITY ? 0.f : mb;
      const float keep = ex2(M - ms);
      M = mb;
      W *= keep;
      y = make_float4(y.x * keep, y.y * keep, y.z * keep, y.w * keep);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i0 + k * pg < n) {  // (no weight is skipped, as above)
          const float e = w[k].y * ex2(w[k].x - ms);
          W += e;
          y.x = fmaf(e, v[k].x, y.x);
          y.y = fmaf(e, v[k].y, y.y);
          y.z = fmaf(e, v[k].z, y.z);
          y.w = fmaf(e, v[k].w, y.w);
        }
    }
    if (pg > 1) {  // the groups of a row, in order
      __syncthreads();
      s_o[tid] = y;
      if (lane == 0) s_ml[grp] = make_float2(M, W);
      __syncthreads();
      if (sub == 0) {
        for (int k = 1; k < pg; ++k) M = fmaxf(M, s_ml[grp + k].x);
        const float ms = M == -INFINITY ? 0.f : M;
        y = make_float4(0.f, 0.f, 0.f, 0.f);
        W = 0.f;
        for (int k = 0; k < pg; ++k) {
          const float2 u = s_ml[grp + k];
          const float e = ex2(u.x - ms);
          const float4 v = s_o[tid + k * kLanes];
          W = fmaf(e, u.y, W);
          y.x = fmaf(e, v.x, y.x);
          y.y = fmaf(e, v.y, y.y);
          y.z = fmaf(e, v.z, y.z);
          y.w = fmaf(e, v.w, y.w);
        }
      }
    }
    if (in && sub == 0) {
      const float inv = W == 0.f ? 0.f : 1.f / W;
      const int r = mg * irows + rr, t = row_tok(a, r);
      store_row4(reinterpret_cast<T*>(a.out) +
                     (((size_t)b * a.ntok + t) * a.nh + g * a.group + (r - t * a.group)) * HD + 4 * lane,
                 make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    }
  }
}

template <typename T, int HD, int NT>
q2_status split_t(const Kv8Attn& a, const uint8_t* kc, const uint8_t* vc, cudaStream_t st) {
  using SM = SplitSmem<HD, NT>;
  auto* kernel = kv8_split_kernel<T, HD, NT>;
  static std::atomic<uint64_t> done{0};
  if (first_on_device(done)) {
    Q2_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SM::kTotal));
    done_on_device(done);
  }
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)a.batch * a.nkv * a.max_seq;
  Q2_TRY(make_tmap_2d_u8(&km, kc, rows, HD, HD, kKeys, HD, HD));
  Q2_TRY(make_tmap_2d_u8(&vm, vc, rows, HD, HD, kKeys, HD, HD));
  const int items = a.batch * a.nkv * a.mgroups;
  Q2_LAUNCH(kernel, dim3(a.whole ? items : a.ctas), dim3(kThreads), SM::kTotal, st, true, a, km, vm);
  if (a.whole) return Q2_OK;
  // few items: a CTA per row of each, else one per item
  Q2_LAUNCH(kv8_join_kernel<T, HD>, dim3(items, items <= 32 ? a.irows : 1), dim3(kJoinThreads), 0, st, true, a);
  return Q2_OK;
}

template <typename T, int HD>
q2_status split_hd(const Kv8Attn& a, const uint8_t* kc, const uint8_t* vc, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (a.nt == 4) return split_t<T, HD, 4>(a, kc, vc, st);
  return a.nt == 1 ? split_t<T, HD, 1>(a, kc, vc, st) : split_t<T, HD, 2>(a, kc, vc, st);
}

template <typename T>
q2_status split(const Kv8Attn& a, int hd, const uint8_t* kc, const uint8_t* vc, cudaStream_t st) {
  switch (hd) {
    case 32: return split_hd<T, 32>(a, kc, vc, st);
    case 64: return split_hd<T, 64>(a, kc, vc, st);
    default: return split_hd<T, 128>(a, kc, vc, st);
  }
}

// Row tiles per warp, warps per item, items per kv head, CTAs and workspace of
// the split kernel.
struct SplitPlan {
  int nt, nm, irows, mgroups, ctas;
  bool whole;  // every item gets a CTA of its own
  size_t cut_bytes, bytes;
};
SplitPlan split_plan(size_t batch, size_t ntok, size_t nh, size_t nkv, size_t hd, size_t max_seq, int dtype) {
  SplitPlan p;
  const int rows = (int)(ntok * (nh / nkv));
  // Four tiles convert K and V half as often as two, but leave a warp alone with
  // them: 30 rows (4 sequences of up to 20011 positions) 26 us with two, 30 with
  // four; 384 rows over 32768 positions 100 and 82.  (fp32's second terms leave no
  // registers for four.)
  p.nt = rows <= 8 ? 1 : rows <= 64 || dtype == Q2_F32 ? 2 : 4;
  const int warps = ceil_div(rows, 8 * p.nt);
  p.nm = warps > 2 ? 4 : warps;
  p.irows = 8 * p.nt * p.nm;
  p.mgroups = ceil_div(rows, p.irows);
  p.ctas = num_sms() * (p.nt == 1 ? 3 : 2);  // all resident at once
  if (p.ctas > kCtasMax) p.ctas = kCtasMax;
  // Items whole: no scan of the lengths, nothing to join, one launch, no
  // workspace.  Where a warp has at most six units of an item to itself (12 / 2
  // heads, us on the GPU with / without: one sequence in a cache of 128 positions
  // 4.5 / 6.8, of 577 9.2 / 11.8, of 760 10.3 / 8.4; 4 of 577 9.2 / 12.1, of 760
  // 10.3 / 12.2; 16 of 760 10.3 / 13.5; 64 of 300 8.0 / 14.4, of 760 12.1 / 16.2, of
  // 2000 21.7 / 20.0: past the rule), and where items by far outnumber the
  // resident CTAs and are not so long that the last ones leave the machine idle
  // (128 sequences x 8 heads: ragged up to 2000 positions 43 / 55, of 2000 each 62
  // / 62, of 6000 each 155 / 141).
  const unsigned long long units = (max_seq + kKeys - 1) / kKeys, items = (unsigned long long)batch * nkv * p.mgroups;
  p.whole = units * p.nm <= 24 || (items >= 2ull * p.ctas && units <= 128);
  p.cut_bytes = (items * sizeof(int4) + 255) / 256 * 256;
  p.bytes = p.whole ? 0 : p.cut_bytes + (size_t)2 * p.ctas * p.irows * (hd + 2) * sizeof(float);
  return p;
}

q2_status set_flag(Kv8Attn* a) {
  a->err = op_error_flag();
  Q2_CHECK_ARG(a->err, Q2_ERR_CUDA, "cannot resolve the device error flag");
  return Q2_OK;
}
q2_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0 || (ws && !(reinterpret_cast<uintptr_t>(ws) & 255) && have >= need)) return Q2_OK;
  set_error("kv8 attention: the workspace is NULL, not 256-byte aligned or smaller than "
            "q2_kv8_attention_workspace says");
  return Q2_ERR_INVALID_ARG;
}

// ------------------------------------------------------------------ prompt rows

// The tcgen05 attention takes 128 rows of one query head a tile, whether they
// exist or not, and the copy of K and V comes before it; the split kernel's time
// goes with the rows of a kv head.  12 / 2 heads over 32768 keys: 64 prompt
// tokens (384 rows) 82 us in the split kernel against 115, 128 (768 rows) 141
// against 112; 512 tokens over 512 keys 48 against 24.
constexpr int kTcRows = 512;
bool use_tc(size_t ntok, size_t group, size_t hd, int dtype) {
  return dtype == Q2_BF16 && hd == 128 && ntok >= 16 && ntok * group >= kTcRows;
}

// Workspace: the tcgen05 attention's counters and slots, the NaN words (a memset
// clears the counters, another these), K, V.
struct TcPlan {
  size_t nan, k, v, bytes;
};
TcPlan tc_plan(size_t rows, size_t total, size_t nh, size_t nkv) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  TcPlan p;
  const size_t cache = up(total * nkv * 128 * 2);
  p.nan = up(attn_tc_ws_need((int)rows, (int)(total - rows), (int)nh));
  p.k = p.nan + up(nkv * 128 * sizeof(int));
  p.v = p.k + cache;
  p.bytes = p.v + cache;
  return p;
}

q2_status attn_tc(Kv8Attn a, const void* kc, const void* vc, void* ws, size_t ws_bytes, cudaStream_t st) {
  const TcPlan p = tc_plan(a.ntok, a.fixed_len, a.nh, a.nkv);
  Q2_TRY(check_workspace(ws, ws_bytes, p.bytes));
  Q2_TRY(set_flag(&a));
  char* base = static_cast<char*>(ws);
  Q2_CUDA_TRY(cudaMemsetAsync(base, 0, 4096, st));
  Q2_CUDA_TRY(cudaMemsetAsync(base + p.nan, 0, (size_t)a.nkv * 128 * sizeof(int), st));
  Kv8Read r = {};
  r.k = base + p.k;
  r.v = base + p.v;
  r.kc = static_cast<const uint8_t*>(kc);
  r.vc = static_cast<const uint8_t*>(vc);
  r.ks = a.ks;
  r.vs = a.vs;
  r.tok_stride = 128;
  r.head_stride = (long long)a.fixed_len * 128;
  r.batch = 1;
  r.ntok = a.fixed_len;
  r.nkv = a.nkv;
  r.hd = 128;
  r.max_seq = a.max_seq;
  r.vnan = reinterpret_cast<int*>(base + p.nan);
  Q2_TRY(launch_kv8_read(r, Q2_BF16, a.err, st));
  AttnRows t = {};
  t.q = a.q;
  t.q_row_stride = t.out_row_stride = (long long)a.nh * 128;
  t.k = r.k;
  t.v = r.v;
  t.kv_tok_stride = 128;
  t.kv_head_stride = r.head_stride;
  t.out = a.out;
  t.rows = a.ntok;
  t.nh = a.nh;
  t.nkv = a.nkv;
  t.hd = 128;
  t.base = a.fixed_len - a.ntok + 1;
  t.row_step = 1;
  t.scale = a.scale;
  return launch_attn_tc_nan(t, ws, a.err, st, r.vnan);
}

q2_status attn(Kv8Attn a, int hd, int dtype, const void* kc, const void* vc, void* ws, size_t ws_bytes,
               cudaStream_t st) {
  const SplitPlan p = split_plan(a.batch, a.ntok, a.nh, a.nkv, hd, a.max_seq, dtype);
  if ((unsigned long long)a.batch * a.nkv * p.mgroups * a.nblk >= (1ull << 29)) {
    set_error("kv8 attention: batch * kv heads * query row groups * key blocks must stay below 2^29");
    return Q2_ERR_SHAPE;
  }
  Q2_TRY(check_workspace(ws, ws_bytes, p.bytes));
  Q2_TRY(set_flag(&a));
  a.group = a.nh / a.nkv;
  a.magic = a.group == 1 ? 0u : (unsigned)(((1ull << 32) + a.group - 1) / a.group);
  a.nt = p.nt;
  a.nm = p.nm;
  a.irows = p.irows;
  a.mgroups = p.mgroups;
  a.ctas = p.ctas;
  a.whole = p.whole;
  a.cut = static_cast<int4*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.cut_bytes);
  const auto* k = static_cast<const uint8_t*>(kc);
  const auto* v = static_cast<const uint8_t*>(vc);
  return dtype == Q2_BF16 ? split<__nv_bfloat16>(a, hd, k, v, st) : split<float>(a, hd, k, v, st);
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
               Q2_ERR_INVALID_ARG, who ": the codes must be 16-byte aligned");                                   \
  Q2_CHECK_ARG((reinterpret_cast<uintptr_t>(out) & 15) == 0, Q2_ERR_INVALID_ARG, who ": out must be 16-byte aligned")

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
  Q2_CHECK_ARG((unsigned long long)batch * nkv * max_seq < (1ull << 31), Q2_ERR_SHAPE,
               "kv8_attention: need batch * nkv * max_seq < 2^31");
  Kv8Attn a = {};
  a.q = q;
  a.q_seq_stride = q_strides ? q_strides[0] : (long long)(ntok * nh * hd);
  a.q_tok_stride = q_strides ? q_strides[1] : (long long)(nh * hd);
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
  return attn(a, (int)hd, dtype, kc, vc, workspace, workspace_bytes, as_stream(stream));
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
  Q2_CHECK_ARG((unsigned long long)nkv * max_seq < (1ull << 31), Q2_ERR_SHAPE,
               "kv8_self_attention: need nkv * max_seq < 2^31");
  Kv8Attn a = {};
  a.q = q;
  a.q_seq_stride = 0;
  a.q_tok_stride = (long long)(nh * hd);
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
  // (the tcgen05 attention reads q and writes out in 16-byte pieces, and takes the
  // largest score, and masks, before it scales: right for a positive scale alone)
  if (use_tc(seqlen, nh / nkv, hd, dtype) && scale > 0.f &&
      ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) == 0)
    return attn_tc(a, kc, vc, workspace, workspace_bytes, as_stream(stream));
  return attn(a, (int)hd, dtype, kc, vc, workspace, workspace_bytes, as_stream(stream));
}

q2_status q2_kv8_attention_workspace(size_t batch, size_t ntok, size_t total_len, size_t nh, size_t nkv, size_t hd,
                                     size_t max_seq, int dtype, size_t* bytes) {
  clear_error();
  Q2_KV8_ATTN_CHECK("kv8_attention_workspace");
  Q2_CHECK_ARG(bytes, Q2_ERR_INVALID_ARG, "kv8_attention_workspace: NULL bytes");
  Q2_CHECK_ARG(ntok < 65536, Q2_ERR_SHAPE, "kv8_attention_workspace: need ntok < 65536");
  Q2_CHECK_ARG(total_len == 0 || (batch == 1 && ntok <= total_len && total_len <= max_seq), Q2_ERR_SHAPE,
               "kv8_attention_workspace: with a total_len, batch must be 1, ntok at most total_len and that at most max_seq");
  *bytes = 0;
  if (batch == 0 || ntok == 0) return Q2_OK;
  *bytes = split_plan(batch, ntok, nh, nkv, hd, max_seq, dtype).bytes;
  if (total_len && use_tc(ntok, nh / nkv, hd, dtype)) {
    const size_t tc = tc_plan(ntok, total_len, nh, nkv).bytes;
    if (tc > *bytes) *bytes = tc;  // (either path, as the scale and the alignment of q and out have it)
  }
  return Q2_OK;
}

}  // extern "C"
