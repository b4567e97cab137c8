// kv8_attn.cu -- attention over the 8-bit KV cache.
//
// Split kernel (any head dim, fp32 or bf16, one to many query rows).  The
// query rows of a kv head (ntok rows x nh / nkv heads) go on the M side of
// mma.sync m16n8k16 (16 rows an m-tile, up to four m-tiles a work item), keys
// on N for the scores, head dims on N for the output.  A work item is (sequence,
// m-tiles, kv head); its unit of work is 32 keys, half a block.  All items'
// units, in order, are dealt to a grid of resident CTAs in equal runs (lengths
// are read on the device), so ragged batches and a single long sequence load
// every SM alike; an item cut by a run's end leaves partial results that a
// second kernel joins in order (the same result every time).
//
// Bound by HBM (a byte per cached element): a unit's K and V rows arrive by TMA
// (swizzled to the head's row length).  Four warps a CTA; the nm warps that
// share an item's units (one m-tile each) share 3 nm slots, a warp with an
// m-tile of its own has three: its next two units are in flight while it
// computes.  (With whole blocks and one ring for the CTA a warp's next tile
// could only start when its last was done: 48 us instead of KV8_B64_US for 64
// sequences of up to 4096 positions.)  e4m3 values are exact in fp16 and
// Blackwell converts two per instruction, so the products run in fp16 with
// fp32 accumulation:
//   scores  a lane's 32 contiguous bytes of a key row (16-byte loads, no bank
//           conflicts under the swizzle) feed eight MMAs: the order of the dims
//           inside a dot product is free, the query's fragments take the same;
//   output  ldmatrix.trans on byte pairs gives a lane two keys x two dims; one
//           byte permute splits them into the even and the odd dim's operand.
// The query rows are scaled by a power of two into fp16's range (exact for
// bf16; fp32 queries are split into a high and a low fp16 part, two MMAs, and
// so are their probabilities).  Softmax in fp32, online, with p = 2^(s - m + 14):
// the common factor cancels and keeps probabilities down to 2^-28 of the
// largest at fp16's full 11 bits.  The scale of K multiplies the scores; the
// output is accumulated in units of the current block's V scale and moved to
// the next block's where that differs (a power of two: exact).
#include "common.cuh"
#include "e4m3.cuh"
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
constexpr int kDepth = 3;                       // slots per warp
constexpr int kCtasMax = 512;
constexpr float kPBias = 14.f;                  // p <= 2^14 in fp16

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
  int nm;       // m-tiles of an item: 1, 2 or 4
  int mgroups;  // items of a (sequence, kv head)
  float scale;
  void* out;    // [batch][ntok][nh][hd]
  float* part;  // [2 * CTAs][16 nm][hd + 2]: rows of partial items, then m and l of each row
  int ctas;     // of the split kernel
  int* err;
};

// --------------------------------------------------------------- work division

__device__ __forceinline__ int seq_len(const Kv8Attn& a, int b) {
  const int n = a.lens ? a.lens[b] : a.fixed_len;
  return n > a.max_seq || n < 0 ? 0 : n;
}
// Query token of row r of a kv head's rows (r < 2^20: the rounding of the magic
// number adds less than r / 2^29 < 1 / group).
__device__ __forceinline__ int row_tok(const Kv8Attn& a, int r) {
  return a.group == 1 ? r : (int)__umulhi((unsigned)r, a.magic);
}
// Units that an item's rows see (the last row sees the most).
__device__ __forceinline__ int item_units(const Kv8Attn& a, int len, int mg) {
  const int last = min(a.ntok * a.group, (mg + 1) * a.nm * 16) - 1;
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

template <typename T, int HD>
struct SplitSmem {
  static constexpr size_t kTile = (size_t)kKeys * HD;
  static constexpr size_t kSlot = 2 * kTile;
  // a warp's rows at an item's end, over its share of the slots (free then);
  // rows 16 floats longer against conflicts
  static constexpr int kRowF = HD + 16;
  static constexpr size_t kShare = kDepth * kSlot > 16 * kRowF * 4 ? kDepth * kSlot : (16 * kRowF * 4 + 1023) / 1024 * 1024;
  static constexpr size_t kML = kWarps * kShare;
  static constexpr size_t kNan = kML + (size_t)kWarps * 16 * 2 * 4;  // per warp: first NaN position of each dim
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

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 2)
    kv8_split_kernel(const Kv8Attn a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using SM = SplitSmem<T, HD>;
  constexpr bool kWide = sizeof(T) == 4;  // fp32: two fp16 parts of q and of p
  constexpr int kTerms = kWide ? 2 : 1;
  constexpr int kNt = kKeys / 8, kC = HD / 16;
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
  pdl_launch_dependents();
  pdl_wait();

  // this CTA's run of units
  int before, e0, e1;
  const int total = scan_entries(a, tid, s_int + 4, &before, &e0, &e1);
  const int run = run_units(a, total);
  const int u0 = (int)min((long long)blockIdx.x * run, (long long)total), u1 = min(total, u0 + run);
  if (u0 < u1)
    for (int e = e0; e < e1; ++e) {
      const int n = entry_units(a, e);
      if (before <= u0 && u0 < before + n) {
        s_int[0] = e;
        s_int[1] = u0 - before;
      }
      before += n;
    }
  if (blockIdx.x == 0 && a.lens)
    for (int b = tid; b < a.batch; b += kThreads)
      if (a.lens[b] > a.max_seq) atomicOr(a.err, kErrCapacity);
  __syncthreads();
  if (u0 >= u1) return;
  UnitWalk w;
  w.seek(a, s_int[0], s_int[1]);

  const int kw = kWarps / a.nm;            // warps that split the keys of an m-tile
  const int mt = warp % a.nm, kg = warp / a.nm;
  const int gq = lane >> 2, tq = lane & 3;
  const int G = a.group, rows = a.ntok * G;
  const int mi = lane >> 3, mr = lane & 7;
  const float sl2 = a.scale * kLog2e;
  // the slots of this warp's group (the nm warps of one kg), a ring; the warp
  // of m-tile 0 fills them
  const int slots = kDepth * a.nm, slot0 = kg * slots;
  uint8_t* ring = smem + (size_t)kg * a.nm * SM::kShare;
  int fill_s = 0, use_s = 0;
  uint32_t fill_ph = 0, use_ph = 0;
  int* first_nan = reinterpret_cast<int*>(smem + SM::kNan) + warp * HD;

  for (int u = u0; u < u1;) {
    const int n = min(w.nu - w.at, u1 - u);        // units of this item here
    const bool whole = n == w.nu;
    const int m0 = (w.mg * a.nm + mt) * 16;        // the m-tile's first row
    const bool two = m0 + 8 < rows;                // rows 8..15 exist
    const size_t head = (size_t)w.b * a.nkv + w.g;
    const float* ksp = a.ks + head * a.nblk;
    const float* vsp = a.vs + head * a.nblk;
    const int tile_row = (int)head * a.max_seq;

    // units kg, kg + kw, ... of the n are this group's
    int fill = kg;
    auto fill_next = [&]() {
      if (fill >= n) return;
      if (!tc_wait_asleep(&empty[slot0 + fill_s], fill_ph ^ 1u)) atomicOr(a.err, kErrTimeout);
      uint64_t* bar = &full[slot0 + fill_s];
      uint8_t* st = ring + (size_t)fill_s * SM::kSlot;
      const int row = tile_row + (w.at + fill) * kKeys;
      mbar_arrive_expect_tx(bar, (uint32_t)SM::kSlot);
      tma_load_2d(st, &kmap, 0, row, bar);
      tma_load_2d(st + SM::kTile, &vmap, 0, row, bar);
      fill += kw;
      if (++fill_s == slots) {
        fill_s = 0;
        fill_ph ^= 1u;
      }
    };
    if (mt == 0 && lane == 0)
      for (int i = 0; i < slots; ++i) fill_next();
    float ks_n = 0.f, vs_n = 0.f;
    if (kg < n) {
      ks_n = __ldg(ksp + (w.at + kg) * kKeys / kBlk);
      vs_n = __ldg(vsp + (w.at + kg) * kKeys / kBlk);
    }

    // query fragments: rows gq and gq + 8, the lane's HD / 4 contiguous dims
    uint32_t qa[kTerms][HD / 16][4];
    float sc[2];
    int lim[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m0 + gq + 8 * h;
      float f[HD / 4];
      lim[h] = 0;
      if (r < rows) {
        const int t = row_tok(a, r), hq = r - t * G;
        lim[h] = w.len - a.ntok + 1 + t;
        const T* src = reinterpret_cast<const T*>(a.q) + (long long)w.b * a.q_seq_stride +
                       (long long)t * a.q_tok_stride + (long long)(w.g * G + hq) * HD + tq * (HD / 4);
        if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
          constexpr int kV = Storage<T>::kVec;
#pragma unroll
          for (int j = 0; j < HD / 4 / kV; ++j) unpack16<T>(__ldg(reinterpret_cast<const uint4*>(src) + j), f + j * kV);
        } else {
#pragma unroll
          for (int j = 0; j < HD / 4; ++j) f[j] = to_f(src[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < HD / 4; ++j) f[j] = 0.f;
      }
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < HD / 4; ++j) m = fmaxf(m, fabsf(f[j]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // 2^k brings the row's largest magnitude to [256, 512)
      const int k = m > 0.f ? min(126, 127 + 8 - (int)(__float_as_uint(m) >> 23)) : 0;
      const float up = __uint_as_float((uint32_t)(127 + k) << 23);
      sc[h] = sl2 * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
      for (int j = 0; j < HD / 16; ++j) {
        const float x0 = f[4 * j] * up, x1 = f[4 * j + 1] * up, x2 = f[4 * j + 2] * up, x3 = f[4 * j + 3] * up;
        qa[0][j][h] = pack_f16x2(x0, x1);
        qa[0][j][2 + h] = pack_f16x2(x2, x3);
        if constexpr (kWide) {
          const float2 y0 = unpack_f16x2(qa[0][j][h]), y1 = unpack_f16x2(qa[0][j][2 + h]);
          qa[1][j][h] = pack_f16x2(x0 - y0.x, x1 - y0.y);
          qa[1][j][2 + h] = pack_f16x2(x2 - y1.x, x3 - y1.y);
        }
      }
    }
    // keys below every row's limit need no mask
    const int clear = w.len - a.ntok + 1 + row_tok(a, min(m0, rows - 1));
    bool some_nan = false;  // first_nan is in use

    float o[kC][8];  // per chunk of 16 dims: even dims' tile, odd dims' tile
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) o[c][j] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float unit = 0.f, unit_max = 0.f;

    for (int x = kg; x < n; x += kw) {
      const int key0 = (w.at + x) * kKeys;
      const float ksc = ks_n, vsc = vs_n;
      if (x + kw < n) {
        ks_n = __ldg(ksp + (key0 + kw * kKeys) / kBlk);
        vs_n = __ldg(vsp + (key0 + kw * kKeys) / kBlk);
      }
      if (!tc_wait_asleep(&full[slot0 + use_s], use_ph) && lane == 0) atomicOr(a.err, kErrTimeout);
      uint8_t* tile = ring + (size_t)use_s * SM::kSlot;
      const uint32_t kt = smem_u32(tile), vt = kt + (uint32_t)SM::kTile;
      if (m0 < rows) {  // (three m-tiles of four: the last has no rows)
        // ---- scores: four key tiles side by side, so that no MMA waits for the last
        float s[kNt][4];
        uint32_t kb[kNt][HD / 16];
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
          const int r = nt * 8 + gq;
          if constexpr (HD == 128) {
            lds_words<16>(kt + tile_off<HD>(r, 2 * tq), kb[nt]);
            lds_words<16>(kt + tile_off<HD>(r, 2 * tq + 1), kb[nt] + 4);
          } else if constexpr (HD == 64) {
            lds_words<16>(kt + tile_off<HD>(r, tq), kb[nt]);
          } else {
            lds_words<8>(kt + tile_off<HD>(r, tq >> 1) + 8 * (tq & 1), kb[nt]);
          }
        }
#pragma unroll
        for (int j = 0; j < HD / 16; ++j)
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            const uint32_t b0 = e4m3x2_to_f16x2((uint16_t)(kb[nt][j] & 0xffffu));
            const uint32_t b1 = e4m3x2_to_f16x2((uint16_t)(kb[nt][j] >> 16));
            mma_f16(s[nt], qa[0][j], b0, b1);
            if constexpr (kWide) mma_f16(s[nt], qa[1][j], b0, b1);
          }
        // ---- the unit of this block's V scale (never 2^60 below the largest so
        // far: the output in units of it stays in range)
        unit_max = fmaxf(unit_max, vsc);
        const float unit_new = fmaxf(fmaxf(vsc, unit_max * 0x1p-60f), 0x1p-126f);
        const float ratio = unit_new == unit ? 1.f : unit / unit_new;
        const float pf = vsc == unit_new ? 1.f : vsc / unit_new;
        unit = unit_new;
        // ---- softmax of rows gq (h = 0) and gq + 8 (h = 1)
        const bool edge = key0 + kKeys > clear;
        uint32_t pa[kTerms][kNt / 2][4];
        float move[2] = {ratio, ratio};  // of the output: to the new maximum and unit
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) {
#pragma unroll
            for (int e = 0; e < kTerms; ++e)
#pragma unroll
              for (int kk = 0; kk < kNt / 2; ++kk) pa[e][kk][1] = pa[e][kk][3] = 0u;
            continue;
          }
          const float f = sc[h] * ksc;
          float mx = -INFINITY;
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float v = s[nt][2 * h + j] * f;
              if (edge && key0 + nt * 8 + 2 * tq + j >= lim[h]) v = -INFINITY;
              s[nt][2 * h + j] = v;
              mx = fmaxf(mx, v);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m_run[h], mx);
          const float ms = mn == -INFINITY ? 0.f : mn;
          const float alpha = ex2(m_run[h] - ms);
          move[h] *= alpha;
          m_run[h] = mn;
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float p = ex2(s[nt][2 * h + j] - ms + kPBias);
              s[nt][2 * h + j] = p;
              sum += p;
            }
          l_run[h] = l_run[h] * alpha + sum;
          if (pf != 1.f) {
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              s[nt][2 * h] *= pf;
              s[nt][2 * h + 1] *= pf;
            }
          }
#pragma unroll
          for (int kk = 0; kk < kNt / 2; ++kk)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const float p0 = s[2 * kk + v][2 * h], p1 = s[2 * kk + v][2 * h + 1];
              pa[0][kk][2 * v + h] = pack_f16x2(p0, p1);
              if constexpr (kWide) {
                const float2 hi = unpack_f16x2(pa[0][kk][2 * v + h]);
                pa[1][kk][2 * v + h] = pack_f16x2(p0 - hi.x, p1 - hi.y);
              }
            }
        }
        if (__any_sync(0xffffffffu, move[0] != 1.f || move[1] != 1.f)) {
#pragma unroll
          for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) o[c][j] *= move[(j >> 1) & 1];
        }
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
        // ---- output
#pragma unroll
        for (int kk = 0; kk < kNt / 2; ++kk) {
          uint32_t r[kC / 2][4];
#pragma unroll
          for (int c2 = 0; c2 < kC / 2; ++c2)
            ldsm4_t(vt + tile_off<HD>(16 * kk + (mi & 1) * 8 + mr, 2 * c2 + (mi >> 1)), r[c2]);
          if (drop_nan) {
#pragma unroll
            for (int c2 = 0; c2 < kC / 2; ++c2)
#pragma unroll
              for (int z = 0; z < 4; ++z) r[c2][z] &= ~nan_bytes(r[c2][z]);
          }
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            // bytes (key, dim): (0, even), (0, odd), (1, even), (1, odd)
            const uint32_t y0 = __byte_perm(r[c / 2][2 * (c & 1)], 0u, 0x3120);
            const uint32_t y1 = __byte_perm(r[c / 2][2 * (c & 1) + 1], 0u, 0x3120);
            const uint32_t e0v = e4m3x2_to_f16x2((uint16_t)(y0 & 0xffffu)), e1v = e4m3x2_to_f16x2((uint16_t)(y1 & 0xffffu));
            const uint32_t d0v = e4m3x2_to_f16x2((uint16_t)(y0 >> 16)), d1v = e4m3x2_to_f16x2((uint16_t)(y1 >> 16));
            mma_f16(o[c], pa[0][kk], e0v, e1v);
            mma_f16(o[c] + 4, pa[0][kk], d0v, d1v);
            if constexpr (kWide) {
              mma_f16(o[c], pa[1][kk], e0v, e1v);
              mma_f16(o[c] + 4, pa[1][kk], d0v, d1v);
            }
          }
        }
        if (edge) fence_async_smem();  // zeroed rows before the slot's next copy
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&empty[slot0 + use_s]);
        if (mt == 0) fill_next();
      }
      __syncwarp();
      if (++use_s == slots) {
        use_s = 0;
        use_ph ^= 1u;
      }
    }

    // ---- the item's rows: each warp's normalised output, maximum and sum, over
    // its share of the slots (all consumed: its group's, once every warp is here)
    asm volatile("bar.sync 1, 128;" ::: "memory");
    float* Ow = reinterpret_cast<float*>(smem + (size_t)warp * SM::kShare);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = l_run[h];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int r = gq + 8 * h;
      if (some_nan) {
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (first_nan[16 * c + 4 * tq + j] < lim[h]) o[c][2 * h + (j >> 1) + 4 * (j & 1)] = NAN;
      }
#pragma unroll
      for (int c = 0; c < kC; ++c)
        *reinterpret_cast<float4*>(Ow + r * SM::kRowF + 16 * c + 4 * tq) =
            make_float4(o[c][2 * h] * inv * unit, o[c][4 + 2 * h] * inv * unit, o[c][2 * h + 1] * inv * unit,
                        o[c][5 + 2 * h] * inv * unit);
      if (tq == 0) {
        MLw[2 * (16 * warp + r)] = m_run[h];
        MLw[2 * (16 * warp + r) + 1] = l;
      }
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    // ---- joined over the key-splitting warps: to the output, or to this CTA's
    // first (slot 0: the item began at or before the run) or last partial
    const int part = 2 * blockIdx.x + (u != u0 ? 1 : 0);
    const int irows = 16 * a.nm, here = min(irows, rows - w.mg * irows);
    for (int j = tid; j < here * (HD / 4); j += kThreads) {
      const int rr = j / (HD / 4), d = j % (HD / 4) * 4;  // row rr % 16 of warp rr / 16; the next key part is nm warps on
      float M = -INFINITY;
      for (int k = 0; k < kw; ++k) M = fmaxf(M, MLw[2 * (rr + 16 * a.nm * k)]);
      const float ms = M == -INFINITY ? 0.f : M;
      float W = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < kw; ++k) {
        const int at = rr + 16 * a.nm * k;
        const float l = MLw[2 * at + 1];
        if (l == 0.f) continue;
        const float e = l * ex2(MLw[2 * at] - ms);
        const float4 v = *reinterpret_cast<const float4*>(
            smem + (size_t)(at >> 4) * SM::kShare + ((at & 15) * SM::kRowF + d) * 4);
        W += e;
        y.x = fmaf(e, v.x, y.x);
        y.y = fmaf(e, v.y, y.y);
        y.z = fmaf(e, v.z, y.z);
        y.w = fmaf(e, v.w, y.w);
      }
      const float inv = W == 0.f ? 0.f : 1.f / W;
      y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      if (whole) {
        const int r = w.mg * irows + rr, t = row_tok(a, r);
        store_row4(reinterpret_cast<T*>(a.out) +
                       (((size_t)w.b * a.ntok + t) * a.nh + w.g * G + (r - t * G)) * HD + d,
                   y);
      } else {
        const size_t at = (size_t)part * irows + rr;
        *reinterpret_cast<float4*>(a.part + at * HD + d) = y;
        if (d == 0)
          *reinterpret_cast<float2*>(a.part + (size_t)2 * a.ctas * irows * HD + 2 * at) = make_float2(M, W);
      }
    }
    u += n;
    w.at += n;
    if (u < u1) {
      fence_async_smem();  // the rows before the slots' next copies
      asm volatile("bar.sync 1, 128;" ::: "memory");
      w.next_item(a);
    }
  }
}

// Joins the partial rows of the items that a run's end cut, in the runs' order,
// and zeroes the rows of items without a visible key.  One CTA per row.
template <typename T, int HD>
__global__ void __launch_bounds__(128) kv8_join_kernel(const Kv8Attn a) {
  constexpr int kLanes = HD / 4, kGroups = 128 / kLanes;
  constexpr int kMost = kCtasMax;  // an item's partial rows: at most one per CTA of the split kernel
  __shared__ float s_w[kMost], s_m[kMost];
  __shared__ int s_int[8];
  __shared__ float s_red[8];
  __shared__ float4 s_o[128];
  pdl_launch_dependents();
  const int r = blockIdx.x, g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int irows = 16 * a.nm, mg = r / irows, rr = r - mg * irows;
  const int G = a.group, t = row_tok(a, r);
  const int e = b * a.mgroups + mg;
  int before, e0, e1;
  pdl_wait();
  const int total = scan_entries(a, tid, s_int, &before, &e0, &e1);
  if (e0 <= e && e < e1) {
    for (int x = e0; x < e; ++x) before += entry_units(a, x);
    s_int[4] = before;
  }
  __syncthreads();
  T* out = reinterpret_cast<T*>(a.out) + (((size_t)b * a.ntok + t) * a.nh + g * G + (r - t * G)) * HD;
  const int nu = item_units(a, seq_len(a, b), mg);
  const int lane = tid % kLanes, grp = tid / kLanes;
  if (nu == 0) {
    if (grp == 0) store_row4(out + 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  const int run = run_units(a, total), us = s_int[4] + g * nu;
  const int c0 = us / run, n = (us + nu - 1) / run - c0 + 1;
  if (n == 1) return;  // the split kernel has written it
  const float* ml = a.part + (size_t)2 * a.ctas * irows * HD;
  auto row_of = [&](int i) { return (size_t)(2 * (c0 + i) + (us > (c0 + i) * run ? 1 : 0)) * irows + rr; };
  float M = -INFINITY;
  for (int i = tid; i < n; i += 128) {
    const float2 v = *reinterpret_cast<const float2*>(ml + 2 * row_of(i));
    s_m[i] = v.x;
    s_w[i] = v.y;
    M = fmaxf(M, v.x);
  }
  M = warp_max(M);
  if ((tid & 31) == 0) s_red[tid >> 5] = M;
  __syncthreads();
  M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
  const float ms = M == -INFINITY ? 0.f : M;
  float W = 0.f;
  for (int i = tid; i < n; i += 128) {
    const float x = s_w[i] == 0.f ? 0.f : s_w[i] * ex2(s_m[i] - ms);
    s_w[i] = x;
    W += x;
  }
  W = warp_sum(W);
  if ((tid & 31) == 0) s_red[4 + (tid >> 5)] = W;
  __syncthreads();
  W = (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = grp; i < n; i += kGroups) {
    const float x = s_w[i];
    if (x == 0.f) continue;
    const float4 v = *reinterpret_cast<const float4*>(a.part + row_of(i) * HD + 4 * lane);
    y.x = fmaf(x, v.x, y.x);
    y.y = fmaf(x, v.y, y.y);
    y.z = fmaf(x, v.z, y.z);
    y.w = fmaf(x, v.w, y.w);
  }
  s_o[tid] = y;
  __syncthreads();
  if (grp == 0) {
    for (int k = 1; k < kGroups; ++k) {
      const float4 v = s_o[k * kLanes + lane];
      y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
    store_row4(out + 4 * lane, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
  }
}

template <typename T, int HD>
q2_status split_t(const Kv8Attn& a, const uint8_t* kc, const uint8_t* vc, cudaStream_t st) {
  using SM = SplitSmem<T, HD>;
  auto* kernel = kv8_split_kernel<T, HD>;
  Q2_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SM::kTotal));
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)a.batch * a.nkv * a.max_seq;
  Q2_TRY(make_tmap_2d_u8(&km, kc, rows, HD, HD, kKeys, HD, HD));
  Q2_TRY(make_tmap_2d_u8(&vm, vc, rows, HD, HD, kKeys, HD, HD));
  Q2_LAUNCH(kernel, dim3(a.ctas), dim3(kThreads), SM::kTotal, st, true, a, km, vm);
  Q2_LAUNCH(kv8_join_kernel<T, HD>, dim3(a.ntok * a.group, a.nkv, a.batch), dim3(128), 0, st, true, a);
  return Q2_OK;
}

template <typename T>
q2_status split(const Kv8Attn& a, int hd, const uint8_t* kc, const uint8_t* vc, cudaStream_t st) {
  switch (hd) {
    case 32: return split_t<T, 32>(a, kc, vc, st);
    case 64: return split_t<T, 64>(a, kc, vc, st);
    default: return split_t<T, 128>(a, kc, vc, st);
  }
}

// m-tiles per item, items per kv head, CTAs and workspace of the split kernel.
struct SplitPlan {
  int nm, mgroups, ctas;
  size_t bytes;
};
SplitPlan split_plan(size_t ntok, size_t nh, size_t nkv, size_t hd) {
  SplitPlan p;
  const int mtiles = ceil_div((long long)(ntok * (nh / nkv)), 16);
  p.nm = mtiles > 2 ? 4 : mtiles;
  p.mgroups = ceil_div(mtiles, p.nm);
  p.ctas = num_sms() * 2;  // all resident at once
  if (p.ctas > kCtasMax) p.ctas = kCtasMax;
  p.bytes = (size_t)2 * p.ctas * 16 * p.nm * (hd + 2) * sizeof(float);
  return p;
}

q2_status attn(Kv8Attn a, int hd, int dtype, const void* kc, const void* vc, void* ws, size_t ws_bytes,
               cudaStream_t st) {
  const SplitPlan p = split_plan(a.ntok, a.nh, a.nkv, hd);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < p.bytes) {
    set_error("kv8 attention: the workspace is NULL, not 256-byte aligned or smaller than "
              "q2_kv8_attention_workspace says");
    return Q2_ERR_INVALID_ARG;
  }
  if ((unsigned long long)a.batch * a.nkv * p.mgroups * a.nblk >= (1ull << 29)) {
    set_error("kv8 attention: batch * kv heads * query row groups * key blocks must stay below 2^29");
    return Q2_ERR_SHAPE;
  }
  a.group = a.nh / a.nkv;
  a.magic = a.group == 1 ? 0u : (unsigned)(((1ull << 32) + a.group - 1) / a.group);
  a.nm = p.nm;
  a.mgroups = p.mgroups;
  a.ctas = p.ctas;
  a.part = static_cast<float*>(ws);
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
  a.err = flag;
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
  int* flag = op_error_flag();
  Q2_CHECK_ARG(flag, Q2_ERR_CUDA, "cannot resolve the device error flag");
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
  a.err = flag;
  return attn(a, (int)hd, dtype, kc, vc, workspace, workspace_bytes, as_stream(stream));
}

q2_status q2_kv8_attention_workspace(size_t batch, size_t ntok, size_t total_len, size_t nh, size_t nkv, size_t hd,
                                     int dtype, size_t* bytes) {
  clear_error();
  const size_t max_seq = 1;
  Q2_KV8_ATTN_CHECK("kv8_attention_workspace");
  Q2_CHECK_ARG(bytes, Q2_ERR_INVALID_ARG, "kv8_attention_workspace: NULL bytes");
  Q2_CHECK_ARG(ntok < 65536, Q2_ERR_SHAPE, "kv8_attention_workspace: need ntok < 65536");
  (void)batch;
  (void)total_len;
  *bytes = ntok ? split_plan(ntok, nh, nkv, hd).bytes : 0;
  return Q2_OK;
}

}  // extern "C"
