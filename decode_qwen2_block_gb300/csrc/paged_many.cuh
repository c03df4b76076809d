// Attention over a paged K/V cache for many rows: prompts and chunks of them
// (rows of one sequence, causal), and a prefix that all sequences share (its
// keys are read once for the rows of the whole batch).
//
// Bound by the tensor cores and the exponentials: 4 D flops and one 2^x per
// score.  A unit is two blocks of 128 / G tokens, each with the G query heads of
// one kv head: 256 rows that share every K/V tile of 128 slots.  The CTAs (one
// per SM) take equal ranges of the line of all units' tiles, as the few-row
// kernel does (see paged.h).  Twelve warps:
//   warp 0     producer: q of both blocks once per unit, then K and V tiles, page
//              by page (each lane one box of 64 columns), into a ring of tiles.
//   warps 1, 2 MMA issuers (lane 0) of block 0 and 1: S = Q K^T (M = N = 128), then in
//              turn O += P V and the next tile's S, so that one block's products run
//              under the other's softmax.  An issuer a block: issuing an MMA takes
//              the thread as long as the MMA itself (64 clocks), so what one thread
//              does in between (a wait, a commit: 250 clocks) leaves the tensor core
//              idle; one issuer for both blocks took 4150 clocks a tile instead.
//   warps 4-7, 8-11   softmax of block 0 and 1, a thread per row: scores from TMEM,
//              online softmax in base 2 with lazy rescaling of O, P (fp16)
//              over S's own columns (TMEM: S0 S1 O0 O1 = 512 columns).
// Over an 8-bit cache (k8) the producer's ring holds codes and scales, and four more warps
// (12-15, a thread a slot) make each tile fp16 in the ring that the MMAs read: exact, so
// all else is as over an fp16 cache.
// MMAs of one thread execute in order: a block's S_j+1 is written after its PV_j has
// read P_j, and a commit behind S_j+1 says that PV_j is complete too.
// Slots that no row of the unit sees have their V rows zeroed before PV (0 * NaN
// is NaN).  Every wait is bounded.
//
// Measured with the merge, in a graph, 12 heads on 2 kv heads of 128: 8 prompts of 700 -
// 2000 tokens 80 us (648 TFLOP/s; the kernel alone 690), 512 tokens behind 3584 slots
// 27 us.  From batches of 1 - 10 equal units a CTA, none cut, of 1 - 16 tiles: a tile takes
// 1.66 us (3400 clocks, 2048 of them its 32 MMAs: S = Q K^T reads 128 bytes of shared
// memory per clock, all there is, while the next tiles' 64 KB arrive), a unit's begin and
// end 2.6 us (5400 clocks, 1.6 tiles), all else of the call, with the merge that finds
// nothing cut, 10.6 us.
// k8, the same way: a tile 2.07 us (64 columns 1.69, fp16 1.53): the conversion reads 32 KB and
// writes 64 KB of shared memory beside the MMAs' own reads; leaving either out would
// save 0.2 - 0.3 us, its arithmetic nothing.  The softmax warps as converters, in their waits:
// 2.89; codes from memory into the converters' registers, no ring of them: 2.60.
#pragma once

#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kv8.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "tcgen05.cuh"

namespace blk {
namespace {

// k8: the cache is in 8 bits, and a fourth group of four warps makes its tiles fp16.
template <bool k8>
constexpr int kThreadsOf = k8 ? 512 : 384;
// Registers: a softmax thread holds a row of 128 scores.  The block is launched
// with 168 a thread (384 x 168 = 64512); warps 0-3 keep 72, the softmax warps take
// 216 (the prefix's variant 88 and 208: 56.2 us against 59.4): 128 x 72 + 256 x
// 216 = 128 x 88 + 256 x 208 = 64512.  The launch bounds allow 168 and the compiler takes
// them all, but nothing forces it: a larger share would wait forever for registers that the
// block does not have, so configure_paged_many looks at the count.
// k8: 128 a thread at the launch, kConv for the warps that convert.
template <bool k8>
constexpr int kRegsLaunch = k8 ? 128 : 168;
template <int D, bool kPrefix, bool k8>
struct Regs {
  static constexpr int kFew = k8 ? (D == 128 ? 56 : 40) : kPrefix ? 88 : 72;
  static constexpr int kMany = k8 ? (D == 128 ? 208 : 216) : kPrefix ? 208 : 216;
  static constexpr int kConv = k8 ? 40 : 0;
  static_assert(128 * (kFew + kConv) + 256 * kMany <= kThreadsOf<k8> * kRegsLaunch<k8>, "register split");
};
constexpr int kTile = kPagedManyTile;
constexpr int kInfos = 8;
constexpr float kRescaleLog2 = 8.f;   // see the softmax
// Weights are formed 2^7 times their size (O and l carry the factor, it cancels), so that
// fp16 holds them to 2^-11 of themselves down to 2^-21 of the greatest and to half of
// 2^-31 below; with kRescaleLog2 they reach 2^15, half of what fp16 holds (see weight_plain
// for scores that need more room).
constexpr float kWeightLog2 = 7.f;
constexpr int kMinTiles = 2;          // of a CTA: a piece of less is all begin and end
constexpr int kHead = kPagedManyHead;

struct alignas(16) ManyInfo {
  int flags;                 // 1 first tile of the piece, 2 last, 4 the end, 8 block 1 has rows
  int slot0, lo, hi;         // first slot; slots that some row sees: [lo, hi)
  int first;                 // slot of the unit's first token
  int ntok, r0, g;           // tokens, batch row of the first, kv head
  int dst;                   // -1 whole, else the partial slot
  int pad[3];
};

template <int D, bool k8>
struct MSmem {
  static constexpr int NB = D / kKv8Block;
  static constexpr int kQBlk = 128 * D * 2;                  // [D / 64][128 rows][128 B]
  static constexpr int kKV = kTile * D * 2;                  // K or V tile, the same form
  static constexpr int kRing = D == 128 ? (k8 ? 4 : 5) : 8;
  static constexpr int kS = (kRing + 1) / 2;                 // see the kernel
  static constexpr int kRingOff = 2 * kQBlk;
  // 8 bits: K or V tiles' codes [128 slots][D], then their scales [128 slots][D / 32]
  static constexpr int kCodes = k8 ? kTile * D : 0, kScales = k8 ? kTile * NB : 0;
  static constexpr int kCRing = k8 ? (D == 128 ? 2 : 4) : 0;
  static constexpr int kCOff = kRingOff + kRing * kKV;
  static constexpr int kScOff = kCOff + kCRing * kCodes;
  static constexpr int kInfoOff = kScOff + kCRing * kScales;
  static constexpr int kBarOff = kInfoOff + kInfos * (int)sizeof(ManyInfo);
  static constexpr int kEnd = kBarOff + (kRing + 2 * kS + 8 + (k8 ? 2 * kCRing + 1 : 0)) * 8 + 16;
  static constexpr size_t kBytes = (size_t)kEnd + 1024;
  static constexpr uint32_t kSCol = 0, kOCol = 256;
  static_assert(kBarOff % 8 == 0 && kBytes + (k8 ? 256 : 0) <= 232448, "shared memory");
};

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ int4 lds128(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {   // 2^x; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 bytes; `wide`: dst is 32-byte aligned (else 16).
__device__ __forceinline__ void st_global32(void* dst, const uint32_t* v, bool wide) {
  if (!wide) {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Pairs of fp32 in one instruction, and the maximum of three.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A unit of the own parts: tokens tok .. tok + ntok - 1 of a sequence.
struct Unit {
  int tok, ntok, r0;         // first token, tokens, batch row of the first
  int L, lo, hi;             // the sequence's history; slots that some row sees: [lo, hi)
};
__device__ __forceinline__ Unit unit_of(const PagedAttnParams& p, const PagedSeq& s, int u, int utok) {
  Unit x;
  x.tok = u * utok;
  x.ntok = min(utok, s.n - x.tok);
  x.r0 = s.r0 + x.tok;
  x.L = s.L;
  x.lo = paged_lo(p, s.L + x.tok);
  x.hi = s.L + x.tok + x.ntok;
  return x;
}
__device__ __forceinline__ int unit_tiles(const Unit& x) {
  return (x.hi + kTile - 1) / kTile - x.lo / kTile;
}

// Exclusive sum over the block of one value per thread; `total` is the sum.
template <int kThreads>
__device__ __forceinline__ int64_t block_excl(int64_t v, int64_t* warp_sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
  return before + x - v;
}

template <bool k8>
using ManyParams = std::conditional_t<k8, PagedMany8Params, PagedManyParams>;

template <int D, bool kPrefix, bool k8>
__global__ void __launch_bounds__(kThreadsOf<k8>, 1)
    paged_many_kernel(const __grid_constant__ ManyParams<k8> q) {
  using Sm = MSmem<D, k8>;
  using R3 = Regs<D, kPrefix, k8>;
  constexpr int kThreads = kThreadsOf<k8>;
  // Ring item 2 j is K of tile j, item 2 j + 1 its V.  The commit behind a block's S of
  // tile j says that everything it issued up to there is done: with both blocks'
  // the items up to 2 j and, at a piece's end, q are free.  The producer waits for
  // that, for item i with j = (i - R + 1) / 2, at most kS - 1 tiles behind the
  // issuers: kS barriers in turn, so that no phase is overtaken.
  constexpr int R = Sm::kRing, H = D / 64, kS = Sm::kS;
  const PagedAttnParams& p = q.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + Sm::kRingOff;
  volatile ManyInfo* infos = reinterpret_cast<volatile ManyInfo*>(smem + Sm::kInfoOff);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + Sm::kBarOff);
  uint64_t* q_full = kv_full + R;       // [2] q of a block
  uint64_t* s_full = q_full + 2;        // [2][kS] S of a block in TMEM, tile j's at j % kS
  uint64_t* p_full = s_full + 2 * kS;   // [2] P of a block in TMEM (O rescaled)
  uint64_t* o_full = p_full + 2;        // [2] O complete at the end of a piece
  uint64_t* drain = o_full + 2;         // [2]
  // 8 bits: codes there, codes read (a ring of their own), q of a piece used up
  constexpr int C = Sm::kCRing;
  uint64_t* c_full = drain + 2;
  uint64_t* c_empty = c_full + C;
  uint64_t* q_free = c_empty + C;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(k8 ? q_free + 1 : drain + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  // what needs nothing of the kernels before: barriers, TMEM, tensor maps
  if (threadIdx.x == 0) {
    for (int s = 0; s < R; ++s) mbar_init(&kv_full[s], k8 ? 2 : 1);
    if constexpr (k8) {
      for (int s = 0; s < C; ++s) {
        mbar_init(&c_full[s], 1 + 32);      // the copies of codes, and each lane's scales
        mbar_init(&c_empty[s], 2);
      }
      mbar_init(q_free, 2);
    }
    for (int k = 0; k < 2 * kS; ++k) mbar_init(&s_full[k], 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(&p_full[k], 5);      // the softmax warps and the other block's issuer
      mbar_init(&o_full[k], 1);
      mbar_init(&q_full[k], 1);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
            smem_u32(tmem_slot)),
        "r"(512u)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    prefetch_tmap(&p.tm_q);
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  griddep_wait();
  griddep_launch();
  // this CTA's range of the line of tiles
  const int utok = 2 * q.btok;
  int64_t T1;
  __shared__ int64_t wsum[kThreads / 32], start_cum;
  __shared__ int start_b, start_u;
  int64_t before = 0, mine = 0;
  int k0 = 0, k1 = 0;
  // own: units before each sequence, and the sequences where a thread has one each (in
  // the q area, until q comes)
  int* uoff = reinterpret_cast<int*>(smem);
  PagedSeq* seqs = reinterpret_cast<PagedSeq*>(smem + (kMaxSeqs + 16) * 4);
  static_assert((kMaxSeqs + 16) * 4 + kThreads * sizeof(PagedSeq) <= 2 * Sm::kQBlk, "q area");
  const bool few_seqs = p.B <= kThreads;
  auto seq = [&](int b) { return few_seqs ? seqs[b] : load_seq(p, b); };
  if constexpr (kPrefix) {
    T1 = (int64_t)q.units * ((p.prefix_len + kTile - 1) / kTile + kHead);
  } else {
    // Every CTA sums the units' tiles itself: units of all sequences first (a run
    // of sequences per thread), then their tiles (a run of units per thread).  (By the
    // producer warp alone, without barriers: one prompt's chunk 28.0 -> 27.6 us, but 8
    // prompts 80.4 -> 82.4, a lane having nine units of theirs one after another.)
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int64_t n = 0, R64;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const PagedSeq s = load_seq(p, b);
      n += (s.n + utok - 1) / utok;
      bad |= s.bad;
      if (few_seqs) seqs[b] = s;
      if (p.upb && cta == 0)           // entries of units that are not there
        for (int u = (s.n + utok - 1) / utok; u < p.upb; ++u)
          for (int g = 0; g < p.Hkv; ++g) p.cut[(g * p.B + b) * p.upb + u].c0 = -1;
    }
    if (bad && cta == 0) set_error(p.err, kDevPage);
    int64_t at = block_excl<kThreads>(n, wsum, R64);
    for (int b = b0; b < b1; ++b) {
      uoff[b] = (int)at;
      at += (seq(b).n + utok - 1) / utok;
    }
    __syncthreads();
    const int units = (int)R64, pu = (units + kThreads - 1) / kThreads;
    k0 = min(units, (int)threadIdx.x * pu);
    k1 = min(units, k0 + pu);
    if (k0 < k1) {
      int lo = 0, hi = p.B;            // last sequence with uoff <= k0: it has unit k0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (uoff[mid] <= k0) lo = mid; else hi = mid;
      }
      PagedSeq s = seq(lo);
      for (int k = k0, u = k0 - uoff[lo]; k < k1; ++k, ++u) {
        while (u * utok >= s.n) {
          s = seq(++lo);
          u = 0;
        }
        mine += unit_tiles(unit_of(p, s, u, utok)) + kHead;
      }
    }
    before = block_excl<kThreads>(mine, wsum, T1);
  }
  const int64_t T = T1 * p.Hkv;
  int nc = p.nc;
  if constexpr (!kPrefix) {
    const int64_t enough = (T + kMinTiles - 1) / kMinTiles;
    nc = (int)(enough < p.nc ? (enough < 1 ? 1 : enough) : p.nc);
  }
  const int64_t t0 = cta < nc ? range_of(T, cta, nc) : T;
  const int64_t t1 = cta < nc ? range_of(T, cta + 1, nc) : T;
  if (t0 >= t1) {
    if (threadIdx.x == 0 && !kPrefix && !p.upb) p.cut[cta].c0 = -1;
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot),
                   "r"(512u)
                   : "memory");
    }
    return;
  }
  const int g0 = small_div(t0, T1);
  if constexpr (!kPrefix) {
    const int64_t x = t0 - g0 * T1;
    if (mine > 0 && before <= x && x < before + mine) {    // the range begins in this thread's run
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (uoff[mid] <= k0) lo = mid; else hi = mid;
      }
      PagedSeq s = seq(lo);
      int64_t cum = before;
      for (int u = k0 - uoff[lo];; ++u) {
        while (u * utok >= s.n) {
          s = seq(++lo);
          u = 0;
        }
        const int wt = unit_tiles(unit_of(p, s, u, utok)) + kHead;
        if (x < cum + wt) {
          start_b = lo;
          start_u = u;
          start_cum = cum;
          break;
        }
        cum += wt;
      }
    }
    __syncthreads();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // uoff's place takes q by TMA
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // S of tile j of both blocks is done (j < 0: nothing to wait for): everything that was
  // issued before it is, too
  auto s_done = [&](int j) {
    const bool done = j < 0 || (mbar_wait_near(&s_full[j % kS], (uint32_t)(j / kS) & 1u, p.err) &&
                                mbar_wait_near(&s_full[kS + j % kS], (uint32_t)(j / kS) & 1u, p.err));
    return __all_sync(0xffffffffu, done);
  };
  if (k8 && warp >= 12) {
    if constexpr (k8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R3::kConv));
      // ------------------------------------------------------------- converters
      // Two warps make K tiles fp16 and two V tiles, 32 slots and 64 columns at a time: a lane's
      // codes and scales to the place and order that a tile of an fp16 cache would have, zeros
      // where no row of the unit sees the slot.  (All four warps on one tile after another: the
      // waits around each follow one another, 2.20 us a tile of 128 columns against 2.07.)
      const int own = (warp - 12) >> 1, r0 = (warp & 1) * 64 + lane;
      for (int i = own;; i += 2) {       // ring item i: K (even) or V of tile i / 2
        if (!__all_sync(0xffffffffu, mbar_wait_near(&c_full[i % C], (uint32_t)(i / C) & 1u, p.err))) break;
        const int4 f = lds128(smem_u32(const_cast<ManyInfo*>(&infos[(i >> 1) % kInfos])));
        const bool end = (f.x & 4) != 0;
        if (end && own == 1) break;
        if (!s_done((i - R + 1) >> 1)) break;        // what lay in the item's place is used up
        if (!end) {
#pragma unroll 1
          for (int part = 0; part < D / 32; ++part) {          // rows r0 / r0 + 32, columns 0 - 63 / 64 - 127
            const int r = r0 + (part & 1) * 32, half = part >> 1;
            const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
            const uint32_t from = smem_u32(smem + Sm::kCOff) + (i % C) * Sm::kCodes + r * D;
            const uint32_t to = smem_u32(ring) + (i % R) * Sm::kKV + half * 16384 + r * 128;
            uint4 c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int4 v = lds128(from + (((half * 4 + k) ^ sw) << 4));
              c[k] = make_uint4(v.x, v.y, v.z, v.w);
            }
            uint32_t w = kv8_lds_scales<Sm::NB>(smem_u32(smem + Sm::kScOff) + (i % C) * Sm::kScales + r * Sm::NB);
            w = f.y + r >= f.z && f.y + r < f.w ? w >> (half * 16) : 0;
            if (part == D / 32 - 1) {
              __syncwarp();
              if (lane == 0) mbar_arrive(&c_empty[i % C]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t b = k >> 1;        // the block's scale, doubled to fp16
              // (any scale's form: what these warps compute is not what they take their time for)
              const Kv8Unit<true> u(__byte_perm(w, 0, b << 12 | 4 << 8 | b << 4 | 4));
              sts128(to + (((2 * k) ^ (r & 7)) << 4), u(c[k].x, 0x4140), u(c[k].x, 0x4342),
                     u(c[k].y, 0x4140), u(c[k].y, 0x4342));
              sts128(to + (((2 * k + 1) ^ (r & 7)) << 4), u(c[k].z, 0x4140), u(c[k].z, 0x4342),
                     u(c[k].w, 0x4140), u(c[k].w, 0x4342));
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[i % R]);
        if (end) break;
      }
    }
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R3::kMany));
    // --------------------------------------------------------------- softmax
    const int blk = (warp - 4) >> 2;
    const int qt = warp & 3;                     // TMEM lane quarter of this warp
    const int r = qt * 32 + lane;                // row of the block
    const uint32_t loff = (uint32_t)(qt * 32) << 16;
    const uint32_t tS = tmem + Sm::kSCol + blk * 128 + loff;
    const uint32_t tO = tmem + Sm::kOCol + blk * 128 + loff;
    const float sl2 = p.scale_log2;
    const int rt = r / p.G;                      // token of the row in its block
    // 32-byte stores where the rows allow them (pointers are 16-byte aligned, as the
    // workspace's parts are with respect to one another by 256)
    const bool wide = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.out_stride % 16 == 0;
    const bool wide_part = reinterpret_cast<uintptr_t>(p.part) % 32 == 0;
    float m = -INFINITY, l = 0.f, most = kRescaleLog2;
    int seg = 0, last = 0, low = 0;              // slots that the row sees: [low, last]
    bool row_ok = false;                         // the row is a token's
    bool ok = true;
    // decisions before a warp-collective TMEM access are uniform over the warp
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_near(bar, parity, p.err));
    };
    for (int it = 0; ok; ++it) {
      if (!wait_all(&s_full[blk * kS + it % kS], (uint32_t)(it / kS) & 1u)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // the scores and the tile's description on their way together
      float sv[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tc_ld32(tS + c, sv + c);
      const uint32_t fi = smem_u32(const_cast<ManyInfo*>(&infos[it % kInfos]));
      const int4 fa = lds128(fi), fb = lds128(fi + 16);
      const int flags = fa.x, slot0 = fa.y, lo = fa.z, hi = fa.w;
      const int first = fb.x, ntok = fb.y;
      tc_wait_ld();
      if (flags & 4) break;
      if (blk == 1 && !(flags & 8)) {    // the unit has no rows in block 1
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[blk]);
        if (flags & 2) {
          if (!wait_all(&o_full[blk], (uint32_t)seg & 1u)) { ok = false; break; }
          ++seg;
        }
        continue;
      }
      if (flags & 1) {                   // a new piece
        const int t = blk * q.btok + rt; // token of the unit
        row_ok = rt < q.btok && t < ntok;
        last = kPrefix ? hi - 1 : first + min(t, ntok - 1);
        low = kPrefix ? 0 : max(lo, paged_window(p, last));
        m = -INFINITY;
        l = 0.f;
      }
      const int first_last = kPrefix ? hi - 1 : first + blk * q.btok;   // of the block's first row
      if (slot0 + kTile - 1 > first_last) {      // some row sees less than the tile
        const int lim = last - slot0;
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c > lim) sv[c] = -INFINITY;
      }
      if (!kPrefix && (slot0 < lo || p.window > 0)) {
        const int lim = low - slot0;
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c < lim) sv[c] = -INFINITY;
      }
      float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
      for (int c = 0; c < kTile; c += 8) {
        a0 = max3(a0, sv[c], sv[c + 1]);
        a1 = max3(a1, sv[c + 2], sv[c + 3]);
        a2 = max3(a2, sv[c + 4], sv[c + 5]);
        a3 = max3(a3, sv[c + 6], sv[c + 7]);
      }
      // (log2 units, less kWeightLog2; so is m)
      const float mx = fmaf(fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)), sl2, -kWeightLog2);
      // A row's reference maximum moves (and O, l are rescaled) only when the
      // maximum grew by more than 2^8 since: P <= 2^15 fits fp16, and 1 / l at the
      // end makes the choice exact.  (most: kRescaleLog2, counted from m as it stands.)
      // (Rows of no token hold whatever lay there: they take no part, or the moment
      // of a move, and with it the rounding of P, would differ from call to call.)
      const bool need = row_ok && ((m == -INFINITY) ? (mx != -INFINITY) : (mx - m > most));
      const bool move = __any_sync(0xffffffffu, need);
      if (move) {
        float mn = fmaxf(m, mx);
        if (mn != m && weight_plain(mn)) mn += kWeightLog2;
        most = weight_plain(mn) ? kRescaleLog2 - kWeightLog2 : kRescaleLog2;
        const float alpha = (m == -INFINITY || mn == m) ? 1.f : ex2(m - mn);
        m = mn;
        l *= alpha;
        if (!(flags & 1)) {             // (PV of the tile before is complete: S came behind it)
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            tc_ld32(tO + c, ov);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] *= alpha;
            tc_st32(tO + c, ov);
          }
        }
      }
      const float nref = (m == -INFINITY) ? 0.f : -m;
      const uint64_t sl22 = pack2(sl2, sl2), nref2 = pack2(nref, nref);
      uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = unpack2(fma2(pack2(sv[c + 2 * i], sv[c + 2 * i + 1]), sl22, nref2));
          const float e0 = ex2(x.x), e1 = ex2(x.y);
          if (i & 1) sum1 = add2(sum1, pack2(e0, e1));
          else sum0 = add2(sum0, pack2(e0, e1));
          const __half2 h2 = __floats2half2_rn(e0, e1);
          pk[i] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        tc_st16(tS + c / 2, pk);
      }
      if (!k8 && (slot0 < lo || slot0 + kTile > hi)) {
        // rows of V that no row of the unit sees are zero before PV (either block's
        // warps write the zeros before their own PV)
        const int vi = 2 * it + 1;
        ok = wait_all(&kv_full[vi % R], (uint32_t)(vi / R) & 1u);
        if (slot0 + r < lo || slot0 + r >= hi) {
          uint8_t* vrow = ring + (vi % R) * Sm::kKV + (size_t)r * 128;
#pragma unroll
          for (int hh = 0; hh < H; ++hh)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(vrow + hh * 16384 + k * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[blk]);
      const float2 sum = unpack2(add2(sum0, sum1));
      l += sum.x + sum.y;
      if (flags & 2) {
        if (!wait_all(&o_full[blk], (uint32_t)seg & 1u)) { ok = false; break; }
        ++seg;
        tc_fence_after();
        const int t = blk * q.btok + rt, r0 = fb.z, g = fb.w, hq = g * p.G + (r - rt * p.G);
        const int dst = lds128(fi + 32).x;
        const bool fin = dst < 0 && !p.own;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int64_t at = dst < 0 ? (int64_t)(r0 + t) * p.Hq + hq
                                   : ((int64_t)cta * 2 + dst) * p.slot_rows + blk * 128 + r;
        if (!fin && row_ok) (dst < 0 ? p.own_ml : p.ml)[at] = make_float2(m, l);
        __half* ho = p.out + (int64_t)(r0 + t) * p.out_stride + (int64_t)hq * D;
        float* fo = (dst < 0 ? p.own : p.part) + at * D;
        // a lane stores its own row, 32 bytes (a whole sector) at a time; the row is
        // read from TMEM at once (piece by piece between the stores took 3 times as long)
        float ov[D];
#pragma unroll
        for (int c = 0; c < D; c += 32) tc_ld32(tO + c, ov + c);
        tc_wait_ld();
        if (row_ok) {
          if (fin) {
#pragma unroll
            for (int c = 0; c < D; c += 16) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const __half2 h2 = __floats2half2_rn(ov[c + 2 * k] * inv, ov[c + 2 * k + 1] * inv);
                w[k] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              st_global32(ho + c, w, wide);
            }
          } else {
#pragma unroll
            for (int c = 0; c < D; c += 8)
              st_global32(fo + c, reinterpret_cast<const uint32_t*>(ov) + c, wide_part);
          }
        }
        tc_fence_before();
      }
    }
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R3::kFew));
  if (warp == 0) {
    // -------------------------------------------------------------- producer
    const int ps_lg = p.page_lg, boxes = kTile >> ps_lg;     // pages of a tile
    // 64 columns of one page (8 bits: all)
    const uint32_t box_bytes = (k8 ? (uint32_t)D : 128u) << ps_lg;
    int g = g0;
    int b, ui;                         // sequence (prefix: 0) and unit in it
    int64_t cum;                       // tiles before that unit
    int base32 = -1;
    PagedSeq mys = {};
    if constexpr (kPrefix) {
      const int64_t w = (p.prefix_len + kTile - 1) / kTile + kHead;
      b = 0;
      ui = small_div(t0 - g * T1, w);
      cum = ui * w;
    } else {
      b = start_b;
      ui = start_u;
      cum = start_cum;
    }
    int64_t lin = t0;
    int it = 0, seg = 0, item = 0;     // tiles, pieces, ring items so far
    int qn0 = 0, qn1 = 0;              // q loads of block 0, 1
    bool ok = true;
    if (!kPrefix && !p.upb && lane == 0) p.cut[cta].c0 = -1;   // until a unit is cut here
    auto wait_s = [&](int j) { ok = __all_sync(0xffffffffu, ok) && s_done(j); };
    // room for ring item `item` (8 bits: for its codes)
    auto wait_item = [&] {
      if constexpr (k8)
        ok = __all_sync(0xffffffffu, ok && (item < C || mbar_wait_near(&c_empty[item % C],
                                                                       (uint32_t)(item / C - 1) & 1u, p.err)));
      else wait_s((item - R + 1) >> 1);      // (arithmetic shift: below 0 nothing to wait for)
    };
    auto scales_of = [&](int v) -> const uint8_t* {
      if constexpr (k8) return v ? q.vs : q.ks;
      return nullptr;
    };
    while (lin < t1 && ok) {
      Unit u;
      if constexpr (kPrefix) {
        if (ui >= q.units) {
          ui = 0;
          cum = 0;
          ++g;
        }
        u.tok = ui * utok;
        u.ntok = min(utok, p.N - u.tok);
        u.r0 = u.tok;
        u.L = 0;
        u.lo = 0;
        u.hi = (int)p.prefix_len;
      } else {
        if (b >= p.B) {                // the next kv head begins again with the first sequence
          b = 0;
          ui = 0;
          cum = 0;
          ++g;
        }
        if ((b & ~31) != base32) {     // 32 sequences at a time, one per lane
          base32 = b & ~31;
          mys = base32 + lane < p.B ? (seg == 0 ? seq(base32 + lane) : load_seq(p, base32 + lane))
                                    : PagedSeq{};
        }
        PagedSeq s;
        s.r0 = __shfl_sync(0xffffffffu, mys.r0, b & 31);
        s.n = __shfl_sync(0xffffffffu, mys.n, b & 31);
        s.L = __shfl_sync(0xffffffffu, mys.L, b & 31);
        if (ui * utok >= s.n) {
          ++b;
          ui = 0;
          continue;
        }
        u = unit_of(p, s, ui, utok);
      }
      const int j0 = u.lo / kTile, nt = (u.hi + kTile - 1) / kTile - j0;
      const int64_t us = (int64_t)g * T1 + cum;
      const int64_t ue = us + kHead + nt;
      const int xa = (int)max((int64_t)0, lin - us - kHead);
      const int xb = (int)min((int64_t)nt, t1 - us - kHead);
      lin = ue;
      cum += nt + kHead;
      ++ui;
      if (xb <= xa) continue;          // its head alone lies here
      const bool whole = xa == 0 && xb == nt;
      const int dst = whole ? -1 : (xa == 0 ? 1 : 0);
      const bool two = u.ntok > q.btok;
      if (xa == 0) {
        if constexpr (kPrefix) {
          // until the own parts' kernel says otherwise a row has no own part
          for (int t = lane; t < u.ntok; t += 32)
            p.row_info[(int64_t)(u.r0 + t) * p.Hkv + g] = make_int4(-2, 0, 0, 0);
        } else {
          const int c1 = whole ? cta : cta_of(T, ue - 1, nc);
          const PagedPiece now = {whole ? -1 : cta, u.ntok * p.G, c1, u.r0, g};
          if (lane == 0 && (p.upb || !whole))
            p.cut[p.upb ? (g * p.B + b) * p.upb + ui - 1 : cta] = now;
          if (p.row_info)
            for (int t = lane; t < u.ntok; t += 32)
              p.row_info[(int64_t)(u.r0 + t) * p.Hkv + g] =
                  make_int4(whole ? -1 : cta, c1, 0,
                            t / q.btok * 128 + t % q.btok * p.G);
        }
      }
      const int32_t* row = kPrefix ? p.prefix_pages : p.table + (int64_t)b * p.max_blocks;
      const int64_t pre = kPrefix ? 0 : p.pre_here;
      for (int x = xa; x < xb && ok; ++x, ++it) {
        const int slot0 = (j0 + x) * kTile;
        // lane: half lane / 8 of the columns (8 bits: all of them), page lane % 8 of the tile
        const int i = lane & 7, half = lane >> 3, first = slot0 + (i << ps_lg);
        const bool take = half < (k8 ? 1 : H) && i < boxes && first < u.hi && first + (1 << ps_lg) > u.lo;
        int64_t page = -1;
        if (take) page = (first < pre ? p.prefix_pages : row)[first >> ps_lg];
        const bool in = page >= 0 && page < p.n_pages;
        if (take && !in) set_error(p.err, kDevPage);
        const int z = in ? (int)(page * p.Hkv + g) : (int)(p.n_pages * p.Hkv);   // zeros
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, take)) * box_bytes;
        const int at = half * (kTile * 128) + ((i << ps_lg) * 128);
        // 8 bits: the lane's 16 bytes of a tile's scales, those of 16 / NB slots
        const int sslot = lane * (16 / Sm::NB);
        bool sthere = false;
        int64_t srow = 0;
        if constexpr (k8) {
          const int spage = __shfl_sync(0xffffffffu, (int)page, (sslot >> ps_lg) & 7);
          sthere = sslot < kTile && slot0 + sslot < u.hi && slot0 + sslot + 16 / Sm::NB > u.lo &&
                   spage >= 0 && spage < p.n_pages;
          if (sthere)
            srow = ((((int64_t)spage * p.Hkv + g) << ps_lg) + (sslot & ((1 << ps_lg) - 1))) * Sm::NB;
        }
        // ring item `item`: K or V of this tile
        auto copy = [&](const CUtensorMap* map, const uint8_t* scales) {
          if constexpr (k8) {
            const int c = item % C;
            if (lane == 0) mbar_arrive_expect_tx(&c_full[c], bytes);
            __syncwarp();
            if (take)
              kv8_tma_codes(smem_u32(smem + Sm::kCOff) + c * Sm::kCodes + (i << ps_lg) * D, map, 0, z, &c_full[c]);
            if (sslot < kTile)
              kv8_copy16(smem_u32(smem + Sm::kScOff) + c * Sm::kScales + lane * 16, scales + srow, sthere);
            kv8_copies_arrive(&c_full[c]);
          } else {
            if (lane == 0) mbar_arrive_expect_tx(&kv_full[item % R], bytes);
            __syncwarp();
            if (take) tma_3d(ring + (item % R) * Sm::kKV + at, map, half * 64, 0, z, &kv_full[item % R]);
          }
          ++item;
        };
        wait_item();
        if (!ok) break;
        if (lane == 0) {
          volatile ManyInfo& f = infos[it % kInfos];
          f.slot0 = slot0;
          f.lo = u.lo;
          f.hi = u.hi;
          f.first = u.L + u.tok;
          f.ntok = u.ntok;
          f.r0 = u.r0;
          f.g = g;
          f.flags = (x == xa ? 1 : 0) | (x == xb - 1 ? 2 : 0) | (two ? 8 : 0);
          f.dst = dst;
        }
        copy(&p.tm_k, scales_of(0));
        if constexpr (k8) {            // (V first: it needs no wait for the piece before)
          wait_item();
          if (!ok) break;
          copy(&p.tm_v, scales_of(1));
        }
        if (x == xa) {
          // q of the piece before is used up
          if constexpr (k8)
            ok = __all_sync(0xffffffffu, seg == 0 || mbar_wait_near(q_free, (uint32_t)(seg - 1) & 1u, p.err));
          else
            wait_s(it - 1);
          if (!ok) break;
          // (a barrier a block: block 0 begins when its q is there)
          ++qn0;
          qn1 += two;
          if (lane == 0) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
              if (blk == 1 && !two) break;
              mbar_arrive_expect_tx(&q_full[blk], q.btok * p.G * D * 2);
              for (int hh = 0; hh < H; ++hh)
                tma_3d(smem + blk * Sm::kQBlk + hh * 16384, &p.tm_q, hh * 64, g * p.G,
                       u.r0 + blk * q.btok, &q_full[blk]);
            }
          }
        }
        if constexpr (!k8) {
          wait_item();
          if (!ok) break;
          copy(&p.tm_v, scales_of(1));
        }
      }
      ++seg;
    }
    if (ok) wait_item();
    if (ok) {
      if (lane == 0) infos[it % kInfos].flags = 4;
      __syncwarp();
      if constexpr (k8) {              // (to K's warps and to V's)
        for (int k = 0; k < 2; ++k) {
          wait_item();
          if (!ok) break;
          mbar_arrive(&c_full[item % C]);
          if (lane == 0) mbar_arrive(&c_full[item % C]);
          ++item;
        }
      } else {
        if (lane == 0) mbar_arrive(&kv_full[item % R]);
      }
    }
    if (!ok) {
      // copies in flight land before shared memory goes away
      if (qn0 > 0) mbar_wait(&q_full[0], (uint32_t)(qn0 - 1) & 1u, nullptr);
      if (qn1 > 0) mbar_wait(&q_full[1], (uint32_t)(qn1 - 1) & 1u, nullptr);
      constexpr int N = k8 ? C : R;
      for (int j = max(0, item - N); j < item; ++j)
        mbar_wait(k8 ? &c_full[j % N] : &kv_full[j % N], (uint32_t)(j / N) & 1u, nullptr);
    }
  } else if (warp < 3) {
    // -------------------------------------------- MMA issuer of block warp - 1
    if (lane == 0) {
      constexpr uint32_t id_s = tc_idesc(128, kTile, 0), id_o = tc_idesc(128, D, 1);
      const int blk = warp - 1;
      const uint32_t qb = smem_u32(smem) + blk * Sm::kQBlk, ra = smem_u32(ring);
      const uint32_t tS = tmem + Sm::kSCol + blk * 128, tO = tmem + Sm::kOCol + blk * 128;
      int qs = 0;                      // pieces whose q was waited for
      auto landed = [&](int i) {       // ring item i
        return mbar_wait_near(&kv_full[i % R], (uint32_t)(i / R) & 1u, p.err);
      };
      // S of tile it (flags f).  At the end of the range, or where the unit has no
      // rows in this block, the commit alone.
      // Descriptors: their low words hold the address, so a step adds to those (kd_lo:
      // K of tile it, formed before the waits).
      const uint32_t d_hi = (uint32_t)(tc_desc_kmajor(0) >> 32);
      const uint32_t q_lo = (uint32_t)tc_desc_kmajor(qb), r_lo = (uint32_t)tc_desc_kmajor(ra);
      const uint32_t v_hi = (uint32_t)(tc_desc_mnmajor(0) >> 32), rv_lo = (uint32_t)tc_desc_mnmajor(ra);
      auto desc = [](uint32_t hi, uint32_t lo) { return (uint64_t)hi << 32 | lo; };
      auto start_s = [&](int it, int f, uint32_t kd_lo) -> bool {
        if ((f & 1) && (blk == 0 || (f & 8))) {    // a new piece: its q
          if (!mbar_wait_near(&q_full[blk], (uint32_t)qs & 1u, p.err)) return false;
          ++qs;
        }
        tc_fence_after();
        if (!(f & 4) && (blk == 0 || (f & 8))) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
            tc_mma(tS, desc(d_hi, q_lo + o), desc(d_hi, kd_lo + o), id_s, ks != 0);
          }
        }
        if (blk == 1 || it > 0) mbar_arrive(&p_full[1 - blk]);
        tc_commit(&s_full[blk * kS + it % kS]);
        if constexpr (k8) {
          if ((f & 2) && !(f & 4)) tc_commit(q_free);      // the piece's last S
        }
        return true;
      };
      // The issuers take turns, block 0 first, so that the blocks' softmaxes stay half
      // a tile apart: issuing whenever P was there they fell into step (both softmaxes,
      // then both blocks' products: 4500 clocks a tile).  The turn is an arrival on the
      // other block's p_full: one wait for both.
      int f = 0;
      bool ok = landed(0);
      if (ok) {
        f = infos[0].flags;
        ok = start_s(0, f, r_lo);
      }
      for (int it = 0; ok && !(f & 4); ++it) {
        // everything but P first: while the softmax works this thread has the time
        if (!landed(2 * it + 1) || !landed(2 * it + 2)) break;
        const int fn = infos[(it + 1) % kInfos].flags;
        const uint32_t vd_lo = rv_lo + ((2 * it + 1) % R) * (Sm::kKV >> 4);
        const uint32_t kd_lo = r_lo + ((2 * it + 2) % R) * (Sm::kKV >> 4);
        if (!mbar_wait_near(&p_full[blk], (uint32_t)it & 1u, p.err)) break;
        tc_fence_after();
        if (blk == 0 || (f & 8)) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc_mma_ts(tO, tS + kk * 8, desc(v_hi, vd_lo + (kk * 16 * 128 >> 4)), id_o,
                      !(f & 1) || kk != 0);
        }
        if (f & 2) tc_commit(&o_full[blk]);
        if (!start_s(it + 1, fn, kd_lo)) break;
        f = fn;
      }
      // issued MMAs finish before TMEM and shared memory go away
      tc_commit(&drain[blk]);
      mbar_wait(&drain[blk], 0, nullptr);
    }
  }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
}

template <int D, bool kPrefix, bool k8>
cudaError_t launch_many(const ManyParams<k8>& p, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.a.nc);
  cfg.blockDim = dim3(kThreadsOf<k8>);
  cfg.dynamicSmemBytes = MSmem<D, k8>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_many_kernel<D, kPrefix, k8>, p);
}

template <int D, bool kPrefix, bool k8>
cudaError_t configure_one(bool* usable) {
  cudaFuncAttributes fa;
  const cudaError_t e = cudaFuncGetAttributes(&fa, paged_many_kernel<D, kPrefix, k8>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kRegsLaunch<k8>) *usable = false;
  return cudaFuncSetAttribute(paged_many_kernel<D, kPrefix, k8>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MSmem<D, k8>::kBytes);
}

}  // namespace
}  // namespace blk
