// Attention over a paged K/V cache in 8 bits (kv8.h) for few new rows per sequence: at
// most 32 rows (token, query head of the kv head's group) of one sequence share a pass
// over its codes.  The batch, the line of tiles that the CTAs share evenly, units, pieces
// and their merge are those of paged_few.cu; K and V become fp16 in registers, exactly.
//
//   out[r, h] = softmax(q[r, h] . K / sqrt(D)) V  over the slots row r sees
//
// Bound by memory and by issue: D + D / 32 bytes a row of K or V, and for each pair of
// codes a byte permute, a subtraction and a product before mma.sync can take them.
//   warp 4     producer: codes and scales, page by page (at most 64 slots), by TMA.
//   warps 0-3  16 slots each of every 64-slot tile: S = Q K^T, the warp's own running
//              maximum and sum, O = P V of all columns.  Nothing is exchanged between
//              warps until the unit ends (the weights' fragments are the scores' own), so
//              a warp waits for no other while tiles come.
// A lane's codes are wide loads because the MMA's inner index may run over the columns in
// any order if q's does too: lane (grp, tig) takes 16-byte pieces tig (and tig + 4) of its
// slot's row, whose j-th four codes are inner indexes 2 tig, 2 tig + 1, 2 tig + 8,
// 2 tig + 9 of product j.  For V the inner index is the slot and the lane's four are
// words of four columns each; two permutes a pair of words bring equal columns together.
// Slots are dealt to the scores' columns so that neither read meets bank conflicts.
// A slot that no row sees has its V scale taken as 0, so its codes count for nothing.
#include <math.h>

#include "common.cuh"
#include "kv8.cuh"
#include "paged_dev.cuh"

namespace blk {
namespace {

constexpr int kTile = 64;            // slots of a tile
constexpr int kWarps = 4, kConsumers = 32 * kWarps, kThreads = kConsumers + 32;
constexpr int kHead = 1;             // a unit's begin and end in the line, in tiles
constexpr float kWeightLog2 = 14.f;  // weights are formed 2^14 times their size (see paged_few.cu)

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// The scales of a slot: D / 32 bytes.
template <int NB>
__device__ __forceinline__ uint32_t lds_scales(uint32_t addr) {
  if constexpr (NB == 4) return lds32(addr);
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
// Codes of a page: (0, y, z), all columns of some slots.
__device__ __forceinline__ void tma_codes(uint32_t dst, const CUtensorMap* map, int y, int z,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// The scales of a page that is not there (a box's, at most).
__device__ const uint4 kZeroScales[kTile * 4 / 16] = {};
__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error 2^-22; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ __half2 unit_of_bits(uint32_t h) {   // s / 64 of two fp16 s
  return __hmul2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(1.f / 64.f));
}

struct TileInfo {      // what the consumers need of a tile
  int slot0;           // its first slot
  int lo, hi;          // slots that some row of the unit sees: [lo, hi)
  int L, n;            // the unit's history and new tokens
  int r0, g;           // its first batch row, its kv head
  int flags;           // 1 first tile of the piece, 2 last, 4 end of the CTA's range
  int dst;             // -1 the whole unit, else the partial slot
};

template <int D, int MT>
struct FSmem {
  static constexpr int NB = D / kKv8Block;
  static constexpr int kKV = kTile * D;                         // K or V codes of a tile
  static constexpr int kSc = kTile * NB;                        // their scales
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kQStride = D * 2 + 16;                   // bytes (conflict-free reads)
  static constexpr int kQBytes = 16 * MT * kQStride;
  static constexpr int kQBufs = MT;                             // two row tiles re-read q for every tile
  static constexpr int kXBytes = 3 * NB * 16 * 32 * 4;          // a unit's end: O on its way
  static constexpr int kScOff = kStages * 2 * kKV;
  static constexpr int kQOff = kScOff + kStages * 2 * kSc;
  static constexpr int kXOff = kQOff + kQBufs * kQBytes;
  static constexpr int kStatOff = kXOff + kXBytes;              // [16 MT][4 warps] maxima, then sums
  static constexpr int kInfoOff = kStatOff + 2 * 4 * 16 * MT * 4;
  static constexpr int kBarOff = (kInfoOff + kStages * (int)sizeof(TileInfo) + 15) / 16 * 16;
  static constexpr int kEnd = kBarOff + (2 * kStages + kQBufs) * 8 + 64;
  static constexpr size_t kBytes = (size_t)kEnd + 1024;         // the ring is 1024-aligned
  static_assert(kBytes + 3072 <= 233472 / 2, "two CTAs per SM");   // (1 KB the system's, statics)
};

__device__ __forceinline__ int seq_tiles(const PagedAttnParams& p, const PagedSeq& s) {
  if (s.n == 0) return 0;
  return (s.L + s.n + kTile - 1) / kTile - paged_lo(p, s.L) / kTile;
}
__device__ __forceinline__ int seq_weight(const PagedAttnParams& p, const PagedSeq& s) {
  return s.n == 0 ? 0 : seq_tiles(p, s) + kHead;
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 2)
    paged_few_kv8_kernel(const __grid_constant__ PagedFew8Params q8) {
  using Sm = FSmem<D, MT>;
  constexpr int S = Sm::kStages, NB = Sm::NB;
  const PagedAttnParams& p = q8.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem), sring = smem_u32(smem + Sm::kScOff),
                 qbase = smem_u32(smem + Sm::kQOff), xbase = smem_u32(smem + Sm::kXOff);
  float* stat_m = reinterpret_cast<float*>(smem + Sm::kStatOff);
  float* stat_l = stat_m + 4 * 16 * MT;
  volatile TileInfo* infos = reinterpret_cast<volatile TileInfo*>(smem + Sm::kInfoOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Sm::kBarOff);
  uint64_t* empty = full + S;
  uint64_t* q_empty = empty + S;
  __shared__ int64_t wsum[kThreads / 32];
  __shared__ int start_b, abort_s;
  __shared__ int64_t start_cum;
  __shared__ PagedSeq first_seqs[128];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // what needs nothing of the kernels before
  if (tid == 0) {
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    for (int s = 0; s < Sm::kQBufs; ++s) mbar_init(&q_empty[s], kWarps);
    fence_mbar_init();
    start_b = 0;
    start_cum = 0;
    abort_s = 0;
  }
  // (early: the producer waits, before q and the new slots)
  if (!p.early) {
    griddep_wait();
    griddep_launch();
  }
  // tiles of all sequences (one kv head), and those before this thread's
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int64_t mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const PagedSeq s = load_seq(p, b);
    mine += seq_weight(p, s);
    bad |= s.bad;
    if (b < 128) first_seqs[b] = s;
    if (p.upb && s.n == 0 && blockIdx.x == 0)
      for (int g = 0; g < p.Hkv; ++g) p.cut[g * p.B + b].c0 = -1;
  }
  if (bad && blockIdx.x == 0) set_error(p.err, kDevPage);
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int64_t before = 0, T1 = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += wsum[w];
    T1 += wsum[w];
  }
  before += inc - mine;
  const int64_t T = T1 * p.Hkv;
  const int nc = (int)(T < p.nc ? (T < 1 ? 1 : T) : p.nc);
  const int cta = blockIdx.x;
  const int64_t t0 = cta < nc ? range_of(T, cta, nc) : T, t1 = cta < nc ? range_of(T, cta + 1, nc) : T;
  if (t0 >= t1) {   // (uniform over the CTA)
    if (p.early) {
      griddep_wait();
      griddep_launch();
    }
    if (tid == 0 && !p.upb) p.cut[cta].c0 = -1;
    return;
  }
  const int g0 = small_div(t0, T1);
  const int64_t x0 = t0 - g0 * T1;
  if (mine > 0 && before <= x0 && x0 < before + mine) {
    int64_t cum = before;
    int b = b0;
    for (; b + 1 < b1; ++b) {
      const int wt = seq_weight(p, load_seq(p, b));
      if (x0 < cum + wt) break;
      cum += wt;
    }
    start_b = b;
    start_cum = cum;
  }
  __syncthreads();

  if (warp == kWarps) {
    // -------------------------------------------------------------- producer
    const int bs_lg = p.page_lg < 6 ? p.page_lg : 6, bs = 1 << bs_lg;   // slots of a box
    const int boxes = kTile >> bs_lg;
    const uint32_t box_bytes = (uint32_t)bs * (D + NB);
    int b = start_b, g = g0;
    int64_t cum = start_cum, lin = t0;
    int it = 0, seg = 0, base32 = -1;
    PagedSeq mys = {};
    bool ok = true, waited = !p.early;
    auto wait_before = [&] {           // for what the kernel before this one writes
      if (!waited) {
        griddep_wait();
        griddep_launch();
        waited = true;
      }
    };
    PagedPiece cut = {-1, 0, 0, 0, 0};
    while (lin < t1 && ok) {
      if (b >= p.B) {        // the next kv head begins again with the first sequence
        b = 0;
        cum = 0;
        ++g;
      }
      if ((b & ~31) != base32) {
        base32 = b & ~31;
        if (it == 0 && seg == 0 && base32 < 128) mys = base32 + lane < p.B ? first_seqs[base32 + lane] : PagedSeq{};
        else if (base32 + lane < p.B) mys = load_seq(p, base32 + lane);
        else mys = PagedSeq{};
      }
      PagedSeq s;
      s.r0 = __shfl_sync(0xffffffffu, mys.r0, b & 31);
      s.n = __shfl_sync(0xffffffffu, mys.n, b & 31);
      s.L = __shfl_sync(0xffffffffu, mys.L, b & 31);
      const int nt = seq_tiles(p, s);
      if (nt == 0) {
        ++b;
        continue;
      }
      const int64_t us = (int64_t)g * T1 + cum;      // the unit's first tile in the line
      const int64_t ue = us + kHead + nt;
      const int xa = (int)max((int64_t)0, lin - us - kHead);
      const int xb = (int)min((int64_t)nt, t1 - us - kHead);
      lin = ue;
      cum += nt + kHead;
      if (xb <= xa) {        // its head alone lies here
        ++b;
        continue;
      }
      const bool whole = xa == 0 && xb == nt;
      const int dst = whole ? -1 : (xa == 0 ? 1 : 0);
      if (xa == 0) {
        const int c1 = whole ? cta : cta_of(T, ue - 1, nc);
        const PagedPiece now = {whole ? -1 : cta, s.n * p.G, c1, s.r0, g};
        if (!whole) cut = now;
        if (p.upb && lane == 0) p.cut[g * p.B + b] = now;
        if (p.row_info)
          for (int t = lane; t < s.n; t += 32)
            p.row_info[(int64_t)(s.r0 + t) * p.Hkv + g] =
                make_int4(whole ? -1 : cta, c1, 0, t * p.G);
      }
      const int lo = paged_lo(p, s.L), hi = s.L + s.n, j0 = lo / kTile;
      const int32_t* row = p.table + (int64_t)b * p.max_blocks;
      for (int x = xa; x < xb; ++x, ++it) {
        const int st = it % S;
        const int slot0 = (j0 + x) * kTile;
        // box i of the tile: slots slot0 + i * bs ..; lanes 0-15 take K, 16-31 V
        const int i = lane & 15, first = slot0 + (i << bs_lg);
        const bool take = i < boxes && first < hi && first + bs > lo;
        int64_t page = -1;
        if (take) page = (first < p.pre_here ? p.prefix_pages : row)[first >> p.page_lg];
        const bool in = page >= 0 && page < p.n_pages;
        if (take && !in) set_error(p.err, kDevPage);
        if (it >= S && !mbar_wait_near(&empty[st], (uint32_t)(it / S - 1) & 1u, p.err)) ok = false;
        constexpr int Q = Sm::kQBufs;
        if (x == xa && seg >= Q && !mbar_wait_near(&q_empty[seg % Q], (uint32_t)(seg / Q - 1) & 1u, p.err))
          ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const unsigned m = __ballot_sync(0xffffffffu, take);
        const int qrows = x == xa ? s.n * p.G : 0;
        if (lane == 0) {
          volatile TileInfo& f = infos[st];
          f.slot0 = slot0;
          f.lo = lo;
          f.hi = hi;
          f.L = s.L;
          f.n = s.n;
          f.r0 = s.r0;
          f.g = g;
          f.flags = (x == xa ? 1 : 0) | (x == xb - 1 ? 2 : 0);
          f.dst = dst;
          mbar_arrive_expect_tx(&full[st], __popc(m) * box_bytes + qrows * D * 2);
        }
        if (slot0 + kTile > s.L) wait_before();
        __syncwarp();
        if (take) {
          const int v = lane >> 4, y = first & ((1 << p.page_lg) - 1);
          // a bad page reads as zeros: the coordinate lies behind the pool
          const int z = in ? (int)(page * p.Hkv + g) : (int)(p.n_pages * p.Hkv);
          tma_codes(ring + (st * 2 + v) * Sm::kKV + (i << bs_lg) * D, v ? &p.tm_v : &p.tm_k, y, z,
                    &full[st]);
          // (not by a tensor map: a box of those would have to lie at 128 bytes here)
          const uint8_t* sc = (v ? q8.vs : q8.ks) + (((int64_t)z << p.page_lg) + y) * NB;
          bulk_g2s(smem + Sm::kScOff + (st * 2 + v) * Sm::kSc + (i << bs_lg) * NB,
                   in ? sc : reinterpret_cast<const uint8_t*>(kZeroScales), bs * NB, &full[st]);
        }
        if (qrows > 0) wait_before();
        for (int r = lane; r < qrows; r += 32) {
          const int t = r / p.G, hh = r - t * p.G;
          bulk_g2s(smem + Sm::kQOff + (seg % Q) * Sm::kQBytes + r * Sm::kQStride,
                   p.q + (int64_t)(s.r0 + t) * p.q_stride + (int64_t)(g * p.G + hh) * D, D * 2,
                   &full[st]);
        }
      }
      ++b;
      ++seg;
    }
    wait_before();                     // (a range of heads alone has no tile)
    if (lane == 0 && !p.upb) {
      if (!ok) cut.c0 = -1;
      p.cut[cta] = cut;
    }
    const int st = it % S;
    if (ok && it >= S && !mbar_wait_near(&empty[st], (uint32_t)(it / S - 1) & 1u, p.err)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      if (lane == 0) {
        infos[st].flags = 4;
        mbar_arrive(&full[st]);
      }
    } else {
      // copies in flight land before shared memory goes away
      for (int k = max(0, it - S); k < it; ++k)
        mbar_wait(&full[k % S], (uint32_t)(k / S) & 1u, nullptr);
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  const int grp = lane >> 2, tig = lane & 3;
  const int slab = warp * 16;
  const float sl2 = p.scale_log2;
  // The slot (of 8) behind column c of a score tile.  With rows of 128 bytes and the
  // 128-byte swizzle rows 0 - 3 and 4 - 7 have a piece in different halves, so columns
  // 2 i, 2 i + 1 are slots i, i + 4; rows of 64 bytes alternate by themselves.
  auto slot_of = [](int c) { return D == 128 ? (c >> 1) | ((c & 1) << 2) : c; };
  auto row_sw = [](int r) { return D == 128 ? r & 7 : (r >> 1) & 3; };
  const int kr = slab + slot_of(grp);                 // + 8 t: K row of the lane's column
  const uint32_t k_off = kr * D + ((tig ^ row_sw(kr)) << 4);      // (^ 64: piece tig + 4)
  const int se = slab + slot_of(2 * tig), so = slab + slot_of(2 * tig + 1);   // V rows, + 8 p
  // lanes of odd tig read the odd slot first: their rows' pieces then lie elsewhere
  const int r_a = tig & 1 ? so : se, r_b = tig & 1 ? se : so;
  const uint32_t va_off = r_a * D + ((((grp >> 2) ^ row_sw(r_a))) << 4) + (grp & 3) * 4;
  const uint32_t vb_off = r_b * D + ((((grp >> 2) ^ row_sw(r_b))) << 4) + (grp & 3) * 4;
  const uint32_t sel_lo = tig & 1 ? 0x1504 : 0x5140, sel_hi = tig & 1 ? 0x3726 : 0x7362;
  // a K piece's block of 32 columns, as a permute that doubles its scale's byte to fp16
  const uint32_t kb = tig >> 1, sel_k0 = kb << 12 | 4 << 8 | kb << 4 | 4, sel_k1 = sel_k0 + 0x2020;
  const uint32_t q_lane = qbase + grp * Sm::kQStride + tig * 32;
  // top: the row's maximum (log2 units) less kWeightLog2; m_r: what exponents are taken
  // against, the same but where weight_plain
  float top[MT][2], m_r[MT][2], l_r[MT][2], O[MT][NB * 4][4];
  int last[MT][2], low[MT][2];
  uint32_t qf[MT == 1 ? D / 16 : 1][4];               // the unit's q, if there is room for it
  // q's A fragments of products 2 x, 2 x + 1 (x < D / 32) of row tile mt
  auto load_q = [&](uint32_t qb, int mt, int x, uint32_t* a, uint32_t* b) {
    const uint32_t at = qb + mt * 16 * Sm::kQStride + (x >> 1) * 128 + (x & 1) * 16;
    const uint4 u = lds128(at), w = lds128(at + 8 * Sm::kQStride);
    a[0] = u.x; a[1] = w.x; a[2] = u.y; a[3] = w.y;
    b[0] = u.z; b[1] = w.z; b[2] = u.w; b[3] = w.w;
  };
  int seg = 0;
  for (int it = 0;; ++it) {
    const int st = it % S;
    if (!__all_sync(0xffffffffu, mbar_wait_near(&full[st], (uint32_t)(it / S) & 1u, p.err))) {
      // the wait ran out: the other warps, at the next unit's end or on their way there,
      // find the flag behind its barrier; nobody waits for this one
      if (lane == 0) *(volatile int*)&abort_s = 1;
      __threadfence_block();
      asm volatile("bar.arrive 1, %0;" ::"r"(kConsumers) : "memory");
      return;
    }
    const int flags = infos[st].flags;
    if (flags & 4) return;
    const int slot0 = infos[st].slot0, n = infos[st].n;
    const int vlo = infos[st].lo - slot0, vhi = infos[st].hi - slot0;   // seen: [vlo, vhi) of the tile
    const uint32_t kt = ring + st * 2 * Sm::kKV, vt = kt + Sm::kKV;
    const uint32_t ks = sring + st * 2 * Sm::kSc, vs = ks + Sm::kSc;
    const uint32_t qb = q_lane + (seg % Sm::kQBufs) * Sm::kQBytes;
    if (flags & 1) {
      const int L = infos[st].L;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const int row = mt * 16 + grp + 8 * h2;
          last[mt][h2] = L + min(row / p.G, n - 1);
          low[mt][h2] = paged_window(p, last[mt][h2]);
          top[mt][h2] = m_r[mt][h2] = -INFINITY;
          l_r[mt][h2] = 0.f;
#pragma unroll
          for (int i = 0; i < NB * 4; ++i) O[mt][i][2 * h2] = O[mt][i][2 * h2 + 1] = 0.f;
        }
      if constexpr (MT == 1) {
#pragma unroll
        for (int x = 0; x < D / 32; ++x) load_q(qb, 0, x, qf[2 * x], qf[2 * x + 1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[0]);       // q's place is free
      }
    }
    if (slab < vhi && slab + 16 > vlo) {
      // every row sees every slot of this warp's 16: n - 1 slots from the end are
      // behind the first row, windows begin at most n - 1 slots behind vlo
      const bool clear = slab + 16 <= vhi - (n - 1) && slab >= (p.window > 0 ? vlo + (n - 1) : vlo);
      float sc[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int t = 0; t < 2; ++t) sc[mt][t][0] = sc[mt][t][1] = sc[mt][t][2] = sc[mt][t][3] = 0.f;
      const uint32_t w0 = lds_scales<NB>(ks + kr * NB), w1 = lds_scales<NB>(ks + (kr + 8) * NB);
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint4 c0 = lds128(kt + (k_off ^ (h << 6))), c1 = lds128(kt + (k_off ^ (h << 6)) + 8 * D);
        const uint32_t cw[2][4] = {{c0.x, c0.y, c0.z, c0.w}, {c1.x, c1.y, c1.z, c1.w}};
        const uint32_t sel = h ? sel_k1 : sel_k0;
        const __half2 u[2] = {unit_of_bits(__byte_perm(w0, 0, sel)), unit_of_bits(__byte_perm(w1, 0, sel))};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t qa[MT][2][4];
          if constexpr (MT > 1) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) load_q(qb, mt, 2 * h + x, qa[mt][0], qa[mt][1]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t b0 = kv8_pair(cw[t][2 * x + y], 0x4140, u[t]);
              const uint32_t b1 = kv8_pair(cw[t][2 * x + y], 0x4342, u[t]);
              if constexpr (MT == 1) {
                mma16816(sc[0][t], qf[4 * h + 2 * x + y], b0, b1);
              } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma16816(sc[mt][t], qa[mt][y], b0, b1);
              }
            }
        }
      }
      if (!clear) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = (e & 1 ? so : se) + 8 * t, slot = slot0 + c;
              const bool seen = c >= vlo && slot <= last[mt][e >> 1] && slot >= low[mt][e >> 1];
              if (!seen) sc[mt][t][e] = -INFINITY;
            }
      }
      float corr[MT][2], mx[MT][2];
      bool moved = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          float x = fmaxf(fmaxf(sc[mt][0][2 * h2], sc[mt][0][2 * h2 + 1]),
                          fmaxf(sc[mt][1][2 * h2], sc[mt][1][2 * h2 + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          mx[mt][h2] = fmaxf(top[mt][h2], fmaf(x, sl2, -kWeightLog2));
          moved |= mx[mt][h2] != top[mt][h2];
        }
      if (__any_sync(0xffffffffu, moved)) {       // (seldom, after a unit's first tiles)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const float t = mx[mt][h2], mn = t == top[mt][h2] ? m_r[mt][h2]
                                             : weight_plain(t) ? t + kWeightLog2 : t;
            corr[mt][h2] = mn == -INFINITY ? 1.f : ex2(m_r[mt][h2] - mn);
            top[mt][h2] = t;
            m_r[mt][h2] = mn;
            l_r[mt][h2] *= corr[mt][h2];
          }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < NB * 4; ++i) {
            O[mt][i][0] *= corr[mt][0];
            O[mt][i][1] *= corr[mt][0];
            O[mt][i][2] *= corr[mt][1];
            O[mt][i][3] *= corr[mt][1];
          }
      }
      uint32_t pa[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const float nref = m_r[mt][h2] == -INFINITY ? 0.f : -m_r[mt][h2];      // 2^-inf = 0
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float e0 = ex2(fmaf(sc[mt][t][2 * h2], sl2, nref));
            const float e1 = ex2(fmaf(sc[mt][t][2 * h2 + 1], sl2, nref));
            sum += e0 + e1;
            const __half2 ph = __floats2half2_rn(e0, e1);
            pa[mt][2 * t + h2] = *reinterpret_cast<const uint32_t*>(&ph);
          }
          l_r[mt][h2] += sum;
        }
      // O += P V
      uint32_t sw[2][2];               // scales of the even and odd slot, + 8 p
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sw[x][0] = lds_scales<NB>(vs + (se + 8 * x) * NB);
        sw[x][1] = lds_scales<NB>(vs + (so + 8 * x) * NB);
        if (slab < vlo || slab + 16 > vhi) {
          if (se + 8 * x < vlo || se + 8 * x >= vhi) sw[x][0] = 0;
          if (so + 8 * x < vlo || so + 8 * x >= vhi) sw[x][1] = 0;
        }
      }
#pragma unroll
      for (int g = 0; g < NB; ++g) {
        uint32_t lo2[2], hi2[2];
        __half2 u[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t a = lds32(vt + (va_off ^ (g << 5)) + x * 8 * D);
          const uint32_t b = lds32(vt + (vb_off ^ (g << 5)) + x * 8 * D);
          lo2[x] = __byte_perm(a, b, sel_lo);      // columns 0, 1: even and odd slot's codes
          hi2[x] = __byte_perm(a, b, sel_hi);      // columns 2, 3
          u[x] = unit_of_bits(__byte_perm(sw[x][0], sw[x][1], (4 + g) << 12 | g << 4) & 0xff00ff00u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t sel = j & 1 ? 0x4342 : 0x4140;
          const uint32_t b0 = kv8_pair(j < 2 ? lo2[0] : hi2[0], sel, u[0]);
          const uint32_t b1 = kv8_pair(j < 2 ? lo2[1] : hi2[1], sel, u[1]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mma16816(O[mt][g * 4 + j], pa[mt], b0, b1);
        }
      }
    }
    if (flags & 2) {
      // The piece's end: the warps' maxima meet, each brings its sums to the greatest,
      // and warp w < D / 32 adds all warps' O of column block w.
      const int rows = n * p.G, r0 = infos[st].r0, g = infos[st].g, dst = infos[st].dst;
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (MT > 1 && lane == 0) mbar_arrive(&q_empty[seg % Sm::kQBufs]);
      ++seg;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2)
          if (tig == 0) stat_m[(mt * 16 + grp + 8 * h2) * 4 + warp] = m_r[mt][h2];
      named_sync(1, kConsumers);
      if (*(volatile int*)&abort_s) return;       // (set before a warp's arrival, see above)
      float M[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const int row = mt * 16 + grp + 8 * h2;
          const float4 m4 = *reinterpret_cast<const float4*>(stat_m + row * 4);
          M[mt][h2] = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
          const float f = m_r[mt][h2] == -INFINITY ? 0.f : ex2(m_r[mt][h2] - M[mt][h2]);
          float l = l_r[mt][h2] * f;
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          if (tig == 0) stat_l[row * 4 + warp] = l;
#pragma unroll
          for (int i = 0; i < NB * 4; ++i) {
            O[mt][i][2 * h2] *= f;
            O[mt][i][2 * h2 + 1] *= f;
          }
        }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt > 0) named_sync(1, kConsumers);    // the first row tile's O is read
        // a lane's O of a column block: columns 8 tig .. + 7 of rows grp and grp + 8
#pragma unroll
        for (int d = 0; d < NB; ++d)
          if (d != warp) {
            const uint32_t to = xbase + (d * 3 + (warp < d ? warp : warp - 1)) * 2048;
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int row = grp + 8 * h2;
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 to + row * 128 + (((2 * tig + x) ^ (row & 7)) << 4)),
                             "f"(O[mt][d * 4][2 * h2 + x]), "f"(O[mt][d * 4 + 1][2 * h2 + x]),
                             "f"(O[mt][d * 4 + 2][2 * h2 + x]), "f"(O[mt][d * 4 + 3][2 * h2 + x])
                             : "memory");
              }
          }
        named_sync(1, kConsumers);
        if (warp >= NB) continue;
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const int row = grp + 8 * h2, urow = mt * 16 + row;
          float v[8];
#pragma unroll
          for (int s = 0; s < kWarps; ++s)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float4 f;
              if (s == warp) {
#pragma unroll
                for (int d = 0; d < NB; ++d)
                  if (d == warp)
                    f = make_float4(O[mt][d * 4][2 * h2 + x], O[mt][d * 4 + 1][2 * h2 + x],
                                    O[mt][d * 4 + 2][2 * h2 + x], O[mt][d * 4 + 3][2 * h2 + x]);
              } else {
                const uint32_t from = xbase + (warp * 3 + (s < warp ? s : s - 1)) * 2048;
                const uint4 w = lds128(from + row * 128 + (((2 * tig + x) ^ (row & 7)) << 4));
                f = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                                __uint_as_float(w.w));
              }
              if (s == 0) {
                v[4 * x] = f.x; v[4 * x + 1] = f.y; v[4 * x + 2] = f.z; v[4 * x + 3] = f.w;
              } else {
                v[4 * x] += f.x; v[4 * x + 1] += f.y; v[4 * x + 2] += f.z; v[4 * x + 3] += f.w;
              }
            }
          if (urow >= rows) continue;
          const float4 l4 = *reinterpret_cast<const float4*>(stat_l + urow * 4);
          const float l = (l4.x + l4.y) + (l4.z + l4.w);
          const int t = urow / p.G, hq = g * p.G + (urow - t * p.G);
          const int col = warp * 32 + 8 * tig;
          if (dst < 0 && !p.own) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __half2 h = __floats2half2_rn(v[2 * k] * inv, v[2 * k + 1] * inv);
              w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(p.out + (int64_t)(r0 + t) * p.out_stride + (int64_t)hq * D + col) =
                make_uint4(w[0], w[1], w[2], w[3]);
          } else {
            const int64_t at = dst < 0 ? (int64_t)(r0 + t) * p.Hq + hq
                                       : ((int64_t)cta * 2 + dst) * p.slot_rows + urow;
            float4* o = reinterpret_cast<float4*>((dst < 0 ? p.own : p.part) + at * D + col);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
            if (warp == 0 && tig == 0)
              (dst < 0 ? p.own_ml : p.ml)[at] = make_float2(M[mt][h2], l);
          }
        }
      }
      continue;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
}

template <int D, int MT>
cudaError_t launch_few(const PagedFew8Params& p, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.a.nc);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = FSmem<D, MT>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_few_kv8_kernel<D, MT>, p);
}

template <int D, int MT>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(paged_few_kv8_kernel<D, MT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FSmem<D, MT>::kBytes);
}

}  // namespace

cudaError_t launch_paged_few_kv8(const PagedFew8Params& p, cudaStream_t s, bool pdl) {
  if (p.a.max_new * p.a.G > p.a.slot_rows || p.a.nc < 1 || p.a.nc > 512) return cudaErrorInvalidValue;
  const int mt = p.a.slot_rows / 16;
  if (p.a.D == 128) return mt == 1 ? launch_few<128, 1>(p, s, pdl) : launch_few<128, 2>(p, s, pdl);
  if (p.a.D == 64) return mt == 1 ? launch_few<64, 1>(p, s, pdl) : launch_few<64, 2>(p, s, pdl);
  return cudaErrorInvalidValue;
}

cudaError_t configure_paged_few_kv8() {
  cudaError_t e = configure_one<128, 1>();
  if (e == cudaSuccess) e = configure_one<128, 2>();
  if (e == cudaSuccess) e = configure_one<64, 1>();
  if (e == cudaSuccess) e = configure_one<64, 2>();
  return e;
}

}  // namespace blk
