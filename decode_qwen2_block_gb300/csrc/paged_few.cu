// Attention over a paged K/V cache for few new rows per sequence (decode, or a
// few drafted tokens): at most 32 rows (token, query head of the kv head's
// group) of one sequence share a pass over its K/V.
//
//   out[r, h] = softmax(q[r, h] . K / sqrt(D)) V  over the slots row r sees,
//   [max(0, p - W + 1), p] for a row in slot p (W the window, 0 = all).
//
// Bound by memory: every K/V byte is read once for all rows of the unit.  The
// batch is ragged and its lengths live on the device, so the CTAs cut the
// line of all units' 64-slot tiles into equal ranges (see paged.h) instead of
// splitting every sequence alike: each sums the sequences' tile counts itself
// (B <= 4096 lengths), finds its range and walks it.
//   warp 4     producer: walks (kv head, sequence, tile), looks up the pages and
//              copies K and V boxes of one page (at most 64 slots, all of D) by
//              TMA with the 128-byte swizzle; the unit's q rows come with its
//              first tile as bulk copies into rows padded by 16 bytes.
//   warps 0-3  16 slots each: S = Q K^T by mma.sync m16n8k16 (the rows are the M
//              side: at most 32, a tcgen05 MMA's 128 rows would be padding),
//              the row maxima meet in shared memory, P (fp16, see kWeightLog2)
//              goes there too, and each warp forms O for its quarter of the columns
//              over all 64 slots.
//              So a unit's end needs no merge of O between warps, which with
//              short sequences would cost more than their tiles.
// Slots of a tile that no row of the unit sees (behind the last, before the
// first window, pages that were not loaded) have their V rows zeroed in shared
// memory: 0 * NaN would reach O.  Every wait is bounded.
//
// Measured with the merge, in a graph: 64 sequences of 1 - 8191 slots, 12 heads on 2
// kv heads of 128, 46 us (5.5 TB/s of 6.8 that a copy reaches); 16 of 32768 slots, 32
// heads on 2, 87 us (6.2 TB/s); 32 of 4096 with 4 - 5 tokens each (30 rows) 29 us, 22 of
// them streaming at 5.1 TB/s; 8 of 1024 8.6 us, all latency: 1.3 us until the CTA knows
// its range, 1.6 until its first tile is there, 1.5 for it, then the merge.  On the
// many-row kernel these take 70, 102, 36 and 17 us.
#include <math.h>

#include "common.cuh"
#include "paged.h"
#include "paged_dev.cuh"

namespace blk {
namespace {

constexpr int kTile = 64;            // slots of a tile
constexpr int kConsumers = 128, kThreads = 160;
// What a unit's beginning and end (q, the pieces' ends) count for in the line, in
// tiles; they lie before its first tile.  (30 rows a unit, with 0 / 1 / 2: 32.8 / 32.1 /
// 32.7 us.)
constexpr int kHead = 1;
// Weights are formed 2^14 times their size (O and l carry the factor, it cancels): fp16
// then holds them to 2^-11 of themselves down to 2^-28 of the greatest and to half of
// 2^-38 below.  Formed at their size those below 2^-14 would lose bits and those below
// 2^-25 be lost: e^-15 of one slot's weight is off by 2.6 % in every one of 32,000
// others.  The greatest, 2^14, leaves a factor 2 of room
// (see weight_plain for scores that need more).
constexpr float kWeightLog2 = 14.f;

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Box (0, 0, 0, z) at slot y of a page: all D / 64 halves of the page's slots.
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int y, int z,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(0), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void st_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}

__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error 2^-22; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  static constexpr int kKV = kTile * D * 2;                     // K or V of a tile
  static constexpr int kStages = 98304 / (2 * kKV);
  static constexpr int kQStride = D * 2 + 16;                   // bytes (conflict-free ldmatrix)
  static constexpr int kQBytes = 16 * MT * kQStride;
  static constexpr int kPStride = kTile * 2 + 16;
  static constexpr int kQOff = kStages * 2 * kKV;
  static constexpr int kPOff = kQOff + kQBytes;
  static constexpr int kStatOff = kPOff + 16 * MT * kPStride;   // [16 MT][4 warps] floats
  static constexpr int kSumOff = kStatOff + 4 * 16 * MT * 4;    // [16 MT][4 warps] floats
  static constexpr int kInfoOff = kSumOff + 4 * 16 * MT * 4;
  static constexpr int kBarOff = (kInfoOff + kStages * (int)sizeof(TileInfo) + 15) / 16 * 16;
  static constexpr int kEnd = kBarOff + (2 * kStages + 1) * 8 + 64;
  static constexpr size_t kBytes = (size_t)kEnd + 1024;         // the ring is 1024-aligned
  static_assert(kBytes + 2048 <= 233472 / 2, "two CTAs per SM");   // (1 KB the system's, statics)
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
    paged_few_kernel(const __grid_constant__ PagedAttnParams p) {
  using Sm = FSmem<D, MT>;
  constexpr int S = Sm::kStages;
  constexpr int kCPR = D / 8;           // 16-byte pieces of a row
  constexpr int kNT = D / 32;           // 8-column tiles of O per warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem), qbase = smem_u32(smem + Sm::kQOff),
                 pbase = smem_u32(smem + Sm::kPOff);
  float* stat = reinterpret_cast<float*>(smem + Sm::kStatOff);   // the warps' row maxima
  // the warps' row sums at a piece's end: apart, as a warp that has read its own goes on
  // to the next tile's maxima while others still read (the next sums are two barriers off)
  float* stat_l = reinterpret_cast<float*>(smem + Sm::kSumOff);
  volatile TileInfo* infos = reinterpret_cast<volatile TileInfo*>(smem + Sm::kInfoOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Sm::kBarOff);
  uint64_t* empty = full + S;
  uint64_t* q_empty = empty + S;
  __shared__ int64_t wsum[kThreads / 32];
  __shared__ int start_b, abort_s;
  __shared__ int64_t start_cum;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // what needs nothing of the kernels before
  if (tid == 0) {
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    mbar_init(q_empty, 4);
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
  // (the first 128 sequences go to the producer through P's place, still unused)
  PagedSeq* first_seqs = reinterpret_cast<PagedSeq*>(smem + Sm::kPOff);
  static_assert(sizeof(PagedSeq) * 128 <= 16 * MT * Sm::kPStride, "room for 128 sequences");
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

  if (warp == 4) {
    // -------------------------------------------------------------- producer
    const int bs_lg = p.page_lg < 6 ? p.page_lg : 6, bs = 1 << bs_lg;   // slots of a box
    const int boxes = kTile >> bs_lg;
    const uint32_t box_bytes = (uint32_t)bs * D * 2;
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
        if (x == xa && seg > 0 && !mbar_wait_near(q_empty, (uint32_t)(seg - 1) & 1u, p.err))
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
          const uint32_t to = ring + st * 2 * Sm::kKV + (lane < 16 ? 0 : Sm::kKV) + i * box_bytes;
          // a bad page reads as zeros: the coordinate lies behind the pool
          const int z = in ? (int)(page * p.Hkv + g) : (int)(p.n_pages * p.Hkv);
          tma_page(to, lane < 16 ? &p.tm_k : &p.tm_v, first & ((1 << p.page_lg) - 1), z,
                   &full[st]);
        }
        if (qrows > 0) wait_before();
        for (int r = lane; r < qrows; r += 32) {
          const int t = r / p.G, hh = r - t * p.G;
          bulk_g2s(smem + Sm::kQOff + r * Sm::kQStride,
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
  const int grp = lane >> 2, tig = lane & 3, mm = lane >> 3;
  const int bs_lg = p.page_lg < 6 ? p.page_lg : 6;
  const int slab = warp * 16;
  const float sl2 = p.scale_log2;
  // top: the row's maximum (log2 units) less kWeightLog2; m_r: what exponents are taken
  // against, the same but where weight_plain
  float top[MT][2], m_r[MT][2], l_r[MT][2], O[MT][kNT][4];
  int last[MT][2], low[MT][2];
  uint32_t qf[D / 16][MT][4];          // the unit's q: A fragments
  // A K or V tile is boxes [D / 64][bs slots][128 B] with the 128-byte swizzle:
  // row r, 16-byte piece c is at row_off(r) + (c / 8) half + ((c % 8 ^ r % 8) << 4).
  const int half = 128 << bs_lg;
  auto row_off = [&](int r) -> uint32_t {
    return (uint32_t)((r >> bs_lg) * (D / 64) * half + (r & ((1 << bs_lg) - 1)) * 128);
  };
  uint32_t k_off[4], v_col[kNT / 2], v_row[4];      // this lane's ldmatrix offsets
  {
    const int kr = slab + (mm >> 1) * 8 + (lane & 7);
#pragma unroll
    for (int k = 0; k < 4; ++k) k_off[k] = row_off(kr) + (((k * 2 + (mm & 1)) ^ (kr & 7)) << 4);
#pragma unroll
    for (int i = 0; i < kNT / 2; ++i) {
      const int c = warp * kNT + 2 * i + (mm >> 1);
      v_col[i] = (c >> 3) * half + (((c & 7) ^ (lane & 7)) << 4) +
                 ((mm & 1) * 8 + (lane & 7)) * 128;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v_row[k] = row_off(k * 16);
  }
  const uint32_t q_lane = qbase + ((mm & 1) * 8 + (lane & 7)) * Sm::kQStride + (mm >> 1) * 16;
  const uint32_t p_lane = pbase + ((mm & 1) * 8 + (lane & 7)) * Sm::kPStride + (mm >> 1) * 16;
  const uint32_t p_st = pbase + grp * Sm::kPStride + (slab + 2 * tig) * 2;
  for (int it = 0;; ++it) {
    const int st = it % S;
    if (!__all_sync(0xffffffffu, mbar_wait_near(&full[st], (uint32_t)(it / S) & 1u, p.err))) {
      // the wait ran out: the other warps, at the first barrier or on their way there,
      // find the flag behind it; nobody waits for this one
      if (lane == 0) *(volatile int*)&abort_s = 1;
      __threadfence_block();
      asm volatile("bar.arrive 1, %0;" ::"r"(kConsumers) : "memory");
      return;
    }
    const int flags = infos[st].flags;
    if (flags & 4) return;
    const int slot0 = infos[st].slot0, n = infos[st].n;
    const int vlo = infos[st].lo - slot0, vhi = infos[st].hi - slot0;   // seen: [vlo, vhi) of the tile
    const uint32_t kb = ring + st * 2 * Sm::kKV, vb = kb + Sm::kKV;
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
          for (int i = 0; i < kNT; ++i) O[mt][i][2 * h2] = O[mt][i][2 * h2 + 1] = 0.f;
        }
    }
    if (flags & 1) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) ldsm_x4(q_lane + mt * 16 * Sm::kQStride + ks * 32, qf[ks][mt]);
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty);       // q's place is free
    }
    const bool active = slab < vhi && slab + 16 > vlo;
    // every row sees every slot of this warp's 16: n - 1 slots from the end are
    // behind the first row, windows begin at most n - 1 slots behind vlo
    const bool clear = slab + 16 <= vhi - (n - 1) && slab >= (p.window > 0 ? vlo + (n - 1) : vlo);
    float sc[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) sc[mt][k][0] = sc[mt][k][1] = sc[mt][k][2] = sc[mt][k][3] = 0.f;
    if (active) {
      // S = Q K^T of this warp's 16 slots
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t bk[4];
        ldsm_x4(kb + k_off[ks & 3] + (ks >> 2) * half, bk);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816(sc[mt][0], qf[ks][mt], bk[0], bk[1]);
          mma16816(sc[mt][1], qf[ks][mt], bk[2], bk[3]);
        }
      }
    }
    // raw scores, -inf where the row does not see the slot; the warps' maxima meet
    if (!clear) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = slab + k * 8 + 2 * tig + (e & 1), slot = slot0 + c;
            const bool seen =
                active && c >= vlo && slot <= last[mt][e >> 1] && slot >= low[mt][e >> 1];
            if (!seen) sc[mt][k][e] = -INFINITY;
          }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        float mx = fmaxf(fmaxf(sc[mt][0][2 * h2], sc[mt][0][2 * h2 + 1]),
                         fmaxf(sc[mt][1][2 * h2], sc[mt][1][2 * h2 + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (tig == 0) stat[(mt * 16 + grp + 8 * h2) * 4 + warp] = mx;
      }
    named_sync(1, kConsumers);
    if (*(volatile int*)&abort_s) return;       // (set before a warp's arrival, see above)
    float corr[MT][2], m_new[MT][2];
    bool moved = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const int row = mt * 16 + grp + 8 * h2;
        const float4 m4 = *reinterpret_cast<const float4*>(stat + row * 4);
        const float mx = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
        const float t = fmaxf(top[mt][h2], fmaf(mx, sl2, -kWeightLog2));
        moved |= t != top[mt][h2];
        top[mt][h2] = t;
        m_new[mt][h2] = m_r[mt][h2];
      }
    if (moved) {                        // (seldom, after a unit's first tiles)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2)
          m_new[mt][h2] = weight_plain(top[mt][h2]) ? top[mt][h2] + kWeightLog2 : top[mt][h2];
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const float mn = m_new[mt][h2];
        corr[mt][h2] = mn == -INFINITY ? 1.f : ex2(m_r[mt][h2] - mn);
        m_r[mt][h2] = mn;
        const float nref = mn == -INFINITY ? 0.f : -mn;      // 2^-inf = 0
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float e0 = ex2(fmaf(sc[mt][k][2 * h2], sl2, nref));
          const float e1 = ex2(fmaf(sc[mt][k][2 * h2 + 1], sl2, nref));
          sum += e0 + e1;
          const __half2 ph = __floats2half2_rn(e0, e1);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(p_st + (mt * 16 + 8 * h2) * Sm::kPStride +
                                                      k * 16),
                       "r"(*reinterpret_cast<const uint32_t*>(&ph))
                       : "memory");
        }
        l_r[mt][h2] = l_r[mt][h2] * corr[mt][h2] + sum;
      }
    if (active && (slab < vlo || slab + 16 > vhi)) {
      for (int i = lane; i < 16 * kCPR; i += 32) {
        const int r = slab + i / kCPR, c = i % kCPR;
        if (r < vlo || r >= vhi) st_zero16(vb + row_off(r) + (c >> 3) * half + (((c & 7) ^ (r & 7)) << 4));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before a later copy there
    }
    named_sync(1, kConsumers);
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < kNT; ++i) {
          O[mt][i][0] *= corr[mt][0];
          O[mt][i][1] *= corr[mt][0];
          O[mt][i][2] *= corr[mt][1];
          O[mt][i][3] *= corr[mt][1];
        }
    }
    // O += P V for this warp's D / 4 columns
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks * 16 >= vhi || ks * 16 + 16 <= vlo) continue;
      uint32_t bv[kNT / 2][4];
#pragma unroll
      for (int i = 0; i < kNT / 2; ++i) ldsm_x4_t(vb + v_row[ks] + v_col[i], bv[i]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t a[4];
        ldsm_x4(p_lane + mt * 16 * Sm::kPStride + ks * 32, a);
#pragma unroll
        for (int i = 0; i < kNT / 2; ++i) {
          mma16816(O[mt][2 * i], a, bv[i][0], bv[i][1]);
          mma16816(O[mt][2 * i + 1], a, bv[i][2], bv[i][3]);
        }
      }
    }
    if (flags & 2) {
      // the piece's end: the warps' sums of l meet, then rows go out
      const int rows = n * p.G, r0 = infos[st].r0, g = infos[st].g, dst = infos[st].dst;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          float l = l_r[mt][h2];
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          if (tig == 0) stat_l[(mt * 16 + grp + 8 * h2) * 4 + warp] = l;
        }
      named_sync(1, kConsumers);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const int row = mt * 16 + grp + 8 * h2;
          if (row >= rows) continue;
          const float4 l4 = *reinterpret_cast<const float4*>(stat_l + row * 4);
          const float l = (l4.x + l4.y) + (l4.z + l4.w);
          const int t = row / p.G, hq = g * p.G + (row - t * p.G);
          const int col = warp * (D / 4) + 2 * tig;
          if (dst < 0 && !p.own) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            __half* o = p.out + (int64_t)(r0 + t) * p.out_stride + (int64_t)hq * D + col;
#pragma unroll
            for (int i = 0; i < kNT; ++i)
              *reinterpret_cast<__half2*>(o + i * 8) =
                  __floats2half2_rn(O[mt][i][2 * h2] * inv, O[mt][i][2 * h2 + 1] * inv);
          } else {
            const int64_t at = dst < 0 ? (int64_t)(r0 + t) * p.Hq + hq
                                       : ((int64_t)cta * 2 + dst) * p.slot_rows + row;
            float* o = (dst < 0 ? p.own : p.part) + at * D + col;
#pragma unroll
            for (int i = 0; i < kNT; ++i)
              *reinterpret_cast<float2*>(o + i * 8) =
                  make_float2(O[mt][i][2 * h2], O[mt][i][2 * h2 + 1]);
            if (warp == 0 && tig == 0)
              (dst < 0 ? p.own_ml : p.ml)[at] = make_float2(m_r[mt][h2], l);
          }
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
}

// ------------------------------------------------------------------- merging
// A row's result from its pieces: sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c
// with M = max_c m_c, pieces in their order.  kWPR warps take a row, each a run of
// its pieces (their sums are added in order, so the bits do not depend on
// timing): eight where few rows have many pieces (one long sequence alone is cut
// into 150), one where many rows have a few.  Bound by latency: the pieces' places,
// then the pieces, a round trip each.  The attention with one / two / eight warps a
// row (a row's entry searched for in each): 96 rows of 16 pieces 14.2 / 10.7 / 10.3 us,
// 768 rows 48.9 / 48.3 / 49.7, 32000 rows of two (39 MB) 80 / 90 / 127.
template <int D, int kWPR, bool kByUnit>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedMergeParams q) {
  // a row's lanes: half a warp where rows are many (two rows' pieces in flight per warp)
  constexpr int kLanes = kWPR == 1 ? 16 : 32, kV = D / kLanes;     // columns per lane
  const PagedAttnParams& p = q.a;
  __shared__ float sacc[kWPR > 1 ? 8 : 1][D + 2];
  __shared__ int cut_row[kByUnit ? 1 : 512], wsum[8];
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = (lane % kLanes) * kV;
  // With a prefix the blocks share all rows and heads.  Else they share the rows of the
  // cut units: where there is an entry for every unit, blockIdx.x is one and the blocks
  // of a column share its rows; else they share the rows of the CTAs' entries together
  // (a CTA's entry a column left most blocks without work: 512 tokens 28.4 -> 30.7 us;
  // finding a row's entry took 64 decoding sequences from 45.9 to 47.5, 512 tokens from
  // 27.0 to 27.8).
  PagedPiece u = {};
  int64_t items, b0 = blockIdx.x, nb = gridDim.x;
  if constexpr (kByUnit) {
    u = p.cut[blockIdx.x];
    // (an attention that timed out may have left its entry as it was)
    const bool cut = u.c0 >= 0 && u.c0 <= u.c1 && u.c1 < p.nc && u.rows > 0 &&
                     u.rows <= p.slot_rows && u.r0 >= 0 && u.r0 <= p.N - u.rows / p.G &&
                     u.g >= 0 && u.g < p.Hkv;
    items = cut ? u.rows : 0;
    b0 = blockIdx.y;
    nb = gridDim.y;
  } else if (q.prefix) {
    items = (int64_t)p.N * p.Hq;
  } else {
    // rows of the cut units before each CTA's (two CTAs a thread; nc <= 512)
    int n2[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = 2 * tid + k;
      if (i < p.nc) {
        const int2 h = *reinterpret_cast<const int2*>(&p.cut[i]);     // c0, rows
        n2[k] = h.x >= 0 ? h.y : 0;
      }
    }
    int x = n2[0] + n2[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) x += wsum[w];
      all += wsum[w];
    }
    cut_row[2 * tid] = x - n2[0] - n2[1];
    cut_row[2 * tid + 1] = x - n2[1];
    __syncthreads();
    items = all;
  }
  constexpr int kRows = 256 / kLanes / kWPR;  // rows of a block at a time
  for (int64_t item0 = b0 * kRows; item0 < items; item0 += nb * kRows) {
    const int64_t item = item0 + tid / kLanes / kWPR;
    bool here = item < items;                 // (a block's warps stay together: barriers below)
    if (kWPR == 1 && !here) break;
    // pieces: own ones in slots of CTAs c0..c1 (or a whole one), then the prefix's
    int c0 = 0, c1 = 0, row = 0, r = 0, hq = 0, pc0 = 0, pc1 = -1, prow = 0;
    bool own_whole = false, pre_whole = false;
    if (kByUnit || !q.prefix) {
      int i = (int)item;             // row of the unit
      if constexpr (!kByUnit) {
        int lo = 0, hi = p.nc;
        while (hi - lo > 1) {        // (an item behind the last takes no piece)
          const int mid = (lo + hi) >> 1;
          if (cut_row[mid] <= i) lo = mid; else hi = mid;
        }
        u = p.cut[lo];
        i -= cut_row[lo];
      }
      const int tl = i / p.G, hh = i - tl * p.G;
      c0 = u.c0;
      c1 = u.c1;
      row = q.own_btok ? tl / q.own_btok * 128 + tl % q.own_btok * p.G + hh : i;
      r = u.r0 + tl;
      hq = u.g * p.G + hh;
    } else {
      r = (int)(item / p.Hq);
      hq = (int)(item - (int64_t)r * p.Hq);
      const int g = hq / p.G, hh = hq - g * p.G;
      const int4 f = here ? p.row_info[(int64_t)r * p.Hkv + g] : make_int4(-2, 0, 0, 0);
      // (else a row behind the batch, or refused)
      here = paged_row_part(f.x, f.y, f.w, p.nc, p.slot_rows, p.G);
      if (kWPR == 1 && !here) continue;
      own_whole = f.x == -1;
      c0 = f.x;
      c1 = f.y;
      row = f.w + hh;
      // the prefix's unit of this row: pre_tok tokens in blocks of pre_btok
      const int u = r / q.pre_tok, tl = r - u * q.pre_tok;
      const int64_t w = q.pre_tiles + kPagedManyHead;
      const int64_t ue = ((int64_t)g * q.pre_units + u + 1) * w, T = p.Hkv * q.pre_units * w;
      const int64_t x0 = (ue - q.pre_tiles + 1) * q.pre_nc - 1, x1 = ue * q.pre_nc - 1;
      if (T * q.pre_nc < ((int64_t)1 << 31)) {       // (a 64-bit division takes 100 clocks)
        pc0 = (int)x0 / (int)T;
        pc1 = (int)x1 / (int)T;
      } else {
        pc0 = (int)(x0 / T);
        pc1 = (int)(x1 / T);
      }
      pre_whole = pc0 == pc1;
      prow = tl / q.pre_btok * 128 + tl % q.pre_btok * p.G + hh;
    }
    const int n_own = own_whole ? 1 : c1 - c0 + 1;
    const int n_all = !here ? 0 : n_own + (!kByUnit && q.prefix ? pc1 - pc0 + 1 : 0);
    auto piece = [&](int i, const float*& o, float2& ml) {
      if (kByUnit || i < n_own) {
        const int64_t at = own_whole ? (int64_t)r * p.Hq + hq
                                     : ((int64_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * p.slot_rows + row;
        o = (own_whole ? p.own : p.part) + at * D;
        ml = __ldcg((own_whole ? p.own_ml : p.ml) + at);
      } else {
        const int k = i - n_own;
        const int64_t at = pre_whole ? (int64_t)r * p.Hq + hq
                                     : ((int64_t)(pc0 + k) * 2 + (k == 0 ? 1 : 0)) * q.pre_rows + prow;
        o = (pre_whole ? q.pre_own : q.pre_part) + at * D;
        ml = __ldcg((pre_whole ? q.pre_own_ml : q.pre_ml) + at);
      }
    };
    const int wr = warp % kWPR;
    const int i0 = wr * n_all / kWPR, i1 = (wr + 1) * n_all / kWPR;
    float M = -INFINITY, l = 0.f, acc[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) acc[k] = 0.f;
    constexpr int kU = 4;                     // pieces' loads in flight (8: fewer warps fit, slower)
    for (int i = i0; i < i1; i += kU) {
      float v[kU][kV];
      float2 ml[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        ml[u] = make_float2(-INFINITY, 0.f);
        if (i + u < i1) {
          const float* o;
          piece(i + u, o, ml[u]);
          if constexpr (kV == 2) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(o + c));
            v[u][0] = x.x; v[u][1] = x.y;
          } else {
#pragma unroll
            for (int e = 0; e < kV; e += 4) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(o + c + e));
              v[u][e] = x.x; v[u][e + 1] = x.y; v[u][e + 2] = x.z; v[u][e + 3] = x.w;
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (ml[u].y == 0.f) continue;         // nothing seen there (a sum of NaN goes on)
        const float mn = fmaxf(M, ml[u].x);
        const float so = M == -INFINITY ? 0.f : exp2f(M - mn), w = exp2f(ml[u].x - mn);
        l = __fmaf_rn(w, ml[u].y, __fmul_rn(l, so));
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[k] = __fmaf_rn(w, v[u][k], __fmul_rn(acc[k], so));
        M = mn;
      }
    }
    if constexpr (kWPR > 1) {
      __syncthreads();                        // sacc of the rows before is read
      if (here) {
#pragma unroll
        for (int k = 0; k < kV; ++k) sacc[warp][c + k] = acc[k];
        if (lane == 0) {
          sacc[warp][D] = M;
          sacc[warp][D + 1] = l;
        }
      }
      __syncthreads();
      if (wr != 0 || !here) continue;
      M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWPR; ++k) M = fmaxf(M, sacc[warp + k][D]);
      l = 0.f;
#pragma unroll
      for (int k = 0; k < kV; ++k) acc[k] = 0.f;
#pragma unroll
      for (int k = 0; k < kWPR; ++k) {
        const float mg = sacc[warp + k][D];
        const float w = mg == -INFINITY ? 0.f : exp2f(mg - M);
        l = __fmaf_rn(w, sacc[warp + k][D + 1], l);
#pragma unroll
        for (int e = 0; e < kV; ++e) acc[e] = __fmaf_rn(w, sacc[warp + k][c + e], acc[e]);
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __half* d = p.out + (int64_t)r * p.out_stride + (int64_t)hq * D + c;
#pragma unroll
    for (int k = 0; k < kV; k += 2)
      *reinterpret_cast<__half2*>(d + k) = __floats2half2_rn(acc[k] * inv, acc[k + 1] * inv);
  }
}

template <int D, int MT>
cudaError_t launch_few(const PagedAttnParams& p, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.nc);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = FSmem<D, MT>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_few_kernel<D, MT>, p);
}

template <int D, int MT>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(paged_few_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)FSmem<D, MT>::kBytes);
}

}  // namespace

bool paged_few_rows(int G, int64_t max_new) { return max_new * G <= kPagedFewRows; }

void paged_few_slots(int num_sms, int G, int64_t max_new, int* nc, int* slot_rows) {
  *nc = 2 * num_sms;
  *slot_rows = max_new * G <= 16 ? 16 : 32;
}

cudaError_t launch_paged_few(const PagedAttnParams& p, cudaStream_t s, bool pdl) {
  if (p.max_new * p.G > p.slot_rows || p.nc < 1 || p.nc > 512) return cudaErrorInvalidValue;
  const int mt = p.slot_rows / 16;
  if (p.D == 128)
    return mt == 1 ? launch_few<128, 1>(p, s, pdl) : launch_few<128, 2>(p, s, pdl);
  if (p.D == 64)
    return mt == 1 ? launch_few<64, 1>(p, s, pdl) : launch_few<64, 2>(p, s, pdl);
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_merge(const PagedMergeParams& p, int num_sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // Rows to merge, at most: with a prefix every row, else those of the units that can be
  // cut, each in an entry of its own.  The fewer they are, the more warps take one
  // (figures at the kernel); the grid has few CTAs that find nothing to do, as those
  // still have to come and go.
  const PagedAttnParams& a = p.a;
  const bool few = a.slot_rows <= kPagedFewRows;
  const int64_t entries = a.upb ? (int64_t)a.B * a.Hkv * a.upb : a.nc, all = (int64_t)a.N * a.Hq;
  const int64_t rows = few ? a.max_new * a.G : a.slot_rows;          // of a unit
  const int64_t cut = p.prefix || entries * rows > all ? all : entries * rows;
  const int wpr = cut > 16 * num_sms ? 1 : cut > 4 * num_sms ? 2 : 8;
  const int64_t per = wpr == 1 ? 16 : 8 / wpr;
  if (a.upb) {
    cfg.gridDim = dim3((unsigned)entries, (unsigned)((rows + per - 1) / per));
  } else {
    const int64_t want = (cut + per - 1) / per, fit = (int64_t)num_sms * 8;
    cfg.gridDim = dim3((unsigned)(want < fit ? want : fit));
  }
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int d = a.D == 128, v = wpr == 1 ? 0 : wpr == 2 ? 1 : 2;
  if (a.upb) {
    void (*const k[2][3])(PagedMergeParams) = {
        {paged_merge_kernel<64, 1, true>, paged_merge_kernel<64, 2, true>,
         paged_merge_kernel<64, 8, true>},
        {paged_merge_kernel<128, 1, true>, paged_merge_kernel<128, 2, true>,
         paged_merge_kernel<128, 8, true>}};
    return cudaLaunchKernelEx(&cfg, k[d][v], p);
  }
  void (*const k[2][3])(PagedMergeParams) = {
      {paged_merge_kernel<64, 1, false>, paged_merge_kernel<64, 2, false>,
       paged_merge_kernel<64, 8, false>},
      {paged_merge_kernel<128, 1, false>, paged_merge_kernel<128, 2, false>,
       paged_merge_kernel<128, 8, false>}};
  return cudaLaunchKernelEx(&cfg, k[d][v], p);
}

cudaError_t configure_paged_few() {
  cudaError_t e = configure_one<128, 1>();
  if (e == cudaSuccess) e = configure_one<128, 2>();
  if (e == cudaSuccess) e = configure_one<64, 1>();
  if (e == cudaSuccess) e = configure_one<64, 2>();
  return e;
}

}  // namespace blk
