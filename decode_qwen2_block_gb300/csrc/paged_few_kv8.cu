// Attention over a paged K/V cache in 8 bits (kv8.h) for few new rows per sequence: at
// most 32 rows (token, query head of the kv head's group) of one sequence share a pass
// over its codes.  The batch, the line of tiles that the CTAs share evenly, units, pieces
// and their merge are those of paged_few.cu; K and V become fp16 in registers, exactly.
//
//   out[r, h] = softmax(q[r, h] . K / sqrt(D)) V  over the slots row r sees
//
// Bound by memory and by issue: D + D / 32 bytes a row of K or V, and for each pair of
// codes a byte permute and a fused multiply-add before mma.sync can take them.
//   warp 4     producer: codes page by page by TMA, scales by 16-byte copies.
//   warps 0-3  16 slots each of every 64-slot tile (32 of 128 slots where a row has 64 columns
//              and half the work): S' = K Q' (the slots are the M side, so
//              that rows come in eights), the warp's own running maximum and sum, O' = V' P'
//              of all columns.  Nothing is exchanged between warps until the unit ends,
//              so a warp waits for no other while tiles come.
// A lane's K codes are wide loads because the MMA's inner index may run over the columns in
// any order if q's does too: lane (grp, tig) takes 16-byte pieces tig (and tig + 4) of its
// slot's row, whose j-th four codes are inner indexes 2 tig, 2 tig + 1, 2 tig + 8,
// 2 tig + 9 of product j.  V's codes come transposed (ldmatrix of 16 x 16 bytes): four slots
// of a column a word.  Slots are dealt to the scores' rows so that neither read meets bank
// conflicts.
// A slot that no row sees has its V scale taken as 0, so its codes count for nothing.
//
// Measured with the merge, in a graph: 96 ragged sequences (291 MB, 6 heads a kv head) 62 us
// over pages of 16 and 59 over pages of 64 (5.0 TB/s), 8 of 131072 slots 90 us (6.1 TB/s) and
// with 16 heads a kv head 112, 24 of 5000 slots 30, 37, 45 and 55 us for 8, 16, 24 and 32 rows.
// A cold pass over the first spends 56 us here at 67 % of the memory's peak and 50 % of the
// issue slots: a warp waits for its own chain of loads, products and exponentials.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kv8.cuh"
#include "paged_dev.cuh"

namespace blk {
namespace {

constexpr int kHead = 1;             // a unit's begin and end in the line, in tiles
// Weights are rounded to fp16, mma.sync's type for the second product (l sums them before
// that, in fp32).  They are formed 2^10 times their size (O and l carry the factor, it
// cancels), and a row's reference maximum follows only when a score passes it by 2^5: weights reach 2^15,
// half of what fp16 holds (see weight_plain for scores that need more room), and keep 11
// bits down to 2^-24 of the greatest.  Following every rise, as the fp16 caches' kernel does
// with 2^14 (11 bits down to 2^-28), rescales O for nearly every tile while a piece has few.
constexpr float kWeightLog2 = 10.f, kRescaleLog2 = 5.f, kUnseen = 1e38f;   // (scores stay below 2^37)

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
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
// Two matrices of 16 x 16 bytes, transposed: lanes 0 - 15 point to the first one's rows, 16 -
// 31 to the second's; lane (grp, tig) gets rows 4 tig .. + 3 of columns grp, 8 + grp of each.
__device__ __forceinline__ void ldsm_bytes_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error 2^-22; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {    // an 8 x 8 matrix of fp16
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

struct TileInfo {      // what the consumers need of a tile
  int slot0;           // its first slot
  int lo, hi;          // slots that some row of the unit sees: [lo, hi)
  int L, n;            // the unit's history and new tokens
  int r0, g;           // its first batch row, its kv head
  int flags;           // 1 first tile of the piece, 2 last, 4 end of the CTA's range
  int dst;             // -1 the whole unit, else the partial slot
};

template <int D, int NT>
struct FSmem {
  static constexpr int NB = D / kKv8Block;
  // Up to 16 rows: four warps that take slots, and one; three CTAs an SM, as more warps hide more
  // of a slab's chain of loads, products and exponentials, while O's registers leave room
  // (65536 / 16 warps).  More rows: O alone is up to 128 registers, so eight warps with 216 each
  // and the producer's group with 72 (216 * 256 + 72 * 128 = 168 * 384).
  static constexpr bool kWide = NT > kKv8NarrowTiles;
  static constexpr int kCtas = kWide ? 1 : 3;
  static constexpr int kWarps = kWide ? 8 : 4, kConsumers = 32 * kWarps;
  static constexpr int kThreads = kConsumers + (kWide ? 128 : 32);
  static constexpr int kTile = kv8_few_tile(D, kWide);          // slots of a tile
  static constexpr int NS = kTile / (16 * kWarps);              // groups of 16 that a warp takes
  static constexpr int kKV = kTile * D;                         // K or V codes of a tile
  static constexpr int kSc = kTile * NB;                        // their scales
  static constexpr int kScCopies = 2 * kSc / 512;               // 16 bytes of those a lane
  static constexpr int kQStride = D * 2 + 16;                   // bytes (conflict-free reads)
  static constexpr int kQBytes = 8 * NT * kQStride;
  static constexpr bool kQRegs = NT == 1;                       // else q is re-read for every tile
  static constexpr int kQBufs = kQRegs ? 1 : 2;
  static constexpr int kStage = 2 * (kKV + kSc);
  static constexpr int kStages =
      (233472 / kCtas - 1024 - 2304 - 1024 - 1024 - (kWide ? 2048 : 0) - kQBufs * kQBytes) / kStage;
  static constexpr int kScOff = kStages * 2 * kKV;
  static constexpr int kQOff = kScOff + kStages * 2 * kSc;
  static constexpr int kStatOff = kQOff + kQBufs * kQBytes;     // [8 NT][warps] maxima, sums, [8 NT] tops
  static constexpr int kInfoOff = kStatOff + (2 * kWarps + 1) * 8 * NT * 4;
  static constexpr int kBarOff = (kInfoOff + kStages * (int)sizeof(TileInfo) + 15) / 16 * 16;
  static constexpr int kEnd = kBarOff + (2 * kStages + kQBufs) * 8 + 64;
  static constexpr size_t kBytes = (size_t)kEnd + 1024;         // the ring is 1024-aligned
  static_assert(kStages >= 3 && kWarps * NB * 1024 <= 2 * kKV, "O goes through a tile's place");
  static_assert(kBytes + 3328 <= 233472 / kCtas && kBytes <= 230000, "shared memory");   // (1 KB the system's, statics)
};

template <int kTile>
__device__ __forceinline__ int seq_tiles(const PagedAttnParams& p, const PagedSeq& s) {
  if (s.n == 0) return 0;
  return (s.L + s.n + kTile - 1) / kTile - paged_lo(p, s.L) / kTile;
}
template <int kTile>
__device__ __forceinline__ int seq_weight(const PagedAttnParams& p, const PagedSeq& s) {
  return s.n == 0 ? 0 : seq_tiles<kTile>(p, s) + kHead;
}

template <int D, int NT>
__global__ void __launch_bounds__(FSmem<D, NT>::kThreads, FSmem<D, NT>::kCtas)
    paged_few_kv8_kernel(const __grid_constant__ PagedFew8Params q8) {
  using Sm = FSmem<D, NT>;
  constexpr int S = Sm::kStages, NB = Sm::NB, NS = Sm::NS, kTile = Sm::kTile;
  constexpr int kWarps = Sm::kWarps, kConsumers = Sm::kConsumers, kThreads = Sm::kThreads;
  const PagedAttnParams& p = q8.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem), sring = smem_u32(smem + Sm::kScOff),
                 qbase = smem_u32(smem + Sm::kQOff);
  float* stat_m = reinterpret_cast<float*>(smem + Sm::kStatOff);
  float* stat_l = stat_m + kWarps * 8 * NT;
  float* stat_top = stat_l + kWarps * 8 * NT;
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
      mbar_init(&full[s], 1 + 32);      // the boxes and q, and each lane's scales
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
    mine += seq_weight<kTile>(p, s);
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
      const int wt = seq_weight<kTile>(p, load_seq(p, b));
      if (x0 < cum + wt) break;
      cum += wt;
    }
    start_b = b;
    start_cum = cum;
  }
  __syncthreads();

  if (warp >= kWarps) {
    if constexpr (Sm::kWide) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      if (warp > kWarps) return;
    }
    // -------------------------------------------------------------- producer
    constexpr int kBoxLg = kTile == 64 ? 6 : 7;      // (a page has 128 slots at most)
    const int bs_lg = p.page_lg < kBoxLg ? p.page_lg : kBoxLg, bs = 1 << bs_lg;   // slots of a box
    const int boxes = kTile >> bs_lg;
    const uint32_t box_bytes = (uint32_t)bs * D;
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
    // Page ids come 32 table entries at a time, a lane each, the next 32 and the next
    // sequence's first ahead of their use: a tile is a few hundred clocks of work, as long
    // as one of these loads takes.
    auto entries = [&](int b, int lo, int hi, int base) -> int {
      const int e = base + lane;
      if (b >= p.B || e < lo >> p.page_lg || e > (hi - 1) >> p.page_lg) return -1;
      return (e < (int)(p.pre_here >> p.page_lg) ? p.prefix_pages : p.table + (int64_t)b * p.max_blocks)[e];
    };
    int ids = -1, ids_next = -1, ids_seq = -1, seq_ahead = -1;      // the last: whose ids_seq are
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
      const int nt = seq_tiles<kTile>(p, s);
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
      int base = (((j0 + xa) * kTile) >> p.page_lg) & ~31;
      ids = seq_ahead == b && xa == 0 ? ids_seq : entries(b, lo, hi, base);
      ids_next = entries(b, lo, hi, base + 32);
      seq_ahead = -1;
      if (((b + 1) & ~31) == base32) {       // (its lengths are here)
        const int n2 = __shfl_sync(0xffffffffu, mys.n, (b + 1) & 31);
        const int L2 = __shfl_sync(0xffffffffu, mys.L, (b + 1) & 31);
        if (n2 > 0 && lin < t1) {
          const int lo2 = paged_lo(p, L2);
          ids_seq = entries(b + 1, lo2, L2 + n2, ((lo2 / kTile * kTile) >> p.page_lg) & ~31);
          seq_ahead = b + 1;
        }
      }
      for (int x = xa; x < xb; ++x, ++it) {
        const int st = it % S;
        const int slot0 = (j0 + x) * kTile;
        // box i of the tile: slots slot0 + i * bs ..; lanes 0-15 take K, 16-31 V
        const int i = lane & 15, first = slot0 + (i << bs_lg);
        const bool take = i < boxes && first < hi && first + bs > lo;
        if ((slot0 >> p.page_lg) - base >= 32) {
          base += 32;
          ids = ids_next;
          ids_next = entries(b, lo, hi, base + 32);
        }
        const int page = __shfl_sync(0xffffffffu, ids, (first >> p.page_lg) & 31);
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
          const int z = in ? (int)((int64_t)page * p.Hkv + g) : (int)(p.n_pages * p.Hkv);
          kv8_tma_codes(ring + (st * 2 + v) * Sm::kKV + (i << bs_lg) * D, v ? &p.tm_v : &p.tm_k, y, z,
                    &full[st]);
        }
        // the scales: 16 bytes a lane and copy whatever the page (a copy of each page's own costs as
        // much as one of its codes: 96 sequences over pages of 16 took 69 us with those, 62 so)
#pragma unroll
        for (int c = 0; c < Sm::kScCopies; ++c) {
          const int piece = c * 32 + lane, sv = piece / (Sm::kSc / 16);
          const int at = piece % (Sm::kSc / 16) * (16 / NB), slot = slot0 + at;      // at: of the tile
          const int spage = __shfl_sync(0xffffffffu, ids, (slot >> p.page_lg) & 31);
          const bool there = slot < hi && slot + 16 / NB > lo && spage >= 0 && spage < p.n_pages;
          const int64_t row = (((int64_t)spage * p.Hkv + g) << p.page_lg) + (slot & ((1 << p.page_lg) - 1));
          kv8_copy16(sring + (st * 2 + sv) * Sm::kSc + at * NB, (sv ? q8.vs : q8.ks) + (there ? row * NB : 0),
                     there);
        }
        kv8_copies_arrive(&full[st]);
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
      if (lane == 0) infos[st].flags = 4;
      __syncwarp();
      mbar_arrive(&full[st]);
      if (lane == 0) mbar_arrive(&full[st]);
    } else {
      // copies in flight land before shared memory goes away
      for (int k = max(0, it - S); k < it; ++k)
        mbar_wait(&full[k % S], (uint32_t)(k / S) & 1u, nullptr);
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  if constexpr (Sm::kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
  const int grp = lane >> 2, tig = lane & 3;
  const int slab = warp * 16 * NS;                    // the warp's slots of a tile
  const float sl2 = p.scale_log2;
  // The slot (of 16) behind row c of score tile t.  Equal pieces of rows 2 i, 2 i + 1 of a
  // tile lie in different halves of the banks (K's loads: the swizzle parts rows 0 - 3 from
  // 4 - 7 where a row has 128 bytes, even from odd ones where it has 64), and rows 4 i ..
  // 4 i + 3 of both tiles are eight rows of different places (V's).
  auto slot_of = [](int t, int c) {
    return D == 128 ? 8 * (c >> 2) + 2 * ((c >> 1) & 1) + 4 * (c & 1) + t
                    : 8 * (c >> 2) + 4 * ((c >> 1) & 1) + (c & 1) + 2 * t;
  };
  auto piece_at = [](int r, int c) {                  // piece c of row r of a tile's codes
    return r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
  };
  constexpr int kT1 = D == 128 ? 1 : 2;               // from tile 0's slot to tile 1's
  const int kr = slab + slot_of(0, grp);              // the lane's K slots: kr, kr + kT1
  const uint32_t k_off0 = piece_at(kr, tig), k_off1 = piece_at(kr + kT1, tig);   // (^ 64: piece tig + 4)
  // V: inner indexes 2 tig, 2 tig + 1 of tile 0 are slots ve, ve + vo; of tile 1 kT1 further.
  // The matrix row that the lane points to, and which of a pair of pieces.
  const int ve = slab + slot_of(0, 2 * tig);
  constexpr int vo = D == 128 ? 4 : 1;
  const int vr = slab + slot_of((lane >> 1) & 1, 2 * ((lane >> 2) & 3) + (lane & 1));
  const uint32_t v_off = piece_at(vr, lane >> 4);     // (^ 32 g: pieces 2 g, 2 g + 1)
  // a K piece's block of 32 columns, as a permute that doubles its scale's byte to fp16
  const uint32_t kb = tig >> 1, sel_k0 = kb << 12 | 4 << 8 | kb << 4 | 4, sel_k1 = sel_k0 + 0x2020;
  const uint32_t q_lane = qbase + grp * Sm::kQStride + tig * 32;
  // The lane's rows: 8 nt + 2 tig + e.  nref: less what their exponents are taken against (log2
  // units, less kWeightLog2 but where weight_plain; kUnseen: nothing seen yet).  most: the
  // exponent at which that follows, of all the lane's rows the least.  O: columns 16 i + grp
  // and + 8 of either row.  (Registers bound 32 rows: with each row's limit and slots in them
  // 24 x 6000 slots took 59.9 us, so 55.7, though 24 rows 45.8 and so 46.9.)
  float nref[NT][2], most = 0.f, l_r[NT][2], O[NT][NB * 2][4];
  uint32_t toks[(NT + 1) / 2] = {};     // the rows' tokens (of at most 32), a byte each; 0x80: no row
  uint32_t qf[Sm::kQRegs ? D / 16 : 1][2];
  // q's fragments of products 2 x, 2 x + 1 (x < D / 32) of row tile nt
  auto load_q = [&](uint32_t qb, int nt, int x, uint32_t* a, uint32_t* b) {
    const uint4 u = lds128(qb + nt * 8 * Sm::kQStride + (x >> 1) * 128 + (x & 1) * 16);
    a[0] = u.x; a[1] = u.y;
    b[0] = u.z; b[1] = u.w;
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
#pragma unroll
      for (int w = 0; w < (NT + 1) / 2; ++w) toks[w] = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = (nt * 8 + 2 * tig + e) / p.G;
          toks[nt >> 1] |= (uint32_t)(t < n ? t : 0x80) << ((nt & 1) * 16 + e * 8);
          nref[nt][e] = kUnseen;
          l_r[nt][e] = 0.f;
        }
      most = kWeightLog2 + kRescaleLog2;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < NB * 2; ++i) O[nt][i][0] = O[nt][i][1] = O[nt][i][2] = O[nt][i][3] = 0.f;
      if constexpr (Sm::kQRegs) {
#pragma unroll
        for (int x = 0; x < D / 32; ++x) load_q(qb, 0, x, qf[2 * x], qf[2 * x + 1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[0]);       // q's place is free
      }
    }
    if (slab < vhi && slab + 16 * NS > vlo) {
      // every row sees every slot of this warp's: n - 1 slots from the end are behind the
      // first row, windows begin at most n - 1 slots behind vlo
      const bool clear = slab + 16 * NS <= vhi - (n - 1) && slab >= (p.window > 0 ? vlo + (n - 1) : vlo);
      // the scales: K's of the lane's two slots, V's of its four ([tile][even, odd])
      uint32_t kw[NS][2], sw[NS][2][2], large = 0;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if constexpr (D == 128) {
          const uint2 k2 = lds64(ks + (kr + 16 * s) * NB), e2 = lds64(vs + (ve + 16 * s) * NB),
                      o2 = lds64(vs + (ve + vo + 16 * s) * NB);
          kw[s][0] = k2.x; kw[s][1] = k2.y;
          sw[s][0][0] = e2.x; sw[s][1][0] = e2.y;
          sw[s][0][1] = o2.x; sw[s][1][1] = o2.y;
        } else {
          const uint2 v4 = lds64(vs + (ve + 16 * s) * NB);     // (one behind the other)
          kw[s][0] = lds16(ks + (kr + 16 * s) * NB);
          kw[s][1] = lds16(ks + (kr + kT1 + 16 * s) * NB);
          sw[s][0][0] = v4.x & 0xffffu; sw[s][0][1] = v4.x >> 16;
          sw[s][1][0] = v4.y & 0xffffu; sw[s][1][1] = v4.y >> 16;
        }
        if (slab < vlo || slab + 16 * NS > vhi) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const int c = ve + 16 * s + t * kT1 + o * vo;
              if (c < vlo || c >= vhi) sw[s][t][o] = 0;
            }
        }
        large |= kv8_big_scales(kw[s][0]) | kv8_big_scales(kw[s][1]) | kv8_big_scales(sw[s][0][0]) |
                 kv8_big_scales(sw[s][0][1]) | kv8_big_scales(sw[s][1][0]) | kv8_big_scales(sw[s][1][1]);
      }
      // One row tile asks whether a scale is large and keeps the values' shorter form for when
      // none is (half the conversion's arithmetic).  More row tiles have enough products to
      // hide the longer one behind, and no register for the question: 16 heads a kv head,
      // 8 x 131072 slots 118 -> 111 us without it, 24 sequences of 24 rows 48.5 -> 46;
      // one row tile without it 62 -> 64 (96 ragged sequences).
      const bool any_big = NT > 1 || __any_sync(0xffffffffu, (large & 0x80808080u) != 0);
      // (one row tile: two sums, so that products follow one another half as far)
      constexpr int kSums = NT == 1 ? 2 : 1;
      float sc[NS][NT][kSums][4];
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < kSums; ++k)
            sc[s][nt][k][0] = sc[s][nt][k][1] = sc[s][nt][k][2] = sc[s][nt][k][3] = 0.f;
      auto scores = [&](auto big) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint4 c[NS][2];
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            c[s][0] = lds128(kt + (k_off0 ^ (h << 6)) + s * 16 * D);
            c[s][1] = lds128(kt + (k_off1 ^ (h << 6)) + s * 16 * D);
          }
          const uint32_t sel = h ? sel_k1 : sel_k0;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            [[maybe_unused]] uint32_t qv[Sm::kQRegs ? 1 : NT][2][2];
            if constexpr (!Sm::kQRegs) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) load_q(qb, nt, 2 * h + x, qv[nt][0], qv[nt][1]);
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              const Kv8Unit<decltype(big)::value> u0(__byte_perm(kw[s][0], 0, sel)),
                  u1(__byte_perm(kw[s][1], 0, sel));
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t w0 = x ? (y ? c[s][0].w : c[s][0].z) : (y ? c[s][0].y : c[s][0].x);
                const uint32_t w1 = x ? (y ? c[s][1].w : c[s][1].z) : (y ? c[s][1].y : c[s][1].x);
                const uint32_t a[4] = {u0(w0, 0x4140), u1(w1, 0x4140), u0(w0, 0x4342), u1(w1, 0x4342)};
                if constexpr (Sm::kQRegs) {
                  const uint32_t* b = qf[4 * h + 2 * x + y];
                  mma16816(sc[s][0][y % kSums], a, b[0], b[1]);
                } else {
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma16816(sc[s][nt][0], a, qv[nt][y][0], qv[nt][y][1]);
                }
              }
            }
          }
        }
      };
      if constexpr (NT > 1) scores(std::true_type());
      else if (__builtin_expect(any_big, 0)) scores(std::true_type());
      else scores(std::false_type());
      bool need = false;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if constexpr (kSums == 2) {
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[s][0][0][k] += sc[s][0][1][k];
        }
        if (!clear) {
          const int L = infos[st].L;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int last = L + (int)(toks[nt >> 1] >> ((nt & 1) * 16 + e * 8) & 0x7f);
              const int low = paged_window(p, last);
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const int c = kr + 16 * s + kT1 * t, slot = slot0 + c;
                if (!(c >= vlo && slot <= last && slot >= low)) sc[s][nt][0][2 * t + e] = -INFINITY;
              }
            }
        }
      }
      float top[NT][2];                   // of the lane's slots
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[0][nt][0][e], sc[0][nt][0][2 + e]);
#pragma unroll
          for (int s = 1; s < NS; ++s) x = fmaxf(x, fmaxf(sc[s][nt][0][e], sc[s][nt][0][2 + e]));
          top[nt][e] = x;
          need |= fmaf(x, sl2, nref[nt][e]) > most;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[nt][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (fmaf(x, sl2, nref[nt][e]) > most) {       // (alike in the row's lanes)
              const float t = fmaf(x, sl2, -kWeightLog2);
              const bool plain = weight_plain(t);
              // Never below where it stands: the limit may be another row's, and a reference
              // that fell with a row's scores would let O and l grow without end.
              const float mn = fmaxf(plain ? t + kWeightLog2 : t, -nref[nt][e]);
              const float f = ex2(-nref[nt][e] - mn);     // (nothing seen: 0)
              nref[nt][e] = -mn;
              // (places of no row hold whatever lay there: the bits of others do not depend on it)
              if (plain && !(toks[nt >> 1] >> ((nt & 1) * 16 + e * 8) & 0x80)) most = kRescaleLog2;
              l_r[nt][e] *= f;
#pragma unroll
              for (int i = 0; i < NB * 2; ++i) {
                O[nt][i][e] *= f;
                O[nt][i][2 + e] *= f;
              }
            }
          }
      }
      uint32_t pb[NS][NT][2];
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = ex2(fmaf(sc[s][nt][0][k], sl2, nref[nt][k & 1]));   // 2^-inf = 0
          l_r[nt][0] += w[0] + w[2];
          l_r[nt][1] += w[1] + w[3];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const __half2 h = __floats2half2_rn(w[2 * t], w[2 * t + 1]);
            pb[s][nt][t] = transposed(*reinterpret_cast<const uint32_t*>(&h));
          }
        }
      // O' += V' P'
      auto values = [&](auto big) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int g = 0; g < NB; ++g) {
            uint32_t v[4];
            ldsm_bytes_t(vt + (v_off ^ (g << 5)) + s * 16 * D, v);
            const uint32_t sel = (4 + g) << 12 | g << 4;
            const Kv8Unit<decltype(big)::value> u0(__byte_perm(sw[s][0][0], sw[s][0][1], sel) & 0xff00ff00u),
                u1(__byte_perm(sw[s][1][0], sw[s][1][1], sel) & 0xff00ff00u);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t a[4] = {u0(v[2 * j], 0x4140), u0(v[2 * j + 1], 0x4140), u1(v[2 * j], 0x4342),
                                     u1(v[2 * j + 1], 0x4342)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(O[nt][g * 2 + j], a, pb[s][nt][0], pb[s][nt][1]);
            }
          }
      };
      if constexpr (NT > 1) values(std::true_type());
      else if (__builtin_expect(any_big, 0)) values(std::true_type());
      else values(std::false_type());
    }
    if (flags & 2) {
      // The piece's end: the warps' maxima meet, each brings its sums to the greatest,
      // and warp w < D / 32 adds all warps' O of column block w.  O goes through the place
      // of the last tile's codes, which all warps have read behind the first barrier.
      const int rows = n * p.G, r0 = infos[st].r0, g = infos[st].g, dst = infos[st].dst;
      const uint32_t xbase = kt;
      __syncwarp();
      if (!Sm::kQRegs && lane == 0) mbar_arrive(&q_empty[seg % Sm::kQBufs]);
      ++seg;
      float m_r[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m_r[nt][e] = nref[nt][e] == kUnseen ? -INFINITY : -nref[nt][e];
          if (grp == 0) stat_m[(nt * 8 + 2 * tig + e) * kWarps + warp] = m_r[nt][e];
        }
      named_sync(1, kConsumers);
      if (*(volatile int*)&abort_s) return;       // (set before a warp's arrival, see above)
      auto max_of = [&](int row) {
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; w += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(stat_m + row * kWarps + w);
          m = fmaxf(m, fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)));
        }
        return m;
      };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = nt * 8 + 2 * tig + e;
          // (stat_m is read here alone: a warp that has written its O may be at the next piece's)
          const float M = max_of(row), f = m_r[nt][e] == -INFINITY ? 0.f : ex2(m_r[nt][e] - M);
          if (warp == 0 && grp == 0) stat_top[row] = M;
          float l = l_r[nt][e] * f;
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          if (grp == 0) stat_l[row * kWarps + warp] = l;
#pragma unroll
          for (int i = 0; i < NB * 2; ++i) {
            O[nt][i][e] *= f;
            O[nt][i][2 + e] *= f;
          }
        }
      // O's way: [block of 32 columns][warp][row of the tile][32 columns], eight columns
      // moved by the row's pair and four by its parity (no bank conflicts on either side)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        __syncwarp();
        if (nt > 0) named_sync(1, kConsumers);     // the row tile before is read
#pragma unroll
        for (int d = 0; d < NB; ++d)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x)            // column 8 x + grp of block d
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(
                               xbase + (d * kWarps + warp) * 1024 + (2 * tig + e) * 128 +
                               ((x ^ tig) << 5) + ((grp ^ (4 * e)) << 2)),
                           "f"(O[nt][d * 2 + (x >> 1)][2 * (x & 1) + e])
                           : "memory");
        named_sync(1, kConsumers);
        if (warp < NB) {
          // row lane / 4, columns 8 (lane % 4) .. + 7
          const int r8 = lane >> 2, row = nt * 8 + r8;
          const uint32_t from = xbase + warp * kWarps * 1024 + r8 * 128 + (((lane & 3) ^ (r8 >> 1)) << 5);
          float v[8] = {};
#pragma unroll
          for (int s = 0; s < kWarps; ++s)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint4 w = lds128(from + s * 1024 + ((x ^ (r8 & 1)) << 4));
              v[4 * x] += __uint_as_float(w.x);
              v[4 * x + 1] += __uint_as_float(w.y);
              v[4 * x + 2] += __uint_as_float(w.z);
              v[4 * x + 3] += __uint_as_float(w.w);
            }
          if (row < rows) {
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; w += 4) {
              const float4 l4 = *reinterpret_cast<const float4*>(stat_l + row * kWarps + w);
              l += (l4.x + l4.y) + (l4.z + l4.w);
            }
            const int t = row / p.G, hq = g * p.G + (row - t * p.G);
            const int col = warp * 32 + 8 * (lane & 3);
            if (dst < 0 && !p.own) {
              const float inv = l > 0.f ? 1.f / l : 0.f;
              uint32_t w[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const __half2 h = __floats2half2_rn(v[2 * c] * inv, v[2 * c + 1] * inv);
                w[c] = *reinterpret_cast<const uint32_t*>(&h);
              }
              *reinterpret_cast<uint4*>(p.out + (int64_t)(r0 + t) * p.out_stride + (int64_t)hq * D + col) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            } else {
              const int64_t at = dst < 0 ? (int64_t)(r0 + t) * p.Hq + hq
                                         : ((int64_t)cta * 2 + dst) * p.slot_rows + row;
              float4* o = reinterpret_cast<float4*>((dst < 0 ? p.own : p.part) + at * D + col);
              o[0] = make_float4(v[0], v[1], v[2], v[3]);
              o[1] = make_float4(v[4], v[5], v[6], v[7]);
              if (warp == 0 && (lane & 3) == 0)
                (dst < 0 ? p.own_ml : p.ml)[at] = make_float2(stat_top[row], l);
            }
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next copy there
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
}

template <int D, int NT>
cudaError_t launch_few(const PagedFew8Params& p, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.a.nc);
  cfg.blockDim = dim3(FSmem<D, NT>::kThreads);
  cfg.dynamicSmemBytes = FSmem<D, NT>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_few_kv8_kernel<D, NT>, p);
}

template <int D, int NT>
cudaError_t configure_one(bool* wide) {
  if (FSmem<D, NT>::kWide) {           // their warps share out the registers that the block is launched with
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, paged_few_kv8_kernel<D, NT>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != 168) *wide = false;
  }
  return cudaFuncSetAttribute(paged_few_kv8_kernel<D, NT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FSmem<D, NT>::kBytes);
}

}  // namespace

void paged_few_kv8_slots(int num_sms, int G, int64_t max_new, int* nc, int* slot_rows) {
  *nc = (kv8_few_wide(G, max_new) ? 1 : 3) * num_sms;      // FSmem::kCtas
  *slot_rows = max_new * G <= 16 ? 16 : 32;
}

cudaError_t launch_paged_few_kv8(const PagedFew8Params& p, cudaStream_t s, bool pdl) {
  if (p.a.max_new * p.a.G > p.a.slot_rows || p.a.nc < 1 || p.a.nc > 512) return cudaErrorInvalidValue;
  const int tiles = (int)((p.a.max_new * p.a.G + 7) / 8) - 1;      // of eight rows
  using F = cudaError_t (*)(const PagedFew8Params&, cudaStream_t, bool);
  constexpr F f[2][4] = {{launch_few<64, 1>, launch_few<64, 2>, launch_few<64, 3>, launch_few<64, 4>},
                         {launch_few<128, 1>, launch_few<128, 2>, launch_few<128, 3>, launch_few<128, 4>}};
  if ((p.a.D != 64 && p.a.D != 128) || tiles < 0 || tiles > 3) return cudaErrorInvalidValue;
  return f[p.a.D == 128][tiles](p, s, pdl);
}

cudaError_t configure_paged_few_kv8(bool* wide) {
  *wide = true;
  for (auto f : {configure_one<64, 1>, configure_one<64, 2>, configure_one<64, 3>, configure_one<64, 4>,
                 configure_one<128, 1>, configure_one<128, 2>, configure_one<128, 3>, configure_one<128, 4>}) {
    const cudaError_t e = f(wide);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace blk
