// Attention over a paged K/V cache for many rows: prompts and chunks of them
// (rows of one sequence, causal), and a prefix that all sequences share (its
// keys are read once for the rows of the whole batch).
//
// Bound by the tensor cores and the exponentials: 4 D flops and one 2^x per
// score.  A unit is two blocks of 128 / G tokens, each with the G query heads of
// one kv head: 256 rows that share every K/V tile of 128 slots.  The CTAs (one
// per SM) take equal ranges of the line of all units' tiles, as the few-row
// kernel does (see paged.h).  Ten warps:
//   warp 0     producer: q of both blocks once per unit, then K and V tiles, page
//              by page (each lane one box of 64 columns), into a ring of tiles.
//   warp 1     MMA issuer (lane 0): S = Q K^T (M = N = 128) and O += P V for the
//              two blocks in turn: S0 S1 | PV0 S0' | PV1 S1' | ..., so that one
//              block's products run under the other's softmax.
//   warps 2-5, 6-9   softmax of block 0 and 1, a thread per row: scores from TMEM,
//              online softmax in base 2 with lazy rescaling of O, P (fp16)
//              over S's own columns (TMEM: S0 S1 O0 O1 = 512 columns).
// MMAs of one thread execute in order: S_j+1 is written after PV_j has read P_j,
// and a commit behind S_j+1 says that PV_j is complete too.
// Slots that no row of the unit sees have their V rows zeroed before PV (0 * NaN
// is NaN).  Every wait is bounded.
#include <math.h>

#include "common.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "tcgen05.cuh"

namespace blk {
namespace {

constexpr int kThreads = 320;
constexpr int kTile = kPagedManyTile;
constexpr int kInfos = 8;
constexpr float kRescaleLog2 = 8.f;   // see the softmax
constexpr int kMinTiles = 2;

struct ManyInfo {
  int slot0, lo, hi;         // first slot; slots that some row sees: [lo, hi)
  int first;                 // slot of the unit's first token
  int ntok, r0, tok0, g;     // tokens, batch row of the first, its number, kv head
  int flags;                 // 1 first tile of the piece, 2 last, 4 the end, 8 block 1 has rows
  int dst;                   // -1 whole, else the partial slot
};

template <int D>
struct MSmem {
  static constexpr int kQBlk = 128 * D * 2;                  // [D / 64][128 rows][128 B]
  static constexpr int kKV = kTile * D * 2;                  // K or V tile, the same form
  static constexpr int kRing = D == 128 ? 5 : 8;
  static constexpr int kRingOff = 2 * kQBlk;
  static constexpr int kInfoOff = kRingOff + kRing * kKV;
  static constexpr int kBarOff = kInfoOff + kInfos * (int)sizeof(ManyInfo);
  static constexpr int kEnd = kBarOff + (2 * kRing + 10) * 8 + 16;
  static constexpr size_t kBytes = (size_t)kEnd + 1024;
  static constexpr uint32_t kSCol = 0, kOCol = 256;
  static_assert(kBarOff % 8 == 0 && kBytes <= 232448, "shared memory");
};

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {   // 2^x; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ schedule
// The units of a ragged batch and the tiles before each, for one kv head: unit
// u of sequence b are its tokens 2 btok u ...  One CTA; bound by latency (about
// 3 us), for calls that take tens of microseconds.
__global__ void __launch_bounds__(1024)
    paged_sched_kernel(const __grid_constant__ PagedManyParams q, int64_t* pref, PagedUnit* unit) {
  extern __shared__ int off[];          // [B + 1] units before each sequence
  __shared__ int64_t wsum[32];
  __shared__ int64_t run;
  griddep_wait();
  griddep_launch();
  const PagedAttnParams& p = q.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int utok = 2 * q.btok;
  auto scan = [&](int64_t v, int64_t& total) -> int64_t {   // exclusive, over the block
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    return before + x - v;
  };
  const int per = (p.B + 1023) / 1024;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int64_t mine = 0, total;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const PagedSeq s = load_seq(p, b);
    mine += (s.n + utok - 1) / utok;
    bad |= s.bad;
  }
  if (bad) set_error(p.err, kDevPage);
  int64_t at = scan(mine, total);
  for (int b = b0; b < b1; ++b) {
    off[b] = (int)min(at, (int64_t)q.units);
    at += (load_seq(p, b).n + utok - 1) / utok;
  }
  // more units than rows allow: row ranges that overlap (the host's row_start is wrong)
  const int R = (int)min(total, (int64_t)q.units);
  if (total > q.units && tid == 0) set_error(p.err, kDevPage);
  if (tid == 0) run = 0;
  __syncthreads();
  for (int k0 = 0; k0 < R; k0 += 1024) {
    const int k = k0 + tid;
    int64_t tiles = 0;
    if (k < R) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= k) lo = mid; else hi = mid;
      }
      const PagedSeq s = load_seq(p, lo);
      PagedUnit u;
      u.b = lo;
      u.tok = (k - off[lo]) * utok;
      u.ntok = min(utok, s.n - u.tok);
      u.r0 = s.r0 + u.tok;
      u.L = s.L;
      u.n = s.n;
      u.lo = paged_lo(p, s.L + u.tok);
      u.hi = s.L + u.tok + u.ntok;
      unit[k] = u;
      tiles = (u.hi + kTile - 1) / kTile - u.lo / kTile;
    }
    int64_t chunk;
    const int64_t ex = scan(tiles, chunk);
    if (k < R) pref[k] = run + ex;
    __syncthreads();
    if (tid == 0) run += chunk;
    __syncthreads();
  }
  if (tid == 0) {
    pref[R] = run;
    pref[-1] = R;
  }
}

template <int D, bool kPrefix>
__global__ void __launch_bounds__(kThreads, 1)
    paged_many_kernel(const __grid_constant__ PagedManyParams q) {
  using Sm = MSmem<D>;
  constexpr int R = Sm::kRing, H = D / 64;
  const PagedAttnParams& p = q.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + Sm::kRingOff;
  volatile ManyInfo* infos = reinterpret_cast<volatile ManyInfo*>(smem + Sm::kInfoOff);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + Sm::kBarOff);
  uint64_t* kv_empty = kv_full + R;
  uint64_t* q_full = kv_empty + R;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;       // [2] S of a block in TMEM
  uint64_t* p_full = s_full + 2;        // [2] its P in TMEM (O rescaled)
  uint64_t* o_full = p_full + 2;        // [2] O complete at the end of a piece
  uint64_t* drain = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  griddep_wait();
  griddep_launch();
  // this CTA's range of the line of tiles
  int64_t T1;
  int n_units;
  if constexpr (kPrefix) {
    n_units = q.units;
    T1 = (int64_t)q.units * ((p.prefix_len + kTile - 1) / kTile);
  } else {
    n_units = (int)q.pref[-1];
    T1 = q.pref[n_units];
  }
  const int64_t T = T1 * p.Hkv;
  int nc = p.nc;
  if constexpr (!kPrefix) {
    const int64_t enough = (T + kMinTiles - 1) / kMinTiles;
    nc = (int)(enough < p.nc ? (enough < 1 ? 1 : enough) : p.nc);
  }
  const int64_t t0 = cta < nc ? T * cta / nc : T, t1 = cta < nc ? T * (cta + 1) / nc : T;
  if (t0 >= t1) {
    if (threadIdx.x == 0 && !kPrefix) p.cut[cta].c0 = -1;
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(&s_full[k], 1);
      mbar_init(&p_full[k], 4);
      mbar_init(&o_full[k], 1);
    }
    mbar_init(drain, 1);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    const int ps_lg = p.page_lg, boxes = kTile >> ps_lg;     // pages of a tile
    const uint32_t box_bytes = (128u << ps_lg);              // 64 columns of one page
    int g = (int)(t0 / T1), k;
    int64_t cum;                       // tiles before unit k
    {
      const int64_t x = t0 - (int64_t)g * T1;
      if constexpr (kPrefix) {
        const int64_t nt = (p.prefix_len + kTile - 1) / kTile;
        k = (int)(x / nt);
        cum = k * nt;
      } else {
        int lo = 0, hi = n_units;      // last unit with pref <= x: 32 probes a round
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32;
          const int i = lo + (lane + 1) * step;
          const bool le = i < hi && q.pref[i] <= x;
          const int c = __popc(__ballot_sync(0xffffffffu, le));
          const int nlo = lo + c * step;
          hi = min(hi, nlo + step);
          lo = nlo;
        }
        k = lo;
        cum = q.pref[k];
      }
    }
    int64_t lin = t0;
    int it = 0, seg = 0, qn = 0, item = 0;   // tiles, pieces, q loads, ring items so far
    bool ok = true;
    PagedPiece cut;
    cut.c0 = -1;
    auto wait_slot = [&](int i) {      // ring item i's place is free
      if (i >= R && !mbar_wait(&kv_empty[i % R], (uint32_t)(i / R - 1) & 1u, p.err)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
    };
    while (lin < t1 && ok) {
      if (k >= n_units) {
        k = 0;
        cum = 0;
        ++g;
      }
      PagedUnit u;
      if constexpr (kPrefix) {
        u.b = 0;
        u.tok = k * 2 * q.btok;
        u.ntok = min(2 * q.btok, p.N - u.tok);
        u.r0 = u.tok;
        u.L = u.n = 0;
        u.lo = 0;
        u.hi = (int)p.prefix_len;
      } else {
        u = q.unit[k];
      }
      const int j0 = u.lo / kTile, nt = (u.hi + kTile - 1) / kTile - j0;
      const int64_t us = (int64_t)g * T1 + cum;
      const int xa = (int)(lin - us), xb = (int)min((int64_t)nt, t1 - us);
      const bool whole = xa == 0 && xb == nt;
      const int dst = whole ? -1 : (lin == t0 ? 0 : 1);
      const bool two = u.ntok > q.btok;
      if (xa == 0) {
        if constexpr (kPrefix) {
          // until the own parts' kernel says otherwise a row has no own part
          for (int t = lane; t < u.ntok; t += 32)
            p.row_info[(int64_t)(u.r0 + t) * p.Hkv + g] = make_int4(-2, 0, 0, 0);
        } else {
          const int c1 = whole ? cta : (int)(((us + nt) * nc - 1) / T);
          if (!whole) {
            cut.c0 = cta;
            cut.c1 = c1;
            cut.s0 = dst;
            cut.rows = u.ntok * p.G;
            cut.r0 = u.r0;
            cut.g = g;
          }
          if (p.row_info)
            for (int t = lane; t < u.ntok; t += 32)
              p.row_info[(int64_t)(u.r0 + t) * p.Hkv + g] =
                  make_int4(whole ? -1 : cta, c1, whole ? 0 : dst,
                            t / q.btok * 128 + t % q.btok * p.G);
        }
      }
      const int32_t* row = kPrefix ? p.prefix_pages : p.table + (int64_t)u.b * p.max_blocks;
      for (int x = xa; x < xb && ok; ++x, ++it) {
        const int slot0 = (j0 + x) * kTile;
        // lane: half lane / 8 of the columns (D / 64 of them), page lane % 8 of the tile
        const int i = lane & 7, half = lane >> 3, first = slot0 + (i << ps_lg);
        const bool take = half < H && i < boxes && first < u.hi && first + (1 << ps_lg) > u.lo;
        int64_t page = -1;
        if (take) page = row[first >> ps_lg];
        const bool in = page >= 0 && page < p.n_pages;
        if (take && !in) set_error(p.err, kDevPage);
        const int z = in ? (int)(page * p.Hkv + g) : (int)(p.n_pages * p.Hkv);   // zeros
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, take)) * box_bytes;
        const int at = half * (kTile * 128) + ((i << ps_lg) * 128);
        if (x == xa) {
          if (seg > 0 && !mbar_wait(q_empty, (uint32_t)(seg - 1) & 1u, p.err)) ok = false;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++qn;
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * q.btok * p.G * D * 2);
            for (int blk = 0; blk < (two ? 2 : 1); ++blk)
              for (int hh = 0; hh < H; ++hh)
                tma_3d(smem + blk * Sm::kQBlk + hh * 16384, &p.tm_q, hh * 64, g * p.G,
                       u.r0 + blk * q.btok, q_full);
          }
        }
        wait_slot(item);
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
          mbar_arrive_expect_tx(&kv_full[item % R], bytes);
        }
        __syncwarp();
        if (take) tma_3d(ring + (item % R) * Sm::kKV + at, &p.tm_k, half * 64, 0, z, &kv_full[item % R]);
        ++item;
        wait_slot(item);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&kv_full[item % R], bytes);
        __syncwarp();
        if (take) tma_3d(ring + (item % R) * Sm::kKV + at, &p.tm_v, half * 64, 0, z, &kv_full[item % R]);
        ++item;
      }
      lin = us + xb;
      cum += nt;
      ++k;
      ++seg;
    }
    if (!kPrefix && lane == 0) {
      volatile PagedPiece& c = p.cut[cta];
      c.c1 = cut.c1;
      c.s0 = cut.s0;
      c.rows = cut.rows;
      c.r0 = cut.r0;
      c.g = cut.g;
      c.c0 = ok ? cut.c0 : -1;
    }
    if (ok) wait_slot(item);
    if (ok) {
      if (lane == 0) {
        infos[it % kInfos].flags = 4;
        mbar_arrive(&kv_full[item % R]);
      }
    } else {
      // copies in flight land before shared memory goes away
      if (qn > 0) mbar_wait(q_full, (uint32_t)(qn - 1) & 1u, nullptr);
      for (int j = max(0, item - R); j < item; ++j)
        mbar_wait(&kv_full[j % R], (uint32_t)(j / R) & 1u, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = tc_idesc(128, kTile, 0), id_o = tc_idesc(128, D, 1);
      const uint32_t qa = smem_u32(smem), ra = smem_u32(ring);
      bool ok = true;
      int seg = -1;                    // piece of the tile whose S was issued last
      auto issue_s = [&](int blk, int it) {   // S of block blk, tile it
        const uint32_t kb = ra + (2 * it % R) * Sm::kKV, qb = qa + blk * Sm::kQBlk;
        const uint32_t tS = tmem + Sm::kSCol + blk * 128;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = (ks >> 2) * 16384;
          tc_mma(tS, tc_desc_kmajor(qb + o) + ((ks & 3) * 32 >> 4),
                 tc_desc_kmajor(kb + o) + ((ks & 3) * 32 >> 4), id_s, ks != 0);
        }
      };
      auto issue_pv = [&](int blk, int it, bool acc) {
        const uint32_t vb = ra + ((2 * it + 1) % R) * Sm::kKV;
        const uint32_t tP = tmem + Sm::kSCol + blk * 128, tO = tmem + Sm::kOCol + blk * 128;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          tc_mma_ts(tO, tP + kk * 8, tc_desc_mnmajor(vb + kk * 16 * 128), id_o,
                    acc || kk != 0);
      };
      // K of tile it has landed (and q of a new piece); its flags
      auto begin = [&](int it) -> int {
        const int i = 2 * it;
        if (!mbar_wait(&kv_full[i % R], (uint32_t)(i / R) & 1u, p.err)) return -1;
        const int f = infos[it % kInfos].flags;
        if (f & 4) return f;
        if (f & 1) {
          ++seg;
          if (!mbar_wait(q_full, (uint32_t)seg & 1u, p.err)) return -1;
        }
        return f;
      };
      auto end_s0 = [&](int it, int f) {
        if (f & 4) mbar_arrive(&s_full[0]);
        else {
          issue_s(0, it);
          tc_commit(&s_full[0]);
        }
      };
      auto end_s1 = [&](int it, int f) {
        if (f & 4) {
          mbar_arrive(&s_full[1]);
          return;
        }
        if (f & 8) {
          issue_s(1, it);
          tc_commit(&s_full[1]);
        } else {
          mbar_arrive(&s_full[1]);
        }
        tc_commit(&kv_empty[2 * it % R]);
        if (f & 2) tc_commit(q_empty);
      };
      int f = begin(0);
      ok = f >= 0;
      if (ok) {
        tc_fence_after();
        end_s0(0, f);
        end_s1(0, f);
      }
      for (int it = 0; ok && !(f & 4); ++it) {
        const int vi = 2 * it + 1;
        int fn = 0;
        if (!mbar_wait(&p_full[0], (uint32_t)it & 1u, p.err) ||
            !mbar_wait(&kv_full[vi % R], (uint32_t)(vi / R) & 1u, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        issue_pv(0, it, !(f & 1));
        if (f & 2) tc_commit(&o_full[0]);
        fn = begin(it + 1);
        if (fn < 0) {
          ok = false;
          break;
        }
        end_s0(it + 1, fn);
        if (!mbar_wait(&p_full[1], (uint32_t)it & 1u, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (f & 8) issue_pv(1, it, !(f & 1));
        if (f & 2) {
          if (f & 8) tc_commit(&o_full[1]);
          else mbar_arrive(&o_full[1]);
        }
        tc_commit(&kv_empty[vi % R]);
        end_s1(it + 1, fn);
        f = fn;
      }
      // issued MMAs finish before TMEM and shared memory go away
      tc_commit(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int blk = (warp - 2) >> 2;
    const int qt = warp & 3;                     // TMEM lane quarter of this warp
    const int r = qt * 32 + lane;                // row of the block
    const uint32_t loff = (uint32_t)(qt * 32) << 16;
    const uint32_t tS = tmem + Sm::kSCol + blk * 128 + loff;
    const uint32_t tO = tmem + Sm::kOCol + blk * 128 + loff;
    const float sl2 = p.scale_log2;
    const int rt = r / p.G;                      // token of the row in its block
    float m = -INFINITY, l = 0.f;
    int seg = 0;
    bool ok = true;
    // decisions before a warp-collective TMEM access are uniform over the warp
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err));
    };
    for (int it = 0; ok; ++it) {
      if (!wait_all(&s_full[blk], (uint32_t)it & 1u)) { ok = false; break; }
      tc_fence_after();
      volatile const ManyInfo& f = infos[it % kInfos];
      const int flags = f.flags;
      if (flags & 4) break;
      const int slot0 = f.slot0, lo = f.lo, hi = f.hi, first = f.first, ntok = f.ntok;
      const bool here = blk == 0 || (flags & 8);
      if (!here) {       // the unit has no rows in block 1
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[blk]);
        if (flags & 2) {
          if (!wait_all(&o_full[blk], (uint32_t)seg & 1u)) { ok = false; break; }
          ++seg;
        }
        continue;
      }
      const int t = blk * q.btok + rt;           // token of the unit
      const int last = kPrefix ? hi - 1 : first + min(t, ntok - 1);
      if (flags & 1) {
        m = -INFINITY;
        l = 0.f;
      }
      // rows of V that no row of the unit sees: zero before PV (block 0 for both)
      if (blk == 0 && (slot0 < lo || slot0 + kTile > hi)) {
        const int vi = 2 * it + 1;
        if (!wait_all(&kv_full[vi % R], (uint32_t)(vi / R) & 1u)) { ok = false; break; }
        if (slot0 + r < lo || slot0 + r >= hi) {
          uint8_t* vrow = ring + (vi % R) * Sm::kKV + (size_t)r * 128;
#pragma unroll
          for (int hh = 0; hh < H; ++hh)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(vrow + hh * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      float sv[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tc_ld32(tS + c, sv + c);
      tc_wait_ld();
      const int first_last = kPrefix ? hi - 1 : first + blk * q.btok;   // of the block's first row
      if (slot0 + kTile - 1 > first_last) {      // some row sees less than the tile
        const int lim = last - slot0;
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c > lim) sv[c] = -INFINITY;
      }
      if (!kPrefix) {
        const int low = max(lo, (int)window_lo(p.window, last)) - slot0;
        if (__any_sync(0xffffffffu, low > 0)) {
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (c < low) sv[c] = -INFINITY;
        }
      }
      float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
      for (int c = 0; c < kTile; c += 4) {
        a0 = fmaxf(a0, sv[c]);
        a1 = fmaxf(a1, sv[c + 1]);
        a2 = fmaxf(a2, sv[c + 2]);
        a3 = fmaxf(a3, sv[c + 3]);
      }
      const float mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * sl2;   // log2 units
      // A row's reference maximum moves (and O, l are rescaled) only when the
      // maximum grew by more than 2^8 since: P <= 256 fits fp16, and 1 / l at the
      // end makes the choice exact.
      const bool need = (m == -INFINITY) ? (mx != -INFINITY) : (mx - m > kRescaleLog2);
      const bool move = __any_sync(0xffffffffu, need);
      const float mn = move ? fmaxf(m, mx) : m;
      const float alpha = (m == -INFINITY || mn == m) ? 1.f : ex2(m - mn);
      const float nref = (mn == -INFINITY) ? 0.f : -mn;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float e0 = ex2(fmaf(sv[c + 2 * i], sl2, nref));
          const float e1 = ex2(fmaf(sv[c + 2 * i + 1], sl2, nref));
          s0 += e0;
          s1 += e1;
          const __half2 h2 = __floats2half2_rn(e0, e1);
          pk[i] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        tc_st16(tS + c / 2, pk);
      }
      l = l * alpha + (s0 + s1);
      m = mn;
      if (move && !(flags & 1)) {       // (PV of the tile before is complete: S came behind it)
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
      tc_wait_st();
      tc_fence_before();
      const int r0 = f.r0, g = f.g, dst = f.dst;
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[blk]);
      if (flags & 2) {
        if (!wait_all(&o_full[blk], (uint32_t)seg & 1u)) { ok = false; break; }
        ++seg;
        tc_fence_after();
        const bool row_ok = rt < q.btok && t < ntok;
        const int hq = g * p.G + (r - rt * p.G);
        if (dst < 0 && !p.own) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
          __half* d = p.out + (int64_t)(r0 + t) * p.out_stride + (int64_t)hq * D;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            tc_ld32(tO + c, ov);
            tc_wait_ld();
            if (row_ok) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint4 w;
                __half2* hp = reinterpret_cast<__half2*>(&w);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  hp[e] = __floats2half2_rn(ov[8 * k + 2 * e] * inv, ov[8 * k + 2 * e + 1] * inv);
                *reinterpret_cast<uint4*>(d + c + 8 * k) = w;
              }
            }
          }
        } else {
          const int64_t at = dst < 0 ? (int64_t)(r0 + t) * p.Hq + hq
                                     : ((int64_t)cta * 2 + dst) * p.slot_rows + blk * 128 + r;
          float* d = (dst < 0 ? p.own : p.part) + at * D;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            tc_ld32(tO + c, ov);
            tc_wait_ld();
            if (row_ok) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<float4*>(d + c + 4 * k) =
                    make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
            }
          }
          if (row_ok) (dst < 0 ? p.own_ml : p.ml)[at] = make_float2(m, l);
        }
        tc_fence_before();
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

template <int D, bool kPrefix>
cudaError_t launch_many(const PagedManyParams& p, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.a.nc);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = MSmem<D>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_many_kernel<D, kPrefix>, p);
}

template <int D, bool kPrefix>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(paged_many_kernel<D, kPrefix>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MSmem<D>::kBytes);
}

}  // namespace

cudaError_t launch_paged_sched(const PagedManyParams& p, int64_t* pref, PagedUnit* unit,
                               cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = (size_t)(p.a.B + 1) * sizeof(int);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_sched_kernel, p, pref, unit);
}

cudaError_t launch_paged_many(const PagedManyParams& p, cudaStream_t s, bool pdl) {
  if (p.a.nc < 1 || p.a.nc > 512 || p.units < 1) return cudaErrorInvalidValue;
  if (p.a.D == 128)
    return p.prefix ? launch_many<128, true>(p, s, pdl) : launch_many<128, false>(p, s, pdl);
  if (p.a.D == 64)
    return p.prefix ? launch_many<64, true>(p, s, pdl) : launch_many<64, false>(p, s, pdl);
  return cudaErrorInvalidValue;
}

cudaError_t configure_paged_many() {
  cudaError_t e = configure_one<128, true>();
  if (e == cudaSuccess) e = configure_one<128, false>();
  if (e == cudaSuccess) e = configure_one<64, true>();
  if (e == cudaSuccess) e = configure_one<64, false>();
  return e;
}

}  // namespace blk
