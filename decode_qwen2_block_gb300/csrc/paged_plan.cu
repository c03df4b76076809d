// The bookkeeping of a paged K/V cache on the GPU: block tables, slot map and
// positions of a step from the requests' lengths, and the copy of K/V rows
// into their pages (the serving form of the KV append in the decoder block's
// decode phase, §4 "three-phase split": new K/V follow the history).
#include "common.cuh"
#include "paged.h"

namespace blk {
namespace {

constexpr int kPlanThreads = 512;

// Last i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_le(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// One step's plan.  With n_b new tokens after L_b slots, sequence b's rows
// begin at sum of n over the sequences before it, it holds ceil(L_b / page)
// pages and takes ceil((L_b + n_b) / page) less those from the free list,
// beginning behind what the sequences before it took.  Both are sums over the
// sequences, so every CTA forms them in shared memory by itself (B <= 4096
// lengths, a few KB) and fills its share of the slots and table entries: one
// launch, nothing waits on another CTA.  One scan gives both sums, packed in 64
// bits: a sequence whose rows run past N is refused after the scan, but then so is
// every later one with rows, and what it would have taken moves nobody's pages.
// Pages of a row are formed from the lengths and the free list, never read back
// from the table entries that this launch writes.  Bound by latency: 64 decoding
// sequences are one CTA and three round trips to L2, 3.1 - 3.5 us in a graph (with a
// scan each and the lengths read in turn 3.9); 200 prompts with 100,000 slots 4.6.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PagePlanParams p) {
  extern __shared__ int sm[];
  int* rs = sm;                  // [B + 1] first row, at most N
  int* base = sm + p.B + 1;      // [B] first free page taken
  uint8_t* bad = reinterpret_cast<uint8_t*>(base + p.B);   // [B] refused
  __shared__ int64_t warp_sums[kPlanThreads / 32];
  __shared__ int used_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) used_s = 0;
  griddep_wait();
  griddep_launch();
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  const int64_t cap = p.max_blocks << p.page_lg, mask = ((int64_t)1 << p.page_lg) - 1;
  struct Len { int64_t n, L; };
  auto load = [&](int b) { return Len{p.new_lens ? p.new_lens[b] : 1, p.cache_lens[b]}; };
  const Len first = b0 < b1 ? load(b0) : Len{0, 0};
  auto len = [&](int b) { return b == b0 ? first : load(b); };
  auto rows_of = [&](const Len& s) { return s.n < 0 || s.n > p.N ? (int64_t)0 : s.n; };
  // (rows past N apart)
  auto fits = [&](const Len& s) {
    return s.n >= 0 && s.n <= p.N && s.L >= 0 && s.L <= cap && s.L + s.n <= cap;
  };
  auto need_of = [&](const Len& s) {
    return fits(s) ? ((s.L + s.n + mask) >> p.page_lg) - ((s.L + mask) >> p.page_lg) : (int64_t)0;
  };
  // rows (at most 4096 x 2^20) in the low 34 bits, pages (at most 4096 x 2^16 + 4096) above
  constexpr int kPack = 34;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Len s = len(b);
    mine += rows_of(s) + (need_of(s) << kPack);
  }
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t before = x - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const int64_t s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
  constexpr int64_t kRows = ((int64_t)1 << kPack) - 1;
  int64_t r = before & kRows, take = before >> kPack;
  int top = 0;
  bool any_bad = false;
  for (int b = b0; b < b1; ++b) {
    const Len s = len(b);
    const int64_t r1 = r + rows_of(s), need = need_of(s);
    const bool no = !fits(s) || r1 > p.N || (need > 0 && take + need > p.n_free);
    rs[b] = (int)min(r, p.N);
    base[b] = (int)min(take, p.n_free);
    bad[b] = no;
    if (blockIdx.x == 0) p.row_start[b] = r;
    if (!no && need > 0) top = (int)(take + need);
    any_bad |= no;
    r = r1;
    take += need;
  }
  if (tid == 0) {
    rs[p.B] = (int)min(total & kRows, p.N);
    if (blockIdx.x == 0) p.row_start[p.B] = total & kRows;
  }
  if (top > 0) atomicMax(&used_s, top);
  if (any_bad && blockIdx.x == 0) set_error(p.err, kDevPage);
  __syncthreads();
  const int used = used_s;
  if (tid == 0 && blockIdx.x == 0) *p.used = used;
  const int64_t gt = (int64_t)blockIdx.x * kPlanThreads + tid;
  const int64_t gn = (int64_t)gridDim.x * kPlanThreads;
  for (int64_t i = gt; i < p.N; i += gn) {
    int64_t slot = -1, ps = 0;
    if (i < rs[p.B]) {
      const int b = last_le(rs, p.B, (int)i);
      if (!bad[b]) {
        const int64_t L = p.cache_lens[b];
        ps = L + (i - rs[b]);
        const int64_t blkno = ps >> p.page_lg, held = (L + mask) >> p.page_lg;
        const int64_t pg = blkno < held ? p.table[(int64_t)b * p.max_blocks + blkno]
                                        : p.free_pages[base[b] + (blkno - held)];
        slot = pg < 0 ? -1 : (pg << p.page_lg) + (ps & mask);
      }
    }
    p.slot_map[i] = slot;
    p.pos[i] = ps;
  }
  for (int64_t u = gt; u < used; u += gn) {
    const int b = last_le(base, p.B, (int)u);
    const int64_t held = (p.cache_lens[b] + mask) >> p.page_lg;
    p.table[(int64_t)b * p.max_blocks + held + (u - base[b])] = p.free_pages[u];
  }
}

// Copies row r's K and V (Hkv heads of D) to slot slot_map[r].  A thread moves
// the same 16 bytes of K and of V; bound by memory (2 x 2 x Hkv x D x 2 bytes a
// row), kUnroll items in flight per thread.  32761 rows of 2 x 128 from a contiguous
// cache: 11.5 us, 5.8 TB/s read and written (a plain copy reaches 6.8); with one / four /
// eight items a thread 11.9 / 12.1 / 14.6.
constexpr int kUnroll = 2;
__global__ void __launch_bounds__(256) page_append_kernel(const PageAppendParams p) {
  // In this order: the few-row attention of a paged step, launched behind this kernel, reads
  // what is older than it (lengths, tables, the history's slots) ahead of its own wait, and
  // those kernels are complete only because this one has waited before it lets it start.
  griddep_wait();
  griddep_launch();
  const uint32_t cpr = p.D >> 3;                  // 16-byte pieces of a head's row
  const uint32_t per_row = p.Hkv * cpr;
  const int64_t total = (int64_t)p.N * per_row;   // < 2^32: checked by the launcher
  const int64_t step = (int64_t)gridDim.x * 256;
  const int64_t mask = ((int64_t)1 << p.page_lg) - 1;
  for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x; i0 < total; i0 += step * kUnroll) {
    uint4 kv[kUnroll], vv[kUnroll];
    int64_t slot[kUnroll], to[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * step;
      slot[u] = -1;
      if (i < total) {       // the rows are there whatever their slots: nothing waits for these
        const uint32_t r = (uint32_t)i / per_row, e = (uint32_t)i - r * per_row;
        const uint32_t h = e / cpr, c = e - h * cpr;
        slot[u] = p.slot_map[r];
        const int64_t src = (int64_t)r * p.row_stride + h * p.head_stride + c * 8;
        kv[u] = __ldcs(reinterpret_cast<const uint4*>(p.k + src));
        vv[u] = __ldcs(reinterpret_cast<const uint4*>(p.v + src));
        to[u] = ((int64_t)h << p.page_lg) * p.D + c * 8;
        if (slot[u] != -1 && (slot[u] < 0 || slot[u] >= p.n_slots)) {
          if (e == 0) set_error(p.err, kDevPage);
          slot[u] = -1;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (slot[u] >= 0) {
        const int64_t dst =
            (((slot[u] >> p.page_lg) * p.Hkv << p.page_lg) + (slot[u] & mask)) * p.D + to[u];
        *reinterpret_cast<uint4*>(p.k_pages + dst) = kv[u];
        *reinterpret_cast<uint4*>(p.v_pages + dst) = vv[u];
      }
  }
}

template <typename K, typename P>
cudaError_t launch(K kernel, int grid, int threads, size_t smem, cudaStream_t s, bool pdl,
                   const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanParams& p, int num_sms, cudaStream_t s, bool pdl) {
  // a slot a thread while there are SMs (100,000 slots: four a thread 6.8 us, one 5.4)
  const int64_t want = (p.N + kPlanThreads - 1) / kPlanThreads;
  const int grid = (int)(want < 1 ? 1 : (want > num_sms ? num_sms : want));
  const size_t smem = (size_t)(2 * p.B + 1) * sizeof(int) + p.B;   // 36 KB at 4096 sequences
  return launch(page_plan_kernel, grid, kPlanThreads, smem, s, pdl, p);
}

cudaError_t launch_page_append(const PageAppendParams& p, int num_sms, cudaStream_t s, bool pdl) {
  const int64_t total = (int64_t)p.N * p.Hkv * (p.D / 8);
  if (total >= (int64_t)1 << 32) return cudaErrorInvalidValue;
  // two waves of CTAs, so that the second's loads fill the first's ends (one: 12.1 us)
  const int64_t want = (total + 255) / 256, most = (int64_t)num_sms * 16;
  const int grid = (int)(want < 1 ? 1 : (want > most ? most : want));
  return launch(page_append_kernel, grid, 256, 0, s, pdl, p);
}

}  // namespace blk
