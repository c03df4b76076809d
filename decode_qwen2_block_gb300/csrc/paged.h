// Serving over a paged K/V cache: parameter blocks and launchers of the plan
// (block tables, slot map), append and attention kernels.
//
// Pools: K and V each [n_pages][Hkv][page][D] fp16, page 16, 32, 64 or 128
// slots.  Slot s of a sequence is slot s % page of page block_table[s / page].
// Row t of sequence b (rows row_start[b] .. row_start[b + 1] - 1 of the batch)
// sits in slot cache_lens[b] + t.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace blk {

constexpr int kMaxSeqs = 4096;      // sequences of one batch

// ------------------------------------------------------- plan and append
struct PagePlanParams {
  const int64_t* cache_lens;   // [B]
  const int64_t* new_lens;     // [B], null: one each
  const int32_t* free_pages;   // [n_free]
  int32_t* table;              // [B][max_blocks]
  int64_t* row_start;          // [B + 1]
  int64_t* slot_map;           // [N]
  int64_t* pos;                // [N]
  int64_t* used;               // [1]
  int64_t max_blocks, n_free, N;
  int B, page_lg;
  int* err;
};
cudaError_t launch_page_plan(const PagePlanParams& p, int num_sms, cudaStream_t s, bool pdl);

struct PageAppendParams {
  const __half* k;             // row r, head h at r * row_stride + h * head_stride
  const __half* v;
  int64_t row_stride, head_stride;
  const int64_t* slot_map;     // [N]
  __half* k_pages;
  __half* v_pages;
  int64_t n_slots;             // n_pages * page
  int N, Hkv, D, page_lg;
  int* err;
};
cudaError_t launch_page_append(const PageAppendParams& p, int num_sms, cudaStream_t s, bool pdl);

// -------------------------------------------------------------- attention
// A kernel's CTAs share the batch's K/V tiles evenly: the tiles of every unit
// (a group of rows of one sequence and one kv head) are numbered in one line
// and CTA i takes tiles [i T / n, (i + 1) T / n).  A unit inside one CTA is
// finished there; of a cut unit every CTA leaves a partial (its unnormalised
// O and sum l, fp32, both of 2^(score - m) with the m that it took, in log2 units) in one
// of its two slots: slot 1 of the piece that begins the unit, slot 0 of those that go on.  In the line a unit
// also has a head before its first tile, for what its begin and end cost.
struct alignas(8) PagedPiece { // what merging needs of one cut unit
  int c0;                      // first CTA that holds a piece of it (-1: no unit)
  int rows;                    // partial rows of the unit
  int c1;                      // last CTA that holds a piece
  int r0;                      // batch row of its first token
  int g;                       // kv head
};

struct PagedAttnParams {
  CUtensorMap tm_k, tm_v;      // pools (few rows: boxes of one page or 64 slots, all of D;
                               //   many rows: 64 columns of one page or 128 slots)
  CUtensorMap tm_q;            // many rows: q as (D, Hq, N), box (64, G, tokens)
  const __half* q;             // row r at r * q_stride: [Hq][D]
  int64_t q_stride;
  __half* out;                 // row r at r * out_stride
  int64_t out_stride;
  const int64_t* row_start;    // [B + 1]
  const int64_t* cache_lens;   // [B]
  const int32_t* table;        // [B][max_blocks]
  const int32_t* prefix_pages; // [prefix_len / page] or null
  int64_t max_blocks, n_pages;
  int64_t max_len;             // slots of the longest sequence, new ones with it; it fits the
                               //   table's rows and 31 bits
  int64_t prefix_len;          // every sequence has at least the shared prefix's slots
  int64_t pre_here;            // slots of it that the own parts take with them (their pages from
                               //   prefix_pages); the others belong to the prefix's own launch
  int own_lo;                  // the first slot of the own parts: prefix_len - pre_here
  int window;                  // of the handle; 0: all slots
  int early;                   // few rows: lengths, tables and the slots of the history are
                               //   older than the kernel before this one, which writes q
                               //   and the new slots; nothing else of it is waited for.
                               //   That kernel (qkv_finish_kernel, page_append_kernel) waits
                               //   for its own predecessors before it lets this one start
  int B, N, Hq, Hkv, D, G, page_lg, max_new;
  float scale_log2;
  int nc;                      // CTAs of the kernel
  int slot_rows;               // partial rows of one slot
  float* part;                 // [nc][2][slot_rows][D]
  float2* ml;                  // [nc][2][slot_rows] (m, l)
  PagedPiece* cut;             // [nc]: the unit that begins in CTA i and goes on behind it;
                               //   with upb: [Hkv][B][upb], of every unit (at most nc)
  int upb;                     // units of a sequence at most, if there are entries for all
  // shared prefix: own parts are merged with the prefix's, so whole units
  // leave their (O, m, l) by row and head, and every row says where its own
  // part is
  float* own;                  // [N][Hq][D]
  float2* own_ml;              // [N][Hq]
  int4* row_info;              // [N][Hkv]: c0 (-1 whole, -2 no part), c1, 0, partial row of head 0
                               //   (an attention that timed out leaves entries unwritten: the
                               //   merge takes those that paged_row_part accepts)
  int* err;
};

// Whether a row_info entry names a row's own part: a whole one, or pieces in the slots of
// CTAs c0 .. c1 whose G rows lie in a slot.  Anything else (no part, or what lay in the
// workspace where an attention that timed out wrote no entry) is no part: an address is
// formed from accepted entries only.
__host__ __device__ inline bool paged_row_part(int c0, int c1, int row, int nc, int slot_rows, int G) {
  return c0 == -1 || (c0 >= 0 && c0 <= c1 && c1 < nc && row >= 0 && row <= slot_rows - G);
}

// Rows of one unit that the few-row kernel takes (16 per MMA row tile): at 30 rows it
// takes 29 us for what takes the many-row kernel 35, with 64 rows (four row tiles) it
// was the slower one.
constexpr int kPagedFewRows = 32;
bool paged_few_rows(int G, int64_t max_new);
// CTAs of the kernel and partial rows of a slot.
void paged_few_slots(int num_sms, int G, int64_t max_new, int* nc, int* slot_rows);
cudaError_t launch_paged_few(const PagedAttnParams& p, cudaStream_t s, bool pdl);
cudaError_t configure_paged_few();

// Many rows: prompts and long runs of new tokens, and the shared prefix (its
// rows are the whole batch's).  Units are 2 blocks of 128 / G tokens.
struct PagedManyParams {
  PagedAttnParams a;
  int prefix;                  // 1: the shared prefix's parts, of all N rows
  int btok;                    // tokens of a block
  int units;                   // prefix: units of one kv head
};
inline int paged_btok(int G) { return 128 / G; }
constexpr int kPagedManyRows = 256;     // partial rows of a slot
constexpr int kPagedManyTile = 128;     // slots of a tile
// A unit's begin and end in the line, in tiles (8 prompts, with 1 / 3 / 5: 84 / 81 / 85
// us; they take the time of 1.6, and a piece that the line cuts off takes them again).
constexpr int kPagedManyHead = 3;
cudaError_t launch_paged_many(const PagedManyParams& p, cudaStream_t s, bool pdl);
// `usable` becomes false, and the kernels must not be launched, where the compiler gave one
// another register count than its warps share out.
cudaError_t configure_paged_many(bool* usable);

// Merges cut units (and, with a prefix, every row's own and prefix parts).
struct PagedMergeParams {
  PagedAttnParams a;           // the own parts
  int prefix;                  // 1: merge by rows with the prefix's partials
  int own_btok;                // tokens of a block of 128 partial rows (0: rows lie close)
  const float* pre_part;       // prefix partials [pre_nc][2][pre_rows][D]
  const float2* pre_ml;
  const float* pre_own;        // prefix parts of units inside one CTA, by row and head
  const float2* pre_own_ml;
  int pre_nc, pre_rows, pre_units, pre_tiles, pre_tok, pre_btok;
};
cudaError_t launch_paged_merge(const PagedMergeParams& p, int num_sms, cudaStream_t s);

}  // namespace blk
