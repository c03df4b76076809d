// A paged K/V cache in 8 bits: parameter blocks and launchers.
//
// A row (slot, kv head) of D values is D / 32 blocks of 32 columns.  A block whose
// greatest magnitude is a has the scale
//   s = the least E5M2 number with 127 s / 64 >= a,
// codes c = rint(64 x / s) (ties to even; |c| <= 127), kept as c + 128 in a byte, and
// stands for c s / 64.  An E5M2 number is the upper byte of an fp16 number.  c has 7 bits
// and s 3, and their product's last bit is worth 2^-22 or more: the value is an fp16
// number, so reading a block back, and the attention's use of it, round nothing.
// A block with an infinity or a NaN has the scale NaN: all of it reads as NaN.
//
// Pools: codes K and V each [n_pages][Hkv][page][D] bytes, scales [n_pages][Hkv][page][D / 32].
#pragma once

#include "paged.h"

namespace blk {

constexpr int kKv8Block = 32;       // columns of a scale

struct Kv8Pools {
  uint8_t *k, *v;              // codes
  uint8_t *ks, *vs;            // scales
};

struct Kv8AppendParams {
  const __half* k;             // row r, head h at r * row_stride + h * head_stride
  const __half* v;
  int64_t row_stride, head_stride;
  const int64_t* slot_map;     // [N]
  Kv8Pools to;
  int64_t n_slots;             // n_pages * page
  int N, Hkv, D, page_lg;
  int* err;
};
cudaError_t launch_kv8_append(const Kv8AppendParams& p, int num_sms, cudaStream_t s, bool pdl);

struct Kv8ReadParams {
  __half* k;                   // row r, head h at r * row_stride + h * head_stride
  __half* v;
  int64_t row_stride, head_stride;
  const int64_t* slot_map;     // [N]
  Kv8Pools from;
  int64_t n_slots;
  int N, Hkv, D, page_lg;
  int* err;
};

// Whether rows that the read writes lie over each other, and several threads would write one
// place: rows of D values at r * row_stride + h * head_stride (r < n, h < H), and the same `apart`
// elements further (V's from K's).  Heads may lie within rows or rows within heads; the span of
// what lies within fits the stride of the other.
inline bool kv8_rows_meet(int64_t n, int64_t H, int64_t row_stride, int64_t head_stride, int64_t D,
                          int64_t apart) {
  int64_t a = head_stride, na = H, b = row_stride, nb = n;          // within, around
  if (n > 1 && (H == 1 || row_stride < (H - 1) * head_stride + D)) {
    a = row_stride, na = n;
    b = head_stride, nb = H;
  }
  if ((na > 1 && a < D) || (nb > 1 && b < (na > 1 ? (na - 1) * a : 0) + D)) return true;
  // a row of one over a row of the other: |apart - i a - j b| < D for some |i| < na, |j| < nb,
  // and with |i a| + D <= b only the two j around apart / b can give that
  const int64_t d = apart < 0 ? -apart : apart;
  const int64_t j0 = nb > 1 ? d / b : 0;
  for (int64_t j = j0; j < nb && j <= j0 + 1; ++j) {
    const int64_t rest = d - (nb > 1 ? j * b : 0), at = rest < 0 ? -rest : rest;
    const int64_t i = na > 1 ? at / a : 0, left = at - (na > 1 ? i * a : 0);
    if (i < na && left < D) return true;
    if (na > 1 && i + 1 < na && a - left < D) return true;
  }
  return false;
}

cudaError_t launch_kv8_read(const Kv8ReadParams& p, int num_sms, cudaStream_t s, bool pdl);

// Attention over such pools: the kernels of paged.h over codes and scales.
// Few rows (paged_few_rows): as launch_paged_few, the merge of cut units behind it.
// Up to 8 kKv8NarrowTiles rows and more run on different shapes of the kernel; kv8_few_tile:
// slots of a tile.
constexpr int kKv8NarrowTiles = 2;
inline bool kv8_few_wide(int G, int64_t max_new) { return max_new * G > 8 * kKv8NarrowTiles; }
constexpr int kv8_few_tile(int D, bool wide) { return (D == 128 ? 64 : 128) << wide; }
struct PagedFew8Params {
  PagedAttnParams a;           // tm_k, tm_v: codes, boxes of all columns of a page's slots, a
                               //   tile's at most
  const uint8_t *ks, *vs;      // scales
};
void paged_few_kv8_slots(int num_sms, int G, int64_t max_new, int* nc, int* slot_rows);
cudaError_t launch_paged_few_kv8(const PagedFew8Params& p, cudaStream_t s, bool pdl);
// `wide` becomes false, and the shape for more rows must not be launched, where the compiler
// gave it another register count than its warps share out.
cudaError_t configure_paged_few_kv8(bool* wide);


// Many rows: as launch_paged_many (tm_k, tm_v: codes, boxes of all columns of one page).
struct PagedMany8Params : PagedManyParams {
  const uint8_t *ks, *vs;      // scales
};
cudaError_t launch_paged_many_kv8(const PagedMany8Params& p, cudaStream_t s, bool pdl);
cudaError_t configure_paged_many_kv8(bool* usable);

}  // namespace blk
