// Device code shared by the tree attention's kernels: a request's sizes, the
// walk over a CTA's share, the drafts that a row attends.
#pragma once

#include <cstdint>

#include "attn_common.cuh"
#include "tree_params.h"

namespace convgb300 {

struct TreeSize {
  int keys, drafts;
};

__device__ __forceinline__ TreeSize tree_size(const TreeParams& p, int b) {
  TreeSize s;
  s.keys = max(0, min(p.kv_lengths[b], p.c.table_width * p.c.page_size));
  s.drafts = min(p.draft_lengths ? max(0, min(p.draft_lengths[b], p.q_len)) : p.q_len, s.keys);
  return s;
}
__device__ __forceinline__ int tree_row_tiles(const TreeParams& p, const TreeSize& s) {
  return (s.drafts * p.group + p.tile_rows - 1) / p.tile_rows;
}
__device__ __forceinline__ int tree_key_tiles(const TreeSize& s) {
  return (s.keys + kTreeKeys - 1) / kTreeKeys;
}
__device__ __forceinline__ long long tree_steps(const TreeParams& p, int b) {
  const TreeSize s = tree_size(p, b);
  return static_cast<long long>(tree_row_tiles(p, s)) * tree_key_tiles(s) * p.kv_heads;
}

// The items of a CTA's share, in order.  Row tiles of a key head follow one
// another, so that CTAs side by side read the same keys.
struct TreeWalk {
  const TreeParams& p;
  long long left;  // steps after this item
  int b, item;
  TreeSize size;
  int row_tiles, nt;
  int hk, row_tile, t0, t1;  // key tiles [t0, t1) of nt
  bool live;

  __device__ TreeWalk(const TreeParams& params, const SplitStart& st) : p(params) {
    b = st.b;
    left = st.left;
    live = left > 0;
    if (!live) return;
    request();
    item = static_cast<int>(st.rest / nt);
    place(static_cast<int>(st.rest - static_cast<long long>(item) * nt));
  }
  __device__ void request() {
    size = tree_size(p, b);
    row_tiles = tree_row_tiles(p, size);
    nt = tree_key_tiles(size);
  }
  __device__ void place(int tile) {
    hk = item / row_tiles;
    row_tile = item - hk * row_tiles;
    t0 = tile;
    t1 = static_cast<int>(min(static_cast<long long>(nt), tile + left));
    left -= t1 - t0;
  }
  __device__ void next() {
    live = left > 0;
    if (!live) return;
    if (++item == p.kv_heads * row_tiles) {
      item = 0;
      do {  // (requests without drafts have no steps)
        ++b;
        request();
      } while (row_tiles == 0);
    }
    place(0);
  }
  __device__ bool whole() const { return t0 == 0 && t1 == nt; }
};

// The drafts that draft i attends, as bits: itself and, with `parents` (a
// shared copy of the request's), those on its way to the root; without, all up
// to it.  A way only goes to smaller numbers, so it ends.
__device__ __forceinline__ void draft_bits(const int* parents, int i, uint32_t (&bits)[kTreeWords]) {
#pragma unroll
  for (int w = 0; w < kTreeWords; ++w) {
    const int upto = i - 32 * w;  // the word's last bit
    bits[w] = parents || upto < 0 ? 0u : upto >= 31 ? 0xFFFFFFFFu : (2u << upto) - 1u;
  }
  if (!parents) return;
  for (int at = i;;) {
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w)
      if (at >> 5 == w) bits[w] |= 1u << (at & 31);
    const int up = parents[at];
    if (up < 0 || up >= at) return;
    at = up;
  }
}

// A power of two for a query's row, so that its largest element is in [2^14,
// 2^15) as fp16: the factor, and what takes it out again.  (fp16 rows keep
// theirs.)
template <typename T>
__device__ __forceinline__ float row_factor(float top, float* back) {
  if constexpr (std::is_same<T, __half>::value) {
    *back = 1.f;
    return 1.f;
  }
  // top = m 2^k: 2^(14 - k), within fp32's normal numbers.
  const int k = static_cast<int>(__float_as_uint(top) >> 23) - 127;
  const int f = top > 0.f && top < INFINITY ? max(-113, min(14 - k, 126)) : 0;
  *back = __int_as_float((127 - f) << 23);
  return __int_as_float((127 + f) << 23);
}

// Two bf16 numbers: the larger magnitude, and both times `up` as fp16.
__device__ __forceinline__ float larger_of(uint32_t v) {
  return fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xFFFF0000u)));
}
__device__ __forceinline__ uint32_t to_half(uint32_t v, float up) {
  return round2<__half>(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
}

// y = (score in log2 units) + (exponent of the value's scale): probabilities
// are held as 2^(y - maximum + kTreeShift), see tree_few.cu.  The maximum may
// lag by kTreeLag, so they stay within 2^15; small ones are rounded in steps of
// 2^-28 of the largest at worst.  (Rescaling costs a row's whole output: scores
// of cached keys that differ in size grow by 2^8 now and then, hardly by 2^11.)
constexpr float kTreeShift = 4.f, kTreeLag = 11.f;

}  // namespace convgb300
