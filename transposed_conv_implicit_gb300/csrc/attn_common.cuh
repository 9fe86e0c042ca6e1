// Device code shared by the attention kernels: rounding, barriers, and the
// ways a call's work is cut between CTAs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "attn_params.h"
#include "attn_ptx.cuh"
#include "conv_params.h"

namespace convgb300 {

template <typename T>
__device__ __forceinline__ uint32_t round2(float a, float b);
template <>
__device__ __forceinline__ uint32_t round2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t round2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// bar.sync over `count` threads that also ANDs a predicate across them.
__device__ __forceinline__ bool barrier_all(uint32_t id, uint32_t count, bool v) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(count)
      : "memory");
  return out != 0;
}

// Barriers that a warp waits for together, a lane for each: a wait beside
// running 128 x 128 products from shared memory takes some 300 cycles, whether
// the barrier is through or not (the products take all of the bandwidth), and
// one set takes no more.  The lanes poll in step: where they left the loop one
// by one, the warp's products afterwards issued at half their rate (the forward
// pass at 2 x 16 heads, 16384 x 4096 x 128: 1819 us, in step 768).
struct WaitSet {
  uint32_t bar, parity, lane;
  __device__ WaitSet(uint64_t* b, uint32_t q, int at) : bar(smem_u32(b)), parity(q), lane(at & 7) {}
  template <int i>
  __device__ void also(uint64_t* b, uint32_t q, bool on = true) {
    if (on && lane == i) {
      bar = smem_u32(b);
      parity = q;
    }
  }
};

__device__ __forceinline__ bool wait_set_bounded(const WaitSet& s, volatile int* abort_flag,
                                                 unsigned int* status, unsigned int code,
                                                 long long limit_cycles) {
  const auto through = [&]() { return __all_sync(0xFFFFFFFFu, mbar_try_wait(s.bar, s.parity)); };
  if (through()) return true;
  const long long t0 = cycle_count();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
      if (through()) return true;
    if (__any_sync(0xFFFFFFFFu, *abort_flag)) return false;
    if (__any_sync(0xFFFFFFFFu, cycle_count() - t0 > limit_cycles)) {
      if ((threadIdx.x & 31) == 0) {
        atomicOr(status, code);
        *abort_flag = 1;
      }
      __syncwarp();
      return false;
    }
  }
}

__device__ __forceinline__ int valid_keys(const AttnShape& a, int b) {
  return a.kv_lengths ? max(0, min(a.kv_lengths[b], a.kv_len)) : a.kv_len;
}

// Key tiles of a row with n keys; a row without keys takes one, fully masked.
__device__ __forceinline__ int key_tiles(int n, int box) { return n > box ? (n + box - 1) / box : 1; }

// A split launch's shares: CTA c takes steps [total * c / ctas, total * (c + 1) / ctas).
__device__ __forceinline__ long long share_begin(long long total, int ctas, int c) {
  return total * c / ctas;
}
// The CTA whose share holds step s.
__device__ __forceinline__ int share_of(long long total, int ctas, long long s) {
  return static_cast<int>(((s + 1) * ctas - 1) / total);
}

// Where a CTA's share begins.
struct SplitStart {
  long long left;  // steps of this CTA
  long long rest;  // steps of batch b before the share
  int b;
};

// One warp: this CTA's share of the steps of all batches, steps(b) each, or
// `uniform` each when that is not negative.  (Each lane sums some batches.)
template <typename F>
__device__ SplitStart split_start(int batch, long long uniform, int lane, F steps) {
  SplitStart st{};
  long long total = 0;
  if (uniform >= 0) {
    total = uniform * batch;
  } else {
    for (int b = lane; b < batch; b += 32) total += steps(b);
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  }
  const long long lo = share_begin(total, gridDim.x, blockIdx.x);
  st.left = share_begin(total, gridDim.x, blockIdx.x + 1) - lo;
  st.rest = lo;
  if (st.left == 0) return st;
  if (uniform >= 0) {
    st.b = static_cast<int>(lo / uniform);
    st.rest -= st.b * uniform;
    return st;
  }
  for (int b0 = 0; b0 < batch; b0 += 32) {
    const int b = b0 + lane;
    const long long mine = b < batch ? steps(b) : 0ll;
    long long upto = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > st.rest);
    if (past) {
      const int at = __ffs(past) - 1;
      st.b = b0 + at;
      st.rest -= __shfl_sync(0xFFFFFFFFu, upto - mine, at);
      return st;
    }
    st.rest -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  return st;
}

// Block-wide: steps of all batches and of those before b.  `sums`: 2 x warps.
template <typename F>
__device__ void split_prefix(int batch, long long uniform, int b, long long (*sums)[32], F steps,
                             long long* before, long long* total) {
  if (uniform >= 0) {
    *before = uniform * b;
    *total = uniform * batch;
    return;
  }
  long long t = 0, u = 0;
  for (int i = threadIdx.x; i < batch; i += blockDim.x) {
    const long long v = steps(i);
    t += v;
    if (i < b) u += v;
  }
  for (int o = 16; o; o >>= 1) {
    t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
  }
  if ((threadIdx.x & 31) == 0) {
    sums[0][threadIdx.x >> 5] = t;
    sums[1][threadIdx.x >> 5] = u;
  }
  __syncthreads();
  *total = *before = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) {
    *total += sums[0][i];
    *before += sums[1][i];
  }
}

// Row tiles (forward, dq): a batch has item_rows items of its key tiles each.
template <typename P>
__device__ __forceinline__ long long row_steps(const P& p, int b) {
  return key_tiles(valid_keys(p.a, b), p.kv_box) * p.item_rows;
}
template <typename P>
__device__ __forceinline__ long long row_steps_uniform(const P& p) {
  return p.a.kv_lengths ? -1 : key_tiles(p.a.kv_len, p.kv_box) * p.item_rows;
}
template <typename P>
__device__ SplitStart split_rows(const P& p, int lane) {
  return split_start(p.a.batch, row_steps_uniform(p), lane, [&](int b) { return row_steps(p, b); });
}

// Whether a split launch cuts no item: a CTA then takes the items that begin in
// its share.
__device__ __forceinline__ bool whole_items(const AttnFwdParams&) { return false; }
__device__ __forceinline__ bool whole_items(const AttnBwdParams& p) { return p.q_whole; }

// Walks a CTA's work: every role walks the same sequence.
template <bool kSplit, bool kMask, typename P>
struct Walk {
  const P& p;
  long long pos;       // pairs: item index; split: steps left after this item
  int b, hk, row_tile; // row_tile: the first of the item's row tiles
  int tiles_here;      // row tiles of the item
  int n;               // valid keys
  int t0, t1, nt;      // key tiles [t0, t1) of nt
  uint32_t act;        // tiles from act_base on that are worked on (with a mask)
  int act_base;
  bool live;

  __device__ Walk(const P& params, const SplitStart& st) : p(params) {
    if constexpr (kSplit) {
      b = st.b;
      pos = st.left;
      live = pos > 0;
      if (live) {
        const int per = key_tiles(valid_keys(p.a, b), p.kv_box);
        const int item = static_cast<int>(st.rest / per);
        const int tile = static_cast<int>(st.rest - static_cast<long long>(item) * per);
        set_split(item, tile);
        if (whole_items(p) && tile > 0) {  // an item that began in another share
          pos = st.left - (per - tile);
          next();
        }
      }
    } else {
      pos = blockIdx.x;
      set_pair();
    }
  }
  __device__ void set_split(int item, int tile) {
    n = valid_keys(p.a, b);
    nt = key_tiles(n, p.kv_box);
    hk = item / p.row_tiles;
    row_tile = item - hk * p.row_tiles;
    tiles_here = 1;
    t0 = tile;
    t1 = whole_items(p) ? nt : static_cast<int>(min(static_cast<long long>(nt), tile + pos));
    pos -= t1 - t0;
  }
  __device__ void set_pair() {
    if constexpr (!kSplit) {
      live = pos < p.items;
      if (!live) return;
      const int item = static_cast<int>(pos);
      const int bh = fast_div(item, p.div_pairs);
      row_tile = 2 * (item - bh * static_cast<int>(p.div_pairs.d));
      b = fast_div(bh, p.div_kv_heads);
      hk = bh - b * p.a.kv_heads;
      tiles_here = min(2, p.row_tiles - row_tile);
      n = valid_keys(p.a, b);
      nt = key_tiles(n, p.kv_box);
      t0 = 0;
      t1 = nt;
    }
  }
  __device__ void next() {
    if (kSplit) {
      live = pos > 0;
      if (!live) return;
      int item = hk * p.row_tiles + row_tile + 1;
      if (item == p.item_rows) {
        item = 0;
        ++b;
      }
      set_split(item, 0);
    } else {
      pos += gridDim.x;
      set_pair();
    }
  }
  // First token and head of row tile `row_tile + g`.
  __device__ void place(int g, int* token, int* head) const {
    const int rt = row_tile + g;
    if (p.tile_heads > 1) {
      *token = rt * p.tile_tokens;
      *head = hk * p.a.group;
    } else {
      const int hg = fast_div(rt, p.div_token_tiles);
      *token = (rt - hg * p.token_tiles) * kAttnRows;
      *head = hk * p.a.group + hg;
    }
  }
  // Keys of tile t that some row of the item's tiles may attend, by the mask
  // (of all queries of the tiles of 128 that the rows lie in).
  __device__ uint4 any_keys(int t) const {
    const AttnShape& a = p.a;
    uint4 any = make_uint4(0, 0, 0, 0);
    for (int g = 0; g < tiles_here; ++g) {
      int token, head;
      place(g, &token, &head);
      const int q0 = a.any_q ? token >> 7 : 0;
      const int q1 = a.any_q ? (min(token + p.tile_tokens, a.q_len) - 1) >> 7 : 0;
      const int heads = a.any_h ? p.tile_heads : 1;
      for (int h = head; h < head + heads; ++h)
        for (int q = q0; q <= q1; ++q) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              a.mask_any + (b * a.any_b + h * a.any_h + q * a.any_q) * a.mask_words + (t * p.kv_box >> 5));
          any.x |= v.x;
          any.y |= v.y;
          any.z |= v.z;
          any.w |= v.w;
        }
    }
    return any;
  }
  // The key tiles of [t0, t1) that are worked on, in order: all, or with a
  // mask those that some row attends (the first one if there is none).  Every
  // lane of a warp calls these together.
  __device__ int first() {
    act = 0;
    act_base = t0;
    if (!kMask || t1 - t0 == 1) return t0;
    const int t = search(t0);
    return t < t1 ? t : t0;
  }
  __device__ int after(int t) {
    if (!kMask || t1 - t0 == 1) return t + 1;
    const int at = t - act_base;
    const uint32_t rest = static_cast<uint32_t>(at) < 31u ? act & (0xFFFFFFFEu << at) : 0u;
    return rest ? act_base + __ffs(rest) - 1 : search(act_base + 32);
  }
  __device__ int search(int from) {
    for (act_base = from; act_base < t1; act_base += 32) {
      const int t = act_base + (threadIdx.x & 31);
      bool on = false;
      if (t < t1) {
        const uint4 v = any_keys(t);
        on = (v.x | v.y | v.z | v.w) != 0;
      }
      act = __ballot_sync(0xFFFFFFFFu, on);
      if (act) return act_base + __ffs(act) - 1;
    }
    return t1;
  }
  // Keys of tile t that are valid, and the columns multiplied for them.
  __device__ int tile_keys(int t) const { return max(0, min(p.kv_box, n - t * p.kv_box)); }
  __device__ int tile_cols(int t) const { return max(16, (tile_keys(t) + 15) & ~15); }
};

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

// The forward pass holds P times 2^kShift (the running maximum in log2 units,
// `mc`, is less by it), and its sums with it.  In fp16 P then reaches 2^15 (the
// maximum may lag by 2^8), so that probabilities far below a row's largest are not
// rounded among the type's subnormal numbers.  (No more: the exponent's argument
// is rounded at the shift's size, 1.7e-7 of P here.)
template <typename T>
constexpr float kShift = std::is_same<T, __half>::value ? 7.f : 0.f;

template <typename T>
__device__ __forceinline__ float row_lse(float mc, float l) {
  return fmaf(mc + kShift<T>, kLn2, logf(l * exp2f(-kShift<T>)));
}

// Floats of a tile of 128 queries in the statistics: minus lse, minus delta, and in
// fp16 |do|^2.
template <typename T>
constexpr int kStatPitch = std::is_same<T, __half>::value ? 384 : 256;

// fp16: ds is rounded after a scaling by a power of two, so that it does not
// leave the type's range on either side.  |ds_ij| <= 2 |do_i| max |v|, over the
// values of the request's key head.  dq_i sums over the keys only: every query
// has a scale of its own.  dk sums over the queries: one scale for a thread
// block's share of a key head's queries, taken out again before the shares meet.
//
// The largest of n squares, 0 without any.  One warp.
__device__ __forceinline__ float largest(const float* v, int n, int lane) {
  float x = 0.f;
#pragma unroll 8
  for (int i = lane; i < n; i += 32) x = fmaxf(x, v[i]);
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)));  // (as bits they are in order)
}
// The largest |v|^2 of a request's key head, and |do|^2 of its queries' steps
// [i0, i1) (tiles of 128 tokens, over the query heads that share it).
__device__ __forceinline__ float largest_value(const AttnBwdParams& p, int b, int hk, int lane) {
  return largest(p.value_norms + (static_cast<long long>(b) * p.a.kv_heads + hk) * p.key_groups,
                 p.key_groups, lane);
}
__device__ __forceinline__ float largest_row(const AttnBwdParams& p, int b, int hk, int i0, int i1, int lane) {
  const int per = kAttnRows / (kAttnRowUnroll * p.row_slots);  // entries of a tile
  return largest(p.row_norms + ((static_cast<long long>(b) * p.a.heads + hk * p.a.group) * p.q_tiles + i0) * per,
                 (i1 - i0) * per, lane);
}
// The power of two for |do|^2 <= x and |v|^2 <= y: |ds| 2^k <= 2^15.  By the
// exponents alone: x y < 2^e, so 2 |do| |v| < 2^(1 + ceil(e / 2)).  (Squares of
// fp16 numbers and their sums are normal, and k is within +-61.)
__device__ __forceinline__ float ds_scale(float x, float y) {
  if (x == 0.f || y == 0.f) return 1.f;
  const int e = (__float_as_int(x) >> 23) + (__float_as_int(y) >> 23) - 2 * 126;
  return __int_as_float((127 + 14 - ((e + 1) >> 1)) << 23);
}

// Clears the rows of a tile (kBlocks blocks of 128-byte rows) below `limit`
// whose bit of `keep` is not set.  One warp, four rows a store: a lane per row
// took ten times as long, its stores meeting in the same banks.
template <int kBlocks>
__device__ __forceinline__ void clear_rows(uint8_t* tile, uint32_t block_bytes, int limit, uint4 keep,
                                           int lane) {
  const uint32_t words[4] = {keep.x, keep.y, keep.z, keep.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (words[i] == 0xFFFFFFFFu) continue;
    for (int r0 = lane >> 3; r0 < 32; r0 += 4) {
      const int r = i * 32 + r0;
      if (r < limit && !((words[i] >> r0) & 1u))
#pragma unroll
        for (int c = 0; c < kBlocks; ++c)
          *reinterpret_cast<uint4*>(tile + c * block_bytes + r * 128 + (lane & 7) * 16) =
              make_uint4(0, 0, 0, 0);
    }
  }
}

// The first n of 128 keys.
__device__ __forceinline__ uint4 first_keys(int n) {
  const auto word = [n](int i) {
    const int rest = n - i * 32;
    return rest >= 32 ? 0xFFFFFFFFu : rest <= 0 ? 0u : (1u << rest) - 1u;
  };
  return make_uint4(word(0), word(1), word(2), word(3));
}

// Writes 32 fp32 columns of a row, scaled: rounded to T.
template <typename T>
__device__ __forceinline__ void store_cols(T* dst, const uint32_t* v, int n, float f) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    if (i < n) {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[j] = round2<T>(__uint_as_float(v[i + 2 * j]) * f, __uint_as_float(v[i + 2 * j + 1]) * f);
      *reinterpret_cast<uint4*>(dst + i) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}
__device__ __forceinline__ void store_cols_f32(float* dst, const uint32_t* v, int n, float f) {
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    if (i < n)
      *reinterpret_cast<float4*>(dst + i) =
          make_float4(__uint_as_float(v[i]) * f, __uint_as_float(v[i + 1]) * f,
                      __uint_as_float(v[i + 2]) * f, __uint_as_float(v[i + 3]) * f);
}

// Joining the shares of tiles that a launch cut: one block takes kJoinRows
// rows of a tile, each warp kJoinUnroll at a time, and the shares' slots are
// listed once per block, so that the rows' reads are all in flight together
// (with the slots found row by row, in 64-bit divisions, the join of a 1021 x
// 523 training pass took 112 us).
constexpr int kJoinRows = 32, kJoinUnroll = 4, kJoinThreads = 256;
constexpr int kMaxShares = 320;  // CTAs of a launch: two per SM at most

struct JoinSlots {
  long long sums[2][32];
  int slots[kMaxShares];
  int count;  // 0: the tile was written whole
};

// Slots of the shares of steps [s0, s0 + steps) of `total`, in order.
__device__ __forceinline__ void list_slots(JoinSlots& j, long long total, int ctas, long long s0,
                                           long long steps) {
  __shared__ int range[2];
  if (threadIdx.x == 0) {
    range[0] = share_of(total, ctas, s0);
    range[1] = share_of(total, ctas, s0 + steps - 1);
    j.count = 0;
  }
  __syncthreads();
  const int c0 = range[0], c1 = range[1];
  if (c0 == c1) return;
  if (total >= ctas) {  // every CTA has a share
    for (int c = c0 + threadIdx.x; c <= c1; c += blockDim.x)
      j.slots[c - c0] = 2 * c + (c == c0 ? 1 : 0);
    if (threadIdx.x == 0) j.count = c1 - c0 + 1;
  } else if (threadIdx.x == 0) {
    int n = 0;
    for (int c = c0; c <= c1; ++c)
      if (share_begin(total, ctas, c) != share_begin(total, ctas, c + 1))
        j.slots[n++] = 2 * c + (c == c0 ? 1 : 0);
    j.count = n;
  }
  __syncthreads();
}

}  // namespace convgb300
