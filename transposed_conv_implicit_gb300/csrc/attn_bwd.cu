// Cross attention backward on the tensor cores.
//
//   p_ij = exp(s_ij - lse_i),  dv_j = sum_i p_ij do_i,  dp_ij = do_i . v_j
//   ds_ij = p_ij (dp_ij - delta_i),  delta_i = do_i . o_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
//
// Three kernels, none with atomics, so that every sum has a fixed order:
//  - rows: delta and the statistics of every query (bound by reading do, o);
//  - dq: a row tile of 128 (token, head) rows stays, key tiles stream by.
//    S = q k^T and dp = do v^T (lanes = queries) land in TMEM, ds replaces dp
//    there and is the A operand of dq += ds k: three products per tile.  S is
//    free once it is read and dp has two buffers, so that both are ready when
//    the exponentials come to them;
//  - dk, dv: 128 keys stay, query tiles stream by, over all query heads that
//    share the key head.  S^T = k q^T and dp^T = v do^T (lanes = keys), so
//    that p^T and ds^T are A operands in TMEM where they are made: dv += p^T
//    do, dk += ds^T q: four products per tile.
// The scores are multiplied twice (seven products where five would do): the
// price of dq and dk, dv each summing in registers of their own CTA, without
// adding fp32 partial sums of dq through L2 once per key tile.
//
// 2 x 16 heads, 8192 x 2048 x 128 (bound by the products): rows 27 us (5.0
// TB/s), dq 254 (1.62 PFLOP/s), dk and dv 350 (1.57 PFLOP/s), joins 31.  What
// held the products back were waits: products of 128 x 128 from shared memory
// take all of its bandwidth, and an mbarrier that is looked at beside them
// answers after some 300 cycles.  16 softmax warps (a quarter of the columns
// each) take 3 % less than 8.
//
// Each kernel's (tile, step) sequence is cut into equal shares, one per SM,
// unless whole tiles even out;
// the tiles that a share boundary cuts go through fp32 partial sums, which a
// last kernel adds in order.  Rows that take no part are cleared in shared
// memory before a product sums over them.
//
// p and ds are rounded to the inputs' type.  In fp16 both are scaled by
// powers of two first: p <= 1 by 2^15, and ds by what the norms of do and v
// allow, for dq row by row and for dk by shares of a key head's queries
// (attn_common.cuh); the results are scaled back in fp32.  (With one scale for
// the whole call, rows of do 2^16 smaller than the largest lost 0.4 % of dq at
// 2048 keys.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "attn_common.cuh"
#include "attn_internal.h"
#include "attn_params.h"

namespace convgb300 {

namespace {

constexpr int kMaxRing = 8;

// ------------------------------------------------------------------ rows
template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t v);
template <>
__device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 widen2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

template <typename T>
__device__ __forceinline__ float dot8(uint4 x, uint4 y) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = widen2<T>(a[i]), v = widen2<T>(b[i]);
    s = fmaf(u.x, v.x, s);
    s = fmaf(u.y, v.y, s);
  }
  return s;
}

// With more than one tile of keys, delta is taken from the rounded output, which
// leaves ds an error of the output's rounding, for a pass over the keys that is
// saved (one tile: the dq kernel sums it and puts it in).
// stats[b][h][token tile][2][128]: minus lse in log2 units, plus p_shift (-inf
// for queries without keys and past the end, which makes p zero), and minus
// delta: as the products' sums take them.  In fp16 also |do|^2, and the largest
// ones of every warp's rows of do and of v.  Rows of do without keys and of v
// without queries count as zeros, and so do rows that are not finite: their
// gradients are not, either.
template <typename T>
__global__ void __launch_bounds__(256) attn_rows_kernel(const __grid_constant__ AttnBwdParams p) {
  constexpr bool kNorms = std::is_same<T, __half>::value;
  const AttnShape& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Power-of-two lanes per row, 16 bytes each; a warp takes kAttnRowUnroll x slots
  // neighbouring tokens of one head (no more than 128), so that its statistics
  // fill whole sectors.
  const int words = a.head_dim >> 3;
  const int width = 32 / p.row_slots;
  const int at = lane & (width - 1), slot = lane / width;
  const int group = kAttnRowUnroll * p.row_slots;
  grid_dependency_wait();
  grid_launch_dependents();
  const bool values = blockIdx.x >= static_cast<unsigned>(p.row_blocks);
  const int block = values ? blockIdx.x - p.row_blocks : blockIdx.x;
  const int blocks = values ? gridDim.x - p.row_blocks : p.row_blocks;
  const int heads = values ? a.kv_heads : a.heads;
  const int groups = values ? p.key_groups : p.q_tiles * kAttnRows / group;
  const FastDiv div_heads = values ? p.div_kv_heads : p.div_heads;
  const FastDiv div_groups = values ? p.div_key_groups : p.div_groups;
  const int units = groups * heads * a.batch;  // heads innermost, then tokens
  for (int unit = block * 8 + warp; unit < units; unit += blocks * 8) {
    const int bt = fast_div(unit, div_heads), h = unit - bt * heads;
    const int b = fast_div(bt, div_groups), part = bt - b * groups, t0 = part * group + slot;
    const int length = values ? valid_keys(a, b) : a.q_len;
    const long long row0 = (static_cast<long long>(b) * a.heads + h) * a.q_len;
    // Keys of the tile of 128 around t0 that some query of the key head attends.
    uint4 used = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (kNorms && values && a.mask_bits) {
      const int rows = (a.any_h ? a.group : 1) * (a.any_q ? p.q_tiles : 1);
      used = make_uint4(0u, 0u, 0u, 0u);
      for (int i = lane; i < rows; i += 32) {
        const int hg = a.any_q ? i / p.q_tiles : i, qt = a.any_q ? i - hg * p.q_tiles : 0;
        const uint4 v = *reinterpret_cast<const uint4*>(
            a.mask_any + (b * a.any_b + (h * a.group + hg) * a.any_h + qt * a.any_q) * a.mask_words + (t0 >> 7) * 4);
        used.x |= v.x;
        used.y |= v.y;
        used.z |= v.z;
        used.w |= v.w;
      }
      used.x = __reduce_or_sync(0xFFFFFFFFu, used.x);
      used.y = __reduce_or_sync(0xFFFFFFFFu, used.y);
      used.z = __reduce_or_sync(0xFFFFFFFFu, used.z);
      used.w = __reduce_or_sync(0xFFFFFFFFu, used.w);
    }
    uint4 x[kAttnRowUnroll], y[kAttnRowUnroll];
    float lse[kAttnRowUnroll];
#pragma unroll
    for (int u = 0; u < kAttnRowUnroll; ++u) {
      const int t = t0 + u * p.row_slots;
      x[u] = y[u] = make_uint4(0, 0, 0, 0);
      lse[u] = -INFINITY;
      if (t >= length || at >= words) continue;
      if (values) {
        x[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + b * a.vs[0] + t * a.vs[1] +
                                               h * a.vs[2] + at * 8);
      } else {
        x[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.dout) + b * a.dos[0] +
                                               t * a.dos[1] + h * a.dos[2] + at * 8);
        if (a.kv_len > p.kv_box)
          y[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.out) + b * a.os[0] +
                                                 t * a.os[1] + h * a.os[2] + at * 8);
        if (at == 0) lse[u] = a.lse[row0 + t];
      }
    }
    float dot[kAttnRowUnroll], sq[kAttnRowUnroll];
#pragma unroll
    for (int u = 0; u < kAttnRowUnroll; ++u) {
      dot[u] = dot8<T>(x[u], y[u]);
      sq[u] = kNorms ? dot8<T>(x[u], x[u]) : 0.f;
    }
    for (int o = width >> 1; o; o >>= 1)
#pragma unroll
      for (int u = 0; u < kAttnRowUnroll; ++u) {
        dot[u] += __shfl_xor_sync(0xFFFFFFFFu, dot[u], o);
        if (kNorms) sq[u] += __shfl_xor_sync(0xFFFFFFFFu, sq[u], o);
      }
    if (!kNorms && at != 0) continue;
    float norm = 0.f;
#pragma unroll
    for (int u = 0; u < kAttnRowUnroll; ++u) {
      const int t = t0 + u * p.row_slots;
      if (kNorms) {
        const int bit = t & 127;
        const uint32_t word = bit < 32 ? used.x : bit < 64 ? used.y : bit < 96 ? used.z : used.w;
        if (!(sq[u] < INFINITY) || !((word >> (bit & 31)) & 1u)) sq[u] = 0.f;  // (NaN compares false)
      }
      if (at == 0 && !values) {
        const float lse2 = lse[u] == -INFINITY ? lse[u] : p.p_shift - lse[u] * kLog2e;
        if (lse2 == -INFINITY) dot[u] = sq[u] = 0.f;
        float* st = p.stats + ((static_cast<long long>(b) * a.heads + h) * p.q_tiles + (t >> 7)) * kStatPitch<T>;
        st[t & 127] = lse2;
        st[128 + (t & 127)] = -dot[u];
        if (kNorms) st[256 + (t & 127)] = sq[u];
      }
      if (at == 0) norm = fmaxf(norm, sq[u]);
    }
    if (kNorms) {
      norm = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(norm)));
      if (lane == 0)
        (values ? p.value_norms : p.row_norms)[(static_cast<long long>(b) * heads + h) * groups + part] = norm;
    }
  }
}

struct Bars {
  uint64_t a_full[2], a_empty[2];                 // q, do (dq kernel); k, v (dk, dv kernel)
  uint64_t x_full[kMaxRing], x_empty[kMaxRing];   // k ring; q ring
  uint64_t y_full[kMaxRing], y_empty[kMaxRing];   // v ring; do ring
  uint64_t st_full[2], st_empty[2];               // dk, dv: the queries' statistics
  uint64_t s_full, p_full, acc_done, acc_free;
  uint64_t s_free;                                // dq: the scores have been read
  // dq: by step parity.  The step after next cannot arrive before everyone has
  // waited for this one, so no wait sees a phase go by.
  uint64_t dp_full[2], ds_full[2];
  uint64_t drain[2];
  SplitStart start;
  uint32_t tmem;
  int abort_flag;
};

static_assert(sizeof(Bars) <= 1024, "shared-memory plan of the dk, dv kernel");

constexpr int kSoftWarps = 16;  // a quarter of the lanes and of the columns each
constexpr int kMmaWarp = kSoftWarps;
// dq: two warps issue products, so that one's waits pass beside the other's.
constexpr int kGradWarp = kSoftWarps + 1, kLoadWarp = kSoftWarps + 2, kDqThreads = 32 * (kSoftWarps + 3);
// dk, dv: one does.
constexpr int kKeyLoadWarp = kSoftWarps + 1, kDkvThreads = 32 * (kSoftWarps + 2);

// ------------------------------------------------------------------ dq
// kOne: all keys are one tile, and each row's delta is summed here, from p and
// dp in fp32 (with few keys ds is a small difference, which the rounding of the
// output that delta is else taken from would swamp: against 3 keys the
// gradients were 1.8 times as far off); the dk, dv kernel then takes it too.
template <typename T, int DP, bool kMask, bool kOne>
__global__ void __launch_bounds__(kDqThreads, 1)
    attn_dq_kernel(const __grid_constant__ AttnBwdParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kBlocks = DP / 64;
  constexpr uint32_t kATile = 128u * 128u * kBlocks;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + p.off_bar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars.abort_flag;
  unsigned int* status = p.status;
  const long long limit = p.timeout_cycles;
  const uint32_t kv_block = static_cast<uint32_t>(p.kv_box) * 128u;
  const uint32_t kv_tile = kv_block * kBlocks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.a_full[i]), 1);
      mbar_init(smem_u32(&bars.a_empty[i]), 1);
      mbar_init(smem_u32(&bars.dp_full[i]), 1);
      mbar_init(smem_u32(&bars.ds_full[i]), kSoftWarps);
    }
    mbar_init(smem_u32(&bars.s_full), 1);
    mbar_init(smem_u32(&bars.s_free), kSoftWarps);
    for (int i = 0; i < p.x_stages; ++i) {
      mbar_init(smem_u32(&bars.x_full[i]), 1);
      mbar_init(smem_u32(&bars.x_empty[i]), 1);
    }
    for (int i = 0; i < p.y_stages; ++i) {
      mbar_init(smem_u32(&bars.y_full[i]), 1);
      mbar_init(smem_u32(&bars.y_empty[i]), 1);
    }
    mbar_init(smem_u32(&bars.acc_done), 1);
    mbar_init(smem_u32(&bars.acc_free), kSoftWarps);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&bars.drain[i]), 1);
    bars.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars.tmem), 512);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&p.map_q);
    tma_prefetch_desc(&p.map_do);
    tma_prefetch_desc(&p.map_k);
    tma_prefetch_desc(&p.map_v);
  }
  grid_dependency_wait();
  if (warp == 0) {
    const SplitStart st = split_rows(p, lane);
    if (lane == 0) bars.start = st;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();  // (TMEM is held: what starts now cannot take it first)
  const uint32_t tmem = bars.tmem;
  const SplitStart start = bars.start;
  // TMEM columns: S, dp (two buffers; ds over them), dq.
  const uint32_t t_dp = tmem + 128, t_acc = tmem + 384;

  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned int code) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(bar), parity, abort_flag, status,
                                                     code, limit));
  };
  auto wait_set = [&](const WaitSet& s) {
    return wait_set_bounded(s, abort_flag, status, kAttnMmaTimeout, limit);
  };

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    const uint32_t lead = lane == 0 ? 1u : 0u;
    const uint32_t a_bytes = static_cast<uint32_t>(p.tile_heads * p.tile_tokens) * 128u * kBlocks;
    bool ok = true;
    int xs = 0, ys = 0;
    uint32_t xph = 0, yph = 0, aph = 0;
    long long nx = 0, ny = 0, na = 0;
    for (Walk<true, kMask, AttnBwdParams> w(p, start); ok && w.live; w.next()) {
      int token, head;
      w.place(0, &token, &head);
      for (int i = 0; ok && i < 2; ++i) {
        ok = wait(&bars.a_empty[i], aph ^ 1u, kAttnProducerTimeout);
        if (!ok) break;
        const uint32_t bar = smem_u32(&bars.a_full[i]);
        mbar_arrive_expect_tx_if(lead, bar, a_bytes);
        const CUtensorMap* map = i ? &p.map_do : &p.map_q;
        const int* mul = i ? p.do_mul : p.q_mul;
        for (int c = 0; c < kBlocks; ++c)
          tma_load_4d_if(lead, smem_u32(smem + p.off_a) + i * kATile + c * 16384u, map, bar, c * 64,
                         head * mul[0], token, w.b * mul[1]);
        if (i == 1) ++na;
      }
      aph ^= 1u;
      for (int t = w.first(); ok && t < w.t1; t = w.after(t)) {
        ok = wait(&bars.x_empty[xs], xph ^ 1u, kAttnProducerTimeout);
        if (!ok) break;
        if (!(p.fault_mode == 1 && nx == 0)) {
          mbar_arrive_expect_tx_if(lead, smem_u32(&bars.x_full[xs]), kv_tile);
          for (int c = 0; c < kBlocks; ++c)
            tma_load_4d_if(lead, smem_u32(smem + p.off_x) + xs * kv_tile + c * kv_block, &p.map_k,
                           smem_u32(&bars.x_full[xs]), c * 64, w.hk * p.k_mul[0], t * p.kv_box,
                           w.b * p.k_mul[1]);
        }
        ++nx;
        if (++xs == p.x_stages) {
          xs = 0;
          xph ^= 1u;
        }
        ok = wait(&bars.y_empty[ys], yph ^ 1u, kAttnProducerTimeout);
        if (!ok) break;
        mbar_arrive_expect_tx_if(lead, smem_u32(&bars.y_full[ys]), kv_tile);
        for (int c = 0; c < kBlocks; ++c)
          tma_load_4d_if(lead, smem_u32(smem + p.off_y) + ys * kv_tile + c * kv_block, &p.map_v,
                         smem_u32(&bars.y_full[ys]), c * 64, w.hk * p.v_mul[0], t * p.kv_box,
                         w.b * p.v_mul[1]);
        ++ny;
        if (++ys == p.y_stages) {
          ys = 0;
          yph ^= 1u;
        }
      }
    }
    if (!ok) {
      // Let every copy still in flight land before the CTA exits.
      for (long long q = nx - p.x_stages; q < nx; ++q)
        if (q >= 0)
          mbar_wait_drain(smem_u32(&bars.x_full[q % p.x_stages]),
                          static_cast<uint32_t>((q / p.x_stages) & 1), limit / 8 + 1);
      for (long long q = ny - p.y_stages; q < ny; ++q)
        if (q >= 0)
          mbar_wait_drain(smem_u32(&bars.y_full[q % p.y_stages]),
                          static_cast<uint32_t>((q / p.y_stages) & 1), limit / 8 + 1);
      if (na > 0)
        for (int i = 0; i < 2; ++i)
          mbar_wait_drain(smem_u32(&bars.a_full[i]), static_cast<uint32_t>((na - 1) & 1),
                          limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp < kLoadWarp && warp >= kMmaWarp) {
    // ------------------------------------------------------------ products
    // One warp issues S and dp, the other dq.
    const bool grads = warp == kGradWarp;
    const int k_steps = (p.a.head_dim + 15) >> 4;
    const uint32_t idesc_s = attn_idesc(kBf16, 0, false, false);
    const uint32_t idesc_acc = attn_idesc(kBf16, k_steps * 16, false, true);
    const uint32_t lead_k = lead_mn(kv_block);
    const uint32_t a_lo = smem_u32(smem + p.off_a) >> 4, x_lo = smem_u32(smem + p.off_x) >> 4,
                   y_lo = smem_u32(smem + p.off_y) >> 4;
    const uint32_t tile_lo = kv_tile >> 4, block_lo = kv_block >> 4;
    bool ok = true;
    int xs = 0, ys = 0, xs_before[2] = {0, 0};  // stages; k's one and two steps before
    uint32_t xph = 0, yph = 0, xph_before[2] = {0, 0}, count = 0, items = 0;
    // A (128 rows) times a key/value tile, over the head dimension.
    auto rows_by_keys = [&](uint32_t d, uint32_t a, uint32_t b, int cols) {
      const uint32_t id = idesc_s | (static_cast<uint32_t>(cols >> 3) << 17);
      mma_ss_x4(d, kLeadK | a, kLeadK | b, id, 0u, k_steps);
      if (k_steps > 4) mma_ss_x4(d, kLeadK | (a + 1024u), kLeadK | (b + block_lo), id, 1u, k_steps - 4);
    };
    for (Walk<true, kMask, AttnBwdParams> w(p, start); ok && w.live; w.next(), ++items) {
      bool first = true;
      for (int t = w.first(), after; ok && t < w.t1; t = after, first = false) {
        after = w.after(t);
        const bool last = after >= w.t1;
        const int cols = w.tile_cols(t);
        const uint32_t buf = count & 1u;
        if (!grads) {
          // This step's S and dp run beside the step before's exponentials and
          // ds.  (dp's buffer held the ds that dq took two steps ago.)
          WaitSet ready(&bars.x_full[xs], xph, lane);
          ready.also<1>(&bars.s_free, (count - 1) & 1u, count > 0);
          ready.also<2>(&bars.a_full[0], items & 1u, first);
          ok = wait_set(ready);
          if (!ok) break;
          tc_fence_after();
          rows_by_keys(tmem, a_lo, x_lo + xs * tile_lo, cols);
          mma_commit_warp(smem_u32(&bars.s_full));
          WaitSet rest(&bars.y_full[ys], yph, lane);
          rest.also<1>(&bars.x_empty[xs_before[1]], xph_before[1], count > 1);
          rest.also<2>(&bars.a_full[1], items & 1u, first);
          ok = wait_set(rest);
          if (!ok) break;
          tc_fence_after();
          rows_by_keys(t_dp + buf * 128, a_lo + (kATile >> 4), y_lo + ys * tile_lo, cols);
          mma_commit_warp(smem_u32(&bars.dp_full[buf]));
          mma_commit_warp(smem_u32(&bars.y_empty[ys]));
          if (last) {
            mma_commit_warp(smem_u32(&bars.a_empty[0]));
            mma_commit_warp(smem_u32(&bars.a_empty[1]));
          }
          if (++ys == p.y_stages) {
            ys = 0;
            yph ^= 1u;
          }
        } else {
          const int keys = w.tile_keys(t);
          uint4 used = first_keys(keys);
          if (kMask) {
            const uint4 any = w.any_keys(t);
            used = make_uint4(used.x & any.x, used.y & any.y, used.z & any.z, used.w & any.w);
          }
          WaitSet ready(&bars.ds_full[buf], (count >> 1) & 1u, lane);
          ready.also<1>(&bars.x_full[xs], xph);
          ready.also<2>(&bars.acc_free, (items - 1) & 1u, first && items > 0);
          ok = wait_set(ready);
          if (!ok) break;
          // Keys that no row takes part with are cleared: nothing they hold
          // meets a zero of ds.
          if (kMask || (keys < cols && p.a.kv_lengths)) {
            clear_rows<kBlocks>(smem + p.off_x + xs * kv_tile, kv_block, cols, used, lane);
            fence_proxy_async_shared();
            __syncwarp();
          }
          tc_fence_after();
          const int steps = cols >> 4;
          const uint32_t kb = lead_k | (x_lo + xs * tile_lo), ds = t_dp + buf * 128;
          mma_ts_x4<32>(t_acc, ds, kb, idesc_acc, first ? 0u : 1u, steps);
          if (steps > 4) mma_ts_x4<32>(t_acc, ds + 64, kb + 512u, idesc_acc, 1u, steps - 4);
          mma_commit_warp(smem_u32(&bars.x_empty[xs]));
          if (last) mma_commit_warp(smem_u32(&bars.acc_done));
        }
        xs_before[1] = xs_before[0];
        xph_before[1] = xph_before[0];
        xs_before[0] = xs;
        xph_before[0] = xph;
        if (++xs == p.x_stages) {
          xs = 0;
          xph ^= 1u;
        }
        ++count;
      }
    }
    if (!ok) {
      mma_commit_warp(smem_u32(&bars.drain[grads]));
      mbar_wait_drain(smem_u32(&bars.drain[grads]), 0, limit / 8 + 1);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ p and ds
    // Four warps share a quarter of the lanes; each takes 32 of the keys.
    const int part = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
    const float c2 = p.scale_log2;
    const int d = p.a.head_dim;
    const int row_token = p.tile_heads > 1 ? r / p.tile_heads : r;
    const int row_head = p.tile_heads > 1 ? r - row_token * p.tile_heads : 0;
    uint32_t count = 0, items = 0;
    bool ok = true;
    float values = 0.f;  // fp16: the largest |v|^2 of the key head of (of_b, of_hk)
    int of_b = -1, of_hk = -1;
    for (Walk<true, kMask, AttnBwdParams> w(p, start); ok && w.live; w.next()) {
      if (!kBf16 && (w.b != of_b || w.hk != of_hk)) {
        of_b = w.b;
        of_hk = w.hk;
        values = largest_value(p, of_b, of_hk, lane);
      }
      int token, head;
      w.place(0, &token, &head);
      token += row_token;
      head += row_head;
      const bool row_ok = row_token < p.tile_tokens && token < p.a.q_len;
      float lse2 = -INFINITY, delta = 0.f, norm = 0.f;  // (the first two negated)
      const uint32_t* bits = nullptr;
      float* st = nullptr;
      if (row_ok) {
        st = p.stats + ((static_cast<long long>(w.b) * p.a.heads + head) * p.q_tiles + (token >> 7)) * kStatPitch<T>;
        lse2 = st[token & 127];
        if (!kOne) delta = st[128 + (token & 127)];
        if (!kBf16) norm = st[256 + (token & 127)];
        if (kMask)
          bits = p.a.mask_bits +
                 (w.b * p.a.mask_b + head * p.a.mask_h + token * p.a.mask_q) * p.a.mask_words;
      }
      // (p is held times 2^p_shift here too; ds's scale takes it out.)
      const float scale_ds = kBf16 ? 1.f : ds_scale(norm, values), sc = scale_ds * p.p_unscale;
      const uint64_t c22 = pack2(c2, c2), l2 = pack2(lse2, lse2), sc2 = pack2(sc, sc);
      for (int t = w.first(); t < w.t1; t = w.after(t)) {
        const int keys = w.tile_keys(t), cols = w.tile_cols(t);
        const int rest = keys - part * 32;  // of this warp's columns
        uint32_t on = rest >= 32 ? 0xFFFFFFFFu : rest <= 0 ? 0u : (1u << rest) - 1u;
        if (kMask) on &= bits ? bits[(t * p.kv_box >> 5) + part] : 0u;
        // (kOne: the warps of a row meet below, where a failed one tells the others.)
        ok = wait(&bars.s_full, count & 1u, kAttnSoftmaxTimeout);
        if (!kOne && !ok) break;
        tc_fence_after();
        const uint32_t ts = tmem + part * 32 + lane_field;
        const uint32_t td = t_dp + (count & 1u) * 128 + part * 32 + lane_field;
        const bool mine = part * 32 < cols && (!kOne || ok);
        uint32_t s[32];
        if (mine) {
          tmem_ld_x32(ts, s);
          tmem_wait_ld_x32(s);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.s_free));
        if (mine) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            unpack2(fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c22, l2), x, y);
            s[2 * i] = __float_as_uint(exp2_approx(x));
            s[2 * i + 1] = __float_as_uint(exp2_approx(y));
          }
        }
        ok = ok && wait(&bars.dp_full[count & 1u], (count >> 1) & 1u, kAttnSoftmaxTimeout);
        if (!kOne && !ok) break;
        tc_fence_after();
        if constexpr (kOne) {
          float sum = 0.f;
          if (mine && ok) {
            uint32_t dp[32];
            tmem_ld_x32(td, dp);
            tmem_wait_ld_x32(dp);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((on >> i) & 1u) sum = fmaf(__uint_as_float(s[i]), __uint_as_float(dp[i]), sum);
          }
          float* parts = reinterpret_cast<float*>(smem + p.off_stat);
          parts[part * 128 + r] = sum;
          ok = barrier_all(1 + quarter, 128, ok);
          if (!ok) break;
          delta = -p.p_unscale * ((parts[r] + parts[128 + r]) + (parts[256 + r] + parts[384 + r]));
          if (part == 0 && st) st[128 + (token & 127)] = delta;
        }
        const uint64_t dl2 = pack2(delta * sc, delta * sc);
        if (mine) {
          uint32_t dp[32], h[16];
          tmem_ld_x32(td, dp);
          tmem_wait_ld_x32(dp);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            unpack2(mul2(fma2(pack2(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1])), sc2, dl2),
                         pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]))), x, y);
            dp[2 * i] = __float_as_uint(x);
            dp[2 * i + 1] = __float_as_uint(y);
          }
          if (on != 0xFFFFFFFFu) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((on >> i) & 1u)) dp[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            h[i] = round2<T>(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1]));
          tmem_st_x16(td, h);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.ds_full[count & 1u]));
        ++count;
      }
      ok = ok && wait(&bars.acc_done, items & 1u, kAttnSoftmaxTimeout);
      if (kOne) ok = barrier_all(1 + quarter, 128, ok);  // (the sums' parts have been read, too)
      ++items;
      if (!ok) break;
      tc_fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.nt;
      const long long slot = 2ll * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      const float f = p.a.scale / scale_ds;
      const int col = part * 32;
      if (col < DP) {
        uint32_t v[32];
        tmem_ld_x32(t_acc + col + lane_field, v);
        tmem_wait_ld_x32(v);
        if (row_ok && col < d) {
          if (whole)
            store_cols(static_cast<T*>(p.a.dq) + w.b * p.a.dqs[0] + token * p.a.dqs[1] +
                           head * p.a.dqs[2] + col,
                       v, d - col, f);
          else
            store_cols_f32(p.part_q + (slot * kAttnRows + r) * 128 + col, v, d - col,
                           kBf16 ? 1.f : 1.f / scale_ds);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.acc_free));
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dk, dv
// Key tiles of 128 of each batch's valid keys; an item is one key tile of one
// key head, its steps the query tiles of the heads that share it.
__device__ __forceinline__ long long key_steps(const AttnBwdParams& p, int b) {
  return static_cast<long long>((valid_keys(p.a, b) + kAttnRows - 1) / kAttnRows) * p.a.kv_heads *
         p.item_steps;
}
__device__ __forceinline__ long long key_steps_uniform(const AttnBwdParams& p) {
  // (Short keys: one tile for every request, also one without keys.)
  if (p.region) return static_cast<long long>(p.a.kv_heads) * p.item_steps;
  return p.a.kv_lengths ? -1 : key_steps(p, 0);
}

template <bool kMask>
struct KeyWalk {
  const AttnBwdParams& p;
  long long left;  // steps after this item
  int b, hk, tile, n;
  int i0, i1;      // steps [i0, i1) of item_steps
  int i, head, qt;  // the present step, its query head and tile
  uint32_t act;    // steps from act_base on that are worked on (with a mask)
  int act_base;
  bool live;
  __device__ KeyWalk(const AttnBwdParams& params, const SplitStart& st) : p(params) {
    left = st.left;
    live = left > 0;
    b = st.b;
    if (!live) return;
    n = valid_keys(p.a, b);
    const long long item = st.rest / p.item_steps;
    const int tiles = (n + kAttnRows - 1) / kAttnRows;
    hk = static_cast<int>(item / tiles);
    tile = static_cast<int>(item - static_cast<long long>(hk) * tiles);
    const int from = static_cast<int>(st.rest - item * p.item_steps);
    if (p.kv_whole && from > 0) {  // an item that began in another share
      left -= p.item_steps - from;
      next();
    } else {
      take(from);
    }
  }
  __device__ void take(int from) {
    i0 = from;
    i1 = p.kv_whole ? p.item_steps
                    : static_cast<int>(min(static_cast<long long>(p.item_steps), from + left));
    left -= i1 - i0;
    const int h = from / p.q_tiles;
    qt = from - h * p.q_tiles;
    head = hk * p.a.group + h;
  }
  // The steps of [i0, i1) that are worked on, in order: all, or with a mask
  // those whose queries attend some key of the tile (the first one if there is
  // none).  Every lane of a warp calls these together.  `i`, `head` and `qt`
  // are the present step's.
  __device__ void first() {
    act = 0;
    act_base = i = i0;
    if (!kMask || i1 - i0 == 1) return;
    const int to = search(i0);
    if (to < i1) go(to);
  }
  __device__ int after() {
    if (!kMask || i1 - i0 == 1) return i + 1;
    const int at = i - act_base;
    const uint32_t rest = static_cast<uint32_t>(at) < 31u ? act & (0xFFFFFFFEu << at) : 0u;
    return rest ? act_base + __ffs(rest) - 1 : search(act_base + 32);
  }
  __device__ void go(int to) {
    qt += to - i;
    i = to;
    while (qt >= p.q_tiles) {
      qt -= p.q_tiles;
      ++head;
    }
  }
  __device__ int search(int from) {
    const AttnShape& a = p.a;
    for (act_base = from; act_base < i1; act_base += 32) {
      const int s = act_base + (threadIdx.x & 31);
      bool on = false;
      if (s < i1) {
        const int h = s / p.q_tiles;
        const uint4 v = *reinterpret_cast<const uint4*>(
            a.mask_any +
            (b * a.any_b + (hk * a.group + h) * a.any_h + (s - h * p.q_tiles) * a.any_q) * a.mask_words +
            tile * 4);
        on = (v.x | v.y | v.z | v.w) != 0;
      }
      act = __ballot_sync(0xFFFFFFFFu, on);
      if (act) return act_base + __ffs(act) - 1;
    }
    return i1;
  }
  __device__ void next() {
    live = left > 0;
    if (!live) return;
    if (++tile * kAttnRows >= n) {
      tile = 0;
      if (++hk == p.a.kv_heads) {
        hk = 0;
        do n = valid_keys(p.a, ++b);
        while (n == 0);
      }
    }
    take(0);
  }
  __device__ int cols() const { return qt == p.q_tiles - 1 ? p.last_cols : kAttnRows; }
  __device__ int keys() const { return min(kAttnRows, n - tile * kAttnRows); }
};

template <typename T, int DP, bool kMask>
__global__ void __launch_bounds__(kDkvThreads, 1)
    attn_dkv_kernel(const __grid_constant__ AttnBwdParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kBlocks = DP / 64;
  constexpr uint32_t kTile = 128u * 128u * kBlocks;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + p.off_bar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars.abort_flag;
  unsigned int* status = p.status;
  const long long limit = p.timeout_cycles;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.a_full[i]), 1);
      mbar_init(smem_u32(&bars.a_empty[i]), 1);
    }
    for (int i = 0; i < p.x_stages; ++i) {
      mbar_init(smem_u32(&bars.x_full[i]), 1);
      mbar_init(smem_u32(&bars.x_empty[i]), 1);
    }
    for (int i = 0; i < p.y_stages; ++i) {
      mbar_init(smem_u32(&bars.y_full[i]), 1);
      mbar_init(smem_u32(&bars.y_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.st_full[i]), 1);
      mbar_init(smem_u32(&bars.st_empty[i]), kSoftWarps);
    }
    mbar_init(smem_u32(&bars.s_full), 1);
    mbar_init(smem_u32(&bars.dp_full[0]), 1);
    mbar_init(smem_u32(&bars.p_full), kSoftWarps);
    mbar_init(smem_u32(&bars.ds_full[0]), kSoftWarps);
    mbar_init(smem_u32(&bars.acc_done), 1);
    mbar_init(smem_u32(&bars.acc_free), kSoftWarps);
    mbar_init(smem_u32(&bars.drain[0]), 1);
    bars.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars.tmem), 512);
    tmem_relinquish();
  }
  if (warp == kKeyLoadWarp && lane == 0) {
    tma_prefetch_desc(&p.map_q);
    tma_prefetch_desc(&p.map_do);
    tma_prefetch_desc(&p.map_k);
    tma_prefetch_desc(&p.map_v);
  }
  grid_dependency_wait();
  if (warp == 0) {
    const SplitStart st = split_start(p.a.batch, key_steps_uniform(p), lane,
                                      [&](int b) { return key_steps(p, b); });
    if (lane == 0) bars.start = st;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();  // (TMEM is held: what starts now cannot take it first)
  const uint32_t tmem = bars.tmem;
  const SplitStart start = bars.start;
  // TMEM columns: S^T (p^T over it), dp^T (ds^T over it), dv, dk.
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 256 + DP;

  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned int code) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(bar), parity, abort_flag, status,
                                                     code, limit));
  };
  auto wait_set = [&](const WaitSet& s) {
    return wait_set_bounded(s, abort_flag, status, kAttnMmaTimeout, limit);
  };

  if (warp == kKeyLoadWarp) {
    // ------------------------------------------------------------ loads
    const uint32_t lead = lane == 0 ? 1u : 0u;
    const uint32_t kv_bytes = static_cast<uint32_t>(p.kv_box) * 128u * kBlocks;
    const uint32_t q_bytes = static_cast<uint32_t>(p.q_box) * 128u * kBlocks;
    bool ok = true;
    int xs = 0, ys = 0;
    uint32_t xph = 0, yph = 0, aph = 0;
    long long nx = 0, ny = 0, na = 0, nst = 0;
    for (KeyWalk<kMask> w(p, start); ok && w.live; w.next()) {
      for (int i = 0; ok && i < 2; ++i) {
        ok = wait(&bars.a_empty[i], aph ^ 1u, kAttnProducerTimeout);
        if (!ok) break;
        const uint32_t bar = smem_u32(&bars.a_full[i]);
        mbar_arrive_expect_tx_if(lead, bar, kv_bytes);
        const CUtensorMap* map = i ? &p.map_v : &p.map_k;
        const int* mul = i ? p.v_mul : p.k_mul;
        for (int c = 0; c < kBlocks; ++c)
          tma_load_4d_if(lead, smem_u32(smem + p.off_a) + i * kTile + c * 16384u, map, bar, c * 64,
                         w.hk * mul[0], w.tile * kAttnRows, w.b * mul[1]);
        if (i == 1) ++na;
      }
      aph ^= 1u;
      for (w.first(); ok && w.i < w.i1; w.go(w.after())) {
        const int h = w.head, qt = w.qt;
        ok = wait(&bars.x_empty[xs], xph ^ 1u, kAttnProducerTimeout);
        if (!ok) break;
        uint32_t bar = smem_u32(&bars.x_full[xs]);
        if (!(p.fault_mode == 1 && nx == 0)) {
          mbar_arrive_expect_tx_if(lead, bar, q_bytes);
          for (int c = 0; c < kBlocks; ++c)
            tma_load_4d_if(lead, smem_u32(smem + p.off_x) + xs * kTile + c * 16384u, &p.map_q, bar,
                           c * 64, h * p.q_mul[0], qt * kAttnRows, w.b * p.q_mul[1]);
        }
        const uint32_t ss = static_cast<uint32_t>(nx & 1);
        ok = wait(&bars.st_empty[ss], static_cast<uint32_t>((nx >> 1) & 1) ^ 1u, kAttnProducerTimeout);
        if (ok) {
          const uint32_t sbar = smem_u32(&bars.st_full[ss]);
          mbar_arrive_expect_tx_if(lead, sbar, 1024u);
          if (lead)
            bulk_load(smem_u32(smem + p.off_stat) + ss * 1024u,
                      p.stats + ((static_cast<long long>(w.b) * p.a.heads + h) * p.q_tiles + qt) * kStatPitch<T>,
                      1024u, sbar);
          __syncwarp();
          ++nst;
        }
        ++nx;
        if (!ok) break;
        if (++xs == p.x_stages) {
          xs = 0;
          xph ^= 1u;
        }
        ok = wait(&bars.y_empty[ys], yph ^ 1u, kAttnProducerTimeout);
        if (!ok) break;
        bar = smem_u32(&bars.y_full[ys]);
        mbar_arrive_expect_tx_if(lead, bar, q_bytes);
        for (int c = 0; c < kBlocks; ++c)
          tma_load_4d_if(lead, smem_u32(smem + p.off_y) + ys * kTile + c * 16384u, &p.map_do, bar,
                         c * 64, h * p.do_mul[0], qt * kAttnRows, w.b * p.do_mul[1]);
        ++ny;
        if (++ys == p.y_stages) {
          ys = 0;
          yph ^= 1u;
        }
      }
    }
    if (!ok) {
      for (long long q = nx - p.x_stages; q < nx; ++q)
        if (q >= 0)
          mbar_wait_drain(smem_u32(&bars.x_full[q % p.x_stages]),
                          static_cast<uint32_t>((q / p.x_stages) & 1), limit / 8 + 1);
      for (long long q = ny - p.y_stages; q < ny; ++q)
        if (q >= 0)
          mbar_wait_drain(smem_u32(&bars.y_full[q % p.y_stages]),
                          static_cast<uint32_t>((q / p.y_stages) & 1), limit / 8 + 1);
      for (long long q = nst - 2; q < nst; ++q)
        if (q >= 0)
          mbar_wait_drain(smem_u32(&bars.st_full[q & 1]), static_cast<uint32_t>((q >> 1) & 1),
                          limit / 8 + 1);
      if (na > 0)
        for (int i = 0; i < 2; ++i)
          mbar_wait_drain(smem_u32(&bars.a_full[i]), static_cast<uint32_t>((na - 1) & 1),
                          limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    // dv of a step and S^T of the next as soon as p is there, dk and dp^T as
    // soon as ds is: one wait for each pair.  (2 x 16 heads, 8192 x 2048 x
    // 128: 350 us; two warps with a pair each 372, taking turns 358.)
    const int k_steps = (p.a.head_dim + 15) >> 4;
    const uint32_t idesc_s = attn_idesc(kBf16, 0, false, false);
    const uint32_t idesc_acc = attn_idesc(kBf16, k_steps * 16, false, true);
    const uint32_t lead_b = lead_mn(16384);
    const uint32_t a_lo = smem_u32(smem + p.off_a) >> 4, x_lo = smem_u32(smem + p.off_x) >> 4,
                   y_lo = smem_u32(smem + p.off_y) >> 4;
    constexpr uint32_t kTileLo = kTile >> 4;
    bool ok = true;
    int xs = 0, ys = 0, x_now = 0, y_now = 0;  // stages to come, and the present step's
    uint32_t xph = 0, yph = 0, count = 0, items = 0;
    auto keys_by_rows = [&](uint32_t d, uint32_t a, uint32_t b, int cols) {
      const uint32_t id = idesc_s | (static_cast<uint32_t>(cols >> 3) << 17);
      mma_ss_x4(d, kLeadK | a, kLeadK | b, id, 0u, k_steps);
      if (k_steps > 4) mma_ss_x4(d, kLeadK | (a + 1024u), kLeadK | (b + 1024u), id, 1u, k_steps - 4);
    };
    // A (in TMEM, quarters of 32 columns) times a query tile, over its rows.
    auto accumulate = [&](uint32_t acc, uint32_t a, uint32_t b, int cols, bool fresh) {
      const int steps = cols >> 4;
      mma_ts_x4<32>(acc, a, lead_b | b, idesc_acc, fresh ? 0u : 1u, steps);
      if (steps > 4) mma_ts_x4<32>(acc, a + 64, lead_b | (b + 512u), idesc_acc, 1u, steps - 4);
    };
    // Queries without keys are cleared: nothing they hold meets a zero of p or ds.
    auto clear = [&](uint8_t* tile, int stat_stage) {
      const float* st = reinterpret_cast<const float*>(smem + p.off_stat + stat_stage * 1024);
      uint4 used;
      used.x = __ballot_sync(0xFFFFFFFFu, st[lane] != -INFINITY);
      used.y = __ballot_sync(0xFFFFFFFFu, st[32 + lane] != -INFINITY);
      used.z = __ballot_sync(0xFFFFFFFFu, st[64 + lane] != -INFINITY);
      used.w = __ballot_sync(0xFFFFFFFFu, st[96 + lane] != -INFINITY);
      clear_rows<kBlocks>(tile, 16384, kAttnRows, used, lane);
      fence_proxy_async_shared();
      __syncwarp();
    };
    // S^T of step n, and its dp^T (their barriers are through).
    auto step_s = [&](uint32_t n, int cols, bool last) {
      if (kMask) {
        ok = wait(&bars.st_full[n & 1u], (n >> 1) & 1u, kAttnMmaTimeout);
        if (!ok) return;
        clear(smem + p.off_x + xs * kTile, n & 1u);
      }
      keys_by_rows(t_s, a_lo, x_lo + xs * kTileLo, cols);
      mma_commit_warp(smem_u32(&bars.s_full));
      if (last) mma_commit_warp(smem_u32(&bars.a_empty[0]));
      if (++xs == p.x_stages) {
        xs = 0;
        xph ^= 1u;
      }
    };
    auto step_dp = [&](uint32_t n, int cols, bool last) {
      if (kMask) clear(smem + p.off_y + ys * kTile, n & 1u);
      keys_by_rows(t_dp, a_lo + kTileLo, y_lo + ys * kTileLo, cols);
      mma_commit_warp(smem_u32(&bars.dp_full[0]));
      if (last) mma_commit_warp(smem_u32(&bars.a_empty[1]));
      if (++ys == p.y_stages) {
        ys = 0;
        yph ^= 1u;
      }
    };
    KeyWalk<kMask> w(p, start);
    bool live = w.live, first = true;
    int after = 0, cols = 0;
    if (live) {
      w.first();
      after = w.after();
      cols = w.cols();
      WaitSet rows(&bars.x_full[0], 0, lane);
      rows.also<1>(&bars.a_full[0], 0);
      ok = wait_set(rows);
      tc_fence_after();
      if (ok) step_s(0, cols, after >= w.i1);
      if (ok) {
        WaitSet grads(&bars.y_full[0], 0, lane);
        grads.also<1>(&bars.a_full[1], 0);
        ok = wait_set(grads);
        tc_fence_after();
        if (ok) step_dp(0, cols, after >= w.i1);
      }
    }
    while (ok && live) {
      // The next step's place first: between the products below there is only
      // what they need.
      const bool last = after >= w.i1;
      const int this_cols = cols;
      bool more = true;
      if (last) {
        w.next();
        more = w.live;
        if (more) w.first();
      } else {
        w.go(after);
      }
      if (more) {
        after = w.after();
        cols = w.cols();
      }
      const uint32_t next_item = (items + 1) & 1u;
      WaitSet to_p(&bars.p_full, count & 1u, lane);
      to_p.also<1>(&bars.x_full[xs], xph, more);
      to_p.also<2>(&bars.a_full[0], next_item, more && last);
      to_p.also<3>(&bars.acc_free, (items - 1) & 1u, first && items > 0);
      ok = wait_set(to_p);
      if (!ok) break;
      tc_fence_after();
      accumulate(t_dv, t_s, y_lo + y_now * kTileLo, this_cols, first);
      mma_commit_warp(smem_u32(&bars.y_empty[y_now]));
      y_now = ys;
      if (more) step_s(count + 1, cols, after >= w.i1);
      if (!ok) break;
      WaitSet to_ds(&bars.ds_full[0], count & 1u, lane);
      to_ds.also<1>(&bars.y_full[ys], yph, more);
      to_ds.also<2>(&bars.a_full[1], next_item, more && last);
      ok = wait_set(to_ds);
      if (!ok) break;
      tc_fence_after();
      accumulate(t_dk, t_dp, x_lo + x_now * kTileLo, this_cols, first);
      if (last) mma_commit_warp(smem_u32(&bars.acc_done));
      mma_commit_warp(smem_u32(&bars.x_empty[x_now]));
      if (++x_now == p.x_stages) x_now = 0;
      if (more) step_dp(count + 1, cols, after >= w.i1);
      if (last) ++items;
      ++count;
      first = last;
      live = more;
    }
    if (!ok) {
      mma_commit_warp(smem_u32(&bars.drain[0]));
      mbar_wait_drain(smem_u32(&bars.drain[0]), 0, limit / 8 + 1);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ p and ds
    // One thread per key and 32 of the queries.
    const int part = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
    const float c2 = p.scale_log2;
    const uint64_t c22 = pack2(c2, c2);
    const int d = p.a.head_dim;
    const uint32_t ts = t_s + part * 32 + lane_field, td = t_dp + part * 32 + lane_field;
    uint32_t* mask_tile = reinterpret_cast<uint32_t*>(smem + p.off_mask);
    uint32_t count = 0, items = 0;
    bool ok = true;
    for (KeyWalk<kMask> w(p, start); ok && w.live; w.next()) {
      const bool key_ok = r < w.keys();
      const bool keys_whole = w.keys() == kAttnRows;
      const float scale_ds = kBf16 ? 1.f
                                   : ds_scale(largest_row(p, w.b, w.hk, w.i0, w.i1, lane),
                                              largest_value(p, w.b, w.hk, lane));
      const float sc = scale_ds * p.p_unscale;
      const uint64_t sc2 = pack2(sc, sc);
      for (w.first(); w.i < w.i1; w.go(w.after())) {
        const bool mine = part * 32 < w.cols();
        uint32_t on = 0xFFFFFFFFu;
        if (kMask) {
          // The tile's mask words, [query][4 words of 32 keys]: every warp reads
          // its word of 32 queries, one bit per lane.
          const int h = w.head, t0 = w.qt * kAttnRows;
          uint32_t* buf = mask_tile + (count & 1u) * 512;
          const int row = threadIdx.x >> 2, word = threadIdx.x & 3;
          uint32_t q = 0;
          if (t0 + row < p.a.q_len)
            q = p.a.mask_bits[(w.b * p.a.mask_b + h * p.a.mask_h + (t0 + row) * p.a.mask_q) *
                                  p.a.mask_words + w.tile * 4 + word];
          buf[row * 4 + word] = q;
          ok = barrier_all(1, 32 * kSoftWarps, ok);
          if (!ok) break;
          on = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) on |= ((buf[(part * 32 + j) * 4 + quarter] >> lane) & 1u) << j;
        }
        if (!key_ok) on = 0;
        const bool select = kMask || !keys_whole;
        const uint32_t ss = count & 1u;
        ok = wait(&bars.st_full[ss], (count >> 1) & 1u, kAttnSoftmaxTimeout) &&
             wait(&bars.s_full, count & 1u, kAttnSoftmaxTimeout);
        if (!kMask && !ok) break;
        const float* st = reinterpret_cast<const float*>(smem + p.off_stat + ss * 1024) + part * 32;
        uint32_t s[32];
        if (ok) {
          tc_fence_after();
          if (mine) {
            tmem_ld_x32(ts, s);
            tmem_wait_ld_x32(s);
            uint32_t h[16];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(st + j);
              float x[4];
              unpack2(fma2(pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), c22, l.x), x[0], x[1]);
              unpack2(fma2(pack2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), c22, l.y), x[2], x[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) s[j + k] = __float_as_uint(exp2_approx(x[k]));
            }
            if (select) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((on >> j) & 1u)) s[j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
              h[j] = round2<T>(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
            tmem_st_x16(ts, h);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.p_full));
          ok = wait(&bars.dp_full[0], count & 1u, kAttnSoftmaxTimeout);
        }
        if (ok) {
          tc_fence_after();
          if (mine) {
            uint32_t dp[32], h[16];
            tmem_ld_x32(td, dp);
            tmem_wait_ld_x32(dp);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(st + 128 + j);
              uint64_t u = add2(pack2(__uint_as_float(dp[j]), __uint_as_float(dp[j + 1])), l.x);
              uint64_t v = add2(pack2(__uint_as_float(dp[j + 2]), __uint_as_float(dp[j + 3])), l.y);
              if (!kBf16) {
                u = mul2(u, sc2);
                v = mul2(v, sc2);
              }
              float x[4];
              unpack2(mul2(u, pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1]))), x[0], x[1]);
              unpack2(mul2(v, pack2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]))), x[2], x[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) dp[j + k] = __float_as_uint(x[k]);
            }
            if (select) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((on >> j) & 1u)) dp[j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
              h[j] = round2<T>(__uint_as_float(dp[2 * j]), __uint_as_float(dp[2 * j + 1]));
            tmem_st_x16(td, h);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&bars.ds_full[0]));
            mbar_arrive(smem_u32(&bars.st_empty[ss]));
          }
        }
        ++count;
        // (With a mask the warps meet at the next barrier, where a failed one
        // tells the others.)
        if (!ok && !kMask) break;
      }
      // (With a mask all warps leave the item together: one that gave up alone
      // would be missed at the next item's barriers.)
      ok = ok && wait(&bars.acc_done, items & 1u, kAttnSoftmaxTimeout);
      if (kMask) ok = barrier_all(1, 32 * kSoftWarps, ok);
      ++items;
      if (!ok) break;
      tc_fence_after();
      // Parts 0 and 1 take dv, 2 and 3 dk: half of the columns each.
      const int which = part >> 1;
      const bool whole = w.i0 == 0 && w.i1 == p.item_steps;
      const long long slot = 2ll * blockIdx.x + (w.i0 == 0 ? 1 : 0);
      const float f = which ? p.a.scale / scale_ds : p.p_unscale;
      const int j = w.tile * kAttnRows + r;
      T* dst = which ? static_cast<T*>(p.a.dk) + w.b * p.a.dks[0] + j * p.a.dks[1] + w.hk * p.a.dks[2]
                    : static_cast<T*>(p.a.dv) + w.b * p.a.dvs[0] + j * p.a.dvs[1] + w.hk * p.a.dvs[2];
#pragma unroll
      for (int i = 0; i < DP / 2; i += 32) {
        const int c = (part & 1) * (DP / 2) + i;
        uint32_t v[32];
        tmem_ld_x32((which ? t_dk : t_dv) + c + lane_field, v);
        tmem_wait_ld_x32(v);
        if (c < d) {
          if (whole) {
            if (j < p.a.kv_len) store_cols(dst + c, v, d - c, f);
          } else {
            store_cols_f32(p.part_kv + ((slot * 2 + which) * kAttnRows + r) * 128 + c, v, d - c,
                           kBf16 ? 1.f : which ? 1.f / scale_ds : p.p_unscale);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.acc_free));
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ joins
// Adds the shares of tiles that the launches before cut, in order, and clears
// the gradients of keys past each request's length.  Blocks of kJoinRows rows:
// the row tiles of dq first, then the key tiles of dk and dv.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
    attn_bwd_join_kernel(const __grid_constant__ AttnBwdParams p, int q_ctas, int kv_ctas,
                         long long q_blocks) {
  __shared__ JoinSlots join;
  const AttnShape& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d0 = lane * 4;
  const int r0 = blockIdx.y * kJoinRows + warp * kJoinUnroll;
  grid_dependency_wait();
  grid_launch_dependents();
  long long before, total;
  if (blockIdx.x < q_blocks) {
    const int b = static_cast<int>(blockIdx.x / p.item_rows);
    const int item = static_cast<int>(blockIdx.x - b * p.item_rows);
    split_prefix(a.batch, row_steps_uniform(p), b, join.sums, [&](int i) { return row_steps(p, i); },
                 &before, &total);
    const int nt = key_tiles(valid_keys(a, b), p.kv_box);
    list_slots(join, total, q_ctas, before + static_cast<long long>(item) * nt, nt);
    const int shares = join.count;
    if (shares == 0) return;
    const int hk = item / p.row_tiles, rt = item - hk * p.row_tiles;
    int token0, head0, rows;
    if (p.tile_heads > 1) {
      token0 = rt * p.tile_tokens;
      head0 = hk * a.group;
      rows = min(p.tile_tokens, a.q_len - token0) * p.tile_heads;
    } else {
      const int hg = rt / p.token_tiles;
      token0 = (rt - hg * p.token_tiles) * kAttnRows;
      head0 = hk * a.group + hg;
      rows = min(kAttnRows, a.q_len - token0);
    }
    if (r0 >= rows || d0 >= a.head_dim) return;
    float4 acc[kJoinUnroll];
#pragma unroll
    for (int u = 0; u < kJoinUnroll; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int c = 0; c < shares; ++c)
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u) {
        const float4 v = *reinterpret_cast<const float4*>(
            p.part_q + (static_cast<long long>(join.slots[c]) * kAttnRows + min(r0 + u, rows - 1)) * 128 + d0);
        acc[u].x += v.x; acc[u].y += v.y; acc[u].z += v.z; acc[u].w += v.w;
      }
#pragma unroll
    for (int u = 0; u < kJoinUnroll; ++u) {
      const int r = r0 + u;
      if (r >= rows) break;
      const int dt = p.tile_heads > 1 ? r / p.tile_heads : r;
      const int token = token0 + dt, head = p.tile_heads > 1 ? head0 + r - dt * p.tile_heads : head0;
      *reinterpret_cast<uint2*>(static_cast<T*>(a.dq) + b * a.dqs[0] + token * a.dqs[1] +
                                head * a.dqs[2] + d0) =
          make_uint2(round2<T>(acc[u].x * a.scale, acc[u].y * a.scale),
                     round2<T>(acc[u].z * a.scale, acc[u].w * a.scale));
    }
    return;
  }
  const int all_tiles = (a.kv_len + kAttnRows - 1) / kAttnRows;
  const long long at = blockIdx.x - q_blocks;
  const long long bh = at / all_tiles;
  const int tile = static_cast<int>(at - bh * all_tiles);
  const int b = static_cast<int>(bh / a.kv_heads), hk = static_cast<int>(bh - static_cast<long long>(b) * a.kv_heads);
  const int n = p.item_steps == 0 ? 0 : p.region ? a.kv_len : valid_keys(a, b), tiles = (n + kAttnRows - 1) / kAttnRows;
  const int rows = min(kAttnRows, a.kv_len - tile * kAttnRows);
  int shares = 0;
  if (tile < tiles) {
    if (p.kv_whole) return;
    split_prefix(a.batch, key_steps_uniform(p), b, join.sums, [&](int i) { return key_steps(p, i); },
                 &before, &total);
    list_slots(join, total, kv_ctas, before + (static_cast<long long>(hk) * tiles + tile) * p.item_steps,
               p.item_steps);
    shares = join.count;
    if (shares == 0) return;
  }
  if (r0 >= rows || d0 >= a.head_dim) return;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float4 acc[kJoinUnroll];
#pragma unroll
    for (int u = 0; u < kJoinUnroll; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int c = 0; c < shares; ++c)
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u) {
        const float4 v = *reinterpret_cast<const float4*>(
            p.part_kv +
            ((static_cast<long long>(join.slots[c]) * 2 + half) * kAttnRows + min(r0 + u, rows - 1)) * 128 + d0);
        acc[u].x += v.x; acc[u].y += v.y; acc[u].z += v.z; acc[u].w += v.w;
      }
    const float f = half ? a.scale : 1.f;
#pragma unroll
    for (int u = 0; u < kJoinUnroll; ++u) {
      if (r0 + u >= rows) break;
      const int j = tile * kAttnRows + r0 + u;
      T* dst = half ? static_cast<T*>(a.dk) + b * a.dks[0] + j * a.dks[1] + hk * a.dks[2]
                    : static_cast<T*>(a.dv) + b * a.dvs[0] + j * a.dvs[1] + hk * a.dvs[2];
      *reinterpret_cast<uint2*>(dst + d0) =
          make_uint2(round2<T>(acc[u].x * f, acc[u].y * f), round2<T>(acc[u].z * f, acc[u].w * f));
    }
  }
}

template <typename T, int DP, bool kMask, bool kOne>
cudaError_t launch_dq(const AttnBwdParams& p, int grid, size_t smem, cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  cudaError_t e = raise_smem(attn_dq_kernel<T, DP, kMask, kOne>, configured, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_dq_kernel<T, DP, kMask, kOne>, dim3(grid), dim3(kDqThreads), smem, stream, p);
}

template <typename T, int DP, bool kMask>
cudaError_t launch_dkv(const AttnBwdParams& p, int grid, size_t smem, cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  cudaError_t e = raise_smem(attn_dkv_kernel<T, DP, kMask>, configured, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_dkv_kernel<T, DP, kMask>, dim3(grid), dim3(kDkvThreads), smem, stream, p);
}

// Calls f with the operands' type, whether a row is wider than 64 columns and
// whether there is a mask.
template <typename F>
cudaError_t with_variant(const AttnBwdParams& p, F f) {
  const auto by_mask = [&](auto type, auto wide) {
    return p.a.mask_bits ? f(type, wide, std::true_type{}) : f(type, wide, std::false_type{});
  };
  const auto by_width = [&](auto type) {
    return p.a.head_dim > 64 ? by_mask(type, std::true_type{}) : by_mask(type, std::false_type{});
  };
  return p.a.dtype == 0 ? by_width(__nv_bfloat16{}) : by_width(__half{});
}

}  // namespace

size_t attn_bwd_bar_bytes() { return sizeof(Bars); }

cudaError_t launch_attn_rows(const AttnBwdParams& p, cudaStream_t stream) {
  const dim3 grid(p.row_blocks + p.value_blocks);
  return p.a.dtype == 0
             ? launch_pdl(attn_rows_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, p)
             : launch_pdl(attn_rows_kernel<__half>, grid, dim3(256), 0, stream, p);
}

cudaError_t launch_attn_dq(const AttnBwdParams& p, int grid, size_t smem, cudaStream_t stream) {
  return with_variant(p, [&](auto type, auto wide, auto mask) {
    constexpr int kDp = wide() ? 128 : 64;
    return p.a.kv_len <= p.kv_box ? launch_dq<decltype(type), kDp, mask(), true>(p, grid, smem, stream)
                                  : launch_dq<decltype(type), kDp, mask(), false>(p, grid, smem, stream);
  });
}

cudaError_t launch_attn_dkv(const AttnBwdParams& p, int grid, size_t smem, cudaStream_t stream) {
  return with_variant(p, [&](auto type, auto wide, auto mask) {
    return launch_dkv<decltype(type), wide() ? 128 : 64, mask()>(p, grid, smem, stream);
  });
}

cudaError_t launch_attn_bwd_join(const AttnBwdParams& p, int q_ctas, int kv_ctas,
                                 long long q_blocks, long long kv_blocks, cudaStream_t stream) {
  if (q_blocks + kv_blocks == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(q_blocks + kv_blocks), kAttnRows / kJoinRows);
  return p.a.dtype == 0 ? launch_pdl(attn_bwd_join_kernel<__nv_bfloat16>, grid, dim3(kJoinThreads), 0,
                                     stream, p, q_ctas, kv_ctas, q_blocks)
                        : launch_pdl(attn_bwd_join_kernel<__half>, grid, dim3(kJoinThreads), 0, stream,
                                     p, q_ctas, kv_ctas, q_blocks);
}

}  // namespace convgb300
