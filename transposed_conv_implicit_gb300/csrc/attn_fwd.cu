// Cross attention forward on the tensor cores.
//
//   s = scale q k^T,  p = exp(s - max),  out = (p v) / sum p
//
// in one pass over the keys with the running maximum and sum of each row.  A
// softmax group of four warps owns a row tile of 128 (token, head) rows, one
// thread per row: S (fp32, 128 TMEM lanes x keys) comes from one tcgen05.mma
// over the head dimension, the thread reads its row, and writes P (16-bit)
// over it, which the second tcgen05.mma takes straight from TMEM as its A
// operand against V, whose rows run along N in shared memory.  The output
// accumulates in TMEM; it is rescaled only when a row's maximum grows by more
// than a factor of 2^8 (P stays within 2^8 and the sum in fp32, so nothing is
// lost meanwhile), which after the first tiles hardly happens.
//
// Two schedules:
//  - pairs: a persistent CTA per SM takes two row tiles of one key head at a
//    time; each key/value tile is loaded once for both, and while one group
//    does its exponentials the tensor core multiplies for the other.
//  - split: two CTAs per SM, one row tile each; the sequence of (row tile, key
//    tile) steps of the whole call is cut into equal shares, so that few rows
//    over many keys still fill the GPU and ragged lengths balance.  A row tile
//    cut between CTAs goes through fp32 partial rows in the workspace, which
//    a second kernel joins in order.  Query heads that share a key head sit
//    side by side in a row tile when that makes fewer tiles.
//
// P is rounded to the inputs' type (the product's operand type; in fp16 times 2^7,
// with which it stays within 2^15), the sum is taken of the unrounded fp32 values;
// O is rounded once.
//
// A group's products (P v, then the next S) are one batch that its own warp
// issues; the groups' batches take turns.  With a mask, key tiles that none of
// the rows' tiles of 128 queries attends are skipped.
//
// Bound by the products and, beside them, the exponentials: 2 x 16 heads, 16384
// x 4096 x 128 takes 771 us, 1.43 PFLOP/s (567 us at the rate of a large matrix
// product).  Split, by reading the keys: one token of 64 requests x 32 heads
// against up to 4096 keys, 141 us, 5.8 TB/s.  Masked (each query sees its own
// segment), 3 x 1021 x 12 heads x 80 against 1531: 41 us, of which the mask's
// packing takes 6; 104 without the skipping.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "attn_internal.h"
#include "attn_params.h"
#include "attn_common.cuh"

namespace convgb300 {

namespace {

constexpr float kRescaleLog2 = 8.f;

template <typename T, int DP, int G>
struct Layout {
  static constexpr bool kSplit = G == 1;
  static constexpr int kBlocks = DP / 64;
  // Pairs: three warpgroups, so that the softmax groups can take the third
  // one's registers: (208 + 208 + 80) * 128 <= 168 * 384.
  static constexpr int kThreads = G == 2 ? 384 : 192;
  // One warp issues each group's products: a warp's issue is in order, and
  // the waits, descriptors and commits of two groups together take longer
  // than their products.
  static constexpr int kMmaWarp = 4 * G, kLoadWarp = 5 * G;
  static constexpr uint32_t kQTile = 128u * 128u * kBlocks;
  static constexpr uint32_t kTmemCols = G == 2 ? 512 : 256;
};

constexpr int kMaxStages = 8;

struct Bars {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t q_full[2][2], q_empty[2][2];  // [group][stage]
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], o_free[2];  // p_half: of the first 64 keys
  uint64_t turn[2];  // the groups' products take turns
  uint64_t drain[2];
  SplitStart start;
  uint32_t tmem;
  int abort_flag;
};

template <typename T, int DP, int G, bool kMask>
__global__ void __launch_bounds__(Layout<T, DP, G>::kThreads, G == 2 ? 1 : 2)
    attn_fwd_kernel(const __grid_constant__ AttnFwdParams p) {
  using L = Layout<T, DP, G>;
  constexpr bool kBf16 = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + p.off_bar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars.abort_flag;
  unsigned int* status = p.status;
  const long long limit = p.timeout_cycles;
  const uint32_t kv_block = static_cast<uint32_t>(p.kv_box) * 128u;  // 64 columns of a key tile
  const uint32_t kv_tile = kv_block * L::kBlocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&bars.kv_full[s]), 1);
      mbar_init(smem_u32(&bars.kv_empty[s]), G);
    }
    for (int g = 0; g < G; ++g) {
      for (int s = 0; s < p.q_stages; ++s) {
        mbar_init(smem_u32(&bars.q_full[g][s]), 1);
        mbar_init(smem_u32(&bars.q_empty[g][s]), 1);
      }
      mbar_init(smem_u32(&bars.s_full[g]), 1);
      mbar_init(smem_u32(&bars.p_half[g]), 4);
      mbar_init(smem_u32(&bars.p_full[g]), 4);
      mbar_init(smem_u32(&bars.o_done[g]), 1);
      mbar_init(smem_u32(&bars.o_free[g]), 4);
    }
    for (int g = 0; g < G; ++g) {
      mbar_init(smem_u32(&bars.turn[g]), 1);
      mbar_init(smem_u32(&bars.drain[g]), 1);
    }
    bars.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == L::kMmaWarp) {
    tmem_alloc(smem_u32(&bars.tmem), L::kTmemCols);
    tmem_relinquish();
  }
  if (warp == L::kLoadWarp && lane == 0) {
    tma_prefetch_desc(&p.map_q);
    tma_prefetch_desc(&p.map_k);
    tma_prefetch_desc(&p.map_v);
    tma_prefetch_desc(&p.map_out);
  }
  grid_dependency_wait();
  if (L::kSplit && warp == 0) {
    const SplitStart st = split_rows(p, lane);
    if (lane == 0) bars.start = st;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();  // (TMEM is held: what starts now cannot take it first)
  const uint32_t tmem = bars.tmem;
  const SplitStart start = L::kSplit ? bars.start : SplitStart{};

  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned int code) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(bar), parity, abort_flag, status,
                                                     code, limit));
  };

  auto wait_set = [&](const WaitSet& s) {
    return wait_set_bounded(s, abort_flag, status, kAttnMmaTimeout, limit);
  };

  if (warp == L::kLoadWarp) {
    // ------------------------------------------------------------ loads
    if (G == 2) give_registers<80>();
    const uint32_t lead = lane == 0 ? 1u : 0u;
    const uint32_t q_bytes =
        static_cast<uint32_t>(p.tile_heads * p.tile_tokens) * 128u * L::kBlocks;
    bool ok = true;
    int stage = 0, qs = 0;
    uint32_t phase = 0, q_phase = 0;
    long long issued = 0;
    long long q_issued[2] = {0, 0};
    for (Walk<L::kSplit, kMask, AttnFwdParams> w(p, start); ok && w.live; w.next()) {
      // Both groups' stages move together.  A group without a row tile in
      // this item has its stage's phase completed for it (group 1 first, so
      // that its wait precedes everything that ends the phase).
      for (int g = G - 1; ok && g >= 0; --g) {
        if (!wait(&bars.q_empty[g][qs], q_phase ^ 1u, kAttnProducerTimeout)) {
          ok = false;
          break;
        }
        const uint32_t bar = smem_u32(&bars.q_full[g][qs]);
        ++q_issued[g];
        if (g >= w.tiles_here) {
          if (lead) mbar_arrive(bar);
          continue;
        }
        int token, head;
        w.place(g, &token, &head);
        mbar_arrive_expect_tx_if(lead, bar, q_bytes);
#pragma unroll
        for (int c = 0; c < L::kBlocks; ++c)
          tma_load_4d_if(lead,
                         smem_u32(smem + p.off_q) + (g * p.q_stages + qs) * L::kQTile + c * 16384u,
                         &p.map_q, bar, c * 64, head * p.q_mul[0], token, w.b * p.q_mul[1]);
      }
      if (++qs == p.q_stages) {
        qs = 0;
        q_phase ^= 1u;
      }
      for (int t = w.first(); ok && t < w.t1; t = w.after(t)) {
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (!wait(&bars.kv_empty[stage], phase ^ 1u, kAttnProducerTimeout)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&bars.kv_full[stage]);
          const CUtensorMap* map = kv ? &p.map_v : &p.map_k;
          const int* mul = kv ? p.v_mul : p.k_mul;
          // (fault_mode 1, a test hook: every CTA leaves its first key tile un-armed.)
          if (!(p.fault_mode == 1 && issued == 0)) {
            mbar_arrive_expect_tx_if(lead, bar, kv_tile);
#pragma unroll
            for (int c = 0; c < L::kBlocks; ++c)
              tma_load_4d_if(lead, smem_u32(smem + p.off_kv) + stage * kv_tile + c * kv_block, map,
                             bar, c * 64, w.hk * mul[0], t * p.kv_box, w.b * mul[1]);
          }
          ++issued;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    if (!ok) {
      // Let every copy still in flight land before the CTA exits.
      for (long long q = issued - p.stages; q < issued; ++q)
        if (q >= 0)
          mbar_wait_drain(smem_u32(&bars.kv_full[q % p.stages]),
                          static_cast<uint32_t>((q / p.stages) & 1), limit / 8 + 1);
      for (int g = 0; g < G; ++g)
        for (long long q = q_issued[g] - p.q_stages; q < q_issued[g]; ++q)
          if (q >= 0)
            mbar_wait_drain(smem_u32(&bars.q_full[g][q % p.q_stages]),
                            static_cast<uint32_t>((q / p.q_stages) & 1), limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp >= L::kMmaWarp && warp < L::kMmaWarp + G) {
    // ------------------------------------------------------------ products
    // The converged warp walks the MMAs of its group; one elected lane issues.
    if (G == 2) give_registers<80>();
    const int g = warp - L::kMmaWarp;
    const int k_steps = (p.a.head_dim + 15) >> 4;
    const uint32_t idesc_s = attn_idesc(kBf16, 0, false, false);
    const uint32_t idesc_o = attn_idesc(kBf16, static_cast<uint32_t>(k_steps) * 16u, false, true);
    const uint32_t lead_v = lead_mn(kv_block);
    const uint32_t q_lo = (smem_u32(smem + p.off_q) + g * p.q_stages * L::kQTile) >> 4;
    const uint32_t kv_lo = smem_u32(smem + p.off_kv) >> 4;
    const uint32_t kv_tile_lo = kv_tile >> 4, kv_block_lo = kv_block >> 4;
    const uint32_t ts = tmem + g * 128, to = tmem + G * 128 + g * DP;
    bool ok = true;
    int stage = 0, qs = 0;
    uint32_t phase = 0, q_phase = 0, tiles = 0, items = 0;
    auto advance = [&]() {
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    auto next_q = [&]() {
      if (++qs == p.q_stages) {
        qs = 0;
        q_phase ^= 1u;
      }
    };
    uint32_t turns = 0;  // strictly in turn: both groups have the same steps
    auto take_turn = [&]() {
      return G == 1 || wait(&bars.turn[g], (turns & 1u) ^ (g == 0 ? 1u : 0u), kAttnMmaTimeout);
    };
    auto end_turn = [&]() {
      if (G == 2 && lane == 0) mbar_arrive(smem_u32(&bars.turn[g ^ 1]));
      ++turns;
    };
    Walk<L::kSplit, kMask, AttnFwdParams> w(p, start);
    // Items without a row tile for this group: their stages are passed on.
    // (Only once the group's own batches are issued: it would hold the last
    // values' stage all along.  The queries' stage first, when the loads have
    // come to it: the other group's last turn of an item waits for keys that
    // are loaded behind the next item's queries.)
    auto absent = [&]() { return G == 2 && w.live && g >= w.tiles_here; };
    auto skip_absent = [&]() {
      while (ok && absent()) {
        ok = wait(&bars.q_full[g][qs], q_phase, kAttnMmaTimeout);
        if (!ok) break;
        mma_commit_warp(smem_u32(&bars.q_empty[g][qs]));
        next_q();
        for (int t = w.first(); ok && t < w.t1; t = w.after(t)) {
          for (int i = 0; ok && i < 2; ++i) {
            ok = wait(&bars.kv_full[stage], phase, kAttnMmaTimeout);
            if (ok && lane == 0) mbar_arrive(smem_u32(&bars.kv_empty[stage]));
            advance();
          }
          ok = ok && take_turn();
          if (ok) end_turn();
        }
        w.next();
      }
    };
    // S of key stage `k_stage`, into the group's columns.
    auto scores = [&](int k_stage, int cols) {
      const uint32_t a = kLeadK | (q_lo + qs * (L::kQTile >> 4));
      const uint32_t b = kLeadK | (kv_lo + k_stage * kv_tile_lo);
      const uint32_t id = idesc_s | (static_cast<uint32_t>(cols >> 3) << 17);
      mma_ss_x4(ts, a, b, id, 0u, k_steps);
      if (k_steps > 4) mma_ss_x4(ts, a + 1024u, b + kv_block_lo, id, 1u, k_steps - 4);
      mma_commit_warp(smem_u32(&bars.s_full[g]));
    };
    int t = 0, after = 0, cols = 0;
    bool first = true;
    // The next item that has a row tile for the group, and its first scores.
    auto begin = [&]() {
      skip_absent();
      if (!ok || !w.live) return false;
      t = w.first();
      after = w.after(t);
      cols = w.tile_cols(t);
      first = true;
      ok = wait(&bars.q_full[g][qs], q_phase, kAttnMmaTimeout) &&
           wait(&bars.kv_full[stage], phase, kAttnMmaTimeout);
      if (!ok) return false;
      tc_fence_after();
      scores(stage, cols);
      mma_commit_warp(smem_u32(&bars.kv_empty[stage]));
      if (after >= w.t1) mma_commit_warp(smem_u32(&bars.q_empty[g][qs]));
      advance();
      return true;
    };
    bool live = begin();
    while (ok && live) {
      // This step's values, then the next step's keys.
      const int v_stage = stage, keys = w.tile_keys(t), this_cols = cols;
      if (kMask || p.a.kv_lengths) ok = wait(&bars.kv_full[stage], phase, kAttnMmaTimeout);
      if (!ok) break;
      const uint32_t v_phase = phase;
      advance();
      // Values that no row of the CTA takes part with are cleared, so that
      // nothing they hold meets a zero of P: keys past the request's length
      // (past the tensor's end the load has filled zeros), and masked keys.
      // (Each group's warp clears them; both write the same zeros.)
      if (kMask || (keys < this_cols && p.a.kv_lengths)) {
        uint4 used = first_keys(keys);
        if (kMask) {
          const uint4 any = w.any_keys(t);
          used = make_uint4(used.x & any.x, used.y & any.y, used.z & any.z, used.w & any.w);
        }
        clear_rows<L::kBlocks>(smem + p.off_kv + v_stage * kv_tile, kv_block, this_cols, used, lane);
        fence_proxy_async_shared();
        __syncwarp();
      }
      bool more = true, next_item = false;
      if (after >= w.t1) {
        w.next();
        next_q();
        more = w.live && !absent();
        next_item = true;
        if (more) t = w.first();
      } else {
        t = after;
      }
      if (more) {
        after = w.after(t);
        cols = w.tile_cols(t);
      }
      WaitSet tiles_in(&bars.kv_full[v_stage], v_phase, lane);
      tiles_in.also<1>(&bars.kv_full[stage], phase, more);
      tiles_in.also<2>(&bars.q_full[g][qs], q_phase, more && next_item);
      tiles_in.also<3>(&bars.o_free[g], (items - 1) & 1u, first && items > 0);
      ok = wait_set(tiles_in);
      if (first) ++items;
      // The first 64 keys' products start before the others' P is there.  The
      // groups take turns with whole batches (P v, then the next S): products
      // of two batches in between one another would end together, and both
      // groups' exponentials would leave the tensor core idle.
      WaitSet ready(&bars.p_half[g], tiles & 1u, lane);
      ready.also<1>(&bars.turn[g], (turns & 1u) ^ (g == 0 ? 1u : 0u), G == 2);
      ok = ok && wait_set(ready);
      if (!ok) break;
      tc_fence_after();
      const uint32_t b = lead_v | (kv_lo + v_stage * kv_tile_lo);
      const int steps = this_cols >> 4;
      mma_ts_x4(to, ts, b, idesc_o, first ? 0u : 1u, steps);
      ok = wait(&bars.p_full[g], tiles & 1u, kAttnMmaTimeout);
      if (!ok) break;
      tc_fence_after();
      if (steps > 4) mma_ts_x4(to, ts + 32, b + 512u, idesc_o, 1u, steps - 4);
      ++tiles;
      // (Announced before the next scores are: who has seen those can tell this
      // product's phase from the one before.)
      mma_commit_warp(smem_u32(&bars.o_done[g]));
      const int k_stage = stage;
      if (more) {
        scores(stage, cols);
        advance();
      }
      end_turn();
      mma_commit_warp(smem_u32(&bars.kv_empty[v_stage]));
      if (more) {
        mma_commit_warp(smem_u32(&bars.kv_empty[k_stage]));
        if (after >= w.t1) mma_commit_warp(smem_u32(&bars.q_empty[g][qs]));
      }
      first = next_item;
      live = more || begin();
    }
    if (!ok) {
      // Every MMA already issued must finish before TMEM is released.
      mma_commit_warp(smem_u32(&bars.drain[g]));
      mbar_wait_drain(smem_u32(&bars.drain[g]), 0, limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp < 4 * G) {
    // ------------------------------------------------------------ softmax
    if (G == 2) take_registers<208>();
    const int g = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + g * 128 + lane_field;
    const uint32_t to = tmem + G * 128 + g * DP + lane_field;
    const uint32_t bar_id = 1 + g;
    const float c2 = p.scale_log2;
    const int d = p.a.head_dim;
    uint8_t* stage_out = smem + p.off_out + g * 16384;
    // The thread's row of every tile: (token, head) from the tile's first.
    const int row_token = p.tile_heads > 1 ? r / p.tile_heads : r;
    const int row_head = p.tile_heads > 1 ? r - row_token * p.tile_heads : 0;
    uint32_t tiles = 0;  // S tiles seen: barrier parity
    bool ok = true;
    for (Walk<L::kSplit, kMask, AttnFwdParams> w(p, start); ok && w.live; w.next()) {
      if (g >= w.tiles_here) continue;
      int token, head;
      w.place(g, &token, &head);
      token += row_token;
      head += row_head;
      const bool row_ok = row_token < p.tile_tokens && token < p.a.q_len;
      const bool warp_ok = __any_sync(0xFFFFFFFFu, row_ok);
      const uint32_t* bits = nullptr;
      if (kMask && row_ok)
        bits = p.a.mask_bits +
               (w.b * p.a.mask_b + head * p.a.mask_h + token * p.a.mask_q) * p.a.mask_words;
      float m = -INFINITY, mc = 0.f, l = 0.f;
      bool first = true;
      for (int t = w.first(); t < w.t1; t = w.after(t), first = false) {
        const int keys = w.tile_keys(t), cols = w.tile_cols(t);
        uint32_t word[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
        if (kMask) {
          // A tile of kv_box keys starts inside a row of whole 128-key words
          // only when it is the row's single tile (kv_box < 128).
          uint4 q = make_uint4(0, 0, 0, 0);
          if (bits) q = *reinterpret_cast<const uint4*>(bits + (t * p.kv_box >> 5));
          word[0] = q.x; word[1] = q.y; word[2] = q.z; word[3] = q.w;
        }
        ok = wait(&bars.s_full[g], tiles & 1u, kAttnSoftmaxTimeout);
        if (!ok) break;
        tc_fence_after();
        // The row's running maximum takes in `mx`.
        auto grow = [&](float mx) __attribute__((always_inline)) {
          if (first) {
            m = mx;
            mc = m == -INFINITY ? 0.f : fmaf(m, c2, -kShift<T>);
          } else {
            const bool grown = (mx - m) * c2 > kRescaleLog2;  // (false for -inf - -inf = NaN)
            if (__any_sync(0xFFFFFFFFu, grown)) {
              float f = 1.f;
              if (grown) {
                const float next = fmaf(mx, c2, -kShift<T>);
                f = m == -INFINITY ? 0.f : exp2_approx(mc - next);
                m = mx;
                mc = next;
                l *= f;
              }
              // The product of the tile before has to be done.
              ok = wait(&bars.o_done[g], (tiles - 1) & 1u, kAttnSoftmaxTimeout);
              if (!ok) return;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < d; c += 16) {  // (16 columns: the scores stay in registers)
                uint32_t o[16];
                tmem_ld_x16(to + c, o);
                tmem_wait_ld_x16(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st_x16(to + c, o);
              }
              tmem_wait_st();
            }
          }
        };
        if (keys == 128 && !kMask) {
          // A whole tile: straight-line code.
          if (warp_ok) {
            uint32_t s[128];
            // (The second half of the scores loads beside the first one's maximum.)
            tmem_ld_x32(ts, s);
            tmem_ld_x32(ts + 32, s + 32);
            tmem_wait_ld();
            tmem_pin<64>(s);
            tmem_ld_x32(ts + 64, s + 64);
            tmem_ld_x32(ts + 96, s + 96);
            float top[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top[i] = fmaxf(__uint_as_float(s[i]), __uint_as_float(s[4 + i]));
#pragma unroll
            for (int i = 8; i < 64; i += 8)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                top[j] = max3(top[j], __uint_as_float(s[i + j]), __uint_as_float(s[i + 4 + j]));
            tmem_wait_ld();
            tmem_pin<64>(s + 64);
#pragma unroll
            for (int i = 64; i < 128; i += 8)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                top[j] = max3(top[j], __uint_as_float(s[i + j]), __uint_as_float(s[i + 4 + j]));
            grow(max3(fmaxf(top[0], top[1]), top[2], top[3]));
            if (!ok) break;
            const uint64_t c22 = pack2(c2, c2), mc2 = pack2(-mc, -mc);
            uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t h[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(s[c * 32 + 2 * i]),
                                   __uint_as_float(s[c * 32 + 2 * i + 1])),
                             c22, mc2),
                        x, y);
                x = exp2_approx(x);
                y = exp2_approx(y);
                sum[i & 3] = add2(sum[i & 3], pack2(x, y));
                h[i] = round2<T>(x, y);
              }
              if (c == 3) {
                // (By now the stores of the first half have arrived.)
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.p_half[g]));
              }
              tmem_st_x16(ts + c * 16, h);
            }
            float x, y;
            unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), x, y);
            l += x + y;
            tmem_wait_st();
          } else if (lane == 0) {
            mbar_arrive(smem_u32(&bars.p_half[g]));
          }
        } else {
          // A part of a tile, or a mask: two passes over the scores, 32 at a
          // time.  (P of a chunk lies over scores read before it is stored.)
          if (warp_ok) {
            auto chunk = [&](int c, uint32_t* s) __attribute__((always_inline)) {
              tmem_ld_x32(ts + c * 32, s);
              tmem_wait_ld_x32(s);
              uint32_t on = c == 0 ? word[0] : c == 1 ? word[1] : c == 2 ? word[2] : word[3];
              const int rest = keys - c * 32;
              if (rest < 32) on &= rest <= 0 ? 0u : (1u << rest) - 1u;
              if (on != 0xFFFFFFFFu) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!((on >> i) & 1u)) s[i] = 0xFF800000u;  // -infinity
              }
            };
            const int chunks = (cols + 31) >> 5;
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              uint32_t s[32];
              chunk(c, s);
              float top[4] = {mx, mx, mx, mx};
#pragma unroll
              for (int i = 0; i < 32; i += 8)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  top[j] = max3(top[j], __uint_as_float(s[i + j]), __uint_as_float(s[i + 4 + j]));
              mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
            }
            grow(mx);
            if (!ok) break;
            const uint64_t c22 = pack2(c2, c2), mc2 = pack2(-mc, -mc);
            uint64_t sum[2] = {0, 0};
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              uint32_t s[32], h[16];
              chunk(c, s);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c22, mc2),
                        x, y);
                x = exp2_approx(x);
                y = exp2_approx(y);
                sum[i & 1] = add2(sum[i & 1], pack2(x, y));
                h[i] = round2<T>(x, y);
              }
              tmem_st_x16(ts + c * 16, h);
            }
            float x, y;
            unpack2(add2(sum[0], sum[1]), x, y);
            l += x + y;
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.p_half[g]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[g]));
        ++tiles;
      }
      if (ok) ok = wait(&bars.o_done[g], (tiles - 1) & 1u, kAttnSoftmaxTimeout);
      // The staging buffer's last store has been read; every warp agrees that
      // the item is complete.
      if (quarter == 0 && lane == 0) bulk_wait_read_all();
      ok = barrier_all(bar_id, 128, ok);
      if (!ok) break;
      tc_fence_after();
      const bool whole = !L::kSplit || (w.t0 == 0 && w.t1 == w.nt);
      if (!whole) {
        // A share of the row's keys: unnormalised, with its maximum and sum.
        const long long slot = 2ll * blockIdx.x + (w.t0 == 0 ? 1 : 0);
        if (warp_ok) {
          float* dst = p.part_out + (slot * kAttnRows + r) * 128;
#pragma unroll 1
          for (int c = 0; c < d; c += 32) {
            uint32_t o[32];
            tmem_ld_x32(to + c, o);
            tmem_wait_ld_x32(o);
            if (row_ok)
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                if (c + i < d)
                  *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
          if (row_ok)
            *reinterpret_cast<float2*>(p.part_stat + (slot * kAttnRows + r) * 2) =
                make_float2(m == -INFINITY ? -INFINITY : mc, l);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.o_free[g]));
        continue;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (p.a.lse && row_ok)
        p.a.lse[(static_cast<long long>(w.b) * p.a.heads + head) * p.a.q_len + token] =
            l == 0.f ? -INFINITY : row_lse<T>(mc, l);
      int token0, head0;
      w.place(g, &token0, &head0);
#pragma unroll 1
      for (int blk = 0; blk < L::kBlocks; ++blk) {
        if (blk * 64 >= d) break;
        if (blk > 0) {
          if (quarter == 0 && lane == 0) bulk_wait_read_all();
          named_barrier(bar_id, 128);
        }
        if (warp_ok) {
          uint32_t o[64];
          tmem_ld_x32(to + blk * 64, o);
          tmem_ld_x32(to + blk * 64 + 32, o + 32);
          tmem_wait_ld();
          tmem_pin<64>(o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              h[j] = round2<T>(__uint_as_float(o[i * 8 + 2 * j]) * inv,
                               __uint_as_float(o[i * 8 + 2 * j + 1]) * inv);
            // 16-byte words of a row sit at their index XOR the row's low bits (128-byte swizzle).
            *reinterpret_cast<uint4*>(stage_out + r * 128 + ((i ^ (r & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        fence_proxy_async_shared();
        if (blk == L::kBlocks - 1 || (blk + 1) * 64 >= d) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.o_free[g]));
        }
        named_barrier(bar_id, 128);
        if (quarter == 0 && lane == 0) {
          tma_store_4d(&p.map_out, smem_u32(stage_out), blk * 64, head0, token0, w.b);
          bulk_commit_group();
        }
      }
    }
    // Shared memory stays until the last store has read it.
    if (quarter == 0 && lane == 0) bulk_wait_read_all();
    __syncwarp();
  } else {
    if (G == 2) give_registers<80>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == L::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Joins the shares of row tiles that a split launch cut, in order, with
// weights 2^(m_f - max m) over the shares' maxima.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
    attn_join_kernel(const __grid_constant__ AttnFwdParams p, int ctas) {
  __shared__ JoinSlots join;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnShape& a = p.a;
  const int b = static_cast<int>(blockIdx.x / p.item_rows);
  const int item = static_cast<int>(blockIdx.x - b * p.item_rows);
  grid_dependency_wait();
  grid_launch_dependents();
  long long before, total;
  split_prefix(a.batch, row_steps_uniform(p), b, join.sums, [&](int i) { return row_steps(p, i); },
               &before, &total);
  const int nt = key_tiles(valid_keys(a, b), p.kv_box);
  list_slots(join, total, ctas, before + static_cast<long long>(item) * nt, nt);
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
  const int d0 = lane * 4;
  const int r0 = blockIdx.y * kJoinRows + warp * kJoinUnroll;
  if (r0 >= rows) return;
  // (Rows past the tile's read its last row again and write nothing.)
  float m[kJoinUnroll], l[kJoinUnroll];
  float4 acc[kJoinUnroll];
#pragma unroll
  for (int u = 0; u < kJoinUnroll; ++u) {
    m[u] = -INFINITY;
    l[u] = 0.f;
    acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int c = lane; c < shares; c += 32)
#pragma unroll
    for (int u = 0; u < kJoinUnroll; ++u) {
      const long long row = static_cast<long long>(join.slots[c]) * kAttnRows + min(r0 + u, rows - 1);
      m[u] = fmaxf(m[u], p.part_stat[row * 2]);
    }
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int u = 0; u < kJoinUnroll; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(0xFFFFFFFFu, m[u], o));
#pragma unroll 2
  for (int c = 0; c < shares; ++c)
#pragma unroll
    for (int u = 0; u < kJoinUnroll; ++u) {
      const long long row = static_cast<long long>(join.slots[c]) * kAttnRows + min(r0 + u, rows - 1);
      const float2 st = *reinterpret_cast<const float2*>(p.part_stat + row * 2);
      // A share whose pairs are all left out holds zeros.
      const float f = st.x == -INFINITY && st.y == 0.f ? 0.f : exp2_approx(st.x - m[u]);
      l[u] = fmaf(f, st.y, l[u]);
      if (d0 < a.head_dim) {
        const float4 v = *reinterpret_cast<const float4*>(p.part_out + row * 128 + d0);
        acc[u].x = fmaf(f, v.x, acc[u].x);
        acc[u].y = fmaf(f, v.y, acc[u].y);
        acc[u].z = fmaf(f, v.z, acc[u].z);
        acc[u].w = fmaf(f, v.w, acc[u].w);
      }
    }
#pragma unroll
  for (int u = 0; u < kJoinUnroll; ++u) {
    const int r = r0 + u;
    if (r >= rows) break;
    const int dt = p.tile_heads > 1 ? r / p.tile_heads : r;
    const int token = token0 + dt, head = p.tile_heads > 1 ? head0 + r - dt * p.tile_heads : head0;
    const float inv = l[u] == 0.f ? 0.f : 1.f / l[u];
    if (d0 < a.head_dim)
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out_w) + b * a.os[0] + token * a.os[1] +
                                head * a.os[2] + d0) =
          make_uint2(round2<T>(acc[u].x * inv, acc[u].y * inv), round2<T>(acc[u].z * inv, acc[u].w * inv));
    if (a.lse && lane == 0)
      a.lse[(static_cast<long long>(b) * a.heads + head) * a.q_len + token] =
          l[u] == 0.f ? -INFINITY : row_lse<T>(m[u], l[u]);
  }
}

// Outputs of a call without keys.
__global__ void __launch_bounds__(256) attn_no_keys_kernel(const AttnShape a) {
  const long long rows = static_cast<long long>(a.batch) * a.q_len * a.heads;
  const int words = a.head_dim / 8;
  grid_dependency_wait();
  grid_launch_dependents();
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < rows * words;
       i += step) {
    const long long row = i / words;
    const int h = static_cast<int>(row % a.heads);
    const long long bt = row / a.heads;
    const long long b = bt / a.q_len, t = bt - b * a.q_len;
    *reinterpret_cast<uint4*>(static_cast<__half*>(a.out_w) + b * a.os[0] + t * a.os[1] +
                              h * a.os[2] + (i - row * words) * 8) = make_uint4(0, 0, 0, 0);
    if (a.lse && i == row * words) a.lse[(b * a.heads + h) * a.q_len + t] = -INFINITY;
  }
}

template <typename T, int DP, int G, bool kMask>
cudaError_t launch_masked(const AttnFwdParams& p, int grid, size_t smem, cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  const cudaError_t err = raise_smem(attn_fwd_kernel<T, DP, G, kMask>, configured, smem);
  if (err != cudaSuccess) return err;
  return launch_pdl(attn_fwd_kernel<T, DP, G, kMask>, dim3(grid), dim3(Layout<T, DP, G>::kThreads), smem, stream, p);
}

template <typename T, int DP, int G>
cudaError_t launch_one(const AttnFwdParams& p, int grid, size_t smem, cudaStream_t stream) {
  return p.a.mask_bits ? launch_masked<T, DP, G, true>(p, grid, smem, stream)
                       : launch_masked<T, DP, G, false>(p, grid, smem, stream);
}

template <typename T>
cudaError_t launch_type(const AttnFwdParams& p, bool split, int grid, size_t smem,
                        cudaStream_t stream) {
  const bool wide = p.a.head_dim > 64;
  cudaError_t err;
  if (!split)
    return wide ? launch_one<T, 128, 2>(p, grid, smem, stream)
                : launch_one<T, 64, 2>(p, grid, smem, stream);
  err = wide ? launch_one<T, 128, 1>(p, grid, smem, stream)
             : launch_one<T, 64, 1>(p, grid, smem, stream);
  // Rows of one key tile are never cut.
  if (err != cudaSuccess || p.a.kv_len <= p.kv_box) return err;
  const int rows = p.tile_heads * p.tile_tokens;
  return launch_pdl(attn_join_kernel<T>,
                    dim3(static_cast<unsigned>(p.item_rows * p.a.batch), (rows + kJoinRows - 1) / kJoinRows),
                    dim3(kJoinThreads), 0, stream, p, grid);
}

}  // namespace

cudaError_t launch_attn_no_keys(const AttnShape& a, cudaStream_t stream) {
  const long long words = static_cast<long long>(a.batch) * a.q_len * a.heads * (a.head_dim / 8);
  const int grid = static_cast<int>(words / 256 < 2048 ? words / 256 + 1 : 2048);
  return launch_pdl(attn_no_keys_kernel, dim3(grid), dim3(256), 0, stream, a);
}

size_t attn_fwd_bar_bytes() { return sizeof(Bars); }

cudaError_t launch_attn_fwd(const AttnFwdParams& p, bool split, int grid, size_t smem,
                            cudaStream_t stream) {
  return p.a.dtype == 0 ? launch_type<__nv_bfloat16>(p, split, grid, smem, stream)
                        : launch_type<__half>(p, split, grid, smem, stream);
}

}  // namespace convgb300
