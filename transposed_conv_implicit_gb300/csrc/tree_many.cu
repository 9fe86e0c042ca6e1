// Attention of drafted tokens to the paged 8-bit cache, many rows to a key
// head, on the tensor cores.
//
//   s = scale q K^T,  p = exp(s - max),  out = (p V) / sum p
//
// The forward attention's scheme: a softmax group of four warps owns a row
// tile of 128 (draft, head) rows, one thread per row; S (fp32, TMEM) comes from
// one tcgen05.mma over the head dimension, the thread writes P (fp16) over it,
// and the second tcgen05.mma takes P from TMEM against V; the output stays in
// TMEM and is rescaled only when a row's maximum grows by more than 2^kTreeLag.
// A tile of 128 keys goes by halves of 64: while a group's threads turn one
// half's scores into P, the tensor core multiplies the other's.  (By whole
// tiles, with the scores read twice, 196 us at 16 x 64 drafts x 32 heads against
// 8192 keys.)
//
// The keys come as 8-bit codes from pages of any strides, and the products
// want 16-bit operands in shared memory: eight warps copy codes with cp.async
// (each lane what it will read itself, two tiles ahead), widen them and store
// them where TMA would have put 128-byte rows with the 128-byte swizzle.  That
// is work for each key tile, so a CTA has two softmax groups that share the
// widened tiles:
//  - an item of more than 128 rows: the groups are two row tiles;
//  - an item of up to 128 rows: both groups hold the same rows, and take the
//    key tiles in turn.  A row is the same lane of tensor memory in both, so
//    where the CTA has all of the item each group reads the other's output
//    there and writes half of the columns; else each leaves a share of its own
//    for the join.
// The sequence of all items' key tiles is cut evenly between the CTAs (one per
// SM), as for few rows.  A CTA leaves at most two items' shares: of one that
// began in front of its part, and of one that ends behind it.
//
// Bound by the order of exponentials, widening (issue slots 53 %) and products (47
// % of their pipe), of which neither is full: 64 drafts of 16 requests x 32/8 heads
// x 128 against 8192 keys 168 us, its join with it (0.81 PFLOP/s; 0.99 for each
// further key).
//
// Numbers, as for few rows, but that scales are common to 16 keys: codes become
// fp16 times their row's scale relative to the largest of the slice of 16 that
// the row lies in (a key's by 2^-24 at least, a value's by 2^-31: rows further
// below become 0), whose exponents go to the slice's scores (keys: E) and with
// the probabilities (values: F): w = 2^(y - M), y = s log2(e) + F, M the running
// maximum of y less kTreeShift; the sum of probabilities adds 2^-F w.  (With
// every row's scale applied in fp32 and rounded to the queries' type the
// widening took 60 instructions for 16 codes, 28 now, and the whole pass 213 us
// at 16 x 64 drafts x 32 heads against 8192 keys.)
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "tree_common.cuh"

namespace convgb300 {

namespace {

constexpr int kRowsMany = 128;               // of a group
constexpr int kWordStages = 3;               // widened tiles of keys or values
constexpr int kCodeStages = 3;               // tiles of codes in flight
constexpr int kHalfKeys = 64;                // of a tile: scores and probabilities go by halves
constexpr int kSlotsMany = 4;                // tiles whose validity and scales are kept
// Two softmax groups, a group of which two warps issue the products, and the
// widening's warps, which take a slice of 16 keys each.  Registers of a thread:
// (136 + 136 + 64 + 72 + 72) * 128 = 96 * 640.
constexpr int kWidenWarps = 8;
constexpr int kThreadsMany = 32 * (12 + kWidenWarps);
constexpr uint32_t kBlockBytes = 128 * 128;  // 128 keys (or rows) x 64 elements

template <int DP>
struct Many {
  static constexpr int kBlocks = DP / 64;
  static constexpr uint32_t kTile = kBlockBytes * kBlocks;       // a widened tile; a row tile
  static constexpr uint32_t kOffWords = 2 * kTile;
  static constexpr int kPieces = 2 * kBlocks;                    // 16-byte words a lane takes of a tile
  static constexpr uint32_t kCodeWarp = kPieces * 512 + 2 * 128; // a warp's codes and scales of a tile
  static constexpr uint32_t kOffCodes = kOffWords + kWordStages * kTile;
  static constexpr uint32_t kOffShared = kOffCodes + kCodeStages * kWidenWarps * kCodeWarp;
};

struct ManyShared {
  uint64_t kv_full[kWordStages], kv_empty[kWordStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];  // [group][half of a tile]
  uint64_t drain[2];
  uint64_t meet;  // the groups, over an item whose rows both hold: statistics are there, outputs have been read
  SplitStart start;
  uint32_t tmem;
  int abort_flag;
  alignas(16) uint16_t valid[kSlotsMany][kWidenWarps];  // keys of a tile that are there
  alignas(16) float scale[kSlotsMany][3][kWidenWarps];  // of a slice: 2^E, F, 2^-F (see above)
  int parents[2][kMaxDrafts];
  uint32_t bits[2][kTreeWords][kRowsMany];  // drafts that a row attends
  float2 stat[2][kRowsMany];                // a group's maximum and sum, for the other group
};

// 2^-below as fp16, twice; 0 below 2^-24.
__device__ __forceinline__ uint32_t half_power(int below) {
  const uint32_t h = below <= 14 ? static_cast<uint32_t>(15 - below) << 10 : below <= 24 ? 1u << (24 - below) : 0u;
  return h | (h << 16);
}
constexpr int kValueLift = 7;  // values stay below 448 2^7 < 65504

// Sixteen codes as fp16 times `factor`.
__device__ __forceinline__ void widen16(uint4 codes, uint32_t factor, uint4& first, uint4& second) {
  const uint32_t u[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    widen_codes4(u[i], w[2 * i], w[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(w[2 * i + j]) : "r"(factor));
  }
  first = make_uint4(w[0], w[1], w[2], w[3]);
  second = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int DP>
constexpr size_t many_smem() {
  static_assert(Many<DP>::kOffShared + sizeof(ManyShared) <= 227 * 1024, "a block's shared memory");
  return Many<DP>::kOffShared + sizeof(ManyShared);
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreadsMany, 1)
    tree_many_kernel(const __grid_constant__ TreeParams p) {
  using L = Many<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  ManyShared& sh = *reinterpret_cast<ManyShared*>(smem + L::kOffShared);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh.abort_flag;
  unsigned int* status = p.status;
  const long long limit = p.timeout_cycles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kWordStages; ++s) {
      mbar_init(smem_u32(&sh.kv_full[s]), kWidenWarps);
      mbar_init(smem_u32(&sh.kv_empty[s]), 2);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&sh.q_full[g]), 4);
      mbar_init(smem_u32(&sh.q_empty[g]), 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(smem_u32(&sh.s_full[g][h]), 1);
        mbar_init(smem_u32(&sh.p_full[g][h]), 4);
        mbar_init(smem_u32(&sh.o_done[g][h]), 1);
      }
      mbar_init(smem_u32(&sh.drain[g]), 1);
    }
    mbar_init(smem_u32(&sh.meet), 8);
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  grid_dependency_wait();
  if (warp == 0) {
    const SplitStart st = split_start(p.batch, -1, lane, [&](int b) { return tree_steps(p, b); });
    if (lane == 0) sh.start = st;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();  // (TMEM is held: what starts now cannot take it first)
  const uint32_t tmem = sh.tmem;
  const SplitStart start = sh.start;
  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned int code) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(bar), parity, abort_flag, status, code, limit));
  };

  if (warp >= 12) {
    // ------------------------------------------------------------ codes to operands
    give_registers<72>();
    const int w8 = warp - 12;
    const uint32_t codes = smem_u32(smem + L::kOffCodes) + w8 * L::kCodeWarp;
    // A lane's rows of the warp's slice of 16 (which lies in one page): row8 and row8 + 8; its 16
    // codes of each 64: col.  (Two rows of four lanes together store to all banks.)
    const int row8 = lane >> 2, col = lane & 3;
    // Bytes that the lane copies of a row's 64 codes: none behind its end.
    const int whole_bytes[2] = {col * 16 < p.c.head_dim ? 16 : 0, (4 + col) * 16 < p.c.head_dim ? 16 : 0};
    // What is copied next: tile lt of item lw, where the warp's slice of it lies (`page` as the table
    // has it, read a tile ahead so that nothing waits for it; an item's first one is waited for).
    TreeWalk lw(p, start);
    int lt = 0, page = -1, next_page = -1, from = 0, offset = 0, keys = 0;
    const uint8_t *k_lane = nullptr, *v_lane = nullptr, *s_lane = nullptr;
    auto page_at = [&](int t) {
      const int slice = t * kWidenWarps + w8;
      return slice * 16 < lw.size.keys ? p.c.table[lw.b * p.c.table_stride + fast_div(slice, p.div_slices)] : -1;
    };
    auto begin_item = [&]() {
      if (!lw.live) return;
      lt = lw.t0;
      page = page_at(lt);
      k_lane = p.c.k + lw.hk * p.c.ks[2] + row8 * p.c.ks[1] + col * 16;
      v_lane = p.c.v + lw.hk * p.c.vs[2] + row8 * p.c.vs[1] + col * 16;
      s_lane = p.c.scales + static_cast<long long>(lw.hk) * p.c.page_size * 2 + 2 * (row8 & ~1);
    };
    begin_item();
    auto copy_rows = [&](const uint8_t* rows, long long eight, uint32_t to) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int c = 0; c < L::kBlocks; ++c)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           to + ((k * L::kBlocks + c) * 32 + lane) * 16),
                       "l"(rows + (k ? eight : 0) + c * 64), "r"(8 * k + row8 < keys ? whole_bytes[c] : 0)
                       : "memory");
    };
    auto load_keys = [&](int stage) {
      if (lw.live) {
        const int slice = lt * kWidenWarps + w8;
        const bool real = static_cast<unsigned int>(page) < static_cast<unsigned int>(p.c.pages);
        from = real ? page : 0;
        offset = (slice - fast_div(slice, p.div_slices) * static_cast<int>(p.div_slices.d)) * 16;
        keys = real ? lw.size.keys - slice * 16 : 0;  // that are there
        if (lt + 1 < lw.t1) next_page = page_at(lt + 1);
        const uint32_t to = codes + stage * (kWidenWarps * L::kCodeWarp);
        copy_rows(k_lane + (from * p.c.ks[0] + offset * p.c.ks[1]), p.ks8, to);
        // The scales of two keys each, of which those that are there.
        const uint8_t* sc = s_lane + (from * p.scale_page + offset * 2);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int there = keys - 8 * k - (row8 & ~1);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                           to + L::kPieces * 512 + (k * 32 + lane) * 4),
                       "l"(sc + 16 * k), "r"(there >= 2 ? 4 : there == 1 ? 2 : 0)
                       : "memory");
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto load_values = [&](int stage) {
      if (lw.live) {
        copy_rows(v_lane + (from * p.c.vs[0] + offset * p.c.vs[1]), p.vs8,
                  codes + stage * (kWidenWarps * L::kCodeWarp));
        if (++lt < lw.t1) {
          page = next_page;
        } else {
          lw.next();
          begin_item();
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    static_assert(kCodeStages == 3, "a tile's keys, and its values, are copied a tile ahead");
    load_keys(0);
    load_values(1);
    bool ok = true;
    int code_stage = 0, stage = 0;
    uint32_t phase = 0, tiles = 0;
    for (TreeWalk w(p, start); ok && w.live; w.next()) {
      for (int t = w.t0; ok && t < w.t1; ++t, ++tiles) {
        uint32_t factor[2][2];  // of the rows' codes: keys', values'
        bool there[2];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int ahead = code_stage == 0 ? kCodeStages - 1 : code_stage - 1;
          if (kv == 0)
            load_keys(ahead);
          else
            load_values(ahead);
          asm volatile("cp.async.wait_group %0;" ::"n"(kCodeStages - 1) : "memory");
          const uint32_t from_codes = codes + code_stage * (kWidenWarps * L::kCodeWarp);
          uint4 u[2][L::kBlocks];
          uint32_t two[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (kv == 0)
              two[k] = lds32(from_codes + L::kPieces * 512 + (k * 32 + lane) * 4) >> (16 * (row8 & 1)) & 0xFFFFu;
#pragma unroll
            for (int c = 0; c < L::kBlocks; ++c)
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(u[k][c].x), "=r"(u[k][c].y), "=r"(u[k][c].z), "=r"(u[k][c].w)
                           : "r"(from_codes + ((k * L::kBlocks + c) * 32 + lane) * 16));
          }
          ok = ok && wait(&sh.kv_empty[stage], phase ^ 1u, kAttnProducerTimeout);
          if (!ok) break;
          if (kv == 0) {
            // The rows' bytes, and the slice's largest.
            uint32_t mine = 0;
            int key_most = 0, value_most = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              there[k] = (two[k] & 0xFFu) != 0;
              if (there[k]) mine |= 1u << (8 * k + row8);
              if (!there[k]) two[k] = 0;
              key_most = max(key_most, static_cast<int>(two[k] & 0xFFu));
              value_most = max(value_most, static_cast<int>(two[k] >> 8));
            }
            key_most = __reduce_max_sync(0xFFFFFFFFu, key_most);
            value_most = __reduce_max_sync(0xFFFFFFFFu, value_most);
            mine = __reduce_or_sync(0xFFFFFFFFu, mine);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              factor[0][k] = half_power(key_most - static_cast<int>(two[k] & 0xFFu));
              factor[1][k] = half_power(value_most - static_cast<int>(two[k] >> 8) - kValueLift);
            }
            if (lane == 0) {
              const int f = value_most - 127 - kValueLift, slot = tiles % kSlotsMany;
              sh.valid[slot][w8] = static_cast<uint16_t>(mine);
              sh.scale[slot][0][w8] = __uint_as_float(static_cast<uint32_t>(key_most) << 23);
              sh.scale[slot][1][w8] = static_cast<float>(f);
              sh.scale[slot][2][w8] = __uint_as_float(static_cast<uint32_t>(min(254, 127 - f)) << 23);
            }
          }
          uint8_t* to = smem + L::kOffWords + stage * L::kTile + (w8 * 16 + row8) * 128;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int c = 0; c < L::kBlocks; ++c) {
              uint4 a, b;
              // (Where nothing was written there may be NaN.)
              widen16(there[k] ? u[k][c] : make_uint4(0, 0, 0, 0), factor[kv][k], a, b);
              uint8_t* row = to + c * kBlockBytes + k * 1024;
              *reinterpret_cast<uint4*>(row + (((2 * col) ^ row8) << 4)) = a;
              *reinterpret_cast<uint4*>(row + (((2 * col + 1) ^ row8) << 4)) = b;
            }
          fence_proxy_async_shared();
          __syncwarp();
          // (fault_mode 1, a test hook: every CTA leaves its first keys un-announced.)
          if (lane == 0 && !(p.fault_mode == 1 && tiles == 0 && kv == 0)) mbar_arrive(smem_u32(&sh.kv_full[stage]));
          code_stage = code_stage == kCodeStages - 1 ? 0 : code_stage + 1;
          if (++stage == kWordStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp == 8 || warp == 9) {
    // ------------------------------------------------------------ products
    give_registers<64>();
    const int g = warp - 8;
    const int k_steps = p.c.head_dim >> 4;
    const uint32_t idesc_s = attn_idesc(false, kHalfKeys, false, false);
    const uint32_t idesc_o = attn_idesc(false, static_cast<uint32_t>(p.c.head_dim), false, true);
    const uint32_t q_lo = kLeadK | ((smem_u32(smem) + g * L::kTile) >> 4);
    const uint32_t word_lo = smem_u32(smem + L::kOffWords) >> 4;
    const uint32_t ts = tmem + g * 128, to = tmem + 256 + g * DP;
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0, tiles = 0, items = 0;
    auto advance = [&]() {
      if (++stage == kWordStages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    // A tile's keys, or values, that the other group alone uses.
    auto pass = [&]() {
      ok = ok && wait(&sh.kv_full[stage], phase, kAttnMmaTimeout);
      if (ok && lane == 0) mbar_arrive(smem_u32(&sh.kv_empty[stage]));
      advance();
    };
    // Scores of a half of the tile whose keys are in stage `at`.
    auto scores = [&](int at, int half) {
      const uint32_t b = kLeadK | (word_lo + at * (L::kTile >> 4) + half * (kHalfKeys * 128 >> 4));
      mma_ss_x4(ts + half * kHalfKeys, q_lo, b, idesc_s, 0u, k_steps);
      if (k_steps > 4)
        mma_ss_x4(ts + half * kHalfKeys, q_lo + (kBlockBytes >> 4), b + (kBlockBytes >> 4), idesc_s, 1u, k_steps - 4);
      mma_commit_warp(smem_u32(&sh.s_full[g][half]));
    };
    for (TreeWalk w(p, start); ok && w.live; w.next()) {
      const bool single = w.size.drafts * p.group - w.row_tile * p.tile_rows <= kRowsMany;
      ok = wait(&sh.q_full[g], items & 1u, kAttnMmaTimeout);
      ++items;
      // Its own tiles: t, t + step, ...; the others pass.
      const int step = single ? 2 : 1;
      int t = w.t0 + (single ? g : 0);
      auto both_scores = [&]() {  // of the stage that comes next
        ok = ok && wait(&sh.kv_full[stage], phase, kAttnMmaTimeout);
        if (!ok) return;
        tc_fence_after();
        scores(stage, 0);
        scores(stage, 1);
        mma_commit_warp(smem_u32(&sh.kv_empty[stage]));
        advance();
      };
      if (single && g == 1) {
        pass();
        pass();
      }
      if (t < w.t1) both_scores();
      for (bool first = true; ok && t < w.t1; first = false) {
        // Half of the values, then the next tile's scores in that half's place (softmax has the
        // other half's scores meanwhile).  Where tiles are taken in turn, the next tile's keys come
        // when these values have left.
        const int v_stage = stage;
        ok = wait(&sh.kv_full[v_stage], phase, kAttnMmaTimeout);
        if (!ok) break;
        advance();
        const bool more = !single && t + 1 < w.t1;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          ok = wait(&sh.p_full[g][half], tiles & 1u, kAttnMmaTimeout);
          if (ok && more && half == 0) ok = wait(&sh.kv_full[stage], phase, kAttnMmaTimeout);
          if (!ok) break;
          tc_fence_after();
          mma_ts_x4(to, ts + half * kHalfKeys,
                    lead_mn(kBlockBytes) | (word_lo + v_stage * (L::kTile >> 4) + half * (kHalfKeys * 128 >> 4)),
                    idesc_o, first && half == 0 ? 0u : 1u, 4);
          // (A barrier for each half: who has seen the scores of a half knows the products of the
          // tile before to be done, so a wait for this half's cannot take the phase before for it.
          // With one barrier for both the two halves' phases could be taken for one another.)
          mma_commit_warp(smem_u32(&sh.o_done[g][half]));
          if (half == 1) mma_commit_warp(smem_u32(&sh.kv_empty[v_stage]));
          if (more) scores(stage, half);
        }
        if (!ok) break;
        ++tiles;
        if (more) {
          mma_commit_warp(smem_u32(&sh.kv_empty[stage]));
          advance();
        }
        if (single && t + 1 < w.t1) {
          pass();
          pass();
        }
        t += step;
        if (single && t < w.t1) both_scores();
      }
      // (The queries' place is free once these have been read.)
      mma_commit_warp(smem_u32(&sh.q_empty[g]));
    }
    if (!ok) {
      // Every MMA already issued must finish before TMEM is released.
      mma_commit_warp(smem_u32(&sh.drain[g]));
      mbar_wait_drain(smem_u32(&sh.drain[g]), 0, limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    take_registers<136>();
    const int g = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + g * 128 + lane_field, to = tmem + 256 + g * DP + lane_field;
    const uint32_t to_other = tmem + 256 + (g ^ 1) * DP + lane_field;
    const uint32_t bar_id = 1 + g;
    const int d = p.c.head_dim;
    uint32_t tiles = 0, items = 0, seen = 0;  // own tiles: barrier parity; all tiles: validity's slot
    bool ok = true, met = false;  // met: the other group may still be reading this one's last output
    for (TreeWalk w(p, start); ok && w.live; w.next()) {
      const int left = w.size.drafts * p.group - w.row_tile * p.tile_rows;
      const bool single = left <= kRowsMany;
      const bool whole = w.whole(), pair = single && whole;
      const int row = w.row_tile * p.tile_rows + (single ? r : g * kRowsMany + r);
      const bool row_ok = row < w.size.drafts * p.group;
      const bool warp_ok = __any_sync(0xFFFFFFFFu, row_ok);
      const int draft = row_ok ? fast_div(row, p.div_group) : 0;
      const int head = w.hk * p.group + (row_ok ? row - draft * p.group : 0);
      const int prefix = w.size.keys - w.size.drafts;
      ok = (!met || wait(&sh.meet, 1u, kAttnSoftmaxTimeout)) &&
           wait(&sh.q_empty[g], (items & 1u) ^ 1u, kAttnSoftmaxTimeout);
      ok = barrier_all(bar_id, 128, ok);
      if (!ok) break;
      met = pair;
      ++items;
      float rf = 0.f;  // of the row's scores: scale, and the query's power of two
      {
        // The queries as fp16, as TMA would place them: copied there as they are, kAtOnce of the
        // warp's rows side by side, then (bfloat16) each word by the lane that copied it.  Short
        // loops: a row a lane, or eight words in registers, took 24000 cycles an item for code that
        // runs once and is fetched every time.
        constexpr int kLanes = DP / 8, kAtOnce = 32 / kLanes;
        const int col = lane % kLanes;
        const int first_row = w.row_tile * p.tile_rows + (single ? 0 : g * kRowsMany) + quarter * 32;
        uint8_t* place = smem + g * L::kTile + (col >> 3) * kBlockBytes + quarter * 32 * 128;
#pragma unroll 2
        for (int i = 0; i < 32; i += kAtOnce) {
          const int at = i + lane / kLanes;  // of the warp's rows
          const bool on = first_row + at < w.size.drafts * p.group && col * 8 < d;
          const int at_draft = on ? fast_div(first_row + at, p.div_group) : 0;
          const int at_head = w.hk * p.group + (on ? first_row + at - at_draft * p.group : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_u32(place + at * 128 + (((col & 7) ^ (at & 7)) << 4))),
                       "l"(p.q + w.b * p.qs[0] + at_draft * p.qs[1] + at_head * p.qs[2] + (on ? col * 8 : 0)),
                       "r"(on ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        if constexpr (std::is_same<T, __half>::value) {
          rf = p.scale_log2;
        } else {
#pragma unroll 2
          for (int i = 0; i < 32; i += kAtOnce) {
            const int at = i + lane / kLanes;
            uint4* word = reinterpret_cast<uint4*>(place + at * 128 + (((col & 7) ^ (at & 7)) << 4));
            const uint4 v = *word;
            float top = fmaxf(fmaxf(larger_of(v.x), larger_of(v.y)), fmaxf(larger_of(v.z), larger_of(v.w)));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            float back;
            const float up = row_factor<T>(top, &back);
            *word = make_uint4(to_half(v.x, up), to_half(v.y, up), to_half(v.z, up), to_half(v.w, up));
            const float mine = __shfl_sync(0xFFFFFFFFu, back, (lane % kAtOnce) * kLanes);
            if (lane - lane % kAtOnce == i) rf = p.scale_log2 * mine;
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.q_full[g]));
      }
      if (w.t1 * kTreeKeys > prefix) {  // this share comes to the drafts
        if (p.parents)
          for (int i = r; i < w.size.drafts; i += 128) sh.parents[g][i] = p.parents[w.b * p.parent_stride + i];
        named_barrier(bar_id, 128);
        uint32_t mine[kTreeWords];
        draft_bits(p.parents ? sh.parents[g] : nullptr, draft, mine);
#pragma unroll
        for (int i = 0; i < kTreeWords; ++i) sh.bits[g][i][r] = mine[i];
      }
      float mc = -INFINITY, l = 0.f;  // the running maximum less kTreeShift, the sum
      bool first = true;
      const int step = single ? 2 : 1;
      for (int t = w.t0 + (single ? g : 0); ok && t < w.t1; t += step) {
        const int slot = static_cast<int>((seen + t - w.t0) % kSlotsMany);
#pragma unroll 1
        for (int half = 0; half < 2; ++half, first = false) {
          ok = wait(&sh.s_full[g][half], tiles & 1u, kAttnSoftmaxTimeout);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ts_half = ts + half * kHalfKeys;
          uint32_t s[64];
          if (warp_ok) {
            tmem_ld_x32(ts_half, s);
            tmem_ld_x32(ts_half + 32, s + 32);
          }
          // Of the half's slices: the factor of their scores (not 0, for the sake of scores that are
          // left out: -infinity times it), what goes to their exponents and to their sums.
          const float4 scale4 = *reinterpret_cast<const float4*>(sh.scale[slot][0] + 4 * half);
          const float4 lift4 = *reinterpret_cast<const float4*>(sh.scale[slot][1] + 4 * half);
          const float4 back4 = *reinterpret_cast<const float4*>(sh.scale[slot][2] + 4 * half);
          const uint2 valid2 = *reinterpret_cast<const uint2*>(sh.valid[slot] + 4 * half);
          constexpr float kLeast = 1.17549435e-38f;
          const float factor[4] = {fmaxf(scale4.x * rf, kLeast), fmaxf(scale4.y * rf, kLeast),
                                   fmaxf(scale4.z * rf, kLeast), fmaxf(scale4.w * rf, kLeast)};
          const float lift[4] = {lift4.x, lift4.y, lift4.z, lift4.w};
          const float back[4] = {back4.x, back4.y, back4.z, back4.w};
          uint32_t word[2] = {valid2.x, valid2.y};
          bool all = (valid2.x & valid2.y) == 0xFFFFFFFFu;
          if (t * kTreeKeys + (half + 1) * kHalfKeys > prefix) {
            all = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // Bits from d0 on: in front of 0 all, behind the row's words none.
              const int d0 = t * kTreeKeys + half * kHalfKeys + 32 * i - prefix, at = d0 >> 5;
              const uint32_t lo = at < 0 ? 0xFFFFFFFFu : at < kTreeWords ? sh.bits[g][at][r] : 0u;
              const uint32_t hi = at + 1 < 0 ? 0xFFFFFFFFu : at + 1 < kTreeWords ? sh.bits[g][at + 1][r] : 0u;
              word[i] &= __funnelshift_r(lo, hi, d0 & 31);
            }
          }
          if (warp_ok) {
            tmem_wait_ld();
            tmem_pin<64>(s);
            if (!all) {  // (the same for the whole warp)
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (!((word[i >> 5] >> (i & 31)) & 1u)) s[i] = 0xFF800000u;  // -infinity
            }
            // The running maximum takes in the half's largest y.
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t* v = s + 16 * i;
              float x = max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
              float y = max3(__uint_as_float(v[3]), __uint_as_float(v[4]), __uint_as_float(v[5]));
              x = max3(x, __uint_as_float(v[6]), __uint_as_float(v[7]));
              y = max3(y, __uint_as_float(v[8]), __uint_as_float(v[9]));
              x = max3(x, __uint_as_float(v[10]), __uint_as_float(v[11]));
              y = max3(y, __uint_as_float(v[12]), __uint_as_float(v[13]));
              x = max3(x, __uint_as_float(v[14]), __uint_as_float(v[15]));
              mx = fmaxf(mx, fmaf(fmaxf(x, y), factor[i], lift[i]));
            }
            mx -= kTreeShift;
            if (first) {
              mc = mx;
            } else {
              const bool grown = mx - mc > kTreeLag;  // (false for -inf - -inf = NaN)
              if (__any_sync(0xFFFFFFFFu, grown)) {
                float f = 1.f;
                if (grown) {
                  f = exp2_approx(mc - mx);  // (0 from -inf)
                  mc = mx;
                  l *= f;
                }
                // The product of the half before has to be done.
                ok = wait(&sh.o_done[g][half ^ 1], (tiles - (half ^ 1)) & 1u, kAttnSoftmaxTimeout);
                if (!ok) break;
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
            // P lies over the scores.
            const float base = mc == -INFINITY ? 0.f : mc;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t h[16];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const float f = factor[2 * c + q], e = lift[2 * c + q] - base;
                const uint64_t ff = pack2(f, f), ee = pack2(e, e);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int i = 8 * q; i < 8 * q + 8; ++i) {
                  float x, y;
                  unpack2(fma2(pack2(__uint_as_float(s[32 * c + 2 * i]), __uint_as_float(s[32 * c + 2 * i + 1])),
                               ff, ee),
                          x, y);
                  x = exp2_approx(x);
                  y = exp2_approx(y);
                  sum[i & 1] = add2(sum[i & 1], pack2(x, y));
                  h[i] = round2<__half>(x, y);
                }
                float x, y;
                unpack2(add2(sum[0], sum[1]), x, y);
                l = fmaf(x + y, back[2 * c + q], l);
              }
              tmem_st_x16(ts_half + c * 16, h);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[g][half]));
        }
        ++tiles;
      }
      seen += w.t1 - w.t0;
      if (ok && !first)  // the last tile's products, each half's
        ok = wait(&sh.o_done[g][0], (tiles - 1) & 1u, kAttnSoftmaxTimeout) &&
             wait(&sh.o_done[g][1], (tiles - 1) & 1u, kAttnSoftmaxTimeout);
      ok = barrier_all(bar_id, 128, ok);
      if (!ok) break;
      tc_fence_after();
      // Both groups' parts of a row: their weights, as the join has them.  (A part without keys is
      // left out, whatever its output holds; one whose maximum is -infinity all the same holds NaN of
      // the row's own.)
      float weight = 1.f, weight_other = 0.f;
      bool on = true, on_other = false;
      if (pair) {
        sh.stat[g][r] = make_float2(mc, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.meet));
        ok = wait(&sh.meet, 0u, kAttnSoftmaxTimeout);
        ok = barrier_all(bar_id, 128, ok);
        if (!ok) break;
        tc_fence_after();
        const float2 a = sh.stat[0][r], b = sh.stat[1][r];
        const float top = fmaxf(a.x, b.x);
        const bool on_a = a.x != -INFINITY || a.y != 0.f, on_b = b.x != -INFINITY || b.y != 0.f;
        const float fa = a.x == -INFINITY ? 0.f : exp2_approx(a.x - top);
        const float fb = b.x == -INFINITY ? 0.f : exp2_approx(b.x - top);
        mc = top;
        l = fmaf(fb, b.y, fa * a.y);
        weight = g ? fb : fa;
        weight_other = g ? fa : fb;
        on = g ? on_b : on_a;
        on_other = g ? on_a : on_b;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // A share: unnormalised, with its maximum and sum.  (Both groups' shares of one row tile
      // lie behind one another; one without a tile leaves no rows.)
      const long long at = (2ll * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * (2 * kRowsMany) + g * kRowsMany + r;
      if (warp_ok && (!first || whole)) {
        // Through the warp's part of the queries' place (whose products have ended), so that rows
        // leave side by side.  (A row a lane, 16 bytes at a time, took 9 us an item.)
        uint8_t* staged = smem + g * L::kTile + quarter * (L::kTile / 4);
        const int row_first = row - lane;
        if (whole) {
          constexpr int kChunks = DP / 8, kAtOnce = 32 / kChunks;  // 16-byte words of a row
#pragma unroll 1
          for (int c = pair ? 32 * g : 0; c < d; c += pair ? 64 : 32) {
            uint32_t o[32];
            tmem_ld_x32(to + c, o);
            tmem_wait_ld_x32(o);
            if (pair) {
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                uint32_t v[16];
                tmem_ld_x16(to_other + c + j, v);
                tmem_wait_ld_x16(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float mine = on ? weight * __uint_as_float(o[j + i]) : 0.f;
                  o[j + i] = __float_as_uint(on_other ? fmaf(weight_other, __uint_as_float(v[i]), mine) : mine);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t h[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                h[j] = round2<T>(__uint_as_float(o[8 * i + 2 * j]) * inv, __uint_as_float(o[8 * i + 2 * j + 1]) * inv);
              *reinterpret_cast<uint4*>(staged + lane * (DP * 2) + ((((c >> 3) + i) ^ (lane % kChunks)) << 4)) =
                  make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
          __syncwarp();
          const int col = lane % kChunks;
#pragma unroll 4
          for (int i = 0; i < 32; i += kAtOnce) {
            const int at = i + lane / kChunks, at_row = row_first + at;
            if (at_row < w.size.drafts * p.group && col * 8 < d && (!pair || ((col >> 2) & 1) == g)) {
              const int at_draft = fast_div(at_row, p.div_group);
              const int at_head = w.hk * p.group + at_row - at_draft * p.group;
              *reinterpret_cast<uint4*>(p.out + w.b * p.os[0] + at_draft * p.os[1] + at_head * p.os[2] + col * 8) =
                  *reinterpret_cast<const uint4*>(staged + at * (DP * 2) + ((col ^ (at % kChunks)) << 4));
            }
          }
        } else {
          float* part = p.part_out + (at - lane) * 128;
#pragma unroll 1
          for (int c = 0; c < d; c += 32) {  // 32 columns: eight words of a row
            uint32_t o[32];
            tmem_ld_x32(to + c, o);
            tmem_wait_ld_x32(o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(staged + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                  make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            __syncwarp();
            const int col = lane & 7;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const int from = i + (lane >> 3);
              if (row_first + from < w.size.drafts * p.group && c + col * 4 < d)
                *reinterpret_cast<uint4*>(part + from * 128 + c + col * 4) =
                    *reinterpret_cast<const uint4*>(staged + from * 128 + ((col ^ (from & 7)) << 4));
            }
            __syncwarp();
          }
        }
        __syncwarp();
      }
      if (row_ok) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_stat + at * 2) = make_float2(mc, l);
        else if (p.lse && (!pair || g == 0))
          p.lse[(static_cast<long long>(w.b) * p.heads + head) * p.q_len + draft] =
              l == 0.f ? -INFINITY : fmaf(mc, kLn2, logf(l));
      }
      tc_fence_before();
      if (pair) {  // (before the next item this group waits for the other's arrival here)
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.meet));
      }
    }
  } else {
    give_registers<64>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int DP>
cudaError_t many_launch(const TreeParams& p, int grid, cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  const cudaError_t err = raise_smem(tree_many_kernel<T, DP>, configured, many_smem<DP>());
  if (err != cudaSuccess) return err;
  return launch_pdl(tree_many_kernel<T, DP>, dim3(grid), dim3(kThreadsMany), many_smem<DP>(), stream, p);
}

}  // namespace

cudaError_t launch_tree_many(const TreeParams& p, int dtype, int grid, cudaStream_t stream) {
  if (dtype == CONV_DTYPE_BF16)
    return p.c.head_dim <= 64 ? many_launch<__nv_bfloat16, 64>(p, grid, stream)
                              : many_launch<__nv_bfloat16, 128>(p, grid, stream);
  return p.c.head_dim <= 64 ? many_launch<__half, 64>(p, grid, stream)
                            : many_launch<__half, 128>(p, grid, stream);
}

}  // namespace convgb300
