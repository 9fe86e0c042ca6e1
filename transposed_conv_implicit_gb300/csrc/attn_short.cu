// Cross attention with at most 128 keys and heads of up to 64 elements (an
// image's pixels reading a caption): every row's keys are one tile, so nothing
// runs along the keys and the passes are bound by reading q (and do) and
// writing out (and dq).
//
// Forward: several small persistent CTAs per SM, each with one row tile of
// 128 (token, head) rows in flight, so that one CTA's loads, products,
// exponentials and stores run beside the others'.  The output leaves through
// the queries' shared-memory buffer; keys and values stay while consecutive
// tiles share them.
//
// 16 x 4096 x 8 heads x 40 against 77 keys: 32 us, 2.6 TB/s; the floor is 12.5
// us of memory traffic.  A row tile passes loads, scores, exponentials,
// products and stores one after another (5300 cycles, 37 % of the issue slots
// with four CTAs per SM, whose scores and outputs fill TMEM).
//
// Backward, one pass over q and do for all three gradients: a row's scores
// and dp = do v^T are whole in TMEM, so delta = sum_j p_j dp_j is summed right
// there (no read of out).  p and ds go to shared memory as the queries' rows;
// the same bytes are the A operand of dv += p^T do and dk += ds^T q (rows along
// M) and, in bf16, of dq = ds k (rows along K).  In fp16 dq's ds has the queries'
// own scales, which a sum over the queries cannot have: it lies in TMEM, over dp
// (the same call in fp16, with the norms' kernel and the join: 99 us, 95 with one
// scale for both).  dk and dv stay in TMEM over a CTA's share of a key head's
// query tiles and are joined through the workspace.
// The same call: 57 us and 10 for the join (the floor is 19): shared memory
// carries p and ds three times and the 128-row operands of five products, some
// 2000 cycles a step of 2700.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "attn_common.cuh"
#include "attn_internal.h"
#include "attn_params.h"

namespace convgb300 {

namespace {

constexpr uint32_t kTile = 128 * 128;  // 128 rows of 64 elements

// -infinity where the key takes no part.
__device__ __forceinline__ void mask_keys(uint32_t* s, int valid) {
  if (valid < 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= valid) s[i] = 0xFF800000u;
  }
}

// ------------------------------------------------------------------ forward
struct OneBars {
  uint64_t kv_full, kv_empty, q_full[2], q_empty[2], s_full, p_full, o_done, o_free, drain;
  uint32_t tmem;
  int abort_flag;
};

constexpr int kOneThreads = 192;  // 4 softmax warps, products, loads

// A CTA's items (row tiles), in order.
struct OneWalk {
  const AttnFwdParams& p;
  int item, end;
  int b, hk, row_tile;
  __device__ explicit OneWalk(const AttnFwdParams& params) : p(params) {
    item = static_cast<int>(share_begin(p.items, gridDim.x, blockIdx.x));
    end = static_cast<int>(share_begin(p.items, gridDim.x, blockIdx.x + 1));
    if (!live()) return;
    const int bh = fast_div(item, p.div_pairs);  // (of row tiles here)
    row_tile = item - bh * p.row_tiles;
    b = fast_div(bh, p.div_kv_heads);
    hk = bh - b * p.a.kv_heads;
  }
  __device__ bool live() const { return item < end; }
  // To the next item; true when it has other keys.
  __device__ bool next() {
    ++item;
    if (++row_tile < p.row_tiles) return false;
    row_tile = 0;
    if (++hk == p.a.kv_heads) {
      hk = 0;
      ++b;
    }
    return true;
  }
  __device__ void place(int* token, int* head) const {
    if (p.tile_heads > 1) {
      *token = row_tile * p.tile_tokens;
      *head = hk * p.a.group;
    } else {
      const int hg = fast_div(row_tile, p.div_token_tiles);
      *token = (row_tile - hg * p.token_tiles) * kAttnRows;
      *head = hk * p.a.group + hg;
    }
  }
  __device__ int keys() const { return min(valid_keys(p.a, b), p.kv_box); }
};

__device__ __forceinline__ int cols_of(int keys) { return max(16, (keys + 15) & ~15); }

// kCtas per SM: 4 where scores and output fit 128 TMEM columns, else 2.
template <typename T, int kCtas>
__global__ void __launch_bounds__(kOneThreads, kCtas)
    attn_one_kernel(const __grid_constant__ AttnFwdParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kCols = kCtas == 4 ? 128 : 256;
  extern __shared__ __align__(1024) uint8_t smem[];
  OneBars& bars = *reinterpret_cast<OneBars*>(smem + p.off_bar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars.abort_flag;
  unsigned int* status = p.status;
  const long long limit = p.timeout_cycles;
  const uint32_t kv_tile = static_cast<uint32_t>(p.kv_box) * 128u;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars.kv_full), 1);
    mbar_init(smem_u32(&bars.kv_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.q_full[i]), 1);
      mbar_init(smem_u32(&bars.q_empty[i]), 1);
    }
    mbar_init(smem_u32(&bars.s_full), 1);
    mbar_init(smem_u32(&bars.p_full), 4);
    mbar_init(smem_u32(&bars.o_done), 1);
    mbar_init(smem_u32(&bars.o_free), 4);
    mbar_init(smem_u32(&bars.drain), 1);
    bars.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(&bars.tmem), kCols);
    tmem_relinquish();
  }
  if (warp == 5 && lane == 0) {
    tma_prefetch_desc(&p.map_q);
    tma_prefetch_desc(&p.map_k);
    tma_prefetch_desc(&p.map_v);
    tma_prefetch_desc(&p.map_out);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t tmem = bars.tmem;
  const uint32_t t_out = tmem + (kCtas == 4 ? static_cast<uint32_t>(p.kv_box) : 128u);

  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned int code) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(bar), parity, abort_flag, status,
                                                     code, limit));
  };

  if (warp == 5) {
    // ------------------------------------------------------------ loads
    const uint32_t lead = lane == 0 ? 1u : 0u;
    const uint32_t q_bytes = static_cast<uint32_t>(p.tile_heads * p.tile_tokens) * 128u;
    bool ok = true, fresh = true;
    uint32_t count = 0, runs = 0;
    OneWalk w(p);
    for (; ok && w.live(); ++count) {
      if (fresh) {
        ok = wait(&bars.kv_empty, (runs & 1u) ^ 1u, kAttnProducerTimeout);
        if (!ok) break;
        // (fault_mode 1, a test hook: every CTA leaves its first keys un-armed.)
        if (!(p.fault_mode == 1 && runs == 0)) {
          const uint32_t bar = smem_u32(&bars.kv_full);
          mbar_arrive_expect_tx_if(lead, bar, 2 * kv_tile);
          tma_load_4d_if(lead, smem_u32(smem + p.off_kv), &p.map_k, bar, 0, w.hk * p.k_mul[0], 0,
                         w.b * p.k_mul[1]);
          tma_load_4d_if(lead, smem_u32(smem + p.off_kv) + kv_tile, &p.map_v, bar, 0,
                         w.hk * p.v_mul[0], 0, w.b * p.v_mul[1]);
        }
        ++runs;
      }
      const uint32_t s = count & 1u;
      ok = wait(&bars.q_empty[s], ((count >> 1) & 1u) ^ 1u, kAttnProducerTimeout);
      if (!ok) break;
      int token, head;
      w.place(&token, &head);
      mbar_arrive_expect_tx_if(lead, smem_u32(&bars.q_full[s]), q_bytes);
      tma_load_4d_if(lead, smem_u32(smem + p.off_q) + s * kTile, &p.map_q, smem_u32(&bars.q_full[s]),
                     0, head * p.q_mul[0], token, w.b * p.q_mul[1]);
      fresh = w.next();
    }
    if (!ok) {
      // Let every copy still in flight land before the CTA exits.
      if (runs > 0) mbar_wait_drain(smem_u32(&bars.kv_full), (runs - 1) & 1u, limit / 8 + 1);
      for (uint32_t i = count > 2 ? count - 2 : 0; i < count; ++i)
        mbar_wait_drain(smem_u32(&bars.q_full[i & 1u]), (i >> 1) & 1u, limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp == 4) {
    // ------------------------------------------------------------ products
    const int k_steps = (p.a.head_dim + 15) >> 4;
    const uint32_t idesc_o = attn_idesc(kBf16, static_cast<uint32_t>(k_steps) * 16u, false, true);
    const uint32_t q_lo = kLeadK | (smem_u32(smem + p.off_q) >> 4);
    const uint32_t k_lo = kLeadK | (smem_u32(smem + p.off_kv) >> 4);
    const uint32_t v_lo = lead_mn(kv_tile) | ((smem_u32(smem + p.off_kv) + kv_tile) >> 4);
    bool ok = true;
    uint32_t count = 0, runs = 0;
    int cols = 0;
    OneWalk w(p);
    // The keys of a run of items; values past the request's length are cleared.
    auto take_keys = [&]() {
      ok = wait(&bars.kv_full, runs & 1u, kAttnMmaTimeout);
      ++runs;
      const int keys = w.keys();
      cols = cols_of(keys);
      if (ok && keys < cols && p.a.kv_lengths) {
        const int r = keys + (lane >> 3);
        uint4* v = reinterpret_cast<uint4*>(smem + p.off_kv + kv_tile);
        for (int i = r; i < cols; i += 4) v[i * 8 + (lane & 7)] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_shared();
        __syncwarp();
      }
    };
    auto scores = [&]() {
      const uint32_t s = count & 1u;
      ok = ok && wait(&bars.q_full[s], (count >> 1) & 1u, kAttnMmaTimeout);
      if (!ok) return;
      tc_fence_after();
      mma_ss_x4(tmem, q_lo + s * (kTile >> 4), k_lo,
                attn_idesc(kBf16, static_cast<uint32_t>(cols), false, false), 0u, k_steps);
      mma_commit_warp(smem_u32(&bars.s_full));
    };
    bool live = w.live();
    if (live) {
      take_keys();
      scores();
    }
    while (ok && live) {
      const int steps = cols >> 4;
      const bool other = w.next();
      live = w.live();
      ok = wait(&bars.p_full, count & 1u, kAttnMmaTimeout);
      if (ok && count > 0) ok = wait(&bars.o_free, (count - 1) & 1u, kAttnMmaTimeout);
      if (!ok) break;
      tc_fence_after();
      mma_ts_x4(t_out, tmem, v_lo, idesc_o, 0u, steps);
      if (steps > 4) mma_ts_x4(t_out, tmem + 32, v_lo + 512u, idesc_o, 1u, steps - 4);
      mma_commit_warp(smem_u32(&bars.o_done));
      if (other) mma_commit_warp(smem_u32(&bars.kv_empty));
      ++count;
      if (live) {
        if (other) take_keys();
        scores();
      }
    }
    if (!ok) {
      mma_commit_warp(smem_u32(&bars.drain));
      mbar_wait_drain(smem_u32(&bars.drain), 0, limit / 8 + 1);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int r = warp * 32 + lane;
    const uint32_t lane_field = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t ts = tmem + lane_field, to = t_out + lane_field;
    const float c2 = p.scale_log2;
    const int row_token = p.tile_heads > 1 ? r / p.tile_heads : r;
    const int row_head = p.tile_heads > 1 ? r - row_token * p.tile_heads : 0;
    const bool leader = warp == 0 && lane == 0;
    bool ok = true, fresh = true;
    uint32_t count = 0;
    int keys = 0;
    OneWalk w(p);
    for (; w.live(); ++count) {
      if (fresh) keys = w.keys();
      int token0, head0;
      w.place(&token0, &head0);
      const int token = token0 + row_token;
      const bool row_ok = row_token < p.tile_tokens && token < p.a.q_len;
      const bool warp_ok = __any_sync(0xFFFFFFFFu, row_ok);
      const int b = w.b;
      fresh = w.next();
      ok = ok && wait(&bars.s_full, count & 1u, kAttnSoftmaxTimeout);
      float mc = 0.f, l = 0.f;
      if (ok) {
        tc_fence_after();
        if (leader && count > 0) {
          // The store before has been read: its buffer takes the next queries.
          bulk_wait_read_all();
          mbar_arrive(smem_u32(&bars.q_empty[(count - 1) & 1u]));
        }
        __syncwarp();
        if (warp_ok) {
          // Two passes over the scores, 32 at a time.  (P of a chunk lies over
          // scores read before it is stored.)
          const int chunks = (cols_of(keys) + 31) >> 5;
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            uint32_t s[32];
            tmem_ld_x32(ts + c * 32, s);
            tmem_wait_ld_x32(s);
            mask_keys(s, keys - c * 32);
            float top[4] = {mx, mx, mx, mx};
#pragma unroll
            for (int i = 0; i < 32; i += 8)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                top[j] = max3(top[j], __uint_as_float(s[i + j]), __uint_as_float(s[i + 4 + j]));
            mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
          }
          mc = mx == -INFINITY ? 0.f : fmaf(mx, c2, -kShift<T>);
          const uint64_t c22 = pack2(c2, c2), mc2 = pack2(-mc, -mc);
          uint64_t sum[2] = {0, 0};
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            uint32_t s[32], h[16];
            tmem_ld_x32(ts + c * 32, s);
            tmem_wait_ld_x32(s);
            mask_keys(s, keys - c * 32);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x, y;
              unpack2(fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c22, mc2), x,
                      y);
              x = exp2_approx(x);
              y = exp2_approx(y);
              sum[i & 1] = add2(sum[i & 1], pack2(x, y));
              h[i] = round2<T>(x, y);
            }
            tmem_st_x16(ts + c * 16, h);
          }
          float x, y;
          unpack2(add2(sum[0], sum[1]), x, y);
          l = x + y;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.p_full));
        ok = wait(&bars.o_done, count & 1u, kAttnSoftmaxTimeout);
      }
      uint8_t* stage = smem + p.off_q + (count & 1u) * kTile;
      if (ok) {
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (p.a.lse && row_ok)
          p.a.lse[(static_cast<long long>(b) * p.a.heads + head0 + row_head) * p.a.q_len + token] =
              l == 0.f ? -INFINITY : row_lse<T>(mc, l);
        if (warp_ok) {
#pragma unroll 1
          for (int c = 0; c < p.a.head_dim; c += 16) {  // (16 columns: no further than they are ours)
            uint32_t o[16];
            tmem_ld_x16(to + c, o);
            tmem_wait_ld_x16(o);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t h[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                h[j] = round2<T>(__uint_as_float(o[i * 8 + 2 * j]) * inv,
                                 __uint_as_float(o[i * 8 + 2 * j + 1]) * inv);
              // 16-byte words of a row sit at their index XOR the row's low bits.
              *reinterpret_cast<uint4*>(stage + r * 128 + ((((c >> 3) + i) ^ (r & 7)) << 4)) =
                  make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.o_free));
      }
      ok = barrier_all(1, 128, ok);
      if (!ok) break;
      if (leader) {
        tma_store_4d(&p.map_out, smem_u32(stage), 0, head0, token0, b);
        bulk_commit_group();
      }
    }
    // Shared memory stays until the last store has read it.
    if (leader) bulk_wait_read_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// ------------------------------------------------------------------ backward
// 8 warps for p and ds, 4 that write dq, 2 that issue products, loads.
constexpr int kShortSoftmax = 8, kShortEpi = 8, kShortScores = 12, kShortGrads = 13, kShortLoad = 14;
constexpr int kShortThreads = 32 * 15;
constexpr int kShortStages = 3;     // query tiles in flight

struct ShortBars {
  uint64_t kv_full, kv_empty;
  uint64_t qd_full[kShortStages], qd_empty[kShortStages];
  uint64_t s_full[2], buf_free[2], dq_full[2];  // by TMEM buffer
  uint64_t pds_full, pds_empty, acc_done, acc_free, drain[2];
  float exchange[2][2][128];  // by step parity: a half row's share of delta
  uint32_t tmem;
  int abort_flag;
};

// A CTA's steps: query tiles of 128 tokens of one head, over the items (key
// heads) of all batches.
struct ShortWalk {
  const AttnBwdParams& p;
  long long left;
  int b, hk, i0, i1, head, qt;
  bool live;
  __device__ explicit ShortWalk(const AttnBwdParams& params) : p(params) {
    const long long total = static_cast<long long>(p.a.batch) * p.a.kv_heads * p.item_steps;
    const long long lo = share_begin(total, gridDim.x, blockIdx.x);
    left = share_begin(total, gridDim.x, blockIdx.x + 1) - lo;
    live = left > 0;
    if (!live) return;
    const long long item = lo / p.item_steps;
    b = static_cast<int>(item / p.a.kv_heads);
    hk = static_cast<int>(item - static_cast<long long>(b) * p.a.kv_heads);
    take(static_cast<int>(lo - item * p.item_steps));
  }
  __device__ void take(int from) {
    i0 = from;
    i1 = static_cast<int>(min(static_cast<long long>(p.item_steps), from + left));
    left -= i1 - i0;
    const int h = from / p.q_tiles;
    qt = from - h * p.q_tiles;
    head = hk * p.a.group + h;
  }
  __device__ void step() {
    if (++qt == p.q_tiles) {
      qt = 0;
      ++head;
    }
  }
  __device__ void next() {
    live = left > 0;
    if (!live) return;
    if (++hk == p.a.kv_heads) {
      hk = 0;
      ++b;
    }
    take(0);
  }
  // The present step's place in the statistics, in tiles.
  __device__ long long stats_at() const {
    return (static_cast<long long>(b) * p.a.heads + head) * p.q_tiles + qt;
  }
  __device__ int keys() const { return min(valid_keys(p.a, b), p.kv_box); }
  __device__ int rows16() const { return qt == p.q_tiles - 1 ? p.last_cols : kAttnRows; }
};

// fp16: a row's scale of ds is the share's times 2^down.  At most 2^24, the
// largest that a factor of fp16 takes back: rows still smaller beside the share's
// largest have less room above fp16's smallest numbers.
__device__ __forceinline__ int row_down(float norm, float values, float share) {
  const int own = __float_as_int(ds_scale(norm, values)) >> 23, all = __float_as_int(share) >> 23;
  return norm == 0.f ? 0 : min(24, own - all);
}
__device__ __forceinline__ float power(int e) { return __int_as_float((127 + e) << 23); }
__device__ __forceinline__ __half2 half_down(int e) {  // 2^-e, e in [0, 24]
  return __half2half2(__ushort_as_half(static_cast<unsigned short>(e <= 14 ? (15 - e) << 10 : 1 << (24 - e))));
}
__device__ __forceinline__ uint32_t times(uint32_t pair, __half2 f) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&pair), f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__global__ void __launch_bounds__(kShortThreads, 1)
    attn_short_bwd_kernel(const __grid_constant__ AttnBwdParams p) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) uint8_t smem[];
  ShortBars& bars = *reinterpret_cast<ShortBars*>(smem + p.off_bar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars.abort_flag;
  unsigned int* status = p.status;
  const long long limit = p.timeout_cycles;
  const uint32_t kv_tile = static_cast<uint32_t>(p.kv_box) * 128u;
  // Shared memory: q and do stages, p and ds (two blocks of 64 keys each), the
  // staging of dq, k and v.
  uint8_t* qd = smem + p.off_x;
  uint8_t* pds = smem + p.off_y;
  uint8_t* out = smem + p.off_stat;
  uint8_t* kv = smem + p.off_a;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars.kv_full), 1);
    mbar_init(smem_u32(&bars.kv_empty), 2);
    for (int i = 0; i < kShortStages; ++i) {
      mbar_init(smem_u32(&bars.qd_full[i]), 1);
      mbar_init(smem_u32(&bars.qd_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.s_full[i]), 1);
      mbar_init(smem_u32(&bars.buf_free[i]), 4);
      mbar_init(smem_u32(&bars.dq_full[i]), 1);
    }
    mbar_init(smem_u32(&bars.pds_full), kShortSoftmax);
    mbar_init(smem_u32(&bars.pds_empty), 1);
    mbar_init(smem_u32(&bars.acc_done), 1);
    mbar_init(smem_u32(&bars.acc_free), kShortSoftmax);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&bars.drain[i]), 1);
    bars.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kShortScores) {
    tmem_alloc(smem_u32(&bars.tmem), 512);
    tmem_relinquish();
  }
  if (warp == kShortLoad && lane == 0) {
    tma_prefetch_desc(&p.map_q);
    tma_prefetch_desc(&p.map_do);
    tma_prefetch_desc(&p.map_k);
    tma_prefetch_desc(&p.map_v);
    tma_prefetch_desc(&p.map_dq);
  }
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();  // (TMEM is held: what starts now cannot take it first)
  const uint32_t tmem = bars.tmem;
  // TMEM columns: dv, dk, then buffers of S (dq over it) and dp (in fp16 ds over it).
  const uint32_t t_dv = tmem, t_dk = tmem + 64, t_buf = tmem + 128;
  const uint32_t region = static_cast<uint32_t>(p.region), bufs = static_cast<uint32_t>(p.bufs);

  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned int code) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(bar), parity, abort_flag, status,
                                                     code, limit));
  };
  // Buffer and phase of step n.
  auto buf_of = [&](uint32_t n) { return bufs == 2 ? n & 1u : 0u; };
  auto phase_of = [&](uint32_t n) { return (bufs == 2 ? n >> 1 : n) & 1u; };

  if (warp == kShortLoad) {
    // ------------------------------------------------------------ loads
    const uint32_t lead = lane == 0 ? 1u : 0u;
    const uint32_t q_bytes = static_cast<uint32_t>(p.q_box) * 128u;
    bool ok = true;
    int s = 0;
    uint32_t sph = 0, items = 0;
    long long issued = 0;
    for (ShortWalk w(p); ok && w.live; w.next()) {
      ok = wait(&bars.kv_empty, (items & 1u) ^ 1u, kAttnProducerTimeout);
      if (!ok) break;
      // (fault_mode 1, a test hook: every CTA leaves its first keys un-armed.)
      if (!(p.fault_mode == 1 && items == 0)) {
        const uint32_t bar = smem_u32(&bars.kv_full);
        mbar_arrive_expect_tx_if(lead, bar, 2 * kv_tile);
        tma_load_4d_if(lead, smem_u32(kv), &p.map_k, bar, 0, w.hk * p.k_mul[0], 0, w.b * p.k_mul[1]);
        tma_load_4d_if(lead, smem_u32(kv) + kv_tile, &p.map_v, bar, 0, w.hk * p.v_mul[0], 0,
                       w.b * p.v_mul[1]);
      }
      ++items;
      for (int i = w.i0; i < w.i1; ++i, w.step()) {
        ok = wait(&bars.qd_empty[s], sph ^ 1u, kAttnProducerTimeout);
        if (!ok) break;
        const uint32_t bar = smem_u32(&bars.qd_full[s]);
        mbar_arrive_expect_tx_if(lead, bar, 2 * q_bytes);
        tma_load_4d_if(lead, smem_u32(qd) + s * 2 * kTile, &p.map_q, bar, 0, w.head * p.q_mul[0],
                       w.qt * kAttnRows, w.b * p.q_mul[1]);
        tma_load_4d_if(lead, smem_u32(qd) + s * 2 * kTile + kTile, &p.map_do, bar, 0,
                       w.head * p.do_mul[0], w.qt * kAttnRows, w.b * p.do_mul[1]);
        ++issued;
        if (++s == kShortStages) {
          s = 0;
          sph ^= 1u;
        }
      }
    }
    if (!ok) {
      if (items > 0) mbar_wait_drain(smem_u32(&bars.kv_full), (items - 1) & 1u, limit / 8 + 1);
      for (long long q = issued - kShortStages; q < issued; ++q)
        if (q >= 0)
          mbar_wait_drain(smem_u32(&bars.qd_full[q % kShortStages]),
                          static_cast<uint32_t>((q / kShortStages) & 1), limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp == kShortScores) {
    // ------------------------------------------------------------ S and dp
    const int k_steps = (p.a.head_dim + 15) >> 4;
    const uint32_t q_lo = kLeadK | (smem_u32(qd) >> 4), kv_lo = kLeadK | (smem_u32(kv) >> 4);
    bool ok = true;
    int s = 0;
    uint32_t sph = 0, count = 0, items = 0;
    for (ShortWalk w(p); ok && w.live; w.next()) {
      ok = wait(&bars.kv_full, items & 1u, kAttnMmaTimeout);
      if (!ok) break;
      ++items;
      const int keys = w.keys(), cols = cols_of(keys);
      if (keys < cols && p.a.kv_lengths) {
        // Keys past the request's length are cleared (k meets the zeros of ds;
        // v is only a factor of scores that are left out).
        uint4* k = reinterpret_cast<uint4*>(kv);
        for (int i = keys + (lane >> 3); i < cols; i += 4) k[i * 8 + (lane & 7)] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_shared();
        __syncwarp();
      }
      const uint32_t id = attn_idesc(kBf16, static_cast<uint32_t>(cols), false, false);
      for (int i = w.i0; i < w.i1; ++i, ++count) {
        ok = wait(&bars.qd_full[s], sph, kAttnMmaTimeout);
        // (The buffer's last dq has been read.)
        if (count >= bufs)
          ok = ok && wait(&bars.buf_free[buf_of(count)], phase_of(count) ^ 1u, kAttnMmaTimeout);
        if (!ok) break;
        tc_fence_after();
        const uint32_t t = t_buf + buf_of(count) * 2 * region, q = q_lo + s * (2 * kTile >> 4);
        mma_ss_x4(t, q, kv_lo, id, 0u, k_steps);
        mma_ss_x4(t + region, q + (kTile >> 4), kv_lo + (kv_tile >> 4), id, 0u, k_steps);
        mma_commit_warp(smem_u32(&bars.s_full[buf_of(count)]));
        if (++s == kShortStages) {
          s = 0;
          sph ^= 1u;
        }
      }
      if (ok) mma_commit_warp(smem_u32(&bars.kv_empty));
    }
    if (!ok) {
      // Every MMA already issued must finish before TMEM is released.
      mma_commit_warp(smem_u32(&bars.drain[0]));
      mbar_wait_drain(smem_u32(&bars.drain[0]), 0, limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp == kShortGrads) {
    // ------------------------------------------------------------ dq, dv, dk
    const int k_steps = (p.a.head_dim + 15) >> 4;
    const uint32_t n_out = static_cast<uint32_t>(k_steps) * 16u;
    const uint32_t idesc_acc = attn_idesc(kBf16, n_out, true, true);   // p^T do, ds^T q
    const uint32_t idesc_dq = attn_idesc(kBf16, n_out, false, true);   // ds k
    const uint32_t mn = lead_mn(kTile);
    const uint32_t q_lo = mn | (smem_u32(qd) >> 4), k_lo = lead_mn(kv_tile) | (smem_u32(kv) >> 4);
    const uint32_t p_lo = smem_u32(pds) >> 4, ds_lo = p_lo + (2 * kTile >> 4);
    bool ok = true;
    int s = 0;
    uint32_t count = 0, items = 0;
    for (ShortWalk w(p); ok && w.live; w.next()) {
      if (items > 0) ok = wait(&bars.acc_free, (items - 1) & 1u, kAttnMmaTimeout);
      ++items;
      const int steps = cols_of(w.keys()) >> 4;
      for (int i = w.i0; ok && i < w.i1; ++i, ++count, w.step()) {
        const uint32_t q = q_lo + s * (2 * kTile >> 4), go_on = i == w.i0 ? 0u : 1u;
        const uint32_t t_dq = t_buf + buf_of(count) * 2 * region;
        const int row_steps = w.rows16() >> 4;
        ok = wait(&bars.pds_full, count & 1u, kAttnMmaTimeout);
        if (!ok) break;
        tc_fence_after();
        // dq first: others wait for it.
        if (kBf16) {
          mma_x4<2, 128>(t_dq, kLeadK | ds_lo, k_lo, idesc_dq, 0u, steps);
          if (steps > 4)
            mma_x4<2, 128>(t_dq, kLeadK | (ds_lo + (kTile >> 4)), k_lo + 512u, idesc_dq, 1u, steps - 4);
        } else {  // (a chunk of 16 keys lies over its own dp)
          mma_ts_x4<32, 16>(t_dq, t_dq + region, k_lo, idesc_dq, 0u, steps);
          if (steps > 4)
            mma_ts_x4<32, 16>(t_dq, t_dq + region + 64, k_lo + 512u, idesc_dq, 1u, steps - 4);
        }
        mma_commit_warp(smem_u32(&bars.dq_full[buf_of(count)]));
        mma_x4<128, 128>(t_dv, mn | p_lo, q + (kTile >> 4), idesc_acc, go_on, row_steps);
        if (row_steps > 4)
          mma_x4<128, 128>(t_dv, mn | (p_lo + 512u), q + (kTile >> 4) + 512u, idesc_acc, 1u, row_steps - 4);
        mma_x4<128, 128>(t_dk, mn | ds_lo, q, idesc_acc, go_on, row_steps);
        if (row_steps > 4)
          mma_x4<128, 128>(t_dk, mn | (ds_lo + 512u), q + 512u, idesc_acc, 1u, row_steps - 4);
        mma_commit_warp(smem_u32(&bars.pds_empty));
        mma_commit_warp(smem_u32(&bars.qd_empty[s]));
        if (++s == kShortStages) s = 0;
      }
      if (ok) {
        mma_commit_warp(smem_u32(&bars.acc_done));
        mma_commit_warp(smem_u32(&bars.kv_empty));
      }
    }
    if (!ok) {
      mma_commit_warp(smem_u32(&bars.drain[1]));
      mbar_wait_drain(smem_u32(&bars.drain[1]), 0, limit / 8 + 1);
    }
    __syncwarp();
  } else if (warp >= kShortEpi && warp < kShortEpi + 4) {
    // ------------------------------------------------------------ dq out
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
    const bool leader = warp == kShortEpi && lane == 0;
    bool ok = true;
    uint32_t count = 0;
    for (ShortWalk w(p); ok && w.live; w.next()) {
      const float values = kBf16 ? 0.f : largest_value(p, w.b, w.hk, lane);
      const float scale_ds = kBf16 ? 1.f : ds_scale(largest_row(p, w.b, w.hk, w.i0, w.i1, lane), values);
      const float* st = p.stats + w.stats_at() * kStatPitch<T> + 256 + r;
      float norm = kBf16 ? 0.f : *st;
      for (int i = w.i0; i < w.i1; ++i, ++count, w.step()) {
        const float f = kBf16 ? p.a.scale : p.a.scale / (power(row_down(norm, values, scale_ds)) * scale_ds);
        st += kStatPitch<T>;
        if (!kBf16 && i + 1 < w.i1) norm = *st;  // (for the step after)
        ok = wait(&bars.dq_full[buf_of(count)], phase_of(count), kAttnSoftmaxTimeout);
        if (leader) bulk_wait_read_all();
        ok = barrier_all(5, 128, ok);  // (the staging buffer is free)
        if (!ok) break;
        tc_fence_after();
        const uint32_t t = t_buf + buf_of(count) * 2 * region + lane_field;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          if (c < p.a.head_dim) {
            uint32_t v[32];
            tmem_ld_x32(t + c, v);
            tmem_wait_ld_x32(v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                h[j] = round2<T>(__uint_as_float(v[k * 8 + 2 * j]) * f,
                                 __uint_as_float(v[k * 8 + 2 * j + 1]) * f);
              *reinterpret_cast<uint4*>(out + r * 128 + ((((c >> 3) + k) ^ (r & 7)) << 4)) =
                  make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
        tc_fence_before();
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.buf_free[buf_of(count)]));
        named_barrier(5, 128);
        if (leader) {
          tma_store_4d(&p.map_dq, smem_u32(out), 0, w.head, w.qt * kAttnRows, w.b);
          bulk_commit_group();
        }
      }
    }
    if (leader) bulk_wait_read_all();
    __syncwarp();
  } else {
    // ------------------------------------------------------------ p and ds
    // Two warps share a quarter of the rows: 16-key chunks [0, mid) and [mid, all).
    const int half = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
    const float c2 = p.scale_log2;
    const uint64_t c22 = pack2(c2, c2);
    const int d = p.a.head_dim;
    uint32_t count = 0, items = 0;
    bool ok = true;
    for (ShortWalk w(p); ok && w.live; w.next()) {
      const int keys = w.keys(), all = cols_of(keys) >> 4, mid = (all + 1) >> 1;
      const int c0 = half ? mid : 0, c1 = half ? all : mid;
      // ds's scales: of this share of the key head's queries, for dk, and of a row.
      float values = 0.f, scale_ds = 1.f;
      if (!kBf16) {
        values = largest_value(p, w.b, w.hk, lane);
        scale_ds = ds_scale(largest_row(p, w.b, w.hk, w.i0, w.i1, lane), values);
      }
      float lse = -INFINITY, norm = 0.f;
      const float* st = p.stats + w.stats_at() * kStatPitch<T> + r;
      auto load_row = [&]() {
        if constexpr (kBf16) {
          const int token = w.qt * kAttnRows + r;
          lse = token < p.a.q_len
                    ? p.a.lse[(static_cast<long long>(w.b) * p.a.heads + w.head) * p.a.q_len + token]
                    : -INFINITY;
        } else {  // (as the rows kernel left them: lse is l2 already)
          lse = st[0];
          norm = st[256];
          st += kStatPitch<T>;
        }
      };
      load_row();
      for (int i = w.i0; i < w.i1; ++i, ++count) {
        // Minus lse in log2 units; a row without keys or past the end: p = 0.
        const float l2 = !kBf16 || lse == -INFINITY ? lse : -lse * kLog2e;
        const int down = kBf16 ? 0 : row_down(norm, values, scale_ds);
        const float sc = power(down) * scale_ds * p.p_unscale;
        const uint64_t sc2 = pack2(sc, sc);
        const __half2 to_share = half_down(down);
        if (kBf16) w.step();
        if (i + 1 < w.i1) load_row();  // (for the step after)
        ok = ok && wait(&bars.s_full[buf_of(count)], phase_of(count), kAttnSoftmaxTimeout);
        const uint32_t ts = t_buf + buf_of(count) * 2 * region + lane_field;
        uint32_t s[64];
        const uint64_t l22 = pack2(l2, l2);
        uint64_t sum = 0;
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c0 + c < c1) tmem_ld_x16(ts + (c0 + c) * 16, s + c * 16);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c0 + c < c1) {
              uint32_t dp[16];
              tmem_ld_x16(ts + region + (c0 + c) * 16, dp);
              tmem_wait_ld_x16(s + c * 16);
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(s[c * 16 + j]), __uint_as_float(s[c * 16 + j + 1])), c22,
                             l22), x, y);
                x = exp2_approx(x);
                y = exp2_approx(y);
                s[c * 16 + j] = __float_as_uint(x);
                s[c * 16 + j + 1] = __float_as_uint(y);
              }
              tmem_wait_ld_x16(dp);
              const int valid = keys - (c0 + c) * 16;
              if (valid < 16) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (j >= valid) s[c * 16 + j] = dp[j] = 0u;
              }
#pragma unroll
              for (int j = 0; j < 16; j += 2)
                sum = fma2(pack2(__uint_as_float(s[c * 16 + j]), __uint_as_float(s[c * 16 + j + 1])),
                           pack2(__uint_as_float(dp[j]), __uint_as_float(dp[j + 1])), sum);
            }
          }
        }
        // delta over both halves of the row; then the products before have
        // read p and ds.
        float x, y;
        unpack2(sum, x, y);
        float* ex = &bars.exchange[count & 1u][0][0];
        ex[half * 128 + r] = x + y;
        ok = barrier_all(1 + quarter, 64, ok);
        if (!ok) break;
        const float delta = (ex[r] + ex[128 + r]) * p.p_unscale;
        const uint64_t dl = pack2(-delta, -delta);
        if (count > 0) ok = wait(&bars.pds_empty, (count - 1) & 1u, kAttnSoftmaxTimeout);
        // (A failure here is told to the other half at its next barrier.)
        if (ok) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c0 + c < c1) {
              // (dp is read again: held beside p, it would not fit the registers.)
              uint32_t dp[16], hp[8], hd[8], hr[8];  // (hr: ds by its row's scale)
              tmem_ld_x16(ts + region + (c0 + c) * 16, dp);
              tmem_wait_ld_x16(dp);
              const int valid = keys - (c0 + c) * 16;
              if (valid < 16) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (j >= valid) dp[j] = 0u;
              }
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint64_t pp = pack2(__uint_as_float(s[c * 16 + 2 * j]), __uint_as_float(s[c * 16 + 2 * j + 1]));
                uint64_t u = add2(pack2(__uint_as_float(dp[2 * j]), __uint_as_float(dp[2 * j + 1])), dl);
                unpack2(mul2(kBf16 ? u : mul2(u, sc2), pp), x, y);
                hd[j] = round2<T>(x, y);
                if (!kBf16) {
                  hr[j] = hd[j];
                  hd[j] = times(hd[j], to_share);
                }
                unpack2(pp, x, y);
                hp[j] = round2<T>(x, y);
              }
              // Two 16-byte words of the row's block of 64 keys, swizzled.
              const int chunk = c0 + c, word = (chunk & 3) * 2;
              if (!kBf16) tmem_st_x8(ts + region + chunk * 16, hr);
              uint8_t* row = pds + (chunk >> 2) * kTile + r * 128;
              const int w0 = (word ^ (r & 7)) << 4, w1 = ((word + 1) ^ (r & 7)) << 4;
              *reinterpret_cast<uint4*>(row + w0) = make_uint4(hp[0], hp[1], hp[2], hp[3]);
              *reinterpret_cast<uint4*>(row + w1) = make_uint4(hp[4], hp[5], hp[6], hp[7]);
              row += 2 * kTile;
              *reinterpret_cast<uint4*>(row + w0) = make_uint4(hd[0], hd[1], hd[2], hd[3]);
              *reinterpret_cast<uint4*>(row + w1) = make_uint4(hd[4], hd[5], hd[6], hd[7]);
            }
          }
          if (!kBf16) tmem_wait_st();
          tc_fence_before();
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.pds_full));
        }
      }
      // Both halves leave the item together, ok or not: one that gave up alone would
      // be missed at the next item's barriers.
      ok = ok && wait(&bars.acc_done, items & 1u, kAttnSoftmaxTimeout);
      ok = barrier_all(1 + quarter, 64, ok);
      ++items;
      if (!ok) break;
      tc_fence_after();
      // Half 0 takes dv, half 1 dk.
      const bool whole = w.i0 == 0 && w.i1 == p.item_steps;
      const long long slot = 2ll * blockIdx.x + (w.i0 == 0 ? 1 : 0);
      const float f = half ? p.a.scale / scale_ds : p.p_unscale;
      T* dst = half ? static_cast<T*>(p.a.dk) + w.b * p.a.dks[0] + r * p.a.dks[1] + w.hk * p.a.dks[2]
                    : static_cast<T*>(p.a.dv) + w.b * p.a.dvs[0] + r * p.a.dvs[1] + w.hk * p.a.dvs[2];
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t v[32];
        tmem_ld_x32((half ? t_dk : t_dv) + c + lane_field, v);
        tmem_wait_ld_x32(v);
        if (r >= keys) {  // (their rows of p and ds were never written)
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        if (c < d && r < p.a.kv_len) {
          if (whole)
            store_cols(dst + c, v, d - c, f);
          else
            store_cols_f32(p.part_kv + ((slot * 2 + half) * kAttnRows + r) * 128 + c, v, d - c,
                           kBf16 ? 1.f : half ? 1.f / scale_ds : p.p_unscale);
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
  if (warp == kShortScores) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int kCtas>
cudaError_t launch_one_fwd(const AttnFwdParams& p, int grid, size_t smem, cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  const cudaError_t e = raise_smem(attn_one_kernel<T, kCtas>, configured, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_one_kernel<T, kCtas>, dim3(grid), dim3(kOneThreads), smem, stream, p);
}

template <typename T>
cudaError_t launch_short(const AttnBwdParams& p, int grid, size_t smem, cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  const cudaError_t e = raise_smem(attn_short_bwd_kernel<T>, configured, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_short_bwd_kernel<T>, dim3(grid), dim3(kShortThreads), smem, stream, p);
}

}  // namespace

size_t attn_one_bar_bytes() { return sizeof(OneBars); }
size_t attn_short_bar_bytes() { return sizeof(ShortBars); }
int attn_short_stages() { return kShortStages; }

cudaError_t launch_attn_one(const AttnFwdParams& p, int ctas, int grid, size_t smem,
                            cudaStream_t stream) {
  if (p.a.dtype == 0)
    return ctas == 4 ? launch_one_fwd<__nv_bfloat16, 4>(p, grid, smem, stream)
                     : launch_one_fwd<__nv_bfloat16, 2>(p, grid, smem, stream);
  return ctas == 4 ? launch_one_fwd<__half, 4>(p, grid, smem, stream)
                   : launch_one_fwd<__half, 2>(p, grid, smem, stream);
}

cudaError_t launch_attn_short_bwd(const AttnBwdParams& p, int grid, size_t smem,
                                  cudaStream_t stream) {
  return p.a.dtype == 0 ? launch_short<__nv_bfloat16>(p, grid, smem, stream)
                        : launch_short<__half>(p, grid, smem, stream);
}

}  // namespace convgb300
