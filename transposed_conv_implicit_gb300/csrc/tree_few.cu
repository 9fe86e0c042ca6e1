// Attention of drafted tokens to the paged 8-bit cache, few rows to a key
// head: up to 32 rows (draft, query head) go through the keys together.
//
//   s = scale q K^T,  p = exp(s - max),  out = (p V) / sum p
//
// in one pass with the running maximum and sum of each row.  Bound by reading
// the cache: 4 operations for each row and byte of it.  So that nothing else
// takes longer, codes go straight from the copies' landing place into the
// operands of mma.sync products (a tcgen05 product of 128 rows would multiply
// mostly rows that are not there, and wants the widened operands in shared
// memory first), and no warp waits for another: each of a CTA's warps takes
// every fourth slice of 16 keys, with a maximum, sum and output of its own, and
// each lane copies with cp.async exactly the bytes it will read itself.
//
// The order of a product's inner dimension is free, and so is that of the
// output's columns, so a lane takes 16 bytes side by side of a key's row (as
// four inner steps' operands) and of a value's row (as a column of each of the
// 16 output tiles).
//
// Measured: one token of 64 requests x 32/8 heads x 128 against up to 4096 keys
// 94 us, its join with it (4.3 TB/s; 5.4 for each further key); 7 drafts of 32
// requests against up to 8192 keys 124 us.  (Turned over, with the rows along N,
// single tokens need half the products and 128 registers, and take 99.7 us: the
// copies alone take 89 to 95.)
//
// Numbers: e4m3 codes are exact in fp16, and stay unscaled.  A key's scale goes
// to its scores.  A value's scale 2^e goes to its probability: p 2^e is held as
// w = 2^(y - M), y = s log2(e) + e, with M the running maximum of y, which
// keeps w in fp16's range whatever the scales are; the sum of probabilities
// adds w 2^-e in fp32.  bf16 queries become fp16 after a power of two for each
// row, which the scores give back.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "tree_common.cuh"

namespace convgb300 {

namespace {

constexpr int kWarps = kTreeFewWarps, kThreads = 32 * kWarps;
constexpr int kSlice = 16;  // keys of a warp's step
static_assert(kTreeKeys % (kSlice * kWarps) == 0, "steps hold whole rounds of the warps");

template <int DP>
struct Few {
  static constexpr int kKeyWords = DP / 64;     // 16-byte words a lane takes of a key's row
  static constexpr int kValueBytes = DP / 8;    // bytes a lane takes of a value's row
  static constexpr int kTiles = DP / 8;         // output tiles of 8 columns
  static constexpr int kSteps = DP / 16;        // inner steps of the scores
  static constexpr int kStages = 4;
  static constexpr int kKeyBytes = 2 * kKeyWords * 512;
  static constexpr int kStageBytes = kKeyBytes + 4 * 32 * kValueBytes + 256;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kPitch = DP + 4;         // floats of a row where the warps meet
};

template <int DP>
constexpr size_t few_smem(int rows) {
  // The ring; where the warps meet lies over it.
  return std::max<size_t>(Few<DP>::kRing, static_cast<size_t>(kWarps) * rows * Few<DP>::kPitch * 4);
}

// Copies kBytes, of which `bytes` come from src and the rest is cleared.
template <int kBytes>
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, int bytes) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ uint4 read16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 read8(uint32_t src) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(src) : "memory");
  return v;
}

// d += a b: 16 rows, 8 columns, 16 inner elements of fp16.
__device__ __forceinline__ void product(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ void store4(uint16_t* dst, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(round2<T>(a, b), round2<T>(c, d));
}

// kGroups: groups of 16 rows.
template <typename T, int DP, int kGroups>
__global__ void __launch_bounds__(kThreads, kGroups == 1 ? 3 : 2)
    tree_few_kernel(const __grid_constant__ TreeParams p) {
  using L = Few<DP>;
  constexpr int kRows = 16 * kGroups;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ SplitStart shared_start;
  __shared__ int parents[kMaxDrafts];
  __shared__ uint32_t bits[kRows][kTreeWords];
  __shared__ float stat[kWarps][kRows][2];
  __shared__ float row_stat[kRows][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;  // a product's row (and row + 8), and columns 2 c4, 2 c4 + 1
  const uint32_t ring = smem_u32(smem) + warp * (L::kStages * L::kStageBytes);
  grid_dependency_wait();
  if (warp == 0) {
    const SplitStart st = split_start(p.batch, -1, lane, [&](int b) { return tree_steps(p, b); });
    if (lane == 0) shared_start = st;
  }
  __syncthreads();
  grid_launch_dependents();
  for (TreeWalk w(p, shared_start); w.live; w.next()) {
    const int prefix = w.size.keys - w.size.drafts;
    const int rows = min(kRows, w.size.drafts * p.group - w.row_tile * kRows);
    const int row0 = w.row_tile * kRows;
    // Slices of 16 keys, this warp's every fourth.
    const int end = min(w.t1 * (kTreeKeys / kSlice), (w.size.keys + kSlice - 1) / kSlice);
    int load_at = w.t0 * (kTreeKeys / kSlice) + warp;
    // The lane's part of a slice: rows g and g + 8 of the keys, 2 c4, 2 c4 + 1 and 8 further of the
    // values, the scales of the latter.
    const uint8_t* k_lane = p.c.k + w.hk * p.c.ks[2] + g * p.c.ks[1] + c4 * 16;
    const uint8_t* v_lane = p.c.v + w.hk * p.c.vs[2] + 2 * c4 * p.c.vs[1] + g * L::kValueBytes;
    const uint8_t* s_lane = p.c.scales + static_cast<long long>(w.hk) * p.c.page_size * 2 + 4 * c4;
    // Bytes that the lane copies of a row: none behind its end.
    const int k_bytes[2] = {c4 * 16 < p.c.head_dim ? 16 : 0, (c4 + 4) * 16 < p.c.head_dim ? 16 : 0};
    const int v_bytes = g * L::kValueBytes < p.c.head_dim ? L::kValueBytes : 0;
    // (The next slice's page is read a slice ahead, as the table has it, so that nothing waits for it.)
    const int* table = p.c.table + w.b * p.c.table_stride;
    auto page_at = [&](int slice) { return slice < end ? table[fast_div(slice, p.div_slices)] : -1; };
    int load_page = page_at(load_at);
    auto load = [&](int stage) {
      if (load_at < end) {
        const bool real = static_cast<unsigned int>(load_page) < static_cast<unsigned int>(p.c.pages);
        const int page = real ? load_page : 0;
        const int offset = (load_at - fast_div(load_at, p.div_slices) * static_cast<int>(p.div_slices.d)) * kSlice;
        const int keys = real ? w.size.keys - load_at * kSlice : 0;  // of the slice, that are there
        load_page = page_at(load_at + kWarps);
        const uint8_t* k = k_lane + (page * p.c.ks[0] + offset * p.c.ks[1]);
        const uint8_t* v = v_lane + (page * p.c.vs[0] + offset * p.c.vs[1]);
        const uint8_t* sc = s_lane + (page * p.scale_page + offset * 2);
        const uint32_t dst = ring + stage * L::kStageBytes + lane * 16;
        const uint32_t dst_v = ring + stage * L::kStageBytes + L::kKeyBytes + lane * L::kValueBytes;
        const uint32_t dst_s = ring + stage * L::kStageBytes + L::kKeyBytes + 4 * 32 * L::kValueBytes + lane * 8;
        auto copy = [&](auto whole) __attribute__((always_inline)) {
          constexpr bool kWhole = decltype(whole)::value;  // all 16 keys are there
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < L::kKeyWords; ++i)
              copy_bytes<16>(dst + (n * L::kKeyWords + i) * 512, k + (n ? p.ks8 : 0) + i * 64,
                             kWhole || 8 * n + g < keys ? k_bytes[i] : 0);
#pragma unroll
          for (int n = 0; n < 4; ++n)
            copy_bytes<L::kValueBytes>(dst_v + n * 32 * L::kValueBytes,
                                       v + ((n & 1) ? p.c.vs[1] : 0) + ((n >> 1) ? p.vs8 : 0),
                                       kWhole || 2 * c4 + (n & 1) + 8 * (n >> 1) < keys ? v_bytes : 0);
          // (Where a key is not there its byte arrives as 0, which says so.)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int there = keys - (2 * c4 + 8 * n);  // of two keys
            copy_bytes<4>(dst_s + n * 4, sc + 16 * n, kWhole || there >= 2 ? 4 : there == 1 ? 2 : 0);
          }
        };
        if (keys >= kSlice)
          copy(std::true_type());
        else
          copy(std::false_type());
      }
      load_at += kWarps;
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) load(i);

    // The rows' drafts, where this share comes to them.
    if (w.t1 * kTreeKeys > prefix) {
      const bool tree = p.parents != nullptr;
      if (tree)
        for (int i = threadIdx.x; i < w.size.drafts; i += kThreads)
          parents[i] = p.parents[w.b * p.parent_stride + i];
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < kRows) {
        uint32_t mine[kTreeWords];
        const int r = min(static_cast<int>(threadIdx.x), rows - 1);
        draft_bits(tree ? parents : nullptr, fast_div(row0 + r, p.div_group), mine);
#pragma unroll
        for (int i = 0; i < kTreeWords; ++i) bits[threadIdx.x][i] = mine[i];
      }
      __syncthreads();
    }

    // Queries: a lane's 16 elements of rows g and g + 8 are the operands of four inner steps.
    uint32_t qa[kGroups][L::kSteps][4];
    float factor[kGroups][2];  // of the rows' scores: scale, and the query's power of two
#pragma unroll
    for (int m = 0; m < kGroups; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = m * 16 + h * 8 + g;
        const int draft = fast_div(row0 + min(r, rows - 1), p.div_group);
        const int head = w.hk * p.group + row0 + min(r, rows - 1) - draft * p.group;
        const uint16_t* q = p.q + w.b * p.qs[0] + draft * p.qs[1] + head * p.qs[2];
        uint4 raw[L::kKeyWords][2];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < L::kKeyWords; ++i) {
          const int at = (c4 + 4 * i) * 16;
          const bool on = r < rows && at < p.c.head_dim;
          raw[i][0] = on ? *reinterpret_cast<const uint4*>(q + at) : make_uint4(0, 0, 0, 0);
          raw[i][1] = on ? *reinterpret_cast<const uint4*>(q + at + 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 u = raw[i][j >> 2];
            if constexpr (!std::is_same<T, __half>::value)
              top = fmaxf(top, larger_of((j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w));
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        float back;
        const float up = row_factor<T>(top, &back);
        factor[m][h] = p.scale_log2 * back;
#pragma unroll
        for (int i = 0; i < L::kKeyWords; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 u = raw[i][j >> 2];
            const uint32_t v = (j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w;
            // Elements 2 j, 2 j + 1: inner step 4 i + j / 2, its first or second pair.
            qa[m][4 * i + j / 2][h + 2 * (j & 1)] = std::is_same<T, __half>::value ? v : to_half(v, up);
          }
      }

    float o[kGroups][L::kTiles][4];
    float top[kGroups][2], sum[kGroups][2];  // top: the running maximum less kTreeShift
#pragma unroll
    for (int m = 0; m < kGroups; ++m) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[m][h] = -INFINITY;
        sum[m][h] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < L::kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
    }
    int stage = 0;
    for (int slice = w.t0 * (kTreeKeys / kSlice) + warp; slice < end; slice += kWarps) {
      copy_wait<L::kStages - 2>();
      const uint32_t src = ring + stage * L::kStageBytes;
      // Scores of the slice's keys 2 c4, 2 c4 + 1 (n = 0) and 8 further (n = 1).
      // (Two chains of products for each, which wait for one another's sums.)
      float s[kGroups][2][4], odd[kGroups][2][4];
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[m][n][i] = odd[m][n][i] = 0.f;
#pragma unroll
      for (int i = 0; i < L::kKeyWords; ++i) {
        uint32_t u[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint4 v = read16(src + (n * L::kKeyWords + i) * 512 + lane * 16);
          u[n][0] = v.x; u[n][1] = v.y; u[n][2] = v.z; u[n][3] = v.w;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            uint32_t b0, b1;
            widen_codes4(u[n][t], b0, b1);
#pragma unroll
            for (int m = 0; m < kGroups; ++m)
              product((t & 1) && kGroups == 1 ? odd[m][n] : s[m][n], qa[m][4 * i + t], b0, b1);
          }
      }
      if constexpr (kGroups == 1)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[0][n][i] += odd[0][n][i];
      const uint2 bytes = read8(src + L::kKeyBytes + 4 * 32 * L::kValueBytes + lane * 8);
      float key_scale[4], value_exp[4], value_back[4];
      uint32_t there = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t two = (j >> 1 ? bytes.y : bytes.x) >> (16 * (j & 1));
        const uint32_t kb = two & 0xFFu, vb = (two >> 8) & 0xFFu;
        key_scale[j] = __uint_as_float(kb << 23);
        value_exp[j] = __uint_as_float(0x4B000000u | vb) - 8388735.f;  // vb - 127
        value_back[j] = __uint_as_float((254u - vb) << 23);
        if (kb) there |= 1u << j;
      }
      const bool drafts = (slice + 1) * kSlice > prefix;
      if (drafts || __any_sync(0xFFFFFFFFu, there != 15u)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)  // (a value's byte of 255 would make the probability of 0 NaN)
          if (!((there >> j) & 1u)) value_back[j] = 0.f;
#pragma unroll
        for (int m = 0; m < kGroups; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = slice * kSlice + 2 * c4 + (j & 1) + 8 * (j >> 1) - prefix;  // a draft from 0 on
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              bool on = (there >> j) & 1u;
              if (on && d >= 0) on = (bits[m * 16 + h * 8 + g][d >> 5] >> (d & 31)) & 1u;
              float& x = s[m][j >> 1][2 * h + (j & 1)];
              x = on ? fmaf(x, key_scale[j] * factor[m][h], value_exp[j]) : -INFINITY;
            }
          }
      } else {
#pragma unroll
        for (int m = 0; m < kGroups; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = s[m][j >> 1][2 * h + (j & 1)];
              x = fmaf(x, key_scale[j] * factor[m][h], value_exp[j]);
            }
      }
      // Running maxima: a row's four lanes meet only where one has grown.
      bool grown = false;
      float most[kGroups][2];
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          most[m][h] = fmaxf(fmaxf(s[m][0][2 * h], s[m][0][2 * h + 1]), fmaxf(s[m][1][2 * h], s[m][1][2 * h + 1]));
          grown = grown || most[m][h] > top[m][h] + (kTreeShift + kTreeLag);
        }
      if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
        for (int m = 0; m < kGroups; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = most[m][h];
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2)) - kTreeShift;
            if (x > top[m][h]) {
              const float f = exp2_approx(top[m][h] - x);  // (0 at first)
              top[m][h] = x;
              sum[m][h] *= f;
#pragma unroll
              for (int n = 0; n < L::kTiles; ++n) {
                o[m][n][2 * h] *= f;
                o[m][n][2 * h + 1] *= f;
              }
            }
          }
      }
      uint32_t pa[kGroups][4];
#pragma unroll
      for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float base = top[m][h] == -INFINITY ? 0.f : top[m][h];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float x = exp2_approx(s[m][n][2 * h] - base), y = exp2_approx(s[m][n][2 * h + 1] - base);
            sum[m][h] = fmaf(x, value_back[2 * n], fmaf(y, value_back[2 * n + 1], sum[m][h]));
            pa[m][h + 2 * n] = round2<__half>(x, y);
          }
        }
      // The values: bytes of two keys side by side are the operands of two output tiles.
      uint32_t u[4][L::kValueBytes / 4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t at = src + L::kKeyBytes + (n * 32 + lane) * L::kValueBytes;
        if constexpr (L::kValueBytes == 16) {
          const uint4 v = read16(at);
          u[n][0] = v.x; u[n][1] = v.y; u[n][2] = v.z; u[n][3] = v.w;
        } else {
          const uint2 v = read8(at);
          u[n][0] = v.x; u[n][1] = v.y;
        }
      }
      if (__any_sync(0xFFFFFFFFu, there != 15u)) {  // (rows that were never written may hold NaN)
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (!((there >> n) & 1u))
#pragma unroll
            for (int i = 0; i < L::kValueBytes / 4; ++i) u[n][i] = 0;
      }
#pragma unroll
      for (int i = 0; i < L::kValueBytes / 4; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t pick = half ? 0x7362u : 0x5140u;
          uint32_t b[2][2];
          widen_codes4(__byte_perm(u[0][i], u[1][i], pick), b[0][0], b[1][0]);
          widen_codes4(__byte_perm(u[2][i], u[3][i], pick), b[0][1], b[1][1]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int m = 0; m < kGroups; ++m) product(o[m][4 * i + 2 * half + j], pa[m], b[j][0], b[j][1]);
        }
      // (All lanes have read the stage that the next copies go to, each its own bytes.)
      load(stage == 0 ? L::kStages - 1 : stage - 1);
      stage = stage == L::kStages - 1 ? 0 : stage + 1;
    }
    copy_wait<0>();

    // The warps meet: maxima first, then each one's rows relative to the largest.
#pragma unroll
    for (int m = 0; m < kGroups; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sum[m][h] += __shfl_xor_sync(0xFFFFFFFFu, sum[m][h], 1);
        sum[m][h] += __shfl_xor_sync(0xFFFFFFFFu, sum[m][h], 2);
        if (c4 == 0) {
          stat[warp][m * 16 + h * 8 + g][0] = top[m][h];
          stat[warp][m * 16 + h * 8 + g][1] = sum[m][h];
        }
      }
    __syncthreads();
    float* meet = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int m = 0; m < kGroups; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = m * 16 + h * 8 + g;
        float all = stat[0][r][0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) all = fmaxf(all, stat[i][r][0]);
        const float f = top[m][h] == -INFINITY ? 0.f : exp2_approx(top[m][h] - all);
        float* to = meet + (warp * kRows + r) * L::kPitch;
        // Column n of tile j is element n * kTiles + j: a lane's two columns are side by side.
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < L::kTiles; j += 4)
            *reinterpret_cast<float4*>(to + (2 * c4 + e) * L::kTiles + j) =
                make_float4(o[m][j][2 * h + e] * f, o[m][j + 1][2 * h + e] * f, o[m][j + 2][2 * h + e] * f,
                            o[m][j + 3][2 * h + e] * f);
        if (warp == 0 && c4 == 0) {
          float l = 0.f;
#pragma unroll
          for (int i = 0; i < kWarps; ++i)
            // (Without keys a warp's sum is 0, or NaN of the row's own.)
            l = fmaf(stat[i][r][1], stat[i][r][0] == -INFINITY ? 0.f : exp2_approx(stat[i][r][0] - all), l);
          row_stat[r][0] = all;
          row_stat[r][1] = l;
        }
      }
    __syncthreads();
    const bool whole = w.whole();
    const long long slot = 2ll * blockIdx.x + (w.t0 == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < rows * (DP / 4); i += kThreads) {
      const int r = i / (DP / 4), d = (i - r * (DP / 4)) * 4;
      if (d >= p.c.head_dim) continue;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(meet + (j * kRows + r) * L::kPitch + d);
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
      }
      const float m = row_stat[r][0], l = row_stat[r][1];
      if (!whole) {
        *reinterpret_cast<float4*>(p.part_out + (slot * kRows + r) * 128 + d) = a;
        if (d == 0) *reinterpret_cast<float2*>(p.part_stat + (slot * kRows + r) * 2) = make_float2(m, l);
        continue;
      }
      const int draft = fast_div(row0 + r, p.div_group);
      const int head = w.hk * p.group + row0 + r - draft * p.group;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      store4<T>(p.out + w.b * p.os[0] + draft * p.os[1] + head * p.os[2] + d, a.x * inv, a.y * inv, a.z * inv,
                a.w * inv);
      if (d == 0 && p.lse)
        p.lse[(static_cast<long long>(w.b) * p.heads + head) * p.q_len + draft] =
            l == 0.f ? -INFINITY : fmaf(m, kLn2, logf(l));
    }
    __syncthreads();  // (the ring takes the next item's copies)
  }
}

// Joins the shares of items that the launch cut, in order, with weights
// 2^(m_c - max m).  A warp takes kPer neighbouring rows of an item, whose lanes
// hold four columns; the shares' slots are listed once per block, before the
// launch that wrote them has ended, and a row's reads are in flight together.
// (Found share by share, with 64-bit divisions, the join of 5 requests x 29
// drafts took 45 us; that of 16 x 64 drafts takes 20 under the profiler.)
constexpr int kTreeJoinWarps = 8, kTreeJoinThreads = 32 * kTreeJoinWarps;
constexpr int kTreeMaxShares = 1024;  // of an item: two for each CTA at most
template <typename T, int kPer>
__global__ void __launch_bounds__(kTreeJoinThreads)
    tree_join_kernel(const __grid_constant__ TreeParams p, int ctas) {
  __shared__ long long sums[2][32];
  __shared__ int slots[kTreeMaxShares];  // rows of the workspace, or -1
  __shared__ int range[2];
  const int items = p.kv_heads * p.max_tiles;
  const int b = static_cast<int>(blockIdx.x / items), at = static_cast<int>(blockIdx.x - b * items);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (The launch before has waited for those in front of it before this one could start: the
  // lengths are there.)
  const TreeSize size = tree_size(p, b);
  const int row_tiles = tree_row_tiles(p, size), nt = tree_key_tiles(size);
  const int hk = row_tiles > 0 ? at / row_tiles : 0, row0 = (at - hk * row_tiles) * p.tile_rows;
  const int rows = min(p.tile_rows, size.drafts * p.group - row0);
  const int r0 = static_cast<int>(blockIdx.y * kTreeJoinWarps) * kPer;
  // Of an item of up to half a tile, many rows' CTAs leave two shares (their groups') where they
  // have a part of it.
  const int halves = p.many && rows <= p.tile_rows / 2 ? 2 : 1;
  int shares = 0;
  if (at < p.kv_heads * row_tiles && r0 < rows && nt > 1) {
    long long before, total;
    split_prefix(p.batch, -1, b, sums, [&](int i) { return tree_steps(p, i); }, &before, &total);
    if (threadIdx.x < 2) {
      const long long first = before + static_cast<long long>(at) * nt;
      range[threadIdx.x] = share_of(total, ctas, threadIdx.x ? first + nt - 1 : first);
    }
    __syncthreads();
    const int c0 = range[0];
    shares = range[1] == c0 ? 1 : (range[1] - c0 + 1) * halves;
    for (int i = threadIdx.x; i < shares; i += kTreeJoinThreads) {
      const int c = c0 + (halves == 2 ? i >> 1 : i);
      // (With fewer steps than CTAs some CTAs' shares are empty.)
      const bool none = total < ctas && share_begin(total, ctas, c) == share_begin(total, ctas, c + 1);
      slots[i] = none ? -1 : (2 * c + (c == c0 ? 1 : 0)) * p.tile_rows +
                                 (halves == 2 && (i & 1) ? p.tile_rows / 2 : 0);
    }
    __syncthreads();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (shares <= 1) return;  // nothing here, or written whole
  const int r = r0 + warp * kPer, d = lane * 4;
  if (r >= rows) return;
  const bool on = d < p.c.head_dim;
  // A few shares at a time, their statistics and rows in flight together, with the running maximum.
  // (Rows past the item's read its last one again and write nothing.)
  constexpr int kAtOnce = kPer == 1 ? 8 : 3;
  float m[kPer], l[kPer];
  float4 a[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    m[k] = -INFINITY;
    l[k] = 0.f;
    a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int c0 = 0; c0 < shares; c0 += kAtOnce) {
    float2 st[kAtOnce][kPer];
    float4 v[kAtOnce][kPer];
#pragma unroll
    for (int c = 0; c < kAtOnce; ++c) {
      const int slot = c0 + c < shares ? slots[c0 + c] : -1;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const long long row = max(slot, 0) + min(r + k, rows - 1);
        st[c][k] = make_float2(-INFINITY, 0.f);
        v[c][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (slot >= 0) {
          st[c][k] = *reinterpret_cast<const float2*>(p.part_stat + row * 2);
          if (on) v[c][k] = *reinterpret_cast<const float4*>(p.part_out + row * 128 + d);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      float top = m[k];
#pragma unroll
      for (int c = 0; c < kAtOnce; ++c) top = fmaxf(top, st[c][k].x);
      const float down = m[k] == -INFINITY ? 0.f : exp2_approx(m[k] - top);
      m[k] = top;
      l[k] *= down;
      a[k].x *= down;
      a[k].y *= down;
      a[k].z *= down;
      a[k].w *= down;
#pragma unroll
      for (int c = 0; c < kAtOnce; ++c) {
        // A share without keys leaves no rows, what lies there is not used; one whose maximum is
        // -infinity all the same holds NaN of the row's own.
        if (st[c][k].x == -INFINITY && st[c][k].y == 0.f) continue;
        const float f = st[c][k].x == -INFINITY ? 0.f : exp2_approx(st[c][k].x - top);
        l[k] = fmaf(f, st[c][k].y, l[k]);
        a[k].x = fmaf(f, v[c][k].x, a[k].x);
        a[k].y = fmaf(f, v[c][k].y, a[k].y);
        a[k].z = fmaf(f, v[c][k].z, a[k].z);
        a[k].w = fmaf(f, v[c][k].w, a[k].w);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (r + k >= rows) break;
    const int draft = fast_div(row0 + r + k, p.div_group);
    const int head = hk * p.group + row0 + r + k - draft * p.group;
    const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
    if (on)
      store4<T>(p.out + b * p.os[0] + draft * p.os[1] + head * p.os[2] + d, a[k].x * inv, a[k].y * inv,
                a[k].z * inv, a[k].w * inv);
    if (lane == 0 && p.lse)
      p.lse[(static_cast<long long>(b) * p.heads + head) * p.q_len + draft] =
          l[k] == 0.f ? -INFINITY : fmaf(m[k], kLn2, logf(l[k]));
  }
}

template <typename T, int DP, int kGroups>
cudaError_t few_launch(const TreeParams& p, int grid, cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  const size_t smem = few_smem<DP>(16 * kGroups);
  const cudaError_t err = raise_smem(tree_few_kernel<T, DP, kGroups>, configured, smem);
  if (err != cudaSuccess) return err;
  return launch_pdl(tree_few_kernel<T, DP, kGroups>, dim3(grid), dim3(kThreads), smem, stream, p);
}

template <typename T>
cudaError_t few_launch_type(const TreeParams& p, int grid, cudaStream_t stream) {
  if (p.c.head_dim <= 64)
    return p.tile_rows == 16 ? few_launch<T, 64, 1>(p, grid, stream) : few_launch<T, 64, 2>(p, grid, stream);
  return p.tile_rows == 16 ? few_launch<T, 128, 1>(p, grid, stream) : few_launch<T, 128, 2>(p, grid, stream);
}

}  // namespace

int tree_few_ctas(int tile_rows) { return tile_rows == 16 ? 3 : 2; }

cudaError_t launch_tree_few(const TreeParams& p, int dtype, int grid, cudaStream_t stream) {
  return dtype == CONV_DTYPE_BF16 ? few_launch_type<__nv_bfloat16>(p, grid, stream)
                                  : few_launch_type<__half>(p, grid, stream);
}

template <typename T, int kPer>
cudaError_t join_launch(const TreeParams& p, int ctas, cudaStream_t stream) {
  const int rows = std::min(p.tile_rows, p.q_len * p.group), of_block = kTreeJoinWarps * kPer;
  return launch_pdl(tree_join_kernel<T, kPer>,
                    dim3(static_cast<unsigned>(p.batch) * p.kv_heads * p.max_tiles, (rows + of_block - 1) / of_block),
                    dim3(kTreeJoinThreads), 0, stream, p, ctas);
}

cudaError_t launch_tree_join(const TreeParams& p, int dtype, int ctas, cudaStream_t stream) {
  // Four rows a warp where there are more rows than warps that run at once: attention of 128 items
  // of 256 rows takes 178 us with one, 168 with four; of 20 items of 87 rows (18 shares each) 25 and 32.
  const long long rows = static_cast<long long>(p.batch) * p.q_len * p.heads;
  const bool four = rows > 64ll * attn_sm_count();
  if (dtype == CONV_DTYPE_BF16)
    return four ? join_launch<__nv_bfloat16, 4>(p, ctas, stream) : join_launch<__nv_bfloat16, 1>(p, ctas, stream);
  return four ? join_launch<__half, 4>(p, ctas, stream) : join_launch<__half, 1>(p, ctas, stream);
}

}  // namespace convgb300
