// Layer norm, forward and backward, and its C entry points.
//
//   y = (x - m) r w + b,  m = mean x,  r = 1 / sqrt(mean (x - m)^2 + eps)
//   dx = r (g - mean g - h mean(g h)),  g = dy w,  h = (x - m) r
//   dw = sum_rows dy h,  db = sum_rows dy
//
// Deviations are taken from c, the first sum's mean rounded to the rows' type:
//   m = c + d,  d = mean (x - c),  mean (x - m)^2 = mean (x - c)^2 - d^2
// A row of one value has c equal to it, so its deviations are 0 whatever the sum's
// rounding (from the mean in fp32 they were the last bit of it, times r: y = 0.8
// for 60000 in 1000 channels).  The difference loses a bit at most: elements lie on
// the type's grid, so where d is some half of its step the deviations are that large
// too.
//
// Bound by memory: x in, y out; x and dy in, dx out.  Measured: 65536 x 320
// forward 18 us (4.7 TB/s; 6.7 for each further row), backward 24 us (5.3), 30 with
// the weights' sums; 16381 x 4096 forward 52 us (5.1 TB/s), backward 70 us (5.8),
// 82 with the weights' sums; with 321 and 4099 channels 32 and 114 us forward, 91
// and 266 for both passes.  A row lies in
// the registers of `lanes` lanes (a power of two up to a warp, or a whole block),
// up to kWords words of kVec elements each, so it is read once: the mean, the
// deviations from it and the result come from the same registers.  Lanes take
// words that are neighbours, and rows go around the groups of the grid.
//
// Rows come through a ring in shared memory, two ahead (each lane copies what it
// will read itself, so nothing waits but for its own copies).  Backward, a lane
// keeps the same columns in every row, so dw and db add up in
// its registers over all rows of its group; groups of a block meet in shared
// memory and blocks in the workspace, in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/conv_gb300_decoder.h"
#include "attn_internal.h"
#include "attn_ptx.cuh"
#include "conv_params.h"

namespace convgb300 {

namespace {

constexpr int kMaxChannels = 16384;
constexpr long long kMaxLnRows = 0x7F000000ll;  // (a step of the grid beyond still counts in 31 bits)
constexpr int kLnBwdBlocksPerSm = 4;  // rows of partial sums in the workspace
constexpr int kLnStages = 3;          // rows of a lane in the ring

struct LnParams {
  const void *x, *weight, *bias, *dy;
  void* y;  // y or dx
  float *mean, *rstd;
  float* partial;  // backward: [blocks][2][C]
  float *dweight, *dbias;
  int channels, words, lanes;  // words of kVec elements, lanes of a row
  int rows, blocks;
  bool weight_f32;  // of kShift alone: the others are built for a type
  float eps, inv_c;
  FastDiv div_length;
  long long xs[2], ds[2], ys[2];  // batch, token
};

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }

__device__ __forceinline__ float2 halves(uint32_t v, __nv_bfloat16) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float2 halves(uint32_t v, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
__device__ __forceinline__ uint32_t joined(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t joined(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A word of kVec elements as loaded: 16 bytes, or one element.
template <int kVec>
struct Word;
template <>
struct Word<8> {
  uint4 v;
};
template <>
struct Word<1> {
  uint16_t v;
};

template <int kVec>
__device__ __forceinline__ Word<kVec> load_word(const uint16_t* p) {
  Word<kVec> w;
  if constexpr (kVec == 8)
    w.v = *reinterpret_cast<const uint4*>(p);
  else
    w.v = *p;
  return w;
}
template <int kVec>
__device__ __forceinline__ Word<kVec> no_word() {
  Word<kVec> w;
  if constexpr (kVec == 8)
    w.v = make_uint4(0, 0, 0, 0);
  else
    w.v = 0;
  return w;
}
// Elements as fp32 pairs, so that arithmetic goes two at a time (a single
// element's pair has a 0).
template <int kVec>
struct Pairs {
  static constexpr int kCount = kVec == 8 ? 4 : 1;
  uint64_t v[kCount];
};
template <typename T, int kVec>
__device__ __forceinline__ Pairs<kVec> widen(const Word<kVec>& w) {
  Pairs<kVec> o;
  if constexpr (kVec == 8) {
    const uint32_t u[4] = {w.v.x, w.v.y, w.v.z, w.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = halves(u[i], T());
      o.v[i] = pack2(h.x, h.y);
    }
  } else {
    o.v[0] = pack2(to_float(*reinterpret_cast<const T*>(&w.v)), 0.f);
  }
  return o;
}
template <typename T, int kVec>
__device__ __forceinline__ void store_word(uint16_t* p, const Pairs<kVec>& o) {
  uint32_t u[Pairs<kVec>::kCount];
#pragma unroll
  for (int i = 0; i < Pairs<kVec>::kCount; ++i) {
    float a, b;
    unpack2(o.v[i], a, b);
    if constexpr (kVec == 8)
      u[i] = joined(a, b, T());
    else
      *reinterpret_cast<T*>(p) = from_float<T>(a);
  }
  if constexpr (kVec == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
// Elements [at, at + kVec) of weight or bias; `fill` without one.
template <typename W, int kVec>
__device__ __forceinline__ Pairs<kVec> load_weight(const void* w, int at, float fill) {
  Pairs<kVec> o;
  if (!w) {
#pragma unroll
    for (int i = 0; i < Pairs<kVec>::kCount; ++i) o.v[i] = pack2(fill, fill);
    return o;
  }
  if constexpr (kVec == 8 && sizeof(W) == 4) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    o.v[0] = pack2(a.x, a.y);
    o.v[1] = pack2(a.z, a.w);
    o.v[2] = pack2(b.x, b.y);
    o.v[3] = pack2(b.z, b.w);
  } else if constexpr (kVec == 8) {
    Word<8> v;
    v.v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + at));
    o = widen<W, 8>(v);
  } else {
    o.v[0] = pack2(to_float(static_cast<const W*>(w)[at]), 0.f);
  }
  return o;
}
__device__ __forceinline__ float both_of(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}

// Sums over the lanes of a row, given to all of them.  kBlock: the row is the
// whole block's; `turn` alternates between two sets of slots, so that one
// barrier a sum does.
template <bool kBlock, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int lanes, float (*slots)[2][32], int& turn) {
  for (int step = kBlock ? 16 : lanes >> 1; step > 0; step >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], step);
  if constexpr (kBlock) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) slots[turn][i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
      for (int w = 0; w < warps; ++w) v[i] += slots[turn][i][w];
    }
    turn ^= 1;
  }
}

// 1/sqrt(x): the hardware's approximation and one Newton step (which would make
// NaN of the infinity that belongs to 0).
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  return r < INFINITY ? r * fmaf(-0.5f * x * r, r, 1.5f) : r;
}

__device__ __forceinline__ long long row_at(const LnParams& p, int row, const long long s[2]) {
  const int b = fast_div(row, p.div_length);
  return b * s[0] + (row - b * static_cast<int>(p.div_length.d)) * s[1];
}

// 16 bytes, of which the first `bytes` are read and the others become zeros.
__device__ __forceinline__ void ring_copy(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint4 ring_word(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}

__device__ __forceinline__ void ring_put(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// kShift: rows that begin inside a 16-byte word, as those of an odd number of
// channels do.  A row that begins k elements into a word comes as the words that it
// touches; what a lane computes with is elements [8 w, 8 w + 8) all the same, put
// together from two words of the ring, its own and its neighbour's, so that a row's
// result does not depend on where the row lies.  The results go back through the
// ring in the same way, and to memory as whole words but for a row's two ends.
// (65536 x 321 forward 32 us at 61 % of the issue slots, element by element without
// a ring 86.)
__device__ __forceinline__ int place(const uint16_t* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 7;
}
// Elements [k, k + 8) of the words at `a` and `b`; zeros in place of a word that the
// ring does not have.
__device__ __forceinline__ uint4 shifted(uint32_t a, uint32_t b, bool has_b, int k) {
  const uint4 lo = ring_word(a);
  uint4 hi = make_uint4(0, 0, 0, 0);
  if (has_b) hi = ring_word(b);
  uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int j = 0; j < 6; ++j) u[j] = k & 4 ? u[j + 2] : u[j];
#pragma unroll
  for (int j = 0; j < 5; ++j) u[j] = k & 2 ? u[j + 1] : u[j];
  const int odd = k & 1 ? 16 : 0;
  return make_uint4(__funnelshift_r(u[0], u[1], odd), __funnelshift_r(u[1], u[2], odd),
                    __funnelshift_r(u[2], u[3], odd), __funnelshift_r(u[3], u[4], odd));
}
// Copies word w of a row of `channels` that begins at `row`, in a tensor that begins
// at `base` (nothing before it is read).
__device__ __forceinline__ void shift_copy(uint32_t dst, const uint16_t* row, const uint16_t* base, int w,
                                           bool first, int channels, bool live) {
  const int k = place(row), left = channels + k - 8 * w;
  if (first && live && row - base < k) {
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= k && j < left) u[j >> 1] |= static_cast<uint32_t>(row[j - k]) << (16 * (j & 1));
    ring_put(dst, make_uint4(u[0], u[1], u[2], u[3]));
    return;
  }
  const bool on = live && left > 0;
  const uintptr_t word = reinterpret_cast<uintptr_t>(row) & ~uintptr_t{15};  // (not read unless `on`)
  ring_copy(dst, reinterpret_cast<const void*>(word + (on ? 16 * w : 0)), on ? min(16, 2 * left) : 0);
}
// Stores word w of such a row.
__device__ __forceinline__ void shift_store(uint16_t* row, const uint4& v, int w, int k, int channels) {
  const int first = 8 * w - k;
  uint16_t* p = row + first;
  if (first >= 0 && first + 8 <= channels) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  if (first + 8 <= channels) {  // from element k on: one, two and four of them
    const int even = k + (k & 1);
    if (k & 1) p[k] = static_cast<uint16_t>((k & 4 ? k & 2 ? u[3] : u[2] : k & 2 ? u[1] : u[0]) >> 16);
    if (even & 2) *reinterpret_cast<uint32_t*>(p + even) = even & 4 ? u[3] : u[1];
    if (even <= 4) *reinterpret_cast<uint2*>(p + 4) = make_uint2(u[2], u[3]);
  } else if (first >= 0) {  // up to the row's end: four, two and one
    const int n = channels - first;
    if (n & 4) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    if (n & 2) *reinterpret_cast<uint32_t*>(p + (n & 4)) = n & 4 ? u[2] : u[0];
    if (n & 1) p[n - 1] = static_cast<uint16_t>(n & 4 ? n & 2 ? u[3] : u[2] : n & 2 ? u[1] : u[0]);
  } else {  // a row within one word
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (first + j >= 0 && first + j < channels) p[j] = static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1)));
  }
}
// An element of weight or bias, whose type is a choice of the run here: they are
// read once a block.
template <typename T>
__device__ __forceinline__ float weight_at(const LnParams& p, const void* w, int at, float none) {
  if (at >= p.channels) return 0.f;
  if (!w) return none;
  return p.weight_f32 ? static_cast<const float*>(w)[at] : to_float(static_cast<const T*>(w)[at]);
}
template <bool kBlock>
__device__ __forceinline__ void row_sync() {
  if constexpr (kBlock) __syncthreads();
  else __syncwarp();
}
template <typename T>
__device__ __forceinline__ uint4 joined8(const Pairs<8>& o) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    unpack2(o.v[j], a, b);
    u[j] = joined(a, b, T());
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Stores a row whose words lie at `held`.
template <int kWords>
__device__ __forceinline__ void store_shifted(uint16_t* row, uint32_t held, uint32_t pitch, int before, int at,
                                              int lanes, int channels) {
  const int k = place(row), words = channels > 0 ? (channels + k + 7) >> 3 : 0;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const int w = at + i * lanes;
    if (w >= words) break;
    // Elements [8 w - k, 8 w - k + 8): the last k of the word before, the first of this.
    // (In front of the first lie elements that are not stored.)
    const uint32_t own = held + i * pitch, left = i > 0 || at > 0 ? own + before : own;
    shift_store(row, k == 0 ? ring_word(own) : shifted(left, own, true, 8 - k), w, k, channels);
  }
}

// A row whose squares, or whose sum, pass fp32's range, as bfloat16's from some 2^60
// on do: from the elements times 2^-80, whose squares stay below 2^96, element by
// element from memory (such rows are few, and nothing is held for them).  All lanes
// of a warp, or a block, come here; rows of `past` are written.
template <typename T, bool kBlock>
__device__ __noinline__ void layer_norm_far_row(const LnParams& p, int row, bool live, bool past, int at, int lanes,
                                                float (*slots)[2][32], int turn) {
  constexpr float kDown = 0x1p-80f, kUp = 0x1p80f;
  const T* x = static_cast<const T*>(p.x) + (live ? row_at(p, row, p.xs) : 0);
  T* y = static_cast<T*>(p.y) + (live ? row_at(p, row, p.ys) : 0);
  const int end = live ? p.channels : 0;
  float first[1] = {0.f}, sum[2] = {0.f, 0.f};
  for (int e = at; e < end; e += lanes) first[0] += to_float(x[e]) * kDown;
  row_sum<kBlock, 1>(first, lanes, slots, turn);
  const float near = to_float(from_float<T>(first[0] * p.inv_c));
  for (int e = at; e < end; e += lanes) {
    const float d = to_float(x[e]) * kDown - near;
    sum[0] += d;
    sum[1] = fmaf(d, d, sum[1]);
  }
  row_sum<kBlock, 2>(sum, lanes, slots, turn);
  if (!past || !live) return;
  const float off = sum[0] * p.inv_c, difference = fmaf(-off, off, sum[1] * p.inv_c);
  const float var = difference < 0.f ? 0.f : difference, var_up = var * kUp * kUp;
  // (eps is nothing beside a variance that passes fp32, and all of it in a row of one value.)
  const float scale = var_up < INFINITY ? inverse_root(var_up + p.eps) * kUp : inverse_root(var);
  if (at == 0) {
    if (p.mean) p.mean[row] = (near + off) * kUp;
    if (p.rstd) p.rstd[row] = scale * kDown;
  }
  for (int e = at; e < end; e += lanes) {
    const float h = fmaf(to_float(x[e]) * kDown - near, scale, -off * scale);
    y[e] = from_float<T>(fmaf(h, weight_at<T>(p, p.weight, e, 1.f), weight_at<T>(p, p.bias, e, 0.f)));
  }
}

// kFull: a row's words are as many as its lanes take (320 channels on 8 lanes of 5).
template <typename T, typename W, int kVec, int kWords, bool kBlock, bool kFull, bool kShift>
__global__ void __launch_bounds__(kBlock ? (kVec == 8 ? 512 : 1024) : 256, kBlock ? 1 : 3)
    layer_norm_fwd_kernel(const __grid_constant__ LnParams p) {
  constexpr bool kRing = kVec == 8;
  __shared__ float slots[2][2][32];
  // [kLnStages][kWords][threads] words; kShift: then weight and bias in fp32, each
  // word's first half [words] and its second half [words] (from memory in every row:
  // 65536 x 321 in 41 us, so 33).
  extern __shared__ __align__(16) uint8_t shared[];
  const int lanes = kBlock ? static_cast<int>(blockDim.x) : p.lanes;
  const int at = kBlock ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (lanes - 1);
  const int groups = kBlock ? 1 : static_cast<int>(blockDim.x) / lanes;
  const int group = kBlock ? 0 : static_cast<int>(threadIdx.x) / lanes;
  int turn = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  const int step = gridDim.x * groups;
  const uint32_t ring = smem_u32(shared) + threadIdx.x * 16, pitch = blockDim.x * 16;
  auto copy = [&](int row0, int stage) {
    const int row = row0 + group;
    const bool live = row0 < p.rows && row < p.rows;
    const uint16_t* x = static_cast<const uint16_t*>(p.x) + (live ? row_at(p, row, p.xs) : 0);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int w = at + i * lanes;
      const uint32_t to = ring + (stage * kWords + i) * pitch;
      if constexpr (kShift) {
        shift_copy(to, x, static_cast<const uint16_t*>(p.x), w, i == 0 && at == 0, p.channels, live);
      } else {
        const bool on = live && (kFull || w < p.words);
        ring_copy(to, x + (on ? w * kVec : 0), on ? 16 : 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int stage = 0;
  if constexpr (kRing) {
    copy(blockIdx.x * groups, 0);
    copy(blockIdx.x * groups + step, 1);
  }
  const float4* affine = reinterpret_cast<const float4*>(shared + kLnStages * kWords * blockDim.x * 16);
  const int words = kShift ? (p.channels + 7) >> 3 : p.words;
  // The words before and after a lane's own, in the ring.
  const int before = at > 0 ? -16 : 16 * (lanes - 1) - static_cast<int>(pitch);
  const int after = at + 1 < lanes ? 16 : static_cast<int>(pitch) - 16 * at;
  if constexpr (kShift) {
    float* to = reinterpret_cast<float*>(shared + kLnStages * kWords * blockDim.x * 16);
    for (int e = threadIdx.x; e < 8 * words; e += blockDim.x) {
      float* t = to + (e & 4) * words + (e >> 3) * 4 + (e & 3);
      t[0] = weight_at<T>(p, p.weight, e, 1.f);
      t[8 * words] = weight_at<T>(p, p.bias, e, 0.f);
    }
    __syncthreads();
  }
  // (Every lane goes through every step: groups without a row left load nothing.)
  for (int row0 = blockIdx.x * groups; row0 < p.rows; row0 += step) {
    const int row = row0 + group;
    const bool live = row < p.rows;
    Word<kVec> raw[kWords];
    const uint32_t held = ring + stage * kWords * pitch;
    if constexpr (kRing) {
      if constexpr (kShift) {
        // The others' copies have come, and the last row's results have left the ring.
        asm volatile("cp.async.wait_group %0;" ::"n"(kLnStages - 2) : "memory");
        row_sync<kBlock>();
      }
      copy(row0 + 2 * step, stage == 0 ? 2 : stage - 1);
      if constexpr (!kShift) asm volatile("cp.async.wait_group %0;" ::"n"(kLnStages - 1) : "memory");
      if constexpr (kShift) {
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + (live ? row_at(p, row, p.xs) : 0);
        const int k = place(x);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const uint32_t own = held + i * pitch;
          raw[i].v = shifted(own, own + after, i + 1 < kWords || at + 1 < lanes, k);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) raw[i].v = ring_word(held + i * pitch);
      }
      stage = stage == kLnStages - 1 ? 0 : stage + 1;
    } else {
      const uint16_t* x = static_cast<const uint16_t*>(p.x) + (live ? row_at(p, row, p.xs) : 0);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int w = at + i * lanes;
        raw[i] = live && (kFull || w < p.words) ? load_word<kVec>(x + w * kVec) : no_word<kVec>();
      }
    }
    constexpr int kPairs = Pairs<kVec>::kCount;
    Pairs<kVec> f[kWords];
    uint64_t total = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      f[i] = widen<T, kVec>(raw[i]);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) total = add2(total, f[i].v[j]);
    }
    float first[1] = {both_of(total)};
    row_sum<kBlock, 1>(first, lanes, slots, turn);
    const float near = to_float(from_float<T>(first[0] * p.inv_c));
    const uint64_t minus = pack2(-near, kVec == 8 ? -near : 0.f);
    total = 0;
    uint64_t squares = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int w = at + i * lanes;
      if (kFull || w < words) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) f[i].v[j] = add2(f[i].v[j], minus);
        if constexpr (kShift)
          if (w == words - 1) {  // zeros behind the row
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
              float a, b;
              unpack2(f[i].v[j], a, b);
              f[i].v[j] = pack2(8 * w + 2 * j < p.channels ? a : 0.f, 8 * w + 2 * j + 1 < p.channels ? b : 0.f);
            }
          }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          total = add2(total, f[i].v[j]);
          squares = fma2(f[i].v[j], f[i].v[j], squares);
        }
      }
    }
    float sum[2] = {both_of(total), both_of(squares)};
    row_sum<kBlock, 2>(sum, lanes, slots, turn);
    const bool far = !std::is_same<T, __half>::value && !(sum[1] < INFINITY);  // (fp16's stay within fp32)
    const float off = sum[0] * p.inv_c, var = fmaf(-off, off, sum[1] * p.inv_c);
    const float rstd = inverse_root((var < 0.f ? 0.f : var) + p.eps);
    const bool here = live && !far;  // written here
    if (kShift || here) {
      if (here && at == 0) {
        if (p.mean) p.mean[row] = near + off;
        if (p.rstd) p.rstd[row] = rstd;
      }
      uint16_t* y = static_cast<uint16_t*>(p.y) + (live ? row_at(p, row, p.ys) : 0);
      const uint64_t rr = pack2(rstd, rstd), shift = pack2(-off * rstd, -off * rstd);
      if constexpr (kShift && !kBlock) __syncwarp();  // (all lanes have read the row; a block's, before its sums)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int w = at + i * lanes;
        if (!kFull && w >= words) break;
        Pairs<kVec> wt, bs;
        if constexpr (kShift) {
          const float4 a = affine[w], b = affine[words + w], c = affine[2 * words + w], d = affine[3 * words + w];
          wt.v[0] = pack2(a.x, a.y), wt.v[1] = pack2(a.z, a.w), wt.v[2] = pack2(b.x, b.y), wt.v[3] = pack2(b.z, b.w);
          bs.v[0] = pack2(c.x, c.y), bs.v[1] = pack2(c.z, c.w), bs.v[2] = pack2(d.x, d.y), bs.v[3] = pack2(d.z, d.w);
        } else {
          wt = load_weight<W, kVec>(p.weight, w * kVec, 1.f);
          bs = load_weight<W, kVec>(p.bias, w * kVec, 0.f);
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) f[i].v[j] = fma2(fma2(f[i].v[j], rr, shift), wt.v[j], bs.v[j]);
        if constexpr (kShift) ring_put(held + i * pitch, joined8<T>(f[i]));
        else store_word<T, kVec>(y + w * kVec, f[i]);
      }
      if constexpr (kShift) {
        row_sync<kBlock>();
        store_shifted<kWords>(y, held, pitch, before, at, lanes, here ? p.channels : 0);
      }
    }
    if constexpr (!std::is_same<T, __half>::value)
      if (kBlock ? far : __any_sync(0xFFFFFFFFu, far))
        layer_norm_far_row<T, kBlock>(p, row, live, far, at, lanes, slots, turn);
  }
}

// kWide: rows of blocks of more than 256 threads, which leave a lane no
// registers to keep its weights and the products of the first pass.  (With
// them kept, a row of 4096 takes 360 instructions of a warp, 880 without;
// twice the lanes with two words each: 188 us for both passes over 16381 rows,
// 153 with four.)
template <typename T, typename W, int kVec, int kWords, bool kBlock, bool kWide, bool kFull, bool kShift>
__global__ void __launch_bounds__(!kBlock ? 128 : kVec == 1 ? 1024 : kWide ? 512 : 256, !kShift ? 1 : kBlock ? 2 : 3)
    layer_norm_bwd_kernel(const __grid_constant__ LnParams p) {
  constexpr bool kRing = kVec == 8, kKeep = kVec == 8 && !kWide, kKeepRow = kKeep && !kShift;
  __shared__ float slots[2][2][32];
  // [kLnStages][2 * kWords][threads] words; then, where a block has several groups, [2][C].
  extern __shared__ __align__(16) uint8_t shared[];
  float* sums = reinterpret_cast<float*>(shared);
  const int lanes = kBlock ? static_cast<int>(blockDim.x) : p.lanes;
  const int at = kBlock ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (lanes - 1);
  const int groups = kBlock ? 1 : static_cast<int>(blockDim.x) / lanes;
  const int group = kBlock ? 0 : static_cast<int>(threadIdx.x) / lanes;
  int turn = 0;
  constexpr int kPairs = Pairs<kVec>::kCount;
  uint64_t dw[kWords * kPairs], db[kWords * kPairs];
#pragma unroll
  for (int i = 0; i < kWords * kPairs; ++i) dw[i] = db[i] = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  const int words = kShift ? (p.channels + 7) >> 3 : p.words;
  Pairs<kVec> weight[kKeep ? kWords : 1];
  if constexpr (kShift)
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const int e = 8 * (at + i * lanes) + 2 * j;
        weight[i].v[j] = pack2(weight_at<T>(p, p.weight, e, 1.f), weight_at<T>(p, p.weight, e + 1, 1.f));
      }
  else if constexpr (kKeep)
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      weight[i] = load_weight<W, kVec>(kFull || at + i * lanes < p.words ? p.weight : nullptr, (at + i * lanes) * kVec, 1.f);
  const int step = gridDim.x * groups;
  const uint32_t ring = smem_u32(shared) + threadIdx.x * 16, pitch = blockDim.x * 16;
  const int before = at > 0 ? -16 : 16 * (lanes - 1) - static_cast<int>(pitch);
  const int after = at + 1 < lanes ? 16 : static_cast<int>(pitch) - 16 * at;
  float stat[2] = {0.f, 0.f}, next_stat[2] = {0.f, 0.f};  // mean and rstd of the next rows, as they are copied
  auto copy = [&](int row0, int stage) {
    const int row = row0 + group;
    const bool live = row < p.rows && row0 < p.rows;
    const uint16_t* x = static_cast<const uint16_t*>(p.x) + (live ? row_at(p, row, p.xs) : 0);
    const uint16_t* dy = static_cast<const uint16_t*>(p.dy) + (live ? row_at(p, row, p.ds) : 0);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int w = at + i * lanes;
      const uint32_t to = ring + (stage * 2 * kWords + i) * pitch;
      if constexpr (kShift) {
        shift_copy(to, x, static_cast<const uint16_t*>(p.x), w, i == 0 && at == 0, p.channels, live);
        shift_copy(to + kWords * pitch, dy, static_cast<const uint16_t*>(p.dy), w, i == 0 && at == 0, p.channels, live);
      } else {
        const bool on = live && (kFull || w < p.words);
        ring_copy(to, x + (on ? w * kVec : 0), on ? 16 : 0);
        ring_copy(to + kWords * pitch, dy + (on ? w * kVec : 0), on ? 16 : 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int stage = 0;
  if constexpr (kRing) {
    copy(blockIdx.x * groups, 0);
    copy(blockIdx.x * groups + step, 1);
  }
  if (static_cast<int>(blockIdx.x) * groups + group < p.rows) {
    next_stat[0] = p.mean[blockIdx.x * groups + group];
    next_stat[1] = p.rstd[blockIdx.x * groups + group];
  }
  for (int row0 = blockIdx.x * groups; row0 < p.rows; row0 += step) {
    const int row = row0 + group;
    const bool live = row < p.rows;
    Word<kVec> rx[kWords], rd[kWords];
    stat[0] = next_stat[0];
    stat[1] = next_stat[1];
    if (row + step < p.rows) {
      next_stat[0] = p.mean[row + step];
      next_stat[1] = p.rstd[row + step];
    }
    const uint32_t held = ring + stage * 2 * kWords * pitch;
    if constexpr (kRing) {
      if constexpr (kShift) {
        // The others' copies have come, and the last row's results have left the ring.
        asm volatile("cp.async.wait_group %0;" ::"n"(kLnStages - 2) : "memory");
        row_sync<kBlock>();
      }
      copy(row0 + 2 * step, stage == 0 ? 2 : stage - 1);
      if constexpr (!kShift) asm volatile("cp.async.wait_group %0;" ::"n"(kLnStages - 1) : "memory");
      if constexpr (kShift) {
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + (live ? row_at(p, row, p.xs) : 0);
        const uint16_t* dy = static_cast<const uint16_t*>(p.dy) + (live ? row_at(p, row, p.ds) : 0);
        const int kx = place(x), kd = place(dy);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const bool next = i + 1 < kWords || at + 1 < lanes;
          const uint32_t own = held + i * pitch, own_d = own + kWords * pitch;
          rx[i].v = shifted(own, own + after, next, kx);
          rd[i].v = shifted(own_d, own_d + after, next, kd);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const uint32_t from = held + i * pitch;
          rx[i].v = ring_word(from);
          rd[i].v = ring_word(from + kWords * pitch);
        }
      }
      stage = stage == kLnStages - 1 ? 0 : stage + 1;
    } else {
      const uint16_t* x = static_cast<const uint16_t*>(p.x) + (live ? row_at(p, row, p.xs) : 0);
      const uint16_t* dy = static_cast<const uint16_t*>(p.dy) + (live ? row_at(p, row, p.ds) : 0);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int w = at + i * lanes;
        const bool on = live && (kFull || w < p.words);
        rx[i] = on ? load_word<kVec>(x + w * kVec) : no_word<kVec>();
        rd[i] = on ? load_word<kVec>(dy + w * kVec) : no_word<kVec>();
      }
    }
    const float mean = live ? stat[0] : 0.f, rstd = live ? stat[1] : 0.f;
    // (The mean goes off first: of x rstd - mean rstd little is left where a row is nearly of one value.)
    const uint64_t rr = pack2(rstd, rstd), minus = pack2(-mean, kVec == 8 ? -mean : 0.f);
    uint64_t sum_g = 0, sum_gh = 0;
    Pairs<kVec> hs[kKeepRow ? kWords : 1], fs[kKeepRow ? kWords : 1];  // h, and dy w
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int w = at + i * lanes;
      if (!kFull && w >= words) break;
      const Pairs<kVec> x = widen<T, kVec>(rx[i]), g = widen<T, kVec>(rd[i]);
      Pairs<kVec> wt;
      if constexpr (kKeep) wt = weight[i];
      else wt = load_weight<W, kVec>(p.weight, w * kVec, 1.f);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const uint64_t h = mul2(add2(x.v[j], minus), rr), f = mul2(g.v[j], wt.v[j]);
        // (Rows left out hold zeros of dy; so does a single element's other half.)
        dw[i * kPairs + j] = fma2(g.v[j], h, dw[i * kPairs + j]);
        db[i * kPairs + j] = add2(db[i * kPairs + j], g.v[j]);
        sum_g = add2(sum_g, f);
        sum_gh = fma2(f, h, sum_gh);
        if constexpr (kKeepRow) {
          hs[i].v[j] = h;
          fs[i].v[j] = f;
        }
      }
    }
    float sum[2] = {both_of(sum_g), both_of(sum_gh)};
    if (kShift && !(fabsf(mean * rstd) < INFINITY)) {  // the zeros behind a row, less its mean, are no numbers
      sum[1] = 0.f;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const Pairs<kVec> x = widen<T, kVec>(rx[i]), g = widen<T, kVec>(rd[i]);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const int e = 8 * (at + i * lanes) + 2 * j;
          float a, b, c, d;
          unpack2(mul2(add2(x.v[j], minus), rr), a, b);
          unpack2(mul2(g.v[j], weight[i].v[j]), c, d);
          sum[1] += (e < p.channels ? a * c : 0.f) + (e + 1 < p.channels ? b * d : 0.f);
        }
      }
    }
    row_sum<kBlock, 2>(sum, lanes, slots, turn);
    if (!kShift && !live) continue;
    const float c0 = -rstd * (sum[0] * p.inv_c), c1 = -rstd * (sum[1] * p.inv_c);
    const uint64_t cc0 = pack2(c0, c0), cc1 = pack2(c1, c1);
    uint16_t* dx = static_cast<uint16_t*>(p.y) + (live ? row_at(p, row, p.ys) : 0);
    if constexpr (kShift && !kBlock) __syncwarp();  // (all lanes have read the row; a block's, before its sums)
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int w = at + i * lanes;
      if (!kFull && w >= words) break;
      Pairs<kVec> o;
      if constexpr (kKeepRow) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) o.v[j] = fma2(fs[i].v[j], rr, fma2(hs[i].v[j], cc1, cc0));
      } else {
        const Pairs<kVec> x = widen<T, kVec>(rx[i]), g = widen<T, kVec>(rd[i]);
        Pairs<kVec> wt;
        if constexpr (kKeep) wt = weight[i];
        else wt = load_weight<W, kVec>(p.weight, w * kVec, 1.f);
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
          o.v[j] = fma2(mul2(g.v[j], wt.v[j]), rr, fma2(mul2(add2(x.v[j], minus), rr), cc1, cc0));
      }
      if constexpr (kShift) ring_put(held + i * pitch, joined8<T>(o));
      else store_word<T, kVec>(dx + w * kVec, o);
    }
    if constexpr (kShift) {
      row_sync<kBlock>();
      store_shifted<kWords>(dx, held, pitch, before, at, lanes, live ? p.channels : 0);
    }
  }
  if constexpr (kRing) asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!p.partial) return;
  __syncthreads();  // (the sums lie over the ring)
  float* out = p.partial + static_cast<long long>(blockIdx.x) * 2 * p.channels;
  // Element w * kVec + e of a lane's sums.
  auto put = [&](float* to, int w, const uint64_t* v, bool more) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      float a, b;
      unpack2(v[j], a, b);
      const int c = w * kVec + 2 * j;
      float* t = to + c;
      if (!kShift || c < p.channels) t[0] = more ? t[0] + a : a;
      if (kVec == 8 && (!kShift || c + 1 < p.channels)) t[1] = more ? t[1] + b : b;
    }
  };
  if constexpr (kBlock) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int w = at + i * lanes;
      if (!kFull && w >= words) break;
      put(out, w, dw + i * kPairs, false);
      put(out + p.channels, w, db + i * kPairs, false);
    }
  } else {
    // The groups of a warp, then the warps one after the other.
    for (int step_lanes = lanes; step_lanes < 32; step_lanes <<= 1)
#pragma unroll
      for (int i = 0; i < kWords * kPairs; ++i) {
        dw[i] = add2(dw[i], __shfl_xor_sync(0xFFFFFFFFu, dw[i], step_lanes));
        db[i] = add2(db[i], __shfl_xor_sync(0xFFFFFFFFu, db[i], step_lanes));
      }
    const int warps = static_cast<int>(blockDim.x) >> 5, warp = threadIdx.x >> 5;
    for (int next = 0; next < warps; ++next) {
      if (warp == next && (threadIdx.x & 31) < lanes)
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const int w = at + i * lanes;
          if (!kFull && w >= words) break;
          put(sums, w, dw + i * kPairs, next > 0);
          put(sums + p.channels, w, db + i * kPairs, next > 0);
        }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < 2 * p.channels; i += blockDim.x) out[i] = sums[i];
  }
}

// Sums the blocks' shares: a block takes 32 columns, its warps every 32nd share
// each, in order.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps)
    layer_norm_sum_kernel(const __grid_constant__ LnParams p) {
  __shared__ float part[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;  // of [2][C]
  grid_dependency_wait();
  grid_launch_dependents();
  float s = 0.f;
  if (col < 2 * p.channels) {
    const float* from = p.partial + col;
#pragma unroll 8
    for (int b = warp; b < p.blocks; b += kSumWarps) s += from[static_cast<long long>(b) * 2 * p.channels];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < 2 * p.channels) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) s += part[w][lane];
    if (col < p.channels) {
      if (p.dweight) p.dweight[col] = s;
    } else if (p.dbias) {
      p.dbias[col - p.channels] = s;
    }
  }
}

// How a row's words lie on lanes.
struct LnShape {
  int vec, words, lanes, per_lane, threads;
  bool block, shift;
};

// Words that a row touches at most, wherever in one it begins.
int ln_shift_words(int channels) { return (channels + 14) / 8; }

// How a row lies on lanes: as few idle words as possible, then few words a lane.
// Forward up to five a lane (320 channels on 8 lanes of 5: 19.8 us, on 16 of 3
// 24.1); backward four, with what it keeps of a row.  Longer rows take a block.
LnShape ln_shape(int channels, bool vectors, bool shift, bool backward) {
  LnShape s{};
  s.vec = vectors ? 8 : 1;
  s.shift = shift;
  s.words = shift ? ln_shift_words(channels) : channels / s.vec;
  const int most = backward ? 4 : 5;
  long long best = -1;
  for (int lanes = vectors ? 32 : 0; lanes >= 1; lanes >>= 1) {
    const int per = (s.words + lanes - 1) / lanes;
    if (per > most) continue;
    const long long idle = static_cast<long long>(lanes) * per - s.words;
    const long long cost = idle * 32 / lanes + (lanes > 8 ? 0 : 1);
    if (best < 0 || cost < best) {
      best = cost;
      s.lanes = lanes;
      s.per_lane = per;
    }
  }
  s.threads = backward ? 128 : 256;
  if (best >= 0) return s;
  s.block = true;
  // Three or four words a lane, whichever leaves fewer lanes idle.
  const auto warps = [&](int per) { return (s.words + 32 * per - 1) / (32 * per) * 32; };
  const int four = std::max(64, warps(4)), three = std::max(64, warps(3));
  s.threads = !vectors ? 1024 : three <= 256 && three * 3 < four * 4 ? three : four;
  s.lanes = s.threads;
  s.per_lane = (s.words + s.threads - 1) / s.threads;
  return s;
}

int ln_groups(const LnShape& s) { return s.block ? 1 : s.threads / s.lanes; }

template <typename T, typename W, int kVec, int kWords, bool kBlock, bool kWide, bool kFull, bool kShift>
cudaError_t ln_launch_bwd(LnParams p, const LnShape& s, long long need, int sms, cudaStream_t stream) {
  const auto kernel = layer_norm_bwd_kernel<T, W, kVec, kWords, kBlock, kWide, kFull, kShift>;
  const size_t ring = kVec == 8 ? static_cast<size_t>(kLnStages) * 2 * kWords * s.threads * 16 : 0;
  const size_t smem = std::max(ring, s.block ? size_t{0} : static_cast<size_t>(2) * p.channels * sizeof(float));
  static std::atomic<size_t> configured[kMaxDevices];
  cudaError_t err = raise_smem(kernel, configured, smem);
  if (err != cudaSuccess) return err;
  // As many blocks as run at once: each keeps its columns' sums over all of its rows.
  int fit = 0;
  static BlocksPerSm known[kMaxDevices][kWarpCounts];
  err = blocks_per_sm(kernel, known, s.threads, smem, &fit);
  if (err != cudaSuccess) return err;
  p.blocks = static_cast<int>(
      std::min<long long>(need, static_cast<long long>(std::min(fit, kLnBwdBlocksPerSm)) * sms));
  err = launch_pdl(kernel, dim3(p.blocks), dim3(s.threads), smem, stream, p);
  if (err != cudaSuccess || !p.partial) return err;
  return launch_pdl(layer_norm_sum_kernel, dim3((2 * p.channels + 31) / 32), dim3(32 * kSumWarps), 0,
                    stream, p);
}

// (A launcher's parameters are its kernel's, as what it remembers is of one kernel.)
template <typename T, typename W, int kVec, int kWords, bool kBlock, bool kFull, bool kShift>
cudaError_t ln_launch_fwd(const LnParams& p, const LnShape& s, long long need, int sms, cudaStream_t stream) {
  const auto kernel = layer_norm_fwd_kernel<T, W, kVec, kWords, kBlock, kFull, kShift>;
  size_t smem = kVec == 8 ? static_cast<size_t>(kLnStages) * kWords * s.threads * 16 : 0;
  if (kShift) smem += static_cast<size_t>(s.words) * 16 * sizeof(float);
  static std::atomic<size_t> configured[kMaxDevices];
  cudaError_t err = raise_smem(kernel, configured, smem);
  if (err != cudaSuccess) return err;
  int fit = 0;
  static BlocksPerSm known[kMaxDevices][kWarpCounts];
  err = blocks_per_sm(kernel, known, s.threads, smem, &fit);
  if (err != cudaSuccess) return err;
  const int grid = static_cast<int>(std::min<long long>(need, static_cast<long long>(fit) * sms));
  return launch_pdl(kernel, dim3(grid), dim3(s.threads), smem, stream, p);
}

template <typename T, typename W, int kVec, int kWords, bool kBlock, bool kWide, bool kFull, bool kShift>
cudaError_t ln_launch(const LnParams& p, const LnShape& s, bool backward, int sms, cudaStream_t stream) {
  const long long need = (static_cast<long long>(p.rows) + ln_groups(s) - 1) / ln_groups(s);
  if (!backward) return ln_launch_fwd<T, W, kVec, kWords, kBlock, kFull, kShift>(p, s, need, sms, stream);
  // (Five words a lane are for the forward pass alone: see ln_shape.)
  if constexpr (kVec == 8 && kWords == 5) return cudaErrorInvalidValue;
  else return ln_launch_bwd<T, W, kVec, kWords, kBlock, kWide, kFull, kShift>(p, s, need, sms, stream);
}
template <typename T, typename W>
cudaError_t ln_launch_shape(const LnParams& p, const LnShape& s, bool backward, int sms,
                            cudaStream_t stream) {
  const auto part = [&](auto vec, auto words) {  // rows on a warp's lanes
    constexpr int kVec = decltype(vec)::value, kWords = decltype(words)::value;
    if (s.shift) return ln_launch<T, T, kVec, kWords, false, false, false, true>(p, s, backward, sms, stream);
    if (s.lanes * kWords == s.words)
      return ln_launch<T, W, kVec, kWords, false, false, true, false>(p, s, backward, sms, stream);
    return ln_launch<T, W, kVec, kWords, false, false, false, false>(p, s, backward, sms, stream);
  };
  const auto whole = [&](auto vec, auto words, auto wide) {  // rows on a block
    constexpr int kVec = decltype(vec)::value, kWords = decltype(words)::value;
    constexpr bool kWide = decltype(wide)::value;
    if constexpr (kVec == 8 && !kWide)
      if (s.shift) return ln_launch<T, T, kVec, kWords, true, false, false, true>(p, s, backward, sms, stream);
    if constexpr (kVec == 8)
      if (s.lanes * kWords == s.words)
        return ln_launch<T, W, kVec, kWords, true, kWide, true, false>(p, s, backward, sms, stream);
    return ln_launch<T, W, kVec, kWords, true, kWide, false, false>(p, s, backward, sms, stream);
  };
  using N1 = std::integral_constant<int, 1>;
  using N2 = std::integral_constant<int, 2>;
  using N3 = std::integral_constant<int, 3>;
  using N4 = std::integral_constant<int, 4>;
  using N5 = std::integral_constant<int, 5>;
  using N8 = std::integral_constant<int, 8>;
  using N16 = std::integral_constant<int, 16>;
  const int n = s.per_lane;
  if (s.vec == 8) {
    if (s.block && s.threads > 256) return whole(N8(), N4(), std::true_type());
    if (s.block)
      return n <= 3 ? whole(N8(), N3(), std::false_type()) : whole(N8(), N4(), std::false_type());
    return n == 1 ? part(N8(), N1()) : n == 2 ? part(N8(), N2()) : n == 3 ? part(N8(), N3())
         : n == 4 ? part(N8(), N4()) : part(N8(), N5());
  }
  return n <= 8 ? whole(N1(), N8(), std::false_type()) : whole(N1(), N16(), std::false_type());
}

bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

conv_status_t ln_strides(const long long in[2], int batch, int length, bool output, long long out[2]) {
  const int extent[2] = {batch, length};
  for (int i = 0; i < 2; ++i) {
    out[i] = extent[i] > 1 ? in[i] : 0;
    if (extent[i] > 1 && (in[i] < 0 || (in[i] == 0 && output))) return CONV_ERR_INVALID_VALUE;
    if (out[i] >= 1ll << 40) return CONV_ERR_NOT_SUPPORTED;
  }
  return CONV_OK;
}

conv_status_t ln_check(const layer_norm_args_t& a, bool backward, LnParams* p) {
  if (a.dtype != CONV_DTYPE_BF16 && a.dtype != CONV_DTYPE_F16) return CONV_ERR_NOT_SUPPORTED;
  if (a.batch < 0 || a.length < 0 || a.channels <= 0) return CONV_ERR_INVALID_VALUE;
  if (a.channels > kMaxChannels || static_cast<long long>(a.batch) * a.length > kMaxLnRows)
    return CONV_ERR_NOT_SUPPORTED;
  if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return CONV_ERR_INVALID_VALUE;
  const bool rows = a.batch > 0 && a.length > 0;
  if (rows && (!a.x || (backward ? !a.dy || !a.dx || !a.mean || !a.rstd : !a.y)))
    return CONV_ERR_INVALID_VALUE;
  const uintptr_t weight_size = a.weight_f32 ? 4 : 2;
  if (off(a.x, 2) || off(a.weight, weight_size) || off(a.mean, 4) || off(a.rstd, 4))
    return CONV_ERR_MISALIGNED;
  if (backward ? off(a.dy, 2) || off(a.dx, 2) || off(a.dweight, 4) || off(a.dbias, 4)
               : off(a.y, 2) || off(a.bias, weight_size))
    return CONV_ERR_MISALIGNED;
  conv_status_t st = ln_strides(a.x_stride, a.batch, a.length, false, p->xs);
  if (st == CONV_OK && backward) st = ln_strides(a.dy_stride, a.batch, a.length, false, p->ds);
  if (st == CONV_OK)
    st = ln_strides(backward ? a.dx_stride : a.y_stride, a.batch, a.length, true, p->ys);
  return st;
}

conv_status_t ln_run(const layer_norm_args_t* args, bool backward, void* workspace,
                     size_t workspace_bytes, cudaStream_t stream) {
  if (!args) return CONV_ERR_INVALID_VALUE;
  const layer_norm_args_t& a = *args;
  LnParams p{};
  conv_status_t st = ln_check(a, backward, &p);
  if (st != CONV_OK) return st;
  const bool sums = backward && (a.dweight || a.dbias);
  if (backward) {
    if (!workspace) return CONV_ERR_INVALID_VALUE;
    if (off(workspace, 16)) return CONV_ERR_MISALIGNED;
    // (Partial sums are of dweight and dbias alone.)
    const size_t need = sums ? layer_norm_workspace_size(a.channels) : CONV_STATUS_BYTES;
    if (need == 0) return CONV_ERR_CUDA;
    if (workspace_bytes < need) return CONV_ERR_WORKSPACE_TOO_SMALL;
  }
  const int sms = attn_sm_count();
  if (sms <= 0) return CONV_ERR_CUDA;
  p.rows = a.batch * a.length;
  if (p.rows == 0 && !sums) return CONV_OK;
  p.x = a.x;
  p.weight = a.weight;
  p.bias = a.bias;
  p.dy = a.dy;
  p.y = backward ? a.dx : a.y;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.dweight = a.dweight;
  p.dbias = a.dbias;
  p.channels = a.channels;
  p.eps = a.eps;
  p.inv_c = 1.f / static_cast<float>(a.channels);
  p.div_length = make_fast_div(static_cast<uint32_t>(std::max(1, a.length)));
  bool vectors = a.channels % 8 == 0;
  const void* ptrs[] = {a.x, p.y, backward ? a.dy : nullptr};
  for (const void* q : ptrs) vectors = vectors && !off(q, 16);
  vectors = vectors && !off(a.weight, 16) && (backward || !off(a.bias, 16));
  for (int i = 0; i < 2; ++i)
    vectors = vectors && p.xs[i] % 8 == 0 && p.ys[i] % 8 == 0 && p.ds[i] % 8 == 0;
  // (Up to 1024 words, which a block of 256 threads takes.)
  const bool shift = !vectors && ln_shift_words(a.channels) <= 1024;
  p.weight_f32 = a.weight_f32 != 0;
  const LnShape s = ln_shape(a.channels, vectors || shift, shift, backward);
  p.words = s.words;
  p.lanes = s.lanes;
  if (backward) {
    if (sums) p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + CONV_STATUS_BYTES);
    if (p.rows == 0)  // sums over nothing
      return launch_pdl(layer_norm_sum_kernel, dim3((2 * p.channels + 31) / 32), dim3(32 * kSumWarps),
                        0, stream, p) == cudaSuccess
                 ? CONV_OK
                 : CONV_ERR_CUDA;
  }
  cudaError_t err;
  if (a.dtype == CONV_DTYPE_BF16)
    err = a.weight_f32 ? ln_launch_shape<__nv_bfloat16, float>(p, s, backward, sms, stream)
                       : ln_launch_shape<__nv_bfloat16, __nv_bfloat16>(p, s, backward, sms, stream);
  else
    err = a.weight_f32 ? ln_launch_shape<__half, float>(p, s, backward, sms, stream)
                       : ln_launch_shape<__half, __half>(p, s, backward, sms, stream);
  return err == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace

}  // namespace convgb300

extern "C" {

size_t layer_norm_workspace_size(int channels) {
  using namespace convgb300;
  if (channels <= 0 || channels > kMaxChannels) return 0;
  const int sms = attn_sm_count();
  if (sms <= 0) return 0;
  return CONV_STATUS_BYTES +
         static_cast<size_t>(kLnBwdBlocksPerSm) * sms * 2 * channels * sizeof(float);
}

conv_status_t layer_norm_fwd(const layer_norm_args_t* args, void* stream) {
  return convgb300::ln_run(args, false, nullptr, 0, static_cast<cudaStream_t>(stream));
}

conv_status_t layer_norm_bwd(const layer_norm_args_t* args, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return convgb300::ln_run(args, true, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
