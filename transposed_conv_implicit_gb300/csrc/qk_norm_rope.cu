// Norm of queries and keys for each head with the position rotation, forward
// and backward, and their C entry points.
//
// For a row x of one head: r = 1/sqrt(mean x^2 + eps), y = x r w, and the
// pairs (a, b) of y turn by the position's angle.  The rotation is
// orthogonal, so the backward pass turns dy back (g = R^T dy) and
//   dw = sum_rows g x r,   dx = r (g w - x r^2 mean(g w x)).
//
// Bound by memory: x in, y out (dx: x and dy in, dx out) and a few operations
// per element.  A row is D/8 lanes with one 16-byte word each, so every lane
// sees its row's sums after a few shuffles and its pair's other member in one
// more exchange, and nothing is read twice.  The warp packs 32 / (D/8) rows
// side by side (6 rows of 40 elements on 30 lanes), and each lane keeps
// kUnroll rows of one token in flight, which share one read of the angle
// tables when there are enough heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/conv_gb300_attention.h"
#include "attn_internal.h"
#include "conv_params.h"
#include "attn_ptx.cuh"

namespace convgb300 {

namespace {

constexpr int kThreadsQn = 256;
constexpr int kWarpsQn = kThreadsQn / 32;
// Rows in flight per lane: the backward pass holds two tensors and their
// product for each.
constexpr int kUnrollFwd = 4, kUnrollBwd = 2;
constexpr int kBlocksFwd = 3, kBlocksBwd = 3;  // thread blocks per SM (launch bounds)

struct QnTensor {
  const void* x;
  const void* weight;
  const int* positions;
  const void* dy;
  void* y;         // y or dx
  float* dweight;
  float* partial;  // backward: [blocks][D]
  int weight_f32;
  int length, heads;
  int blocks;      // thread blocks that share this tensor's rows
  int units_per_token;
  int rows;          // batch * length * heads
  int many, units;
  FastDiv div_upt, div_length, div_heads;
  long long position_stride;
  uint32_t xs[3], ds[3], ys[3];  // batch, token, head; in 8 elements
};

struct QnParams {
  QnTensor t[2];
  const float* cos;
  const float* sin;
  int head_dim, rot, lanes, slots;  // lanes per row, rows side by side in a warp
  int table_rows, adjacent;
  float eps, inv_d;
};

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 load(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t store(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 load(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t store(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// V elements of a row as loaded, and as fp32 pairs.
template <int V>
struct Raw {
  uint32_t w[V / 2];
};
template <int V>
struct Pairs {
  uint64_t v[V / 2];
};

template <int V>
__device__ __forceinline__ Raw<V> load_raw(const uint16_t* p) {
  Raw<V> r;
  if constexpr (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    r.w[0] = u.x; r.w[1] = u.y;
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ Pairs<V> widen(const Raw<V>& r) {
  Pairs<V> o;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float2 f = Pair<T>::load(r.w[i]);
    o.v[i] = pack2(f.x, f.y);
  }
  return o;
}

template <typename T, int V>
__device__ __forceinline__ void store_row(uint16_t* p, const Pairs<V>& v) {
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    float x, y;
    unpack2(v.v[i], x, y);
    w[i] = Pair<T>::store(x, y);
  }
  if constexpr (V == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// The pairs' other members: the lane's own words the other way round
// (adjacent), or those of lane `other`.  Every lane of the warp takes part.
template <typename T, int V, bool kAdjacent>
__device__ __forceinline__ Pairs<V> partners(const Raw<V>& r, const Pairs<V>& own, int other) {
  if constexpr (kAdjacent) {
    Pairs<V> q;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      float x, y;
      unpack2(own.v[i], x, y);
      q.v[i] = pack2(y, x);
    }
    return q;
  } else {
    Raw<V> q;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) q.w[i] = __shfl_sync(0xFFFFFFFFu, r.w[i], other);
    return widen<T, V>(q);
  }
}

// Sums over the `lanes` lanes of a row (lane `at` of it), given to all of
// them, for kUnroll rows at once.  Rows need not fill a power of two: lanes
// past the end add nothing.
template <int kUnroll>
__device__ __forceinline__ void row_sums(float (&v)[kUnroll], int lanes, int at, int first) {
  if ((lanes & (lanes - 1)) == 0) {
    for (int step = lanes >> 1; step > 0; step >>= 1)
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u] += __shfl_xor_sync(0xFFFFFFFFu, v[u], step);
    return;
  }
  int step = 16;
  while (step >= lanes) step >>= 1;
  for (; step > 0; step >>= 1) {
    const bool adds = at + step < lanes && at < step;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const float o = __shfl_down_sync(0xFFFFFFFFu, v[u], step);
      if (adds) v[u] += o;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) v[u] = __shfl_sync(0xFFFFFFFFu, v[u], first);
}

// 1/sqrt(x): the hardware's approximation and one Newton step.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  return r * fmaf(-0.5f * x * r, r, 1.5f);
}

// The lane's angles for a token: each of its elements x turns into
//   x * c - partner * s
// (the sine of a pair's second member is negated).  Lanes that are not
// rotated have c = 1, s = 0.
template <int V, bool kAdjacent>
__device__ __forceinline__ void load_angles(const QnParams& p, const QnTensor& t, int b, int l,
                                            int e0, bool rotated, Pairs<V>& c, Pairs<V>& s) {
  if (!rotated) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      c.v[i] = pack2(1.f, 1.f);
      s.v[i] = 0;
    }
    return;
  }
  int pos = t.positions ? t.positions[b * t.position_stride + l] : l;
  pos = max(0, min(pos, p.table_rows - 1));
  const int half = p.rot >> 1;
  const uint64_t row = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * static_cast<uint32_t>(half);
  if constexpr (kAdjacent) {
    const float4 fc = *reinterpret_cast<const float4*>(p.cos + row + (e0 >> 1));
    const float4 fs = *reinterpret_cast<const float4*>(p.sin + row + (e0 >> 1));
    const float cc[4] = {fc.x, fc.y, fc.z, fc.w}, ss[4] = {fs.x, fs.y, fs.z, fs.w};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      c.v[i] = pack2(cc[i & 3], cc[i & 3]);
      s.v[i] = pack2(ss[i & 3], -ss[i & 3]);
    }
  } else {
    const bool second = e0 >= half;
    const uint64_t at = row + (second ? e0 - half : e0);
    const float sign = second ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 fc = *reinterpret_cast<const float4*>(p.cos + at + i);
      const float4 fs = *reinterpret_cast<const float4*>(p.sin + at + i);
      c.v[i / 2] = pack2(fc.x, fc.y);
      c.v[i / 2 + 1] = pack2(fc.z, fc.w);
      s.v[i / 2] = pack2(fs.x * sign, fs.y * sign);
      s.v[i / 2 + 1] = pack2(fs.z * sign, fs.w * sign);
    }
  }
}

__device__ __forceinline__ uint64_t offset8(uint32_t i, uint32_t stride8) {
  return static_cast<uint64_t>(i) * stride8;
}

// kMany: a unit's rows are heads of one token, which share its angles.
// Otherwise they are consecutive (token, head) rows, each with its own.
template <typename T, int V, bool kAdjacent, bool kBackward, bool kMany>
__device__ __forceinline__ void norm_rows(const QnParams& p, const QnTensor& t, int block,
                                          const float (*weight)[256], float (*red)[256]) {
  constexpr int kUnroll = kBackward ? kUnrollBwd : kUnrollFwd;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = lane / p.lanes;
  const int at = lane - slot * p.lanes;
  const int first = slot * p.lanes;
  const bool live = slot < p.slots;
  const int e0 = at * V;
  const int half = p.rot >> 1;
  const bool rotated = live && e0 < p.rot;
  const int other = rotated && !kAdjacent ? first + (e0 >= half ? at - half / V : at + half / V) : lane;
  const uint16_t* px = static_cast<const uint16_t*>(t.x) + e0;
  const uint16_t* pg = static_cast<const uint16_t*>(t.dy) + e0;
  uint16_t* py = static_cast<uint16_t*>(t.y) + e0;
  const uint64_t* w0 = reinterpret_cast<const uint64_t*>(weight[0] + e0);
  const uint64_t* w1 = reinterpret_cast<const uint64_t*>(weight[1] + e0);
  Pairs<V> dw;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) dw.v[i] = 0;

  // The angles of a token; forward, with the weights in them.
  auto angles = [&](int b, int l, Pairs<V>& c, Pairs<V>& s) {
    load_angles<V, kAdjacent>(p, t, b, l, e0, rotated, c, s);
    if constexpr (!kBackward) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        c.v[i] = mul2(c.v[i], w0[i]);
        s.v[i] = mul2(s.v[i], w1[i]);
      }
    }
  };
  const uint64_t head_step = offset8(p.slots, t.ys[2]);  // to the next row's head (kMany)
  const int step = t.blocks * kWarpsQn;
  for (int unit = block * kWarpsQn + warp; unit < t.units; unit += step) {
    Raw<V> x[kUnroll], g[kUnroll];
    Pairs<V> c, s;
    int b[kUnroll], l[kUnroll];
    uint64_t oy[kMany ? 1 : kUnroll];
    bool ok[kUnroll];
    if constexpr (kMany) {
      const int token = fast_div(unit, t.div_upt);
      const int h0 = (unit - token * t.units_per_token) * p.slots * kUnroll + slot;
      b[0] = fast_div(token, t.div_length);
      l[0] = token - b[0] * t.length;
      uint64_t ox = offset8(b[0], t.xs[0]) + offset8(l[0], t.xs[1]) + offset8(h0, t.xs[2]);
      uint64_t og = offset8(b[0], t.ds[0]) + offset8(l[0], t.ds[1]) + offset8(h0, t.ds[2]);
      oy[0] = offset8(b[0], t.ys[0]) + offset8(l[0], t.ys[1]) + offset8(h0, t.ys[2]);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        ok[u] = live && h0 + u * p.slots < t.heads;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) x[u].w[i] = g[u].w[i] = 0u;
        if (ok[u]) {
          x[u] = load_raw<V>(px + ox * 8);
          if constexpr (kBackward) g[u] = load_raw<V>(pg + og * 8);
        }
        ox += offset8(p.slots, t.xs[2]);
        og += offset8(p.slots, t.ds[2]);
      }
      angles(b[0], l[0], c, s);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int row = (unit * kUnroll + u) * p.slots + slot;
        const int token = fast_div(row, t.div_heads);
        const int head = row - token * t.heads;
        b[u] = fast_div(token, t.div_length);
        l[u] = token - b[u] * t.length;
        ok[u] = live && row < t.rows;
        oy[u] = offset8(b[u], t.ys[0]) + offset8(l[u], t.ys[1]) + offset8(head, t.ys[2]);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) x[u].w[i] = g[u].w[i] = 0u;
        if (ok[u]) {
          x[u] = load_raw<V>(px + (offset8(b[u], t.xs[0]) + offset8(l[u], t.xs[1]) +
                                   offset8(head, t.xs[2])) * 8);
          if constexpr (kBackward)
            g[u] = load_raw<V>(pg + (offset8(b[u], t.ds[0]) + offset8(l[u], t.ds[1]) +
                                     offset8(head, t.ds[2])) * 8);
        } else {
          b[u] = l[u] = 0;
        }
      }
    }
    float r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const Pairs<V> v = widen<T, V>(x[u]);
      uint64_t sq = mul2(v.v[0], v.v[0]);
#pragma unroll
      for (int i = 1; i < V / 2; ++i) sq = fma2(v.v[i], v.v[i], sq);
      float lo, hi;
      unpack2(sq, lo, hi);
      r[u] = lo + hi;
    }
    row_sums(r, p.lanes, at, first);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u] = inverse_root(fmaf(r[u], p.inv_d, p.eps));
    if constexpr (!kBackward) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if constexpr (!kMany) angles(b[u], l[u], c, s);
        Pairs<V> v = widen<T, V>(x[u]);
        const Pairs<V> q = partners<T, V, kAdjacent>(x[u], v, other);
        const uint64_t rr = pack2(r[u], r[u]), mr = pack2(-r[u], -r[u]);
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
          v.v[i] = fma2(mul2(q.v[i], s.v[i]), mr, mul2(mul2(v.v[i], c.v[i]), rr));
        if (ok[u]) store_row<T, V>(py + (kMany ? oy[0] + u * head_step : oy[u]) * 8, v);
      }
    } else {
      float dot[kUnroll];
      Pairs<V> gw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if constexpr (!kMany) angles(b[u], l[u], c, s);
        const Pairs<V> own = widen<T, V>(g[u]);
        const Pairs<V> q = partners<T, V, kAdjacent>(g[u], own, other);
        const Pairs<V> v = widen<T, V>(x[u]);
        const uint64_t rr = pack2(r[u], r[u]);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const uint64_t back = fma2(q.v[i], s.v[i], mul2(own.v[i], c.v[i]));  // turned back
          const uint64_t xhat = mul2(v.v[i], rr);                             // the normed row
          dw.v[i] = fma2(back, xhat, dw.v[i]);  // (rows left out hold zeros)
          gw[u].v[i] = mul2(back, w0[i]);
          sum = fma2(gw[u].v[i], xhat, sum);
        }
        float lo, hi;
        unpack2(sum, lo, hi);
        dot[u] = lo + hi;
      }
      row_sums(dot, p.lanes, at, first);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        Pairs<V> v = widen<T, V>(x[u]);
        const float f = -dot[u] * p.inv_d * r[u];
        const uint64_t rr = pack2(r[u], r[u]), ff = pack2(f, f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v.v[i] = mul2(rr, fma2(v.v[i], ff, gw[u].v[i]));
        if (ok[u]) store_row<T, V>(py + (kMany ? oy[0] + u * head_step : oy[u]) * 8, v);
      }
    }
  }
  if constexpr (kBackward) {
    // The block's share of dw: slots of a warp, then warps, in order.
    for (int sl = 0; sl < p.slots; ++sl) {
      if (slot == sl) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          float x, y;
          unpack2(dw.v[i], x, y);
          red[warp][e0 + 2 * i] = x + (sl ? red[warp][e0 + 2 * i] : 0.f);
          red[warp][e0 + 2 * i + 1] = y + (sl ? red[warp][e0 + 2 * i + 1] : 0.f);
        }
      }
      __syncwarp();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.head_dim; d += kThreadsQn) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWarpsQn; ++i) sum += red[i][d];
      t.partial[static_cast<long long>(block) * p.head_dim + d] = sum;
    }
  }
}

template <typename T, int V, bool kAdjacent, bool kBackward>
__global__ void __launch_bounds__(kThreadsQn, kBackward ? kBlocksBwd : kBlocksFwd)
    qk_norm_rope_kernel(const __grid_constant__ QnParams p) {
  __shared__ __align__(16) float weight[2][256];
  __shared__ float red[kBackward ? kWarpsQn : 1][256];
  const bool is_k = blockIdx.x >= static_cast<unsigned>(p.t[0].blocks);
  const QnTensor& t = p.t[is_k ? 1 : 0];
  const int block = is_k ? blockIdx.x - p.t[0].blocks : blockIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  // The weights, and those of each element's partner.
  for (int e = threadIdx.x; e < 256; e += kThreadsQn) {
    int far = e;
    if (e < p.rot) far = kAdjacent ? e ^ 1 : e < (p.rot >> 1) ? e + (p.rot >> 1) : e - (p.rot >> 1);
    float w[2] = {0.f, 0.f};
    if (e < p.head_dim) {
      w[0] = t.weight_f32 ? static_cast<const float*>(t.weight)[e]
                          : Pair<T>::load(static_cast<const uint16_t*>(t.weight)[e]).x;
      w[1] = t.weight_f32 ? static_cast<const float*>(t.weight)[far]
                          : Pair<T>::load(static_cast<const uint16_t*>(t.weight)[far]).x;
    }
    weight[0][e] = w[0];
    weight[1][e] = w[1];
  }
  __syncthreads();
  if (t.many)
    norm_rows<T, V, kAdjacent, kBackward, true>(p, t, block, weight, red);
  else
    norm_rows<T, V, kAdjacent, kBackward, false>(p, t, block, weight, red);
}

// dw = the blocks' shares, summed in a fixed order: one thread block per
// tensor, kReduceRows interleaved runs of rows, then the runs.
constexpr int kReduceRows = 8;
__global__ void __launch_bounds__(1024) qk_norm_rope_dw_kernel(const __grid_constant__ QnParams p) {
  __shared__ float part[kReduceRows][256];
  grid_dependency_wait();
  const QnTensor& t = p.t[blockIdx.x];
  if (t.blocks == 0) {
    // A tensor without rows: the gradient of its weight is zero.
    if (t.dweight)
      for (int d = threadIdx.x; d < p.head_dim; d += blockDim.x) t.dweight[d] = 0.f;
    return;
  }
  const int run = threadIdx.x >> 7;
  for (int d = threadIdx.x & 127; d < p.head_dim; d += 128) {
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    int i = run;
    for (; i + 3 * kReduceRows < t.blocks; i += 4 * kReduceRows) {
      s0 += t.partial[static_cast<long long>(i) * p.head_dim + d];
      s1 += t.partial[static_cast<long long>(i + kReduceRows) * p.head_dim + d];
      s2 += t.partial[static_cast<long long>(i + 2 * kReduceRows) * p.head_dim + d];
      s3 += t.partial[static_cast<long long>(i + 3 * kReduceRows) * p.head_dim + d];
    }
    for (; i < t.blocks; i += kReduceRows)
      s0 += t.partial[static_cast<long long>(i) * p.head_dim + d];
    part[run][d] = (s0 + s1) + (s2 + s3);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.head_dim; d += blockDim.x) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kReduceRows; ++i) sum += part[i][d];
    t.dweight[d] = sum;
  }
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Fills one tensor's strides, with those of dimensions of extent 1 cleared.
conv_status_t take_strides(const long long in[3], int batch, int length, int heads, bool output,
                           uint32_t out[3]) {
  const int extent[3] = {batch, length, heads};
  for (int i = 0; i < 3; ++i) {
    out[i] = 0;
    if (extent[i] <= 1) continue;
    if (in[i] < 0 || (output && in[i] == 0)) return CONV_ERR_INVALID_VALUE;
    if (in[i] % 8 != 0) return CONV_ERR_MISALIGNED;
    if (in[i] / 8 > 0xFFFFFFFFll) return CONV_ERR_NOT_SUPPORTED;
    out[i] = static_cast<uint32_t>(in[i] / 8);
  }
  return CONV_OK;
}

conv_status_t take_tensor(const qk_norm_rope_args_t& a, const qk_norm_rope_tensor_t& in,
                          bool backward, QnTensor* t) {
  *t = QnTensor{};
  if (!in.x) {
    // Left out; a weight gradient asked for all the same is zero.
    if (backward) t->dweight = in.dweight;
    return CONV_OK;
  }
  if (in.length < 0 || in.heads <= 0) return CONV_ERR_INVALID_VALUE;
  if (!in.weight || (backward ? (!in.dy || !in.dx || !in.dweight) : !in.y))
    return CONV_ERR_INVALID_VALUE;
  const void* ptrs[] = {in.x, in.weight, backward ? in.dy : in.y, backward ? in.dx : in.y};
  for (const void* q : ptrs)
    if (misaligned(q)) return CONV_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(in.positions) & 3u) return CONV_ERR_MISALIGNED;
  if (backward && (reinterpret_cast<uintptr_t>(in.dweight) & 3u)) return CONV_ERR_MISALIGNED;
  conv_status_t st = take_strides(in.x_stride, a.batch, in.length, in.heads, false, t->xs);
  if (st == CONV_OK && backward)
    st = take_strides(in.dy_stride, a.batch, in.length, in.heads, false, t->ds);
  if (st == CONV_OK)
    st = take_strides(backward ? in.dx_stride : in.y_stride, a.batch, in.length, in.heads, true,
                      t->ys);
  if (st != CONV_OK) return st;
  t->x = in.x;
  t->weight = in.weight;
  t->weight_f32 = in.weight_f32;
  t->positions = in.positions;
  t->position_stride = a.batch > 1 ? in.position_stride : 0;
  t->dy = in.dy;
  t->y = backward ? in.dx : in.y;
  t->dweight = in.dweight;
  t->length = in.length;
  t->heads = in.heads;
  const long long tokens = static_cast<long long>(a.batch) * in.length;
  if (tokens * in.heads > 0x7FFF0000ll) return CONV_ERR_NOT_SUPPORTED;  // rows count in 31 bits
  t->rows = static_cast<int>(tokens * in.heads);
  return CONV_OK;
}

template <typename T, bool kBackward>
cudaError_t launch_qn(const QnParams& p, int v, int grid, cudaStream_t stream) {
  const dim3 g(grid), b(kThreadsQn);
  if (p.adjacent) return launch_pdl(qk_norm_rope_kernel<T, 8, true, kBackward>, g, b, 0, stream, p);
  if (v == 8) return launch_pdl(qk_norm_rope_kernel<T, 8, false, kBackward>, g, b, 0, stream, p);
  return launch_pdl(qk_norm_rope_kernel<T, 4, false, kBackward>, g, b, 0, stream, p);
}

template <bool kBackward>
cudaError_t launch_qn_dtype(int dtype, int v, const QnParams& p, int grid, cudaStream_t stream) {
  return dtype == CONV_DTYPE_BF16 ? launch_qn<__nv_bfloat16, kBackward>(p, v, grid, stream)
                                  : launch_qn<__half, kBackward>(p, v, grid, stream);
}

conv_status_t run_qk_norm_rope(const qk_norm_rope_args_t* args, bool backward, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
  if (!args) return CONV_ERR_INVALID_VALUE;
  const qk_norm_rope_args_t& a = *args;
  if (a.dtype != CONV_DTYPE_BF16 && a.dtype != CONV_DTYPE_F16) return CONV_ERR_NOT_SUPPORTED;
  if (a.batch < 0 || a.head_dim <= 0 || a.rot_dim < 0 || a.rot_dim > a.head_dim || !(a.eps >= 0.f) ||
      !std::isfinite(a.eps))
    return CONV_ERR_INVALID_VALUE;
  if (a.head_dim % 8 != 0 || a.head_dim > 256 || a.rot_dim % 8 != 0) return CONV_ERR_NOT_SUPPORTED;
  if (a.rot_dim > 0) {
    if (!a.cos || !a.sin || a.table_rows <= 0) return CONV_ERR_INVALID_VALUE;
    if (misaligned(a.cos) || misaligned(a.sin)) return CONV_ERR_MISALIGNED;
  }
  // Halves that split a 16-byte word (rot_dim an odd multiple of 8) take
  // 8-byte words, so that a pair's members sit in whole words of two lanes.
  const int v = !a.adjacent_pairs && a.rot_dim % 16 != 0 ? 4 : 8;
  if (a.head_dim / v > 32) return CONV_ERR_NOT_SUPPORTED;
  QnParams p{};
  conv_status_t st = take_tensor(a, a.q, backward, &p.t[0]);
  if (st == CONV_OK) st = take_tensor(a, a.k, backward, &p.t[1]);
  if (st != CONV_OK) return st;
  if (backward) {
    if (!workspace) return CONV_ERR_INVALID_VALUE;
    if (misaligned(workspace)) return CONV_ERR_MISALIGNED;
    if (workspace_bytes < qk_norm_rope_workspace_size(a.head_dim))
      return CONV_ERR_WORKSPACE_TOO_SMALL;
  }
  const int sms = attn_sm_count();
  if (sms <= 0) return CONV_ERR_CUDA;
  p.cos = a.cos;
  p.sin = a.sin;
  p.head_dim = a.head_dim;
  p.rot = a.rot_dim;
  p.lanes = a.head_dim / v;
  p.slots = 32 / p.lanes;
  p.table_rows = a.table_rows;
  p.adjacent = a.adjacent_pairs != 0;
  p.eps = a.eps;
  p.inv_d = 1.0f / static_cast<float>(a.head_dim);
  long long units = 0;
  for (QnTensor& t : p.t) {
    if (!t.x || t.rows == 0) continue;
    // One token to a unit where its heads fill most of the unit's rows (the
    // angles are then read once for all of them); else rows back to back.
    const int unit_rows = p.slots * (backward ? kUnrollBwd : kUnrollFwd);
    t.units_per_token = (t.heads + unit_rows - 1) / unit_rows;
    t.many = 4 * t.heads >= 3 * t.units_per_token * unit_rows;
    t.units = t.many ? t.rows / t.heads * t.units_per_token : (t.rows + unit_rows - 1) / unit_rows;
    t.div_heads = make_fast_div(static_cast<uint32_t>(t.heads));
    t.div_upt = make_fast_div(static_cast<uint32_t>(t.units_per_token));
    t.div_length = make_fast_div(static_cast<uint32_t>(t.length));
    units += t.units;
  }
  // The grid fills the SMs once; the two tensors share the blocks in
  // proportion to their units.
  const long long most = static_cast<long long>(sms) * (backward ? kBlocksBwd : kBlocksFwd);
  int grid = 0;
  for (QnTensor& t : p.t) {
    if (t.units == 0) continue;
    const long long want = (t.units + kWarpsQn - 1) / kWarpsQn;
    const long long share =
        units <= most * kWarpsQn ? want : std::max(1ll, (most - 1) * t.units / units);
    t.blocks = static_cast<int>(std::min(want, share));
    grid += t.blocks;
  }
  if (backward) {
    float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + CONV_STATUS_BYTES);
    p.t[0].partial = part;
    p.t[1].partial = part + static_cast<long long>(p.t[0].blocks) * a.head_dim;
  }
  cudaError_t err = cudaSuccess;
  if (grid > 0)
    err = backward ? launch_qn_dtype<true>(a.dtype, v, p, grid, stream)
                   : launch_qn_dtype<false>(a.dtype, v, p, grid, stream);
  if (err == cudaSuccess && backward)
    err = launch_pdl(qk_norm_rope_dw_kernel, dim3(2), dim3(1024), 0, stream, p);
  return err == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace

}  // namespace convgb300

extern "C" {

size_t qk_norm_rope_workspace_size(int head_dim) {
  const int sms = convgb300::attn_sm_count();
  if (head_dim <= 0 || sms <= 0) return 0;
  // One row of partial sums per thread block.
  return CONV_STATUS_BYTES +
         static_cast<size_t>(sms) * convgb300::kBlocksBwd * head_dim * sizeof(float);
}

conv_status_t qk_norm_rope_fwd(const qk_norm_rope_args_t* args, void* stream) {
  return convgb300::run_qk_norm_rope(args, false, nullptr, 0, static_cast<cudaStream_t>(stream));
}

conv_status_t qk_norm_rope_bwd(const qk_norm_rope_args_t* args, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return convgb300::run_qk_norm_rope(args, true, workspace, workspace_bytes,
                                     static_cast<cudaStream_t>(stream));
}

}  // extern "C"
