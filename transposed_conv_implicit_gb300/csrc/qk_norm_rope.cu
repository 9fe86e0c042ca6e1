// Norm of queries and keys for each head with the position rotation, forward
// and backward, and their C entry points.
//
// For a row x of one head: r = 1/sqrt(mean x^2 + eps), y = x r w, and the
// pairs (a, b) of y turn by the position's angle.  The rotation is
// orthogonal, so the backward pass turns dy back (g = R^T dy) and
//   dw = sum_rows g x r,   dx = r (g w - x r^2 mean(g w x)).
//
// Bound by memory: x in, y out (dx: x and dy in, dx out) and a few operations
// per element.  A lane holds two words of its row (the members of a word's
// pairs, when halves turn), so that the rotation needs no exchange and the sums
// a few shuffles, and nothing is read twice.  The warp packs 32 / lanes rows
// side by side (10 rows of 40 elements on 30 lanes).  Forward, a lane keeps
// four rows in flight in registers; backward, two, which come through a ring in
// shared memory.  Measured: 8 x (8192 + 4096) x 16 heads x 128 forward 141 us
// (5.7 TB/s), 8 x (4096 x 16 + 2048 x 4 heads) x 128 backward 90 us (5.1 TB/s),
// 16 x 4096 x 8 heads x 40 backward, neighbouring pairs, 49 us (2.6 TB/s: 240
// instructions for 10 short rows).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/conv_gb300_attention.h"
#include "../../include/conv_gb300_testing.h"
#include "attn_internal.h"
#include "conv_params.h"
#include "attn_ptx.cuh"

namespace convgb300 {

namespace {

constexpr int kThreadsQn = 128;
constexpr int kWarpsQn = kThreadsQn / 32;
// Rows in flight per lane, and thread blocks per SM (the register budget):
// the backward pass holds two tensors and a product for each row.
constexpr int kRowsFwd = 4, kRowsBwd = 2;
constexpr int kStagesBwd = 2;  // steps of the backward pass's ring
constexpr int kBlocksFwd = 4, kBlocksBwd = 4;

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
  int rows;          // batch * length * heads
  int tokens;        // batch * length
  int many;          // a lane keeps its token and walks its heads (else rows back to back)
  int run;           // steps of a unit: many, a token's; else one
  int units;
  FastDiv div_length, div_heads;
  long long position_stride;
  uint32_t xs[3], ds[3], ys[3];  // batch, token, head; in 8 elements
};

struct QnParams {
  QnTensor t[2];
  const float* cos;
  const float* sin;
  int head_dim, rot;
  int lanes, slots;   // lanes per row, rows side by side in a warp
  int rot_lanes;      // lanes that hold rotated elements
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

// Each pair's members the other way round.
template <int V>
__device__ __forceinline__ Pairs<V> swapped(const Pairs<V>& own) {
  Pairs<V> q;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    float x, y;
    unpack2(own.v[i], x, y);
    q.v[i] = pack2(y, x);
  }
  return q;
}

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
template <int V>
__device__ __forceinline__ Raw<V> no_raw() {
  Raw<V> r;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) r.w[i] = 0u;
  return r;
}

// One word of a lane's own ring slot: global -> shared without registers;
// zeros when the row is left out.
template <int kBytes>
__device__ __forceinline__ void ring_load(uint32_t dst, const void* src, bool ok) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes),
                 "r"(ok ? kBytes : 0)
                 : "memory");
}
template <int V>
__device__ __forceinline__ Raw<V> ring_read(uint32_t src) {
  Raw<V> r;
  if constexpr (V == 8)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "r"(src)
                 : "memory");
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(src) : "memory");
  return r;
}

// Sums over the `lanes` lanes of a row (lane `at` of it), given to all of
// them, for R rows at once.  Rows need not fill a power of two:
// lanes past the end add nothing.
template <int R>
__device__ __forceinline__ void row_sums(float (&v)[R], int lanes, int at, int first) {
  if ((lanes & (lanes - 1)) == 0) {
    for (int step = lanes >> 1; step > 0; step >>= 1)
#pragma unroll
      for (int u = 0; u < R; ++u) v[u] += __shfl_xor_sync(0xFFFFFFFFu, v[u], step);
    return;
  }
  int step = 16;
  while (step >= lanes) step >>= 1;
  for (; step > 0; step >>= 1) {
    const bool adds = at + step < lanes && at < step;
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const float o = __shfl_down_sync(0xFFFFFFFFu, v[u], step);
      if (adds) v[u] += o;
    }
  }
#pragma unroll
  for (int u = 0; u < R; ++u) v[u] = __shfl_sync(0xFFFFFFFFu, v[u], first);
}

// 1/sqrt(x): the hardware's approximation and one Newton step.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  return r * fmaf(-0.5f * x * r, r, 1.5f);
}

__device__ __forceinline__ uint64_t offset8(uint32_t i, uint32_t stride8) {
  return static_cast<uint64_t>(i) * stride8;
}

// What a lane holds of a row: V elements at ea and V at eb (which may be
// missing).  Rotated halves: the two members of V pairs; else words some
// lanes apart, so that each access of a warp is contiguous.
struct LaneAt {
  int ea, eb;
  bool rot_a, rot_b, has_b;
};

template <int V, bool kAdjacent>
__device__ __forceinline__ LaneAt lane_at(const QnParams& p, int at) {
  LaneAt o;
  if (!kAdjacent && at < p.rot_lanes) {
    o.ea = at * V;
    o.eb = (p.rot >> 1) + at * V;
    o.rot_a = o.rot_b = o.has_b = true;
    return o;
  }
  const int from = kAdjacent ? 0 : p.rot, lane = kAdjacent ? at : at - p.rot_lanes;
  o.ea = from + lane * V;
  o.eb = o.ea + (kAdjacent ? p.lanes : p.lanes - p.rot_lanes) * V;
  o.has_b = o.eb < p.head_dim;
  o.rot_a = kAdjacent && o.ea < p.rot;
  o.rot_b = kAdjacent && o.eb < p.rot;
  return o;
}

// A lane's angles for a position, so that x -> x c + q s with q the pair's
// other member: the other word's element (halves), or the word's neighbour
// (adjacent).  The rotation: s = -sin for first members, +sin for second
// ones; `back` turns the other way.
template <int V>
struct Angles {
  Pairs<V> ca, sa, cb, sb;
};

template <int V, bool kAdjacent, bool kBack>
__device__ __forceinline__ void load_angles(const QnParams& p, int pos, const LaneAt& at,
                                            Angles<V>& o) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    o.ca.v[i] = o.cb.v[i] = pack2(1.f, 1.f);
    o.sa.v[i] = o.sb.v[i] = 0;
  }
  if (!at.rot_a) return;
  pos = max(0, min(pos, p.table_rows - 1));
  const uint64_t row =
      static_cast<uint64_t>(static_cast<uint32_t>(pos)) * static_cast<uint32_t>(p.rot >> 1);
  constexpr float f = kBack ? 1.f : -1.f;  // of a first member's sine
  if constexpr (kAdjacent) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int e = w ? at.eb : at.ea;
      if (w && !at.rot_b) break;
      const float4 fc = *reinterpret_cast<const float4*>(p.cos + row + (e >> 1));
      const float4 fs = *reinterpret_cast<const float4*>(p.sin + row + (e >> 1));
      const float cc[4] = {fc.x, fc.y, fc.z, fc.w}, ss[4] = {fs.x, fs.y, fs.z, fs.w};
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        (w ? o.cb : o.ca).v[i] = pack2(cc[i & 3], cc[i & 3]);
        (w ? o.sb : o.sa).v[i] = pack2(f * ss[i & 3], -f * ss[i & 3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 fc = *reinterpret_cast<const float4*>(p.cos + row + at.ea + i);
      const float4 fs = *reinterpret_cast<const float4*>(p.sin + row + at.ea + i);
      o.ca.v[i / 2] = o.cb.v[i / 2] = pack2(fc.x, fc.y);
      o.ca.v[i / 2 + 1] = o.cb.v[i / 2 + 1] = pack2(fc.z, fc.w);
      o.sa.v[i / 2] = pack2(f * fs.x, f * fs.y);
      o.sa.v[i / 2 + 1] = pack2(f * fs.z, f * fs.w);
      o.sb.v[i / 2] = pack2(-f * fs.x, -f * fs.y);
      o.sb.v[i / 2 + 1] = pack2(-f * fs.z, -f * fs.w);
    }
  }
}

template <int V>
__device__ __forceinline__ Pairs<V> weights(const float* weight, int e, bool ok) {
  Pairs<V> w;
#pragma unroll
  for (int i = 0; i < V / 2; i += 2) {
    const float4 f = ok ? *reinterpret_cast<const float4*>(weight + e + 2 * i)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    w.v[i] = pack2(f.x, f.y);
    w.v[i + 1] = pack2(f.z, f.w);
  }
  return w;
}

// Forward, the weights go into the angles: q is the other member before its
// own weight.
template <int V, bool kAdjacent>
__device__ __forceinline__ void weigh(const float* weight, const LaneAt& la, Angles<V>& an) {
  const Pairs<V> wa = weights<V>(weight, la.ea, true), wb = weights<V>(weight, la.eb, la.has_b);
  const Pairs<V> fa = kAdjacent ? swapped<V>(wa) : wb, fb = kAdjacent ? swapped<V>(wb) : wa;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    an.ca.v[i] = mul2(an.ca.v[i], wa.v[i]);
    an.sa.v[i] = mul2(an.sa.v[i], fa.v[i]);
    an.cb.v[i] = mul2(an.cb.v[i], wb.v[i]);
    an.sb.v[i] = mul2(an.sb.v[i], fb.v[i]);
  }
}

template <int V>
struct Loaded {
  Raw<V> xa, xb, ga, gb;
};

template <int V>
__device__ __forceinline__ Loaded<V> load_row(const uint16_t* x, const LaneAt& la, bool ok) {
  Loaded<V> o;
  o.xa = o.xb = no_raw<V>();
  if (ok) {
    o.xa = load_raw<V>(x + la.ea);
    if (la.has_b) o.xb = load_raw<V>(x + la.eb);
  }
  return o;
}

// A row's sum of squares, this lane's part.
template <typename T, int V>
__device__ __forceinline__ float square_sum(const Loaded<V>& x) {
  const Pairs<V> va = widen<T, V>(x.xa), vb = widen<T, V>(x.xb);
  uint64_t sq = mul2(va.v[0], va.v[0]);
#pragma unroll
  for (int i = 1; i < V / 2; ++i) sq = fma2(va.v[i], va.v[i], sq);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) sq = fma2(vb.v[i], vb.v[i], sq);
  float lo, hi;
  unpack2(sq, lo, hi);
  return lo + hi;
}

template <typename T, int V, bool kAdjacent>
__device__ __forceinline__ void forward_row(const Loaded<V>& x, float r, const Angles<V>& an,
                                            uint16_t* y, const LaneAt& la) {
  const Pairs<V> va = widen<T, V>(x.xa), vb = widen<T, V>(x.xb);
  const Pairs<V> qa = kAdjacent ? swapped<V>(va) : vb, qb = kAdjacent ? swapped<V>(vb) : va;
  const uint64_t rr = pack2(r, r);
  Pairs<V> ya, yb;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    ya.v[i] = mul2(rr, fma2(qa.v[i], an.sa.v[i], mul2(va.v[i], an.ca.v[i])));
    yb.v[i] = mul2(rr, fma2(qb.v[i], an.sb.v[i], mul2(vb.v[i], an.cb.v[i])));
  }
  store_row<T, V>(y + la.ea, ya);
  if (la.has_b) store_row<T, V>(y + la.eb, yb);
}

// Turns dy back and weighs it (fa, fb), adds the row's share of dw, and
// returns this lane's part of the dot product with the normed row.
template <typename T, int V, bool kAdjacent>
__device__ __forceinline__ float turn_back(const Loaded<V>& x, float r, const Angles<V>& an,
                                           const float* weight, const LaneAt& la, Pairs<V>& fa,
                                           Pairs<V>& fb, Pairs<V>& dwa, Pairs<V>& dwb) {
  const Pairs<V> da = widen<T, V>(x.ga), db = widen<T, V>(x.gb);
  const Pairs<V> qa = kAdjacent ? swapped<V>(da) : db, qb = kAdjacent ? swapped<V>(db) : da;
  const Pairs<V> va = widen<T, V>(x.xa), vb = widen<T, V>(x.xb);
  const Pairs<V> wa = weights<V>(weight, la.ea, true), wb = weights<V>(weight, la.eb, la.has_b);
  const uint64_t rr = pack2(r, r);
  uint64_t sum = 0;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const uint64_t ta = fma2(qa.v[i], an.sa.v[i], mul2(da.v[i], an.ca.v[i]));
    const uint64_t tb = fma2(qb.v[i], an.sb.v[i], mul2(db.v[i], an.cb.v[i]));
    const uint64_t ha = mul2(va.v[i], rr), hb = mul2(vb.v[i], rr);
    dwa.v[i] = fma2(ta, ha, dwa.v[i]);  // (rows left out hold zeros)
    dwb.v[i] = fma2(tb, hb, dwb.v[i]);
    fa.v[i] = mul2(ta, wa.v[i]);
    fb.v[i] = mul2(tb, wb.v[i]);
    sum = fma2(fa.v[i], ha, sum);
    sum = fma2(fb.v[i], hb, sum);
  }
  float lo, hi;
  unpack2(sum, lo, hi);
  return lo + hi;
}

// dx = r f - x r^3 mean(f x): `dot` is mean(f x r).
template <typename T, int V>
__device__ __forceinline__ void backward_row(const Loaded<V>& x, float r, float dot,
                                             const Pairs<V>& fa, const Pairs<V>& fb, uint16_t* y,
                                             const LaneAt& la) {
  Pairs<V> va = widen<T, V>(x.xa), vb = widen<T, V>(x.xb);
  const float f = -dot * r * r;
  const uint64_t rr = pack2(r, r), ff = pack2(f, f);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    va.v[i] = fma2(va.v[i], ff, mul2(rr, fa.v[i]));
    vb.v[i] = fma2(vb.v[i], ff, mul2(rr, fb.v[i]));
  }
  store_row<T, V>(y + la.ea, va);
  if (la.has_b) store_row<T, V>(y + la.eb, vb);
}

// A step's rows and where they go.
template <int V, int R>
struct Rows {
  Loaded<V> x[R];
  bool ok[R];
  uint16_t* y[R];
};

// One step; `angles(u)` gives those of row u.
template <typename T, int V, int R, bool kAdjacent, typename F>
__device__ __forceinline__ void norm_step(const QnParams& p, const Rows<V, R>& s, const LaneAt& la, int at, int first, F angles) {
  float r[R];
#pragma unroll
  for (int u = 0; u < R; ++u) r[u] = square_sum<T, V>(s.x[u]);
  row_sums<R>(r, p.lanes, at, first);
#pragma unroll
  for (int u = 0; u < R; ++u) r[u] = inverse_root(fmaf(r[u], p.inv_d, p.eps));
#pragma unroll
  for (int u = 0; u < R; ++u) {
    const Angles<V>& an = angles(u);
    if (s.ok[u]) forward_row<T, V, kAdjacent>(s.x[u], r[u], an, s.y[u], la);
  }
}

// kMany: each slot of the warp takes one token and walks its heads, R at a
// time, with the token's angles in registers.  Otherwise rows are consecutive
// (token, head) pairs, each with its own angles.
template <typename T, int V, bool kAdjacent, bool kMany>
__device__ __forceinline__ void norm_rows(const QnParams& p, const QnTensor& t, int block,
                                          const float* weight) {
  constexpr int R = kRowsFwd;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = lane / p.lanes;
  const int at = lane - slot * p.lanes, first = slot * p.lanes;
  const bool live = slot < p.slots;
  const LaneAt la = lane_at<V, kAdjacent>(p, live ? at : 0);
  const uint16_t* px = static_cast<const uint16_t*>(t.x);
  uint16_t* py = static_cast<uint16_t*>(t.y);
  const int stride = t.blocks * kWarpsQn;
  Angles<V> an;
  if constexpr (kMany) {
    // (The next token's position is read one unit ahead.)
    int b = 0, l = 0, pos = 0;
    bool here = false;
    auto place = [&](int unit) {
      const int token = unit * p.slots + slot;
      here = live && token < t.tokens;
      b = fast_div(here ? token : 0, t.div_length);
      l = (here ? token : 0) - b * t.length;
      pos = t.positions ? t.positions[b * t.position_stride + l] : l;
    };
    int unit = block * kWarpsQn + warp;
    if (unit < t.units) place(unit);
    const uint64_t sx = offset8(t.xs[2], 8), sy = offset8(t.ys[2], 8);
    while (unit < t.units) {
      const uint16_t* x0 = px + (offset8(b, t.xs[0]) + offset8(l, t.xs[1])) * 8;
      uint16_t* y0 = py + (offset8(b, t.ys[0]) + offset8(l, t.ys[1])) * 8;
      const int this_pos = pos, heads = here ? t.heads : 0;
      unit += stride;
      if (unit < t.units) place(unit);
      int head = 0;
      for (int i = 0; i < t.run; ++i) {
        Rows<V, R> s;
#pragma unroll
        for (int u = 0; u < R; ++u) {
          s.ok[u] = head + u < heads;
          s.x[u] = load_row<V>(x0 + u * sx, la, s.ok[u]);
          s.y[u] = y0 + u * sy;
        }
        if (i == 0) {
          load_angles<V, kAdjacent, false>(p, this_pos, la, an);
          weigh<V, kAdjacent>(weight, la, an);
        }
        norm_step<T, V, R, kAdjacent>(p, s, la, at, first,
                                      [&](int) -> const Angles<V>& { return an; });
        head += R;
        x0 += R * sx;
        y0 += R * sy;
      }
    }
  } else {
    for (int unit = block * kWarpsQn + warp; unit < t.units; unit += stride) {
      Rows<V, R> s;
      int pos[R];
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const int row = (unit * R + u) * p.slots + slot;
        s.ok[u] = live && row < t.rows;
        const int token = fast_div(row, t.div_heads), head = row - token * t.heads;
        const int b = fast_div(token, t.div_length), l = token - b * t.length;
        s.x[u] = load_row<V>(
            px + (offset8(b, t.xs[0]) + offset8(l, t.xs[1]) + offset8(head, t.xs[2])) * 8, la, s.ok[u]);
        s.y[u] = py + (offset8(b, t.ys[0]) + offset8(l, t.ys[1]) + offset8(head, t.ys[2])) * 8;
        pos[u] = !s.ok[u] ? 0 : t.positions ? t.positions[b * t.position_stride + l] : l;
      }
      norm_step<T, V, R, kAdjacent>(
          p, s, la, at, first, [&](int u) -> const Angles<V>& {
            load_angles<V, kAdjacent, false>(p, pos[u], la, an);
            weigh<V, kAdjacent>(weight, la, an);
            return an;
          });
    }
  }
}

// Backward: the rows come through a ring of kStages steps in shared memory,
// each lane's words in slots of its own (no barriers), with where the row's
// result goes and its position beside them; kStages - 1 steps are in flight.
template <typename T, int V, bool kAdjacent, bool kMany>
__device__ __forceinline__ void norm_rows_back(const QnParams& p, const QnTensor& t, int block,
                                               const float* weight, float* red, uint32_t ring) {
  constexpr int R = kRowsBwd, S = kStagesBwd;
  constexpr uint32_t kWord = V * 2, kPitch = kThreadsQn * kWord, kRow = 4 * kPitch + 16 * kThreadsQn;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = lane / p.lanes;
  const int at = lane - slot * p.lanes, first = slot * p.lanes;
  const bool live = slot < p.slots;
  const LaneAt la = lane_at<V, kAdjacent>(p, live ? at : 0);
  const uint32_t words = ring + threadIdx.x * kWord;                      // x a, x b, dy a, dy b
  const uint32_t notes = ring + 4 * kPitch + threadIdx.x * 16;            // y offset, row ok, position
  const uint16_t* px = static_cast<const uint16_t*>(t.x);
  const uint16_t* pg = static_cast<const uint16_t*>(t.dy);
  uint16_t* py = static_cast<uint16_t*>(t.y);
  const int stride = t.blocks * kWarpsQn;
  Pairs<V> dwa, dwb;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) dwa.v[i] = dwb.v[i] = 0;

  // The loading side: step `part` of a unit.
  const uint64_t sx = offset8(t.xs[2], 8), sg = offset8(t.ds[2], 8), sy = offset8(t.ys[2], 8);
  int unit = block * kWarpsQn + warp, part = 0, left = 0;
  const uint16_t *x0 = px, *g0 = pg;
  auto load_step = [&](int stage) {
    if (unit < t.units) {
      if (kMany && part == 0) {
        const int token = unit * p.slots + slot;
        left = live && token < t.tokens ? t.heads : 0;
        const int b = fast_div(left ? token : 0, t.div_length);
        const int l = (left ? token : 0) - b * t.length;
        x0 = px + (offset8(b, t.xs[0]) + offset8(l, t.xs[1])) * 8;
        g0 = pg + (offset8(b, t.ds[0]) + offset8(l, t.ds[1])) * 8;
      }
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const uint32_t w = words + (stage * R + u) * kRow, n = notes + (stage * R + u) * kRow;
        const uint16_t *x, *g;
        bool ok;
        if constexpr (kMany) {
          ok = u < left;
          x = ok ? x0 + u * sx : px;
          g = ok ? g0 + u * sg : pg;
        } else {
          const int row = (unit * R + u) * p.slots + slot;
          ok = live && row < t.rows;
          const int token = fast_div(ok ? row : 0, t.div_heads);
          const int head = (ok ? row : 0) - token * t.heads;
          const int b = fast_div(token, t.div_length), l = token - b * t.length;
          x = px + (offset8(b, t.xs[0]) + offset8(l, t.xs[1]) + offset8(head, t.xs[2])) * 8;
          g = pg + (offset8(b, t.ds[0]) + offset8(l, t.ds[1]) + offset8(head, t.ds[2])) * 8;
          const uint64_t y = (offset8(b, t.ys[0]) + offset8(l, t.ys[1]) + offset8(head, t.ys[2])) * 8;
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(n), "r"(static_cast<uint32_t>(y)),
                       "r"(static_cast<uint32_t>(y >> 32))
                       : "memory");
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(n + 8), "r"(ok ? 1u : 0u) : "memory");
          if (t.positions)
            ring_load<4>(n + 12, t.positions + b * t.position_stride + l, true);
          else
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(n + 12), "r"(l) : "memory");
        }
        const int eb = la.has_b ? la.eb : la.ea;
        ring_load<kWord>(w, x + la.ea, ok);
        ring_load<kWord>(w + kPitch, x + eb, ok && la.has_b);
        ring_load<kWord>(w + 2 * kPitch, g + la.ea, ok);
        ring_load<kWord>(w + 3 * kPitch, g + eb, ok && la.has_b);
      }
      if constexpr (kMany) {
        left -= R;
        x0 += R * sx;
        g0 += R * sg;
      }
      if (!kMany || ++part == t.run) {
        part = 0;
        unit += stride;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // The arithmetic's side (many: the next token's position is read one unit ahead).
  int now = unit, now_part = 0, heads = 0, next_heads = 0, next_pos = 0;
  uint16_t *y0 = py, *next_y = py;
  auto place = [&](int at_unit) {
    const int token = at_unit * p.slots + slot;
    next_heads = live && token < t.tokens ? t.heads : 0;
    const int b = fast_div(next_heads ? token : 0, t.div_length);
    const int l = (next_heads ? token : 0) - b * t.length;
    next_pos = t.positions ? t.positions[b * t.position_stride + l] : l;
    next_y = py + (offset8(b, t.ys[0]) + offset8(l, t.ys[1])) * 8;
  };
  if (kMany && now < t.units) place(now);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) load_step(i);

  Angles<V> an;
  int stage = 0;
  while (now < t.units) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    const uint32_t w = words + stage * R * kRow, n = notes + stage * R * kRow;
    uint16_t* y[R];
    bool ok[R];
    int pos[R];
    float r[R];
    if constexpr (kMany) {
      if (now_part == 0) {
        heads = next_heads;
        y0 = next_y;
        load_angles<V, kAdjacent, true>(p, next_pos, la, an);
        if (now + stride < t.units) place(now + stride);
      }
#pragma unroll
      for (int u = 0; u < R; ++u) {
        ok[u] = u < heads;
        y[u] = y0 + u * sy;
      }
      heads -= R;
      y0 += R * sy;
    } else {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        uint32_t lo, hi, good, at_pos;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(lo), "=r"(hi), "=r"(good), "=r"(at_pos)
                     : "r"(n + u * kRow)
                     : "memory");
        y[u] = py + ((static_cast<uint64_t>(hi) << 32) | lo);
        ok[u] = good != 0;
        pos[u] = static_cast<int>(at_pos);
      }
    }
    // (The stage read in the step before is free.)
    load_step(stage == 0 ? S - 1 : stage - 1);
#pragma unroll
    for (int u = 0; u < R; ++u) {
      Loaded<V> x;
      x.xa = ring_read<V>(w + u * kRow);
      x.xb = ring_read<V>(w + u * kRow + kPitch);
      r[u] = square_sum<T, V>(x);
    }
    row_sums<R>(r, p.lanes, at, first);
    float dot[R];
    Pairs<V> fa[R], fb[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      r[u] = inverse_root(fmaf(r[u], p.inv_d, p.eps));
      if (!kMany) load_angles<V, kAdjacent, true>(p, pos[u], la, an);
      Loaded<V> x;
      x.xa = ring_read<V>(w + u * kRow);
      x.xb = ring_read<V>(w + u * kRow + kPitch);
      x.ga = ring_read<V>(w + u * kRow + 2 * kPitch);
      x.gb = ring_read<V>(w + u * kRow + 3 * kPitch);
      dot[u] = turn_back<T, V, kAdjacent>(x, r[u], an, weight, la, fa[u], fb[u], dwa, dwb);
    }
    row_sums<R>(dot, p.lanes, at, first);
#pragma unroll
    for (int u = 0; u < R; ++u) {
      Loaded<V> x;
      x.xa = ring_read<V>(w + u * kRow);
      x.xb = ring_read<V>(w + u * kRow + kPitch);
      if (ok[u]) backward_row<T, V>(x, r[u], dot[u] * p.inv_d, fa[u], fb[u], y[u], la);
    }
    if (!kMany || ++now_part == t.run) {
      now_part = 0;
      now += stride;
    }
    if (++stage == S) stage = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // The block's share of dw: slots of a warp, then warps, in order.
  float* mine = red + warp * 256;
  for (int sl = 0; sl < p.slots; ++sl) {
    if (slot == sl) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        float x, y;
        unpack2(dwa.v[i], x, y);
        mine[la.ea + 2 * i] = x + (sl ? mine[la.ea + 2 * i] : 0.f);
        mine[la.ea + 2 * i + 1] = y + (sl ? mine[la.ea + 2 * i + 1] : 0.f);
        if (!la.has_b) continue;
        unpack2(dwb.v[i], x, y);
        mine[la.eb + 2 * i] = x + (sl ? mine[la.eb + 2 * i] : 0.f);
        mine[la.eb + 2 * i + 1] = y + (sl ? mine[la.eb + 2 * i + 1] : 0.f);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.head_dim; d += kThreadsQn) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarpsQn; ++i) sum += red[i * 256 + d];
    t.partial[static_cast<long long>(block) * p.head_dim + d] = sum;
  }
}

// Shared memory of the backward kernel: weights, the warps' shares of dw, the ring.
template <int V>
constexpr size_t qn_back_smem() {
  return 1024 + kWarpsQn * 1024 +
         static_cast<size_t>(kStagesBwd) * kRowsBwd * kThreadsQn * (4 * V * 2 + 16);
}

template <typename T, int V, bool kAdjacent, bool kBackward>
__global__ void __launch_bounds__(kThreadsQn, kBackward ? kBlocksBwd : kBlocksFwd)
    qk_norm_rope_kernel(const __grid_constant__ QnParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  float* weight = reinterpret_cast<float*>(smem);
  const bool is_k = blockIdx.x >= static_cast<unsigned>(p.t[0].blocks);
  const QnTensor& t = p.t[is_k ? 1 : 0];
  const int block = is_k ? blockIdx.x - p.t[0].blocks : blockIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  for (int e = threadIdx.x; e < p.head_dim; e += kThreadsQn)
    weight[e] = t.weight_f32 ? static_cast<const float*>(t.weight)[e]
                             : Pair<T>::load(static_cast<const uint16_t*>(t.weight)[e]).x;
  __syncthreads();
  if constexpr (kBackward) {
    float* red = weight + 256;
    const uint32_t ring = smem_u32(smem) + 1024 + kWarpsQn * 1024;
    if (t.many)
      norm_rows_back<T, V, kAdjacent, true>(p, t, block, weight, red, ring);
    else
      norm_rows_back<T, V, kAdjacent, false>(p, t, block, weight, red, ring);
  } else {
    if (t.many)
      norm_rows<T, V, kAdjacent, true>(p, t, block, weight);
    else
      norm_rows<T, V, kAdjacent, false>(p, t, block, weight);
  }
}

// dw = the blocks' shares, summed in a fixed order: one thread block per
// tensor and 32 elements, its warps taking every 32nd share each, so that all
// of a lane's reads are in flight together.
__global__ void __launch_bounds__(1024) qk_norm_rope_dw_kernel(const __grid_constant__ QnParams p) {
  __shared__ float part[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const QnTensor& t = p.t[blockIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = blockIdx.x * 32 + lane;
  if (!t.dweight) return;
  float sum = 0.f;
  if (d < p.head_dim) {
#pragma unroll 8
    for (int i = warp; i < t.blocks; i += 32)
      sum += t.partial[static_cast<long long>(i) * p.head_dim + d];
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && d < p.head_dim) {
    sum = 0.f;  // (a tensor without rows: the gradient of its weight is zero)
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += part[i][lane];
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
  t->tokens = static_cast<int>(tokens);
  return CONV_OK;
}

template <typename T, int V, bool kAdjacent, bool kBackward>
cudaError_t launch_qn_one(const QnParams& p, int grid, cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  const size_t smem = kBackward ? qn_back_smem<V>() : 1024;
  if (smem > 48 * 1024) {
    const cudaError_t e = raise_smem(qk_norm_rope_kernel<T, V, kAdjacent, kBackward>, configured, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(qk_norm_rope_kernel<T, V, kAdjacent, kBackward>, dim3(grid), dim3(kThreadsQn),
                    smem, stream, p);
}

template <typename T, bool kBackward>
cudaError_t launch_qn(const QnParams& p, int v, int grid, cudaStream_t stream) {
  if (p.adjacent) return launch_qn_one<T, 8, true, kBackward>(p, grid, stream);
  if (v == 8) return launch_qn_one<T, 8, false, kBackward>(p, grid, stream);
  return launch_qn_one<T, 4, false, kBackward>(p, grid, stream);
}

template <bool kBackward>
cudaError_t launch_qn_dtype(int dtype, int v, const QnParams& p, int grid, cudaStream_t stream) {
  return dtype == CONV_DTYPE_BF16 ? launch_qn<__nv_bfloat16, kBackward>(p, v, grid, stream)
                                  : launch_qn<__half, kBackward>(p, v, grid, stream);
}

// Thread blocks of the two tensors: a warp for every unit where those fit the
// SMs once, else a share of the blocks in proportion to the units.  They add up
// to no more than `most`, for which the workspace holds rows of partial sums.
// (The choice goes by the sum of both tensors' whole blocks: each rounds up by
// itself, so units that fit may still need a block more than there are.)
void share_blocks(QnTensor (&t)[2], int most) {
  long long units = 0, want[2];
  for (int i = 0; i < 2; ++i) {
    units += t[i].units;
    want[i] = (t[i].units + kWarpsQn - 1) / kWarpsQn;
  }
  for (int i = 0; i < 2; ++i) {
    if (t[i].units == 0) continue;
    const long long share = want[0] + want[1] <= most
                                ? want[i]
                                : std::max(1ll, (most - 1ll) * t[i].units / units);
    t[i].blocks = static_cast<int>(std::min(want[i], share));
  }
}

// Rows of partial sums that the backward pass's workspace holds.
int partial_rows(int sms) { return sms * kBlocksBwd; }

// Checks a call and takes its arguments over; `v`: the elements of a lane's word.
conv_status_t plan_qk_norm_rope(const qk_norm_rope_args_t& a, bool backward, QnParams* out, int* v) {
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
  // 8-byte words, so that a pair's members sit in whole words (32 lanes at the
  // most, for 256 elements).
  *v = !a.adjacent_pairs && a.rot_dim % 16 != 0 ? 4 : 8;
  const int rot_lanes = (a.rot_dim + 2 * *v - 1) / (2 * *v);
  const int lanes = a.adjacent_pairs ? (a.head_dim + 15) / 16
                                     : rot_lanes + (a.head_dim - a.rot_dim + 2 * *v - 1) / (2 * *v);
  QnParams& p = *out;
  p = QnParams{};
  conv_status_t st = take_tensor(a, a.q, backward, &p.t[0]);
  if (st == CONV_OK) st = take_tensor(a, a.k, backward, &p.t[1]);
  if (st != CONV_OK) return st;
  p.cos = a.cos;
  p.sin = a.sin;
  p.head_dim = a.head_dim;
  p.rot = a.rot_dim;
  p.lanes = lanes;
  p.rot_lanes = rot_lanes;
  p.slots = 32 / p.lanes;
  p.table_rows = a.table_rows;
  p.adjacent = a.adjacent_pairs != 0;
  p.eps = a.eps;
  p.inv_d = 1.0f / static_cast<float>(a.head_dim);
  return CONV_OK;
}

// Units and thread blocks of both tensors on `sms` SMs; returns the grid.
int share_qk_norm_rope(QnParams& p, bool backward, int sms) {
  for (QnTensor& t : p.t) {
    if (!t.x || t.rows == 0) continue;
    // Lanes keep their token where there are tokens for every warp and heads
    // to fill their steps: the angles are then read once for all heads.  Else
    // rows back to back, which few tokens spread further.  (Both sides: 141 us
    // against 182 for the long forward call above, 90 against 100 and 48.6
    // against 49.4 for the backward ones.)
    const int rows_step = backward ? kRowsBwd : kRowsFwd;
    const int parts = (t.heads + rows_step - 1) / rows_step;
    const int warps = sms * (backward ? kBlocksBwd : kBlocksFwd) * kWarpsQn;
    t.many = t.tokens / p.slots >= warps && 4 * t.heads >= 3 * parts * rows_step;
    t.run = t.many ? parts : 1;
    t.units = t.many ? (t.tokens + p.slots - 1) / p.slots
                     : (t.rows + p.slots * rows_step - 1) / (p.slots * rows_step);
    t.div_heads = make_fast_div(static_cast<uint32_t>(t.heads));
    t.div_length = make_fast_div(static_cast<uint32_t>(t.length));
  }
  // The grid fills the SMs once.
  share_blocks(p.t, backward ? partial_rows(sms) : sms * kBlocksFwd);
  return p.t[0].blocks + p.t[1].blocks;
}

conv_status_t run_qk_norm_rope(const qk_norm_rope_args_t* args, bool backward, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
  if (!args) return CONV_ERR_INVALID_VALUE;
  const qk_norm_rope_args_t& a = *args;
  QnParams p;
  int v = 0;
  const conv_status_t st = plan_qk_norm_rope(a, backward, &p, &v);
  if (st != CONV_OK) return st;
  if (backward) {
    if (!workspace) return CONV_ERR_INVALID_VALUE;
    if (misaligned(workspace)) return CONV_ERR_MISALIGNED;
    if (workspace_bytes < qk_norm_rope_workspace_size(a.head_dim))
      return CONV_ERR_WORKSPACE_TOO_SMALL;
  }
  const int sms = attn_sm_count();
  if (sms <= 0) return CONV_ERR_CUDA;
  const int grid = share_qk_norm_rope(p, backward, sms);
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
    err = launch_pdl(qk_norm_rope_dw_kernel, dim3((a.head_dim + 31) / 32, 2), dim3(1024), 0, stream, p);
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
         static_cast<size_t>(convgb300::partial_rows(sms)) * head_dim * sizeof(float);
}

conv_status_t qk_norm_rope_fwd(const qk_norm_rope_args_t* args, void* stream) {
  return convgb300::run_qk_norm_rope(args, false, nullptr, 0, static_cast<cudaStream_t>(stream));
}

conv_status_t qk_norm_rope_bwd(const qk_norm_rope_args_t* args, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return convgb300::run_qk_norm_rope(args, true, workspace, workspace_bytes,
                                     static_cast<cudaStream_t>(stream));
}

conv_status_t conv_testing_qk_norm_rope_blocks(const qk_norm_rope_args_t* args, int backward,
                                               int num_sms, int out[3]) {
  using namespace convgb300;
  QnParams p;
  int v = 0;
  const conv_status_t st = plan_qk_norm_rope(*args, backward != 0, &p, &v);
  if (st != CONV_OK) return st;
  share_qk_norm_rope(p, backward != 0, num_sms);
  out[0] = p.t[0].blocks;
  out[1] = p.t[1].blocks;
  out[2] = partial_rows(num_sms);
  return CONV_OK;
}

}  // extern "C"
