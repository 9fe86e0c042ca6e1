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
#include "ptx.cuh"

namespace convgb300 {

namespace {

constexpr int kThreadsQn = 256;
constexpr int kWarpsQn = kThreadsQn / 32;
constexpr int kUnroll = 4;          // rows in flight per lane
constexpr int kMaxBlocksQn = 8;     // per SM: 2048 resident threads

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
  int slots_heads; // heads side by side in a warp (many heads: the slots; else all heads)
  int units_per_token;
  long long tokens;  // batch * length
  long long units;
  long long position_stride;
  long long xs[3], ds[3], ys[3];  // batch, token, head
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

template <typename T, int V>
__device__ __forceinline__ void load_row(const void* base, long long off, float (&v)[V]) {
  const T* p = static_cast<const T*>(base) + off;
  uint32_t w[V / 2];
  if (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[V / 2 - 2] = u.z; w[V / 2 - 1] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  }
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float2 f = Pair<T>::load(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(void* base, long long off, const float (&v)[V]) {
  T* p = static_cast<T*>(base) + off;
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) w[i] = Pair<T>::store(v[2 * i], v[2 * i + 1]);
  if (V == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[V / 2 - 2], w[V / 2 - 1]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// Sum over the `lanes` lanes of a row (lane `at` of it), given to all of
// them.  Rows need not fill a power of two: lanes past the end add nothing.
__device__ __forceinline__ float row_sum(float v, int lanes, int at, int first) {
  int step = 16;
  while (step >= lanes) step >>= 1;
  for (; step > 0; step >>= 1) {
    const float o = __shfl_down_sync(0xFFFFFFFFu, v, step);
    if (at + step < lanes && at < step) v += o;
  }
  return __shfl_sync(0xFFFFFFFFu, v, first);
}

// The lane's angles: cos[] and sin[] of its V/2 pairs (adjacent), or of its V
// elements, the second half's sine negated (halves), so that
//   turned = x * c - partner * s.
template <int V>
__device__ __forceinline__ void load_angles(const QnParams& p, const QnTensor& t, long long token,
                                            int e0, float (&c)[V], float (&s)[V]) {
  const long long b = token / t.length;
  const int l = static_cast<int>(token - b * t.length);
  int pos = t.positions ? t.positions[b * t.position_stride + l] : l;
  pos = max(0, min(pos, p.table_rows - 1));
  const int half = p.rot >> 1;
  const long long row = static_cast<long long>(pos) * half;
  if (p.adjacent) {
    const float4 fc = *reinterpret_cast<const float4*>(p.cos + row + (e0 >> 1));
    const float4 fs = *reinterpret_cast<const float4*>(p.sin + row + (e0 >> 1));
    const float cc[4] = {fc.x, fc.y, fc.z, fc.w}, ss[4] = {fs.x, fs.y, fs.z, fs.w};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = cc[(i >> 1) & 3];
      s[i] = (i & 1) ? -ss[(i >> 1) & 3] : ss[(i >> 1) & 3];
    }
    return;
  }
  const bool second = e0 >= half;
  const long long at = row + (second ? e0 - half : e0);
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 fc = *reinterpret_cast<const float4*>(p.cos + at + i);
    const float4 fs = *reinterpret_cast<const float4*>(p.sin + at + i);
    c[i] = fc.x; c[i + 1] = fc.y; c[i + 2] = fc.z; c[i + 3] = fc.w;
    s[i] = fs.x; s[i + 1] = fs.y; s[i + 2] = fs.z; s[i + 3] = fs.w;
  }
  if (second) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = -s[i];
  }
}

// v turned by the angles (sign +1) or back (-1).  Every lane of the warp
// takes part: the pair's other member comes from lane `other`.
template <int V>
__device__ __forceinline__ void turn(const QnParams& p, bool rotated, int other, float sign,
                                     const float (&c)[V], const float (&s)[V], float (&v)[V]) {
  float q[V];
  if (p.adjacent) {
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = v[i ^ 1];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = __shfl_sync(0xFFFFFFFFu, v[i], other);
  }
  if (rotated) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = v[i] * c[i] - sign * (q[i] * s[i]);
  }
}

// kMany: at least as many heads as row slots in a warp; the unit's rows are
// heads of one token.  Otherwise a warp's slots take all heads of several
// tokens.
template <typename T, int V, bool kBackward>
__global__ void __launch_bounds__(kThreadsQn)
    qk_norm_rope_kernel(const __grid_constant__ QnParams p) {
  __shared__ float red[kWarpsQn][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_k = blockIdx.x >= static_cast<unsigned>(p.t[0].blocks);
  const QnTensor& t = p.t[is_k ? 1 : 0];
  const int block = is_k ? blockIdx.x - p.t[0].blocks : blockIdx.x;
  const int slot = lane / p.lanes;
  const int at = lane - slot * p.lanes;
  const int first = slot * p.lanes;
  const bool live = slot < p.slots;
  const int e0 = at * V;
  const int half = p.rot >> 1;
  const bool rotated = live && e0 < p.rot;
  const int other = rotated ? first + (e0 >= half ? at - half / V : at + half / V) : lane;
  const bool many = t.heads >= p.slots;
  grid_dependency_wait();

  float w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) w[i] = 0.f;
  if (live) {
    if (t.weight_f32) {
      const float* wp = static_cast<const float*>(t.weight) + e0;
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = wp[i];
    } else {
      load_row<T, V>(t.weight, e0, w);
    }
  }
  float dw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = 0.f;

  const long long step = static_cast<long long>(t.blocks) * kWarpsQn;
  for (long long unit = static_cast<long long>(block) * kWarpsQn + warp; unit < t.units;
       unit += step) {
    float x[kUnroll][V], g[kUnroll][V], c[V], s[V];
    long long token[kUnroll];
    int head[kUnroll];
    bool ok[kUnroll];
    // Which rows: fixed token and heads slot, slot + slots, ..., or all heads
    // of tokens token0 + slot / heads, ...
    if (many) {
      const long long tk = unit / t.units_per_token;
      const int h0 = static_cast<int>(unit - tk * t.units_per_token) * p.slots * kUnroll + slot;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        token[u] = tk;
        head[u] = h0 + u * p.slots;
        ok[u] = live && head[u] < t.heads;
      }
    } else {
      const int side = slot / t.heads;            // which of the warp's tokens
      const int tokens = p.slots / t.heads;       // tokens side by side
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        token[u] = (unit * kUnroll + u) * tokens + side;
        head[u] = slot - side * t.heads;
        ok[u] = live && side < tokens && token[u] < t.tokens;
      }
    }
    long long off_y[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      off_y[u] = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[u][i] = 0.f;
        g[u][i] = 0.f;
      }
      if (ok[u]) {
        const long long b = token[u] / t.length, l = token[u] - b * t.length;
        off_y[u] = b * t.ys[0] + l * t.ys[1] + head[u] * t.ys[2] + e0;
        load_row<T, V>(t.x, b * t.xs[0] + l * t.xs[1] + head[u] * t.xs[2] + e0, x[u]);
        if (kBackward)
          load_row<T, V>(t.dy, b * t.ds[0] + l * t.ds[1] + head[u] * t.ds[2] + e0, g[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (rotated && ok[u] && (u == 0 || !many)) load_angles<V>(p, t, token[u], e0, c, s);
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) sq = fmaf(x[u][i], x[u][i], sq);
      sq = row_sum(sq, p.lanes, at, first);
      const float r = 1.0f / sqrtf(fmaf(sq, p.inv_d, p.eps));
      if (!kBackward) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[u][i] = x[u][i] * r * w[i];
        turn<V>(p, rotated, other, 1.f, c, s, x[u]);
        if (ok[u]) store_row<T, V>(t.y, off_y[u], x[u]);
      } else {
        turn<V>(p, rotated, other, -1.f, c, s, g[u]);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[u][i] *= r;                                // the normed row
          if (ok[u]) dw[i] = fmaf(g[u][i], x[u][i], dw[i]);
          g[u][i] *= w[i];
          dot = fmaf(g[u][i], x[u][i], dot);
        }
        dot = row_sum(dot, p.lanes, at, first) * p.inv_d;
#pragma unroll
        for (int i = 0; i < V; ++i) g[u][i] = r * (g[u][i] - x[u][i] * dot);
        if (ok[u]) store_row<T, V>(t.y, off_y[u], g[u]);
      }
    }
  }
  grid_launch_dependents();
  if (!kBackward) return;
  // The block's share of dw: slots of a warp, then warps, in order.
  for (int sl = 0; sl < p.slots; ++sl) {
    if (slot == sl) {
#pragma unroll
      for (int i = 0; i < V; ++i) red[warp][e0 + i] = dw[i] + (sl ? red[warp][e0 + i] : 0.f);
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
                           long long out[3]) {
  const int extent[3] = {batch, length, heads};
  for (int i = 0; i < 3; ++i) {
    out[i] = extent[i] > 1 ? in[i] : 0;
    if (extent[i] > 1 && output && in[i] == 0) return CONV_ERR_INVALID_VALUE;
    if (out[i] % 8 != 0) return CONV_ERR_MISALIGNED;
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
  t->tokens = static_cast<long long>(a.batch) * in.length;
  return CONV_OK;
}

template <typename T, int V, bool kBackward>
cudaError_t launch_qn(const QnParams& p, int grid, cudaStream_t stream) {
  return launch_pdl(qk_norm_rope_kernel<T, V, kBackward>, dim3(grid), dim3(kThreadsQn), 0, stream,
                    p);
}

template <bool kBackward>
cudaError_t launch_qn_dtype(int dtype, int v, const QnParams& p, int grid, cudaStream_t stream) {
  if (dtype == CONV_DTYPE_BF16)
    return v == 8 ? launch_qn<__nv_bfloat16, 8, kBackward>(p, grid, stream)
                  : launch_qn<__nv_bfloat16, 4, kBackward>(p, grid, stream);
  return v == 8 ? launch_qn<__half, 8, kBackward>(p, grid, stream)
                : launch_qn<__half, 4, kBackward>(p, grid, stream);
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
    if (!t.x || t.tokens == 0) continue;
    if (t.heads >= p.slots) {
      t.units_per_token = (t.heads + p.slots * kUnroll - 1) / (p.slots * kUnroll);
      t.units = t.tokens * t.units_per_token;
    } else {
      const long long rows = static_cast<long long>(p.slots / t.heads) * kUnroll;
      t.units = (t.tokens + rows - 1) / rows;
    }
    units += t.units;
  }
  // The grid fills the SMs once; the two tensors share the blocks in
  // proportion to their units.
  const long long most = static_cast<long long>(sms) * kMaxBlocksQn;
  int grid = 0;
  for (QnTensor& t : p.t) {
    if (t.units == 0) continue;
    const long long want = (t.units + kWarpsQn - 1) / kWarpsQn;
    long long share = units <= most * kWarpsQn ? want : std::max(1ll, (most - 1) * t.units / units);
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
         static_cast<size_t>(sms) * convgb300::kMaxBlocksQn * head_dim * sizeof(float);
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
