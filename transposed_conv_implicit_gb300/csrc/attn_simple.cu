// Cross attention on CUDA cores, forward and backward: small fp32 tiles in
// shared memory, right for every case the entry points accept.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_internal.h"
#include "attn_params.h"
#include "ptx.cuh"

namespace convgb300 {

namespace {

constexpr int kRows = 16;      // resident rows (queries; keys in the key pass)
constexpr int kCols = 32;      // streamed rows
constexpr int kThreadsS = 128; // 8 threads per resident row
constexpr int kMaxD = 128;
constexpr int kPitch = kMaxD + 4;

__device__ __forceinline__ float get(const void* p, long long i, int dtype) {
  return dtype == 0 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                    : __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void put(void* p, long long i, int dtype, float v) {
  if (dtype == 0)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ int valid_keys(const AttnShape& a, int b) {
  return a.kv_lengths ? max(0, min(a.kv_lengths[b], a.kv_len)) : a.kv_len;
}

__device__ __forceinline__ bool takes_part(const AttnShape& a, int b, int h, int i, int j, int n) {
  if (j >= n) return false;
  if (!a.mask_bits) return true;
  const long long row = b * a.mask_b + h * a.mask_h + i * a.mask_q;
  return (a.mask_bits[row * a.mask_words + (j >> 5)] >> (j & 31)) & 1u;
}

// rows [r0, r0 + count) of (b, head) into fp32 rows of kPitch; rows past the
// limit and, with `keep`, unwanted rows become zero.
__device__ __forceinline__ void load_tile(float* dst, const void* src, const long long s[3], int b,
                                          int head, int r0, int count, int limit, int d, int dtype) {
  for (int i = threadIdx.x; i < count * d; i += kThreadsS) {
    const int r = i / d, c = i - r * d;
    float v = 0.f;
    if (r0 + r < limit)
      v = get(src, b * s[0] + static_cast<long long>(r0 + r) * s[1] + head * s[2] + c, dtype);
    dst[r * kPitch + c] = v;
  }
}

__device__ __forceinline__ float dot_rows(const float* x, const float* y, int d) {
  float s = 0.f;
  for (int c = 0; c < d; ++c) s = fmaf(x[c], y[c], s);
  return s;
}

// Rows of a streamed tile that no resident row takes part with are cleared,
// so that nothing they hold reaches a product.
__device__ __forceinline__ void clear_unused(float* x, float* y, const uint32_t* used, int d) {
  for (int i = threadIdx.x; i < kCols * d; i += kThreadsS) {
    const int r = i / d, c = i - r * d;
    if (!((*used >> r) & 1u)) {
      x[r * kPitch + c] = 0.f;
      if (y) y[r * kPitch + c] = 0.f;
    }
  }
}

struct Tiles {
  float a[kRows * kPitch], b[kRows * kPitch];
  float x[kCols * kPitch], y[kCols * kPitch];
  float p[kRows * (kCols + 1)], ds[kRows * (kCols + 1)];
  float lse[kCols], delta[kCols];
  uint32_t used;
};

// kGrad false: out and lse.  kGrad true: dq.
template <bool kGrad>
__global__ void __launch_bounds__(kThreadsS) attn_simple_query_kernel(const AttnShape a) {
  extern __shared__ float raw[];
  Tiles& t = *reinterpret_cast<Tiles*>(raw);
  const int d = a.head_dim, dt = a.dtype;
  const int h = blockIdx.y % a.heads, b = blockIdx.y / a.heads, g = h / a.group;
  const int i0 = blockIdx.x * kRows;
  const int row = threadIdx.x >> 3, part = threadIdx.x & 7, i = i0 + row;
  grid_dependency_wait();
  const int n = valid_keys(a, b);
  load_tile(t.a, a.q, a.qs, b, h, i0, kRows, a.q_len, d, dt);
  if (kGrad) load_tile(t.b, a.dout, a.dos, b, h, i0, kRows, a.q_len, d, dt);
  __syncthreads();
  const long long lse_at = (static_cast<long long>(b) * a.heads + h) * a.q_len + i;
  float lse = -INFINITY, delta = 0.f, top = -INFINITY, sum = 0.f, acc[kMaxD / 8];
  for (float& v : acc) v = 0.f;
  if (kGrad && i < a.q_len) {
    lse = a.lse[lse_at];
    for (int c = part; c < d; c += 8)
      delta = fmaf(t.b[row * kPitch + c], get(a.out, b * a.os[0] + i * a.os[1] + h * a.os[2] + c, dt),
                   delta);
  }
  if (kGrad)
    for (int s = 4; s; s >>= 1) delta += __shfl_xor_sync(0xFFFFFFFFu, delta, s);
  for (int j0 = 0; j0 < n; j0 += kCols) {
    __syncthreads();
    if (threadIdx.x == 0) t.used = 0;
    load_tile(t.x, a.k, a.ks, b, g, j0, kCols, n, d, dt);
    load_tile(t.y, a.v, a.vs, b, g, j0, kCols, n, d, dt);
    __syncthreads();
    float s[kCols / 8], most = -INFINITY;
    uint32_t used = 0;
    for (int u = 0; u < kCols / 8; ++u) {
      const int j = part + 8 * u;
      s[u] = -INFINITY;
      if (i < a.q_len && takes_part(a, b, h, i, j0 + j, n)) {
        s[u] = a.scale * dot_rows(t.a + row * kPitch, t.x + j * kPitch, d);
        used |= 1u << j;
      }
      most = fmaxf(most, s[u]);
    }
    atomicOr(&t.used, used);
    float* p = t.p + row * (kCols + 1);
    if (!kGrad) {
      for (int m = 4; m; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, m));
      const float next = fmaxf(top, most), base = next == -INFINITY ? 0.f : next;
      const float shrink = expf(top - base);
      sum *= shrink;
      for (float& v : acc) v *= shrink;
      top = next;
      for (int u = 0; u < kCols / 8; ++u) {
        const bool on = (used >> (part + 8 * u)) & 1u;
        const float e = on ? expf(s[u] - base) : 0.f;
        sum += e;
        p[part + 8 * u] = e;
      }
    } else {
      for (int u = 0; u < kCols / 8; ++u) {
        const int j = part + 8 * u;
        const bool on = (used >> j) & 1u;
        p[j] = on ? expf(s[u] - lse) * (dot_rows(t.b + row * kPitch, t.y + j * kPitch, d) - delta)
                  : 0.f;
      }
    }
    __syncthreads();
    clear_unused(t.x, t.y, &t.used, d);
    __syncthreads();
    const float* z = kGrad ? t.x : t.y;
    for (int u = 0; part + 8 * u < d; ++u)
      for (int j = 0; j < kCols; ++j) acc[u] = fmaf(p[j], z[j * kPitch + part + 8 * u], acc[u]);
  }
  if (!kGrad)
    for (int m = 4; m; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
  if (i >= a.q_len) return;
  const float end = kGrad ? a.scale : (sum > 0.f || sum != sum ? 1.f / sum : 0.f);
  void* dst = kGrad ? a.dq : a.out_w;
  const long long* s = kGrad ? a.dqs : a.os;
  for (int u = 0; part + 8 * u < d; ++u)
    put(dst, b * s[0] + i * s[1] + h * s[2] + part + 8 * u, dt, acc[u] * end);
  if (!kGrad && a.lse && part == 0) a.lse[lse_at] = sum == 0.f ? -INFINITY : top + logf(sum);
}

__global__ void __launch_bounds__(kThreadsS) attn_simple_key_kernel(const AttnShape a) {
  extern __shared__ float raw[];
  Tiles& t = *reinterpret_cast<Tiles*>(raw);
  const int d = a.head_dim, dt = a.dtype;
  const int g = blockIdx.y % a.kv_heads, b = blockIdx.y / a.kv_heads;
  const int j0 = blockIdx.x * kRows;
  const int row = threadIdx.x >> 3, part = threadIdx.x & 7, j = j0 + row;
  grid_dependency_wait();
  const int n = valid_keys(a, b);
  load_tile(t.a, a.k, a.ks, b, g, j0, kRows, n, d, dt);
  load_tile(t.b, a.v, a.vs, b, g, j0, kRows, n, d, dt);
  float dk[kMaxD / 8], dv[kMaxD / 8];
  for (float& v : dk) v = 0.f;
  for (float& v : dv) v = 0.f;
  if (j0 < n) {
    for (int h = g * a.group; h < (g + 1) * a.group; ++h) {
      for (int i0 = 0; i0 < a.q_len; i0 += kCols) {
        __syncthreads();
        load_tile(t.x, a.q, a.qs, b, h, i0, kCols, a.q_len, d, dt);
        load_tile(t.y, a.dout, a.dos, b, h, i0, kCols, a.q_len, d, dt);
        if (threadIdx.x == 0) t.used = 0;
        __syncthreads();
        if (threadIdx.x < kCols) {
          const int i = i0 + threadIdx.x;
          t.lse[threadIdx.x] =
              i < a.q_len ? a.lse[(static_cast<long long>(b) * a.heads + h) * a.q_len + i]
                          : -INFINITY;
          float delta = 0.f;
          if (i < a.q_len)
            for (int c = 0; c < d; ++c)
              delta = fmaf(t.y[threadIdx.x * kPitch + c],
                           get(a.out, b * a.os[0] + i * a.os[1] + h * a.os[2] + c, dt), delta);
          t.delta[threadIdx.x] = delta;
        }
        __syncthreads();
        float* p = t.p + row * (kCols + 1);
        float* ds = t.ds + row * (kCols + 1);
        uint32_t used = 0;
        for (int u = 0; u < kCols / 8; ++u) {
          const int c = part + 8 * u;
          p[c] = ds[c] = 0.f;
          if (t.lse[c] == -INFINITY) continue;
          used |= 1u << c;  // the query attends some key: its row is finite
          if (!takes_part(a, b, h, i0 + c, j, n)) continue;
          p[c] = expf(a.scale * dot_rows(t.a + row * kPitch, t.x + c * kPitch, d) - t.lse[c]);
          ds[c] = p[c] * (dot_rows(t.b + row * kPitch, t.y + c * kPitch, d) - t.delta[c]);
        }
        atomicOr(&t.used, used);
        __syncthreads();
        clear_unused(t.x, t.y, &t.used, d);
        __syncthreads();
        for (int u = 0; part + 8 * u < d; ++u)
          for (int c = 0; c < kCols; ++c) {
            dv[u] = fmaf(p[c], t.y[c * kPitch + part + 8 * u], dv[u]);
            dk[u] = fmaf(ds[c], t.x[c * kPitch + part + 8 * u], dk[u]);
          }
      }
    }
  }
  if (j >= a.kv_len) return;
  for (int u = 0; part + 8 * u < d; ++u) {
    const int c = part + 8 * u;
    put(a.dk, b * a.dks[0] + j * a.dks[1] + g * a.dks[2] + c, dt, j < n ? dk[u] * a.scale : 0.f);
    put(a.dv, b * a.dvs[0] + j * a.dvs[1] + g * a.dvs[2] + c, dt, j < n ? dv[u] : 0.f);
  }
}

template <typename K>
cudaError_t launch_tiles(K kernel, dim3 grid, const AttnShape& a, cudaStream_t stream) {
  if (grid.x == 0 || grid.y == 0) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(Tiles)));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, grid, dim3(kThreadsS), sizeof(Tiles), stream, a);
}

}  // namespace

cudaError_t launch_attn_simple_fwd(const AttnShape& a, cudaStream_t stream) {
  return launch_tiles(attn_simple_query_kernel<false>,
                      dim3((a.q_len + kRows - 1) / kRows, a.batch * a.heads), a, stream);
}

cudaError_t launch_attn_simple_bwd(const AttnShape& a, cudaStream_t stream) {
  cudaError_t e = launch_tiles(attn_simple_query_kernel<true>,
                               dim3((a.q_len + kRows - 1) / kRows, a.batch * a.heads), a, stream);
  if (e != cudaSuccess) return e;
  return launch_tiles(attn_simple_key_kernel,
                      dim3((a.kv_len + kRows - 1) / kRows, a.batch * a.kv_heads), a, stream);
}

}  // namespace convgb300
