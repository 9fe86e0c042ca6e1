// Writing the paged 8-bit cache and reading it back, and their C entry points.
//
// A row of D elements becomes D e4m3 codes and one byte, the exponent of a
// power-of-two scale.  e4m3 has a mantissa of its own for every element, so a
// finer scale would not make the rounding finer (2^-4 of an element either
// way); with a power of two the scaling is exact, the codes are the same
// whatever width it is computed in, and attention can add exponents where it
// would multiply.
//
// Bound by memory: 2 D bytes in and D + 1 out for each row, or the other way.
// Measured: 16 x up to 4096 tokens of 8 heads x 128 written in 55.7 us (5.5
// TB/s; 65.7 with the largest element found in fp32); 12 x up to 3001 of 4 heads
// x 80 read back in 14.5 us (3.7 TB/s, a third of it start and end).
// A lane takes 16 elements (two 16-byte words in, one out), the lanes of a row
// (a power of two, D / 16 of them at work) find its largest element with
// shuffles, and the key and the value of a token and head go together, so that
// their exponents leave in one store.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cache_common.cuh"

namespace convgb300 {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 2;  // in flight for each lane (four: 19 us to read back what two do in 14)

struct CacheParams {
  CacheView c;
  uint16_t *k, *v;
  const int *starts, *lengths;
  long long ks[3], vs[3];  // of k and v: batch, token, head
  int length, rows, lanes;  // rows: batch * length * kv_heads
  FastDiv div_length, div_heads;
};

__device__ __forceinline__ float magnitude(float x) {
  x = fabsf(x);
  return x < INFINITY ? x : 0.f;  // (not for infinities and NaN)
}

__device__ __forceinline__ float2 both(uint32_t v, __nv_bfloat16) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float2 both(uint32_t v, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// The byte of a row whose largest element is `top`: top = m 2^k, 1 <= m < 2,
// fits 448 = 1.75 2^8 with the exponent k - 8, or k - 7 where m > 1.75.  (No less
// than -64: attention divides its sums of probabilities by values' scales.)
__device__ __forceinline__ uint32_t scale_byte(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return top == 0.f ? 127u : static_cast<uint32_t>(max(e, 127 - 64));
}

// A row: request, token, head, and whether it is taken at all.
struct Row {
  int b, i, head;
  bool taken;
};
__device__ __forceinline__ Row row_of(const CacheParams& p, long long row) {
  Row o{0, 0, 0, false};
  if (row >= p.rows) return o;
  const int token = fast_div(static_cast<int>(row), p.div_heads);
  o.head = static_cast<int>(row) - token * static_cast<int>(p.div_heads.d);
  o.b = fast_div(token, p.div_length);
  o.i = token - o.b * static_cast<int>(p.div_length.d);
  o.taken = !p.lengths || o.i < p.lengths[o.b];
  return o;
}
// Where the token goes: page and offset, or page -1.
__device__ __forceinline__ int2 place_of(const CacheParams& p, const Row& o) {
  const long long at = (p.starts ? static_cast<long long>(p.starts[o.b]) : 0ll) + o.i;
  if (!o.taken || at < 0 || at >= static_cast<long long>(p.c.table_width) * p.c.page_size)
    return make_int2(-1, 0);
  const int index = fast_div(static_cast<int>(at), p.c.div_page);
  return make_int2(page_of(p.c, o.b, index), static_cast<int>(at) - index * p.c.page_size);
}

template <typename T>
__device__ __forceinline__ uint4 quantise(const uint4 (&raw)[2], uint32_t byte) {
  const float f = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte)
  const uint64_t ff = pack2(f, f);
  const uint32_t u[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t code[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 a = both(u[2 * i + j], T());
      float x, y;
      unpack2(mul2(pack2(a.x, a.y), ff), x, y);
      code[j] = round_codes(x, y);
    }
    w[i] = code[0] | (static_cast<uint32_t>(code[1]) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The larger magnitudes of two pairs of numbers; NaN only where both are.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return r;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, __half) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return r;
}
// The largest element of a lane's sixteen: among them infinities, or the finite ones.
template <typename T>
__device__ __forceinline__ float largest_of(const uint4 (&raw)[2]) {
  const T t{};
  const uint32_t a = larger(larger(raw[0].x, raw[0].y, t), larger(raw[0].z, raw[0].w, t), t);
  const uint32_t b = larger(larger(raw[1].x, raw[1].y, t), larger(raw[1].z, raw[1].w, t), t);
  const float2 f = both(larger(a, b, t), t);
  return fmaxf(fmaxf(f.x, f.y), 0.f);  // (0 for NaN)
}
template <typename T>
__device__ __forceinline__ float largest_finite_of(const uint4 (&raw)[2]) {
  const uint32_t u[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 a = both(u[i], T());
    top = fmaxf(top, fmaxf(magnitude(a.x), magnitude(a.y)));
  }
  return top;
}

template <typename T>
__global__ void __launch_bounds__(kCacheThreads)
    kv_cache_write_kernel(const __grid_constant__ CacheParams p) {
  const int at = threadIdx.x & (p.lanes - 1);
  const int groups = kCacheThreads / p.lanes;
  grid_dependency_wait();
  grid_launch_dependents();
  const long long step = static_cast<long long>(gridDim.x) * groups;
  const bool lane_on = at * 16 < p.c.head_dim;
  for (long long row0 = static_cast<long long>(blockIdx.x) * groups; row0 < p.rows; row0 += kCacheRows * step) {
    // (The elements are asked for before the page, which takes two loads that depend on one another.)
    Row o[kCacheRows];
    uint4 k[kCacheRows][2], v[kCacheRows][2];
    int2 place[kCacheRows];
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
      o[u] = row_of(p, row0 + u * step + threadIdx.x / p.lanes);
      k[u][0] = k[u][1] = v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      if (o[u].taken && lane_on) {
        const uint4* kp =
            reinterpret_cast<const uint4*>(p.k + o[u].b * p.ks[0] + o[u].i * p.ks[1] + o[u].head * p.ks[2]) + 2 * at;
        const uint4* vp =
            reinterpret_cast<const uint4*>(p.v + o[u].b * p.vs[0] + o[u].i * p.vs[1] + o[u].head * p.vs[2]) + 2 * at;
        k[u][0] = kp[0];
        k[u][1] = kp[1];
        v[u][0] = vp[0];
        v[u][1] = vp[1];
      }
    }
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) place[u] = place_of(p, o[u]);
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
      float kt = largest_of<T>(k[u]), vt = largest_of<T>(v[u]);
      if (__any_sync(0xFFFFFFFFu, fmaxf(kt, vt) == INFINITY)) {
        kt = largest_finite_of<T>(k[u]);
        vt = largest_finite_of<T>(v[u]);
      }
      for (int s = p.lanes >> 1; s > 0; s >>= 1) {
        kt = fmaxf(kt, __shfl_xor_sync(0xFFFFFFFFu, kt, s));
        vt = fmaxf(vt, __shfl_xor_sync(0xFFFFFFFFu, vt, s));
      }
      const int page = place[u].x, offset = place[u].y;
      if (page < 0 || !lane_on) continue;
      const uint32_t kb = scale_byte(kt), vb = scale_byte(vt);
      *reinterpret_cast<uint4*>(p.c.k + page * p.c.ks[0] + offset * p.c.ks[1] + o[u].head * p.c.ks[2] + at * 16) =
          quantise<T>(k[u], kb);
      *reinterpret_cast<uint4*>(p.c.v + page * p.c.vs[0] + offset * p.c.vs[1] + o[u].head * p.c.vs[2] + at * 16) =
          quantise<T>(v[u], vb);
      if (at == 0)
        *reinterpret_cast<uint16_t*>(p.c.scales + scale_at(p.c, page, o[u].head, offset)) =
            static_cast<uint16_t>(kb | (vb << 8));
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kCacheThreads)
    kv_cache_read_kernel(const __grid_constant__ CacheParams p) {
  const int at = threadIdx.x & (p.lanes - 1);
  const int groups = kCacheThreads / p.lanes;
  grid_dependency_wait();
  grid_launch_dependents();
  if (at * 16 >= p.c.head_dim) return;
  const long long step = static_cast<long long>(gridDim.x) * groups;
  for (long long row0 = static_cast<long long>(blockIdx.x) * groups; row0 < p.rows; row0 += kCacheRows * step) {
    Row o[kCacheRows];
    int2 place[kCacheRows];
    uint4 k[kCacheRows], v[kCacheRows];
    uint32_t bytes[kCacheRows];
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
      o[u] = row_of(p, row0 + u * step + threadIdx.x / p.lanes);
      place[u] = place_of(p, o[u]);
    }
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
      const int page = place[u].x, offset = place[u].y;
      k[u] = v[u] = make_uint4(0, 0, 0, 0);
      bytes[u] = 0;
      if (page >= 0) {
        k[u] = *reinterpret_cast<const uint4*>(p.c.k + page * p.c.ks[0] + offset * p.c.ks[1] +
                                               o[u].head * p.c.ks[2] + at * 16);
        v[u] = *reinterpret_cast<const uint4*>(p.c.v + page * p.c.vs[0] + offset * p.c.vs[1] +
                                               o[u].head * p.c.vs[2] + at * 16);
        bytes[u] = *reinterpret_cast<const uint16_t*>(p.c.scales + scale_at(p.c, page, o[u].head, offset));
      }
    }
#pragma unroll
    for (int u = 0; u < kCacheRows; ++u) {
      if (!o[u].taken) continue;
      if ((bytes[u] & 0xFFu) == 0) {  // nothing was written there
        k[u] = v[u] = make_uint4(0, 0, 0, 0);
        bytes[u] = 0;
      }
      uint4* ko = reinterpret_cast<uint4*>(p.k + o[u].b * p.ks[0] + o[u].i * p.ks[1] + o[u].head * p.ks[2]) + 2 * at;
      uint4* vo = reinterpret_cast<uint4*>(p.v + o[u].b * p.vs[0] + o[u].i * p.vs[1] + o[u].head * p.vs[2]) + 2 * at;
      restore<T>(k[u], bytes[u] & 0xFFu, ko[0], ko[1]);
      restore<T>(v[u], bytes[u] >> 8, vo[0], vo[1]);
    }
  }
}

bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

conv_status_t cache_run(const kv_cache_args_t* args, bool write, cudaStream_t stream) {
  if (!args) return CONV_ERR_INVALID_VALUE;
  const kv_cache_args_t& a = *args;
  if (a.dtype != CONV_DTYPE_BF16 && a.dtype != CONV_DTYPE_F16) return CONV_ERR_NOT_SUPPORTED;
  if (a.batch < 0 || a.length < 0) return CONV_ERR_INVALID_VALUE;
  const bool rows = a.batch > 0 && a.length > 0;
  CacheParams p{};
  conv_status_t st = take_cache(a.batch, a.kv_heads, a.head_dim, a.pages, a.page_size, a.table_width,
                                a.table_stride, a.k_cache, a.v_cache, a.scales, a.block_table,
                                a.k_cache_stride, a.v_cache_stride, write, rows, &p.c);
  if (st != CONV_OK) return st;
  if (rows && (!a.k || !a.v)) return CONV_ERR_INVALID_VALUE;
  if (off(a.k, 16) || off(a.v, 16) || off(a.starts, 4) || off(a.lengths, 4)) return CONV_ERR_MISALIGNED;
  st = take_row_strides(a.k_stride, a.batch, a.length, a.kv_heads, !write, p.ks);
  if (st == CONV_OK) st = take_row_strides(a.v_stride, a.batch, a.length, a.kv_heads, !write, p.vs);
  if (st != CONV_OK) return st;
  if (!rows) return CONV_OK;
  if (static_cast<long long>(a.batch) * a.length > kMaxCacheRows / a.kv_heads) return CONV_ERR_NOT_SUPPORTED;
  p.k = static_cast<uint16_t*>(a.k);
  p.v = static_cast<uint16_t*>(a.v);
  p.starts = a.starts;
  p.lengths = a.lengths;
  p.length = a.length;
  p.rows = a.batch * a.length * a.kv_heads;
  p.lanes = 1;
  while (p.lanes * 16 < a.head_dim) p.lanes <<= 1;
  p.div_length = make_fast_div(static_cast<uint32_t>(a.length));
  p.div_heads = make_fast_div(static_cast<uint32_t>(a.kv_heads));
  const int sms = attn_sm_count();
  if (sms <= 0) return CONV_ERR_CUDA;
  const long long groups = kCacheThreads / p.lanes;
  const dim3 grid(static_cast<unsigned>(std::min<long long>((p.rows + groups - 1) / groups, 16ll * sms)));
  const auto kernel = a.dtype == CONV_DTYPE_BF16
                          ? (write ? kv_cache_write_kernel<__nv_bfloat16> : kv_cache_read_kernel<__nv_bfloat16>)
                          : (write ? kv_cache_write_kernel<__half> : kv_cache_read_kernel<__half>);
  return launch_pdl(kernel, grid, dim3(kCacheThreads), 0, stream, p) == cudaSuccess ? CONV_OK
                                                                                   : CONV_ERR_CUDA;
}

}  // namespace

conv_status_t take_row_strides(const long long in[3], int batch, int length, int heads, bool output,
                               long long out[3]) {
  const int extent[3] = {batch, length, heads};
  for (int i = 0; i < 3; ++i) {
    out[i] = extent[i] > 1 ? in[i] : 0;
    if (extent[i] > 1 && (in[i] < 0 || (in[i] == 0 && output))) return CONV_ERR_INVALID_VALUE;
    if (out[i] % 8 != 0) return CONV_ERR_MISALIGNED;
    if (out[i] >= 1ll << 40) return CONV_ERR_NOT_SUPPORTED;
  }
  return CONV_OK;
}

conv_status_t take_cache(int batch, int kv_heads, int head_dim, int pages, int page_size,
                         int table_width, long long table_stride, const void* k, const void* v,
                         const void* scales, const int* table, const long long ks[3],
                         const long long vs[3], bool written, bool needed, CacheView* out) {
  if (kv_heads <= 0 || head_dim <= 0 || pages < 0 || page_size <= 0 || table_width < 0)
    return CONV_ERR_INVALID_VALUE;
  if (head_dim % 16 != 0 || head_dim > 128 || page_size % 16 != 0) return CONV_ERR_NOT_SUPPORTED;
  if (static_cast<long long>(table_width) * page_size > kMaxCacheRows) return CONV_ERR_NOT_SUPPORTED;
  if (needed && (pages == 0 || !k || !v || !scales || (table_width > 0 && !table)))
    return CONV_ERR_INVALID_VALUE;
  if (batch > 1 && table_stride < 0) return CONV_ERR_INVALID_VALUE;
  if (off(k, 16) || off(v, 16) || off(scales, 16) || off(table, 4)) return CONV_ERR_MISALIGNED;
  const int extent[3] = {pages, page_size, kv_heads};
  for (int i = 0; i < 3; ++i) {
    const long long s[2] = {extent[i] > 1 ? ks[i] : 0, extent[i] > 1 ? vs[i] : 0};
    for (const long long x : s) {
      if (extent[i] > 1 && (x < 0 || (x == 0 && written))) return CONV_ERR_INVALID_VALUE;
      if (x % 16 != 0) return CONV_ERR_MISALIGNED;
      if (x >= 1ll << 40) return CONV_ERR_NOT_SUPPORTED;
    }
    out->ks[i] = s[0];
    out->vs[i] = s[1];
  }
  out->k = static_cast<uint8_t*>(const_cast<void*>(k));
  out->v = static_cast<uint8_t*>(const_cast<void*>(v));
  out->scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  out->table = table;
  out->table_stride = batch > 1 ? table_stride : 0;
  out->pages = pages;
  out->page_size = page_size;
  out->table_width = table_width;
  out->kv_heads = kv_heads;
  out->head_dim = head_dim;
  out->div_page = make_fast_div(static_cast<uint32_t>(page_size));
  return CONV_OK;
}

}  // namespace convgb300

extern "C" {

conv_status_t kv_cache_write(const kv_cache_args_t* args, void* stream) {
  return convgb300::cache_run(args, true, static_cast<cudaStream_t>(stream));
}

conv_status_t kv_cache_read(const kv_cache_args_t* args, void* stream) {
  return convgb300::cache_run(args, false, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
