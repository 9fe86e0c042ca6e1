// The paged 8-bit cache, as its kernels see it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "../../include/conv_gb300_decoder.h"
#include "attn_common.cuh"
#include "attn_internal.h"
#include "conv_params.h"

namespace convgb300 {

// Pages and the table that lists them.  Strides in bytes: {page, token, head}.
struct CacheView {
  uint8_t *k, *v, *scales;
  const int* table;
  long long table_stride;
  long long ks[3], vs[3];
  int pages, page_size, table_width, kv_heads, head_dim;
  FastDiv div_page;  // by tokens of a page
};

// The page of a token that the table covers, or -1.
__device__ __forceinline__ int page_of(const CacheView& c, int b, int index) {
  const int page = c.table[b * c.table_stride + index];
  return static_cast<unsigned int>(page) < static_cast<unsigned int>(c.pages) ? page : -1;
}

__device__ __forceinline__ long long scale_at(const CacheView& c, int page, int head, int offset) {
  return ((static_cast<long long>(page) * c.kv_heads + head) * c.page_size + offset) * 2;
}

// Two e4m3 codes as fp16 (exact).
__device__ __forceinline__ uint32_t widen_codes(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
// Four codes: {0, 1} and {2, 3}.
__device__ __forceinline__ void widen_codes4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
// Two numbers as e4m3 codes (a in the lower byte): nearest, ties to even, limited to 448.
__device__ __forceinline__ uint16_t round_codes(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Sixteen codes times 2^(byte - 127) (0 for rows that were never written),
// rounded to T and limited to its numbers.
template <typename T>
__device__ __forceinline__ void restore(uint4 codes, uint32_t byte, uint4& first, uint4& second) {
  constexpr bool kHalf = std::is_same<T, __half>::value;
  const float f = __uint_as_float(byte << 23);
  const uint64_t ff = pack2(f, f);
  const uint32_t u[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t w[8];
  auto each = [&](auto rounded) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2];
      widen_codes4(u[i], h[0], h[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        float x, y;
        unpack2(mul2(pack2(a.x, a.y), ff), x, y);
        w[2 * i + j] = rounded(x, y);
      }
    }
  };
  // Codes up to 448 can pass the largest number from these scales on (bfloat16's, by a row that
  // was rounded up).  NaN stays.
  if (byte < (kHalf ? 127u + 8u : 127u + 120u)) {
    each([](float x, float y) { return round2<T>(x, y); });
  } else {
    each([](float x, float y) {
      constexpr float kMost = kHalf ? 65504.f : 0x1.FEp127f;
      return round2<T>(x > kMost ? kMost : x < -kMost ? -kMost : x, y > kMost ? kMost : y < -kMost ? -kMost : y);
    });
  }
  first = make_uint4(w[0], w[1], w[2], w[3]);
  second = make_uint4(w[4], w[5], w[6], w[7]);
}

// Sizes, pages and strides that writing, reading and attention check alike;
// fills the view.  `written`: the cache may not repeat a row.
conv_status_t take_cache(int batch, int kv_heads, int head_dim, int pages, int page_size,
                         int table_width, long long table_stride, const void* k, const void* v,
                         const void* scales, const int* table, const long long ks[3],
                         const long long vs[3], bool written, bool needed, CacheView* out);

// {batch, token, head} strides of a 16-bit tensor (see take_strides).
conv_status_t take_row_strides(const long long in[3], int batch, int length, int heads, bool output,
                               long long out[3]);

constexpr long long kMaxCacheRows = 0x7FFF0000ll;

}  // namespace convgb300
