// The paged 8-bit cache, as its kernels see it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/conv_gb300_decoder.h"
#include "attn_internal.h"
#include "attn_ptx.cuh"
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
