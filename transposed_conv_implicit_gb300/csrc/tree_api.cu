// Tree attention, host side: argument checks, plan, workspace layout and the C
// entry points of include/conv_gb300_decoder.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "tree_params.h"

namespace convgb300 {

namespace {

// Rows of a key head up to which the kernel for few rows takes them (in tiles of 32, which read
// the keys once each).  Its time and the other kernel's: 48 rows, 2 requests x 8192 keys 38 and 45
// us, 32 x 4096 160 and 155; 64 rows, 32 x 2048 101 and 108; 96 rows, 16 x 4096 131 and 95.
constexpr int kFewRows = 64;

struct TreePlan {
  bool many;
  int tile_rows, max_tiles, grid;
  size_t part_bytes;
};

conv_status_t check_sizes(const tree_attention_args_t& a) {
  if (a.dtype != CONV_DTYPE_BF16 && a.dtype != CONV_DTYPE_F16) return CONV_ERR_NOT_SUPPORTED;
  if (a.batch < 0 || a.q_len < 0 || a.heads <= 0 || a.kv_heads <= 0 || a.heads % a.kv_heads != 0 ||
      a.head_dim <= 0 || a.page_size <= 0 || a.table_width < 0)
    return CONV_ERR_INVALID_VALUE;
  if (a.head_dim % 16 != 0 || a.head_dim > 128 || a.page_size % 16 != 0 || a.q_len > kMaxDrafts ||
      static_cast<long long>(a.table_width) * a.page_size > kMaxCacheRows ||
      static_cast<long long>(a.batch) * std::max(1, a.q_len) > kMaxCacheRows / a.heads)
    return CONV_ERR_NOT_SUPPORTED;
  return CONV_OK;
}

TreePlan plan(const tree_attention_args_t& a, int sms) {
  TreePlan f{};
  const int rows = a.q_len * (a.heads / a.kv_heads);
  f.many = rows > kFewRows;
  f.tile_rows = f.many ? kTreeManyRows : rows <= 16 ? 16 : 32;
  f.max_tiles = std::max(1, (rows + f.tile_rows - 1) / f.tile_rows);
  const long long key_tiles =
      (static_cast<long long>(a.table_width) * a.page_size + kTreeKeys - 1) / kTreeKeys;
  const long long items = static_cast<long long>(a.batch) * a.kv_heads * f.max_tiles;
  const long long most = static_cast<long long>(f.many ? 1 : tree_few_ctas(f.tile_rows)) * sms;
  // (More items than CTAs by far: their steps are as many at least.)
  f.grid = static_cast<int>(items >= most ? most : std::min(most, items * std::max(1ll, key_tiles)));
  if (key_tiles > 1)
    f.part_bytes = static_cast<size_t>(2) * f.grid * f.tile_rows * (128 + 2) * sizeof(float);
  return f;
}

size_t workspace_bytes_of(const TreePlan& f) { return CONV_STATUS_BYTES + f.part_bytes; }

bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

conv_status_t run(const tree_attention_args_t* args, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
  if (!args) return CONV_ERR_INVALID_VALUE;
  const tree_attention_args_t& a = *args;
  conv_status_t st = check_sizes(a);
  if (st != CONV_OK) return st;
  if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return CONV_ERR_INVALID_VALUE;
  const bool rows = a.batch > 0 && a.q_len > 0;
  TreeParams p{};
  st = take_cache(a.batch, a.kv_heads, a.head_dim, a.pages, a.page_size, a.table_width, a.table_stride,
                  a.k_cache, a.v_cache, a.scales, a.block_table, a.k_cache_stride, a.v_cache_stride,
                  false, rows, &p.c);
  if (st != CONV_OK) return st;
  if (rows && (!a.q || !a.out || !a.kv_lengths)) return CONV_ERR_INVALID_VALUE;
  if (a.parents && a.batch > 1 && a.parent_stride < 0) return CONV_ERR_INVALID_VALUE;
  if (off(a.q, 16) || off(a.out, 16) || off(a.lse, 4) || off(a.kv_lengths, 4) ||
      off(a.draft_lengths, 4) || off(a.parents, 4))
    return CONV_ERR_MISALIGNED;
  st = take_row_strides(a.q_stride, a.batch, a.q_len, a.heads, false, p.qs);
  if (st == CONV_OK) st = take_row_strides(a.out_stride, a.batch, a.q_len, a.heads, true, p.os);
  if (st != CONV_OK) return st;
  if (!workspace) return CONV_ERR_INVALID_VALUE;
  if (off(workspace, 16)) return CONV_ERR_MISALIGNED;
  const int sms = attn_sm_count();
  if (sms <= 0) return CONV_ERR_CUDA;
  const TreePlan f = plan(a, sms);
  if (workspace_bytes < workspace_bytes_of(f)) return CONV_ERR_WORKSPACE_TOO_SMALL;
  if (!rows || a.table_width == 0) return CONV_OK;  // (without a table there are no drafts)
  p.q = static_cast<const uint16_t*>(a.q);
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.kv_lengths = a.kv_lengths;
  p.draft_lengths = a.draft_lengths;
  p.parents = a.parents;
  p.parent_stride = a.batch > 1 ? a.parent_stride : 0;
  p.batch = a.batch;
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.group = a.heads / a.kv_heads;
  p.q_len = a.q_len;
  p.tile_rows = f.tile_rows;
  p.max_tiles = f.max_tiles;
  p.scale_log2 = a.scale * 1.44269504088896341f;
  p.div_group = make_fast_div(static_cast<uint32_t>(p.group));
  p.div_slices = make_fast_div(static_cast<uint32_t>(a.page_size / 16));
  p.ks8 = 8 * p.c.ks[1];
  p.vs8 = 8 * p.c.vs[1];
  p.scale_page = 2ll * a.kv_heads * a.page_size;
  p.part_out = reinterpret_cast<float*>(static_cast<char*>(workspace) + CONV_STATUS_BYTES);
  p.part_stat = p.part_out + static_cast<size_t>(2) * f.grid * f.tile_rows * 128;
  p.many = f.many;
  p.status = static_cast<unsigned int*>(workspace);
  p.timeout_cycles = wait_limit_cycles();
  p.fault_mode = wait_fault_mode();
  const cudaError_t err = f.many ? launch_tree_many(p, a.dtype, f.grid, stream)
                                 : launch_tree_few(p, a.dtype, f.grid, stream);
  if (err != cudaSuccess) return CONV_ERR_CUDA;
  if (f.part_bytes && launch_tree_join(p, a.dtype, f.grid, stream) != cudaSuccess) return CONV_ERR_CUDA;
  return CONV_OK;
}

}  // namespace

}  // namespace convgb300

extern "C" {

size_t tree_attention_workspace_size(const tree_attention_args_t* args) {
  using namespace convgb300;
  if (!args || check_sizes(*args) != CONV_OK) return 0;
  const int sms = attn_sm_count();
  if (sms <= 0) return 0;
  return workspace_bytes_of(plan(*args, sms));
}

conv_status_t tree_attention_fwd(const tree_attention_args_t* args, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  return convgb300::run(args, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
