// Launch parameters shared by the tree attention's entry points and kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cache_common.cuh"

namespace convgb300 {

constexpr int kMaxDrafts = 256;            // of a request
constexpr int kTreeWords = kMaxDrafts / 32;
constexpr int kTreeKeys = 128;             // keys of a step: what a share of the work counts

// Rows of a key head: (draft, query head of the group), the draft's heads side
// by side.  A row tile holds tile_rows of them.  An item is a row tile of a key
// head of a request, steps are its tiles of kTreeKeys keys; the sequence of all
// items' steps is cut evenly between the CTAs.
struct TreeParams {
  CacheView c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int *kv_lengths, *draft_lengths, *parents;
  long long parent_stride;
  long long qs[3], os[3];  // batch, token, head
  int batch, heads, kv_heads, group, q_len;
  int tile_rows;
  float scale_log2;        // scale * log2(e)
  FastDiv div_group;
  FastDiv div_slices;      // by slices of 16 keys of a page
  long long ks8, vs8;      // eight tokens on in the cache
  long long scale_page;    // bytes of a page's scales
  // Rows whose keys are shared out: [2 * CTAs][tile_rows][128] unnormalised,
  // and their maximum (log2 units) and sum.  A share that begins in the middle
  // of an item leaves its rows in slot 2 c, one that begins with it in 2 c + 1:
  // there is one of either at most, since items that a CTA has whole are
  // written by it.
  float* part_out;
  float* part_stat;
  int max_tiles;           // most row tiles of a key head
  bool many;               // tree_many.cu: two shares, behind one another, of items of up to half a tile
  unsigned int* status;
  long long timeout_cycles;
  int fault_mode;          // test hook: 1 = every CTA with work leaves its first keys un-announced
};

// Few rows (tree_few.cu).
constexpr int kTreeFewWarps = 4;
int tree_few_ctas(int tile_rows);  // a SM
cudaError_t launch_tree_few(const TreeParams& p, int dtype, int grid, cudaStream_t stream);
// Many rows (tree_many.cu): one CTA a SM, row tiles of twice 128 rows.
constexpr int kTreeManyRows = 256;
cudaError_t launch_tree_many(const TreeParams& p, int dtype, int grid, cudaStream_t stream);
// Joins the shares of `ctas` CTAs.
cudaError_t launch_tree_join(const TreeParams& p, int dtype, int ctas, cudaStream_t stream);

}  // namespace convgb300
