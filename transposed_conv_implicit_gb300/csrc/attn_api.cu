// Cross attention, host side: argument checks, workspace layout and the C
// entry points of include/conv_gb300_attention.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/conv_gb300_attention.h"
#include "../../include/conv_gb300_testing.h"
#include "attn_internal.h"
#include "attn_params.h"

namespace convgb300 {


namespace {

constexpr int kMaxHeadDim = 128;

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Strides with those of dimensions of extent 1 cleared.  Outputs may not
// overlap themselves; no tensor repeats one token.
conv_status_t take_strides(const long long in[3], int batch, int length, int heads, bool output,
                           long long out[3]) {
  const int extent[3] = {batch, length, heads};
  for (int i = 0; i < 3; ++i) {
    out[i] = extent[i] > 1 ? in[i] : 0;
    if (extent[i] > 1 && (in[i] < 0 || (in[i] == 0 && (output || i == 1))))
      return CONV_ERR_INVALID_VALUE;
    if (out[i] % 8 != 0) return CONV_ERR_MISALIGNED;
  }
  return CONV_OK;
}

// Sizes and types, which the workspace size needs too.
conv_status_t check_sizes(const cross_attention_args_t& a) {
  if (a.dtype != CONV_DTYPE_BF16 && a.dtype != CONV_DTYPE_F16) return CONV_ERR_NOT_SUPPORTED;
  if (a.batch < 0 || a.q_len < 0 || a.kv_len < 0 || a.heads <= 0 || a.kv_heads <= 0 ||
      a.head_dim <= 0 || a.heads % a.kv_heads != 0)
    return CONV_ERR_INVALID_VALUE;
  if (a.head_dim % 8 != 0 || a.head_dim > kMaxHeadDim) return CONV_ERR_NOT_SUPPORTED;
  // Rows count in 31 bits (padded to whole tiles).
  const long long rows = (static_cast<long long>(a.q_len) + kAttnRows) * a.heads;
  const long long states = (static_cast<long long>(a.kv_len) + kAttnRows) * a.kv_heads;
  if (a.batch > 0 && std::max(rows, states) > 0x7FFFFFFFll / a.batch) return CONV_ERR_NOT_SUPPORTED;
  return CONV_OK;
}

// The packed mask's extents after broadcasting.
struct MaskShape {
  int batches, heads, queries, words, tiles;
  size_t bytes, any_bytes;
};

MaskShape mask_shape(const cross_attention_args_t& a) {
  MaskShape m{};
  if (!a.mask) return m;
  m.batches = a.mask_stride[0] == 0 ? 1 : a.batch;
  m.heads = a.mask_stride[1] == 0 ? 1 : a.heads;
  m.queries = a.mask_stride[2] == 0 ? 1 : a.q_len;
  m.words = (a.kv_len + 127) / 128 * 4;
  m.tiles = (m.queries + kAttnRows - 1) / kAttnRows;
  m.bytes = static_cast<size_t>(m.batches) * m.heads * m.queries * m.words * 4;
  m.any_bytes = static_cast<size_t>(m.batches) * m.heads * m.tiles * m.words * 4;
  return m;
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// ------------------------------------------------------------------ forward plan
// How the rows of one key head are cut into row tiles, and which schedule
// runs them (attn_fwd.cu).
struct FwdPlan {
  int tile_heads, tile_tokens, token_tiles, row_tiles;
  int kv_box;
  bool split;
  int one;               // one key tile: CTAs per SM of its kernel, or 0
  int grid;
  long long items;       // pairs: launch items
  size_t part_bytes;     // split: partial rows and their statistics
};

// Shared memory of the kernel for one tile of keys: two buffers of queries (and
// output), keys and values, barriers.
uint32_t one_bar_offset(int kv_box) { return 2 * 16384 + 2 * kv_box * 128; }
size_t one_smem(int kv_box) { return one_bar_offset(kv_box) + attn_one_bar_bytes(); }

FwdPlan plan_fwd(const cross_attention_args_t& a, int sms, bool may_pack) {
  FwdPlan f{};
  const int group = a.heads / a.kv_heads;
  const int token_tiles = (a.q_len + kAttnRows - 1) / kAttnRows;
  f.token_tiles = std::max(1, token_tiles);
  f.tile_heads = 1;
  f.tile_tokens = std::min(kAttnRows, std::max(1, a.q_len));
  long long row_tiles = static_cast<long long>(group) * f.token_tiles;
  // The query heads of a key head side by side, where that makes fewer tiles.
  if (may_pack && group > 1 && group <= kAttnRows) {
    const int tokens = kAttnRows / group;
    const int packed = (a.q_len + tokens - 1) / tokens;
    if (packed < row_tiles) {
      f.tile_heads = group;
      f.tile_tokens = std::min(tokens, std::max(1, a.q_len));
      row_tiles = std::max(1, packed);
    }
  }
  f.row_tiles = static_cast<int>(row_tiles);
  f.kv_box = std::min(kAttnRows, std::max(16, (a.kv_len + 15) / 16 * 16));
  const long long nt = std::max(1, (a.kv_len + f.kv_box - 1) / f.kv_box);
  const long long heads = static_cast<long long>(a.batch) * a.kv_heads;
  // One tile of keys, narrow heads, no mask: the kernel made for it (16 x 4096
  // x 8 heads x 40 against 77 keys: 31 us, 47 in pairs).  Four
  // CTAs per SM where scores and output fit in 128 TMEM columns, three of them
  // where shared memory (228 KB, 1 KB a CTA taken) has no room for a fourth: with
  // equal shares for more CTAs than run at once, some begin when others end (96
  // keys x 32: 24.5 us, with shares for four 34.9; 112 x 16: 28.8 and 38.6).
  if (a.kv_len > 0 && a.kv_len <= kAttnRows && a.head_dim <= 64 && !a.mask) {
    f.one = f.kv_box + (a.head_dim + 15) / 16 * 16 <= 128 ? 4 : 2;
    f.items = heads * row_tiles;
    const long long fit = std::min<long long>(f.one, 228 * 1024 / (one_smem(f.kv_box) + 1024));
    f.grid = static_cast<int>(std::min(f.items, fit * sms));
    return f;
  }
  f.items = heads * ((row_tiles + 1) / 2);
  // Pairs take whole rounds of items; split shares steps out evenly.  A
  // pair's step covers two row tiles on a whole SM.
  const long long rounds = (f.items + sms - 1) / sms;
  const double pairs_cost = static_cast<double>(rounds) * nt;
  // The join costs what 4 steps do.  Both sides, whole calls: one token of 64
  // requests x 32 heads x 128 against up to 4096 keys, 171 us as pairs and 141
  // split; 3 x 1021 x 12 heads x 80 against 1531, masked, 42 and 59; 2 x 16 heads,
  // 16384 x 4096 x 128, 774 and 963.
  const double split_cost = static_cast<double>(heads) * row_tiles * nt / (2.0 * sms) * 1.25 + (nt > 1 ? 4 : 0);
  f.split = split_cost < pairs_cost;
  const long long steps = heads * row_tiles * nt;
  f.grid = static_cast<int>(f.split ? std::min<long long>(steps, 2ll * sms)
                                    : std::min<long long>(f.items, sms));
  if (f.split && nt > 1)
    f.part_bytes = static_cast<size_t>(2) * f.grid * kAttnRows * (128 + 2) * sizeof(float);
  return f;
}

// ------------------------------------------------------------------ backward plan
// Rows that a warp of the rows kernel reads side by side: 16 bytes a lane, a power
// of two of lanes a row.
int row_slots(int head_dim) {
  int width = 1;
  while (width < head_dim / 8) width <<= 1;
  return 32 / width;
}

struct BwdPlan {
  int q_tiles, item_steps, kv_tiles;
  int q_grid, kv_grid;     // CTAs of the dq and the dk, dv kernel
  bool q_whole, kv_whole;  // no item is cut between CTAs
  int per_tile, key_groups;  // neighbouring rows whose norms are joined: of a tile of queries, of the keys
  bool brief;              // one tile of keys, narrow heads, no mask: one kernel
  size_t stat_bytes, row_norm_bytes, value_norm_bytes, part_q_bytes, part_kv_bytes;
};

BwdPlan plan_bwd(const cross_attention_args_t& a, const FwdPlan& f, int sms) {
  BwdPlan p{};
  p.q_tiles = (a.q_len + kAttnRows - 1) / kAttnRows;
  p.item_steps = a.heads / a.kv_heads * p.q_tiles;
  p.kv_tiles = (a.kv_len + kAttnRows - 1) / kAttnRows;
  const long long heads = static_cast<long long>(a.batch) * a.kv_heads;
  const long long nt = std::max(1, (a.kv_len + f.kv_box - 1) / f.kv_box);
  p.q_grid = static_cast<int>(std::min<long long>(heads * f.row_tiles * nt, sms));
  p.kv_grid = static_cast<int>(std::min<long long>(heads * p.kv_tiles * p.item_steps, sms));
  // Even shares cut items and join them, which costs about what kJoinSteps
  // steps do; whole items leave some CTAs idle at the end.  (2 x 1021 x 12
  // heads x 80 against 523, masked, the training pass: 107 us with dq's items
  // cut, 99 whole.)
  constexpr double kJoinSteps = 5;
  const auto whole = [sms](long long items, long long steps) {
    return static_cast<double>((items + sms - 1) / sms) * steps <=
           static_cast<double>(items) * steps / sms + (steps > 1 ? kJoinSteps : 0);
  };
  p.q_whole = whole(heads * f.row_tiles, nt);
  p.kv_whole = whole(heads * p.kv_tiles, p.item_steps) && !(f.one && a.q_len > 0);
  p.brief = f.one && a.q_len > 0;
  if (p.brief) p.kv_grid = static_cast<int>(std::min<long long>(heads * p.item_steps, sms));
  const int group = kAttnRowUnroll * row_slots(a.head_dim);
  p.per_tile = kAttnRows / group;
  p.key_groups = (a.kv_len + group - 1) / group;
  // (Of one size for both types; bf16 has no use for the norms.)
  p.stat_bytes = static_cast<size_t>(a.batch) * a.heads * p.q_tiles * 384 * sizeof(float);
  p.row_norm_bytes = static_cast<size_t>(a.batch) * a.heads * p.q_tiles * p.per_tile * sizeof(float);
  p.value_norm_bytes = static_cast<size_t>(heads) * p.key_groups * sizeof(float);
  const size_t tile = static_cast<size_t>(kAttnRows) * 128 * sizeof(float);
  p.part_q_bytes = nt > 1 && !p.q_whole ? 2 * tile * p.q_grid : 0;
  p.part_kv_bytes = p.item_steps > 1 && !p.kv_whole ? 4 * tile * p.kv_grid : 0;
  return p;
}

struct Layout {
  MaskShape mask;
  size_t mask_at, any_at, part_at, stat_at, row_norm_at, value_norm_at, part_q_at, part_kv_at, total;
};

Layout layout(const cross_attention_args_t& a, bool backward, const FwdPlan& f, const BwdPlan& g) {
  Layout l{};
  l.mask = mask_shape(a);
  l.mask_at = CONV_STATUS_BYTES;
  l.any_at = round_up(l.mask_at + l.mask.bytes, 256);
  l.part_at = round_up(l.any_at + l.mask.any_bytes, 256);
  if (!backward) {
    l.total = round_up(l.part_at + f.part_bytes, 256);
    return l;
  }
  l.stat_at = l.part_at;
  l.row_norm_at = round_up(l.stat_at + g.stat_bytes, 256);
  l.value_norm_at = round_up(l.row_norm_at + g.row_norm_bytes, 256);
  l.part_q_at = round_up(l.value_norm_at + g.value_norm_bytes, 256);
  l.part_kv_at = round_up(l.part_q_at + g.part_q_bytes, 256);
  l.total = round_up(l.part_kv_at + g.part_kv_bytes, 256);
  return l;
}

// {D, heads, tokens, batch} of a tensor with strides s (0: one entry, or a
// broadcast), rows of 64 elements, 128-byte swizzle.
conv_status_t encode_map(CUtensorMap* map, const void* base, const AttnShape& a, int heads,
                         int tokens, const long long s[3], int box_heads, int box_tokens) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tiled_map_encoder();
  if (!encode) return CONV_ERR_CUDA;
  const long long any = 16 * ((a.head_dim + 7) / 8);  // stride of a single entry: unused
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.head_dim),
                        static_cast<cuuint64_t>(s[2] ? heads : 1),
                        static_cast<cuuint64_t>(s[1] ? tokens : 1),
                        static_cast<cuuint64_t>(s[0] ? a.batch : 1)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(s[2] ? 2 * s[2] : any),
                           static_cast<cuuint64_t>(s[1] ? 2 * s[1] : any),
                           static_cast<cuuint64_t>(s[0] ? 2 * s[0] : any)};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens),
                       1};
  cuuint32_t step[4] = {1, 1, 1, 1};
  const CUresult r = encode(
      map,
      a.dtype == CONV_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
      4, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CONV_OK : CONV_ERR_CUDA;
}

conv_status_t run_fwd(const AttnShape& s, const FwdPlan& f, char* ws, const Layout& l,
                      cudaStream_t stream) {
  AttnFwdParams p{};
  p.a = s;
  p.tile_heads = f.tile_heads;
  p.tile_tokens = f.tile_tokens;
  p.token_tiles = f.token_tiles;
  p.row_tiles = f.row_tiles;
  p.div_pairs = make_fast_div(static_cast<uint32_t>(f.one ? f.row_tiles : (f.row_tiles + 1) / 2));
  p.div_kv_heads = make_fast_div(static_cast<uint32_t>(s.kv_heads));
  p.div_token_tiles = make_fast_div(static_cast<uint32_t>(f.token_tiles));
  p.kv_box = f.kv_box;
  p.items = f.items;
  p.item_rows = static_cast<long long>(s.kv_heads) * f.row_tiles;
  p.scale_log2 = s.scale * 1.44269504088896341f;
  conv_status_t st = encode_map(&p.map_q, s.q, s, s.heads, s.q_len, s.qs, f.tile_heads, f.tile_tokens);
  if (st == CONV_OK) st = encode_map(&p.map_k, s.k, s, s.kv_heads, s.kv_len, s.ks, 1, f.kv_box);
  if (st == CONV_OK) st = encode_map(&p.map_v, s.v, s, s.kv_heads, s.kv_len, s.vs, 1, f.kv_box);
  if (st == CONV_OK)
    st = encode_map(&p.map_out, s.out_w, s, s.heads, s.q_len, s.os, f.tile_heads, f.tile_tokens);
  if (st != CONV_OK) return st;
  p.q_mul[0] = s.qs[2] != 0;
  p.q_mul[1] = s.qs[0] != 0;
  p.k_mul[0] = s.ks[2] != 0;
  p.k_mul[1] = s.ks[0] != 0;
  p.v_mul[0] = s.vs[2] != 0;
  p.v_mul[1] = s.vs[0] != 0;
  p.status = reinterpret_cast<unsigned int*>(ws);
  p.timeout_cycles = wait_limit_cycles();
  p.fault_mode = wait_fault_mode();
  if (f.one) {
    p.off_q = 0;
    p.off_kv = 2 * 16384;
    p.off_bar = one_bar_offset(f.kv_box);
    return launch_attn_one(p, f.one, f.grid, one_smem(f.kv_box), stream) == cudaSuccess
               ? CONV_OK
               : CONV_ERR_CUDA;
  }
  // Shared memory: queries, the key/value ring, output staging, barriers.
  const bool wide = s.head_dim > 64;
  const uint32_t q_tile = wide ? 32768 : 16384, kv_tile = f.kv_box * (wide ? 256 : 128);
  const uint32_t ring = f.split ? (wide ? 65536 : 81920) : (wide ? 131072 : 98304);
  const int groups = f.split ? 1 : 2;
  p.q_stages = f.split || wide ? 1 : 2;
  p.stages = std::min<uint32_t>(8, ring / kv_tile);
  p.off_q = 0;
  p.off_kv = p.off_q + groups * p.q_stages * q_tile;
  p.off_out = p.off_kv + p.stages * kv_tile;
  p.off_bar = p.off_out + groups * 16384;
  const size_t smem = p.off_bar + attn_fwd_bar_bytes();
  if (f.split) {
    p.part_out = reinterpret_cast<float*>(ws + l.part_at);
    p.part_stat = p.part_out + static_cast<size_t>(2) * f.grid * kAttnRows * 128;
  }
  return launch_attn_fwd(p, f.split, f.grid, smem, stream) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

// The maps of q, do, k and v, and where they are broadcast.
conv_status_t encode_maps(AttnBwdParams* p, const AttnShape& s, int box_heads, int box_tokens,
                          int kv_box) {
  conv_status_t st = encode_map(&p->map_q, s.q, s, s.heads, s.q_len, s.qs, box_heads, box_tokens);
  if (st == CONV_OK)
    st = encode_map(&p->map_do, s.dout, s, s.heads, s.q_len, s.dos, box_heads, box_tokens);
  if (st == CONV_OK) st = encode_map(&p->map_k, s.k, s, s.kv_heads, s.kv_len, s.ks, 1, kv_box);
  if (st == CONV_OK) st = encode_map(&p->map_v, s.v, s, s.kv_heads, s.kv_len, s.vs, 1, kv_box);
  p->q_mul[0] = s.qs[2] != 0;
  p->q_mul[1] = s.qs[0] != 0;
  p->do_mul[0] = s.dos[2] != 0;
  p->do_mul[1] = s.dos[0] != 0;
  p->k_mul[0] = s.ks[2] != 0;
  p->k_mul[1] = s.ks[0] != 0;
  p->v_mul[0] = s.vs[2] != 0;
  p->v_mul[1] = s.vs[0] != 0;
  return st;
}

conv_status_t run_bwd(const AttnShape& s, const FwdPlan& f, const BwdPlan& g, char* ws,
                      const Layout& l, cudaStream_t stream) {
  AttnBwdParams p{};
  p.a = s;
  p.tile_heads = f.tile_heads;
  p.tile_tokens = f.tile_tokens;
  p.token_tiles = f.token_tiles;
  p.row_tiles = f.row_tiles;
  p.div_token_tiles = make_fast_div(static_cast<uint32_t>(f.token_tiles));
  p.kv_box = f.kv_box;
  p.q_tiles = g.q_tiles;
  p.q_box = std::min(kAttnRows, std::max(16, (s.q_len + 15) / 16 * 16));
  p.item_steps = g.item_steps;
  p.last_cols = (s.q_len - std::max(0, g.q_tiles - 1) * kAttnRows + 15) / 16 * 16;
  p.item_rows = static_cast<long long>(s.kv_heads) * f.row_tiles;
  p.scale_log2 = s.scale * 1.44269504088896341f;
  const bool half = s.dtype == CONV_DTYPE_F16;
  p.p_shift = half ? 15.f : 0.f;
  p.p_unscale = half ? 1.f / 32768.f : 1.f;
  p.stats = reinterpret_cast<float*>(ws + l.stat_at);
  p.row_norms = reinterpret_cast<float*>(ws + l.row_norm_at);
  p.value_norms = reinterpret_cast<float*>(ws + l.value_norm_at);
  p.key_groups = g.key_groups;
  p.part_q = reinterpret_cast<float*>(ws + l.part_q_at);
  p.part_kv = reinterpret_cast<float*>(ws + l.part_kv_at);
  p.status = reinterpret_cast<unsigned int*>(ws);
  p.timeout_cycles = wait_limit_cycles();
  p.fault_mode = wait_fault_mode();
  const bool queries = s.q_len > 0, keys = s.kv_len > 0;
  const bool wide = s.head_dim > 64;
  const uint32_t block = wide ? 32768 : 16384;  // 128 rows
  if (queries && keys) {
    // Row statistics.
    p.div_heads = make_fast_div(static_cast<uint32_t>(s.heads));
    p.row_slots = row_slots(s.head_dim);
    const int groups = g.q_tiles * g.per_tile;
    p.div_groups = make_fast_div(static_cast<uint32_t>(groups));
    p.div_kv_heads = make_fast_div(static_cast<uint32_t>(s.kv_heads));
    p.div_key_groups = make_fast_div(static_cast<uint32_t>(g.key_groups));
    const long long units = static_cast<long long>(s.batch) * s.heads * groups;
    p.row_blocks = static_cast<int>(std::min<long long>(kAttnRowBlocks, (units + 7) / 8));
    const long long value_units = static_cast<long long>(s.batch) * s.kv_heads * g.key_groups;
    p.value_blocks =
        half ? static_cast<int>(std::min<long long>(kAttnRowBlocks, (value_units + 7) / 8)) : 0;
    p.q_whole = g.q_whole;
    p.kv_whole = g.kv_whole;
    // (Short keys: delta is summed beside the scores; fp16 still wants the norms.)
    if ((!g.brief || half) && launch_attn_rows(p, stream) != cudaSuccess) return CONV_ERR_CUDA;
    if (g.brief) {
      conv_status_t st = encode_maps(&p, s, 1, p.q_box, f.kv_box);
      if (st == CONV_OK) st = encode_map(&p.map_dq, s.dq, s, s.heads, s.q_len, s.dqs, 1, p.q_box);
      if (st != CONV_OK) return st;
      // TMEM: dv and dk (64 columns each), then buffers of scores and dp.
      p.region = std::max(f.kv_box, (s.head_dim + 15) / 16 * 16);
      p.bufs = 128 + 4 * p.region <= 512 ? 2 : 1;
      // Shared memory: q and do, p and ds, dq's staging, k and v, barriers.
      p.off_x = 0;
      p.off_y = attn_short_stages() * 32768;
      p.off_stat = p.off_y + 4 * 16384;
      p.off_a = p.off_stat + 16384;
      p.off_bar = p.off_a + 2 * f.kv_box * 128;
      if (launch_attn_short_bwd(p, g.kv_grid, p.off_bar + attn_short_bar_bytes(), stream) != cudaSuccess)
        return CONV_ERR_CUDA;
      if (g.item_steps == 1) return CONV_OK;  // no item is cut
      return launch_attn_bwd_join(p, 0, g.kv_grid, 0, static_cast<long long>(s.batch) * s.kv_heads,
                                  stream) == cudaSuccess
                 ? CONV_OK
                 : CONV_ERR_CUDA;
    }
    // dq.
    conv_status_t st = encode_maps(&p, s, f.tile_heads, f.tile_tokens, f.kv_box);
    if (st != CONV_OK) return st;
    const uint32_t kv_tile = f.kv_box * (wide ? 256 : 128);
    // (One key tile: two of its stages do, and leave room for the sums of delta.)
    const bool one = s.kv_len <= f.kv_box;
    p.x_stages = one ? 2 : wide ? 3 : 4;
    p.y_stages = wide ? 2 : 4;
    p.off_a = 0;
    p.off_stat = 2 * block;
    p.off_x = p.off_stat + (one ? 2048 : 0);
    p.off_y = p.off_x + p.x_stages * kv_tile;
    p.off_bar = p.off_y + p.y_stages * kv_tile;
    if (launch_attn_dq(p, g.q_grid, p.off_bar + attn_bwd_bar_bytes(), stream) != cudaSuccess)
      return CONV_ERR_CUDA;
    // dk, dv: the queries in tiles of 128 tokens of one head.
    st = encode_map(&p.map_q, s.q, s, s.heads, s.q_len, s.qs, 1, p.q_box);
    if (st == CONV_OK) st = encode_map(&p.map_do, s.dout, s, s.heads, s.q_len, s.dos, 1, p.q_box);
    if (st != CONV_OK) return st;
    p.x_stages = wide && s.mask_bits ? 2 : 3;
    p.y_stages = 2;
    p.off_x = 2 * block;
    p.off_y = p.off_x + p.x_stages * block;
    p.off_stat = p.off_y + p.y_stages * block;
    p.off_mask = p.off_stat + 2048;
    p.off_bar = p.off_mask + (s.mask_bits ? 4096 : 0);
    if (launch_attn_dkv(p, g.kv_grid, p.off_bar + attn_bwd_bar_bytes(), stream) != cudaSuccess)
      return CONV_ERR_CUDA;
  } else if (queries) {
    AttnShape z = s;  // no keys: dq is zero
    z.out_w = s.dq;
    z.lse = nullptr;
    for (int i = 0; i < 3; ++i) z.os[i] = s.dqs[i];
    return launch_attn_no_keys(z, stream) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
  }
  // Tiles that were cut between CTAs, and keys without queries.
  const long long heads = static_cast<long long>(s.batch) * s.kv_heads;
  const long long q_blocks = queries && s.kv_len > f.kv_box && !g.q_whole ? heads * f.row_tiles : 0;
  const bool kv_join = g.item_steps == 0 || (g.item_steps > 1 && !g.kv_whole) || s.kv_lengths;
  const long long kv_blocks = kv_join ? heads * g.kv_tiles : 0;
  return launch_attn_bwd_join(p, g.q_grid, g.kv_grid, q_blocks, kv_blocks, stream) == cudaSuccess
             ? CONV_OK
             : CONV_ERR_CUDA;
}

conv_status_t check_args(const cross_attention_args_t& a, bool backward, AttnShape* s) {
  conv_status_t st = check_sizes(a);
  if (st != CONV_OK) return st;
  if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return CONV_ERR_INVALID_VALUE;
  // (Tensors without elements need no memory.)
  const bool queries = a.batch > 0 && a.q_len > 0, keys = a.batch > 0 && a.kv_len > 0;
  if ((queries && (!a.q || !a.out)) || (keys && (!a.k || !a.v))) return CONV_ERR_INVALID_VALUE;
  if (backward && ((queries && (!a.lse || !a.dout || !a.dq)) || (keys && (!a.dk || !a.dv))))
    return CONV_ERR_INVALID_VALUE;
  const void* ptrs[] = {a.q, a.k, a.v, a.out};
  for (const void* p : ptrs)
    if (off16(p)) return CONV_ERR_MISALIGNED;
  const void* grads[] = {a.dout, a.dq, a.dk, a.dv};
  for (const void* p : grads)
    if (backward && off16(p)) return CONV_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(a.lse) & 3u) || (reinterpret_cast<uintptr_t>(a.kv_lengths) & 3u))
    return CONV_ERR_MISALIGNED;
  *s = AttnShape{};
  st = take_strides(a.q_stride, a.batch, a.q_len, a.heads, false, s->qs);
  if (st == CONV_OK) st = take_strides(a.k_stride, a.batch, a.kv_len, a.kv_heads, false, s->ks);
  if (st == CONV_OK) st = take_strides(a.v_stride, a.batch, a.kv_len, a.kv_heads, false, s->vs);
  if (st == CONV_OK)
    st = take_strides(a.out_stride, a.batch, a.q_len, a.heads, !backward, s->os);
  if (backward) {
    if (st == CONV_OK) st = take_strides(a.dout_stride, a.batch, a.q_len, a.heads, false, s->dos);
    if (st == CONV_OK) st = take_strides(a.dq_stride, a.batch, a.q_len, a.heads, true, s->dqs);
    if (st == CONV_OK) st = take_strides(a.dk_stride, a.batch, a.kv_len, a.kv_heads, true, s->dks);
    if (st == CONV_OK) st = take_strides(a.dv_stride, a.batch, a.kv_len, a.kv_heads, true, s->dvs);
  }
  if (st != CONV_OK) return st;
  s->dtype = a.dtype;
  s->batch = a.batch;
  s->heads = a.heads;
  s->kv_heads = a.kv_heads;
  s->q_len = a.q_len;
  s->kv_len = a.kv_len;
  s->head_dim = a.head_dim;
  s->group = a.heads / a.kv_heads;
  s->scale = a.scale;
  s->q = a.q;
  s->k = a.k;
  s->v = a.v;
  s->out = a.out;
  s->out_w = a.out;
  s->lse = a.lse;
  s->kv_lengths = a.kv_lengths;
  if (backward) {
    s->dout = a.dout;
    s->dq = a.dq;
    s->dk = a.dk;
    s->dv = a.dv;
  }
  return CONV_OK;
}

conv_status_t run(const cross_attention_args_t* args, bool backward, void* workspace,
                  size_t workspace_bytes, cudaStream_t stream) {
  if (!args) return CONV_ERR_INVALID_VALUE;
  const cross_attention_args_t& a = *args;
  AttnShape s;
  conv_status_t st = check_args(a, backward, &s);
  if (st != CONV_OK) return st;
  if (!workspace) return CONV_ERR_INVALID_VALUE;
  if (off16(workspace)) return CONV_ERR_MISALIGNED;
  const int sms = attn_sm_count();
  if (sms <= 0) return CONV_ERR_CUDA;
  // (Tensors broadcast over heads have no head axis to load side by side.)
  const bool may_pack = s.qs[2] != 0 && (!backward || s.dos[2] != 0);
  const FwdPlan f = plan_fwd(a, sms, may_pack);
  const BwdPlan g = backward ? plan_bwd(a, f, sms) : BwdPlan{};
  const Layout l = layout(a, backward, f, g);
  if (workspace_bytes < l.total) return CONV_ERR_WORKSPACE_TOO_SMALL;
  if (a.batch == 0 || (!backward && a.q_len == 0)) return CONV_OK;
  char* ws = static_cast<char*>(workspace);
  if (a.mask && a.kv_len > 0 && a.q_len > 0) {
    uint32_t* bits = reinterpret_cast<uint32_t*>(ws + l.mask_at);
    s.mask_bits = bits;
    s.mask_words = l.mask.words;
    s.mask_q = l.mask.queries > 1 ? 1 : 0;
    s.mask_h = l.mask.heads > 1 ? l.mask.queries : 0;
    s.mask_b = l.mask.batches > 1 ? static_cast<long long>(l.mask.heads) * l.mask.queries : 0;
    uint32_t* any = reinterpret_cast<uint32_t*>(ws + l.any_at);
    s.mask_any = any;
    s.any_q = l.mask.queries > 1 ? 1 : 0;
    s.any_h = l.mask.heads > 1 ? l.mask.tiles : 0;
    s.any_b = l.mask.batches > 1 ? static_cast<long long>(l.mask.heads) * l.mask.tiles : 0;
    if (launch_mask_pack(a.mask, a.mask_stride, l.mask.batches, l.mask.heads, l.mask.queries,
                         a.kv_len, l.mask.words, bits, any, stream) != cudaSuccess)
      return CONV_ERR_CUDA;
  }
  if (backward) return run_bwd(s, f, g, ws, l, stream);
  if (a.kv_len > 0) return run_fwd(s, f, ws, l, stream);
  return launch_attn_no_keys(s, stream) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace

}  // namespace convgb300

extern "C" {

size_t cross_attention_workspace_size(const cross_attention_args_t* args, int backward) {
  using namespace convgb300;
  if (!args || check_sizes(*args) != CONV_OK) return 0;
  const int sms = attn_sm_count();
  if (sms <= 0) return 0;
  // Whichever way the queries turn out to be strided.
  size_t total = 0;
  for (int packed = 0; packed < 2; ++packed) {
    const FwdPlan f = plan_fwd(*args, sms, packed != 0);
    const BwdPlan g = plan_bwd(*args, f, sms);
    total = std::max(total, layout(*args, false, f, g).total);
    if (backward) total = std::max(total, layout(*args, true, f, g).total);
  }
  return total;
}

conv_status_t cross_attention_fwd(const cross_attention_args_t* args, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return convgb300::run(args, false, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

conv_status_t cross_attention_bwd(const cross_attention_args_t* args, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return convgb300::run(args, true, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

conv_status_t conv_testing_cross_attention_plan(const cross_attention_args_t* args, int num_sms,
                                                int out[3]) {
  using namespace convgb300;
  const conv_status_t st = check_sizes(*args);
  if (st != CONV_OK) return st;
  const FwdPlan f = plan_fwd(*args, num_sms, true);
  out[0] = f.one ? 2 : f.split ? 1 : 0;
  out[1] = f.grid;
  out[2] = f.one ? static_cast<int>(one_smem(f.kv_box)) : 0;
  return CONV_OK;
}

}  // extern "C"
