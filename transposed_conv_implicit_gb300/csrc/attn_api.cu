// Cross attention, host side: argument checks, workspace layout and the C
// entry points of include/conv_gb300_attention.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/conv_gb300_attention.h"
#include "attn_internal.h"
#include "attn_params.h"

namespace convgb300 {


cudaError_t launch_attn_simple_fwd(const AttnShape& a, cudaStream_t stream);
cudaError_t launch_attn_simple_bwd(const AttnShape& a, cudaStream_t stream);

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
  // Heads and batches share a launch's grid.
  if (static_cast<long long>(a.batch) * a.heads > 65535) return CONV_ERR_NOT_SUPPORTED;
  return CONV_OK;
}

// The packed mask's extents after broadcasting.
struct MaskShape {
  int batches, heads, queries, words;
  size_t bytes;
};

MaskShape mask_shape(const cross_attention_args_t& a) {
  MaskShape m{};
  if (!a.mask) return m;
  m.batches = a.mask_stride[0] == 0 ? 1 : a.batch;
  m.heads = a.mask_stride[1] == 0 ? 1 : a.heads;
  m.queries = a.mask_stride[2] == 0 ? 1 : a.q_len;
  m.words = (a.kv_len + 127) / 128 * 4;
  m.bytes = static_cast<size_t>(m.batches) * m.heads * m.queries * m.words * 4;
  return m;
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

struct Layout {
  MaskShape mask;
  size_t mask_at, total;
};

Layout layout(const cross_attention_args_t& a) {
  Layout l{};
  l.mask = mask_shape(a);
  l.mask_at = CONV_STATUS_BYTES;
  l.total = round_up(l.mask_at + l.mask.bytes, 256);
  return l;
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
  const Layout l = layout(a);
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
    if (launch_mask_pack(a.mask, a.mask_stride, l.mask.batches, l.mask.heads, l.mask.queries,
                         a.kv_len, l.mask.words, bits, stream) != cudaSuccess)
      return CONV_ERR_CUDA;
  }
  const cudaError_t e =
      backward ? launch_attn_simple_bwd(s, stream) : launch_attn_simple_fwd(s, stream);
  return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

}  // namespace

}  // namespace convgb300

extern "C" {

size_t cross_attention_workspace_size(const cross_attention_args_t* args, int backward) {
  using namespace convgb300;
  if (!args || check_sizes(*args) != CONV_OK) return 0;
  return layout(*args).total;
}

conv_status_t cross_attention_fwd(const cross_attention_args_t* args, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return convgb300::run(args, false, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

conv_status_t cross_attention_bwd(const cross_attention_args_t* args, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return convgb300::run(args, true, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
