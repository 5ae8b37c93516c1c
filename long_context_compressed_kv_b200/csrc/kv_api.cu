// C-ABI entry points of the 16-bit K/V layers: argument checks and launches.
#include <math.h>

#include "common.cuh"
#include "kv_kernels.h"
#include "tc_kernels.h"

using namespace v4a;

namespace {

// Workspace: [status header | parts | their statistics | the sums' maxima | the
// parts' outputs | the sums]
constexpr size_t kPartsOff = sizeof(WsHeader);
constexpr size_t kMlOff = kPartsOff + sizeof(KvPart) * 2 * kKvMaxCtas;
constexpr size_t kFoldMOff = kMlOff + sizeof(float2) * 2 * kKvMaxCtas * kKvPartRows;
constexpr size_t kOutOff = kFoldMOff + sizeof(float) * kKvMaxCtas * kKvPartRows;
static_assert(kMlOff % 16 == 0 && kFoldMOff % 16 == 0 && kOutOff % 16 == 0, "workspace alignment");

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

v4attn_status check_kv_desc(const v4attn_kv_desc* d) {
  if (!d || d->Hq < 1 || d->Hkv < 1) return V4A_ERR_INVALID_ARG;
  if (d->Hq % d->Hkv) return V4A_ERR_INVALID_ARG;
  if (d->Hq > 1024 || d->Hq / d->Hkv > 128) return V4A_ERR_UNSUPPORTED;
  if (d->d != 64 && d->d != 128) return V4A_ERR_UNSUPPORTED;
  if (d->dtype != V4A_BF16 && d->dtype != V4A_F16) return V4A_ERR_UNSUPPORTED;
  if (d->d_rope < 0 || d->d_rope > d->d) return V4A_ERR_INVALID_ARG;
  if (d->d_rope % 16) return V4A_ERR_UNSUPPORTED;
  if (d->d_rope && !(d->rope_theta > 0.f && isfinite(d->rope_theta))) return V4A_ERR_INVALID_ARG;
  if (d->n_win < 0 || !isfinite(d->softmax_scale)) return V4A_ERR_INVALID_ARG;
  return V4A_OK;
}

v4attn_status check_rows(const v4attn_kv_desc* d, const void* p, int64_t tok, int64_t head) {
  if (!p || !aligned(p, 16)) return V4A_ERR_INVALID_ARG;
  if (tok < d->d || head < d->d || (tok | head) % 8) return V4A_ERR_INVALID_ARG;
  // far beyond any device's memory; keeps byte offsets inside 63 bits and TMA's 40-bit strides
  if (tok > (1ll << 36) || head > (1ll << 36)) return V4A_ERR_INVALID_ARG;
  return V4A_OK;
}

template <class Args>
v4attn_status check_batch(const v4attn_kv_desc* d, const Args* a, const void* ws, size_t ws_bytes) {
  if (a->T > (1 << 20) || a->B > 65535) return V4A_ERR_UNSUPPORTED;
  if (!a->k_cache || !a->v_cache || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16))
    return V4A_ERR_INVALID_ARG;
  if (!a->q_start || !a->kv_len || !a->block_table || !aligned(a->q_start, 4) ||
      !aligned(a->kv_len, 8) || !aligned(a->block_table, 4))
    return V4A_ERR_INVALID_ARG;
  if (a->n_blocks < 1 || a->blocks_per_seq < 1) return V4A_ERR_INVALID_ARG;
  // positions and the pools' row numbers are 32-bit
  if (a->blocks_per_seq > (1 << 23) || a->n_blocks > kKvMaxRows / ((int64_t)d->Hkv * kKvBlock))
    return V4A_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 16) || ws_bytes < v4attn_kv_workspace_size(d)) return V4A_ERR_WORKSPACE;
  return V4A_OK;
}

template <class Args>
KvBatch batch(const Args* a, void* ws) {
  KvBatch b;
  b.T = a->T;
  b.B = a->B;
  b.q_start = a->q_start;
  b.kv_len = a->kv_len;
  b.bt = a->block_table;
  b.bps = a->blocks_per_seq;
  b.n_blocks = a->n_blocks;
  b.status = reinterpret_cast<uint32_t*>(ws);
  return b;
}

KvRows rows(const void* p, int64_t tok, int64_t head) {
  KvRows r;
  r.p = p;
  r.tok = tok;
  r.head = head;
  return r;
}

v4attn_status run_attention(const v4attn_kv_desc* d, const v4attn_kv_attn_args* a, void* ws,
                            size_t ws_bytes, cudaStream_t st, bool sparse) {
  v4attn_status s = check_kv_desc(d);
  if (s != V4A_OK) return s;
  if (!a || a->T < 0 || a->B < 0) return V4A_ERR_INVALID_ARG;
  if (a->T == 0 || a->B == 0) return V4A_OK;
  if ((s = check_batch(d, a, ws, ws_bytes)) != V4A_OK) return s;
  if ((s = check_rows(d, a->q, a->q_token_stride, a->q_head_stride)) != V4A_OK) return s;
  if ((s = check_rows(d, a->out, a->out_token_stride, a->out_head_stride)) != V4A_OK) return s;
  if (!aligned(a->sink, 4) || !aligned(a->lse, 4) || !aligned(a->idx, 4)) return V4A_ERR_INVALID_ARG;
  if (sparse) {
    if (d->n_win != 0 || a->n_local < 0 || a->n_sel < 0) return V4A_ERR_INVALID_ARG;
    if (a->n_sel > kKvMaxSel) return V4A_ERR_UNSUPPORTED;
    if (a->n_sel > 0 && (!a->idx || (a->n_lists != 1 && a->n_lists != d->Hkv)))
      return V4A_ERR_INVALID_ARG;
  }
  KvAttnParams P;
  P.b = batch(a, ws);
  P.Hq = d->Hq;
  P.Hkv = d->Hkv;
  P.g = d->Hq / d->Hkv;
  P.d = d->d;
  P.f16 = d->dtype == V4A_F16;
  P.scale = d->softmax_scale > 0.f ? d->softmax_scale : 1.0f / sqrtf((float)d->d);
  P.n_win = sparse || d->n_win >= (1 << 30) ? 0 : d->n_win;   // positions stay below 2^30
  P.q = rows(a->q, a->q_token_stride, a->q_head_stride);
  P.out = rows(a->out, a->out_token_stride, a->out_head_stride);
  P.k_cache = a->k_cache;
  P.v_cache = a->v_cache;
  P.sparse = sparse;
  P.idx = sparse ? a->idx : nullptr;
  P.n_lists = sparse && a->n_sel ? a->n_lists : 1;
  P.n_sel = sparse ? a->n_sel : 0;
  P.n_local = sparse ? a->n_local : 0;
  P.sink = a->sink;
  P.lse = a->lse;
  uint8_t* w8 = reinterpret_cast<uint8_t*>(ws);
  P.parts = reinterpret_cast<KvPart*>(w8 + kPartsOff);
  P.part_ml = reinterpret_cast<float2*>(w8 + kMlOff);
  P.part_o = reinterpret_cast<float*>(w8 + kOutOff);
  P.fold_m = reinterpret_cast<float*>(w8 + kFoldMOff);
  P.fold_o = reinterpret_cast<float4*>(P.part_o + (size_t)2 * kKvMaxCtas * kKvPartRows * d->d);
  return cuda_status(launch_kv_attn(P, st));
}

}  // namespace

extern "C" {

size_t v4attn_kv_workspace_size(const v4attn_kv_desc* desc) {
  if (check_kv_desc(desc) != V4A_OK) return 0;
  return kOutOff + sizeof(float) * 3 * kKvMaxCtas * kKvPartRows * desc->d;
}

v4attn_status v4attn_kv_append(const v4attn_kv_desc* desc, const v4attn_kv_append_args* a, void* ws,
                               size_t ws_bytes, cudaStream_t stream) {
  v4attn_status s = check_kv_desc(desc);
  if (s != V4A_OK) return s;
  if (!a || a->T < 0 || a->B < 0) return V4A_ERR_INVALID_ARG;
  if (a->T == 0 || a->B == 0) return V4A_OK;
  if ((s = check_batch(desc, a, ws, ws_bytes)) != V4A_OK) return s;
  if ((s = check_rows(desc, a->k, a->k_token_stride, a->k_head_stride)) != V4A_OK) return s;
  if ((s = check_rows(desc, a->v, a->v_token_stride, a->v_head_stride)) != V4A_OK) return s;
  if (!a->q != !a->q_out) return V4A_ERR_INVALID_ARG;
  KvAppendParams P;
  if (a->q) {
    if ((s = check_rows(desc, a->q, a->q_token_stride, a->q_head_stride)) != V4A_OK) return s;
    if ((s = check_rows(desc, a->q_out, a->q_out_token_stride, a->q_out_head_stride)) != V4A_OK)
      return s;
    P.q = rows(a->q, a->q_token_stride, a->q_head_stride);
    P.q_out = rows(a->q_out, a->q_out_token_stride, a->q_out_head_stride);
  }
  P.b = batch(a, ws);
  P.Hq = desc->Hq;
  P.Hkv = desc->Hkv;
  P.d = desc->d;
  P.d_rope = desc->d_rope;
  P.halves = desc->rope_halves != 0;
  P.f16 = desc->dtype == V4A_F16;
  P.k = rows(a->k, a->k_token_stride, a->k_head_stride);
  P.v = rows(a->v, a->v_token_stride, a->v_head_stride);
  P.k_cache = a->k_cache;
  P.v_cache = a->v_cache;
  // theta^(-2k/d_rope) by repeated products in long double: 64 of them, the
  // logarithm's and the power's own roundings (64-bit mantissas) stay below
  // 2^-55, so that a frequency carries its rounding to double and no more.  With
  // that of its product with the position an angle is off by 2^-52 p: 2.4e-7 rad
  // at the last of 2^30 positions (products in double: up to 4e-6).
  const long double step =
      desc->d_rope ? exp2l(log2l(desc->rope_theta) * (-2.0L / desc->d_rope)) : 0.0L;
  long double f = 0.159154943091895335768883763372514362L;   // 1 / (2 pi)
  for (int k = 0; k < 64; ++k, f *= step) P.freq[k] = k < desc->d_rope / 2 ? (double)f : 0.0;
  return cuda_status(launch_kv_append(P, stream));
}

v4attn_status v4attn_paged_attention(const v4attn_kv_desc* desc, const v4attn_kv_attn_args* args,
                                     void* ws, size_t ws_bytes, cudaStream_t stream) {
  return run_attention(desc, args, ws, ws_bytes, stream, false);
}

v4attn_status v4attn_block_sparse_attention(const v4attn_kv_desc* desc,
                                            const v4attn_kv_attn_args* args, void* ws,
                                            size_t ws_bytes, cudaStream_t stream) {
  return run_attention(desc, args, ws, ws_bytes, stream, true);
}

}  // extern "C"
