// Attention over a paged 16-bit K/V cache ("16-bit K/V layers" in v4attn.h),
// dense (causal, optional window) and over selected blocks.
//
// One CTA per (token, query head); each of its warps takes every fourth key,
// the lanes sharing a key's dims, with the running maximum and sum of a
// softmax; the warps' parts meet in shared memory.
#include "common.cuh"
#include "kv_kernels.h"

namespace v4a {

namespace {
constexpr int kWarps = 4;
}

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps) kv_attn_kernel(KvAttnParams P) {
  constexpr int E = D / 32;
  __shared__ float part[kWarps][D], ms[kWarps], ls[kWarps];
  const int t = blockIdx.x, hq = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = hq / P.g;
  int b = 0;
  for (int i = 0; i < P.b.B; i += 32 * kWarps)
    b += __syncthreads_count(i + tid < P.b.B && P.b.q_start[i + tid + 1] <= t);
  if (b >= P.b.B) return;
  const int q0 = P.b.q_start[b], q1 = P.b.q_start[b + 1];
  if (t < q0 || q0 < 0 || q1 > P.b.T) {
    if ((b > 0 || t >= q0) && tid == 0) flag(P.b.status, ST_BAD_SEQ);
    return;
  }
  int64_t p = P.b.kv_len[b] - (q1 - q0) + (t - q0);
  const int64_t cap = (int64_t)P.b.bps * kKvBlock;
  if ((p < 0 || p >= cap) && tid == 0) flag(P.b.status, ST_BAD_POSITION);
  p = min(p, cap - 1);
  auto load = [](const void* base, int64_t i) {
    return F16 ? __half2float(reinterpret_cast<const __half*>(base)[i])
               : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i]);
  };
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = load(P.q.p, t * P.q.tok + hq * P.q.head + lane + 32 * e) * P.scale;
    o[e] = 0.f;
  }
  const int32_t* list = P.sparse && P.n_sel
                            ? P.idx + ((int64_t)t * P.n_lists + (P.n_lists > 1 ? h : 0)) * P.n_sel
                            : nullptr;
  auto block = [&](int64_t lb) {       // the keys of logical block lb
    const int32_t pb = P.b.bt[(int64_t)b * P.b.bps + lb];
    if (pb < 0 || pb >= P.b.n_blocks) {
      if (lane == 0) flag(P.b.status, ST_BAD_INDEX);
      return;
    }
    for (int c = warp; c < kKvBlock; c += kWarps) {
      const int64_t j = lb * kKvBlock + c;
      if (j > p || (P.n_win && j <= p - P.n_win)) continue;
      const int64_t at = (((int64_t)pb * P.Hkv + h) * kKvBlock + c) * D;
      float s = 0.f;
      for (int e = 0; e < E; ++e) s += q[e] * load(P.k_cache, at + lane + 32 * e);
      s = warp_sum(s);
      const float mn = fmaxf(m, s), a = expf(m - mn), w = expf(s - mn);
      l = l * a + w;
      for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * load(P.v_cache, at + lane + 32 * e);
      m = mn;
    }
  };
  const int64_t last = p < 0 ? -1 : p / kKvBlock;
  if (!P.sparse) {
    const int64_t first = P.n_win ? max((int64_t)0, p - P.n_win + 1) / kKvBlock : 0;
    for (int64_t lb = first; lb <= last; ++lb) block(lb);
  } else {
    const int64_t local = max((int64_t)0, last - P.n_local + 1);
    int32_t before = -1;
    for (int i = 0; i < P.n_sel; ++i) {
      const int32_t e = list[i];
      if (e > before && e < local && e <= last) block(e);
      before = max(before, e);
    }
    for (int64_t lb = local; lb <= last; ++lb) block(lb);
  }
  for (int e = 0; e < E; ++e) part[warp][lane + 32 * e] = o[e];
  if (lane == 0) {
    ms[warp] = m;
    ls[warp] = l;
  }
  __syncthreads();
  float mm = P.sink ? P.sink[hq] : -INFINITY;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ms[w]);
  const float mz = mm == -INFINITY ? 0.f : mm;
  float den = P.sink ? expf(P.sink[hq] - mz) : 0.f;
  for (int w = 0; w < kWarps; ++w) den += ls[w] * expf(ms[w] - mz);
  for (int i = tid; i < D; i += 32 * kWarps) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += part[w][i] * expf(ms[w] - mz);
    x = den > 0.f || den != den ? x / den : 0.f;
    uint16_t* out = reinterpret_cast<uint16_t*>(const_cast<void*>(P.out.p)) + t * P.out.tok +
                    hq * P.out.head + i;
    if (F16)
      *reinterpret_cast<__half*>(out) = __float2half_rn(x);
    else
      *out = f32_to_bf16_bits(x);
  }
  if (tid == 0 && P.lse) P.lse[(int64_t)t * P.Hq + hq] = mz + logf(den);
}

cudaError_t launch_kv_attn(const KvAttnParams& P, cudaStream_t st) {
  const dim3 grid(P.b.T, P.Hq);
  if (P.d == 128 && P.f16) kv_attn_kernel<128, true><<<grid, 32 * kWarps, 0, st>>>(P);
  else if (P.d == 128) kv_attn_kernel<128, false><<<grid, 32 * kWarps, 0, st>>>(P);
  else if (P.f16) kv_attn_kernel<64, true><<<grid, 32 * kWarps, 0, st>>>(P);
  else kv_attn_kernel<64, false><<<grid, 32 * kWarps, 0, st>>>(P);
  return cudaGetLastError();
}

}  // namespace v4a
