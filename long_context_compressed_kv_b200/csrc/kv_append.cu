// Appending new tokens to a paged 16-bit K/V cache, the position rotation
// applied on the way ("16-bit K/V layers" in v4attn.h).
//
// Per token t of sequence b at position p: K rows and (optionally) the query's
// rows rotated by R(p) on their last d_rope dims,
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a),  a = p theta^(-2k/d_rope),
// V rows copied.  Every value is read once and written once: HBM bound for
// long chunks, launch latency for decode steps.
#include "common.cuh"
#include "kv_kernels.h"

namespace v4a {

namespace {

constexpr int kThreads = 256;

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if (F16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rotate pairs k0 .. k0+7: `a`, `b` are 8 values each; ADJ: the pairs are
// adjacent within the 16 values, else a holds the first, b the second members.
template <bool F16, bool ADJ>
__device__ __forceinline__ void rotate16(uint4& a, uint4& b, const float2* cs) {
  uint32_t* w[2] = {reinterpret_cast<uint32_t*>(&a), reinterpret_cast<uint32_t*>(&b)};
  if (ADJ) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& x = w[i >> 2][i & 3];
      const float2 v = unpack2<F16>(x), c = cs[i];
      x = pack2<F16>(v.x * c.x - v.y * c.y, v.x * c.y + v.y * c.x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<F16>(w[0][i]), y = unpack2<F16>(w[1][i]);
      const float2 c = cs[2 * i], e = cs[2 * i + 1];
      w[0][i] = pack2<F16>(x.x * c.x - y.x * c.y, x.y * e.x - y.y * e.y);
      w[1][i] = pack2<F16>(x.x * c.y + y.x * c.x, x.y * e.y + y.y * e.x);
    }
  }
}

}  // namespace

// One CTA per token; a thread moves 16 values (two 16-byte vectors) of a row
// at a time: 16 consecutive ones, or, where the pairs lie half of d_rope
// apart, 8 and their 8 partners.
template <bool F16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendParams P) {
  __shared__ float2 cs[64];
  const int t = blockIdx.x, tid = threadIdx.x;
  // the token's sequence: the number of sequences that end at or before it
  int b = 0;
  for (int i = 0; i < P.b.B; i += kThreads)
    b += __syncthreads_count(i + tid < P.b.B && P.b.q_start[i + tid + 1] <= t);
  if (b >= P.b.B) return;
  const int q0 = P.b.q_start[b], q1 = P.b.q_start[b + 1];
  if (t < q0 || q0 < 0 || q1 > P.b.T) {
    if ((b > 0 || t >= q0) && tid == 0) flag(P.b.status, ST_BAD_SEQ);
    return;
  }
  const int64_t p = P.b.kv_len[b] - (q1 - q0) + (t - q0);
  if (p < 0 || p >= (int64_t)P.b.bps * kKvBlock) {
    if (tid == 0) flag(P.b.status, ST_BAD_POSITION);
    return;
  }
  const int32_t blk = P.b.bt[(int64_t)b * P.b.bps + p / kKvBlock];
  const bool page = blk >= 0 && blk < P.b.n_blocks;
  if (!page && tid == 0) flag(P.b.status, ST_BAD_INDEX);
  const int half = P.d_rope / 2;
  if (tid < half) {
    // turns in double, reduced to half a turn either way before going to float
    double r = (double)p * P.freq[tid];
    r -= rint(r);
    float c, s;
    sincospif(2.0f * (float)r, &s, &c);
    cs[tid] = make_float2(c, s);
  }
  __syncthreads();
  const int units = P.d / 16, keep = (P.d - P.d_rope) / 16;
  const int hq = P.q.p ? P.Hq : 0;
  const int n = (hq + 2 * P.Hkv) * units;
  for (int i = tid; i < n; i += kThreads) {
    const int row = i / units, u = i - row * units;
    const uint16_t* src;
    uint16_t* dst;
    if (row < hq) {
      src = reinterpret_cast<const uint16_t*>(P.q.p) + t * P.q.tok + row * P.q.head;
      dst = reinterpret_cast<uint16_t*>(const_cast<void*>(P.q_out.p)) + t * P.q_out.tok +
            row * P.q_out.head;
    } else {
      if (!page) break;
      const bool is_v = row >= hq + P.Hkv;
      const int h = row - hq - (is_v ? P.Hkv : 0);
      const KvRows& r = is_v ? P.v : P.k;
      src = reinterpret_cast<const uint16_t*>(r.p) + t * r.tok + h * r.head;
      dst = reinterpret_cast<uint16_t*>(is_v ? P.v_cache : P.k_cache) +
            (((int64_t)blk * P.Hkv + h) * kKvBlock + p % kKvBlock) * P.d;
    }
    const bool turn = row < hq + P.Hkv && u >= keep;
    int o0 = 16 * u, o1 = 16 * u + 8;
    if (turn && P.halves) {
      o0 = 16 * keep + 8 * (u - keep);
      o1 = o0 + half;
    }
    uint4 a = *reinterpret_cast<const uint4*>(src + o0);
    uint4 c = *reinterpret_cast<const uint4*>(src + o1);
    if (turn) {
      if (P.halves)
        rotate16<F16, false>(a, c, cs + 8 * (u - keep));
      else
        rotate16<F16, true>(a, c, cs + 8 * (u - keep));
    }
    *reinterpret_cast<uint4*>(dst + o0) = a;
    *reinterpret_cast<uint4*>(dst + o1) = c;
  }
}

cudaError_t launch_kv_append(const KvAppendParams& P, cudaStream_t st) {
  if (P.f16)
    kv_append_kernel<true><<<P.b.T, kThreads, 0, st>>>(P);
  else
    kv_append_kernel<false><<<P.b.T, kThreads, 0, st>>>(P);
  return cudaGetLastError();
}

}  // namespace v4a
