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

// Rotate four adjacent pairs by the angles cs[0..3].
template <bool F16>
__device__ __forceinline__ void rotate_adjacent(uint4& a, const float2* cs) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2<F16>(w[i]), c = cs[i];
    w[i] = pack2<F16>(v.x * c.x - v.y * c.y, v.x * c.y + v.y * c.x);
  }
}
// Rotate eight pairs, a their first members, b their second.
template <bool F16>
__device__ __forceinline__ void rotate_halves(uint4& a, uint4& b, const float2* cs) {
  uint32_t* u = reinterpret_cast<uint32_t*>(&a);
  uint32_t* w = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<F16>(u[i]), y = unpack2<F16>(w[i]);
    const float2 c = cs[2 * i], e = cs[2 * i + 1];
    u[i] = pack2<F16>(x.x * c.x - y.x * c.y, x.y * e.x - y.y * e.y);
    w[i] = pack2<F16>(x.x * c.y + y.x * c.x, x.y * e.y + y.y * e.x);
  }
}

}  // namespace

// One CTA per token; a thread moves 16 values (two 16-byte vectors) of a row
// at a time, half the row apart, or, where that is how the pairs lie, half of
// d_rope: so the lanes' vectors are next to each other in every access.  The rows' addresses need only the token, so a
// thread's first NB units are on their way before its sequence, position
// and table entry (three dependent loads) and the angles are known.
template <bool F16, int NT, int NB>
__global__ void __launch_bounds__(NT) kv_append_kernel(const __grid_constant__ KvAppendParams P) {
  __shared__ float2 cs[64];
  const int t = blockIdx.x, tid = threadIdx.x;
  // launched while the grid before still runs (as the attention behind it is)
  next_grid();
  wait_grid();
  const int lu = P.d == 128 ? 3 : 2, units = 1 << lu;      // units of 16 values in a row
  const int keep = (P.d - P.d_rope) / 16, half = P.d_rope / 2;
  const int hq = P.q.p ? P.Hq : 0;
  const int n = (hq + 2 * P.Hkv) * units;
  // unit i: its row, and its two vectors' places in the row
  auto place = [&](int i, int& row, int& o0, int& o1) {
    row = i >> lu;
    const int u = i & (units - 1);
    if (!P.halves) {
      o0 = 8 * u;
      o1 = o0 + P.d / 2;
    } else if (u < keep) {
      o0 = 8 * u;
      o1 = o0 + 8 * keep;
    } else {
      o0 = 8 * (u + keep);
      o1 = o0 + half;
    }
  };
  uint4 a[NB], c[NB];
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int i = i0 + j * NT;
      if (i >= n) break;
      int row, o0, o1;
      place(i, row, o0, o1);
      const KvRows& r = row < hq ? P.q : row < hq + P.Hkv ? P.k : P.v;
      const int h = row < hq ? row : row < hq + P.Hkv ? row - hq : row - hq - P.Hkv;
      const uint16_t* src = reinterpret_cast<const uint16_t*>(r.p) + t * r.tok + h * r.head;
      a[j] = __ldcs(reinterpret_cast<const uint4*>(src + o0));
      c[j] = __ldcs(reinterpret_cast<const uint4*>(src + o1));
    }
  };
  load(tid);
  // The token's sequence: the number of sequences that end at or before it,
  // where starts do not fall.  Whether they do comes with the barrier below.
  int b = 0;
  bool bad = false;
  for (int i = tid; i < P.b.B; i += NT) {
    const int s0 = P.b.q_start[i], s1 = P.b.q_start[i + 1];
    b += s1 <= t;
    bad = bad || s0 < 0 || s1 < s0 || s1 > P.b.T;
  }
  if (P.b.B <= NT) {
    b = __syncthreads_count(b);
  } else {
    __shared__ int part[NT / 32];
    b = __reduce_add_sync(0xffffffffu, b);
    if ((tid & 31) == 0) part[tid / 32] = b;
    __syncthreads();
    b = 0;
    for (int i = 0; i < NT / 32; ++i) b += part[i];
  }
  // its position and pool block; false: it belongs to no sequence
  int64_t p;
  int32_t blk;
  bool page;
  uint32_t wrong;
  auto find = [&]() -> bool {
    wrong = 0;
    if (b >= P.b.B) return false;
    if (t < P.b.q_start[b]) return false;
    p = P.b.kv_len[b] - P.b.q_start[b + 1] + t;
    if (p < 0 || p >= (int64_t)P.b.bps * kKvBlock) {
      wrong = ST_BAD_POSITION;
      return false;
    }
    blk = P.b.bt[(int64_t)b * P.b.bps + p / kKvBlock];
    page = blk >= 0 && blk < P.b.n_blocks;
    if (!page) wrong = ST_BAD_INDEX;
    return true;
  };
  bool mine = find();
  auto turn = [&]() {
    if (mine && tid < half) {
      // turns in double, reduced to half a turn either way before going to float
      double r = (double)p * P.freq[tid];
      r -= rint(r);
      float co, si;
      sincospif(2.0f * (float)r, &si, &co);
      cs[tid] = make_float2(co, si);
    }
  };
  turn();
  if (__syncthreads_or(bad)) {
    // Some start falls or leaves [0, T].  The token's sequence is the first that
    // ends behind it; it is taken if it begins at or before the token and at no
    // less than any start before it (sequences taken share no row, and no other
    // can hold the token).
    __shared__ int first, most;
    if (tid == 0) {
      first = P.b.B;
      most = 0;
    }
    __syncthreads();
    wrong = 0;
    int low = P.b.B;
    for (int i = tid; i < P.b.B; i += NT)
      if (P.b.q_start[i + 1] > t) low = min(low, i);
    if (low < P.b.B) atomicMin(&first, low);
    __syncthreads();
    b = first;
    int top = 0;
    for (int i = tid; i <= b && i < P.b.B; i += NT) top = max(top, P.b.q_start[i]);
    if (top > 0) atomicMax(&most, top);
    __syncthreads();
    mine = b < P.b.B && P.b.q_start[b] >= most && P.b.q_start[b + 1] <= P.b.T && find();
    turn();
    if (t == 0 && tid == 0) flag(P.b.status, ST_BAD_SEQ);
    __syncthreads();
  }
  if (wrong && tid == 0) flag(P.b.status, wrong);
  if (!mine) return;
  for (int i0 = tid; i0 < n; i0 += NB * NT) {
    if (i0 != tid) load(i0);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int i = i0 + j * NT;
      if (i >= n) break;
      int row, o0, o1;
      place(i, row, o0, o1);
      uint16_t* dst;
      if (row < hq) {
        dst = reinterpret_cast<uint16_t*>(const_cast<void*>(P.q_out.p)) + t * P.q_out.tok +
              row * P.q_out.head;
      } else {
        if (!page) break;
        const bool is_v = row >= hq + P.Hkv;
        const int h = row - hq - (is_v ? P.Hkv : 0);
        dst = reinterpret_cast<uint16_t*>(is_v ? P.v_cache : P.k_cache) +
              (((int64_t)blk * P.Hkv + h) * kKvBlock + p % kKvBlock) * P.d;
      }
      if (row < hq + P.Hkv) {
        const int off = 16 * keep;                           // first rotated dim
        if (!P.halves) {
          if (o0 >= off) rotate_adjacent<F16>(a[j], cs + (o0 - off) / 2);
          if (o1 >= off) rotate_adjacent<F16>(c[j], cs + (o1 - off) / 2);
        } else if (o0 >= off) {
          rotate_halves<F16>(a[j], c[j], cs + (o0 - off));
        }
      }
      *reinterpret_cast<uint4*>(dst + o0) = a[j];
      *reinterpret_cast<uint4*>(dst + o1) = c[j];
    }
  }
}

namespace {
template <int NT, int NB>
cudaError_t launch(const KvAppendParams& P, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.b.T, 1, 1);
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return P.f16 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<true, NT, NB>, P)
               : cudaLaunchKernelEx(&cfg, kv_append_kernel<false, NT, NB>, P);
}
}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& P, cudaStream_t st) {
  // Threads a token by its units: 80 rows of 128 values (640 units) take 53.0 us
  // for 8192 tokens and 3.2 us for 16 on 320 threads, 55.6 and 4.5 us on 128; 40
  // rows of 64 (160 units) 5.8 us for 1204 tokens on 320, 3.9 us on 128.
  const int units = ((P.q.p ? P.Hq : 0) + 2 * P.Hkv) * P.d / 16;
  return units > 256 ? launch<320, 2>(P, st) : launch<128, 3>(P, st);
}

}  // namespace v4a
