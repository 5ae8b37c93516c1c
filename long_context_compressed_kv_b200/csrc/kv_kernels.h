// Kernel parameter blocks and launchers of the 16-bit K/V layers (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace v4a {

constexpr int kKvBlock = 128;       // positions a pool block holds
constexpr int kKvMaxRows = 0x7FFFFF00;   // rows of a pool (TMA coordinates are 32-bit)
constexpr int kKvMaxSel = 2048;     // entries of a query's block list
constexpr int kKvMaxCtas = 160;     // CTAs of the attention kernel (one an SM)
constexpr int kKvPartRows = 256;    // rows of an item: two tiles

#if defined(__CUDACC__)
// The kernels of a call, and calls in a row, are launched while the one before
// still runs (programmatic dependent launch): no global memory is touched before
// wait_grid(), which returns when the grid before is complete and flushed.
__device__ __forceinline__ void wait_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_grid() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// A ragged batch of new tokens over paged caches (see "16-bit K/V layers" in
// v4attn.h).
struct KvBatch {
  int T, B;
  const int32_t* q_start;
  const int64_t* kv_len;
  const int32_t* bt;
  int bps;
  int64_t n_blocks;
  uint32_t* status;
};

// rows [T][H][d] of a 16-bit type, strides in elements
struct KvRows {
  const void* p = nullptr;
  int64_t tok = 0, head = 0;
};

struct KvAppendParams {
  KvBatch b;
  int Hq, Hkv, d, d_rope, halves, f16;
  KvRows q, k, v, q_out;              // q.p null: no queries
  void *k_cache, *v_cache;
  double freq[64];                    // theta^(-2k/d_rope) / (2 pi): turns per position
};

// A part of an item (rows of one K/V head's queries) whose key blocks were cut.
struct KvPart {
  int rows;           // 0: none
  int ends;           // holds the item's last blocks
  int h, tok0;        // K/V head, first token row
};

struct KvAttnParams {
  KvBatch b;
  int Hq, Hkv, g, d, f16;             // g = Hq / Hkv
  float scale;
  int n_win;                          // 0: no window
  KvRows q, out;                      // out: written
  const void *k_cache, *v_cache;
  int sparse;                         // block lists and n_local instead of the window
  const int32_t* idx;
  int n_lists, n_sel, n_local;
  const float* sink;
  float* lse;
  int tt = 0;                         // tokens a tile (set at launch)
  // workspace: two parts a CTA (its first and last pieces), their rows'
  // (log2 of a weight's unit, sum of weights) and unnormalised outputs
  KvPart* parts;                      // [kKvMaxCtas][2]
  float2* part_ml;                    // [kKvMaxCtas][2][kKvPartRows]
  float* part_o;                      // [kKvMaxCtas][2][kKvPartRows][d]
  // and, a CTA's own, its two slots' sums over an item's blocks so far and the
  // maxima that these go with
  float4* fold_o;                     // [kKvMaxCtas][2][d / 4][kKvPartRows / 2]
  float* fold_m;                      // [kKvMaxCtas][2][kKvPartRows / 2]
};

cudaError_t launch_kv_append(const KvAppendParams& P, cudaStream_t st);
cudaError_t launch_kv_attn(const KvAttnParams& P, cudaStream_t st);

}  // namespace v4a
