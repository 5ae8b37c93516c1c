// Attention over a paged 16-bit K/V cache ("16-bit K/V layers" in v4attn.h),
// dense (causal, optional window) and over selected blocks, for single tokens,
// chunks and ragged mixes of both: one persistent tcgen05 kernel, and a merge
// of the parts of queries whose keys were split over CTAs.
//
// Mathematics: softmax(q K^T) V in one pass over the keys, 128 (a pool block)
// at a time: S = Q K^T, running maximum m and sum l of each row,
// P = 2^shift exp2(s scale log2e - m), O = O 2^(m_old - m) + P V.  O is rescaled
// only when m would grow by more than 2^8.  S, m, l and O are fp32; l sums P
// before its rounding.  P is rounded to the cache's type, which the tensor core
// wants of both operands of P V: a weight is off by half a step at most, as the
// output is by its own rounding.  The shift, the same for a row's weights and
// their sum, places P in the type's range (see kShift).
//
// Bounds.  Decode steps: HBM, 8 (g = 8) FLOP a byte.  32 steps of up to 16384
// positions, 64 heads on 8, d = 128: 172 to 180 us by the card, 6.16 to 6.45 TB/s
// of K and V.  Chunks: the tensor pipe (2 x 1024 of its cycles a block and pair of
// tiles), short of that the chain scores -> P -> P V -> next scores of a slot,
// which the other slot's half hides: 2048 tokens on 32768 after some seconds, under
// the power cap: 2.0 to 2.1 ms, 1.04 PFLOP/s (first launches 1.74 ms, 1.22
// PFLOP/s, pipe 64% busy).  At d = 64 the exponentials (16 a cycle and SM) take
// longer than the tensor pipe.  Short calls: launch, work list, first load and
// merge, about 10 us.
//
// Rows.  The g = Hq / Hkv query heads that share a K/V head are rows of one
// tile: row r is token r / g, head r % g, tt = 128 / g tokens a tile.  An item
// is (sequence, K/V head, up to 2 tt tokens).  A CTA has two slots, each with
// its own S / P and O in TMEM and its own softmax warpgroup:
//   more than tt tokens (chunks): a slot a tile, both on the same key blocks,
//     so a block is loaded once for 256 rows; a block that no row of a tile sees
//     (past the diagonal, before the window, not selected) its slot skips (four
//     prompts of up to 4096, 32 heads, after some seconds: 460 us without, 443
//     with; 2048 tokens on 32768: 2079 and 2067);
//   else (decode steps): both slots hold the one tile, even and odd blocks,
//     merged at the end.  Up to 64 rows are MMAs of M = 64, row r in lane
//     32 (r / 16) + r % 16, and up to 16 rows, in calls of mostly such, the
//     products are turned: S^T = K Q^T and O^T = V^T P^T with the rows as N = 16,
//     a softmax thread a key, P^T in shared memory.  The bytes bound these
//     calls either way, but the MMAs' padding costs power and, under the power
//     cap, clock: 32 steps of up to 16384 positions, after some seconds, take
//     208 us at 1.34 GHz with M = 128, 192 at 1.58 with M = 64 and 179 turned on one
//     card; 180 at 1.75 with M = 64 and 172 at 1.96 turned on another.
// The MMA thread issues P V of one slot and the next Q K^T of the same slot
// while the other slot's warps work on their scores.
//
// Work split: the items' key blocks, laid end to end, are cut into equal
// ranges, one a CTA, so ragged lengths and the causal triangle balance
// whatever their mix (lengths are read on the device; the host knows only
// T).  A CTA's first and last pieces may be parts of an item: their O, m and l
// go to the workspace (at most two a CTA) and kv_merge_kernel joins them.
//
// Warps: 0-3 / 4-7 softmax of slot 0 / 1 (a thread a row, TMEM lane quarter =
// warp % 4), 8 MMA issue, 9 work list and TMA loads, 10-11 idle (they complete the
// third warpgroup, whose registers the softmax warpgroups take over).
#include <algorithm>

#include "common.cuh"
#include "kv_kernels.h"
#include "tc_common.cuh"
#include "tc_kernels.h"

namespace v4a {

namespace {

constexpr int NK = kKvBlock;                   // keys a block
constexpr int MROWS = 128;                     // rows a tile
// Three warpgroups: 384 threads launched with 168 registers each (64512 of
// the SM's 65536); the third gives up what the softmax warpgroups, which hold
// a row's 128 scores, take: 2 x 208 + 88 = 3 x 168.
constexpr int NTHREADS = 384;
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kWindow = 2048;                  // blocks whose selection is joined at a time
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Columns of P after which its first MMAs go out, while the rest is formed (a
// slot's scores, P, P V and next scores follow one another, and that chain is
// what a step lasts): attend of 2048 tokens on 32768, 64 heads on 8: none early
// 1853 us, 32 columns 1785, 64 1750, 96 1792.
constexpr int kEarly = 64;
constexpr float kGrow = 8.0f;                  // log2 of the growth that rescales O
// log2 of a weight of 1.  fp16 ends at 2^-24: with P up to 2^(7 + 8) of 2^16 a
// weight counts down to 2^-32 of the largest (unshifted, keys below 2^-25 added
// to the sum but not to O: 900 of them behind one key 2^25.5 above were lost).
// bf16 has fp32's range, and P up to 1 leaves O that of the values' sum.
template <bool F16>
constexpr float kShift = F16 ? 7.0f : -kGrow;
// Blocks that a slot's O takes up in one go.  The tensor core adds to its fp32
// sums by cutting off, up to 2^-23 of them each 16 keys: with values of one sign
// O loses 2^-20.3 of itself a block, and 4096 blocks in a slot (160 decode steps on
// 2^20 positions) made it 0.34% too small.  After kFold blocks O is added to a sum
// outside the tensor core, and begins again: 2^-12 at most, 2^-12.3 measured.
constexpr int kFold = 256;
// Cost of an item besides its blocks, in blocks (Q load, epilogue): 32 decode
// steps of up to 16384 positions 189 us at 1, 183 at 2.
constexpr int kItemCost = 2;
// Least cost of a CTA's range: one step on 1999 positions 18.3 us at 3, 16.5 at
// 2, 14.8 at 1 (nothing else of the measured set moves).
constexpr int kMinRange = 1;

// MMAs of a piece: rows are M = 128 (all items of two tiles), M = 64, or N = 16
constexpr int kFull = 0, kHalf = 1, kTurned = 2;
constexpr int kTurnedRows = 16;                // the least N that M = 128 takes

// What a piece (a range of an item's blocks) tells the MMA and softmax warps.
struct Piece {
  int n;             // blocks
  int dual;          // two tiles (a slot each) or one
  int form;          // of its MMAs: kFull, kHalf or kTurned
  int to0, from1;    // dense, two tiles: slot 0 takes blocks 0 .. to0-1, slot 1 from1 .. n-1
  int first, last;   // of the item's blocks in this CTA's range
  int part;          // -1: the whole item, rows go to the output; else the part to write
  int b, h, tok0, ntok;   // sequence, K/V head, first token row, tokens
  int pos0;          // position of the first token
  int len;           // positions with keys
  int end;           // no piece: the CTA is done
};

// The scores that a slot's warps find ready.
struct Step {
  int tile;          // ring count of the block's V tile, -1: no scores, the piece's O is complete
  int blk;           // logical block, -1: not to be seen
  uint32_t mask;     // the item's tokens that take it (sparse)
};
constexpr int kMeta = 8;

template <int D, bool SPARSE>
struct Cfg {
  static constexpr int kTile = MROWS * D * 2;           // bytes of a Q, K or V tile
  // ring of K / V tiles: what 227 KB leave beside two Q tiles (and the lists)
  static constexpr int kStages = D == 128 ? (SPARSE ? 4 : 5) : 10;
};

template <int D, bool SPARSE>
struct Smem {
  using C = Cfg<D, SPARSE>;
  alignas(1024) uint8_t q[2][C::kTile];
  alignas(1024) uint8_t kv[C::kStages][C::kTile];
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t qfull, qempty, sready[2], pready[2], pearly[2], pfull[2], pempty[2], o1ready, o1free, done;
  // of the blocks on their way, by their count (a ring longer than they can be ahead):
  int blk[kMeta];                  // logical block, -1: not to be seen
  uint32_t mask[kMeta];            // its tokens (sparse)
  Step step[2];                    // what the MMA thread says with each slot's scores
  Piece piece[2];
  float m1[MROWS], l1[MROWS];      // slot 1's statistics for the merge in the CTA
  // turned items: what the four warps of a slot tell one another, round by round
  // (write, meet at xbar, read).  Two of each, taken in turn: a warp writes for
  // round n + 2 once all have met in round n + 1, so have read what round n held.
  uint64_t xbar[2];
  alignas(16) float xsum[2][2][4][kTurnedRows];
  alignas(4) uint8_t xflag[2][2][4];
  uint32_t tmem_base;
  uint32_t list_mask[SPARSE ? kWindow : 1];
  int list_blk[SPARSE ? kWindow : 1];
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// to += from, or to = from: 16 columns of fp32
__device__ __forceinline__ void add16(uint32_t to, uint32_t from, bool add) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) b[e] = 0;
  tmem_ld16_nowait(from, a);
  if (add) tmem_ld16_nowait(to, b);
  tmem_ld_wait();
#pragma unroll
  for (int e = 0; e < 16; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) + __uint_as_float(b[e]));
  tmem_st16(to, a);
  tmem_st_wait();
}
// MMA whose A operand (P) is read from tensor memory: M = 128 rows at lanes
// 0..127, two 16-bit elements of K a column
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 lanes an instruction
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  if (F16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// the largest of the warp's values
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// Adds a head's sink to a row's sum l of weights in units of 2^top; returns the
// factor of the weights so far.  Sinks beyond fp32 in the base of the
// exponentials (inf and above 2.36e38) take all of the weight.
__device__ __forceinline__ float join_sink(float sink, float& top, float& l) {
  const float sk = sink * kLog2e, mm = fmaxf(top, sk), ms = mm == -INFINITY ? 0.f : mm;
  const float f = ex2(top - ms);
  l = l * f + (sk == ms ? 1.0f : ex2(sk - ms));
  top = ms;
  return f;
}
// log of the denominator 2^top l; the sink itself, bit for bit, of a row without
// keys, and where the sink takes all.  A row that sees nothing but NaN has no
// maximum either (maxima pass over NaN): its sum tells them apart.
__device__ __forceinline__ float log_sum(float top, float l, bool no_key, const float* sink, int h) {
  if ((no_key && l == l) || (sink && top == INFINITY && l == 1.0f))
    return sink ? sink[h] : -INFINITY;
  return (top + log2f(l)) * kLn2;
}
// Registers a thread of the calling warpgroup may use from here on.
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// ---------------------------------------------------------------- work list
// Everything below is a function of the lengths alone, so every CTA finds its
// own range without a word from the others.

// 64-bit quotient; the 32-bit one where that is all it takes (a third of the time)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

struct SeqInfo {
  int q0, n;         // first token row, tokens (0 when its q_start is bad)
  int base;          // position of the first token
  int len;           // positions with keys: kv_len cut to the table
};

// fall: the sequence ends below its start
__device__ __forceinline__ SeqInfo seq_info(const KvAttnParams& P, int b, bool report, bool& fall) {
  SeqInfo s;
  const int q0 = P.b.q_start[b], q1 = P.b.q_start[b + 1];
  fall = q1 < q0;
  const int64_t len = P.b.kv_len[b], cap = (int64_t)P.b.bps * NK;
  const bool bad = q0 < 0 || q1 < q0 || q1 > P.b.T;
  s.q0 = q0;
  s.n = bad ? 0 : q1 - q0;
  s.len = (int)max((int64_t)0, min(len, cap));
  // a kv_len out of range still gives a 32-bit position
  s.base = (int)(max((int64_t)0, min(len, (int64_t)1 << 30)) - s.n);
  if (report) {
    if (bad) flag(P.b.status, ST_BAD_SEQ);
    if (s.n > 0 && (len > cap || len < s.n)) flag(P.b.status, ST_BAD_POSITION);
  }
  return s;
}

// Blocks of tokens i0 .. i1-1 of a sequence: first block and count.  Sparse
// items of one token walk their list's entries instead (n_sel + n_local).
struct Span {
  int lo, n;
};
__device__ __forceinline__ bool by_list(const KvAttnParams& P, int ntok) {
  return P.sparse && ntok == 1;
}
__device__ __forceinline__ Span item_span(const KvAttnParams& P, const SeqInfo& s, int i0, int i1) {
  Span r;
  const int last = min(s.base + i1 - 1, s.len - 1);
  if (by_list(P, i1 - i0)) {
    r.lo = 0;
    r.n = last < 0 ? 0 : min(P.n_sel + min(P.n_local, 1 << 23), last / NK + 1 + P.n_sel);
    return r;
  }
  const int hi = last < 0 ? 0 : last / NK + 1;
  r.lo = P.n_win ? min(max(0, s.base + i0 - P.n_win + 1) / NK, hi) : 0;
  r.n = hi - r.lo;
  return r;
}

// Cost of all items of one head of a sequence, found by the whole warp.
__device__ __forceinline__ int64_t head_cost(const KvAttnParams& P, const SeqInfo& s, int per_item,
                                             int lane) {
  const int items = (s.n + per_item - 1) / per_item;
  int64_t sum = 0;
  for (int k = lane; k < items; k += 32)
    sum += item_span(P, s, k * per_item, min(s.n, (k + 1) * per_item)).n + kItemCost;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

__device__ __forceinline__ SeqInfo shfl_seq(const SeqInfo& s, int src) {
  SeqInfo r;
  r.q0 = __shfl_sync(0xffffffffu, s.q0, src);
  r.n = __shfl_sync(0xffffffffu, s.n, src);
  r.base = __shfl_sync(0xffffffffu, s.base, src);
  r.len = __shfl_sync(0xffffffffu, s.len, src);
  return r;
}

// After a start that falls: does sequence b0 + lane, which begins at q0, begin
// below one before it?  Such are left out, so that sequences taken share no row.
// (Out of line: the common path keeps its registers.)
__device__ __noinline__ bool begins_below(const KvBatch& b, int b0, int q0, int lane) {
  int top = 0;
  for (int i = lane; i < b0; i += 32) top = max(top, b.q_start[i]);
  top = __reduce_max_sync(0xffffffffu, top);
  int m = b0 + lane < b.B ? b.q_start[b0 + lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) m = max(m, v);
  }
  return q0 < max(m, top);
}

// The warp's place in the laid-out work: walks (sequence, head, item).
struct Walk {
  int b0;            // sequences b0 .. b0+31, one a lane
  SeqInfo mine;      // this lane's sequence
  int64_t head;      // cost of one head of this lane's sequence
  int per_item;
  bool falls = false;   // a start before this group's end is below the one before it

  __device__ __forceinline__ void load(const KvAttnParams& P, int first, int lane, bool report) {
    b0 = first;
    mine = SeqInfo{0, 0, 0, 0};
    bool fall = false;
    if (b0 + lane < P.b.B) mine = seq_info(P, b0 + lane, report, fall);
    falls = __any_sync(0xffffffffu, fall) || falls;
    if (falls && begins_below(P.b, b0, mine.q0, lane)) mine.n = 0;
    head = 0;
    if (mine.n > 0 && mine.n <= per_item) head = item_span(P, mine, 0, mine.n).n + kItemCost;
    unsigned many = __ballot_sync(0xffffffffu, mine.n > per_item);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const int64_t c = head_cost(P, shfl_seq(mine, src), per_item, lane);
      if (lane == src) head = c;
    }
  }
};

// ---------------------------------------------------------------- kernel

template <int D, bool F16, bool SPARSE, bool TURN, bool LONG>
struct Kernel {
  using S = Smem<D, SPARSE>;
  using C = Cfg<D, SPARSE>;
  static constexpr int NST = C::kStages;
  static constexpr int TM_S = 0, TM_O = 2 * NK;          // TMEM columns: S0 S1 O0 O1
  // all of tensor memory, so its allocation starts at column 0
  static constexpr int kCols = 512;

  // -------------------------------------------------------------- loads
  static __device__ void produce(const KvAttnParams& P, S& s, const CUtensorMap* tm_q,
                                 const CUtensorMap* tm_k, const CUtensorMap* tm_v) {
    const int lane = threadIdx.x & 31;
    uint32_t* status = P.b.status;
    const int tt = P.tt, per_item = 2 * tt;
    wait_grid();
    Walk w;
    w.per_item = per_item;
    int64_t total = 0;
    for (int b0 = 0; b0 < P.b.B; b0 += 32) {
      w.load(P, b0, lane, blockIdx.x == 0);
      int64_t c = w.head * P.Hkv;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
      total += c;
    }
    int64_t range = quotient(total + gridDim.x - 1, gridDim.x);
    if (range < kMinRange) range = kMinRange;
    const int64_t x0 = range * blockIdx.x, x1 = min(total, x0 + range);
    KvPart* rec = P.parts + 2 * blockIdx.x;
    if (lane < 2) rec[lane] = KvPart{0, 0, 0, 0};
    __syncwarp();

    int pieces = 0, it = 0, items = 0;
    bool ok = true;
    // publish a piece (lane 0 writes it)
    auto publish = [&](const Piece& pc) -> bool {
      const int i = pieces & 1, u = pieces >> 1;
      if (u >= 1 && !mbar_wait_warp(&s.pempty[i], (u - 1) & 1, status, 0)) return false;
      if (lane == 0) {
        s.piece[i] = pc;
        mbar_arrive(&s.pfull[i]);
      }
      __syncwarp();
      ++pieces;
      return true;
    };
    // Q of the current item, one tile a slot (rows past the sequence's tokens are
    // never stored), once the item before has read its own: asked for when two
    // blocks of the item are on their way, or at its end
    int q_tiles = 0, q_head = 0, q_tok = 0, ahead = 0;
    auto load_q = [&]() -> bool {
      if (q_tiles == 0) return true;
      if (items >= 1 && !mbar_wait_warp(&s.qempty, (items - 1) & 1, status, 2)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(&s.qfull, q_tiles * D * 2 * P.g * tt);
        for (int t = 0; t < q_tiles; ++t)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(s.q[t] + c * (MROWS * 128), tm_q, &s.qfull, 64 * c, q_head, q_tok + t * tt);
      }
      __syncwarp();
      ++items;
      q_tiles = ahead = 0;
      return true;
    };
    // one block's K and V tiles (pb < 0: rows outside the pool, which TMA fills with zeros)
    auto load_block = [&](int h, int lb, int pb, uint32_t mask) -> bool {
      const int row = pb < 0 ? kKvMaxRows : (pb * P.Hkv + h) * NK;
#pragma unroll 1
      for (int j = 0; j < 2; ++j, ++it) {
        const int st = it % NST, u = it / NST;
        if (u >= 1 && !mbar_wait_warp(&s.empty[st], (u - 1) & 1, status, 1)) return false;
        if (lane == 0) {
          if (j == 0) {
            s.blk[(it >> 1) % kMeta] = pb < 0 ? -1 : lb;
            s.mask[(it >> 1) % kMeta] = mask;
          }
          mbar_arrive_expect_tx(&s.full[st], C::kTile);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_2d(s.kv[st] + c * (MROWS * 128), j ? tm_v : tm_k, &s.full[st], 64 * c, row);
        }
        __syncwarp();
      }
      return q_tiles == 0 || ++ahead < 2 || load_q();
    };
    // the pool block of logical block lb (lane-wise); -1 where the table holds none
    auto entry = [&](int b, int lb, bool want) -> int {
      return want ? __ldg(P.b.bt + (int64_t)b * P.b.bps + lb) : -1;
    };
    auto checked = [&](int pb, bool want) -> int {
      if (want && (pb < 0 || pb >= P.b.n_blocks)) {
        pb = -1;
        flag(status, ST_BAD_INDEX);
      }
      return pb;
    };
    auto page = [&](int b, int lb, bool want) -> int { return checked(entry(b, lb, want), want); };

    // find the first item of the range
    int64_t at = 0;                    // place of the current group of sequences
    for (int b0 = 0; ok && b0 < P.b.B && at < x1; b0 += 32) {
      if (P.b.B > 32) w.load(P, b0, lane, false);
      const int64_t all = w.head * P.Hkv;
      int64_t c = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += v;
      }
      const int64_t end = at + c, begin = end - all;     // this lane's sequence
      const int64_t group_end = __shfl_sync(0xffffffffu, end, 31);
      unsigned todo = __ballot_sync(0xffffffffu, all > 0 && begin < x1 && end > x0);
      while (ok && todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const SeqInfo q = shfl_seq(w.mine, src);
        const int64_t sb = __shfl_sync(0xffffffffu, begin, src);
        const int64_t hc = __shfl_sync(0xffffffffu, w.head, src);
        const int nit = (q.n + per_item - 1) / per_item;
        int h = x0 > sb ? (int)quotient(x0 - sb, hc) : 0;
        int64_t hx = sb + h * hc;                            // place of head h's first item
        int k = 0;
        int64_t ix = hx;
        // first item of this head that reaches past x0, 32 at a time
        if (x0 > hx && nit > 1) {
          for (;;) {
            int cst = 0;
            if (k + lane < nit)
              cst = item_span(P, q, (k + lane) * per_item, min(q.n, (k + lane + 1) * per_item)).n +
                    kItemCost;
            int64_t pre = cst;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int64_t v = __shfl_up_sync(0xffffffffu, pre, o);
              if (lane >= o) pre += v;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, cst > 0 && ix + pre > x0);
            if (hit) {
              const int l0 = __ffs(hit) - 1;
              ix += __shfl_sync(0xffffffffu, pre - cst, l0);
              k += l0;
              break;
            }
            ix += __shfl_sync(0xffffffffu, pre, 31);
            k += 32;
            if (k >= nit) break;                             // (cannot happen: the head holds x0)
          }
        }
        for (; ok && h < P.Hkv && ix < x1; ++h, k = 0) {
          for (; ok && k < nit && ix < x1; ++k) {
            const int i0 = k * per_item, i1 = min(q.n, i0 + per_item);
            const Span sp = item_span(P, q, i0, i1);
            const int64_t iend = ix + sp.n + kItemCost;
            // this CTA's blocks of the item: the first kItemCost places carry none
            const int c0 = (int)(max(x0, ix) - ix), c1 = (int)(min(x1, iend) - ix);
            const int e0 = max(c0 - kItemCost, 0), e1 = max(c1 - kItemCost, 0);
            Piece pc;
            pc.dual = i1 - i0 > tt;
            const int rows = (i1 - i0) * P.g;
            pc.form = TURN && rows <= kTurnedRows ? kTurned : rows <= MROWS / 2 ? kHalf : kFull;
            if (pc.dual) pc.form = kFull;
            pc.b = w.b0 + src;
            pc.h = h;
            pc.tok0 = q.q0 + i0;
            pc.ntok = i1 - i0;
            pc.pos0 = q.base + i0;
            pc.len = q.len;
            pc.end = 0;
            pc.part = c0 == 0 && ix + c1 == iend ? -1 : 2 * (int)blockIdx.x + (c0 == 0 ? 1 : 0);
            if (pc.part >= 0 && lane == 0) {
              KvPart r;
              r.rows = pc.ntok * P.g;
              r.ends = ix + c1 == iend;
              r.h = h;
              r.tok0 = pc.tok0;
              rec[pc.part & 1] = r;
            }
            q_tiles = pc.dual + 1;
            q_head = h * P.g;
            q_tok = pc.tok0;
            // (the first table entries are on their way while Q is asked for)
            int pb = SPARSE ? 0 : entry(pc.b, sp.lo + e0 + lane, e0 + lane < e1);
            if (items == 0) ok = load_q();
            if (!SPARSE) {
              pc.first = pc.last = 1;
              pc.n = e1 - e0;
              // of two tiles the first may end before the last block, and the
              // windows of the second may begin behind the first
              pc.to0 = min(pc.n, (pc.pos0 + tt - 1) / NK - sp.lo - e0 + 1);
              pc.from1 = P.n_win ? max(0, (pc.pos0 + tt - P.n_win + 1) / NK - sp.lo - e0) : 0;
              ok = ok && publish(pc);
              for (int e = e0; ok && e < e1; e += 32) {
                if (e > e0) pb = entry(pc.b, sp.lo + e + lane, e + lane < e1);
                pb = checked(pb, e + lane < e1);
                const int m = min(32, e1 - e);
                for (int i = 0; ok && i < m; ++i)
                  ok = load_block(h, sp.lo + e + i, __shfl_sync(0xffffffffu, pb, i), 0xffffffffu);
              }
            } else {
              ok = ok && sparse_piece(P, s, pc, e0, e1, lane, publish, load_block, load_q, page);
            }
            ok = ok && load_q();
            ix = iend;
          }
          if (ix >= x1) break;
        }
      }
      at = group_end;
    }
    if (ok) {
      Piece pc{};
      pc.end = 1;
      publish(pc);
    }
    // no load may still be landing when the CTA exits
    if (lane == 0) {
      for (int k = 0; k < NST && k < it; ++k) {
        const int i2 = it - 1 - k;
        mbar_wait(&s.full[i2 % NST], (i2 / NST) & 1);      // time bound only
      }
      if (items > 0) mbar_wait(&s.qfull, (items - 1) & 1);
    }
  }

  // Selected blocks of a piece.  One token: list entries e0 .. e1-1 (its list,
  // then its last blocks).  More: the blocks e0 .. e1-1 that any of them
  // selected, with a bit for each token that did, joined in shared memory
  // kWindow blocks at a time.
  template <class Pub, class Load, class LoadQ, class Page>
  static __device__ bool sparse_piece(const KvAttnParams& P, S& s, Piece pc, int e0, int e1, int lane,
                                      Pub& publish, Load& load_block, LoadQ& load_q, Page& page) {
    const int li = P.n_lists > 1 ? pc.h : 0;
    auto list_of = [&](int tok) { return P.idx + ((int64_t)(pc.tok0 + tok) * P.n_lists + li) * P.n_sel; };
    // the warp's 32 entries from i0 on; good: they count, before: largest entry before them
    auto entries = [&](const int32_t* list, int i0, int last, int& before, bool& good) -> int {
      const int e = i0 + lane < P.n_sel ? __ldg(list + i0 + lane) : -1;
      int top = e;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, v);
      }
      int prev = __shfl_up_sync(0xffffffffu, top, 1);
      prev = lane == 0 ? before : max(prev, before);
      good = e >= 0 && e > prev && e <= last;
      before = max(before, __shfl_sync(0xffffffffu, top, 31));
      return e;
    };
    bool ok = true, first = true;
    if (by_list(P, pc.ntok)) {
      const int p = min(pc.pos0, pc.len - 1), last = p < 0 ? -1 : p / NK;
      const int local = max(0, last - P.n_local + 1);          // first of the last blocks
      // the list's blocks in front of them (n_sel <= kWindow)
      int n = 0, before = -1;
      for (int i = 0; i < min(P.n_sel, e1); i += 32) {
        bool good;
        const int e = entries(list_of(0), i, last, before, good);
        good = good && e < local && i + lane >= e0 && i + lane < e1;
        const unsigned m = __ballot_sync(0xffffffffu, good);
        if (good) s.list_blk[n + __popc(m & ((1u << lane) - 1))] = e;
        n += __popc(m);
      }
      // then the last blocks, entries n_sel + i
      const int l0 = max(e0 - P.n_sel, 0), l1 = min(e1 - P.n_sel, last - local + 1);
      const int nl = max(0, l1 - l0);
      __syncwarp();
      pc.first = pc.last = 1;
      pc.n = n + nl;
      ok = publish(pc);
      for (int e = 0; ok && e < pc.n; e += 32) {
        int lb = 0;
        if (e + lane < pc.n) lb = e + lane < n ? s.list_blk[e + lane] : local + l0 + e + lane - n;
        const int pb = page(pc.b, lb, e + lane < pc.n);
        const int m = min(32, pc.n - e);
        for (int i = 0; ok && i < m; ++i)
          ok = load_block(pc.h, __shfl_sync(0xffffffffu, lb, i), __shfl_sync(0xffffffffu, pb, i),
                          0xffffffffu);
      }
      return ok;
    }
    int w0 = e0;
    do {
      const int w1 = min(e1, w0 + kWindow);
      for (int i = lane; i < w1 - w0; i += 32) s.list_mask[i] = 0;
      __syncwarp();
      if (lane < pc.ntok) {                                    // a lane a token
        const int p = min(pc.pos0 + lane, pc.len - 1), last = p < 0 ? -1 : p / NK;
        const int local = max(0, last - P.n_local + 1);
        const int32_t* list = list_of(lane);
        int before = -1;
        for (int i = 0; i < P.n_sel; i += 8) {
          int e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = i + j < P.n_sel ? __ldg(list + i + j) : -1;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (e[j] > before && e[j] <= last && e[j] >= w0 && e[j] < w1)
              atomicOr(&s.list_mask[e[j] - w0], 1u << lane);
            before = max(before, e[j]);
          }
        }
        for (int e = max(local, w0); e <= last && e < w1; ++e)
          atomicOr(&s.list_mask[e - w0], 1u << lane);
      }
      __syncwarp();
      int n = 0;
      for (int i = 0; i < w1 - w0; i += 32) {
        const uint32_t mk = i + lane < w1 - w0 ? s.list_mask[i + lane] : 0;
        const unsigned m = __ballot_sync(0xffffffffu, mk != 0);
        __syncwarp();
        const int to = n + __popc(m & ((1u << lane) - 1));     // <= i + lane: in place
        if (mk) {
          s.list_mask[to] = mk;
          s.list_blk[to] = w0 + i + lane;
        }
        n += __popc(m);
        __syncwarp();
      }
      pc.first = first;
      pc.last = w1 == e1;
      pc.n = n;
      ok = publish(pc);
      first = false;
      for (int e = 0; ok && e < n; e += 32) {
        const int lb = e + lane < n ? s.list_blk[e + lane] : 0;
        const uint32_t mk = e + lane < n ? s.list_mask[e + lane] : 0;
        const int pb = page(pc.b, lb, e + lane < n);
        const int m = min(32, n - e);
        for (int i = 0; ok && i < m; ++i)
          ok = load_block(pc.h, __shfl_sync(0xffffffffu, lb, i), __shfl_sync(0xffffffffu, pb, i),
                          __shfl_sync(0xffffffffu, mk, i));
      }
      // A piece two windows on waits for this one's to be handed back, which takes
      // the item's Q: asked for now, if fewer than two blocks were on their way.
      // (It waits for the item before alone, all of whose blocks are.)
      if (w1 < e1) ok = ok && load_q();
      w0 = w1;
    } while (ok && w0 < e1);
    return ok;
  }

  // -------------------------------------------------------------- MMA issue
  // The tensor-core instructions take their descriptors from the warp's uniform
  // registers.  The lane that elect.sync names runs this alone: the compiler then
  // knows the branch for one lane's, and its values for uniform ones.  (A branch
  // on lane == 0: 122 cycles an MMA; the whole warp together, the instructions
  // predicated on one lane and every wait taken by all: 71, but 5% more time in
  // all than this.)
  static __device__ void issue(const KvAttnParams& P, S& s) {
    wait_grid();
    if (elect_one()) issue_one(P, s);
    __syncwarp();
  }
  static __device__ __forceinline__ void issue_one(const KvAttnParams& P, S& s) {
    uint32_t* status = P.b.status;
    constexpr uint64_t k_bits = smem_desc_bits(16, 1024, 2);             // K-major, 128B swizzle
    constexpr uint64_t v_bits = smem_desc_bits(MROWS * 128, 1024, 2);    // MN-major, 128B swizzle
    constexpr uint32_t fmt = F16 ? 0 : 1;
    auto id_qk = [](int half) {
      return half ? idesc_f(fmt, fmt, MROWS / 2, NK, false, false)
                  : idesc_f(fmt, fmt, MROWS, NK, false, false);
    };
    auto id_pv = [](int half) {
      return half ? idesc_f(fmt, fmt, MROWS / 2, D, false, true)
                  : idesc_f(fmt, fmt, MROWS, D, false, true);
    };
    const uint32_t q_at = smem_u32(s.q) >> 4, kv_at = smem_u32(s.kv) >> 4;
    int base = 0, items = 0, np[2] = {0, 0}, ne[2] = {0, 0}, pend[2] = {-1, -1};
    uint32_t acc[2] = {0, 0};                              // blocks that a slot has taken
    auto wait_tile = [&](int i) { return mbar_wait_at(&s.full[i % NST], (i / NST) & 1, status, 3); };
    // turned: P^T is a B operand in shared memory, in the place of the second Q tile:
    // 32 bytes (16 rows) a key, 16-byte halves exchanged in every other four keys
    const uint64_t p_desc = smem_desc(s.q[1], smem_desc_bits(16, 256, 6));
    auto qk = [&](int slot, int qslot, int tile, int form) {
      tc_fence_after();
      const uint64_t a = k_bits | (q_at + qslot * (C::kTile / 16));
      const uint64_t b = k_bits | (kv_at + tile % NST * (C::kTile / 16));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        // 64 dims (4 steps of 32 bytes) a swizzled half of 128 rows x 128 bytes
        const uint32_t off = (kk / 4) * (MROWS * 128 / 16) + (kk % 4) * 2;
        mma_f16(TM_S + slot * NK, a + off, b + off, id_qk(form), kk > 0);
      }
    };
    // does O hold blocks already?
    auto begun = [&](int slot) -> uint32_t { return LONG ? acc[slot] % kFold : acc[slot]; };
    auto taken = [&](int slot) { acc[slot] = LONG ? acc[slot] + 1 : 1; };
    auto pv = [&](int slot, int tile, bool rest, int form) {
      tc_fence_after();
      const uint64_t b = v_bits | (kv_at + tile % NST * (C::kTile / 16));
#pragma unroll
      for (int kk = 0; kk < NK / 16; ++kk)        // 16 keys: 8 columns of P, 16 rows x 128 bytes
        if ((kk >= kEarly / 16) == rest)
          mma_f16_ts(TM_O + slot * D, TM_S + slot * NK + 8 * kk, b + 128 * kk, id_pv(form),
                 kk > 0 ? 1u : begun(slot));
      if (rest) taken(slot);
    };
    auto qk_turned = [&](int slot, int tile) {
      tc_fence_after();
      const uint64_t a = k_bits | (kv_at + tile % NST * (C::kTile / 16));
      const uint64_t b = k_bits | q_at;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * (MROWS * 128 / 16) + (kk % 4) * 2;
        mma_f16(TM_S + slot * NK, a + off, b + off, idesc_f(fmt, fmt, NK, kTurnedRows, false, false),
                kk > 0);
      }
    };
    auto pv_turned = [&](int slot, int tile) {
      tc_fence_after();
      const uint64_t a = v_bits | (kv_at + tile % NST * (C::kTile / 16));
      const uint64_t b = p_desc + slot * (kTurnedRows * 2 * NK / 16);
#pragma unroll
      for (int kk = 0; kk < NK / 16; ++kk)
        mma_f16(TM_O + slot * D, a + 128 * kk, b + 32 * kk,
                idesc_f(fmt, fmt, D, kTurnedRows, true, true), kk > 0 ? 1u : begun(slot));
      taken(slot);
    };
    // A slot's warps answer each step on pready: with P, or, where there were no
    // scores, that they have read the step (open: the answer is outstanding).
    bool open[2] = {false, false};
    auto answered = [&](int slot) -> bool {
      if (!open[slot]) return true;
      open[slot] = false;
      ++np[slot];
      return mbar_wait_at(&s.pready[slot], (np[slot] - 1) & 1, status, 6);
    };
    // What the scores just issued are of (tile < 0: the piece's O is what comes).
    // The warps wait for this arrive and for the tensor core's.
    auto signal = [&](int slot, int tile, int blk, uint32_t mask) -> bool {
      if (!answered(slot)) return false;
      s.step[slot] = Step{tile, blk, mask};
      mbar_arrive(&s.sready[slot]);
      tc_commit(&s.sready[slot]);
      open[slot] = true;
      return true;
    };
    // the P V still to issue of a slot (pend: its V tile), once P is there
    // (landed: the tile is known to be)
    auto flush = [&](int slot, bool landed, int form) -> bool {
      if (pend[slot] < 0) return true;
      if (!landed && !wait_tile(pend[slot])) return false;
      if (!mbar_wait_at(&s.pearly[slot], ne[slot] & 1, status, 14)) return false;
      ++ne[slot];
      pv(slot, pend[slot], false, form);
      if (!answered(slot)) return false;
      pv(slot, pend[slot], true, form);
      pend[slot] = -1;
      return true;
    };
    bool ok = true;
    for (int pieces = 0; ok; ++pieces) {
      const int pi = pieces & 1;
      if (!mbar_wait_at(&s.pfull[pi], (pieces >> 1) & 1, status, 4)) break;
      const int n = s.piece[pi].n, dual = s.piece[pi].dual,
                first = s.piece[pi].first, last = s.piece[pi].last,
                end = s.piece[pi].end, form = s.piece[pi].form, to0 = s.piece[pi].to0,
                from1 = s.piece[pi].from1;
      mbar_arrive(&s.pempty[pi]);
      if (end) break;
      if (first) {
        acc[0] = acc[1] = 0;
        if (!mbar_wait_at(&s.qfull, items & 1, status, 5)) break;
        ++items;
      }
      pend[0] = pend[1] = -1;
      const uint32_t tile_bits = (1u << min(P.tt, 31)) - 1;
      // Block i's K at tile base + 2 i, its V at base + 2 i + 1.  A slot's step: the
      // P V of its block before, then the Q K^T of its next; past the last block
      // the P V alone, and word that O is complete.
      if (dual) {
        for (int i = 0; ok && i <= n; ++i) {
          const int kt = base + 2 * i, mi = (kt >> 1) % kMeta;
          int blk = 0;
          uint32_t mask = 0;
          const bool both = pend[0] >= 0 && pend[1] >= 0;
#pragma unroll
          for (int slot = 0; slot < 2; ++slot) {
            if (!(ok = ok && flush(slot, slot == 1 && both, kFull))) break;
            if (slot == 1 && i > 0) tc_commit(&s.empty[(kt - 1) % NST]);
            if (i == n) {
              ok = signal(slot, -1, 0, 0);
              continue;
            }
            if (slot == 0) {
              if (!(ok = wait_tile(kt))) break;
              blk = s.blk[mi];
              mask = SPARSE ? s.mask[mi] : 0xffffffffu;
            }
            if (SPARSE ? ((mask >> (slot * P.tt)) & tile_bits) != 0 : slot ? i >= from1 : i < to0) {
              qk(slot, slot, kt, kFull);
              ok = signal(slot, kt + 1, blk, mask);
              pend[slot] = kt + 1;
            }
          }
          if (ok && i < n) tc_commit(&s.empty[kt % NST]);
        }
      } else if (TURN && form == kTurned) {
        for (int i = 0; ok && i < n + 2; i += 2) {
#pragma unroll
          for (int slot = 0; slot < 2; ++slot) {
            const int j = i + slot, kt = base + 2 * j, mi = (kt >> 1) % kMeta;
            if (!ok || j >= n + 2) break;
            if (pend[slot] >= 0) {
              if (!(ok = wait_tile(pend[slot]) && answered(slot))) break;
              pv_turned(slot, pend[slot]);
              pend[slot] = -1;
              tc_commit(&s.empty[(kt - 3) % NST]);
            }
            if (j >= n) {
              ok = signal(slot, -1, 0, 0);
              continue;
            }
            if (!(ok = wait_tile(kt))) break;
            qk_turned(slot, kt);
            tc_commit(&s.empty[kt % NST]);
            ok = signal(slot, kt + 1, s.blk[mi], SPARSE ? s.mask[mi] : 0xffffffffu);
            pend[slot] = kt + 1;
          }
        }
      } else {
        for (int i = 0; ok && i < n + 2; i += 2) {         // a slot's first block past n: its end
#pragma unroll
          for (int slot = 0; slot < 2; ++slot) {
            const int j = i + slot, kt = base + 2 * j, mi = (kt >> 1) % kMeta;
            if (!ok || j >= n + 2) break;
            const bool had = pend[slot] >= 0;
            if (!(ok = flush(slot, false, form))) break;
            if (had) tc_commit(&s.empty[(kt - 3) % NST]);
            if (j >= n) {
              ok = signal(slot, -1, 0, 0);
              continue;
            }
            if (!(ok = wait_tile(kt))) break;
            qk(slot, 0, kt, form);
            tc_commit(&s.empty[kt % NST]);
            ok = signal(slot, kt + 1, s.blk[mi], SPARSE ? s.mask[mi] : 0xffffffffu);
            pend[slot] = kt + 1;
          }
        }
      }
      if (!ok) break;
      if (last) tc_commit(&s.qempty);
      base += 2 * n;
    }
    tc_commit(&s.done);
    mbar_wait(&s.done, 0);                                 // time bound only
  }

  // -------------------------------------------------------------- softmax
  // The row's weights 2^(v sl2 - off) to its P columns; returns their sum.
  static __device__ __forceinline__ float weights(const float* v, float sl2, float off,
                                                  uint32_t t_p, uint32_t kp, uint64_t* early) {
    const uint64_t scale = pair(sl2, sl2), shift = pair(-off, -off);
    uint64_t s0 = 0, s1 = 0;                                 // two pairs of zeros
#pragma unroll
    for (int c = 0; c < NK; c += 32) {
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const uint64_t x = fma2(pair(v[c + e], v[c + e + 1]), scale, shift);
        float a, b;
        unpair(x, a, b);
        a = ex2(a);
        b = ex2(b);
        if (e & 2)
          s1 = add2(s1, pair(a, b));
        else
          s0 = add2(s0, pair(a, b));
        pk[e / 2] = pack16<F16>(a, b);
        if (SPARSE) pk[e / 2] &= kp;
      }
      tmem_st16(t_p + c / 2, pk);
      if (c == kEarly - 32) {                                // the MMAs over these may begin
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(early);
      }
    }
    float a, b;
    unpair(add2(s0, s1), a, b);
    return a + b;
  }

  // An item of at most 16 rows, with the products turned: S^T = K Q^T (a thread a
  // key, a column a row) and O^T = V^T P^T (a lane a dim).  The four warps agree
  // on each row's maximum; sums stay a thread's own until the end.
  // From piece `pieces` (seen by the caller) to the item's last, which it leaves
  // in `pieces`.
  static __device__ __forceinline__ bool turned_item(const KvAttnParams& P, S& s, int slot, int wq,
                                                     int lane, uint32_t t_s, uint32_t t_o, float sl2,
                                                     float grow, int& pieces, int& ns, int& no1,
                                                     int& nx) {
    constexpr int R = kTurnedRows;
    uint32_t* status = P.b.status;
    const int r = wq * 32 + lane;
    uint8_t* pt = s.q[1] + slot * (R * 2 * NK) + r * 32;
    const int swap = (r >> 2 & 1) * 16;
    const int rows = s.piece[pieces & 1].ntok * P.g;
    float m[R], off[R], l[R];
#pragma unroll
    for (int c = 0; c < R; ++c) {
      // rows of no token: no maximum to pass, no weight
      m[c] = c < rows ? -INFINITY : INFINITY;
      off[c] = c < rows ? 0.f : INFINITY;
      l[c] = 0.f;
    }
    bool has_o = false;
    int nb = 0;                                  // blocks of the item seen
    const uint32_t t_sum = t_s + 2 * R;          // O of earlier runs of kFold blocks
    // the four warps' writes before are seen by all behind it
    auto met = [&]() -> bool {
      const bool ok = mbar_wait_warp(&s.xbar[slot], nx & 1, status, 12);
      ++nx;
      return ok;
    };
    auto told = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.xbar[slot]);
    };
    for (bool more = false;; more = true, ++pieces) {
      const int pi = pieces & 1;
      if (more && !mbar_wait_warp(&s.pfull[pi], (pieces >> 1) & 1, status, 7)) return false;
      const Piece& pc = s.piece[pi];
      const int vlo = P.n_win ? pc.pos0 - P.n_win + 1 : 0, vhi = pc.len;
      // keys that every row sees
      const int all_hi = min(pc.pos0, pc.len - 1);
      const int all_lo = P.n_win ? pc.pos0 + pc.ntok - P.n_win : (int)0x80000000;
      const int lane_tok = min(lane / P.g, 31);
      bool end = false;
      do {                                         // runs of kFold blocks
        if (LONG && nb > 0 && nb % kFold == 0) {
          // P V of the run's last block is complete when the next scores are there
          if (!mbar_wait_warp(&s.sready[slot], ns & 1, status, 8)) return false;
          tc_fence_after();
          if (s.step[slot].tile >= 0) add16(t_sum, t_o, nb > kFold);
        }
        for (;;) {
          if (!mbar_wait_warp(&s.sready[slot], ns & 1, status, 8)) return false;
          ++ns;
          const Step stp = s.step[slot];
          tc_fence_after();
          if (stp.tile < 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.pready[slot]);
            end = true;
            break;
          }
          float v[R], p[R];
          {
            uint32_t raw[R];
            tmem_ld16_nowait(t_s, raw);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < R; ++c) v[c] = __uint_as_float(raw[c]);
          }
          const int blk = stp.blk, kb = blk * NK, key = kb + r;
          if (blk >= 0 && (kb + NK > vhi || kb < vlo)) {
            // V rows that nobody sees are zeroed, as below
            const int st = stp.tile % NST;
            if (!mbar_wait_warp(&s.full[st], (stp.tile / NST) & 1, status, 9)) return false;
            if (key >= vhi || key < vlo) {
              const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  *reinterpret_cast<uint4*>(s.kv[st] + c * (MROWS * 128) + r * 128 + e * 16) = z;
            }
          }
          // rows that see this thread's key, a bit each: tokens from `from` on, to `to`
          uint32_t vis = 0xffff;
          if (blk < 0 || kb + NK - 1 > all_hi || kb < all_lo) {
            const int from = min(max(key - pc.pos0, 0), R) * P.g;
            vis = blk < 0 || key >= pc.len ? 0 : vis << min(from, R);
            if (P.n_win) {
              const int to = min(max(key - pc.pos0 + P.n_win, 0), R) * P.g;
              vis &= (1u << min(to, R)) - 1;
            }
            vis &= 0xffff;
          }
          if (SPARSE) vis &= __ballot_sync(0xffffffffu, (stp.mask >> lane_tok) & 1);
          if (__any_sync(0xffffffffu, vis != 0xffff)) {
#pragma unroll
            for (int c = 0; c < R; ++c) v[c] = vis >> c & 1 ? v[c] : -INFINITY;
          }
          // Does a maximum grow?  A first block's do.
          bool grows = !has_o;
          if (has_o) {
            bool up = false;
#pragma unroll
            for (int c = 0; c < R; ++c) up = up || v[c] > m[c] + grow;
            up = __any_sync(0xffffffffu, up);
            if (lane == 0) s.xflag[slot][nx & 1][wq] = up;
            told();
            // the weights as if none did, while the other warps' word comes
#pragma unroll
            for (int c = 0; c < R; ++c) p[c] = ex2(fmaf(v[c], sl2, -off[c]));
            const uint32_t* flags = reinterpret_cast<const uint32_t*>(s.xflag[slot][nx & 1]);
            if (!met()) return false;
            grows = *flags != 0;
          }
          if (grows) {
            float w = 0.f;
#pragma unroll
            for (int c = 0; c < R; ++c) {
              const float x = warp_max(v[c]);
              if (lane == c) w = x;
            }
            float(*x)[R] = s.xsum[slot][nx & 1];
            if (lane < R) x[wq][lane] = w;
            told();
            if (!met()) return false;
            float a[R];
#pragma unroll
            for (int c = 0; c < R; ++c) {
              const float mx = max3(fmaxf(x[0][c], x[1][c]), x[2][c], x[3][c]);
              const float mn = mx > m[c] + grow ? mx : m[c];
              a[c] = mx > m[c] + grow ? ex2((m[c] - mn) * sl2) : 1.0f;
              m[c] = mn;
              off[c] = mn == -INFINITY ? 0.f : fmaf(mn, sl2, -kShift<F16>);
              l[c] *= a[c];
              p[c] = ex2(fmaf(v[c], sl2, -off[c]));
            }
            if (has_o) {
              // P V of the block before is complete: its commit came with these scores
              uint32_t o[R];
              tmem_ld16_nowait(t_o, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < R; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * a[c]);
              tmem_st16(t_o, o);
              tmem_st_wait();
              if (LONG && nb >= kFold) {
                tmem_ld16_nowait(t_sum, o);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < R; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * a[c]);
                tmem_st16(t_sum, o);
                tmem_st_wait();
              }
            }
          }
          uint32_t pk[R / 2];
#pragma unroll
          for (int c = 0; c < R; ++c) l[c] += p[c];
#pragma unroll
          for (int c = 0; c < R; c += 2) pk[c / 2] = pack16<F16>(p[c], p[c + 1]);
          *reinterpret_cast<uint4*>(pt + swap) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          *reinterpret_cast<uint4*>(pt + (swap ^ 16)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.pready[slot]);
          has_o = true;
          if (LONG && ++nb % kFold == 0) break;
        }
      } while (LONG && !end);
      if (pc.last) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.pempty[pi]);
    }
    // -------------------------------------------------------------- epilogue
    // From here a lane (of every warp) holds row `lane % 16`: short code, since it is
    // run once an item and its instructions come from memory.
    const Piece& pc = s.piece[pieces & 1];
    const int c0 = lane & (R - 1);
    float mr = -INFINITY, lr = 0.f;
    if (LONG && nb > kFold) add16(t_o, t_sum, true);
    if (has_o) {
      // sums over the warp's lanes, halving the rows a lane holds each time
#pragma unroll
      for (int o = R / 2; o > 0; o >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int c = 0; c < o; ++c) {
          const float keep = upper ? l[c + o] : l[c], send = upper ? l[c] : l[c + o];
          l[c] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], R);
      float(*x)[R] = s.xsum[slot][nx & 1];
      if (lane < R) x[wq][lane] = l[0];
      told();
#pragma unroll
      for (int c = 0; c < R; ++c) mr = c0 == c ? m[c] : mr;
      if (!met()) return false;
      lr = (x[0][c0] + x[1][c0]) + (x[2][c0] + x[3][c0]);
    }
    auto release = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.pempty[pieces & 1]);
    };
    if (slot == 1) {
      if (r < R) {
        s.m1[r] = mr;
        s.l1[r] = has_o ? lr : -1.0f;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o1ready);
      if (!mbar_wait_warp(&s.o1free, no1 & 1, status, 10)) return false;
      ++no1;
      release();
      return true;
    }
    if (!mbar_wait_warp(&s.o1ready, no1 & 1, status, 11)) return false;
    ++no1;
    tc_fence_after();
    const bool has1 = s.l1[0] >= 0.f || s.l1[0] != s.l1[0];
    uint32_t o0[R], o1[R];
#pragma unroll
    for (int c = 0; c < R; ++c) o0[c] = o1[c] = 0;
    if (has_o) tmem_ld16_nowait(t_o, o0);
    if (has1) tmem_ld16_nowait(t_o + D, o1);
    // the factors of the row's two sums, the log2 of a weight's unit, its sum of weights
    float f0 = 1.0f, f1 = 0.f;
    if (has1) {
      const float m1 = s.m1[c0], mm = fmaxf(mr, m1), ms = mm == -INFINITY ? 0.f : mm;
      f0 = ex2((mr - ms) * sl2);
      f1 = ex2((m1 - ms) * sl2);
      lr = lr * f0 + s.l1[c0] * f1;
      mr = mm;
    }
    const int tok = pc.tok0 + c0 / P.g, hq = pc.h * P.g + c0 % P.g, part = pc.part;
    const bool mine = c0 < rows;
    float top = fmaf(mr, sl2, -kShift<F16>);
    if (part < 0) {
      float f = 1.0f;
      if (P.sink && mine) f = join_sink(P.sink[hq], top, lr);
      f = lr == 0.f ? 0.f : f / lr;
      f0 *= f;
      f1 *= f;
      if (P.lse && mine && r < R)
        P.lse[(int64_t)tok * P.Hq + hq] = log_sum(top, lr, mr == -INFINITY, P.sink, hq);
    } else if (mine && r < R) {
      P.part_ml[(int64_t)part * (2 * MROWS) + r] = make_float2(top, lr);
    }
    tmem_ld_wait();
    // this lane's dim; rows of 64 dims lie in the first 16 lanes of each quarter
    const int dim = D == 128 ? r : wq * 16 + (lane & 15);
    const bool stores = D == 128 || lane < 16;
    const int64_t at = (int64_t)tok * P.out.tok + (int64_t)hq * P.out.head;
    uint16_t* out = reinterpret_cast<uint16_t*>(const_cast<void*>(P.out.p)) + dim;
    float* part_o = P.part_o + (int64_t)part * (2 * MROWS) * D + dim;
#pragma unroll
    for (int c = 0; c < R; ++c) {
      // (a row without keys in one of the slots has its factor 0 and O 0)
      const float x = fmaf(__uint_as_float(o1[c]), __shfl_sync(0xffffffffu, f1, c),
                           __uint_as_float(o0[c]) * __shfl_sync(0xffffffffu, f0, c));
      const int64_t to = __shfl_sync(0xffffffffu, at, c);
      if (c < rows && stores) {
        if (part < 0)
          out[to] = (uint16_t)pack16<F16>(x, 0.f);
        else
          part_o[c * D] = x;
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.o1free);
    release();
    return true;
  }

  static __device__ void softmax(const KvAttnParams& P, S& s) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp >> 2, r = (warp & 3) * 32 + lane;
    uint32_t* status = P.b.status;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = lanes + TM_S + slot * NK, t_o = lanes + TM_O + slot * D;
    const float sl2 = P.scale * kLog2e;
    const float grow = fminf(kGrow / sl2, 1e37f);            // finite: a row's first key passes -inf
    int ns = 0, no1 = 0, nx = 0;
    wait_grid();
    float m = -INFINITY, l = 0.f;
    bool has_o = false;
    int nb = 0;                                              // blocks of the item seen
    for (int pieces = 0;; ++pieces) {
      const int pi = pieces & 1;
      if (!mbar_wait_warp(&s.pfull[pi], (pieces >> 1) & 1, status, 7)) return;
      const Piece& pc = s.piece[pi];
      if (pc.end) return;
      if (TURN && pc.form == kTurned) {
        if (!turned_item(P, s, slot, warp & 3, lane, t_s, t_o, sl2, grow, pieces, ns, no1, nx)) return;
        continue;
      }
      // the piece's entry is handed back when the warp has finished with it
      auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.pempty[pi]);
      };
      // this lane's row of the tile (MROWS: none), its token and head
      const int row = pc.form == kFull ? r : lane < 16 ? (warp & 3) * 16 + lane : MROWS;
      const int rt = row / P.g, rh = row - rt * P.g;
      const int tok = rt + (pc.dual ? slot * P.tt : 0);      // of the item
      const bool valid = rt < P.tt && tok < pc.ntok;
      const bool active = __any_sync(0xffffffffu, valid);
      // keys that the row sees: lo .. hi; rows of no token take all, unstored
      const int p = pc.pos0 + tok;
      const int hi = valid ? min(p, pc.len - 1) : 0x7FFFFFFF;
      const int lo = valid && P.n_win ? p - P.n_win + 1 : (int)0x80000000;
      // keys that every row of the warp sees
      const int all_hi = __reduce_min_sync(0xffffffffu, hi), all_lo = __reduce_max_sync(0xffffffffu, lo);
      // rows of V that no query of the item sees: before its first window, past its end
      const int vlo = P.n_win ? pc.pos0 - P.n_win + 1 : 0, vhi = pc.len;
      // The row's O to its sum over earlier runs (or, at the item's end, that sum to
      // O), each in units of the maximum that it was formed with.  The sums of a
      // slot's rows lie in the workspace, four dims of all of them side by side.
      auto fold = [&](bool end) {
        const int own = (int)blockIdx.x * 2 + slot, at = own * MROWS + (row & (MROWS - 1));
        float4* sum = P.fold_o + (int64_t)own * MROWS * (D / 4) + (row & (MROWS - 1));
        const bool more = valid && nb > kFold;
        const float was = more ? P.fold_m[at] : -INFINITY;
        const float f = was == -INFINITY ? 0.f : ex2((was - m) * sl2);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          float4 w[8];
          tmem_ld32_nowait(t_o + c, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            w[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (more) w[e] = sum[(c / 4 + e) * MROWS];
          }
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            w[e].x = fmaf(w[e].x, f, __uint_as_float(o[4 * e]));
            w[e].y = fmaf(w[e].y, f, __uint_as_float(o[4 * e + 1]));
            w[e].z = fmaf(w[e].z, f, __uint_as_float(o[4 * e + 2]));
            w[e].w = fmaf(w[e].w, f, __uint_as_float(o[4 * e + 3]));
          }
          if (end) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              o[4 * e] = __float_as_uint(w[e].x);
              o[4 * e + 1] = __float_as_uint(w[e].y);
              o[4 * e + 2] = __float_as_uint(w[e].z);
              o[4 * e + 3] = __float_as_uint(w[e].w);
            }
            tmem_st16(t_o + c, o);
            tmem_st16(t_o + c + 16, o + 16);
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[(c / 4 + e) * MROWS] = w[e];
          }
          __syncwarp();
        }
        if (end) tmem_st_wait();
        if (valid && !end) P.fold_m[at] = m;
      };
      if (pc.first) {
        m = -INFINITY;
        l = 0.f;
        has_o = false;
        nb = 0;
      }
      bool end = false;
      do {                                                   // runs of kFold blocks
        if (LONG && nb > 0 && nb % kFold == 0) {
          // P V of the run's last block is complete when the next scores are there
          if (!mbar_wait_warp(&s.sready[slot], ns & 1, status, 8)) return;
          tc_fence_after();
          if (active && s.step[slot].tile >= 0) fold(false);
        }
        for (;;) {
          if (!mbar_wait_warp(&s.sready[slot], ns & 1, status, 8)) return;
          ++ns;
          const Step stp = s.step[slot];
          tc_fence_after();
          if (stp.tile < 0) {                                  // the last P V is complete
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.pready[slot]);
            end = true;
            break;
          }
          const int blk = stp.blk, kb = blk * NK;
          if (blk >= 0 && (kb + NK > vhi || kb < vlo)) {
            // V rows that nobody sees may hold anything, and 0 x NaN is NaN: zero them
            const int key = kb + r, st = stp.tile % NST;
            if (!mbar_wait_warp(&s.full[st], (stp.tile / NST) & 1, status, 9)) return;
            if (key >= vhi || key < vlo) {
              const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  *reinterpret_cast<uint4*>(s.kv[st] + c * (MROWS * 128) + r * 128 + e * 16) = z;
            }
            fence_proxy_async_smem();
          }
          if (active) {
            float v[NK];
            {
              uint32_t raw[NK];
#pragma unroll
              for (int c = 0; c < NK; c += 32) tmem_ld32_nowait(t_s + c, raw + c);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < NK; ++c) v[c] = __uint_as_float(raw[c]);
            }
            // columns lc .. hc are seen; keep: the row's token takes the block
            const bool keep = blk >= 0 && (!SPARSE || !valid || ((stp.mask >> tok) & 1));
            const int hc = blk < 0 ? -1 : hi - kb, lc = lo == (int)0x80000000 ? 0 : lo - kb;
            if (blk < 0 || kb + NK - 1 > all_hi) {
#pragma unroll
              for (int c = 0; c < NK; ++c) v[c] = c <= hc ? v[c] : -INFINITY;
            }
            if (!SPARSE && kb < all_lo) {
#pragma unroll
              for (int c = 0; c < NK; ++c) v[c] = c >= lc ? v[c] : -INFINITY;
            }
            float x[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = v[c];
#pragma unroll
            for (int c = 4; c < NK - 4; c += 8) {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = max3(x[e], v[c + 2 * e], v[c + 2 * e + 1]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = max3(x[c], v[NK - 4 + c], x[c]);
            float mx = max3(max3(x[0], x[1], x[2]), x[3], x[3]);
            if (SPARSE && !keep) mx = -INFINITY;
            const bool up = mx > m + grow;
            if (__any_sync(0xffffffffu, up)) {
              const float mn = up ? mx : m;
              const float a = up ? ex2((m - mn) * sl2) : 1.0f;
              m = mn;
              l *= a;
              if (has_o) {
                // P V of the block before is complete: its commit came with these scores
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  uint32_t o[16];
                  tmem_ld16_nowait(t_o + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                  tmem_st16(t_o + c, o);
                }
              }
            }
            const float off = m == -INFINITY ? 0.f : fmaf(m, sl2, -kShift<F16>);
            const float sum = weights(v, sl2, off, t_s, keep ? 0xffffffffu : 0u, &s.pearly[slot]);
            l += SPARSE && !keep ? 0.f : sum;
          } else {
            __syncwarp();                                      // every lane's zeros before the word of them
            if (lane == 0) mbar_arrive(&s.pearly[slot]);
          }
          if (active) tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.pready[slot]);
          has_o = true;
          if (LONG && ++nb % kFold == 0) break;
        }
      } while (LONG && !end);
      if (LONG && pc.last && active && nb > kFold) fold(true);
      if (!pc.last) {
        release();
        continue;
      }
      // ---------------------------------------------------------- epilogue
      if (!pc.dual && slot == 1) {
        s.m1[r] = m;
        s.l1[r] = has_o ? l : -1.0f;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o1ready);
        if (!mbar_wait_warp(&s.o1free, no1 & 1, status, 10)) return;
        ++no1;
        release();
        continue;
      }
      float a0 = 1.0f, a1 = 0.f;
      bool has1 = false;
      if (!pc.dual) {
        if (!mbar_wait_warp(&s.o1ready, no1 & 1, status, 11)) return;
        ++no1;
        tc_fence_after();
        has1 = s.l1[r] >= 0.f || s.l1[r] != s.l1[r];
        if (has1) {
          const float m1 = s.m1[r], mm = fmaxf(m, m1), ms = mm == -INFINITY ? 0.f : mm;
          a0 = ex2((m - ms) * sl2);
          a1 = ex2((m1 - ms) * sl2);
          l = l * a0 + s.l1[r] * a1;
          m = mm;
        }
        has1 = __any_sync(0xffffffffu, has1);                // the same in every lane
      }
      const int part = pc.part;
      float top = fmaf(m, sl2, -kShift<F16>), f = 1.0f;      // log2 of a weight's unit
      if (part < 0) {
        const int hq = pc.h * P.g + rh;
        if (P.sink && valid) f = join_sink(P.sink[hq], top, l);
        if (valid && P.lse)
          P.lse[(int64_t)(pc.tok0 + tok) * P.Hq + hq] = log_sum(top, l, m == -INFINITY, P.sink, hq);
        f = l == 0.f ? 0.f : f / l;
      } else if (valid) {
        float2* ml = P.part_ml + (int64_t)part * (2 * MROWS) + (pc.dual ? slot * MROWS : 0) + row;
        *ml = make_float2(top, l);
      }
      __syncwarp();
      if (active) {
        uint16_t* out = reinterpret_cast<uint16_t*>(const_cast<void*>(P.out.p)) +
                        (int64_t)(pc.tok0 + tok) * P.out.tok +
                        (int64_t)(pc.h * P.g + rh) * P.out.head;
        float* part_o = P.part_o +
                        ((int64_t)part * (2 * MROWS) + (pc.dual ? slot * MROWS : 0) + row) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16], o1[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = o1[e] = 0;
          if (has_o) tmem_ld16_nowait(t_o + c, o);
          if (has1) tmem_ld16_nowait(t_o + D + c, o1);
          tmem_ld_wait();
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e] = __uint_as_float(o[e]) * a0;
            if (has1) x[e] = fmaf(__uint_as_float(o1[e]), a1, x[e]);
          }
          if (valid && part < 0) {
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              uint4 w;
              w.x = pack16<F16>(x[e] * f, x[e + 1] * f);
              w.y = pack16<F16>(x[e + 2] * f, x[e + 3] * f);
              w.z = pack16<F16>(x[e + 4] * f, x[e + 5] * f);
              w.w = pack16<F16>(x[e + 6] * f, x[e + 7] * f);
              *reinterpret_cast<uint4*>(out + c + e) = w;
            }
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(part_o + c + e) =
                  make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      if (!pc.dual) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o1free);
      }
      release();
    }
  }
};

}  // namespace

template <int D, bool F16, bool SPARSE, bool TURN, bool LONG>
__global__ void __launch_bounds__(NTHREADS, 1)
    kv_attn_kernel(const __grid_constant__ KvAttnParams P, const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  using K = Kernel<D, F16, SPARSE, TURN, LONG>;
  using S = typename K::S;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < K::NST; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    mbar_init(&s.qfull, 1);
    mbar_init(&s.qempty, 1);
    mbar_init(&s.o1ready, 4);
    mbar_init(&s.o1free, 4);
    mbar_init(&s.done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.sready[i], 2);
      mbar_init(&s.pready[i], 4);
      mbar_init(&s.pearly[i], 4);
      mbar_init(&s.xbar[i], 4);
      mbar_init(&s.pfull[i], 1);
      mbar_init(&s.pempty[i], 9);
    }
    fence_mbar_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 8) tmem_alloc(&s.tmem_base, K::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  next_grid();
  if (warp >= 8) {
    regs_down<kOtherRegs>();
    if (warp == 9)
      K::produce(P, s, &tm_q, &tm_k, &tm_v);
    else if (warp == 8)
      K::issue(P, s);
  } else {
    regs_up<kSoftmaxRegs>();
    K::softmax(P, s);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(0, K::kCols);
  }
}

// Joins the parts of the items that were cut: block (c, y) the item whose first
// part is CTA c's last piece, some of its rows.  Its further parts are the first
// pieces of the CTAs behind c; the sums are taken in one order on every run.
// Launched while the kernel before still runs, it waits for its end here: the
// parts are small and in L2, so its launch would cost as much as its work.
template <int D, bool F16>
__global__ void __launch_bounds__(256) kv_merge_kernel(const __grid_constant__ KvAttnParams P, int n_cta) {
  next_grid();
  wait_grid();
  const int c = blockIdx.x;
  // the CTA whose first piece ends the item (kKvMaxCtas <= 256 threads look at once)
  __shared__ int last_s;
  const int cand = c + 1 + threadIdx.x;
  const int ends = cand < n_cta ? P.parts[2 * cand].ends : 0;
  const KvPart r = P.parts[2 * c + 1];
  if (r.rows == 0) return;
  if (threadIdx.x == 0) last_s = n_cta - 1;
  __syncthreads();
  if (ends) atomicMin(&last_s, cand);
  __syncthreads();
  const int last = last_s;
  // 256 threads: D / 8 to a row's dims, `lanes` to its parts, the rest to rows
  constexpr int kPer = D / 8;
  const int n_part = last - c + 1;
  const int lanes = n_part > 16 ? 16 : n_part > 4 ? 4 : 1, rows = 256 / kPer / lanes;
  const int d0 = (threadIdx.x % kPer) * 8, pl = threadIdx.x / kPer % lanes,
            rl = threadIdx.x / kPer / lanes;
  __shared__ float xs[256][9], ts[256];
  for (int i0 = blockIdx.y * rows; i0 < r.rows; i0 += gridDim.y * rows) {
    const int i = min(i0 + rl, r.rows - 1);
    const int tok = i / P.g, hd = i - tok * P.g;
    const int row = tok / P.tt * MROWS + (tok % P.tt) * P.g + hd;
    // four parts at a time, their loads all on their way before the first is used
    float top = -INFINITY, l = 0.f, x[8] = {};
    for (int q0 = c + pl; q0 <= last; q0 += 4 * lanes) {
      float2 ml[4];
      float4 u[4], v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = q0 + j * lanes;
        ml[j] = make_float2(-INFINITY, 0.f);
        u[j] = v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q <= last) {
          const int64_t at = (int64_t)(q == c ? 2 * c + 1 : 2 * q) * (2 * MROWS) + row;
          ml[j] = P.part_ml[at];
          u[j] = *reinterpret_cast<const float4*>(P.part_o + at * D + d0);
          v[j] = *reinterpret_cast<const float4*>(P.part_o + at * D + d0 + 4);
        }
      }
      const float t4 = fmaxf(top, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
      const float z = t4 == -INFINITY ? 0.f : t4, f0 = ex2(top - z);
      top = t4;
      l *= f0;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= f0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = ex2(ml[j].x - z);
        l += ml[j].y * f;
        x[0] += u[j].x * f;
        x[1] += u[j].y * f;
        x[2] += u[j].z * f;
        x[3] += u[j].w * f;
        x[4] += v[j].x * f;
        x[5] += v[j].y * f;
        x[6] += v[j].z * f;
        x[7] += v[j].w * f;
      }
    }
    const float off = top == -INFINITY ? 0.f : top;
    if (lanes > 1) {                     // the lanes' sums, in the lanes' order
      __syncthreads();
      ts[threadIdx.x] = top;
      xs[threadIdx.x][8] = l;
#pragma unroll
      for (int e = 0; e < 8; ++e) xs[threadIdx.x][e] = x[e];
      __syncthreads();
      if (pl == 0) {
        for (int k = 1; k < lanes; ++k) top = fmaxf(top, ts[threadIdx.x + k * kPer]);
        const float o2 = top == -INFINITY ? 0.f : top;
        const float f0 = ex2(off - o2);
        l *= f0;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= f0;
        for (int k = 1; k < lanes; ++k) {
          const int o = threadIdx.x + k * kPer;
          const float f = ts[o] == -INFINITY ? 0.f : ex2(ts[o] - o2);
          l += xs[o][8] * f;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += xs[o][e] * f;
        }
      }
    }
    if (pl == 0 && i0 + rl < r.rows) {
      const int hq = r.h * P.g + hd;
      const bool none = top == -INFINITY;
      float f = 1.0f;
      if (P.sink) f = join_sink(P.sink[hq], top, l);
      f = l == 0.f ? 0.f : f / l;
      uint4 w;
      w.x = pack16<F16>(x[0] * f, x[1] * f);
      w.y = pack16<F16>(x[2] * f, x[3] * f);
      w.z = pack16<F16>(x[4] * f, x[5] * f);
      w.w = pack16<F16>(x[6] * f, x[7] * f);
      uint16_t* out = reinterpret_cast<uint16_t*>(const_cast<void*>(P.out.p)) +
                      (int64_t)(r.tok0 + tok) * P.out.tok + (int64_t)hq * P.out.head + d0;
      *reinterpret_cast<uint4*>(out) = w;
      if (P.lse && d0 == 0)
        P.lse[(int64_t)(r.tok0 + tok) * P.Hq + hq] = log_sum(top, l, none, P.sink, hq);
    }
  }
}

// ---------------------------------------------------------------- host side

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

template <int D, bool F16, bool SPARSE, bool TURN, bool LONG>
cudaError_t launch(const KvAttnParams& P, const CUtensorMap& q, const CUtensorMap& k,
                   const CUtensorMap& v, int grid, int dev, cudaStream_t st) {
  const size_t smem = sizeof(Smem<D, SPARSE>);
  static_assert(sizeof(Smem<D, SPARSE>) <= 232448, "shared memory of a CTA");
  static unsigned long long configured = 0;
  if (dev >= 64 || !(configured & (1ull << dev))) {
    const cudaError_t e =
        cudaFuncSetAttribute(kv_attn_kernel<D, F16, SPARSE, TURN, LONG>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured |= 1ull << dev;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(NTHREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kv_attn_kernel<D, F16, SPARSE, TURN, LONG>, P, q, k, v);
  if (e != cudaSuccess) return e;
  // rows of an item: at most two tiles, at most the call's tokens
  cfg.gridDim = dim3(grid, std::min(16, std::min(P.b.T, 2 * P.tt) * P.g), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_merge_kernel<D, F16>, P, grid);
}

// The most blocks that a slot can be given of an item: those of the table, of the
// windows of an item's tokens, or those that they can select; half of them where
// no item has two tiles (and a window of a joined selection one more).
int64_t most_blocks(const KvAttnParams& P) {
  const int64_t tokens = std::min(P.b.T, 2 * P.tt);
  int64_t n = P.b.bps;
  if (P.n_win) n = std::min<int64_t>(n, (P.n_win + tokens - 2) / NK + 2);
  if (P.sparse) n = std::min<int64_t>(n, tokens * ((int64_t)P.n_sel + P.n_local));
  return P.b.T <= P.tt ? (n + P.b.bps / kWindow + 2) / 2 : n;
}

}  // namespace

cudaError_t launch_kv_attn(const KvAttnParams& params, cudaStream_t st) {
  KvAttnParams P = params;
  auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!enc) return cudaErrorNotSupported;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // tokens a tile: as many as fill its 128 rows; sparse tiles name their tokens
  // by the bits of a word, 32 for the two tiles
  P.tt = MROWS / P.g;
  if (P.sparse && P.tt > 16) P.tt = 16;
  const CUtensorMapDataType ty =
      P.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t ones[3] = {1, 1, 1};
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)P.d, (cuuint64_t)P.Hq, (cuuint64_t)P.b.T};
    const cuuint64_t strides[2] = {(cuuint64_t)P.q.head * 2, (cuuint64_t)P.q.tok * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)P.g, (cuuint32_t)P.tt};
    if (enc(&mq, ty, 3, const_cast<void*>(P.q.p), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[2] = {(cuuint64_t)P.d, (cuuint64_t)(P.b.n_blocks * P.Hkv * NK)};
    const cuuint64_t strides[1] = {(cuuint64_t)P.d * 2};
    const cuuint32_t box[2] = {64, NK};
    if (enc(i ? &mv : &mk, ty, 2, const_cast<void*>(i ? P.v_cache : P.k_cache), dims, strides, box,
            ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const int grid = sms < kKvMaxCtas ? sms : kKvMaxCtas;
  // Decode steps (sequences of 16 rows on average) on the kernel that can turn its
  // products.  It is not the only one because of the longer code: 2048 tokens on
  // 32768 would take 1755 us there, 1725 on the other; a mixed batch of 9
  // sequences 53.3 and 49.5.
  const bool turn = (int64_t)P.b.T * P.g <= (int64_t)P.b.B * kTurnedRows;
  // Calls that can give a slot more blocks than O takes up at once on the kernel
  // that adds O up (2048 tokens on 131072: 9.53 ms without, 9.66 with; 32 steps of up
  // to 131072 1.29 and 1.29; 64 steps on selected blocks 111.8 us and 113.7).  It is
  // not the only one because of its other loop: a mixed batch of 9 sequences 51.3
  // and 51.6 us, four prompts of up to 4096 450 and 457.
  const bool many = most_blocks(P) > kFold;
#define KV_LAUNCH(D, F, S)                                                    \
  (turn ? many ? launch<D, F, S, true, true>(P, mq, mk, mv, grid, dev, st)    \
               : launch<D, F, S, true, false>(P, mq, mk, mv, grid, dev, st)   \
   : many ? launch<D, F, S, false, true>(P, mq, mk, mv, grid, dev, st)        \
          : launch<D, F, S, false, false>(P, mq, mk, mv, grid, dev, st))
  if (P.d == 128) {
    if (P.sparse) return P.f16 ? KV_LAUNCH(128, true, true) : KV_LAUNCH(128, false, true);
    return P.f16 ? KV_LAUNCH(128, true, false) : KV_LAUNCH(128, false, false);
  }
  if (P.sparse) return P.f16 ? KV_LAUNCH(64, true, true) : KV_LAUNCH(64, false, true);
  return P.f16 ? KV_LAUNCH(64, true, false) : KV_LAUNCH(64, false, false);
#undef KV_LAUNCH
}

}  // namespace v4a
