// Attention over a paged key/value cache on tcgen05, with an optional prefix
// of keys that all sequences of the batch share.
//
// Work is cut into items: the keys of one sequence (or the prefix) for one key
// head and up to two 128-row query tiles. A query tile stacks the G = H / Hkv
// query heads of its tokens (row = token * G + head), and for the prefix the
// tokens of all sequences, so its keys and values are read once for the
// batch. The items' 128-key tiles, laid end to end, are split evenly over one
// CTA per SM, whatever the lengths are: a CTA runs the end of an item, whole
// items, and the beginning of another. What a CTA computes of a split item is
// a partial result (unnormalised O, row maximum, row sum) in the workspace,
// and a second kernel joins the partials of each row. All lengths are read on
// the device, so a captured call follows them.
//
// Where a sequence has several items per key head, a team of CTAs takes
// neighbouring ones over the same keys in step, so that a key tile comes from
// HBM once for the team (find_share).
//
// One CTA, 384 threads, the hand-off and tensor-memory layout of the FP8
// attention kernel:
//   warp 10: walks the CTA's share and posts its pieces of items in a ring in
//     shared memory, ahead of the others;
//   warp 11: loads the pieces' query tiles by TMA;
//   warp 8: loads K_t and V_t, key tile by key tile (one box per page and 64
//     channels), into a ring of 32 KB slots, past the ends of pieces;
//   warp 9: allocates TMEM and issues the products: S = Q_i K_t^T (SS) into
//     one S buffer, O_i += P_i V_t (TS, P_i in tensor memory); Q K^T of the next
//     key tile goes ahead of the P V of this one, also across pieces;
//   warps 0-3 / 4-7: softmax of query tile 0 / 1 (thread = query row = TMEM
//     lane). A piece of one query tile takes the two groups in turn, so the
//     output of one piece overlaps the products of the next.
//
// Measured and bound by (152 SMs): single rows, HBM: 8 of up to 58,758 keys, 42
// heads, 1.40 ms (7.2 TB/s); 64 of 4,096 keys, 40 heads on 8, 165 us (6.5 TB/s).
// Pages of 16 keys, the loading warp: a box of 2 KB takes it about 100 cycles (96
// rows of up to 8,191 keys, 32 heads on 4: 165 us; pages of 32 and more 139 us, 6.2
// TB/s). Chunks, the chain through the one S buffer: product 512 cycles, seen 200,
// read 250, seen 200, twice per key tile and two query tiles, 2,700 cycles against
// 2,048 of products (1,896 rows of 58,758 keys, 42 heads: 2,853 thousand cycles, 1.54 to
// 1.82 ms with the clock that the power cap leaves, 1,560 to 1,320 TFLOP/s; of 16,384
// keys, 840 thousand, 1,500). Short items, instruction fetch: the kernel is 125 KB, and an
// item runs a small part of it once (6 causal chunks of up to 901 rows and 6,007
// keys, 32 heads on 8: 141 us, products 69).
#include <algorithm>

#include "h3_attn_common.cuh"

namespace h3 {
namespace {

// Ring of 32 KB slots in the order K_0 K_1 V_0 K_2 V_1 ..: the order of use, so
// that no V waits in the ring for longer than the products need it.
constexpr int PA_SLOTS = 5;
__device__ __forceinline__ int k_seq(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int v_seq(int t) { return 2 * t + 2; }
constexpr int PA_PIECES = 8;   // pieces posted ahead
constexpr int PA_MAX_CTAS = 160;
constexpr int PA_CTRL_BYTES = 1024;
// A query tile of so many tokens is loaded token by token; so many rows of a warp
// are stored by themselves (store_transposed); so many rows of a query tile lie in
// all four lane quarters (softmax_tile_quad).
constexpr int PA_FEW_TOKENS = 4, PA_FEW_ROWS = 8, PA_QUAD_ROWS = 8;
// 12 warps: with three on each SM sub-partition the launch gives every thread
// 168 registers; warps 8-11 hand most of theirs to the softmax warps, which
// hold a row's 128 scores and 64 packed weights (168: 508 bytes of spills)
constexpr int PA_THREADS = 384;
constexpr int PA_REGS_SOFTMAX = 192, PA_REGS_OTHER = 120;
static_assert(2 * PA_REGS_SOFTMAX + PA_REGS_OTHER <= 3 * 168, "registers of the launch");
constexpr size_t PA_SMEM_BYTES = 1024 + (PA_SLOTS + 2) * TILE_BYTES + PA_CTRL_BYTES;
static_assert(PA_SMEM_BYTES <= 227 * 1024, "paged attention shared memory");

enum BarPA {
  PA_KV_FULL = 0,
  PA_KV_EMPTY = PA_KV_FULL + PA_SLOTS,
  PA_Q_FULL = PA_KV_EMPTY + PA_SLOTS,
  PA_Q_EMPTY = PA_Q_FULL + 2,  // last Q K^T done (commit), its shared memory not needed (4 warps)
  PA_S = PA_Q_EMPTY + 2,       // S written for query tile i (MMA commit)
  PA_SFREE = PA_S + 2,         // S read by its softmax (4 warp arrivals)
  PA_P = PA_SFREE + 2,         // P_i written (4 warp arrivals)
  PA_PVD = PA_P + 2,           // P_i V done (MMA commit)
  PA_PC_FULL = PA_PVD + 2,     // piece posted
  PA_PC_EMPTY = PA_PC_FULL + PA_PIECES,  // piece read (8 softmax warps, MMA warp, loads); of
                                         // several runs: done with their place
  PA_JOIN = PA_PC_EMPTY + PA_PIECES,     // a quarter's result is in shared memory (4 arrivals)
  PA_DRAIN = PA_JOIN + 2,
  PA_BARS
};
constexpr uint32_t TPA_S = 0, TPA_O = 128, TPA_P = 384;

struct PagedArgs {
  PagedBatch b;
  int64_t ld_o;
  __nv_bfloat16* o;
  int H, Hkv, G;
  int tok;           // tokens of one query tile: floor(128 / G)
  int item;          // tokens of an item: those of two query tiles, or of one
  int max_team;      // CTAs of a team, at most
  int total_rows;    // rows of the cache's tensor map: num_pages * Hkv * page_size
  float scale_log2;  // softmax_scale * log2(e)
  int causal;
  const int32_t* prefix_pages;
  int prefix_len;
  int rows_own;      // the rows' own keys are another kernel's: its results are in row_o, row_ml
  // workspace
  int* teams;        // [2] CTAs per team of the two segments
  int4* cut;         // [CTA] the item that goes on after the CTA's share: tok0, ntok (0: none),
                     // key head, last CTA that has a part of it
  int2* spread;      // with a prefix: [segment][T * Hkv] first and last CTA of the item that
                     // begins with token t, at t * Hkv + key head
  float* part_o;     // split items: [slot][part_rows][128]
  float* part_ml;    // [slot][part_rows][2]
  int part_rows;
  float* row_o;      // with a prefix: [segment][T * H][128]
  float* row_ml;     // [segment][T * H][2]
  int ctas;
  DevErr err;
};

// A sequence as the kernels see it: segment 0 is the prefix with the rows of
// the whole batch, segment 1 the sequences' own keys. Row ranges are clamped
// to [0, T), lengths to what the page table holds.
struct SeqInfo {
  int c0, q_len;
  int kv;
  int off;  // row i sees keys j <= off + i (the limit is clamped to kv)
};

__device__ __forceinline__ SeqInfo seq_info(const PagedArgs& a, int seg, int b) {
  const int first = seg == 0 ? 0 : b, last = seg == 0 ? a.b.B : b + 1;
  SeqInfo s;
  s.c0 = min(max(__ldg(a.b.cu_q + first), 0), a.b.T);
  s.q_len = min(max(__ldg(a.b.cu_q + last), s.c0), a.b.T) - s.c0;
  const int cap = a.b.max_pages << a.b.page_log2;
  const int len = seg == 0 ? a.prefix_len : max(__ldg(a.b.kv_len + b), 0);
  s.kv = seg == 0 ? len : min(len, cap);
  s.off = seg == 1 && a.causal ? len - s.q_len : s.kv;
  return s;
}

// 128-key tiles that the query tiles [0, end) of an item's tokens see: at
// least one, so that a row without keys is written too.
__device__ __forceinline__ int key_tiles(const SeqInfo& s, int end_tok) {
  const int lim = min(max(s.off + end_tok, 0), s.kv);
  return max((lim + BKV - 1) >> 7, 1);
}

__device__ __forceinline__ bool uneven(const PagedArgs& a, int seg) { return seg == 1 && a.causal; }

// What beginning an item costs, in key tiles, in the shares: its first scores
// and its output are not hidden behind other products.
constexpr int PA_ITEM_COST = 2;
// An item of up to so many key tiles is not split: it goes to the CTA in whose
// share it begins. One of more than a query tile's rows leaves a large partial result
// (256 KB written and read for two query tiles), so it is kept whole up to more tiles,
// and up to a share's worth, which leaves the CTAs within an item of one another.
// (Against 4 for all: a causal chunk of 618 rows, 64 heads on 8, 33.6 -> 27.6 us; 4 of
// 500 rows and 2,000 keys, 32 on 8, 75 -> 64; 7 of up to 1,469 rows and 2,203 keys, 12
// heads, 85 -> 71; 6 of up to 901 rows and 1,500 keys, 8 heads, 47.6 -> 50.7. Up to a
// share and 4 tiles more: 2 of up to 1,623 rows and 2,230 keys, 12 heads, 46 -> 59.)
constexpr int PA_WHOLE = 4, PA_WHOLE_ROWS = 8, PA_WHOLE_SHARE = 32;
// Least share of a CTA: a partial result costs more than a tile's time (8 rows
// behind 12,000 keys, 16 heads on 2: 18.8 us for 2, 19.6 for 1, 22.8 for 4, 29.8 for 8;
// a row of 12,000 keys, 4 heads: 16.1, 16.3, 17.3, 21.6).
constexpr int PA_MIN_SHARE = 2;

// Cost of one key head of a sequence, for teams of g CTAs (the items of a team
// run over as many key tiles as the one that sees most).
__device__ __forceinline__ int64_t head_cost(const PagedArgs& a, int seg, const SeqInfo& s,
                                              int g) {
  const int item = a.item * g;
  const int n = (s.q_len + item - 1) / item;
  if (n == 0) return 0;
  if (!uneven(a, seg)) return static_cast<int64_t>(n) * (key_tiles(s, s.q_len) + PA_ITEM_COST);
  int64_t sum = static_cast<int64_t>(n) * PA_ITEM_COST;
#pragma unroll 1
  for (int i = 1; i <= n; ++i) sum += key_tiles(s, min(i * item, s.q_len));
  return sum;
}

// Key tiles that are summed in one accumulator. The tensor cores cut an FP32
// accumulator off, towards zero, with every 16 keys: for values of one sign a sum
// over n keys comes out low by up to n 2^-27 of it, and by 4.3 n 10^-9 on average (on
// 2^24 keys of one CTA 7 %; 1.8 % where a quarter of the keys is summed for itself).
// So a part of an item of more tiles is several pieces, one after the other, each of
// which adds its result to that of those before it, in FP32 rounded to nearest (then
// 0.08 and 0.02 %). An instance of the kernel for itself, for tables and prefixes with
// room for so many keys: the code for runs is fetched with every short item (1,024
// rows of 256 keys, 32 heads on 8: 255 us with it, 234 without).
constexpr int PA_RUN = 1024;

// Teams of up to so many CTAs (find_share picks the size).
constexpr int PA_MAX_TEAM = 8;

// A CTA's part of an item, or a run of it, as posted to the other warps.
struct Piece {
  int tok0, ntok;  // tokens (ntok 0: no more pieces)
  int hk;          // key head
  int kt0, kt1;    // key tiles
  int kv;          // keys of the sequence
  int lim0;        // token i of the piece sees min(lim0 + i, kv) keys
  int dest;        // >= 0: partial slot; -1: the output; -2 - seg: the segment's rows
  int b;           // sequence, -1: the prefix
  int before, more;  // RUNS: 0, or there are runs of the part before and after this one
  int pad;
};
static_assert(sizeof(Piece) == 48, "16-byte loads");

// a / b for a >= 0, b > 0; in 32 bits where they fit.
__device__ __noinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0)
    return static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
  return a / b;
}

// This CTA's share of a segment: `cost` units from unit `at` of sequence b on. A
// share is the same cost (`per`) for every team but the last ones. An item of n key tiles is PA_ITEM_COST + n units, of
// which the last n are its key tiles.
struct Share {
  int64_t cost, at, per;
  int b, g;
};

// One key tile of the online softmax of the calling thread's row, in base 2
// with the scale folded in; the scores are in sr, columns >= valid are masked.
// The running maximum is raised only when a row exceeds it by more than
// RESCALE_THRESHOLD (then O and the sum are rescaled), so a weight can be up
// to 2^8; a row that has seen no key yet keeps maximum -inf and sum 0.
// Only rows that exist (row_ok) ask for it: the others hold what was left in
// shared memory, whose scores would have the tiles of a lone row rescaled. The
// weights go to tensor memory rounded to bf16 (the type of V in the product);
// the sum is of the unrounded ones, in FP32. wait_pv: the tile's previous P V
// is done with P and O. Returns false when a wait failed.
template <class WaitPV>
__device__ __forceinline__ bool softmax_tile_paged(uint32_t (&sr)[128], uint32_t tP, uint32_t tO,
                                                   int valid, bool o_live, bool row_ok,
                                                   float scale_log2, float& m, float& l,
                                                   WaitPV&& wait_pv) {
  if (__any_sync(0xffffffffu, valid < BKV)) {
#pragma unroll
    for (int c = 0; c < 128; ++c)
      if (c >= valid) sr[c] = 0xff800000u;
  }
  float ma = -INFINITY, mb = -INFINITY, mc = -INFINITY, md = -INFINITY;
#pragma unroll
  for (int c = 0; c < 128; c += 8) {
    ma = max3f(ma, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
    mb = max3f(mb, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
    mc = max3f(mc, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
    md = max3f(md, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
  }
  const float mx = max3f(ma, mb, fmaxf(mc, md)) * scale_log2;
  bool pv_done = !o_live;
  if (__any_sync(0xffffffffu, row_ok && mx > m + RESCALE_THRESHOLD)) {
    const float m_new = fmaxf(m, mx);
    const float alpha = m_new == m ? 1.0f : ex2_approx(m - m_new);  // 0 from -inf
    l *= alpha;
    if (o_live) {
      if (!wait_pv()) return false;
      pv_done = true;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t ov[16];
        tmem_ld16(tO + c * 16, ov);
        tmem_ld_wait();
        tmem_reg_fence(ov);
#pragma unroll
        for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
        tmem_st16(tO + c * 16, ov);
      }
      tmem_st_wait();
    }
    m = m_new;
  }
  const float neg_m = m == -INFINITY ? 0.f : -m;
  float la = 0.f, lb = 0.f, lc = 0.f, ld = 0.f;
  uint32_t pk[64];
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    float x0, x1;
    ffma2_bc(x0, x1, __uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1]), scale_log2, neg_m);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    if (i & 1)
      fadd2(lc, ld, p0, p1);
    else
      fadd2(la, lb, p0, p1);
    pk[i] = pack_bf16x2(p0, p1);
  }
  l += (la + lb) + (lc + ld);
  if (!pv_done && !wait_pv()) return false;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    tmem_st16(tP + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(&pk[c * 16]));
  tmem_st_wait();
  return true;
}

// The same for a piece of at most PA_QUAD_ROWS rows, which lie in all four lane
// quarters of the query tile: warp w takes keys 32 w .. 32 w + 31 of the key
// tile, with a maximum, sum and O of its own (its other weights in tensor memory
// are 0); the four are joined when the piece ends. A quarter of the latency and
// of the code of a warp that takes a row's 128 keys alone. The code counts: short
// items run every path of this kernel once in a few microseconds, and it is
// longer than what an SM keeps of it (64 rows of 256 keys, 42 heads, under a table of
// more: 73 us against 90 without; 1,024 of them, 32 heads on 8: 237 / 320; 32 rows behind
// 6,000 keys, 32 on 8: 27.6 / 29.3; 96 rows of up to 8,191 keys, 32 on 4: 164 / 170).
template <class WaitPV, class FreeS>
__device__ __forceinline__ bool softmax_tile_quad(uint32_t tS, uint32_t tP, uint32_t tO, int valid,
                                                  bool o_live, bool row_ok, float scale_log2,
                                                  float& m, float& l, WaitPV&& wait_pv,
                                                  FreeS&& free_s) {
  uint32_t x[32];
  tmem_ld32(tS, x);
  tmem_ld_wait();
  tmem_reg_fence(x);
  free_s();
  if (__any_sync(0xffffffffu, valid < 32)) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= valid) x[i] = 0xff800000u;
  }
  float ma = -INFINITY, mb = -INFINITY;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    ma = max3f(ma, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
    mb = max3f(mb, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
  }
  const float mx = fmaxf(ma, mb) * scale_log2;
  const bool raise = __any_sync(0xffffffffu, row_ok && mx > m + RESCALE_THRESHOLD);
  float alpha = 1.0f;
  if (raise) {
    const float m_new = fmaxf(m, mx);
    if (m_new != m) alpha = ex2_approx(m - m_new);  // 0 from -inf
    l *= alpha;
    m = m_new;
  }
  const float neg_m = m == -INFINITY ? 0.f : -m;
  float la = 0.f, lb = 0.f;
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    ffma2_bc(x0, x1, __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]), scale_log2, neg_m);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    fadd2(la, lb, p0, p1);
    pk[i] = pack_bf16x2(p0, p1);
  }
  l += la + lb;
  if (o_live && !wait_pv()) return false;
  if (raise && o_live) {
#pragma unroll 1
    for (int c = 0; c < 128; c += 16) {
      uint32_t ov[16];
      tmem_ld16(tO + c, ov);
      tmem_ld_wait();
      tmem_reg_fence(ov);
#pragma unroll
      for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
      tmem_st16(tO + c, ov);
    }
  }
  tmem_st16(tP, pk);
  tmem_st_wait();
  return true;
}

// Adds what the runs of a part before this one have of the calling thread's row, at
// `to` and `ml` in the workspace, to what this one has, maximum and sum (m, l) and O in
// tensor memory (`first`: there is none before it), and leaves that there for the next
// run (keep) or as this one's result. By the whole warp.
__device__ __noinline__ float2 join_runs(uint32_t tO, float* to, float2* ml, bool row_ok, bool first,
                                         bool keep, float m, float l) {
  float c = 0.f, w = 1.f;  // weights of the runs before and of this one
  if (!first && row_ok) {
    const float2 x = *ml;
    const float top = fmaxf(x.x, m);
    c = x.x == top ? 1.f : ex2_approx(x.x - top);  // (equal: -inf too, no key so far)
    w = m == top ? 1.f : ex2_approx(m - top);
    m = top;
    l = fmaf(x.y, c, l * w);
  }
  if (keep && row_ok) *ml = make_float2(m, l);
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    uint32_t ov[16];
    tmem_ld16(tO + i * 16, ov);
    tmem_ld_wait();
    tmem_reg_fence(ov);
    float4* at = reinterpret_cast<float4*>(to) + i * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(ov[4 * j + e]) * w;
      if (!first && row_ok) {
        const float4 y = at[j];
        x[0] = fmaf(y.x, c, x[0]);
        x[1] = fmaf(y.y, c, x[1]);
        x[2] = fmaf(y.z, c, x[2]);
        x[3] = fmaf(y.w, c, x[3]);
      }
      if (keep && row_ok) at[j] = make_float4(x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) ov[4 * j + e] = __float_as_uint(x[e]);
    }
    if (!keep) tmem_st16(tO + i * 16, ov);
  }
  if (!keep) tmem_st_wait();
  __syncwarp();  // another lane may write to the place next
  return make_float2(m, l);
}

// Writes 64 bytes (four 16-byte units, w) of every lane's row at byte `at`, with
// stores of 64 bytes of eight rows each: one that takes 16 bytes of 32 rows
// touches 32 lines and holds the load/store unit for as many cycles. For
// PA_FEW_ROWS rows of a warp and fewer there is nothing to gain. Groups of four
// lanes transpose their units, then to[j] (the row of lane j of the group, at this
// lane's unit) gets what is now in unit j, for j < left.
__device__ __forceinline__ void store_transposed(uint32_t (&w)[16], char* const (&to)[4], int left,
                                                 int at) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s <= 2; ++s) {  // partner lane ^ s holds the other half of each pair of units
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & s) continue;
      const bool hi = (lane & s) != 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t &lo_w = w[i * 4 + k], &hi_w = w[(i + s) * 4 + k];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? lo_w : hi_w, s);
        if (hi)
          lo_w = got;
        else
          hi_w = got;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left)
      *reinterpret_cast<uint4*>(to[j] + at) =
          make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// RUNS: parts may be longer than PA_RUN.
template <bool RUNS>
__global__ void __launch_bounds__(PA_THREADS, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmQ1,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const PagedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sKV = smem;
  uint8_t* sQ = smem + PA_SLOTS * TILE_BYTES;
  uint8_t* ctrl = sQ + 2 * TILE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ctrl);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + PA_BARS + 1);
  Piece* ring = reinterpret_cast<Piece*>(ctrl + 384);   // [PA_PIECES]
  static_assert((PA_BARS + 1) * 8 + 16 <= 384 && 384 + PA_PIECES * sizeof(Piece) <= PA_CTRL_BYTES,
                "control region");
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // the joining kernel may be set up while this one runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // a barrier per thread (one thread for all of them: 2,400 cycles)
  if (threadIdx.x < PA_BARS) {
    const int i = threadIdx.x;
    uint32_t count = 1;
    if (i >= PA_SFREE && i < PA_PVD) count = 4;
    if (i >= PA_PC_EMPTY && i < PA_JOIN) count = 11;
    if (i >= PA_JOIN && i < PA_DRAIN) count = 4;
    if (i >= PA_Q_EMPTY && i < PA_S) count = 5;
    mbar_init(bar(i), count);
    fence_mbar_init();
  }
  if (threadIdx.x == PA_THREADS - 32) {
    tma_prefetch_desc(&tmQ1);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PA_REGS_OTHER));
    if (warp == 10) {
      // ------------------------------------------------------- the share
      // Every lane sums the cost of a run of sequences; the lane whose run holds
      // the share's beginning finds where. Teams are of the size with the least
      // time, a tile of a lone CTA taken as 6 and of a team's as 5: a 64 KB key
      // tile takes a CTA about 2,300 cycles of products for two query tiles, and
      // about 2,800 where every CTA reads it from HBM for itself. (Loops are
      // kept rolled: the instruction cache is short for this kernel.)
      auto find_share = [&](int seg) {
        const int n = seg == 0 ? 1 : a.b.B;
        const int run = (n + 31) / 32;
        const int b0 = min(lane * run, n), b1 = min(b0 + run, n);
        Share sh{0, 0, 1, 0, 1};
        int64_t mine = 0;
        float least = 0.f;
        int most = 1;  // no team is larger than the items of a sequence
        SeqInfo s{};
#pragma unroll 1
        for (int g = 1; g <= most; g += g < 4 ? 1 : 2) {
          int64_t own = 0;
          int rows = 0;
#pragma unroll 1
          for (int b = b0; b < b1; ++b) {
            if (g == 1 || run > 1) s = seq_info(a, seg, b);
            own += head_cost(a, seg, s, g);
            rows = max(rows, s.q_len);
          }
          if (g == 1) {
            rows = __reduce_max_sync(0xffffffffu, rows);
            most = min(min(a.max_team, a.ctas), (rows + a.item - 1) / a.item);
          }
          own *= a.Hkv;
          float W = static_cast<float>(own);
#pragma unroll
          for (int d = 16; d >= 1; d >>= 1) W += __shfl_xor_sync(0xffffffffu, W, d);
          const float cost = ceilf(W / static_cast<float>(a.ctas / g)) * (g == 1 ? 6.f : 5.f);
          if (g == 1 || cost < least) {
            least = cost;
            mine = own;
            sh.g = g;
          }
        }
        int64_t total = mine;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        const int teams = a.ctas / sh.g, team = static_cast<int>(blockIdx.x) / sh.g;
        sh.per = max(div64(total + teams - 1, teams), int64_t{PA_MIN_SHARE});
        const int64_t begin = team * sh.per;
        if (team >= teams || begin >= total) return sh;
        sh.cost = min(sh.per, total - begin);
        int64_t at = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, at, d);
          if (lane >= d) at += v;
        }
        at -= mine;
        const uint32_t who = __ballot_sync(0xffffffffu, begin >= at && begin < at + mine);
        int b = b0;
        if (who >> lane & 1u) {
#pragma unroll 1
          for (; b < b1; ++b) {
            const int64_t c = head_cost(a, seg, seq_info(a, seg, b), sh.g) * a.Hkv;
            if (begin < at + c) break;
            at += c;
          }
        }
        const int src = __ffs(who) - 1;
        sh.b = __shfl_sync(0xffffffffu, b, src & 31);
        sh.at = begin - __shfl_sync(0xffffffffu, at, src & 31);
        return sh;
      };
      int np = 0;
      auto post = [&](const Piece& p) {
        const int r = np % PA_PIECES;
        if (!mbar_wait_warp(bar(PA_PC_EMPTY + r), ((np / PA_PIECES) & 1) ^ 1, a.err,
                            ERR_WAIT_ATTN_PRODUCER))
          return false;
        if (lane == 0) {
          ring[r] = p;
          mbar_arrive(bar(PA_PC_FULL + r));
        }
        __syncwarp();
        ++np;
        return true;
      };
      bool ok = true;
      const int first_seg = a.prefix_len > 0 ? 0 : 1;
#pragma unroll 1
      for (int seg = first_seg; ok && seg < (a.rows_own ? 1 : 2); ++seg) {
        const Share sh = find_share(seg);
        if (blockIdx.x == 0 && lane == 0) a.teams[seg] = sh.g;
        const int member = static_cast<int>(blockIdx.x) % sh.g;
        const int item = a.item;
        const int n = seg == 0 ? 1 : a.b.B;
        int4 cut = make_int4(0, 0, 0, 0);
        int64_t left = sh.cost;
        int b = sh.b, hk = 0, qg = 0, u = 0, items = 0, groups = 0;  // u: unit of the item
        SeqInfo s{};
        auto group_cost = [&]() {
          return key_tiles(s, min((qg + 1) * item * sh.g, s.q_len)) + PA_ITEM_COST;
        };
        auto enter = [&]() {
          s = seq_info(a, seg, b);
          items = (s.q_len + item - 1) / item;
          groups = (items + sh.g - 1) / sh.g;
        };
        if (left > 0) {
          enter();
          const int64_t per_head = max(head_cost(a, seg, s, sh.g), int64_t{1});
          hk = static_cast<int>(div64(sh.at, per_head));
          int64_t r = sh.at - hk * per_head;
          if (!uneven(a, seg)) {
            const int nk = group_cost();
            qg = static_cast<int>(div64(r, nk));
            r -= static_cast<int64_t>(qg) * nk;
          } else {
#pragma unroll 1
            for (int nk = group_cost(); r >= nk && qg + 1 < groups; nk = group_cost()) {
              r -= nk;
              ++qg;
            }
          }
          u = static_cast<int>(r);
        }
#pragma unroll 1
        while (ok && left > 0) {
          const int cost = group_cost();
          const int most = s.q_len * a.G > BQ
                               ? max(PA_WHOLE_ROWS, static_cast<int>(min(sh.per, int64_t{PA_WHOLE_SHARE})))
                               : PA_WHOLE;
          const bool small = cost <= most + PA_ITEM_COST;
          const int rest = cost - u;
          const int take = small ? rest : static_cast<int>(min(static_cast<int64_t>(rest), left));
          const int qt = qg * sh.g + member;
          const int nk = key_tiles(s, min((qt + 1) * item, s.q_len));  // of this CTA's item
          const int kt0 = small ? 0 : max(u - PA_ITEM_COST, 0);
          const int kt1 = min(max(u + take - PA_ITEM_COST, 0), nk);
          if (qt < items && kt0 < kt1 && !(small && u > 0)) {
            Piece p{};
            p.hk = hk;
            p.b = seg == 0 ? -1 : b;
            p.kt0 = kt0;
            p.kt1 = kt1;
            p.tok0 = s.c0 + qt * item;
            p.ntok = min(item, s.q_len - qt * item);
            p.kv = s.kv;
            p.lim0 = uneven(a, seg) ? s.off + qt * item + 1 : s.kv;
            const bool whole = p.kt0 == 0 && p.kt1 == nk;
            p.dest = !whole ? ((seg - first_seg) * PA_MAX_CTAS + static_cast<int>(blockIdx.x)) * 2 +
                                  (p.kt0 > 0 ? 0 : 1)
                            : (first_seg == 0 ? -2 - seg : -1);
            if (p.kt0 == 0) {
              // the shares that the rest of the item falls into
              const int more = static_cast<int>(div64(nk - p.kt1 + sh.per - 1, sh.per));
              const int last = static_cast<int>(blockIdx.x) + more * sh.g;
              if (!whole) cut = make_int4(p.tok0, p.ntok, hk, last);
              if (first_seg == 0 && lane == 0)
                a.spread[(static_cast<int64_t>(seg) * a.b.T + p.tok0) * a.Hkv + hk] =
                    make_int2(blockIdx.x, last);
            }
            if constexpr (RUNS) {
#pragma unroll 1
              do {
                p.kt1 = min(p.kt0 + PA_RUN, kt1);
                p.more = kt1 - p.kt1;
                ok = post(p);
                p.before = 1;
                p.kt0 = p.kt1;
              } while (ok && p.more > 0);
            } else {
              ok = post(p);
            }
          }
          left -= take;
          u += take;
          if (u < cost) break;  // the end of the share
          u = 0;
          if (++qg == groups) {
            qg = 0;
            if (++hk == a.Hkv) {
              hk = 0;
              groups = 0;
#pragma unroll 1
              while (left > 0 && groups == 0 && ++b < n) enter();
              if (b >= n) break;
            }
          }
        }
        if (seg == 1 && lane == 0) a.cut[blockIdx.x] = cut;
      }
      if (ok) post(Piece{});
    } else if (warp == 8) {
      // ------------------------------------------------------- TMA loads
      const int nbox = BKV >> a.b.page_log2;  // pages of a key tile
      const int box = lane & (nbox - 1), half = lane / nbox;
      const uint32_t box_dst = half * BOX_BYTES + ((box << a.b.page_log2) << 7);
      int np = 0;
      bool ok = true;
      struct Tile {
        int kt, kt1, kv, hk;
        const int32_t* pages;
        int page;  // this lane's page, -1: none
      };
      // the key tile after d (of the next piece when d is its piece's last),
      // with the lane's page on its way; false: no more, or a wait failed
      auto advance = [&](Tile& d) {
        if (++d.kt >= d.kt1) {
          const int r = np % PA_PIECES;
          if (!mbar_wait_warp(bar(PA_PC_FULL + r), (np / PA_PIECES) & 1, a.err,
                              ERR_WAIT_ATTN_PRODUCER))
            return ok = false;
          const Piece& p = ring[r];
          const int ntok = p.ntok, b = p.b;
          d.kt = p.kt0;
          d.kt1 = p.kt1;
          d.kv = p.kv;
          d.hk = p.hk;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(PA_PC_EMPTY + r));
          if (ntok == 0) return false;
          d.pages = b < 0 ? a.prefix_pages
                          : a.b.page_table + static_cast<int64_t>(b) * a.b.max_pages;
          ++np;
        }
        // a page is loaded when it begins below the sequence's end
        const int i = d.kt * nbox + box;
        d.page = half < 2 && (static_cast<int64_t>(i) << a.b.page_log2) < d.kv ? __ldg(d.pages + i)
                                                                              : -1;
        return true;
      };
      uint32_t used = 0, parity = 0;  // per slot: loaded at all; phase of its last load
      // K or V of key tile d, the seq-th load
      auto load = [&](const Tile& d, const CUtensorMap* map, int seq) {
        const int live = min(nbox, (d.kv - d.kt * BKV + (1 << a.b.page_log2) - 1) >> a.b.page_log2);
        const uint32_t bytes = static_cast<uint32_t>(max(live, 0)) << (a.b.page_log2 + 8);
        // a page outside the pool: a row past the map's end, which loads zeros
        const int row = d.page >= 0 && d.page < a.b.num_pages
                            ? (d.page * a.Hkv + d.hk) << a.b.page_log2
                            : a.total_rows;
        const int slot = seq % PA_SLOTS;
        if (!mbar_wait_warp(bar(PA_KV_EMPTY + slot), ((seq / PA_SLOTS) & 1) ^ 1, a.err,
                            ERR_WAIT_ATTN_PRODUCER))
          return false;
        const uint32_t full = bar(PA_KV_FULL + slot);
        if (lane == 0) {
          if (bytes > 0)
            mbar_arrive_expect_tx(full, bytes);
          else
            mbar_arrive(full);
        }
        __syncwarp();
        used |= 1u << slot;
        parity = (parity & ~(1u << slot)) | static_cast<uint32_t>((seq / PA_SLOTS) & 1) << slot;
        if (half < 2 && box < live)
          tma_load_2d(smem_u32(sKV + slot * TILE_BYTES) + box_dst, map, full, half * 64, row);
        return true;
      };
      Tile cur{}, nxt{};
      bool have = false;
      for (int t = -1; ok; ++t) {  // K of tile t + 1, then V of tile t
        const bool more = advance(nxt);
        if (!ok || !(have || more)) break;
#pragma unroll 1
        for (int v = more ? 0 : 1; ok && v <= (have ? 1 : 0); ++v)
          ok = load(v ? cur : nxt, v ? &tmV : &tmK, v ? v_seq(t) : k_seq(t + 1));
        cur = nxt;
        have = more;
        if (!have) break;
      }
      // no copy of this CTA may still be landing when it exits
      if (lane == 0) {
        const uint64_t t0 = globaltimer_ns();
        const uint64_t lim = drain_limit_ns(a.err);
        for (int slot = 0; slot < PA_SLOTS; ++slot)
          if (used >> slot & 1u) mbar_wait_drain(bar(PA_KV_FULL + slot), parity >> slot & 1u, t0, lim);
      }
    } else if (warp == 11) {
      // ------------------------------------------------------ query tiles
      // a query tile of few tokens is loaded token by token (tmQ1): the box of a
      // whole tile would read up to 128 rows for one (64 single rows behind a
      // shared prefix, 42 heads: its loads held up those of the keys)
      uint32_t phase = 3, used = 0;  // per query tile: parity of Q_EMPTY; loaded at all
      bool ok = true;
      for (int np = 0; ok; ++np) {
        const int r = np % PA_PIECES;
        if (!mbar_wait_warp(bar(PA_PC_FULL + r), (np / PA_PIECES) & 1, a.err,
                            ERR_WAIT_ATTN_PRODUCER))
          break;
        const int tok0 = ring[r].tok0, ntok = ring[r].ntok, hk = ring[r].hk;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PA_PC_EMPTY + r));
        if (ntok == 0) break;
        const bool two = ntok > a.tok;
#pragma unroll 1
        for (int g = two ? 0 : np & 1; g <= (two ? 1 : np & 1); ++g) {
          ok = mbar_wait_warp(bar(PA_Q_EMPTY + g), phase >> g & 1u, a.err, ERR_WAIT_ATTN_PRODUCER);
          if (!ok) break;
          const uint32_t dst = smem_u32(sQ + g * TILE_BYTES), full = bar(PA_Q_FULL + g);
          const int t0 = tok0 + g * (two ? a.tok : 0);
          const int n = min(ntok - (t0 - tok0), a.tok);
          if (n * a.G <= PA_QUAD_ROWS) {  // in all four lane quarters
            if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(n * a.G) * 1024);
            __syncwarp();
            const int w = lane & 3, h = lane >> 2 & 1;
#pragma unroll 1
            for (int i = lane >> 3; i < n; i += 4)
              tma_load_3d(dst + h * BOX_BYTES + w * 4096 + i * a.G * 128, &tmQ1, full, h * 64,
                          hk * a.G, t0 + i);
          } else if (lane == 0) {
            if (n <= PA_FEW_TOKENS) {
              mbar_arrive_expect_tx(full, static_cast<uint32_t>(n * a.G) * 256);
#pragma unroll 1
              for (int i = 0; i < n; ++i) {
                tma_load_3d(dst + i * a.G * 128, &tmQ1, full, 0, hk * a.G, t0 + i);
                tma_load_3d(dst + i * a.G * 128 + BOX_BYTES, &tmQ1, full, 64, hk * a.G, t0 + i);
              }
            } else {
              mbar_arrive_expect_tx(full, static_cast<uint32_t>(a.tok * a.G) * 256);
              tma_load_3d(dst, &tmQ, full, 0, hk * a.G, t0);
              tma_load_3d(dst + BOX_BYTES, &tmQ, full, 64, hk * a.G, t0);
            }
          }
          __syncwarp();
          phase ^= 1u << g;
          used |= 1u << g;
        }
      }
      if (lane == 0) {  // no copy may still be landing when the CTA exits
        const uint64_t t0 = globaltimer_ns();
        for (int g = 0; g < 2; ++g)
          if (used >> g & 1u)
            mbar_wait_drain(bar(PA_Q_FULL + g), phase >> g & 1u, t0, drain_limit_ns(a.err));
      }
    } else if (warp == 9) {
      // ------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc_qk = idesc_bf16_f32(BQ, BKV, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BQ, DH, true);
      const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = sdesc_sw128(smem_u32(sKV), 16, 1024);
      const uint64_t dv = sdesc_sw128(smem_u32(sKV), BOX_BYTES, 1024);
      // parities of the phases waited for next, one bit per barrier (an array
      // indexed by query tile would live in local memory, on the issue path)
      uint32_t phase = 0;
      auto wait = [&](int b) {
        const bool done = mbar_wait_warp(bar(b), phase >> b & 1u, a.err, ERR_WAIT_ATTN_MMA);
        phase ^= 1u << b;
        return done;
      };
      static_assert(PA_PVD <= 32, "a bit per barrier");
      struct Tile {
        int g0;  // query tile, or the first of two
        bool two, first, last;
      };
      int np = 0, left = 0;
      Tile proto{0, false, false, false};
      bool ok = true;
      // the next key tile; false: no more, or a wait failed (ok false)
      auto next_tile = [&](Tile& d) {
        bool first = false;
        if (left == 0) {
          const int r = np % PA_PIECES;
          if (!mbar_wait_warp(bar(PA_PC_FULL + r), (np / PA_PIECES) & 1, a.err, ERR_WAIT_ATTN_MMA))
            return ok = false;
          // through a warp reduction, whose result is a uniform value: what
          // follows from it, the products' operands included, then stays in
          // the uniform datapath
          const int ntok = __reduce_max_sync(0xffffffffu, ring[r].ntok);
          left = __reduce_max_sync(0xffffffffu, ring[r].kt1 - ring[r].kt0);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(PA_PC_EMPTY + r));
          if (ntok == 0) return false;
          proto.two = ntok > a.tok;
          proto.g0 = proto.two ? 0 : np & 1;
          ++np;
          first = true;
        }
        d = proto;
        d.first = first;
        d.last = --left == 0;
        return true;
      };
      // slots of the next K_t and V_t to be used: from K_1 and V_0 on every
      // other one of the ring
      int k_slot = k_seq(0), v_slot = v_seq(0);
      bool k_first = true;
      auto step = [](int& slot) { slot += slot < PA_SLOTS - 2 ? 2 : 2 - PA_SLOTS; };
      int last_s = -1;  // query tile whose S is in the buffer
      auto qk = [&](int g, int prev, bool lead, bool tail, bool first, bool last) {  // S = Q_g K_t^T
        if (first && !wait(PA_Q_FULL + g)) return false;
        if (lead && !wait(PA_KV_FULL + k_slot)) return false;
        if (prev >= 0 && !wait(PA_SFREE + prev)) return false;
        tc_fence_after();
        const uint64_t qd = dq + static_cast<uint32_t>(g * (TILE_BYTES >> 4));
        const uint64_t kd = dk + static_cast<uint32_t>(k_slot * (TILE_BYTES >> 4));
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          // 16-byte offset of K step kk (16 channels) in a K-major tile
          const uint32_t off = ((kk >> 2) * BOX_BYTES + (kk & 3) * 32) >> 4;
          mma_ss_el(tmem + TPA_S, qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
        }
        mma_commit_el(bar(PA_S + g));
        if (last) mma_commit_el(bar(PA_Q_EMPTY + g));
        if (tail) {
          mma_commit_el(bar(PA_KV_EMPTY + k_slot));
          if (k_first)
            k_slot = k_seq(1), k_first = false;
          else
            step(k_slot);
        }
        return true;
      };
      auto pv = [&](int g, bool lead, bool tail, uint32_t acc) {  // O_g (+)= P_g V_t
        if (lead && !wait(PA_KV_FULL + v_slot)) return false;
        if (!wait(PA_P + g)) return false;
        tc_fence_after();
        const uint64_t vd = dv + static_cast<uint32_t>(v_slot * (TILE_BYTES >> 4));
#pragma unroll
        for (int kk = 0; kk < BKV / 16; ++kk)  // 16 keys: 8 columns of P, 2 KB of V
          mma_ts_el(tmem + TPA_O + g * 128, tmem + TPA_P + g * 64 + kk * 8,
                    vd + kk * (2048 >> 4), idesc_pv, kk > 0 ? 1u : acc);
        mma_commit_el(bar(PA_PVD + g));
        if (tail) {
          mma_commit_el(bar(PA_KV_EMPTY + v_slot));
          step(v_slot);
        }
        return true;
      };
      // Q K^T of the next key tile before P V of this one; with two query tiles
      // their products alternate, so one's softmax overlaps the other's products
      Tile cur{}, nxt{};
      bool have = false, more = true;  // cur, nxt exist
      while (ok) {
        if (have && cur.two && left >= 2) {
          // the next key tile is of the same piece and not its last: the same
          // four products with everything but the slots known
          uint32_t acc = cur.first ? 0u : 1u;
          do {
            ok = qk(0, 1, true, false, false, false) && pv(0, true, false, acc) &&
                 qk(1, 0, false, true, false, false) && pv(1, false, true, acc);
            acc = 1u;
            --left;
          } while (ok && left >= 2);
          cur.first = false;
          continue;
        }
        more = next_tile(nxt);
        if (!ok || !(have || more)) break;
        // a new piece on a query tile that is still in use: its output first
        const bool out_first = have && more && nxt.first && (cur.two || nxt.two);
        // (rolled: the instruction cache holds the short items' path better, 371
        // against 402 thousand cycles for 64 rows behind a 29,034-key prefix; the
        // steady loop of a long chunk loses 4 %)
#pragma unroll 1
        for (int i = 0; ok && i < 4; ++i) {
          const bool is_qk = out_first ? i >= 2 : (i & 1) == 0;
          const int second = out_first ? i & 1 : i >> 1;
          if (is_qk) {
            if (more && (!second || nxt.two)) {
              const int g = second ? 1 : nxt.g0, prev = last_s;
              last_s = g;
              ok = qk(g, prev, !second, second || !nxt.two, nxt.first, nxt.last);
            }
          } else if (have && (!second || cur.two)) {
            ok = pv(second ? 1 : cur.g0, !second, second || !cur.two, cur.first ? 0u : 1u);
          }
        }
        cur = nxt;
        have = more;
        if (!have) break;
      }
      // every product must be done with shared and tensor memory before the CTA
      // frees them: commit and wait, bounded
      mma_commit_el(bar(PA_DRAIN));
      mbar_wait_drain(bar(PA_DRAIN), 0u, globaltimer_ns(), drain_limit_ns(a.err));
    }
  } else {
    // ---------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PA_REGS_SOFTMAX));
    const int tile = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + TPA_S;
    const uint32_t tO = tmem + lane_base + TPA_O + tile * 128;
    const uint32_t tP = tmem + lane_base + TPA_P + tile * 64;
    const int row_tok = row / a.G, row_head = row % a.G, lane_tok = lane / a.G;
    bool p_clear = false;  // this warp's weights outside its 32 keys are 0
    int joins = 0;   // pieces joined from the four quarters
    // the last piece of several runs, if this warp has not seen it done with their place,
    // which may be this piece's too
    int run_piece = -1;
    int n = 0;       // S tiles of this query tile so far
    int tiles = 0;   // key tiles of this CTA so far
    bool ok = true;
    auto wait_pv = [&](int count) {
      const bool done = mbar_wait_warp(bar(PA_PVD + tile), count & 1, a.err, ERR_WAIT_ATTN_SOFTMAX);
      tc_fence_after();
      return done;
    };
    for (int np = 0; ok; ++np) {
      const int r = np % PA_PIECES;
      if (!mbar_wait_warp(bar(PA_PC_FULL + r), (np / PA_PIECES) & 1, a.err, ERR_WAIT_ATTN_SOFTMAX))
        break;
      const Piece p = ring[r];
      const bool two = p.ntok > a.tok, mine = two || (np & 1) == tile;
      const bool run = RUNS && p.before + p.more > 0;
      __syncwarp();
      if (lane == 0 && !(mine && run)) mbar_arrive(bar(PA_PC_EMPTY + r));
      if (p.ntok == 0) break;
      if (!mine) {
        if (run) run_piece = np;
        tiles += p.kt1 - p.kt0;
        continue;
      }
      const int tok0 = two ? tile * a.tok : 0;                        // within the piece
      const int rows = (two ? (tile ? p.ntok - a.tok : a.tok) : p.ntok) * a.G;
      // rows of this lane quarter's own numbering; a few rows are in all quarters
      const bool quad = rows <= PA_QUAD_ROWS;
      const bool active = quad || quarter * 32 < rows;
      const bool row_ok = (quad ? lane : row) < rows;
      const int tok = tok0 + (quad ? lane_tok : row_tok);
      const int lim = min(max(p.lim0 + tok, 0), p.kv) - (quad ? quarter * 32 : 0);
      // only the results of few rows need the query tile's shared memory
      if (!quad && lane == 0) mbar_arrive(bar(PA_Q_EMPTY + tile));
      // keys past the sequence's end hold anything: their weights are 0, and so
      // their values have to be finite
      auto clear_values = [&](int kt) {
        const int live = p.kv - kt * BKV;  // keys of the tile that exist
        if (live >= BKV) return true;
        const int seq = v_seq(tiles), slot = seq % PA_SLOTS;
        if (!mbar_wait_warp(bar(PA_KV_FULL + slot), (seq / PA_SLOTS) & 1, a.err,
                            ERR_WAIT_ATTN_SOFTMAX))
          return false;
        // eight lanes per 128-byte half of a row
        uint4* v = reinterpret_cast<uint4*>(sKV + slot * TILE_BYTES) + (lane & 7);
        for (int r = max(live, 0) + quarter * 4 + (lane >> 3); r < BKV; r += 16)
          v[r * 8] = v[BOX_BYTES / 16 + r * 8] = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        return true;
      };
      float m = -INFINITY, l = 0.f;
      for (int kt = p.kt0; kt < p.kt1; ++kt, ++tiles, ++n) {
        ok = mbar_wait_warp(bar(PA_S + tile), n & 1, a.err, ERR_WAIT_ATTN_SOFTMAX);
        if (!ok) break;
        tc_fence_after();
        auto free_s = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(PA_SFREE + tile));
        };
        auto pv_before = [&] { return wait_pv(n - 1); };
        const int valid = lim - kt * BKV;
        const bool o_live = kt > p.kt0;
        if (!active) {
          // no row of this warp exists: it takes part in the hand-offs only (and
          // waits for the P V, so that its arrivals stay in step)
          free_s();
          ok = !o_live || pv_before();
        } else if (quad) {
          if (!p_clear) {
            const uint32_t z[16] = {};
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) tmem_st16(tP + c, z);
            tmem_st_wait();
            p_clear = true;
          }
          ok = softmax_tile_quad(tS + quarter * 32, tP + quarter * 16, tO, valid, o_live, row_ok,
                                 a.scale_log2, m, l, pv_before, free_s);
        } else {
          p_clear = false;
          uint32_t sr[128];
          {
            uint32_t (&c0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
            uint32_t (&c1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[32]);
            uint32_t (&c2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[64]);
            uint32_t (&c3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[96]);
            tmem_ld32(tS + 0, c0);
            tmem_ld32(tS + 32, c1);
            tmem_ld32(tS + 64, c2);
            tmem_ld32(tS + 96, c3);
            tmem_ld_wait();
            tmem_reg_fence(sr);
          }
          free_s();
          ok = softmax_tile_paged(sr, tP, tO, valid, o_live, row_ok, a.scale_log2, m, l,
                                  pv_before);
        }
        ok = ok && clear_values(kt);
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PA_P + tile));
      }
      if (!ok || !wait_pv(n - 1)) break;
      if (lim > p.kt0 * BKV) m = fmaxf(m, KEYS_SEEN);
      if (RUNS && run_piece >= 0) {
        ok = mbar_wait_warp(bar(PA_PC_EMPTY + run_piece % PA_PIECES), (run_piece / PA_PIECES) & 1,
                            a.err, ERR_WAIT_ATTN_SOFTMAX);
        if (!ok) break;
        run_piece = -1;
      }
      if (run) {
        if (active) {
          // a part's runs meet where its partial result goes, or where this CTA's last one
          // of the segment will; rows in all lane quarters have four places
          const int slot = p.dest >= 0 ? p.dest
                                       : ((p.dest == -1 ? 0 : -2 - p.dest) * PA_MAX_CTAS +
                                          static_cast<int>(blockIdx.x)) * 2 + 1;
          const int64_t at = static_cast<int64_t>(slot) * a.part_rows + tok0 * a.G +
                             (quad ? quarter * rows + lane : row);
          const float2 x = join_runs(tO, a.part_o + at * DH, reinterpret_cast<float2*>(a.part_ml) + at,
                                     row_ok, p.before == 0, p.more > 0, m, l);
          m = x.x;
          l = x.y;
        }
        run_piece = np;
        if (lane == 0) mbar_arrive(bar(PA_PC_EMPTY + r));
        if (p.more > 0) {
          tc_fence_before();  // O has been read
          if (quad && lane == 0) mbar_arrive(bar(PA_Q_EMPTY + tile));
          continue;
        }
      }
      if (quad) {
        // the four quarters' results meet in the part of the query tile that
        // few rows leave free: row r of quarter w, 512 bytes in the order of
        // 16-byte units XOR r
        uint8_t* sj = sQ + tile * TILE_BYTES + 1024;
        auto unit = [&](int w, int r, int c) {
          return reinterpret_cast<float4*>(sj + (r >> 2) * BOX_BYTES + w * 4096 + (r & 3) * 512) +
                 (c ^ r);
        };
        float2* sml = reinterpret_cast<float2*>(sj + 2048);  // + w * 4096: [row]
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t ov[16];
          tmem_ld16(tO + c * 16, ov);
          tmem_ld_wait();
          tmem_reg_fence(ov);
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *unit(quarter, lane, 4 * c + i) =
                  make_float4(__uint_as_float(ov[4 * i]), __uint_as_float(ov[4 * i + 1]),
                              __uint_as_float(ov[4 * i + 2]), __uint_as_float(ov[4 * i + 3]));
          }
        }
        if (row_ok) sml[quarter * 512 + lane] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PA_JOIN + tile));
        ok = mbar_wait_warp(bar(PA_JOIN + tile), joins & 1, a.err, ERR_WAIT_ATTN_SOFTMAX);
        ++joins;
        if (!ok) break;
        for (int r = quarter; r < rows; r += 4) {
          float2 ml[4];
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            ml[w] = sml[w * 512 + r];
            top = fmaxf(top, ml[w].x);
          }
          float sum = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float f = top == -INFINITY ? 0.f : ex2_approx(ml[w].x - top);
            const float4 x = *unit(w, r, lane);
            sum = fmaf(ml[w].y, f, sum);
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
          }
          const int64_t orow = static_cast<int64_t>(p.tok0 + tok0 + r / a.G);
          const int head = p.hk * a.G + r % a.G;
          if (p.dest == -1) {
            const float inv = top == -INFINITY ? 0.f : 1.0f / sum;  // no key: zeros
            *reinterpret_cast<uint2*>(a.o + orow * a.ld_o + head * DH + lane * 4) =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
          } else {
            const int64_t at = p.dest >= 0
                                   ? static_cast<int64_t>(p.dest) * a.part_rows + tok0 * a.G + r
                                   : (static_cast<int64_t>(-2 - p.dest) * a.b.T + orow) * a.H + head;
            reinterpret_cast<float4*>((p.dest >= 0 ? a.part_o : a.row_o) + at * DH)[lane] = o;
            if (lane == 0)
              *reinterpret_cast<float2*>((p.dest >= 0 ? a.part_ml : a.row_ml) + at * 2) =
                  make_float2(top, sum);
          }
        }
        // O has been read before a later piece's P V overwrites it, and the query
        // tile may be loaded again
        tc_fence_before();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PA_Q_EMPTY + tile));
        continue;
      }
      if (!active) continue;
      const int64_t orow = static_cast<int64_t>(p.tok0 + tok);
      const int head = p.hk * a.G + row_head;
      char* dst;
      if (p.dest == -1) {
        dst = reinterpret_cast<char*>(a.o + orow * a.ld_o + head * DH);
      } else {
        int64_t at;
        float* ml;
        if (p.dest >= 0) {
          at = static_cast<int64_t>(p.dest) * a.part_rows + tok0 * a.G + row;
          dst = reinterpret_cast<char*>(a.part_o + at * DH);
          ml = a.part_ml;
        } else {
          at = (static_cast<int64_t>(-2 - p.dest) * a.b.T + orow) * a.H + head;
          dst = reinterpret_cast<char*>(a.row_o + at * DH);
          ml = a.row_ml;
        }
        if (row < rows) *reinterpret_cast<float2*>(ml + at * 2) = make_float2(m, l);
      }
      const float inv = p.dest == -1 ? (m == -INFINITY ? 0.f : 1.0f / l) : 1.0f;  // no key: zeros
      if (rows - quarter * 32 <= PA_FEW_ROWS) {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t ov[16];
          tmem_ld16(tO + c * 16, ov);
          tmem_ld_wait();
          tmem_reg_fence(ov);
          if (row < rows) {
            uint4* to = reinterpret_cast<uint4*>(dst);
            if (p.dest == -1) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                ov[i] = pack_bf16x2(__uint_as_float(ov[2 * i]) * inv,
                                    __uint_as_float(ov[2 * i + 1]) * inv);
              to[2 * c] = make_uint4(ov[0], ov[1], ov[2], ov[3]);
              to[2 * c + 1] = make_uint4(ov[4], ov[5], ov[6], ov[7]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                to[4 * c + i] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
            }
          }
        }
      } else {
        char* to[4];  // the four lanes' rows, at this lane's unit
#pragma unroll
        for (int j = 0; j < 4; ++j)
          to[j] = reinterpret_cast<char*>(
                      __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst),
                                  (lane & ~3) + j)) + (lane & 3) * 16;
        const int have = rows - (row & ~3);  // rows of the four that exist
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t ov[32];
          tmem_ld32(tO + c * 32, ov);
          tmem_ld_wait();
          tmem_reg_fence(ov);
          if (p.dest == -1) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = pack_bf16x2(__uint_as_float(ov[2 * i]) * inv,
                                 __uint_as_float(ov[2 * i + 1]) * inv);
            store_transposed(w, to, have, c * 64);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              store_transposed(*reinterpret_cast<uint32_t(*)[16]>(&ov[h * 16]), to, have,
                               c * 128 + h * 64);
          }
        }
      }
      tc_fence_before();  // O has been read before a later piece's P V overwrites it
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    // the join, which waits for this kernel's end, has to find the rows' results too
    if (a.rows_own) asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}

// Joins. With a prefix every row passes one, so warps in flight count: four CTAs per SM
// (64 registers) and four partials at a time (6 chunks of 300 rows behind 1,000 keys, 42
// heads: 132 us; three CTAs 142, three and eight partials 160). Where the items are so
// few that a row has more than PA_JOIN_MANY partials, up to eight warps of a CTA share
// them: 2 sequences of up to 6 rows and 27,758 keys, 24 heads on 1, 22 us against 38
// with a warp per row (and 2 of up to 3 rows and 8,277 keys, 32 heads on 4, about 19
// partials, 19.7 against 18.5).
constexpr int PA_JOIN_CTAS = 4, PA_JOIN_N = 4, PA_JOIN_WARPS = 8, PA_JOIN_MANY = 32;
// A row's result while its partials are joined, four channels per lane.
struct Joined {
  float m = -INFINITY, l = 0.f;  // maximum -inf: no key (see KEYS_SEEN)
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
};

// Adds up to 32 partial results to j, N of them in flight: lane i holds the (maximum,
// sum) of the i-th, load(i) gives this lane's channels of it. In the order of their
// keys, so the sums do not depend on which CTA came first.
template <int N, class Load>
__device__ __forceinline__ void join_parts(Joined& j, int n, float2 ml, Load&& load) {
  float top = ml.x;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float m = fmaxf(j.m, top);
  if (m == -INFINITY) return;  // no key so far
  const float c = ex2_approx(j.m - m), w = ex2_approx(ml.x - m);
  float l = ml.y * w;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  j.m = m;
  j.l = j.l * c + l;
  j.o.x *= c;
  j.o.y *= c;
  j.o.z *= c;
  j.o.w *= c;
  for (int i0 = 0; i0 < n; i0 += N) {
    float4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i0 + i < n) x[i] = load(i0 + i);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, (i0 + i) & 31);
      if (i0 + i < n) {
        j.o.x = fmaf(x[i].x, wi, j.o.x);
        j.o.y = fmaf(x[i].y, wi, j.o.y);
        j.o.z = fmaf(x[i].z, wi, j.o.z);
        j.o.w = fmaf(x[i].w, wi, j.o.w);
      }
    }
  }
}

__device__ __forceinline__ float4 load_part(const float* row) {
  return __ldcg(reinterpret_cast<const float4*>(row) + (threadIdx.x & 31));
}

// Row r of an item that CTAs c0, c0 + g, .. c1 have parts of (the end of the first
// one's share, the beginning of the others'): the sub-th of `subs` equal runs of them.
template <int N>
__device__ __forceinline__ void join_split(Joined& j, const PagedArgs& a, int seg, int c0, int c1,
                                           int g, int r, int sub, int subs) {
  const int lane = threadIdx.x & 31;
  const int n = (c1 - c0) / g + 1, run = (n + subs - 1) / subs;
  const int end = min((sub + 1) * run, n);
  auto slot = [&](int i) {
    return static_cast<int64_t>((seg * PA_MAX_CTAS + c0 + i * g) * 2 + (i == 0 ? 1 : 0)) *
               a.part_rows + r;
  };
  for (int base = sub * run; base < end; base += 32) {
    const float2 ml = base + lane < end
                          ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot(base + lane))
                          : make_float2(-INFINITY, 0.f);
    join_parts<N>(j, min(end - base, 32), ml,
                  [&](int i) { return load_part(a.part_o + slot(base + i) * DH); });
  }
}

// Warps of a CTA that share a row, when the grid's warps are for so many rows.
__device__ __forceinline__ int join_subs(int64_t rows) {
  int n = 1;
  while (n < PA_JOIN_WARPS && rows * n * 2 <= static_cast<int64_t>(gridDim.x) * PA_JOIN_WARPS) n *= 2;
  return n;
}

// Adds what the other warps of the row have to the first one's. All of the CTA.
__device__ __forceinline__ void join_warps(Joined& j, float4 (&part)[PA_JOIN_WARPS][32],
                                           float2 (&ml)[PA_JOIN_WARPS], int subs) {
  if (subs == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp & (subs - 1);
  __syncthreads();  // the row before has been read
  part[warp][lane] = j.o;
  if (lane == 0) ml[warp] = make_float2(j.m, j.l);
  __syncthreads();
  if (sub != 0) return;
  const float2 mine = lane < subs ? ml[warp + lane] : make_float2(-INFINITY, 0.f);
  Joined all;
  join_parts<PA_JOIN_N>(all, subs, mine, [&](int i) { return part[warp + i][lane]; });
  j = all;
}

__device__ __forceinline__ void store_joined(const Joined& j, const PagedArgs& a, int t, int head) {
  const float inv = j.m == -INFINITY ? 0.f : 1.0f / j.l;  // no key: zeros
  *reinterpret_cast<uint2*>(a.o + t * a.ld_o + head * DH + (threadIdx.x & 31) * 4) =
      make_uint2(pack_bf16x2(j.o.x * inv, j.o.y * inv), pack_bf16x2(j.o.z * inv, j.o.w * inv));
}

// Without a prefix: block (c, y) joins rows of the item that goes on after CTA
// c's share, a warp per row.
constexpr int PA_JOIN_Y = 8;
__global__ void __launch_bounds__(32 * PA_JOIN_WARPS) paged_join_kernel(const PagedArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const int4 cut = __ldcg(a.cut + c);
  const int rows = cut.y * a.G;
  const int g = rows > 0 ? __ldcg(a.teams + 1) : 1;
  for (int r = blockIdx.y * PA_JOIN_WARPS + (threadIdx.x >> 5); r < rows;
       r += PA_JOIN_Y * PA_JOIN_WARPS) {
    Joined j;
    join_split<8>(j, a, 0, c, cut.w, g, r, 0, 1);
    store_joined(j, a, cut.x + r / a.G, cut.z * a.G + r % a.G);
  }
}

// The same where rows have many partials: the rows of those items, laid end to end,
// are spread over the grid's CTAs, several warps to a row.
__global__ void __launch_bounds__(32 * PA_JOIN_WARPS)
    paged_join_many_kernel(const PagedArgs a) {
  __shared__ int start[PA_MAX_CTAS + 1];  // first row of every CTA's cut item
  __shared__ float4 part[PA_JOIN_WARPS][32];
  __shared__ float2 ml[PA_JOIN_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0) {
    constexpr int RUN = PA_MAX_CTAS / 32;
    int rows[RUN], sum = 0;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      const int c = lane * RUN + i;
      rows[i] = c < a.ctas ? __ldcg(a.cut + c).y * a.G : 0;
      sum += rows[i];
    }
    int at = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, d);
      if (lane >= d) at += v;
    }
    if (lane == 31) start[PA_MAX_CTAS] = at;
    at -= sum;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      start[lane * RUN + i] = at;
      at += rows[i];
    }
  }
  __syncthreads();
  const int total = start[PA_MAX_CTAS];
  const int subs = join_subs(total), each = PA_JOIN_WARPS / subs;
  const int sub = warp & (subs - 1);
  const int g = total > 0 ? __ldcg(a.teams + 1) : 1;
  for (int base = blockIdx.x * each; base < total; base += gridDim.x * each) {
    const int w = base + warp / subs;
    Joined j;
    int4 cut{};
    int r = 0;
    if (w < total) {
      // the last CTA whose item begins at or before the row (those without rows
      // begin where the next one does)
      int before = 0;
#pragma unroll
      for (int i = 0; i < PA_MAX_CTAS / 32; ++i) before += start[i * 32 + lane + 1] <= w ? 1 : 0;
      const int c = __reduce_add_sync(0xffffffffu, before);
      cut = __ldcg(a.cut + c);
      r = w - start[c];
      join_split<8>(j, a, 0, c, cut.w, g, r, sub, subs);
    }
    join_warps(j, part, ml, subs);
    if (w < total && sub == 0) store_joined(j, a, cut.x + r / a.G, cut.z * a.G + r % a.G);
  }
}

// With a prefix: every row is joined from its results of the prefix and of its
// own keys, each whole or split, or the second by h3_paged_rows.cu; a warp per
// (token, head). What bounds it is the chain of loads of a row (sequence, ranges,
// places, results), so those of both segments are in flight together.
// MANY: several warps to a row.
template <bool MANY>
__global__ void __launch_bounds__(32 * PA_JOIN_WARPS, MANY ? 1 : PA_JOIN_CTAS)
    paged_join_prefix_kernel(const PagedArgs a) {
  __shared__ float4 part[PA_JOIN_WARPS][32];
  __shared__ float2 ml[PA_JOIN_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(a.b.T) * a.H;
  const int subs = MANY ? join_subs(rows) : 1, each = PA_JOIN_WARPS / subs;
  const int sub = warp & (subs - 1);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int team[2] = {__ldcg(a.teams), a.rows_own ? 1 : __ldcg(a.teams + 1)};
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * each; base < rows;
       base += static_cast<int64_t>(gridDim.x) * each) {
    const int64_t w = base + warp / subs;
    const int t = static_cast<int>(min(w, rows - 1) / a.H);
    const int head = static_cast<int>(min(w, rows - 1) % a.H), hk = head / a.G;
    const int b = w < rows ? ends_up_to(a.b.cu_q, a.b.B, t) : a.b.B;  // the row's sequence
    bool in[2] = {false, false};
    int2 at[2];  // first and last CTA that has a part of the row's item
    int row[2];  // of the item
#pragma unroll
    for (int seg = 0; seg < 2; ++seg) {
      at[seg] = make_int2(0, 0);
      row[seg] = 0;
      if (b >= a.b.B) continue;
      const SeqInfo s = seq_info(a, seg, b);
      in[seg] = t >= s.c0 && t < s.c0 + s.q_len;
      const int first = in[seg] ? (t - s.c0) / a.item * a.item : 0;
      row[seg] = (t - s.c0 - first) * a.G + head % a.G;
      if (in[seg] && (seg == 0 || !a.rows_own))
        at[seg] = __ldcg(a.spread + (static_cast<int64_t>(seg) * a.b.T + s.c0 + first) * a.Hkv + hk);
    }
    Joined j;
    const int64_t i1 = rows + w;
    if (in[0] && in[1] && at[0].x == at[0].y && at[1].x == at[1].y) {  // both whole
      if (sub == 0) {
        const float2 ml0 = __ldcg(reinterpret_cast<const float2*>(a.row_ml) + w);
        const float2 ml1 = __ldcg(reinterpret_cast<const float2*>(a.row_ml) + i1);
        const float4 x0 = load_part(a.row_o + w * DH), x1 = load_part(a.row_o + i1 * DH);
        const float m = fmaxf(ml0.x, ml1.x);
        const float f0 = m == -INFINITY ? 0.f : ex2_approx(ml0.x - m);
        const float f1 = m == -INFINITY ? 0.f : ex2_approx(ml1.x - m);
        j.m = m;
        j.l = ml0.y * f0 + ml1.y * f1;
        j.o = make_float4(x0.x * f0 + x1.x * f1, x0.y * f0 + x1.y * f1, x0.z * f0 + x1.z * f1,
                          x0.w * f0 + x1.w * f1);
      }
    } else {
#pragma unroll 1
      for (int seg = 0; seg < 2; ++seg) {
        if (!(seg ? in[1] : in[0])) continue;
        const int2 p = seg ? at[1] : at[0];
        if (p.x == p.y) {
          if (sub != 0) continue;
          const int64_t i = seg ? i1 : w;
          const float2 v = lane == 0 ? __ldcg(reinterpret_cast<const float2*>(a.row_ml) + i)
                                     : make_float2(-INFINITY, 0.f);
          join_parts<1>(j, 1, v, [&](int) { return load_part(a.row_o + i * DH); });
        } else {
          join_split<MANY ? 8 : PA_JOIN_N>(
                     j, a, seg, min(max(p.x, 0), a.ctas - 1), min(max(p.y, 0), a.ctas - 1),
                     seg ? team[1] : team[0], seg ? row[1] : row[0], sub, subs);
        }
      }
    }
    if constexpr (MANY) join_warps(j, part, ml, subs);
    if (sub == 0 && (in[0] || in[1])) store_joined(j, a, t, head);
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace: team sizes and cut items; the split items' partials; with a
// prefix, where each item lies and a result of every row per segment.
struct PagedWs {
  size_t cut, spread, part_o, part_ml, row_o, row_ml, total;
  int part_rows;
};
PagedWs paged_ws(int T, int H, int prefix_len) {
  PagedWs w;
  const size_t rows = static_cast<size_t>(T) * H;
  const bool prefix = prefix_len > 0;
  // rows of one item: at most two query tiles, at most what the call has; where the
  // runs of a part meet, up to PA_QUAD_ROWS of them in every lane quarter
  w.part_rows = static_cast<int>(std::min<size_t>(2 * BQ, rows + 3 * std::min<size_t>(PA_QUAD_ROWS, rows)));
  const size_t slots = (prefix ? 2 : 1) * PA_MAX_CTAS * 2;
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  w.cut = take(PA_MAX_CTAS * sizeof(int4));
  w.part_o = take(slots * w.part_rows * DH * 4);
  w.part_ml = take(slots * w.part_rows * 8);
  w.spread = take(prefix ? 2 * rows * sizeof(int2) : 0);  // Hkv <= H
  w.row_o = take(prefix ? 2 * rows * DH * 4 : 0);
  w.row_ml = take(prefix ? 2 * rows * 8 : 0);
  w.total = off;
  return w;
}

}  // namespace

size_t paged_workspace_bytes(int T, int H, int prefix_len) {
  return paged_ws(T, H, prefix_len).total;
}

h3_status launch_paged_attention(const void* q, int64_t ld_q, void* o, int64_t ld_o, int H,
                                 float scale, bool causal, const void* k_cache,
                                 const void* v_cache, int Hkv, const PagedBatch& batch,
                                 const int32_t* prefix_pages, int prefix_len, void* workspace,
                                 cudaStream_t s) {
  const int64_t own = static_cast<int64_t>(batch.max_pages) << batch.page_log2;
  const bool runs = std::max<int64_t>(own, prefix_len) > PA_RUN * BKV;
  const auto kernel = runs ? paged_attention_kernel<true> : paged_attention_kernel<false>;
  static std::atomic<bool> done[2][64];
  h3_status st = set_smem_limit(done[runs], kernel, PA_SMEM_BYTES,
                                "paged attention: set shared memory size");
  if (st != H3_OK) return st;
  const PagedWs w = paged_ws(batch.T, H, prefix_len);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  PagedArgs a{};
  a.b = batch;
  a.ld_o = ld_o;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.tok = BQ / a.G;
  // One query tile per item, and no teams, where none is split and there is a CTA for
  // each of them (2 sequences of 185 rows and 446 keys, 32 heads on 8: 14.4 us against
  // 16.5; one of 512 rows and keys, 4 heads: 13.3 / 15.6).
  const bool whole = prefix_len == 0 && own <= PA_WHOLE * BKV;
  const int ctas = std::min(num_sms(), PA_MAX_CTAS);
  const bool one = whole && (batch.T / a.tok + static_cast<int64_t>(batch.B)) * Hkv <= ctas;
  a.item = one ? a.tok : 2 * a.tok;
  a.max_team = one ? 1 : PA_MAX_TEAM;
  a.total_rows = (batch.num_pages * Hkv) << batch.page_log2;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal ? 1 : 0;
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.teams = reinterpret_cast<int*>(base);
  a.cut = reinterpret_cast<int4*>(base + w.cut);
  a.spread = reinterpret_cast<int2*>(base + w.spread);
  a.part_o = reinterpret_cast<float*>(base + w.part_o);
  a.part_ml = reinterpret_cast<float*>(base + w.part_ml);
  a.part_rows = w.part_rows;
  a.row_o = reinterpret_cast<float*>(base + w.row_o);
  a.row_ml = reinterpret_cast<float*>(base + w.row_ml);
  a.ctas = ctas;
  if ((st = dev_err(&a.err)) != H3_OK) return st;
  CUtensorMap tq, tq1, tk, tv;
  const uint32_t page = 1u << batch.page_log2;
  if ((st = make_tmap_bf16_3d(&tq, q, DH, H, batch.T, DH * 2, static_cast<uint64_t>(ld_q) * 2, 64,
                              a.G, a.tok)) != H3_OK ||
      (st = make_tmap_bf16_3d(&tq1, q, DH, H, batch.T, DH * 2, static_cast<uint64_t>(ld_q) * 2, 64,
                              a.G, 1)) != H3_OK ||
      (st = make_tmap_bf16_2d(&tk, k_cache, DH, a.total_rows, DH * 2, 64, page)) != H3_OK ||
      (st = make_tmap_bf16_2d(&tv, v_cache, DH, a.total_rows, DH * 2, 64, page)) != H3_OK)
    return st;
  // The rows' own keys behind a prefix, many items of few keys, go to the kernel of
  // short rows (64 rows of up to 512 keys behind 29,034, 42 heads: 172 us against 194;
  // 128 rows of up to 200 keys behind 12,000, 8 heads: 43 / 50; of up to 1,000 behind
  // 40,000: 98 / 96). With fewer items its launch costs what it saves (64 rows of up
  // to 200 keys behind 40,000, 32 heads on 4: 55 / 53).
  a.rows_own = prefix_len > 0 && static_cast<int64_t>(batch.T) * Hkv > 2 * num_sms() &&
               paged_rows_fit(batch.T, H, Hkv, batch.B, own, 0);
  if (a.rows_own &&
      (st = launch_paged_rows(q, ld_q, o, ld_o, H, scale, causal, k_cache, v_cache, Hkv, batch,
                              nullptr, 0, a.row_o + static_cast<int64_t>(batch.T) * H * DH,
                              a.row_ml + static_cast<int64_t>(batch.T) * H * 2, s)) != H3_OK)
    return st;
  // the next kernel's blocks may take their places while the one before runs; they
  // wait for its end before they read what it wrote
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = a.rows_own;
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(PA_THREADS);
  cfg.dynamicSmemBytes = PA_SMEM_BYTES;
  st = cuda_fail(cudaLaunchKernelEx(&cfg, kernel, tq, tq1, tk, tv, a),
                 "paged attention launch");
  if (st != H3_OK) return st;
  if (whole) return H3_OK;  // nothing is split, nothing to join
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(32 * PA_JOIN_WARPS);
  cfg.dynamicSmemBytes = 0;
  // items of the prefix, or at least so many of the sequences' own keys
  const int64_t tiles = (batch.T + a.item - 1) / a.item;
  const int64_t items = (prefix_len > 0 ? tiles : std::max<int64_t>(tiles, batch.B)) * Hkv;
  const bool many = items * PA_JOIN_MANY <= a.ctas;
  const int64_t rows = static_cast<int64_t>(batch.T) * H;
  cudaError_t e;
  if (many) {
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(rows, a.ctas * 3)));
    e = prefix_len > 0 ? cudaLaunchKernelEx(&cfg, paged_join_prefix_kernel<true>, a)
                       : cudaLaunchKernelEx(&cfg, paged_join_many_kernel, a);
  } else if (prefix_len > 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(
        std::min<int64_t>((rows + PA_JOIN_WARPS - 1) / PA_JOIN_WARPS, a.ctas * 8)));
    e = cudaLaunchKernelEx(&cfg, paged_join_prefix_kernel<false>, a);
  } else {
    cfg.gridDim = dim3(a.ctas, PA_JOIN_Y);
    e = cudaLaunchKernelEx(&cfg, paged_join_kernel, a);
  }
  return cuda_fail(e, "paged attention join launch");
}

}  // namespace h3
