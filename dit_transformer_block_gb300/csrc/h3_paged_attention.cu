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
// One CTA, 384 threads (two warps idle), the hand-off and tensor-memory layout of the FP8
// attention kernel:
//   warp 8: walks the CTA's pieces of items, posts each in a ring in shared
//     memory, and loads by TMA its query tiles and, key tile by key tile, K_t
//     and V_t (one box per page and 64 channels) into a ring of 32 KB slots;
//   warp 9: allocates TMEM and issues the products: S = Q_i K_t^T (SS) into
//     one S buffer, O_i += P_i V_t (TS, P_i in tensor memory); Q K^T of the next
//     key tile goes ahead of the P V of this one, also across pieces;
//   warps 0-3 / 4-7: softmax of query tile 0 / 1 (thread = query row = TMEM
//     lane). A piece of one query tile takes the two groups in turn, so the
//     output of one piece overlaps the products of the next.
#include <algorithm>

#include "h3_attn_common.cuh"

namespace h3 {
namespace {

constexpr int PA_SLOTS = 5;    // 32 KB each: K_t, V_t, K_t+1, ...
constexpr int PA_PIECES = 8;   // pieces posted ahead
constexpr int PA_MAX_CTAS = 160;
constexpr int PA_CTRL_BYTES = 1024;
// 12 warps: with three on each SM sub-partition the launch gives every thread
// 168 registers; warps 8-11 hand most of theirs to the softmax warps, which
// hold a row's 128 scores and 64 packed weights (168: 508 bytes of spills)
constexpr int PA_THREADS = 384;
constexpr int PA_REGS_SOFTMAX = 216, PA_REGS_OTHER = 72;
static_assert(2 * PA_REGS_SOFTMAX + PA_REGS_OTHER <= 3 * 168, "registers of the launch");
constexpr size_t PA_SMEM_BYTES = 1024 + (PA_SLOTS + 2) * TILE_BYTES + PA_CTRL_BYTES;
static_assert(PA_SMEM_BYTES <= 227 * 1024, "paged attention shared memory");

enum BarPA {
  PA_KV_FULL = 0,
  PA_KV_EMPTY = PA_KV_FULL + PA_SLOTS,
  PA_Q_FULL = PA_KV_EMPTY + PA_SLOTS,
  PA_Q_EMPTY = PA_Q_FULL + 2,
  PA_S = PA_Q_EMPTY + 2,       // S written for query tile i (MMA commit)
  PA_SFREE = PA_S + 2,         // S read by its softmax (4 warp arrivals)
  PA_P = PA_SFREE + 2,         // P_i written (4 warp arrivals)
  PA_PVD = PA_P + 2,           // P_i V done (MMA commit)
  PA_PC_FULL = PA_PVD + 2,     // piece posted
  PA_PC_EMPTY = PA_PC_FULL + PA_PIECES,  // piece read (8 softmax warps, MMA warp)
  PA_DRAIN = PA_PC_EMPTY + PA_PIECES,
  PA_BARS
};
constexpr uint32_t TPA_S = 0, TPA_O = 128, TPA_P = 384;

struct PagedArgs {
  PagedBatch b;
  int64_t ld_o;
  __nv_bfloat16* o;
  int H, Hkv, G;
  int tok;           // tokens of one query tile: floor(128 / G)
  int total_rows;    // rows of the cache's tensor map: num_pages * Hkv * page_size
  float scale_log2;  // softmax_scale * log2(e)
  int causal;
  const int32_t* prefix_pages;
  int prefix_len;
  // workspace
  int64_t* totals;   // [2] key tiles of the two segments
  int64_t* first;    // [T] tile offset of the sequence whose first row is t
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

// Key tiles of one key head of a sequence.
__device__ __forceinline__ int64_t head_tiles(const PagedArgs& a, int seg, const SeqInfo& s) {
  const int item = 2 * a.tok;
  const int n = (s.q_len + item - 1) / item;
  if (n == 0) return 0;
  if (!uneven(a, seg)) return static_cast<int64_t>(n) * key_tiles(s, s.q_len);
  int64_t sum = 0;
  for (int i = 1; i <= n; ++i) sum += key_tiles(s, min(i * item, s.q_len));
  return sum;
}

// The CTAs' shares of a segment of W tiles: CTA c has [c W / n, (c + 1) W / n).
__device__ __forceinline__ int64_t share_begin(int64_t W, int n, int c) { return c * W / n; }
__device__ __forceinline__ int share_of(int64_t W, int n, int64_t w) {
  return static_cast<int>(((w + 1) * n - 1) / W);
}

// A CTA's part of an item, as posted to the other warps.
struct Piece {
  int tok0, ntok;  // tokens (ntok 0: no more pieces)
  int hk;          // key head
  int kt0, kt1;    // key tiles
  int kv;          // keys of the sequence
  int lim0;        // token i of the piece sees min(lim0 + i, kv) keys
  int dest;        // >= 0: partial slot; -1: the output; -2 - seg: the segment's rows
};
static_assert(sizeof(Piece) == 32, "two 16-byte loads");

// The first sequence of this CTA's share, found by all threads together.
struct Share {
  int64_t begin, end;
  int64_t base;  // tile offset of sequence b
  int b;
};

// One key tile of the online softmax of the calling thread's row, in base 2
// with the scale folded in; the scores are in sr, columns >= valid are masked.
// The running maximum is raised only when a row exceeds it by more than
// RESCALE_THRESHOLD (then O and the sum are rescaled), so a weight can be up
// to 2^8; a row that has seen no key yet keeps maximum -inf and sum 0. The
// weights go to tensor memory rounded to bf16 (the type of V in the product);
// the sum is of the unrounded ones, in FP32. wait_pv: the tile's previous P V
// is done with P and O. Returns false when a wait failed.
template <class WaitPV>
__device__ __forceinline__ bool softmax_tile_paged(uint32_t (&sr)[128], uint32_t tP, uint32_t tO,
                                                   int valid, bool o_live, float scale_log2,
                                                   float& m, float& l, WaitPV&& wait_pv) {
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
  if (__any_sync(0xffffffffu, mx > m + RESCALE_THRESHOLD)) {
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

__global__ void __launch_bounds__(PA_THREADS, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ,
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
  Piece* ring = reinterpret_cast<Piece*>(ctrl + 384);                 // [PA_PIECES]
  int64_t* warp_sum = reinterpret_cast<int64_t*>(ctrl + 640);         // [12]
  Share* share = reinterpret_cast<Share*>(ctrl + 736);                // [2]
  static_assert((PA_BARS + 1) * 8 + 16 <= 384 && 384 + PA_PIECES * 32 <= 640 &&
                    736 + 2 * sizeof(Share) <= PA_CTRL_BYTES,
                "control region");
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // the joining kernel may be set up while this one runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < PA_BARS; ++i) {
      uint32_t count = 1;
      if (i >= PA_SFREE && i < PA_PVD) count = 4;
      if (i >= PA_PC_EMPTY && i < PA_DRAIN) count = 9;
      mbar_init(bar(i), count);
    }
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // this CTA's share of each segment: every thread sums the tiles of a run of
  // sequences, a scan over the threads gives the offsets
  const int first_seg = a.prefix_len > 0 ? 0 : 1;
  for (int seg = first_seg; seg < 2; ++seg) {
    const int n = seg == 0 ? 1 : a.b.B;
    const int run = (n + PA_THREADS - 1) / PA_THREADS;
    const int b0 = min(static_cast<int>(threadIdx.x) * run, n), b1 = min(b0 + run, n);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += head_tiles(a, seg, seq_info(a, seg, b)) * a.Hkv;
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    __syncthreads();  // warp_sum of the previous segment has been read
    if (lane == 31) warp_sum[warp] = incl;
    if (threadIdx.x == 0) share[seg] = Share{0, 0, 0, 0};
    __syncthreads();
    int64_t before = 0, W = 0;
    for (int i = 0; i < PA_THREADS / 32; ++i) {
      if (i < warp) before += warp_sum[i];
      W += warp_sum[i];
    }
    int64_t at = before + incl - mine;
    const int64_t begin = share_begin(W, a.ctas, blockIdx.x);
    const int64_t end = share_begin(W, a.ctas, blockIdx.x + 1);
    const bool here = begin < end && begin >= at && begin < at + mine;
    if (here || blockIdx.x == 0) {
      if (blockIdx.x == 0 && threadIdx.x == 0) a.totals[seg] = W;
      for (int b = b0; b < b1; ++b) {
        const SeqInfo s = seq_info(a, seg, b);
        const int64_t tiles = head_tiles(a, seg, s) * a.Hkv;
        if (begin < end && begin >= at && begin < at + tiles) share[seg] = Share{begin, end, at, b};
        if (blockIdx.x == 0 && seg == 1 && s.q_len > 0) a.first[s.c0] = at;
        at += tiles;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PA_REGS_OTHER));
  if (warp == 8) {
    // ------------------------------------------- pieces and TMA loads
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int nbox = BKV >> a.b.page_log2;  // pages of a key tile
    const int box = lane & (nbox - 1), half = lane / nbox;
    const uint32_t box_dst = half * BOX_BYTES + ((box << a.b.page_log2) << 7);
    const uint32_t q_bytes = static_cast<uint32_t>(a.tok * a.G) * 256;
    int np = 0, seq = 0, nq[2] = {0, 0};
    bool ok = true;
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
    auto run_piece = [&](const Piece& p, const int32_t* pages) {
      const bool two = p.ntok > a.tok;
      const int g0 = two ? 0 : np & 1;
      if (!post(p)) return false;
      for (int g = g0; g <= (two ? 1 : g0); ++g) {
        if (!mbar_wait_warp(bar(PA_Q_EMPTY + g), (nq[g] & 1) ^ 1, a.err, ERR_WAIT_ATTN_PRODUCER))
          return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(PA_Q_FULL + g), q_bytes);
          const uint32_t dst = smem_u32(sQ + g * TILE_BYTES);
          const int t0 = p.tok0 + (two ? g * a.tok : 0);
          tma_load_3d(dst, &tmQ, bar(PA_Q_FULL + g), 0, p.hk * a.G, t0);
          tma_load_3d(dst + BOX_BYTES, &tmQ, bar(PA_Q_FULL + g), 64, p.hk * a.G, t0);
        }
        ++nq[g];
      }
      // a page is loaded when it begins below the sequence's end
      auto page_of = [&](int kt) {
        const int i = kt * nbox + box;
        return half < 2 && kt < p.kt1 && (static_cast<int64_t>(i) << a.b.page_log2) < p.kv
                   ? __ldg(pages + i)
                   : -1;
      };
      int page = page_of(p.kt0);
      for (int kt = p.kt0; kt < p.kt1; ++kt) {
        const int next = page_of(kt + 1);
        const int live = min(nbox, (p.kv - kt * BKV + (1 << a.b.page_log2) - 1) >> a.b.page_log2);
        const uint32_t bytes = static_cast<uint32_t>(max(live, 0)) << (a.b.page_log2 + 8);
        // a page outside the pool: a row past the map's end, which loads zeros
        const int row = page >= 0 && page < a.b.num_pages
                            ? (page * a.Hkv + p.hk) << a.b.page_log2
                            : a.total_rows;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++seq) {
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
          if (half < 2 && box < live)
            tma_load_2d(smem_u32(sKV + slot * TILE_BYTES) + box_dst, kv ? &tmV : &tmK, full,
                        half * 64, row);
        }
        page = next;
      }
      return true;
    };
    for (int seg = first_seg; ok && seg < 2; ++seg) {
      const Share sh = share[seg];
      int64_t w = sh.begin, base = sh.base;
      int b = sh.b;
      const int n = seg == 0 ? 1 : a.b.B;
      const int item = 2 * a.tok;
      if (w >= sh.end) continue;
      SeqInfo s = seq_info(a, seg, b);
      int64_t per_head = head_tiles(a, seg, s);
      while (ok && w < sh.end) {
        while (w >= base + per_head * a.Hkv && b + 1 < n) {
          base += per_head * a.Hkv;
          s = seq_info(a, seg, ++b);
          per_head = head_tiles(a, seg, s);
        }
        if (per_head == 0 || w >= base + per_head * a.Hkv) break;
        Piece p;
        p.hk = static_cast<int>((w - base) / per_head);
        int64_t r = (w - base) - p.hk * per_head;
        int qt, nk;
        if (uneven(a, seg)) {
          for (qt = 0;; ++qt) {
            nk = key_tiles(s, min((qt + 1) * item, s.q_len));
            if (r < nk) break;
            r -= nk;
          }
        } else {
          nk = key_tiles(s, s.q_len);
          qt = static_cast<int>(r / nk);
          r -= static_cast<int64_t>(qt) * nk;
        }
        p.kt0 = static_cast<int>(r);
        p.kt1 = static_cast<int>(min(static_cast<int64_t>(nk), r + (sh.end - w)));
        w += p.kt1 - p.kt0;
        p.tok0 = s.c0 + qt * item;
        p.ntok = min(item, s.q_len - qt * item);
        p.kv = s.kv;
        p.lim0 = uneven(a, seg) ? s.off + qt * item + 1 : s.kv;
        const bool whole = p.kt0 == 0 && p.kt1 == nk;
        p.dest = !whole ? ((seg - first_seg) * PA_MAX_CTAS + static_cast<int>(blockIdx.x)) * 2 +
                              (p.kt0 > 0 ? 0 : 1)
                        : (first_seg == 0 ? -2 - seg : -1);
        ok = run_piece(p, seg == 0 ? a.prefix_pages
                                   : a.b.page_table + static_cast<int64_t>(b) * a.b.max_pages);
      }
    }
    if (ok) ok = post(Piece{0, 0, 0, 0, 0, 0, 0, 0});
    // no copy of this CTA may still be landing when it exits
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      const uint64_t lim = drain_limit_ns(a.err);
      for (int g = 0; g < 2; ++g)
        if (nq[g] > 0) mbar_wait_drain(bar(PA_Q_FULL + g), (nq[g] - 1) & 1, t0, lim);
      for (int i = max(seq - PA_SLOTS, 0); i < seq; ++i)
        mbar_wait_drain(bar(PA_KV_FULL + i % PA_SLOTS), (i / PA_SLOTS) & 1, t0, lim);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_qk = idesc_bf16_f32(BQ, BKV, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(BQ, DH, true);
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dk = sdesc_sw128(smem_u32(sKV), 16, 1024);
    const uint64_t dv = sdesc_sw128(smem_u32(sKV), BOX_BYTES, 1024);
    auto wait = [&](int b, int count) {
      return mbar_wait_warp(bar(b), count & 1, a.err, ERR_WAIT_ATTN_MMA);
    };
    // 16-byte offset of K step kk (16 channels) in a K-major tile
    auto kmaj = [](int kk) {
      return static_cast<uint32_t>(((kk >> 2) * BOX_BYTES + (kk & 3) * 32) >> 4);
    };
    struct Tile {
      int g0;      // query tile, or the first of two
      bool two, first, last;
      int t;       // key tiles of this CTA before it
    };
    int np = 0, left = 0, tiles = 0;
    Tile proto{0, false, false, false, 0};
    bool ok = true;
    // the next key tile; false: no more, or a wait failed (ok false)
    auto next_tile = [&](Tile& d) {
      bool first = false;
      if (left == 0) {
        const int r = np % PA_PIECES;
        if (!wait(PA_PC_FULL + r, np / PA_PIECES)) return ok = false;
        const int ntok = ring[r].ntok;
        left = ring[r].kt1 - ring[r].kt0;
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
      d.t = tiles++;
      return true;
    };
    int nq[2] = {0, 0}, ns[2] = {0, 0}, npv[2] = {0, 0};
    int last_s = -1;  // query tile whose S is in the buffer
    auto qk = [&](const Tile& d, int g) {  // S = Q_g K_t^T
      const int seq = 2 * d.t, slot = seq % PA_SLOTS;
      if (d.first && !wait(PA_Q_FULL + g, nq[g]++)) return false;
      if (!wait(PA_KV_FULL + slot, seq / PA_SLOTS)) return false;
      if (last_s >= 0 && !wait(PA_SFREE + last_s, ns[last_s] - 1)) return false;
      tc_fence_after();
      const uint64_t qd = dq + static_cast<uint32_t>(g * (TILE_BYTES >> 4));
      const uint64_t kd = dk + static_cast<uint32_t>(slot * (TILE_BYTES >> 4));
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk)
        mma_ss_el(tmem + TPA_S, qd + kmaj(kk), kd + kmaj(kk), idesc_qk, kk > 0 ? 1u : 0u);
      mma_commit_el(bar(PA_S + g));
      if (d.last) mma_commit_el(bar(PA_Q_EMPTY + g));
      if (!d.two || g == 1) mma_commit_el(bar(PA_KV_EMPTY + slot));
      ++ns[g];
      last_s = g;
      return true;
    };
    auto pv = [&](const Tile& d, int g) {  // O_g (+)= P_g V_t
      const int seq = 2 * d.t + 1, slot = seq % PA_SLOTS;
      if (!wait(PA_P + g, npv[g]) || !wait(PA_KV_FULL + slot, seq / PA_SLOTS)) return false;
      tc_fence_after();
      const uint64_t vd = dv + static_cast<uint32_t>(slot * (TILE_BYTES >> 4));
#pragma unroll
      for (int kk = 0; kk < BKV / 16; ++kk)
        mma_ts_el(tmem + TPA_O + g * 128, tmem + TPA_P + g * 64 + kk * 8, vd + kk * (2048 >> 4),
                  idesc_pv, (!d.first || kk > 0) ? 1u : 0u);
      mma_commit_el(bar(PA_PVD + g));
      if (!d.two || g == 1) mma_commit_el(bar(PA_KV_EMPTY + slot));
      ++npv[g];
      return true;
    };
    Tile cur, nxt;
    bool more = next_tile(cur);
    if (more) ok = qk(cur, cur.g0) && (!cur.two || qk(cur, 1));
    // Q K^T of the next key tile before P V of this one; with two query tiles
    // their products alternate, so one's softmax overlaps the other's products
    while (ok && more) {
      more = next_tile(nxt);
      if (!ok) break;
      ok = (!more || qk(nxt, nxt.g0)) && pv(cur, cur.g0);
      if (ok && more && nxt.two) ok = qk(nxt, 1);
      if (ok && cur.two) ok = pv(cur, 1);
      cur = nxt;
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
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(PA_PC_EMPTY + r));
      if (p.ntok == 0) break;
      const bool two = p.ntok > a.tok;
      if (!two && (np & 1) != tile) {
        tiles += p.kt1 - p.kt0;
        continue;
      }
      const int tok0 = two ? tile * a.tok : 0;                        // within the piece
      const int rows = (two ? (tile ? p.ntok - a.tok : a.tok) : p.ntok) * a.G;
      const bool active = quarter * 32 < rows;
      const int tok = tok0 + row / a.G;
      const int lim = min(max(p.lim0 + tok, 0), p.kv);
      float m = -INFINITY, l = 0.f;
      for (int kt = p.kt0; kt < p.kt1; ++kt, ++tiles, ++n) {
        if (!mbar_wait_warp(bar(PA_S + tile), n & 1, a.err, ERR_WAIT_ATTN_SOFTMAX)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[128];
        if (active) {
          tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
          tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
          tmem_ld_wait();
          tmem_reg_fence(sr);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PA_SFREE + tile));
        const int live = p.kv - kt * BKV;  // keys of the tile that exist
        if (live < BKV) {
          // places behind the last key hold anything: their weights are 0, and
          // so their values have to be finite
          const int seq = 2 * tiles + 1, slot = seq % PA_SLOTS;
          if (!mbar_wait_warp(bar(PA_KV_FULL + slot), (seq / PA_SLOTS) & 1, a.err,
                              ERR_WAIT_ATTN_SOFTMAX)) {
            ok = false;
            break;
          }
          if (row >= live) {
            uint8_t* v = sKV + slot * TILE_BYTES + row * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              reinterpret_cast<uint4*>(v)[i] = make_uint4(0, 0, 0, 0);
              reinterpret_cast<uint4*>(v + BOX_BYTES)[i] = make_uint4(0, 0, 0, 0);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        const bool o_live = kt > p.kt0;
        if (active)
          ok = softmax_tile_paged(sr, tP, tO, lim - kt * BKV, o_live, a.scale_log2, m, l,
                                  [&] { return wait_pv(n - 1); });
        else  // this warp's P barrier phase must not run ahead of the others'
          ok = !o_live || wait_pv(n - 1);
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(PA_P + tile));
      }
      if (!ok || !wait_pv(n - 1)) break;
      if (!active) continue;
      const bool row_ok = row < rows;
      const int64_t orow = static_cast<int64_t>(p.tok0 + tok);
      const int head = p.hk * a.G + row % a.G;
      if (p.dest == -1) {
        const float inv = l == 0.f ? 0.f : 1.0f / l;  // no key: zeros
        __nv_bfloat16* dst = a.o + orow * a.ld_o + head * DH;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t ov[16], pk[8];
          tmem_ld16(tO + c * 16, ov);
          tmem_ld_wait();
          tmem_reg_fence(ov);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            pk[i] = pack_bf16x2(__uint_as_float(ov[2 * i]) * inv, __uint_as_float(ov[2 * i + 1]) * inv);
          if (row_ok) {
            reinterpret_cast<uint4*>(dst)[2 * c] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            reinterpret_cast<uint4*>(dst)[2 * c + 1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          }
        }
      } else {
        float *po, *pml;
        if (p.dest >= 0) {
          const int64_t at = static_cast<int64_t>(p.dest) * a.part_rows + tok0 * a.G + row;
          po = a.part_o + at * DH;
          pml = a.part_ml + at * 2;
        } else {
          const int64_t at = (static_cast<int64_t>(-2 - p.dest) * a.b.T + orow) * a.H + head;
          po = a.row_o + at * DH;
          pml = a.row_ml + at * 2;
        }
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t ov[16];
          tmem_ld16(tO + c * 16, ov);
          tmem_ld_wait();
          tmem_reg_fence(ov);
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<uint4*>(po)[4 * c + i] =
                  make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
          }
        }
        if (row_ok) *reinterpret_cast<float2*>(pml) = make_float2(m, l);
      }
      // O has been read before a later piece's P V overwrites it
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial results of each row: one warp per (token, head), four
// channels per lane, partials in the order of their keys (so the sums do not
// depend on which CTA came first). Without a prefix only rows of split items
// have any; with one, every row has those of the prefix and of its own keys.
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(a.b.T) * a.H;
  const int first_seg = a.prefix_len > 0 ? 0 : 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t w = blockIdx.x * 8LL + (threadIdx.x >> 5); w < rows; w += gridDim.x * 8LL) {
    const int t = static_cast<int>(w / a.H), head = static_cast<int>(w % a.H);
    const int hk = head / a.G;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    bool any = first_seg == 0;
    auto add = [&](const float* po, const float* pml) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(pml));
      const float4 x = __ldcg(reinterpret_cast<const float4*>(po) + lane);
      const float m_new = fmaxf(m, ml.x);
      if (m_new == -INFINITY) return;  // no key so far
      const float c = ex2_approx(m - m_new), d = ex2_approx(ml.x - m_new);
      o.x = o.x * c + x.x * d;
      o.y = o.y * c + x.y * d;
      o.z = o.z * c + x.z * d;
      o.w = o.w * c + x.w * d;
      l = l * c + ml.y * d;
      m = m_new;
    };
    // the row's sequence: the number of ends at or below it
    int b = 0;
    for (int i = lane; i < a.b.B; i += 32) b += __ldg(a.b.cu_q + i + 1) <= t ? 1 : 0;
    b = __reduce_add_sync(0xffffffffu, b);
    if (b >= a.b.B) continue;
    const SeqInfo own = seq_info(a, 1, b);
    if (t < own.c0 || t >= own.c0 + own.q_len) continue;
    for (int seg = first_seg; seg < 2; ++seg) {
      const SeqInfo s = seg == 0 ? seq_info(a, 0, 0) : own;
      if (t < s.c0 || t >= s.c0 + s.q_len) continue;  // only if cu_q is out of order
      const int item = 2 * a.tok;
      const int qt = (t - s.c0) / item, r = (t - s.c0 - qt * item) * a.G + head % a.G;
      const int64_t W = __ldcg(reinterpret_cast<const long long*>(a.totals) + seg);
      int64_t at = seg == 0 ? 0 : __ldcg(reinterpret_cast<const long long*>(a.first) + s.c0);
      int nk = key_tiles(s, s.q_len);
      if (uneven(a, seg)) {
        int64_t sum = 0, all = 0;
        const int n = (s.q_len + item - 1) / item;
        for (int i = lane; i < n; i += 32) {
          const int k = key_tiles(s, min((i + 1) * item, s.q_len));
          all += k;
          if (i < qt) sum += k;
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, d);
          all += __shfl_xor_sync(0xffffffffu, all, d);
        }
        at += hk * all + sum;
        nk = key_tiles(s, min((qt + 1) * item, s.q_len));
      } else {
        const int n = (s.q_len + item - 1) / item;
        at += (static_cast<int64_t>(hk) * n + qt) * nk;
      }
      const int c0 = min(max(share_of(W, a.ctas, at), 0), a.ctas - 1);
      const int c1 = min(max(share_of(W, a.ctas, at + nk - 1), c0), a.ctas - 1);
      if (c0 == c1) {
        if (first_seg == 0) {
          const int64_t i = (static_cast<int64_t>(seg) * a.b.T + t) * a.H + head;
          add(a.row_o + i * DH, a.row_ml + i * 2);
        }
        continue;
      }
      any = true;
      for (int c = c0; c <= c1; ++c) {
        const int64_t begin = share_begin(W, a.ctas, c);
        if (begin == share_begin(W, a.ctas, c + 1)) continue;  // fewer tiles than CTAs
        const int slot = ((seg - first_seg) * PA_MAX_CTAS + c) * 2 + (begin > at ? 0 : 1);
        const int64_t i = static_cast<int64_t>(slot) * a.part_rows + r;
        add(a.part_o + i * DH, a.part_ml + i * 2);
      }
    }
    if (!any) continue;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    *reinterpret_cast<uint2*>(a.o + t * a.ld_o + head * DH + lane * 4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace: the segments' totals, the sequences' offsets [T], the split
// items' partials and, with a prefix, a result of every row per segment.
struct PagedWs {
  size_t first, part_o, part_ml, row_o, row_ml, total;
  int part_rows;
};
PagedWs paged_ws(int T, int H, int prefix_len) {
  PagedWs w;
  const size_t rows = static_cast<size_t>(T) * H;
  // rows of one item: at most two query tiles, at most what the call has
  w.part_rows = static_cast<int>(std::min<size_t>(2 * BQ, rows));
  const size_t slots = (prefix_len > 0 ? 2 : 1) * PA_MAX_CTAS * 2;
  size_t off = 256;
  w.first = off;
  off += align256(static_cast<size_t>(T) * 8);
  w.part_o = off;
  off += align256(slots * w.part_rows * DH * 4);
  w.part_ml = off;
  off += align256(slots * w.part_rows * 8);
  w.row_o = off;
  if (prefix_len > 0) off += align256(2 * rows * DH * 4);
  w.row_ml = off;
  if (prefix_len > 0) off += align256(2 * rows * 8);
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
  static std::atomic<bool> done[64];
  h3_status st = set_smem_limit(done, paged_attention_kernel, PA_SMEM_BYTES,
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
  a.total_rows = (batch.num_pages * Hkv) << batch.page_log2;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal ? 1 : 0;
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.totals = reinterpret_cast<int64_t*>(base);
  a.first = reinterpret_cast<int64_t*>(base + w.first);
  a.part_o = reinterpret_cast<float*>(base + w.part_o);
  a.part_ml = reinterpret_cast<float*>(base + w.part_ml);
  a.part_rows = w.part_rows;
  a.row_o = reinterpret_cast<float*>(base + w.row_o);
  a.row_ml = reinterpret_cast<float*>(base + w.row_ml);
  a.ctas = std::min(num_sms(), PA_MAX_CTAS);
  if ((st = dev_err(&a.err)) != H3_OK) return st;
  CUtensorMap tq, tk, tv;
  const uint32_t page = 1u << batch.page_log2;
  if ((st = make_tmap_bf16_3d(&tq, q, DH, H, batch.T, DH * 2, static_cast<uint64_t>(ld_q) * 2, 64,
                              a.G, a.tok)) != H3_OK ||
      (st = make_tmap_bf16_2d(&tk, k_cache, DH, a.total_rows, DH * 2, 64, page)) != H3_OK ||
      (st = make_tmap_bf16_2d(&tv, v_cache, DH, a.total_rows, DH * 2, 64, page)) != H3_OK)
    return st;
  paged_attention_kernel<<<a.ctas, PA_THREADS, PA_SMEM_BYTES, s>>>(tq, tk, tv, a);
  if ((st = cuda_fail(cudaGetLastError(), "paged attention launch")) != H3_OK) return st;
  // the join kernel's blocks may take their places while the first kernel
  // runs; they wait for its end before they read anything
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const int64_t want = (static_cast<int64_t>(batch.T) * H + 7) / 8;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(want, a.ctas * 8)));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_fail(cudaLaunchKernelEx(&cfg, paged_join_kernel, a), "paged attention join launch");
}

}  // namespace h3
