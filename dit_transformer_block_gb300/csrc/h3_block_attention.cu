// Block-sparse attention: every block of 256 query rows attends over its own list of key
// blocks (64 or 128 keys), on tcgen05 with S, P and O in tensor memory.
//
// One CTA per (query block, head): two query tiles of 128 rows share each key tile, so
// a 64 KB key and value tile feeds four products (2,048 cycles) and a CTA draws 32 bytes
// per cycle from L2. Two tiles with lists of their own would need twice that, which is
// what an SM gets at best: hence lists of 256 rows. A key tile is one listed block of 128
// keys, or two of 64.
//   * tensor memory: S (128 columns, the two query tiles in turn), O and P (bf16) of both;
//     a softmax reads S into registers and frees it at once, so the other tile's Q K^T
//     overlaps it, and P V reads P from tensor memory. P has
//     the 8 bits of V's type, since both operands of a product have one type: 0.0023 of the output's
//     norm off 64 bits, of which its own rounding to bf16 is 0.0017. (P in two parts would be half
//     as much tensor work again.) The sum that O is divided by is of the weights before rounding;
//   * warps 0-3 / 4-7: softmax of query tile 0 / 1 (thread = row); warp 8: lists and TMA loads,
//     keys and values in five 32 KB slots in the order in which they are used; warp 9:
//     issues the products;
//   * the lists may hold anything: an id outside the keys is loaded from past the last
//     row (zeros) and its keys are masked, as are those past the end of the last block.
// Where the (query block, head)s are fewer than the SMs, a cluster of CTAs shares a list
// and joins its partial results through distributed shared memory, in rank order.
// Bound by the products of bf16 and by the power they draw: 58,758 rows of 42 heads, 92 blocks of
// 64 keys each, 7.4 TFLOP: 4.43 ms (1,680 TFLOP/s), 4.8 to 4.95 ms in a run of seconds. 1,896 rows,
// 96 blocks, 336 items on 152 SMs: 218 us for 128 of products, three waves of which the last is a
// fifth full. 22 rows of 40 heads, 23 blocks of 128: 12.7 us, of which the keys and values once are
// 4.6: seven or eight tiles one after another, each with a whole tile's products, and the join.
#include <algorithm>

#include "h3_attn_common.cuh"
#include "h3_blocks.cuh"
#include "h3_launch.cuh"

namespace h3 {
namespace {

constexpr int BS_SLOTS = 5;
constexpr int BS_COUNTS = 8;  // key tiles whose key counts are kept
constexpr size_t BS_SMEM_BYTES = 1024 + BS_SLOTS * TILE_BYTES + 2 * TILE_BYTES + 512;
static_assert(BS_SMEM_BYTES <= 227 * 1024, "block attention shared memory");
constexpr float BS_KEYS_SEEN = -3.402823466e+38f;

enum BarB {
  BB_Q = 0,
  BB_FULL = 1,
  BB_EMPTY = BB_FULL + BS_SLOTS,
  BB_S = BB_EMPTY + BS_SLOTS,  // S_i written (MMA commit)
  BB_SFREE = BB_S + 2,         // S_i read by the softmax (4 warp arrivals)
  BB_P = BB_SFREE + 2,         // P_i written (4 warp arrivals)
  BB_PVD = BB_P + 2,           // P_i V_j done (MMA commit)
  BB_O = BB_PVD + 2,
  BB_DRAIN = BB_O + 1,
  BB_NUM = BB_DRAIN + 1
};
constexpr uint32_t TB_S = 0, TB_O = 128, TB_P = 384;
// barriers, the TMEM address word, key counts of the tiles under way
static_assert(BB_NUM * 8 + 16 + BS_COUNTS * 4 <= 512, "barrier + count region");
// the join: O of 256 rows in the slots, (maximum, sum) behind it
static_assert(2 * BQ * DH * 4 + 2 * BQ * 8 <= BS_SLOTS * TILE_BYTES, "join region");

struct BlockAttnArgs {
  __nv_bfloat16* o;
  int64_t ld_o;
  const int32_t* ids;
  const int32_t* counts;
  int Lq, Lk, nq, nk;
  int most;        // entries of a list
  int kb;          // keys of a block
  int group;       // query heads per key head
  int cluster;     // CTAs per list
  float scale_log2;
  DevErr err;
};

// Number of the load, in slot order, of K_j and V_j of n tiles: K0 K1 V0 K2 V1 ...
__device__ __forceinline__ int load_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int load_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

// One key tile of the online softmax for the calling thread's row, as in the dense
// kernel (base 2, the scale folded in, the running maximum raised only when exceeded by
// more than RESCALE_THRESHOLD). v0, v1: real keys among the tile's first and last 64. A
// maximum of -inf says that the row has seen no key; rows whose scores are all NaN or
// -inf have the least float instead, so that they end as NaN.
template <class WaitPV>
__device__ __forceinline__ bool softmax_blocks(uint32_t (&sr)[128], uint32_t tP, uint32_t tO,
                                               int v0, int v1, bool o_live, float scale_log2,
                                               float& m, float& l, WaitPV&& wait_pv) {
  if ((v0 & v1) != 64) {  // (both are at most 64)
#pragma unroll
    for (int c = 0; c < 64; ++c) {
      if (c >= v0) sr[c] = 0xff800000u;
      if (c >= v1) sr[64 + c] = 0xff800000u;
    }
  }
  float ma = -INFINITY, mb = -INFINITY, mc = -INFINITY, md = -INFINITY;
#pragma unroll
  for (int c = 0; c < 128; c += 8) {
    ma = max3f(ma, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
    mb = max3f(mb, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
    mc = max3f(mc, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
    md = max3f(md, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
  }
  float mx = max3f(ma, mb, fmaxf(mc, md)) * scale_log2;
  if (v0 + v1 > 0) mx = fmaxf(mx, BS_KEYS_SEEN);
  bool pv_done = !o_live;
  if (__any_sync(0xffffffffu, mx > m + RESCALE_THRESHOLD)) {
    const float m_new = fmaxf(m, mx);
    const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
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
  const float neg_m = m == -INFINITY ? 0.f : -m;  // no key so far: weights of exp2(-inf)
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

__global__ void __launch_bounds__(Q2_THREADS, 1)
    attention_blocks_kernel(const __grid_constant__ CUtensorMap tmQ,
                            const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const BlockAttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sKV = smem;
  uint8_t* sQ = smem + BS_SLOTS * TILE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sQ + 2 * TILE_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + BB_NUM);
  // real keys of key tile j: low half its first 64, high half its last 64
  volatile uint32_t* keys = tmem_slot + 4;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % a.cluster;
  const int qb = static_cast<int>(blockIdx.x) / a.cluster;
  const int h = blockIdx.y;
  const int q0 = qb * 2 * BQ;
  const bool two = q0 + BQ < a.Lq;  // the second query tile has rows
  const int per_tile = BKV / a.kb;  // listed blocks of a key tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < BB_NUM; ++i) mbar_init(bar(i), (i >= BB_SFREE && i < BB_PVD) ? 4 : 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  const int64_t item = static_cast<int64_t>(h) * a.nq + qb;
  const int32_t* list = a.ids + item * a.most;
  // the loading warp has the list's first entries before its length is known (a CTA that does not
  // begin with them reads its own later)
  int now = -1, next = -1;
  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    wait_previous();
    if (lane < a.most) now = list[lane];
    if (32 + lane < a.most) next = list[32 + lane];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_previous();
  const int count = min(max(*(a.counts + item), 0), a.most);
  // this CTA's key tiles
  const int tiles = (count + per_tile - 1) / per_tile;
  const int tile0 = static_cast<int>(static_cast<int64_t>(tiles) * rank / a.cluster);
  const int n = static_cast<int>(static_cast<int64_t>(tiles) * (rank + 1) / a.cluster) - tile0;

  float m = -INFINITY, l = 0.f;  // softmax warps: the row's maximum and sum
  bool ok = true;
  if (warp == 8) {
    // ---------------------------------------------------------- lists and loads
    // The whole warp goes along, since a lane reads one of 32 entries of the list, a batch ahead
    // of their use; lane 0 waits and loads.
    if (n > 0) {
      const int colq = h * DH, colk = h / a.group * DH;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(BB_Q), (two ? 2 : 1) * TILE_BYTES);
        for (int i = 0; i < (two ? 2 : 1); ++i)
          for (int c = 0; c < 2; ++c)
            tma_load_2d(smem_u32(sQ + i * TILE_BYTES + c * BOX_BYTES), &tmQ, bar(BB_Q), colq + c * 64,
                        q0 + i * BQ);
      }
      const int first = tile0 * per_tile, end = min(count, (tile0 + n) * per_tile);
      auto entry = [&](int i) { return first + i < end ? list[first + i] : -1; };
      if (first > 0) {
        now = entry(lane);
        next = entry(32 + lane);
      } else {
        if (lane >= end) now = -1;
        if (32 + lane >= end) next = -1;
      }
      int issued = 0;
      // the first rows of a tile's blocks; past the last key where there is none
      auto rows_of = [&](int j, int (&row)[2], int (&real)[2]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (e < per_tile) {
            const int at = j * per_tile + e;
            const int id = __shfl_sync(0xffffffffu, now, at & 31);
            if ((at & 31) == 31) {
              now = next;
              next = entry(at + 33 + lane);
            }
            const bool in = id >= 0 && id < a.nk;
            row[e] = in ? id * a.kb : a.Lk;
            real[e] = in ? min(a.kb, a.Lk - row[e]) : 0;
          }
        }
      };
      auto load = [&](const CUtensorMap* map, const int (&row)[2]) {
        const int st = issued % BS_SLOTS;
        int done = 1;
        if (lane == 0) {
          done = mbar_wait(bar(BB_EMPTY + st), (static_cast<uint32_t>(issued / BS_SLOTS) & 1u) ^ 1u,
                           a.err, ERR_WAIT_ATTN_PRODUCER);
          if (done) {
            const uint32_t full = bar(BB_FULL + st);
            mbar_arrive_expect_tx(full, TILE_BYTES);
            const uint32_t dst = smem_u32(sKV + st * TILE_BYTES);
            for (int e = 0; e < per_tile; ++e)
              for (int c = 0; c < 2; ++c)
                tma_load_2d(dst + c * BOX_BYTES + e * a.kb * 128, map, full, colk + c * 64, row[e]);
          }
        }
        done = __shfl_sync(0xffffffffu, done, 0);
        issued += done;
        return done != 0;
      };
      int row[2] = {}, before[2] = {}, real[2] = {};
      for (int j = 0; j <= n; ++j) {  // K_j, then V_{j-1}
        before[0] = row[0], before[1] = row[1];
        if (j < n) {
          rows_of(j, row, real);
          if (lane == 0)
            keys[j % BS_COUNTS] = a.kb == 64
                                      ? static_cast<uint32_t>(real[0]) | static_cast<uint32_t>(real[1]) << 16
                                      : static_cast<uint32_t>(min(real[0], 64)) |
                                            static_cast<uint32_t>(max(real[0] - 64, 0)) << 16;
          if (!load(&tmK, row)) break;
        }
        if (j > 0 && !load(&tmV, before)) break;
      }
      if (lane == 0) {
        launch_next();
        // no copy of this CTA may still be landing when it exits
        const uint64_t t0 = globaltimer_ns();
        const uint64_t lim = drain_limit_ns(a.err);
        mbar_wait_drain(bar(BB_Q), 0u, t0, lim);
        for (int i = issued > BS_SLOTS ? issued - BS_SLOTS : 0; i < issued; ++i)
          mbar_wait_drain(bar(BB_FULL + i % BS_SLOTS), static_cast<uint32_t>(i / BS_SLOTS) & 1u, t0,
                          lim);
      }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_qk = idesc_bf16_f32(BQ, BKV, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(BQ, DH, true);
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dk = sdesc_sw128(smem_u32(sKV), 16, 1024);
    const uint64_t dv = sdesc_sw128(smem_u32(sKV), BOX_BYTES, 1024);
    auto wait = [&](int b, uint32_t parity) {
      return mbar_wait_warp(bar(b), parity, a.err, ERR_WAIT_ATTN_MMA);
    };
    auto wait_load = [&](int i) {
      return wait(BB_FULL + i % BS_SLOTS, static_cast<uint32_t>(i / BS_SLOTS) & 1u);
    };
    auto slot = [](int i) { return static_cast<uint32_t>((i % BS_SLOTS) * (TILE_BYTES >> 4)); };
    auto qk = [&](int i, int j) {  // S = Q_i K_j^T
      const uint64_t qd = dq + static_cast<uint32_t>(i * (TILE_BYTES >> 4));
      const uint64_t kd = dk + slot(load_k(j));
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk) {
        const uint32_t off = static_cast<uint32_t>(((kk >> 2) * BOX_BYTES + (kk & 3) * 32) >> 4);
        mma_ss_el(tmem + TB_S, qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
      }
      mma_commit_el(bar(BB_S + i));
    };
    auto pv = [&](int i, int j) {  // O_i += P_i V_j
      const uint64_t vd = dv + slot(load_v(j, n));
#pragma unroll
      for (int kk = 0; kk < BKV / 16; ++kk)
        mma_ts_el(tmem + TB_O + i * 128, tmem + TB_P + i * 64 + kk * 8, vd + kk * (2048 >> 4),
                  idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
      mma_commit_el(bar(BB_PVD + i));
    };
    auto free_load = [&](int i) { mma_commit_el(bar(BB_EMPTY + i % BS_SLOTS)); };
    if (n > 0) {
      bool go = wait(BB_Q, 0u) && wait_load(0);
      if (go) {
        tc_fence_after();
        qk(0, 0);
        if (two) {
          go = wait(BB_SFREE, 0u);
          if (go) {
            tc_fence_after();
            qk(1, 0);
          }
        }
        if (go) free_load(load_k(0));
      }
      // per key tile QK0(j+1) once S1(j) is read, PV0(j), QK1(j+1) once S0(j+1) is, PV1(j);
      // with one query tile QK0(j+1) once S0(j) is read, PV0(j)
      for (int j = 0; go && j < n; ++j) {
        const uint32_t par = static_cast<uint32_t>(j) & 1u;
        const bool more = j + 1 < n;
        if (more) {
          if (!wait_load(load_k(j + 1)) || !wait(BB_SFREE + (two ? 1 : 0), par)) break;
          tc_fence_after();
          qk(0, j + 1);
          if (!two) free_load(load_k(j + 1));
        }
        if (!wait_load(load_v(j, n)) || !wait(BB_P, par)) break;
        tc_fence_after();
        pv(0, j);
        if (two) {
          if (more) {
            if (!wait(BB_SFREE, par ^ 1u)) break;
            tc_fence_after();
            qk(1, j + 1);
            free_load(load_k(j + 1));
          }
          if (!wait(BB_P + 1, par)) break;
          tc_fence_after();
          pv(1, j);
        }
        free_load(load_v(j, n));
      }
    }
    mma_commit_el(bar(BB_O));
    // every product must be done with shared and tensor memory before the CTA frees them
    mma_commit_el(bar(BB_DRAIN));
    mbar_wait_drain(bar(BB_DRAIN), 0u, globaltimer_ns(), drain_limit_ns(a.err));
  } else if (two || warp < 4) {
    // ---------------------------------------------------------- softmax
    const int tile = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + TB_S;
    const uint32_t tO = tmem + lane_base + TB_O + tile * 128;
    const uint32_t tP = tmem + lane_base + TB_P + tile * 64;
    for (int j = 0; j < n; ++j) {
      if (!mbar_wait_warp(bar(BB_S + tile), static_cast<uint32_t>(j) & 1u, a.err,
                          ERR_WAIT_ATTN_SOFTMAX)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t real = keys[j % BS_COUNTS];
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
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BB_SFREE + tile));
      auto wait_pv = [&]() {  // P_i V_{j-1} done with P_i and O_i
        const bool done = mbar_wait_warp(bar(BB_PVD + tile), static_cast<uint32_t>(j - 1) & 1u,
                                         a.err, ERR_WAIT_ATTN_SOFTMAX);
        tc_fence_after();
        return done;
      };
      if (!softmax_blocks(sr, tP, tO, static_cast<int>(real & 0xffffu),
                          static_cast<int>(real >> 16), j > 0, a.scale_log2, m, l, wait_pv)) {
        ok = false;
        break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BB_P + tile));
    }
    if (ok) ok = mbar_wait_warp(bar(BB_O), 0u, a.err, ERR_WAIT_ATTN_SOFTMAX);
    tc_fence_after();
    const int row = tile * BQ + (warp & 3) * 32 + lane;
    const bool row_ok = q0 + row < a.Lq;
    if (a.cluster == 1) {
      __nv_bfloat16* orow = a.o + static_cast<int64_t>(q0 + row) * a.ld_o + h * DH;
      if (n == 0) {  // no key: zeros
        if (row_ok)
          for (int c = 0; c < DH / 8; ++c) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0, 0, 0, 0);
      } else if (ok) {
        // (a list of nothing but ids outside the keys: O is 0, and stays so)
        store_o_row(tO, m == -INFINITY ? 1.f : l, orow, row_ok, nullptr);
      }
    } else {
      // partial results to shared memory, where no load and no product is under way any
      // more: float4 c of row r at c ^ (r & 31), so that a warp's stores spread over the banks
      float4* po = reinterpret_cast<float4*>(sKV) + row * (DH / 4);
      if (n > 0) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t ov[32];
          tmem_ld32(tO + c * 32, ov);
          tmem_ld_wait();
          tmem_reg_fence(ov);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            po[(c * 8 + i) ^ lane] =
                make_float4(__uint_as_float(ov[4 * i]), __uint_as_float(ov[4 * i + 1]),
                            __uint_as_float(ov[4 * i + 2]), __uint_as_float(ov[4 * i + 3]));
        }
      }
      reinterpret_cast<float2*>(sKV + 2 * BQ * DH * 4)[row] =
          make_float2(n > 0 ? m : -INFINITY, l);
    }
  }

  __syncwarp();
  tc_fence_before();
  if (a.cluster == 1) {
    __syncthreads();
  } else {
    cluster_sync_all();
    // rows in turn over the cluster's warps, a lane four channels
    const int rows = min(2 * BQ, a.Lq - q0);
    const uint32_t base = smem_u32(sKV);
    for (int r = rank * 10 + warp; r < rows; r += a.cluster * 10) {
      float top = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      // every part's loads are under way before the first is used
      float2 ml[8];
      float4 y[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        if (p < a.cluster) {
          const uint32_t at = mapa_shared(base, p);
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                       : "=f"(ml[p].x), "=f"(ml[p].y)
                       : "r"(at + 2 * BQ * DH * 4 + r * 8)
                       : "memory");
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(y[p].x), "=f"(y[p].y), "=f"(y[p].z), "=f"(y[p].w)
                       : "r"(at + r * (DH * 4) + ((lane ^ (r & 31)) * 16))
                       : "memory");
        }
      }
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        if (p >= a.cluster || ml[p].x == -INFINITY) continue;  // (or no key there: y is anything)
        const float next = fmaxf(top, ml[p].x);
        const float f = top == -INFINITY ? 0.f : ex2_approx(top - next), w = ex2_approx(ml[p].x - next);
        top = next;
        sum = fmaf(ml[p].y, w, sum * f);
        acc.x = fmaf(y[p].x, w, acc.x * f);
        acc.y = fmaf(y[p].y, w, acc.y * f);
        acc.z = fmaf(y[p].z, w, acc.z * f);
        acc.w = fmaf(y[p].w, w, acc.w * f);
      }
      const float inv = top == -INFINITY ? 0.f : 1.0f / sum;
      *reinterpret_cast<uint2*>(a.o + static_cast<int64_t>(q0 + r) * a.ld_o + h * DH + lane * 4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
    cluster_sync_all();  // a peer may still be reading this CTA's results
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

h3_status launch_attention_blocks(const void* q, int64_t ld_q, const void* k, int64_t ld_k,
                                  const void* v, int64_t ld_v, void* o, int64_t ld_o,
                                  const int32_t* ids, const int32_t* counts, int max_blocks, int Lq,
                                  int Lk, int H, int Hkv, int k_block, float scale,
                                  cudaStream_t s) {
  static std::atomic<bool> done[64];
  h3_status st = set_smem_limit(done, attention_blocks_kernel, BS_SMEM_BYTES,
                                "block attention: set shared memory size");
  if (st != H3_OK) return st;
  BlockAttnArgs a{};
  a.o = static_cast<__nv_bfloat16*>(o);
  a.ld_o = ld_o;
  a.ids = ids;
  a.counts = counts;
  a.Lq = Lq;
  a.Lk = Lk;
  a.nq = (Lq + 2 * BQ - 1) / (2 * BQ);
  a.nk = (Lk + k_block - 1) / k_block;
  a.most = max_blocks;
  a.kb = k_block;
  a.group = H / Hkv;
  a.scale_log2 = scale * 1.4426950408889634f;
  if ((st = dev_err(&a.err)) != H3_OK) return st;
  // a list is shared by as many CTAs as all of them find room for, two key tiles each at least
  const int64_t items = static_cast<int64_t>(a.nq) * H;
  const int64_t tiles = (static_cast<int64_t>(max_blocks) * k_block + BKV - 1) / BKV;
  static std::atomic<int> room[64][9];
  a.cluster = 1;
  for (int c = 8; c >= 2; --c) {
    if (items * c > num_sms() || tiles < 2 * c) continue;
    if (clusters_at_once(room, attention_blocks_kernel, Q2_THREADS, BS_SMEM_BYTES, c) >= items) {
      a.cluster = c;
      break;
    }
  }
  CUtensorMap tq, tk, tv;
  const uint64_t wq = static_cast<uint64_t>(H) * DH, wk = static_cast<uint64_t>(Hkv) * DH;
  if ((st = make_tmap_bf16_2d(&tq, q, wq, Lq, ld_q * 2, 64, BQ)) != H3_OK) return st;
  if ((st = make_tmap_bf16_2d(&tk, k, wk, Lk, ld_k * 2, 64, k_block)) != H3_OK) return st;
  if ((st = make_tmap_bf16_2d(&tv, v, wk, Lk, ld_v * 2, 64, k_block)) != H3_OK) return st;
  return cuda_fail(launch_overlapped(attention_blocks_kernel,
                                     dim3(static_cast<unsigned>(a.nq) * a.cluster, H), Q2_THREADS,
                                     BS_SMEM_BYTES, a.cluster, s, tq, tk, tv, a),
                   "block attention launch");
}

}  // namespace h3
