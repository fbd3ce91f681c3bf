// Choosing key blocks for block-sparse attention: scores of pooled blocks, and the
// selection of the best of every query block.
//
// Scores: the mean row of every query block and key block (FP32), then one product of
// the means per head. The pooling reads q and k once and is bound by HBM. A product with
// rounded means would choose other blocks, so it has FP32's accuracy: each mean is the sum
// of two TF32 numbers, and three products of those (all but that of the two smaller parts)
// run on the tensor cores; for few query blocks it runs on the CUDA cores.
//
// Selection: the max_blocks-th largest score is found by counting, then one pass writes
// the chosen indices in ascending order. A warp per row of scores, longer ones a CTA.
//
// Measured, pooling and product together: 58,758 rows of 42 + 42 heads, 1.30 GB, in blocks of 64
// keys: 230 us; 1,896 rows of 40 heads and 29,034 of 8, in blocks of 128: 20 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "h3_blocks.cuh"
#include "h3_internal.cuh"
#include "h3_launch.cuh"

namespace h3 {
namespace {

constexpr int DHB = 128;

// ------------------------------------------------------------------ pooling
// One CTA per SM goes over (block of rows, two neighbouring heads) after the other. Its rows
// come in pieces of at most 128 rows x 256 channels (64 KB) by TMA, three of them under way,
// so that HBM is read without a pause whatever the sums do. Each of eight warps sums 32 of the
// channels, eight rows at a time, and has their mean without another warp's: four boxes
// of 64 channels, swizzled, so that its eight rows lie in different banks.
// (1,896 + 29,034 rows of 40 and 8 heads, 79 MB, with their product: 20 us; 24 where every CTA
// loads its block into registers, 28 with the rows of a piece spread over the warps, which then
// have to meet. 58,758 rows of 42 + 42 heads, 1.26 GB: 200 us, 195 and 206.)
constexpr int POOL_WARPS = 8;
constexpr int POOL_THREADS = POOL_WARPS * 32 + 32;  // and a warp that loads
constexpr int POOL_ROWS = 128, POOL_SLOTS = 3;
constexpr int POOL_BOX_BYTES = POOL_ROWS * 128;     // 64 channels
constexpr int POOL_SLOT_BYTES = 4 * POOL_BOX_BYTES;
constexpr size_t POOL_SMEM_BYTES = 1024 + POOL_SLOTS * POOL_SLOT_BYTES + 2 * POOL_SLOTS * 8;
static_assert(POOL_SMEM_BYTES <= 227 * 1024, "pooling shared memory");

struct PoolSide {
  int L, heads, block, blocks;
  int pairs;   // pairs of heads
  int items;   // blocks * pairs
  float* out;  // [heads][blocks][128]
  float* low;  // as out, or NULL: out is then rounded to TF32, and this is what that leaves
};

// The nearest number of 11 significant bits (ties away from zero).
__device__ __forceinline__ float to_tf32(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u);
}

__global__ void __launch_bounds__(POOL_THREADS, 1)
    pool_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const PoolSide q, const PoolSide k, const DevErr err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + POOL_SLOTS * POOL_SLOT_BYTES);  // full, empty
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < POOL_SLOTS; ++i) {
      mbar_init(bar(i), 1);
      mbar_init(bar(POOL_SLOTS + i), POOL_WARPS);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  __syncthreads();
  wait_previous();
  const int items = q.items + k.items;

  if (warp == POOL_WARPS) {
    if (lane == 0) {
      int st = 0, issued = 0;
      uint32_t phase = 1;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const bool is_q = item < q.items;
        const PoolSide& s = is_q ? q : k;
        const int id = item - (is_q ? 0 : q.items);
        const int row0 = id / s.pairs * s.block, head0 = id % s.pairs * 2;
        const int rows = min(s.block, s.L - row0), box = min(s.block, POOL_ROWS);
        for (int r = 0; r < rows; r += POOL_ROWS) {
          ok = mbar_wait(bar(POOL_SLOTS + st), phase, err, ERR_WAIT_POOL_PRODUCER);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(st), box * 2 * DHB * 2);
          for (int c = 0; c < 4; ++c)
            tma_load_2d(smem_u32(smem + st * POOL_SLOT_BYTES + c * POOL_BOX_BYTES), is_q ? &tmQ : &tmK,
                        bar(st), head0 * DHB + c * 64, row0 + r);
          ++issued;
          if (++st == POOL_SLOTS) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
      launch_next();
      const uint64_t t0 = globaltimer_ns();
      for (int i = issued > POOL_SLOTS ? issued - POOL_SLOTS : 0; i < issued; ++i)
        mbar_wait_drain(bar(i % POOL_SLOTS), static_cast<uint32_t>(i / POOL_SLOTS) & 1u, t0,
                        drain_limit_ns(err));
    }
    return;
  }
  // lane: row lane / 4 of eight, channels 8 (lane % 4) .. of the warp's 32: half of a box's row
  const int sub = lane >> 2, chunk = (warp & 1) * 4 + (lane & 3);
  const uint32_t off = (warp >> 1) * POOL_BOX_BYTES + sub * 128 + ((chunk ^ sub) << 4);
  int st = 0;
  uint32_t phase = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const bool is_q = item < q.items;
    const PoolSide& s = is_q ? q : k;
    const int id = item - (is_q ? 0 : q.items);
    const int blk = id / s.pairs, head = id % s.pairs * 2 + (warp >> 2);
    const int rows = min(s.block, s.L - blk * s.block);
    float acc[8] = {};
    for (int r0 = 0; r0 < rows; r0 += POOL_ROWS) {
      // (where a wait runs out, this one returns and so does every later one, soon)
      mbar_wait(bar(st), phase, err, ERR_WAIT_POOL_SUMS);
      const uint8_t* x = smem + st * POOL_SLOT_BYTES + off;
      const int n = min(POOL_ROWS, rows - r0);
#pragma unroll 8
      for (int r = sub; r < n; r += 8, x += 1024) {
        const uint4 v = *reinterpret_cast<const uint4*>(x);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[2 * j] += bf16_lo(w[j]);
          acc[2 * j + 1] += bf16_hi(w[j]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(POOL_SLOTS + st));
      if (++st == POOL_SLOTS) {
        st = 0;
        phase ^= 1u;
      }
    }
    // over the eight rows, each step leaving a lane half of its channels; then channel
    // 8 (lane % 4) + sub is lane's
#pragma unroll
    for (int m = 4, n = 4; m >= 1; m >>= 1, n >>= 1) {
      const bool high = (sub & m) != 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < n) {
          const float give = high ? acc[j] : acc[j + n], keep = high ? acc[j + n] : acc[j];
          acc[j] = keep + __shfl_xor_sync(0xffffffffu, give, m * 4);
        }
      }
    }
    if (head < s.heads) {
      const float mean = acc[0] / static_cast<float>(rows);
      const int64_t at = (static_cast<int64_t>(head) * s.blocks + blk) * DHB + (warp & 3) * 32 +
                         (lane & 3) * 8 + sub;
      if (s.low != nullptr) {
        // (NaN and infinity go whole into the first part)
        const float hi = fabsf(mean) < INFINITY ? to_tf32(mean) : mean;
        s.out[at] = hi;
        s.low[at] = fabsf(mean) < INFINITY ? to_tf32(mean - hi) : 0.f;
      } else {
        s.out[at] = mean;
      }
    }
  }
}

// ------------------------------------------------------------------ product
// Few query blocks (at most eight): scores[h] = scale * mq[h] mk[g]^T, a warp 16 key blocks of a
// head, whose query means its lanes hold, four channels each.
constexpr int FEW = 8, FEW_WARPS = 4, FEW_KEYS = 16;

__global__ void __launch_bounds__(FEW_WARPS * 32)
    block_scores_few_kernel(const float* mq, const float* mk, float* scores, int nq, int nk, int group,
                            float scale) {
  const int lane = threadIdx.x & 31, h = blockIdx.y, g = h / group;
  const int b0 = (blockIdx.x * FEW_WARPS + (threadIdx.x >> 5)) * FEW_KEYS;
  wait_previous();
  const float4* kp = reinterpret_cast<const float4*>(mk + static_cast<int64_t>(g) * nk * DHB) + lane;
  const float4* qp = reinterpret_cast<const float4*>(mq + static_cast<int64_t>(h) * nq * DHB) + lane;
  float4 x[FEW], y[FEW_KEYS];
#pragma unroll
  for (int t = 0; t < FEW; ++t)
    x[t] = t < nq ? qp[t * (DHB / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < FEW_KEYS; ++i)
    y[i] = b0 + i < nk ? kp[static_cast<int64_t>(b0 + i) * (DHB / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
  launch_next();
#pragma unroll
  for (int t = 0; t < FEW; ++t) {
    if (t >= nq) break;
    // 16 sums over the lanes, each step leaving a lane half of them: it ends with key block
    // lane / 2's
    float d[FEW_KEYS];
#pragma unroll
    for (int i = 0; i < FEW_KEYS; ++i)
      d[i] = fmaf(x[t].x, y[i].x, x[t].y * y[i].y) + fmaf(x[t].z, y[i].z, x[t].w * y[i].w);
#pragma unroll
    for (int m = 16, n = 8; n >= 1; m >>= 1, n >>= 1) {
      const bool high = (lane & m) != 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) {
          const float give = high ? d[j] : d[j + n], keep = high ? d[j + n] : d[j];
          d[j] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
      }
    }
    const float sum = d[0] + __shfl_xor_sync(0xffffffffu, d[0], 1);
    const int b = b0 + (lane >> 1);
    if ((lane & 1) == 0 && b < nk)
      scores[(static_cast<int64_t>(h) * nq + t) * nk + b] = sum * scale;
  }
}

// A score from means in two parts, in FP32: the steps of the kernel for few query blocks, a warp's
// lanes having four channels each. The parts add up to the mean (11 bits each; the first alone
// where it is infinite or NaN).
__device__ __noinline__ float score_of_parts(const float* qh, const float* ql, const float* kh,
                                             const float* kl) {
  const int lane = threadIdx.x & 31;
  auto mean = [&](const float* high, const float* low) {
    const float4 a = reinterpret_cast<const float4*>(high)[lane];
    const float4 b = reinterpret_cast<const float4*>(low)[lane];
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
  };
  const float4 x = mean(qh, ql), y = mean(kh, kl);
  float d = fmaf(x.x, y.x, x.y * y.y) + fmaf(x.z, y.z, x.w * y.w);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
  return d;
}

// scores[h] = scale * mq[h] mk[g]^T: a CTA per SM takes one tile of 128 query blocks x 128 key
// blocks of a head after the other (230 x 919 blocks of 42 heads in 17 us, 30 with a CTA per tile
// and 75 by FP32 FMAs). A stage is 32 channels (128 bytes a row) of both parts of both operands;
// warp 0 loads (TMA), warp 1 issues, per 8 channels, three products into one of two FP32
// accumulators, and warps 2 to 5 write the other's scores, row by row through shared memory,
// since a row of them starts at any 4 bytes. A score that is not finite is formed again in FP32:
// an infinite part times the other operand's second part, of any sign or 0, is no part of it. (9,660
// x 919 scores of NaN alone: 7.8 ms instead of 0.23, pooling included.)
constexpr int TC_TILE = 128, TC_STAGES = 3, TC_STEPS = DHB / 32;
constexpr int TC_PART = TC_TILE * 128;         // 16 KB: 128 rows x 32 channels
constexpr int TC_STAGE_BYTES = 4 * TC_PART;    // A high, A low, B high, B low
constexpr int TC_THREADS = 192;
constexpr int TC_OUT = 32 * 128;               // a warp's 32 rows x 32 scores
constexpr size_t TC_SMEM_BYTES = 1024 + TC_STAGES * TC_STAGE_BYTES + 4 * TC_OUT + 128;
static_assert(TC_SMEM_BYTES <= 227 * 1024, "block scores shared memory");
enum BarTc {
  BT_FULL = 0,                     // stage landed
  BT_EMPTY = BT_FULL + TC_STAGES,  // stage read by the products
  BT_DONE = BT_EMPTY + TC_STAGES,  // [2] accumulator written
  BT_READ = BT_DONE + 2,           // [2] accumulator read (4 warps)
  BT_DRAIN = BT_READ + 2,
  BT_NUM
};
static_assert(BT_NUM * 8 + 8 <= 128, "barrier region");

__device__ __forceinline__ void mma_tf32_el(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct ScoreSizes {
  const float *qh, *ql, *kh, *kl;  // the means' two parts, [heads][blocks][128]
  int nq, nk, group;
  int across, down, tiles;  // tiles of a head along the key blocks, the query blocks; of all heads
};

// Head, first query block and first key block of a tile.
__device__ __forceinline__ void score_tile(int tile, const ScoreSizes& z, int& h, int& t0, int& b0) {
  const int r = tile / z.across;
  b0 = (tile - r * z.across) * TC_TILE;
  h = r / z.down;
  t0 = (r - h * z.down) * TC_TILE;
}

__global__ void __launch_bounds__(TC_THREADS, 1)
    block_scores_kernel(const __grid_constant__ CUtensorMap tmQh, const __grid_constant__ CUtensorMap tmQl,
                        const __grid_constant__ CUtensorMap tmKh, const __grid_constant__ CUtensorMap tmKl,
                        float* scores, const ScoreSizes z, float scale, const DevErr err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* out = smem + TC_STAGES * TC_STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(out + 4 * TC_OUT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + BT_NUM);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < BT_NUM; ++i) mbar_init(bar(i), i == BT_READ || i == BT_READ + 1 ? 4 : 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmQh);
    tma_prefetch_desc(&tmQl);
    tma_prefetch_desc(&tmKh);
    tma_prefetch_desc(&tmKl);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 2 * TC_TILE);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_previous();

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0, st = 0;
      uint32_t phase = 1;
      bool ok = true;
      for (int tile = blockIdx.x; tile < z.tiles && ok; tile += gridDim.x) {
        // (rows past the head's last block are the next head's, or zeros; nothing is stored of them)
        int h, t0, b0;
        score_tile(tile, z, h, t0, b0);
        const int qrow = h * z.nq + t0, krow = h / z.group * z.nk + b0;
        for (int c = 0; c < TC_STEPS; ++c) {
          if (!(ok = mbar_wait(bar(BT_EMPTY + st), phase, err, ERR_WAIT_SCORES_PRODUCER))) break;
          const uint32_t full = bar(BT_FULL + st), dst = smem_u32(smem + st * TC_STAGE_BYTES);
          mbar_arrive_expect_tx(full, TC_STAGE_BYTES);
          tma_load_2d(dst, &tmQh, full, c * 32, qrow);
          tma_load_2d(dst + TC_PART, &tmQl, full, c * 32, qrow);
          tma_load_2d(dst + 2 * TC_PART, &tmKh, full, c * 32, krow);
          tma_load_2d(dst + 3 * TC_PART, &tmKl, full, c * 32, krow);
          ++issued;
          if (++st == TC_STAGES) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
      launch_next();
      const uint64_t at = globaltimer_ns();
      for (int c = issued > TC_STAGES ? issued - TC_STAGES : 0; c < issued; ++c)
        mbar_wait_drain(bar(BT_FULL + c % TC_STAGES), static_cast<uint32_t>(c / TC_STAGES) & 1u, at,
                        drain_limit_ns(err));
    }
  } else if (warp == 1) {
    // instruction descriptor: f32 accumulator, TF32 operands (format 2), both K-major
    constexpr uint32_t idesc = (1u << 4) | (2u << 7) | (2u << 10) |
                               (static_cast<uint32_t>(TC_TILE >> 3) << 17) |
                               (static_cast<uint32_t>(TC_TILE >> 4) << 24);
    const uint64_t base = sdesc_sw128(smem_u32(smem), 16, 1024);
    auto wait = [&](int b, uint32_t parity) {
      return mbar_wait_warp(bar(b), parity, err, ERR_WAIT_SCORES_MMA);
    };
    int st = 0, n = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < z.tiles && ok; tile += gridDim.x, ++n) {
      const int acc = n & 1;
      if (!(ok = wait(BT_READ + acc, (static_cast<uint32_t>(n >> 1) & 1u) ^ 1u))) break;
      for (int c = 0; c < TC_STEPS; ++c) {
        if (!(ok = wait(BT_FULL + st, phase))) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * TC_TILE;
        const uint64_t ah = base + static_cast<uint32_t>(st * (TC_STAGE_BYTES >> 4));
        const uint64_t al = ah + (TC_PART >> 4), bh = ah + (2 * TC_PART >> 4);
        const uint64_t bl = ah + (3 * TC_PART >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mma_tf32_el(d, ah + k * 2, bl + k * 2, idesc, (c | k) != 0 ? 1u : 0u);
          mma_tf32_el(d, al + k * 2, bh + k * 2, idesc, 1u);
          mma_tf32_el(d, ah + k * 2, bh + k * 2, idesc, 1u);
        }
        mma_commit_el(bar(BT_EMPTY + st));
        if (++st == TC_STAGES) {
          st = 0;
          phase ^= 1u;
        }
      }
      if (ok) mma_commit_el(bar(BT_DONE + acc));
    }
    mma_commit_el(bar(BT_DRAIN));
    mbar_wait_drain(bar(BT_DRAIN), 0u, globaltimer_ns(), drain_limit_ns(err));
  } else {
    const int quarter = warp & 3;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    // 32 rows x 32 scores: float4 c of row r at c ^ (r & 7)
    float4* rows = reinterpret_cast<float4*>(out + (warp - 2) * TC_OUT);
    const float* words = reinterpret_cast<const float*>(rows);
    int n = 0;
    for (int tile = blockIdx.x; tile < z.tiles; tile += gridDim.x, ++n) {
      int h, t0, b0;
      score_tile(tile, z, h, t0, b0);
      const int acc = n & 1;
      if (!mbar_wait_warp(bar(BT_DONE + acc), static_cast<uint32_t>(n >> 1) & 1u, err,
                          ERR_WAIT_SCORES_EPILOGUE))
        break;
      tc_fence_after();
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_row + acc * TC_TILE + c * 32, v[c]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_reg_fence(v[c]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BT_READ + acc));
      const int first = t0 + quarter * 32, m = min(32, z.nq - first);
      float* o = scores + (static_cast<int64_t>(h) * z.nq + first) * z.nk + b0 + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (m <= 0 || b0 + c * 32 >= z.nk) break;
        float odd = 0.f;  // NaN where a score is not finite
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 f =
              make_float4(__uint_as_float(v[c][4 * j]) * scale, __uint_as_float(v[c][4 * j + 1]) * scale,
                          __uint_as_float(v[c][4 * j + 2]) * scale, __uint_as_float(v[c][4 * j + 3]) * scale);
          odd = fmaf(f.x, 0.f, fmaf(f.y, 0.f, fmaf(f.z, 0.f, fmaf(f.w, 0.f, odd))));
          rows[lane * 8 + (j ^ (lane & 7))] = f;
        }
        __syncwarp();
        const bool mine = b0 + c * 32 + lane < z.nk;
        auto word = [&](int r) { return words[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)]; };
        auto store = [&](int r) {
          if (mine) o[static_cast<int64_t>(r) * z.nk + c * 32] = word(r);
        };
        if (m == 32) {
#pragma unroll
          for (int r = 0; r < 32; ++r) store(r);
        } else {
          for (int r = 0; r < m; ++r) store(r);
        }
        if (__any_sync(0xffffffffu, odd != odd)) {
          for (int r = 0; r < m; ++r) {
            uint32_t again = __ballot_sync(0xffffffffu, mine && !(fabsf(word(r)) < INFINITY));
            while (again != 0u) {
              const int i = __ffs(again) - 1;
              again &= again - 1u;
              const int64_t qa = (static_cast<int64_t>(h) * z.nq + first + r) * DHB;
              const int64_t ka = (static_cast<int64_t>(h / z.group) * z.nk + b0 + c * 32 + i) * DHB;
              const float f = score_of_parts(z.qh + qa, z.ql + qa, z.kh + ka, z.kl + ka) * scale;
              if (lane == i) o[static_cast<int64_t>(r) * z.nk + c * 32] = f;
            }
          }
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * TC_TILE);
  }
}

// ---------------------------------------------------------------- selection
// Scores as integers of the same order, -0 as +0; NONE for what is never selected (-inf, NaN),
// below all others, and KEPT for the blocks that always are, above them.
constexpr uint32_t NONE = 0x007fffffu, KEPT = 0xffffffffu;

__device__ __forceinline__ uint32_t select_key(float f) {
  const uint32_t u = __float_as_uint(fmaxf(f, -INFINITY) + 0.f);  // (of a NaN the maximum is -inf)
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

constexpr int SEL_WARPS = 4;

// Rows r of a 32 x 32 bit matrix, one in every lane, to its columns.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
  constexpr uint32_t keep[5] = {0x0000ffffu, 0x00ff00ffu, 0x0f0f0f0fu, 0x33333333u, 0x55555555u};
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int m = 16 >> i;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, m);
    x = (lane & m) != 0 ? (x & ~keep[i]) | ((y >> m) & keep[i]) : (x & keep[i]) | ((y & keep[i]) << m);
  }
  return x;
}

// Sum of v over the lanes before this one.
__device__ __forceinline__ int lanes_before(int v, int lane) {
  int t = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, t, m);
    if (lane >= m) t += o;
  }
  return t - v;
}

// Rows of at most 32 * IPT scores (IPT up to 32): a warp per row, whose keys stay in its
// registers. The threshold T (the least selected key) is looked for between lo and hi, of
// which at least and fewer than `most` keys are not below; every step counts the keys from a
// place between them on. The first place is where a normal distribution of the row's mean and
// deviation (of every other 32 scores) has `most` (z deviations above the mean), the second as
// far from it as that density says, a dozen keys further, and from then on the middle: rows
// as scores are take two or three steps, any others at most 32 more. With at most 32 keys left
// between lo and hi, a lane takes one, and they go from the largest down. Bound by
// instructions, 1,740 to a row of 919 and 0.55 of the issue slots; so indices are not written 32
// scores at a time but from each lane's bits, a 32 x 32 matrix that is transposed, where a lane
// then has 32 neighbouring ones. (9,660 rows of 919 scores, 91 selected, in 22 us, 6 for their bytes;
// 27 with the indices written by a vote per 32 scores. That is of normal scores; of log-normal
// ones 32, of a peak around one place 36, of a wave with the frame's length 23.)
template <int IPT>
__global__ void __launch_bounds__(SEL_WARPS * 32)
    block_select_warp_kernel(const float* scores, int32_t* ids, int32_t* counts, int rows, int nk,
                             int most, int first, int last, float z, float density) {
  __shared__ uint32_t left[SEL_WARPS][32];
  wait_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * SEL_WARPS + warp;
  if (row >= rows) return;
  const float* s = scores + static_cast<int64_t>(row) * nk;
  int32_t* out = ids + static_cast<int64_t>(row) * most;
  uint32_t key[IPT];
  float sum = 0.f, sum2 = 0.f;
#pragma unroll
  for (int r = 0; r < IPT; ++r)
    key[r] = __float_as_uint(r * 32 + lane < nk ? s[r * 32 + lane] : -INFINITY);
#pragma unroll
  for (int r = 0; r < IPT; ++r) {
    const float f = __uint_as_float(key[r]);
    if ((r & 1) == 0) {
      const float v = f > -INFINITY ? f : 0.f;
      sum += v;
      sum2 = fmaf(v, v, sum2);
    }
    key[r] = select_key(f);
  }
  const int kept = min(first + last, nk);
  if (kept > 0) {
#pragma unroll
    for (int r = 0; r < IPT; ++r)
      if (r * 32 < first || r * 32 + 32 > nk - last) {
        const int i = r * 32 + lane;
        if (i < nk && (i < first || i >= nk - last)) key[r] = KEPT;
      }
  }
  // T, and how many of the keys equal to it are selected (the first of them)
  uint32_t T = NONE;
  int equal = 0;
  if (kept >= most) {
    T = KEPT - 1u;
  } else if (nk > most) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, m);
      sum2 += __shfl_xor_sync(0xffffffffu, sum2, m);
    }
    const float n = static_cast<float>((nk + 63) / 64 * 32);  // (of the mean; a guess is enough)
    const float mean = sum / n;
    const float dev = sqrtf(fmaxf(sum2 / n - mean * mean, 0.f));
    const float per_key = dev / (static_cast<float>(nk) * density);
    uint32_t lo = NONE, hi = KEPT;
    int c_lo = nk, c_hi = kept;  // keys from lo, from hi on
    float at = fmaf(z, dev, mean);
    for (int step = 0;; ++step) {
      uint32_t place = lo + (hi - lo) / 2;
      if (step < 2) {
        const uint32_t k = select_key(at);
        if (k > lo && k < hi) place = k;
      }
      int c = 0;
#pragma unroll
      for (int r = 0; r < IPT; ++r) c += key[r] >= place;
      c = __reduce_add_sync(0xffffffffu, c);
      if (c >= most) {
        lo = place, c_lo = c;
        if (c == most) break;
        at = fmaf(static_cast<float>(c - most + 12), per_key, at);
      } else {
        hi = place, c_hi = c;
        at = fmaf(static_cast<float>(c - most - 12), per_key, at);
      }
      if (c_lo - c_hi <= 32 || hi - lo == 1u) break;
    }
    int need = most - c_hi;
    if (c_lo == most) {
      T = lo - 1u;  // all from lo on
    } else if (hi - lo == 1u) {
      T = lo;
      equal = need;
    } else {
      // the keys between, read again where they lie
      uint32_t bits = 0;
#pragma unroll
      for (int r = 0; r < IPT; ++r) bits |= key[r] - lo < hi - lo ? 1u << r : 0u;
      uint32_t mine = transpose_bits(bits, lane);  // scores 32 lane .. 32 lane + 31
      if (lane * 32 + 32 > nk) mine &= lane * 32 < nk ? (1u << (nk & 31)) - 1u : 0u;
      int at_left = lanes_before(__popc(mine), lane);
      while (mine != 0u) {
        const int j = __ffs(mine) - 1;
        mine &= mine - 1u;
        left[warp][at_left++] = select_key(s[lane * 32 + j]);
      }
      __syncwarp();
      uint32_t k = lane < c_lo - c_hi ? left[warp][lane] : 0u;
      for (;;) {
        T = __reduce_max_sync(0xffffffffu, k);
        const int same = __popc(__ballot_sync(0xffffffffu, k == T));
        if (same >= need || T == 0u) {
          equal = same == need ? 0 : need;
          if (same == need) --T;  // all of them: what is above T - 1
          break;
        }
        need -= same;
        if (k == T) k = 0u;
      }
    }
    if (T <= NONE) T = NONE, equal = 0;  // fewer than wanted: all but -inf and NaN
  }
  launch_next();
  uint32_t bits = 0, same = 0;
#pragma unroll
  for (int r = 0; r < IPT; ++r) bits |= key[r] > T ? 1u << r : 0u;
  bits = transpose_bits(bits, lane);
  if (equal > 0) {
#pragma unroll
    for (int r = 0; r < IPT; ++r) same |= key[r] == T ? 1u << r : 0u;
    same = transpose_bits(same, lane);
    int take = min(max(equal - lanes_before(__popc(same), lane), 0), __popc(same));
    while (take-- > 0) {  // the first of them
      bits |= same & (0u - same);
      same &= same - 1u;
    }
  }
  const int mine = __popc(bits);
  int at = lanes_before(mine, lane);
  const int n = __shfl_sync(0xffffffffu, at + mine, 31);
  while (bits != 0u) {
    out[at++] = lane * 32 + __ffs(bits) - 1;
    bits &= bits - 1u;
  }
  for (int i = n + lane; i < most; i += 32) out[i] = -1;
  if (lane == 0) counts[row] = n;
}

// Longer rows: a CTA per row, a radix search of 8 bits a pass over the scores in L1 and L2, up to
// four of them, and two passes that write. (9,660 rows of 1,025 / 2,048 / 4,096 scores, a tenth of
// them selected: 103 / 134 / 226 us, 6 / 13 / 26 for their bytes, whatever the scores; a warp takes 21
// to 36 for 1,024. The border is where a lane's 32 bits of the matrix above end.)
template <int T>
__global__ void __launch_bounds__(T)
    block_select_kernel(const float* scores, int32_t* ids,
                        int32_t* counts, int nk, int most, int first, int last) {
  __shared__ int hist[256];
  __shared__ int found[3];       // bin, still needed in it, how many it holds
  __shared__ int warp_gt[T / 32], warp_eq[T / 32];
  const int64_t row = blockIdx.x;
  const float* s = scores + row * nk;
  int32_t* out = ids + row * most;
  wait_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto key = [&](int i) { return i < first || i >= nk - last ? KEPT : select_key(s[i]); };

  // threshold: what is above it is selected, and of what is equal to it the first `equal`
  uint32_t prefix = 0, mask = 0, threshold = NONE;
  int need = most, equal = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += T) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < nk; i += T) {
      const uint32_t k = key(i);
      if (k > NONE && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds bins 255 - 8 l .. 248 - 8 l: counts from the top down
      int c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - 8 * lane - j];
      int above = sum;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, above, m);
        if (lane >= m) above += t;
      }
      const int total = __shfl_sync(0xffffffffu, above, 31);
      above -= sum;  // in the bins above this lane's
      if (total <= need) {  // (first pass only: fewer than wanted, all of them)
        if (lane == 0) found[0] = -1;
      } else if (above < need && above + sum >= need) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (above < need && above + c[j] >= need) {
            found[0] = 255 - 8 * lane - j;
            found[1] = need - above;
            found[2] = c[j];
          }
          above += c[j];
        }
      }
    }
    __syncthreads();
    if (found[0] < 0) break;  // threshold NONE
    prefix |= static_cast<uint32_t>(found[0]) << shift;
    mask |= 255u << shift;
    need = found[1];
    if (need == found[2]) {  // all of the bin
      threshold = max(prefix, NONE + 1u) - 1u;
      equal = 0;
      break;
    }
    threshold = prefix;
    equal = need;
  }

  const int per = (nk + T - 1) / T;
  const int i0 = min(tid * per, nk), i1 = min(i0 + per, nk);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    gt += k > threshold;
    eq += k == threshold;
  }
  int sg = gt, se = eq;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, sg, m), b = __shfl_up_sync(0xffffffffu, se, m);
    if (lane >= m) sg += a, se += b;
  }
  if (lane == 31) warp_gt[warp] = sg, warp_eq[warp] = se;
  __syncthreads();
  sg -= gt, se -= eq;
  int total_gt = 0;
  for (int w = 0; w < T / 32; ++w) {
    if (w < warp) sg += warp_gt[w], se += warp_eq[w];
    total_gt += warp_gt[w];
  }
  launch_next();
  const int n = total_gt + equal;
  int at = sg + min(se, equal);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    if (k > threshold || (k == threshold && se++ < equal)) out[at++] = i;
  }
  for (int i = n + tid; i < most; i += T) out[i] = -1;
  if (tid == 0) counts[row] = n;
}

}  // namespace

size_t block_scores_workspace_bytes(int nq, int nk, int H, int Hkv) {
  const size_t means = static_cast<size_t>(nq) * H + static_cast<size_t>(nk) * Hkv;
  return means * DHB * sizeof(float) * (nq > FEW ? 2 : 1);
}

h3_status launch_block_scores(const void* q, int64_t ld_q, const void* k, int64_t ld_k,
                              float* scores, int Lq, int Lk, int H, int Hkv, int k_block,
                              float scale, void* workspace, cudaStream_t s) {
  const int nq = (Lq + H3_QUERY_BLOCK - 1) / H3_QUERY_BLOCK, nk = (Lk + k_block - 1) / k_block;
  const bool few = nq <= FEW;
  const int64_t q_rows = static_cast<int64_t>(nq) * H, k_rows = static_cast<int64_t>(nk) * Hkv;
  float* mq = static_cast<float*>(workspace);
  float* mk = mq + q_rows * DHB;
  float* lq = few ? nullptr : mk + k_rows * DHB;
  float* lk = few ? nullptr : lq + q_rows * DHB;
  const PoolSide qs{Lq, H, H3_QUERY_BLOCK, nq, (H + 1) / 2, nq * ((H + 1) / 2), mq, lq};
  const PoolSide ks{Lk, Hkv, k_block, nk, (Hkv + 1) / 2, nk * ((Hkv + 1) / 2), mk, lk};
  static std::atomic<bool> done_pool[64];
  h3_status st = set_smem_limit(done_pool, pool_kernel, POOL_SMEM_BYTES,
                                "block pooling: set shared memory size");
  if (st != H3_OK) return st;
  DevErr err;
  if ((st = dev_err(&err)) != H3_OK) return st;
  CUtensorMap tq, tk;
  if ((st = make_tmap_bf16_2d(&tq, q, static_cast<uint64_t>(H) * DHB, Lq, ld_q * 2, 64,
                              std::min(H3_QUERY_BLOCK, POOL_ROWS))) != H3_OK)
    return st;
  if ((st = make_tmap_bf16_2d(&tk, k, static_cast<uint64_t>(Hkv) * DHB, Lk, ld_k * 2, 64,
                              std::min(k_block, POOL_ROWS))) != H3_OK)
    return st;
  st = cuda_fail(launch_overlapped(pool_kernel, dim3(std::min(qs.items + ks.items, num_sms())),
                                   POOL_THREADS, POOL_SMEM_BYTES, 1, s, tq, tk, qs, ks, err),
                 "block pooling launch");
  if (st != H3_OK) return st;
  if (few) {
    const dim3 grid((nk + FEW_WARPS * FEW_KEYS - 1) / (FEW_WARPS * FEW_KEYS), H);
    return cuda_fail(launch_overlapped(block_scores_few_kernel, grid, FEW_WARPS * 32, 0, 1, s, mq, mk,
                                       scores, nq, nk, H / Hkv, scale),
                     "block scores launch");
  }
  static std::atomic<bool> done[64];
  st = set_smem_limit(done, block_scores_kernel, TC_SMEM_BYTES, "block scores: set shared memory size");
  if (st != H3_OK) return st;
  CUtensorMap t[4];
  const float* parts[4] = {mq, lq, mk, lk};
  for (int i = 0; i < 4; ++i)
    if ((st = make_tmap_f32_2d(&t[i], parts[i], DHB, i < 2 ? q_rows : k_rows, DHB * 4, 32, TC_TILE)) !=
        H3_OK)
      return st;
  ScoreSizes z{mq, lq, mk, lk, nq, nk, H / Hkv, (nk + TC_TILE - 1) / TC_TILE, (nq + TC_TILE - 1) / TC_TILE, 0};
  z.tiles = z.across * z.down * H;
  return cuda_fail(launch_overlapped(block_scores_kernel, dim3(std::min(z.tiles, num_sms())), TC_THREADS,
                                     TC_SMEM_BYTES, 1, s, t[0], t[1], t[2], t[3], scores, z, scale, err),
                   "block scores launch");
}

h3_status launch_block_select(const float* scores, int32_t* ids, int32_t* counts, int rows,
                              int nk, int max_blocks, int keep_first, int keep_last,
                              cudaStream_t s) {
  cudaError_t e;
  if (nk <= 1024) {
    // z: where a normal distribution has max_blocks / nk of it above (Abramowitz and Stegun,
    // Handbook of Mathematical Functions, 26.2.23: off by less than 4.5e-4), and its density there
    const double share = std::min(0.999, std::max(1e-6, static_cast<double>(max_blocks) / nk));
    const double p = std::min(share, 1.0 - share);
    const double t = std::sqrt(-2.0 * std::log(p));
    double z = t - (2.515517 + t * (0.802853 + t * 0.010328)) /
                       (1.0 + t * (1.432788 + t * (0.189269 + t * 0.001308)));
    const double density = 0.3989422804014327 * std::exp(-0.5 * z * z);
    if (share > 0.5) z = -z;
    const int grid = (rows - 1) / SEL_WARPS + 1;
    const float zf = static_cast<float>(z), df = static_cast<float>(std::max(density, 1e-4));
    auto kernel = nk <= 128    ? block_select_warp_kernel<4>
                  : nk <= 256  ? block_select_warp_kernel<8>
                  : nk <= 512  ? block_select_warp_kernel<16>
                  : nk <= 768  ? block_select_warp_kernel<24>
                               : block_select_warp_kernel<32>;
    e = launch_overlapped(kernel, dim3(grid), SEL_WARPS * 32, 0, 1, s, scores, ids, counts, rows, nk,
                          max_blocks, keep_first, keep_last, zf, df);
  } else {
    e = launch_overlapped(block_select_kernel<512>, dim3(rows), 512, 0, 1, s, scores, ids, counts, nk,
                          max_blocks, keep_first, keep_last);
  }
  return cuda_fail(e, "block select launch");
}

}  // namespace h3
