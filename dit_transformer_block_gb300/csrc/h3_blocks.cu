// Choosing key blocks for block-sparse attention: scores of pooled blocks, and the
// selection of the best of every query block.
//
// Scores: the mean row of every query block and key block (FP32), then one product of
// the means per head. The pooling reads q and k once and is bound by HBM; the product
// has 1 / block of the attention's own Q K^T to do, in FP32 on the CUDA cores, since a
// score that is rounded to fewer bits changes which blocks are chosen.
//
// Selection: the max_blocks-th largest score is found by counting, then one pass writes
// the chosen indices in ascending order. A warp per row of scores, longer ones a CTA.
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
constexpr int POOL_WARPS = 8;

struct PoolSide {
  const __nv_bfloat16* x;
  int64_t ld;
  int L, heads, block, blocks;
  int pairs;   // pairs of heads
  float* out;  // [heads][blocks][128]
};

// A CTA takes a block of rows and two neighbouring heads: a warp reads 512 contiguous
// bytes of a row, its rows POOL_WARPS apart, and the warps' sums meet in shared memory.
__global__ void __launch_bounds__(POOL_WARPS * 32)
    pool_kernel(const PoolSide q, const PoolSide k, const int q_ctas) {
  __shared__ float part[POOL_WARPS][2 * DHB];
  const bool is_q = static_cast<int>(blockIdx.x) < q_ctas;
  const PoolSide& s = is_q ? q : k;
  const int id = static_cast<int>(blockIdx.x) - (is_q ? 0 : q_ctas);
  const int blk = id / s.pairs, head0 = id % s.pairs * 2;
  wait_previous();
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int row0 = blk * s.block;
  const int rows = min(s.block, s.L - row0);
  const bool real = head0 + (lane >> 4) < s.heads;
  float acc[8] = {};
  if (real) {
    const __nv_bfloat16* p = s.x + static_cast<int64_t>(row0 + warp) * s.ld + head0 * DHB + lane * 8;
    const int64_t step = POOL_WARPS * s.ld;
    int r = warp;
    auto add = [&](const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[2 * j] += bf16_lo(w[j]);
        acc[2 * j + 1] += bf16_hi(w[j]);
      }
    };
    constexpr int U = 8;  // rows in flight
    for (; r + (U - 1) * POOL_WARPS < rows; r += U * POOL_WARPS, p += U * step) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const uint4*>(p + u * step);
#pragma unroll
      for (int u = 0; u < U; ++u) add(v[u]);
    }
    for (; r < rows; r += POOL_WARPS, p += step) add(*reinterpret_cast<const uint4*>(p));
  }
  launch_next();
  float4* mine = reinterpret_cast<float4*>(&part[warp][lane * 8]);
  mine[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  mine[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  __syncthreads();
  const int head = head0 + (threadIdx.x >> 7);
  if (head < s.heads) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < POOL_WARPS; ++w) t += part[w][threadIdx.x];
    s.out[(static_cast<int64_t>(head) * s.blocks + blk) * DHB + (threadIdx.x & 127)] =
        t / static_cast<float>(rows);
  }
}

// ------------------------------------------------------------------ product
constexpr int SC_N = 128;    // key blocks of a CTA
constexpr int SC_K = 32;     // channels per step
constexpr int SC_THREADS = 128;

// (d0, d1) += (a, a) * (b0, b1)
__device__ __forceinline__ void ffma2_acc(uint64_t& d, float a, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %1};\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "fma.rn.f32x2 %0, x, y, %0;\n\t}"
      : "+l"(d)
      : "f"(a), "f"(b0), "f"(b1));
}

// scores[h] = scale * mq[h] mk[g]^T: TMQ x 128 of it per CTA. A thread has TMQ / 8 neighbouring
// query blocks and eight key blocks 16 apart, two to a packed FMA; both operands lie
// channel by channel in shared memory, 32 channels at a time, the next ones on their way.
template <int TMQ>
__global__ void __launch_bounds__(SC_THREADS)
    block_scores_kernel(const float* mq, const float* mk,
                        float* scores, int nq, int nk, int group, float scale) {
  constexpr int RQ = TMQ / 8;              // rows of a thread
  constexpr int AV = TMQ * SC_K / 4 / SC_THREADS;  // float4 that a thread loads of A
  constexpr int BV = SC_N * SC_K / 4 / SC_THREADS;
  __shared__ __align__(16) float sa[SC_K][TMQ + 4];
  __shared__ __align__(16) float sb[SC_K][SC_N + 4];
  const int h = blockIdx.z, g = h / group;
  const int t0 = blockIdx.y * TMQ, b0 = blockIdx.x * SC_N;
  const float4* qa = reinterpret_cast<const float4*>(mq + (static_cast<int64_t>(h) * nq + t0) * DHB);
  const float4* kb = reinterpret_cast<const float4*>(mk + (static_cast<int64_t>(g) * nk + b0) * DHB);
  wait_previous();
  const int tid = threadIdx.x;
  // A: thread's row tid % TMQ, its AV float4 from (tid / TMQ) * AV on; B: row tid, all of them
  const int ar = tid % TMQ, ac = tid / TMQ * AV;
  const bool a_in = t0 + ar < nq, b_in = b0 + tid < nk;
  float4 av[AV], bv[BV];
  auto fetch = [&](int k4) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < AV; ++i) av[i] = a_in ? qa[ar * (DHB / 4) + k4 + ac + i] : z;
#pragma unroll
    for (int i = 0; i < BV; ++i) bv[i] = b_in ? kb[tid * (DHB / 4) + k4 + i] : z;
  };
  uint64_t acc[RQ][4];
#pragma unroll
  for (int i = 0; i < RQ; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
  const int ty = tid >> 4, tx = tid & 15;
  fetch(0);
#pragma unroll 1
  for (int k0 = 0; k0 < DHB; k0 += SC_K) {
    if (k0 > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < AV; ++i) {
      const float w[4] = {av[i].x, av[i].y, av[i].z, av[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) sa[4 * (ac + i) + c][ar] = w[c] * scale;
    }
#pragma unroll
    for (int i = 0; i < BV; ++i) {
      const float w[4] = {bv[i].x, bv[i].y, bv[i].z, bv[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) sb[4 * i + c][tid] = w[c];
    }
    __syncthreads();
    if (k0 + SC_K < DHB) fetch((k0 + SC_K) / 4);
#pragma unroll 8
    for (int c = 0; c < SC_K; ++c) {
      float x[RQ], y[8];
#pragma unroll
      for (int i = 0; i < RQ; ++i) x[i] = sa[c][ty * RQ + i];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = sb[c][tx + 16 * j];
#pragma unroll
      for (int i = 0; i < RQ; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) ffma2_acc(acc[i][j], x[i], y[2 * j], y[2 * j + 1]);
    }
  }
  launch_next();
#pragma unroll
  for (int i = 0; i < RQ; ++i) {
    const int t = t0 + ty * RQ + i;
    if (t >= nq) break;
    float* o = scores + (static_cast<int64_t>(h) * nq + t) * nk + b0 + tx;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = static_cast<uint32_t>(acc[i][j >> 1] >> (32 * (j & 1)));
      if (b0 + tx + 16 * j < nk) o[16 * j] = __uint_as_float(w);
    }
  }
}

// ---------------------------------------------------------------- selection
// Scores as integers of the same order: 0 for what is never selected (-inf, NaN), the
// largest for the blocks that always are; -0 and +0 are the same.
__device__ __forceinline__ uint32_t select_key(float f, bool kept) {
  if (kept) return 0xffffffffu;
  if (!(f > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr uint32_t KEPT = 0xffffffffu;
constexpr int SEL_WARPS = 4;

// Rows of at most 32 * IPT scores: a warp per row, whose keys stay in its registers. The
// threshold T (the least selected key) is looked for between lo and hi, of which at least
// and fewer than `most` keys are not below; every step counts the keys from a place between them
// on. The first place is where a normal distribution of the row's mean and deviation has
// `most` (z deviations above the mean), the second as far from it as that density says, a
// dozen keys further, and from then on the middle: rows as scores are take two or three
// steps, any others at most 32 more. With at most 32 keys left between lo and hi, a lane
// takes one and ranks it among them.
template <int IPT>
__global__ void __launch_bounds__(SEL_WARPS * 32)
    block_select_warp_kernel(const float* scores, int32_t* ids,
                             int32_t* counts, int rows, int nk, int most, int first,
                             int last, float z, float density) {
  __shared__ uint32_t left[SEL_WARPS][32];
  wait_previous();
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x * SEL_WARPS + warp;
  if (row >= rows) return;
  const float* s = scores + static_cast<int64_t>(row) * nk;
  int32_t* out = ids + static_cast<int64_t>(row) * most;
  uint32_t key[IPT];
  float sum = 0.f, sum2 = 0.f;
  int valid = 0, kept = 0;
  {
    float f[IPT];
#pragma unroll
    for (int r = 0; r < IPT; ++r) {
      const int i = r * 32 + lane;
      f[r] = i < nk ? __ldcs(s + i) : -INFINITY;
    }
#pragma unroll
    for (int r = 0; r < IPT; ++r) {
      const int i = r * 32 + lane;
      key[r] = select_key(f[r], i < nk && (i < first || i >= nk - last));
      valid += key[r] != 0u;
      kept += key[r] == KEPT;
      const float v = key[r] != 0u && key[r] != KEPT ? f[r] : 0.f;
      sum += v;
      sum2 = fmaf(v, v, sum2);
    }
  }
  valid = __reduce_add_sync(0xffffffffu, valid);
  kept = __reduce_add_sync(0xffffffffu, kept);
  // T, and how many of the keys equal to it are selected (the first of them)
  uint32_t T = 0;
  int equal = 0;
  if (kept >= most) {
    T = KEPT - 1u;
  } else if (valid > most) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, m);
      sum2 += __shfl_xor_sync(0xffffffffu, sum2, m);
    }
    const float n = static_cast<float>(valid - kept);
    const float mean = sum / n;
    const float dev = sqrtf(fmaxf(sum2 / n - mean * mean, 0.f));
    uint32_t lo = 1u, hi = KEPT;
    int c_lo = valid, c_hi = kept;  // keys from lo, from hi on
    float at = fmaf(z, dev, mean);
    for (int step = 0;; ++step) {
      uint32_t place = lo + (hi - lo) / 2;
      if (step < 2 && at > -INFINITY && at < INFINITY) {
        const uint32_t k = select_key(at, false);
        if (k > lo && k < hi) place = k;
      }
      int c = 0;
#pragma unroll
      for (int r = 0; r < IPT; ++r) c += key[r] >= place;
      c = __reduce_add_sync(0xffffffffu, c);
      if (c >= most) {
        lo = place, c_lo = c;
        if (c == most) break;
        at += (c - most + 12) * dev / (n * density);
      } else {
        hi = place, c_hi = c;
        at -= (most - c + 12) * dev / (n * density);
      }
      if (c_lo - c_hi <= 32 || hi - lo == 1u) break;
    }
    const int need = most - c_hi;
    if (c_lo == most) {
      T = lo - 1u;  // all from lo on
    } else if (hi - lo == 1u) {
      T = lo;
      equal = need;
    } else {
      int base = 0;
#pragma unroll
      for (int r = 0; r < IPT; ++r) {
        const bool in = key[r] >= lo && key[r] < hi;
        const uint32_t b = __ballot_sync(0xffffffffu, in);
        if (in) left[warp][base + __popc(b & ((1u << lane) - 1u))] = key[r];
        base += __popc(b);
      }
      __syncwarp();
      const uint32_t mine = lane < base ? left[warp][lane] : 0u;
      int above = 0, rank = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, j);
        above += other > mine;
        rank += other > mine || (other == mine && j < lane);
      }
      const uint32_t b = __ballot_sync(0xffffffffu, rank == need - 1 && lane < base);
      const int who = __ffs(b) - 1;
      T = __shfl_sync(0xffffffffu, mine, who);
      equal = need - __shfl_sync(0xffffffffu, above, who);
    }
  }
  launch_next();
  const uint32_t below = (1u << lane) - 1u;
  int n = 0, eq = 0;
#pragma unroll
  for (int r = 0; r < IPT; ++r) {
    const uint32_t same = __ballot_sync(0xffffffffu, key[r] == T && T != 0u);
    const bool in = key[r] > T || (key[r] == T && T != 0u && eq + __popc(same & below) < equal);
    const uint32_t b = __ballot_sync(0xffffffffu, in);
    if (in) out[n + __popc(b & below)] = r * 32 + lane;
    n += __popc(b);
    eq += __popc(same);
  }
  for (int i = n + lane; i < most; i += 32) out[i] = -1;
  if (lane == 0) counts[row] = n;
}

// Longer rows: a CTA per row, a radix search of 8 bits a pass over the scores in L1 and L2.
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
  auto key = [&](int i) { return select_key(*(s + i), i < first || i >= nk - last); };

  // threshold: what is above it is selected, and of what is equal to it the first `equal`
  uint32_t prefix = 0, mask = 0, threshold = 0;
  int need = most, equal = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += T) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < nk; i += T) {
      const uint32_t k = key(i);
      if (k != 0u && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
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
    if (found[0] < 0) break;  // threshold 0
    prefix |= static_cast<uint32_t>(found[0]) << shift;
    mask |= 255u << shift;
    need = found[1];
    if (need == found[2]) {  // all of the bin
      threshold = prefix != 0u ? prefix - 1u : 0u;
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
  return (static_cast<size_t>(nq) * H + static_cast<size_t>(nk) * Hkv) * DHB * sizeof(float);
}

h3_status launch_block_scores(const void* q, int64_t ld_q, const void* k, int64_t ld_k,
                              float* scores, int Lq, int Lk, int H, int Hkv, int k_block,
                              float scale, void* workspace, cudaStream_t s) {
  const int nq = (Lq + H3_QUERY_BLOCK - 1) / H3_QUERY_BLOCK, nk = (Lk + k_block - 1) / k_block;
  float* mq = static_cast<float*>(workspace);
  float* mk = mq + static_cast<int64_t>(nq) * H * DHB;
  const PoolSide qs{static_cast<const __nv_bfloat16*>(q), ld_q, Lq, H, H3_QUERY_BLOCK, nq,
                    (H + 1) / 2, mq};
  const PoolSide ks{static_cast<const __nv_bfloat16*>(k), ld_k, Lk, Hkv, k_block, nk,
                    (Hkv + 1) / 2, mk};
  const int q_ctas = nq * qs.pairs;
  h3_status st = cuda_fail(launch_overlapped(pool_kernel, dim3(q_ctas + nk * ks.pairs),
                                             POOL_WARPS * 32, 0, 1, s, qs, ks, q_ctas),
                           "block pooling launch");
  if (st != H3_OK) return st;
  const int tile = nq <= 16 ? 16 : 64;
  const dim3 grid((nk + SC_N - 1) / SC_N, (nq + tile - 1) / tile, H);
  return cuda_fail(launch_overlapped(tile == 16 ? block_scores_kernel<16> : block_scores_kernel<64>,
                                     grid, SC_THREADS, 0, 1, s, mq, mk, scores, nq, nk, H / Hkv,
                                     scale),
                   "block scores launch");
}

h3_status launch_block_select(const float* scores, int32_t* ids, int32_t* counts, int rows,
                              int nk, int max_blocks, int keep_first, int keep_last,
                              cudaStream_t s) {
  cudaError_t e;
  if (nk <= 2048) {
    // z: where a normal distribution has max_blocks / nk of it above (Abramowitz and Stegun,
    // Handbook of Mathematical Functions, 26.2.23: off by less than 4.5e-4), and its density there
    const double share = std::min(0.999, std::max(1e-6, static_cast<double>(max_blocks) / nk));
    const double p = std::min(share, 1.0 - share);
    const double t = std::sqrt(-2.0 * std::log(p));
    double z = t - (2.515517 + t * (0.802853 + t * 0.010328)) /
                       (1.0 + t * (1.432788 + t * (0.189269 + t * 0.001308)));
    const double density = 0.3989422804014327 * std::exp(-0.5 * z * z);
    if (share > 0.5) z = -z;
    const int grid = (rows + SEL_WARPS - 1) / SEL_WARPS;
    const float zf = static_cast<float>(z), df = static_cast<float>(std::max(density, 1e-4));
    auto kernel = nk <= 128    ? block_select_warp_kernel<4>
                  : nk <= 256  ? block_select_warp_kernel<8>
                  : nk <= 512  ? block_select_warp_kernel<16>
                  : nk <= 768  ? block_select_warp_kernel<24>
                  : nk <= 1024 ? block_select_warp_kernel<32>
                               : block_select_warp_kernel<64>;
    e = launch_overlapped(kernel, dim3(grid), SEL_WARPS * 32, 0, 1, s, scores, ids, counts, rows, nk,
                          max_blocks, keep_first, keep_last, zf, df);
  } else {
    e = launch_overlapped(block_select_kernel<512>, dim3(rows), 512, 0, 1, s, scores, ids, counts, nk,
                          max_blocks, keep_first, keep_last);
  }
  return cuda_fail(e, "block select launch");
}

}  // namespace h3
