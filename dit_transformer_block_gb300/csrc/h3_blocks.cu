// Choosing key blocks for block-sparse attention: scores of pooled blocks, and the
// selection of the best of every query block.
//
// Scores: the mean row of every query block and key block (FP32), then one product of
// the means per head. The pooling reads q and k once and is bound by HBM; the product
// has 1 / block of the attention's own Q K^T to do, in FP32 on the CUDA cores, since a
// score that is rounded to fewer bits changes which blocks are chosen.
//
// Selection: a radix search for the max_blocks-th largest score (8 bits a pass), then one
// pass that writes the chosen indices in ascending order. A CTA per row of scores.
#include <cuda_bf16.h>

#include <algorithm>

#include "h3_blocks.cuh"
#include "h3_internal.cuh"

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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
      for (int u = 0; u < U; ++u) v[u] = __ldg(reinterpret_cast<const uint4*>(p + u * step));
#pragma unroll
      for (int u = 0; u < U; ++u) add(v[u]);
    }
    for (; r < rows; r += POOL_WARPS, p += step) add(__ldg(reinterpret_cast<const uint4*>(p)));
  }
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
constexpr int SC_T = 64;     // query blocks x key blocks of a CTA
constexpr int SC_LD = 68;    // floats between two channels' rows of a tile
constexpr size_t SC_SMEM = 2 * DHB * SC_LD * sizeof(float);

// scores[h] = scale * mq[h] mk[g]^T: 64 x 64 of it per CTA, 8 x 4 per thread, both
// tiles whole (128 channels) in shared memory, channel by channel.
__global__ void __launch_bounds__(128)
    block_scores_kernel(const float* __restrict__ mq, const float* __restrict__ mk,
                        float* __restrict__ scores, int nq, int nk, int group, float scale) {
  extern __shared__ float sm[];
  float* sa = sm;
  float* sb = sm + DHB * SC_LD;
  const int h = blockIdx.z, g = h / group;
  const int t0 = blockIdx.y * SC_T, b0 = blockIdx.x * SC_T;
  const float* qa = mq + static_cast<int64_t>(h) * nq * DHB;
  const float* kb = mk + static_cast<int64_t>(g) * nk * DHB;
  {
    const int row = threadIdx.x & 63, half = threadIdx.x >> 6;
    const bool qok = t0 + row < nq, kok = b0 + row < nk;
    const float4* qp = reinterpret_cast<const float4*>(qa + static_cast<int64_t>(t0 + row) * DHB);
    const float4* kp = reinterpret_cast<const float4*>(kb + static_cast<int64_t>(b0 + row) * DHB);
#pragma unroll 8
    for (int i = 0; i < 16; ++i) {
      const int c = half * 16 + i;
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 u = qok ? __ldg(qp + c) : z;
      const float4 w = kok ? __ldg(kp + c) : z;
      float* pa = sa + 4 * c * SC_LD + row;
      float* pb = sb + 4 * c * SC_LD + row;
      pa[0] = u.x * scale, pa[SC_LD] = u.y * scale;
      pa[2 * SC_LD] = u.z * scale, pa[3 * SC_LD] = u.w * scale;
      pb[0] = w.x, pb[SC_LD] = w.y, pb[2 * SC_LD] = w.z, pb[3 * SC_LD] = w.w;
    }
  }
  __syncthreads();
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  float acc[8][4] = {};
#pragma unroll 4
  for (int c = 0; c < DHB; ++c) {
    const float4 a0 = *reinterpret_cast<const float4*>(sa + c * SC_LD + ty * 8);
    const float4 a1 = *reinterpret_cast<const float4*>(sa + c * SC_LD + ty * 8 + 4);
    const float4 b = *reinterpret_cast<const float4*>(sb + c * SC_LD + tx * 4);
    const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = t0 + ty * 8 + i;
    if (t >= nq) break;
    float* o = scores + (static_cast<int64_t>(h) * nq + t) * nk + b0 + tx * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (b0 + tx * 4 + j < nk) o[j] = acc[i][j];
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

template <int T>
__global__ void __launch_bounds__(T)
    block_select_kernel(const float* __restrict__ scores, int32_t* __restrict__ ids,
                        int32_t* __restrict__ counts, int nk, int most, int first, int last) {
  __shared__ int hist[256];
  __shared__ int found[3];       // bin, still needed in it, how many it holds
  __shared__ int warp_gt[T / 32], warp_eq[T / 32];
  const int64_t row = blockIdx.x;
  const float* s = scores + row * nk;
  int32_t* out = ids + row * most;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto key = [&](int i) { return select_key(__ldg(s + i), i < first || i >= nk - last); };

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
  static std::atomic<bool> done[64];
  h3_status st = set_smem_limit(done, block_scores_kernel, SC_SMEM,
                                "block scores: set shared memory size");
  if (st != H3_OK) return st;
  const int nq = (Lq + H3_QUERY_BLOCK - 1) / H3_QUERY_BLOCK, nk = (Lk + k_block - 1) / k_block;
  float* mq = static_cast<float*>(workspace);
  float* mk = mq + static_cast<int64_t>(nq) * H * DHB;
  const PoolSide qs{static_cast<const __nv_bfloat16*>(q), ld_q, Lq, H, H3_QUERY_BLOCK, nq,
                    (H + 1) / 2, mq};
  const PoolSide ks{static_cast<const __nv_bfloat16*>(k), ld_k, Lk, Hkv, k_block, nk,
                    (Hkv + 1) / 2, mk};
  const int q_ctas = nq * qs.pairs;
  pool_kernel<<<q_ctas + nk * ks.pairs, POOL_WARPS * 32, 0, s>>>(qs, ks, q_ctas);
  if ((st = cuda_fail(cudaGetLastError(), "block pooling launch")) != H3_OK) return st;
  const dim3 grid((nk + SC_T - 1) / SC_T, (nq + SC_T - 1) / SC_T, H);
  block_scores_kernel<<<grid, 128, SC_SMEM, s>>>(mq, mk, scores, nq, nk, H / Hkv, scale);
  return cuda_fail(cudaGetLastError(), "block scores launch");
}

h3_status launch_block_select(const float* scores, int32_t* ids, int32_t* counts, int rows,
                              int nk, int max_blocks, int keep_first, int keep_last,
                              cudaStream_t s) {
  if (nk <= 2048)
    block_select_kernel<128><<<rows, 128, 0, s>>>(scores, ids, counts, nk, max_blocks, keep_first,
                                                  keep_last);
  else
    block_select_kernel<512><<<rows, 512, 0, s>>>(scores, ids, counts, nk, max_blocks, keep_first,
                                                  keep_last);
  return cuda_fail(cudaGetLastError(), "block select launch");
}

}  // namespace h3
