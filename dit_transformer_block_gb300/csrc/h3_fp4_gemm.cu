// Block-scaled 4-bit GEMM on CTA pairs: C[:L] = epilogue(A[:L] B^T), E2M1 operands whose
// scales the tensor cores apply (tcgen05 kind::mxf4 / kind::mxf4nvf4, cta_group::2), FP32
// accumulation in tensor memory, bf16 output.
//
// A pair takes 256 x 256 of the output: a CTA holds 128 rows of A and of B (half of the
// columns) in shared memory and 128 x 256 of the accumulator in tensor memory. One
// CTA's tile of 128 x 256 would read 12 KB of shared memory per instruction and
// 128 cycles, three quarters of what it can; as a pair it is 8 KB.
//   * stage: 256 values of K (128 bytes per row, 128-byte swizzle) of both operands and
//     their scales, which lie in memory as the tensor cores want them (tiles of 128 rows x
//     4 scales, 512 bytes);
//   * warp 0 of each CTA: TMA producer (one lane), counted on the even CTA's barriers; of the
//     even CTA, warp 1 issues four products of K = 64 per stage, and two warps the copies of
//     a stage's scales from shared to tensor memory (both CTAs' at once) in turn: twelve (NV)
//     or six (MX) copies take longer to issue than the products to run;
//   * warps 2-9: epilogue, two per lane quarter. A warp reads its 128 columns of the accumulator
//     at once, so that the next tile's products wait for one read and not for the stores, then
//     writes bf16 through 4 KB of shared memory of its own with TMA. The CTA's sixteen stores of
//     a tile spread over the next tile's products (seven cycles apart for every 64 values of K,
//     whose product takes 128, or less in SwiGLU): in one go they hold up the loads, and the
//     products wait (2,432 tiles of K = 5,120: 239 us instead of 247 in MX, 251 and 257 in NV, of
//     K = 2,560 138 and 147, 144 and 155; 220 and 228 of K = 5,120 if nothing were stored);
//   * tensor memory: 256 columns of accumulator, a buffer of scales per stage.
// A CTA gets its operands at a rate that its copies in flight allow, so where there are few tiles
// (few rows: the weights' bytes count) several pairs in a cluster share one tile's K. They put
// their sums into shared memory and each adds up a share of the rows, in the order of K (22 x
// 5,376 x 5,376 with weights in HBM: 10.7 us with the quantisation; the product alone 8.7, 7.8 with
// its weights in L2, where HBM would take 2.3 for their 15 MB. What the rest of it is has not been
// found: a pair's seven stages are two rounds of loads).
// 58,758 x 16,128 x 5,376: MX 1,436 us (7,100 TFLOP/s), NV 1,515 us (6,730). Products of K = 64 and
// nothing else run at 9,220 TFLOP/s. With the loads beside them a stage takes 600 cycles instead
// of 512 with five stages (686 with four, 857 with three, 605 with six), nearly the same where half
// of B's loads, the scales' loads or their copies are left out; the stores add what is said above.
#include <cuda_bf16.h>

#include <algorithm>

#include "h3_fp4.cuh"
#include "h3_internal.cuh"
#include "h3_launch.cuh"

namespace h3 {
namespace {

constexpr int ROWS = 128;                    // rows of A, and of B, per CTA
constexpr int BN4 = 256;                     // output columns of a pair
constexpr int STAGE_CODES = 256;             // values of K per stage
constexpr int OP_BYTES = ROWS * STAGE_CODES / 2;  // 16 KB
constexpr int SFA_BYTES = 2048, SFB_BYTES = 2 * 2048;
constexpr int STAGE4_BYTES = 2 * OP_BYTES + SFA_BYTES + SFB_BYTES;
constexpr int STAGES4 = 5;
constexpr int EPI_WARPS = 8, COPY_WARPS = 2;
static_assert(COPY_WARPS <= STAGES4, "a copy warp's next stage is at most one round of slots on");
constexpr int THREADS4 = (2 + EPI_WARPS + COPY_WARPS) * 32;
constexpr int GROUP_M4 = 16;                 // raster: 16 x 256 rows per sweep of the columns
constexpr int OUT_BYTES = 32 * 128;          // a warp's 32 rows x 64 columns of output
constexpr int SCALE_BYTES = 3 * BN4 * 4;          // scales of a tile's columns (NV), three tiles
constexpr size_t SMEM4_BYTES = 1024 + STAGES4 * STAGE4_BYTES + EPI_WARPS * OUT_BYTES + 256 + SCALE_BYTES;
static_assert(SMEM4_BYTES <= 227 * 1024, "fp4 gemm shared memory");

// Tensor memory: the accumulator, then a buffer of scales per stage: A's, from SFB on B's.
template <bool NV>
struct Tmem4 {
  static constexpr uint32_t SFB = NV ? 16 : 8, SF_COLS = 3 * SFB, SF = BN4;
  static_assert(SF + STAGES4 * SF_COLS <= 512, "tensor memory");
};

enum Bar4 {
  B4_FULL = 0,                    // stage landed in both CTAs (even CTA)
  B4_EMPTY = B4_FULL + STAGES4,   // stage read by the products
  B4_SF = B4_EMPTY + STAGES4,     // stage's scales in tensor memory (even CTA)
  B4_TFULL = B4_SF + STAGES4,     // accumulator written
  B4_TEMPTY = B4_TFULL + 1,       // accumulator read (16 warps, even CTA)
  B4_DRAIN = B4_TEMPTY + 1,       // [1 + COPY_WARPS]
  B4_NUM = B4_DRAIN + 1 + COPY_WARPS
};
static_assert(B4_NUM * 8 + 8 <= 256, "barrier region");

// Instruction descriptor of the 4-bit kinds with E2M1 operands and an f32 accumulator:
// [4,6) scale id of B, [7,10) and [10,12) operand formats (1 = E2M1), [17,23) N >> 3, bit
// 23 scale format (0 = E4M3, 1 = E8M0), [24,29) M >> 4, [29,31) scale id of A, bit 31 0
// for K = 64. A scale id is the byte of its 32-bit column where a product's scales begin.
__host__ __device__ constexpr uint32_t idesc_e2m1(int M, int N, bool e8m0, uint32_t scale_id) {
  return (scale_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         ((e8m0 ? 1u : 0u) << 23) | (static_cast<uint32_t>(M >> 4) << 24) | (scale_id << 29);
}

// Descriptor of 32 rows x 16 contiguous bytes without swizzle (8-row groups 128 bytes
// apart): the source of a scale copy.
__device__ __forceinline__ uint64_t sdesc_rows16(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46);
}
// 512 bytes of scales (32 rows of 16 bytes) to 4 columns of tensor memory, the same in
// every lane quarter, in both CTAs from their own shared memory.
__device__ __forceinline__ void scale_copy_pair_el(uint32_t taddr, uint64_t desc) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(desc)
      : "memory");
}
template <bool NV>
__device__ __forceinline__ void mma_fp4_pair_el(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (NV)
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 2D tiled load into this CTA's shared memory, counted on a barrier of either CTA of the
// pair (its shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m,
                                                 uint32_t cluster_bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}

// 32 rows x 64 columns from shared memory (128-byte swizzle) to the output, clipped at its
// edges.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int32_t x,
                                             int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}
// 16 bytes of the shared memory of any CTA of the cluster.
__device__ __forceinline__ void ld_cluster_v4(float4& v, uint32_t addr) {
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// This thread's stores have read their shared memory / are done.
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void store_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

struct Gemm4Args {
  __nv_bfloat16* C;  // (SPLIT)
  const float* ra;  // row scales (NV)
  const float* rb;
  int M, N, K;
  int num_m, num_n, num_k;  // tiles of 256 rows, of columns, stages
  int num_tiles;
  int sf_tiles;             // scale tiles along K
  int parts;                // pairs that share a tile's K
  int up_rows;              // SwiGLU: first row of the up half of B
  int pace;                 // cycles from one of a CTA's sixteen stores of a tile to the next
  DevErr err;
};

__device__ __forceinline__ void tile_coords4(int tile, const Gemm4Args& a, int& mb, int& nb) {
  const int group_size = GROUP_M4 * a.num_n;
  const int group = tile / group_size;
  const int first_m = group * GROUP_M4;
  const int gm = min(a.num_m - first_m, GROUP_M4);
  const int r = tile - group * group_size;
  mb = first_m + r % gm;
  nb = r / gm;
}

// bf16 SiLU(g) * u of two gates and two ups, rounded to bf16 first: g / (1 + 2^(-g log2 e)), the
// exponential within 2^-22 + 2^-23 |g| of it (its argument is a rounded product) and the reciprocal
// within 2^-23, which is flushed to 0 from where the sum is above 2^126 (SiLU below 2^-119). (A tile's epilogue bounds products of few stages: 9,728 x 8,192 x
// 256 54 us in MX and 74 in NV; 85 and 104 with __expf and __fdividef, which look after subnormal
// operands, and each value rounded by itself; an IEEE division made a tile's epilogue 4 us
// longer.)
__device__ __forceinline__ uint32_t swiglu2(float g0, float g1, float u0, float u1) {
  const uint32_t g = pack_bf16x2(g0, g1), u = pack_bf16x2(u0, u1);
  auto silu = [](float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2_approx(-1.4426950408889634f * x)));
    return x * r;
  };
  return pack_bf16x2(silu(bf16_lo(g)) * bf16_lo(u), silu(bf16_hi(g)) * bf16_hi(u));
}
// (a0, a1) * (b0, b1)
__device__ __forceinline__ void fmul2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// SPLIT: the cluster's pairs share one tile; else a pair takes one tile after another.
template <bool NV, bool SWIGLU, bool SPLIT>
__global__ void __launch_bounds__(THREADS4, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmC, const Gemm4Args a) {
  using TM = Tmem4<NV>;
  constexpr int ATOM_STEPS = NV ? 1 : 2;  // products that a scale tile serves
  constexpr int ATOMS = 4 / ATOM_STEPS;   // scale tiles of a stage and 128 rows
  // bytes of a stage in one CTA
  constexpr uint32_t LOADED = 2 * OP_BYTES + 3 * ATOMS * 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sOut = smem + STAGES4 * STAGE4_BYTES;
  uint8_t* sScale = sOut + EPI_WARPS * OUT_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sScale + SCALE_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B4_NUM);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };

  const uint32_t crank = cluster_ctarank();
  const uint32_t rank = crank & 1u;         // in the pair
  const uint32_t even = crank & ~1u;        // the pair's even CTA
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int part = SPLIT ? static_cast<int>(crank >> 1) : 0;
  const int pair = SPLIT ? static_cast<int>(blockIdx.x) / (2 * a.parts) : blockIdx.x >> 1;
  const int pairs = SPLIT ? a.num_tiles : gridDim.x >> 1;
  // this pair's stages of K
  const int kb0 = SPLIT ? a.num_k * part / a.parts : 0;
  const int kb1 = SPLIT ? a.num_k * (part + 1) / a.parts : a.num_k;

  if (threadIdx.x == 0) {
    for (int i = 0; i < B4_NUM; ++i) {
      uint32_t count = 1;
      if (i == B4_TEMPTY) count = 2 * EPI_WARPS;
      mbar_init(bar(i), count);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_previous();

  // stages of this pair, over all of its tiles
  const int total = (a.num_tiles - pair + pairs - 1) / pairs * (kb1 - kb0);

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      int issued = 0, st = 0;
      uint32_t phase = 1;
      bool ok = true;
      const uint32_t full0 = mapa_shared(bar(B4_FULL), even);  // the even CTA's
      for (int tile = pair; tile < a.num_tiles && ok; tile += pairs) {
        int mb, nb;
        tile_coords4(tile, a, mb, nb);
        const int a_blk = 2 * mb + static_cast<int>(rank);
        // the pair's two blocks of 128 rows of B: neighbours, or gate and up
        const int b_blk0 = SWIGLU ? nb : 2 * nb;
        const int b_blk1 = SWIGLU ? a.up_rows / ROWS + nb : 2 * nb + 1;
        const int b_row = (leader ? b_blk0 : b_blk1) * ROWS;
        // (blocks past the operands' rows, and a row's scales past its end, which no product
        // uses, come from wherever they lie in the scales, or as zeros from past their end)
        const int k_tile = kb0 * ATOMS;
        int sa = a_blk * a.sf_tiles + k_tile;
        int sb0 = b_blk0 * a.sf_tiles + k_tile, sb1 = b_blk1 * a.sf_tiles + k_tile;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(bar(B4_EMPTY + st), phase, a.err, ERR_WAIT_GEMM_PRODUCER)) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + st * 8;
          const uint32_t dst = smem_u32(smem + st * STAGE4_BYTES);
          if (leader) mbar_arrive_expect_tx(bar(B4_FULL + st), 2 * LOADED);
          const int kx = kb * (STAGE_CODES / 2);
          tma_load_2d_pair(dst, &tmA, full, kx, a_blk * ROWS);
          tma_load_2d_pair(dst + OP_BYTES, &tmB, full, kx, b_row);
          tma_load_2d_pair(dst + 2 * OP_BYTES, &tmSA, full, 0, sa);
          tma_load_2d_pair(dst + 2 * OP_BYTES + SFA_BYTES, &tmSB, full, 0, sb0);
          tma_load_2d_pair(dst + 2 * OP_BYTES + SFA_BYTES + 2048, &tmSB, full, 0, sb1);
          sa += ATOMS, sb0 += ATOMS, sb1 += ATOMS;
          ++issued;
          if (++st == STAGES4) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
      launch_next();
      // No copy may still be landing when a CTA exits. The even CTA's barriers count those of
      // both, and neither leaves before the other; where a wait ran out they may never
      // complete, and the time of this wait is what the copies have to land.
      if (leader) {
        const uint64_t t0 = globaltimer_ns();
        for (int i = issued > STAGES4 ? issued - STAGES4 : 0; i < issued; ++i)
          mbar_wait_drain(bar(B4_FULL + i % STAGES4), static_cast<uint32_t>(i / STAGES4) & 1u, t0,
                          drain_limit_ns(a.err));
      } else if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    if (leader) {
      constexpr uint32_t idesc0 = idesc_e2m1(2 * ROWS, BN4, !NV, 0);
      constexpr uint32_t idesc2 = idesc_e2m1(2 * ROWS, BN4, !NV, 2);
      const uint16_t both = static_cast<uint16_t>(3u << even);
      const uint64_t da0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      auto wait = [&](uint32_t b, uint32_t parity) {
        return mbar_wait_warp(b, parity, a.err, ERR_WAIT_GEMM_MMA);
      };
      // stages with all of their four products, and the products of one behind them
      const int whole = a.K / STAGE_CODES + (a.K % STAGE_CODES > 192 ? 1 : 0);
      const int last = (a.K - whole * STAGE_CODES + 63) / 64;
      int st = 0;
      uint32_t phase = 0, acc_phase = 1;
      bool ok = true;
      for (int tile = pair; tile < a.num_tiles && ok; tile += pairs, acc_phase ^= 1u) {
        if (!wait(bar(B4_TEMPTY), acc_phase)) break;
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait(bar(B4_FULL) + st * 8, phase) || !wait(bar(B4_SF) + st * 8, phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = da0 + static_cast<uint32_t>(st * (STAGE4_BYTES >> 4));
          const uint64_t bd = ad + (OP_BYTES >> 4);
          const uint32_t sf = tmem + TM::SF + static_cast<uint32_t>(st) * TM::SF_COLS;
          auto product = [&](int k) {
            mma_fp4_pair_el<NV>(tmem, ad + k * 2, bd + k * 2, (!NV && (k & 1)) ? idesc2 : idesc0,
                                sf + (k / ATOM_STEPS) * 4, sf + TM::SFB + (k / ATOM_STEPS) * 8,
                                (kb > kb0 || k > 0) ? 1u : 0u);
          };
          // a whole stage without a branch between its products (with one before each the
          // pipe ran at 0.79 of this: 7,250 against 9,220 TFLOP/s without loads and stores)
          if (kb < whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) product(k);
          } else {
            product(0);
            if (last > 1) product(1);
            if (last > 2) product(2);
          }
          mma_commit_pair_mc_el(bar(B4_EMPTY) + st * 8, both);
          if (++st == STAGES4) {
            st = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair_mc_el(bar(B4_TFULL), both);
      }
      // every product must be done with both CTAs' memories before either frees them
      mma_commit_pair_mc_el(bar(B4_DRAIN), static_cast<uint16_t>(1u << even));
      mbar_wait_drain(bar(B4_DRAIN), 0u, globaltimer_ns(), drain_limit_ns(a.err));
    }
  } else if (warp >= 2 + EPI_WARPS) {
    // ------------------------------------------------------ scale copies
    // two warps, a stage each in turn: issuing a stage's copies takes longer than its products
    if (leader) {
      const int c = warp - 2 - EPI_WARPS;
      const uint64_t ds0 = sdesc_rows16(smem_u32(smem) + 2 * OP_BYTES);
      auto wait = [&](int b, uint32_t parity) {
        return mbar_wait_warp(bar(b), parity, a.err, ERR_WAIT_GEMM_MMA);
      };
      // (the stage was loaded again only after the products that read its buffer)
      for (int it = c, st = c, phase = 0; it < total; it += COPY_WARPS) {
        // The slot's stage before this one may be the other warp's, and its load the last to land:
        // while it has not, the barrier's parity is that of the phase this one waits for. So the slot's
        // copies before this one are waited for first: their barrier goes no further without this warp,
        // however long it is held (a wait for the other warp's loads could miss one).
        if (!wait(B4_SF + st, phase ^ 1) || !wait(B4_FULL + st, phase)) break;
        tc_fence_after();
        const uint64_t s = ds0 + static_cast<uint32_t>(st * (STAGE4_BYTES >> 4));
        const uint32_t sf = tmem + TM::SF + static_cast<uint32_t>(st) * TM::SF_COLS;
#pragma unroll
        for (int t = 0; t < ATOMS; ++t) {
          scale_copy_pair_el(sf + t * 4, s + t * (512 >> 4));
          scale_copy_pair_el(sf + TM::SFB + t * 8, s + ((SFA_BYTES + t * 512) >> 4));
          scale_copy_pair_el(sf + TM::SFB + t * 8 + 4, s + ((SFA_BYTES + 2048 + t * 512) >> 4));
        }
        mma_commit_pair_mc_el(bar(B4_SF + st), static_cast<uint16_t>(1u << even));
        st += COPY_WARPS;
        if (st >= STAGES4) {
          st -= STAGES4;
          phase ^= 1;
        }
      }
      mma_commit_pair_mc_el(bar(B4_DRAIN + 1 + c), static_cast<uint16_t>(1u << even));
      mbar_wait_drain(bar(B4_DRAIN + 1 + c), 0u, globaltimer_ns(), drain_limit_ns(a.err));
    }
  } else {
    // ------------------------------------------------------ epilogue warps
    const int quarter = warp & 3;     // TMEM lane quarter this warp may access
    const int side = (warp - 2) >> 2; // which of the quarter's two warps
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    // this lane's row of the warp's 32 x 64 columns, 16-byte pieces swizzled as TMA reads them
    const uint32_t out = smem_u32(sOut + (warp - 2) * OUT_BYTES);
    auto put = [&](int piece, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
      st_shared_v4(out + lane * 128 + ((piece ^ (lane & 7)) << 4), x, y, z, w);
    };
    uint32_t phase = 0;
    int turn = 0;
    for (int tile = pair; tile < a.num_tiles; tile += pairs, phase ^= 1u) {
      int mb, nb;
      tile_coords4(tile, a, mb, nb);
      const int row0 = (2 * mb + static_cast<int>(rank)) * ROWS + quarter * 32;
      // scales of the row and, in shared memory, of the warp's 128 columns (or 64 and 64), read
      // while the products run
      float ra = 1.f;
      float4* rb = nullptr;
      if constexpr (NV) {
        if (row0 + lane < a.M) ra = *(a.ra + row0 + lane);
        const int b = SWIGLU ? (lane >> 4) * a.up_rows + nb * (BN4 / 2) + side * 64 + (lane & 15) * 4
                             : nb * BN4 + side * (BN4 / 2) + lane * 4;
        // (the four warps of a side write the same; none is three tiles behind another)
        rb = reinterpret_cast<float4*>(sScale) + (turn * 2 + side) * 32;
        if (SWIGLU || b < a.N) rb[lane] = *reinterpret_cast<const float4*>(a.rb + b);
        __syncwarp();
        if (++turn == 3) turn = 0;
      }
      if (!mbar_wait_warp(bar(B4_TFULL), phase, a.err, ERR_WAIT_GEMM_EPILOGUE)) break;
      tc_fence_after();
      // chunks of 32 columns: the warp's half of the tile; gate and up of its half
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld32(t_row + (SWIGLU ? (c >> 1) * (BN4 / 2) + side * 64 + (c & 1) * 32
                                  : side * (BN4 / 2) + c * 32),
                  v[c]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_reg_fence(v[c]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(bar(B4_TEMPTY));
        else
          mbar_arrive_remote(mapa_shared(bar(B4_TEMPTY), even));
      }
      if constexpr (SPLIT) {
        // to shared memory, where no load and no product is under way any more: 16 bytes c of row
        // r at c ^ (r & 31)
        if (row0 < a.M) {
          const uint32_t sums = smem_u32(smem) + (quarter * 32 + lane) * (BN4 * 4);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int col = SWIGLU ? (c >> 1) * (BN4 / 2) + side * 64 + (c & 1) * 32
                                   : side * (BN4 / 2) + c * 32;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4(sums + (((col / 4 + j) ^ lane) << 4), v[c][4 * j], v[c][4 * j + 1],
                           v[c][4 * j + 2], v[c][4 * j + 3]);
          }
        }
        continue;
      }
      if (row0 >= a.M) continue;
      const long long drained = clock64();
      // the turn-th sixteenth of the next tile's products
      auto wait_turn = [&](int turn) {
        if (tile + pairs < a.num_tiles)
          while (static_cast<uint64_t>(clock64() - drained) < static_cast<uint32_t>(turn * a.pace))
            __nanosleep(64);
        __syncwarp();
      };
      // eight products, v[c][8 j ..], scaled
      auto scaled = [&](int c, int j, float (&f)[8]) {
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = __uint_as_float(v[c][8 * j + t]);
        if constexpr (NV) {
          float b[8];
          *reinterpret_cast<float4*>(b) = rb[c * 8 + 2 * j];
          *reinterpret_cast<float4*>(b + 4) = rb[c * 8 + 2 * j + 1];
#pragma unroll
          for (int t = 0; t < 8; t += 2) {
            fmul2(f[t], f[t + 1], ra, ra);
            fmul2(f[t], f[t + 1], b[t], b[t + 1]);
          }
        }
      };
      auto send = [&](int col) {  // what is put, to the output's columns from col on
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmC, out, col, row0);
          store_commit();
          store_wait_read();
        }
        __syncwarp();
      };
      if constexpr (SWIGLU) {
        const int col0 = nb * (BN4 / 2) + side * 64;
        wait_turn(2 * (warp - 2));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float g[8], u[8];
            scaled(c, j, g);
            scaled(2 + c, j, u);
            uint32_t o[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
              o[t] = swiglu2(g[2 * t], g[2 * t + 1], u[2 * t], u[2 * t + 1]);
            put(c * 4 + j, o[0], o[1], o[2], o[3]);
          }
        }
        send(col0);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col0 = nb * BN4 + side * (BN4 / 2) + h * 64;
          if (col0 < a.N) {
            wait_turn(warp - 2 + h * EPI_WARPS);
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              float f[8];
              scaled(2 * h + (p >> 2), p & 3, f);
              put(p, pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                  pack_bf16x2(f[6], f[7]));
            }
            send(col0);
          }
        }
      }
    }
    if (lane == 0) store_wait();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if constexpr (SPLIT) {
    // this pair's share of the tile's rows: a warp takes one after the other, a lane four columns
    // of it, twice (the second of which are the up half's in SwiGLU)
    constexpr int WIDTH = SWIGLU ? BN4 / 2 : BN4;
    int mb, nb;
    tile_coords4(pair, a, mb, nb);
    const int first = (2 * mb + static_cast<int>(rank)) * ROWS;
    const int rows = max(0, min(ROWS, a.M - first));
    const uint32_t sums = smem_u32(smem);
    for (int r = rows * part / a.parts + warp; r < rows * (part + 1) / a.parts; r += THREADS4 / 32) {
      // every part's loads are under way before the first is used
      float4 y[4][2];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (p < a.parts) {
          const uint32_t at = mapa_shared(sums + r * (BN4 * 4), 2 * p + rank);
#pragma unroll
          for (int u = 0; u < 2; ++u) ld_cluster_v4(y[p][u], at + (((lane + 32 * u) ^ (r & 31)) << 4));
        }
      }
      float f[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int t = 0; t < 4; ++t) f[u][t] = 0.f;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if (p < a.parts) {
            f[u][0] += y[p][u].x, f[u][1] += y[p][u].y;
            f[u][2] += y[p][u].z, f[u][3] += y[p][u].w;
          }
        }
        const int b = nb * WIDTH + lane * 4 + u * (SWIGLU ? a.up_rows : 128);
        if (NV && (SWIGLU || b < a.N)) {
          const float ra = *(a.ra + first + r);
          const float4 rb = *reinterpret_cast<const float4*>(a.rb + b);
          f[u][0] *= ra, f[u][1] *= ra, f[u][2] *= ra, f[u][3] *= ra;
          f[u][0] *= rb.x, f[u][1] *= rb.y, f[u][2] *= rb.z, f[u][3] *= rb.w;
        }
      }
      __nv_bfloat16* c = a.C + static_cast<int64_t>(first + r) * a.N + nb * WIDTH + lane * 4;
      auto store = [&](int u, uint32_t x, uint32_t y) {
        if (nb * WIDTH + lane * 4 + u * 128 < a.N)
          *reinterpret_cast<uint2*>(c + u * 128) = make_uint2(x, y);
      };
      if constexpr (SWIGLU) {
        store(0, swiglu2(f[0][0], f[0][1], f[1][0], f[1][1]),
              swiglu2(f[0][2], f[0][3], f[1][2], f[1][3]));
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          store(u, pack_bf16x2(f[u][0], f[u][1]), pack_bf16x2(f[u][2], f[u][3]));
      }
    }
    cluster_sync_all();  // a peer may still be reading this CTA's sums
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool NV, bool SWIGLU>
h3_status launch4(const Fp4Operand& A, const Fp4Operand& B, void* C, int L, int N, int K,
                  cudaStream_t s) {
  static std::atomic<bool> done[64], done_split[64];
  h3_status st = set_smem_limit(done, gemm_fp4_kernel<NV, SWIGLU, false>, SMEM4_BYTES,
                                "fp4 gemm: set shared memory size");
  if (st != H3_OK) return st;
  const int b_rows = SWIGLU ? 2 * N : N;
  const int tile_n = SWIGLU ? BN4 / 2 : BN4;
  Gemm4Args a{};
  a.C = static_cast<__nv_bfloat16*>(C);
  a.ra = A.row_scale;
  a.rb = B.row_scale;
  a.M = L;
  a.N = N;
  a.K = K;
  a.num_m = (L + 2 * ROWS - 1) / (2 * ROWS);
  a.num_n = (N + tile_n - 1) / tile_n;
  a.num_k = (K + STAGE_CODES - 1) / STAGE_CODES;
  a.num_tiles = a.num_m * a.num_n;
  a.sf_tiles = fp4_tiles(K, NV);
  // seven eighths of the products' 128 cycles for every 64 values of K; SwiGLU's last warp has that
  // much to do after its turn (9,728 x 8,192 x 2,048 MX 111 us, 124 without the allowance)
  a.pace = std::max(0, a.num_k * (STAGE_CODES / 64) * 112 - (SWIGLU ? (NV ? 1800 : 1400) : 0)) / 16;
  a.up_rows = SWIGLU ? N : 0;
  if ((st = dev_err(&a.err)) != H3_OK) return st;
  CUtensorMap tmA, tmB, tmSA, tmSB, tmC;
  const uint64_t row_bytes = static_cast<uint64_t>(K) / 2;
  if ((st = make_tmap_u8_2d(&tmA, A.codes, row_bytes, L, row_bytes, 128, ROWS)) != H3_OK) return st;
  if ((st = make_tmap_u8_2d(&tmB, B.codes, row_bytes, b_rows, row_bytes, 128, ROWS)) != H3_OK)
    return st;
  // scales: rows of a tile each, a stage's at a time
  const uint64_t ta = static_cast<uint64_t>((L + ROWS - 1) / ROWS) * a.sf_tiles;
  const uint64_t tb = static_cast<uint64_t>((b_rows + ROWS - 1) / ROWS) * a.sf_tiles;
  constexpr uint32_t atoms = NV ? 4 : 2;
  if ((st = make_tmap_u32_rows(&tmSA, A.scales, 128, ta, atoms)) != H3_OK) return st;
  if ((st = make_tmap_u32_rows(&tmSB, B.scales, 128, tb, atoms)) != H3_OK) return st;
  if ((st = make_tmap_bf16_2d(&tmC, C, N, L, static_cast<uint64_t>(N) * 2, 64, 32)) != H3_OK) return st;
  // As many pairs to a tile as all tiles find room for, of four stages each at least, or, where
  // there are more rows for the sums to be exchanged of, eight (4-bit rows and product, weights
  // in HBM: 22 x 5,376 x 5,376 10.4 us by three pairs, 13.2 by one; 256 rows 14.5 by three of
  // seven stages, 13.5 by two, 14.3 by one; K and N 2,048 22 rows 8.4 by two pairs of four
  // stages, 8.7 by one, 128 rows 10.3 and 9.5; 512 x 2,560 x 10,240 18.0 by three, 21.7 by one)
  const int least = L > 64 ? 8 : 4;
  static std::atomic<int> room[64][9];
  a.parts = 1;
  for (int p = 4; p >= 2; --p) {
    if (a.num_tiles * 2 * p > num_sms() || a.num_k < least * p) continue;
    st = set_smem_limit(done_split, gemm_fp4_kernel<NV, SWIGLU, true>, SMEM4_BYTES,
                        "fp4 gemm: set shared memory size");
    if (st != H3_OK) return st;
    if (clusters_at_once(room, gemm_fp4_kernel<NV, SWIGLU, true>, THREADS4, SMEM4_BYTES, 2 * p) >=
        a.num_tiles) {
      a.parts = p;
      break;
    }
  }
  const int grid = 2 * (a.parts > 1 ? a.num_tiles * a.parts : std::min(a.num_tiles, num_sms() / 2));
  return cuda_fail(
      launch_overlapped(a.parts > 1 ? gemm_fp4_kernel<NV, SWIGLU, true>
                                    : gemm_fp4_kernel<NV, SWIGLU, false>,
                        dim3(grid), THREADS4, SMEM4_BYTES, 2 * a.parts, s, tmA, tmB, tmSA, tmSB, tmC, a),
      "fp4 gemm launch");
}

}  // namespace

h3_status launch_gemm_fp4(const Fp4Operand& a, const Fp4Operand& b, void* C, int L, int N, int K,
                          bool nv, bool swiglu, cudaStream_t s) {
  if (nv)
    return swiglu ? launch4<true, true>(a, b, C, L, N, K, s) : launch4<true, false>(a, b, C, L, N, K, s);
  return swiglu ? launch4<false, true>(a, b, C, L, N, K, s) : launch4<false, false>(a, b, C, L, N, K, s);
}

}  // namespace h3
