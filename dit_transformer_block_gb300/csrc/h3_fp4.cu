// Quantisation of bf16 rows to microscaled 4-bit floating point (E2M1 codes).
//
// A CTA takes a row, a lane eight neighbouring values of it; four lanes (MX, blocks of 32)
// or two (NV, blocks of 16) share a block and find its largest magnitude by shuffles of
// the values' bits, which order like the magnitudes, NaN above infinity above all
// others. NV first needs the largest of the row, so the row stays in registers. Bound by
// HBM: 2 bytes in, 0.53 or 0.56 out per value.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "h3_fp4.cuh"
#include "h3_internal.cuh"
#include "h3_launch.cuh"

namespace h3 {
namespace {

// Eight E2M1 codes, the first in the low half of the low byte.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

constexpr uint32_t BF16_INF = 0x7f80u;

// Bits of the largest magnitude among a lane's eight values.
__device__ __forceinline__ uint32_t top_bits(const uint4& v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                              __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

template <bool NV, int T, int VPT>
__global__ void __launch_bounds__(T)
    quantize_fp4_kernel(const __nv_bfloat16* x, int64_t ldx,
                        uint8_t* codes, uint8_t* scales,
                        float* row_scale, int K) {
  __shared__ uint32_t red[T / 32];
  const int row = blockIdx.x;
  const int K8 = K >> 3;
  // lanes' worth of a row, whole tiles of four scales
  const int K8s = NV ? (K8 + 7) & ~7 : (K8 + 15) & ~15;
  const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(row) * ldx);
  wait_previous();
  const int tid = threadIdx.x;
  uint4 v[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * T;
    v[i] = c < K8 ? __ldcs(src + c) : make_uint4(0, 0, 0, 0);
  }
  uint32_t top[VPT], row_top = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    uint32_t t = top_bits(v[i]);
    t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
    if constexpr (!NV) t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
    top[i] = t;
    if (t < BF16_INF) row_top = max(row_top, t);
  }
  float to_scale = 0.f, to_code = 0.f;
  if constexpr (NV) {
    row_top = __reduce_max_sync(0xffffffffu, row_top);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = row_top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w) row_top = max(row_top, red[w]);
    const float amax = __uint_as_float(row_top << 16);
    const bool some = amax >= FP4_LEAST_ROW;
    if (some) {
      to_scale = __fdiv_rn(448.0f, amax);
      to_code = __fdiv_rn(2688.0f, amax);
    }
    if (threadIdx.x == 0) row_scale[row] = some ? __fdiv_rn(amax, 2688.0f) : 0.f;
  }
  launch_next();
  const int per = NV ? 2 : 4;  // lanes of a block
  uint8_t* srow = scales + static_cast<int64_t>(row >> 7) * (K8s / (4 * per)) * 512 +
                  (row & 31) * 16 + ((row & 127) >> 5) * 4;
  uint32_t* dst = reinterpret_cast<uint32_t*>(codes + static_cast<int64_t>(row) * (K >> 1));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * T;
    if (c >= K8s) break;
    const bool bad = top[i] >= BF16_INF;
    float mul;
    uint32_t byte;
    if constexpr (NV) {
      const float amax = __uint_as_float(top[i] << 16);
      byte = __nv_cvt_float_to_fp8(__fmul_rn(amax, to_scale), __NV_SATFINITE, __NV_E4M3);
      const float sf = __half2float(__half(__nv_cvt_fp8_to_halfraw(byte, __NV_E4M3)));
      mul = byte != 0u ? __fdiv_rn(to_code, sf) : 0.f;
      if (bad) byte = 0x7fu;
    } else {
      const int e = static_cast<int>(top[i] >> 7) - 2;
      byte = bad ? 255u : static_cast<uint32_t>(max(e, 0));
      mul = __uint_as_float((254u - min(byte, 253u)) << 23);
    }
    if (c < K8) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __fmul_rn(bf16_lo(w[j]), mul);
        f[2 * j + 1] = __fmul_rn(bf16_hi(w[j]), mul);
      }
      dst[c] = bad ? 0u : e2m1x8(f);
    }
    const int b = c / per;
    if (c % per == 0) srow[static_cast<int64_t>(b >> 2) * 512 + (b & 3)] = static_cast<uint8_t>(byte);
  }
}

template <bool NV>
h3_status launch(const void* x, int64_t ldx, void* codes, void* scales, float* row_scale, int R,
                 int K, cudaStream_t s) {
  const auto* xx = static_cast<const __nv_bfloat16*>(x);
  auto* cc = static_cast<uint8_t*>(codes);
  auto* ss = static_cast<uint8_t*>(scales);
  const int k8s = (K / 8 + 15) & ~15;
#define H3_Q4(T, V) \
  launch_overlapped(quantize_fp4_kernel<NV, T, V>, dim3(R), T, 0, 1, s, xx, ldx, cc, ss, row_scale, K)
  const cudaError_t e = k8s <= 128    ? H3_Q4(128, 1)
                        : k8s <= 256  ? H3_Q4(256, 1)
                        : k8s <= 512  ? H3_Q4(256, 2)
                        : k8s <= 768  ? H3_Q4(256, 3)
                        : k8s <= 1024 ? H3_Q4(256, 4)
                        : k8s <= 1536 ? H3_Q4(256, 6)
                                      : H3_Q4(256, 8);
#undef H3_Q4
  return cuda_fail(e, "quantize_fp4_rows launch");
}

}  // namespace

h3_status launch_quantize_fp4_rows(const void* x, int64_t ldx, void* codes, void* scales,
                                   float* row_scale, int R, int K, bool nv, cudaStream_t s) {
  return nv ? launch<true>(x, ldx, codes, scales, row_scale, R, K, s)
            : launch<false>(x, ldx, codes, scales, nullptr, R, K, s);
}

}  // namespace h3
