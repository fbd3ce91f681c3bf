// Norms before and after a branch, fused with the branch's gate and the scaled
// residual: a CTA per row, or a warp, which stays in registers from its loads to its stores.
//
// Per row: p = n(delta) * post_gain, r = resid_scale * resid + gate * p, h = n(r) * pre_gain * (1
// + scale) + shift, with n a LayerNorm without affine or a division by the root mean square.
// Everything between the loads and the stores is FP32, and the mean is taken before the squares
// (two passes over registers), so a row far from zero loses a few units of 2^-24 |mean|, off
// every value, and not of |mean|^2. Bound by HBM: 4 + 2 bytes per element in, 4 + 2 out (58,758
// rows of 5,376, 3.79 GB: LayerNorm 593 us, 6.4 TB/s, RMS 543 us, 7.0 TB/s; 22 rows: 3.6 us, the
// latency of a load, of two or four sums over the CTA and of a launch). Launched like an ordinary
// kernel, since its loads of vectors that all rows share take the read-only path: without it, and
// launched ahead of the end of the kernel before it, LayerNorm took 665 us.
#include <cuda_bf16.h>

#include <algorithm>

#include "h3_internal.cuh"
#include "h3_launch.cuh"

namespace h3 {
namespace {

// Half of the least power of two that is not below n.
constexpr int warps_half(int n) {
  int m = 1;
  while (m < n) m *= 2;
  return m / 2;
}

// Threads of a row: a warp (of NORM_WARPS in a CTA), or a CTA.
constexpr int NORM_WARPS = 4;
template <int T>
__device__ __forceinline__ int thread_of() {
  return static_cast<int>(T == 32 ? threadIdx.x & 31 : threadIdx.x);
}

template <int T>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if constexpr (T == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float t = (lane < T / 32) ? red[lane] : 0.f;
#pragma unroll
  for (int m = warps_half(T / 32); m >= 1; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
  return __shfl_sync(0xffffffffu, t, 0);
}

// x <- n(x) over a row of D values, VPT float4 of it in this thread's registers
// (zeros beyond the row). red: two buffers of T / 32 floats, the second reduction's
// being free of the first's readers. False, the same in every thread of the row, where the sum of
// the squares is not finite (nor is it where the sum of the values is not): x is of no use then.
template <int T, int VPT, bool RMS>
__device__ __forceinline__ bool norm_row(float4 (&x)[VPT], int D4, float inv_d, float eps,
                                         float* red) {
  if constexpr (!RMS) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) s += (x[v].x + x[v].y) + (x[v].z + x[v].w);
    const float mean = row_sum<T>(s, red) * inv_d;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (thread_of<T>() + v * T < D4) {
        x[v].x -= mean;
        x[v].y -= mean;
        x[v].z -= mean;
        x[v].w -= mean;
      }
    }
  }
  float q = 0.f;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    q += (x[v].x * x[v].x + x[v].y * x[v].y) + (x[v].z * x[v].z + x[v].w * x[v].w);
  const float squares = row_sum<T>(q, red + T / 32);
  if (!(squares < INFINITY)) return false;
  const float rstd = rsqrtf(squares * inv_d + eps);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    x[v].x *= rstd;
    x[v].y *= rstd;
    x[v].z *= rstd;
    x[v].w *= rstd;
  }
  return true;
}

struct NormArgs {
  const float* resid;
  const __nv_bfloat16* delta;
  float* resid_out;
  __nv_bfloat16* normed;
  const float* post_gain;
  const float* gate;
  const float* pre_gain;
  const float* shift;
  const float* scale;
  const int32_t* seg;
  int num_seg;
  int64_t seg_stride;
  float resid_scale, eps, inv_d;
  int D4, L;
};

// n(x) = (x * k - mean) * rstd of a row that load(c) gives the float4 c of. k is 1, or 2^-80 where the
// sums of that are not finite: 8,192 squares of any values times 2^-80 have a finite sum, and of eps
// there is left what keeps a row of equal values from 0 / 0. (What is infinite or NaN stays so.)
struct RowNorm {
  float k, mean, rstd;

  template <int T, bool RMS, class Load>
  __device__ __forceinline__ void find(const Load& load, const NormArgs& a, float* red) {
    float eps = a.eps;
    mean = 0.f;
#pragma unroll 1
    for (k = 1.f;;) {
      float q = 0.f;
#pragma unroll 1
      for (int pass = RMS ? 1 : 0; pass < 2; ++pass) {
        float s = 0.f;
#pragma unroll 1
        for (int c = thread_of<T>(); c < a.D4; c += T) {
          const float4 x = load(c);
          const float u[4] = {x.x * k - mean, x.y * k - mean, x.z * k - mean, x.w * k - mean};
          s += pass == 0 ? (u[0] + u[1]) + (u[2] + u[3])
                         : (u[0] * u[0] + u[1] * u[1]) + (u[2] * u[2] + u[3] * u[3]);
        }
        if constexpr (T > 32) __syncthreads();  // the last sum's parts are read
        q = row_sum<T>(s, red) * a.inv_d;
        if (pass == 0) mean = q;
      }
      rstd = rsqrtf(q + eps);
      if (q < INFINITY || k < 1.f) return;
      k = 8.271806125530277e-25f;                       // 2^-80
      if (eps > 0.f) eps = 1.1754943508222875e-38f;  // 2^-126
      mean = 0.f;
    }
  }
  __device__ __forceinline__ float4 operator()(float4 x) const {
    return make_float4((x.x * k - mean) * rstd, (x.y * k - mean) * rstd, (x.z * k - mean) * rstd,
                       (x.w * k - mean) * rstd);
  }
};

// A row some of whose sums are not finite, once more and from memory, a float4 at a time: from the branch
// on, or (stored) from the new residual on, which then lies in resid_out, or in resid where there is none.
// Out of line: on the rows' registers, inlined, 58,758 x 5,376 RMS took 636 us instead of 540.
template <int T, bool RMS, bool POST>
__device__ __noinline__ void large_row(const NormArgs& a, int64_t row, bool stored, float* red) {
  const float4* rrow = reinterpret_cast<const float4*>(a.resid) + row * a.D4;
  const uint2* drow = reinterpret_cast<const uint2*>(a.delta) + row * a.D4;
  float4* orow = reinterpret_cast<float4*>(a.resid_out) + row * a.D4;
  int64_t off = 0;
  if (a.seg != nullptr)
    off = static_cast<int64_t>(min(max(a.seg[row], 0), a.num_seg - 1)) * a.seg_stride;
  auto vec = [](const float* p, int c, float d) {
    return p != nullptr ? reinterpret_cast<const float4*>(p)[c] : make_float4(d, d, d, d);
  };
  const float* gate = a.gate != nullptr ? a.gate + off : nullptr;
  RowNorm n{1.f, 0.f, 1.f};
  if (!stored) {  // (there is a branch, and its sums are not finite)
    auto branch = [&](int c) {
      const uint2 d = drow[c];
      return make_float4(bf16_lo(d.x), bf16_hi(d.x), bf16_lo(d.y), bf16_hi(d.y));
    };
    if constexpr (POST) n.find<T, RMS>(branch, a, red);
#pragma unroll 1
    for (int c = thread_of<T>(); c < a.D4; c += T) {
      const float4 p = n(branch(c)), b = vec(POST ? a.post_gain : nullptr, c, 1.f), g = vec(gate, c, 1.f);
      const float4 x = rrow[c];
      const float f = a.resid_scale;
      orow[c] = make_float4(fmaf(g.x, p.x * b.x, f * x.x), fmaf(g.y, p.y * b.y, f * x.y),
                            fmaf(g.z, p.z * b.z, f * x.z), fmaf(g.w, p.w * b.w, f * x.w));
    }
  }
  launch_next();
  if (a.normed == nullptr) return;
  // (a thread reads what it has stored itself)
  const float4* from = a.resid_out != nullptr ? orow : rrow;
  auto value = [&](int c) { return from[c]; };
  n.find<T, RMS>(value, a, red);
  uint2* hrow = reinterpret_cast<uint2*>(a.normed) + row * a.D4;
  const float* scale = a.scale != nullptr ? a.scale + off : nullptr;
  const float* shift = a.shift != nullptr ? a.shift + off : nullptr;
#pragma unroll 1
  for (int c = thread_of<T>(); c < a.D4; c += T) {
    const float4 x = n(value(c)), s = vec(scale, c, 0.f), g = vec(a.pre_gain, c, 1.f), b = vec(shift, c, 0.f);
    hrow[c] = make_uint2(
        pack_bf16x2(fmaf(x.x, (1.f + s.x) * g.x, b.x), fmaf(x.y, (1.f + s.y) * g.y, b.y)),
        pack_bf16x2(fmaf(x.z, (1.f + s.z) * g.z, b.z), fmaf(x.w, (1.f + s.w) * g.w, b.w)));
  }
}

// CTAs that an SM holds: as many as the row's registers leave, which the call of large_row would lessen
// (58,758 rows, us with it left out / in and bounded / in: 5,376 LayerNorm 585 / 593 / 596, RMS 540 /
// 543 / 629; 4,096 RMS 409 / 406 / 443; the others alike).
constexpr int norm_ctas(int threads, int vpt) {
  return 65536 / (threads * (vpt == 2 ? 32 : vpt == 3 ? 42 : vpt == 4 ? 56 : 64));
}

template <int T, int VPT, bool RMS, bool POST>
__global__ void __launch_bounds__(T == 32 ? NORM_WARPS * 32 : T,
                                  norm_ctas(T == 32 ? NORM_WARPS * 32 : T, VPT))
    sandwich_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[4 * (T / 32)];
  const int tid = thread_of<T>();
  const int64_t row =
      T == 32 ? static_cast<int64_t>(blockIdx.x) * NORM_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (T == 32 && row >= a.L) return;
  const int D4 = a.D4;
  const float4* rrow = reinterpret_cast<const float4*>(a.resid) + row * D4;
  float4 x[VPT], y[VPT];
  // every load of the row is requested before the first use
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = tid + v * T;
    x[v] = c < D4 ? __ldcs(rrow + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const bool branch = a.delta != nullptr;
  if (branch) {
    const uint2* drow = reinterpret_cast<const uint2*>(a.delta) + row * D4;
    uint2 d[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = tid + v * T;
      d[v] = c < D4 ? __ldcs(drow + c) : make_uint2(0, 0);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      y[v] = make_float4(bf16_lo(d[v].x), bf16_hi(d[v].x), bf16_lo(d[v].y), bf16_hi(d[v].y));
  }
  int64_t off = 0;
  if (a.seg != nullptr)
    off = static_cast<int64_t>(min(max(__ldg(a.seg + row), 0), a.num_seg - 1)) * a.seg_stride;
  auto vec = [](const float* p, int c) { return __ldg(reinterpret_cast<const float4*>(p) + c); };

  if (branch) {
    if constexpr (POST) {
      if (!norm_row<T, VPT, RMS>(y, D4, a.inv_d, a.eps, red)) {
        large_row<T, RMS, POST>(a, row, false, red);
        return;
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = tid + v * T;
      if (c < D4) {
        if (POST && a.post_gain != nullptr) {
          const float4 g = vec(a.post_gain, c);
          y[v].x *= g.x;
          y[v].y *= g.y;
          y[v].z *= g.z;
          y[v].w *= g.w;
        }
        float4 g = make_float4(1.f, 1.f, 1.f, 1.f);
        if (a.gate != nullptr) g = vec(a.gate + off, c);
        x[v].x = fmaf(g.x, y[v].x, a.resid_scale * x[v].x);
        x[v].y = fmaf(g.y, y[v].y, a.resid_scale * x[v].y);
        x[v].z = fmaf(g.z, y[v].z, a.resid_scale * x[v].z);
        x[v].w = fmaf(g.w, y[v].w, a.resid_scale * x[v].w);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      x[v].x *= a.resid_scale;
      x[v].y *= a.resid_scale;
      x[v].z *= a.resid_scale;
      x[v].w *= a.resid_scale;
    }
  }
  if (a.resid_out != nullptr) {
    float4* orow = reinterpret_cast<float4*>(a.resid_out) + row * D4;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = tid + v * T;
      if (c < D4) __stcs(orow + c, x[v]);
    }
  }
  launch_next();
  if (a.normed == nullptr) return;
  if (!norm_row<T, VPT, RMS>(x, D4, a.inv_d, a.eps, red + 2 * (T / 32))) {
    large_row<T, RMS, POST>(a, row, true, red);
    return;
  }
  uint2* hrow = reinterpret_cast<uint2*>(a.normed) + row * D4;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = tid + v * T;
    if (c < D4) {
      float4 m = make_float4(1.f, 1.f, 1.f, 1.f), b = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.scale != nullptr) {
        const float4 s = vec(a.scale + off, c);
        m = make_float4(1.f + s.x, 1.f + s.y, 1.f + s.z, 1.f + s.w);
      }
      if (a.pre_gain != nullptr) {
        const float4 g = vec(a.pre_gain, c);
        m.x *= g.x;
        m.y *= g.y;
        m.z *= g.z;
        m.w *= g.w;
      }
      if (a.shift != nullptr) b = vec(a.shift + off, c);
      __stcs(hrow + c, make_uint2(pack_bf16x2(fmaf(x[v].x, m.x, b.x), fmaf(x[v].y, m.y, b.y)),
                                  pack_bf16x2(fmaf(x[v].z, m.z, b.z), fmaf(x[v].w, m.w, b.w))));
    }
  }
}

template <int T, int VPT, bool RMS>
void launch_width(const NormArgs& a, bool post, cudaStream_t s) {
  const int grid = T == 32 ? (a.L - 1) / NORM_WARPS + 1 : a.L, threads = T == 32 ? NORM_WARPS * 32 : T;
  if (post)
    sandwich_norm_kernel<T, VPT, RMS, true><<<grid, threads, 0, s>>>(a);
  else
    sandwich_norm_kernel<T, VPT, RMS, false><<<grid, threads, 0, s>>>(a);
}

// Few threads with many vectors each have less to exchange, and more of a row's registers are of
// the row; many have more loads under way. A LayerNorm, which exchanges twice as often, takes
// fewer from 641 float4 on. (58,758 rows, us for LayerNorm / RMS: 512 wide 59 / 59, 74 / 66 with
// 128 threads; 1,152 128 / 125, 187 / 142 with 256; 2,048 210 / 210, 231 / 208 with 256; 4,096
// LayerNorm 429, 454 with 512, RMS 413, 418 with 256; 5,376 LayerNorm 591, 600 with 512 and 613
// with 224, RMS 545, 572 with 384.)
template <bool RMS>
void launch_rows(const NormArgs& a, bool post, cudaStream_t s) {
  const int d4 = a.D4;
  if (d4 <= 64) return launch_width<32, 2, RMS>(a, post, s);
  if (d4 <= 128) return launch_width<32, 4, RMS>(a, post, s);
  if (d4 <= 256) return launch_width<64, 4, RMS>(a, post, s);
  if (d4 <= 320) return launch_width<64, 5, RMS>(a, post, s);
  if (d4 <= 384) return launch_width<128, 3, RMS>(a, post, s);
  if (d4 <= 512) return launch_width<128, 4, RMS>(a, post, s);
  if (d4 <= 640) return launch_width<160, 4, RMS>(a, post, s);
  if (d4 > 1536) return launch_width<512, 4, RMS>(a, post, s);
  if constexpr (RMS) {
    if (d4 <= 768) return launch_width<256, 3, RMS>(a, post, s);
    if (d4 <= 1024) return launch_width<512, 2, RMS>(a, post, s);
    launch_width<512, 3, RMS>(a, post, s);
  } else {
    if (d4 <= 768) return launch_width<192, 4, RMS>(a, post, s);
    if (d4 <= 1024) return launch_width<256, 4, RMS>(a, post, s);
    if (d4 <= 1280) return launch_width<256, 5, RMS>(a, post, s);
    launch_width<384, 4, RMS>(a, post, s);
  }
}

}  // namespace

h3_status launch_sandwich_norm(const float* resid, const void* delta, float* resid_out,
                               void* normed, bool post_norm, const float* post_gain,
                               const float* gate, float resid_scale, const float* pre_gain,
                               const float* shift, const float* scale, const int32_t* seg,
                               int num_seg, int64_t seg_stride, bool rms, int L, int D, float eps,
                               cudaStream_t s) {
  const NormArgs a{resid, static_cast<const __nv_bfloat16*>(delta),
                   resid_out, static_cast<__nv_bfloat16*>(normed),
                   post_gain, gate, pre_gain, shift, scale, seg, num_seg, seg_stride,
                   resid_scale, eps, 1.0f / static_cast<float>(D), D / 4, L};
  if (rms)
    launch_rows<true>(a, post_norm, s);
  else
    launch_rows<false>(a, post_norm, s);
  return cuda_fail(cudaGetLastError(), "sandwich_norm launch");
}

}  // namespace h3
