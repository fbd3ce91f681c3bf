// Paged key/value cache: writing the rows of a call to it, with Q/K RMSNorm and
// RoPE on the way.
//
// A cache holds pages of `page` keys (a power of two from 16 to 128), laid out
// [pages, Hkv, page, 128]: the keys of one page and head are one contiguous
// block. Row t of the call belongs to the sequence b with cu_q[b] <= t <
// cu_q[b + 1]; kv_len[b] is that sequence's length with the call's rows in it,
// and key j lies in page page_table[b * max_pages + j / page], row j % page.
#include <cuda_bf16.h>

#include <algorithm>

#include "h3_internal.cuh"
#include "h3_rope.cuh"

namespace h3 {
namespace {

constexpr int DHP = QK_HEAD_DIM;

struct SeqRow {
  int b;      // sequence of the row, or -1: behind the last sequence (or before the first)
  int i;      // row within the sequence
  int q_len;  // rows of the sequence
};

// The sequence of row t, by the whole warp.
__device__ __forceinline__ SeqRow find_row(const int32_t* __restrict__ cu_q, int B, int t) {
  const int n = ends_up_to(cu_q, B, t);
  SeqRow r{-1, 0, 0};
  if (n < B) {
    const int first = __ldg(cu_q + n), end = __ldg(cu_q + n + 1);
    if (first >= 0 && first <= t && t < end) r = {n, t - first, end - first};
  }
  return r;
}

// ------------------------------------------------------------------ append
// A CTA takes up to APPEND_ROWS consecutive rows, or a slice of the heads of
// one: a warp per row finds its place, a thread per (row, pair) its angles, and
// then every half-warp takes one 128-channel head after the other (8 channels
// per lane) of the row's H query, Hkv key and Hkv value heads, APPEND_BATCH of
// them requested at a time, the first ones before the places and angles are
// known. (A warp that looked up its own row's place for every 8 heads spent its
// life on the three dependent loads of that: 1.06 ms for 58,758 rows of 126
// heads.)
// Measured at 58,758 rows of 42 + 84 heads, interleaved pairs: 642 us (5.9 TB/s
// of 3.8 GB; at the 64 registers of eight CTAs per SM 28 bytes are spilled); 256
// threads with 4 rows 665-776, batches of 8 heads 675. Split-half pairs, with a
// shuffle per channel: 754 us at six CTAs per SM (80 registers, no spills; eight
// CTAs 1,069, five 797).
constexpr int APPEND_THREADS = 128, APPEND_ROWS = 2, APPEND_BATCH = 4;
template <bool HALF>
constexpr int APPEND_CTAS = HALF ? 6 : 8;  // per SM
constexpr int APPEND_STEP = APPEND_THREADS / 16;  // heads at a time

struct AppendArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t ld_q, ld_k, ld_v;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  const float* q_gain;  // given with k_gain where there is a q
  const float* k_gain;  // NULL: no norm
  const int32_t* pos;
  float eps;
  int H, Hkv;
  int rows, slice;  // rows, and heads of a row, per CTA
  PagedBatch b;
};

// 8 channels (one lane's) of a head: normed by its RMS and gain if there is one,
// its pairs turned by (cos, sin) from cs on. Which products are fused is written out,
// so that the result has the bits of the in-place Q/K kernel.
template <bool HALF>
__device__ __forceinline__ uint4 norm_turn(uint4 w, bool norm, const float (&gain)[8], float eps,
                                           const float2* turn, bool first, int src_lane) {
  const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(wd[j]);
    f[2 * j + 1] = bf16_hi(wd[j]);
  }
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float inv = rsqrtf(ss * (1.0f / DHP) + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * inv * gain[j];
  }
  const float4* cs = reinterpret_cast<const float4*>(turn);
  uint32_t o[4];
  if constexpr (HALF) {
    float y[8];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float4 c = cs[t];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 2 * t + e;
        const float co = e ? c.z : c.x, si = e ? c.w : c.y;
        const float p = __shfl_sync(0xffffffffu, f[j], src_lane);  // the pair's other element
        y[j] = first ? fmaf(f[j], co, -__fmul_rn(p, si)) : fmaf(p, si, __fmul_rn(f[j], co));
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = pack_bf16x2(y[2 * t], y[2 * t + 1]);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float4 c = cs[t >> 1];
      const float co = t & 1 ? c.z : c.x, si = t & 1 ? c.w : c.y;
      const float x = f[2 * t], y = f[2 * t + 1];
      o[t] = pack_bf16x2(fmaf(x, co, -__fmul_rn(y, si)), fmaf(x, si, __fmul_rn(y, co)));
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool HALF>
__global__ void __launch_bounds__(APPEND_THREADS, APPEND_CTAS<HALF>)
    kv_append_kernel(const AppendArgs a, const RopeTable tab) {
  __shared__ float2 turn[APPEND_ROWS][DHP / 2];  // (cos, sin)
  // the row's key: page * Hkv * page_size + row in page (for head 0), -1: no
  // place, -2: the row is in no sequence
  __shared__ int64_t place[APPEND_ROWS];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.b.T - row0));
  const int lane = threadIdx.x & 31, sub = lane & 15, warp = threadIdx.x >> 5;
  const int hw = threadIdx.x >> 4;
  // the slice's heads, and their first and end among q, k and v heads
  const int lo = blockIdx.y * a.slice, hi = min(lo + a.slice, a.H + 2 * a.Hkv);

  // heads h, h + STEP, .. of row r
  uint4 x[APPEND_BATCH];
  auto request = [&](int r, int h0) {
    const int64_t t = row0 + r;
    const uint4* q = reinterpret_cast<const uint4*>(a.q + t * a.ld_q) + sub;
    const uint4* k = reinterpret_cast<const uint4*>(a.k + t * a.ld_k) + sub - a.H * 16;
    const uint4* v = reinterpret_cast<const uint4*>(a.v + t * a.ld_v) + sub - (a.H + a.Hkv) * 16;
#pragma unroll
    for (int i = 0; i < APPEND_BATCH; ++i) {
      const int h = h0 + hw + i * APPEND_STEP;
      x[i] = make_uint4(0, 0, 0, 0);
      if (h < hi) x[i] = (h < a.H ? q : h < a.H + a.Hkv ? k : v)[h * 16];
    }
  };
  request(0, lo);

  if (warp < rows) {
    const int t = static_cast<int>(row0) + warp;
    const SeqRow s = find_row(a.b.cu_q, a.b.B, t);
    int64_t at = -2;
    if (s.b >= 0) {
      at = -1;
      const int64_t j = static_cast<int64_t>(__ldg(a.b.kv_len + s.b)) - s.q_len + s.i;
      if (j >= 0 && (j >> a.b.page_log2) < a.b.max_pages) {
        const int page = __ldg(a.b.page_table + static_cast<int64_t>(s.b) * a.b.max_pages +
                               (j >> a.b.page_log2));
        if (page >= 0 && page < a.b.num_pages)
          at = ((static_cast<int64_t>(page) * a.Hkv) << a.b.page_log2) +
               (j & ((1 << a.b.page_log2) - 1));
      }
    }
    if (lane == 0) place[warp] = at;
  }
  if (static_cast<int>(threadIdx.x) < rows * (DHP / 2)) {
    const int r = threadIdx.x / (DHP / 2), pr = threadIdx.x % (DHP / 2);
    float sn, cs;
    rope_angle(__ldg(a.pos + 3 * (row0 + r) + tab.axis[pr]), tab.turn[pr], sn, cs);
    turn[r][pr] = make_float2(cs, sn);
  }
  // (k_gain is there whenever q_gain is; asked for it alone, 58,758 split-half rows of
  // 126 heads take 762 us, not 754)
  const bool norm = a.k_gain != nullptr || a.q_gain != nullptr;
  float gq[8] = {}, gk[8] = {};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (a.q_gain != nullptr) gq[j] = __ldg(a.q_gain + sub * 8 + j);
    if (a.k_gain != nullptr) gk[j] = __ldg(a.k_gain + sub * 8 + j);
  }
  const int src_lane = (lane & 16) + (HALF ? tab.half_src[sub] : 0);
  const bool first = HALF ? tab.half_first[sub] != 0 : true;
  const int pair0 = HALF ? tab.half_pair0[sub] : sub * 4;
  __syncthreads();

  for (int r = 0; r < rows; ++r) {
    const int64_t at = place[r];
    const float2* cs = &turn[r][pair0];
    uint4* q = reinterpret_cast<uint4*>(a.q_out + (row0 + r) * a.H * DHP) + sub;
    // head h of the keys and values: (page * Hkv + h) * page_size + row in page
    const int64_t head = static_cast<int64_t>(16) << a.b.page_log2;
    uint4* k = reinterpret_cast<uint4*>(a.k_cache) + at * 16 + sub - a.H * head;
    uint4* v = reinterpret_cast<uint4*>(a.v_cache) + at * 16 + sub - (a.H + a.Hkv) * head;
    for (int h0 = lo; h0 < hi; h0 += APPEND_STEP * APPEND_BATCH) {
#pragma unroll
      for (int i = 0; i < APPEND_BATCH; ++i) {
        const int hb = h0 + (hw & ~1) + i * APPEND_STEP, h = hb + (hw & 1);
        if (hb >= hi) break;  // neither half-warp has one
        if (hb >= a.H + a.Hkv) {  // values, for both
          if (h < hi && at >= 0) v[h * head] = x[i];
          continue;
        }
        float g[8];
        const bool is_q = h < a.H;
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = is_q ? gq[j] : gk[j];
        const uint4 y = norm_turn<HALF>(x[i], norm, g, a.eps, cs, first, src_lane);
        if (is_q) {
          if (at != -2) q[h * 16] = y;
        } else if (h < hi && at >= 0) {
          if (h < a.H + a.Hkv)
            k[h * head] = y;
          else
            v[h * head] = x[i];
        }
      }
      if (h0 + APPEND_STEP * APPEND_BATCH < hi)
        request(r, h0 + APPEND_STEP * APPEND_BATCH);
      else if (r + 1 < rows)
        request(r + 1, lo);
    }
  }
}

}  // namespace

h3_status launch_kv_append(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                           int64_t ld_v, void* q_out, int H, const float* q_gain,
                           const float* k_gain, const int32_t* pos, const int* axis_dims,
                           int pairing, float theta, float eps, void* k_cache, void* v_cache,
                           int Hkv, const PagedBatch& batch, cudaStream_t s) {
  AppendArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.ld_q = ld_q;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.pos = pos;
  a.eps = eps;
  a.H = H;
  a.Hkv = Hkv;
  a.b = batch;
  // the table of 64 powers takes longer to form than the launch; it depends on
  // these four numbers alone, which a model never changes
  thread_local RopeTable tab;
  thread_local int tab_axis[3] = {0, 0, 0};
  thread_local float tab_theta = 0.f;
  if (tab_theta != theta || !std::equal(axis_dims, axis_dims + 3, tab_axis)) {
    tab = rope_table(axis_dims, theta);
    std::copy(axis_dims, axis_dims + 3, tab_axis);
    tab_theta = theta;
  }
  // several rows per CTA once every SM has 16 CTAs of them (2,600 rows of 42 + 84 heads:
  // one row 38 us, two 44; 58,758: 667, 642); the heads of few rows are spread over two
  // CTAs per SM
  const int heads = H + 2 * Hkv, sms = num_sms();
  a.rows = batch.T >= 16 * APPEND_ROWS * sms ? APPEND_ROWS : 1;
  const int slices = std::min(std::max(2 * sms / batch.T, 1), (heads + APPEND_STEP - 1) / APPEND_STEP);
  a.slice = (heads + slices - 1) / slices;
  a.slice = (a.slice + APPEND_STEP - 1) / APPEND_STEP * APPEND_STEP;
  const dim3 blocks((batch.T + a.rows - 1) / a.rows, (heads + a.slice - 1) / a.slice);
  if (pairing == 1)
    kv_append_kernel<true><<<blocks, APPEND_THREADS, 0, s>>>(a, tab);
  else
    kv_append_kernel<false><<<blocks, APPEND_THREADS, 0, s>>>(a, tab);
  return cuda_fail(cudaGetLastError(), "kv_append_paged launch");
}

}  // namespace h3
