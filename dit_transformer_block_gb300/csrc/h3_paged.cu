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

// The sequence of row t: the number of ends cu_q[1..B] at or below t, counted
// by the whole warp.
__device__ __forceinline__ SeqRow find_row(const int32_t* __restrict__ cu_q, int B, int t) {
  int n = 0;
  for (int i = threadIdx.x & 31; i < B; i += 32) n += __ldg(cu_q + i + 1) <= t ? 1 : 0;
  n = __reduce_add_sync(0xffffffffu, n);
  SeqRow r{-1, 0, 0};
  if (n < B) {
    const int first = __ldg(cu_q + n), end = __ldg(cu_q + n + 1);
    if (first >= 0 && first <= t && t < end) r = {n, t - first, end - first};
  }
  return r;
}

// ------------------------------------------------------------------ append
// A warp takes 2 U heads of one row (lanes 0-15 and 16-31 one head each, 8
// channels per lane, as in the in-place Q/K kernel) from the row's list of H
// query, Hkv key and Hkv value heads.
constexpr int APPEND_WARPS = 8;

struct AppendArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t ld_q, ld_k, ld_v;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  const float* q_gain;  // NULL: no norm
  const float* k_gain;
  const int32_t* pos;
  float eps;
  int H, Hkv;
  int units;  // warps per row
  PagedBatch b;
};

template <bool HALF, int U>
__global__ void __launch_bounds__(APPEND_WARPS * 32)
    kv_append_kernel(const AppendArgs a, const RopeTable tab) {
  const int64_t w = blockIdx.x * static_cast<int64_t>(APPEND_WARPS) + (threadIdx.x >> 5);
  const int64_t row64 = w / a.units;
  if (row64 >= a.b.T) return;
  const int row = static_cast<int>(row64);
  const int h0 = static_cast<int>(w - row64 * a.units) * 2 * U;
  const int lane = threadIdx.x & 31, sub = lane & 15, half = lane >> 4;
  const int heads = a.H + 2 * a.Hkv;

  // the heads are requested first, the row's place and angles found meanwhile
  uint4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + 2 * u + half;
    x[u] = make_uint4(0, 0, 0, 0);
    if (h < heads) {
      const __nv_bfloat16* src =
          h < a.H ? a.q + row * a.ld_q + h * DHP
                  : (h < a.H + a.Hkv ? a.k + row * a.ld_k + (h - a.H) * DHP
                                     : a.v + row * a.ld_v + (h - a.H - a.Hkv) * DHP);
      x[u] = *reinterpret_cast<const uint4*>(src + sub * 8);
    }
  }
  const SeqRow s = find_row(a.b.cu_q, a.b.B, row);
  if (s.b < 0) return;
  // cache row of the row's key: page * Hkv * page_size + row in page (for head 0), or -1
  int64_t key_row = -1;
  {
    const int64_t j = static_cast<int64_t>(__ldg(a.b.kv_len + s.b)) - s.q_len + s.i;
    if (j >= 0 && (j >> a.b.page_log2) < a.b.max_pages) {
      const int page = __ldg(a.b.page_table + static_cast<int64_t>(s.b) * a.b.max_pages +
                             (j >> a.b.page_log2));
      if (page >= 0 && page < a.b.num_pages)
        key_row = ((static_cast<int64_t>(page) * a.Hkv) << a.b.page_log2) +
                  (j & ((1 << a.b.page_log2) - 1));
    }
  }

  const int32_t p3[3] = {__ldg(a.pos + 3LL * row), __ldg(a.pos + 3LL * row + 1),
                         __ldg(a.pos + 3LL * row + 2)};
  constexpr int NP = HALF ? 8 : 4;
  float cs[NP], sn[NP], c4[4], s4[4];
  const int src_lane = (half << 4) + (HALF ? tab.half_src[sub] : 0);
  const bool first = HALF ? tab.half_first[sub] != 0 : true;
  const int pair0 = (HALF ? tab.half_pair0[sub] : sub * 4) + (first ? 0 : 4);
#pragma unroll
  for (int t = 0; t < 4; ++t) rope_angle(p3[tab.axis[pair0 + t]], tab.turn[pair0 + t], s4[t], c4[t]);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if constexpr (HALF) {
      const float oc = __shfl_sync(0xffffffffu, c4[t], src_lane);
      const float os = __shfl_sync(0xffffffffu, s4[t], src_lane);
      cs[t] = first ? c4[t] : oc;
      sn[t] = first ? s4[t] : os;
      cs[4 + t] = first ? oc : c4[t];
      sn[4 + t] = first ? os : s4[t];
    } else {
      cs[t] = c4[t];
      sn[t] = s4[t];
    }
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (h0 + 2 * u >= heads) break;  // uniform across the warp
    const int h = h0 + 2 * u + half;
    const uint32_t wd[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(wd[j]);
      f[2 * j + 1] = bf16_hi(wd[j]);
    }
    if (a.k_gain != nullptr || a.q_gain != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
      for (int m = 8; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float inv = rsqrtf(ss * (1.0f / DHP) + a.eps);
      const float4* gp = reinterpret_cast<const float4*>((h < a.H ? a.q_gain : a.k_gain) + sub * 8);
      const float4 g0 = __ldg(gp), g1 = __ldg(gp + 1);
      const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * inv * g[j];
    }
    uint32_t o[4];
    if constexpr (HALF) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = __shfl_sync(0xffffffffu, f[j], src_lane);  // the pair's other element
        y[j] = first ? f[j] * cs[j] - p * sn[j] : p * sn[j] + f[j] * cs[j];
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] = pack_bf16x2(y[2 * t], y[2 * t + 1]);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        o[t] = pack_bf16x2(f[2 * t] * cs[t] - f[2 * t + 1] * sn[t],
                           f[2 * t] * sn[t] + f[2 * t + 1] * cs[t]);
    }
    if (h < a.H) {
      *reinterpret_cast<uint4*>(a.q_out + (static_cast<int64_t>(row) * a.H + h) * DHP + sub * 8) =
          make_uint4(o[0], o[1], o[2], o[3]);
    } else if (h < heads && key_row >= 0) {
      const bool is_k = h < a.H + a.Hkv;
      const int hk = h - a.H - (is_k ? 0 : a.Hkv);
      __nv_bfloat16* dst = (is_k ? a.k_cache : a.v_cache) +
                           (key_row + (static_cast<int64_t>(hk) << a.b.page_log2)) * DHP + sub * 8;
      *reinterpret_cast<uint4*>(dst) = is_k ? make_uint4(o[0], o[1], o[2], o[3]) : x[u];
    }
  }
}

}  // namespace

h3_status launch_kv_append(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                           int64_t ld_v, void* q_out, int H, const float* q_gain,
                           const float* k_gain, const int32_t* pos, const int* axis_dims,
                           int pairing, float theta, float eps, void* k_cache, void* v_cache,
                           int Hkv, const PagedBatch& batch, cudaStream_t s) {
  constexpr int U = 4;
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
  a.units = (H + 2 * Hkv + 2 * U - 1) / (2 * U);
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
  const int64_t blocks =
      (static_cast<int64_t>(batch.T) * a.units + APPEND_WARPS - 1) / APPEND_WARPS;
  if (blocks > 0x7fffffff)
    return fail(H3_ERR_UNSUPPORTED, "kv_append_paged: T=%d rows of %d heads are too many", batch.T,
                H + 2 * Hkv);
  if (pairing == 1)
    kv_append_kernel<true, U><<<static_cast<int>(blocks), APPEND_WARPS * 32, 0, s>>>(a, tab);
  else
    kv_append_kernel<false, U><<<static_cast<int>(blocks), APPEND_WARPS * 32, 0, s>>>(a, tab);
  return cuda_fail(cudaGetLastError(), "kv_append_paged launch");
}

}  // namespace h3
