// Host-side declarations shared by the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/h3block.h"
#include "h3_ptx.cuh"

namespace h3 {

// ---- error state (h3_abi.cu)
h3_status fail(h3_status s, const char* fmt, ...);
h3_status cuda_fail(cudaError_t e, const char* what);
void clear_error();
// Device error word and wait limit for kernels launched on the current device.
h3_status dev_err(DevErr* out);
int num_sms();

// Raises `kernel`'s dynamic shared-memory limit to `bytes` on the current
// device, once per device (done[] holds the devices already set; ordinals
// past its end are set on every call). Safe to call from several threads:
// the attribute call is idempotent and the flags are atomic.
template <typename Kernel>
h3_status set_smem_limit(std::atomic<bool> (&done)[64], Kernel kernel, size_t bytes,
                         const char* what) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, what);
  if (dev < 64 && done[dev].load(std::memory_order_acquire)) return H3_OK;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e != cudaSuccess) return cuda_fail(e, what);
  if (dev < 64) done[dev].store(true, std::memory_order_release);
  return H3_OK;
}

// ---- TMA descriptors (h3_abi.cu). A 2D bf16 tensor of `outer` rows x `inner`
// elements with the given row stride, boxes of box_inner x box_outer, 128-byte
// swizzle, zero fill outside the tensor.
h3_status make_tmap_bf16_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                            uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer);
// Same for a tensor of bytes (FP8 codes).
h3_status make_tmap_u8_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                          uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer);

// Same for a tensor of float32.
h3_status make_tmap_f32_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                           uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer);

// `outer` contiguous rows of `inner` 32-bit words (at most 256), boxes of box_outer whole
// rows, no swizzle, zero fill past the last row.
h3_status make_tmap_u32_rows(CUtensorMap* m, const void* base, uint32_t inner, uint64_t outer,
                             uint32_t box_outer);

// A 3D bf16 tensor [d2, d1, d0] with row strides s1 and s2 in bytes, boxes of
// b2 x b1 x b0, otherwise the same.
h3_status make_tmap_bf16_3d(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1,
                            uint64_t d2, uint64_t s1, uint64_t s2, uint32_t b0, uint32_t b1,
                            uint32_t b2);

// ---- kernel launchers (arguments already validated)
h3_status launch_swiglu(const void* gate_up, void* out, int L, int F, cudaStream_t s);
// pairing: 0 interleaved pairs (2j, 2j + 1), 1 split-half pairs
// (o + j, o + d/2 + j) per section (every section a multiple of 16 wide).
h3_status launch_qk_norm_rope(void* q, void* k, int64_t row_stride, const float* q_gain,
                              const float* k_gain, const int32_t* pos, const int* axis_dims,
                              int L, int H, float theta, float eps, cudaStream_t s,
                              int pairing = 0);
// The RoPE (cos, sin) table of rows [0, L) (see launch_rope_table), written
// by the modulation kernel beside its own work when requested.
struct RopeRequest {
  const int32_t* pos;    // [L, 3] positions
  const int* axis_dims;  // host [3]
  float theta;
  float2* out;           // [L, 64]
};
// seg (optional): per-row token-group index into a table whose groups are
// seg_stride floats apart (gate/shift/scale point at group 0).
// codes (optional): write the normalised row as per-row E4M3 codes [L, D]
// and scales code_scale [L] (launch_quantize_fp8_rows of the bf16 row)
// instead of the bf16 row `normed`.
h3_status launch_mod_norm_residual(float* resid, const void* delta, const float* gate,
                                   const float* shift, const float* scale, void* normed, int L,
                                   int D, float eps, cudaStream_t s, const int32_t* seg = nullptr,
                                   int num_seg = 1, int64_t seg_stride = 0,
                                   const RopeRequest* rope = nullptr, uint8_t* codes = nullptr,
                                   float* code_scale = nullptr);

// Norms before and after a branch (h3_norms.cu); see h3_sandwich_norm.
h3_status launch_sandwich_norm(const float* resid, const void* delta, float* resid_out,
                               void* normed, bool post_norm, const float* post_gain,
                               const float* gate, float resid_scale, const float* pre_gain,
                               const float* shift, const float* scale, const int32_t* seg,
                               int num_seg, int64_t seg_stride, bool rms, int L, int D, float eps,
                               cudaStream_t s);

// (cos, sin) of every RoPE angle of rows [0, L): out[i * 64 + p] for channel
// pair p of a 128-channel head, the angle formed and reduced exactly as
// launch_qk_norm_rope does.
h3_status launch_rope_table(const int32_t* pos, const int* axis_dims, int L, float theta,
                            float2* out, cudaStream_t s);

// frames [B, C, N] float32 (N = T*H*W, N % 4 == 0) -> [B, N, C] uint8.
h3_status launch_frames_to_u8(const float* in, uint8_t* out, int B, int C, int64_t N,
                              cudaStream_t s);

enum GemmEpilogue : int {
  GEMM_STORE_BF16 = 0,     // C = bf16(acc)
  GEMM_SWIGLU = 1,         // B rows [gate | up] of F each; C[:, j] = SiLU(g) * u, width F
  GEMM_RESIDUAL = 2,       // C is the FP32 residual: C[:, j] += gate[j] * bf16(acc)
  GEMM_QK_NORM_ROPE = 3,   // C = bf16(acc), then RMSNorm + RoPE on the q and k heads
};
// Operands of the fused epilogues (unused fields may stay zero).
struct GemmExtra {
  // GEMM_RESIDUAL: per-column gate [N]; with seg, row i reads the gate at
  // gate + clamp(seg[i], 0, num_seg - 1) * seg_stride.
  const float* gate = nullptr;
  const int32_t* seg = nullptr;
  int num_seg = 1;
  int64_t seg_stride = 0;
  // GEMM_QK_NORM_ROPE: columns [0, d_model) are q heads, [d_model, 2 d_model)
  // k heads (128 channels each), the rest pass through; every head of a row is
  // rounded to bf16, scaled by 1/rms and its gain, rotated by the row's
  // (cos, sin) table [L, 64] (h3::launch_rope_table) and rounded again.
  const float* q_gain = nullptr;
  const float* k_gain = nullptr;
  const float2* rope = nullptr;
  int d_model = 0;
  float eps = 0.f;
  // split-half RoPE pairs (pairing 1): eight pieces of eight pairs, piece i
  // rotating columns piece_first[i] + j with piece_second[i] + j by table
  // entry piece_pair[i] + j (set by rope_pieces)
  int pairing = 0;
  int piece_first[8] = {};
  int piece_second[8] = {};
  int piece_pair[8] = {};
};
// Fills ex's split-half pieces for the RoPE sections axis_dims (each a
// multiple of 16, summing to 128) and sets ex->pairing = 1.
void rope_pieces(const int* axis_dims, GemmExtra* ex);
// C[:L, :] = epilogue(A[:L, :K] @ B^T). A row stride lda, B [N, K] row stride
// ldb, C row stride ldc (elements of C). For GEMM_SWIGLU, N is the width of C
// (= F) and B holds 2N rows.
h3_status launch_gemm(const void* A, int64_t lda, const void* B, int64_t ldb, void* C,
                      int64_t ldc, int L, int N, int K, GemmEpilogue ep, cudaStream_t s,
                      const GemmExtra* extra = nullptr);

// FP8 (E4M3) operands with per-row scales: C[:L] = epilogue(bf16-free
// (A @ B^T) * sa[row] * sb[col]). A [L, K] codes (row stride lda bytes), B
// [N or 2N, K] codes (row stride ldb bytes), sa [L], sb [N or 2N].
h3_status launch_gemm_fp8(const void* A, int64_t lda, const float* sa, const void* B, int64_t ldb,
                          const float* sb, void* C, int64_t ldc, int L, int N, int K,
                          GemmEpilogue ep, cudaStream_t s, const GemmExtra* extra = nullptr);
// Per-row absmax quantisation of bf16 x [R, K] (row stride ldx elements) to
// E4M3 codes q [R, K] (row stride ldq bytes) and float32 scales [R].
h3_status launch_quantize_fp8_rows(const void* x, int64_t ldx, void* q, int64_t ldq, float* scale,
                                   int R, int K, cudaStream_t s);

// o[:L] = attention(q, k, v); q/k/v rows of stride ld_in elements, o of ld_out.
// skip_eps < 0: dense attention (the CTA-pair kernel). skip_eps >= 0:
// Skip-Softmax (the pair kernel's instance with its vote), a key tile is left out for
// a query tile when every valid row's tile maximum is below eps times the
// row's exact running maximum over the kept tiles (eps = 0 never skips); kept
// (optional, [ceil(L/128), H]) receives the number of key tiles kept per
// (query tile, head).
h3_status launch_attention(const void* q, const void* k, const void* v, int64_t ld_in,
                           void* o, int64_t ld_out, int L, int H, float scale, cudaStream_t s,
                           float skip_eps = -1.f, int* kept = nullptr);

// SAGE-style FP8 attention: operands (h3_sage.cu) and the FP8 attention
// kernel (h3_attention.cu). Codes [L, H*128] bytes with row stride ldc; sq,
// sk [ceil(L/128), H]; sv, k_mean [H, 128]; scratch of sage_scratch_bytes.
size_t sage_scratch_bytes(int L, int H);
h3_status launch_sage_quantize(const void* q, const void* k, const void* v, int64_t ld, int L,
                               int H, uint8_t* qc, uint8_t* kc, uint8_t* vc, int64_t ldc,
                               float* sq, float* sk, float* sv, float* k_mean, void* scratch,
                               cudaStream_t s);
// skip_eps >= 0: Skip-Softmax on the FP8 logits (kept tile counts to `kept`
// [ceil(L/128), H] when not null), as in launch_attention.
h3_status launch_attention_fp8(const void* qc, const void* kc, const void* vc, int64_t ld_codes,
                               const float* sq, const float* sk, const float* sv, void* o,
                               int64_t ld_out, int L, int H, float scale, cudaStream_t s,
                               float skip_eps = -1.f, int* kept = nullptr);

// ---- paged key/value cache (h3_paged.cu, h3_paged_attention.cu)
// Rows and pages of one call (device arrays; see h3_kv_batch).
struct PagedBatch {
  int T, B;
  int max_pages;
  int num_pages, page_log2;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* page_table;
};
#ifdef __CUDACC__
// A partial result of a row is (maximum, sum, O). A maximum of -inf says that the
// row has seen no key, and nothing else does: of rows whose scores are all NaN
// (which a maximum drops) or all -inf it is this, the least float. Their sums (NaN,
// 0) then go through the joins with weights like any other's, and the row has no
// value, NaN, however its keys were split.
constexpr float KEYS_SEEN = -3.402823466e+38f;

// The number of sequence ends cu_q[1..B] at or below row t, by a whole warp: 32
// of them at a time, so three reads for any B up to 32,768. Arrays that are out
// of order give some number in [0, B].
__device__ __forceinline__ int ends_up_to(const int32_t* cu_q, int B, int t) {
  int at = 0, n = B;  // the answer is in [at, at + n]
  while (n > 0) {
    const int step = (n + 31) >> 5;
    const int i = (static_cast<int>(threadIdx.x & 31) + 1) * step;  // the i-th end from at on
    const uint32_t below = __ballot_sync(0xffffffffu, i <= n && __ldg(cu_q + at + min(i, n)) <= t);
    const int skip = __popc(below) * step;
    at += skip;
    n = min(step - 1, n - skip);
  }
  return at;
}
#endif
// q (optional, with q_out), k, v: rows of ld elements; pairing as
// launch_qk_norm_rope; gains NULL: rotation only.
h3_status launch_kv_append(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                           int64_t ld_v, void* q_out, int H, const float* q_gain,
                           const float* k_gain, const int32_t* pos, const int* axis_dims,
                           int pairing, float theta, float eps, void* k_cache, void* v_cache,
                           int Hkv, const PagedBatch& batch, cudaStream_t s);
// prefix_len keys in prefix_pages (or 0) come before every sequence's own.
size_t paged_workspace_bytes(int T, int H, int prefix_len);
h3_status launch_paged_attention(const void* q, int64_t ld_q, void* o, int64_t ld_o, int H,
                                 float scale, bool causal, const void* k_cache,
                                 const void* v_cache, int Hkv, const PagedBatch& batch,
                                 const int32_t* prefix_pages, int prefix_len, void* workspace,
                                 cudaStream_t s);
// The same for single rows over at most so many keys (h3_paged_rows.cu), where
// paged_rows_fit; no workspace. With part_o and part_ml, sums and (maximum, sum) of
// every row and head go there instead of the output.
bool paged_rows_fit(int T, int H, int Hkv, int B, int64_t keys, int prefix_len);
h3_status launch_paged_rows(const void* q, int64_t ld_q, void* o, int64_t ld_o, int H, float scale,
                            bool causal, const void* k_cache, const void* v_cache, int Hkv,
                            const PagedBatch& batch, const int32_t* prefix_pages, int prefix_len,
                            float* part_o, float* part_ml, cudaStream_t s);

}  // namespace h3
