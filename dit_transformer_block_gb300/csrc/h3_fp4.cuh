// Declarations of the 4-bit rows and their products (h3_fp4.cu, h3_fp4_gemm.cu).
#pragma once
#include "h3_internal.cuh"

namespace h3 {

// A row of NV values whose largest is below this has scales of 0: 2688 / amax stays finite.
constexpr float FP4_LEAST_ROW = 7.888609052210118e-31f;  // 2^-100

// Tiles of 128 rows x 4 scales along a row.
inline int fp4_tiles(int K, bool nv) { return nv ? (K + 63) / 64 : (K + 127) / 128; }

h3_status launch_quantize_fp4_rows(const void* x, int64_t ldx, void* codes, void* scales,
                                   float* row_scale, int R, int K, bool nv, cudaStream_t s);
// One operand: codes [rows, K / 2], scales in tiles, row scales (NV only).
struct Fp4Operand {
  const void* codes;
  const void* scales;
  const float* row_scale;
};
// C[:L, :N] = bf16 of A B^T, or with swiglu SiLU(A Bg^T) * (A Bu^T) of B = [2 N, K], rows [gate | up].
h3_status launch_gemm_fp4(const Fp4Operand& a, const Fp4Operand& b, void* C, int L, int N, int K,
                          bool nv, bool swiglu, cudaStream_t s);

}  // namespace h3
