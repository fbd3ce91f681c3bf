// Rotary position embedding of 128-channel heads: the per-pair table the
// kernels take and the device angle, shared by every kernel that rotates heads.
#pragma once
#include <cmath>
#include <cstdint>

namespace h3 {

constexpr int QK_HEAD_DIM = 128;

struct RopeTable {
  // turns per unit position of each pair, omega / (2 pi) in 0.64 fixed point
  // (omega / (2 pi) rounded to double, then scaled exactly by 2^64)
  uint64_t turn[QK_HEAD_DIM / 2];
  int axis[QK_HEAD_DIM / 2];      // which position (t, h, w) drives the pair
  // split-half layout, per 8-channel slice s of a head: the slice holding the
  // partners, whether s holds first elements, and the pair of its channel 0
  int half_src[QK_HEAD_DIM / 8];
  int half_first[QK_HEAD_DIM / 8];
  int half_pair0[QK_HEAD_DIM / 8];
};

// Angle of a pair at position p: its turns p * omega / (2 pi) modulo 1, exact
// in 64-bit fixed point (the integer product wraps modulo 2^64, i.e. whole
// turns), read as a signed fraction t of a half turn in [-1, 1) (one rounding
// to float32), then sin and cos of pi * t in FP32. No FP64 arithmetic, whose
// rate on this GPU is a small fraction of FP32's.
__device__ __forceinline__ void rope_angle(int32_t p, uint64_t turn, float& sn, float& cs) {
  const uint64_t f = static_cast<uint64_t>(static_cast<int64_t>(p)) * turn;
  const float t = __ll2float_rn(static_cast<int64_t>(f)) * 0x1p-63f;
  sincospif(t, &sn, &cs);
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

inline RopeTable rope_table(const int* axis_dims, float theta) {
  RopeTable tab{};
  int pr = 0;
  int o = 0;  // first channel of section a
  for (int a = 0; a < 3; ++a) {
    const int d = axis_dims[a];
    for (int j = 0; j < d / 2; ++j, ++pr) {
      const double omega =
          std::pow(static_cast<double>(theta), -2.0 * j / static_cast<double>(d));
      // omega / (2 pi) < 1: scaled by 2^64 it is an integer below 2^63 with
      // at most 53 significant bits, which the conversion keeps exactly
      tab.turn[pr] = static_cast<uint64_t>(std::ldexp(omega / kTwoPi, 64));
      tab.axis[pr] = a;
    }
    // split-half slices (meaningful when d % 16 == 0): slice s of the first
    // half pairs with slice s + d/16 of the second half
    for (int c = 0; c + 8 <= d; c += 8) {
      const int s = (o + c) / 8;
      const bool fst = c < d / 2;
      tab.half_first[s] = fst ? 1 : 0;
      tab.half_src[s] = fst ? s + d / 16 : s - d / 16;
      tab.half_pair0[s] = o / 2 + (fst ? c : c - d / 2);
    }
    o += d;
  }
  return tab;
}

}  // namespace h3
