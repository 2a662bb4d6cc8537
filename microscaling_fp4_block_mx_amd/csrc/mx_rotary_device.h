// mx_rotary_device.h - what the kernels of the heads' norms and rotations share:
// sums over the lanes of a head in 64 bits, the root, cosines and sines.
#ifndef MX_ROTARY_DEVICE_H
#define MX_ROTARY_DEVICE_H
#include "mx_layer_device.h"

namespace mxl {

template <int CTRL>
__device__ __forceinline__ double dppd(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = dpp<CTRL>((uint32_t)b), hi = dpp<CTRL>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, hi << 32 | lo);
}
// Sum over L = 4, 8 or 16 neighbouring lanes, the same bits on each of them
// (quad_perm, then mirrors of 8 and of 16 lanes: a quad's lanes agree by then).
template <int L>
__device__ __forceinline__ double sum_lanes(double v) {
  v += dppd<0xB1>(v);
  v += dppd<0x4E>(v);
  if constexpr (L >= 8) v += dppd<0x141>(v);
  if constexpr (L >= 16) v += dppd<0x140>(v);
  return v;
}

// 1 / sqrt(x) to the last bits of 64 (two steps of Newton's on the hardware's
// estimate); 0 of infinity, NaN of 0 and of NaN.
__device__ __forceinline__ double inverse_root(double x) {
  double r = __builtin_amdgcn_rsq(x);
  const double h = 0.5 * x;
  r = __builtin_fma(r, __builtin_fma(-h * r, r, 0.5), r);
  r = __builtin_fma(r, __builtin_fma(-h * r, r, 0.5), r);
  return x == __builtin_inf() ? 0.0 : r;
}

// Eight floats from p, 16-byte aligned.
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
  const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    f[j] = a[j];
    f[4 + j] = b[j];
  }
}

// The row of the table that a position has, and whether it has one (row 0, if
// not: nothing outside the table is read).
struct Angles {
  const float *row;
  bool none;
};
__device__ __forceinline__ Angles angles_of(const float *table, int64_t length, int rot, int position) {
  const bool none = position < 0 || position >= length;
  return Angles{table + (none ? 0 : (int64_t)position * rot), none};
}

}  // namespace mxl
#endif  // MX_ROTARY_DEVICE_H
