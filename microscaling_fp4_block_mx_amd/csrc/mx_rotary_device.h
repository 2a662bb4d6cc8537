// mx_rotary_device.h - what the kernels of the heads' norms and rotations share:
// sums over the lanes of a head in 64 bits, the root, cosines and sines.
#ifndef MX_ROTARY_DEVICE_H
#define MX_ROTARY_DEVICE_H
#include "mx.h"
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

// Items A and B (of eight dims) of lane t of a head, and whether they turn.
// PAIRED: neighbours; else A and the item half of the rotated dims further on,
// and neighbours behind the rotated dims. Either way the lane's eight pairs
// are pairs 8 t .. 8 t + 7.
template <bool PAIRED>
__device__ __forceinline__ void items_of(int t, int rot, int &a, int &b, bool &turns) {
  turns = 16 * t < rot;
  const int half = rot >> 4;
  a = !PAIRED && turns ? t : 2 * t;
  b = !PAIRED && turns ? t + half : 2 * t + 1;
}

// Turns a lane's pairs, or back.
template <bool PAIRED, bool BACK>
__device__ __forceinline__ void turn(double (&a)[8], double (&b)[8], const float (&c)[8], const float (&s)[8]) {
  auto pair = [&](double &x, double &y, int e) {
    const double cd = c[e], sd = BACK ? -s[e] : s[e], x0 = x;
    x = __builtin_fma(x0, cd, -(y * sd));
    y = __builtin_fma(y, cd, x0 * sd);
  };
#pragma unroll
  for (int e = 0; e < 8; e++) {
    if constexpr (!PAIRED) pair(a[e], b[e], e);
    else if (e < 4) pair(a[2 * e], a[2 * e + 1], e);
    else pair(b[2 * e - 8], b[2 * e - 7], e);
  }
}

template <bool BF16>
__device__ __forceinline__ void widen64(const Raw<BF16> &r, double (&d)[8]) {
  float f[8];
  widen<BF16>(r, f);
#pragma unroll
  for (int j = 0; j < 8; j++) d[j] = f[j];
}
// Weights stay in the caches: default policy.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_weight(const void *w, int item) {
  const u32x4 *p = reinterpret_cast<const u32x4 *>(w) + (BF16 ? 1 : 2) * item;
  Raw<BF16> r;
  r.v[0] = p[0];
  if constexpr (!BF16) r.v[1] = p[1];
  return r;
}

// Cosines and sines of a lane's pairs; NaN cosines where a position has none.
struct Turns {
  float c[8], s[8];
  __device__ __forceinline__ void load(const mx_rotary_t &r, int position, int t) {
    const Angles at = angles_of(r.table, r.length, r.rot, position);
    load8(at.row + 8 * t, c);
    load8(at.row + (r.rot >> 1) + 8 * t, s);
    if (at.none) {
#pragma unroll
      for (int j = 0; j < 8; j++) c[j] = __builtin_nanf("");
    }
  }
};

}  // namespace mxl
#endif  // MX_ROTARY_DEVICE_H
