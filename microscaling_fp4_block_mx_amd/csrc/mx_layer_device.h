// mx_layer_device.h - device helpers of the transformer-layer kernels: wide
// loads of eight elements, cross-lane sums and maxima, E4M3 encoding.
#ifndef MX_LAYER_DEVICE_H
#define MX_LAYER_DEVICE_H
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxl {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---- cross-lane ---------------------------------------------------------------
// DPP controls: quad_perm 1,0,3,2 / 2,3,0,1 (lane^1, lane^2), row_ror 4 / 8
// (rotation inside 16 lanes). Rows of 16 are whole wherever these are used.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
__device__ __forceinline__ uint32_t max4(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  return max(v, dpp<0x4E>(v));
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max4(v);
  v = max(v, dpp<0x124>(v));
  return max(v, dpp<0x128>(v));
}
__device__ __forceinline__ float sum16(float v) {
  v += dppf<0xB1>(v);
  v += dppf<0x4E>(v);
  v += dppf<0x124>(v);
  return v + dppf<0x128>(v);
}
// Sum over the wave, the same bits on every lane.
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// ---- eight elements --------------------------------------------------------------
template <bool BF16>
struct Raw {
  u32x4 v[BF16 ? 1 : 2];
};
// To the compiler another value from here on: what it made of the old one is
// not kept in registers for later.
template <bool BF16>
__device__ __forceinline__ void renew(Raw<BF16> &r) {
  asm("" : "+v"(r.v[0]));
  if constexpr (!BF16) asm("" : "+v"(r.v[1]));
}
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void *base, int64_t item) {
  Raw<BF16> r;
  if constexpr (BF16) {
    r.v[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(base) + item);
  } else {
    r.v[0] = reinterpret_cast<const u32x4 *>(base)[2 * item];
    r.v[1] = reinterpret_cast<const u32x4 *>(base)[2 * item + 1];
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ void widen(const Raw<BF16> &r, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) {
    if constexpr (BF16) {
      const uint32_t w = r.v[0][j >> 1];
      f[j] = __uint_as_float((j & 1) ? (w & 0xFFFF0000u) : (w << 16));
    } else {
      f[j] = __uint_as_float(r.v[j >> 2][j & 3]);
    }
  }
}
// bf16 nearest-even of a and b in one word (a low).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}
template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t item, const float (&f)[8]) {
  if constexpr (BF16) {
    const u32x4 w = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                     pack_bf16(f[6], f[7])};
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(base) + item);
  } else {
    f32x4 *p = reinterpret_cast<f32x4 *>(base) + 2 * item;
    p[0] = f32x4{f[0], f[1], f[2], f[3]};
    p[1] = f32x4{f[4], f[5], f[6], f[7]};
  }
}

// One element.
template <bool BF16>
__device__ __forceinline__ float load_one(const void *base, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(base)[i] << 16);
  else return reinterpret_cast<const float *>(base)[i];
}

// ---- E4M3 -------------------------------------------------------------------------
// Scale byte of a block whose largest |x| has these fp32 bits: floor(log2) - 8
// + 127, clamped at 0; 255 for NaN or infinity.
__device__ __forceinline__ uint32_t scale_byte8(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const uint32_t e = amax_bits >> 23;
  return e > 8u ? e - 8u : 0u;
}
__device__ __forceinline__ uint32_t amax8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  return m;
}
// 448 at scale byte s, where 32 bits hold it (s <= 246, as of finite numbers).
__device__ __forceinline__ float limit8(uint32_t s) {
  return __uint_as_float(((s + 8u) << 23) | 0x600000u);
}
// Eight codes at scale byte s: nearest, ties to even, saturating at 448
// (clamped to `lim` first: the convert turns larger values into NaN); in a
// block with s = 255 the sign bits alone.
__device__ __forceinline__ u32x2 encode8(const float (&f)[8], uint32_t s, float lim) {
  if (__builtin_expect(s == 255u, 0)) {
    uint32_t b[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++) b[j >> 2] |= (__float_as_uint(f[j]) >> 31) << (8 * (j & 3) + 7);
    return u32x2{b[0], b[1]};
  }
  const float sc = __uint_as_float(s << 23);
  float c[8];
#pragma unroll
  for (int j = 0; j < 8; j++) c[j] = __builtin_amdgcn_fmed3f(f[j], -lim, lim);
  s16x2 a = {0, 0}, b = {0, 0};
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[0], c[1], sc, false);
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[2], c[3], sc, true);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[4], c[5], sc, false);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[6], c[7], sc, true);
  return u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}
__device__ __forceinline__ u32x2 encode8(const float (&f)[8], uint32_t s) {
  return encode8(f, s, limit8(s));
}

}  // namespace mxl
#endif  // MX_LAYER_DEVICE_H
