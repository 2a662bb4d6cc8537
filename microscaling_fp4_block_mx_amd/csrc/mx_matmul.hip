// mx_matmul.hip - product of two MXFP8 matrices on the matrix cores:
//   C[m][n] = sum_k A[m][k] 2^(sa-127) B[n][k] 2^(sb-127)
// A [M, K] and B [N, K] are E4M3 codes, row-major, with one E8M0 byte per 32
// or 128 elements of a row. K is a multiple of 32; M and N are any.
//
// bf16 output runs the scaled 8-bit matrix products, which multiply codes and
// apply the E8M0 bytes themselves. Lane layouts (checked on the card): in
// v_mfma_scale_f32_16x16x128_f8f6f4 lane l holds row l % 16; with g = l / 16
// its first 16 bytes are k = 16 g .. 16 g + 15 and its second 16 bytes are
// k = 64 + 16 g ..; the scale byte that lane l supplies belongs to row l % 16
// and elements k = 32 g .. 32 g + 31. Inside each group of eight products the
// matrix core drops bits more than about 2^-14 below the largest product
// (1.4e-5 of the result's norm on normal data), which is far inside bf16's
// rounding (1.7e-3) but not inside fp32's. fp32 output therefore widens the
// codes to bf16, scales applied, and runs the bf16 products at half the rate.
// That is exact for bytes 3 to 246; below, subnormal codes lose what lies under
// 2^-133; where a wave meets one above (no quantizer here makes it), whose
// values would be infinite, it does its tiles anew with the scales applied to
// each block's sum.
//
// The weight-side operand B is the matrix core's "A" operand, so that a
// lane's accumulators are columns n of one row m of C.
#include <algorithm>

#include "mx_layer.h"
#include "mx_layer_device.h"

namespace mxl {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Two 16-byte halves as one operand.
__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// D += A B^T over 128 elements, scale bytes J of sa and sb.
template <int J>
__device__ __forceinline__ f32x4 mfma8(i32x8 a, i32x8 b, f32x4 d, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, 0, 0, J, (int)sa, J, (int)sb);
}

// Eight codes (two words) widened to bf16 with scale 2^(s-127).
__device__ __forceinline__ bf16x8 widen8(int w0, int w1, float s) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}
// An operand of 32 codes widened: four runs of eight; halves have their own scale.
struct Wide {
  bf16x8 v[4];
};
__device__ __forceinline__ Wide widen32(i32x8 c, uint32_t s0, uint32_t s1) {
  const float f0 = __uint_as_float(s0 << 23), f1 = __uint_as_float(s1 << 23);
  return Wide{{widen8(c[0], c[1], f0), widen8(c[2], c[3], f0), widen8(c[4], c[5], f1),
               widen8(c[6], c[7], f1)}};
}
__device__ __forceinline__ f32x4 mfma16(const Wide &a, const Wide &b, f32x4 d) {
#pragma unroll
  for (int i = 0; i < 4; i++)
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
  return d;
}

struct MatArgs {
  const uint8_t *a, *sa, *b, *sb;
  int64_t m, n, k;
  int64_t nb;      // scale bytes per row
  int out_bf16;
  int tm, tn;      // tiles along m and n
  int steps;       // slabs of 128 of one split (a multiple of 4 unless one split)
  void *c;         // output, or partial sums [split][m][n] fp32
  int partial;
};

// Bytes of w above 246, as their top bits.
__device__ __forceinline__ uint32_t far_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x09090909u) & w & 0x80808080u;
}

// MT x NT tiles of 16 rows of A (from row m0) and of B (from n0), elements k0
// to k1, for any scale bytes: 32 elements at a time, unscaled, straight from
// memory, the sums scaled before they are added. Rare, so of little code and
// few registers.
template <bool BLK32, int MT, int NT>
__device__ __forceinline__ void far_tiles(const MatArgs &g, int64_t m0, int64_t n0, int64_t k0, int64_t k1,
                                          int lane, f32x4 (&acc)[MT][NT]) {
  const int l16 = lane & 15, lg = lane >> 4;
  auto codes = [&](const uint8_t *base, int64_t row, int64_t k) {
    const u32x2 w = *reinterpret_cast<const u32x2 *>(base + row * g.k + k + 8 * lg);
    return widen8((int)w[0], (int)w[1], 1.0f);
  };
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll 1
  for (int64_t k = k0; k < k1; k += 32) {
    const int64_t at = k / (BLK32 ? 32 : 128);
    bf16x8 a[MT];
    int sa[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const int64_t row = min(m0 + 16 * i + l16, g.m - 1);
      a[i] = codes(g.a, row, k);
      sa[i] = g.sa[row * g.nb + at];
    }
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const bf16x8 b = codes(g.b, min(n0 + 16 * j + l16, g.n - 1), k);
      int sb[4];
#pragma unroll
      for (int e = 0; e < 4; e++) sb[e] = g.sb[min(n0 + 16 * j + 4 * lg + e, g.n - 1) * g.nb + at];
#pragma unroll
      for (int i = 0; i < MT; i++) {
        const f32x4 t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a[i], f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const bool nan = sa[i] == 255 || sb[e] == 255;
          acc[i][j][e] += nan ? __builtin_nanf("") : __builtin_ldexpf(t[e], sa[i] + sb[e] - 254);
        }
      }
    }
  }
}

// ---- tiled kernel -----------------------------------------------------------------
//
// A workgroup of (SIDE / TM) (SIDE / TN) waves owns a square tile. K runs in
// slabs of 128, one v_mfma_scale_f32_16x16x128_f8f6f4 deep, which go from
// global memory straight into LDS (16 bytes a lane, a row's 128 bytes one
// request), through BUFS buffers. A wave multiplies A's tiles one after the
// other with all of its B tiles, which it holds; it reads A two tiles ahead
// and, in the slab's last two tiles, the next slab's B and first A, so LDS is
// not waited for. The one barrier of a slab stands before those: the next
// slab has landed, and this one has been read, so that its buffer's next
// loads may start. A wave issues in order and a load waits at issue while
// the memory unit is taken, so loads are dealt out between products.
//
// The 16-byte chunk c of row r sits at position c ^ f(r), f chosen so that
// the 16 rows that a quarter of a read instruction touches fall on different
// banks. The chunks are swapped on the global side (a lane picks which chunk
// it loads), since a direct load writes LDS linearly. Scale bytes of four
// slabs are one word per row (and, with blocks of 32, per block of a slab)
// in LDS; the matrix core picks the slab's byte.
//
// 8192 x 8192 x 4096, bf16 out: 200 to 205 us with blocks of 128 (2.7 PFLOP/s),
// 211 to 215 with blocks of 32, the matrix cores busy 62 % of the cycles and
// the card at 2.0 of its 2.4 GHz; 4096 x 4096 x 4096 52 to 57 us. fp32 out 427 us
// (1.3 PFLOP/s): twice the products and the widening.

__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

constexpr uint32_t kOut = 0x80000000u;  // an offset past every buffer: loads give 0

// 16 bytes a lane from the buffer straight into LDS, lane after lane from
// `lds` on (wave-uniform). In assembly, since the compiler would otherwise
// make every later LDS read wait for it; the kernel waits where it must.
// It has no output register, and its memory clobber keeps the order.
__device__ __forceinline__ void load_lds16(i32x4 buffer, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               ::"s"(lds), "v"(offset), "s"(buffer) : "memory", "m0");
}
__device__ __forceinline__ i32x4 buffer_of(const void *base, uint32_t bytes) {
  const uint64_t p = (uint64_t)base;
  return i32x4{__builtin_amdgcn_readfirstlane((int)p), __builtin_amdgcn_readfirstlane((int)(p >> 32) & 0xFFFF),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

template <int SIDE, int TM, int TN, int BUFS, bool BLK32, bool EXACT>
struct Tiled {
  static constexpr int BM = SIDE, BN = SIDE;
  static constexpr int WAVES = (BM / TM) * (BN / TN), T = WAVES * 64;
  static constexpr int MT = TM / 16, NT = TN / 16;
  static constexpr int ROWS = BM + BN, G = BLK32 ? 4 : 1;
  static constexpr int PER = T / 8;           // rows one load of the workgroup covers
  static constexpr int LOADS = ROWS / PER;    // direct loads per thread and slab
  static constexpr int SROWS = (ROWS + T - 1) / T;  // rows of scales per thread
  static_assert(MT % 4 == 0 && ROWS % PER == 0 && BM % PER == 0 && PER % 16 == 0, "tile and threads");

  // LDS: A's BUFS slabs, then B's, so that one address per chunk and constant
  // offsets reach everything a lane reads
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static_assert(4 % BUFS == 0 && BUFS * A_BYTES <= 65536 && BUFS * B_BYTES <= 65536, "constant offsets");

  struct Loader {
    i32x4 ar, br;     // buffers of the tile's rows of A and B
    uint32_t o;       // offset of this thread's first chunk in either
    int kc, k;        // first element of the chunk
    uint32_t lds;     // where this wave's first chunk goes in slab 0
  };
  // Load i of slab `slab`'s codes into buffer `buf`. Offsets are checked
  // against the end of the tile's rows by the buffer, past a row's end the
  // offset is moved out: both give zeros.
  static __device__ __forceinline__ void load(const Loader &l, int slab, int buf, int i) {
    constexpr int AL = BM / PER;
    const int k0 = slab * 128;
    const uint32_t o = k0 + l.kc < l.k ? l.o + k0 : kOut;
    if (i < AL)
      load_lds16(l.ar, o + (uint32_t)(i * PER) * l.k, l.lds + buf * A_BYTES + i * T * 16);
    else
      load_lds16(l.br, o + (uint32_t)((i - AL) * PER) * l.k,
                 l.lds + BUFS * A_BYTES + buf * B_BYTES + (i - AL) * T * 16);
  }

  struct Places {
    const uint8_t *a0, *a1, *b0, *b1;  // this lane's two chunks of tile 0 of A and B
  };
  static __device__ __forceinline__ i32x8 read_a(const Places &p, int buf, int i) {
    return join(*reinterpret_cast<const u32x4 *>(p.a0 + buf * A_BYTES + 2048 * i),
                *reinterpret_cast<const u32x4 *>(p.a1 + buf * A_BYTES + 2048 * i));
  }
  static __device__ __forceinline__ i32x8 read_b(const Places &p, int buf, int j) {
    return join(*reinterpret_cast<const u32x4 *>(p.b0 + buf * B_BYTES + 2048 * j),
                *reinterpret_cast<const u32x4 *>(p.b1 + buf * B_BYTES + 2048 * j));
  }
};

// f(a word of the width that rows of n columns, n no multiple of 16 bytes, are
// aligned to) (8000 x 8100 x 4096, bf16: 249 us column by
// column, 227).
template <bool OUT16, typename F>
__device__ __forceinline__ void by_alignment(int64_t n, F f) {
  if constexpr (OUT16) {
    if (n % 4 == 0) f(u32x2{});
    else if (n % 2 == 0) f(uint32_t{});
    else f(uint16_t{});
  } else {
    if (n % 2 == 0) f(u32x2{});
    else f(uint32_t{});
  }
}

// A wave's MT x NT accumulator tiles to C, 16 rows at a time through `turn`
// (wave-private LDS). Row r's 16-byte chunks are moved by r so that the
// writes of one instruction, which share a chunk number, spread over banks.
// The stores keep the operands of other tiles in the caches (8192 x 8192 x
// 4096, three sets of operands in turn: 218 -> 204 us).
template <int MT, int NT, bool OUT16>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[MT][NT], uint8_t *turn, void *c,
                                           int64_t m, int64_t n, int64_t m0, int64_t n0, int lane) {
  constexpr int E = OUT16 ? 2 : 4, ROW = 16 * NT * E, CH = ROW / 16, V = 16 / E;
  const int l16 = lane & 15, lg = lane >> 4;
  const bool whole = n % V == 0;
#pragma unroll
  for (int i = 0; i < MT; i++) {
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int col = 16 * j + 4 * lg;  // four columns of row l16
      uint8_t *p = turn + l16 * ROW + ((col / V + l16) & (CH - 1)) * 16 + col % V * E;
      const f32x4 v = acc[i][j];
      if constexpr (OUT16) *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      else *reinterpret_cast<f32x4 *>(p) = v;
    }
    // one wave: its LDS operations run in order; the fences keep the compiler's
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (whole) {
#pragma unroll
      for (int u = 0; u < (16 * CH + 63) / 64; u++) {
        const int at = u * 64 + lane, row = at / CH, ch = at % CH;
        const int64_t mm = m0 + 16 * i + row, nn = n0 + ch * V;
        if (row < 16 && mm < m && nn < n)
          __builtin_nontemporal_store(
              *reinterpret_cast<const u32x4 *>(turn + row * ROW + ((ch + row) & (CH - 1)) * 16),
              reinterpret_cast<u32x4 *>(reinterpret_cast<uint8_t *>(c) + (mm * n + nn) * E));
      }
    } else {
      // rows begin between 16-byte marks: pieces as wide as their alignment
      auto pieces = [&](auto one) {
        constexpr int W = sizeof(one) / E, Q = 16 * NT / W;  // columns a piece, pieces a row
        static_assert(Q <= 64, "a row in one instruction");
        for (int u = 0; u < Q / 4; u++) {
          const int row = u * (64 / Q) + lane / Q, col = lane % Q * W;
          const uint8_t *p = turn + row * ROW + ((col / V + row) & (CH - 1)) * 16 + col % V * E;
          const int64_t mm = m0 + 16 * i + row, nn = n0 + col;
          if (mm < m && nn < n)
            *reinterpret_cast<decltype(one) *>(reinterpret_cast<uint8_t *>(c) + (mm * n + nn) * E) =
                *reinterpret_cast<const decltype(one) *>(p);
        }
      };
      by_alignment<OUT16>(n, pieces);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// The same for tiles of 64 whose four waves hold 16 columns each: their parts
// meet in LDS first, so that rows are written 64 columns at a time and not 16
// (333 x 4099 x 1568: 0.5 us less of 14).
template <bool OUT16>
__device__ __forceinline__ void store_tile64(const f32x4 (&acc)[4][1], uint8_t *turn, void *c, int64_t m,
                                             int64_t n, int64_t m0, int64_t n0, int wave, int lane) {
  constexpr int E = OUT16 ? 2 : 4, ROW = 64 * E, CH = ROW / 16, V = 16 / E;
  const int l16 = lane & 15, lg = lane >> 4;
  const int col = 16 * wave + 4 * lg;  // four columns of row 16 i + l16
  auto place = [&](int row, int column) {
    return turn + row * ROW + ((column / V + row) & (CH - 1)) * 16 + column % V * E;
  };
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const f32x4 v = acc[i][0];
    uint8_t *p = place(16 * i + l16, col);
    if constexpr (OUT16) *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    else *reinterpret_cast<f32x4 *>(p) = v;
  }
  __syncthreads();
  if (n % V == 0) {
#pragma unroll
    for (int u = 0; u < CH / 4; u++) {
      const int at = u * 256 + wave * 64 + lane, row = at / CH, cc = at % CH * V;
      if (m0 + row < m && n0 + cc < n)
        __builtin_nontemporal_store(
            *reinterpret_cast<const u32x4 *>(place(row, cc)),
            reinterpret_cast<u32x4 *>(reinterpret_cast<uint8_t *>(c) + ((m0 + row) * n + n0 + cc) * E));
    }
  } else {
    auto pieces = [&](auto one) {
      constexpr int W = sizeof(one) / E, Q = 64 / W;
#pragma unroll
      for (int u = 0; u < Q / 4; u++) {
        const int row = (4 * u + wave) * (64 / Q) + lane / Q, col = lane % Q * W;
        if (m0 + row < m && n0 + col < n)
          *reinterpret_cast<decltype(one) *>(reinterpret_cast<uint8_t *>(c) + ((m0 + row) * n + n0 + col) * E) =
              *reinterpret_cast<const decltype(one) *>(place(row, col));
      }
    };
    by_alignment<OUT16>(n, pieces);
  }
}

// two waves a SIMD, a workgroup of 8 or two of 4, unless LDS holds only one of 4
template <int SIDE, int TM, int TN, int BUFS, bool BLK32, bool EXACT>
__global__ __launch_bounds__((SIDE / TM) * (SIDE / TN) * 64, SIDE == 128 && BUFS == 4 ? 1 : 2) void k_matmul8(const MatArgs g) {
  using K = Tiled<SIDE, TM, TN, BUFS, BLK32, EXACT>;
  constexpr int BM = SIDE, BN = SIDE;
  constexpr int MT = K::MT, NT = K::NT, ROWS = K::ROWS, G = K::G;
  __shared__ __attribute__((aligned(16))) uint8_t slabs[BUFS * ROWS * 128];
  __shared__ uint32_t scl[2][G][ROWS];

  // XCD-aware order: workgroups are dealt round robin to the 8 XCDs; each
  // XCD gets a contiguous eighth of the tiles (the first ones one more, where
  // eight does not divide them), walked in strips of 8 tile rows so that its
  // L2 holds the panels in use. (Launch order: 3333 x 5555 x 4096 104 us, this
  // 96; 333 x 4099 x 1568 14 and 11; 4099 x 1536 x 4096 33 and 35.)
  const int tiles = g.tm * g.tn;
  int t = blockIdx.x;
  t = (t & 7) * (tiles >> 3) + min(t & 7, tiles & 7) + (t >> 3);
  const int strip = 8 * g.tn, s0 = t / strip, in = t - s0 * strip;
  const int high = min(8, g.tm - 8 * s0);
  const int64_t m0 = (int64_t)(8 * s0 + in % high) * BM, n0 = (int64_t)(in / high) * BN;

  const int first = blockIdx.y * g.steps;
  const int nk = min(g.steps, (int)((g.k + 127) >> 7) - first);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;

  // direct loads: load i covers rows i PER + tid / 8, chunk position tid % 8;
  // the swizzle repeats every 16 rows
  typename K::Loader ld;
  ld.k = (int)g.k;
  ld.lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)slabs + wave * 1024;
  {
    const int r = threadIdx.x >> 3;
    ld.kc = ((threadIdx.x & 7) ^ swz(r)) * 16;
    ld.o = (uint32_t)r * ld.k + ld.kc;
    ld.ar = buffer_of(g.a + m0 * g.k, (uint32_t)(min((int64_t)BM, g.m - m0) * g.k));
    ld.br = buffer_of(g.b + n0 * g.k, (uint32_t)(min((int64_t)BN, g.n - n0) * g.k));
  }

  // scales: thread r holds row r of the tile (A rows, then B rows), clamped
  // to the matrix. Four slabs take 16 bytes of a row with blocks of 32 and 4
  // with blocks of 128; where they would pass the row's end, the row's last
  // ones are read and shifted down (the elements past the end are zeros). A
  // row with fewer has one chunk only; the loads for chunks that do not
  // exist read something valid and are not used.
  constexpr int SB = 4 * G, SR = K::SROWS, T = K::T;
  const bool brief = g.nb < SB;
  const int slast = brief ? 0 : (int)g.nb - SB;
  const uint8_t *sp[SR];  // wave-uniform: a wave's rows are all A's or all B's
  uint32_t so[SR], raw[SR][G];
#pragma unroll
  for (int q = 0; q < SR; q++) {
    const int row = min((int)threadIdx.x + q * T, ROWS - 1);
    const bool is_a = min(wave * 64 + q * T, ROWS - 1) < BM;
    static_assert(BM % 64 == 0, "a wave's rows");
    sp[q] = brief ? g.a : is_a ? g.sa + m0 * g.nb : g.sb + n0 * g.nb;  // codes: at least 32 bytes
    so[q] = brief ? 0 : (uint32_t)((is_a ? min((int64_t)row, g.m - 1 - m0)
                                         : min((int64_t)row - BM, g.n - 1 - n0)) * g.nb);
  }
  auto load_scales = [&](int chunk) {
    const int at = (first + 4 * chunk) * G, from = min(at, slast), by = at - from;
#pragma unroll
    for (int q = 0; q < SR; q++) {
      if constexpr (BLK32) {
        __builtin_memcpy(raw[q], sp[q] + from + so[q], 16);
        if (by) {  // wave-uniform, only near the row's end; by < 16 where the slab exists
          unsigned __int128 w;
          __builtin_memcpy(&w, raw[q], 16);
          w >>= 8 * min(by, 15);
          __builtin_memcpy(raw[q], &w, 16);
        }
      } else {
        uint32_t w;
        __builtin_memcpy(&w, sp[q] + from + so[q], 4);
        raw[q][0] = w >> (8 * min(by, 3));
      }
    }
  };
  auto put_scales = [&](int buf) {
#pragma unroll
    for (int q = 0; q < SR; q++) {
      const int row = threadIdx.x + q * T;
      if (ROWS % T == 0 || row < ROWS) {
        if constexpr (BLK32) {  // word s holds slab s's four blocks: turn the 4 x 4 bytes
          const uint32_t *w = raw[q];
          const uint32_t p0 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u),
                         p1 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u),
                         q0 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u),
                         q1 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
          scl[buf][0][row] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);
          scl[buf][1][row] = __builtin_amdgcn_perm(p1, p0, 0x07060302u);
          scl[buf][2][row] = __builtin_amdgcn_perm(q1, q0, 0x05040100u);
          scl[buf][3][row] = __builtin_amdgcn_perm(q1, q0, 0x07060302u);
        } else {
          scl[buf][0][row] = raw[q][0];
        }
      }
    }
  };

  const int wm = wave % (BM / TM) * TM, wn = wave / (BM / TM) * TN;
  // this lane's operand rows: A row wm + 16 i + l16, B row wn + 16 j + l16;
  // the swizzle does not depend on i and j
  const int ra = wm + l16, rb = wn + l16;
  const int lo = (lg ^ swz(l16)) * 16, hi = lo ^ 64;
  const uint8_t *pa = slabs + ra * 128, *pb = slabs + BUFS * K::A_BYTES + rb * 128;
  const typename K::Places pl = {pa + lo, pa + hi, pb + lo, pb + hi};
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[i][j] = f32x4{0, 0, 0, 0};

  if (brief) {
#pragma unroll
    for (int q = 0; q < SR; q++) {
#pragma unroll
      for (int e = 0; e < G; e++) raw[q][e] = 0;
      const int row = min((int)threadIdx.x + q * T, ROWS - 1);
      const uint8_t *p = row < BM ? g.sa + min(m0 + row, g.m - 1) * g.nb
                                  : g.sb + min(n0 + row - BM, g.n - 1) * g.nb;
      for (int j = 0; j < (int)g.nb; j++) {
        const uint32_t b = (uint32_t)p[j] << (8 * (j & 3));
#pragma unroll
        for (int e = 0; e < G; e++)
          if (j >> 2 == e) raw[q][e] |= b;
      }
    }
  } else {
    load_scales(0);
  }
  put_scales(0);

  // Loads of a slab: the first START of them in the last two tiles of the
  // slab whose buffer they take, the others in the first two of the next.
  constexpr int LOADS = K::LOADS, START = MT >= 8 ? LOADS / 2 : LOADS;
#pragma unroll
  for (int i = 0; i < (BUFS - 1) * LOADS + START; i++)
    K::load(ld, first + i / LOADS, i / LOADS, i % LOADS);
  // the first slab has landed (the others may be in flight)
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"((BUFS - 2) * LOADS + START) : "memory");
  uint32_t as[MT][2], bs[NT][2], far = 0;  // far: bytes past what widening takes
  auto get_scales = [&](int buf) {
    // exact: the lane's halves lie in blocks lg / 2 and 2 + lg / 2 of a slab
    const int g0 = !BLK32 ? 0 : EXACT ? lg >> 1 : lg, g1 = EXACT && BLK32 ? 2 + (lg >> 1) : g0;
#pragma unroll
    for (int i = 0; i < MT; i++) {
      as[i][0] = scl[buf][g0][ra + 16 * i];
      as[i][1] = EXACT && BLK32 ? scl[buf][g1][ra + 16 * i] : as[i][0];
    }
#pragma unroll
    for (int j = 0; j < NT; j++) {
      bs[j][0] = scl[buf][g0][BM + rb + 16 * j];
      bs[j][1] = EXACT && BLK32 ? scl[buf][g1][BM + rb + 16 * j] : bs[j][0];
    }
    if constexpr (EXACT) {
#pragma unroll
      for (int h = 0; h < (BLK32 ? 2 : 1); h++) {
#pragma unroll
        for (int i = 0; i < MT; i++) far |= far_bytes(as[i][h]);
#pragma unroll
        for (int j = 0; j < NT; j++) far |= far_bytes(bs[j][h]);
      }
    }
  };
  i32x8 a[4], b[NT];
  get_scales(0);
#pragma unroll
  for (int j = 0; j < NT; j++) b[j] = K::read_b(pl, 0, j);
  a[0] = K::read_a(pl, 0, 0);
  a[1] = K::read_a(pl, 0, 1);

  auto step = [&](int s, auto jt) {
    // slab s is the J-th of its chunk of four; its buffer, the one before and after
    constexpr int J = decltype(jt)::value, CUR = J % BUFS, PREV = (J + 3) % BUFS, NEXT = (J + 1) % BUFS;
    Wide bw[EXACT ? NT : 1];
    if constexpr (EXACT) {
#pragma unroll
      for (int j = 0; j < NT; j++)
        bw[j] = widen32(b[j], bs[j][0] >> (8 * J) & 255, bs[j][1] >> (8 * J) & 255);
    }
    if constexpr (J == 0) load_scales((s >> 2) + 1);
#pragma unroll
    for (int i = 0; i < MT; i++) {
      if (i == MT - 2) {
        // the next slab (this wave's loads of it) has landed and this one
        // has been read; past the barrier that holds for every wave
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"((BUFS - 2) * LOADS) : "memory");
        // the next chunk's scales: read two slabs on
        if constexpr (J == 1) put_scales(((s >> 2) + 1) & 1);
      }
      // a slab's loads in up to four parts of at most HALF
      constexpr int HALF = (START + 1) / 2;
#pragma unroll
      for (int q = 0; q < LOADS; q++) {
        if (i < 2 && q >= START + i * HALF && q < START + (i + 1) * HALF)
          K::load(ld, first + s - 1 + BUFS, PREV, q);
        if (i >= MT - 2 && q < START && q >= (i - MT + 2) * HALF && q < (i - MT + 3) * HALF)
          K::load(ld, first + s + BUFS, CUR, q);
      }
      // past the barrier, reads are of the next slab
      a[(i + 2) & 3] = i < MT - 2 ? K::read_a(pl, CUR, i + 2) : K::read_a(pl, NEXT, i + 2 - MT);
      if constexpr (EXACT) {
        const Wide aw = widen32(a[i & 3], as[i][0] >> (8 * J) & 255, as[i][1] >> (8 * J) & 255);
#pragma unroll
        for (int j = 0; j < NT; j++) acc[i][j] = mfma16(bw[j], aw, acc[i][j]);
      }
#pragma unroll
      for (int j = 0; j < NT; j++) {
        if constexpr (!EXACT)
          acc[i][j] = mfma8<J>(b[j], a[i & 3], acc[i][j], bs[j][0], as[i][0]);
        // the last use of a B tile: its next one takes its place
        if (i == MT - 1) {
          __builtin_amdgcn_sched_barrier(0);
          b[j] = K::read_b(pl, NEXT, j);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (J == 3) get_scales(((s >> 2) + 1) & 1);
  };
  // whole chunks of four slabs, then the rest. (A way out between the steps
  // of the loop would let the compiler move reads past it.)
  int s = 0;
  for (; s + 4 <= nk; s += 4) {
    step(s, std::integral_constant<int, 0>());
    step(s + 1, std::integral_constant<int, 1>());
    step(s + 2, std::integral_constant<int, 2>());
    step(s + 3, std::integral_constant<int, 3>());
  }
  if (s < nk) step(s, std::integral_constant<int, 0>());
  if (s + 1 < nk) step(s + 1, std::integral_constant<int, 1>());
  if (s + 2 < nk) step(s + 2, std::integral_constant<int, 2>());
  // nothing may still be landing in LDS, and every wave is done reading it
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if constexpr (EXACT) {
    if (__builtin_expect(__any(far != 0), 0))
      far_tiles<BLK32, MT, NT>(g, m0 + wm, n0 + wn, (int64_t)first * 128, min(g.k, (int64_t)(first + nk) * 128),
                               lane, acc);
  }

  // Output: a lane's accumulators are 4-column runs of one row, which would
  // be written in pieces of 8 or 16 bytes, so they are turned in LDS: by each
  // wave for itself, 16 rows at a time, where it holds 64 columns.
  float *out32 = reinterpret_cast<float *>(g.c) + (g.partial ? (int64_t)blockIdx.y * g.m * g.n : 0);
  if constexpr (SIDE == 64) {
    static_assert(MT == 4 && NT == 1 && T == 256, "four waves side by side");
    if (g.out_bf16 && !g.partial) store_tile64<true>(acc, slabs, g.c, g.m, g.n, m0, n0, wave, lane);
    else store_tile64<false>(acc, slabs, out32, g.m, g.n, m0, n0, wave, lane);
  } else {
    uint8_t *turn = slabs + wave * (16 * TN * 4);
    static_assert(K::WAVES * 16 * TN * 4 <= BUFS * ROWS * 128, "turning space");
    if (g.out_bf16 && !g.partial)
      store_tile<MT, NT, true>(acc, turn, g.c, g.m, g.n, m0 + wm, n0 + wn, lane);
    else
      store_tile<MT, NT, false>(acc, turn, out32, g.m, g.n, m0 + wm, n0 + wn, lane);
  }
}

// Sum of the splits' partial results in order, rounded to the output type.
__global__ __launch_bounds__(256) void k_sum_splits(const float *__restrict__ p, int splits,
                                                    int64_t count, int out_bf16,
                                                    void *__restrict__ c) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  const bool whole = i + 4 <= count && count % 4 == 0;
  float v[4] = {0, 0, 0, 0};
  for (int s = 0; s < splits; s++) {
    const float *q = p + s * count + i;
    if (whole) {
      const f32x4 w = *reinterpret_cast<const f32x4 *>(q);
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] += w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (i + j < count) v[j] += q[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if (i + j >= count) break;
    if (out_bf16) reinterpret_cast<uint16_t *>(c)[i + j] = (uint16_t)pack_bf16(v[j], 0.0f);
    else reinterpret_cast<float *>(c)[i + j] = v[j];
  }
}

// ---- few rows -----------------------------------------------------------------------
//
// 16 rows of A (single tokens, small batches), or a few times 16: bound by
// reading B, 1 x 8192 x 4096 in 8.7 us (3.9 TB/s; launch and one trip to
// memory are half of it). A workgroup owns 16 CT columns (rows of B) and its
// waves split K into contiguous ranges; a wave loads B's codes straight into
// the matrix core's layout (each row's 128 bytes of a slab are one cache
// line), four slabs at a time so that 8 CT KiB per wave are in flight, and A's
// rows come from the caches. The waves' sums are added in order through LDS.
template <int CT, bool BLK32, bool EXACT>
__global__ __launch_bounds__(512) void k_matmul8_rows(const MatArgs g) {
  constexpr int U = 4, WAVES = 8;
  __shared__ float part[WAVES][16][16 * CT + 1];
  const int64_t n0 = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * (16 * CT);
  if (n0 >= g.n) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int all = (int)((g.k + 127) >> 7), per = (all + WAVES - 1) / WAVES;
  const int first = wave * per, last = min(all, first + per);
  const uint8_t *bp[CT], *sbp[CT];
#pragma unroll
  for (int c = 0; c < CT; c++) {
    const int64_t n = min(n0 + 16 * c + l16, g.n - 1);
    bp[c] = g.b + n * g.k;
    sbp[c] = g.sb + n * g.nb;
  }
  const int64_t m0 = (int64_t)blockIdx.y * 16, m = min(m0 + l16, g.m - 1);
  const uint8_t *ap = g.a + m * g.k, *sap = g.sa + m * g.nb;
  const int64_t nb1 = g.nb - 1;
  const u32x4 zero = {0, 0, 0, 0};
  f32x4 acc[1][CT];
  uint32_t largest = 0;  // scale byte
#pragma unroll
  for (int c = 0; c < CT; c++) acc[0][c] = f32x4{0, 0, 0, 0};
  for (int s = first; s < last; s += U) {
    i32x8 bv[U][CT], av[U];
    uint32_t bs[U][CT][2], as[U][2];
#pragma unroll
    for (int u = 0; u < U; u++) {
      // chunks past K (or past this wave's range) are zeros
      const int64_t k0 = (int64_t)(s + u) * 128 + 16 * lg, k1 = k0 + 64;
      const bool h0 = s + u < last && k0 < g.k, h1 = s + u < last && k1 < g.k;
#pragma unroll
      for (int c = 0; c < CT; c++)
        bv[u][c] =
            join(h0 ? *reinterpret_cast<const u32x4 *>(bp[c] + k0) : zero,
                 h1 ? *reinterpret_cast<const u32x4 *>(bp[c] + k1) : zero);
      av[u] = join(h0 ? *reinterpret_cast<const u32x4 *>(ap + k0) : zero,
                   h1 ? *reinterpret_cast<const u32x4 *>(ap + k1) : zero);
#pragma unroll
      for (int h = 0; h < (EXACT && BLK32 ? 2 : 1); h++) {
        const int64_t at = min(!BLK32 ? (int64_t)(s + u)
                                      : (int64_t)(s + u) * 4 + (EXACT ? 2 * h + (lg >> 1) : lg),
                               nb1);
#pragma unroll
        for (int c = 0; c < CT; c++) bs[u][c][h] = sbp[c][at];
        as[u][h] = sap[at];
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      if constexpr (EXACT) {
        const Wide aw = widen32(av[u], as[u][0], as[u][BLK32 ? 1 : 0]);
        largest = max(largest, max(as[u][0], as[u][BLK32 ? 1 : 0]));
#pragma unroll
        for (int c = 0; c < CT; c++) {
          acc[0][c] = mfma16(widen32(bv[u][c], bs[u][c][0], bs[u][c][BLK32 ? 1 : 0]), aw, acc[0][c]);
          largest = max(largest, max(bs[u][c][0], bs[u][c][BLK32 ? 1 : 0]));
        }
      } else {
#pragma unroll
        for (int c = 0; c < CT; c++) acc[0][c] = mfma8<0>(bv[u][c], av[u], acc[0][c], bs[u][c][0], as[u][0]);
      }
    }
  }
  if constexpr (EXACT) {
    if (__builtin_expect(__any(largest > 246u), 0))
      far_tiles<BLK32, 1, CT>(g, m0, n0, (int64_t)first * 128, min(g.k, (int64_t)last * 128), lane, acc);
  }
#pragma unroll
  for (int c = 0; c < CT; c++)
#pragma unroll
    for (int e = 0; e < 4; e++) part[wave][l16][16 * c + 4 * lg + e] = acc[0][c][e];
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * CT; i += WAVES * 64) {
    const int r = i / (16 * CT), c = i % (16 * CT);
    if (m0 + r < g.m && n0 + c < g.n) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; w++) v += part[w][r][c];
      const int64_t at = (m0 + r) * g.n + n0 + c;
      if (g.out_bf16) reinterpret_cast<uint16_t *>(g.c)[at] = (uint16_t)pack_bf16(v, 0.0f);
      else reinterpret_cast<float *>(g.c)[at] = v;
    }
  }
}

// ---- which kernel -------------------------------------------------------------------

// A choice of kernel for rows [0, m) of A. Figures are microseconds with
// bfloat16 outputs and blocks of 128 unless said otherwise, three sets of
// operands in turn.
struct Plan {
  int columns;          // > 0: the few-rows kernel with this many column tiles
  int side, bufs;       // else square tiles of this side
  int splits, steps;    // of K; slabs of one
  int64_t rest;         // the last rows, done by the few-rows kernel
};

static int64_t tiles_of(int64_t m, int64_t n, int side) {
  return ((m + side - 1) / side) * ((n + side - 1) / side);
}
// At least four fifths of the compute units busy, over all rounds of tiles
static bool full_rounds(int64_t tiles) { return tiles * 5 >= ((tiles + 255) / 256) * 256 * 4; }

static Plan plan_of(int64_t m, int64_t n, int64_t k, int out_bf16) {
  const int all = (int)((k + 127) >> 7);
  Plan p = {0, 0, 0, 1, all, 0};
  // Up to 16 rows: one reading of B decides. 32 columns a workgroup where
  // that still gives every compute unit one (16 x 8192 x 4096: 11.0, with 16
  // columns 13.2), else 16 (16 x 4096 x 4096: 7.9, with 32 10.4).
  if (m <= 16) {
    p.columns = n >= 32 * 256 ? 2 : 1;
    return p;
  }
  // Up to 64 rows: the same in groups of 16, as long as every compute unit
  // gets at most one workgroup (32 x 512 x 4096: 7.2, tiles of 64 9.8; 64 x
  // 1024 x 8192: 12.9 and 21; but 48 x 4096 x 4096: 18.4 and 12).
  if (m <= 64 && ((m + 15) / 16) * ((n + 15) / 16) <= 256) {
    p.columns = 1;
    return p;
  }
  // Tiles of 256 use the matrix cores best where they fill the card in whole
  // rounds (4096 x 4096 x 4096: 52 to 57, tiles of 128 63), not where the last
  // round is nearly empty (4099 x 4096 x 1536: 40 and 35). If up to 16 rows open
  // that round, they go to the few-rows kernel (4099 rows: 28, 4112: 28; 4112 x
  // 4096 x 4096: 59, tiles of 256 alone 88, of 128 80). Tiles of 256 leave no
  // registers to widen codes in, which fp32 outputs do.
  const int64_t t256 = tiles_of(m, n, 256), t128 = tiles_of(m, n, 128), t64 = tiles_of(m, n, 64);
  if (out_bf16) {
    const int64_t rest = m % 256 <= 16 && m > 256 ? m % 256 : 0;
    if (full_rounds(t256)) {
      p.side = 256;
      p.bufs = 2;
      return p;
    }
    if (rest && full_rounds(tiles_of(m - rest, n, 256))) {
      p.side = 256;
      p.bufs = 2;
      p.rest = rest;
      return p;
    }
  }
  // Tiles of 128: two workgroups a compute unit with two buffers each (2048 x
  // 4096 x 4096: 33, one with four 40), one with four where there is only one
  // for each (1024 x 4096 x 4096: 21 and 25). Fewer tiles than 144 leave too
  // many idle: then tiles of 64 (512 x 4096 x 4096: 16, tiles of 128 19.5).
  if (t128 >= 144) {
    p.side = 128;
    p.bufs = t128 > 256 ? 2 : 4;
    return p;
  }
  p.side = 64;
  p.bufs = 4;
  // Split K where tiles of 64 leave half of the card idle, at least 16 slabs
  // each, since the sum costs 3 to 4 us (256 x 1024 x 8192: 13.5, unsplit 21;
  // 128 x 2048 x 2048 unsplit: 6.5, split 8.5; up to 64 rows, 64 x 8192 x 4096:
  // 12.5, split 13.5).
  const int want = m <= 64 ? 1 : (int)std::min<int64_t>(256 / t64, all / 16);
  if (want > 1) {
    p.steps = ((all + want - 1) / want + 3) & ~3;
    p.splits = (all + p.steps - 1) / p.steps;
  }
  return p;
}

template <bool BLK32, bool EXACT>
static hipError_t launch(const Plan &p, MatArgs g, hipStream_t st) {
  if (p.columns) {
    // a grid's dimension holds fewer than 2^32 threads
    const int64_t columns = (g.n + 16 * p.columns - 1) / (16 * p.columns), x = std::min<int64_t>(columns, 1 << 22);
    const dim3 grid((uint32_t)x, (uint32_t)((g.m + 15) / 16), (uint32_t)((columns + x - 1) / x));
    if (p.columns == 1) k_matmul8_rows<1, BLK32, EXACT><<<grid, 512, 0, st>>>(g);
    else k_matmul8_rows<2, BLK32, EXACT><<<grid, 512, 0, st>>>(g);
    return hipGetLastError();
  }
  g.tm = (int)((g.m + p.side - 1) / p.side);
  g.tn = (int)((g.n + p.side - 1) / p.side);
  g.steps = p.steps;
  const dim3 grid((uint32_t)(g.tm * g.tn), (uint32_t)p.splits);
  if constexpr (!EXACT) {
    if (p.side == 256) {
      k_matmul8<256, 128, 64, 2, BLK32, false><<<grid, 512, 0, st>>>(g);
      return hipGetLastError();
    }
  }
  if (p.side == 128 && p.bufs == 2) k_matmul8<128, 64, 64, 2, BLK32, EXACT><<<grid, 256, 0, st>>>(g);
  else if (p.side == 128) k_matmul8<128, 64, 64, 4, BLK32, EXACT><<<grid, 256, 0, st>>>(g);
  else k_matmul8<64, 64, 16, 4, BLK32, EXACT><<<grid, 256, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace mxl

using namespace mxl;

size_t mxi_matmul8_workspace(int64_t m, int64_t n, int64_t k, int block, int out_bf16) {
  (void)block;
  const Plan p = plan_of(m, n, k, out_bf16);
  return p.splits > 1 ? (size_t)p.splits * m * n * sizeof(float) : 0;
}

hipError_t mxi_launch_matmul8(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b,
                              const uint8_t *b_scales, int64_t m, int64_t n, int64_t k, int block,
                              int out_bf16, void *c, void *workspace, hipStream_t st) {
  const Plan p = plan_of(m, n, k, out_bf16);
  if (p.rest) {
    const int64_t at = m - p.rest, nb = (k + block - 1) / block;
    const hipError_t e = mxi_launch_matmul8(a + at * k, a_scales + at * nb, b, b_scales, p.rest, n, k, block,
                                            out_bf16, reinterpret_cast<uint8_t *>(c) + at * n * 2, workspace, st);
    if (e != hipSuccess) return e;
    m = at;
  }
  MatArgs g = {a, a_scales, b, b_scales, m, n, k, (k + block - 1) / block, out_bf16, 0, 0, 0,
               p.splits > 1 ? workspace : c, p.splits > 1};
  hipError_t e;
  if (out_bf16) e = block == 32 ? launch<true, false>(p, g, st) : launch<false, false>(p, g, st);
  else e = block == 32 ? launch<true, true>(p, g, st) : launch<false, true>(p, g, st);
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t count = m * n;
  k_sum_splits<<<dim3((uint32_t)((count + 1023) / 1024)), 256, 0, st>>>(
      reinterpret_cast<const float *>(workspace), p.splits, count, out_bf16, c);
  return hipGetLastError();
}
