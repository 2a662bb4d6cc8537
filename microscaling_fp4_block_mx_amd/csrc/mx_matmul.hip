// mx_matmul.hip - product of two MXFP8 matrices on the matrix cores:
//   C[m][n] = sum_k A[m][k] 2^(sa-127) B[n][k] 2^(sb-127)
// A [M, K] and B [N, K] are E4M3 codes, row-major, with one E8M0 byte per 32
// or 128 elements of a row. K is a multiple of 32; M and N are any.
//
// bf16 output runs v_mfma_scale_f32_16x16x128_f8f6f4, which multiplies codes
// and applies the E8M0 bytes itself. Lane layout (checked on the card): lane
// l holds row l % 16; with g = l / 16 its first 16 bytes are k = 16 g ..
// 16 g + 15 and its second 16 bytes are k = 64 + 16 g ..; the scale byte that
// lane l supplies belongs to row l % 16 and elements k = 32 g .. 32 g + 31.
// Inside each group of eight products the matrix core drops bits more than
// about 2^-14 below the largest product (1.4e-5 of the result's norm on
// normal data), which is far inside bf16's rounding (1.7e-3) but not inside
// fp32's. fp32 output therefore widens the codes to bf16, scales applied
// (both exact), and runs v_mfma_f32_16x16x32_bf16 at half the rate.
//
// The weight-side operand B is the matrix core's "A" operand, so that a
// lane's accumulators are consecutive columns n of one row m of C: column
// n = 4 NT (r / 4) + 4 t + r % 4 of a wave's 16 NT columns is row r of its
// tile t, which makes the 4 NT accumulators of a lane one contiguous run.
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

// L consecutive columns of a row of C from column n on; vec: 16-byte stores
// are aligned and whole.
template <int L>
__device__ __forceinline__ void store_run(void *c, int out_bf16, int64_t at, const float (&v)[L],
                                          int64_t left, bool vec) {
  if (out_bf16) {
    uint16_t *p = reinterpret_cast<uint16_t *>(c) + at;
    if (vec && left >= L && L % 8 == 0) {
#pragma unroll
      for (int j = 0; j + 8 <= L; j += 8)
        *reinterpret_cast<u32x4 *>(p + j) =
            u32x4{pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]),
                  pack_bf16(v[j + 4], v[j + 5]), pack_bf16(v[j + 6], v[j + 7])};
    } else {
#pragma unroll
      for (int j = 0; j < L; j++)
        if (j < left) p[j] = (uint16_t)pack_bf16(v[j], 0.0f);
    }
  } else {
    float *p = reinterpret_cast<float *>(c) + at;
    if (vec && left >= L) {
#pragma unroll
      for (int j = 0; j < L; j += 4)
        *reinterpret_cast<f32x4 *>(p + j) = f32x4{v[j], v[j + 1], v[j + 2], v[j + 3]};
    } else {
#pragma unroll
      for (int j = 0; j < L; j++)
        if (j < left) p[j] = v[j];
    }
  }
}

struct MatArgs {
  const uint8_t *a, *sa, *b, *sb;
  int64_t m, n, k;
  int64_t nb;      // scale bytes per row
  int out_bf16;
  int tm, tn;      // tiles along m and n
  int steps;       // K steps of 128 of one split (a multiple of 4 unless one split)
  void *c;         // output, or partial sums [split][m][n] fp32
  int partial;
};

// ---- tiled kernel -----------------------------------------------------------------
//
// A workgroup of (BM / TM) (BN / TN) waves owns a BM x BN tile; K runs in
// steps of 128. Codes go from global memory straight into LDS (16 bytes a
// lane), double-buffered, one barrier per step: a step first reads its
// operands from LDS into registers, then starts the next step's loads into
// the other buffer, then multiplies. Rows are 128 bytes; 16-byte chunk c of
// row r sits at position c ^ f(r), f chosen so that the 16 rows one read
// instruction touches spread over all banks. The chunks are swapped on the
// global side (a lane picks which chunk it loads), since a direct load
// writes LDS linearly. Scale bytes of four steps are packed into one word
// per row (and per 32-element block: four words) in LDS; the matrix core
// picks the step's byte.

// Swizzle of A rows (16 consecutive rows per read) and B rows (see the column
// order above: rows 4 NT apart in fours).
__device__ __forceinline__ int swz_a(int r) { return (r >> 1) & 7; }
template <int NT>
__device__ __forceinline__ int swz_b(int r) {
  return ((r >> 1) & 1) | (((r / (4 * NT)) & 3) << 1);
}

constexpr uint32_t kOut = 0x80000000u;  // an offset past every buffer: loads give 0

template <int BM, int BN, int TM, int TN, bool BLK32, bool EXACT>
__global__ __launch_bounds__((BM / TM) * (BN / TN) * 64) void k_matmul8(const MatArgs g) {
  constexpr int WAVES = (BM / TM) * (BN / TN), T = WAVES * 64;
  constexpr int MT = TM / 16, NT = TN / 16;
  constexpr int ROWS = BM + BN, G = BLK32 ? 4 : 1;
  constexpr int LOADS = ROWS * 8 / T;  // direct loads per thread and step
  static_assert(ROWS <= T && ROWS * 8 % T == 0 && BM * 8 % T == 0, "tile and threads");
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][ROWS * 128];
  __shared__ uint32_t scl[2][G][ROWS];

  // XCD-aware order: workgroups are dealt round robin to the 8 XCDs; each
  // XCD gets a contiguous eighth of the tiles, walked in strips of 8 tile
  // rows so that its L2 holds the panels in use.
  const int tiles = g.tm * g.tn;
  int t = blockIdx.x;
  if (tiles % 8 == 0) t = (t & 7) * (tiles >> 3) + (t >> 3);
  const int strip = 8 * g.tn, s0 = t / strip, in = t - s0 * strip;
  const int high = min(8, g.tm - 8 * s0);
  const int64_t m0 = (int64_t)(8 * s0 + in % high) * BM, n0 = (int64_t)(in / high) * BN;

  const int first = blockIdx.y * g.steps;
  const int all = (int)((g.k + 127) >> 7);
  const int nk = min(g.steps, all - first);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;

  // direct loads: load i covers LDS rows (i T + tid) / 8, chunk position tid % 8
  const uint8_t *abase = g.a + m0 * g.k, *bbase = g.b + n0 * g.k;
  const uint32_t abytes = (uint32_t)(min((int64_t)BM, g.m - m0) * g.k);
  const uint32_t bbytes = (uint32_t)(min((int64_t)BN, g.n - n0) * g.k);
  const __amdgpu_buffer_rsrc_t ar =
      __builtin_amdgcn_make_buffer_rsrc((void *)abase, 0, abytes, 0x00020000);
  const __amdgpu_buffer_rsrc_t br =
      __builtin_amdgcn_make_buffer_rsrc((void *)bbase, 0, bbytes, 0x00020000);
  uint32_t off[LOADS];
  int kc[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; i++) {
    const int r = (i * T + (int)threadIdx.x) >> 3, p = threadIdx.x & 7;
    const bool is_a = i * T / 8 < BM;
    const int rr = is_a ? r : r - BM;
    kc[i] = (p ^ (is_a ? swz_a(rr) : swz_b<NT>(rr))) * 16;
    off[i] = (uint32_t)rr * (uint32_t)g.k + kc[i];
  }
  const int k32 = (int)g.k;
  auto load = [&](int step, int buf) {
    const int kb = (first + step) * 128;
#pragma unroll
    for (int i = 0; i < LOADS; i++) {
      // past the row's end: zeros (past the last row the buffer's end does it)
      const uint32_t o = kb + kc[i] < k32 ? off[i] + kb : kOut;
      auto *dst = (__attribute__((address_space(3))) void *)(codes[buf] + (i * T + wave * 64) * 16);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(i * T / 8 < BM ? ar : br, dst, 16, o, 0, 0, 0);
    }
  };

  // scales: thread r holds row r of the tile (A rows, then B rows), clamped
  // to the matrix; bytes past a row's end repeat its last one
  const int srow = min((int)threadIdx.x, ROWS - 1);
  const uint8_t *sp = srow < BM ? g.sa + min(m0 + srow, g.m - 1) * g.nb
                                : g.sb + min(n0 + srow - BM, g.n - 1) * g.nb;
  uint32_t sw[G];
  auto load_scales = [&](int chunk) {
    const int64_t at = ((int64_t)first + 4 * chunk) * G;
    uint8_t b[4 * G];
    if (at + 4 * G <= g.nb) {
      __builtin_memcpy(b, sp + at, 4 * G);
    } else {
#pragma unroll
      for (int j = 0; j < 4 * G; j++) b[j] = sp[min(at + j, g.nb - 1)];
    }
#pragma unroll
    for (int q = 0; q < G; q++)
      sw[q] = (uint32_t)b[q] | (uint32_t)b[G + q] << 8 | (uint32_t)b[2 * G + q] << 16 |
              (uint32_t)b[3 * G + q] << 24;
  };
  auto put_scales = [&](int buf) {
    if ((int)threadIdx.x < ROWS) {
#pragma unroll
      for (int q = 0; q < G; q++) scl[buf][q][threadIdx.x] = sw[q];
    }
  };

  const int wm = wave % (BM / TM) * TM, wn = wave / (BM / TM) * TN;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[i][j] = f32x4{0, 0, 0, 0};

  load(0, 0);
  load_scales(0);
  put_scales(0);
  uint32_t as[MT][2], bs[NT][2];
  auto step = [&](int s, auto jt) {
    constexpr int J = decltype(jt)::value;
    const int buf = s & 1;
    // this step's loads have landed, and every wave is done with the other buffer
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if constexpr (J == 0) {
      const int sb = (s >> 2) & 1;
#pragma unroll
      for (int i = 0; i < MT; i++) {
        const int r = wm + 16 * i + l16;
        if constexpr (EXACT && BLK32) {
          as[i][0] = scl[sb][lg >> 1][r];
          as[i][1] = scl[sb][2 + (lg >> 1)][r];
        } else {
          as[i][0] = scl[sb][BLK32 ? lg : 0][r];
        }
      }
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const int r = BM + wn + 4 * NT * (l16 >> 2) + 4 * j + (l16 & 3);
        if constexpr (EXACT && BLK32) {
          bs[j][0] = scl[sb][lg >> 1][r];
          bs[j][1] = scl[sb][2 + (lg >> 1)][r];
        } else {
          bs[j][0] = scl[sb][BLK32 ? lg : 0][r];
        }
      }
    }
    i32x8 av[MT], bv[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int r = wn + 4 * NT * (l16 >> 2) + 4 * j + (l16 & 3);
      const uint8_t *p = codes[buf] + (BM + r) * 128;
      const int x = swz_b<NT>(r);
      bv[j] = join(*reinterpret_cast<const u32x4 *>(p + (lg ^ x) * 16),
                   *reinterpret_cast<const u32x4 *>(p + ((lg + 4) ^ x) * 16));
    }
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const int r = wm + 16 * i + l16;
      const uint8_t *p = codes[buf] + r * 128;
      const int x = swz_a(r);
      av[i] = join(*reinterpret_cast<const u32x4 *>(p + (lg ^ x) * 16),
                   *reinterpret_cast<const u32x4 *>(p + ((lg + 4) ^ x) * 16));
    }
    if (s + 1 < nk) load(s + 1, buf ^ 1);
    if constexpr (J == 0) {
      if (s + 4 < nk) load_scales((s >> 2) + 1);
    }
    if constexpr (EXACT) {
      Wide bw[NT];
#pragma unroll
      for (int j = 0; j < NT; j++)
        bw[j] = widen32(bv[j], bs[j][0] >> (8 * J) & 255, bs[j][BLK32 ? 1 : 0] >> (8 * J) & 255);
#pragma unroll
      for (int i = 0; i < MT; i++) {
        const Wide aw =
            widen32(av[i], as[i][0] >> (8 * J) & 255, as[i][BLK32 ? 1 : 0] >> (8 * J) & 255);
#pragma unroll
        for (int j = 0; j < NT; j++) acc[i][j] = mfma16(bw[j], aw, acc[i][j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++)
          acc[i][j] = mfma8<J>(bv[j], av[i], acc[i][j], bs[j][0], as[i][0]);
    }
    if constexpr (J == 3) put_scales(((s >> 2) + 1) & 1);
  };
  for (int s = 0; s < nk; s += 4) {
    step(s, std::integral_constant<int, 0>());
    if (s + 1 < nk) step(s + 1, std::integral_constant<int, 1>());
    if (s + 2 < nk) step(s + 2, std::integral_constant<int, 2>());
    if (s + 3 < nk) step(s + 3, std::integral_constant<int, 3>());
  }

  void *c = g.c;
  int out_bf16 = g.out_bf16;
  if (g.partial) {
    c = reinterpret_cast<float *>(g.c) + (int64_t)blockIdx.y * g.m * g.n;
    out_bf16 = 0;
  }
  const bool vec = g.n % (out_bf16 ? 8 : 4) == 0;
  const int64_t n = n0 + wn + 4 * NT * lg;
#pragma unroll
  for (int i = 0; i < MT; i++) {
    const int64_t m = m0 + wm + 16 * i + l16;
    if (m < g.m && n < g.n) {
      float v[4 * NT];
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) v[4 * j + e] = acc[i][j][e];
      store_run<4 * NT>(c, out_bf16, m * g.n + n, v, g.n - n, vec);
    }
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
// Up to 16 RT rows of A (single tokens, small batches): bound by reading B
// once. A workgroup owns 16 columns (rows of B) and its waves split K into
// contiguous ranges; a wave loads B's codes straight into the matrix core's
// layout (each row's 128 bytes of a step are one cache line), four steps at a
// time so that 8 KiB per wave are in flight, and A's rows come from the
// caches. The waves' sums are added in order through LDS.
template <int RT, bool BLK32, bool EXACT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_matmul8_rows(const MatArgs g) {
  constexpr int U = RT > 2 ? 2 : 4;
  __shared__ float part[WAVES][16 * RT][17];
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int all = (int)((g.k + 127) >> 7), per = (all + WAVES - 1) / WAVES;
  const int first = wave * per, last = min(all, first + per);
  const int64_t n = min(n0 + l16, g.n - 1);
  const uint8_t *bp = g.b + n * g.k, *sbp = g.sb + n * g.nb;
  const uint8_t *ap[RT], *sap[RT];
#pragma unroll
  for (int r = 0; r < RT; r++) {
    const int64_t m = min((int64_t)(16 * r + l16), g.m - 1);
    ap[r] = g.a + m * g.k;
    sap[r] = g.sa + m * g.nb;
  }
  const int64_t nb1 = g.nb - 1;
  const u32x4 zero = {0, 0, 0, 0};
  f32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; r++) acc[r] = f32x4{0, 0, 0, 0};
  for (int s = first; s < last; s += U) {
    i32x8 bv[U], av[U][RT];
    uint32_t bs[U][2], as[U][RT][2];
#pragma unroll
    for (int u = 0; u < U; u++) {
      // chunks past K (or past this wave's range) are zeros
      const int64_t k0 = (int64_t)(s + u) * 128 + 16 * lg, k1 = k0 + 64;
      const bool h0 = s + u < last && k0 < g.k, h1 = s + u < last && k1 < g.k;
      bv[u] = join(h0 ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(bp + k0)) : zero,
                   h1 ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(bp + k1)) : zero);
#pragma unroll
      for (int r = 0; r < RT; r++)
        av[u][r] = join(h0 ? *reinterpret_cast<const u32x4 *>(ap[r] + k0) : zero,
                        h1 ? *reinterpret_cast<const u32x4 *>(ap[r] + k1) : zero);
#pragma unroll
      for (int h = 0; h < (EXACT && BLK32 ? 2 : 1); h++) {
        const int64_t at = min(!BLK32 ? (int64_t)(s + u)
                                      : (int64_t)(s + u) * 4 + (EXACT ? 2 * h + (lg >> 1) : lg),
                               nb1);
        bs[u][h] = sbp[at];
#pragma unroll
        for (int r = 0; r < RT; r++) as[u][r][h] = sap[r][at];
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      if constexpr (EXACT) {
        const Wide bw = widen32(bv[u], bs[u][0], bs[u][BLK32 ? 1 : 0]);
#pragma unroll
        for (int r = 0; r < RT; r++)
          acc[r] = mfma16(bw, widen32(av[u][r], as[u][r][0], as[u][r][BLK32 ? 1 : 0]), acc[r]);
      } else {
#pragma unroll
        for (int r = 0; r < RT; r++)
          acc[r] = mfma8<0>(bv[u], av[u][r], acc[r], bs[u][0], as[u][r][0]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; r++)
#pragma unroll
    for (int e = 0; e < 4; e++) part[wave][16 * r + l16][4 * lg + e] = acc[r][e];
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * RT; i += WAVES * 64) {
    const int m = i >> 4, c = i & 15;
    if (m < g.m && n0 + c < g.n) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; w++) v += part[w][m][c];
      const int64_t at = (int64_t)m * g.n + n0 + c;
      if (g.out_bf16) reinterpret_cast<uint16_t *>(g.c)[at] = (uint16_t)pack_bf16(v, 0.0f);
      else reinterpret_cast<float *>(g.c)[at] = v;
    }
  }
}

// ---- which kernel -------------------------------------------------------------------

struct Plan {
  int rows;             // > 0: the few-rows kernel with this many row tiles
  int bm, bn;           // tile
  int splits, steps;
};

static Plan plan_of(int64_t m, int64_t n, int64_t k, int out_bf16) {
  Plan p = {0, 0, 0, 1, 0};
  const int all = (int)((k + 127) >> 7);
  if (m <= 64) {
    p.rows = m <= 16 ? 1 : m <= 32 ? 2 : 4;
    return p;
  }
  auto tiles = [&](int bm, int bn) { return ((m + bm - 1) / bm) * ((n + bn - 1) / bn); };
  if (out_bf16 && tiles(256, 256) >= 192) {
    p.bm = p.bn = 256;
  } else if (tiles(128, 128) >= 192) {
    p.bm = p.bn = 128;
  } else {
    p.bm = p.bn = 64;
  }
  p.steps = all;
  const int64_t t = tiles(p.bm, p.bn);
  // split K where the tiles leave most of the card idle, at least eight steps each
  if (t < 192) {
    int want = (int)std::min<int64_t>((384 + t - 1) / t, all / 8);
    if (want > 1) {
      p.steps = ((all + want - 1) / want + 3) & ~3;
      p.splits = (all + p.steps - 1) / p.steps;
    }
  }
  return p;
}

template <bool BLK32, bool EXACT>
static hipError_t launch(const Plan &p, MatArgs g, hipStream_t st) {
  if (p.rows) {
    const dim3 grid((uint32_t)((g.n + 15) / 16));
    if (p.rows == 1) k_matmul8_rows<1, BLK32, EXACT, 8><<<grid, 512, 0, st>>>(g);
    else if (p.rows == 2) k_matmul8_rows<2, BLK32, EXACT, 8><<<grid, 512, 0, st>>>(g);
    else k_matmul8_rows<4, BLK32, EXACT, 8><<<grid, 512, 0, st>>>(g);
    return hipGetLastError();
  }
  g.tm = (int)((g.m + p.bm - 1) / p.bm);
  g.tn = (int)((g.n + p.bn - 1) / p.bn);
  g.steps = p.steps;
  const dim3 grid((uint32_t)(g.tm * g.tn), (uint32_t)p.splits);
  if constexpr (!EXACT) {
    if (p.bm == 256) {
      k_matmul8<256, 256, 128, 64, BLK32, false><<<grid, 512, 0, st>>>(g);
      return hipGetLastError();
    }
  }
  if (p.bm == 128) k_matmul8<128, 128, 64, 64, BLK32, EXACT><<<grid, 256, 0, st>>>(g);
  else k_matmul8<64, 64, 32, 32, BLK32, EXACT><<<grid, 256, 0, st>>>(g);
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
