// mx_norm.hip - RMS norm with the residual's addition and MXFP8 output, its
// gradient, and the MXFP8 quantizer with blocks of 32 or 128 along rows and
// columns.
//
// Norm: h = x + r, y_j = w_j h_j / sqrt(sum h^2 / k + eps), then MXFP8 of y
// in blocks of 32 or 128 along the row. h enters the sum unrounded (the copy
// of it that is written is rounded to the input's type); a wave sums in fp32,
// the waves' sums and the root are in 64 bits, and y keeps what its products
// round off until the last addition: a block's scale byte changes where its
// largest value crosses a power of two, so a bit of y can be one of the byte.
// One workgroup holds one row in registers, so x, r are read once and codes,
// scales, h written once: bound by HBM.
//
// Gradient (with s = 1 / sqrt(sum h^2 / k + eps), g = w dy):
//   dx_j = s (g_j - h_j s^2 sum(g h) / k) [+ through_j]
//   dw_j = sum over rows of dy_j h_j s
// Both row sums come from one pass over registers; each workgroup walks a
// run of rows and keeps its share of dw in registers, written once as a row
// of partial sums that a second launch adds in a fixed order (no atomics).
#include "mx_layer.h"
#include "mx_layer_device.h"

namespace mxl {

// Sum of one or two values over the workgroup; every thread gets the same
// bits. `part` is this call's own LDS (two calls in flight alternate).
template <int T>
__device__ __forceinline__ f32x2 block_sum2(float a, float b, f32x2 *part) {
  a = sum64(a);
  b = sum64(b);
  if constexpr (T == 64) return f32x2{a, b};
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = f32x2{a, b};
  __syncthreads();
  f32x2 t = part[0];
#pragma unroll
  for (int i = 1; i < T / 64; i++) {
    t.x += part[i].x;
    t.y += part[i].y;
  }
  return t;
}

// The same for one value, added up in 64 bits from the waves' sums on.
template <int T>
__device__ __forceinline__ double block_sum(float a, float *part) {
  a = sum64(a);
  if constexpr (T == 64) return a;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
  __syncthreads();
  double t = part[0];
#pragma unroll
  for (int i = 1; i < T / 64; i++) t += part[i];
  return t;
}

// The same of a value that is in 64 bits from the start.
template <int T>
__device__ __forceinline__ double block_sum64(double a, double *part) {
#pragma unroll 1
  for (int d = 1; d < 64; d <<= 1) a += __shfl_xor(a, d);
  if constexpr (T == 64) return a;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
  __syncthreads();
  double t = part[0];
#pragma unroll 1  // few registers: rare, and beside rows held in all the others
  for (int i = 1; i < T / 64; i++) t += part[i];
  return t;
}

// Whether a sum of squares in 32 bits is none to go by: squares overflowed, or
// are so small that bits of them, or of their products with a gradient, may
// have been lost (`floor`: what is added to the sum).
__device__ __forceinline__ bool out_of_range(float sum, float floor) {
  return !(sum < 0x1p127f) || sum + floor < 0x1p-40f;
}

// T threads of N items (eight elements) hold a row. 8191 x 8192 bf16 with a
// residual, blocks of 32: 75 us, 6.3 TB/s of 7 bytes an element; 5 x 4096,
// where one trip to memory and one sum are all there is: 3.4 us.
template <bool BF16, int T, int N>
__global__ __launch_bounds__(T) void k_rmsnorm(const void *x, const void *residual,
                                               const void *__restrict__ weight, int64_t rows, int k, float eps,
                                               int wide, uint8_t *__restrict__ codes,
                                               uint8_t *__restrict__ scales, void *h) {
  __shared__ float part[T / 64];
  __shared__ double part64[T / 64];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= rows) return;
  const int items = k >> 3;
  const int64_t base = row * items;
  Raw<BF16> xr[N], rr[N], wr[N];
#pragma unroll
  for (int u = 0; u < N; u++) {
    const int it = threadIdx.x + u * T;
    if (it < items) {
      xr[u] = load_raw<BF16>(x, base + it);
      if (residual) rr[u] = load_raw<BF16>(residual, base + it);
    }
  }
#pragma unroll
  for (int u = 0; u < N; u++) {  // the weight stays in the caches: default policy
    const int it = threadIdx.x + u * T;
    if (it < items) {
      const u32x4 *p = reinterpret_cast<const u32x4 *>(weight) + (BF16 ? 1 : 2) * it;
      wr[u].v[0] = p[0];
      if constexpr (!BF16) wr[u].v[1] = p[1];
    }
  }
  float f[N][8], ss = 0.0f;
#pragma unroll
  for (int u = 0; u < N; u++) {
    const int it = threadIdx.x + u * T;
    if (it < items) {
      widen<BF16>(xr[u], f[u]);
      if (residual) {
        float r[8];
        widen<BF16>(rr[u], r);
#pragma unroll
        for (int j = 0; j < 8; j++) f[u][j] += r[j];
        if (h) store8<BF16>(h, base + it, f[u]);
      }
#pragma unroll
      for (int j = 0; j < 8; j++) ss = __builtin_fmaf(f[u][j], f[u][j], ss);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) f[u][j] = 0.0f;
    }
  }
  double sum = block_sum<T>(ss, part);
  int up = 0;  // the row is held times 2^up
  if (__builtin_expect(out_of_range((float)sum, eps * k), 0)) {
    // the same for the whole workgroup: the sum again in 64 bits, whose root
    // decides the power of two that brings the row near 1
    double wide = 0.0;
#pragma unroll
    for (int u = 0; u < N; u++)
#pragma unroll
      for (int j = 0; j < 8; j++) wide += (double)f[u][j] * f[u][j];
    sum = block_sum64<T>(wide, part64);
    const double mean = sum / k + eps;
    if (mean > 0.0 && mean < __builtin_inf()) {  // neither zeros, NaN nor infinities
      up = -(__builtin_amdgcn_frexp_exp(mean) / 2);
#pragma unroll
      for (int u = 0; u < N; u++)
#pragma unroll
        for (int j = 0; j < 8; j++) f[u][j] = __builtin_ldexpf(f[u][j], up);
    }
  }
  const double exact = __builtin_ldexp(1.0 / __builtin_sqrt(sum / k + eps), -up);
  const float s = (float)exact, s_low = (float)(exact - s);
  const int lanes = wide ? 16 : 4;  // lanes that share a block (wave-uniform)
  const int64_t nb = (items + lanes - 1) / lanes;
#pragma unroll
  for (int u = 0; u < N; u++) {
    const int it = threadIdx.x + u * T;
    float y[8];
    uint32_t m = 0;
    if (it < items) {
      float w[8];
      widen<BF16>(wr[u], w);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float n = f[u][j] * s;
        const float low = __builtin_fmaf(f[u][j], s, -n) + f[u][j] * s_low;
        y[j] = __builtin_fmaf(n, w[j], low * w[j]);
      }
      m = amax8(y);
      if (m >= 0x7F800000u) {  // infinities: their low parts are NaN
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = f[u][j] * s * w[j];
        m = amax8(y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) y[j] = 0.0f;
    }
    // lanes past the row's end take part with zeros: they may sit in the
    // last, short block
    m = wide ? max16(m) : max4(m);
    if (it < items) {
      const uint32_t sb = scale_byte8(m);
      reinterpret_cast<u32x2 *>(codes)[base + it] = encode8(y, sb);
      if ((it & (lanes - 1)) == 0) scales[row * nb + it / lanes] = (uint8_t)sb;
    }
  }
}

// Bound by HBM: 8192 x 4096 bf16 with a second gradient, 46 to 48 us (5.7 TB/s
// of 8 bytes an element) and 4 for the sum of 512 partial rows; 8192 x 8192
// 93 us. Rows of more than 16,384 elements do not fit the registers whole: 2048
// x 32768 209 us (2.6 TB/s), fp32 491; fp32 4096 x 12288, which does, 158.
template <bool BF16, int T, int N>
__global__ __launch_bounds__(T) void k_rmsnorm_backward(
    const void *dy, const void *h, const void *__restrict__ weight, const void *through,
    int64_t rows, int k, float eps, void *dx, float *__restrict__ partial) {
  // One item a thread: the next row is loaded while this one is summed and
  // written. More take the registers for their own row and widen them, and
  // read the weight again (from the caches), at each use.
  constexpr bool AHEAD = N == 1;
  __shared__ f32x2 part[2][T / 64];
  __shared__ double part64[2][T / 64];
  const int items = k >> 3;
  Raw<BF16> dr[N], hr[N], tr[N], wr[N];
  auto fetch = [&](const void *from, int64_t row, Raw<BF16> (&to)[N]) {
#pragma unroll
    for (int u = 0; u < N; u++) {
      const int it = threadIdx.x + u * T;
      if (it < items) to[u] = load_raw<BF16>(from, row * items + it);
    }
  };
  float dw[N][8];
#pragma unroll
  for (int u = 0; u < N; u++) {
#pragma unroll
    for (int j = 0; j < 8; j++) dw[u][j] = 0.0f;
    wr[u] = dr[u] = hr[u] = tr[u] = Raw<BF16>{};
  }
  const float inv_k = 1.0f / (float)k;
  if (AHEAD) {
    fetch(weight, 0, wr);
    fetch(dy, blockIdx.x, dr);
    fetch(h, blockIdx.x, hr);
    if (through) fetch(through, blockIdx.x, tr);
  }
  int flip = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, flip ^= 1) {
    const int64_t next = row + gridDim.x;
    if (!AHEAD) {
      fetch(dy, row, dr);
      fetch(h, row, hr);
      fetch(weight, 0, wr);
      if (through) fetch(through, row, tr);
    }
    float ss = 0.0f, sg = 0.0f;
    Raw<BF16> d[N], g[N];  // of this row; past its end zeros
#pragma unroll
    for (int u = 0; u < N; u++) {
      d[u] = dr[u];
      g[u] = hr[u];
      float dv[8], hv[8], w[8];
      widen<BF16>(d[u], dv);
      widen<BF16>(g[u], hv);
      widen<BF16>(wr[u], w);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        ss = __builtin_fmaf(hv[j], hv[j], ss);
        sg = __builtin_fmaf(dv[j] * w[j], hv[j], sg);
      }
    }
    if (AHEAD && next < rows) {
      fetch(dy, next, dr);
      fetch(h, next, hr);
    }
    // alternate halves of `part`: a wave may still be reading the last row's
    const f32x2 t = block_sum2<T>(ss, sg, part[flip]);
    float s = 1.0f / __builtin_sqrtf(t.x * inv_k + eps);
    float c = t.y * inv_k * s * s;
    const bool lost = __builtin_fabsf(t.y) < 0x1p-80f && t.y != 0.0f;
    if (__builtin_expect(out_of_range(t.x, eps * k) || !(__builtin_fabsf(t.y) < 0x1p127f) || lost, 0)) {
      // the same for the whole workgroup: the sums again in 64 bits, element by
      // element from memory, which costs other rows no registers. s and c
      // themselves are in range wherever the results are: s h is about 1.
      double sh = 0.0, sgh = 0.0;
      int start = threadIdx.x, count = k;
      float more = eps;
      // unknown to the compiler, which would make addresses and quotients ahead
      // of all rows and hold them
      asm volatile("" : "+v"(start), "+s"(count), "+s"(more));
#pragma unroll 1
      for (int e = start; e < count; e += T) {
        const double hv = load_one<BF16>(h, row * k + e);
        sh += hv * hv;
        sgh += (double)load_one<BF16>(dy, row * k + e) * load_one<BF16>(weight, e) * hv;
      }
      const double mean = block_sum64<T>(sh, part64[0]) / count + more;
      s = (float)(1.0 / __builtin_sqrt(mean));
      c = (float)(block_sum64<T>(sgh, part64[1]) / count / mean);
    }
#pragma unroll
    for (int u = 0; u < N; u++) {
      const int it = threadIdx.x + u * T;
      if (it < items) {
        float dv[8], hv[8], w[8], o[8], th[8];
        if (!AHEAD && (BF16 || N < 4)) {  // widened again: what the sums widened is not held for this
          renew<BF16>(d[u]);
          renew<BF16>(g[u]);
          renew<BF16>(wr[u]);
        }
        widen<BF16>(d[u], dv);
        widen<BF16>(g[u], hv);
        widen<BF16>(wr[u], w);
        if (through) widen<BF16>(tr[u], th);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          o[j] = s * __builtin_fmaf(-hv[j], c, dv[j] * w[j]);
          if (through) o[j] += th[j];
          dw[u][j] = __builtin_fmaf(dv[j], hv[j] * s, dw[u][j]);
        }
        store8<BF16>(dx, row * items + it, o);
      }
    }
    if (AHEAD && through && next < rows) fetch(through, next, tr);
  }
#pragma unroll
  for (int u = 0; u < N; u++) {
    const int it = threadIdx.x + u * T;
    if (it < items) {
      f32x4 *p = reinterpret_cast<f32x4 *>(partial + (int64_t)blockIdx.x * k) + 2 * it;
      p[0] = f32x4{dw[u][0], dw[u][1], dw[u][2], dw[u][3]};
      p[1] = f32x4{dw[u][4], dw[u][5], dw[u][6], dw[u][7]};
    }
  }
}

// dweight_j = sum over the n partial rows: 16 columns per workgroup, thread
// (r, c) adds rows r, r + 16, ... of column c, then the 16 sums in order.
__global__ __launch_bounds__(256) void k_sum_rows(const float *__restrict__ partial, int n, int k,
                                                  float *__restrict__ out) {
  __shared__ float part[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;  // k is a multiple of 32: every column exists
  float a[8] = {0, 0, 0, 0, 0, 0, 0, 0};  // independent: the loads of a round go together
  int i = r;
  for (; i + 7 * 16 < n; i += 8 * 16)
#pragma unroll
    for (int q = 0; q < 8; q++) a[q] += partial[(int64_t)(i + 16 * q) * k + col];
  for (; i < n; i += 16) a[0] += partial[(int64_t)i * k + col];
  part[r][c] = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
  __syncthreads();
  if (r == 0) {
    float t = 0.0f;
#pragma unroll
    for (int q = 0; q < 16; q++) t += part[q][c];
    out[col] = t;
  }
}

// ---- quantizer: blocks along rows and along columns from one read -----------------
//
// A workgroup takes a tile of 128 rows x 128 columns. Rows: thread t holds
// item t % 16 (eight columns) of rows t / 16 + 16 u; a block of 128 is 16
// lanes, one of 32 is four. Columns: the tile goes through LDS (bf16 pairs
// or floats) and thread t takes rows 8 (t % 16) .. + 7 of columns, so that
// again 16 or 4 lanes share a block. Rows past the end count as zeros; the
// transposed codes of a ragged last 32 rows are written as zeros.
//
// Bound by HBM when large: 8192 x 8192 bf16 both ways 53 us (5.1 TB/s), fp32
// 77 us; 4099 x 1536 9.4 us. 1,024 threads: a tile is one round of loads, so
// more of them means more in flight (256 threads: 62, 106 and 11 us). Tiles
// next to each other along a row run together (along a column: 57, 87, 9.4).
constexpr int kQuantThreads = 1024;
template <bool BF16>
__global__ __launch_bounds__(kQuantThreads) void k_quantize8_blocks(
    const void *__restrict__ x, int64_t rows, int64_t k, int wide, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales, uint8_t *__restrict__ codes_t, uint8_t *__restrict__ scales_t) {
  // 65 (129) words per row: the transposed reads, 8 rows apart, spread over the banks
  constexpr int P = BF16 ? 65 : 129, RS = kQuantThreads / 16, U = 128 / RS;
  __shared__ uint32_t tile[128 * P];
  const int64_t r0 = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 128, c0 = (int64_t)blockIdx.x * 128;
  if (r0 >= rows) return;
  const int q = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int lanes = wide ? 16 : 4;
  const int64_t col = c0 + 8 * q;
  const bool in_k = col < k;  // k is a multiple of 32: items are whole
  const int64_t nb = (k + 8 * lanes - 1) / (8 * lanes);
  Raw<BF16> raw[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t row = r0 + r + RS * u;
    if (in_k && row < rows) {
      raw[u] = load_raw<BF16>(x, (row * k + col) >> 3);
    } else {
      raw[u].v[0] = u32x4{0, 0, 0, 0};
      if constexpr (!BF16) raw[u].v[1] = u32x4{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t row = r0 + r + RS * u;
    if (codes_t) {
      uint32_t *d = tile + (r + RS * u) * P + (BF16 ? 4 : 8) * q;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        d[j] = raw[u].v[0][j];
        if constexpr (!BF16) d[4 + j] = raw[u].v[1][j];
      }
    }
    if (codes) {
      float f[8];
      widen<BF16>(raw[u], f);
      uint32_t m = amax8(f);
      m = wide ? max16(m) : max4(m);
      if (in_k && row < rows) {
        const uint32_t sb = scale_byte8(m);
        *reinterpret_cast<u32x2 *>(codes + row * k + col) = encode8(f, sb);
        if ((q & (lanes - 1)) == 0) scales[row * nb + col / (8 * lanes)] = (uint8_t)sb;
      }
    }
  }
  if (!codes_t) return;
  __syncthreads();
  const int64_t rows_p = (rows + 31) & ~(int64_t)31;
  const int64_t row = r0 + 8 * q;
  const int64_t nbt = (rows + 8 * lanes - 1) / (8 * lanes);
#pragma unroll
  for (int u = 0; u < (BF16 ? U / 2 : U); u++) {
    // columns c (and c + 1 of the same word for bf16)
    const int c = BF16 ? 2 * (r + RS * u) : r + RS * u;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; j++) w[j] = tile[(8 * q + j) * P + (BF16 ? c >> 1 : c)];
#pragma unroll
    for (int e = 0; e < (BF16 ? 2 : 1); e++) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; j++)
        f[j] = __uint_as_float(!BF16 ? w[j] : e ? (w[j] & 0xFFFF0000u) : (w[j] << 16));
      uint32_t m = amax8(f);
      m = wide ? max16(m) : max4(m);
      const int64_t cc = c0 + c + e;
      if (cc < k && row < rows_p) {
        const uint32_t sb = scale_byte8(m);
        *reinterpret_cast<u32x2 *>(codes_t + cc * rows_p + row) = encode8(f, sb);
        if ((q & (lanes - 1)) == 0) scales_t[cc * nbt + row / (8 * lanes)] = (uint8_t)sb;
      }
    }
  }
}

// Threads and items per thread that hold a row of `items` items. Few rows:
// as many threads as there are items (latency); many rows: up to `per` items
// for a thread.
struct Shape {
  int t, n;
};
static Shape row_shape(int64_t items, int per) {
  for (int t = 64; t <= 1024; t *= 2) {
    if (items <= t && (t == 64 || per == 1)) return {t, 1};
    if (items <= (int64_t)t * per) return {t, per};
  }
  int n = per;
  while ((int64_t)1024 * n < items) n *= 2;
  return {1024, n};
}

// FOUR: also the shapes that row_shape(.., 4) gives.
template <bool FOUR, typename F>
static hipError_t with_shape(Shape s, F f) {
  auto at = [&](auto t) {
    if constexpr (FOUR)
      if (s.n == 4) return f(t, std::integral_constant<int, 4>());
    return f(t, std::integral_constant<int, 1>());
  };
  switch (s.t) {
    case 64: return at(std::integral_constant<int, 64>());
    case 128: return at(std::integral_constant<int, 128>());
    case 256: return at(std::integral_constant<int, 256>());
    case 512: return at(std::integral_constant<int, 512>());
  }
  constexpr std::integral_constant<int, 1024> t;
  switch (s.n) {
    case 1: return f(t, std::integral_constant<int, 1>());
    case 2: return f(t, std::integral_constant<int, 2>());
    case 4: return f(t, std::integral_constant<int, 4>());
    default: return f(t, std::integral_constant<int, 8>());
  }
}

}  // namespace mxl

using namespace mxl;

hipError_t mxi_launch_rmsnorm(const void *x, const void *residual, const void *weight, int bf16,
                              int64_t rows, int64_t k, float eps, int block, uint8_t *codes,
                              uint8_t *scales, void *h, hipStream_t st) {
  // one item a thread and four: 5 x 4096 3.0 and 4.1 us, 512 x 4096 5.4 and 6.2,
  // 1024 x 4096 8.2 and 7.9, 8191 x 8192 92 and 78
  const Shape s = row_shape(k / 8, rows < 768 ? 1 : 4);
  // a grid's dimension holds fewer than 2^32 threads
  const int64_t across = rows < (1 << 21) ? rows : 1 << 21;
  const dim3 grid((uint32_t)across, (uint32_t)((rows + across - 1) / across));
  auto go = [&](auto bf) {
    return with_shape<true>(s, [&](auto t, auto n) {
      k_rmsnorm<decltype(bf)::value, decltype(t)::value, decltype(n)::value>
          <<<grid, dim3(decltype(t)::value), 0, st>>>(
              x, residual, weight, rows, (int)k, eps, block == 128, codes, scales, h);
      return hipGetLastError();
    });
  };
  return bf16 ? go(std::true_type()) : go(std::false_type());
}

int64_t mxi_rmsnorm_partials(int64_t rows, int64_t k) {
  const Shape s = row_shape(k / 8, 1);
  // 1,024 threads per compute unit; on 8192 x 4096 with a residual, 54 us
  // (1,536: 57, 2,048: 61; two items a thread and 1,024: 77)
  const int64_t most = (int64_t)256 * (1024 / s.t);
  return rows < most ? rows : most;
}

hipError_t mxi_launch_rmsnorm_backward(const void *dy, const void *h, const void *weight,
                                       const void *through, int bf16, int64_t rows, int64_t k,
                                       float eps, void *dx, float *dweight, float *partial,
                                       hipStream_t st) {
  const Shape s = row_shape(k / 8, 1);
  const int64_t grid = mxi_rmsnorm_partials(rows, k);
  auto go = [&](auto bf) {
    return with_shape<false>(s, [&](auto t, auto n) {
      k_rmsnorm_backward<decltype(bf)::value, decltype(t)::value, decltype(n)::value>
          <<<dim3((uint32_t)grid), dim3(decltype(t)::value), 0, st>>>(
              dy, h, weight, through, rows, (int)k, eps, dx, partial);
      return hipGetLastError();
    });
  };
  if (grid > 0) {
    const hipError_t e = bf16 ? go(std::true_type()) : go(std::false_type());
    if (e != hipSuccess) return e;
  }
  k_sum_rows<<<dim3((uint32_t)(k / 16)), dim3(256), 0, st>>>(partial, (int)grid, (int)k, dweight);
  return hipGetLastError();
}

hipError_t mxi_launch_quantize8_blocks(const void *x, int bf16, int64_t rows, int64_t k, int block,
                                       uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                                       uint8_t *scales_t, hipStream_t st) {
  // tiles down over two dimensions of the grid, of which one is short
  const int64_t down = (rows + 127) / 128, y = down < 32768 ? down : 32768;
  const dim3 grid((uint32_t)((k + 127) / 128), (uint32_t)y, (uint32_t)((down + y - 1) / y));
  if (bf16)
    k_quantize8_blocks<true><<<grid, kQuantThreads, 0, st>>>(x, rows, k, block == 128, codes, scales, codes_t,
                                                   scales_t);
  else
    k_quantize8_blocks<false><<<grid, kQuantThreads, 0, st>>>(x, rows, k, block == 128, codes, scales,
                                                    codes_t, scales_t);
  return hipGetLastError();
}
