// mx_kv.hip - a paged key/value cache in 8 bits and the attention that reads it.
//
// Cache: keys [page, head, token, dim], values [page, head, dim, token] (so
// that both products read 16 codes at once along their summed dimension),
// E4M3, one E8M0 byte per page and head for each of the two.
//
// Append. A page's byte is the largest of what its kept tokens have and what
// the new tokens need; where it grows, the kept codes are re-rounded to it.
// One workgroup per (sequence's page, head).
//
// Attention, o = sum_j softmax_j(scale q.k_j) v_j, takes the cache's keys to
// the 8-bit matrix cores as they are: v_mfma_scale_f32_16x16x128_f8f6f4
// multiplies codes and bytes. q is split into two E4M3 numbers, x = hi + lo,
// whose products land in the same accumulator. They hold all eight significant
// bits of an element above 2^-13 of the row's largest one; lo's smallest step
// lies 2^-20 below that one. (Inside a group of eight products the matrix core
// drops bits more than about 2^-14 below the group's largest.) Scores are taken transposed (tokens are the accumulator's
// rows), so that the weights p come out in the very lanes and order in which
// the second product wants them. Maxima, sums and accumulators are fp32.
//
// The second product is a bfloat16 one: values are widened to it (exact, their
// bytes applied), weights rounded to it, which moves each by at most 2^-9 of
// itself however far below the largest it lies. (Two E4M3 parts, as q has,
// end 2^-22 below the largest weight: a tail of many such keys is lost.) The
// weights' sum is a product with a row of ones, of the weights as rounded.
//
// Two kernels. Few rows (single tokens) are bound by reading the cache: one
// wave per 128 tokens at a time, the sequence split over workgroups. With
// g = lane / 16, tile t (of 16 rows) and accumulator i hold token 64 (t / 4) +
// 16 g + 4 (t % 4) + i of 128, and the second product's lane holds tokens
// 16 g .. + 15 and 64 + 16 g .. + 15.
//
// Many rows (prompts) share tiles of 128 tokens through LDS and are bound by
// instruction issue: per 32 rows and 128 tokens, 2,200 cycles of products
// beside 2,400 of vector arithmetic, half of it the exponentials. There the
// workgroup widens the values once. Token 32 (t / 2) + 8 g + 4 (t % 2) + i.
#include <algorithm>

#include "mx_layer.h"
#include "mx_layer_device.h"

namespace mxl {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int clamp_page(int32_t id, int64_t pages) {
  return (int)min((uint32_t)id, (uint32_t)(pages - 1));
}

// ---- append -------------------------------------------------------------------------

struct AppendArgs {
  const void *k, *v;
  int64_t k_stride, v_stride;  // elements between tokens
  mx_kv_cache_t c;
  mx_kv_batch_t b;
  int shift;        // log2(page)
  uint32_t blocks;  // units times heads
};

// Which sequence a unit of work belongs to: sequence i owns units from
// cu[i] / per + extra i on, which leaves it at least n / per + extra. The
// wave's lanes look at up to 64 sequences at once (one trip to memory for up
// to 64 sequences, two up to 4096).
__device__ __forceinline__ int find_sequence(const int32_t *cu, int batch, int per, int extra,
                                             int unit) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 63) >> 6, at = lo + lane * step;
    const bool below = lane * step < n && cu[at] / per + extra * at <= unit;
    // the lanes that hold are the first ones; sequence lo always does
    const int skip = max((int)__popcll(__ballot(below)) - 1, 0) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Four codes moved from scale byte s to s + d (d > 0), or to a NaN block.
__device__ __forceinline__ uint32_t move4(uint32_t w, int d, bool nan) {
  if (nan) return w & 0x80808080u;
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_ldexpf(a.x, -d), __builtin_ldexpf(a.y, -d), 0,
                                          false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_ldexpf(b.x, -d), __builtin_ldexpf(b.y, -d), r, true);
  return (uint32_t)r;
}

// Items of eight elements that a thread keeps between the two passes (what a
// page of 64 tokens of 128 dims takes); larger pages read the rest twice.
constexpr int kKeep = 4;

// One workgroup per page and head. Prompts are bound by HBM: 6 sequences of up
// to 8,000 tokens, 8 heads of 128, 201 MB in 41 us (4.9 TB/s); with the values'
// bytes written to LDS one at a time 44.6, with the tokens read twice 72. A
// token per sequence is a chain of loads that wait for each other (cu, table
// and lengths, scale, codes): 64 sequences 5 us, 256 8.5.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_at(const void *base, int64_t elem) {
  return load_raw<BF16>(reinterpret_cast<const uint8_t *>(base) + elem * (BF16 ? 2 : 4), 0);
}

template <bool BF16, int T>
__global__ __launch_bounds__(T) void k_kv_append(const AppendArgs a) {
  // new values' codes, [dim][token]; rows are one word longer than a page's,
  // so that the rows that an instruction writes to fall on different banks
  extern __shared__ __attribute__((aligned(16))) uint8_t vt[];
  __shared__ uint32_t am[2][T / 64];
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= a.blocks) return;
  const int unit = block / a.c.heads, head = block % a.c.heads;
  const int P = a.c.page, D = a.c.dim;
  const int i = find_sequence(a.b.cu, a.b.batch, P, 2, unit);
  const int c0 = a.b.cu[i], n = a.b.cu[i + 1] - c0, held = a.b.lengths[i];
  const int j = (held >> a.shift) + (unit - (c0 / P + 2 * i));  // page of the sequence
  // (a unit before the first sequence's has pages before the sequence's first)
  if (n <= 0 || held < 0 || j < held >> a.shift || j >= a.b.width || ((int64_t)j << a.shift) >= (int64_t)held + n)
    return;
  const int kept = max(0, held - (j << a.shift));            // slots that stay
  const int end = min((int64_t)P, (int64_t)held + n - ((int64_t)j << a.shift));  // slots in use after
  const int64_t id = a.b.table[(int64_t)i * a.b.width + j];
  if (id < 0 || id >= a.c.pages) return;  // no page: its tokens are dropped
  const int64_t src0 = (int64_t)c0 + ((int64_t)j << a.shift) - held;  // token of slot 0
  const int64_t most = a.b.tokens - 1;
  const int64_t at = id * a.c.heads + head;
  // An item is eight dims of a token. Lanes l, l + 16, l + 32, l + 48 of a wave
  // hold four tokens that share a word of a values' row.
  const int wide = D == 128, first = kept & ~3;
  uint32_t was_k = 0, was_v = 0;
  if (kept) {
    was_k = a.c.k_scales[at];
    was_v = a.c.v_scales[at];
  }
  auto word_of = [&](int it) {  // first of the four slots
    return first + (wide ? it >> 6 << 2 : (it >> 6 << 3) + ((it & 8) >> 1));
  };
  auto slot_of = [&](int it) { return word_of(it) + ((it >> 4) & 3); };
  auto dim_of = [&](int it) { return (it & (wide ? 15 : 7)) * 8; };
  // whether any lane of the wave has a slot in use: the wave's lanes go together
  auto any = [&](int it) { return first + (wide ? it >> 6 << 2 : it >> 6 << 3) < end; };
  auto mine = [&](int it) { return slot_of(it) >= kept && slot_of(it) < end; };
  auto load = [&](const void *x, int64_t stride, int it) {
    const int64_t tok = min(max(src0 + slot_of(it), (int64_t)0), most);
    return load_at<BF16>(x, tok * stride + (int64_t)head * D + dim_of(it));
  };

  Raw<BF16> kr[kKeep], vr[kKeep];
#pragma unroll
  for (int u = 0; u < kKeep; u++) {
    const int it = threadIdx.x + T * u;
    kr[u] = vr[u] = Raw<BF16>{};
    if (mine(it)) {
      kr[u] = load(a.k, a.k_stride, it);
      vr[u] = load(a.v, a.v_stride, it);
    }
  }
  uint32_t mk = 0, mv = 0;
  auto take = [&](const Raw<BF16> &k, const Raw<BF16> &v) {
    float f[8];
    widen<BF16>(k, f);
    mk = max(mk, amax8(f));
    widen<BF16>(v, f);
    mv = max(mv, amax8(f));
  };
#pragma unroll
  for (int u = 0; u < kKeep; u++) take(kr[u], vr[u]);  // zeros where there is none
  for (int it = threadIdx.x + T * kKeep; any(it); it += T)
    if (mine(it)) take(load(a.k, a.k_stride, it), load(a.v, a.v_stride, it));
  mk = max16(mk);
  mv = max16(mv);
  mk = max(mk, (uint32_t)__shfl_xor((int)mk, 16));
  mv = max(mv, (uint32_t)__shfl_xor((int)mv, 16));
  mk = max(mk, (uint32_t)__shfl_xor((int)mk, 32));
  mv = max(mv, (uint32_t)__shfl_xor((int)mv, 32));
  if ((threadIdx.x & 63) == 0) {
    am[0][threadIdx.x >> 6] = mk;
    am[1][threadIdx.x >> 6] = mv;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; w++) {
    mk = max(mk, am[0][w]);
    mv = max(mv, am[1][w]);
  }
  const uint32_t sk = max(scale_byte8(mk), was_k), sv = max(scale_byte8(mv), was_v);
  uint8_t *kc = a.c.k_codes + at * P * D, *vc = a.c.v_codes + at * P * D;
  // kept codes move to the new bytes 16 at a time, four such pieces asked for
  // together; what a piece holds past the kept tokens stays
  auto move = [&](int pieces, auto place, auto keeps, int d, bool nan) {
    for (int c = threadIdx.x; c < pieces; c += 4 * T) {
      u32x4 v[4];
#pragma unroll
      for (int u = 0; u < 4; u++) v[u] = *reinterpret_cast<const u32x4 *>(place(min(c + u * T, pieces - 1)));
#pragma unroll
      for (int u = 0; u < 4; u++) {
        if (c + u * T >= pieces) break;
        const int keep = keeps(c + u * T);
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int n = min(max(keep - 4 * e, 0), 4);
          const uint32_t mask = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1;
          w[e] = (move4(v[u][e], d, nan) & mask) | (v[u][e] & ~mask);
        }
        *reinterpret_cast<u32x4 *>(place(c + u * T)) = w;
      }
    }
  };
  if (kept && sk > was_k)
    move(kept * D / 16, [&](int c) { return kc + 16 * c; }, [](int) { return 16; }, (int)(sk - was_k), sk == 255u);
  if (kept && sv > was_v) {
    const int n = (kept + 15) >> 4;
    move(D * n, [&](int c) { return vc + c / n * P + c % n * 16; },
         [&](int c) { return kept - c % n * 16; }, (int)(sv - was_v), sv == 255u);
    __syncthreads();  // before the new tokens' bytes of the same words
  }
  // a kept byte may be any: above 246 every finite number is below 448 scales
  auto limit = [](uint32_t b) { return b > 246u ? 0x1.fffffep127f : limit8(b); };
  const float most_k = limit(sk), most_v = limit(sv);
  const int row = P + 4;
  auto put = [&](const Raw<BF16> &k, const Raw<BF16> &v, int it) {
    float f[8];
    if (mine(it)) {
      widen<BF16>(k, f);
      *reinterpret_cast<u32x2 *>(kc + slot_of(it) * D + dim_of(it)) = encode8(f, sk, most_k);
    }
    widen<BF16>(v, f);
    const u32x2 w = encode8(f, sv, most_v);
    // four lanes' tokens t = 2 b + a, eight dims each, become two dims of four
    // tokens: halves of the dims change places over b, then quarters over a
    const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
    const uint32_t lo = __builtin_amdgcn_perm(x[1], x[0], 0x05040100u);  // dims 0, 1 of tokens a, a + 2
    const uint32_t hi = __builtin_amdgcn_perm(x[1], x[0], 0x07060302u);  // dims 2, 3
    const auto y = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
    uint32_t *to = reinterpret_cast<uint32_t *>(vt + (dim_of(it) + 2 * ((it >> 4) & 3)) * row + word_of(it));
    to[0] = __builtin_amdgcn_perm(y[1], y[0], 0x06020400u);
    to[row >> 2] = __builtin_amdgcn_perm(y[1], y[0], 0x07030501u);
  };
#pragma unroll
  for (int u = 0; u < kKeep; u++)
    if (any(threadIdx.x + T * u)) put(kr[u], vr[u], threadIdx.x + T * u);
  for (int it = threadIdx.x + T * kKeep; any(it); it += T)
    put(load(a.k, a.k_stride, it), load(a.v, a.v_stride, it), it);
  __syncthreads();
  const int piece0 = kept >> 4, chunks = ((end + 15) >> 4) - piece0;  // of a row, with new tokens in them
  for (int it = threadIdx.x; it < D * chunks; it += T) {
    const int d = it / chunks, s = (piece0 + it % chunks) * 16;
    const int lo = max(kept, s), hi = min(end, s + 16);
    uint8_t *dst = vc + (int64_t)d * P;
    if (lo == s && hi == s + 16) {
      const uint32_t *from = reinterpret_cast<const uint32_t *>(vt + d * row + s);
      *reinterpret_cast<u32x4 *>(dst + s) = u32x4{from[0], from[1], from[2], from[3]};
    } else {
      for (int q = lo; q < hi; q++) dst[q] = vt[d * row + q];
    }
  }
  if (threadIdx.x == 0) {
    if (!kept || sk != was_k) a.c.k_scales[at] = (uint8_t)sk;
    if (!kept || sv != was_v) a.c.v_scales[at] = (uint8_t)sv;
  }
}

// ---- attention ----------------------------------------------------------------------

struct AttnArgs {
  const uint16_t *q;
  int64_t q_stride;
  int q_heads, group;
  mx_kv_cache_t c;
  mx_kv_batch_t b;
  int shift;
  int block_tokens;  // tokens of a workgroup's block of rows
  int chunk;         // kv tiles (of 128 tokens) per split
  int splits, units;
  float scale2;      // softmax scale times log2(e)
  uint16_t *out;
  float *part;       // [token, q head, split][dim + 2]: sums, then maximum and total
};

__device__ __forceinline__ i32x8 join8(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
// D += A B^T over 128 elements; A's scale is byte JA of sa, B's byte JB of sb.
template <int JA, int JB>
__device__ __forceinline__ f32x4 mma(i32x8 a, i32x8 b, f32x4 d, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, 0, 0, JA, (int)sa, JB, (int)sb);
}

// D += A B^T over 32 bf16 elements.
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 d) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), d, 0, 0, 0);
}

// A row of q as the second operand: hi and lo, each 32 codes (dim 128), or
// hi in the first 16 bytes and lo in the second (dim 64, where one product
// of length 128 takes both against the keys' codes given twice). Byte i of
// `bytes` is the E8M0 byte of v[i]; lo's is 4 below hi's.
template <int D>
struct Query {
  i32x8 v[D / 64];
  uint32_t bytes;
};

__device__ __forceinline__ void split4(const float (&x)[4], float to, float back, uint32_t &hi,
                                       uint32_t &lo) {
  s16x2 h = {0, 0}, l = {0, 0};
  h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, x[0], x[1], to, false);
  h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, x[2], x[3], to, true);
  hi = __builtin_bit_cast(uint32_t, h);
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, to, false);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, to, true);
  l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, x[0] - a.x, x[1] - a.y, back, false);
  l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, x[2] - b.x, x[3] - b.y, back, true);
  lo = __builtin_bit_cast(uint32_t, l);
}

template <int D>
__device__ __forceinline__ Query<D> load_query(const uint16_t *row, int lg) {
  float f[D / 64][16];
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < D / 64; h++) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(row + 64 * h + 16 * lg);
    const u32x4 w[2] = {p[0], p[1]};
#pragma unroll
    for (int j = 0; j < 16; j++) {
      const uint32_t x = w[j >> 3][(j >> 1) & 3];
      f[h][j] = __uint_as_float((j & 1) ? (x & 0xFFFF0000u) : (x << 16));
      m = max(m, __float_as_uint(f[h][j]) & 0x7FFFFFFFu);
    }
  }
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  // the row's largest lands in [128, 256); NaN or infinity makes the row NaN
  const bool bad = m >= 0x7F800000u;
  const uint32_t e = m >> 23, byte = e > 11u ? e - 7u : 4u;
  const float to = __uint_as_float(byte << 23), back = __uint_as_float((byte - 4u) << 23);
  Query<D> q;
  i32x8 hi, lo;
#pragma unroll
  for (int h = 0; h < D / 64; h++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float x[4] = {f[h][4 * j], f[h][4 * j + 1], f[h][4 * j + 2], f[h][4 * j + 3]};
      uint32_t a, b;
      split4(x, to, back, a, b);
      hi[4 * h + j] = bad ? 0 : (int)a;
      lo[4 * h + j] = bad ? 0 : (int)b;
    }
  if constexpr (D == 64) {
#pragma unroll
    for (int j = 0; j < 4; j++) hi[4 + j] = lo[j];
    q.v[0] = hi;
    q.bytes = bad ? 255u : lg < 2 ? byte : byte - 4u;
  } else {
    q.v[0] = hi;
    q.v[1] = lo;
    q.bytes = bad ? 0xFFFFu : byte | (byte - 4u) << 8;
  }
  return q;
}

// Largest of the four lanes l % 16 + 16 g (a row of scores is spread over them).
__device__ __forceinline__ float max_groups(float v) {
  typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
  const uint32_t x = __float_as_uint(v);
  const u32x2v a = __builtin_bit_cast(u32x2v, __builtin_amdgcn_permlane16_swap(x, x, false, false));
  const uint32_t y = __float_as_uint(__builtin_fmaxf(__uint_as_float(a.x), __uint_as_float(a.y)));
  const u32x2v b = __builtin_bit_cast(u32x2v, __builtin_amdgcn_permlane32_swap(y, y, false, false));
  return __builtin_fmaxf(__uint_as_float(b.x), __uint_as_float(b.y));
}

// Running state of 16 rows: maximum (in units of log2), sums, total.
template <int D>
struct Rows {
  f32x4 o[D / 16], l;
  float m;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < D / 16; d++) o[d] = f32x4{0, 0, 0, 0};
    l = f32x4{0, 0, 0, 0};
    m = -__builtin_inff();
  }
};

// Masks RT x 16 rows of 128 scores past `limit` where `masked` (tile t's
// accumulator i is token places(t) + i) and moves the running maxima; `less`
// is what a weight's exponent, s c - less, takes off. Branches are taken for
// all rows at once.
//
// FUSED: the exponent is one operation, which leaves the largest score's off 0
// by what rounding took from the maximum: up to half a unit in its last place.
// From 2^24 on that would be whole powers of two (all weights 0, or infinite),
// so there the scores are multiplied by c as the maximum was, and c becomes 1.
// Else every exponent is a product and a difference (few rows, whose arithmetic
// waits for the cache anyway: the branch made 16 sequences of 16,000 tokens, 64
// dims, 37 -> 41 us).
template <int D, int RT, bool FUSED, typename F>
__device__ __forceinline__ void running_max(f32x4 (&s)[RT][8], Rows<D> (&r)[RT], float &c, bool masked,
                                            const int (&limit)[RT], F places, float (&less)[RT]) {
  if (masked) {
#pragma unroll
    for (int x = 0; x < RT; x++)
#pragma unroll
      for (int t = 0; t < 8; t++) {
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (places(t) + i > limit[x]) s[x][t][i] = -__builtin_inff();
        __builtin_amdgcn_sched_barrier(0);  // few conditions alive at a time
      }
  }
  float m[RT];
  bool moved = false, large = false;
#pragma unroll
  for (int x = 0; x < RT; x++) {
    float top = s[x][0][0];
#pragma unroll
    for (int t = 0; t < 8; t++)
#pragma unroll
      for (int i = 0; i < 4; i++) top = __builtin_fmaxf(top, s[x][t][i]);
    m[x] = __builtin_fmaxf(r[x].m, max_groups(top) * c);
    moved |= m[x] != r[x].m;
    // nothing seen yet: weights are 0
    less[x] = m[x] == -__builtin_inff() ? 0.0f : m[x];
    large |= FUSED && __builtin_fabsf(less[x]) >= 0x1p24f;
  }
  if (FUSED && __any(large)) {
#pragma unroll
    for (int x = 0; x < RT; x++)
#pragma unroll
      for (int t = 0; t < 8; t++) s[x][t] *= c;
    c = 1.0f;
  }
  if (__any(moved)) {
#pragma unroll
    for (int x = 0; x < RT; x++) {
      const float alpha = __builtin_amdgcn_exp2f(r[x].m - less[x]);
#pragma unroll
      for (int d = 0; d < D / 16; d++) r[x].o[d] *= alpha;
      r[x].l *= alpha;
      r[x].m = m[x];
    }
  }
}

// Weights of RT x 16 rows and 128 tokens, rounded to bfloat16: tiles 2 j and
// 2 j + 1 are the eight tokens of a lane in the second product's step j.
template <int RT, bool FUSED>
__device__ __forceinline__ void weights(const f32x4 (&s)[RT][8], float c, const float (&less)[RT],
                                        u32x4 (&p)[RT][4]) {
#pragma unroll
  for (int x = 0; x < RT; x++)
#pragma unroll
    for (int t = 0; t < 8; t++) {
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; i++)
        e[i] = __builtin_amdgcn_exp2f(FUSED ? __builtin_fmaf(s[x][t][i], c, -less[x]) : s[x][t][i] * c - less[x]);
      p[x][t >> 1][2 * (t & 1)] = pack_bf16(e[0], e[1]);
      p[x][t >> 1][2 * (t & 1) + 1] = pack_bf16(e[2], e[3]);
    }
}

// Sum of the 128 weights on top of l: a product with a row of ones.
__device__ __forceinline__ f32x4 add_weights(const u32x4 (&p)[4], f32x4 l) {
  const uint32_t one = 0x3F803F80u;
#pragma unroll
  for (int j = 0; j < 4; j++) l = mma16(u32x4{one, one, one, one}, p[j], l);
  return l;
}

// 16 codes widened with scale 2^(byte-127). `far`: a lane's byte may be above
// 246; its values past bfloat16's range (no quantizer makes them) become the
// largest, so that a weight of 0 still drops them.
__device__ __forceinline__ void widen16(u32x4 c, uint32_t byte, bool far, u32x4 (&w)[2]) {
  const float f = __uint_as_float(byte << 23);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    w[j >> 1][2 * (j & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[j], f, false));
    w[j >> 1][2 * (j & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[j], f, true));
  }
  if (far) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      uint32_t x = w[j >> 2][j & 3];
      if ((x & 0x7FFFu) == 0x7F80u) x -= 1u;
      if ((x & 0x7FFF0000u) == 0x7F800000u) x -= 0x10000u;
      w[j >> 2][j & 3] = x;
    }
  }
}

// Zero the codes of tokens past the sequence's end (what a page holds there
// may decode to NaN): the lane's 16 bytes start at token `from`, `len` valid.
__device__ __forceinline__ u32x4 keep_tokens(u32x4 v, int valid) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int b = min(max(valid - 4 * j, 0), 4);
    v[j] &= b == 4 ? 0xFFFFFFFFu : (1u << (8 * b)) - 1u;
  }
  return v;
}

struct Block {  // a block of query rows and the keys it sees
  int tok0, count;  // first token of the block, tokens in it
  int len;          // tokens in the sequence's cache
  int seen0;        // keys the block's first token sees; the next one more
  const int32_t *table;
  int last_page;
};
__device__ __forceinline__ bool find_block(const AttnArgs &a, int unit, Block &b) {
  // everything here is the same for the whole workgroup: kept in scalar registers
  auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const int i = uniform(find_sequence(a.b.cu, a.b.batch, a.block_tokens, 1, unit));
  const int c0 = uniform(a.b.cu[i]), n = uniform(a.b.cu[i + 1]) - c0;
  const int at = (unit - (c0 / a.block_tokens + i)) * a.block_tokens;
  if (at >= n || at < 0 || c0 < 0 || (int64_t)c0 + n > a.b.tokens) return false;
  const int64_t room = (int64_t)a.b.width << a.shift;
  b.len = (int)min((int64_t)max(uniform(a.b.lengths[i]), 0), room);
  b.tok0 = c0 + at;
  b.count = min(a.block_tokens, n - at);
  b.seen0 = b.len - n + at + 1;
  b.table = a.b.table + (int64_t)i * a.b.width;
  b.last_page = max(0, (b.len - 1) >> a.shift);
  return true;
}

// The pages of the four runs of 32 tokens of a tile: lane j holds run j % 4's;
// past the end the last page. Page numbers are clamped where they are used:
// at the load, the clamp would have the wave wait for what it just asked for.
__device__ __forceinline__ const int32_t *page_at(const AttnArgs &a, const Block &b, int tile, int lane) {
  return b.table + min((tile * 128 + 32 * (lane & 3)) >> a.shift, b.last_page);
}
__device__ __forceinline__ int page_of(const AttnArgs &a, const Block &b, int tile, int lane) {
  return *page_at(a, b, tile, lane);
}
struct Runs {
  int a, b, c, d;
};
__device__ __forceinline__ Runs runs_of(const AttnArgs &a, int mine) {
  auto page = [&](int j) { return clamp_page(__builtin_amdgcn_readlane(mine, j), a.c.pages); };
  return Runs{page(0), page(1), page(2), page(3)};
}
__device__ __forceinline__ int of_run(const Runs &r, int j) {  // j may differ from lane to lane
  const int lo = (j & 1) ? r.b : r.a, hi = (j & 1) ? r.d : r.c;
  return (j & 2) ? hi : lo;
}

// Scale bytes of a tile's pages: lane j % 4 holds run j's key byte, lane 4 +
// j its value byte. `bytes_of` turns them into one word: bytes 0 and 1 are for
// the keys that this lane's row holds in tiles 0 .. 3 and 4 .. 7 (the matrix
// core picks them), bytes 2 and 3 for the values of its two runs of tokens,
// lg / 2 and 2 + lg / 2. A page whose values
// are NaN must reach only the rows that see it: its keys are made NaN
// instead (masked scores are dropped, visible ones make the row NaN) and its
// values, whose codes are signed zeros, get a finite scale.
__device__ __forceinline__ const uint8_t *byte_at(const AttnArgs &a, int page, int head, int lane) {
  const int64_t at = (int64_t)clamp_page(page, a.c.pages) * a.c.heads + head;
  return ((lane & 4) ? a.c.v_scales : a.c.k_scales) + at;
}
__device__ __forceinline__ uint32_t bytes_of(uint32_t mine, int l16, int lg) {
  uint32_t k[4], v[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    k[j] = (uint32_t)__builtin_amdgcn_readlane((int)mine, j);
    v[j] = (uint32_t)__builtin_amdgcn_readlane((int)mine, 4 + j);
    k[j] = v[j] == 255u ? 255u : k[j];
    v[j] = v[j] == 255u ? 127u : v[j];
  }
  const uint32_t even = k[0] | k[2] << 8, odd = k[1] | k[3] << 8;
  const uint32_t v02 = v[0] | v[2] << 8, v13 = v[1] | v[3] << 8;
  return ((l16 & 8) ? odd : even) | ((lg & 2) ? v13 : v02) << 16;
}

// The same of one tile for the many-rows kernel: the keys' bytes of the four
// runs in one word, and run j's value byte.
__device__ __forceinline__ void page_bytes(uint32_t mine, int j, uint32_t &keys, uint32_t &value) {
  keys = 0;
  value = 0;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)mine, e);
    const uint32_t v = (uint32_t)__builtin_amdgcn_readlane((int)mine, 4 + e);
    keys |= (v == 255u ? 255u : k) << (8 * e);
    value = j == e ? (v == 255u ? 127u : v) : value;
  }
}

// Scores of half a tile (64 tokens), whose keys' bytes are byte H of sc.
template <int D, int H>
__device__ __forceinline__ void scores(const i32x8 (&kv)[4], const Query<D> &q, uint32_t sc,
                                       f32x4 (&s)[8]) {
#pragma unroll
  for (int t = 0; t < 4; t++) {
    s[4 * H + t] = mma<H, 0>(kv[t], q.v[0], f32x4{0, 0, 0, 0}, sc, q.bytes);
    if constexpr (D == 128) s[4 * H + t] = mma<H, 1>(kv[t], q.v[1], s[4 * H + t], sc, q.bytes);
  }
}

// 16 bytes a lane straight into LDS, lane after lane from `lds` on. In
// assembly, since the compiler would otherwise make every later LDS read
// wait for it; the kernel waits where it must. No output register.
__device__ __forceinline__ void load_lds16(const uint8_t *base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"s"(lds), "v"(offset), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void load_lds16(uint64_t address, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt"
               ::"s"(lds), "v"(address) : "memory", "m0");
}
// A word, or a byte widened to one, a lane.
__device__ __forceinline__ void load_lds4(const int32_t *p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void load_lds1(const uint8_t *p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)p;
}

// Few rows: a workgroup of four waves takes up to 16 RT rows of one sequence
// and kv head and one split of its keys; wave w takes tiles w, w + 4, ....
//
// A tile comes in four parts (the keys of 64 tokens twice, then the values of
// half the dims twice), whole rows straight into LDS. A wave has room of its
// own for two parts: as soon as one has been read the one after the next is
// asked for in its place, so that some part is always on its way and no wave
// waits for another. Page numbers and scale bytes come the same way: a load
// into a register would have the compiler wait for everything asked for
// since. Keys lie as rows of D bytes (tokens), values as rows of 128 bytes
// (dims); the 16-byte chunk c of row r sits at position c ^ f(r), f chosen so
// that the 16 rows of a read fall on different banks, the chunks being swapped
// on the global side.
//
// Bound by the cache's bytes: 16 sequences of up to 65,000 tokens, 8 kv heads
// of 128 dims, 1.19 GB in 211 to 220 us (5.4 to 5.6 TB/s; a plain reading of as
// much reaches 7.0). Loads into registers, a tile at a time, took 250: half of a line per
// request, and nothing on its way while a wave computes.
template <int D>
__device__ __forceinline__ int swz_rows(int r) {
  if constexpr (D == 128) return ((r >> 1) & 1) | (((r >> 4) & 3) << 1);
  return (r >> 4) & 3;
}
// (32 rows of 128 dims: one wave a SIMD, two would spill: 92 and 113 us for 16
// sequences of 4 tokens in 16,000, 8 query heads to a kv head. Weights in two
// bfloat16 parts would take the error against 64 bits from 0.0019 of the
// result's norm to its rounding's 0.0017, and the same call to 100 us, 4
// sequences of 700 tokens from 9.0 to 9.6.)
template <int D, int RT>
__global__ __launch_bounds__(256, D == 128 && RT == 2 ? 1 : 2) void k_attn_rows(const AttnArgs a) {
  constexpr int DT = D / 16, W = 4, S = 128 * D, L = S / 2048;  // bytes of a tile's keys, loads of a part
  __shared__ __attribute__((aligned(16))) uint8_t codes[W][S];
  __shared__ uint32_t pages[W][64], bytes[W][64];
  __shared__ float merge_ml[W][16][2];
  static_assert(S >= 16 * (D + 4) * 4, "the waves' sums go where the codes were");
  // a grid's third dimension counts splits, or, where there are none, what the
  // first one has no room for
  const int unit = a.splits > 1 ? blockIdx.x : blockIdx.z * gridDim.x + blockIdx.x;
  Block b;
  if (unit >= a.units || !find_block(a, unit, b)) return;
  const int head = blockIdx.y, split = a.splits > 1 ? blockIdx.z : 0;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int end = min(b.len, b.seen0 + b.count - 1);  // keys any row sees
  const int tiles = (max(end, 0) + 127) >> 7;
  // (the last split takes whatever the caller's bound on the lengths left out)
  const int t0 = split * a.chunk, t1 = split + 1 == a.splits ? tiles : min(tiles, t0 + a.chunk);
  if (split > 0 && t0 >= tiles) return;  // the sum takes only splits that exist
  const int rows = b.count * a.group;

  const int64_t PD = (int64_t)a.c.page * D;
  const int mask = a.c.page - 1, P = a.c.page;
  // loads: 64 / (D / 16) rows of keys each, all of one run of 32 tokens, and 8
  // rows of values, whose chunk lies in one of four runs
  constexpr int KR = 1024 / D;  // rows of a load
  uint8_t *own = codes[wave];
  const uint32_t lds = lds_address(own);
  const int kr = lane / (D / 16), kc = lane & (D / 16 - 1);
  auto load_keys = [&](int tile, const Runs &id, int part) {
#pragma unroll
    for (int i = part * L; i < part * L + L; i++) {
      const int j = i * KR >> 5;  // run
      const uint8_t *base = a.c.k_codes + ((int64_t)of_run(id, j) * a.c.heads + head) * PD +
                            (int64_t)((tile * 128 + i * KR) & mask) * D;
      load_lds16((uint64_t)base + (uint32_t)(kr * D + (kc ^ swz_rows<D>(i * KR + kr)) * 16), lds + i * 1024);
    }
  };
  const int vr = lane >> 3;
  auto load_values = [&](int tile, const Runs &id, int part) {
#pragma unroll
    for (int h = 0; h < 2; h++) {  // rows 16 n + 8 h ..: one swizzle
      const int vc = (lane & 7) ^ (((vr + 8 * h) >> 1) & 7);
      uint64_t v = (uint64_t)a.c.v_codes + ((int64_t)of_run(id, vc >> 1) * a.c.heads + head) * PD +
                   (uint32_t)(((tile * 128 + 16 * vc) & mask) + (vr + 8 * h + part * (D / 2)) * P);
#pragma unroll
      for (int i = 0; i < L / 2; i++, v += 16 * P) load_lds16(v, lds + part * (S / 2) + (2 * i + h) * 1024);
    }
  };
  // a part has landed: only the L loads of the next one are younger
  auto landed = [] { asm volatile("s_waitcnt vmcnt(%0)" ::"i"(L) : "memory"); };
  // what was read is in registers: the part's place may be written
  auto taken = [] { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
  // operand addresses: keys' row 64 (t / 4) + 16 (l16 / 4) + 4 (t % 4) + l16 % 4
  // of tile t, values' row 16 d + l16
  const int krow = 16 * (l16 >> 2) + (l16 & 3);
  const uint8_t *kp0 = own + krow * D + 16 * (lg ^ swz_rows<D>(krow));
  const uint8_t *kp1 = own + krow * D + 16 * ((lg + 4) ^ swz_rows<D>(krow));
  const uint8_t *vp0 = own + l16 * 128 + 16 * (lg ^ ((l16 >> 1) & 7));
  const uint8_t *vp1 = own + l16 * 128 + 16 * ((lg + 4) ^ ((l16 >> 1) & 7));

  Query<D> q[RT];
  Rows<D> r[RT];
  int seen[RT];
#pragma unroll
  for (int x = 0; x < RT; x++) {
    const int row = min(16 * x + l16, rows - 1);
    const int tok = row / a.group;
    seen[x] = b.seen0 + tok;
    q[x] = load_query<D>(a.q + (int64_t)(b.tok0 + tok) * a.q_stride +
                             ((int64_t)head * a.group + row % a.group) * D, lg);
    r[x].clear();
  }
  // ask for what comes before a tile's codes: its scale bytes, and the pages of
  // the wave's tile after it
  auto prepare = [&](int tile, int now) {
    load_lds1(byte_at(a, now, head, lane), lds_address(bytes[wave]));
    load_lds4(page_at(a, b, tile + W, lane), lds_address(pages[wave]));
  };
  Runs id = {0, 0, 0, 0};
  if (t0 + wave < t1) {
    const int now = page_of(a, b, t0 + wave, lane);
    id = runs_of(a, now);
    prepare(t0 + wave, now);
    load_keys(t0 + wave, id, 0);
    load_keys(t0 + wave, id, 1);
  }
  for (int tile = t0 + wave; tile < t1; tile += W) {
    const int next = tile + W;
    f32x4 s[RT][8];
    uint32_t sc = 0;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      landed();
      if (h == 0) sc = bytes_of(bytes[wave][lane], l16, lg);
      i32x8 kv[4];
#pragma unroll
      for (int t = 0; t < 4; t++) {
        const int at = (64 * h + 4 * t) * D;
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(kp0 + at);
        if constexpr (D == 64) kv[t] = join8(lo, lo);
        else kv[t] = join8(lo, *reinterpret_cast<const u32x4 *>(kp1 + at));
      }
      taken();
      load_values(tile, id, h);
#pragma unroll
      for (int x = 0; x < RT; x++) {
        if (h == 0) scores<D, 0>(kv, q[x], sc, s[x]);
        else scores<D, 1>(kv, q[x], sc, s[x]);
      }
    }
    int limit[RT];
    float less[RT], c = a.scale2;
#pragma unroll
    for (int x = 0; x < RT; x++) limit[x] = seen[x] - 1 - tile * 128 - 16 * lg;
    running_max<D, RT, false>(s, r, c, tile * 128 + 128 > b.seen0, limit,
                       [](int t) { return 64 * (t >> 2) + 4 * (t & 3); }, less);
    u32x4 p[RT][4];
    weights<RT, false>(s, c, less, p);
    const uint32_t vb0 = sc >> 16 & 255u, vb1 = sc >> 24;
    const bool far = __any(max(vb0, vb1) > 246u);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      if (h == 0 || next < t1) landed();
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      i32x8 vv[DT / 2];
#pragma unroll
      for (int d = 0; d < DT / 2; d++)
        vv[d] = join8(*reinterpret_cast<const u32x4 *>(vp0 + h * (S / 2) + 2048 * d),
                      *reinterpret_cast<const u32x4 *>(vp1 + h * (S / 2) + 2048 * d));
      taken();
      if (next < t1) {
        if (h == 0) {
          const int now = (int)pages[wave][lane];
          id = runs_of(a, now);
          prepare(next, now);
        }
        load_keys(next, id, h);
      }
      if (tile * 128 + 128 > b.len) {
        // the sequence's last tile: what its pages hold past the end may decode
        // to NaN and is cleared
#pragma unroll
        for (int d = 0; d < DT / 2; d++) {
          const u32x4 v0 = {(uint32_t)vv[d][0], (uint32_t)vv[d][1], (uint32_t)vv[d][2], (uint32_t)vv[d][3]};
          const u32x4 v1 = {(uint32_t)vv[d][4], (uint32_t)vv[d][5], (uint32_t)vv[d][6], (uint32_t)vv[d][7]};
          const int from = b.len - tile * 128 - 16 * lg;
          vv[d] = join8(keep_tokens(v0, from), keep_tokens(v1, from - 64));
        }
      }
#pragma unroll
      for (int d = 0; d < DT / 2; d++) {
        u32x4 w[4];
#pragma unroll
        for (int q = 0; q < 2; q++) {
          u32x4 wide[2];
          widen16(u32x4{(uint32_t)vv[d][4 * q], (uint32_t)vv[d][4 * q + 1], (uint32_t)vv[d][4 * q + 2],
                        (uint32_t)vv[d][4 * q + 3]}, q ? vb1 : vb0, far, wide);
          w[2 * q] = wide[0];
          w[2 * q + 1] = wide[1];
        }
#pragma unroll
        for (int x = 0; x < RT; x++) {
          f32x4 &o = r[x].o[h * (DT / 2) + d];
#pragma unroll
          for (int j = 0; j < 4; j++) o = mma16(w[j], p[x][j], o);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < RT; x++) r[x].l = add_weights(p[x], r[x].l);
  }
  // no load may land on the sums below
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  auto merge_o = [&](int w, int row, int d) -> float & {
    return reinterpret_cast<float *>(codes[w])[row * (D + 4) + d];
  };
  // merge the four waves, 16 rows at a time
#pragma unroll
  for (int x = 0; x < RT; x++) {
    if (x) __syncthreads();
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int e = 0; e < 4; e++) merge_o(wave, l16, 16 * d + 4 * lg + e) = r[x].o[d][e];
    if (lg == 0) {
      merge_ml[wave][l16][0] = r[x].m;
      merge_ml[wave][l16][1] = r[x].l[0];
    }
    __syncthreads();
    // thread: row threadIdx / 16, D / 16 consecutive dims
    const int row = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * (D / 16);
    float m = merge_ml[0][row][0];
#pragma unroll
    for (int w = 1; w < W; w++) m = __builtin_fmaxf(m, merge_ml[w][row][0]);
    const float ms = m == -__builtin_inff() ? 0.0f : m;
    float l = 0.0f, o[D / 16];
#pragma unroll
    for (int e = 0; e < D / 16; e++) o[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; w++) {
      const float f = __builtin_amdgcn_exp2f(merge_ml[w][row][0] - ms);
      l += f * merge_ml[w][row][1];
#pragma unroll
      for (int e = 0; e < D / 16; e++) o[e] += f * merge_o(w, row, d0 + e);
    }
    const int rr = 16 * x + row;
    if (rr < rows) {
      const int64_t tok = b.tok0 + rr / a.group;
      const int64_t qh = (int64_t)head * a.group + rr % a.group;
      if (a.splits > 1) {
        float *p = a.part + ((tok * a.q_heads + qh) * a.splits + split) * (D + 4);
#pragma unroll
        for (int e = 0; e < D / 16; e++) p[d0 + e] = o[e];
        if (d0 == 0) {
          p[D] = m;
          p[D + 1] = l;
        }
      } else {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t *p = a.out + (tok * a.q_heads + qh) * D + d0;
#pragma unroll
        for (int e = 0; e < D / 16; e += 2)
          *reinterpret_cast<uint32_t *>(p + e) = pack_bf16(o[e] * inv, o[e + 1] * inv);
      }
    }
  }
}

// How many splits of a token's block the first kernel wrote, as it had it.
__device__ __forceinline__ int splits_of(const AttnArgs &a, int tok) {
  const int i = find_sequence(a.b.cu, a.b.batch, 1, 0, tok);
  const int c0 = a.b.cu[i], n = a.b.cu[i + 1] - c0;
  const int64_t room = (int64_t)a.b.width << a.shift;
  const int len = (int)min((int64_t)max(a.b.lengths[i], 0), room);
  const int at = (tok - c0) / a.block_tokens * a.block_tokens;
  const int end = min(len, len - n + at + min(a.block_tokens, n - at));
  const int tiles = (max(end, 0) + 127) >> 7;
  return max(1, min(a.splits, (tiles + a.chunk - 1) / a.chunk));
}

// Joins a few splits of many rows: D / 4 threads a (token, query head), which
// all go through the splits' maxima and then through their sums.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join_few(const AttnArgs a) {
  constexpr int C = D / 4, R = 256 / C, P = D + 4;
  const int tok = blockIdx.x, c = threadIdx.x % C, qh = blockIdx.y * R + threadIdx.x / C;
  const int live = splits_of(a, tok);
  if (qh >= a.q_heads) return;
  const int64_t row = (int64_t)tok * a.q_heads + qh;
  const float *p = a.part + row * a.splits * P;
  float m = -__builtin_inff();
  for (int s = 0; s < live; s++) m = __builtin_fmaxf(m, p[s * P + D]);
  const float ms = m == -__builtin_inff() ? 0.0f : m;
  f32x4 o = {0, 0, 0, 0};
  float l = 0.0f;
  for (int s = 0; s < live; s++) {
    const float f = __builtin_amdgcn_exp2f(p[s * P + D] - ms);
    const f32x4 v = *reinterpret_cast<const f32x4 *>(p + s * P + 4 * c);
    l = __builtin_fmaf(f, p[s * P + D + 1], l);
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = __builtin_fmaf(f, v[e], o[e]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<u32x2 *>(a.out + row * D + 4 * c) =
      u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
}

// Joins many splits, or those of few rows, of one (token, query head): thread
// s takes split s's maximum and total, then D / 4 threads a row add up splits
// s, s + G, ....
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a) {
  constexpr int C = D / 4, G = 256 / C, P = D + 4;
  __shared__ float factor[256];
  __shared__ float red[4];
  __shared__ f32x4 sums[G][C];
  const int64_t row = blockIdx.x;
  const int tok = (int)(row / a.q_heads);
  const int live = splits_of(a, tok);
  const float *p = a.part + row * a.splits * P;
  const int wave = threadIdx.x >> 6;

  float m = -__builtin_inff();
  for (int s = threadIdx.x; s < live; s += 256) m = __builtin_fmaxf(m, p[(int64_t)s * P + D]);
  for (int d = 1; d < 64; d <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d));
  if ((threadIdx.x & 63) == 0) red[wave] = m;
  __syncthreads();
  m = __builtin_fmaxf(__builtin_fmaxf(red[0], red[1]), __builtin_fmaxf(red[2], red[3]));
  const float ms = m == -__builtin_inff() ? 0.0f : m;
  const int c = threadIdx.x % C, g = threadIdx.x / C;
  f32x4 o = {0, 0, 0, 0};
  float l = 0.0f;
  for (int s0 = 0; s0 < live; s0 += 256) {
    const int s = s0 + threadIdx.x, many = min(256, live - s0);
    float f = 0.0f;
    if (s < live) {
      f = __builtin_amdgcn_exp2f(p[(int64_t)s * P + D] - ms);
      l = __builtin_fmaf(f, p[(int64_t)s * P + D + 1], l);
    }
    __syncthreads();  // the last round's factors have been used
    factor[threadIdx.x] = f;
    __syncthreads();
#pragma unroll 4
    for (int q = g; q < many; q += G) {
      const f32x4 v = *reinterpret_cast<const f32x4 *>(p + (int64_t)(s0 + q) * P + 4 * c);
      const float w = factor[q];
#pragma unroll
      for (int e = 0; e < 4; e++) o[e] = __builtin_fmaf(w, v[e], o[e]);
    }
  }
  l = sum64(l);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[wave] = l;
  sums[g][c] = o;
  __syncthreads();
  l = (red[0] + red[1]) + (red[2] + red[3]);
  if (g == 0) {
#pragma unroll
    for (int q = 1; q < G; q++) o += sums[q][c];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<u32x2 *>(a.out + row * D + 4 * c) =
        u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
  }
}

// Many rows: four waves of 32 rows share tiles of 128 tokens through LDS; two
// workgroups share a compute unit, so that one's softmax runs beside the
// other's products. Rows are `tokens x group` of one kv head. Keys are loaded
// directly, double-buffered; values go through registers, where they are
// widened, a tile ahead of use, into one buffer (a second barrier a tile).
//
// Keys lie in LDS as rows of D bytes (tokens), values as rows of 256 bytes
// (dims). The 16-byte chunk c of row r sits at position c ^ f(r), f chosen so
// that the 16 rows of a read fall on different banks (the keys' chunks are
// swapped on the global side); for values c ^ (c / 8) ^ r, so that the eight
// even chunks that a row's lanes write do too. A load of keys covers rows of
// one run of 32 tokens, whose page is wave-uniform; a lane's chunk of values
// lies in one of four.
//
// 2 x up to 2,048 tokens of 8,192, 32 query heads on 8 of 128 dims: 404 to 419
// us (1.0 PFLOP/s) in a long run, heads of 64 296 to 302; a few calls after a
// pause 466 to 514. (Weights in two E4M3 parts and 8-bit values took 510 and 381
// where this, measured beside it, took 480 and 326.)
template <int D>
__device__ __forceinline__ int swz_k(int r) {
  if constexpr (D == 128) return ((r >> 1) & 1) | (((r >> 3) & 3) << 1);
  return (r >> 3) & 3;
}

template <int D>
__global__ __launch_bounds__(256, 2) void k_attn_tiles(const AttnArgs a) {
  constexpr int DT = D / 16, RT = 2, S = 128 * D;
  constexpr int KL = S / 4096, VL = KL;  // direct loads per thread and tile
  __shared__ __attribute__((aligned(16))) uint8_t ks[2 * S], vs[2 * S];
  // kv heads fastest: the eight XCDs, which are dealt workgroups in turn,
  // keep to few heads each. The last blocks of a sequence see the most keys:
  // they start first.
  const uint32_t block = blockIdx.z * gridDim.x + blockIdx.x;
  const int head = block % a.c.heads, from_last = block / a.c.heads;
  Block b;
  if (from_last >= a.units || !find_block(a, a.units - 1 - from_last, b)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int end = min(b.len, b.seen0 + b.count - 1);
  const int tiles = (max(end, 0) + 127) >> 7;
  // this split's tiles, from an even one on (the buffers take turns); the last
  // split takes whatever the caller's bound on the lengths left out
  const int split = blockIdx.y, t0 = split * a.chunk;
  const int t1 = split + 1 == a.splits ? tiles : min(tiles, t0 + a.chunk);
  if (split > 0 && t0 >= tiles) return;  // the sum takes only splits that exist
  const int rows = b.count * a.group;
  Query<D> q[RT];
  Rows<D> r[RT];
  int seen[RT];
#pragma unroll
  for (int x = 0; x < RT; x++) {
    const int row = min(32 * wave + 16 * x + l16, rows - 1);
    const int tok = row / a.group;
    seen[x] = b.seen0 + tok;
    q[x] = load_query<D>(a.q + (int64_t)(b.tok0 + tok) * a.q_stride +
                             ((int64_t)head * a.group + row % a.group) * D, lg);
    r[x].clear();
  }
  const int64_t PD = (int64_t)a.c.page * D;
  const int mask = a.c.page - 1, P = a.c.page;

  // loads: this thread's offsets in a page's keys (rows tid / 8 or tid / 4 of
  // a run; every other load's rows swizzle by 64 bytes more) and values
  const int kr = threadIdx.x / (D / 16), kc = (threadIdx.x & (D / 16 - 1)) ^ swz_k<D>(kr);
  const uint32_t koff = (uint32_t)((kr & 31) * D + kc * 16);
  const int vr = threadIdx.x >> 3, vc = threadIdx.x & 7;  // row and 16 tokens of values
  const uint32_t klds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)ks + wave * 1024;
  u32x4 raw[VL];
  auto load = [&](int tile, int buf, const Runs &id) {
    int64_t page[4];  // wave-uniform: where each run's page begins, in keys and values alike
#pragma unroll
    for (int j = 0; j < 4; j++) page[j] = ((int64_t)of_run(id, j) * a.c.heads + head) * PD;
#pragma unroll
    for (int i = 0; i < KL; i++) {
      const int j = D == 128 ? i : 2 * i + (wave >> 1);  // wave-uniform
      const int64_t at = D == 128 ? page[i] : (wave >> 1) ? page[2 * i + 1] : page[2 * i];
      load_lds16(a.c.k_codes + at + (int64_t)((tile * 128 + 32 * j) & mask) * D, koff, klds + buf * S + i * 4096);
    }
    const int64_t lo = (vc & 2) ? page[1] : page[0], hi = (vc & 2) ? page[3] : page[2];
    const uint8_t *v = a.c.v_codes + ((vc & 4) ? hi : lo) + (((tile * 128 + 16 * vc) & mask) + vr * P);
#pragma unroll
    for (int i = 0; i < VL; i++) raw[i] = *reinterpret_cast<const u32x4 *>(v + 32 * i * P);
  };
  // operand addresses in LDS: keys' row 32 (t / 2) + 8 (l16 / 4) + 4 (t % 2) +
  // l16 % 4 of tile t; values' row 16 d + l16, tokens 32 j + 8 lg ..
  const int krow = 8 * (l16 >> 2) + (l16 & 3);
  const uint8_t *kp0 = ks + krow * D + 16 * (lg ^ swz_k<D>(krow));
  const uint8_t *kp1 = ks + krow * D + 16 * ((lg + 4) ^ swz_k<D>(krow));
  const uint8_t *vp[4];
#pragma unroll
  for (int j = 0; j < 4; j++) vp[j] = vs + l16 * 256 + 16 * ((4 * j + lg) ^ (j >> 1) ^ l16);

  int mine = 0;        // pages of the next tile
  uint32_t bytes = 0;  // scale bytes of this one
  if (t0 < t1) {
    const int now = page_of(a, b, t0, lane);
    bytes = *byte_at(a, now, head, lane);
    mine = page_of(a, b, t0 + 1, lane);
    load(t0, 0, runs_of(a, now));
  }
  int flip = S;
  for (int tile = t0; tile < t1; tile++) {
    // this tile's codes, its scale bytes and the next one's pages have
    // arrived, and every wave is done with the other buffer
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    uint32_t sc, mv;
    page_bytes(bytes, vc >> 1, sc, mv);
    if (tile * 128 + 128 > b.len) {
      // the sequence's last tile: what its pages hold past the end may decode
      // to NaN and is cleared
      asm volatile("");  // a branch, not arithmetic in every tile
#pragma unroll
      for (int i = 0; i < VL; i++) raw[i] = keep_tokens(raw[i], b.len - tile * 128 - 16 * vc);
    }
#pragma unroll
    for (int i = 0; i < VL; i++) {
      u32x4 w[2];
      widen16(raw[i], mv, __any(mv > 246u), w);
      const int row = vr + 32 * i;
#pragma unroll
      for (int h = 0; h < 2; h++)
        *reinterpret_cast<u32x4 *>(vs + row * 256 + 16 * ((2 * vc + h) ^ (vc >> 2) ^ (row & 15))) = w[h];
    }
    const Runs id = runs_of(a, mine);
    __builtin_amdgcn_sched_barrier(0);
    if (tile + 1 < t1) {
      bytes = *byte_at(a, mine, head, lane);
      mine = page_of(a, b, tile + 2, lane);
      load(tile + 1, (tile + 1) & 1, id);
    }
    auto keys = [&](int t) {
      const int at = (32 * (t >> 1) + 4 * (t & 1)) * D;
      const u32x4 lo = *reinterpret_cast<const u32x4 *>(kp0 + at);
      if constexpr (D == 64) return join8(lo, lo);
      else return join8(lo, *reinterpret_cast<const u32x4 *>(kp1 + at));
    };
    // operands are read two tiles ahead
    f32x4 s[RT][8];
    i32x8 f[3] = {keys(0), keys(1)};
    auto score = [&](auto run) {  // the two tiles of a run of 32 tokens
      constexpr int J = decltype(run)::value;
#pragma unroll
      for (int t = 2 * J; t < 2 * J + 2; t++) {
        if (t + 2 < 8) f[(t + 2) % 3] = keys(t + 2);
#pragma unroll
        for (int x = 0; x < RT; x++) s[x][t] = mma<J, 0>(f[t % 3], q[x].v[0], f32x4{0, 0, 0, 0}, sc, q[x].bytes);
        if constexpr (D == 128) {
#pragma unroll
          for (int x = 0; x < RT; x++) s[x][t] = mma<J, 1>(f[t % 3], q[x].v[1], s[x][t], sc, q[x].bytes);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    score(std::integral_constant<int, 0>());
    score(std::integral_constant<int, 1>());
    score(std::integral_constant<int, 2>());
    score(std::integral_constant<int, 3>());
    // all scores are taken here, while a key operand is at hand (the compiler
    // would move some past the branches below, and keep the operands)
#pragma unroll
    for (int x = 0; x < RT; x++)
#pragma unroll
      for (int t = 0; t < 8; t++) asm volatile("" : "+v"(s[x][t]));
    int limit[RT];
    float less[RT], c = a.scale2;
#pragma unroll
    for (int x = 0; x < RT; x++) limit[x] = seen[x] - 1 - tile * 128 - 8 * lg;
    running_max<D, RT, true>(s, r, c, tile * 128 + 128 > b.seen0, limit,
                       [](int t) { return 32 * (t >> 1) + 4 * (t & 1); }, less);
    u32x4 p[RT][4];  // of tokens 32 j + 8 lg ..
    weights<RT, true>(s, c, less, p);
    // the widened values of every wave are in LDS
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    u32x4 g[2][4];
    auto values = [&](int d) {
#pragma unroll
      for (int j = 0; j < 4; j++) g[d & 1][j] = *reinterpret_cast<const u32x4 *>(vp[j] + 4096 * d);
    };
    values(0);
#pragma unroll
    for (int d = 0; d < DT; d++) {
      if (d + 1 < DT) values(d + 1);
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int x = 0; x < RT; x++) r[x].o[d] = mma16(g[d & 1][j], p[x][j], r[x].o[d]);
    }
#pragma unroll
    for (int x = 0; x < RT; x++) r[x].l = add_weights(p[x], r[x].l);
    kp0 += flip;  // to the other buffer
    kp1 += flip;
    flip = -flip;
  }
#pragma unroll
  for (int x = 0; x < RT; x++) {
    const int row = 32 * wave + 16 * x + l16;
    if (row < rows) {
      const float l = r[x].l[0], inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int64_t tok = b.tok0 + row / a.group;
      const int64_t qh = (int64_t)head * a.group + row % a.group;
      if (a.splits > 1) {
        float *p = a.part + ((tok * a.q_heads + qh) * a.splits + split) * (D + 4);
#pragma unroll
        for (int d = 0; d < DT; d++) *reinterpret_cast<f32x4 *>(p + 16 * d + 4 * lg) = r[x].o[d];
        if (lg == 0) {
          p[D] = r[x].m;
          p[D + 1] = l;
        }
      } else {
        uint16_t *p = a.out + (tok * a.q_heads + qh) * D + 4 * lg;
#pragma unroll
        for (int d = 0; d < DT; d++) {
          const f32x4 o = r[x].o[d];
          *reinterpret_cast<u32x2 *>(p + 16 * d) =
              u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
        }
      }
    }
  }
}

static int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) s++;
  return s;
}

// Workgroups along one dimension of a grid, whose threads are fewer than 2^32,
// and along another for the rest.
struct Spread {
  uint32_t first, second;
};
static Spread spread(int64_t blocks) {
  const int64_t first = std::min<int64_t>(blocks, 1 << 22);
  return {(uint32_t)first, (uint32_t)((blocks + first - 1) / first)};
}

struct AttnPlan {
  bool few;
  int rt, block_tokens, chunk, splits;
  int most_splits;  // of any sequence up to max_length
  int64_t units;
};
static AttnPlan attn_plan(int64_t tokens, int batch, int q_heads, int heads, int64_t max_length) {
  AttnPlan p;
  const int group = q_heads / heads;
  const int64_t mean = (tokens + batch - 1) / batch * group;  // rows of a sequence
  // 16 sequences of 16,000 tokens: 16 rows each 64 us (the other kernel, of
  // 128 rows: 105), 32 rows 94 (109)
  p.few = mean <= 32 && group <= 32;
  p.rt = p.few ? (mean <= 16 && group <= 16 ? 1 : 2) : 2;
  p.block_tokens = (p.few ? 16 * p.rt : 128) / group;
  p.units = tokens / p.block_tokens + batch;
  const int tiles = (int)((max_length + 127) / 128);
  p.chunk = tiles > 0 ? tiles : 1;
  p.splits = p.most_splits = 1;
  // No split has fewer than eight tiles, and there are at most `want`: a bound
  // that grows with the length, where the number of splits itself does not
  // (chunks are rounded up).
  auto bound = [&](int64_t want) { return (int)std::max<int64_t>(1, std::min<int64_t>(want, (tiles + 7) / 8)); };
  if (p.few) {
    // enough workgroups to fill the card four times over, since sequences
    // shorter than the longest leave splits empty (16 ragged ones of up to
    // 65,000: 220 us; twice over 238, eight times 224), and at least two tiles
    // a wave: below that the sum over splits costs more than it saves
    const int64_t base = std::max<int64_t>(1, (int64_t)batch * heads);
    const int64_t want = std::max<int64_t>(1, 2048 / base);
    const int64_t c = std::max<int64_t>(8, (tiles + want - 1) / want);
    p.chunk = (int)((c + 3) / 4 * 4);
    p.splits = std::max(1, (tiles + p.chunk - 1) / p.chunk);
    p.most_splits = bound(want);
  } else {
    // two workgroups a compute unit where blocks of rows leave half of that
    // empty (1 x 512 tokens of 4,096, 32 query heads on 8: 85 us in one piece,
    // 54 so; 1 x 256 of 8,192: 163 and 56), and at least eight tiles each: with
    // four 1 x 1,024 of 1,024 take 37, in one piece 29
    const int64_t base = std::max<int64_t>(1, (tokens + p.block_tokens - 1) / p.block_tokens * heads);
    const int64_t want = 512 / base;
    if (want > 1) {
      const int64_t c = std::max<int64_t>(8, (tiles + want - 1) / want);
      p.chunk = (int)((c + 1) & ~1);
      p.splits = std::max(1, (tiles + p.chunk - 1) / p.chunk);
      p.most_splits = bound(want);
    }
  }
  return p;
}

}  // namespace mxl

using namespace mxl;

hipError_t mxi_launch_kv_append(const void *k, const void *v, int bf16, int64_t k_stride,
                                int64_t v_stride, const mx_kv_cache_t &cache,
                                const mx_kv_batch_t &batch, hipStream_t st) {
  const int64_t blocks = (batch.tokens / cache.page + 2 * (int64_t)batch.batch) * cache.heads;
  const AppendArgs a = {k, v, k_stride, v_stride, cache, batch, log2_of(cache.page), (uint32_t)blocks};
  const Spread xy = spread(blocks);
  const dim3 grid(xy.first, xy.second);
  const size_t lds = (size_t)cache.dim * (cache.page + 4);
  // a few new tokens per sequence: one wave a page, so that all pages are at
  // work at once (256 sequences of one token: 8.5 us; four
  // waves, and kept codes moved a word at a time: 19)
  const bool few = batch.tokens <= 4 * (int64_t)batch.batch;
  if (bf16) few ? k_kv_append<true, 64><<<grid, 64, lds, st>>>(a) : k_kv_append<true, 256><<<grid, 256, lds, st>>>(a);
  else few ? k_kv_append<false, 64><<<grid, 64, lds, st>>>(a) : k_kv_append<false, 256><<<grid, 256, lds, st>>>(a);
  return hipGetLastError();
}

size_t mxi_kv_attention_workspace(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                  int64_t max_length) {
  const AttnPlan p = attn_plan(tokens, batch, q_heads, heads, max_length);
  return p.most_splits > 1 ? (size_t)tokens * q_heads * p.most_splits * (dim + 4) * sizeof(float) : 0;
}

hipError_t mxi_launch_kv_attention(const void *q, int64_t q_stride, int q_heads,
                                   const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                                   int64_t max_length, float scale, void *out, void *workspace,
                                   hipStream_t st) {
  const AttnPlan p = attn_plan(batch.tokens, batch.batch, q_heads, cache.heads, max_length);
  const AttnArgs a = {reinterpret_cast<const uint16_t *>(q), q_stride, q_heads,
                      q_heads / cache.heads, cache, batch, log2_of(cache.page), p.block_tokens,
                      p.chunk, p.splits, (int)p.units, scale * 1.44269504088896340736f,
                      reinterpret_cast<uint16_t *>(out), reinterpret_cast<float *>(workspace)};
  // (few rows are split for at most 1,024 sequences)
  const Spread xz = spread(p.few ? p.units : p.units * cache.heads);
  const dim3 grid(xz.first, (uint32_t)cache.heads, p.splits > 1 ? (uint32_t)p.splits : xz.second);
  if (!p.few) {
    const dim3 tgrid(xz.first, (uint32_t)p.splits, xz.second);
    if (cache.dim == 64) k_attn_tiles<64><<<tgrid, 256, 0, st>>>(a);
    else k_attn_tiles<128><<<tgrid, 256, 0, st>>>(a);
  } else if (cache.dim == 64) {
    if (p.rt == 1) k_attn_rows<64, 1><<<grid, 256, 0, st>>>(a);
    else k_attn_rows<64, 2><<<grid, 256, 0, st>>>(a);
  } else {
    if (p.rt == 1) k_attn_rows<128, 1><<<grid, 256, 0, st>>>(a);
    else k_attn_rows<128, 2><<<grid, 256, 0, st>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  // 16,384 rows of 4 splits: 14 us less than with a workgroup a row; 512 rows of
  // 16: 7 us more
  if (p.splits <= 16 && batch.tokens * q_heads >= 4096) {
    const int rows = 1024 / cache.dim;  // of a workgroup
    const dim3 jgrid((uint32_t)batch.tokens, (uint32_t)((q_heads + rows - 1) / rows));
    if (cache.dim == 64) k_attn_join_few<64><<<jgrid, 256, 0, st>>>(a);
    else k_attn_join_few<128><<<jgrid, 256, 0, st>>>(a);
    return hipGetLastError();
  }
  const dim3 jgrid((uint32_t)(batch.tokens * q_heads));
  if (cache.dim == 64) k_attn_join<64><<<jgrid, 256, 0, st>>>(a);
  else k_attn_join<128><<<jgrid, 256, 0, st>>>(a);
  return hipGetLastError();
}
