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
// Attention, o = sum_j softmax_j(scale q.k_j) v_j, runs on the 8-bit matrix
// cores without widening the cache. v_mfma_scale_f32_16x16x128_f8f6f4 takes
// the cache's codes and bytes as they are; the other operand (q, then the
// softmax's weights p) is split into two E4M3 numbers, x = hi + lo, whose
// products land in the same accumulator: q's eight significant bits are held
// exactly, p is off by at most 2^-9 of itself (bf16: 2^-8; measured, the
// output's error is 1.07 of bf16 rounding's own). Scores are taken
// transposed (tokens are the accumulator's rows), so that the weights come
// out in the very lanes and order in which the second product wants them:
// with g = lane / 16, tile t (of 16 rows) and accumulator i hold token
// 64 (t / 4) + 16 g + 4 (t % 4) + i of a run of 128, and the second product's
// lane holds tokens 16 g .. + 15 and 64 + 16 g .. + 15. The weights' sum is a
// ninth product with a row of ones. Maxima, sums and accumulators are fp32.
//
// Two kernels: few rows (single tokens) read the cache straight into
// registers, one wave per 128 tokens at a time, the sequence split over
// workgroups; many rows (prompts) share tiles of 128 tokens through LDS.
#include <algorithm>

#include "mx_layer.h"
#include "mx_layer_device.h"

namespace mxl {

__device__ __forceinline__ int clamp_page(int32_t id, int64_t pages) {
  return (int)min((uint32_t)id, (uint32_t)(pages - 1));
}

// ---- append -------------------------------------------------------------------------

struct AppendArgs {
  const void *k, *v;
  int64_t k_stride, v_stride;  // elements between tokens
  mx_kv_cache_t c;
  mx_kv_batch_t b;
  int shift;  // log2(page)
};

// Which sequence a unit of work belongs to: sequence i owns units from
// cu[i] / per + extra i on, which leaves it at least n / per + extra.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int batch, int per, int extra,
                                             int unit) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] / per + extra * mid <= unit) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <bool BF16>
__device__ __forceinline__ uint32_t amax_row8(const void *base, int64_t elem, float (&f)[8]) {
  widen<BF16>(load_raw<BF16>(reinterpret_cast<const uint8_t *>(base) + elem * (BF16 ? 2 : 4), 0), f);
  return amax8(f);
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

constexpr int kMaxPage = 256, kMaxDim = 128;

template <bool BF16>
__global__ __launch_bounds__(256) void k_kv_append(const AppendArgs a) {
  // new values' codes, [dim][token]; rows are 16 bytes longer than a page's
  // so that a row's byte writes and the next row's fall on other banks
  __shared__ __attribute__((aligned(16))) uint8_t vt[kMaxDim * (kMaxPage + 16)];
  __shared__ uint32_t am[2][4];
  const int unit = blockIdx.x, head = blockIdx.y, P = a.c.page, D = a.c.dim;
  const int i = find_sequence(a.b.cu, a.b.batch, P, 2, unit);
  const int c0 = a.b.cu[i], n = a.b.cu[i + 1] - c0, held = a.b.lengths[i];
  const int j = (held >> a.shift) + unit - (c0 / P + 2 * i);  // page of the sequence
  if (n <= 0 || held < 0 || j >= a.b.width || ((int64_t)j << a.shift) >= (int64_t)held + n) return;
  const int kept = max(0, held - (j << a.shift));            // slots that stay
  const int end = min((int64_t)P, (int64_t)held + n - ((int64_t)j << a.shift));  // slots in use after
  const int64_t id = clamp_page(a.b.table[(int64_t)i * a.b.width + j], a.c.pages);
  const int64_t src0 = (int64_t)c0 + ((int64_t)j << a.shift) - held;  // token of slot 0
  const int64_t most = a.b.tokens - 1;
  const int64_t at = id * a.c.heads + head;
  const int per = D >> 3, items = (end - kept) * per;  // items of eight elements

  uint32_t mk = 0, mv = 0;
  for (int it = threadIdx.x; it < items; it += 256) {
    const int slot = kept + it / per, d = (it % per) * 8;
    const int64_t tok = min(max(src0 + slot, (int64_t)0), most);
    float f[8];
    mk = max(mk, amax_row8<BF16>(a.k, tok * a.k_stride + (int64_t)head * D + d, f));
    mv = max(mv, amax_row8<BF16>(a.v, tok * a.v_stride + (int64_t)head * D + d, f));
  }
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
  uint32_t was_k = 0, was_v = 0;
  if (kept) {
    was_k = a.c.k_scales[at];
    was_v = a.c.v_scales[at];
  }
  __syncthreads();
  mk = max(max(am[0][0], am[0][1]), max(am[0][2], am[0][3]));
  mv = max(max(am[1][0], am[1][1]), max(am[1][2], am[1][3]));
  const uint32_t sk = max(scale_byte8(mk), was_k), sv = max(scale_byte8(mv), was_v);
  uint8_t *kc = a.c.k_codes + at * P * D, *vc = a.c.v_codes + at * P * D;
  if (kept && sk > was_k) {
    uint32_t *w = reinterpret_cast<uint32_t *>(kc);
    for (int it = threadIdx.x; it < kept * D / 4; it += 256)
      w[it] = move4(w[it], (int)(sk - was_k), sk == 255u);
  }
  if (kept && sv > was_v) {
    // whole words of four tokens; a word that also holds slots past `kept`
    // keeps those bytes
    const int words = (kept + 3) >> 2;
    for (int it = threadIdx.x; it < D * words; it += 256) {
      const int d = it / words, s = (it % words) * 4;
      uint32_t *w = reinterpret_cast<uint32_t *>(vc + (int64_t)d * P + s);
      const uint32_t old = *w, moved = move4(old, (int)(sv - was_v), sv == 255u);
      const uint32_t mask = kept - s >= 4 ? 0xFFFFFFFFu : (1u << (8 * (kept - s))) - 1;
      *w = (moved & mask) | (old & ~mask);
    }
    __syncthreads();  // before the new tokens' bytes of the same words
  }
  const int row = P + 16;
  for (int it = threadIdx.x; it < items; it += 256) {
    const int slot = kept + it / per, d = (it % per) * 8;
    const int64_t tok = min(max(src0 + slot, (int64_t)0), most);
    float f[8];
    amax_row8<BF16>(a.k, tok * a.k_stride + (int64_t)head * D + d, f);
    *reinterpret_cast<u32x2 *>(kc + slot * D + d) = encode8(f, sk);
    amax_row8<BF16>(a.v, tok * a.v_stride + (int64_t)head * D + d, f);
    const u32x2 w = encode8(f, sv);
#pragma unroll
    for (int e = 0; e < 8; e++) vt[(d + e) * row + slot] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
  }
  __syncthreads();
  const int chunks = P >> 4;
  for (int it = threadIdx.x; it < D * chunks; it += 256) {
    const int d = it / chunks, s = (it % chunks) * 16;
    const int lo = max(kept, s), hi = min(end, s + 16);
    if (lo >= hi) continue;
    uint8_t *dst = vc + (int64_t)d * P;
    if (lo == s && hi == s + 16) {
      *reinterpret_cast<u32x4 *>(dst + s) = *reinterpret_cast<const u32x4 *>(vt + d * row + s);
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
  int splits;
  float scale2;      // softmax scale times log2(e)
  uint16_t *out;
  float *part;       // [token, q head, split][dim + 2]: sums, then maximum and total
};

__device__ __forceinline__ i32x8 join8(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
__device__ __forceinline__ f32x4 mma(i32x8 a, i32x8 b, f32x4 d, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, 0, 0, 0, (int)sa, 0, (int)sb);
}

// A row of q as the second operand: hi and lo, each 32 codes (dim 128), or
// hi in the first 16 bytes and lo in the second (dim 64, where one product
// of length 128 takes both against the keys' codes given twice). `byte` is
// the E8M0 byte of hi; lo's is byte - 4.
template <int D>
struct Query {
  i32x8 v[D / 64];
  uint32_t byte[D / 64];
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
    q.byte[0] = bad ? 255u : lg < 2 ? byte : byte - 4u;
  } else {
    q.v[0] = hi;
    q.v[1] = lo;
    q.byte[0] = bad ? 255u : byte;
    q.byte[1] = bad ? 255u : byte - 4u;
  }
  return q;
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

// Weights of 128 scores (see the order above): masks tokens past `limit`
// where `masked`, moves the running maximum, and gives hi and lo operands
// 256 p = hi + lo / 16.
template <int D>
__device__ __forceinline__ void softmax_tile(f32x4 (&s)[8], Rows<D> &r, float c, bool masked,
                                             int limit, i32x8 &hi, i32x8 &lo) {
  if (masked) {
#pragma unroll
    for (int t = 0; t < 8; t++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (64 * (t >> 2) + 4 * (t & 3) + i > limit) s[t][i] = -__builtin_inff();
  }
  float top = s[0][0];
#pragma unroll
  for (int t = 0; t < 8; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) top = __builtin_fmaxf(top, s[t][i]);
  top = __builtin_fmaxf(top, __shfl_xor(top, 16));
  top = __builtin_fmaxf(top, __shfl_xor(top, 32));
  const float m = __builtin_fmaxf(r.m, top * c);
  const float ms = m == -__builtin_inff() ? 0.0f : m;  // nothing seen yet: weights are 0
  if (__any(m != r.m)) {
    const float alpha = __builtin_amdgcn_exp2f(r.m - ms);
#pragma unroll
    for (int d = 0; d < D / 16; d++) r.o[d] *= alpha;
    r.l *= alpha;
    r.m = m;
  }
  const float to8 = 8.0f - ms;  // 256 p
#pragma unroll
  for (int t = 0; t < 8; t++) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; i++) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], c, to8));
    uint32_t a, b;
    split4(p, 1.0f, 0.0625f, a, b);
    hi[t] = (int)a;
    lo[t] = (int)b;
  }
}

constexpr uint32_t kHi = 127 - 8, kLo = 127 - 12;  // bytes of the weights' two parts

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
  const int i = find_sequence(a.b.cu, a.b.batch, a.block_tokens, 1, unit);
  const int c0 = a.b.cu[i], n = a.b.cu[i + 1] - c0;
  const int at = (unit - (c0 / a.block_tokens + i)) * a.block_tokens;
  if (at >= n || at < 0 || c0 < 0 || (int64_t)c0 + n > a.b.tokens) return false;
  const int64_t room = (int64_t)a.b.width << a.shift;
  b.len = (int)min((int64_t)max(a.b.lengths[i], 0), room);
  b.tok0 = c0 + at;
  b.count = min(a.block_tokens, n - at);
  b.seen0 = b.len - n + at + 1;
  b.table = a.b.table + (int64_t)i * a.b.width;
  b.last_page = max(0, (b.len - 1) >> a.shift);
  return true;
}

// The pages of the four runs of 32 tokens of tile `tile`, past the end the last page.
struct Pages {
  int id[4];
};
__device__ __forceinline__ Pages pages_of(const AttnArgs &a, const Block &b, int tile) {
  Pages p;
#pragma unroll
  for (int j = 0; j < 4; j++)
    p.id[j] = clamp_page(b.table[min((tile * 128 + 32 * j) >> a.shift, b.last_page)], a.c.pages);
  return p;
}
__device__ __forceinline__ int pick4(const int (&x)[4], int i) {
  const int a = (i & 1) ? x[1] : x[0], b = (i & 1) ? x[3] : x[2];
  return (i & 2) ? b : a;
}

// Scale bytes of a tile as the matrix core wants them. A page whose values
// are NaN must reach only the rows that see it: its keys are made NaN
// instead (masked scores are dropped, visible ones make the row NaN) and its
// values, whose codes are signed zeros, get a finite scale.
struct TileScales {
  uint32_t k[2], v;
};
__device__ __forceinline__ TileScales scales_of(const AttnArgs &a, const Pages &p, int head,
                                                int l16, int lg) {
  int ks[4], vs[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int64_t at = (int64_t)p.id[j] * a.c.heads + head;
    vs[j] = a.c.v_scales[at];
    ks[j] = vs[j] == 255 ? 255 : a.c.k_scales[at];
    vs[j] = vs[j] == 255 ? 127 : vs[j];
  }
  TileScales s;
  s.k[0] = (uint32_t)((l16 & 8) ? ks[1] : ks[0]);
  s.k[1] = (uint32_t)((l16 & 8) ? ks[3] : ks[2]);
  s.v = (uint32_t)pick4(vs, lg);
  return s;
}

template <int D>
__device__ __forceinline__ void scores(const i32x8 *kv, const Query<D> &q, const TileScales &sc,
                                       f32x4 (&s)[8]) {
#pragma unroll
  for (int t = 0; t < 8; t++) {
    s[t] = mma(kv[t], q.v[0], f32x4{0, 0, 0, 0}, sc.k[t >> 2], q.byte[0]);
    if constexpr (D == 128) s[t] = mma(kv[t], q.v[1], s[t], sc.k[t >> 2], q.byte[1]);
  }
}

__device__ __forceinline__ i32x8 ones() {
  const int w = 0x38383838;
  return i32x8{w, w, w, w, w, w, w, w};
}

// One lane's run of outputs of a row: 4 D / 16 consecutive numbers.
template <int D>
__device__ __forceinline__ void store_out(uint16_t *p, const float (&v)[D / 4]) {
#pragma unroll
  for (int j = 0; j < D / 4; j += 8)
    *reinterpret_cast<u32x4 *>(p + j) =
        u32x4{pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]),
              pack_bf16(v[j + 4], v[j + 5]), pack_bf16(v[j + 6], v[j + 7])};
}

// Few rows: a workgroup of four waves takes up to 16 RT rows of one sequence
// and kv head and one split of its keys; wave w takes tiles w, w + 4, ....
template <int D, int RT>
__global__ __launch_bounds__(256) void k_attn_rows(const AttnArgs a) {
  constexpr int DT = D / 16, W = 4;
  __shared__ float merge_o[W][16][D + 4];
  __shared__ float merge_ml[W][16][2];
  Block b;
  if (!find_block(a, blockIdx.x, b)) return;
  const int head = blockIdx.y, split = blockIdx.z;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int end = min(b.len, b.seen0 + b.count - 1);  // keys any row sees
  const int tiles = (max(end, 0) + 127) >> 7;
  // (the last split takes whatever the caller's bound on the lengths left out)
  const int t0 = split * a.chunk, t1 = split + 1 == a.splits ? tiles : min(tiles, t0 + a.chunk);
  if (split > 0 && t0 >= tiles) return;  // the sum takes only splits that exist
  const int rows = b.count * a.group;

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
  const int64_t PD = (int64_t)a.c.page * D;
  const int mask = a.c.page - 1;
  Pages pg;
  if (t0 + wave < t1) pg = pages_of(a, b, t0 + wave);
  for (int tile = t0 + wave; tile < t1; tile += W) {
    const TileScales sc = scales_of(a, pg, head, l16, lg);
    i32x8 kv[8], vv[DT];
    // keys: row (token) of this lane in tile t; its page by run of 32 tokens
    const uint8_t *kp[2], *vp[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      kp[h] = a.c.k_codes + ((int64_t)((l16 & 8) ? pg.id[2 * h + 1] : pg.id[2 * h]) * a.c.heads + head) * PD;
      vp[h] = a.c.v_codes + ((int64_t)((lg & 2) ? pg.id[2 * h + 1] : pg.id[2 * h]) * a.c.heads + head) * PD;
    }
#pragma unroll
    for (int t = 0; t < 8; t++) {
      const int tok = tile * 128 + 64 * (t >> 2) + 16 * (l16 >> 2) + 4 * (t & 3) + (l16 & 3);
      const uint8_t *p = kp[t >> 2] + (tok & mask) * D + 16 * lg;
      const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
      if constexpr (D == 128)
        kv[t] = join8(x, __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + 64)));
      else
        kv[t] = join8(x, x);
    }
#pragma unroll
    for (int d = 0; d < DT; d++) {
      const int dim = 4 * DT * (l16 >> 2) + 4 * d + (l16 & 3);
      const int s0 = (tile * 128 + 16 * lg) & mask, s1 = (tile * 128 + 64 + 16 * lg) & mask;
      vv[d] = join8(__builtin_nontemporal_load(
                        reinterpret_cast<const u32x4 *>(vp[0] + (int64_t)dim * a.c.page + s0)),
                    __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4 *>(vp[1] + (int64_t)dim * a.c.page + s1)));
    }
    if (tile + W < t1) pg = pages_of(a, b, tile + W);
    const bool tail = tile * 128 + 128 > b.len;
    const bool masked = tile * 128 + 128 > b.seen0;
    if (tail) {
#pragma unroll
      for (int d = 0; d < DT; d++) {
        const u32x4 lo = {(uint32_t)vv[d][0], (uint32_t)vv[d][1], (uint32_t)vv[d][2], (uint32_t)vv[d][3]};
        const u32x4 hi = {(uint32_t)vv[d][4], (uint32_t)vv[d][5], (uint32_t)vv[d][6], (uint32_t)vv[d][7]};
        const int from = b.len - tile * 128 - 16 * lg;
        vv[d] = join8(keep_tokens(lo, from), keep_tokens(hi, from - 64));
      }
    }
#pragma unroll
    for (int x = 0; x < RT; x++) {
      f32x4 s[8];
      scores<D>(kv, q[x], sc, s);
      i32x8 hi, lo;
      softmax_tile<D>(s, r[x], a.scale2, masked, seen[x] - 1 - tile * 128 - 16 * lg, hi, lo);
#pragma unroll
      for (int d = 0; d < DT; d++) {
        r[x].o[d] = mma(vv[d], hi, r[x].o[d], sc.v, kHi);
        r[x].o[d] = mma(vv[d], lo, r[x].o[d], sc.v, kLo);
      }
      r[x].l = mma(ones(), hi, r[x].l, 127, kHi);
      r[x].l = mma(ones(), lo, r[x].l, 127, kLo);
    }
  }
  // merge the four waves, 16 rows at a time
#pragma unroll
  for (int x = 0; x < RT; x++) {
    if (x) __syncthreads();
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int e = 0; e < 4; e++) merge_o[wave][l16][4 * DT * lg + 4 * d + e] = r[x].o[d][e];
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
      for (int e = 0; e < D / 16; e++) o[e] += f * merge_o[w][row][d0 + e];
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

// Joins the splits of one (token, query head): a wave, two (one) dims a lane.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= a.b.tokens * a.q_heads) return;
  const int tok = (int)(row / a.q_heads);
  // the token's sequence and how many keys its block saw, as the first kernel had it
  int lo = 0, hi = a.b.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.b.cu[mid] <= tok) lo = mid;
    else hi = mid - 1;
  }
  const int c0 = a.b.cu[lo], n = a.b.cu[lo + 1] - c0;
  const int64_t room = (int64_t)a.b.width << a.shift;
  const int len = (int)min((int64_t)max(a.b.lengths[lo], 0), room);
  const int at = (tok - c0) / a.block_tokens * a.block_tokens;
  const int end = min(len, len - n + at + min(a.block_tokens, n - at));
  const int tiles = (max(end, 0) + 127) >> 7;
  const int live = max(1, min(a.splits, (tiles + a.chunk - 1) / a.chunk));
  const float *p = a.part + row * a.splits * (D + 4);
  float m = -__builtin_inff();
  for (int s = 0; s < live; s++) m = __builtin_fmaxf(m, p[(int64_t)s * (D + 4) + D]);
  const float ms = m == -__builtin_inff() ? 0.0f : m;
  float l = 0.0f, o[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; e++) o[e] = 0.0f;
  for (int s = 0; s < live; s++) {
    const float *ps = p + (int64_t)s * (D + 4);
    const float f = __builtin_amdgcn_exp2f(ps[D] - ms);
    l += f * ps[D + 1];
#pragma unroll
    for (int e = 0; e < D / 64; e++) o[e] += f * ps[lane * (D / 64) + e];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t *out = a.out + row * D + lane * (D / 64);
  if constexpr (D == 128) *reinterpret_cast<uint32_t *>(out) = pack_bf16(o[0] * inv, o[1] * inv);
  else *out = (uint16_t)pack_bf16(o[0] * inv, 0.0f);
}

// Many rows: four waves of 32 rows share tiles of 128 tokens through LDS,
// loaded directly and double-buffered. Rows are `tokens x group` of one kv
// head. Chunks of 16 bytes are swapped within their row so that the 16 rows
// a read touches spread over all banks.
template <int D>
__device__ __forceinline__ int swz_k(int r) {
  if constexpr (D == 128) return ((r >> 1) & 1) | (((r >> 4) & 3) << 1);
  return (r >> 4) & 3;
}
template <int D>
__device__ __forceinline__ int swz_v(int r) {
  return ((r >> 1) & 1) | (((r / (D / 4)) & 3) << 1);
}

template <int D>
__global__ __launch_bounds__(256, 2) void k_attn_tiles(const AttnArgs a) {
  constexpr int DT = D / 16, RT = 2, T = 256;
  constexpr int KL = 128 * D / 16 / T, VL = KL;  // direct loads per thread and tile
  __shared__ __attribute__((aligned(16))) uint8_t ks[2][128 * D], vs[2][128 * D];
  Block b;
  // the last blocks of a sequence see the most keys: they start first
  if (!find_block(a, gridDim.x - 1 - blockIdx.x, b)) return;
  const int head = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int end = min(b.len, b.seen0 + b.count - 1);
  const int tiles = (max(end, 0) + 127) >> 7;
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
  const int mask = a.c.page - 1;
  auto load = [&](int tile, int buf, const Pages &pg) {
#pragma unroll
    for (int i = 0; i < KL; i++) {
      constexpr int CH = D / 16;  // chunks per row
      const int e = i * T + (int)threadIdx.x, row = e / CH, c = (e % CH) ^ swz_k<D>(row);
      const uint8_t *src = a.c.k_codes +
                           ((int64_t)pick4(pg.id, row >> 5) * a.c.heads + head) * PD +
                           ((tile * 128 + row) & mask) * D + 16 * c;
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void *)src,
          (__attribute__((address_space(3))) void *)(ks[buf] + (i * T + wave * 64) * 16), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < VL; i++) {
      const int e = i * T + (int)threadIdx.x, row = e >> 3, c = (e & 7) ^ swz_v<D>(row);
      const uint8_t *src = a.c.v_codes + ((int64_t)pick4(pg.id, c >> 1) * a.c.heads + head) * PD +
                           (int64_t)row * a.c.page + ((tile * 128 + 16 * c) & mask);
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void *)src,
          (__attribute__((address_space(3))) void *)(vs[buf] + (i * T + wave * 64) * 16), 16, 0, 0);
    }
  };
  Pages pg, nx;
  if (tiles > 0) {
    pg = pages_of(a, b, 0);
    load(0, 0, pg);
  }
  for (int tile = 0; tile < tiles; tile++) {
    const int buf = tile & 1;
    const TileScales sc = scales_of(a, pg, head, l16, lg);
    if (tile + 1 < tiles) nx = pages_of(a, b, tile + 1);
    // this tile's loads have landed, and every wave is done with the other buffer
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tile + 1 < tiles) load(tile + 1, buf ^ 1, nx);
    f32x4 s[RT][8];
#pragma unroll
    for (int t = 0; t < 8; t++) {
      const int row = 64 * (t >> 2) + 16 * (l16 >> 2) + 4 * (t & 3) + (l16 & 3);
      const uint8_t *p = ks[buf] + row * D;
      const u32x4 lo = *reinterpret_cast<const u32x4 *>(p + 16 * (lg ^ swz_k<D>(row)));
      u32x4 hi = lo;
      if constexpr (D == 128) hi = *reinterpret_cast<const u32x4 *>(p + 16 * ((lg + 4) ^ swz_k<D>(row)));
      const i32x8 kv = join8(lo, hi);
#pragma unroll
      for (int x = 0; x < RT; x++) {
        s[x][t] = mma(kv, q[x].v[0], f32x4{0, 0, 0, 0}, sc.k[t >> 2], q[x].byte[0]);
        if constexpr (D == 128) s[x][t] = mma(kv, q[x].v[1], s[x][t], sc.k[t >> 2], q[x].byte[1]);
      }
    }
    const bool masked = tile * 128 + 128 > b.seen0;
    i32x8 hi[RT], lo[RT];
#pragma unroll
    for (int x = 0; x < RT; x++)
      softmax_tile<D>(s[x], r[x], a.scale2, masked, seen[x] - 1 - tile * 128 - 16 * lg, hi[x], lo[x]);
    const bool tail = tile * 128 + 128 > b.len;
#pragma unroll
    for (int d = 0; d < DT; d++) {
      const int row = 4 * DT * (l16 >> 2) + 4 * d + (l16 & 3);
      const uint8_t *p = vs[buf] + row * 128;
      u32x4 v0 = *reinterpret_cast<const u32x4 *>(p + 16 * (lg ^ swz_v<D>(row)));
      u32x4 v1 = *reinterpret_cast<const u32x4 *>(p + 16 * ((lg + 4) ^ swz_v<D>(row)));
      if (tail) {
        const int from = b.len - tile * 128 - 16 * lg;
        v0 = keep_tokens(v0, from);
        v1 = keep_tokens(v1, from - 64);
      }
      const i32x8 vv = join8(v0, v1);
#pragma unroll
      for (int x = 0; x < RT; x++) {
        r[x].o[d] = mma(vv, hi[x], r[x].o[d], sc.v, kHi);
        r[x].o[d] = mma(vv, lo[x], r[x].o[d], sc.v, kLo);
      }
    }
#pragma unroll
    for (int x = 0; x < RT; x++) {
      r[x].l = mma(ones(), hi[x], r[x].l, 127, kHi);
      r[x].l = mma(ones(), lo[x], r[x].l, 127, kLo);
    }
    pg = nx;
  }
#pragma unroll
  for (int x = 0; x < RT; x++) {
    const int row = 32 * wave + 16 * x + l16;
    if (row < rows) {
      const float l = r[x].l[0], inv = l == 0.0f ? 0.0f : 1.0f / l;
      float v[D / 4];
#pragma unroll
      for (int d = 0; d < DT; d++)
#pragma unroll
        for (int e = 0; e < 4; e++) v[4 * d + e] = r[x].o[d][e] * inv;
      const int64_t tok = b.tok0 + row / a.group;
      const int64_t qh = (int64_t)head * a.group + row % a.group;
      store_out<D>(a.out + (tok * a.q_heads + qh) * D + 4 * DT * lg, v);
    }
  }
}

static int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) s++;
  return s;
}

struct AttnPlan {
  bool few;
  int rt, block_tokens, chunk, splits;
  int64_t units;
};
static AttnPlan attn_plan(int64_t tokens, int batch, int q_heads, int heads, int64_t max_length) {
  AttnPlan p;
  const int group = q_heads / heads;
  const int64_t mean = (tokens + batch - 1) / batch * group;  // rows of a sequence
  p.few = mean <= 32 && group <= 32;
  p.rt = p.few ? (mean <= 16 && group <= 16 ? 1 : 2) : 2;
  p.block_tokens = (p.few ? 16 * p.rt : 128) / group;
  p.units = tokens / p.block_tokens + batch;
  const int tiles = (int)((max_length + 127) / 128);
  p.chunk = tiles > 0 ? tiles : 1;
  p.splits = 1;
  if (p.few) {
    // enough workgroups to fill the card twice over; at least a tile a wave
    const int64_t base = std::max<int64_t>(1, (int64_t)batch * heads);
    const int64_t want = std::max<int64_t>(1, 4096 / base);
    const int64_t c = std::max<int64_t>(4, (tiles + want - 1) / want);
    p.chunk = (int)((c + 3) / 4 * 4);
    p.splits = std::max(1, (tiles + p.chunk - 1) / p.chunk);
  }
  return p;
}

}  // namespace mxl

using namespace mxl;

hipError_t mxi_launch_kv_append(const void *k, const void *v, int bf16, int64_t k_stride,
                                int64_t v_stride, const mx_kv_cache_t &cache,
                                const mx_kv_batch_t &batch, hipStream_t st) {
  const AppendArgs a = {k, v, k_stride, v_stride, cache, batch, log2_of(cache.page)};
  const dim3 grid((uint32_t)(batch.tokens / cache.page + 2 * (int64_t)batch.batch),
                  (uint32_t)cache.heads);
  if (bf16) k_kv_append<true><<<grid, 256, 0, st>>>(a);
  else k_kv_append<false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

size_t mxi_kv_attention_workspace(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                  int64_t max_length) {
  const AttnPlan p = attn_plan(tokens, batch, q_heads, heads, max_length);
  return p.splits > 1 ? (size_t)tokens * q_heads * p.splits * (dim + 4) * sizeof(float) : 0;
}

hipError_t mxi_launch_kv_attention(const void *q, int64_t q_stride, int q_heads,
                                   const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                                   int64_t max_length, float scale, void *out, void *workspace,
                                   hipStream_t st) {
  const AttnPlan p = attn_plan(batch.tokens, batch.batch, q_heads, cache.heads, max_length);
  const AttnArgs a = {reinterpret_cast<const uint16_t *>(q), q_stride, q_heads,
                      q_heads / cache.heads, cache, batch, log2_of(cache.page), p.block_tokens,
                      p.chunk, p.splits, scale * 1.44269504088896340736f,
                      reinterpret_cast<uint16_t *>(out), reinterpret_cast<float *>(workspace)};
  const dim3 grid((uint32_t)p.units, (uint32_t)cache.heads, (uint32_t)p.splits);
  if (!p.few) {
    if (cache.dim == 64) k_attn_tiles<64><<<grid, 256, 0, st>>>(a);
    else k_attn_tiles<128><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
  }
  if (cache.dim == 64) {
    if (p.rt == 1) k_attn_rows<64, 1><<<grid, 256, 0, st>>>(a);
    else k_attn_rows<64, 2><<<grid, 256, 0, st>>>(a);
  } else {
    if (p.rt == 1) k_attn_rows<128, 1><<<grid, 256, 0, st>>>(a);
    else k_attn_rows<128, 2><<<grid, 256, 0, st>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 jgrid((uint32_t)((batch.tokens * q_heads + 3) / 4));
  if (cache.dim == 64) k_attn_join<64><<<jgrid, 256, 0, st>>>(a);
  else k_attn_join<128><<<jgrid, 256, 0, st>>>(a);
  return hipGetLastError();
}
