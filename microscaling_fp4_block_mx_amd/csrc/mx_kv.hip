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
// itself however far below the largest it lies, down to 2^-126. (Two E4M3 parts,
// as q has, end 2^-22 below the largest weight: a tail of many such keys is lost.) The
// weights' sum is a product with a row of ones, of the weights as rounded.
//
// Three kernels. Few rows (single tokens) are bound by reading the cache: one
// wave per 128 tokens at a time, the sequence split over workgroups. With
// g = lane / 16, tile t (of 16 rows) and accumulator i hold token 64 (t / 4) +
// 16 g + 4 (t % 4) + i of 128, and the second product's lane holds tokens
// 16 g .. + 15 and 64 + 16 g .. + 15.
//
// Many rows (prompts) share tiles of 128 tokens through LDS and are bound by
// instruction issue: per 32 rows and 128 tokens, 2,200 cycles of products
// beside 2,400 of vector arithmetic, half of it the exponentials. There the
// workgroup widens the values once. Token 32 (t / 2) + 8 g + 4 (t % 2) + i.
//
// Trees of drafted tokens lie between: the second kernel's way through a tile, with
// the tiles of a whole batch shared out evenly, and a join of its own.
#include <algorithm>

#include "mx_layer.h"
#include "mx_rotary_device.h"

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
  // keys through a norm and a rotation on the way, where the kernel has them
  const void *weight;  // or NULL: no norm
  float eps;
  mx_rotary_t r;
};

// Which sequence a unit of work belongs to: sequence i owns units from
// units(cu[i]) + extra i on, units being a quotient by some number `per`, which
// leaves it at least n / per + extra. The
// wave's lanes look at up to 64 sequences at once (one trip to memory for up
// to 64 sequences, two up to 4096).
template <typename F>
__device__ __forceinline__ int find_sequence(const int32_t *cu, int batch, F units, int extra, int unit) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 63) >> 6, at = lo + lane * step;
    const bool below = lane * step < n && units(cu[at]) + extra * at <= unit;
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

// The first `keep` of 16 codes moved, the others as they are.
__device__ __forceinline__ u32x4 move16(u32x4 v, int keep, int d, bool nan) {
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const int n = min(max(keep - 4 * e, 0), 4);
    const uint32_t mask = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1;
    w[e] = (move4(v[e], d, nan) & mask) | (v[e] & ~mask);
  }
  return w;
}

// Items of eight elements that a thread keeps between the two passes (what a
// page of 64 tokens of 128 dims takes); larger pages read the rest twice.
constexpr int kKeep = 4;

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_at(const void *base, int64_t elem) {
  return load_raw<BF16>(reinterpret_cast<const uint8_t *>(base) + elem * (BF16 ? 2 : 4), 0);
}

// A workgroup's page of a sequence, and its head.
struct AppendPage {
  int head, page;       // the page's number in its sequence
  int kept, end;        // slots that stay, slots in use after
  int64_t src0, most;   // token of slot 0; the last token there is
  int64_t at;           // of the page and head in the scales
  __device__ __forceinline__ int64_t token(int slot) const { return min(max(src0 + slot, (int64_t)0), most); }
};
// TOGETHER: the heads of a page run on one of the eight XCDs, which are dealt
// workgroups in turn (its cache then has what they share).
template <bool TOGETHER>
__device__ __forceinline__ bool find_page(const AppendArgs &a, AppendPage &p) {
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= a.blocks) return false;
  const int P = a.c.page;
  int unit;
  if constexpr (TOGETHER) {
    unit = (block >> 3) / a.c.heads * 8 + (block & 7);
    p.head = (block >> 3) % a.c.heads;
  } else {
    unit = block / a.c.heads;
    p.head = block % a.c.heads;
  }
  auto pages = [&](int tokens) { return (tokens + (tokens >> 31 & (P - 1))) >> a.shift; };  // tokens / P
  const int i = find_sequence(a.b.cu, a.b.batch, pages, 2, unit);
  const int c0 = a.b.cu[i], n = a.b.cu[i + 1] - c0, held = a.b.lengths[i];
  const int j = (held >> a.shift) + (unit - (pages(c0) + 2 * i));  // page of the sequence
  // (a unit before the first sequence's has pages before the sequence's first)
  if (n <= 0 || held < 0 || j < held >> a.shift || j >= a.b.width || ((int64_t)j << a.shift) >= (int64_t)held + n)
    return false;
  p.page = j;
  p.kept = max(0, held - (j << a.shift));
  p.end = min((int64_t)P, (int64_t)held + n - ((int64_t)j << a.shift));
  const int64_t id = a.b.table[(int64_t)i * a.b.width + j];
  if (id < 0 || id >= a.c.pages) return false;  // no page: its tokens are dropped
  p.src0 = (int64_t)c0 + ((int64_t)j << a.shift) - held;
  p.most = a.b.tokens - 1;
  p.at = id * a.c.heads + p.head;
  return true;
}

// Items of eight dims of a token. Lanes l, l + 16, l + 32, l + 48 of a wave hold
// four tokens that share a word of a values' row.
struct AppendItems {
  int first, kept, end, wide;
  __device__ __forceinline__ AppendItems(const AppendPage &p, int dim)
      : first(p.kept & ~3), kept(p.kept), end(p.end), wide(dim == 128) {}
  __device__ __forceinline__ int word(int it) const {  // first of the four slots
    return first + (wide ? it >> 6 << 2 : (it >> 6 << 3) + ((it & 8) >> 1));
  }
  __device__ __forceinline__ int slot(int it) const { return word(it) + ((it >> 4) & 3); }
  __device__ __forceinline__ int dim(int it) const { return (it & (wide ? 15 : 7)) * 8; }
  // whether any lane of the wave has a slot in use: the wave's lanes go together
  __device__ __forceinline__ bool any(int it) const { return first + (wide ? it >> 6 << 2 : it >> 6 << 3) < end; }
  __device__ __forceinline__ bool mine(int it) const { return slot(it) >= kept && slot(it) < end; }
};

// Largest over the workgroup of two numbers that its threads have; `am` is this
// call's own.
template <int T>
__device__ __forceinline__ void largest2(uint32_t &x, uint32_t &y, uint32_t (&am)[2][T / 64]) {
  x = max16(x);
  y = max16(y);
  x = max(x, (uint32_t)__shfl_xor((int)x, 16));
  y = max(y, (uint32_t)__shfl_xor((int)y, 16));
  x = max(x, (uint32_t)__shfl_xor((int)x, 32));
  y = max(y, (uint32_t)__shfl_xor((int)y, 32));
  if ((threadIdx.x & 63) == 0) {
    am[0][threadIdx.x >> 6] = x;
    am[1][threadIdx.x >> 6] = y;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; w++) {
    x = max(x, am[0][w]);
    y = max(y, am[1][w]);
  }
}

// Kept codes move to a new byte 16 at a time, four such pieces asked for
// together; what a piece holds past the kept tokens stays.
template <int T, typename F, typename G>
__device__ __forceinline__ void move_codes(int pieces, F place, G keeps, int d, bool nan) {
  for (int c = threadIdx.x; c < pieces; c += 4 * T) {
    u32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; u++) v[u] = *reinterpret_cast<const u32x4 *>(place(min(c + u * T, pieces - 1)));
#pragma unroll
    for (int u = 0; u < 4; u++) {
      if (c + u * T >= pieces) break;
      *reinterpret_cast<u32x4 *>(place(c + u * T)) = move16(v[u], keeps(c + u * T), d, nan);
    }
  }
}
template <int T>
__device__ __forceinline__ void move_keys(uint8_t *kc, int kept, int D, uint32_t from, uint32_t to) {
  if (kept && to > from)
    move_codes<T>(kept * D / 16, [&](int c) { return kc + 16 * c; }, [](int) { return 16; }, (int)(to - from), to == 255u);
}
template <int T>
__device__ __forceinline__ void move_values(uint8_t *vc, int kept, int D, int P, uint32_t from, uint32_t to) {
  if (!kept || to <= from) return;
  const int n = (kept + 15) >> 4;
  move_codes<T>(D * n, [&](int c) { return vc + c / n * P + c % n * 16; }, [&](int c) { return kept - c % n * 16; },
                (int)(to - from), to == 255u);
  __syncthreads();  // before the new tokens' bytes of the same words
}

// a kept byte may be any: above 246 every finite number is below 448 scales
__device__ __forceinline__ float append_limit(uint32_t b) { return b > 246u ? 0x1.fffffep127f : limit8(b); }

// A value item's codes into vt, [dim][token], whose rows are `row` bytes.
template <bool BF16>
__device__ __forceinline__ void put_value(uint8_t *vt, int row, const AppendItems &items, const Raw<BF16> &v, int it,
                                          uint32_t byte, float most) {
  float f[8];
  widen<BF16>(v, f);
  const u32x2 w = encode8(f, byte, most);
  // four lanes' tokens t = 2 b + a, eight dims each, become two dims of four
  // tokens: halves of the dims change places over b, then quarters over a
  const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
  const uint32_t lo = __builtin_amdgcn_perm(x[1], x[0], 0x05040100u);  // dims 0, 1 of tokens a, a + 2
  const uint32_t hi = __builtin_amdgcn_perm(x[1], x[0], 0x07060302u);  // dims 2, 3
  const auto y = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
  uint32_t *to = reinterpret_cast<uint32_t *>(vt + (items.dim(it) + 2 * ((it >> 4) & 3)) * row + items.word(it));
  to[0] = __builtin_amdgcn_perm(y[1], y[0], 0x06020400u);
  to[row >> 2] = __builtin_amdgcn_perm(y[1], y[0], 0x07030501u);
}
// The new tokens' bytes from vt to the page.
template <int T>
__device__ __forceinline__ void write_values(uint8_t *vc, const uint8_t *vt, int row, int kept, int end, int D, int P) {
  const int piece0 = kept >> 4, chunks = ((end + 15) >> 4) - piece0;  // of a row, with new tokens in them
  const bool all = chunks == P >> 4;  // a power of two
  const int shift = 31 - __builtin_clz(P >> 4);
  for (int it = threadIdx.x; it < D * chunks; it += T) {
    const int d = all ? it >> shift : it / chunks, s = (piece0 + it - d * chunks) * 16;
    const int lo = max(kept, s), hi = min(end, s + 16);
    uint8_t *dst = vc + (int64_t)d * P;
    if (lo == s && hi == s + 16) {
      const uint32_t *from = reinterpret_cast<const uint32_t *>(vt + d * row + s);
      *reinterpret_cast<u32x4 *>(dst + s) = u32x4{from[0], from[1], from[2], from[3]};
    } else {
      for (int q = lo; q < hi; q++) dst[q] = vt[d * row + q];
    }
  }
}

// One workgroup per page and head. Prompts are bound by HBM: 6 sequences of up
// to 8,000 tokens, 8 heads of 128, 201 MB in 41 us (4.9 TB/s); with the values'
// bytes written to LDS one at a time 44.6, with the tokens read twice 72. A
// token per sequence is a chain of loads that wait for each other (cu, table
// and lengths, scale, codes): 64 sequences 5 us, 256 8.5.
template <bool BF16, int T>
__global__ __launch_bounds__(T) void k_kv_append(const AppendArgs a) {
  // new values' codes, [dim][token]; rows are one word longer than a page's,
  // so that the rows that an instruction writes to fall on different banks
  extern __shared__ __attribute__((aligned(16))) uint8_t vt[];
  __shared__ uint32_t am[2][T / 64];
  AppendPage p;
  if (!find_page<false>(a, p)) return;
  const int P = a.c.page, D = a.c.dim;
  const AppendItems items(p, D);
  uint32_t was_k = 0, was_v = 0;
  if (p.kept) {
    was_k = a.c.k_scales[p.at];
    was_v = a.c.v_scales[p.at];
  }
  auto load = [&](const void *x, int64_t stride, int it) {
    return load_at<BF16>(x, p.token(items.slot(it)) * stride + (int64_t)p.head * D + items.dim(it));
  };
  Raw<BF16> kr[kKeep], vr[kKeep];
#pragma unroll
  for (int u = 0; u < kKeep; u++) {
    const int it = threadIdx.x + T * u;
    kr[u] = vr[u] = Raw<BF16>{};
    if (items.mine(it)) {
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
  for (int it = threadIdx.x + T * kKeep; items.any(it); it += T)
    if (items.mine(it)) take(load(a.k, a.k_stride, it), load(a.v, a.v_stride, it));
  largest2<T>(mk, mv, am);
  const uint32_t sk = max(scale_byte8(mk), was_k), sv = max(scale_byte8(mv), was_v);
  uint8_t *kc = a.c.k_codes + p.at * P * D, *vc = a.c.v_codes + p.at * P * D;
  move_keys<T>(kc, p.kept, D, was_k, sk);
  move_values<T>(vc, p.kept, D, P, was_v, sv);
  const float most_k = append_limit(sk), most_v = append_limit(sv);
  const int row = P + 4;
  auto put = [&](const Raw<BF16> &k, const Raw<BF16> &v, int it) {
    if (items.mine(it)) {
      float f[8];
      widen<BF16>(k, f);
      *reinterpret_cast<u32x2 *>(kc + items.slot(it) * D + items.dim(it)) = encode8(f, sk, most_k);
    }
    put_value<BF16>(vt, row, items, v, it, sv, most_v);
  };
#pragma unroll
  for (int u = 0; u < kKeep; u++)
    if (items.any(threadIdx.x + T * u)) put(kr[u], vr[u], threadIdx.x + T * u);
  for (int it = threadIdx.x + T * kKeep; items.any(it); it += T)
    put(load(a.k, a.k_stride, it), load(a.v, a.v_stride, it), it);
  __syncthreads();
  write_values<T>(vc, vt, row, p.kept, p.end, D, P);
  if (threadIdx.x == 0) {
    if (!p.kept || sk != was_k) a.c.k_scales[p.at] = (uint8_t)sk;
    if (!p.kept || sv != was_v) a.c.v_scales[p.at] = (uint8_t)sv;
  }
}

// The same with the keys' norm (if there is a weight) and rotation on the way, in
// 64 bits: a page's byte changes where its largest number crosses a power of two,
// so the last bit of a key can be one of the byte. dim / 16 lanes hold a token's
// key, two items each, both members of a pair in one lane. The values go first,
// while the keys are on their way: what is held of the two at once decides how
// many waves a unit has.
template <bool BF16, int T, int D, bool PAIRED>
__global__ __launch_bounds__(T, BF16 ? 4 : 1) void k_kv_append_rotary(const AppendArgs a) {
  constexpr int kTurn = kKeep / 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t vt[];
  __shared__ uint32_t am[2][2][T / 64];
  AppendPage p;
  if (!find_page<(T > 64)>(a, p)) return;
  const int P = a.c.page;
  const AppendItems items(p, D);
  // the same for all threads, and in scalar registers: the branches that they
  // decide are the workgroup's
  auto uniform = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); };
  uint32_t was_k = 0, was_v = 0;
  if (p.kept) {
    was_k = uniform(a.c.k_scales[p.at]);
    was_v = uniform(a.c.v_scales[p.at]);
  }
  auto load_value = [&](int it) {
    return load_at<BF16>(a.v, p.token(items.slot(it)) * a.v_stride + (int64_t)p.head * D + items.dim(it));
  };
  // Key item `it` is lane t of a token, dims 8 ka .. and 8 kb ... (T is a multiple
  // of the lanes of a token: t, ka and kb are the same for all of a thread's items.)
  constexpr int lanes = D / 16;
  const int t = threadIdx.x % lanes;
  auto slot_of = [&](int it) { return p.kept + it / lanes; };
  int ka, kb;
  bool turns;
  items_of<PAIRED>(t, a.r.rot, ka, kb, turns);
  Raw<BF16> wa = {}, wb = {};
  if (a.weight) {
    wa = load_weight<BF16>(a.weight, ka);
    wb = load_weight<BF16>(a.weight, kb);
  }
  struct Key {
    Raw<BF16> a, b;
    int position;
  };
  auto load_key = [&](int it) {
    Key k;
    const int slot = slot_of(it);
    const int64_t tok = p.token(slot);
    const uint8_t *x = reinterpret_cast<const uint8_t *>(a.k) + (tok * a.k_stride + (int64_t)p.head * D) * (BF16 ? 2 : 4);
    k.a = load_raw<BF16>(x, ka);
    k.b = load_raw<BF16>(x, kb);
    k.position = a.r.positions && turns ? a.r.positions[tok] : (p.page << a.shift) + slot;
    return k;
  };
  struct Turned {  // as it enters the cache
    float a[8], b[8];
  };
  auto turned = [&](const Key &k) {
    double x[8], y[8];
    widen64<BF16>(k.a, x);
    widen64<BF16>(k.b, y);
    if (a.weight) {
      double ss = 0.0;
#pragma unroll
      for (int e = 0; e < 8; e++) ss = __builtin_fma(x[e], x[e], __builtin_fma(y[e], y[e], ss));
      const double root = inverse_root(sum_lanes<lanes>(ss) * (1.0 / D) + a.eps);
      // widened each time: held in 64 bits they would cost a wave of four
      renew<BF16>(wa);
      renew<BF16>(wb);
      float u[8], v[8];
      widen<BF16>(wa, u);
      widen<BF16>(wb, v);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        x[e] = x[e] * root * u[e];
        y[e] = y[e] * root * v[e];
      }
    }
    if (turns) {
      Turns angles;
      angles.load(a.r, k.position, t);
      turn<PAIRED, false>(x, y, angles.c, angles.s);
    }
    Turned r;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      r.a[e] = (float)x[e];
      r.b[e] = (float)y[e];
    }
    return r;
  };

  Raw<BF16> vr[kKeep];
  Key kr[kTurn];
#pragma unroll
  for (int u = 0; u < kKeep; u++) {
    const int it = threadIdx.x + T * u;
    vr[u] = Raw<BF16>{};
    if (items.mine(it)) vr[u] = load_value(it);
  }
#pragma unroll
  for (int u = 0; u < kTurn; u++)
    if (slot_of(threadIdx.x + T * u) < p.end) kr[u] = load_key(threadIdx.x + T * u);
  uint8_t *kc = a.c.k_codes + p.at * P * D, *vc = a.c.v_codes + p.at * P * D;
  const int row = P + 4;

  uint32_t mk = 0, mv = 0, none = 0;
  auto take = [&](const Raw<BF16> &v) {
    float f[8];
    widen<BF16>(v, f);
    mv = max(mv, amax8(f));
  };
#pragma unroll
  for (int u = 0; u < kKeep; u++) take(vr[u]);  // zeros where there is none
  for (int it = threadIdx.x + T * kKeep; items.any(it); it += T)
    if (items.mine(it)) take(load_value(it));
  largest2<T>(mv, none, am[0]);
  const uint32_t sv = max(scale_byte8(uniform(mv)), was_v);
  move_values<T>(vc, p.kept, D, P, was_v, sv);
  const float most_v = append_limit(sv);
#pragma unroll
  for (int u = 0; u < kKeep; u++)
    if (items.any(threadIdx.x + T * u)) put_value<BF16>(vt, row, items, vr[u], threadIdx.x + T * u, sv, most_v);
  for (int it = threadIdx.x + T * kKeep; items.any(it); it += T)
    put_value<BF16>(vt, row, items, load_value(it), it, sv, most_v);

  Turned tr[kTurn];
  auto take_key = [&](const Turned &r) { mk = max(mk, max(amax8(r.a), amax8(r.b))); };
#pragma unroll
  for (int u = 0; u < kTurn; u++)
    if (slot_of(threadIdx.x + T * u) < p.end) {  // (the lanes of a token go together)
      tr[u] = turned(kr[u]);
      take_key(tr[u]);
      __builtin_amdgcn_sched_barrier(0);  // one key's numbers at a time
    }
  for (int it = threadIdx.x + T * kTurn; slot_of(it) < p.end; it += T) take_key(turned(load_key(it)));
  largest2<T>(mk, none, am[1]);  // (and vt is whole)
  const uint32_t sk = max(scale_byte8(uniform(mk)), was_k);
  move_keys<T>(kc, p.kept, D, was_k, sk);
  const float most_k = append_limit(sk);
  auto put_key = [&](const Turned &r, int it) {
    uint8_t *to = kc + slot_of(it) * D;
    *reinterpret_cast<u32x2 *>(to + 8 * ka) = encode8(r.a, sk, most_k);
    *reinterpret_cast<u32x2 *>(to + 8 * kb) = encode8(r.b, sk, most_k);
  };
#pragma unroll
  for (int u = 0; u < kTurn; u++)
    if (slot_of(threadIdx.x + T * u) < p.end) put_key(tr[u], threadIdx.x + T * u);
  for (int it = threadIdx.x + T * kTurn; slot_of(it) < p.end; it += T) put_key(turned(load_key(it)), it);
  write_values<T>(vc, vt, row, p.kept, p.end, D, P);
  if (threadIdx.x == 0) {
    if (!p.kept || sk != was_k) a.c.k_scales[p.at] = (uint8_t)sk;
    if (!p.kept || sv != was_v) a.c.v_scales[p.at] = (uint8_t)sv;
  }
}

// ---- keep ---------------------------------------------------------------------------
//
// Accepted tokens of a tree, at held + path[j], move to held + j. A page that
// tokens move into gets the largest of its kept tokens' byte (where it has any)
// and those that the moved ones had; codes are rounded once more where their
// byte grows. A path's nodes come in order, so no token lies before where it
// goes: pages are done in order, and what a later one needs is still in place. A
// workgroup takes a sequence and head. Latency is all there is: counts, tables,
// bytes and codes, each a trip to memory that waits for the last.
struct KeepArgs {
  mx_kv_cache_t c;
  const int32_t *table, *lengths, *path, *count;
  int batch, width, path_width, shift;
};
constexpr int kMoved = 64;  // tokens on the move at a time

__global__ __launch_bounds__(256) void k_kv_keep(const KeepArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t ks[kMoved * 128], vs[kMoved * 128];
  __shared__ uint8_t kb[256], vb[256];  // bytes that a page's tokens come with
  __shared__ int from_page[256], from_slot[256];
  __shared__ int stays, ends;
  __shared__ uint32_t most_k, most_v;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= (int64_t)a.batch * a.c.heads) return;
  const int i = (int)(block / a.c.heads), head = (int)(block % a.c.heads), tid = threadIdx.x;
  const int P = a.c.page, D = a.c.dim, held = a.lengths[i];
  const int many = min(a.count[i], a.path_width);
  const int32_t *path = a.path + (int64_t)i * a.path_width;
  const int32_t *table = a.table + (int64_t)i * a.width;
  if (held < 0 || many <= 0) return;
  if (tid == 0) {
    stays = many;
    ends = many;
  }
  __syncthreads();
  for (int j = tid; j < many; j += 256) {
    const int p = path[j], last = j ? path[j - 1] : -1;
    if (p != j) atomicMin(&stays, j);
    // not in order, or past the table's room: the path ends there
    if (p <= last || (((int64_t)held + p) >> a.shift) >= a.width) atomicMin(&ends, j);
  }
  __syncthreads();
  const int first = stays, end = ends;
  if (first >= end) return;  // (end > 0: the last token to move lies inside the table)
  for (int page = (held + first) >> a.shift; page <= (held + end - 1) >> a.shift; page++) {
    const int begin = page << a.shift, lo = max(held + first, begin);
    const int n = min(held + end, begin + P) - lo, kept = lo - begin;
    const int64_t id = table[page];
    if (id < 0 || id >= a.c.pages) continue;  // no page: its tokens are dropped
    const int64_t at = id * a.c.heads + head;
    const uint32_t was_k = kept ? a.c.k_scales[at] : 0u, was_v = kept ? a.c.v_scales[at] : 0u;
    if (tid == 0) {
      most_k = was_k;
      most_v = was_v;
    }
    __syncthreads();
    for (int s = tid; s < n; s += 256) {  // (n is at most a page: one token a thread)
      const int src = held + path[lo - held + s];
      const int from = table[src >> a.shift];
      const bool none = from < 0 || from >= a.c.pages;  // its tokens become zeros
      from_page[s] = none ? -1 : from;
      from_slot[s] = src & (P - 1);
      const int64_t b = (int64_t)from * a.c.heads + head;
      kb[s] = none ? 0 : a.c.k_scales[b];
      vb[s] = none ? 0 : a.c.v_scales[b];
      atomicMax(&most_k, (uint32_t)kb[s]);
      atomicMax(&most_v, (uint32_t)vb[s]);
    }
    __syncthreads();
    const uint32_t sk = most_k, sv = most_v;
    uint8_t *kc = a.c.k_codes + at * P * D, *vc = a.c.v_codes + at * P * D;
    for (int s0 = 0; s0 < n; s0 += kMoved) {
      const int m = min(n - s0, kMoved);
      // what moves is read before anything is written
      for (int it = tid; it < m * D / 16; it += 256) {
        const int s = s0 + it / (D / 16), d = it % (D / 16) * 16;
        u32x4 w = {0, 0, 0, 0};
        if (from_page[s] >= 0)
          w = *reinterpret_cast<const u32x4 *>(a.c.k_codes + (((int64_t)from_page[s] * a.c.heads + head) * P + from_slot[s]) * D + d);
        *reinterpret_cast<u32x4 *>(ks + it * 16) = w;
      }
      for (int it = tid; it < m * D; it += 256) {
        const int s = s0 + it / D, d = it % D;
        vs[it] = from_page[s] < 0 ? 0
                                  : a.c.v_codes[(((int64_t)from_page[s] * a.c.heads + head) * D + d) * P + from_slot[s]];
      }
      __syncthreads();
      if (s0 == 0) {  // the kept tokens, to the new bytes
        if (kept && sk > was_k)
          for (int c = tid; c < kept * D / 16; c += 256) {
            u32x4 *p = reinterpret_cast<u32x4 *>(kc + 16 * c);
            *p = move16(*p, 16, (int)(sk - was_k), sk == 255u);
          }
        if (kept && sv > was_v) {
          const int pieces = (kept + 15) >> 4;
          for (int c = tid; c < D * pieces; c += 256) {
            u32x4 *p = reinterpret_cast<u32x4 *>(vc + c / pieces * P + c % pieces * 16);
            *p = move16(*p, kept - c % pieces * 16, (int)(sv - was_v), sv == 255u);
          }
        }
        __syncthreads();  // before the moved tokens' bytes of the same words
      }
      for (int it = tid; it < m * D / 16; it += 256) {
        const int s = it / (D / 16), d = it % (D / 16) * 16, by = (int)(sk - kb[s0 + s]);
        u32x4 w = *reinterpret_cast<const u32x4 *>(ks + it * 16);
        if (by) w = move16(w, 16, by, sk == 255u);
        *reinterpret_cast<u32x4 *>(kc + (kept + s0 + s) * D + d) = w;
      }
      for (int it = tid; it < m * D; it += 256) {
        const int s = it % m, d = it / m, by = (int)(sv - vb[s0 + s]);
        uint32_t w = vs[s * D + d];
        if (by) w = move4(w, by, sv == 255u);
        vc[d * P + kept + s0 + s] = (uint8_t)w;
      }
      __syncthreads();
    }
    if (tid == 0) {
      a.c.k_scales[at] = (uint8_t)sk;
      a.c.v_scales[at] = (uint8_t)sv;
    }
    __syncthreads();
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
  const uint32_t *tree;  // [token][words]: which new tokens of its sequence a token sees, or NULL: causal
  int words;
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
struct RawQuery {
  u32x4 w[D / 64][2];
};
template <int D>
__device__ __forceinline__ RawQuery<D> load_raw_query(const uint16_t *row, int lg) {
  RawQuery<D> q;
#pragma unroll
  for (int h = 0; h < D / 64; h++) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(row + 64 * h + 16 * lg);
    q.w[h][0] = p[0];
    q.w[h][1] = p[1];
  }
  return q;
}
template <int D>
__device__ __forceinline__ Query<D> split_query(const RawQuery<D> &raw) {
  const int lg = (threadIdx.x & 63) >> 4;
  float f[D / 64][16];
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < D / 64; h++) {
#pragma unroll
    for (int j = 0; j < 16; j++) {
      const uint32_t x = raw.w[h][j >> 3][(j >> 1) & 3];
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
template <int D>
__device__ __forceinline__ Query<D> load_query(const uint16_t *row, int lg) {
  return split_query<D>(load_raw_query<D>(row, lg));
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

// Masks RT x 16 rows of 128 scores where `masked` (tile t's accumulator i of row
// x is hidden(x, t, i)) and moves the running maxima; `less` is what a weight's
// exponent, s c - less, takes off. Branches are taken for all rows at once.
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
                                            F hidden, float (&less)[RT]) {
  if (masked) {
#pragma unroll
    for (int x = 0; x < RT; x++)
#pragma unroll
      for (int t = 0; t < 8; t++) {
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (hidden(x, t, i)) s[x][t][i] = -__builtin_inff();
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
  int seen0;        // keys the block's first token sees; the next one more (tree: keys that all see)
  int fresh;        // new tokens of the sequence
  const int32_t *table;
  int last_page;
};
template <bool TREE>
__device__ __forceinline__ bool find_block(const AttnArgs &a, int unit, Block &b) {
  // everything here is the same for the whole workgroup: kept in scalar registers
  auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const int i = uniform(find_sequence(a.b.cu, a.b.batch, [&](int x) { return x / a.block_tokens; }, 1, unit));
  const int c0 = uniform(a.b.cu[i]), n = uniform(a.b.cu[i + 1]) - c0;
  const int at = (unit - (c0 / a.block_tokens + i)) * a.block_tokens;
  if (at >= n || at < 0 || c0 < 0 || (int64_t)c0 + n > a.b.tokens) return false;
  const int64_t room = (int64_t)a.b.width << a.shift;
  b.len = (int)min((int64_t)max(uniform(a.b.lengths[i]), 0), room);
  b.tok0 = c0 + at;
  b.count = min(a.block_tokens, n - at);
  b.seen0 = TREE ? b.len - n : b.len - n + at + 1;
  b.fresh = n;
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
// 32 bits of a row of a tree's masks from bit `from` on, of which `n` count:
// keys before the new tokens (negative) are seen, bits past the row's are not.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t *row, int words, int n, int from) {
  const int w = from >> 5;
  auto word = [&](int i) { return i < 0 ? 0xFFFFFFFFu : i < words ? row[i] : 0u; };
  const uint32_t v = __builtin_amdgcn_alignbit(word(w + 1), word(w), (uint32_t)from & 31u);
  const int keep = n - from;
  return keep >= 32 ? v : keep <= 0 ? 0u : v & ((1u << keep) - 1u);
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
template <int D, int RT, bool TREE>
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
  if (unit >= a.units || !find_block<TREE>(a, unit, b)) return;
  const int head = blockIdx.y, split = a.splits > 1 ? blockIdx.z : 0;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int end = TREE ? b.len : min(b.len, b.seen0 + b.count - 1);  // keys any row sees
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
    seen[x] = TREE ? tok : b.seen0 + tok;
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
    const bool masked = tile * 128 + 128 > b.seen0;
    int limit[RT];  // tree: bit 4 t + i is what the row sees of accumulator i of tile t
    float less[RT], c = a.scale2;
#pragma unroll
    for (int x = 0; x < RT; x++) {
      if constexpr (!TREE) {
        limit[x] = seen[x] - 1 - tile * 128 - 16 * lg;
      } else if (masked) {
        const uint32_t *row = a.tree + (int64_t)(b.tok0 + seen[x]) * a.words;
        const int from = tile * 128 + 16 * lg - b.seen0;
        limit[x] = (int)((tree_bits(row, a.words, b.fresh, from) & 0xFFFFu) |
                         tree_bits(row, a.words, b.fresh, from + 64) << 16);
      }
    }
    running_max<D, RT, false>(s, r, c, masked, [&](int x, int t, int i) {
      return TREE ? !(limit[x] >> (4 * t + i) & 1) : 64 * (t >> 2) + 4 * (t & 3) + i > limit[x];
    }, less);
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

// How many splits of a token's block the first kernel wrote, as it had it; none
// of a token of no sequence, whose row of the output stays.
__device__ __forceinline__ int splits_of(const AttnArgs &a, int tok) {
  const int i = find_sequence(a.b.cu, a.b.batch, [](int x) { return x; }, 0, tok);
  const int c0 = a.b.cu[i], c1 = a.b.cu[i + 1], n = c1 - c0;
  if (c0 < 0 || tok < c0 || tok >= c1 || c1 > a.b.tokens) return 0;
  const int64_t room = (int64_t)a.b.width << a.shift;
  const int len = (int)min((int64_t)max(a.b.lengths[i], 0), room);
  const int at = (tok - c0) / a.block_tokens * a.block_tokens;
  const int end = a.tree ? len : min(len, len - n + at + min(a.block_tokens, n - at));
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
  if (!live || qh >= a.q_heads) return;
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
  if (!live) return;
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

// A wave's R parts of 16 rows, part x from row part_of(x) of the block on.
template <int D, bool TREE, int R, typename G, typename F>
__device__ __forceinline__ void attend_parts(const AttnArgs &a, const Block &b, int head, int t0, int t1,
                                             uint8_t (&ks)[256 * D], uint8_t (&vs)[256 * D], G part_of, F write) {
  constexpr int DT = D / 16, S = 128 * D;
  constexpr int KL = S / 4096, VL = KL;  // direct loads per thread and tile
  constexpr int N = R ? R : 1;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int rows = b.count * a.group;
  // pages are asked for first, then q, which is split while the first tile is on its way
  const int first_page = page_of(a, b, t0, lane);
  RawQuery<D> raw_q[N];
  Query<D> q[N];
  Rows<D> r[N];
  int seen[N];
#pragma unroll
  for (int x = 0; x < R; x++) {
    const int row = min(part_of(x) + l16, rows - 1);
    const int tok = row / a.group;
    seen[x] = TREE ? tok : b.seen0 + tok;
    raw_q[x] = load_raw_query<D>(a.q + (int64_t)(b.tok0 + tok) * a.q_stride +
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
    bytes = *byte_at(a, first_page, head, lane);
    mine = page_of(a, b, t0 + 1, lane);
    load(t0, 0, runs_of(a, first_page));
  }
#pragma unroll
  for (int x = 0; x < R; x++) q[x] = split_query<D>(raw_q[x]);
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
      load(tile + 1, (tile + 1 - t0) & 1, id);
    }
    if constexpr (R == 0) {  // the second barrier of the others
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      continue;
    } else {
      auto keys = [&](int t) {
        const int at = (32 * (t >> 1) + 4 * (t & 1)) * D;
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(kp0 + at);
        if constexpr (D == 64) return join8(lo, lo);
        else return join8(lo, *reinterpret_cast<const u32x4 *>(kp1 + at));
      };
      // operands are read two tiles ahead
      f32x4 s[R][8];
      i32x8 f[3] = {keys(0), keys(1)};
      auto score = [&](auto run) {  // the two tiles of a run of 32 tokens
        constexpr int J = decltype(run)::value;
#pragma unroll
        for (int t = 2 * J; t < 2 * J + 2; t++) {
          if (t + 2 < 8) f[(t + 2) % 3] = keys(t + 2);
#pragma unroll
          for (int x = 0; x < R; x++) s[x][t] = mma<J, 0>(f[t % 3], q[x].v[0], f32x4{0, 0, 0, 0}, sc, q[x].bytes);
          if constexpr (D == 128) {
#pragma unroll
            for (int x = 0; x < R; x++) s[x][t] = mma<J, 1>(f[t % 3], q[x].v[1], s[x][t], sc, q[x].bytes);
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
      for (int x = 0; x < R; x++)
#pragma unroll
        for (int t = 0; t < 8; t++) asm volatile("" : "+v"(s[x][t]));
      const bool masked = tile * 128 + 128 > b.seen0;
      int limit[R];  // tree: bit 4 t + i is what the row sees of accumulator i of tile t
      float less[R], c = a.scale2;
#pragma unroll
      for (int x = 0; x < R; x++) {
        if constexpr (!TREE) {
          limit[x] = seen[x] - 1 - tile * 128 - 8 * lg;
        } else if (masked) {
          const uint32_t *row = a.tree + (int64_t)(b.tok0 + seen[x]) * a.words;
          uint32_t bits = 0;
#pragma unroll
          for (int j = 0; j < 4; j++)
            bits |= (tree_bits(row, a.words, b.fresh, tile * 128 + 32 * j + 8 * lg - b.seen0) & 0xFFu) << (8 * j);
          limit[x] = (int)bits;
        }
      }
      running_max<D, R, true>(s, r, c, masked, [&](int x, int t, int i) {
        return TREE ? !(limit[x] >> (4 * t + i) & 1) : 32 * (t >> 1) + 4 * (t & 1) + i > limit[x];
      }, less);
      u32x4 p[R][4];  // of tokens 32 j + 8 lg ..
      weights<R, true>(s, c, less, p);
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
          for (int x = 0; x < R; x++) r[x].o[d] = mma16(g[d & 1][j], p[x][j], r[x].o[d]);
      }
#pragma unroll
      for (int x = 0; x < R; x++) r[x].l = add_weights(p[x], r[x].l);
      kp0 += flip;  // to the other buffer
      kp1 += flip;
      flip = -flip;
    }
  }
#pragma unroll
  for (int x = 0; x < R; x++) {
    const int row = part_of(x) + l16;
    if (row < rows) write(row, r[x]);
  }
}

// One block of rows and its tiles t0 .. t1 - 1, 16 RT rows a wave; `write(row, state)`
// takes what comes of each row. A prompt's block is full but for its last. A tree's
// rows are often fewer: they are dealt out a part of 16 at a time, and a wave does
// those that it has (the way through the tiles is its own, the barriers are as many).
template <int D, bool TREE, int RT, typename F>
__device__ __forceinline__ void attend_tiles(const AttnArgs &a, const Block &b, int head, int t0, int t1,
                                             uint8_t (&ks)[256 * D], uint8_t (&vs)[256 * D], F write) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (!TREE) {
    attend_parts<D, TREE, RT>(a, b, head, t0, t1, ks, vs, [&](int x) { return 16 * (RT * wave + x); }, write);
  } else {
    auto part_of = [&](int x) { return 16 * (4 * x + wave); };
    const int rows = __builtin_amdgcn_readfirstlane(b.count * a.group);
    if (part_of(RT - 1) < rows) attend_parts<D, TREE, RT>(a, b, head, t0, t1, ks, vs, part_of, write);
    else if (RT == 2 && part_of(0) < rows) attend_parts<D, TREE, 1>(a, b, head, t0, t1, ks, vs, part_of, write);
    else attend_parts<D, TREE, 0>(a, b, head, t0, t1, ks, vs, part_of, write);
  }
}

// Where a row's result goes: to the output, or what is left to be joined.
template <int D>
__device__ __forceinline__ void write_row(const AttnArgs &a, const Block &b, int head, int row, const Rows<D> &r) {
  const int lg = (threadIdx.x & 63) >> 4;
  const float l = r.l[0], inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t tok = b.tok0 + row / a.group, qh = (int64_t)head * a.group + row % a.group;
  uint16_t *p = a.out + (tok * a.q_heads + qh) * D + 4 * lg;
#pragma unroll
  for (int d = 0; d < D / 16; d++) {
    const f32x4 o = r.o[d];
    *reinterpret_cast<u32x2 *>(p + 16 * d) = u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
  }
}
template <int D>
__device__ __forceinline__ void write_part(float *p, const Rows<D> &r) {
  const int lg = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int d = 0; d < D / 16; d++) *reinterpret_cast<f32x4 *>(p + 16 * d + 4 * lg) = r.o[d];
  if (lg == 0) {
    p[D] = r.m;
    p[D + 1] = r.l[0];
  }
}

template <int D, bool TREE>
__global__ __launch_bounds__(256, 2) void k_attn_tiles(const AttnArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t ks[256 * D], vs[256 * D];
  // kv heads fastest: the eight XCDs, which are dealt workgroups in turn,
  // keep to few heads each. The last blocks of a sequence see the most keys:
  // they start first.
  const uint32_t block = blockIdx.z * gridDim.x + blockIdx.x;
  const int head = block % a.c.heads, from_last = block / a.c.heads;
  Block b;
  if (from_last >= a.units || !find_block<TREE>(a, a.units - 1 - from_last, b)) return;
  const int end = TREE ? b.len : min(b.len, b.seen0 + b.count - 1);
  const int tiles = (max(end, 0) + 127) >> 7;
  // this split's tiles; the last split takes whatever the caller's bound on the
  // lengths left out
  const int split = blockIdx.y, t0 = split * a.chunk;
  const int t1 = split + 1 == a.splits ? tiles : min(tiles, t0 + a.chunk);
  if (split > 0 && t0 >= tiles) return;  // the sum takes only splits that exist
  attend_tiles<D, TREE, 2>(a, b, head, t0, t1, ks, vs, [&](int row, const Rows<D> &r) {
    if (a.splits > 1) {
      const int64_t tok = b.tok0 + row / a.group, qh = (int64_t)head * a.group + row % a.group;
      write_part<D>(a.part + ((tok * a.q_heads + qh) * a.splits + split) * (D + 4), r);
    } else {
      write_row<D>(a, b, head, row, r);
    }
  });
}

// Trees whose rows fill no card in blocks: every workgroup gets an even share of
// all the tiles there are. Blocks of rows lie end to end, each as long as it has
// tiles and some for its beginning, sequence after sequence; workgroup g of a head takes
// places g per .. (g + 1) per - 1, which may be the end of one block, some whole
// ones and the beginning of another. What a block got from several workgroups
// is left in their room (the first and the last block of each: two rooms) and
// joined. 16 sequences of up to 24 tokens in 8,000 to 32,000, 32 query heads on 8 of
// 128 dims: 150 to 154 us a call in a long run, traced 151 and 8 for the join (splits of
// one length for all sequences, which left units idle for 41 % of the time, 241 and 8).
// Bound by what a wave does in a row (scores, weights, sums): 3.9 TB/s, matrix cores
// 33 % and vector arithmetic 41 % of a unit's cycles.
constexpr int kLeastTiles = 4;    // of a workgroup's share
constexpr int kSharers = 64;      // sequences: one a lane
constexpr int kBegin = 2;         // what beginning a block counts for, in tiles (4 trees of up to
                                  // 63 in 8,000: 36 us with nothing, 33 with one, 32 with two)
struct Stretch {
  int c0, n, len;     // the lane's sequence: first token, tokens, length
  int blocks, tiles;  // its blocks of rows, places of each: kBegin, then its tiles
  int64_t end;        // of its places
  int64_t total, per; // places there are, places of a workgroup
  __device__ __forceinline__ explicit Stretch(const AttnArgs &a) {
    const int lane = threadIdx.x & 63;
    c0 = n = len = blocks = 0;
    if (lane < a.b.batch) {
      c0 = a.b.cu[lane];
      n = a.b.cu[lane + 1] - c0;
      const int64_t room = (int64_t)a.b.width << a.shift;
      len = (int)min((int64_t)max(a.b.lengths[lane], 0), room);
      if (n > 0 && c0 >= 0 && (int64_t)c0 + n <= a.b.tokens) blocks = (n + a.block_tokens - 1) / a.block_tokens;
    }
    tiles = ((len + 127) >> 7) + kBegin;
    end = (int64_t)blocks * tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up((long long)end, d);
      end += lane >= d ? o : 0;
    }
    total = __shfl((long long)end, 63);
    per = max((int64_t)kLeastTiles, (total + a.splits - 1) / a.splits);
  }
  // what lane i knows, for all lanes of the wave together: none may have left
  __device__ __forceinline__ static int of(int v, int i) { return __builtin_amdgcn_readlane(v, i); }
  __device__ __forceinline__ int64_t begin_of(int i) const {
    return __shfl((long long)(end - (int64_t)blocks * tiles), i);
  }
};

// RT: 16-row parts of a wave, a block being 64 RT rows.
template <int D, int RT>
__global__ __launch_bounds__(256, 2) void k_attn_share(const AttnArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t ks[256 * D], vs[256 * D];
  __shared__ int of[5][kSharers];  // what a sequence's lane knows: not held in registers meanwhile
  auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const int head = blockIdx.x % a.c.heads, g = blockIdx.x / a.c.heads;
  int64_t left;
  int i, block, t0;
  {
    const Stretch s(a);
    if (threadIdx.x < kSharers) {
      of[0][threadIdx.x] = s.c0;
      of[1][threadIdx.x] = s.n;
      of[2][threadIdx.x] = s.len;
      of[3][threadIdx.x] = s.blocks;
      of[4][threadIdx.x] = s.tiles;
    }
    const int64_t first = g * s.per;
    left = min(s.total - first, s.per);
    i = __builtin_ctzll(__ballot(s.end > first) | 1ull << 63);
    const int64_t into = first - s.begin_of(i);
    block = (int)(into / Stretch::of(s.tiles, i));
    t0 = (int)(into % Stretch::of(s.tiles, i));
  }
  __syncthreads();
  i = uniform(i);
  block = uniform(block);
  t0 = uniform(t0);
  bool later = false;
  while (left > 0 && i < kSharers) {
    if (block >= uniform(of[3][i])) {  // on to the next sequence
      i++;
      block = 0;
      continue;
    }
    const int n = uniform(of[1][i]), tiles = uniform(of[4][i]);
    const int t1 = uniform((int)min((int64_t)tiles, t0 + left));
    Block b;
    b.len = uniform(of[2][i]);
    b.tok0 = uniform(of[0][i]) + block * a.block_tokens;
    b.count = min(a.block_tokens, n - block * a.block_tokens);
    b.seen0 = b.len - n;
    b.fresh = n;
    b.table = a.b.table + (int64_t)i * a.b.width;
    b.last_page = max(0, (b.len - 1) >> a.shift);
    const bool whole = t0 == 0 && t1 == tiles;
    float *room_of = a.part + ((int64_t)blockIdx.x * 2 + later) * 128 * (D + 4);
    attend_tiles<D, true, RT>(a, b, head, max(0, t0 - kBegin), max(0, t1 - kBegin), ks, vs, [&](int row, const Rows<D> &r) {
      if (whole) write_row<D>(a, b, head, row, r);
      else write_part<D>(room_of + row * (D + 4), r);
    });
    left -= t1 - t0;
    t0 = 0;
    block++;
    later = true;
    __syncthreads();  // every wave is done with the tiles in LDS
  }
}

// Joins what workgroups left of the rows of a token: D / 4 threads a row.
template <int D>
__global__ __launch_bounds__(256) void k_attn_share_join(const AttnArgs a) {
  constexpr int C = D / 4, R = 256 / C, P = D + 4;
  const int tok = blockIdx.x, c = threadIdx.x % C, qh = blockIdx.y * R + threadIdx.x / C;
  const Stretch s(a);
  const uint64_t owner = __ballot(s.blocks > 0 && tok >= s.c0 && tok < s.c0 + s.n);
  if (!owner) return;
  const int i = __builtin_ctzll(owner);
  const int c0 = Stretch::of(s.c0, i), tiles = Stretch::of(s.tiles, i), block = (tok - c0) / a.block_tokens;
  const int64_t begin = s.begin_of(i) + (int64_t)block * tiles;
  const int g0 = (int)(begin / s.per), g1 = (int)((begin + tiles - 1) / s.per);
  if (g0 == g1) return;  // one workgroup had it all
  // (not before: lane i is asked for its sequence above, and may have no query head)
  if (qh >= a.q_heads) return;
  const int head = qh / a.group;
  const int row = (tok - c0 - block * a.block_tokens) * a.group + qh % a.group;
  auto part = [&](int g) {  // of a workgroup that began before this block the later room
    return a.part + ((((int64_t)g * a.c.heads + head) * 2 + (g * s.per < begin)) * 128 + row) * P;
  };
  // four workgroups' at a time, whose loads go together
  float m = -__builtin_inff(), l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  for (int g = g0; g <= g1; g += 4) {
    float pm[4], pl[4];
    f32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const float *p = part(min(g + u, g1));
      pm[u] = g + u <= g1 ? p[D] : -__builtin_inff();
      pl[u] = p[D + 1];
      v[u] = *reinterpret_cast<const f32x4 *>(p + 4 * c);
    }
    const float top = __builtin_fmaxf(__builtin_fmaxf(m, __builtin_fmaxf(pm[0], pm[1])), __builtin_fmaxf(pm[2], pm[3]));
    const float ms = top == -__builtin_inff() ? 0.0f : top, old = __builtin_amdgcn_exp2f(m - ms);
    l *= old;
    o *= old;
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const float f = __builtin_amdgcn_exp2f(pm[u] - ms);
      if (g + u > g1) break;
      l = __builtin_fmaf(f, pl[u], l);
#pragma unroll
      for (int e = 0; e < 4; e++) o[e] = __builtin_fmaf(f, v[u][e], o[e]);
    }
    m = top;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<u32x2 *>(a.out + ((int64_t)tok * a.q_heads + qh) * D + 4 * c) =
      u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
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

// Workgroups of a head that share a tree's tiles, and 16-row parts of their waves;
// none where the kernels of causal attention take it: up to 16 rows, more sequences
// than a wave has lanes, blocks enough to fill the card over and over, and heads for
// which one workgroup each would be more than two a compute unit. Figures: us a call
// of sequences of up to so many new tokens, 32 query heads on 8. 17 to 32 rows of 128
// dims share where sequences may be longer than 1,024 (16 x 12 in 32,000: 121, with
// a wave to 32 rows 204; 48 x 8 in 3,000 51 and 78; 16 x 8 in 700 18 and 15), of 64 dims
// they do not (48 x 8 in 6,000: 56 and 55). Blocks of 64 rows up to 48 in the mean,
// since a sequence of more than 64 is then two blocks, which both read its keys (16 x
// 16 in 32,000, 48 rows in the mean: 121, in blocks of 128 rows 124; 16 x 24, 64 rows:
// 164 and 152). Two workgroups a compute unit, of four tiles at least (16 x 48 in 2,000:
// 36, of eight 40). 64 sequences that share beside the same that do not, as 65
// would: 64 x 12 in 8,000 141 and 165, 64 x 24 178 and 257, in 700 43 and 40.
struct TreePlan {
  int share, rt, block_tokens;
};
static TreePlan tree_plan(const AttnPlan &p, int64_t tokens, int batch, int q_heads, int heads, int dim,
                          int64_t max_length) {
  if (p.few && (p.rt == 1 || dim == 64 || max_length <= 1024)) return TreePlan{};
  if (batch > kSharers || heads > 512 || p.units * heads > 4096) return TreePlan{};
  const int group = q_heads / heads;
  const int rt = (tokens + batch - 1) / batch * group <= 48 && group <= 64 ? 1 : 2;
  const int block_tokens = 64 * rt / group;
  const int64_t tiles = (tokens / block_tokens + batch) * std::max<int64_t>(1, (max_length + 127) / 128);
  const int64_t share = std::min<int64_t>(512 / heads, (tiles + kLeastTiles - 1) / kLeastTiles);
  return TreePlan{(int)std::max<int64_t>(1, share), rt, block_tokens};
}
template <int D>
static void launch_share(const AttnArgs &a, int rt, hipStream_t st) {
  if (rt == 1) k_attn_share<D, 1><<<a.splits * a.c.heads, 256, 0, st>>>(a);
  else k_attn_share<D, 2><<<a.splits * a.c.heads, 256, 0, st>>>(a);
  const int rows = 1024 / D;  // of a workgroup that joins
  k_attn_share_join<D><<<dim3((uint32_t)a.b.tokens, (uint32_t)((a.q_heads + rows - 1) / rows)), 256, 0, st>>>(a);
}

}  // namespace mxl

using namespace mxl;

// A few new tokens per sequence: one wave a page, so that all pages are at
// work at once (256 sequences of one token: 8.5 us; four
// waves, and kept codes moved a word at a time: 19)
static bool few_tokens(const AppendArgs &a) { return a.b.tokens <= 4 * (int64_t)a.b.batch; }
static AppendArgs append_args(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                              const mx_kv_cache_t &cache, const mx_kv_batch_t &batch) {
  const int64_t blocks = (batch.tokens / cache.page + 2 * (int64_t)batch.batch) * cache.heads;
  return AppendArgs{k, v, k_stride, v_stride, cache, batch, log2_of(cache.page), (uint32_t)blocks, nullptr, 0.0f, {}};
}

hipError_t mxi_launch_kv_append(const void *k, const void *v, int bf16, int64_t k_stride,
                                int64_t v_stride, const mx_kv_cache_t &cache,
                                const mx_kv_batch_t &batch, hipStream_t st) {
  const AppendArgs a = append_args(k, v, k_stride, v_stride, cache, batch);
  const Spread xy = spread(a.blocks);
  const dim3 grid(xy.first, xy.second);
  const size_t lds = (size_t)cache.dim * (cache.page + 4);
  const bool few = few_tokens(a);
  if (bf16) few ? k_kv_append<true, 64><<<grid, 64, lds, st>>>(a) : k_kv_append<true, 256><<<grid, 256, lds, st>>>(a);
  else few ? k_kv_append<false, 64><<<grid, 64, lds, st>>>(a) : k_kv_append<false, 256><<<grid, 256, lds, st>>>(a);
  return hipGetLastError();
}

template <bool BF16, bool PAIRED>
static hipError_t launch_append_rotary(AppendArgs a, hipStream_t st) {
  if (!few_tokens(a)) a.blocks = (a.blocks / a.c.heads + 7) / 8 * 8 * a.c.heads;  // whole rounds of the XCDs
  const Spread xy = spread(a.blocks);
  const dim3 grid(xy.first, xy.second);
  const size_t lds = (size_t)a.c.dim * (a.c.page + 4);
  const bool few = few_tokens(a);
  if (a.c.dim == 64) few ? k_kv_append_rotary<BF16, 64, 64, PAIRED><<<grid, 64, lds, st>>>(a) : k_kv_append_rotary<BF16, 256, 64, PAIRED><<<grid, 256, lds, st>>>(a);
  else few ? k_kv_append_rotary<BF16, 64, 128, PAIRED><<<grid, 64, lds, st>>>(a) : k_kv_append_rotary<BF16, 256, 128, PAIRED><<<grid, 256, lds, st>>>(a);
  return hipGetLastError();
}
hipError_t mxi_launch_kv_append_rotary(const void *k, const void *v, int bf16, int64_t k_stride,
                                       int64_t v_stride, const void *weight, float eps,
                                       const mx_rotary_t &rotary, const mx_kv_cache_t &cache,
                                       const mx_kv_batch_t &batch, hipStream_t st) {
  AppendArgs a = append_args(k, v, k_stride, v_stride, cache, batch);
  a.weight = weight;
  a.eps = eps;
  a.r = rotary;
  if (bf16) return rotary.paired ? launch_append_rotary<true, true>(a, st) : launch_append_rotary<true, false>(a, st);
  return rotary.paired ? launch_append_rotary<false, true>(a, st) : launch_append_rotary<false, false>(a, st);
}

hipError_t mxi_launch_kv_keep(const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                              const int32_t *path, int path_width, const int32_t *count,
                              hipStream_t st) {
  const KeepArgs a = {cache, batch.table, batch.lengths, path, count, batch.batch, batch.width,
                      path_width, log2_of(cache.page)};
  const Spread xy = spread((int64_t)batch.batch * cache.heads);
  k_kv_keep<<<dim3(xy.first, xy.second), 256, 0, st>>>(a);
  return hipGetLastError();
}

size_t mxi_kv_attention_tree_workspace(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                       int64_t max_length) {
  const AttnPlan p = attn_plan(tokens, batch, q_heads, heads, max_length);
  if (const int64_t share = tree_plan(p, tokens, batch, q_heads, heads, dim, max_length).share)
    return (size_t)(share * heads * 2 * 128) * (dim + 4) * sizeof(float);
  return mxi_kv_attention_workspace(tokens, batch, q_heads, heads, dim, max_length);
}

size_t mxi_kv_attention_workspace(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                  int64_t max_length) {
  const AttnPlan p = attn_plan(tokens, batch, q_heads, heads, max_length);
  return p.most_splits > 1 ? (size_t)tokens * q_heads * p.most_splits * (dim + 4) * sizeof(float) : 0;
}

template <bool TREE>
static hipError_t launch_attention(const void *q, int64_t q_stride, int q_heads,
                                   const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                                   const uint32_t *tree, int words, int64_t max_length, float scale,
                                   void *out, void *workspace, hipStream_t st) {
  const AttnPlan p = attn_plan(batch.tokens, batch.batch, q_heads, cache.heads, max_length);
  const AttnArgs a = {reinterpret_cast<const uint16_t *>(q), q_stride, q_heads,
                      q_heads / cache.heads, cache, batch, log2_of(cache.page), p.block_tokens,
                      p.chunk, p.splits, (int)p.units, scale * 1.44269504088896340736f,
                      reinterpret_cast<uint16_t *>(out), reinterpret_cast<float *>(workspace),
                      tree, words};
  if constexpr (TREE) {
    const TreePlan plan = tree_plan(p, batch.tokens, batch.batch, q_heads, cache.heads, cache.dim, max_length);
    if (plan.share) {
      AttnArgs t = a;
      t.splits = plan.share;
      t.block_tokens = plan.block_tokens;
      if (cache.dim == 64) launch_share<64>(t, plan.rt, st);
      else launch_share<128>(t, plan.rt, st);
      return hipGetLastError();
    }
  }
  // (few rows are split for at most 1,024 sequences)
  const Spread xz = spread(p.few ? p.units : p.units * cache.heads);
  const dim3 grid(xz.first, (uint32_t)cache.heads, p.splits > 1 ? (uint32_t)p.splits : xz.second);
  if (!p.few) {
    const dim3 tgrid(xz.first, (uint32_t)p.splits, xz.second);
    if (cache.dim == 64) k_attn_tiles<64, TREE><<<tgrid, 256, 0, st>>>(a);
    else k_attn_tiles<128, TREE><<<tgrid, 256, 0, st>>>(a);
  } else if (cache.dim == 64) {
    if (p.rt == 1) k_attn_rows<64, 1, TREE><<<grid, 256, 0, st>>>(a);
    else k_attn_rows<64, 2, TREE><<<grid, 256, 0, st>>>(a);
  } else {
    if (p.rt == 1) k_attn_rows<128, 1, TREE><<<grid, 256, 0, st>>>(a);
    else k_attn_rows<128, 2, TREE><<<grid, 256, 0, st>>>(a);
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

hipError_t mxi_launch_kv_attention(const void *q, int64_t q_stride, int q_heads,
                                   const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                                   int64_t max_length, float scale, void *out, void *workspace,
                                   hipStream_t st) {
  return launch_attention<false>(q, q_stride, q_heads, cache, batch, nullptr, 0, max_length, scale, out, workspace, st);
}

hipError_t mxi_launch_kv_attention_tree(const void *q, int64_t q_stride, int q_heads,
                                        const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                                        const uint32_t *mask, int words, int64_t max_length,
                                        float scale, void *out, void *workspace, hipStream_t st) {
  return launch_attention<true>(q, q_stride, q_heads, cache, batch, mask, words, max_length, scale, out, workspace, st);
}
