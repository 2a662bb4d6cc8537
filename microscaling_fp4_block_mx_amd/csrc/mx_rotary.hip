// mx_rotary.hip - norms of queries and keys per head with the position rotation,
// and their gradients.
//
// n = w x / sqrt(sum x^2 / dim + eps) over a head's dims, then pairs of dims
// turn: y_a = n_a c - n_b s, y_b = n_b c + n_a s. Gradient: the rotation's
// transpose takes dy back to the norm's output (n = R^T dy), then with
// r = 1 / sqrt(..), g = w n: dx = r (g - x r^2 mean(g x)), dw = sum n x r.
//
// dim / 16 lanes hold a head, 16 elements each: two items of eight, chosen so
// that both members of every pair lie in one lane. A workgroup takes heads of q or
// of k, so that the weight stays in registers; a wave takes a run of neighbouring
// (token, head) pairs, 64 / (dim / 16) at a time, and loads cosines and sines where
// the token changes. Bound by HBM: each element is read and written once.
#include <algorithm>

#include "mx_layer.h"
#include "mx_rotary_device.h"

namespace mxl {

// What a wave does: which of the two tensors, and its run of pairs.
struct Runs {
  int heads[2], blocks[2];  // workgroups that take q, then those that take k
  int steps;                // of a wave: 64 / (dim / 16) pairs each
  int64_t tokens;
};
struct RotateArgs {
  const void *x[2], *weight[2];  // of q and k
  void *y[2];
  int64_t xs[2], ys[2];  // elements between tokens
  Runs runs;
  float eps;
  mx_rotary_t r;
};

// A lane's place in its wave's run.
template <int S>
struct Place {
  int64_t token, tokens;
  int head, heads, left;
  __device__ __forceinline__ Place(const Runs &r, int k, int slot) {
    const int64_t wave = (int64_t)(blockIdx.x - (k ? r.blocks[0] : 0)) * 4 + (threadIdx.x >> 6);
    const int64_t pair = wave * r.steps * S + slot;
    heads = r.heads[k];
    tokens = r.tokens;
    left = r.steps;
    token = pair / heads;
    head = (int)(pair % heads);
  }
  __device__ __forceinline__ bool is() const { return left > 0 && token < tokens; }
  __device__ __forceinline__ void next() {
    left--;
    token += S / heads;
    head += S % heads;
    if (head >= heads) {
      head -= heads;
      token++;
    }
  }
};

template <bool BF16>
__device__ __forceinline__ void store64(void *base, int64_t item, const double (&d)[8]) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; j++) f[j] = (float)d[j];
  store8<BF16>(base, item, f);
}
template <bool BF16>
__device__ __forceinline__ const uint8_t *element(const void *base, int64_t i) {
  return reinterpret_cast<const uint8_t *>(base) + i * (BF16 ? 2 : 4);
}
// Bound by HBM: 8191 tokens of 32 and 8 heads of 128, bf16, 168 MB in 37 us (4.6
// TB/s); 5 tokens, where a position, its angles and the head are trips to memory in a
// row, 3.5 us.
template <bool BF16, int D, bool PAIRED>
__global__ __launch_bounds__(256, BF16 ? 4 : 3) void k_norm_rotate(const RotateArgs p) {
  constexpr int L = D / 16, S = 64 / L;
  const int lane = threadIdx.x & 63, t = lane % L;
  const int k = (int)blockIdx.x >= p.runs.blocks[0];
  Place<S> at(p.runs, k, lane / L);
  int a, b;
  bool turns;
  items_of<PAIRED>(t, p.r.rot, a, b, turns);
  Raw<BF16> xa = {}, xb = {};
  int position = 0;
  auto fetch = [&] {
    if (!at.is()) return;
    const uint8_t *x = element<BF16>(p.x[k], at.token * p.xs[k] + (int64_t)at.head * D);
    xa = load_raw<BF16>(x, a);
    xb = load_raw<BF16>(x, b);
    if (turns) position = p.r.positions[at.token];
  };
  fetch();
  const bool norm = p.weight[k] != nullptr;
  Raw<BF16> wa = {}, wb = {};
  if (norm) {
    wa = load_weight<BF16>(p.weight[k], a);
    wb = load_weight<BF16>(p.weight[k], b);
  }
  Turns angles;
  int64_t turned = -1;  // the token whose angles these are
  while (at.is()) {     // (the lanes of a head go together)
    double da[8], db[8];
    widen64<BF16>(xa, da);
    widen64<BF16>(xb, db);
    if (turns && at.token != turned) {
      angles.load(p.r, position, t);
      turned = at.token;
    }
    uint8_t *y = const_cast<uint8_t *>(element<BF16>(p.y[k], at.token * p.ys[k] + (int64_t)at.head * D));
    at.next();
    fetch();
    if (norm) {
      double ss = 0.0;
#pragma unroll
      for (int j = 0; j < 8; j++) ss = __builtin_fma(da[j], da[j], __builtin_fma(db[j], db[j], ss));
      const double root = inverse_root(sum_lanes<L>(ss) * (1.0 / D) + p.eps);
      // widened each time: held in 64 bits they would cost a wave of four
      renew<BF16>(wa);
      renew<BF16>(wb);
      float va[8], vb[8];
      widen<BF16>(wa, va);
      widen<BF16>(wb, vb);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        da[j] = da[j] * root * va[j];
        db[j] = db[j] * root * vb[j];
      }
    }
    if (turns) turn<PAIRED, false>(da, db, angles.c, angles.s);
    store64<BF16>(y, a, da);
    store64<BF16>(y, b, db);
  }
}

struct RotateGradArgs {
  const void *dy[2], *x[2], *weight[2];
  void *dx[2];
  float *dweight[2];
  int64_t dys[2], xs[2], dxs[2];
  Runs runs;
  float eps;
  mx_rotary_t r;
  float *partial;  // [workgroup][dim]
};

// A lane's dims stay the same over its wave's run, so its share of dweight stays
// in registers; the next pairs are on their way while these are worked on. Bound by
// HBM: 8192 tokens of 32 and 8 heads of 128, bf16, 252 MB in 55 us (4.6 TB/s; a large
// copy reaches 5.2) and 4.5 for the sum of the partial rows. Three waves a SIMD (with
// dweight in 32 bits) took the same; one pair at a time without the next, a token
// a wave, 100.
template <bool BF16, int D, bool PAIRED>
__global__ __launch_bounds__(256) void k_norm_rotate_backward(const RotateGradArgs p) {
  constexpr int L = D / 16, S = 64 / L;
  __shared__ double part[4][D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = lane % L, slot = lane / L;
  const int k = (int)blockIdx.x >= p.runs.blocks[0];
  Place<S> at(p.runs, k, slot);
  int a, b;
  bool turns;
  items_of<PAIRED>(t, p.r.rot, a, b, turns);
  const bool norm = p.weight[k] != nullptr;
  Raw<BF16> ya = {}, yb = {}, xa = {}, xb = {};
  int position = 0;
  auto fetch = [&] {
    if (!at.is()) return;
    const uint8_t *dy = element<BF16>(p.dy[k], at.token * p.dys[k] + (int64_t)at.head * D);
    ya = load_raw<BF16>(dy, a);
    yb = load_raw<BF16>(dy, b);
    if (norm) {
      const uint8_t *x = element<BF16>(p.x[k], at.token * p.xs[k] + (int64_t)at.head * D);
      xa = load_raw<BF16>(x, a);
      xb = load_raw<BF16>(x, b);
    }
    if (turns) position = p.r.positions[at.token];
  };
  fetch();
  float wa[8] = {}, wb[8] = {};
  if (norm) {
    widen<BF16>(load_weight<BF16>(p.weight[k], a), wa);
    widen<BF16>(load_weight<BF16>(p.weight[k], b), wb);
  }
  double dw[16];
#pragma unroll
  for (int j = 0; j < 16; j++) dw[j] = 0.0;
  Turns angles;
  int64_t turned = -1;
  while (at.is()) {
    double na[8], nb[8], da[8], db[8];
    widen64<BF16>(ya, na);
    widen64<BF16>(yb, nb);
    widen64<BF16>(xa, da);
    widen64<BF16>(xb, db);
    if (turns && at.token != turned) {
      angles.load(p.r, position, t);
      turned = at.token;
    }
    uint8_t *dx = const_cast<uint8_t *>(element<BF16>(p.dx[k], at.token * p.dxs[k] + (int64_t)at.head * D));
    at.next();
    fetch();
    if (turns) turn<PAIRED, true>(na, nb, angles.c, angles.s);
    if (norm) {
      double ss = 0.0, sg = 0.0;
#pragma unroll
      for (int j = 0; j < 8; j++) ss = __builtin_fma(da[j], da[j], __builtin_fma(db[j], db[j], ss));
      const double r = inverse_root(sum_lanes<L>(ss) * (1.0 / D) + p.eps);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        da[j] *= r;
        db[j] *= r;
        dw[j] = __builtin_fma(na[j], da[j], dw[j]);
        dw[8 + j] = __builtin_fma(nb[j], db[j], dw[8 + j]);
        na[j] *= wa[j];
        nb[j] *= wb[j];
        sg = __builtin_fma(na[j], da[j], __builtin_fma(nb[j], db[j], sg));
      }
      const double m = sum_lanes<L>(sg) * (1.0 / D);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        na[j] = r * __builtin_fma(-da[j], m, na[j]);
        nb[j] = r * __builtin_fma(-db[j], m, nb[j]);
      }
    }
    store64<BF16>(dx, a, na);
    store64<BF16>(dx, b, nb);
  }
  if (!norm) return;
  // the heads of a wave, then the four waves, in a fixed order
#pragma unroll
  for (int j = 0; j < 16; j++) {
    double v = dw[j];
#pragma unroll
    for (int d = L; d < 64; d <<= 1) v += __shfl_xor(v, d);
    if (slot == 0) part[wave][8 * (j < 8 ? a : b) + (j & 7)] = v;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 256)
    p.partial[(int64_t)blockIdx.x * D + d] = (float)((part[0][d] + part[1][d]) + (part[2][d] + part[3][d]));
}

// dweight = sum of the partial rows of q's workgroups, or of k's: a workgroup per
// 16 columns, 64 rows at a time.
__global__ __launch_bounds__(1024) void k_sum_weights(const float *__restrict__ partial, int rows_q, int rows_k,
                                                      int dim, float *dq, float *dk) {
  __shared__ float part[64][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  const int first = blockIdx.y ? rows_q : 0, n = blockIdx.y ? rows_k : rows_q;
  float *to = blockIdx.y ? dk : dq;
  if (!to) return;
  float v[4] = {0, 0, 0, 0};  // independent: their loads go together
  for (int i = r; i < n; i += 256)
#pragma unroll
    for (int q = 0; q < 4; q++)
      if (i + 64 * q < n) v[q] += partial[(int64_t)(first + i + 64 * q) * dim + col];
  part[r][c] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (r == 0) {
    float total = 0.0f;
#pragma unroll
    for (int q = 0; q < 64; q++) total += part[q][c];
    to[col] = total;
  }
}

// Splits tokens x heads of q and k over at most `most` workgroups of four waves
// (if both have heads at least two), each wave a run of `steps` rounds.
static Runs runs_of(int64_t tokens, int q_heads, int k_heads, int dim, int64_t most) {
  Runs r = {};
  r.heads[0] = q_heads;
  r.heads[1] = std::max(1, k_heads);
  r.tokens = tokens;
  const int at_once = 4 * 64 / (dim / 16);  // pairs of a workgroup's round
  auto blocks = [&](int heads, int64_t steps) {
    const int64_t each = at_once * steps;
    return (tokens * heads + each - 1) / each;
  };
  auto all = [&](int64_t steps) { return blocks(q_heads, steps) + (k_heads ? blocks(k_heads, steps) : 0); };
  int64_t steps = std::max<int64_t>(1, all(1) / most);
  while (all(steps) > most) steps += steps / 64 + 1;  // (rounding up may leave one too many)
  r.steps = (int)steps;
  r.blocks[0] = (int)blocks(q_heads, steps);
  r.blocks[1] = k_heads ? (int)blocks(k_heads, steps) : 0;
  return r;
}

template <bool BF16, int D>
static void launch_rotate(const RotateArgs &a, hipStream_t st) {
  const int blocks = a.runs.blocks[0] + a.runs.blocks[1];
  if (a.r.paired) k_norm_rotate<BF16, D, true><<<blocks, 256, 0, st>>>(a);
  else k_norm_rotate<BF16, D, false><<<blocks, 256, 0, st>>>(a);
}
template <bool BF16, int D>
static void launch_rotate_backward(const RotateGradArgs &a, hipStream_t st) {
  const int blocks = a.runs.blocks[0] + a.runs.blocks[1];
  if (a.r.paired) k_norm_rotate_backward<BF16, D, true><<<blocks, 256, 0, st>>>(a);
  else k_norm_rotate_backward<BF16, D, false><<<blocks, 256, 0, st>>>(a);
}

}  // namespace mxl

using namespace mxl;

// Most workgroups. Forward: four times what the card holds, so that the last ones
// leave little of it idle (1,024 37.9 us, 2,048 38.6, 4,096 36.7, 12,000, a round each, 46).
// The gradient's: what the card holds, since each adds a partial row (512 55 us, 1,024
// 61).
constexpr int64_t kForwardBlocks = 4096, kGradientBlocks = 512;

hipError_t mxi_launch_norm_rotate(const mx_heads_t &q, const mx_heads_t *k, int bf16,
                                  int64_t tokens, int dim, float eps, const mx_rotary_t &rotary,
                                  hipStream_t st) {
  RotateArgs a = {};
  const mx_heads_t both[2] = {q, k ? *k : mx_heads_t{}};
  for (int i = 0; i < 2; i++) {
    a.x[i] = both[i].x;
    a.weight[i] = both[i].weight;
    a.y[i] = both[i].y;
    a.xs[i] = both[i].x_stride;
    a.ys[i] = both[i].y_stride;
  }
  a.runs = runs_of(tokens, q.heads, both[1].heads, dim, kForwardBlocks);
  a.eps = eps;
  a.r = rotary;
  if (bf16) {
    if (dim == 64) launch_rotate<true, 64>(a, st);
    else if (dim == 128) launch_rotate<true, 128>(a, st);
    else launch_rotate<true, 256>(a, st);
  } else {
    if (dim == 64) launch_rotate<false, 64>(a, st);
    else if (dim == 128) launch_rotate<false, 128>(a, st);
    else launch_rotate<false, 256>(a, st);
  }
  return hipGetLastError();
}

// The most workgroups of the gradient's launch (one of q and one of k at least).
int64_t mxi_norm_rotate_partials(int64_t tokens) { return std::min(2 * tokens, kGradientBlocks); }

hipError_t mxi_launch_norm_rotate_backward(const mx_heads_grad_t &q, const mx_heads_grad_t *k,
                                           int bf16, int64_t tokens, int dim, float eps,
                                           const mx_rotary_t &rotary, float *partial,
                                           hipStream_t st) {
  RotateGradArgs a = {};
  const mx_heads_grad_t both[2] = {q, k ? *k : mx_heads_grad_t{}};
  for (int i = 0; i < 2; i++) {
    a.dy[i] = both[i].dy;
    a.x[i] = both[i].x;
    a.weight[i] = both[i].weight;
    a.dx[i] = both[i].dx;
    a.dweight[i] = both[i].weight ? both[i].dweight : nullptr;
    a.dys[i] = both[i].dy_stride;
    a.xs[i] = both[i].x_stride;
    a.dxs[i] = both[i].dx_stride;
  }
  a.eps = eps;
  a.r = rotary;
  a.partial = partial;
  if (tokens > 0) {
    a.runs = runs_of(tokens, q.heads, both[1].heads, dim, mxi_norm_rotate_partials(tokens));
    if (bf16) {
      if (dim == 64) launch_rotate_backward<true, 64>(a, st);
      else if (dim == 128) launch_rotate_backward<true, 128>(a, st);
      else launch_rotate_backward<true, 256>(a, st);
    } else {
      if (dim == 64) launch_rotate_backward<false, 64>(a, st);
      else if (dim == 128) launch_rotate_backward<false, 128>(a, st);
      else launch_rotate_backward<false, 256>(a, st);
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.dweight[0] || a.dweight[1])
    k_sum_weights<<<dim3((uint32_t)dim / 16, 2), 1024, 0, st>>>(partial, a.runs.blocks[0], a.runs.blocks[1], dim,
                                                                a.dweight[0], a.dweight[1]);
  return hipGetLastError();
}
