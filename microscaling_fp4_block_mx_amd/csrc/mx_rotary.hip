// mx_rotary.hip - norms of queries and keys per head with the position rotation,
// and their gradients.
//
// n = w x / sqrt(sum x^2 / dim + eps) over a head's dims, then pairs of dims
// turn: y_a = n_a c - n_b s, y_b = n_b c + n_a s. Gradient: the rotation's
// transpose takes dy back to the norm's output (n = R^T dy), then with
// r = 1 / sqrt(..), g = w n: dx = r (g - x r^2 mean(g x)), dw = sum n x r.
//
// dim / 16 lanes hold a head, 16 elements each: two items of eight, chosen so
// that both members of every pair lie in one lane. A wave takes a token, its
// heads in turn; cosines and sines are loaded once for all of them. Bound by
// HBM: each element is read and written once.
#include <algorithm>

#include "mx_layer.h"
#include "mx_rotary_device.h"

namespace mxl {

struct RotateArgs {
  const void *x[2], *weight[2];  // of q and k
  void *y[2];
  int64_t xs[2], ys[2];  // elements between tokens
  int q_heads, heads;    // q's, and both
  int chunks;            // waves that share a token
  int64_t work;          // tokens times chunks
  float eps;
  mx_rotary_t r;
};

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

// Turns a lane's pairs; `sign` -1: back.
template <bool PAIRED>
__device__ __forceinline__ void turn(double (&a)[8], double (&b)[8], const float (&c)[8], const float (&s)[8],
                                     double sign) {
  auto pair = [&](double &x, double &y, int e) {
    const double cd = c[e], sd = sign * s[e], x0 = x;
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
// Weights stay in the caches: default policy.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_weight(const void *w, int item) {
  const u32x4 *p = reinterpret_cast<const u32x4 *>(w) + (BF16 ? 1 : 2) * item;
  Raw<BF16> r;
  r.v[0] = p[0];
  if constexpr (!BF16) r.v[1] = p[1];
  return r;
}

constexpr int kAhead = 4;  // heads of a lane whose loads go together

template <bool BF16, int D, bool PAIRED>
__global__ __launch_bounds__(256) void k_norm_rotate(const RotateArgs p) {
  constexpr int L = D / 16, S = 64 / L;
  const int64_t id = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (id >= p.work) return;
  const int64_t token = id / p.chunks;
  const int lane = threadIdx.x & 63, t = lane % L, slot = lane / L;
  int a, b;
  bool turns;
  items_of<PAIRED>(t, p.r.rot, a, b, turns);
  float c[8], s[8];
  if (turns) {
    const Angles at = angles_of(p.r.table, p.r.length, p.r.rot, p.r.positions[token]);
    load8(at.row + 8 * t, c);
    load8(at.row + (p.r.rot >> 1) + 8 * t, s);
    if (at.none) {
#pragma unroll
      for (int j = 0; j < 8; j++) c[j] = __builtin_nanf("");
    }
  }
  for (int h0 = (int)(id % p.chunks) * S + slot; h0 - slot < p.heads; h0 += S * p.chunks * kAhead) {
    Raw<BF16> xa[kAhead], xb[kAhead];
    auto head_of = [&](int u) { return h0 + u * S * p.chunks; };
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      xa[u] = xb[u] = Raw<BF16>{};
      const int h = head_of(u), k = h >= p.q_heads;
      if (h < p.heads) {
        const uint8_t *x = element<BF16>(p.x[k], token * p.xs[k] + (int64_t)(k ? h - p.q_heads : h) * D);
        xa[u] = load_raw<BF16>(x, a);
        xb[u] = load_raw<BF16>(x, b);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      const int h = head_of(u), k = h >= p.q_heads;
      double da[8], db[8], ss = 0.0;
      widen64<BF16>(xa[u], da);
      widen64<BF16>(xb[u], db);
#pragma unroll
      for (int j = 0; j < 8; j++) ss = __builtin_fma(da[j], da[j], __builtin_fma(db[j], db[j], ss));
      ss = sum_lanes<L>(ss);  // (every lane takes part)
      if (h >= p.heads) continue;
      if (p.weight[k]) {
        const double root = inverse_root(ss * (1.0 / D) + p.eps);
        double wa[8], wb[8];
        widen64<BF16>(load_weight<BF16>(p.weight[k], a), wa);
        widen64<BF16>(load_weight<BF16>(p.weight[k], b), wb);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          da[j] = da[j] * root * wa[j];
          db[j] = db[j] * root * wb[j];
        }
      }
      if (turns) turn<PAIRED>(da, db, c, s, 1.0);
      uint8_t *y = const_cast<uint8_t *>(
          element<BF16>(p.y[k], token * p.ys[k] + (int64_t)(k ? h - p.q_heads : h) * D));
      store64<BF16>(y, a, da);
      store64<BF16>(y, b, db);
    }
  }
}

struct RotateGradArgs {
  const void *dy[2], *x[2], *weight[2];
  void *dx[2];
  float *dweight[2];
  int64_t dys[2], xs[2], dxs[2];
  int q_heads, heads;
  int64_t tokens;
  float eps;
  mx_rotary_t r;
  float *partial;  // [workgroup][q, k][dim]
};

template <bool BF16, int D, bool PAIRED>
__global__ __launch_bounds__(256) void k_norm_rotate_backward(const RotateGradArgs p) {
  constexpr int L = D / 16, S = 64 / L;
  __shared__ float part[4][2][D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = lane % L, slot = lane / L;
  int a, b;
  bool turns;
  items_of<PAIRED>(t, p.r.rot, a, b, turns);
  float dw[2][16];
#pragma unroll
  for (int j = 0; j < 16; j++) dw[0][j] = dw[1][j] = 0.0f;
  for (int64_t token = (int64_t)blockIdx.x * 4 + wave; token < p.tokens; token += (int64_t)gridDim.x * 4) {
    float c[8], s[8];
    if (turns) {
      const Angles at = angles_of(p.r.table, p.r.length, p.r.rot, p.r.positions[token]);
      load8(at.row + 8 * t, c);
      load8(at.row + (p.r.rot >> 1) + 8 * t, s);
      if (at.none) {
#pragma unroll
        for (int j = 0; j < 8; j++) c[j] = __builtin_nanf("");
      }
    }
    for (int h0 = 0; h0 < p.heads; h0 += S) {
      const int h = h0 + slot, k = h >= p.q_heads;
      const bool mine = h < p.heads;
      const int64_t head = (int64_t)(k ? h - p.q_heads : h) * D;
      Raw<BF16> ya = {}, yb = {}, xa = {}, xb = {};
      if (mine) {
        const uint8_t *dy = element<BF16>(p.dy[k], token * p.dys[k] + head);
        ya = load_raw<BF16>(dy, a);
        yb = load_raw<BF16>(dy, b);
        if (p.weight[k]) {
          const uint8_t *x = element<BF16>(p.x[k], token * p.xs[k] + head);
          xa = load_raw<BF16>(x, a);
          xb = load_raw<BF16>(x, b);
        }
      }
      double na[8], nb[8], da[8], db[8], wa[8], wb[8], ss = 0.0, sg = 0.0;
      widen64<BF16>(ya, na);
      widen64<BF16>(yb, nb);
      widen64<BF16>(xa, da);
      widen64<BF16>(xb, db);
      if (turns) turn<PAIRED>(na, nb, c, s, -1.0);
      const bool norm = mine && p.weight[k];
      Raw<BF16> ra = {}, rb = {};
      if (norm) {
        ra = load_weight<BF16>(p.weight[k], a);
        rb = load_weight<BF16>(p.weight[k], b);
      }
      widen64<BF16>(ra, wa);
      widen64<BF16>(rb, wb);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        ss = __builtin_fma(da[j], da[j], __builtin_fma(db[j], db[j], ss));
        sg = __builtin_fma(na[j] * wa[j], da[j], __builtin_fma(nb[j] * wb[j], db[j], sg));
      }
      ss = sum_lanes<L>(ss);
      sg = sum_lanes<L>(sg);
      if (!mine) continue;
      if (norm) {
        const double r = inverse_root(ss * (1.0 / D) + p.eps), m = sg * (1.0 / D) * r * r;
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float ga = (float)(na[j] * (da[j] * r)), gb = (float)(nb[j] * (db[j] * r));
          dw[0][j] += k ? 0.0f : ga;
          dw[0][8 + j] += k ? 0.0f : gb;
          dw[1][j] += k ? ga : 0.0f;
          dw[1][8 + j] += k ? gb : 0.0f;
          na[j] = r * __builtin_fma(-da[j], m, na[j] * wa[j]);
          nb[j] = r * __builtin_fma(-db[j], m, nb[j] * wb[j]);
        }
      }
      uint8_t *dx = const_cast<uint8_t *>(element<BF16>(p.dx[k], token * p.dxs[k] + head));
      store64<BF16>(dx, a, na);
      store64<BF16>(dx, b, nb);
    }
  }
  if (!p.partial) return;
  // the heads of a wave, then the four waves, in a fixed order
#pragma unroll
  for (int k = 0; k < 2; k++)
#pragma unroll
    for (int j = 0; j < 16; j++) {
      float v = dw[k][j];
#pragma unroll
      for (int d = L; d < 64; d <<= 1) v += __shfl_xor(v, d);
      if (slot == 0) part[wave][k][8 * (j < 8 ? a : b) + (j & 7)] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += 256) {
    const int k = i / D, d = i % D;
    p.partial[(int64_t)blockIdx.x * 2 * D + i] = (part[0][k][d] + part[1][k][d]) + (part[2][k][d] + part[3][k][d]);
  }
}

// dweight = sum of n partial rows: a workgroup per 16 of the 2 D columns.
__global__ __launch_bounds__(256) void k_sum_weights(const float *__restrict__ partial, int n, int dim,
                                                     float *dq, float *dk) {
  __shared__ float part[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float v = 0.0f;
  for (int i = r; i < n; i += 16) v += partial[(int64_t)i * 2 * dim + col];
  part[r][c] = v;
  __syncthreads();
  float *to = col < dim ? dq : dk;
  if (r == 0 && to) {
    float total = 0.0f;
#pragma unroll
    for (int q = 0; q < 16; q++) total += part[q][c];
    to[col < dim ? col : col - dim] = total;
  }
}

// Workgroups along one dimension of a grid, whose threads are fewer than 2^32,
// and along another for the rest.
static dim3 spread_grid(int64_t blocks) {
  const int64_t first = std::min<int64_t>(blocks, 1 << 22);
  return dim3((uint32_t)first, (uint32_t)((blocks + first - 1) / first));
}

template <bool BF16, int D>
static void launch_rotate(const RotateArgs &a, hipStream_t st) {
  const dim3 grid = spread_grid((a.work + 3) / 4);
  if (a.r.paired) k_norm_rotate<BF16, D, true><<<grid, 256, 0, st>>>(a);
  else k_norm_rotate<BF16, D, false><<<grid, 256, 0, st>>>(a);
}
template <bool BF16, int D>
static void launch_rotate_backward(const RotateGradArgs &a, int blocks, hipStream_t st) {
  if (a.r.paired) k_norm_rotate_backward<BF16, D, true><<<blocks, 256, 0, st>>>(a);
  else k_norm_rotate_backward<BF16, D, false><<<blocks, 256, 0, st>>>(a);
}

}  // namespace mxl

using namespace mxl;

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
  a.q_heads = q.heads;
  a.heads = q.heads + both[1].heads;
  a.chunks = 1;
  a.work = tokens * a.chunks;
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

int64_t mxi_norm_rotate_partials(int64_t tokens) { return std::min<int64_t>((tokens + 3) / 4, 1024); }

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
  a.q_heads = q.heads;
  a.heads = q.heads + both[1].heads;
  a.tokens = tokens;
  a.eps = eps;
  a.r = rotary;
  const bool sums = a.dweight[0] || a.dweight[1];
  a.partial = sums ? partial : nullptr;
  const int blocks = (int)mxi_norm_rotate_partials(tokens);
  if (tokens > 0) {
    if (bf16) {
      if (dim == 64) launch_rotate_backward<true, 64>(a, blocks, st);
      else if (dim == 128) launch_rotate_backward<true, 128>(a, blocks, st);
      else launch_rotate_backward<true, 256>(a, blocks, st);
    } else {
      if (dim == 64) launch_rotate_backward<false, 64>(a, blocks, st);
      else if (dim == 128) launch_rotate_backward<false, 128>(a, blocks, st);
      else launch_rotate_backward<false, 256>(a, blocks, st);
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (sums) k_sum_weights<<<2 * dim / 16, 256, 0, st>>>(partial, blocks, dim, a.dweight[0], a.dweight[1]);
  return hipGetLastError();
}
