// mx_verify.hip - verification of drafted tokens against the target model's
// probabilities, from given random numbers.
//
// At a node of a sequence's tree, with the target's row p and (where the draft's
// probabilities are given) the draft's row q: the first child's token x is taken
// if u0 q(x) < p(x). If it is not, w = max(p - q, 0), or p without a draft, and
// the first t with w_0 + .. + w_t > u1 sum(w) is drawn; a child with that token
// is followed, else t is the sequence's next token. The result is distributed as
// the target's own samples: a taken x and a t drawn from the residual together
// are p, and t does not depend on the other children's tokens.
//
// Sums of a row run over up to hundreds of thousands of numbers and decide at
// their borders: 64 bits. Two launches. The first finds each node's first child and
// whether it is taken, and with that which nodes the walk can reach and has to draw at
// (of a chain with a draft one; without a draft all that it can reach): only their rows
// are read, and summed in chunks. The second finds each one's chunk, reads it again and
// draws; then it walks down.
#include <algorithm>

#include "mx_layer.h"
#include "mx_layer_device.h"
#include "mx_rotary_device.h"

namespace mxl {

constexpr int kNodes = 1024;   // nodes of a sequence that are looked at
constexpr int kChunk = 2048;   // elements of a row that a wave sums at a time

struct VerifyArgs {
  const void *target, *draft;
  const int32_t *ids, *parents, *cu;
  const float *numbers;
  int64_t tokens, vocab;
  int batch, width, chunks;
  int32_t *path, *count, *token;
  // scratch: each node's first child (or -1), with kTaken where it is taken; each
  // sequence's nodes to draw at, in order, with kResidual where from p - q, and how
  // many; their chunks' sums of w and of p
  int32_t *kid, *draws, *many;
  double *sums;
};
constexpr int32_t kTaken = 1 << 30, kResidual = 1 << 30;

// A probability: what is negative, infinite or no number counts as 0.
__device__ __forceinline__ float clean(float p) { return __float_as_uint(p) - 1u < 0x7F7FFFFFu ? p : 0.0f; }

struct Sequence {
  int64_t first;
  int nodes;
};
__device__ __forceinline__ Sequence sequence_of(const VerifyArgs &a, int i) {
  const int64_t c0 = a.cu[i], n = a.cu[i + 1] - c0;
  if (c0 < 0 || n <= 0 || c0 + n > a.tokens) return Sequence{0, 0};
  return Sequence{c0, (int)(n < kNodes ? n : kNodes)};
}

// What a sequence's walk can meet, found by the whole workgroup.
struct Plan {
  int up[kNodes], kid[kNodes], id[kNodes], depth[kNodes], draws[kNodes];
  int many;
};
template <bool BF16>
__device__ __forceinline__ void make_plan(const VerifyArgs &a, const Sequence &s, Plan &p) {
  const int lane = threadIdx.x & 63;
  for (int j = threadIdx.x; j < s.nodes; j += blockDim.x) {
    p.up[j] = a.parents[s.first + j];
    p.id[j] = a.ids[s.first + j];
    p.kid[j] = kNodes;
  }
  __syncthreads();
  // nodes that the root reaches in fewer than `width` steps have a depth
  for (int j = threadIdx.x; j < s.nodes; j += blockDim.x) {
    int x = j, d = 0;
    while (x > 0 && d < a.width) {
      const int up = p.up[x];
      x = up >= 0 && up < x ? up : -1;
      d++;
    }
    p.depth[j] = x == 0 && d < a.width ? d : -1;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < s.nodes; j += blockDim.x)
    if (p.depth[j] > 0) atomicMin(&p.kid[p.up[j]], j);
  __syncthreads();
  for (int j = threadIdx.x; j < s.nodes; j += blockDim.x) {
    const int k = p.kid[j];
    int to = k == kNodes ? -1 : k;
    if (a.draft && to >= 0) {
      const int64_t row = s.first + j, x = p.id[k];
      if (x >= 0 && x < a.vocab) {
        const double t = clean(load_one<BF16>(a.target, row * a.vocab + x));
        const double q = clean(load_one<BF16>(a.draft, row * a.vocab + x));
        if ((double)a.numbers[2 * row] * q < t) to |= kTaken;
      }
    }
    p.kid[j] = to;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    int found = 0;
    for (int j0 = 0; j0 < s.nodes; j0 += 64) {
      const int j = j0 + lane;
      // drawn at: reached, unless its first child is taken. With a draft a first
      // child is reached where it is taken, another where the first one is not.
      bool draws = j < s.nodes && p.depth[j] >= 0 && (p.kid[j] < 0 || !(p.kid[j] & kTaken));
      for (int x = j; draws && x > 0; x = p.up[x]) {
        const int k = p.kid[p.up[x]];
        if (a.draft) draws = k == (x | kTaken) || (k != x && !(k & kTaken));
      }
      const uint64_t all = __ballot(draws);
      if (draws) p.draws[found + __popcll(all & ((1ull << lane) - 1))] = j | (a.draft && p.kid[j] >= 0 ? kResidual : 0);
      found += __popcll(all);
    }
    if (lane == 0) p.many = found;
  }
  __syncthreads();
}

// A wave's part of a row: step u of lane l holds 16 bytes of neighbouring elements,
// zeros outside the row. Rows begin anywhere: chunks are laid out from the 16-byte
// boundary before a row on. A step is a run of the row, or, LANES, a lane has one.
template <bool BF16>
struct Part {
  static constexpr int A = BF16 ? 8 : 4, U = kChunk / 64 / A;
  u32x4 v[U];
};
template <bool BF16, bool LANES>
__device__ __forceinline__ Part<BF16> load_part(const void *base, const VerifyArgs &a, int64_t row, int chunk) {
  constexpr int A = Part<BF16>::A, U = Part<BF16>::U, E = BF16 ? 2 : 4;
  constexpr int STEP = LANES ? A : 64 * A;  // elements from step to step
  const int64_t begin = row * a.vocab, end = begin + a.vocab;
  const int64_t from = (begin & ~(int64_t)(A - 1)) + (int64_t)chunk * kChunk + (threadIdx.x & 63) * (LANES ? A * U : A);
  const uint8_t *x = reinterpret_cast<const uint8_t *>(base) + from * E;
  Part<BF16> p;
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t at = from + u * STEP;
    p.v[u] = u32x4{0, 0, 0, 0};
    if (at >= begin && at + A <= end) p.v[u] = *reinterpret_cast<const u32x4 *>(x + u * STEP * E);
  }
  // the row's first and last elements, where they share their 16 bytes with others'
  if ((begin | end) & (A - 1)) {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t at = from + u * STEP;
      if (at >= end || at + A <= begin || (at >= begin && at + A <= end)) continue;
#pragma unroll
      for (int e = 0; e < A; e++) {
        if (at + e < begin || at + e >= end) continue;
        const uint8_t *one = x + (u * STEP + e) * E;
        if constexpr (BF16) p.v[u][e >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t *>(one) << (16 * (e & 1));
        else p.v[u][e] = *reinterpret_cast<const uint32_t *>(one);
      }
    }
  }
  return p;
}
// Element e of 16 bytes as a probability.
template <bool BF16>
__device__ __forceinline__ float probability(u32x4 v, int e) {
  const uint32_t w = BF16 ? v[e >> 1] : v[e];
  return clean(__uint_as_float(!BF16 ? w : (e & 1) ? w & 0xFFFF0000u : w << 16));
}
__device__ __forceinline__ double shfl(double v, int lane) { return __shfl(v, lane); }
// Sum over the wave, the same bits on every lane.
__device__ __forceinline__ double sum64d(double v) {
  v = sum_lanes<16>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
// Sums of the lanes up to and including this one: within 16 lanes by shifts of 1,
// 2, 4 and 8 (row_shr), then the last lane of a row to the next one, and that of
// the first two rows to the others (row_bcast 15 and 31).
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double scan64(double v) {
  v += shifted<0x111, 0xF>(v);
  v += shifted<0x112, 0xF>(v);
  v += shifted<0x114, 0xF>(v);
  v += shifted<0x118, 0xF>(v);
  v += shifted<0x142, 0xA>(v);
  return v + shifted<0x143, 0xC>(v);
}

// Weight of an element of a row that is drawn from.
template <bool BF16>
__device__ __forceinline__ double weight_of(u32x4 p, u32x4 q, bool residual, int e) {
  const double t = probability<BF16>(p, e);
  if (!residual) return t;
  return __builtin_fmax(t - (double)probability<BF16>(q, e), 0.0);
}

// A wave a chunk; a workgroup's z takes rows z, z + gridDim.z, ... of a sequence. Each
// finds out by itself which those are (a launch of its own for that took 3 to 5.5 us);
// one of a sequence leaves it for the walk. 64 chains of 8 over 128,000 tokens, fp32:
// 65 MB.
template <bool BF16>
__global__ __launch_bounds__(256) void k_verify_sums(const VerifyArgs a) {
  __shared__ Plan plan;
  auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const int chunk = uniform(blockIdx.x * 4 + (threadIdx.x >> 6)), i = blockIdx.y;
  const Sequence s = sequence_of(a, i);
  if ((int)blockIdx.z >= max(s.nodes, 1)) return;
  make_plan<BF16>(a, s, plan);
  const int many = uniform(plan.many);
  if (blockIdx.x == 0 && blockIdx.z == 0) {
    for (int j = threadIdx.x; j < s.nodes; j += 256) {
      a.kid[s.first + j] = plan.kid[j];
      if (j < many) a.draws[s.first + j] = plan.draws[j];
    }
    if (threadIdx.x == 0) a.many[i] = many;
  }
  if (chunk >= a.chunks) return;
  for (int r = blockIdx.z; r < many; r += gridDim.z) {
    const int draws = uniform(plan.draws[r]);
    const int64_t row = s.first + (draws & ~kResidual);
    const bool residual = draws & kResidual;
    const Part<BF16> p = load_part<BF16, false>(a.target, a, row, chunk);
    Part<BF16> q = {};
    if (residual) q = load_part<BF16, false>(a.draft, a, row, chunk);
    double w = 0.0, t = 0.0;
    if (residual) {
#pragma unroll
      for (int u = 0; u < Part<BF16>::U; u++)
#pragma unroll
        for (int e = 0; e < Part<BF16>::A; e++) {
          w += weight_of<BF16>(p.v[u], q.v[u], true, e);
          t += weight_of<BF16>(p.v[u], q.v[u], false, e);
        }
    } else {
#pragma unroll
      for (int u = 0; u < Part<BF16>::U; u++)
#pragma unroll
        for (int e = 0; e < Part<BF16>::A; e++) t += weight_of<BF16>(p.v[u], q.v[u], false, e);
      w = t;
    }
    w = sum64d(w);
    t = sum64d(t);
    if ((threadIdx.x & 63) == 0) {
      double *to = a.sums + ((s.first + r) * a.chunks + chunk) * 2;
      to[0] = w;
      to[1] = t;
    }
  }
}

// Draws from a row, the whole wave together; -1 where nothing in it is positive.
template <bool BF16>
__device__ __forceinline__ int64_t draw_from(const VerifyArgs &a, int64_t slot, int64_t row, bool residual) {
  const int lane = threadIdx.x & 63;
  const double *sums = a.sums + slot * a.chunks * 2;
  const double number = a.numbers[2 * row + 1];
  double total = 0.0, head = 0.0;  // head: of the first 64 chunks
  int which = 0;                   // w, or, where w has nothing, p
  for (; which < 2; which++) {
    head = lane < a.chunks ? sums[2 * lane + which] : 0.0;
    double t = head;
    for (int c = lane + 64; c < a.chunks; c += 64) t += sums[2 * c + which];
    total = sum64d(t);
    if (total > 0.0) break;
  }
  if (which == 2) return -1;
  if (which == 1) residual = false;
  const double bound = number * total;
  // the chunk in which the sum passes the bound; if rounding leaves it below, the last with anything
  double before = 0.0, base = 0.0;
  int chunk = -1;
  for (int c0 = 0; c0 < a.chunks; c0 += 64) {
    const double v = c0 == 0 ? head : c0 + lane < a.chunks ? sums[2 * (c0 + lane) + which] : 0.0;
    const double incl = scan64(v);
    const uint64_t any = __ballot(v > 0.0), past = __ballot(v > 0.0 && before + incl > bound);
    const uint64_t take = past ? past & -past : any ? 1ull << (63 - __builtin_clzll(any)) : 0;
    if (take) {
      const int l = __builtin_ctzll(take);
      chunk = c0 + l;
      base = before + (shfl(incl, l) - shfl(v, l));
      if (past) break;
    }
    before += shfl(incl, 63);
  }
  chunk = __builtin_amdgcn_readfirstlane(chunk);
  constexpr int A = Part<BF16>::A, U = Part<BF16>::U;
  const Part<BF16> p = load_part<BF16, true>(a.target, a, row, chunk);
  Part<BF16> q = {};
  if (residual) q = load_part<BF16, true>(a.draft, a, row, chunk);
  // the lane in which it does, from the lanes' sums, then its step, then its element
  double part[U], mine = 0.0;
#pragma unroll
  for (int u = 0; u < U; u++) {
    part[u] = 0.0;
#pragma unroll
    for (int e = 0; e < A; e++) part[u] += weight_of<BF16>(p.v[u], q.v[u], residual, e);
    asm volatile("" : "+v"(part[u]));  // formed here and held, not formed again below
    mine += part[u];
    __builtin_amdgcn_sched_barrier(0);  // few numbers in 64 bits at a time
  }
  const double incl = scan64(mine);
  const uint64_t any = __ballot(mine > 0.0), past = __ballot(mine > 0.0 && base + incl > bound);
  if (!any) return -1;
  const int l = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(any);
  double at = base + (incl - mine), sum = at;
  int step = 0;
  u32x4 mine_p = {0, 0, 0, 0}, mine_q = {0, 0, 0, 0};
  bool over = false;
#pragma unroll
  for (int u = 0; u < U; u++) {
    if (part[u] > 0.0 && !over) {
      step = u;
      mine_p = p.v[u];
      mine_q = q.v[u];
      sum = at;
      over = at + part[u] > bound;
    }
    at += part[u];
  }
  int last = -1;
  bool done = false;
#pragma unroll
  for (int e = 0; e < A; e++) {
    const double w = weight_of<BF16>(mine_p, mine_q, residual, e);
    sum += w;
    if (w > 0.0 && !done) {
      last = e;
      done = sum > bound;
    }
  }
  // (places count from the boundary before the row)
  const int64_t found = (int64_t)chunk * kChunk + (lane * U + step) * A + last - ((row * a.vocab) & (A - 1));
  return __shfl((long long)(last < 0 ? -1 : found), l);
}

// A wave a row to draw at, all of a sequence's at once where they are 16 or fewer.
template <bool BF16>
__global__ __launch_bounds__(1024) void k_verify_walk(const VerifyArgs a) {
  __shared__ int up[kNodes], kid[kNodes], id[kNodes], drawn[kNodes];
  // (the wave's number and what follows from it is in scalar registers)
  auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const int i = blockIdx.x, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int found = a.tokens ? a.many[i] : 0;
  const Sequence s = sequence_of(a, i);
  int32_t *path = a.path + (int64_t)i * a.width;
  // the wave's row is asked for beside how many there are, before what the walk needs
  const int first = wave < s.nodes ? a.draws[s.first + wave] : 0;
  for (int j = threadIdx.x; j < s.nodes; j += blockDim.x) {
    up[j] = a.parents[s.first + j];
    kid[j] = a.kid[s.first + j];
    id[j] = a.ids[s.first + j];
  }
  if (wave < s.nodes) {
    int draws = uniform(first);
    const int many = uniform(found);
    for (int r = wave; r < many; r += blockDim.x >> 6) {
      if (r != wave) draws = uniform(a.draws[s.first + r]);
      const int j = draws & ~kResidual;
      if (j >= s.nodes) continue;  // (another sequence's, where cu falls)
      const int64_t t = draw_from<BF16>(a, s.first + r, s.first + j, draws & kResidual);
      if (lane == 0) drawn[j] = (int)t;
    }
  }
  __syncthreads();
  if (wave) return;
  // (nodes rise and stay inside, also where cu falls and sequences share rows of
  // the scratch)
  int node = 0, steps = 0, token = -1;
  while (s.nodes) {
    if (lane == 0) path[steps] = node;
    steps++;
    const int k = kid[node], taken = k & ~kTaken;
    if (k >= 0 && (k & kTaken) && taken > node && taken < s.nodes && steps < a.width) {
      node = taken;
      continue;
    }
    token = drawn[node];
    token = token >= 0 && token < a.vocab ? token : -1;
    int next = -1;
    for (int j0 = node + 1; j0 < s.nodes && token >= 0 && steps < a.width && next < 0; j0 += 64) {
      const int j = j0 + lane;
      const bool hit = j < s.nodes && up[j] == node && id[j] == token && !(a.draft && j == k);
      const uint64_t all = __ballot(hit);
      if (all) next = j0 + __builtin_ctzll(all);
    }
    if (next < 0) break;
    node = next;
  }
  for (int j = steps + lane; j < a.width; j += 64) path[j] = -1;
  if (lane == 0) {
    a.count[i] = steps;
    a.token[i] = token;
  }
}

static int verify_chunks(int64_t vocab) { return (int)((vocab + 7 + kChunk - 1) / kChunk); }
static size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace mxl

using namespace mxl;

size_t mxi_verify_workspace(int64_t tokens, int batch, int64_t vocab) {
  return (size_t)tokens * verify_chunks(vocab) * 16 + 2 * round16((size_t)tokens * 4) + round16((size_t)batch * 4);
}

hipError_t mxi_launch_verify(const void *target, const void *draft, int bf16, const int32_t *ids,
                             const int32_t *parents, const int32_t *cu, const float *numbers,
                             int64_t tokens, int batch, int64_t vocab, int width, int32_t *path,
                             int32_t *count, int32_t *token, void *workspace, hipStream_t st) {
  VerifyArgs a = {target, draft, ids, parents, cu, numbers, tokens, vocab, batch, width,
                  verify_chunks(vocab), path, count, token, nullptr, nullptr, nullptr, nullptr};
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.sums = reinterpret_cast<double *>(ws);
  ws += (size_t)tokens * a.chunks * 16;
  a.kid = reinterpret_cast<int32_t *>(ws);
  ws += round16((size_t)tokens * 4);
  a.draws = reinterpret_cast<int32_t *>(ws);
  ws += round16((size_t)tokens * 4);
  a.many = reinterpret_cast<int32_t *>(ws);
  if (tokens == 0) {  // outputs alone
    k_verify_walk<false><<<batch, 64, 0, st>>>(a);
    return hipGetLastError();
  }
  const int groups = (a.chunks + 3) / 4;
  const int64_t mean = std::max<int64_t>(1, tokens / batch);
  // workgroups for four a compute unit: each makes the plan (64 chains of 8 over 128,000
  // tokens 21.8 us, with four times as many 27.6)
  const int rows = (int)std::min<int64_t>(mean, std::max<int64_t>(1, 1024 / ((int64_t)groups * batch)));
  const dim3 grid((uint32_t)groups, (uint32_t)batch, (uint32_t)rows);
  const int threads = 64 * (int)std::min<int64_t>(16, mean);
  if (bf16) {
    k_verify_sums<true><<<grid, 256, 0, st>>>(a);
    k_verify_walk<true><<<batch, threads, 0, st>>>(a);
  } else {
    k_verify_sums<false><<<grid, 256, 0, st>>>(a);
    k_verify_walk<false><<<batch, threads, 0, st>>>(a);
  }
  return hipGetLastError();
}
