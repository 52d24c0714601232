// Routing of tokens over experts: top-k selection, per-expert counts and the balance loss, and
// the gradient of the logits.  Arithmetic is fp32, counts are integers.
//
//   p = softmax(l);  the k largest logits of a token are chosen, the lowest index first among
//   equals;  gate = p there, or normalised over the chosen;  N = tokens that count
//   loss = E / (k N^2) sum_e counts_e sum_t p_te
//   c_e = dloss E counts_e / (k N^2);  dl = p (c + dgate at the chosen - sum_e p (...))
//
// G lanes hold one token's logits, eight (times NC) neighbouring experts each, so a warp works
// on 32 / G tokens, each logit is read once, and a lane meets the same experts in every token:
// the sums over tokens of p stay in its registers.
#include <algorithm>

#include "mb_block.h"
#include "mb_device.cuh"
#include "mb_rows.cuh"
#include "muonbank.h"

namespace mb {
namespace {

constexpr int WARPS = 16;             // per CTA, two CTAs per SM
constexpr int THREADS = WARPS * 32;
constexpr unsigned FULL = 0xFFFFFFFFu;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float MINUS_INF = -__builtin_huge_valf();

// The softmax takes these approximations in place of expf and a division: one instruction per element in a
// kernel that instructions bound.  The results of a call are within 1.7e-7 of their size (with expf and a
// division 5e-8 to 6e-8); exponentials below 2^-126 are 0, which against a sum of at least 1 changes none but
// their own.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Exact keys in the order of the logits: -inf (an expert that is not available) is 0, NaN is
// above everything, both zeros are one.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  if (l != l) return 0xFFFFFFFFu;
  if (u == 0xFF800000u) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (key == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  if (key == 0u) return MINUS_INF;
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
  if constexpr (G == 32) return __reduce_max_sync(FULL, x);
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) {
    const uint32_t y = __shfl_xor_sync(FULL, x, o);
    x = y > x ? y : x;
  }
  return x;
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t x) {
  if constexpr (G == 32) return __reduce_min_sync(FULL, x);
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) {
    const uint32_t y = __shfl_xor_sync(FULL, x, o);
    x = y < x ? y : x;
  }
  return x;
}
template <int G>
__device__ __forceinline__ float group_add(float x) {
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
  return x;
}
template <int G>
__device__ __forceinline__ float group_fmax(float x) {
  if constexpr (G == 32) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
  }
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(FULL, x, o));
  return x;
}

__device__ __forceinline__ void count_one(int* counter) {
  asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(smem_u32(counter)) : "memory");
}

// Whether any lane of this lane's group says so.
template <int G>
__device__ __forceinline__ bool any_of_group(bool x, int lane) {
  if constexpr (G == 32) return __any_sync(FULL, x) != 0;
  const uint32_t votes = __ballot_sync(FULL, x) >> (lane & ~(G - 1));
  return (votes & ((1u << (G & 31)) - 1u)) != 0;
}

// Expert of element j of piece c of lane g in its group.
template <int G>
__device__ __forceinline__ int expert_of(int c, int g, int j) { return (c * G + g) * 8 + j; }

// The lane's logits of one token as loaded (one load ahead of their use); experts past the
// last, and tokens that are not read, are -inf.
template <typename T, bool VEC, int G, int NC>
struct Logits {
  Eight<T> v[VEC ? NC : 1];
  float f[VEC ? 1 : 8 * NC];
  bool on;
  __device__ __forceinline__ void load(const T* row, bool read, int experts, int g) {
    on = read;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e0 = expert_of<G>(c, g, 0);
      if constexpr (VEC) {
        if (on && e0 < experts) v[c].load(row + e0);
        else v[c].fill(minus_inf_bits(T()));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[8 * c + j] = on && e0 + j < experts ? to_float(row[e0 + j]) : MINUS_INF;
      }
    }
  }
  __device__ __forceinline__ void get(float (&l)[8 * NC]) const {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float x[8];
      if constexpr (VEC) v[c].get(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) l[8 * c + j] = VEC ? x[j] : f[8 * c + j];
    }
  }
};

__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
  const uint32_t lo = min(a, b);
  b = max(a, b);
  a = lo;
}

// All eight in order (19 comparisons).
__device__ __forceinline__ void sort8(uint32_t (&k)[8]) {
  order2(k[0], k[2]), order2(k[1], k[3]), order2(k[4], k[6]), order2(k[5], k[7]);
  order2(k[0], k[4]), order2(k[1], k[5]), order2(k[2], k[6]), order2(k[3], k[7]);
  order2(k[0], k[1]), order2(k[2], k[3]), order2(k[4], k[5]), order2(k[6], k[7]);
  order2(k[2], k[4]), order2(k[3], k[5]);
  order2(k[1], k[4]), order2(k[3], k[6]);
  order2(k[1], k[2]), order2(k[3], k[4]), order2(k[5], k[6]);
}
__device__ __forceinline__ void sort4(uint32_t (&k)[4]) {
  order2(k[0], k[1]), order2(k[2], k[3]), order2(k[0], k[2]), order2(k[1], k[3]), order2(k[1], k[2]);
}

// A lane's least D (4 or 8) of V keys, in order, by networks of minima and maxima: D at a time, the
// least D of both sorted runs being a bitonic sequence.
template <int D, int V>
__device__ __forceinline__ void least(const uint32_t (&key)[V], uint32_t (&out)[D]) {
#pragma unroll
  for (int q = 0; q < V; q += D) {
    uint32_t f[D];
#pragma unroll
    for (int j = 0; j < D; ++j) f[j] = key[q + j];
    if constexpr (D == 8) sort8(f);
    else sort4(f);
    if (q == 0) {
#pragma unroll
      for (int j = 0; j < D; ++j) out[j] = f[j];
    } else {
#pragma unroll
      for (int j = 0; j < D; ++j) out[j] = min(out[j], f[D - 1 - j]);
#pragma unroll
      for (int d = D / 2; d > 0; d /= 2)
#pragma unroll
        for (int j = 0; j < D; ++j)
          if ((j & d) == 0) order2(out[j], out[j + d]);
    }
  }
}

// The counts and the loss from the CTAs' sums ({sum of p, count} of every expert, n rows of them);
// called by the threads of a CTA for the experts [e_begin, e_end); returns (to every thread) the
// share of  sum_e counts_e sum_t p_te  of these experts.  sums: 33 entries per warp.
__device__ __forceinline__ float finish_experts(const RouterParams& p, int n, int e_begin, int e_end, int2* sums) {
  // 32 experts by (threads / 32) slices of the rows at a time, added in a fixed order
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, slices = blockDim.x >> 5;
  float share = 0.f;
  for (int e0 = e_begin; e0 < e_end; e0 += 32) {
    const int e = e0 + lane;
    float a = 0.f;
    int c = 0;
    if (e < e_end) {
#pragma unroll 10
      for (int i = slice; i < n; i += slices) {
        const int2 v = p.parts_sums[static_cast<size_t>(i) * p.experts + e];
        a += __int_as_float(v.x);
        c += v.y;
      }
    }
    sums[slice * 33 + lane] = make_int2(__float_as_int(a), c);
    __syncthreads();
    for (int i = slice; i < 32; i += slices) {         // expert e0 + i: the slices' sums over a warp's lanes
      const int2 v = lane < slices ? sums[lane * 33 + i] : make_int2(0, 0);
      a = group_add<32>(__int_as_float(v.x));
      c = __reduce_add_sync(FULL, v.y);
      if (e0 + i < e_end) {
        if (lane == 0) p.counts[e0 + i] = c;
        share += a * static_cast<float>(c);
      }
    }
    __syncthreads();
  }
  if (lane == 0) sums[slice].x = __float_as_int(share);
  __syncthreads();
  share = group_add<32>(lane < slices ? __int_as_float(sums[lane].x) : 0.f);
  __syncthreads();
  return share;
}

__device__ __forceinline__ float loss_of(float share, int used, int experts, int k) {
  if (used == 0) return 0.f;
  const float n = static_cast<float>(used);
  return share * (static_cast<float>(experts) / (static_cast<float>(k) * n)) / n;
}

// ---------------------------------------------------------------- forward

// A lane keeps the r-th chosen experts with r % G equal to its place in the group.
template <int G, int V = 8>
struct Slots {
  static constexpr int N = 32 / G < V ? 32 / G : V;    // k <= V G and k <= 32
};

// A token's softmax and its k largest logits for any values, in little code, because it is rare and
// its instructions have to be fetched first: every round looks for the best that comes after the one
// before it, over exact keys.  Puts the chosen experts into `order` (-1: none).  The terms of the
// softmax are exp(l - m); NaN or +inf among the logits makes the sum NaN, and with it every
// probability of the token.
struct ExactSoftmax {
  float m, sum;
  bool some;
};
template <typename T, int G, int V>
__device__ __forceinline__ ExactSoftmax select_exact(const T* row, bool mine, int experts, int g, int k, uint32_t* order) {
  ExactSoftmax x{0.f, 0.f, false};
  uint32_t before = 0xFFFFFFFFu, top = 0;
  uint32_t before_e = 0xFFFFFFFFu;                     // the first round takes any
#pragma unroll 1
  for (int r = 0; r < k; ++r) {
    uint32_t best = 0, who = 0x7FFFFFFFu;
#pragma unroll 4
    for (int j = 0; j < V; ++j) {
      const uint32_t e = expert_of<G>(j / 8, g, j & 7);
      const uint32_t key = mine && e < static_cast<uint32_t>(experts) ? key_of(to_float(row[e])) : 0;
      const bool after = r == 0 || key < before || (key == before && e > before_e);
      if (after && key > best) {
        best = key;
        who = e;
      }
    }
    before = group_max<G>(best);
    before_e = group_min<G>(best == before && before != 0 ? who : 0x7FFFFFFFu);
    if (r == 0) top = before;
    order[r] = before != 0 ? before_e : 0xFFFFFFFFu;   // the same value from every lane of the group
  }
  x.some = top != 0;
  x.m = value_of(top);
#pragma unroll 4
  for (int j = 0; j < V; ++j) {
    const int e = expert_of<G>(j / 8, g, j & 7);
    const float l = mine && e < experts ? to_float(row[e]) : MINUS_INF;
    x.sum += l == MINUS_INF ? 0.f : expf(l - x.m);
  }
  x.sum = group_add<G>(x.sum);
  if (top >= 0xFF800000u) x.sum = __uint_as_float(0x7FC00000u);
  return x;
}

// Puts keys 0..k, whose upper bits are in order, in the order of their logits (the lower number first
// among equals, as they come).
template <uint32_t IDX, typename T>
__device__ __forceinline__ void put_right(uint32_t* order, int k, const T* row) {
  bool moved = true;
#pragma unroll 1
  for (int pass = 0; pass < k && moved; ++pass) {
    moved = false;
#pragma unroll 1
    for (int r = 0; r < k; ++r) {
      const uint32_t a = order[r], b = order[r + 1];
      if (((a ^ b) & ~IDX) == 0 && to_float(row[a & IDX]) < to_float(row[b & IDX])) {
        order[r] = b;
        order[r + 1] = a;
        moved = true;
      }
    }
  }
}

// Selection without conditions per element.  With c = max * log2(e) rounded up, x = l log2(e) - c
// is at most 0, monotone in l, and the exponent the softmax needs anyway.  The bits of such an x
// grow as l falls, so a key of x's upper bits and the expert's number in the low ones sorts by
// falling logit, then by number, with one minimum per comparison.  A lane keeps its best few keys
// (D: eight of up to 8 lanes, four of 32); rounds of a minimum over the group take the best and pop
// it from its lane.  Where a lane gave all it kept, the rounds are done again over all keys (with
// k = 8 that is one token in 1000 of 256 experts, and every one of equal logits).
//
// Neighbours in the order whose keys agree in the upper bits are compared themselves and put right by
// their group's first lane.  Some tokens this cannot decide: more than the first left out agrees
// with the last chosen, and is larger; fewer than k are above -inf in x though not in the logits; or
// the sum is not that of a softmax (NaN, infinities, overflow).  They are left out, marked in
// `index`, and a second loop selects for them exactly (in the first loop that path cost a fifth of
// its instructions even where it was not taken).
//
// A lane holds 16 experts and not eight up to 128 experts, although that leaves registers for half
// the warps: 262144 tokens of 128 experts, k = 8, take 65 us and not 100, bf16 of 64 39 and not 47.
// Of 256 experts eight are faster (131072 tokens 64 us, with 16 lanes of 16 experts 70); beyond, the
// lanes are 32 and hold 16 or 32.
//
// Bound by instructions, not by HBM: 420 per token of 256 experts with k = 8, at 77 % of the issue
// slots; the loads alone (134 MB) would take 21 us.
constexpr int UNDECIDED = -2;

template <typename T, bool VEC, int G, int NC>
__global__ void __launch_bounds__(THREADS, NC == 1 ? 2 : 1) router_kernel(const RouterParams p) {
  begin_after_previous();
  // [WARPS][experts] sums of p, [experts] counts, [WARPS][TOK][k + 1] chosen keys
  extern __shared__ float dyn[];
  __shared__ float warp_share[WARPS];
  __shared__ int warp_used[WARPS];
  constexpr int V = 8 * NC;
  constexpr int TOK = 32 / G;                          // tokens per warp
  constexpr int SLOTS = Slots<G, V>::N;
  constexpr bool BYTE = V * G <= 256;                  // the expert's number is a byte
  constexpr uint32_t IDX = BYTE ? 255 : V * G - 1;     // its bits of a key
  constexpr uint32_t CLOSED = 0xFF800000u;             // a key from here on: x = -inf
  constexpr uint32_t NONE = 0xFFFFFFFFu;               // no key
  constexpr int D = G < 32 ? 8 : 4;                    // keys a lane keeps
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane % G;
  int* scount = reinterpret_cast<int*>(dyn + WARPS * p.experts);
  uint32_t* order = reinterpret_cast<uint32_t*>(scount + p.experts) + (warp * TOK + lane / G) * (p.k + 1);
  for (int e = threadIdx.x; e < p.experts; e += THREADS) scount[e] = 0;
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) psum[j] = 0.f;
  uint32_t bytes[V / 4];                               // the numbers of the lane's experts, four to a word
#pragma unroll
  for (int q = 0; q < V / 4; ++q) bytes[q] = static_cast<uint32_t>(expert_of<G>(q / 2, g, 4 * (q & 1))) * 0x01010101u + 0x03020100u;
  int used_here = 0;
  bool left_over = false;
  const int stride = static_cast<int>(gridDim.x) * WARPS * TOK;   // tokens < 2^31, checked before the launch
  Logits<T, VEC, G, NC> next;
  long long token = static_cast<long long>(blockIdx.x * WARPS + warp) * TOK + lane / G;
  const T* row = static_cast<const T*>(p.logits) + token * p.stride;   // of `token`, then of the next one to load
  const long long row_step = stride * p.stride;
  auto fetch = [&](long long t) { next.load(row, t < p.tokens && (!p.valid || p.valid[t] != 0), p.experts, g); };
  long long at = token * p.k + g;                      // of the lane's first chosen expert in index and gate
  const long long at_step = static_cast<long long>(stride) * p.k;
  const long long first = token - lane / G;            // of the warp's tokens: the loop runs by it
  if (first < p.tokens) fetch(token);
  for (long long base = first; base < p.tokens; base += stride, token += stride) {
    float l[V];
    next.get(l);
    bool on = next.on;
    const T* here = row;
    row += row_step;
    if (base + stride < p.tokens) fetch(token + stride);
    float m = l[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
    m = group_fmax<G>(m);
    if (__any_sync(FULL, on && m == MINUS_INF)) {      // no expert is open, or NaN hides behind -inf
      bool nan = false;
#pragma unroll
      for (int j = 0; j < V; ++j) nan |= l[j] != l[j];
      nan = any_of_group<G>(nan, lane);
      on &= m > MINUS_INF || nan;
      // x = -inf, and with it a closed key, for the places past the last expert too: -inf - (-inf) would be
      // NaN, their keys would come before closed ones, and the comparisons below would read past the row
      if (m == MINUS_INF && nan) m = 0.f;
    }
    const float down = 0.f - __fmul_ru(m, LOG2E);      // +0 for a maximum of either zero
    float e[V], sum = 0.f;
    uint32_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float x = fmaf(l[j], LOG2E, down);
      e[j] = exp2_approx(x);
      sum += e[j];
      if constexpr (BYTE)         // in place of the lowest byte
        key[j] = __byte_perm(__float_as_uint(x), bytes[j / 4], 0x3210 + 4 + (j & 3));
      else
        key[j] = (__float_as_uint(x) & ~IDX) | static_cast<uint32_t>(expert_of<G>(j / 8, g, j & 7));
    }
    sum = group_add<G>(sum);
    uint32_t own[D];
    least<D, V>(key, own);
    const uint32_t deepest = own[D - 1];
    // the k best of the group and the first after them, in order; a lane that has given the last
    // of its kept keys gives it again
#pragma unroll 3
    for (int r = 0; r <= p.k; ++r) {
      const uint32_t best = group_min<G>(own[0]);
      const bool won = own[0] == best;
      order[r] = best;                                 // the same value from every lane of the group
#pragma unroll
      for (int d = 0; d + 1 < D; ++d) own[d] = won ? own[d + 1] : own[d];
      if constexpr (D == V) own[D - 1] = won ? NONE : own[D - 1];
    }
    __syncwarp();
    if (D < V && p.k >= D && __any_sync(FULL, on && deepest <= order[p.k - 1])) {
      // a lane gave all it kept: the rounds again, over all keys
      uint32_t taken = 0;
      bool none = true;
      __syncwarp();
#pragma unroll 1
      for (int r = 0; r <= p.k; ++r) {
        uint32_t mine = NONE;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const uint32_t x = (__float_as_uint(fmaf(l[j], LOG2E, down)) & ~IDX) |
                             static_cast<uint32_t>(expert_of<G>(j / 8, g, j & 7));
          if (none || x > taken) mine = min(mine, x);
        }
        const uint32_t best = group_min<G>(mine);
        order[r] = best;
        if (mine == best) {
          taken = best;
          none = false;
        }
      }
      __syncwarp();
    }
    int idx[SLOTS];
    float w[SLOTS];                                    // the chosen logits, then the softmax's terms
    bool wrong = false;                                // a key's successor has the larger logit
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int r = s * G + g;
      idx[s] = -1;
      w[s] = 0.f;
      if (s * G < p.k && r < p.k && on) {
        const uint32_t mine = order[r], then = order[r + 1];
        if (mine < CLOSED) {
          idx[s] = static_cast<int>(mine & IDX);
          w[s] = to_float(here[idx[s]]);
          if ((mine & ~IDX) == (then & ~IDX)) wrong |= !(w[s] >= to_float(here[then & IDX]));
        }
      }
    }
    if (__any_sync(FULL, wrong)) {
      if (g == 0 && on) put_right<IDX>(order, p.k, here);
      __syncwarp();
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        if (idx[s] >= 0) {
          idx[s] = static_cast<int>(order[s * G + g] & IDX);
          w[s] = to_float(here[idx[s]]);
        }
      }
    }
    const uint32_t last = order[p.k - 1], after = order[p.k];
    bool unsure = on && !(sum >= 0.5f);
    if (__any_sync(FULL, on && last >= CLOSED)) {      // fewer than k above -inf: in the logits, or only in x?
#pragma unroll
      for (int j = 0; j < V; ++j) unsure |= on && l[j] > MINUS_INF && fmaf(l[j], LOG2E, down) == MINUS_INF;
    }
    const bool tie = on && last < CLOSED && (last & ~IDX) == (after & ~IDX);
    if (__any_sync(FULL, tie)) {                       // no other that agrees with the last may be larger
      const float worst = tie ? to_float(here[last & IDX]) : 0.f;
      uint32_t larger = 0;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (tie && ((__float_as_uint(fmaf(l[j], LOG2E, down)) ^ last) & ~IDX) == 0 && !(l[j] <= worst)) larger |= 1u << j;
      while (larger != 0) {
        const int j = __ffs(static_cast<int>(larger)) - 1, e = expert_of<G>(j / 8, g, j & 7);
        larger &= larger - 1;
        bool chosen = false;
#pragma unroll 1
        for (int r = 0; r < p.k; ++r) chosen |= (order[r] & IDX) == static_cast<uint32_t>(e);
        unsure |= !chosen;
      }
    }
    unsure = any_of_group<G>(unsure, lane);
    left_over |= unsure;
    const bool used = on && !unsure;
    const float inv = used ? reciprocal(sum) : 0.f;
    if (used) {
#pragma unroll
      for (int j = 0; j < V; ++j) psum[j] = fmaf(e[j], inv, psum[j]);
      if (g == 0) ++used_here;
    }
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) w[s] = idx[s] >= 0 ? exp2_approx(fmaf(w[s], LOG2E, down)) : 0.f;
    float scale = inv;
    if (p.normalize) {
      float chosen = 0.f;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) chosen += w[s];
      chosen = group_add<G>(chosen);                   // by every lane, whether its token counts or not
      scale = used ? reciprocal(chosen) : 0.f;
    }
    int* to_index = p.index + at;
    float* to_gate = p.gate + at;
    at += at_step;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (s * G >= p.k) break;
      if (s * G + g < p.k && token < p.tokens) {
        to_index[s * G] = unsure ? UNDECIDED : idx[s];
        to_gate[s * G] = w[s] * scale;                 // w is 0 at a place without an expert
        if (used && idx[s] >= 0) count_one(&scount[idx[s]]);
      }
    }
    __syncwarp();                                      // the order has been read
  }
  __syncwarp();
  // the tokens left over, exactly: a lane looks up one of the warp's next 32, then their groups work
  for (long long from = first; __any_sync(FULL, left_over) && from < p.tokens; from += G * static_cast<long long>(stride)) {
    const long long look = from + lane / TOK * static_cast<long long>(stride) + lane % TOK;
    uint32_t todo = __ballot_sync(FULL, look < p.tokens && p.index[look * p.k] == UNDECIDED);
    while (todo != 0) {
      const int round = (__ffs(static_cast<int>(todo)) - 1) / TOK;
      const bool mine = (todo >> (round * TOK + lane / G) & 1u) != 0;
      todo &= ~((TOK == 32 ? FULL : (1u << (TOK & 31)) - 1u) << (round * TOK));
      const long long t = from + round * static_cast<long long>(stride) + lane / G;
      const T* row = static_cast<const T*>(p.logits) + t * p.stride;
      const ExactSoftmax x = select_exact<T, G, V>(row, mine, p.experts, g, p.k, order);
      __syncwarp();
      const float inv = x.some ? 1.f / x.sum : 0.f;
      int idx[SLOTS];
      float w[SLOTS], chosen = 0.f;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        const int r = s * G + g;
        idx[s] = mine && r < p.k ? static_cast<int>(order[r]) : -1;
        w[s] = idx[s] >= 0 ? expf(to_float(row[idx[s]]) - x.m) : 0.f;
        chosen += w[s];
      }
      chosen = group_add<G>(chosen);
      const float scale = p.normalize && x.some && x.sum == x.sum ? 1.f / chosen : inv;
      if (mine && x.some) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = expert_of<G>(j / 8, g, j & 7);
          const float l = e < p.experts ? to_float(row[e]) : MINUS_INF;
          psum[j] += l == MINUS_INF && x.sum == x.sum ? 0.f : exp2_approx((l - x.m) * LOG2E) * inv;
        }
        if (g == 0) ++used_here;
      }
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        const int r = s * G + g;
        if (mine && r < p.k) {
          p.index[t * p.k + r] = idx[s];
          p.gate[t * p.k + r] = idx[s] >= 0 ? w[s] * scale : 0.f;
          if (idx[s] >= 0) count_one(&scount[idx[s]]);
        }
      }
      __syncwarp();
    }
  }
  // the CTA's sums, in a fixed order: the warp's token groups, then its warps
#pragma unroll
  for (int j = 0; j < V; ++j) {
    for (int o = G; o < 32; o <<= 1) psum[j] += __shfl_xor_sync(FULL, psum[j], o);
    const int e = expert_of<G>(j / 8, g, j & 7);
    if (lane < G && e < p.experts) dyn[warp * p.experts + e] = psum[j];
  }
  used_here = __reduce_add_sync(FULL, used_here);
  if (lane == 0) warp_used[warp] = used_here;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < WARPS; ++w) total += warp_used[w];
  float share = 0.f;
  for (int e = threadIdx.x; e < p.experts; e += THREADS) {
    float a = 0.f;
    for (int w = 0; w < WARPS; ++w) a += dyn[w * p.experts + e];
    const int c = scount[e];
    if (gridDim.x > 1) {
      p.parts_sums[static_cast<size_t>(blockIdx.x) * p.experts + e] = make_int2(__float_as_int(a), c);
    } else {
      p.counts[e] = c;
      share += a * static_cast<float>(c);
    }
  }
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) p.part_used[blockIdx.x] = total;
    return;
  }
  // the only CTA finishes by itself
  share = group_add<32>(share);
  if (lane == 0) warp_share[warp] = share;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < WARPS; ++w) share += warp_share[w];
    p.loss[0] = loss_of(share, total, p.experts, p.k);
    p.used[0] = total;
  }
}

// A cluster of CTAs shares the experts; the first one adds the shares of the loss.
constexpr int FINISH_CTAS = 8;

__global__ void __launch_bounds__(1024) router_finish_kernel(const RouterParams p) {
  begin_after_previous();
  __shared__ int2 sums[32 * 33];
  __shared__ float share;
  const uint32_t rank = cluster_ctarank();
  int used = 0;                                        // of the first warp, asked for before the sums
  if (rank == 0 && threadIdx.x < 32) {
#pragma unroll 10
    for (int i = threadIdx.x; i < p.parts; i += 32) used += p.part_used[i];
  }
  const int per = (p.experts + FINISH_CTAS - 1) / FINISH_CTAS;
  const int e0 = static_cast<int>(rank) * per, e1 = e0 + per < p.experts ? e0 + per : p.experts;
  const float mine = finish_experts(p, p.parts, e0, e1, sums);
  if (threadIdx.x == 0) share = mine;
  cluster_sync_all();
  if (rank == 0 && threadIdx.x < 32) {
    const float of = threadIdx.x < FINISH_CTAS ? __uint_as_float(ld_cluster_u32(map_to_rank(&share, threadIdx.x))) : 0.f;
    const float all = group_add<32>(of);
    used = __reduce_add_sync(FULL, used);
    if (threadIdx.x == 0) {
      p.loss[0] = loss_of(all, used, p.experts, p.k);
      p.used[0] = used;
    }
  }
  cluster_sync_all();                                  // the shares are read before their CTAs end
}

// ---------------------------------------------------------------- backward

// With a_e = c_e (+ dgate at the chosen experts, unnormalised gates), dl = p (a - sum p a); with
// normalised gates gate (dgate - sum gate dgate) is added at the chosen ones instead.  What
// belongs to the chosen experts goes to their lanes through shared memory.
//
// Bound by HBM, the next token being loaded ahead: 262144 fp32 tokens of 256 experts with k = 8 take
// 92 us, 6.1 TB/s; narrow tokens (64 experts: 34 us, 4.4 TB/s) by the instructions per token.
template <typename T, bool VEC, int G, int NC>
__global__ void __launch_bounds__(THREADS, NC == 1 ? 2 : 1) router_bwd_kernel(const RouterBwdParams p) {
  begin_after_previous();
  extern __shared__ __align__(16) float dyn[];         // [WARPS][TOK][8 G NC], zero between tokens
  constexpr int V = 8 * NC;
  constexpr int TOK = 32 / G;
  constexpr int SLOTS = Slots<G>::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane % G;
  float* add = dyn + (warp * TOK + lane / G) * (G * V);
  const long long stride = static_cast<long long>(gridDim.x) * WARPS * TOK;
  const T* logits = static_cast<const T*>(p.logits);
  Logits<T, VEC, G, NC> next;
  int next_e[SLOTS];                                   // the lane's chosen experts of the next token
  float next_d[SLOTS], next_w[SLOTS];                  // ... their dgate and gate
  auto fetch = [&](long long base) {
    const long long token = base + lane / G;
    const bool on = token < p.tokens && (!p.valid || p.valid[token] != 0);
    next.load(logits + token * p.stride, on, p.experts, g);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (s * G >= p.k) break;
      const int r = s * G + g;
      const bool has = on && r < p.k && p.dgate;
      next_e[s] = has ? p.index[token * p.k + r] : -1;
      next_d[s] = has ? p.dgate[token * p.k + r] : 0.f;
      next_w[s] = has && p.normalize ? p.gate[token * p.k + r] : 0.f;
    }
  };
  long long base = (static_cast<long long>(blockIdx.x) * WARPS + warp) * TOK;
  if (base < p.tokens) fetch(base);                    // before the counts, so that their latencies overlap
#pragma unroll
  for (int j = 0; j < V; ++j) add[expert_of<G>(j / 8, g, j & 7)] = 0.f;
  float c[V];
  {
    const int n = *p.used;
    const float dloss = p.dloss ? *p.dloss : 0.f;
    int count[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert_of<G>(j / 8, g, j & 7);
      count[j] = e < p.experts ? p.counts[e] : 0;
    }
    const float nf = static_cast<float>(n > 0 ? n : 1);
    const float d = n > 0 ? dloss * (static_cast<float>(p.experts) / (static_cast<float>(p.k) * nf)) / nf : 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = d * static_cast<float>(count[j]);
  }
  __syncwarp();
  for (; base < p.tokens; base += stride) {
    const long long token = base + lane / G;
    float l[V];
    next.get(l);
    const bool on = next.on;
    int mine[SLOTS];
    float part[SLOTS];
    if (p.dgate) {
      float dot = 0.f;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        if (s * G >= p.k) break;
        mine[s] = next_e[s] < p.experts ? next_e[s] : -1;
        part[s] = next_d[s];
        if (p.normalize && mine[s] >= 0) dot = fmaf(next_w[s], next_d[s], dot);
      }
      if (p.normalize) {
        dot = group_add<G>(dot);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          if (s * G >= p.k) break;
          part[s] = next_w[s] * (part[s] - dot);
        }
      }
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        if (s * G >= p.k) break;
        if (mine[s] >= 0) add[mine[s]] = part[s];
      }
    }
    if (base + stride < p.tokens) fetch(base + stride);
    float m = l[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
    m = group_fmax<G>(m);
    const float shift = m * LOG2E;
    float e[V], sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      e[j] = exp2_approx(fmaf(l[j], LOG2E, -shift));
      sum += e[j];
    }
    sum = group_add<G>(sum);
    // a softmax's sum is between 1 and the number of experts: else NaN, infinities, overflow (of the
    // exponents, to either side), or no open expert
    if (__any_sync(FULL, on && !(sum >= 0.5f && sum <= 2.f * ROUTER_MAX_EXPERTS))) {
      bool any = false;
      float again = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        any |= !(l[j] == MINUS_INF);
        e[j] = l[j] == MINUS_INF ? 0.f : expf(l[j] - m);
        again += e[j];
      }
      again = group_add<G>(again);
      sum = group_max<G>(any ? 1u : 0u) != 0u ? again : __uint_as_float(0x7F800000u);   // 1 / sum = 0: every p is 0
    }
    const float inv = on ? reciprocal(sum) : 0.f;
    __syncwarp();
    float out[V], pa = 0.f;
#pragma unroll
    for (int q = 0; q < NC; ++q) {
      const float4* from = reinterpret_cast<const float4*>(add + expert_of<G>(q, g, 0));
      const float4 x = from[0], y = from[1];
      const float t[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = 8 * q + j;
        e[i] = on ? e[i] * inv : 0.f;
        out[i] = t[j];
        pa = fmaf(e[i], p.normalize ? c[i] : c[i] + t[j], pa);
      }
    }
    pa = group_add<G>(pa);
    if (token < p.tokens) {
      T* to = static_cast<T*>(p.dlogits) + token * p.dstride;
#pragma unroll
      for (int q = 0; q < NC; ++q) {
        const int e0 = expert_of<G>(q, g, 0);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 8 * q + j;
          f[j] = p.normalize ? fmaf(e[i], c[i] - pa, out[i]) : e[i] * (c[i] + out[i] - pa);
        }
        if constexpr (VEC) {
          if (e0 < p.experts) {
            Eight<T> o;
            o.set(f);
            o.store(to + e0);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e0 + j < p.experts) to[e0 + j] = from_float<T>(f[j]);
        }
      }
    }
    if (p.dgate) {
      __syncwarp();
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        if (s * G >= p.k) break;
        if (mine[s] >= 0) add[mine[s]] = 0.f;
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------- launches

int lanes_for(int experts) {
  int g = 1;
  while (g < 32 && g * 8 < experts) g *= 2;
  return g;
}

// Lanes of a token and pieces of eight experts per lane in the forward pass.
struct FwdShape {
  int g, nc, ctas;     // and CTAs per SM
};
FwdShape fwd_shape(int experts) {
  if (experts <= 8) return {1, 1, 2};
  if (experts > 128) return {32, experts > 512 ? 4 : experts > 256 ? 2 : 1, experts > 256 ? 1 : 2};
  int g = 1;
  while (g * 16 < experts) g *= 2;
  return {g, 2, 1};
}

template <typename P>
using Kernel = void (*)(P);

template <typename T, bool VEC>
Kernel<RouterParams> fwd_kernel(int g, int nc) {
  if (nc == 4) return router_kernel<T, VEC, 32, 4>;
  if (nc == 1) return g == 1 ? router_kernel<T, VEC, 1, 1> : router_kernel<T, VEC, 32, 1>;
  switch (g) {
    case 1: return router_kernel<T, VEC, 1, 2>;
    case 2: return router_kernel<T, VEC, 2, 2>;
    case 4: return router_kernel<T, VEC, 4, 2>;
    case 8: return router_kernel<T, VEC, 8, 2>;
    default: return router_kernel<T, VEC, 32, 2>;
  }
}
template <typename T, bool VEC>
Kernel<RouterBwdParams> bwd_kernel(int g, int nc) {
  if (nc == 4) return router_bwd_kernel<T, VEC, 32, 4>;
  if (nc == 2) return router_bwd_kernel<T, VEC, 32, 2>;
  switch (g) {
    case 1: return router_bwd_kernel<T, VEC, 1, 1>;
    case 2: return router_bwd_kernel<T, VEC, 2, 1>;
    case 4: return router_bwd_kernel<T, VEC, 4, 1>;
    case 8: return router_bwd_kernel<T, VEC, 8, 1>;
    case 16: return router_bwd_kernel<T, VEC, 16, 1>;
    default: return router_bwd_kernel<T, VEC, 32, 1>;
  }
}

bool vec_rows(const void* p, long long stride, int size, int rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (stride * size) % 16 == 0);
}

int pieces_for(int experts, int g) {
  const int nc = (experts + 8 * g - 1) / (8 * g);
  return nc <= 1 ? 1 : nc == 2 ? 2 : 4;
}

template <typename T>
cudaError_t fwd(const RouterParams& p, cudaStream_t s, int* launches) {
  const bool vec = p.experts % 8 == 0 && vec_rows(p.logits, p.stride, sizeof(T), p.tokens);
  const FwdShape f = fwd_shape(p.experts);
  const auto kernel = vec ? fwd_kernel<T, true>(f.g, f.nc) : fwd_kernel<T, false>(f.g, f.nc);
  const auto bytes = [&](int experts, int k) {
    return (static_cast<size_t>(WARPS + 1) * experts + WARPS * (32 / f.g) * (k + 1)) * 4;
  };
  const size_t smem = bytes(p.experts, p.k);
  const int places = 8 * f.g * f.nc;                   // the most experts of this kernel
  cudaError_t e;
  if ((e = allow_shared(kernel, smem, bytes(places, std::min(places, ROUTER_MAX_K)))) != cudaSuccess) return e;
  if ((e = launch_after(kernel, dim3(p.parts), dim3(THREADS), smem, s, p)) != cudaSuccess) return e;
  *launches = 1;
  if (p.parts == 1) return cudaSuccess;
  *launches = 2;
  return launch_after(router_finish_kernel, dim3(FINISH_CTAS), dim3(1024), 0, s, p, FINISH_CTAS);
}

template <typename T>
cudaError_t bwd(const RouterBwdParams& p, int sms, cudaStream_t s) {
  const bool vec = p.experts % 8 == 0 && vec_rows(p.logits, p.stride, sizeof(T), p.tokens) &&
                   vec_rows(p.dlogits, p.dstride, sizeof(T), p.tokens);
  const int g = lanes_for(p.experts), nc = pieces_for(p.experts, g);
  const auto kernel = vec ? bwd_kernel<T, true>(g, nc) : bwd_kernel<T, false>(g, nc);
  const size_t smem = static_cast<size_t>(THREADS) * 8 * nc * 4;
  const int per = WARPS * (32 / g);
  const int want = static_cast<int>((static_cast<long long>(p.tokens) + per - 1) / per), most = 2 * sms;
  const cudaError_t e = allow_shared(kernel, smem, smem);          // by the kernel alone
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(want < most ? want : most), dim3(THREADS), smem, s, p);
}

}  // namespace

// CTAs of the forward pass: as many as the SMs hold, with at least two tokens per group of lanes in
// each where there are enough of them (one CTA also finishes the sums without a second launch).
int router_parts(int tokens, int experts, int sms) {
  const FwdShape f = fwd_shape(experts);
  const long long per = WARPS * (32 / f.g) * 2, want = (tokens + per - 1) / per;
  const long long most = std::min<long long>(static_cast<long long>(f.ctas) * sms, ROUTER_MAX_PARTS);
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

cudaError_t launch_router(RouterParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 0;
  p.parts = router_parts(p.tokens, p.experts, sms);
  if (type == MB_F32) return fwd<float>(p, s, launches);
  if (type == MB_BF16) return fwd<__nv_bfloat16>(p, s, launches);
  return fwd<__half>(p, s, launches);
}

cudaError_t launch_router_backward(RouterBwdParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 1;
  if (type == MB_F32) return bwd<float>(p, sms, s);
  if (type == MB_BF16) return bwd<__nv_bfloat16>(p, sms, s);
  return bwd<__half>(p, sms, s);
}

}  // namespace mb
