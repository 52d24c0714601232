// Rotary positions with one or several axes on q and k, forward and inverse (the gradient).
//
// Pair i of a head's elements turns by t = positions[axis(i)] * inv_freq[i], the same angle for
// every head of q and k at that token:  u' = u cos t - v sin t,  v' = v cos t + u sin t.
// Elements past the pairs are copied.  The angle is one fp32 product, as a formula in 32 bits
// has it (an angle of thousands of radians is off by its own rounding, 2^-24 of it); sines
// and cosines are the full-range functions.
//
// The copy of the elements through the SMs is what bounds it.  A CTA takes a tile of tokens,
// makes the tile's sines and cosines once in shared memory, about one per thread, and streams
// every head past them.  64 x 1024 bf16 tokens of 24 heads of 64 take 62 us (6.5 TB/s), fp32 121 us
// (6.6 TB/s); pairs of adjacent elements 5.3 and 6.4 TB/s; heads of odd 16-bit lengths are
// moved by single elements, at 2.4 TB/s.
#include <algorithm>

#include "mb_block.h"
#include "mb_rows.cuh"
#include "muonbank.h"

namespace mb {
namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ float position(const RotaryParams& p, long long i) {
  if (p.pos_type == MB_I32) return static_cast<float>(static_cast<const int*>(p.pos)[i]);
  if (p.pos_type == MB_I64) return static_cast<float>(static_cast<const long long*>(p.pos)[i]);
  return static_cast<const float*>(p.pos)[i];
}

// One access of N elements: 2, 4, 8 or 16 bytes.
template <typename T, int N>
struct Run {
  static constexpr int BYTES = N * static_cast<int>(sizeof(T));
  uint32_t u[BYTES <= 4 ? 1 : BYTES / 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(u) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(u) = *reinterpret_cast<const uint2*>(p);
    else if constexpr (BYTES == 4) u[0] = *reinterpret_cast<const uint32_t*>(p);
    else u[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(u);
    else if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(u);
    else if constexpr (BYTES == 4) *reinterpret_cast<uint32_t*>(p) = u[0];
    else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(u[0]);
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = __uint_as_float(u[i]);
    } else if constexpr (N == 1) {
      f[0] = unpack2(u[0], T()).x;
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 a = unpack2(u[i], T());
        f[2 * i] = a.x;
        f[2 * i + 1] = a.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&f)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = __float_as_uint(f[i]);
    } else if constexpr (N == 1) {
      u[0] = pack2(f[0], 0.f, T());
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) u[i] = pack2(f[2 * i], f[2 * i + 1], T());
    }
  }
};

// Where a token's heads start in q and k and in their results, and its first axis' position.
struct TokenBase {
  long long src[2], dst[2], pos;
};

// Items that a thread loads before it works on them: single ones of 16-byte 16-bit runs, which
// leave room for all of an SM's threads (64x1024 tokens of 24 heads of 64: 65 us, four ahead 83),
// two of 16-byte fp32 runs, four of shorter ones.
template <typename T, int N>
constexpr int ITEMS_AHEAD = N * sizeof(T) < 16 ? 4 : sizeof(T) == 2 ? 1 : 2;

// Every access is of N elements.  An item is a run of N pairs of a split head (its first and its
// second halves), a run of an interleaved head (of N / 2 pairs, or of one for N = 1), or a run of the
// copied rest.  A thread loads AHEAD items before it works on them.
template <typename T, int N, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const RotaryParams p) {
  begin_after_previous();
  extern __shared__ float2 cs[];                     // [tile][pairs] cosine, sine; then the tile's TokenBases
  TokenBase* base = reinterpret_cast<TokenBase*>(cs + static_cast<size_t>(p.tile) * p.pairs);
  constexpr int AHEAD = ITEMS_AHEAD<T, N>;
  constexpr bool TWO = !INTERLEAVED || N == 1;         // an item with pairs is two runs
  const int token0 = static_cast<int>(blockIdx.x) * p.tile;      // tokens of the call < 2^31
  const int left = static_cast<int>(p.all_tokens) - token0;
  const int here = left < p.tile ? left : p.tile;
  for (int tt = threadIdx.x; tt < here; tt += THREADS) {
    const int b = (token0 + tt) / p.tokens, at = token0 + tt - b * p.tokens;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      base[tt].src[k] = b * p.x[k].src_b + at * p.x[k].src_t;
      base[tt].dst[k] = b * p.x[k].dst_b + at * p.x[k].dst_t;
    }
    base[tt].pos = b * p.pos_b + at * p.pos_t;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < here * p.pairs; e += THREADS) {
    const int tt = e / p.pairs, i = e - tt * p.pairs;
    int axis = 0;
    while (axis < p.axes - 1 && i >= p.section_end[axis]) ++axis;
    const float angle = __fmul_rn(position(p, axis * p.pos_a + base[tt].pos), p.inv_freq[i]);
    float sn, c;
    sincosf(angle, &sn, &c);
    cs[e] = make_float2(c, p.sign * sn);
  }
  __syncthreads();
  // a thread keeps its place within a head and goes over (token, head) in steps of `slots`
  const int turned = (TWO ? p.pairs : 2 * p.pairs) / N;          // items with pairs
  const int per_head = turned + (p.dim - 2 * p.pairs) / N;
  const int heads = p.x[0].heads + p.x[1].heads;
  const int slots = per_head < THREADS ? THREADS / per_head : 1;
  const int slot = per_head < THREADS ? threadIdx.x / per_head : 0;
  const int first_item = per_head < THREADS ? threadIdx.x - slot * per_head : threadIdx.x;
  if (slot >= slots) return;
  const int step_t = slots / heads, step_h = slots - step_t * heads;
  for (int item = first_item; item < per_head; item += THREADS) {
    const bool turn = item < turned;
    // where the item's runs start in its head, and its first pair
    const int e0 = !turn ? 2 * p.pairs + (item - turned) * N : N == 1 && INTERLEAVED ? 2 * item : item * N;
    const int e1 = N == 1 && INTERLEAVED ? e0 + 1 : e0 + p.pairs;
    const int pair = TWO ? item * N : item * (N / 2);
    int tt = slot / heads, h = slot - tt * heads;
    while (tt < here) {
      Run<T, N> v0[AHEAD], v1[AHEAD];
      T* dst[AHEAD];
      int at[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        at[i] = tt < here ? tt : -1;
        if (tt < here) {
          const int k = h < p.x[0].heads ? 0 : 1;
          const int hk = h - (k ? p.x[0].heads : 0);
          const T* src = static_cast<const T*>(p.x[k].src) + base[tt].src[k] + hk * p.x[k].src_h;
          dst[i] = static_cast<T*>(p.x[k].dst) + base[tt].dst[k] + hk * p.x[k].dst_h;
          v0[i].load(src + e0);
          if (TWO && turn) v1[i].load(src + e1);
          tt += step_t;
          h += step_h;
          if (h >= heads) {
            h -= heads;
            ++tt;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (at[i] < 0) break;
        if (turn) {
          const float2* a = cs + static_cast<size_t>(at[i]) * p.pairs + pair;
          float f0[N], f1[N];
          v0[i].get(f0);
          if constexpr (TWO) {
            v1[i].get(f1);
#pragma unroll
            for (int j = 0; j < N; ++j) {
              const float2 r = a[j];
              const float u = f0[j], w = f1[j];
              f0[j] = u * r.x - w * r.y;
              f1[j] = w * r.x + u * r.y;
            }
            v1[i].set(f1);
            v1[i].store(dst[i] + e1);
          } else {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
              const float2 r = a[j];
              const float u = f0[2 * j], w = f0[2 * j + 1];
              f0[2 * j] = u * r.x - w * r.y;
              f0[2 * j + 1] = w * r.x + u * r.y;
            }
          }
          v0[i].set(f0);
        }
        v0[i].store(dst[i] + e0);
      }
    }
  }
}

// The widest access (in bytes, a power of two) that every run's start and length allow.
template <typename T>
int access_bytes(const RotaryParams& p) {
  unsigned long long bits = 16;
  for (const RotaryTensor& x : p.x) {
    if (x.heads == 0) continue;
    bits |= reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(x.dst) |
            static_cast<unsigned long long>(x.src_b | x.src_t | x.src_h | x.dst_b | x.dst_t | x.dst_h) * sizeof(T);
  }
  bits |= static_cast<unsigned long long>((p.interleaved ? 2 * p.pairs : p.pairs) | (p.dim - 2 * p.pairs)) * sizeof(T);
  return static_cast<int>(bits & (~bits + 1));
}

template <typename T, int N>
cudaError_t rotary(RotaryParams p, int sms, cudaStream_t s) {
  const int turned = (!p.interleaved || N == 1 ? p.pairs : 2 * p.pairs) / N;
  const int per_head = turned + (p.dim - 2 * p.pairs) / N;
  const int heads = p.x[0].heads + p.x[1].heads;
  // about one sine and cosine per thread and at least one item; up to four times as many tokens if
  // that wastes less of the threads' last round; no more than fills the SMs
  const int slots = per_head < THREADS ? THREADS / per_head : 1;
  long long least = std::max(1, THREADS / p.pairs);
  if (least * heads < slots) least = (slots + heads - 1) / heads;
  const long long most = std::max(1, ROTARY_MAX_PAIRS / p.pairs), spread = (p.all_tokens + sms - 1) / sms;
  least = std::min(least, std::min(most, spread));
  long long tile = least;
  double best = 0;
  for (long long t = least; t <= std::min(4 * least, std::min(most, spread)); ++t) {
    const double rounds = static_cast<double>((t * heads + slots - 1) / slots), used = t * heads / (rounds * slots);
    if (used > best + 0.02) {
      best = used;
      tile = t;
    }
  }
  p.tile = static_cast<int>(tile);
  const size_t smem = static_cast<size_t>(tile) * p.pairs * sizeof(float2) + static_cast<size_t>(tile) * sizeof(TokenBase);
  const unsigned grid = static_cast<unsigned>((p.all_tokens + tile - 1) / tile);
  auto kernel = p.interleaved ? rotary_kernel<T, N, true> : rotary_kernel<T, N, false>;
  // a tile has at most ROTARY_MAX_PAIRS pairs and four times THREADS tokens
  const cudaError_t e =
      allow_shared(kernel, smem, ROTARY_MAX_PAIRS * sizeof(float2) + 4 * THREADS * sizeof(TokenBase));
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(grid), dim3(THREADS), smem, s, p);
}

template <typename T>
cudaError_t rotary_any(const RotaryParams& p, int sms, cudaStream_t s) {
  switch (access_bytes<T>(p) / static_cast<int>(sizeof(T))) {
    case 8: return rotary<T, 16 / static_cast<int>(sizeof(T))>(p, sms, s);
    case 4: return rotary<T, 4>(p, sms, s);
    case 2: return rotary<T, 2>(p, sms, s);
    default: return rotary<T, 1>(p, sms, s);
  }
}

}  // namespace

cudaError_t launch_rotary(RotaryParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 1;
  if (type == MB_F32) return rotary_any<float>(p, sms, s);
  if (type == MB_BF16) return rotary_any<__nv_bfloat16>(p, sms, s);
  return rotary_any<__half>(p, sms, s);
}

}  // namespace mb
