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
// every head past them.
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

// One 16-byte access of N elements.
template <typename T>
struct Vec16 {
  static constexpr int N = 16 / sizeof(T);
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(u[i]);
      } else {
        const float2 a = unpack2(u[i], T());
        f[2 * i] = a.x;
        f[2 * i + 1] = a.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&f)[N]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) u[i] = __float_as_uint(f[i]);
      else u[i] = pack2(f[2 * i], f[2 * i + 1], T());
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// Where a token's heads start in q and k, and in their results.
struct TokenBase {
  long long src[2], dst[2];
};

// VEC: every access is 16 bytes; an item is two vectors of a split head (the pairs' first and
// second halves), one of an interleaved head, or one of the copied rest.  Otherwise an item is
// one pair or one copied element.
template <typename T, bool VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const RotaryParams p) {
  extern __shared__ float2 cs[];                     // [tile][pairs] cosine, sine; then the tile's TokenBases
  TokenBase* base = reinterpret_cast<TokenBase*>(cs + static_cast<size_t>(p.tile) * p.pairs);
  constexpr int N = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
  const long long token0 = static_cast<long long>(blockIdx.x) * p.tile;
  const long long left = p.all_tokens - token0;
  const int here = left < p.tile ? static_cast<int>(left) : p.tile;
  for (int e = threadIdx.x; e < here * p.pairs; e += THREADS) {
    const int tt = e / p.pairs, i = e - tt * p.pairs;
    const long long token = token0 + tt, b = token / p.tokens, at = token - b * p.tokens;
    int axis = 0;
    while (axis < p.axes - 1 && i >= p.section_end[axis]) ++axis;
    const float angle = __fmul_rn(position(p, axis * p.pos_a + b * p.pos_b + at * p.pos_t), p.inv_freq[i]);
    float sn, c;
    sincosf(angle, &sn, &c);
    cs[e] = make_float2(c, p.sign * sn);
  }
  for (int tt = threadIdx.x; tt < here; tt += THREADS) {
    const long long token = token0 + tt, b = token / p.tokens, at = token - b * p.tokens;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      base[tt].src[k] = b * p.x[k].src_b + at * p.x[k].src_t;
      base[tt].dst[k] = b * p.x[k].dst_b + at * p.x[k].dst_t;
    }
  }
  __syncthreads();
  // a thread keeps its place within a head and goes over (token, head) in steps of `slots`
  const int turned = VEC ? (INTERLEAVED ? 2 * p.pairs : p.pairs) / N : p.pairs;   // items with pairs
  const int per_head = turned + (p.dim - 2 * p.pairs) / N;
  const int heads = p.x[0].heads + p.x[1].heads;
  const int slots = per_head < THREADS ? THREADS / per_head : 1;
  const int slot = per_head < THREADS ? threadIdx.x / per_head : 0;
  const int first_item = per_head < THREADS ? threadIdx.x - slot * per_head : threadIdx.x;
  if (slot >= slots) return;
  const int step_t = slots / heads, step_h = slots - step_t * heads;
  for (int item = first_item; item < per_head; item += THREADS) {
    int tt = slot / heads, h = slot - tt * heads;
    while (tt < here) {
      const int k = h < p.x[0].heads ? 0 : 1;
      const int hk = h - (k ? p.x[0].heads : 0);
      const T* src = static_cast<const T*>(p.x[k].src) + base[tt].src[k] + hk * p.x[k].src_h;
      T* dst = static_cast<T*>(p.x[k].dst) + base[tt].dst[k] + hk * p.x[k].dst_h;
      const float2* a = cs + static_cast<size_t>(tt) * p.pairs;
      if (item >= turned) {
        const int e = 2 * p.pairs + (item - turned) * N;
        if constexpr (VEC) {
          Vec16<T> v;
          v.load(src + e);
          v.store(dst + e);
        } else {
          dst[e] = src[e];
        }
      } else if constexpr (VEC && INTERLEAVED) {
        Vec16<T> v;
        float f[N];
        v.load(src + item * N);
        v.get(f);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float2 r = a[item * (N / 2) + j];
          const float u = f[2 * j], w = f[2 * j + 1];
          f[2 * j] = u * r.x - w * r.y;
          f[2 * j + 1] = w * r.x + u * r.y;
        }
        v.set(f);
        v.store(dst + item * N);
      } else if constexpr (VEC) {
        Vec16<T> v0, v1;
        float f0[N], f1[N];
        v0.load(src + item * N);
        v1.load(src + p.pairs + item * N);
        v0.get(f0);
        v1.get(f1);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float2 r = a[item * N + j];
          const float u = f0[j], w = f1[j];
          f0[j] = u * r.x - w * r.y;
          f1[j] = w * r.x + u * r.y;
        }
        v0.set(f0);
        v1.set(f1);
        v0.store(dst + item * N);
        v1.store(dst + p.pairs + item * N);
      } else {
        const int i0 = INTERLEAVED ? 2 * item : item, i1 = INTERLEAVED ? 2 * item + 1 : item + p.pairs;
        const float2 r = a[item];
        const float u = to_float(src[i0]), w = to_float(src[i1]);
        dst[i0] = from_float<T>(u * r.x - w * r.y);
        dst[i1] = from_float<T>(w * r.x + u * r.y);
      }
      tt += step_t;
      h += step_h;
      if (h >= heads) {
        h -= heads;
        ++tt;
      }
    }
  }
}

// Whether every 16-byte access of the vector form is aligned.
bool vec_tensor(const RotaryTensor& x, int size) {
  if (x.heads == 0) return true;
  const long long strides = x.src_b | x.src_t | x.src_h | x.dst_b | x.dst_t | x.dst_h;
  return ((reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(x.dst)) & 15u) == 0 &&
         (strides * size) % 16 == 0;
}

template <typename T>
cudaError_t rotary(RotaryParams p, int sms, cudaStream_t s) {
  constexpr int N = 16 / sizeof(T);
  const bool vec = vec_tensor(p.x[0], sizeof(T)) && vec_tensor(p.x[1], sizeof(T)) &&
                   (p.interleaved ? 2 * p.pairs : p.pairs) % N == 0 && (p.dim - 2 * p.pairs) % N == 0;
  const int per_head = (vec ? (p.interleaved ? 2 * p.pairs : p.pairs) / N : p.pairs) +
                       (p.dim - 2 * p.pairs) / (vec ? N : 1);
  const int heads = p.x[0].heads + p.x[1].heads;
  // about one sine and cosine per thread, and at least one item; no more than fills the SMs
  long long tile = THREADS / p.pairs;
  const long long items = static_cast<long long>(heads) * per_head;
  if (tile * items < THREADS) tile = (THREADS + items - 1) / items;
  const long long most = ROTARY_MAX_PAIRS / p.pairs, spread = (p.all_tokens + sms - 1) / sms;
  if (tile > most) tile = most;
  if (tile > spread) tile = spread;
  if (tile < 1) tile = 1;
  p.tile = static_cast<int>(tile);
  const size_t smem = static_cast<size_t>(tile) * p.pairs * sizeof(float2) + static_cast<size_t>(tile) * sizeof(TokenBase);
  const unsigned grid = static_cast<unsigned>((p.all_tokens + tile - 1) / tile);
  auto kernel = vec ? (p.interleaved ? rotary_kernel<T, true, true> : rotary_kernel<T, true, false>)
                    : (p.interleaved ? rotary_kernel<T, false, true> : rotary_kernel<T, false, false>);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, THREADS, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(RotaryParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 1;
  if (type == MB_F32) return rotary<float>(p, sms, s);
  if (type == MB_BF16) return rotary<__nv_bfloat16>(p, sms, s);
  return rotary<__half>(p, sms, s);
}

}  // namespace mb
