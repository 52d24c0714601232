// What the layer norm's two directions share: sums over a row's threads, weight and bias in shared
// memory, and the rules by which the host picks how rows are accessed.
#pragma once

#include <algorithm>

#include "mb_block.h"
#include "mb_rows.cuh"
#include "muonbank.h"

namespace mb {

__device__ __forceinline__ void group_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sums over the threads of a row, N of them at once; every thread gets them, formed in the same
// order in each.  `part` has one entry per warp of the CTA; a group of more than one warp waits
// at its own barrier, and takes the two halves of `part` in turn (a half is written again only
// after the barrier behind the other half's use).
template <int N, int WARPS>
struct RowSums {
  float (*part)[WARPS][N];
  int tpr, warp, first_warp, barrier, parity;
  __device__ __forceinline__ RowSums(float (*smem)[WARPS][N], int tpr_, int group)
      : part(smem), tpr(tpr_), warp(threadIdx.x >> 5), first_warp(group * (tpr_ >> 5)), barrier(1 + group), parity(0) {}
  __device__ __forceinline__ void operator()(float (&s)[N]) {
    if (tpr <= 32) {
      for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], o);
      return;
    }
    const int lane = threadIdx.x & 31;
    int which;
    const float sum = warp_sums<N>(s, lane, &which);
    if ((lane & (32 / N - 1)) == 0) part[parity][warp][which] = sum;
    group_barrier(barrier, tpr);
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = 0.f;
    for (int u = 0; u < tpr >> 5; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] += part[parity][first_warp + u][k];
    parity ^= 1;
  }
};

// The same over a whole CTA, for the kernels that give it one row at a time.
__device__ __forceinline__ float cta_sum(float s, float* smem) {
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  __syncthreads();                         // the previous sum has been read
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (int i = 0; i < static_cast<int>(blockDim.x) >> 5; ++i) s += smem[i];
  return s;
}

// A weight or bias in shared memory, in fp32, so that threads read their pieces of it without bank
// conflicts: VEC and SCALAR as [piece][half][thread][4] (16-byte reads); SHIFT, where every row may
// start at another element of its first piece, as eight planes by the column's last three bits.
template <Access A, int NV>
struct Staged {
  static __host__ __device__ int floats(int tpr) { return A == Access::SHIFT ? 8 * (NV * tpr + 2) : NV * 8 * tpr; }
  template <typename T>
  static __device__ __forceinline__ void put(float* to, const void* p, bool f32, float otherwise, int cols, int tpr) {
    if constexpr (A == Access::SHIFT) {
      const int plane = NV * tpr + 2;
      for (int i = threadIdx.x; i < 8 * plane; i += blockDim.x) {
        const int r = i / plane, c = (i - r * plane - 1) * 8 + r;
        to[i] = c >= 0 && c < cols ? param<T>(p, f32, otherwise, c) : 0.f;
      }
    } else {
      for (int i = threadIdx.x; i < NV * tpr; i += blockDim.x) {     // piece i / tpr of thread i % tpr
        const int v = i / tpr, t = i - v * tpr;
        float2 f[4];
        param_pairs<T, A>(p, f32, otherwise, Place{cols, tpr, t, 0}, v, f);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4*>(to + (v * 8 + 4 * h) * tpr + t * 4) =
              make_float4(f[2 * h].x, f[2 * h].y, f[2 * h + 1].x, f[2 * h + 1].y);
      }
    }
  }
  static __device__ __forceinline__ void get(const float* from, const Place& p, int v, float2 (&f)[4]) {
    if constexpr (A == Access::SHIFT) {
      const int plane = NV * p.tpr + 2;
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = j - p.shift;                     // the column is 8 (v tpr + t) + d
        e[j] = from[(d & 7) * plane + v * p.tpr + p.t + 1 + (d >> 3)];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = make_float2(e[2 * j], e[2 * j + 1]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 x = *reinterpret_cast<const float4*>(from + (v * 8 + 4 * h) * p.tpr + p.t * 4);
        f[2 * h] = make_float2(x.x, x.y);
        f[2 * h + 1] = make_float2(x.z, x.w);
      }
    }
  }
};

// Sums over up to 32 warps' entries of N values; every lane gets them.  By exchanges, one entry per lane:
// a loop over the entries in every lane is slower from five of them on
// (the backward pass of 2^27 bf16 elements in rows of 8192, 16 entries: 135 us and not 148) and even below.
template <int N>
__device__ __forceinline__ void sums_of_warps(const float (*part)[N], int warps, int lane, float (&sums)[N]) {
  float s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = lane < warps ? part[lane][i] : 0.f;
  int which;
  const float sum = warp_sums<N>(s, lane, &which);
#pragma unroll
  for (int i = 0; i < N; ++i) sums[i] = __shfl_sync(0xFFFFFFFFu, sum, i * (32 / N));
}

// A chunk of 16 bytes as pairs, and back.
__device__ __forceinline__ void chunk_pairs(const uint4& c, float2 (&f)[2], float) {
  f[0] = make_float2(__uint_as_float(c.x), __uint_as_float(c.y));
  f[1] = make_float2(__uint_as_float(c.z), __uint_as_float(c.w));
}
template <typename T>
__device__ __forceinline__ void chunk_pairs(const uint4& c, float2 (&f)[4], T) {
  f[0] = unpack2(c.x, T());
  f[1] = unpack2(c.y, T());
  f[2] = unpack2(c.z, T());
  f[3] = unpack2(c.w, T());
}
__device__ __forceinline__ uint4 chunk_of(const float2 (&f)[2], float) {
  return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
}
template <typename T>
__device__ __forceinline__ uint4 chunk_of(const float2 (&f)[4], T) {
  return make_uint4(pack2(f[0].x, f[0].y, T()), pack2(f[1].x, f[1].y, T()), pack2(f[2].x, f[2].y, T()),
                    pack2(f[3].x, f[3].y, T()));
}

// ---------------------------------------------------------------- host side

inline bool aligned_rows(const void* p, long long stride, int size, long long rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (stride * size) % 16 == 0);
}
inline bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether row r of q starts as far from a 16-byte boundary as row r of p, for every r.
inline bool same_shift(const void* p, long long p_stride, const void* q, long long q_stride, int size, long long rows) {
  return ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) == 0 &&
         (rows <= 1 || (p_stride - q_stride) * size % 16 == 0);
}

inline int pow2_at_least(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

// Whether 16-byte accesses that start at each row's own boundary serve it (SHIFT): rows long enough
// that what such an access takes in beyond a row belongs to the next, and not the same row again.
inline bool shiftable(long long stride, int cols, long long rows) {
  return cols >= 16 && (rows <= 1 || stride >= cols);
}

inline int cta_count(long long rows, long long per_cta, int most) {
  const long long want = (rows + per_cta - 1) / per_cta;
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

}  // namespace mb
