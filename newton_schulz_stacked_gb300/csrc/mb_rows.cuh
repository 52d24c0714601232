// What the block operators (layer norm, rotary, router) share: the element types, a thread's
// eight elements of a row, and sums over the threads of a row.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace mb {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
// -inf as Eight::fill takes it.
__device__ __forceinline__ uint32_t minus_inf_bits(float) { return 0xFF800000u; }
__device__ __forceinline__ uint32_t minus_inf_bits(__nv_bfloat16) { return 0xFF80FF80u; }
__device__ __forceinline__ uint32_t minus_inf_bits(__half) { return 0xFC00FC00u; }

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// Two neighbouring 16-bit values of one 32-bit word (the low half is the first).
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight consecutive elements at a 16-byte boundary, as loaded (one 16-byte access for the
// 16-bit types, two for fp32).
template <typename T>
struct Eight {
  static constexpr int WORDS = sizeof(T) / 2;   // 16-byte words
  uint4 w[WORDS];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() { fill(0); }
  // Every element as the 32-bit pattern `u` holds it (a pair of 16-bit elements, or one of fp32).
  __device__ __forceinline__ void fill(uint32_t u) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = make_uint4(u, u, u, u);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(u[i], T());
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(w);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = pack2(v[2 * i], v[2 * i + 1], T());
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
};

// How the threads of a row take its elements, in pieces of eight:
//   VEC     neighbouring elements in 16-byte accesses: rows start at 16-byte boundaries and hold a
//           multiple of eight elements;
//   SHIFT   the same accesses for rows that start anywhere: pieces start at the row's 16-byte
//           boundaries, `shift` elements before it, and the first and last hold less;
//   SCALAR  single elements, one per thread in turn.
enum class Access { SCALAR, VEC, SHIFT };

// A thread's place in a row of `cols` elements that `tpr` threads hold together.
struct Place {
  int cols, tpr, t, shift;
};

// Elements from the last 16-byte boundary to p.
template <typename T>
__device__ __forceinline__ int shift_of(const T* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / static_cast<int>(sizeof(T));
}

// Piece v of a thread's share of a row: its eight elements as loaded, at the columns col(v, j).
// What lies outside the row reads as zero.
template <typename T, Access A>
struct Piece;

template <typename T>
struct Piece<T, Access::VEC> {
  Eight<T> e;
  static __device__ __forceinline__ int col(const Place& p, int v, int j) { return (v * p.tpr + p.t) * 8 + j; }
  static __device__ __forceinline__ bool in(const Place& p, int v, int) { return col(p, v, 0) < p.cols; }
  __device__ __forceinline__ void load(const T* row, const Place& p, int v, bool on, bool) {
    if (on && in(p, v, 0)) e.load(row + col(p, v, 0));
    else e.zero();
  }
  __device__ __forceinline__ void get(const Place&, int, float (&f)[8]) const { e.get(f); }
  static __device__ __forceinline__ void store(T* row, const Place& p, int v, const float (&f)[8]) {
    if (in(p, v, 0)) {
      Eight<T> o;
      o.set(f);
      o.store(row + col(p, v, 0));
    }
  }
};

template <typename T>
struct Piece<T, Access::SHIFT> {
  Eight<T> e;
  static __device__ __forceinline__ int col(const Place& p, int v, int j) {
    return (v * p.tpr + p.t) * 8 - p.shift + j;
  }
  static __device__ __forceinline__ bool in(const Place& p, int v, int j) {
    const int c = col(p, v, j);
    return c >= 0 && c < p.cols;
  }
  // The first and last piece take in neighbours of the row, which get() drops (another thread may
  // be writing over those meanwhile); `edge`: the first or last row, beyond which nothing may be
  // read, so its own elements are picked one by one.
  __device__ __forceinline__ void load(const T* row, const Place& p, int v, bool on, bool edge) {
    const int c = col(p, v, 0);
    const bool some = on && c + 8 > 0 && c < p.cols, whole = c >= 0 && c + 8 <= p.cols;
    if (some && (whole || !edge)) {
      e.load(row + c);
    } else if (some) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = in(p, v, j) ? to_float(row[c + j]) : 0.f;
      e.set(f);
    } else {
      e.zero();
    }
  }
  __device__ __forceinline__ void get(const Place& p, int v, float (&f)[8]) const {
    e.get(f);
    const int c = col(p, v, 0);
    if (c < 0 || c + 8 > p.cols) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!in(p, v, j)) f[j] = 0.f;
    }
  }
  static __device__ __forceinline__ void store(T* row, const Place& p, int v, const float (&f)[8]) {
    const int c = col(p, v, 0);
    if (c >= 0 && c + 8 <= p.cols) {
      Eight<T> o;
      o.set(f);
      o.store(row + c);
    } else if (c + 8 > 0 && c < p.cols) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (in(p, v, j)) row[c + j] = from_float<T>(f[j]);
    }
  }
};

template <typename T>
struct Piece<T, Access::SCALAR> {
  T e_[8];             // converted when they are used: a conversion here would wait for the load
  static __device__ __forceinline__ int col(const Place& p, int v, int j) { return (v * 8 + j) * p.tpr + p.t; }
  static __device__ __forceinline__ bool in(const Place& p, int v, int j) { return col(p, v, j) < p.cols; }
  __device__ __forceinline__ void load(const T* row, const Place& p, int v, bool on, bool) {
#pragma unroll
    for (int j = 0; j < 8; ++j) e_[j] = on && in(p, v, j) ? row[col(p, v, j)] : from_float<T>(0.f);
  }
  __device__ __forceinline__ void get(const Place&, int, float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = to_float(e_[j]);
  }
  static __device__ __forceinline__ void store(T* row, const Place& p, int v, const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (in(p, v, j)) row[col(p, v, j)] = from_float<T>(f[j]);
  }
};

// A piece as four pairs, for the packed fp32 instructions (two operations per issue).
template <typename P>
__device__ __forceinline__ void get_pairs(const P& x, const Place& p, int v, float2 (&f)[4]) {
  float e[8];
  x.get(p, v, e);
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = make_float2(e[2 * j], e[2 * j + 1]);
}
template <typename P, typename T>
__device__ __forceinline__ void store_pairs(T* row, const Place& p, int v, const float2 (&f)[4]) {
  const float o[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
  P::store(row, p, v, o);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Element c of a parameter vector (weight or bias) in fp32 or in the activations' type T; null
// reads as `otherwise`.
template <typename T>
__device__ __forceinline__ float param(const void* p, bool f32, float otherwise, int c) {
  if (!p) return otherwise;
  return f32 ? static_cast<const float*>(p)[c] : to_float(static_cast<const T*>(p)[c]);
}
// ... and a thread's piece of it.
template <typename T, Access A>
__device__ __forceinline__ void param_pairs(const void* p, bool f32, float otherwise, const Place& at, int v,
                                            float2 (&f)[4]) {
  float e[8];
  if (A == Access::VEC && p) {
    if (f32) {
      Piece<float, Access::VEC> w;
      w.load(static_cast<const float*>(p), at, v, true, false);
      w.get(at, v, e);
    } else {
      Piece<T, Access::VEC> w;
      w.load(static_cast<const T*>(p), at, v, true, false);
      w.get(at, v, e);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      e[j] = Piece<T, A>::in(at, v, j) ? param<T>(p, f32, otherwise, Piece<T, A>::col(at, v, j)) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = make_float2(e[2 * j], e[2 * j + 1]);
}

// Sum over the aligned group of `width` lanes (a power of two); every lane gets it.
__device__ __forceinline__ float group_sum(float x, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// Sums of N values (1, 2, 4 or 8) over a warp, one of them per lane: the halves of the lanes that
// split at 16, 8, ... keep half of the values each, so N values cost N - 1 exchanges and then
// five less log2(N), not 5 N.  Returns the sum of value *which.
template <int N>
__device__ __forceinline__ float warp_sums(float (&s)[N], int lane, int* which) {
  int k = 0, o = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? s[n + i] : s[i], give = up ? s[i] : s[n + i];
      s[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
    }
    k += up ? n : 0;
  }
#pragma unroll
  for (; o > 0; o >>= 1) s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], o);
  *which = k;
  return s[0];
}

// Asynchronous copies of 16 bytes to shared memory by single threads, in groups that complete in order;
// copies_wait<N> waits for all but the thread's last N groups.
__device__ __forceinline__ void copy_16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from)
               : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The begin of a kernel launched with launch_after: its CTAs may be on their SMs before the kernel
// ahead of it in the stream has ended, and wait here until that one's writes are visible; then the
// next such kernel may do the same.  A launch costs 1 to 2 us less of the stream's time so.
__device__ __forceinline__ void begin_after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace mb
