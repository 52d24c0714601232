// AdamW over a list of tensors (the ones that are in no bank) in one launch, moments in fp32 or in 8 bits.
//
// Per element, each operation rounded to fp32 on its own (no contraction), so that any program that does the
// same operations in the same order gets the same bits, and with them the same 8-bit codes:
//   m <- m b1 + g (1 - b1);   v <- v b2 + (g g) (1 - b2);   r = sqrt(v)
//   w <- w decay - (m / (r root + eps)) rate
// with decay = 1 - lr wd, rate = lr / (1 - b1^t), root = 1 / sqrt(1 - b2^t) formed in double.
//
// 8-bit moments: e4m3 codes of m and of r, the root of v (half of v's exponent range, and what the update
// divides by), each block of 256 elements with its own scale, the block's largest magnitude over 448.  A warp
// holds a block in registers, eight elements per lane, so that the two maxima are two warp reductions and every
// code is read and written once.  A positive r keeps at least the least positive code: a root that fell to zero
// would leave eps alone under the next step's m.
//
// Bound by memory: 26 bytes per element with bf16 weights, their low halves, bf16 gradients and fp32 moments,
// 14 with 8-bit ones.  The list of tensors travels in the launch's parameters, so that a call is one launch, needs
// no memory of its own and can be captured.
#include <cuda_fp8.h>

#include <cmath>

#include "mb_block.h"
#include "mb_device.cuh"
#include "mb_rows.cuh"
#include "muonbank.h"

namespace mb {
namespace {

constexpr int BLOCK = 256;              // elements of a warp's turn, and of a scale
// Small CTAs: 2 x 38633472 elements with 8-bit moments took 238 us in CTAs of 256 threads, 212 of 128, 186 of 64, 211 of 32 (24
// warps per SM each: 80 registers), since a CTA's registers are free again only when its last warp is done.
constexpr int THREADS = 64, WARPS = THREADS / 32, CTAS = 12;
constexpr float TOP = 448.f;            // the largest e4m3 number
constexpr float LEAST_SCALED = 0x1p-100f;   // a block whose largest magnitude is below this is held as zeros

struct AdamTensor {
  void* param;
  const void* grad;
  void *avg, *sq;
  uint16_t* mantissa;       // or null
  float *avg_scale, *sq_scale;
  long long n;
  float decay, rate;
  int first;                // its first CTA in the launch
  int position;             // in the call's list (the random bits' key)
  uint8_t param_type, grad_type, aligned;
};

// What a call's tensors share; also the first words of a device-scalar call's workspace, which {decay, rate} of every
// tensor follow.
struct AdamScalars {
  float b1, c1, b2, c2, root, eps;
  uint32_t key;
  float minus_zero;
};

template <int CAP>
struct AdamParams {
  AdamScalars s;
  const AdamScalars* dev;   // or null: use s and the tensors' decay and rate
  const float* grad_scale;  // or null
  int count, random;
  AdamTensor t[CAP];
};
constexpr int FEW = 32, MANY = 320;     // the launch copies the whole block: a short list takes a small one
static_assert(sizeof(AdamParams<MANY>) <= 32764, "kernel parameters");

// A hash of 32-bit words: multiplications by odd constants (2^32 over the golden ratio; the first fractional bits of the
// roots of 2 and 3) between shifted exclusive-ors.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x *= 0x9E3779B1u;
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// Two fp32 operations in one instruction, each rounded on its own.  A product is a fused one with -0 as its summand, which
// changes no value and comes from memory: packed products, explicit roundings or a constant -0 or not, were contracted
// with the sums that follow them.
__device__ __forceinline__ uint64_t bits_of(float2 v) {
  return static_cast<uint64_t>(__float_as_uint(v.y)) << 32 | __float_as_uint(v.x);
}
__device__ __forceinline__ float2 pair_of(uint64_t u) {
  return make_float2(__uint_as_float(static_cast<uint32_t>(u)), __uint_as_float(static_cast<uint32_t>(u >> 32)));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b, float minus_zero) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(bits_of(a)), "l"(bits_of(b)), "l"(bits_of(make_float2(minus_zero, minus_zero))));
  return pair_of(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)));
  return pair_of(d);
}

// ---------------------------------------------------------------- a lane's eight elements, of a type known at run time

struct Raw {
  uint4 a, b;
};

__device__ __forceinline__ Raw load_eight(const void* p, long long at, int type) {
  Raw r;
  if (type == MB_F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    r.a = q[0];
    r.b = q[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  }
  return r;
}

__device__ __forceinline__ void widen(const Raw& r, int type, float2 (&v)[4]) {
  const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  // (branches, the same for the warp: as a choice of values all three would be computed)
  if (type == MB_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = unpack2(u[i], __nv_bfloat16());
  } else if (type == MB_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = unpack2(u[i], __half());
  }
}

__device__ __forceinline__ float load_one(const void* p, long long at, int type) {
  if (type == MB_F32) return static_cast<const float*>(p)[at];
  if (type == MB_BF16) return to_float(static_cast<const __nv_bfloat16*>(p)[at]);
  return to_float(static_cast<const __half*>(p)[at]);
}

__device__ __forceinline__ void store_one(void* p, long long at, int type, float v) {
  if (type == MB_F32) static_cast<float*>(p)[at] = v;
  else if (type == MB_BF16) static_cast<__nv_bfloat16*>(p)[at] = from_float<__nv_bfloat16>(v);
  else static_cast<__half*>(p)[at] = from_float<__half>(v);
}

__device__ __forceinline__ void store_eight(void* p, long long at, int type, const float2 (&v)[4]) {
  if (type == MB_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    return;
  }
  uint32_t u[4];
  if (type == MB_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack2(v[i].x, v[i].y, __nv_bfloat16());
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack2(v[i].x, v[i].y, __half());
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(u[0], u[1], u[2], u[3]);
}

// ---------------------------------------------------------------- 8-bit moments

__device__ __forceinline__ float2 widen_codes(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t codes_of(float2 v) { return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3); }

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The largest magnitude of the warp's finite values.  The bits of non-negative floats are ordered as their values are, and
// those of infinities and NaN are above: only a warp that has one of them looks at each.
template <bool ROOT>
__device__ __forceinline__ float block_size(const float2 (&v)[4], bool& all_finite) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // (a root has no sign but NaN's, which is above all the same)
    if (ROOT) top = max(top, max(__float_as_uint(v[j].x), __float_as_uint(v[j].y)));
    else top = max(top, max(magnitude(v[j].x), magnitude(v[j].y)));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  all_finite = top < 0x7F800000u;
  if (!all_finite) {
    top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = magnitude(j & 1 ? v[j / 2].y : v[j / 2].x);
      top = max(top, a < 0x7F800000u ? a : 0u);
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  return __uint_as_float(top);
}

// The e4m3 number that q becomes with 16 random bits: a step of the number's exponent (20 dropped mantissa bits) times
// bits / 2^16 is added before the rest is dropped.  Below 2^-6, where the numbers are evenly spaced, the same is done
// one exponent up, 2^-6 higher.
__device__ __forceinline__ float round_at_random(float q, uint32_t bits16) {
  float a = fabsf(q);
  const bool low = a < 0x1p-6f;
  a = low ? __fadd_rn(a, 0x1p-6f) : a;
  a = __uint_as_float((__float_as_uint(a) + (bits16 << 4)) & 0xFFF00000u);
  a = fminf(low ? __fsub_rn(a, 0x1p-6f) : a, TOP);
  return isnan(q) ? q : copysignf(a, q);
}

// A block's values over its scale, as e4m3 numbers still in fp32 (rounded where `random`, else by codes_of); a value that is
// not finite becomes NaN, alone.  Returns the scale.
template <bool ROOT>
__device__ __forceinline__ float scale_block(const float2 (&v)[4], float2 (&q)[4], bool random, const uint32_t (&bits)[8]) {
  bool all_finite;
  const float size = block_size<ROOT>(v, all_finite);
  const bool some = size >= LEAST_SCALED;
  const float inv = some ? __fmul_rn(__frcp_rn(size), TOP) : 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = __fmul2_rn(v[j], both(inv));
  if (!all_finite) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[j].x = fabsf(q[j].x) < 480.f ? q[j].x : __uint_as_float(0x7FC00000u);
      q[j].y = fabsf(q[j].y) < 480.f ? q[j].y : __uint_as_float(0x7FC00000u);
    }
  }
  if (random) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[j].x = round_at_random(q[j].x, ROOT ? bits[2 * j] >> 16 : bits[2 * j] & 0xFFFFu);
      q[j].y = round_at_random(q[j].y, ROOT ? bits[2 * j + 1] >> 16 : bits[2 * j + 1] & 0xFFFFu);
    }
  }
  if (ROOT && some) {
    // (roots are never negative) the least code for what is positive below it: rare, so the lane's least is looked at first
    float least = TOP;
#pragma unroll
    for (int j = 0; j < 4; ++j) least = fminf(least, fminf(q[j].x, q[j].y));
    if (least < 0x1p-9f) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q[j].x = v[j].x > 0.f && q[j].x < 0x1p-9f ? 0x1p-9f : q[j].x;
        q[j].y = v[j].y > 0.f && q[j].y < 0x1p-9f ? 0x1p-9f : q[j].y;
      }
    }
  }
  return some ? __fmul_rn(size, 1.f / TOP) : 0.f;
}

// ---------------------------------------------------------------- the step

// A lane's eight elements: as pairs, the operations two at a time.
struct Lane {
  float2 g[4], w[4], m[4], v[4], r[4];
};

// The step of eight elements.  EIGHT: v comes as its root r.
template <bool EIGHT>
__device__ __forceinline__ void step_eight(Lane& e, const AdamScalars& s, float decay, float rate, const float* grad_scale) {
  const float z = s.minus_zero;
  if (grad_scale) {
    const float2 gs = both(*grad_scale);
#pragma unroll
    for (int j = 0; j < 4; ++j) e.g[j] = mul2(e.g[j], gs, z);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (EIGHT) e.v[j] = mul2(e.r[j], e.r[j], z);
    e.m[j] = add2(mul2(e.m[j], both(s.b1), z), mul2(e.g[j], both(s.c1), z));
    e.v[j] = add2(mul2(e.v[j], both(s.b2), z), mul2(mul2(e.g[j], e.g[j], z), both(s.c2), z));
    e.r[j] = make_float2(__fsqrt_rn(e.v[j].x), __fsqrt_rn(e.v[j].y));
    const float2 d = add2(mul2(e.r[j], both(s.root), z), both(s.eps));
    const float2 q = make_float2(__fdiv_rn(e.m[j].x, d.x), __fdiv_rn(e.m[j].y, d.y));
    e.w[j] = add2(mul2(e.w[j], both(decay), z), mul2(q, both(-rate), z));
  }
}

// The moments of a whole block as codes still in fp32 (m, v), their scales stored.  where: the lane's elements.
__device__ __forceinline__ void pack_moments(Lane& e, const AdamTensor& T, uint32_t key, bool random, long long at, int lane,
                                             uint32_t first, uint32_t apart) {
  uint32_t bits[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) bits[j] = 0;
  if (random) {
    const uint32_t k = mix(key + static_cast<uint32_t>(T.position)) + first;
#pragma unroll
    for (int j = 0; j < 8; ++j) bits[j] = mix(k + apart * j);
  }
  float2 q[4];
  const float ms = scale_block<false>(e.m, q, random, bits);
#pragma unroll
  for (int j = 0; j < 4; ++j) e.m[j] = q[j];
  const float vs = scale_block<true>(e.r, q, random, bits);
#pragma unroll
  for (int j = 0; j < 4; ++j) e.v[j] = q[j];
  if (lane == 0) {
    T.avg_scale[at / BLOCK] = ms;
    T.sq_scale[at / BLOCK] = vs;
  }
}

// What a lane loads of a whole aligned block: eight neighbouring elements in 16-byte accesses (8-byte ones of codes), held
// as they come, so that the next block's can be on their way under this block's arithmetic.
template <bool EIGHT>
struct Loaded {
  Raw g, p;
  uint4 low;
  Raw m, v;
  uint2 mc, vc;
  float ms, vs;
  __device__ __forceinline__ void load(const AdamTensor& T, long long at, int lane) {
    const long long first = at + 8 * lane;
    g = load_eight(T.grad, first, T.grad_type);
    p = load_eight(T.param, first, T.param_type);
    if (T.mantissa) low = *reinterpret_cast<const uint4*>(T.mantissa + first);
    if constexpr (EIGHT) {
      mc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.avg) + first);
      vc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.sq) + first);
      ms = T.avg_scale[at / BLOCK];
      vs = T.sq_scale[at / BLOCK];
    } else {
      m = load_eight(T.avg, first, MB_F32);
      v = load_eight(T.sq, first, MB_F32);
    }
  }
  __device__ __forceinline__ void get(const AdamTensor& T, Lane& e, float z) const {
    widen(g, T.grad_type, e.g);
    if (T.mantissa) {
      const uint32_t l[4] = {low.x, low.y, low.z, low.w}, h[4] = {p.a.x, p.a.y, p.a.z, p.a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        e.w[j] = make_float2(__uint_as_float(__byte_perm(l[j], h[j], 0x5410)), __uint_as_float(__byte_perm(l[j], h[j], 0x7632)));
    } else {
      widen(p, T.param_type, e.w);
    }
    if constexpr (EIGHT) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e.m[j] = mul2(widen_codes((j < 2 ? mc.x : mc.y) >> (16 * (j & 1)) & 0xFFFFu), both(ms), z);
        e.r[j] = mul2(widen_codes((j < 2 ? vc.x : vc.y) >> (16 * (j & 1)) & 0xFFFFu), both(vs), z);
      }
    } else {
      widen(m, MB_F32, e.m);
      widen(v, MB_F32, e.v);
    }
  }
};

template <bool EIGHT>
__device__ __forceinline__ void store_block(const Lane& e, const AdamTensor& T, long long at, int lane) {
  const long long first = at + 8 * lane;
  if (T.mantissa) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = __float_as_uint(e.w[j].x), b = __float_as_uint(e.w[j].y);
      hi[j] = __byte_perm(a, b, 0x7632);
      lo[j] = __byte_perm(a, b, 0x5410);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(T.param) + first) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(T.mantissa + first) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  } else {
    store_eight(T.param, first, T.param_type, e.w);
  }
  if constexpr (EIGHT) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.avg) + first) =
        make_uint2(codes_of(e.m[0]) | codes_of(e.m[1]) << 16, codes_of(e.m[2]) | codes_of(e.m[3]) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.sq) + first) =
        make_uint2(codes_of(e.v[0]) | codes_of(e.v[1]) << 16, codes_of(e.v[2]) | codes_of(e.v[3]) << 16);
  } else {
    store_eight(T.avg, first, MB_F32, e.m);
    store_eight(T.sq, first, MB_F32, e.v);
  }
}

// A block of a tensor that is not aligned, or a tensor's last: a lane has every 32nd element, zeros past the end.
template <bool EIGHT>
__device__ __forceinline__ void step_single(const AdamTensor& T, const AdamScalars& s, float decay, float rate,
                                            const float* grad_scale, bool random, long long at, int lane) {
  const long long first = at + lane;
  Lane e;
  float* const eg = &e.g[0].x;
  float* const ew = &e.w[0].x;
  float* const em = &e.m[0].x;
  float* const ev = &e.v[0].x;
  float* const er = &e.r[0].x;
  float ms = 0.f, vs = 0.f;
  if constexpr (EIGHT) {
    ms = T.avg_scale[at / BLOCK];
    vs = T.sq_scale[at / BLOCK];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long i = first + 32 * j;
    eg[j] = ew[j] = em[j] = ev[j] = er[j] = 0.f;
    if (i >= T.n) continue;
    eg[j] = load_one(T.grad, i, T.grad_type);
    // a bf16 weight with a low half is taken by its bits
    ew[j] = T.mantissa
                ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(T.param)[i]) << 16 | T.mantissa[i])
                : load_one(T.param, i, T.param_type);
    if constexpr (EIGHT) {
      em[j] = __fmul_rn(widen_codes(static_cast<const uint8_t*>(T.avg)[i]).x, ms);
      er[j] = __fmul_rn(widen_codes(static_cast<const uint8_t*>(T.sq)[i]).x, vs);
    } else {
      em[j] = static_cast<const float*>(T.avg)[i];
      ev[j] = static_cast<const float*>(T.sq)[i];
    }
  }
  step_eight<EIGHT>(e, s, decay, rate, grad_scale);
  if constexpr (EIGHT) {
    // past the end there is nothing whose size would count (NaN, where grad_scale is one)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (first + 32 * j >= T.n) em[j] = er[j] = 0.f;
    pack_moments(e, T, s.key, random, at, lane, static_cast<uint32_t>(first), 32u);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long i = first + 32 * j;
    if (i >= T.n) continue;
    if (T.mantissa) {
      static_cast<uint16_t*>(T.param)[i] = static_cast<uint16_t>(__float_as_uint(ew[j]) >> 16);
      T.mantissa[i] = static_cast<uint16_t>(__float_as_uint(ew[j]));
    } else {
      store_one(T.param, i, T.param_type, ew[j]);
    }
    if constexpr (EIGHT) {
      static_cast<uint8_t*>(T.avg)[i] = static_cast<uint8_t>(codes_of(make_float2(em[j], 0.f)));
      static_cast<uint8_t*>(T.sq)[i] = static_cast<uint8_t>(codes_of(make_float2(ev[j], 0.f)));
    } else {
      static_cast<float*>(T.avg)[i] = em[j];
      static_cast<float*>(T.sq)[i] = ev[j];
    }
  }
}

// Blocks of 256 elements that a warp takes in turn, the next one's loads under this one's arithmetic: 8-bit moments 186 us with
// four or eight, 199 with two; fp32 288 with two, 292 with four, 296 with eight.
template <bool EIGHT>
constexpr int CHUNK = WARPS * (EIGHT ? 4 : 2) * BLOCK;

template <int CAP, bool EIGHT>
__global__ void __launch_bounds__(THREADS, CTAS) adamw_kernel(const __grid_constant__ AdamParams<CAP> p) {
  begin_after_previous();
  int i = 0, end = p.count;
  while (end - i > 1) {
    const int mid = (i + end) >> 1;
    if (p.t[mid].first <= static_cast<int>(blockIdx.x)) i = mid;
    else end = mid;
  }
  const AdamTensor& T = p.t[i];
  const AdamScalars s = p.dev ? *p.dev : p.s;
  float decay = T.decay, rate = T.rate;
  if (p.dev) {
    const float* each = reinterpret_cast<const float*>(p.dev + 1) + 2 * T.position;
    decay = each[0];
    rate = each[1];
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long at = static_cast<long long>(blockIdx.x - T.first) * CHUNK<EIGHT> + warp * BLOCK;
  const long long stop = min(static_cast<long long>(blockIdx.x - T.first + 1) * CHUNK<EIGHT>, T.n);
  if (T.aligned) {
    Loaded<EIGHT> next;
    if (at + BLOCK <= stop) next.load(T, at, lane);
    for (; at + BLOCK <= stop; at += WARPS * BLOCK) {
      Lane e;
      next.get(T, e, s.minus_zero);
      if (at + (WARPS + 1) * BLOCK <= stop) next.load(T, at + WARPS * BLOCK, lane);
      step_eight<EIGHT>(e, s, decay, rate, p.grad_scale);
      if constexpr (EIGHT) pack_moments(e, T, s.key, p.random, at, lane, static_cast<uint32_t>(at) + 8 * lane, 1u);
      store_block<EIGHT>(e, T, at, lane);
    }
  }
  for (; at < stop; at += WARPS * BLOCK) step_single<EIGHT>(T, s, decay, rate, p.grad_scale, p.random, at, lane);
}

// ---------------------------------------------------------------- scalars

// b1^t and the like in double, as the host forms them for a call by value.
struct Derived {
  AdamScalars s;
  double rate_per_lr;      // 1 / (1 - b1^t), as a divisor: lr / this
};

__host__ __device__ inline double product(double a, double b) {
#ifdef __CUDA_ARCH__
  return __dmul_rn(a, b);
#else
  volatile double p = a * b;    // not contracted with what follows
  return p;
#endif
}

__host__ __device__ inline Derived derive(double beta1, double beta2, double eps, double step, uint32_t seed) {
  Derived d{};
  d.s.b1 = static_cast<float>(beta1);
  d.s.c1 = static_cast<float>(1.0 - beta1);
  d.s.b2 = static_cast<float>(beta2);
  d.s.c2 = static_cast<float>(1.0 - beta2);
  d.s.root = static_cast<float>(1.0 / sqrt(1.0 - pow(beta2, step)));
  d.s.eps = static_cast<float>(eps);
  d.s.minus_zero = -0.f;
  d.s.key = mix(mix(seed) + static_cast<uint32_t>(static_cast<unsigned long long>(step)));
  d.rate_per_lr = 1.0 - pow(beta1, step);
  return d;
}

__host__ __device__ inline void derive_each(double lr, double wd, float lr_mul, float wd_mul, double rate_per_lr, float* decay,
                                            float* rate) {
  const double l = product(lr, lr_mul);
  *decay = static_cast<float>(1.0 - product(l, product(wd, wd_mul)));
  *rate = static_cast<float>(l / rate_per_lr);
}

__host__ __device__ inline bool good_scalars(double lr, double wd, double beta1, double beta2, double eps, double step) {
  // (a comparison with NaN is false)
  return fabs(lr) < 1e30 && fabs(wd) < 1e30 && beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1 && eps >= 0 && eps < 1e30 &&
         step >= 1 && step <= 9007199254740992.0;
}

struct ScalarTensors {
  const double* src;       // {lr, wd, beta1, beta2, eps, step}
  AdamScalars* out;
  uint32_t seed;
  int begin, count;        // of the call's tensors, in this launch
  int* status;
  float lr_mul[512], wd_mul[512];
};

__global__ void adamw_scalars_kernel(const __grid_constant__ ScalarTensors p) {
  begin_after_previous();
  const double lr = p.src[0], wd = p.src[1], beta1 = p.src[2], beta2 = p.src[3], eps = p.src[4], step = p.src[5];
  const Derived d = derive(beta1, beta2, eps, step, p.seed);
  if (threadIdx.x == 0) {
    if (!good_scalars(lr, wd, beta1, beta2, eps, step)) latch_status(p.status, DEV_BAD_SCALAR);
    if (p.begin == 0) *p.out = d.s;
  }
  float* each = reinterpret_cast<float*>(p.out + 1) + 2 * p.begin;
  for (int i = threadIdx.x; i < p.count; i += blockDim.x)
    derive_each(lr, wd, p.lr_mul[i], p.wd_mul[i], d.rate_per_lr, &each[2 * i], &each[2 * i + 1]);
}

// ---------------------------------------------------------------- checks and launches

#define MB_TRY(expr)            \
  do {                          \
    int r_ = (expr);            \
    if (r_ != MB_OK) return r_; \
  } while (0)

bool float_type(int type) { return type == MB_F32 || type == MB_BF16 || type == MB_F16; }
int type_size(int type) { return type == MB_F32 ? 4 : 2; }

int check_pointer(const void* p, int size) {
  if (!p) return MB_ERR_NULL;
  return reinterpret_cast<uintptr_t>(p) % size == 0 ? MB_OK : MB_ERR_ALIGN;
}

int check_tensor(const mb_adamw_tensor& t) {
  if (t.n < 0 || t.n > (1ll << 40)) return MB_ERR_SHAPE;
  if (!float_type(t.param_type) || !float_type(t.grad_type)) return MB_ERR_ARG;
  if (t.state_type != MB_F32 && t.state_type != MB_E4M3) return MB_ERR_ARG;
  if (t.mantissa && t.param_type != MB_BF16) return MB_ERR_ARG;
  if (!std::isfinite(t.lr_mul) || !std::isfinite(t.wd_mul)) return MB_ERR_ARG;
  if (t.n == 0) return MB_OK;
  MB_TRY(check_pointer(t.param, type_size(t.param_type)));
  MB_TRY(check_pointer(t.grad, type_size(t.grad_type)));
  const int state = t.state_type == MB_F32 ? 4 : 1;
  MB_TRY(check_pointer(t.exp_avg, state));
  MB_TRY(check_pointer(t.exp_avg_sq, state));
  if (t.mantissa) MB_TRY(check_pointer(t.mantissa, 2));
  if (t.state_type == MB_E4M3) {
    MB_TRY(check_pointer(t.avg_scale, 4));
    MB_TRY(check_pointer(t.sq_scale, 4));
  }
  return MB_OK;
}

bool at_16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool at_8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The launches of the list's tensors with one kind of moments: one, unless the list is longer than a launch's parameters
// or its CTAs are more than a grid has.
template <int CAP, bool EIGHT>
cudaError_t launch_kind(const mb_adamw_tensor* list, int n, const AdamScalars& s, double lr, double wd, double rate_per_lr,
                        const AdamScalars* dev, const float* grad_scale, bool random, cudaStream_t st, int* launches) {
  AdamParams<CAP> p;
  p.s = s;
  p.dev = dev;
  p.grad_scale = grad_scale;
  p.random = random;
  p.count = 0;
  long long blocks = 0;
  auto launch = [&]() {
    if (p.count == 0) return cudaSuccess;
    ++*launches;
    const cudaError_t e = launch_after(adamw_kernel<CAP, EIGHT>, dim3(static_cast<unsigned>(blocks)), dim3(THREADS), 0, st, p);
    p.count = 0;
    blocks = 0;
    return e;
  };
  for (int i = 0; i < n; ++i) {
    const mb_adamw_tensor& t = list[i];
    if (t.n == 0 || (t.state_type == MB_E4M3) != EIGHT) continue;
    const long long need = (t.n + CHUNK<EIGHT> - 1) / CHUNK<EIGHT>;
    if (p.count == CAP || blocks + need > (1ll << 30)) {
      const cudaError_t e = launch();
      if (e != cudaSuccess) return e;
    }
    AdamTensor& a = p.t[p.count++];
    a.param = t.param;
    a.grad = t.grad;
    a.avg = t.exp_avg;
    a.sq = t.exp_avg_sq;
    a.mantissa = t.mantissa;
    a.avg_scale = t.avg_scale;
    a.sq_scale = t.sq_scale;
    a.n = t.n;
    a.decay = a.rate = 0.f;
    if (!dev) derive_each(lr, wd, t.lr_mul, t.wd_mul, rate_per_lr, &a.decay, &a.rate);
    a.first = static_cast<int>(blocks);
    a.position = i;
    a.param_type = static_cast<uint8_t>(t.param_type);
    a.grad_type = static_cast<uint8_t>(t.grad_type);
    a.aligned = at_16(t.param) && at_16(t.grad) && at_16(t.mantissa) &&
                (EIGHT ? at_8(t.exp_avg) && at_8(t.exp_avg_sq) : at_16(t.exp_avg) && at_16(t.exp_avg_sq));
    blocks += need;
  }
  return launch();
}

int run(const mb_adamw_tensor* list, int n, const AdamScalars& s, double lr, double wd, double rate_per_lr,
        const AdamScalars* dev, const float* grad_scale, bool random, cudaStream_t st, int launches) {
  int wide = 0, narrow = 0;
  for (int i = 0; i < n; ++i)
    if (list[i].n > 0) ++(list[i].state_type == MB_E4M3 ? narrow : wide);
  cudaError_t e = cudaSuccess;
  if (wide > 0)
    e = (wide <= FEW ? launch_kind<FEW, false> : launch_kind<MANY, false>)(list, n, s, lr, wd, rate_per_lr, dev, grad_scale,
                                                                           random, st, &launches);
  if (e == cudaSuccess && narrow > 0)
    e = (narrow <= FEW ? launch_kind<FEW, true> : launch_kind<MANY, true>)(list, n, s, lr, wd, rate_per_lr, dev, grad_scale,
                                                                           random, st, &launches);
  if (e != cudaSuccess) return api_cuda_fail(e);
  api_launched(MB_MARK_ADAMW, launches, st);
  return MB_OK;
}

int check_list(const mb_adamw_tensor* list, int n, const float* grad_scale) {
  if (n < 0 || n > MB_ADAMW_MAX_TENSORS) return MB_ERR_TOO_MANY;
  if (n > 0 && !list) return MB_ERR_NULL;
  for (int i = 0; i < n; ++i) MB_TRY(check_tensor(list[i]));
  return grad_scale ? check_pointer(grad_scale, 4) : MB_OK;
}

}  // namespace
}  // namespace mb

using namespace mb;

extern "C" {

int adamw_multi_step(const mb_adamw_tensor* tensors, int n_tensors, double lr, double wd, double beta1, double beta2,
                     double eps, int64_t step, const float* grad_scale, int stochastic, uint32_t seed, void* cuda_stream) {
  MB_TRY(check_list(tensors, n_tensors, grad_scale));
  if (!good_scalars(lr, wd, beta1, beta2, eps, static_cast<double>(step))) return MB_ERR_ARG;
  if (n_tensors == 0) return MB_OK;
  int sms = 0;
  MB_TRY(api_device_sms(&sms));
  const Derived d = derive(beta1, beta2, eps, static_cast<double>(step), seed);
  return run(tensors, n_tensors, d.s, lr, wd, d.rate_per_lr, nullptr, grad_scale, stochastic != 0,
             static_cast<cudaStream_t>(cuda_stream), 0);
}

int adamw_multi_step_dev_workspace_bytes(int n_tensors, size_t* out_bytes) {
  if (!out_bytes) return MB_ERR_NULL;
  if (n_tensors < 0 || n_tensors > MB_ADAMW_MAX_TENSORS) return MB_ERR_TOO_MANY;
  *out_bytes = sizeof(AdamScalars) + static_cast<size_t>(n_tensors) * 2 * sizeof(float);
  return MB_OK;
}

int adamw_multi_step_dev(const mb_adamw_tensor* tensors, int n_tensors, const double* scalars_dev, const float* grad_scale,
                         int stochastic, uint32_t seed, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  MB_TRY(check_list(tensors, n_tensors, grad_scale));
  MB_TRY(check_pointer(scalars_dev, 8));
  size_t need = 0;
  MB_TRY(adamw_multi_step_dev_workspace_bytes(n_tensors, &need));
  if (!workspace || workspace_bytes < need) return MB_ERR_WORKSPACE;
  if (!at_16(workspace)) return MB_ERR_ALIGN;
  if (n_tensors == 0) return MB_OK;
  int* status = nullptr;
  MB_TRY(api_device_status(&status));
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  AdamScalars* out = static_cast<AdamScalars*>(workspace);
  int launches = 0;
  for (int begin = 0; begin < n_tensors; begin += 512, ++launches) {
    ScalarTensors p;
    p.src = scalars_dev;
    p.out = out;
    p.seed = seed;
    p.begin = begin;
    p.count = n_tensors - begin < 512 ? n_tensors - begin : 512;
    p.status = status;
    for (int i = 0; i < p.count; ++i) {
      p.lr_mul[i] = tensors[begin + i].lr_mul;
      p.wd_mul[i] = tensors[begin + i].wd_mul;
    }
    const cudaError_t e = launch_after(adamw_scalars_kernel, dim3(1), dim3(256), 0, st, p);
    if (e != cudaSuccess) return api_cuda_fail(e);
  }
  return run(tensors, n_tensors, AdamScalars{}, 0.0, 0.0, 1.0, out, grad_scale, stochastic != 0, st, launches);
}

}  // extern "C"
