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
constexpr int THREADS = 256, WARPS = THREADS / 32;
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
  uint32_t pad;
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

__device__ __forceinline__ void widen(const Raw& r, int type, float (&v)[8]) {
  const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (type == MB_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
  } else if (type == MB_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(u[i], __nv_bfloat16());
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(u[i], __half());
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
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

__device__ __forceinline__ void store_eight(void* p, long long at, int type, const float (&v)[8]) {
  if (type == MB_F32) {
    uint4* q = reinterpret_cast<uint4*>(static_cast<float*>(p) + at);
    q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    return;
  }
  uint32_t u[4];
  if (type == MB_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack2(v[2 * i], v[2 * i + 1], __nv_bfloat16());
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack2(v[2 * i], v[2 * i + 1], __half());
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(u[0], u[1], u[2], u[3]);
}

// ---------------------------------------------------------------- 8-bit moments

__device__ __forceinline__ float2 widen_codes(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The largest magnitude of the warp's finite values.  The bits of non-negative floats are ordered as their values are.
__device__ __forceinline__ float block_size(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    top = max(top, a < 0x7F800000u ? a : 0u);
  }
  return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
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

// A block's values over its scale, as e4m3 numbers still in fp32; a value that is not finite becomes NaN, alone.  Returns
// the scale.
template <bool ROOT>
__device__ __forceinline__ float scale_block(const float (&v)[8], float (&q)[8], bool random, const uint32_t (&bits)[8]) {
  const float size = block_size(v);
  const bool some = size >= LEAST_SCALED;
  const float inv = some ? __fmul_rn(__frcp_rn(size), TOP) : 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float x = __fmul_rn(v[j], inv);
    x = fabsf(x) < 480.f ? x : __uint_as_float(0x7FC00000u);
    if (random) x = round_at_random(x, ROOT ? bits[j] >> 16 : bits[j] & 0xFFFFu);
    if (ROOT && some && v[j] > 0.f) x = x < 0x1p-9f ? 0x1p-9f : x;
    q[j] = x;
  }
  return some ? __fmul_rn(size, 1.f / TOP) : 0.f;
}

// ---------------------------------------------------------------- the step

__device__ __forceinline__ float step_one(float g, float& m, float& v, float& r, float w, const AdamScalars& s, float decay,
                                          float rate) {
  m = __fadd_rn(__fmul_rn(m, s.b1), __fmul_rn(g, s.c1));
  v = __fadd_rn(__fmul_rn(v, s.b2), __fmul_rn(__fmul_rn(g, g), s.c2));
  r = __fsqrt_rn(v);
  const float d = __fadd_rn(__fmul_rn(r, s.root), s.eps);
  return __fsub_rn(__fmul_rn(w, decay), __fmul_rn(__fdiv_rn(m, d), rate));
}

// One block of 256 elements from `at` on, by one warp.  VEC: eight neighbouring elements to a lane in 16-byte accesses
// (8-byte ones of codes); else every 32nd element, what lies past the end as zeros.
template <bool EIGHT, bool VEC>
__device__ __forceinline__ void step_block(const AdamTensor& T, const AdamScalars& s, float decay, float rate,
                                           const float* grad_scale, bool random, long long at, int lane) {
  const int pt = T.param_type, gt = T.grad_type;
  float g[8], w[8], m[8], v[8], r[8];
  long long where[8];
  bool in[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    where[j] = VEC ? at + 8 * lane + j : at + 32 * j + lane;
    in[j] = VEC || where[j] < T.n;
  }
  if constexpr (VEC) {
    const long long first = at + 8 * lane;
    const Raw gr = load_eight(T.grad, first, gt), pr = load_eight(T.param, first, pt);
    uint4 low = make_uint4(0, 0, 0, 0);
    if (T.mantissa) low = *reinterpret_cast<const uint4*>(T.mantissa + first);
    if constexpr (EIGHT) {
      const uint2 mc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.avg) + first);
      const uint2 vc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.sq) + first);
      const float ms = T.avg_scale[at / BLOCK], vs = T.sq_scale[at / BLOCK];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = widen_codes((j < 2 ? mc.x : mc.y) >> (16 * (j & 1)) & 0xFFFFu);
        const float2 b = widen_codes((j < 2 ? vc.x : vc.y) >> (16 * (j & 1)) & 0xFFFFu);
        m[2 * j] = __fmul_rn(a.x, ms);
        m[2 * j + 1] = __fmul_rn(a.y, ms);
        r[2 * j] = __fmul_rn(b.x, vs);
        r[2 * j + 1] = __fmul_rn(b.y, vs);
      }
    } else {
      const Raw mr = load_eight(T.avg, first, MB_F32), vr = load_eight(T.sq, first, MB_F32);
      widen(mr, MB_F32, m);
      widen(vr, MB_F32, v);
    }
    widen(gr, gt, g);
    widen(pr, pt, w);
    if (T.mantissa) {
      const uint32_t l[4] = {low.x, low.y, low.z, low.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[2 * j] = __uint_as_float(__float_as_uint(w[2 * j]) | (l[j] & 0xFFFFu));
        w[2 * j + 1] = __uint_as_float(__float_as_uint(w[2 * j + 1]) | (l[j] >> 16));
      }
    }
  } else {
    float ms = 0.f, vs = 0.f;
    if constexpr (EIGHT) {
      ms = T.avg_scale[at / BLOCK];
      vs = T.sq_scale[at / BLOCK];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = w[j] = m[j] = v[j] = r[j] = 0.f;
      if (!in[j]) continue;
      g[j] = load_one(T.grad, where[j], gt);
      // a bf16 weight with a low half is taken by its bits
      w[j] = T.mantissa ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(T.param)[where[j]]) << 16 |
                                          T.mantissa[where[j]])
                        : load_one(T.param, where[j], pt);
      if constexpr (EIGHT) {
        m[j] = __fmul_rn(widen_codes(static_cast<const uint8_t*>(T.avg)[where[j]]).x, ms);
        r[j] = __fmul_rn(widen_codes(static_cast<const uint8_t*>(T.sq)[where[j]]).x, vs);
      } else {
        m[j] = static_cast<const float*>(T.avg)[where[j]];
        v[j] = static_cast<const float*>(T.sq)[where[j]];
      }
    }
  }
  if constexpr (EIGHT) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(r[j], r[j]);
  }
  if (grad_scale) {
    const float gs = *grad_scale;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(g[j], gs);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = step_one(g[j], m[j], v[j], r[j], w[j], s, decay, rate);
  float ms = 0.f, vs = 0.f;
  if constexpr (EIGHT) {
    // past the end there is nothing whose size would count
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = in[j] ? m[j] : 0.f;
      r[j] = in[j] ? r[j] : 0.f;
    }
    uint32_t bits[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) bits[j] = 0;
    if (random) {
      const uint32_t key = mix(s.key + static_cast<uint32_t>(T.position));
#pragma unroll
      for (int j = 0; j < 8; ++j) bits[j] = mix(static_cast<uint32_t>(where[j]) + key);
    }
    float q[8];
    ms = scale_block<false>(m, q, random, bits);
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = q[j];
    vs = scale_block<true>(r, q, random, bits);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = q[j];
    if (lane == 0) {
      T.avg_scale[at / BLOCK] = ms;
      T.sq_scale[at / BLOCK] = vs;
    }
  }
  if constexpr (VEC) {
    const long long first = at + 8 * lane;
    if (T.mantissa) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = __float_as_uint(w[2 * j]), b = __float_as_uint(w[2 * j + 1]);
        hi[j] = __byte_perm(a, b, 0x7632);
        lo[j] = __byte_perm(a, b, 0x5410);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(T.param) + first) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(T.mantissa + first) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    } else {
      store_eight(T.param, first, pt, w);
    }
    if constexpr (EIGHT) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.avg) + first) =
          make_uint2(codes_of(m[0], m[1]) | codes_of(m[2], m[3]) << 16, codes_of(m[4], m[5]) | codes_of(m[6], m[7]) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.sq) + first) =
          make_uint2(codes_of(v[0], v[1]) | codes_of(v[2], v[3]) << 16, codes_of(v[4], v[5]) | codes_of(v[6], v[7]) << 16);
    } else {
      store_eight(T.avg, first, MB_F32, m);
      store_eight(T.sq, first, MB_F32, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!in[j]) continue;
      if (T.mantissa) {
        static_cast<uint16_t*>(T.param)[where[j]] = static_cast<uint16_t>(__float_as_uint(w[j]) >> 16);
        T.mantissa[where[j]] = static_cast<uint16_t>(__float_as_uint(w[j]));
      } else {
        store_one(T.param, where[j], pt, w[j]);
      }
      if constexpr (EIGHT) {
        static_cast<uint8_t*>(T.avg)[where[j]] = static_cast<uint8_t>(codes_of(m[j], 0.f));
        static_cast<uint8_t*>(T.sq)[where[j]] = static_cast<uint8_t>(codes_of(v[j], 0.f));
      } else {
        static_cast<float*>(T.avg)[where[j]] = m[j];
        static_cast<float*>(T.sq)[where[j]] = v[j];
      }
    }
  }
}

// Blocks of 256 elements that a warp takes in turn.
constexpr int TURNS = 2;
constexpr int CHUNK = WARPS * TURNS * BLOCK;

template <int CAP, bool EIGHT>
__global__ void __launch_bounds__(THREADS) adamw_kernel(const __grid_constant__ AdamParams<CAP> p) {
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
  const long long begin = static_cast<long long>(blockIdx.x - T.first) * CHUNK + warp * BLOCK;
#pragma unroll
  for (int u = 0; u < TURNS; ++u) {
    const long long at = begin + u * (WARPS * BLOCK);
    if (at >= T.n) return;
    if (T.aligned && at + BLOCK <= T.n) step_block<EIGHT, true>(T, s, decay, rate, p.grad_scale, p.random, at, lane);
    else step_block<EIGHT, false>(T, s, decay, rate, p.grad_scale, p.random, at, lane);
  }
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
    const long long need = (t.n + CHUNK - 1) / CHUNK;
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
