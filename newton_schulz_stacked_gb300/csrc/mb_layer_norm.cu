// Layer norm over the rows of [rows, cols]: forward, and backward with the reduction of the
// weight's and bias's gradients over the rows.  All arithmetic is fp32.
//
//   m = mean_j x_j;  r = 1 / sqrt(mean_j (x_j - m)^2 + eps);  h = (x - m) r;  y = h w + b
//   g = dy w;  dx = r (g - mean_j g - h mean_j(g h));  dw = sum_rows dy h;  db = sum_rows dy
//
// Both directions are bound by HBM (two and three passes of the elements' size): a row is read
// once and stays in its threads' registers through the statistics and the result.
#include <algorithm>

#include "mb_block.h"
#include "mb_rows.cuh"
#include "muonbank.h"

namespace mb {
namespace {

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

// ---------------------------------------------------------------- forward

// a += the squares of the piece's differences from m, within the row.
template <typename P>
__device__ __forceinline__ void add_squares(const P& x, float m, int cols, int v, int t, int tpr, float2& a) {
  float2 f[4];
  get_pairs(x, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 d = __fadd2_rn(f[j], both(-m));
    if (!P::in(v, 2 * j, t, tpr, cols)) d.x = 0.f;
    if (!P::in(v, 2 * j + 1, t, tpr, cols)) d.y = 0.f;
    a = __ffma2_rn(d, d, a);
  }
}
// f <- (f - m) r w + b
__device__ __forceinline__ void normalise(float2 (&f)[4], float m, float r, const float2 (&w)[4], const float2 (&b)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[j], both(-m)), both(r)), w[j], b[j]);
}
// A weight or bias as pairs.
template <typename T, bool VEC>
__device__ __forceinline__ void load_param_pairs(const void* p, bool f32, float otherwise, int cols, int t, int tpr,
                                                 float2 (&f)[4]) {
  float v[8];
  load_param<T, VEC>(p, f32, otherwise, cols, 0, t, tpr, v);
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = make_float2(v[2 * j], v[2 * j + 1]);
}

// A weight or bias in shared memory, in fp32: [piece][half][thread][4], so that 16-byte reads of
// neighbouring threads meet no bank twice.
template <typename T, bool VEC, int NV>
__device__ __forceinline__ void stage_param(const void* p, bool f32, float otherwise, int cols, int t, int tpr, float* to) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float f[8];
    load_param<T, VEC>(p, f32, otherwise, cols, v, t, tpr, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) to[(v * 8 + (j & 4)) * tpr + t * 4 + (j & 3)] = f[j];
  }
}
__device__ __forceinline__ void staged_param(const float* from, int v, int t, int tpr, float2 (&f)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 x = *reinterpret_cast<const float4*>(from + ((v * 8 + 4 * h) * tpr + t * 4));
    f[2 * h] = make_float2(x.x, x.y);
    f[2 * h + 1] = make_float2(x.z, x.w);
  }
}

// CTAs per SM of the kernel below: 80 registers with 16-bit vectors, else 128.
template <typename T, bool VEC>
constexpr int fwd_ctas() { return VEC && sizeof(T) == 2 ? 3 : 2; }

// Rows of up to 1024 elements: tpr lanes of a warp hold a row in NV pieces of eight elements each
// and take R rows at a time, the next R already being loaded; no barrier in the loop.  Weight and
// bias wait in shared memory, in fp32 and in the order in which the lanes read them.  The variance
// sums squares of differences from the mean, over the registers: no cancellation however far the
// mean is from zero.
template <typename T, bool VEC, int NV, int R>
__global__ void __launch_bounds__(256, fwd_ctas<T, VEC>()) ln_fwd_kernel(const LnFwdParams p) {
  extern __shared__ __align__(16) float wb[];          // [2][NV][8 or (halves of) 4][tpr]
  using P = Piece<T, VEC>;
  const int tpr = p.tpr, cols = p.cols;
  const int t = threadIdx.x % tpr, g = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const float inv_n = 1.f / static_cast<float>(cols);
  const long long step = static_cast<long long>(groups) * R, stride = step * gridDim.x;
  P x[R][NV], next[R][NV];
  auto fetch = [&](long long base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * groups + g;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        next[r][v].load(static_cast<const T*>(p.x) + row * p.x_stride, cols, v, t, tpr, row < p.rows);
    }
  };
  long long base = blockIdx.x * step;
  fetch(base);
  if (g == 0) {
    stage_param<T, VEC, NV>(p.w, p.w_f32, 1.f, cols, t, tpr, wb);
    stage_param<T, VEC, NV>(p.b, p.w_f32, 0.f, cols, t, tpr, wb + NV * 8 * tpr);
  }
  __syncthreads();
  for (; base < p.rows; base += stride) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int v = 0; v < NV; ++v) x[r][v] = next[r][v];
    if (base + stride < p.rows) fetch(base + stride);
    float s[R], m[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 a = both(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float2 f[4];
        get_pairs(x[r][v], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) a = __fadd2_rn(a, f[j]);      // elements past the row are zero
      }
      s[r] = a.x + a.y;
    }
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], o);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = s[r] * inv_n;
      float2 a = both(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v) add_squares<P>(x[r][v], m[r], cols, v, t, tpr, a);
      s[r] = a.x + a.y;
    }
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], o);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = rsqrtf(fmaf(s[r], inv_n, p.eps));
      const long long row = base + r * groups + g;
      if (t == 0 && row < p.rows) {
        if (p.mean) p.mean[row] = m[r];
        if (p.rstd) p.rstd[row] = s[r];
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 w[4], b[4];
      staged_param(wb, v, t, tpr, w);
      staged_param(wb, NV + v, t, tpr, b);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const long long row = base + r * groups + g;
        if (row < p.rows) {
          float2 f[4];
          get_pairs(x[r][v], f);
          normalise(f, m[r], s[r], w, b);
          store_pairs<P>(static_cast<T*>(p.y) + row * p.y_stride, cols, v, t, tpr, f);
        }
      }
    }
  }
}

// Rows of up to 8192 elements: a thread owns eight columns and keeps their weight and bias; a
// group of tpr threads (whole warps) covers a row and takes R rows at a time, the next R already
// being loaded.
template <typename T, bool VEC, int R, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 288 ? 2 : 1) ln_fwd_group_kernel(const LnFwdParams p) {
  __shared__ float part[2][MAXT / 32][R];
  using P = Piece<T, VEC>;
  const int tpr = p.tpr, cols = p.cols, groups = blockDim.x / tpr;
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  const float inv_n = 1.f / static_cast<float>(cols);
  const long long step = static_cast<long long>(groups) * R, stride = step * gridDim.x;
  P x[R], next[R];
  auto fetch = [&](long long row0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      next[r].load(static_cast<const T*>(p.x) + (row0 + r) * p.x_stride, cols, 0, t, tpr, row0 + r < p.rows);
  };
  long long row0 = blockIdx.x * step + g * R;
  fetch(row0);
  float2 w[4], b[4];
  load_param_pairs<T, VEC>(p.w, p.w_f32, 1.f, cols, t, tpr, w);
  load_param_pairs<T, VEC>(p.b, p.w_f32, 0.f, cols, t, tpr, b);
  RowSums<R, MAXT / 32> sums(part, tpr, g);
  for (; row0 < p.rows; row0 += stride) {
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = next[r];
    if (row0 + stride < p.rows) fetch(row0 + stride);
    float s[R], m[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 f[4], a;
      get_pairs(x[r], f);
      a = __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3]));
      s[r] = a.x + a.y;
    }
    sums(s);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = s[r] * inv_n;
      float2 a = both(0.f);
      add_squares<P>(x[r], m[r], cols, 0, t, tpr, a);
      s[r] = a.x + a.y;
    }
    sums(s);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r < p.rows) {
        s[r] = rsqrtf(fmaf(s[r], inv_n, p.eps));
        if (t == 0) {
          if (p.mean) p.mean[row0 + r] = m[r];
          if (p.rstd) p.rstd[row0 + r] = s[r];
        }
        float2 f[4];
        get_pairs(x[r], f);
        normalise(f, m[r], s[r], w, b);
        store_pairs<P>(static_cast<T*>(p.y) + (row0 + r) * p.y_stride, cols, 0, t, tpr, f);
      }
    }
  }
}

// Rows too wide for registers: one CTA per row reads it three times (the second and third
// time out of L2 for all but the widest).
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) ln_fwd_wide_kernel(const LnFwdParams p) {
  __shared__ float smem[32];
  using P = Piece<T, VEC>;
  const int t = threadIdx.x, tpr = blockDim.x, cols = p.cols;
  const int nv = (cols + 8 * tpr - 1) / (8 * tpr);
  const float inv_n = 1.f / static_cast<float>(cols);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.x_stride;
    float s = 0.f, q = 0.f, f[8];
    for (int v = 0; v < nv; ++v) {
      P x;
      x.load(xr, cols, v, t, tpr);
      x.get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += f[j];
    }
    const float m = cta_sum(s, smem) * inv_n;
    for (int v = 0; v < nv; ++v) {
      P x;
      x.load(xr, cols, v, t, tpr);
      x.get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = P::in(v, j, t, tpr, cols) ? f[j] - m : 0.f;
        q = fmaf(d, d, q);
      }
    }
    const float rs = rsqrtf(fmaf(cta_sum(q, smem), inv_n, p.eps));
    if (t == 0) {
      if (p.mean) p.mean[row] = m;
      if (p.rstd) p.rstd[row] = rs;
    }
    for (int v = 0; v < nv; ++v) {
      P x;
      float w[8], b[8];
      x.load(xr, cols, v, t, tpr);
      x.get(f);
      load_param<T, VEC>(p.w, p.w_f32, 1.f, cols, v, t, tpr, w);
      load_param<T, VEC>(p.b, p.w_f32, 0.f, cols, v, t, tpr, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf((f[j] - m) * rs, w[j], b[j]);
      P::store(static_cast<T*>(p.y) + row * p.y_stride, cols, v, t, tpr, f);
    }
  }
}

// ---------------------------------------------------------------- backward

__device__ __forceinline__ void put_param_grad(void* out, bool f32, int c, float v, __nv_bfloat16) {
  if (f32) static_cast<float*>(out)[c] = v;
  else static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void put_param_grad(void* out, bool f32, int c, float v, __half) {
  if (f32) static_cast<float*>(out)[c] = v;
  else static_cast<__half*>(out)[c] = __float2half_rn(v);
}
__device__ __forceinline__ void put_param_grad(void* out, bool, int c, float v, float) {
  static_cast<float*>(out)[c] = v;
}

// A thread owns eight columns: a group of tpr threads covers a row, takes R rows at a time (the
// next R already being loaded) and adds dy h and dy of its columns over all its rows in registers,
// so the weight's gradient needs no second pass over dy and x.  The CTA's groups add theirs in
// shared memory at the end, the CTAs through `parts` (fixed orders throughout: results repeat bit
// for bit).
template <typename T, bool VEC, int R, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 288 ? 2 : 1) ln_bwd_kernel(const LnBwdParams p) {
  extern __shared__ float dyn[];                       // [threads][16] at the end
  __shared__ float part[2][MAXT / 32][2 * R];
  using P = Piece<T, VEC>;
  const int tpr = p.tpr, cols = p.cols, groups = p.groups;
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  const float inv_n = 1.f / static_cast<float>(cols);
  // every group of the CTA goes round the same number of times (a warp may hold several groups)
  const long long step = static_cast<long long>(groups) * R, stride = step * gridDim.x;
  P next_x[R], next_dy[R];
  float next_m[R], next_rs[R];
  auto fetch = [&](long long row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = row0 + g * R + r;
      const bool on = row < p.rows;
      next_x[r].load(static_cast<const T*>(p.x) + row * p.x_stride, cols, 0, t, tpr, on);
      next_dy[r].load(static_cast<const T*>(p.dy) + row * p.dy_stride, cols, 0, t, tpr, on);
      next_m[r] = on ? p.mean[row] : 0.f;
      next_rs[r] = on ? p.rstd[row] : 0.f;
    }
  };
  long long base = blockIdx.x * step;
  fetch(base);
  float2 w[4], dw[4], db[4];
  load_param_pairs<T, VEC>(p.w, p.w_f32, 1.f, cols, t, tpr, w);
#pragma unroll
  for (int j = 0; j < 4; ++j) dw[j] = db[j] = both(0.f);
  RowSums<2 * R, MAXT / 32> sums(part, tpr, g);
  for (; base < p.rows; base += stride) {
    const long long row0 = base + g * R;
    float2 h[R][4], gr[R][4];                          // (x - m) r and dy w of the rows
    float rs[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 df[4], s1 = both(0.f), s2 = both(0.f);
      rs[r] = next_rs[r];
      get_pairs(next_x[r], h[r]);
      get_pairs(next_dy[r], df);
      const float m = next_m[r];
#pragma unroll
      for (int j = 0; j < 4; ++j) {                    // past the row dy is 0, and h of no consequence
        h[r][j] = __fmul2_rn(__fadd2_rn(h[r][j], both(-m)), both(rs[r]));
        gr[r][j] = __fmul2_rn(df[j], w[j]);
        s1 = __fadd2_rn(s1, gr[r][j]);
        s2 = __ffma2_rn(gr[r][j], h[r][j], s2);
        dw[j] = __ffma2_rn(df[j], h[r][j], dw[j]);
        db[j] = __fadd2_rn(db[j], df[j]);
      }
      s[2 * r] = s1.x + s1.y;
      s[2 * r + 1] = s2.x + s2.y;
    }
    if (base + stride < p.rows) fetch(base + stride);
    sums(s);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r < p.rows) {
        const float c1 = s[2 * r] * inv_n, c2 = s[2 * r + 1] * inv_n;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[r][j] = __fmul2_rn(__fadd2_rn(gr[r][j], __ffma2_rn(h[r][j], both(-c2), both(-c1))), both(rs[r]));
        store_pairs<P>(static_cast<T*>(p.dx) + (row0 + r) * p.dx_stride, cols, 0, t, tpr, h[r]);
      }
    }
  }
  let_next_kernel_start();
  if (!p.dw && !p.db) return;
  // the CTA's sum over its groups: [16 values][threads], so that threads touch neighbouring words
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    dyn[j * blockDim.x + threadIdx.x] = j & 1 ? dw[j / 2].y : dw[j / 2].x;
    dyn[(8 + j) * blockDim.x + threadIdx.x] = j & 1 ? db[j / 2].y : db[j / 2].x;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * tpr; e += blockDim.x) {
    const int k = e / tpr, tt = e - k * tpr, j = k & 7;
    if (!P::in(0, j, tt, tpr, cols)) continue;
    float sum = 0.f;
    for (int u = 0; u < groups; ++u) sum += dyn[k * blockDim.x + u * tpr + tt];
    const int c = P::col(0, j, tt, tpr);
    if (p.parts) {
      p.parts[(static_cast<size_t>(blockIdx.x) * 2 + (k >> 3)) * cols + c] = sum;
    } else {
      void* out = k < 8 ? p.dw : p.db;
      if (out) put_param_grad(out, p.w_f32, c, sum, T());
    }
  }
}

// Threads of a CTA (one per SM) of the kernel below, by what the registers of NV pieces allow.
template <int NV>
constexpr int BWD_THREADS = NV == 2 ? 512 : NV == 3 ? 384 : 256;

// Rows of 257 to 1024 elements: a warp holds a row in NV pieces per lane and sums over it by
// exchanges alone; the next row is already being loaded.  Sums of the gradient as above.
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(BWD_THREADS<NV>, 1) ln_bwd_warp_kernel(const LnBwdParams p) {
  extern __shared__ __align__(16) float dyn[];         // the weight [NV][8][32]; at the end [warps][NV][16][32] sums
  using P = Piece<T, VEC>;
  constexpr int WARPS = BWD_THREADS<NV> / 32;
  const int cols = p.cols, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inv_n = 1.f / static_cast<float>(cols);
  const long long stride = static_cast<long long>(gridDim.x) * WARPS;
  long long row = static_cast<long long>(blockIdx.x) * WARPS + warp;
  P next_x[NV], next_dy[NV];
  float next_m = 0.f, next_rs = 0.f;
  const T *x = static_cast<const T*>(p.x) + row * p.x_stride, *dy = static_cast<const T*>(p.dy) + row * p.dy_stride;
  T* dx = static_cast<T*>(p.dx) + row * p.dx_stride;
  auto fetch = [&](long long r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      next_x[v].load(x, cols, v, lane, 32);
      next_dy[v].load(dy, cols, v, lane, 32);
    }
    next_m = p.mean[r];
    next_rs = p.rstd[r];
    x += stride * p.x_stride;
    dy += stride * p.dy_stride;
  };
  if (row < p.rows) fetch(row);
  if (warp == 0) stage_param<T, VEC, NV>(p.w, p.w_f32, 1.f, cols, lane, 32, dyn);
  __syncthreads();
  float2 dw[NV][4], db[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[v][j] = db[v][j] = both(0.f);
  for (; row < p.rows; row += stride) {
    float2 h[NV][4], gr[NV][4], s1 = both(0.f), s2 = both(0.f);
    const float2 m = both(-next_m), rs = both(next_rs);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 w[4];
      staged_param(dyn, v, lane, 32, w);
      get_pairs(next_x[v], h[v]);
      get_pairs(next_dy[v], gr[v]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {                    // past the row dy is 0, and h of no consequence
        const float2 d = gr[v][j];
        h[v][j] = __fmul2_rn(__fadd2_rn(h[v][j], m), rs);
        gr[v][j] = __fmul2_rn(d, w[j]);
        s1 = __fadd2_rn(s1, gr[v][j]);
        s2 = __ffma2_rn(gr[v][j], h[v][j], s2);
        dw[v][j] = __ffma2_rn(d, h[v][j], dw[v][j]);
        db[v][j] = __fadd2_rn(db[v][j], d);
      }
    }
    if (row + stride < p.rows) fetch(row + stride);
    const float c1 = group_sum(s1.x + s1.y, 32) * inv_n, c2 = group_sum(s2.x + s2.y, 32) * inv_n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[v][j] = __fmul2_rn(__fadd2_rn(gr[v][j], __ffma2_rn(h[v][j], both(-c2), both(-c1))), rs);
      store_pairs<P>(dx, cols, v, lane, 32, h[v]);
    }
    dx += stride * p.dx_stride;
  }
  let_next_kernel_start();
  if (!p.dw && !p.db) return;
  __syncthreads();                                     // the weight has been read
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float* to = dyn + ((warp * NV + v) * 16 + j) * 32 + lane;
      to[0] = j & 1 ? dw[v][j / 2].y : dw[v][j / 2].x;
      to[8 * 32] = j & 1 ? db[v][j / 2].y : db[v][j / 2].x;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < NV * 16 * 32; e += blockDim.x) {
    const int tt = e & 31, k = (e >> 5) & 15, v = e >> 9, j = k & 7;
    if (!P::in(v, j, tt, 32, cols)) continue;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < WARPS; ++u) sum += dyn[u * NV * 512 + e];
    const int c = P::col(v, j, tt, 32);
    if (p.parts) {
      p.parts[(static_cast<size_t>(blockIdx.x) * 2 + (k >> 3)) * cols + c] = sum;
    } else {
      void* out = k < 8 ? p.dw : p.db;
      if (out) put_param_grad(out, p.w_f32, c, sum, T());
    }
  }
}

struct LnPartsParams {
  const float* parts;
  int n, cols, w_f32;
  void *dw, *db;
};

// dw and db from the partial sums: 32 columns by 32 slices of the parts per CTA.
template <typename T>
__global__ void __launch_bounds__(1024) ln_parts_kernel(const LnPartsParams p) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  wait_for_previous_kernel();
  float a = 0.f;
  if (c < 2ll * p.cols) {
#pragma unroll 10
    for (int i = slice; i < p.n; i += 32) a += p.parts[static_cast<size_t>(i) * 2 * p.cols + c];
  }
  s[slice][lane] = a;
  __syncthreads();
  // column 32 blockIdx + slice: its slices' sums over the lanes
  const long long mine = static_cast<long long>(blockIdx.x) * 32 + slice;
  a = group_sum(s[lane][slice], 32);
  if (lane == 0 && mine < 2ll * p.cols) {
    void* out = mine < p.cols ? p.dw : p.db;
    if (out) put_param_grad(out, p.w_f32, static_cast<int>(mine < p.cols ? mine : mine - p.cols), a, T());
  }
}

// Wide rows: dx with one CTA per row, which reads the row twice ...
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) ln_bwd_wide_kernel(const LnBwdParams p) {
  __shared__ float smem[32];
  using P = Piece<T, VEC>;
  const int t = threadIdx.x, tpr = blockDim.x, cols = p.cols;
  const int nv = (cols + 8 * tpr - 1) / (8 * tpr);
  const float inv_n = 1.f / static_cast<float>(cols);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* dr = static_cast<const T*>(p.dy) + row * p.dy_stride;
    const float m = p.mean[row], rs = p.rstd[row];
    float s1 = 0.f, s2 = 0.f, xf[8], df[8], w[8];
    for (int v = 0; v < nv; ++v) {
      P x, dy;
      x.load(xr, cols, v, t, tpr);
      dy.load(dr, cols, v, t, tpr);
      load_param<T, VEC>(p.w, p.w_f32, 1.f, cols, v, t, tpr, w);
      x.get(xf);
      dy.get(df);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = P::in(v, j, t, tpr, cols) ? (xf[j] - m) * rs : 0.f;
        s1 = fmaf(df[j], w[j], s1);
        s2 = fmaf(df[j] * w[j], h, s2);
      }
    }
    const float c1 = cta_sum(s1, smem) * inv_n, c2 = cta_sum(s2, smem) * inv_n;
    for (int v = 0; v < nv; ++v) {
      P x, dy;
      x.load(xr, cols, v, t, tpr);
      dy.load(dr, cols, v, t, tpr);
      load_param<T, VEC>(p.w, p.w_f32, 1.f, cols, v, t, tpr, w);
      x.get(xf);
      dy.get(df);
#pragma unroll
      for (int j = 0; j < 8; ++j) xf[j] = rs * (fmaf(df[j], w[j], -c1) - (xf[j] - m) * rs * c2);
      P::store(static_cast<T*>(p.dx) + row * p.dx_stride, cols, v, t, tpr, xf);
    }
  }
}

// ... and, before it (dx may lie over x or dy), the weight's gradient with one thread per
// column and slab of rows.
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_wide_params_kernel(const LnBwdParams p) {
  const long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float dw = 0.f, db = 0.f;
#pragma unroll 4
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float d = to_float(static_cast<const T*>(p.dy)[row * p.dy_stride + c]);
    const float h = (to_float(static_cast<const T*>(p.x)[row * p.x_stride + c]) - p.mean[row]) * p.rstd[row];
    dw = fmaf(d, h, dw);
    db += d;
  }
  float* out = p.parts + static_cast<size_t>(blockIdx.y) * 2 * p.cols;
  out[c] = dw;
  out[p.cols + c] = db;
}

// ---------------------------------------------------------------- launches

bool vec_rows(const void* p, long long stride, int size, long long rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (stride * size) % 16 == 0);
}
bool vec_param(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int pow2_at_least(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

// How groups of threads share rows of up to 8192 elements: 576 threads per SM at 112 registers in
// two or three CTAs up to rows of 2304 elements, then one CTA of 128 or 64 registers.
struct GroupShape {
  int tpr, groups;      // threads per row, rows side by side in a CTA
  int most;             // the kernel's MAXT
  int rows;             // rows at a time of a group
  int ctas;             // per SM
};
GroupShape group_shape(int cols, bool vec) {
  const int pieces = (cols + 7) / 8;
  GroupShape g{};
  g.tpr = pieces <= 32 ? pow2_at_least(pieces) : (pieces + 31) / 32 * 32;
  g.most = g.tpr <= 288 ? 288 : g.tpr <= 512 ? 512 : 1024;
  g.groups = g.tpr < 32 ? 256 / g.tpr : g.most / g.tpr;
  g.rows = vec && g.most <= 512 ? 2 : 1;
  g.ctas = g.most == 288 ? std::min(3, 576 / (g.groups * g.tpr)) : 1;
  return g;
}
int cta_count(long long rows, long long per_cta, int most) {
  const long long want = (rows + per_cta - 1) / per_cta;
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

template <typename T, bool VEC>
cudaError_t fwd(LnFwdParams p, int sms, cudaStream_t s) {
  const int pieces = (p.cols + 7) / 8;
  if (p.cols > LN_MAX_COLS) {
    ln_fwd_wide_kernel<T, VEC><<<cta_count(p.rows, 1, 2 * sms), 1024, 0, s>>>(p);
  } else if (pieces > 128) {
    const GroupShape g = group_shape(p.cols, VEC);
    p.tpr = g.tpr;
    const int grid = cta_count(p.rows, g.groups * g.rows, g.ctas * sms), threads = g.groups * g.tpr;
    constexpr int R = VEC ? 2 : 1;
    if (g.most == 288) ln_fwd_group_kernel<T, VEC, R, 288><<<grid, threads, 0, s>>>(p);
    else if (g.most == 512) ln_fwd_group_kernel<T, VEC, R, 512><<<grid, threads, 0, s>>>(p);
    else ln_fwd_group_kernel<T, VEC, 1, 1024><<<grid, threads, 0, s>>>(p);
  } else {
    const int nv = (pieces + 31) / 32;
    constexpr int R1 = VEC ? 4 : 2, R2 = VEC ? 2 : 1;  // rows at a time of one and two pieces
    const int r = nv == 1 ? R1 : nv == 2 ? R2 : 1;
    p.tpr = pieces >= 32 ? 32 : pow2_at_least(pieces);
    const int grid = cta_count(p.rows, static_cast<long long>(256 / p.tpr) * r, fwd_ctas<T, VEC>() * sms);
    const size_t smem = static_cast<size_t>(2 * nv * 8) * p.tpr * sizeof(float);
    if (nv == 1) ln_fwd_kernel<T, VEC, 1, R1><<<grid, 256, smem, s>>>(p);
    else if (nv == 2) ln_fwd_kernel<T, VEC, 2, R2><<<grid, 256, smem, s>>>(p);
    else if (nv == 3) ln_fwd_kernel<T, VEC, 3, 1><<<grid, 256, smem, s>>>(p);
    else ln_fwd_kernel<T, VEC, 4, 1><<<grid, 256, smem, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_any(const LnFwdParams& p, int sms, cudaStream_t s) {
  const bool vec = p.cols % 8 == 0 && vec_rows(p.x, p.x_stride, sizeof(T), p.rows) &&
                   vec_rows(p.y, p.y_stride, sizeof(T), p.rows) && vec_param(p.w) && vec_param(p.b);
  return vec ? fwd<T, true>(p, sms, s) : fwd<T, false>(p, sms, s);
}

template <typename T>
cudaError_t add_parts(const LnBwdParams& p, int n, cudaStream_t s) {
  LnPartsParams q{p.parts, n, p.cols, p.w_f32, p.dw, p.db};
  return launch_after(ln_parts_kernel<T>, dim3((2u * p.cols + 31) / 32), dim3(1024), 0, s, q);
}

template <typename T, bool VEC>
cudaError_t bwd(LnBwdParams p, int sms, cudaStream_t s, int* launches) {
  const bool params = p.dw || p.db;
  cudaError_t e;
  if (p.cols > LN_MAX_COLS) {
    if (params) {
      const int slabs = static_cast<int>(p.rows < 1 ? 1 : p.rows < 64 ? p.rows : 64);
      ln_bwd_wide_params_kernel<T><<<dim3((p.cols + 255) / 256, slabs), 256, 0, s>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      if ((e = add_parts<T>(p, slabs, s)) != cudaSuccess) return e;
      *launches += 2;
    }
    if (p.rows == 0) return cudaSuccess;
    ln_bwd_wide_kernel<T, VEC><<<cta_count(p.rows, 1, 2 * sms), 1024, 0, s>>>(p);
    *launches += 1;
    return cudaGetLastError();
  }
  int grid, threads;
  size_t smem;
  void (*kernel)(LnBwdParams);
  const int pieces = (p.cols + 7) / 8;
  if (pieces > 32 && pieces <= 128) {
    const int nv = (pieces + 31) / 32;
    threads = nv == 2 ? BWD_THREADS<2> : nv == 3 ? BWD_THREADS<3> : BWD_THREADS<4>;
    grid = cta_count(p.rows, threads / 32, std::min(LN_MAX_PARTS, sms));
    smem = static_cast<size_t>(nv) * (params ? 16 * threads : 8 * 32) * sizeof(float);
    kernel = nv == 2 ? ln_bwd_warp_kernel<T, VEC, 2> : nv == 3 ? ln_bwd_warp_kernel<T, VEC, 3> : ln_bwd_warp_kernel<T, VEC, 4>;
  } else {
    const GroupShape g = group_shape(p.cols, VEC);
    p.tpr = g.tpr;
    p.groups = g.groups;
    threads = g.groups * g.tpr;
    grid = cta_count(p.rows, g.groups * g.rows, std::min(LN_MAX_PARTS, g.ctas * sms));
    smem = params ? static_cast<size_t>(threads) * 16 * sizeof(float) : 0;
    constexpr int R = VEC ? 2 : 1;
    kernel = g.most == 288   ? ln_bwd_kernel<T, VEC, R, 288>
             : g.most == 512 ? ln_bwd_kernel<T, VEC, R, 512> : ln_bwd_kernel<T, VEC, 1, 1024>;
  }
  if (grid == 1 || !params) p.parts = nullptr;
  if (smem > 40 * 1024 &&
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem))) !=
          cudaSuccess)
    return e;
  kernel<<<grid, threads, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  *launches += 1;
  if (!p.parts) return cudaSuccess;
  *launches += 1;
  return add_parts<T>(p, grid, s);
}

template <typename T>
cudaError_t bwd_any(const LnBwdParams& p, int sms, cudaStream_t s, int* launches) {
  const bool vec = p.cols % 8 == 0 && vec_rows(p.x, p.x_stride, sizeof(T), p.rows) &&
                   vec_rows(p.dy, p.dy_stride, sizeof(T), p.rows) && vec_rows(p.dx, p.dx_stride, sizeof(T), p.rows) &&
                   vec_param(p.w);
  return vec ? bwd<T, true>(p, sms, s, launches) : bwd<T, false>(p, sms, s, launches);
}

}  // namespace

cudaError_t launch_layer_norm(LnFwdParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 1;
  if (type == MB_F32) return fwd_any<float>(p, sms, s);
  if (type == MB_BF16) return fwd_any<__nv_bfloat16>(p, sms, s);
  return fwd_any<__half>(p, sms, s);
}

cudaError_t launch_layer_norm_backward(LnBwdParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 0;
  if (type == MB_F32) return bwd_any<float>(p, sms, s, launches);
  if (type == MB_BF16) return bwd_any<__nv_bfloat16>(p, sms, s, launches);
  return bwd_any<__half>(p, sms, s, launches);
}

}  // namespace mb
