// Layer norm over the rows of [rows, cols]: forward, and backward with the reduction of the
// weight's and bias's gradients over the rows.  All arithmetic is fp32.
//
//   m = mean_j x_j;  r = 1 / sqrt(mean_j (x_j - m)^2 + eps);  h = (x - m) r;  y = h w + b
//   g = dy w;  dx = r (g - mean_j g - h mean_j(g h));  dw = sum_rows dy h;  db = sum_rows dy
//
// Both directions are bound by HBM (two and three passes of the elements' size): a row is read
// once and stays in its threads' registers through the statistics and the result.
#include "mb_block.h"
#include "mb_rows.cuh"
#include "muonbank.h"

namespace mb {
namespace {

// Sum over the threads of a row: `tpr` lanes of a warp, or the whole CTA (MULTI) through
// shared memory.  Every thread gets the sum, formed in the same order in each of them.
template <bool MULTI, int R>
__device__ __forceinline__ void row_sum(float (&s)[R], int tpr, float* smem) {
  const int width = MULTI ? 32 : tpr;
  for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], o);
  if constexpr (MULTI) {
    static_assert(R == 1, "a CTA holds one row at a time");
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    __syncthreads();                       // the previous sum has been read
    if ((threadIdx.x & 31) == 0) smem[warp] = s[0];
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < nw; ++i) t += smem[i];
    s[0] = t;
  }
}

// ---------------------------------------------------------------- forward

// R rows at a time per group of tpr threads (MULTI: one row per CTA), NV pieces of eight
// elements per thread and row.  The variance sums squares of differences from the mean, over
// the registers: no cancellation however far the mean is from zero.
template <typename T, bool VEC, int NV, int R, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 1024 : 256) ln_fwd_kernel(const LnFwdParams p) {
  __shared__ float smem[32];
  using P = Piece<T, VEC>;
  const int tpr = p.tpr, cols = p.cols;
  const int t = MULTI ? threadIdx.x : threadIdx.x % tpr;
  const int groups = MULTI ? 1 : blockDim.x / tpr, g = MULTI ? 0 : threadIdx.x / tpr;
  const float inv_n = 1.f / static_cast<float>(cols);
  const long long step = static_cast<long long>(groups) * R;
  for (long long base = blockIdx.x * step; base < p.rows; base += gridDim.x * step) {
    P x[R][NV];
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * groups + g;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        x[r][v].load(static_cast<const T*>(p.x) + row * p.x_stride, cols, v, t, tpr, row < p.rows);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
        x[r][v].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[r] += f[j];      // elements past the row are zero
      }
    }
    row_sum<MULTI, R>(s, tpr, smem);
    float m[R], q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = s[r] * inv_n;
      q[r] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
        x[r][v].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = P::in(v, j, t, tpr, cols) ? f[j] - m[r] : 0.f;
          q[r] = fmaf(d, d, q[r]);
        }
      }
    }
    row_sum<MULTI, R>(q, tpr, smem);
    float rs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rs[r] = rsqrtf(fmaf(q[r], inv_n, p.eps));
      const long long row = base + r * groups + g;
      if (t == 0 && row < p.rows) {
        if (p.mean) p.mean[row] = m[r];
        if (p.rstd) p.rstd[row] = rs[r];
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w[8], b[8];
      load_param<T, VEC>(p.w, p.w_f32, 1.f, cols, v, t, tpr, w);
      load_param<T, VEC>(p.b, p.w_f32, 0.f, cols, v, t, tpr, b);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const long long row = base + r * groups + g;
        if (row < p.rows) {
          float f[8];
          x[r][v].get(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = fmaf((f[j] - m[r]) * rs[r], w[j], b[j]);
          P::store(static_cast<T*>(p.y) + row * p.y_stride, cols, v, t, tpr, f);
        }
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
    float s[1] = {0.f}, q[1] = {0.f}, f[8];
    for (int v = 0; v < nv; ++v) {
      P x;
      x.load(xr, cols, v, t, tpr);
      x.get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += f[j];
    }
    row_sum<true, 1>(s, tpr, smem);
    const float m = s[0] * inv_n;
    for (int v = 0; v < nv; ++v) {
      P x;
      x.load(xr, cols, v, t, tpr);
      x.get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = P::in(v, j, t, tpr, cols) ? f[j] - m : 0.f;
        q[0] = fmaf(d, d, q[0]);
      }
    }
    row_sum<true, 1>(q, tpr, smem);
    const float rs = rsqrtf(fmaf(q[0], inv_n, p.eps));
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

__device__ __forceinline__ void group_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

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

// A thread owns eight columns: a group of tpr threads covers a row, takes R rows at a time and
// adds dy h and dy of its columns over all its rows in registers, so the weight's gradient needs
// no second pass over dy and x.  The CTA's groups add theirs in shared memory at the end, the
// CTAs through `parts` (fixed orders throughout: results repeat bit for bit).
template <typename T, bool VEC, int R, int MAXT>
__global__ void __launch_bounds__(MAXT) ln_bwd_kernel(const LnBwdParams p) {
  extern __shared__ float dyn[];                       // [threads][16] at the end
  __shared__ float part[2][MAXT / 32][2 * R];
  using P = Piece<T, VEC>;
  const int tpr = p.tpr, cols = p.cols, groups = p.groups;
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = tpr >> 5, first_warp = g * warps;  // of this group, if it has whole warps
  const float inv_n = 1.f / static_cast<float>(cols);
  float w[8], dw[8], db[8];
  load_param<T, VEC>(p.w, p.w_f32, 1.f, cols, 0, t, tpr, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.f;
  const long long nblocks = (p.rows + R - 1) / R;
  const long long stride = static_cast<long long>(gridDim.x) * groups;
  // every group of the CTA goes round the same number of times (a warp may hold several groups)
  const long long rounds = (nblocks - static_cast<long long>(blockIdx.x) * groups + stride - 1) / stride;
  int parity = 0;
  for (long long i = 0; i < rounds; ++i, parity ^= 1) {
    const long long row0 = (static_cast<long long>(blockIdx.x) * groups + g + i * stride) * R;
    P x[R], dy[R];
    float m[R], rs[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool on = row0 + r < p.rows;
      x[r].load(static_cast<const T*>(p.x) + (row0 + r) * p.x_stride, cols, 0, t, tpr, on);
      dy[r].load(static_cast<const T*>(p.dy) + (row0 + r) * p.dy_stride, cols, 0, t, tpr, on);
      m[r] = on ? p.mean[row0 + r] : 0.f;
      rs[r] = on ? p.rstd[row0 + r] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float xf[8], df[8];
      x[r].get(xf);
      dy[r].get(df);
      s[2 * r] = s[2 * r + 1] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {                    // dy is zero past the row, and h is finite for a finite row
        const float h = P::in(0, j, t, tpr, cols) ? (xf[j] - m[r]) * rs[r] : 0.f;
        const float gr = df[j] * w[j];
        s[2 * r] += gr;
        s[2 * r + 1] = fmaf(gr, h, s[2 * r + 1]);
        dw[j] = fmaf(df[j], h, dw[j]);
        db[j] += df[j];
      }
    }
    const int width = tpr < 32 ? tpr : 32;
    for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], o);
    if (warps > 1) {
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < 2 * R; ++k) part[parity][warp][k] = s[k];
      group_barrier(1 + g, tpr);        // the other parity's sums are read before anyone passes the next one
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) s[k] = 0.f;
      for (int u = 0; u < warps; ++u)
#pragma unroll
        for (int k = 0; k < 2 * R; ++k) s[k] += part[parity][first_warp + u][k];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r < p.rows) {
        float xf[8], df[8];
        x[r].get(xf);
        dy[r].get(df);
        const float c1 = s[2 * r] * inv_n, c2 = s[2 * r + 1] * inv_n;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float h = (xf[j] - m[r]) * rs[r];
          xf[j] = rs[r] * (fmaf(df[j], w[j], -c1) - h * c2);
        }
        P::store(static_cast<T*>(p.dx) + (row0 + r) * p.dx_stride, cols, 0, t, tpr, xf);
      }
    }
  }
  let_next_kernel_start();
  if (!p.dw && !p.db) return;
  // the CTA's sum over its groups: [16 values][threads], so that threads touch neighbouring words
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    dyn[j * blockDim.x + threadIdx.x] = dw[j];
    dyn[(8 + j) * blockDim.x + threadIdx.x] = db[j];
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

struct LnPartsParams {
  const float* parts;
  int n, cols, w_f32;
  void *dw, *db;
};

// dw and db from the partial sums: 32 columns by 8 slices of the parts per CTA.
template <typename T>
__global__ void __launch_bounds__(256) ln_parts_kernel(const LnPartsParams p) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  wait_for_previous_kernel();
  float a = 0.f;
  if (c < 2ll * p.cols) {
#pragma unroll 4
    for (int i = slice; i < p.n; i += 8) a += p.parts[static_cast<size_t>(i) * 2 * p.cols + c];
  }
  s[slice][lane] = a;
  __syncthreads();
  if (slice == 0 && c < 2ll * p.cols) {
    for (int i = 1; i < 8; ++i) a += s[i][lane];
    void* out = c < p.cols ? p.dw : p.db;
    if (out) put_param_grad(out, p.w_f32, static_cast<int>(c < p.cols ? c : c - p.cols), a, T());
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
    float s1[1] = {0.f}, s2[1] = {0.f}, xf[8], df[8], w[8];
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
        s1[0] = fmaf(df[j], w[j], s1[0]);
        s2[0] = fmaf(df[j] * w[j], h, s2[0]);
      }
    }
    row_sum<true, 1>(s1, tpr, smem);
    row_sum<true, 1>(s2, tpr, smem);
    const float c1 = s1[0] * inv_n, c2 = s2[0] * inv_n;
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

template <typename T, bool VEC>
cudaError_t fwd(LnFwdParams p, int sms, cudaStream_t s) {
  const int pieces = (p.cols + 7) / 8;
  if (p.cols > LN_FWD_MAX_COLS) {
    const int grid = static_cast<int>(p.rows < 2 * sms ? p.rows : 2 * sms);
    ln_fwd_wide_kernel<T, VEC><<<grid, 1024, 0, s>>>(p);
    return cudaGetLastError();
  }
  if (pieces > 128) {                       // one CTA per row
    int nv = 1;
    while (nv < 4 && pieces > 256 * nv) nv *= 2;
    const int threads = (pieces + 32 * nv - 1) / (32 * nv) * 32;
    p.tpr = threads;
    const long long cap = 1ll << 30;
    const int grid = static_cast<int>(p.rows < cap ? p.rows : cap);
    if (nv == 1) ln_fwd_kernel<T, VEC, 1, 1, true><<<grid, threads, 0, s>>>(p);
    else if (nv == 2) ln_fwd_kernel<T, VEC, 2, 1, true><<<grid, threads, 0, s>>>(p);
    else ln_fwd_kernel<T, VEC, 4, 1, true><<<grid, threads, 0, s>>>(p);
    return cudaGetLastError();
  }
  const int nv = (pieces + 31) / 32;
  p.tpr = pieces >= 32 ? 32 : pow2_at_least(pieces);
  const int r = nv == 1 ? 4 : nv == 2 ? 2 : 1;
  const long long per_cta = static_cast<long long>(256 / p.tpr) * r;
  const long long want = (p.rows + per_cta - 1) / per_cta, cap = 1ll << 30;
  const int grid = static_cast<int>(want < cap ? want : cap);
  if (nv == 1) ln_fwd_kernel<T, VEC, 1, 4, false><<<grid, 256, 0, s>>>(p);
  else if (nv == 2) ln_fwd_kernel<T, VEC, 2, 2, false><<<grid, 256, 0, s>>>(p);
  else if (nv == 3) ln_fwd_kernel<T, VEC, 3, 1, false><<<grid, 256, 0, s>>>(p);
  else ln_fwd_kernel<T, VEC, 4, 1, false><<<grid, 256, 0, s>>>(p);
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
  return launch_after(ln_parts_kernel<T>, dim3((2u * p.cols + 31) / 32), dim3(256), 0, s, q);
}

template <typename T, bool VEC>
cudaError_t bwd(LnBwdParams p, int sms, cudaStream_t s, int* launches) {
  const bool params = p.dw || p.db;
  cudaError_t e;
  if (p.cols > LN_BWD_MAX_COLS) {
    if (params) {
      const int slabs = static_cast<int>(p.rows < 1 ? 1 : p.rows < 64 ? p.rows : 64);
      ln_bwd_wide_params_kernel<T><<<dim3((p.cols + 255) / 256, slabs), 256, 0, s>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      if ((e = add_parts<T>(p, slabs, s)) != cudaSuccess) return e;
      *launches += 2;
    }
    if (p.rows == 0) return cudaSuccess;
    const int grid = static_cast<int>(p.rows < 2 * sms ? p.rows : 2 * sms);
    ln_bwd_wide_kernel<T, VEC><<<grid, 1024, 0, s>>>(p);
    *launches += 1;
    return cudaGetLastError();
  }
  const int pieces = (p.cols + 7) / 8;
  p.tpr = pieces <= 32 ? pow2_at_least(pieces) : (pieces + 31) / 32 * 32;
  const int r = p.tpr <= 512 ? 4 : 1, most = p.tpr <= 512 ? 512 : 1024;
  p.groups = most / p.tpr;
  // whole warps only: groups of fewer than 32 threads fill them
  const int threads = p.groups * p.tpr;
  const long long blocks = (p.rows + r - 1) / r, want = (blocks + p.groups - 1) / p.groups;
  int grid = static_cast<int>(want < sms ? want : sms);
  if (grid > LN_MAX_PARTS) grid = LN_MAX_PARTS;
  if (grid < 1) grid = 1;                   // no rows: the sums are zero, and written
  if (grid == 1 || !params) p.parts = nullptr;
  const size_t smem = params ? static_cast<size_t>(threads) * 16 * sizeof(float) : 0;
  auto kernel = r == 4 ? ln_bwd_kernel<T, VEC, 4, 512> : ln_bwd_kernel<T, VEC, 1, 1024>;
  if (smem > 48 * 1024 &&
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
