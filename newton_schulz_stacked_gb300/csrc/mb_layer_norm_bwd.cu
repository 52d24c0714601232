// Layer norm over the rows of [rows, cols], backward, with the reduction of the weight's and bias's
// gradients over the rows.  All arithmetic is fp32.
//
//   h = (x - m) r;  g = dy w;  dx = r (g - mean_j g - h mean_j(g h))
//   dw = sum_rows dy h;  db = sum_rows dy
//
// HBM bounds it (x and dy are read, dx is written once): both sums over a row and the sums over
// the rows come from the same pass.
#include "mb_layer_norm.cuh"

namespace mb {
namespace {

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
// for bit).  SHIFT: a group's rows are a multiple of 16 bytes apart, so that it keeps its columns.
template <typename T, Access A, int R, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 288 ? 2 : 1) ln_bwd_kernel(const LnBwdParams p) {
  begin_after_previous();
  extern __shared__ float dyn[];                       // [16][threads] at the end
  __shared__ float part[2][MAXT / 32][2 * R];
  __shared__ int shifts[256];
  using P = Piece<T, A>;
  const int tpr = p.tpr, cols = p.cols, groups = p.groups;
  const int g = threadIdx.x / tpr;
  Place at{cols, tpr, static_cast<int>(threadIdx.x) - g * tpr, 0};
  const float inv_n = 1.f / static_cast<float>(cols);
  // every group of the CTA goes round the same number of times (a warp may hold several groups)
  const long long step = static_cast<long long>(groups) * R, stride = step * gridDim.x;
  P next_x[R], next_dy[R];
  float next_m[R], next_rs[R];
  long long base = blockIdx.x * step;
  if (A == Access::SHIFT) {
    at.shift = shift_of(static_cast<const T*>(p.x) + (base + g) * p.x_stride);
    if (at.t == 0) shifts[g] = at.shift;
  }
  auto fetch = [&](long long row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = row0 + g * R + r;
      const bool on = row < p.rows, edge = row == 0 || row == p.rows - 1;
      next_x[r].load(static_cast<const T*>(p.x) + row * p.x_stride, at, 0, on, edge);
      next_dy[r].load(static_cast<const T*>(p.dy) + row * p.dy_stride, at, 0, on, edge);
      next_m[r] = on ? p.mean[row] : 0.f;
      next_rs[r] = on ? p.rstd[row] : 0.f;
    }
  };
  fetch(base);
  float2 w[4], dw[4], db[4];
  param_pairs<T, A>(p.w, p.w_f32, 1.f, at, 0, w);
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
      get_pairs(next_x[r], at, 0, h[r]);
      get_pairs(next_dy[r], at, 0, df);
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
        store_pairs<P>(static_cast<T*>(p.dx) + (row0 + r) * p.dx_stride, at, 0, h[r]);
      }
    }
  }
  if (!p.dw && !p.db) return;
  // the CTA's sum over its groups: [16 values][threads], so that threads touch neighbouring words
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    dyn[j * blockDim.x + threadIdx.x] = j & 1 ? dw[j / 2].y : dw[j / 2].x;
    dyn[(8 + j) * blockDim.x + threadIdx.x] = j & 1 ? db[j / 2].y : db[j / 2].x;
  }
  __syncthreads();
  const int count = A == Access::SHIFT ? 2 * cols : 16 * tpr;
  for (int e = threadIdx.x; e < count; e += blockDim.x) {
    float sum = 0.f;
    int c, k;                                          // the column, and whether of dw or db
    if constexpr (A == Access::SHIFT) {
      k = e >= cols;
      c = e - k * cols;
      for (int u = 0; u < groups; ++u) {
        const int i = c + shifts[u];
        sum += dyn[(k * 8 + (i & 7)) * blockDim.x + u * tpr + (i >> 3)];
      }
    } else {
      const int i = e / tpr, tt = e - i * tpr;
      const Place there{cols, tpr, tt, 0};
      if (!P::in(there, 0, i & 7)) continue;
      for (int u = 0; u < groups; ++u) sum += dyn[i * blockDim.x + u * tpr + tt];
      c = P::col(there, 0, i & 7);
      k = i >> 3;
    }
    if (p.parts) {
      p.parts[(static_cast<size_t>(blockIdx.x) * 2 + k) * cols + c] = sum;
    } else {
      void* out = k ? p.db : p.dw;
      if (out) put_param_grad(out, p.w_f32, c, sum, T());
    }
  }
}

// Threads of a CTA (one per SM) of the kernel below, by what the registers of NV pieces allow: more of
// them spill (2^26 fp32 elements in rows of 768: 126 us, with 384 threads 143; of 512 122 and, with 512
// threads, 137; 2^27 bf16 elements in unaligned rows of 511 162 and 205, of 761 170 and 263).
template <typename T, Access A, int NV>
constexpr int BWD_THREADS = NV == 2 ? (sizeof(T) == 2 && A == Access::VEC ? 512 : 384)
                          : NV == 3 && sizeof(T) == 2 && A == Access::VEC ? 384 : 256;

// Most pieces of a row in this kernel: 16-bit aligned rows of more than 768 elements are faster through
// the ring below (2^27 bf16 elements in rows of 1024 131 us and not 143), fp32 ones not (2^26 in rows of
// 1024 131 and 122).
template <typename T, Access A>
constexpr int WARP_PIECES = A == Access::VEC && sizeof(T) == 2 ? 96 : 128;

// Rows of 257 to 1024 elements: a warp holds a row in NV pieces per lane and sums over it by
// exchanges alone; the next row is already being loaded.  Sums of the gradient as above.
template <typename T, Access A, int NV>
__global__ void __launch_bounds__(BWD_THREADS<T, A, NV>, 1) ln_bwd_warp_kernel(const LnBwdParams p) {
  begin_after_previous();
  extern __shared__ __align__(16) float dyn[];         // the weight; at the end [warps][NV][16][32] sums
  using P = Piece<T, A>;
  constexpr int WARPS = BWD_THREADS<T, A, NV> / 32;
  static_assert(A != Access::SHIFT, "single elements are as fast here");
  const int cols = p.cols, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inv_n = 1.f / static_cast<float>(cols);
  const long long stride = static_cast<long long>(gridDim.x) * WARPS;
  long long row = static_cast<long long>(blockIdx.x) * WARPS + warp;
  P next_x[NV], next_dy[NV];
  float next_m = 0.f, next_rs = 0.f;
  const T *x = static_cast<const T*>(p.x) + row * p.x_stride, *dy = static_cast<const T*>(p.dy) + row * p.dy_stride;
  T* dx = static_cast<T*>(p.dx) + row * p.dx_stride;
  const Place at{cols, 32, lane, 0};
  auto fetch = [&](long long r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      next_x[v].load(x, at, v, true, false);
      next_dy[v].load(dy, at, v, true, false);
    }
    next_m = p.mean[r];
    next_rs = p.rstd[r];
    x += stride * p.x_stride;
    dy += stride * p.dy_stride;
  };
  if (row < p.rows) fetch(row);
  Staged<A, NV>::template put<T>(dyn, p.w, p.w_f32, 1.f, cols, 32);
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
      Staged<A, NV>::get(dyn, at, v, w);
      get_pairs(next_x[v], at, v, h[v]);
      get_pairs(next_dy[v], at, v, gr[v]);
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
      store_pairs<P>(dx, at, v, h[v]);
    }
    dx += stride * p.dx_stride;
  }
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
    const int j = (e >> 5) & 7, v = e >> 9, k = (e >> 8) & 1;      // k: of dw or db
    const Place there{cols, 32, e & 31, 0};
    if (!P::in(there, v, j)) continue;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < WARPS; ++u) sum += dyn[u * NV * 512 + e];
    const int c = P::col(there, v, j);
    if (p.parts) {
      p.parts[(static_cast<size_t>(blockIdx.x) * 2 + k) * cols + c] = sum;
    } else {
      void* out = k ? p.db : p.dw;
      if (out) put_param_grad(out, p.w_f32, c, sum, T());
    }
  }
}

// Longer aligned rows, up to 8192 elements: a group of up to 512 threads holds a row, 16 elements per
// thread in 16-byte chunks.  Every thread copies its own chunks of the next rows into its own places
// of a ring in shared memory (so nothing but its own wait orders them), and a row is finished while
// the next one's sums are under way: one barrier per row, behind a row's worth of other work.  2^27
// bf16 elements in rows of 1536 to 4096 take 125 to 151 us, of 8192 135 (6.0 TB/s; with the next row in
// registers 167 to 179, and 230); fp32 245 to 277 (of 8192 414).  Rows of 4097 to 5376 leave a third to
// half of the threads out and take 163 to 174: 24 elements per thread, so that two fit, spill (185).
template <typename T>
struct Ring {
  static constexpr int E = 16 / sizeof(T);             // elements of a chunk
  static constexpr int NC = 16 / E;                    // chunks per thread
  static constexpr int R = 4 / NC;                     // rows at a time
  static constexpr int STAGES = 3;                     // times R rows: 192 KB with 512 threads
  static constexpr int MAX_THREADS = 512;
  static size_t bytes(int threads) { return static_cast<size_t>(STAGES) * R * 2 * NC * threads * 16; }
};

template <typename T>
__global__ void __launch_bounds__(Ring<T>::MAX_THREADS, 1) ln_bwd_ring_kernel(const LnBwdParams p) {
  begin_after_previous();
  using Shape = Ring<T>;
  constexpr int E = Shape::E, NC = Shape::NC, NP = E / 2, STAGES = Shape::STAGES, R = Shape::R;
  constexpr int WARPS = Shape::MAX_THREADS / 32;
  extern __shared__ __align__(16) float dyn[];         // the ring [STAGES][R][x, dy][NC][threads]; at the end [32][threads] sums
  __shared__ float part[2][WARPS][2 * R];              // of every row: sum g, sum g h
  const int tpr = p.tpr, cols = p.cols, groups = p.groups, threads = blockDim.x;
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv_n = 1.f / static_cast<float>(cols);
  uint4* const mine = reinterpret_cast<uint4*>(dyn) + threadIdx.x;
  auto place = [&](int stage, int r, int k, int c) { return mine + (((stage * R + r) * 2 + k) * NC + c) * threads; };
  auto col = [&](int c) { return (c * tpr + t) * E; };

  // R rows at a time; they go round the CTAs first
  const long long stride = static_cast<long long>(gridDim.x) * groups * R;
  long long row = (blockIdx.x + static_cast<long long>(gridDim.x) * g) * R, ahead = row;
  const T *x = static_cast<const T*>(p.x) + row * p.x_stride, *dy = static_cast<const T*>(p.dy) + row * p.dy_stride;
  auto fetch = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (ahead + r < p.rows) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (col(c) < cols) {
            copy_16(place(stage, r, 0, c), x + r * p.x_stride + col(c));
            copy_16(place(stage, r, 1, c), dy + r * p.dy_stride + col(c));
          }
        }
      }
    }
    copies_end_group();
    ahead += stride;
    x += stride * p.x_stride;
    dy += stride * p.dy_stride;
  };
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (col(c) >= cols) {
      for (int k = 0; k < STAGES * R * 2; ++k) *place(0, 0, k, c) = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s);
  float next_m[R], next_rs[R];
  auto fetch_stats = [&](long long row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool on = row0 + r < p.rows;
      next_m[r] = on ? p.mean[row0 + r] : 0.f;
      next_rs[r] = on ? p.rstd[row0 + r] : 0.f;
    }
  };
  fetch_stats(row);
  float2 w[NC][NP], dw[NC][NP], db[NC][NP];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const bool in = col(c) < cols;
      w[c][j].x = in ? param<T>(p.w, p.w_f32, 1.f, col(c) + 2 * j) : 0.f;
      w[c][j].y = in ? param<T>(p.w, p.w_f32, 1.f, col(c) + 2 * j + 1) : 0.f;
      dw[c][j] = db[c][j] = both(0.f);
    }
  }

  float m[R], rs[R];                                   // of the rows to be finished
  int stage = 0, before = STAGES - 1, parity = 0;      // places of the present rows and of the ones before
  T* dx = static_cast<T*>(p.dx) + row * p.dx_stride;
  auto finish = [&](int from, int half, long long row0) {
    float sums[2 * R];
    sums_of_warps<2 * R>(part[half] + g * (tpr >> 5), tpr >> 5, lane, sums);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (R > 1 && row0 + r >= p.rows) break;
      const float2 c1 = both(-sums[2 * r] * inv_n), c2 = both(-sums[2 * r + 1] * inv_n), scale = both(rs[r]);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float2 h[NP], d[NP];
        chunk_pairs(*place(from, r, 0, c), h, T());
        chunk_pairs(*place(from, r, 1, c), d, T());
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          h[j] = __fmul2_rn(__fadd2_rn(h[j], both(-m[r])), scale);
          h[j] = __fmul2_rn(__ffma2_rn(d[j], w[c][j], __ffma2_rn(h[j], c2, c1)), scale);
        }
        if (col(c) < cols) *reinterpret_cast<uint4*>(dx + r * p.dx_stride + col(c)) = chunk_of(h, T());
      }
    }
    dx += stride * p.dx_stride;
  };
  bool first = true;
  for (; row < p.rows; row += stride) {
    copies_wait<STAGES - 2>();
    float m_now[R], rs_now[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m_now[r] = next_m[r];
      rs_now[r] = next_rs[r];
    }
    fetch_stats(row + stride);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 s1 = both(0.f), s2 = both(0.f);
      if (R == 1 || row + r < p.rows) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float2 h[NP], d[NP];
          chunk_pairs(*place(stage, r, 0, c), h, T());
          chunk_pairs(*place(stage, r, 1, c), d, T());
#pragma unroll
          for (int j = 0; j < NP; ++j) {               // past the row dy is 0, and h of no consequence
            h[j] = __fmul2_rn(__fadd2_rn(h[j], both(-m_now[r])), both(rs_now[r]));
            const float2 gr = __fmul2_rn(d[j], w[c][j]);
            s1 = __fadd2_rn(s1, gr);
            s2 = __ffma2_rn(gr, h[j], s2);
            dw[c][j] = __ffma2_rn(d[j], h[j], dw[c][j]);
            db[c][j] = __fadd2_rn(db[c][j], d[j]);
          }
        }
      }
      s[2 * r] = s1.x + s1.y;
      s[2 * r + 1] = s2.x + s2.y;
    }
    int which;
    const float sum = warp_sums<2 * R>(s, lane, &which);
    if ((lane & (16 / R - 1)) == 0) part[parity][warp][which] = sum;
    if (!first) finish(before, parity ^ 1, row - stride);
    first = false;
    fetch(before);                                     // its rows have been finished
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = m_now[r];
      rs[r] = rs_now[r];
    }
    before = stage;
    stage = stage + 1 < STAGES ? stage + 1 : 0;
    parity ^= 1;
    group_barrier(1 + g, tpr);
  }
  if (!first) finish(before, parity ^ 1, row - stride);
  if (!p.dw && !p.db) return;
  copies_wait<0>();
  __syncthreads();
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      dyn[(c * E + j) * threads + threadIdx.x] = j & 1 ? dw[c][j / 2].y : dw[c][j / 2].x;
      dyn[(16 + c * E + j) * threads + threadIdx.x] = j & 1 ? db[c][j / 2].y : db[c][j / 2].x;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 32 * tpr; e += threads) {
    const int i = e / tpr, tt = e - i * tpr, k = i >> 4, n = i & 15;   // k: of dw or db
    const int c = (n / E * tpr + tt) * E + n % E;
    if (c >= cols) continue;
    float sum = 0.f;
    for (int u = 0; u < groups; ++u) sum += dyn[i * threads + u * tpr + tt];
    if (p.parts) {
      p.parts[(static_cast<size_t>(blockIdx.x) * 2 + k) * cols + c] = sum;
    } else {
      void* out = k ? p.db : p.dw;
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
  begin_after_previous();
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
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
template <typename T, Access A>
__global__ void __launch_bounds__(1024) ln_bwd_wide_kernel(const LnBwdParams p) {
  begin_after_previous();
  __shared__ float smem[32];
  using P = Piece<T, A>;
  const Place at{p.cols, static_cast<int>(blockDim.x), static_cast<int>(threadIdx.x), 0};
  const int nv = (p.cols + 8 * at.tpr - 1) / (8 * at.tpr);
  const float inv_n = 1.f / static_cast<float>(p.cols);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* dr = static_cast<const T*>(p.dy) + row * p.dy_stride;
    const float2 m = both(-p.mean[row]), rs = both(p.rstd[row]);
    float2 s1 = both(0.f), s2 = both(0.f), h[4], g[4], w[4];
    P x, dy;
    auto piece = [&](int v) {                          // h and g of piece v
      x.load(xr, at, v, true, false);
      dy.load(dr, at, v, true, false);
      param_pairs<T, A>(p.w, p.w_f32, 1.f, at, v, w);
      get_pairs(x, at, v, h);
      get_pairs(dy, at, v, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = __fmul2_rn(__fadd2_rn(h[j], m), rs);
        g[j] = __fmul2_rn(g[j], w[j]);
      }
    };
    for (int v = 0; v < nv; ++v) {
      piece(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s1 = __fadd2_rn(s1, g[j]);
        s2 = __ffma2_rn(g[j], h[j], s2);
      }
    }
    const float c1 = cta_sum(s1.x + s1.y, smem) * inv_n, c2 = cta_sum(s2.x + s2.y, smem) * inv_n;
    for (int v = 0; v < nv; ++v) {
      piece(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __fmul2_rn(__fadd2_rn(g[j], __ffma2_rn(h[j], both(-c2), both(-c1))), rs);
      store_pairs<P>(static_cast<T*>(p.dx) + row * p.dx_stride, at, v, h);
    }
  }
}

// ... and, before it (dx may lie over x or dy), the weight's gradient with one thread per
// column and slab of rows.
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_wide_params_kernel(const LnBwdParams p) {
  begin_after_previous();
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

// How groups of threads share rows: up to 256 elements, and unaligned ones of more than 1024.  256
// threads in two CTAs of 128 registers; longer rows 576 threads per SM at 96 registers in two or
// three CTAs up to 2304 elements, then one CTA of 128 or 64 registers.
struct GroupShape {
  int tpr, groups;      // threads per row, rows side by side in a CTA
  int most;             // the kernel's MAXT
  int ctas;             // per SM
};
GroupShape group_shape(int pieces) {
  if (pieces <= 32) {
    const int tpr = pow2_at_least(pieces);
    return {tpr, 256 / tpr, 256, 2};
  }
  const int tpr = (pieces + 31) / 32 * 32, most = tpr <= 288 ? 288 : tpr <= 512 ? 512 : 1024;
  return {tpr, most / tpr, most, most == 288 ? std::min(3, 576 / (most / tpr * tpr)) : 1};
}
template <typename T>
cudaError_t add_parts(const LnBwdParams& p, int n, cudaStream_t s) {
  LnPartsParams q{p.parts, n, p.cols, p.w_f32, p.dw, p.db};
  return launch_after(ln_parts_kernel<T>, dim3((2u * p.cols + 31) / 32), dim3(1024), 0, s, q);
}

template <typename T, Access A>
cudaError_t bwd_wide(const LnBwdParams& p, int sms, cudaStream_t s, int* launches) {
  cudaError_t e;
  if (p.dw || p.db) {
    const int slabs = static_cast<int>(p.rows < 1 ? 1 : p.rows < LN_WIDE_SLABS ? p.rows : LN_WIDE_SLABS);
    if ((e = launch_after(ln_bwd_wide_params_kernel<T>, dim3((p.cols + 255) / 256, slabs), dim3(256), 0, s, p)) != cudaSuccess)
      return e;
    if ((e = add_parts<T>(p, slabs, s)) != cudaSuccess) return e;
    *launches += 2;
  }
  if (p.rows == 0) return cudaSuccess;
  *launches += 1;
  return launch_after(ln_bwd_wide_kernel<T, A>, dim3(cta_count(p.rows, 1, 2 * sms)), dim3(1024), 0, s, p);
}

// A kernel and its launch.
struct BwdLaunch {
  void (*kernel)(LnBwdParams);
  int grid, threads, rows_per_cta;
  size_t smem, most_smem;      // of this launch; of any launch of the kernel
};

template <typename T, Access A>
BwdLaunch bwd_warp_launch(const LnBwdParams& p, int pieces, int sms) {
  const bool params = p.dw || p.db;
  const int nv = (pieces + 31) / 32;
  BwdLaunch l{};
  l.threads = nv == 2 ? BWD_THREADS<T, A, 2> : nv == 3 ? BWD_THREADS<T, A, 3> : BWD_THREADS<T, A, 4>;
  l.rows_per_cta = l.threads / 32;
  l.grid = cta_count(p.rows, l.rows_per_cta, std::min(LN_MAX_PARTS, sms));
  const int staged = nv == 2 ? Staged<A, 2>::floats(32) : nv == 3 ? Staged<A, 3>::floats(32) : Staged<A, 4>::floats(32);
  l.most_smem = static_cast<size_t>(std::max(staged, 16 * nv * l.threads)) * sizeof(float);
  l.smem = params ? l.most_smem : static_cast<size_t>(staged) * sizeof(float);
  l.kernel = nv == 2 ? ln_bwd_warp_kernel<T, A, 2> : ln_bwd_warp_kernel<T, A, 3>;
  if constexpr (WARP_PIECES<T, A> > 96) {
    if (nv == 4) l.kernel = ln_bwd_warp_kernel<T, A, 4>;
  }
  return l;
}

template <typename T>
BwdLaunch bwd_ring_launch(LnBwdParams& p, int sms) {
  using Shape = Ring<T>;
  p.tpr = (p.cols + 16 * 32 - 1) / (16 * 32) * 32;
  p.groups = Shape::MAX_THREADS / p.tpr;
  BwdLaunch l{};
  l.threads = p.groups * p.tpr;
  l.rows_per_cta = p.groups * Shape::R;
  l.grid = cta_count(p.rows, Shape::R, std::min(LN_MAX_PARTS, sms));
  l.smem = Shape::bytes(l.threads);
  l.most_smem = Shape::bytes(Shape::MAX_THREADS);
  l.kernel = ln_bwd_ring_kernel<T>;
  return l;
}
template <typename T, Access A>
BwdLaunch bwd_group_launch(LnBwdParams& p, int pieces, int sms) {
  const GroupShape g = group_shape(pieces);
  p.tpr = g.tpr;
  p.groups = g.groups;
  constexpr int R = A == Access::VEC ? 2 : 1;
  BwdLaunch l{};
  l.threads = g.groups * g.tpr;
  l.rows_per_cta = g.groups * R;
  l.grid = cta_count(p.rows, l.rows_per_cta, std::min(LN_MAX_PARTS, g.ctas * sms));
  l.smem = p.dw || p.db ? static_cast<size_t>(l.threads) * 16 * sizeof(float) : 0;
  l.most_smem = static_cast<size_t>(g.most) * 16 * sizeof(float);
  l.kernel = ln_bwd_kernel<T, A, R, 256>;
  if constexpr (A != Access::VEC) {
    if (g.most == 288) l.kernel = ln_bwd_kernel<T, A, 1, 288>;
    if (g.most == 512) l.kernel = ln_bwd_kernel<T, A, 1, 512>;
    if (g.most == 1024) l.kernel = ln_bwd_kernel<T, A, 1, 1024>;
  }
  return l;
}

template <typename T, Access A>
cudaError_t bwd(LnBwdParams p, int sms, cudaStream_t s, int* launches) {
  const int pieces = (p.cols + (A == Access::SHIFT ? 14 : 7)) / 8;
  BwdLaunch l;
  if constexpr (A == Access::SHIFT) {
    l = bwd_group_launch<T, A>(p, pieces, sms);
    // a group's rows lie grid * rows_per_cta apart, which has to be a multiple of 16 bytes whatever
    // the row; eight rows always are one
    while (l.grid > 1 && l.grid * l.rows_per_cta % 8 != 0) --l.grid;
    if (l.grid * l.rows_per_cta % 8 != 0 && p.rows > l.rows_per_cta) return bwd<T, Access::SCALAR>(p, sms, s, launches);
  } else {
    if (pieces > 32 && pieces <= WARP_PIECES<T, A>) l = bwd_warp_launch<T, A>(p, pieces, sms);
    else if (A == Access::VEC && pieces > 32) l = bwd_ring_launch<T>(p, sms);
    else l = bwd_group_launch<T, A>(p, pieces, sms);
  }
  if (l.grid == 1 || !(p.dw || p.db)) p.parts = nullptr;
  cudaError_t e;
  if ((e = allow_shared(l.kernel, l.smem, l.most_smem)) != cudaSuccess) return e;
  if ((e = launch_after(l.kernel, dim3(l.grid), dim3(l.threads), l.smem, s, p)) != cudaSuccess) return e;
  *launches += 1;
  if (!p.parts) return cudaSuccess;
  *launches += 1;
  return add_parts<T>(p, l.grid, s);
}

template <typename T>
cudaError_t bwd_any(const LnBwdParams& p, int sms, cudaStream_t s, int* launches) {
  constexpr int SIZE = sizeof(T);
  const bool vec = p.cols % 8 == 0 && aligned_rows(p.x, p.x_stride, SIZE, p.rows) &&
                   aligned_rows(p.dy, p.dy_stride, SIZE, p.rows) && aligned_rows(p.dx, p.dx_stride, SIZE, p.rows) &&
                   aligned(p.w);
  if (p.cols > LN_BWD_MAX_COLS)
    return vec ? bwd_wide<T, Access::VEC>(p, sms, s, launches) : bwd_wide<T, Access::SCALAR>(p, sms, s, launches);
  if (vec) return bwd<T, Access::VEC>(p, sms, s, launches);
  // not where a warp holds a row and reads 64 or 128 bytes at a time by single elements too: 2^26 bf16
  // elements in rows of 777 take 151 us so and 90 by single ones, of 303 188 and 115; in rows of 201 145 and
  // 165, of 2003 123 and 313 (fp32: 169 and 127, 201 and 145; 165 and 190, 154 and 211)
  if ((p.cols + 14 <= 256 || p.cols > 1024) && p.cols + 14 <= LN_BWD_MAX_COLS && shiftable(p.x_stride, p.cols, p.rows) &&
      shiftable(p.dy_stride, p.cols, p.rows) && same_shift(p.x, p.x_stride, p.dy, p.dy_stride, SIZE, p.rows) &&
      same_shift(p.x, p.x_stride, p.dx, p.dx_stride, SIZE, p.rows))
    return bwd<T, Access::SHIFT>(p, sms, s, launches);
  return bwd<T, Access::SCALAR>(p, sms, s, launches);
}

}  // namespace

cudaError_t launch_layer_norm_backward(LnBwdParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 0;
  if (type == MB_F32) return bwd_any<float>(p, sms, s, launches);
  if (type == MB_BF16) return bwd_any<__nv_bfloat16>(p, sms, s, launches);
  return bwd_any<__half>(p, sms, s, launches);
}

}  // namespace mb
