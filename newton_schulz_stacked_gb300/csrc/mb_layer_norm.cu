// Layer norm over the rows of [rows, cols], forward.  All arithmetic is fp32.
//
//   m = mean_j x_j;  r = 1 / sqrt(mean_j (x_j - m)^2 + eps);  h = (x - m) r;  y = h w + b
//
// HBM bounds it (the elements are read and written once): a row stays in its threads' registers
// through the statistics and the result.  49152 x 1024 bf16 take 34.8 us (5.8 TB/s), 2^26 elements in
// rows of 32 to 4096 5.2 to 6.3 TB/s.
#include "mb_layer_norm.cuh"

namespace mb {
namespace {

// a += the squares of the piece's differences from m, within the row.
template <typename P>
__device__ __forceinline__ void add_squares(const P& x, float m, const Place& p, int v, float2& a) {
  float2 f[4];
  get_pairs(x, p, v, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 d = __fadd2_rn(f[j], both(-m));
    if (!P::in(p, v, 2 * j)) d.x = 0.f;
    if (!P::in(p, v, 2 * j + 1)) d.y = 0.f;
    a = __ffma2_rn(d, d, a);
  }
}
template <typename P>
__device__ __forceinline__ void add_piece(const P& x, const Place& p, int v, float2& a) {
  float2 f[4];
  get_pairs(x, p, v, f);
  a = __fadd2_rn(a, __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3])));
}
// f <- (f - m) r w + b
__device__ __forceinline__ void normalise(float2 (&f)[4], float m, float r, const float2 (&w)[4], const float2 (&b)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[j], both(-m)), both(r)), w[j], b[j]);
}

// CTAs of 256 threads per SM of the kernel below: 80 registers for up to four 16-bit pieces, else
// 128, and 255 for 16 fp32 pieces.
template <typename T, Access A, int NV>
constexpr int FWD_CTAS = A != Access::SCALAR && sizeof(T) == 2 && NV <= 4 ? 3 : sizeof(T) == 4 && NV > 8 ? 1 : 2;

// Rows of up to 4096 elements (512 by single elements): tpr lanes of a warp hold a row in NV pieces each and take R rows at a
// time; no barrier in the loop.  Up to four pieces the next rows are already being loaded (AHEAD);
// with more, a warp's own row is enough in flight.  Weight and bias wait in shared memory.  The
// variance sums squares of differences from the mean, over the registers: no cancellation however
// far the mean is from zero.
template <typename T, Access A, int NV, int R>
__global__ void __launch_bounds__(256, FWD_CTAS<T, A, NV>) ln_fwd_kernel(const LnFwdParams p) {
  begin_after_previous();
  extern __shared__ __align__(16) float wb[];          // the weight, then the bias
  using P = Piece<T, A>;
  constexpr bool AHEAD = A != Access::SCALAR && NV <= 4;
  const int tpr = p.tpr, g = threadIdx.x / tpr, groups = blockDim.x / tpr;
  Place at{p.cols, tpr, static_cast<int>(threadIdx.x) % tpr, 0};
  const float inv_n = 1.f / static_cast<float>(p.cols);
  const long long step = static_cast<long long>(groups) * R, stride = step * gridDim.x;
  P x[R][NV], next[AHEAD ? R : 1][AHEAD ? NV : 1];
  auto fetch = [&](auto& to, long long base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * groups + g;
      const T* from = static_cast<const T*>(p.x) + row * p.x_stride;
      if (A == Access::SHIFT) at.shift = shift_of(from);
#pragma unroll
      for (int v = 0; v < NV; ++v) to[r][v].load(from, at, v, row < p.rows, row == 0 || row == p.rows - 1);
    }
  };
  long long base = blockIdx.x * step;
  if constexpr (AHEAD) fetch(next, base);
  Staged<A, NV>::template put<T>(wb, p.w, p.w_f32, 1.f, p.cols, tpr);
  Staged<A, NV>::template put<T>(wb + Staged<A, NV>::floats(tpr), p.b, p.w_f32, 0.f, p.cols, tpr);
  __syncthreads();
  for (; base < p.rows; base += stride) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < NV; ++v) x[r][v] = next[r][v];
      if (base + stride < p.rows) fetch(next, base + stride);
    } else {
      fetch(x, base);
    }
    float s[R], m[R];
    int shift[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      shift[r] = A == Access::SHIFT ? shift_of(static_cast<const T*>(p.x) + (base + r * groups + g) * p.x_stride) : 0;
      at.shift = shift[r];
      float2 a = both(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v) add_piece(x[r][v], at, v, a);    // elements past the row are zero
      s[r] = a.x + a.y;
    }
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], o);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = s[r] * inv_n;
      at.shift = shift[r];
      float2 a = both(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v) add_squares(x[r][v], m[r], at, v, a);
      s[r] = a.x + a.y;
    }
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], o);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = rsqrtf(fmaf(s[r], inv_n, p.eps));
      const long long row = base + r * groups + g;
      if (at.t == 0 && row < p.rows) {
        if (p.mean) p.mean[row] = m[r];
        if (p.rstd) p.rstd[row] = s[r];
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 w[4], b[4];
      if (A != Access::SHIFT) {
        Staged<A, NV>::get(wb, at, v, w);
        Staged<A, NV>::get(wb + Staged<A, NV>::floats(tpr), at, v, b);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const long long row = base + r * groups + g;
        if (row < p.rows) {
          at.shift = shift[r];
          if (A == Access::SHIFT) {
            Staged<A, NV>::get(wb, at, v, w);
            Staged<A, NV>::get(wb + Staged<A, NV>::floats(tpr), at, v, b);
          }
          float2 f[4];
          get_pairs(x[r][v], at, v, f);
          normalise(f, m[r], s[r], w, b);
          store_pairs<P>(static_cast<T*>(p.y) + row * p.y_stride, at, v, f);
        }
      }
    }
  }
}

// Aligned rows through a ring in shared memory: a group of up to 512 threads holds a row, 16 elements
// per thread in 16-byte chunks, R rows at a time.  Every thread copies its own chunks of the next rows
// into its own places (so nothing but its own wait orders them).  While the sum of one set of rows is
// formed, the squares of the set before are, with the mean known, and the set before that is finished:
// one barrier per set, behind other work.  (Eight elements per thread, of 1024 threads, were slower:
// 2^27 bf16 elements in rows of 8192 136 us and not 107.)
template <typename T>
struct FwdRing {
  static constexpr int E = 16 / sizeof(T);             // elements of a chunk
  static constexpr int NC = 16 / E;                    // chunks per thread
  static constexpr int R = 4 / NC;                     // rows at a time
  static constexpr int STAGES = 5;                     // times R rows: 160 KB with 512 threads
  static constexpr int MAX_THREADS = 512;
  static size_t bytes(int threads) { return static_cast<size_t>(STAGES) * R * NC * threads * 16; }
};

template <typename T>
__global__ void __launch_bounds__(FwdRing<T>::MAX_THREADS, 1) ln_fwd_ring_kernel(const LnFwdParams p) {
  begin_after_previous();
  using Shape = FwdRing<T>;
  constexpr int E = Shape::E, NC = Shape::NC, NP = E / 2, STAGES = Shape::STAGES, R = Shape::R;
  extern __shared__ __align__(16) uint4 ring[];        // [STAGES][R][NC][threads]
  __shared__ float part[2][Shape::MAX_THREADS / 32][2 * R];        // sums of R rows, sums of squares of R
  const int tpr = p.tpr, cols = p.cols, threads = blockDim.x, groups = threads / tpr;
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv_n = 1.f / static_cast<float>(cols);
  uint4* const mine = ring + threadIdx.x;
  auto place = [&](int stage, int r, int c) { return mine + ((stage * R + r) * NC + c) * threads; };
  auto col = [&](int c) { return (c * tpr + t) * E; };

  // sets of R rows, which go round the CTAs first
  const long long stride = static_cast<long long>(gridDim.x) * groups * R;
  const long long row0 = (blockIdx.x + static_cast<long long>(gridDim.x) * g) * R;
  const int sets = row0 < p.rows ? static_cast<int>((p.rows - row0 + stride - 1) / stride) : 0;
  long long ahead = row0;
  const T* x = static_cast<const T*>(p.x) + row0 * p.x_stride;
  auto fetch = [&](int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (ahead + r < p.rows) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (col(c) < cols) copy_16(place(stage, r, c), x + r * p.x_stride + col(c));
      }
    }
    copies_end_group();
    ahead += stride;
    x += stride * p.x_stride;
  };
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (col(c) >= cols) {
      for (int k = 0; k < STAGES * R; ++k) *place(0, k, c) = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int s = 0; s < STAGES - 2; ++s) fetch(s);
  float2 w[NC][NP], b[NC][NP];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const bool in = col(c) < cols;
      w[c][j].x = in ? param<T>(p.w, p.w_f32, 1.f, col(c) + 2 * j) : 0.f;
      w[c][j].y = in ? param<T>(p.w, p.w_f32, 1.f, col(c) + 2 * j + 1) : 0.f;
      b[c][j].x = in ? param<T>(p.b, p.w_f32, 0.f, col(c) + 2 * j) : 0.f;
      b[c][j].y = in ? param<T>(p.b, p.w_f32, 0.f, col(c) + 2 * j + 1) : 0.f;
    }
  }

  float m1[R], m2[R];                                  // means of the sets one and two before
#pragma unroll
  for (int r = 0; r < R; ++r) m1[r] = m2[r] = 0.f;
  int at0 = 0, at1 = STAGES - 1, at2 = STAGES - 2;     // places of the present set and of those before
  long long row = row0 - 2 * stride;                   // of the set to be finished
  T* y = static_cast<T*>(p.y) + row * p.y_stride;
  for (int k = 0; k < sets + 2; ++k) {
    const int parity = k & 1;
    float sums[2 * R], s[2 * R];
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) sums[i] = s[i] = 0.f;
    if (k > 0) {
      sums_of_warps<2 * R>(part[parity ^ 1] + g * (tpr >> 5), tpr >> 5, lane, sums);
    }
    copies_wait<STAGES - 3>();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m2[r] = m1[r];
      m1[r] = sums[r] * inv_n;
      float2 a = both(0.f), q = both(0.f);
      if (k < sets && row + 2 * stride + r < p.rows) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {                 // past the row there are zeros
          float2 f[NP];
          chunk_pairs(*place(at0, r, c), f, T());
#pragma unroll
          for (int j = 0; j < NP; ++j) a = __fadd2_rn(a, f[j]);
        }
      }
      if (k > 0 && k <= sets && row + stride + r < p.rows) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (col(c) < cols) {
            float2 f[NP];
            chunk_pairs(*place(at1, r, c), f, T());
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              f[j] = __fadd2_rn(f[j], both(-m1[r]));
              q = __ffma2_rn(f[j], f[j], q);
            }
          }
        }
      }
      s[r] = a.x + a.y;
      s[R + r] = q.x + q.y;
    }
    int which;
    const float sum = warp_sums<2 * R>(s, lane, &which);
    if ((lane & (16 / R - 1)) == 0) part[parity][warp][which] = sum;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (k > 1 && row + r < p.rows) {
        const float rs = rsqrtf(fmaf(sums[R + r], inv_n, p.eps));
        if (t == 0) {
          if (p.mean) p.mean[row + r] = m2[r];
          if (p.rstd) p.rstd[row + r] = rs;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float2 f[NP];
          chunk_pairs(*place(at2, r, c), f, T());
#pragma unroll
          for (int j = 0; j < NP; ++j)
            f[j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[j], both(-m2[r])), both(rs)), w[c][j], b[c][j]);
          if (col(c) < cols) *reinterpret_cast<uint4*>(y + r * p.y_stride + col(c)) = chunk_of(f, T());
        }
      }
    }
    row += stride;
    y += stride * p.y_stride;
    fetch(at2);                                        // its set has been finished
    at2 = at1;
    at1 = at0;
    at0 = at0 + 1 < STAGES ? at0 + 1 : 0;
    group_barrier(1 + g, tpr);
  }
}

// Rows of up to 32768 elements (16384 by single elements): one CTA per row, which its threads hold
// in NV pieces each; several CTAs per SM keep loads in flight while others wait at their sums.
template <typename T, Access A, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) ln_fwd_cta_kernel(const LnFwdParams p) {
  begin_after_previous();
  __shared__ float smem[32];
  using P = Piece<T, A>;
  const Place at{p.cols, static_cast<int>(blockDim.x), static_cast<int>(threadIdx.x), 0};
  const float inv_n = 1.f / static_cast<float>(p.cols);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    P x[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) x[v].load(static_cast<const T*>(p.x) + row * p.x_stride, at, v, true, false);
    float2 a = both(0.f), q = both(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) add_piece(x[v], at, v, a);
    const float m = cta_sum(a.x + a.y, smem) * inv_n;
#pragma unroll
    for (int v = 0; v < NV; ++v) add_squares(x[v], m, at, v, q);
    const float rs = rsqrtf(fmaf(cta_sum(q.x + q.y, smem), inv_n, p.eps));
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = m;
      if (p.rstd) p.rstd[row] = rs;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 f[4], w[4], b[4];
      param_pairs<T, A>(p.w, p.w_f32, 1.f, at, v, w);
      param_pairs<T, A>(p.b, p.w_f32, 0.f, at, v, b);
      get_pairs(x[v], at, v, f);
      normalise(f, m, rs, w, b);
      store_pairs<P>(static_cast<T*>(p.y) + row * p.y_stride, at, v, f);
    }
  }
}

// Rows too wide for registers: one CTA per row reads it three times (the second and third
// time out of L2 for all but the widest).
template <typename T, Access A>
__global__ void __launch_bounds__(1024) ln_fwd_wide_kernel(const LnFwdParams p) {
  begin_after_previous();
  __shared__ float smem[32];
  using P = Piece<T, A>;
  const Place at{p.cols, static_cast<int>(blockDim.x), static_cast<int>(threadIdx.x), 0};
  const int nv = (p.cols + 8 * at.tpr - 1) / (8 * at.tpr);
  const float inv_n = 1.f / static_cast<float>(p.cols);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.x_stride;
    float2 a = both(0.f), q = both(0.f);
    P x;
    for (int v = 0; v < nv; ++v) {
      x.load(xr, at, v, true, false);
      add_piece(x, at, v, a);
    }
    const float m = cta_sum(a.x + a.y, smem) * inv_n;
    for (int v = 0; v < nv; ++v) {
      x.load(xr, at, v, true, false);
      add_squares(x, m, at, v, q);
    }
    const float rs = rsqrtf(fmaf(cta_sum(q.x + q.y, smem), inv_n, p.eps));
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = m;
      if (p.rstd) p.rstd[row] = rs;
    }
    for (int v = 0; v < nv; ++v) {
      float2 f[4], w[4], b[4];
      x.load(xr, at, v, true, false);
      param_pairs<T, A>(p.w, p.w_f32, 1.f, at, v, w);
      param_pairs<T, A>(p.b, p.w_f32, 0.f, at, v, b);
      get_pairs(x, at, v, f);
      normalise(f, m, rs, w, b);
      store_pairs<P>(static_cast<T*>(p.y) + row * p.y_stride, at, v, f);
    }
  }
}

// ---------------------------------------------------------------- launches

template <typename T, Access A, int NV, int R>
cudaError_t fwd_warp(LnFwdParams p, int sms, cudaStream_t s) {
  const int grid = cta_count(p.rows, static_cast<long long>(256 / p.tpr) * R, FWD_CTAS<T, A, NV> * sms);
  const size_t smem = 2 * static_cast<size_t>(Staged<A, NV>::floats(p.tpr)) * sizeof(float);
  return launch_after(ln_fwd_kernel<T, A, NV, R>, dim3(grid), dim3(256), smem, s, p);
}

template <typename T>
cudaError_t fwd_ring(LnFwdParams p, int sms, cudaStream_t s) {
  using Shape = FwdRing<T>;
  p.tpr = (p.cols + 16 * 32 - 1) / (16 * 32) * 32;
  const int threads = Shape::MAX_THREADS / p.tpr * p.tpr;
  const size_t smem = Shape::bytes(threads);
  const cudaError_t e = allow_shared(ln_fwd_ring_kernel<T>, smem, Shape::bytes(Shape::MAX_THREADS));
  if (e != cudaSuccess) return e;
  return launch_after(ln_fwd_ring_kernel<T>, dim3(cta_count(p.rows, Shape::R, sms)), dim3(threads), smem, s, p);
}

template <typename T, Access A>
cudaError_t fwd(LnFwdParams p, int sms, cudaStream_t s) {
  constexpr bool SCALAR = A == Access::SCALAR, SHIFT = A == Access::SHIFT;
  const int pieces = (p.cols + (SHIFT ? 14 : 7)) / 8;
  p.tpr = pieces >= 32 ? 32 : pow2_at_least(pieces);
  if constexpr (A == Access::VEC) {
    // 9728 bf16 rows of 8192 elements take 60 us so and 84 by a CTA per row (fp32 104 and 119), of 4096 33
    // and, by a warp per row, 36 (fp32 rows up to 4096 are as fast so); but 608 rows of 8192 8.6 and 6.0,
    // and 1216 of 4096 8.6 and 6.8: a ring pays from about 2^16 elements per SM
    if (pieces > (sizeof(T) == 2 ? 256 : 512) && pieces <= 1024 && p.rows * p.cols >= 65536ll * sms)
      return fwd_ring<T>(p, sms, s);
  }
  if constexpr (!SHIFT) {
    if (pieces <= 32) return fwd_warp<T, A, 1, SCALAR ? 2 : 4>(p, sms, s);
    if (pieces <= 64) return fwd_warp<T, A, 2, SCALAR ? 1 : 2>(p, sms, s);
  }
  if constexpr (!SCALAR) {
    if (pieces <= 96) return fwd_warp<T, A, 3, 1>(p, sms, s);
    if (pieces <= 128) return fwd_warp<T, A, 4, 1>(p, sms, s);
    if (pieces <= 256) return fwd_warp<T, A, 8, 1>(p, sms, s);
  }
  if constexpr (A == Access::VEC) {
    if (pieces <= 512) return fwd_warp<T, A, 16, 1>(p, sms, s);
  }
  if constexpr (!SHIFT) {
    constexpr int NV = SCALAR ? 2 : 8, MAXT = SCALAR ? 1024 : 512;
    if (pieces <= NV * MAXT) {
      const int threads = (pieces + 32 * NV - 1) / (32 * NV) * 32;
      return launch_after(ln_fwd_cta_kernel<T, A, NV, MAXT>, dim3(cta_count(p.rows, 1, 1 << 20)), dim3(threads), 0, s, p);
    }
    return launch_after(ln_fwd_wide_kernel<T, A>, dim3(cta_count(p.rows, 1, 2 * sms)), dim3(1024), 0, s, p);
  }
  return cudaErrorInvalidValue;                        // SHIFT is for 513 to 2034 elements
}

template <typename T>
cudaError_t fwd_any(const LnFwdParams& p, int sms, cudaStream_t s) {
  constexpr int SIZE = sizeof(T);
  if (p.cols % 8 == 0 && aligned_rows(p.x, p.x_stride, SIZE, p.rows) && aligned_rows(p.y, p.y_stride, SIZE, p.rows) &&
      aligned(p.w) && aligned(p.b))
    return fwd<T, Access::VEC>(p, sms, s);
  // 2^26 elements in rows of 1001 take 102 us so and 146 by single elements (bf16; fp32 114 and 149), in
  // rows of 2003 92 and 142 (109 and 146), of 777 126 and 177 (134 and 181); in rows of 303 224 and 168 (195 and 178), of 3001 184 and 152
  if (p.cols > 512 && p.cols + 14 <= 2048 && shiftable(p.x_stride, p.cols, p.rows) &&
      same_shift(p.x, p.x_stride, p.y, p.y_stride, SIZE, p.rows))
    return fwd<T, Access::SHIFT>(p, sms, s);
  return fwd<T, Access::SCALAR>(p, sms, s);
}

}  // namespace

cudaError_t launch_layer_norm(LnFwdParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 1;
  if (type == MB_F32) return fwd_any<float>(p, sms, s);
  if (type == MB_BF16) return fwd_any<__nv_bfloat16>(p, sms, s);
  return fwd_any<__half>(p, sms, s);
}

}  // namespace mb
