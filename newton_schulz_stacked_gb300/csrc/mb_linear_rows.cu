// The passes over rows around the products of mb_linear: dz = dy act'(z) with its sums over slabs of rows, and rows copied to
// 16-byte boundaries for operands that TMA cannot address; and the product over a few rows, which is a pass over W.
#include <type_traits>

#include "mb_block.h"
#include "mb_linear.cuh"

namespace mb {
namespace {

// A CTA takes 256 columns of a slab of rows, a warp every eighth row, a lane eight columns: neighbouring ones where the rows
// allow 16-byte accesses, else pairs or single ones 64 or 32 apart.  Bound by memory.  The sums are those of dz
// before it is rounded, one row of parts for every piece of a slab that lies in one group: slab number + group number,
// which no two pieces share.
constexpr int SLOPE_COLS = 256, SLOPE_WARPS = 8;

// The column of a lane's element j.
template <int ACCESS>
__device__ __forceinline__ int lane_col(int lane, int j) {
  return ACCESS == 16 ? 8 * lane + j : ACCESS == 4 ? 64 * (j / 2) + 2 * lane + j % 2 : 32 * j + lane;
}

// Eight elements of a row, zeros past the last column.
template <typename T, int ACCESS>
__device__ __forceinline__ void load_lane(const T* row, int c0, int cols, int lane, float (&v)[8]) {
  if constexpr (ACCESS == 16) {
    Eight<T> e;
    e.load(row + c0 + 8 * lane);
    e.get(v);
  } else if constexpr (ACCESS == 4) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const int c = c0 + lane_col<4>(lane, j);
      const float2 f = unpack2(c < cols ? *reinterpret_cast<const uint32_t*>(row + c) : 0u, T());
      v[j] = f.x;
      v[j + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + lane_col<2>(lane, j);
      v[j] = c < cols ? to_float(row[c]) : 0.f;
    }
  }
}

template <typename T, int ACCESS>
__device__ __forceinline__ void store_lane(T* row, int c0, int cols, int lane, const float (&v)[8]) {
  if constexpr (ACCESS == 16) {
    Eight<T> e;
    e.set(v);
    e.store(row + c0 + 8 * lane);
  } else if constexpr (ACCESS == 4) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const int c = c0 + lane_col<4>(lane, j);
      if (c < cols) *reinterpret_cast<uint32_t*>(row + c) = pack2(v[j], v[j + 1], T());
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + lane_col<2>(lane, j);
      if (c < cols) row[c] = from_float<T>(v[j]);
    }
  }
}

template <typename T, int ACT, int ACCESS>
__device__ __forceinline__ void slope_rows(const LinearSlopeParams& p, int begin, int end, int c0, int warp, int lane,
                                           float (&sum)[8]) {
  const T* dy = static_cast<const T*>(p.dy);
  const T* z = static_cast<const T*>(p.z);
  T* dz = static_cast<T*>(p.dz);
  const int first = c0 + lane_col<ACCESS>(lane, 0);
  const int most = p.low ? p.low : p.cols;       // columns that are written: with low halves the gap before them too
  if (first >= (ACT == MB_ACT_NONE ? p.cols : most)) return;
#pragma unroll 2
  for (int row = begin + warp; row < end; row += SLOPE_WARPS) {
    float v[8], x[8];
    const bool some = ACCESS != 16 || first < p.cols;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = x[j] = 0.f;
    if (some) load_lane<T, ACCESS>(dy + row * p.dy_ld, c0, p.cols, lane, v);
    if (ACT != MB_ACT_NONE) {
      if (some) load_lane<T, ACCESS>(z + row * p.z_ld, c0, p.cols, lane, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= slope<ACT>(x[j]);
      T* to = dz + row * p.dz_ld;
      store_lane<T, ACCESS>(to, c0, most, lane, v);
      if (p.low) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float left = v[j] - to_float(from_float<T>(v[j]));
          x[j] = isfinite(left) ? left : 0.f;      // (an infinite half: all of it)
        }
        store_lane<T, ACCESS>(to + p.low, c0, most, lane, x);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += v[j];
  }
}

template <typename T, int ACCESS>
__global__ void __launch_bounds__(32 * SLOPE_WARPS) linear_slope_kernel(const __grid_constant__ LinearSlopeParams p) {
  __shared__ float partial[SLOPE_WARPS][SLOPE_COLS];
  __shared__ int groups[2 * (LINEAR_MAX_GROUPS + 1)];
  begin_after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Groups G{groups, groups + LINEAR_MAX_GROUPS + 1, p.groups};
  if (warp == 0) fill_groups(G, p.ends, p.rows, lane);
  __syncthreads();
  const int slab = blockIdx.y, c0 = blockIdx.x * SLOPE_COLS;
  const int begin = slab * p.slab, end = min(begin + p.slab, G.row[G.n]);
  // the first group whose rows end past the slab's begin
  int lo = 0, hi = G.n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (G.row[mid + 1] > begin) hi = mid;
    else lo = mid + 1;
  }
  int row = begin;
  for (int g = lo; g < G.n && row < end; ++g) {
    const int stop = min(end, G.row[g + 1]);
    if (stop <= row) continue;
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
    with_activation(p.z ? p.act : MB_ACT_NONE, [&](auto act) {
      slope_rows<T, decltype(act)::value, ACCESS>(p, row, stop, c0, warp, lane, sum);
    });
    row = stop;
    if (!p.parts) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) partial[warp][lane_col<ACCESS>(lane, j)] = sum[j];
    __syncthreads();
    const int col = threadIdx.x;
    if (c0 + col < p.cols) {
      float all = 0.f;
#pragma unroll
      for (int i = 0; i < SLOPE_WARPS; ++i) all += partial[i][col];
      p.parts[static_cast<long long>(slab + g) * p.cols + c0 + col] = all;
    }
    __syncthreads();
  }
}

constexpr int PACK_COLS = 256;
__global__ void __launch_bounds__(256) linear_pack_kernel(const __grid_constant__ LinearPackParams p) {
  begin_after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a warp for 256 columns of a row: pairs of elements, or single ones, read along the row, all before the first is stored
  const int c0 = blockIdx.y * PACK_COLS, cols = min(p.cols - c0, PACK_COLS);
  for (long long row = static_cast<long long>(blockIdx.x) * 8 + warp; row < p.rows; row += static_cast<long long>(gridDim.x) * 8) {
    const uint16_t* from = p.src + row * p.src_ld + c0;
    uint16_t* to = p.dst + row * p.dst_ld + c0;
    if (p.pairs) {
      uint32_t v[PACK_COLS / 64];
#pragma unroll
      for (int i = 0; i < PACK_COLS / 64; ++i)
        if (lane + 32 * i < cols / 2) v[i] = reinterpret_cast<const uint32_t*>(from)[lane + 32 * i];
#pragma unroll
      for (int i = 0; i < PACK_COLS / 64; ++i)
        if (lane + 32 * i < cols / 2) reinterpret_cast<uint32_t*>(to)[lane + 32 * i] = v[i];
    } else {
      uint16_t v[PACK_COLS / 32];
#pragma unroll
      for (int i = 0; i < PACK_COLS / 32; ++i)
        if (lane + 32 * i < cols) v[i] = from[lane + 32 * i];
#pragma unroll
      for (int i = 0; i < PACK_COLS / 32; ++i)
        if (lane + 32 * i < cols) to[lane + 32 * i] = v[i];
    }
  }
}

// dbias of 32 columns of one group: the sums over the slabs that hold its rows, a run of them to each warp, then the warps', in
// order.
constexpr int BIAS_WARPS = 16;
template <typename T>
__global__ void __launch_bounds__(32 * BIAS_WARPS) linear_bias_kernel(const __grid_constant__ LinearBiasParams p) {
  __shared__ float partial[BIAS_WARPS][32];
  __shared__ int groups[2 * (LINEAR_MAX_GROUPS + 1)];
  begin_after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Groups G{groups, groups + LINEAR_MAX_GROUPS + 1, p.groups};
  if (warp == 0) fill_groups(G, p.ends, p.rows, lane);
  __syncthreads();
  const int g = blockIdx.y, col = blockIdx.x * 32 + lane;
  const int begin = G.row[g], end = G.row[g + 1];
  const int first = begin / p.slab, slabs = end > begin ? (end - 1) / p.slab - first + 1 : 0;
  const int from = static_cast<int>(static_cast<long long>(slabs) * warp / BIAS_WARPS);
  const int to = static_cast<int>(static_cast<long long>(slabs) * (warp + 1) / BIAS_WARPS);
  float sum = 0.f;
  if (col < p.cols) {
    const float* at = p.parts + static_cast<long long>(first + g) * p.cols + col;
#pragma unroll 8
    for (int s = from; s < to; ++s) sum += at[static_cast<long long>(s) * p.cols];
  }
  partial[warp][lane] = sum;
  __syncthreads();
  if (warp > 0 || col >= p.cols) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < BIAS_WARPS; ++i) sum += partial[i][lane];
  const long long out = static_cast<long long>(g) * p.cols + col;
  if (p.f32) static_cast<float*>(p.db)[out] = sum;
  else static_cast<T*>(p.db)[out] = from_float<T>(sum);
}

// y of one row (off 16-byte boundaries up to 8): bound by reading W, which the tensor cores' tiles of 256 rows would only wait
// for.  A CTA takes four columns of y (rows of W) of one group, its warps every eighth 256 elements of them, each lane eight
// for all rows of x in fp32; the lanes' sums, then the warps', are added in order.  1x4096->4096 7.8 us, 1x4096->16384 23.6
// (5.7 TB/s); with more rows the conversions and sums would bound it (8x4096->4096 21.0).
constexpr int FEW_WARPS = 8, FEW_COLS = 4;

// The rows of the blockIdx.y'th group that has any, and zeros in the columns from col0 on of the rows of no group.
struct FewRows {
  int g, begin, end;
};
template <typename T>
__device__ __forceinline__ FewRows few_rows(const LinearFewParams& p, int* groups, int col0, int cols) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  FewRows f{0, 0, p.rows};
  if (!p.ends) return f;
  Groups G{groups, groups + LINEAR_MAX_GROUPS + 1, p.groups};
  if (warp == 0 && fill_groups(G, p.ends, p.rows, lane) && blockIdx.x == 0 && blockIdx.y == 0 && lane == 0)
    latch_status(p.status, DEV_BAD_SCALAR);
  __syncthreads();
  const int last = G.row[G.n];
  f.begin = f.end = last;
  int before = static_cast<int>(blockIdx.y);
  for (int g0 = 0; g0 < G.n; g0 += 32) {
    const int at = g0 + lane;
    const bool some = at < G.n && G.row[at + 1] > G.row[at];
    const unsigned all = __ballot_sync(0xffffffffu, some);
    const unsigned found = __ballot_sync(0xffffffffu, some && __popc(all & ((1u << lane) - 1)) == before);
    if (found) {
      f.g = g0 + __ffs(found) - 1;
      f.begin = G.row[f.g];
      f.end = G.row[f.g + 1];
      break;
    }
    before -= __popc(all);
  }
  if (blockIdx.y == 0 && blockIdx.z == 0) {
    for (int i = threadIdx.x; i < (p.rows - last) * cols; i += blockDim.x) {
      const long long row = last + i / cols;
      const int col = col0 + i % cols;
      if (col >= p.out) continue;
      static_cast<T*>(p.y)[row * p.y_ld + col] = from_float<T>(0.f);
      if (p.z) static_cast<T*>(p.z)[row * p.z_ld + col] = from_float<T>(0.f);
    }
  }
  return f;
}

// One sum on its way out.
template <typename T>
__device__ __forceinline__ void finish_one(const LinearFewParams& p, float v, int g, long long row, int col) {
  const long long at = static_cast<long long>(g) * p.out + col;
  if (p.bias) v += p.bias_f32 ? static_cast<const float*>(p.bias)[at] : to_float(static_cast<const T*>(p.bias)[at]);
  if (p.z) static_cast<T*>(p.z)[row * p.z_ld + col] = from_float<T>(v);
  with_activation(p.act, [&](auto act) { v = activate<decltype(act)::value>(make_float2(v, 0.f)).x; });
  if (p.residual) v += to_float(static_cast<const T*>(p.residual)[row * p.residual_ld + col]);
  static_cast<T*>(p.y)[row * p.y_ld + col] = from_float<T>(v);
}

template <typename T, int ACCESS, int ROWS>
__global__ void __launch_bounds__(32 * FEW_WARPS, ROWS == 1 ? 4 : 2) linear_few_kernel(const __grid_constant__ LinearFewParams p) {
  __shared__ int groups[2 * (LINEAR_MAX_GROUPS + 1)];
  __shared__ float partial[FEW_WARPS][ROWS * FEW_COLS];
  begin_after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col0 = blockIdx.x * FEW_COLS;
  const FewRows f = few_rows<T>(p, groups, col0, FEW_COLS);
  const int g = f.g, begin = f.begin, end = f.end;
  const T* x = static_cast<const T*>(p.x);
  const int n = end - begin;
  if (n == 0) return;
  const T* w = static_cast<const T*>(p.w) + (static_cast<long long>(g) * p.out + col0) * p.in;
  float2 sum[FEW_COLS][ROWS];                    // of even and odd elements
#pragma unroll
  for (int c = 0; c < FEW_COLS; ++c)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) sum[c][r] = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int k = 256 * warp; k < p.in; k += 256 * FEW_WARPS) {
    if (ACCESS == 16 && k + 8 * lane >= p.in) continue;
    float a[FEW_COLS][8], b[8];
#pragma unroll
    for (int c = 0; c < FEW_COLS; ++c)           // (past the last column: that one again)
      load_lane<T, ACCESS>(w + static_cast<long long>(min(c, p.out - 1 - col0)) * p.in, k, p.in, lane, a[c]);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {             // (and past the last row)
      load_lane<T, ACCESS>(x + (begin + min(r, n - 1)) * p.x_ld, k, p.in, lane, b);
#pragma unroll
      for (int c = 0; c < FEW_COLS; ++c)
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          sum[c][r] = __ffma2_rn(make_float2(a[c][j], a[c][j + 1]), make_float2(b[j], b[j + 1]), sum[c][r]);
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int c = 0; c < FEW_COLS; ++c) {
      float s = sum[c][r].x + sum[c][r].y;
#pragma unroll
      for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (lane == 0) partial[warp][r * FEW_COLS + c] = s;
    }
  __syncthreads();
  const int r = threadIdx.x / FEW_COLS, col = col0 + threadIdx.x % FEW_COLS;
  if (r >= n || col >= p.out) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < FEW_WARPS; ++i) v += partial[i][threadIdx.x];
  finish_one<T>(p, v, g, begin + r, col);
}

// y of up to 512 rows, the products by warps' MMAs (16 x 8 x 16) whose operands come straight from memory.  With up to 32 rows
// bound by reading W (16x4096->4096 10.0 us, 3.4 TB/s) and the chain of waits on it; with more, every 32 rows read W again
// (from the L2) and every 16 columns x, and the number of CTAs is what counts (512x768->768 8.0 us, 768 CTAs).  A lane's
// 16 bytes of a row hold what two MMAs take of it, in an order of the contraction that is the same for x and W.  A CTA
// takes 16 columns of y (rows of W) and 16 or 32 rows of one group, each of its warps 32 elements of the contraction in turn,
// which are added in order.  A call is a chain of waits on memory: long contractions go to 16 warps
// (16x4096->1024 8.3 us, by 8 warps 13.2), short ones of 32 rows to 8 (32x768->2816 4.9, by 16 6.1).
constexpr int SOME_COLS = 16, SOME_LD = SOME_COLS + 2;

template <typename T>
__device__ __forceinline__ void warp_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename T, int TILES, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) linear_some_kernel(const __grid_constant__ LinearFewParams p) {
  constexpr int AHEAD = TILES == 2 && WARPS == 16 ? 4 : 2;
  __shared__ int groups[2 * (LINEAR_MAX_GROUPS + 1)];
  // (written in pairs)
  static_assert(SOME_LD % 2 == 0, "a row of sums begins at a pair");
  __shared__ alignas(16) float partial[WARPS][16 * TILES][SOME_LD];
  begin_after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col0 = blockIdx.x * SOME_COLS;
  FewRows f = few_rows<T>(p, groups, col0, SOME_COLS);
  f.begin += static_cast<int>(blockIdx.z) * 16 * TILES;
  const int n = min(f.end - f.begin, 16 * TILES), quad = lane >> 2, k0 = 8 * (lane & 3);
  if (n <= 0) return;
  const T* w[2];
  const T* x[2 * TILES];
#pragma unroll
  for (int i = 0; i < 2; ++i)                    // (past the last column, or row: that one again)
    w[i] = static_cast<const T*>(p.w) + (static_cast<long long>(f.g) * p.out + min(col0 + 8 * i + quad, p.out - 1)) * p.in + k0;
#pragma unroll
  for (int i = 0; i < 2 * TILES; ++i)
    x[i] = static_cast<const T*>(p.x) + (f.begin + min(8 * i + quad, n - 1)) * p.x_ld + k0;
  float sum[TILES][2][4];
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[t][i / 4][i % 4] = 0.f;
#pragma unroll AHEAD
  for (int k = 32 * warp; k < p.in; k += 32 * WARPS) {
    const bool some = k + k0 < p.in;
    uint4 a[2 * TILES], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = some ? *reinterpret_cast<const uint4*>(w[i] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * TILES; ++i) a[i] = some ? *reinterpret_cast<const uint4*>(x[i] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        warp_mma<T>(sum[t][i], a[2 * t].x, a[2 * t + 1].x, a[2 * t].y, a[2 * t + 1].y, b[i].x, b[i].y);
        warp_mma<T>(sum[t][i], a[2 * t].z, a[2 * t + 1].z, a[2 * t].w, a[2 * t + 1].w, b[i].z, b[i].w);
      }
  }
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 16 * t + quad, col = 8 * i + 2 * (lane & 3);
      *reinterpret_cast<float2*>(&partial[warp][row][col]) = make_float2(sum[t][i][0], sum[t][i][1]);
      *reinterpret_cast<float2*>(&partial[warp][row + 8][col]) = make_float2(sum[t][i][2], sum[t][i][3]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < n * SOME_COLS; i += 32 * WARPS) {
    const int row = i / SOME_COLS, col = i % SOME_COLS;
    if (col0 + col >= p.out) continue;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < WARPS; ++j) v += partial[j][row][col];
    finish_one<T>(p, v, f.g, f.begin + row, col0 + col);
  }
}

template <typename T>
cudaError_t launch_few_type(const LinearFewParams& p, cudaStream_t s) {
  const int groups = p.groups < p.rows ? p.groups : p.rows;
  const dim3 grid((p.out + FEW_COLS - 1) / FEW_COLS, groups), wide((p.out + SOME_COLS - 1) / SOME_COLS, groups, (p.rows + 31) / 32), block(32 * FEW_WARPS);
  if (p.access != 16 && p.rows == 1) return launch_after(linear_few_kernel<T, 2, 1>, grid, block, 0, s, p);
  if (p.access != 16) return launch_after(linear_few_kernel<T, 2, LINEAR_FEW_ROWS>, grid, block, 0, s, p);
  if (p.rows == 1) return launch_after(linear_few_kernel<T, 16, 1>, grid, block, 0, s, p);
  if (p.rows <= 16) return launch_after(linear_some_kernel<T, 1, 16>, wide, dim3(512), 0, s, p);
  if (p.in <= 1024) return launch_after(linear_some_kernel<T, 2, 8>, wide, dim3(256), 0, s, p);
  return launch_after(linear_some_kernel<T, 2, 16>, wide, dim3(512), 0, s, p);
}

template <typename T>
cudaError_t launch_slope_type(const LinearSlopeParams& p, cudaStream_t s) {
  const dim3 grid((p.cols + SLOPE_COLS - 1) / SLOPE_COLS, (p.rows + p.slab - 1) / p.slab);
  const dim3 block(32 * SLOPE_WARPS);
  if (p.access == 16) return launch_after(linear_slope_kernel<T, 16>, grid, block, 0, s, p);
  if (p.access == 4) return launch_after(linear_slope_kernel<T, 4>, grid, block, 0, s, p);
  return launch_after(linear_slope_kernel<T, 2>, grid, block, 0, s, p);
}

}  // namespace

cudaError_t launch_linear_bias(const LinearBiasParams& p, int type, cudaStream_t s) {
  const dim3 grid((p.cols + 31) / 32, p.groups), block(32 * BIAS_WARPS);
  return type == MB_BF16 ? launch_after(linear_bias_kernel<__nv_bfloat16>, grid, block, 0, s, p)
                         : launch_after(linear_bias_kernel<__half>, grid, block, 0, s, p);
}

cudaError_t launch_linear_slope(const LinearSlopeParams& p, int type, cudaStream_t s) {
  return type == MB_BF16 ? launch_slope_type<__nv_bfloat16>(p, s) : launch_slope_type<__half>(p, s);
}

cudaError_t launch_linear_few(const LinearFewParams& p, int type, cudaStream_t s) {
  return type == MB_BF16 ? launch_few_type<__nv_bfloat16>(p, s) : launch_few_type<__half>(p, s);
}

cudaError_t launch_linear_pack(const LinearPackParams& p, int sms, cudaStream_t s) {
  const int pieces = (p.cols + PACK_COLS - 1) / PACK_COLS;
  const long long need = (p.rows + 7) / 8, most = pieces < 8 ? 8ll * sms / pieces : sms;
  return launch_after(linear_pack_kernel, dim3(static_cast<unsigned>(need < most ? need : most), pieces), dim3(256), 0, s, p);
}

}  // namespace mb
