// The passes over rows around the products of mb_linear: dz = dy act'(z) with its sums over slabs of rows, and rows copied to
// 16-byte boundaries for operands that TMA cannot address.
#include <type_traits>

#include "mb_block.h"
#include "mb_linear.cuh"

namespace mb {
namespace {

// A CTA takes 256 columns of a slab of rows, a warp every eighth row, a lane eight columns (neighbouring where the rows are
// aligned, else every 32nd).  Bound by memory.  The sums are those of dz before it is rounded, one row of parts for every
// piece of a slab that lies in one group: slab number + group number, which no two pieces share.
constexpr int SLOPE_COLS = 256, SLOPE_WARPS = 8;

template <typename T, int ACT, bool ALIGNED>
__device__ __forceinline__ void slope_rows(const LinearSlopeParams& p, int begin, int end, int c0, int warp, int lane,
                                           float (&sum)[8]) {
  const T* dy = static_cast<const T*>(p.dy);
  const T* z = static_cast<const T*>(p.z);
  T* dz = static_cast<T*>(p.dz);
  const int first = ALIGNED ? c0 + 8 * lane : c0 + lane;
  if (first >= p.cols) return;
#pragma unroll 2
  for (int row = begin + warp; row < end; row += SLOPE_WARPS) {
    const T* g = dy + row * p.dy_ld + first;
    float v[8], x[8];
    if constexpr (ALIGNED) {
      Eight<T> a, b;
      a.load(g);
      if (ACT != MB_ACT_NONE) {
        b.load(z + row * p.z_ld + first);
        b.get(x);
      }
      a.get(v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = first + 32 * j < p.cols ? to_float(g[32 * j]) : 0.f;
        if (ACT != MB_ACT_NONE) x[j] = first + 32 * j < p.cols ? to_float(z[row * p.z_ld + first + 32 * j]) : 0.f;
      }
    }
    if (ACT != MB_ACT_NONE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= slope<ACT>(x[j]);
      T* to = dz + row * p.dz_ld + first;
      if constexpr (ALIGNED) {
        Eight<T> a;
        a.set(v);
        a.store(to);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (first + 32 * j < p.cols) to[32 * j] = from_float<T>(v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += v[j];
  }
}

template <typename T, bool ALIGNED>
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
      slope_rows<T, decltype(act)::value, ALIGNED>(p, row, stop, c0, warp, lane, sum);
    });
    row = stop;
    if (!p.parts) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) partial[warp][ALIGNED ? 8 * lane + j : 32 * j + lane] = sum[j];
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

__global__ void __launch_bounds__(256) linear_pack_kernel(const __grid_constant__ LinearPackParams p) {
  begin_after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a warp per row: single elements, read along the row
  for (long long row = static_cast<long long>(blockIdx.x) * 8 + warp; row < p.rows; row += static_cast<long long>(gridDim.x) * 8) {
    const uint16_t* from = p.src + row * p.src_ld;
    uint16_t* to = p.dst + row * p.dst_ld;
#pragma unroll 4
    for (int c = lane; c < p.cols; c += 32) to[c] = from[c];
  }
}

}  // namespace

cudaError_t launch_linear_slope(const LinearSlopeParams& p, int type, cudaStream_t s) {
  const dim3 grid((p.cols + SLOPE_COLS - 1) / SLOPE_COLS, (p.rows + p.slab - 1) / p.slab);
  const dim3 block(32 * SLOPE_WARPS);
  if (type == MB_BF16)
    return p.aligned ? launch_after(linear_slope_kernel<__nv_bfloat16, true>, grid, block, 0, s, p)
                     : launch_after(linear_slope_kernel<__nv_bfloat16, false>, grid, block, 0, s, p);
  return p.aligned ? launch_after(linear_slope_kernel<__half, true>, grid, block, 0, s, p)
                   : launch_after(linear_slope_kernel<__half, false>, grid, block, 0, s, p);
}

cudaError_t launch_linear_pack(const LinearPackParams& p, int sms, cudaStream_t s) {
  const long long need = (p.rows + 7) / 8, most = 8ll * sms;
  return launch_after(linear_pack_kernel, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(256), 0, s, p);
}

}  // namespace mb
