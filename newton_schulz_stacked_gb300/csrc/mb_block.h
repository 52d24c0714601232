// Internal interfaces of the block operators (layer norm, rotary, router) between their C
// entries (mb_block_api.cu) and the kernel files, and the API state they share with mb_api.cu.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mb {

// ---------------------------------------------------------------- from mb_api.cu

int api_cuda_fail(cudaError_t e);    // keeps the message, returns MB_ERR_CUDA
int api_device_sms(int* sms);        // checks the current device; its SM count
int api_device_status(int** status); // checks the current device; its latched status word
// A tensor map of `batch` matrices of rows x cols 2-byte elements, row stride ld (a multiple of 8) elements, in boxes of
// box_rows x 64 in the 128-byte swizzle; after one of the two calls above.
int api_encode_rows(CUtensorMap* map, const void* base, bool bf16, int64_t cols, int64_t rows, int64_t batch, int64_t ld,
                    int box_rows);
void api_launched(int label, int launches, cudaStream_t stream);   // counts launches and marks their end

// ---------------------------------------------------------------- layer norm

// Partial sums of the weight's gradient, rows of [2][cols]: one per CTA, or, of rows of more than LN_BWD_MAX_COLS
// elements, one per slab of rows.
constexpr int LN_MAX_PARTS = 456;
constexpr int LN_BWD_MAX_COLS = 8192;    // wider rows are read again from memory
constexpr int LN_WIDE_SLABS = 64;

struct LnFwdParams {
  const void* x;
  long long x_stride;
  const void *w, *b;       // may be null
  int w_f32;               // weight and bias are fp32 (else the activations' type)
  void* y;
  long long y_stride;
  float *mean, *rstd;      // may be null
  long long rows;
  int cols;
  float eps;
  int tpr;                 // threads per row
};

struct LnBwdParams {
  const void* dy;
  long long dy_stride;
  const void* x;
  long long x_stride;
  const void* w;
  int w_f32;
  const float *mean, *rstd;
  void* dx;
  long long dx_stride;
  void *dw, *db;           // may be null
  float* parts;            // [parts][2][cols] partial sums (null: none wanted, or one CTA writes dw and db itself)
  long long rows;
  int cols;
  int tpr, groups;         // threads per row, rows side by side in a CTA
};

cudaError_t launch_layer_norm(LnFwdParams p, int type, int sms, cudaStream_t s, int* launches);
cudaError_t launch_layer_norm_backward(LnBwdParams p, int type, int sms, cudaStream_t s, int* launches);

// ---------------------------------------------------------------- rotary

constexpr int ROTARY_MAX_AXES = 4;
constexpr int ROTARY_MAX_PAIRS = 4096;

struct RotaryTensor {
  const void* src;
  void* dst;
  int heads;                                         // 0: absent
  long long src_b, src_t, src_h, dst_b, dst_t, dst_h;  // strides in elements; heads' elements are contiguous
};

struct RotaryParams {
  RotaryTensor x[2];
  const void* pos;
  int pos_type;
  long long pos_a, pos_b, pos_t;   // strides of the positions
  const float* inv_freq;
  int axes, section_end[ROTARY_MAX_AXES];
  int pairs, dim, interleaved;
  float sign;                      // -1: the inverse rotation
  int batch, tokens;
  int tile;                        // tokens per CTA
  long long all_tokens;            // batch * tokens
};

cudaError_t launch_rotary(RotaryParams p, int type, int sms, cudaStream_t s, int* launches);

// ---------------------------------------------------------------- router

constexpr int ROUTER_MAX_EXPERTS = 1024;
constexpr int ROUTER_MAX_K = 32;
constexpr int ROUTER_MAX_PARTS = 304;    // CTAs of the forward pass, each with its partial sums

struct RouterParams {
  const void* logits;
  long long stride;
  const uint8_t* valid;    // may be null
  int tokens, experts, k, normalize;
  int* index;              // [tokens, k]
  float* gate;             // [tokens, k]
  int* counts;             // [experts]
  float* loss;             // [1]
  int* used;               // [1]
  int2* parts_sums;        // [parts][experts] {sum of p (fp32 bits), count}
  int* part_used;          // [parts]
  int parts;
};

struct RouterBwdParams {
  const void* logits;
  long long stride;
  const uint8_t* valid;
  int tokens, experts, k, normalize;
  const int* index;
  const float* gate;
  const int* counts;
  const int* used;
  const float* dloss;      // [1], may be null
  const float* dgate;      // [tokens, k], may be null
  void* dlogits;
  long long dstride;
};

int router_parts(int tokens, int experts, int sms);
cudaError_t launch_router(RouterParams p, int type, int sms, cudaStream_t s, int* launches);
cudaError_t launch_router_backward(RouterBwdParams p, int type, int sms, cudaStream_t s, int* launches);

// Lets a launch with `smem` bytes of dynamic shared memory be made.  `most`: the most that any launch of this
// kernel asks for, so that every call sets the same limit: a smaller one, set by another host thread between
// this and the launch, would refuse the launch.  What a launch occupies goes by its own size.
template <typename P>
cudaError_t allow_shared(void (*kernel)(P), size_t smem, size_t most) {
  if (smem <= 40 * 1024) return cudaSuccess;         // with a kernel's own arrays within the 48 KB of every launch
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
}

// A launch that may start while the kernel before it in the stream drains: its kernel begins with
// begin_after_previous, before it reads or writes anything.
template <typename P>
cudaError_t launch_after(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const P& p,
                         int cluster = 0) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute a[2]{};
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  if (cluster > 1) {
    a[1].id = cudaLaunchAttributeClusterDimension;
    a[1].val.clusterDim.x = cluster;
    a[1].val.clusterDim.y = 1;
    a[1].val.clusterDim.z = 1;
  }
  cfg.attrs = a;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace mb
