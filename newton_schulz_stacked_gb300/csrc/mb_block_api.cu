// C entries of the block operators: argument checks, workspace layout, launches.
#include <cmath>

#include "mb_block.h"
#include "muonbank.h"

namespace mb {
namespace {

#define MB_TRY(expr)            \
  do {                          \
    int r_ = (expr);            \
    if (r_ != MB_OK) return r_; \
  } while (0)

int type_size(int type) {
  switch (type) {
    case MB_F32: case MB_I32: return 4;
    case MB_BF16: case MB_F16: return 2;
    case MB_I64: return 8;
    default: return 0;
  }
}

bool float_type(int type) { return type == MB_F32 || type == MB_BF16 || type == MB_F16; }

// A pointer to elements of `size` bytes; `need`: it may not be null.
int check_elements(const void* p, int size, bool need) {
  if (!p) return need ? MB_ERR_NULL : MB_OK;
  return reinterpret_cast<uintptr_t>(p) % size == 0 ? MB_OK : MB_ERR_ALIGN;
}

int check_block_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MB_OK;
  if (!ws || have < need) return MB_ERR_WORKSPACE;
  return reinterpret_cast<uintptr_t>(ws) % 256 == 0 ? MB_OK : MB_ERR_ALIGN;
}

// A row stride: `write` rows must not overlap.
bool bad_stride(int64_t stride, int64_t rows, int64_t cols, bool write) {
  return stride < 0 || (write && rows > 1 && stride < cols);
}

int norm_checks(int64_t rows, int64_t cols, int type, int w_type) {
  if (rows < 0 || cols < 1 || cols > (1ll << 30)) return MB_ERR_SHAPE;
  if (!float_type(type) || (w_type != type && w_type != MB_F32)) return MB_ERR_ARG;
  return MB_OK;
}

size_t norm_workspace(int64_t rows, int64_t cols) {
  const int64_t most = cols > LN_BWD_MAX_COLS ? LN_WIDE_SLABS : LN_MAX_PARTS;
  const int64_t parts = rows < 1 ? 1 : rows < most ? rows : most;
  return static_cast<size_t>(parts) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

int router_checks(int64_t tokens, int64_t experts) {
  if (tokens < 0 || tokens >= (1ll << 31) || experts < 1 || experts > ROUTER_MAX_EXPERTS) return MB_ERR_SHAPE;
  return MB_OK;
}

int router_call_checks(int64_t tokens, int64_t experts, int top_k, int type) {
  MB_TRY(router_checks(tokens, experts));
  if (top_k < 1 || top_k > experts || top_k > ROUTER_MAX_K) return MB_ERR_SHAPE;
  if (tokens * top_k >= (1ll << 31)) return MB_ERR_SHAPE;
  return float_type(type) ? MB_OK : MB_ERR_ARG;
}

struct RouterWorkspace {
  size_t sums, used, end;
};

RouterWorkspace router_workspace(int64_t tokens, int64_t experts) {
  const size_t parts = router_parts(static_cast<int>(tokens), static_cast<int>(experts), 1 << 20);
  RouterWorkspace w{};
  if (parts == 1) return w;                // one CTA finishes its sums in shared memory
  w.sums = 0;
  w.used = w.sums + parts * experts * sizeof(int2);
  w.end = w.used + parts * 4;
  return w;
}

int check_heads(const mb_head_tensor& x, const mb_rotary_desc& d, int size, RotaryTensor* out) {
  if (x.heads < 0 || x.heads > 65536) return MB_ERR_SHAPE;
  *out = RotaryTensor{};
  if (x.heads == 0) return MB_OK;
  const int64_t n[3] = {d.batch, d.tokens, x.heads};
  int64_t src[3] = {x.src_batch, x.src_token, x.src_head}, dst[3] = {x.dst_batch, x.dst_token, x.dst_head};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) src[i] = dst[i] = 0;        // a stride that is never taken
    else if (src[i] < 0 || dst[i] <= 0) return MB_ERR_SHAPE;
  }
  const bool some = d.batch > 0 && d.tokens > 0;
  MB_TRY(check_elements(x.src, size, some));
  MB_TRY(check_elements(x.dst, size, some));
  *out = RotaryTensor{x.src, x.dst, static_cast<int>(x.heads), src[0], src[1], src[2], dst[0], dst[1], dst[2]};
  return MB_OK;
}

int rotary_call(const mb_rotary_desc* desc, float sign, void* cuda_stream) {
  if (!desc) return MB_ERR_NULL;
  const mb_rotary_desc& d = *desc;
  if (!float_type(d.type)) return MB_ERR_ARG;
  if (d.position_type != MB_I32 && d.position_type != MB_I64 && d.position_type != MB_F32) return MB_ERR_ARG;
  if (d.batch < 0 || d.tokens < 0 || d.batch >= (1ll << 31) || d.tokens >= (1ll << 31) ||
      d.batch * d.tokens >= (1ll << 31))
    return MB_ERR_SHAPE;
  if (d.pairs < 1 || d.pairs > ROTARY_MAX_PAIRS || d.dim < 2 * d.pairs || d.dim > 65536) return MB_ERR_SHAPE;
  if (d.axes < 1 || d.axes > ROTARY_MAX_AXES) return MB_ERR_SHAPE;
  RotaryParams p{};
  int64_t end = 0;
  for (int a = 0; a < d.axes; ++a) {
    if (d.sections[a] < 0) return MB_ERR_SHAPE;
    end += d.sections[a];
    p.section_end[a] = static_cast<int>(end < ROTARY_MAX_PAIRS ? end : ROTARY_MAX_PAIRS);
  }
  if (end != d.pairs) return MB_ERR_SHAPE;
  if (d.pos_axis < 0 || d.pos_batch < 0 || d.pos_token < 0) return MB_ERR_SHAPE;
  const int size = type_size(d.type);
  MB_TRY(check_heads(d.q, d, size, &p.x[0]));
  MB_TRY(check_heads(d.k, d, size, &p.x[1]));
  const int heads = p.x[0].heads + p.x[1].heads;
  if (heads < 1 || heads > 65536) return MB_ERR_SHAPE;
  const bool some = d.batch > 0 && d.tokens > 0;
  MB_TRY(check_elements(d.positions, type_size(d.position_type), some));
  MB_TRY(check_elements(d.inv_freq, 4, some));
  if (!some) return MB_OK;
  p.pos = d.positions;
  p.pos_type = d.position_type;
  p.pos_a = d.pos_axis;
  p.pos_b = d.pos_batch;
  p.pos_t = d.pos_token;
  p.inv_freq = d.inv_freq;
  p.axes = d.axes;
  p.pairs = d.pairs;
  p.dim = d.dim;
  p.interleaved = d.interleaved != 0;
  p.sign = sign;
  p.batch = static_cast<int>(d.batch);
  p.tokens = static_cast<int>(d.tokens);
  p.all_tokens = d.batch * d.tokens;
  int sms = 0, launches = 0;
  MB_TRY(api_device_sms(&sms));
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = launch_rotary(p, d.type, sms, st, &launches);
  if (e != cudaSuccess) return api_cuda_fail(e);
  api_launched(MB_MARK_ROTARY, launches, st);
  return MB_OK;
}

}  // namespace
}  // namespace mb

using namespace mb;

extern "C" {

int mb_layer_norm(const void* x, int64_t x_stride, int type, const void* w, const void* b, int w_type, void* y,
                  int64_t y_stride, float* mean, float* rstd, int64_t rows, int64_t cols, float eps,
                  void* cuda_stream) {
  MB_TRY(norm_checks(rows, cols, type, w_type));
  if (!std::isfinite(eps) || eps < 0.f) return MB_ERR_ARG;
  if (bad_stride(x_stride, rows, cols, false) || bad_stride(y_stride, rows, cols, true)) return MB_ERR_SHAPE;
  MB_TRY(check_elements(x, type_size(type), rows > 0));
  MB_TRY(check_elements(y, type_size(type), rows > 0));
  MB_TRY(check_elements(w, type_size(w_type), false));
  MB_TRY(check_elements(b, type_size(w_type), false));
  MB_TRY(check_elements(mean, 4, false));
  MB_TRY(check_elements(rstd, 4, false));
  if (rows == 0) return MB_OK;
  int sms = 0, launches = 0;
  MB_TRY(api_device_sms(&sms));
  LnFwdParams p{x, x_stride, w, b, w_type == MB_F32, y, y_stride, mean, rstd, rows, static_cast<int>(cols), eps, 0};
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = launch_layer_norm(p, type, sms, st, &launches);
  if (e != cudaSuccess) return api_cuda_fail(e);
  api_launched(MB_MARK_LAYER_NORM, launches, st);
  return MB_OK;
}

int mb_layer_norm_workspace_bytes(int64_t rows, int64_t cols, size_t* out_bytes) {
  if (!out_bytes) return MB_ERR_NULL;
  MB_TRY(norm_checks(rows, cols, MB_F32, MB_F32));
  *out_bytes = norm_workspace(rows, cols);
  return MB_OK;
}

int mb_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride, int type,
                           const void* w, int w_type, const float* mean, const float* rstd, void* dx,
                           int64_t dx_stride, void* dw, void* db, int64_t rows, int64_t cols, void* workspace,
                           size_t workspace_bytes, void* cuda_stream) {
  MB_TRY(norm_checks(rows, cols, type, w_type));
  if (bad_stride(x_stride, rows, cols, false) || bad_stride(dy_stride, rows, cols, false) ||
      bad_stride(dx_stride, rows, cols, true))
    return MB_ERR_SHAPE;
  const int size = type_size(type), w_size = type_size(w_type);
  MB_TRY(check_elements(dy, size, rows > 0));
  MB_TRY(check_elements(x, size, rows > 0));
  MB_TRY(check_elements(dx, size, rows > 0));
  MB_TRY(check_elements(mean, 4, rows > 0));
  MB_TRY(check_elements(rstd, 4, rows > 0));
  MB_TRY(check_elements(w, w_size, false));
  MB_TRY(check_elements(dw, w_size, false));
  MB_TRY(check_elements(db, w_size, false));
  if (dw || db) MB_TRY(check_block_workspace(workspace, workspace_bytes, norm_workspace(rows, cols)));
  else if (rows == 0) return MB_OK;
  int sms = 0, launches = 0;
  MB_TRY(api_device_sms(&sms));
  LnBwdParams p{};
  p.dy = dy;
  p.dy_stride = dy_stride;
  p.x = x;
  p.x_stride = x_stride;
  p.w = w;
  p.w_f32 = w_type == MB_F32;
  p.mean = mean;
  p.rstd = rstd;
  p.dx = dx;
  p.dx_stride = dx_stride;
  p.dw = dw;
  p.db = db;
  p.parts = static_cast<float*>(workspace);
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = launch_layer_norm_backward(p, type, sms, st, &launches);
  if (e != cudaSuccess) return api_cuda_fail(e);
  api_launched(MB_MARK_LAYER_NORM_BACKWARD, launches, st);
  return MB_OK;
}

int mb_rotary(const mb_rotary_desc* desc, void* cuda_stream) { return rotary_call(desc, 1.f, cuda_stream); }
int mb_rotary_backward(const mb_rotary_desc* desc, void* cuda_stream) { return rotary_call(desc, -1.f, cuda_stream); }

int mb_router_workspace_bytes(int64_t tokens, int64_t experts, size_t* out_bytes) {
  if (!out_bytes) return MB_ERR_NULL;
  MB_TRY(router_checks(tokens, experts));
  *out_bytes = router_workspace(tokens, experts).end;
  return MB_OK;
}

int mb_router(const void* logits, int64_t stride, int type, const uint8_t* valid, int64_t tokens, int64_t experts,
              int top_k, int normalize, int32_t* index, float* gate, int32_t* counts, float* loss, int32_t* used,
              void* workspace, size_t workspace_bytes, void* cuda_stream) {
  MB_TRY(router_call_checks(tokens, experts, top_k, type));
  if (bad_stride(stride, tokens, experts, false)) return MB_ERR_SHAPE;
  MB_TRY(check_elements(logits, type_size(type), tokens > 0));
  MB_TRY(check_elements(index, 4, tokens > 0));
  MB_TRY(check_elements(gate, 4, tokens > 0));
  MB_TRY(check_elements(counts, 4, true));
  MB_TRY(check_elements(loss, 4, true));
  MB_TRY(check_elements(used, 4, true));
  const RouterWorkspace w = router_workspace(tokens, experts);
  MB_TRY(check_block_workspace(workspace, workspace_bytes, w.end));
  int sms = 0, launches = 0;
  MB_TRY(api_device_sms(&sms));
  RouterParams p{};
  p.logits = logits;
  p.stride = stride;
  p.valid = valid;
  p.tokens = static_cast<int>(tokens);
  p.experts = static_cast<int>(experts);
  p.k = top_k;
  p.normalize = normalize != 0;
  p.index = index;
  p.gate = gate;
  p.counts = counts;
  p.loss = loss;
  p.used = used;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.parts_sums = reinterpret_cast<int2*>(ws + w.sums);
  p.part_used = reinterpret_cast<int*>(ws + w.used);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = launch_router(p, type, sms, st, &launches);
  if (e != cudaSuccess) return api_cuda_fail(e);
  api_launched(MB_MARK_ROUTER, launches, st);
  return MB_OK;
}

int mb_router_backward(const float* dloss, const float* dgate, const void* logits, int64_t stride, int type,
                       const uint8_t* valid, int64_t tokens, int64_t experts, int top_k, int normalize,
                       const int32_t* index, const float* gate, const int32_t* counts, const int32_t* used,
                       void* dlogits, int64_t dlogits_stride, void* cuda_stream) {
  MB_TRY(router_call_checks(tokens, experts, top_k, type));
  if (bad_stride(stride, tokens, experts, false) || bad_stride(dlogits_stride, tokens, experts, true))
    return MB_ERR_SHAPE;
  const bool some = tokens > 0;
  MB_TRY(check_elements(logits, type_size(type), some));
  MB_TRY(check_elements(dlogits, type_size(type), some));
  MB_TRY(check_elements(dloss, 4, false));
  MB_TRY(check_elements(dgate, 4, false));
  MB_TRY(check_elements(index, 4, some && dgate));
  MB_TRY(check_elements(gate, 4, some && dgate));
  MB_TRY(check_elements(counts, 4, some));
  MB_TRY(check_elements(used, 4, some));
  if (!some) return MB_OK;
  int sms = 0, launches = 0;
  MB_TRY(api_device_sms(&sms));
  const RouterBwdParams p{logits, stride, valid, static_cast<int>(tokens), static_cast<int>(experts), top_k,
                          normalize != 0, index, gate, counts, used, dloss, dgate, dlogits, dlogits_stride};
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = launch_router_backward(p, type, sms, st, &launches);
  if (e != cudaSuccess) return api_cuda_fail(e);
  api_launched(MB_MARK_ROUTER_BACKWARD, launches, st);
  return MB_OK;
}

}  // extern "C"
