// Routing of tokens over experts: top-k selection, per-expert counts and the balance loss, and
// the gradient of the logits.  Arithmetic is fp32, counts are integers.
//
//   p = softmax(l);  the k largest logits of a token are chosen, the lowest index first among
//   equals;  gate = p there, or normalised over the chosen;  N = tokens that count
//   loss = E / (k N^2) sum_e counts_e sum_t p_te
//   c_e = dloss E counts_e / (k N^2);  dl = p (c + dgate at the chosen - sum_e p (...))
//
// G lanes hold one token's logits, eight (times NC) neighbouring experts each, so a warp works
// on 32 / G tokens, each logit is read once, and a lane meets the same experts in every token:
// the sums over tokens of p stay in its registers.
#include "mb_block.h"
#include "mb_device.cuh"
#include "mb_rows.cuh"
#include "muonbank.h"

namespace mb {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr unsigned FULL = 0xFFFFFFFFu;

// Unsigned keys in the order of the logits: -inf (an expert that is not available) is 0, NaN is
// above everything, both zeros are one.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  if (l != l) return 0xFFFFFFFFu;
  if (u == 0xFF800000u) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (key == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  if (key == 0u) return __uint_as_float(0xFF800000u);
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
  if constexpr (G == 32) return __reduce_max_sync(FULL, x);
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) {
    const uint32_t y = __shfl_xor_sync(FULL, x, o);
    x = y > x ? y : x;
  }
  return x;
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t x) {
  if constexpr (G == 32) return __reduce_min_sync(FULL, x);
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) {
    const uint32_t y = __shfl_xor_sync(FULL, x, o);
    x = y < x ? y : x;
  }
  return x;
}
template <int G>
__device__ __forceinline__ float group_add(float x) {
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
  return x;
}
template <int G>
__device__ __forceinline__ float group_fmax(float x) {
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(FULL, x, o));
  return x;
}

// Expert of element j of piece c of lane g in its group.
template <int G>
__device__ __forceinline__ int expert_of(int c, int g, int j) { return (c * G + g) * 8 + j; }

// The lane's logits of one token; experts past the last read as -inf.
template <typename T, bool VEC, int G, int NC>
__device__ __forceinline__ void load_logits(const T* row, bool on, int experts, int g, float (&l)[8 * NC]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e0 = expert_of<G>(c, g, 0);
    if constexpr (VEC) {
      if (on && e0 < experts) {
        Eight<T> v;
        float f[8];
        v.load(row + e0);
        v.get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) l[8 * c + j] = f[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) l[8 * c + j] = __uint_as_float(0xFF800000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        l[8 * c + j] = on && e0 + j < experts ? to_float(row[e0 + j]) : __uint_as_float(0xFF800000u);
    }
  }
}

// The counts and the loss from the CTAs' sums: E experts in `n` rows of sums; called by the
// `threads` threads of one CTA for the experts [e_begin, e_end); returns (to every thread) the
// share of  sum_e counts_e sum_t p_te  of these experts.  smem: threads floats and ints.
__device__ __forceinline__ float finish_experts(const RouterParams& p, int n, int e_begin, int e_end, float* sf,
                                                int* si) {
  // 32 experts by (threads / 32) slices of the rows at a time, added in a fixed order
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, slices = blockDim.x >> 5;
  float share = 0.f;
  for (int e0 = e_begin; e0 < e_end; e0 += 32) {
    const int e = e0 + lane;
    float a = 0.f;
    int c = 0;
    if (e < e_end) {
#pragma unroll 4
      for (int i = slice; i < n; i += slices) {
        a += p.part_prob[static_cast<size_t>(i) * p.experts + e];
        c += p.part_count[static_cast<size_t>(i) * p.experts + e];
      }
    }
    sf[threadIdx.x] = a;
    si[threadIdx.x] = c;
    __syncthreads();
    if (slice == 0) {
      for (int i = 1; i < slices; ++i) {
        a += sf[i * 32 + lane];
        c += si[i * 32 + lane];
      }
      if (e < e_end) {
        p.counts[e] = c;
        share += a * static_cast<float>(c);
      }
    }
    __syncthreads();
  }
  if (slice == 0) {
    share = group_add<32>(share);
    if (lane == 0) sf[0] = share;
  }
  __syncthreads();
  return sf[0];
}

__device__ __forceinline__ float loss_of(float share, int used, int experts, int k) {
  if (used == 0) return 0.f;
  const float n = static_cast<float>(used);
  return share * (static_cast<float>(experts) / (static_cast<float>(k) * n)) / n;
}

// ---------------------------------------------------------------- forward

template <typename T, bool VEC, int G, int NC>
__global__ void __launch_bounds__(THREADS) router_kernel(const RouterParams p) {
  extern __shared__ float dyn[];                       // [WARPS][experts] sums of p, then [experts] counts
  __shared__ float sf[THREADS];
  __shared__ int si[THREADS];
  constexpr int V = 8 * NC;
  constexpr int TOK = 32 / G;                          // tokens per warp
  constexpr int SLOTS = G >= 32 ? 1 : 32 / G > 8 ? 8 : 32 / G;   // chosen experts a lane keeps (k <= 8 G and k <= 32)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane % G;
  int* scount = reinterpret_cast<int*>(dyn + WARPS * p.experts);
  for (int e = threadIdx.x; e < p.experts; e += THREADS) scount[e] = 0;
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) psum[j] = 0.f;
  int used_here = 0;
  const long long stride = static_cast<long long>(gridDim.x) * WARPS * TOK;
  for (long long base = (static_cast<long long>(blockIdx.x) * WARPS + warp) * TOK; base < p.tokens; base += stride) {
    const long long token = base + lane / G;
    const bool on = token < p.tokens && (!p.valid || p.valid[token] != 0);
    float l[V];
    load_logits<T, VEC, G, NC>(static_cast<const T*>(p.logits) + token * p.stride, on, p.experts, g, l);
    uint32_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = key_of(l[j]);
    // the lane's best two, the lower index first among equals; `last` is the last one taken from it
    uint32_t k1 = 0, k2 = 0;
    int i1 = 0, i2 = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool b1 = key[j] > k1, b2 = key[j] > k2;
      k2 = b1 ? k1 : b2 ? key[j] : k2;
      i2 = b1 ? i1 : b2 ? j : i2;
      k1 = b1 ? key[j] : k1;
      i1 = b1 ? j : i1;
    }
    bool second = true;                                // k2, i2 hold the lane's next
    uint32_t sel_key[SLOTS];
    int sel_idx[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      sel_key[s] = 0;
      sel_idx[s] = -1;
    }
    uint32_t top = 0;
    for (int r = 0; r < p.k; ++r) {
      const uint32_t best = group_max<G>(k1);
      if (r == 0) top = best;
      const uint32_t mine = k1 == best && best != 0 ? expert_of<G>(i1 / 8, g, i1 & 7) : 0x7FFFFFFFu;
      const uint32_t who = group_min<G>(mine);
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        if (r == s * G + g) {
          sel_key[s] = best;
          sel_idx[s] = best != 0 ? static_cast<int>(who) : -1;
        }
      }
      const bool won = best != 0 && mine == who;
      if (won) {
        if (second) {
          k1 = k2;
          i1 = i2;
          second = false;
        } else {                                       // the best of what comes after the one just taken
          const uint32_t lk = k1;
          const int li = i1;
          k1 = 0;
          i1 = 0;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const bool after = key[j] < lk || (key[j] == lk && j > li);
            if (after && key[j] > k1) {
              k1 = key[j];
              i1 = j;
            }
          }
        }
      }
    }
    const bool used = on && top != 0;
    const float m = value_of(top);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      l[j] = key[j] == 0 ? 0.f : expf(l[j] - m);
      sum += l[j];
    }
    sum = group_add<G>(sum);
    // NaN or +inf among the logits makes the sum NaN, and with it every probability of the token
    if (top == 0xFFFFFFFFu || top == 0xFF800000u) sum = __uint_as_float(0x7FC00000u);
    const float inv = used ? 1.f / sum : 0.f;
    if (used) {
#pragma unroll
      for (int j = 0; j < V; ++j) psum[j] = fmaf(l[j], inv, psum[j]);
      if (g == 0) ++used_here;
    }
    float w[SLOTS], chosen = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      w[s] = sel_idx[s] >= 0 ? expf(value_of(sel_key[s]) - m) : 0.f;
      chosen += w[s];
    }
    float scale = inv;
    if (p.normalize) {
      chosen = group_add<G>(chosen);
      scale = used ? (sum != sum ? sum : 1.f / chosen) : 0.f;
    }
    if (token < p.tokens) {
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        const int r = s * G + g;
        if (r < p.k) {
          p.index[token * p.k + r] = sel_idx[s];
          p.gate[token * p.k + r] = sel_idx[s] >= 0 ? w[s] * scale : 0.f;
          if (sel_idx[s] >= 0) atomicAdd(&scount[sel_idx[s]], 1);
        }
      }
    }
  }
  // the CTA's sums, in a fixed order: the warp's token groups, then its warps
#pragma unroll
  for (int j = 0; j < V; ++j) {
    for (int o = G; o < 32; o <<= 1) psum[j] += __shfl_xor_sync(FULL, psum[j], o);
    const int e = expert_of<G>(j / 8, g, j & 7);
    if (lane < G && e < p.experts) dyn[warp * p.experts + e] = psum[j];
  }
  used_here = __reduce_add_sync(FULL, used_here);
  if (lane == 0) si[warp] = used_here;
  let_next_kernel_start();
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += THREADS) {
    float a = 0.f;
    for (int w = 0; w < WARPS; ++w) a += dyn[w * p.experts + e];
    p.part_prob[static_cast<size_t>(blockIdx.x) * p.experts + e] = a;
    p.part_count[static_cast<size_t>(blockIdx.x) * p.experts + e] = scount[e];
  }
  int total = 0;
  for (int w = 0; w < WARPS; ++w) total += si[w];
  if (threadIdx.x == 0) p.part_used[blockIdx.x] = total;
  if (gridDim.x == 1) {                                // the only CTA finishes by itself
    __syncthreads();
    const float share = finish_experts(p, 1, 0, p.experts, sf, si);
    if (threadIdx.x == 0) {
      p.loss[0] = loss_of(share, total, p.experts, p.k);
      p.used[0] = total;
    }
  }
}

// A cluster of CTAs shares the experts; the first one adds the shares of the loss.
constexpr int FINISH_CTAS = 8;

__global__ void __launch_bounds__(512) router_finish_kernel(const RouterParams p) {
  __shared__ float sf[512];
  __shared__ int si[512];
  __shared__ float share;
  wait_for_previous_kernel();
  const uint32_t rank = cluster_ctarank();
  const int per = (p.experts + FINISH_CTAS - 1) / FINISH_CTAS;
  const int e0 = static_cast<int>(rank) * per, e1 = e0 + per < p.experts ? e0 + per : p.experts;
  const float mine = finish_experts(p, p.parts, e0, e1, sf, si);
  if (threadIdx.x == 0) share = mine;
  cluster_sync_all();
  if (rank == 0 && threadIdx.x == 0) {
    float all = 0.f;
    for (int i = 0; i < FINISH_CTAS; ++i) all += __uint_as_float(ld_cluster_u32(map_to_rank(&share, i)));
    int used = 0;
    for (int i = 0; i < p.parts; ++i) used += p.part_used[i];
    p.loss[0] = loss_of(all, used, p.experts, p.k);
    p.used[0] = used;
  }
  cluster_sync_all();                                  // the shares are read before their CTAs end
}

// ---------------------------------------------------------------- backward

template <typename T, bool VEC, int G, int NC>
__global__ void __launch_bounds__(THREADS) router_bwd_kernel(const RouterBwdParams p) {
  extern __shared__ float dyn[];                       // [WARPS][TOK][G * 8 * NC] what the gates add, zero between tokens
  constexpr int V = 8 * NC;
  constexpr int TOK = 32 / G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane % G;
  float* add = dyn + (warp * TOK + lane / G) * (G * V);
#pragma unroll
  for (int j = 0; j < V; ++j) add[expert_of<G>(j / 8, g, j & 7)] = 0.f;
  float c[V];
  {
    const int n = *p.used;
    const float nf = static_cast<float>(n > 0 ? n : 1);
    const float d = p.dloss && n > 0
                        ? *p.dloss * (static_cast<float>(p.experts) / (static_cast<float>(p.k) * nf)) / nf : 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert_of<G>(j / 8, g, j & 7);
      c[j] = e < p.experts ? d * static_cast<float>(p.counts[e]) : 0.f;
    }
  }
  __syncwarp();
  const long long stride = static_cast<long long>(gridDim.x) * WARPS * TOK;
  for (long long base = (static_cast<long long>(blockIdx.x) * WARPS + warp) * TOK; base < p.tokens; base += stride) {
    const long long token = base + lane / G;
    const bool on = token < p.tokens && (!p.valid || p.valid[token] != 0);
    float l[V];
    load_logits<T, VEC, G, NC>(static_cast<const T*>(p.logits) + token * p.stride, on, p.experts, g, l);
    // the gates' share: t_r = gate_r dgate_r (- gate_r sum gate dgate if normalised), put where
    // the expert's lane finds it
    float dot = 0.f;
    if (p.dgate && on) {
      for (int r = g; r < p.k; r += G) {
        if (p.index[token * p.k + r] >= 0) dot = fmaf(p.gate[token * p.k + r], p.dgate[token * p.k + r], dot);
      }
    }
    dot = group_add<G>(dot);
    if (p.dgate && on) {
      for (int r = g; r < p.k; r += G) {
        const int e = p.index[token * p.k + r];
        if (e >= 0 && e < p.experts)
          add[e] = p.gate[token * p.k + r] * (p.dgate[token * p.k + r] - (p.normalize ? dot : 0.f));
      }
    }
    float m = l[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
    m = group_fmax<G>(m);
    float sum = 0.f;
    bool any = false;                                  // some logit is not -inf (NaN counts)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool off = l[j] == __uint_as_float(0xFF800000u);
      any |= !off;
      l[j] = off ? 0.f : expf(l[j] - m);
      sum += l[j];
    }
    sum = group_add<G>(sum);
    float pc = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) pc = fmaf(l[j], c[j], pc);
    pc = group_add<G>(pc);
    const bool some = group_max<G>(any ? 1u : 0u) != 0u;
    const float inv = some ? 1.f / sum : 0.f;
    const float back = pc * inv + (p.normalize ? 0.f : dot);
    __syncwarp();
    if (token < p.tokens) {
      T* out = static_cast<T*>(p.dlogits) + token * p.dstride;
#pragma unroll
      for (int q = 0; q < NC; ++q) {
        const int e0 = expert_of<G>(q, g, 0);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float pr = l[8 * q + j] * inv;
          f[j] = fmaf(pr, c[8 * q + j] - back, add[e0 + j]);
        }
        if constexpr (VEC) {
          if (e0 < p.experts) {
            Eight<T> o;
            o.set(f);
            o.store(out + e0);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e0 + j < p.experts) out[e0 + j] = from_float<T>(f[j]);
        }
      }
    }
    __syncwarp();
    if (p.dgate && on) {
      for (int r = g; r < p.k; r += G) {
        const int e = p.index[token * p.k + r];
        if (e >= 0 && e < p.experts) add[e] = 0.f;
      }
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------- launches

int lanes_for(int experts) {
  int g = 1;
  while (g < 32 && g * 8 < experts) g *= 2;
  return g;
}

template <typename P>
using Kernel = void (*)(P);

template <typename T, bool VEC>
Kernel<RouterParams> fwd_kernel(int g, int nc) {
  if (nc == 4) return router_kernel<T, VEC, 32, 4>;
  if (nc == 2) return router_kernel<T, VEC, 32, 2>;
  switch (g) {
    case 1: return router_kernel<T, VEC, 1, 1>;
    case 2: return router_kernel<T, VEC, 2, 1>;
    case 4: return router_kernel<T, VEC, 4, 1>;
    case 8: return router_kernel<T, VEC, 8, 1>;
    case 16: return router_kernel<T, VEC, 16, 1>;
    default: return router_kernel<T, VEC, 32, 1>;
  }
}
template <typename T, bool VEC>
Kernel<RouterBwdParams> bwd_kernel(int g, int nc) {
  if (nc == 4) return router_bwd_kernel<T, VEC, 32, 4>;
  if (nc == 2) return router_bwd_kernel<T, VEC, 32, 2>;
  switch (g) {
    case 1: return router_bwd_kernel<T, VEC, 1, 1>;
    case 2: return router_bwd_kernel<T, VEC, 2, 1>;
    case 4: return router_bwd_kernel<T, VEC, 4, 1>;
    case 8: return router_bwd_kernel<T, VEC, 8, 1>;
    case 16: return router_bwd_kernel<T, VEC, 16, 1>;
    default: return router_bwd_kernel<T, VEC, 32, 1>;
  }
}

bool vec_rows(const void* p, long long stride, int size, int rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (stride * size) % 16 == 0);
}

int pieces_for(int experts, int g) {
  const int nc = (experts + 8 * g - 1) / (8 * g);
  return nc <= 1 ? 1 : nc == 2 ? 2 : 4;
}

template <typename T>
cudaError_t fwd(const RouterParams& p, cudaStream_t s, int* launches) {
  const bool vec = p.experts % 8 == 0 && vec_rows(p.logits, p.stride, sizeof(T), p.tokens);
  const int g = lanes_for(p.experts), nc = pieces_for(p.experts, g);
  const auto kernel = vec ? fwd_kernel<T, true>(g, nc) : fwd_kernel<T, false>(g, nc);
  const size_t smem = static_cast<size_t>(WARPS + 1) * p.experts * 4;
  kernel<<<p.parts, THREADS, smem, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  *launches = 1;
  if (p.parts == 1) return cudaSuccess;
  *launches = 2;
  return launch_after(router_finish_kernel, dim3(FINISH_CTAS), dim3(512), 0, s, p, FINISH_CTAS);
}

template <typename T>
cudaError_t bwd(const RouterBwdParams& p, int sms, cudaStream_t s) {
  const bool vec = p.experts % 8 == 0 && vec_rows(p.logits, p.stride, sizeof(T), p.tokens) &&
                   vec_rows(p.dlogits, p.dstride, sizeof(T), p.tokens);
  const int g = lanes_for(p.experts), nc = pieces_for(p.experts, g);
  const auto kernel = vec ? bwd_kernel<T, true>(g, nc) : bwd_kernel<T, false>(g, nc);
  const size_t smem = static_cast<size_t>(THREADS) * 8 * nc * 4;
  const int per = WARPS * (32 / g);
  const int want = static_cast<int>((static_cast<long long>(p.tokens) + per - 1) / per), most = 4 * sms;
  kernel<<<want < most ? want : most, THREADS, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// CTAs of the forward pass: up to two per SM, at least two tokens per group of lanes in each
// where there are enough of them (one CTA also finishes the sums without a second launch).
int router_parts(int tokens, int experts, int sms) {
  const int per = WARPS * (32 / lanes_for(experts)) * 2;
  int want = static_cast<int>((static_cast<long long>(tokens) + per - 1) / per);
  if (want > 2 * sms) want = 2 * sms;
  if (want > ROUTER_MAX_PARTS) want = ROUTER_MAX_PARTS;
  return want < 1 ? 1 : want;
}

cudaError_t launch_router(RouterParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 0;
  p.parts = router_parts(p.tokens, p.experts, sms);
  if (type == MB_F32) return fwd<float>(p, s, launches);
  if (type == MB_BF16) return fwd<__nv_bfloat16>(p, s, launches);
  return fwd<__half>(p, s, launches);
}

cudaError_t launch_router_backward(RouterBwdParams p, int type, int sms, cudaStream_t s, int* launches) {
  *launches = 1;
  if (type == MB_F32) return bwd<float>(p, sms, s);
  if (type == MB_BF16) return bwd<__nv_bfloat16>(p, sms, s);
  return bwd<__half>(p, sms, s);
}

}  // namespace mb
