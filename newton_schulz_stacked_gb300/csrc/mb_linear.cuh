// What the kernels of mb_linear share: a call's groups of rows, its tiles, activations, and a warp's 32 x 32 chunk of a
// result on its way to memory.
#pragma once

#include <type_traits>

#include "mb_device.cuh"
#include "mb_linear.h"
#include "mb_rows.cuh"
#include "muonbank.h"

namespace mb {

// ---------------------------------------------------------------- groups

// Where the groups' rows and tiles begin, in shared memory: rows of group g are [row[g], row[g + 1]), its tiles of 256 rows
// [tile[g], tile[g + 1]).
struct Groups {
  int* row;
  int* tile;
  int n;
};
constexpr int GROUPS_BYTES = 2 * (LINEAR_MAX_GROUPS + 1) * 4;

// One warp fills them in from the ends in device memory.  Ends that fall, or pass the number of rows, are held to what can
// be (each at least the one before, at most `rows`), so that no access leaves the tensors; true if any was.
__device__ __forceinline__ bool fill_groups(const Groups& G, const int* ends, int rows, int lane) {
  int before = 0, tiles = 0;
  bool bad = false;
  if (lane == 0) G.row[0] = G.tile[0] = 0;
  for (int g0 = 0; g0 < G.n; g0 += 32) {
    const int g = g0 + lane;
    const int given = g >= G.n || !ends ? rows : ends[g];
    int end = min(max(given, 0), rows);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int other = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end = max(end, other);
    }
    end = max(end, before);
    bad |= g < G.n && end != given;
    const int left = __shfl_up_sync(0xffffffffu, end, 1);
    const int begin = lane == 0 ? before : left;
    int sum = (end - begin + LINEAR_TILE - 1) / LINEAR_TILE;
    if (g >= G.n) sum = 0;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int other = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += other;
    }
    if (g < G.n) {
      G.row[g + 1] = end;
      G.tile[g + 1] = tiles + sum;
    }
    before = __shfl_sync(0xffffffffu, end, 31);
    tiles += __shfl_sync(0xffffffffu, sum, 31);
  }
  return __any_sync(0xffffffffu, bad);
}

// ---------------------------------------------------------------- tiles

// One pair's unit of work: a tile of a job, or a part of its contraction.
struct Unit {
  int job, group;
  int tile;                // of the job
  int split;
  int m0, m_end;           // D's rows: the tile's first, and where the group's (or matrix's) end
  int n0, wide;            // D's columns
  int k_begin, k_end;      // over_rows: the group's rows
  int kb0, kb1;            // blocks of 64 of the contraction
};

// (the host refuses what 31 bits cannot number: a division of 64 bits takes a role longer than a block's MMAs)
__device__ __forceinline__ int job_units(const LinearJob& J, const Groups& G) {
  return (J.over_rows ? G.n * J.m_tiles : G.tile[G.n]) * J.n_tiles * J.splits;
}

__device__ __forceinline__ void decode_tile(const LinearJob& J, const Groups& G, int tile, Unit& u) {
  u.tile = tile;
  int m = tile / J.n_tiles;
  const int n = tile - m * J.n_tiles;
  int blocks;
  if (J.over_rows) {
    u.group = m / J.m_tiles;
    m -= u.group * J.m_tiles;
    u.m0 = m * LINEAR_TILE;
    u.m_end = J.M;
    u.k_begin = G.row[u.group];
    u.k_end = G.row[u.group + 1];
    blocks = (u.k_end - u.k_begin + LINEAR_DEEP - 1) / LINEAR_DEEP;
  } else {
    int lo = 0, hi = G.n;                        // the group whose tiles hold m
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (G.tile[mid] <= m) lo = mid;
      else hi = mid;
    }
    u.group = lo;
    u.m0 = G.row[lo] + (m - G.tile[lo]) * LINEAR_TILE;
    u.m_end = G.row[lo + 1];
    u.k_begin = 0;
    u.k_end = J.K;
    blocks = (J.K + LINEAR_DEEP - 1) / LINEAR_DEEP;
  }
  u.n0 = n * J.wide;
  // the last columns' tile is as narrow as its operand's layout allows
  const int left = J.N - u.n0, step = J.b_mn ? 128 : 64;
  u.wide = min(J.wide, (left + step - 1) & -step);
  u.kb0 = 0;
  u.kb1 = blocks;
  if (J.splits > 1) {                            // (blocks < 2^24, splits < 2^5)
    u.kb0 = blocks * u.split / J.splits;
    u.kb1 = blocks * (u.split + 1) / J.splits;
  }
}

// The units that a pair takes, in order: of the first job every `pairs`th; where those do not come out even, the pairs that have
// one less take `extra` of the second job's each; then every `pairs`th of what is left.
struct Deal {
  int pair, pairs, first, units;   // first: the first job's units
  int firsts, extras;              // that this pair takes
  int rest, skipped;               // pairs with an extra share begin at `skipped`; the units from `rest` on are left
  __device__ __forceinline__ Deal(int pair_, int pairs_, int first_, int units_, int extra) {
    pair = pair_;
    pairs = pairs_;
    first = first_;
    units = units_;
    firsts = pair < first ? (first - pair + pairs - 1) / pairs : 0;
    skipped = first % pairs;
    const int others = pairs - skipped;
    extra = skipped > 0 ? min(extra, (units - first) / others) : 0;
    extras = pair >= skipped ? extra : 0;
    rest = first + extra * others;
  }
  // The pair's unit number i; none from `units` on.
  __device__ __forceinline__ int operator()(int i) const {
    if (i < firsts) return pair + i * pairs;
    i -= firsts;
    if (i < extras) return first + (pair - skipped) + i * (pairs - skipped);
    return rest + pair + (i - extras) * pairs;
  }
  __device__ __forceinline__ int count() const {
    const int left = units - rest - pair;
    return firsts + extras + (left > 0 ? (left + pairs - 1) / pairs : 0);
  }
};

__device__ __forceinline__ void decode_unit(const LinearParams& P, const Groups& G, int first_units, int at, Unit& u) {
  u.job = at >= first_units ? 1 : 0;
  if (u.job) at -= first_units;
  const LinearJob& J = P.job[u.job];
  u.split = 0;
  if (J.splits > 1) {
    const int tile = at / J.splits;
    u.split = at - tile * J.splits;
    at = tile;
  }
  decode_tile(J, G, at, u);
}

// ---------------------------------------------------------------- activations

// exp2 and the reciprocal are the hardware's, within about 2^-22 of their values: a result is rounded to 16 bits.
__device__ __forceinline__ float sigmoid(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
constexpr float GELU_SCALE = 1.5957691216057308f;    // 2 sqrt(2 / pi): tanh(u) = 2 sigmoid(2 u) - 1
constexpr float GELU_CUBE = 0.044715f;

// (comparisons are written so that NaN stays NaN)
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == MB_ACT_RELU) return z < 0.f ? 0.f : z;
  if (ACT == MB_ACT_RELU2) {
    const float r = z < 0.f ? 0.f : z;
    return r * r;
  }
  if (ACT == MB_ACT_SILU) return z * sigmoid(z);
  if (ACT == MB_ACT_GELU) return z * sigmoid(GELU_SCALE * fmaf(GELU_CUBE * z * z, z, z));
  return z;
}

template <int ACT>
__device__ __forceinline__ float slope(float z) {
  if (ACT == MB_ACT_RELU) return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
  if (ACT == MB_ACT_RELU2) return z < 0.f ? 0.f : 2.f * z;
  if (ACT == MB_ACT_SILU) {
    const float p = sigmoid(z);
    return p * fmaf(z, 1.f - p, 1.f);
  }
  if (ACT == MB_ACT_GELU) {
    const float p = sigmoid(GELU_SCALE * fmaf(GELU_CUBE * z * z, z, z));
    return p * fmaf(GELU_SCALE * z * (1.f - p), fmaf(3.f * GELU_CUBE * z, z, 1.f), 1.f);
  }
  return 1.f;
}

// f<ACT>() with the run-time activation as a constant.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  switch (act) {
    case MB_ACT_RELU: f(std::integral_constant<int, MB_ACT_RELU>()); break;
    case MB_ACT_RELU2: f(std::integral_constant<int, MB_ACT_RELU2>()); break;
    case MB_ACT_SILU: f(std::integral_constant<int, MB_ACT_SILU>()); break;
    case MB_ACT_GELU: f(std::integral_constant<int, MB_ACT_GELU>()); break;
    default: f(std::integral_constant<int, MB_ACT_NONE>()); break;
  }
}

// ---------------------------------------------------------------- chunks of 32 x 32

// A warp's chunk in shared memory: rows of 64 bytes whose 16-byte pieces are exchanged by row, so that lanes that each take
// a row, and lanes that each take a piece of neighbouring rows, hit distinct banks.
constexpr int CHUNK_BYTES = 32 * 64;
__device__ __forceinline__ uint32_t chunk_at(int row, int piece) {
  return static_cast<uint32_t>(row * 64 + 16 * (piece ^ ((row >> 1) & 3)));
}

// Rows [0, rows) and columns [0, cols) of the chunk to memory, neighbouring lanes along rows.
template <int ACCESS>
__device__ __forceinline__ void store_chunk(const uint8_t* buf, uint16_t* to, long long ld, int rows, int cols, int lane) {
  constexpr int LANES = 64 / ACCESS, STEP = 32 / LANES;      // lanes of a row, rows at a time
  const int piece = lane % LANES, col = piece * (ACCESS / 2);
#pragma unroll
  for (int i = 0; i < LANES; ++i) {
    const int row = i * STEP + lane / LANES;
    if (row < rows && col < cols) {
      const uint8_t* from = buf + chunk_at(row, piece * ACCESS / 16) + piece * ACCESS % 16;
      uint16_t* at = to + row * ld + col;
      if constexpr (ACCESS == 16) *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(from);
      else if constexpr (ACCESS == 4) *reinterpret_cast<uint32_t*>(at) = *reinterpret_cast<const uint32_t*>(from);
      else *at = *reinterpret_cast<const uint16_t*>(from);
    }
  }
}
__device__ __forceinline__ void store_chunk(int access, const uint8_t* buf, void* to, long long ld, int rows, int cols, int lane) {
  uint16_t* at = static_cast<uint16_t*>(to);
  if (access == 16) store_chunk<16>(buf, at, ld, rows, cols, lane);
  else if (access == 4) store_chunk<4>(buf, at, ld, rows, cols, lane);
  else store_chunk<2>(buf, at, ld, rows, cols, lane);
}

// The same from memory; what lies outside is left as it is.
template <int ACCESS>
__device__ __forceinline__ void load_chunk(uint8_t* buf, const uint16_t* from, long long ld, int rows, int cols, int lane) {
  constexpr int LANES = 64 / ACCESS, STEP = 32 / LANES;
  const int piece = lane % LANES, col = piece * (ACCESS / 2);
#pragma unroll
  for (int i = 0; i < LANES; ++i) {
    const int row = i * STEP + lane / LANES;
    if (row < rows && col < cols) {
      uint8_t* to = buf + chunk_at(row, piece * ACCESS / 16) + piece * ACCESS % 16;
      const uint16_t* at = from + row * ld + col;
      if constexpr (ACCESS == 16) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(at);
      else if constexpr (ACCESS == 4) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(at);
      else *reinterpret_cast<uint16_t*>(to) = *at;
    }
  }
}
__device__ __forceinline__ void load_chunk(int access, uint8_t* buf, const void* from, long long ld, int rows, int cols, int lane) {
  const uint16_t* at = static_cast<const uint16_t*>(from);
  if (access == 16) load_chunk<16>(buf, at, ld, rows, cols, lane);
  else if (access == 4) load_chunk<4>(buf, at, ld, rows, cols, lane);
  else load_chunk<2>(buf, at, ld, rows, cols, lane);
}

// The lane's row of the chunk: rounded to T into it, or widened out of it.
template <typename T>
__device__ __forceinline__ void put_row(uint8_t* buf, const float (&v)[32], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(buf + chunk_at(lane, i)) =
        make_uint4(pack2(v[8 * i], v[8 * i + 1], T()), pack2(v[8 * i + 2], v[8 * i + 3], T()),
                   pack2(v[8 * i + 4], v[8 * i + 5], T()), pack2(v[8 * i + 6], v[8 * i + 7], T()));
}
template <typename T>
__device__ __forceinline__ void add_row(const uint8_t* buf, float (&v)[32], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 q = *reinterpret_cast<const uint4*>(buf + chunk_at(lane, i));
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2(u[j], T());
      v[8 * i + 2 * j] += f.x;
      v[8 * i + 2 * j + 1] += f.y;
    }
  }
}

// What an epilogue's warp holds: its rows of the tile, its chunk buffer, and the forward pass's bias of its columns.
struct WarpPlace {
  int row0;                // D's row of lane 0
  int rows;                // of the 32, how many belong to the group
  int lane;
  uint8_t* buf;            // CHUNK_BYTES
  float* bias;             // of the chunks that it takes, 32 each
};

// The chunk in the buffer to a result: whole by TMA where the layout allows it (BULK), else by row-wise stores.  The buffer
// may be written again after `chunk_left`.
template <bool BULK>
__device__ __forceinline__ void send_chunk(const WarpPlace& w, bool bulk, const CUtensorMap* map, int batch, int access, void* to,
                                           long long ld, int col0, int cols) {
  if (BULK && bulk && w.rows >= 32) {
    fence_proxy_async_smem();
    __syncwarp();
    if (w.lane == 0) {
      tma_store_3d(map, w.buf, col0, w.row0, batch);
      bulk_commit();
    }
  } else {
    __syncwarp();
    store_chunk(access, w.buf, static_cast<uint16_t*>(to) + w.row0 * ld + col0, ld, w.rows, cols, w.lane);
  }
}
template <bool BULK>
__device__ __forceinline__ void chunk_left(const WarpPlace& w) {
  if (BULK && w.lane == 0) bulk_wait_read_all();
  __syncwarp();
}

// One chunk's sums to the results: columns col0 .. col0 + 31, `bias` those columns' (forward).
//   z = v + bias;  y = act(z) + residual;  each rounded once.
// Both leave through one buffer: a second one would cost the products a stage of their ring, and with it 10 % of their rate.
template <bool FORWARD, typename T, bool BULK>
__device__ __forceinline__ void finish_chunk(const LinearParams& P, const LinearJob& J, const Unit& u, const WarpPlace& w,
                                             float (&v)[32], int col0, const float* bias) {
  const int cols = J.N - col0;
  if (w.rows <= 0 || cols <= 0) return;            // (the same for all lanes)
  if constexpr (FORWARD) {
    if (P.bias) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 b = reinterpret_cast<const float4*>(bias)[i];
        v[4 * i] += b.x;
        v[4 * i + 1] += b.y;
        v[4 * i + 2] += b.z;
        v[4 * i + 3] += b.w;
      }
    }
    if (P.z) {
      chunk_left<BULK>(w);
      put_row<T>(w.buf, v, w.lane);
      send_chunk<BULK>(w, J.bulk, &P.z_map, 0, P.z_access, P.z, P.z_ld, col0, cols);
    }
    with_activation(P.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = activate<decltype(act)::value>(v[i]);
    });
  }
  chunk_left<BULK>(w);
  if constexpr (FORWARD) {
    if (P.residual) {
      load_chunk(P.residual_access, w.buf, static_cast<const uint16_t*>(P.residual) + w.row0 * P.residual_ld + col0,
                 P.residual_ld, w.rows, cols, w.lane);
      __syncwarp();
      add_row<T>(w.buf, v, w.lane);                // (a lane reads and writes its own row)
    }
  }
  put_row<T>(w.buf, v, w.lane);
  send_chunk<BULK>(w, J.bulk, &J.d, u.group * J.over_rows, J.access, static_cast<uint16_t*>(J.out) + u.group * J.group_stride,
                   J.ld, col0, cols);
}

// The bias of the warp's chunks of a unit (chunk i: columns n0 + 32 (half + 2 i)), zeros past the last column.
template <typename T>
__device__ __forceinline__ void fetch_bias(const LinearParams& P, const LinearJob& J, const Unit& u, const WarpPlace& w, int half) {
  if (!P.bias) return;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = u.n0 + 32 * (half + 2 * i) + w.lane;
    const long long at = static_cast<long long>(u.group) * J.N + col;
    float b = 0.f;
    if (col < J.N)
      b = P.bias_f32 ? static_cast<const float*>(P.bias)[at] : to_float(static_cast<const T*>(P.bias)[at]);
    w.bias[32 * i + w.lane] = b;
  }
  __syncwarp();
}

// Where the warp `warp` of CTA `rank` keeps the fp32 sums of one chunk of a unit: 8 float4 per lane, 32 lanes side by side.
__device__ __forceinline__ float4* part_of(const LinearJob& J, const Unit& u, int split, uint32_t rank, int warp, int chunk) {
  const long long tile = split * J.part_tiles + u.tile;
  return reinterpret_cast<float4*>(J.parts) + (((tile * 2 + rank) * 8 + warp) * (J.wide / 64) + chunk) * 8 * 32;
}

}  // namespace mb
