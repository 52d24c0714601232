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
  int kb0, kb1;            // the unit's blocks of 64 of the contraction (the same in each pass)
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
  if (J.splits > 1) {                            // (blocks < 2^25, splits < 2^5)
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
    if (units <= pairs) first = units;             // one each
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
__device__ __forceinline__ float inverse_one_plus_exp2(float t) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ float sigmoid(float x) { return inverse_one_plus_exp2(x * -1.4426950408889634f); }
constexpr float GELU_SCALE = 1.5957691216057308f;    // 2 sqrt(2 / pi): tanh(u) = 2 sigmoid(2 u) - 1
constexpr float GELU_CUBE = 0.044715f;

// max(z, 0), NaN for NaN.
__device__ __forceinline__ float relu(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
  return r;
}

// Two at a time: what the exponentials leave to do goes two to an instruction.
template <int ACT>
__device__ __forceinline__ float2 activate(float2 z) {
  if constexpr (ACT == MB_ACT_GELU) {
    // z s(z (a + b z^2)), the exponent's log2(e) in a and b
    constexpr float A = -GELU_SCALE * 1.4426950408889634f, B = A * GELU_CUBE;
    const float2 t = __fmul2_rn(z, __ffma2_rn(__fmul2_rn(z, z), make_float2(B, B), make_float2(A, A)));
    return __fmul2_rn(z, make_float2(inverse_one_plus_exp2(t.x), inverse_one_plus_exp2(t.y)));
  } else if constexpr (ACT == MB_ACT_SILU) {
    const float2 t = __fmul2_rn(z, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    return __fmul2_rn(z, make_float2(inverse_one_plus_exp2(t.x), inverse_one_plus_exp2(t.y)));
  } else if constexpr (ACT == MB_ACT_RELU2) {
    const float2 t = make_float2(relu(z.x), relu(z.y));
    return __fmul2_rn(t, t);
  } else if constexpr (ACT == MB_ACT_RELU) {
    return make_float2(relu(z.x), relu(z.y));
  } else {
    return z;
  }
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
    // past 16 p is 0 or 1 and the slope is p, which a product that overflows (z^3 from 10^13 on) would make NaN; an
    // infinite z makes it (z 0)
    const float c = fminf(fmaxf(z, -16.f), 16.f);
    return p * fmaf(GELU_SCALE * c * (1.f - p), fmaf(3.f * GELU_CUBE * c, c, 1.f), fmaf(z, 0.f, 1.f));
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

// ---------------------------------------------------------------- dz by pieces

__device__ __forceinline__ unsigned load_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Orders this thread's generic accesses of global memory with asynchronous (TMA) ones.
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// dz of rows [begin, end) of one group, columns col .. col + 7, eight rows on their way at a time; the sums of dz.
template <typename T, int ACT, int ROWS>
__device__ __forceinline__ void slope_rows_of(const T* dy, long long dy_ld, const T* z, long long z_ld, T* dz, long long dz_ld,
                                              float (&sum)[8]) {
  Eight<T> g[ROWS], x[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    g[i].load(dy + i * dy_ld);
    x[i].load(z + i * z_ld);
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float v[8], s[8];
    g[i].get(v);
    x[i].get(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] *= slope<ACT>(s[j]);
      sum[j] += v[j];
    }
    g[i].set(v);
    g[i].store(dz + i * dz_ld);
  }
}
template <typename T, int ACT>
__device__ __forceinline__ void slope_piece(const LinearSlopeParams& p, int begin, int end, int col, float (&sum)[8]) {
  constexpr int ROWS = 8;
  const T* dy = static_cast<const T*>(p.dy) + begin * p.dy_ld + col;
  const T* z = static_cast<const T*>(p.z) + begin * p.z_ld + col;
  T* dz = static_cast<T*>(p.dz) + begin * p.dz_ld + col;
  int left = end - begin;
  for (; left >= ROWS; left -= ROWS, dy += ROWS * p.dy_ld, z += ROWS * p.z_ld, dz += ROWS * p.dz_ld)
    slope_rows_of<T, ACT, ROWS>(dy, p.dy_ld, z, p.z_ld, dz, p.dz_ld, sum);
  for (; left > 0; --left, dy += p.dy_ld, z += p.z_ld, dz += p.dz_ld)
    slope_rows_of<T, ACT, 1>(dy, p.dy_ld, z, p.z_ld, dz, p.dz_ld, sum);
}

// Piece number `at` by one warp, and its report.
template <typename T>
__device__ __forceinline__ void do_piece(const LinearAhead& A, const Groups& G, int at, int lane) {
  const LinearSlopeParams& p = A.slope;
  const int turn = at / A.column_groups, column = at - turn * A.column_groups;
  const int step = turn / A.ways, slab = (turn - step * A.ways) * A.per_way + step;
  if (slab >= A.slabs) return;                     // (the last range may be shorter)
  const int col = column * 256 + 8 * lane;
  const int begin = slab * LINEAR_PIECE_ROWS, end = min(begin + LINEAR_PIECE_ROWS, G.row[G.n]);
  int g = 0;
  if (G.n > 1) {                                   // the first group whose rows end past the piece's begin
    int hi = G.n;
    while (g < hi) {
      const int mid = (g + hi) >> 1;
      if (G.row[mid + 1] > begin) hi = mid;
      else g = mid + 1;
    }
  }
  for (int row = begin; g < G.n && row < end; ++g) {
    const int stop = min(end, G.row[g + 1]);
    if (stop <= row) continue;
    if (col < p.cols) {
      float sum[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = 0.f;
      with_activation(p.act, [&](auto act) { slope_piece<T, decltype(act)::value>(p, row, stop, col, sum); });
      if (p.parts) {
        float4* to = reinterpret_cast<float4*>(p.parts + static_cast<long long>(slab + g) * p.cols + col);
        to[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        to[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
      }
    }
    row = stop;
  }
  fence_async_global();
  __syncwarp();
  if (lane == 0) add_release(&A.done[slab], 1u);
}

// Which slabs of dz a producer has seen done: [begin, end).
struct Seen {
  int begin = 0, end = 0;
  // Waits (bounded, as a whole warp) until the slabs of rows [from, to) are.
  __device__ __forceinline__ bool rows(const LinearAhead& A, int from, int to, int lane, const volatile int* abort_flag) {
    const int first = from / LINEAR_PIECE_ROWS, last = min((to - 1) / LINEAR_PIECE_ROWS, A.slabs - 1);
    if (last < first || (first >= begin && last < end)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 0;; ++i) {
      const int slab = first + lane;
      const bool ok = slab < A.slabs && load_acquire(&A.done[slab]) >= static_cast<unsigned>(A.column_groups);
      const unsigned missing = ~__ballot_sync(0xffffffffu, ok);
      begin = first;
      end = first + (missing ? __ffs(missing) - 1 : 32);
      if (last < end) break;
      __nanosleep(200);
      if (__any_sync(0xffffffffu, *abort_flag || globaltimer_ns() - t0 > WAIT_LIMIT_NS)) return false;
    }
    // each lane has acquired a slab of its own, and any one of them issues the loads of all: votes order no memory
    __syncwarp();
    fence_async_global();
    return true;
  }
};

// ---------------------------------------------------------------- chunks of 32 rows x 64 columns

// A warp's chunk in shared memory: rows of 128 bytes whose 16-byte pieces are exchanged by row (TMA's 128-byte swizzle), so
// that lanes that each take a row, and lanes that each take a piece of neighbouring rows, hit distinct banks.  Whole lines
// of memory: the TMA unit takes about two cycles for a row of a box whatever its length, and stores of 64-byte rows held
// up the products' loads (65536x768->2816 with gelu, z and a bias: 284 us in boxes of 32 columns, 267 in these).
constexpr int CHUNK_COLS = 64;
constexpr int CHUNK_BYTES = 32 * CHUNK_COLS * 2;
__device__ __forceinline__ uint32_t chunk_at(int row, int piece) {
  return static_cast<uint32_t>(row * 128 + 16 * (piece ^ (row & 7)));
}

// The chunk's row-wise copies in accesses of ACCESS bytes, neighbouring lanes along rows: f(place in the buffer, place in memory)
// for rows [0, rows) and columns [0, cols).
template <int ACCESS, typename F>
__device__ __forceinline__ void each_piece(uint16_t* at, long long ld, int rows, int cols, int lane, F&& f) {
  constexpr int PIECES = CHUNK_COLS * 2 / ACCESS;              // of a row
  constexpr int LANES = PIECES < 32 ? PIECES : 32, STEP = 32 / LANES;
#pragma unroll
  for (int part = 0; part < PIECES / LANES; ++part) {
    const int piece = part * LANES + lane % LANES, col = piece * (ACCESS / 2);
    const int row = lane / LANES;
    uint16_t* to = at + row * ld + col;
    const int some = col < cols ? rows : 0;
#pragma unroll 16
    for (int i = 0; i < 32 / STEP; ++i, to += STEP * ld)
      if (i * STEP + row < some) f(chunk_at(i * STEP + row, piece * ACCESS / 16) + piece * ACCESS % 16, to);
  }
}
template <int ACCESS>
using AccessWord = std::conditional_t<ACCESS == 16, uint4, std::conditional_t<ACCESS == 4, uint32_t, uint16_t>>;

// To memory, or from there (what lies outside is left as it is).
template <int ACCESS>
__device__ __forceinline__ void store_chunk(const uint8_t* buf, uint16_t* to, long long ld, int rows, int cols, int lane) {
  each_piece<ACCESS>(to, ld, rows, cols, lane, [&](uint32_t at, uint16_t* p) {
    *reinterpret_cast<AccessWord<ACCESS>*>(p) = *reinterpret_cast<const AccessWord<ACCESS>*>(buf + at);
  });
}
template <int ACCESS>
__device__ __forceinline__ void load_chunk(uint8_t* buf, const uint16_t* from, long long ld, int rows, int cols, int lane) {
  each_piece<ACCESS>(const_cast<uint16_t*>(from), ld, rows, cols, lane, [&](uint32_t at, const uint16_t* p) {
    *reinterpret_cast<AccessWord<ACCESS>*>(buf + at) = *reinterpret_cast<const AccessWord<ACCESS>*>(p);
  });
}
__device__ __forceinline__ void store_chunk(int access, const uint8_t* buf, uint16_t* to, long long ld, int rows, int cols, int lane) {
  if (access == 16) store_chunk<16>(buf, to, ld, rows, cols, lane);
  else if (access == 4) store_chunk<4>(buf, to, ld, rows, cols, lane);
  else store_chunk<2>(buf, to, ld, rows, cols, lane);
}

// A lane's row of a chunk: 64 sums, as pairs.
struct Row {
  float2 v[CHUNK_COLS / 2];
};

// Rounded to T into the buffer.
template <typename T>
__device__ __forceinline__ void put_row(uint8_t* buf, const Row& r, int lane) {
#pragma unroll
  for (int i = 0; i < CHUNK_COLS / 8; ++i)
    *reinterpret_cast<uint4*>(buf + chunk_at(lane, i)) =
        make_uint4(pack2(r.v[4 * i].x, r.v[4 * i].y, T()), pack2(r.v[4 * i + 1].x, r.v[4 * i + 1].y, T()),
                   pack2(r.v[4 * i + 2].x, r.v[4 * i + 2].y, T()), pack2(r.v[4 * i + 3].x, r.v[4 * i + 3].y, T()));
}
// Eight elements added to the pairs from 4 i on.
template <typename T>
__device__ __forceinline__ void add_piece(Row& r, int i, uint4 q) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) r.v[4 * i + j] = __fadd2_rn(r.v[4 * i + j], unpack2(u[j], T()));
}

// The bias of a chunk's columns, two to a lane, zeros past the last.  Asked for before the sums are there: with the ring in
// shared memory next to nothing is left to cache it, and a chunk that waits for it takes 1700 cycles longer.
template <typename T>
__device__ __forceinline__ float2 bias_of(const LinearParams& P, const LinearJob& J, int group, int col0, int lane) {
  const int col = col0 + 2 * lane;
  const long long at = static_cast<long long>(group) * J.N + col;
  float2 b = make_float2(0.f, 0.f);
  if (!P.bias) return b;
  if (P.bias_f32) {
    const float* p = static_cast<const float*>(P.bias) + at;
    if (col < J.N) b.x = p[0];
    if (col + 1 < J.N) b.y = p[1];
  } else {
    const T* p = static_cast<const T*>(P.bias) + at;
    if (col < J.N) b.x = to_float(p[0]);
    if (col + 1 < J.N) b.y = to_float(p[1]);
  }
  return b;
}
__device__ __forceinline__ void add_bias(Row& r, float2 bias) {
#pragma unroll
  for (int i = 0; i < CHUNK_COLS / 2; ++i)
    r.v[i] = __fadd2_rn(r.v[i], make_float2(__shfl_sync(0xffffffffu, bias.x, i), __shfl_sync(0xffffffffu, bias.y, i)));
}

// What an epilogue's warp holds: its rows of the tile and its chunk buffer.
struct WarpPlace {
  int row0;                // D's row of lane 0
  int rows;                // of the 32, how many belong to the group
  int lane;
  uint8_t* buf;            // CHUNK_BYTES
};

// What the buffer held has left it.
template <bool BULK>
__device__ __forceinline__ void chunk_left(const WarpPlace& w) {
  if (BULK && w.lane == 0) bulk_wait_read_all();
  __syncwarp();
}

// The chunk in the buffer to a result: whole by TMA where the layout allows it (BULK), else by row-wise stores.
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

// The residual's chunks on their way by TMA into a buffer of the warp's own, a chunk ahead: their way from memory is longer
// than a short product's tile (65536x768->2816 with a residual: 593 us where it is waited for, 228 so).  Rows that TMA cannot address are read into
// the chunk's buffer when they are needed.
struct ResidualFeed {
  uint8_t* buf;            // CHUNK_BYTES, or null: not by TMA
  uint64_t* landed;
  uint32_t asked, used;
  __device__ __forceinline__ void ask(const LinearParams& P, const LinearJob& J, const WarpPlace& w, int col0) {
    if (!buf || w.rows <= 0 || col0 >= J.N) return;
    ++asked;
    if (w.lane != 0) return;
    mbar_expect_tx(landed, CHUNK_BYTES);
    tma_load_3d(buf, &P.residual_map, landed, col0, w.row0, 0);
  }
};

// One chunk's sums to the results: columns col0 .. col0 + 63.
//   z = v + bias;  y = act(z) + residual;  each rounded once.
// Both leave through one buffer: a second one would cost the products a stage of their ring, and with it 10 % of their rate.
// False if a wait for the residual ran out.
template <bool FORWARD, typename T, bool BULK>
__device__ __forceinline__ bool finish_chunk(const LinearParams& P, const LinearJob& J, const Unit& u, const WarpPlace& w, Row& r,
                                             int col0, float2 bias, ResidualFeed& res, const volatile int* abort_flag) {
  const int cols = J.N - col0;
  if (w.rows <= 0 || cols <= 0) return true;       // (the same for all lanes)
  if constexpr (FORWARD) {
    if (P.bias) add_bias(r, bias);
    if (P.z) {
      chunk_left<BULK>(w);
      put_row<T>(w.buf, r, w.lane);
      send_chunk<BULK>(w, J.bulk, &P.z_map, 0, P.z_access, P.z, P.z_ld, col0, cols);
    }
    with_activation(P.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < CHUNK_COLS / 2; ++i) r.v[i] = activate<decltype(act)::value>(r.v[i]);
    });
  }
  if constexpr (FORWARD) {
    if (BULK && res.buf) {
      if (!__all_sync(0xffffffffu, mbar_wait_or_abort(res.landed, res.used & 1, abort_flag))) return false;
      ++res.used;
#pragma unroll
      for (int i = 0; i < CHUNK_COLS / 8; ++i)
        add_piece<T>(r, i, *reinterpret_cast<const uint4*>(res.buf + chunk_at(w.lane, i)));
      __syncwarp();                                // read: the next may land
      if (col0 + 2 * CHUNK_COLS < u.n0 + u.wide) res.ask(P, J, w, col0 + 2 * CHUNK_COLS);
    }
  }
  chunk_left<BULK>(w);
  if constexpr (FORWARD) {
    if (P.residual && !(BULK && res.buf)) {
      const uint16_t* from = static_cast<const uint16_t*>(P.residual) + w.row0 * P.residual_ld + col0;
      if (P.residual_access == 16) load_chunk<16>(w.buf, from, P.residual_ld, w.rows, cols, w.lane);
      else if (P.residual_access == 4) load_chunk<4>(w.buf, from, P.residual_ld, w.rows, cols, w.lane);
      else load_chunk<2>(w.buf, from, P.residual_ld, w.rows, cols, w.lane);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < CHUNK_COLS / 8; ++i)     // (a lane reads and writes its own row)
        add_piece<T>(r, i, *reinterpret_cast<const uint4*>(w.buf + chunk_at(w.lane, i)));
    }
  }
  put_row<T>(w.buf, r, w.lane);
  send_chunk<BULK>(w, J.bulk, &J.d, u.group * J.over_rows, J.access, static_cast<uint16_t*>(J.out) + u.group * J.group_stride,
                   J.ld, col0, cols);
  return true;
}

// Where the warp `warp` of CTA `rank` keeps the fp32 sums of one chunk of a unit: 16 float4 per lane, 32 lanes side by side.
__device__ __forceinline__ float4* part_of(const LinearJob& J, const Unit& u, int split, uint32_t rank, int warp, int chunk) {
  const long long tile = split * J.part_tiles + u.tile;
  return reinterpret_cast<float4*>(J.parts) + (((tile * 2 + rank) * 8 + warp) * (J.wide / 128) + chunk) * 16 * 32;
}

}  // namespace mb
