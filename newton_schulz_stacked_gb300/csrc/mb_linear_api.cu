// C entries of the products with bias, activation and residual: checks, the plan of a call (what is copied, how the
// products are cut), tensor maps and the launches.
#include <algorithm>
#include <cmath>

#include "mb_block.h"
#include "mb_device.cuh"
#include "mb_linear.h"
#include "muonbank.h"

namespace mb {
namespace {

#define MB_TRY(expr)            \
  do {                          \
    int r_ = (expr);            \
    if (r_ != MB_OK) return r_; \
  } while (0)

constexpr int64_t MAX_ROWS = 1ll << 30, MAX_WIDTH = 1ll << 20;
constexpr int64_t MAX_PAIRS = 76;        // what the cuts are planned for: the pairs of a GB300's 152 SMs
constexpr int MAX_SPLITS = 16;
// Up to so many elements (of x or y) dz's rounding is kept in a second half.  Over random cases of 1 to 64 rows and widths of 64
// to 2048 the gradients' errors with one half were 1.4 times those of rounding the exact sums, and more than 1.5 times in 3 %,
// none of them above 1610 elements.  The second pass takes 1x768->768 from 10.5 to 12.6 us and 1x2048->2048 from 18 to 28 (in a
// graph), which wider calls are spared.
constexpr int64_t TWO_HALVES = 1 << 11;
// From so many elements on dz is formed under the products' MMAs, below by a launch before them.  Both, with dx, dW and db on
// one GB300, in us: 32768x768->768 100 and 90, 8192x1024->4096 140 and 136, 32768x2048->2048 379 and 390, 65536x768->2816
// 471 and 530, 131072x1024->2816 over 64 groups 1190 and 1278.  (The two products side by side on a share of the pairs
// each, so that neither runs ahead of dz, took 486 and 1199.)
constexpr int64_t AHEAD_ELEMENTS = 3ll << 24;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t parts_of(int64_t n, int64_t by) { return (n + by - 1) / by; }
bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// ---------------------------------------------------------------- checks

int check_two(const void* p, bool need) {
  if (!p) return need ? MB_ERR_NULL : MB_OK;
  return aligned(p, 2) ? MB_OK : MB_ERR_ALIGN;
}

int check_shape(int64_t rows, int64_t in, int64_t out, int64_t groups, const int32_t* ends) {
  if (rows < 0 || rows > MAX_ROWS || in < 1 || in > MAX_WIDTH || out < 1 || out > MAX_WIDTH) return MB_ERR_SHAPE;
  if (groups < 1 || groups > LINEAR_MAX_GROUPS || (!ends && groups != 1)) return MB_ERR_SHAPE;
  if (groups * in * out > (1ll << 40)) return MB_ERR_SHAPE;
  // tiles are numbered with 32 bits
  const int64_t widest = in > out ? in : out;
  if ((parts_of(rows, LINEAR_TILE) + groups) * parts_of(widest, 128) >= (1ll << 30)) return MB_ERR_SHAPE;
  if (groups * parts_of(out, LINEAR_TILE) * parts_of(in, 128) >= (1ll << 30)) return MB_ERR_SHAPE;
  return aligned(ends, 4) ? MB_OK : MB_ERR_ALIGN;
}

int check_types(int type, int bias_type, int act) {
  if (type != MB_BF16 && type != MB_F16) return MB_ERR_ARG;
  if (bias_type != type && bias_type != MB_F32) return MB_ERR_ARG;
  return act >= MB_ACT_NONE && act <= MB_ACT_GELU ? MB_OK : MB_ERR_ARG;
}

bool bad_stride(int64_t stride, int64_t rows, int64_t cols, bool write) {
  return stride < 0 || stride > (1ll << 36) || (write && rows > 1 && stride < cols);
}

// ---------------------------------------------------------------- operands

// A matrix of 2-byte elements as TMA reads it: the caller's, or a copy of it in the workspace.
struct Operand {
  const void* base;
  int64_t ld;
  bool copy;
  size_t at;               // the copy's place in the workspace
  int64_t rows, cols;
  const void* src;
  int64_t src_ld;
};

Operand operand(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  Operand o{p, ld, false, 0, rows, cols, p, ld};
  if (rows <= 1) o.ld = up(cols, 8);             // a stride that is never taken
  o.copy = !aligned(p, 16) || o.ld % 8 != 0 || o.ld < cols;
  if (o.copy) o.ld = up(cols, 8);
  return o;
}

int access_of(const void* p, int64_t ld, int64_t cols, int64_t rows) {
  const int64_t step = rows > 1 ? ld : 0;
  if (aligned(p, 16) && step % 8 == 0 && cols % 8 == 0) return 16;
  return aligned(p, 4) && step % 2 == 0 && cols % 2 == 0 ? 4 : 2;
}

// ---------------------------------------------------------------- plans

struct Workspace {
  size_t end = 0;
  size_t take(int64_t bytes) {
    const size_t at = end;
    end += static_cast<size_t>(up(bytes, 1024));
    return at;
  }
};

// How a product's tiles are cut: their width, and the parts of the contraction.
struct Cut {
  int wide, splits;
  int64_t tiles, blocks;   // tiles (the most that there can be), blocks of the contraction (on average)
  int64_t n;               // columns
  size_t at;               // of the parts' sums
};

// Time in blocks of 256 x 256 x 64 (0.29 us): one of 128 columns takes 0.85 of it (measured: dW of 65536 rows 458 cycles
// against 551), a tile's begin about one.
double unit_time(const Cut& c) { return static_cast<double>(c.blocks) / c.splits * (c.wide == 256 ? 1.0 : 0.85) + 1; }

// The units of the second product that a pair takes for one of the first that others have more than it.
int extra_units(const Cut& first, const Cut& second) { return static_cast<int>(unit_time(first) / unit_time(second) + 0.5); }

// What the parts of a contraction cost: the join's launch, and 256 KB of sums for each unit there and back.
double join_time(const Cut& c) { return c.splits > 1 ? 10 + 0.27 * c.wide / 256 * static_cast<double>(c.tiles * c.splits) : 0; }

// The time of the busiest pair and the last epilogue.
double busiest(const Cut& first, const Cut* second) {
  const double a = unit_time(first), b = second ? unit_time(*second) : 0;
  const int64_t n = first.tiles * first.splits, rounds = n / MAX_PAIRS, over = n % MAX_PAIRS;
  double t;
  if (!second) {
    t = (rounds + (over > 0)) * a;
  } else {
    const int64_t extra = over > 0 ? extra_units(first, *second) : 0;
    const int64_t rest = second->tiles - extra * (MAX_PAIRS - over);
    const int64_t more = rest > 0 ? parts_of(rest, MAX_PAIRS) : 0;
    const double with = (rounds + (over > 0)) * a + more * b, without = rounds * a + (extra + more) * b;
    t = with > without ? with : without;
  }
  return t + 8 + join_time(first);
}

// The cut of tiles and contraction that takes the busiest pair least time, wide and whole where others gain little.
Cut cut(int64_t m_tiles, int64_t n, int64_t blocks, const Cut* second) {
  Cut best{};
  double least = 0;
  for (int wide = n <= 128 ? 128 : 256; wide >= 128; wide /= 2)
    for (int s = 1; s <= MAX_SPLITS && (s == 1 || blocks / s >= 8); ++s) {
      const Cut c{wide, s, m_tiles * parts_of(n, wide), blocks, n, 0};
      const double t = busiest(c, second);
      if (best.wide == 0 || t < 0.97 * least) {
        best = c;
        least = t;
      }
    }
  return best;
}

// Two products of few tiles, with a pair for every unit: both in parts where that is shorter.
void cut_few(Cut& first, Cut& second) {
  Cut a = first, b = second;
  double least = 0;
  bool any = false;
  for (int ways = 0; ways < 4; ++ways)
    for (int i = 1; i <= MAX_SPLITS && (i == 1 || first.blocks / i >= 4); ++i)
      for (int j = 1; j <= MAX_SPLITS && (j == 1 || second.blocks / j >= 4); ++j) {
        const int a_wide = ways & 1 ? 128 : 256, b_wide = ways & 2 ? 128 : 256;
        const Cut f{a_wide, i, first.tiles / parts_of(first.n, first.wide) * parts_of(first.n, a_wide), first.blocks, first.n, 0};
        const Cut s{b_wide, j, second.tiles / parts_of(second.n, second.wide) * parts_of(second.n, b_wide), second.blocks, second.n, 0};
        if (f.tiles * i + s.tiles * j > MAX_PAIRS) continue;
        const double t = std::max(unit_time(f), unit_time(s)) + 8 + join_time(f) + join_time(s);
        if (!any || t < 0.97 * least) {
          any = true;
          least = t;
          a = f;
          b = s;
        }
      }
  if (any && least < busiest(first, &second)) {
    first = a;
    second = b;
  }
}

void reserve_parts(Cut& c, Workspace& ws) {
  if (c.splits > 1) c.at = ws.take(c.splits * c.tiles * c.wide * LINEAR_TILE * 4);
}

struct ForwardPlan {
  Operand x, w;
  Cut y;
  size_t end;
};

ForwardPlan plan_forward(const mb_linear_desc& d) {
  ForwardPlan p{};
  Workspace ws;
  p.x = operand(d.x, d.x_stride, d.rows, d.in);
  p.w = operand(d.weight, d.in, static_cast<int64_t>(d.groups) * d.out, d.in);
  if (p.x.copy) p.x.at = ws.take(p.x.rows * p.x.ld * 2);
  if (p.w.copy) p.w.at = ws.take(p.w.rows * p.w.ld * 2);
  p.y = cut(parts_of(d.rows, LINEAR_TILE) + (d.ends ? d.groups : 0), d.out, parts_of(d.in, LINEAR_DEEP), nullptr);
  reserve_parts(p.y, ws);
  p.end = ws.end;
  return p;
}

struct BackwardPlan {
  bool slope;              // dz is formed (else it is dy)
  bool ahead;              // by the products' launch
  size_t counters;         // ahead: the next piece, and the column groups done of each slab
  int64_t counter_bytes;
  int low;                 // columns from dz to its low halves, or 0
  Operand dz, x, w;
  Cut dx, dw;
  int slab;
  int64_t slabs;
  size_t db_parts, end;
};

BackwardPlan plan_backward(const mb_linear_backward_desc& d) {
  BackwardPlan p{};
  Workspace ws;
  const bool products = d.dx || d.dweight;
  p.slope = d.activation != MB_ACT_NONE;
  if (p.slope) {
    // The products take dz rounded to 16 bits, half a step in every term; the smallest calls take it in two halves.
    p.low = d.rows * (d.in < d.out ? d.in : d.out) <= TWO_HALVES ? static_cast<int>(up(d.out, LINEAR_DEEP)) : 0;
    const int64_t width = p.low ? p.low + d.out : d.out;
    p.dz = Operand{nullptr, p.low ? 2 * p.low : up(width, 8), false, 0, d.rows, width, nullptr, 0};
    p.dz.at = ws.take(d.rows * p.dz.ld * 2);
  } else if (products) {
    p.dz = operand(d.dy, d.dy_stride, d.rows, d.out);
    if (p.dz.copy) p.dz.at = ws.take(p.dz.rows * p.dz.ld * 2);
  }
  if (d.dweight) {
    p.x = operand(d.x, d.x_stride, d.rows, d.in);
    if (p.x.copy) p.x.at = ws.take(p.x.rows * p.x.ld * 2);
  }
  if (d.dx) {
    p.w = operand(d.weight, d.in, static_cast<int64_t>(d.groups) * d.out, d.in);
    if (p.w.copy) p.w.at = ws.take(p.w.rows * p.w.ld * 2);
    p.dx = cut(parts_of(d.rows, LINEAR_TILE) + (d.ends ? d.groups : 0), d.in, parts_of(d.out, LINEAR_DEEP) * (p.low ? 2 : 1), nullptr);
    if (d.dweight) p.dx.splits = 1;              // dealt out after the other's units, which even them out
  }
  if (d.dweight)
    p.dw = cut(d.groups * parts_of(d.out, LINEAR_TILE), d.in, parts_of(parts_of(d.rows, d.groups), LINEAR_DEEP) * (p.low ? 2 : 1),
               d.dx ? &p.dx : nullptr);
  if (d.dx && d.dweight) cut_few(p.dw, p.dx);
  if (d.dweight) reserve_parts(p.dw, ws);
  if (d.dx) reserve_parts(p.dx, ws);
  p.ahead = p.slope && !p.low && products && d.rows * static_cast<int64_t>(d.out) >= AHEAD_ELEMENTS &&
            access_of(d.dy, d.dy_stride, d.out, d.rows) == 16 && access_of(d.z, d.z_stride, d.out, d.rows) == 16;
  if (p.ahead) {
    p.slab = LINEAR_PIECE_ROWS;
    p.slabs = parts_of(d.rows, p.slab);
    p.counter_bytes = (1 + p.slabs) * 4;
    p.counters = ws.take(p.counter_bytes);
    if (d.dbias) p.db_parts = ws.take((p.slabs + d.groups) * d.out * 4);
    p.end = ws.end;
    return p;
  }
  // slabs of rows: about four CTAs for an SM, 8 (a row for each warp) to 1024 rows
  const int64_t columns = parts_of(d.out, 256);
  int64_t slab = up(parts_of(d.rows * columns, 608), 8);
  slab = slab < 8 ? 8 : slab > 1024 ? 1024 : slab;
  if (parts_of(d.rows, slab) > 65535) slab = up(parts_of(d.rows, 65535), 32);
  p.slab = static_cast<int>(slab);
  p.slabs = parts_of(d.rows, slab);
  if (d.dbias) p.db_parts = ws.take((p.slabs + d.groups) * d.out * 4);
  p.end = ws.end;
  return p;
}

// ---------------------------------------------------------------- calls

struct Call {
  cudaStream_t stream;
  int type, sms, launches;
  int* status;
  uint8_t* ws;

  // The operand's copy in the workspace, where it needs one.
  int lay_out(Operand& o) {
    if (!o.copy) return MB_OK;
    o.base = ws + o.at;
    const LinearPackParams p{static_cast<const uint16_t*>(o.src), o.src_ld, reinterpret_cast<uint16_t*>(ws + o.at), o.ld,
                             o.rows, static_cast<int>(o.cols), access_of(o.src, o.src_ld, o.cols, o.rows) >= 4};
    const cudaError_t e = launch_linear_pack(p, sms, stream);
    if (e != cudaSuccess) return api_cuda_fail(e);
    ++launches;
    return MB_OK;
  }
  int map(CUtensorMap* m, const Operand& o, int64_t rows, int64_t batch, int box_rows) const {
    return api_encode_rows(m, o.base, type == MB_BF16, o.cols, rows, batch, o.ld, box_rows);
  }
  int result_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t batch, int64_t ld) const {
    return api_encode_rows(m, p, type == MB_BF16, cols, rows, batch, rows > 1 ? ld : up(cols, 8), 32);
  }
};

// Whether TMA can read chunks of a matrix: rows at 16-byte boundaries.  To write them, rows have to end at such boundaries
// too: past a row's end it leaves only whole 16-byte pieces alone.
bool bulk_loads(const void* p, int64_t ld, int64_t cols, int64_t rows) {
  return aligned(p, 16) && (rows <= 1 || (ld % 8 == 0 && ld >= cols));
}
bool bulk_stores(const void* p, int64_t ld, int64_t cols, int64_t rows) { return cols % 8 == 0 && bulk_loads(p, ld, cols, rows); }

void set_cut(LinearJob& j, const Cut& c, uint8_t* ws) {
  j.wide = c.wide;
  j.n_tiles = static_cast<int>(parts_of(j.N, c.wide));
  j.splits = c.splits;
  j.parts = c.splits > 1 ? reinterpret_cast<float*>(ws + c.at) : nullptr;
  j.part_tiles = c.tiles;
}

int run_products(const LinearParams& p, const Cut* const cuts[2], bool forward, Call& call) {
  int64_t units = 0;
  for (int j = 0; j < p.jobs; ++j) units += cuts[j]->tiles * cuts[j]->splits;
  // (a launch without tiles still has rows to clear and sums to finish)
  const int pairs = static_cast<int>(p.jobs == 0 ? MAX_PAIRS : units < 1 ? 1 : units < 4096 ? units : 4096);
  cudaError_t e = launch_linear(p, call.type, forward, pairs, call.stream);
  if (e != cudaSuccess) return api_cuda_fail(e);
  ++call.launches;
  for (int j = 0; j < p.jobs; ++j) {
    if (cuts[j]->splits == 1) continue;
    e = launch_linear_join(p, j, call.type, forward, cuts[j]->tiles, call.stream);
    if (e != cudaSuccess) return api_cuda_fail(e);
    ++call.launches;
  }
  return MB_OK;
}

int begin_call(Call& call, int type, void* workspace, size_t bytes, size_t need, void* cuda_stream) {
  if (need > 0) {
    if (!workspace || bytes < need) return MB_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MB_ERR_ALIGN;
  }
  call = Call{static_cast<cudaStream_t>(cuda_stream), type, 0, 0, nullptr, static_cast<uint8_t*>(workspace)};
  MB_TRY(api_device_sms(&call.sms));
  return api_device_status(&call.status);
}

int check_forward(const mb_linear_desc& d) {
  MB_TRY(check_shape(d.rows, d.in, d.out, d.groups, d.ends));
  MB_TRY(check_types(d.type, d.bias_type, d.activation));
  if (bad_stride(d.x_stride, d.rows, d.in, false) || bad_stride(d.y_stride, d.rows, d.out, true) ||
      (d.residual && bad_stride(d.residual_stride, d.rows, d.out, false)) ||
      (d.z && bad_stride(d.z_stride, d.rows, d.out, true)))
    return MB_ERR_SHAPE;
  const bool some = d.rows > 0;
  MB_TRY(check_two(d.x, some));
  MB_TRY(check_two(d.y, some));
  MB_TRY(check_two(d.weight, some));
  MB_TRY(check_two(d.residual, false));
  MB_TRY(check_two(d.z, false));
  if (d.bias && !aligned(d.bias, d.bias_type == MB_F32 ? 4 : 2)) return MB_ERR_ALIGN;
  return MB_OK;
}

int check_backward(const mb_linear_backward_desc& d) {
  MB_TRY(check_shape(d.rows, d.in, d.out, d.groups, d.ends));
  MB_TRY(check_types(d.type, d.bias_type, d.activation));
  const bool slope = d.activation != MB_ACT_NONE, some = d.rows > 0;
  if (bad_stride(d.dy_stride, d.rows, d.out, false) || (d.dweight && bad_stride(d.x_stride, d.rows, d.in, false)) ||
      (slope && bad_stride(d.z_stride, d.rows, d.out, false)) || (d.dx && bad_stride(d.dx_stride, d.rows, d.in, true)))
    return MB_ERR_SHAPE;
  MB_TRY(check_two(d.dy, some));
  MB_TRY(check_two(d.x, some && d.dweight));
  MB_TRY(check_two(d.weight, some && d.dx));
  MB_TRY(check_two(d.z, some && slope));
  MB_TRY(check_two(d.dx, false));
  MB_TRY(check_two(d.dweight, false));
  if (d.dbias && !aligned(d.dbias, d.bias_type == MB_F32 ? 4 : 2)) return MB_ERR_ALIGN;
  return MB_OK;
}

int few_access(const mb_linear_desc& d) {
  return std::min(access_of(d.x, d.x_stride, d.in, d.rows), access_of(d.weight, d.in, d.in, 2));
}

// A kernel of mb_linear_rows.cu as its time goes: columns and rows of a CTA, how deep its warps reach in one step; then in ns what
// a CTA costs an otherwise full GPU, the same per element of `in`, and a CTA that finds no rows; in us a step's wait and
// the begin; and the rate at which W comes, in TB/s.
struct RowsForm {
  int cols, rows, deep;
  double cta, per_in, idle, step, begin, rate;
};

// The time of a product by rows, in us: its CTAs' work or the chain of waits along the contraction, whichever is longer, and the
// lesser of the two as far as it shows.
double time_by_rows(const mb_linear_desc& d, bool wide) {
  const RowsForm some16{16, 16, 512, 3.3, 0.0039, 1.8, 0.51, 1.8, 7.4}, short32{16, 32, 256, 3.0, 0.008, 0.9, 0.59, 1.6, 5.5},
      long32{16, 32, 512, 14.0, 0.0077, 2.9, 0.58, 1.0, 3.9}, one{4, 1, 2048, 1.7, 0.0007, 1.0, 0.41, 1.3, 9.5},
      one_single{4, 1, 2048, 1.8, 0.0005, 1.0, 0.5, 1.4, 4.0}, few_single{4, 8, 2048, 13.0, 0.0062, 1.0, 4.1, 0.8, 20.0};
  const RowsForm& f = !wide ? (d.rows == 1 ? one_single : few_single)
                            : d.rows == 1 ? one : d.rows <= 16 ? some16 : d.in <= 1024 ? short32 : long32;
  const int64_t columns = parts_of(d.out, f.cols), slabs = parts_of(d.rows, f.rows);
  const int64_t some = std::min<int64_t>(d.groups, d.rows);      // groups that can have rows
  double ctas = columns * std::max(some, slabs) * (f.cta + f.per_in * d.in);
  if (d.groups > 1) ctas += columns * some * slabs * f.idle * (1 + d.groups / 64.0);     // (each looks the groups through)
  const double waits = f.step * parts_of(d.in, f.deep) + 2e-6 * d.in * d.out * some / f.rate;
  return f.begin + std::sqrt(1e-6 * ctas * ctas + waits * waits);
}

// And by tiles, from the same cut as the call's: a tile of a short contraction takes as long as its results take to leave.
double time_by_tiles(const mb_linear_desc& d, bool wide) {
  const Cut c = plan_forward(d).y;
  const int64_t some = std::min<int64_t>(d.groups, d.rows), tiles = std::max(some, parts_of(d.rows, LINEAR_TILE)) * parts_of(d.out, c.wide);
  const Cut held{c.wide, c.splits, tiles, c.blocks, c.n, 0};
  const double weights = 2e-6 * d.in * d.out * d.groups;         // MB
  double t = 2.3 + 0.33 * (parts_of(tiles * c.splits, MAX_PAIRS) * std::max(unit_time(c), 7.6 * c.wide / 256) + 8 + join_time(held)) +
             0.07 * weights * some / d.groups;
  if (!wide) t += 2.5 + 0.57 * (weights + 2e-6 * d.rows * d.in); // laid out at 16-byte boundaries first
  return t;
}

// Whether a few rows go by the kernels without tiles.  The two times above are fitted to 540 calls on one GB300 (in a graph, W from
// memory; 1 to 512 rows, in and out 8 to 65536, 1 to 256 groups): within about 15 % each, and the choice by them costs 1 %
// over the better side of each call.  Both sides of some, us, by rows and by tiles: one row 768->768 1.8 and 8.6, 4096->4096
// 7.9 and 22, 8->65536 28 and 15; 16 rows 4096->4096 10.0 and 20, 65536->64 99 and 28; 64 rows 768->768 3.5 and 8.5,
// 4096->1024 10.2 and 14.5, 64->32768 16 and 9.4, 65536->64 125 and 28; 256 rows 768->768 4.6 and 8.9, 64->8192 15 and 6.8; 512
// rows 64->64 2.0 and 5.3, 768->768 8.0 and 9.0, 64->2816 11 and 6.6, 64->8192 29 and 7.3, 8->65536 208 and 37, 4096->128
// 6.5 and 12.  Over groups: 64 rows of 8 256->1024 5.0 and 7.7, 1024->2816 24 and 19; of 64 1024->64 7.3 and 12, 1024->2816 170 and
// 67.  Off 16-byte boundaries elements come one by one: one row 4095->4095 10 and 33; eight 765->765 6.9 and 12, 33->65535
// 220 and 34.  No product by tiles takes less than 5.
bool by_rows(const mb_linear_desc& d) {
  const bool wide = few_access(d) == 16;
  if (d.rows > (!wide ? LINEAR_FEW_ROWS : d.groups > 1 ? LINEAR_SOME_GROUPED : LINEAR_SOME_ROWS)) return false;
  const double t = time_by_rows(d, wide);
  return t < 5 || t < time_by_tiles(d, wide);
}

int few_rows(const mb_linear_desc& d, cudaStream_t stream) {
  LinearFewParams p{d.x, d.x_stride, d.weight, d.bias, d.bias_type == MB_F32, d.activation, d.residual, d.residual_stride,
                    d.z, d.z_stride, d.y, d.y_stride, static_cast<int>(d.rows), d.in, d.out, d.groups, d.ends, 0, nullptr};
  int sms = 0;
  MB_TRY(api_device_sms(&sms));
  MB_TRY(api_device_status(&p.status));
  p.access = few_access(d);
  const cudaError_t e = launch_linear_few(p, d.type, stream);
  if (e != cudaSuccess) return api_cuda_fail(e);
  api_launched(MB_MARK_LINEAR, 1, stream);
  return MB_OK;
}

}  // namespace
}  // namespace mb

using namespace mb;

extern "C" {

int mb_linear_workspace_bytes(const mb_linear_desc* desc, size_t* out_bytes) {
  if (!desc || !out_bytes) return MB_ERR_NULL;
  MB_TRY(check_forward(*desc));
  *out_bytes = desc->rows == 0 || by_rows(*desc) ? 0 : plan_forward(*desc).end;
  return MB_OK;
}

int mb_linear(const mb_linear_desc* desc, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  if (!desc) return MB_ERR_NULL;
  const mb_linear_desc& d = *desc;
  MB_TRY(check_forward(d));
  if (d.rows == 0) return MB_OK;
  if (by_rows(d)) return few_rows(d, static_cast<cudaStream_t>(cuda_stream));
  ForwardPlan plan = plan_forward(d);
  Call call{};
  MB_TRY(begin_call(call, d.type, workspace, workspace_bytes, plan.end, cuda_stream));
  MB_TRY(call.lay_out(plan.x));
  MB_TRY(call.lay_out(plan.w));
  LinearParams p{};
  p.jobs = 1;
  p.rows = static_cast<int>(d.rows);
  p.groups = d.groups;
  p.ends = d.ends;
  p.status = call.status;
  p.status_from = 1;
  p.bias = d.bias;
  p.bias_f32 = d.bias_type == MB_F32;
  p.act = d.activation;
  p.residual = d.residual;
  p.residual_ld = d.residual_stride;
  p.residual_access = access_of(d.residual, d.residual_stride, d.out, d.rows);
  p.z = d.z;
  p.z_ld = d.z_stride;
  p.z_access = access_of(d.z, d.z_stride, d.out, d.rows);
  LinearJob& j = p.job[0];
  j.passes = 1;
  j.N = d.out;
  j.K = d.in;
  j.out = d.y;
  j.ld = d.y_stride;
  j.access = access_of(d.y, d.y_stride, d.out, d.rows);
  set_cut(j, plan.y, call.ws);
  MB_TRY(call.map(&j.a, plan.x, d.rows, 1, 128));
  MB_TRY(call.map(&j.b, plan.w, d.out, d.groups, j.wide / 2));
  j.bulk = j.splits == 1 && bulk_stores(d.y, d.y_stride, d.out, d.rows) &&
           (!d.z || bulk_stores(d.z, d.z_stride, d.out, d.rows));
  if (j.bulk) {
    MB_TRY(call.result_map(&j.d, d.y, d.rows, d.out, 1, d.y_stride));
    if (d.z) MB_TRY(call.result_map(&p.z_map, d.z, d.rows, d.out, 1, d.z_stride));
  }
  p.residual_bulk = d.residual && j.splits == 1 && bulk_loads(d.residual, d.residual_stride, d.out, d.rows);
  if (p.residual_bulk) MB_TRY(call.result_map(&p.residual_map, d.residual, d.rows, d.out, 1, d.residual_stride));
  const Cut* const cuts[2] = {&plan.y, nullptr};
  MB_TRY(run_products(p, cuts, true, call));
  api_launched(MB_MARK_LINEAR, call.launches, call.stream);
  return MB_OK;
}

int mb_linear_backward_workspace_bytes(const mb_linear_backward_desc* desc, size_t* out_bytes) {
  if (!desc || !out_bytes) return MB_ERR_NULL;
  MB_TRY(check_backward(*desc));
  *out_bytes = desc->rows == 0 ? 0 : plan_backward(*desc).end;
  return MB_OK;
}

int mb_linear_backward(const mb_linear_backward_desc* desc, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  if (!desc) return MB_ERR_NULL;
  const mb_linear_backward_desc& d = *desc;
  MB_TRY(check_backward(d));
  if (!d.dx && !d.dweight && !d.dbias) return MB_OK;
  Call call{};
  if (d.rows == 0) {                             // sums over nothing
    MB_TRY(begin_call(call, d.type, workspace, workspace_bytes, 0, cuda_stream));
    const size_t n = static_cast<size_t>(d.groups) * d.out;
    cudaError_t e = cudaSuccess;
    if (d.dweight) e = cudaMemsetAsync(d.dweight, 0, n * d.in * 2, call.stream);
    if (e == cudaSuccess && d.dbias) e = cudaMemsetAsync(d.dbias, 0, n * (d.bias_type == MB_F32 ? 4 : 2), call.stream);
    return e == cudaSuccess ? MB_OK : api_cuda_fail(e);
  }
  BackwardPlan plan = plan_backward(d);
  MB_TRY(begin_call(call, d.type, workspace, workspace_bytes, plan.end, cuda_stream));
  if (plan.slope) plan.dz.base = call.ws + plan.dz.at;
  else if (d.dx || d.dweight) MB_TRY(call.lay_out(plan.dz));
  if (d.dweight) MB_TRY(call.lay_out(plan.x));
  if (d.dx) MB_TRY(call.lay_out(plan.w));
  LinearParams p{};
  if (plan.slope || d.dbias) {
    LinearSlopeParams s{};
    s.dy = d.dy;
    s.dy_ld = d.dy_stride;
    s.z = plan.slope ? d.z : nullptr;
    s.z_ld = d.z_stride;
    s.dz = plan.slope ? call.ws + plan.dz.at : nullptr;
    s.dz_ld = plan.dz.ld;
    s.low = plan.low;
    s.act = d.activation;
    s.rows = static_cast<int>(d.rows);
    s.cols = d.out;
    s.groups = d.groups;
    s.ends = d.ends;
    s.parts = d.dbias ? reinterpret_cast<float*>(call.ws + plan.db_parts) : nullptr;
    s.slab = plan.slab;
    s.access = access_of(d.dy, d.dy_stride, d.out, d.rows);
    if (plan.slope && access_of(d.z, d.z_stride, d.out, d.rows) < s.access) s.access = access_of(d.z, d.z_stride, d.out, d.rows);
    if (plan.ahead) {
      LinearAhead& a = p.ahead;
      a.slope = s;
      a.next = reinterpret_cast<unsigned*>(call.ws + plan.counters);
      a.done = a.next + 1;
      a.slabs = static_cast<int>(plan.slabs);
      a.column_groups = static_cast<int>(parts_of(d.out, 256));
      // the units of dW go through their parts of the rows side by side
      a.ways = d.dweight && d.groups == 1 ? plan.dw.splits : 1;
      a.per_way = static_cast<int>(parts_of(plan.slabs, a.ways));
      const cudaError_t e = cudaMemsetAsync(a.next, 0, plan.counter_bytes, call.stream);
      if (e != cudaSuccess) return api_cuda_fail(e);
    } else {
      const cudaError_t e = launch_linear_slope(s, d.type, call.stream);
      if (e != cudaSuccess) return api_cuda_fail(e);
      ++call.launches;
    }
  }
  p.rows = static_cast<int>(d.rows);
  p.groups = d.groups;
  p.ends = d.ends;
  p.status = call.status;
  p.status_from = 1;
  p.db = plan.ahead ? nullptr : d.dbias;
  p.db_parts = reinterpret_cast<const float*>(call.ws + plan.db_parts);
  p.db_f32 = d.bias_type == MB_F32;
  p.db_cols = d.out;
  p.slab = plan.slab;
  const Cut* cuts[2] = {nullptr, nullptr};
  if (d.dweight) {                               // the longer units first
    LinearJob& j = p.job[p.jobs];
    cuts[p.jobs++] = &plan.dw;
    j.over_rows = j.a_mn = j.b_mn = 1;
    j.passes = plan.low ? 2 : 1;
    j.pass_cols = plan.low;
    j.M = d.out;
    j.m_tiles = static_cast<int>(parts_of(d.out, LINEAR_TILE));
    j.N = d.in;
    j.out = d.dweight;
    j.ld = d.in;
    j.group_stride = static_cast<int64_t>(d.out) * d.in;
    j.access = access_of(d.dweight, d.in, d.in, 2);
    set_cut(j, plan.dw, call.ws);
    MB_TRY(call.map(&j.a, plan.dz, d.rows, 1, 64));
    MB_TRY(call.map(&j.b, plan.x, d.rows, 1, 64));
    j.bulk = j.splits == 1 && bulk_stores(d.dweight, d.in, d.in, 2);
    if (j.bulk) MB_TRY(call.result_map(&j.d, d.dweight, d.out, d.in, d.groups, d.in));
  }
  if (d.dx) {
    LinearJob& j = p.job[p.jobs];
    cuts[p.jobs++] = &plan.dx;
    j.b_mn = 1;
    j.passes = plan.low ? 2 : 1;
    j.pass_cols = plan.low;
    j.N = d.in;
    j.K = d.out;
    j.out = d.dx;
    j.ld = d.dx_stride;
    j.access = access_of(d.dx, d.dx_stride, d.in, d.rows);
    set_cut(j, plan.dx, call.ws);
    MB_TRY(call.map(&j.a, plan.dz, d.rows, 1, 128));
    MB_TRY(call.map(&j.b, plan.w, d.out, d.groups, 64));
    j.bulk = j.splits == 1 && bulk_stores(d.dx, d.dx_stride, d.in, d.rows);
    if (j.bulk) MB_TRY(call.result_map(&j.d, d.dx, d.rows, d.in, 1, d.dx_stride));
  }
  if (p.jobs == 2) p.extra = extra_units(plan.dw, plan.dx);
  MB_TRY(run_products(p, cuts, false, call));
  if (plan.ahead && d.dbias) {
    const LinearBiasParams b{reinterpret_cast<const float*>(call.ws + plan.db_parts), d.dbias, d.bias_type == MB_F32, d.out,
                             plan.slab, static_cast<int>(d.rows), d.groups, d.ends};
    const cudaError_t e = launch_linear_bias(b, d.type, call.stream);
    if (e != cudaSuccess) return api_cuda_fail(e);
    ++call.launches;
  }
  api_launched(MB_MARK_LINEAR_BACKWARD, call.launches, call.stream);
  return MB_OK;
}

}  // extern "C"
