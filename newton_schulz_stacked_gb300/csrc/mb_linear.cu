// The products of mb_linear on the sm_103a tensor cores: y = act(x W^T + b) + residual over groups of rows, and the two
// products of its gradient, dx = dz W and dW = dz^T x, in one launch.
//
// Pairs of CTAs compute tiles of 256 rows x 256 (or 128) columns with M = 256 tcgen05 MMAs (cta_group::2): CTA r of a
// pair holds rows 128 r .. of the A operand and half of the B operand's, staged by TMA with 128-byte swizzle in 64-deep
// blocks, and receives its 128 rows x all columns of the fp32 sums in TMEM (two accumulators, so that one tile's epilogue
// runs under the next one's MMAs).  Where dz comes in two halves (LOW) each has an accumulator of its own, and the epilogue adds
// them.  An operand whose contraction runs along memory is staged K-major, one box a block;
// the others (W in dx, both in dW) as boxes of 64 x 64 in MN-major layout.
//
// The units are dealt to the pairs in turn (Deal); the roles find them themselves from the groups' first rows and tiles, which
// each CTA works out in shared memory from the ends in device memory, so that the host need not know them.  Tiles never
// cross groups; a tile's operand rows past its group belong to the next group and are computed but not stored.  In dW
// the contraction runs over the group's rows and its last block may reach into the next group's: there the loads complete on
// a barrier of their own CTA, a warp clears the rows past the group's end in both operands (zero times the next group's
// infinity would not be zero), and the MMAs wait for both CTAs' warps.  Rows past the tensor, and columns past its
// width, are read as zeros by TMA.
//
// Roles (12 warps, both CTAs):
//   warps 0 and 11  TMA producers of the A and the B operand, a ring of STAGES blocks; the bytes of both CTAs complete
//                   on the even CTA's barrier
//   warp 1          TMEM; in the even CTA it issues the MMAs and releases stages in both CTAs
//   warps 2..9      epilogue of the CTA's 128 rows, two warps per 32 TMEM lanes, chunks of 32 x 64 through shared memory to
//                   TMA or row-wise stores; before its first tile each takes a share of what else the call leaves to do: zeros in
//                   rows of no group, dbias from the slabs' sums
//   warp 10         clears the blocks that reach past a group
// Where dz has to be formed first (dy act'(z), a pass over memory as long as half the products), the epilogue warps of the
// backward pass do it in pieces while the MMAs run, in the order in which the products need the rows; the A operand's
// producers wait for the slabs of rows that they load.  Pieces are claimed from a counter, so that a CTA that is not
// resident yet holds none.
// Producers and issuer run as whole warps, the same in all lanes, and elect a lane for each TMA copy, MMA or commit: those take
// their operands from uniform registers, and values that one lane alone has worked out are moved there one by one.
// Every bounded wait of a warp is decided by all of its lanes: each looks at a clock of its own, and a lane that gave up alone
// would leave the others at the warp's next barrier.
//
// A long contraction over few tiles is cut into parts whose fp32 sums go to the workspace, and linear_join_kernel adds them.
//
// What bounds it: a block of 256 x 256 x 64 takes 551 cycles where its MMAs need 512 (8192^3 600 us, 1.83 PFLOP/s).  Short
// contractions with results of their width are bound by what an SM moves to and from the L2 (65536x768->2816, relu^2 with z
// and a bias: 235 us, tensor pipe 0.5 busy), calls below about 20 us by their launch and the first tile's way.
#include <atomic>
#include <climits>
#include <type_traits>

#include "mb_block.h"
#include "mb_linear.cuh"

namespace mb {
namespace {

constexpr int BM = 128;
constexpr int STAGES = 6;
constexpr int TILE_BYTES = BM * LINEAR_DEEP * 2;     // 16 KB: a CTA's rows of one operand's block
constexpr int BOX_BYTES = 64 * LINEAR_DEEP * 2;      // 8 KB: one 64 x 64 box
constexpr int EPI_WARPS = 8;
constexpr int A_WARP = 0, FIX_WARP = 2 + EPI_WARPS, B_WARP = FIX_WARP + 1;
constexpr int THREADS = 32 * (B_WARP + 1);
// What not every call needs takes the memory of the ring's last stages: the residual's buffers a whole one, the places of more
// than FEW_GROUPS groups the A half of one.
constexpr int FEW_GROUPS = 140;
static_assert(EPI_WARPS * CHUNK_BYTES <= 2 * TILE_BYTES, "the residual's buffers fit a stage");
constexpr int SMEM = 2 * STAGES * TILE_BYTES + EPI_WARPS * CHUNK_BYTES + 2 * (FEW_GROUPS + 1) * 4 + 1024 /* alignment */ +
                     448 /* barriers, notes */;
static_assert(SMEM <= 232448, "shared memory per CTA");
static_assert(GROUPS_BYTES <= TILE_BYTES, "the groups' places fit a stage's");
constexpr uint32_t ACC_COLS = 256, TMEM_COLS = 512;

// Instruction descriptor, kind::f16, fp32 sums, M = 256 (a pair).
template <typename T>
__device__ __forceinline__ uint32_t instruction(int n, int a_mn, int b_mn) {
  const uint32_t kind = std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u;
  return (1u << 4) | kind | static_cast<uint32_t>(a_mn) << 15 | static_cast<uint32_t>(b_mn) << 16 |
         static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(256 >> 4) << 24;
}

// 32 lanes x 32 columns of sums: the load, and the wait that its registers are ready after.
__device__ __forceinline__ void tmem_ld_32x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_ready(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ int same(int v) { return __shfl_sync(0xffffffffu, v, 0); }
// A unit as the producers and the MMA issuer take it: the same in all lanes, and known to be (shuffled from one).
__device__ __forceinline__ void decode_same(const LinearParams& P, const Groups& G, int first_units, int at, Unit& u) {
  decode_unit(P, G, first_units, at, u);
  u.job = same(u.job);
  u.group = same(u.group);
  u.m0 = same(u.m0);
  u.n0 = same(u.n0);
  u.wide = same(u.wide);
  u.k_begin = same(u.k_begin);
  u.k_end = same(u.k_end);
  u.kb0 = same(u.kb0);
  u.kb1 = same(u.kb1);
}

// How long a unit's sums may take: a block 0.3 us, and where 2^28 rows are one group's its 2^22 blocks 1.15 s.
constexpr uint64_t BLOCK_LIMIT_NS = 4000;
__device__ __forceinline__ uint64_t unit_limit_ns(const Unit& u) {
  return WAIT_LIMIT_NS + static_cast<uint64_t>(u.kb1 - u.kb0) * BLOCK_LIMIT_NS;
}

// What the MMA issuer has to know of a block, written by the A operand's producer of the even CTA: it need not decode units
// itself, which took it longer (750 cycles) than a block's MMAs.
struct BlockNote {
  uint32_t idesc, flags;
};
enum : uint32_t {
  NOTE_FIRST = 1,          // of its unit: the accumulator starts anew
  NOTE_LAST = 2,
  NOTE_NOTHING = 4,        // a unit without blocks, one of zeros in their place: no MMAs
  NOTE_PAST = 8,           // reaches past its group: wait until it is cleared
  NOTE_A_MN = 16,
  NOTE_B_MN = 32,
  NOTE_SECOND = 64         // the second pass begins: other sums, anew
};

// The block of a pass that reaches into the next group's rows (the last, or none: INT_MAX).
__device__ __forceinline__ int past_from(const LinearParams& P, const LinearJob& J, const Unit& u) {
  const int whole = (u.k_end - u.k_begin) / LINEAR_DEEP;
  return J.over_rows && u.k_end < P.rows && whole * LINEAR_DEEP < u.k_end - u.k_begin ? whole : INT_MAX;
}

// How a CTA loads one operand of a unit, block after block: held in registers, since a loop that reads the parameters again
// for each block (as the compiler does behind a barrier's memory clobber) costs the producer more than the MMAs take.
struct Feed {
  const CUtensorMap* map;
  int x, y, x_step, y_step, batch, boxes;   // x, y: of a pass's first block
  int pass_cols;           // from one pass to the next
  uint32_t bytes;          // of both operands
  int past_from;
};
__device__ __forceinline__ Feed feed_of(const LinearParams& P, const Unit& u, bool for_a, uint32_t rank) {
  const LinearJob& J = P.job[u.job];
  Feed f;
  f.map = for_a ? &J.a : &J.b;
  const int mn = for_a ? u.m0 + static_cast<int>(rank) * BM : u.n0 + static_cast<int>(rank) * (u.wide >> 1);
  const int k = u.k_begin;
  const bool turned = for_a ? J.a_mn : J.b_mn;
  f.x = turned ? mn : k;
  f.y = turned ? k : mn;
  f.x_step = turned ? 0 : LINEAR_DEEP;
  f.y_step = turned ? LINEAR_DEEP : 0;
  f.pass_cols = for_a ? J.pass_cols : 0;
  f.batch = for_a || J.over_rows ? 0 : u.group;
  f.boxes = !turned ? 1 : for_a ? 2 : u.wide >> 7;
  f.bytes = TILE_BYTES + (J.b_mn ? (u.wide >> 7) * BOX_BYTES : (J.wide >> 1) * LINEAR_DEEP * 2);
  f.past_from = past_from(P, J, u);
  return f;
}

__device__ __forceinline__ int claim_piece(unsigned* next, int lane) {
  unsigned p = 0;
  if (lane == 0) p = atomicAdd(next, 1u);
  return static_cast<int>(__shfl_sync(0xffffffffu, p, 0));
}

// A share of the work beside the tiles, by the epilogue's warps: warp `me` of `all`.
template <typename T>
__device__ void side_work(const LinearParams& P, const Groups& G, long long me, long long all, int lane) {
  if (P.ends && P.jobs > 0 && !P.job[P.jobs - 1].over_rows) {
    // zeros in the rows of no group
    const LinearJob& J = P.job[P.jobs - 1];
    for (long long row = G.row[G.n] + me; row < P.rows; row += all) {
      for (int which = 0; which < 2; ++which) {
        uint16_t* out = static_cast<uint16_t*>(which ? P.z : J.out);
        if (!out) continue;
        out += row * (which ? P.z_ld : J.ld);
        if ((which ? P.z_access : J.access) == 16)
          for (int c = lane; c < J.N / 8; c += 32) reinterpret_cast<uint4*>(out)[c] = make_uint4(0, 0, 0, 0);
        else
          for (int c = lane; c < J.N; c += 32) out[c] = 0;
      }
    }
  }
  if (P.db) {
    // dbias of 8 columns of one group: its sums over the slabs that hold its rows, every fourth to a lane of each column (with 32
    // columns to a warp the chain of loads took 8 us for 98 slabs)
    const int across = (P.db_cols + 7) / 8;
    for (long long i = me; i < static_cast<long long>(G.n) * across; i += all) {
      const int g = static_cast<int>(i / across), col = static_cast<int>(i % across) * 8 + (lane & 7);
      float sum = 0.f;
      const int begin = G.row[g], end = G.row[g + 1];
      if (end > begin && col < P.db_cols) {
        const int last = (end - 1) / P.slab;
#pragma unroll 8
        for (int s = begin / P.slab + (lane >> 3); s <= last; s += 4) sum += P.db_parts[static_cast<long long>(s + g) * P.db_cols + col];
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (lane >= 8 || col >= P.db_cols) continue;
      const long long at = static_cast<long long>(g) * P.db_cols + col;
      if (P.db_f32) static_cast<float*>(P.db)[at] = sum;
      else static_cast<T*>(P.db)[at] = from_float<T>(sum);
    }
  }
}

template <bool FORWARD, typename T, bool LOW>
__global__ void __launch_bounds__(THREADS, 1) linear_kernel(const __grid_constant__ LinearParams P) {
  constexpr int PASSES = LOW ? 2 : 1;
  constexpr int TURNS = LOW ? 1 : 2;           // tiles whose sums TMEM holds
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * TILE_BYTES;
  uint8_t* sChunk = sB + STAGES * TILE_BYTES;
  const bool few = P.groups <= FEW_GROUPS;
  const bool with_residual = FORWARD && P.residual_bulk;
  const uint32_t stages = STAGES - (few ? 0 : 1) - (with_residual ? 1 : 0);
  uint64_t* full = reinterpret_cast<uint64_t*>(sChunk + EPI_WARPS * CHUNK_BYTES);   // [STAGES] (even) both CTAs' operands landed
  uint64_t* empty = full + STAGES;           // [STAGES] the pair's MMAs are done with the stage
  uint64_t* past_bar = empty + STAGES;       // [STAGES] this CTA's part of a block that reaches past its group landed
  uint64_t* cleared = past_bar + STAGES;         // [STAGES] (even) both CTAs have cleared it
  uint64_t* tfull = cleared + STAGES;        // [2] accumulator ready for the epilogue
  uint64_t* tempty = tfull + 2;              // [2] (even) both CTAs' epilogues drained the accumulator
  uint64_t* landed = tempty + 2;             // [EPI_WARPS] the warp's chunk of the residual
  BlockNote* notes = reinterpret_cast<BlockNote*>(landed + EPI_WARPS);      // [STAGES]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(notes + STAGES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Groups G;
  G.row = few ? reinterpret_cast<int*>(tmem_slot + 4) : reinterpret_cast<int*>(sA + stages * TILE_BYTES);
  G.tile = G.row + P.groups + 1;
  G.n = P.groups;

  const int warp = same(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool even = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&past_bar[s], 1);
      mbar_init(&cleared[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * EPI_WARPS);
    }
    for (int i = 0; i < EPI_WARPS; ++i) mbar_init(&landed[i], 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  begin_after_previous();
  if (warp == FIX_WARP && fill_groups(G, P.ends, P.rows, lane) && blockIdx.x == 0 && P.status_from && lane == 0)
    latch_status(P.status, DEV_BAD_SCALAR);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();      // both CTAs' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&]() {
    latch_status(P.status, DEV_TIMEOUT);
    *abort_flag = 1;
  };
  // The pair's MMAs write the odd CTA's accumulators at the even CTA's TMEM address.
  if (threadIdx.x == 0 && ld_cluster_u32(map_to_rank(tmem_slot, rank ^ 1u)) != tmem) {
    latch_status(P.status, DEV_PAIR_TMEM);
    *abort_flag = 1;
  }

  const int first_units = P.jobs > 0 ? job_units(P.job[0], G) : 0;
  const Deal deal(blockIdx.x >> 1, gridDim.x >> 1, first_units,
                  first_units + (P.jobs > 1 ? job_units(P.job[1], G) : 0), P.extra);
  const int mine = deal.count();

  if (warp == A_WARP || warp == B_WARP) {
    // ---------------- TMA producer of one operand (both CTAs); the A operand's also announces the bytes of both
    const bool for_a = warp == A_WARP;
    const uint32_t full_even = map_to_rank(&full[0], 0), past_own = map_to_rank(&past_bar[0], rank);
    uint8_t* const ring = for_a ? sA : sB;
    uint32_t st = 0, ph = 0, it = 0;
    bool ok = true;
    Seen seen;
    for (int i = 0; i < mine && ok && !__any_sync(0xffffffffu, *abort_flag); ++i) {
      Unit u;
      decode_same(P, G, first_units, deal(i), u);
      const Feed f = feed_of(P, u, for_a, rank);
      const LinearJob& J = P.job[u.job];
      const uint32_t idesc = instruction<T>(u.wide, J.a_mn, J.b_mn);
      const uint32_t flags = (J.a_mn ? NOTE_A_MN : 0u) | (J.b_mn ? NOTE_B_MN : 0u) | (u.kb0 < u.kb1 ? 0u : NOTE_NOTHING);
      // (a unit without blocks has one for its note)
      const int blocks = max((u.kb1 - u.kb0) * PASSES, 1);
      const bool await = !FORWARD && !LOW && for_a && P.ahead.next && !(flags & NOTE_NOTHING);   // dz is still being made
      if (await && !J.over_rows) {
        const int row = u.m0 + static_cast<int>(rank) * BM;
        ok = seen.rows(P.ahead, row, min(row + BM, u.m_end), lane, abort_flag);
        if (!ok) break;
      }
      int at_block = u.kb0;                        // of its pass
      int x = f.x + at_block * f.x_step, y = f.y + at_block * f.y_step;
      // A unit without blocks (of dW) loads one from behind the rows, zeros that cost no traffic: each block has all four
      // producers' copies in it, so that the stages' phases cannot pass one of them that is late by two turns of the ring.
      if (flags & NOTE_NOTHING) y = P.rows;
      for (int left = blocks; left > 0; --left, ++it) {
        if (it >= stages) {
          ok = __all_sync(0xffffffffu, mbar_wait_cluster_or_abort(&empty[st], ph ^ 1u, abort_flag));
          if (!ok) break;
        }
        if (await && J.over_rows) {
          ok = seen.rows(P.ahead, y, min(y + LINEAR_DEEP, u.k_end), lane, abort_flag);
          if (!ok) break;
        }
        const bool past_end = !(flags & NOTE_NOTHING) && at_block >= f.past_from;
        const uint32_t bar = (past_end ? past_own : full_even) + 8u * st;
        uint8_t* to = ring + st * TILE_BYTES;
        if (elect_lane()) {
          if (for_a) {
            if (even) {
              notes[st] = BlockNote{idesc, flags | (left == blocks ? NOTE_FIRST : LOW && at_block == u.kb0 ? NOTE_SECOND : 0u) |
                                               (left == 1 ? NOTE_LAST : 0u) | (past_end ? NOTE_PAST : 0u)};
              if (past_end) mbar_arrive(&full[st]);
              else mbar_expect_tx(&full[st], 2u * f.bytes);
            }
            if (past_end) mbar_expect_tx(&past_bar[st], f.bytes);
          }
          tma_load_3d_pair(to, f.map, bar, x, y, f.batch);
          if (f.boxes > 1) tma_load_3d_pair(to + BOX_BYTES, f.map, bar, x + 64, y, f.batch);
        }
        __syncwarp();
        x += f.x_step;
        y += f.y_step;
        ++at_block;
        if (LOW && at_block == u.kb1) {            // the next pass
          at_block = u.kb0;
          x = f.x + at_block * f.x_step + f.pass_cols;
          y = f.y + at_block * f.y_step;
        }
        if (++st == stages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok) fail();
    // this CTA stays until the multicast releases of every stage it filled have arrived
    for (uint32_t i = it > stages ? it - stages : 0u; i < it; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait_cluster_or_abort(&empty[i % stages], (i / stages) & 1, abort_flag))) {
        fail();
        break;
      }
    }
  } else if (warp == 1) {
    if (even) {
      // ---------------- MMA issuer of the pair: block after block as the notes say
      const uint64_t desc = smem_desc_sw128(0, 0, 1024);             // but for the address and the step between boxes
      const uint32_t a_ring = smem_u32(sA) >> 4, b_ring = smem_u32(sB) >> 4;
      uint32_t past_phase = 0, st = 0, ph = 0, dacc = tmem, idesc = 0, a_step = 0, b_step = 0;
      uint64_t a_desc = desc, b_desc = desc;
      int k = 0;
      bool ok = true;
      while (k < mine) {
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&full[st], ph, abort_flag));
        if (!ok) break;
        const uint32_t flags = same(notes[st].flags);
        if (flags & NOTE_FIRST) {
          idesc = same(notes[st].idesc);
          a_step = (flags & NOTE_A_MN ? 2048u : 32u) >> 4;
          b_step = (flags & NOTE_B_MN ? 2048u : 32u) >> 4;
          a_desc = desc | static_cast<uint64_t>((flags & NOTE_A_MN ? BOX_BYTES : 16) >> 4) << 16;
          b_desc = desc | static_cast<uint64_t>((flags & NOTE_B_MN ? BOX_BYTES : 16) >> 4) << 16;
          dacc = tmem + k % TURNS * ACC_COLS;
          if (k >= TURNS) {
            ok = __all_sync(0xffffffffu, mbar_wait_cluster_or_abort(&tempty[k % TURNS], (k / TURNS - 1) & 1, abort_flag));
            if (!ok) break;
          }
        } else if (LOW && (flags & NOTE_SECOND)) {
          dacc += ACC_COLS;
        }
        if (flags & NOTE_PAST) {
          ok = __all_sync(0xffffffffu, mbar_wait_cluster_or_abort(&cleared[st], (past_phase >> st) & 1u, abort_flag));
          if (!ok) break;
          past_phase ^= 1u << st;
        }
        tc_fence_after();
        const uint64_t a0 = a_desc + (a_ring + st * (TILE_BYTES >> 4)), b0 = b_desc + (b_ring + st * (TILE_BYTES >> 4));
        if (elect_lane()) {
          if (!(flags & NOTE_NOTHING)) {
#pragma unroll
            for (int kk = 0; kk < LINEAR_DEEP / 16; ++kk)
              umma_bf16_pair(dacc, a0 + kk * a_step, b0 + kk * b_step, idesc,
                             (flags & (LOW ? NOTE_FIRST | NOTE_SECOND : NOTE_FIRST)) && kk == 0 ? 0u : 1u);
          }
          umma_commit_pair_both(&empty[st]);   // the stage may be refilled in both CTAs
          if (flags & NOTE_LAST) umma_commit_pair_both(&tfull[k % TURNS]);
        }
        __syncwarp();
        if (flags & NOTE_LAST) ++k;
        if (++st == stages) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (!ok) fail();
    }
    __syncwarp();
  } else if (warp == FIX_WARP) {
    // ---------------- blocks that reach past a group: their rows from the group's end on become zero
    uint32_t it = 0, past_phase = 0;
    const uint32_t cleared_even = map_to_rank(&cleared[0], 0);
    for (int i = 0; i < mine && !__any_sync(0xffffffffu, *abort_flag); ++i) {
      Unit u;
      decode_unit(P, G, first_units, deal(i), u);
      const LinearJob& J = P.job[u.job];
      const int part = u.kb1 - u.kb0, blocks = max(part * PASSES, 1);     // (without blocks: a stage for the note)
      const int past = past_from(P, J, u);
      bool ok = true;
      for (int pass = 0; pass < PASSES && past >= u.kb0 && past < u.kb1; ++pass) {
        const int st = (it + pass * part + past - u.kb0) % stages;
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&past_bar[st], (past_phase >> st) & 1u, abort_flag, unit_limit_ns(u)));
        if (!ok) break;
        past_phase ^= 1u << st;
        // a box's rows of 128 bytes are its rows of the contraction (the swizzle stays within a row)
        const int keep = u.k_end - u.k_begin - past * LINEAR_DEEP;
        for (int box = 0; box < 2 + (u.wide >> 7); ++box) {
          uint8_t* base = box < 2 ? sA + st * TILE_BYTES + box * BOX_BYTES : sB + st * TILE_BYTES + (box - 2) * BOX_BYTES;
          for (int j = keep * 8 + lane; j < LINEAR_DEEP * 8; j += 32) reinterpret_cast<uint4*>(base)[j] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cleared_even + 8u * static_cast<uint32_t>(st));
      }
      if (!ok) {
        fail();
        break;
      }
      it += blocks;
    }
    __syncwarp();
  } else {
    // ---------------- epilogue
    const int ew = warp - 2, quad = warp & 3, half = ew >> 2;
    WarpPlace w;
    w.lane = lane;
    w.buf = sChunk + ew * CHUNK_BYTES;
    // (the last stage's two halves, four warps' buffers in each)
    ResidualFeed res{with_residual ? (half ? sB : sA) + (STAGES - 1) * TILE_BYTES + (ew & 3) * CHUNK_BYTES : nullptr, &landed[ew], 0, 0};
    const uint32_t tempty_even = map_to_rank(&tempty[0], 0);
    side_work<T>(P, G, static_cast<long long>(blockIdx.x) * EPI_WARPS + ew, static_cast<long long>(gridDim.x) * EPI_WARPS, lane);
    // the piece of dz that this warp has claimed (none from `pieces` on)
    const int pieces = !FORWARD && !LOW && P.ahead.next ? P.ahead.ways * P.ahead.per_way * P.ahead.column_groups : 0;
    int piece = pieces > 0 ? claim_piece(P.ahead.next, lane) : 0;
    for (int k = 0; k < mine || piece < pieces; ++k) {
      // pieces while no sums are ready, each claimed under the work on the one before
      while (piece < pieces &&
             !(k < mine && __all_sync(0xffffffffu, mbar_test(&tfull[k % TURNS], (k / TURNS) & 1))) &&
             !__any_sync(0xffffffffu, *abort_flag)) {
        const int now = piece;
        piece = claim_piece(P.ahead.next, lane);
        do_piece<T>(P.ahead, G, now, lane);
      }
      if (k >= mine) break;
      Unit u;
      decode_unit(P, G, first_units, deal(k), u);
      const LinearJob& J = P.job[u.job];
      const int buf = k % TURNS;
      w.row0 = u.m0 + static_cast<int>(rank) * BM + quad * 32;
      w.rows = min(32, u.m_end - w.row0);
      float2 bias[2] = {};
      if constexpr (FORWARD) {
        res.ask(P, J, w, u.n0 + CHUNK_COLS * half);
        bias[0] = bias_of<T>(P, J, u.group, u.n0 + CHUNK_COLS * half, lane);
        bias[1] = bias_of<T>(P, J, u.group, u.n0 + CHUNK_COLS * (half + 2), lane);
      }
      if (!__all_sync(0xffffffffu, mbar_wait_or_abort(&tfull[buf], (k / TURNS) & 1, abort_flag, unit_limit_ns(u)))) {
        fail();
        break;
      }
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      tc_fence_after();
      const uint32_t tacc = tmem + buf * ACC_COLS + (static_cast<uint32_t>(quad * 32) << 16);
      const int chunks = u.wide / CHUNK_COLS;
      bool ok = true;
      for (int c = half; c < chunks && ok; c += 2) {
        uint32_t r[2][32];
        __syncwarp();
        tmem_ld_32x32(tacc + CHUNK_COLS * c, r[0]);
        tmem_ld_32x32(tacc + CHUNK_COLS * c + 32, r[1]);
        tmem_ld_ready(r[0]);
        tmem_ld_ready(r[1]);
        Row v;
#pragma unroll
        for (int i = 0; i < CHUNK_COLS / 2; ++i)
          v.v[i] = make_float2(__uint_as_float(r[i / 16][2 * i % 32]), __uint_as_float(r[i / 16][2 * i % 32 + 1]));
        if (u.kb0 == u.kb1) {                                // without blocks the accumulator holds another tile
#pragma unroll
          for (int i = 0; i < CHUNK_COLS / 2; ++i) v.v[i] = make_float2(0.f, 0.f);
        } else if (LOW) {
          // what dz's rounding left, but where the sums without it are no numbers: zero times infinity is none
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __syncwarp();
            tmem_ld_32x32(tacc + ACC_COLS + CHUNK_COLS * c + 32 * h, r[0]);
            tmem_ld_ready(r[0]);
#pragma unroll
            for (int i = 0; i < CHUNK_COLS / 4; ++i) {
              float2& s = v.v[CHUNK_COLS / 4 * h + i];
              s.x = isfinite(s.x) ? s.x + __uint_as_float(r[0][2 * i]) : s.x;
              s.y = isfinite(s.y) ? s.y + __uint_as_float(r[0][2 * i + 1]) : s.y;
            }
          }
        }
        if (J.splits > 1) {
          float4* part = part_of(J, u, u.split, rank, ew, c >> 1);
#pragma unroll
          for (int i = 0; i < CHUNK_COLS / 4; ++i)
            part[32 * i + lane] = make_float4(v.v[2 * i].x, v.v[2 * i].y, v.v[2 * i + 1].x, v.v[2 * i + 1].y);
        } else {
          ok = finish_chunk<FORWARD, T, true>(P, J, u, w, v, u.n0 + CHUNK_COLS * c, c < 2 ? bias[0] : bias[1], res, abort_flag);
        }
      }
      if (!ok) {
        fail();
        break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_even + 8u * buf);    // the even CTA's MMA issuer may reuse the accumulator
    }
    // copies in flight (a residual's only after an abort) end before the CTA does
    if (res.asked != res.used) mbar_wait(res.landed, res.used & 1);
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();      // no multicast or remote arrival targets a CTA that has left
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// The parts of a job's contraction added, then the epilogue: a CTA for one chunk of one epilogue warp, whose warps take every
// fourth part each, and the first of them the others' sums in order.  The parts' loads are a chain of waits on the L2 that the
// ways shorten (16 parts by one warp: 9 us).
constexpr int JOIN_WAYS = 4;
template <bool FORWARD, typename T>
__global__ void __launch_bounds__(32 * JOIN_WAYS) linear_join_kernel(const __grid_constant__ LinearParams P, int job) {
  __shared__ int groups[2 * (LINEAR_MAX_GROUPS + 1)];
  __shared__ alignas(16) uint8_t chunk[CHUNK_BYTES];
  __shared__ float4 sums[JOIN_WAYS - 1][CHUNK_COLS / 4 * 32];
  begin_after_previous();
  const LinearJob& J = P.job[job];
  Groups G{groups, groups + LINEAR_MAX_GROUPS + 1, P.groups};
  const int way = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (way == 0) fill_groups(G, P.ends, P.rows, lane);
  __syncthreads();
  const int tile = blockIdx.x >> 1;
  const uint32_t rank = blockIdx.x & 1;
  if (tile >= job_units(J, G) / J.splits) return;
  Unit u;
  u.job = job;
  u.split = 0;
  decode_tile(J, G, tile, u);
  const int ew = blockIdx.y & (EPI_WARPS - 1), quad = (ew + 2) & 3, half = ew >> 2;         // as warps 2..9 of the kernel above
  WarpPlace w;
  w.lane = lane;
  w.buf = chunk;
  w.row0 = u.m0 + static_cast<int>(rank) * BM + quad * 32;
  w.rows = min(32, u.m_end - w.row0);
  if (w.rows <= 0) return;
  const int c = half + 2 * (blockIdx.y / EPI_WARPS), col0 = u.n0 + CHUNK_COLS * c;
  if (c >= u.wide / CHUNK_COLS || col0 >= J.N) return;
  const float2 bias = FORWARD ? bias_of<T>(P, J, u.group, col0, lane) : make_float2(0.f, 0.f);
  ResidualFeed none{nullptr, nullptr, 0, 0};
  Row v;
  const auto add = [&](const float4* part) {
#pragma unroll
    for (int i = 0; i < CHUNK_COLS / 4; ++i) {
      const float4 q = part[32 * i + lane];
      v.v[2 * i] = __fadd2_rn(v.v[2 * i], make_float2(q.x, q.y));
      v.v[2 * i + 1] = __fadd2_rn(v.v[2 * i + 1], make_float2(q.z, q.w));
    }
  };
#pragma unroll
  for (int i = 0; i < CHUNK_COLS / 2; ++i) v.v[i] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int s = way; s < J.splits; s += JOIN_WAYS) add(part_of(J, u, s, rank, ew, c >> 1));
  if (way > 0) {
#pragma unroll
    for (int i = 0; i < CHUNK_COLS / 4; ++i)
      sums[way - 1][32 * i + lane] = make_float4(v.v[2 * i].x, v.v[2 * i].y, v.v[2 * i + 1].x, v.v[2 * i + 1].y);
  }
  __syncthreads();
  if (way > 0) return;
#pragma unroll 1
  for (int i = 0; i < JOIN_WAYS - 1; ++i) add(sums[i]);
  finish_chunk<FORWARD, T, false>(P, J, u, w, v, col0, bias, none, nullptr);
}

// Per-device set-up (the shared-memory limit, the number of pairs that can be resident) is done by the first call on each
// device; concurrent first calls do the same idempotent work.
template <bool FORWARD, typename T, bool LOW>
cudaError_t launch_form(const LinearParams& p, int pairs_wanted, cudaStream_t s) {
  static std::atomic<int> resident[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int most = resident[dev].load(std::memory_order_acquire);
  if (most == 0) {
    e = cudaFuncSetAttribute(linear_kernel<FORWARD, T, LOW>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&most, linear_kernel<FORWARD, T, LOW>, &cfg);
    if (e != cudaSuccess) return e;
    if (most <= 0) return cudaErrorInvalidConfiguration;
    resident[dev].store(most, std::memory_order_release);
  }
  const int pairs = pairs_wanted < most ? pairs_wanted : most;
  return launch_after(linear_kernel<FORWARD, T, LOW>, dim3(2 * pairs), dim3(THREADS), SMEM, s, p, 2);
}

template <bool FORWARD, typename T>
cudaError_t launch_join_form(const LinearParams& p, int job, long long tiles, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * tiles), EPI_WARPS * (p.job[job].wide / 128));
  cfg.blockDim = dim3(32 * JOIN_WAYS);
  cfg.stream = s;
  cudaLaunchAttribute a[1]{};
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_join_kernel<FORWARD, T>, p, job);
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, int type, bool forward, int pairs_wanted, cudaStream_t s) {
  const bool low = p.jobs > 0 && p.job[0].passes > 1;      // (both jobs contract dz)
  if (type == MB_BF16)
    return forward ? launch_form<true, __nv_bfloat16, false>(p, pairs_wanted, s)
           : low   ? launch_form<false, __nv_bfloat16, true>(p, pairs_wanted, s)
                   : launch_form<false, __nv_bfloat16, false>(p, pairs_wanted, s);
  return forward ? launch_form<true, __half, false>(p, pairs_wanted, s)
         : low   ? launch_form<false, __half, true>(p, pairs_wanted, s)
                 : launch_form<false, __half, false>(p, pairs_wanted, s);
}

cudaError_t launch_linear_join(const LinearParams& p, int job, int type, bool forward, long long tiles, cudaStream_t s) {
  if (type == MB_BF16)
    return forward ? launch_join_form<true, __nv_bfloat16>(p, job, tiles, s) : launch_join_form<false, __nv_bfloat16>(p, job, tiles, s);
  return forward ? launch_join_form<true, __half>(p, job, tiles, s) : launch_join_form<false, __half>(p, job, tiles, s);
}

}  // namespace mb
