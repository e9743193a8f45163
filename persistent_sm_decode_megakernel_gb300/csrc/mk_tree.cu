// Attention of trees of drafted tokens over a paged KV cache (mk_tree_attention).
//
// Of one sequence and kv head the tree's nodes times the heads of the group are rows of one matrix Q, and its
// slots -- the cached positions and the nodes' own, which follow them -- are columns:
//   S = Q K^T,  P = 2^(S - m),  O = P V,  out = O / sum P,
// with a running maximum m per row.  Only the last one or two tiles of slots hold nodes, so all others
// are plain matrix products, and run on the fifth-generation tensor cores: S and O in tensor memory, K and V by
// tensor-map copies from the pages, P from the threads' registers into tensor memory, where it is the
// second product's first operand.
//
// Bound: the tensor cores, next to the keys' and values' bytes.  A tile of 64 slots costs a block of 128 rows 8 products
// for the scores, each 48 cycles (with both operands in shared memory its traffic decides: 64 columns take 48, not 32),
// and 4 of 64 for each part of the probabilities at 128 dims: two blocks of 16-bit queries 1792 cycles, the tile's arrival
// at the copy bandwidth 1100 to 1400, by the clock.  16 rows of 64 nodes over 16384 to 32768 positions, 32 heads over 8: 443 us,
// 3.8 TB/s and 0.97 PFLOP/s of the 32-bit product (half as much again is multiplied); one row of 16 nodes over 32768, 32-bit
// queries in two parts: 38.5 us; one of 8 nodes over 512: 12.9 us, the latency of a piece (7 us, most of it code executed
// for the first time) and of the join (3 us).
//
// The work is split as the single tokens' attention splits it: the segments (row, kv head), each of its tiles,
// follow one another in one line; every CTA of one wave takes an equal share of it; the pieces of a segment that
// spans CTAs go to the workspace and a second kernel joins them in order:
//   M = max M_i,  L = sum L_i 2^(M_i - M),  out = sum O_i 2^(M_i - M) / L.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "mk_internal.h"
#include "mk_device.cuh"
#include "mk_paged.cuh"
#include "mk_tmem.cuh"
#include "mk_tree.h"

namespace mk {
namespace {

constexpr int kMaxNodes = 128, kMaxGroup = 16;
constexpr int kRows = 128;               // rows of a block: the tensor cores' M
constexpr int kGroupThreads = 128;       // a softmax warpgroup: a thread per row
// two of them, then warps: the copies, each one's products, with SOLO the second one's copies
__host__ __device__ constexpr int tree_threads(int mode) { return 2 * kGroupThreads + (mode == 2 ? 128 : 96); }
constexpr int kTile = 64;                // slots that are copied, multiplied and weighted at a time
constexpr int kMaxStages = 10;
constexpr int kCopyWarp = 8, kMmaWarp = 9;
constexpr int kSmemBytes = 227 * 1024;
constexpr int kLead = 4;                 // tiles that a piece costs besides its own
constexpr int kJoinThreads = 256;
// Products that are added up in tensor memory at the most.  The tensor cores cut a sum off where it is longer than 32 bits
// instead of rounding it, always towards zero, so that a long piece's sums would fall behind by up to 2^-23 a product (32768
// positions in one piece: 2e-4 of every value).  After so many a row's thread takes its sums out, adds them, rounded, to those
// before, in the workspace, and begins anew.  512 in 16-bit outputs: a quarter of fp16's least half step (16 rows x 64 nodes x
// 24576, 32 heads over 8: 422 us without, 435 with it; 32-bit outputs over fp16 612 and 650, over bf16 1065 and 1175).
template <typename Q>
constexpr int kSumProducts = sizeof(Q) == 4 ? 128 : 512;
constexpr long long kWaitCycles = 4000000000ll;  // limit of a wait inside the kernel: two seconds

struct TreeArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  float* part;                           // [CTA][2][HD + 2][rows]: weighted values, maximum, sum
  float* sums;                           // [CTA][warpgroup][HD][q_rows]: weighted values of a piece's tiles so far
  int4* joins;                           // [CTA]: first and last share, row, kv head
  const int32_t *lens, *parents, *rows, *table;
  int32_t* status;
  long long q_row, q_node, q_head, o_row, o_node, o_head, page_stride, table_stride;
  int n_rows, n_nodes, hq, hkv, group, window, page_size, n_pages, table_rows, cap;
  int nodes_per_block, blocks;           // blocks of 128 rows that a segment's rows make up
  int parts;                             // CTAs of a share: each takes one block (PAIR: two) of its segments
  int shares;                            // of the line of work: one for each CTA of a part (SOLO: two)
  int part_rows;                         // rows of a piece in the workspace
  int q_rows;                            // rows of a block that hold queries, in whole 32s
  int tpp;                               // 16s of positions in a page
  unsigned tpp_inverse;                  // 2^32 / tpp, rounded up
  int box;                               // positions of a copy
  int q_vec, o_vec;                      // 16-byte accesses
  float scale, softcap;                  // scores to units of log 2: scale s, or softcap tanh(scale s)
  float q_sign;                          // -1: queries are negated (the scale was negative), 0: they are zero
  uint32_t q_and, q_xor;                 // the same for a pair of 16-bit ones
  int group_inverse;                     // 2^16 / group, rounded up
};

// Slots [lo, hi) of a row that some node may see, its tiles [t0, t0 + n).
struct Span {
  int lo, hi, t0, n, trow, len;
};
__device__ __forceinline__ Span span_of(const TreeArgs& a, int r) {
  Span s;
  s.trow = a.rows ? a.rows[r] : r;
  s.len = a.lens[r];
  const bool there = s.len >= 0 && (unsigned)s.trow < (unsigned)a.table_rows;
  s.hi = there ? (int)min((unsigned)s.len + (unsigned)a.n_nodes, (unsigned)a.cap) : 0;
  s.lo = there && a.window > 0 ? max(0, s.len - a.window + 1) : 0;  // the roots' first position
  s.t0 = s.lo / kTile;
  s.n = s.hi > s.lo ? (s.hi + kTile - 1) / kTile - s.t0 : 0;
  return s;
}

// A CTA's pieces, one after another; every warp of it walks them by itself.
struct Walk {
  int at, end, share, lead, row, before;  // next unit and end; the row that holds `at`, the units before it
};
struct Piece {
  Span sp;
  int r, head, first, count;              // tiles [first, first + count) of the segment's
  int last_unit;                          // of its segment
  bool whole;
};
__device__ __forceinline__ bool next_piece(const TreeArgs& a, Walk& w, Piece& p) {
  while (w.at < w.end) {
    p.sp = span_of(a, w.row);
    const int each = p.sp.n > 0 ? p.sp.n + w.lead : 0, units = each * a.hkv;
    if (w.at >= w.before + units) {
      w.before += units;
      ++w.row;
      continue;
    }
    p.r = w.row;
    p.head = (int)((unsigned)(w.at - w.before) / (unsigned)each);
    const int seg = w.before + p.head * each, stop = min(w.end, seg + each);
    p.first = max(0, w.at - seg - w.lead);
    p.count = stop - seg - w.lead - p.first;
    p.last_unit = seg + each - 1;
    p.whole = p.count == p.sp.n;
    w.at = stop;
    if (p.count > 0) return true;         // (none: of a segment's lead alone)
  }
  return false;
}

// C: the cache's type.  Q: the queries' and outputs' type.  NQ parts of C make up a query element, NP a
// probability.  How the two warpgroups of a CTA work:
//   PAIR: on two blocks of rows, one each, against the same tiles;
//   SOLO: on a share of the line each, by themselves, as two CTAs would;
//   TURNS: on one block, taking turns at the tiles and joining at a piece's end.
//
// Tensor memory, 256 columns a warpgroup: 128 of scores, 128 of O.  The scores have two buffers of a tile, so that
// the tensor cores work on one while the warpgroup is at the other (one buffer where P has three parts: it
// takes the place of the scores it comes from).
enum Mode : int { TURNS = 0, PAIR_MODE = 1, SOLO_MODE = 2 };
template <typename C, typename Q, int HD, int NQ, int NP, int MODE>
struct Shape {
  static constexpr bool PAIR = MODE == PAIR_MODE, SOLO = MODE == SOLO_MODE;
  static constexpr int BUFFERS = NP == 3 ? 1 : 2;
  // A ring of stages for each that takes its tiles: a product warp must see every load of its ring, in order.  (With one
  // ring of which each takes every second tile, one could look for a load whose stage still waits for the other's load
  // before it: loads land in any order, and the parity of a phase but one ago reads as done.)
  static constexpr int RINGS = PAIR ? 1 : 2;
  // Tiles of a warpgroup whose values are summed in tensor memory before the sum is put away (kSumProducts).
  static constexpr int kSumTiles = kSumProducts<Q> / (NP * kTile / 16);
  static constexpr int AHEAD = BUFFERS;             // tiles of a ring whose scores are asked for before the first values
  static constexpr int BLOCKS = PAIR ? 2 : 1;       // blocks of rows of a piece
  static constexpr int QUERIES = MODE == TURNS ? 1 : 2;  // places of a block's queries
  static __host__ __device__ constexpr int q_part(int rows) { return rows * HD * 2; }
  static __host__ __device__ constexpr int q_bytes(int rows) { return QUERIES * NQ * q_part(rows); }
  static_assert(NQ * 2 >= (int)sizeof(Q), "the outputs go through the queries' place");
  static constexpr int kStage = kTile * HD * 2;
  struct State {
    uint64_t full[kMaxStages], empty[kMaxStages], s_full[2][2], p_full[2][2], o_done[2][2], q_full[2], q_seen, finished;  // [warpgroup][buffer]
    uint32_t tmem;
    int abort;
    Walk walk[2];
    int sums[tree_threads(MODE) / 32][2];
    int parents[2][kMaxNodes];
    unsigned char bad[2][16];                // of the last tiles: groups of 16 slots on a bad page
    unsigned odd[8][2];                   // slots whose values are not all finite, of the last tiles
    float scale[QUERIES * kRows];
    float ml[2][kRows][2];
  };
  // stages of a ring: with SOLO four, and only the rows that hold queries have a place (the products read
  // on over what lies behind it, for rows that nobody looks at)
  static constexpr int kRoom = kSmemBytes - 1024 - (int)sizeof(State) - q_bytes(kRows);
  static constexpr int kAll = kRoom / kStage < kMaxStages ? kRoom / kStage : kMaxStages, kStages = SOLO ? 4 : kAll / RINGS;
  // (more than half of an SM's: there is one CTA on it, which takes all of the tensor memory)
  static __host__ __device__ constexpr int bytes(int rows) {
    const int used = 1024 + q_bytes(rows) + RINGS * kStages * kStage + (int)sizeof(State);
    return used > 120 * 1024 ? used : 120 * 1024;
  }
  static_assert(kStages >= 3 && RINGS * kStages <= kMaxStages && (SOLO || bytes(kRows) <= kSmemBytes), "shared memory");
  static_assert(!SOLO || bytes(32) <= kSmemBytes, "shared memory");
  // what the products of the last row of queries' place read beyond it lies in the ring
  static_assert(!SOLO || 8 * kStage >= kRows * 128, "shared memory");
  // the place of tile i's keys and values among the copies to a ring of a piece's `count` tiles in it: K0 .. K(AHEAD - 1), V0, K(AHEAD), V1, ..
  static __device__ __forceinline__ unsigned k_load(int i) { return i < AHEAD ? i : 2 * i - AHEAD + 1; }
  static __device__ __forceinline__ unsigned v_load(int i, int count) { return i + min(count, AHEAD + i); }
};

template <typename T>
constexpr float kShift = 0.f;             // fp16 probabilities are held times 2^10, so that small ones stay normal
template <>
constexpr float kShift<__half> = 10.f;
template <typename T>
constexpr float kSlack = 8.f;             // a maximum may be passed by this much before what is summed is rescaled
template <>
constexpr float kSlack<__half> = 5.f;

// the page of a row that a slot lies in: a multiplication of the slot's number in 16s (exact below 2^26, pages of up to 64 of them)
__device__ __forceinline__ int page_index(const TreeArgs& a, int slot) {
  const int t = slot >> 4;
  return a.tpp == 1 ? t : (int)__umulhi((unsigned)t, a.tpp_inverse);
}

// the node of a block that a row of it is of: row / group, exact for rows below 128 and groups up to 16
__device__ __forceinline__ int node_of(const TreeArgs& a, int row) { return row * a.group_inverse >> 16; }

// Waits for a phase of a barrier, a whole warp together (what follows may need it so), false where it did not come: a wait
// that takes too long sets *abort, and from then on none waits: the work goes on over whatever lies there, within its bounds,
// to its end.  With abort NULL: up to the limit in any case (what is in flight when a CTA ends).
// A barrier tells two phases apart: nobody looks for a phase before the one before it is over, nor after the next one is.
// Each phase is answered by its waiters before the next can end, and a ring's loads are waited for one by one, in order.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* abort) {
  bool come = mbar_try_wait(bar, parity);
  if (!come) {
    const long long begin = clock64();
    while (!(come = mbar_wait_hint(bar, parity, 100000))) {
      if (abort && *(volatile int*)abort) break;
      if (clock64() - begin > kWaitCycles) {
        if (abort) *(volatile int*)abort = 1;
        break;
      }
    }
  }
  __syncwarp();
  return come;
}
// the same for a whole warp, which goes on together
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, abort));
}
__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 1, %0;" ::"n"(2 * kGroupThreads) : "memory"); }
template <bool BOTH>
__device__ __forceinline__ void tile_sync(int wg) {
  if (BOTH)
    groups_sync();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(2 + wg), "n"(kGroupThreads) : "memory");
}

// whether a pair of 16-bit elements holds one that is infinite or NaN; the pair without it
template <typename C>
__device__ __forceinline__ uint32_t odd_mask(uint32_t w) {
  constexpr uint32_t e = std::is_same<C, __half>::value ? 0x7c00u : 0x7f80u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w >> 16 & e) == e ? 0xffff0000u : 0u);
}

// 32 bits of a 128-bit set from bit `off` on (any number), zeros beyond its ends
__device__ __forceinline__ unsigned bits_at(const unsigned (&set)[4], int off) {
  const int q = off >> 5;
  unsigned lo = 0, hi = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo = q == i ? set[i] : lo;
    hi = q + 1 == i ? set[i] : hi;
  }
  return __funnelshift_r(lo, hi, off & 31);
}
// ones at [x, y) of 32 bits
__device__ __forceinline__ unsigned ones(int x, int y) {
  x = min(max(x, 0), 32);
  y = min(max(y, 0), 32);
  const unsigned to = y == 32 ? 0xffffffffu : (1u << y) - 1, from = x == 32 ? 0xffffffffu : (1u << x) - 1;
  return y > x ? to & ~from : 0u;
}

// cap tanh(x / (2 log2 e)) = cap - 2 cap / (2^x + 1), off by 2^-22 cap: two of the hardware's approximations (2 ulp, 1 ulp) in the
// place of tanhf's 25 instructions, which took three times a tile's softmax.  For 16-bit outputs and caps up to 64, where that
// is 2^-16 of a score, a sixteenth of fp16's half step in a probability (33 rows x 7 nodes x 700, 16 heads over 8, cap 30: 35 us,
// with the finer one below 50).
constexpr float kCoarseCap = 64.f;
__device__ __forceinline__ float capped(float x, float cap) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(x) + 1.f));
  return fmaf(-2.f * cap, r, cap);
}

// cap tanh(x) for 32-bit outputs and larger caps, off by 2^-23 cap at most and by 2^-23 of itself up to a third of the cap, so
// that a cap far above the scores costs them nothing: small ones by the series of tanh (through x^11), the others with one
// step of Newton's behind the reciprocal's approximation.
__device__ __forceinline__ float capped_fine(float x, float cap) {
  const float d = ex2(x * (2.f * kLog2e)) + 1.f;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  r = d < 1e30f ? r * fmaf(-d, r, 2.f) : r;  // (infinity's is 0, NaN's NaN)
  const float q = x * x;
  float t = fmaf(q, -1382.f / 155925.f, 62.f / 2835.f);
  t = fmaf(q, t, -17.f / 315.f);
  t = fmaf(q, t, 2.f / 15.f);
  t = fmaf(q, t, -1.f / 3.f);
  t = fmaf(q * x, t, x);
  return q < 0.09f ? cap * t : fmaf(-2.f * cap, r, cap);
}

// A row's sums from tensor memory to the workspace, added to `f` times those that are there (-1: none are), and zeros in their
// place; and back, to be added once more.  (A row's words are its own thread's.  Calls, so that the loop over the tiles, which is
// short of registers, has no part of it.  What only adds does not wait for what is there; sums below the normal numbers it
// takes for zero.)
template <int HD>
__device__ __noinline__ void put_away(uint32_t t_o, float* sums, int rows, float f) {
  const bool fresh = f < 0.f, adds = __all_sync(0xffffffffu, f == 1.f);
#pragma unroll 1
  for (int x = 0; x < HD / 16; ++x) {
    uint32_t o[16];
    tmem_ld(t_o + 16 * x, o);
    tmem_wait_ld();
    float* at = sums + (size_t)16 * x * rows;
    if (adds) {
#pragma unroll
      for (int y = 0; y < 16; ++y) atomicAdd(at + y * rows, __uint_as_float(o[y]));
    } else {
      float had[16];
#pragma unroll
      for (int y = 0; y < 16; ++y) had[y] = fresh ? 0.f : __ldcg(at + y * rows);
#pragma unroll
      for (int y = 0; y < 16; ++y) __stcg(at + y * rows, fmaf(f, had[y], __uint_as_float(o[y])));
    }
#pragma unroll
    for (int y = 0; y < 16; ++y) o[y] = 0;
    tmem_st(t_o + 16 * x, o);
  }
  tmem_wait_st();
}
template <int HD>
__device__ __noinline__ void take_back(uint32_t t_o, const float* sums, int rows, float f) {
#pragma unroll 1
  for (int x = 0; x < HD / 16; ++x) {
    uint32_t o[16];
    float had[16];
#pragma unroll
    for (int y = 0; y < 16; ++y) had[y] = __ldcg(sums + (size_t)(16 * x + y) * rows);
    tmem_ld(t_o + 16 * x, o);
    tmem_wait_ld();
#pragma unroll
    for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(fmaf(f, had[y], __uint_as_float(o[y])));
    tmem_st(t_o + 16 * x, o);
  }
  tmem_wait_st();
}

// two sums or products at a time
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}

template <typename C, typename Q, int HD, int NQ, int NP, int MODE>
__global__ void __launch_bounds__(tree_threads(MODE), 1) tree_kernel(const __grid_constant__ TreeArgs a,
                                                                const __grid_constant__ CUtensorMap k_map,
                                                                const __grid_constant__ CUtensorMap v_map) {
  using SH = Shape<C, Q, HD, NQ, NP, MODE>;
  using State = typename SH::State;
  constexpr bool PAIR = SH::PAIR, SOLO = SH::SOLO;
  constexpr int ST = SH::kStages, HALVES = HD / 64, AHEAD = SH::AHEAD, kTreeThreads = tree_threads(MODE);
  constexpr int WORKERS = SOLO ? kGroupThreads : 2 * kGroupThreads;  // softmax threads of a piece
  constexpr uint32_t kType = std::is_same<C, __half>::value ? 0 : 1;
  extern __shared__ unsigned char tree_smem[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(tree_smem) + 1023) & ~uintptr_t(1023));
  const int place_rows = SOLO ? a.q_rows : kRows, q_part = SH::q_part(place_rows);
  unsigned char *s_q = base, *s_kv = base + SH::q_bytes(place_rows);
  State* st = reinterpret_cast<State*>(s_kv + SH::RINGS * ST * SH::kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int part = blockIdx.x % a.parts;
  // the share of warpgroup g (SOLO: the first of all CTAs come first)
  auto share_of = [&](int g) { return (int)blockIdx.x / a.parts + (SOLO ? g * (a.shares / 2) : 0); };
  if (warp == kCopyWarp) {
    constexpr int ALL = SH::RINGS * ST;
    if (lane < ALL) {
      mbar_init(&st->full[lane], 1);
      mbar_init(&st->empty[lane], SH::BLOCKS);
    } else if (lane < ALL + 2) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&st->s_full[lane - ALL][b], 1);
        mbar_init(&st->p_full[lane - ALL][b], kGroupThreads);
        mbar_init(&st->o_done[lane - ALL][b], 1);
      }
    } else if (lane == ALL + 2) {
      mbar_init(&st->q_full[0], WORKERS);
      mbar_init(&st->q_full[1], WORKERS);
      mbar_init(&st->q_seen, 2);
      mbar_init(&st->finished, 2);
      st->abort = 0;
    }
    mbar_fence_init();
    fence_proxy_async();
  }
  // the rows that hold queries, rounded up to whole warps' worth; the others of the blocks stay zero
  const int first_node = part * SH::BLOCKS * a.nodes_per_block;
  const int q_rows = PAIR ? 2 * kRows : min(place_rows, (min(a.nodes_per_block, a.n_nodes - first_node) * a.group + 31) / 32 * 32);
  for (int x = q_rows * 8 + tid; x < kRows * 8 && MODE == TURNS; x += kTreeThreads) {
#pragma unroll
    for (int y = 0; y < NQ * HALVES; ++y) reinterpret_cast<uint4*>(s_q)[y * kRows * 8 + x] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (MODE == TURNS && tid >= q_rows && tid < kRows) st->scale[tid] = 1.f;
  pdl_wait();
  // ---- this CTA's share of the line
  {
    const int per = (a.n_rows + kTreeThreads - 1) / kTreeThreads;
    const int r0 = min(a.n_rows, tid * per), r1 = min(a.n_rows, r0 + per);
    int tiles = 0, rows = 0;
    for (int r = r0; r < r1; ++r) {
      const int n = span_of(a, r).n;
      tiles += n;
      rows += n > 0;
    }
    int ti = tiles, ri = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, ti, o), y = __shfl_up_sync(0xffffffffu, ri, o);
      if (lane >= o) {
        ti += x;
        ri += y;
      }
    }
    if (lane == 31) {
      st->sums[warp][0] = ti;
      st->sums[warp][1] = ri;
    }
    if (warp == kMmaWarp) tmem_alloc_all(&st->tmem);
    __syncthreads();
    ti -= tiles;
    ri -= rows;
    int all_tiles = 0, all_rows = 0;
#pragma unroll
    for (int w = 0; w < kTreeThreads / 32; ++w) {
      const int x = st->sums[w][0], y = st->sums[w][1];
      ti += w < warp ? x : 0;
      ri += w < warp ? y : 0;
      all_tiles += x;
      all_rows += y;
    }
    // with a CTA for every tile the latency of a piece is all there is
    const int lead = all_tiles * a.hkv <= a.shares ? 0 : kLead;
    const int units = (all_tiles + all_rows * lead) * a.hkv, each = max(1, (units + a.shares - 1) / a.shares);
    const int mine = (tiles + rows * lead) * a.hkv;
#pragma unroll
    for (int g = 0; g < (SOLO ? 2 : 1); ++g) {
      const int share = share_of(g), at = min(units, each * share);
      int b = (ti + ri * lead) * a.hkv;
      if (at < units && at >= b && at < b + mine) {
        for (int r = r0; r < r1; ++r) {
          const int n = span_of(a, r).n, u = n > 0 ? (n + lead) * a.hkv : 0;
          if (at >= b && at < b + u) st->walk[g] = Walk{at, min(units, at + each), each, lead, r, b};
          b += u;
        }
      }
      if (tid == 0) {
        if (at >= units) st->walk[g] = Walk{at, at, each, lead, a.n_rows, 0};
        a.joins[share * a.parts + part] = make_int4(0, -1, 0, 0);
      }
    }
    // rows without slots: zeros; what is not there is reported
    if (all_rows < a.n_rows)
      for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
        if (span_of(a, r).n != 0) continue;
        for (int x = tid; x < a.n_nodes * a.hq * HD; x += kTreeThreads) {
          const int h = x / HD;
          static_cast<Q*>(a.out)[r * a.o_row + h / a.hq * a.o_node + h % a.hq * a.o_head + x % HD] = Conv<Q>::down(0.f);
        }
        for (int x = tid; x < a.n_nodes * a.hq && a.lse; x += kTreeThreads)
          a.lse[(long long)r * a.n_nodes * a.hq + x] = -INFINITY;
      }
    if (blockIdx.x == gridDim.x - 1)
      for (int r = tid; r < a.n_rows; r += kTreeThreads) {
        const Span s = span_of(a, r);
        if (s.len >= 0 && (unsigned)s.trow >= (unsigned)a.table_rows)
          report(a.status, MK_ERR_PAGES, PO_TREE, r, s.trow);
        else if (s.len >= a.cap) {  // every node's slot is past the table (there may be no tile whose softmax could tell)
          bool some = false;
          for (int i = 0; i < a.n_nodes; ++i) some = some || a.parents[(long long)r * a.n_nodes + i] == -1;
          if (some) report(a.status, MK_ERR_PAGES, PO_TREE, r, s.len);
        }
      }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  pdl_launch();
  const uint32_t tmem = __shfl_sync(0xffffffffu, st->tmem, 0);
  // whose share this warp works on
  const int own = !SOLO ? 0 : warp < kCopyWarp ? warp >> 2 : warp == kCopyWarp ? 0 : warp == kMmaWarp ? 0 : 1;
  Walk w = st->walk[own];
  w = Walk{__shfl_sync(0xffffffffu, w.at, 0), __shfl_sync(0xffffffffu, w.end, 0), __shfl_sync(0xffffffffu, w.share, 0),
           __shfl_sync(0xffffffffu, w.lead, 0), __shfl_sync(0xffffffffu, w.row, 0), __shfl_sync(0xffffffffu, w.before, 0)};
  const int self = share_of(own) * a.parts + part;  // the place of its pieces
  Piece p;
  unsigned loads = 0, loads1 = 0;         // tiles of keys or values asked for, or used; TURNS' copies: of the second ring
  // whose ring (TURNS' one copying warp: the first, and the second behind it)
  const int ring = PAIR ? 0 : warp < kCopyWarp ? warp >> 2 : warp == kMmaWarp + 1 || warp == kMmaWarp + 2 ? 1 : 0;
  s_kv += ring * ST * SH::kStage;
  uint64_t *full = st->full + ring * ST, *empty = st->empty + ring * ST;
  if (warp == kCopyWarp || (SOLO && warp == kMmaWarp + 2)) {
    // ------------------------------------------------------------------------- copies
    constexpr int LEAD = MODE == TURNS ? 2 * AHEAD : AHEAD;  // tiles whose keys come before the first values
    unsigned tiles = 0;
    bool run = true, begun = false;
    while (run && next_piece(a, w, p)) {
      if (begun) {  // the queries of a piece to come: to L2 while the one before it is worked on
        constexpr int LINES = HD * (int)sizeof(Q) / 128;
        const int nodes = min(SH::BLOCKS * a.nodes_per_block, a.n_nodes - first_node);
        for (int x = lane; x < nodes * a.group * LINES; x += 32) {
          const int y = x / LINES, nd = y / a.group;  // (of both blocks)
          prefetch_l2_line(static_cast<const Q*>(a.q) + p.r * a.q_row + (long long)(first_node + nd) * a.q_node +
                           (long long)(p.head * a.group + y - nd * a.group) * a.q_head + x % LINES * (128 / sizeof(Q)));
        }
      }
      const int boxes = kTile / a.box, half = lane / boxes;  // a lane per copy: 64 dims of some positions
      const int at0 = (p.sp.t0 + p.first) * kTile + lane % boxes * a.box;
      const bool on = half < HALVES;
      // whether anything of this lane's part of tile i is to be read, and the table's entry for it (asked for some tiles
      // ahead, looked at when it is used)
      auto read_of = [&](int i) {
        const int t = at0 + i * kTile;
        return i < p.count && on && t < p.sp.hi && t + a.box > p.sp.lo;
      };
      const int32_t* table = a.table + (long long)p.sp.trow * a.table_stride;
      auto entry_of = [&](int i) { return read_of(i) ? table[page_index(a, at0 + i * kTile)] : 0; };
      auto copy = [&](const CUtensorMap* map, int i, int page) {
        const int r = MODE == TURNS ? i & 1 : 0;
        const unsigned l = r ? loads1 : loads;
        const int s = r * ST + l % ST;
        if (!wait_warp(&empty[s], (l / ST & 1) ^ 1, &st->abort)) return false;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], SH::kStage);
        __syncwarp();
        const uint32_t dst = smem_addr(s_kv + s * SH::kStage) + half * kTile * 128 + lane % boxes * a.box * 128;
        const int t = at0 + i * kTile;
        const bool there = read_of(i) && (unsigned)page < (unsigned)a.n_pages;
        if (on)  // (a page outside the map: zeros)
          tma_box_4d(dst, map, 64 * half, there ? t - page_index(a, t) * a.page_size : 0, p.head, there ? page : a.n_pages, &full[s]);
        loads += 1 - r;
        loads1 += r;
        return true;
      };
      // the pages of the next tiles: the keys' is LEAD tiles before the values'
      int page[LEAD + 2];
#pragma unroll
      for (int i = 0; i < LEAD + 1; ++i) page[i] = entry_of(i);
      auto keys = [&](int i, int pg) {
        const bool none = half == 0 && read_of(i) && (unsigned)pg >= (unsigned)a.n_pages;
        unsigned bad = 0;
        if (__any_sync(0xffffffffu, none)) {  // the groups of 16 slots on a bad page
          if (none) bad = ((1u << (a.box / 16)) - 1) << (lane % boxes * (a.box / 16));
          bad = __reduce_or_sync(0xffffffffu, bad);
        }
        if (lane == 0) st->bad[own][tiles % 16] = (unsigned char)bad;
        __syncwarp();
        ++tiles;
        run = run && copy(&k_map, i, pg);
      };
#pragma unroll
      for (int i = 0; i < LEAD; ++i)
        if (i < p.count) keys(i, page[i]);
      // (the first queries do not queue behind the keys and values that fill the ring)
      if (!begun) wait_phase(&st->q_full[own], 0, &st->abort);
      begun = true;
      for (int i = 0; i < p.count && run; ++i) {
        page[LEAD + 1] = entry_of(i + LEAD + 1);
        run = copy(&v_map, i, page[0]);
        if (i + LEAD < p.count) keys(i + LEAD, page[LEAD]);
#pragma unroll
        for (int y = 0; y < LEAD + 1; ++y) page[y] = page[y + 1];
      }
    }
    // every copy has landed before the CTA ends
    for (unsigned i = loads > ST ? loads - ST : 0; i < loads; ++i) wait_phase(&full[i % ST], i / ST & 1, nullptr);
    for (unsigned i = loads1 > ST ? loads1 - ST : 0; i < loads1; ++i) wait_phase(&full[ST + i % ST], i / ST & 1, nullptr);
  } else if (warp >= kMmaWarp) {
    // ----------------------------------------------------------------------- products
    // A warp for each warpgroup: one alone takes longer to issue a job than the tensor cores to do it.  The whole
    // warp walks, so that what the instructions take stays in uniform registers; one lane issues.
    const int g = warp - kMmaWarp;
    const uint64_t q_desc = smem_desc(smem_addr(s_q) + (MODE == TURNS ? 0 : g) * NQ * q_part, 16, 1024);
    const uint64_t k_desc = smem_desc(smem_addr(s_kv), 16, 1024), v_desc = smem_desc(smem_addr(s_kv), kTile * 128, 1024);
    const uint32_t t_s = tmem + g * 256, t_o = t_s + 128;
    unsigned p_phase = 0, pieces = 0;     // p_phase: a bit per buffer
    while (next_piece(a, w, p)) {
      const int n = MODE != TURNS ? p.count : (p.count - g + 1) / 2;  // jobs: this warpgroup's tiles
      wait_phase(&st->q_full[own], pieces & 1, &st->abort);
      ++pieces;
      if (MODE == TURNS) {  // (a piece of one tile can be over before the second warp has looked: the next queries wait for both)
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->q_seen);
      }
      // The tensor cores take what one thread issues in order: a buffer's next scores come after the product
      // that read its P.
      auto scores = [&](int x) {
        const unsigned l = loads + SH::k_load(x), s = l % ST;
        const int b = SH::BUFFERS == 2 ? x & 1 : 0;
        wait_phase(&full[s], l / ST & 1, &st->abort);
        tmem_fence_after();
        if (elect_one()) {
          const uint64_t kd = k_desc + s * (SH::kStage / 16);
#pragma unroll
          for (int y = NQ - 1; y >= 0; --y)  // the smallest parts first: each product's sum is cut off, not rounded
#pragma unroll
            for (int c = 0; c < HD / 16; ++c)  // (the address counts in 16 bytes)
              mma_ss(t_s + b * kTile, q_desc + (y * q_part + (c >> 2) * place_rows * 128 + (c & 3) * 32) / 16,
                     kd + ((c >> 2) * kTile * 128 + (c & 3) * 32) / 16, mma_desc(kType, false, kRows, kTile), y < NQ - 1 || c > 0);
          mma_commit(&st->s_full[g][b]);
          mma_commit(&empty[s]);
        }
        __syncwarp();
      };
      auto values = [&](int x) {
        const unsigned l = loads + SH::v_load(x, n), s = l % ST;
        const int b = SH::BUFFERS == 2 ? x & 1 : 0;
        wait_phase(&full[s], l / ST & 1, &st->abort);
        wait_phase(&st->p_full[g][b], p_phase >> b & 1, &st->abort);
        p_phase ^= 1u << b;
        tmem_fence_after();
        if (elect_one()) {
          const uint64_t vd = v_desc + s * (SH::kStage / 16);
#pragma unroll
          for (int y = NP - 1; y >= 0; --y)
#pragma unroll
            for (int c = 0; c < kTile / 16; ++c)
              mma_ts(t_o, t_s + b * kTile + y * (kTile / 2) + c * 8, vd + c * 2048 / 16, mma_desc(kType, true, kRows, HD), true);
          mma_commit(&st->o_done[g][b]);
          mma_commit(&empty[s]);
        }
        __syncwarp();
      };
      for (int x = 0; x < min(n, SH::BUFFERS); ++x) scores(x);
      for (int x = 0; x < n; ++x) {
        values(x);
        if (x + SH::BUFFERS < n) scores(x + SH::BUFFERS);
      }
      loads += 2 * n;
    }
    if (elect_one()) mma_commit(&st->finished);
    __syncwarp();
    wait_phase(&st->finished, 0, nullptr);
  } else {
    // ------------------------------------------------------------------------ softmax
    const int g = warp >> 2, row = tid & (kGroupThreads - 1);  // warpgroup, row of its block
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;         // this warp's lanes of the tensor memory
    const uint32_t t_s0 = tmem + g * 256 + lanes, t_o = t_s0 + 128;
    const int node = first_node + (PAIR ? g * a.nodes_per_block : 0) + node_of(a, row), h = row - node_of(a, row) * a.group;
    const bool valid = row < a.nodes_per_block * a.group && node < a.n_nodes;
    const bool warp_valid = __any_sync(0xffffffffu, valid);
    auto workers_sync = [&]() { SOLO ? tile_sync<false>(g) : groups_sync(); };
    unsigned tiles = 0, s_phase = 0, pieces = 0;  // tiles and pieces so far; a bit per buffer: the next phase of its scores
    int row_of = -1;                      // whose tree `seen` is of
    unsigned seen[4] = {0, 0, 0, 0};
    int depth = 0;
    bool there = false;
    const int id = SOLO ? row : tid;      // of the piece's threads
    float* sums = a.sums + (size_t)(blockIdx.x * 2 + g) * HD * a.q_rows + row;  // what is put away
    while (next_piece(a, w, p)) {
      workers_sync();                      // what the last piece left in shared and tensor memory was read
      if (MODE == TURNS && pieces > 0) wait_phase(&st->q_seen, (pieces - 1) & 1, &st->abort);
      ++pieces;
      int parent = 0;                     // (asked for before the queries, stored behind them)
      const bool other_row = p.r != row_of;
      if (other_row && id < a.n_nodes) parent = a.parents[(long long)p.r * a.n_nodes + id];
      // ---- the queries, K-major, 128-byte swizzled; neighbouring lanes take neighbouring chunks of a row.  (What
      // is executed once or twice waits for its instructions: the loop is short, and ends with the rows.)
      {
        constexpr int CH = HD / 8, STEP = WORKERS / CH, U = PAIR ? 8 : NQ == 1 ? 4 : sizeof(Q) == 2 ? 2 : 1;
        const int c = id % CH;
        const Q* src = static_cast<const Q*>(a.q) + p.r * a.q_row + (long long)p.head * a.group * a.q_head + 8 * c;
#pragma unroll 1
        for (int x0 = id / CH; x0 < q_rows; x0 += U * STEP) {
          Raw8<Q> raw[U];
#pragma unroll
          for (int z = 0; z < U; ++z) {
            const int x = x0 + z * STEP, y = x % kRows, nd = node_of(a, y);  // row of all blocks, of its own
            raw[z] = {};
            if (x < q_rows && nd < a.nodes_per_block && x / kRows * a.nodes_per_block + nd < a.n_nodes - first_node) {
              const Q* from = src + (first_node + x / kRows * a.nodes_per_block + nd) * a.q_node + (y - nd * a.group) * a.q_head;
              if (a.q_vec)
                raw[z].load(from);
              else
                raw[z].gather(from);
            }
          }
#pragma unroll
          for (int z = 0; z < U; ++z) {
            const int x = x0 + z * STEP, y = x % kRows;
            uint32_t parts[4][NQ];
            if constexpr (std::is_same<C, Q>::value) {
              parts[0][0] = (raw[z].w[0].x & a.q_and) ^ a.q_xor;
              parts[1][0] = (raw[z].w[0].y & a.q_and) ^ a.q_xor;
              parts[2][0] = (raw[z].w[0].z & a.q_and) ^ a.q_xor;
              parts[3][0] = (raw[z].w[0].w & a.q_and) ^ a.q_xor;
            } else {
              float v[8];
              raw[z].up(v);
              float up = a.q_sign;
              if constexpr (kScaled<C, Q>) {  // the chunks of a row are in neighbouring lanes
                float most = fabsf(v[0]);
#pragma unroll
                for (int e = 1; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
#pragma unroll
                for (int o = 1; o < CH; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                const int shift = shift_of(most);
                up *= power_of(shift);
                if (c == 0 && x < q_rows) st->scale[(SOLO ? g * kRows : 0) + x] = a.scale * power_of(-shift);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) split2<C, NQ>(v[2 * e] * up, v[2 * e + 1] * up, parts[e]);
            }
            if (x < q_rows)
#pragma unroll
              for (int n = 0; n < NQ; ++n)
                *reinterpret_cast<uint4*>(s_q + ((SOLO ? g : x / kRows) * NQ + n) * q_part + (c >> 3) * place_rows * 128 + y * 128 +
                                          (((c & 7) ^ (y & 7)) << 4)) = make_uint4(parts[0][n], parts[1][n], parts[2][n], parts[3][n]);
          }
        }
      }
      {
        uint32_t zero[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) zero[i] = 0;
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) tmem_st(t_o + 32 * i, zero);
        tmem_wait_st();
      }
      if (other_row && id < a.n_nodes) st->parents[own][id] = parent;
      fence_proxy_async_shared();
      tmem_fence_before();
      mbar_arrive(&st->q_full[own]);
      workers_sync();                     // parents and scales are there
      const float scale = kScaled<C, Q> ? st->scale[(MODE != TURNS ? g * kRows : 0) + row] : a.scale;
      if (other_row) {                    // the node's ancestors that its window holds
        row_of = p.r;
#pragma unroll
        for (int i = 0; i < 4; ++i) seen[i] = 0;
        depth = 0;
        there = valid;
        for (int i = node; there;) {
          if (a.window == 0 || depth < a.window)
#pragma unroll
            for (int x = 0; x < 4; ++x) seen[x] |= (i >> 5) == x ? 1u << (i & 31) : 0u;
          const int up = st->parents[own][i];
          if (up == -1) break;
          there = up >= 0 && up < i;
          i = up;
          ++depth;
        }
        if (!there) {
#pragma unroll
          for (int i = 0; i < 4; ++i) seen[i] = 0;
        } else if ((unsigned)p.sp.len + (unsigned)node >= (unsigned)a.cap) {
          report(a.status, MK_ERR_PAGES, PO_TREE, p.r, p.sp.len);
        }
      }
      // the first position that a node of so many ancestors sees (lengths up to 2^31 - 1)
      auto from = [&](int up) {
        const unsigned end = (unsigned)p.sp.len + 1u + (unsigned)up;
        return a.window > 0 && end > (unsigned)a.window ? (int)min(end - (unsigned)a.window, 0x7fffffffu) : 0;
      };
      const int lo = there ? from(depth) : p.sp.len;
      const int plain_lo = from(a.n_nodes - 1);  // tiles in [plain_lo, len) are seen by all nodes whole
      float m = -INFINITY, l = 0.f;
      float away = -INFINITY;             // the maximum of the sums that were put away
      // before the sums so far are touched: the last product is done (of the buffer at hand it is: its scores came after it)
      auto sums_done = [&](int buf) {
        if (SH::BUFFERS == 2) wait_phase(&st->o_done[g][buf ^ 1], (s_phase >> (buf ^ 1) & 1) ^ 1, &st->abort);
        tmem_fence_after();
      };
      const int n = MODE != TURNS ? p.count : (p.count - g + 1) / 2;  // this warpgroup's tiles of the piece
      int turn = 0;                       // those that it has taken
      for (int i = MODE != TURNS ? 0 : g; i < p.count; i += MODE != TURNS ? 1 : 2, ++turn) {
        const int t0 = (p.sp.t0 + p.first + i) * kTile;
        const int buf = SH::BUFFERS == 2 ? turn & 1 : 0;
        const uint32_t t_s = t_s0 + buf * kTile;
        wait_phase(&st->s_full[g][buf], s_phase >> buf & 1, &st->abort);
        s_phase ^= 1u << buf;
        tmem_fence_after();
        const unsigned bad = *(volatile unsigned char*)&st->bad[own][(tiles + i) % 16];
        const bool partial = t0 < plain_lo || t0 + kTile > min(p.sp.len, p.sp.hi) || bad != 0;
        unsigned vis[2] = {0, 0};
        if (warp_valid) {
          if (turn > 0 && turn % SH::kSumTiles == 0) {
            sums_done(buf);
            put_away<HD>(t_o, sums, a.q_rows, turn == SH::kSumTiles ? -1.f : away == m ? 1.f : ex2(away - m));
            away = m;
          }
          float factor = scale;
          uint32_t s[2][32];
          tmem_ld(t_s, s[0]);
          tmem_ld(t_s + 32, s[1]);
          tmem_wait_ld();
          if (a.softcap > 0.f) {
            factor = 1.f;
            if (std::is_same<Q, float>::value || a.softcap > kCoarseCap * kLog2e) {
#pragma unroll
              for (int x = 0; x < kTile; ++x)
                s[x >> 5][x & 31] = __float_as_uint(capped_fine(__uint_as_float(s[x >> 5][x & 31]) * scale, a.softcap));
            } else {
              const float twice = scale * (2.f * kLog2e);
#pragma unroll
              for (int x = 0; x < kTile; ++x)
                s[x >> 5][x & 31] = __float_as_uint(capped(__uint_as_float(s[x >> 5][x & 31]) * twice, a.softcap));
            }
          }
          if (partial) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int b = t0 + 32 * x;
              vis[x] = ones(lo - b, p.sp.len - b) | bits_at(seen, b - p.sp.len);
              vis[x] &= ones(0, p.sp.hi - b);
              const unsigned none = (bad >> (2 * x) & 1 ? 0x0000ffffu : 0u) | (bad >> (2 * x) & 2 ? 0xffff0000u : 0u);
              if (vis[x] & none)           // (only what some node sees is missed: the slots of absent ones need no page)
                report(a.status, MK_ERR_PAGES, PO_TREE, p.r,
                       a.table[(long long)p.sp.trow * a.table_stride + page_index(a, b + __ffs(vis[x] & none) - 1)]);
              vis[x] &= ~none;
#pragma unroll
              for (int y = 0; y < 32; ++y) s[x][y] = vis[x] >> y & 1 ? s[x][y] : 0xff800000u;
            }
          }
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int x = 0; x < kTile; x += 2)
            tops[x >> 1 & 3] = fmaxf(fmaxf(tops[x >> 1 & 3], __uint_as_float(s[x >> 5][x & 31])), __uint_as_float(s[x >> 5][(x & 31) + 1]));
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * factor;
          // what was summed under a smaller maximum is brought to the new one, where it is much smaller
          const bool grown = top > m + kSlack<C>;
          const float to = grown ? top : m;
          const bool rescale = __any_sync(0xffffffffu, grown && m > -INFINITY);
          if (rescale) {
            sums_done(buf);
            const float f = grown ? ex2(m - to) : 1.f;
            l *= f;
#pragma unroll 1
            for (int x = 0; x < HD / 16; ++x) {
              uint32_t o[16];
              tmem_ld(t_o + 16 * x, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st(t_o + 16 * x, o);
            }
          }
          m = to;
          const float less = kShift<C> - (m == -INFINITY ? 0.f : m);
          const float2 factor2 = make_float2(factor, factor), less2 = make_float2(less, less);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t parts[NP][32];
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            float2 y = make_float2(__uint_as_float(s[x >> 4][2 * (x & 15)]), __uint_as_float(s[x >> 4][2 * (x & 15) + 1]));
            y = fma2(y, factor2, less2);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            sum[x & 1] = add2(sum[x & 1], y);
            uint32_t z[NP];
            split2<C, NP>(y.x, y.y, z);
#pragma unroll
            for (int e = 0; e < NP; ++e) parts[e][x] = z[e];
          }
#pragma unroll
          for (int e = 0; e < NP; ++e) tmem_st(t_s + e * (kTile / 2), parts[e]);
          const float2 both = add2(sum[0], sum[1]);
          l += both.x + both.y;
          tmem_wait_st();
        }
        if (partial) {
          // Values that are not finite must not meet the zero of one who does not see them: they are taken
          // out of the tile and added for those who do.  (Kept for eight tiles: one warpgroup may be ahead of the
          // other by what the ring holds, five tiles.)
          unsigned* found = st->odd[PAIR ? i & 7 : 2 * g + (turn & 1)];
          if (row < 2) found[row] = 0;
          tile_sync<PAIR>(g);
          const unsigned v_at = loads + SH::v_load(turn, n);
          wait_phase(&full[v_at % ST], v_at / ST & 1, &st->abort);
          uint4* v = reinterpret_cast<uint4*>(s_kv + v_at % ST * SH::kStage);
          constexpr int step = PAIR ? 2 * kGroupThreads : kGroupThreads;
#pragma unroll
          for (int z = 0; z < SH::kStage / 16 / step; ++z) {
            const int x = (PAIR ? tid : row) + z * step;
            const uint4 y = v[x];
            const uint32_t o0 = odd_mask<C>(y.x), o1 = odd_mask<C>(y.y), o2 = odd_mask<C>(y.z), o3 = odd_mask<C>(y.w);
            if (o0 | o1 | o2 | o3) {
              v[x] = make_uint4(y.x & ~o0, y.y & ~o1, y.z & ~o2, y.w & ~o3);
              const int slot = x / 8 % kTile;
              atomicOr(&found[slot >> 5], 1u << (slot & 31));
            }
          }
          fence_proxy_async_shared();
          tile_sync<PAIR>(g);
          const unsigned odd[2] = {found[0], found[1]};
          if (odd[0] | odd[1]) sums_done(buf);
#pragma unroll 1
          for (int x2 = 0; x2 < 2; ++x2) {
            for (unsigned rest = x2 ? odd[1] : odd[0]; rest; rest &= rest - 1) {
              const int x = 32 * x2 + __ffs(rest) - 1, t = t0 + x;
              const bool sees = (x2 ? vis[1] : vis[0]) >> (x & 31) & 1;
              if (!__any_sync(0xffffffffu, sees)) continue;
              // (who sees it has its page)
              const C* src = static_cast<const C*>(a.v) +
                             (long long)a.table[(long long)p.sp.trow * a.table_stride + t / a.page_size] * a.page_stride +
                             ((long long)p.head * a.page_size + t % a.page_size) * HD;
              float pr = 0.f;
#pragma unroll
              for (int z = 0; z < NP; ++z) {
                const uint32_t y = tmem_ld1(t_s + z * (kTile / 2) + (x >> 1));
                tmem_wait_ld();
                const float2 pair = unpack2<C>(y);
                pr += x & 1 ? pair.y : pair.x;
              }
              for (int c = 0; c < HD / 16; ++c) {
                uint32_t o[16];
                tmem_ld(t_o + 16 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  const float v = Conv<C>::up(src[16 * c + y]);
                  if (sees && !(fabsf(v) < INFINITY)) o[y] = __float_as_uint(fmaf(pr, v, __uint_as_float(o[y])));
                }
                tmem_st(t_o + 16 * c, o);
                tmem_wait_st();
              }
            }
          }
        }
        tmem_fence_before();
        mbar_arrive(&st->p_full[g][buf]);
      }
      for (int b = 0; b < SH::BUFFERS; ++b) wait_phase(&st->o_done[g][b], (s_phase >> b & 1) ^ 1, &st->abort);
      tiles += p.count;
      loads += 2 * n;
      // ---- the piece's result
      if (n > SH::kSumTiles && warp_valid) {
        tmem_fence_after();
        take_back<HD>(t_o, sums, a.q_rows, away == m ? 1.f : ex2(away - m));
      }
      if (!there) {                       // (an absent node's row went through the whole tiles with the others)
        m = -INFINITY;
        l = 0.f;
      }
      if (MODE == TURNS) {
        st->ml[g][row][0] = m;
        st->ml[g][row][1] = l;
        tmem_fence_before();
        groups_sync();
      }
      tmem_fence_after();
      if (id == 0 && !p.whole && p.first == 0)
        a.joins[self] = make_int4(share_of(own), (int)((unsigned)p.last_unit / (unsigned)w.share), p.r, p.head);
      if (!warp_valid) continue;
      float M = m, L = l, f0 = 1.f, f1 = 0.f;
      if (MODE == TURNS) {
        const float m0 = st->ml[0][row][0], m1 = st->ml[1][row][0];
        M = fmaxf(m0, m1);
        const float Ms = M == -INFINITY ? 0.f : M;
        f0 = ex2(m0 - Ms);
        f1 = ex2(m1 - Ms);
        L = fmaf(f0, st->ml[0][row][1], f1 * st->ml[1][row][1]);
      }
      const int slot = p.first == 0;      // 0: continues a segment, 1: begins one
      float* keep = a.part + (size_t)(self * 2 + slot) * a.part_rows * (HD + 2) + (PAIR ? g * kRows : 0) + row;
      const float inv = L == 0.f ? 0.f : 1.f / L;
      // this thread's dims: all of them, or the warpgroup's half.  What is whole goes through the queries' place
      // in shared memory (read by now), a warp's rows in rows of its own, so that whole runs are written.
      constexpr int DIMS = MODE != TURNS ? HD : HD / 2, kRun = DIMS * (int)sizeof(Q), RCH = kRun / 16, kTwist = RCH < 8 ? RCH - 1 : 7;
      const int d0 = MODE != TURNS ? 0 : g * DIMS;
      unsigned char* run = s_q + (MODE != TURNS ? g * NQ * q_part : 0) + (warp & 3) * 32 * HD * (int)sizeof(Q) + (MODE != TURNS ? 0 : g) * 32 * kRun;
#pragma unroll 1
      for (int c = 0; c < DIMS / 32; ++c) {
        uint32_t o[32];
        if (MODE != TURNS) {
          tmem_ld(t_o + 32 * c, o);
          tmem_wait_ld();
        } else {
          uint32_t o1[32];
          tmem_ld(tmem + lanes + 128 + d0 + 32 * c, o);
          tmem_ld(tmem + lanes + 256 + 128 + d0 + 32 * c, o1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(fmaf(f0, __uint_as_float(o[e]), f1 * __uint_as_float(o1[e])));
        }
        if (p.whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) x[y] = L == 0.f ? 0.f : __uint_as_float(o[8 * e + y]) * inv;
            union {
              Q q[8];
              uint4 v[sizeof(Q) / 2];
            } to;
#pragma unroll
            for (int y = 0; y < 8; ++y) to.q[y] = Conv<Q>::down(x[y]);
#pragma unroll
            for (int y = 0; y < (int)sizeof(Q) / 2; ++y) {
              const int ch = (4 * c + e) * ((int)sizeof(Q) / 2) + y;
              *reinterpret_cast<uint4*>(run + lane * kRun + ((ch ^ (lane & kTwist)) << 4)) = to.v[y];
            }
          }
        } else if (valid) {
#pragma unroll
          for (int e = 0; e < 32; ++e) keep[(d0 + 32 * c + e) * a.part_rows] = __uint_as_float(o[e]);
        }
      }
      if (p.whole) {
        __syncwarp();
        Q* out = static_cast<Q*>(a.out) + p.r * a.o_row + (long long)p.head * a.group * a.o_head + d0;
#pragma unroll 2
        for (int x = lane; x < 32 * RCH; x += 32) {
          const int y = (warp & 3) * 32 + x / RCH, ch = x % RCH, nd = node_of(a, y);
          const int at = first_node + (PAIR ? g * a.nodes_per_block : 0) + nd;
          if (nd >= a.nodes_per_block || at >= a.n_nodes) continue;
          const uint4 v = *reinterpret_cast<const uint4*>(run + x / RCH * kRun + ((ch ^ (x / RCH & kTwist)) << 4));
          Q* dst = out + at * a.o_node + (y - nd * a.group) * a.o_head + ch * (16 / sizeof(Q));
          if (a.o_vec) {
            *reinterpret_cast<uint4*>(dst) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 16 / (int)sizeof(Q); ++e) dst[e] = reinterpret_cast<const Q*>(&v)[e];
          }
        }
      }
      if (valid && (MODE != TURNS || g == 0)) {
        if (p.whole) {
          if (a.lse)
            a.lse[((long long)p.r * a.n_nodes + node) * a.hq + p.head * a.group + h] =
                ((M == -INFINITY ? 0.f : M) - kShift<C> + log2f(L)) * kLn2;
        } else {
          keep[(size_t)HD * a.part_rows] = M;
          keep[(size_t)(HD + 1) * a.part_rows] = L;
        }
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (tid == 0 && st->abort) report(a.status, MK_ERR_TIMEOUT, PO_TREE, -1, blockIdx.x);
  if (warp == kMmaWarp) tmem_free_all(tmem);
}

// Joins the pieces of the segments that span CTAs: a CTA per 32 rows and 32 dims of a block, a lane per row, a
// warp 4 dims; the pieces in order, eight of them in flight.
template <typename Q, int HD>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeArgs a, float shift) {
  constexpr int W = kJoinThreads / 32, E = 32 / W, U = 8;
  __shared__ float s_o[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch();
  const int4 job = a.joins[blockIdx.x];
  if (job.y < 0) return;
  const int part = blockIdx.x % a.parts, row0 = blockIdx.y * 32, d0 = blockIdx.z * 32;
  const int per = a.part_rows > kRows ? 2 : 1, r = job.z;
  const int row = min(row0 + lane, a.part_rows - 1);  // (past the last: loaded and not used)
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int b = job.x; b <= job.y; b += U) {
    float pm[U], pl[U], po[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int y = min(b + u, job.y);
      const float* src = a.part + (size_t)((y * a.parts + part) * 2 + (y == job.x)) * a.part_rows * (HD + 2) + row;
      pm[u] = src[(size_t)HD * a.part_rows];
      pl[u] = src[(size_t)(HD + 1) * a.part_rows];
#pragma unroll
      for (int e = 0; e < E; ++e) po[u][e] = src[(size_t)(d0 + warp * E + e) * a.part_rows];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u > job.y) continue;
      const float mn = fmaxf(m, pm[u]), ms = mn == -INFINITY ? 0.f : mn;
      const float f0 = ex2(m - ms), f1 = ex2(pm[u] - ms);
      l = l * f0 + pl[u] * f1;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f0 + po[u][e] * f1;
      m = mn;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[lane][warp * E + e] = l == 0.f ? 0.f : o[e] / l;
  // where row x of the blocks goes: its node and head, or no node
  auto place = [&](int x, int* node, int* head) {
    const int y = x % kRows, nd = node_of(a, y);
    *node = (part * per + x / kRows) * a.nodes_per_block + nd;
    *head = job.w * a.group + y - nd * a.group;
    return x < a.part_rows && nd < a.nodes_per_block && *node < a.n_nodes;
  };
  int node, head;
  if (warp == 0 && d0 == 0 && a.lse && place(row0 + lane, &node, &head))
    a.lse[((long long)r * a.n_nodes + node) * a.hq + head] = ((m == -INFINITY ? 0.f : m) - shift + log2f(l)) * kLn2;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int x = warp * E + e;
    if (place(row0 + x, &node, &head))
      static_cast<Q*>(a.out)[r * a.o_row + node * a.o_node + head * a.o_head + d0 + lane] = Conv<Q>::down(s_o[x][lane]);
  }
}

// a thread per node
__global__ void __launch_bounds__(kMaxNodes) places_kernel(const int32_t* lens, const int32_t* parents, const int32_t* rows, int n_nodes,
                                                            int32_t* positions, int32_t* slots, int32_t* table_rows) {
  __shared__ int s_parent[kMaxNodes];
  const int r = blockIdx.x, node = threadIdx.x;
  pdl_wait();
  pdl_launch();
  if (node < n_nodes) s_parent[node] = parents[(long long)r * n_nodes + node];
  const int len = lens[r];
  __syncthreads();
  if (node >= n_nodes) return;
  int depth = 0, i = node;
  bool there = len >= 0 && len <= 0x7fffffff - kMaxNodes;
  while (there) {
    const int up = s_parent[i];
    if (up == -1) break;
    there = up >= 0 && up < i;
    i = up;
    ++depth;
  }
  const long long at = (long long)r * n_nodes + node;
  positions[at] = there ? len + depth : -1;
  slots[at] = there ? len + node : -1;
  table_rows[at] = rows ? rows[r] : r;
}

// --------------------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
  }();
  return fn;
}

// Pages as [page][kv head][position][dim]; a copy lands 64 dims of `box` positions, 128-byte swizzled.  A
// page number of n_pages lies outside the map: the copy fills zeros.
mk_status page_map(CUtensorMap* map, const mk_page_view& c, void* base, int box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return paged_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.n_kv_heads, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c.head_dim * 2, (cuuint64_t)c.page_size * c.head_dim * 2, (cuuint64_t)c.page_stride * 2};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, c.dtype == MK_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
                         strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return paged_fail(MK_ERR_INVALID, "the pages' tensor map was refused (" + std::to_string((int)r) + ")");
  return MK_OK;
}

// How a call's rows are dealt: blocks of 128, and CTAs that take one (16-bit queries of the cache's type: two)
// of a share's blocks.
struct Deal {
  int nodes_per_block, blocks, parts, part_rows, q_rows;
  bool pair;
};
Deal deal(int n_nodes, int group, bool same_type) {
  Deal d;
  d.nodes_per_block = kRows / group;
  d.blocks = (n_nodes + d.nodes_per_block - 1) / d.nodes_per_block;
  d.pair = same_type && d.blocks > 1;
  d.parts = d.pair ? (d.blocks + 1) / 2 : d.blocks;
  d.part_rows = d.pair ? 2 * kRows : d.blocks > 1 ? kRows : n_nodes * group;
  d.q_rows = std::min(kRows, (std::min(n_nodes, d.nodes_per_block) * group + 31) / 32 * 32);
  return d;
}

// floats of the sums that are put away
size_t sums_count(int n_sm, int head_dim, int q_rows) { return (size_t)n_sm * 2 * head_dim * q_rows; }

template <typename C, typename Q, int HD, int NQ, int NP, int MODE>
mk_status launch_mode(TreeArgs a, const mk_page_view& view, int n_sm, void* stream) {
  using SH = Shape<C, Q, HD, NQ, NP, MODE>;
  const int ctas = std::max(1, n_sm / a.parts) * a.parts;
  a.shares = ctas / a.parts * (SH::SOLO ? 2 : 1);
  a.box = 16;
  while (a.box < kTile && a.page_size % (2 * a.box) == 0) a.box *= 2;
  CUtensorMap k_map, v_map;
  mk_status s = page_map(&k_map, view, view.k, a.box);
  if (!s) s = page_map(&v_map, view, view.v, a.box);
  if (s) return s;
  auto kernel = tree_kernel<C, Q, HD, NQ, NP, MODE>;
  const int smem = SH::bytes(SH::SOLO ? a.q_rows : kRows);
  static SmemLimit limit;
  s = limit.raise(kernel, SH::SOLO ? kSmemBytes : smem, "mk_tree_attention");
  if (s) return s;
  s = launch_dependent(kernel, dim3(ctas), dim3(tree_threads(MODE)), smem, stream, "mk_tree_attention", a, k_map, v_map);
  if (s) return s;
  return launch_dependent(tree_join_kernel<Q, HD>, dim3(a.shares * a.parts, (a.part_rows + 31) / 32, HD / 32), dim3(kJoinThreads),
                          0, stream, "mk_tree_attention (join)", a, kShift<C>);
}
template <typename C, typename Q, int HD, int NQ, int NP>
mk_status launch_tree(const TreeArgs& a, const mk_page_view& view, bool pair, int n_sm, void* stream) {
  if constexpr (NQ == 1) {
    if (pair) return launch_mode<C, Q, HD, NQ, NP, PAIR_MODE>(a, view, n_sm, stream);
  }
  // SOLO where there are segments enough for a third of the CTAs (8 nodes, 8 kv heads, bf16: 16 rows of 4500 to 9000
  // positions 79 us, TURNS 102; 64 rows 279, 373), TURNS where there are fewer and a piece's latency counts (32-bit queries
  // over fp16, one row of 512 positions: 13.2 us, SOLO 13.8; one of 32768 38.7, 40.4)
  const bool solo = 3LL * a.n_rows * a.hkv * a.parts >= n_sm;
  if (solo && Shape<C, Q, HD, NQ, NP, SOLO_MODE>::bytes(a.q_rows) <= kSmemBytes)
    return launch_mode<C, Q, HD, NQ, NP, SOLO_MODE>(a, view, n_sm, stream);
  return launch_mode<C, Q, HD, NQ, NP, TURNS>(a, view, n_sm, stream);
}
template <typename C, typename Q, int NQ, int NP>
mk_status launch_tree(const TreeArgs& a, const mk_page_view& view, bool pair, int n_sm, void* stream) {
  return view.head_dim == 64 ? launch_tree<C, Q, 64, NQ, NP>(a, view, pair, n_sm, stream)
                             : launch_tree<C, Q, 128, NQ, NP>(a, view, pair, n_sm, stream);
}

}  // namespace

mk_status tree_places(const int32_t* lens, const int32_t* parents, const int32_t* rows, int n_rows, int n_nodes, int32_t* positions,
                      int32_t* slots, int32_t* table_rows, void* stream) {
  return launch_dependent(places_kernel, dim3(n_rows), dim3(kMaxNodes), 0, stream, "the nodes' places", lens, parents, rows, n_nodes,
                          positions, slots, table_rows);
}

}  // namespace mk

extern "C" mk_status mk_tree_attention_workspace(int n_nodes, int n_heads, int n_kv_heads, int head_dim, size_t* bytes) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    if (!bytes) return paged_fail(MK_ERR_INVALID, "bytes is NULL");
    if (n_nodes < 1 || n_nodes > kMaxNodes) return paged_fail(MK_ERR_INVALID, "n_nodes must be in [1, 128]");
    if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > kMaxGroup)
      return paged_fail(MK_ERR_INVALID, "n_heads / n_kv_heads must be a whole number in [1, 16]");
    if (head_dim != 64 && head_dim != 128) return paged_fail(MK_ERR_INVALID, "head_dim must be 64 or 128");
    int n_sm = 0;
    const mk_status s = sm_count(&n_sm);
    if (s) return s;
    size_t rows = 0;  // of a CTA's pieces at once: two shares' of one block, or one's of two
    for (bool same : {false, true}) {
      const Deal d = deal(n_nodes, n_heads / n_kv_heads, same);
      rows = std::max<size_t>(rows, d.pair ? d.part_rows : 2 * d.part_rows);
    }
    *bytes = (size_t)n_sm * (2 * sizeof(int4) + 2 * rows * (head_dim + 2) * sizeof(float)) +
             sums_count(n_sm, head_dim, deal(n_nodes, n_heads / n_kv_heads, true).q_rows) * sizeof(float);
    return MK_OK;
  });
}

extern "C" mk_status mk_tree_attention(const mk_tree_args* args, const mk_page_view* cache, int32_t* status, void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    const std::string e = check_view(cache);
    if (!e.empty()) return paged_fail(MK_ERR_INVALID, e);
    if (!args || !args->q || !args->out || !args->lens || !args->parents) return paged_fail(MK_ERR_INVALID, "NULL argument");
    if (args->dtype < MK_F16 || args->dtype > MK_F32) return paged_fail(MK_ERR_INVALID, "dtype");
    if (args->n_nodes < 1 || args->n_nodes > kMaxNodes) return paged_fail(MK_ERR_INVALID, "n_nodes must be in [1, 128]");
    if (args->n_heads < 1 || args->n_heads % cache->n_kv_heads || args->n_heads / cache->n_kv_heads > kMaxGroup)
      return paged_fail(MK_ERR_INVALID, "n_heads / n_kv_heads must be a whole number in [1, 16]");
    if (args->n_rows < 0 || (long long)args->n_rows * args->n_nodes * args->n_heads > 0x7fffffffLL / cache->head_dim)
      return paged_fail(MK_ERR_INVALID, "n_rows * n_nodes * n_heads * head_dim must be in [0, 2^31)");
    if (args->window < 0) return paged_fail(MK_ERR_INVALID, "window must not be negative");
    const float softcap = cap_of(args->softcap), factor = softcap > 0.f ? args->scale / softcap : args->scale * kLog2e;
    if (!(args->softcap >= 0.f && 2.f * args->softcap * kLog2e < INFINITY) || !(std::abs(factor) * 2.f * kLog2e < INFINITY))
      return paged_fail(MK_ERR_INVALID, "scale or softcap is not finite, too large, or softcap negative or too small for scale");
    const size_t esz = args->dtype == MK_F32 ? 4 : 2;
    if (!aligned_to(args->q, esz) || !aligned_to(args->out, esz))
      return paged_fail(MK_ERR_INVALID, "q and out must be aligned to their type");
    const long long rn = args->n_rows, nn = args->n_nodes, hn = args->n_heads, hd = cache->head_dim;
    if (overlaps(rn, args->o_row, nn, args->o_node, hd) || overlaps(rn, args->o_row, hn, args->o_head, hd) ||
        overlaps(nn, args->o_node, hn, args->o_head, hd))
      return paged_fail(MK_ERR_INVALID, "the vectors of out overlap");
    // the line of work counts in 32 bits, in tiles of 64 at the least
    const long long cap = (long long)cache->table_width * cache->page_size;
    const long long most = (args->window > 0 ? std::min(cap, (long long)args->window + kMaxNodes + kTile) : cap) / kTile + 2 + kLead;
    if (most * rn > 0x7f000000LL / cache->n_kv_heads)
      return paged_fail(MK_ERR_INVALID, "n_rows * n_kv_heads * (the table's positions / 64 + 6) must be below 2^31 - 2^24");
    if (!args->workspace || !aligned_to(args->workspace, 16)) return paged_fail(MK_ERR_INVALID, "the workspace is missing or unaligned");
    if (args->n_rows == 0) return MK_OK;
    size_t need = 0;
    mk_status s = mk_tree_attention_workspace(args->n_nodes, args->n_heads, cache->n_kv_heads, cache->head_dim, &need);
    if (s) return s;
    if (args->workspace_bytes < need)
      return paged_fail(MK_ERR_INVALID, "the workspace is too small (mk_tree_attention_workspace)");
    int n_sm = 0;
    s = sm_count(&n_sm);
    if (s) return s;
    TreeArgs a{};
    a.q = args->q; a.k = cache->k; a.v = cache->v; a.out = args->out; a.lse = args->lse;
    a.lens = args->lens; a.parents = args->parents; a.rows = args->rows; a.table = cache->table; a.status = status;
    a.q_row = args->q_row; a.q_node = args->q_node; a.q_head = args->q_head;
    a.o_row = args->o_row; a.o_node = args->o_node; a.o_head = args->o_head;
    a.page_stride = cache->page_stride; a.table_stride = cache->table_stride;
    a.n_rows = args->n_rows; a.n_nodes = args->n_nodes; a.hq = args->n_heads; a.hkv = cache->n_kv_heads;
    a.group = a.hq / a.hkv; a.window = args->window; a.page_size = cache->page_size; a.n_pages = cache->n_pages;
    a.table_rows = cache->n_rows; a.cap = (int)cap;
    a.tpp = a.page_size / 16;
    a.tpp_inverse = a.tpp > 1 ? (unsigned)(((1ULL << 32) + a.tpp - 1) / a.tpp) : 0;
    const Deal d = deal(a.n_nodes, a.group, args->dtype == cache->dtype);
    a.nodes_per_block = d.nodes_per_block; a.blocks = d.blocks; a.parts = d.parts; a.part_rows = d.part_rows;
    a.q_rows = d.q_rows;
    a.joins = static_cast<int4*>(args->workspace);
    a.sums = reinterpret_cast<float*>(a.joins + 2 * n_sm);
    a.part = a.sums + sums_count(n_sm, cache->head_dim, d.q_rows);
    const long long per = 16 / (long long)esz;
    a.q_vec = aligned_to(a.q, 16) && a.q_row % per == 0 && a.q_node % per == 0 && a.q_head % per == 0;
    a.o_vec = aligned_to(a.out, 16) && a.o_row % per == 0 && a.o_node % per == 0 && a.o_head % per == 0;
    a.scale = factor == 0.f ? 1.f : std::abs(factor);
    a.q_sign = factor == 0.f ? 0.f : factor < 0.f ? -1.f : 1.f;
    a.q_and = factor == 0.f ? 0u : 0xffffffffu;
    a.q_xor = factor < 0.f ? 0x80008000u : 0u;
    a.group_inverse = (65536 + a.group - 1) / a.group;
    a.softcap = softcap * kLog2e;
    // 16-bit queries of the cache's type are exact in one part, others are split into 2 parts of fp16 (22
    // bits, each head at a power of two of its own) or 3 of bf16 (24 bits); probabilities likewise, 2 parts of bf16 (16
    // bits) being enough for an output of 16 bits, as for single tokens.  (One part, 8 or 11 bits, is as far off as the
    // output's own rounding: 2.3e-3 from 64 bits where that gives 1.7e-3.)
    if (cache->dtype == MK_F16) {
      if (args->dtype == MK_F16) return launch_tree<__half, __half, 1, 2>(a, *cache, d.pair, n_sm, stream);
      if (args->dtype == MK_BF16) return launch_tree<__half, __nv_bfloat16, 2, 2>(a, *cache, d.pair, n_sm, stream);
      return launch_tree<__half, float, 2, 2>(a, *cache, d.pair, n_sm, stream);
    }
    if (args->dtype == MK_BF16) return launch_tree<__nv_bfloat16, __nv_bfloat16, 1, 2>(a, *cache, d.pair, n_sm, stream);
    if (args->dtype == MK_F16) return launch_tree<__nv_bfloat16, __half, 2, 2>(a, *cache, d.pair, n_sm, stream);
    return launch_tree<__nv_bfloat16, float, 3, 3>(a, *cache, d.pair, n_sm, stream);
  });
}
