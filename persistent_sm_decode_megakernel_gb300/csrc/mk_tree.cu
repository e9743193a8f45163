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

namespace mk {
namespace {

constexpr int kMaxNodes = 128, kMaxGroup = 16;
constexpr int kRows = 128;               // rows of a block: the tensor cores' M
constexpr int kGroupThreads = 128;       // a softmax warpgroup: a thread per row
constexpr int kTreeThreads = 3 * kGroupThreads;  // two of them, and one with a warp for the copies, one for the products
// registers of a thread: 168 at the launch (384 threads), of which the third group gives its share to the others
constexpr int kMoreRegs = 216, kFewRegs = 72;
static_assert(2 * kMoreRegs + kFewRegs <= 3 * 168, "registers");
constexpr int kCopyWarp = 8, kMmaWarp = 9;
constexpr int kSmemBytes = 227 * 1024;
constexpr int kLead = 2;                 // tiles that a piece costs besides its own
constexpr int kJoinThreads = 256;
constexpr unsigned long long kWaitNs = 2000000000ull;  // limit of a wait inside the kernel

struct TreeArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  float* part;                           // [CTA][2][rows][HD + 4]: weighted values, maximum, sum
  int4* joins;                           // [CTA]: first and last share, row, kv head
  const int32_t *lens, *parents, *rows, *table;
  int32_t* status;
  long long q_row, q_node, q_head, o_row, o_node, o_head, page_stride, table_stride;
  int n_rows, n_nodes, hq, hkv, group, window, page_size, n_pages, table_rows, cap;
  int nodes_per_block, blocks;           // blocks of 128 rows that a segment's rows make up
  int parts;                             // CTAs of a share: each takes one block (PAIR: two) of its segments
  int shares;
  int part_rows;                         // rows of a piece in the workspace
  int box;                               // positions of a copy
  int q_vec, o_vec;                      // 16-byte accesses
  float scale, softcap;                  // scores to units of log 2: scale s, or softcap tanh(scale s)
  float q_sign;                          // -1: queries are negated (the scale was negative), 0: they are zero
};

// Slots [lo, hi) of a row that some node may see, its tiles [t0, t0 + n).
struct Span {
  int lo, hi, t0, n, trow, len;
};
template <int TILE>
__device__ __forceinline__ Span span_of(const TreeArgs& a, int r) {
  Span s;
  s.trow = a.rows ? a.rows[r] : r;
  s.len = a.lens[r];
  const bool there = s.len >= 0 && (unsigned)s.trow < (unsigned)a.table_rows;
  s.hi = there ? (int)min((unsigned)s.len + (unsigned)a.n_nodes, (unsigned)a.cap) : 0;
  s.lo = there && a.window > 0 ? max(0, s.len - a.window + 1) : 0;  // the roots' first position
  s.t0 = s.lo / TILE;
  s.n = s.hi > s.lo ? (s.hi + TILE - 1) / TILE - s.t0 : 0;
  return s;
}

// A CTA's pieces, one after another; every warp of it walks them by itself.
struct Walk {
  int at, end, share, lead, row, before;  // next unit and end; the row that holds `at`, the units before it
};
struct Piece {
  Span sp;
  int r, head, first, count;              // tiles [first, first + count) of the segment's
  int last_share;                         // the share its segment ends in
  bool whole;
};
template <int TILE>
__device__ __forceinline__ bool next_piece(const TreeArgs& a, Walk& w, Piece& p) {
  while (w.at < w.end) {
    p.sp = span_of<TILE>(a, w.row);
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
    p.last_share = (int)((unsigned)(seg + each - 1) / (unsigned)w.share);
    p.whole = p.count == p.sp.n;
    w.at = stop;
    if (p.count > 0) return true;         // (none: of a segment's lead alone)
  }
  return false;
}

// C: the cache's type.  Q: the queries' and outputs' type.  NQ parts of C make up a query element, NP a
// probability.  PAIR: the CTA takes two blocks of rows, a warpgroup each, against the same tiles; else one
// block, the warpgroups taking turns at the tiles and joining at a piece's end.
template <typename C, int HD, int NQ, int NP, bool PAIR>
struct Shape {
  static constexpr int TILE = NP == 3 ? 64 : 128;  // slots: S and all parts of P lie in the same 128 columns
  static constexpr int BLOCKS = PAIR ? 2 : 1;
  static constexpr int kQPart = kRows * HD * 2, kQBytes = BLOCKS * NQ * kQPart;
  static constexpr int kStage = TILE * HD * 2;
  struct State {
    uint64_t full[8], empty[8], s_full[2], p_full[2], o_done[2], q_full, finished;
    uint32_t tmem;
    int abort;
    Walk walk;
    int sums[kTreeThreads / 32][2];
    int parents[kMaxNodes];
    unsigned char bad[16];                // of the last tiles: groups of 16 slots on a bad page
    unsigned odd[2][4];                   // slots whose values are not all finite, of a warpgroup's tile (PAIR: of two tiles in turn)
    float scale[BLOCKS][kRows];
    float ml[2][kRows][2];
  };
  static constexpr int kRoom = kSmemBytes - 1024 - (int)sizeof(State) - kQBytes;
  static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
  static constexpr int kBytes = 1024 + kQBytes + kStages * kStage + (int)sizeof(State);
  static_assert(kStages >= 3, "shared memory");
  static_assert(kBytes <= kSmemBytes && kBytes > kSmemBytes / 2, "one CTA per SM: it takes all of the tensor memory");
};

template <typename T>
constexpr float kShift = 0.f;             // fp16 probabilities are held times 2^10, so that small ones stay normal
template <>
constexpr float kShift<__half> = 10.f;
template <typename T>
constexpr float kSlack = 8.f;             // a maximum may be passed by this much before what is summed is rescaled
template <>
constexpr float kSlack<__half> = 5.f;

// Waits for a phase of a barrier: a wait that takes too long sets *abort, and from then on none waits.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long begin = globaltimer_ns();
  while (!mbar_wait_hint(bar, parity, 100000)) {
    if (*(volatile int*)abort) return false;
    if (globaltimer_ns() - begin > kWaitNs) {
      *(volatile int*)abort = 1;
      return false;
    }
  }
  return true;
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

template <typename C, typename Q, int HD, int NQ, int NP, bool PAIR>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a,
                                                                const __grid_constant__ CUtensorMap k_map,
                                                                const __grid_constant__ CUtensorMap v_map) {
  using SH = Shape<C, HD, NQ, NP, PAIR>;
  using State = typename SH::State;
  constexpr int TILE = SH::TILE, ST = SH::kStages, HALVES = HD / 64, WORDS = TILE / 32;
  constexpr uint32_t kType = std::is_same<C, __half>::value ? 0 : 1;
  extern __shared__ unsigned char tree_smem[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(tree_smem) + 1023) & ~uintptr_t(1023));
  unsigned char *s_q = base, *s_kv = base + SH::kQBytes;
  State* st = reinterpret_cast<State*>(s_kv + ST * SH::kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&st->full[i], 1);
      mbar_init(&st->empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&st->s_full[w], 1);
      mbar_init(&st->p_full[w], kGroupThreads);
      mbar_init(&st->o_done[w], 1);
    }
    mbar_init(&st->q_full, 2 * kGroupThreads);
    mbar_init(&st->finished, 1);
    st->abort = 0;
    mbar_fence_init();
    fence_proxy_async();
  }
  pdl_wait();
  // ---- this CTA's share of the line
  const int per = (a.n_rows + kTreeThreads - 1) / kTreeThreads;
  const int r0 = min(a.n_rows, tid * per), r1 = min(a.n_rows, r0 + per);
  {
    int tiles = 0, rows = 0;
    for (int r = r0; r < r1; ++r) {
      const int n = span_of<TILE>(a, r).n;
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
    const int at = min(units, each * share);
    if (tid == 0) {
      st->walk = Walk{at, min(units, at + each), each, lead, a.n_rows, 0};
      a.joins[blockIdx.x] = make_int4(0, -1, 0, 0);
    }
    __syncthreads();
    int b = (ti + ri * lead) * a.hkv;
    const int mine = (tiles + rows * lead) * a.hkv;
    if (at < units && at >= b && at < b + mine)
      for (int r = r0; r < r1; ++r) {
        const int n = span_of<TILE>(a, r).n, u = n > 0 ? (n + lead) * a.hkv : 0;
        if (at >= b && at < b + u) {
          st->walk.row = r;
          st->walk.before = b;
        }
        b += u;
      }
    // rows without slots: zeros; what is not there is reported
    if (all_rows < a.n_rows)
      for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
        if (span_of<TILE>(a, r).n != 0) continue;
        for (int x = tid; x < a.n_nodes * a.hq * HD; x += kTreeThreads) {
          const int h = x / HD;
          static_cast<Q*>(a.out)[r * a.o_row + h / a.hq * a.o_node + h % a.hq * a.o_head + x % HD] = Conv<Q>::down(0.f);
        }
        for (int x = tid; x < a.n_nodes * a.hq && a.lse; x += kTreeThreads)
          a.lse[(long long)r * a.n_nodes * a.hq + x] = -INFINITY;
      }
    if (blockIdx.x == gridDim.x - 1)
      for (int r = tid; r < a.n_rows; r += kTreeThreads) {
        const Span s = span_of<TILE>(a, r);
        if (s.len >= 0 && (unsigned)s.trow >= (unsigned)a.table_rows)
          report(a.status, MK_ERR_PAGES, PO_TREE, r, s.trow);
        else if (s.len >= 0 && (unsigned)s.len + (unsigned)a.n_nodes > (unsigned)a.cap)
          report(a.status, MK_ERR_PAGES, PO_TREE, r, s.len);
      }
  }
  __syncthreads();
  tmem_fence_after();
  pdl_launch();
  const uint32_t tmem = st->tmem;
  Walk w = st->walk;
  Piece p;
  unsigned loads = 0;                     // tiles of keys or values asked for, or used

  if (warp >= kCopyWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
  if (warp == kCopyWarp) {
    // ------------------------------------------------------------------------- copies
    // in the order in which the products take them: K0 (K1) V0 K2 V1 .. or, PAIR, K0 V0 K1 V1 ..
    unsigned tiles = 0;
    bool run = true;
    while (run && next_piece<TILE>(a, w, p)) {
      const int boxes = TILE / a.box, mine = lane / boxes;  // a lane per copy: 64 dims of some positions
      const int at0 = (p.sp.t0 + p.first) * TILE + lane % boxes * a.box;
      const bool on = mine < HALVES;
      auto page_of = [&](int i) {          // the page of this lane's part of tile i, n_pages where nothing is to be read
        const int t = at0 + i * TILE;
        if (i >= p.count || !on || t >= p.sp.hi || t + a.box <= p.sp.lo) return a.n_pages;
        const int page = a.table[(long long)p.sp.trow * a.table_stride + t / a.page_size];
        if ((unsigned)page < (unsigned)a.n_pages) return page;
        if (mine == 0) report(a.status, MK_ERR_PAGES, PO_TREE, p.r, page);
        return -1;
      };
      auto copy = [&](const CUtensorMap* map, int i, int page) {
        const int s = loads % ST;
        if (!wait_phase(&st->empty[s], (loads / ST & 1) ^ 1, &st->abort)) return false;
        if (lane == 0) mbar_arrive_expect_tx(&st->full[s], SH::kStage);
        __syncwarp();
        const uint32_t dst = smem_addr(s_kv + s * SH::kStage) + mine * TILE * 128 + lane % boxes * a.box * 128;
        if (on)
          tma_box_4d(dst, map, 64 * mine, page < 0 || page >= a.n_pages ? 0 : (at0 + i * TILE) % a.page_size, p.head,
                     page < 0 ? a.n_pages : page, &st->full[s]);
        ++loads;
        return true;
      };
      auto note = [&](int page) {          // the groups of 16 slots of a tile on a bad page
        unsigned bad = on && mine == 0 && page < 0 ? ((1u << (a.box / 16)) - 1) << (lane % boxes * (a.box / 16)) : 0u;
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (lane == 0) st->bad[tiles % 16] = (unsigned char)bad;
        __syncwarp();
        ++tiles;
      };
      int now = page_of(0), ahead = page_of(1);
      note(now);
      run = copy(&k_map, 0, now);
      for (int i = 0; i < p.count && run; ++i) {
        const int later = page_of(i + 2);
        if (PAIR) run = copy(&v_map, i, now);
        if (run && i + 1 < p.count) {
          note(ahead);
          run = copy(&k_map, i + 1, ahead);
        }
        if (!PAIR && run) run = copy(&v_map, i, now);
        now = ahead;
        ahead = later;
      }
    }
    // every copy has landed before the CTA ends
    for (unsigned i = loads > ST ? loads - ST : 0; i < loads; ++i) wait_phase(&st->full[i % ST], i / ST & 1, &st->abort);
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t q0 = smem_addr(s_q), kv0 = smem_addr(s_kv);
      unsigned p_count[2] = {0, 0}, pieces = 0;
      while (next_piece<TILE>(a, w, p)) {
        const int n = PAIR ? 2 * p.count : p.count;
        auto k_load = [&](int i) { return loads + (PAIR ? 2 * i : i == 0 ? 0 : 2 * i - 1); };
        auto v_load = [&](int i) { return loads + (PAIR ? 2 * i + 1 : i + 1 < p.count ? 2 * i + 2 : 2 * p.count - 1); };
        wait_phase(&st->q_full, pieces & 1, &st->abort);
        ++pieces;
        tmem_fence_after();
        auto scores = [&](int x) {
          const int i = PAIR ? x >> 1 : x, g = x & 1;
          const unsigned l = k_load(i), s = l % ST;
          wait_phase(&st->full[s], l / ST & 1, &st->abort);
          tmem_fence_after();
          const uint32_t d = tmem + g * 256, kb = kv0 + s * SH::kStage, qb = q0 + (PAIR ? g : 0) * NQ * SH::kQPart;
#pragma unroll
          for (int y = 0; y < NQ; ++y)
#pragma unroll
            for (int c = 0; c < HD / 16; ++c)
              mma_ss(d, smem_desc(qb + y * SH::kQPart + (c >> 2) * kRows * 128 + (c & 3) * 32, 16, 1024),
                     smem_desc(kb + (c >> 2) * TILE * 128 + (c & 3) * 32, 16, 1024), mma_desc(kType, false, kRows, TILE), y + c > 0);
          mma_commit(&st->s_full[g]);
          if (!PAIR || g == 1) mma_commit(&st->empty[s]);
        };
        auto values = [&](int x) {
          const int i = PAIR ? x >> 1 : x, g = x & 1;
          const unsigned l = v_load(i), s = l % ST;
          wait_phase(&st->full[s], l / ST & 1, &st->abort);
          wait_phase(&st->p_full[g], p_count[g]++ & 1, &st->abort);
          tmem_fence_after();
          const uint32_t d = tmem + g * 256 + 128, pa = tmem + g * 256, vb = kv0 + s * SH::kStage;
#pragma unroll
          for (int y = 0; y < NP; ++y)
#pragma unroll
            for (int c = 0; c < TILE / 16; ++c)
              mma_ts(d, pa + y * (TILE / 2) + c * 8, smem_desc(vb + c * 2048, TILE * 128, 1024), mma_desc(kType, true, kRows, HD), true);
          mma_commit(&st->o_done[g]);
          if (!PAIR || g == 1) mma_commit(&st->empty[s]);
        };
        scores(0);
        if (n > 1) scores(1);
        for (int x = 0; x < n; ++x) {
          values(x);
          if (x + 2 < n) scores(x + 2);
        }
        loads += 2 * p.count;
      }
      mma_commit(&st->finished);
      wait_phase(&st->finished, 0, &st->abort);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMoreRegs));
    // ------------------------------------------------------------------------ softmax
    const int g = warp >> 2, row = tid & (kGroupThreads - 1);  // warpgroup, row of its block
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;         // this warp's lanes of the tensor memory
    const uint32_t t_s = tmem + g * 256 + lanes, t_o = t_s + 128;
    const int block = PAIR ? 2 * part + g : part;
    const int node = block * a.nodes_per_block + row / a.group, h = row % a.group;
    const bool valid = row < a.nodes_per_block * a.group && node < a.n_nodes;
    const bool warp_valid = __any_sync(0xffffffffu, valid);
    unsigned tiles = 0, mine = 0;         // tiles of the CTA, and of this warpgroup
    int row_of = -1;                      // whose tree `seen` is of
    unsigned seen[4] = {0, 0, 0, 0};
    int depth = 0;
    bool there = false;
    while (next_piece<TILE>(a, w, p)) {
      groups_sync();                      // what the last piece left in shared and tensor memory was read
      if (p.r != row_of)
        for (int i = tid; i < a.n_nodes; i += 2 * kGroupThreads) st->parents[i] = a.parents[(long long)p.r * a.n_nodes + i];
      // ---- the queries, K-major, 128-byte swizzled
      if (PAIR || g == 0) {
        const Q* src = static_cast<const Q*>(a.q) + p.r * a.q_row + node * a.q_node + (long long)(p.head * a.group + h) * a.q_head;
        unsigned char* dst = s_q + (PAIR ? g : 0) * NQ * SH::kQPart + row * 128;
        constexpr bool SCALED = kScaled<C, Q>;
        float up = a.q_sign;
        if (SCALED) {
          float most = 0.f;
          if (valid)
#pragma unroll 4
            for (int c = 0; c < HD / 8; ++c) {
              Raw8<Q> raw;
              if (a.q_vec)
                raw.load(src + 8 * c);
              else
                raw.gather(src + 8 * c);
              float v[8];
              raw.up(v);
#pragma unroll
              for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
            }
          const int shift = shift_of(most);
          up *= power_of(shift);
          st->scale[PAIR ? g : 0][row] = a.scale * power_of(-shift);
        }
#pragma unroll 4
        for (int c = 0; c < HD / 8; ++c) {
          Raw8<Q> raw = {};
          if (valid) {
            if (a.q_vec)
              raw.load(src + 8 * c);
            else
              raw.gather(src + 8 * c);
          }
          float v[8];
          raw.up(v);
          uint32_t x[4][NQ];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            split2<C, NQ>(valid ? v[2 * e] * up : 0.f, valid ? v[2 * e + 1] * up : 0.f, x[e]);
#pragma unroll
          for (int y = 0; y < NQ; ++y)
            *reinterpret_cast<uint4*>(dst + y * SH::kQPart + (c >> 3) * kRows * 128 + (((c & 7) ^ (row & 7)) << 4)) =
                make_uint4(x[0][y], x[1][y], x[2][y], x[3][y]);
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
      fence_proxy_async();
      tmem_fence_before();
      mbar_arrive(&st->q_full);
      groups_sync();                      // parents and scales are there
      const float scale = kScaled<C, Q> ? st->scale[PAIR ? g : 0][row] : a.scale;
      if (p.r != row_of) {                // the node's ancestors that its window holds
        row_of = p.r;
#pragma unroll
        for (int i = 0; i < 4; ++i) seen[i] = 0;
        depth = 0;
        there = valid;
        for (int i = node; there;) {
          if (a.window == 0 || depth < a.window)
#pragma unroll
            for (int x = 0; x < 4; ++x) seen[x] |= (i >> 5) == x ? 1u << (i & 31) : 0u;
          const int up = st->parents[i];
          if (up == -1) break;
          there = up >= 0 && up < i;
          i = up;
          ++depth;
        }
        if (!there)
#pragma unroll
          for (int i = 0; i < 4; ++i) seen[i] = 0;
      }
      // the first position that a node of so many ancestors sees (lengths up to 2^31 - 1)
      auto from = [&](int up) {
        const unsigned end = (unsigned)p.sp.len + 1u + (unsigned)up;
        return a.window > 0 && end > (unsigned)a.window ? (int)min(end - (unsigned)a.window, 0x7fffffffu) : 0;
      };
      const int lo = there ? from(depth) : p.sp.len;
      const int plain_lo = from(a.n_nodes - 1);  // tiles in [plain_lo, len) are seen by all nodes whole
      float m = -INFINITY, l = 0.f;
      for (int i = PAIR ? 0 : g; i < p.count; i += PAIR ? 1 : 2) {
        const int t0 = (p.sp.t0 + p.first + i) * TILE;
        wait_phase(&st->s_full[g], mine & 1, &st->abort);
        tmem_fence_after();
        const unsigned bad_tile = *(volatile unsigned char*)&st->bad[(tiles + i) % 16];
        const bool partial = t0 < plain_lo || t0 + TILE > min(p.sp.len, p.sp.hi) || bad_tile != 0;
        unsigned vis[WORDS];
        if (partial) {
#pragma unroll
          for (int x = 0; x < WORDS; ++x) {
            const int b = t0 + 32 * x;
            vis[x] = ones(lo - b, p.sp.len - b) | bits_at(seen, b - p.sp.len);
            vis[x] &= ones(0, p.sp.hi - b);
            if (bad_tile >> (2 * x) & 1) vis[x] &= 0xffff0000u;
            if (bad_tile >> (2 * x) & 2) vis[x] &= 0x0000ffffu;
          }
          // values that are not finite must not meet the zero of one who does not see them: they are taken
          // out of the tile and added for those who do
          if (row < 4) st->odd[PAIR ? i & 1 : g][row] = 0;
          tile_sync<PAIR>(g);
          const unsigned v_at = loads + (PAIR ? 2 * i + 1 : i + 1 < p.count ? 2 * i + 2 : 2 * p.count - 1);
          wait_phase(&st->full[v_at % ST], v_at / ST & 1, &st->abort);
          uint4* v = reinterpret_cast<uint4*>(s_kv + v_at % ST * SH::kStage);
          constexpr int step = PAIR ? 2 * kGroupThreads : kGroupThreads;
          for (int x = PAIR ? tid : row; x < SH::kStage / 16; x += step) {
            uint4 y = v[x];
            const uint32_t o0 = odd_mask<C>(y.x), o1 = odd_mask<C>(y.y), o2 = odd_mask<C>(y.z), o3 = odd_mask<C>(y.w);
            if (o0 | o1 | o2 | o3) {
              v[x] = make_uint4(y.x & ~o0, y.y & ~o1, y.z & ~o2, y.w & ~o3);
              const int slot = x / 8 % TILE;
              atomicOr(&st->odd[PAIR ? i & 1 : g][slot >> 5], 1u << (slot & 31));
            }
          }
          fence_proxy_async();
          tile_sync<PAIR>(g);
        }
        if (warp_valid) {
          float factor = scale;
          if (a.softcap > 0.f) {
            factor = 1.f;
#pragma unroll 1
            for (int x = 0; x < TILE / 16; ++x) {
              uint32_t y[16];
              tmem_ld(t_s + 16 * x, y);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(a.softcap * tanhf(__uint_as_float(y[e]) * scale));
              tmem_st(t_s + 16 * x, y);
            }
            tmem_wait_st();
          }
          uint32_t s[WORDS][32];
#pragma unroll
          for (int x = 0; x < WORDS; ++x) tmem_ld(t_s + 32 * x, s[x]);
          tmem_wait_ld();
          if (partial) {
#pragma unroll
            for (int x = 0; x < WORDS; ++x)
#pragma unroll
              for (int y = 0; y < 32; ++y) s[x][y] = vis[x] >> y & 1 ? s[x][y] : 0xff800000u;
          }
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int x = 0; x < TILE; ++x) tops[x & 3] = fmaxf(tops[x & 3], __uint_as_float(s[x >> 5][x & 31]));
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * factor;
          // what was summed under a smaller maximum is brought to the new one, where it is much smaller
          const bool grown = top > m + kSlack<C>;
          const float to = grown ? top : m;
          if (__any_sync(0xffffffffu, grown && m > -INFINITY)) {
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
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < WORDS; ++b) {
            uint32_t parts[NP][16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float p0 = ex2(fmaf(__uint_as_float(s[b][2 * x]), factor, less));
              const float p1 = ex2(fmaf(__uint_as_float(s[b][2 * x + 1]), factor, less));
              sum[2 * (x & 1)] += p0;
              sum[2 * (x & 1) + 1] += p1;
              uint32_t y[NP];
              split2<C, NP>(p0, p1, y);
#pragma unroll
              for (int z = 0; z < NP; ++z) parts[z][x] = y[z];
            }
#pragma unroll
            for (int z = 0; z < NP; ++z) tmem_st(t_s + z * (TILE / 2) + 16 * b, parts[z]);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
          if (partial) {
#pragma unroll 1
            for (int x = 0; x < TILE; ++x) {
              if (!(st->odd[PAIR ? i & 1 : g][x >> 5] >> (x & 31) & 1)) continue;
              unsigned word = 0;
#pragma unroll
              for (int y = 0; y < WORDS; ++y) word = (x >> 5) == y ? vis[y] : word;
              const bool sees = word >> (x & 31) & 1;
              if (!__any_sync(0xffffffffu, sees)) continue;
              const int t = t0 + x;
              int page = -1;
              if (t < p.sp.hi) page = a.table[(long long)p.sp.trow * a.table_stride + t / a.page_size];
              if ((unsigned)page >= (unsigned)a.n_pages) continue;
              const C* src = static_cast<const C*>(a.v) + (long long)page * a.page_stride +
                             ((long long)p.head * a.page_size + t % a.page_size) * HD;
              float pr = 0.f;
#pragma unroll
              for (int z = 0; z < NP; ++z) {
                const uint32_t y = tmem_ld1(t_s + z * (TILE / 2) + (x >> 1));
                tmem_wait_ld();
                const float2 both = unpack2<C>(y);
                pr += x & 1 ? both.y : both.x;
              }
              for (int c = 0; c < HD / 32; ++c) {
                uint32_t o[32];
                tmem_ld(t_o + 32 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; ++y) {
                  const float v = Conv<C>::up(src[32 * c + y]);
                  if (sees && !(fabsf(v) < INFINITY)) o[y] = __float_as_uint(fmaf(pr, v, __uint_as_float(o[y])));
                }
                tmem_st(t_o + 32 * c, o);
                tmem_wait_st();
              }
            }
          }
        }
        tmem_fence_before();
        mbar_arrive(&st->p_full[g]);
        ++mine;
      }
      if (mine) wait_phase(&st->o_done[g], (mine - 1) & 1, &st->abort);
      tiles += p.count;
      loads += 2 * p.count;
      // ---- the piece's result
      if (!there) {                       // (an absent node's row went through the whole tiles with the others)
        m = -INFINITY;
        l = 0.f;
      }
      if (!PAIR) {
        st->ml[g][row][0] = m;
        st->ml[g][row][1] = l;
        tmem_fence_before();
        groups_sync();
      }
      tmem_fence_after();
      if (!warp_valid) continue;
      float M = m, L = l, f0 = 1.f, f1 = 0.f;
      if (!PAIR) {
        const float m0 = st->ml[0][row][0], m1 = st->ml[1][row][0];
        M = fmaxf(m0, m1);
        const float Ms = M == -INFINITY ? 0.f : M;
        f0 = ex2(m0 - Ms);
        f1 = ex2(m1 - Ms);
        L = fmaf(f0, st->ml[0][row][1], f1 * st->ml[1][row][1]);
      }
      const float Ms = M == -INFINITY ? 0.f : M;
      const long long at = ((long long)p.r * a.n_nodes + node) * a.hq + p.head * a.group + h;
      Q* dst = static_cast<Q*>(a.out) + p.r * a.o_row + node * a.o_node + (long long)(p.head * a.group + h) * a.o_head;
      const int slot = p.first == 0;      // 0: continues a segment, 1: begins one
      float* keep = a.part + (((size_t)blockIdx.x * 2 + slot) * a.part_rows + (PAIR ? g : 0) * kRows + row) * (HD + 4);
      const float inv = L == 0.f ? 0.f : 1.f / L;
      constexpr int CHUNKS = PAIR ? HD / 32 : HD / 64;  // of this thread: all of the dims, or the warpgroup's half
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int d = 32 * ((PAIR ? 0 : g * CHUNKS) + c);
        uint32_t o[32];
        if (PAIR) {
          tmem_ld(t_o + d, o);
          tmem_wait_ld();
        } else {
          uint32_t o1[32];
          tmem_ld(tmem + lanes + 128 + d, o);
          tmem_ld(tmem + lanes + 256 + 128 + d, o1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(fmaf(f0, __uint_as_float(o[e]), f1 * __uint_as_float(o1[e])));
        }
        if (!valid) continue;
        if (p.whole) {
          float x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = L == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
          if (a.o_vec) {
#pragma unroll
            for (int e = 0; e < 4; ++e) store8<Q>(dst + d + 8 * e, *reinterpret_cast<const float(*)[8]>(x + 8 * e));
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) dst[d + e] = Conv<Q>::down(x[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) reinterpret_cast<uint4*>(keep + d)[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (valid && (PAIR || g == 0)) {
        if (p.whole) {
          if (a.lse) a.lse[at] = (Ms - kShift<C> + log2f(L)) * kLn2;
        } else {
          keep[HD] = M;
          keep[HD + 1] = L;
        }
      }
      if (tid == 0 && !p.whole && p.first == 0) a.joins[blockIdx.x] = make_int4(share, p.last_share, p.r, p.head);
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (tid == 0 && st->abort) report(a.status, MK_ERR_TIMEOUT, PO_TREE, -1, blockIdx.x);
  if (warp == kMmaWarp) tmem_free_all(tmem);
}

// Joins the pieces of the segments that span CTAs: a warp per row of a block, a lane HD / 32 dims.
template <typename Q, int HD>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeArgs a, float shift) {
  constexpr int E = HD / 32, ROW = HD + 4, U = 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch();
  const int4 job = a.joins[blockIdx.x];
  const int part = blockIdx.x % a.parts, row = blockIdx.y * (kJoinThreads / 32) + warp;
  if (job.y < 0 || row >= a.part_rows) return;
  const int per = a.part_rows > kRows ? 2 : 1, block = part * per + row / kRows, x = row % kRows;
  const int node = block * a.nodes_per_block + x / a.group, head = job.w * a.group + x % a.group, r = job.z;
  if (x >= a.nodes_per_block * a.group || node >= a.n_nodes) return;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int b = job.x; b <= job.y; b += U) {
    float pm[U], pl[U], po[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int y = min(b + u, job.y);     // past the last: loaded and not used
      const float* src = a.part + (((size_t)(y * a.parts + part) * 2 + (y == job.x)) * a.part_rows + row) * ROW;
#pragma unroll
      for (int e = 0; e < E; ++e) po[u][e] = src[32 * e + lane];
      pm[u] = src[HD];
      pl[u] = src[HD + 1];
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
  Q* out = static_cast<Q*>(a.out) + r * a.o_row + node * a.o_node + head * a.o_head;
#pragma unroll
  for (int e = 0; e < E; ++e) out[32 * e + lane] = Conv<Q>::down(l == 0.f ? 0.f : o[e] / l);
  if (lane == 0 && a.lse)
    a.lse[((long long)r * a.n_nodes + node) * a.hq + head] = ((m == -INFINITY ? 0.f : m) - shift + log2f(l)) * kLn2;
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
  int nodes_per_block, blocks, parts, part_rows;
  bool pair;
};
Deal deal(int n_nodes, int group, bool same_type) {
  Deal d;
  d.nodes_per_block = kRows / group;
  d.blocks = (n_nodes + d.nodes_per_block - 1) / d.nodes_per_block;
  d.pair = same_type && d.blocks > 1;
  d.parts = d.pair ? (d.blocks + 1) / 2 : d.blocks;
  d.part_rows = d.pair ? 2 * kRows : d.blocks > 1 ? kRows : n_nodes * group;
  return d;
}

template <typename C, typename Q, int HD, int NQ, int NP, bool PAIR>
mk_status launch_tree(TreeArgs& a, const mk_page_view& view, void* stream) {
  using SH = Shape<C, HD, NQ, NP, PAIR>;
  a.box = 16;
  while (a.box < SH::TILE && a.page_size % (2 * a.box) == 0) a.box *= 2;
  CUtensorMap k_map, v_map;
  mk_status s = page_map(&k_map, view, view.k, a.box);
  if (!s) s = page_map(&v_map, view, view.v, a.box);
  if (s) return s;
  auto kernel = tree_kernel<C, Q, HD, NQ, NP, PAIR>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::kBytes);
  if (e != cudaSuccess) return paged_fail(MK_ERR_CUDA, std::string("mk_tree_attention: ") + cudaGetErrorString(e));
  s = launch_dependent(kernel, dim3(a.shares * a.parts), dim3(kTreeThreads), SH::kBytes, stream, "mk_tree_attention", a, k_map, v_map);
  if (s) return s;
  const int per = kJoinThreads / 32;
  return launch_dependent(tree_join_kernel<Q, HD>, dim3(a.shares * a.parts, (a.part_rows + per - 1) / per), dim3(kJoinThreads), 0,
                          stream, "mk_tree_attention (join)", a, kShift<C>);
}
template <typename C, typename Q, int NQ, int NP>
mk_status launch_tree(TreeArgs& a, const mk_page_view& view, bool pair, void* stream) {
  if constexpr (NQ == 1) {
    if (pair)
      return view.head_dim == 64 ? launch_tree<C, Q, 64, NQ, NP, true>(a, view, stream)
                                 : launch_tree<C, Q, 128, NQ, NP, true>(a, view, stream);
  }
  return view.head_dim == 64 ? launch_tree<C, Q, 64, NQ, NP, false>(a, view, stream)
                             : launch_tree<C, Q, 128, NQ, NP, false>(a, view, stream);
}

}  // namespace
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
    size_t rows = 0;
    for (bool same : {false, true}) rows = std::max<size_t>(rows, deal(n_nodes, n_heads / n_kv_heads, same).part_rows);
    *bytes = (size_t)n_sm * (sizeof(int4) + 2 * rows * (head_dim + 4) * sizeof(float));
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
    const float factor = args->softcap > 0.f ? args->scale / args->softcap : args->scale * kLog2e;
    if (!(args->softcap >= 0.f && args->softcap * kLog2e < INFINITY) || !(std::abs(factor) < INFINITY))
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
    const long long most = (args->window > 0 ? std::min(cap, (long long)args->window + kMaxNodes + 64) : cap) / 64 + 2 + kLead;
    if (most * rn > 0x7f000000LL / cache->n_kv_heads)
      return paged_fail(MK_ERR_INVALID, "n_rows * n_kv_heads * (the table's positions / 64 + 4) must be below 2^31 - 2^24");
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
    const Deal d = deal(a.n_nodes, a.group, args->dtype == cache->dtype);
    a.nodes_per_block = d.nodes_per_block; a.blocks = d.blocks; a.parts = d.parts; a.part_rows = d.part_rows;
    a.shares = std::max(1, n_sm / d.parts);
    a.joins = static_cast<int4*>(args->workspace);
    a.part = reinterpret_cast<float*>(a.joins + n_sm);
    const long long per = 16 / (long long)esz;
    a.q_vec = aligned_to(a.q, 16) && a.q_row % per == 0 && a.q_node % per == 0 && a.q_head % per == 0;
    a.o_vec = aligned_to(a.out, 16) && a.o_row % per == 0 && a.o_node % per == 0 && a.o_head % per == 0;
    a.scale = factor == 0.f ? 1.f : std::abs(factor);
    a.q_sign = factor == 0.f ? 0.f : factor < 0.f ? -1.f : 1.f;
    a.softcap = args->softcap * kLog2e;
    // 16-bit queries of the cache's type are exact in one part, others are split into 2 parts of fp16 (22
    // bits, each head at a power of two of its own) or 3 of bf16 (24 bits).  A probability has one part where the
    // outputs have 16 bits, and 2 of fp16 or 3 of bf16 where they have 32.
    if (cache->dtype == MK_F16) {
      if (args->dtype == MK_F16) return launch_tree<__half, __half, 1, 1>(a, *cache, d.pair, stream);
      if (args->dtype == MK_BF16) return launch_tree<__half, __nv_bfloat16, 2, 1>(a, *cache, d.pair, stream);
      return launch_tree<__half, float, 2, 2>(a, *cache, d.pair, stream);
    }
    if (args->dtype == MK_BF16) return launch_tree<__nv_bfloat16, __nv_bfloat16, 1, 1>(a, *cache, d.pair, stream);
    if (args->dtype == MK_F16) return launch_tree<__nv_bfloat16, __half, 2, 1>(a, *cache, d.pair, stream);
    return launch_tree<__nv_bfloat16, float, 3, 3>(a, *cache, d.pair, stream);
  });
}
