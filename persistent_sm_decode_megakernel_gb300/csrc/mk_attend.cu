// Attention of one new token per row over a paged KV cache (mk_paged_attention).
//
// The rows' positions are cut into tiles of 16 (a tile lies in one page).  The segments
// (row, kv head), each of its row's tiles, follow one another in one line of work, and every
// CTA of a single wave takes an equal, contiguous share of that line: batches of any raggedness
// load the SMs evenly, and one long sequence is split over all of them.  A segment that lies
// in one CTA is finished there; the pieces of one that spans CTAs go to the workspace as
// (running maximum, sum, weighted values) and a second small kernel joins them in order:
//   M = max M_i,  L = sum L_i 2^(M_i - M),  out = sum O_i 2^(M_i - M) / L.
#include <algorithm>
#include <type_traits>

#include "mk_internal.h"
#include "mk_device.cuh"
#include "mk_paged.cuh"

namespace mk {
namespace {

constexpr int kTile = 16;               // positions per tile: the k extent of the value product
constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
// CTAs of one wave per SM: 168 registers a thread at 128 dims, 128 at 64
constexpr int ctas_per_sm(int hd) { return hd == 128 ? 3 : 4; }
constexpr int kJoinThreads = 256;
constexpr int kMaxGroup = 16;           // query heads per kv head
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

struct AttendArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  float* part;                          // [n_cta][2][heads of a group][HD + 4]
  int4* joins;                          // [n_cta] what to join: first and last CTA, row, kv head
  const int32_t *lens, *rows, *table;
  int32_t* status;
  long long q_row, q_head, o_row, o_head, page_stride, table_stride;
  int n_rows, hq, hkv, group, len_add, window, page_size, n_pages, table_rows, cap;  // cap: positions of a table row
  int tpp;                              // tiles per page
  unsigned tpp_inverse;                 // 2^32 / tpp, rounded up
  int n_cta;
  int q_vec;                            // q in accesses of 16 bytes
  int by_segment;                       // joins[row * hkv + kv head] (they fit), else joins[first CTA]
  float scale, softcap;                 // scores to units of log 2: scale s, or softcap tanh(scale s)
};

// The span of a row: positions [lo, hi) and their tiles [t0, t0 + n).
struct Span {
  int lo, hi, t0, n, trow;
};
__device__ __forceinline__ int length_of(const AttendArgs& a, int r) {
  int len;
  asm("add.sat.s32 %0, %1, %2;" : "=r"(len) : "r"(a.lens[r]), "r"(a.len_add));
  return len;
}
__device__ __forceinline__ Span span_of(const AttendArgs& a, int r) {
  Span s;
  s.trow = a.rows ? a.rows[r] : r;
  const int len = (unsigned)s.trow < (unsigned)a.table_rows ? max(0, length_of(a, r)) : 0;
  // the window counts from the row's own end, also where the table ends earlier
  s.hi = min(len, a.cap);
  s.lo = a.window > 0 ? min(max(0, len - a.window), s.hi) : 0;
  s.t0 = s.lo / kTile;
  s.n = s.hi > s.lo ? (s.hi + kTile - 1) / kTile - s.t0 : 0;
  return s;
}
// Rows that have no row of the table, and lengths beyond it, are reported.
__device__ __noinline__ void check_rows(const AttendArgs& a) {
  for (int r = threadIdx.x; r < a.n_rows; r += kAttThreads) {
    const int len = length_of(a, r), trow = a.rows ? a.rows[r] : r;
    if ((unsigned)trow >= (unsigned)a.table_rows) {
      if (len > 0) report(a.status, MK_ERR_PAGES, PO_ATTEND, r, trow);
    } else if (len > a.cap) {
      report(a.status, MK_ERR_PAGES, PO_ATTEND, r, len);
    }
  }
}
// Rows without positions: zeros.
template <typename Q>
__device__ __noinline__ void fill_rows(const AttendArgs& a, int hd) {
  for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
    if (span_of(a, r).n != 0) continue;
    for (int x = threadIdx.x; x < a.hq * hd; x += kAttThreads)
      static_cast<Q*>(a.out)[(long long)r * a.o_row + (long long)(x / hd) * a.o_head + x % hd] = Conv<Q>::down(0.f);
    for (int h = threadIdx.x; h < a.hq; h += kAttThreads) {
      if (a.lse) a.lse[(long long)r * a.hq + h] = -INFINITY;
      if (a.by_segment && h < a.hkv) a.joins[r * a.hkv + h] = make_int4(0, -1, 0, 0);
    }
  }
}

// The line of work, in units: every segment counts its tiles and `lead` units in front of them
// for what a piece costs besides its tiles (the query, the table, the merge).  CTA c takes
// [c share, (c + 1) share).  Of what a CTA takes, a segment's lead is where it begins: the
// segment's first tiles are of the CTA that holds their units, whoever holds the lead.
//   lead: with fewer tiles than the wave's warps the latency of a piece is all there is, and
//     equal tiles are best; else kLead, without which a CTA that meets a dozen segments of two
//     tiles each ran twice as long as the others (61 ragged rows of up to 700 positions).
//   pitch: the units of every segment, its lead being what its tiles leave, so that each is
//     whole in a CTA of its own; 0: n + lead.  Taken when there is a CTA for each and the longest is
//     no longer than an equal share and the lead that a second piece would add (61 ragged rows
//     of up to 700 positions: 13.7 us; in equal shares 1.1 more).
constexpr int kLead = 8;
struct Line {
  int units, share, lead, pitch;
  bool gaps;  // rows without positions
};
__device__ __forceinline__ int segment_units(int n, int lead, int pitch) { return pitch ? pitch : n + lead; }
__device__ __forceinline__ int row_units(const AttendArgs& a, int n, int lead, int pitch) {
  return n > 0 ? segment_units(n, lead, pitch) * a.hkv : 0;
}
// The line, and in *row and *before (shared memory; the caller syncs) the row that holds this
// CTA's first unit and the units before it.  What stands before the first load is as short as
// it can be, all of it in 32 bits (the host refuses longer lines): executed once, it waits for
// its instructions, 7 cycles for each.
__device__ __forceinline__ Line find_row(const AttendArgs& a, int (*sums)[3], int* row, int* before) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_rows + kAttThreads - 1) / kAttThreads;
  const int r0 = min(a.n_rows, tid * per), r1 = min(a.n_rows, r0 + per);
  int tiles = 0, rows = 0, most = 0;  // rows: with positions; most: the longest
  for (int r = r0; r < r1; ++r) {
    const int n = span_of(a, r).n;
    tiles += n;
    rows += n > 0;
    most = max(most, n);
  }
  int ti = tiles, ri = rows;
  most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, ti, o), y = __shfl_up_sync(0xffffffffu, ri, o);
    if (lane >= o) {
      ti += x;
      ri += y;
    }
  }
  if (lane == 31) {
    sums[warp][0] = ti;
    sums[warp][1] = ri;
    sums[warp][2] = most;
  }
  __syncthreads();
  ti -= tiles;  // before this thread's rows
  ri -= rows;
  int all_tiles = 0, all_rows = 0;
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) {
    const int x = sums[w][0], y = sums[w][1];
    ti += w < warp ? x : 0;
    ri += w < warp ? y : 0;
    all_tiles += x;
    all_rows += y;
    most = max(most, sums[w][2]);
  }
  Line l;
  const int segments = all_rows * a.hkv;
  l.lead = all_tiles * a.hkv <= a.n_cta * kAttWarps ? 0 : kLead;
  l.units = all_tiles * a.hkv + segments * l.lead;
  l.share = max(kAttWarps, (int)((unsigned)(l.units + a.n_cta - 1) / (unsigned)a.n_cta));
  l.gaps = all_rows < a.n_rows;
  l.pitch = 0;
  if (l.lead && segments <= a.n_cta && most <= l.share + kLead) {
    l.pitch = most;
    l.share = most;
    l.units = segments * most;
  }
  auto units = [&](int tiles, int rows) { return (l.pitch ? rows * l.pitch : tiles + rows * l.lead) * a.hkv; };
  const int at = min(l.units, l.share * (int)blockIdx.x);  // (n_cta shares pass the line by less than 2^20)
  int b = units(ti, ri);
  if (at >= b && at < b + units(tiles, rows))
    for (int r = r0; r < r1; ++r) {
      const int n = row_units(a, per == 1 ? tiles : span_of(a, r).n, l.lead, l.pitch);
      if (at >= b && at < b + n) {
        *row = r;
        *before = b;
      }
      b += n;
    }
  return l;
}

// the page a tile lies in: t / tpp by a multiplication (exact for t <= 2^26, tpp <= 64)
__device__ __forceinline__ int page_index(const AttendArgs& a, int t) {
  return a.tpp == 1 ? t : (int)__umulhi((unsigned)t, a.tpp_inverse);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
// two floats as PARTS packed pairs whose sums are the floats: each part is the rest rounded
template <typename T, int PARTS>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    p[i] = pack2<T>(x, y);
    const float2 r = unpack2<T>(p[i]);
    x -= r.x;
    y -= r.y;
  }
}

// fp16 probabilities are held times 2^14 so that small ones stay normal numbers; bf16 has
// the range of fp32
template <typename T>
constexpr float kProbShift = 0.f;
template <>
constexpr float kProbShift<__half> = 14.f;

// A query that is split into fp16 parts is first brought near the top of their range, every head
// by a power of two of its own (2^shift times its largest element lies in [2^14, 2^15)) that the
// score's factor takes back: else the second part of an element below 1/8 was a subnormal
// number, and one below 2^-25 or above 65504 lost altogether.
template <typename C, typename Q>
constexpr bool kScaled = std::is_same<C, __half>::value && !std::is_same<Q, __half>::value;
__device__ __forceinline__ int shift_of(float largest) {
  const int e = __float_as_int(largest) >> 23;  // (largest >= 0; zeros, infinities and NaN stay as they are)
  return e == 0 || e == 255 ? 0 : min(127 + 14 - e, 126);
}
__device__ __forceinline__ float power_of(int e) { return __int_as_float((127 + e) << 23); }  // 2^e, |e| <= 126

// four bytes from global to shared memory, without a register between
__device__ __forceinline__ void cp_async4(int* dst, const int* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// 2^x by the hardware's approximation (2 ulp; results below the normal range become 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared memory of the kernel: the query as A fragments [part][32-dim chunk][32 lanes][16 B]
// (WIDE: [part][chunk][2 row halves][32 lanes]), then the warps' partials for the CTA's merge.
struct AttState {
  const int32_t* table;        // the row's pages
  int at, end, share, before;  // next unit, end of the CTA's units, share; units before `row`
  int sums[kAttWarps][3];
  int row, head, slot, lead, pitch, bad, bad_page;
  float scale[kMaxGroup];      // kScaled: a head's factor from products to scores
  int pages[kAttWarps][64];    // of a warp's tiles: the k-th one's at k mod 64
};
template <int HD, bool WIDE, int NQ>
struct AttSmem {
  static constexpr int kHeads = WIDE ? 16 : 8;
  static constexpr int kQBytes = NQ * (HD / 32) * (WIDE ? 2 : 1) * 32 * 16;
  static constexpr int kRow = HD + 4;                        // floats per head of a partial
  static constexpr int kPartFloats = kAttWarps * kHeads * kRow;
  static constexpr int kMlFloats = kAttWarps * kHeads * 2;
  static constexpr int kBytes = kQBytes + 4 * (kPartFloats + kMlFloats) + (int)sizeof(AttState);
};

// C: the cache's type.  Q: the queries' and outputs' type.  NQ parts of C make up a query
// element, NP a probability.  A tensor-core tile m16n8k16 has 16 rows:
//   WIDE = false (up to 8 heads): row g holds head g's first part, row g + 8 the second; a
//     third part takes a second instruction;
//   WIDE = true (up to 16 heads): a row per head, one instruction per part.
// Keys and values go from global memory straight into the B fragments, without shared memory:
//   scores: the dims of a 32-dim chunk may be summed in any order, so lane (g, c) loads 16
//     bytes -- dims [32 i + 8 c, + 8) of position g -- and uses them as the fragments of two
//     k-steps; the query's fragments take the same order;
//   values: lane (n, c) loads 16 bytes -- dims [64 h + 8 n, + 8) -- of the four positions
//     2c, 2c + 1, 2c + 8, 2c + 9 its score columns stand for; byte permutes pair the
//     positions, and column n of the j-th instruction is dim 64 h + 8 n + j.
// So every load is 16 bytes, a warp's rows are read in whole 64- and 128-byte runs, no
// barrier stands between the loads and the products, and the warps of an SM hide each
// other's latency.  Bound: the keys' and values' bytes (16 rows of 16384 to 32768 positions,
// 1.67 GB: 245 us, 6.8 TB/s), of short rows the chain from the lengths over the table to the
// first keys, 3 us of it, and a tile after another of a warp, 1 us each (one row of 512: 6.7 us
// with the join, one of 32768: 29.2).  The pages of a warp's tiles lie in shared memory and
// come there without a register between: held by the lanes, they cost the long rows 2 %.
template <typename C, typename Q, int HD, bool WIDE, int NQ, int NP>
__global__ void __launch_bounds__(kAttThreads, ctas_per_sm(HD)) attend_kernel(const __grid_constant__ AttendArgs a) {
  using SM = AttSmem<HD, WIDE, NQ>;
  constexpr int CH = HD / 32, VH = HD / 64, HEADS = SM::kHeads, ROW = SM::kRow;
  constexpr int RH = WIDE ? 2 : 1;  // row halves that are heads of their own
  extern __shared__ __align__(16) unsigned char att_smem[];
  uint4* s_q = reinterpret_cast<uint4*>(att_smem);
  float* s_part = reinterpret_cast<float*>(att_smem + SM::kQBytes);
  float* s_ml = s_part + SM::kPartFloats;
  AttState* st = reinterpret_cast<AttState*>(s_ml + SM::kMlFloats);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_launch();
  const Line line = find_row(a, st->sums, &st->row, &st->before);
  if (blockIdx.x == gridDim.x - 1) check_rows(a);
  if (line.gaps) fill_rows<Q>(a, HD);
  if (tid == 0 && !a.by_segment) a.joins[blockIdx.x] = make_int4(0, -1, 0, 0);
  const int begin = line.share * (int)blockIdx.x;
  if (begin >= line.units) return;
  // what a piece needs again at its end lives in shared memory: the loop over the tiles has
  // few registers to spare
  if (tid == 0) {
    st->at = begin;
    st->end = min(line.units, begin + line.share);
    st->share = line.share;
    st->lead = line.lead;
    st->pitch = line.pitch;
    st->bad = 0;
  }
  __syncthreads();
  while (true) {
    int base, cnt, mine, lo, hi;  // this warp's tiles: base, + kAttWarps, ...
    {
      int rbase = st->before, at = st->at, seg;  // seg: the segment's first unit
      int r = st->row, j, first, each;
      Span sp;
      while (true) {
        sp = span_of(a, r);
        const int n = row_units(a, sp.n, st->lead, st->pitch);
        if (at < rbase + n) {
          each = segment_units(sp.n, st->lead, st->pitch);
          const int lead = each - sp.n;
          j = (int)((unsigned)(at - rbase) / (unsigned)each);
          seg = rbase + j * each;
          const int stop = min(st->end, seg + each);
          first = max(0, at - seg - lead);
          cnt = stop - seg - lead - first;  // tiles of this piece
          at = stop;
          if (cnt > 0 || at >= st->end) break;  // (no tiles: of a segment's lead alone)
        } else {
          rbase += n;
          ++r;
        }
      }
      __syncthreads();  // the state is read
      if (cnt <= 0) return;
      if (tid == 0) {
        const bool whole = cnt == sp.n;
        st->row = r;
        st->before = rbase;
        st->head = j;
        st->table = a.table + (long long)sp.trow * a.table_stride;
        st->slot = whole ? 2 : first == 0;  // 0: continues a segment, 1: begins one, 2: is one
        if (first == 0) {  // the segment's begin knows where it ends
          const int last = (int)((unsigned)(seg + each - 1) / (unsigned)st->share);
          if (a.by_segment)
            a.joins[r * a.hkv + j] = whole ? make_int4(0, -1, 0, 0) : make_int4(blockIdx.x, last, r, j);
          else if (!whole)
            a.joins[blockIdx.x] = make_int4(blockIdx.x, last, r, j);
        }
        st->at = at;
      }
      base = sp.t0 + first + warp;
      mine = cnt > warp ? (cnt - warp + kAttWarps - 1) / kAttWarps : 0;
      lo = sp.lo;
      hi = sp.hi;
    }
    __syncthreads();
    // the pages of this warp's first 32 tiles; from then on the next 32 are fetched ahead
    int* pages = st->pages[warp];
    auto entry = [&](int k) { return st->table + page_index(a, base + k * kAttWarps); };
    const int page0 = lane < mine ? *entry(lane) : -1;
    // the query's fragments: chunk i, lane (g, c): dims [32 i + 8 c, + 8) of head g.  Asked for
    // here, stored behind the first keys' loads, which need not wait for them.
    constexpr int kAsk = CH * HEADS * 4 / kAttThreads > 0 ? CH * HEADS * 4 / kAttThreads : 1;
    constexpr bool SCALED = kScaled<C, Q>;  // a head's chunks are then in neighbouring lanes of one warp
    Raw8<Q> ask[kAsk];
#pragma unroll
    for (int z = 0; z < kAsk; ++z) {
      const int y = tid + z * kAttThreads, h = SCALED ? y / (4 * CH) : (y >> 2) % HEADS;
      const int i = SCALED ? (y >> 2) % CH : y / (4 * HEADS);
      const Q* src = static_cast<const Q*>(a.q) + (long long)st->row * a.q_row +
                     (long long)(st->head * a.group + h) * a.q_head + 32 * i + 8 * (y & 3);
      ask[z] = {};
      if (i < CH && h < a.group) {
        if (a.q_vec)
          ask[z].load(src);
        else
          ask[z].gather(src);
      }
    }
    const long long plane = (long long)st->head * a.page_size * HD;  // the kv head's part of a page
    // a tile's offset in the pages, and the positions [p0, p1) of it that count
    long long off;
    int p0, p1;
    auto locate = [&](int k) {
      const int t = base + k * kAttWarps;
      const int page = pages[k & 63];
      p0 = max(0, lo - t * kTile);
      p1 = min(kTile, hi - t * kTile);
      off = (long long)page * a.page_stride + plane + (t - page_index(a, t) * a.tpp) * (kTile * HD);
      if ((unsigned)page >= (unsigned)a.n_pages) {  // its positions are masked, and reported at the end
        st->bad_page = page;
        st->bad = 1;
        p0 = p1 = 0;
        off = 0;
      }
    };
    uint4 kf[2][CH];
    auto load_k = [&]() {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int p = n * 8 + g;
        const C* src = static_cast<const C*>(a.k) + off + p * HD + 8 * c;
        if (p1 - p0 == kTile) {  // a whole tile: nothing to fill in
#pragma unroll
          for (int i = 0; i < CH; ++i) kf[n][i] = ldg_stream(src + 32 * i);
        } else {
#pragma unroll
          for (int i = 0; i < CH; ++i)
            kf[n][i] = p >= p0 && p < p1 ? ldg_stream(src + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    pages[lane] = page0;
    __syncwarp();
    if (mine > 0) {
      locate(0);
      load_k();
    }
#pragma unroll
    for (int z = 0; z < kAsk; ++z) {
      const int y = tid + z * kAttThreads, h = SCALED ? y / (4 * CH) : (y >> 2) % HEADS;
      const int i = SCALED ? (y >> 2) % CH : y / (4 * HEADS);
      if (SCALED ? h >= HEADS : i >= CH) continue;  // (whole warps)
      uint32_t w[4][NQ];
      if constexpr (std::is_same<C, Q>::value) {
        w[0][0] = ask[z].w[0].x;
        w[1][0] = ask[z].w[0].y;
        w[2][0] = ask[z].w[0].z;
        w[3][0] = ask[z].w[0].w;
      } else {
        float v[8];
        ask[z].up(v);
        if constexpr (SCALED) {
          float most = fabsf(v[0]);
#pragma unroll
          for (int e = 1; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
#pragma unroll
          for (int x = 1; x < 4 * CH; x <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
          const int shift = shift_of(most);
          const float up = power_of(shift);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= up;
          if (y % (4 * CH) == 0) st->scale[h] = a.scale * power_of(-shift);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) split2<C, NQ>(v[2 * e], v[2 * e + 1], w[e]);
      }
#pragma unroll
      for (int p = 0; p < NQ; ++p) {
        const int slot = WIDE ? ((p * CH + i) * 2 + (h >> 3)) * 32 : (p * CH + i) * 32;
        s_q[slot + (h & 7) * 4 + (y & 3)] = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
      }
    }
    float o[VH][8][4];
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[h][x][e] = 0.f;
    float m[RH], l[RH];  // row g (WIDE: and row g + 8)
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
    __syncthreads();
    float scale[RH];  // of row g (WIDE: and row g + 8)
#pragma unroll
    for (int h = 0; h < RH; ++h) scale[h] = SCALED ? st->scale[g + 8 * h] : a.scale;
    // The warp's sums of weighted values to shared memory.  The tensor cores truncate what they add
    // up: a sum of n tiles comes out too small, by 2.5e-8 n of itself, or 5e-8 n where the values have one
    // sign (128 rows of 32768 positions, 862 tiles a warp: 4.3e-5).  Where 32-bit outputs show it, it is added every 32 tiles to what lies
    // there, rounded to nearest and brought to the new maximum (below 3.8e-6, in the same time).  Outputs of 16
    // bits round at 2^-12 and 2^-9, and with over 8 heads the registers that it takes cost 15 to 20 %
    // of the time: there the sum stays in the tensor cores.
    constexpr bool FLUSH = std::is_same<Q, float>::value && !WIDE;
    auto flush = [&](bool first) {
#pragma unroll
      for (int h = 0; h < RH; ++h) {
        const int head = g + 8 * h;
        float* ml = s_ml + (warp * HEADS + head) * 2;
        const float ms = m[h] == -INFINITY ? 0.f : m[h], f = first ? 0.f : ex2(ml[0] - ms);
        float* dst = s_part + (warp * HEADS + head) * ROW;
#pragma unroll
        for (int d = 0; d < VH; ++d)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // columns 2c + e: dims 64 d + 16 c + 8 e + y
            float4* p = reinterpret_cast<float4*>(dst + 64 * d + 16 * c + 8 * e);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                w[y] = WIDE ? o[d][4 * q + y][2 * h + e] : o[d][4 * q + y][e] + o[d][4 * q + y][2 + e];
              if (!first) {
                const float4 v = p[q];
                w[0] = fmaf(f, v.x, w[0]);
                w[1] = fmaf(f, v.y, w[1]);
                w[2] = fmaf(f, v.z, w[2]);
                w[3] = fmaf(f, v.w, w[3]);
              }
              p[q] = make_float4(w[0], w[1], w[2], w[3]);
            }
          }
        __syncwarp();
        if (c == 0) ml[0] = m[h];
      }
    };
    for (int k = 0; k < mine; ++k) {
      if ((k & 31) == 0) {
        __syncwarp();  // what is overwritten was read
        if (FLUSH && k > 0) {
          flush(k == 32);
#pragma unroll
          for (int h = 0; h < VH; ++h)
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[h][x][e] = 0.f;
          __syncwarp();
        }
        if (k + 32 + lane < mine) cp_async4(pages + ((k + 32 + lane) & 63), entry(k + 32 + lane));
      }
      const int q0 = p0, q1 = p1;
      // the tile's values: in flight while the scores are computed
      uint4 vf[VH][4];
      const C* src = static_cast<const C*>(a.v) + off + 2 * c * HD + 8 * g;
      if (q1 - q0 == kTile) {
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int h = 0; h < VH; ++h) vf[h][y] = ldg_stream(src + ((y & 1) + 8 * (y >> 1)) * HD + 64 * h);
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int p = 2 * c + (y & 1) + 8 * (y >> 1);
#pragma unroll
          for (int h = 0; h < VH; ++h)
            vf[h][y] = p >= q0 && p < q1 ? ldg_stream(src + ((y & 1) + 8 * (y >> 1)) * HD + 64 * h)
                                         : make_uint4(0u, 0u, 0u, 0u);
        }
      }
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int p = 0; p < NQ; p += WIDE ? 1 : 2) {
          uint4 u, w;  // rows 0..7 and rows 8..15 of the A tile
          if (WIDE) {
            u = s_q[((p * CH + i) * 2) * 32 + lane];
            w = s_q[((p * CH + i) * 2 + 1) * 32 + lane];
          } else {
            u = s_q[(p * CH + i) * 32 + lane];
            w = p + 1 < NQ ? s_q[((p + 1) * CH + i) * 32 + lane] : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            Mma<C>::run(s[n], make_uint4(u.x, w.x, u.y, w.y), kf[n][i].x, kf[n][i].y);
            Mma<C>::run(s[n], make_uint4(u.z, w.z, u.w, w.w), kf[n][i].z, kf[n][i].w);
          }
        }
      }
      // the next tile's keys
      if (k + 1 < mine) {
        if (((k + 1) & 31) == 0) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
        }
        locate(k + 1);
        load_k();
      }
      // ---- softmax of the tile, in units of log 2; lane (g, c): columns 2c, 2c + 1 of each half
      uint32_t ph[RH][2][NP];  // [row half][column half][part]
#pragma unroll
      for (int h = 0; h < RH; ++h) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = s[e >> 1][2 * h + (e & 1)];
          // the second part's row; one part has none, and there 0 times an infinite key is NaN
          if (!WIDE && NQ > 1) y += s[e >> 1][2 + (e & 1)];
          x[e] = y * scale[h];
        }
        if (a.softcap > 0.f) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = a.softcap * tanhf(x[e]);
        }
        if (q1 - q0 != kTile) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int p = 2 * c + (e & 1) + 8 * (e >> 1);
            if (p < q0 || p >= q1) x[e] = -INFINITY;
          }
        }
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[h], top), ms = mn == -INFINITY ? 0.f : mn;
        if (__any_sync(0xffffffffu, mn > m[h])) {  // rescale what was summed under a smaller maximum
          const float f = ex2(m[h] - ms);
          l[h] *= f;
#pragma unroll
          for (int d = 0; d < VH; ++d)
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              o[d][y][2 * h] *= f;
              o[d][y][2 * h + 1] *= f;
              if (!WIDE) {
                o[d][y][2] *= f;
                o[d][y][3] *= f;
              }
            }
          m[h] = mn;
        }
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2(x[e] - ms + kProbShift<C>);
          l[h] += p[e];
        }
        split2<C, NP>(p[0], p[1], ph[h][0]);
        split2<C, NP>(p[2], p[3], ph[h][1]);
      }
      // ---- values: pair the positions (2c, 2c + 1) and (2c + 8, 2c + 9) of every dim
#pragma unroll
      for (int d = 0; d < VH; ++d) {
        const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vf[d][0]);
        const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vf[d][1]);
        const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vf[d][2]);
        const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vf[d][3]);
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const uint32_t sel = y & 1 ? 0x7632u : 0x5410u;
          const uint32_t b0 = __byte_perm(v0[y >> 1], v1[y >> 1], sel), b1 = __byte_perm(v2[y >> 1], v3[y >> 1], sel);
#pragma unroll
          for (int p = 0; p < NP; p += WIDE ? 1 : 2) {
            if (WIDE) {
              Mma<C>::run(o[d][y], make_uint4(ph[0][0][p], ph[RH - 1][0][p], ph[0][1][p], ph[RH - 1][1][p]), b0, b1);
            } else {
              const int p2 = p + 1 < NP ? p + 1 : 0;
              Mma<C>::run(o[d][y], make_uint4(ph[0][0][p], p2 ? ph[0][0][p2] : 0u, ph[0][1][p], p2 ? ph[0][1][p2] : 0u),
                          b0, b1);
            }
          }
        }
      }
    }
    // ---- merge the warps' pieces in shared memory, fixed order
    flush(!FLUSH || mine <= 32);
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      float lh = l[h];
      lh += __shfl_xor_sync(0xffffffffu, lh, 1);
      lh += __shfl_xor_sync(0xffffffffu, lh, 2);
      if (c == 0) s_ml[(warp * HEADS + g + 8 * h) * 2 + 1] = lh;
    }
    __syncthreads();
    const int r = st->row, j = st->head, slot = st->slot;
    if (tid == 0 && st->bad) {
      report(a.status, MK_ERR_PAGES, PO_ATTEND, r, st->bad_page);
      st->bad = 0;
    }
    for (int x = tid; x < a.group * (HD / 4); x += kAttThreads) {
      const int h = x / (HD / 4), d = (x % (HD / 4)) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) M = fmaxf(M, s_ml[(w * HEADS + h) * 2]);
      const float Ms = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        const float f = ex2(s_ml[(w * HEADS + h) * 2] - Ms);
        const float4 v = *reinterpret_cast<const float4*>(s_part + (w * HEADS + h) * ROW + d);
        L = fmaf(f, s_ml[(w * HEADS + h) * 2 + 1], L);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (slot == 2) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        Q* dst = static_cast<Q*>(a.out) + (long long)r * a.o_row + (long long)(j * a.group + h) * a.o_head + d;
        dst[0] = Conv<Q>::down(acc.x * inv);
        dst[1] = Conv<Q>::down(acc.y * inv);
        dst[2] = Conv<Q>::down(acc.z * inv);
        dst[3] = Conv<Q>::down(acc.w * inv);
        if (d == 0 && a.lse)
          a.lse[(long long)r * a.hq + j * a.group + h] = (Ms - kProbShift<C> + log2f(L)) * kLn2;
      } else {
        float* dst = a.part + (((size_t)blockIdx.x * 2 + slot) * a.group + h) * ROW;
        *reinterpret_cast<float4*>(dst + d) = acc;
        if (d == 0) {
          dst[HD] = M;
          dst[HD + 1] = L;
        }
      }
    }
    if (st->at >= st->end) return;
  }
}

// Joins the pieces of the segments that span CTAs: one CTA per (segment, head of its group);
// warps take the pieces in turn, each lane HD / 32 dims.  Bound: the launch and two dependent
// loads, 1.2 us behind one row of 512 positions, 2 us when nothing is to be joined in 2000 CTAs.
template <typename Q, int HD>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttendArgs a, float shift) {
  constexpr int W = kJoinThreads / 32, E = HD / 32, ROW = HD + 4;
  __shared__ float s_o[W][HD], s_ml[W][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
  pdl_wait();
  pdl_launch();
  const int4 job = a.joins[blockIdx.x];
  const int c0 = job.x, c1 = job.y, r = job.z, head = job.w * a.group + h;
  if (c1 < 0) return;  // finished by its CTA
  Q* out = static_cast<Q*>(a.out) + (long long)r * a.o_row + (long long)head * a.o_head;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  constexpr int U = 8;  // pieces in flight per warp
  for (int b = c0 + warp; b <= c1; b += W * U) {
    float pm[U], pl[U], po[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = min(b + u * W, c1);  // past the last: loaded and not used
      const float* p = a.part + (((size_t)x * 2 + (x == c0)) * a.group + h) * ROW;
#pragma unroll
      for (int e = 0; e < E; ++e) po[u][e] = p[e * 32 + lane];
      pm[u] = p[HD];
      pl[u] = p[HD + 1];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u * W > c1) continue;
      const float mn = fmaxf(m, pm[u]), ms = mn == -INFINITY ? 0.f : mn;
      const float f0 = ex2(m - ms), f1 = ex2(pm[u] - ms);
      l = l * f0 + pl[u] * f1;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f0 + po[u][e] * f1;
      m = mn;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][e * 32 + lane] = o[e];
  if (lane == 0) {
    s_ml[warp][0] = m;
    s_ml[warp][1] = l;
  }
  __syncthreads();
  if (tid < HD) {
    float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, s_ml[w][0]);
    const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = ex2(s_ml[w][0] - Ms);
      L = fmaf(f, s_ml[w][1], L);
      acc = fmaf(f, s_o[w][tid], acc);
    }
    out[tid] = Conv<Q>::down(L == 0.f ? 0.f : acc / L);
    if (tid == 0 && a.lse) a.lse[(long long)r * a.hq + head] = (Ms - shift + log2f(L)) * kLn2;
  }
}

template <typename C, typename Q, int HD, bool WIDE, int NQ, int NP>
mk_status launch_attend(const AttendArgs& a, void* stream) {
  auto k = attend_kernel<C, Q, HD, WIDE, NQ, NP>;
  constexpr int smem = AttSmem<HD, WIDE, NQ>::kBytes;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return paged_fail(MK_ERR_CUDA, std::string("mk_paged_attention: ") + cudaGetErrorString(e));
  }
  const mk_status s = launch_dependent(k, dim3(a.n_cta), dim3(kAttThreads), smem, stream, "mk_paged_attention", a);
  if (s) return s;
  const int jobs = a.by_segment ? a.n_rows * a.hkv : a.n_cta;
  return launch_dependent(join_kernel<Q, HD>, dim3(jobs, a.group), dim3(kJoinThreads), 0, stream,
                          "mk_paged_attention (join)", a, kProbShift<C>);
}
template <typename C, typename Q, int NQ, int NP>
mk_status launch_attend(const AttendArgs& a, int hd, void* stream) {
  const bool wide = a.group > 8;
  if (hd == 64) return wide ? launch_attend<C, Q, 64, true, NQ, NP>(a, stream) : launch_attend<C, Q, 64, false, NQ, NP>(a, stream);
  return wide ? launch_attend<C, Q, 128, true, NQ, NP>(a, stream) : launch_attend<C, Q, 128, false, NQ, NP>(a, stream);
}

}  // namespace

// the line of work counts in 32 bits
std::string check_line(const mk_page_view* c, long long n_rows, int window) {
  const long long cap = (long long)c->table_width * c->page_size;
  const long long most = (window > 0 ? std::min(cap, (long long)window + kTile) : cap) / kTile + 1 + kLead;
  if (most * n_rows > 0x7f000000LL / c->n_kv_heads)
    return "n_rows * n_kv_heads * (the table's positions / 16 + 9) must be below 2^31 - 2^24";
  return "";
}
}  // namespace mk

extern "C" mk_status mk_paged_attention_workspace(int n_heads, int n_kv_heads, int head_dim, size_t* bytes) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    if (!bytes) return paged_fail(MK_ERR_INVALID, "bytes is NULL");
    if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > kMaxGroup)
      return paged_fail(MK_ERR_INVALID, "n_heads / n_kv_heads must be a whole number in [1, 16]");
    if (head_dim != 64 && head_dim != 128) return paged_fail(MK_ERR_INVALID, "head_dim must be 64 or 128");
    int n_sm = 0;
    const mk_status s = sm_count(&n_sm);
    if (s) return s;
    const size_t n_cta = (size_t)n_sm * ctas_per_sm(head_dim);
    *bytes = n_cta * (sizeof(int4) + 2 * (n_heads / n_kv_heads) * (head_dim + 4) * sizeof(float));
    return MK_OK;
  });
}

extern "C" mk_status mk_paged_attention(const mk_attend_args* args, const mk_page_view* cache, int32_t* status,
                                        void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    const std::string e = check_view(cache);
    if (!e.empty()) return paged_fail(MK_ERR_INVALID, e);
    if (!args || !args->q || !args->out || !args->lens) return paged_fail(MK_ERR_INVALID, "NULL argument");
    if (args->dtype < MK_F16 || args->dtype > MK_F32) return paged_fail(MK_ERR_INVALID, "dtype");
    if (args->n_heads < 1 || args->n_heads % cache->n_kv_heads || args->n_heads / cache->n_kv_heads > kMaxGroup)
      return paged_fail(MK_ERR_INVALID, "n_heads / n_kv_heads must be a whole number in [1, 16]");
    if (args->n_rows < 0 || (long long)args->n_rows * args->n_heads > 0x7fffffffLL)
      return paged_fail(MK_ERR_INVALID, "n_rows out of range");
    if (args->window < 0) return paged_fail(MK_ERR_INVALID, "window must not be negative");
    const float factor = args->softcap > 0.f ? args->scale / args->softcap : args->scale * kLog2e;
    if (!(args->softcap >= 0.f && args->softcap * kLog2e < INFINITY) || !(fabsf(factor) < INFINITY))
      return paged_fail(MK_ERR_INVALID, "scale or softcap is not finite, too large, or softcap negative or too small for scale");
    const size_t esz = args->dtype == MK_F32 ? 4 : 2;
    if (!aligned_to(args->q, esz) || !aligned_to(args->out, esz))
      return paged_fail(MK_ERR_INVALID, "q and out must be aligned to their type");
    if (overlaps(args->n_rows, args->o_row, args->n_heads, args->o_head, cache->head_dim))
      return paged_fail(MK_ERR_INVALID, "the vectors of out overlap");
    const std::string line = check_line(cache, args->n_rows, args->window);
    if (!line.empty()) return paged_fail(MK_ERR_INVALID, line);
    if (!args->workspace || !aligned_to(args->workspace, 16))
      return paged_fail(MK_ERR_INVALID, "the workspace is missing or unaligned");
    if (args->n_rows == 0) return MK_OK;
    size_t need = 0;
    mk_status s = mk_paged_attention_workspace(args->n_heads, cache->n_kv_heads, cache->head_dim, &need);
    if (s) return s;
    if (args->workspace_bytes < need)
      return paged_fail(MK_ERR_INVALID, "the workspace is too small (mk_paged_attention_workspace)");
    int n_sm = 0;
    s = sm_count(&n_sm);
    if (s) return s;
    AttendArgs a{};
    a.q = args->q; a.k = cache->k; a.v = cache->v; a.out = args->out; a.lse = args->lse;
    a.joins = static_cast<int4*>(args->workspace);
    a.lens = args->lens; a.rows = args->rows; a.table = cache->table; a.status = status;
    a.q_row = args->q_row; a.q_head = args->q_head; a.o_row = args->o_row; a.o_head = args->o_head;
    a.page_stride = cache->page_stride; a.table_stride = cache->table_stride;
    a.n_rows = args->n_rows; a.hq = args->n_heads; a.hkv = cache->n_kv_heads; a.group = args->n_heads / cache->n_kv_heads;
    a.len_add = args->len_add; a.window = args->window; a.page_size = cache->page_size; a.n_pages = cache->n_pages;
    a.table_rows = cache->n_rows; a.cap = cache->table_width * cache->page_size;  // at most 2^30
    a.tpp = a.page_size / kTile;
    a.tpp_inverse = a.tpp > 1 ? (unsigned)(((1ULL << 32) + a.tpp - 1) / a.tpp) : 0;
    a.n_cta = n_sm * ctas_per_sm(cache->head_dim);
    a.part = reinterpret_cast<float*>(a.joins + a.n_cta);
    a.q_vec = aligned_to(a.q, 16) && a.q_row * (long long)esz % 16 == 0 && a.q_head * (long long)esz % 16 == 0;
    a.by_segment = (long long)a.n_rows * a.hkv <= a.n_cta;
    a.scale = factor;
    a.softcap = args->softcap * kLog2e;
    // 16-bit queries of the cache's type are exact in one part.  Other queries are split into
    // 2 parts of fp16 (22 bits, each head at a power of two of its own) or 3 of bf16 (24 bits);
    // probabilities likewise, 2 parts of
    // bf16 (16 bits) being enough for an output of 16 bits: 16 rows of 16384 to 32768 positions
    // lie 1.66e-3 (all of it the output's rounding) from the 64-bit result with 2 parts and
    // with 3, and a batch of 61 short rows takes 13.7 us with 2, 14.3 with 3.
    if (cache->dtype == MK_F16) {
      if (args->dtype == MK_F16) return launch_attend<__half, __half, 1, 2>(a, cache->head_dim, stream);
      if (args->dtype == MK_BF16) return launch_attend<__half, __nv_bfloat16, 2, 2>(a, cache->head_dim, stream);
      return launch_attend<__half, float, 2, 2>(a, cache->head_dim, stream);
    }
    if (args->dtype == MK_BF16) return launch_attend<__nv_bfloat16, __nv_bfloat16, 1, 2>(a, cache->head_dim, stream);
    if (args->dtype == MK_F16) return launch_attend<__nv_bfloat16, __half, 2, 2>(a, cache->head_dim, stream);
    return launch_attend<__nv_bfloat16, float, 3, 3>(a, cache->head_dim, stream);
  });
}
