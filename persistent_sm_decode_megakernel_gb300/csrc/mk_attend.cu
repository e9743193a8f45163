// Attention of one new token per row over a paged KV cache (mk_paged_attention).
//
// The rows' positions are cut into tiles of 16 (a tile lies in one page).  The segments
// (row, kv head), each of its row's tiles, follow one another in one line of work, and every
// CTA of a single wave takes an equal, contiguous share of that line: batches of any raggedness
// load the SMs evenly, and one long sequence is split over all of them.  A segment that lies
// in one CTA is finished there; the pieces of one that spans CTAs go to the workspace as
// (running maximum, sum, weighted values) and a second small kernel joins them in order:
//   M = max M_i,  L = sum L_i 2^(M_i - M),  out = sum O_i 2^(M_i - M) / L.
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
  int n_rows, hq, hkv, group, len_add, window, page_size, n_pages, table_rows, width;
  int tpp;                              // tiles per page
  unsigned tpp_inverse;                 // 2^32 / tpp, rounded up
  int n_cta;
  int by_segment;                       // joins[row * hkv + kv head] (they fit), else joins[first CTA]
  float scale, softcap;                 // scores to units of log 2: scale s, or softcap tanh(scale s)
};

// The span of a row: positions [lo, hi) and their tiles [t0, t0 + n).
struct Span {
  int lo, hi, t0, n, trow;
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, int r, bool tell) {
  Span s;
  s.trow = a.rows ? a.rows[r] : r;
  long long len = (long long)a.lens[r] + a.len_add;
  const long long cap = (long long)a.width * a.page_size;
  if ((unsigned)s.trow >= (unsigned)a.table_rows) {
    if (tell && len > 0) report(a.status, MK_ERR_PAGES, PO_ATTEND, r, s.trow);
    len = 0;
  }
  if (tell && len > cap) report(a.status, MK_ERR_PAGES, PO_ATTEND, r, (int)min(len, 0x7fffffffLL));
  // the window counts from the row's own end, also where the table ends earlier
  const long long lo = a.window > 0 ? max(0LL, len - a.window) : 0LL;
  s.hi = (int)max(0LL, min(len, cap));
  s.lo = (int)min(lo, (long long)s.hi);
  s.t0 = s.lo / kTile;
  s.n = s.hi > s.lo ? (s.hi + kTile - 1) / kTile - s.t0 : 0;
  return s;
}

// The line of work, in units: every segment counts its tiles and `lead` units in front of them
// for what a piece costs besides its tiles (the query, the table, the merge).  CTA c takes
// [c share, (c + 1) share).  Of what a CTA takes, a segment's lead is where it begins: the
// segment's first tiles are of the CTA that holds their units, whoever holds the lead.
//   lead: with fewer tiles than the wave's warps the latency of a piece is all there is, and
//     equal tiles are best; else kLead, without which a CTA that meets a dozen segments of two
//     tiles each ran twice as long as the others (61 ragged rows of up to 700 positions).
constexpr int kLead = 8;
struct Line {
  long long units, share;
  int lead;
};
__device__ __forceinline__ long long row_units(const AttendArgs& a, int n, int lead) {
  return n > 0 ? (long long)(n + lead) * a.hkv : 0LL;
}
// The line, and in *row and *before (shared memory; the caller syncs) the row that holds this
// CTA's first unit and the units before it.
__device__ __forceinline__ Line find_row(const AttendArgs& a, long long (*sums)[2], int* row, long long* before) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_rows + kAttThreads - 1) / kAttThreads;
  const int r0 = min(a.n_rows, tid * per), r1 = min(a.n_rows, r0 + per);
  long long tiles = 0;
  int rows = 0;  // with positions
  for (int r = r0; r < r1; ++r) {
    const int n = span_of(a, r, blockIdx.x == 0).n;
    tiles += n;
    rows += n > 0;
  }
  long long ti = tiles;
  int ri = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, ti, o);
    const int y = __shfl_up_sync(0xffffffffu, ri, o);
    if (lane >= o) {
      ti += x;
      ri += y;
    }
  }
  if (lane == 31) {
    sums[warp][0] = ti;
    sums[warp][1] = ri;
  }
  __syncthreads();
  long long all_tiles = 0, all_rows = 0;
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) {
    if (w == warp) {
      ti += all_tiles - tiles;  // before this thread's rows
      ri += (int)all_rows - rows;
    }
    all_tiles += sums[w][0];
    all_rows += sums[w][1];
  }
  Line l;
  l.lead = all_tiles * a.hkv <= (long long)a.n_cta * kAttWarps ? 0 : kLead;
  l.units = (all_tiles + all_rows * l.lead) * a.hkv;
  l.share = max((long long)kAttWarps, (l.units + a.n_cta - 1) / a.n_cta);
  const long long at = l.share * blockIdx.x;
  long long b = (ti + (long long)ri * l.lead) * a.hkv;
  if (at >= b && at < b + (tiles + (long long)rows * l.lead) * a.hkv)
    for (int r = r0; r < r1; ++r) {
      const long long n = row_units(a, per == 1 ? (int)tiles : span_of(a, r, false).n, l.lead);
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

// 2^x by the hardware's approximation (2 ulp; results below the normal range become 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared memory of the kernel: the query as A fragments [part][32-dim chunk][32 lanes][16 B]
// (WIDE: [part][chunk][2 row halves][32 lanes]), then the warps' partials for the CTA's merge.
struct AttState {
  long long at, end, share, before;  // next unit, end of the CTA's units, share; units before `row`
  long long sums[kAttWarps][2];
  int row, head, slot, lead, bad, bad_page;
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
// other's latency.
//
// A warp takes NT tiles at a time: with 64 dims two, so that as many bytes are in flight.
template <typename C, typename Q, int HD, bool WIDE, int NQ, int NP>
__global__ void __launch_bounds__(kAttThreads, ctas_per_sm(HD)) attend_kernel(const __grid_constant__ AttendArgs a) {
  using SM = AttSmem<HD, WIDE, NQ>;
  constexpr int CH = HD / 32, VH = HD / 64, HEADS = SM::kHeads, ROW = SM::kRow, NT = 1;
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
  // rows without positions: zeros
  for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
    if (span_of(a, r, false).n != 0) continue;
    for (int x = tid; x < a.hq * HD; x += kAttThreads)
      static_cast<Q*>(a.out)[(long long)r * a.o_row + (long long)(x / HD) * a.o_head + x % HD] = Conv<Q>::down(0.f);
    for (int h = tid; h < a.hq; h += kAttThreads) {
      if (a.lse) a.lse[(long long)r * a.hq + h] = -INFINITY;
      if (a.by_segment && h < a.hkv) a.joins[r * a.hkv + h] = make_int4(0, -1, 0, 0);
    }
  }
  if (tid == 0 && !a.by_segment) a.joins[blockIdx.x] = make_int4(0, -1, 0, 0);
  if (line.share * blockIdx.x >= line.units) return;
  __syncthreads();
  // what a piece needs again at its end lives in shared memory: the loop over the tiles has
  // few registers to spare
  if (tid == 0) {
    st->at = line.share * blockIdx.x;
    st->end = min(line.units, line.share * (blockIdx.x + 1LL));
    st->share = line.share;
    st->lead = line.lead;
    st->bad = 0;
  }
  __syncthreads();
  while (true) {
    int base, cnt, mine, lo, hi;  // this warp's tiles: base, + kAttWarps, ...
    const int32_t* trow;
    {
      long long rbase = st->before, at = st->at, seg;  // seg: the segment's first unit
      int r = st->row, j, first;
      Span sp;
      while (true) {
        sp = span_of(a, r, false);
        const long long n = row_units(a, sp.n, st->lead);
        if (at < rbase + n) {
          const int each = sp.n + st->lead;
          j = (int)((at - rbase) / each);
          seg = rbase + (long long)j * each;
          const long long stop = min(st->end, seg + each);
          first = (int)max(0LL, at - seg - st->lead);
          cnt = (int)(stop - seg - st->lead) - first;  // tiles of this piece
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
        st->slot = whole ? 2 : first == 0;  // 0: continues a segment, 1: begins one, 2: is one
        if (first == 0) {  // the segment's begin knows where it ends
          const int last = (int)((seg + st->lead + sp.n - 1) / st->share);
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
      trow = a.table + (long long)sp.trow * a.table_stride;
    }
    __syncthreads();
    // lane i holds the page of this warp's (32 b + i)-th tile; the next 32 are fetched ahead
    auto page_of = [&](int k) -> int { return k < mine ? trow[page_index(a, base + k * kAttWarps)] : -1; };
    int pages = page_of(lane), pages_next = -1;
    // the query's fragments: chunk i, lane (g, c): dims [32 i + 8 c, + 8) of head g
#pragma unroll 1
    for (int y = tid; y < CH * HEADS * 4; y += kAttThreads) {
      const int h = (y >> 2) % HEADS, i = y / (4 * HEADS);
      const Q* src = static_cast<const Q*>(a.q) + (long long)st->row * a.q_row +
                     (long long)(st->head * a.group + min(h, a.group - 1)) * a.q_head + 32 * i + 8 * (y & 3);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = h < a.group ? Conv<Q>::up(src[e]) : 0.f;
      uint32_t w[4][NQ];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2<C, NQ>(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
      for (int p = 0; p < NQ; ++p) {
        const int slot = WIDE ? ((p * CH + i) * 2 + (h >> 3)) * 32 : (p * CH + i) * 32;
        s_q[slot + (h & 7) * 4 + (y & 3)] = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
      }
    }
    const long long plane = (long long)st->head * a.page_size * HD;  // the kv head's part of a page
    // a tile's offset in the pages, and the positions [p0, p1) of it that count
    long long off[NT];
    int p0[NT], p1[NT];
    auto locate = [&](int k) {
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const int t = base + (k + x) * kAttWarps;
        const int page = __shfl_sync(0xffffffffu, pages, (k + x) & 31);
        p0[x] = max(0, lo - t * kTile);
        p1[x] = min(kTile, hi - t * kTile);
        off[x] = (long long)page * a.page_stride + plane + (t - page_index(a, t) * a.tpp) * (kTile * HD);
        if ((unsigned)page >= (unsigned)a.n_pages || k + x >= mine) {
          if (k + x < mine) {  // no such page: its positions are masked, and reported at the end
            st->bad_page = page;
            st->bad = 1;
          }
          p0[x] = p1[x] = 0;
          off[x] = 0;
        }
      }
    };
    uint4 kf[NT][2][CH];
    auto load_k = [&]() {
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int p = n * 8 + g;
          const C* src = static_cast<const C*>(a.k) + off[x] + p * HD + 8 * c;
          if (p1[x] - p0[x] == kTile) {  // a whole tile: nothing to fill in
#pragma unroll
            for (int i = 0; i < CH; ++i) kf[x][n][i] = ldg_stream(src + 32 * i);
          } else {
#pragma unroll
            for (int i = 0; i < CH; ++i)
              kf[x][n][i] = p >= p0[x] && p < p1[x] ? ldg_stream(src + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
          }
        }
    };
    if (mine > 0) {
      locate(0);
      load_k();
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
    for (int k = 0; k < mine; k += NT) {
      if ((k & 31) == 0) pages_next = page_of(k + 32 + lane);
      int q0[NT], q1[NT];
      // values of these tiles: in flight while the scores are computed
      uint4 vf[NT][VH][4];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        q0[x] = p0[x];
        q1[x] = p1[x];
        const C* src = static_cast<const C*>(a.v) + off[x] + 2 * c * HD + 8 * g;
        if (p1[x] - p0[x] == kTile) {
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int h = 0; h < VH; ++h) vf[x][h][y] = ldg_stream(src + ((y & 1) + 8 * (y >> 1)) * HD + 64 * h);
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int p = 2 * c + (y & 1) + 8 * (y >> 1);
#pragma unroll
            for (int h = 0; h < VH; ++h)
              vf[x][h][y] = p >= p0[x] && p < p1[x] ? ldg_stream(src + ((y & 1) + 8 * (y >> 1)) * HD + 64 * h)
                                                    : make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
      float s[NT][2][4];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][n][e] = 0.f;
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
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              Mma<C>::run(s[x][n], make_uint4(u.x, w.x, u.y, w.y), kf[x][n][i].x, kf[x][n][i].y);
              Mma<C>::run(s[x][n], make_uint4(u.z, w.z, u.w, w.w), kf[x][n][i].z, kf[x][n][i].w);
            }
        }
      }
      // the next tiles' keys
      if (((k + NT) & 31) == 0) pages = pages_next;
      if (k + NT < mine) {
        locate(k + NT);
        load_k();
      }
      // ---- softmax of the tiles, in units of log 2; lane (g, c): columns 2c, 2c + 1 of each half
      uint32_t ph[NT][RH][2][NP];  // [tile][row half][column half][part]
#pragma unroll
      for (int h = 0; h < RH; ++h) {
        float x[NT][4], top = -INFINITY;
#pragma unroll
        for (int z = 0; z < NT; ++z) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = s[z][e >> 1][2 * h + (e & 1)];
            // the second part's row; one part has none, and there 0 times an infinite key is NaN
            if (!WIDE && NQ > 1) y += s[z][e >> 1][2 + (e & 1)];
            x[z][e] = y * a.scale;
          }
          if (a.softcap > 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[z][e] = a.softcap * tanhf(x[z][e]);
          }
          if (q1[z] - q0[z] != kTile) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int p = 2 * c + (e & 1) + 8 * (e >> 1);
              if (p < q0[z] || p >= q1[z]) x[z][e] = -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, x[z][e]);
        }
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
#pragma unroll
        for (int z = 0; z < NT; ++z) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(x[z][e] - ms + kProbShift<C>);
            l[h] += p[e];
          }
          split2<C, NP>(p[0], p[1], ph[z][h][0]);
          split2<C, NP>(p[2], p[3], ph[z][h][1]);
        }
      }
      // ---- values: pair the positions (2c, 2c + 1) and (2c + 8, 2c + 9) of every dim
#pragma unroll
      for (int z = 0; z < NT; ++z)
#pragma unroll
        for (int d = 0; d < VH; ++d) {
          const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vf[z][d][0]);
          const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vf[z][d][1]);
          const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vf[z][d][2]);
          const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vf[z][d][3]);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const uint32_t sel = y & 1 ? 0x7632u : 0x5410u;
            const uint32_t b0 = __byte_perm(v0[y >> 1], v1[y >> 1], sel), b1 = __byte_perm(v2[y >> 1], v3[y >> 1], sel);
#pragma unroll
            for (int p = 0; p < NP; p += WIDE ? 1 : 2) {
              if (WIDE) {
                Mma<C>::run(o[d][y], make_uint4(ph[z][0][0][p], ph[z][RH - 1][0][p], ph[z][0][1][p], ph[z][RH - 1][1][p]),
                            b0, b1);
              } else {
                const int p2 = p + 1 < NP ? p + 1 : 0;
                Mma<C>::run(o[d][y], make_uint4(ph[z][0][0][p], p2 ? ph[z][0][0][p2] : 0u, ph[z][0][1][p],
                                                p2 ? ph[z][0][1][p2] : 0u), b0, b1);
              }
            }
          }
        }
    }
    // ---- merge the warps' pieces in shared memory, fixed order
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      float lh = l[h];
      lh += __shfl_xor_sync(0xffffffffu, lh, 1);
      lh += __shfl_xor_sync(0xffffffffu, lh, 2);
      const int head = g + 8 * h;
      if (c == 0) {
        s_ml[(warp * HEADS + head) * 2] = m[h];
        s_ml[(warp * HEADS + head) * 2 + 1] = lh;
      }
      float* dst = s_part + (warp * HEADS + head) * ROW;
#pragma unroll
      for (int d = 0; d < VH; ++d)
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // columns 2c + e: dims 64 d + 16 c + 8 e + y
          float w[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) w[y] = WIDE ? o[d][y][2 * h + e] : o[d][y][e] + o[d][y][2 + e];
          float4* p = reinterpret_cast<float4*>(dst + 64 * d + 16 * c + 8 * e);
          p[0] = make_float4(w[0], w[1], w[2], w[3]);
          p[1] = make_float4(w[4], w[5], w[6], w[7]);
        }
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
// warps take the pieces in turn, each lane HD / 32 dims.
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
    if (!(args->softcap >= 0.f && args->softcap < INFINITY) || !(fabsf(args->scale) < INFINITY)) return paged_fail(MK_ERR_INVALID, "scale or softcap");
    const size_t esz = args->dtype == MK_F32 ? 4 : 2;
    if (!aligned_to(args->q, esz) || !aligned_to(args->out, esz))
      return paged_fail(MK_ERR_INVALID, "q and out must be aligned to their type");
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
    a.table_rows = cache->n_rows; a.width = cache->table_width;
    a.tpp = a.page_size / kTile;
    a.tpp_inverse = a.tpp > 1 ? (unsigned)(((1ULL << 32) + a.tpp - 1) / a.tpp) : 0;
    a.n_cta = n_sm * ctas_per_sm(cache->head_dim);
    a.part = reinterpret_cast<float*>(a.joins + a.n_cta);
    a.by_segment = (long long)a.n_rows * a.hkv <= a.n_cta;
    a.scale = args->softcap > 0.f ? args->scale / args->softcap : args->scale * kLog2e;
    a.softcap = args->softcap * kLog2e;
    // 16-bit queries of the cache's type are exact in one part.  Other queries are split into
    // 2 parts of fp16 (22 bits) or 3 of bf16 (24 bits); probabilities likewise, 2 parts of
    // bf16 (16 bits) being enough for an output of 16 bits.
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
