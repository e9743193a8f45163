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
constexpr int kJoinThreads = 256;
constexpr int kMaxGroup = 16;           // query heads per kv head
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

struct AttendArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  float* part;                          // [n_cta][2][heads of a group][HD + 4]
  const int32_t *lens, *rows, *table;
  int32_t* status;
  long long q_row, q_head, o_row, o_head, page_stride, table_stride;
  int n_rows, hq, hkv, group, len_add, window, page_size, n_pages, table_rows, width;
  int n_cta, min_share;
  float scale, softcap;
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

// Sums of the rows' tiles over a CTA of THREADS, thread t taking the rows from t * per:
// returns the total; *before: the tiles of the rows before this thread's (upto < 0), or of the
// rows below `upto`.
template <int THREADS>
__device__ __forceinline__ long long sum_rows(const AttendArgs& a, long long* sums, bool tell, int upto,
                                              long long* before) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_rows + THREADS - 1) / THREADS, r0 = min(a.n_rows, tid * per), r1 = min(a.n_rows, r0 + per);
  long long mine = 0, below = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = span_of(a, r, tell).n;
    mine += n;
    if (r < upto) below += n;
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 31) sums[warp] = inc;
  if (lane == 0) sums[THREADS / 32 + warp] = below;
  __syncthreads();
  long long base = 0, total = 0, bel = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) base += sums[w];
    total += sums[w];
    bel += sums[THREADS / 32 + w];
  }
  __syncthreads();
  *before = upto >= 0 ? bel : base + inc - mine;
  return total;
}

// units (tiles of one kv head) a CTA takes: equal shares of one wave, but no fewer than
// min_share, so that a short call is not cut into pieces whose join costs more than they save
__device__ __forceinline__ long long share_of(const AttendArgs& a, long long units) {
  return max((long long)a.min_share, (units + a.n_cta - 1) / a.n_cta);
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
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

// keys and values are read once: they need not stay in L1
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Shared memory of the kernel: the query as A fragments [part][32-dim chunk][32 lanes][16 B]
// (WIDE: [part][chunk][2 row halves][32 lanes]), then the warps' partials for the CTA's merge.
template <int HD, bool WIDE, int NQ>
struct AttSmem {
  static constexpr int kHeads = WIDE ? 16 : 8;
  static constexpr int kQBytes = NQ * (HD / 32) * (WIDE ? 2 : 1) * 32 * 16;
  static constexpr int kRow = HD + 4;                        // floats per head of a partial
  static constexpr int kPartFloats = kAttWarps * kHeads * kRow;
  static constexpr int kMlFloats = kAttWarps * kHeads * 2;
  static constexpr int kBytes = kQBytes + 4 * (kPartFloats + kMlFloats) + 16 * kAttWarps + 32;
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
template <typename C, typename Q, int HD, bool WIDE, int NQ, int NP>
__global__ void __launch_bounds__(kAttThreads, HD == 128 ? 3 : 4) attend_kernel(const __grid_constant__ AttendArgs a) {
  using SM = AttSmem<HD, WIDE, NQ>;
  constexpr int CH = HD / 32, VH = HD / 64, HEADS = SM::kHeads, ROW = SM::kRow;
  constexpr int RH = WIDE ? 2 : 1;  // row halves that are heads of their own
  extern __shared__ __align__(16) unsigned char att_smem[];
  uint4* s_q = reinterpret_cast<uint4*>(att_smem);
  float* s_part = reinterpret_cast<float*>(att_smem + SM::kQBytes);
  float* s_ml = s_part + SM::kPartFloats;
  long long* s_sum = reinterpret_cast<long long*>(s_ml + SM::kMlFloats);  // [2 kAttWarps]
  long long* s_before = s_sum + 2 * kAttWarps;                            // units before the first row
  int* s_row = reinterpret_cast<int*>(s_before + 1);                      // the first row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_launch();
  long long before;
  const long long units = sum_rows<kAttThreads>(a, s_sum, blockIdx.x == 0, -1, &before) * a.hkv;
  const long long share = share_of(a, units);
  long long at = share * blockIdx.x;
  const long long end = min(units, at + share);
  if (at >= end) return;
  {  // the row that holds unit `at` is among one thread's rows
    const int per = (a.n_rows + kAttThreads - 1) / kAttThreads;
    const int r0 = min(a.n_rows, tid * per), r1 = min(a.n_rows, r0 + per);
    long long b = before * a.hkv;
    for (int r = r0; r < r1; ++r) {
      const long long n = (long long)span_of(a, r, false).n * a.hkv;
      if (at >= b && at < b + n) {
        *s_row = r;
        *s_before = b;
      }
      b += n;
    }
  }
  __syncthreads();
  int r = *s_row;
  long long rbase = *s_before;  // units before row r
  while (at < end) {
    const Span sp = span_of(a, r, false);
    const long long in_row = at - rbase;
    if (in_row >= (long long)sp.n * a.hkv) {  // next row (rows without positions have no units)
      rbase += (long long)sp.n * a.hkv;
      ++r;
      continue;
    }
    const int j = (int)(in_row / sp.n), first = (int)(in_row - (long long)j * sp.n);
    const int cnt = (int)min((long long)(sp.n - first), end - at);  // tiles of this piece
    // ---- the query's fragments: chunk i, lane (g, c): dims [32 i + 8 c, + 8) of head g
    __syncthreads();
    for (int x = tid; x < CH * HEADS * 4; x += kAttThreads) {
      const int cc = x & 3, h = (x >> 2) % HEADS, i = x / (4 * HEADS);
      float v[8];
      const Q* src = static_cast<const Q*>(a.q) + (long long)r * a.q_row +
                     (long long)(j * a.group + min(h, a.group - 1)) * a.q_head + 32 * i + 8 * cc;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = h < a.group ? Conv<Q>::up(src[e]) : 0.f;
      uint32_t w[4][NQ];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2<C, NQ>(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
      for (int p = 0; p < NQ; ++p) {
        const int slot = WIDE ? ((p * CH + i) * 2 + (h >> 3)) * 32 : (p * CH + i) * 32;
        s_q[slot + (h & 7) * 4 + cc] = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
      }
    }
    __syncthreads();
    // ---- this warp's tiles: first + warp, + kAttWarps, ...
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
    const int32_t* trow = a.table + (long long)sp.trow * a.table_stride;
    const int tpp = a.page_size / kTile;  // tiles per page
    const int mine = cnt > warp ? (cnt - warp + kAttWarps - 1) / kAttWarps : 0;
    // lane i holds the page of this warp's (32 b + i)-th tile; the next 32 are fetched ahead
    auto page_of = [&](int k) -> int { return k < mine ? trow[(sp.t0 + first + warp + k * kAttWarps) / tpp] : -1; };
    int pages = page_of(lane), pages_next = -1;
    const C* kbase = static_cast<const C*>(a.k) + (long long)j * a.page_size * HD;
    const C* vbase = static_cast<const C*>(a.v) + (long long)j * a.page_size * HD;
    // a tile's offset in the pages, and the positions [p0, p1) of it that count
    auto locate = [&](int k, long long* off, int* p0, int* p1) {
      const int t = sp.t0 + first + warp + k * kAttWarps;
      const int page = __shfl_sync(0xffffffffu, pages, k & 31);
      *p0 = max(0, sp.lo - t * kTile);
      *p1 = min(kTile, sp.hi - t * kTile);
      *off = (long long)page * a.page_stride + (t % tpp) * (kTile * HD);
      if ((unsigned)page >= (unsigned)a.n_pages) {
        if (lane == 0) report(a.status, MK_ERR_PAGES, PO_ATTEND, r, page);
        *p0 = *p1 = 0;
        *off = 0;
      }
    };
    uint4 kf[2][CH];
    auto load_k = [&](long long off, int p0, int p1) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int p = n * 8 + g;
        const C* src = kbase + off + p * HD + 8 * c;
#pragma unroll
        for (int i = 0; i < CH; ++i)
          kf[n][i] = p >= p0 && p < p1 ? ldg_stream(src + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    long long off = 0;
    int p0 = 0, p1 = 0;
    if (mine > 0) {
      locate(0, &off, &p0, &p1);
      load_k(off, p0, p1);
    }
    for (int k = 0; k < mine; ++k) {
      if ((k & 31) == 0) pages_next = page_of(k + 32 + lane);
      const int q0 = p0, q1 = p1;
      // values of this tile: in flight while the scores are computed
      uint4 vf[VH][4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int p = 2 * c + (x & 1) + 8 * (x >> 1);
        const C* src = vbase + off + p * HD + 8 * g;
#pragma unroll
        for (int h = 0; h < VH; ++h)
          vf[h][x] = p >= q0 && p < q1 ? ldg_stream(src + 64 * h) : make_uint4(0u, 0u, 0u, 0u);
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
      if (((k + 1) & 31) == 0) pages = pages_next;
      if (k + 1 < mine) {
        locate(k + 1, &off, &p0, &p1);
        load_k(off, p0, p1);
      }
      // ---- softmax of the tile, in units of log 2; lane (g, c): columns 2c, 2c + 1 of each half
      uint32_t ph[RH][2][NP];  // [row half][column half][part]
#pragma unroll
      for (int h = 0; h < RH; ++h) {
        float x[4], top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int p = 2 * c + (e & 1) + 8 * (e >> 1);
          float y = s[e >> 1][2 * h + (e & 1)];
          // the second part's row; one part has none, and there 0 times an infinite key is NaN
          if (!WIDE && NQ > 1) y += s[e >> 1][2 + (e & 1)];
          y *= a.scale;
          if (a.softcap > 0.f) y = a.softcap * tanhf(y / a.softcap);
          x[e] = p >= q0 && p < q1 ? y * kLog2e : -INFINITY;
          top = fmaxf(top, x[e]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[h], top), ms = mn == -INFINITY ? 0.f : mn;
        if (__any_sync(0xffffffffu, mn > m[h])) {  // rescale what was summed under a smaller maximum
          const float f = exp2f(m[h] - ms);
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
          p[e] = exp2f(x[e] - ms + kProbShift<C>);
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
    const bool whole = first == 0 && cnt == sp.n;
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
        const float f = exp2f(s_ml[(w * HEADS + h) * 2] - Ms);
        const float4 v = *reinterpret_cast<const float4*>(s_part + (w * HEADS + h) * ROW + d);
        L = fmaf(f, s_ml[(w * HEADS + h) * 2 + 1], L);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        Q* dst = static_cast<Q*>(a.out) + (long long)r * a.o_row + (long long)(j * a.group + h) * a.o_head + d;
        dst[0] = Conv<Q>::down(acc.x * inv);
        dst[1] = Conv<Q>::down(acc.y * inv);
        dst[2] = Conv<Q>::down(acc.z * inv);
        dst[3] = Conv<Q>::down(acc.w * inv);
        if (d == 0 && a.lse)
          a.lse[(long long)r * a.hq + j * a.group + h] = (Ms - kProbShift<C> + log2f(L)) * kLn2;
      } else {  // slot 0: a piece that continues a segment, slot 1: one that begins it
        float* dst = a.part + (((size_t)blockIdx.x * 2 + (first == 0)) * a.group + h) * ROW;
        *reinterpret_cast<float4*>(dst + d) = acc;
        if (d == 0) {
          dst[HD] = M;
          dst[HD + 1] = L;
        }
      }
    }
    at += cnt;
  }
}

// Joins the pieces of the segments that span CTAs, and writes the rows without positions.
// One CTA per (row, query head); warps take the pieces in turn, each lane HD / 32 dims.
template <typename Q, int HD>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttendArgs a, float shift) {
  constexpr int W = kJoinThreads / 32, E = HD / 32, ROW = HD + 4;
  __shared__ long long sums[2 * W];
  __shared__ float s_o[W][HD], s_ml[W][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / a.hq, head = blockIdx.x % a.hq, j = head / a.group, h = head % a.group;
  pdl_wait();
  pdl_launch();
  const Span sp = span_of(a, r, false);
  Q* out = static_cast<Q*>(a.out) + (long long)r * a.o_row + (long long)head * a.o_head;
  if (sp.n == 0) {
    for (int d = tid; d < HD; d += kJoinThreads) out[d] = Conv<Q>::down(0.f);
    if (tid == 0 && a.lse) a.lse[(long long)r * a.hq + head] = -INFINITY;
    return;
  }
  long long before;
  const long long units = sum_rows<kJoinThreads>(a, sums, false, r, &before) * a.hkv;
  const long long share = share_of(a, units), from = before * a.hkv + (long long)j * sp.n;
  const int c0 = (int)(from / share), c1 = (int)((from + sp.n - 1) / share);
  if (c0 == c1) return;  // finished by its CTA
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  constexpr int U = 4;  // pieces in flight per warp
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
      const float f0 = exp2f(m - ms), f1 = exp2f(pm[u] - ms);
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
      const float f = exp2f(s_ml[w][0] - Ms);
      L = fmaf(f, s_ml[w][1], L);
      acc = fmaf(f, s_o[w][tid], acc);
    }
    out[tid] = Conv<Q>::down(L == 0.f ? 0.f : acc / L);
    if (tid == 0 && a.lse) a.lse[(long long)r * a.hq + head] = (Ms - shift + log2f(L)) * kLn2;
  }
}

// CTAs of one wave: resident per SM by the launch bounds, the same for every instance of a
// head_dim, so that the workspace's size depends on nothing else
int ctas_per_sm(int hd) { return hd == 128 ? 3 : 4; }

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
  return launch_dependent(join_kernel<Q, HD>, dim3((unsigned)(a.n_rows * a.hq)), dim3(kJoinThreads), 0, stream,
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
  if (!bytes) return paged_fail(MK_ERR_INVALID, "bytes is NULL");
  if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > kMaxGroup)
    return paged_fail(MK_ERR_INVALID, "n_heads / n_kv_heads must be a whole number in [1, 16]");
  if (head_dim != 64 && head_dim != 128) return paged_fail(MK_ERR_INVALID, "head_dim must be 64 or 128");
  int n_sm = 0;
  const mk_status s = sm_count(&n_sm);
  if (s) return s;
  *bytes = (size_t)n_sm * ctas_per_sm(head_dim) * 2 * (n_heads / n_kv_heads) * (head_dim + 4) * sizeof(float);
  return MK_OK;
}

extern "C" mk_status mk_paged_attention(const mk_attend_args* args, const mk_page_view* cache, int32_t* status,
                                        void* stream) {
  using namespace mk;
  const std::string e = check_view(cache);
  if (!e.empty()) return paged_fail(MK_ERR_INVALID, e);
  if (!args || !args->q || !args->out || !args->lens) return paged_fail(MK_ERR_INVALID, "NULL argument");
  if (args->dtype < MK_F16 || args->dtype > MK_F32) return paged_fail(MK_ERR_INVALID, "dtype");
  if (args->n_heads < 1 || args->n_heads % cache->n_kv_heads || args->n_heads / cache->n_kv_heads > kMaxGroup)
    return paged_fail(MK_ERR_INVALID, "n_heads / n_kv_heads must be a whole number in [1, 16]");
  if (args->n_rows < 0 || (long long)args->n_rows * args->n_heads > 0x7fffffffLL)
    return paged_fail(MK_ERR_INVALID, "n_rows out of range");
  if (args->window < 0) return paged_fail(MK_ERR_INVALID, "window must not be negative");
  if (!(args->softcap >= 0.f) || !(args->scale == args->scale)) return paged_fail(MK_ERR_INVALID, "scale or softcap");
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
  a.part = static_cast<float*>(args->workspace);
  a.lens = args->lens; a.rows = args->rows; a.table = cache->table; a.status = status;
  a.q_row = args->q_row; a.q_head = args->q_head; a.o_row = args->o_row; a.o_head = args->o_head;
  a.page_stride = cache->page_stride; a.table_stride = cache->table_stride;
  a.n_rows = args->n_rows; a.hq = args->n_heads; a.hkv = cache->n_kv_heads; a.group = args->n_heads / cache->n_kv_heads;
  a.len_add = args->len_add; a.window = args->window; a.page_size = cache->page_size; a.n_pages = cache->n_pages;
  a.table_rows = cache->n_rows; a.width = cache->table_width;
  a.n_cta = n_sm * ctas_per_sm(cache->head_dim);
  a.min_share = kAttWarps;
  a.scale = args->scale; a.softcap = args->softcap;
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
}
