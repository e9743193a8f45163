// Attention over chosen pages: the bounds of a page's keys (mk_update_bounds), the pages' scores by them
// (mk_page_scores) and the choice (mk_sparse_attention; the attention itself is mk_attend.cu's).
#include <algorithm>

#include "mk_attend.h"
#include "mk_internal.h"
#include "mk_device.cuh"
#include "mk_paged.cuh"

namespace mk {
namespace {

constexpr int kMaxGroup = 16;

// ------------------------------------------------------------------------------ bounds
constexpr int kBoundThreads = 128;

struct BoundArgs {
  const void* k;
  void* bounds;
  const int32_t *lens, *rows, *table;
  int32_t* status;
  long long page_stride, table_stride;
  int n_rows, n_new, hkv, page_size, n_pages, table_rows, width, candidates;
};

template <typename C>
struct Pair;
template <>
struct Pair<__half> {
  using T = __half2;
  static constexpr uint32_t kInf = 0x7c007c00u;
};
template <>
struct Pair<__nv_bfloat16> {
  using T = __nv_bfloat162;
  static constexpr uint32_t kInf = 0x7f807f80u;
};
template <typename C>
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y) {
  using T = typename Pair<C>::T;
  const T r = __hmin2_nan(*reinterpret_cast<const T*>(&x), *reinterpret_cast<const T*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename C>
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  using T = typename Pair<C>::T;
  const T r = __hmax2_nan(*reinterpret_cast<const T*>(&x), *reinterpret_cast<const T*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A CTA takes HEADS kv heads of one page: a thread 16 bytes of every kBoundThreads / (HD / 8)-th key of each,
// pairs of elements compared as they lie there; what the threads found is joined in shared memory.  Bound: the keys'
// bytes; a thread has eight loads in flight, of two heads where a page has few positions (16 prompts of 4096 to
// 8192 positions in pages of 32, 221 MB: 33.9 us, 6.5 TB/s; one head to a CTA 40.5); of a step's one page a row the
// chain from the length over the table to the keys (2.8 us).
template <typename C, int HD, int HEADS>
__global__ void __launch_bounds__(kBoundThreads) bounds_kernel(const __grid_constant__ BoundArgs a) {
  constexpr int VEC = HD / 8, STEP = kBoundThreads / VEC;
  __shared__ uint4 s_low[HEADS][kBoundThreads], s_high[HEADS][kBoundThreads];
  const int tid = threadIdx.x, r = blockIdx.x / a.candidates, c = blockIdx.x % a.candidates, head = blockIdx.y * HEADS;
  pdl_wait();
  pdl_launch();
  const int trow = a.rows ? a.rows[r] : r, cap = a.width * a.page_size;
  int len = a.lens[r];
  if (len <= 0) return;
  const bool tell = c == 0 && head == 0 && tid == 0;
  if ((unsigned)trow >= (unsigned)a.table_rows) {
    if (tell) report(a.status, MK_ERR_PAGES, PO_BOUNDS, r, trow);
    return;
  }
  if (len > cap) {
    if (tell) report(a.status, MK_ERR_PAGES, PO_BOUNDS, r, len);
    len = cap;
  }
  const int first = max(0, len - a.n_new) / a.page_size, j = first + c;  // (the last positions that are in the table)
  if ((long long)j * a.page_size >= len) return;
  const int page = a.table[(long long)trow * a.table_stride + j];
  if ((unsigned)page >= (unsigned)a.n_pages) {
    if (head == 0 && tid == 0) report(a.status, MK_ERR_PAGES, PO_BOUNDS, r, page);
    return;
  }
  const int held = min(a.page_size, len - j * a.page_size), v = tid % VEC;
  const C* src = static_cast<const C*>(a.k) + page * a.page_stride + (long long)head * a.page_size * HD + v * 8;
  constexpr uint32_t kInf = Pair<C>::kInf, kNeg = kInf | 0x80008000u;
  auto join = [](uint4& low, uint4& high, const uint4& l, const uint4& h) {
    low = make_uint4(min2<C>(low.x, l.x), min2<C>(low.y, l.y), min2<C>(low.z, l.z), min2<C>(low.w, l.w));
    high = make_uint4(max2<C>(high.x, h.x), max2<C>(high.y, h.y), max2<C>(high.z, h.z), max2<C>(high.w, h.w));
  };
  uint4 low[HEADS], high[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    low[h] = make_uint4(kInf, kInf, kInf, kInf);
    high[h] = make_uint4(kNeg, kNeg, kNeg, kNeg);
  }
  constexpr int U = 8 / HEADS;
  for (int p = tid / VEC; p < held; p += U * STEP) {
    uint4 x[HEADS][U];
#pragma unroll
    for (int h = 0; h < HEADS; ++h)  // past the last key or head: the last one again, no matter
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[h][u] = ldg_stream(src + ((long long)min(h, a.hkv - 1 - head) * a.page_size + min(p + u * STEP, held - 1)) * HD);
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
#pragma unroll
      for (int u = 0; u < U; ++u) join(low[h], high[h], x[h][u], x[h][u]);
  }
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    s_low[h][tid] = low[h];
    s_high[h][tid] = high[h];
  }
  __syncthreads();
  // a thread per head, bound and 16 bytes
  for (int x = tid; x < HEADS * 2 * VEC; x += kBoundThreads) {
    const int h = x / (2 * VEC), at = x % VEC;
    const bool up = x / VEC % 2;
    if (head + h >= a.hkv) break;
    uint4 l = s_low[h][at], u = s_high[h][at];
    for (int y = 1; y < STEP; ++y) join(l, u, s_low[h][y * VEC + at], s_high[h][y * VEC + at]);
    C* dst = static_cast<C*>(a.bounds) + (((long long)page * a.hkv + head + h) * 2 + up) * HD + at * 8;
    *reinterpret_cast<uint4*>(dst) = up ? u : l;
  }
}

// ------------------------------------------------------------------------------ scores
constexpr int kScoreWarps = 8, kScoreThreads = 32 * kScoreWarps;
constexpr int kScorePages = 8;             // pages that a warp takes at a time

struct ScoreArgs {
  const void *q, *bounds;
  const int32_t *lens, *rows, *table;
  float* scores;
  int32_t* status;
  long long q_row, q_head, table_stride;
  int n_rows, hkv, group, page_size, n_pages, table_rows, width, chunk, q_vec;  // chunk: pages of a CTA
};

__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

// As q_d low_d or q_d high_d is the greater by q_d's sign alone, a score is one product of length 2 HD: of the
// queries' negative elements and then their positive ones with a page's lower bounds and then its upper ones,
// which lie one behind the other.  A warp takes eight pages: tensor-core tiles m16n8k16 of 16 rows of heads (up to
// 8 heads: row g the head's first part, row g + 8 the second; more: a row per head) and 8 columns of pages, whose
// fragments come straight from memory, 16 bytes a lane, as the elements may be summed in any order the two
// operands share.  The lower and the upper half are summed apart, in two chains.  Where a sum is not finite (an
// infinite bound times the zero of the other sign) the warp takes those pages once more without the tensor
// cores.  Bound: the bounds' bytes (16
// rows of 1024 to 2048 pages of 16 positions, 105 MB: 21.6 us, 4.9 TB/s; warps that multiplied on CUDA cores and added
// up through the lanes took 84); of one row the chain from the length over the table to the bounds (3.5 us).
template <typename C, typename Q, int HD, bool WIDE, int NQ>
struct ScoreSmem {
  static constexpr int I = HD / 16;        // chunks of 32 elements of both halves
  static constexpr int RH = WIDE ? 2 : 1;
  uint4 q[kScoreWarps][NQ][I][RH][32];
  float scale[kScoreWarps][16];
};
template <typename C, typename Q, int HD, bool WIDE, int NQ>
__global__ void __launch_bounds__(kScoreThreads, 2) scores_kernel(const __grid_constant__ ScoreArgs a) {
  using SM = ScoreSmem<C, Q, HD, WIDE, NQ>;
  constexpr int I = SM::I, RH = SM::RH;
  extern __shared__ __align__(16) unsigned char score_smem[];
  SM* sm = reinterpret_cast<SM*>(score_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_launch();
  const int trow = a.rows ? a.rows[r] : r, cap = a.width * a.page_size;
  const bool tell = blockIdx.x == 0 && threadIdx.x == 0;
  int len = max(0, a.lens[r]);
  if ((unsigned)trow >= (unsigned)a.table_rows) {
    if (tell && len > 0) report(a.status, MK_ERR_PAGES, PO_SCORES, r, trow);
    len = 0;
  }
  if (len > cap) {
    if (tell) report(a.status, MK_ERR_PAGES, PO_SCORES, r, len);
    len = cap;
  }
  const int pages = (len + a.page_size - 1) / a.page_size;
  const int begin = blockIdx.x * a.chunk, end = min(a.width, begin + a.chunk);
  const int per = min(a.hkv, kScoreWarps), subs = kScoreWarps / per, sub = warp / per;
  if (sub >= subs) return;
  const int32_t* table = a.table + (long long)(len > 0 ? trow : 0) * a.table_stride;
  const int step = subs * kScorePages, first = begin + sub * kScorePages;
  // the table's entry for this lane's column, asked for some turns ahead, and the page it names, -1 where that is none
  const int last = min(pages, end);
  auto entry_of = [&](int j) { return j < last ? table[j] : 0; };
  auto page_of = [&](int j, int entry, bool tell_bad) {
    if (j >= last) return -1;
    if ((unsigned)entry < (unsigned)a.n_pages) return entry;
    if (tell_bad && c == 0) report(a.status, MK_ERR_PAGES, PO_SCORES, r, entry);
    return -1;
  };
  for (int head = warp % per; head < a.hkv; head += per) {
    float* out = a.scores + ((long long)r * a.hkv + head) * a.width;
    const Q* q0 = static_cast<const Q*>(a.q) + (long long)r * a.q_row + (long long)head * a.group * a.q_head + 8 * c;
    const C* b0 = static_cast<const C*>(a.bounds) + (long long)head * 2 * HD + 8 * c;
    uint4 raw[I];
    auto load = [&](int page) {
#pragma unroll
      for (int i = 0; i < I; ++i)
        raw[i] = page >= 0 ? ldg_stream(b0 + (long long)page * a.hkv * 2 * HD + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    };
    const int entry = entry_of(first + g);
    int ahead = entry_of(first + step + g), page = -1;
    // ---- the queries' fragments: chunk i, lane (g, c): elements [32 i + 8 c, + 8) of head g
    if (first < pages) {
      __syncwarp();
#pragma unroll 1
      for (int rh = 0; rh < RH; ++rh) {
        const int h = g + 8 * rh;
        Raw8<Q> x[I / 2];
#pragma unroll
        for (int i = 0; i < I / 2; ++i) {
          x[i] = {};
          if (h < a.group) {
            if (a.q_vec)
              x[i].load(q0 + h * a.q_head + 32 * i);
            else
              x[i].gather(q0 + h * a.q_head + 32 * i);
          }
        }
        if (rh == 0) {  // (the first bounds go out behind the queries)
          page = page_of(first + g, entry, head == 0);
          load(page);
        }
        float up = 1.f;
        if constexpr (kScaled<C, Q>) {
          float most = 0.f;
#pragma unroll
          for (int i = 0; i < I / 2; ++i) {
            float v[8];
            x[i].up(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
          }
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const int shift = shift_of(most);
          up = power_of(shift);
          if (c == 0) sm->scale[warp][h] = power_of(-shift);
        }
#pragma unroll
        for (int i = 0; i < I / 2; ++i) {
          float v[8];
          x[i].up(v);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w[4][NQ];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = v[2 * e] * up, z = v[2 * e + 1] * up;
              split2<C, NQ>((half ? y > 0.f : y < 0.f) || y != y ? y : 0.f, (half ? z > 0.f : z < 0.f) || z != z ? z : 0.f, w[e]);
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
              sm->q[warp][n][half * (I / 2) + i][rh][lane] = make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]);
          }
        }
      }
      __syncwarp();
    }
    for (int j0 = first; j0 < end; j0 += step) {
      float best[2] = {-INFINITY, -INFINITY};  // of pages j0 + 2 c and the next one
      if (j0 < pages) {
        uint4 now[I];
#pragma unroll
        for (int i = 0; i < I; ++i) now[i] = raw[i];
        const int mine = page;
        page = page_of(j0 + step + g, ahead, head == 0);
        ahead = entry_of(j0 + 2 * step + g);
        if (j0 + step < pages) load(page);
        constexpr int SETS = WIDE ? NQ : (NQ + 1) / 2;
        float d[SETS][2][4];
#pragma unroll
        for (int n = 0; n < SETS; ++n)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[n][half][e] = 0.f;
#pragma unroll
            for (int i = half * (I / 2); i < (half + 1) * (I / 2); ++i) {
              const int n0 = WIDE ? n : 2 * n;
              const uint4 u = sm->q[warp][n0][i][0][lane];
              const uint4 w = WIDE ? sm->q[warp][n0][i][RH - 1][lane]
                              : n0 + 1 < NQ ? sm->q[warp][n0 + 1 < NQ ? n0 + 1 : 0][i][0][lane] : make_uint4(0u, 0u, 0u, 0u);
              Mma<C>::run(d[n][half], make_uint4(u.x, w.x, u.y, w.y), now[i].x, now[i].y);
              Mma<C>::run(d[n][half], make_uint4(u.z, w.z, u.w, w.w), now[i].z, now[i].w);
            }
          }
        bool odd = false;
#pragma unroll
        for (int rh = 0; rh < RH; ++rh) {
          const int h = g + 8 * rh;
          const float scale = kScaled<C, Q> ? sm->scale[warp][h] : 1.f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float s = 0.f;
#pragma unroll
            for (int n = SETS - 1; n >= 0; --n) {  // the smallest parts first
              if (!WIDE && 2 * n + 1 < NQ) s += d[n][0][2 + e] + d[n][1][2 + e];
              s += d[n][0][2 * rh + e] + d[n][1][2 * rh + e];
            }
            s *= scale;
            odd = odd || !(fabsf(s) < INFINITY);
            if (h < a.group) best[e] = fmaxf(best[e], s);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) best[e] = fmaxf(best[e], __shfl_xor_sync(0xffffffffu, best[e], o));
        // the four lanes of a page together; what is not a half's to add adds nothing, but a NaN bound is one under any query
        if (__any_sync(0xffffffffu, odd)) {
          float most = -INFINITY;
          for (int h = 0; h < a.group; ++h) {
            float s = 0.f;
#pragma unroll 1
            for (int i = 0; i < I / 2; ++i)
              for (int e = 0; e < 8; ++e) {
                const float x = Conv<Q>::up(q0[h * a.q_head + 32 * i + e]);
                float lo = 0.f, hi = 0.f;
                if (mine >= 0) {
                  lo = Conv<C>::up(b0[(long long)mine * a.hkv * 2 * HD + 32 * i + e]);
                  hi = Conv<C>::up(b0[(long long)mine * a.hkv * 2 * HD + HD + 32 * i + e]);
                }
                s += !(lo == lo && hi == hi) ? lo + hi : x == 0.f ? 0.f : x > 0.f ? x * hi : x * lo;
              }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            most = max_nan(most, s);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) best[e] = __shfl_sync(0xffffffffu, most, 4 * (2 * c + e));
        }
        const unsigned there = __ballot_sync(0xffffffffu, mine >= 0);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!(there >> (4 * (2 * c + e)) & 1)) best[e] = -INFINITY;
      }
      if (g == 0)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (j0 + 2 * c + e < end) out[j0 + 2 * c + e] = best[e];
    }
  }
}

// ------------------------------------------------------------------------------ choice
constexpr int kChooseThreads = 512, kChooseKeys = 4;

struct ChooseArgs {
  const float* scores;
  const int32_t *lens, *rows, *table;
  int32_t *pages, *chosen, *out_lens, *status;  // pages: numbers for the caller; chosen: the attention's table
  long long scores_row, scores_head, table_stride;
  int n_rows, hkv, page_size, table_rows, width, n_blocks, first, last;
};

// the order of the scores as whole numbers: NaN as +inf, zeros of either sign alike
__device__ __forceinline__ uint32_t key_of(float x) { return orderable(x != x ? INFINITY : x + 0.f); }

// One CTA per row and kv head: the key of the last page to be taken by its bytes, from the top (a count of
// the pages that share the bytes found so far, 256 counters a turn; equal bytes of a warp count at once, as the
// first bytes of most scores are), then the pages in order: all with a greater key and the first of those
// with the same.  Keys of up to kChooseThreads * kChooseKeys pages stay in registers.  Bound: latency, some barriers
// a byte (128 segments of 512 to 1024 pages: about 5 of the 56 us of the whole call; one launch before the attention's).
template <bool KEPT>
__global__ void __launch_bounds__(kChooseThreads) choose_kernel(const __grid_constant__ ChooseArgs a) {
  constexpr int W = kChooseThreads / 32;
  __shared__ int s_count[256], s_warp[2][W][2], s_digit, s_left, s_whole;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x, head = blockIdx.y;
  pdl_wait();
  pdl_launch();
  const int trow = a.rows ? a.rows[r] : r, cap = a.width * a.page_size;
  int len = max(0, a.lens[r]);
  const bool tell = head == 0 && tid == 0;
  if ((unsigned)trow >= (unsigned)a.table_rows) {
    if (tell && len > 0) report(a.status, MK_ERR_PAGES, PO_SPARSE, r, trow);
    len = 0;
  }
  if (len > cap) {
    if (tell) report(a.status, MK_ERR_PAGES, PO_SPARSE, r, len);
    len = cap;
  }
  const int n = (len + a.page_size - 1) / a.page_size, taken = min(n, a.n_blocks);
  const int32_t* table = a.table + (long long)(len > 0 ? trow : 0) * a.table_stride;
  const float* score = a.scores + r * a.scores_row + head * a.scores_head;
  const long long at = ((long long)r * a.hkv + head) * a.n_blocks;
  // the page that ends inside is the last one taken
  if (tell) a.out_lens[r] = len - (n - taken) * a.page_size;
  const int begin = n > a.n_blocks ? a.first : 0, end = n > a.n_blocks ? n - a.last : 0;  // pages that are chosen among
  int left = n > a.n_blocks ? a.n_blocks - a.first - a.last : 0;                            // how many of them
  uint32_t limit = 0xffffffffu;  // above it: taken; at it: the first `left`
  bool whole = false;            // at or above it: taken
  uint32_t kept[KEPT ? kChooseKeys : 1];
  if (KEPT) {
#pragma unroll
    for (int i = 0; i < kChooseKeys; ++i) {
      const int j = i * kChooseThreads + tid;
      kept[i] = j >= begin && j < end && left > 0 ? key_of(score[j]) : 0u;
    }
  }
  if (left > 0) {
    uint32_t prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kChooseThreads) s_count[i] = 0;
      __syncthreads();
      auto count = [&](int j, uint32_t k) {
        const bool in = j >= begin && j < end && (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)));
        const unsigned digit = in ? k >> shift & 255u : 256u;
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        if (in && lane == __ffs(same) - 1) atomicAdd(&s_count[digit], __popc(same));
      };
      if (KEPT) {
#pragma unroll
        for (int i = 0; i < kChooseKeys; ++i)
          if (i * kChooseThreads < end) count(i * kChooseThreads + tid, kept[i]);
      } else {
        for (int base = 0; base < end; base += kChooseThreads) count(base + tid, base + tid < end ? key_of(score[base + tid]) : 0u);
      }
      __syncthreads();
      if (tid < 32) {  // the greatest digit with at least `left` pages at or above it; a lane 8 digits
        int c[8], mine = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          c[e] = s_count[255 - (lane * 8 + e)];
          mine += c[e];
        }
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += x;
        }
        before -= mine;
        if (before < left && before + mine >= left) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (before < left && before + c[e] >= left) {
              s_digit = 255 - (lane * 8 + e);
              s_left = left - before;
              s_whole = c[e] == left - before;
            }
            before += c[e];
          }
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift;
      left = s_left;
      // all that share the bytes so far are taken: nothing is left to tell apart
      whole = s_whole;
      if (whole) break;
    }
    limit = prefix;
  }
  int out = 0, same = 0;  // pages written, pages met at the limit
  auto take = [&](int i, uint32_t k) {
    const int j = i * kChooseThreads + tid;
    const bool among = j >= begin && j < end && left > 0;
    const bool equal = among && !whole && k == limit;
    const bool more = j < n && (j < begin || j >= end || (among && (whole ? k >= limit : k > limit)));
    // those with the same key come before this one as far as they are taken: their places are counted apart
    const unsigned eq = __ballot_sync(0xffffffffu, equal), mo = __ballot_sync(0xffffffffu, more);
    int(*counts)[2] = s_warp[i & 1];
    if (lane == 0) {
      counts[warp][0] = __popc(eq);
      counts[warp][1] = __popc(mo);
    }
    __syncthreads();
    int rank = same + __popc(eq & ((1u << lane) - 1)), place = out + __popc(mo & ((1u << lane) - 1));
    int all_eq = 0, all_mo = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      rank += w < warp ? counts[w][0] : 0;
      place += w < warp ? counts[w][1] : 0;
      all_eq += counts[w][0];
      all_mo += counts[w][1];
    }
    if (more || (equal && rank < left)) {
      place += min(rank, left);
      a.chosen[at + place] = table[j];
      if (a.pages) a.pages[at + place] = j;
    }
    same += all_eq;
    out += all_mo;
  };
  if (KEPT) {
#pragma unroll
    for (int i = 0; i < kChooseKeys; ++i)
      if (i * kChooseThreads < n) take(i, kept[i]);
  } else {
    for (int i = 0; i * kChooseThreads < n; ++i) {
      const int j = i * kChooseThreads + tid;
      take(i, j >= begin && j < end && left > 0 ? key_of(score[j]) : 0u);
    }
  }
  for (int i = taken + tid; i < a.n_blocks; i += kChooseThreads) {
    a.chosen[at + i] = -1;
    if (a.pages) a.pages[at + i] = -1;
  }
}

template <typename C, typename Q, int HD, bool WIDE, int NQ>
mk_status launch_scores(const ScoreArgs& a, void* stream) {
  auto kernel = scores_kernel<C, Q, HD, WIDE, NQ>;
  constexpr int smem = sizeof(ScoreSmem<C, Q, HD, WIDE, NQ>);
  static SmemLimit limit;
  const mk_status s = smem > 48 * 1024 ? limit.raise(kernel, smem, "mk_page_scores") : MK_OK;
  if (s) return s;
  return launch_dependent(kernel, dim3((a.width + a.chunk - 1) / a.chunk, a.n_rows), dim3(kScoreThreads), smem, stream, "mk_page_scores", a);
}
template <typename C, typename Q, int NQ>
mk_status launch_scores(const ScoreArgs& a, int hd, void* stream) {
  if (a.group > 8) return hd == 64 ? launch_scores<C, Q, 64, true, NQ>(a, stream) : launch_scores<C, Q, 128, true, NQ>(a, stream);
  return hd == 64 ? launch_scores<C, Q, 64, false, NQ>(a, stream) : launch_scores<C, Q, 128, false, NQ>(a, stream);
}

size_t choice_bytes(long long n_rows, int n_kv_heads, int n_blocks) {
  return round16(4 * (size_t)n_rows) + round16(4 * (size_t)n_rows * n_kv_heads * n_blocks);
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_update_bounds(const mk_bounds_args* args, const mk_page_view* cache, int32_t* status, void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    const std::string e = check_view(cache);
    if (!e.empty()) return paged_fail(MK_ERR_INVALID, e);
    if (!args || !args->bounds || !args->lens) return paged_fail(MK_ERR_INVALID, "NULL argument");
    if (!aligned_to(args->bounds, 16)) return paged_fail(MK_ERR_INVALID, "bounds must be 16-byte aligned");
    if (args->n_new < 1) return paged_fail(MK_ERR_INVALID, "n_new must be positive");
    BoundArgs a{};
    a.k = cache->k; a.bounds = args->bounds; a.lens = args->lens; a.rows = args->rows; a.table = cache->table;
    a.status = status; a.page_stride = cache->page_stride; a.table_stride = cache->table_stride;
    a.n_rows = args->n_rows; a.n_new = args->n_new; a.hkv = cache->n_kv_heads; a.page_size = cache->page_size;
    a.n_pages = cache->n_pages; a.table_rows = cache->n_rows; a.width = cache->table_width;
    // n_new positions lie in at most this many pages
    a.candidates = (int)std::min<long long>(a.width, (args->n_new + 2LL * a.page_size - 2) / a.page_size);
    if (args->n_rows < 0 || (long long)args->n_rows * a.candidates > 0x7fffffffLL)
      return paged_fail(MK_ERR_INVALID, "n_rows * the pages of n_new positions must be in [0, 2^31)");
    if (args->n_rows == 0) return MK_OK;
    // two heads to a CTA where a page's keys of one are no eight loads of a thread, and CTAs are many
    int n_sm = 0;
    const mk_status s = sm_count(&n_sm);
    if (s) return s;
    const bool two = a.page_size * cache->head_dim < 8192 && (long long)a.n_rows * a.candidates * a.hkv >= 64LL * n_sm;
    const dim3 grid(a.n_rows * a.candidates, two ? (a.hkv + 1) / 2 : a.hkv);
    auto go = [&](auto kernel) { return launch_dependent(kernel, grid, dim3(kBoundThreads), 0, stream, "mk_update_bounds", a); };
    auto typed = [&](auto zero) {
      using C = decltype(zero);
      if (cache->head_dim == 64) return two ? go(bounds_kernel<C, 64, 2>) : go(bounds_kernel<C, 64, 1>);
      return two ? go(bounds_kernel<C, 128, 2>) : go(bounds_kernel<C, 128, 1>);
    };
    return cache->dtype == MK_F16 ? typed(__half()) : typed(__nv_bfloat16());
  });
}

extern "C" mk_status mk_page_scores(const mk_scores_args* args, const mk_page_view* cache, int32_t* status, void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    const std::string e = check_view(cache);
    if (!e.empty()) return paged_fail(MK_ERR_INVALID, e);
    if (!args || !args->q || !args->bounds || !args->lens || !args->scores) return paged_fail(MK_ERR_INVALID, "NULL argument");
    if (args->dtype < MK_F16 || args->dtype > MK_F32) return paged_fail(MK_ERR_INVALID, "dtype");
    if (args->n_heads < 1 || args->n_heads % cache->n_kv_heads || args->n_heads / cache->n_kv_heads > kMaxGroup)
      return paged_fail(MK_ERR_INVALID, "n_heads / n_kv_heads must be a whole number in [1, 16]");
    if (args->n_rows < 0 || args->n_rows > 65535) return paged_fail(MK_ERR_INVALID, "n_rows must be in [0, 65535]");
    if (!aligned_to(args->bounds, 16) || !aligned_to(args->scores, 4) || !aligned_to(args->q, args->dtype == MK_F32 ? 4 : 2))
      return paged_fail(MK_ERR_INVALID, "bounds must be 16-byte aligned, q and scores to their type");
    if (args->n_rows == 0) return MK_OK;
    ScoreArgs a{};
    a.q = args->q; a.bounds = args->bounds; a.lens = args->lens; a.rows = args->rows; a.table = cache->table;
    a.scores = args->scores; a.status = status; a.q_row = args->q_row; a.q_head = args->q_head;
    a.table_stride = cache->table_stride; a.n_rows = args->n_rows; a.hkv = cache->n_kv_heads;
    a.group = args->n_heads / cache->n_kv_heads; a.page_size = cache->page_size; a.n_pages = cache->n_pages;
    a.table_rows = cache->n_rows; a.width = cache->table_width;
    const long long per = args->dtype == MK_F32 ? 4 : 8;
    a.q_vec = aligned_to(a.q, 16) && a.q_row % per == 0 && a.q_head % per == 0;
    // pages of a CTA: as many as leave two CTAs for every SM (one wave), in whole turns of its warps, up to 96 or what whole
    // turns leave of that (8 kv heads, 16 ragged rows of up to 2048 pages: 21.6 us; 64 pages 25.7, 128 23.5, 256 34.4)
    int n_sm = 0;
    const mk_status s = sm_count(&n_sm);
    if (s) return s;
    const int turn = kScorePages * std::max(1, kScoreWarps / a.hkv);
    const long long want = (long long)a.width * a.n_rows / (2LL * n_sm);
    a.chunk = (int)std::min<long long>(96 / turn, std::max<long long>(1, want / turn)) * turn;
    // queries of the bounds' type are exact in one part, others are split as the attention splits them: into 2 parts of
    // fp16 (22 bits, each head at a power of two of its own; a third part would bring 32-bit queries' scores from 2.6e-7
    // to 1e-7 of 64 bits and take 16 rows of 24576 positions in pages of 16 from 21.6 to 29.9 us) or 3 of bf16 (24 bits; fp16
    // queries: 2, 16 bits and more than their 11)
    const int d = cache->head_dim;
    if (cache->dtype == MK_F16) {
      if (args->dtype == MK_F16) return launch_scores<__half, __half, 1>(a, d, stream);
      if (args->dtype == MK_BF16) return launch_scores<__half, __nv_bfloat16, 2>(a, d, stream);
      return launch_scores<__half, float, 2>(a, d, stream);
    }
    if (args->dtype == MK_BF16) return launch_scores<__nv_bfloat16, __nv_bfloat16, 1>(a, d, stream);
    if (args->dtype == MK_F16) return launch_scores<__nv_bfloat16, __half, 2>(a, d, stream);
    return launch_scores<__nv_bfloat16, float, 3>(a, d, stream);
  });
}

extern "C" mk_status mk_sparse_attention_workspace(int n_rows, int n_heads, int n_kv_heads, int head_dim, int n_blocks,
                                                   size_t* bytes) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    if (!bytes) return paged_fail(MK_ERR_INVALID, "bytes is NULL");
    if (n_rows < 0 || n_blocks < 1 || n_blocks > 65536)
      return paged_fail(MK_ERR_INVALID, "n_rows must not be negative, n_blocks in [1, 65536]");
    const mk_status s = mk_paged_attention_workspace(n_heads, n_kv_heads, head_dim, bytes);
    if (s) return s;
    *bytes = round16(*bytes) + choice_bytes(n_rows, n_kv_heads, n_blocks);
    return MK_OK;
  });
}

extern "C" mk_status mk_sparse_attention(const mk_attend_args* attend, const mk_sparse_args* args, const mk_page_view* cache,
                                         int32_t* status, void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    const std::string e = check_view(cache);
    if (!e.empty()) return paged_fail(MK_ERR_INVALID, e);
    if (!attend || !args || !args->scores || !attend->lens) return paged_fail(MK_ERR_INVALID, "NULL argument");
    if (!aligned_to(args->scores, 4)) return paged_fail(MK_ERR_INVALID, "scores must be aligned to their type");
    if (attend->window) return paged_fail(MK_ERR_INVALID, "chosen pages have no window");
    if (args->first < 0 || args->last < 1 || args->n_blocks < 1 || args->n_blocks > 65536 ||
        (long long)args->first + args->last > args->n_blocks)
      return paged_fail(MK_ERR_INVALID, "first must not be negative, last positive, n_blocks at least their sum and at most 65536");
    if ((long long)args->n_blocks * cache->page_size > (1LL << 30))
      return paged_fail(MK_ERR_INVALID, "n_blocks * page_size must be at most 2^30");
    size_t need = 0;
    mk_status s = mk_sparse_attention_workspace(attend->n_rows, attend->n_heads, cache->n_kv_heads, cache->head_dim,
                                                args->n_blocks, &need);
    if (s) return s;
    if (!attend->workspace || !aligned_to(attend->workspace, 16) || attend->workspace_bytes < need)
      return paged_fail(MK_ERR_INVALID, "the workspace is missing, unaligned or too small (mk_sparse_attention_workspace)");
    ChooseArgs c{};
    c.scores = args->scores; c.scores_row = args->scores_row; c.scores_head = args->scores_head;
    c.lens = attend->lens; c.rows = attend->rows; c.table = cache->table; c.table_stride = cache->table_stride;
    c.pages = args->pages; c.status = status;
    c.out_lens = static_cast<int32_t*>(attend->workspace);
    c.chosen = reinterpret_cast<int32_t*>(static_cast<char*>(attend->workspace) + round16(4 * (size_t)attend->n_rows));
    c.n_rows = attend->n_rows; c.hkv = cache->n_kv_heads; c.page_size = cache->page_size; c.table_rows = cache->n_rows;
    c.width = cache->table_width; c.n_blocks = args->n_blocks; c.first = args->first; c.last = args->last;
    // what the attention sees: a table row per row and kv head
    mk_page_view view = *cache;
    view.table = c.chosen; view.n_rows = attend->n_rows; view.table_width = args->n_blocks;
    view.table_stride = (long long)cache->n_kv_heads * args->n_blocks;
    mk_attend_args x = *attend;
    x.lens = c.out_lens; x.len_add = 0; x.rows = nullptr;
    const size_t used = choice_bytes(attend->n_rows, cache->n_kv_heads, args->n_blocks);
    x.workspace = static_cast<char*>(attend->workspace) + used;
    x.workspace_bytes = attend->workspace_bytes - used;
    auto choose = [&]() {
      return launch_dependent(c.width <= kChooseThreads * kChooseKeys ? choose_kernel<true> : choose_kernel<false>,
                              dim3(c.n_rows, c.hkv), dim3(kChooseThreads), 0, stream, "mk_sparse_attention (choice)", c);
    };
    return attend_pages(x, view, args->n_blocks, status, stream, choose);
  });
}
