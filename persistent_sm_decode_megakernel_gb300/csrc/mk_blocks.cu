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

// A CTA takes one kv head of one page: a thread 16 bytes of every kBoundThreads / (HD / 8)-th key,
// pairs of elements compared as they lie there; what the threads found is joined in shared memory.
template <typename C, int HD>
__global__ void __launch_bounds__(kBoundThreads) bounds_kernel(const __grid_constant__ BoundArgs a) {
  constexpr int VEC = HD / 8, STEP = kBoundThreads / VEC;
  __shared__ uint4 s_low[kBoundThreads], s_high[kBoundThreads];
  const int tid = threadIdx.x, r = blockIdx.x / a.candidates, c = blockIdx.x % a.candidates, head = blockIdx.y;
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
  uint4 low = make_uint4(kInf, kInf, kInf, kInf), high = make_uint4(kNeg, kNeg, kNeg, kNeg);
  auto join = [&](const uint4& l, const uint4& h) {
    low = make_uint4(min2<C>(low.x, l.x), min2<C>(low.y, l.y), min2<C>(low.z, l.z), min2<C>(low.w, l.w));
    high = make_uint4(max2<C>(high.x, h.x), max2<C>(high.y, h.y), max2<C>(high.z, h.z), max2<C>(high.w, h.w));
  };
  constexpr int U = 8;
  for (int p = tid / VEC; p < held; p += U * STEP) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = ldg_stream(src + (long long)min(p + u * STEP, held - 1) * HD);  // the last one again: no matter
#pragma unroll
    for (int u = 0; u < U; ++u) join(x[u], x[u]);
  }
  s_low[tid] = low;
  s_high[tid] = high;
  __syncthreads();
  if (tid >= 2 * VEC) return;
  const bool up = tid >= VEC;
  for (int y = 0; y < STEP; ++y) join(s_low[y * VEC + v], s_high[y * VEC + v]);
  C* dst = static_cast<C*>(a.bounds) + (((long long)page * a.hkv + head) * 2 + up) * HD + v * 8;
  *reinterpret_cast<uint4*>(dst) = up ? high : low;
}

// ------------------------------------------------------------------------------ scores
constexpr int kScoreThreads = 256;

struct ScoreArgs {
  const void *q, *bounds;
  const int32_t *lens, *rows, *table;
  float* scores;
  int32_t* status;
  long long q_row, q_head, table_stride;
  int n_rows, hkv, group, page_size, n_pages, table_rows, width;
};

// A warp takes a page of one row and kv head, a lane HD / 32 elements; the heads' sums go through the lanes.
template <typename C, typename Q, int HD>
__global__ void __launch_bounds__(kScoreThreads) scores_kernel(const __grid_constant__ ScoreArgs a) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = blockIdx.y, r = blockIdx.z;
  pdl_wait();
  pdl_launch();
  const int j = blockIdx.x * (kScoreThreads / 32) + warp;
  if (j >= a.width) return;
  const int trow = a.rows ? a.rows[r] : r, cap = a.width * a.page_size;
  const bool tell = j == 0 && head == 0 && lane == 0;
  int len = a.lens[r];
  if ((unsigned)trow >= (unsigned)a.table_rows) {
    if (tell && len > 0) report(a.status, MK_ERR_PAGES, PO_SCORES, r, trow);
    len = 0;
  }
  if (len > cap && tell) report(a.status, MK_ERR_PAGES, PO_SCORES, r, len);
  float best = -INFINITY;
  if (len > 0 && (long long)j * a.page_size < len) {
    const int page = a.table[(long long)trow * a.table_stride + j];
    if ((unsigned)page >= (unsigned)a.n_pages) {
      if (head == 0 && lane == 0) report(a.status, MK_ERR_PAGES, PO_SCORES, r, page);
    } else {
      const C* b = static_cast<const C*>(a.bounds) + ((long long)page * a.hkv + head) * 2 * HD + lane;
      float lo[E], hi[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        lo[e] = Conv<C>::up(b[32 * e]);
        hi[e] = Conv<C>::up(b[HD + 32 * e]);
      }
      for (int h = 0; h < a.group; ++h) {
        const Q* q = static_cast<const Q*>(a.q) + (long long)r * a.q_row + (long long)(head * a.group + h) * a.q_head + lane;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float x = Conv<Q>::up(q[32 * e]);
          s = fmaf(x, x > 0.f ? hi[e] : lo[e], s);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        best = s != s || best != best ? NAN : fmaxf(best, s);
      }
    }
  }
  if (lane == 0) a.scores[((long long)r * a.hkv + head) * a.width + j] = best;
}

// ------------------------------------------------------------------------------ choice
constexpr int kChooseThreads = 256;

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
// the pages that share the bytes found so far, 256 counters a turn), then the pages in order: all with
// a greater key and the first of those with the same.
__global__ void __launch_bounds__(kChooseThreads) choose_kernel(const __grid_constant__ ChooseArgs a) {
  __shared__ int s_count[256], s_warp[kChooseThreads / 32][2], s_digit, s_left;
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
  const int n = (int)(((long long)len + a.page_size - 1) / a.page_size), taken = min(n, a.n_blocks);
  const int32_t* table = a.table + (long long)(len > 0 ? trow : 0) * a.table_stride;
  const float* score = a.scores + r * a.scores_row + head * a.scores_head;
  const long long at = ((long long)r * a.hkv + head) * a.n_blocks;
  // the page that ends inside is the last one taken
  if (tell) a.out_lens[r] = len - (n - taken) * a.page_size;
  const int begin = n > a.n_blocks ? a.first : 0, end = n > a.n_blocks ? n - a.last : 0;  // pages that are chosen among
  int left = n > a.n_blocks ? a.n_blocks - a.first - a.last : 0;                            // how many of them
  uint32_t limit = 0xffffffffu;  // above it: taken; at it: the first `left`
  if (left > 0) {
    uint32_t prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kChooseThreads) s_count[i] = 0;
      __syncthreads();
      for (int j = begin + tid; j < end; j += kChooseThreads) {
        const uint32_t k = key_of(score[j]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_count[k >> shift & 255], 1);
      }
      __syncthreads();
      if (tid < 32) {  // the greatest digit with at least `left` pages at or above it; a lane 8 digits
        int mine = 0;
        for (int e = 0; e < 8; ++e) mine += s_count[255 - (lane * 8 + e)];
        int before = mine;
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += x;
        }
        before -= mine;
        if (before < left && before + mine >= left)
          for (int e = 0; e < 8; ++e) {
            const int c = s_count[255 - (lane * 8 + e)];
            if (before < left && before + c >= left) {
              s_digit = 255 - (lane * 8 + e);
              s_left = left - before;
            }
            before += c;
          }
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift;
      left = s_left;
      __syncthreads();
    }
    limit = prefix;
  }
  int out = 0, same = 0;  // pages written, pages met at the limit
  for (int base = 0; base < n; base += kChooseThreads) {
    const int j = base + tid;
    const bool among = j >= begin && j < end;
    const uint32_t k = among && left > 0 ? key_of(score[j]) : 0;
    const bool equal = among && left > 0 && k == limit;
    bool in = j < n && (!among || (left > 0 && k > limit));
    const unsigned eq = __ballot_sync(0xffffffffu, equal);
    if (lane == 0) s_warp[warp][0] = __popc(eq);
    __syncthreads();
    int rank = same + __popc(eq & ((1u << lane) - 1));
    for (int w = 0; w < kChooseThreads / 32; ++w) {
      rank += w < warp ? s_warp[w][0] : 0;
      same += s_warp[w][0];
    }
    in = in || (equal && rank < left);
    const unsigned got = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_warp[warp][1] = __popc(got);
    __syncthreads();
    int place = out + __popc(got & ((1u << lane) - 1));
    for (int w = 0; w < kChooseThreads / 32; ++w) {
      place += w < warp ? s_warp[w][1] : 0;
      out += s_warp[w][1];
    }
    if (in) {
      a.chosen[at + place] = table[j];
      if (a.pages) a.pages[at + place] = j;
    }
    __syncthreads();
  }
  for (int i = taken + tid; i < a.n_blocks; i += kChooseThreads) {
    a.chosen[at + i] = -1;
    if (a.pages) a.pages[at + i] = -1;
  }
}

template <typename C>
mk_status launch_scores(const ScoreArgs& a, int dtype, int hd, dim3 grid, void* stream) {
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, dim3(kScoreThreads), 0, stream, "mk_page_scores", a); };
  if (dtype == MK_F32) return hd == 64 ? go(scores_kernel<C, float, 64>) : go(scores_kernel<C, float, 128>);
  if (dtype == MK_F16) return hd == 64 ? go(scores_kernel<C, __half, 64>) : go(scores_kernel<C, __half, 128>);
  return hd == 64 ? go(scores_kernel<C, __nv_bfloat16, 64>) : go(scores_kernel<C, __nv_bfloat16, 128>);
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
    const dim3 grid(a.n_rows * a.candidates, a.hkv);
    auto go = [&](auto kernel) { return launch_dependent(kernel, grid, dim3(kBoundThreads), 0, stream, "mk_update_bounds", a); };
    if (cache->dtype == MK_F16) return cache->head_dim == 64 ? go(bounds_kernel<__half, 64>) : go(bounds_kernel<__half, 128>);
    return cache->head_dim == 64 ? go(bounds_kernel<__nv_bfloat16, 64>) : go(bounds_kernel<__nv_bfloat16, 128>);
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
    const dim3 grid((a.width + kScoreThreads / 32 - 1) / (kScoreThreads / 32), a.hkv, a.n_rows);
    return cache->dtype == MK_F16 ? launch_scores<__half>(a, args->dtype, cache->head_dim, grid, stream)
                                  : launch_scores<__nv_bfloat16>(a, args->dtype, cache->head_dim, grid, stream);
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
    auto choose = [&]() { return launch_dependent(choose_kernel, dim3(c.n_rows, c.hkv), dim3(kChooseThreads), 0, stream,
                                                  "mk_sparse_attention (choice)", c); };
    return attend_pages(x, view, args->n_blocks, status, stream, choose);
  });
}
