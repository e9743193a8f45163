// Page table updates of a paged KV cache (mk_update_pages: fork, free, reserve) and its
// compaction (mk_compact_pages), with the copies of pages over all layers.
//
// Both are a plan of integers and a copy.  mk_update_pages takes three steps: `count` (a CTA
// per row) moves the holders' counts from the old table to the shared part of the new one and
// saves the old table; `plan` (one CTA) decides who copies a page, takes the lowest free
// pages by a scan of the counts and commits, or finds that it cannot; `apply` (all SMs) writes
// the table rows and copies the pages -- or, after a refusal, gives the counts back.  Tables
// of up to kCountInPlan entries are counted by the plan's CTA itself, which saves a launch.
// The counts are integer sums, so the order of their atomics does not show.
#include <algorithm>

#include "mk_paged.cuh"

namespace mk {
namespace {

constexpr int kMaxRows = 4096;
constexpr int kRowThreads = 256;
constexpr int kCopyThreads = 256;
constexpr int kUnitBytes = kCopyThreads * 16;  // a copy's unit: one 16-byte access per thread
constexpr int kInFlight = 6;                   // units a thread has in flight
constexpr int kCopyCtasPerSm = 4;
constexpr int kNarrowThreads = 256, kWideThreads = 1024;  // of the plan: one row per thread where that will do
constexpr int kCountInPlan = 2048;             // entries of a table that the plan counts itself
using u64 = unsigned long long;

struct PoolArgs {
  char *k, *v;
  int32_t *table, *refs, *lens, *status;
  const int32_t *parents, *reserve;
  long long page_bytes, page_stride, layer_stride, table_stride;
  int n_layers, n_pages, page_size, n_rows, width;
  // workspace
  int32_t *head;                     // [0] refused, [1] copies
  int32_t *held, *ends, *at, *copy;  // per row: pages taken over, pages after, first fresh page, copies its last
  int32_t *snap;                     // [n_rows][width]: the old table, entries that name no page as -1
  int32_t *fresh;                    // fresh pages in order (compaction: destinations)
  int32_t *src, *dst;                // the copies (compaction: sources in src, destinations in fresh)
  int32_t *rank;                     // compaction: [n_pages] a moved page's place in src, or -1
};

// what the workspace holds, in order
size_t lay_out(PoolArgs* a, void* ws, long long rows, long long width, long long pages) {
  char* p = static_cast<char*>(ws);
  size_t at = 0;
  auto take = [&](int32_t** out, long long n) {
    *out = reinterpret_cast<int32_t*>(p + at);
    at += round16(sizeof(int32_t) * (size_t)n);
  };
  take(&a->head, 4);
  take(&a->held, rows);
  take(&a->ends, rows);
  take(&a->at, rows);
  take(&a->copy, rows);
  take(&a->src, std::max(rows, pages));
  take(&a->dst, rows);
  take(&a->fresh, pages);
  take(&a->rank, pages);
  take(&a->snap, rows * width);
  return at;
}

// What row r takes over: its parent, the parent's positions and pages; false when the
// parent or its length cannot be (the whole call is then refused).
struct Take {
  int parent, len, held;
};
__device__ __forceinline__ bool take_of(const PoolArgs& a, int r, Take* t) {
  const int p = a.parents ? a.parents[r] : r;
  t->parent = p;
  t->len = t->held = 0;
  if (p == -1) return true;
  if ((unsigned)p >= (unsigned)a.n_rows) return false;
  const int n = a.lens[p];
  if (n < 0 || n > (long long)a.width * a.page_size) return false;
  t->len = n;
  t->held = (int)(((long long)n + a.page_size - 1) / a.page_size);
  return true;
}

__device__ __forceinline__ int page_or_none(const PoolArgs& a, int id) { return (unsigned)id < (unsigned)a.n_pages ? id : -1; }

// one entry of the table: saved, and the counts moved to what the row will hold there
__device__ __forceinline__ void count_entry(const PoolArgs& a, int r, int i, const Take& t, bool ok) {
  const int raw = a.table[(long long)r * a.table_stride + i], o = page_or_none(a, raw);
  int n = -1;
  if (ok && i < t.held) n = page_or_none(a, a.table[(long long)t.parent * a.table_stride + i]);
  if (raw >= a.n_pages) report(a.status, MK_ERR_PAGES, PO_UPDATE, r, raw);
  a.snap[(long long)r * a.width + i] = o;
  if (!ok || o == n) return;
  if (o >= 0) atomicSub(a.refs + o, 1);
  if (n >= 0) atomicAdd(a.refs + n, 1);
}

__global__ void __launch_bounds__(kRowThreads) count_kernel(const __grid_constant__ PoolArgs a) {
  pdl_wait();
  pdl_launch();
  const int r = blockIdx.x;
  Take t;
  const bool ok = take_of(a, r, &t);
  for (int i = threadIdx.x; i < a.width; i += kRowThreads) count_entry(a, r, i, t, ok);
}

// exclusive prefix sum of a number per thread over the CTA; the total in *total
template <int THREADS>
__device__ __forceinline__ u64 block_scan(u64 x, u64* sums, u64* total) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  u64 inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  u64 base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) base = all;
    all += sums[w];
  }
  *total = all;
  __syncthreads();
  return base + inc - x;
}

// Appends to `out` the ids in [from, to) for which want(refs[id]) holds, ascending, until
// `most` are found; returns how many were found (at most `most`).
template <int THREADS, typename Want>
__device__ __forceinline__ int list_pages(const int32_t* refs, int from, int to, int most, int32_t* out, u64* sums,
                                          Want want) {
  int found = 0;
  for (int base = from; base < to && found < most; base += THREADS * 4) {
    const int p0 = base + (int)threadIdx.x * 4;
    int held[4];
    bool is[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) held[x] = p0 + x < to ? __ldcg(refs + p0 + x) : 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) is[x] = p0 + x < to && want(held[x]);
    u64 total;
    int at = found + (int)block_scan<THREADS>(is[0] + is[1] + is[2] + is[3], sums, &total);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (is[x] && at < most) out[at] = p0 + x;
      at += is[x];
    }
    found = min(most, found + (int)total);
  }
  return found;
}

// COUNT: the counting of the whole table as well.  (refs is read past L1: atomics change it.)
// One CTA: a scan over the rows and one over the free pages decide every place, in an order
// that does not depend on timing.  Bound: its chain of loads and barriers (4 rows forked, plan
// and copies: 6.6 us).
template <int THREADS, int ROWS, bool COUNT>
__global__ void __launch_bounds__(THREADS) plan_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ u64 s_sums[THREADS / 32];
  __shared__ int s_last[ROWS];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch();
  if (COUNT) {
    for (int x = tid; x < a.n_rows * a.width; x += THREADS) {
      const int r = x / a.width;
      Take t;
      const bool ok = take_of(a, r, &t);
      count_entry(a, r, x - r * a.width, t, ok);
    }
    __syncthreads();
  }
  constexpr int PER = (ROWS + THREADS - 1) / THREADS;
  const int per = (a.n_rows + THREADS - 1) / THREADS;
  const int r0 = min(a.n_rows, tid * per), r1 = min(a.n_rows, r0 + per);
  int len[PER], held[PER], ends[PER], copies[PER], holders[PER];
  bool bad = false;
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const int r = r0 + x;
    len[x] = held[x] = ends[x] = copies[x] = holders[x] = 0;
    if (r >= r1) continue;
    Take t;
    bool ok = take_of(a, r, &t);
    const int room = ok && t.parent >= 0 && a.reserve ? max(0, a.reserve[r]) : 0;
    const long long e = ((long long)t.len + room + a.page_size - 1) / a.page_size;
    if (room > 0 && e > a.width) ok = false;
    if (!ok) {
      report(a.status, MK_ERR_PAGES, PO_UPDATE, r, t.parent);
      bad = true;
      t.len = t.held = 0;
    }
    len[x] = t.len;
    held[x] = t.held;
    ends[x] = ok && room > 0 ? (int)e : t.held;
    // the page this row will write into: its last, when it is partly filled
    int last = -1;
    if (ok && room > 0 && t.len % a.page_size) last = a.snap[(long long)t.parent * a.width + t.held - 1];
    s_last[r] = last;
    if (last >= 0) holders[x] = __ldcg(a.refs + last);
  }
  const bool any_bad = __syncthreads_or(bad);
  // of the rows that write into one page, each copies it while another holder is left
  u64 need = 0;
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const int r = r0 + x;
    if (r >= r1) continue;
    if (holders[x] > 1) {
      const int last = s_last[r];
      int before = 0;
      for (int q = 0; q < r; ++q) before += s_last[q] == last;
      copies[x] = before < holders[x] - 1;
    }
    // pages needed (at most 4096 rows of 2^26), and the copies among them in the low 13 bits
    need += ((u64)(copies[x] + ends[x] - held[x]) << 13) + copies[x];
  }
  u64 total;
  const u64 before = block_scan<THREADS>(need, s_sums, &total);
  const u64 pages = total >> 13;
  bool refused = any_bad;
  if (!refused && pages > 0) {
    const int most = (int)min(pages, (u64)a.n_pages);
    const int found = list_pages<THREADS>(a.refs, 0, a.n_pages, most, a.fresh, s_sums, [](int n) { return n == 0; });
    if ((u64)found < pages) {
      refused = true;
      if (tid == 0) report(a.status, MK_ERR_PAGES, PO_UPDATE, -1, (int)min(pages - found, (u64)0x7fffffff));
    }
  }
  if (tid == 0) {
    a.head[0] = refused;
    a.head[1] = refused ? 0 : (int)(total & 8191);
  }
  if (refused) return;
  __syncthreads();  // every read of refs is done, a.fresh is written
  for (int i = tid; i < (int)pages; i += THREADS) a.refs[a.fresh[i]] = 1;
  int at = (int)(before >> 13), c = (int)(before & 8191);
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const int r = r0 + x;
    if (r >= r1) continue;
    a.held[r] = held[x];
    a.ends[r] = ends[x];
    a.at[r] = at;
    a.copy[r] = copies[x];
    if (copies[x]) {
      a.src[c] = s_last[r];
      a.dst[c] = a.fresh[at];
      atomicSub(a.refs + s_last[r], 1);
      ++c;
    }
    at += copies[x] + ends[x] - held[x];
    a.lens[r] = len[x];  // every thread has read the old lengths it needs
  }
}

// Copies pages src[i] -> dst[i] in every plane: units of 4 KB dealt to the CTAs round robin,
// so that a few pages still use every SM; a thread has up to six 16-byte loads in flight.  W: the
// unit numbers' type -- 32 bits where they fit, as 64-bit divisions took a third of the
// instructions of a large copy.  Bound: DRAM.  Measured (128 rows forked, 80 pages of 64 KB in
// 48 planes; 450 pages of 16 KB compacted; whole calls): 73 and 120 us with four CTAs per SM
// and six loads, 83 and 118 with four loads, 113 and 161 with eight, 72 and 163 with five CTAs
// and four loads.
template <typename W>
__device__ __forceinline__ void copy_units(const PoolArgs& a, const int32_t* src, const int32_t* dst, W units, W upp) {
  const W planes = 2u * a.n_layers, grid = gridDim.x;
  for (W u0 = blockIdx.x; u0 < units; u0 += grid * kInFlight) {
    uint4 x[kInFlight];
    char* to[kInFlight];
#pragma unroll
    for (int q = 0; q < kInFlight; ++q) {
      const W u = u0 + q * grid;
      to[q] = nullptr;
      if (u >= units) continue;
      const W pl = u / upp, i = pl / planes, p = pl - i * planes;
      const long long off = (long long)(u - pl * upp) * kUnitBytes + threadIdx.x * 16;
      if (off >= a.page_bytes) continue;
      char* base = ((p & 1) ? a.v : a.k) + (long long)(p >> 1) * a.layer_stride + off;
      x[q] = *reinterpret_cast<const uint4*>(base + (long long)src[i] * a.page_stride);
      to[q] = base + (long long)dst[i] * a.page_stride;
    }
#pragma unroll
    for (int q = 0; q < kInFlight; ++q)
      if (to[q]) *reinterpret_cast<uint4*>(to[q]) = x[q];
  }
}
__device__ __forceinline__ void copy_pages(const PoolArgs& a, const int32_t* src, const int32_t* dst, int n) {
  const u64 upp = (u64)((a.page_bytes + kUnitBytes - 1) / kUnitBytes), units = (u64)n * 2u * a.n_layers * upp;
  if (units + (u64)gridDim.x * kInFlight < (1ull << 32))
    copy_units<unsigned>(a, src, dst, (unsigned)units, (unsigned)upp);
  else
    copy_units<u64>(a, src, dst, units, upp);
}

__global__ void __launch_bounds__(kCopyThreads) apply_kernel(const __grid_constant__ PoolArgs a) {
  pdl_wait();
  pdl_launch();
  if (a.head[0]) {  // refused: the counts go back to what the table says
    for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
      Take t;
      if (!take_of(a, r, &t)) continue;
      for (int i = threadIdx.x; i < a.width; i += kCopyThreads) {
        const int o = a.snap[(long long)r * a.width + i];
        const int n = i < t.held ? a.snap[(long long)t.parent * a.width + i] : -1;
        if (o == n) continue;
        if (o >= 0) atomicAdd(a.refs + o, 1);
        if (n >= 0) atomicSub(a.refs + n, 1);
      }
    }
    return;
  }
  for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
    const int held = a.held[r], ends = a.ends[r], at = a.at[r], copy = a.copy[r];
    const int p = a.parents ? a.parents[r] : r;
    const int32_t* from = a.snap + (long long)max(p, 0) * a.width;
    for (int i = threadIdx.x; i < a.width; i += kCopyThreads) {
      int id = -1;
      if (i < held)
        id = copy && i == held - 1 ? a.fresh[at] : from[i];
      else if (i < ends)
        id = a.fresh[at + copy + i - held];
      a.table[(long long)r * a.table_stride + i] = id;
    }
  }
  copy_pages(a, a.src, a.dst, a.head[1]);
}

// The u pages in use move below u: the i-th held page above goes to the i-th free one below, so
// that no copy waits for another.  One CTA; bound by its scans (2500 pages: 8 us).
__global__ void __launch_bounds__(kWideThreads) compact_plan_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ u64 s_sums[kWideThreads / 32];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch();
  int mine = 0;
  for (int i = tid; i < a.n_pages; i += kWideThreads) {
    mine += a.refs[i] > 0;
    a.rank[i] = -1;
  }
  u64 total;
  block_scan<kWideThreads>(mine, s_sums, &total);
  const int used = (int)total;
  const int n = list_pages<kWideThreads>(a.refs, used, a.n_pages, a.n_pages, a.src, s_sums, [](int c) { return c > 0; });
  list_pages<kWideThreads>(a.refs, 0, used, n, a.fresh, s_sums, [](int c) { return c <= 0; });
  __syncthreads();  // a.src and a.fresh are written, refs read
  for (int i = tid; i < n; i += kWideThreads) {
    const int s = a.src[i];
    a.rank[s] = i;
    a.refs[a.fresh[i]] = a.refs[s];
    a.refs[s] = 0;
  }
  if (tid == 0) a.head[1] = n;
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const __grid_constant__ PoolArgs a) {
  pdl_wait();
  pdl_launch();
  const long long cells = (long long)a.n_rows * a.width;
  for (long long x = (long long)blockIdx.x * kCopyThreads + threadIdx.x; x < cells; x += (long long)gridDim.x * kCopyThreads) {
    const int r = (int)(x / a.width);
    int32_t* cell = a.table + (long long)r * a.table_stride + (int)(x - (long long)r * a.width);
    const int id = *cell;
    if (id < 0) continue;
    if (id >= a.n_pages) {
      report(a.status, MK_ERR_PAGES, PO_COMPACT, r, id);
      continue;
    }
    const int k = a.rank[id];
    if (k >= 0) *cell = a.fresh[k];
  }
  copy_pages(a, a.src, a.fresh, a.head[1]);
}

mk_status fill(PoolArgs* a, const mk_page_pool* p, void* ws, size_t ws_bytes, int32_t* status) {
  if (!p || !p->k || !p->v || !p->table || !p->refs)
    return paged_fail(MK_ERR_INVALID, "the page pool or one of its pointers is NULL");
  if (!aligned_to(p->k, 16) || !aligned_to(p->v, 16)) return paged_fail(MK_ERR_INVALID, "pages must be 16-byte aligned");
  if (p->n_layers < 1 || p->n_pages < 1 || p->n_rows < 1 || p->table_width < 1)
    return paged_fail(MK_ERR_INVALID, "n_layers, n_pages, n_rows and table_width must be positive");
  if (p->n_pages >= (1 << 30)) return paged_fail(MK_ERR_INVALID, "n_pages out of range");
  if (p->n_rows > kMaxRows) return paged_fail(MK_ERR_INVALID, "n_rows must be at most 4096");
  if (p->page_size < 16 || p->page_size > 1024 || p->page_size % 16)
    return paged_fail(MK_ERR_INVALID, "page_size must be a multiple of 16 in [16, 1024]");
  if ((long long)p->table_width * p->page_size > (1LL << 30))
    return paged_fail(MK_ERR_INVALID, "table_width * page_size must be at most 2^30");
  if (p->table_stride < p->table_width) return paged_fail(MK_ERR_INVALID, "table_stride is smaller than table_width");
  if (p->page_bytes < 16 || p->page_bytes % 16 || p->page_stride % 16 || p->layer_stride % 16)
    return paged_fail(MK_ERR_INVALID, "page_bytes, page_stride and layer_stride must be multiples of 16");
  if (p->page_stride < p->page_bytes || (p->n_layers > 1 && p->layer_stride < p->page_bytes))
    return paged_fail(MK_ERR_INVALID, "page_stride and layer_stride must hold a page");
  const size_t need = lay_out(a, ws, p->n_rows, p->table_width, p->n_pages);
  if (!ws || !aligned_to(ws, 16) || ws_bytes < need)
    return paged_fail(MK_ERR_INVALID, "the workspace is missing, unaligned or too small (mk_update_pages_workspace)");
  a->k = static_cast<char*>(p->k); a->v = static_cast<char*>(p->v);
  a->table = p->table; a->refs = p->refs; a->status = status;
  a->page_bytes = p->page_bytes; a->page_stride = p->page_stride; a->layer_stride = p->layer_stride;
  a->table_stride = p->table_stride;
  a->n_layers = p->n_layers; a->n_pages = p->n_pages; a->page_size = p->page_size; a->n_rows = p->n_rows;
  a->width = p->table_width;
  return MK_OK;
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_update_pages_workspace(int n_rows, int table_width, int n_pages, size_t* bytes) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    if (!bytes) return paged_fail(MK_ERR_INVALID, "bytes is NULL");
    if (n_rows < 1 || n_rows > kMaxRows || table_width < 1 || n_pages < 1)
      return paged_fail(MK_ERR_INVALID, "n_rows must be in [1, 4096], table_width and n_pages positive");
    PoolArgs a{};
    *bytes = lay_out(&a, nullptr, n_rows, table_width, n_pages);
    return MK_OK;
  });
}

extern "C" mk_status mk_update_pages(const mk_update_args* args, const mk_page_pool* pool, int32_t* status, void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    if (!args || !args->lens) return paged_fail(MK_ERR_INVALID, "NULL argument");
    PoolArgs a{};
    mk_status s = fill(&a, pool, args->workspace, args->workspace_bytes, status);
    if (s) return s;
    a.lens = args->lens;
    a.parents = args->parents;
    a.reserve = args->reserve;
    int n_sm = 0;
    s = sm_count(&n_sm);
    if (s) return s;
    const bool narrow = a.n_rows <= kNarrowThreads;
    if (narrow && (long long)a.n_rows * a.width <= kCountInPlan) {
      s = launch_dependent(plan_kernel<kNarrowThreads, kNarrowThreads, true>, dim3(1), dim3(kNarrowThreads), 0, stream,
                           "mk_update_pages (plan)", a);
    } else {
      s = launch_dependent(count_kernel, dim3(a.n_rows), dim3(kRowThreads), 0, stream, "mk_update_pages (count)", a);
      if (s) return s;
      s = launch_dependent(narrow ? plan_kernel<kNarrowThreads, kNarrowThreads, false> : plan_kernel<kWideThreads, kMaxRows, false>,
                           dim3(1), dim3(narrow ? kNarrowThreads : kWideThreads), 0, stream, "mk_update_pages (plan)", a);
    }
    if (s) return s;
    return launch_dependent(apply_kernel, dim3(n_sm * kCopyCtasPerSm), dim3(kCopyThreads), 0, stream,
                            "mk_update_pages (apply)", a);
  });
}

extern "C" mk_status mk_compact_pages(const mk_page_pool* pool, void* workspace, size_t workspace_bytes, int32_t* status,
                                      void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    PoolArgs a{};
    mk_status s = fill(&a, pool, workspace, workspace_bytes, status);
    if (s) return s;
    int n_sm = 0;
    s = sm_count(&n_sm);
    if (s) return s;
    s = launch_dependent(compact_plan_kernel, dim3(1), dim3(kWideThreads), 0, stream, "mk_compact_pages (plan)", a);
    if (s) return s;
    return launch_dependent(compact_apply_kernel, dim3(n_sm * kCopyCtasPerSm), dim3(kCopyThreads), 0, stream,
                            "mk_compact_pages (apply)", a);
  });
}
