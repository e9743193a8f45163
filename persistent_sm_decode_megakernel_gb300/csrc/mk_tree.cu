// Attention of a tree of drafted tokens over a paged KV cache (mk_tree_attention): the simplest form, a
// warp per row, node and head.
#include <algorithm>

#include "mk_internal.h"
#include "mk_device.cuh"
#include "mk_paged.cuh"

namespace mk {
namespace {

constexpr int kMaxNodes = 128, kMaxGroup = 16, kTreeThreads = 128;

struct TreeArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  const int32_t *lens, *parents, *rows, *table;
  int32_t* status;
  long long q_row, q_node, q_head, o_row, o_node, o_head, page_stride, table_stride;
  int n_rows, n_nodes, hq, hkv, group, window, page_size, n_pages, table_rows, cap;
  float scale, softcap;
};

template <typename C, typename Q, int HD>
__global__ void __launch_bounds__(kTreeThreads) tree_simple_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int E = HD / 32;
  __shared__ float s_q[kTreeThreads / 32][HD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch();
  const long long unit = (long long)blockIdx.x * (kTreeThreads / 32) + warp;
  if (unit >= (long long)a.n_rows * a.n_nodes * a.hq) return;
  const int h = (int)(unit % a.hq), node = (int)(unit / a.hq % a.n_nodes), r = (int)(unit / a.hq / a.n_nodes);
  const int trow = a.rows ? a.rows[r] : r, len = a.lens[r];
  unsigned seen[4] = {0, 0, 0, 0};
  int depth = 0, first = node;  // first: the ancestor the window ends at
  bool there = len >= 0;
  for (int i = node; there;) {
    if (!a.window || depth < a.window) seen[i >> 5] |= 1u << (i & 31);
    const int p = a.parents[(long long)r * a.n_nodes + i];
    if (p == -1) break;
    there = p >= 0 && p < i;
    i = p;
    ++depth;
  }
  (void)first;
  if (there && (unsigned)trow >= (unsigned)a.table_rows) {
    if (lane == 0) report(a.status, MK_ERR_PAGES, PO_TREE, r, trow);
    there = false;
  }
  const Q* q = static_cast<const Q*>(a.q) + r * a.q_row + node * a.q_node + h * a.q_head;
  for (int d = lane; d < HD; d += 32) s_q[warp][d] = Conv<Q>::up(q[d]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[E];
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const long long end = (long long)len + a.n_nodes;
  if (there && end > a.cap && lane == 0) report(a.status, MK_ERR_PAGES, PO_TREE, r, (int)(end < 0x7fffffffLL ? end : 0x7fffffffLL));
  const int hi = there ? (int)(end < a.cap ? end : a.cap) : 0;
  const int lo = a.window ? (int)max(0LL, (long long)len + depth + 1 - a.window) : 0;
  for (int t0 = min(lo, max(len, 0)) / 32 * 32; t0 < hi; t0 += 32) {
    const int t = t0 + lane, x = t - len;
    bool in = t < hi && (x < 0 ? t >= lo : (seen[(x >> 5) & 3] >> (x & 31) & 1) != 0);
    int page = -1;
    if (t < hi) {
      page = a.table[(long long)trow * a.table_stride + t / a.page_size];
      if ((unsigned)page >= (unsigned)a.n_pages) {
        if (in) report(a.status, MK_ERR_PAGES, PO_TREE, r, page);
        in = false;
      }
    }
    const long long off = (long long)page * a.page_stride + ((long long)(h / a.group) * a.page_size + t % a.page_size) * HD;
    float s = -INFINITY;
    if (in) {
      s = 0.f;
      const C* k = static_cast<const C*>(a.k) + off;
      for (int d = 0; d < HD; ++d) s = fmaf(s_q[warp][d], Conv<C>::up(k[d]), s);
      s *= a.scale;
      if (a.softcap > 0.f) s = a.softcap * tanhf(s);
    }
    float top = s;
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    const float mn = fmaxf(m, top), ms = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ms), p = in ? exp2f(s - ms) : 0.f;
    float sum = p;
    for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    l = l * f + sum;
    m = mn;
    for (int e = 0; e < E; ++e) o[e] *= f;
    for (int y = 0; y < 32; ++y) {
      const bool on = __shfl_sync(0xffffffffu, (int)in, y);
      const float py = __shfl_sync(0xffffffffu, p, y);
      const long long oy = __shfl_sync(0xffffffffu, off, y);
      if (!on) continue;
      const C* v = static_cast<const C*>(a.v) + oy;
      for (int e = 0; e < E; ++e) o[e] = fmaf(py, Conv<C>::up(v[32 * e + lane]), o[e]);
    }
  }
  Q* out = static_cast<Q*>(a.out) + r * a.o_row + node * a.o_node + h * a.o_head;
  for (int e = 0; e < E; ++e) out[32 * e + lane] = Conv<Q>::down(l == 0.f ? 0.f : o[e] / l);
  if (lane == 0 && a.lse)
    a.lse[((long long)r * a.n_nodes + node) * a.hq + h] = ((m == -INFINITY ? 0.f : m) + log2f(l)) * 0.69314718055994531f;
}

template <typename C, typename Q>
mk_status launch_tree(const TreeArgs& a, int hd, void* stream) {
  const long long warps = (long long)a.n_rows * a.n_nodes * a.hq;
  const dim3 grid((unsigned)((warps + kTreeThreads / 32 - 1) / (kTreeThreads / 32)));
  return launch_dependent(hd == 64 ? tree_simple_kernel<C, Q, 64> : tree_simple_kernel<C, Q, 128>, grid, dim3(kTreeThreads), 0,
                          stream, "mk_tree_attention", a);
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_tree_attention_workspace(int n_heads, int n_kv_heads, int head_dim, size_t* bytes) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    if (!bytes) return paged_fail(MK_ERR_INVALID, "bytes is NULL");
    if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > kMaxGroup)
      return paged_fail(MK_ERR_INVALID, "n_heads / n_kv_heads must be a whole number in [1, 16]");
    if (head_dim != 64 && head_dim != 128) return paged_fail(MK_ERR_INVALID, "head_dim must be 64 or 128");
    *bytes = 16;
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
    size_t need = 0;
    const mk_status s = mk_tree_attention_workspace(args->n_heads, cache->n_kv_heads, cache->head_dim, &need);
    if (s) return s;
    if (args->n_rows < 0 || (long long)args->n_rows * args->n_nodes * args->n_heads > 0x7fffffffLL)
      return paged_fail(MK_ERR_INVALID, "n_rows out of range");
    if (args->window < 0) return paged_fail(MK_ERR_INVALID, "window must not be negative");
    const float log2e = 1.4426950408889634f;
    const float factor = args->softcap > 0.f ? args->scale / args->softcap : args->scale * log2e;
    if (!(args->softcap >= 0.f && args->softcap * log2e < INFINITY) || !(std::abs(factor) < INFINITY))
      return paged_fail(MK_ERR_INVALID, "scale or softcap is not finite, too large, or softcap negative or too small for scale");
    const size_t esz = args->dtype == MK_F32 ? 4 : 2;
    if (!aligned_to(args->q, esz) || !aligned_to(args->out, esz))
      return paged_fail(MK_ERR_INVALID, "q and out must be aligned to their type");
    const long long rn = args->n_rows, nn = args->n_nodes, hn = args->n_heads, hd = cache->head_dim;
    if (overlaps(rn, args->o_row, nn, args->o_node, hd) || overlaps(rn, args->o_row, hn, args->o_head, hd) ||
        overlaps(nn, args->o_node, hn, args->o_head, hd))
      return paged_fail(MK_ERR_INVALID, "the vectors of out overlap");
    if (!args->workspace || !aligned_to(args->workspace, 16) || args->workspace_bytes < need)
      return paged_fail(MK_ERR_INVALID, "the workspace is missing, unaligned or too small (mk_tree_attention_workspace)");
    if (args->n_rows == 0) return MK_OK;
    TreeArgs a{};
    a.q = args->q; a.k = cache->k; a.v = cache->v; a.out = args->out; a.lse = args->lse;
    a.lens = args->lens; a.parents = args->parents; a.rows = args->rows; a.table = cache->table; a.status = status;
    a.q_row = args->q_row; a.q_node = args->q_node; a.q_head = args->q_head;
    a.o_row = args->o_row; a.o_node = args->o_node; a.o_head = args->o_head;
    a.page_stride = cache->page_stride; a.table_stride = cache->table_stride;
    a.n_rows = args->n_rows; a.n_nodes = args->n_nodes; a.hq = args->n_heads; a.hkv = cache->n_kv_heads;
    a.group = a.hq / a.hkv; a.window = args->window; a.page_size = cache->page_size; a.n_pages = cache->n_pages;
    a.table_rows = cache->n_rows; a.cap = cache->table_width * cache->page_size;
    a.scale = factor;
    a.softcap = args->softcap * log2e;
    const int d = cache->head_dim;
    if (cache->dtype == MK_F16) {
      if (args->dtype == MK_F16) return launch_tree<__half, __half>(a, d, stream);
      if (args->dtype == MK_BF16) return launch_tree<__half, __nv_bfloat16>(a, d, stream);
      return launch_tree<__half, float>(a, d, stream);
    }
    if (args->dtype == MK_BF16) return launch_tree<__nv_bfloat16, __nv_bfloat16>(a, d, stream);
    if (args->dtype == MK_F16) return launch_tree<__nv_bfloat16, __half>(a, d, stream);
    return launch_tree<__nv_bfloat16, float>(a, d, stream);
  });
}
