// Acceptance of drafted tokens (mk_accept_drafts): the walk along the model's choices and the move of
// the accepted tokens' keys and values, in one launch.
//
// A cluster of CTAs takes a row.  Each of them walks the tree itself (a warp looks at all of the
// nodes at once, one turn per accepted token), moves its share of the vectors and waits for the others
// before one of them writes the row's new length, which the walk of all has read.  An accepted node's
// slot only ever lies at or behind its place (path[j] >= j), and a thread takes the same 16 bytes of
// all of a head's accepted vectors in order, several loads before their stores: what is overwritten was
// read before.  Bound: the vectors' bytes, read and written once, in pieces of a vector (64 rows of up to 12 tokens, 24
// layers, 91 MB: 20 us, 4.5 TB/s; more loads in flight per thread leave fewer CTAs on an SM: 12 took 45); for a few rows
// the chain from the tree over the table to the stores (one row of 4 tokens: 4.5 us).
#include "mk_paged.cuh"

namespace mk {
namespace {

constexpr int kAcceptThreads = 256;
constexpr int kAcceptCluster = 8;  // CTAs of a row
constexpr int kMaxNodes = 128;

struct AcceptArgs {
  char *k, *v;
  int32_t *lens, *out_tokens, *out_path, *out_count, *status;
  const int32_t *tokens, *parents, *choices, *table;
  long long page_stride, layer_stride, table_stride;
  int n_layers, n_pages, page_size, width, hkv, n_nodes, vec;  // vec: 16-byte pieces of a vector
};

__global__ void __cluster_dims__(kAcceptCluster, 1, 1) __launch_bounds__(kAcceptThreads, 4)
accept_kernel(const __grid_constant__ AcceptArgs a) {
  __shared__ int s_token[kMaxNodes], s_parent[kMaxNodes], s_choice[kMaxNodes], s_path[kMaxNodes], s_count;
  __shared__ long long s_src[kMaxNodes], s_dst[kMaxNodes];  // bytes from a plane's begin to the vectors of its first head
  const int tid = threadIdx.x, lane = tid & 31, r = blockIdx.x / kAcceptCluster, rank = blockIdx.x % kAcceptCluster;
  const int n = a.n_nodes;
  pdl_wait();
  pdl_launch();
  const long long at = (long long)r * n;
  for (int i = tid; i < n; i += kAcceptThreads) {
    s_token[i] = a.tokens[at + i];
    s_parent[i] = a.parents[at + i];
    s_choice[i] = a.choices[at + i];
  }
  const int len = a.lens[r];
  if (tid == 0) s_count = 0;
  __syncthreads();
  if (tid < 32 && len >= 0 && s_parent[0] == -1) {
    int cur = 0, count = 0;
    while (true) {
      if (lane == 0) s_path[count] = cur;
      ++count;
      const int wanted = s_choice[cur];
      int next = n;  // a child is behind its parent
      for (int b = 0; b < n && next == n; b += 32) {
        const int i = b + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, i < n && i > cur && s_parent[i] == cur && s_token[i] == wanted);
        if (hit) next = b + __ffs(hit) - 1;
      }
      if (next == n) break;
      cur = next;
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  int count = s_count;
  // places, and whether all of them are
  bool bad = false;
  int told = 0;
  for (int j = tid; j < count; j += kAcceptThreads) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const long long t = (long long)len + (w ? j : s_path[j]);
      const int i = (int)(t / a.page_size);
      int page = -1;
      if (i < a.width) page = a.table[(long long)r * a.table_stride + i];
      if ((unsigned)page >= (unsigned)a.n_pages) {
        bad = true;
        told = (int)t;
      }
      (w ? s_dst : s_src)[j] = page * a.page_stride + (t - (long long)i * a.page_size) * a.vec * 16;
    }
  }
  if (__syncthreads_or(bad)) {
    if (bad && rank == 0) report(a.status, MK_ERR_PAGES, PO_ACCEPT, r, told);
    count = 0;
  }
  const int planes = 2 * a.n_layers * a.hkv, vec = a.vec;
  constexpr int U = 6;  // vectors in flight
  for (int x = rank * kAcceptThreads + tid; x < planes * vec && count > 1; x += kAcceptCluster * kAcceptThreads) {
    const int piece = x % vec, plane = x / vec, head = plane % a.hkv, l = plane / a.hkv;
    char* base = (l & 1 ? a.v : a.k) + (long long)(l >> 1) * a.layer_stride + (long long)head * a.page_size * vec * 16 + piece * 16;
    for (int j0 = 1; j0 < count; j0 += U) {
      uint4 got[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u < count)
          got[u] = *reinterpret_cast<const uint4*>(base + s_src[j0 + u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u < count && s_path[j0 + u] != j0 + u)
          *reinterpret_cast<uint4*>(base + s_dst[j0 + u]) = got[u];
    }
  }
  // every CTA of the row has read its length
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  if (rank != 0) return;
  for (int j = tid; j < n; j += kAcceptThreads) {
    a.out_path[at + j] = j < count ? s_path[j] : -1;
    a.out_tokens[at + j] = j < count ? s_choice[s_path[j]] : -1;
  }
  if (tid == 0) {
    a.out_count[r] = count;
    if (count) a.lens[r] = len + count;
  }
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_accept_drafts(const mk_accept_args* args, const mk_page_pool* p, int32_t* status, void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
    if (!p || !p->k || !p->v || !p->table)
      return paged_fail(MK_ERR_INVALID, "the page pool or one of its pointers is NULL");
    if (!args || !args->lens || !args->tokens || !args->parents || !args->choices || !args->out_tokens || !args->out_path ||
        !args->out_count)
      return paged_fail(MK_ERR_INVALID, "NULL argument");
    if (!aligned_to(p->k, 16) || !aligned_to(p->v, 16)) return paged_fail(MK_ERR_INVALID, "pages must be 16-byte aligned");
    if (p->n_layers < 1 || p->n_pages < 1 || p->n_rows < 1 || p->table_width < 1)
      return paged_fail(MK_ERR_INVALID, "n_layers, n_pages, n_rows and table_width must be positive");
    if (p->page_size < 16 || p->page_size > 1024 || p->page_size % 16)
      return paged_fail(MK_ERR_INVALID, "page_size must be a multiple of 16 in [16, 1024]");
    if ((long long)p->table_width * p->page_size > (1LL << 30))
      return paged_fail(MK_ERR_INVALID, "table_width * page_size must be at most 2^30");
    if (p->table_stride < p->table_width) return paged_fail(MK_ERR_INVALID, "table_stride is smaller than table_width");
    if (args->n_nodes < 1 || args->n_nodes > kMaxNodes) return paged_fail(MK_ERR_INVALID, "n_nodes must be in [1, 128]");
    if (args->n_kv_heads < 1 || args->n_kv_heads > 65535)
      return paged_fail(MK_ERR_INVALID, "n_kv_heads must be in [1, 65535]");
    const long long vectors = (long long)args->n_kv_heads * p->page_size;
    if (p->page_bytes < 16 || p->page_bytes % vectors || p->page_bytes / vectors % 16 || p->page_bytes / vectors > 256)
      return paged_fail(MK_ERR_INVALID, "page_bytes must be n_kv_heads * page_size vectors of a multiple of 16 bytes up to 256");
    if (p->page_stride % 16 || p->layer_stride % 16 || p->page_stride < p->page_bytes ||
        (p->n_layers > 1 && p->layer_stride < p->page_bytes))
      return paged_fail(MK_ERR_INVALID, "page_stride and layer_stride must hold a page and be multiples of 16");
    if ((long long)p->n_layers * args->n_kv_heads > (1 << 24) || p->n_rows > (1 << 27))
      return paged_fail(MK_ERR_INVALID, "n_layers * n_kv_heads must be at most 2^24, n_rows at most 2^27");
    AcceptArgs a{};
    a.k = static_cast<char*>(p->k); a.v = static_cast<char*>(p->v);
    a.lens = args->lens; a.out_tokens = args->out_tokens; a.out_path = args->out_path; a.out_count = args->out_count;
    a.status = status;
    a.tokens = args->tokens; a.parents = args->parents; a.choices = args->choices; a.table = p->table;
    a.page_stride = p->page_stride; a.layer_stride = p->layer_stride; a.table_stride = p->table_stride;
    a.n_layers = p->n_layers; a.n_pages = p->n_pages; a.page_size = p->page_size; a.width = p->table_width;
    a.hkv = args->n_kv_heads; a.n_nodes = args->n_nodes; a.vec = (int)(p->page_bytes / vectors / 16);
    return launch_dependent(accept_kernel, dim3(p->n_rows * kAcceptCluster), dim3(kAcceptThreads), 0, stream,
                            "mk_accept_drafts", a);
  });
}
