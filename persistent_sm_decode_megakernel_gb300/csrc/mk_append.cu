// Rotary positions and the append into a paged KV cache (mk_rope_append), the frequencies
// (mk_rope_freqs) and the status word shared by the paged operators.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>

#include "mk_paged.cuh"

namespace mk {

mk_status sm_count(int* n) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && known[dev]) {
    *n = known[dev];
    return MK_OK;
  }
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return paged_fail(MK_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
  if (dev < 64) known[dev] = *n;
  return MK_OK;
}

std::string check_view(const mk_page_view* c) {
  if (!c) return "the page view is NULL";
  if (!c->k || !c->v || !c->table) return "the page view's k, v or table is NULL";
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return "pages must be 16-byte aligned";
  if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
  if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16)
    return "page_size must be a multiple of 16 in [16, 1024]";
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_rows < 1 || c->table_width < 1)
    return "n_pages, n_kv_heads, n_rows and table_width must be positive";
  if (c->n_kv_heads > 65535) return "n_kv_heads must be at most 65535";
  if ((long long)c->table_width * c->page_size > (1LL << 30)) return "table_width * page_size must be at most 2^30";
  if (c->table_stride < c->table_width) return "table_stride is smaller than table_width";
  if (c->page_stride < (long long)c->n_kv_heads * c->page_size * c->head_dim || c->page_stride % 8)
    return "page_stride must hold a page and be a multiple of 8";
  if (c->dtype != MK_F16 && c->dtype != MK_BF16) return "the cache's dtype must be MK_F16 or MK_BF16";
  return "";
}

namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxFreqs = 64;  // head_dim / 2 at most

struct AppendArgs {
  const void *q, *k, *v;
  void *qo, *kc, *vc;
  long long q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h, page_stride, table_stride;
  const int32_t *positions, *rows, *table;
  const double* freqs;
  int32_t* status;
  int hq, hkv, page_size, n_pages, n_rows, width, n_freqs;
  float mscale;
};

// One CTA per token.  A head is cut into items of 16 elements, one per thread at a time: in
// the half layout item c < n_freqs / 8 holds elements [8c, 8c + 8) and their partners
// [n_freqs + 8c, ..), so that a rotation stays in one thread, and the others 16 consecutive
// ones; interleaved, every item is 16 consecutive elements.  Without 16-byte alignment, or
// when n_freqs does not fill whole items, the same work goes element pair by element pair.
//
// The angle position * freq is taken in 64 bits in units of pi and reduced there to
// [-1, 1] before sine and cosine, which is what keeps far positions exact (at position 10^6
// a 32-bit product would be off by 0.06 rad); once per pair and token, shared by all heads
// through shared memory, 64-bit arithmetic costs nothing beside the vectors' traffic.
template <typename T, typename C, int HD, bool INTER, bool VEC>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float s_cos[kMaxFreqs], s_sin[kMaxFreqs];
  pdl_wait();
  pdl_launch();
  const int t = blockIdx.x, tid = threadIdx.x;
  const int pos = a.positions[t];
  if (pos < 0) return;
  const int row = a.rows ? a.rows[t] : t;
  const int slot = pos / a.page_size;
  int page = -1;
  if ((unsigned)row < (unsigned)a.n_rows && slot < a.width) page = a.table[(long long)row * a.table_stride + slot];
  const bool placed = (unsigned)page < (unsigned)a.n_pages;
  if (!placed && tid == 0) report(a.status, MK_ERR_PAGES, PO_APPEND, row, pos);
  if (tid < a.n_freqs) {
    const double turns = (double)pos * (a.freqs[tid] * 0.31830988618379067154);  // angle / pi
    const double r = turns - 2.0 * rint(turns * 0.5);
    float s, c;
    sincospif((float)r, &s, &c);
    s_cos[tid] = c * a.mscale;
    s_sin[tid] = s * a.mscale;
  }
  __syncthreads();
  const long long in_page = (long long)page * a.page_stride + (long long)(pos - slot * a.page_size) * HD;
  C* kc = static_cast<C*>(a.kc) + in_page;
  C* vc = static_cast<C*>(a.vc) + in_page;
  // heads in the order queries, keys, values; a token without a place has its queries only
  const int heads = a.hq + (placed ? 2 * a.hkv : 0);
  constexpr int PER = VEC ? HD / 16 : HD / 2;  // items, or pairs, of a head
  for (int i = tid; i < heads * PER; i += kAppendThreads) {
    const int h = i / PER, c = i % PER;
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    const int hk = is_v ? h - a.hq - a.hkv : h - a.hq;
    const T* src = is_q   ? static_cast<const T*>(a.q) + t * a.q_t + h * a.q_h
                   : is_v ? static_cast<const T*>(a.v) + t * a.v_t + hk * a.v_h
                          : static_cast<const T*>(a.k) + t * a.k_t + hk * a.k_h;
    T* qd = static_cast<T*>(a.qo) + t * a.o_t + h * a.o_h;
    C* cd = (is_v ? vc : kc) + (long long)hk * a.page_size * HD;
    if (VEC) {
      const bool turned = c < a.n_freqs / 8;
      // in the half layout a head's rotating items come in two pieces, for values too
      const int e0 = !INTER && turned ? 8 * c : 16 * c, e1 = !INTER && turned ? a.n_freqs + 8 * c : 16 * c + 8;
      float x[8], y[8];
      load8(src + e0, x);
      load8(src + e1, y);
      if (turned && !is_v) {
        if (INTER) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float c0 = s_cos[8 * c + j], s0 = s_sin[8 * c + j], c1 = s_cos[8 * c + 4 + j], s1 = s_sin[8 * c + 4 + j];
            const float xa = x[2 * j], ya = y[2 * j];
            x[2 * j] = xa * c0 - x[2 * j + 1] * s0;
            x[2 * j + 1] = x[2 * j + 1] * c0 + xa * s0;
            y[2 * j] = ya * c1 - y[2 * j + 1] * s1;
            y[2 * j + 1] = y[2 * j + 1] * c1 + ya * s1;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float cs = s_cos[8 * c + j], sn = s_sin[8 * c + j], xa = x[j];
            x[j] = xa * cs - y[j] * sn;
            y[j] = y[j] * cs + xa * sn;
          }
        }
      }
      if (is_q) {
        store8(qd + e0, x);
        store8(qd + e1, y);
      } else {
        store8(cd + e0, x);
        store8(cd + e1, y);
      }
    } else {
      const int e0 = !INTER && c < a.n_freqs ? c : 2 * c, e1 = !INTER && c < a.n_freqs ? a.n_freqs + c : 2 * c + 1;
      float x = Conv<T>::up(src[e0]), y = Conv<T>::up(src[e1]);
      if (c < a.n_freqs && !is_v) {
        const float xa = x;
        x = xa * s_cos[c] - y * s_sin[c];
        y = y * s_cos[c] + xa * s_sin[c];
      }
      if (is_q) {
        qd[e0] = Conv<T>::down(x);
        qd[e1] = Conv<T>::down(y);
      } else {
        cd[e0] = Conv<C>::down(x);
        cd[e1] = Conv<C>::down(y);
      }
    }
  }
}

template <typename T, typename C, int HD>
mk_status launch_append(const AppendArgs& a, int n, bool inter, bool vec, void* stream) {
  auto k = inter ? (vec ? append_kernel<T, C, HD, true, true> : append_kernel<T, C, HD, true, false>)
                 : (vec ? append_kernel<T, C, HD, false, true> : append_kernel<T, C, HD, false, false>);
  return launch_dependent(k, dim3(n), dim3(kAppendThreads), 0, stream, "mk_rope_append", a);
}
template <typename T>
mk_status launch_append(const AppendArgs& a, int n, int cache_dtype, int hd, bool inter, bool vec, void* stream) {
  if (cache_dtype == MK_F16)
    return hd == 64 ? launch_append<T, __half, 64>(a, n, inter, vec, stream)
                    : launch_append<T, __half, 128>(a, n, inter, vec, stream);
  return hd == 64 ? launch_append<T, __nv_bfloat16, 64>(a, n, inter, vec, stream)
                  : launch_append<T, __nv_bfloat16, 128>(a, n, inter, vec, stream);
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_rope_append(const mk_append_args* args, const mk_page_view* cache, int32_t* status,
                                    void* stream) {
  using namespace mk;
  const std::string e = check_view(cache);
  if (!e.empty()) return paged_fail(MK_ERR_INVALID, e);
  if (!args || !args->k || !args->v || !args->positions) return paged_fail(MK_ERR_INVALID, "NULL argument");
  if (!args->q != !args->q_out) return paged_fail(MK_ERR_INVALID, "q and q_out must both be given or both be NULL");
  if (args->dtype < MK_F16 || args->dtype > MK_F32) return paged_fail(MK_ERR_INVALID, "dtype");
  if (args->n_tokens < 0 || args->n_heads < 0 || args->n_heads > 65535 || (args->q && args->n_heads < 1))
    return paged_fail(MK_ERR_INVALID, "n_tokens or n_heads out of range");
  if (args->n_freqs < 0 || 2 * (long long)args->n_freqs > cache->head_dim)
    return paged_fail(MK_ERR_INVALID, "n_freqs must be in [0, head_dim / 2]");
  if (args->n_freqs && !args->freqs) return paged_fail(MK_ERR_INVALID, "freqs is NULL");
  if (args->interleaved != 0 && args->interleaved != 1) return paged_fail(MK_ERR_INVALID, "interleaved must be 0 or 1");
  const size_t esz = args->dtype == MK_F32 ? 4 : 2;
  for (const void* p : {args->q, args->k, args->v, (const void*)args->q_out})
    if (!aligned_to(p, esz)) return paged_fail(MK_ERR_INVALID, "q, k, v and q_out must be aligned to their type");
  if (args->q == args->q_out && args->q && (args->q_token != args->o_token || args->q_head != args->o_head))
    return paged_fail(MK_ERR_INVALID, "q_out in the place of q needs q's strides");
  if (args->n_tokens == 0) return MK_OK;
  AppendArgs a{};
  a.q = args->q; a.k = args->k; a.v = args->v; a.qo = args->q_out;
  a.kc = cache->k; a.vc = cache->v;
  a.q_t = args->q_token; a.q_h = args->q_head; a.k_t = args->k_token; a.k_h = args->k_head;
  a.v_t = args->v_token; a.v_h = args->v_head; a.o_t = args->o_token; a.o_h = args->o_head;
  a.page_stride = cache->page_stride; a.table_stride = cache->table_stride;
  a.positions = args->positions; a.rows = args->rows; a.table = cache->table; a.freqs = args->freqs; a.status = status;
  a.hq = args->q ? args->n_heads : 0;
  a.hkv = cache->n_kv_heads; a.page_size = cache->page_size; a.n_pages = cache->n_pages; a.n_rows = cache->n_rows;
  a.width = cache->table_width; a.n_freqs = args->n_freqs; a.mscale = args->mscale;
  // 16-byte accesses need aligned vectors and whole rotating items
  bool vec = args->n_freqs % 8 == 0;
  const long long per = 16 / (long long)esz;
  for (const void* p : {args->q, args->k, args->v, (const void*)args->q_out}) vec = vec && aligned_to(p, 16);
  for (long long s : {a.k_t, a.k_h, a.v_t, a.v_h}) vec = vec && s % per == 0;
  if (args->q)
    for (long long s : {a.q_t, a.q_h, a.o_t, a.o_h}) vec = vec && s % per == 0;
  const bool inter = args->interleaved != 0;
  if (args->dtype == MK_F32)
    return launch_append<float>(a, args->n_tokens, cache->dtype, cache->head_dim, inter, vec, stream);
  if (args->dtype == MK_F16)
    return launch_append<__half>(a, args->n_tokens, cache->dtype, cache->head_dim, inter, vec, stream);
  return launch_append<__nv_bfloat16>(a, args->n_tokens, cache->dtype, cache->head_dim, inter, vec, stream);
}

extern "C" mk_status mk_rope_freqs(const mk_rope_desc* d, double* freqs, float* mscale) {
  using namespace mk;
  if (!d || !freqs || !mscale) return paged_fail(MK_ERR_INVALID, "NULL argument");
  if (!(d->theta > 0) || !std::isfinite(d->theta)) return paged_fail(MK_ERR_INVALID, "theta must be positive");
  if (d->n_rot < 2 || d->n_rot % 2 || d->n_rot > 128) return paged_fail(MK_ERR_INVALID, "n_rot must be even, in [2, 128]");
  if (d->kind < 0 || d->kind > 4) return paged_fail(MK_ERR_INVALID, "kind must be 0..4");
  if (d->kind && (!(d->factor >= 1) || !std::isfinite(d->factor)))
    return paged_fail(MK_ERR_INVALID, "factor must be at least 1");
  if (d->kind == 2 && d->n_rot < 4) return paged_fail(MK_ERR_INVALID, "the scaled base needs n_rot >= 4");
  const double pi = 3.14159265358979323846;
  double fast = d->beta_fast, slow = d->beta_slow;
  if (d->kind >= 3) {
    if (!(d->original > 0) || !std::isfinite(d->original)) return paged_fail(MK_ERR_INVALID, "original must be positive");
    if (fast == 0) fast = d->kind == 3 ? 32 : 4;
    if (slow == 0) slow = 1;
    if (!(fast > slow) || !(slow > 0))
      return paged_fail(MK_ERR_INVALID, "beta_fast must be above beta_slow, both positive");
    if (d->kind == 3 && !(d->theta > 1)) return paged_fail(MK_ERR_INVALID, "the blend needs theta above 1");
  }
  const int n = d->n_rot / 2;
  const double theta = d->kind == 2 ? d->theta * std::pow(d->factor, (double)d->n_rot / (d->n_rot - 2)) : d->theta;
  // the (fractional) pair index that turns `turns` times within `original` positions
  auto index_of = [&](double turns) {
    return d->n_rot * std::log(d->original / (turns * 2 * pi)) / (2 * std::log(d->theta));
  };
  double lo = 0, hi = 0;
  if (d->kind == 3) {
    lo = std::max(0.0, std::floor(index_of(fast)));
    hi = std::min((double)d->n_rot - 1, std::ceil(index_of(slow)));
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < n; ++i) {
    const double f = std::pow(theta, -2.0 * i / d->n_rot);
    double r = f;
    if (d->kind == 1) r = f / d->factor;
    if (d->kind == 3) {
      const double far = std::min(1.0, std::max(0.0, (i - lo) / (hi - lo)));  // share of the divided frequency
      r = f * (1 - far) + f / d->factor * far;
    }
    if (d->kind == 4) {
      const double turns = d->original * f / (2 * pi);  // original / wavelength
      const double near = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
      r = f * near + f / d->factor * (1 - near);
    }
    freqs[i] = r;
  }
  *mscale = d->kind == 3 ? (float)(0.1 * std::log(d->factor) + 1.0) : 1.0f;
  return MK_OK;
}

extern "C" mk_status mk_paged_status(int32_t* status, void* stream) {
  using namespace mk;
  if (!status) return paged_fail(MK_ERR_INVALID, "status is NULL");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t got[4] = {};
  cudaError_t e = cudaMemcpyAsync(got, status, sizeof got, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && got[0]) e = cudaMemsetAsync(status, 0, sizeof got, s);
  if (e != cudaSuccess) return paged_fail(MK_ERR_CUDA, std::string("mk_paged_status: ") + cudaGetErrorString(e));
  if (!got[0]) return MK_OK;
  static const char* const ops[] = {"?", "append", "attention", "page update", "compaction", "selection"};
  char buf[160];
  snprintf(buf, sizeof buf, "%s: %s at row %d, value %d", ops[got[1] >= 1 && got[1] <= 5 ? got[1] : 0],
           got[0] == MK_ERR_NAN ? "a NaN or infinite logit" : "a bad page, row, length or parent, or too few free pages",
           got[2], got[3]);
  return paged_fail((mk_status)got[0], buf);
}
