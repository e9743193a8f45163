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
constexpr int kCtasPerSm = 3, kWarpsPerSm = kCtasPerSm * kAppendThreads / 32;

struct AppendArgs {
  const void *q, *k, *v;
  void *qo, *kc, *vc;
  long long q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h, page_stride, table_stride;
  const int32_t *positions, *rows, *table;
  const double* freqs;
  int32_t* status;
  int n_tokens, share, hq, hkv, page_size, n_pages, n_rows, width, n_freqs;
  float mscale;
};

// The angle position * freq is taken in turns, as a whole number of 2^-64: the frequency's
// mantissa times 1 / (2 pi) to 64 bits, shifted, times the position; whole turns fall off the
// top, what is left is good to 2^-33 of a turn at any position and goes to sine and cosine in
// units of pi.  A 32-bit product would be off by 0.06 rad at position 10^6, and 64-bit floating
// point has so little throughput here that it alone cost 8 of 42 us of a long prompt.
__device__ __forceinline__ void turn_of(const AppendArgs& a, int pos, int i, float* c, float* s) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(a.freqs[i]);
  const int exponent = (int)(bits >> 52 & 2047) - 1023;               // freq = m 2^(exponent - 52)
  const unsigned long long m = (bits & 0xFFFFFFFFFFFFFull) | 1ull << 52;
  constexpr unsigned long long kInv = 0xa2f9836e4e441529ull;                // 2^66 / (2 pi)
  const unsigned long long hi = __umul64hi(m, kInv), lo = m * kInv;
  const int shift = 54 - exponent;                                     // freq 2^64 / (2 pi) = (hi, lo) 2^-shift
  unsigned long long turns = 0;                                        // (frequencies of 2^54 and more: none)
  if (shift >= 64 && shift < 128)
    turns = hi >> (shift - 64);
  else if (shift > 0 && shift < 64)
    turns = hi << (64 - shift) | lo >> shift;
  turns *= (unsigned long long)pos;
  if (bits >> 63) turns = 0ull - turns;
  sincospif((float)(int)(turns >> 32) * 0x1p-31f, s, c);
  *c *= a.mscale;
  *s *= a.mscale;
}

// where a token goes: the page and the row of it (page -1: nowhere)
__device__ __forceinline__ int2 place_of(const AppendArgs& a, int t, int pos, bool tell) {
  const int row = a.rows ? a.rows[t] : t, slot = pos / a.page_size;
  int page = -1;
  if ((unsigned)row < (unsigned)a.n_rows && slot < a.width) page = a.table[(long long)row * a.table_stride + slot];
  if ((unsigned)page >= (unsigned)a.n_pages) {
    if (tell) report(a.status, MK_ERR_PAGES, PO_APPEND, row, pos);
    page = -1;
  }
  return make_int2(page, pos - slot * a.page_size);
}

// A token is taken by 2^share warps, no warp waiting for another.  A head is cut into items of 16
// elements, one per lane: in the half layout item c < n_freqs / 8 holds elements [8c, 8c + 8) and
// their partners [n_freqs + 8c, ..), so that a rotation stays in one lane, and the others 16
// consecutive ones; interleaved, every item is 16 consecutive elements.  A lane has the same
// item of every head it takes (4 heads of 128 dims per turn of the warp, 8 of 64: queries
// first, then keys, then values), so its cosines and sines stay in registers.  The vectors of
// the next turns are in flight while it works, the first ones while the warp looks up its
// token's place and angles.  Bound: the vectors' bytes, read and written once (8192 tokens of 48
// heads of 128 dims, 201 MB: 37.2 us, 5.4 TB/s); for a few tokens the chain of loads from the
// position over the table to the store (one token: 2.6 us).
template <typename T, typename C, int HD, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, kCtasPerSm) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int ITEMS = HD / 16, HPW = 32 / ITEMS, WARPS = kAppendThreads / 32, U = 2;
  __shared__ __align__(16) float s_turn[WARPS][2][kMaxFreqs];  // cosines and sines of a warp's token
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % ITEMS;
  pdl_wait();
  pdl_launch();
  const unsigned unit = blockIdx.x * WARPS + warp;  // below 2^32: the host sees to it
  const int parts = 1 << a.share;
  if ((unit >> a.share) >= (unsigned)a.n_tokens) return;
  const int t = (int)(unit >> a.share);
  const int heads = a.hq + 2 * a.hkv, first = (unit & (parts - 1)) * HPW + lane / ITEMS, step = parts * HPW;
  const bool turned = c < a.n_freqs / 8;
  const int e0 = !INTER && turned ? 8 * c : 16 * c, e1 = !INTER && turned ? a.n_freqs + 8 * c : 16 * c + 8;
  const int qh = (int)a.q_h, kh = (int)a.k_h, vh = (int)a.v_h, oh = (int)a.o_h, hk = a.hq + a.hkv;
  const T* qs = static_cast<const T*>(a.q) + t * a.q_t + e0;
  const T* ks = static_cast<const T*>(a.k) + t * a.k_t - a.hq * a.k_h + e0;
  const T* vs = static_cast<const T*>(a.v) + t * a.v_t - hk * a.v_h + e0;
  Raw8<T> rx[U], ry[U];
  auto load = [&](int u, int h) {
    if (h >= heads) return;
    const T* base = h < a.hq ? qs : h < hk ? ks : vs;
    const int each = h < a.hq ? qh : h < hk ? kh : vh;
    const T* src = base + (long long)h * each;
    rx[u].load(src);
    ry[u].load(src + (e1 - e0));
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, first + u * step);
  const int pos = a.positions[t];
  if (pos < 0) return;
  int2 place = make_int2(0, 0);
  if (lane == 0) place = place_of(a, t, pos, (unit & (parts - 1)) == 0);
  for (int f = lane; f < a.n_freqs; f += 32) turn_of(a, pos, f, &s_turn[warp][0][f], &s_turn[warp][1][f]);
  place.x = __shfl_sync(0xffffffffu, place.x, 0);
  place.y = __shfl_sync(0xffffffffu, place.y, 0);
  __syncwarp();
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = turned ? s_turn[warp][0][8 * c + j] : 1.f;
    sn[j] = turned ? s_turn[warp][1][8 * c + j] : 0.f;
  }
  T* qd = static_cast<T*>(a.qo) + t * a.o_t + e0;
  const long long row = (long long)place.x * a.page_stride + (long long)place.y * HD + e0;
  const int head = a.page_size * HD;
  C* kd = static_cast<C*>(a.kc) + row - (long long)a.hq * head;
  C* vd = static_cast<C*>(a.vc) + row - (long long)hk * head;
  for (int h0 = first; h0 - lane / ITEMS < heads; h0 += U * step) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      if (h >= heads) break;
      float x[8], y[8];
      rx[u].up(x);
      ry[u].up(y);
      load(u, h + U * step);
      if (turned && h < hk) {
        if (INTER) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float xa = x[2 * j], ya = y[2 * j];
            x[2 * j] = xa * cs[j] - x[2 * j + 1] * sn[j];
            x[2 * j + 1] = x[2 * j + 1] * cs[j] + xa * sn[j];
            y[2 * j] = ya * cs[4 + j] - y[2 * j + 1] * sn[4 + j];
            y[2 * j + 1] = y[2 * j + 1] * cs[4 + j] + ya * sn[4 + j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xa = x[j];
            x[j] = xa * cs[j] - y[j] * sn[j];
            y[j] = y[j] * cs[j] + xa * sn[j];
          }
        }
      }
      if (h < a.hq) {
        T* dst = qd + (long long)h * oh;
        store8<T>(dst, x);
        store8<T>(dst + (e1 - e0), y);
      } else if (place.x >= 0) {
        C* dst = (h < hk ? kd : vd) + (long long)h * head;
        store8<C>(dst, x);
        store8<C>(dst + (e1 - e0), y);
      }
    }
  }
}

// The same without 16-byte alignment, or when n_freqs does not fill whole items: element
// pair by element pair, one CTA per token.
template <typename T, typename C, int HD, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) append_pairs_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float s_cos[kMaxFreqs], s_sin[kMaxFreqs];
  __shared__ int2 s_place;
  pdl_wait();
  pdl_launch();
  const int t = blockIdx.x, tid = threadIdx.x, pos = a.positions[t];
  if (pos < 0) return;
  if (tid == 0) s_place = place_of(a, t, pos, true);
  if (tid < a.n_freqs) turn_of(a, pos, tid, &s_cos[tid], &s_sin[tid]);
  __syncthreads();
  const int2 place = s_place;
  const int heads = a.hq + (place.x >= 0 ? 2 * a.hkv : 0);
  for (int i = tid; i < heads * (HD / 2); i += kAppendThreads) {
    const int h = i / (HD / 2), c = i % (HD / 2);
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv, turned = c < a.n_freqs;
    const int hk = is_v ? h - a.hq - a.hkv : h - a.hq;
    const T* src = is_q   ? static_cast<const T*>(a.q) + t * a.q_t + h * a.q_h
                   : is_v ? static_cast<const T*>(a.v) + t * a.v_t + hk * a.v_h
                          : static_cast<const T*>(a.k) + t * a.k_t + hk * a.k_h;
    const int e0 = !INTER && turned ? c : 2 * c, e1 = !INTER && turned ? a.n_freqs + c : 2 * c + 1;
    float x = Conv<T>::up(src[e0]), y = Conv<T>::up(src[e1]);
    if (turned && !is_v) {
      const float xa = x;
      x = xa * s_cos[c] - y * s_sin[c];
      y = y * s_cos[c] + xa * s_sin[c];
    }
    if (is_q) {
      T* dst = static_cast<T*>(a.qo) + t * a.o_t + h * a.o_h;
      dst[e0] = Conv<T>::down(x);
      dst[e1] = Conv<T>::down(y);
    } else {
      C* dst = static_cast<C*>(is_v ? a.vc : a.kc) + (long long)place.x * a.page_stride +
               ((long long)hk * a.page_size + place.y) * HD;
      dst[e0] = Conv<C>::down(x);
      dst[e1] = Conv<C>::down(y);
    }
  }
}

template <typename T, typename C, int HD>
mk_status launch_append(AppendArgs a, int n_sm, bool inter, bool vec, void* stream) {
  const char* what = "mk_rope_append";
  if (!vec)
    return launch_dependent(inter ? append_pairs_kernel<T, C, HD, true> : append_pairs_kernel<T, C, HD, false>,
                            dim3(a.n_tokens), dim3(kAppendThreads), 0, stream, what, a);
  // a warp takes at least four turns of a token, or down to one while warps are free
  constexpr int WARPS = kAppendThreads / 32, HPW = 512 / HD;
  const int turns = (a.hq + 2 * a.hkv + HPW - 1) / HPW;
  // (the warps are counted in 32 bits)
  while (((long long)a.n_tokens << (a.share + 1)) <= 0xFFFFFFF0LL &&
         ((8LL << a.share) <= turns ||
          ((2LL << a.share) <= turns && ((long long)a.n_tokens << (a.share + 1)) <= (long long)kWarpsPerSm * n_sm)))
    ++a.share;
  const long long ctas = (((long long)a.n_tokens << a.share) + WARPS - 1) / WARPS;
  return launch_dependent(inter ? append_kernel<T, C, HD, true> : append_kernel<T, C, HD, false>, dim3((unsigned)ctas),
                          dim3(kAppendThreads), 0, stream, what, a);
}
template <typename T>
mk_status launch_append(const AppendArgs& a, int n_sm, int cache_dtype, int hd, bool inter, bool vec, void* stream) {
  if (cache_dtype == MK_F16)
    return hd == 64 ? launch_append<T, __half, 64>(a, n_sm, inter, vec, stream)
                    : launch_append<T, __half, 128>(a, n_sm, inter, vec, stream);
  return hd == 64 ? launch_append<T, __nv_bfloat16, 64>(a, n_sm, inter, vec, stream)
                  : launch_append<T, __nv_bfloat16, 128>(a, n_sm, inter, vec, stream);
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_rope_append(const mk_append_args* args, const mk_page_view* cache, int32_t* status,
                                    void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
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
    if (args->q && overlaps(args->n_tokens, args->o_token, args->n_heads, args->o_head, cache->head_dim))
      return paged_fail(MK_ERR_INVALID, "the vectors of q_out overlap");
    if (args->n_tokens == 0) return MK_OK;
    AppendArgs a{};
    a.q = args->q; a.k = args->k; a.v = args->v; a.qo = args->q_out;
    a.kc = cache->k; a.vc = cache->v;
    a.q_t = args->q_token; a.q_h = args->q_head; a.k_t = args->k_token; a.k_h = args->k_head;
    a.v_t = args->v_token; a.v_h = args->v_head; a.o_t = args->o_token; a.o_h = args->o_head;
    a.page_stride = cache->page_stride; a.table_stride = cache->table_stride;
    a.positions = args->positions; a.rows = args->rows; a.table = cache->table; a.freqs = args->freqs; a.status = status;
    a.n_tokens = args->n_tokens; a.hq = args->q ? args->n_heads : 0;
    a.hkv = cache->n_kv_heads; a.page_size = cache->page_size; a.n_pages = cache->n_pages; a.n_rows = cache->n_rows;
    a.width = cache->table_width; a.n_freqs = args->n_freqs; a.mscale = args->mscale;
    // 16-byte accesses need aligned vectors and whole rotating items (and head strides of 32 bits)
    bool vec = args->n_freqs % 8 == 0;
    for (long long s : {a.q_h, a.k_h, a.v_h, a.o_h}) vec = vec && s >= INT32_MIN && s <= INT32_MAX;
    const long long per = 16 / (long long)esz;
    for (const void* p : {args->q, args->k, args->v, (const void*)args->q_out}) vec = vec && aligned_to(p, 16);
    for (long long s : {a.k_t, a.k_h, a.v_t, a.v_h}) vec = vec && s % per == 0;
    if (args->q)
      for (long long s : {a.q_t, a.q_h, a.o_t, a.o_h}) vec = vec && s % per == 0;
    const bool inter = args->interleaved != 0;
    int n_sm = 0;
    const mk_status s = sm_count(&n_sm);
    if (s) return s;
    if (args->dtype == MK_F32)
      return launch_append<float>(a, n_sm, cache->dtype, cache->head_dim, inter, vec, stream);
    if (args->dtype == MK_F16)
      return launch_append<__half>(a, n_sm, cache->dtype, cache->head_dim, inter, vec, stream);
    return launch_append<__nv_bfloat16>(a, n_sm, cache->dtype, cache->head_dim, inter, vec, stream);
  });
}

extern "C" mk_status mk_rope_freqs(const mk_rope_desc* d, double* freqs, float* mscale) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
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
  });
}

extern "C" mk_status mk_paged_status(int32_t* status, void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
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
  });
}
