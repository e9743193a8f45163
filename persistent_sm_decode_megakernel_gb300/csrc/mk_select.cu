// One step of a beam search over beams and vocabulary (mk_beam_select).
//
// A row's candidates are ordered by logit alone, so the log-softmax is not needed to choose
// among them: one pass over the logits yields, per chunk of a row, the maximum, the sum of
// exponentials and the chunk's `beams` largest logits; a second kernel (one CTA per group)
// joins the chunks -- lse = M + log sum_c S_c e^(M_c - M), in 64 bits -- and picks the best of
// score + logit - lse over the group's beams.
//
// Keys: a logit's bits as an ordered unsigned number, above the complement of its token, so
// that a larger key is a larger logit or an equal one of a lower token, and no two are equal.
#include <algorithm>

#include "mk_internal.h"
#include "mk_device.cuh"
#include "mk_paged.cuh"

namespace mk {
namespace {

constexpr int kMaxBeams = 32;
constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kPickThreads = 256;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kList = 1024;  // candidates of a chunk above its threshold that are ranked at once

using u64 = unsigned long long;

struct SelectArgs {
  const void* logits;
  const float* scores;
  const int32_t* ended;
  int32_t *out_tokens, *out_parents, *out_ended, *status;
  float* out_scores;
  u64* cand;        // [rows][chunks][beams], best first; 0: none
  float4* stat;     // [rows][chunks]: maximum, sum of e^(x - maximum) in two parts, unused
  long long row_stride;
  int rows, beams, vocab, chunk, chunks, eos;
};

__device__ __forceinline__ u64 key_of(float x, int token) { return (u64)orderable(x) << 32 | (0xFFFFFFFFu - (unsigned)token); }
__device__ __forceinline__ float value_of(u64 key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ int token_of(u64 key) { return (int)(0xFFFFFFFFu - (unsigned)key); }

// the largest of the warp's keys (each lane's own, 0: none)
__device__ __forceinline__ u64 warp_max(u64 k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (u64)hi << 32 | lo;
}

// One chunk of PER * 256 logits per CTA, all of it in registers.  The `beams` largest are
// found through a threshold: the beams-th largest of a warp's 32 lane maxima has at least
// `beams` elements at or above it, the largest such bound over the warps few more (about
// 60..150 of 8192 for 8 beams); those go to a list in shared memory and each counts how many
// of the list are above it, which is its place.  Were the list to overflow (logits laid out
// so that a few lanes hold all the large ones), the beams come out one block maximum at a
// time.  Bound: the logits' bytes for many rows, the launch and the block steps for few.
template <typename T, int PER, bool VEC>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ u64 s_list[kList], s_warp[kScanWarps];
  __shared__ double s_d[kScanWarps];
  __shared__ float s_f[kScanWarps];
  __shared__ int s_n;
  constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;  // elements of an access
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  pdl_wait();
  pdl_launch();
  if (a.ended[row]) return;  // it offers one token, whatever its logits
  const T* src = static_cast<const T*>(a.logits) + (long long)row * a.row_stride;
  const int first = chunk * a.chunk, n = min(a.chunk, a.vocab - first);
  float x[PER];
#pragma unroll
  for (int i = 0; i < PER / V; ++i) {
    const int e = (i * kScanThreads + tid) * V;
    if (VEC) {
      alignas(16) T raw[V];
      if (e + V <= n) {
        *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(src + first + e);
#pragma unroll
        for (int y = 0; y < V; ++y) x[i * V + y] = Conv<T>::up(raw[y]);
      } else {
#pragma unroll
        for (int y = 0; y < V; ++y) x[i * V + y] = e + y < n ? Conv<T>::up(src[first + e + y]) : -INFINITY;
      }
    } else {
      x[i] = e < n ? Conv<T>::up(src[first + e]) : -INFINITY;
    }
  }
  // element x[i * V + y] is token first + (i * 256 + tid) * V + y: rising in a thread
  auto at = [&](int i) { return ((i / V) * kScanThreads + tid) * V + i % V; };
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!(x[i] < INFINITY)) {  // NaN or +inf
      bad = true;
      x[i] = -INFINITY;
    }
    x[i] += 0.f;  // -0 and +0 are one value, and so a tie
    top = fmaxf(top, x[i]);
  }
  if (bad) report(a.status, MK_ERR_NAN, PO_SELECT, row, chunk);
  // the thread's own largest key: the first element that reaches top (none in an empty tail)
  int best = -1;
#pragma unroll
  for (int i = PER - 1; i >= 0; --i)
    if (x[i] == top && at(i) < n) best = at(i);
  const u64 own = best >= 0 ? key_of(top, first + best) : 0ull;
  // the warp's beams-th largest lane maximum
  u64 left = own, kth = 0ull;
  for (int b = 0; b < a.beams; ++b) {
    kth = warp_max(left);
    if (kth == 0ull) break;  // fewer lanes with elements than beams: no bound from this warp
    if (left == kth) left = 0ull;
  }
  float wtop = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wtop = fmaxf(wtop, __shfl_xor_sync(0xffffffffu, wtop, o));
  if (lane == 0) {
    s_warp[warp] = kth;
    s_f[warp] = wtop;
  }
  if (tid == 0) s_n = 0;
  __syncthreads();
  u64 bound = 0ull;
  float m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kScanWarps; ++w) {
    bound = s_warp[w] > bound ? s_warp[w] : bound;
    m = fmaxf(m, s_f[w]);
  }
  // sum of e^(x - m): fours in 32 bits, a compensated sum of them per thread, and from there
  // on in 64 bits, so that the sum of any vocabulary is good to a few 2^-24 of its terms
  float s = 0.f, comp = 0.f;
  if (m > -INFINITY) {
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const float q = (expf(x[i] - m) + expf(x[i + 1] - m)) + (expf(x[i + 2] - m) + expf(x[i + 3] - m));
      const float t = s + q, r = t - s;  // t + the bracket below is s + q exactly
      comp += (s - (t - r)) + (q - r);
      s = t;
    }
  }
  if (own >= bound) {  // its largest is at or above the bound: the others may be
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= n) continue;
      const u64 k = key_of(x[i], first + at(i));
      if (k < bound) continue;
      const int p = atomicAdd(&s_n, 1);
      if (p < kList) s_list[p] = k;
    }
  }
  double d = (double)s + (double)comp;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) s_d[warp] = d;
  __syncthreads();
  if (tid == 0) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) sum += s_d[w];
    a.stat[(long long)row * a.chunks + chunk] = make_float4(m, (float)sum, (float)(sum - (double)(float)sum), 0.f);
  }
  const int count = s_n;
  u64* out = a.cand + ((long long)row * a.chunks + chunk) * a.beams;
  if (count <= kList) {
    for (int e = tid; e < count; e += kScanThreads) {
      const u64 k = s_list[e];
      int above = 0;
      for (int f = 0; f < count; ++f) above += s_list[f] > k;
      if (above < a.beams) out[above] = k;
    }
    for (int b = count + tid; b < a.beams; b += kScanThreads) out[b] = 0ull;
    return;
  }
  u64 last = ~0ull;
  for (int b = 0; b < a.beams; ++b) {  // the largest key below the last one taken
    u64 k = 0ull;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at(i) >= n) continue;
      const u64 y = key_of(x[i], first + at(i));
      if (y < last && y > k) k = y;
    }
    k = warp_max(k);
    __syncthreads();
    if (lane == 0) s_warp[warp] = k;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) k = s_warp[w] > k ? s_warp[w] : k;
    if (tid == 0) out[b] = k;
    last = k;
  }
}

// One CTA per group, a warp per beam at a time: the beam's best from its chunks' lists (8 keys
// per lane in registers, the best so far carried from batch to batch), its lse, and its
// candidates' scores; then every candidate's place among the group's is the sum over the
// beams of how many of that beam's sorted list are ahead of it.
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ double s_key[kMaxBeams][kMaxBeams];
  __shared__ int s_token[kMaxBeams][kMaxBeams], s_len[kMaxBeams];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = blockIdx.x, K = a.beams;
  pdl_wait();
  pdl_launch();
  for (int b = warp; b < K; b += kPickWarps) {
    const int row = group * K + b;
    float sc = a.scores[row];
    if (!(sc == sc)) {
      if (lane == 0) report(a.status, MK_ERR_NAN, PO_SELECT, row, -1);
      sc = -INFINITY;
    }
    if (a.ended[row]) {
      if (lane == 0) {
        s_len[b] = 1;
        s_key[b][0] = (double)sc;
        s_token[b][0] = a.eos;
      }
      continue;
    }
    const float4* st = a.stat + (long long)row * a.chunks;
    float m = -INFINITY;
    for (int c = lane; c < a.chunks; c += 32) m = fmaxf(m, st[c].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double sum = 0.0;
    if (m > -INFINITY)
      for (int c = lane; c < a.chunks; c += 32) {
        const float4 s = st[c];
        if (s.x > -INFINITY) sum += ((double)s.y + (double)s.z) * exp((double)s.x - (double)m);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const double lse = m > -INFINITY ? (double)m + log(sum) : 0.0;
    const u64* cand = a.cand + (long long)row * a.chunks * K;
    const long long total = (long long)a.chunks * K;
    u64 mine = 0ull;  // lane k: the k-th best so far
    for (long long base = 0; base < total; base += 256) {
      u64 k[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const long long e = base + x * 32 + lane;
        k[x] = e < total ? cand[e] : 0ull;
      }
      u64 carry = mine;
      for (int q = 0; q < K; ++q) {
        u64 best = carry;
#pragma unroll
        for (int x = 0; x < 8; ++x) best = k[x] > best ? k[x] : best;
        const u64 win = warp_max(best);
        if (win == 0ull) {
          if (lane >= q) mine = 0ull;
          break;
        }
        if (best == win) {  // one lane: the keys differ
          if (carry == win) carry = 0ull;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (k[x] == win) k[x] = 0ull;
        }
        if (lane == q) mine = win;
      }
    }
    if (lane < K) {
      const float v = value_of(mine);
      double key = v > -INFINITY ? (double)sc + ((double)v - lse) : -INFINITY;
      if (!(key == key)) key = -INFINITY;
      s_key[b][lane] = key;
      s_token[b][lane] = token_of(mine);
    }
    if (lane == 0) s_len[b] = K;
  }
  __syncthreads();
  for (int x = tid; x < K * K; x += kPickThreads) {
    const int b = x / K, e = x % K;
    if (e >= s_len[b]) continue;
    const double key = s_key[b][e];
    int place = e;
    for (int o = 0; o < K && place < K; ++o) {
      if (o == b) continue;
      // how many of beam o's, best first, are ahead: larger, or as large and of a lower beam
      int lo = 0, hi = s_len[o];
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const double y = s_key[o][mid];
        if (y > key || (y == key && o < b))
          lo = mid + 1;
        else
          hi = mid;
      }
      place += lo;
    }
    if (place >= K) continue;
    const int out = group * K + place, token = s_token[b][e];
    a.out_tokens[out] = token;
    a.out_parents[out] = group * K + b;
    a.out_scores[out] = (float)key;
    a.out_ended[out] = (a.ended[group * K + b] != 0 || token == a.eos) ? 1 : 0;
  }
}

// Elements of a chunk: 32 per thread when that still leaves a CTA per SM and more, else 8, so
// that one row's logits spread over more SMs.
constexpr int kPerLarge = 32, kPerSmall = 8;
int chunk_of(long long rows, int vocab, int n_sm) {
  const long long large = kPerLarge * kScanThreads;
  return rows * ((vocab + large - 1) / large) >= n_sm ? (int)large : kPerSmall * kScanThreads;
}

size_t lay_out(SelectArgs* a, void* ws, long long rows, int beams, int chunks) {
  char* p = static_cast<char*>(ws);
  const size_t cand = round16(sizeof(u64) * rows * chunks * beams);
  a->cand = reinterpret_cast<u64*>(p);
  a->stat = reinterpret_cast<float4*>(p + cand);
  return cand + sizeof(float4) * rows * chunks;
}

template <typename T>
mk_status launch_scan(const SelectArgs& a, bool vec, void* stream) {
  const bool large = a.chunk == kPerLarge * kScanThreads;
  auto k = large ? (vec ? scan_kernel<T, kPerLarge, true> : scan_kernel<T, kPerLarge, false>)
                 : (vec ? scan_kernel<T, kPerSmall, true> : scan_kernel<T, kPerSmall, false>);
  return launch_dependent(k, dim3((unsigned)(a.rows * a.chunks)), dim3(kScanThreads), 0, stream, "mk_beam_select", a);
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_beam_select_workspace(int groups, int beams, int vocab, size_t* bytes) {
  using namespace mk;
  if (!bytes) return paged_fail(MK_ERR_INVALID, "bytes is NULL");
  if (groups < 1 || beams < 1 || beams > kMaxBeams || vocab < beams)
    return paged_fail(MK_ERR_INVALID, "groups must be positive, beams in [1, 32] and at most vocab");
  const long long rows = (long long)groups * beams;
  if (rows * (vocab / (kPerSmall * kScanThreads) + 1) > 0x7fffffffLL)
    return paged_fail(MK_ERR_INVALID, "groups * beams * vocab out of range");
  int n_sm = 0;
  const mk_status s = sm_count(&n_sm);
  if (s) return s;
  const int chunk = chunk_of(rows, vocab, n_sm);
  SelectArgs a{};
  *bytes = lay_out(&a, nullptr, rows, beams, (int)(((long long)vocab + chunk - 1) / chunk));
  return MK_OK;
}

extern "C" mk_status mk_beam_select(const mk_select_args* args, int32_t* status, void* stream) {
  using namespace mk;
  if (!args || !args->logits || !args->scores || !args->ended || !args->out_tokens || !args->out_parents ||
      !args->out_scores || !args->out_ended)
    return paged_fail(MK_ERR_INVALID, "NULL argument");
  if (args->dtype < MK_F16 || args->dtype > MK_F32) return paged_fail(MK_ERR_INVALID, "dtype");
  if (args->eos < -1 || args->eos >= args->vocab) return paged_fail(MK_ERR_INVALID, "eos must be a token or -1");
  if (args->row_stride < args->vocab) return paged_fail(MK_ERR_INVALID, "row_stride is smaller than vocab");
  const size_t esz = args->dtype == MK_F32 ? 4 : 2;
  if (!aligned_to(args->logits, esz)) return paged_fail(MK_ERR_INVALID, "logits must be aligned to their type");
  if ((const void*)args->out_scores == (const void*)args->scores || args->out_ended == args->ended)
    return paged_fail(MK_ERR_INVALID, "outputs must not overlap the inputs");
  if (!args->workspace || !aligned_to(args->workspace, 16))
    return paged_fail(MK_ERR_INVALID, "the workspace is missing or unaligned");
  size_t need = 0;
  mk_status s = mk_beam_select_workspace(args->groups, args->beams, args->vocab, &need);
  if (s) return s;
  if (args->workspace_bytes < need) return paged_fail(MK_ERR_INVALID, "the workspace is too small (mk_beam_select_workspace)");
  int n_sm = 0;
  s = sm_count(&n_sm);
  if (s) return s;
  SelectArgs a{};
  a.logits = args->logits; a.scores = args->scores; a.ended = args->ended;
  a.out_tokens = args->out_tokens; a.out_parents = args->out_parents; a.out_scores = args->out_scores;
  a.out_ended = args->out_ended; a.status = status;
  a.row_stride = args->row_stride; a.rows = args->groups * args->beams; a.beams = args->beams; a.vocab = args->vocab;
  a.chunk = chunk_of(a.rows, a.vocab, n_sm);
  a.chunks = (int)(((long long)a.vocab + a.chunk - 1) / a.chunk);
  a.eos = args->eos;
  lay_out(&a, args->workspace, a.rows, a.beams, a.chunks);
  const bool vec = aligned_to(args->logits, 16) && (args->row_stride * (long long)esz) % 16 == 0;
  s = args->dtype == MK_F32   ? launch_scan<float>(a, vec, stream)
      : args->dtype == MK_F16 ? launch_scan<__half>(a, vec, stream)
                              : launch_scan<__nv_bfloat16>(a, vec, stream);
  if (s) return s;
  return launch_dependent(pick_kernel, dim3(args->groups), dim3(kPickThreads), 0, stream, "mk_beam_select (pick)", a);
}
