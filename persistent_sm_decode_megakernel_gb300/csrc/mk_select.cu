// One step of a beam search over beams and vocabulary (mk_beam_select).
//
// A row's candidates are ordered by logit alone, so the log-softmax is not needed to choose
// among them: one pass over the logits yields, per part of a row, the maximum, the sum of
// exponentials and the part's `beams` largest logits; a second kernel (one CTA per group)
// joins the parts -- lse = M + log sum_c S_c e^(M_c - M), in 64 bits -- and picks the best of
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
constexpr int kIter = 16 * kScanThreads;  // elements of a step
constexpr int kList = 1024;               // entries of a CTA's list

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

// (-0 and +0 are one value, and so a tie)
__device__ __forceinline__ u64 key_of(float x, int token) {
  return (u64)orderable(x + 0.f) << 32 | (0xFFFFFFFFu - (unsigned)token);
}
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

// e^x for x <= 0: 2^(x log2 e) by the hardware's approximation, log2 e in two parts so that
// the product has no systematic error
__device__ __forceinline__ float exp_of(float x) {
  const float hi = 1.44269502162933349609375f, lo = 1.92596299112661746887e-8f;  // their sum is log2 e to 2^-50
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(x, lo, x * hi)));
  return y;
}

// a double as an unsigned number of the same order (NaN does not occur)
__device__ __forceinline__ u64 ordered(double x) {
  const u64 u = (u64)__double_as_longlong(x);
  return (u >> 63) ? ~u : u | (1ull << 63);
}

// A CTA reads its part of a row once, kIter elements at a time with the next ones in flight.
// The `beams` largest are kept in a list in shared memory, entered by what lies above a bound.
// The first bound comes from the lanes: the beams-th largest of a warp's 32 lane maxima has
// at least `beams` elements at or above it.  From then on it is the list's beams-th key: the
// list is cut down to its best after the first elements and whenever it has grown, each entry
// counting how many are above it, which is its place; of a part in random order about
// beams / i keys enter at the i-th elements.  Were one step's entries to overflow the list
// (rising logits), they come out one block maximum at a time.  The sum of exponentials runs
// against each thread's own maximum: fours in 32 bits, a compensated sum of them, and from
// there on in 64 bits, so that the sum of any vocabulary is good to a few 2^-24 of its terms.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kScanThreads, 4) scan_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ u64 s_list[kList], s_warp[kScanWarps];
  __shared__ double s_d[kScanWarps];
  __shared__ float s_f[kScanWarps];
  __shared__ int s_n[3];  // entries of the step, in turn: one is cleared while one is read
  constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;  // elements of an access
  constexpr int PER = kIter / kScanThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.beams;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  pdl_wait();
  pdl_launch();
  if (a.ended[row]) return;  // it offers one token, whatever its logits
  const T* src = static_cast<const T*>(a.logits) + (long long)row * a.row_stride;
  const int first = chunk * a.chunk, n = min(a.chunk, a.vocab - first);
  // element i * V + y of step `it` is token first + it * kIter + (i * 256 + tid) * V + y
  auto at = [&](int it, int i) { return it * kIter + ((i / V) * kScanThreads + tid) * V + i % V; };
  auto load = [&](int it, float (&x)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; i += V) {
      const int e = at(it, i);
      if (VEC && e + V <= n) {
        alignas(16) T raw[V];
        *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(src + first + e);
#pragma unroll
        for (int y = 0; y < V; ++y) x[i + y] = Conv<T>::up(raw[y]);
      } else {
#pragma unroll
        for (int y = 0; y < V; ++y) x[i + y] = e + y < n ? Conv<T>::up(src[first + e + y]) : -INFINITY;
      }
    }
  };
  if (tid < 3) s_n[tid] = 0;
  float x[PER], next[PER];
  load(0, next);
  const int steps = (n + kIter - 1) / kIter;
  int held = 0;       // entries of the list
  u64 bound = 0ull;   // keys above it enter
  bool bad = false;
  float m = -INFINITY, s = 0.f, comp = 0.f;
  for (int it = 0; it < steps; ++it) {
    float top = -INFINITY, q = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      x[i] = next[i];
      top = fmaxf(top, x[i]);
      q = fmaf(0.f, x[i], q);  // NaN as soon as one is not finite
    }
    if (it + 1 < steps) load(it + 1, next);
    if (q != q) {  // -inf is a value; NaN and +inf are reported and count as -inf
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (!(x[i] < INFINITY)) {
          bad = true;
          x[i] = -INFINITY;
        }
        top = fmaxf(top, x[i]);
      }
    }
    if (it == 0) {
      // the lane's own largest key: the first element that reaches top (none in an empty tail)
      int best = -1;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i)
        if (x[i] == top && at(0, i) < n) best = at(0, i);
      u64 left = best >= 0 ? key_of(top, first + best) : 0ull, kth = 0ull;
      for (int b = 0; b < K; ++b) {
        kth = warp_max(left);
        if (kth == 0ull) break;  // fewer lanes with elements than beams: no bound from this warp
        if (left == kth) left = 0ull;
      }
      if (lane == 0) s_warp[warp] = kth;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kScanWarps; ++w) bound = s_warp[w] > bound ? s_warp[w] : bound;
      if (bound) --bound;  // that key itself enters
    }
    if (orderable(top) >= (uint32_t)(bound >> 32)) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const u64 k = key_of(x[i], first + at(it, i));
        if (k <= bound || at(it, i) >= n) continue;
        const int p = held + atomicAdd(&s_n[it % 3], 1);
        if (p < kList) s_list[p] = k;
      }
    }
    if (top > m) {
      if (m > -INFINITY) {
        const float f = exp_of(m - top);
        s *= f;
        comp *= f;
      }
      m = top;
    }
    if (m > -INFINITY) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const float q = (exp_of(x[i] - m) + exp_of(x[i + 1] - m)) + (exp_of(x[i + 2] - m) + exp_of(x[i + 3] - m));
        const float t = s + q, r = t - s;  // t + the bracket below is s + q exactly
        comp += (s - (t - r)) + (q - r);
        s = t;
      }
    }
    if (tid == 0) s_n[(it + 1) % 3] = 0;
    __syncthreads();
    int count = held + s_n[it % 3];
    if (count > kList) {  // the step's entries one by one: the largest below the last one taken
      u64 last = ~0ull;
      for (int b = 0; b < K; ++b) {
        u64 k = 0ull;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const u64 y = key_of(x[i], first + at(it, i));
          if (at(it, i) < n && y > bound && y < last && y > k) k = y;
        }
        k = warp_max(k);
        __syncthreads();
        if (lane == 0) s_warp[warp] = k;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) k = s_warp[w] > k ? s_warp[w] : k;
        if (tid == 0) s_list[held + b] = k;  // held <= kList / 2
        last = k;
      }
      count = held + K;
      __syncthreads();
    }
    held = count;
    if (it == 0 || it == steps - 1 || count > kList / 2) {  // the list's best, in order
      u64 mine[kList / kScanThreads];
      int place[kList / kScanThreads];
#pragma unroll
      for (int q = 0; q < kList / kScanThreads; ++q) {
        const int e = q * kScanThreads + tid;
        place[q] = K;
        mine[q] = 0ull;
        if (e >= count) continue;
        mine[q] = s_list[e];
        int above = 0;
        for (int f = 0; f < count; ++f) above += s_list[f] > mine[q];
        place[q] = above;
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kList / kScanThreads; ++q)
        if (place[q] < K) s_list[place[q]] = mine[q];
      __syncthreads();
      held = min(count, K);
      if (held == K) bound = s_list[K - 1];
    }
  }
  if (bad) report(a.status, MK_ERR_NAN, PO_SELECT, row, chunk);
  u64* out = a.cand + ((long long)row * a.chunks + chunk) * K;
  for (int b = tid; b < K; b += kScanThreads) out[b] = b < held ? s_list[b] : 0ull;
  float M = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_f[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kScanWarps; ++w) M = fmaxf(M, s_f[w]);
  double d = 0.0;
  if (m > -INFINITY) {
    const float f = exp_of(m - M);
    d = ((double)s + (double)comp) * (double)f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) s_d[warp] = d;
  __syncthreads();
  if (tid == 0) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) sum += s_d[w];
    a.stat[(long long)row * a.chunks + chunk] = make_float4(M, (float)sum, (float)(sum - (double)(float)sum), 0.f);
  }
}

// One CTA per group, a warp per beam: the beam's best from its parts' lists (8 keys per lane
// in registers, the best so far carried from batch to batch), its lse, and its candidates'
// scores in 64 bits, kept as ordered integers; then every candidate's place among the group's
// is the sum over the beams of how many of that beam's sorted list are ahead of it.  Bound:
// one chain of loads, 64-bit exp and log, and the list steps; nothing here grows with vocab.
__global__ void __launch_bounds__(32 * kMaxBeams) pick_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ u64 s_key[kMaxBeams][kMaxBeams];
  __shared__ double s_score[kMaxBeams][kMaxBeams];
  __shared__ int s_token[kMaxBeams][kMaxBeams], s_len[kMaxBeams], s_ended[kMaxBeams];
  const int tid = threadIdx.x, lane = tid & 31, b = tid >> 5, group = blockIdx.x, K = a.beams;
  pdl_wait();
  pdl_launch();
  {
    const int row = group * K + b, total = a.chunks * K;
    const float4* st = a.stat + (long long)row * a.chunks;
    const u64* cand = a.cand + (long long)row * total;
    // everything the beam needs is asked for at once
    const int ended = a.ended[row];
    float sc = a.scores[row];
    float4 part = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    u64 k[8];
    if (!ended) {
      if (lane < a.chunks) part = st[lane];
#pragma unroll
      for (int x = 0; x < 8; ++x) k[x] = x * 32 + lane < total ? cand[x * 32 + lane] : 0ull;
    }
    if (!(sc == sc)) {
      if (lane == 0) report(a.status, MK_ERR_NAN, PO_SELECT, row, -1);
      sc = -INFINITY;
    }
    if (lane == 0) {
      s_len[b] = ended ? 1 : K;
      s_ended[b] = ended;
    }
    if (ended) {
      if (lane == 0) {
        s_score[b][0] = (double)sc;
        s_key[b][0] = ordered((double)sc);
        s_token[b][0] = a.eos;
      }
    } else {
      u64 mine = 0ull;  // lane q: the q-th best so far
      for (int base = 0; base < total; base += 256) {
        if (base) {
#pragma unroll
          for (int x = 0; x < 8; ++x) k[x] = base + x * 32 + lane < total ? cand[base + x * 32 + lane] : 0ull;
        }
        const int rows = min(8, (total - base + 31) / 32);  // registers in use
        u64 carry = mine;
        for (int q = 0; q < K; ++q) {
          u64 best = carry;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (x < rows) best = k[x] > best ? k[x] : best;
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
      float m = part.x;
      for (int c = lane + 32; c < a.chunks; c += 32) m = fmaxf(m, st[c].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      double sum = 0.0;
      for (int c = lane; c < a.chunks; c += 32) {
        if (c >= 32) part = st[c];
        if (part.x > -INFINITY) sum += ((double)part.y + (double)part.z) * exp((double)part.x - (double)m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const double lse = m > -INFINITY ? (double)m + log(sum) : 0.0;
      if (lane < K) {
        const float v = value_of(mine);
        double s = v > -INFINITY ? (double)sc + ((double)v - lse) : -INFINITY;
        if (!(s == s)) s = -INFINITY;
        s_score[b][lane] = s;
        s_key[b][lane] = ordered(s);
        s_token[b][lane] = token_of(mine);
      }
    }
  }
  __syncthreads();
  for (int x = tid; x < K * K; x += 32 * K) {
    const int b = x / K, e = x % K;
    if (e >= s_len[b]) continue;
    const u64 key = s_key[b][e];
    int place = e;
    for (int o = 0; o < K; ++o) {
      if (o == b) continue;
      // how many of beam o's, best first, are ahead: larger, or as large and of a lower beam
      int lo = 0, hi = s_len[o];
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_key[o][mid] >= key + (o < b ? 0 : 1))
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
    a.out_scores[out] = (float)s_score[b][e];
    a.out_ended[out] = (s_ended[b] != 0 || token == a.eos) ? 1 : 0;
  }
}

// Elements of a CTA's part of a row: the rows' parts fill the resident CTAs (4 per SM) once,
// in whole groups of accesses (2048), and down to one group per CTA when there are few rows.
constexpr int kPart = 8 * kScanThreads;
int chunk_of(long long rows, int vocab, int n_sm) {
  const long long parts = std::max(1LL, 4LL * n_sm / rows), each = ((long long)vocab + parts - 1) / parts;
  return (int)std::min((each + kPart - 1) / kPart * kPart, 1LL << 30);
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
  auto k = vec ? scan_kernel<T, true> : scan_kernel<T, false>;
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
  if (rows * (vocab / kPart + 1) > 0x7fffffffLL)
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
  return launch_dependent(pick_kernel, dim3(args->groups), dim3(32 * args->beams), 0, stream, "mk_beam_select (pick)", a);
}
