// One step of a beam search over beams and vocabulary (mk_beam_select).
//
// A row's candidates are ordered by logit alone, so the log-softmax is not needed to choose
// among them: one pass over the logits yields, per part of a row, the maximum, the sum of
// exponentials and the part's `beams` largest logits; a second kernel (one CTA per group)
// joins the parts -- lse = N ln 2 + ln sum_c S_c 2^(N_c - N) -- and picks the best of
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
constexpr float kLargest = 0x1p126f;  // of a logit: beyond it lies infinity
// Up to here x log2 e, rounded to a whole number n in 32 bits, is off by less than 0.1, so that
// 2^(x log2 e - n) is at most about 1; from 2^32 on the rounding alone is worth 128 powers of two
constexpr float kNear = 0x1p20f;
constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
// elements of a step per thread, and CTAs per SM: one short step, or several long ones (a step
// costs about 90 instructions beside its 6 per element; 128 rows of 128256: 18.4 us, steps of
// half the length in twice the CTAs 20.2, CTAs of 128 threads 19.8 to 24)
constexpr int kPerSmall = 8, kCtasSmall = 4, kPerLarge = 32, kCtasLarge = 2;
constexpr int kList = 1024;               // entries of a CTA's list

using u64 = unsigned long long;

// of a part of a row: n, and the sum of 2^(x log2 e - n) in units of 2^-sum_bits; far: n is the
// part's largest logit, and the sum that of e^(x - n)
struct __align__(16) Stat {
  float n;
  int far;
  u64 sum;
};

struct SelectArgs {
  const void* logits;
  const float* scores;
  const int32_t* ended;
  int32_t *out_tokens, *out_parents, *out_ended, *status;
  float* out_scores;
  u64* cand;        // [rows][chunks][beams], best first; 0: none
  Stat* stat;       // [rows][chunks]
  long long row_stride;
  int rows, beams, vocab, chunk, chunks, eos, sum_bits;
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

// the least logit above x (x not +inf): what lies below -kLargest is -inf
__device__ __forceinline__ float above(float x) {
  const uint32_t u = orderable(x + 0.f) + 1u;
  return value_of((u64)(x == -INFINITY ? orderable(-kLargest) : u) << 32);
}

// the largest of the warp's keys (each lane's own, 0: none)
__device__ __forceinline__ u64 warp_max(u64 k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (u64)hi << 32 | lo;
}

// 2^(x log2 e - n) by the hardware's approximation; log2 e in two parts, so that the exponent
// is off by its own rounding alone
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.92596299112661746887e-8f;  // to 2^-50
__device__ __forceinline__ float term_of(float x, float n) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(x, kLog2eLo, fmaf(x, kLog2eHi, -n))));
  return y;
}
// the same of a natural exponent y, the difference of two logits
__device__ __forceinline__ float exp_of(float y) { return term_of(y, 0.f); }
// 2^d for a whole d in [-126, 127], exactly; 0 below
__device__ __forceinline__ float power_of(float d) { return d < -126.f ? 0.f : __int_as_float((127 + (int)d) << 23); }

// Numbers as a pair of floats (hi + lo, |lo| at most half a step of hi), so that scores are
// compared before they are rounded to 32 bits (a score of -100 has steps of 2^-17 there; the
// log-sum-exp in it is good to 2^-19, so that no more than that is decided): 48 bits, from
// 32-bit instructions -- 64-bit log alone took 1.3 us of a launch of 5.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float x, float y) {
  const float s = x + y, r = s - x;
  return {s, (x - (s - r)) + (y - r)};
}
// ln(u 2^shift), u > 0: u = 2^e f with f in [0.7, 1.42), ln f = 2 t + 2 t^3 / 3 + .. of
// t = (f - 1) / (f + 1), |t| < 0.18.  The leading term is taken in pairs, the others (below
// 0.004) in 32 bits: off by less than 2^-30 and the pair's own rounding.
__device__ __forceinline__ Pair ln_of(u64 u, float shift) {
  const int z = __clzll((long long)(u | 1));
  const u64 m = u << z;                     // the leading bit on top
  const bool half = (m >> 48) > 0xB504u;    // f above sqrt 2: take f / 2
  const float unit = half ? 0x1p-24f : 0x1p-23f;
  const float fh = (float)(unsigned)(m >> 40) * unit, fl = (float)(unsigned)((m >> 16) & 0xFFFFFFu) * (unit * 0x1p-24f);
  const float e = (float)(63 - z + (half ? 1 : 0)) + shift;
  const float nh = fh - 1.f;                // exact
  const Pair den = two_sum(fh, 1.f);
  float inv;  // approximate: what it leaves over goes into tl
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(den.hi));
  const float th = nh * inv;
  const float tl = (fmaf(-th, den.hi, nh) + (fl - th * (den.lo + fl))) * inv;
  const float w = th * th;
  const float rest = w * fmaf(w, fmaf(w, fmaf(w, fmaf(w, fmaf(w, 2.f / 13, 2.f / 11), 2.f / 9), 2.f / 7), 2.f / 5), 2.f / 3);
  const float l2h = 0.693147182464599609375f, l2l = -1.90465429995776804525e-9f;  // ln 2 to 2^-52
  const float ph = e * l2h, pl = fmaf(e, l2h, -ph) + e * l2l;
  const Pair s = two_sum(ph, 2.f * th);
  return two_sum(s.hi, s.lo + (pl + fmaf(th, rest, 2.f * tl)));
}
// score + (v - lse), -inf where it lies below the floats, and a pair as an unsigned number of
// the same order
__device__ __forceinline__ Pair score_of(float score, float v, Pair lse) {
  const Pair d = two_sum(v, -lse.hi), s = two_sum(score, d.hi);
  const Pair t = two_sum(s.hi, s.lo + (d.lo - lse.lo));
  return t.hi > -INFINITY ? t : Pair{-INFINITY, 0.f};  // (past the range t is NaN)
}
__device__ __forceinline__ u64 ordered(Pair p) { return (u64)orderable(p.hi + 0.f) << 32 | orderable(p.lo + 0.f); }

// A CTA reads its part of a row once, kIter elements at a time with the next ones in flight.
// The `beams` largest are kept in a list in shared memory, entered by what lies above a bound.
// The first bound comes from the lanes' maxima.  From then on it is the list's beams-th key: the
// list is cut down to its best after steps 1, 4, 16, .., each entry counting how many are
// above it, which is its place; of a part in random order about three times `beams` keys
// enter between two of those (no cut after the first step: 24.8 us for 128 rows of 128256, in
// place of 18.4; one after every step: 22.3).  Should the list overflow (rising
// logits, or equal ones in the first step), what came since the last cut is read again, once
// per beam.  The sum of exponentials runs against whole powers of two, so that joining threads,
// steps and parts rounds nothing: a step's in 32 bits, a compensated sum of them per thread,
// and from there on whole numbers.  Bound: the logits' bytes for many rows (the arithmetic, one
// exponential each, is most of that time again), the launch and the block steps for few.
// That holds for logits up to kNear in magnitude.  A step of a thread whose largest logit lies
// beyond takes no part: it counts for nothing beside a part whose largest logit is within, and
// a part whose largest logit is beyond (all masked by a large finite number; it is known after
// the last cut) is read once more, its sum against that logit itself, x - max being exact where
// it matters.
// (Both kernels, 4 rows of 32000: 5.3 us; 128 of 128256, 66 MB: 18.4 us, 3.6 TB/s.)
template <typename T, bool VEC, int PER>
__global__ void __launch_bounds__(kScanThreads, PER == kPerLarge ? kCtasLarge : kCtasSmall) scan_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ u64 s_list[kList], s_warp[kScanWarps];
  __shared__ float s_f[kScanWarps];
  __shared__ int s_n;
  constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;  // elements of an access
  constexpr int kIter = PER * kScanThreads;         // elements of a step
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.beams;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  pdl_wait();
  pdl_launch();
  if (a.ended[row]) return;  // it offers one token, whatever its logits
  const int first = chunk * a.chunk, n = min(a.chunk, a.vocab - first);
  const T* src = static_cast<const T*>(a.logits) + (long long)row * a.row_stride + first;
  // element i * V + y of step `it` is token first + it * kIter + (i * 256 + tid) * V + y
  auto at = [&](int it, int i) { return it * kIter + ((i / V) * kScanThreads + tid) * V + i % V; };
  auto load = [&](int it, float (&x)[PER]) {
    if (VEC && (it + 1) * kIter <= n) {
#pragma unroll
      for (int i = 0; i < PER; i += V) {
        alignas(16) T raw[V];
        *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(src + at(it, i));
#pragma unroll
        for (int y = 0; y < V; ++y) x[i + y] = Conv<T>::up(raw[y]);
      }
    } else {  // a part's last step: what lies in it
#pragma unroll
      for (int i = 0; i < PER; i += V) {
        const int e = at(it, i);
        if (VEC && e + V <= n) {
          alignas(16) T raw[V];
          *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(src + e);
#pragma unroll
          for (int y = 0; y < V; ++y) x[i + y] = Conv<T>::up(raw[y]);
        } else {
#pragma unroll
          for (int y = 0; y < V; ++y) x[i + y] = e + y < n ? Conv<T>::up(src[e + y]) : -INFINITY;
        }
      }
    }
  };
  if (tid == 0) s_n = 0;
  float x[PER], next[PER];
  load(0, next);
  const int steps = (n + kIter - 1) / kIter;
  float floor_ = -INFINITY;    // logits below it do not enter
  int cut = 1;                 // the list is cut down after this many steps
  int kept = 0, from = 0;      // entries of the list after the last cut, and elements before it
  bool bad = false;
  float ref = -INFINITY, s = 0.f, comp = 0.f;  // (s + comp) 2^ref: the thread's sum of e^x
  for (int it = 0; it < steps; ++it) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      x[i] = next[i];
      top = fmaxf(top, x[i]);
    }
    if (it + 1 < steps) load(it + 1, next);
    // the step's sum against a whole power of two at or above the thread's largest: sums
    // under another power are rescaled without rounding
    float q = 0.f;
    auto terms = [&] {
      const float up = ceilf(top * kLog2eHi);
      if (up > ref) {
        if (ref > -INFINITY) {
          const float f = power_of(ref - up);
          s *= f;
          comp *= f;
        }
        ref = up;
      }
      float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < PER; ++i) w[i % 4] += term_of(x[i], ref);
      q = (w[0] + w[1]) + (w[2] + w[3]);
    };
    if (fabsf(top) <= kNear) {
      terms();
    } else if (fabsf(top) <= kLargest) {
#pragma unroll
      for (int i = 0; i < PER; ++i) q = fmaf(x[i], 0.f, q);  // 0, or NaN where something is to be looked at
    }
    if (!(fabsf(top) <= kLargest) || q != q) {  // NaN and +inf are reported and count as -inf
      top = -INFINITY;
      q = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (!(x[i] <= kLargest)) {
          bad = true;
          x[i] = -INFINITY;
        }
        if (x[i] < -kLargest) x[i] = -INFINITY;
        top = fmaxf(top, x[i]);
      }
      if (fabsf(top) <= kNear) terms();
    }
    const float sum = s + q, r = sum - s;  // sum + the bracket below is s + q exactly
    comp += (s - (sum - r)) + (q - r);
    s = sum;
    if (it == 0) {
      // a warp's r-th largest lane maximum, r = beams / 8 rounded up: the least of the warps'
      // has at least `beams` elements at or above it (a warp with fewer lanes sets no bound)
      float left = at(0, 0) < n ? top : -INFINITY, kth = -INFINITY;
      for (int b = 0; b < (K + kScanWarps - 1) / kScanWarps; ++b) {
        const uint32_t u = __reduce_max_sync(0xffffffffu, orderable(left));
        kth = value_of((u64)u << 32);
        const unsigned who = __ballot_sync(0xffffffffu, orderable(left) == u);
        if (lane == __ffs(who) - 1) left = -INFINITY;
      }
      if (lane == 0) s_f[warp] = kth;
      __syncthreads();
      floor_ = s_f[0];
#pragma unroll
      for (int w = 1; w < kScanWarps; ++w) floor_ = fminf(floor_, s_f[w]);
    }
    if (top >= floor_) {
      unsigned hits = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) hits |= x[i] >= floor_ ? 1u << i : 0u;
      while (hits) {
        const int i = __ffs(hits) - 1;
        hits &= hits - 1;
        const int e = at(it, i);
        float y = x[0];
#pragma unroll
        for (int z = 1; z < PER; ++z) y = z == i ? x[z] : y;
        if (e >= n) continue;
        const u64 k = key_of(y < -kLargest ? -INFINITY : y, first + e);
        const int p = atomicAdd(&s_n, 1);
        if (p < kList) s_list[p] = k;
      }
    }
    if (it + 1 == cut)
      cut *= 4;
    else if (it + 1 < steps)
      continue;
    // ---- after steps 1, 4, 16, .. and the last: the list's best, in order
    __syncthreads();
    int count = s_n;
    const int seen = min(n, (it + 1) * kIter);
    if (count > kList) {  // too many: the largest since the last cut and of its list one by one, each below the last
      u64 last = ~0ull;
      for (int b = 0; b < K; ++b) {
        u64 k = tid < kept && s_list[tid] < last ? s_list[tid] : 0ull;
#pragma unroll 16
        for (int e = from + tid; e < seen; e += kScanThreads) {
          float y = Conv<T>::up(src[e]);
          if (!(y <= kLargest) || y < -kLargest) y = -INFINITY;
          const u64 z = key_of(y, first + e);
          if (z < last && z > k) k = z;
        }
        k = warp_max(k);
        __syncthreads();
        if (lane == 0) s_warp[warp] = k;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) k = s_warp[w] > k ? s_warp[w] : k;
        if (tid == 0) s_list[kList - K + b] = k;  // (what entered there is in memory still)
        last = k;
      }
      count = K;
      __syncthreads();
      if (tid < K) s_list[tid] = s_list[kList - K + tid];
      __syncthreads();
    } else {
      // a short list takes a pair of threads per entry, each counting over one half
      const int share = count <= kScanThreads / 2 ? 2 : 1, part = share == 2 ? tid & 1 : 0;
      const int f0 = part ? (count + 1) / 2 : 0, f1 = share == 2 && !part ? (count + 1) / 2 : count;
      u64 mine[kList / kScanThreads];
      int place[kList / kScanThreads];
#pragma unroll
      for (int z = 0; z < kList / kScanThreads; ++z) {
        place[z] = K;
        mine[z] = 0ull;
        if (z * kScanThreads >= count) continue;  // uniform
        const int e = z * kScanThreads + tid / share;
        int above = 0;
        if (e < count) {
          mine[z] = s_list[e];
#pragma unroll 4
          for (int f = f0; f < f1; ++f) above += s_list[f] > mine[z];
        }
        if (share == 2) above += __shfl_xor_sync(0xffffffffu, above, 1);
        if (e < count) place[z] = above;
      }
      __syncthreads();
#pragma unroll
      for (int z = 0; z < kList / kScanThreads; ++z)
        if (place[z] < K) s_list[place[z]] = mine[z];
    }
    if (tid == 0) s_n = min(count, K);
    __syncthreads();
    kept = min(count, K);
    from = seen;
    // of what follows, equal logits lose to the list's, whose tokens are lower
    if (count >= K) floor_ = above(value_of(s_list[K - 1]));
  }
  if (bad) report(a.status, MK_ERR_NAN, PO_SELECT, row, chunk);
  u64* out = a.cand + ((long long)row * a.chunks + chunk) * K;
  for (int b = tid; b < K; b += kScanThreads) out[b] = b < s_n ? s_list[b] : 0ull;
  const float largest = value_of(s_list[0]);
  // (256 below the bound: what is left out then is less than e^-256 of the part's largest term)
  const bool far = fabsf(largest) > kNear - 256.f && fabsf(largest) <= kLargest;
  if (far) {
    ref = s = comp = 0.f;
    for (int it = 0; it < steps; ++it) {
      load(it, x);
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float y = x[i] <= kLargest ? exp_of(x[i] - largest) : 0.f;
        q += y;
      }
      const float sum = s + q, r = sum - s;
      comp += (s - (sum - r)) + (q - r);
      s = sum;
    }
  }
  float top_ref = ref;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top_ref = fmaxf(top_ref, __shfl_xor_sync(0xffffffffu, top_ref, o));
  if (lane == 0) s_f[warp] = top_ref;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kScanWarps; ++w) top_ref = fmaxf(top_ref, s_f[w]);
  // the thread's sum as a whole number of units: exact sums from here on, in any order
  u64 d = 0;
  if (ref > -INFINITY) {
    const float f = power_of(ref - top_ref), unit = power_of((float)a.sum_bits);
    d = (u64)__float2ull_rn(s * f * unit) + (u64)__float2ll_rn(comp * f * unit);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) s_warp[warp] = d;
  __syncthreads();
  if (tid == 0) {
    u64 all = 0;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) all += s_warp[w];
    a.stat[(long long)row * a.chunks + chunk] = Stat{far ? largest : top_ref, far, all};
  }
}

// The warp's K largest of R keys per lane and of *best (lane q: the q-th largest so far), into
// *best.  Keys differ, 0 is none.  A lane's keys are sorted first, so that taking one is a
// shift (looking for the next largest each time: a call of 2 x 32 of 32000 34.6 us in place of 24.8).
template <int R>
__device__ __forceinline__ void take_best(const u64 (&k)[8], int K, int lane, u64* best) {
  u64 s[R + 1];
#pragma unroll
  for (int x = 0; x < R; ++x) s[x] = k[x];
  s[R] = *best;
#pragma unroll
  for (int x = R; x > 0; --x)
#pragma unroll
    for (int y = 0; y < x; ++y) {
      const u64 hi = s[y] > s[y + 1] ? s[y] : s[y + 1], lo = s[y] > s[y + 1] ? s[y + 1] : s[y];
      s[y] = hi;
      s[y + 1] = lo;
    }
  u64 mine = 0ull;
#pragma unroll 1
  for (int q = 0; q < K; ++q) {  // (without branches: twice as fast)
    const u64 win = warp_max(s[0]);
    const bool taken = s[0] == win;
    mine = lane == q ? win : mine;
#pragma unroll
    for (int x = 0; x < R; ++x) s[x] = taken ? s[x + 1] : s[x];
    s[R] = taken ? 0ull : s[R];
  }
  *best = mine;
}

// One CTA per group, a warp per beam: the beam's best from its parts' lists (8 keys per lane
// in registers, the best so far carried from batch to batch), its lse, and its candidates'
// scores as pairs of floats, compared as ordered integers; then the beams' lists, each sorted,
// are merged, a lane per beam.  Bound: one chain of loads, the logarithm and the list steps,
// each instruction waiting for the last.  Every warp goes through all of its beam's part, ended beam or not:
// inside a branch that the compiler cannot see to be the same for a whole warp, a shuffle took
// 285 cycles and a reduction 700, in place of 17 and 22 (the kernel 9500, in place of 3500).
__global__ void __launch_bounds__(32 * kMaxBeams) pick_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ u64 s_key[kMaxBeams][kMaxBeams];
  __shared__ float s_score[kMaxBeams][kMaxBeams];
  __shared__ int s_token[kMaxBeams][kMaxBeams], s_len[kMaxBeams], s_ended[kMaxBeams];
  const int lane = threadIdx.x & 31, b = threadIdx.x >> 5, group = blockIdx.x, K = a.beams;
  const int row = group * K + b, total = a.chunks * K;
  const Stat* st = a.stat + (long long)row * a.chunks;
  const u64* cand = a.cand + (long long)row * total;
  pdl_wait();
  pdl_launch();
  // everything the beam needs is asked for at once (of an ended one nothing was written, and
  // what is computed from that is not used)
  const int ended = a.ended[row];
  float sc = a.scores[row];
  Stat part{-INFINITY, 0, 0ull};
  if (lane < a.chunks) part = st[lane];
  u64 k[8];
  k[0] = lane < total ? cand[lane] : 0ull;
  k[1] = 32 + lane < total ? cand[32 + lane] : 0ull;
  if (total > 64) {
#pragma unroll
    for (int x = 2; x < 8; ++x) k[x] = x * 32 + lane < total ? cand[x * 32 + lane] : 0ull;
  }
  const bool no_score = !(sc < INFINITY);
  sc = no_score ? -INFINITY : sc;
  // the parts' sums against the largest power: whole numbers, shifted
  float ref = part.n;
  for (int c = 32; c < a.chunks; c += 32) ref = fmaxf(ref, c + lane < a.chunks ? st[c + lane].n : -INFINITY);
  ref = value_of((u64)__reduce_max_sync(0xffffffffu, orderable(ref)) << 32);
  auto share = [&](const Stat& s) { return s.n > ref - 64.f ? s.sum >> (int)(ref - s.n) : 0ull; };
  u64 sum = share(part);
  for (int c = 32; c < a.chunks; c += 32) sum += share(c + lane < a.chunks ? st[c + lane] : Stat{-INFINITY, 0, 0ull});
  int far = part.far;
  for (int c = 32; c < a.chunks; c += 32) far |= c + lane < a.chunks ? st[c + lane].far : 0;
  far = __any_sync(0xffffffffu, far);
  float base = 0.f;  // the row's sum is e^base 2^shift times the whole number
  if (far) {
    // a part against its largest logit: the row's sum against the row's, natural exponents
    base = -INFINITY;
    for (int c = lane; c < a.chunks; c += 32) base = fmaxf(base, value_of(cand[c * K]));
    base = value_of((u64)__reduce_max_sync(0xffffffffu, orderable(base)) << 32);
    sum = 0ull;
    for (int c = lane; c < a.chunks; c += 32) {
      const Stat p = st[c];
      const float f = p.far ? exp_of(p.n - base) : p.n > -INFINITY ? term_of(-base, -p.n) : 0.f;
      sum += __double2ull_rn(__ull2double_rn(p.sum) * f);
    }
    ref = 0.f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  Pair lse = ln_of(sum, ref - (float)a.sum_bits);
  if (far) {
    const Pair p = two_sum(base, lse.hi);
    lse = two_sum(p.hi, p.lo + lse.lo);
  }
  u64 mine = 0ull;  // lane q: the q-th best
  if (total <= 64)
    take_best<2>(k, K, lane, &mine);
  else
    for (int base = 0; base < total; base += 256) {
      if (base) {
#pragma unroll
        for (int x = 0; x < 8; ++x) k[x] = base + x * 32 + lane < total ? cand[base + x * 32 + lane] : 0ull;
      }
      take_best<8>(k, K, lane, &mine);
    }
  if (lane < K) {
    const float v = value_of(mine);
    Pair s = ref > -INFINITY && v > -INFINITY && sc > -INFINITY ? score_of(sc, v, lse) : Pair{-INFINITY, 0.f};
    if (ended) s = Pair{sc, 0.f};
    s_score[b][lane] = s.hi;
    s_key[b][lane] = ordered(s);
    s_token[b][lane] = ended ? a.eos : token_of(mine);
  }
  if (lane == 0) {
    s_len[b] = ended ? 1 : K;
    s_ended[b] = ended;
    if (no_score) report(a.status, MK_ERR_NAN, PO_SELECT, row, -1);
  }
  __syncthreads();
  if (b) return;  // (23.1 us for 2 x 32 of 32000, in place of 24.8 with every warp alike)
  // lane o holds beam o's best that is not yet taken
  u64 head = lane < K ? s_key[lane][0] : 0ull;
  int next = 1, from = 0, entry = 0;
  const int len = lane < K ? s_len[lane] : 0;
#pragma unroll 1
  for (int q = 0; q < K; ++q) {
    const u64 win = warp_max(head);
    const int who = __ffs(__ballot_sync(0xffffffffu, head == win)) - 1;  // ties: the lowest beam
    const int taken = __shfl_sync(0xffffffffu, next, who) - 1;
    from = lane == q ? who : from;
    entry = lane == q ? taken : entry;
    if (lane == who) {
      head = next < len ? s_key[lane][next] : 0ull;
      ++next;
    }
  }
  if (lane < K) {
    const int out = group * K + lane, token = s_token[from][entry];
    a.out_tokens[out] = token;
    a.out_parents[out] = group * K + from;
    a.out_scores[out] = s_score[from][entry];
    a.out_ended[out] = (s_ended[from] != 0 || token == a.eos) ? 1 : 0;
  }
}

// Elements of a CTA's part of a row: the rows' parts fill the resident CTAs once -- of long steps
// when a part is then longer than one of them, else of short steps (2048 elements; one each where
// there are CTAs for it), so that few rows still spread over many SMs.
constexpr int kPart = kPerSmall * kScanThreads;
int chunk_of(long long rows, int vocab, int n_sm) {
  const long long parts = std::max(1LL, (long long)kCtasLarge * n_sm / rows), each = ((long long)vocab + parts - 1) / parts;
  if (each > kPerLarge * kScanThreads) return (int)std::min((each + kPart - 1) / kPart * kPart, 1LL << 30);
  const long long most = std::max(1LL, (long long)kCtasSmall * n_sm / rows);
  const long long one = ((long long)vocab + most - 1) / most;
  return one <= kPart ? kPart : (int)((one + kPart - 1) / kPart * kPart);
}

size_t lay_out(SelectArgs* a, void* ws, long long rows, int beams, int chunks) {
  char* p = static_cast<char*>(ws);
  const size_t cand = round16(sizeof(u64) * rows * chunks * beams);
  a->cand = reinterpret_cast<u64*>(p);
  a->stat = reinterpret_cast<Stat*>(p + cand);
  return cand + sizeof(Stat) * rows * chunks;
}

template <typename T>
mk_status launch_scan(const SelectArgs& a, bool vec, void* stream) {
  const bool small = a.chunk <= kPerLarge * kScanThreads;  // (a long step would not be full)
  auto k = small ? (vec ? scan_kernel<T, true, kPerSmall> : scan_kernel<T, false, kPerSmall>)
                 : (vec ? scan_kernel<T, true, kPerLarge> : scan_kernel<T, false, kPerLarge>);
  return launch_dependent(k, dim3((unsigned)(a.rows * a.chunks)), dim3(kScanThreads), 0, stream, "mk_beam_select", a);
}

}  // namespace
}  // namespace mk

extern "C" mk_status mk_beam_select_workspace(int groups, int beams, int vocab, size_t* bytes) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
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
  });
}

extern "C" mk_status mk_beam_select(const mk_select_args* args, int32_t* status, void* stream) {
  using namespace mk;
  return c_entry([&]() -> mk_status {
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
    a.sum_bits = 62;  // a row's sum, at most vocab, stays below 2^63
    while ((1LL << (62 - a.sum_bits)) < a.vocab) --a.sum_bits;
    lay_out(&a, args->workspace, a.rows, a.beams, a.chunks);
    const bool vec = aligned_to(args->logits, 16) && (args->row_stride * (long long)esz) % 16 == 0;
    s = args->dtype == MK_F32   ? launch_scan<float>(a, vec, stream)
        : args->dtype == MK_F16 ? launch_scan<__half>(a, vec, stream)
                                : launch_scan<__nv_bfloat16>(a, vec, stream);
    if (s) return s;
    return launch_dependent(pick_kernel, dim3(args->groups), dim3(32 * args->beams), 0, stream, "mk_beam_select (pick)", a);
  });
}
