// Beam search over a batch of groups of K beams: choosing the M best
// continuations of each group (gdn_beam_select), and moving the surviving
// beams' recurrent states into place (gdn_state_reorder).
//
// Selection.  A candidate is (beam k, token v) with the score
//   c = score_k + logit_kv - log sum_v' exp(logit_kv').
// Within a beam the order by c is the order by logit, so each row's best M are
// found from the logits alone while its sum is still being formed, and the
// logits are read once.  One kernel, a cluster of CTAs per group: the group's
// K rows, cut into S segments each, are dealt to the cluster's CTAs.  A CTA
// forms a segment's maximum and sum of exponentials and its best M as 64-bit
// keys (ordered value, then the complement of the index: keys are distinct, and
// the lower index wins a tie), and leaves them in the first CTA's shared
// memory, which then forms the rows' log sums and merges the K S lists by score
// (64-bit floating point, ties to the lowest beam, then to the largest logit, then
// to the lowest token).
// Work is cut by element index, never by address, so rows with equal logits
// get equal sums bit for bit, wherever they lie.
//
// The best M of n values, by 256 threads, without sorting them: each thread's
// largest; of those, the largest of each of g >= M groups of threads; the
// least of these g has at least M values at or above it, and in random data
// about g ln g.  These are collected and ranked by counting.
//
// What bounds it: for one group the chain behind the last load, which no other
// work hides (best of the threads, limit, second look, rank, cluster, merge), on
// the 16 SMs of one cluster; for many, about 90 instructions a vector of 8
// elements, 32 of them for the sum of exponentials, at 44% of the issue rate with 14
// warps on an SM.  Measured on a B200 (calls in a CUDA graph), bf16: 1 group, K = 4,
// V = 32000, M = 8 9.9 us, of which the chain is about 8; 1 group, K = 8, V =
// 130000, M = 16 15.4; 32 groups, K = 8, V = 130001 in rows of 130048, M = 16 29.2 us
// (66.6 MB, 2.3 TB/s of the copy's 6.5).  fp32, the same 32 groups: 41.5 us.  A
// mask of -inf or -1e9 over 99 % of the tokens costs nothing (29.0); one of the
// type's lowest value, whose rows are read a second time from the caches by the
// threads that have met nothing else, 48.7.
#include <float.h>

#include <atomic>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCap = 1024;  // candidates of one segment held at once
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNear = 1073741824.f;  // 2^30: see Offset

// Order-preserving map of a float (not NaN; -0 taken as +0) to an unsigned.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ u64 key_of(float x, uint32_t idx) {
  return (u64)ordered(x) << 32 | (uint32_t)~idx;
}
// What a logit counts as: NaN as -inf (never chosen before a number).
__device__ __forceinline__ float tame(float x) { return fmaxf(x, -INFINITY); }
// a - b, 0 for equal infinities: where the largest is +inf, the entries that are
// it share the row equally and the others have nothing.
__device__ __forceinline__ float gap(float a, float b) {
  return a == b ? 0.f : __fadd_rn(a, -b);
}

// 16 bytes of a row as floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  // the largest (of numbers, where there are any)
  static __device__ __forceinline__ float top(const uint4& r) {
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                 fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  static __device__ __forceinline__ void get(const uint4& r, float* f) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ float top(const uint4& r) {
    auto p = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 m = __hmax2(__hmax2(p(r.x), p(r.y)), __hmax2(p(r.z), p(r.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void get(const uint4& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// One row, read as vectors of 16 bytes by element index whatever its address.  A
// row that begins on 16 bytes gives a vector in one load.  Any other gives
// aligned words, five where elements of 2 bytes begin in the middle of one, which
// are shifted together only when they are used, so that loads stay in
// flight.  Nothing outside the row is touched: vectors whose words would
// reach over either end are gathered element by element.
template <typename T>
struct Row {
  struct Raw {
    uint32_t w[5];
  };
  const T* p;
  int64_t V;
  bool whole;     // begins on 16 bytes
  uint32_t bits;  // of the first word before the vector

  __device__ __forceinline__ Row(const T* row, int64_t v) : p(row), V(v) {
    const uint32_t at = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
    whole = at == 0;
    bits = (at & 3u) * 8u;
  }
  static __device__ __forceinline__ Raw none() {  // -inf throughout
    Raw r;
#pragma unroll
    for (int k = 0; k < 5; ++k) r.w[k] = Vec<T>::kNegInf;
    return r;
  }
  __device__ __forceinline__ Raw load(int64_t i) const {  // elements i .. i + Vec::n - 1
    constexpr int E = Vec<T>::n;
    Raw r;
    if (whole && i + E <= V) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p + i));
      r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
      r.w[4] = 0;
    } else if (!whole && (bits == 0 || i > 0) && i + E < V) {
      const uint32_t* q =
          reinterpret_cast<const uint32_t*>(reinterpret_cast<const char*>(p + i) - bits / 8);
#pragma unroll
      for (int k = 0; k < 4; ++k) r.w[k] = __ldg(q + k);
      r.w[4] = E == 8 && bits != 0 ? __ldg(q + 4) : 0;
    } else {
      uint32_t o[6];  // the vector's words, none before and behind
      o[0] = o[5] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (E == 4) {
          o[k + 1] = i + k < V ? reinterpret_cast<const uint32_t*>(p)[i + k] : Vec<T>::kNegInf;
        } else {
          const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
          const uint32_t lo = i + 2 * k < V ? h[i + 2 * k] : 0xff80u;
          const uint32_t hi = i + 2 * k + 1 < V ? h[i + 2 * k + 1] : 0xff80u;
          o[k + 1] = lo | hi << 16;
        }
      }
#pragma unroll
      for (int k = 0; k < 5; ++k) r.w[k] = __funnelshift_l(o[k], o[k + 1], bits);
    }
    return r;
  }
  __device__ __forceinline__ uint4 get(const Raw& r) const {
    return make_uint4(__funnelshift_r(r.w[0], r.w[1], bits), __funnelshift_r(r.w[1], r.w[2], bits),
                      __funnelshift_r(r.w[2], r.w[3], bits), __funnelshift_r(r.w[3], r.w[4], bits));
  }
};

// What a sum of exp(x - m) subtracts: c = fl(m log2 e), so that a term is 2^(x
// log2 e - c), one instruction.  c lacks r = m log2 e - c, up to half a step of
// c, which makes each of the sum's terms 2^r times what it should be: at |m| < 2^30
// (so that masks of -1e9 are among them) at most 2^64, put right where sums of
// different m meet.  Beyond it r may pass the exponents that a float has; there
// c = 0 and the difference x - m is formed first.
struct Offset {
  float c, r;
  __device__ __forceinline__ explicit Offset(float m) {
    const bool near = fabsf(m) < kNear;
    c = near ? __fmul_rn(m, kLog2e) : 0.f;
    r = near ? __fmaf_rn(m, kLog2e, -c) : 0.f;
  }
};

// How a beam takes part: read its logits, or only its end token (finished), or
// not at all (its score is -inf or not a number).
enum : int { kLive = 0, kDone = 1, kDead = 2 };
__device__ __forceinline__ int beam_kind(const BeamArgs& a, int64_t row) {
  const float s = a.scores[row];
  if (!(fabsf(s) <= FLT_MAX)) return kDead;
  return a.finished != nullptr && a.finished[row] != 0 ? kDone : kLive;
}

// The least of the g largest-of-group values (see above): `mine` is a thread's
// largest key (0: none), g a power of two, 1 .. 64, a thread's group its
// index modulo g.  All threads; a barrier inside.
__device__ __forceinline__ u64 least_of_groups(u64 mine, int g, u64 (*best)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  best[warp][lane] = mine;
  __syncthreads();
  u64 even = 0, odd = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w += 2) {
    const u64 x = best[w][lane], y = best[w + 1][lane];
    even = x > even ? x : even;
    odd = y > odd ? y : odd;
  }
  u64 v = g == 64 ? (even < odd ? even : odd) : (even > odd ? even : odd);
  for (int o = 16; o > 0; o >>= 1) {
    const u64 x = __shfl_xor_sync(0xffffffffu, v, o);
    v = (o >= g) == (x > v) ? x : v;  // the larger within a group, the lesser of groups
  }
  return v;
}

// For every c in [0, n): use(c, r), once, r the number of keys above key c; TIE:
// of equal keys the one with the lower tie value is above.  All threads,
// several to a c where there are enough; keys and ties 16-byte aligned, n
// rounded up to even of them there (a key behind the last, 0).
template <bool TIE, typename Use>
__device__ __forceinline__ void rank_by_count(const u64* keys, const u64* ties, int n, Use use) {
  const int fit = n > 0 ? kThreads / n : 32;
  const int shift = fit >= 32 ? 5 : fit >= 2 ? 31 - __clz(fit) : 0, team = 1 << shift;
  const int me = threadIdx.x & (team - 1), pairs = (n + 1) >> 1;
  const ulonglong2* two = reinterpret_cast<const ulonglong2*>(keys);
  [[maybe_unused]] const ulonglong2* tie = reinterpret_cast<const ulonglong2*>(ties);
  for (int c = threadIdx.x >> shift; c < ((n + kThreads - 1) & ~(kThreads - 1));
       c += shift > 0 ? 2 * kThreads : kThreads) {  // (teams of several: once is enough)
    int r = 0;
    const u64 k = c < n ? keys[c] : ~0ull;
    [[maybe_unused]] const u64 f = TIE && c < n ? ties[c] : 0;
#pragma unroll 4
    for (int d = me; d < pairs; d += team) {
      const ulonglong2 q = two[d];
      bool x = q.x > k, y = q.y > k;
      if constexpr (TIE) {
        const ulonglong2 e = tie[d];
        x |= (q.x == k) & (e.x < f);
        y |= (q.y == k) & (e.y < f);
      }
      r += (x ? 1 : 0) + (y ? 1 : 0);
    }
    for (int o = team >> 1; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if (c < n && me == 0) use(c, r);
  }
}

// A whole warp: room for `count` items of each lane behind *counter; the first
// of this lane's places.
__device__ __forceinline__ int places(int count, int* counter) {
  const int lane = threadIdx.x & 31;
  int upto = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  int base = 0;
  if (lane == 31 && upto > 0) base = atomicAdd(counter, upto);
  return __shfl_sync(0xffffffffu, base, 31) + upto - count;
}

// Shared memory of a CTA besides the merge's lists.
struct __align__(16) BeamShared {
  u64 best[kWarps][32];
  u64 cand[kCap + 2];
  u64 win_key[kThreads + 2];
  u64 red_k[kWarps], lim;
  int multi[kThreads];
  float red_m[kWarps], red_s[kWarps];
  int n_cand, n_win, n_multi;
  // the merge
  double score[kMaxBeams], log_sum[kMaxBeams];  // score -inf: no finite candidate
  float top[kMaxBeams];
  int n_inf[kMaxBeams];  // +inf logits of a row (at most M counted)
  unsigned char done[kMaxBeams];
};

// One segment of a row: its best M keys, largest first (0: none), put(r, key),
// and its maximum and sum of exp(x - maximum), sums(m, s).  All threads.
template <typename T, typename Put, typename Sums>
__device__ __forceinline__ void scan_segment(const BeamArgs& a, BeamShared& sh, int64_t row,
                                             int seg, Put put, Sums sums) {
  constexpr int E = Vec<T>::n;
  constexpr int U = 4;  // vectors of a thread in flight
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int M = a.M;
  const int64_t e0 = (int64_t)seg * a.seg_len;
  const int64_t e1 = e0 + a.seg_len < a.V ? e0 + a.seg_len : (int64_t)a.V;
  const Row<T> x(static_cast<const T*>(a.logits) + row * a.ld, a.V);
  const int n_vec = e1 > e0 ? (int)((e1 - e0 + E - 1) / E) : 0;
  typename Row<T>::Raw next[U];  // the batch after the one at hand
  auto fetch = [&](int v0) {
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int v = v0 + q * kThreads;
      next[q] = v < n_vec ? x.load(e0 + (int64_t)v * E) : x.none();
    }
  };
  fetch(tid);  // (before the beam's state is known: its loads take as long)
  const int kind = beam_kind(a, row);
  if (kind != kLive) {
    // every token -inf, in index order, but a finished beam's end token 0
    const int64_t end = a.end_token;
    const bool has_end = kind == kDone && end >= e0 && end < e1;
    for (int r = tid; r < M; r += kThreads) {
      u64 k = 0;
      if (has_end && r == 0) {
        k = key_of(0.f, (uint32_t)end);
      } else {
        int64_t v = e0 + r - (has_end ? 1 : 0);
        if (has_end && v >= end) ++v;
        if (v < e1) k = key_of(-INFINITY, (uint32_t)v);
      }
      put(r, k);
    }
    if (tid == 0) sums(0.f, 1.f);
    return;
  }

  if (tid == 0) sh.n_cand = sh.n_win = sh.n_multi = 0;
  // One pass: the sum s of exp(x - m), the thread's best vector (its largest
  // value, the first vector that has it) and the largest value of its other
  // vectors.  m need not be the maximum: it is the first batch's and moves
  // only when exp(x - m) would grow past e^20, so that most batches cost no
  // rescaling (and 2^31 terms of 2^(64 + 20 log2 e) stay below 2^127).  m beyond
  // 2^30 (Offset) and batches with NaN take the long way; a batch of nothing but
  // -inf adds nothing to any sum.
  float m = -FLT_MAX, c = 0.f, s = 0.f, best = -INFINITY, other = -INFINITY;
  uint32_t best_v = (uint32_t)tid;
  for (int v0 = tid; v0 < n_vec; v0 += U * kThreads) {
    uint4 r[U];
    float peak = -INFINITY;
#pragma unroll
    for (int q = 0; q < U; ++q) r[q] = x.get(next[q]);
    if (v0 + U * kThreads < n_vec) fetch(v0 + U * kThreads);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const float top = tame(Vec<T>::top(r[q]));
      other = fmaxf(other, fminf(top, best));
      if (top > best) {
        best = top;
        best_v = (uint32_t)(v0 + q * kThreads);
      }
      peak = fmaxf(peak, top);
    }
    if (peak > m + 20.f) {  // (-FLT_MAX + 20 is -FLT_MAX; what was summed vanishes, if any was)
      const Offset old(m), now(peak);
      s *= sm100::ex2_approx(__fmaf_rn(__fadd_rn(m, -peak), kLog2e, now.r - old.r));
      m = peak;
      c = now.c;
    }
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      float f[E], part = 0.f;
      Vec<T>::get(r[q], f);
#pragma unroll
      for (int j = 0; j < E; ++j) part += sm100::ex2_approx(__fmaf_rn(f[j], kLog2e, -c));
      sum += part;
    }
    if (!(sum <= FLT_MAX) || !(fabsf(m) < kNear)) {
      const float r_m = Offset(m).r;
      const int end = peak > -INFINITY ? min(n_vec, v0 + U * kThreads) : 0;
      sum = 0.f;
#pragma unroll 1
      for (int v = v0; v < end; v += kThreads) {
        float f[E];
        Vec<T>::get(x.get(x.load(e0 + (int64_t)v * E)), f);
#pragma unroll
        for (int j = 0; j < E; ++j)
          sum += sm100::ex2_approx(__fmaf_rn(gap(tame(f[j]), m), kLog2e, r_m));
      }
    }
    s += sum;
  }
  s *= exp2f(-Offset(m).r);
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  const float ws = warp_sum(s * sm100::ex2_approx(__fmul_rn(gap(m, wm), kLog2e)));
  if (lane == 0) {
    sh.red_m[warp] = wm;
    sh.red_s[warp] = ws;
  }
  // (a thread's key here: its best value, then its vector)
  const u64 mine = tid < n_vec ? key_of(best, best_v) : 0;
  int g = 1;
  while (g < M) g *= 2;
  u64 lim = least_of_groups(mine, g, sh.best);  // (0: fewer vectors than groups)
  // Above 64 threads at the limit it is raised to the M-th best of their best:
  // the counting pays for what need not be read again and ranked.
  if (__syncthreads_count(mine >= lim && mine != 0) > 64) {
    const int at = places(mine >= lim && mine != 0, &sh.n_win);
    if (mine >= lim && mine != 0) sh.win_key[at] = mine;
    __syncthreads();
    if (tid == 0) sh.win_key[sh.n_win] = 0;
    __syncthreads();
    rank_by_count<false>(sh.win_key, nullptr, sh.n_win, [&](int i, int r) {
      if (r == M - 1) sh.lim = sh.win_key[i];
    });
    __syncthreads();
    lim = sh.lim;
  }
  // What is at or above the limit lies with the threads whose best is: in their
  // best vector, which each reads again (from the caches), or anywhere in theirs
  // if another vector reaches the limit too; those are shared out over all
  // threads.
  const float lim_x = lim == 0 ? -INFINITY : unordered((uint32_t)(lim >> 32));
  const uint32_t lim_v = ~(uint32_t)lim;
  const bool wins = mine >= lim && mine != 0, many = wins && other >= lim_x;
  {
    const int at = places(many, &sh.n_multi);
    if (many) sh.multi[at] = tid;
  }
  __syncthreads();
  const int per = (n_vec + kThreads - 1) / kThreads, n_multi = sh.n_multi;
  constexpr int R = 3;  // vectors of a thread at a time; at first its own and two shared ones
  for (int i0 = (tid & ~31) - kThreads; i0 < n_multi * per; i0 += R * kThreads) {
    int v[R];
    typename Row<T>::Raw w[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int i = i0 + lane + q * kThreads;
      v[q] = -1;
      if (i < 0) {
        if (wins && !many) v[q] = (int)best_v;
      } else if (i < n_multi * per) {
        v[q] = sh.multi[i / per] + (i % per) * kThreads;
        if (v[q] >= n_vec) v[q] = -1;
      }
      if (v[q] >= 0) w[q] = x.load(e0 + (int64_t)v[q] * E);
    }
    uint32_t hits = 0;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (v[q] < 0) continue;
      float f[E];
      Vec<T>::get(x.get(w[q]), f);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float z = tame(f[j]);
        if ((z > lim_x || (z == lim_x && (uint32_t)v[q] <= lim_v)) &&
            (int64_t)v[q] * E + j < e1 - e0)
          hits |= 1u << (q * E + j);
      }
    }
    if (!__any_sync(0xffffffffu, hits != 0)) continue;
    int k = places(__popc(hits), &sh.n_cand);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if ((hits >> (q * E) & ((1u << E) - 1u)) == 0) continue;
      float f[E];
      Vec<T>::get(x.get(w[q]), f);
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (hits >> (q * E + j) & 1) {
          if (k < kCap) sh.cand[k] = key_of(tame(f[j]), (uint32_t)(e0 + (int64_t)v[q] * E + j));
          ++k;
        }
    }
  }
  if (tid == kThreads - 1) {  // (the last to have a rank to count)
    float bm = sh.red_m[0];
    for (int w = 1; w < kWarps; ++w) bm = fmaxf(bm, sh.red_m[w]);
    float bs = 0.f;
    for (int w = 0; w < kWarps; ++w)
      bs += sh.red_s[w] * sm100::ex2_approx(__fmul_rn(gap(sh.red_m[w], bm), kLog2e));
    sums(bm, bs);
  }
  __syncthreads();
  const int n = sh.n_cand;
  if (n <= kCap) {
    if (tid == 0) sh.cand[n] = 0;
    __syncthreads();
    rank_by_count<false>(sh.cand, nullptr, n, [&](int i, int r) {
      if (r < M) put(r, sh.cand[i]);
    });
    for (int r = n + tid; r < M; r += kThreads) put(r, (u64)0);
    return;
  }
  // More than kCap: a few threads hold a great many of the largest elements
  // (values that recur every kThreads * E elements).  The best M one by one,
  // each the largest key below the one before.
  u64 last = ~0ull;
  for (int r = 0; r < M; ++r) {
    u64 k = 0;
    for (int v = tid; v < n_vec; v += kThreads) {
      const int64_t at = e0 + (int64_t)v * E;
      float f[E];
      Vec<T>::get(x.get(x.load(at)), f);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const u64 q = key_of(tame(f[j]), (uint32_t)(at + j));
        if (at + j < e1 && q < last && q > k) k = q;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const u64 q = __shfl_xor_sync(0xffffffffu, k, o);
      k = q > k ? q : k;
    }
    if (lane == 0) sh.red_k[warp] = k;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) k = sh.red_k[w] > k ? sh.red_k[w] : k;
    __syncthreads();
    if (tid == 0) put(r, k);
    last = k;
  }
}

// Of a row with +inf logits these share the score, and all other tokens score -inf
// and go by index, not by logit: its lists are made anew, of M infinite tokens
// (as 0 above a top of 0), or all and the lowest others.  keys: [M][K S].  All
// threads.  (Apart from the kernel, whose common path it would lengthen.)
__device__ __noinline__ void infinite_rows(u64* keys, BeamShared& sh, int K, int M, int S, int V) {
  const int tid = threadIdx.x;
  for (int k = 0; k < K; ++k) {
    const int n_inf = sh.n_inf[k];
    if (n_inf == 0) continue;
    auto slot = [&](int i) { return i / S * (K * S) + k * S + i % S; };
    if (tid == 0) sh.n_multi = 0;
    __syncthreads();
    for (int i = tid; i < S * M; i += kThreads) {
      const u64 key = keys[slot(i)];
      const bool one = (uint32_t)(key >> 32) == ordered(INFINITY);
      if (one && n_inf < M) sh.multi[atomicAdd(&sh.n_multi, 1)] = (int)~(uint32_t)key;
      keys[slot(i)] = one && n_inf == M ? key_of(0.f, ~(uint32_t)key) : 0;
    }
    __syncthreads();
    if (n_inf < M && tid < M) {
      if (tid < n_inf) keys[slot(tid)] = key_of(0.f, (uint32_t)sh.multi[tid]);
      int below = 0;  // (the lowest M tokens hold enough others)
      bool one = false;
      for (int i = 0; i < n_inf; ++i) {
        below += sh.multi[i] < tid;
        one |= sh.multi[i] == tid;
      }
      const int i = n_inf + tid - below;
      if (!one && i < M && tid < V) keys[slot(i)] = key_of(-INFINITY, (uint32_t)tid);
    }
    __syncthreads();
  }
}

// Order-preserving map of a double (NaN as -inf, -0 as +0) to an unsigned.
__device__ __forceinline__ u64 ordered64(double x) {
  if (x != x) x = -INFINITY;
  const u64 u = (u64)__double_as_longlong(x + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered64(u64 o) {
  return __longlong_as_double((long long)(o ^ ((o >> 63) ? 1ull << 63 : ~0ull)));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) beam_select_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char beam_smem[];
  __shared__ BeamShared sh;
  const int tid = threadIdx.x;
  const int n_cta = (int)gridDim.x, rank = (int)blockIdx.x;  // one cluster along x
  const int64_t g = blockIdx.y;
  const int K = a.K, M = a.M, S = a.n_seg, lists = K * S, N = lists * M;
  // (used in the first CTA) keys [M][lists]: list u = k S + segment; then the
  // merge's candidates; then the segments' sums
  u64* keys = reinterpret_cast<u64*>(beam_smem);
  const int Np = (N + 3) & ~1;  // (room for a key behind the last, 16-byte steps)
  u64* cand_o = keys + Np;
  u64* cand_t = cand_o + Np;
  float2* sums = reinterpret_cast<float2*>(cand_t + Np);
  const uint32_t keys0 = sm100::mapa_shared(sm100::smem_u32(keys), 0);
  const uint32_t sums0 = sm100::mapa_shared(sm100::smem_u32(sums), 0);
  float my_score = 0.f;  // (the first CTA's thread k: beam k's, loaded ahead)
  int my_kind = kDead;
  if (rank == 0 && tid < K) {
    my_score = a.scores[g * K + tid];
    my_kind = beam_kind(a, g * K + tid);
    sh.done[tid] = a.finished != nullptr && a.finished[g * K + tid] != 0;
  }
  if (n_cta > 1) sm100::cluster_sync();  // the first CTA runs before any writes into it

  for (int u = rank; u < lists; u += n_cta) {
    scan_segment<T>(
        a, sh, g * K + u / S, u % S,
        [&](int r, u64 key) {
          asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(keys0 + 8u * (r * lists + u)),
                       "l"(key)
                       : "memory");
        },
        [&](float m, float s) {
          asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(sums0 + 8u * u), "f"(m),
                       "f"(s)
                       : "memory");
        });
    __syncthreads();  // before the next segment uses the shared memory again
  }
  if (n_cta > 1) sm100::cluster_sync();
  if (rank != 0) return;

  // The rows: c = score + ((x - top) - log_sum), the difference of the logits
  // first, since x and top may be as large as the type allows.
  bool inf = false;
  if (tid < K) {
    float m = -FLT_MAX;
    for (int i = 0; i < S; ++i) m = fmaxf(m, sums[tid * S + i].x);
    double s = 0.0;
    for (int i = 0; i < S; ++i) {
      const float2 p = sums[tid * S + i];
      s += (double)(p.y * sm100::ex2_approx(__fmul_rn(gap(p.x, m), kLog2e)));
    }
    // (a row of -inf has s = 0: it takes part like a dead beam)
    const bool some = my_kind != kDead && s > 0.0, live = some && my_kind == kLive;
    sh.score[tid] = some ? (double)my_score : -INFINITY;
    sh.log_sum[tid] = live ? log(s) : 0.0;
    inf = live && m == INFINITY;
    sh.top[tid] = live && !inf ? m : 0.f;
    sh.n_inf[tid] = inf ? (s < (double)M ? (int)s : M) : 0;
  }
  if (tid == 0) sh.n_cand = 0;
  if (__syncthreads_or(inf)) infinite_rows(keys, sh, K, M, S, a.V);
  auto candidate = [&](int i) -> u64 {  // (0: none)
    const u64 key = keys[i];
    const int k = (i % lists) / S;
    const float x = unordered((uint32_t)(key >> 32));
    const double d = (double)x - (double)sh.top[k];
    return key == 0 ? 0 : ordered64(sh.score[k] + (d - sh.log_sum[k]));
  };
  // The best M: those at or above the limit, ranked by counting.  (Equal scores
  // may put more there than ranks need, never fewer.)  Of equal scores the lower
  // beam's goes first, within a beam the larger logit's (where a large top or
  // score makes the scores of different logits one number, they keep the order by
  // which the lists were cut), of equal logits the lower token's: in one word, since
  // K V < 2^31 leaves beam and token 32 bits, the beam the upper `of_k`.
  const int of_k = K > 2 ? 32 - __clz(K - 1) : 1, of_v = 32 - of_k;
  // A thread's i-th key lies on a diagonal of the lists, so that a group of threads
  // has keys of all of them: with a list each, the limit would be the best of the
  // worst beam, and all keys above it to be ranked.
  auto place = [&](int i) {
    const int r = i / lists, u = i % lists - r % lists;
    return r * lists + (u < 0 ? u + lists : u);
  };
  u64 mine = 0;
  for (int i = tid; i < N; i += kThreads) {
    const u64 o = candidate(place(i));
    mine = o > mine ? o : mine;
  }
  int groups = 1;
  while (groups < M) groups *= 2;
  const u64 lim = least_of_groups(mine, groups, sh.best);
  for (int i0 = tid & ~31; i0 < N; i0 += kThreads) {
    const int at = i0 + (tid & 31), i = place(at);
    const u64 o = mine >= lim && at < N ? candidate(i) : 0;
    const bool in = o != 0 && o >= lim;
    if (!__any_sync(0xffffffffu, in)) continue;
    const int c = places(in, &sh.n_cand);
    if (in) {
      cand_o[c] = o;
      const u64 x = ~keys[i];  // logit, token; the lower first
      cand_t[c] = (u64)(i % lists / S) << (32 + of_v) | x >> 32 << of_v | (uint32_t)x;
    }
  }
  __syncthreads();
  const int n = sh.n_cand;
  if (tid == 0) cand_o[n] = 0;
  __syncthreads();
  rank_by_count<true>(cand_o, cand_t, n, [&](int c, int r) {
    if (r >= M) return;
    const u64 o = cand_o[c], t = cand_t[c];
    const int k = (int)(t >> (32 + of_v)), token = (int)((uint32_t)t << of_k >> of_k);
    const int64_t at = g * M + r;
    a.out_scores[at] = (float)unordered64(o);
    a.out_parents[at] = k;
    a.out_tokens[at] = token;
    if (a.out_finished != nullptr) a.out_finished[at] = sh.done[k] || token == a.end_token;
  });
}

// In-place reordering.  A thread owns one W-wide column of a group's K rows of
// one tensor: it loads what each row shall hold, then stores it.  No other
// thread touches the column, so no second copy of the state is needed; rows
// that keep their place are neither read nor written.  Bound by memory: 32
// groups of 8 beams, 7 rows of each written from 4 others or themselves (1.19 GB
// read and written) 191 us, 6.26 TB/s of the copy's 6.54; 2 groups of 4 (34 MB)
// 6.4 us.
template <typename W, int KMAX>
__device__ __forceinline__ void reorder_column(char* base, int64_t row_bytes, int64_t col, int K,
                                               const int* from) {
  W v[KMAX];
  W* p = reinterpret_cast<W*>(base) + col;
  const int64_t step = row_bytes / (int64_t)sizeof(W);
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (j < K && from[j] != j) v[j] = p[from[j] * step];
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (j < K && from[j] != j) p[j * step] = v[j];
}

template <int KMAX>
__global__ void __launch_bounds__(kThreads) state_reorder_kernel(const ReorderArgs a) {
  __shared__ int from[KMAX];
  int t = 0;
  while (t + 1 < a.n_states && (int64_t)blockIdx.x >= a.first_block[t + 1]) ++t;
  const int64_t b = (int64_t)blockIdx.x - a.first_block[t];
  const int64_t g = b / a.blocks_per_group[t];
  const int64_t col = (b % a.blocks_per_group[t]) * kThreads + threadIdx.x;
  if (threadIdx.x < (unsigned)a.K) {
    const int p = a.parents[g * a.K + threadIdx.x];
    const bool ok = p >= 0 && p < a.K;
    if (!ok) atomicOr(a.err, kErrBadIndex);
    from[threadIdx.x] = ok ? p : (int)threadIdx.x;  // a bad parent: the row stays
  }
  __syncthreads();
  const int64_t rb = a.row_bytes[t];
  char* base = static_cast<char*>(a.states[t]) + g * a.K * rb;
  const int w = a.width[t];
  if (col * w >= rb) return;
  if (w == 16) reorder_column<uint4, KMAX>(base, rb, col, a.K, from);
  else if (w == 4) reorder_column<uint32_t, KMAX>(base, rb, col, a.K, from);
  else reorder_column<unsigned char, KMAX>(base, rb, col, a.K, from);
}

}  // namespace

// Clusters of 2^i CTAs that the device holds at once, per type (asked once per
// device; the answers are the same whoever asks, so threads may race).
constexpr int kMaxDevices = 64, kLogMaxCluster = 4;
std::atomic<int> g_fit[kMaxDevices][2][kLogMaxCluster + 1];

gdn_status launch_beam_select(BeamArgs a, cudaStream_t stream) {
  const bool bf16 = a.dtype == GDN_BF16;
  void (*kernel)(BeamArgs) =
      bf16 ? beam_select_kernel<__nv_bfloat16> : beam_select_kernel<float>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GDN_ERR_CUDA;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;

  // The group's cluster: the largest power of two at which all groups are on the
  // device at once, none of its CTAs with less than a vector a thread; at
  // most 16 (more than the portable 8 by leave of cudaFuncSetAttribute).
  // Measured on a B200 (K = 8, V = 130000, M = 16, bf16, in one run): 32 groups in
  // clusters of 16 (two waves) 37.9 us, of 8 29.4, of 4 45.2; 16 groups in
  // clusters of 16 24.1, of 8 24.7.
  const int64_t step = (int64_t)kThreads * (bf16 ? 8 : 4);
  const int64_t vectors = a.K * ((a.V + step - 1) / step);
  int cluster = 1;
  for (int i = kLogMaxCluster; i > 0; --i) {
    std::atomic<int>& slot = g_fit[dev][bf16 ? 0 : 1][i];
    int fit = slot.load(std::memory_order_relaxed);
    if (fit == 0) {
      attr.val.clusterDim.x = 1u << i;
      cfg.gridDim = dim3(1u << i);
      cfg.dynamicSmemBytes = 16384;
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kBeamMergeKeys * 32 + 72) != cudaSuccess ||
          cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
              cudaSuccess)
        return GDN_ERR_CUDA;
      if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess || fit < 1) {
        cudaGetLastError();  // (a size that the device cannot hold)
        fit = -1;
      }
      slot.store(fit, std::memory_order_relaxed);
    }
    if (fit >= a.n_groups && (1 << i) < 2 * vectors) {
      cluster = 1 << i;
      break;
    }
  }
  // Segments of a row: the least time of the busiest CTA, whose every list
  // costs its elements and about as much as 8192 more for the choice among them.
  const int hold = kBeamMergeKeys / (a.K * a.M);
  int segs = 1;
  double least = 0.0;
  for (int s = 1; s <= cluster && s <= hold; ++s) {
    const double cost = ((a.K * s + cluster - 1) / cluster) * ((double)a.V / s + 8192.0);
    if (s == 1 || cost < least) {
      least = cost;
      segs = s;
    }
  }
  a.seg_len = (((int64_t)a.V + segs - 1) / segs + step - 1) / step * step;
  a.n_seg = (int)((a.V + a.seg_len - 1) / a.seg_len);
  const int lists = a.K * a.n_seg;
  attr.val.clusterDim.x = (unsigned)cluster;
  cfg.gridDim = dim3((unsigned)cluster, (unsigned)a.n_groups);
  cfg.dynamicSmemBytes = ((size_t)lists * a.M + 3) * 24 + (size_t)lists * sizeof(float2);
  return launch_status(cudaLaunchKernelEx(&cfg, kernel, a));
}

gdn_status launch_state_reorder(ReorderArgs a, cudaStream_t stream) {
  int64_t blocks = 0;
  for (int t = 0; t < a.n_states; ++t) {
    const int64_t rb = a.row_bytes[t];
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.states[t]) | (uintptr_t)rb;
    a.width[t] = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : 1;
    const int64_t cols = rb / a.width[t];
    a.first_block[t] = blocks;
    a.blocks_per_group[t] = (cols + kThreads - 1) / kThreads;
    blocks += a.blocks_per_group[t] * a.n_groups;
    if (blocks > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  }
  if (blocks == 0) return GDN_OK;
  void (*kernel)(ReorderArgs) = a.K <= 4    ? state_reorder_kernel<4>
                                : a.K <= 8  ? state_reorder_kernel<8>
                                : a.K <= 16 ? state_reorder_kernel<16>
                                            : state_reorder_kernel<32>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  return launch_status(cudaLaunchKernelEx(&cfg, kernel, a));
}

}  // namespace gdn
