// Beam search over a batch of groups of K beams: choosing the M best
// continuations of each group (gdn_beam_select), and moving the surviving
// beams' recurrent states into place (gdn_state_reorder).
//
// Selection.  A candidate is (beam k, token v) with the score
//   c = score_k + logit_kv - log sum_v' exp(logit_kv').
// Within a beam the order by c is the order by logit, so each row's best M are
// found from the logits alone while its sum is still being formed, and the
// logits are read once.  Two kernels:
//   1. beam_scan_kernel, a CTA per segment of a row: the segment's maximum and
//      sum of exponentials, and its best M as 64-bit keys (ordered value, then
//      the complement of the index: keys are distinct, and the lower index
//      wins a tie), largest first;
//   2. beam_merge_kernel, a CTA per group: the rows' log sums, then one warp
//      merges the K x segments lists by score (64-bit floating point, ties to
//      the lowest k V + v).
// Work is cut by element index, never by address, so rows with equal logits
// get equal sums bit for bit, wherever they lie.
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
// What a logit counts as: NaN as -inf (never chosen before a number), +inf as
// the largest finite value (so that equal shares go to the infinite entries).
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

// 16 bytes of a row as floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ void get(const uint4& r, float* f) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ void get(const uint4& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// One row, read as vectors of 16 bytes by element index whatever its address:
// a row that does not begin on 16 bytes is read as aligned pairs and shifted
// together.  Nothing outside the row is touched: vectors whose aligned pair
// would reach over either end are gathered element by element.
template <typename T>
struct Row {
  const T* p;
  int64_t V;
  uint32_t shift;  // bytes from the aligned address below

  __device__ __forceinline__ Row(const T* row, int64_t v)
      : p(row), V(v), shift((uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u)) {}

  __device__ __forceinline__ uint4 load(int64_t i) const {  // elements i .. i + Vec::n - 1
    constexpr int E = Vec<T>::n;
    if (shift == 0) {
      if (i + E <= V) return __ldg(reinterpret_cast<const uint4*>(p + i));
    } else if (i > 0 && i + 2 * E <= V) {
      const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p + i) - shift);
      const uint4 a = __ldg(q), b = __ldg(q + 1);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const uint32_t bits = (shift & 3u) * 8u, word = shift >> 2;
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // (word is uniform over the CTA: selects, no indexed registers)
        const uint32_t lo = word == 0 ? w[k] : word == 1 ? w[k + 1] : word == 2 ? w[k + 2] : w[k + 3];
        const uint32_t hi =
            word == 0 ? w[k + 1] : word == 1 ? w[k + 2] : word == 2 ? w[k + 3] : w[(k + 4) & 7];
        o[k] = __funnelshift_r(lo, hi, bits);
      }
      return make_uint4(o[0], o[1], o[2], o[3]);
    }
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (E == 4) {
        o[k] = i + k < V ? reinterpret_cast<const uint32_t*>(p)[i + k] : Vec<T>::kNegInf;
      } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
        const uint32_t lo = i + 2 * k < V ? h[i + 2 * k] : 0xff80u;
        const uint32_t hi = i + 2 * k + 1 < V ? h[i + 2 * k + 1] : 0xff80u;
        o[k] = lo | hi << 16;
      }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

__device__ __forceinline__ u64 shfl_u64(u64 v, int src) {
  return __shfl_sync(0xffffffffu, v, src);
}

// How a beam takes part: read its logits, or only its end token (finished), or
// not at all (its score is -inf or not a number).
enum : int { kLive = 0, kDone = 1, kDead = 2 };
__device__ __forceinline__ int beam_kind(const BeamArgs& a, int64_t row) {
  const float s = a.scores[row];
  if (!(fabsf(s) <= FLT_MAX)) return kDead;
  return a.finished != nullptr && a.finished[row] != 0 ? kDone : kLive;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(const BeamArgs a) {
  constexpr int E = Vec<T>::n;
  constexpr int U = 4;  // vectors of a thread in flight
  __shared__ u64 sorted[kWarps][32];
  __shared__ u64 cand[kCap];
  __shared__ float red_m[kWarps], red_s[kWarps];
  __shared__ u64 red_k[kWarps];
  __shared__ int winner[kMaxBeamCandidates];
  __shared__ u64 tau;
  __shared__ int n_cand;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / a.n_seg;
  const int seg = (int)(blockIdx.x % a.n_seg);
  const int M = a.M;
  const int64_t e0 = (int64_t)seg * a.seg_len;
  const int64_t e1 = e0 + a.seg_len < a.V ? e0 + a.seg_len : (int64_t)a.V;
  u64* out = a.keys + ((int64_t)row * a.n_seg + seg) * M;
  float2* out_sum = a.sums + (int64_t)row * a.n_seg + seg;
  sm100::launch_dependents();

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
      out[r] = k;
    }
    if (tid == 0) *out_sum = make_float2(0.f, 1.f);
    return;
  }

  const Row<T> x(static_cast<const T*>(a.logits) + row * a.ld, a.V);
  const int n_vec = (int)((e1 - e0 + E - 1) / E);
  if (tid == 0) {
    tau = 1;  // every key
    n_cand = 0;
  }
  // One pass: running maximum m and sum s of exp(x - m); the thread's best
  // element.  m starts at the lowest finite value, not -inf, so that m - m is
  // a number in rows of -inf.
  float m = -FLT_MAX, s = 0.f, best = -INFINITY;
  uint32_t best_at = (uint32_t)(e0 + (int64_t)tid * E);
  for (int v0 = tid; v0 < n_vec; v0 += U * kThreads) {
    uint4 r[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int v = v0 + q * kThreads;
      r[q] = v < n_vec ? x.load(e0 + (int64_t)v * E)
                       : make_uint4(Vec<T>::kNegInf, Vec<T>::kNegInf, Vec<T>::kNegInf,
                                    Vec<T>::kNegInf);
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      float f[E];
      Vec<T>::get(r[q], f);
      float top = f[0];
#pragma unroll
      for (int j = 1; j < E; ++j) top = fmaxf(top, f[j]);
      if (top > best) {
        top = tame(top);
        int at = 0;
#pragma unroll
        for (int j = E - 1; j >= 0; --j)
          if (tame(f[j]) == top) at = j;
        if (top > best) {
          best = top;
          best_at = (uint32_t)(e0 + (int64_t)(v0 + q * kThreads) * E + at);
        }
        if (top > m) {
          s *= sm100::ex2_approx(__fmul_rn(__fadd_rn(m, -top), kLog2e));
          m = top;
        }
      }
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j)
        sum += sm100::ex2_approx(__fmul_rn(__fadd_rn(f[j], -m), kLog2e));
      if (!(sum <= FLT_MAX)) {  // a NaN or +inf among them
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j)
          sum += sm100::ex2_approx(__fmul_rn(__fadd_rn(tame(f[j]), -m), kLog2e));
      }
      s += sum;
    }
  }
  // the segment's maximum and sum
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  const float ws = warp_sum(s * sm100::ex2_approx(__fmul_rn(__fadd_rn(m, -wm), kLog2e)));
  if (lane == 0) {
    red_m[warp] = wm;
    red_s[warp] = ws;
  }
  // The threads' best elements, ranked: the warp sorts its 32 keys, then each
  // key's rank is its place here plus the larger keys of the other warps.
  const u64 mine = tid < n_vec ? key_of(best, best_at) : 0;
  int place = 0;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    const u64 k = shfl_u64(mine, i);
    place += (k > mine || (k == mine && i < lane)) ? 1 : 0;
  }
  sorted[warp][place] = mine;
  __syncthreads();
  if (tid == 0) {
    float bm = red_m[0];
    for (int w = 1; w < kWarps; ++w) bm = fmaxf(bm, red_m[w]);
    float bs = 0.f;
    for (int w = 0; w < kWarps; ++w)
      bs += red_s[w] * sm100::ex2_approx(__fmul_rn(__fadd_rn(red_m[w], -bm), kLog2e));
    *out_sum = make_float2(bm, bs);
  }
  const int n_own = n_vec < kThreads ? n_vec : kThreads;  // threads with elements
  const int n_win = n_own < M ? n_own : M;
  if (place < M && mine != 0) {
    int rank = place;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) continue;
      int lo = 0, hi = 32;  // keys larger than mine in sorted[w]
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sorted[w][mid] > mine) lo = mid + 1; else hi = mid;
      }
      rank += lo;
    }
    if (rank < M) {
      winner[rank] = tid;
      if (rank == M - 1) tau = mine;
    }
  }
  __syncthreads();
  // The segment's best M are >= tau, the M-th best of the threads' best
  // elements, and lie with the threads whose best is >= tau.  Those threads'
  // vectors (from the caches) give the candidates: M and a few more.
  const u64 lim = tau;
  const float lim_x = lim == 1 ? -INFINITY : unordered((uint32_t)(lim >> 32));
  const int per = (n_vec + kThreads - 1) / kThreads;
  for (int i = tid; i < n_win * per; i += kThreads) {
    const int v = winner[i % n_win] + (i / n_win) * kThreads;
    if (v >= n_vec) continue;
    const int64_t at = e0 + (int64_t)v * E;
    float f[E];
    Vec<T>::get(x.load(at), f);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float z = tame(f[j]);
      if (z >= lim_x && at + j < e1) {
        const u64 k = key_of(z, (uint32_t)(at + j));
        if (k >= lim) {
          const int c = atomicAdd(&n_cand, 1);
          if (c < kCap) cand[c] = k;
        }
      }
    }
  }
  __syncthreads();
  const int n = n_cand;
  if (n <= kCap) {
    for (int c = tid; c < n; c += kThreads) {
      const u64 k = cand[c];
      int rank = 0;
      for (int d = 0; d < n; ++d) rank += cand[d] > k ? 1 : 0;
      if (rank < M) out[rank] = k;
    }
    for (int r = n + tid; r < M; r += kThreads) out[r] = 0;
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
      Vec<T>::get(x.load(at), f);
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
    if (lane == 0) red_k[warp] = k;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) k = red_k[w] > k ? red_k[w] : k;
    __syncthreads();
    if (tid == 0) out[r] = k;
    last = k;
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

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  // c = score + ((x - top) - log_sum), the difference of the logits first: x and
  // top may be as large as the type allows
  __shared__ double score[kMaxBeams], log_sum[kMaxBeams];  // score -inf: no finite candidate
  __shared__ float top[kMaxBeams];
  __shared__ unsigned char done[kMaxBeams];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x, K = a.K, M = a.M, S = a.n_seg;
  const int lists = K * S, n_keys = lists * M;
  u64* keys = reinterpret_cast<u64*>(smem);                            // [lists][M]
  unsigned char* used = reinterpret_cast<unsigned char*>(keys + n_keys);  // [lists]
  sm100::dependency_wait();  // the scan's results are in memory

  const u64* src = a.keys + (int64_t)g * n_keys;
  for (int i = tid; i < n_keys; i += kThreads) keys[i] = src[i];
  for (int i = tid; i < lists; i += kThreads) used[i] = 0;
  for (int k = warp; k < K; k += kWarps) {
    const int64_t row = (int64_t)g * K + k;
    float m = -FLT_MAX;
    for (int i = lane; i < S; i += 32) m = fmaxf(m, a.sums[row * S + i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double s = 0.0;
    for (int i = lane; i < S; i += 32) {
      const float2 p = a.sums[row * S + i];
      s += (double)p.y * exp((double)p.x - (double)m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      const int kind = beam_kind(a, row);
      // (a row of -inf has s = 0: it takes part like a dead beam; a finished
      // beam's sums are maximum 0, sum 1)
      const bool some = kind != kDead && s > 0.0;
      score[k] = some ? (double)a.scores[row] : -INFINITY;
      log_sum[k] = some && kind == kLive ? log(s) : 0.0;
      top[k] = some && kind == kLive ? m : 0.f;
      done[k] = a.finished != nullptr && a.finished[row] != 0;
    }
  }
  __syncthreads();
  if (warp != 0) return;

  // One warp: a lane has the lists lane, lane + 32, ...; each round takes the
  // best head of all and moves that list on.
  u64 best = 0;
  uint32_t best_flat = 0xffffffffu;
  int best_list = -1;
  auto pick = [&]() {  // the best head among this lane's lists
    best = 0;
    best_flat = 0xffffffffu;
    best_list = -1;
    for (int l = lane; l < lists; l += 32) {
      const int u = used[l];
      const u64 key = u < M ? keys[l * M + u] : 0;
      if (key == 0) continue;
      const int k = l / S;
      const uint32_t v = ~(uint32_t)key;
      const float x = unordered((uint32_t)(key >> 32));
      const u64 o = ordered64(score[k] + (((double)x - (double)top[k]) - log_sum[k]));
      const uint32_t flat = (uint32_t)k * (uint32_t)a.V + v;
      if (best_list < 0 || o > best || (o == best && flat < best_flat)) {
        best = o;
        best_flat = flat;
        best_list = l;
      }
    }
  };
  pick();
  for (int r = 0; r < M; ++r) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    bool in = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, in ? (uint32_t)best : 0u);
    in = in && (uint32_t)best == lo;
    const uint32_t flat = __reduce_min_sync(0xffffffffu, in ? best_flat : 0xffffffffu);
    if (in && best_flat == flat && best_list >= 0) {
      const int k = best_list / S;
      const int token = (int)(flat - (uint32_t)k * (uint32_t)a.V);
      const int64_t o = (int64_t)g * M + r;
      a.out_scores[o] = (float)unordered64(best);
      a.out_parents[o] = k;
      a.out_tokens[o] = token;
      if (a.out_finished != nullptr) a.out_finished[o] = done[k] || token == a.end_token;
      ++used[best_list];
      pick();
    }
    __syncwarp();
  }
}

// In-place reordering.  A thread owns one W-wide column of a group's K rows of
// one tensor: it loads what each row shall hold, then stores it.  No other
// thread touches the column, so no second copy of the state is needed; rows
// that keep their place are neither read nor written.
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

// How a call is cut: enough segments that the device has several CTAs per SM
// (148 SMs), none shorter than one vector a thread, and no more lists than
// the merge holds in shared memory.
BeamPlan beam_plan(int64_t rows, int32_t K, int32_t V, int32_t M, gdn_dtype dtype) {
  const int64_t step = (int64_t)kThreads * (dtype == GDN_BF16 ? 8 : 4);
  const int64_t target = 4 * 148;
  int64_t n = (target + rows - 1) / rows;
  const int64_t most = (V + step - 1) / step;
  if (n > most) n = most;
  const int64_t hold = kBeamMergeKeys / ((int64_t)K * M);
  if (n > hold) n = hold;
  if (n < 1) n = 1;
  const int64_t len = ((V + n - 1) / n + step - 1) / step * step;
  BeamPlan p;
  p.seg_len = len;
  p.n_seg = (int32_t)((V + len - 1) / len);
  p.sum_bytes = ((size_t)rows * p.n_seg * sizeof(float2) + 255) & ~(size_t)255;
  p.bytes = p.sum_bytes + (((size_t)rows * p.n_seg * M * sizeof(u64) + 255) & ~(size_t)255);
  return p;
}

gdn_status launch_beam_select(BeamArgs a, void* ws, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.n_groups * a.K;
  const BeamPlan p = beam_plan(rows, a.K, a.V, a.M, a.dtype);
  if (rows * p.n_seg > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  a.n_seg = p.n_seg;
  a.seg_len = p.seg_len;
  a.sums = static_cast<float2*>(ws);
  a.keys = reinterpret_cast<u64*>(static_cast<char*>(ws) + p.sum_bytes);
  const unsigned blocks = (unsigned)(rows * p.n_seg);
  if (a.dtype == GDN_BF16)
    beam_scan_kernel<__nv_bfloat16><<<blocks, kThreads, 0, stream>>>(a);
  else
    beam_scan_kernel<float><<<blocks, kThreads, 0, stream>>>(a);
  if (cudaPeekAtLastError() != cudaSuccess) return GDN_ERR_CUDA;
  const size_t smem = (size_t)a.K * p.n_seg * (a.M * sizeof(u64) + 1);
  static std::atomic<bool> attr_set[64];  // per device; setting it twice does no harm
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GDN_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kBeamMergeSmem) != cudaSuccess)
      return GDN_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_relaxed);
  }
  // the merge may be scheduled while the scan still runs; it waits for the
  // scan's end before it reads
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_groups);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_merge_kernel, (const BeamArgs)a) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
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
  if (a.K <= 4)
    state_reorder_kernel<4><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else if (a.K <= 8)
    state_reorder_kernel<8><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else if (a.K <= 16)
    state_reorder_kernel<16><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else
    state_reorder_kernel<32><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
