// Gated linear recurrence: per channel c and token t
//   h_t = a_t h_{t-1} + b_t x_t,   a_t = exp(log_alpha_t),   y_t = h_t,
// with b = 1, a given gate beta, or 1 - a, over a packed batch of sequences;
// its backward; and the one-token step.
//
// The pair (A, h) of a run of tokens (the product of its a, and its h from
// a zero start) composes associatively: run 1 then run 2 gives
// (A1 A2, A2 h1 + h2).  A sequence's first token takes a = 0 and adds
// a_t h_0 to its input, so packed sequences need no other care.
//
// Layout.  A CTA of 8 warps owns a tile of 64 tokens x 32 VEC channels: warp
// w has tokens 8 w .. 8 w + 7, a lane VEC neighbouring channels.  The carry
// along the tokens passes three levels, each in a fixed order (results do not
// depend on timing): 8 tokens in a thread's registers, 8 warps through
// shared memory, and the CTAs of a cluster, which hold consecutive tiles of
// the same channels, through distributed shared memory.  The cluster walks
// the packed tokens in steps of (cluster size) tiles, the carry kept in
// registers; nothing is exchanged through global memory, so there is no
// workspace and no flag to wait on.  Every input is read once and every
// output written once; the next tile's inputs are loaded into registers
// while this one is folded.
#include <atomic>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kTok = kGlrTile / kWarps;  // tokens per thread and tile
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;
static_assert(kTok == 8 && kGlrTile == 64, "one lane per token of a warp's run");

enum : int { kGateNone = GDN_GLR_GATE_NONE, kGateBeta = GDN_GLR_GATE_BETA,
             kGateComp = GDN_GLR_GATE_COMPLEMENT };

// VEC neighbouring channels of one token as they lie in memory.
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) { r = __ldg(p); }
  __device__ __forceinline__ void zero() { r = 0.f; }
  __device__ __forceinline__ void get(float* f) const { f[0] = r; }
  static __device__ __forceinline__ void store(float* p, const float* f) { *p = f[0]; }
};
template <>
struct Raw<float, 2> {
  float2 r;
  __device__ __forceinline__ void load(const float* p) {
    r = __ldg(reinterpret_cast<const float2*>(p));
  }
  __device__ __forceinline__ void zero() { r = make_float2(0.f, 0.f); }
  __device__ __forceinline__ void get(float* f) const { f[0] = r.x; f[1] = r.y; }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  unsigned short r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = __ldg(reinterpret_cast<const unsigned short*>(p));
  }
  __device__ __forceinline__ void zero() { r = 0; }
  __device__ __forceinline__ void get(float* f) const { f[0] = __uint_as_float((uint32_t)r << 16); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    *p = __float2bfloat16_rn(f[0]);
  }
};
template <>
struct Raw<__nv_bfloat16, 2> {
  uint32_t r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
  __device__ __forceinline__ void zero() { r = 0; }
  // (a bf16 is the high half of its fp32 value)
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(r << 16);
    f[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    *reinterpret_cast<uint32_t*>(p) = sm100::pack_bf16(f[0], f[1]);
  }
};

// a = exp(l) and 1 - a.  Channels that remember a thousand tokens have a
// within 1e-3 of 1, where an error of exp in one direction adds up over all of
// them.  So near 0, exp(l) - 1 is summed from its Taylor series (the first
// term left out, l^7/5040, is below 2^-24 of the sum for |l| < 1/4) and a is
// 1 + that, rounded once; further out the hardware 2^x, good to 2^-22,
// serves, since such a channel forgets within a few tokens.
__device__ __forceinline__ void decay(float l, float& a, float& one_minus_a) {
  float p = __fmaf_rn(l, 1.f / 720.f, 1.f / 120.f);
  p = __fmaf_rn(l, p, 1.f / 24.f);
  p = __fmaf_rn(l, p, 1.f / 6.f);
  p = __fmaf_rn(l, p, 0.5f);
  p = __fmaf_rn(l, p, 1.f);
  p = __fmul_rn(l, p);
  const float e = sm100::ex2_approx(__fmul_rn(l, 1.4426950408889634f));
  const bool near = fabsf(l) < 0.25f;
  a = near ? __fadd_rn(1.f, p) : e;
  one_minus_a = near ? -p : __fadd_rn(1.f, -e);
}

// Input gate b of one channel: its factor of x.
template <int GATE>
__device__ __forceinline__ float gate_of(float beta, float one_minus_a) {
  return GATE == kGateNone ? 1.f : GATE == kGateBeta ? beta : one_minus_a;
}

// Last sequence s with cu[s] <= t (so that empty sequences are passed over).
// Any contents of cu give an s in [0, n_seq).
__device__ __forceinline__ int seq_at(const int32_t* cu, int n_seq, int64_t t) {
  int lo = 0, hi = n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Which of a warp's kTok tokens from t0 on begin or end a sequence (bit i:
// token t0 + i); lane i (< kTok) also gets token i's sequence.
struct Marks {
  uint32_t first, last;
  int seq;
};
__device__ __forceinline__ Marks marks_of(const int32_t* cu, int n_seq, int64_t total_T,
                                          int64_t t0, int lane) {
  Marks m;
  m.seq = 0;
  if (cu == nullptr) {
    m.first = t0 == 0 ? 1u : 0u;
    const int64_t d = total_T - 1 - t0;
    m.last = d >= 0 && d < kTok ? 1u << (int)d : 0u;
    return m;
  }
  bool f = false, l = false;
  const int64_t t = t0 + lane;
  if (lane < kTok && t < total_T) {
    m.seq = seq_at(cu, n_seq, t);
    f = __ldg(cu + m.seq) == t;
    l = __ldg(cu + m.seq + 1) == t + 1;
  }
  m.first = __ballot_sync(0xffffffffu, f);
  m.last = __ballot_sync(0xffffffffu, l);
  return m;
}

// One composed run of tokens per channel.
template <int VEC>
struct __align__(8 * VEC) Run {
  float A[VEC], h[VEC];
};

// h behind a run that is entered with h.  A run whose A is 0 forgets what was
// before it, even an infinity or NaN: those belong to another sequence.
__device__ __forceinline__ float through(float A, float run_h, float h) {
  return A == 0.f ? run_h : __fmaf_rn(A, h, run_h);
}

// Rows of a [n_seq, C] state: load / store VEC channels of sequence s.
template <int VEC>
__device__ __forceinline__ void state_get(const float* p, int64_t s, int C, int c, float* f) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = p == nullptr ? 0.f : p[s * C + c + j];
}
template <int VEC>
__device__ __forceinline__ void state_put(float* p, int64_t s, int C, int c, const float* f) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) p[s * C + c + j] = f[j];
}

// Sequences without tokens carry their state through: out[s] = in[s] (or 0).
// Also reports a malformed cu_seqlens.  Rows are shared out over the
// cluster's warps.
template <int VEC>
__device__ __forceinline__ void empty_sequences(const int32_t* cu, int n_seq, int64_t total_T,
                                                const float* in, float* out, int C, int c,
                                                bool c_ok, int first_row, int stride, int* err) {
  for (int s = first_row; s < n_seq; s += stride) {
    int64_t lo = 0, hi = total_T;
    if (cu != nullptr) {
      lo = __ldg(cu + s);
      hi = __ldg(cu + s + 1);
      const bool ok = lo >= 0 && hi >= lo && hi <= total_T && (s != 0 || lo == 0) &&
                      (s != n_seq - 1 || hi == total_T);
      if (!ok) {
        if (err != nullptr && (threadIdx.x & 31) == 0) atomicOr(err, kErrBadSeqlens);
        continue;
      }
    }
    if (lo == hi && out != nullptr && c_ok) {
      float f[VEC];
      state_get<VEC>(in, s, C, c, f);
      state_put<VEC>(out, s, C, c, f);
    }
  }
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <typename Tin, int VEC, int GATE>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_kernel(const GlrArgs p) {
  __shared__ Run<VEC> warp_run[kWarps][32];
  __shared__ Run<VEC> tile_run[2][kMaxCluster][32];
  using R = Raw<Tin, VEC>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_cta = (int)gridDim.x, rank = (int)blockIdx.x;  // one cluster along x
  const int C = p.C;
  const int c = ((int)blockIdx.y * 32 + lane) * VEC;
  const bool c_ok = c < C;
  const int64_t T = p.total_T;
  const int64_t n_tiles = (T + kGlrTile - 1) / kGlrTile;
  const int64_t n_steps = (n_tiles + n_cta - 1) / n_cta;
  const Tin* X = static_cast<const Tin*>(p.x) + c;
  const Tin* L = static_cast<const Tin*>(p.log_alpha) + c;
  const Tin* B = static_cast<const Tin*>(p.beta) + c;
  Tin* Y = static_cast<Tin*>(p.y) + c;

  R rx[kTok], rl[kTok], rb[kTok];
  auto load = [&](int64_t step) {
    const int64_t t0 = (step * n_cta + rank) * kGlrTile + warp * kTok;
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const int64_t t = t0 + i;
      if (c_ok && t < T) {
        rx[i].load(X + t * C);
        rl[i].load(L + t * C);
        if (GATE == kGateBeta) rb[i].load(B + t * C);
      } else {  // a = exp(0) = 1, x = 0: leaves a state as it is
        rx[i].zero();
        rl[i].zero();
        if (GATE == kGateBeta) rb[i].zero();
      }
    }
  };

  float carry[VEC];  // state before this step's first tile
#pragma unroll
  for (int j = 0; j < VEC; ++j) carry[j] = 0.f;
  if (n_steps > 0) {
    load(0);
    sm100::cluster_sync();  // every CTA runs before any writes into another's shared memory
  }

  for (int64_t step = 0; step < n_steps; ++step) {
    const int64_t tile = step * n_cta + rank;
    const int64_t t0 = tile * kGlrTile + warp * kTok;
    const Marks m = marks_of(p.cu_seqlens, p.n_seq, T, t0, lane);
    float a[kTok][VEC], u[kTok][VEC];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      float x[VEC], l[VEC], b[VEC];
      rx[i].get(x);
      rl[i].get(l);
      if (GATE == kGateBeta) rb[i].get(b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float q;
        decay(l[j], a[i][j], q);
        const float g = gate_of<GATE>(b[j], q);
        u[i][j] = GATE == kGateNone ? x[j] : __fmul_rn(g, x[j]);
      }
    }
    if (step + 1 < n_steps) load(step + 1);
    if (m.first != 0) {
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const int s = __shfl_sync(0xffffffffu, m.seq, i);
        if ((m.first >> i & 1) && c_ok) {
          float h0[VEC];
          state_get<VEC>(p.initial_state, s, C, c, h0);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            // (without a state, 0: a = inf or NaN stays the caller's own)
            if (p.initial_state != nullptr) u[i][j] = __fmaf_rn(a[i][j], h0[j], u[i][j]);
            a[i][j] = 0.f;
          }
        }
      }
    }
    // this thread's run of tokens, then the warps' runs
    Run<VEC> run;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      run.A[j] = a[0][j];
      run.h[j] = u[0][j];
#pragma unroll
      for (int i = 1; i < kTok; ++i) {
        run.A[j] = __fmul_rn(run.A[j], a[i][j]);
        run.h[j] = (m.first >> i & 1) ? u[i][j] : __fmaf_rn(a[i][j], run.h[j], u[i][j]);
      }
    }
    warp_run[warp][lane] = run;
    __syncthreads();
    Run<VEC> before;  // the warps before this one
    Run<VEC> all;     // the whole tile
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      all.A[j] = 1.f;
      all.h[j] = 0.f;
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) before = all;
      const Run<VEC> r = warp_run[w][lane];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        all.A[j] = __fmul_rn(all.A[j], r.A[j]);
        all.h[j] = through(r.A[j], r.h[j], all.h[j]);
      }
    }
    // warp w hands the tile's run to CTA w of the cluster.  The two buffers
    // alternate: a CTA writes step s + 2 only after the barrier of step s + 1,
    // which every CTA reaches after its reads of step s.
    Run<VEC>(*tr)[32] = tile_run[step & 1];
    if (warp < n_cta) {
      const uint32_t dst = sm100::mapa_shared(sm100::smem_u32(&tr[rank][lane]), (uint32_t)warp);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        st_cluster_f32(dst + 4 * j, all.A[j]);
        st_cluster_f32(dst + 4 * (VEC + j), all.h[j]);
      }
    }
    sm100::cluster_sync();
    float h[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = carry[j];
    for (int r = 0; r < n_cta; ++r) {
      if (r == rank) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[j] = carry[j];
      }
      const Run<VEC> q = tr[r][lane];
#pragma unroll
      for (int j = 0; j < VEC; ++j) carry[j] = through(q.A[j], q.h[j], carry[j]);
    }
    if (p.checkpoints != nullptr && warp == 0 && c_ok && tile < n_tiles)
      state_put<VEC>(p.checkpoints, tile, C, c, h);
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = through(before.A[j], before.h[j], h[j]);
    if (c_ok && p.y != nullptr) {
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          h[j] = (m.first >> i & 1) ? u[i][j] : __fmaf_rn(a[i][j], h[j], u[i][j]);
        if (t0 + i < T) R::store(Y + (t0 + i) * C, h);
        if ((m.last >> i & 1) && p.final_state != nullptr) {
          // (uniform over the warp's channels that exist; lanes past C hold no sequence)
          const int s = p.cu_seqlens == nullptr ? 0 : seq_at(p.cu_seqlens, p.n_seq, t0 + i);
          state_put<VEC>(p.final_state, s, C, c, h);
        }
      }
    }
  }
  empty_sequences<VEC>(p.cu_seqlens, p.n_seq, T, p.initial_state, p.final_state, C, c, c_ok,
                       rank * kWarps + warp, n_cta * kWarps, blockIdx.y == 0 ? p.err : nullptr);
}

// Backward.  With e_t = a_t dh_t (what token t hands to t - 1),
//   dh_t = dy_t + e_{t+1}            (last token: dy_t + dh_T)
//   e_t  = a_t e_{t+1} + a_t dy_t    (last token: a_t (dy_t + dh_T), carrying no e_{t+1})
//   dx = b dh, dbeta = x dh, dlog_alpha = h_{t-1} e   (b = 1 - a: (h_{t-1} - x) e),
//   dh_0 = e of the first token.
// The e run backwards through the same three levels, the cluster walking the
// tiles from the last to the first.  The h_{t-1} of a tile are folded again
// from the tile's checkpoint (the state before it, from the forward), so the
// forward carry needs the first two levels only.
template <typename Tin, int VEC, int GATE>
__global__ void __launch_bounds__(kThreads, 2) glr_bwd_kernel(const GlrArgs p) {
  __shared__ Run<VEC> warp_fwd[kWarps][32], warp_rev[kWarps][32];
  __shared__ Run<VEC> tile_run[2][kMaxCluster][32];
  using R = Raw<Tin, VEC>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_cta = (int)gridDim.x, rank = (int)blockIdx.x;
  const int C = p.C;
  const int c = ((int)blockIdx.y * 32 + lane) * VEC;
  const bool c_ok = c < C;
  const int64_t T = p.total_T;
  const int64_t n_tiles = (T + kGlrTile - 1) / kGlrTile;
  const int64_t n_steps = (n_tiles + n_cta - 1) / n_cta;
  const Tin* X = static_cast<const Tin*>(p.x) + c;
  const Tin* L = static_cast<const Tin*>(p.log_alpha) + c;
  const Tin* B = static_cast<const Tin*>(p.beta) + c;
  const Tin* DY = static_cast<const Tin*>(p.dy) + c;
  Tin* DX = static_cast<Tin*>(p.dx) + c;
  Tin* DL = static_cast<Tin*>(p.dlog_alpha) + c;
  Tin* DB = static_cast<Tin*>(p.dbeta) + c;

  // tiles in reverse: rank r of step s has tile n_tiles - 1 - (s n_cta + r),
  // negative (nothing to do, all neutral) behind the first tile
  R rx[kTok], rl[kTok], rb[kTok], rd[kTok];
  float ck[VEC];
  auto load = [&](int64_t step) {
    const int64_t tile = n_tiles - 1 - (step * n_cta + rank);
    const int64_t t0 = tile * kGlrTile + warp * kTok;
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const int64_t t = t0 + i;
      if (c_ok && t >= 0 && t < T) {
        rx[i].load(X + t * C);
        rl[i].load(L + t * C);
        if (GATE == kGateBeta) rb[i].load(B + t * C);
        rd[i].load(DY + t * C);
      } else {
        rx[i].zero();
        rl[i].zero();
        if (GATE == kGateBeta) rb[i].zero();
        rd[i].zero();
      }
    }
    state_get<VEC>(c_ok && tile >= 0 ? p.checkpoints : nullptr, tile, C, c, ck);
  };

  float carry[VEC];  // e of the token behind this step's last tile
#pragma unroll
  for (int j = 0; j < VEC; ++j) carry[j] = 0.f;
  if (n_steps > 0) {
    load(0);
    sm100::cluster_sync();
  }

  for (int64_t step = 0; step < n_steps; ++step) {
    const int64_t tile = n_tiles - 1 - (step * n_cta + rank);
    const int64_t t0 = tile * kGlrTile + warp * kTok;
    Marks m;
    m.first = m.last = 0;
    m.seq = 0;
    if (tile >= 0) m = marks_of(p.cu_seqlens, p.n_seq, T, t0, lane);
    float a[kTok][VEC], x[kTok][VEC], b[kTok][VEC], d[kTok][VEC], h[VEC];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      float l[VEC], be[VEC];
      rx[i].get(x[i]);
      rl[i].get(l);
      rd[i].get(d[i]);
      if (GATE == kGateBeta) rb[i].get(be);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float q;
        decay(l[j], a[i][j], q);
        b[i][j] = gate_of<GATE>(be[j], q);
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = ck[j];
    if (step + 1 < n_steps) load(step + 1);
    // dh_T joins its sequence's last dy
    if (m.last != 0 && p.d_final_state != nullptr) {
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const int s = __shfl_sync(0xffffffffu, m.seq, i);
        if ((m.last >> i & 1) && c_ok) {
          float f[VEC];
          state_get<VEC>(p.d_final_state, s, C, c, f);
#pragma unroll
          for (int j = 0; j < VEC; ++j) d[i][j] = __fadd_rn(d[i][j], f[j]);
        }
      }
    }
    // h before a token: h_0 of its sequence where that begins
    auto enter = [&](int i, float* hh) {
      if (m.first >> i & 1) {
        const int s = p.cu_seqlens == nullptr ? 0 : seq_at(p.cu_seqlens, p.n_seq, t0 + i);
        state_get<VEC>(c_ok ? p.initial_state : nullptr, s, C, c, hh);
      }
    };
    Run<VEC> fr, rr;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      fr.A[j] = rr.A[j] = 1.f;
      fr.h[j] = rr.h[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      enter(i, fr.h);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        fr.A[j] = (m.first >> i & 1) ? 0.f : __fmul_rn(fr.A[j], a[i][j]);
        fr.h[j] = __fmaf_rn(a[i][j], fr.h[j], __fmul_rn(b[i][j], x[i][j]));
      }
    }
#pragma unroll
    for (int i = kTok - 1; i >= 0; --i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const bool last = m.last >> i & 1;
        rr.A[j] = last ? 0.f : __fmul_rn(rr.A[j], a[i][j]);
        rr.h[j] = __fmul_rn(a[i][j], __fadd_rn(d[i][j], last ? 0.f : rr.h[j]));
      }
    }
    warp_fwd[warp][lane] = fr;
    warp_rev[warp][lane] = rr;
    __syncthreads();
    Run<VEC> behind, all;  // the warps behind this one, the whole tile, in reverse
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      all.A[j] = 1.f;
      all.h[j] = 0.f;
    }
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      if (w == warp) behind = all;
      const Run<VEC> r = warp_rev[w][lane];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        all.A[j] = __fmul_rn(all.A[j], r.A[j]);
        all.h[j] = through(r.A[j], r.h[j], all.h[j]);
      }
    }
    Run<VEC>(*tr)[32] = tile_run[step & 1];  // (two buffers: see the forward)
    if (warp < n_cta) {
      const uint32_t dst = sm100::mapa_shared(sm100::smem_u32(&tr[rank][lane]), (uint32_t)warp);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        st_cluster_f32(dst + 4 * j, all.A[j]);
        st_cluster_f32(dst + 4 * (VEC + j), all.h[j]);
      }
    }
    // the state before this warp's tokens
    for (int w = 0; w < warp; ++w) {
      const Run<VEC> r = warp_fwd[w][lane];
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[j] = through(r.A[j], r.h[j], h[j]);
    }
    sm100::cluster_sync();
    float e[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = carry[j];
    for (int r = 0; r < n_cta; ++r) {
      if (r == rank) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) e[j] = carry[j];
      }
      const Run<VEC> q = tr[r][lane];
#pragma unroll
      for (int j = 0; j < VEC; ++j) carry[j] = through(q.A[j], q.h[j], carry[j]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = through(behind.A[j], behind.h[j], e[j]);
    // h_{t-1} of every token, then the gradients from the last token back
    float hb[kTok][VEC];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      enter(i, h);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        hb[i][j] = h[j];
        h[j] = __fmaf_rn(a[i][j], h[j], __fmul_rn(b[i][j], x[i][j]));
      }
    }
#pragma unroll
    for (int i = kTok - 1; i >= 0; --i) {
      const int64_t t = t0 + i;
      float dx[VEC], dl[VEC], db[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float dh = __fadd_rn(d[i][j], (m.last >> i & 1) ? 0.f : e[j]);
        e[j] = __fmul_rn(a[i][j], dh);
        dx[j] = GATE == kGateNone ? dh : __fmul_rn(b[i][j], dh);
        db[j] = __fmul_rn(x[i][j], dh);
        dl[j] = __fmul_rn(GATE == kGateComp ? __fsub_rn(hb[i][j], x[i][j]) : hb[i][j], e[j]);
      }
      if (c_ok && t >= 0 && t < T) {
        R::store(DX + t * C, dx);
        R::store(DL + t * C, dl);
        if (GATE == kGateBeta) R::store(DB + t * C, db);
        if ((m.first >> i & 1) && p.d_initial_state != nullptr) {
          const int s = p.cu_seqlens == nullptr ? 0 : seq_at(p.cu_seqlens, p.n_seq, t);
          state_put<VEC>(p.d_initial_state, s, C, c, e);
        }
      }
    }
  }
  empty_sequences<VEC>(p.cu_seqlens, p.n_seq, T, p.d_final_state, p.d_initial_state, C, c, c_ok,
                       rank * kWarps + warp, n_cta * kWarps, blockIdx.y == 0 ? p.err : nullptr);
}

// One token: [N, C] arrays, all dense and of one shape, so n = N C values in
// a row.  A thread takes 8 of them with 16-byte accesses; the last n % 8
// are taken singly.
template <typename Tin, int GATE>
__global__ void __launch_bounds__(256) glr_step_kernel(const Tin* __restrict__ x,
                                                       const Tin* __restrict__ la,
                                                       const Tin* __restrict__ beta,
                                                       float* __restrict__ state,
                                                       Tin* __restrict__ y, int64_t n) {
  const int64_t i0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (i0 >= n) return;
  auto one = [&](float xv, float lv, float bv, float h) {
    float a, q;
    decay(lv, a, q);
    const float g = gate_of<GATE>(bv, q);
    return __fmaf_rn(a, h, GATE == kGateNone ? xv : __fmul_rn(g, xv));
  };
  if (i0 + 8 <= n) {
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const float4 xv = Elem<Tin>::load4(x + i0 + k), lv = Elem<Tin>::load4(la + i0 + k);
      float4 bv = make_float4(0.f, 0.f, 0.f, 0.f);
      if (GATE == kGateBeta) bv = Elem<Tin>::load4(beta + i0 + k);
      float4 h = *reinterpret_cast<const float4*>(state + i0 + k);
      h.x = one(xv.x, lv.x, bv.x, h.x);
      h.y = one(xv.y, lv.y, bv.y, h.y);
      h.z = one(xv.z, lv.z, bv.z, h.z);
      h.w = one(xv.w, lv.w, bv.w, h.w);
      *reinterpret_cast<float4*>(state + i0 + k) = h;
      Elem<Tin>::store4(y + i0 + k, h);
    }
  } else {
    for (int64_t i = i0; i < n; ++i) {
      const float h = one(Elem<Tin>::load(x + i), Elem<Tin>::load(la + i),
                          GATE == kGateBeta ? Elem<Tin>::load(beta + i) : 0.f, state[i]);
      state[i] = h;
      Elem<Tin>::store(y + i, h);
    }
  }
}

using ScanKernel = void (*)(GlrArgs);

template <typename Tin, int VEC>
ScanKernel scan_kernel(bool bwd, int gate) {
  switch (gate) {
    case kGateNone:
      return bwd ? glr_bwd_kernel<Tin, VEC, kGateNone> : glr_fwd_kernel<Tin, VEC, kGateNone>;
    case kGateBeta:
      return bwd ? glr_bwd_kernel<Tin, VEC, kGateBeta> : glr_fwd_kernel<Tin, VEC, kGateBeta>;
    default:
      return bwd ? glr_bwd_kernel<Tin, VEC, kGateComp> : glr_fwd_kernel<Tin, VEC, kGateComp>;
  }
}

cudaLaunchConfig_t scan_config(int cluster, int groups, cudaStream_t stream,
                               cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster, (unsigned)groups);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)cluster;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of each size that the device holds at once, per kernel (asked once
// per device; the answers are the same whoever asks, so threads may race).
constexpr int kMaxDevices = 64;
constexpr int kVariants = 2 * 2 * 2 * 3;
std::atomic<int> g_fit[kMaxDevices][kVariants][kMaxCluster + 1];

int clusters_that_fit(int dev, int variant, ScanKernel k, int cluster) {
  std::atomic<int>& slot = g_fit[dev][variant][cluster];
  int n = slot.load(std::memory_order_relaxed);
  if (n != 0) return n;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = scan_config(cluster, 1, nullptr, &attr);
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) return 0;
  slot.store(n, std::memory_order_relaxed);
  return n;
}

gdn_status launch_scan(const GlrArgs& a, bool bwd, cudaStream_t stream) {
  const bool bf16 = a.dtype == GDN_BF16;
  const int vec = a.C % 2 == 0 ? 2 : 1;  // an odd row length leaves every other row odd
  const ScanKernel k =
      bf16 ? (vec == 2 ? scan_kernel<__nv_bfloat16, 2>(bwd, a.gate)
                       : scan_kernel<__nv_bfloat16, 1>(bwd, a.gate))
           : (vec == 2 ? scan_kernel<float, 2>(bwd, a.gate) : scan_kernel<float, 1>(bwd, a.gate));
  const int variant = ((bf16 ? 0 : 1) * 2 + (vec - 1)) * 2 * 3 + (bwd ? 3 : 0) + a.gate;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GDN_ERR_CUDA;
  const int groups = (a.C + 32 * vec - 1) / (32 * vec);
  if (groups > 65535) return GDN_ERR_UNSUPPORTED;
  // The largest cluster (consecutive tiles in flight per channel group) at
  // which all groups' clusters are on the device at once.
  const int64_t n_tiles = (a.total_T + kGlrTile - 1) / kGlrTile;
  int cluster = (int)(n_tiles < kMaxCluster ? (n_tiles < 1 ? 1 : n_tiles) : kMaxCluster);
  while (cluster > 1 && clusters_that_fit(dev, variant, k, cluster) < groups) --cluster;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = scan_config(cluster, groups, stream, &attr);
  return cudaLaunchKernelEx(&cfg, k, a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename Tin>
gdn_status launch_step(const GlrArgs& a, int64_t n, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((n + 8 * 256 - 1) / (8 * 256));
  const Tin* x = static_cast<const Tin*>(a.x);
  const Tin* l = static_cast<const Tin*>(a.log_alpha);
  const Tin* b = static_cast<const Tin*>(a.beta);
  Tin* y = static_cast<Tin*>(a.y);
  switch (a.gate) {
    case kGateNone:
      glr_step_kernel<Tin, kGateNone><<<blocks, 256, 0, stream>>>(x, l, b, a.final_state, y, n);
      break;
    case kGateBeta:
      glr_step_kernel<Tin, kGateBeta><<<blocks, 256, 0, stream>>>(x, l, b, a.final_state, y, n);
      break;
    default:
      glr_step_kernel<Tin, kGateComp><<<blocks, 256, 0, stream>>>(x, l, b, a.final_state, y, n);
  }
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

gdn_status launch_glr_fwd(const GlrArgs& a, cudaStream_t stream) {
  return launch_scan(a, false, stream);
}

gdn_status launch_glr_bwd(const GlrArgs& a, cudaStream_t stream) {
  return launch_scan(a, true, stream);
}

gdn_status launch_glr_step(const GlrArgs& a, cudaStream_t stream) {
  const int64_t n = a.total_T * a.C;
  return a.dtype == GDN_BF16 ? launch_step<__nv_bfloat16>(a, n, stream)
                             : launch_step<float>(a, n, stream);
}

}  // namespace gdn
