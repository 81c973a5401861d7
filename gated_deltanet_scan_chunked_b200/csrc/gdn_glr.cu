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
// Layout.  A CTA of W warps owns a tile of W runs (16 tokens, backward 8) x 64
// channels: warp w has the tile's w-th run, a lane two channels.  The carry
// along the tokens passes three levels, each in a fixed order (results do not
// depend on timing): a thread's run in registers, the tile's runs through
// shared memory, and the CTAs of a cluster, which hold consecutive tiles of
// the same channels, through distributed shared memory.  The cluster walks the
// packed tokens in steps of (cluster size) tiles, the carry kept in registers;
// nothing is exchanged through global memory, so there is no workspace and no
// flag in it to wait on.  Every input is read once and every output written
// once.
//
// Inputs come into two shared-memory stages, so that the next step's loads are
// in flight while this one is folded, and outputs leave through shared memory
// (the forward's from room of their own where there is some, else from the
// places of the inputs that they replace): by TMA where rows of C elements are a
// multiple of 16 bytes (AL), one box of 64 channels a tensor.  Other rows begin
// anywhere, but 4 (fp32) or 8 (bf16) of them together are such a multiple: the
// inputs are then loaded as boxes of every 4th or 8th row, from the 16-byte
// boundary below a piece on and 16 bytes wider, and outputs are stored from
// registers.  (Against 16-byte asynchronous copies of all threads, in one run: fp32,
// C = 1333, 20011 tokens of 24 sequences 80 us for 91, with beta, one sequence 74
// for 100; the backward 135 for 169 and 156 for 211.)
//
// What bounds it.  A dozen operations an element leave it memory bound in
// principle.  In practice a step is a chain (inputs, fold, the cluster's
// exchange, outputs) that the two to four CTAs of an SM overlap: at wide C the
// memory is the limit, at others the part of the SMs that whole clusters of one
// wave can fill, and with three tensors the latency of that chain.  Measured on a
// B200 (a copy runs at 6.54 TB/s; calls in a CUDA graph), time and bytes read and
// written by time:
//   forward, bf16, beta, C = 6144, T = 4096          36.9 us   5.45 TB/s
//   forward, bf16, beta, C = 9216, T = 16384          199 us   6.07 TB/s
//   forward, bf16, b = 1 - a, C = 2560, T = 131072    449 us   4.48 TB/s
//   forward, fp32, b = 1, C = 1333 (unaligned),
//     20011 tokens of 24 sequences                   81.9 us   3.91 TB/s
//   backward, bf16, beta, C = 6144, T = 32768         514 us   5.53 TB/s
//   backward, bf16, beta, C = 2560, T = 4096         36.0 us   4.11 TB/s
//   forward, bf16, beta, C = 2560, T = 128            4.3 us   (one step: its
//     load, the exchange, its store)
//
// Runs in which a sequence begins or ends take a path of their own behind the
// common one: for each such token, in a loop over the marks, the states of
// its sequence are fetched and added at that token (its index known only at run
// time: a select over the run), then the run is folded again with its cuts.
#include <cuda.h>

#include <atomic>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

constexpr int kChan = 64;  // channels of a CTA
constexpr int kMaxCluster = 16;  // (more than 8: by leave of cudaFuncSetAttribute)
constexpr uint32_t kWait = 1u << 24;  // polls of a bounded wait

enum : int { kGateNone = GDN_GLR_GATE_NONE, kGateBeta = GDN_GLR_GATE_BETA,
             kGateComp = GDN_GLR_GATE_COMPLEMENT };

using f2 = float2;  // two channels of a lane

__device__ __forceinline__ f2 both(float v) { return make_float2(v, v); }
// (one packed instruction for both channels, each rounded as by itself)
__device__ __forceinline__ f2 unpacked(uint64_t v) {
  f2 r;
  f2_unpack(v, r.x, r.y);
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  return unpacked(f2_mul(f2_pack(a.x, a.y), f2_pack(b.x, b.y)));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  return unpacked(f2_add(f2_pack(a.x, a.y), f2_pack(b.x, b.y)));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  return unpacked(f2_fma(f2_pack(a.x, a.y), f2_pack(b.x, b.y), f2_pack(c.x, c.y)));
}

// a = exp(l) and 1 - a.  Channels that remember a thousand tokens have a
// within 1e-3 of 1, where an error of exp in one direction adds up over all of
// them.  So for |l| < 1/4, a = 1 + l q(l), rounded once, with
//   q = 1 + l/2 + l^2 (r0 + r1 l + r2 l^2),
// the first terms exact and the r fitted to (e^l - 1 - l - l^2/2) / l^3 so
// that the largest relative error of l q over the range is least: 1.8e-7, at
// its ends, falling with l^2 towards 0.  Further out the hardware 2^x, good to
// 2^-22, serves, since such a channel forgets within a few tokens.
template <int GATE>
__device__ __forceinline__ void decay2(f2 l, f2& a, f2& one_minus_a) {
  f2 q = fma2(l, both(0.008352220989763737f), both(0.04174217954277992f));
  q = fma2(l, q, both(0.16666626930236816f));
  q = fma2(l, q, both(0.5f));
  q = fma2(l, q, both(1.f));
  const f2 n = fma2(l, q, both(1.f)), z = mul2(l, both(1.4426950408889634f));
  const float e0 = sm100::ex2_approx(z.x), e1 = sm100::ex2_approx(z.y);
  const bool near0 = fabsf(l.x) < 0.25f, near1 = fabsf(l.y) < 0.25f;
  a = make_float2(near0 ? n.x : e0, near1 ? n.y : e1);
  if (GATE == kGateComp) {
    const f2 lq = mul2(l, q);
    one_minus_a = make_float2(near0 ? -lq.x : __fadd_rn(1.f, -e0),
                              near1 ? -lq.y : __fadd_rn(1.f, -e1));
  }
}

// The input b x of two channels.
template <int GATE>
__device__ __forceinline__ f2 gated(f2 x, f2 beta, f2 one_minus_a) {
  return GATE == kGateNone ? x : mul2(GATE == kGateBeta ? beta : one_minus_a, x);
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

// Which of a run's tokens from t0 on begin or end a sequence (bit i: token
// t0 + i; tokens outside [0, total_T) neither).  The sequence that the walk has
// come to and its bounds [lo, hi) are kept: most runs of long sequences lie
// inside it and need no look at the offsets.  For another run a lane has one of
// the 32 offsets beyond them: those that fall into the run are its marks, and a
// token's sequence is counted from the walk's over those up to it.  Only where
// 32 are not enough are sequences searched for.
template <int RUN, bool BACK>
struct Marks {
  uint32_t first = 0, last = 0;
  int at;       // sequence of the walk's last token; before the first, none
  int lo, hi;   // its bounds
  int from;     // (this run's) the walk's sequence before the run; none: searched for
  int off;      // (this lane's) an offset beyond it; searched for: token `lane`'s sequence
  static constexpr int kSearched = -2;

  __device__ __forceinline__ explicit Marks(const GlrArgs& p)
      : at(BACK ? p.n_seq : -1), lo(BACK ? 0x7fffffff : 0), hi(BACK ? 0x7fffffff : 0), from(at) {}

  __device__ __forceinline__ void look(const GlrArgs& p, int64_t t0, int lane) {
    first = last = 0;
    if (t0 < 0 || t0 >= p.total_T) return;
    const int t = (int)t0, n = p.total_T - t0 < RUN ? (int)(p.total_T - t0) : RUN;
    if (p.cu_seqlens == nullptr) {
      if (t == 0) first = 1;
      if (t0 + RUN >= p.total_T) last = 1u << (n - 1);
      return;
    }
    if (lo < t && t0 + RUN < hi) return;
    const uint32_t valid = 0xffffffffu >> (32 - n);
    const int i = BACK ? at - lane : at + 1 + lane;
    from = at;
    off = i < 0 ? -1 : i > p.n_seq ? 0x7fffffff : __ldg(p.cu_seqlens + i);
    const int passed = __popc(upto(p, BACK ? t : t + n - 1, lane));
    if (passed < 32) {
      const uint32_t d = (uint32_t)off - (uint32_t)t;  // (others are at or above RUN)
      const uint32_t b = d < RUN ? 1u << d : 0, e = d - 1u < RUN ? 1u << (d - 1u) : 0;
      first = __reduce_or_sync(0xffffffffu, b) & valid;
      last = __reduce_or_sync(0xffffffffu, e) & valid;
      const int x = __shfl_sync(0xffffffffu, off, passed);
      const int y = __shfl_sync(0xffffffffu, off, passed - 1 & 31);
      if (BACK) {
        hi = passed != 0 ? y : hi;
        lo = x;
        at -= passed;
      } else {
        lo = passed != 0 ? y : lo;
        hi = x;
        at += passed;
      }
    } else {
      from = kSearched;
      int l = 0, h = 0;
      if (lane < n) {
        off = seq_at(p.cu_seqlens, p.n_seq, t + lane);
        l = __ldg(p.cu_seqlens + off);
        h = __ldg(p.cu_seqlens + off + 1);
      }
      first = __ballot_sync(0xffffffffu, lane < n && l == t + lane);
      last = __ballot_sync(0xffffffffu, lane < n && h == t + lane + 1);
      const int end = BACK ? 0 : n - 1;
      at = __shfl_sync(0xffffffffu, off, end);
      lo = __shfl_sync(0xffffffffu, l, end);
      hi = __shfl_sync(0xffffffffu, h, end);
    }
  }
  // The lanes whose offset lies between the walk's sequence and token t's.
  __device__ __forceinline__ uint32_t upto(const GlrArgs& p, int t, int lane) const {
    return __ballot_sync(0xffffffffu, BACK ? off > t : from + 1 + lane < p.n_seq && off <= t);
  }
  // Sequence of the run's token i, one of the marked (some index, whatever the
  // offsets hold).
  __device__ __forceinline__ int seq_of(const GlrArgs& p, int64_t t0, int i, int lane) const {
    if (p.cu_seqlens == nullptr) return 0;
    if (from == kSearched) return __shfl_sync(0xffffffffu, off, i);
    const int passed = __popc(upto(p, (int)t0 + i, lane));
    return min(max(BACK ? from - passed : from + passed, 0), p.n_seq - 1);
  }
};

// Value k (known at run time) of a run held in registers, and its replacement.
template <int RUN>
__device__ __forceinline__ f2 pick(const f2 (&v)[RUN], int k) {
  f2 r = v[0];
#pragma unroll
  for (int i = 1; i < RUN; ++i)
    if (i == k) r = v[i];
  return r;
}
template <int RUN>
__device__ __forceinline__ void replace(f2 (&v)[RUN], int k, f2 x) {
#pragma unroll
  for (int i = 0; i < RUN; ++i)
    if (i == k) v[i] = x;
}

// A composed run, two channels.
struct __align__(16) Run {
  f2 A, h;
};

// A run that a sequence's border cuts has A = -0 in its first channel (products
// of a, which is never negative, have no sign): it forgets what was before it,
// even an infinity or NaN, since those belong to another sequence.  A product
// that falls to +0 inside a sequence does not: 0 x NaN stays NaN there, as in
// the recurrence.  CUT: a packed batch, which alone has anything to forget.
__device__ __forceinline__ f2 cut_A() { return both(-0.f); }

// h behind a run that is entered with h.
template <bool CUT>
__device__ __forceinline__ f2 through(const Run& r, f2 h) {
  const f2 n = fma2(r.A, h, r.h);
  return CUT && __float_as_int(r.A.x) < 0 ? r.h : n;
}
// A of two runs, one behind the other.
template <bool CUT>
__device__ __forceinline__ f2 behind_A(f2 a, f2 b) {
  f2 r = mul2(a, b);
  if (CUT)
    r.x = __int_as_float(__float_as_int(r.x) |
                         ((__float_as_int(a.x) | __float_as_int(b.x)) & (int)0x80000000));
  return r;
}

// A lane's two channels: neighbours where rows are aligned, else 32 apart.
template <bool AL>
struct Chan {
  int c0, c1;
  bool ok0, ok1;
  __device__ __forceinline__ Chan(int cb, int lane, int C) {
    c0 = cb + (AL ? 2 * lane : lane);
    c1 = AL ? c0 + 1 : c0 + 32;
    ok0 = c0 < C;
    ok1 = c1 < C;
  }
  // rows of a [.., C] fp32 array (nullptr: zeros)
  __device__ __forceinline__ f2 get(const float* p, int64_t row, int C) const {
    return make_float2(p != nullptr && ok0 ? p[row * C + c0] : 0.f,
                   p != nullptr && ok1 ? p[row * C + c1] : 0.f);
  }
  __device__ __forceinline__ void put(float* p, int64_t row, int C, f2 v) const {
    if (ok0) p[row * C + c0] = v.x;
    if (ok1) p[row * C + c1] = v.y;
  }
};

// Shared-memory image of one input tensor's piece of a tile.
template <typename T, bool AL>
struct Piece {
  static constexpr int kGroup = AL ? 1 : 16 / (int)sizeof(T);  // rows of a map's row
  static constexpr int kPitch = kChan * (int)sizeof(T) + (AL ? 0 : 16);  // bytes of a row
  // rows r = kGroup q + j of one j lie together
  static constexpr int part(int rows) { return (rows / kGroup * kPitch + 127) & ~127; }
  static constexpr int bytes(int rows) { return kGroup * part(rows); }
  static constexpr int at(int rows, int r) { return r % kGroup * part(rows) + r / kGroup * kPitch; }
  // A lane's two channels of one row; rem: where the row's piece begins.
  static __device__ __forceinline__ f2 get(const char* row, int rem, int lane) {
    if (sizeof(T) == 2) {
      uint32_t lo, hi;
      if (AL) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(row + 4 * lane);
        lo = w << 16;
        hi = w & 0xffff0000u;
      } else {
        lo = (uint32_t) * reinterpret_cast<const unsigned short*>(row + rem + 2 * lane) << 16;
        hi = (uint32_t) * reinterpret_cast<const unsigned short*>(row + rem + 2 * lane + 64) << 16;
      }
      return make_float2(__uint_as_float(lo), __uint_as_float(hi));
    }
    if (AL) return *reinterpret_cast<const f2*>(row + 8 * lane);
    return make_float2(*reinterpret_cast<const float*>(row + rem + 4 * lane),
                       *reinterpret_cast<const float*>(row + rem + 4 * lane + 128));
  }
  // Leaves an output in its input's place (AL).
  static __device__ __forceinline__ void put(char* row, int lane, f2 v) {
    if (sizeof(T) == 2)
      *reinterpret_cast<uint32_t*>(row + 4 * lane) = sm100::pack_bf16(v.x, v.y);
    else
      *reinterpret_cast<f2*>(row + 8 * lane) = v;
  }
};

// Stores a lane's two channels of a token row (unaligned rows); q: its first.
template <typename T>
__device__ __forceinline__ void put_out(T* q, const Chan<false>& ch, f2 v) {
  if (ch.ok0) Elem<T>::store(q, v.x);
  if (ch.ok1) Elem<T>::store(q + 32, v.y);
}

// TMA maps of the inputs and (AL) outputs: [total_T, C] with boxes of kChan
// channels x a tile's tokens.  Rows that are no multiple of 16 bytes: `kGroup`
// rows together are one, so the inputs' maps are [total_T / kGroup, kGroup C], and
// a box of every kGroup-th row begins at the 16-byte boundary below its piece,
// 16 bytes wider than it.  The last total_T % kGroup tokens are not in the maps.
struct ScanMaps {
  CUtensorMap in[4], out[3];
};

// Two stages of N input tensors' tiles of ROWS tokens.  Tokens outside [0, T)
// become zeros: a = exp(0) = 1 and x = 0 leave a state as it is.  Loads are
// numbered by step; step s goes to stage s & 1.  APART: the outputs are not left in
// the inputs' places but (AL) in room of their own behind the stages, or (else)
// are stored from registers, and the inputs are read once: a stage may be filled
// again in the middle of its own step, for the step after the next.
template <typename T, bool AL, int ROWS, int N, int THREADS, bool APART>
struct Stages {
  using P = Piece<T, AL>;
  static constexpr int kTensor = P::bytes(ROWS), kStage = N * kTensor;
  static constexpr int kBytes = 2 * kStage + (AL && APART ? kTensor : 0);
  char* at;
  uint64_t* full;  // [2] (AL)

  // (by every thread, before the block's first barrier)
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      sm100::mbar_init(&full[0], 1);
      sm100::mbar_init(&full[1], 1);
      sm100::fence_mbar_init();
    }
  }
  // (by every thread, after a barrier behind the last use of the stage; the
  // outputs that leave from it are read before it is filled again)
  __device__ __forceinline__ void load(int64_t step, bool any, const ScanMaps& maps, int64_t t0,
                                       int64_t total_T, int C, int cb) {
    if (!any || threadIdx.x != 0) return;
    constexpr int G = P::kGroup;
    const uint32_t stage = sm100::smem_u32(at) + (uint32_t)(step & 1) * kStage;
    uint64_t* bar = &full[step & 1];
    if (AL && !APART) sm100::bulk_wait_read_all();
    sm100::mbar_arrive_expect_tx(bar, N * ROWS * P::kPitch);
    // (fewer than G tokens are in no map: the box lies outside it)
    const int y = (int)(t0 / G) + (!AL && total_T < G ? 1 << 20 : 0);
    for (int j = 0; j < G; ++j) {
      const int x = AL ? cb : (j * C + cb) & ~(G - 1);
#pragma unroll
      for (int k = 0; k < N; ++k)
        sm100::tma_load_2d(stage + k * kTensor + j * P::part(ROWS), &maps.in[k], x, y, bar);
    }
  }
  // (by every warp, behind wait; !AL) The tokens of its run, from row `r0` of the
  // tile, that are in no map, each lane's own channels.
  template <int RUN>
  __device__ __forceinline__ void last_tokens(int64_t step, const char* const (&src)[N], int r0,
                                              int64_t t0, int64_t total_T, int C,
                                              const Chan<AL>& ch, int lane) {
    constexpr int G = P::kGroup, E = (int)sizeof(T);
    const int64_t mapped = total_T / G * G;
    if (t0 >= total_T || t0 + RUN <= mapped) return;
    char* stage = at + (int)(step & 1) * kStage;
#pragma unroll 1
    for (int64_t t = t0 > mapped ? t0 : mapped; t < t0 + RUN && t < total_T; ++t) {
      const int r = r0 + (int)(t - t0), rem = (int)((uint32_t)t * (uint32_t)(C * E) & 15u);
      char* row = stage + P::at(ROWS, r) + rem + E * lane;
      const int64_t from = t * C + ch.c0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const T* q = reinterpret_cast<const T*>(src[k]) + from;
        if (ch.ok0) *reinterpret_cast<T*>(row + k * kTensor) = q[0];
        if (ch.ok1) *reinterpret_cast<T*>(row + k * kTensor + 32 * E) = q[32];
      }
    }
    sm100::fence_proxy_async();  // before the stage is filled again
  }
  // (by every thread) Waits for the step's inputs.  ok: no bounded wait ran out
  // yet (then none is made).
  __device__ __forceinline__ bool wait(int64_t step, bool ok) {
    return ok && sm100::mbar_wait(&full[step & 1], (uint32_t)(step >> 1) & 1u, kWait);
  }
  // (by thread 0, before a barrier in front of the next outputs; AL, APART) The
  // last ones have left.
  __device__ __forceinline__ void free_outputs() {
    if (AL && APART && threadIdx.x == 0) sm100::bulk_wait_read_all();
  }
  // (by every thread, its outputs in place; AL) Sends the tile of step `step` off.
  __device__ __forceinline__ void store(int64_t step, int n, const ScanMaps& maps, int64_t t0,
                                        int cb) {
    sm100::fence_proxy_async();  // the outputs, before the copies read them
    if (threadIdx.x >= 32) {
      sm100::named_arrive(1, THREADS);
      return;
    }
    sm100::named_sync(1, THREADS);
    if (threadIdx.x == 0) {
      const uint32_t stage = sm100::smem_u32(at) + (APART ? 2u : (uint32_t)(step & 1)) * kStage;
      for (int k = 0; k < n; ++k)
        sm100::tma_store_2d(&maps.out[k], cb, (int)t0, stage + k * kTensor);
      sm100::bulk_commit();
    }
  }
};

// A tile's run to one CTA of the cluster (its address there), counted on that
// CTA's barrier.
__device__ __forceinline__ void send_run(uint32_t addr, uint32_t bar, const Run& r) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::
          "r"(addr),
      "f"(r.A.x), "f"(r.A.y), "f"(r.h.x), "f"(r.h.y), "r"(bar)
      : "memory");
}

// The runs of a tile's warps, in order or backwards: what lies before this
// warp's run, and the whole.
template <int W, bool BACK, bool CUT>
__device__ __forceinline__ void fold_tile(const Run (*runs)[32], int lane, int warp, Run& before,
                                          Run& all) {
  all.A = both(1.f);
  all.h = both(0.f);
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const int w = BACK ? W - 1 - k : k;
    if (w == warp) before = all;
    const Run r = runs[w][lane];
    all.h = through<CUT>(r, all.h);
    all.A = behind_A<CUT>(all.A, r.A);
  }
}

// The cluster's exchange of tile runs.  In every step each CTA sends its tile's
// run to all CTAs (itself too) and waits on its own barrier for theirs: the
// stores carry the signal, so no fence waits for the outputs of the step
// before.  Two buffers alternate: a CTA sends step s + 2 only after it has
// everyone's step s + 1, which each sends after its reads of step s.
struct Exchange {
  Run (*tiles)[32];  // [2][n_cta]
  uint64_t* bar;     // [2]
  int n_cta, rank;
  bool ok = true;

  // (by every thread, before the cluster's first barrier)
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      sm100::mbar_init(&bar[0], 1);
      sm100::mbar_init(&bar[1], 1);
      sm100::fence_mbar_init();
    }
  }
  // (by every warp: warp w of W sends to CTAs w, w + W, ..)
  template <int W>
  __device__ __forceinline__ void send(int64_t step, int lane, int warp, const Run& all) {
    const int b = (int)(step & 1);
    if (threadIdx.x == 0)
      sm100::mbar_arrive_expect_tx(&bar[b], (uint32_t)n_cta * 32u * (uint32_t)sizeof(Run));
    const uint32_t to = sm100::smem_u32(&tiles[b * n_cta + rank][lane]);
    const uint32_t on = sm100::smem_u32(&bar[b]);
    for (int r = warp; r < n_cta; r += W)
      send_run(sm100::mapa_shared(to, (uint32_t)r), sm100::mapa_shared(on, (uint32_t)r), all);
  }
  // Waits for the step's runs; h: the carry before this CTA's tile; carry
  // moves on past the whole step.
  template <bool CUT>
  __device__ __forceinline__ f2 receive(int64_t step, int lane, f2& carry) {
    const int b = (int)(step & 1);
    // (a thread that gave up never waits again, but still sends every step)
    ok = ok && sm100::mbar_wait_cluster(&bar[b], (uint32_t)(step >> 1) & 1u, kWait);
    f2 h = carry;
#pragma unroll 4
    for (int r = 0; r < n_cta; ++r) {
      if (r == rank) h = carry;
      carry = through<CUT>(tiles[b * n_cta + r][lane], carry);
    }
    return h;
  }
  // The tile's runs: what lies before this warp's, the whole to the cluster.
  template <int W, bool BACK, bool CUT>
  __device__ __forceinline__ Run give(int64_t step, int lane, int warp, const Run (*runs)[32]) {
    Run before, all;
    fold_tile<W, BACK, CUT>(runs, lane, warp, before, all);
    send<W>(step, lane, warp, all);
    return before;
  }
};

// Sequences without tokens carry their state through: out[s] = in[s] (or 0).
// Also reports a malformed cu_seqlens.  Rows are shared out over the
// cluster's warps.
template <bool AL>
__device__ __forceinline__ void empty_sequences(const GlrArgs& p, const float* in, float* out,
                                                const Chan<AL>& ch, int first_row, int stride,
                                                bool report) {
  for (int s = first_row; s < p.n_seq; s += stride) {
    int64_t lo = 0, hi = p.total_T;
    if (p.cu_seqlens != nullptr) {
      lo = __ldg(p.cu_seqlens + s);
      hi = __ldg(p.cu_seqlens + s + 1);
      const bool ok = lo >= 0 && hi >= lo && hi <= p.total_T && (s != 0 || lo == 0) &&
                      (s != p.n_seq - 1 || hi == p.total_T);
      if (!ok) {
        if (report && (threadIdx.x & 31) == 0) atomicOr(p.err, kErrBadSeqlens);
        continue;
      }
    }
    if (lo == hi && out != nullptr) ch.put(out, s, p.C, ch.get(in, s, p.C));
  }
}

// Tokens of a thread's run.  The forward holds a and b x of its run in registers
// (4 a token), the backward more.  Both come with 4 and with 8 warps to a CTA;
// the backward's tiles begin at checkpoints.  (Forward runs of 8 tokens in
// fp32 against 16: 20011 tokens of 24 sequences, C = 1336 98 us for 74, with beta
// 90 for 76, C = 2560 110 for 109; C = 6144 both 263.)
constexpr int kFwdRun = 16, kBwdRun = 8;
static_assert(4 * kBwdRun % kGlrTile == 0 && kGlrTile % kFwdRun == 0, "checkpoints at runs");

// Shared memory of a CTA: the runs of a tile (`sets` arrays, two buffers each),
// the cluster's tiles (two buffers), the barriers, two stages.
constexpr int runs_bytes(int w, int sets) { return 2 * sets * w * 32 * (int)sizeof(Run); }
constexpr int tiles_bytes(int cluster) { return 2 * cluster * 32 * (int)sizeof(Run); }
constexpr int kBarBytes = 128;
static_assert(runs_bytes(1, 1) % 128 == 0 && tiles_bytes(1) % 128 == 0, "stages on 128 bytes");

// CTAs of an SM (of 128 registers a thread, in clusters of 8) with that much
// shared memory for the stages.
constexpr int ctas_of_sm(int w, int stages) {
  const int fit = 227 * 1024 / (runs_bytes(w, 1) + tiles_bytes(8) + kBarBytes + stages + 1024);
  return fit < 16 / w ? fit : 16 / w;
}
// The forward's outputs get room apart where that costs no CTA of an SM in clusters
// of 8 (of two bf16 inputs in clusters of 12 and more it costs the fourth CTA, which
// `choose` sees and avoids): loads then have a step and a half to arrive, not a
// half (bf16, gate beta, us, apart
// against in place: 4 warps, C = 6144, T = 32768 263 for 290, C = 2560, T = 131072
// 444 for 483; 8 warps, two CTAs of an SM in place and one apart, C = 9216, T =
// 16384 216 for 199; fp32, gate beta, 4 warps likewise, C = 2560, T = 32768 233
// for 210).
template <typename T, int GATE, bool AL, int W, bool APART>
using FwdStagesOf = Stages<T, AL, W * kFwdRun, GATE == kGateBeta ? 3 : 2, 32 * W, APART>;
template <typename T, int GATE, bool AL, int W>
constexpr bool kFwdApart = ctas_of_sm(W, FwdStagesOf<T, GATE, AL, W, true>::kBytes) ==
                           ctas_of_sm(W, FwdStagesOf<T, GATE, AL, W, false>::kBytes);
template <typename T, int GATE, bool AL, int W>
using FwdStages = FwdStagesOf<T, GATE, AL, W, kFwdApart<T, GATE, AL, W>>;
static_assert(kFwdApart<float, kGateBeta, false, 8>, "outputs from registers cost no room");
template <typename T, int GATE, bool AL, int W>
using BwdStages = Stages<T, AL, W * kBwdRun, GATE == kGateBeta ? 4 : 3, 32 * W, false>;

template <typename T, int GATE, bool AL, int W>
__global__ void __launch_bounds__(32 * W, 16 / W)
    glr_fwd_kernel(const GlrArgs p, const __grid_constant__ ScanMaps maps) {
  constexpr int RUN = kFwdRun, ROWS = W * RUN;
  constexpr int N = GATE == kGateBeta ? 3 : 2;
  using P = Piece<T, AL>;
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_cta = (int)gridDim.x, rank = (int)blockIdx.x;  // one cluster along x
  Run(*run_buf)[32] = reinterpret_cast<Run(*)[32]>(smem);    // [2][W]
  Exchange ex;
  ex.n_cta = n_cta;
  ex.rank = rank;
  ex.tiles = run_buf + 2 * W;
  ex.bar = reinterpret_cast<uint64_t*>(ex.tiles + 2 * n_cta);
  FwdStages<T, GATE, AL, W> stages;
  stages.full = ex.bar + 2;
  stages.at = reinterpret_cast<char*>(ex.bar) + kBarBytes;

  const int C = p.C, cb = (int)blockIdx.y * kChan;
  const Chan<AL> ch(cb, lane, C);
  const int64_t T_ = p.total_T;
  const int64_t n_tiles = (T_ + ROWS - 1) / ROWS;
  const int64_t n_steps = (n_tiles + n_cta - 1) / n_cta;
  const uint32_t row_bytes = (uint32_t)C * (uint32_t)sizeof(T);
  const char* src[N];
  src[0] = static_cast<const char*>(p.x);
  src[1] = static_cast<const char*>(p.log_alpha);
  if (N == 3) src[N - 1] = static_cast<const char*>(p.beta);
  auto load = [&](int64_t step) {
    stages.load(step, step < n_steps, maps, (step * n_cta + rank) * ROWS, T_, C, cb);
  };

  f2 carry = both(0.f);  // state before this step's first tile
  Marks<RUN, false> m(p);
  if (n_steps > 0) {
    stages.init();
    ex.init();
    sm100::cluster_sync();  // every CTA runs, its barriers set, before any sends
    load(0);
    load(1);
  }
  for (int64_t step = 0; step < n_steps; ++step) {
    const int64_t tile0 = (step * n_cta + rank) * ROWS, t0 = tile0 + warp * RUN;
    m.look(p, t0, lane);
    const bool inside = (m.first | m.last) == 0;
    ex.ok = stages.wait(step, ex.ok);
    if constexpr (!AL)
      stages.template last_tokens<RUN>(step, src, warp * RUN, t0, T_, C, ch, lane);
    char* st = stages.at + (int)(step & 1) * stages.kStage + warp * (RUN / P::kGroup) * P::kPitch;
    [[maybe_unused]] char* to = kFwdApart<T, GATE, AL, W>
                                    ? stages.at + 2 * stages.kStage + warp * RUN * P::kPitch
                                    : st;
    auto in = [&](int k, int i) {  // tensor k at token i of the run
      return P::get(st + k * stages.kTensor + P::at(ROWS, i),
                    AL ? 0 : (int)((uint32_t)(i % P::kGroup) * row_bytes & 15u), lane);
    };
    f2 a[RUN], u[RUN];
    Run run;
    run.A = both(1.f);
    run.h = both(0.f);
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      f2 q;
      decay2<GATE>(in(1, i), a[i], q);
      u[i] = gated<GATE>(in(0, i), GATE == kGateBeta ? in(N - 1, i) : both(0.f), q);
      run.A = mul2(run.A, a[i]);
      run.h = fma2(a[i], run.h, u[i]);
    }
    if (m.first != 0) {  // h_0 joins at first tokens, which forget what was before them
      for (uint32_t f = m.first; f != 0; f &= f - 1) {
        const int k = __ffs((int)f) - 1;
        const f2 h0 = ch.get(p.initial_state, m.seq_of(p, t0, k, lane), C);
        replace(u, k, fma2(pick(a, k), h0, pick(u, k)));
      }
      run.A = cut_A();
#pragma unroll
      for (int i = 0; i < RUN; ++i)
        run.h = (m.first >> i & 1) ? u[i] : fma2(a[i], run.h, u[i]);
    }
    // (two buffers: a warp may still fold this step's runs when others write
    // the next one's)
    Run(*runs)[32] = run_buf + (int)(step & 1) * W;
    runs[warp][lane] = run;
    stages.free_outputs();
    // the runs are complete; this step's inputs are read, the step before is done
    // with its stage
    __syncthreads();
    if (kFwdApart<T, GATE, AL, W>) load(step + 2);
    else if (step > 0) load(step + 1);
    f2 h;
    if (p.cu_seqlens == nullptr) {
      const Run before = ex.template give<W, false, false>(step, lane, warp, runs);
      h = through<false>(before, ex.template receive<false>(step, lane, carry));
    } else {
      const Run before = ex.template give<W, false, true>(step, lane, warp, runs);
      h = through<true>(before, ex.template receive<true>(step, lane, carry));
    }
    if (p.checkpoints != nullptr && t0 % kGlrTile == 0 && t0 < T_)
      ch.put(p.checkpoints, t0 / kGlrTile, C, h);
    if (p.y == nullptr) continue;
    [[maybe_unused]] T* y = static_cast<T*>(p.y) + t0 * C + ch.c0;
    [[maybe_unused]] const int n_tok = T_ - t0 < RUN ? (int)(T_ - t0) : RUN;
    auto out = [&](int i) {  // (called with i ascending)
      if constexpr (AL) {
        P::put(to + i * P::kPitch, lane, h);
      } else {
        if (i < n_tok) put_out<T>(y, ch, h);
        y += C;
      }
    };
    if (inside) {
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        h = fma2(a[i], h, u[i]);
        out(i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        h = (m.first >> i & 1) ? u[i] : fma2(a[i], h, u[i]);
        u[i] = h;
        out(i);
      }
      if (p.final_state != nullptr)
        for (uint32_t f = m.last; f != 0; f &= f - 1) {
          const int k = __ffs((int)f) - 1;
          ch.put(p.final_state, m.seq_of(p, t0, k, lane), C, pick(u, k));
        }
    }
    if (AL && tile0 < T_) stages.store(step, 1, maps, tile0, cb);
  }
  if (!ex.ok) atomicOr(p.err, kErrTimeout);
  if (AL && threadIdx.x == 0) sm100::bulk_wait_all();
  if (n_steps > 0) sm100::cluster_sync();  // (a CTA that gave up waiting may still be sent to)
  empty_sequences<AL>(p, p.initial_state, p.final_state, ch, rank * W + warp, n_cta * W,
                      blockIdx.y == 0);
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
template <typename T, int GATE, bool AL, int W>
__global__ void __launch_bounds__(32 * W, 16 / W)
    glr_bwd_kernel(const GlrArgs p, const __grid_constant__ ScanMaps maps) {
  constexpr int RUN = kBwdRun, ROWS = W * RUN;
  constexpr int N = GATE == kGateBeta ? 4 : 3;  // x, log_alpha, [beta,] dy
  constexpr int kBeta = 2, kDy = N - 1;
  using P = Piece<T, AL>;
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_cta = (int)gridDim.x, rank = (int)blockIdx.x;
  Run(*run_buf)[32] = reinterpret_cast<Run(*)[32]>(smem);  // [2][forward, reverse][W]
  Exchange ex;
  ex.n_cta = n_cta;
  ex.rank = rank;
  ex.tiles = run_buf + 4 * W;
  ex.bar = reinterpret_cast<uint64_t*>(ex.tiles + 2 * n_cta);
  BwdStages<T, GATE, AL, W> stages;
  stages.full = ex.bar + 2;
  stages.at = reinterpret_cast<char*>(ex.bar) + kBarBytes;

  const int C = p.C, cb = (int)blockIdx.y * kChan;
  const Chan<AL> ch(cb, lane, C);
  const int64_t T_ = p.total_T;
  const int64_t n_tiles = (T_ + ROWS - 1) / ROWS;
  const int64_t n_steps = (n_tiles + n_cta - 1) / n_cta;
  const uint32_t row_bytes = (uint32_t)C * (uint32_t)sizeof(T);
  const char* src[N];
  src[0] = static_cast<const char*>(p.x);
  src[1] = static_cast<const char*>(p.log_alpha);
  if (N == 4) src[kBeta] = static_cast<const char*>(p.beta);
  src[kDy] = static_cast<const char*>(p.dy);
  // tiles in reverse: rank r of step s has tile n_tiles - 1 - (s n_cta + r),
  // negative (nothing to do, all neutral) behind the first tile
  auto load = [&](int64_t step) {
    stages.load(step, step < n_steps, maps, (n_tiles - 1 - (step * n_cta + rank)) * ROWS, T_, C,
                cb);
  };

  f2 carry = both(0.f);  // e of the token behind this step's last tile
  Marks<RUN, true> m(p);
  if (n_steps > 0) {
    stages.init();
    ex.init();
    sm100::cluster_sync();
    load(0);
    load(1);
  }
  for (int64_t step = 0; step < n_steps; ++step) {
    const int64_t tile = n_tiles - 1 - (step * n_cta + rank);
    const int64_t t0 = tile * ROWS + warp * RUN;
    m.look(p, t0, lane);
    const bool inside = (m.first | m.last) == 0;
    f2 h = both(0.f);
    if (tile >= 0) h = ch.get(p.checkpoints, tile * (ROWS / kGlrTile), C);
    ex.ok = stages.wait(step, ex.ok);
    if constexpr (!AL)
      stages.template last_tokens<RUN>(step, src, warp * RUN, t0, T_, C, ch, lane);
    char* st = stages.at + (int)(step & 1) * stages.kStage + warp * (RUN / P::kGroup) * P::kPitch;
    auto in = [&](int k, int i) {  // tensor k at token i of the run
      return P::get(st + k * stages.kTensor + P::at(ROWS, i),
                    AL ? 0 : (int)((uint32_t)(i % P::kGroup) * row_bytes & 15u), lane);
    };
    // dy of the run; dh_T joins at its sequence's last token
    auto all_dy = [&](f2(&d)[RUN]) {
#pragma unroll
      for (int i = 0; i < RUN; ++i) d[i] = in(kDy, i);
      if (p.d_final_state != nullptr)
        for (uint32_t f = m.last; f != 0; f &= f - 1) {
          const int k = __ffs((int)f) - 1;
          replace(d, k, add2(pick(d, k), ch.get(p.d_final_state, m.seq_of(p, t0, k, lane), C)));
        }
    };
    f2 a[RUN], u[RUN], om[RUN];  // om: 1 - a
    Run fr, rr;
    fr.A = rr.A = both(1.f);
    fr.h = rr.h = both(0.f);
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      decay2<GATE>(in(1, i), a[i], om[i]);
      u[i] = gated<GATE>(in(0, i), GATE == kGateBeta ? in(kBeta, i) : both(0.f), om[i]);
      fr.A = mul2(fr.A, a[i]);
      fr.h = fma2(a[i], fr.h, u[i]);
    }
    rr.A = fr.A;
    if (inside) {
#pragma unroll
      for (int i = RUN - 1; i >= 0; --i) rr.h = mul2(a[i], add2(in(kDy, i), rr.h));
    } else {
      // (a run cut by a sequence's end forgets what is beyond it)
      f2 d[RUN];
      all_dy(d);
#pragma unroll
      for (int i = RUN - 1; i >= 0; --i)
        rr.h = mul2(a[i], (m.last >> i & 1) ? d[i] : add2(d[i], rr.h));
      if (m.last != 0) rr.A = cut_A();
      if (m.first != 0) {  // as in the forward
        for (uint32_t f = m.first; f != 0; f &= f - 1) {
          const int k = __ffs((int)f) - 1;
          const f2 h0 = ch.get(p.initial_state, m.seq_of(p, t0, k, lane), C);
          replace(u, k, fma2(pick(a, k), h0, pick(u, k)));
        }
        fr.A = cut_A();
#pragma unroll
        for (int i = 0; i < RUN; ++i)
          fr.h = (m.first >> i & 1) ? u[i] : fma2(a[i], fr.h, u[i]);
      }
    }
    Run(*fwd_runs)[32] = run_buf + (int)(step & 1) * 2 * W;  // (two buffers: see the forward)
    Run(*rev_runs)[32] = fwd_runs + W;
    fwd_runs[warp][lane] = fr;
    rev_runs[warp][lane] = rr;
    __syncthreads();  // the runs are complete; the step before is done with its stage
    if (step > 0) load(step + 1);
    // While the cluster's runs are under way: the state before this run, and
    // h_{t-1} of every token (into u).
    Run behind;
    if (p.cu_seqlens == nullptr) {
      behind = ex.template give<W, true, false>(step, lane, warp, rev_runs);
#pragma unroll
      for (int w = 0; w < W - 1; ++w)
        if (w < warp) h = through<false>(fwd_runs[w][lane], h);
    } else {
      behind = ex.template give<W, true, true>(step, lane, warp, rev_runs);
#pragma unroll
      for (int w = 0; w < W - 1; ++w)
        if (w < warp) h = through<true>(fwd_runs[w][lane], h);
    }
    if (m.first == 0) {
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        const f2 next = fma2(a[i], h, u[i]);
        u[i] = h;
        h = next;
      }
    } else {
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        const f2 next = (m.first >> i & 1) ? u[i] : fma2(a[i], h, u[i]);
        u[i] = h;
        h = next;
      }
      for (uint32_t f = m.first; f != 0; f &= f - 1) {  // before a first token: h_0
        const int k = __ffs((int)f) - 1;
        replace(u, k, ch.get(p.initial_state, m.seq_of(p, t0, k, lane), C));
      }
    }
    f2 e = p.cu_seqlens == nullptr
               ? through<false>(behind, ex.template receive<false>(step, lane, carry))
               : through<true>(behind, ex.template receive<true>(step, lane, carry));
    // Token i's gradients, from its x, h_{t-1} (hb), dh, e and b's parts.
    const int64_t o0 = t0 * C + ch.c0;
    [[maybe_unused]] const int n_tok = t0 < 0 ? 0 : T_ - t0 < RUN ? (int)(T_ - t0) : RUN;
    auto out = [&](int i, f2 dh, f2 hb, f2 om_i) {
      const f2 x = in(0, i);
      const f2 dx = gated<GATE>(dh, GATE == kGateBeta ? in(kBeta, i) : both(0.f), om_i);
      if (GATE == kGateComp) hb = fma2(x, both(-1.f), hb);
      const f2 dl = mul2(hb, e), db = mul2(x, dh);
      if constexpr (AL) {
        char* row = st + i * P::kPitch;
        P::put(row, lane, dx);
        P::put(row + stages.kTensor, lane, dl);
        if (GATE == kGateBeta) P::put(row + kBeta * stages.kTensor, lane, db);
      } else if (i < n_tok) {
        const int64_t o = o0 + (int64_t)i * C;
        put_out<T>(static_cast<T*>(p.dx) + o, ch, dx);
        put_out<T>(static_cast<T*>(p.dlog_alpha) + o, ch, dl);
        if (GATE == kGateBeta) put_out<T>(static_cast<T*>(p.dbeta) + o, ch, db);
      }
    };
    if (inside) {
#pragma unroll
      for (int i = RUN - 1; i >= 0; --i) {
        const f2 dh = add2(in(kDy, i), e);
        e = mul2(a[i], dh);
        out(i, dh, u[i], om[i]);
      }
    } else {
      f2 d[RUN];
      all_dy(d);
#pragma unroll
      for (int i = RUN - 1; i >= 0; --i) {
        const f2 dh = (m.last >> i & 1) ? d[i] : add2(d[i], e);
        d[i] = e = mul2(a[i], dh);
        out(i, dh, u[i], om[i]);
      }
      if (p.d_initial_state != nullptr)
        for (uint32_t f = m.first; f != 0; f &= f - 1) {
          const int k = __ffs((int)f) - 1;
          ch.put(p.d_initial_state, m.seq_of(p, t0, k, lane), C, pick(d, k));
        }
    }
    if (AL && tile >= 0) stages.store(step, N - 1, maps, tile * ROWS, cb);
  }
  if (!ex.ok) atomicOr(p.err, kErrTimeout);
  if (AL && threadIdx.x == 0) sm100::bulk_wait_all();
  if (n_steps > 0) sm100::cluster_sync();
  empty_sequences<AL>(p, p.d_final_state, p.d_initial_state, ch, rank * W + warp, n_cta * W,
                      blockIdx.y == 0);
}

// One token: [N, C] arrays, all dense and of one shape, so n = N C values in
// a row.  A thread takes 8 of them, four at a time (16 bytes of fp32, 8 of bf16);
// the last n % 8 are taken singly.  Bound by memory, and by its launch when small:
// bf16 with beta, N = 256, C = 6144 5.2 us (25 MB, 4.8 TB/s), N = 3, C = 2561 2.2 us.
template <typename Tin, int GATE>
__global__ void __launch_bounds__(256) glr_step_kernel(const Tin* __restrict__ x,
                                                       const Tin* __restrict__ la,
                                                       const Tin* __restrict__ beta,
                                                       float* __restrict__ state,
                                                       Tin* __restrict__ y, int64_t n) {
  const int64_t i0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (i0 >= n) return;
  auto two = [&](float x0, float x1, float l0, float l1, float b0, float b1, float& h0,
                 float& h1) {
    f2 a, q = both(0.f);
    decay2<GATE>(make_float2(l0, l1), a, q);
    const f2 u = gated<GATE>(make_float2(x0, x1), make_float2(b0, b1), q);
    const f2 h = fma2(a, make_float2(h0, h1), u);
    h0 = h.x;
    h1 = h.y;
  };
  if (i0 + 8 <= n) {
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const float4 xv = Elem<Tin>::load4(x + i0 + k), lv = Elem<Tin>::load4(la + i0 + k);
      float4 bv = make_float4(0.f, 0.f, 0.f, 0.f);
      if (GATE == kGateBeta) bv = Elem<Tin>::load4(beta + i0 + k);
      float4 h = *reinterpret_cast<const float4*>(state + i0 + k);
      two(xv.x, xv.y, lv.x, lv.y, bv.x, bv.y, h.x, h.y);
      two(xv.z, xv.w, lv.z, lv.w, bv.z, bv.w, h.z, h.w);
      *reinterpret_cast<float4*>(state + i0 + k) = h;
      Elem<Tin>::store4(y + i0 + k, h);
    }
  } else {
    for (int64_t i = i0; i < n; ++i) {
      float h = state[i], unused = 0.f;
      two(Elem<Tin>::load(x + i), 0.f, Elem<Tin>::load(la + i), 0.f,
          GATE == kGateBeta ? Elem<Tin>::load(beta + i) : 0.f, 0.f, h, unused);
      state[i] = h;
      Elem<Tin>::store(y + i, h);
    }
  }
}

using ScanKernel = void (*)(GlrArgs, ScanMaps);

// One compiled scan: its kernel, threads, tokens per tile and shared memory
// (apart from the cluster's part).
struct Scan {
  ScanKernel kernel;
  int threads, rows, smem;
};

enum : int { kFwd8 = 0, kFwd4 = 1, kBwd8 = 2, kBwd4 = 3, kScans = 4 };

template <typename T, bool AL, int GATE, int W>
Scan fwd_scan() {
  constexpr int rows = W * kFwdRun;
  return {glr_fwd_kernel<T, GATE, AL, W>, 32 * W, rows,
          runs_bytes(W, 1) + kBarBytes + FwdStages<T, GATE, AL, W>::kBytes};
}
template <typename T, bool AL, int GATE, int W>
Scan bwd_scan() {
  constexpr int rows = W * kBwdRun;
  return {glr_bwd_kernel<T, GATE, AL, W>, 32 * W, rows,
          runs_bytes(W, 2) + kBarBytes + BwdStages<T, GATE, AL, W>::kBytes};
}
template <typename T, bool AL, int GATE>
Scan scan_of(int what) {
  if (what == kFwd8) return fwd_scan<T, AL, GATE, 8>();
  if (what == kFwd4) return fwd_scan<T, AL, GATE, 4>();
  return what == kBwd8 ? bwd_scan<T, AL, GATE, 8>() : bwd_scan<T, AL, GATE, 4>();
}
template <typename T, bool AL>
Scan scan_gate(int what, int gate) {
  return gate == kGateNone   ? scan_of<T, AL, kGateNone>(what)
         : gate == kGateBeta ? scan_of<T, AL, kGateBeta>(what)
                             : scan_of<T, AL, kGateComp>(what);
}
Scan scan_for(const GlrArgs& a, bool al, int what) {
  if (a.dtype == GDN_BF16)
    return al ? scan_gate<__nv_bfloat16, true>(what, a.gate)
              : scan_gate<__nv_bfloat16, false>(what, a.gate);
  return al ? scan_gate<float, true>(what, a.gate) : scan_gate<float, false>(what, a.gate);
}

cudaLaunchConfig_t scan_config(const Scan& k, int cluster, int smem, int groups,
                               cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster, (unsigned)groups);
  cfg.blockDim = dim3((unsigned)k.threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)cluster;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
                       cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(f)
               : nullptr;
  }();
  return fn;
}

bool encode_map(CUtensorMap* m, const GlrArgs& a, const void* base, int rows, bool al) {
  const EncodeTiledFn fn = encode_tiled();
  const bool bf16 = a.dtype == GDN_BF16;
  // (Piece has the other side of this)
  const int g = al ? 1 : bf16 ? 8 : 4;
  const cuuint64_t whole = (cuuint64_t)(a.total_T / g);
  const cuuint64_t dims[2] = {(cuuint64_t)a.C * g, whole > 0 ? whole : 1};
  const cuuint64_t strides[1] = {(cuuint64_t)a.C * g * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {(cuuint32_t)(al ? kChan : kChan + g), (cuuint32_t)(rows / g)};
  const cuuint32_t one[2] = {1, 1};
  return fn != nullptr &&
         fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
            const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What is known of a device (asked once; the answers are the same whoever asks,
// so threads may race): its shared memory, and how many clusters of each kernel,
// size and share of an SM it holds at once (-1: none).
constexpr int kMaxDevices = 64, kMaxShare = 4;
constexpr int kVariants = 2 * 2 * kScans * 3;
struct Device {
  std::atomic<int> of_block, of_sm, reserved;  // bytes: most of a block, of an SM, a block's own
  std::atomic<int> fit[kVariants][kMaxShare][kMaxCluster + 1];
};
Device g_device[kMaxDevices];

bool know_device(int dev) {
  Device& d = g_device[dev];
  if (d.of_block.load(std::memory_order_acquire) != 0) return true;
  int block = 0, sm = 0, own = 0;
  if (cudaDeviceGetAttribute(&block, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
          cudaSuccess ||
      cudaDeviceGetAttribute(&sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) !=
          cudaSuccess ||
      cudaDeviceGetAttribute(&own, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess)
    return false;
  d.of_sm.store(sm, std::memory_order_relaxed);
  d.reserved.store(own, std::memory_order_relaxed);
  d.of_block.store(block, std::memory_order_release);
  return true;
}

// Shared memory of a CTA of which an SM shall hold at most `share`.
int shared_bytes(const Device& d, const Scan& k, int cluster, int share) {
  const int need = k.smem + tiles_bytes(cluster);
  const int least = d.of_sm.load(std::memory_order_relaxed) / (share + 1) -
                    d.reserved.load(std::memory_order_relaxed) + 128;
  return need > least ? need : least;
}

int clusters_that_fit(int dev, int variant, const Scan& k, int cluster, int share) {
  std::atomic<int>& slot = g_device[dev].fit[variant][share - 1][cluster];
  int n = slot.load(std::memory_order_relaxed);
  if (n != 0) return n;
  const int smem = shared_bytes(g_device[dev], k, cluster, share);
  const int most = g_device[dev].of_block.load(std::memory_order_relaxed);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = scan_config(k, cluster, smem, 1, nullptr, &attr);
  if (smem > most ||
      cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) !=
          cudaSuccess ||
      cudaFuncSetAttribute(k.kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, k.kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();  // (a size that the device cannot hold)
    n = -1;
  }
  slot.store(n, std::memory_order_relaxed);
  return n;
}

// How a scan is cut: its kernel, cluster size and CTAs of an SM, by the least
// estimated time,
//   steps of a cluster  x  waves of clusters  x  a step's time,
// the latter by how many CTAs share an SM.  Clusters are not spread evenly: of
// eight clusters of 16 CTAs two to an SM, some lie together on a few SMs and the
// others' steps are half as long; so no more CTAs are let onto an SM than the
// choice counts on, by the shared memory asked for.  Measured on a B200
// (forward, bf16, gate beta, us a step; the table serves the other types, gates and
// unaligned rows too, whose steps have not been measured each): 8 warps 2.05 alone
// and 2.85 by twos, 4 warps (half the tokens) 1.28, 1.65, 2.1 and 2.5; a further
// wave costs about a tenth; the backward's 4 warps are slower by comparison (on the scale of its 8:
// 1.46, 1.87, 2.26, 2.72).  What this settles (us, bf16):
//   forward, C = 6144, T = 32768: 8 warps in clusters of 2 (one wave, a third
//     of the SMs with two CTAs) 336, of 8 (three waves) 307, 4 warps in
//     clusters of 4 263;
//   forward, C = 2560, T = 131072: 8 warps in clusters of 6 487, of 7 (a second
//     wave for 3 of 40 groups) 668, 4 warps in clusters of 10 444;
//   forward, C = 9216, T = 16384: 8 warps in clusters of 2 199, 4 warps 211;
//   backward, C = 6144, T = 32768: 8 warps in clusters of 2 633, of 5 (two
//     waves) 567, 4 warps in clusters of 5, four to an SM, 515; C = 9216, T =
//     16384: 8 warps in clusters of 2 358, 4 warps in clusters of 7 391; C =
//     2560, T = 4096: 4 warps in clusters of 12, four to an SM, 38.9, of 10,
//     three to an SM, 36.0.
struct Choice {
  Scan scan;
  int cluster, smem;  // cluster 0: none
  double cost;
};

Choice choose(int dev, const GlrArgs& a, bool al, int what, int groups) {
  static const double kStep8[] = {2.05, 2.85}, kFwdStep4[] = {1.28, 1.65, 2.1, 2.5},
                      kBwdStep4[] = {1.46, 1.87, 2.26, 2.72};
  const bool small = what == kFwd4 || what == kBwd4;
  const double* step_us = what == kFwd4 ? kFwdStep4 : what == kBwd4 ? kBwdStep4 : kStep8;
  const Scan k = scan_for(a, al, what);
  const int variant =
      (((a.dtype == GDN_BF16 ? 0 : 1) * 2 + (al ? 0 : 1)) * kScans + what) * 3 + a.gate;
  const int64_t n_tiles = (a.total_T + k.rows - 1) / k.rows;
  const int most = (int)(n_tiles < kMaxCluster ? (n_tiles < 1 ? 1 : n_tiles) : kMaxCluster);
  Choice best = {k, 0, 0, 0.0};
  for (int share = 1; share <= (small ? kMaxShare : 2); ++share)
    for (int r = 1; r <= most; ++r) {
      const int fit = clusters_that_fit(dev, variant, k, r, share);
      if (fit < 1) continue;
      const int waves = (groups + fit - 1) / fit;
      const double cost = (double)((n_tiles + r - 1) / r) * waves * (1.0 + 0.1 * (waves - 1)) *
                          step_us[share - 1];
      if (best.cluster == 0 || cost < best.cost)
        best = {k, r, shared_bytes(g_device[dev], k, r, share), cost};
    }
  return best;
}

gdn_status launch_scan(const GlrArgs& a, bool bwd, cudaStream_t stream) {
  const bool bf16 = a.dtype == GDN_BF16;
  const bool al = (int64_t)a.C * (bf16 ? 2 : 4) % 16 == 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GDN_ERR_CUDA;
  if (!know_device(dev)) return GDN_ERR_CUDA;
  const int groups = (a.C + kChan - 1) / kChan;
  Choice c = choose(dev, a, al, bwd ? kBwd8 : kFwd8, groups);
  const Choice small = choose(dev, a, al, bwd ? kBwd4 : kFwd4, groups);
  if (small.cluster != 0 && (c.cluster == 0 || small.cost < c.cost)) c = small;
  if (c.cluster == 0) return GDN_ERR_CUDA;
  const Scan& k = c.scan;
  ScanMaps maps = {};
  if (a.total_T > 0) {
    // (the order in which the kernels number their tensors)
    const bool beta = a.gate == kGateBeta;
    const void* in[4] = {a.x, a.log_alpha, beta ? a.beta : a.dy, a.dy};
    const void* out[3] = {bwd ? a.dx : a.y, a.dlog_alpha, a.dbeta};
    const int n_in = 2 + (beta ? 1 : 0) + (bwd ? 1 : 0);
    const int n_out = !al ? 0 : bwd ? n_in - 1 : a.y != nullptr ? 1 : 0;
    for (int i = 0; i < n_in; ++i)
      if (!encode_map(&maps.in[i], a, in[i], k.rows, al)) return GDN_ERR_CUDA;
    for (int i = 0; i < n_out; ++i)
      if (!encode_map(&maps.out[i], a, out[i], k.rows, al)) return GDN_ERR_CUDA;
  }
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = scan_config(k, c.cluster, c.smem, groups, stream, &attr);
  return launch_status(cudaLaunchKernelEx(&cfg, k.kernel, a, maps));
}

template <typename Tin>
gdn_status launch_step(const GlrArgs& a, int64_t n, cudaStream_t stream) {
  void (*kernel)(const Tin*, const Tin*, const Tin*, float*, Tin*, int64_t) =
      a.gate == kGateNone   ? glr_step_kernel<Tin, kGateNone>
      : a.gate == kGateBeta ? glr_step_kernel<Tin, kGateBeta>
                            : glr_step_kernel<Tin, kGateComp>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n + 8 * 256 - 1) / (8 * 256)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  return launch_status(cudaLaunchKernelEx(
      &cfg, kernel, static_cast<const Tin*>(a.x), static_cast<const Tin*>(a.log_alpha),
      static_cast<const Tin*>(a.beta), a.final_state, static_cast<Tin*>(a.y), n));
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
