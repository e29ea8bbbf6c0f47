// gated.cuh -- what the gated linear recurrence's kernels share.
//
// Per (batch, KV head), with a log decay g_t per token and a 64 x 64 state:
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,      y_t = scale S_t^T q_t.
// With G the sums of g inside a chunk of 64 tokens, S_in the state before it:
//     y_i   = scale [ sum_{j<=i} e^{G_i-G_j} (q_i.k_j) v_j + e^{G_i} S_in^T q_i ]
//     S_out = e^{G_63} S_in + sum_j e^{G_63-G_j} k_j v_j^T.
// A sequence is cut into segments of whole chunks: the segments' own states
// are formed side by side, a scan turns them into the state before each
// segment, and a last pass walks every segment from there.
#pragma once
#include <math.h>

#include "oal_internal.cuh"

namespace oal {

constexpr int kGC = 64;                 // tokens of a chunk
constexpr int kGS = kD * kDv;           // elements of a state
// exp(g) is 0 in fp32 from here down, so such a gate starts from nothing like
// -inf does; it is counted instead of summed, which keeps the sums small.
constexpr float kGateCut = -104.f;

// A decay over a token, a chunk or a segment, e^x, as an unevaluated sum
// hi + lo.  Many of them in a row multiply a state, and a slow gate's lie next
// to 1, where half a step of fp32 is 2^-25: under a constant gate it would be
// the same one each time, and grow with their number instead of its root
// (4096 chunks: 6e-5 of the state, with the pair 5e-7).  From |x| = 0.5 on a
// state is forgotten before that shows, and lo is 0.
struct GateDecay {
  float hi, lo;
};
__device__ __forceinline__ GateDecay decay_exp(float x) {
  const float hi = expf(x);
  return {hi, fabsf(x) < 0.5f ? expm1f(x) - (hi - 1.f) : 0.f};
}
// (lo may outgrow half a step of hi; not renormalised, a row of these is as deep
// as one of plain products)
__device__ __forceinline__ GateDecay decay_mul(GateDecay a, GateDecay b) {
  const float p = a.hi * b.hi;
  return {p, fmaf(a.lo, b.hi, fmaf(a.hi, b.lo, fmaf(a.hi, b.hi, -p)))};
}
// f s + d.  A decay of 0 (a cut gate) shuts out whatever s is, NaN and
// infinities too.
__device__ __forceinline__ float decay_add(GateDecay f, float s, float d) {
  s = __uint_as_float(__float_as_uint(s) & (f.hi == 0.f ? 0u : ~0u));   // (a select would become a branch)
  return fmaf(f.hi, s, fmaf(f.lo, s, d));
}
// The same for a factor by itself.
__device__ __forceinline__ float decay_by(float f, float x) { return f == 0.f ? 0.f : f * x; }

struct GatedArgs {
  const void *Q, *K, *V, *dY;
  const float *g;
  int B, Hq, Hkv, T;
  float scale;
  const int32_t *lengths;               // null: every sequence has T tokens
  const float *state_in;                // state before token 0, null: zeros
  float *state_out;                     // prefill: state after the last token
  void *Y;
  const float *dstate;                  // backward: gradient of the last state, null: zeros
  float *dstate0;                       // backward: gradient of state_in, may be null
  void *dQ, *dK, *dV;
  float *dg;
  int seg_chunks, nseg;                 // chunks of a segment, segments of T tokens
  float *seg_state;                     // [B Hkv][nseg][64 64]
  GateDecay *seg_decay;                 // [B Hkv][nseg]
  float *seg_grad;                      // backward: the same for the state's gradient
  int *status;
};

// Segment sizes in chunks (gated_simt.cu), and how many of them T tokens have.
int gated_prefill_segment(int B, int Hkv, int T);
inline int gated_segments(int T, int seg_chunks) {
  const int chunks = (int)(((long long)T + kGC - 1) / kGC);
  return (chunks + seg_chunks - 1) / seg_chunks;
}

// Kernels above 48 KB of shared memory ask for it once per device.
oal_status gated_need_smem(const void *kernel, size_t bytes, bool (&done)[kMaxDevices]);

// Length of sequence b, clamped to 0..T; one outside is recorded.
__device__ __forceinline__ int gated_len(const GatedArgs &p, int b) {
  if (!p.lengths) return p.T;
  const int n = p.lengths[b];
  if (n < 0 || n > p.T) {
    if (threadIdx.x == 0) atomicCAS(p.status, kStatusOk, (int)OAL_ERR_INVALID_ARG);
    return n < 0 ? 0 : p.T;
  }
  return n;
}
__device__ __forceinline__ int gated_last_seg(int n, int seg_tokens) {
  return n > 0 ? (n - 1) / seg_tokens : 0;
}

// Sums of g inside a chunk: the sum as an unevaluated pair hi + lo, so the
// difference of two neighbours keeps its digits behind a large drop, and the
// gates cut so far, which are left out of the sum.
struct __align__(16) GateSums {
  float hi[kGC], lo[kGC];
  int cuts[kGC];
};

__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
  s = a + b;
  const float t = s - a;
  e = (a - (s - t)) + (b - t);
}

// The same held by a warp: lane l has tokens 2l and 2l + 1.
struct GateLane {
  float hi[2], lo[2];
  int cuts[2];
};

// Gates of lane l's tokens of the chunk at t0; rows from n on count as gates
// of 1 (g = 0).
__device__ __forceinline__ float2 gate_load(const float *__restrict__ g, int t0, int n) {
  const int t = t0 + 2 * (threadIdx.x & 31);
  return make_float2(t < n ? __ldg(g + t) : 0.f, t + 1 < n ? __ldg(g + t + 1) : 0.f);
}

__device__ __forceinline__ GateLane gate_sums(float2 x) {
  const int lane = threadIdx.x & 31;
  const int c0 = x.x <= kGateCut, c1 = x.y <= kGateCut;
  const float a = c0 ? 0.f : x.x, b = c1 ? 0.f : x.y;
  float hi, lo;
  two_sum(a, b, hi, lo);
  int cuts = c0 + c1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float oh = __shfl_up_sync(0xffffffffu, hi, d), ol = __shfl_up_sync(0xffffffffu, lo, d);
    const int oc = __shfl_up_sync(0xffffffffu, cuts, d);
    if (lane >= d) {
      float s, e;
      two_sum(oh, hi, s, e);
      e += ol + lo;
      hi = s + e;
      lo = e - (hi - s);
      cuts += oc;
    }
  }
  float ph = __shfl_up_sync(0xffffffffu, hi, 1), pl = __shfl_up_sync(0xffffffffu, lo, 1);
  int pc = __shfl_up_sync(0xffffffffu, cuts, 1);
  if (lane == 0) ph = pl = 0.f, pc = 0;
  float s, e;
  two_sum(ph, a, s, e);
  e += pl;
  GateLane out;
  out.hi[0] = s + e;
  out.lo[0] = e - (out.hi[0] - s);
  out.cuts[0] = pc + c0;
  out.hi[1] = hi;
  out.lo[1] = lo;
  out.cuts[1] = cuts;
  return out;
}
__device__ __forceinline__ void gate_store(const GateLane &x, GateSums &out) {
  const int l = threadIdx.x & 31;
  *reinterpret_cast<float2 *>(&out.hi[2 * l]) = make_float2(x.hi[0], x.hi[1]);
  *reinterpret_cast<float2 *>(&out.lo[2 * l]) = make_float2(x.lo[0], x.lo[1]);
  *reinterpret_cast<int2 *>(&out.cuts[2 * l]) = make_int2(x.cuts[0], x.cuts[1]);
}

// exp(x) where `on`, else 0, without a branch: a row of these under branches
// runs one after another (32 of them: 8,000 cycles instead of 300).
__device__ __forceinline__ float gate_exp(bool on, float x) { return expf(on ? x : -INFINITY); }
__device__ __forceinline__ float gate_exp_fast(bool on, float x) { return __expf(on ? x : -INFINITY); }

// Decay between tokens j <= i of the chunk, exp(G_i - G_j).
__device__ __forceinline__ float gate_pair(const GateSums &s, int i, int j) {
  return gate_exp(s.cuts[i] == s.cuts[j], (s.hi[i] - s.hi[j]) + (s.lo[i] - s.lo[j]));
}
// Decay from the chunk's start to token i, exp(G_i).
__device__ __forceinline__ float gate_head(const GateSums &s, int i) {
  return gate_exp(s.cuts[i] == 0, s.hi[i] + s.lo[i]);
}
// Decay over the chunk.
__device__ __forceinline__ GateDecay gate_whole(const GateSums &s) {
  return decay_exp(s.cuts[kGC - 1] == 0 ? s.hi[kGC - 1] + s.lo[kGC - 1] : -INFINITY);
}
// Decay from behind token j to the chunk's end, exp(G_63 - G_j).
__device__ __forceinline__ float gate_tail(const GateSums &s, int j) {
  return gate_pair(s, kGC - 1, j);
}

// The walk over a sequence's segments (chunks in the backward): a thread takes
// kVec values of the state and has the loads of kAhead segments in flight,
// which is all that hides the walk's own chain.  put(i, run) gets the value
// before segment i (walking back: behind it).
template <int kVec>
struct ScanVec {
  float v[kVec];
};
template <int kVec>
__device__ __forceinline__ ScanVec<kVec> scan_load(const float *p) {
  ScanVec<kVec> r;
  if (kVec == 4) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    r.v[0] = x.x, r.v[1] = x.y, r.v[kVec - 2] = x.z, r.v[kVec - 1] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2 *>(p);
    r.v[0] = x.x, r.v[1] = x.y;
  }
  return r;
}
template <int kVec>
__device__ __forceinline__ void scan_store(float *p, const ScanVec<kVec> &r) {
  if (kVec == 4) *reinterpret_cast<float4 *>(p) = make_float4(r.v[0], r.v[1], r.v[kVec - 2], r.v[kVec - 1]);
  else *reinterpret_cast<float2 *>(p) = make_float2(r.v[0], r.v[1]);
}
// own: the thread's values of segment 0's own state; count segments, of which
// the first `formed` in walking order have one; back: from the last to the first.
template <int kVec, int kAhead, typename Put>
__device__ __forceinline__ ScanVec<kVec> scan_walk(const float *own, const GateDecay *decay, const float *from, int count,
                                                   int formed, bool back, Put put) {
  ScanVec<kVec> run = {};
  if (from) run = scan_load<kVec>(from);
  for (int i0 = 0; i0 < count; i0 += kAhead) {
    ScanVec<kVec> v[kAhead];
    GateDecay f[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = back ? count - 1 - i0 - k : i0 + k;
      v[k] = {};
      f[k] = {};
      if (i0 + k < formed) v[k] = scan_load<kVec>(own + (size_t)i * kGS), f[k] = decay[i];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k < count) {
        put(back ? count - 1 - i0 - k : i0 + k, run);
#pragma unroll
        for (int e = 0; e < kVec; ++e) run.v[e] = decay_add(f[k], run.v[e], v[k].v[e]);
      }
  }
  return run;
}
// The same walk by kChains threads a value, each over kAhead segments of a
// round at a time: its part's decay and sum first, then, from the parts before
// it, the states.  All of a round's loads are in flight together.  The threads
// of a block are kChains groups of kScanThreads / kChains; all get the result.
constexpr int kScanThreads = 128;
template <int kVec, int kAhead, int kChains, typename Put>
__device__ __forceinline__ ScanVec<kVec> scan_split(const float *own, const GateDecay *decay, const float *from, int count,
                                                    int formed, bool back, Put put) {
  constexpr int kLanes = kScanThreads / kChains;
  __shared__ GateDecay s_decay[kChains];
  __shared__ ScanVec<kVec> s_sum[kChains][kLanes];
  const int chain = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  ScanVec<kVec> run = {};
  if (from) run = scan_load<kVec>(from);
  for (int i0 = 0; i0 < count; i0 += kAhead * kChains) {
    const int first = i0 + chain * kAhead;
    ScanVec<kVec> v[kAhead], sum = {};
    GateDecay f[kAhead], all = {1.f, 0.f};
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = back ? count - 1 - first - k : first + k;
      v[k] = {};
      f[k] = {1.f, 0.f};
      if (first + k < formed) v[k] = scan_load<kVec>(own + (size_t)i * kGS), f[k] = decay[i];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) sum.v[e] = decay_add(f[k], sum.v[e], v[k].v[e]);
      all = decay_mul(all, f[k]);
    }
    __syncthreads();
    if (lane == 0) s_decay[chain] = all;
    s_sum[chain][lane] = sum;
    __syncthreads();
    ScanVec<kVec> in = run;
#pragma unroll
    for (int z = 0; z < kChains; ++z) {
      if (z == chain) in = run;
      const ScanVec<kVec> part = s_sum[z][lane];
#pragma unroll
      for (int e = 0; e < kVec; ++e) run.v[e] = decay_add(s_decay[z], run.v[e], part.v[e]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (first + k < count) {
        put(back ? count - 1 - first - k : first + k, in);
#pragma unroll
        for (int e = 0; e < kVec; ++e) in.v[e] = decay_add(f[k], in.v[e], v[k].v[e]);
      }
  }
  return run;
}
// Few states and many segments: the split walk (205 segments of 2 states: 7 us;
// one thread a value took 16 with 32 loads ahead, 22 with 8, when this one took
// 8); otherwise the states' own number fills the GPU.
inline bool scan_deep(int states, int segments) { return states <= 16 && segments > 16; }
constexpr int kScanChains = 8;

}  // namespace oal

#define GATED_TRY(x)             \
  do {                           \
    const oal_status _s = (x);   \
    if (_s != OAL_OK) return _s; \
  } while (0)
