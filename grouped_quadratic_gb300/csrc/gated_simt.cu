// gated_simt.cu -- the gated linear recurrence on the CUDA cores in fp32:
// the segments' states, the scan over segments, the outputs, the backward.
//
// A block of 256 threads works on 64 x 64 tiles in shared memory; a thread
// owns rows 4 ty .. 4 ty + 3 and columns tx, tx + 16, tx + 32, tx + 48 of a
// product, so a warp's reads of the left tile are broadcasts and those of the
// right tile meet no bank twice (pitch 68: four words past a row of 64).
// fp32 inputs only.  Bound by the latency of a chunk where there are few: 32 us
// for 2 x 777 tokens of 4 heads in three launches, 44 us for the backward of
// 2 x 513 tokens, 4/2 heads; by the fp32 pipes where there are many.
#include <algorithm>

#include "gated.cuh"

namespace oal {
namespace {

constexpr int kThreads = 256;
constexpr int kP = 68;                   // pitch of a tile row, floats
constexpr int kTile = kGC * kP;

struct Acc {
  float v[4][4];
};

__device__ __forceinline__ void clear(Acc &a) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) a.v[i][j] = 0.f;
}

// out[i][j] += sum_k A[i][k] B[j][k]
__device__ __forceinline__ void mm_nt(const float *A, const float *B, int ty, int tx, Acc &o) {
#pragma unroll 4
  for (int k = 0; k < 64; k += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * kP + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * kP + k);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o.v[i][j] = fmaf(a[i].x, b[j].x, o.v[i][j]);
        o.v[i][j] = fmaf(a[i].y, b[j].y, o.v[i][j]);
        o.v[i][j] = fmaf(a[i].z, b[j].z, o.v[i][j]);
        o.v[i][j] = fmaf(a[i].w, b[j].w, o.v[i][j]);
      }
  }
}
// out[i][j] += sum_k A[i][k] B[k][j]
__device__ __forceinline__ void mm_nn(const float *A, const float *B, int ty, int tx, Acc &o) {
#pragma unroll 4
  for (int k = 0; k < 64; k += 4) {
    float a[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * kP + k);
      a[i][0] = t.x, a[i][1] = t.y, a[i][2] = t.z, a[i][3] = t.w;
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float b = B[(k + kk) * kP + tx + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i) o.v[i][j] = fmaf(a[i][kk], b, o.v[i][j]);
      }
  }
}
// out[i][j] += sum_k w[k] A[k][i] B[k][j]
__device__ __forceinline__ void mm_tn(const float *A, const float *B, const float *w, int ty, int tx, Acc &o) {
#pragma unroll 4
  for (int k = 0; k < 64; ++k) {
    float4 t = *reinterpret_cast<const float4 *>(A + k * kP + 4 * ty);
    if (w) {
      const float f = w[k];
      t.x *= f, t.y *= f, t.z *= f, t.w *= f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float b = B[k * kP + tx + 16 * j];
      o.v[0][j] = fmaf(t.x, b, o.v[0][j]);
      o.v[1][j] = fmaf(t.y, b, o.v[1][j]);
      o.v[2][j] = fmaf(t.z, b, o.v[2][j]);
      o.v[3][j] = fmaf(t.w, b, o.v[3][j]);
    }
  }
}

// Rows t0 .. t0 + 63 of a [T][64] matrix into a tile; rows from n on are 0.
__device__ __forceinline__ void load_tile(const float *src, int t0, int n, float *tile) {
  float4 v[4];
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int x = threadIdx.x + it * kThreads, r = x >> 4, c = (x & 15) * 4;
    v[it] = t0 + r < n ? __ldg(reinterpret_cast<const float4 *>(src + (size_t)(t0 + r) * 64 + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int x = threadIdx.x + it * kThreads, r = x >> 4, c = (x & 15) * 4;
    *reinterpret_cast<float4 *>(tile + r * kP + c) = v[it];
  }
}
__device__ __forceinline__ void load_state(const float *src, float *tile) {
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int x = threadIdx.x + it * kThreads, r = x >> 4, c = (x & 15) * 4;
    *reinterpret_cast<float4 *>(tile + r * kP + c) =
        src ? *reinterpret_cast<const float4 *>(src + r * 64 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}
__device__ __forceinline__ void put(const Acc &a, int ty, int tx, float *tile) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) tile[(4 * ty + i) * kP + tx + 16 * j] = a.v[i][j];
}
__device__ __forceinline__ void store_rows(const Acc &a, int ty, int tx, float *dst, int t0, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t0 + 4 * ty + i < n)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        dst[(size_t)(t0 + 4 * ty + i) * 64 + tx + 16 * j] = a.v[i][j];
}

// The decays of a chunk that every thread reads.
struct Decays {
  GateSums sums;
  float head[kGC], tail[kGC];
  GateDecay whole;
};
// (`gate` as warp 0 loaded it, early, so that its way to memory is not in
// front of the tiles')
__device__ __forceinline__ void chunk_decays(float2 gate, Decays &d) {
  if (threadIdx.x < 32) gate_store(gate_sums(gate), d.sums);
  __syncthreads();
  if (threadIdx.x < kGC) {
    d.head[threadIdx.x] = gate_head(d.sums, threadIdx.x);
    d.tail[threadIdx.x] = gate_tail(d.sums, threadIdx.x);
  }
  if (threadIdx.x == kGC) d.whole = gate_whole(d.sums);
  __syncthreads();
}

// Own state of each segment but a sequence's last (y = 0), or, for the
// backward, own gradient of the state before each segment but the first
// (y = 1):  sum_i e^{G_i} scale q_i dy_i^T over the segment's tokens and the
// query heads of the KV head.
__global__ void __launch_bounds__(kThreads) gated_segment_kernel(GatedArgs p) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ float4 smem4[];
  float *A = reinterpret_cast<float *>(smem4), *B = A + kTile;
  __shared__ Decays dec;
  const int bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg, b = bh / p.Hkv, kv = bh % p.Hkv;
  const int rho = p.Hq / p.Hkv, n = gated_len(p, b);
  const int last = gated_last_seg(n, p.seg_chunks * kGC);
  const bool grad = blockIdx.y != 0;
  if (grad ? seg > last : seg >= last) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const float *g = p.g + (size_t)bh * p.T;
  const int c0 = seg * p.seg_chunks, c1 = min((n + kGC - 1) / kGC, c0 + p.seg_chunks);
  Acc acc;
  clear(acc);
  __shared__ GateDecay decay;                 // (the first thread's)
  if (threadIdx.x == 0) decay = {1.f, 0.f};
  for (int s = 0; s < c1 - c0; ++s) {
    const int t0 = (grad ? c1 - 1 - s : c0 + s) * kGC;
    const float2 gate = gate_load(g, t0, n);
    __syncthreads();
    if (!grad) {
      load_tile(static_cast<const float *>(p.K) + (size_t)bh * p.T * 64, t0, n, A);
      load_tile(static_cast<const float *>(p.V) + (size_t)bh * p.T * 64, t0, n, B);
    } else {
      load_tile(static_cast<const float *>(p.Q) + ((size_t)b * p.Hq + kv * rho) * p.T * 64, t0, n, A);
      load_tile(static_cast<const float *>(p.dY) + ((size_t)b * p.Hq + kv * rho) * p.T * 64, t0, n, B);
    }
    chunk_decays(gate, dec);
    const GateDecay whole = dec.whole;
    if (threadIdx.x == 0) decay = decay_mul(decay, whole);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc.v[i][j] = decay_add(whole, acc.v[i][j], 0.f);
    if (!grad) {
      mm_tn(A, B, dec.tail, ty, tx, acc);
    } else {
      if (threadIdx.x < kGC) dec.tail[threadIdx.x] = p.scale * dec.head[threadIdx.x];
      for (int r = 0; r < rho; ++r) {
        const size_t row = ((size_t)b * p.Hq + kv * rho + r) * p.T * 64;
        __syncthreads();
        if (r > 0) {
          load_tile(static_cast<const float *>(p.Q) + row, t0, n, A);
          load_tile(static_cast<const float *>(p.dY) + row, t0, n, B);
          __syncthreads();
        }
        mm_tn(A, B, dec.tail, ty, tx, acc);
      }
    }
  }
  float *out = (grad ? p.seg_grad : p.seg_state) + ((size_t)bh * p.nseg + seg) * kGS;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) out[(4 * ty + i) * 64 + tx + 16 * j] = acc.v[i][j];
  if (threadIdx.x == 0 && (grad || gridDim.y == 1)) p.seg_decay[(size_t)bh * p.nseg + seg] = decay;
}

// z = 0: own states -> the state before each segment, forwards.  z = 1: own
// gradients -> the gradient of the state behind each segment, backwards, and
// dstate0.  In place.  kLast: the last segment has its own state too, and the
// state behind it is the result.
template <int kVec, int kAhead, int kChains, bool kLast>
__global__ void __launch_bounds__(kScanThreads) gated_scan_kernel(GatedArgs p) {
  pdl_trigger();
  pdl_wait();
  constexpr int kLanes = kScanThreads / kChains;
  const int bh = blockIdx.x, x = kVec * (blockIdx.y * kLanes + threadIdx.x % kLanes);
  const int n = gated_len(p, bh / p.Hkv), last = gated_last_seg(n, p.seg_chunks * kGC);
  const bool grad = blockIdx.z != 0;
  float *s = (grad ? p.seg_grad : p.seg_state) + (size_t)bh * p.nseg * kGS + x;
  const float *from = grad ? p.dstate : p.state_in;
  const GateDecay *decay = p.seg_decay + (size_t)bh * p.nseg;
  if (from) from += (size_t)bh * kGS + x;
  const int count = grad && n == 0 ? 0 : last + 1, formed = grad || kLast ? count : last;
  auto put = [&](int i, const ScanVec<kVec> &v) { scan_store(s + (size_t)i * kGS, v); };
  ScanVec<kVec> run;
  if constexpr (kChains == 1) run = scan_walk<kVec, kAhead>(s, decay, from, count, formed, grad, put);
  else run = scan_split<kVec, kAhead, kChains>(s, decay, from, count, formed, grad, put);
  if (threadIdx.x >= kLanes) return;
  if (grad && p.dstate0) scan_store(p.dstate0 + (size_t)bh * kGS + x, run);
  if (!grad && kLast) scan_store(p.state_out + (size_t)bh * kGS + x, run);
}

// Outputs of a segment, and the state behind the sequence's last one.
__global__ void __launch_bounds__(kThreads) gated_out_kernel(GatedArgs p) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ float4 smem4[];
  float *Q = reinterpret_cast<float *>(smem4), *K = Q + kTile, *V = K + kTile, *P = V + kTile, *S = P + kTile;
  __shared__ Decays dec;
  const int bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg, b = bh / p.Hkv, kv = bh % p.Hkv;
  const int rho = p.Hq / p.Hkv, n = gated_len(p, b);
  const int last = gated_last_seg(n, p.seg_chunks * kGC);
  if (seg > last) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const float *g = p.g + (size_t)bh * p.T;
  load_state(p.nseg > 1 ? p.seg_state + ((size_t)bh * p.nseg + seg) * kGS
                        : p.state_in ? p.state_in + (size_t)bh * kGS : nullptr, S);
  const int c0 = seg * p.seg_chunks, c1 = min((n + kGC - 1) / kGC, c0 + p.seg_chunks);
  for (int c = c0; c < c1; ++c) {
    const int t0 = c * kGC;
    const float2 gate = gate_load(g, t0, n);
    __syncthreads();
    load_tile(static_cast<const float *>(p.K) + (size_t)bh * p.T * 64, t0, n, K);
    load_tile(static_cast<const float *>(p.Q) + ((size_t)b * p.Hq + kv * rho) * p.T * 64, t0, n, Q);
    load_tile(static_cast<const float *>(p.V) + (size_t)bh * p.T * 64, t0, n, V);
    chunk_decays(gate, dec);
    float pair[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        pair[i][j] = gate_pair(dec.sums, 4 * ty + i, min(tx + 16 * j, 4 * ty + i));
    for (int r = 0; r < rho; ++r) {
      const size_t row = ((size_t)b * p.Hq + kv * rho + r) * p.T * 64;
      if (r > 0) {
        __syncthreads();
        load_tile(static_cast<const float *>(p.Q) + row, t0, n, Q);
        __syncthreads();
      }
      Acc a;
      clear(a);
      mm_nt(Q, K, ty, tx, a);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) a.v[i][j] = tx + 16 * j <= 4 * ty + i ? a.v[i][j] * pair[i][j] : 0.f;
      put(a, ty, tx, P);
      clear(a);
      mm_nn(Q, S, ty, tx, a);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) a.v[i][j] = decay_by(dec.head[4 * ty + i], a.v[i][j]);
      __syncthreads();
      mm_nn(P, V, ty, tx, a);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) a.v[i][j] *= p.scale;
      store_rows(a, ty, tx, static_cast<float *>(p.Y) + row, t0, n);
    }
    Acc s;
    const GateDecay whole = dec.whole;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s.v[i][j] = decay_add(whole, S[(4 * ty + i) * kP + tx + 16 * j], 0.f);
    mm_tn(K, V, dec.tail, ty, tx, s);
    __syncthreads();
    put(s, ty, tx, S);
  }
  if (seg == last) {
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int x = threadIdx.x + it * kThreads, r = x >> 4, c = (x & 15) * 4;
      *reinterpret_cast<float4 *>(p.state_out + (size_t)bh * kGS + r * 64 + c) =
          *reinterpret_cast<const float4 *>(S + r * kP + c);
    }
  }
}

// Gradients of one chunk (segments of one chunk): with pair_ij = e^{G_i-G_j},
// R the gradient of the state behind the chunk,
//   z_ij = scale pair_ij dy_i.v_j, p_ij = pair_ij q_i.k_j,
//   dq_i = sum_j z_ij k_j + scale e^{G_i} S_in dy_i
//   dk_j = sum_i z_ij q_i + e^{G_63-G_j} R v_j
//   dv_j = scale sum_i p_ij dy_i + e^{G_63-G_j} R^T k_j
//   dg_t = sum_{j<t<=l} w_lj + sum_{l>=t} q_l.dq_l' + sum_{j<t} k_j.dk_j' + e^{G_63} <S_in, R>
// with w = p scale dy.v, and dq', dk' the terms with S_in and R: every path
// from a token before t to one at or behind t decays by exp(g_t).
__global__ void __launch_bounds__(kThreads) gated_grad_kernel(GatedArgs p) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ float4 smem4[];
  float *Q = reinterpret_cast<float *>(smem4), *K = Q + kTile, *V = K + kTile, *O = V + kTile;
  float *P = O + kTile, *Z = P + kTile, *S = Z + kTile, *R = S + kTile;
  __shared__ Decays dec;
  __shared__ float s_row[kGC], s_far[kGC], s_col[16][kGC], s_dot[kThreads / 32];
  const int bh = blockIdx.x / p.nseg, c = blockIdx.x % p.nseg, b = bh / p.Hkv, kv = bh % p.Hkv;
  const int rho = p.Hq / p.Hkv, n = gated_len(p, b), t0 = c * kGC;
  if (t0 >= n) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const size_t kvrow = (size_t)bh * p.T * 64;
  const float2 gate = gate_load(p.g + (size_t)bh * p.T, t0, n);
  load_tile(static_cast<const float *>(p.K) + kvrow, t0, n, K);
  load_tile(static_cast<const float *>(p.V) + kvrow, t0, n, V);
  load_tile(static_cast<const float *>(p.Q) + ((size_t)b * p.Hq + kv * rho) * p.T * 64, t0, n, Q);
  load_tile(static_cast<const float *>(p.dY) + ((size_t)b * p.Hq + kv * rho) * p.T * 64, t0, n, O);
  load_state(p.seg_state + ((size_t)bh * p.nseg + c) * kGS, S);
  load_state(p.seg_grad + ((size_t)bh * p.nseg + c) * kGS, R);
  chunk_decays(gate, dec);
  float pair[4][4], w[4][4], rows[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      pair[i][j] = gate_pair(dec.sums, 4 * ty + i, min(tx + 16 * j, 4 * ty + i));
      w[i][j] = 0.f;
    }
  Acc dK, dV;
  clear(dK);
  clear(dV);
  for (int r = 0; r < rho; ++r) {
    const size_t row = ((size_t)b * p.Hq + kv * rho + r) * p.T * 64;
    if (r > 0) {
      __syncthreads();
      load_tile(static_cast<const float *>(p.Q) + row, t0, n, Q);
      load_tile(static_cast<const float *>(p.dY) + row, t0, n, O);
      __syncthreads();
    }
    Acc a, z;
    clear(a);
    clear(z);
    mm_nt(Q, K, ty, tx, a);
    mm_nt(O, V, ty, tx, z);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row_i = 4 * ty + i, col_j = tx + 16 * j;
        const bool on = col_j <= row_i;
        a.v[i][j] = on ? p.scale * pair[i][j] * a.v[i][j] : 0.f;
        if (col_j < row_i) w[i][j] = fmaf(a.v[i][j], z.v[i][j], w[i][j]);
        z.v[i][j] = on ? p.scale * pair[i][j] * z.v[i][j] : 0.f;
      }
    put(a, ty, tx, P);
    put(z, ty, tx, Z);
    clear(a);
    mm_nt(O, S, ty, tx, a);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a.v[i][j] = decay_by(p.scale * dec.head[4 * ty + i], a.v[i][j]);
        rows[i] = fmaf(a.v[i][j], Q[(4 * ty + i) * kP + tx + 16 * j], rows[i]);
      }
    __syncthreads();
    mm_nn(Z, K, ty, tx, a);
    store_rows(a, ty, tx, static_cast<float *>(p.dQ) + row, t0, n);
    mm_tn(P, O, nullptr, ty, tx, dV);
    mm_tn(Z, Q, nullptr, ty, tx, dK);
  }
  Acc a;
  clear(a);
  mm_nt(V, R, ty, tx, a);
  float far[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a.v[i][j] = decay_by(dec.tail[4 * ty + i], a.v[i][j]);
      far[i] = fmaf(a.v[i][j], K[(4 * ty + i) * kP + tx + 16 * j], far[i]);
      dK.v[i][j] += a.v[i][j];
    }
  clear(a);
  mm_nn(K, R, ty, tx, a);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dV.v[i][j] += decay_by(dec.tail[4 * ty + i], a.v[i][j]);
  store_rows(dK, ty, tx, static_cast<float *>(p.dK) + kvrow, t0, n);
  store_rows(dV, ty, tx, static_cast<float *>(p.dV) + kvrow, t0, n);

  // dg: row and column sums of w, the far terms and <S_in, R>
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      dot = fmaf(S[(4 * ty + i) * kP + tx + 16 * j], R[(4 * ty + i) * kP + tx + 16 * j], dot);
#pragma unroll
  for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if ((threadIdx.x & 31) == 0) s_dot[threadIdx.x >> 5] = dot;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x = rows[i] + (w[i][0] + w[i][1]) + (w[i][2] + w[i][3]), y = far[i];
#pragma unroll
    for (int d = 8; d; d >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, d);
      y += __shfl_xor_sync(0xffffffffu, y, d);
    }
    if (tx == 0) s_row[4 * ty + i] = x, s_far[4 * ty + i] = y;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_col[ty][tx + 16 * j] = (w[0][j] + w[1][j]) + (w[2][j] + w[3][j]);
  __syncthreads();
  if (threadIdx.x < kGC) {
    float x = s_row[threadIdx.x];
#pragma unroll
    for (int k = 0; k < 16; ++k) x -= s_col[k][threadIdx.x];
    s_row[threadIdx.x] = x;
  }
  __syncthreads();
  if (threadIdx.x < kGC && t0 + threadIdx.x < n) {
    const int t = threadIdx.x;
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) x += s_dot[k];
    x = decay_by(dec.whole.hi, x);
    for (int l = kGC - 1; l >= t; --l) x += s_row[l];
    for (int j = 0; j < t; ++j) x += s_far[j];
    const bool cut = dec.sums.cuts[t] != (t ? dec.sums.cuts[t - 1] : 0);
    p.dg[(size_t)bh * p.T + t0 + t] = cut ? 0.f : x;
  }
}

}  // namespace

oal_status gated_need_smem(const void *kernel, size_t bytes, bool (&done)[kMaxDevices]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return oal_fail(OAL_ERR_CUDA, "no current device");
  if (done[dev]) return OAL_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
    return oal_check_launch("shared memory of a gated kernel");
  done[dev] = true;
  return OAL_OK;
}

// As many segments as give three blocks per SM one wave: what is resident in
// the bf16 output kernel.  Blocks a segment at 2, 2.5, 3, 4 and 6 per SM, us:
// 4 x 32/8 heads x 8192 tokens 97, 92, 84, 95, 87; 65536 tokens 77, 76, 68,
// 84, 76; 4 x 16/16 x 4096 75, 73, 63, 70, 66; 8 x 32/8 x 512 20, 20, 20, 23,
// 23.  Fewer lose more (1 per SM 164, 112, 107, 25).  Only small ragged
// batches gain from more (14/2 heads, 201 tokens: 28 -> 25 with 4).  (The fp32
// kernel, of which two fit an SM, goes by the same rule; it was not measured.)
int gated_prefill_segment(int B, int Hkv, int T) {
  const long long units = (long long)B * Hkv, chunks = ((long long)T + kGC - 1) / kGC;
  const long long want = std::max<long long>(1, 3 * 152 / units);
  return (int)std::max<long long>(1, (chunks + want - 1) / want);
}
template <bool kLast>
static oal_status launch_scan(const GatedArgs &p, int ways, cudaStream_t stream) {
  const int units = p.B * p.Hkv;
  if (scan_deep(units * ways, p.nseg))
    launch_pdl(gated_scan_kernel<2, 32, kScanChains, kLast>, dim3(units, kGS / 2 * kScanChains / kScanThreads, ways),
               dim3(kScanThreads), 0, stream, p);
  else
    launch_pdl(gated_scan_kernel<4, 8, 1, kLast>, dim3(units, kGS / 4 / kScanThreads, ways), dim3(kScanThreads), 0, stream, p);
  return oal_after_launch("gated_scan_kernel", stream);
}
// From the segments' own states to those before them and (last) the one behind
// the last of them; with two ways, the gradients too.
oal_status launch_gated_scan(const GatedArgs &p, int ways, bool last, cudaStream_t stream) {
  return last ? launch_scan<true>(p, ways, stream) : launch_scan<false>(p, ways, stream);
}

oal_status launch_gated_prefill_simt(const GatedArgs &p, cudaStream_t stream) {
  static bool done_seg[kMaxDevices], done_out[kMaxDevices];
  const size_t seg_smem = 2 * kTile * sizeof(float), out_smem = 5 * kTile * sizeof(float);
  GATED_TRY(gated_need_smem(reinterpret_cast<const void *>(gated_segment_kernel), seg_smem, done_seg));
  GATED_TRY(gated_need_smem(reinterpret_cast<const void *>(gated_out_kernel), out_smem, done_out));
  if (p.nseg > 1) {
    launch_pdl(gated_segment_kernel, dim3(p.nseg * p.B * p.Hkv), dim3(kThreads), seg_smem, stream, p);
    GATED_TRY(oal_after_launch("gated_segment_kernel", stream));
    GATED_TRY(launch_scan<false>(p, 1, stream));
  }
  launch_pdl(gated_out_kernel, dim3(p.nseg * p.B * p.Hkv), dim3(kThreads), out_smem, stream, p);
  return oal_after_launch("gated_out_kernel", stream);
}

oal_status launch_gated_backward_simt(const GatedArgs &p, cudaStream_t stream) {
  static bool done_seg[kMaxDevices], done_grad[kMaxDevices];
  const size_t seg_smem = 2 * kTile * sizeof(float), grad_smem = 8 * kTile * sizeof(float);
  GATED_TRY(gated_need_smem(reinterpret_cast<const void *>(gated_segment_kernel), seg_smem, done_seg));
  GATED_TRY(gated_need_smem(reinterpret_cast<const void *>(gated_grad_kernel), grad_smem, done_grad));
  launch_pdl(gated_segment_kernel, dim3(p.nseg * p.B * p.Hkv, 2), dim3(kThreads), seg_smem, stream, p);
  GATED_TRY(oal_after_launch("gated_segment_kernel", stream));
  GATED_TRY(launch_scan<false>(p, 2, stream));
  launch_pdl(gated_grad_kernel, dim3(p.nseg * p.B * p.Hkv), dim3(kThreads), grad_smem, stream, p);
  return oal_after_launch("gated_grad_kernel", stream);
}

}  // namespace oal
