// gated_tc_grad.cu -- the backward of the gated recurrence for bf16 on the
// tensor cores.
//
// With f_ij = scale e^{G_i-G_j} for j <= i of a chunk, S the state before it
// and R the gradient of the state behind it,
//     X = Q K^T, Z = dY V^T,  p = f o X, z = f o Z  (rounded to bf16)
//     dQ = z K + scale e^{G_i} dY S^T
//     dK = z^T Q + e^{G_63-G_j} V R^T,   dV = p^T dY + e^{G_63-G_j} K R
//     dg_t = sum_{j<t<=l} X_lj (f o Z)_lj + sum_{l>=t} q_l.dq_l' + sum_{j<t} k_j.dk_j' + e^{G_63} <S, R>
// (dq', dk': the terms with S and R; they and X, Z enter dg unrounded).
//   gated_tc_own_kernel   a chunk's own state (K, V) and own gradient of the
//                         state before it (Q, dY of all heads), registers
//   gated_scan_kernel     (gated_simt.cu) S and R of every chunk from those
//   gated_tc_grad_kernel  the gradients, chunks in any order: a pair of query
//                         heads is 128 rows; two blocks per SM.  S and R are
//                         operands as three bf16 terms, which hold all of their
//                         bits (R as two for dV, which is rounded to bf16).
// Tensor memory of a block: X, then dY S^T | Z, then z K | 128 columns of
// [p | z]^T [dY | Q], of which the upper left quarter is dV and the lower
// right one dK, on top of K R and V R^T.
#include <algorithm>

#include "gated_tc.cuh"

namespace oal {
namespace {
using namespace gated;

// ---------------------------------------------------------------- own states

constexpr int kOwnThreads = 128;
template <int kOwnStages>
struct OwnSmem {
  uint8_t a[kOwnStages][kTileBytes], b[kOwnStages][kTileBytes];
  alignas(16) float w[kGC];
  uint64_t full[kOwnStages];
  int abort_flag;
};

// blockIdx.y = 0: sum_j e^{G_63-G_j} k_j v_j^T of the chunk, and its decay;
// 1: scale sum_i e^{G_i} q_i dy_i^T over the query heads of the KV head.
// 51 us for 4 x 4096 tokens, 32/8 heads (168 MB in, 67 MB out: 4.6 TB/s); the
// products (mma.sync at a quarter of tcgen05's rate) and the splitting of
// their factors take about as long as the memory does.  The segments' way
// (tcgen05, factors by way of shared memory) took 57 us here, where blocks are
// one to eight chunks long and six of these share an SM.
template <int kOwnStages>
__global__ void __launch_bounds__(kOwnThreads)
gated_tc_own_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, GatedArgs p) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  OwnSmem<kOwnStages> &s = *reinterpret_cast<OwnSmem<kOwnStages> *>(align1024(smem_raw));
  const int bh = blockIdx.x / p.nseg, c = blockIdx.x % p.nseg, b = bh / p.Hkv, kv = bh % p.Hkv;
  const int tid = threadIdx.x, rho = p.Hq / p.Hkv, t0 = c * kGC;
  const bool grad = blockIdx.y != 0;
  if (tid == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kOwnStages; ++i) mbar_init(&s.full[i], 1);
    fence_mbar_init();
  }
  pdl_wait();
  const int n = gated_len(p, b);
  if (t0 >= n) return;
  __syncthreads();
  volatile int *abort_flag = &s.abort_flag;
  const int count = grad ? rho : 1;
  auto load = [&](int r) {
    const int st = r % kOwnStages;
    mbar_arrive_expect_tx(&s.full[st], 2 * kTileBytes);
    tma_load_3d(s.a[st], grad ? &tmQ : &tmK, &s.full[st], 0, t0, grad ? b * p.Hq + kv * rho + r : bh);
    tma_load_3d(s.b[st], grad ? &tmO : &tmV, &s.full[st], 0, t0, grad ? b * p.Hq + kv * rho + r : bh);
  };
  if (tid == 0)
    for (int r = 0; r < min(kOwnStages, count); ++r) load(r);
  if (tid < 32) {
    const GateLane sums = gate_sums(gate_load(p.g + (size_t)bh * p.T, t0, n));
    if (!grad) {
      const GateDecay whole = gate_tails(sums, reinterpret_cast<float2 *>(s.w)[tid]);
      if (tid == 0) p.seg_decay[(size_t)bh * p.nseg + c] = whole;
    } else {
      reinterpret_cast<float2 *>(s.w)[tid] =
          make_float2(p.scale * gate_exp_fast(sums.cuts[0] == 0, sums.hi[0] + sums.lo[0]),
                      p.scale * gate_exp_fast(sums.cuts[1] == 0, sums.hi[1] + sums.lo[1]));
    }
  }
  __syncthreads();
  StateAcc<8> acc;
  state_load(acc, 0, nullptr);
  bool ok = true;
  for (int r = 0; r < count; ++r) {
    const int st = r % kOwnStages;
    ok = ok && mbar_wait(&s.full[st], (r / kOwnStages) & 1, abort_flag, p.status);
    ok = __all_sync(0xffffffffu, ok);
    if (t0 + kGC > n && n < p.T) {   // rows behind the sequence count as zeros
      clear_rows(s.a[st], n - t0, tid, kOwnThreads);
      clear_rows(s.b[st], n - t0, tid, kOwnThreads);
      fence_proxy_async();
      __syncthreads();
    }
    if (ok) state_step(acc, 1.f, 0, s.a[st], s.b[st], s.w);
    __syncthreads();
    if (tid == 0 && ok && r + kOwnStages < count) load(r + kOwnStages);
  }
  if (tid == 0 && !ok)   // copies still in flight land before the block ends
    for (int i = 0; i < min(kOwnStages, count); ++i)
      for (int ph = 0; ph < 2; ++ph) mbar_wait_teardown(&s.full[i], ph, p.status);
  state_store(acc, 0, (grad ? p.seg_grad : p.seg_state) + ((size_t)bh * p.nseg + c) * kGS);
}

// ---------------------------------------------------------------- gradients

// Factors f of keys j0 .. j0 + 7 of the chunk for row i by themselves, where
// `on` has a bit, into two places (a chunk whose gates drop too far for factors; out of line,
// as its instructions would push the others out of the cache).
__device__ __noinline__ void each_decay(const float *g, int t0, int n, int i, int j0, uint32_t on, float scale, float4 *to0,
                                        float4 *to1) {
  const GateLane s = gate_sums(gate_load(g, t0, n));
  const float h0 = __shfl_sync(0xffffffffu, s.hi[0], i >> 1), h1 = __shfl_sync(0xffffffffu, s.hi[1], i >> 1);
  const float l0 = __shfl_sync(0xffffffffu, s.lo[0], i >> 1), l1 = __shfl_sync(0xffffffffu, s.lo[1], i >> 1);
  const float hi = i & 1 ? h1 : h0, lo = i & 1 ? l1 : l0;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int from = (j0 + e) >> 1;
    const float hj = __shfl_sync(0xffffffffu, s.hi[e & 1], from), lj = __shfl_sync(0xffffffffu, s.lo[e & 1], from);
    f[e] = scale * gate_exp_fast(on & (1u << e), (hi - hj) + (lo - lj));
  }
  *to0 = make_float4(f[0], f[1], f[2], f[3]);
  *to1 = make_float4(f[4], f[5], f[6], f[7]);
}

constexpr int kGradThreads = 320;              // eight computing warps, one for the MMAs, one for loads and gates
constexpr uint32_t kGradCols = 256;
struct GradSmem {
  uint8_t kv[2 * kTileBytes];                  // K, V
  uint8_t oq[4 * kTileBytes];                  // dY of two heads, Q of two heads
  uint8_t pz[4 * kTileBytes];                  // p, z of 128 rows; dQ after p; before z R in fp32, then its
                                               // first two terms, and the third before p
  uint8_t st[3 * kTileBytes];                  // S in fp32, then its terms
  struct alignas(16) Gates {
    ChunkGates c;
    float tail[kGC], head[kGC];                // e^{G_63-G_j}, e^{G_i}
  } gates[2];
  struct Sums {                                // parts of dg
    float rows[2][2 * kGC], cols[4][kGC], far[2][kGC], dots[8];
  } sums[2];
  uint64_t kv_full, r_full, gate_full, split_full, far_full, q_full, clean, go, xz_full, pz_full, dq_full, p_free, pair[4],
      meet, chunk_done[2], drain;
  uint32_t tmem;
  WaitState wait;
};
static_assert(2 * (sizeof(GradSmem) + 2 * 1024) <= 228 * 1024, "two blocks per SM");

// Four values as three bf16 terms, which hold all of their 24 bits.
__device__ __forceinline__ void split_put(float4 x, uint8_t *to0, uint8_t *to1, uint8_t *to2) {
  uint2 t[3];
  split3(x.x, x.y, t[0].x, t[1].x, t[2].x);
  split3(x.z, x.w, t[0].y, t[1].y, t[2].y);
  *reinterpret_cast<uint2 *>(to0) = t[0];
  *reinterpret_cast<uint2 *>(to1) = t[1];
  *reinterpret_cast<uint2 *>(to2) = t[2];
}

// dg of a chunk from its parts (one warp, two tokens a lane).
__device__ __noinline__ void chunk_dg(const GradSmem::Sums &u, const ChunkGates &gates, float *dg, int rows) {
  const int lane = threadIdx.x & 31;
  float x = 0.f, r[2], f[2];
#pragma unroll
  for (int z = 0; z < 8; ++z) x += u.dots[z];
  x = decay_by(gates.whole.hi, x);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = 2 * lane + e;
    r[e] = (u.rows[0][t] + u.rows[1][t]) + (u.rows[0][64 + t] + u.rows[1][64 + t]) -
           ((u.cols[0][t] + u.cols[1][t]) + (u.cols[2][t] + u.cols[3][t]));
    f[e] = u.far[0][t] + u.far[1][t];
  }
  float down = r[0] + r[1], up = f[0] + f[1];              // sums from this lane on; up to it
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float a = __shfl_down_sync(0xffffffffu, down, d), v = __shfl_up_sync(0xffffffffu, up, d);
    if (lane + d < 32) down += a;
    if (lane >= d) up += v;
  }
  up = __shfl_up_sync(0xffffffffu, up, 1);
  if (lane == 0) up = 0.f;
  float after = __shfl_down_sync(0xffffffffu, down, 1);
  if (lane == 31) after = 0.f;
  const float d0 = x + (after + r[1] + r[0]) + up, d1 = x + (after + r[1]) + (up + f[0]);
  if (2 * lane < rows) dg[2 * lane] = gates.cut_even >> lane & 1u ? 0.f : d0;
  if (2 * lane + 1 < rows) dg[2 * lane + 1] = gates.cut_odd >> lane & 1u ? 0.f : d1;
}

// dY and Q of heads head .. head + heads - 1 into their tiles, or (to null) into L2.
__device__ __noinline__ void fetch_heads(const CUtensorMap *tmO, const CUtensorMap *tmQ, uint8_t *to, uint64_t *bar, int t0,
                                         int head, int heads) {
  if (to) mbar_arrive_expect_tx(bar, 2 * heads * kTileBytes);
#pragma unroll 1
  for (int h = 0; h < heads; ++h) {
    if (to) {
      tma_load_3d(to + h * kTileBytes, tmO, bar, 0, t0, head + h);
      tma_load_3d(to + (2 + h) * kTileBytes, tmQ, bar, 0, t0, head + h);
    } else {
      tma_prefetch_3d(tmO, 0, t0, head + h);
      tma_prefetch_3d(tmQ, 0, t0, head + h);
    }
  }
}

// 97 us for 4 x 4096 tokens, 32/8 heads (307 MB: 3.2 TB/s).  Bound by the chain
// of a step - tile loads, X and Z, p and z, 24 MMAs, dQ - about 11,000 cycles a
// pair of heads where two blocks per SM leave half of that; tensor pipe 23% busy.
// With S and R as two bf16 terms each, formed by the scan, it took 88, and the
// scan 2 us more; dg was off by 3e-6 instead of 7e-7.
__global__ void __launch_bounds__(kGradThreads, 2)
gated_tc_grad_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                     const __grid_constant__ CUtensorMap tmDQ, GatedArgs p) {
  extern __shared__ uint8_t smem_raw[];
  GradSmem &s = *reinterpret_cast<GradSmem *>(align1024(smem_raw));
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int rho = p.Hq / p.Hkv, npair = (rho + 1) / 2;
  if (tid == 0) {
    s.wait.abort = 0;
    s.wait.status = p.status;
    mbar_init(&s.kv_full, 1), mbar_init(&s.r_full, 1), mbar_init(&s.gate_full, 1), mbar_init(&s.far_full, 1);
    mbar_init(&s.split_full, 8);
    mbar_init(&s.q_full, 1), mbar_init(&s.clean, 8), mbar_init(&s.go, 8), mbar_init(&s.xz_full, 1);
    mbar_init(&s.pz_full, 8), mbar_init(&s.dq_full, 1), mbar_init(&s.p_free, 4), mbar_init(&s.meet, 8);
    mbar_init(&s.chunk_done[0], 8), mbar_init(&s.chunk_done[1], 8), mbar_init(&s.drain, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&s.pair[i], 2);
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 8) {   // (not before: this block must not hold tensor memory that what it waits for may want)
    tmem_alloc(&s.tmem, kGradCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tb = uniform(s.tmem), tx = tb, tz = tb + 64, tkv = tb + 128;
  auto wait = [&](uint64_t *bar, int phase) { return warp_wait(bar, phase & 1, &s.wait); };
  auto arrive = [&](uint64_t *bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // The block's chunks: every gridDim.x-th of (batch, KV head, chunk), the last
  // fastest, counted up digit by digit (a division costs more than the rest).
  struct Place {
    int b, kv, c;
  };
  const int per = p.nseg * p.Hkv;
  const Place by = {(int)gridDim.x / per, (int)gridDim.x % per / p.nseg, (int)gridDim.x % p.nseg};
  auto next_of = [&](Place x) {
    x.c += by.c, x.kv += by.kv, x.b += by.b;
    if (x.c >= p.nseg) x.c -= p.nseg, ++x.kv;
    if (x.kv >= p.Hkv) x.kv -= p.Hkv, ++x.b;
    return x;
  };
  const Place begin_at = {(int)blockIdx.x / per, (int)blockIdx.x % per / p.nseg, (int)blockIdx.x % p.nseg};
  bool ok = true;
  // All sides count alike: k chunks, it steps (a chunk's pairs of heads), cl
  // cleanings.  Every barrier completes once per what it counts, and whoever
  // waits on it is never more than a phase behind: the next but one needs
  // what comes after that wait (chunk_done is a pair for that).
  int k = 0, it = 0, cl = 0;
  // Tiles of heads that do not exist, or rows behind a sequence, are cleared
  // before the tensor cores read them (they are summed over).
  auto cleans = [&](int pr, bool tail) { return tail || (rho - 2 * pr == 1 && (rho > 1 || it == 0)); };

  if (warp == 9) {
    // ---- loads and gates, ahead of the rest; dg behind it
    auto load_q = [&](int t0, int h0, int pr) {
      fetch_heads(&tmO, &tmQ, s.oq, &s.q_full, t0, h0 + 2 * pr, min(2, rho - 2 * pr));
    };
    auto prefetch_q = [&](int t0, int h0, int pr) {
      fetch_heads(&tmO, &tmQ, nullptr, nullptr, t0, h0 + 2 * pr, min(2, rho - 2 * pr));
    };
    // dg of the chunk before: its parts are there once all warps are done with it
    float *dg = nullptr;
    int dg_rows = 0;
    auto finish = [&]() {
      if (!wait(&s.chunk_done[(k - 1) & 1], (k - 1) >> 1)) return false;
      chunk_dg(s.sums[(k - 1) & 1], s.gates[(k - 1) & 1].c, dg, dg_rows);
      return true;
    };
    int q_loads = 0;
#pragma unroll 1
    for (Place x = begin_at; x.b < p.B && ok; x = next_of(x)) {
      const int bh = x.b * p.Hkv + x.kv, t0 = x.c * kGC, n = gated_len(p, x.b), h0 = x.b * p.Hq + x.kv * rho;
      if (t0 >= n) continue;
      // the last step's MMAs have read K, V, S, z and the pair of heads (waited for below)
      if (lane == 0) {
        mbar_arrive_expect_tx(&s.kv_full, 4 * kTileBytes);
        tma_load_3d(s.kv, &tmK, &s.kv_full, 0, t0, bh);
        tma_load_3d(s.kv + kTileBytes, &tmV, &s.kv_full, 0, t0, bh);
        bulk_load(s.st, p.seg_state + ((size_t)bh * p.nseg + x.c) * kGS, kGS * sizeof(float), &s.kv_full);
        mbar_arrive_expect_tx(&s.r_full, 2 * kTileBytes);
        bulk_load(s.pz + 2 * kTileBytes, p.seg_grad + ((size_t)bh * p.nseg + x.c) * kGS, kGS * sizeof(float), &s.r_full);
        load_q(t0, h0, 0), ++q_loads;
        if (npair > 1) prefetch_q(t0, h0, 1);
      }
      __syncwarp();
      // (two chunks back, these gates were read for the last time before that dg)
      const float2 gate = gate_load(p.g + (size_t)bh * p.T, t0, n);
      const GateLane sums = gate_sums(gate);
      GradSmem::Gates &to = s.gates[k & 1];
      chunk_gates<true>(gate, sums, to.c, reinterpret_cast<float2 *>(to.tail)[lane]);
      reinterpret_cast<float2 *>(to.head)[lane] = make_float2(gate_exp_fast(sums.cuts[0] == 0, sums.hi[0] + sums.lo[0]),
                                                              gate_exp_fast(sums.cuts[1] == 0, sums.hi[1] + sums.lo[1]));
      arrive(&s.gate_full);
      if (k > 0 && !finish()) ok = false;
      if (!ok) break;
      dg = p.dg + (size_t)bh * p.T + t0;
      dg_rows = n - t0;
      ++k;
#pragma unroll 1
      for (int pr = 0; pr < npair && ok; ++pr, ++it) {
        if (lane == 0) {
          if (pr + 2 < npair) prefetch_q(t0, h0, pr + 2);
          const Place y = next_of(x);
          if (pr == npair - 1 && y.b < p.B) {
            const int nbh = y.b * p.Hkv + y.kv;
            const size_t at = ((size_t)nbh * p.nseg + y.c) * kGS;
            tma_prefetch_3d(&tmK, 0, y.c * kGC, nbh);
            tma_prefetch_3d(&tmV, 0, y.c * kGC, nbh);
            prefetch_l2(p.seg_state + at, kGS * sizeof(float));
            prefetch_l2(p.seg_grad + at, kGS * sizeof(float));
            prefetch_q(y.c * kGC, y.b * p.Hq + y.kv * rho, 0);
          }
        }
        __syncwarp();
        ok = wait(&s.dq_full, it);
        if (ok && lane == 0 && pr + 1 < npair) load_q(t0, h0, pr + 1), ++q_loads;
        __syncwarp();
      }
    }
    if (ok && k > 0) finish();
    if (lane == 0 && !ok) {   // the last loads may not have been waited for
      for (int ph = 0; ph < 2; ++ph) {
        mbar_wait_teardown(&s.kv_full, ph, p.status);
        mbar_wait_teardown(&s.r_full, ph, p.status);
      }
      if (q_loads > 0) mbar_wait_teardown(&s.q_full, (q_loads - 1) & 1, p.status);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---- the MMAs
    const uint32_t id_k = idesc_bf16_f32(128, 64, 0), id_mn = idesc_bf16_f32(128, 64, 1);
    const uint32_t id_kv = idesc_bf16_f32(128, 128, 1) | (1u << 15);   // A with rows along its minor axis too
    const uint64_t od = sdesc_sw128(smem_u32(s.oq), 16, 1024), qd = sdesc_sw128(smem_u32(s.oq) + 2 * kTileBytes, 16, 1024);
    const uint64_t kd = sdesc_sw128(smem_u32(s.kv), 16, 1024), vd = sdesc_sw128(smem_u32(s.kv) + kTileBytes, 16, 1024);
    // the terms of S one behind the other, of R the first two at z, the third at p
    constexpr uint64_t kNext = kTileBytes >> 4;
    const uint64_t sd = sdesc_sw128(smem_u32(s.st), 16, 1024);
    const uint64_t rd = sdesc_sw128(smem_u32(s.pz) + 2 * kTileBytes, 16, 1024), zd = rd;
    const uint64_t rd3 = sdesc_sw128(smem_u32(s.pz), 16, 1024);
    // [p | z] and [dY | Q]: two 64-column atoms, 16 KB apart
    const uint64_t pzd = sdesc_sw128(smem_u32(s.pz), 2 * kTileBytes, 1024);
    const uint64_t oqd = sdesc_sw128(smem_u32(s.oq), 2 * kTileBytes, 1024);
#pragma unroll 1
    for (Place x = begin_at; x.b < p.B && ok; x = next_of(x)) {
      const int t0 = x.c * kGC, n = gated_len(p, x.b);
      if (t0 >= n) continue;
      const bool tail = t0 + kGC > n && n < p.T;
      ok = wait(&s.kv_full, k);
#pragma unroll 1
      for (int pr = 0; pr < npair && ok; ++pr) {
        ok = wait(&s.q_full, it);
        if (ok && cleans(pr, tail)) ok = wait(&s.clean, cl++);
        ok = ok && wait(&s.go, it);       // X and Z are free
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j) umma_ss_warp(tx, qd + 2 * j, kd + 2 * j, id_k, j > 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) umma_ss_warp(tz, od + 2 * j, vd + 2 * j, id_k, j > 0);
        umma_commit_warp(&s.xz_full);
        if (pr == 0) {
          // [K; V] R and [K; V] R^T side by side: K R above on the left, V R^T below on the right
          ok = wait(&s.split_full, k) && (k == 0 || wait(&s.chunk_done[(k - 1) & 1], (k - 1) >> 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < 8; ++j) umma_ss_warp(tkv, kd + 2 * (j & 3), rd + kNext * (j >> 2) + 128 * (j & 3), id_mn, j > 0);
#pragma unroll
          for (int j = 0; j < 8; ++j) umma_ss_warp(tkv + 64, kd + 2 * (j & 3), rd + kNext * (j >> 2) + 2 * (j & 3), id_k, j > 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) umma_ss_warp(tkv + 64, kd + 2 * j, rd3 + 2 * j, id_k, 1u);
          umma_commit_warp(&s.far_full);
          ++k;
        }
        ok = wait(&s.pz_full, it);        // p and z are there, X and Z are read
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 12; ++j) umma_ss_warp(tx, od + 2 * (j & 3), sd + kNext * (j >> 2) + 2 * (j & 3), id_k, j > 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) umma_ss_warp(tz, zd + 2 * j, kd + 128 * j, id_mn, j > 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) umma_ss_warp(tkv, pzd + 128 * j, oqd + 128 * j, id_kv, 1u);
        umma_commit_warp(&s.dq_full);
        ++it;
      }
    }
    umma_commit_warp(&s.drain);
    if (lane == 0) mbar_wait_teardown(&s.drain, 0, p.status);   // no MMA in flight at the block's end
    __syncwarp();
  } else {
    const int quad = warp & 3, hf = warp >> 2;                 // lanes of tensor memory; keys (dims) 32 hf .. + 31
    const int m = 32 * quad + lane, i = m & 63;                // row: head m / 64 of the pair, token i
    const bool own = hf == (quad & 1), pre = !hf && (quad & 1);   // keys of the row's half of the chunk; of the half before
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    int met = 0, paired = 0;
    arrive(&s.go);
#pragma unroll 1
    for (Place x = begin_at; x.b < p.B && ok; x = next_of(x)) {
      const int bh = x.b * p.Hkv + x.kv, t0 = x.c * kGC, n = gated_len(p, x.b), h0 = x.b * p.Hq + x.kv * rho;
      if (t0 >= n) continue;
      const bool tail = t0 + kGC > n && n < p.T;
      const GradSmem::Gates &gates = s.gates[k & 1];
      GradSmem::Sums &sums = s.sums[k & 1];
      ok = wait(&s.gate_full, k) && wait(&s.kv_full, k);
      if (!ok) break;
      auto clean = [&](int pr) {
        const int keep = tail ? n - t0 : 64, keep1 = rho - 2 * pr == 1 ? 0 : keep;
        clear_rows(s.oq, keep, tid, 256);
        clear_rows(s.oq + kTileBytes, keep1, tid, 256);
        clear_rows(s.oq + 2 * kTileBytes, keep, tid, 256);
        clear_rows(s.oq + 3 * kTileBytes, keep1, tid, 256);
        fence_proxy_async();
        arrive(&s.clean);
      };
      if (cleans(0, tail)) {                                   // with the first pair: K and V too
        ok = wait(&s.q_full, it);
        if (!ok) break;
        if (tail) {
          clear_rows(s.kv, n - t0, tid, 256);
          clear_rows(s.kv + kTileBytes, n - t0, tid, 256);
        }
        clean(0);
      }
      float cfar = 0.f;
      ok = wait(&s.r_full, k);
      if (!ok) break;
      {
        // S and R (row-major, as the scan left them) into their terms, in the same
        // place: all of them read, then written.  <S, R> on the way.
        float4 sv[4], rv[4];
        float dot = 0.f;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          sv[z] = reinterpret_cast<const float4 *>(s.st)[tid + 256 * z];
          rv[z] = reinterpret_cast<const float4 *>(s.pz + 2 * kTileBytes)[tid + 256 * z];
          dot = fmaf(sv[z].x, rv[z].x, fmaf(sv[z].y, rv[z].y, dot));
          dot = fmaf(sv[z].z, rv[z].z, fmaf(sv[z].w, rv[z].w, dot));
        }
        arrive(&s.meet);
        ok = wait(&s.meet, met++) && (it == 0 || wait(&s.p_free, it - 1));   // (dQ has left the third term's place)
        if (!ok) break;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int f = tid + 256 * z;
          const uint32_t at = tile_at(f >> 4, (f & 15) >> 1) + 8 * (f & 1);
          split_put(sv[z], s.st + at, s.st + kTileBytes + at, s.st + 2 * kTileBytes + at);
          split_put(rv[z], s.pz + 2 * kTileBytes + at, s.pz + 3 * kTileBytes + at, s.pz + at);
        }
        fence_proxy_async();
        arrive(&s.split_full);
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        if (lane == 0) sums.dots[warp] = dot;
        // K R (rows 0 .. 63) and V R^T (64 .. 127) times the keys' decays to the chunk's end
        ok = wait(&s.far_full, k);
        if (!ok) break;
        tc_fence_after();
        const float tj = gates.tail[i];
        const uint32_t from = tkv + (quad & 2 ? 64u : 0u) + 32u * hf + lanes;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t x[16];
          tmem_ld16(from + 16 * h, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(decay_by(tj, __uint_as_float(x[e])));
          if (quad & 2) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint4 kk = *reinterpret_cast<const uint4 *>(s.kv + tile_at(i, 4 * hf + 2 * h + z));
              const uint32_t u[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                cfar = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(x[8 * z + 2 * e]), cfar);
                cfar = fmaf(__uint_as_float(u[e] & 0xFFFF0000u), __uint_as_float(x[8 * z + 2 * e + 1]), cfar);
              }
            }
          }
          tmem_st16(from + 16 * h, x);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      ++k;                                                     // (R has been read: p and z take its place)
      const int mode = gates.c.mode;
      const float fq = p.scale * gates.head[i];
      const float fr = p.scale * gates.c.row[i];
      const float *rest = pre ? gates.c.before : gates.c.rest + 32 * hf;
      int begin = 0;
      cut_before(gates.c, i, begin);
      const uint32_t live = 0xFFFFFFFFu << min(31, max(0, begin - 32 * hf));
      const uint32_t mask = own ? live & (0xFFFFFFFFu >> (31 - lane)) : pre && begin < 32 ? live : 0u;
      float w[32], racc = 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) w[e] = 0.f;
#pragma unroll 1
      for (int pr = 0; pr < npair; ++pr) {
        ok = wait(&s.q_full, it);
        if (!ok) break;
        if (pr > 0 && cleans(pr, tail)) clean(pr);
        ok = wait(&s.xz_full, it);
        if (!ok) break;
        tc_fence_after();
        if (it > 0) {                                          // the outputs of the step before have left the place of p
          ok = wait(&s.p_free, it - 1);
          if (!ok) break;
        }
        if (own || pre) {
          if (mode == kEach)   // the factors lie where their p and z will
#pragma unroll 1
            for (int h = 0; h < 4; ++h)
              each_decay(p.g + (size_t)bh * p.T, t0, n, i, 32 * hf + 8 * h, mask >> (8 * h), p.scale,
                         reinterpret_cast<float4 *>(s.pz + tile_at(m, 4 * hf + h)),
                         reinterpret_cast<float4 *>(s.pz + 2 * kTileBytes + tile_at(m, 4 * hf + h)));
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t x[8], y[8];
            tmem_ld8(tx + lanes + 32 * hf + 8 * h, x);
            tmem_ld8(tz + lanes + 32 * hf + 8 * h, y);
            float f[8];
            if (mode != kEach) {
#pragma unroll
              for (int e = 0; e < 8; e += 4) {
                const float4 r = *reinterpret_cast<const float4 *>(rest + 8 * h + e);
                f[e] = fr * r.x, f[e + 1] = fr * r.y, f[e + 2] = fr * r.z, f[e + 3] = fr * r.w;
              }
            } else {
              const float4 r0 = *reinterpret_cast<const float4 *>(s.pz + tile_at(m, 4 * hf + h));
              const float4 r1 = *reinterpret_cast<const float4 *>(s.pz + 2 * kTileBytes + tile_at(m, 4 * hf + h));
              f[0] = r0.x, f[1] = r0.y, f[2] = r0.z, f[3] = r0.w;
              f[4] = r1.x, f[5] = r1.y, f[6] = r1.z, f[7] = r1.w;
            }
            tmem_wait_ld();
            uint32_t pw[4], zw[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              float pv[2], zv[2];
#pragma unroll
              for (int d = 0; d < 2; ++d) {
                const int j = 8 * h + e + d;
                const float fv = mask & (1u << j) ? f[e + d] : 0.f, xv = __uint_as_float(x[e + d]);
                zv[d] = fv * __uint_as_float(y[e + d]);
                pv[d] = fv * xv;
                w[j] = fmaf(xv, zv[d], w[j]);
              }
              pw[e >> 1] = pack_bf16x2(pv[0], pv[1]);
              zw[e >> 1] = pack_bf16x2(zv[0], zv[1]);
            }
            *reinterpret_cast<uint4 *>(s.pz + tile_at(m, 4 * hf + h)) = make_uint4(pw[0], pw[1], pw[2], pw[3]);
            *reinterpret_cast<uint4 *>(s.pz + 2 * kTileBytes + tile_at(m, 4 * hf + h)) = make_uint4(zw[0], zw[1], zw[2], zw[3]);
          }
        } else {                                               // later keys: nothing
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            *reinterpret_cast<uint4 *>(s.pz + tile_at(m, 4 * hf + z)) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(s.pz + 2 * kTileBytes + tile_at(m, 4 * hf + z)) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        uint4 q[4];                                            // the row's queries, before their buffer is refilled
#pragma unroll
        for (int z = 0; z < 4; ++z) q[z] = *reinterpret_cast<const uint4 *>(s.oq + 2 * kTileBytes + tile_at(m, 4 * hf + z));
        fence_proxy_async();
        tc_fence_before();
        arrive(&s.pz_full);
        ok = wait(&s.dq_full, it);
        if (!ok) break;
        tc_fence_after();
        ++it;
        const int hd = 2 * pr + (m >> 6);
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.dQ) + ((size_t)(h0 + hd) * p.T + t0 + i) * 64) + 4 * hf;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t x[16], y[16];
          tmem_ld16(tx + lanes + 32 * hf + 16 * h, x);
          tmem_ld16(tz + lanes + 32 * hf + 16 * h, y);
          tmem_wait_ld();
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint4 qq = q[z];
            const uint32_t u[4] = {qq.x, qq.y, qq.z, qq.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = decay_by(fq, __uint_as_float(x[8 * z + 2 * e])), d = decay_by(fq, __uint_as_float(x[8 * z + 2 * e + 1]));
              racc = fmaf(__uint_as_float(u[e] << 16), a, racc);
              racc = fmaf(__uint_as_float(u[e] & 0xFFFF0000u), d, racc);
              o[e] = pack_bf16x2(a + __uint_as_float(y[8 * z + 2 * e]), d + __uint_as_float(y[8 * z + 2 * e + 1]));
            }
            const uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
            if (!tail) *reinterpret_cast<uint4 *>(s.pz + tile_at(m, 4 * hf + 2 * h + z)) = out;   // p has been read
            else if (hd < rho && t0 + i < n) dst[2 * h + z] = out;
          }
          q[0] = q[2], q[1] = q[3];
        }
        fence_proxy_async();
        tc_fence_before();
        arrive(&s.go);
        arrive(&s.pair[quad]);
        if (hf == 0) {                                         // both halves of these 32 rows are there
          ok = wait(&s.pair[quad], paired);
          if (!ok) break;
          if (lane == 0) {
            const int row = 32 * (quad & 1);
            if (!tail && hd < rho && t0 + row < n) tma_store_3d(&tmDQ, s.pz + 32 * quad * 128, 0, t0 + row, h0 + hd);
            bulk_commit();
            bulk_wait_read();
            mbar_arrive(&s.p_free);
          }
          __syncwarp();
        }
        ++paired;
      }
      if (!ok) break;
      // dV from rows 0 .. 63, dK from rows 64 .. 127; the sums for dg
      {
        const uint32_t from = tkv + (quad & 2 ? 64u : 0u) + 32u * hf + lanes;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(quad & 2 ? p.dK : p.dV) + ((size_t)bh * p.T + t0 + i) * 64) + 4 * hf;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t x[16];
          tmem_ld16(from + 16 * h, x);
          tmem_wait_ld();
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = pack_bf16x2(__uint_as_float(x[8 * z + 2 * e]), __uint_as_float(x[8 * z + 2 * e + 1]));
            const uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
            if (t0 + i < n) dst[2 * h + z] = out;              // (not by way of shared memory: R is on its way there)
          }
        }
        tc_fence_before();
        float sum = racc;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          w[e] = own && e == lane ? 0.f : w[e];                // a token's own pair decays by nothing
          sum += w[e];
        }
        sums.rows[hf][m] = sum;
        // lane l ends with the sum over the warp's rows of column l
#pragma unroll
        for (int d = 16; d; d >>= 1)
#pragma unroll
          for (int e = 0; e < d; ++e) {
            const float keep = lane & d ? w[e + d] : w[e], give = lane & d ? w[e] : w[e + d];
            w[e] = keep + __shfl_xor_sync(0xffffffffu, give, d);
          }
        sums.cols[quad][32 * hf + lane] = w[0];
        if (quad & 2) sums.far[hf][i] = cfar;
      }
      arrive(&s.chunk_done[(k - 1) & 1]);
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tb, kGradCols);
  }
}

}  // namespace

oal_status launch_gated_scan(const GatedArgs &p, int ways, bool last, cudaStream_t stream);

oal_status launch_gated_backward_tc(const GatedArgs &p, cudaStream_t stream) {
  static bool done_own[2][kMaxDevices], done_grad[kMaxDevices];
  const int total = p.nseg * p.B * p.Hkv;
  // Few chunks: more heads of each in flight (256 chunks of 7 heads: 46 us a
  // backward against 57); many: more blocks per SM (2048 chunks of 4 heads:
  // 50 us this kernel against 58).
  const bool few = total <= 3 * 152;
  const auto own = few ? gated_tc_own_kernel<4> : gated_tc_own_kernel<2>;
  const size_t own_smem = (few ? sizeof(OwnSmem<4>) : sizeof(OwnSmem<2>)) + 1024, grad_smem = sizeof(GradSmem) + 1024;
  GATED_TRY(gated_need_smem(reinterpret_cast<const void *>(own), own_smem, done_own[few]));
  GATED_TRY(gated_need_smem(reinterpret_cast<const void *>(gated_tc_grad_kernel), grad_smem, done_grad));
  const long long hq = (long long)p.B * p.Hq, hkv = (long long)p.B * p.Hkv;
  CUtensorMap tmQ, tmK, tmV, tmO, tmDQ;
  GATED_TRY(make_map(&tmQ, p.Q, p.T, hq));
  GATED_TRY(make_map(&tmK, p.K, p.T, hkv));
  GATED_TRY(make_map(&tmV, p.V, p.T, hkv));
  GATED_TRY(make_map(&tmO, p.dY, p.T, hq));
  GATED_TRY(make_map(&tmDQ, p.dQ, p.T, hq, 32));
  launch_pdl(own, dim3(total, 2), dim3(kOwnThreads), own_smem, stream, tmQ, tmK, tmV, tmO, p);
  GATED_TRY(oal_after_launch("gated_tc_own_kernel", stream));
  GATED_TRY(launch_gated_scan(p, 2, false, stream));
  launch_pdl(gated_tc_grad_kernel, dim3(std::min(total, 2 * 152)), dim3(kGradThreads), grad_smem, stream, tmQ, tmK, tmV,
             tmO, tmDQ, p);
  return oal_after_launch("gated_tc_grad_kernel", stream);
}

}  // namespace oal
