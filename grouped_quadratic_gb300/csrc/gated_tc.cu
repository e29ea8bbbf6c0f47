// gated_tc.cu -- the gated linear recurrence for bf16 on the tensor cores.
//
// Prefill.  gated_tc_segment_kernel forms the segments' own states,
// gated_scan_kernel (gated_simt.cu) the state before each segment and the last
// one, and gated_tc_out_kernel walks every segment: per chunk of 64 tokens and
// pair of query heads of the KV head (128 rows: 64 tokens of each)
//     X = Q K^T,  D = Q S_in           tcgen05, operands as TMA left them
//     P = X o decays (bf16)            four warps, tensor memory -> registers -> tensor memory
//     D += P V                         tcgen05, P from tensor memory
// and the state itself in registers (gated_mma.cuh).
//
// Where the sums G of a chunk span at most 60, a row's factor is taken out of
// its sum, one product a score and one a result:
//     y_i = scale e^{G_i} [ S_in^T q_i + sum_j (q_i.k_j) e^{-G_j} v_j ].
// The sum is up to e^60 = 1e26 times the result: where that leaves fp32 (results
// of 3e12 and more), a block whose results are not finite takes its segment
// again without this way (one more packed product per two results to see that;
// the next way for every chunk cost 8% of a prefill).
// Where each half spans at most 60, a decay is the product of two factors,
//     e^{G_i-G_j} = e^{G_i-R} e^{R-G_j},
// with R = 0 for the first 32 rows and G_31 for the others, which meet before a
// score does, and S_in^T q_i takes e^{G_i} in tensor memory; a cut gate leaves
// the sums alone and masks the scores and S_in instead.  Other chunks form every
// decay exp(G_i - G_j) by itself.  Prefill of 4 x 8192 tokens, 32/8 heads: 83.5 us
// by the first way, 91.6 by the second (g = -1.5), 184 by the third (g = -3), 143
// where every segment is taken again.
//
// Rounded to bf16, because the tensor cores take both factors in the inputs'
// type: P, and the state that a chunk reads, by 2^-8 at most each.  Y is off by
// 2.35e-3 in the mean, of which 1.66e-3 are its own rounding.  Second terms would
// be 8 more MMAs to a step's 12 and another 8 KB a block, where three blocks
// leave none.
#include <algorithm>

#include "gated_tc.cuh"

namespace oal {
namespace {
using namespace gated;

constexpr int kStages = 3;                  // chunks in flight of the segment kernel
constexpr int kSegThreads = 128;
constexpr int kOutThreads = 160;            // four computing warps and one that issues
constexpr uint32_t kOutCols = 128;          // tensor memory: X (then P) 64, D 64
constexpr uint32_t kColX = 0, kColD = 64;

// ---------------------------------------------------------------- segments

// sum_j w_j a_j b_j^T over the 64 rows j of two bf16 tiles, as a sum of fp32
// products: w_j a_j is formed in fp32 and goes in as three bf16 terms, which
// hold all of its 24 bits.  The terms lie in shared memory as the tiles do, the
// first in the place of a: one MMA of 128 rows takes the first two (64 rows of
// the state each), another the second again and the third.  Every sum starts
// from zero, because the tensor cores cut what they add to an accumulator; the
// state is in registers, thread m (of 128) holding row m % 64 as the first
// term's sum or that of the other two.
constexpr uint32_t kSumCols = 128;
constexpr int kSumIssuer = 3;               // the warp that issues (the first one loads)
// Threads 0 .. 127; `terms` has room for two tiles.
__device__ __forceinline__ void sum_split(uint8_t *a, uint8_t *terms, const float *w) {
#pragma unroll
  for (int z = 0; z < 4; ++z) {
    const int row = (threadIdx.x >> 3) + 16 * z;
    const uint32_t at = tile_at(row, threadIdx.x & 7);
    const float f = w[row];
    const uint4 x4 = *reinterpret_cast<const uint4 *>(a + at);
    const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
    uint32_t t[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo = f * __uint_as_float(x[e] << 16), hi = f * __uint_as_float(x[e] & 0xFFFF0000u);
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const uint32_t word = pack_bf16x2(lo, hi);
        lo -= __uint_as_float(word << 16), hi -= __uint_as_float(word & 0xFFFF0000u);
        t[q][e] = word;
      }
    }
    *reinterpret_cast<uint4 *>(a + at) = make_uint4(t[0][0], t[0][1], t[0][2], t[0][3]);
    *reinterpret_cast<uint4 *>(terms + at) = make_uint4(t[1][0], t[1][1], t[1][2], t[1][3]);
    *reinterpret_cast<uint4 *>(terms + kTileBytes + at) = make_uint4(t[2][0], t[2][1], t[2][2], t[2][3]);
  }
  fence_proxy_async();
}
// The products (one warp); `bar` completes with them.  `terms` lies behind `a`.
__device__ __forceinline__ void sum_issue(uint32_t tm, const uint8_t *a, const uint8_t *b, const uint8_t *terms, uint64_t *bar) {
  const uint32_t id = idesc_bf16_f32(128, 64, 1) | (1u << 15);   // both with rows along their minor axis
  const uint64_t ad = sdesc_sw128(smem_u32(a), smem_u32(terms) - smem_u32(a), 1024);
  const uint64_t td = sdesc_sw128(smem_u32(terms), kTileBytes, 1024), bd = sdesc_sw128(smem_u32(b), 16, 1024);
#pragma unroll
  for (int j = 0; j < 4; ++j) umma_ss_warp(tm, ad + 128 * j, bd + 128 * j, id, j > 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) umma_ss_warp(tm + 64, td + 128 * j, bd + 128 * j, id, j > 0);
  umma_commit_warp(bar);
}
// s = f s + the sums.
__device__ __forceinline__ void sum_add(float (&s)[64], GateDecay f, uint32_t tm) {
  const int warp = threadIdx.x >> 5;
  const uint32_t from = tm + ((uint32_t)(32 * warp) << 16);
  if (f.hi == 0.f) {   // a cut gate: as in decay_add, but one branch instead of 64 masks
#pragma unroll
    for (int e = 0; e < 64; ++e) s[e] = 0.f;
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t x[16];
    tmem_ld16(from + 16 * h, x);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) s[16 * h + e] = fmaf(f.hi, s[16 * h + e], fmaf(f.lo, s[16 * h + e], __uint_as_float(x[e])));
  }
  if (warp >= 2) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      uint32_t x[16];
      tmem_ld16(from + 64 + 16 * h, x);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) s[16 * h + e] += __uint_as_float(x[e]);
    }
  }
}
// The state, by way of 64 x 68 floats of shared memory that nothing else uses now (all 128 threads).
__device__ __forceinline__ void sum_store(const float (&s)[64], float *room, float *dst) {
  float *row = room + (threadIdx.x & 63) * 68;
  if (threadIdx.x >= 64)
#pragma unroll
    for (int h = 0; h < 16; ++h) *reinterpret_cast<float4 *>(row + 4 * h) = make_float4(s[4 * h], s[4 * h + 1], s[4 * h + 2], s[4 * h + 3]);
  __syncthreads();
  if (threadIdx.x < 64)
#pragma unroll
    for (int h = 0; h < 16; ++h) {
      const float4 x = *reinterpret_cast<const float4 *>(row + 4 * h);
      *reinterpret_cast<float4 *>(row + 4 * h) =
          make_float4(s[4 * h] + x.x, s[4 * h + 1] + x.y, s[4 * h + 2] + x.z, s[4 * h + 3] + x.w);
    }
  __syncthreads();
#pragma unroll
  for (int z = 0; z < 8; ++z) {
    const int x = threadIdx.x + 128 * z;
    reinterpret_cast<float4 *>(dst)[x] = *reinterpret_cast<const float4 *>(room + (x >> 4) * 68 + 4 * (x & 15));
  }
}

constexpr int kGateBatch = 8;               // chunks whose decays are formed together, two a warp
struct SegSmem {
  uint8_t a[kStages][kTileBytes], b[kStages][kTileBytes];
  uint8_t terms[2][kTileBytes];
  struct alignas(16) {
    float tail[kGC];                      // e^{G_63-G_j}
    GateDecay whole;                      // e^{G_63}
  } gates[kGateBatch];
  uint64_t full[kStages], done, drain;
  uint32_t tmem;
  WaitState wait;
};
static_assert(3 * (sizeof(SegSmem) + 2 * 1024) <= 228 * 1024, "three blocks per SM");

// Own state of each segment: K and V once.
// A chunk's decays are a chain of shuffles as long as its products: eight
// chunks' are formed side by side, or every chunk would wait for its own.
// 24.5 us for 4 x 8192 tokens of 8 KV heads (2.8 TB/s); mma.sync, 96 products a
// warp and chunk, made the whole prefill 85.9 us where this made it 80.5.  A
// chunk is 2,500 cycles of a block, three of which share the SM -
// splitting 500, MMAs 800, their sums 300, waits - after 5,000 until the first
// one is there.  A warp of its own for loads, decays and MMAs with two places
// for the sums took 2 us more: the decays, 2,000 cycles a chunk there, were in
// its way.
__global__ void __launch_bounds__(kSegThreads, 3)
gated_tc_segment_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        GatedArgs p) {
  extern __shared__ uint8_t smem_raw[];
  SegSmem &s = *reinterpret_cast<SegSmem *>(align1024(smem_raw));
  const int bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg, b = bh / p.Hkv;
  const int tid = threadIdx.x, warp = warp_index();
  if (tid == 0) {
    s.wait.abort = 0;
    s.wait.status = p.status;
    for (int i = 0; i < kStages; ++i) mbar_init(&s.full[i], 1);
    mbar_init(&s.done, 1), mbar_init(&s.drain, 1);
    fence_mbar_init();
  }
  pdl_wait();
  const int n = gated_len(p, b);
  if (seg > gated_last_seg(n, p.seg_chunks * kGC)) return;
  const int c0 = seg * p.seg_chunks, nc = max(0, min((n + kGC - 1) / kGC - c0, p.seg_chunks));
  const float *g = p.g + (size_t)bh * p.T;
  auto gate_of = [&](int c) { return gate_load(g, (c0 + c) * kGC, c < nc ? n : 0); };
  float2 gate0 = gate_of(warp), gate1 = gate_of(warp + 4);
  int loads = 0;
  auto load = [&]() {
    const int st = loads % kStages;
    mbar_arrive_expect_tx(&s.full[st], 2 * kTileBytes);
    tma_load_3d(s.a[st], &tmK, &s.full[st], 0, (c0 + loads) * kGC, bh);
    tma_load_3d(s.b[st], &tmV, &s.full[st], 0, (c0 + loads) * kGC, bh);
    ++loads;
  };
  if (tid == 0)
    while (loads < min(kStages, nc)) load();
  if (warp == kSumIssuer) {
    tmem_alloc(&s.tmem, kSumCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // (not before: what comes behind must not hold tensor memory that this block waits for)
  const uint32_t tm = uniform(s.tmem);
  float acc[64];
  GateDecay decay = {1.f, 0.f}, whole = decay;   // whole: of the chunk whose sums come next
#pragma unroll
  for (int e = 0; e < 64; ++e) acc[e] = 0.f;
  bool ok = true;
  auto take = [&](int c) {
    ok = ok && warp_wait(&s.done, c & 1, &s.wait);
    if (!ok) return;
    tc_fence_after();
    sum_add(acc, whole, tm);
    tc_fence_before();
  };
#pragma unroll 1
  for (int c = 0, st = 0, turn = 0; c < nc; ++c) {
    if (c % kGateBatch == 0) {   // (the chunk before is behind a barrier)
      const GateLane s0 = gate_sums(gate0), s1 = gate_sums(gate1);
      auto &to0 = s.gates[warp], &to1 = s.gates[warp + 4];
      to0.whole = gate_tails(s0, reinterpret_cast<float2 *>(to0.tail)[tid & 31]);
      to1.whole = gate_tails(s1, reinterpret_cast<float2 *>(to1.tail)[tid & 31]);
      gate0 = gate_of(c + kGateBatch + warp), gate1 = gate_of(c + kGateBatch + warp + 4);
      __syncthreads();
    }
    const auto &gates = s.gates[c % kGateBatch];
    ok = ok && warp_wait(&s.full[st], turn & 1, &s.wait);
    if (c > 0) {
      take(c - 1);               // its tiles and terms have been read
      if (tid == 0 && ok && loads < nc) load();
    }
    whole = gates.whole;
    decay = decay_mul(decay, whole);
    if (n < p.T && (c0 + c + 1) * kGC > n) {   // rows behind the sequence count as zeros
      clear_rows(s.a[st], n - (c0 + c) * kGC, tid, kSegThreads);
      clear_rows(s.b[st], n - (c0 + c) * kGC, tid, kSegThreads);
      __syncthreads();
    }
    if (ok) sum_split(s.a[st], s.terms[0], gates.tail);
    tc_fence_before();
    __syncthreads();
    if (warp == kSumIssuer && ok) {
      tc_fence_after();
      sum_issue(tm, s.a[st], s.b[st], s.terms[0], &s.done);
    }
    if (++st == kStages) st = 0, ++turn;
  }
  if (nc > 0) take(nc - 1);
  if (warp == kSumIssuer) {   // nothing in flight at the block's end
    umma_commit_warp(&s.drain);
    if ((tid & 31) == 0) mbar_wait_teardown(&s.drain, 0, p.status);
    __syncwarp();
  }
  if (tid == 0 && !ok)
    for (int i = max(0, loads - kStages); i < loads; ++i)
      mbar_wait_teardown(&s.full[i % kStages], (i / kStages) & 1, p.status);
  tc_fence_before();
  __syncthreads();
  sum_store(acc, reinterpret_cast<float *>(s.a), p.seg_state + ((size_t)bh * p.nseg + seg) * kGS);
  if (tid == 0) p.seg_decay[(size_t)bh * p.nseg + seg] = decay;
  if (warp == kSumIssuer) {
    tc_fence_after();
    tmem_dealloc(tm, kSumCols);
  }
}

// ---------------------------------------------------------------- outputs

struct OutSmem {
  uint8_t k[2][kTileBytes], v[2][kTileBytes];
  uint8_t q[2][2 * kTileBytes];          // two heads' queries, then their outputs
  uint8_t state[kTileBytes];             // the state before the chunk, bf16
  ChunkGates gates[2];                   // by the issuing warp
  PairWeights tail[2];                   // e^{G_63-G_j}
  uint64_t kv_full[2], q_full[2], gate_full, x_full, d_full, p_full, y_full, go, meet, drain;
  uint32_t tmem;
  int again;                             // a result was not finite
  WaitState wait;
};
static_assert(3 * (sizeof(OutSmem) + 2 * 1024) <= 228 * 1024, "three blocks per SM");

// Scores and D of a chunk whose gates drop too far for the other ways: every
// decay by itself, P in the place of X, D scaled by e^{G_i} (one row a thread).
__device__ __noinline__ void slow_scores(const float *g, int t0, int n, int i, uint32_t tm) {
  const GateLane s = gate_sums(gate_load(g, t0, n));
  const bool odd = i & 1;
  const float h0 = __shfl_sync(0xffffffffu, s.hi[0], i >> 1), h1 = __shfl_sync(0xffffffffu, s.hi[1], i >> 1);
  const float l0 = __shfl_sync(0xffffffffu, s.lo[0], i >> 1), l1 = __shfl_sync(0xffffffffu, s.lo[1], i >> 1);
  const int c0 = __shfl_sync(0xffffffffu, s.cuts[0], i >> 1), c1 = __shfl_sync(0xffffffffu, s.cuts[1], i >> 1);
  const float hi = odd ? h1 : h0, lo = odd ? l1 : l0;
  const int cut = odd ? c1 : c0;
  const float head = gate_exp_fast(cut == 0, hi + lo);
  for (int h = 0; h < 4; ++h) {         // P's 8 columns lie in front of the X still to be read
    uint32_t x[16], d[16];
    tmem_ld16(tm + kColX + 16 * h, x);
    tmem_ld16(tm + kColD + 16 * h, d);
    tmem_wait_ld();
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int from = 8 * h + (e >> 1), j = 16 * h + e;
      const float hj = __shfl_sync(0xffffffffu, s.hi[e & 1], from), lj = __shfl_sync(0xffffffffu, s.lo[e & 1], from);
      const int cj = __shfl_sync(0xffffffffu, s.cuts[e & 1], from);
      const float w = gate_exp_fast(j <= i && cj == cut, (hi - hj) + (lo - lj));
      f[e] = j <= i ? __uint_as_float(x[e]) * w : 0.f;
      d[e] = __float_as_uint(decay_by(head, __uint_as_float(d[e])));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
    tmem_st8(tm + kColX + 8 * h, x);
    tmem_st16(tm + kColD + 16 * h, d);
  }
}

// A block walks a segment, three blocks per SM (76 KB of shared memory, 128
// columns of tensor memory, 108 registers).  57.5 us for 4 x 8192 tokens, 32/8
// heads: 5.2 TB/s of DRAM traffic, 77% of a copy's; the rest is the chain
// load - X - P - P V - outputs that three blocks do not quite hide.  Two teams
// of four warps, a pair of heads each, with two blocks per SM took 86 us where
// this took 68.
__global__ void __launch_bounds__(kOutThreads, 3)
gated_tc_out_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmY,
                    GatedArgs p) {
  extern __shared__ uint8_t smem_raw[];
  OutSmem &s = *reinterpret_cast<OutSmem *>(align1024(smem_raw));
  const int bh = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg, b = bh / p.Hkv, kv = bh % p.Hkv;
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int rho = p.Hq / p.Hkv, npair = (rho + 1) / 2;
  auto init = [&]() {
    s.again = 0;
    for (int i = 0; i < 2; ++i) mbar_init(&s.kv_full[i], 1), mbar_init(&s.q_full[i], 1);
    mbar_init(&s.gate_full, 1);
    mbar_init(&s.x_full, 1);
    mbar_init(&s.d_full, 1);
    mbar_init(&s.p_full, 4);
    mbar_init(&s.y_full, 1);
    mbar_init(&s.go, 4);
    mbar_init(&s.meet, 4);
    mbar_init(&s.drain, 1);
    fence_mbar_init();
  };
  if (tid == 0) {
    s.wait.abort = 0;
    s.wait.status = p.status;
    init();
  }
  pdl_wait();
  const int n = gated_len(p, b), last = gated_last_seg(n, p.seg_chunks * kGC);
  if (seg > last) return;
  if (warp == 4) {
    tmem_alloc(&s.tmem, kOutCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // (not before: what comes behind must not hold tensor memory that this block waits for)
  const uint32_t tb = uniform(s.tmem);
  const int c0 = seg * p.seg_chunks, nc = max(0, min((n + kGC - 1) / kGC - c0, p.seg_chunks));
  const int steps = nc * npair;              // step it: chunk it / npair, heads 2 (it % npair), + 1
  const int h0 = b * p.Hq + kv * rho;
  // rows behind a sequence that ends before T must stay: its last tile is
  // stored row by row instead of by TMA (which drops rows from T on)
  auto by_rows = [&](int t0) { return t0 + kGC > n && n < p.T; };

  for (bool careful = false;; careful = true) {
    if (warp == 4) {
      const uint32_t id_k = idesc_bf16_f32(128, 64, 0), id_mn = idesc_bf16_f32(128, 64, 1);
      auto load_q = [&](int it) {
        const int pr = it % npair, heads = min(2, rho - 2 * pr), st = it & 1;
        mbar_arrive_expect_tx(&s.q_full[st], heads * kTileBytes);
        for (int h = 0; h < heads; ++h)
          tma_load_3d(s.q[st] + h * kTileBytes, &tmQ, &s.q_full[st], 0, (c0 + it / npair) * kGC, h0 + 2 * pr + h);
      };
      auto prefetch_q = [&](int it) {
        const int pr = it % npair, heads = min(2, rho - 2 * pr);
        for (int h = 0; h < heads; ++h) tma_prefetch_3d(&tmQ, 0, (c0 + it / npair) * kGC, h0 + 2 * pr + h);
      };
      auto load_kv = [&](int c) {
        mbar_arrive_expect_tx(&s.kv_full[c & 1], 2 * kTileBytes);
        tma_load_3d(s.k[c & 1], &tmK, &s.kv_full[c & 1], 0, (c0 + c) * kGC, bh);
        tma_load_3d(s.v[c & 1], &tmV, &s.kv_full[c & 1], 0, (c0 + c) * kGC, bh);
      };
      int kv_loads = 0, q_loads = 0;
      if (lane == 0) {
        for (; kv_loads < min(2, nc); ++kv_loads) load_kv(kv_loads);
        for (; q_loads < min(2, steps); ++q_loads) load_q(q_loads);
      }
      const uint64_t sd = sdesc_sw128(smem_u32(s.state), 16, 1024);
      // X of step it, while the step before writes its outputs
      auto issue_x = [&](int it) {
        const int c = it / npair;
        if (!warp_wait(&s.q_full[it & 1], (it >> 1) & 1, &s.wait) ||
            !warp_wait(&s.kv_full[c & 1], (c >> 1) & 1, &s.wait))
          return false;
        const uint64_t qd = sdesc_sw128(smem_u32(s.q[it & 1]), 16, 1024);
        const uint64_t kd = sdesc_sw128(smem_u32(s.k[c & 1]), 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_ss_warp(tb + kColX, qd + 2 * k, kd + 2 * k, id_k, k > 0);
        umma_commit_warp(&s.x_full);
        return true;
      };
      const float *g = p.g + (size_t)bh * p.T;
      float2 gate = gate_load(g, c0 * kGC, n);
      auto make_gates = [&](int c) {
        const float2 now = gate;
        if (c + 1 < nc) gate = gate_load(g, (c0 + c + 1) * kGC, n);
        float2 tail;
        chunk_gates<false>(now, gate_sums(now), s.gates[c & 1], tail, careful);
        weights_put(s.tail[c & 1], tail.x, tail.y);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.gate_full);
      };
      __syncwarp();
      if (nc > 0) make_gates(0);
      bool ok = steps == 0 || issue_x(0);
#pragma unroll 1
      for (int it = 0; it < steps && ok; ++it) {
        const int c = it / npair, pr = it % npair;
        // the step before is done: its D is read, its outputs and (a new chunk)
        // the state are in shared memory
        ok = warp_wait(&s.go, it & 1, &s.wait);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = sdesc_sw128(smem_u32(s.q[it & 1]), 16, 1024);
        const uint64_t vd = sdesc_sw128(smem_u32(s.v[c & 1]), 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_ss_warp(tb + kColD, qd + 2 * k, sd + 128 * k, id_mn, k > 0);
        umma_commit_warp(&s.d_full);
        if (lane == 0) {
          if (pr == 0 && c > 0 && c + 1 < nc) load_kv(c + 1), ++kv_loads;
          if (it + 2 < steps) prefetch_q(it + 2);
        }
        __syncwarp();
        ok = warp_wait(&s.p_full, it & 1, &s.wait);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_ts_warp(tb + kColD, tb + kColX + 8 * k, vd + 128 * k, id_mn, 1u);
        umma_commit_warp(&s.y_full);
        // the outputs of the step before have left their buffer (p_full says so)
        if (lane == 0 && it > 0 && it + 1 < steps) load_q(it + 1), ++q_loads;
        __syncwarp();
        // P, which lies in X, has been read
        if (it + 1 < steps) ok = warp_wait(&s.y_full, it & 1, &s.wait) && issue_x(it + 1);
        if (pr == 0 && c + 1 < nc) make_gates(c + 1);
      }
      umma_commit_warp(&s.drain);
      if (lane == 0) {   // nothing in flight at the block's end
        mbar_wait_teardown(&s.drain, 0, p.status);
        for (int i = max(0, kv_loads - 2); i < kv_loads; ++i) mbar_wait_teardown(&s.kv_full[i & 1], (i >> 1) & 1, p.status);
        for (int i = max(0, q_loads - 2); i < q_loads; ++i) mbar_wait_teardown(&s.q_full[i & 1], (i >> 1) & 1, p.status);
      }
      __syncwarp();
    } else {
      const int i = tid & 63, half = warp & 1;            // token of this thread's row, its 32-token half
      const uint32_t tm = tb + ((uint32_t)(32 * warp) << 16);
      StateAcc<8> acc;
      state_load(acc, 0, p.seg_state + ((size_t)bh * p.nseg + seg) * kGS);
      state_round(acc, 0, s.state);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.go);
      float row = 0.f;                                      // factor of the row's result
      float in = 1.f, into = 1.f;                          // of its scores, and (kHalves) of S_in^T q_i
      uint32_t wrong = 0u;                                 // 0, or NaN once a result was not finite
      int begin = 0, mode = kPlain;                        // first key of the row
      bool ok = true;
      // the four computing warps meet (a wait that ends, unlike a barrier of threads)
      int met = 0;
      auto meet = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.meet);
        return warp_wait(&s.meet, met++ & 1, &s.wait);
      };
#pragma unroll 1
      for (int it = 0; it < steps && ok; ++it) {
        const int c = it / npair, pr = it % npair, t0 = (c0 + c) * kGC;
        const ChunkGates &gates = s.gates[c & 1];
        if (pr == 0) {
          ok = warp_wait(&s.gate_full, c & 1, &s.wait);
          if (!ok) break;
          mode = gates.mode;
          const float r = gates.row[i];
          row = mode == kPlain ? p.scale * r : p.scale;
          in = mode == kPlain ? 1.f : r;
          begin = 0;
          into = half ? r * gates.first : r;
          if (cut_before(gates, i, begin)) into = 0.f;     // keys from the row's last cut gate on, nothing from S_in
          ok = warp_wait(&s.kv_full[c & 1], (c >> 1) & 1, &s.wait);
        }
        ok = ok && warp_wait(&s.x_full, it & 1, &s.wait);
        if (!ok) break;
        tc_fence_after();
        if (pr == 0 && t0 + kGC > n) {                     // rows behind the sequence count as zeros
          clear_rows(s.k[c & 1], n - t0, tid, 128);
          clear_rows(s.v[c & 1], n - t0, tid, 128);
          fence_proxy_async();
          ok = meet();
          if (!ok) break;
        }
        if (mode != kEach) {
          // P's columns lie in front of the X still to be read: first the first
          // half's keys for rows of the second, then the keys of the row's own half
          uint32_t x[2][16], pk[16];
          if (half) {
            tmem_ld16(tm + kColX, x[0]);
            tmem_ld16(tm + kColX + 16, x[1]);
            tmem_wait_ld();
            if (mode == kHalves) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e >> 4][e & 15] = e >= begin ? x[e >> 4][e & 15] : 0u;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 r = *reinterpret_cast<const float4 *>(gates.before + 16 * h + e);
                pk[8 * h + (e >> 1)] =
                    pack_bf16x2(__uint_as_float(x[h][e]) * (in * r.x), __uint_as_float(x[h][e + 1]) * (in * r.y));
                pk[8 * h + (e >> 1) + 1] =
                    pack_bf16x2(__uint_as_float(x[h][e + 2]) * (in * r.z), __uint_as_float(x[h][e + 3]) * (in * r.w));
              }
            tmem_st16(tm + kColX, pk);
          }
          const uint32_t mask = (0xFFFFFFFFu >> (31 - lane)) & (0xFFFFFFFFu << max(0, begin - 32 * half));   // begin <= i
          tmem_ld16(tm + kColX + 32 * half, x[0]);
          tmem_ld16(tm + kColX + 32 * half + 16, x[1]);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 r = *reinterpret_cast<const float4 *>(gates.rest + 32 * half + 16 * h + e);
              const int j = 16 * h + e;
              pk[8 * h + (e >> 1)] = pack_bf16x2(mask & (1u << j) ? __uint_as_float(x[h][e]) * (in * r.x) : 0.f,
                                                 mask & (1u << (j + 1)) ? __uint_as_float(x[h][e + 1]) * (in * r.y) : 0.f);
              pk[8 * h + (e >> 1) + 1] =
                  pack_bf16x2(mask & (1u << (j + 2)) ? __uint_as_float(x[h][e + 2]) * (in * r.z) : 0.f,
                              mask & (1u << (j + 3)) ? __uint_as_float(x[h][e + 3]) * (in * r.w) : 0.f);
            }
          tmem_st16(tm + kColX + 16 * half, pk);
          if (!half) {
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = 0u;
            tmem_st16(tm + kColX + 16, pk);
          }
        } else {
          ok = warp_wait(&s.d_full, it & 1, &s.wait);
          if (!ok) break;
          tc_fence_after();
          slow_scores(p.g + (size_t)bh * p.T, t0, n, i, tm);
        }
        if (mode == kHalves) {
          ok = warp_wait(&s.d_full, it & 1, &s.wait);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            uint32_t x[16];
            tmem_ld16(tm + kColD + 16 * h, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = into == 0.f ? 0u : __float_as_uint(__uint_as_float(x[e]) * into);
            tmem_st16(tm + kColD + 16 * h, x);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          bulk_wait_read();                                // the outputs of the step before are out of shared memory
          mbar_arrive(&s.p_full);
        }
        // the state, while P V runs: half of the chunk with its first pair, the rest with its last
        if (pr == 0) {
          state_scale(acc, gates.whole);
          state_add<0, 2>(acc, 0, s.k[c & 1], s.v[c & 1], s.tail[c & 1]);
        }
        if (pr == npair - 1) {
          state_add<2, 4>(acc, 0, s.k[c & 1], s.v[c & 1], s.tail[c & 1]);
          ok = warp_wait(&s.d_full, it & 1, &s.wait);   // the chunk's last Q S_in is done
          if (!ok) break;
          state_round(acc, 0, s.state);
        }
        ok = warp_wait(&s.y_full, it & 1, &s.wait);
        if (!ok) break;
        tc_fence_after();
        const int hd = 2 * pr + (warp >> 1);
        const bool rows = by_rows(t0);
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.Y) + ((size_t)(h0 + hd) * p.T + t0 + i) * 64);
        uint8_t *tile = s.q[it & 1] + (warp >> 1) * kTileBytes;
        uint32_t x[4][16];
#pragma unroll
        for (int h = 0; h < 4; ++h) tmem_ld16(tm + kColD + 16 * h, x[h]);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = pack_bf16x2(__uint_as_float(x[h][2 * e]) * row, __uint_as_float(x[h][2 * e + 1]) * row);
          if (hd < rho && t0 + i < n)
#pragma unroll
            for (int e = 0; e < 8; ++e) wrong = bf2_fma(y[e], 0u, wrong);
          const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
          if (!rows) {
            *reinterpret_cast<uint4 *>(tile + tile_at(i, 2 * h)) = lo;
            *reinterpret_cast<uint4 *>(tile + tile_at(i, 2 * h + 1)) = hi;
          } else if (hd < rho && t0 + i < n) {
            dst[2 * h] = lo;
            dst[2 * h + 1] = hi;
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!rows && hd < rho && t0 + 32 * half < n) tma_store_3d(&tmY, tile + 32 * half * 128, 0, t0 + 32 * half, h0 + hd);
          bulk_commit();
          mbar_arrive(&s.go);
        }
      }
      if (lane == 0) bulk_wait_all();
      if (wrong & 0x7FFF7FFFu) s.again = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (careful || !s.again || s.wait.abort) break;
    // once more, from the start: nothing is in flight, the barriers begin anew
    tc_fence_after();
    __syncthreads();
    if (tid == 0) {
      uint64_t *bars[] = {&s.kv_full[0], &s.kv_full[1], &s.q_full[0], &s.q_full[1], &s.gate_full, &s.x_full,
                          &s.d_full,     &s.p_full,     &s.y_full,    &s.go,        &s.meet,      &s.drain};
      for (uint64_t *bar : bars) mbar_inval(bar);
      init();
    }
    __syncthreads();
  }
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tb, kOutCols);
  }
}

}  // namespace

oal_status launch_gated_scan(const GatedArgs &p, int ways, bool last, cudaStream_t stream);

oal_status launch_gated_prefill_tc(const GatedArgs &p, cudaStream_t stream) {
  static bool done_seg[kMaxDevices], done_out[kMaxDevices];
  const size_t seg_smem = sizeof(SegSmem) + 1024, out_smem = sizeof(OutSmem) + 1024;
  GATED_TRY(gated_need_smem(reinterpret_cast<const void *>(gated_tc_segment_kernel), seg_smem, done_seg));
  GATED_TRY(gated_need_smem(reinterpret_cast<const void *>(gated_tc_out_kernel), out_smem, done_out));
  CUtensorMap tmQ, tmK, tmV, tmY;
  GATED_TRY(make_map(&tmQ, p.Q, p.T, (long long)p.B * p.Hq));
  GATED_TRY(make_map(&tmK, p.K, p.T, (long long)p.B * p.Hkv));
  GATED_TRY(make_map(&tmV, p.V, p.T, (long long)p.B * p.Hkv));
  GATED_TRY(make_map(&tmY, p.Y, p.T, (long long)p.B * p.Hq, 32));
  const dim3 grid(p.nseg * p.B * p.Hkv);
  launch_pdl(gated_tc_segment_kernel, grid, dim3(kSegThreads), seg_smem, stream, tmK, tmV, p);
  GATED_TRY(oal_after_launch("gated_tc_segment_kernel", stream));
  GATED_TRY(launch_gated_scan(p, 1, true, stream));
  launch_pdl(gated_tc_out_kernel, grid, dim3(kOutThreads), out_smem, stream, tmQ, tmK, tmV, tmY, p);
  return oal_after_launch("gated_tc_out_kernel", stream);
}

}  // namespace oal
