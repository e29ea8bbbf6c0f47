// paged_tc.cu -- attention over a paged cache for bf16 on the tensor cores
// (tcgen05), for chunks of new tokens.
//
// A block takes two tiles of 128 rows (row h' * nt + t': nt tokens of all rho
// query heads of a KV head) over the keys that they see, 128 keys at a time:
//     S = Q K^T                 tcgen05, operands as TMA left them
//     P = 2^{s - m} (bf16)      four warps a tile, a row a thread: tensor memory -> registers -> tensor memory
//     O += P V                  tcgen05, P from tensor memory
// One warp loads keys and one values (a page is a box of TMA's, or part of one),
// one issues the first product and one the second: a wait on a barrier that is
// complete costs an issuing warp about 130 cycles beside MMAs that read shared
// memory, and one warp for both took 1,320 cycles for the 512 of its MMAs.  P lies
// beside S, so that the next scores of a tile come as soon as its warps have
// taken the present ones into registers.
//
// m is the row's maximum at some time, at most 2^8 below the present one: O is
// multiplied by a power of two (through registers) only when it falls behind
// further, which after the first keys is rare.
//
// What bounds it: 512 cycles of MMA and as many of the exponentials' units for
// 128 x 128 scores.
#include <algorithm>

#include "gated_tc.cuh"
#include "paged.cuh"

namespace oal {
namespace {
using namespace gated;

constexpr int kTcThreads = 384;           // two tiles' warps, and four that load and issue
constexpr int kLoadK = 8, kScoreWarp = 9, kValueWarp = 10, kLoadV = 11;
constexpr int kKeys = 128;
constexpr int kTile = 128 * 128;          // bytes of 128 rows of 64
constexpr int kRing = 4;                  // key tiles in flight, of K and of V
constexpr uint32_t kColP = 256, kColO = 384;   // tensor memory: S of each tile (128 columns), P (64), O (64)
constexpr float kBehind = 8.f;
// Up to here tanh(f) = f (c0 + c1 f^2 + .. + c4 f^8) to 6e-8, by least squares at
// Chebyshev's points: no exponential and no division, whose units the softmax
// needs.  64 chats of up to 201 tokens, cap 30, window 1024: 140 us without it.
constexpr float kTanhSpan = 0.625f;

struct TcSmem {
  uint8_t q[2][kTile], k[kRing][kTile], v[kRing][kTile];
  uint64_t q_full, k_full[kRing], k_free[kRing], v_full[kRing], v_free[kRing], v_raw;
  uint64_t s_full[2], s_read[2], p_full[2], o_done[2], drain[2];
  int lo[8], hi[8];                       // keys that the rows of each warp see
  uint32_t tmem;
  WaitState wait;
};
constexpr size_t kTcBytes = sizeof(TcSmem) + 1024;

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// 32 columns of the thread's row, and the maximum of those that are numbers (of
// their amounts)
template <bool kAbs>
__device__ __forceinline__ float tmem_ld32_max(uint32_t taddr, uint32_t *r) {
  float top;
#define OAL_LD32_MAX(abs)                                                                                              \
  asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x32.max" abs                                                        \
               ".f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"  \
               "%26,%27,%28,%29,%30,%31}, %32, [%33];"                                                                 \
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),       \
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),              \
                 "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),            \
                 "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),            \
                 "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(top)                                                      \
               : "r"(taddr))
  if (kAbs)
    OAL_LD32_MAX(".abs");
  else
    OAL_LD32_MAX("");
#undef OAL_LD32_MAX
  return top;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The key tiles of the block's two tiles of rows, whose products are issued by
// key tile, first tile first.
// (Selected, not indexed: an index would put them into local memory, and what
// is loaded from there is not known to be the same in all lanes.)
struct TcWork {
  int from0, to0, from1, to1;             // key tiles
  __device__ __forceinline__ int from(int x) const { return x ? from1 : from0; }
  __device__ __forceinline__ int to(int x) const { return x ? to1 : to0; }
  __device__ __forceinline__ bool has(int x, int j) const { return j >= from(x) && j < to(x); }
};

// kCap: scores are capped; kBias: they take a distance.
template <bool kCap, bool kBias>
__global__ void __launch_bounds__(kTcThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, PagedArgs p, int nt) {
  constexpr bool kExtra = kCap || kBias;
  extern __shared__ uint8_t smem_raw[];
  TcSmem &s = *reinterpret_cast<TcSmem *>(align1024(smem_raw));
  const uint32_t units = (uint32_t)(p.B * p.Hkv);
  const int bh = blockIdx.x % units, b = bh / p.Hkv, kv = bh % p.Hkv, split = blockIdx.y;
  const int t0 = (gridDim.x / units - 1 - blockIdx.x / units) * 2 * nt;   // the last tokens, which see most, first
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  if (tid == 0) {
    s.wait.abort = 0;
    s.wait.status = p.status;
    mbar_init(&s.q_full, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&s.k_full[i], 1), mbar_init(&s.k_free[i], 1);
      mbar_init(&s.v_full[i], 1), mbar_init(&s.v_free[i], 1);
    }
    mbar_init(&s.v_raw, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1), mbar_init(&s.s_read[i], 4);
      mbar_init(&s.p_full[i], 4), mbar_init(&s.o_done[i], 1);
      mbar_init(&s.drain[i], 1);
    }
    fence_mbar_init();
  }
  pdl_wait();
  const PagedSeq seq = paged_seq(p, b, tid == 0);
  if (t0 >= seq.n) return;
  if (warp == kScoreWarp) {
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  int from = 0, to = INT32_MAX;
  if (p.splits > 1) {
    from = paged_base(p, seq, t0) + split * p.split_keys;
    to = from + p.split_keys;
  }
  // the thread's row, and the keys that it sees
  const int x = warp >> 2, r = tid & 127;                    // (warps 0 .. 7)
  const int h1 = r / nt, t = t0 + x * nt + r % nt;
  const bool live = warp < 8 && h1 < p.rho && t < seq.n;
  int2 sees = make_int2(0, 0);
  if (warp < 8) {
    if (live) sees = paged_sees(p, seq, b, t);
    const int a = max(sees.x, from), z = min(sees.y, to);
    const int lo = __reduce_min_sync(0xffffffffu, a < z ? a : INT32_MAX);
    const int hi = __reduce_max_sync(0xffffffffu, a < z ? z : 0);
    if (lane == 0) s.lo[warp] = lo, s.hi[warp] = hi;
  }
  // rows behind the last token's: scores of 0
  for (int e = nt * p.rho * 8 + tid; e < 128 * 8; e += kTcThreads)
    reinterpret_cast<uint4 *>(s.q[0])[e] = reinterpret_cast<uint4 *>(s.q[1])[e] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // (not before: what comes behind must not hold tensor memory that this block waits for)
  const uint32_t tb = uniform(s.tmem);
  const int lo0 = min(min(s.lo[0], s.lo[1]), min(s.lo[2], s.lo[3])), hi0 = max(max(s.hi[0], s.hi[1]), max(s.hi[2], s.hi[3]));
  const int lo1 = min(min(s.lo[4], s.lo[5]), min(s.lo[6], s.lo[7])), hi1 = max(max(s.hi[4], s.hi[5]), max(s.hi[6], s.hi[7]));
  const int lo = uniform(min(lo0, lo1)), hi = uniform(max(hi0, hi1));
  TcWork work;
  work.from0 = uniform(hi0 > 0 ? lo0 / kKeys : 0), work.to0 = uniform((hi0 + kKeys - 1) / kKeys);
  work.from1 = uniform(hi1 > 0 ? lo1 / kKeys : 0), work.to1 = uniform((hi1 + kKeys - 1) / kKeys);
  const bool one = work.to0 > 0, two = work.to1 > 0;
  if (one && two) {                       // no key tile between them without a user: the rings go by key tiles
    work.to0 = max(work.to0, work.from1);
    work.to1 = max(work.to1, work.from0);
  }
  const int j_first = !one ? work.from1 : !two ? work.from0 : min(work.from0, work.from1);
  const int j_last = max(work.to0, work.to1);

  if (warp == kLoadK || warp == kLoadV) {
    const bool keys = warp == kLoadK;
    uint64_t *full = keys ? s.k_full : s.v_full, *free = keys ? s.k_free : s.v_free;
    uint8_t *ring = keys ? s.k[0] : s.v[0];
    const CUtensorMap *map = keys ? &tmK : &tmV;
    if (keys && lane == 0 && j_first < j_last) {
      const int bytes = nt * p.rho * 128;
      mbar_arrive_expect_tx(&s.q_full, (one ? bytes : 0) + (two ? bytes : 0));
      if (one) tma_load_4d(s.q[0], &tmQ, &s.q_full, 0, t0, 0, bh);
      if (two) tma_load_4d(s.q[1], &tmQ, &s.q_full, 0, t0 + nt, 0, bh);
    }
    // a lane loads a page's part of the tile
    const int page_rows = min(1 << p.page_shift, kKeys), boxes = kKeys / page_rows;
    auto page_of = [&](int j) {           // none: zeros
      const int key = j * kKeys + lane * page_rows;
      if (lane >= boxes || j >= j_last || key + page_rows <= lo || key >= hi) return -1;
      return paged_page(p, b, key);
    };
    bool ok = true;
    int loads = 0, raw = 0, raw_at = -1;  // raw: tiles that were cleared; the last of them, if it is not handed over
    int page = page_of(j_first);
#pragma unroll 1
    for (int j = j_first; j < j_last; ++j) {
      const int st = loads % kRing, round = loads / kRing;
      const int at = page >= 0 ? page : max(p.n_pages, 1);
      const int y = (j * kKeys + lane * page_rows) & ((1 << p.page_shift) - 1);
      page = page_of(j + 1);
      if (round > 0) ok = warp_wait(&free[st], (round - 1) & 1, &s.wait);
      if (!ok) break;
      // values outside of what the rows see meet weights of 0, which an infinity or NaN would survive: zeros
      const bool edge = !keys && (j * kKeys < lo || (j + 1) * kKeys > hi);
      uint64_t *bar = edge ? &s.v_raw : &full[st];
      if (lane == 0) mbar_arrive_expect_tx(bar, kTile);
      __syncwarp();
      if (lane < boxes) tma_load_4d(ring + st * kTile + lane * page_rows * 128, map, bar, 0, y, kv, at);
      ++loads;
      if (edge) {
        raw_at = loads - 1;
        ok = warp_wait(bar, raw++ & 1, &s.wait);
        if (!ok) break;
        for (int e = lane; e < kKeys * 8; e += 32) {
          const int key = j * kKeys + (e >> 3);
          if (key < lo || key >= hi) reinterpret_cast<uint4 *>(ring + st * kTile)[e] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        raw_at = -1;
      }
    }
    if (lane == 0) {                      // nothing in flight at the block's end
      if (keys && j_first < j_last) mbar_wait_teardown(&s.q_full, 0, p.status);
      if (raw_at >= 0) mbar_wait_teardown(&s.v_raw, (raw - 1) & 1, p.status);
      for (int i = max(0, loads - kRing); i < loads; ++i)
        if (i != raw_at) mbar_wait_teardown(&full[i % kRing], (i / kRing) & 1, p.status);
    }
    __syncwarp();
  } else if (warp == kScoreWarp || warp == kValueWarp) {
    // The tiles' scores (values) in their order; j, x: the present ones
    const uint64_t rest = sdesc_sw128(0, 16, 1024);
    auto desc = [&](const uint8_t *at) { return rest | (uint64_t)uniform(smem_u32(at) >> 4); };   // (below 2^18)
    auto step = [&](int &j, int &x) {
      do {
        if (++x == 2) x = 0, ++j;
      } while (j < j_last && !work.has(x, j));
    };
    int j = j_first, x = work.has(0, j_first) ? 0 : 1, st = 0, round = 0;
    bool ok = true, fresh = true;         // fresh: the ring's tile is not known to be there
    if (warp == kScoreWarp) {
      const uint32_t id = idesc_bf16_f32(128, kKeys, 0);
      int n0 = 0, n1 = 0;                 // scores of each tile
      if (j < j_last) ok = warp_wait(&s.q_full, 0, &s.wait);
#pragma unroll 1
      while (j < j_last && ok) {
        const int n = x ? n1 : n0;
        if (fresh) ok = warp_wait(&s.k_full[st], round & 1, &s.wait);
        if (n > 0) ok = ok && warp_wait(&s.s_read[x], (n - 1) & 1, &s.wait);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = desc(s.q[x]), kd = desc(s.k[st]);
        const uint32_t to_s = uniform(tb + 128 * x);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_ss_warp(to_s, qd + 2 * k, kd + 2 * k, id, k > 0);
        umma_commit_warp(&s.s_full[x]);
        n0 += 1 - x, n1 += x;
        const int before = j;
        step(j, x);
        fresh = j != before;
        if (fresh) {
          umma_commit_warp(&s.k_free[st]);
          if (++st == kRing) st = 0, ++round;
        }
      }
    } else {
      const uint32_t id = idesc_bf16_f32(128, 64, 1);
      int n0 = 0, n1 = 0;                 // products of each tile
#pragma unroll 1
      while (j < j_last && ok) {
        const int n = x ? n1 : n0;
        if (fresh) ok = warp_wait(&s.v_full[st], round & 1, &s.wait);
        ok = ok && warp_wait(&s.p_full[x], n & 1, &s.wait);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = desc(s.v[st]);
        const uint32_t from_p = uniform(tb + kColP + 64 * x), to_o = uniform(tb + kColO + 64 * x), more = n > 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_ts_warp(to_o, from_p + 8 * k, vd + 128 * k, id, k > 0 ? 1u : more);
        umma_commit_warp(&s.o_done[x]);
        n0 += 1 - x, n1 += x;
        const int before = j;
        step(j, x);
        fresh = j != before;
        if (fresh) {
          umma_commit_warp(&s.v_free[st]);
          if (++st == kRing) st = 0, ++round;
        }
      }
    }
    uint64_t *drain = &s.drain[warp == kValueWarp];
    umma_commit_warp(drain);
    if (lane == 0) mbar_wait_teardown(drain, 0, p.status);
    __syncwarp();
  } else {
    const uint32_t tm = tb + ((uint32_t)(32 * (warp & 3)) << 16), to_o = tm + kColO + 64 * x;
    const int h = kv * p.rho + h1;
    const float scale2 = p.scale * kLog2e;
    const float cap_in = kCap ? 2.f * kLog2e * p.scale / p.cap : 0.f, cap_out = p.cap * kLog2e;
    const float in_cap = kCap ? p.scale / p.cap : 0.f;
    auto times = [&](float c) { return pair(c * cap_out, c * cap_out); };
    const uint64_t tanh0 = times(0.9999998807907104f), tanh1 = times(-0.3333197236061096f), tanh2 = times(0.13304771482944489f),
                   tanh3 = times(-0.05183185636997223f), tanh4 = times(0.015063672326505184f);
    const float slope = kBias && live ? p.slopes[h] * kLog2e : 0.f;
    const float by = kExtra ? 1.f : scale2;                // of what is held as a score
    // (a row that is none is not to make the others look at masks)
    const int see0 = live ? max(sees.x, from) : 0, see1 = live ? min(sees.y, to) : INT32_MAX;
    float m = -INFINITY;
    uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
    bool ok = true;
    int n = 0;                                               // the tile's key tiles so far
#pragma unroll 1
    for (int j = work.from(x); j < work.to(x); ++j, ++n) {
      const int j0 = j * kKeys;
      ok = warp_wait(&s.s_full[x], n & 1, &s.wait);
      if (!ok) break;
      tc_fence_after();
      uint32_t w[128];
      float top[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) top[c] = tmem_ld32_max<kCap>(tm + 128 * x + 32 * c, w + 32 * c);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.s_read[x]);            // the next scores may come
      if (kCap) {
        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * in_cap;
        if (__all_sync(0xffffffffu, most <= kTanhSpan)) {
#pragma unroll
          for (int e = 0; e < 128; e += 2) {
            const uint64_t f = mul2(pair(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), pair(in_cap, in_cap)), f2 = mul2(f, f);
            uint64_t q = fma2(f2, tanh4, tanh3);
            q = fma2(q, f2, tanh2), q = fma2(q, f2, tanh1), q = fma2(q, f2, tanh0);
            float a, z;
            unpair(mul2(f, q), a, z);
            w[e] = __float_as_uint(a), w[e + 1] = __float_as_uint(z);
          }
        } else {                            // cap tanh(f) = cap - 2 cap / (e^{2 f} + 1)
#pragma unroll
          for (int e = 0; e < 128; ++e) {
            float z;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(ex2(__uint_as_float(w[e]) * cap_in) + 1.f));
            w[e] = __float_as_uint(fmaf(-2.f * cap_out, z, cap_out));
          }
        }
      }
      if (kBias) {                          // with the scale where no cap has taken it in; packed where no key lies behind its row
        const float far = (float)(seq.past + t - j0), times = kCap ? 1.f : scale2;
        if (__all_sync(0xffffffffu, far >= 127.f)) {
          const uint64_t times2 = pair(times, times), slope2 = pair(slope, slope), start2 = pair(-slope * far, -slope * far);
#pragma unroll
          for (int e = 0; e < 128; e += 2) {
            float a, z;
            unpair(fma2(pair(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), times2,
                        fma2(pair((float)e, (float)(e + 1)), slope2, start2)), a, z);
            w[e] = __float_as_uint(a), w[e + 1] = __float_as_uint(z);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            w[e] = __float_as_uint(fmaf(-slope, fabsf(far - (float)e), __uint_as_float(w[e]) * times));
        }
      }
      const bool cut = !__all_sync(0xffffffffu, see0 <= j0 && see1 >= j0 + kKeys);
      if (cut) {
        const uint32_t off = (uint32_t)(see0 - j0), len = (uint32_t)max(see1 - see0, 0);
#pragma unroll
        for (int e = 0; e < 128; ++e) w[e] = (uint32_t)e - off < len ? w[e] : 0xFF800000u;
      }
      if (kExtra || cut) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          top[c] = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            top[c] = fmaxf(top[c], fmaxf(__uint_as_float(w[32 * c + e]), __uint_as_float(w[32 * c + e + 1])));
        }
      }
      const float now = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
      const bool behind = (now - m) * by > kBehind;          // (from -inf: always)
      if (__any_sync(0xffffffffu, behind)) {
        const float keep = behind ? ex2((m - now) * by) : 1.f;
        if (behind) m = now;
        float a, z;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          unpair(sum[c], a, z);
          sum[c] = pair(a * keep, z * keep);
        }
        if (n > 0) {
          ok = warp_wait(&s.o_done[x], (n - 1) & 1, &s.wait);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[16];
            tmem_ld16(to_o + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
            tmem_st16(to_o + 16 * c, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : -m * by;
      const uint64_t by2 = pair(by, by), base2 = pair(base, base);
      // weights, rounded to bf16 because the tensor cores take both factors in the values' type
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float a, z;
          unpair(fma2(pair(__uint_as_float(w[32 * c + e]), __uint_as_float(w[32 * c + e + 1])), by2, base2), a, z);
          a = ex2(a), z = ex2(z);
          sum[e >> 1 & 1] = add2(sum[e >> 1 & 1], pair(a, z));
          w[16 * c + (e >> 1)] = pack_bf16x2(a, z);
        }
        if (c == 0) {                       // the product before is done: P may be written over
          if (n > 0) ok = warp_wait(&s.o_done[x], (n - 1) & 1, &s.wait);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st16(tm + kColP + 64 * x + 16 * c, *reinterpret_cast<uint32_t (*)[16]>(w + 16 * c));
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.p_full[x]);
    }
    float f[4];
    unpair(sum[0], f[0], f[1]), unpair(sum[1], f[2], f[3]);
    const float total = (f[0] + f[1]) + (f[2] + f[3]);
    if (n > 0 && ok) ok = warp_wait(&s.o_done[x], (n - 1) & 1, &s.wait);
    if (ok) {
      tc_fence_after();
      bool wrong = false;
      const size_t row = ((size_t)bh * p.splits + split) * ((size_t)p.T * p.rho) + (size_t)t * p.rho + h1;
      const float inv = see0 < see1 ? 1.f / total : 0.f;
      if (p.splits > 1 && live) p.part_ml[row] = make_float2(m == -INFINITY ? m : m * by, total);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[16];
        if (n > 0) {
          tmem_ld16(to_o + 16 * c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0u;
        }
        if (!live) continue;
        if (p.splits > 1) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + row * 64 + 16 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = inv == 0.f ? 0.f : __uint_as_float(o[2 * e]) * inv;
            const float z = inv == 0.f ? 0.f : __uint_as_float(o[2 * e + 1]) * inv;
            wrong |= !(fabsf(a) + fabsf(z) < INFINITY);
            pk[e] = pack_bf16x2(a, z);
          }
          uint4 *dst = reinterpret_cast<uint4 *>(paged_y<__nv_bfloat16>(p, b, h, t) + 16 * c);
          dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]), dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        }
      }
      for (uint32_t again = __ballot_sync(0xffffffffu, wrong); again; again &= again - 1) {
        const int who = __ffs(again) - 1;
        const int h2 = __shfl_sync(0xffffffffu, h, who), t2 = __shfl_sync(0xffffffffu, t, who);
        const int a = __shfl_sync(0xffffffffu, sees.x, who), z = __shfl_sync(0xffffffffu, sees.y, who);
        const float2 y = paged_row_again<__nv_bfloat16>(p, seq, b, h2, t2, a, z);
        __syncwarp();
        *reinterpret_cast<uint32_t *>(paged_y<__nv_bfloat16>(p, b, h2, t2) + 2 * lane) = pack_bf16x2(y.x, y.y);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kScoreWarp) tmem_dealloc(tb, 512);
}

oal_status tc_map(CUtensorMap *m, const void *ptr, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                  const cuuint32_t (&box)[4]) {
  auto fn = encode_fn();
  if (!fn) return oal_fail(OAL_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint32_t es[4] = {1, 1, 1, 1};
  if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return oal_fail(OAL_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  return OAL_OK;
}

template <bool kCap, bool kBias>
oal_status run(const PagedArgs &p, cudaStream_t stream) {
  static bool done[kMaxDevices];
  auto kernel = paged_tc_kernel<kCap, kBias>;
  oal_status st = paged_need_smem(reinterpret_cast<const void *>(kernel), kTcBytes, done);
  if (st != OAL_OK) return st;
  const int nt = p.tile_rows / (2 * p.rho);
  CUtensorMap mq, mk, mv;
  st = tc_map(&mq, p.Q, {64, (cuuint64_t)p.T, (cuuint64_t)p.rho, (cuuint64_t)p.B * p.Hkv},
              {128, (cuuint64_t)p.T * 128, (cuuint64_t)p.T * p.rho * 128}, {64, (cuuint32_t)nt, (cuuint32_t)p.rho, 1});
  const cuuint64_t page = (cuuint64_t)1 << p.page_shift;
  const cuuint64_t dims[4] = {64, page, (cuuint64_t)p.Hkv, (cuuint64_t)std::max(p.n_pages, 1)};
  const cuuint64_t strides[3] = {128, page * 128, (cuuint64_t)p.page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min<cuuint64_t>(page, kKeys), 1, 1};
  if (st == OAL_OK) st = tc_map(&mk, p.Kp, dims, strides, box);
  if (st == OAL_OK) st = tc_map(&mv, p.Vp, dims, strides, box);
  if (st != OAL_OK) return st;
  const dim3 grid((unsigned)((long long)p.B * p.Hkv * ((p.T + 2 * nt - 1) / (2 * nt))), (unsigned)p.splits);
  launch_pdl(kernel, grid, dim3(kTcThreads), kTcBytes, stream, mq, mk, mv, p, nt);
  st = oal_after_launch("paged_tc_kernel", stream);
  return st != OAL_OK || p.splits == 1 ? st : launch_paged_join(p, 1, stream);
}

}  // namespace

// Rows of a block: two tiles of as many tokens as fit.
int paged_tc_rows(int T, int rho) { return 2 * rho * std::min(T, 128 / rho); }

oal_status launch_paged_tc(const PagedArgs &p, cudaStream_t stream) {
  if (p.cap > 0.f) return p.slopes ? run<true, true>(p, stream) : run<true, false>(p, stream);
  return p.slopes ? run<false, true>(p, stream) : run<false, false>(p, stream);
}

}  // namespace oal
