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
// The launch has a block for every pair of tiles; one that has loaded its keys asks
// for the work of one that has not started (cluster launch control), whose scores
// are there when the results of the first leave: 4 x 8192 tokens, 32/8 heads, 845
// to 865 us from box to box (1.3 PFLOP/s), with blocks that end 8% more.  Asked for
// at a block's start, work went to blocks that were longer at theirs (documents 18.4
// -> 24 us).
//
// m is the row's maximum at some time, at most 2^8 below the present one: O is
// multiplied by a power of two (through registers) only when it falls behind
// further, which after the first keys is rare.
//
// What bounds it: for 128 x 128 scores of both tiles 1,024 cycles of MMAs, 1,024 of
// the exponentials' units, 1,400 of the softmax's instructions with nothing to wait
// for; a whole launch takes 1,780 for each (2048 tokens on 63488 keys, three items a
// block) or 1,830 (4 x 8192, 27 items), items' starts and ends among them; what else
// the other 300 go to is not known.  The loop of a row's scores needs nearly all
// registers: a few more values that live across it (the row's head, its place) cost
// 15% in spilled ones, so they are formed again behind it.  (With caps or distances 16
// to 32 bytes are stored apart, 24 to 68 loaded.)
#include <stddef.h>

#include <algorithm>

#include "gated_tc.cuh"
#include "paged_again.cuh"

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

// Two tiles of rows and the keys that they see: what a block works on next.
struct TcItem {
  int bh, t0, split;                      // bh: -1 = no more
  int n, past, total;                     // the sequence
  int from, to;                           // the split's keys
  int lo, hi, from0, to0, from1, to1;     // keys and key tiles that rows see
};
struct TcSmem {
  uint8_t q[2][kTile], k[kRing][kTile], v[kRing][kTile];
  uint64_t q_full, q_free, k_full[kRing], k_free[kRing], v_full[kRing], v_free[kRing], v_raw;
  uint64_t s_full[2], s_read[2], p_full[2], o_done[2], drain[2];
  uint64_t item_full[2], item_free[2], next_full;
  ulonglong2 next;                        // the answer to a request for another block's work
  TcItem item[4];                         // the present one, the next, and two whose rows may be formed again
  uint32_t again[4][8];                   // their rows whose result is not finite, by warp
  int stop;                               // there are such: no more items
  uint32_t tmem;
  WaitState wait;
  // (only where a split has more than kFold key tiles)
  float fold_l[256], fold_o[2][64][128];  // sums and results of the key tiles so far, by row
};
// The tensor cores cut what they add to an accumulator instead of rounding it, a
// loss in proportion to the keys: values of one sign came out 6e-4 low after 65536
// keys, 6.6e-3 after 2^20.  So O starts anew every kFold key tiles (1.3e-4), and
// what it held is added in fp32 to a sum in shared memory, a row a thread.
constexpr int kFold = 128;
constexpr size_t kTcBytes = offsetof(TcSmem, fold_l) + 1024, kTcFoldBytes = sizeof(TcSmem) + 1024;
static_assert(kTcFoldBytes <= 227 * 1024, "shared memory of a block");

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

// The key tiles of an item's two tiles of rows, whose products are issued by key
// tile, first tile first.
// (Selected, not indexed: an index would put them into local memory, and what
// is loaded from there is not known to be the same in all lanes.)
struct TcWork {
  int from0, to0, from1, to1;             // key tiles
  int first, last;                        // of both
  __device__ __forceinline__ int from(int x) const { return x ? from1 : from0; }
  __device__ __forceinline__ int to(int x) const { return x ? to1 : to0; }
  __device__ __forceinline__ bool has(int x, int j) const { return j >= from(x) && j < to(x); }
  __device__ __forceinline__ void step(int &j, int &x) const {
    do {
      if (++x == 2) x = 0, ++j;
    } while (j < last && !has(x, j));
  }
};
__device__ __forceinline__ TcWork tc_work(const TcItem &i) {
  TcWork w;
  w.from0 = uniform(i.from0), w.to0 = uniform(i.to0), w.from1 = uniform(i.from1), w.to1 = uniform(i.to1);
  w.first = w.to0 == 0 ? w.from1 : w.to1 == 0 ? w.from0 : min(w.from0, w.from1);
  w.last = max(w.to0, w.to1);
  return w;
}

// Asks for the work of a block of this launch that has not started, which then
// never does (PTX's cluster launch control); the answer completes 16 bytes on bar.
__device__ __forceinline__ void next_ask(ulonglong2 *answer, uint64_t *bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ bool next_read(const ulonglong2 &answer, int &x, int &y) {
  uint32_t got;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\tmov.b128 a, {%3, %4};\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\tselp.u32 %0, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::y.b32.b128 %2, a;\n\t}"
      : "=r"(got), "=r"(x), "=r"(y)
      : "l"(answer.x), "l"(answer.y));
  return got != 0;
}

// kCap: scores are capped; kBias: they take a distance; kFolds: a split has more
// than kFold key tiles (kernels of their own: the code that others do not run cost
// them 1 to 6%).
template <bool kCap, bool kBias, bool kFolds>
__global__ void __launch_bounds__(kTcThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, PagedArgs p, int nt) {
  constexpr bool kExtra = kCap || kBias;
  extern __shared__ uint8_t smem_raw[];
  TcSmem &s = *reinterpret_cast<TcSmem *>(align1024(smem_raw));
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  if (tid == 0) {
    s.wait.abort = 0, s.stop = 0;
    s.wait.status = p.status;
    mbar_init(&s.q_full, 1), mbar_init(&s.q_free, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&s.k_full[i], 1), mbar_init(&s.k_free[i], 1);
      mbar_init(&s.v_full[i], 1), mbar_init(&s.v_free[i], 1);
    }
    mbar_init(&s.v_raw, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1), mbar_init(&s.s_read[i], 4);
      mbar_init(&s.p_full[i], 4), mbar_init(&s.o_done[i], 1);
      mbar_init(&s.drain[i], 1);
      mbar_init(&s.item_full[i], 1), mbar_init(&s.item_free[i], kTcThreads / 32 - 1);
    }
    mbar_init(&s.next_full, 1);
    fence_mbar_init();
  }
  // rows behind the last token's: scores of 0
  for (int e = nt * p.rho * 8 + tid; e < 128 * 8; e += kTcThreads)
    reinterpret_cast<uint4 *>(s.q[0])[e] = reinterpret_cast<uint4 *>(s.q[1])[e] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async();
  pdl_wait();
  if (warp == kScoreWarp) {
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // (not before: what comes behind must not hold tensor memory that this block waits for)
  const uint32_t tb = uniform(s.tmem);
  const int x = warp >> 2;                // the warp's tile (warps 0 .. 7)
  // an item, as every warp but the first loading one takes it: copied, its place free at once
  auto take = [&](int it, TcItem &item) {
    if (!warp_wait(&s.item_full[it & 1], (it >> 1) & 1, &s.wait)) return false;
    item = s.item[it & 3];
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.item_free[it & 1]);
    return uniform(item.bh) != 0xFFFFFFFFu;
  };

  if (warp == kLoadK || warp == kLoadV) {
    const bool keys = warp == kLoadK;
    uint64_t *full = keys ? s.k_full : s.v_full, *free = keys ? s.k_free : s.v_free;
    uint8_t *ring = keys ? s.k[0] : s.v[0];
    const CUtensorMap *map = keys ? &tmK : &tmV;
    bool ok = true;
    int loads = 0, raw = 0, raw_at = -1;  // raw: tiles that were cleared; the last of them, if it is not handed over
    // The item's tiles.  A lane loads a page's part of one.
    const int page_rows = min(1 << p.page_shift, kKeys), boxes = kKeys / page_rows;
    auto load = [&](const TcItem &item) {
      const int b = item.bh / p.Hkv, kv = item.bh % p.Hkv, lo = uniform(item.lo), hi = uniform(item.hi);
      const int j_first = lo / kKeys, j_last = uniform(max(item.to0, item.to1));
      auto page_of = [&](int j) {         // none: zeros
        const int key = j * kKeys + lane * page_rows;
        if (lane >= boxes || j >= j_last || key + page_rows <= lo || key >= hi) return -1;
        return paged_page(p, b, key);
      };
      int page = page_of(j_first);
#pragma unroll 1
      for (int j = j_first; j < j_last; ++j) {
        const int st = loads % kRing, round = loads / kRing;
        const int at = page >= 0 ? page : max(p.n_pages, 1);
        const int y = (j * kKeys + lane * page_rows) & ((1 << p.page_shift) - 1);
        page = page_of(j + 1);
        if (round > 0) ok = warp_wait(&free[st], (round - 1) & 1, &s.wait);
        if (!ok) return;
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
          if (!ok) return;
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
    };
    int queries = 0;                      // items whose queries were loaded
    if (keys) {
      // this warp finds the block's items, its own first, then those of blocks that have not started
      const uint32_t units = (uint32_t)(p.B * p.Hkv);
      int bx = blockIdx.x, by = blockIdx.y, asked = 0;
#pragma unroll 1
      for (int it = 0;;) {
        TcItem item;
        item.bh = bx % units, item.split = by;
        item.t0 = (gridDim.x / units - 1 - bx / units) * 2 * nt;   // the last tokens, which see most, first
        const int b = item.bh / p.Hkv;
        const PagedSeq seq = paged_seq(p, b, lane == 0);
        item.n = seq.n, item.past = seq.past, item.total = seq.total;
        item.from = 0, item.to = INT32_MAX;
        if (p.splits > 1) {
          item.from = paged_base(p, seq, item.t0) + by * p.split_keys;
          item.to = item.from + p.split_keys;
        }
        int lo0 = INT32_MAX, hi0 = 0, lo1 = INT32_MAX, hi1 = 0;
        for (int i = lane; i < 2 * nt && item.t0 + i < seq.n; i += 32) {
          const int2 sees = paged_sees(p, seq, b, item.t0 + i);
          const int a = max(sees.x, item.from), z = min(sees.y, item.to);
          if (a < z && i < nt) lo0 = min(lo0, a), hi0 = max(hi0, z);
          if (a < z && i >= nt) lo1 = min(lo1, a), hi1 = max(hi1, z);
        }
        lo0 = __reduce_min_sync(0xffffffffu, lo0), hi0 = __reduce_max_sync(0xffffffffu, hi0);
        lo1 = __reduce_min_sync(0xffffffffu, lo1), hi1 = __reduce_max_sync(0xffffffffu, hi1);
        item.lo = min(lo0, lo1), item.hi = max(hi0, hi1);
        item.from0 = hi0 > 0 ? lo0 / kKeys : 0, item.to0 = (hi0 + kKeys - 1) / kKeys;
        item.from1 = hi1 > 0 ? lo1 / kKeys : 0, item.to1 = (hi1 + kKeys - 1) / kKeys;
        if (hi0 > 0 && hi1 > 0) {           // no key tile between them without a user: the rings go by key tiles
          item.to0 = max(item.to0, item.from1);
          item.to1 = max(item.to1, item.from0);
        }
        // (nothing to do: no token, or a split that no row's keys reach into, of which nothing is joined)
        if (item.t0 < seq.n && (p.splits == 1 || item.hi > 0)) {
          if (it >= 2) ok = warp_wait(&s.item_free[it & 1], ((it >> 1) - 1) & 1, &s.wait);
          if (!ok) break;
          if (lane == 0) {
            s.item[it & 3] = item;
            mbar_arrive(&s.item_full[it & 1]);
          }
          __syncwarp();
          ++it;
          if (item.hi > 0) {
            if (queries > 0) ok = warp_wait(&s.q_free, (queries - 1) & 1, &s.wait);
            if (!ok) break;
            if (lane == 0) {
              const int bytes = nt * p.rho * 128;
              mbar_arrive_expect_tx(&s.q_full, (hi0 > 0 ? bytes : 0) + (hi1 > 0 ? bytes : 0));
              if (hi0 > 0) tma_load_4d(s.q[0], &tmQ, &s.q_full, 0, item.t0, 0, item.bh);
              if (hi1 > 0) tma_load_4d(s.q[1], &tmQ, &s.q_full, 0, item.t0 + nt, 0, item.bh);
            }
            __syncwarp();
            ++queries;
            load(item);
            if (!ok) break;
          }
        }
        // (asked for when this one's keys are on their way: earlier would take it from a block that is done sooner)
        bool more = !uniform(*(volatile int *)&s.stop);
        if (more) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&s.next_full, 16);
            next_ask(&s.next, &s.next_full);
          }
          __syncwarp();
          ++asked;
          ok = warp_wait(&s.next_full, (asked - 1) & 1, &s.wait);
          if (!ok) break;
          more = next_read(s.next, bx, by);
          bx = uniform(bx), by = uniform(by);
          fence_proxy_async();              // (read before the next answer is written)
          __syncwarp();
        }
        if (!more) {                        // the end, for the others
          if (it >= 2) ok = warp_wait(&s.item_free[it & 1], ((it >> 1) - 1) & 1, &s.wait);
          if (ok && lane == 0) {
            s.item[it & 3].bh = -1;
            mbar_arrive(&s.item_full[it & 1]);
          }
          break;
        }
      }
      if (lane == 0 && asked > 0) mbar_wait_teardown(&s.next_full, (asked - 1) & 1, p.status);
    } else {
      TcItem item;
#pragma unroll 1
      for (int it = 0; ok && take(it, item); ++it)
        if (item.hi > 0) load(item);
    }
    if (lane == 0) {                      // nothing in flight at the block's end
      if (queries > 0) mbar_wait_teardown(&s.q_full, (queries - 1) & 1, p.status);
      if (raw_at >= 0) mbar_wait_teardown(&s.v_raw, (raw - 1) & 1, p.status);
      for (int i = max(0, loads - kRing); i < loads; ++i)
        if (i != raw_at) mbar_wait_teardown(&full[i % kRing], (i / kRing) & 1, p.status);
    }
    __syncwarp();
  } else if (warp == kScoreWarp || warp == kValueWarp) {
    // The tiles' scores (values) in their order; j, y: the present ones
    const uint64_t rest = sdesc_sw128(0, 16, 1024);
    auto desc = [&](const uint8_t *at) { return rest | (uint64_t)uniform(smem_u32(at) >> 4); };   // (below 2^18)
    int st = 0, round = 0, queries = 0;
    int c0 = 0, c1 = 0;                   // scores (products) of each tile so far, of all items
    bool ok = true;
    TcItem item;
#pragma unroll 1
    for (int it = 0; ok && take(it, item); ++it) {
      const TcWork work = tc_work(item);
      if (work.first >= work.last) continue;
      int j = work.first, y = work.has(0, j) ? 0 : 1;
      bool fresh = true;                  // the ring's tile is not known to be there
      if (warp == kScoreWarp) {
        const uint32_t id = idesc_bf16_f32(128, kKeys, 0);
        ok = warp_wait(&s.q_full, queries++ & 1, &s.wait);
#pragma unroll 1
        while (j < work.last && ok) {
          const int c = y ? c1 : c0;
          if (fresh) ok = warp_wait(&s.k_full[st], round & 1, &s.wait);
          if (c > 0) ok = ok && warp_wait(&s.s_read[y], (c - 1) & 1, &s.wait);
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = desc(s.q[y]), kd = desc(s.k[st]);
          const uint32_t to_s = uniform(tb + 128 * y);
#pragma unroll
          for (int k = 0; k < 4; ++k) umma_ss_warp(to_s, qd + 2 * k, kd + 2 * k, id, k > 0);
          umma_commit_warp(&s.s_full[y]);
          c0 += 1 - y, c1 += y;
          const int before = j;
          work.step(j, y);
          fresh = j != before;
          if (fresh) {
            umma_commit_warp(&s.k_free[st]);
            if (++st == kRing) st = 0, ++round;
          }
        }
        umma_commit_warp(&s.q_free);
      } else {
        const uint32_t id = idesc_bf16_f32(128, 64, 1);
#pragma unroll 1
        while (j < work.last && ok) {
          const int c = y ? c1 : c0;
          if (fresh) ok = warp_wait(&s.v_full[st], round & 1, &s.wait);
          ok = ok && warp_wait(&s.p_full[y], c & 1, &s.wait);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = desc(s.v[st]);
          const uint32_t from_p = uniform(tb + kColP + 64 * y), to_o = uniform(tb + kColO + 64 * y), since = (uint32_t)(j - work.from(y));
          const uint32_t more = kFolds ? since & (kFold - 1) : since;   // O holds something to add to
#pragma unroll
          for (int k = 0; k < 8; ++k) umma_ts_warp(to_o, from_p + 8 * k, vd + 128 * k, id, k > 0 ? 1u : more != 0u);
          umma_commit_warp(&s.o_done[y]);
          c0 += 1 - y, c1 += y;
          const int before = j;
          work.step(j, y);
          fresh = j != before;
          if (fresh) {
            umma_commit_warp(&s.v_free[st]);
            if (++st == kRing) st = 0, ++round;
          }
        }
      }
    }
    uint64_t *drain = &s.drain[warp == kValueWarp];
    umma_commit_warp(drain);
    if (lane == 0) mbar_wait_teardown(drain, 0, p.status);
    __syncwarp();
  } else {
    const uint32_t tm = tb + ((uint32_t)(32 * (warp & 3)) << 16), to_o = tm + kColO + 64 * x;
    bool ok = true;
    int count = 0, it = 0;                                   // key tiles so far, of all items; items
    // The thread's row of an item: its query head in the KV head's, its token.  (Formed anew where it is wanted.)
    auto row_of = [&](const TcItem &item, int &h, int &t) {
      int r = tid & 127;
      asm volatile("" : "+r"(r));
      h = r / nt, t = item.t0 + x * nt + (r - h * nt);
      return h < p.rho && t < item.n;
    };
#pragma unroll 1
    for (; ok; ++it) {
      const TcItem &item = s.item[it & 3];                     // (read again at the end: registers are short in between)
      ok = warp_wait(&s.item_full[it & 1], (it >> 1) & 1, &s.wait);
      if (!ok || uniform(item.bh) == 0xFFFFFFFFu) break;
      int see0, see1, at;                                      // the keys that the row sees, its position
      float slope = 0.f;
      {
        int h, t;
        const bool row = row_of(item, h, t);
        PagedSeq seq;
        seq.n = item.n, seq.past = item.past, seq.total = item.total;
        const int2 sees = row ? paged_sees(p, seq, item.bh / p.Hkv, t) : make_int2(0, 0);
        // (a row that is none is not to make the others look at masks)
        see0 = row ? max(sees.x, item.from) : 0, see1 = row ? min(sees.y, item.to) : INT32_MAX;
        at = seq.past + t;
        if (kBias && row) slope = p.slopes[item.bh % p.Hkv * p.rho + h] * kLog2e;
      }
      const int j_from = uniform(x ? item.from1 : item.from0), j_to = uniform(x ? item.to1 : item.to0);
      const float scale2 = p.scale * kLog2e;
      const float cap_in = kCap ? 2.f * kLog2e * p.scale / p.cap : 0.f, cap_out = p.cap * kLog2e;
      const float in_cap = kCap ? p.scale / p.cap : 0.f;
      auto times = [&](float c) { return pair(c * cap_out, c * cap_out); };
      const uint64_t tanh0 = times(kTanh0), tanh1 = times(kTanh1), tanh2 = times(kTanh2), tanh3 = times(kTanh3),
                     tanh4 = times(kTanh4);
      const float by = kExtra ? 1.f : scale2;                // of what is held as a score
      float m = -INFINITY;
      uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll 1
      for (int j = j_from; j < j_to; ++j, ++count) {
        const int j0 = j * kKeys;
        ok = warp_wait(&s.s_full[x], count & 1, &s.wait);
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
          // (The polynomial takes no exponential and no division, whose units the softmax needs: 64 chats of up to 201
          // tokens, cap 30, window 1024, 140 us without it.  What a row that is none holds is not to change the others.)
          if (__all_sync(0xffffffffu, most <= kTanhSpan || see1 == INT32_MAX)) {
#pragma unroll
            for (int e = 0; e < 128; e += 2) {
              const uint64_t f = mul2(pair(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), pair(in_cap, in_cap)), f2 = mul2(f, f);
              uint64_t q = fma2(f2, tanh4, tanh3);
              q = fma2(q, f2, tanh2), q = fma2(q, f2, tanh1), q = fma2(q, f2, tanh0);
              float a, z;
              unpair(mul2(f, q), a, z);
              w[e] = __float_as_uint(a), w[e + 1] = __float_as_uint(z);
            }
          } else if (p.cap <= kCapNear) {
#pragma unroll
            for (int e = 0; e < 128; ++e) w[e] = __float_as_uint(paged_cap_near(__uint_as_float(w[e]), cap_in, cap_out));
          } else {
#pragma unroll
            for (int e = 0; e < 128; ++e) w[e] = __float_as_uint(paged_cap_far(__uint_as_float(w[e]), in_cap, cap_in, cap_out));
          }
        }
        if (kBias) {                          // with the scale where no cap has taken it in; packed where no key lies behind its row
          const float far = (float)(at - j0), times = kCap ? 1.f : scale2;
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
        if (kFolds && j > j_from && ((j - j_from) & (kFold - 1)) == 0) {
          ok = warp_wait(&s.o_done[x], (count - 1) & 1, &s.wait);
          if (!ok) break;
          tc_fence_after();
          const bool more = j - j_from > kFold;
          float a, z, l = more ? s.fold_l[tid] : 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            unpair(sum[c], a, z);
            l += a + z, sum[c] = pair(0.f, 0.f);
          }
          s.fold_l[tid] = l;
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            uint32_t o[16];
            tmem_ld16(to_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float &at = s.fold_o[x][c + e][tid & 127];
              at = __uint_as_float(o[e]) + (more ? at : 0.f);
            }
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
          if (j > j_from) {
            ok = warp_wait(&s.o_done[x], (count - 1) & 1, &s.wait);
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
          if (kFolds && j - j_from >= kFold) {
            s.fold_l[tid] *= keep;
#pragma unroll 4
            for (int c = 0; c < 64; ++c) s.fold_o[x][c][tid & 127] *= keep;
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
            ok = warp_wait(&s.o_done[x], (count & 1) ^ 1, &s.wait);   // (none before: at once)
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
      const bool folded = kFolds && j_to - j_from > kFold;
      const float total = (f[0] + f[1]) + (f[2] + f[3]) + (folded ? s.fold_l[tid] : 0.f);
      if (j_from < j_to && ok) ok = warp_wait(&s.o_done[x], (count - 1) & 1, &s.wait);
      if (ok) {
        tc_fence_after();
        const int bh = uniform(item.bh), b = bh / p.Hkv, split = item.split;
        int h1, t;
        const bool live = row_of(item, h1, t);
        const int h = bh % p.Hkv * p.rho + h1;
        bool wrong = false;
        const size_t row = ((size_t)bh * p.splits + split) * ((size_t)p.T * p.rho) + (size_t)t * p.rho + h1;
        const float inv = see0 < see1 ? 1.f / total : 0.f;
        if (p.splits > 1 && live) p.part_ml[row] = make_float2(m == -INFINITY ? m : m * by, total);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[16];
          if (j_from < j_to) {
            tmem_ld16(to_o + 16 * c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0u;
          }
          if (folded) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + s.fold_o[x][16 * c + e][tid & 127]);
          }
          if (!live) continue;
          if (p.splits > 1) {
            uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + row * 64 + 16 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
              wrong |= !(fabsf(__uint_as_float(o[4 * e])) + fabsf(__uint_as_float(o[4 * e + 1])) +
                         fabsf(__uint_as_float(o[4 * e + 2])) + fabsf(__uint_as_float(o[4 * e + 3])) < INFINITY);
            }
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
        const uint32_t again = __ballot_sync(0xffffffffu, wrong && see0 < see1);
        if (lane == 0) s.again[it & 3][warp] = again;
        if (lane == 0 && again) s.stop = 1;   // (the loading warp reads it before it goes three items further)
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.item_free[it & 1]);
    }
    // Rows whose result is not finite, now that nothing waits for this warp, of the last three items: the first item
    // with such rows lets go of its place before the loading warp hands out the second item behind it.
#pragma unroll 1
    for (int i = max(0, it - 3); ok && i < it; ++i) {
      const uint32_t again = s.again[i & 3][warp];
      if (again == 0u) continue;
      const TcItem &item = s.item[i & 3];
      int h, t;
      row_of(item, h, t);
      PagedSeq seq;
      seq.n = item.n, seq.past = item.past, seq.total = item.total;
      const int bh = item.bh;
      int2 sees = make_int2(0, 0);
      if (again >> lane & 1u) sees = paged_sees(p, seq, bh / p.Hkv, t);
      paged_rows_again(p, bh, item.split, seq.past, bh % p.Hkv * p.rho + h, t, max(sees.x, item.from), min(sees.y, item.to));
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

template <bool kCap, bool kBias, bool kFolds>
oal_status run(const PagedArgs &p, cudaStream_t stream) {
  static bool done[kMaxDevices];
  auto kernel = paged_tc_kernel<kCap, kBias, kFolds>;
  constexpr size_t bytes = kFolds ? kTcFoldBytes : kTcBytes;
  oal_status st = paged_need_smem(reinterpret_cast<const void *>(kernel), bytes, done);
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
  launch_pdl(kernel, grid, dim3(kTcThreads), bytes, stream, mq, mk, mv, p, nt);
  st = oal_after_launch("paged_tc_kernel", stream);
  return st != OAL_OK || p.splits == 1 ? st : launch_paged_join(p, 1, stream);
}

}  // namespace

// Rows of a block: two tiles of as many tokens as fit.
int paged_tc_rows(int T, int rho) { return 2 * rho * std::min(T, 128 / rho); }

template <bool kFolds>
static oal_status run_tc(const PagedArgs &p, cudaStream_t stream) {
  if (p.cap > 0.f) return p.slopes ? run<true, true, kFolds>(p, stream) : run<true, false, kFolds>(p, stream);
  return p.slopes ? run<false, true, kFolds>(p, stream) : run<false, false, kFolds>(p, stream);
}
oal_status launch_paged_tc(const PagedArgs &p, cudaStream_t stream) {
  return p.split_keys > kFold * kKeys ? run_tc<true>(p, stream) : run_tc<false>(p, stream);
}

}  // namespace oal
