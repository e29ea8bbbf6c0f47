// gated_tc.cuh -- what the gated recurrence's tensor-core kernels share: bulk
// stores, warp-wide waits, the modes of a chunk's gates, tensor maps.
#pragma once
#include <cudaTypedefs.h>

#include "gated_mma.cuh"

namespace oal {
namespace gated {
using namespace tc;

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// A value that is the same in all lanes, as one the compiler knows to be so:
// branches on it are uniform, and what follows from it (descriptors, tensor-
// memory addresses) stays in uniform registers, where an MMA wants it.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int warp_index() { return (int)uniform(threadIdx.x >> 5); }
// Without a time hint the hardware puts a waiting warp to sleep until the phase
// completes (or a while has passed); with one the wait is a loop of probes and
// naps, which takes issue slots and instruction fetches from the others.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// What every wait of a block shares, in shared memory.
struct WaitState {
  int *status;                            // the device status word
  int abort;                              // a wait gave up: the others give up too
};
// The rest of a wait that did not end at once (out of line: these kernels'
// instructions barely fit the caches).  Bounded like mbar_wait.
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, WaitState *w) {
  const uint64_t t0 = cycles_now();
  volatile int *abort = &w->abort;
  while (!try_wait(bar, parity)) {
    if (*abort) return false;
    const uint64_t el = cycles_now() - t0;
    if (el > kWaitFloorCycles && el > wait_limit(w->status)) {
      *abort = 1;
      atomicCAS(w->status, 0, 4 /* OAL_ERR_TIMEOUT */);
      return false;
    }
  }
  return true;
}
// A wait by a whole warp, whose lanes agree on the outcome (the tensor-memory
// instructions that follow want all of them).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, WaitState *w) {
  bool ok = try_wait(smem_u32(bar), parity);
  if (!ok) ok = wait_on(smem_u32(bar), parity, w);
  return __all_sync(0xffffffffu, ok);
}
// The first 1024-byte boundary of the dynamic shared memory.  (By an offset: a
// pointer rounded as an integer is one the compiler no longer knows to be
// shared, and every access through it a generic one.)
__device__ __forceinline__ uint8_t *align1024(uint8_t *p) { return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u); }

// What a chunk's gates ask for: nothing (R = 0, no cuts), R per half and
// masks, or every decay by itself.
constexpr int kPlain = 0, kHalves = 1, kEach = 2;
constexpr float kSpan = 60.f;

struct alignas(16) ChunkGates {
  float rest[kGC], row[kGC];              // e^{R-G_j}, e^{G_i-R}
  float before[kGC / 2];                  // e^{R'-G_j}, R' that of the second half's rows
  GateDecay whole;                        // e^{G_63} (0 if cut)
  float first;                            // e^{R'}
  uint32_t cut_even, cut_odd;             // bit l: the gate of token 2l (2l + 1) is cut
  int mode;
};
// e^{a-b} of two sums hi + lo.  kExact: to fp32's last bits, which the fast
// exponential of a sum rounded to fp32 is not where that is large (3e-6 at 60).
template <bool kExact>
__device__ __forceinline__ float gate_exp_sums(float ah, float al, float bh, float bl) {
  if (!kExact) return __expf((ah - bh) + (al - bl));
  float x, e;
  two_sum(ah, -bh, x, e);
  x = expf(x);
  return fmaf(x, e + (al - bl), x);
}
// Fills them, and the lane's decays to the chunk's end (one warp; `gate` as
// loaded, `sums` of it); never as kPlain if so told.
template <bool kExact>
__device__ __forceinline__ void chunk_gates(float2 gate, const GateLane &sums, ChunkGates &to, float2 &tail,
                                            bool not_plain = false) {
  const int lane = threadIdx.x & 31;
  const uint32_t even = __ballot_sync(0xffffffffu, gate.x <= kGateCut);
  const uint32_t odd = __ballot_sync(0xffffffffu, gate.y <= kGateCut);
  const GateDecay whole = gate_tails(sums, tail);
  const float mh = __shfl_sync(0xffffffffu, sums.hi[1], 15), ml = __shfl_sync(0xffffffffu, sums.lo[1], 15);
  const float span = fmaxf(fabsf(sums.hi[0]), fabsf(sums.hi[1]));
  const bool plain = __all_sync(0xffffffffu, span <= kSpan) && (even | odd) == 0u && !not_plain;
  const float bh = plain ? 0.f : mh, bl = plain ? 0.f : ml;          // R'
  const float rh = lane < 16 ? 0.f : bh, rl = lane < 16 ? 0.f : bl;   // R
  const float near = fmaxf(fabsf(sums.hi[0] - rh), fabsf(sums.hi[1] - rh));
  const bool halves = __all_sync(0xffffffffu, near <= kSpan);
  float2 rest, row, before;
  rest.x = gate_exp_sums<kExact>(rh, rl, sums.hi[0], sums.lo[0]), rest.y = gate_exp_sums<kExact>(rh, rl, sums.hi[1], sums.lo[1]);
  row.x = gate_exp_sums<kExact>(sums.hi[0], sums.lo[0], rh, rl), row.y = gate_exp_sums<kExact>(sums.hi[1], sums.lo[1], rh, rl);
  before.x = gate_exp_sums<kExact>(bh, bl, sums.hi[0], sums.lo[0]);
  before.y = gate_exp_sums<kExact>(bh, bl, sums.hi[1], sums.lo[1]);
  reinterpret_cast<float2 *>(to.rest)[lane] = rest;
  reinterpret_cast<float2 *>(to.row)[lane] = row;
  if (lane < 16) reinterpret_cast<float2 *>(to.before)[lane] = before;
  if (lane == 0) {
    to.whole = whole;
    to.first = __expf(bh + bl);
    to.cut_even = even;
    to.cut_odd = odd;
    to.mode = plain ? kPlain : halves ? kHalves : kEach;
  }
}
// Whether a gate up to token i's is cut; `begin` then becomes the last such token.
__device__ __forceinline__ bool cut_before(const ChunkGates &gates, int i, int &begin) {
  const uint32_t upto = (2u << (i >> 1)) - 1u;     // bits l with 2 l <= i
  const uint32_t even = gates.cut_even & upto, odd = gates.cut_odd & (i & 1 ? upto : upto >> 1);
  if ((even | odd) == 0u) return false;
  begin = max(2 * (31 - __clz(even)), 2 * (31 - __clz(odd)) + 1);
  return true;
}

// Rows from `rows` on of a tile become zeros; thread `at` of `threads`.
static __device__ __noinline__ void clear_rows(void *tile, int rows, int at, int threads) {
  for (int x = at; x < 64 * 8; x += threads)
    if ((x >> 3) >= rows) reinterpret_cast<uint4 *>(tile)[x] = make_uint4(0u, 0u, 0u, 0u);
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (PFN_cuTensorMapEncodeTiled_v12000)f;
  }();
  return fn;
}

// [heads][T][64] bf16 in boxes of 64 columns, 128-byte swizzle; rows from T on
// read as zeros and are not written.
inline oal_status make_map(CUtensorMap *m, const void *ptr, int T, long long heads, int rows = kGC) {
  auto fn = encode_fn();
  if (!fn) return oal_fail(OAL_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[3] = {64, (cuuint64_t)T, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {128, (cuuint64_t)T * 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1}, es[3] = {1, 1, 1};
  if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return oal_fail(OAL_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  return OAL_OK;
}

}  // namespace gated

}  // namespace oal
