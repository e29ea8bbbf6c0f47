// state_remap.cu -- copying, forking, compacting and freeing the slots of a
// pool of states in place: new[i] = old[map[i]], zeros where map[i] is -1.
//
// Every source has to be read before any target is written, whatever cycles
// the map holds.  The slots are cut into slices of a few words; a block takes
// a slice of ALL slots that change, holds the old words that move in
// registers, waits for its threads, and writes them and the zeros.  Slices do
// not meet, so no block waits for another, and no workspace is needed.  Each
// moved slot's source is read once and its target written once: HBM-bound.
// The fewer slots move, the longer the runs of a slice: 512 moving slots leave
// runs of 128 bytes, 64 of 1 KB.  26 us for 64 slots of 1.1 MB (4.5 TB/s, in
// 8-byte words, as such slots start on 8), 37 us for 512 moves and 512 zeros
// of 131 KB (5.4 TB/s).  Words placed anew for every slice, with a division
// each, cost 20% more.
#include <algorithm>

#include "gated.cuh"

namespace oal {
namespace {

constexpr int kMoveThreads = 1024;
constexpr int kMoveMost = OAL_REMAP_MAX_SLOTS;           // one word of each slot at least

// Word: the widest type that slot_bytes is a multiple of (a packed prefix
// state has 557,700 bytes a head, so slots need not start on 16).
template <typename Word, int kWords, bool kAhead>
__global__ void __launch_bounds__(kMoveThreads)
state_remap_kernel(Word *pool, long long slot_words, int n, const int32_t *__restrict__ map, int *status) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ int2 s_move[];      // (target, source) of the slots that move; from the end: those to be zeroed
  __shared__ int s_count, s_zeros;
  if (threadIdx.x == 0) s_count = s_zeros = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kMoveThreads) {
    const int from = map[i];
    if (from < -1 || from >= n) {
      atomicCAS(status, kStatusOk, (int)OAL_ERR_INVALID_ARG);
    } else if (from == -1) {
      s_move[n - 1 - atomicAdd(&s_zeros, 1)].x = i;          // (any order: targets differ)
    } else if (from != i) {
      s_move[atomicAdd(&s_count, 1)] = make_int2(i, from);
    }
  }
  __syncthreads();
  const int count = s_count, zeros = s_zeros;
  if (count + zeros == 0) return;
  // words of a slice: as many as the block holds, at most what spreads the
  // slot over the grid
  const long long spread = (slot_words + gridDim.x - 1) / gridDim.x;
  const int width = (int)min((long long)(kWords * kMoveThreads / max(count, 1)), spread);
  const long long step = (long long)gridDim.x * width;
  // this thread's words of every slice: the move, and the place in the slice
  // (16 bits each; past the last move: past the slice)
  uint32_t at[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int x = threadIdx.x + k * kMoveThreads, m = x / width;
    at[k] = m < count ? (uint32_t)m << 16 | (uint32_t)(x - m * width) : 0xFFFFu;
  }
  auto gather = [&](long long w0, Word (&held)[kWords]) {
    const int wide = (int)max(0LL, min((long long)width, slot_words - w0));
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      if ((int)(at[k] & 0xFFFFu) < wide) held[k] = pool[s_move[at[k] >> 16].y * slot_words + (w0 + (at[k] & 0xFFFFu))];
  };
  auto scatter = [&](long long w0, const Word (&held)[kWords]) {
    const int wide = (int)min((long long)width, slot_words - w0);
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      if ((int)(at[k] & 0xFFFFu) < wide) pool[s_move[at[k] >> 16].x * slot_words + (w0 + (at[k] & 0xFFFFu))] = held[k];
    for (int x = threadIdx.x; x < zeros * width; x += kMoveThreads) {
      const int m = x / width, w = x - m * width;
      if (w < wide) pool[s_move[n - 1 - m].x * slot_words + w0 + w] = Word();
    }
  };
  // (kAhead: the next slice is on its way while this one is written)
  Word held[kAhead ? 2 : 1][kWords];
  long long w0 = (long long)blockIdx.x * width;
  if (kAhead) gather(w0, held[0]);
  for (; w0 < slot_words; w0 += step) {
    if (!kAhead) gather(w0, held[0]);
    __syncthreads();                     // the slice at w0 is read by all
    if (kAhead) gather(w0 + step, held[kAhead]);
    scatter(w0, held[0]);
    if (!kAhead) continue;
    w0 += step;
    if (w0 >= slot_words) break;
    __syncthreads();
    gather(w0 + step, held[0]);
    scatter(w0, held[kAhead]);
  }
}

template <typename Word>
oal_status remap(void *pool, size_t slot_bytes, int n, const int32_t *map, int *status, cudaStream_t stream) {
  static bool done[2][kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return oal_fail(OAL_ERR_CUDA, "no current device");
  // Four words a thread and two slices in flight; more slots than that has
  // words for take eight and one slice.
  const bool few = n <= 4 * kMoveThreads;
  const auto kernel = few ? state_remap_kernel<Word, 4, true> : state_remap_kernel<Word, 8, false>;
  if (!done[few][dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kMoveMost * sizeof(int2))) !=
        cudaSuccess)
      return oal_check_launch("shared memory of the remap kernel");
    done[few][dev] = true;
  }
  const long long words = (long long)(slot_bytes / sizeof(Word));
  const int blocks = (int)std::min<long long>(words, 152);
  launch_pdl(kernel, dim3(blocks), dim3(kMoveThreads), (size_t)n * sizeof(int2), stream,
             static_cast<Word *>(pool), words, n, map, status);
  return oal_after_launch("state_remap_kernel", stream);
}

}  // namespace

oal_status launch_state_remap(void *pool, size_t slot_bytes, int n, const int32_t *map, cudaStream_t stream) {
  int *status = oal_device_status_word();
  if (!status) return oal_fail(OAL_ERR_CUDA, "no device status word");
  if (slot_bytes % 16 == 0) return remap<uint4>(pool, slot_bytes, n, map, status, stream);
  if (slot_bytes % 8 == 0) return remap<uint2>(pool, slot_bytes, n, map, status, stream);
  if (slot_bytes % 4 == 0) return remap<uint32_t>(pool, slot_bytes, n, map, status, stream);
  if (slot_bytes % 2 == 0) return remap<uint16_t>(pool, slot_bytes, n, map, status, stream);
  return remap<uint8_t>(pool, slot_bytes, n, map, status, stream);
}

}  // namespace oal
