// gated_decode.cu -- one token of the gated linear recurrence:
//     S = exp(g) S + k v^T,   y = scale S^T q
// per (sequence, KV head), the state of sequence b in slot slots[b] of a pool.
//
// The state is read and written once (32 KB a unit), q, k, v and y are small:
// HBM-bound for a batch, a few dependent loads long for one sequence.  One
// block a unit holds the state in registers: thread (row group, column
// group) owns kRows rows of 4 columns, all of whose loads are in flight
// before the first use.  Replayed with the states in L2: 2.6 us for 2 units,
// 4.9 for 512, 18 for 4096; four blocks a unit, 16 columns each, took 2.9,
// 6.8 and 37, and with cold states were ahead at no number of units either.
// Before its state a block looks through the slots of the sequences before its
// own, work that grows with the square of the batch: at 4096 sequences of 8
// heads the call takes 179 us, the bytes alone 158.
#include "gated.cuh"

namespace oal {
namespace {

constexpr int kDecThreads = 128;
constexpr int kHeads = 8;                // query heads read out together

template <typename T>
__global__ void __launch_bounds__(kDecThreads)
gated_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                    const float *__restrict__ g, int B, int Hq, int Hkv, float scale,
                    const int32_t *__restrict__ slots, int n_slots, float *__restrict__ state,
                    T *__restrict__ y, int *status) {
  pdl_trigger();
  pdl_wait();
  constexpr int kCols = kDv, kCg = kCols / 4, kRg = kDecThreads / kCg, kRows = kD / kRg;
  constexpr int kWarps = kDecThreads / 32;
  __shared__ float s_q[kHeads][kD];
  __shared__ float s_red[kWarps][kHeads][kCols];
  const int unit = blockIdx.x;
  const int b = unit / Hkv, kv = unit % Hkv, rho = Hq / Hkv;
  const int tid = threadIdx.x, cg = tid % kCg, rg = tid / kCg;
  int slot = b;
  if (slots) {
    slot = slots[b];
    // a slot that an earlier sequence of the batch holds is that one's
    int twice = 0;
    for (int i = tid; i < b; i += kDecThreads) twice |= slots[i] == slot;
    twice = __syncthreads_or(twice && slot >= 0);
    const bool bad = slot < -1 || slot >= n_slots || twice;
    if (bad && tid == 0) atomicCAS(status, kStatusOk, (int)OAL_ERR_INVALID_ARG);
    if (bad || slot == -1) {   // no state: zeros
      for (int x = tid; x < rho * kCols; x += kDecThreads)
        y[((size_t)b * Hq + kv * rho + x / kCols) * 64 + x % kCols] = from_f32<T>(0.f);
      return;
    }
  }
  float *s = state + ((size_t)slot * Hkv + kv) * kGS + 4 * cg;
  float4 S[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) S[r] = *reinterpret_cast<const float4 *>(s + (rg * kRows + r) * 64);
  const size_t kvrow = (size_t)unit * 64;
  const GateDecay a = decay_exp(__ldg(g + unit));
  float vv[4], kk[kRows];
#pragma unroll
  for (int e = 0; e < 4; ++e) vv[e] = to_f32(v[kvrow + 4 * cg + e]);
#pragma unroll
  for (int r = 0; r < kRows; ++r) kk[r] = to_f32(k[kvrow + rg * kRows + r]);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    S[r].x = decay_add(a, S[r].x, kk[r] * vv[0]), S[r].y = decay_add(a, S[r].y, kk[r] * vv[1]);
    S[r].z = decay_add(a, S[r].z, kk[r] * vv[2]), S[r].w = decay_add(a, S[r].w, kk[r] * vv[3]);
    *reinterpret_cast<float4 *>(s + (rg * kRows + r) * 64) = S[r];
  }
  for (int h0 = 0; h0 < rho; h0 += kHeads) {
    const int nh = min(kHeads, rho - h0);
    const size_t qrow = ((size_t)b * Hq + kv * rho + h0) * 64;
    __syncthreads();
    for (int x = tid; x < nh * kD; x += kDecThreads) s_q[x / kD][x % kD] = to_f32(q[qrow + x]);
    __syncthreads();
    for (int h = 0; h < nh; ++h) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float w = s_q[h][rg * kRows + r];
        o.x = fmaf(w, S[r].x, o.x), o.y = fmaf(w, S[r].y, o.y);
        o.z = fmaf(w, S[r].z, o.z), o.w = fmaf(w, S[r].w, o.w);
      }
#pragma unroll
      for (int d = kCg; d < 32; d <<= 1) {   // the warp's row groups of this column group
        o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
      }
      if ((tid & 31) < kCg) *reinterpret_cast<float4 *>(&s_red[tid >> 5][h][4 * cg]) = o;
    }
    __syncthreads();
    for (int x = tid; x < nh * kCols; x += kDecThreads) {
      const int h = x / kCols, c = x % kCols;
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) o += s_red[w][h][c];
      y[qrow + h * 64 + c] = from_f32<T>(scale * o);
    }
  }
}

}  // namespace

template <typename T>
static oal_status run(const void *q, const void *k, const void *v, const float *g, int B, int Hq, int Hkv,
                      float scale, const int32_t *slots, int n_slots, float *state, void *y,
                      cudaStream_t stream) {
  int *status = oal_device_status_word();
  if (!status) return oal_fail(OAL_ERR_CUDA, "no device status word");
  launch_pdl(gated_decode_kernel<T>, dim3(B * Hkv), dim3(kDecThreads), 0, stream, static_cast<const T *>(q),
             static_cast<const T *>(k), static_cast<const T *>(v), g, B, Hq, Hkv, scale, slots, n_slots,
             state, static_cast<T *>(y), status);
  return oal_after_launch("gated_decode_kernel", stream);
}

oal_status launch_gated_decode(const void *q, const void *k, const void *v, int is_bf16, const float *g, int B,
                               int Hq, int Hkv, float scale, const int32_t *slots, int n_slots, float *state,
                               void *y, cudaStream_t stream) {
  return is_bf16 ? run<__nv_bfloat16>(q, k, v, g, B, Hq, Hkv, scale, slots, n_slots, state, y, stream)
                 : run<float>(q, k, v, g, B, Hq, Hkv, scale, slots, n_slots, state, y, stream);
}

}  // namespace oal
