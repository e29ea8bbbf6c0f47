// gated_mma.cuh -- register-level tensor-core products of the gated
// recurrence on 64 x 64 bf16 tiles in shared memory (rows of 128 bytes, the
// 16-byte chunk c of row r at chunk c ^ (r & 7), as a 128-byte-swizzled TMA
// copy leaves it).
//
// The states live in registers, split over four warps (warp w owns rows
// 16 w .. 16 w + 15), because every chunk scales them by a decay and adds a
// product: in tensor memory that would be a read and a write of the state per
// chunk besides the product.
#pragma once
#include "gated.cuh"
#include "tc_ptx.cuh"

namespace oal {

constexpr int kTileBytes = kGC * 128;     // one 64 x 64 bf16 tile

__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Columns 8 nb0 .. 8 (nb0 + kNb) - 1 of a 64 x 64 fp32 matrix over four warps:
// v[nb][0..3] = rows r, r, r + 8, r + 8 (r = 16 warp + lane / 4), columns
// 8 (nb0 + nb) + 2 (lane % 4) and the next.
template <int kNb>
struct StateAcc {
  float v[kNb][4];
};

// A weight per token of a chunk as two bf16 terms (the sum is off by at most
// 2^-16 of it), in pairs: word l has tokens 2l and 2l + 1.
struct __align__(16) PairWeights {
  uint32_t hi[kGC / 2], lo[kGC / 2];
};
__device__ __forceinline__ void weights_put(PairWeights &w, float x, float y) {
  const int lane = threadIdx.x & 31;
  const uint32_t hi = tc::pack_bf16x2(x, y);
  w.hi[lane] = hi;
  w.lo[lane] = tc::pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// s += sum_j w_j a_j b_j^T over the 64 rows j of two tiles (kFrom, kTo: of the
// rows, 16 at a time).  w_j a_j goes in as two bf16 terms: hi = bf16(w_hi a),
// whose rounding error w_hi a - hi is a bf16 number itself, and
// lo = bf16(w_lo a + that), three packed products for two values; the terms'
// sum is off by at most 2^-15 of w a where one rounded factor would be off by
// 2^-8.  b is exact.  (For a state that is rounded to bf16 before it is read;
// state_step is the exact one.  Here the tensor cores add to the state itself
// and cut: 1.3e-4 low after 1024 chunks.)
// The terms of one accumulator are kNb products apart, and the next
// 16 rows' operand is under way while these multiply.
template <int kFrom, int kTo, int kNb>
__device__ __forceinline__ void state_add(StateAcc<kNb> &s, int nb0, const void *a_tile, const void *b_tile,
                                          const PairWeights &w) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int mat = lane >> 3, r = lane & 7, q = lane & 3;
  // (16 rows further on is 2048 bytes: the swizzle goes by the row's low three bits)
  const uint32_t at = tc::smem_u32(a_tile) + tile_at(8 * (mat >> 1) + r, 2 * warp + (mat & 1));
  uint32_t bt[kNb / 2];
#pragma unroll
  for (int np = 0; np < kNb / 2; ++np)
    bt[np] = tc::smem_u32(b_tile) + tile_at(8 * (mat & 1) + r, nb0 + 2 * np + (mat >> 1));
  uint32_t a[4], b[kNb / 2][4];
  ldsm4t(at + 2048 * kFrom, a);
#pragma unroll
  for (int ks = kFrom; ks < kTo; ++ks) {
#pragma unroll
    for (int np = 0; np < kNb / 2; ++np) ldsm4t(bt[np] + 2048 * ks, b[np]);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t wh = w.hi[8 * ks + 4 * (e >> 1) + q], wl = w.lo[8 * ks + 4 * (e >> 1) + q];
      hi[e] = bf2_mul(wh, a[e]);
      lo[e] = bf2_fma(wl, a[e], bf2_fma(wh, a[e], hi[e] ^ 0x80008000u));
    }
    if (ks + 1 < kTo) ldsm4t(at + 2048 * (ks + 1), a);
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) mma16816(s.v[nb], hi, b[nb >> 1][2 * (nb & 1)], b[nb >> 1][2 * (nb & 1) + 1]);
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) mma16816(s.v[nb], lo, b[nb >> 1][2 * (nb & 1)], b[nb >> 1][2 * (nb & 1) + 1]);
  }
}
// s = f s + sum_j w_j a_j b_j^T over the 64 rows j of two tiles, w in fp32 in
// shared memory, as a sum of fp32 products: w_j a_j is formed in fp32 and goes
// in as three bf16 terms, which hold all of its 24 bits, and the tiles' sum
// starts from zero, because the tensor cores cut what they add to an
// accumulator instead of rounding it (a state of 2,000 tokens was off by 3e-6
// when they added to it, by 2e-7 this way).
__device__ __forceinline__ void split3(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  hi = tc::pack_bf16x2(x, y);
  x -= __uint_as_float(hi << 16), y -= __uint_as_float(hi & 0xFFFF0000u);
  mid = tc::pack_bf16x2(x, y);
  x -= __uint_as_float(mid << 16), y -= __uint_as_float(mid & 0xFFFF0000u);
  lo = tc::pack_bf16x2(x, y);
}
template <int kNb>
__device__ __forceinline__ void state_step(StateAcc<kNb> &s, float f, int nb0, const void *a_tile, const void *b_tile,
                                           const float *w) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int mat = lane >> 3, r = lane & 7, q = lane & 3;
  const uint32_t at = tc::smem_u32(a_tile) + tile_at(8 * (mat >> 1) + r, 2 * warp + (mat & 1));
  uint32_t bt[kNb / 2];
#pragma unroll
  for (int np = 0; np < kNb / 2; ++np)
    bt[np] = tc::smem_u32(b_tile) + tile_at(8 * (mat & 1) + r, nb0 + 2 * np + (mat >> 1));
  StateAcc<kNb> d = {};
  uint32_t a[4], b[kNb / 2][4];
  ldsm4t(at, a);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
    for (int np = 0; np < kNb / 2; ++np) ldsm4t(bt[np] + 2048 * ks, b[np]);
    uint32_t t[3][4];
    const float2 w0 = *reinterpret_cast<const float2 *>(w + 16 * ks + 2 * q);
    const float2 w1 = *reinterpret_cast<const float2 *>(w + 16 * ks + 8 + 2 * q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = e < 2 ? w0 : w1;
      split3(__uint_as_float(a[e] << 16) * x.x, __uint_as_float(a[e] & 0xFFFF0000u) * x.y, t[0][e], t[1][e], t[2][e]);
    }
    if (ks < 3) ldsm4t(at + 2048 * (ks + 1), a);
#pragma unroll
    for (int z = 0; z < 3; ++z)
#pragma unroll
      for (int nb = 0; nb < kNb; ++nb) mma16816(d.v[nb], t[z], b[nb >> 1][2 * (nb & 1)], b[nb >> 1][2 * (nb & 1) + 1]);
  }
#pragma unroll
  for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) s.v[nb][e] = fmaf(f, s.v[nb][e], d.v[nb][e]);
}
template <int kNb>
__device__ __forceinline__ void state_scale(StateAcc<kNb> &s, GateDecay f) {
#pragma unroll
  for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) s.v[nb][e] = decay_add(f, s.v[nb][e], 0.f);
}
template <int kNb>
__device__ __forceinline__ void state_load(StateAcc<kNb> &s, int nb0, const float *src) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int r = 16 * warp + (lane >> 2), c = 8 * nb0 + 2 * (lane & 3);
#pragma unroll
  for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = src ? *reinterpret_cast<const float2 *>(src + (r + 8 * h) * 64 + 8 * nb + c) : make_float2(0.f, 0.f);
      s.v[nb][2 * h] = x.x, s.v[nb][2 * h + 1] = x.y;
    }
}
template <int kNb>
__device__ __forceinline__ void state_store(const StateAcc<kNb> &s, int nb0, float *dst) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int r = 16 * warp + (lane >> 2), c = 8 * nb0 + 2 * (lane & 3);
#pragma unroll
  for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2 *>(dst + (r + 8 * h) * 64 + 8 * nb + c) = make_float2(s.v[nb][2 * h], s.v[nb][2 * h + 1]);
}
// The columns rounded to bf16 into a tile (row d of the state = row d of the tile).
template <int kNb>
__device__ __forceinline__ void state_round(const StateAcc<kNb> &s, int nb0, void *tile) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int r = 16 * warp + (lane >> 2), c = 4 * (lane & 3);
  uint8_t *t = static_cast<uint8_t *>(tile);
#pragma unroll
  for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint32_t *>(t + tile_at(r + 8 * h, nb0 + nb) + c) =
          tc::pack_bf16x2(s.v[nb][2 * h], s.v[nb][2 * h + 1]);
}

// Decays from behind a lane's two tokens to the end of the chunk, and over the
// whole chunk (returned).
__device__ __forceinline__ GateDecay gate_tails(const GateLane &x, float2 &out) {
  const float eh = __shfl_sync(0xffffffffu, x.hi[1], 31), el = __shfl_sync(0xffffffffu, x.lo[1], 31);
  const int ec = __shfl_sync(0xffffffffu, x.cuts[1], 31);
  out = make_float2(gate_exp_fast(x.cuts[0] == ec, (eh - x.hi[0]) + (el - x.lo[0])),
                    gate_exp_fast(x.cuts[1] == ec, (eh - x.hi[1]) + (el - x.lo[1])));
  return decay_exp(ec == 0 ? eh + el : -INFINITY);
}

}  // namespace oal
