// rope.cu -- rotary positions, and appending to a paged cache with the rotation
// on the way.
//
// Pair r of a row at position p turns by the angle p f_r.  Angles are held in
// turns as 64-bit fractions: p times round(2^64 f_r / 2 pi), modulo 2^64, is the
// angle modulo a turn to 2^-33 of a turn whatever the position (32 bits), in two
// integer products where a float loses a bit for every doubling of p.  The
// nearest quarter turn is taken out exactly and the rest (at most an eighth)
// goes through sincospif.
//
// A block takes 4 tokens: their angles once, into shared memory, for all of its
// heads, while the first rows are on their way; then every row is read once and
// written once: HBM-bound.  A thread moves two 16-byte pieces whose elements pair
// up.  4 x 8192 tokens, 32/8 heads, bf16, as views of a projection: 53.8 us (6.24
// TB/s), appending them 63.7 (6.32); blocks of 4, 8 and 16 tokens 53.8, 54.7 and
// 60.0.  Few tokens: the heads are spread over blocks instead, and the angles are
// formed again in each.
#include <algorithm>

#include "paged.cuh"

namespace oal {
namespace {

constexpr int kRopeThreads = 64;
constexpr int kRopeTokens = 4;

struct alignas(16) Piece {
  uint4 w;
};
template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);

__device__ __forceinline__ void piece_get(const Piece &x, float (&f)[8]) {
  const uint32_t w[4] = {x.w.x, x.w.y, x.w.z, x.w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) f[2 * e] = __uint_as_float(w[e] << 16), f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
}
__device__ __forceinline__ void piece_get(const Piece &x, float (&f)[4]) {
  f[0] = __uint_as_float(x.w.x), f[1] = __uint_as_float(x.w.y), f[2] = __uint_as_float(x.w.z), f[3] = __uint_as_float(x.w.w);
}
__device__ __forceinline__ Piece piece_put(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
  return Piece{make_uint4(w[0], w[1], w[2], w[3])};
}
__device__ __forceinline__ Piece piece_put(const float (&f)[4]) {
  return Piece{make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]))};
}

template <typename T, bool kHalves>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(RopeArgs p, int heads_a_block) {
  pdl_trigger();
  pdl_wait();
  constexpr int E = kPiece<T>, kUnits = 32 / E;       // pairs of a unit, units of a row
  constexpr int kStep = kRopeThreads / kUnits / kRopeTokens;   // heads of a pass
  __shared__ float2 s_turn[kRopeTokens][33];
  const int tid = threadIdx.x, unit = tid % kUnits, tok = tid / kUnits % kRopeTokens;
  const uint32_t T_ = (uint32_t)p.T, n0 = blockIdx.x * kRopeTokens, all = (uint32_t)p.B * T_;
  const int a0 = kHalves ? unit * E : 2 * unit * E, a1 = a0 + (kHalves ? 32 : E);

  // the thread's token: in its sequence, and (page) its place in the cache
  const uint32_t n = min(n0 + tok, all - 1), b = n / T_, t = n - b * T_;
  bool live = n0 + tok < all;
  if (live && p.lengths) {
    const int len = p.lengths[b];
    if (len < 0 || len > p.T) atomicCAS(p.status, kStatusOk, (int)OAL_ERR_INVALID_ARG);
    live = (int)t < len;
  }
  long long page = -1;
  if (p.Kp && live) {
    const long long at = (long long)p.past[b] + t;
    int i = -1;
    if (at >= 0 && (at >> p.page_shift) < p.max_pages) i = p.table[(size_t)b * p.max_pages + (at >> p.page_shift)];
    if (i >= 0 && i < p.n_pages)
      page = i * p.page_stride + (at & ((1 << p.page_shift) - 1)) * 64;
    else
      atomicCAS(p.status, kStatusOk, (int)OAL_ERR_INVALID_ARG);
  }
  const int heads = p.Hq + (p.K ? p.Hkv : 0) + (p.V ? p.Hkv : 0);
  const int h0 = blockIdx.y * heads_a_block, h1 = live ? min(heads, h0 + heads_a_block) : 0;
  auto source = [&](int h) {
    if (h < p.Hq) return static_cast<const T *>(p.Q) + b * p.q.b + t * p.q.t + h * p.q.h;
    h -= p.Hq;
    if (h < p.Hkv) return static_cast<const T *>(p.K) + b * p.k.b + t * p.k.t + h * p.k.h;
    return static_cast<const T *>(p.V) + b * p.v.b + t * p.v.t + (h - p.Hkv) * p.v.h;
  };
  auto target = [&](int h) -> T * {       // null: nowhere
    if (h < p.Hq) return static_cast<T *>(p.Yq) + (((size_t)b * p.Hq + h) * p.T + t) * 64;
    h -= p.Hq;
    const bool key = h < p.Hkv;
    if (!p.Kp) return static_cast<T *>(p.Yk) + (((size_t)b * p.Hkv + h) * p.T + t) * 64;
    if (page < 0) return nullptr;
    if (!key) h -= p.Hkv;
    return static_cast<T *>(key ? p.Kp : p.Vp) + page + ((long long)h << p.page_shift) * 64;
  };
  // the first rows are on their way while the angles are formed
  int h = h0 + tid / (kUnits * kRopeTokens);
  Piece x0 = {}, x1 = {};
  if (h < h1) {
    const T *src = source(h);
    x0 = *reinterpret_cast<const Piece *>(src + a0), x1 = *reinterpret_cast<const Piece *>(src + a1);
  }
  if (p.turns) {
    for (int x = tid; x < kRopeTokens * 32; x += kRopeThreads) {
      const int r = x & 31;
      const uint32_t m = n0 + (x >> 5);
      if (m >= all) break;
      long long at;
      if (p.positions) {
        const long long axis = p.axes[r];
        const bool bad = axis < 0 || axis >= p.n_axes;
        if (bad) atomicCAS(p.status, kStatusOk, (int)OAL_ERR_INVALID_ARG);
        at = p.positions[(bad ? 0 : axis) * all + m];
      } else {
        at = (long long)(m % T_) + (p.past ? p.past[m / T_] : 0);
      }
      const unsigned long long turn = (unsigned long long)at * p.turns[r];
      const unsigned long long quarter = turn + (1ull << 61);
      float s, c;
      sincospif((float)(long long)(turn - (quarter & (3ull << 62))) * 0x1p-63f, &s, &c);
      const int k = (int)(quarter >> 62);
      if (k & 1) { const float x2 = c; c = -s, s = x2; }
      if (k & 2) c = -c, s = -s;
      s_turn[x >> 5][r] = make_float2(c, p.inverse ? -s : s);
    }
  }
  __syncthreads();
  float2 turn[E];
  if (p.turns) {
#pragma unroll
    for (int e = 0; e < E; ++e) turn[e] = s_turn[tok][unit * E + e];
  }
  const int turned = p.turns ? p.Hq + p.Hkv : 0;      // heads that turn
#pragma unroll 4
  for (; h < h1; h += kStep) {
    Piece y0 = x0, y1 = x1;
    if (h + kStep < h1) {
      const T *src = source(h + kStep);
      x0 = *reinterpret_cast<const Piece *>(src + a0), x1 = *reinterpret_cast<const Piece *>(src + a1);
    }
    if (h < turned) {
      float a[E], c[E];
      piece_get(y0, a), piece_get(y1, c);
      if (kHalves) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float u = a[e], w = c[e];
          a[e] = fmaf(u, turn[e].x, -(w * turn[e].y)), c[e] = fmaf(w, turn[e].x, u * turn[e].y);
        }
      } else {   // pairs inside each piece
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float2 t0 = turn[e], t1 = turn[E / 2 + e];
          float u = a[2 * e], w = a[2 * e + 1];
          a[2 * e] = fmaf(u, t0.x, -(w * t0.y)), a[2 * e + 1] = fmaf(w, t0.x, u * t0.y);
          u = c[2 * e], w = c[2 * e + 1];
          c[2 * e] = fmaf(u, t1.x, -(w * t1.y)), c[2 * e + 1] = fmaf(w, t1.x, u * t1.y);
        }
      }
      y0 = piece_put(a), y1 = piece_put(c);
    }
    T *dst = target(h);
    if (dst) *reinterpret_cast<Piece *>(dst + a0) = y0, *reinterpret_cast<Piece *>(dst + a1) = y1;
  }
}

template <typename T>
oal_status run(const RopeArgs &p, int form, const char *name, cudaStream_t stream) {
  const int heads = p.Hq + (p.K ? p.Hkv : 0) + (p.V ? p.Hkv : 0);
  const long long tiles = ((long long)p.B * p.T + kRopeTokens - 1) / kRopeTokens;
  constexpr int pass = kRopeThreads / (32 / kPiece<T>) / kRopeTokens;      // heads of a pass
  const int per = (heads + pass - 1) / pass;
  const int groups = (int)std::min<long long>(per, std::max<long long>(1, 608 / tiles));
  const int each = (per + groups - 1) / groups * pass;
  const dim3 grid((unsigned)tiles, (unsigned)((heads + each - 1) / each));
  if (form == OAL_ROPE_HALVES)
    launch_pdl(rope_kernel<T, true>, grid, dim3(kRopeThreads), 0, stream, p, each);
  else
    launch_pdl(rope_kernel<T, false>, grid, dim3(kRopeThreads), 0, stream, p, each);
  return oal_after_launch(name, stream);
}

}  // namespace

oal_status launch_rope(const RopeArgs &p, int is_bf16, int form, const char *name, cudaStream_t stream) {
  return is_bf16 ? run<__nv_bfloat16>(p, form, name, stream) : run<float>(p, form, name, stream);
}

}  // namespace oal
