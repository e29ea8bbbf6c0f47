// paged_again.cuh -- rows of bf16 whose result is not finite, formed once more.
//
// A weight of 0 for a key that a row does not see leaves nothing of its value,
// unless that is an infinity or NaN.  The kernels see that in the result and form
// such rows again here, over the keys of their own split.  A look at the keys first
// tells most rows that do see a bad one (they stay as they are: not finite); the
// others take 16 at a time a walk in which values that are not finite count as
// zeros, and a row that sees one after all gets NaN.
//
// Products by mma.sync, straight from global memory.  Both products may take
// their columns in any order, so a thread takes 16 neighbouring dimensions of a
// key (two 16-byte loads) and 8 neighbouring columns of a value (one).
//
// A NaN in the middle of a sequence that all tokens behind it see, or two of three,
// against the call without it: 8192 tokens of 32/8 heads 0.21 -> 1.2 and 0.27 -> 1.8
// ms, 131072 tokens of 4/1 heads 5.8 -> 35 and 7.6 -> 54 ms, 64 x 4 tokens on 8000
// 0.17 -> 0.35 ms.
#pragma once
#include "gated_mma.cuh"
#include "paged.cuh"

namespace oal {

__device__ __forceinline__ bool not_finite2(uint32_t w) {   // of two bf16
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Lane l has row l: query head h (of all), token t, the keys [lo, hi) that it
// sees of this split; lo >= hi: left as it is.  Writes Y, or the split's partial
// result.
static __device__ __forceinline__ void paged_rows_again(const PagedArgs &p, int bh, int split, int past, int h, int t,
                                                     int lo, int hi) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, b = bh / p.Hkv, kv = bh % p.Hkv;
  const bool plain = !(p.cap > 0.f) && !p.slopes;
  const float scale2 = p.scale * kLog2e;
  const __nv_bfloat16 *Kp = static_cast<const __nv_bfloat16 *>(p.Kp), *Vp = static_cast<const __nv_bfloat16 *>(p.Vp);
  // Where the first and the last bad key lie: a row that sees one of them is as it is.
  const int from = __reduce_min_sync(0xffffffffu, lo < hi ? lo : INT32_MAX), to = __reduce_max_sync(0xffffffffu, lo < hi ? hi : 0);
  int bad0 = INT32_MAX, bad1 = -1;
#pragma unroll 1
  for (int j0 = from < to ? from & ~15 : to; j0 < to; j0 += 32) {
    uint4 x[16];                            // a lane takes 16 bytes of every fourth key, and of its value
    const int page[2] = {paged_page_again(p, b, j0), j0 + 16 < to ? paged_page_again(p, b, j0 + 16) : -1};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const size_t at = paged_row(p, max(page[i >> 2], 0), kv, j0 + 4 * i + (lane >> 3)) + 8 * (lane & 7);
      x[i] = x[8 + i] = make_uint4(0u, 0u, 0u, 0u);
      if (page[i >> 2] >= 0) x[i] = *reinterpret_cast<const uint4 *>(Kp + at), x[8 + i] = *reinterpret_cast<const uint4 *>(Vp + at);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = j0 + 4 * (i & 7) + (lane >> 3);
      if (key >= from && key < to && (not_finite2(x[i].x) || not_finite2(x[i].y) || not_finite2(x[i].z) || not_finite2(x[i].w)))
        bad0 = min(bad0, key), bad1 = max(bad1, key);
    }
  }
  bad0 = __reduce_min_sync(0xffffffffu, bad0), bad1 = __reduce_max_sync(0xffffffffu, bad1);
  if ((lo <= bad0 && bad0 < hi) || (lo <= bad1 && bad1 < hi)) hi = lo;
  uint32_t rows = __ballot_sync(0xffffffffu, lo < hi);
#pragma unroll 1
  while (rows != 0u) {                      // 16 of them at a time
    uint32_t after = rows;
    for (int i = 0; i < 16; ++i) after &= after - 1u;
    const bool mine = (rows & ~after) >> lane & 1u;
    const int k0 = __reduce_min_sync(0xffffffffu, mine ? lo : INT32_MAX), k1 = __reduce_max_sync(0xffffffffu, mine ? hi : 0);
    uint32_t q[4][4];
    int row_h[2], row_t[2], row_lo[2], row_hi[2];
    float slope[2], m[2], l[2], o[8][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {           // the thread's rows: g and g + 8 of the 16
      const int nth = (int)__fns(rows & ~after, 0, 8 * u + g + 1), who = nth & 31;
      row_h[u] = __shfl_sync(0xffffffffu, h, who), row_t[u] = __shfl_sync(0xffffffffu, t, who);
      row_lo[u] = __shfl_sync(0xffffffffu, lo, who), row_hi[u] = __shfl_sync(0xffffffffu, hi, who);
      if (nth < 0) row_hi[u] = row_lo[u];   // (fewer than 16)
      uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
      slope[u] = 0.f;
      if (row_lo[u] < row_hi[u]) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.Q) +
                                                           (((size_t)b * p.Hq + row_h[u]) * p.T + row_t[u]) * 64 + 16 * c);
        x = src[0], y = src[1];
        if (p.slopes) slope[u] = p.slopes[row_h[u]];
      }
      q[0][u] = x.x, q[0][2 + u] = x.y, q[1][u] = x.z, q[1][2 + u] = x.w;
      q[2][u] = y.x, q[2][2 + u] = y.y, q[3][u] = y.z, q[3][2 + u] = y.w;
      m[u] = -INFINITY, l[u] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    bool lost[2] = {row_lo[0] >= row_hi[0], row_lo[1] >= row_hi[1]};   // nothing more to find out
    // Keys j0 + 8 n + g, dimensions 16 c ..; values j0 + 2 c, + 1, + 8, + 9, columns 8 g ..: of 16 keys, which lie on
    // one page.  (Those that no row sees are read along: masked, or values whose weights are 0.)  A step ahead.
    uint4 k[2][2], v[4], k_next[2][2], v_next[4];
    auto load = [&](int page, int j0) {
      const size_t at = page >= 0 ? paged_row(p, page, kv, j0) : 0;
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint4 *src = reinterpret_cast<const uint4 *>(Kp + at + (8 * n + g) * 64 + 16 * c);
        k_next[n][0] = page >= 0 ? src[0] : none, k_next[n][1] = page >= 0 ? src[1] : none;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 *src = reinterpret_cast<const uint4 *>(Vp + at + (2 * c + (i & 1) + 8 * (i >> 1)) * 64 + 8 * g);
        v_next[i] = page >= 0 ? src[0] : none;
      }
    };
    const int start = k0 & ~15;
    load(paged_page_again(p, b, start), start);
    int page = start + 16 < k1 ? paged_page_again(p, b, start + 16) : -1;
#pragma unroll 1
    for (int j0 = start; j0 < k1; j0 += 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i >> 1][i & 1] = k_next[i >> 1][i & 1], v[i] = v_next[i];
      if (j0 + 16 < k1) load(page, j0 + 16);
      page = j0 + 32 < k1 ? paged_page_again(p, b, j0 + 32) : -1;
      uint32_t bad = 0u;                    // bit i: value j0 + i is not finite
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (not_finite2(v[i].x) || not_finite2(v[i].y) || not_finite2(v[i].z) || not_finite2(v[i].w)) {
          bad |= 1u << (2 * c + (i & 1) + 8 * (i >> 1));
          v[i] = make_uint4(finite2(v[i].x), finite2(v[i].y), finite2(v[i].z), finite2(v[i].w));
        }
      }
      bad = __reduce_or_sync(0xffffffffu, bad);
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
        mma16816(s[n], q[0], k[n][0].x, k[n][0].y), mma16816(s[n], q[1], k[n][0].z, k[n][0].w);
        mma16816(s[n], q[2], k[n][1].x, k[n][1].y), mma16816(s[n], q[3], k[n][1].z, k[n][1].w);
      }
      float base[2], keep[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float top = m[u];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j0 + 2 * c + (i & 1) + 8 * (i >> 1);
          float &x = s[i >> 1][2 * u + (i & 1)];
          x = plain ? x * scale2 : paged_score(p, x, slope[u], abs(past + row_t[u] - j)) * kLog2e;
          x = j >= row_lo[u] && j < row_hi[u] ? x : -INFINITY;
          top = fmaxf(top, x);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        base[u] = top == -INFINITY ? 0.f : top;
        keep[u] = ex2_ftz(m[u] - base[u]), m[u] = top;
        l[u] *= keep[u];
        const uint32_t from = row_lo[u] > j0 ? 0xFFFFu << min(row_lo[u] - j0, 16) : 0xFFFFu;
        const uint32_t to = row_hi[u] > j0 ? 0xFFFFu >> max(16 - (row_hi[u] - j0), 0) : 0u;
        lost[u] |= (bad & from & to) != 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float &x = s[i >> 1][2 * u + (i & 1)];
          x = ex2_ftz(x - base[u]);
          l[u] += x;
        }
      }
      const uint32_t w[4] = {tc::pack_bf16x2(s[0][0], s[0][1]), tc::pack_bf16x2(s[0][2], s[0][3]),
                             tc::pack_bf16x2(s[1][0], s[1][1]), tc::pack_bf16x2(s[1][2], s[1][3])};
#pragma unroll
      for (int n = 0; n < 8; ++n) {         // column n of the threads' eight
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] *= keep[e >> 1];
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = n < 2 ? v[i].x : n < 4 ? v[i].y : n < 6 ? v[i].z : v[i].w;
        const uint32_t half_of = n & 1 ? 0x7632u : 0x5410u;
        mma16816(o[n], w, __byte_perm(x[0], x[1], half_of), __byte_perm(x[2], x[3], half_of));
      }
      if (__all_sync(0xffffffffu, lost[0] && lost[1])) break;
    }
    // columns 16 c + n (and + 8) of rows g, g + 8
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float sum = l[u];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (row_lo[u] >= row_hi[u]) continue;
      if (lost[u]) sum = __uint_as_float(0x7FFFFFFFu);
      if (p.splits > 1) {
        const size_t row = ((size_t)bh * p.splits + split) * ((size_t)p.T * p.rho) + (size_t)row_t[u] * p.rho + row_h[u] % p.rho;
        float4 *dst = reinterpret_cast<float4 *>(p.part_o + row * 64 + 16 * c);
        dst[0] = make_float4(o[0][2 * u], o[1][2 * u], o[2][2 * u], o[3][2 * u]);
        dst[1] = make_float4(o[4][2 * u], o[5][2 * u], o[6][2 * u], o[7][2 * u]);
        dst[2] = make_float4(o[0][2 * u + 1], o[1][2 * u + 1], o[2][2 * u + 1], o[3][2 * u + 1]);
        dst[3] = make_float4(o[4][2 * u + 1], o[5][2 * u + 1], o[6][2 * u + 1], o[7][2 * u + 1]);
        if (c == 0) p.part_ml[row] = make_float2(m[u], sum);
      } else {
        const float inv = 1.f / sum;
        uint4 *dst = reinterpret_cast<uint4 *>(paged_y<__nv_bfloat16>(p, b, row_h[u], row_t[u]) + 16 * c);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          dst[e] = make_uint4(tc::pack_bf16x2(o[0][2 * u + e] * inv, o[1][2 * u + e] * inv),
                              tc::pack_bf16x2(o[2][2 * u + e] * inv, o[3][2 * u + e] * inv),
                              tc::pack_bf16x2(o[4][2 * u + e] * inv, o[5][2 * u + e] * inv),
                              tc::pack_bf16x2(o[6][2 * u + e] * inv, o[7][2 * u + e] * inv));
      }
    }
    rows = after;
  }
}

}  // namespace oal
