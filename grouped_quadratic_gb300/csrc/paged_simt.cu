// paged_simt.cu -- attention over a paged cache on the CUDA cores, for fp32.
//
//     y = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},   m = max_j s_j
// in one pass over the keys: maximum, sum and result of the keys so far are
// multiplied by e^{m_old - m_new} when the maximum grows.
//
// A block takes kRows rows (queries of one KV head, row t * rho + h') and walks
// 64 keys at a time through shared memory; a thread holds kRows / 8 rows of 4
// keys (scores) or 4 columns (results).  fp32 products: bound by the FMA pipes
// and shared memory together (8 16-byte loads for 64 FMAs), four blocks per SM
// hiding each other's loads and barriers.  1 x 3000 tokens, 4 heads: 179 us (27
// TFLOP/s); with the next tile in registers, two blocks per SM, 199.  One token: 16
// sequences of 8 KV heads on 4096 keys 105 us (2.6 TB/s), one of 2 on 32768 21 us;
// no tile is in flight while one is worked on.
#include <algorithm>

#include "paged.cuh"

namespace oal {
namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 64;
constexpr int kPitch = 68;                // floats of a row in shared memory: 4 banks on

template <int kRows>
struct SimtSmem {
  float q[kRows][kPitch], p[kRows][kPitch];
  float k[kKeys][kPitch], v[kKeys][kPitch];
};

__device__ __forceinline__ float4 row4(const float *row, int c) { return *reinterpret_cast<const float4 *>(row + c); }
__device__ __forceinline__ ulonglong2 row2(const float *row, int c) { return *reinterpret_cast<const ulonglong2 *>(row + c); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// One row once more, by a warp, over the keys [lo, hi) that it sees of a split:
// for rows whose result is not finite, which the value of a key that they do not
// see may be to blame for (0 times infinity or NaN).  A row that does see a bad key
// stays as it is, which a look at its keys tells first; then lanes take 32 keys for
// the scores, and the columns 2 l and 2 l + 1 of the values.
static __device__ __noinline__ void paged_row_again(const PagedArgs &p, int bh, int split, int past, int h, int t, int lo, int hi) {
  const int lane = threadIdx.x & 31, b = bh / p.Hkv, kv = bh % p.Hkv;
  const float *Kp = static_cast<const float *>(p.Kp), *Vp = static_cast<const float *>(p.Vp);
  const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p.Q) + (((size_t)b * p.Hq + h) * p.T + t) * 64);
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll 1
  for (int j0 = lo & ~15; j0 < hi; j0 += 16) {      // (16 keys lie on one page)
    const int page = paged_page_again(p, b, j0);
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {           // a lane takes 16 bytes of every other key
      const int j = j0 + 2 * i + (lane >> 4);
      if (page < 0 || j < lo || j >= hi) continue;
      const size_t at = paged_row(p, page, kv, j) + 4 * (lane & 15);
      const float4 k = *reinterpret_cast<const float4 *>(Kp + at), v = *reinterpret_cast<const float4 *>(Vp + at);
      worst += (k.x * 0.f + k.y * 0.f) + (k.z * 0.f + k.w * 0.f);         // (0 unless one is not finite)
      worst += (v.x * 0.f + v.y * 0.f) + (v.z * 0.f + v.w * 0.f);
    }
    if (__any_sync(0xffffffffu, worst != worst)) return;
  }
#pragma unroll 1
  for (int j0 = lo & ~31; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    const bool seen = j >= lo && j < hi;
    const int page = seen ? paged_page_again(p, b, j) : -1;
    float x = -INFINITY;
    if (seen) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (page >= 0) {
        const float4 *k = reinterpret_cast<const float4 *>(Kp + paged_row(p, page, kv, j));
#pragma unroll 8
        for (int d = 0; d < 16; ++d) {
          const float4 a = q[d], c = k[d];
          s.x = fmaf(a.x, c.x, s.x), s.y = fmaf(a.y, c.y, s.y), s.z = fmaf(a.z, c.z, s.z), s.w = fmaf(a.w, c.w, s.w);
        }
      }
      x = paged_score(p, (s.x + s.y) + (s.z + s.w), slope, abs(past + t - j));
    }
    float top = fmaxf(m, x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float base = top == -INFINITY ? 0.f : top, keep = expf(m - base), w = expf(x - base);
    m = top;
    l = l * keep + w, o0 *= keep, o1 *= keep;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
      const int pg = __shfl_sync(0xffffffffu, page, i);       // (-1: not seen, or zeros)
      const float f = __shfl_sync(0xffffffffu, w, i);
      if (pg >= 0) {
        const float2 v = *reinterpret_cast<const float2 *>(Vp + paged_row(p, pg, kv, j0 + i) + 2 * lane);
        o0 = fmaf(f, v.x, o0), o1 = fmaf(f, v.y, o1);
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (p.splits > 1) {
    const size_t row = ((size_t)bh * p.splits + split) * ((size_t)p.T * p.rho) + (size_t)t * p.rho + h % p.rho;
    *reinterpret_cast<float2 *>(p.part_o + row * 64 + 2 * lane) = make_float2(o0, o1);
    if (lane == 0) p.part_ml[row] = make_float2(m * kLog2e, l);
  } else {
    *reinterpret_cast<float2 *>(paged_y<float>(p, b, h, t) + 2 * lane) = make_float2(o0 / l, o1 / l);
  }
}

template <int kRows>
__global__ void __launch_bounds__(kThreads, kRows == 32 ? 4 : 1)
paged_simt_kernel(PagedArgs p) {
  pdl_trigger();
  pdl_wait();
  constexpr int R = kRows / 8;            // rows of a thread
  extern __shared__ uint8_t smem_raw[];
  SimtSmem<kRows> &s = *reinterpret_cast<SimtSmem<kRows> *>(smem_raw);
  __shared__ int s_lo, s_hi;
  const int bh = blockIdx.y, b = bh / p.Hkv, kv = bh % p.Hkv, split = blockIdx.z;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int r0 = blockIdx.x * kRows;
  const PagedSeq seq = paged_seq(p, b, tid == 0);
  const int t_first = r0 / p.rho;
  if (t_first >= seq.n) return;
  if (tid == 0) s_lo = INT32_MAX, s_hi = 0;
  __syncthreads();
  int lo[R], hi[R], at[R];                // keys seen, position
  float slope[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + ty * R + i, t = r / p.rho, h = r % p.rho;
    const bool live = t < seq.n;
    const int2 sees = live ? paged_sees(p, seq, b, t) : make_int2(0, 0);
    lo[i] = sees.x, hi[i] = sees.y, at[i] = seq.past + t;
    slope[i] = live && p.slopes ? p.slopes[kv * p.rho + h] : 0.f;
    if (tx == 0 && hi[i] > 0) atomicMin(&s_lo, lo[i]), atomicMax(&s_hi, hi[i]);
  }
  for (int x = tid; x < kRows * 16; x += kThreads) {
    const int r = r0 + (x >> 4), t = r / p.rho, h = r % p.rho;
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < seq.n)
      q = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.Q) +
                                            (((size_t)b * p.Hq + kv * p.rho + h) * p.T + t) * 64 + 4 * (x & 15));
    *reinterpret_cast<float4 *>(&s.q[x >> 4][4 * (x & 15)]) = q;
  }
  __syncthreads();
  int k0 = s_lo, k1 = s_hi;
  if (p.splits > 1) {
    const int from = paged_base(p, seq, t_first) + split * p.split_keys;
    k0 = max(k0, from), k1 = min(k1, from + p.split_keys);
    if (k0 >= k1) return;                 // (no row's interval reaches in: nothing is joined)
  }

  float m[R], l[R];
  float4 o[R];
#pragma unroll
  for (int i = 0; i < R; ++i) m[i] = -INFINITY, l[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  // A thread moves piece tid % 16 of rows tid / 16 + 8 i of a tile; 16 keys lie on one page.
  int page[kKeys / 16];
  auto look = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kKeys / 16; ++i) {
      const int j = j0 + 16 * i;
      page[i] = j < k1 && j + 16 > k0 ? paged_page(p, b, j) : -1;
    }
  };
  float4 kn[kKeys / 8], vn[kKeys / 8];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kKeys / 8; ++i) {
      const int j = j0 + (tid >> 4) + 8 * i;
      kn[i] = vn[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (page[i >> 1] >= 0 && j >= k0 && j < k1) {
        const size_t from = paged_row(p, page[i >> 1], kv, j) + 4 * (tid & 15);
        kn[i] = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.Kp) + from);
        vn[i] = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.Vp) + from);
      }
    }
  };
  look(k0 & ~(kKeys - 1));
  for (int j0 = k0 & ~(kKeys - 1); j0 < k1; j0 += kKeys) {
    fetch(j0);
    look(j0 + kKeys);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKeys / 8; ++i) {
      *reinterpret_cast<float4 *>(&s.k[(tid >> 4) + 8 * i][4 * (tid & 15)]) = kn[i];
      *reinterpret_cast<float4 *>(&s.v[(tid >> 4) + 8 * i][4 * (tid & 15)]) = vn[i];
    }
    __syncthreads();
    uint64_t x2[R][4];                    // sums over even and odd elements, side by side: half the instructions
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x2[i][e] = 0u;
#pragma unroll 4
    for (int d = 0; d < 64; d += 4) {
      ulonglong2 k[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = row2(s.k[tx + 16 * e], d);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const ulonglong2 q = row2(s.q[ty * R + i], d);
#pragma unroll
        for (int e = 0; e < 4; ++e) x2[i][e] = fma2(q.y, k[e].y, fma2(q.x, k[e].x, x2[i][e]));
      }
    }
    float x[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = __uint_as_float((uint32_t)x2[i][e]) + __uint_as_float((uint32_t)(x2[i][e] >> 32));
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float top = m[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + tx + 16 * e;
        const bool seen = j >= max(lo[i], k0) && j < min(hi[i], k1);
        x[i][e] = seen ? paged_score(p, x[i][e], slope[i], abs(at[i] - j)) : -INFINITY;
        top = fmaxf(top, x[i][e]);
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = expf(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = expf(x[i][e] - base);
        s.p[ty * R + i][tx + 16 * e] = w;
        sum += w;
      }
      m[i] = top;
      l[i] = l[i] * keep + sum;
      o[i].x *= keep, o[i].y *= keep, o[i].z *= keep, o[i].w *= keep;
    }
    __syncwarp();                         // (a row's weights come from its own half warp)
#pragma unroll 4
    for (int j = 0; j < kKeys; j += 4) {
      float4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = row4(s.v[j + e], 4 * tx);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float4 w = row4(s.p[ty * R + i], j);
        o[i].x = fmaf(w.x, v[0].x, fmaf(w.y, v[1].x, fmaf(w.z, v[2].x, fmaf(w.w, v[3].x, o[i].x))));
        o[i].y = fmaf(w.x, v[0].y, fmaf(w.y, v[1].y, fmaf(w.z, v[2].y, fmaf(w.w, v[3].y, o[i].y))));
        o[i].z = fmaf(w.x, v[0].z, fmaf(w.y, v[1].z, fmaf(w.z, v[2].z, fmaf(w.w, v[3].z, o[i].z))));
        o[i].w = fmaf(w.x, v[0].w, fmaf(w.y, v[1].w, fmaf(w.z, v[2].w, fmaf(w.w, v[3].w, o[i].w))));
      }
    }
  }

#pragma unroll
  for (int i = 0; i < R; ++i) {
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
    const int r = r0 + ty * R + i, t = r / p.rho, h = kv * p.rho + r % p.rho;
    const bool live = t < seq.n;
    const int a = max(lo[i], k0), z = min(hi[i], k1);          // of this split
    const float all = fabsf(o[i].x) + fabsf(o[i].y) + fabsf(o[i].z) + fabsf(o[i].w) + l[i];
    const bool wrong = live && a < z && !(all < INFINITY);
    if (live && p.splits > 1) {
      const size_t row = ((size_t)bh * p.splits + split) * ((size_t)p.T * p.rho) + r;
      *reinterpret_cast<float4 *>(p.part_o + row * 64 + 4 * tx) = o[i];
      if (tx == 0) p.part_ml[row] = make_float2(m[i] * kLog2e, l[i]);
    } else if (live) {
      // (a row that sees nothing: zeros whatever its o is, which a bad value times a weight of 0 may have reached)
      const float inv = 1.f / l[i];
      *reinterpret_cast<float4 *>(paged_y<float>(p, b, h, t) + 4 * tx) =
          a < z ? make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const uint32_t again = __ballot_sync(0xffffffffu, wrong);
    __syncwarp();                         // (other lanes write these rows then)
    for (int half = 0; half < 2; ++half)
      if (again >> (16 * half) & 0xFFFFu) {
        const int who = 16 * half;
        paged_row_again(p, bh, split, seq.past, __shfl_sync(0xffffffffu, h, who), __shfl_sync(0xffffffffu, t, who),
                        __shfl_sync(0xffffffffu, a, who), __shfl_sync(0xffffffffu, z, who));
      }
  }
}

template <int kRows>
oal_status run(const PagedArgs &p, cudaStream_t stream) {
  static bool done[kMaxDevices];
  const oal_status ready =
      paged_need_smem(reinterpret_cast<const void *>(paged_simt_kernel<kRows>), sizeof(SimtSmem<kRows>), done);
  if (ready != OAL_OK) return ready;
  const dim3 grid((unsigned)(((long long)p.T * p.rho + kRows - 1) / kRows), (unsigned)(p.B * p.Hkv), (unsigned)p.splits);
  launch_pdl(paged_simt_kernel<kRows>, grid, dim3(kThreads), sizeof(SimtSmem<kRows>), stream, p);
  const oal_status st = oal_after_launch("paged_simt_kernel", stream);
  return st != OAL_OK || p.splits == 1 ? st : launch_paged_join(p, 0, stream);
}

}  // namespace

oal_status launch_paged_simt(const PagedArgs &p, cudaStream_t stream) {
  return p.tile_rows == 8 ? run<8>(p, stream) : run<32>(p, stream);
}

}  // namespace oal
