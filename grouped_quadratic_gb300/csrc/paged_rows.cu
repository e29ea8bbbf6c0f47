// paged_rows.cu -- attention over a paged cache for bf16 and few rows: the next
// token of each sequence, or a handful of drafted ones.
//
// A block takes the queries of a KV head (16 kTiles rows at a time) over a run
// of keys; each of its warps walks its own groups of 32 keys, with a ring of
// asynchronous copies, an online softmax and a result of its own, and meets the
// others only at the end.  The products are mma.sync: 16 rows fill them, where a
// tcgen05 tile would be seven eighths empty and its scores with four threads a
// row; the work is HBM's, each key and value read once: 64 tokens on 2048 to 8192
// keys, 32/8 heads, 112 to 117 us (5.9 TB/s).
#include <algorithm>

#include "paged_again.cuh"

namespace oal {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kGroup = 32;                // keys of a warp's step
constexpr int kStages = 2;                // (three blocks per SM then; 3 and 4 leave two and one: 64 sequences 124, 143, 210 us)
constexpr int kGroupBytes = kGroup * 128; // of K, and of V
constexpr int kRing = kStages * 2 * kGroupBytes;

__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldm4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// kExtra: scores are capped or take a distance.
template <int kTiles, bool kExtra>
__global__ void __launch_bounds__(kThreads, 3)
paged_rows_kernel(PagedArgs p) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  constexpr int kRows = 16 * kTiles;
  static_assert(kRing >= kRows * 66 * 4, "the warps' results meet where the rings were");
  const int bh = blockIdx.y, b = bh / p.Hkv, kv = bh % p.Hkv, split = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int r0 = blockIdx.x * kRows, all = p.T * p.rho;
  const PagedSeq seq = paged_seq(p, b, threadIdx.x == 0);
  const int t_first = r0 / p.rho;
  if (t_first >= seq.n) return;

  // keys that some row sees, and those that all rows see
  int k0 = INT32_MAX, k1 = 0, in0 = 0, in1 = INT32_MAX;
  int lo = 0, hi = 0;                     // of row `lane`
  if (lane < kRows && r0 + lane < all && (r0 + lane) / p.rho < seq.n) {
    const int2 sees = paged_sees(p, seq, b, (r0 + lane) / p.rho);
    lo = sees.x, hi = sees.y;
    if (hi > 0) k0 = lo, k1 = hi;
    in0 = lo, in1 = hi;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    k0 = min(k0, __shfl_xor_sync(0xffffffffu, k0, d)), k1 = max(k1, __shfl_xor_sync(0xffffffffu, k1, d));
    in0 = max(in0, __shfl_xor_sync(0xffffffffu, in0, d)), in1 = min(in1, __shfl_xor_sync(0xffffffffu, in1, d));
  }
  if (p.splits > 1) {
    const int from = paged_base(p, seq, t_first) + split * p.split_keys;
    k0 = max(k0, from), k1 = min(k1, from + p.split_keys);
    if (k0 >= k1) return;                 // (no row's interval reaches in: nothing is joined)
  }

  uint32_t q[kTiles][4][4];
  int row_lo[kTiles][2], row_hi[kTiles][2], row_at[kTiles][2];
  float slope[kTiles][2];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = 16 * i + 8 * u + g, r = r0 + at, t = r / p.rho, h = kv * p.rho + r % p.rho;
      row_lo[i][u] = __shfl_sync(0xffffffffu, lo, at & 31), row_hi[i][u] = __shfl_sync(0xffffffffu, hi, at & 31);
      row_at[i][u] = seq.past + t;
      const bool live = r < all && t < seq.n;
      slope[i][u] = kExtra && live && p.slopes ? p.slopes[h] * kLog2e : 0.f;
      const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.Q) +
                                                              (((size_t)b * p.Hq + h) * p.T + t) * 64) + c;
#pragma unroll
      for (int k = 0; k < 4; ++k) q[i][k][u] = live ? src[8 * k] : 0u, q[i][k][2 + u] = live ? src[8 * k + 4] : 0u;
    }

  const uint32_t ring = smem_at(smem_raw) + warp * kRing;
  const int first = k1 > 0 ? (k0 & ~(kGroup - 1)) + warp * kGroup : 0;   // (no row sees anything: no step)
  const int steps = first < k1 ? (k1 - first + kWarps * kGroup - 1) / (kWarps * kGroup) : 0;
  // pages of a group's two halves (a page has 16 keys at least); -1: no key of it is wanted
  int page[kGroup / 16];
  auto look = [&](int it) {
#pragma unroll
    for (int u = 0; u < kGroup / 16; ++u) {
      const int j = first + it * kWarps * kGroup + 16 * u;
      page[u] = it < steps && j < k1 && j + 16 > k0 ? paged_page(p, b, j) : -1;
    }
  };
  const uint32_t to = (lane >> 3) * 128;    // (row lane / 8 + 4 i, piece lane % 8 on the swizzle)
  auto load = [&](int it) {
    if (it < steps) {
      const uint32_t dst = ring + it % kStages * (2 * kGroupBytes) + to;
      const int j0 = first + it * kWarps * kGroup + (lane >> 3);
#pragma unroll
      for (int i = 0; i < kGroup / 4; ++i) {
        const int j = j0 + 4 * i, pg = page[i >> 2];
        const bool there = pg >= 0 && j >= k0 && j < k1;
        const size_t from = there ? paged_row(p, pg, kv, j) + 8 * (lane & 7) : 0;
        const uint32_t at = dst + 512 * i + (((lane & 7) ^ ((lane >> 3) + 4 * (i & 1))) << 4);
        copy16(at, static_cast<const __nv_bfloat16 *>(p.Kp) + from, there);
        copy16(at + kGroupBytes, static_cast<const __nv_bfloat16 *>(p.Vp) + from, there);
      }
    }
    copy_commit();
  };

  float m[kTiles][2], l[kTiles][2], o[kTiles][8][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
#pragma unroll
    for (int u = 0; u < 2; ++u) m[i][u] = -INFINITY, l[i][u] = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
  }
  const float scale2 = p.scale * kLog2e;
  const float cap_in = kExtra && p.cap > 0.f ? 2.f * kLog2e * p.scale / p.cap : 0.f, cap_out = p.cap * kLog2e;

#pragma unroll
  for (int it = 0; it < kStages - 1; ++it) look(it), load(it);
  look(kStages - 1);
#pragma unroll 1
  for (int it = 0; it < steps; ++it) {
    copy_wait<kStages - 2>();
    __syncwarp();
    load(it + kStages - 1);
    look(it + kStages);
    const int j0 = first + it * kWarps * kGroup;
    const uint32_t kt = ring + it % kStages * (2 * kGroupBytes), vt = kt + kGroupBytes;
    float s[kTiles][kGroup / 8][4];
#pragma unroll
    for (int n = 0; n < kGroup / 8; ++n) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[4];
        ldm4(kt + (8 * n + (lane & 7)) * 128 + (((4 * h + (lane >> 3)) ^ (lane & 7)) << 4), x);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) mma(s[i][n], q[i][2 * h], x[0], x[1]), mma(s[i][n], q[i][2 * h + 1], x[2], x[3]);
      }
    }
    const bool whole = j0 >= max(in0, k0) && j0 + kGroup <= min(in1, k1);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      float top[2] = {m[i][0], m[i][1]};
      if (kExtra && p.cap > kCapNear) {
#pragma unroll
        for (int n = 0; n < kGroup / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][n][e] = paged_cap_far(s[i][n][e], p.scale / p.cap, cap_in, cap_out);
      } else if (kExtra && p.cap > 0.f) {
#pragma unroll
        for (int n = 0; n < kGroup / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][n][e] = paged_cap_near(s[i][n][e], cap_in, cap_out);
      } else {
#pragma unroll
        for (int n = 0; n < kGroup / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][n][e] *= scale2;
      }
      if (kExtra) {                         // (one conversion a row: those take the exponentials' units)
        const float far[2] = {(float)(row_at[i][0] - j0 - 2 * c), (float)(row_at[i][1] - j0 - 2 * c)};
#pragma unroll
        for (int n = 0; n < kGroup / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[i][n][e] = fmaf(-slope[i][e >> 1], fabsf(far[e >> 1] - (float)(8 * n + (e & 1))), s[i][n][e]);
      }
      if (!whole) {
#pragma unroll
        for (int n = 0; n < kGroup / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int u = e >> 1, j = j0 + 8 * n + 2 * c + (e & 1);
            if (!(j >= max(row_lo[i][u], k0) && j < min(row_hi[i][u], k1))) s[i][n][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int n = 0; n < kGroup / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[i][n][e]);
      float keep[2];
      bool grew = false;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 1));
        top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 2));
        grew |= top[u] > m[i][u];
        const float base = top[u] == -INFINITY ? 0.f : top[u];
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(keep[u]) : "f"(m[i][u] - base));
        m[i][u] = top[u], top[u] = base;
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) l[i][u] *= keep[u];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][n][e] *= keep[e >> 1];
      }
#pragma unroll
      for (int n = 0; n < kGroup / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s[i][n][e]) : "f"(s[i][n][e] - top[e >> 1]));
          l[i][e >> 1] += s[i][n][e];
        }
    }
    // the weights, rounded to bf16 (by 2^-8 of each at most), are left factors as they lie
#pragma unroll
    for (int k = 0; k < kGroup / 16; ++k) {
      uint32_t w[kTiles][4];
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i][e] = pack(s[i][2 * k + (e >> 1)][2 * (e & 1)], s[i][2 * k + (e >> 1)][2 * (e & 1) + 1]);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t x[4];
        ldm4t(vt + (16 * k + (lane & 15)) * 128 + (((2 * n + (lane >> 4)) ^ (lane & 7)) << 4), x);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) mma(o[i][2 * n], w[i], x[0], x[1]), mma(o[i][2 * n + 1], w[i], x[2], x[3]);
      }
    }
    __syncwarp();
  }
  copy_wait<0>();
  __syncthreads();

  // the warps' rows meet in shared memory
  float *mine = reinterpret_cast<float *>(smem_raw) + warp * kRows * 66;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float sum = l[i][u];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      float *row = mine + (16 * i + 8 * u + g) * 66;
      if (c == 0) row[64] = m[i][u], row[65] = sum;
#pragma unroll
      for (int n = 0; n < 8; ++n) *reinterpret_cast<float2 *>(row + 8 * n + 2 * c) = make_float2(o[i][n][2 * u], o[i][n][2 * u + 1]);
    }
  }
  __syncthreads();
  uint32_t again = 0u;                    // the warp's rows whose result is not finite
  for (int at = warp; at < kRows; at += kWarps) {
    const int r = r0 + at, t = r / p.rho, h = kv * p.rho + r % p.rho;
    if (r >= all || t >= seq.n) break;
    const float *row = reinterpret_cast<const float *>(smem_raw) + at * 66;
    float top = -INFINITY, sum = 0.f;
    float2 y = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, row[w * kRows * 66 + 64]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float *x = row + w * kRows * 66;
      const float f = exp2f(x[64] - base);
      sum = fmaf(f, x[65], sum), y.x = fmaf(f, x[2 * lane], y.x), y.y = fmaf(f, x[2 * lane + 1], y.y);
    }
    if (__any_sync(0xffffffffu, !(fabsf(y.x) + fabsf(y.y) + sum < INFINITY))) again |= 1u << at;
    if (p.splits > 1) {
      const size_t to_row = ((size_t)bh * p.splits + split) * all + r;
      *reinterpret_cast<float2 *>(p.part_o + to_row * 64 + 2 * lane) = y;
      if (lane == 0) p.part_ml[to_row] = make_float2(top, sum);
      continue;
    }
    if (__shfl_sync(0xffffffffu, hi, at) > 0)
      y.x /= sum, y.y /= sum;
    else
      y = make_float2(0.f, 0.f);
    *reinterpret_cast<uint32_t *>(paged_y<__nv_bfloat16>(p, b, h, t) + 2 * lane) = pack(y.x, y.y);
  }
  if (again != 0u) {
    const int r = r0 + lane;
    const bool mine = again >> lane & 1u;
    __syncwarp();                         // (other lanes write these rows now)
    paged_rows_again(p, bh, split, seq.past, kv * p.rho + r % p.rho, r / p.rho, mine ? max(lo, k0) : 0, mine ? min(hi, k1) : 0);
  }
}

template <int kTiles, bool kExtra>
oal_status run(const PagedArgs &p, cudaStream_t stream) {
  static bool done[kMaxDevices];
  auto kernel = paged_rows_kernel<kTiles, kExtra>;
  const oal_status ready = paged_need_smem(reinterpret_cast<const void *>(kernel), kWarps * kRing, done);
  if (ready != OAL_OK) return ready;
  const dim3 grid((unsigned)((p.T * p.rho + 16 * kTiles - 1) / (16 * kTiles)), (unsigned)(p.B * p.Hkv), (unsigned)p.splits);
  launch_pdl(kernel, grid, dim3(kThreads), kWarps * kRing, stream, p);
  const oal_status st = oal_after_launch("paged_rows_kernel", stream);
  return st != OAL_OK || p.splits == 1 ? st : launch_paged_join(p, 1, stream);
}

}  // namespace

oal_status launch_paged_rows(const PagedArgs &p, cudaStream_t stream) {
  const bool extra = p.cap > 0.f || p.slopes;
  if (p.tile_rows == 16) return extra ? run<1, true>(p, stream) : run<1, false>(p, stream);
  return extra ? run<2, true>(p, stream) : run<2, false>(p, stream);
}

}  // namespace oal
