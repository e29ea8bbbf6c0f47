// paged.cuh -- rotary positions, the paged cache and the attention over it:
// arguments and what the kernels share.
#pragma once
#include "oal_internal.cuh"

namespace oal {

// ---------------------------------------------------------------- rotation, append

// Element (b, h, t, 0) of a tensor whose rows of 64 are contiguous.
struct RowStrides {
  long long b, h, t;
};

struct RopeArgs {
  const void *Q, *K, *V;                  // K, V may be null
  void *Yq, *Yk;                          // contiguous; Yk null where K goes to pages
  void *Kp, *Vp;                          // pages, or null
  RowStrides q, k, v;
  int B, Hq, Hkv, T;
  const unsigned long long *turns;        // [32] angle a position, in turns of 2^64; null: nothing turns
  const long long *axes;                  // [32] axis of each pair
  const int32_t *positions;               // [n_axes][B][T], or null: past + t
  int n_axes;
  const int32_t *past, *lengths;          // [B] or null
  const int32_t *table;
  int n_pages, page_shift, max_pages;
  long long page_stride;
  int inverse;
  int *status;
};

// ---------------------------------------------------------------- attention

struct PagedArgs {
  const void *Q, *Kp, *Vp;
  void *Y;
  const int32_t *table, *past, *lengths, *prefix, *first;   // lengths, prefix, first may be null
  const float *slopes;                    // [Hq] or null
  int B, Hq, Hkv, T, rho;
  int n_pages, page_shift, max_pages;
  long long page_stride;                  // elements from page to page
  float scale, cap;                       // cap: 0 = none
  int window;                             // 0 = none
  int *status;
  // The split of the keys: an item's tile of `tile_rows` rows (row t * rho + h'
  // of the KV head's queries) over keys base + [s, s + 1) * split_keys.
  int tile_rows, splits, split_keys;
  float *part_o;                          // [B * Hkv][splits][T * rho][64], not yet divided
  float2 *part_ml;                        // the same rows' maximum (base 2) and sum
};

// A sequence's place in its pages.
struct PagedSeq {
  int n, past, total;                     // new tokens, tokens before them, keys
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs &p, int b, bool record) {
  PagedSeq s;
  const int n = p.lengths ? p.lengths[b] : p.T, past = p.past[b];
  const int room = p.max_pages << p.page_shift;
  s.n = min(max(n, 0), p.T);
  s.past = min(max(past, 0), room);
  s.total = min(s.past + s.n, room);
  if (record && (n != s.n || past != s.past || s.past + s.n > room))
    atomicCAS(p.status, kStatusOk, (int)OAL_ERR_INVALID_ARG);
  return s;
}

// The keys that token t may see: every mask leaves an interval [lo, hi).
__device__ __forceinline__ int2 paged_sees(const PagedArgs &p, const PagedSeq &s, int b, int t) {
  const int i = s.past + t;
  int lo = p.window ? max(0, i + 1 - p.window) : 0, hi = i + 1;
  if (p.first) lo = max(lo, p.first[(size_t)b * p.T + t]);
  if (p.prefix) hi = max(hi, p.prefix[b]);
  hi = min(hi, s.total);
  if (lo >= hi) lo = hi = 0;
  return make_int2(lo, hi);
}

// First key of the splits of the tile that starts at token t: at or before
// every key that the tile's rows see, and known without looking at the rows.
constexpr int kSplitAlign = 128;
__device__ __forceinline__ int paged_base(const PagedArgs &p, const PagedSeq &s, int t) {
  return p.window ? max(0, s.past + t + 1 - p.window) & ~(kSplitAlign - 1) : 0;
}

// The page that holds key j, or -1 (a bad entry, which is recorded; its keys
// count as zeros).
__device__ __forceinline__ int paged_page(const PagedArgs &p, int b, int j) {
  const int page = p.table[(size_t)b * p.max_pages + (j >> p.page_shift)];
  if (page >= 0 && page < p.n_pages) return page;
  atomicCAS(p.status, kStatusOk, (int)OAL_ERR_INVALID_ARG);
  return -1;
}
// The same for keys that were looked up before (loads may pass it).
__device__ __forceinline__ int paged_page_again(const PagedArgs &p, int b, int j) {
  const int page = p.table[(size_t)b * p.max_pages + (j >> p.page_shift)];
  return page >= 0 && page < p.n_pages ? page : -1;
}
__device__ __forceinline__ size_t paged_row(const PagedArgs &p, int page, int kv, int j) {
  return (size_t)page * p.page_stride +
         (((size_t)kv << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * 64;
}

// The score in units of the exponent's base 2: cap, then distance.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float paged_score(const PagedArgs &p, float qk, float slope, int distance) {
  float s = qk * p.scale;
  if (p.cap > 0.f) s = p.cap * tanhf(s / p.cap);
  s -= slope * (float)distance;
  return s;
}

// Caps of bf16's scores, in units of the exponent's base 2: cap tanh(f), f = qk
// in_cap, in two forms.  cap - 2 cap / (e^{2 f} + 1) is off by up to 2^-22 of the cap,
// which is nothing up to kCapNear (1.5e-5 of a score) and more than small scores
// are under large caps.  Up to kTanhSpan, tanh(f) = f (c0 + c1 f^2 + .. + c4 f^8) to
// 6e-8 of itself, by least squares at Chebyshev's points.
constexpr float kCapNear = 64.f, kTanhSpan = 0.625f;
constexpr float kTanh0 = 0.9999998807907104f, kTanh1 = -0.3333197236061096f, kTanh2 = 0.13304771482944489f,
                kTanh3 = -0.05183185636997223f, kTanh4 = 0.015063672326505184f;
__device__ __forceinline__ float paged_cap_near(float qk, float cap_in, float cap_out) {   // cap_in = 2 log2(e) in_cap
  float w;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(qk * cap_in));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(w + 1.f));
  return fmaf(-2.f * cap_out, w, cap_out);
}
__device__ __forceinline__ float paged_cap_far(float qk, float in_cap, float cap_in, float cap_out) {
  const float f = qk * in_cap, f2 = f * f;
  const float q = fmaf(fmaf(fmaf(fmaf(f2, kTanh4, kTanh3), f2, kTanh2), f2, kTanh1), f2, kTanh0);
  return fabsf(f) <= kTanhSpan ? cap_out * (f * q) : paged_cap_near(qk, cap_in, cap_out);
}

// Rows of 64 for Y.
template <typename T>
__device__ __forceinline__ T *paged_y(const PagedArgs &p, int b, int h, int t) {
  return static_cast<T *>(p.Y) + (((size_t)b * p.Hq + h) * p.T + t) * 64;
}

// A kernel's dynamic shared memory, once a device.
oal_status paged_need_smem(const void *kernel, size_t bytes, bool (&done)[kMaxDevices]);
oal_status launch_paged_join(const PagedArgs &p, int is_bf16, cudaStream_t stream);

}  // namespace oal
