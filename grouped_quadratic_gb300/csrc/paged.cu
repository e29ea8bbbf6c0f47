// paged.cu -- attention over a paged cache: which kernel, how the keys are split,
// and the join of split rows.
#include <algorithm>

#include "paged.cuh"

namespace oal {

oal_status launch_paged_simt(const PagedArgs &p, cudaStream_t stream);
oal_status launch_paged_rows(const PagedArgs &p, cudaStream_t stream);
int paged_tc_rows(int T, int rho);
oal_status launch_paged_tc(const PagedArgs &p, cudaStream_t stream);

namespace {

// Joins the rows of split keys: y = sum_s 2^{m_s - m} o_s / sum_s 2^{m_s - m} l_s
// over the splits that the row sees something of.  A row has kJoinWarps warps,
// each with every kJoinWarps-th split, in order, and their sums are added in
// order: the same bits every time.  Eight splits a warp are one step, 2 us with
// the launch, and each further step costs another 2: 129 splits took 10 us with
// four warps; but 6,216 rows of 4 splits take 16 us (cold) with four warps, 6.6
// with one.
constexpr int kJoinThreads = 128;
template <typename T, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps > 4 ? 32 * kJoinWarps : kJoinThreads)
paged_join_kernel(PagedArgs p) {
  pdl_trigger();
  pdl_wait();
  constexpr int kRows = kJoinWarps > 4 ? 1 : kJoinThreads / 32 / kJoinWarps;   // of a block
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  __shared__ float2 s_y[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % kJoinWarps;
  const int bh = blockIdx.y, b = bh / p.Hkv, kv = bh % p.Hkv;
  const int r = blockIdx.x * kRows + (threadIdx.x >> 5) / kJoinWarps;
  if (r >= p.T * p.rho) return;
  const PagedSeq seq = paged_seq(p, b, false);
  const int t = r / p.rho, h = kv * p.rho + r % p.rho;
  if (t >= seq.n) return;
  const int2 sees = paged_sees(p, seq, b, t);
  const int base = paged_base(p, seq, r / p.tile_rows * p.tile_rows / p.rho);
  float2 y = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  if (sees.y > 0) {
    const int s0 = (sees.x - base) / p.split_keys, s1 = (sees.y - 1 - base) / p.split_keys;
    const size_t rows = (size_t)p.T * p.rho;
    const size_t first = (size_t)bh * p.splits * rows + r;
    for (int s = s0 + warp; s <= s1; s += 8 * kJoinWarps) {   // eight splits' loads in flight
      float2 ml[8], o[8];
      float top = m;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = s + e * kJoinWarps;
        ml[e] = make_float2(-INFINITY, 0.f), o[e] = make_float2(0.f, 0.f);
        if (at <= s1) {
          ml[e] = p.part_ml[first + at * rows];
          o[e] = *reinterpret_cast<const float2 *>(p.part_o + (first + at * rows) * 64 + 2 * lane);
        }
        top = fmaxf(top, ml[e].x);
      }
      const float zero = top == -INFINITY ? 0.f : top, keep = exp2f(m - zero);
      l *= keep, y.x *= keep, y.y *= keep, m = top;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float w = s + e * kJoinWarps <= s1 ? exp2f(ml[e].x - zero) : 0.f;
        l = fmaf(w, ml[e].y, l), y.x = fmaf(w, o[e].x, y.x), y.y = fmaf(w, o[e].y, y.y);
      }
    }
  }
  if (kJoinWarps > 1) {                   // (one row a block)
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    s_y[warp][lane] = y;
    __syncthreads();
    if (warp != 0) return;
    float top = s_m[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, s_m[w]);
    if (top == -INFINITY) top = 0.f;
    l = 0.f, y = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = exp2f(s_m[w] - top);
      const float2 o = s_y[w][lane];
      l = fmaf(f, s_l[w], l), y.x = fmaf(f, o.x, y.x), y.y = fmaf(f, o.y, y.y);
    }
  }
  if (sees.y > 0)
    y.x /= l, y.y /= l;
  else
    y = make_float2(0.f, 0.f);
  T *to = paged_y<T>(p, b, h, t) + 2 * lane;
  to[0] = from_f32<T>(y.x), to[1] = from_f32<T>(y.y);
}

}  // namespace

oal_status launch_paged_join(const PagedArgs &p, int is_bf16, cudaStream_t stream) {
  // warps a row: so that eight splits each are enough, up to 16
  const int warps = p.splits <= 8 ? 1 : p.splits <= 32 ? 4 : 16, each = warps == 1 ? kJoinThreads / 32 : 1;
  const dim3 grid((unsigned)((p.T * p.rho + each - 1) / each), (unsigned)(p.B * p.Hkv));
  auto kernel = is_bf16 ? (warps == 1   ? paged_join_kernel<__nv_bfloat16, 1>
                           : warps == 4 ? paged_join_kernel<__nv_bfloat16, 4>
                                        : paged_join_kernel<__nv_bfloat16, 16>)
                        : (warps == 1   ? paged_join_kernel<float, 1>
                           : warps == 4 ? paged_join_kernel<float, 4>
                                        : paged_join_kernel<float, 16>);
  launch_pdl(kernel, grid, dim3(warps == 16 ? 512 : kJoinThreads), 0, stream, p);
  return oal_after_launch("paged_join_kernel", stream);
}

oal_status paged_need_smem(const void *kernel, size_t bytes, bool (&done)[kMaxDevices]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return oal_fail(OAL_ERR_CUDA, "no current device");
  if (done[dev]) return OAL_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
    return oal_check_launch("shared memory of a paged kernel");
  done[dev] = true;
  return OAL_OK;
}

// Keys of a split at least: a bf16 block's start and end cost more than 256 keys, an fp32 block's less.
// (256 for both: 2 x 300 tokens of 4 fp32 heads 32 us instead of 24.5; 128 for both: one bf16 token on 32768
// keys 3 us more.)
static int split_least(int is_bf16) { return is_bf16 ? 256 : 128; }
constexpr int kRowsMost = 32;             // rows a KV head up to which bf16 goes by paged_rows_kernel
// Keys of a split of paged_rows_kernel at most.  Its four warps add to accumulators that the tensor cores cut: values
// of one sign come out 1.7e-3 low after 2^20 keys, 4e-4 after these, a tenth of a bf16's rounding.
constexpr int kRowsKeys = 1 << 18;

// The kernel's tile of rows, and into how many pieces the keys of a tile may be
// cut: as many as fill the GPU, where the tiles alone do not.  The grid is made
// for the longest sequence that the table has room for; blocks behind a
// sequence's end return at once.  So a table far wider than its sequences leaves
// the GPU part empty: 8 tokens on 4096 keys each, 32/8 heads, 15.0 us with a table
// of 4096 keys and 32.9 with one of 131072; 128 tokens on 2000, 13.0 and 28.0.
//
// paged_rows_kernel, three blocks of which fit an SM: with few units (pairs of
// sequence and KV head) about one wave, four blocks per SM of which a ragged
// batch leaves some empty; with many, enough waves to even out their ends.  4,
// 8 and 16 blocks per SM, us: 16 sequences of 8 heads with 2048 to 8192 keys
// 35.3, 37.8, 42.2; 8 with 32768 at most 57.8, 60.7, 66.4; 32 with 5 drafted
// tokens on 3000 43.9, 47.3, 52.5; but 64 with 8192 129, 117.8, 116.6, all of
// one length 209, 180, 168.
static long long plan_tiles(PagedArgs &p, int is_bf16) {
  const long long rows = (long long)p.T * p.rho, units = (long long)p.B * p.Hkv;
  long long want;                         // blocks
  if (is_bf16 && rows > kRowsMost) {
    p.tile_rows = paged_tc_rows(p.T, p.rho);
    want = 152 * 4;
  } else if (is_bf16) {
    p.tile_rows = rows <= 16 ? 16 : 32;
    want = units * ((rows + p.tile_rows - 1) / p.tile_rows) <= 2 * 152 ? 152 * 4 : 152 * 16;
  } else {
    p.tile_rows = rows <= 8 ? 8 : 32;
    want = 152 * 4 * 2;
  }
  const long long tiles = units * ((rows + p.tile_rows - 1) / p.tile_rows);
  const long long least = split_least(is_bf16), most = (((long long)p.max_pages << p.page_shift) + least - 1) / least;
  return std::max<long long>(1, std::min(most, want / tiles));
}
// ... and must be, of so many keys.
static long long plan_fewest(const PagedArgs &p, int is_bf16, long long span) {
  return is_bf16 && (long long)p.T * p.rho <= kRowsMost ? (span + kRowsKeys - 1) / kRowsKeys : 1;
}
static void plan_split(PagedArgs &p, int is_bf16, long long pieces) {
  const long long room = (long long)p.max_pages << p.page_shift;
  long long span = room;                  // keys from a tile's first to its last
  if (p.window && !p.prefix) span = std::min(room, (long long)p.window + p.tile_rows / p.rho + 1 + kSplitAlign);
  auto keys_of = [&](long long n) {
    const long long keys = std::max<long long>(split_least(is_bf16), (span + n - 1) / n);
    return (keys + kSplitAlign - 1) / kSplitAlign * kSplitAlign;
  };
  const long long rows = (long long)p.T * p.rho, units = (long long)p.B * p.Hkv;
  pieces = std::max(pieces, plan_fewest(p, is_bf16, span));
  if (is_bf16 && rows > kRowsMost && pieces > 1) {
    // paged_tc_kernel: the fewest waves of one block per SM, a wave's time in keys: its blocks' and 700 that a block
    // costs beside; 300 and the partial results of 130 rows a key for the join.  114 tiles on 65536 keys: 4 pieces,
    // three full waves, 371 us; 5 pieces 399, 3 pieces 465.  16 tiles on 4300 keys: 3 pieces 23.0, 2 and 4 26.5, 28.2.
    const long long tiles = units * ((rows + p.tile_rows - 1) / p.tile_rows), most = pieces;
    long long best = INT64_MAX;
    for (long long n = 1; n <= most; ++n) {
      const long long keys = keys_of(n), cuts = (span + keys - 1) / keys;
      const long long cost = (tiles * cuts + 151) / 152 * (keys + 700) + (cuts > 1 ? 300 + units * rows * cuts / 130 : 0);
      if (cost < best) best = cost, pieces = n;
    }
  }
  p.split_keys = (int)keys_of(pieces);
  p.splits = (int)std::max<long long>(1, (span + p.split_keys - 1) / p.split_keys);
}

static size_t part_rows(const PagedArgs &p, long long splits) {
  return splits == 1 ? 0 : (size_t)p.B * p.Hkv * splits * p.T * p.rho;
}
constexpr size_t kPartBytes = 64 * sizeof(float) + sizeof(float2);
size_t paged_workspace_bytes(PagedArgs p, int is_bf16) {
  const long long room = (long long)p.max_pages << p.page_shift;            // (whatever the window)
  const size_t bytes = part_rows(p, std::max(plan_tiles(p, is_bf16), plan_fewest(p, is_bf16, room))) * kPartBytes;
  return std::max<size_t>(256, (bytes + 255) & ~(size_t)255);
}

oal_status launch_paged(PagedArgs p, int is_bf16, void *ws, cudaStream_t stream) {
  plan_split(p, is_bf16, plan_tiles(p, is_bf16));
  p.part_o = static_cast<float *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(p.part_o + part_rows(p, p.splits) * 64);
  if (!is_bf16) return launch_paged_simt(p, stream);
  return (long long)p.T * p.rho > kRowsMost ? launch_paged_tc(p, stream) : launch_paged_rows(p, stream);
}

}  // namespace oal
