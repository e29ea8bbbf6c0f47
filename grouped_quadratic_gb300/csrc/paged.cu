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

// Joins the rows of split keys, one warp a row: y = sum_s 2^{m_s - m} o_s /
// sum_s 2^{m_s - m} l_s over the splits that the row sees something of, in
// their order.
constexpr int kJoinThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(PagedArgs p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / p.Hkv, kv = bh % p.Hkv;
  const int r = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  if (r >= p.T * p.rho) return;
  const PagedSeq seq = paged_seq(p, b, false);
  const int t = r / p.rho, h = kv * p.rho + r % p.rho;
  if (t >= seq.n) return;
  const int2 sees = paged_sees(p, seq, b, t);
  const int base = paged_base(p, seq, r / p.tile_rows * p.tile_rows / p.rho);
  float2 y = make_float2(0.f, 0.f);
  if (sees.y > 0) {
    const int s0 = (sees.x - base) / p.split_keys, s1 = (sees.y - 1 - base) / p.split_keys;
    const size_t rows = (size_t)p.T * p.rho;
    const size_t first = (size_t)bh * p.splits * rows + r;
    float m = -INFINITY;
    for (int s = s0 + lane; s <= s1; s += 32) m = fmaxf(m, p.part_ml[first + s * rows].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (m == -INFINITY) m = 0.f;
    float l = 0.f;
#pragma unroll 4
    for (int s = s0; s <= s1; ++s) {
      const float2 ml = p.part_ml[first + s * rows];
      const float2 o = *reinterpret_cast<const float2 *>(p.part_o + (first + s * rows) * 64 + 2 * lane);
      const float w = exp2f(ml.x - m);
      l = fmaf(w, ml.y, l), y.x = fmaf(w, o.x, y.x), y.y = fmaf(w, o.y, y.y);
    }
    y.x /= l, y.y /= l;
    if (__any_sync(0xffffffffu, !(fabsf(y.x) + fabsf(y.y) < INFINITY)))
      y = paged_row_again<T>(p, b, h, t, sees.x, sees.y);
  }
  T *to = paged_y<T>(p, b, h, t) + 2 * lane;
  to[0] = from_f32<T>(y.x), to[1] = from_f32<T>(y.y);
}

}  // namespace

oal_status launch_paged_join(const PagedArgs &p, int is_bf16, cudaStream_t stream) {
  const unsigned rows = kJoinThreads / 32;
  const dim3 grid((unsigned)(((long long)p.T * p.rho + rows - 1) / rows), (unsigned)(p.B * p.Hkv));
  if (is_bf16)
    launch_pdl(paged_join_kernel<__nv_bfloat16>, grid, dim3(kJoinThreads), 0, stream, p);
  else
    launch_pdl(paged_join_kernel<float>, grid, dim3(kJoinThreads), 0, stream, p);
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

constexpr int kSplitLeast = 256;          // keys of a split at least

// The kernel's tile of rows, and into how many pieces the keys of a tile may be
// cut: as many as fill the GPU, where the tiles alone do not.  The grid is made
// for the longest sequence that the table has room for; blocks behind a
// sequence's end return at once.
static long long plan_tiles(PagedArgs &p, int is_bf16) {
  const long long rows = (long long)p.T * p.rho, units = (long long)p.B * p.Hkv;
  long long want;                         // blocks
  if (is_bf16 && rows > 32) {
    p.tile_rows = paged_tc_rows(p.T, p.rho);
    want = 152 * 4;
  } else if (is_bf16) {
    p.tile_rows = rows <= 16 ? 16 : 32;
    want = 152 * 2 * 4;
  } else {
    p.tile_rows = rows <= 8 ? 8 : 32;
    want = 152 * 4 * 2;
  }
  const long long tiles = units * ((rows + p.tile_rows - 1) / p.tile_rows);
  const long long most = (((long long)p.max_pages << p.page_shift) + kSplitLeast - 1) / kSplitLeast;
  return std::max<long long>(1, std::min(most, want / tiles));
}
static void plan_split(PagedArgs &p, long long pieces) {
  const long long room = (long long)p.max_pages << p.page_shift;
  long long span = room;                  // keys from a tile's first to its last
  if (p.window && !p.prefix) span = std::min(room, (long long)p.window + p.tile_rows / p.rho + 1 + kSplitAlign);
  const long long keys = std::max<long long>(kSplitLeast, (span + pieces - 1) / pieces);
  p.split_keys = (int)((keys + kSplitAlign - 1) / kSplitAlign * kSplitAlign);
  p.splits = (int)std::max<long long>(1, (span + p.split_keys - 1) / p.split_keys);
}

static size_t part_rows(const PagedArgs &p, long long splits) {
  return splits == 1 ? 0 : (size_t)p.B * p.Hkv * splits * p.T * p.rho;
}
constexpr size_t kPartBytes = 64 * sizeof(float) + sizeof(float2);
size_t paged_workspace_bytes(PagedArgs p, int is_bf16) {
  const size_t bytes = part_rows(p, plan_tiles(p, is_bf16)) * kPartBytes;   // whatever the window
  return std::max<size_t>(256, (bytes + 255) & ~(size_t)255);
}

oal_status launch_paged(PagedArgs p, int is_bf16, void *ws, cudaStream_t stream) {
  plan_split(p, plan_tiles(p, is_bf16));
  p.part_o = static_cast<float *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(p.part_o + part_rows(p, p.splits) * 64);
  if (!is_bf16) return launch_paged_simt(p, stream);
  return (long long)p.T * p.rho > 32 ? launch_paged_tc(p, stream) : launch_paged_rows(p, stream);
}

}  // namespace oal
