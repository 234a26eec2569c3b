// Attention of packed rows over the paged cache: prompts of several sequences, and decode
// rows of sequences that share a prefix.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

#include <algorithm>

namespace qd {
namespace {

constexpr int kD = 128;
constexpr float kLog2e = 1.4426950408889634f;

// One warp per (row, q head), four dims per lane, one key at a time.
template <typename T>
__global__ void __launch_bounds__(128) attn_rows_kernel(const AttnRowsArgs a, int* err) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int row = (int)(w / a.Hq), h = (int)(w % a.Hq), g = h / (a.Hq / a.Hkv);
  bool bad = a.cu[0] < 0 || a.cu[a.n_seg] > a.n_rows;
  for (int i = lane; i < a.n_seg; i += 32) bad = bad || a.cu[i + 1] < a.cu[i];
  if (__any_sync(0xffffffffu, bad)) {
    if (w == 0 && lane == 0) set_error(err, QD_DEVERR_POS);
    return;
  }
  if (row < a.cu[0] || row >= a.cu[a.n_seg] || row >= a.n_rows) return;
  int lo = 0, hi = a.n_seg;   // the last segment that starts at or before the row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu[mid] <= row) lo = mid; else hi = mid;
  }
  const int seq = a.shared_lens ? row : lo;
  const int len = a.seq_lens[seq];
  const int n = a.shared_lens ? len : len - (a.cu[lo + 1] - row) + 1;
  if (len < 0 || len > a.max_pages * a.page_size) {
    if (lane == 0) set_error(err, QD_DEVERR_POS);
    return;
  }
  const size_t o = (size_t)h * kD + 4 * lane;
  float q[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = (float)((const T*)a.q)[(size_t)row * a.q_stride + o + e] * a.scale * kLog2e;
  for (int t = 0; t < n; ++t) {
    const PagedSlot sl = paged_slot(a.page_table + (size_t)seq * a.max_pages, t, a.page_size, a.n_pages);
    if (!sl.ok && lane == 0) set_error(err, QD_DEVERR_PAGE);
    const size_t at = (((size_t)sl.page * a.Hkv + g) * a.page_size + sl.slot) * kD + 4 * lane;
    const uint2 k = *(const uint2*)((const __nv_bfloat16*)a.k_pages + at);
    const uint2 v = *(const uint2*)((const __nv_bfloat16*)a.v_pages + at);
    const float s = warp_sum(q[0] * bf_lo(k.x) + q[1] * bf_hi(k.x) + q[2] * bf_lo(k.y) + q[3] * bf_hi(k.y));
    const float mn = fmaxf(m, s), al = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
    l = l * al + p;
    acc[0] = acc[0] * al + p * bf_lo(v.x);
    acc[1] = acc[1] * al + p * bf_hi(v.x);
    acc[2] = acc[2] * al + p * bf_lo(v.y);
    acc[3] = acc[3] * al + p * bf_hi(v.y);
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) ((T*)a.out)[(size_t)row * a.Hq * kD + o + e] = (T)(n > 0 ? acc[e] / l : 0.f);
}

}  // namespace

size_t attn_rows_workspace_bytes() { return 16; }
size_t attn_shared_workspace_bytes(int, int, int) { return 16; }

cudaError_t launch_attn_prompt(const AttnRowsArgs& a, const Launch& L) {
  const dim3 grid((unsigned)(((long long)a.n_rows * a.Hq + 3) / 4));
  return a.q_f32 ? launch_ex(attn_rows_kernel<float>, grid, dim3(128), 0, L, a, L.err)
                 : launch_ex(attn_rows_kernel<__nv_bfloat16>, grid, dim3(128), 0, L, a, L.err);
}

cudaError_t launch_attn_shared(const AttnRowsArgs& a, const Launch& L) { return launch_attn_prompt(a, L); }

}  // namespace qd
