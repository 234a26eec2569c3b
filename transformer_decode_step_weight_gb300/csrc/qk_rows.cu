// Norms of the q and k heads of packed rows, the position rotation in the same pass, and the
// write of K and V into the paged cache: what stands between the QKV projection of several
// sequences' rows and the attention over them (qd_attn_prompt, qd_attn_prompt_window, the decode
// attentions).
//
//   y = w * x / sqrt(mean(x^2) + eps), y'[i] = y[i] cos_i - y[i + 64] sin_i,
//   y'[i + 64] = y[i + 64] cos_i + y[i] sin_i,  (cos_i, sin_i) = table[pos[axis(i)], i], i < 64
//
// HBM-bound: every row is read once and its q, k and v written once, some 37 KB a row (32 q heads,
// 8 kv heads, f32 in, bf16 out). A warp has one row and up to 8 of its heads, two at a time: a half
// warp holds a head, lane i of it dims 4 i .. and 64 + 4 i .., so that the two of a rotated pair meet
// in one lane and loads are 16 bytes (f32). All of a warp's loads go out before the first use, and
// the row's angles are read once for its 8 heads; the row's sequence and page are looked up beside
// them. Sums and angles are f32, the result is rounded once (with `cast` also after the division
// and after the weight, as the decode step of a bf16 model does).
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace qd {
namespace {

constexpr int kD = 128;
constexpr int kTh = 256;
constexpr int kPairs = 4;              // pairs of heads per warp

struct F8 {
  float4 a, b;                         // dims 4 i .., 64 + 4 i ..
};
QD_DEV F8 load8(const float* p) { return F8{*(const float4*)p, *(const float4*)(p + 64)}; }
QD_DEV float4 widen(uint2 w) { return make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)); }
QD_DEV F8 load8(const __nv_bfloat16* p) { return F8{widen(*(const uint2*)p), widen(*(const uint2*)(p + 64))}; }
QD_DEV uint2 narrow(float4 v) {
  return make_uint2(f2bf_bits(v.x) | f2bf_bits(v.y) << 16, f2bf_bits(v.z) | f2bf_bits(v.w) << 16);
}
QD_DEV void store8(float* p, const F8& v) {
  *(float4*)p = v.a;
  *(float4*)(p + 64) = v.b;
}
QD_DEV void store8(__nv_bfloat16* p, const F8& v) {
  *(uint2*)p = narrow(v.a);
  *(uint2*)(p + 64) = narrow(v.b);
}

// The sequence of packed row r, by a whole warp: the number of segments that end at or before r,
// in two looks of 32 (batch <= 1024). Not a segment of r's if r lies outside all of them.
QD_DEV int segment_of(const int32_t* cu, int batch, int r, int lane) {
  const int step = (batch + 31) >> 5;
  const int e = min((lane + 1) * step, batch);
  const int c = __popc(__ballot_sync(0xffffffffu, (lane == 0 || e > lane * step) && cu[e] <= r));
  const int first = min(c * step, batch - 1);
  const int i = min(first + lane + 1, batch);
  const int n = __popc(__ballot_sync(0xffffffffu, lane < step && first + lane < batch && cu[i] <= r));
  return min(first + n, batch - 1);
}

template <typename TI, typename TO, bool CAST>
__global__ void __launch_bounds__(kTh) qk_rows_kernel(const __grid_constant__ QkRowsArgs p, const PageDiv div,
                                                      int units, int* err) {
  const int lane = threadIdx.x & 31, hl = lane & 15;
  const long long item = (long long)blockIdx.x * (kTh / 32) + (threadIdx.x >> 5);
  if (blockIdx.x == 0) {   // segments that make no sense
    for (int i = threadIdx.x; i < p.batch; i += kTh) {
      const int lo = p.cu[i], hi = p.cu[i + 1];
      if (lo < 0 || hi < lo || hi > p.n_rows) set_error(err, QD_DEVERR_POS);
    }
  }
  const int r = (int)(item / units);
  if (r >= p.n_rows) return;
  const int heads = p.Hq + 2 * p.Hkv;
  const int h0 = (int)(item % units) * 2 * kPairs + (lane >> 4);   // heads h0, h0 + 2, ...
  const TI* x = (const TI*)p.qkv + (long long)r * p.stride + 4 * hl;
  F8 v[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    if (h0 + 2 * i < heads) v[i] = load8(x + (long long)(h0 + 2 * i) * kD);

  const int b = segment_of(p.cu, p.batch, r, lane);
  const int row0 = p.cu[b], end = p.cu[b + 1], len = p.seq_lens[b];
  if (r < row0 || r >= end) return;   // a row outside every sequence
  const long long cap = (long long)p.max_pages * p.page_size, at = (long long)len - end + r;
  bool ok = len <= cap && at >= 0;
  // the position of each of the lane's four frequencies
  int pos[4];
  const uint32_t axes = (p.axes[hl >> 2] >> (8 * (hl & 3))) & 0xffu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    pos[i] = p.positions ? p.positions[(long long)((axes >> (2 * i)) & 3u) * p.n_rows + r] : (int)at;
    ok = ok && pos[i] >= 0 && pos[i] < p.rope_max_pos;
  }
  if (!__all_sync(0xffffffffu, ok)) {
    if (lane == 0) set_error(err, QD_DEVERR_POS);
    return;
  }
  float4 cs[2];   // (cos, sin) of frequencies 4 hl, + 1 and + 2, + 3
  if (p.n_axes == 1) {
    const float4* t = (const float4*)(p.rope + (long long)pos[0] * (kD / 2) + 4 * hl);
    cs[0] = t[0];
    cs[1] = t[1];
  } else {
    float2 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = p.rope[(long long)pos[i] * (kD / 2) + 4 * hl + i];
    cs[0] = make_float4(t[0].x, t[0].y, t[1].x, t[1].y);
    cs[1] = make_float4(t[2].x, t[2].y, t[3].x, t[3].y);
  }
  long long slot = -1;   // of head 0 in the cache
  if (h0 + 2 * kPairs > p.Hq) {
    const PagedSlot sl = paged_slot(p.page_table + (long long)b * p.max_pages, (int)at, p.page_size, div, p.n_pages);
    if (sl.ok) slot = ((long long)sl.page * p.Hkv * p.page_size + sl.slot) * kD + 4 * hl;
    else if (lane == 0) set_error(err, QD_DEVERR_PAGE);
  }
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int h = h0 + 2 * i;
    F8 y = v[i];
    // (both halves of the warp take part in the sum)
    float ss = 0.f;
    if (h < p.Hq + p.Hkv)
      ss = (y.a.x * y.a.x + y.a.y * y.a.y) + (y.a.z * y.a.z + y.a.w * y.a.w) +
           ((y.b.x * y.b.x + y.b.y * y.b.y) + (y.b.z * y.b.z + y.b.w * y.b.w));
#pragma unroll
    for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (h >= heads) continue;
    if (h < p.Hq + p.Hkv) {
      const float inv = 1.0f / sqrtf(ss / (float)kD + p.eps);
      const __nv_bfloat16* w = (const __nv_bfloat16*)(h < p.Hq ? p.q_norm : p.k_norm) + 4 * hl;
      const F8 g = load8(w);
      auto norm = [&](float& e, float gw) {
        e *= inv;
        if (CAST) e = round_bf16(e);
        e *= gw;
        if (CAST) e = round_bf16(e);
      };
      norm(y.a.x, g.a.x); norm(y.a.y, g.a.y); norm(y.a.z, g.a.z); norm(y.a.w, g.a.w);
      norm(y.b.x, g.b.x); norm(y.b.y, g.b.y); norm(y.b.z, g.b.z); norm(y.b.w, g.b.w);
      auto turn = [](float& lo, float& hi, float c, float s) {
        const float l = lo * c - hi * s;
        hi = hi * c + lo * s;
        lo = l;
      };
      turn(y.a.x, y.b.x, cs[0].x, cs[0].y);
      turn(y.a.y, y.b.y, cs[0].z, cs[0].w);
      turn(y.a.z, y.b.z, cs[1].x, cs[1].y);
      turn(y.a.w, y.b.w, cs[1].z, cs[1].w);
    }
    if (h < p.Hq) {
      store8((TO*)p.q_out + ((long long)r * p.Hq + h) * kD + 4 * hl, y);
    } else if (slot >= 0) {
      const int g = h - p.Hq;
      __nv_bfloat16* pages = (__nv_bfloat16*)(g < p.Hkv ? p.k_pages : p.v_pages);
      store8(pages + slot + (long long)(g < p.Hkv ? g : g - p.Hkv) * p.page_size * kD, y);
    }
  }
}

template <typename TI, typename TO, bool CAST>
cudaError_t launch(const QkRowsArgs& a, const Launch& L) {
  const int units = ceil_div(a.Hq + 2 * a.Hkv, 2 * kPairs);
  const long long ctas = ((long long)a.n_rows * units + kTh / 32 - 1) / (kTh / 32);
  return launch_ex(qk_rows_kernel<TI, TO, CAST>, dim3((unsigned)ctas), dim3(kTh), 0, L, a, make_page_div(a.page_size),
                   units, L.err);
}

template <typename TI, typename TO>
cudaError_t launch(const QkRowsArgs& a, const Launch& L) {
  return a.cast ? launch<TI, TO, true>(a, L) : launch<TI, TO, false>(a, L);
}

}  // namespace

cudaError_t launch_qk_rows(const QkRowsArgs& a, const Launch& L) {
  if (a.in_f32) return a.out_f32 ? launch<float, float>(a, L) : launch<float, __nv_bfloat16>(a, L);
  return a.out_f32 ? launch<__nv_bfloat16, float>(a, L) : launch<__nv_bfloat16, __nv_bfloat16>(a, L);
}

}  // namespace qd
