// Norms of the q and k heads of packed rows, the position rotation in the same pass, and the
// write of K and V into the paged cache: what stands between the QKV projection of several
// sequences' rows and the attention over them (qd_attn_prompt, qd_attn_prompt_window, the decode
// attentions).
//
//   y = w * x / sqrt(mean(x^2) + eps), y'[i] = y[i] cos_i - y[i + 64] sin_i,
//   y'[i + 64] = y[i + 64] cos_i + y[i] sin_i,  (cos_i, sin_i) = table[pos[axis(i)], i], i < 64
//
// HBM-bound: every row is read once and its q, k and v written once, some 37 KB a row (32 q heads,
// 8 kv heads, f32 in, bf16 out). A warp takes 8 heads of a row at a time, two beside each other: a half
// warp holds a head, lane i of it dims 4 i .. and 64 + 4 i .., so that the two of a rotated pair meet
// in one lane and loads are 16 bytes (f32). It walks an equal run of (row, 8 heads), the loads of the next
// under way while it works on one; a row's sequence, page and angles are looked up once for all of its
// heads in the run. Sums and angles are f32, the result is rounded once (with `cast` also after the
// division and after the weight, as the decode step of a bf16 model does).
//
// 8192 rows with three position axes: 51 us, 6.0 TB/s (one item a warp, without the next under way: 65;
// with a root and a division a head, and bf16 values rounded one by one: 56). 64 rows of one token: 4.8 us.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

#include <algorithm>

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
// The same as it was read, so that bf16 values wait in half the registers
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  F8 v;
  QD_DEV void load(const float* p) { v = load8(p); }
  QD_DEV F8 wide() const { return v; }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 a, b;
  QD_DEV void load(const __nv_bfloat16* p) {
    a = *(const uint2*)p;
    b = *(const uint2*)(p + 64);
  }
  QD_DEV F8 wide() const { return F8{widen(a), widen(b)}; }
};
QD_DEV uint2 narrow(float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  return make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
}
QD_DEV void store8(float* p, const F8& v) {
  *(float4*)p = v.a;
  *(float4*)(p + 64) = v.b;
}
QD_DEV void store8(__nv_bfloat16* p, const F8& v) {
  *(uint2*)p = narrow(v.a);
  *(uint2*)(p + 64) = narrow(v.b);
}

// w * (v * inv), with CAST rounded to bf16 after each product (that of two bf16 values is exact before it)
template <bool CAST>
QD_DEV void norm4(float4& v, float inv, uint2 w) {
  if constexpr (CAST) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv), hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
    const float2 a = __bfloat1622float2(lo), b = __bfloat1622float2(hi);
    const float2 x = __bfloat1622float2(__floats2bfloat162_rn(a.x * bf_lo(w.x), a.y * bf_hi(w.x)));
    const float2 y = __bfloat1622float2(__floats2bfloat162_rn(b.x * bf_lo(w.y), b.y * bf_hi(w.y)));
    v = make_float4(x.x, x.y, y.x, y.y);
  } else {
    v = make_float4(v.x * inv * bf_lo(w.x), v.y * inv * bf_hi(w.x), v.z * inv * bf_lo(w.y), v.w * inv * bf_hi(w.y));
  }
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

// What a row's heads need besides their values.
struct Row {
  int r;
  bool ok;                             // written at all
  float4 cs[2];                        // (cos, sin) of frequencies 4 hl, + 1 and + 2, + 3
  long long slot;                      // dim 4 hl of head 0 in the cache; -1: none
};
QD_DEV Row look_up(const QkRowsArgs& p, const PageDiv& div, int r, int lane, int* err) {
  const int hl = lane & 15;
  Row w;
  w.r = r;
  w.ok = false;
  w.slot = -1;
  const int b = segment_of(p.cu, p.batch, r, lane);
  const int row0 = p.cu[b], end = p.cu[b + 1], len = p.seq_lens[b];
  if (r < row0 || r >= end) return w;   // a row outside every sequence
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
  w.ok = __all_sync(0xffffffffu, ok);
  if (!w.ok) {
    if (lane == 0) set_error(err, QD_DEVERR_POS);
    return w;
  }
  if (p.n_axes == 1) {
    const float4* t = (const float4*)(p.rope + (long long)pos[0] * (kD / 2) + 4 * hl);
    w.cs[0] = t[0];
    w.cs[1] = t[1];
  } else {
    float2 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = p.rope[(long long)pos[i] * (kD / 2) + 4 * hl + i];
    w.cs[0] = make_float4(t[0].x, t[0].y, t[1].x, t[1].y);
    w.cs[1] = make_float4(t[2].x, t[2].y, t[3].x, t[3].y);
  }
  const PagedSlot sl = paged_slot(p.page_table + (long long)b * p.max_pages, (int)at, p.page_size, div, p.n_pages);
  if (sl.ok) w.slot = ((long long)sl.page * p.Hkv * p.page_size + sl.slot) * kD + 4 * hl;
  else if (lane == 0) set_error(err, QD_DEVERR_PAGE);
  return w;
}

template <typename TI, typename TO, bool CAST>
__global__ void __launch_bounds__(kTh, 2) qk_rows_kernel(const __grid_constant__ QkRowsArgs p, const PageDiv div,
                                                         int units, int* err) {
  const int lane = threadIdx.x & 31, hl = lane & 15;
  if (blockIdx.x == 0) {   // segments that make no sense
    for (int i = threadIdx.x; i < p.batch; i += kTh) {
      const int lo = p.cu[i], hi = p.cu[i + 1];
      if (lo < 0 || hi < lo || hi > p.n_rows) set_error(err, QD_DEVERR_POS);
    }
  }
  // the warp's run of (row, 8 heads)
  const long long items = (long long)p.n_rows * units;
  const long long warps = (long long)gridDim.x * (kTh / 32), me = (long long)blockIdx.x * (kTh / 32) + (threadIdx.x >> 5);
  long long it = items * me / warps;
  const long long last = items * (me + 1) / warps;
  if (it >= last) return;
  const int heads = p.Hq + 2 * p.Hkv;
  int r = (int)(it / units), u = (int)(it % units);
  Raw<TI> v[kPairs];
  auto load = [&](int row, int unit) {
    const TI* x = (const TI*)p.qkv + (long long)row * p.stride + 4 * hl;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int h = (unit * kPairs + i) * 2 + (lane >> 4);
      if (h < heads) v[i].load(x + (long long)h * kD);
    }
  };
  load(r, u);
  Row w = look_up(p, div, r, lane, err);
  Raw<__nv_bfloat16> gq, gk;
  gq.load((const __nv_bfloat16*)p.q_norm + 4 * hl);
  gk.load((const __nv_bfloat16*)p.k_norm + 4 * hl);
#pragma unroll 1
  for (;;) {
    F8 y[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) y[i] = v[i].wide();
    const int h0 = u * kPairs * 2 + (lane >> 4);   // heads h0, h0 + 2, ...
    const bool more = ++it < last;
    if (more) {
      if (++u == units) {
        u = 0;
        ++r;
      }
      load(r, u);
    }
    if (w.ok) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int h = h0 + 2 * i;
        // (both halves of the warp take part in the sum)
        float ss = 0.f;
        if (h < p.Hq + p.Hkv)
          ss = (y[i].a.x * y[i].a.x + y[i].a.y * y[i].a.y) + (y[i].a.z * y[i].a.z + y[i].a.w * y[i].a.w) +
               ((y[i].b.x * y[i].b.x + y[i].b.y * y[i].b.y) + (y[i].b.z * y[i].b.z + y[i].b.w * y[i].b.w));
#pragma unroll
        for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (h >= heads) continue;
        if (h < p.Hq + p.Hkv) {
          const float inv = rsqrtf(ss * (1.0f / kD) + p.eps);
          const uint2 ga = h < p.Hq ? gq.a : gk.a, gb = h < p.Hq ? gq.b : gk.b;
          norm4<CAST>(y[i].a, inv, ga);
          norm4<CAST>(y[i].b, inv, gb);
          auto turn = [](float& lo, float& hi, float c, float s) {
            const float l = lo * c - hi * s;
            hi = hi * c + lo * s;
            lo = l;
          };
          turn(y[i].a.x, y[i].b.x, w.cs[0].x, w.cs[0].y);
          turn(y[i].a.y, y[i].b.y, w.cs[0].z, w.cs[0].w);
          turn(y[i].a.z, y[i].b.z, w.cs[1].x, w.cs[1].y);
          turn(y[i].a.w, y[i].b.w, w.cs[1].z, w.cs[1].w);
        }
        if (h < p.Hq) {
          store8((TO*)p.q_out + ((long long)w.r * p.Hq + h) * kD + 4 * hl, y[i]);
        } else if (w.slot >= 0) {
          const int g = h - p.Hq;
          __nv_bfloat16* pages = (__nv_bfloat16*)(g < p.Hkv ? p.k_pages : p.v_pages);
          store8(pages + w.slot + (long long)(g < p.Hkv ? g : g - p.Hkv) * p.page_size * kD, y[i]);
        }
      }
    }
    if (!more) break;
    if (w.r != r) w = look_up(p, div, r, lane, err);
  }
}

template <typename TI, typename TO, bool CAST>
cudaError_t launch(const QkRowsArgs& a, const Launch& L) {
  const int units = ceil_div(a.Hq + 2 * a.Hkv, 2 * kPairs);
  // two CTAs an SM, each warp an equal run of items
  const long long ctas = std::min(2LL * dev_info().sm_count, ((long long)a.n_rows * units + kTh / 32 - 1) / (kTh / 32));
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
