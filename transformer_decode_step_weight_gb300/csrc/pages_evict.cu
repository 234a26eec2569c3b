// Eviction from the cache by the weights that keys have drawn (attention_window.cu,
// attention_weights.cu): of each sequence over its budget, every layer and kv head keeps its own
// tokens: the first n_sinks, the last n_recent, and those of the largest weights between. The kept
// ones move down in their order, K, V and weights, and the pages that are left over go back.
//
// Three launches: one CTA checks the whole call and lists the sequences that lose tokens (nothing
// changes where one of them cannot be done), a CTA per (layer, sequence, kv head) selects and moves,
// and the trim of pages.cu cuts tables, lengths and counts.
//
// Selection: the border between kept and not by radix over the weights as ordered integers (11, 11
// and 10 bits, a shared-memory histogram each; the row, some 10 KB, comes from L2), then one pass
// in token order in which equal weights count from the left. Moving is bound by HBM (6.0 TB/s read and written):
// 64 rows of K and V at a time through a ring of asynchronous copies. A kept token's new place r is
// below those of all later ones, and they lie at r + 1 or behind it, so a batch may be written while
// the loads of later ones are under way; it only has to have landed whole itself.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "page_plan.h"
#include "scan.cuh"

#include <algorithm>

namespace qd {
namespace {

constexpr int kPlan = 1024;
constexpr int kBins = 2048;
constexpr int kList = 1024;            // kept tokens found before they are moved
// Threads of a (layer, sequence, kv head), rows moved at a time, places of the ring: two CTAs an SM. One
// sequence of 28 layers 37 us, four of 36 layers 296; 256 threads with 32 rows, two places and four CTAs 46 and 307.
constexpr int kTh = 512, kBatch = 64, kStages = 3;
constexpr int kMaxHeadDim = 256;

// The tokens that stay, of n, without asking the weights: the first and the last.
struct Always {
  int first, last;
};
__host__ __device__ inline Always always(int keep, int n_sinks, int n_recent) {
  const int f = n_sinks < keep ? n_sinks : keep;
  return Always{f, n_recent < keep - f ? n_recent : keep - f};
}

// One CTA: sequences that lose tokens into ws.dst, their number into head[1], new lengths (-1: as it
// is) into ws.src.
__global__ void __launch_bounds__(kPlan) pages_evict_plan_kernel(PageState c, PagesWs ws, const int32_t* keep,
                                                                 int n_sinks, int n_recent, int* err) {
  __shared__ int warp_sums[kPlan / 32], s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = c.page_size;
  const long long cap = (long long)c.max_pages * ps;
  pdl_launch_dependents();   // the moves wait for this kernel before they read the list
  if (tid == 0) s_bad = 0;
  __syncthreads();
  for (int s = warp; s < c.max_seqs; s += kPlan / 32) {
    const int n = c.lens[s], k = keep[s];
    if (k < 0 || k >= n) {
      if (n < 0 && k >= 0 && lane == 0) atomicOr(&s_bad, QD_DEVERR_CACHE);
      continue;
    }
    if (n > cap) {
      if (lane == 0) atomicOr(&s_bad, QD_DEVERR_CACHE);
      continue;
    }
    // pages from the first token that may go on: they exist, and those that are written have one owner (none are
    // where first tokens alone stay)
    const int first = always(k, n_sinks, n_recent).first;
    const int p0 = first / ps, written = first < k ? pages_of(k, ps) : 0, all = pages_of(n, ps);
    int bad = 0;
    for (int i = p0 + lane; i < all; i += 32) {
      const int page = c.table[(size_t)s * c.max_pages + i];
      if (page < 0 || page >= c.n_pages) bad |= QD_DEVERR_CACHE | QD_DEVERR_PAGE;
      else if (i < written && c.refs[page] != 1) bad |= QD_DEVERR_CACHE;
    }
    if (bad) atomicOr(&s_bad, bad);
  }
  __syncthreads();
  const int bad = s_bad;
  if (bad && tid == 0) set_error(err, bad);
  int base = 0;
  for (int s0 = 0; s0 < c.max_seqs; s0 += kPlan) {
    const int s = s0 + tid;
    bool hit = false;
    if (s < c.max_seqs) {
      const int k = keep[s];
      hit = !bad && k >= 0 && k < c.lens[s];
      ws.src[s] = hit ? k : -1;
    }
    int total;
    const int at = block_scan(hit ? 1 : 0, warp_sums, total);
    if (hit) ws.dst[base + at - 1] = s;
    base += total;
  }
  if (tid == 0) ws.head[1] = base;
}

// A weight as an integer in the same order: -0 as 0, NaN as -infinity.
QD_DEV uint32_t order_of(float w) {
  const uint32_t b = __float_as_uint(w != w ? -INFINITY : w + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}

// Adds the bins from the top: the bin in which the `want`-th value from above lies, and how many lie
// above that bin (the whole CTA; 1 <= want <= all).
QD_DEV void find_bin(const int* hist, int want, int* warp_sums, int* s_out, int& bin, int& above) {
  constexpr int kPer = kBins / kTh;
  const int top = kBins - 1 - threadIdx.x * kPer;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) n += hist[top - i];
  int total;
  int at = block_scan(n, warp_sums, total) - n;
  if (at < want && at + n >= want) {
    int b = top;
    for (; at + hist[b] < want; --b) at += hist[b];
    s_out[0] = b;
    s_out[1] = at;
  }
  __syncthreads();
  bin = s_out[0];
  above = s_out[1];
  __syncthreads();
}

template <int VECS>
__global__ void __launch_bounds__(kTh, 2) pages_evict_kernel(const __grid_constant__ PagePtrs pk, PageState c, PagesWs ws,
                                                             const __grid_constant__ PageEvict e, const PageDiv div,
                                                             int layer0) {
  extern __shared__ __align__(128) unsigned char ring[];   // [kStages][K and V][kBatch rows]
  // (the bins are done with when the list begins)
  __shared__ int s_mem[3 * kList > kBins ? 3 * kList : kBins], warp_sums[kTh / 32], s_out[2];
  int *s_hist = s_mem, *s_src = s_mem, *s_dst = s_mem + kList;   // cache rows from and to; -1: it stays where it is
  float* s_val = (float*)(s_mem + 2 * kList);
  const int tid = threadIdx.x, g = blockIdx.x, l = blockIdx.z;
  const int vecs = VECS ? VECS : e.head_dim / 8, row = vecs * 16;   // a token's K in 16-byte pieces, and in bytes
  unsigned char *kp = pk.p[2 * l], *vp = pk.p[2 * l + 1];
  const long long cap = (long long)c.max_pages * c.page_size;
  pdl_wait();
  const int count = ws.head[1];
#pragma unroll 1
  for (int k = blockIdx.y; k < count; k += gridDim.y) {
    const int s = ws.dst[k], n = c.lens[s], keep = ws.src[s];
    const Always a = always(keep, e.n_sinks, e.n_recent);
    const int end = n - a.last, want = keep - a.first - a.last;   // the middle: [a.first, end), `want` of it stay
    float* w = e.weights + (((long long)(layer0 + l) * c.max_seqs + s) * e.n_kv_heads + g) * cap;

    // ---- the border: tokens above it stay, `equal` of those on it
    uint32_t border = 0xffffffffu;
    int equal = 0;
    if (want > 0) {
      int left = want;
      uint32_t prefix = 0;
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < kBins; i += kTh) s_hist[i] = 0;
        __syncthreads();
        for (int i = a.first + tid; i < end; i += kTh) {
          const uint32_t x = order_of(w[i]);
          if (pass == 0 || x >> (shift + bits) == prefix) atomicAdd(&s_hist[(x >> shift) & ((1u << bits) - 1u)], 1);
        }
        __syncthreads();
        int bin, above;
        find_bin(s_hist, left, warp_sums, s_out, bin, above);
        prefix = prefix << bits | (uint32_t)bin;
        left -= above;
      }
      border = prefix;
      equal = left;
    }

    // ---- kept tokens in order, up to kList at a time, and their moves
    auto place = [&](int t) {   // the cache row of a token
      const PagedSlot sl = paged_slot(c.table + (long long)s * c.max_pages, t, c.page_size, div, c.n_pages);
      return (sl.page * e.n_kv_heads + g) * c.page_size + sl.slot;
    };
    int next = a.first, kept = a.first, on_border = 0;   // the next token to look at; kept so far
#pragma unroll 1
    while (next < n) {
      int m = 0;                         // in the list
#pragma unroll 1
      while (next < n && m + kTh <= kList) {
        const int t = next + tid;
        const float v = t < n ? w[t] : 0.f;
        const uint32_t x = order_of(v);
        const bool middle = t < end;
        // both counts in one scan: equal ones so far below, kept ones above
        const int eq = t < n && middle && x == border && equal > 0;
        int total;
        const int eq_at = block_scan(eq, warp_sums, total) - eq;
        const bool stays = t < n && (!middle || (want > 0 && (x > border || (eq && on_border + eq_at < equal))));
        on_border += total;
        const int at = block_scan(stays ? 1 : 0, warp_sums, total);
        if (stays) {
          const int i = m + at - 1;
          const bool moves = t != kept + i;
          s_src[i] = moves ? place(t) : -1;
          s_dst[i] = moves ? place(kept + i) : -1;
          s_val[i] = v;
        }
        m += total;
        next += kTh;
      }
      __syncthreads();
      for (int i = tid; i < m; i += kTh)
        if (s_dst[i] >= 0) w[kept + i] = s_val[i];
      const int batches = (m + kBatch - 1) / kBatch;
      auto load = [&](int b) {
        if (b < batches) {
          const uint32_t dst = smem_u32(ring) + (uint32_t)(b % kStages) * (2 * kBatch * row);
#pragma unroll 4
          for (int i = tid; i < kBatch * vecs; i += kTh) {
            const int r = b * kBatch + i / vecs, v = i % vecs;
            if (r < m && s_src[r] >= 0) {
              const long long o = ((long long)s_src[r] * vecs + v) * 16;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 16), "l"(kp + o) : "memory");
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + kBatch * row + i * 16), "l"(vp + o)
                           : "memory");
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int b = 0; b < kStages - 1; ++b) load(b);
#pragma unroll 1
      for (int b = 0; b < batches; ++b) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();                 // batch b has landed whole, and the one before has been written
        load(b + kStages - 1);
        const unsigned char* src = ring + (size_t)(b % kStages) * (2 * kBatch * row);
#pragma unroll 4
        for (int i = tid; i < kBatch * vecs; i += kTh) {
          const int r = b * kBatch + i / vecs, v = i % vecs;
          if (r < m && s_dst[r] >= 0) {
            const long long o = ((long long)s_dst[r] * vecs + v) * 16;
            *(uint4*)(kp + o) = *(const uint4*)(src + i * 16);
            *(uint4*)(vp + o) = *(const uint4*)(src + kBatch * row + i * 16);
          }
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();                   // before the list and the ring are used again
      kept += m;
    }
    for (int i = keep + tid; i < n; i += kTh) w[i] = 0.f;
    __syncthreads();
  }
}

template <int VECS>
cudaError_t move(const PageState& c, const PageCopy& pc, const PageEvict& e, const PagesWs& ws, Launch L) {
  constexpr size_t kRowSmem = (size_t)kStages * 2 * kBatch * 2;
  cudaError_t rc = allow_smem<pages_evict_kernel<VECS>>(kRowSmem * kMaxHeadDim);   // (asked for once)
  for (int l0 = 0; rc == cudaSuccess && l0 < pc.n_layers; l0 += kPagePtrs / 2) {
    const int nl = std::min(kPagePtrs / 2, pc.n_layers - l0);
    PagePtrs pk = {};
    for (int i = 0; i < nl; ++i) {
      pk.p[2 * i] = (unsigned char*)pc.k_cache[l0 + i];
      pk.p[2 * i + 1] = (unsigned char*)pc.v_cache[l0 + i];
    }
    rc = launch_ex(pages_evict_kernel<VECS>, dim3(e.n_kv_heads, std::min(c.max_seqs, 64), nl), dim3(kTh),
                   kRowSmem * e.head_dim, L, pk, c, ws, e, make_page_div(c.page_size), l0);
    L.pdl = false;
  }
  return rc;
}

}  // namespace

cudaError_t launch_pages_evict(const PageState& c, const PageCopy& pc, const PageEvict& e, void* workspace,
                               const Launch& L) {
  const PagesWs ws = pages_ws(c, workspace);
  Launch first = L, moves = L, last = L;
  first.pdl = last.pdl = false;
  moves.pdl = true;
  cudaError_t rc = launch_ex(pages_evict_plan_kernel, dim3(1), dim3(kPlan), 0, first, c, ws, e.keep, e.n_sinks,
                             e.n_recent, L.err);
  if (rc != cudaSuccess) return rc;
  // (the model's own head size: no division by the row's length)
  rc = e.head_dim == 128 ? move<16>(c, pc, e, ws, moves) : move<0>(c, pc, e, ws, moves);
  if (rc != cudaSuccess) return rc;
  return launch_pages_trim(c, ws.src, last);
}

}  // namespace qd
