// Page operations on the paged K/V cache: copy, fork, extend, trim, compact.
//
// State, all in device memory: table[s, i] is the page of sequence s's tokens
// [i ps, (i + 1) ps) (-1 past its last page), lens[s] its tokens, refs[p] the number of
// table entries that name page p (0: free). There is no free list: a page is free when
// nothing names it, and new pages are the lowest free ids, taken in sequence order, so
// the result of a call depends on its arguments alone and not on the history or on the
// order of threads. (Integer atomics on refs commute.)
//
// A fork shares every page of its parent, the partly filled last one too; whoever is
// extended first copies that page (copy on write), and the last sharer keeps it. A call
// that cannot be carried out whole (no free pages left, a length past the table, a bad
// sequence id) changes nothing and sets QD_DEVERR_CACHE. A table entry that names no page is a fault
// of the caller's, met only where the work is under way: it is passed over and QD_DEVERR_PAGE set.
//
// The copies are bound by HBM (16 KB per CTA turn, eight 16-byte loads per thread under way, eight
// CTAs per SM): 783 MB read and written in some 130 us, 6.0 TB/s. Planning is latency: one CTA,
// since a scan over the counts of a few thousand pages costs less than a grid's barrier. 63 forks
// of a 4101-token prompt, 36 layers: fork 4 us, the plan of the extension 10, one page each (149 MB
// written) 27; compaction of 40 sequences' pages, 28 layers: 136 us; two pages, 36 layers: 2.5 us.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "page_plan.h"
#include "scan.cuh"

#include <algorithm>

namespace qd {
namespace {

constexpr int kPlan = 1024;            // threads of the planning kernels (one CTA)
constexpr int kCopyTh = 128;
constexpr int kCopyVec = 8;            // 16-byte pieces in flight per thread
constexpr int kItem = kCopyTh * kCopyVec * 16;   // bytes a CTA copies at a time
constexpr int kForkTh = 128;

// One CTA walks the pages [lo, hi) in ascending order, 16 per thread at a time (each
// warp 512 consecutive ones, 16 coalesced loads in flight), and calls put(rank, page) for
// those with (refs == 0) == want_free, rank counting from `base`; stops once `limit` are
// found. Returns base + the number found so far (the whole CTA). hi <= 2^30: the indexes of the
// last turn stay within 32 bits.
template <typename Put>
QD_DEV int walk_pages(const int32_t* refs, int lo, int hi, bool want_free, int base, int limit, int* warp_sums,
                      Put put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kPer = 16;
  for (int b = lo; b < hi && base < limit; b += kPlan * kPer) {
    const int first = b + warp * 32 * kPer + lane;
    int r[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) r[k] = first + 32 * k < hi ? refs[first + 32 * k] : -1;
    unsigned hit[kPer];
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      hit[k] = __ballot_sync(0xffffffffu, r[k] >= 0 && (r[k] == 0) == want_free);
      n += __popc(hit[k]);
    }
    int total;
    // lane 31 of every warp carries the warp's count: the scan there is the running total
    int at = block_scan(lane == 31 ? n : 0, warp_sums, total);
    at = base + __shfl_sync(0xffffffffu, at, 31) - n;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if ((hit[k] >> lane) & 1) {
        const int rank = at + __popc(hit[k] & ((1u << lane) - 1u));
        if (rank < limit) put(rank, first + 32 * k);
      }
      at += __popc(hit[k]);
    }
    base += total;
  }
  return base;
}

// ---- page copies: pair i of the list, every cache pointer, in items of 16 KB. The
// copies of one source (a page forked to many children) are neighbours, so it comes from
// L2 after its first read.
__global__ void __launch_bounds__(kCopyTh) pages_copy_kernel(const __grid_constant__ PagePtrs pk, int n_ptrs,
                                                             const int32_t* src, const int32_t* dst, int n,
                                                             const int32_t* n_dev, int n_pages, long long page_bytes,
                                                             int* err) {
  pdl_wait();
  if (n_dev) n = *n_dev;
  const int per_page = (int)((page_bytes + kItem - 1) / kItem);
  const long long items = (long long)n * n_ptrs * per_page;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int pair = (int)(it % n);
    const long long rest = it / n;
    const int c = (int)(rest % per_page), l = (int)(rest / per_page);
    const int a = src[pair], b = dst[pair];
    if (a < 0 || b < 0) continue;   // a pair with a negative id is skipped
    if (a >= n_pages || b >= n_pages) {
      if (threadIdx.x == 0) set_error(err, QD_DEVERR_PAGE);
      continue;
    }
    const long long o = (long long)c * kItem + threadIdx.x * 16;
    const unsigned char* from = pk.p[l] + (long long)a * page_bytes + o;
    unsigned char* to = pk.p[l] + (long long)b * page_bytes + o;
    uint4 v[kCopyVec];
#pragma unroll
    for (int j = 0; j < kCopyVec; ++j)
      if (o + j * kCopyTh * 16 < page_bytes) v[j] = *(const uint4*)(from + j * kCopyTh * 16);
#pragma unroll
    for (int j = 0; j < kCopyVec; ++j)
      if (o + j * kCopyTh * 16 < page_bytes) *(uint4*)(to + j * kCopyTh * 16) = v[j];
  }
}

// ---- fork: CTA i gives child i its parent's row. Each CTA checks the whole call first
// (a bitmap of the children); the lengths are written by the last CTA to finish, so that
// every CTA has seen the children empty.
__global__ void __launch_bounds__(kForkTh) pages_fork_kernel(PageState c, PagesWs ws, const int32_t* parents,
                                                             const int32_t* children, int n, int* err) {
  extern __shared__ uint32_t seen[];
  __shared__ int s_bad, s_last;
  const int tid = threadIdx.x, words = (c.max_seqs + 31) / 32;
  const long long cap = (long long)c.max_pages * c.page_size;
  for (int i = tid; i < words; i += kForkTh) seen[i] = 0;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kForkTh) {
    const int p = parents[i], q = children[i];
    bool ok = p >= 0 && p < c.max_seqs && q >= 0 && q < c.max_seqs && p != q;
    if (ok) ok = c.lens[p] >= 0 && c.lens[p] <= cap && c.lens[q] == 0;
    if (ok) ok = !((atomicOr(&seen[q >> 5], 1u << (q & 31)) >> (q & 31)) & 1u);
    if (!ok) s_bad = 1;
  }
  __syncthreads();
  if (s_bad) {   // the same in every CTA
    if (tid == 0) set_error(err, QD_DEVERR_CACHE);
    return;
  }
  const int par = parents[blockIdx.x], kid = children[blockIdx.x];
  const int len = c.lens[par], np = pages_of(len, c.page_size);
  for (int i = tid; i < c.max_pages; i += kForkTh) {
    int e = -1;
    if (i < np) {
      e = c.table[(size_t)par * c.max_pages + i];
      if (e >= 0 && e < c.n_pages) atomicAdd(c.refs + e, 1);
      else set_error(err, QD_DEVERR_PAGE);
    }
    c.table[(size_t)kid * c.max_pages + i] = e;
  }
  if (tid == 0) ws.src[blockIdx.x] = len;
  __syncthreads();
  if (tid == 0) s_last = atom_add_acq_rel_gpu(ws.head, 1) == n - 1;
  __syncthreads();
  if (!s_last) return;
  for (int i = tid; i < n; i += kForkTh) c.lens[children[i]] = __ldcg(ws.src + i);
  if (tid == 0) ws.head[0] = 0;
}

// ---- extend: one CTA plans. Per sequence: the pages it needs (and whether its shared
// last page has to be copied), a prefix sum over the sequences, the lowest free ids into
// ws.map, then the table rows, the counts and the list of copies.
__global__ void __launch_bounds__(kPlan) pages_extend_kernel(PageState c, PagesWs ws, const int32_t* n_new, int* err) {
  extern __shared__ __align__(16) int32_t sh[];
  pdl_launch_dependents();   // the copies wait for this kernel before they read the list
  int32_t* cand = sh;                     // [max_seqs] a shared last page, or -1
  int32_t* at = cand + c.max_seqs;        // [max_seqs] first new page of the sequence
  int32_t* need = at + c.max_seqs;        // [max_seqs] the page's count, then what it takes (PageNeed)
  __shared__ PageSum sums[kPlan / 32];
  __shared__ int warp_sums[kPlan / 32], s_bad, s_copies;
  const int tid = threadIdx.x, ps = c.page_size;
  const long long cap = (long long)c.max_pages * ps;
  if (tid == 0) s_bad = s_copies = 0;
  __syncthreads();
  for (int s = tid; s < c.max_seqs; s += kPlan) {
    const int n = max(n_new[s], 0), len = c.lens[s];
    int q = -1;
    if (n > 0) {
      if (len < 0 || (long long)len + n > cap) {
        atomicOr(&s_bad, QD_DEVERR_CACHE);
      } else if (len % ps) {
        const int p = c.table[(size_t)s * c.max_pages + len / ps];
        if (p < 0 || p >= c.n_pages) atomicOr(&s_bad, QD_DEVERR_CACHE | QD_DEVERR_PAGE);
        else if (const int r = c.refs[p]; r > 1) {
          q = p;
          need[s] = r;
        }
      }
    }
    cand[s] = q;
  }
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      set_error(err, s_bad);
      ws.head[1] = 0;
    }
    return;
  }
  PageSum base = 0;
  for (int s0 = 0; s0 < c.max_seqs; s0 += kPlan) {
    const int s = s0 + tid;
    PageSum w = 0;
    if (s < c.max_seqs) {
      const int q = cand[s];
      bool copy = false;
      if (q >= 0) {   // the sharers extended before this one have left the page
        int before = 0, j = 0;
        for (; j + 4 <= s; j += 4) {
          const int4 p = *(const int4*)(cand + j);
          before += (p.x == q) + (p.y == q) + (p.z == q) + (p.w == q);
        }
        for (; j < s; ++j) before += cand[j] == q;
        copy = need[s] - before > 1;
      }
      const PageNeed x = page_need(c.lens[s], max(n_new[s], 0), ps, copy);
      need[s] = (int)x.bits;
      w = x.pages();
    }
    PageSum total;
    const PageSum incl = block_scan(w, sums, total);
    if (s < c.max_seqs) at[s] = (int)(base + incl - w);   // (used where all of them exist)
    base += total;
  }
  const PageSum want = base;
  // at most n_pages ids fit the list (and exist)
  const int found = want > c.n_pages
                        ? 0
                        : walk_pages(c.refs, 0, c.n_pages, true, 0, (int)want, warp_sums,
                                     [&](int rank, int page) { ws.map[rank] = page; });
  __syncthreads();
  if (found < want) {
    if (tid == 0) {
      set_error(err, QD_DEVERR_CACHE);
      ws.head[1] = 0;
    }
    return;
  }
  // one warp per sequence writes its row
  const int lane = tid & 31, warp = tid >> 5;
  for (int s = warp; s < c.max_seqs; s += kPlan / 32) {
    const int n = max(n_new[s], 0);
    if (n == 0) continue;
    const int len = c.lens[s], had = pages_of(len, ps);
    const PageNeed x = {(uint32_t)need[s]};
    const int w = x.pages();
    const bool copy = x.copy();
    const int row0 = copy ? had - 1 : had;
    for (int i = lane; i < w; i += 32) {
      const int page = ws.map[at[s] + i];
      c.table[(size_t)s * c.max_pages + row0 + i] = page;
      c.refs[page] = 1;
      if (copy && i == 0) {
        // the place of a copy in the list does not matter: the pairs are disjoint
        const int k = atomicAdd(&s_copies, 1);
        ws.src[k] = cand[s];
        ws.dst[k] = page;
        atomicSub(c.refs + cand[s], 1);
      }
    }
    __syncwarp();
    if (lane == 0) c.lens[s] = len + n;
  }
  __syncthreads();
  if (tid == 0) ws.head[1] = s_copies;
}

// ---- trim: one CTA per sequence
__global__ void __launch_bounds__(kForkTh) pages_trim_kernel(PageState c, const int32_t* new_lens, int* err) {
  const int s = blockIdx.x, n = new_lens[s], len = c.lens[s];
  if (n < 0 || n >= len) return;
  const int had = min(pages_of(len, c.page_size), c.max_pages);
  for (int i = pages_of(n, c.page_size) + threadIdx.x; i < had; i += kForkTh) {
    int32_t* e = c.table + (size_t)s * c.max_pages + i;
    if (*e >= 0 && *e < c.n_pages) atomicSub(c.refs + *e, 1);
    else set_error(err, QD_DEVERR_PAGE);
    *e = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) c.lens[s] = n;
}

// ---- compact: one CTA plans. n = pages in use; the used ids >= n move, in ascending
// order, to the free ids < n.
__global__ void __launch_bounds__(kPlan) pages_compact_kernel(PageState c, PagesWs ws, int32_t* n_live) {
  __shared__ int warp_sums[kPlan / 32];
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  const int n = walk_pages(c.refs, 0, c.n_pages, false, 0, INT32_MAX, warp_sums, [](int, int) {});
  const int holes = walk_pages(c.refs, 0, n, true, 0, INT32_MAX, warp_sums,
                               [&](int rank, int page) { ws.dst[rank] = page; });
  walk_pages(c.refs, n, c.n_pages, false, 0, INT32_MAX, warp_sums, [&](int rank, int page) { ws.src[rank] = page; });
  __syncthreads();
  for (int i = tid; i < holes; i += kPlan) {
    const int a = ws.src[i], b = ws.dst[i];
    ws.map[a] = b;
    c.refs[b] = c.refs[a];
    c.refs[a] = 0;
  }
  if (tid == 0) {
    ws.head[1] = holes;
    ws.head[2] = n;
    *n_live = n;
  }
}

// table entries of the moved pages; one CTA per sequence, its pages only
__global__ void __launch_bounds__(kForkTh) pages_remap_kernel(PageState c, PagesWs ws, int* err) {
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x, n = ws.head[2];
  const int had = min(pages_of(max(c.lens[s], 0), c.page_size), c.max_pages);
  for (int i = threadIdx.x; i < had; i += kForkTh) {
    int32_t* e = c.table + (size_t)s * c.max_pages + i;
    if (*e < 0 || *e >= c.n_pages) set_error(err, QD_DEVERR_PAGE);
    else if (*e >= n) *e = ws.map[*e];
  }
}

cudaError_t copy_pairs(const PageCopy& pc, const int32_t* src, const int32_t* dst, int n, const int32_t* n_dev,
                       int n_pages, const Launch& L) {
  const int per_page = (int)((pc.page_bytes + kItem - 1) / kItem);
  for (int l0 = 0; l0 < pc.n_layers; l0 += kPagePtrs / 2) {
    const int nl = std::min(kPagePtrs / 2, pc.n_layers - l0);
    PagePtrs pk = {};
    for (int i = 0; i < nl; ++i) {
      pk.p[2 * i] = (unsigned char*)pc.k_cache[l0 + i];
      pk.p[2 * i + 1] = (unsigned char*)pc.v_cache[l0 + i];
    }
    const long long fill = 8LL * dev_info().sm_count;
    const long long items = n_dev ? fill : (long long)n * 2 * nl * per_page;
    Launch Lc = L;
    Lc.pdl = l0 == 0 && L.pdl;
    cudaError_t e = launch_ex(pages_copy_kernel, dim3((unsigned)std::min(items, fill)), dim3(kCopyTh), 0, Lc, pk,
                              2 * nl, src, dst, n, n_dev, n_pages, (long long)pc.page_bytes, L.err);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t pages_workspace_bytes(int max_seqs, int n_pages) {
  return (64 + 3 * (size_t)std::max(max_seqs, n_pages)) * 4;
}

cudaError_t launch_pages_copy(const PageCopy& pc, const int32_t* src, const int32_t* dst, int n, int n_pages,
                              const Launch& L) {
  return copy_pairs(pc, src, dst, n, nullptr, n_pages, L);
}

cudaError_t launch_pages_fork(const PageState& c, const int32_t* parents, const int32_t* children, int n,
                              void* workspace, const Launch& L) {
  const size_t smem = (size_t)((c.max_seqs + 31) / 32) * 4;
  return launch_ex(pages_fork_kernel, dim3(n), dim3(kForkTh), smem, L, c, pages_ws(c, workspace), parents, children, n,
                   L.err);
}

cudaError_t launch_pages_extend(const PageState& c, const PageCopy& pc, const int32_t* n_new, void* workspace,
                                const Launch& L) {
  const PagesWs ws = pages_ws(c, workspace);
  Launch first = L;
  first.pdl = false;
  cudaError_t e =
      launch_ex(pages_extend_kernel, dim3(1), dim3(kPlan), (size_t)c.max_seqs * 12, first, c, ws, n_new, L.err);
  if (e != cudaSuccess) return e;
  return copy_pairs(pc, ws.src, ws.dst, 0, ws.head + 1, c.n_pages, L);
}

cudaError_t launch_pages_trim(const PageState& c, const int32_t* new_lens, const Launch& L) {
  return launch_ex(pages_trim_kernel, dim3(c.max_seqs), dim3(kForkTh), 0, L, c, new_lens, L.err);
}

cudaError_t launch_pages_compact(const PageState& c, const PageCopy& pc, int32_t* n_live, void* workspace,
                                 const Launch& L) {
  const PagesWs ws = pages_ws(c, workspace);
  Launch first = L;
  first.pdl = false;
  cudaError_t e = launch_ex(pages_compact_kernel, dim3(1), dim3(kPlan), 0, first, c, ws, n_live);
  if (e != cudaSuccess) return e;
  e = launch_ex(pages_remap_kernel, dim3(c.max_seqs), dim3(kForkTh), 0, L, c, ws, L.err);
  if (e != cudaSuccess) return e;
  return copy_pairs(pc, ws.src, ws.dst, 0, ws.head + 1, c.n_pages, L);
}

}  // namespace qd
