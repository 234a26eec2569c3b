// Verification of drafted tokens by their probabilities (speculative sampling).
//
// Per sequence, with drafts d_0 .. d_{n-1}, the draft model's distributions q_i they were
// drawn from, the target's p_0 .. p_n and uniform random numbers u: draft i is accepted
// while u_i q_i(d_i) < p_i(d_i). At the first rejection m the next token is drawn from
// r = max(p_m - q_m, 0) (from p_m where that is zero everywhere), after n accepted drafts
// from r = p_n: the least token j with sum_{i <= j} r_i > u_last sum_i r_i. Entries of r
// that are not finite count as 0.
//
// Which token is drawn hangs on where a sum over the vocabulary crosses a border, so the
// sums are kept in pairs of floats (binary64 adds run at 1/64 of the binary32 rate here). A thread
// adds up groups of at most 32 tokens, each in a pair of its own whose low part is not renormalised
// (off by at most 496 2^-49 of the group), and where it has more of them the groups in three floats;
// the threads' sums go through 14 additions of pairs (1.5 2^-48 each), the chunks' are added in
// binary64. So a border is misplaced by less than 2^-39 of the total whatever the vocabulary and the
// batch; in models of the sums by 2^-43 at most, 2^-45 where the tokens are not all alike.
//
// One launch: CTA (chunk c, sequence b) finds m (k gathered values, the same in every
// CTA), sums its chunk of the one or two rows that matter, and the sequence's last CTA
// (ticket) finds the chunk that holds the border, reads that chunk again and writes the
// state. Bytes: one or two vocabulary rows per sequence, whatever k. Chunks are as long as eight CTAs
// per SM need; five of them (48 registers a thread) are resident at a time. 64 sequences with 5 rows of
// 151936: 27 us for 78 MB (3, 4, 6, 8, 12, 16 CTAs per SM: 36.5, 36, 30, 27, 27, 28 us; one or two groups
// of four tokens per thread under way instead of four: 28 to 31), bound by waits: a
// warp spends 4.2 cycles per instruction on memory and 4.1 at barriers (HBM 23 % busy).
// One sequence: 10 to 11 us, a chain of dependent reads (drafts, their probabilities, the rows, the chunk
// sums, the chunk again, the state).
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

#include <algorithm>

namespace qd {
namespace {

constexpr int kTh = 256;
constexpr int kGroup = 32;   // tokens whose sum one pair of floats holds

// an unevaluated sum hi + lo
struct Pair {
  float hi, lo;
};
QD_DEV Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
QD_DEV Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
QD_DEV double value(Pair a) { return (double)a.hi + (double)a.lo; }

struct VsParams {
  const float *target, *draft_p, *u;
  long long t_stride, d_stride;   // elements from one row to the next
  const int32_t *draft, *n_draft;
  int B, k, V, chunk, vec;        // vec: both matrices' rows start on 16-byte boundaries
  int32_t *tok, *pos, *step, *out;
  int max_steps;
  int32_t* n_accept;
  double* part;                   // [B, chunks]
  int* cnt;                       // [B] tickets
  int* err;
};

// s + r of one token. r = p - q exactly: rounded, and what the rounding left (p > q >= 0 where
// it counts). The low part gathers what the high part loses and is not renormalised.
QD_DEV void add_mass(Pair& s, float p, float q) {
  const float r = __fsub_rn(p, q);
  const bool some = r > 0.f && r < INFINITY;
  const float e = __fsub_rn(__fsub_rn(p, r), q);
  const Pair t = two_sum(s.hi, some ? r : 0.f);
  s.hi = t.hi;
  s.lo = __fadd_rn(s.lo, __fadd_rn(t.lo, some ? e : 0.f));
}

// A thread's groups of tokens but for the last.
struct Groups {
  float t0 = 0.f, t1 = 0.f, t2 = 0.f;
  QD_DEV void take(Pair& g) {
    const Pair a = two_sum(t0, g.hi), b = two_sum(t1, a.lo), c = two_sum(b.hi, g.lo);
    t0 = a.hi;
    t1 = c.hi;
    t2 = __fadd_rn(t2, __fadd_rn(b.lo, c.lo));
    g = Pair{0.f, 0.f};
  }
  QD_DEV Pair with(Pair g) {   // and the last
    take(g);
    const Pair s = two_sum(t0, t1);
    return two_sum(s.hi, __fadd_rn(s.lo, t2));
  }
};

// four tokens from j on; 0 past `end`
QD_DEV float4 load4(const float* p, int j, int end, int vec) {
  if (vec && j + 4 <= end) return *(const float4*)(p + j);
  return make_float4(j < end ? p[j] : 0.f, j + 1 < end ? p[j + 1] : 0.f, j + 2 < end ? p[j + 2] : 0.f,
                     j + 3 < end ? p[j + 3] : 0.f);
}

// inclusive sum over the CTA's threads in thread order; total: the whole sum
__device__ __noinline__ Pair block_scan(Pair v, Pair* warp_sums, Pair* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const Pair x = {__shfl_up_sync(0xffffffffu, v.hi, o), __shfl_up_sync(0xffffffffu, v.lo, o)};
    if (lane >= o) v = add(x, v);
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  Pair before{0.f, 0.f}, all{0.f, 0.f};
#pragma unroll 1
  for (int w = 0; w < kTh / 32; ++w) {
    if (w == warp) before = all;
    all = add(all, warp_sums[w]);
  }
  *total = all;
  return add(before, v);
}

// The CTA's sum of r over the tokens [j0, end): thread t takes every kTh-th four of them.
// kMany: more than kGroup for a thread.
template <bool kMany>
QD_DEV double chunk_sum(const float* p, const float* q, int j0, int end, int vec, Pair* warp_sums) {
  Pair s{0.f, 0.f}, total;
  Groups before;
  constexpr int kU = 4;
  for (int j = j0 + threadIdx.x * 4; j < end; j += kTh * 4 * kU) {
    float4 a[kU], b[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      a[u] = load4(p, j + u * kTh * 4, end, vec);
      b[u] = q ? load4(q, j + u * kTh * 4, end, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      add_mass(s, a[u].x, b[u].x);
      add_mass(s, a[u].y, b[u].y);
      add_mass(s, a[u].z, b[u].z);
      add_mass(s, a[u].w, b[u].w);
    }
    if (kMany) before.take(s);
  }
  if (kMany) s = before.with(s);
  block_scan(s, warp_sums, &total);
  return value(total);
}

template <bool kMany>
__global__ void __launch_bounds__(kTh) verify_sample_kernel(const __grid_constant__ VsParams p) {
  __shared__ int s_m, s_n, s_last, s_tok, s_chunk, s_some, s_first;
  __shared__ Pair warp_sums[kTh / 32], s_prev[kTh];
  __shared__ double s_want;
  const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int kd = p.k - 1, nc = (int)gridDim.x;
  const float ul = p.u[(size_t)b * p.k + kd];
  if (tid < 32) {
    int n = p.n_draft ? p.n_draft[b] : kd;
    if (n < 0 || n > kd) {
      if (lane == 0 && c == 0) set_error(p.err, QD_DEVERR_POS);
      n = max(0, min(n, kd));
    }
    int m = 0;
    for (int i0 = 0; i0 < n && m == i0; i0 += 32) {   // 32 drafts at a time, as long as all are accepted
      const int i = i0 + lane;
      bool ok = false;
      if (i < n) {
        const int d = p.draft[(size_t)b * kd + i];
        if (d >= 0 && d < p.V) {
          const float pd = p.target[((size_t)b * p.k + i) * p.t_stride + d];
          const float qd = p.draft_p[((size_t)b * kd + i) * p.d_stride + d];
          ok = (double)p.u[(size_t)b * p.k + i] * (double)qd < (double)pd;   // the product is exact
        }
      }
      const unsigned no = ~__ballot_sync(0xffffffffu, ok);
      m += no ? __ffs(no) - 1 : 32;
    }
    if (lane == 0) {
      s_m = m;
      s_n = n;
    }
  }
  __syncthreads();
  const int m = s_m;
  const float* pr = p.target + ((size_t)b * p.k + m) * p.t_stride;
  const float* qr = m < s_n ? p.draft_p + ((size_t)b * kd + m) * p.d_stride : nullptr;
  double* part = p.part + (size_t)b * nc;
  {
    const double sum = chunk_sum<kMany>(pr, qr, c * p.chunk, min((c + 1) * p.chunk, p.V), p.vec, warp_sums);
    if (tid == 0) {
      part[c] = sum;
      s_last = atom_add_acq_rel_gpu(p.cnt + b, 1) == nc - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;

  // ---- the sequence's last CTA: the chunk that holds the border
#pragma unroll 1
  for (int attempt = 0;; ++attempt) {
    if (tid < 32) {
      double total = 0.0;
#pragma unroll 4
      for (int i = lane; i < nc; i += 32) total += __ldcg(part + i);
#pragma unroll
      for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      // the first chunk whose running sum passes the border; the last one with any mass
      // where rounding leaves none
      const double border = (double)ul * total;
      double before = 0.0, b_hit = 0.0, b_some = 0.0;
      int hit = -1, some = -1;
      for (int i0 = 0; i0 < nc && hit < 0; i0 += 32) {
        const double own = i0 + lane < nc ? __ldcg(part + i0 + lane) : 0.0;
        double v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double x = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += x;
        }
        const double excl = __shfl_up_sync(0xffffffffu, v, 1);
        const double start = before + (lane ? excl : 0.0);
        const unsigned over = __ballot_sync(0xffffffffu, own > 0.0 && before + v > border);
        const unsigned any = __ballot_sync(0xffffffffu, own > 0.0);
        if (any) {
          some = i0 + 31 - __clz(any);
          b_some = __shfl_sync(0xffffffffu, start, 31 - __clz(any));
        }
        if (over) {
          hit = i0 + __ffs(over) - 1;
          b_hit = __shfl_sync(0xffffffffu, start, __ffs(over) - 1);
        }
        before += __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) {
        s_chunk = hit >= 0 ? hit : some;
        // (not below 0: the scan adds in another order for each chunk, so the sum before one
        // may pass the border by a rounding without the chunk before it having done so)
        s_want = fmax(0.0, border - (hit >= 0 ? b_hit : b_some));
      }
    }
    __syncthreads();
    if (s_chunk >= 0 || qr == nullptr || attempt) break;
    // nothing left of p - q: draw from p, whose chunk sums nobody has made yet
    qr = nullptr;
#pragma unroll 1
    for (int ch = 0; ch < nc; ++ch) {
      const double sum = chunk_sum<kMany>(pr, nullptr, ch * p.chunk, min((ch + 1) * p.chunk, p.V), p.vec, warp_sums);
      if (tid == 0) part[ch] = sum;
    }
    __threadfence();
    __syncthreads();
  }
  if (tid == 0) {
    s_tok = s_some = -1;
    s_first = kTh;
  }
  __syncthreads();
  if (s_chunk >= 0) {
    // ---- its tokens in order: thread t takes chunk / kTh consecutive ones. The first thread with any
    // mass whose running sum passes the border holds the token (of all threads, the first: the sums
    // are added in another order for each, so in their last bits they may fall from one to the next);
    // where rounding leaves none, the chunk's last token with any mass
    const int each = p.chunk / kTh, j0 = s_chunk * p.chunk + tid * each;
    const int end = min(p.V, j0 + each);
    Pair s{0.f, 0.f}, total;
    Groups earlier;
    int last = -1;
#pragma unroll 4
    for (int j = j0; j < end; j += 4) {
      const float4 x = load4(pr, j, end, p.vec), y = qr ? load4(qr, j, end, p.vec) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        add_mass(s, xs[i], ys[i]);
        const float r = xs[i] - ys[i];
        if (r > 0.f && r < INFINITY) last = j + i;
      }
      if (kMany && ((j - j0) & 12) == 12) earlier.take(s);
    }
    if (kMany) s = earlier.with(s);
    const Pair incl = block_scan(s, warp_sums, &total);
    s_prev[tid] = incl;
    const double want = s_want;
    const Pair neg{-(float)want, -(float)(want - (double)(float)want)};
    auto over = [&](Pair a) {
      const Pair d = add(a, neg);
      return d.hi > 0.f || (d.hi == 0.f && d.lo > 0.f);
    };
    if (last >= 0) atomicMax(&s_some, last);
    const unsigned past = __ballot_sync(0xffffffffu, last >= 0 && over(incl));
    if (lane == 0 && past) atomicMin(&s_first, (tid & ~31) + __ffs(past) - 1);
    __syncthreads();
    if (tid == s_first) {
      // what the tokens before it leave to the border (below 0), and the group at hand
      Pair base = tid ? add(s_prev[tid - 1], neg) : neg, a{0.f, 0.f};
#pragma unroll 4
      for (int j = j0; j < end; ++j) {
        const float x = pr[j], y = qr ? qr[j] : 0.f, r = x - y;
        add_mass(a, x, y);
        if (r > 0.f && r < INFINITY) {
          s_tok = j;
          const Pair d = add(base, a);
          if (d.hi > 0.f || (d.hi == 0.f && d.lo > 0.f)) break;
        }
        if (kMany && ((j - j0) & (kGroup - 1)) == kGroup - 1) {
          base = add(base, a);
          a = Pair{0.f, 0.f};
        }
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    int t = s_tok >= 0 ? s_tok : s_some;
    if (t < 0) {   // a row without any positive finite entry
      set_error(p.err, QD_DEVERR_NAN);
      t = 0;
    }
    const int st = p.step[b];
    for (int i = 0; i <= m; ++i) {
      const long long at = (long long)st + i;
      if (at >= 0 && at < p.max_steps) p.out[(size_t)b * p.max_steps + at] = i < m ? p.draft[(size_t)b * kd + i] : t;
      else set_error(p.err, QD_DEVERR_STEPS);
    }
    p.tok[b] = t;
    p.pos[b] += m + 1;
    p.step[b] = st + m + 1;
    p.n_accept[b] = m;
    p.cnt[b] = 0;
  }
}

constexpr int kMaxChunks = 1024;   // chunk sums per sequence in the workspace
constexpr size_t kTicketBytes = 65536 * 4;

}  // namespace

// Tickets first, with room for every batch (their place must not depend on the call: they are
// zero between calls of different sizes), then the chunk sums.
size_t verify_sample_workspace_bytes(int B) { return kTicketBytes + (size_t)B * kMaxChunks * 8; }
int verify_sample_max_vocab() { return kMaxChunks * kTh * 16; }

cudaError_t launch_verify_sample(const VerifySampleArgs& a, const Launch& L) {
  VsParams p = {};
  p.target = a.target; p.draft_p = a.draft_probs; p.u = a.u;
  p.t_stride = a.t_stride; p.d_stride = a.d_stride;
  p.draft = a.draft; p.n_draft = a.n_draft;
  p.B = a.B; p.k = a.k; p.V = a.V;
  p.tok = a.tok; p.pos = a.pos; p.step = a.step; p.out = a.out_tokens; p.max_steps = a.max_steps;
  p.n_accept = a.n_accept;
  p.cnt = (int*)a.workspace;
  p.part = (double*)((unsigned char*)a.workspace + kTicketBytes);
  p.err = L.err;
  p.vec = ((uintptr_t)a.target & 15u) == 0 && a.t_stride % 4 == 0 &&
          (a.k == 1 || (((uintptr_t)a.draft_probs & 15u) == 0 && a.d_stride % 4 == 0));
  // about eight CTAs per SM, chunks a multiple of 1024 tokens
  const int chunks = (int)std::max(1LL, std::min((long long)kMaxChunks, 8LL * dev_info().sm_count / a.B));
  p.chunk = ceil_div(ceil_div(a.V, chunks), kTh * 4) * kTh * 4;
  return launch_ex(p.chunk > kTh * kGroup ? verify_sample_kernel<true> : verify_sample_kernel<false>,
                   dim3(ceil_div(a.V, p.chunk), a.B), dim3(kTh), 0, L, p);
}

}  // namespace qd
