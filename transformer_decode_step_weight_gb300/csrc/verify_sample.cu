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
// sums are kept in pairs of floats (48 bits, by exact two-sums; binary64 adds run at
// 1/64 of the binary32 rate here): a border is misplaced by about 2^-45 of the total.
//
// One launch: CTA (chunk c, sequence b) finds m (k gathered values, the same in every
// CTA), sums its chunk of the one or two rows that matter, and the sequence's last CTA
// (ticket) finds the chunk that holds the border, reads that chunk again and writes the
// state. Bytes: one or two vocabulary rows per sequence, whatever k.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

#include <algorithm>

namespace qd {
namespace {

constexpr int kTh = 256;

// an unevaluated sum hi + lo
struct Pair {
  float hi, lo;
};
QD_DEV Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
// a + b for a running sum a and one value b (three roundings of the low parts: 2^-46 of
// the sum)
QD_DEV Pair add_small(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, __fadd_rn(__fadd_rn(s.lo, b.lo), a.lo));
}
QD_DEV Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
  const Pair v = two_sum(s.hi, __fadd_rn(s.lo, t.hi));
  return two_sum(v.hi, __fadd_rn(v.lo, t.lo));
}
QD_DEV double value(Pair a) { return (double)a.hi + (double)a.lo; }
QD_DEV Pair shfl_up(Pair a, int o) {
  return Pair{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}

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

// r of one token, exactly (hi is p - q rounded, lo what the rounding left; hi > 0 just
// where p > q)
QD_DEV Pair mass(float p, float q) {
  const Pair r = two_sum(p, -q);
  return r.hi > 0.f && r.hi < INFINITY ? r : Pair{0.f, 0.f};
}

// the 4 N values of r from token j on (j a multiple of 4), 0 past the vocabulary; q null:
// r = p
template <int N>
QD_DEV void load_mass(const float* p, const float* q, int j, int V, int vec, Pair* r) {
  float a[4 * N], b[4 * N];
  if (vec && j + 4 * N <= V) {
#pragma unroll
    for (int i = 0; i < N; ++i) *(float4*)(a + 4 * i) = *(const float4*)(p + j + 4 * i);
    if (q)
#pragma unroll
      for (int i = 0; i < N; ++i) *(float4*)(b + 4 * i) = *(const float4*)(q + j + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) a[i] = j + i < V ? p[j + i] : 0.f;
    if (q)
#pragma unroll
      for (int i = 0; i < 4 * N; ++i) b[i] = j + i < V ? q[j + i] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) r[i] = mass(a[i], q ? b[i] : 0.f);
}

// inclusive sum over the CTA's threads in thread order, in pairs; total: the whole sum
QD_DEV Pair block_scan(Pair v, Pair* warp_sums, Pair& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair x = shfl_up(v, o);
    if (lane >= o) v = add(x, v);
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  Pair before{0.f, 0.f}, all{0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kTh / 32; ++w) {
    if (w == warp) before = all;
    all = add(all, warp_sums[w]);
  }
  total = all;
  return add(before, v);
}

// N: float4 loads per thread, chunk = kTh * 4 N tokens
template <int N>
__global__ void __launch_bounds__(kTh) verify_sample_kernel(const VsParams p) {
  __shared__ int s_m, s_n, s_last, s_tok, s_chunk;
  __shared__ Pair warp_sums[kTh / 32];
  __shared__ double s_before, s_total;
  const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int kd = p.k - 1;
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
  // ---- the chunk's sum: thread t takes the float4 at t, t + kTh, ... of the chunk
  {
    Pair s{0.f, 0.f};
    Pair r[4 * N];
    const int j0 = c * p.chunk;
#pragma unroll
    for (int i = 0; i < N; ++i) load_mass<1>(pr, qr, j0 + (i * kTh + tid) * 4, p.V, p.vec, r + 4 * i);
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) s = add_small(s, r[i]);
    Pair total;
    block_scan(s, warp_sums, total);
    if (tid == 0) {
      p.part[(size_t)b * gridDim.x + c] = value(total);
      s_last = atom_add_acq_rel_gpu(p.cnt + b, 1) == (int)gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  // ---- the sequence's last CTA: the chunk that holds the border
  if (tid == 0) s_tok = -1;
  const float ul = p.u[(size_t)b * p.k + p.k - 1];
  for (int attempt = 0; attempt < 2; ++attempt) {
    if (attempt == 1) {   // nothing left of p - q: draw from p, whose chunk sums nobody has made yet
      if (qr == nullptr) break;
      qr = nullptr;
      for (int ch = 0; ch < (int)gridDim.x; ++ch) {
        Pair s{0.f, 0.f}, total;
        Pair r[4 * N];
#pragma unroll
        for (int i = 0; i < N; ++i) load_mass<1>(pr, qr, ch * p.chunk + (i * kTh + tid) * 4, p.V, p.vec, r + 4 * i);
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) s = add_small(s, r[i]);
        block_scan(s, warp_sums, total);
        if (tid == 0) p.part[(size_t)b * gridDim.x + ch] = value(total);
      }
      __threadfence();
      __syncthreads();
    }
    if (tid < 32) {
      const double* part = p.part + (size_t)b * gridDim.x;
      const int nc = (int)gridDim.x;
      double total = 0.0;
      for (int i0 = 0; i0 < nc; i0 += 32) {
        double v = i0 + lane < nc ? __ldcg(part + i0 + lane) : 0.0;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        total += v;
      }
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
        s_before = hit >= 0 ? b_hit : b_some;
        s_total = border;
      }
    }
    __syncthreads();
    if (s_chunk >= 0) break;
  }
  if (s_chunk >= 0) {
    // ---- its tokens in order: thread t takes 4 N consecutive ones
    const int j = s_chunk * p.chunk + tid * 4 * N;
    Pair r[4 * N];
    load_mass<N>(pr, qr, j, p.V, p.vec, r);
    Pair s{0.f, 0.f}, total;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) s = add_small(s, r[i]);
    const Pair incl = block_scan(s, warp_sums, total);
    // the border as a pair, relative to the chunk's start
    const double want = s_total - s_before;
    const Pair lim{(float)want, (float)(want - (double)(float)want)};
    const Pair neg{-lim.hi, -lim.lo};
    auto over = [&](Pair a) {
      const Pair d = add(a, neg);
      return d.hi > 0.f || (d.hi == 0.f && d.lo > 0.f);
    };
    const bool mine = over(incl);
    const unsigned vote = __ballot_sync(0xffffffffu, mine);
    __shared__ int s_first[kTh / 32], s_some[kTh / 32];
    // running sums never fall, so the first thread past the border holds the token; where
    // rounding leaves none, the chunk's last token with any mass
    int last = -1;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i)
      if (r[i].hi > 0.f) last = j + i;
#pragma unroll
    for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
    if (lane == 0) {
      s_first[tid >> 5] = vote ? (tid & ~31) + __ffs(vote) - 1 : kTh;
      s_some[tid >> 5] = last;
    }
    __syncthreads();
    int first = kTh, some = -1;
#pragma unroll
    for (int w = 0; w < kTh / 32; ++w) {
      first = min(first, s_first[w]);
      some = max(some, s_some[w]);
    }
    if (first == kTh) {
      if (tid == 0) s_tok = some;
    } else {
      // the sum before thread `first`, from its left neighbour
      __shared__ Pair s_prev[kTh];
      s_prev[tid] = incl;
      __syncthreads();
      if (tid == first) {
        Pair a = tid ? s_prev[tid - 1] : Pair{0.f, 0.f};
        int t = -1;
        for (int i = 0; i < 4 * N; ++i) {
          a = add_small(a, r[i]);
          if (r[i].hi > 0.f) {
            t = j + i;
            if (over(a)) break;
          }
        }
        s_tok = t >= 0 ? t : some;
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    int t = s_tok;
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
  // chunks of 4096 tokens; of 1024 where those would leave SMs without work
  const bool small = (long long)a.B * ceil_div(a.V, kTh * 16) < dev_info().sm_count;
  p.chunk = kTh * (small ? 4 : 16);
  const dim3 grid(ceil_div(a.V, p.chunk), a.B);
  return small ? launch_ex(verify_sample_kernel<1>, grid, dim3(kTh), 0, L, p)
               : launch_ex(verify_sample_kernel<4>, grid, dim3(kTh), 0, L, p);
}

}  // namespace qd
