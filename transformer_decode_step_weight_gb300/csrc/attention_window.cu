// Decode attention of one row per sequence over the keys that a sliding window and a few first
// tokens leave visible, with, where asked for, the weight that each key got added to a sum per
// (sequence, kv head, token) (what eviction goes by, pages_evict.cu).
//
// The visible keys of a sequence are counted through, the first tokens and then the window, so that
// nothing hidden is read and nothing is masked but the end: key i of n lies at token i below the
// first tokens' end and at i + skip above. CTA (split, kv head, sequence), each warp its own blocks
// of 16 keys through a ring of 8 KB stages (16-byte asynchronous copies, any page size); S^T[16 keys
// x 8 heads] = K Q^T and O^T[128 dims x 8 heads] += V^T P^T on mma.sync m16n8k16, the heads of the
// kv head padded to 8. f32 q: q and the softmax weights as three bf16 parts (24 bits); bf16 q: as it
// is, the weights in two parts (2^-16 of each, below the result's own rounding; the second costs a
// quarter more products beside the loads that bound the kernel). Each block's sums are added with
// rounding, since the products' own accumulation truncates. The splits are joined in their order by
// the last of them (ticket).
//
// HBM-bound: 1.08 GB in 174 us (6.2 TB/s) at 64 sequences x 4100 keys (32 q heads, 8 kv heads); one sequence's
// 1028 keys 7.6 us, the launch and a chain of dependent reads (length, pages, keys, partial results).
//
// The weights need every split's statistics first, so the scores (f32, log2 units) are kept in the
// workspace, a sixteenth of K and V's bytes at four q heads a kv head, and a second kernel turns
// them into weights: reading K again would be half of all bytes. A thread owns a key, so no atomics. 16
// sequences x 4400 to 7200 keys: 84 us, of which the second kernel some 8 (13 with one key a thread at a time).
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "mma_sync.cuh"

#include <algorithm>

namespace qd {
namespace {

constexpr int kD = 128;
constexpr int kW = 4;
constexpr int kTh = kW * 32;               // == kD
constexpr int kBlock = 16;                 // keys a warp takes at a time
constexpr int kStages = 2;
constexpr int kStage = 2 * kBlock * kD * 2;   // K and V of a block: 8 KB
constexpr int kHeads = 8;
constexpr int kMaxSplits = 64;
constexpr int kBatch = 32;                 // partial results joined at a time
constexpr int kTickets = 4096;
static_assert(kTickets * 4 == kAttnWindowHeadBytes, "");
constexpr float kLog2e = 1.4426950408889634f;
// A split's result: O [rep][128], m, l [rep], rounded up to whole 16-byte pieces, in which O is
// written and read.
__host__ __device__ constexpr size_t split_floats(int rep) { return (size_t)rep * kD + (2 * rep + 3) / 4 * 4; }

struct Params {
  const void* q;
  long long q_stride;
  const __nv_bfloat16 *k_pages, *v_pages;
  const int32_t *page_table, *seq_lens;
  int Hq, Hkv, rep, page_size, max_pages, n_pages, min_chunk;
  long long cap, window, sinks;
  float scale_log2;
  void* out;
  PageDiv div;
  float* part;      // [B Hkv][splits][split_floats(rep)]
  int* tickets;     // [B Hkv], zero between calls
  float* scores;    // [B Hkv][score_stride]: [key][rep], log2 units; null: not wanted
  long long score_stride;
  float* stats;     // [B Hkv][2][rep]: largest score, 1 / sum
  float* sums;      // [B Hkv][cap]
  int* err;
};

// The keys that the row at token len - 1 sees: n of them, `first` at their own places, the others
// `skip` further on.
struct Shown {
  int n, first, skip;
};
QD_DEV Shown shown(const Params& p, int len) {
  const long long n = min((long long)len, p.window + p.sinks);
  return Shown{(int)n, (int)min(n, p.sinks), (int)(len - n)};
}
QD_DEV int token_of(const Shown& s, int i) { return i < s.first ? i : i + s.skip; }

template <typename T, int QP, int WP, bool SCORES>
__global__ void __launch_bounds__(kTh, 3) attn_window_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float s_m[kBatch][kHeads], s_l[kBatch][kHeads];
  __shared__ float s_max[kHeads], s_scale[kHeads], s_sum[kHeads];
  __shared__ int s_last;
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const int len = p.seq_lens[b];
  if (len < 0 || len > p.cap) {   // the sequence is left as it was
    if (tid == 0) set_error(p.err, QD_DEVERR_POS);
    return;
  }
  const Shown see = shown(p, len);
  int chunk = (see.n + (int)gridDim.x - 1) / (int)gridDim.x;
  chunk = max(p.min_chunk, (chunk + kW * kBlock - 1) / (kW * kBlock) * (kW * kBlock));
  const int n_act = max(1, (see.n + chunk - 1) / chunk);
  if (split >= n_act) return;
  const int lo = split * chunk, hi = min(lo + chunk, see.n);
  const int blocks = (hi - lo + kBlock - 1) / kBlock;
  const int mine = blocks > warp ? (blocks - warp + kW - 1) / kW : 0;   // blocks warp, warp + 4, ...

  // lane k of the first 16 looks key k of a block up one block before its copies go out
  const int32_t* pt = p.page_table + (size_t)b * p.max_pages;
  auto look = [&](int i) {
    const int key = lo + (i * kW + warp) * kBlock + lane;
    int row = -1;
    if (i < mine && lane < kBlock && key < hi) {
      const PagedSlot sl = paged_slot(pt, token_of(see, key), p.page_size, p.div, p.n_pages);
      if (!sl.ok) set_error(p.err, QD_DEVERR_PAGE);
      row = (sl.page * p.Hkv + g) * p.page_size + sl.slot;
    }
    return row;
  };
  int row = look(0);

  // ---- q: heads padded to 8 with zeros, as bf16 parts in the layout of the B operand
  const size_t head0 = (size_t)b * p.Hq + (size_t)g * p.rep, pair = (size_t)b * p.Hkv + g;
  const int qn = lane >> 2, qk = (lane & 3) * 2;
  uint32_t qf[QP][8][2];
  {
    const T* q = (const T*)p.q + (long long)b * p.q_stride + (long long)(g * p.rep + min(qn, p.rep - 1)) * kD + qk;
    const bool ok = qn < p.rep;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (QP == 1) {
          qf[0][ks][e] = ok ? *(const uint32_t*)(q + ks * 16 + 8 * e) : 0u;
        } else {
          const float2 v = *(const float2*)(q + ks * 16 + 8 * e);
          float x = ok ? v.x : 0.f, y = ok ? v.y : 0.f;
#pragma unroll
          for (int part = 0; part < QP; ++part) {
            const uint32_t w = bf2(x, y);
            qf[part][ks][e] = w;
            x -= bf_lo(w);
            y -= bf_hi(w);
          }
        }
      }
  }

  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // heads qk, qk + 1
  float o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  const int rA = (lane & 7) + ((lane >> 3) & 1) * 8, cA = lane >> 4;
  const int rV = (lane & 7) + ((lane >> 4) & 1) * 8, cV = (lane >> 3) & 1;

#pragma unroll 1
  for (int i = 1 - kStages; i < mine; ++i) {
    const int nx = i + kStages - 1;
    if (nx < mine) {
      const int next = look(nx + 1);
      const uint32_t dst = ring + (nx % kStages) * kStage + swz(lane >> 4, lane & 15);
      const __nv_bfloat16 *kp = p.k_pages + (lane & 15) * 8, *vp = p.v_pages + (lane & 15) * 8;
#pragma unroll
      for (int j = 0; j < kBlock; j += 2) {
        const int r = __shfl_sync(0xffffffffu, row, j + (lane >> 4)), n = r < 0 ? 0 : 16;
        const long long off = (long long)max(r, 0) * kD;
        // rows j and j + 1: 256 bytes each, pieces at c ^ (row & 7)
        const uint32_t d = (dst + j * 256) ^ (uint32_t)((j & 6) << 4);
        cp16(d, kp + off, n);
        cp16(d + kBlock * 256, vp + off, n);
      }
      row = next;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (i < 0) continue;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint32_t sK = ring + (i % kStages) * kStage, sV = sK + kBlock * 256;
    float sc[4] = {0.f, 0.f, 0.f, 0.f}, sx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t a[4];
      ldsm_x4(a, sK + swz(rA, 2 * ks + cA));
      mma16816(ks & 1 ? sx : sc, a, qf[0][ks][0], qf[0][ks][1]);
      if constexpr (QP == 3) {
        mma16816(ks & 1 ? sc : sx, a, qf[1][ks][0], qf[1][ks][1]);
        mma16816(ks & 1 ? sx : sc, a, qf[2][ks][0], qf[2][ks][1]);
      }
    }
    const int key0 = lo + (i * kW + warp) * kBlock + (lane >> 2);
    const bool in0 = key0 < hi, in1 = key0 + 8 < hi;
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[e] = (e < 2 ? in0 : in1) ? (sc[e] + sx[e]) * p.scale_log2 : -INFINITY;
    if constexpr (SCORES) {
      float* to = p.scores + pair * p.score_stride + (long long)key0 * p.rep + qk;
      if (p.rep > 1) {
        if (in0 && qk < p.rep) *(float2*)to = make_float2(sc[0], sc[1]);
        if (in1 && qk < p.rep) *(float2*)(to + 8 * p.rep) = make_float2(sc[2], sc[3]);
      } else if (qk == 0) {
        if (in0) to[0] = sc[0];
        if (in1) to[8] = sc[2];
      }
    }
    float x0 = fmaxf(sc[0], sc[2]), x1 = fmaxf(sc[1], sc[3]);
#pragma unroll
    for (int d = 4; d <= 16; d <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
    }
    const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
    const float a0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), a1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
    // nothing but scores of -inf so far: weights 2^(-inf - 0)
    const float r0 = n0 == -INFINITY ? 0.f : n0, r1 = n1 == -INFINITY ? 0.f : n1;
    float w[4] = {in0 ? ex2(sc[0] - r0) : 0.f, in0 ? ex2(sc[1] - r1) : 0.f, in1 ? ex2(sc[2] - r0) : 0.f,
                  in1 ? ex2(sc[3] - r1) : 0.f};
    l0 = l0 * a0 + (w[0] + w[2]);   // this lane's keys; the lanes are added at the end
    l1 = l1 * a1 + (w[1] + w[3]);
    m0 = n0;
    m1 = n1;
    uint32_t pb[WP][2];
#pragma unroll
    for (int part = 0; part < WP; ++part) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t x = bf2(w[2 * e], w[2 * e + 1]);
        pb[part][e] = transpose8(x);
        w[2 * e] -= bf_lo(x);
        w[2 * e + 1] -= bf_hi(x);
      }
    }
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      uint32_t a[4];
      ldsm_x4_t(a, sV + swz(rV, 2 * mt + cV));
      // the smallest parts first
      float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int part = WP - 1; part >= 0; --part) mma16816(x, a, pb[part][0], pb[part][1]);
      o[mt][0] = fmaf(o[mt][0], a0, x[0]);
      o[mt][1] = fmaf(o[mt][1], a1, x[1]);
      o[mt][2] = fmaf(o[mt][2], a0, x[2]);
      o[mt][3] = fmaf(o[mt][3], a1, x[3]);
    }
    __syncwarp();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
  __syncthreads();   // the rings are idle

  // ---- the four warps' results: O [warp][head][dim] in the rings' place
  float* sO = (float*)smem;
  {
    const int d0 = lane >> 2;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sO[(warp * kHeads + qk + (e & 1)) * kD + mt * 16 + d0 + 8 * (e >> 1)] = o[mt][e];
    if (lane < 4) {
      s_m[warp][qk] = m0;
      s_m[warp][qk + 1] = m1;
      s_l[warp][qk] = l0;
      s_l[warp][qk + 1] = l1;
    }
  }
  if (tid < kHeads) {
    s_max[tid] = -INFINITY;
    s_sum[tid] = 0.f;
  }

  // A thread's share of a result: columns 4 (tid % 32) of head tid / 32, and of head 4 + tid / 32
  const int c4 = lane, h0 = warp;
  float4 acc[2];
  acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  // n more partial results, whose statistics are in s_m, s_l; afterwards s_m holds their weights.
  // s_max, s_sum carry the running maximum and sum of each head.
  auto weigh = [&](int n) {
    __syncthreads();
    if (tid < p.rep) {
      float M = s_max[tid];
      for (int k = 0; k < n; ++k) M = fmaxf(M, s_m[k][tid]);
      // what has seen nothing yet: weight 1 for a sum and an O of 0 (or NaN)
      const float old = s_max[tid] == -INFINITY ? 1.f : ex2(s_max[tid] - M);
      float sum = s_sum[tid] * old;   // (a weight of 0 keeps a NaN)
      for (int k = 0; k < n; ++k) {
        const float x = s_m[k][tid] == -INFINITY ? 1.f : ex2(s_m[k][tid] - M);
        s_m[k][tid] = x;
        sum = fmaf(x, s_l[k][tid], sum);
      }
      s_scale[tid] = old;
      s_max[tid] = M;
      s_sum[tid] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (h0 + 4 * u < p.rep) {
        const float f = s_scale[h0 + 4 * u];
        acc[u].x *= f;
        acc[u].y *= f;
        acc[u].z *= f;
        acc[u].w *= f;
      }
  };
  auto add = [&](int u, float x, const float4& v) {   // (a weight of 0 keeps a NaN)
    acc[u].x = fmaf(x, v.x, acc[u].x);
    acc[u].y = fmaf(x, v.y, acc[u].y);
    acc[u].z = fmaf(x, v.z, acc[u].z);
    acc[u].w = fmaf(x, v.w, acc[u].w);
  };
  weigh(kW);
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (h0 + 4 * u < p.rep)
#pragma unroll
      for (int k = 0; k < kW; ++k)
        add(u, s_m[k][h0 + 4 * u], *(const float4*)(sO + (k * kHeads + h0 + 4 * u) * kD + 4 * c4));

  if (n_act > 1) {   // a partial: O [rep][128], m, l [rep]
    const size_t per = split_floats(p.rep);
    float* base = p.part + pair * gridDim.x * per;
    float* my = base + split * per;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (h0 + 4 * u < p.rep) *(float4*)(my + (h0 + 4 * u) * kD + 4 * c4) = acc[u];
    if (tid < p.rep) {
      my[p.rep * kD + tid] = s_max[tid];
      my[p.rep * kD + p.rep + tid] = s_sum[tid];
    }
    __syncthreads();
    if (tid == 0) s_last = atom_add_acq_rel_gpu(p.tickets + pair, 1) == n_act - 1;
    __syncthreads();
    if (!s_last) return;
    if (tid == 0) p.tickets[pair] = 0;
    if (tid < kHeads) {
      s_max[tid] = -INFINITY;
      s_sum[tid] = 0.f;
    }
    acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < n_act; k0 += kBatch) {
      const int n = min(kBatch, n_act - k0);
      __syncthreads();
      for (int e = tid; e < n * kHeads; e += kTh) {
        const int k = e / kHeads, h = e % kHeads;
        if (h < p.rep) {
          const float* m = base + (k0 + k) * per + p.rep * kD;
          s_m[k][h] = __ldcg(m + h);
          s_l[k][h] = __ldcg(m + p.rep + h);
        }
      }
      weigh(n);
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        if (h0 + 4 * u >= p.rep) break;
#pragma unroll 8
        for (int k = 0; k < n; ++k)
          add(u, s_m[k][h0 + 4 * u], __ldcg((const float4*)(base + (k0 + k) * per + (h0 + 4 * u) * kD) + c4));
      }
    }
  }
  if (SCORES && tid < p.rep) {
    p.stats[pair * 2 * p.rep + tid] = s_max[tid];
    p.stats[pair * 2 * p.rep + p.rep + tid] = 1.0f / s_sum[tid];
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (h0 + 4 * u < p.rep) {
      const float inv = len > 0 ? 1.0f / s_sum[h0 + 4 * u] : 0.f;
      const size_t at = (head0 + h0 + 4 * u) * kD + 4 * c4;
      if constexpr (QP == 1)
        *(uint2*)((__nv_bfloat16*)p.out + at) =
            make_uint2(bf2(acc[u].x * inv, acc[u].y * inv), bf2(acc[u].z * inv, acc[u].w * inv));
      else
        *(float4*)((float*)p.out + at) = make_float4(acc[u].x * inv, acc[u].y * inv, acc[u].z * inv, acc[u].w * inv);
    }
}

// The keys' weights, from the scores and the rows' statistics: CTA (part of the keys, kv head, sequence)
constexpr int kAddTh = 256, kAddKeys = 4;
template <int REP>
__global__ void __launch_bounds__(kAddTh) attn_add_weights_kernel(const __grid_constant__ Params p) {
  const int g = blockIdx.y, b = blockIdx.z;
  const size_t pair = (size_t)b * p.Hkv + g;
  const int len = p.seq_lens[b];
  pdl_wait();
  if (len <= 0 || len > p.cap) return;
  const Shown see = shown(p, len);
  float m[REP], inv[REP];
#pragma unroll
  for (int h = 0; h < REP; ++h) {
    m[h] = __ldcg(p.stats + pair * 2 * REP + h);
    inv[h] = __ldcg(p.stats + pair * 2 * REP + REP + h);
  }
  const float* scores = p.scores + pair * p.score_stride;
  float* sums = p.sums + pair * p.cap;
  // kAddKeys keys a thread at a time, all their loads under way
#pragma unroll 1
  for (int i0 = blockIdx.x * kAddTh * kAddKeys + threadIdx.x; i0 < see.n; i0 += gridDim.x * kAddTh * kAddKeys) {
    float s[kAddKeys][REP], old[kAddKeys];
#pragma unroll
    for (int k = 0; k < kAddKeys; ++k) {
      const int i = min(i0 + k * kAddTh, see.n - 1);
      if constexpr (REP >= 4) {
#pragma unroll
        for (int h = 0; h < REP; h += 4) *(float4*)(s[k] + h) = __ldcs((const float4*)(scores + (long long)i * REP + h));
      } else {
#pragma unroll
        for (int h = 0; h < REP; ++h) s[k][h] = __ldcs(scores + (long long)i * REP + h);
      }
      old[k] = sums[token_of(see, i)];
    }
#pragma unroll
    for (int k = 0; k < kAddKeys; ++k) {
      const int i = i0 + k * kAddTh;
      float w = 0.f;
#pragma unroll
      for (int h = 0; h < REP; ++h) w = fmaf(ex2(s[k][h] - m[h]), inv[h], w);
      if (i < see.n) sums[token_of(see, i)] = old[k] + w;
    }
  }
}

// Splits per (sequence, kv head). Long rows: many more CTAs than fit at once, so that the last wave
// is a small share of all. Tickets are taken only where there are splits to join, so by fewer
// than kTickets pairs; their place does not depend on the call.
int splits(int B, int Hkv) {
  const long long pairs = (long long)B * Hkv;
  return (int)std::max(1LL, std::min((long long)kMaxSplits, (kTickets + pairs - 1) / pairs));
}
// Keys per split at least: few pairs take short splits, since then the chain of loads is the time.
// 8 pairs of 1028 keys: 64 8.9 us, 128 7.7, 256 9.6, 512 12.1; 128 pairs of 5700 keys with weights:
// 256 98 us, 512 93, 1024 87, 2048 88; 512 pairs of 4100: 64 to 512 176 us, 1024 174, 2048 184.
// The borders go by pairs alone, not by the visible keys, and lie where these were measured. With 8 kv heads
// (bf16 q; us at 260, 1028 and 4096 visible keys): 1 sequence 7.6, 7.7, 10.9; 4 11, 13, 22; 8 14, 18, 33; 15 15, 23, 53;
// 16 13, 29, 57; 32 15, 35, 94; 64 20, 57, 166. So just above a border a short window is split worst: 16 sequences'
// 1028 keys go to splits of 1024 and 4, and half of the CTAs have next to nothing to do.
int min_chunk(int B, int Hkv) {
  const long long pairs = (long long)B * Hkv;
  return pairs >= 128 ? 1024 : pairs >= 32 ? 256 : 128;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t part_bytes(int B, int Hq, int Hkv) {
  const int n = splits(B, Hkv);
  return n > 1 ? round256((size_t)B * Hkv * n * split_floats(Hq / Hkv) * 4) : 0;
}
size_t stat_bytes(int B, int Hq) { return round256((size_t)B * Hq * 2 * 4); }
long long score_floats(int rep, long long keys) { return (rep * keys + 3) / 4 * 4; }

template <typename T, int QP, int WP>
cudaError_t launch(const Params& p, int B, const Launch& L) {
  const size_t smem = (size_t)kW * kStages * kStage;
  const dim3 grid(splits(B, p.Hkv), p.Hkv, B);
  if (!p.scores) {
    cudaError_t e = allow_smem<attn_window_kernel<T, QP, WP, false>>(smem);
    return e != cudaSuccess ? e : launch_ex(attn_window_kernel<T, QP, WP, false>, grid, dim3(kTh), smem, L, p);
  }
  cudaError_t e = allow_smem<attn_window_kernel<T, QP, WP, true>>(smem);
  return e != cudaSuccess ? e : launch_ex(attn_window_kernel<T, QP, WP, true>, grid, dim3(kTh), smem, L, p);
}

}  // namespace

size_t attn_window_workspace_bytes(int B, int Hq, int Hkv, long long max_keys) {
  const size_t base = kAttnWindowHeadBytes + part_bytes(B, Hq, Hkv);
  return max_keys <= 0 ? base
                       : base + stat_bytes(B, Hq) + (size_t)B * Hkv * score_floats(Hq / Hkv, max_keys) * 4;
}

cudaError_t launch_attn_window(const AttnRowsArgs& a, const Launch& L) {
  Params p = {};
  p.q = a.q; p.q_stride = a.q_stride;
  p.k_pages = (const __nv_bfloat16*)a.k_pages; p.v_pages = (const __nv_bfloat16*)a.v_pages;
  p.page_table = a.page_table; p.seq_lens = a.seq_lens;
  p.Hq = a.Hq; p.Hkv = a.Hkv; p.rep = a.Hq / a.Hkv;
  p.page_size = a.page_size; p.max_pages = a.max_pages; p.n_pages = a.n_pages;
  p.min_chunk = min_chunk(a.n_rows, a.Hkv);
  p.cap = (long long)a.max_pages * a.page_size;
  p.window = a.window; p.sinks = a.n_sinks;
  p.scale_log2 = a.scale * kLog2e;
  p.out = a.out;
  p.div = make_page_div(a.page_size);
  unsigned char* ws = (unsigned char*)a.workspace;
  p.tickets = (int*)ws;
  p.part = (float*)(ws + kAttnWindowHeadBytes);
  if (a.key_weights) {
    p.stats = (float*)(ws + kAttnWindowHeadBytes + part_bytes(a.n_rows, a.Hq, a.Hkv));
    p.scores = (float*)((unsigned char*)p.stats + stat_bytes(a.n_rows, a.Hq));
    p.score_stride = score_floats(p.rep, attn_shown_keys(a));
    p.sums = a.key_weights;
  }
  p.err = L.err;
  Launch first = L;
  first.pdl = false;
  cudaError_t e = a.q_f32 ? launch<float, 3, 3>(p, a.n_rows, first) : launch<__nv_bfloat16, 1, 2>(p, a.n_rows, first);
  if (e != cudaSuccess || !a.key_weights) return e;
  const long long pairs = (long long)a.n_rows * a.Hkv, fill = 8LL * dev_info().sm_count;
  const dim3 grid((unsigned)std::max(1LL, std::min((attn_shown_keys(a) + kAddTh * kAddKeys - 1) / (kAddTh * kAddKeys), (fill + pairs - 1) / pairs)),
                  a.Hkv, a.n_rows);
  Launch second = L;
  second.pdl = true;
  switch (p.rep) {
    case 1: return launch_ex(attn_add_weights_kernel<1>, grid, dim3(kAddTh), 0, second, p);
    case 2: return launch_ex(attn_add_weights_kernel<2>, grid, dim3(kAddTh), 0, second, p);
    case 4: return launch_ex(attn_add_weights_kernel<4>, grid, dim3(kAddTh), 0, second, p);
    default: return launch_ex(attn_add_weights_kernel<8>, grid, dim3(kAddTh), 0, second, p);
  }
}

}  // namespace qd
