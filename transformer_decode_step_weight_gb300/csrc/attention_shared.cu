// Decode attention of sequences that share prefixes. Two launches: attention_rows.cu reads
// each group's shared tokens once for all of its sequences and leaves (O, m, l) of every
// (sequence, q head); the kernel here reads each sequence's own tokens and joins the two.
// It may be launched while the first one runs and waits for it only to join, but a CTA of the first
// takes all of an SM's shared memory and nearly all of its registers, so that it begins early only on
// SMs that have no prefix work left: mostly the two run one after the other. 64 sequences with 4096
// shared tokens (f32, 32 q heads, 8 kv heads): 48 us (the own tokens alone 21, the prefix alone with its
// join 34, either with the launches' 9); 32768 shared tokens (bf16): 66 us, 134 MB of K and V.
//
// Own tokens: CTA (split, kv head, sequence); HBM-bound, so the work only has to keep enough
// bytes in flight, and most of a short sequence's time is the chain of loads before its first
// key (group, page table, keys), which is why three CTAs share an SM and a split has at least
// 512 keys. Each of the four warps walks its own 16-key blocks through a private ring of 8 KB
// stages (16-byte asynchronous copies, any page size, rows past the sequence zero-filled),
// with no CTA barrier in the loop: S^T[16 keys x 8 heads] = K Q^T and O^T[128 dims x 8 heads]
// += V^T P^T on mma.sync m16n8k16, the heads of the kv head padded to 8, P^T transposed in
// registers. f32 q: q and P as three bf16 parts (as in attention_rows.cu); bf16 q: one. The
// prefix's pieces and the splits are joined in a fixed order by the sequence's last CTA
// (ticket): spread over all of them, since one SM reads the 64 KB pieces of a prefix's row tile at
// 16 bytes per cycle (30 us for 12 pieces where attention_rows.cu joined them itself).
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

#include <algorithm>
#include <cstdlib>

namespace qd {
namespace {

constexpr int kD = 128;
constexpr int kW = 4;
constexpr int kTh = kW * 32;               // == kD
constexpr int kBlock = 16;                 // keys a warp takes at a time
constexpr int kStages = 2;
constexpr int kStage = 2 * kBlock * kD * 2;   // K and V of a block: 8 KB
constexpr int kHeads = 8;
constexpr int kMinChunk = 512;             // keys per split, at least
constexpr int kMaxSplits = 64;
constexpr int kBatch = 32;                 // partial results joined at a time
constexpr float kLog2e = 1.4426950408889634f;
// A split's result: O [rep][128], m, l [rep], rounded up to whole 16-byte pieces, in which O is
// written and read.
__host__ __device__ constexpr size_t split_floats(int rep) { return (size_t)rep * kD + (2 * rep + 3) / 4 * 4; }

struct SParams {
  const void* q;
  long long q_stride;
  const __nv_bfloat16 *k_pages, *v_pages;
  const int32_t *page_table, *cu, *seq_lens, *shared_lens;
  int n_groups, B, Hq, Hkv, rep, page_size, max_pages, n_pages;
  long long cap;
  float scale_log2;
  void* out;
  const float *pre_o, *pre_m, *pre_l;
  const AttnFrom* from;
  AttnPieces pieces;
  PageDiv div;
  long long share_min;
  float* part;      // [B Hkv][splits][split_floats(rep)]
  int* tickets;     // [B Hkv], zero between calls
  int* err;
};

QD_DEV void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
QD_DEV void ldsm_x4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
QD_DEV void ldsm_x4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
QD_DEV uint32_t transpose8(uint32_t x) {   // an 8 x 8 tile of 16-bit values over the warp
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
QD_DEV void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
QD_DEV uint32_t bf2(float lo, float hi) { return f2bf_bits(lo) | (f2bf_bits(hi) << 16); }
QD_DEV uint32_t swz(int r, int c) { return (uint32_t)(r * 256 + ((c ^ (r & 7)) << 4)); }

QD_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T, int PARTS>
__global__ void __launch_bounds__(kTh, 3) attn_suffix_kernel(const __grid_constant__ SParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float s_m[kBatch][kHeads], s_l[kBatch][kHeads];
  __shared__ float s_max[kHeads], s_scale[kHeads], s_sum[kHeads];
  __shared__ int s_last;
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- the sequence's group (every warp for itself), and whether the groups make sense
  const int len = p.seq_lens[b];
  int grp = -1, shared = 0;
  long long saved = 0;
  bool bad = false;
  for (int i0 = 0; i0 < p.n_groups; i0 += 32) {
    const int i = i0 + lane;
    bool in = false;
    int n = 0;
    if (i < p.n_groups) {
      const int lo = p.cu[i], hi = p.cu[i + 1];
      n = p.shared_lens[i];
      bad = bad || lo < 0 || hi < lo || hi > p.B;
      if (hi > lo && n > 0 && n <= p.cap) saved += (long long)n * (hi - lo - 1);
      in = lo <= b && b < hi;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, in);
    if (hit) {
      grp = i0 + __ffs(hit) - 1;
      shared = __shfl_sync(0xffffffffu, n, __ffs(hit) - 1);
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  const bool wrong = len < 0 || len > p.cap || shared < 0 || shared > p.cap;
  if (bad || grp < 0 || wrong) {   // the sequence is left as it was
    if (tid == 0 && (bad || grp >= 0)) set_error(p.err, QD_DEVERR_POS);
    pdl_wait();
    return;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) saved += __shfl_xor_sync(0xffffffffu, saved, d);
  const int t0 = saved < p.share_min ? 0 : min(shared, len), own = len - t0;   // as attention_rows.cu decides
  int chunk = (own + (int)gridDim.x - 1) / (int)gridDim.x;
  chunk = max(kMinChunk, (chunk + kW * kBlock - 1) / (kW * kBlock) * (kW * kBlock));
  const int n_act = max(1, (own + chunk - 1) / chunk);
  if (split >= n_act) {
    pdl_wait();
    return;
  }
  const int lo = t0 + split * chunk, hi = min(lo + chunk, len);
  const int blocks = hi > lo ? (hi - lo + kBlock - 1) / kBlock : 0;
  const int mine = blocks > warp ? (blocks - warp + kW - 1) / kW : 0;   // blocks warp, warp + 4, ...

  // ---- q: heads padded to 8 with zeros, as bf16 parts in the layout of the B operand
  const size_t head0 = (size_t)b * p.Hq + (size_t)g * p.rep;
  const int qn = lane >> 2, qk = (lane & 3) * 2;
  uint32_t qf[PARTS][8][2];
  {
    const T* q = (const T*)p.q + (long long)b * p.q_stride + (long long)(g * p.rep + min(qn, p.rep - 1)) * kD + qk;
    const bool ok = qn < p.rep;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (PARTS == 1) {
          qf[0][ks][e] = ok ? *(const uint32_t*)(q + ks * 16 + 8 * e) : 0u;
        } else {
          const float2 v = *(const float2*)(q + ks * 16 + 8 * e);
          float x = ok ? v.x : 0.f, y = ok ? v.y : 0.f;
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            const uint32_t w = bf2(x, y);
            qf[part][ks][e] = w;
            x -= bf_lo(w);
            y -= bf_hi(w);
          }
        }
      }
  }

  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  const int32_t* pt = p.page_table + (size_t)b * p.max_pages;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // heads qk, qk + 1
  float o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  const int rA = (lane & 7) + ((lane >> 3) & 1) * 8, cA = lane >> 4;
  const int rV = (lane & 7) + ((lane >> 4) & 1) * 8, cV = (lane >> 3) & 1;

  // lane k of the first 16 looks key k of a block up one block before its copies go out
  auto look = [&](int i) {
    const int key = lo + (i * kW + warp) * kBlock + lane;
    int row = -1;
    if (i < mine && lane < kBlock && key < hi) {
      const PagedSlot sl = paged_slot(pt, key, p.page_size, p.div, p.n_pages);
      if (!sl.ok) set_error(p.err, QD_DEVERR_PAGE);
      row = (sl.page * p.Hkv + g) * p.page_size + sl.slot;
    }
    return row;
  };
  int row = look(0);
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
      if constexpr (PARTS == 3) {
        mma16816(ks & 1 ? sc : sx, a, qf[1][ks][0], qf[1][ks][1]);
        mma16816(ks & 1 ? sx : sc, a, qf[2][ks][0], qf[2][ks][1]);
      }
    }
    const int key0 = lo + (i * kW + warp) * kBlock + (lane >> 2);
    const bool in0 = key0 < hi, in1 = key0 + 8 < hi;
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[e] = (e < 2 ? in0 : in1) ? (sc[e] + sx[e]) * p.scale_log2 : -INFINITY;
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
    uint32_t pb[PARTS][2];
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
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
      o[mt][0] *= a0;
      o[mt][1] *= a1;
      o[mt][2] *= a0;
      o[mt][3] *= a1;
      uint32_t a[4];
      ldsm_x4_t(a, sV + swz(rV, 2 * mt + cV));
      if constexpr (PARTS == 1) {
        mma16816(o[mt], a, pb[0][0], pb[0][1]);
      } else {
        // each block's sum alone, the smallest parts first, then added with rounding: the
        // products' own accumulation truncates (about 2^-24 of the sum at every step)
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int part = PARTS - 1; part >= 0; --part) mma16816(x, a, pb[part][0], pb[part][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][e] += x[e];
      }
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
  __syncthreads();

  // A thread's share of a result: columns 4 (tid % 32) of head tid / 32, and of head 4 + tid / 32
  const int c4 = lane, h0 = warp;
  float4 acc[2];
  // Adds n partial results, the first `skip` of them without keys: get(k, h, what) gives m, l or O.
  // s_max, s_sum carry the running maximum and sum of each head.
  if (tid < kHeads) {
    s_max[tid] = -INFINITY;
    s_sum[tid] = 0.f;
  }
  acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  // statistics of a batch are in s_m, s_l; afterwards s_m holds weights
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
        if (f != 1.f) {
          acc[u].x *= f;
          acc[u].y *= f;
          acc[u].z *= f;
          acc[u].w *= f;
        }
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

  const size_t pair = (size_t)b * p.Hkv + g;
  const size_t per = split_floats(p.rep);
  float* base = p.part + pair * gridDim.x * per;
  if (n_act > 1) {   // a partial: O [rep][128], m, l [rep]
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
    if (!s_last) {
      pdl_wait();
      return;
    }
    if (tid == 0) p.tickets[pair] = 0;
    if (tid < kHeads) {
      s_max[tid] = -INFINITY;
      s_sum[tid] = 0.f;
    }
    acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  pdl_wait();   // the prefix's results are there

  // ---- joined: the splits (unless this CTA has it all already), then the prefix's pieces
  AttnFrom from = {0, 0, 1, 0};
  if (t0 > 0) {
    const int4 f = __ldcg((const int4*)(p.from + pair));
    // (nothing was written where the first kernel gave up; it has said so)
    from.first = max(0, min(f.x, p.pieces.n - 1));
    from.stride = max(1, min(f.z, p.pieces.n));
    from.pieces = max(0, min(f.y, (p.pieces.n - 1 - from.first) / from.stride + 1));
    from.row = max(0, min(f.w, kPieceRows - p.rep));
  }
  const int n_own = n_act > 1 ? n_act : 0, n_pre = t0 > 0 ? max(from.pieces, 1) : 0;
  // partial k: its O rows (128 floats per head) and statistics
  auto where = [&](int k, const float*& O, const float*& m, const float*& l) {
    if (k < n_own) {
      O = base + k * per;
      m = O + p.rep * kD;
      l = m + p.rep;
    } else if (from.pieces == 0) {
      O = p.pre_o + head0 * kD;
      m = p.pre_m + head0;
      l = p.pre_l + head0;
    } else {
      const int i = k - n_own;
      const float* piece =
          p.pieces.base + ((size_t)(from.first + i * from.stride) * 2 + (i == 0 ? 1 : 0)) * kPieceFloats;
      O = piece + (size_t)from.row * kD;
      m = piece + (size_t)kPieceRows * kD + from.row;
      l = m + kPieceRows;
    }
  };
  const int n_all = n_own + n_pre;
#pragma unroll 1
  for (int k0 = 0; k0 < n_all; k0 += kBatch) {
    const int n = min(kBatch, n_all - k0);
    __syncthreads();
    for (int e = tid; e < n * kHeads; e += kTh) {
      const int k = e / kHeads, h = e % kHeads;
      if (h < p.rep) {
        const float *O, *m, *l;
        where(k0 + k, O, m, l);
        s_m[k][h] = __ldcg(m + h);
        s_l[k][h] = __ldcg(l + h);
      }
    }
    weigh(n);
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
      if (h0 + 4 * u >= p.rep) break;
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const float *O, *m, *l;
        where(k0 + k, O, m, l);
        add(u, s_m[k][h0 + 4 * u], __ldcg((const float4*)(O + (h0 + 4 * u) * kD) + c4));
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (h0 + 4 * u < p.rep) {
      const float sum = s_sum[h0 + 4 * u], inv = len > 0 ? 1.0f / sum : 0.f;
      const size_t at = (head0 + h0 + 4 * u) * kD + 4 * c4;
      if constexpr (PARTS == 1)
        *(uint2*)((__nv_bfloat16*)p.out + at) =
            make_uint2(bf2(acc[u].x * inv, acc[u].y * inv), bf2(acc[u].z * inv, acc[u].w * inv));
      else
        *(float4*)((float*)p.out + at) = make_float4(acc[u].x * inv, acc[u].y * inv, acc[u].z * inv, acc[u].w * inv);
    }
}

// Tickets are taken only where there are splits to join, so by fewer pairs than splits() aims
// at; their place does not depend on the call, which keeps them zero between calls of
// different sizes.
constexpr size_t kTicketBytes = 4096;
static_assert(kAttnSeqTickets + kTicketBytes <= kAttnHeadBytes, "");
int want_ctas() { return std::min(4 * dev_info().sm_count, (int)(kTicketBytes / 4)); }

// Splits per (sequence, kv head): about four CTAs per SM.
int splits(int B, int Hkv) {
  const long long want = want_ctas(), pairs = (long long)B * Hkv;
  return (int)std::max(1LL, std::min((long long)kMaxSplits, (want + pairs - 1) / pairs));
}

// Sharing costs a kernel more and the joining of its pieces, some 12 us; reading everything
// for every sequence costs the repeated bytes at about 5.5 TB/s. Measured crossing between 60 and
// 100 MB: 64 x 256 tokens (8 kv heads) 22.8 us shared, 21.4 not; 16 x 2048 25.2 and 33.4; 4 x
// 8192 34.7 and 36.2 (f32). QD_SHARED_MIN_MB (read per call) sets another limit.
long long share_min(int Hkv) {
  const char* v = getenv("QD_SHARED_MIN_MB");
  return (v ? std::max(0LL, std::min(atoll(v), 1000000000LL)) : 80) * 1000000 / ((long long)Hkv * 2 * kD * 2);
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t pre_bytes(int B, int Hq) { return round256((size_t)B * Hq * (kD + 2) * 4); }
size_t from_bytes(int B, int Hkv) { return round256((size_t)B * Hkv * sizeof(AttnFrom)); }

template <typename T, int PARTS>
cudaError_t launch(const SParams& p, int n_splits, const Launch& L) {
  const size_t smem = (size_t)kW * kStages * kStage;
  cudaError_t e = allow_smem<attn_suffix_kernel<T, PARTS>>(smem);
  if (e != cudaSuccess) return e;
  return launch_ex(attn_suffix_kernel<T, PARTS>, dim3(n_splits, p.Hkv, p.B), dim3(kTh), smem, L, p);
}

}  // namespace

// attention_rows.cu's workspace, whose head has the tickets, then the prefix results (and where they
// are) and the splits.
size_t attn_shared_workspace_bytes(int B, int Hq, int Hkv) {
  return round256(attn_rows_workspace_bytes()) + pre_bytes(B, Hq) +
         from_bytes(B, Hkv) + (size_t)B * Hkv * splits(B, Hkv) * split_floats(Hq / Hkv) * 4;
}

cudaError_t launch_attn_shared(const AttnRowsArgs& args, const Launch& L) {
  AttnRowsArgs a = args;
  a.share_min = share_min(a.Hkv);
  float* pre = (float*)((unsigned char*)a.workspace + round256(attn_rows_workspace_bytes()));
  Launch first = L;
  first.pdl = false;   // whatever ran before in the stream is done before either kernel reads
  AttnFrom* from = (AttnFrom*)((unsigned char*)pre + pre_bytes(a.n_rows, a.Hq));
  SParams p = {};
  cudaError_t e = launch_attn_prefix(a, pre, from, &p.pieces, first);
  if (e != cudaSuccess) return e;
  p.q = a.q; p.q_stride = a.q_stride;
  p.k_pages = (const __nv_bfloat16*)a.k_pages; p.v_pages = (const __nv_bfloat16*)a.v_pages;
  p.page_table = a.page_table; p.cu = a.cu; p.seq_lens = a.seq_lens; p.shared_lens = a.shared_lens;
  p.n_groups = a.n_seg; p.B = a.n_rows; p.Hq = a.Hq; p.Hkv = a.Hkv; p.rep = a.Hq / a.Hkv;
  p.page_size = a.page_size; p.max_pages = a.max_pages; p.n_pages = a.n_pages;
  p.cap = (long long)a.max_pages * a.page_size;
  p.scale_log2 = a.scale * kLog2e;
  p.out = a.out;
  p.pre_o = pre;
  p.pre_m = pre + (size_t)a.n_rows * a.Hq * kD;
  p.pre_l = p.pre_m + (size_t)a.n_rows * a.Hq;
  p.from = from;
  p.div = make_page_div(a.page_size);
  p.share_min = a.share_min;
  p.tickets = (int*)((unsigned char*)a.workspace + kAttnSeqTickets);
  p.part = (float*)((unsigned char*)from + from_bytes(a.n_rows, a.Hkv));
  p.err = L.err;
  const int n = splits(a.n_rows, a.Hkv);
  return a.q_f32 ? launch<float, 3>(p, n, L) : launch<__nv_bfloat16, 1>(p, n, L);
}

}  // namespace qd
