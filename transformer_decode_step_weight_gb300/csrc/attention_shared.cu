// Decode attention of sequences that share prefixes. Two launches: attention_rows.cu reads
// each group's shared tokens once for all of its sequences and leaves (O, m, l) of every
// (sequence, q head); the kernel here reads each sequence's own tokens and joins the two.
// It starts while the first one runs and waits for it only to join.
//
// Own tokens: CTA (split, kv head, sequence); HBM-bound, so the split only has to keep
// enough bytes in flight. Each of the four warps walks its own 16-key blocks through a
// private ring of 8 KB stages (16-byte asynchronous copies, any page size, rows past the
// sequence zero-filled), with no CTA barrier in the loop: S^T[16 keys x 8 heads] = K Q^T
// and O^T[128 dims x 8 heads] += V^T P^T on mma.sync m16n8k16, the heads of the kv head
// padded to 8, P^T transposed in registers. f32 q: q and P as three bf16 parts (as in
// attention_rows.cu); bf16 q: one. Warps, then splits (ticket), then the prefix are joined
// in a fixed order.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

#include <algorithm>

namespace qd {
namespace {

constexpr int kD = 128;
constexpr int kW = 4;
constexpr int kTh = kW * 32;               // == kD
constexpr int kBlock = 16;                 // keys a warp takes at a time
constexpr int kStages = 3;
constexpr int kStage = 2 * kBlock * kD * 2;   // K and V of a block: 8 KB
constexpr int kHeads = 8;
constexpr int kMinChunk = 256;             // keys per split, at least
constexpr int kMaxSplits = 64;
constexpr float kLog2e = 1.4426950408889634f;

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
  float* part;      // [B Hkv][splits][rep][130]
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

template <typename T, int PARTS>
__global__ void __launch_bounds__(kTh) attn_suffix_kernel(const SParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sM[kW][kHeads], sL[kW][kHeads], sQ[kHeads][kD];
  __shared__ float s_w[kMaxSplits + 1][kHeads], s_tot[kHeads];
  __shared__ int s_last;
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- the sequence's group (every warp for itself), and whether the groups make sense
  int grp = -1;
  bool bad = false;
  for (int i0 = 0; i0 < p.n_groups; i0 += 32) {
    const int i = i0 + lane;
    bool in = false;
    if (i < p.n_groups) {
      const int lo = p.cu[i], hi = p.cu[i + 1];
      bad = bad || lo < 0 || hi < lo || hi > p.B;
      in = lo <= b && b < hi;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, in);
    if (hit) grp = i0 + __ffs(hit) - 1;
  }
  bad = __any_sync(0xffffffffu, bad);
  const int len = p.seq_lens[b], shared = !bad && grp >= 0 ? p.shared_lens[grp] : 0;
  const bool wrong = len < 0 || len > p.cap || shared < 0 || shared > p.cap;
  if (bad || grp < 0 || wrong) {   // the sequence is left as it was
    if (tid == 0 && (bad || grp >= 0)) set_error(p.err, QD_DEVERR_POS);
    pdl_wait();
    return;
  }
  const int t0 = min(shared, len), own = len - t0;
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

  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  const int32_t* pt = p.page_table + (size_t)b * p.max_pages;
  auto load = [&](int i) {
    const int key0 = lo + (i * kW + warp) * kBlock;
    long long off = -1;
    if (lane < kBlock && key0 + lane < hi) {
      const PagedSlot sl = paged_slot(pt, key0 + lane, p.page_size, p.n_pages);
      if (!sl.ok) set_error(p.err, QD_DEVERR_PAGE);
      off = (((long long)sl.page * p.Hkv + g) * p.page_size + sl.slot) * kD;
    }
    const uint32_t dst = ring + (i % kStages) * kStage;
#pragma unroll
    for (int j = 0; j < kBlock; j += 2) {
      const int r = j + (lane >> 4), c = lane & 15;
      const long long o = __shfl_sync(0xffffffffu, off, r);
      cp16(dst + swz(r, c), p.k_pages + (o < 0 ? 0 : o) + c * 8, o < 0 ? 0 : 16);
      cp16(dst + kBlock * 256 + swz(r, c), p.v_pages + (o < 0 ? 0 : o) + c * 8, o < 0 ? 0 : 16);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < mine) load(i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // ---- q: heads padded to 8 with zeros, as bf16 parts in the layout of the B operand
  const size_t head0 = (size_t)b * p.Hq + (size_t)g * p.rep;
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    float x = 0.f;
    if (h < p.rep) {
      const T v = ((const T*)p.q)[(long long)b * p.q_stride + (long long)(g * p.rep + h) * kD + tid];
      if constexpr (PARTS == 1) x = __bfloat162float(v); else x = v;
    }
    sQ[h][tid] = x;
  }
  __syncthreads();
  const int qn = lane >> 2, qk = (lane & 3) * 2;
  uint32_t qf[PARTS][8][2];
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = sQ[qn][ks * 16 + qk + 8 * e], y = sQ[qn][ks * 16 + qk + 8 * e + 1];
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        const uint32_t w = bf2(x, y);
        qf[part][ks][e] = w;
        x -= bf_lo(w);
        y -= bf_hi(w);
      }
    }

  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // heads qk, qk + 1
  float o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  const int rA = (lane & 7) + ((lane >> 3) & 1) * 8, cA = lane >> 4;
  const int rV = (lane & 7) + ((lane >> 4) & 1) * 8, cV = (lane >> 3) & 1;

  for (int i = 0; i < mine; ++i) {
    if (i + kStages - 1 < mine) load(i + kStages - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
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
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[e] = key0 + (e >> 1) * 8 < hi ? (sc[e] + sx[e]) * p.scale_log2 : -INFINITY;
    float x0 = fmaxf(sc[0], sc[2]), x1 = fmaxf(sc[1], sc[3]);
#pragma unroll
    for (int d = 4; d <= 16; d <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
    }
    const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
    const float a0 = n0 == -INFINITY ? 1.f : exp2f(m0 - n0), a1 = n1 == -INFINITY ? 1.f : exp2f(m1 - n1);
    const bool in0 = key0 < hi, in1 = key0 + 8 < hi;
    float w[4] = {in0 ? exp2f(sc[0] - n0) : 0.f, in0 ? exp2f(sc[1] - n1) : 0.f, in1 ? exp2f(sc[2] - n0) : 0.f,
                  in1 ? exp2f(sc[3] - n1) : 0.f};
    l0 = l0 * a0 + (w[0] + w[2]);   // this lane's keys; the lanes are added at the end
    l1 = l1 * a1 + (w[1] + w[3]);
    m0 = n0;
    m1 = n1;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      o[mt][0] *= a0;
      o[mt][1] *= a1;
      o[mt][2] *= a0;
      o[mt][3] *= a1;
    }
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

  // ---- the four warps
  float* sO = (float*)smem;   // [warp][head][dim]
  {
    const int d0 = lane >> 2;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      sO[(warp * kHeads + qk) * kD + mt * 16 + d0] = o[mt][0];
      sO[(warp * kHeads + qk + 1) * kD + mt * 16 + d0] = o[mt][1];
      sO[(warp * kHeads + qk) * kD + mt * 16 + d0 + 8] = o[mt][2];
      sO[(warp * kHeads + qk + 1) * kD + mt * 16 + d0 + 8] = o[mt][3];
    }
    if (lane < 4) {
      sM[warp][qk] = m0;
      sM[warp][qk + 1] = m1;
      sL[warp][qk] = l0;
      sL[warp][qk + 1] = l1;
    }
  }
  __syncthreads();
  float oo[kHeads], MM[kHeads], LL[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    float M = -INFINITY, Lx = 0.f, O = 0.f;
#pragma unroll
    for (int v = 0; v < kW; ++v) M = fmaxf(M, sM[v][h]);
#pragma unroll
    for (int v = 0; v < kW; ++v) {
      if (blocks <= v) continue;   // a warp without keys
      const float c = sM[v][h] == -INFINITY && M != -INFINITY ? 0.f : exp2f(sM[v][h] - M);
      Lx = fmaf(c, sL[v][h], Lx);
      O = fmaf(c, sO[(v * kHeads + h) * kD + tid], O);
    }
    oo[h] = O;
    MM[h] = M;
    LL[h] = Lx;
  }
  auto store = [&](int h, float O, float M, float Lx) {   // with the prefix, if there is one
    if (t0 > 0) {
      const float pm = __ldcg(p.pre_m + head0 + h), pl = __ldcg(p.pre_l + head0 + h);
      const float po = __ldcg(p.pre_o + (head0 + h) * kD + tid);
      const float N = fmaxf(M, pm);
      const float c = M == -INFINITY ? 0.f : exp2f(M - N), d = pm == -INFINITY ? 0.f : exp2f(pm - N);
      Lx = (M == -INFINITY ? 0.f : c * Lx) + d * pl;
      O = (M == -INFINITY ? 0.f : c * O) + d * po;
    }
    const float r = len > 0 ? O / Lx : 0.f;
    if constexpr (PARTS == 1) ((__nv_bfloat16*)p.out)[(head0 + h) * kD + tid] = __float2bfloat16_rn(r);
    else ((float*)p.out)[(head0 + h) * kD + tid] = r;
  };
  if (n_act == 1) {
    pdl_wait();
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < p.rep) store(h, oo[h], MM[h], LL[h]);
    return;
  }
  const size_t pair = (size_t)b * p.Hkv + g;
  const size_t per = (size_t)p.rep * (kD + 2);
  float* base = p.part + pair * gridDim.x * per;
  float* my = base + split * per;
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
    if (h < p.rep) {
      my[h * kD + tid] = oo[h];
      if (tid == 0) {
        my[p.rep * kD + h] = MM[h];
        my[p.rep * kD + p.rep + h] = LL[h];
      }
    }
  __syncthreads();
  if (tid == 0) s_last = atom_add_acq_rel_gpu(p.tickets + pair, 1) == n_act - 1;
  __syncthreads();
  pdl_wait();
  if (!s_last) return;
  if (tid < p.rep) {
    float M = -INFINITY, Lx = 0.f;
    for (int k = 0; k < n_act; ++k) M = fmaxf(M, __ldcg(base + k * per + p.rep * kD + tid));
    for (int k = 0; k < n_act; ++k) {
      const float x = exp2f(__ldcg(base + k * per + p.rep * kD + tid) - M);
      s_w[k][tid] = x;
      Lx = fmaf(x, __ldcg(base + k * per + p.rep * kD + p.rep + tid), Lx);
    }
    s_w[kMaxSplits][tid] = M;
    s_tot[tid] = Lx;
  }
  __syncthreads();
  for (int h = 0; h < p.rep; ++h) {
    float O = 0.f;
#pragma unroll 8
    for (int k = 0; k < n_act; ++k) O = fmaf(s_w[k][h], __ldcg(base + k * per + h * kD + tid), O);
    store(h, O, s_w[kMaxSplits][h], s_tot[h]);
  }
  if (tid == 0) p.tickets[pair] = 0;
}

// Splits per (sequence, kv head): about two rounds of two CTAs per SM.
int splits(int B, int Hkv) {
  const long long want = 4LL * dev_info().sm_count, pairs = (long long)B * Hkv;
  return (int)std::max(1LL, std::min((long long)kMaxSplits, (want + pairs - 1) / pairs));
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t pre_bytes(int B, int Hq) { return round256((size_t)B * Hq * (kD + 2) * 4); }
size_t ticket_bytes(int B, int Hkv) { return round256((size_t)B * Hkv * 4); }

template <typename T, int PARTS>
cudaError_t launch(const SParams& p, int n_splits, const Launch& L) {
  auto k = attn_suffix_kernel<T, PARTS>;
  const size_t smem = (size_t)kW * kStages * kStage;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_ex(k, dim3(n_splits, p.Hkv, p.B), dim3(kTh), smem, L, p);
}

}  // namespace

// attention_rows.cu's workspace, then the tickets, the prefix results and the splits.
size_t attn_shared_workspace_bytes(int B, int Hq, int Hkv) {
  return round256(attn_rows_workspace_bytes()) + ticket_bytes(B, Hkv) + pre_bytes(B, Hq) +
         (size_t)B * Hkv * splits(B, Hkv) * (Hq / Hkv) * (kD + 2) * 4;
}

cudaError_t launch_attn_shared(const AttnRowsArgs& a, const Launch& L) {
  unsigned char* ws = (unsigned char*)a.workspace + round256(attn_rows_workspace_bytes());
  float* pre = (float*)(ws + ticket_bytes(a.n_rows, a.Hkv));
  Launch first = L;
  first.pdl = false;   // whatever ran before in the stream is done before either kernel reads
  cudaError_t e = launch_attn_prefix(a, pre, first);
  if (e != cudaSuccess) return e;
  SParams p = {};
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
  p.tickets = (int*)ws;
  p.part = (float*)(ws + ticket_bytes(a.n_rows, a.Hkv) + pre_bytes(a.n_rows, a.Hq));
  p.err = L.err;
  const int n = splits(a.n_rows, a.Hkv);
  return a.q_f32 ? launch<float, 3>(p, n, L) : launch<__nv_bfloat16, 1>(p, n, L);
}

}  // namespace qd
