// The attention that packed rows give to each key of their sequence: the softmax weights of a
// prompt's rows (all, or the last few), summed over rows and the q heads of a kv head. Eviction goes
// by these sums (pages_evict.cu); attention_window.cu adds those of single tokens.
//
// Two launches, since a weight needs its row's whole sum: the first finds each row's largest score
// and sum, the second forms the scores again and adds the weights up. Both take tiles of 128 rows (tokens
// times the q heads of a kv head) by 128 keys on tcgen05 and differ in which operand stays. The
// first keeps a row tile of Q and walks the keys: a TMEM lane is a row, whose maximum and sum stay in
// a thread. The second keeps a tile of K and walks the row tiles: a TMEM lane is a key, whose sum stays
// in a thread, so that nothing is added across threads until the end. Row tiles are written out
// by the first launch as they lie in shared memory (an f32 q in three bf16 parts, 24 bits), so the
// second brings them by plain 16-byte copies. A cluster's CTAs share the walk of one tile, for calls
// with few tiles, and the first of them adds their results up in rank order through
// distributed shared memory: no atomics, the same bits each time.
//
// The two MUFU exponentials a (row, key) bound it: 2 x 1024 cycles a pair of tiles, against 256 for
// each product (768 in three parts), which run beside them in the other of two S buffers.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tc_common.cuh"

#include <algorithm>

namespace qd {
namespace {

constexpr int kD = 128;
constexpr int kTile = 128;                  // rows, and keys
constexpr int kChunk = 128 * 128;           // [128 x 64 bf16], 128-byte swizzle
constexpr int kSlot = 2 * kChunk;           // a tile of K, or one part of a tile of Q
constexpr int kTh = 256;
constexpr int kMisc = 3 * 1024;
constexpr int kMaxSeg = 1024;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  const void* q;
  long long q_stride;
  const __nv_bfloat16* k_pages;
  const int32_t *page_table, *cu, *seq_lens;
  int n_seg, n_rows, last, rep, log_rep, Hkv, page_size, max_pages, n_pages;
  int cluster;
  long long cap, window, sinks;
  float scale_log2;
  long long* base;         // [2][kMaxSeg + 1]: row tiles and key tiles before each segment (of one kv head)
  float2* stats;           // [row tiles][128]: largest score in log2 units, 1 / sum
  unsigned char* image;    // [row tiles][parts][kSlot]
  float* sums;             // [n_seg][Hkv][cap]
  PageDiv div;
  int* err;
};

QD_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
QD_DEV uint32_t pack(float lo, float hi) { return f2bf_bits(lo) | f2bf_bits(hi) << 16; }
QD_DEV void cp16(uint32_t dst, const void* src, int bytes) {   // bytes 0: zeros, nothing read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
QD_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
QD_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
QD_DEV float ld_cluster(const float* p, uint32_t rank) {   // the same place in another CTA of the cluster
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// The rows of a sequence that count: n of them from packed row row0 on, row j at token off + j.
struct Seg {
  int row0, n, off, len;
};
QD_DEV Seg segment(const Params& p, int s) {
  Seg a;
  const int lo = p.cu[s], hi = p.cu[s + 1];
  a.len = p.seq_lens[s];
  a.n = a.len < 0 || a.len > p.cap ? 0 : hi - lo;
  if (p.last > 0) a.n = min(a.n, p.last);
  a.row0 = hi - a.n;
  a.off = a.len - a.n;
  return a;
}
QD_DEV int row_tiles(const Params& p, const Seg& a) { return (a.n + (kTile >> p.log_rep) - 1) >> (7 - p.log_rep); }

template <int PARTS, int PASS>
constexpr int kRing = PARTS == 3 && PASS == 1 ? 3 : 2;   // tiles that come
template <int PARTS, int PASS>
constexpr size_t kSmem = kMisc + (size_t)kSlot * (PASS == 1 ? PARTS + kRing<PARTS, PASS> : 1 + PARTS * kRing<PARTS, PASS>);

template <typename T, int PARTS, int PASS>
__global__ void __launch_bounds__(kTh, PARTS == 1 ? 2 : 1) attn_weights_kernel(const __grid_constant__ Params p) {
  constexpr int kStages = kRing<PARTS, PASS>;
  constexpr int kFixed = PASS == 1 ? PARTS : 1, kMoving = PASS == 1 ? 1 : PARTS;   // slots of the tile that stays, of one that comes
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bar = (uint64_t*)smem;                 // [2] S in buffer b is there
  uint32_t* tslot = (uint32_t*)(bar + 2);
  int* s_abort = (int*)(tslot + 1);
  long long* s_scan = (long long*)(smem + 64);     // [8] + [8]
  float* red = (float*)(smem + (PASS == 1 ? 1024 : 256));   // pass 1: m [128], l [128]; pass 2: [128]
  float2* stat = (float2*)(smem + 1024);           // pass 2: [2][128] of the rows of two tiles
  unsigned char* fixed = smem + kMisc;
  unsigned char* moving = fixed + kFixed * kSlot;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hf = warp >> 2;
  const int line = (warp & 3) * 32 + lane;         // TMEM lane
  const uint32_t rank = blockIdx.x % p.cluster;
  const int group = blockIdx.x / p.cluster, groups = gridDim.x / p.cluster;

  // ---- tiles before each segment. Pass 1: every CTA for itself (they wait in the workspace for pass 2)
  long long total;   // row or key tiles of one kv head
  if (tid == 0) *s_abort = 0;
  if (smem_u32(smem) & 1023u) {   // the swizzled tiles rest on it (there is no static shared memory); the same in all CTAs
    if (tid == 0) set_error(p.err, QD_DEVERR_TIMEOUT);
    if (PASS == 2) pdl_wait();
    else if (blockIdx.x == 0 && tid == 0) p.base[kMaxSeg + 1 + p.n_seg] = 0;
    return;
  }
  if (PASS == 1) {
    const int per = (p.n_seg + kTh - 1) / kTh;
    long long rows = 0, keys = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
      const int s = tid * per + i;
      if (s >= p.n_seg) break;
      const int lo = p.cu[s], hi = p.cu[s + 1], len = p.seq_lens[s];
      if (lo < 0 || hi < lo || hi > p.n_rows) {
        bad = true;
        continue;
      }
      if (hi > lo && (len < 0 || len > p.cap) && blockIdx.x == 0) set_error(p.err, QD_DEVERR_POS);
      const Seg a = segment(p, s);
      rows += row_tiles(p, a);
      keys += a.n > 0 ? (a.len + kTile - 1) >> 7 : 0;
    }
    const int any_bad = __syncthreads_or(bad);
    long long r = rows, k = keys;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, r, o), y = __shfl_up_sync(0xffffffffu, k, o);
      if (lane >= o) {
        r += x;
        k += y;
      }
    }
    if (lane == 31) {
      s_scan[warp] = r;
      s_scan[8 + warp] = k;
    }
    __syncthreads();
    total = 0;
    long long all_keys = 0, r0 = r - rows, k0 = k - keys;
    for (int w = 0; w < kTh / 32; ++w) {
      if (w < warp) {
        r0 += s_scan[w];
        k0 += s_scan[8 + w];
      }
      total += s_scan[w];
      all_keys += s_scan[8 + w];
    }
    if (any_bad) {   // starts that make no sense: nothing is added
      total = all_keys = 0;
      if (blockIdx.x == 0 && tid == 0) set_error(p.err, QD_DEVERR_POS);
    }
    // every CTA writes the same values, and reads back its own
    if (tid == 0) {
      p.base[p.n_seg] = total;
      p.base[kMaxSeg + 1 + p.n_seg] = all_keys;
    }
    if (!any_bad)
      for (int i = 0; i < per; ++i) {
        const int s = tid * per + i;
        if (s >= p.n_seg) break;
        p.base[s] = r0;
        p.base[kMaxSeg + 1 + s] = k0;
        const Seg a = segment(p, s);
        r0 += row_tiles(p, a);
        k0 += a.n > 0 ? (a.len + kTile - 1) >> 7 : 0;
      }
  }
  if (tid == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_mbar_init();
  }
  if (warp == 0) tc::alloc(tslot, 256);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = *tslot;
  if (PASS == 2) pdl_wait();
  const long long* base = p.base + (PASS == 1 ? 0 : kMaxSeg + 1);
  total = base[p.n_seg];

  uint32_t made = 0;   // products issued so far
  const float c = p.scale_log2;
  const int tpt = kTile >> p.log_rep;   // tokens of a row tile
  for (long long item = group; item < total * p.Hkv; item += groups) {
    // ---- the segment, kv head and tile of the item: the last segment whose tiles start at or before it
    int s = 0;
    {
      const long long tile0 = item / p.Hkv;
      for (int hi = p.n_seg; hi - s > 1;) {
        const int mid = (s + hi) >> 1;
        if (base[mid] <= tile0) s = mid; else hi = mid;
      }
    }
    const Seg a = segment(p, s);
    const long long in = item - base[s] * p.Hkv;
    const int tiles = row_tiles(p, a);
    const int fixed_tiles = PASS == 1 ? tiles : (a.len + kTile - 1) >> 7;
    const int g = (int)(in / fixed_tiles), ft = (int)(in % fixed_tiles);
    const int32_t* pt = p.page_table + (size_t)s * p.max_pages;
    const long long first_rt = p.base[s] * p.Hkv + (long long)g * tiles;   // of the segment and head

    // ---- what the walk passes: key tiles (first ones, then a window), or row tiles [w0, w1)
    int w0 = 0, w1 = 0, jump_at = 0, jump = 0;   // tile i of the walk: w0 + i, + jump from jump_at on
    int key_lo = 0, key_hi = 0;                  // keys that some row sees: below sinks or from key_lo on, below key_hi
    if (PASS == 1) {
      const int j0 = ft * tpt, j1 = min(j0 + tpt, a.n) - 1;
      key_hi = max(0, a.off + j1 + 1);
      key_lo = (int)max(0LL, a.off + j0 + 1 - p.window);
      jump_at = (int)min((p.sinks + kTile - 1) >> 7, 1LL << 24);
      jump = max(0, (key_lo >> 7) - jump_at);
      w1 = ((key_hi + kTile - 1) >> 7) - jump;
    } else {
      const int key0 = ft * kTile;
      key_hi = a.len;
      key_lo = (int)max(0LL, a.off + 1 - p.window);
      const int j0 = max(0, key0 - a.off);       // the first row that may see it
      long long j1 = a.n - 1;                    // the last
      if (key0 >= p.sinks) j1 = min(j1, key0 + kTile - 1 + p.window - 1 - a.off);
      w0 = j0 >> (7 - p.log_rep);
      w1 = j1 < j0 ? w0 : (int)(j1 >> (7 - p.log_rep)) + 1;
      jump_at = INT32_MAX;
    }
    auto tile_at = [&](int i) { return w0 + i >= jump_at ? w0 + i + jump : w0 + i; };
    const int all = w1 - w0;
    if (PASS == 2 && all <= 0) continue;         // (the same in the whole cluster)
    const int n = all > (int)rank ? (all - (int)rank + p.cluster - 1) / p.cluster : 0;   // tiles rank, rank + cluster, ...
    const bool dead0 = *(volatile int*)s_abort != 0;

    auto load_keys = [&](unsigned char* dst, int kt) {   // 16 threads a key
      const uint32_t d = smem_u32(dst) + (uint32_t)((tid & 15) >> 3) * kChunk;
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i) {
        const int r = i * 16 + (tid >> 4), key = kt * kTile + r;
        long long row = -1;
        if (key < key_hi && (key < p.sinks || key >= key_lo)) {
          const PagedSlot sl = paged_slot(pt, key, p.page_size, p.div, p.n_pages);
          if (!sl.ok) set_error(p.err, QD_DEVERR_PAGE);
          row = ((long long)sl.page * p.Hkv + g) * p.page_size + sl.slot;
        }
        cp16(d + tc::sw128_off(r, tid & 7), p.k_pages + max(row, 0LL) * kD + (tid & 15) * 8, row < 0 ? 0 : 16);
      }
    };
    auto load = [&](int i) {   // tile i of this CTA's walk, if there is one
      if (i < n && !dead0) {
        const int t = tile_at((int)rank + i * p.cluster);
        unsigned char* dst = moving + (size_t)((i % kStages) * kMoving) * kSlot;
        if (PASS == 1) {
          load_keys(dst, t);
        } else {
          const unsigned char* src = p.image + (first_rt + t) * (long long)(PARTS * kSlot);
          const uint32_t d = smem_u32(dst);
#pragma unroll 8
          for (int k = tid; k < PARTS * kSlot / 16; k += kTh) cp16(d + k * 16, src + k * 16, 16);
        }
      }
      cp_commit();
    };

    // ---- the tile that stays
    if (!dead0) {
      if (PASS == 2) {
        load_keys(fixed, ft);   // (joins the first group)
      } else {
        // warp w splits rows 16 w ..; lane: dims 4 lane .. + 3
        const int rows = min(tpt, a.n - ft * tpt) << p.log_rep;
        const T* q = (const T*)p.q + (long long)(a.row0 + ft * tpt) * p.q_stride + ((long long)g << p.log_rep) * kD + 4 * lane;
        unsigned char* out = p.image + (first_rt + ft) * (long long)(PARTS * kSlot);
#pragma unroll 1
        for (int i0 = 0; i0 < 16; i0 += 8) {
          float4 f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = warp * 16 + i0 + i;
            const T* from = q + (long long)(r >> p.log_rep) * p.q_stride + (r & (p.rep - 1)) * kD;
            f[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
              if constexpr (PARTS == 1) {
                const uint2 w = *(const uint2*)from;
                f[i] = make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
              } else {
                f[i] = *(const float4*)from;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t o = (uint32_t)((lane >> 4) * kChunk + (lane & 1) * 8) +
                               tc::sw128_off(warp * 16 + i0 + i, (lane & 15) >> 1);
            float x[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
              const uint2 b = make_uint2(pack(x[0], x[1]), pack(x[2], x[3]));
              *(uint2*)(fixed + part * kSlot + o) = b;
              if (rank == 0) *(uint2*)(out + part * kSlot + o) = b;
              x[0] -= bf_lo(b.x); x[1] -= bf_hi(b.x); x[2] -= bf_lo(b.y); x[3] -= bf_hi(b.y);
            }
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kStages; ++i) load(i);

    // ---- what a thread keeps of its line: pass 1 a row's largest score and sum over half the keys of
    // each tile, pass 2 a key's sum over half the rows
    float m = -INFINITY, l = 0.f;
    // pass 1: the row sees keys below lim, of those from sinks on the ones from `from` on; pass 2: the key is
    // seen by the rows of tokens [j_lo, j_hi)
    int lim = 0, from = 0;
    long long j_lo = 0, j_hi = 0;
    if (PASS == 1) {
      const int j = ft * tpt + (line >> p.log_rep);
      lim = j < a.n ? max(0, a.off + j + 1) : 0;
      from = (int)max(0LL, lim - p.window);
    } else {
      const int key = ft * kTile + line;
      j_lo = max(0, key - a.off);
      j_hi = key >= a.len ? 0 : key < p.sinks ? a.n : min((long long)a.n, key + p.window - a.off);
    }
    const uint32_t fix = smem_u32(fixed), mov = smem_u32(moving);
    [[maybe_unused]] float2 held = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int i = 0; i <= n && n > 0; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      fence_proxy_async_smem();
      tc::fence_before();
      if (PASS == 2 && tid < kTile) {   // the statistics of the rows of tile i - 1, read a turn ahead
        if (i > 0) stat[((i - 1) & 1) * kTile + tid] = held;
        if (i < n) held = __ldcg(p.stats + (first_rt + tile_at((int)rank + i * p.cluster)) * kTile + tid);
      }
      __syncthreads();
      const bool dead = *(volatile int*)s_abort != 0;
      if (i < n && tid == 0 && !dead) {
        tc::fence_after();
        const uint32_t mv = mov + (uint32_t)((i % kStages) * kMoving) * kSlot;
        const uint32_t td = tS + 128 * (made & 1);
#pragma unroll 1
        for (int part = PARTS - 1; part >= 0; --part) {   // small parts first
          const uint64_t da = tc::desc_sw128(PASS == 1 ? fix + part * kSlot : fix);
          const uint64_t db = tc::desc_sw128(PASS == 1 ? mv : mv + part * kSlot);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t o = (uint64_t)((kk >> 2) * (kChunk >> 4) + (kk & 3) * 2);
            tc::mma<kTile>(td, da + o, db + o, kk != 0 || part != PARTS - 1);
          }
        }
        tc::commit(&bar[made & 1]);
      }
      if (i > 0 && !dead) {
        const int t = tile_at((int)rank + (i - 1) * p.cluster);
        const uint32_t ts = tS + 128 * ((made - 1) & 1) + ((uint32_t)((warp & 3) * 32) << 16) + 64 * hf;
        if (PASS == 1) {
          const int key0 = t * kTile + 64 * hf;
          const bool whole = key0 + 64 <= lim && (key0 >= from || key0 + 64 <= p.sinks);
          float v[64];
          tc::ld_32x32(ts, v);
          tc::ld_32x32(ts + 32, v + 32);
          float mx[4] = {m, m, m, m};
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            v[e] *= c;
            if (!whole) v[e] = key0 + e < lim && (key0 + e >= from || key0 + e < p.sinks) ? v[e] : -INFINITY;
            mx[e & 3] = fmaxf(mx[e & 3], v[e]);
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const float ref = top == -INFINITY ? 0.f : top;   // a row that has seen nothing yet: weights 2^(-inf - 0)
          if (top != m) l *= ex2(m - top);                  // 0 while m is -inf (l is 0, or NaN then)
          m = top;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 64; ++e) sum[e & 3] += ex2(v[e] - ref);
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        } else {
          const int t0 = t * tpt;   // the columns of the rows that see the key, within this half
          const int lo = (int)max(0LL, min((long long)tpt, j_lo - t0) << p.log_rep) - 64 * hf;
          const int hi = (int)max(0LL, min((long long)tpt, j_hi - t0) << p.log_rep) - 64 * hf;
          const bool whole = lo <= 0 && hi >= 64;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            float v[32];
            tc::ld_32x32(ts + h, v);
            const float4* st = (const float4*)(stat + ((i - 1) & 1) * kTile + 64 * hf + h);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float4 w = st[e / 2];
              float x = ex2(fmaf(v[e], c, -w.x)) * w.y, y = ex2(fmaf(v[e + 1], c, -w.z)) * w.w;
              if (!whole) {
                x = h + e >= lo && h + e < hi ? x : 0.f;
                y = h + e + 1 >= lo && h + e + 1 < hi ? y : 0.f;
              }
              sum[e & 2] += x;
              sum[(e & 2) + 1] += y;
            }
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
      }
      if (i < n) {
        if (!dead && !mbar_wait_bounded(&bar[made & 1], (made >> 1) & 1, p.err)) *(volatile int*)s_abort = 1;
        tc::fence_after();
        ++made;
        load(i + kStages);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- the two halves of a line, then the cluster's CTAs, in order
    if (PASS == 1) {
      float* rm = red;
      float* rl = red + kTile;
      if (hf == 1) {
        rm[line] = m;
        rl[line] = l;
      }
      __syncthreads();
      auto join = [&](float om, float ol) {
        const float top = fmaxf(m, om);
        l = l * (m == -INFINITY ? 1.f : ex2(m - top)) + ol * (om == -INFINITY ? 1.f : ex2(om - top));
        m = top;
      };
      if (hf == 0) join(rm[line], rl[line]);
      if (p.cluster > 1) {
        __syncthreads();
        if (hf == 0) {
          rm[line] = m;
          rl[line] = l;
        }
        cluster_sync();
        if (rank == 0 && hf == 0)
          for (int r = 1; r < p.cluster; ++r) join(ld_cluster(rm + line, r), ld_cluster(rl + line, r));
        cluster_sync();
      } else {
        __syncthreads();
      }
      if (rank == 0 && hf == 0) p.stats[(first_rt + ft) * kTile + line] = make_float2(m, 1.0f / l);
    } else {
      if (hf == 1) red[line] = l;
      __syncthreads();
      if (hf == 0) l += red[line];
      if (p.cluster > 1) {
        __syncthreads();
        if (hf == 0) red[line] = l;
        cluster_sync();
        if (rank == 0 && hf == 0)
          for (int r = 1; r < p.cluster; ++r) l += ld_cluster(red + line, r);
        cluster_sync();
      } else {
        __syncthreads();
      }
      if (rank == 0 && hf == 0 && j_lo < j_hi && !*(volatile int*)s_abort)
        p.sums[((long long)s * p.Hkv + g) * p.cap + ft * kTile + line] += l;
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::dealloc(tS, 256);
  }
}

template <typename T, int PARTS, int PASS>
cudaError_t launch(Params p, int cluster, const Launch& L) {
  constexpr size_t smem = kSmem<PARTS, PASS>;
  cudaError_t e = allow_smem<attn_weights_kernel<T, PARTS, PASS>>(smem);
  if (e != cudaSuccess) return e;
  p.cluster = cluster;
  const int ctas = dev_info().sm_count * (PARTS == 1 ? 2 : 1) / cluster * cluster;
  return launch_ex_cluster(attn_weights_kernel<T, PARTS, PASS>, dim3(std::max(ctas, cluster)), dim3(kTh), smem, cluster, L, p);
}

// CTAs that share a tile's walk: enough for some four items an SM, at most 8, and no more than tiles to walk.
int cluster_for(long long items, long long walk) {
  int n = 1;
  while (n < 8 && items * n < 4LL * dev_info().sm_count && 2 * n <= walk) n *= 2;
  return n;
}

constexpr size_t kBaseBytes = (2 * (kMaxSeg + 1) * 8 + 255) / 256 * 256;
long long counted_rows(int B, int n_rows, int last) { return last > 0 ? std::min((long long)n_rows, (long long)B * last) : n_rows; }
long long most_row_tiles(int B, int n_rows, int rep, int Hkv, int last) {
  return (counted_rows(B, n_rows, last) * rep / kTile + B) * Hkv;
}

}  // namespace

size_t attn_key_weights_workspace_bytes(int B, int n_rows, int Hq, int Hkv, int last, bool f32) {
  const long long n = most_row_tiles(B, n_rows, Hq / Hkv, Hkv, last);
  return kBaseBytes + (size_t)n * kTile * 8 + (size_t)n * (f32 ? 3 : 1) * kSlot;
}

cudaError_t launch_attn_key_weights(const AttnRowsArgs& a, int last, const Launch& L) {
  Params p = {};
  p.q = a.q; p.q_stride = a.q_stride;
  p.k_pages = (const __nv_bfloat16*)a.k_pages;
  p.page_table = a.page_table; p.cu = a.cu; p.seq_lens = a.seq_lens;
  p.n_seg = a.n_seg; p.n_rows = a.n_rows; p.last = last; p.rep = a.Hq / a.Hkv; p.Hkv = a.Hkv;
  while ((1 << p.log_rep) < p.rep) ++p.log_rep;
  p.page_size = a.page_size; p.max_pages = a.max_pages; p.n_pages = a.n_pages;
  p.cap = (long long)a.max_pages * a.page_size;
  p.window = a.window; p.sinks = a.n_sinks;
  p.scale_log2 = a.scale * kLog2e;
  const long long tiles = most_row_tiles(a.n_seg, a.n_rows, p.rep, a.Hkv, last);
  unsigned char* ws = (unsigned char*)a.workspace;
  p.base = (long long*)ws;
  p.stats = (float2*)(ws + kBaseBytes);
  p.image = ws + kBaseBytes + (size_t)tiles * kTile * 8;
  p.sums = a.key_weights;
  p.div = make_page_div(a.page_size);
  p.err = L.err;
  // The host knows neither the lengths nor the rows of each sequence: both are taken to be even, and the
  // keys as many as the rows, or enough to walk.
  const long long rows = counted_rows(a.n_seg, a.n_rows, last);
  const long long per = std::max(1LL, rows * p.rep / kTile / a.n_seg);   // row tiles of a sequence
  const long long shown = (attn_shown_keys(a) + kTile - 1) / kTile;
  const int c1 = cluster_for(a.n_seg * per * a.Hkv, shown);
  const int c2 = cluster_for(a.n_seg * std::max(1LL, per / p.rep) * a.Hkv, per);
  Launch first = L, second = L;
  first.pdl = false;
  second.pdl = true;
  cudaError_t e = a.q_f32 ? launch<float, 3, 1>(p, c1, first) : launch<__nv_bfloat16, 1, 1>(p, c1, first);
  if (e != cudaSuccess) return e;
  return a.q_f32 ? launch<float, 3, 2>(p, c2, second) : launch<__nv_bfloat16, 1, 2>(p, c2, second);
}

}  // namespace qd
