// The attention that packed rows give to each key of their sequence: the softmax weights of a
// prompt's rows (all, or the last few), summed over rows and the q heads of a kv head. Eviction goes
// by these sums (pages_evict.cu); attention_window.cu adds those of single tokens.
//
// Two launches, since a weight needs its row's whole sum: the first finds each row's largest score
// and sum, the second forms the scores again and adds the weights up. Both take tiles of 128 rows (tokens
// times the q heads of a kv head) by 128 keys on tcgen05, S in one of two tensor-memory buffers while the
// other is read, and differ in what a TMEM lane is and which tile stays in shared memory:
//   kStats   a lane is a row, a row tile of Q stays, the keys are walked; a cluster's CTAs share the
//            walk and join in rank order through distributed shared memory
//   kSums    a lane is a key, a tile of K stays, the row tiles are walked (shared by a cluster in the
//            same way), so a key's sum stays in a thread
//   kSumsOne the same sums where no sequence has more than one row tile (the last few rows of a
//            prompt): the row tile stays and the keys are walked, each tile's sums added at once
// So nothing is added in an order that could change. Row tiles are written out by the first launch as
// they lie in shared memory (an f32 q in three bf16 parts, 24 bits), and the second copies them.
//
// Bounds: the exponentials, one a (row, key) in each launch: 1024 cycles a pair of tiles (MUFU), against 512
// for the product of bf16 tiles; an f32 q's three parts take 1536. PERF_NOTE
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
enum { kStats, kSums, kSumsOne };
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
  float scale_log2, q_sign;   // (the scale positive, its sign with q)
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
// two floats at a time
QD_DEV uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
QD_DEV void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
QD_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
QD_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
QD_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
QD_DEV void ld32(uint32_t taddr, float* v) {   // 32 columns, not waited for
  uint32_t* r = (uint32_t*)v;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
QD_DEV void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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

// kSums walks row tiles, the others key tiles (whose cache rows are looked up two turns ahead)
template <int PARTS, int PASS>
constexpr int kRing = PASS == kSums ? 2 : PARTS == 3 ? 3 : 2;   // tiles of the walk in shared memory
template <int PASS>
constexpr int kMisc = PASS == kSums ? 3 * 1024 : 5 * 1024;   // barriers and small arrays in front of the tiles
template <int PARTS, int PASS>
constexpr size_t kSmem = kMisc<PASS> + (size_t)kSlot * (PASS == kSums ? 1 + PARTS * kRing<PARTS, PASS> : PARTS + kRing<PARTS, PASS>);

template <typename T, int PARTS, int PASS>
__global__ void __launch_bounds__(kTh, PARTS == 1 ? 2 : 1) attn_weights_kernel(const __grid_constant__ Params p) {
  constexpr int kStages = kRing<PARTS, PASS>;
  constexpr bool kRows = PASS == kSums;                           // the walk goes over row tiles
  constexpr int kFixed = kRows ? 1 : PARTS, kMoving = kRows ? PARTS : 1;   // slots of the tile that stays, of one of the walk
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bar = (uint64_t*)smem;                 // [2] S in buffer b is there
  uint64_t* full = bar + 2;                        // [2] kSums: a row tile has landed
  uint32_t* tslot = (uint32_t*)(full + 2);
  int* s_abort = (int*)(tslot + 1);
  long long* s_scan = (long long*)(smem + 64);     // [8] + [8]
  // kSums: cache rows of the key tile, later the sums of a half [128]; statistics of two row tiles
  // [2][negated maxima, 1 / sums][128]. The others: cache rows [stages + 1][128], then kStats m, l [128]
  // each, kSumsOne the sums of a half [2][128] and the row tile's statistics
  int* look_rows = (int*)(smem + (kRows ? 256 : 1024));
  float* red = (float*)(smem + (kRows ? 256 : 3072));
  float* stat = (float*)(smem + (kRows ? 1024 : 4096));
  unsigned char* fixed = smem + kMisc<PASS>;
  unsigned char* moving = fixed + kFixed * kSlot;
  // (the warp's number from one lane, so that it is known to be the same in all of them)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), hf = warp >> 2;
  const int line = (warp & 3) * 32 + lane;         // TMEM lane
  const uint32_t rank = blockIdx.x % p.cluster;
  const int group = blockIdx.x / p.cluster, groups = gridDim.x / p.cluster;

  if (tid == 0) *s_abort = 0;
  if (smem_u32(smem) & 1023u) {   // the swizzled tiles rest on it (there is no static shared memory); the same in all CTAs
    if (tid == 0) set_error(p.err, QD_DEVERR_TIMEOUT);
    if (PASS != kStats) pdl_wait();
    else if (blockIdx.x == 0 && tid == 0) p.base[p.n_seg] = p.base[kMaxSeg + 1 + p.n_seg] = 0;
    return;
  }
  // ---- tiles before each segment: every CTA of the first launch for itself; they wait in the workspace for the second
  if (PASS == kStats) {
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
    long long all_rows = 0, all_keys = 0, r0 = r - rows, k0 = k - keys;
    for (int w = 0; w < kTh / 32; ++w) {
      if (w < warp) {
        r0 += s_scan[w];
        k0 += s_scan[8 + w];
      }
      all_rows += s_scan[w];
      all_keys += s_scan[8 + w];
    }
    if (any_bad) {   // starts that make no sense: nothing is added
      all_rows = all_keys = 0;
      if (blockIdx.x == 0 && tid == 0) set_error(p.err, QD_DEVERR_POS);
    }
    // every CTA writes the same values, and reads back its own
    if (tid == 0) {
      p.base[p.n_seg] = all_rows;
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[i], 1);
      mbar_init(&full[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) tc::alloc(tslot, 256);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = *tslot;
  if (PASS != kStats) pdl_wait();
  const long long* base = p.base + (kRows ? kMaxSeg + 1 : 0);
  const long long items = base[p.n_seg] * p.Hkv;

  uint32_t made = 0, landed = 0;   // products issued, row tiles copied so far
  const float c = p.scale_log2;
  const uint64_t c2 = pack2(c, c);
  const int tpt = kTile >> p.log_rep;   // tokens of a row tile
  // items in turn, there and back: the long ones (late rows, early keys) come first in a segment
  for (long long round = 0; round * groups < items; ++round) {
    const long long item = round * groups + (round & 1 ? groups - 1 - group : group);
    if (item >= items) continue;
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
    const int g = (int)(in % p.Hkv), ft = kRows ? (int)(in / p.Hkv) : tiles - 1 - (int)(in / p.Hkv);
    const int32_t* pt = p.page_table + (size_t)s * p.max_pages;
    const long long first_rt = p.base[s] * p.Hkv + (long long)g * tiles;   // of the segment and head

    // ---- what the walk passes: key tiles (first ones, then a window), or row tiles [w0, w1)
    int w0 = 0, w1 = 0, jump_at = INT32_MAX, jump = 0;   // tile i of the walk: w0 + i, + jump from jump_at on
    int key_lo = 0, key_hi = 0;                  // keys that some row sees: below sinks or from key_lo on, below key_hi
    if (!kRows) {
      const int j0 = ft * tpt, j1 = min(j0 + tpt, a.n) - 1;
      key_hi = max(0, a.off + j1 + 1);
      key_lo = (int)max(0LL, a.off + j0 + 1 - p.window);
      jump_at = (int)((p.sinks + kTile - 1) >> 7);
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
    }
    const int all = w1 - w0;
    if (PASS != kStats && all <= 0) continue;    // (the same in the whole cluster)
    const int n = all > (int)rank ? (all - (int)rank + p.cluster - 1) / p.cluster : 0;   // tiles rank, rank + cluster, ...
    auto tile_at = [&](int i) {
      const int t = w0 + (int)rank + i * p.cluster;
      return t >= jump_at ? t + jump : t;
    };
    const bool dead0 = *(volatile int*)s_abort != 0;

    // ---- keys: threads 0 .. 127 look a key's cache row up (-1: nobody sees it), then 16 threads copy each
    auto look = [&](int kt) {
      const int key = kt * kTile + tid;
      int row = -1;
      if (key < key_hi && (key < p.sinks || key >= key_lo)) {
        const PagedSlot sl = paged_slot(pt, key, p.page_size, p.div, p.n_pages);
        if (!sl.ok) set_error(p.err, QD_DEVERR_PAGE);
        row = (sl.page * p.Hkv + g) * p.page_size + sl.slot;
      }
      return row;
    };
    auto load_keys = [&](unsigned char* dst, const int* rows) {
      const uint32_t d = smem_u32(dst) + (uint32_t)((tid & 15) >> 3) * kChunk;
      const __nv_bfloat16* from = p.k_pages + (tid & 15) * 8;
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i) {
        const int r = i * 16 + (tid >> 4), row = rows[r];
        cp16(d + tc::sw128_off(r, tid & 7), from + (long long)max(row, 0) * kD, row < 0 ? 0 : 16);
      }
    };
    auto load = [&](int i) {   // tile i of this CTA's walk, if there is one
      if constexpr (kRows) {
        if (i < n && !dead0 && tid == 0) {
          mbar_arrive_expect_tx(&full[landed & 1], PARTS * kSlot);
          bulk_g2s(moving + (size_t)((i % kStages) * kMoving) * kSlot,
                   p.image + (first_rt + tile_at(i)) * (long long)(PARTS * kSlot), PARTS * kSlot, &full[landed & 1]);
        }
        if (i < n) ++landed;
      } else {
        if (i < n && !dead0) load_keys(moving + (size_t)(i % kStages) * kSlot, look_rows + i % (kStages + 1) * kTile);
        cp_commit();
      }
    };
    const uint32_t landed0 = landed;
    [[maybe_unused]] int ahead = -1;   // the cache row of this thread's key, a turn ahead

    // ---- the tile that stays, and the first of the walk
    if (tid < kTile) {
      if (kRows) {
        look_rows[tid] = look(ft);
      } else {
        for (int i = 0; i < kStages; ++i)
          if (i < n) look_rows[i * kTile + tid] = look(tile_at(i));
        if (kStages < n) ahead = look(tile_at(kStages));
      }
    }
    if (PASS == kStats && !dead0) {
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
          float x[4] = {f[i].x * p.q_sign, f[i].y * p.q_sign, f[i].z * p.q_sign, f[i].w * p.q_sign};
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
    if (PASS == kSumsOne && !dead0) {
      const unsigned char* src = p.image + (first_rt + ft) * (long long)(PARTS * kSlot);
      const uint32_t d = smem_u32(fixed);
#pragma unroll 8
      for (int k = tid; k < PARTS * kSlot / 16; k += kTh) cp16(d + k * 16, src + k * 16, 16);
      if (tid < kTile) {
        const float2 st = __ldcg(p.stats + (first_rt + ft) * kTile + tid);
        stat[tid] = -st.x;
        stat[kTile + tid] = st.y;
      }
    }
    __syncthreads();
    if (kRows) {
      if (!dead0) load_keys(fixed, look_rows);
      cp_commit();
    }
#pragma unroll
    for (int i = 0; i < kStages; ++i) load(i);   // (kSumsOne: the row tile lands with the first)

    // ---- what a thread keeps of its line over half the columns of each tile: a row's largest score and sum, or a key's sum
    float m = -INFINITY, l = 0.f;
    // kStats: the row sees keys below lim, of those from sinks on the ones from `from` on; else the key of key
    // tile kt is seen by the rows of tokens [j_lo, j_hi)
    int lim = 0, from = 0;
    long long j_lo = 0, j_hi = 0;
    auto seen_by = [&](int kt) {
      const int key = kt * kTile + line;
      j_lo = max(0, key - a.off);
      j_hi = key >= a.len ? 0 : key < p.sinks ? a.n : min((long long)a.n, key + p.window - a.off);
    };
    if (PASS == kStats) {
      const int j = ft * tpt + (line >> p.log_rep);
      lim = j < a.n ? max(0, a.off + j + 1) : 0;
      from = (int)max(0LL, lim - p.window);
    } else if (kRows) {
      seen_by(ft);
    }
    float* sums = p.sums + ((long long)s * p.Hkv + g) * p.cap;
    // kSumsOne: the sums of tile i, whose other half is in red by now. Nobody else adds to them: an atomic
    // only so that the old value is not waited for
    auto flush = [&](int i) {
      if (hf == 0 && j_lo < j_hi) atomicAdd(sums + tile_at(i) * kTile + line, l + red[(i & 1) * kTile + line]);
    };
    const uint32_t fix = smem_u32(fixed), mov = smem_u32(moving);
    [[maybe_unused]] float2 held = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int i = 0; i <= n && n > 0; ++i) {
      if (!kRows || i == 0) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRows ? 0 : kStages - 1) : "memory");
        fence_proxy_async_smem();
      }
      tc::fence_before();
      if (kRows) {
        if (tid < kTile) {   // the statistics of the rows of tile i - 1, read a turn ahead
          if (i > 0) {
            stat[((i - 1) & 1) * 2 * kTile + tid] = -held.x;
            stat[((i - 1) & 1) * 2 * kTile + kTile + tid] = held.y;
          }
          if (i < n) held = __ldcg(p.stats + (first_rt + tile_at(i)) * kTile + tid);
        }
      } else if (tid < kTile) {
        look_rows[(i + kStages) % (kStages + 1) * kTile + tid] = ahead;
        if (i + kStages + 1 < n) ahead = look(tile_at(i + kStages + 1));
      }
      __syncthreads();
      const bool dead = *(volatile int*)s_abort != 0;
      if (i < n && warp == 0 && !dead) {
        bool there = true;
        if (kRows) there = mbar_wait_bounded(&full[(landed0 + i) & 1], ((landed0 + i) >> 1) & 1, p.err);
        if (!there) *(volatile int*)s_abort = 1;
        if (lane == 0 && there) {
          tc::fence_after();
          const uint32_t mv = mov + (uint32_t)((i % kStages) * kMoving) * kSlot;
          const uint32_t td = tS + 128 * (made & 1);
#pragma unroll 1
          for (int part = PARTS - 1; part >= 0; --part) {   // small parts first
            const uint64_t dq = tc::desc_sw128((kRows ? mv : fix) + part * kSlot), dk = tc::desc_sw128(kRows ? fix : mv);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint64_t o = (uint64_t)((kk >> 2) * (kChunk >> 4) + (kk & 3) * 2);
              tc::mma<kTile>(td, (PASS == kStats ? dq : dk) + o, (PASS == kStats ? dk : dq) + o, kk != 0 || part != PARTS - 1);
            }
          }
          tc::commit(&bar[made & 1]);
        }
        __syncwarp();
      }
      if (PASS == kSumsOne && i > 1) flush(i - 2);
      if (i > 0 && !dead) {
        const int t = tile_at(i - 1);
        const uint32_t ts = tS + 128 * ((made - 1) & 1) + ((uint32_t)((warp & 3) * 32) << 16) + 64 * hf;
        float v[64];
        ld32(ts, v);
        ld32(ts + 32, v + 32);
        if (PASS == kStats) {
          const int key0 = t * kTile + 64 * hf;
          wait_ld();
          if (!(key0 + 64 <= lim && (key0 >= from || key0 + 64 <= p.sinks))) {
            const int x = lim - key0, y = from - key0, z = (int)min(p.sinks - key0, 64LL);
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = (e < x) & ((e >= y) | (e < z)) ? v[e] : -INFINITY;
          }
          float mx[4] = {m, m, m, m};
#pragma unroll
          for (int e = 0; e < 64; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], v[e + 2 * k], v[e + 2 * k + 1]);
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          const float ref = top == -INFINITY ? 0.f : -top * c;   // a row that has seen nothing yet: weights 2^(-inf - 0)
          if (top != m) l *= ex2(fmaf(m, c, ref));               // 0 while m is -inf (l is 0, or NaN then)
          m = top;
          const uint64_t r2 = pack2(ref, ref);
          uint64_t sum[2] = {0, 0};   // pairs of sums, +0 each
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float x, y;
            unpack2(fma2(pack2(v[e], v[e + 1]), c2, r2), x, y);
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(ex2(x), ex2(y)));
          }
          float x, y;
          unpack2(add2(sum[0], sum[1]), x, y);
          l += x + y;
        } else {
          // the columns of the rows that see the key, within this half
          if (!kRows) seen_by(t);
          const int t0 = (kRows ? t : ft) * tpt;
          const int lo = (int)max(0LL, min((long long)tpt, j_lo - t0) << p.log_rep) - 64 * hf;
          const int hi = (int)max(0LL, min((long long)tpt, j_hi - t0) << p.log_rep) - 64 * hf;
          const float* st = stat + (kRows ? ((i - 1) & 1) * 2 * kTile : 0) + 64 * hf;
          uint64_t sum[2] = {0, 0};
          wait_ld();
          if (lo <= 0 && hi >= 64) {
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              const ulonglong2 nm = *(const ulonglong2*)(st + e), iv = *(const ulonglong2*)(st + kTile + e);
              float x, y;
              unpack2(fma2(pack2(v[e], v[e + 1]), c2, nm.x), x, y);
              sum[0] = fma2(pack2(ex2(x), ex2(y)), iv.x, sum[0]);
              unpack2(fma2(pack2(v[e + 2], v[e + 3]), c2, nm.y), x, y);
              sum[1] = fma2(pack2(ex2(x), ex2(y)), iv.y, sum[1]);
            }
          } else if (lo < 64 && hi > 0 && lo < hi) {
            float one[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              const float x = ex2(fmaf(v[e], c, st[e])) * st[kTile + e];
              one[e & 3] += (e >= lo) & (e < hi) ? x : 0.f;
            }
            sum[0] = pack2(one[0], one[1]);
            sum[1] = pack2(one[2], one[3]);
          }
          float x, y;
          unpack2(add2(sum[0], sum[1]), x, y);
          if (kRows) {
            l += x + y;
          } else {
            l = x + y;
            if (hf == 1) red[((i - 1) & 1) * kTile + line] = l;
          }
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
    __syncthreads();
    if (PASS == kStats) {
      float* rm = red;
      float* rl = red + kTile;
      m *= c;   // log2 units
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
      }
      if (rank == 0 && hf == 0) p.stats[(first_rt + ft) * kTile + line] = make_float2(m, 1.0f / l);
    } else if (kRows) {
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
      }
      if (rank == 0 && hf == 0 && j_lo < j_hi && !*(volatile int*)s_abort) sums[ft * kTile + line] += l;
    } else if (n > 0 && !*(volatile int*)s_abort) {
      flush(n - 1);
    }
    __syncthreads();   // the small arrays are used again
  }
  if (kRows && *(volatile int*)s_abort && tid == 0)   // after a timeout the copies under way land first (bounded)
    for (uint32_t i = landed < 2 ? 0 : landed - 2; i < landed; ++i) mbar_wait_limit(&full[i & 1], (i >> 1) & 1, p.err, 10000000ull);
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
  const int ctas = std::max(1, dev_info().sm_count * (PARTS == 1 ? 2 : 1) / cluster) * cluster;
  if (PASS == kSumsOne) return launch_ex(attn_weights_kernel<T, PARTS, PASS>, dim3(ctas), dim3(kTh), smem, L, p);
  return launch_ex_cluster(attn_weights_kernel<T, PARTS, PASS>, dim3(ctas), dim3(kTh), smem, cluster, L, p);
}

// CTAs that share a tile's walk: enough for one and a half items a CTA slot, at most 8, and no more than tiles to walk.
int cluster_for(long long items, long long walk, bool f32) {
  int n = 1;
  while (n < 8 && 2 * items * n < 3LL * dev_info().sm_count * (f32 ? 1 : 2) && 2 * n <= walk) n *= 2;
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
  // q takes the sign; a scale of 0 makes q 0, so that masked scores stay -inf times something
  p.scale_log2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
  p.q_sign = a.scale < 0.f ? -1.f : a.scale == 0.f ? 0.f : 1.f;
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
  const int c1 = cluster_for(a.n_seg * per * a.Hkv, shown, a.q_f32);
  const int c2 = cluster_for(a.n_seg * std::max(1LL, per / p.rep) * a.Hkv, per, a.q_f32);
  const bool one = (last > 0 && (long long)last * p.rep <= kTile) || (long long)a.n_rows * p.rep <= kTile;
  Launch first = L, second = L;
  first.pdl = false;
  second.pdl = true;
  cudaError_t e = a.q_f32 ? launch<float, 3, kStats>(p, c1, first) : launch<__nv_bfloat16, 1, kStats>(p, c1, first);
  if (e != cudaSuccess) return e;
  if (one) return a.q_f32 ? launch<float, 3, kSumsOne>(p, c1, second) : launch<__nv_bfloat16, 1, kSumsOne>(p, c1, second);
  return a.q_f32 ? launch<float, 3, kSums>(p, c2, second) : launch<__nv_bfloat16, 1, kSums>(p, c2, second);
}

}  // namespace qd
