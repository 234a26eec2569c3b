// The attention that packed rows give to each key of their sequence: the softmax weights of a
// prompt's rows (all, or the last few), summed over rows and the q heads of a kv head. Eviction goes
// by these sums (pages_evict.cu); attention_window.cu adds those of single tokens.
//
// Two launches, since a weight needs its row's whole sum: the first finds each row's largest score
// and sum, the second forms the scores again and adds the weights up. Both take tiles of 128 rows (tokens
// times the q heads of a kv head) by 128 keys on tcgen05 and differ in what a tensor-memory lane is and
// which tile stays in shared memory:
//   kStats   a lane is a row, a row tile of Q stays, the keys are walked
//   kSums    a lane is a key, a tile of K stays, the row tiles are walked, so a key's sum stays in a thread
//   kSumsOne the same sums where no sequence has more than one row tile (the last few rows of a
//            prompt): the row tile stays and the keys are walked, each tile's sums added at once
// Where there are few tiles, several CTAs share a tile's walk (with one row tile a sequence each CTA takes an
// equal run of the (sequence, kv head, key tile) units) and the last of them joins their parts in order
// (ticket). So nothing is added in an order that could change. Row tiles are written out by the first
// launch as they lie in shared memory (an f32 q in three bf16 parts, 24 bits), and the second copies them.
//
// Sixteen warps read S, a quarter of a tile's columns each, while one warp issues the products into the other of
// two S buffers and one brings tiles; they meet at mbarriers only. With a CTA barrier per tile, the
// loads shared by all warps, a tile took 1900 to 2900 cycles. Bounds: the exponentials, one a (row, key) in
// each launch, 1024 cycles a pair of tiles (MUFU), against 512 for the product of bf16 tiles; an f32
// q's three parts take 1536. A tile takes 1100 to 1600 cycles. Last 32 rows of 8 prompts (bf16, 48
// key tiles each): 59 us, in each launch a start of some 8 us (segments, Q, the first tile) and 20 tiles a CTA, in the
// first at HBM's rate; all 2011 rows of one prompt (f32): 63 us.
//
// Every wait is bounded; after a timeout all roles run through without touching anything.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tc_common.cuh"

#include <algorithm>
#include <cstring>

namespace qd {
namespace {

constexpr int kD = 128;
constexpr int kTile = 128;                  // rows, and keys
constexpr int kChunk = 128 * 128;           // [128 x 64 bf16], 128-byte swizzle
constexpr int kSlot = 2 * kChunk;           // a tile of K, or one part of a tile of Q
constexpr int kWarps = 16;                  // warps that read S
constexpr int kWorkers = 32 * kWarps;
constexpr int kIssue = kWarps;              // the warp that issues the products, then the one that brings tiles
constexpr int kTh = kWorkers + 64;
enum { kStats, kSums, kSumsOne };
constexpr int kMaxSeg = 1024;
constexpr int kMaxParts = 4096;             // items times shares, where a walk is shared
constexpr int kMaxShares = 16;
static_assert(kMaxParts * 4 == kAttnWeightsHeadBytes, "");
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  const void* q;
  long long q_stride;
  const __nv_bfloat16* k_pages;
  const int32_t *page_table, *cu, *seq_lens;
  int n_seg, n_rows, last, rep, log_rep, Hkv, page_size, max_pages, n_pages;
  long long cap, window, sinks;
  float scale_log2, q_sign;   // (the scale positive, its sign with q)
  int box;                 // rows per TMA box; 0: 16-byte copies
  int one;                 // no sequence has more than one row tile
  int* tickets;            // [kMaxParts], zero between launches
  long long* base;         // [2][kMaxSeg + 1], 1: before each segment, of one kv head: row tiles, and key tiles (`one`: those that
                           // its row tile sees); sequences with rows
  float2* parts;           // [kMaxParts][128]: of shared walks
  float* stats;            // [row tiles][2][128]: negated largest scores in log2 units, 1 / sums
  unsigned char* image;    // [row tiles][parts of q][kSlot]
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
// The products are issued by one lane of a warp whose lanes all walk the same way (`lead` says
// which), so that descriptors stay in uniform registers: 250 cycles a product where one lane
// branched off for them.
QD_DEV void mma_lead(bool lead, uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t accumulate) {
  constexpr uint32_t kIdesc = tc::idesc_m128(kTile);
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(da), "l"(db), "r"(kIdesc), "r"(accumulate), "r"((uint32_t)lead)
      : "memory");
}
QD_DEV void commit_lead(bool lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"((uint32_t)lead)
      : "memory");
}
QD_DEV void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// A tile of K lies as groups of 8 keys of 2048 bytes, one 128-byte-swizzled atom for dims 0 .. 63 and one
// for the others, so that one copy brings whole rows of a page.
constexpr int kKeys8 = 2048, kHalf8 = 1024;
QD_DEV uint32_t k_off(int key, int c) {   // of 16-byte piece c of a key's row
  return (uint32_t)((key >> 3) * kKeys8 + (c >> 3) * kHalf8 + (key & 7) * 128 + (((c & 7) ^ (key & 7)) << 4));
}
QD_DEV uint64_t desc_k(uint32_t saddr) {   // K-major, the stride offset leads to the next 8 keys
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(kKeys8 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
QD_DEV void tma_load_keys(void* dst, const CUtensorMap* map, int row, uint64_t* bar) {   // row: a multiple of 8
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(0), "r"(row >> 3), "r"(smem_u32(bar))
      : "memory");
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

// The key tiles that row tile ft of a segment sees: the first tokens', then from jump tiles further on. Keys seen
// by some row lie below hi, and below sinks or from lo on.
struct Walk {
  int lo, hi, jump_at, jump, n;
};
QD_DEV Walk key_walk(const Params& p, const Seg& a, int ft) {
  const int tpt = kTile >> p.log_rep, j0 = ft * tpt, j1 = min(j0 + tpt, a.n) - 1;
  Walk w;
  w.hi = max(0, a.off + j1 + 1);
  w.lo = (int)max(0LL, a.off + j0 + 1 - p.window);
  w.jump_at = (int)((p.sinks + kTile - 1) >> 7);
  w.jump = max(0, (w.lo >> 7) - w.jump_at);
  w.n = ((w.hi + kTile - 1) >> 7) - w.jump;
  return w;
}

// CTAs that share each walk of `walk` tiles on average: those that give G CTAs the shortest run, when an
// item costs some 3 tiles beside its walk and, over several turns, long and short walks come to three
// quarters of the longest; `most` items times shares at most. By a whole warp, a count a lane.
QD_DEV int shares_for(long long items, long long walk, int G, long long most, int lane) {
  const int n = (lane & (kMaxShares - 1)) + 1, groups = G / n;
  uint32_t key = 0xffffffffu;
  if (n == 1 || (n <= walk && groups > 0 && items * n <= most)) {
    const float turns = ceilf((float)items / (float)groups), tiles = ceilf((float)walk / (float)n);
    const float t = turns <= 1.f ? tiles + 3.f : turns * (0.75f * tiles + 3.f);
    key = (uint32_t)fminf(4.f * t, 1e8f) << 5 | (uint32_t)n;
  }
  return (int)(__reduce_min_sync(0xffffffffu, key) & 31u);
}

template <int PARTS, int PASS>
constexpr int kRing = PASS == kSums ? (PARTS == 3 ? 2 : 4) : PARTS == 3 ? 3 : 5;   // tiles of the walk in shared memory
template <int PASS>
constexpr int kMisc = PASS == kSums ? 3 * 1024 : 8 * 1024;   // barriers and small arrays in front of the tiles
template <int PARTS, int PASS>
constexpr size_t kSmem = kMisc<PASS> + (size_t)kSlot * (PASS == kSums ? 1 + PARTS * kRing<PARTS, PASS> : PARTS + kRing<PARTS, PASS>);

// position and phase in a ring
struct Ring {
  uint32_t slot, ph;
  QD_DEV void step(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      ph ^= 1;
    }
  }
};

// An item: the tile that stays and the walk.
struct Item {
  int s, g, ft, n, i0;     // n: tiles that this CTA walks, from the walk's i0 on in steps of the shares; 0: none
  bool none;               // nobody walks any
  Seg a;
  long long first_rt;      // the first row tile of the segment and head
  int w0, jump_at, jump;   // tile i of the walk: w0 + i, + jump from jump_at on
  long long unit0;         // `one`: the unit that the walk begins with, and all its tiles
  int walk;
  int key_lo, key_hi;      // keys that some row sees: below sinks or from key_lo on, below key_hi
  const int32_t* pt;
};

template <typename T, int PARTS, int PASS>
__global__ void __launch_bounds__(kTh, 1) attn_weights_kernel(const __grid_constant__ CUtensorMap tmK,
                                                              const __grid_constant__ Params p) {
  constexpr uint32_t kStages = kRing<PARTS, PASS>;
  constexpr bool kRows = PASS == kSums;                           // the walk goes over row tiles
  constexpr int kFixed = kRows ? 1 : PARTS, kMoving = kRows ? PARTS : 1;   // slots of the tile that stays, of one of the walk
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* full = (uint64_t*)smem;                // [stages] a tile of the walk has landed
  uint64_t* empty = full + 5;                      // [stages] its product is done
  uint64_t* s_full = empty + 5;                    // [2] S in buffer b is there
  uint64_t* s_free = s_full + 2;                   // [2] ... and has been read
  uint64_t* stat_free = s_free + 2;                // [2] kSums: a row tile's statistics have been read
  uint64_t* fix_full = stat_free + 2;              // the tile that stays is there
  uint64_t* fix_free = fix_full + 1;               // ... and is not needed any more
  uint64_t* drained = fix_free + 1;                // after a timeout: the products so far are done
  uint32_t* tslot = (uint32_t*)(drained + 1);
  int* s_abort = (int*)(tslot + 1);
  int* s_last = s_abort + 1;
  long long* s_scan = (long long*)(smem + 256);    // kStats: [3][18]
  // Statistics of row tiles (kSums: two) [negated maxima, 1 / sums][128]. What the quarters of a line
  // have, but for the first: kStats m and l [2][6][128], kSums one quarter's [128], kSumsOne [2][3][128]
  float* stat = (float*)(smem + 1024);
  float* red = (float*)(smem + (kRows ? 512 : 2048));
  unsigned char* fixed = smem + kMisc<PASS>;
  unsigned char* moving = fixed + kFixed * kSlot;
  // (the warp's number from one lane, so that it is known to be the same in all of them)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 0) *s_abort = 0;
  if (PASS == kStats) pdl_launch_dependents();   // the second launch waits for this one before it reads
  if (smem_u32(smem) & 1023u) {   // the swizzled tiles rest on it (there is no static shared memory); the same in all CTAs
    if (tid == 0) set_error(p.err, QD_DEVERR_TIMEOUT);
    if (PASS != kStats) pdl_wait();
    else if (blockIdx.x == 0 && tid == 0) p.base[p.n_seg] = p.base[kMaxSeg + 1 + p.n_seg] = 0;
    return;
  }
  // ---- tiles before each segment: every CTA of the first launch for itself; they wait in the workspace for the second
  if (PASS == kStats) {
    auto key_tiles = [&](const Seg& a) { return a.n <= 0 ? 0 : p.one ? max(0, key_walk(p, a, 0).n) : (a.len + kTile - 1) >> 7; };
    const int per = (p.n_seg + kTh - 1) / kTh;
    long long rows = 0, keys = 0;
    int some = 0;
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
      keys += key_tiles(a);
      some += a.n > 0;
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
    some = __reduce_add_sync(0xffffffffu, some);
    if (lane == 31) {
      s_scan[warp] = r;
      s_scan[kTh / 32 + warp] = k;
      s_scan[2 * (kTh / 32) + warp] = some;
    }
    __syncthreads();
    long long all_rows = 0, all_keys = 0, r0 = r - rows, k0 = k - keys, segs = 0;
    const int with = min(kTh / 32, (p.n_seg + 31) / 32);   // warps that have segments (the others' sums are 0)
    for (int w = 0; w < with; ++w) {
      if (w < warp) {
        r0 += s_scan[w];
        k0 += s_scan[kTh / 32 + w];
      }
      all_rows += s_scan[w];
      all_keys += s_scan[kTh / 32 + w];
      segs += s_scan[2 * (kTh / 32) + w];
    }
    if (any_bad) {   // starts that make no sense: nothing is added
      all_rows = all_keys = 0;
      if (blockIdx.x == 0 && tid == 0) set_error(p.err, QD_DEVERR_POS);
    }
    // every CTA writes the same values, and reads back its own
    if (tid == 0) {
      p.base[p.n_seg] = all_rows;
      p.base[kMaxSeg + 1 + p.n_seg] = all_keys;
      p.base[2 * (kMaxSeg + 1)] = segs;
    }
    if (!any_bad)
      for (int i = 0; i < per; ++i) {
        const int s = tid * per + i;
        if (s >= p.n_seg) break;
        p.base[s] = r0;
        p.base[kMaxSeg + 1 + s] = k0;
        const Seg a = segment(p, s);
        r0 += row_tiles(p, a);
        k0 += key_tiles(a);
      }
  }
  if (tid == 0) {
    for (uint32_t i = 0; i < kStages; ++i) {
      mbar_init(&full[i], kRows || p.box ? 1 : 32);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], kWarps);
      mbar_init(&stat_free[i], kWarps);
    }
    mbar_init(fix_full, PASS == kStats ? kWorkers : kRows && !p.box ? 32 : 1);
    mbar_init(fix_free, 1 + kWarps);
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  if (warp == 0) tc::alloc(tslot, 256);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = *tslot;
  if (PASS != kStats) {
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");   // the row tiles come by the copy engine
  }

  // ---- the items, and this CTA's: in turn, there and back, the long ones (late rows, early keys) of a segment first
  const bool one = !kRows && p.one;
  const long long* base = p.base + (kRows || one ? kMaxSeg + 1 : 0);
  const long long all_rows = p.base[p.n_seg], all_keys = p.base[kMaxSeg + 1 + p.n_seg];
  const long long segs = max(1LL, p.base[2 * (kMaxSeg + 1)]);
  const long long items = (kRows || one ? all_keys : all_rows) * p.Hkv;   // `one`: units
  const int shares = items == 0 || one ? 1
                                       : shares_for(items, max(1LL, (kRows ? all_rows : all_keys) / segs), gridDim.x,
                                                    kMaxParts, lane);
  const int rank = blockIdx.x % shares, group = blockIdx.x / shares, groups = gridDim.x / shares;
  // `one`: CTA c takes per + (c < rem) units
  const long long runs = min((long long)gridDim.x, items), per = runs ? items / runs : 0, rem = runs ? items % runs : 0;
  auto first_of = [&](long long c) { return c * per + min(c, rem); };
  auto owner = [&](long long u) { return u < rem * (per + 1) ? u / (per + 1) : rem + (u - rem * (per + 1)) / per; };
  const long long end = blockIdx.x < runs ? first_of(blockIdx.x + 1) : 0;
  const int tpt = kTile >> p.log_rep;   // tokens of a row tile
  auto next_item = [&](long long& round, long long& item) {   // (`one`: round counts units)
    if (one) {
      item = round;
      return round < end;
    }
    for (; group < groups && round * groups < items; ++round) {
      item = round * groups + (round & 1 ? groups - 1 - group : group);
      if (item < items) {
        ++round;
        return true;
      }
    }
    return false;
  };
  auto look_up = [&](long long& round, long long item) {
    Item x;
    // the last segment whose tiles start at or before it, in one or two looks of the warp
    const long long tile0 = item / p.Hkv;
    const int step = (p.n_seg + 31) >> 5;
    const int some = __popc(__ballot_sync(0xffffffffu, lane * step < p.n_seg && base[min(lane * step, p.n_seg - 1)] <= tile0));
    x.s = max(0, some - 1) * step;
    if (step > 1) {
      const int more = __popc(__ballot_sync(0xffffffffu, lane < step && x.s + lane < p.n_seg && base[min(x.s + lane, p.n_seg - 1)] <= tile0));
      x.s += max(0, more - 1);
    }
    x.a = segment(p, x.s);
    const Seg& a = x.a;
    const long long in = item - base[x.s] * p.Hkv;
    const int tiles = row_tiles(p, a);
    x.pt = p.page_table + (size_t)x.s * p.max_pages;
    x.w0 = x.jump = x.ft = 0;
    x.jump_at = INT32_MAX;
    if (!kRows) {
      if (!one) {
        x.g = (int)(in % p.Hkv);
        x.ft = tiles - 1 - (int)(in / p.Hkv);
      }
      const Walk w = key_walk(p, a, x.ft);
      x.key_lo = w.lo;
      x.key_hi = w.hi;
      x.jump_at = w.jump_at;
      x.jump = w.jump;
      x.walk = w.n;
    } else {
      x.g = (int)(in % p.Hkv);
      x.ft = (int)(in / p.Hkv);
      const int key0 = x.ft * kTile;
      x.key_hi = a.len;
      x.key_lo = (int)max(0LL, a.off + 1 - p.window);
      const int j0 = max(0, key0 - a.off);       // the first row that may see it
      long long j1 = a.n - 1;                    // the last
      if (key0 >= p.sinks) j1 = min(j1, key0 + kTile - 1 + p.window - 1 - a.off);
      x.w0 = j0 >> (7 - p.log_rep);
      x.walk = j1 < j0 ? 0 : (int)(j1 >> (7 - p.log_rep)) + 1 - x.w0;
    }
    x.none = x.walk <= 0;
    x.i0 = rank;
    x.n = x.walk > rank ? (x.walk - rank + shares - 1) / shares : 0;
    x.unit0 = item;
    if (one) {   // (a walk of no tiles has no units)
      x.g = (int)(in / x.walk);
      x.i0 = (int)(in - (long long)x.g * x.walk);
      x.n = (int)min((long long)(x.walk - x.i0), end - item);
      x.unit0 = item - x.i0;
      round += x.n;
    }
    x.first_rt = p.base[x.s] * p.Hkv + (long long)x.g * tiles;
    return x;
  };
  // (kSumsOne: backwards, since the first launch left the last tiles in L2: 58.6 us instead of 59.4)
  auto tile_at = [&](const Item& x, int i) {
    const int t = x.w0 + x.i0 + (PASS == kSumsOne ? x.n - 1 - i : i * shares);
    return t >= x.jump_at ? t + x.jump : t;
  };
  // a wait of a whole warp, bounded by its polls (each returns after 2 us where nothing comes); after a timeout
  // anywhere in the CTA it returns soon
  auto wait = [&](uint64_t* bar, uint32_t ph) {
    for (int i = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, ph)); ++i)
      if ((i & 1023) == 0 && (i == 1 << 20 || __any_sync(0xffffffffu, *(volatile int*)s_abort))) {
        if (i == 1 << 20) set_error(p.err, QD_DEVERR_TIMEOUT);
        *(volatile int*)s_abort = 1;
        break;
      }
  };
  long long round = one ? first_of(blockIdx.x) : 0, item;
  Ring rt = {0, 0}, rb = {0, 0}, rf = {0, 0};   // tiles, buffers of S, items

  if (warp == kIssue + 1) {
    // ---- tiles
    Ring rs = {0, 0};       // statistics
    uint64_t* late = nullptr;
    uint32_t brought = 0;
    // keys of tile kt: TMA: lane l, box l; 16-byte copies: keys l, l + 32, ... (slot -1: seen by nobody). What is
    // read is not used before the tile's turn
    constexpr int kMine = 4;
    struct Look {
      int page[kMine], slot[kMine];
    };
    auto look = [&](const Item& x, int kt) {
      Look k;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int key = kt * kTile + (p.box ? lane * p.box : 32 * j + lane), w = p.box ? p.box : 1;
        k.page[j] = 0;
        k.slot[j] = -1;
        if (key < min(x.key_hi, (kt + 1) * kTile) && (key < p.sinks || key + w > x.key_lo) && (j == 0 || !p.box)) {
          const int lp = (int)((uint64_t)(uint32_t)key * p.div.mul >> (31 + p.div.shift));   // key / page_size (PageDiv)
          k.page[j] = x.pt[lp];
          k.slot[j] = key - lp * p.page_size;
        }
      }
      return k;
    };
    auto row_of = [&](const Item& x, const Look& k, int j) {
      const bool ok = (unsigned)k.page[j] < (unsigned)p.n_pages;
      if (k.slot[j] >= 0 && !ok) set_error(p.err, QD_DEVERR_PAGE);
      return k.slot[j] < 0 ? -1 : ((ok ? k.page[j] : 0) * p.Hkv + x.g) * p.page_size + k.slot[j];
    };
    auto land = [&] {   // the copies before the last ones, or all
      if (late) {
        fence_proxy_async_smem();
        mbar_arrive(late);
        late = nullptr;
      }
    };
    auto bring_keys = [&](const Item& x, const Look& k, unsigned char* dst, uint64_t* bar) {
      if (p.box) {
        const bool go = !__any_sync(0xffffffffu, *(volatile int*)s_abort != 0);
        const int row = row_of(x, k, 0);
        const unsigned boxes = __popc(__ballot_sync(0xffffffffu, row >= 0));
        if (lane == 0) {
          if (go && boxes) mbar_arrive_expect_tx(bar, boxes * p.box * 256);
          else mbar_arrive(bar);
        }
        __syncwarp();
        if (go && row >= 0) tma_load_keys(dst + lane * p.box * 256, &tmK, row, bar);
        __syncwarp();
      } else {
        const uint32_t d0 = smem_u32(dst);
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const int mine = row_of(x, k, j);
#pragma unroll 2
          for (int i = 0; i < 32; i += 2) {   // 16 lanes copy one key's 256 bytes
            const int r = i + (lane >> 4), c = lane & 15;
            const int row = __shfl_sync(0xffffffffu, mine, r);
            cp16(d0 + k_off(32 * j + r, c), p.k_pages + (long long)max(row, 0) * kD + c * 8, row < 0 ? 0 : 16);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (late) asm volatile("cp.async.wait_group 1;" ::: "memory");
        land();
        late = bar;
      }
    };
    auto bring_rows = [&](const Item& x, int t, unsigned char* dst, float* st, uint64_t* bar) {   // a row tile, its statistics
      if (lane == 0) {
        if (*(volatile int*)s_abort) {
          mbar_arrive(bar);
        } else {
          mbar_arrive_expect_tx(bar, PARTS * kSlot + 2 * kTile * 4);
          bulk_g2s(dst, p.image + (x.first_rt + t) * (long long)(PARTS * kSlot), PARTS * kSlot, bar);
          bulk_g2s(st, p.stats + (x.first_rt + t) * 2 * kTile, 2 * kTile * 4, bar);
        }
      }
      __syncwarp();
    };
    while (next_item(round, item)) {
      const Item x = look_up(round, item);
      if (x.n == 0) continue;
      if (PASS != kStats) {
        Look k;
        if (kRows) k = look(x, x.ft);
        wait(fix_free, rf.ph ^ 1);   // (the first time, the phase before the first is over)
        if (kRows) {
          bring_keys(x, k, fixed, fix_full);
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          land();
        } else {
          bring_rows(x, x.ft, fixed, stat, fix_full);
        }
        rf.step(1);
      }
      if (kRows) {
        for (int i = 0; i < x.n; ++i) {
          wait(&empty[rt.slot], rt.ph ^ 1);
          wait(&stat_free[rs.slot], rs.ph ^ 1);
          bring_rows(x, tile_at(x, i), moving + (size_t)rt.slot * kMoving * kSlot, stat + rs.slot * 2 * kTile, &full[rt.slot]);
          rt.step(kStages);
          rs.step(2);
          ++brought;
        }
      } else {
        Look now, next = look(x, tile_at(x, 0)), third = {};
        if (x.n > 1) third = look(x, tile_at(x, 1));
        for (int i = 0; i < x.n; ++i) {
          now = next;
          next = third;
          if (i + 2 < x.n) third = look(x, tile_at(x, i + 2));
          wait(&empty[rt.slot], rt.ph ^ 1);
          bring_keys(x, now, moving + (size_t)rt.slot * kSlot, &full[rt.slot]);
          rt.step(kStages);
          ++brought;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        land();
      }
    }
    if (*(volatile int*)s_abort && lane == 0) {   // after a timeout the copies under way land before the CTA leaves (bounded)
      for (uint32_t i = 0; i < kStages; ++i) {
        const bool again = i < rt.slot;   // filled in this round of the ring
        if (again || brought >= kStages) mbar_wait_limit(&full[i], again ? rt.ph : rt.ph ^ 1, p.err, 10000000ull);
      }
      if (PASS != kStats) mbar_wait_limit(fix_full, rf.ph ^ 1, p.err, 10000000ull);
    }
  } else if (warp == kIssue) {
    // ---- products, by one lane of a warp whose lanes all walk the same way
    const bool lead = lane == 0;
    const uint32_t fix = smem_u32(fixed), mov = smem_u32(moving);
    while (next_item(round, item)) {
      const Item x = look_up(round, item);
      if (x.n == 0) continue;
      wait(fix_full, rf.ph);
      rf.step(1);
#pragma unroll 1
      for (int i = 0; i < x.n; ++i) {
        wait(&full[rt.slot], rt.ph);
        wait(&s_free[rb.slot], rb.ph ^ 1);
        tc::fence_after();
        const uint32_t mv = mov + rt.slot * kMoving * kSlot, td = tS + 128 * rb.slot;
        const uint64_t dk = desc_k(kRows ? fix : mv);
#pragma unroll 1
        for (int part = PARTS - 1; part >= 0; --part) {   // small parts first
          const uint64_t dq = tc::desc_sw128((kRows ? mv : fix) + part * kSlot);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t q = dq + (uint64_t)((kk >> 2) * (kChunk >> 4) + (kk & 3) * 2);
            const uint64_t k = dk + (uint64_t)((kk >> 2) * (kHalf8 >> 4) + (kk & 3) * 2);
            mma_lead(lead, td, PASS == kStats ? q : k, PASS == kStats ? k : q, kk != 0 || part != PARTS - 1);
          }
        }
        commit_lead(lead, &s_full[rb.slot]);
        commit_lead(lead, &empty[rt.slot]);
        rt.step(kStages);
        rb.step(2);
      }
      if (PASS != kStats) commit_lead(lead, fix_free);
    }
    if (*(volatile int*)s_abort) {   // (bounded)
      commit_lead(lead, drained);
      mbar_wait_limit(drained, 0, p.err, 10000000ull);
    }
  } else {
    // ---- what becomes of S. TMEM lane `line`; the quarter's columns
    const int line = (warp & 3) * 32 + lane, quarter = warp >> 2, col0 = 32 * quarter, group_bar = 1 + (warp & 3);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float c = p.scale_log2;
    const uint64_t c2 = pack2(c, c);
    Ring rs = {0, 0};
    uint32_t turn = 0;   // items or tiles that went through red
    auto arrive = [&](uint64_t* bar) {   // of the whole warp
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // Whether this CTA is the last of the item's shares; its part is in p.parts. By the first quarter's 4 warps
    auto last_share = [&](long long it, int of) {
      bar_sync(5, kTile);
      if (tid == 0) {
        *s_last = !*(volatile int*)s_abort && atom_add_acq_rel_gpu(p.tickets + it, 1) == of - 1;
        if (*s_last) p.tickets[it] = 0;
      }
      bar_sync(5, kTile);
      return *(volatile int*)s_last != 0;
    };
    while (next_item(round, item)) {
      const Item x = look_up(round, item);
      if (PASS != kStats && x.none) continue;
      const Seg& a = x.a;
      if (PASS == kStats && x.n > 0) {
        // the row tile, warp w rows 8 w ..; lane: dims 4 lane .. + 3 (everybody has seen the last product of the
        // item before)
        const int rows = min(tpt, a.n - x.ft * tpt) << p.log_rep;
        const T* q = (const T*)p.q + (long long)(a.row0 + x.ft * tpt) * p.q_stride + ((long long)x.g << p.log_rep) * kD + 4 * lane;
        unsigned char* out = p.image + (x.first_rt + x.ft) * (long long)(PARTS * kSlot);
        float4 f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = warp * 8 + i;
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
        auto split = [&](auto put) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t o = (uint32_t)((lane >> 4) * kChunk + (lane & 1) * 8) + tc::sw128_off(warp * 8 + i, (lane & 15) >> 1);
            float e[4] = {f[i].x * p.q_sign, f[i].y * p.q_sign, f[i].z * p.q_sign, f[i].w * p.q_sign};
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
              const uint2 b = make_uint2(pack(e[0], e[1]), pack(e[2], e[3]));
              put(part * kSlot + o, b);
              e[0] -= bf_lo(b.x); e[1] -= bf_hi(b.x); e[2] -= bf_lo(b.y); e[3] -= bf_hi(b.y);
            }
          }
        };
        split([&](uint32_t o, uint2 b) { *(uint2*)(fixed + o) = b; });
        fence_proxy_async_smem();
        mbar_arrive(fix_full);
        // (written out behind the fence, which would wait for it)
        if (x.i0 == 0) split([&](uint32_t o, uint2 b) { *(uint2*)(out + o) = b; });
      }
      if (PASS == kSumsOne && x.n > 0) {   // the statistics came with the row tile
        wait(fix_full, rf.ph);
        rf.step(1);
      }

      // what a thread keeps of its line over a quarter of the columns of each tile: a row's largest score and
      // sum, or a key's sum
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
        const int j = x.ft * tpt + (line >> p.log_rep);
        lim = j < a.n ? max(0, a.off + j + 1) : 0;
        from = (int)max(0LL, lim - p.window);
      } else if (kRows) {
        seen_by(x.ft);
      }
      float* sums = p.sums + ((long long)x.s * p.Hkv + x.g) * p.cap;
#pragma unroll 1
      for (int i = 0; i < x.n; ++i) {
        const int t = tile_at(x, i);
        wait(&s_full[rb.slot], rb.ph);
        if (kRows) {
          // The row tile's statistics came with it, and its own barrier alone says that they are there: s_full tells of
          // the products. The slot is not filled again before this warp has freed the statistics (two at a time)
          wait(&full[rt.slot], rt.ph);
          rt.step(kStages);
        }
        tc::fence_after();
        float v[32];
        ld32(tS + 128 * rb.slot + lanes + col0, v);
        wait_ld();
        tc::fence_before();
        arrive(&s_free[rb.slot]);
        rb.step(2);
        if (PASS == kStats) {
          const int key0 = t * kTile + col0;
          if (!(key0 + 32 <= lim && (key0 >= from || key0 + 32 <= p.sinks))) {
            const int hi = lim - key0, lo = from - key0, z = (int)min(p.sinks - key0, 64LL);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (e < hi) & ((e >= lo) | (e < z)) ? v[e] : -INFINITY;
          }
          float mx[4] = {m, m, m, m};
#pragma unroll
          for (int e = 0; e < 32; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], v[e + 2 * k], v[e + 2 * k + 1]);
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          const float ref = top == -INFINITY ? 0.f : -top * c;   // a row that has seen nothing yet: weights 2^(-inf - 0)
          if (top != m) l *= ex2(fmaf(m, c, ref));               // 0 while m is -inf (l is 0, or NaN then)
          m = top;
          const uint64_t r2 = pack2(ref, ref);
          uint64_t sum[2] = {0, 0};   // pairs of sums, +0 each
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float y0, y1;
            unpack2(fma2(pack2(v[e], v[e + 1]), c2, r2), y0, y1);
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(ex2(y0), ex2(y1)));
          }
          float y0, y1;
          unpack2(add2(sum[0], sum[1]), y0, y1);
          l += y0 + y1;
        } else {
          // the columns of the rows that see the key, within this quarter
          if (!kRows) seen_by(t);
          const int t0 = (kRows ? t : x.ft) * tpt;
          const int lo = (int)max(0LL, min((long long)tpt, j_lo - t0) << p.log_rep) - col0;
          const int hi = (int)max(0LL, min((long long)tpt, j_hi - t0) << p.log_rep) - col0;
          const float* st = stat + (kRows ? rs.slot * 2 * kTile : 0) + col0;
          uint64_t sum[2] = {0, 0};
          if (lo <= 0 && hi >= 32) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const ulonglong2 nm = *(const ulonglong2*)(st + e), iv = *(const ulonglong2*)(st + kTile + e);
              float y0, y1;
              unpack2(fma2(pack2(v[e], v[e + 1]), c2, nm.x), y0, y1);
              sum[0] = fma2(pack2(ex2(y0), ex2(y1)), iv.x, sum[0]);
              unpack2(fma2(pack2(v[e + 2], v[e + 3]), c2, nm.y), y0, y1);
              sum[1] = fma2(pack2(ex2(y0), ex2(y1)), iv.y, sum[1]);
            }
          } else if (lo < 32 && hi > 0 && lo < hi) {
            float one[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float w = ex2(fmaf(v[e], c, st[e])) * st[kTile + e];
              one[e & 3] += (e >= lo) & (e < hi) ? w : 0.f;
            }
            sum[0] = pack2(one[0], one[1]);
            sum[1] = pack2(one[2], one[3]);
          }
          float y0, y1;
          unpack2(add2(sum[0], sum[1]), y0, y1);
          if (kRows) {
            l += y0 + y1;
            arrive(&stat_free[rs.slot]);
            rs.step(2);
          } else {
            // the tile's sums at once. Nobody else adds to them: an atomic only so that the old value is not waited for
            l = y0 + y1;
            float* r = red + (turn++ & 1) * 3 * kTile + line;
            if (quarter > 0) r[(quarter - 1) * kTile] = l;
            bar_sync(group_bar, 4 * 32);
            if (quarter == 0 && j_lo < j_hi && !*(volatile int*)s_abort)
              atomicAdd(sums + t * kTile + line, (l + r[0]) + (r[kTile] + r[2 * kTile]));
          }
        }
      }
      if (PASS != kStats && x.n > 0) arrive(fix_free);

      // ---- the quarters of a line, then the shares, in order
      if (PASS == kStats) {
        m *= c;   // log2 units
        float* r = red + (turn++ & 1) * 6 * kTile + line;
        if (quarter > 0) {
          r[(quarter - 1) * kTile] = m;
          r[(quarter + 2) * kTile] = l;
        }
        bar_sync(group_bar, 4 * 32);
        if (quarter == 0) {
          auto join = [&](float om, float ol) {
            const float top = fmaxf(m, om);
            l = l * (m == -INFINITY ? 1.f : ex2(m - top)) + ol * (om == -INFINITY ? 1.f : ex2(om - top));
            m = top;
          };
#pragma unroll
          for (int k = 0; k < 3; ++k) join(r[k * kTile], r[(k + 3) * kTile]);
          bool out = true;
          if (one) {   // parts [CTA][2], the second where a walk begins
            const long long c0 = owner(x.unit0), c1 = owner(x.unit0 + x.walk - 1);
            if (c0 != c1) {
              p.parts[(blockIdx.x * 2LL + (x.i0 == 0)) * kTile + line] = make_float2(m, l);
              out = last_share(c0, (int)(c1 - c0) + 1);
              if (out) {
                const float2 first = __ldcg(p.parts + (c0 * 2 + 1) * kTile + line);
                m = first.x;
                l = first.y;
                for (long long k = c0 + 1; k <= c1; ++k) {
                  const float2 o = __ldcg(p.parts + k * 2 * kTile + line);
                  join(o.x, o.y);
                }
              }
            }
          } else if (shares > 1) {
            float2* part = p.parts + item * shares * kTile + line;
            part[rank * kTile] = make_float2(m, l);
            out = last_share(item, shares);
            if (out) {
              const float2 first = __ldcg(part);
              m = first.x;
              l = first.y;
              for (int k = 1; k < shares; ++k) {
                const float2 o = __ldcg(part + k * kTile);
                join(o.x, o.y);
              }
            }
          }
          if (out) {
            float* st = p.stats + (x.first_rt + x.ft) * 2 * kTile + line;
            st[0] = -m;
            st[kTile] = 1.0f / l;
          }
        }
      } else if (kRows) {
#pragma unroll 1
        for (int k = 1; k < 4; ++k) {   // (one quarter at a time: there is no more space)
          if (quarter == k) red[line] = l;
          bar_sync(group_bar, 4 * 32);
          if (quarter == 0) l += red[line];
          bar_sync(group_bar, 4 * 32);
        }
        if (quarter == 0) {
          bool out = !*(volatile int*)s_abort;
          if (shares > 1) {
            float* part = (float*)p.parts + item * shares * kTile + line;
            part[rank * kTile] = l;
            out = last_share(item, shares);
            if (out) {
              l = __ldcg(part);
              for (int k = 1; k < shares; ++k) l += __ldcg(part + k * kTile);
            }
          }
          if (out && j_lo < j_hi) sums[x.ft * kTile + line] += l;
        }
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::dealloc(tS, 256);
  }
}

template <typename T, int PARTS, int PASS>
cudaError_t launch(const CUtensorMap& tm, const Params& p, const Launch& L) {
  constexpr size_t smem = kSmem<PARTS, PASS>;
  cudaError_t e = allow_smem<attn_weights_kernel<T, PARTS, PASS>>(smem);
  if (e != cudaSuccess) return e;
  return launch_ex(attn_weights_kernel<T, PARTS, PASS>, dim3(dev_info().sm_count), dim3(kTh), smem, L, tm, p);
}

constexpr size_t kBaseBytes = ((2 * (kMaxSeg + 1) + 1) * 8 + 255) / 256 * 256, kPartBytes = (size_t)kMaxParts * kTile * 8;
long long counted_rows(int B, int n_rows, int last) { return last > 0 ? std::min((long long)n_rows, (long long)B * last) : n_rows; }
long long most_row_tiles(int B, int n_rows, int rep, int Hkv, int last) {
  return (counted_rows(B, n_rows, last) * rep / kTile + B) * Hkv;
}

}  // namespace

size_t attn_key_weights_workspace_bytes(int B, int n_rows, int Hq, int Hkv, int last, bool f32) {
  const long long n = most_row_tiles(B, n_rows, Hq / Hkv, Hkv, last);
  return kAttnWeightsHeadBytes + kBaseBytes + kPartBytes + (size_t)n * 2 * kTile * 4 + (size_t)n * (f32 ? 3 : 1) * kSlot;
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
  p.tickets = (int*)ws;
  p.base = (long long*)(ws + kAttnWeightsHeadBytes);
  p.parts = (float2*)((unsigned char*)p.base + kBaseBytes);
  p.stats = (float*)((unsigned char*)p.parts + kPartBytes);
  p.image = (unsigned char*)p.stats + (size_t)tiles * 2 * kTile * 4;
  p.sums = a.key_weights;
  p.div = make_page_div(a.page_size);
  p.err = L.err;
  p.one = (last > 0 && (long long)last * p.rep <= kTile) || (long long)a.n_rows * p.rep <= kTile;
  // boxes of whole 16-row pieces of a page; other page sizes by 16-byte asynchronous copies
  alignas(64) CUtensorMap tm;
  memset(&tm, 0, sizeof(tm));
  if (a.page_size % 16 == 0) {
    p.box = 16;
    while (p.box < kTile && a.page_size % (2 * p.box) == 0) p.box *= 2;
    cudaError_t e = encode_tmap_bf16_rows128(&tm, a.k_pages, (uint64_t)a.n_pages * a.Hkv * a.page_size, p.box);
    if (e != cudaSuccess) return e;
  }
  Launch first = L, second = L;
  first.pdl = false;
  second.pdl = true;
  cudaError_t e = a.q_f32 ? launch<float, 3, kStats>(tm, p, first) : launch<__nv_bfloat16, 1, kStats>(tm, p, first);
  if (e != cudaSuccess) return e;
  if (p.one) return a.q_f32 ? launch<float, 3, kSumsOne>(tm, p, second) : launch<__nv_bfloat16, 1, kSumsOne>(tm, p, second);
  return a.q_f32 ? launch<float, 3, kSums>(tm, p, second) : launch<__nv_bfloat16, 1, kSums>(tm, p, second);
}

}  // namespace qd
