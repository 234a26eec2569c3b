// Attention of packed rows over the paged cache on tcgen05: the prompts of several
// sequences in one launch, and the shared prefixes of decode rows.
//
// A row tile is 128 rows of one kv head: consecutive packed tokens (prompt form) or
// sequences (shared form) times the Hq / Hkv q heads that read it, so a K/V tile is read
// once for all of them. Work is counted in units of one row tile times 128 keys, ordered
// by (segment, kv head, row tile, keys), and each CTA of the one-per-SM grid takes an equal run
// of them. So ragged prompts, one long prompt and one row behind a long cache all split
// evenly without the host knowing a length; a prompt's row tile that several CTAs share is
// joined, in key order, by the last of them (ticket). A causal row tile counts only the
// tiles that some row of it sees.
//
// Per 128 keys: S = Q K^T (M 128, N 128) into tensor memory, the softmax warps read it,
// keep a reference maximum that moves when a score passes it by more than 2^8 (so that O
// is rescaled rarely), and write the weights back over S as the A operand of O += P V.
// V is read as it lies in the cache (keys x dims) through an MN-major descriptor, so no
// transposed copy exists. Two rings of 32 KB slots hold K and V tiles.
//   * bf16 q: weights rounded to bf16 (each off by 2^-8 of itself at most, as the
//     result's own rounding); sums, statistics and O in f32. Results are 2.0e-3 to 2.5e-3 off the 64-bit
//     form (2-norms), with weights in f32 they would be 1.5e-3 to 1.7e-3; two parts of a weight would cost
//     half as many products again, and those bound the kernel. (With an f32 q: 3e-7.)
//   * f32 q: q and the weights as three bf16 parts each (24 bits; two would leave
//     2.4e-6 of each weight, above what an f32 sum of the same length loses), three times
//     the products.
// A row is held by two threads, one in each half of the softmax warps. bf16: they take whole
// tiles in turn, S runs three tiles ahead of P V in three buffers, each product has a warp that
// issues it, and while one half writes a row tile out the other begins the next. A long prompt is
// bound by the products: they are 1024 of some 1420 cycles per tile (the tensor pipe 72 % active,
// at the clock that power leaves), the exponentials 520, beside them; 8192 tokens of 32 q heads (8
// kv heads) take 390 us, 1410 TFLOP/s, 0.74 of the measured bf16 rate. Both
// halves on one tile, 64 keys each: 558 us; one warp for both products, whatever the softmax did:
// 2100 cycles per tile; two row tiles per CTA, whose S has one buffer each: 643 us. Short row
// tiles (16 messages of 20 to 700 tokens: 71 us) are bound by the start and the end of each, most
// of which is code that the instruction cache does not hold. f32: three products for each of
// bf16's, both halves on one tile, since O is summed in registers.
//
// Keys a row must not see: scores are masked by selection, and V rows that only some rows
// of the tile see are checked for NaN and infinities (0 * NaN would reach every row):
// those entries enter the products as 0 and are added afterwards to the rows that see
// them. Every wait is bounded; after a timeout all roles run through without touching
// anything, so nobody is left waiting.
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tc_common.cuh"

#include <algorithm>
#include <cstring>

namespace qd {
namespace {

constexpr int kD = 128;
constexpr int kRows = 128;               // rows of a row tile (M, TMEM lanes)
constexpr int kKeys = 128;               // keys of a tile
constexpr int kChunk = 128 * 128;        // [128 rows x 64 bf16], 128-byte swizzle
constexpr int kSlot = 2 * kChunk;        // a K or V tile, or one part of a row tile of Q
constexpr int kSoftWarps = 8;
constexpr int kSoft = 32 * kSoftWarps;
// warp roles behind the softmax warps
constexpr int kIssueS = kSoftWarps;         // issues S = Q K^T
constexpr int kProducer = kSoftWarps + 1;   // K tiles; the warp after it V tiles
constexpr int kIssueO = kSoftWarps + 3;     // issues O += P V
constexpr int kThreads = 32 * (kSoftWarps + 4);
// named barriers: 1 and 6 the threads that write a piece out, 2 + quarter the holders of a row,
// kPassed + 4 holder + quarter: the holder has written its reference (7 to 14)
constexpr int kPassed = 7;
// Tiles that the half which begins a row tile takes before the two alternate: about as long as the
// other half needs to write the row tile before out. 8192 tokens with 2, 3, 4, 5, 6, 8, 12, results
// stored row by row: 453, 429, 413, 398, 398, 406, 418 us; as now with 4, 5, 6: 394, 394, 396.
constexpr int kSolo = 5;
constexpr int kMisc = 3 * 1024;              // barriers and small arrays in front of Q and the ring
constexpr int kData = 7 * kSlot;         // 224 KB: Q parts and ring slots
constexpr size_t kSmem = kMisc + kData;  // 227 KB, the whole opt-in shared memory
constexpr int kMaxSlots = 6;
constexpr int kMinUnits = 2;             // units per CTA of a prompt below which fewer CTAs are used
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxTeam = 8;              // row tiles of a group up to which its CTAs form teams
constexpr float kMove = 8.0f;            // log2 units a score may pass the reference maximum
constexpr int kMaxGrid = 192;            // CTAs (SMs) the workspace has room for
constexpr size_t kPartFloats = kPieceFloats;

struct Params {
  const void* q;
  long long q_stride;
  const __nv_bfloat16 *k_pages, *v_pages;
  const int32_t *page_table, *cu, *seq_lens, *shared_lens;
  int n_seg, n_rows, Hq, Hkv, rep, log_rep, page_size, max_pages, n_pages;
  long long cap;
  int box;                 // rows per TMA box; 0: cp.async loads
  float scale_log2, q_sign;
  void* out;
  long long share_min;
  float* part;             // [grid][2][kPartFloats]: O [rows][128], m [rows], l [rows]
  int* tickets;            // [grid], zero between calls
  float *pre_o, *pre_m, *pre_l;   // shared form: O, m, l of each (sequence, q head)
  AttnFrom* from;                 // ... or where their pieces are, per (sequence, kv head)
  PageDiv div;
  int* err;
};

QD_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
QD_DEV uint32_t bf2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &v, 4);
  return u;
}
QD_DEV void bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }
QD_DEV void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// ---- tensor memory
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
QD_DEV void ld16(uint32_t taddr, float* v) {   // 16 columns, not waited for
  uint32_t* r = (uint32_t*)v;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
QD_DEV void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
QD_DEV void st16(uint32_t taddr, const uint32_t* r) {   // 16 columns, not waited for
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
QD_DEV void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// K and V tiles lie as groups of 8 keys of 2048 bytes, one 128-byte-swizzled atom for dims 0 ..
// 63 and one for the others, so that one copy brings whole rows of a page (with a copy for each
// half of the dims a prefix of 32768 tokens in 16-row pages took 2 us more of 68).
constexpr int kKeys8 = 2048, kHalf8 = 1024;
QD_DEV uint32_t kv_off(int key, int c) {   // of 16-byte piece c of a key's row
  return (uint32_t)((key >> 3) * kKeys8 + (c >> 3) * kHalf8 + (key & 7) * 128 + (((c & 7) ^ (key & 7)) << 4));
}
// K: K-major, the stride offset leads to the next 8 keys.
QD_DEV uint64_t desc_k(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(kKeys8 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// V as B of O += P V (A in tensor memory), [keys][dims], i.e. MN-major: the leading offset leads
// to the next 64 dims, the stride offset to the next 8 keys.
QD_DEV uint64_t desc_v(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(kHalf8 >> 4) << 16 | (uint64_t)(kKeys8 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
QD_DEV void tma_load_rows(void* dst, const CUtensorMap* map, int row, uint64_t* bar) {   // row: a multiple of 8
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(0), "r"(row >> 3), "r"(smem_u32(bar))
      : "memory");
}
// The products are issued by one lane of a warp whose lanes all walk the same way, so that
// descriptors stay in uniform registers; `lead` says which lane.
// Step kk of 16 keys, left out by lanes whose `steps` it is not below.
QD_DEV void mma_pv(int steps, int kk, uint32_t tmem_d, uint32_t tmem_a, uint64_t db, uint32_t accumulate) {
  constexpr uint32_t kIdesc = tc::idesc_m128(kD) | (1u << 16);   // B MN-major
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.gt.s32 q, %5, %6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(db), "r"(kIdesc), "r"(accumulate), "r"(steps), "r"(kk)
      : "memory");
}
QD_DEV void mma_qk(bool lead, uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t accumulate) {
  constexpr uint32_t kIdesc = tc::idesc_m128(kKeys);
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(da), "l"(db), "r"(kIdesc), "r"(accumulate), "r"((uint32_t)lead)
      : "memory");
}
QD_DEV void commit(bool lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"((uint32_t)lead)
      : "memory");
}

QD_DEV void tma_load_rows3(void* dst, const CUtensorMap* map, int half, int head, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(64 * half), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}
// 32 rows of a tile's results, dims 64 half .. + 63, from shared memory as Q lies there
QD_DEV void tma_store_rows(const CUtensorMap* map, int half, int head, int row, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"((uint64_t)map),
               "r"(64 * half), "r"(head), "r"(row), "r"(smem_u32(src))
               : "memory");
}
QD_DEV void cp16(uint32_t dst, const void* src, int bytes) {   // bytes 0: zeros, nothing read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// ---- the work of one segment
struct Seg {
  int row0, n;     // its packed rows (prompt tokens, or sequences)
  int off;         // prompt form: row j sees off + j + 1 keys
  int len;         // keys
  int tiles;       // row tiles per kv head; 0: no work
  int steps;       // row tiles that one CTA's run walks through (Work::team)
  bool bad;
};

// The units' split: CTA c of G takes per + (c < rem) of them.
struct Split {
  uint32_t per, rem;
  QD_DEV uint32_t first(uint32_t c) const { return c * per + min(c, rem); }
  QD_DEV int owner(uint32_t u) const {
    const uint32_t big = rem * (per + 1);
    return (int)(u < big ? u / (per + 1) : rem + (u - big) / per);
  }
};

template <bool PROMPT>
struct Work {
  int log_tpt;   // 2^log_tpt packed rows (tokens or sequences) per row tile
  // Shared form: a team of CTAs takes the same run of keys, each member another row tile of
  // every head, so that a K/V tile comes from HBM once for all row tiles at the same moment (as
  // separate runs the row tiles of 64 sequences read a 134 MB prefix twice: 258 MB from DRAM,
  // 68 us instead of 58). A segment with fewer row tiles leaves members idle.
  int team, member;   // (prompt form: 1, 0)

  QD_DEV int tpt() const { return 1 << log_tpt; }
  QD_DEV int step_tile(int t) const { return !PROMPT && team > 1 ? member : t; }
  QD_DEV Seg seg(const Params& p, int s) const {
    Seg a;
    a.row0 = p.cu[s];
    a.n = (int)((uint32_t)p.cu[s + 1] - (uint32_t)a.row0);   // (refused below where the ends make no sense)
    a.len = PROMPT ? p.seq_lens[s] : p.shared_lens[s];
    a.bad = a.n > 0 && (a.len < 0 || a.len > p.cap);
    a.off = a.len - a.n;
    a.tiles = a.bad || a.n <= 0 || (!PROMPT && a.len == 0) ? 0 : (a.n + tpt() - 1) >> log_tpt;
    a.steps = !PROMPT && team > 1 ? min(a.tiles, 1) : a.tiles;
    return a;
  }
  // keys that the last row of row tile t sees (prompt form), at least 0
  QD_DEV int seen(const Seg& a, int t) const {
    return PROMPT ? max(0, a.off + min((t + 1) << log_tpt, a.n)) : a.len;
  }
  QD_DEV int units(const Seg& a, int t) const { return max(1, (seen(a, t) + kKeys - 1) >> 7); }
  // sum over j < n of floor(j / 2^k)
  QD_DEV static long long floor_sum(long long n, int k) {
    const long long q = n >> k;
    return ((q * (q - 1)) >> 1 << k) + q * (n - (q << k));
  }
  // units of the row tiles before t (t <= tiles)
  QD_DEV long long before(const Seg& a, int t) const {
    if (!PROMPT) return (long long)t * units(a, 0);
    const int full = min(t, a.tiles - 1);
    long long sum = t == a.tiles && t > 0 ? units(a, t - 1) : 0;   // (prompt form: steps are tiles)
    if (full <= 0) return sum;
    // tile i < full ends at off + (i + 1) tpt keys: one unit up to 128, else the quotient
    const int one = a.off > kKeys ? 0 : min(full, (kKeys - a.off) >> log_tpt);
    sum += one;
    const long long c = (long long)a.off + ((long long)(one + 1) << log_tpt) + kKeys - 1;
    const long long rest = full - one;
    if (rest > 0) {
      sum += floor_sum((c >> log_tpt) + rest, 7 - log_tpt) - floor_sum(c >> log_tpt, 7 - log_tpt);   // tpt divides 128
    }
    return sum;
  }
};

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

// the largest magnitude, NaN if there is one
QD_DEV float max3_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A place in the work: row tile t of kv head g of segment s, from key tile k0 on.
struct Place {
  int s, g, t, k0;
  Seg a;
};

// not 0 if some of eight bf16 values is NaN or infinite: a half with all exponent bits set
// borrows into its top bit
QD_DEV uint32_t any_odd(const uint4& x) {
  auto odd = [](uint32_t w) { return ((w & 0x7f807f80u) ^ 0x7f807f80u) - 0x00010001u; };
  return (odd(x.x) | odd(x.y) | odd(x.z) | odd(x.w)) & 0x80008000u;
}

// Values of O that are not finite: what the row sees of V's own NaN and infinities in dims
// [d0, d0 + 64) of the keys [first, last) decides (the product of a weight's part and an
// infinity may have given NaN, or an entry was taken out of a masked tile: `taken`). The row's
// values are in memory by now, f32 or (half) bf16, 16-byte piece c at c ^ xr. The lanes have a row
// each (last 0: none) and go through the keys together, 32 at a time, until each value that is not
// finite is known to be NaN. A prompt of 8192 tokens with a NaN in its first value takes 1.1 ms, with
// an infinity there 2.2 (0.39 without).
__device__ __noinline__ void patch_rows(const Params& p, const int32_t* pt, int g, int first, int last, int d0,
                                        unsigned char* row, int xr, bool half, bool taken) {
  const int lane = threadIdx.x & 31;
  auto cell = [&](int k) {
    const int c = (d0 + k) >> (half ? 3 : 2);
    return row + ((c ^ xr) << 4) + (half ? ((d0 + k) & 7) * 2 : ((d0 + k) & 3) * 4);
  };
  unsigned long long nan = 0, pos = 0, neg = 0, open = 0;   // bit k: dim d0 + k; open: not settled
  if (last > 0) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k) {
      const float f = half ? __bfloat162float(*(const __nv_bfloat16*)cell(k)) : *(const float*)cell(k);
      if (taken || !(fabsf(f) < INFINITY)) open |= 1ull << k;
    }
  }
  const int end = __reduce_max_sync(0xffffffffu, last);
#pragma unroll 1
  for (int base = first; base < end; base += 32) {
    if (__all_sync(0xffffffffu, (open & ~nan) == 0)) break;
    int at = -1;   // the cache row of key base + lane
    if (base + lane < end) {
      const PagedSlot sl = paged_slot(pt, base + lane, p.page_size, p.div, p.n_pages);
      at = (sl.page * p.Hkv + g) * p.page_size + sl.slot;
    }
    // eight lanes read the dims of a key
    uint32_t odd = 0;   // bit j: this lane's piece of key base + 4 j + lane / 8
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = __shfl_sync(0xffffffffu, at, 4 * j + (lane >> 3));
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (r >= 0) x = *(const uint4*)(p.v_pages + (long long)r * kD + d0 + 8 * (lane & 7));
      odd |= (any_odd(x) ? 1u : 0u) << j;
    }
    uint32_t rows_odd = __reduce_or_sync(0xffffffffu, odd);
#pragma unroll 1
    for (; rows_odd; rows_odd &= rows_odd - 1) {
      const int j = __ffs(rows_odd) - 1;
#pragma unroll 1
      for (uint32_t who = __ballot_sync(0xffffffffu, (odd >> j) & 1); who; who &= who - 1) {
        const int src = __ffs(who) - 1, n = 4 * j + (src >> 3), dim = 8 * (src & 7);
        const int r = __shfl_sync(0xffffffffu, at, n);
        const unsigned short* v = (const unsigned short*)(p.v_pages + (long long)r * kD + d0 + dim);
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
          const unsigned h = v[e];
          if (base + n >= last || (h & 0x7f80u) != 0x7f80u) continue;   // (the lane's row does not see the key)
          const unsigned long long bit = 1ull << (dim + e);
          if (h & 0x7fu) nan |= bit;
          else if (h & 0x8000u) neg |= bit;
          else pos |= bit;
        }
        nan |= pos & neg;
        __syncwarp();
      }
    }
  }
#pragma unroll 1
  for (int k = 0; k < 64; ++k) {
    if (!(((nan | pos | neg) >> k) & 1)) continue;
    const float f = (nan >> k) & 1 ? NAN : (pos >> k) & 1 ? INFINITY : -INFINITY;
    if (half) *(__nv_bfloat16*)cell(k) = __float2bfloat16_rn(f);
    else *(float*)cell(k) = f;
  }
}

// piece k of the np that CTAs c0, c0 + 1, ... computed of one row tile
QD_DEV const float* piece_of(const Params& p, int c0, int k) {
  return p.part + ((size_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * kPartFloats;
}

// Four values of a joined row that some piece reached with a weight of 0 (below what 32 bits hold):
// the pieces' NaN and infinities count all the same.
template <typename T>
__device__ __noinline__ void patch_joined(const Params& p, int c0, int np, int row, T* out) {
  float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int k = 0; k < np; ++k) {
    const float4 v = __ldcg((const float4*)(piece_of(p, c0, k) + (size_t)row * kD) + (threadIdx.x & 31));
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!(fabsf(f[e]) < INFINITY)) u[e] += f[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (u[e] != 0.f) out[e] = (T)u[e];
}

template <typename T, int PARTS, bool PROMPT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
                     const __grid_constant__ Params p) {
  // bf16: two buffers of Q, so that S of the next piece follows this one's; f32: three parts of
  // one. What goes out is gathered in the place of the Q that it was made with.
  constexpr bool kEarlyQ = PARTS == 1;
  constexpr int kQ = kEarlyQ ? 2 : PARTS;     // slots of Q
  constexpr int kRing = 7 - kQ;
  constexpr int kCols = 64;                   // O columns per softmax thread
  constexpr bool kFresh = PARTS == 3;         // O of each tile alone in TMEM, summed in registers
  constexpr int kBufs = kFresh ? 2 : 3;       // buffers of S: how many tiles it runs ahead of P V
  constexpr int kRingV = kRing > 4 ? 3 : 2, kRingK = kRing - kRingV;   // K slots, then V slots
  static_assert(kRingK >= 2 && kRing <= kMaxSlots, "");
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* data = smem + kMisc;
  uint64_t* full = (uint64_t*)smem;      // [kRing] a K or V tile landed
  uint64_t* empty = full + kMaxSlots;    // [kRing] its products are done
  uint64_t* s_full = empty + kMaxSlots;  // [kBufs] S in buffer b
  uint64_t* p_full = s_full + kBufs;     // [kBufs] the weights in buffer b, O rescaled
  uint64_t* o_done = p_full + kBufs;     // [kBufs] the P V products of buffer b done
  uint64_t* o_free = o_done + kBufs;     // O of a piece has been read
  uint64_t* q_full = o_free + 1;         // [2] Q of a piece (f32: [0])
  uint64_t* drained = q_full + 2;        // [2] after a timeout: an issuer's products so far are done
  uint32_t* tslot = (uint32_t*)(drained + 2);
  int* s_abort = (int*)(tslot + 1);
  int* s_patch = s_abort + 1;            // [2] the last piece with NaN or infinities in a masked V tile
  int* s_last = s_patch + 2;             // [2]
  long long* s_find = (long long*)(smem + 256);   // [0] segment, [1] unit within it, [2] the split
  long long* s_scan = (long long*)(smem + 320);   // [warps] sums of the scan
  int* s_most = (int*)(smem + 448);               // [warps] most row tiles of a segment
  long long* s_saved = (long long*)(smem + 512);  // [warps]
  float* xm = (float*)(smem + 512);               // f32: [2][2][128] traded maxima and sums; bf16: [2][128] each

  // the warp's number from one lane: the roles' branches are then known to be taken by whole
  // warps, and the issuers' descriptors can stay in uniform registers
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  Work<PROMPT> W;
  W.log_tpt = 7 - p.log_rep;
  pdl_launch_dependents();
  if (smem_u32(smem) & 1023u) {   // the swizzled tiles rest on it (there is no static shared memory)
    if (tid == 0) set_error(p.err, QD_DEVERR_TIMEOUT);
    return;
  }

  // ---- this CTA's units
  W.team = 1;
  W.member = 0;
  uint32_t run_no;   // which run of units: one for each team
  {
    const int per = (p.n_seg + kThreads - 1) / kThreads;
    long long own = 0;
    int most = 0;
    long long saved = 0;   // tokens that sharing spares
    bool bad = false;
    for (int i = 0; i < per; ++i) {
      const int s = tid * per + i;
      if (s >= p.n_seg) break;
      // the ends themselves: their difference may pass 32 bits
      const int lo = p.cu[s], hi = p.cu[s + 1];
      bad = bad || lo < 0 || hi < lo || hi > p.n_rows;
      const Seg a = W.seg(p, s);
      if (a.bad && blockIdx.x == 0) set_error(p.err, QD_DEVERR_POS);
      most = max(most, a.tiles);
      if (a.tiles) saved += (long long)a.len * (a.n - 1);
    }
    if (tid == 0) *s_abort = 0;
    most = __reduce_max_sync(0xffffffffu, most);
    if constexpr (!PROMPT) {
#pragma unroll
      for (int o = 16; o; o >>= 1) saved += __shfl_xor_sync(0xffffffffu, saved, o);
    }
    if (lane == 0) {
      s_most[warp] = most;
      s_saved[warp] = saved;
    }
    const int any_bad = __syncthreads_or(bad);
    if (any_bad) {
      if (blockIdx.x == 0 && tid == 0) set_error(p.err, QD_DEVERR_POS);
      return;
    }
    if (!PROMPT) {
      saved = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        most = max(most, s_most[w]);
        saved += s_saved[w];
      }
      if (saved < p.share_min) return;   // the sequences read their prefixes for themselves
      if (most > 1 && most <= kMaxTeam) W.team = most;
      W.member = blockIdx.x % W.team;
    }
    for (int i = 0; i < per; ++i) {
      const int s = tid * per + i;
      if (s >= p.n_seg) break;
      const Seg a = W.seg(p, s);
      if (a.steps) own += W.before(a, a.steps) * p.Hkv;
    }
    long long v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    long long base = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base += s_scan[w];
      total += s_scan[w];
    }
    if (total >= (1LL << 31)) {
      if (blockIdx.x == 0 && tid == 0) set_error(p.err, QD_DEVERR_POS);
      return;
    }
    constexpr uint32_t kMin = PROMPT ? kMinUnits : 1;
    const uint32_t G = min(gridDim.x / W.team, ((uint32_t)total + kMin - 1) / kMin);
    run_no = blockIdx.x / W.team;
    if (run_no >= G) return;
    const Split sp = {(uint32_t)total / G, (uint32_t)total % G};
    const uint32_t u0 = sp.first(run_no);
    long long at = base + v - own;
    if (tid == 0) s_find[2] = (long long)sp.per << 32 | sp.rem;
    if (own > 0 && at <= u0 && u0 < at + own) {
      for (int i = 0; i < per; ++i) {
        const int s = tid * per + i;
        const Seg a = W.seg(p, s);
        const long long n = a.steps ? W.before(a, a.steps) * p.Hkv : 0;
        if (u0 < at + n) {
          s_find[0] = s;
          s_find[1] = u0 - at;
          break;
        }
        at += n;
      }
    }
  }
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&full[i], p.box ? 1 : 32);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kFresh ? kSoft : kSoft / 2);
      mbar_init(&o_done[i], 1);
    }
    s_patch[0] = s_patch[1] = 0;
    mbar_init(o_free, kSoft / 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], !kEarlyQ ? kSoft : p.q_sign > 0.f ? 4 : kSoft / 2);
      mbar_init(&drained[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) tc::alloc(tslot, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tb = *tslot;
  const uint32_t tS = tb, tO = tb + 128 * kBufs, tX = tb + 384;   // (tX: f32 only)
  const Split sp = {(uint32_t)(s_find[2] >> 32), (uint32_t)s_find[2]};
  const uint32_t u1 = sp.first(run_no + 1);
  uint32_t u = sp.first(run_no);

  // a wait of a whole warp, bounded by its polls (each returns after 2 us where nothing comes: half a
  // minute, which patch_rows needs for a billion keys); after a timeout anywhere in the CTA it returns
  // soon
  auto wait = [&](uint64_t* bar, uint32_t ph) {
    for (int i = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, ph)); ++i)
      if ((i & 1023) == 0 && (i == 1 << 24 || __any_sync(0xffffffffu, *(volatile int*)s_abort))) {
        if (i == 1 << 24) set_error(p.err, QD_DEVERR_TIMEOUT);
        *(volatile int*)s_abort = 1;
        break;
      }
  };

  // the place of unit u
  Place at;
  {
    at.s = (int)s_find[0];
    at.a = W.seg(p, at.s);
    const uint32_t head_units = (uint32_t)W.before(at.a, at.a.steps), v = (uint32_t)s_find[1];
    at.g = (int)(v / head_units);
    const uint32_t w = v % head_units;
    int lo = 0;
    for (int hi = at.a.steps; hi - lo > 1;) {   // the last row tile whose units start at or before w
      const int mid = (lo + hi) / 2;
      if (W.before(at.a, mid) <= w) lo = mid; else hi = mid;
    }
    at.t = lo;
    at.k0 = (int)(w - W.before(at.a, lo));
  }
  // the row tile after x's (there is one)
  auto advance = [&](Place& x) {
    x.k0 = 0;
    if (++x.t < x.a.steps) return;
    x.t = 0;
    if (++x.g < p.Hkv) return;
    x.g = 0;
    do {
      x.a = W.seg(p, ++x.s);
    } while (x.a.steps == 0);
  };
  // the place of unit x_u on, where this CTA has work: false if its run ends before
  auto settle = [&](Place& x, uint32_t& x_u) {
    for (;;) {
      if (x_u >= u1) return false;
      if (PROMPT || W.team == 1 || W.member < x.a.tiles) return true;
      x_u += min((uint32_t)(W.units(x.a, 0) - x.k0), u1 - x_u);   // another member's alone
      if (x_u >= u1) return false;
      advance(x);
    }
  };
  // A piece is the part of one row tile that this CTA computes. Each role walks the pieces for
  // itself, so the copies and products of one run into the next; counts that several roles
  // follow: tiles, trades, pieces.
  uint32_t tile = 0, piece_no = 0;
  [[maybe_unused]] uint32_t trades = 0;
  [[maybe_unused]] int begins = 0;   // bf16: the holder of the piece's first tile
  [[maybe_unused]] bool behind = false;
  [[maybe_unused]] int q_last = -1;   // bf16: the last piece whose Q this thread's copies brought
  int late = -1;
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
  Ring rk = {0, 0}, rb = {0, 0};   // K or V slots, buffers of S
  [[maybe_unused]] bool first = true;

  struct Piece {
    int g, t, k0, k1, nk, n;
    int first_row, packed;     // packed rows of the tile: the first, how many
    int seen_max, seen_min;    // keys past the first are nobody's, keys before the second everybody's
    const int32_t* pt;
  };
  auto piece_at = [&](const Place& x) {
    const Seg& a = x.a;
    Piece q;
    q.g = x.g;
    q.t = W.step_tile(x.t);
    q.k0 = x.k0;
    q.nk = W.units(a, W.step_tile(x.t));
    q.k1 = (int)min((uint32_t)q.nk, x.k0 + (u1 - u));
    q.n = q.k1 - x.k0;
    const int row = q.t << W.log_tpt;
    q.first_row = a.row0 + row;
    q.packed = min(W.tpt(), a.n - row);
    q.seen_max = W.seen(a, q.t);
    if (PROMPT) {
      q.seen_min = max(0, a.off + row + 1);
    } else {
      int m = a.len;
      for (int i = lane; i < q.packed; i += 32) {
        const int l = p.seq_lens[q.first_row + i];
        m = min(m, l < 0 || l > p.cap ? 0 : l);
      }
      q.seen_min = __reduce_min_sync(0xffffffffu, m);
    }
    q.pt = p.page_table + (size_t)(PROMPT ? x.s : a.row0) * p.max_pages;
    return q;
  };
  // the place after a piece of n units at x; false: none
  auto next_place = [&](Place& x, uint32_t& x_u, int n) {
    x_u += n;
    if (x_u >= u1) return false;
    advance(x);
    return settle(x, x_u);
  };
  const bool idle = !settle(at, u);

  if (idle) {
    // (a member of a team whose run has no row tile for it)
  } else if (warp >= kSoftWarps) {
    // the softmax warps take the registers that the others leave (256 x 200 + 128 x 104 of the
    // 384 x 168 of the launch)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    while (true) {
      const Piece pc = piece_at(at);
      const int g = pc.g, k0 = pc.k0, n = pc.n, seen_max = pc.seen_max, seen_min = pc.seen_min;
      const int32_t* pt = pc.pt;

      if (warp == kProducer || warp == kProducer + 1) {
        // ---- K or V tiles, a warp each, since a copy takes some 100 cycles to issue. A lane's cache
        // rows of a tile are looked up a tile ahead of their use. TMA: lane l, box l; asynchronous
        // copies: keys l, l + 32, ... (-1: past the keys)
        constexpr int kMine = 4;
        struct Look {
          int row[kMine];
        };
        int bad_page = 0;
        auto look = [&](int i) {
          Look x;
          const int key0 = (k0 + i) * kKeys;
#pragma unroll
          for (int j = 0; j < kMine; ++j) {
            const int key = p.box ? key0 + lane * p.box : key0 + 32 * j + lane;
            x.row[j] = -1;
            if (i < n && key < min(seen_max, key0 + kKeys) && (j == 0 || !p.box)) {
              const PagedSlot sl = paged_slot(pt, key, p.page_size, p.div, p.n_pages);
              if (!sl.ok) bad_page = 1;   // no branch on what is still being read
              x.row[j] = (sl.page * p.Hkv + g) * p.page_size + sl.slot;
            }
          }
          return x;
        };
        const bool is_v = warp != kProducer;
        const CUtensorMap* map = is_v ? &tmV : &tmK;
        const __nv_bfloat16* pages = is_v ? p.v_pages : p.k_pages;
        const uint32_t slots = is_v ? kRingV : kRingK, slot0 = is_v ? kRingK : 0;
        auto load = [&](const Look& x) {
          const uint32_t slot = slot0 + rk.slot;
          wait(&empty[slot], rk.ph ^ 1);   // (the first round's phase before the first is over)
          rk.step(slots);
          unsigned char* dst = data + (kQ + slot) * kSlot;
          if (p.box) {
            const bool go = !__any_sync(0xffffffffu, *(volatile int*)s_abort != 0);
            const unsigned boxes = __popc(__ballot_sync(0xffffffffu, x.row[0] >= 0));
            if (lane == 0) {
              if (go && boxes) mbar_arrive_expect_tx(&full[slot], boxes * p.box * 256);
              else mbar_arrive(&full[slot]);
            }
            __syncwarp();
            if (go && x.row[0] >= 0)
              tma_load_rows(dst + lane * p.box * 256, map, x.row[0], &full[slot]);
            __syncwarp();
          } else {
            // 16 lanes copy one key's 256 bytes
            const uint32_t d0 = smem_u32(dst);
#pragma unroll
            for (int j = 0; j < kMine; ++j)
#pragma unroll 2
              for (int i = 0; i < 32; i += 2) {
                const int r = i + (lane >> 4), c = lane & 15;
                const int row = __shfl_sync(0xffffffffu, x.row[j], r);
                cp16(d0 + kv_off(32 * j + r, c), pages + (long long)max(row, 0) * kD + c * 8, row < 0 ? 0 : 16);
              }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (late >= 0) {   // the entry before this one
              asm volatile("cp.async.wait_group 1;" ::: "memory");
              fence_proxy_async_smem();
              mbar_arrive(&full[late]);
            }
            late = (int)slot;
          }
        };
        Look now = {}, next = {};
#pragma unroll 1
        for (int i = -1; i < n; ++i) {
          now = next;
          next = look(i + 1);
          if (i >= 0) load(now);
        }
        if (late >= 0) {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          fence_proxy_async_smem();
          mbar_arrive(&full[late]);
          late = -1;
        }
        if (bad_page) set_error(p.err, QD_DEVERR_PAGE);
      } else if (warp == kIssueS) {
        // ---- S, up to kBufs tiles ahead of P V. The two products have a warp each, since what
        // a warp does between them is time the tensor cores idle: a product of 64 cycles takes
        // 58 to issue, and the waits and commits of a tile some 150 each (one warp for both: 2100
        // cycles a tile, whatever the softmax and the loads did). Slots are counted, not divided.
        const bool lead = lane == 0;
        const uint32_t qb = kEarlyQ ? piece_no & 1 : 0;
        const uint64_t dq = tc::desc_sw128(smem_u32(data) + qb * kSlot);
        const uint32_t ring0 = smem_u32(data) + kQ * kSlot;
        wait(&q_full[qb], (kEarlyQ ? piece_no >> 1 : piece_no) & 1);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          wait(&full[rk.slot], rk.ph);
          wait(&o_done[rb.slot], rb.ph ^ 1);   // the products that read the buffer (none in the first round)
          tc::fence_after();
          const uint64_t dk = desc_k(ring0 + rk.slot * kSlot);
          const uint32_t ts = tS + 128 * rb.slot;
#pragma unroll 1
          for (int part = PARTS - 1; part >= 0; --part) {   // small parts first
            const uint64_t da = dq + (uint64_t)(part * kSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              mma_qk(lead, ts, da + (kk >> 2) * (kChunk >> 4) + (kk & 3) * 2,
                     dk + (kk >> 2) * (kHalf8 >> 4) + (kk & 3) * 2, kk != 0 || part != PARTS - 1);
            }
          }
          commit(lead, &s_full[rb.slot]);
          commit(lead, &empty[rk.slot]);
          rk.step(kRingK);
          rb.step(kBufs);
        }
      } else {
        // ---- O += P V
        const bool lead = lane == 0;
        const uint32_t ring0 = smem_u32(data) + (kQ + kRingK) * kSlot;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const uint32_t slot = kRingK + rk.slot;
          wait(&full[slot], rk.ph);
          const int key0 = (k0 + i) * kKeys;
          int steps = kKeys / 16;   // of 16 keys that some row sees
          if (key0 + kKeys > seen_min) {
            // a V tile that some row must not see whole: NaN and infinities taken out, rows past
            // everybody's keys to zero up to the last step's end
            const int lo = max(0, seen_min - key0), hi = min(seen_max - key0, kKeys);
            steps = max(1, (hi + 15) >> 4);
            // lane: of key lane / 4 in a group of 8, 16-byte pieces lane & 3, + 4, + 8, + 12
            const int sub = lane >> 2, cc = lane & 3;
            unsigned char* v = data + (kQ + slot) * kSlot + sub * 128;
            const int o4[4] = {(cc ^ sub) << 4, ((cc + 4) ^ sub) << 4, kHalf8 + ((cc ^ sub) << 4),
                               kHalf8 + (((cc + 4) ^ sub) << 4)};
#pragma unroll 1
            for (int key = (lo & ~7) + sub; key < steps * 16; key += 8) {
              unsigned char* cell = v + (key >> 3) * kKeys8;
              if (key >= hi) {
#pragma unroll
                for (int j = 0; j < 4; ++j) *(uint4*)(cell + o4[j]) = make_uint4(0u, 0u, 0u, 0u);
              } else if (key >= lo) {
                uint4 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = *(const uint4*)(cell + o4[j]);
                if (!(any_odd(x[0]) | any_odd(x[1]) | any_odd(x[2]) | any_odd(x[3]))) continue;
                *(volatile int*)(s_patch + (piece_no & 1)) = (int)piece_no + 1;
#pragma unroll 1
                for (int j = 0; j < 32; ++j) {
                  const int c = ((cc + 4 * ((j >> 3) & 1)) ^ sub) << 4;
                  unsigned short* h = (unsigned short*)(cell + (j >> 4) * kHalf8 + c) + (j & 7);
                  if ((*h & 0x7f80u) == 0x7f80u) *h = 0;
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          // O of the piece before has been read by everybody (f32: p_full says so)
          if (!kFresh && i == 0 && piece_no) wait(o_free, (piece_no - 1) & 1);
          wait(&p_full[rb.slot], rb.ph);
          tc::fence_after();
          const uint64_t dv = desc_v(ring0 + rk.slot * kSlot);
          const bool first = kFresh || i == 0;
          const int go = lead ? steps : 0;
#pragma unroll 1
          for (int part = PARTS - 1; part >= 0; --part) {
            // 32 keys' weights over their own 32 scores
            const uint32_t ta = part < 2 ? tS + 128 * rb.slot + 16 * part : tX + 64 * rb.slot;
            const uint32_t t32 = part < 2 ? 32 : 16;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_pv(go, kk, tO, ta + t32 * (kk >> 1) + 8 * (kk & 1), dv + (uint64_t)(kk * 2 * kKeys8 >> 4),
                     kk != 0 || part != PARTS - 1 || !first);
          }
          commit(lead, &o_done[rb.slot]);
          commit(lead, &empty[slot]);
          rk.step(kRingV);
          rb.step(kBufs);
        }
      }
      tile += n;
      ++piece_no;
      if (!next_place(at, u, n)) break;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    while (true) {
      const Piece pc = piece_at(at);
      const Seg& a = at.a;
      const int g = pc.g, t = pc.t, k0 = pc.k0, k1 = pc.k1, nk = pc.nk, n = pc.n;
      const int first_row = pc.first_row, packed = pc.packed;
      const int32_t* pt = pc.pt;
      // ---- softmax: warps w and w + 4 hold the same rows (TMEM lanes)
      const int hf = warp >> 2, row = (warp & 3) * 32 + lane;
      const int rows = packed << p.log_rep;
      const bool valid = row < rows;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;

      // Q of the row tile at x into buffer qb; the copies are waited for in q_ready
      auto q_load = [&](const Place& x, [[maybe_unused]] uint32_t qb) {
        unsigned char* dst = data + (kEarlyQ ? qb * kSlot : 0);
        const T* q = (const T*)p.q + (long long)(x.a.row0 + (W.step_tile(x.t) << W.log_tpt)) * p.q_stride +
                     (long long)(x.g << p.log_rep) * kD;
        const int qrows = min(W.tpt(), x.a.n - (W.step_tile(x.t) << W.log_tpt)) << p.log_rep;
        if constexpr (PARTS == 1) {
          // warp w of the half that calls it copies rows 32 w .. as they are (rows of the box that
          // are not the tile's hold anything)
          if (p.q_sign > 0.f) {
            fence_proxy_async_smem();   // results went out from here
            __syncwarp();
            if (lane == 0 && *(volatile int*)s_abort == 0) {
              const int r0 = (warp & 3) * 32, head = x.g << p.log_rep;
              const int at_row = x.a.row0 + (W.step_tile(x.t) << W.log_tpt) + (r0 >> p.log_rep);
              mbar_arrive_expect_tx(&q_full[qb], 32 * 256);
              tma_load_rows3(dst + r0 * 128, &tmQ, 0, head, at_row, &q_full[qb]);
              tma_load_rows3(dst + kChunk + r0 * 128, &tmQ, 1, head, at_row, &q_full[qb]);
              q_last = (int)(piece_no + (first ? 0u : 1u));
            }
            __syncwarp();
            return;
          }
          // a scale that is not positive: through q_ready, two rows at a time
          constexpr int kPer = 32;
          const uint32_t d0 = smem_u32(dst);
          const int c = lane & 15;
#pragma unroll 4
          for (int i = 0; i < kPer; i += 2) {
            const int r = (warp & 3) * kPer + i + (lane >> 4), ok = r < qrows ? r : 0;
            cp16(d0 + (c >> 3) * kChunk + tc::sw128_off(r, c & 7),
                 q + (long long)(ok >> p.log_rep) * p.q_stride + (ok & (p.rep - 1)) * kD + 8 * c, r < qrows ? 16 : 0);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
          // warp w splits rows 16 w ..; lane: dims 4 lane .. + 3
#pragma unroll 1
          for (int i0 = 0; i0 < 16; i0 += 8) {
            float4 f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = warp * 16 + i0 + i;
              const T* from = q + (long long)(r >> p.log_rep) * p.q_stride + (r & (p.rep - 1)) * kD + 4 * lane;
              f[i] = r < qrows ? *(const float4*)from : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t o = (uint32_t)((lane >> 4) * kChunk + (lane & 1) * 8) +
                                 tc::sw128_off(warp * 16 + i0 + i, (lane & 15) >> 1);
              float x4[4] = {f[i].x * p.q_sign, f[i].y * p.q_sign, f[i].z * p.q_sign, f[i].w * p.q_sign};
#pragma unroll
              for (int part = 0; part < PARTS; ++part) {
                const uint32_t b0 = bf2(x4[0], x4[1]), b1 = bf2(x4[2], x4[3]);
                *(uint2*)(dst + part * kSlot + o) = make_uint2(b0, b1);
                x4[0] -= bf_lo(b0); x4[1] -= bf_hi(b0); x4[2] -= bf_lo(b1); x4[3] -= bf_hi(b1);
              }
            }
          }
        }
      };
      auto q_ready = [&]([[maybe_unused]] uint32_t qb) {
        [[maybe_unused]] unsigned char* dst = data + qb * kSlot;
        if constexpr (PARTS == 1) {
          if (p.q_sign > 0.f) return;
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          {   // a negative scale: this thread's pieces negated; none: zeros
            constexpr int kPer = 32;
            const int c = lane & 15;
            const uint32_t keep = p.q_sign < 0.f ? 0xffffffffu : 0u, flip = p.q_sign < 0.f ? 0x80008000u : 0u;
#pragma unroll 1
            for (int i = 0; i < kPer; i += 2) {
              const int r = (warp & 3) * kPer + i + (lane >> 4);
              uint4* cell = (uint4*)(dst + (c >> 3) * kChunk + tc::sw128_off(r, c & 7));
              const uint4 v = *cell;
              *cell = make_uint4((v.x & keep) ^ flip, (v.y & keep) ^ flip, (v.z & keep) ^ flip, (v.w & keep) ^ flip);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_full[kEarlyQ ? qb : 0]);
      };
      Place nx = at;
      uint32_t nx_u = u;
      if (first && (!kEarlyQ || hf == 0)) {
        q_load(at, 0);
        q_ready(0);
      }
      first = false;
      const bool more = next_place(nx, nx_u, n);
      const uint32_t nq = (piece_no + 1) & 1;   // the next piece's buffer of Q
      // bf16: the holder of the last tile of the piece before, who has seen that piece's last S and
      // written it out, fills its buffer again
      const bool loads = kEarlyQ && more && hf != begins;
      if (loads) q_load(nx, nq);

      int lim = 0;   // keys this row sees
      if (valid) {
        const int j = (t << W.log_tpt) + (row >> p.log_rep);
        if (PROMPT) {
          lim = max(0, a.off + j + 1);
        } else {
          const int l = p.seq_lens[a.row0 + j];
          lim = l < 0 || l > p.cap ? 0 : min(l, a.len);
        }
      }
      // what all valid rows of the warp see (rows that are not valid hold anything)
      const int warp_min = __reduce_min_sync(0xffffffffu, valid ? lim : INT32_MAX);
      const float c = p.scale_log2;
      float ms = -INFINITY, l = 0.f;
      [[maybe_unused]] float osum[kFresh ? kCols : 1];
      if constexpr (kFresh) {
#pragma unroll
        for (int k = 0; k < kCols; ++k) osum[k] = 0.f;
      }
      // 32 scores; those of keys that the row does not see become -inf
      auto mask = [&](float* sv, int key) {
        if (key + 32 > warp_min) {
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[e] = key + e < lim ? sv[e] : -INFINITY;
        }
      };
      auto top = [&](const float* sv, float m) {
        float m4[4] = {m, m, m, m};
#pragma unroll
        for (int e = 0; e < 32; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = max3(m4[k], sv[e + 2 * k], sv[e + 2 * k + 1]);
        return fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
      };
      // the weights of 32 scores (reference maximum nm2, negated), over the scores at ts, which
      // have been read; their sums into ps
      auto weights = [&](const float* s32, uint32_t ts, [[maybe_unused]] uint32_t tx, uint64_t nm2, uint64_t* ps) {
        const uint64_t c2 = pack2(c, c);
        uint32_t w0[16];
        [[maybe_unused]] uint32_t w1[PARTS == 3 ? 16 : 1], w2[PARTS == 3 ? 16 : 1];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          unpack2(fma2(pack2(s32[e], s32[e + 1]), c2, nm2), x, y);
          x = ex2(x);
          y = ex2(y);
          ps[(e >> 1) & 1] = add2(ps[(e >> 1) & 1], pack2(x, y));
          w0[e / 2] = bf2(x, y);
          if constexpr (PARTS == 3) {
            x -= bf_lo(w0[e / 2]);
            y -= bf_hi(w0[e / 2]);
            w1[e / 2] = bf2(x, y);
            w2[e / 2] = bf2(x - bf_lo(w1[e / 2]), y - bf_hi(w1[e / 2]));
          }
        }
        st16(ts, w0);
        if constexpr (PARTS == 3) {
          st16(ts + 16, w1);
          st16(tx, w2);
        }
      };
      const uint32_t ce = tile + n;
      if constexpr (kFresh) {
        // both holders of a row take 64 keys of every tile
        auto trade = [&](float v) -> float {   // with the other holder of the row
          const int par = trades & 1;
          ++trades;
          xm[(par * 2 + hf) * kRows + row] = v;
          bar_sync(2 + (warp & 3), 64);
          return xm[(par * 2 + (hf ^ 1)) * kRows + row];
        };
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const uint32_t ct = tile + i;
          const int b = (int)(ct & 1);
          const int key0 = (k0 + i) * kKeys + 64 * hf;
          const uint32_t ts = tS + 128 * b + lanes + 64 * hf;
          wait(&s_full[b], (ct >> 1) & 1);
          tc::fence_after();
          // the scores are read twice (for the maximum, for the weights), since registers for all
          // of them are not left beside O
          float mx = -INFINITY;
          float sv[32];
#pragma unroll 1
          for (int e = 0; e < kCols; e += 32) {
            ld32(ts + e, sv);
            wait_ld();
            mask(sv, key0 + e);
            mx = top(sv, mx);
          }
          mx = fmaxf(mx, trade(mx));
          mx = mx == -INFINITY ? mx : mx * c;
          const bool move = mx > ms + kMove;
          const float alpha = move ? ex2(ms - mx) : 1.f;   // 0 while ms is -inf
          if (move) {
            l *= alpha;
            ms = mx;
          }
          // a row that has seen nothing yet: weights 2^(-inf - 0)
          const float neg = ms == -INFINITY ? 0.f : -ms;
          const uint64_t nm2 = pack2(neg, neg);
          uint64_t ps[2] = {0, 0};   // pairs of sums, +0 each
#pragma unroll 1
          for (int e = 0; e < kCols; e += 32) {
            ld32(ts + e, sv);
            wait_ld();
            mask(sv, key0 + e);
            weights(sv, ts + e, tX + 64 * b + lanes + 32 * hf + e / 2, nm2, ps);
          }
          // O of the tile before, while S of the tile after is made; the next P V products,
          // which overwrite it, wait for this thread
          if (i > 0) {
            wait(&o_done[b ^ 1], ((ct - 1) >> 1) & 1);
            tc::fence_after();
            const bool any = __any_sync(0xffffffffu, move);
#pragma unroll
            for (int e = 0; e < kCols; e += 32) {
              ld32(tO + lanes + 64 * hf + e, sv);
              wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) osum[e + k] += sv[k];
            }
            if (any)
#pragma unroll
              for (int k = 0; k < kCols; ++k) osum[k] *= alpha;
          }
          float x, y;
          unpack2(add2(ps[0], ps[1]), x, y);
          l += x + y;
          wait_st();
          tc::fence_before();
          mbar_arrive(&p_full[b]);
        }
        wait(&o_done[(ce - 1) & 1], ((ce - 1) >> 1) & 1);
        const float l_other = trade(l);
        l = hf == 0 ? l + l_other : l_other + l;
      } else {
        // The two holders of a row take whole tiles in turn, so that the exponentials of one run
        // beside the loads and maxima of the other: the one that begins the first kSolo tiles, while
        // the other writes out the piece before, then they alternate. The reference maximum of O goes from one to
        // the other (xm), before either's exponentials; a holder's own sum of weights is for its
        // last reference (ms). The holder of the piece's last tile gets the other's sum and writes
        // the piece out, while the other begins the next one.
        const int pass_mine = kPassed + 4 * hf + (warp & 3), pass_other = kPassed + 4 * (hf ^ 1) + (warp & 3);
        float* ref_mine = xm + hf * kRows + row;
        const float* ref_other = xm + (hf ^ 1) * kRows + row;
        auto refer = [&](float m) {
          if (m != ms) {
            l *= ex2(ms - m);   // 0 while ms is -inf
            ms = m;
          }
        };
#pragma unroll 1
        for (int i = hf == begins ? 0 : kSolo; i < n; i += i < kSolo - 1 ? 1 : 2) {
          const uint32_t ct = tile + i, b = ct % kBufs;
          const int key0 = (k0 + i) * kKeys;
          const uint32_t ts = tS + 128 * b + lanes;
          // (whoever has not followed the kBufs tiles before this one waits for the reference first:
          // the barrier of S is then at this tile's phase)
          const bool early = i == kSolo || (i == 0 && behind);
          if (early) bar_sync(pass_other, 64);
          wait(&s_full[b], (ct / kBufs) & 1);
          tc::fence_after();
          if (key0 + kKeys > warp_min) {   // keys that some row of the warp does not see become -inf
#pragma unroll 1
            for (int e = max(0, (warp_min - key0) & ~31); e < kKeys; e += 32) {
              float x[32];
              ld32(ts + e, x);
              wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = key0 + e + k < lim ? x[k] : -INFINITY;
              st16(ts + e, (const uint32_t*)x);
              st16(ts + e + 16, (const uint32_t*)x + 16);
            }
            wait_st();
          }
          float sv[kKeys];
#pragma unroll
          for (int e = 0; e < kKeys; e += 32) ld32(ts + e, sv + e);
          wait_ld();
          float mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < kKeys; e += 32) mx = top(sv + e, mx);
          mx = mx == -INFINITY ? mx : mx * c;
          float old = -INFINITY;
          if (!early && (i > kSolo || (i == 0 && ct > 0))) bar_sync(pass_other, 64);
          if (i > 0) old = i < kSolo ? ms : *ref_other;
          const bool move = mx > old + kMove;
          const float now = move ? mx : old;
          if (i >= kSolo - 1 && i < n - 1) {   // (of the last tile: when the other's sum has been read)
            *ref_mine = now;
            bar_arrive(pass_mine, 64);
          }
          if (loads && i == kSolo) q_ready(nq);
          if (i > 0 && __any_sync(0xffffffffu, move)) {
            // (S of the tile before is there, so the products three tiles before it are done)
            wait(&o_done[(ct - 1) % kBufs], ((ct - 1) / kBufs) & 1);
            tc::fence_after();
            const float alpha = move ? ex2(old - now) : 1.f;   // 0 while the reference is -inf
#pragma unroll 1
            for (int e = 0; e < kD; e += 16) {
              float ov[16];
              ld16(tO + lanes + e, ov);
              wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) ov[k] *= alpha;
              st16(tO + lanes + e, (const uint32_t*)ov);
            }
            wait_st();
          }
          refer(now);
          // a row that has seen nothing yet: weights 2^(-inf - 0)
          const float neg = ms == -INFINITY ? 0.f : -ms;
          const uint64_t nm2 = pack2(neg, neg);
          uint64_t ps[2] = {0, 0};   // pairs of sums, +0 each
#pragma unroll
          for (int e = 0; e < kKeys; e += 32) weights(sv + e, ts + e, 0, nm2, ps);
          float x, y;
          unpack2(add2(ps[0], ps[1]), x, y);
          l += x + y;
          wait_st();
          tc::fence_before();
          mbar_arrive(&p_full[b]);
        }
        if (loads && n <= kSolo) q_ready(nq);   // (no tile of its own)
      }

      // ---- the piece's O, m, l: f32 by both holders of a row, 64 columns each; bf16 by the
      // holder of the last tile
      constexpr int kGroup = kFresh ? kSoft : kSoft / 2;   // threads that write a piece out
      const int gid = tid & (kGroup - 1), gbar = kFresh || hf ? 6 : 1;
      const bool whole = k0 == 0 && k1 == nk;
      const bool final_out = whole && PROMPT;      // else O as it is, with m and l
      float* part = p.part + ((size_t)blockIdx.x * 2 + (k0 == 0 ? 1 : 0)) * kPartFloats;
      // row r of the tile in [n_rows, Hq]: tile0 + out_row(r)
      const size_t tile0 = (size_t)first_row * p.Hq + (g << p.log_rep);
      auto out_row = [&](int r) { return (r >> p.log_rep) * p.Hq + (r & (p.rep - 1)); };   // (x 128: below 2^31)
      float* dst = !whole ? part : (PROMPT ? (float*)p.out : p.pre_o) + tile0 * kD;
      auto put_stats = [&] {
        float* m_at = whole ? p.pre_m + tile0 + out_row(row) : part + (size_t)kRows * kD + row;
        float* l_at = whole ? p.pre_l + tile0 + out_row(row) : part + (size_t)kRows * (kD + 1) + row;
        *m_at = ms;
        *l_at = l;
      };
      bool writes = true;
      if constexpr (kFresh) {
        tc::fence_after();
        const bool dead = *(volatile int*)s_abort != 0;
        const bool patch = *(volatile int*)(s_patch + (piece_no & 1)) == (int)piece_no + 1;
        const int col0 = 64 * hf;
        const float f = !final_out ? 1.f : lim == 0 ? 0.f : 1.0f / l;   // a row that sees no key gives 0
        // values go out by whole rows, through Q's place: 16-byte pieces, swizzled
        unsigned char* mine = data + row * 512;
        const int xr = row & 31;
        float z = 0.f;   // 0 unless a value is not finite
#pragma unroll
        for (int e = 0; e < kCols; e += 32) {
          float ov[32];
          ld32(tO + lanes + col0 + e, ov);
          wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            ov[k] += osum[e + k];
            z = fmaf(ov[k], 0.f, z);
            ov[k] *= f;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *(float4*)(mine + ((((col0 + e) / 4 + k) ^ xr) << 4)) =
                make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
        }
        const bool look = (patch || z != 0.f) && valid && !dead && l == l;
        if (__any_sync(0xffffffffu, look))
          patch_rows(p, pt, g, k0 * kKeys, look ? min(lim, k1 * kKeys) : 0, col0, mine, xr, false, patch);
        if (valid && !dead && !final_out && hf == 0) put_stats();
        // the rows that this warp's lanes and their other holders' wrote
        bar_sync(2 + (warp & 3), 64);
        const int r0 = (warp & 3) * 32 + hf * 16;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int r = r0 + i;
          const uint4 v = *(const uint4*)(data + r * 512 + ((lane ^ (r & 31)) << 4));
          if (r < rows && !dead) *(uint4*)(dst + (size_t)(whole ? out_row(r) : r) * kD + 4 * lane) = v;
        }
      } else {
        float* given = xm + 2 * kRows + row;   // reference and sum of the holder without the last tile
        // the holder of the last tile
        const int ends = n > kSolo && !((n - 1 - kSolo) & 1) ? begins ^ 1 : begins;
        behind = n >= kBufs && n <= kSolo;   // (of the other, who had no tile and begins the next piece)
        begins = ends ^ 1;
        writes = ends == hf;
        if (!writes) {
          given[0] = ms;
          given[kRows] = l;
          bar_arrive(2 + (warp & 3), 64);
        } else {
          bar_sync(2 + (warp & 3), 64);
          const float om = given[0], ol = given[kRows];
          if (more) bar_arrive(kPassed + 4 * hf + (warp & 3), 64);
          l = fmaf(ol, om == -INFINITY ? 1.f : ex2(om - ms), l);   // (its sum is 0 or NaN while it saw nothing)
          // (S of this tile is there, so the products three tiles before it are done)
          wait(&o_done[(ce - 1) % kBufs], ((ce - 1) / kBufs) & 1);
          tc::fence_after();
          const bool dead = *(volatile int*)s_abort != 0;
          const bool patch = *(volatile int*)(s_patch + (piece_no & 1)) == (int)piece_no + 1;
          const float f = !final_out ? 1.f : lim == 0 ? 0.f : 1.0f / l;   // a row that sees no key gives 0
          const bool put = valid && !dead;
          // bf16 results go out by whole rows, through the place of the same rows of Q (which this
          // warp fills again); partial values as they are
          unsigned char* old_q = data + (piece_no & 1) * kSlot;
          unsigned char* mine = final_out ? old_q + row * 128
                                          : (unsigned char*)(dst + (size_t)(whole ? out_row(put ? row : 0) : row) * kD);
          const int xr = row & 7;
          float z = 0.f;   // infinite or NaN if a value is
#pragma unroll 1
          for (int e = 0; e < kD; e += 32) {
            float ov[32];
            ld32(tO + lanes + e, ov);
            wait_ld();
            if (e == kD - 32) {
              tc::fence_before();
              mbar_arrive(o_free);
            }
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              z = max3_abs_nan(z, ov[k], ov[k + 1]);
              ov[k] *= f;
              ov[k + 1] *= f;
            }
            if (final_out) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *(uint4*)(mine + (e >> 6) * kChunk + ((((e & 32) / 8 + k) ^ xr) << 4)) =
                    make_uint4(bf2(ov[8 * k], ov[8 * k + 1]), bf2(ov[8 * k + 2], ov[8 * k + 3]),
                               bf2(ov[8 * k + 4], ov[8 * k + 5]), bf2(ov[8 * k + 6], ov[8 * k + 7]));
            } else if (put) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *(float4*)(mine + 4 * e + 16 * k) = make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
            }
          }
          const bool look = (patch || !(z < INFINITY)) && put && l == l;
          if (__any_sync(0xffffffffu, look)) {
#pragma unroll 1
            for (int d0 = 0; d0 < kD; d0 += 64)
              patch_rows(p, pt, g, k0 * kKeys, look ? min(lim, k1 * kKeys) : 0, d0,
                         mine + (final_out ? (d0 >> 6) * (kChunk - 128) : 0), final_out ? xr : 0, final_out, patch);
          }
          // a warp whose 32 rows are all there hands them to the copy engine (row by row they took
          // 2300 cycles of the warp, as long as a tile), the last rows of a prompt go one by one
          if (final_out && (warp & 3) * 32 + 32 <= rows && !__any_sync(0xffffffffu, dead)) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int r0 = (warp & 3) * 32, head = g << p.log_rep, at_row = first_row + (r0 >> p.log_rep);
              tma_store_rows(&tmO, 0, head, at_row, old_q + r0 * 128);
              tma_store_rows(&tmO, 1, head, at_row, old_q + kChunk + r0 * 128);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            __syncwarp();   // before the next Q
          } else if (final_out) {
            __syncwarp();
            __nv_bfloat16* out = (__nv_bfloat16*)p.out + tile0 * kD + 8 * (lane & 15);
#pragma unroll 4
            for (int i = 0; i < 32; i += 2) {
              const int c = lane & 15, tr = (warp & 3) * 32 + i + (lane >> 4);
              const uint4 v = *(const uint4*)(old_q + (c >> 3) * kChunk + tc::sw128_off(tr, c & 7));
              if (tr < rows && !dead) *(uint4*)(out + out_row(tr) * kD) = v;
            }
            __syncwarp();   // before the next Q
          }
          if (put && !final_out) put_stats();
        }
      }
      if (!PROMPT && writes && k0 == 0 && gid < packed) {   // the kernel that reads the rest joins the pieces
        AttnFrom* f = p.from + (size_t)(first_row + gid) * p.Hkv + g;
        f->first = blockIdx.x;
        f->pieces = whole ? 0 : sp.owner(u + nk - 1) - (int)run_no + 1;
        f->stride = W.team;
        f->row = gid << p.log_rep;
      }
      // ---- a prompt's row tile of several CTAs: the last of them joins the pieces in key order
      if (PROMPT && writes && !whole) {   // the same in all threads that write the piece out
        // where the tile's units lie: the CTAs of its first and last
        const int c0 = k0 == 0 ? (int)blockIdx.x : sp.owner(u - k0);
        const int c1 = k1 == nk ? (int)blockIdx.x : sp.owner(u - k0 + nk - 1);
        volatile int* last = s_last + (kFresh ? 0 : hf);
        bar_sync(gbar, kGroup);
        if (gid == 0) *last = !*(volatile int*)s_abort && atom_add_acq_rel_gpu(p.tickets + c0, 1) == c1 - c0;
        bar_sync(gbar, kGroup);
        if (*last) {
          const int np = c1 - c0 + 1;
          auto piece = [&](int k) { return piece_of(p, c0, k); };
          // A warp joins eight rows at a time: lane k has piece k's statistics (32 pieces at a time),
          // then four columns of O. Everything is read from L2 once, so what counts is how many
          // loads are under way.
          constexpr int kJoin = 8;
#pragma unroll 1
          for (int r0 = (gid >> 5) * kJoin; r0 < rows; r0 += kGroup / 32 * kJoin) {
            float M[kJoin], L[kJoin];
            float4 acc[kJoin];
            uint32_t zero = 0;   // bit j: a weight of row j was 0
#pragma unroll
            for (int j = 0; j < kJoin; ++j) {
              M[j] = -INFINITY;
              L[j] = 0.f;
              acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll 1
            for (int b0 = 0; b0 < np; b0 += 32) {
              const int nb = min(32, np - b0);
              float m4[kJoin], l4[kJoin];
              const float* st = piece(b0 + min(lane, nb - 1)) + (size_t)kRows * kD + r0;
#pragma unroll
              for (int j = 0; j < kJoin; ++j) {
                const bool has = lane < nb && r0 + j < rows;
                m4[j] = has ? __ldcg(st + j) : -INFINITY;
                l4[j] = has ? __ldcg(st + kRows + j) : 0.f;
              }
#pragma unroll
              for (int j = 0; j < kJoin; ++j) {
                float top = m4[j];
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = fmaxf(top, M[j]);
                const float keep = M[j] == -INFINITY ? 1.f : ex2(M[j] - top);   // (O and L are 0 or NaN there)
                // pieces that saw nothing: weight 1 for a sum and an O of 0 (or NaN); a weight of 0 (below
                // what 32 bits hold) keeps a NaN
                m4[j] = m4[j] == -INFINITY ? 1.f : ex2(m4[j] - top);
                zero |= (keep == 0.f || m4[j] == 0.f ? 1u : 0u) << j;
                float sum = m4[j] * l4[j];
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                L[j] = L[j] * keep + sum;
                if (keep != 1.f) {
                  acc[j].x *= keep;
                  acc[j].y *= keep;
                  acc[j].z *= keep;
                  acc[j].w *= keep;
                }
                M[j] = top;
              }
#pragma unroll 1
              for (int k = 0; k < nb; ++k) {
                const float4* src = (const float4*)(piece(b0 + k) + (size_t)r0 * kD) + lane;
                float4 v[kJoin];
#pragma unroll
                for (int j = 0; j < kJoin; ++j)
                  if (r0 + j < rows) v[j] = __ldcg(src + j * (kD / 4));
#pragma unroll
                for (int j = 0; j < kJoin; ++j) {
                  const float x = __shfl_sync(0xffffffffu, m4[j], k);
                  if (r0 + j < rows) {
                    acc[j].x = fmaf(x, v[j].x, acc[j].x);
                    acc[j].y = fmaf(x, v[j].y, acc[j].y);
                    acc[j].z = fmaf(x, v[j].z, acc[j].z);
                    acc[j].w = fmaf(x, v[j].w, acc[j].w);
                  }
                }
              }
            }
#pragma unroll
            for (int j = 0; j < kJoin; ++j) {
              if (r0 + j >= rows) break;
              const size_t o = (tile0 + out_row(r0 + j)) * kD + 4 * lane;
              const bool sees = a.off + (t << W.log_tpt) + ((r0 + j) >> p.log_rep) >= 0;   // (else 0)
              const float iv = sees ? 1.0f / L[j] : 0.f;
              if constexpr (PARTS == 1)
                *(uint2*)((__nv_bfloat16*)p.out + o) =
                    make_uint2(bf2(acc[j].x * iv, acc[j].y * iv), bf2(acc[j].z * iv, acc[j].w * iv));
              else
                *(float4*)((float*)p.out + o) = make_float4(acc[j].x * iv, acc[j].y * iv, acc[j].z * iv, acc[j].w * iv);
              if (L[j] != L[j]) zero &= ~(1u << j);
            }
            zero = __reduce_or_sync(0xffffffffu, zero);
#pragma unroll 1
            for (int j = 0; zero >> j && r0 + j < rows; ++j)
              if ((zero >> j) & 1) patch_joined(p, c0, np, r0 + j, (T*)p.out + (tile0 + out_row(r0 + j)) * kD + 4 * lane);
          }
          bar_sync(gbar, kGroup);
          if (gid == 0) p.tickets[c0] = 0;
        }
      }
      tc::fence_before();
      if (!kEarlyQ && more) {
        bar_sync(6, kSoft);   // everybody is done with Q's place
        q_load(nx, 0);
        q_ready(0);
      }
      tile += n;
      ++piece_no;
      if (!more) break;
      at = nx;
      u = nx_u;
    }
  }
  __syncwarp();
  if ((warp == kProducer || warp == kProducer + 1) && *(volatile int*)s_abort && p.box && lane == 0) {
    // a timeout: the copies that are still under way land before the CTA leaves (bounded)
    const uint32_t slots = warp != kProducer ? kRingV : kRingK, slot0 = warp != kProducer ? kRingK : 0;
    for (uint32_t i = 0; i < slots; ++i) {
      const bool again = i < rk.slot;   // filled in this round of the ring
      if (again || tile >= slots) mbar_wait_limit(&full[slot0 + i], again ? rk.ph : rk.ph ^ 1, p.err, 10000000ull);
    }
  }
  if (q_last >= 0 && *(volatile int*)s_abort)
    mbar_wait_limit(&q_full[q_last & 1], (q_last >> 1) & 1, p.err, 10000000ull);
  if ((warp == kIssueS || warp == kIssueO) && *(volatile int*)s_abort) {   // ... and the products (bounded)
    commit(lane == 0, &drained[warp == kIssueO]);
    mbar_wait_limit(&drained[warp == kIssueO], 0, p.err, 10000000ull);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::dealloc(tb, 512);
  }
}

int grid_ctas() { return std::min(dev_info().sm_count, kMaxGrid); }

template <typename T, int PARTS, bool PROMPT>
cudaError_t launch(const Params& p, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                   const CUtensorMap& to, const Launch& L) {
  cudaError_t e = allow_smem<attn_rows_kernel<T, PARTS, PROMPT>>(kSmem);
  if (e != cudaSuccess) return e;
  return launch_ex(attn_rows_kernel<T, PARTS, PROMPT>, dim3(grid_ctas()), dim3(kThreads), kSmem, L, tk, tv, tq, to,
                   p);
}

// Workspace: the head with the tickets, then the partials.
static_assert(kAttnRowTickets + kMaxGrid * 4 <= kAttnSeqTickets, "");

template <bool PROMPT>
cudaError_t run(const AttnRowsArgs& a, float* pre_o, AttnFrom* from, const Launch& L) {
  Params p = {};
  p.q = a.q; p.q_stride = a.q_stride;
  p.k_pages = (const __nv_bfloat16*)a.k_pages; p.v_pages = (const __nv_bfloat16*)a.v_pages;
  p.page_table = a.page_table; p.cu = a.cu; p.seq_lens = a.seq_lens; p.shared_lens = a.shared_lens;
  p.n_seg = a.n_seg; p.n_rows = a.n_rows; p.Hq = a.Hq; p.Hkv = a.Hkv; p.rep = a.Hq / a.Hkv;
  while ((1 << p.log_rep) < p.rep) ++p.log_rep;
  p.page_size = a.page_size; p.max_pages = a.max_pages; p.n_pages = a.n_pages;
  p.cap = (long long)a.max_pages * a.page_size;
  // q takes the sign; a scale of 0 makes q 0, so that masked scores stay -inf times something
  p.scale_log2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
  p.q_sign = a.scale < 0.f ? -1.f : a.scale == 0.f ? 0.f : 1.f;
  p.out = a.out;
  p.tickets = (int*)((unsigned char*)a.workspace + kAttnRowTickets);
  p.part = (float*)((unsigned char*)a.workspace + kAttnHeadBytes);
  p.pre_o = pre_o;
  p.from = from;
  p.div = make_page_div(a.page_size);
  p.share_min = a.share_min;
  p.pre_m = pre_o ? pre_o + (size_t)a.n_rows * a.Hq * kD : nullptr;
  p.pre_l = pre_o ? p.pre_m + (size_t)a.n_rows * a.Hq : nullptr;
  p.err = L.err;
  // boxes of whole 16-row pieces of a page; other page sizes by 16-byte asynchronous copies
  alignas(64) CUtensorMap tk, tv, tq, to;
  memset(&tk, 0, sizeof(tk));
  memset(&tv, 0, sizeof(tv));
  memset(&tq, 0, sizeof(tq));
  memset(&to, 0, sizeof(to));
  if (!a.q_f32) {
    cudaError_t e = encode_tmap_bf16_heads(&tq, a.q, a.n_rows, a.q_stride, a.Hq, p.rep, 32 / p.rep);
    if (e == cudaSuccess && PROMPT)
      e = encode_tmap_bf16_heads(&to, a.out, a.n_rows, (int64_t)a.Hq * kD, a.Hq, p.rep, 32 / p.rep);
    if (e != cudaSuccess) return e;
  }
  if (a.page_size % 16 == 0) {
    p.box = 16;
    while (p.box < kKeys && a.page_size % (2 * p.box) == 0) p.box *= 2;
    const uint64_t rows = (uint64_t)a.n_pages * a.Hkv * a.page_size;
    cudaError_t e = encode_tmap_bf16_rows128(&tk, a.k_pages, rows, p.box);
    if (e == cudaSuccess) e = encode_tmap_bf16_rows128(&tv, a.v_pages, rows, p.box);
    if (e != cudaSuccess) return e;
  }
  return a.q_f32 ? launch<float, 3, PROMPT>(p, tk, tv, tq, to, L)
                 : launch<__nv_bfloat16, 1, PROMPT>(p, tk, tv, tq, to, L);
}

}  // namespace

size_t attn_rows_workspace_bytes() { return kAttnHeadBytes + (size_t)grid_ctas() * 2 * kPartFloats * 4; }

cudaError_t launch_attn_prompt(const AttnRowsArgs& a, const Launch& L) { return run<true>(a, nullptr, nullptr, L); }

cudaError_t launch_attn_prefix(const AttnRowsArgs& a, float* pre, AttnFrom* from, AttnPieces* pieces,
                               const Launch& L) {
  *pieces = {(const float*)((const unsigned char*)a.workspace + kAttnHeadBytes), grid_ctas()};
  return run<false>(a, pre, from, L);
}

}  // namespace qd
