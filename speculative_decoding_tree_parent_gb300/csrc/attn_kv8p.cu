// Tree-verify attention over an 8-bit paged cache with a scale per (page, KV head), on the
// 5th-generation tensor cores.
//
// Row (node i of sequence b, query head h, g = h / G, G = hq / hkv), over the prefix keys j
// (slot j's page and row) and the tree nodes its mask bits name:
//   x_j = sm_scale * q . k_j,   out = sum_j e^(x_j) v_j / sum_j e^(x_j),
//   prefix: k_j = k_code_j * ks[page_j][g], v_j = v_code_j * vs[page_j][g];  tree: bf16 rows.
//
// K's codes go to the tensor cores as they are (kind::f8f6f4), so QK needs no widened copy of
// K. Its other operand has to be E4M3 too: a row of q, scaled by a power of two to a largest
// element in [2^7, 2^8), is the sum of two E4M3 values, hi = e4m3(q) and lo = e4m3(q - hi): a
// bf16 has 8 significant bits, an E4M3 4, so the sum is exact for elements within 2^9 of the
// row's largest (and off by at most 2^-17 of it below). Two products of twice bf16's rate cost
// what one bf16 product does.
// P V runs in fp16: E4M3 is a subset of fp16, and P needs the range (a key that takes nearly
// all of a row's weight leaves the others' weights 2^20 and more below it, where two E4M3
// terms have run out of exponents). Four warps widen V's codes, one conversion for two.
// The page's scales stay outside the products: ks multiplies the score's fp32 factor, and vs
// enters the exponent, P_j = 2^(x_j log2 e + log2 vs_j - M + 11), where M follows the largest
// x log2 e + log2 vs (P stays below 2^15, and full precision reaches 2^25 below the largest);
// the row sum adds P_j / vs_j per page.
//
// A CTA = (key split, one or two row tiles, sequence x KV head). A row tile is 128 rows: 128 / G
// nodes (rounded down) of G heads each. K/V come in blocks: the split's prefix blocks (64 keys, 4
// pages, TMA page by page), then its tree blocks (32 nodes, bf16). Two slots, each with its own MMA
// issuer, four softmax warps (one row per thread) and TMEM (S of its even and of its odd blocks, P
// over the S it comes from, O): of two tiles a slot has one, and K, V and V's conversion serve both;
// of one tile the slots take the blocks in turn and their sums are joined at the end. QK of a slot's
// next block runs under the softmax of this one.
// q's codes (hi and lo) stand in shared memory, later its bf16 rows for the tree.
// Warps (512 threads, 128 registers): 0 and 15 TMA producers (K, V's codes), 1 and 10 MMA issuers,
// 2-5 and 6-9 softmax, 11-14 V's converters. Every wait is bounded.
// Splits write O / l in fp32 and the log2-sum-exp, joined by a second kernel.
//
// Bound (one GB300): not HBM and not the tensor cores but a slot's chain (S, softmax, P, each handed
// on through a barrier) and the issue of its instructions: about 1700 cycles for a block of 64 keys on
// the long case below, of which the softmax takes the most; two slots go at a time. 128 sequences of one token over
// 543,000 keys (1.1 GB): 275 us, 4.1 TB/s; 32 trees of 64 nodes over 512 .. 8192 keys: 156 us,
// 0.96 of 1.93 PFLOP/s; 8 x 128 nodes over 32768 keys: 923 us, 1.06 PFLOP/s.
// What was measured beside it (when it took 293, 164 and 984 us): one tile a CTA, its blocks of 128
// keys handed to the slots in turn, q in TMEM 300, 246, 1010; two tiles in 128-key blocks with one S
// each 330, 199, 1260; one producer for K and V 404, 161, 973 (one tile's blocks wait for its copies);
// MMAs issued by a whole warp under a predicate instead of one thread 293, 175, 1048. Loops unrolled
// over 128 keys ran at the rate at which their code is fetched, a fifth slower.
#include "attn_common.cuh"
#include "tc_host.cuh"
#include "tc_math.cuh"

namespace specv {
namespace kv8p {

constexpr int kRows = 128;      // rows of a tile
constexpr int kKeys = 64;       // keys of a prefix block
constexpr int kPages = kKeys / 16;
constexpr int kTreeKeys = 32;   // nodes of a tree block (as many bytes as a prefix block)
constexpr int kD = 128;
constexpr int kThreads = 512;
constexpr int kSoft0 = 2, kMma1 = 10, kVProd = 15;  // first softmax warp, slot 1's MMA issuer, V's producer
// stages: K, V codes, V in 16 bits; K's and V's even, so that a slot that takes every other block
// finds its blocks in stages of its own and sees each phase of their barriers
constexpr int kStK = 8, kStC = 6, kStV = 2;
static_assert(kStK % 2 == 0 && kStV % 2 == 0, "a stage has to belong to one slot");
constexpr uint32_t kSlab = 128 * 128;        // 16 KB: half a tile of q, a stage of V
constexpr uint32_t kStage = kKeys * 128;      // 8 KB: a stage of K or of V's codes
constexpr uint32_t kVSlab = kKeys * 128;     // half a stage of V: 64 rows of 64 elements
constexpr uint32_t kTreeSlab = kTreeKeys * 128;
// q: of two tiles the hi and lo codes, then the tree's bf16 rows; of one codes and rows
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 4 * kSlab;
constexpr uint32_t kOffC = kOffK + kStK * kStage;
constexpr uint32_t kOffV = kOffC + kStC * kStage;
static_assert(2 * kTreeSlab == kStage, "a tree block fills a stage");
constexpr uint32_t kOffBar = kOffV + kStV * kSlab;
constexpr int kScales = 32;                  // blocks whose page scales are kept: four groups of eight
constexpr uint32_t kOffScale = kOffBar + 640;
constexpr uint32_t kOffJoin = kOffScale + kScales * kPages * 16;            // float2 [slot][row]: M, sum
constexpr uint32_t kSmem = kOffJoin + 2 * kRows * 8 + 1024;   // + alignment slack
static_assert(kSmem <= 232448, "shared memory over the per-CTA limit");
constexpr uint32_t kTmemCols = 512;          // a tile: S (and P) of even and of odd blocks, O
constexpr int kLptMax = 1024;                // sequences that are ranked by length
constexpr float kShift = 11.f;               // log2 of the largest P when M is set
constexpr float kGrow = 4.f;                 // growth of the largest score that M may lag behind
constexpr uint32_t kIdQK = tc::idesc_e4m3(kRows, kKeys);
constexpr uint32_t kIdPV = tc::idesc_f16(kRows, kD, 1);
constexpr uint32_t kIdTreeQK = tc::idesc_bf16(kRows, kTreeKeys, 0);
constexpr uint32_t kIdTreePV = tc::idesc_bf16(kRows, kD, 1);
constexpr int kMaxSplits = 32;
constexpr int kMaxTreeWords = kMaxTreeNodes / 64;

struct Params {
  const __nv_bfloat16* q;
  const float2* kv_scale;
  const int32_t* page_table;
  int max_pages, num_pages;
  int max_len;  // longest prefix that the row of pages and the caller's bound allow
  const int32_t* prefix_len;
  const uint64_t* mask;
  int mask_words, max_nodes;
  const int32_t* qo;
  int hq, hkv, G, npt;  // npt: nodes of a row tile
  int splits, mtiles, batch, lpt;
  int per_cta;  // row tiles of a CTA: 1 or 2
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float4* part_o;   // [tile][split][32 chunks of 4 columns][128 rows], O / l
  float* part_lse;  // [tile][split][128 rows] log2-sum-exp (-inf: no keys)
  int32_t* status;
  int early;
};

struct Bars {
  // one arrival a phase
  uint64_t k_full[kStK], c_full[kStC], s_full[2][2], pv_done[2][2], fin[2], sc_full[2];
  // four: a warpgroup's warps
  uint64_t q16[2], q8[2], c_empty[kStC], v_full[kStV], p_full[2][2];  // q in bf16 / as codes
  // one a tile
  uint64_t k_empty[kStK], v_empty[kStV];
  uint64_t bad[kMaxTreeWords];  // tree nodes whose V row holds an infinity or NaN
  uint32_t tmem;
  int abort;
};
constexpr int kBar1 = kStK + kStC + 12, kBar4 = kBar1 + 8 + kStC + kStV, kBarAll = kBar4 + kStK + kStV;
static_assert(sizeof(Bars) <= 640, "barrier block over its reserved bytes");

// The blocks of one key split: units are the prefix pages, then the tree blocks (2 each); a
// split takes a contiguous run of units, a tree block goes to the split of its first unit.
struct Split {
  int pg_lo, pg_hi;   // prefix pages
  int np;             // prefix blocks
  int tb_lo;          // first tree block
  int nb;             // blocks in all
};
__device__ __forceinline__ Split split_of(int P, int N, int splits, int s) {
  const int pages = (P + 15) >> 4, nt = (N + kTreeKeys - 1) / kTreeKeys;
  const long units = pages + 2L * nt;
  const int lo = (int)(s * units / splits), hi = (int)((s + 1) * units / splits);
  Split r;
  r.pg_lo = min(lo, pages);
  r.pg_hi = min(hi, pages);
  r.np = (r.pg_hi - r.pg_lo + kPages - 1) / kPages;
  r.tb_lo = lo <= pages ? 0 : (lo - pages + 1) >> 1;
  const int tb_hi = hi <= pages ? 0 : min(nt, (hi - pages + 1) >> 1);
  r.nb = r.np + max(0, tb_hi - r.tb_lo);
  return r;
}

__device__ __forceinline__ uint16_t e4m3x2(float x0, float x1) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x1), "f"(x0));
  return c;
}
__device__ __forceinline__ uint32_t half2_of(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The whole warp waits for a phase, bounded: the hardware holds a try for microseconds before it
// says no, so kTries of them are a second or so. (One lane waiting, with its answer shuffled to the
// others, cost about 1000 cycles a wait to bring the warp back together. The first try stands by
// itself and the others out of line: a loop around it cost a tenth of the kernel's time.)
constexpr int kTries = 1 << 18;
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int i = 0; i < kTries && *abort == 0; ++i) {
    const bool ok = tc::mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort) {
  const bool ok = tc::mbar_try_wait(bar, parity);
  return __builtin_expect(__all_sync(0xffffffffu, ok), 1) || wait_more(bar, parity, abort);
}

// The same for one thread. (Here the further tries in line are the faster form.)
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (tc::mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < kTries && *abort == 0; ++i)
    if (tc::mbar_try_wait(bar, parity)) return true;
  *abort = 1;
  return false;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e != 0;
}

// One arrival for a warp whose lanes have all done their part.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  tc::mbar_arrive_if((threadIdx.x & 31) == 0, bar);
}

// The softmax warps of both slots.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// 16-byte chunk c of row r of a 128-byte-row slab, in the 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// A row of q (bf16) to shared memory as hi and lo E4M3 codes (a slab of 128-byte rows each);
// returns the factor that the codes have to be multiplied by. (A row with an infinity or NaN gets
// a NaN code.) The row is read twice, the second time from the cache: short loops, as this runs
// once a CTA and its code comes from afar.
__device__ __forceinline__ float split_row(const uint4* src, bool valid, uint8_t* qs, int row) {
  uint32_t m = 0;  // the largest magnitude, of the low and of the high halves
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint4 v = valid ? ld(src + k) : make_uint4(0, 0, 0, 0);
    const uint32_t a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu);
    const uint32_t b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
    m = __vmaxu2(m, __vmaxu2(a, b));
  }
  const uint32_t top = max(m & 0xFFFFu, m >> 16);
  const int e = max((int)(top >> 7), 1);       // exponent field of the largest element
  // up * 2^(e - 134) = 1: q * up has its largest element in [2^7, 2^8). Both factors are made
  // of two powers of two, as one may leave fp32's range.
  const int sh = 134 - e;                      // in [-121, 133]
  const float up0 = __uint_as_float((uint32_t)(127 + sh / 2) << 23);
  const float up1 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
#pragma unroll 1
  for (int h = 0; h < 8; ++h) {  // 16 elements, a 16-byte chunk of each
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = valid ? ld(src + 2 * h + i) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t a = w[2 * k], b = w[2 * k + 1];
        const float x0 = __uint_as_float(a << 16) * up0 * up1, x1 = __uint_as_float(a & 0xFFFF0000u) * up0 * up1;
        const float x2 = __uint_as_float(b << 16) * up0 * up1, x3 = __uint_as_float(b & 0xFFFF0000u) * up0 * up1;
        const uint16_t h01 = e4m3x2(x0, x1), h23 = e4m3x2(x2, x3);
        const uint32_t f01 = half2_of(h01), f23 = half2_of(h23);
        const float2 g01 = __half22float2(*reinterpret_cast<const __half2*>(&f01));
        const float2 g23 = __half22float2(*reinterpret_cast<const __half2*>(&f23));
        hi[2 * i + k] = h01 | ((uint32_t)h23 << 16);
        lo[2 * i + k] = e4m3x2(x0 - g01.x, x1 - g01.y) | ((uint32_t)e4m3x2(x2 - g23.x, x3 - g23.y) << 16);
      }
    }
    if (h == 0 && top >= 0x7F80u) hi[0] |= 0x7Fu;
    *reinterpret_cast<uint4*>(qs + swz(row, h)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(qs + kSlab + swz(row, h)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  return __uint_as_float((uint32_t)(127 - sh / 2) << 23) * __uint_as_float((uint32_t)(127 - (sh - sh / 2)) << 23);
}

// The factor from a raw score to log2 units, for a row's and a page's scale; kept above 0 so
// that a key past the prefix stays at -inf (a score is 0 there all the same).
__device__ __forceinline__ float factor(float row, float ks) { return fmaxf(row * ks, 1e-37f); }

// The sequence with the n-th most keys (ties: the lower first), from the lengths: CTAs start in
// the order of their index, so the longest are begun first and the last wave holds the shortest.
__device__ __forceinline__ int nth_longest(const Params& p, int n, int* keys) {
#pragma unroll 1
  for (int t = threadIdx.x; t < p.batch; t += kThreads)
    keys[t] = ld(p.prefix_len + t) + (ld(p.qo + t + 1) - ld(p.qo + t));
  int* found = keys + kLptMax;
  __syncthreads();
#pragma unroll 1
  for (int t = threadIdx.x; t < p.batch; t += kThreads) {
    const int k = keys[t];
    int r = 0;
#pragma unroll 4
    for (int u = 0; u < p.batch; ++u) r += keys[u] > k || (keys[u] == k && u < t) ? 1 : 0;
    if (r == n) *found = t;  // ranks are distinct: exactly one thread writes
  }
  __syncthreads();
  const int b = *found;
  __syncthreads();  // (the scratch becomes the K ring)
  return b;
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_kv8p_kernel(const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                     const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                     const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + kOffBar);
  const uint32_t sb = tc::smem_u32(smem);
  const int split = blockIdx.x, bg = blockIdx.z;
  pdl_trigger();  // the split merge waits for this grid to end
  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&tm_kp);
    tc::prefetch_tmap(&tm_vp);
    tc::prefetch_tmap(&tm_kt);
    tc::prefetch_tmap(&tm_vt);
  }
  if (!p.early) pdl_wait();
  int b = bg / p.hkv;
  const int g = bg - b * p.hkv;
  if (p.lpt) b = nth_longest(p, b, reinterpret_cast<int*>(smem));
  const int base = ld(p.qo + b), N = ld(p.qo + b + 1) - base, P = ld(p.prefix_len + b);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
  const int node0 = p.per_cta * blockIdx.y * p.npt;
  if (node0 >= N) {
    if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0) pdl_wait();  // (the grid must not end before its predecessor)
    return;
  }
  // (the grid and the workspace hold max_nodes nodes a sequence, not the mask row's multiple of 64)
  if (N > p.max_nodes || P < 0 || P > p.max_len) {
    if (threadIdx.x == 0 && split == 0) {
      report_waited(p.status, SPEC_ERR_CAPACITY);
    }
    return;
  }
  const int ntiles = p.per_cta == 2 && node0 + p.npt < N ? 2 : 1;
  const Split sp = split_of(P, N, p.splits, split);
  const int nb = sp.nb, np = sp.np;

  // softmax threads: slot, tile, row (its TMEM lane), and what the row stands for
  const bool soft = warp >= kSoft0 && warp < kMma1;
  // (two tiles: a slot has one of them and every block; one tile: the slots take its blocks in turn)
  const int slot = warp >= kSoft0 + 4 ? 1 : 0, tile = ntiles == 2 ? slot : 0;
  const int step = ntiles == 2 ? 1 : 2;
  const int row = (warp & 3) * 32 + lane;
  const int node = node0 + tile * p.npt + row / p.G;
  const int head = g * p.G + row % p.G;
  const bool valid = soft && row < p.npt * p.G && node < N;
  const size_t orow = (size_t)(base + node) * p.hq + head;
  const int group = p.per_cta * blockIdx.y + tile + p.mtiles * (b * p.hkv + g);

  if (nb == 0) {  // an empty key split: nothing for the merge
    if (soft) {
      pdl_wait();
      if (valid && (ntiles == 2 || slot == 0)) p.part_lse[((size_t)group * p.splits + split) * kRows + row] = -INFINITY;
    }
    return;
  }

  auto bar = [&](uint64_t* x) { return tc::smem_u32(x); };
  volatile int* abort = &bars.abort;
  if (warp == 0) {
    uint64_t* all = reinterpret_cast<uint64_t*>(&bars);
    for (int x = lane; x < kBarAll; x += 32) tc::mbar_init(bar(all + x), x < kBar1 ? 1 : x < kBar4 ? 4 : ntiles);
    if (lane < kMaxTreeWords) bars.bad[lane] = 0;
    if (lane == 0) bars.abort = 0;
    tc::mbar_fence_init();
  } else if (warp == 1) {
    tc::tmem_alloc(bar(reinterpret_cast<uint64_t*>(&bars.tmem)), kTmemCols);
    tc::tmem_relinquish();
  }
  // in flight over the setup: q's rows (to L2), the producer's first page ids
  int ids0 = p.num_pages;
  if (valid) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + orow * kD));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + orow * kD + 64));
  } else if ((warp == 0 || warp == kVProd) && sp.pg_lo + lane < sp.pg_hi) {
    ids0 = ld(p.page_table + (size_t)b * p.max_pages + sp.pg_lo + lane);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars.tmem;
  bool ok = true;

  if (warp == 0 || warp == kVProd) {
    // ------------------------------------------------------------------ TMA producers
    // Warp 0 loads K and the pages' scales, the last one V's codes (one warp issuing all copies of
    // a block took longer than its products). Page ids of eight blocks at a time, one per lane, a
    // batch ahead of their use; an id is checked when its batch comes up.
    const bool isv = warp == kVProd;
    const uint32_t leader = elect_one();
    const int kSt = isv ? kStC : kStK;
    uint64_t* full = isv ? bars.c_full : bars.k_full;
    uint64_t* empty = isv ? bars.c_empty : bars.k_empty;
    const uint32_t ring = sb + (isv ? kOffC : kOffK);
    const CUtensorMap* tm_tree = isv ? &tm_vt : &tm_kt;
    const CUtensorMap* tm_pool = isv ? &tm_vp : &tm_kp;
    auto ids_of = [&](int k) -> int {
      const int lp = sp.pg_lo + 32 * k + lane;
      return lp < sp.pg_hi ? ld(p.page_table + (size_t)b * p.max_pages + lp) : p.num_pages;
    };
    auto checked = [&](int page, int k) -> int {
      if (page >= 0 && page < p.num_pages) return page;
      if (!isv && sp.pg_lo + 32 * k + lane < sp.pg_hi) report_waited(p.status, SPEC_ERR_PAGE);
      return p.num_pages;  // out of range: TMA reads zeros
    };
    auto scale_of = [&](int page) {
      return !isv && page < p.num_pages ? ld(p.kv_scale + (size_t)page * p.hkv + g) : make_float2(1.f, 1.f);
    };
    int ids = checked(ids0, 0), ids_next = ids_of(1);
    float2 sc = scale_of(ids), sc_next = sc;
    int done = 0;  // blocks whose copies were issued
#pragma unroll 1
    for (int j = 0, st = 0, turn = 0; j < nb; ++j, ++st) {
      if (st == kSt) st = 0, ++turn;
      if (turn > 0 && !wait_all(bar(&empty[st]), (turn & 1) ^ 1, abort)) break;
      const uint32_t dst = ring + st * kStage;
      // (one lane issues, the others' part predicated off: a copy by each of eight lanes cost about
      // 60 cycles more a copy)
      tc::expect_tx_if(leader, bar(&full[st]), j < np ? kKeys * 128 : 2 * kTreeSlab);
      if (j < np) {
        if ((j & 7) == 0 && j > 0) {
          ids = ids_next;
          sc = sc_next;
          ids_next = ids_of((j >> 3) + 1);
        }
#pragma unroll
        for (int pp = 0; pp < kPages; ++pp)
          tc::tma_load_4d_if(leader, dst + pp * 2048, tm_pool, bar(&full[st]), 0, 0, g,
                             __shfl_sync(0xffffffffu, ids, (j & 7) * kPages + pp));
        if ((j & 7) == 4) {
          ids_next = checked(ids_next, (j >> 3) + 1);
          sc_next = scale_of(ids_next);
        }
        if (!isv && (j & 7) == 0) {
          // The scales of these eight blocks. What their places held, thirty-two to twenty-five
          // blocks ago, has been read: the stage just filled was released by QK of eight blocks ago,
          // which its slot issued after PV of twelve blocks ago at the latest, so after that block's
          // softmax; the stage filled before it by QK of nine, after the softmax of thirteen.
          const float vs = page_scale(sc.y);
          *reinterpret_cast<float4*>(smem + kOffScale + ((j % kScales) * kPages + lane) * 16) =
              make_float4(page_scale(sc.x), log2f(vs), 1.f / vs, 0.f);
          warp_arrive(bar(&bars.sc_full[(j >> 3) & 1]));
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)  // two 64-column halves
          tc::tma_load_3d_if(leader, dst + h * kTreeSlab, tm_tree, bar(&full[st]), h * 64, g,
                             base + (sp.tb_lo + j - np) * kTreeKeys);
      }
      done = j + 1;
    }
    if (done < nb && lane == 0) {  // given up: leave no copy in flight
      report_waited(p.status, SPEC_ERR_TIMEOUT);
      int zero = 0;
      for (int j = max(0, done - kSt); j < done; ++j)
        tc::mbar_wait(bar(&full[j % kSt]), (j / kSt) & 1, &zero, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == 1 || warp == kMma1) {
    // ------------------------------------------------------------------ MMA issuers, one a slot
    const int t = warp == 1 ? 0 : 1, j0 = ntiles == 2 ? 0 : t;
    if (j0 < nb && elect_one()) {
      const uint32_t ts = tmem + 256 * t, to = ts + 128;
      const uint32_t q8 = sb + kOffQ + (ntiles == 2 ? t : 0) * 2 * kSlab;
      const uint32_t q16 = sb + kOffQ + (ntiles == 2 ? t : 1) * 2 * kSlab;
      bool codes = false, rows = false;  // q has been waited for
      auto qk = [&](int j, int n) {
        const int sk = j % kStK;
        if (j < np && !codes) ok = codes = wait_one(bar(&bars.q8[ntiles == 2 ? t : 0]), 0, abort);
        if (j >= np && !rows) ok = rows = wait_one(bar(&bars.q16[ntiles == 2 ? t : 1]), 0, abort);
        ok = ok && wait_one(bar(&bars.k_full[sk]), (j / kStK) & 1, abort);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t d = ts + 64 * (n & 1);
        const uint64_t kd = tc::sdesc_sw128(sb + kOffK + sk * kStage, 16, 1024);
        if (j < np) {
          const uint64_t qd = tc::sdesc_sw128(q8, 16, 1024);
#pragma unroll
          for (int k = 0; k < 8; ++k)  // hi, then lo
            tc::mma_f8(d, qd + (((k >> 2) * kSlab + (k & 3) * 32) >> 4), kd + (((k & 3) * 32) >> 4), kIdQK, k > 0);
        } else {
          const uint64_t qd = tc::sdesc_sw128(q16, 16, 1024);
#pragma unroll 1
          for (int k = 0; k < 8; ++k)
            tc::mma_bf16(d, qd + (((k >> 2) * kSlab + (k & 3) * 32) >> 4),
                         kd + (((k >> 2) * kTreeSlab + (k & 3) * 32) >> 4), kIdTreeQK, k > 0);
        }
        tc::mma_commit(bar(&bars.s_full[t][n & 1]));
        tc::mma_commit(bar(&bars.k_empty[sk]));
      };
      qk(j0, 0);
#pragma unroll 1
      for (int j = j0, n = 0; ok && j < nb; j += step, ++n) {
        if (j + step < nb) qk(j + step, n + 1);  // S of the next block while the softmax works on this one
        const int sv = j % kStV;
        ok = ok && wait_one(bar(&bars.v_full[sv]), (j / kStV) & 1, abort) &&
             wait_one(bar(&bars.p_full[t][n & 1]), (n >> 1) & 1, abort);
        if (!ok) break;
        tc::fence_after_sync();
        // P stands where its S stood; the QK that next overwrites it follows this PV in order
        const uint64_t vd = tc::sdesc_sw128(sb + kOffV + sv * kSlab, kVSlab, 1024);
        const uint32_t tp = ts + 64 * (n & 1);
        if (j < np) {
#pragma unroll
          for (int k = 0; k < 4; ++k) tc::mma_bf16_ts(to, tp + 8 * k, vd + ((k * 2048) >> 4), kIdPV, n > 0 || k > 0);
        } else {
#pragma unroll 1
          for (int k = 0; k < 4; ++k)  // P's two bf16 terms, two steps of 16 nodes each
            tc::mma_bf16_ts(to, tp + 8 * k, vd + (((k & 1) * 2048) >> 4), kIdTreePV, n > 0 || k > 0);
        }
        tc::mma_commit(bar(&bars.pv_done[t][n & 1]));
        tc::mma_commit(bar(&bars.v_empty[sv]));
      }
      if (!ok) report_waited(p.status, SPEC_ERR_TIMEOUT);
      // every product issued has completed before TMEM is released
      tc::mma_commit(bar(&bars.fin[t]));
      int zero = 0;
      tc::mbar_wait(bar(&bars.fin[t]), 0, &zero, kWaitLimit);
    }
    __syncwarp();
  } else if (warp > kMma1) {
    // ------------------------------------------------------------------ V converters
    const int ct = threadIdx.x - (kMma1 + 1) * 32;
    const int r0 = (ct & 7) | ((ct >> 6) << 3), cc = (ct >> 3) & 7;
    const uint32_t src0 = swz(r0, cc);
    const uint32_t dst0 = (cc >> 2) * kVSlab + swz(r0, (cc & 3) * 2);
    const uint32_t dst1 = (cc >> 2) * kVSlab + swz(r0, (cc & 3) * 2 + 1);
    const int tail = min(P, sp.pg_hi * 16) - (sp.pg_lo + (np - 1) * kPages) * 16;  // rows of the last prefix block
#pragma unroll 1
    for (int j = 0; j < nb; ++j) {
      const int sc_ = j % kStC, sv = j % kStV;
      ok = wait_all(bar(&bars.c_full[sc_]), (j / kStC) & 1, abort);
      if (!ok) break;
      uint8_t* src = smem + kOffC + sc_ * kStage;
      uint8_t* dst = smem + kOffV + sv * kSlab;
      if (j >= np) {
        // bf16 rows as they are, but for rows past the tree and elements that are not finite
        // (a weight of 0 times either would reach rows whose mask leaves the node out)
        const int tb = sp.tb_lo + j - np, nvalid = N - tb * kTreeKeys;
        if (j >= kStV) ok = wait_all(bar(&bars.v_empty[sv]), ((j / kStV) & 1) ^ 1, abort);
        if (!ok) break;
#pragma unroll 1
        for (int it = 0; it < 4; ++it) {
          const int id = it * 128 + ct, half = id >> 8, off = id & 255, r = off >> 3;
          const uint4 w = *reinterpret_cast<const uint4*>(src + half * kTreeSlab + off * 16);
          uint32_t u[4] = {w.x, w.y, w.z, w.w};
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (r >= nvalid) u[k] = 0;
            if ((u[k] & 0x7F80u) == 0x7F80u) {
              u[k] &= 0xFFFF0000u;
              bad = true;
            }
            if ((u[k] & 0x7F800000u) == 0x7F800000u) {
              u[k] &= 0xFFFFu;
              bad = true;
            }
          }
          if (bad) atomicOr(reinterpret_cast<unsigned long long*>(&bars.bad[tb >> 1]), 1ull << (r + 32 * (tb & 1)));
          *reinterpret_cast<uint4*>(dst + half * kVSlab + off * 16) = make_uint4(u[0], u[1], u[2], u[3]);
        }
      } else {
        // 16 codes a piece: row r0 + 16 it, chunk cc (8 lanes take 8 rows, so that loads and stores
        // meet 8 different 16-byte columns; the swizzle depends on r % 8 alone, the same in every
        // piece of a thread)
        if (j == np - 1) {  // rows past the prefix may hold anything (each thread clears what it will read)
#pragma unroll 1
          for (int r = r0; r < kKeys; r += 16)
            if (r >= tail) *reinterpret_cast<uint4*>(src + src0 + (r - r0) * 128) = make_uint4(0, 0, 0, 0);
        }
        uint4 w[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) w[it] = *reinterpret_cast<const uint4*>(src + src0 + it * 2048);
        if (j >= kStV) ok = wait_all(bar(&bars.v_empty[sv]), ((j / kStV) & 1) ^ 1, abort);
        if (!ok) break;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const uint32_t u[4] = {w[it].x, w[it].y, w[it].z, w[it].w};
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            h[2 * k] = half2_of((uint16_t)(u[k] & 0xFFFFu));
            h[2 * k + 1] = half2_of((uint16_t)(u[k] >> 16));
          }
          *reinterpret_cast<uint4*>(dst + dst0 + it * 2048) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + dst1 + it * 2048) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
      tc::fence_proxy_async_smem();
      warp_arrive(bar(&bars.v_full[sv]));
      warp_arrive(bar(&bars.c_empty[sc_]));
    }
    if (!ok && lane == 0) report_waited(p.status, SPEC_ERR_TIMEOUT);
  } else {
    // ------------------------------------------------------------------ softmax
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16, ts = tmem + 256 * slot + quarter, to = ts + 128;
    const bool live = __any_sync(0xffffffffu, valid);  // a warp without rows only keeps step
    const float scale_log2 = p.scale_log2;
    const uint4* qrow = reinterpret_cast<const uint4*>(p.q + orow * kD);
    float2* join = reinterpret_cast<float2*>(smem + kOffJoin);
    float m = -INFINITY, l = 0.f;  // running maximum and sum
    // M follows the row's maximum, and O is rescaled where it moves
    auto raise = [&](int n, float mx) {
      const bool moves = mx > -INFINITY && (m == -INFINITY || mx > m + kGrow);
      if (__any_sync(0xffffffffu, moves)) {
        float alpha = 1.f;
        if (moves) {
          alpha = m == -INFINITY ? 0.f : ex2_approx(m - mx);
          m = mx;
          l *= alpha;
        }
        if (n > 0) {  // O is complete up to the block before
          ok = wait_all(bar(&bars.pv_done[slot][(n - 1) & 1]), ((n - 1) >> 1) & 1, abort) && ok;
          tc::fence_after_sync();
#pragma unroll 1
          for (int ch = 0; ch < kD / 16; ++ch) {
            float o[16];
            tc::tmem_ld16(to + ch * 16, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= alpha;
            tc::tmem_st16(to + ch * 16, o);
          }
        }
      }
      return m == -INFINITY ? 0.f : kShift - m;
    };
    // the tree's q: its rows as they are; of two tiles, where the codes stood
    auto store_q16 = [&]() {
#pragma unroll 1
      for (int k = 0; k < 16; k += 4) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = valid ? ld(qrow + k + e) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(smem + kOffQ + (2 * slot + (k >> 3)) * kSlab + swz(row, (k + e) & 7)) = v[e];
      }
      tc::fence_proxy_async_smem();
      warp_arrive(bar(&bars.q16[slot]));
    };
    float rowf = scale_log2;
    if (np > 0 && (ntiles == 2 || slot == 0)) {
      const float qf = split_row(qrow, valid, smem + kOffQ + tile * 2 * kSlab, row);
      if (ntiles == 1) join[row].x = qf;
      rowf *= qf;
      tc::fence_proxy_async_smem();
      warp_arrive(bar(&bars.q8[slot]));
    }
    if (nb > np && (ntiles == 2 ? np == 0 : slot == 1)) store_q16();
    if (np > 0 && ntiles == 1 && slot == 1) {  // the same row's factor, from the other slot
      ok = wait_all(bar(&bars.q8[0]), 0, abort);
      rowf *= join[row].x;
    }
    int j = ntiles == 2 ? 0 : slot, n = 0;
    int left = min(P, sp.pg_hi * 16) - (sp.pg_lo + j * kPages) * 16;  // prefix keys from this block's first on
#pragma unroll 1
    for (; ok && j < np; j += step, ++n, left -= step * kKeys) {
      if ((j & 7) < step) ok = wait_all(bar(&bars.sc_full[(j >> 3) & 1]), (j >> 4) & 1, abort);
      const float4* scale = reinterpret_cast<const float4*>(smem + kOffScale) + (j % kScales) * kPages;
      float4 f[kPages];
#pragma unroll
      for (int pp = 0; pp < kPages; ++pp) f[pp] = scale[pp];
      ok = ok && wait_all(bar(&bars.s_full[slot][n & 1]), (n >> 1) & 1, abort);
      if (!ok) break;
      tc::fence_after_sync();
      if (j == np - 1 && nb > np && ntiles == 2) store_q16();  // (every QK over the codes is complete)
      const uint32_t tj = ts + 64 * (n & 1);
      if (live) {
        if (left < kKeys) {  // the last block's keys past the prefix
#pragma unroll 1
          for (int c = left; c < kKeys; ++c) tc::tmem_st1_u(tj + c, 0xFF800000u);
          tc::tmem_wait_st();
        }
        float s[kKeys];
        tc::tmem_ld32(tj, s);
        tc::tmem_ld32(tj + 32, s + 32);
        tc::tmem_wait_ld();
        float mx = -INFINITY;  // the largest x log2 e + log2 vs
#pragma unroll
        for (int pp = 0; pp < kPages; ++pp) {
          const float* v = s + 16 * pp;
          float x = fmax3(v[0], v[1], v[2]);
#pragma unroll
          for (int c = 3; c < 15; c += 2) x = fmax3(x, v[c], v[c + 1]);
          f[pp].x = factor(rowf, f[pp].x);
          mx = fmaxf(mx, fmaf(fmaxf(x, v[15]), f[pp].x, f[pp].y));
        }
        const float off = raise(n, mx);
        uint32_t pk[kKeys / 2];
#pragma unroll
        for (int pp = 0; pp < kPages; ++pp) {
          const float oo = off + f[pp].y;
          const float2 f2 = make_float2(f[pp].x, f[pp].x), o2 = make_float2(oo, oo);
          float2 s0 = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float* v = s + 16 * pp + c;
            uint32_t* to2 = pk + 8 * pp + (c >> 1);
            const float2 a = ffma2(make_float2(v[0], v[1]), f2, o2);
            const float2 d = ffma2(make_float2(v[2], v[3]), f2, o2);
            const float2 ea = make_float2(ex2_approx(a.x), ex2_approx(a.y));
            const float2 ed = make_float2(ex2_approx(d.x), ex2_approx(d.y));
            s0 = fadd2(s0, ea);
            s1 = fadd2(s1, ed);
            to2[0] = pack_f16x2(ea.x, ea.y);
            to2[1] = pack_f16x2(ed.x, ed.y);
          }
          l = fmaf((s0.x + s0.y) + (s1.x + s1.y), f[pp].z, l);
        }
        tc::tmem_st32_u(tj, pk);
        tc::tmem_wait_st();
      }
      tc::fence_before_sync();
      if (ok) warp_arrive(bar(&bars.p_full[slot][n & 1]));
    }
    if (ok && j < nb) {
      pdl_wait();  // the mask may come from the kernel before
      const uint32_t* mrow =
          reinterpret_cast<const uint32_t*>(p.mask + (size_t)(base + node) * p.mask_words) + sp.tb_lo;
      uint32_t bits = valid ? __ldcg(mrow + j - np) : 0u;
#pragma unroll 1
      for (; ok && j < nb; j += step, ++n) {  // P as two bf16 terms
        ok = wait_all(bar(&bars.s_full[slot][n & 1]), (n >> 1) & 1, abort);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t tj = ts + 64 * (n & 1);
        if (live) {
          const uint32_t see = bits;
          if (valid && j + step < nb) bits = __ldcg(mrow + j + step - np);
          float s[kTreeKeys];
          tc::tmem_ld32(tj, s);
          tc::tmem_wait_ld();
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < kTreeKeys; ++c) {
            s[c] = ((see >> c) & 1u) ? s[c] * scale_log2 : -INFINITY;
            mx = fmaxf(mx, s[c]);
          }
          const float off = raise(n, mx);
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float a = ex2_approx(s[16 * h + 2 * c] + off), d = ex2_approx(s[16 * h + 2 * c + 1] + off);
              sum0 += a;
              sum1 += d;
              hi[c] = pack_bf16x2(a, d);
              lo[c] = pack_bf16x2(a - __uint_as_float(hi[c] << 16), d - __uint_as_float(hi[c] & 0xFFFF0000u));
            }
            tc::tmem_st8_u(tj + 8 * h, hi);
            tc::tmem_st8_u(tj + 16 + 8 * h, lo);
          }
          l += sum0 + sum1;
          tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        if (ok) warp_arrive(bar(&bars.p_full[slot][n & 1]));
      }
    }
    if (n > 0) ok = ok && wait_all(bar(&bars.pv_done[slot][(n - 1) & 1]), ((n - 1) >> 1) & 1, abort);
    if (!ok && lane == 0) report_waited(p.status, SPEC_ERR_TIMEOUT);

    // -------------------------------------------------------------------- epilogue
    // Of one tile, the slots' sums are joined: both hold the same rows, and each thread takes 64
    // columns of its row, from both O's; of two, a thread has its row's 128 columns.
    float2 other = make_float2(-INFINITY, 0.f);
    if (ntiles == 1) {
      tc::fence_before_sync();
      soft_sync();  // (the factors have been read)
      join[slot * kRows + row] = make_float2(m, l);
      soft_sync();
      other = join[(slot ^ 1) * kRows + row];
    }
    tc::fence_after_sync();
    pdl_wait();  // nothing is written before the kernel before has finished
    if (live) {
      const float top = fmaxf(m, other.x);
      const float w0 = m == -INFINITY ? 0.f : ex2_approx(m - top);
      const float w1 = other.x == -INFINITY ? 0.f : ex2_approx(other.x - top);
      const float sum = l * w0 + other.y * w1;
      float inv = sum == 0.f ? 0.f : 1.f / sum;
      // a tree node that this row sees holds an infinity or NaN in V
#pragma unroll 1
      for (int i = sp.tb_lo >> 1; 2 * i < sp.tb_lo + nb - np; ++i) {
        const uint64_t bad = bars.bad[i];
        if (bad != 0 && valid && (__ldcg(p.mask + (size_t)(base + node) * p.mask_words + i) & bad) != 0)
          inv = __int_as_float(0x7FC00000);
      }
      if (!ok || *abort) inv = 0.f;
      const float i0 = inv * w0, i1 = inv * w1;
      const bool mine = n > 0, theirs = ntiles == 1 && nb > (slot ^ 1);  // an O that was written
      const uint32_t to2 = tmem + 256 * (slot ^ 1) + 128 + quarter;
      float4* po = p.part_o + ((size_t)group * p.splits + split) * (kRows * kD / 4) + row;
      const int c0 = ntiles == 2 ? 0 : 4 * slot, c1 = ntiles == 2 ? 8 : c0 + 4;
#pragma unroll 1
      for (int ch = c0; ch < c1; ++ch) {
        float x[16], y[16];
        __syncwarp();
        tc::tmem_ld16(to + 16 * ch, x);
        if (theirs) tc::tmem_ld16(to2 + 16 * ch, y);
        tc::tmem_wait_ld();
        if (!valid) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          x[k] = mine ? x[k] * i0 : 0.f;
          if (theirs) x[k] += y[k] * i1;
        }
        if (p.splits == 1) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + orow * kD + 16 * ch);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            dst[k] = make_uint4(pack_bf16x2(x[8 * k], x[8 * k + 1]), pack_bf16x2(x[8 * k + 2], x[8 * k + 3]),
                                pack_bf16x2(x[8 * k + 4], x[8 * k + 5]), pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            po[(ch * 4 + k) * kRows] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        }
      }
      if (valid && (ntiles == 2 || slot == 0)) {
        const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum) - kShift;
        if (p.splits > 1) p.part_lse[((size_t)group * p.splits + split) * kRows + row] = lse2;
        else if (p.lse != nullptr) p.lse[orow] = lse2 * kLn2;
      }
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of the key splits: out = sum_s 2^(lse_s - M) O_s / sum_s 2^(lse_s - M). One thread per
// (tile, 4 columns, row), every load issued before any is used.
struct MergeParams {
  const float4* part_o;
  const float* part_lse;
  const int32_t* qo;
  const int32_t* prefix_len;
  int max_len, max_nodes;
  int splits, mtiles, hkv, hq, G, npt;
  long tiles;
  __nv_bfloat16* out;
  float* lse;
};
constexpr int kMergeThreads = 64;

template <int MAXS>
__global__ void __launch_bounds__(kMergeThreads) attn_kv8p_merge_kernel(const MergeParams p) {
  pdl_trigger();
  const long idx = (long)blockIdx.x * kMergeThreads + threadIdx.x;
  if (idx >= p.tiles * 32 * kRows) return;
  const int tile = (int)(idx / (32 * kRows)), rem = (int)(idx - (long)tile * 32 * kRows);
  const int c = rem / kRows, r = rem % kRows;
  const int tt = tile % p.mtiles, bg = tile / p.mtiles, b = bg / p.hkv, g = bg - b * p.hkv;
  const int node = tt * p.npt + r / p.G;
  if (r >= p.npt * p.G) return;
  pdl_wait();  // the attention grid has finished: its partials are visible
  const int base = ld(p.qo + b), N = ld(p.qo + b + 1) - base, P = ld(p.prefix_len + b);
  if (node >= N || N > p.max_nodes || P < 0 || P > p.max_len) return;  // as the attention
  const float* ls = p.part_lse + (size_t)tile * p.splits * kRows + r;
  const float4* po = p.part_o + (size_t)tile * p.splits * (kRows * kD / 4) + c * kRows + r;
  float lv[MAXS];
  float4 o[MAXS];
#pragma unroll
  for (int s = 0; s < MAXS; ++s) {
    lv[s] = s < p.splits ? __ldcg(ls + s * kRows) : -INFINITY;
    o[s] = s < p.splits ? __ldcg(po + (size_t)s * (kRows * kD / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int s = 0; s < MAXS; ++s) M = fmaxf(M, lv[s]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int s = 0; s < MAXS; ++s) {
    if (lv[s] == -INFINITY) continue;  // nothing in it: its row was not written
    const float w = ex2_approx(lv[s] - M);
    L += w;
    acc = make_float4(fmaf(o[s].x, w, acc.x), fmaf(o[s].y, w, acc.y), fmaf(o[s].z, w, acc.z), fmaf(o[s].w, w, acc.w));
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t orow = (size_t)(base + node) * p.hq + g * p.G + r % p.G;
  *reinterpret_cast<uint2*>(p.out + orow * kD + c * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (c == 0 && p.lse != nullptr) p.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ------------------------------------------------------------------------------------ host

static int tiles_of(int max_nodes, int npt) { return ceil_div(max_nodes, npt); }

// Row tiles that a CTA has: two where the sequence has them (they share K, V and V's conversion),
// unless one a CTA is what it takes to put a CTA on every SM without cutting the keys into more
// splits, each of which writes its partial result. (One tree of 64 nodes over 4096 keys, 16 tiles:
// 24 us with one a CTA and 9 splits, 31 with two and 19 or 10. 32 of them, 512 tiles: 243 and 156 us;
// 8 x 128 nodes over 32768 keys, 512 tiles: 976 and 923.)
static int tiles_per_cta(int batch, int max_nodes, int hq, int hkv) {
  const int tiles = tiles_of(max_nodes, kRows / (hq / hkv));
  return tiles > 1 && (long)batch * hkv * ceil_div(tiles, 2) >= sm_count() ? 2 : 1;
}

// Key splits per work item (sequence, KV head, two row tiles), from the sizes alone; one
// CTA fits on an SM. Fewer items than SMs: the splits that cover the SMs. Otherwise the count
// in 1..8 whose waves cost least (a CTA's fixed cost counted as six blocks), if that is at
// least 8% below the unsplit cost (the merge kernel is not in the model).
static int splits_of(int batch, int max_nodes, int hq, int hkv, int max_prefix) {
  const int npt = kRows / (hq / hkv);
  const long items = (long)batch * hkv * ceil_div(tiles_of(max_nodes, npt), tiles_per_cta(batch, max_nodes, hq, hkv));
  const long sms = sm_count();
  const int blocks = ceil_div(max_prefix, kKeys) + ceil_div(max_nodes, kTreeKeys);
  long s = 1;
  if (items > 0 && items < sms) {
    s = sms / items;
  } else if (items > 0) {
    long best = -1;
    for (long c = 1; c <= 8; ++c) {
      const long cost = ((items * c + sms - 1) / sms) * ((blocks + c - 1) / c + 6);
      if (best < 0 || cost < best) {
        best = cost;
        s = c;
      }
    }
    if (s > 1 && best * 100 > ((items + sms - 1) / sms) * (blocks + 6) * 92) s = 1;
  }
  if (s > blocks) s = blocks;
  if (s > kMaxSplits) s = kMaxSplits;
  return s < 1 ? 1 : (int)s;
}

struct Ws {
  size_t o, total;
};
static Ws ws_of(long tiles, int splits) {
  Ws w;
  w.o = align_up(sizeof(float) * tiles * splits * kRows, 256);
  w.total = w.o + sizeof(float) * tiles * splits * kRows * kD;
  return w;
}

}  // namespace kv8p

size_t attn_kv8p_ws_bytes(int batch, int max_nodes, int hq, int hkv, int max_prefix) {
  const int s = kv8p::splits_of(batch, max_nodes, hq, hkv, max_prefix);
  if (s <= 1) return 0;
  return kv8p::ws_of((long)batch * hkv * kv8p::tiles_of(max_nodes, kv8p::kRows / (hq / hkv)), s).total;
}

int launch_attn_kv8p(const void* q, const uint8_t* k_pool, const uint8_t* v_pool, const float* kv_scale, int num_pages,
                     const int32_t* page_table, int max_pages, const int32_t* prefix_len, int max_prefix,
                     const void* k_tree, const void* v_tree, const uint64_t* mask, const int32_t* qo, int batch,
                     int total_nodes, int max_nodes, int hq, int hkv, float sm_scale, void* out, float* lse, void* ws,
                     int32_t* status, cudaStream_t stream) {
  using namespace kv8p;
  const int G = hq / hkv;
  CUtensorMap tm_kp, tm_vp, tm_kt, tm_vt;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)hkv, (cuuint64_t)total_nodes};
    const cuuint64_t str[2] = {(cuuint64_t)kD * 2, (cuuint64_t)hkv * kD * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kTreeKeys};
    if (!encode_bf16(&tm_kt, k_tree, 3, dims, str, box)) return SPEC_ERR_CUDA;
    if (!encode_bf16(&tm_vt, v_tree, 3, dims, str, box)) return SPEC_ERR_CUDA;
  }
  if (max_prefix > 0) {  // one 16-token x 128-code tile (2 KB) per (page, head), 128-byte rows
    const cuuint64_t dims[4] = {(cuuint64_t)kD, 16, (cuuint64_t)hkv, (cuuint64_t)num_pages};
    const cuuint64_t str[3] = {(cuuint64_t)kD, (cuuint64_t)16 * kD, (cuuint64_t)hkv * 16 * kD};
    const cuuint32_t box[4] = {(cuuint32_t)kD, 16, 1, 1};
    if (!encode_tiled(&tm_kp, CU_TENSOR_MAP_DATA_TYPE_UINT8, k_pool, 4, dims, str, box)) return SPEC_ERR_CUDA;
    if (!encode_tiled(&tm_vp, CU_TENSOR_MAP_DATA_TYPE_UINT8, v_pool, 4, dims, str, box)) return SPEC_ERR_CUDA;
  } else {  // no prefix anywhere: the pool's maps are not used
    tm_kp = tm_kt;
    tm_vp = tm_vt;
  }
  static PerDevice smem_set;
  if (per_device(smem_set, [](int) {
        return cudaFuncSetAttribute(attn_kv8p_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess
                   ? 1
                   : 0;
      }) == 0)
    return SPEC_ERR_CUDA;
  Params prm;
  prm.q = static_cast<const __nv_bfloat16*>(q);
  prm.kv_scale = reinterpret_cast<const float2*>(kv_scale);
  prm.page_table = page_table;
  prm.max_pages = max_pages;
  prm.num_pages = num_pages;
  prm.max_len = max_prefix;  // (the caller's rows hold it: checked on the host)
  prm.prefix_len = prefix_len;
  prm.mask = mask;
  prm.mask_words = (max_nodes + 63) >> 6;
  prm.max_nodes = max_nodes;
  prm.qo = qo;
  prm.hq = hq;
  prm.hkv = hkv;
  prm.G = G;
  prm.npt = kRows / G;
  prm.splits = splits_of(batch, max_nodes, hq, hkv, max_prefix);
  prm.mtiles = tiles_of(max_nodes, prm.npt);
  prm.per_cta = tiles_per_cta(batch, max_nodes, hq, hkv);
  prm.scale_log2 = sm_scale * kLog2e;
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.lse = lse;
  const long tiles = (long)batch * hkv * prm.mtiles;
  const Ws w = ws_of(tiles, prm.splits);
  uint8_t* wb = static_cast<uint8_t*>(ws);
  prm.part_lse = prm.splits > 1 ? reinterpret_cast<float*>(wb) : nullptr;
  prm.part_o = prm.splits > 1 ? reinterpret_cast<float4*>(wb + w.o) : nullptr;
  prm.status = status;
  prm.early = early_reads() ? 1 : 0;
  prm.batch = batch;
  // (past eight waves the last one is a small share of the grid)
  prm.lpt = prm.splits == 1 && batch > 1 && batch <= kLptMax && tiles <= 16L * sm_count() ? 1 : 0;
  const dim3 grid(prm.splits, ceil_div(prm.mtiles, prm.per_cta), batch * hkv);
  if (launch_pdl(attn_kv8p_kernel, grid, dim3(kThreads), kSmem, stream, tm_kp, tm_vp, tm_kt, tm_vt, prm) != cudaSuccess)
    return SPEC_ERR_CUDA;
  if (prm.splits > 1) {
    MergeParams mp{prm.part_o, prm.part_lse, qo, prefix_len, prm.max_len, max_nodes, prm.splits, prm.mtiles, hkv,
                   hq, G, prm.npt, tiles, prm.out, lse};
    const long threads = tiles * 32 * kRows;
    const dim3 mg((unsigned)((threads + kMergeThreads - 1) / kMergeThreads)), mb(kMergeThreads);
    const cudaError_t e = prm.splits <= 4    ? launch_pdl(attn_kv8p_merge_kernel<4>, mg, mb, 0, stream, mp)
                          : prm.splits <= 8  ? launch_pdl(attn_kv8p_merge_kernel<8>, mg, mb, 0, stream, mp)
                          : prm.splits <= 20 ? launch_pdl(attn_kv8p_merge_kernel<20>, mg, mb, 0, stream, mp)
                                             : launch_pdl(attn_kv8p_merge_kernel<kMaxSplits>, mg, mb, 0, stream, mp);
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
