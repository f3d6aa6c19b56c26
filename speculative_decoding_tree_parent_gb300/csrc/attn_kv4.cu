// Tree-verify attention over a 4-bit paged cache (kv4.cuh) on the 5th-generation tensor cores.
//
// Row (node i of sequence b, query head h, g = h / G, G = hq / hkv), over the prefix keys j and the tree
// nodes that its mask bits name:
//   x_j = sm_scale * q . k_j,   out = sum_j e^(x_j) v_j / sum_j e^(x_j),
//   prefix: k_j = code * group scale * kv_scale[0][g], v_j likewise;  tree: bf16 rows.
//
// Keys stand on the MMA's 128 rows and queries on its columns: S^T = K q^T and O^T = V^T P^T, so that a block of
// 128 keys costs a decode step of 8 query rows 16 columns, not 128 rows of softmax. It also makes K and V the A operands, which
// come from TMEM: a thread of K's converters has a token, one of V's an element of the head, each reads its codes from
// shared memory, widens them to fp16 (code * group scale has 6 significant bits: exact) and stores its TMEM lane;
// no widened copy passes through shared memory, whose bandwidth would be the bound.
// q, scaled per row by a power of two to a largest element in [2^14, 2^15), is fp16: exact for elements within
// 2^31 of the row's largest, off by at most 2^-39 of it below. The head's scale of K, the softmax scale and that power are one
// fp32 factor per row; the head's scale of V multiplies the finished row.
// Softmax: y = S * factor + off per row, P = 2^y in fp16 while no y passes 15; a block in which one does (and a
// segment's first) moves off so that the row's largest becomes 2^5 and rescales O. The row sum adds P unrounded. fp16 has
// 11 bits of a P down to 2^-14, 2^19 below that largest, and a step of 2^-24 below it: a smaller P is off by at most 2^-30 of
// the row's largest. Tree blocks (32 nodes) run in bf16 from the rows as they are, P as two bf16 terms.
//
// A row tile is R = 16, 32, 64 or 128 rows: R / G nodes of G heads, the least that holds a sequence's nodes. Two slots,
// each with its own MMA issuer, softmax warps and TMEM (S, O): of 128 rows a slot has 64 and every block, below that the
// slots take the blocks in turn and their sums are joined at the end. The work of the batch, (sequence, head, row
// tile) times its blocks, is one list of blocks, which the CTAs (one an SM) cut into equal shares, whatever the lengths:
// a share's first and last tile may be part of a tile, whose fp32 partial results a second kernel joins.
// Warps: 0 and 3 producers (a page's record is one bulk copy; a block is one's or the other's), 1 and 2 MMA issuers,
// then K's converters, V's, and the softmax. Up to 32 rows, where the cache's conversion is most of the work, each operand
// has two groups of four converter warps and a slot one of softmax warps (decode of 128 sequences 244 -> 212 us); of 64
// rows a slot it is one and two (32 trees of 64 nodes 338 -> 321). Every wait is bounded.
//
// What bounds it: of 128 rows the issue of instructions (4 sequences of 128 nodes over 16384: a scheduler issues in 73% of its
// cycles, the tensor pipe is active in 39%; about 8000 warp instructions a block, of which the softmax is 3100, the
// conversions 1700, waits and loops the rest; without the conversions 11% less time, without the exponentials 4%, without all
// of the softmax 24%), of 16 rows the conversions (24%) and the issue of the copies. Every shape spills a few registers (8 to 40
// bytes of stack): of 128 and 64 rows 41 and 35 loads of a warp a block (0.5%) bring some back, of 32 rows 5, of 16 one; they
// are stored a tile at a time. Unrolling the conversions' loops cost more than it gave (their code has to be fetched), a
// third issuer warp for O's products changed nothing. GB300: one token over 517, 32 query heads
// over 8, 12 us; 64 nodes over 4096 27; 128 tokens over 256 to 8190, 64 heads over 8, 182 (3.4 TB/s of records; 197 with
// one producer warp); 32 trees of 64 nodes over 512 to 8192, 32 heads over 8, 217; 8 of 101 to 128 nodes over 32768, 64
// heads over 8, 1075 (0.91 PFLOP/s).
#include "attn_common.cuh"
#include "kv4.cuh"
#include "tc_host.cuh"
#include "tc_math.cuh"

namespace specv {
namespace a4 {

using namespace kv4;

constexpr int kKeys = 128;      // keys of a prefix block
constexpr int kTreeKeys = 32;   // nodes of a tree block
constexpr int kProducer = 0, kMma0 = 1, kProducer2 = 3, kConvK = 4;  // warps (4: the first converter's)
constexpr uint32_t kStage = kKeys / kPage * kRecord;   // 18432: eight records, or a tree block's K and V rows
constexpr uint32_t kTreeV = kTreeKeys * kDim * 2;      // V's rows within it
static_assert(2 * kTreeV <= kStage, "a tree block fits a stage");
constexpr uint32_t kPBuf = kKeys * 128;                // P of a block: 128-byte rows of up to 64 queries
// TMEM's columns: each slot's S and O, then K and V in two buffers each. (512 hold S twice only with K and V once: of 128
// rows that took 1220 us for 8 sequences of 101 to 128 nodes over 32768 tokens, this 1100.)
constexpr uint32_t kColS = 0, kColO = 128, kColK = 256, kColV = 384;
constexpr int kSegs = 4;
// What a tile of R rows costs beside its blocks (q, the result, the pipeline's start, a tree block's more), in blocks: the
// shares count it. Ragged batches, us of a call among others: 32 trees of 64 nodes (128 rows) 235 with 4, 212 with 6, 198 with 8,
// 197 with 10, 200 with 12; 64 of 16 nodes (64 rows) 177, 163, 162, 164, 166; 64 of 8 nodes (32 rows) 121, 111, 107, 108,
// 110; 128 of one node (16 rows) 202 with 3, 196 with 4, 187 with 6, 190 with 8, 193 with 10. (The costs of 16 and 32 rows were
// the best with one producer warp; with two, 6 and 8 would be 5% and 3% better.)
__host__ __device__ constexpr int tile_cost(int R) { return R == 16 ? 4 : R == 32 ? 6 : 8; }
constexpr float kShift = 5.f;   // log2 of a row's largest P where off is set
constexpr float kLimit = 15.f;  // log2 of the largest P

struct Params {
  const __nv_bfloat16* q;
  const uint8_t* pool;
  const float* kv_scale;
  const int32_t* page_table;
  int max_pages, num_pages;
  const int32_t* prefix_len;
  int max_len;
  const __nv_bfloat16* k_tree;
  const __nv_bfloat16* v_tree;
  const uint64_t* mask;
  int mask_words, max_nodes;
  const int32_t* qo;
  int batch, total, hq, hkv, G, npt;  // npt: nodes of a row tile
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  int4* meta;       // [CTA]: (bit 0 a first partial, 1 its tile ends there, 2 a last partial), its b, g, node0
  float* part_lse;  // [CTA][2][R] log2-sum-exp
  float* part_o;    // [CTA][2][R][128], O / l
  int32_t* status;
};

// A run of blocks of one tile.
struct Seg {
  int b, g, node0, base, N, P;
  int j0, nb, np;  // first block within the tile, blocks, prefix blocks among them
  int piece;       // -1: the whole tile; else which partial of the CTA
};

struct Bars {
  uint64_t full[10], empty[10];                  // stages
  uint64_t kt_full[2], kt_free[2], vt_full[2], vt_free[2];
  uint64_t s_full[2], s_free[2], p_full[2][2], pv_done[2][2];  // [slot][buffer]
  uint64_t q_full[2], seg_full[kSegs], seg_empty[kSegs], fin[2];
  int flag[4][2];           // of a softmax group: the block n (at n % 2) in which a row last passed the limit
  Seg seg[kSegs];
  uint32_t bad_pages[10];   // of a stage: pages that are not in the pool
  uint32_t bad_nodes[2][4]; // of a tree block, by V's converter warps: nodes whose V holds an infinity or NaN
  int first_b, first_off;   // where the CTA's share starts
  int warp_sum[32];
  uint32_t tmem;
};
static_assert(sizeof(Bars) <= 1536, "barrier block over its reserved bytes");

// kW: rows of a slot; kDual: a slot has its own half of the tile's rows (else the slots take the blocks in turn).
// kConv: groups of four converter warps for K, and for V (two: each takes every other block, whose stages are its own).
template <int kW, bool kDual>
struct Shape {
  static constexpr int kConv = kW <= 32 ? 2 : 1;
  static constexpr int kConvV = kConvK + 4 * kConv, kSoft0 = kConvV + 4 * kConv;
  // groups of four softmax warps a slot, and the rows of a group
  static constexpr int kG = kW == 64 ? 2 : 1, kC = kW / kG, kThreads = 32 * (kSoft0 + 8 * kG);
  static constexpr int kR = kDual ? 2 * kW : kW, kTileCost = tile_cost(kR);
  // Registers a thread by role (of 32 rows and more), out of what the block is launched with: 72 a thread, as 896 threads
  // leave. A sum above that would wait forever.
  static constexpr int kRegMisc = 40, kRegConv = 56, kRegSoft = kW == 64 ? 88 : 104;
  static_assert(kThreads == 896 && 4 * kRegMisc + 8 * kConv * kRegConv + 8 * kG * kRegSoft <= 28 * 72, "more registers than the launch has");
  static constexpr uint32_t kQSlab = kW * 128;               // 64 elements of a slot's q rows
  static constexpr uint32_t kQ = 2 * kQSlab;                 // q of a slot, one type
  static constexpr int kQs = kDual ? 2 : 1;
  static constexpr uint32_t kOffQ = 0;                       // fp16, then bf16
  static constexpr uint32_t kOffP = kOffQ + 2 * kQs * kQ;    // [slot][buffer]
  static constexpr uint32_t kOffRing = kOffP + 4 * kPBuf;
  static constexpr int kStages = kDual ? 4 : kW == 64 ? 5 : 6;
  static constexpr uint32_t kOffBar = kOffRing + kStages * kStage;
  static constexpr uint32_t kOffRow = kOffBar + 1536;        // float4 [slot][kW / 2]: two factors, two offs
  static constexpr uint32_t kOffDelta = kOffRow + 2 * kW * 8;  // float [2][slot][kW]: factors, what off grew by
  static constexpr uint32_t kOffSum = kOffDelta + 4 * kW * 4;      // float2 [slot][kW]: off, row sum
  static constexpr uint32_t kOffFin = kOffSum + 2 * kW * 8;  // float2 [kR]: weights of the slots' O
  static constexpr uint32_t kOffOut = kOffFin + kR * 8;      // int [kR]: output row, -1: none
  static constexpr uint32_t kOffTree = kOffOut + kR * 4;       // float [slot][kW]: row sums of the tree blocks
  static constexpr uint32_t kOffMask = kOffTree + 2 * kW * 4;  // int [kR]: mask row, -1: none
  static constexpr uint32_t kOffRed = kOffMask + kR * 4;       // float [slot][32][kW]: maxima, or sums, of four tokens
  static constexpr uint32_t kOffScale = kOffRed + 2 * 32 * kW * 4;  // fp16 [warp of V's][8 pages][2 groups][16 tokens]
  static constexpr uint32_t kSmem = kOffScale + kConv * 2048 + 1024;
  static_assert(kSmem <= 232448, "shared memory over the per-CTA limit");
  static_assert(kConv == 1 || kStages % 2 == 0, "a stage has to belong to one group of converters");
  static_assert(kStages <= 10, "more stages than barriers");
};

// ---------------------------------------------------------------------------------- small pieces

// Waits are bounded (kTries of a millisecond) and in line: a kernel that hands registers from warp to warp cannot call
// a function. Without a time to hold it a try comes back so soon that the waiting warps take half of the issue slots.
constexpr uint32_t kTries = 1000, kHoldNs = 1000000;
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, uint32_t tries = kTries) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p, q; .reg .u32 n; mov.u32 n, 0;\n"
      "AGAIN: mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n"
      "@p bra DONE; add.u32 n, n, 1; setp.lt.u32 q, n, %3; @q bra AGAIN;\n"
      "DONE: selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(tries), "r"(kHoldNs)
      : "memory");
  return ok != 0;
}
// The same where a warp goes on whatever comes of it, to where it meets others: `tries` is 0 once a wait has given up, and
// further ones then try once.
__device__ __forceinline__ void wait_on(uint32_t bar, uint32_t parity, uint32_t& tries) {
  if (!wait_one(bar, parity, tries)) tries = 0;
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity) {
  const bool ok = wait_one(bar, parity);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  tc::mbar_arrive_if((threadIdx.x & 31) == 0, bar);
}
__device__ __forceinline__ void named_sync(int id, int n) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// Whether `x` holds in any of the n threads that meet at the barrier (whole warps, converged).
__device__ __forceinline__ bool named_any(int id, int n, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %3, 0; bar.red.or.pred q, %1, %2, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], kind::f16, with the descriptor in halves: of a run of products only the low one moves.
template <bool kFirst>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 b; setp.ne.b32 p, %5, 0; mov.b64 b, {%2, %3}; "
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p; }" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(kFirst ? 0 : 1)
      : "memory");
}
__device__ __forceinline__ float redux_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// 16-byte chunk c of row r of a slab of 128-byte rows, in the 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// Blocks of a tile of a sequence with P prefix keys and N nodes, and the sequence's tiles.
__device__ __forceinline__ int blocks_of(int P, int N) { return (P + kKeys - 1) / kKeys + (N + kTreeKeys - 1) / kTreeKeys; }

template <int kRegs>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ void tmem_ld8(uint32_t at, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// 16 lanes x kW columns of fp32 in the fragment layout: v[4 j + e] of thread t is column 8 j + 2 (t % 4) + e % 2 of lane
// t / 4 + 8 (e / 2).
template <int kW>
__device__ __forceinline__ void tmem_ld_frag(uint32_t at, float* v) {
  static_assert(kW == 16 || kW == 32, "the rows of a softmax group");
  uint32_t r[kW / 2];
  if constexpr (kW == 16) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at)
                 : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < kW / 2; ++i) v[i] = __uint_as_float(r[i]);
}
// Four 8 x 8 matrices of 16-bit elements from the fragment layout; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// ---------------------------------------------------------------------------------- the kernel

template <int kW, bool kDual>
__global__ void __launch_bounds__(Shape<kW, kDual>::kThreads, 1) attn_kv4_kernel(const Params p) {
  using S = Shape<kW, kDual>;
  constexpr int kThreads = S::kThreads, kConvV = S::kConvV, kSoft0 = S::kSoft0, kConv = S::kConv;
  constexpr int kTileCost = S::kTileCost, kG = S::kG, kC = S::kC, kSoft = 256 * kG;  // kSoft: softmax threads
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + S::kOffBar);
  const uint32_t sb = tc::smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  auto bar = [&](uint64_t& x) { return tc::smem_u32(&x); };

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      tc::mbar_init(bar(bars.full[i]), 1);
      tc::mbar_init(bar(bars.empty[i]), 8);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(bars.kt_full[i]), 4);
      tc::mbar_init(bar(bars.kt_free[i]), kDual ? 2 : 1);
      tc::mbar_init(bar(bars.vt_full[i]), 4);
      tc::mbar_init(bar(bars.vt_free[i]), kDual ? 2 : 1);
      tc::mbar_init(bar(bars.s_full[i]), 1);
      tc::mbar_init(bar(bars.s_free[i]), 4 * kG);
      for (int k = 0; k < 2; ++k) {
        tc::mbar_init(bar(bars.p_full[i][k]), 4 * kG);
        tc::mbar_init(bar(bars.pv_done[i][k]), 1);
      }
      tc::mbar_init(bar(bars.q_full[i]), (kDual ? 4 : 8) * kG);
      tc::mbar_init(bar(bars.fin[i]), 1);
      for (int k = 0; k < 4; ++k) bars.flag[i * 2 + (k >> 1)][k & 1] = -1;
    }
    for (int i = 0; i < kSegs; ++i) {
      tc::mbar_init(bar(bars.seg_full[i]), 1);
      tc::mbar_init(bar(bars.seg_empty[i]), 3 + 8 * kG + 8 * kConv);
    }
    tc::mbar_fence_init();
  } else if (warp == 1) {
    tc::tmem_alloc(bar(*reinterpret_cast<uint64_t*>(&bars.tmem)), 512);
    tc::tmem_relinquish();
  }
  pdl_wait();

  // ---- the CTA's share of all blocks: sizes summed over the batch, then the sequence where the share starts
  auto units_of = [&](int b) -> int {
    if (b >= p.batch) return 0;
    const int base = ld(p.qo + b), end = ld(p.qo + b + 1), P = ld(p.prefix_len + b);
    const bool outside = base < 0 || end < base || end > p.total;
    const int N = end - base;
    if (!outside && N == 0) return 0;
    if (outside || N > p.max_nodes || P < 0 || P > p.max_len) {
      if (blockIdx.x == 0) report(p.status, outside ? SPEC_ERR_INDEX : SPEC_ERR_CAPACITY);
      return 0;
    }
    return (N + p.npt - 1) / p.npt * p.hkv * (blocks_of(P, N) + kTileCost);
  };
  int sum = 0;
#pragma unroll 1
  for (int c = tid; c < p.batch; c += kThreads) sum += units_of(c);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) bars.warp_sum[warp] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) sum += bars.warp_sum[w];
  const int each = sum / (int)gridDim.x, more = sum - each * (int)gridDim.x;
  const int start = each * (int)blockIdx.x + min((int)blockIdx.x, more), share = each + ((int)blockIdx.x < more ? 1 : 0);
  if (share > 0 && warp == 0) {
    int before = 0;
#pragma unroll 1
    for (int c = 0; before <= start; c += 32) {  // (some sequence holds the start)
      const int u = units_of(c + lane);
      int upto = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      upto += before;
      if (upto - u <= start && start < upto) {
        bars.first_b = c + lane;
        bars.first_off = start - (upto - u);
      }
      before = __shfl_sync(0xffffffffu, upto, 31);
      if (c + 32 >= p.batch) break;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars.tmem;
  bool ok = true;

  if (share == 0) {
    if (tid == 0) p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp < kConvK) {
    if constexpr (kW >= 32) regs_less<S::kRegMisc>();
    if (warp == kProducer || warp == kProducer2) {
      // ------------------------------------------------------------------ producers: a block is one's or the other's in turn
      const int mine_of = warp == kProducer ? 0 : 1;
      int i = 0, st = 0, turn = 0;  // the CTA's block, its stage
      auto copy = [&](int b, int g, int base, int N, int P, int j0, int nb, int np) {
        const int pages = (P + kPage - 1) / kPage;
        // page ids of four blocks at a time, one a lane, a batch ahead of their use
        auto ids_of = [&](int k) -> int {
          const int lp = (j0 + 4 * k) * (kKeys / kPage) + lane;
          return lp < pages ? ld(p.page_table + (size_t)b * p.max_pages + lp) : -1;
        };
        int ids_next = np > 0 ? ids_of(0) : -1, ids = -1;
#pragma unroll 1
        for (int k = 0; k < nb; ++k) {
          if (k < np && (k & 3) == 0) {
            ids = ids_next;
            if (k + 4 < np) ids_next = ids_of((k >> 2) + 1);
          }
          if ((i & 1) == mine_of) {
            if (turn > 0) ok = wait_all(bar(bars.empty[st]), (turn & 1) ^ 1);
            if (!ok) break;
            const uint32_t dst = sb + S::kOffRing + st * kStage, full = bar(bars.full[st]);
            if (k < np) {
              const int page = __shfl_sync(0xffffffffu, ids, (k & 3) * 8 + (lane & 7));
              const bool used = lane < 8 && (j0 + k) * 8 + lane < pages;
              const bool good = used && page >= 0 && page < p.num_pages;
              if (used && !good) report(p.status, SPEC_ERR_PAGE);
              const uint32_t there = __ballot_sync(0xffffffffu, good), bad = __ballot_sync(0xffffffffu, used && !good);
              if (lane == 0) {
                bars.bad_pages[st] = bad;
                tc::mbar_arrive_expect_tx(full, __popc(there) * kRecord);
              }
              __syncwarp();
              if (good) bulk_load(dst + lane * kRecord, p.pool + ((size_t)page * p.hkv + g) * kRecord, kRecord, full);
            } else {
              const int n0 = (j0 + k - (P + kKeys - 1) / kKeys) * kTreeKeys, rows = min(kTreeKeys, N - n0);
              if (lane == 0) tc::mbar_arrive_expect_tx(full, rows * kDim * 4);
              __syncwarp();
              if (lane < rows) {
                const size_t row = ((size_t)(base + n0 + lane) * p.hkv + g) * kDim;
                bulk_load(dst + lane * kDim * 2, p.k_tree + row, kDim * 2, full);
                bulk_load(dst + kTreeV + lane * kDim * 2, p.v_tree + row, kDim * 2, full);
              }
            }
          }
          ++i;
          if (++st == S::kStages) st = 0, ++turn;
        }
      };
      if (warp == kProducer) {  // it also walks the share and says what its runs are
        int left = share, off = bars.first_off, b = bars.first_b, flags = 0;
        int4 meta = make_int4(0, 0, 0, 0);
#pragma unroll 1
        for (int s = 0;; ++s) {
          if (s >= kSegs) ok = wait_all(bar(bars.seg_empty[s % kSegs]), ((s / kSegs) & 1) ^ 1);
          if (!ok) break;
          int base, N, P, nblk, tiles, t, j0;
          while (left > 0) {
            base = ld(p.qo + b), N = ld(p.qo + b + 1) - base, P = ld(p.prefix_len + b);
            nblk = blocks_of(P, N);  // (b counts: first_b does, and so does every next)
            tiles = (N + p.npt - 1) / p.npt;
            if (off >= tiles * p.hkv * (nblk + kTileCost)) {  // the next sequence that counts, 32 at a time
              off = 0;
              ++b;
              while (b < p.batch) {
                const uint32_t some = __ballot_sync(0xffffffffu, units_of(b + lane) > 0);
                if (some != 0) {
                  b += __ffs(some) - 1;
                  break;
                }
                b += 32;
              }
              if (b >= p.batch) left = 0;  // (not reached: the shares count the same blocks)
              continue;
            }
            t = off / (nblk + kTileCost), j0 = off - t * (nblk + kTileCost);
            if (j0 < nblk) break;
            // (the share begins, or goes on, behind a tile's blocks)
            const int rest = min(nblk + kTileCost - j0, left);
            off += rest;
            left -= rest;
          }
          if (left == 0) {
            if (lane == 0) {
              bars.seg[s % kSegs].nb = 0;
              tc::mbar_arrive(bar(bars.seg_full[s % kSegs]));
            }
            break;
          }
          const int g = t / tiles, node0 = (t - g * tiles) * p.npt;
          const int nb = min(nblk - j0, left);
          const int np = max(0, min((P + kKeys - 1) / kKeys - j0, nb));
          const int piece = j0 > 0 ? 0 : nb < nblk ? 1 : -1;
          if (piece == 0) flags |= j0 + nb == nblk ? 3 : 1;
          if (piece == 1) {
            flags |= 4;
            meta.y = b, meta.z = g, meta.w = node0;
          }
          if (lane == 0) {
            bars.seg[s % kSegs] = Seg{b, g, node0, base, N, P, j0, nb, np, piece};
            tc::mbar_arrive(bar(bars.seg_full[s % kSegs]));
          }
          copy(b, g, base, N, P, j0, nb, np);
          if (!ok) break;
          off += nb;
          left -= nb;
        }
        if (lane == 0) {
          meta.x = flags;
          p.meta[blockIdx.x] = meta;
        }
        __syncwarp();
      } else {
#pragma unroll 1
        for (int s = 0;; ++s) {
          ok = wait_all(bar(bars.seg_full[s % kSegs]), (s / kSegs) & 1);
          if (!ok) break;
          const Seg seg = bars.seg[s % kSegs];
          warp_arrive(bar(bars.seg_empty[s % kSegs]));
          if (seg.nb == 0) break;
          copy(seg.b, seg.g, seg.base, seg.N, seg.P, seg.j0, seg.nb, seg.np);
          if (!ok) break;
        }
      }
      if (!ok && lane == 0) {  // given up: leave no copy in flight
        report(p.status, SPEC_ERR_TIMEOUT);
        int zero = 0;
        for (int j = max(0, i - S::kStages); j < i; ++j)
          if ((j & 1) == mine_of) tc::mbar_wait(bar(bars.full[j % S::kStages]), (j / S::kStages) & 1, &zero, kWaitLimit);
      }
      __syncwarp();
    } else if (warp == kMma0 || warp == kMma0 + 1) {
      // ------------------------------------------------------------------ MMA issuers, one a slot
      const int t = warp - kMma0;
      if (elect_one()) {
        constexpr uint32_t kIdQK = tc::idesc_f16(128, kW, 0), kIdPV = tc::idesc_f16(128, kW, 1);
        constexpr uint32_t kIdTreeQK = tc::idesc_bf16(128, kW, 0), kIdTreePV = tc::idesc_bf16(128, kW, 1);
        // (tc::sdesc_sw128's fields but the address: the 14 bits of it are below)
        constexpr uint32_t kDescLo = (16u >> 4) << 16, kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
        const uint32_t ts = tmem + kColS + 64 * t, to = tmem + kColO + 64 * t;
        const uint32_t qh = sb + S::kOffQ + (kDual ? t : 0) * S::kQ, qb = qh + S::kQs * S::kQ;
        const uint32_t pb = sb + S::kOffP + t * 2 * kPBuf;
        int i = 0;       // the CTA's block
        int n_qk = 0, n_pv = 0;  // the slot's blocks
        int n_q = 0;             // its tiles: those of which it has a block
#pragma unroll 1
        for (int s = 0; ok; ++s) {
          ok = wait_one(bar(bars.seg_full[s % kSegs]), (s / kSegs) & 1);
          if (!ok) break;
          const int nb = bars.seg[s % kSegs].nb, np = bars.seg[s % kSegs].np;
          const int keys = bars.seg[s % kSegs].P - bars.seg[s % kSegs].j0 * kKeys;  // prefix keys from the first block on
          tc::mbar_arrive(bar(bars.seg_empty[s % kSegs]));
          if (nb == 0) break;
          constexpr int kStep = kDual ? 1 : 2;
          const int k0 = kDual ? 0 : (i ^ t) & 1;
          if (k0 < nb) {
            ok = wait_one(bar(bars.q_full[t]), n_q & 1);
            if (!ok) break;
            tc::fence_after_sync();
            ++n_q;
          }
          auto qk = [&](int k) {
            const int at = i + k, kb = at & 1;
            ok = ok && wait_one(bar(bars.kt_full[kb]), (at >> 1) & 1);
            if (n_qk > 0) ok = ok && wait_one(bar(bars.s_free[t]), (n_qk & 1) ^ 1);
            if (!ok) return;
            tc::fence_after_sync();
            const uint32_t a = tmem + kColK + 64 * kb;
            const uint32_t d = (k < np ? qh : qb) >> 4, id = k < np ? kIdQK : kIdTreeQK;
            mma<true>(ts, a, d | kDescLo, kDescHi, id);
#pragma unroll
            for (int c = 1; c < 8; ++c)
              mma<false>(ts, a + 8 * c, (d | kDescLo) + (((c >> 2) * S::kQSlab + (c & 3) * 32) >> 4), kDescHi, id);
            tc::mma_commit(bar(bars.s_full[t]));
            tc::mma_commit(bar(bars.kt_free[kb]));
            ++n_qk;
          };
          if (k0 < nb) qk(k0);
#pragma unroll 1
          for (int k = k0; ok && k < nb; k += kStep) {
            if (k + kStep < nb) qk(k + kStep);  // S of the next block while the softmax works on this one
            const int at = i + k, vb = at & 1, buf = n_pv & 1;
            ok = ok && wait_one(bar(bars.vt_full[vb]), (at >> 1) & 1) &&
                 wait_one(bar(bars.p_full[t][buf]), (n_pv >> 1) & 1);
            if (!ok) break;
            tc::fence_after_sync();
            const uint32_t a = tmem + kColV + 64 * vb;
            const uint32_t d = ((pb + buf * kPBuf) >> 4) | kDescLo;
            const int steps = (keys - k * kKeys + 15) >> 4;
            if (k < np && steps >= 8) {
              if (k == k0) mma<true>(to, a, d, kDescHi, kIdPV);
              else mma<false>(to, a, d, kDescHi, kIdPV);
#pragma unroll
              for (int c = 1; c < 8; ++c) mma<false>(to, a + 8 * c, d + ((c * 2048) >> 4), kDescHi, kIdPV);
            } else {
              // the prefix's last block, or a tree block: P's two bf16 terms, two steps of 16 nodes each
              const uint32_t id = k < np ? kIdPV : kIdTreePV, wrap = k < np ? 7 : 1;
#pragma unroll 1
              for (int c = 0; c < (k < np ? steps : 4); ++c) {
                if (k == k0 && c == 0) mma<true>(to, a, d, kDescHi, id);
                else mma<false>(to, a + 8 * (c & wrap), d + ((c * 2048) >> 4), kDescHi, id);
              }
            }
            tc::mma_commit(bar(bars.pv_done[t][buf]));
            tc::mma_commit(bar(bars.vt_free[vb]));
            ++n_pv;
          }
          i += nb;
        }
        if (!ok) report(p.status, SPEC_ERR_TIMEOUT);
        // every product issued has completed before TMEM is released
        tc::mma_commit(bar(bars.fin[t]));
        int zero = 0;
        tc::mbar_wait(bar(bars.fin[t]), 0, &zero, kWaitLimit);
      }
      __syncwarp();
    }
  } else if (warp < kSoft0) {
    // ---------------------------------------------------------------------- converters
    if constexpr (kW >= 32) regs_less<S::kRegConv>();
    const bool isv = warp >= kConvV;
    const int x = tid & 127;  // K: the token, V: the element
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // a warp of V's: the scales of its two groups, fp16 [page][group][16 tokens]
    uint4* vscale = reinterpret_cast<uint4*>(smem + S::kOffScale) + (isv ? warp - kConvV : 0) * 32;
    const int turn_of = kConv == 2 ? (warp - (isv ? kConvV : kConvK)) >> 2 : 0;  // the blocks of this group: i % 2
    int i = 0, st = 0, turn = 0;
#pragma unroll 1
    for (int s = 0; ok; ++s) {
      ok = wait_all(bar(bars.seg_full[s % kSegs]), (s / kSegs) & 1);
      if (!ok) break;
      const Seg& seg = bars.seg[s % kSegs];
      const int nb = seg.nb, np = seg.np, keys = seg.P - seg.j0 * kKeys;
      const int nodes = seg.N - max(0, seg.j0 - (seg.P + kKeys - 1) / kKeys) * kTreeKeys;  // from the first tree block on
      warp_arrive(bar(bars.seg_empty[s % kSegs]));
      if (nb == 0) break;
#pragma unroll 1
      for (int k = 0; k < nb; ++k, ++i) {
        if (kConv == 2 && (i & 1) != turn_of) {
          if (++st == S::kStages) st = 0, ++turn;
          continue;
        }
        ok = wait_all(bar(bars.full[st]), turn & 1);
        if (!ok) break;
        const uint8_t* src = smem + S::kOffRing + st * kStage;
        const int tb = i & 1;
        uint64_t& tfull = isv ? bars.vt_full[tb] : bars.kt_full[tb];
        uint64_t& tfree = isv ? bars.vt_free[tb] : bars.kt_free[tb];
        const uint32_t to = tmem + (isv ? kColV : kColK) + 64 * tb + lanes;
        if (k < np && !isv) {
          const uint32_t bad = bars.bad_pages[st];
          const uint8_t* rec = src + (x >> 4) * kRecord;
          const uint32_t none = bad != 0 && ((bad >> (x >> 4)) & 1) ? 0u : 0xFFFFu;  // a page outside the pool: zeros
          if (i >= 2) ok = wait_all(bar(tfree), ((i >> 1) & 1) ^ 1);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {  // a part: 32 elements, two groups
            const uint4 c = *reinterpret_cast<const uint4*>(rec + q * 256 + (x & 15) * 16);
            const uint32_t sc = *reinterpret_cast<const uint16_t*>(rec + kOffKs + (x & 15) * 8 + 2 * q) & none;
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            uint32_t h[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t f = half2_of_scales((uint16_t)__byte_perm(sc, 0, e < 2 ? 0x00 : 0x11));
              h[4 * e] = hmul2(half2_of_codes<0>(w[e]), f);
              h[4 * e + 1] = hmul2(half2_of_codes<1>(w[e]), f);
              h[4 * e + 2] = hmul2(half2_of_codes<2>(w[e]), f);
              h[4 * e + 3] = hmul2(half2_of_codes<3>(w[e]), f);
            }
            tc::tmem_st16_u(to + 16 * q, h);
          }
          warp_arrive(bar(bars.empty[st]));
        } else if (k < np) {
          const int valid = keys - k * kKeys;  // tokens of the block (may be more)
          // the scales of the warp's two groups as fp16, 8 tokens a lane, once for the warp's 32 elements
          {
            const int pg = lane >> 2, half = lane & 3;
            uint2 f = *reinterpret_cast<const uint2*>(src + pg * kRecord + kOffVs + (warp & 3) * 32 + half * 8);
            const uint32_t bad = bars.bad_pages[st];
            if (bad != 0 || valid < kKeys) {  // tokens past the prefix, pages outside the pool: scales of 0
              const int n = ((bad >> pg) & 1) ? 0 : valid - pg * kPage - (half & 1) * 8;
              f.x = n >= 4 ? f.x : n <= 0 ? 0u : f.x & (0xFFFFFFFFu >> (32 - 8 * n));
              f.y = n >= 8 ? f.y : n <= 4 ? 0u : f.y & (0xFFFFFFFFu >> (64 - 8 * n));
            }
            __syncwarp();  // (the block before's have been read)
            vscale[lane] = make_uint4(half2_of_scales((uint16_t)f.x), half2_of_scales((uint16_t)(f.x >> 16)),
                                      half2_of_scales((uint16_t)f.y), half2_of_scales((uint16_t)(f.y >> 16)));
            __syncwarp();
          }
          if (i >= 2) ok = wait_all(bar(tfree), ((i >> 1) & 1) ^ 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint4* f = vscale + (lane >> 4) * 2;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {  // two pages
            uint32_t h[16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint2 w = *reinterpret_cast<const uint2*>(src + (2 * q + e) * kRecord + kOffV + x * 8);
              const uint4 lo = f[(2 * q + e) * 4], hi = f[(2 * q + e) * 4 + 1];
              h[8 * e] = hmul2(half2_of_codes<0>(w.x), lo.x), h[8 * e + 1] = hmul2(half2_of_codes<1>(w.x), lo.y);
              h[8 * e + 2] = hmul2(half2_of_codes<2>(w.x), lo.z), h[8 * e + 3] = hmul2(half2_of_codes<3>(w.x), lo.w);
              h[8 * e + 4] = hmul2(half2_of_codes<0>(w.y), hi.x), h[8 * e + 5] = hmul2(half2_of_codes<1>(w.y), hi.y);
              h[8 * e + 6] = hmul2(half2_of_codes<2>(w.y), hi.z), h[8 * e + 7] = hmul2(half2_of_codes<3>(w.y), hi.w);
            }
            tc::tmem_st16_u(to + 16 * q, h);
          }
          warp_arrive(bar(bars.empty[st]));
        } else {
          // a tree block: bf16 rows as they are, K's a node a lane (the same 32 in each warp's quarter), V's turned; V's
          // elements that are not finite become 0 (a weight of 0 times either would reach rows whose mask leaves the
          // node out) and the node is noted
          const int rows = min(kTreeKeys, nodes - (k - np) * kTreeKeys);
          if (i >= 2) ok = wait_all(bar(tfree), ((i >> 1) & 1) ^ 1);
          if (!ok) break;
          tc::fence_after_sync();
          if (!isv) {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t h[16];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint4 v = lane < rows ? *reinterpret_cast<const uint4*>(src + lane * kDim * 2 + q * 64 + e * 16)
                                            : make_uint4(0, 0, 0, 0);
                h[4 * e] = v.x, h[4 * e + 1] = v.y, h[4 * e + 2] = v.z, h[4 * e + 3] = v.w;
              }
              __syncwarp();
              tc::tmem_st16_u(to + 16 * q, h);
            }
          } else {
            uint32_t h[16], bad = 0;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(src + kTreeV) + x;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              uint32_t lo = 2 * e < rows ? v[2 * e * kDim] : 0u, hi = 2 * e + 1 < rows ? v[(2 * e + 1) * kDim] : 0u;
              if ((lo & 0x7F80u) == 0x7F80u) lo = 0, bad |= 1u << (2 * e);
              if ((hi & 0x7F80u) == 0x7F80u) hi = 0, bad |= 2u << (2 * e);
              h[e] = lo | (hi << 16);
            }
            tc::tmem_st16_u(to, h);
            bad = __reduce_or_sync(0xffffffffu, bad);
            if (lane == 0) bars.bad_nodes[tb][warp & 3] = bad;
          }
          warp_arrive(bar(bars.empty[st]));
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        warp_arrive(bar(tfull));
        if (++st == S::kStages) st = 0, ++turn;
      }
    }
    if (!ok && lane == 0) report(p.status, SPEC_ERR_TIMEOUT);
  } else {
    // ---------------------------------------------------------------------- softmax
    if constexpr (kW >= 32) regs_more<S::kRegSoft>();
    const int group = (warp - kSoft0) >> 2, slot = group / kG, cb = group % kG * kC;  // cb: the group's first row
    const int x = tid & 127, wq = warp & 3;  // x: the token of S, the element of O
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t ts = tmem + kColS + 64 * slot + cb + lanes, to = tmem + kColO + 64 * slot + cb + lanes;
    // of the group's rows
    float4* rowinfo = reinterpret_cast<float4*>(smem + S::kOffRow) + (slot * kW + cb) / 2;
    float* red = reinterpret_cast<float*>(smem + S::kOffRed) + group * 32 * kC;
    float* myred = red + (8 * wq + (lane >> 2)) * kC + 2 * (lane & 3);  // of the thread's four tokens, its first two rows
    float* fac = reinterpret_cast<float*>(smem + S::kOffDelta) + slot * kW + cb;  // (what off grew by: 2 kW behind)
    float* tsum = reinterpret_cast<float*>(smem + S::kOffTree) + slot * kW + cb;
    const bool has = 8 * wq < kC;  // the warp has rows of a tree block
    // of the tile's
    float2* sums = reinterpret_cast<float2*>(smem + S::kOffSum);
    float2* fin = reinterpret_cast<float2*>(smem + S::kOffFin);
    int* orow = reinterpret_cast<int*>(smem + S::kOffOut);
    int* mrow = reinterpret_cast<int*>(smem + S::kOffMask);
    const int row0 = (kDual ? slot * kW : 0) + cb;  // the group's first row within the tile
    uint8_t* pbuf = smem + S::kOffP + slot * 2 * kPBuf;
    const int mine = 2 + group;  // the group's barrier; 1: all groups'
    // the thread's part of q: kParts threads a row, kQv pieces of 8 elements each
    constexpr int kParts = (kDual ? kSoft / 2 : kSoft) / kW, kQv = 16 / kParts;
    const int qt = group % (kDual ? kG : 4) * 128 + x, qr = qt / kParts, qc = (qt % kParts) * kQv;
    const uint32_t s_full = bar(bars.s_full[slot]), s_free = bar(bars.s_free[slot]), p_full = bar(bars.p_full[slot][0]);
    uint32_t tries = kTries;
    int n = 0;  // the slot's block
    int i = 0;  // the CTA's block
    const int q_node = ((kDual ? slot * kW : 0) + qr) / p.G, q_head = (kDual ? slot * kW : 0) + qr - q_node * p.G;
#pragma unroll 1
    for (int s = 0;; ++s) {
      const Seg& seg = bars.seg[s % kSegs];
      if (s == 0) {  // (later ones: waited for, and their q asked for, ahead of the result before)
        ok = wait_all(bar(bars.seg_full[0]), 0);
        if (named_any(1, kSoft, !ok)) {
          ok = false;
          break;
        }
      }
      const int nb = seg.nb, np = seg.np;
      if (nb == 0) break;
      // ---- q of the tile: fp16 and bf16 rows, their factors, where the rows go
      {
        uint4 qv[kQv];
        int q_at, q_m;  // the row's place in q and out (and the mask's rows), -1: none
        {
          const int node = seg.node0 + q_node;
          const bool valid = q_node < p.npt && node < seg.N;
          q_m = valid ? seg.base + node : -1;
          q_at = valid ? q_m * p.hq + seg.g * p.G + q_head : -1;
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)max(q_at, 0) * kDim) + qc;
#pragma unroll
          for (int e = 0; e < kQv; ++e) qv[e] = valid ? ld(src + e) : make_uint4(0, 0, 0, 0);
        }
        const int r = (kDual ? slot * kW : 0) + qr;
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < kQv; ++e) {
          const uint4 v = qv[e];
          m = __vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
          m = __vmaxu2(m, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
        }
        m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
        for (int o = kParts / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        // up * 2^(e - 141) = 1: q * up has its largest element in [2^14, 2^15). Both factors are made of two
        // powers of two, as one may leave fp32's range.
        const int sh = 141 - max((int)(m >> 7), 1);
        const float up0 = __uint_as_float((uint32_t)(127 + sh / 2) << 23);
        const float up1 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
        uint8_t* dst = smem + S::kOffQ + (kDual ? slot : 0) * S::kQ;
#pragma unroll
        for (int e = 0; e < kQv; ++e) {
          const int c = qc + e;
          const uint4 v = qv[e];
          const uint32_t off = (c >> 3) * S::kQSlab + swz(qr, c & 7);
          *reinterpret_cast<uint4*>(dst + S::kQs * S::kQ + off) = v;
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t h[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            h[u] = pack_f16x2(__uint_as_float(w[u] << 16) * up0 * up1, __uint_as_float(w[u] & 0xFFFF0000u) * up0 * up1);
          *reinterpret_cast<uint4*>(dst + off) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        if (qt % kParts == 0) {
          const float f = p.scale_log2 * head_scale(p.kv_scale, 0, p.hkv, seg.g) *
                          __uint_as_float((uint32_t)(127 - sh / 2) << 23) *
                          __uint_as_float((uint32_t)(127 - (sh - sh / 2)) << 23);
          for (int to_slot = kDual ? slot : 0; to_slot < (kDual ? slot + 1 : 2); ++to_slot) {
            float* info = reinterpret_cast<float*>(smem + S::kOffRow) + to_slot * 2 * kW + (qr >> 1) * 4 + (qr & 1);
            info[0] = f;
            info[2] = 0.f;
          }
          orow[r] = q_at;
          mrow[r] = q_m;
        }
        if (x < kC) tsum[x] = 0.f;
      }
      tc::fence_proxy_async_smem();
      if constexpr (kDual) {
        warp_arrive(bar(bars.q_full[slot]));
        named_sync(6 + slot, 128 * kG);
      } else {
        // (only to a slot that has a block of the tile: an issuer without one waits for nothing else here, and a phase
        // that it has not seen when the next is over would never be seen)
        __syncwarp();
        tc::mbar_arrive_if(lane == 0 && nb > (i & 1), bar(bars.q_full[0]));
        tc::mbar_arrive_if(lane == 0 && nb > ((i & 1) ^ 1), bar(bars.q_full[1]));
        named_sync(1, kSoft);
      }
      // ---- blocks
      // A thread has four tokens, lane / 4 + 8 e, and of every 8 rows two: their factors and offs, and the sums of its
      // tokens' P, stay in registers.
      constexpr int kJ = kC / 8;
      float2 mul[kJ], off[kJ], l[kJ];
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const float4 f = rowinfo[4 * j + (lane & 3)];
        mul[j] = make_float2(f.x, f.y), off[j] = make_float2(0.f, 0.f), l[j] = make_float2(0.f, 0.f);
      }
      bool row_set = false;  // row x of the slot has seen a key: its off is set
      constexpr int kStep = kDual ? 1 : 2;
      const int k0 = kDual ? 0 : (i ^ slot) & 1;
      int left = seg.P - (seg.j0 + k0) * kKeys;  // prefix keys from the block on
#pragma unroll 1
      for (int k = k0; k < nb; k += kStep, ++n, left -= kStep * kKeys) {
        const bool tree = k >= np, first = k == k0;
        // of a tree block: the mask words of the warp's 8 rows, one a lane, and V's head scale, on their way while S is
        uint32_t words = 0;
        bool node_is = false;
        float v_scale = 1.f;
        if (tree) {
          const int tb = max(0, seg.j0 - (seg.P + kKeys - 1) / kKeys) + k - np;
          node_is = lane < seg.N - tb * kTreeKeys;
          const int m = has && lane < 8 ? mrow[row0 + 8 * wq + lane] : -1;
          if (m >= 0) words = ld(reinterpret_cast<const uint32_t*>(p.mask + (size_t)m * p.mask_words) + tb);
          v_scale = head_scale(p.kv_scale, 1, p.hkv, seg.g);
        }
        wait_on(s_full, n & 1, tries);
        tc::fence_after_sync();
        // ---- off of the rows whose largest y (red, `rows` rows of it) passes the limit, or that had seen no key: the
        // largest becomes 2^5; what was summed before is scaled. What off grew by, in `fac` behind the factors.
        auto move = [&](int rows) {
          named_sync(mine, 128);
          bool moved = false;
          if (x < kC) {
            float* info = reinterpret_cast<float*>(rowinfo) + (x >> 1) * 4 + (x & 1);
            float m = red[x];
#pragma unroll 4
            for (int w = 1; w < rows; ++w) m = fmaxf(m, red[w * kC + x]);
            const float d = m > -INFINITY && (!row_set || m > kLimit) ? kShift - m : 0.f;
            row_set |= m > -INFINITY;
            const float f = ex2_approx(fminf(d, 0.f));  // (off of a row that has a sum only falls)
            info[2] += d;
            fac[x] = f;
            fac[2 * kW + x] = d;
            tsum[x] *= f;
            moved = d != 0.f;
          }
          if (!named_any(mine, 128, moved)) return;
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const float4 f = rowinfo[4 * j + (lane & 3)];
            off[j] = make_float2(f.z, f.w);
            l[j] = fmul2(l[j], *reinterpret_cast<const float2*>(fac + 8 * j + 2 * (lane & 3)));
          }
          if (first) return;
          wait_on(bar(bars.pv_done[slot][(n - 1) & 1]), ((n - 1) >> 1) & 1, tries);  // O up to the block before
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < kC; c += 8) {
            float o[8];
            tmem_ld8(to + c, o);
            tc::tmem_wait_ld();
            uint32_t w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = __float_as_uint(o[u] * fac[c + u]);
            tc::tmem_st8_u(to + c, w);
          }
          tc::tmem_wait_st();
        };
        // (P's buffer is free: the PV of two blocks ago was issued before this block's QK, by the same thread, so S came
        // after it)
        const uint32_t row = tc::smem_u32(pbuf) + (n & 1) * kPBuf + x * 128;
        if (!tree) {
          constexpr int kHalf = kC / 2;
          float y[kC];  // [tokens 0, 8 | 16, 24][j][token][row]
          tmem_ld_frag<kC>(ts, y);
          tmem_ld_frag<kC>(ts + (16u << 16), y + kHalf);
          tc::tmem_wait_ld();
          tc::fence_before_sync();
          float top = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float* v = y + h * kHalf + 4 * j + 2 * e;
                const float2 z = ffma2(make_float2(v[0], v[1]), mul[j], off[j]);
                v[0] = z.x, v[1] = z.y;
              }
          if (left < kKeys) {  // keys past the prefix (what they hold may be NaN)
            const int valid = left - 32 * wq - (lane >> 2);  // from the thread's first on
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const bool past = 16 * h + 8 * e >= valid;
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                  float* v = y + h * kHalf + 4 * j + 2 * e;
                  v[0] = past ? -INFINITY : v[0], v[1] = past ? -INFINITY : v[1];
                }
              }
          }
#pragma unroll
          for (int c = 0; c < kC; c += 2) top = fmax3(top, y[c], y[c + 1]);
          // Whether a row passes the limit in any of the slot's warps: each says so before it lets S go, and asks when
          // its exponentials are done, so that no warp waits for the slowest. (A tile's first block: off is yet to be
          // found.)
          if (__any_sync(0xffffffffu, top > kLimit) && lane == 0) bars.flag[group][n & 1] = n;
          tc::mbar_arrive_if(lane == 0, s_free);
          auto shift = [&] {  // y after a move
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              const float *v = y + 4 * j, *w = v + kHalf;
              *reinterpret_cast<float2*>(myred + 8 * j) =
                  make_float2(fmaxf(fmaxf(v[0], v[2]), fmaxf(w[0], w[2])), fmaxf(fmaxf(v[1], v[3]), fmaxf(w[1], w[3])));
            }
            move(32);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              const float2 d = *reinterpret_cast<const float2*>(fac + 2 * kW + 8 * j + 2 * (lane & 3));
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float* v = y + h * kHalf + 4 * j + 2 * e;
                  const float2 z = fadd2(make_float2(v[0], v[1]), d);
                  v[0] = z.x, v[1] = z.y;
                }
            }
          };
          float2 sum[kJ];
          auto weights = [&] {  // P, and its sums over the thread's tokens
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float* v = y + (e >> 1) * kHalf + 4 * j + 2 * (e & 1);
                const float2 z = make_float2(ex2_approx(v[0]), ex2_approx(v[1]));
                sum[j] = e == 0 ? z : fadd2(sum[j], z);
                w[e] = pack_f16x2(z.x, z.y);
              }
              stmatrix4(row + (((cb / 8 + j) ^ (x & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
          };
          if (__builtin_expect(first, 0)) shift();
          weights();
          if (!first) {
            wait_on(s_free, n & 1, tries);
            if (__builtin_expect(*reinterpret_cast<volatile int*>(&bars.flag[group][n & 1]) == n, 0)) {
              shift();
              weights();
            }
          }
#pragma unroll
          for (int j = 0; j < kJ; ++j) l[j] = fadd2(l[j], sum[j]);
        } else {
          // a tree block: its nodes stand on the lanes of each warp's quarter; a warp takes 8 rows (of 16 the last two none)
          float r[8];
          if (has) {
            float keep = -INFINITY;
            tmem_ld8(ts + 8 * wq, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float o = reinterpret_cast<const float*>(rowinfo + ((8 * wq + u) >> 1))[2 + (u & 1)];
              const uint32_t see = __shfl_sync(0xffffffffu, words, u);
              r[u] = ((see >> lane) & 1u) && node_is ? fmaf(r[u], p.scale_log2, o) : -INFINITY;
              const float m = redux_max(r[u]);
              if (lane == u) keep = m;
            }
            if (lane < 8) red[8 * wq + lane] = keep;
          }
          tc::fence_before_sync();
          warp_arrive(s_free);
          move(1);
          // V's converters have noted the block's nodes before the barrier that they arrive on. (Its phase before
          // this one is over once the slot's PV of the block before is done: then the parity is this block's.)
          if (!first) wait_on(bar(bars.pv_done[slot][(n - 1) & 1]), ((n - 1) >> 1) & 1, tries);
          wait_on(bar(bars.vt_full[(i + k) & 1]), ((i + k) >> 1) & 1, tries);
          if (has) {
            const uint32_t* w = bars.bad_nodes[(i + k) & 1];
            const bool bad = ((w[0] | w[1] | w[2] | w[3]) >> lane) & 1u;
            const float inv = 1.f / v_scale;  // (O is in units of V's head scale)
            uint8_t* dst = pbuf + (n & 1) * kPBuf;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float z = r[u] + fac[2 * kW + 8 * wq + u];
              r[u] = ex2_approx(z > kLimit ? kLimit : z);  // (a NaN stays)
            }
            if (__any_sync(0xffffffffu, bad)) {  // a node whose V holds an infinity or NaN makes the rows that see it NaN
#pragma unroll
              for (int u = 0; u < 8; ++u)
                if (((__shfl_sync(0xffffffffu, words, u) >> lane) & 1u) && node_is && bad) r[u] = __int_as_float(0x7FC00000);
            }
#pragma unroll
            for (int u = 0; u < 8; u += 2) {
              const float a = r[u] * inv, b = r[u + 1] * inv;
              hi[u >> 1] = pack_bf16x2(a, b);
              lo[u >> 1] = pack_bf16x2(a - __uint_as_float(hi[u >> 1] << 16), b - __uint_as_float(hi[u >> 1] & 0xFFFF0000u));
            }
            *reinterpret_cast<uint4*>(dst + swz(lane, (cb >> 3) + wq)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + swz(32 + lane, (cb >> 3) + wq)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            // row sums over the lanes: three steps halve a lane's columns, to the one of its bits 4 to 2
#pragma unroll
            for (int o = 16, h = 4; o > 2; o >>= 1, h >>= 1)
#pragma unroll
              for (int u = 0; u < h; ++u) {
                const bool up = (lane & o) != 0;
                const float give = up ? r[u] : r[u + h], have = up ? r[u + h] : r[u];
                r[u] = have + __shfl_xor_sync(0xffffffffu, give, o);
              }
            r[0] += __shfl_xor_sync(0xffffffffu, r[0], 2);
            r[0] += __shfl_xor_sync(0xffffffffu, r[0], 1);
            if ((lane & 3) == 0) tsum[8 * wq + (lane >> 2)] += r[0];
          }
        }
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        warp_arrive(p_full + 8 * (n & 1));
      }
      // the next tile's q, on its way to the L2 while this one's result is written (in registers it would not fit beside it)
      wait_on(bar(bars.seg_full[(s + 1) % kSegs]), ((s + 1) / kSegs) & 1, tries);
      if (tries != 0) {
        const Seg& next = bars.seg[(s + 1) % kSegs];
        const int node = next.node0 + q_node;
        if (next.nb > 0 && q_node < p.npt && node < next.N)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + ((size_t)(next.base + node) * p.hq + next.g * p.G + q_head) * kDim + qc * 8));
      }
      if (nb > k0) wait_on(bar(bars.pv_done[slot][(n - 1) & 1]), ((n - 1) >> 1) & 1, tries);
      if (named_any(1, kSoft, tries == 0)) {
        ok = false;
        break;
      }
      // ---- the tile's (or the piece's) result
      // row sums over the tokens
#pragma unroll
      for (int j = 0; j < kJ; ++j) *reinterpret_cast<float2*>(myred + 8 * j) = l[j];
      named_sync(mine, 128);
      if (x < kC) {
        float sum = tsum[x];
#pragma unroll 4
        for (int w = 0; w < 32; ++w) sum += red[w * kC + x];
        sums[slot * kW + cb + x] = make_float2(reinterpret_cast<float*>(rowinfo)[(x >> 1) * 4 + 2 + (x & 1)], sum);
      }
      if (!kDual) named_sync(1, kSoft);
      const int piece = seg.piece;
      {
        const int r = row0 + x;
        if (x < kC && (kDual || slot == 0)) {
          float off, sum, w0 = 1.f, w1 = 0.f;
          if constexpr (kDual) {
            const float2 a = sums[slot * kW + cb + x];
            off = a.x, sum = a.y;
          } else {
            const float2 a = sums[cb + x], b = sums[kW + cb + x];
            // the slot whose rows stand higher (the smaller off) gives the scale; one without weights has none
            off = a.y == 0.f ? b.x : b.y == 0.f ? a.x : fminf(a.x, b.x);
            w0 = a.y == 0.f ? 0.f : ex2_approx(off - a.x);
            w1 = b.y == 0.f ? 0.f : ex2_approx(off - b.x);
            sum = a.y * w0 + b.y * w1;
          }
          const float inv = sum == 0.f ? 0.f : head_scale(p.kv_scale, 1, p.hkv, seg.g) / sum;
          fin[r] = make_float2(w0 * inv, w1 * inv);
          const float lse2 = sum == 0.f ? -INFINITY : log2f(sum) - off;
          if (piece >= 0) p.part_lse[((size_t)blockIdx.x * 2 + piece) * S::kR + r] = lse2;
          else if (p.lse != nullptr && orow[r] >= 0) p.lse[orow[r]] = lse2 * kLn2;
        }
      }
      if (kDual) named_sync(mine, 128);  // (a group's rows are its own)
      else named_sync(1, kSoft);
      warp_arrive(bar(bars.seg_empty[s % kSegs]));
      {
        tc::fence_after_sync();
        // columns of this thread: of its group's rows, or its share of both slots'
        constexpr int kCols = kDual ? kC : kC / 2;
        const int c0 = kDual ? cb : group * kCols;
        const uint32_t o0 = tmem + kColO + (kDual ? 64 * slot : 0) + lanes, o1 = tmem + kColO + 64 + lanes;
        const bool have0 = kDual || nb > (i & 1), have1 = !kDual && nb > ((i & 1) ^ 1);
        float* part = p.part_o + ((size_t)blockIdx.x * 2 + max(piece, 0)) * S::kR * kDim + x;
        __nv_bfloat16* out = p.out + x;
#pragma unroll 1
        for (int c = c0; c < c0 + kCols; c += 8) {
          float a[8], b[8];
          tmem_ld8(o0 + c, a);
          if (!kDual) tmem_ld8(o1 + c, b);
          tc::tmem_wait_ld();
          const int r0 = (kDual ? slot * kW : 0) + c;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float2 w = fin[r0 + u];
            a[u] = have0 && w.x != 0.f ? a[u] * w.x : 0.f;
            if (!kDual && have1 && w.y != 0.f) a[u] = fmaf(b[u], w.y, a[u]);
          }
          if (piece >= 0) {
#pragma unroll
            for (int u = 0; u < 8; ++u) part[(r0 + u) * kDim] = a[u];
          } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int at = orow[r0 + u];
              if (at >= 0) out[(size_t)at * kDim] = __float2bfloat16_rn(a[u]);
            }
          }
        }
        tc::fence_before_sync();
      }
      i += nb;
      // (both slots' O have been read, and the tables, before the next tile's q and products)
      named_sync(1, kSoft);
    }
    if (!ok && lane == 0) report(p.status, SPEC_ERR_TIMEOUT);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------- the join of a tile's pieces

struct MergeParams {
  const int4* meta;
  const float* part_lse;
  const float* part_o;
  const int32_t* qo;
  int ctas, R, hq, G, npt;
  __nv_bfloat16* out;
  float* lse;
};
constexpr int kMergeRows = 8;

// out = sum_s 2^(lse_s - M) O_s / sum_s 2^(lse_s - M) over the pieces of a tile: the last of the CTA where the tile
// begins, then the first of each CTA that follows until one ends the tile. A warp a row, four columns a lane.
__global__ void __launch_bounds__(32 * kMergeRows) attn_kv4_merge_kernel(const MergeParams p) {
  pdl_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31, r = blockIdx.y * kMergeRows + (threadIdx.x >> 5);
  const int4 m = ld(p.meta + c0);
  // (of the first 32 CTAs, one a lane: loaded before it is known whether a tile begins here)
  int f = c0 + lane < p.ctas ? ld(&p.meta[c0 + lane].x) : 0;
  float s = c0 + lane < p.ctas ? ld(p.part_lse + ((size_t)(c0 + lane) * 2 + (lane == 0 ? 1 : 0)) * p.R + r) : 0.f;
  if (!(m.x & 4) || r >= p.npt * p.G) return;
  const int base = ld(p.qo + m.y), N = ld(p.qo + m.y + 1) - base, node = m.w + r / p.G;
  if (node >= N) return;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int from = c0;; from += 32) {  // 32 CTAs at a time, one a lane
    const int c = from + lane;
    if (from > c0) {
      f = c < p.ctas ? ld(&p.meta[c].x) : 0;
      s = c < p.ctas ? ld(p.part_lse + (size_t)c * 2 * p.R + r) : 0.f;
    } else if (lane == 0) {
      f = 0;
    }
    const uint32_t ends = __ballot_sync(0xffffffffu, (f & 2) != 0);
    const int n = ends != 0 ? __ffs(ends) : 32;  // lanes that belong to the tile (a CTA without a share has no piece)
    s = lane < n && (c == c0 || (f & 1)) ? s : -INFINITY;
    const float top = fmaxf(M, redux_max(s));
    const float w = s == -INFINITY ? 0.f : ex2_approx(s - top), was = M == -INFINITY ? 0.f : ex2_approx(M - top);
    M = top;
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    L = fmaf(L, was, sum);
    acc = make_float4(acc.x * was, acc.y * was, acc.z * was, acc.w * was);
#pragma unroll 1
    for (int j = 0; j < n; j += 8) {
      float4 o[8];
      float wj[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        wj[u] = __shfl_sync(0xffffffffu, w, (j + u) & 31);
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j + u < n && wj[u] != 0.f)
          o[u] = ld(reinterpret_cast<const float4*>(p.part_o + (((size_t)(from + j + u) * 2 + (from + j + u == c0 ? 1 : 0)) * p.R + r) * kDim) + lane);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (j + u >= n) wj[u] = 0.f;
        acc = make_float4(fmaf(o[u].x, wj[u], acc.x), fmaf(o[u].y, wj[u], acc.y), fmaf(o[u].z, wj[u], acc.z),
                          fmaf(o[u].w, wj[u], acc.w));
      }
    }
    if (ends != 0 || from + 32 >= p.ctas) break;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t row = (size_t)(base + node) * p.hq + m.z * p.G + r % p.G;
  *reinterpret_cast<uint2*>(p.out + row * kDim + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && p.lse != nullptr) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ---------------------------------------------------------------------------------- host

// Rows of a tile: the smallest of 16, 32, 64, 128 that holds a sequence's rows of a KV head (or 128).
static int rows_of(int max_nodes, int G) {
  const long rows = (long)max_nodes * G;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

struct Ws {
  size_t lse, o, total;
};
static Ws ws_of(int ctas, int R) {
  Ws w;
  w.lse = align_up(sizeof(int4) * ctas, 256);
  w.o = align_up(w.lse + sizeof(float) * ctas * 2 * R, 256);
  w.total = w.o + sizeof(float) * ctas * 2 * R * kDim;
  return w;
}

constexpr long kMostBlocks = 0x3FFFFFFF;  // of a call: their sum is an int
static long blocks_of_all(int batch, int max_nodes, int hkv, int max_prefix, int R, int G) {
  return (long)batch * hkv * ceil_div(max_nodes, R / G) *
         (ceil_div(max_prefix, kKeys) + ceil_div(max_nodes, kTreeKeys) + tile_cost(R));
}
// CTAs: one an SM, and no more than there can be blocks.
static int ctas_of(int batch, int max_nodes, int hkv, int max_prefix, int R, int G) {
  const long blocks = blocks_of_all(batch, max_nodes, hkv, max_prefix, R, G);
  return (int)(blocks < sm_count() ? (blocks < 1 ? 1 : blocks) : sm_count());
}

template <int kW, bool kDual>
static cudaError_t launch(const Params& p, int ctas, cudaStream_t stream) {
  using S = Shape<kW, kDual>;
  static PerDevice smem_set;
  if (per_device(smem_set, [](int) {
        return cudaFuncSetAttribute(attn_kv4_kernel<kW, kDual>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) ==
                       cudaSuccess
                   ? 1
                   : 0;
      }) == 0)
    return cudaErrorUnknown;
  return launch_pdl(attn_kv4_kernel<kW, kDual>, dim3(ctas), dim3(S::kThreads), S::kSmem, stream, p);
}

}  // namespace a4

size_t attn_kv4_ws_bytes(int batch, int max_nodes, int hq, int hkv, int max_prefix) {
  using namespace a4;
  const int R = rows_of(max_nodes, hq / hkv);
  if (blocks_of_all(batch, max_nodes, hkv, max_prefix, R, hq / hkv) > kMostBlocks) return 0;
  return ws_of(ctas_of(batch, max_nodes, hkv, max_prefix, R, hq / hkv), R).total;
}

int launch_attn_kv4(const void* q, const uint8_t* pool, const float* kv_scale, int num_pages, const int32_t* page_table,
                    int max_pages, const int32_t* prefix_len, int max_prefix, const void* k_tree, const void* v_tree,
                    const uint64_t* mask, const int32_t* qo, int batch, int total_nodes, int max_nodes, int hq, int hkv,
                    float sm_scale, void* out, float* lse, void* ws, int32_t* status, cudaStream_t stream) {
  using namespace a4;
  const int G = hq / hkv, R = rows_of(max_nodes, G), npt = R / G;
  if (blocks_of_all(batch, max_nodes, hkv, max_prefix, R, G) > kMostBlocks) return SPEC_ERR_UNSUPPORTED;
  const int ctas = ctas_of(batch, max_nodes, hkv, max_prefix, R, G);
  const Ws w = ws_of(ctas, R);
  uint8_t* wb = static_cast<uint8_t*>(ws);
  const Params p{static_cast<const __nv_bfloat16*>(q), pool, kv_scale, page_table, max_pages, num_pages, prefix_len,
                 max_prefix, static_cast<const __nv_bfloat16*>(k_tree), static_cast<const __nv_bfloat16*>(v_tree), mask,
                 (max_nodes + 63) >> 6, max_nodes, qo, batch, total_nodes, hq, hkv, G, npt, sm_scale * kLog2e,
                 static_cast<__nv_bfloat16*>(out), lse, reinterpret_cast<int4*>(wb), reinterpret_cast<float*>(wb + w.lse),
                 reinterpret_cast<float*>(wb + w.o), status};
  const cudaError_t e = R == 16   ? launch<16, false>(p, ctas, stream)
                        : R == 32 ? launch<32, false>(p, ctas, stream)
                        : R == 64 ? launch<64, false>(p, ctas, stream)
                                  : launch<64, true>(p, ctas, stream);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  const MergeParams m{p.meta, p.part_lse, p.part_o, qo, ctas, R, hq, G, npt, p.out, lse};
  if (launch_pdl(attn_kv4_merge_kernel, dim3(ctas, R / kMergeRows), dim3(32 * kMergeRows), 0, stream, m) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
