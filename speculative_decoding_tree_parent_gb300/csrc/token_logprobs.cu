// Log probabilities of given tokens, their rank, the entropy and the top alternatives, from rows of logits.
//
// With y_v = (x_v - M) / T, M the row's largest logit: Z = sum e^y, lp(t) = y_t - ln Z, H = ln Z - sum e^y y / Z.
// Every term of both sums is at most 1 in magnitude and of one sign, so nothing cancels; Z is summed with its remainder, since
// of a token that is nearly certain ln Z is what is left of Z beside 1. rank(t) = 1 + the tokens
// before t in the order (larger logit, lower id on ties); the alternatives are the first of that order.
//
// One pass over the row: each thread keeps the running maximum, Z and sum e^y y of its elements (fp32;
// rescaled where the maximum moves), counts the tokens before t, and notes the largest logit of every
// segment (the elements it takes in one or more turns of the loop) in shared memory. The k-th largest of the threads'
// maxima is a bound that at least k elements reach; the few segments that reach it are read a second time (from
// the L2), and the elements that do are sorted by counting.
//
// Bound: HBM for many rows (a row is read once; of bf16 neither is full: HBM at 68%, the issue of instructions at 66%);
// latency for a few.
// Layout: a cluster of 1 to 8 CTAs a row, so that a few rows still use many SMs; each writes its part into the first CTA's
// shared memory. CTAs of 256 threads, four an SM for bf16 and five for fp32, so that one CTA's end (the alternatives)
// runs beside the others' reading: 4093 bf16 rows of 128256 took 382 us at two CTAs of 512 threads, 220 at four
// of 256 with the arithmetic in pairs, 235 at five (registers spill); 160 fp32 rows 39 us at four and 31 at five. A second
// turn's loads ahead of the first's use changed nothing.
// GB300: 5 rows of 128256 in fp32, 5 alternatives, 9.8 us; 160 rows, 20 alternatives, 30 us (2.8 TB/s); 4093 rows in bf16,
// 1 alternative, 229 us (4.6 TB/s; 218 without Z's remainder), as many in fp32 with 5 alternatives 338 to 356 us (6.2 to 5.9 TB/s,
// as a call among others or alone), 160 bf16 rows along paths, 20 alternatives, 27. What runs once a CTA is kept short:
// on few rows its code has to be fetched (a sort of the maxima within and across warps took 1 us more of 160 rows).
#include <cooperative_groups.h>

#include "common.cuh"
#include "tc_host.cuh"
#include "tc_math.cuh"

namespace specv {
namespace lp {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kSegs = 8;       // segments of a thread at most
constexpr int kUnroll = 4;     // 16-byte loads of a turn (eight: 4093 bf16 rows 239 us instead of 220)
constexpr int kList = 1024;    // segments, and elements, that may reach the bound
constexpr int kMaxSplit = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

struct Params {
  const uint8_t* logits;
  long row_bytes;
  int vocab;
  const int32_t* tokens;      // [batch * cap], nullable
  const int32_t* path;        // [batch][cap], nullable: entry e reads row e
  const int32_t* accept_len;
  const int32_t* qo;
  int batch, cap, total;
  float inv_t;
  int topk;
  float* logprob;
  int32_t* rank;
  float* entropy;
  int32_t* top_ids;
  float* top_lp;
  int32_t* status;
};

// The order's key of a logit: larger for larger values, -0 as 0, NaN above all, 0 for -infinity (no alternative).
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  if (x == -INFINITY) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(float x, int id) {
  const uint32_t o = order_of(x);
  return o == 0 ? 0 : ((uint64_t)o << 32) | (uint32_t)~id;
}

// (a - m) / T in powers of two; no infinity, which times a weight of 0 would be NaN.
__device__ __forceinline__ float apart(float a, float m, float c) { return fmaxf((a - m) * c, -1e30f); }

// Of some elements: the largest logit, Z (and what its rounding lost), sum e^y y in powers of two. Z is at least 1, and
// where it is little more the log probability of the largest is as small, so Z is summed with its remainder.
struct Stat {
  float m, z, lost, w;
};
// a + b into a, what the rounding lost to `lost` (Knuth's sum of two, exact in any order).
__device__ __forceinline__ void add_to(float& a, float& lost, float b) {
  const float sum = a + b, part = sum - a;
  lost += (a - (sum - part)) + (b - part);
  a = sum;
}
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return Stat{m, a.z + b.z, 0.f, a.w + b.w};
  const float da = a.m == -INFINITY ? 0.f : apart(a.m, m, c), db = b.m == -INFINITY ? 0.f : apart(b.m, m, c);
  const float fa = ex2_approx(da), fb = ex2_approx(db);  // (one of them is 1)
  Stat s{m, a.z * fa, fmaf(a.lost, fa, b.lost * fb), fmaf(fmaf(a.z, da, a.w), fa, fmaf(b.z, db, b.w) * fb)};
  add_to(s.z, s.lost, b.z * fb);
  return s;
}
__device__ __forceinline__ float log_of(const Stat& s) {  // ln Z
  return s.z < 2.f ? log1pf((s.z - 1.f) + s.lost) : logf(s.z) + s.lost / s.z;
}

// Two elements of a 16-byte piece (its 4-byte words a, and for fp32 b) as fp32.
template <int VEC>
__device__ __forceinline__ float2 pair_of(uint32_t a, uint32_t b) {
  if constexpr (VEC == 4) return make_float2(__uint_as_float(a), __uint_as_float(b));
  else return make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
}
// The largest of a piece (a NaN is passed over), of m too.
template <int VEC>
__device__ __forceinline__ float largest(const uint4& v, float m) {
  if constexpr (VEC == 4) {
    return fmax3(fmax3(m, __uint_as_float(v.x), __uint_as_float(v.y)), __uint_as_float(v.z), __uint_as_float(v.w));
  } else {
    const __nv_bfloat162 t = __hmax2(__hmax2(reinterpret_cast<const __nv_bfloat162&>(v.x), reinterpret_cast<const __nv_bfloat162&>(v.y)),
                                     __hmax2(reinterpret_cast<const __nv_bfloat162&>(v.z), reinterpret_cast<const __nv_bfloat162&>(v.w)));
    return fmax3(m, __low2float(t), __high2float(t));
  }
}
// Elements of a piece above the threshold (for bf16 in both halves of thr), in fp32.
template <int VEC>
__device__ __forceinline__ float2 above(const uint4& v, uint32_t thr) {
  if constexpr (VEC == 4) {
    const float t = __uint_as_float(thr);
    auto is = [&](uint32_t w) { return __uint_as_float(w) > t ? 1.f : 0.f; };
    return fadd2(make_float2(is(v.x), is(v.y)), make_float2(is(v.z), is(v.w)));
  } else {
    const __nv_bfloat162 t = reinterpret_cast<const __nv_bfloat162&>(thr);
    auto is = [&](const uint32_t& w) { return __hgt2(reinterpret_cast<const __nv_bfloat162&>(w), t); };
    const __nv_bfloat162 n = __hadd2(__hadd2(is(v.x), is(v.y)), __hadd2(is(v.z), is(v.w)));
    return make_float2(__low2float(n), __high2float(n));
  }
}
// The bits of the next smaller value of the row's type (of -infinity and NaN: itself), as above() takes them.
template <int VEC>
__device__ __forceinline__ uint32_t threshold(float x, bool below) {
  constexpr int kDown = VEC == 4 ? 0 : 16;
  uint32_t u = __float_as_uint(x) >> kDown;
  constexpr uint32_t kSign = 0x80000000u >> kDown;
  if (below && x > -INFINITY) u = x == 0.f ? kSign | 1u : (u & kSign) ? u + 1 : u - 1;
  return VEC == 4 ? u : u | (u << 16);
}

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// The join of every n lanes from a multiple of n on (n a power of two), in each of them.
__device__ __forceinline__ Stat join_lanes(Stat s, int n, float c) {
#pragma unroll 1
  for (int o = n >> 1; o > 0; o >>= 1) {
    const Stat other{__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.z, o),
                     __shfl_xor_sync(0xffffffffu, s.lost, o), __shfl_xor_sync(0xffffffffu, s.w, o)};
    s = join(s, other, c);
  }
  return s;
}

struct Shared {
  float seg[kSegs * kThreads];   // the largest logit of every segment (thread t's s-th at s * kThreads + t)
  uint32_t maxima[kThreads];     // threads' maxima as order keys, the larger ones
  uint32_t low[kWarps], bound;
  uint64_t cand[kList];
  uint16_t hit[kList];
  uint64_t top[kMaxTop];         // this CTA's alternatives, in order
  Stat part[kWarps];
  int before[kWarps];
  int n_max, n_hit, n_cand;
  // in the cluster's first CTA, written by all of them: each one's alternatives, sums and count
  uint64_t all[kMaxSplit * kMaxTop];
  Stat stat[kMaxSplit];
  int count[kMaxSplit];
  uint64_t best[kWarps];
};

// Row element `id` (a plain load of its own size).
template <int VEC>
__device__ __forceinline__ float element(const uint8_t* row, int id) {
  if constexpr (VEC == 4) return ld(reinterpret_cast<const float*>(row) + id);
  else return __uint_as_float((uint32_t)ld(reinterpret_cast<const uint16_t*>(row) + id) << 16);
}

// A 16-byte piece of a row: elements [first, first + VEC) of it, those outside [0, vocab) as -infinity.
template <int VEC>
__device__ __forceinline__ uint4 edge(const uint8_t* row, int first, int vocab) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float x = first + i >= 0 && first + i < vocab ? element<VEC>(row, first + i) : -INFINITY;
    if (VEC == 4) w[i] = __float_as_uint(x);
    else w[i / 2] |= (__float_as_uint(x) >> 16) << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// VEC: elements of 16 bytes (4: fp32, 8: bf16). kRank, kEntropy: what is asked for.
template <int VEC, bool kRank, bool kEntropy>
__global__ void __launch_bounds__(kThreads, VEC == 4 ? 5 : 4) token_logprobs_kernel(const Params p) {
  __shared__ Shared sh;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int log_split = __ffs(split) - 1, e = (int)(blockIdx.x >> log_split), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  // ---- which row (the same in every CTA of the cluster); what it hangs on is loaded at once
  long row = e;
  bool none = false, bad = false;
  int token = p.tokens != nullptr ? ld(p.tokens + e) : -1;
  if (p.path != nullptr) {
    const int b = e / p.cap, i = e - b * p.cap;
    const int L = ld(p.accept_len + b), base = ld(p.qo + b), n = ld(p.qo + b + 1) - base, node = ld(p.path + e);
    bad = L < 0 || L >= p.cap || base < 0 || n > p.total - base;
    none = bad || i > L;
    if (!none) bad = none = node < 0 || node >= n;
    row = (long)base + node;
  }
  const bool known = !none && token >= 0 && token < p.vocab;
  if (!none && p.tokens != nullptr && !known) bad = true;
  if (bad && part == 0 && tid == 0) report(p.status, SPEC_ERR_INDEX);
  if (none) {  // past the path: no token
    if (part == 0) {
      if (tid == 0) {
        if (p.logprob != nullptr) p.logprob[e] = 0.f;
        if (p.rank != nullptr) p.rank[e] = -1;
        if (p.entropy != nullptr) p.entropy[e] = 0.f;
      }
      if (tid < p.topk) {
        if (p.top_ids != nullptr) p.top_ids[(long)e * p.topk + tid] = -1;
        if (p.top_lp != nullptr) p.top_lp[(long)e * p.topk + tid] = 0.f;
      }
    }
    return;
  }
  if (split > 1) cluster_arrive();  // (awaited before the first CTA's shared memory is written: by then it runs)
  const uint8_t* src = p.logits + row * p.row_bytes;
  const int V = p.vocab;
  const float c = p.inv_t * kLog2e;
  const float xt = known ? element<VEC>(src, token) : INFINITY;
  // 16-byte pieces from the aligned address at or below the row's first byte: piece v holds the elements
  // from v * VEC - skew on; its first and last may be partial and are read element by element
  const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15) / (16 / VEC));
  const int pieces = (int)((unsigned)(skew + V + VEC - 1) / VEC);  // (V <= 2^24)
  const int v0 = pieces * part >> log_split, v1 = pieces * (part + 1) >> log_split;
  const uint8_t* aligned = src - skew * (16 / VEC);
  constexpr int kTurnPieces = kThreads * kUnroll;
  const int turns = (int)((unsigned)(v1 - v0 + kTurnPieces - 1) / kTurnPieces), per_seg = (int)((unsigned)(turns + kSegs - 1) / kSegs);
  auto fetch = [&](int v) -> uint4 {  // piece v of this CTA's
    const int first = v * VEC - skew;
    constexpr uint32_t kNone = VEC == 4 ? 0xFF800000u : 0xFF80FF80u;  // -infinity
    if (v >= v1) return make_uint4(kNone, kNone, kNone, kNone);
    if (first >= 0 && first + VEC <= V) return ld(reinterpret_cast<const uint4*>(aligned) + v);
    return edge<VEC>(src, first, V);
  };

  Stat s{-INFINITY, 0.f, 0.f, 0.f};
  int before = 0;
  const uint32_t thr_above = threshold<VEC>(xt, false), thr_from = threshold<VEC>(xt, true);
  float seg_top = -INFINITY, my_top = -INFINITY;
  int seg = 0, in_seg = 0;
  // turns inside the row load without looking (the row's first piece may be partial), the others piece by piece
  const int whole = (min(v1, (int)((unsigned)(V + skew) / VEC)) - v0) / kTurnPieces;
#pragma unroll 1
  for (int t = 0; t < turns; ++t) {
    uint4 x[kUnroll];
    const int at = v0 + t * kTurnPieces + tid;
    if (t < whole && at > 0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) x[u] = ld(reinterpret_cast<const uint4*>(aligned) + at + u * kThreads);
    } else {
#pragma unroll 1
      for (int u = 0; u < kUnroll; ++u) {
        const uint4 v = fetch(at + u * kThreads);
#pragma unroll
        for (int w = 0; w < kUnroll; ++w) x[w] = w == u ? v : x[w];
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) top = largest<VEC>(x[u], top);
    seg_top = fmaxf(seg_top, top);
    if (top > s.m) {
      if (s.m != -INFINITY) {
        const float d = apart(s.m, top, c), f = ex2_approx(d);
        s.w = fmaf(s.z, d, s.w) * f;
        s.z *= f;
        s.lost *= f;
      }
      s.m = top;
    }
    const float m = s.m == -INFINITY ? 0.f : s.m;
    float2 z = make_float2(0.f, 0.f), w = z, n = z;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t words[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float2 part;  // of the piece: the fewer sums a 1 goes through, the less Z loses
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float2 v = VEC == 4 ? pair_of<VEC>(words[2 * i & 3], words[(2 * i + 1) & 3]) : pair_of<VEC>(words[i], 0);
        // (one fma would round m c, the same way for every term)
        const float2 y = fmul2(fadd2(v, make_float2(-m, -m)), make_float2(c, c));
        const float2 ex = make_float2(ex2_approx(y.x), ex2_approx(y.y));
        part = i == 0 ? ex : fadd2(part, ex);
        if constexpr (kEntropy) w = ffma2(ex, make_float2(fmaxf(y.x, -1e30f), fmaxf(y.y, -1e30f)), w);
      }
      z = u == 0 ? part : fadd2(z, part);
      if constexpr (kRank) {
        // tokens before t: a larger logit, or an equal one at a lower id (the piece that holds t, and the
        // row's first where it is partial, are looked at again below)
        const int first = (at + u * kThreads) * VEC - skew;
        n = fadd2(n, above<VEC>(x[u], first >= 0 && first + VEC <= token ? thr_from : thr_above));
      }
    }
    add_to(s.z, s.lost, z.x + z.y);
    if constexpr (kEntropy) s.w += w.x + w.y;
    if constexpr (kRank) before += (int)(n.x + n.y);
    if (++in_seg == per_seg) {
      sh.seg[seg * kThreads + tid] = seg_top;
      my_top = fmaxf(my_top, seg_top);
      seg_top = -INFINITY;
      in_seg = 0;
      ++seg;
    }
  }
  if (in_seg > 0) {
    sh.seg[seg * kThreads + tid] = seg_top;
    my_top = fmaxf(my_top, seg_top);
    ++seg;
  }
  if (kRank && xt == -INFINITY) {  // (no value is below it to compare with: whole pieces before t)
#pragma unroll 1
    for (int v = v0 + tid; v < v1; v += kThreads) {
      const int first = v * VEC - skew;
      if (first < 0 || first + VEC > token) continue;
#pragma unroll 1
      for (int i = 0; i < VEC; ++i) before += element<VEC>(src, first + i) == -INFINITY;
    }
  }
  if (kRank && known && warp == 0) {
    const int of_t = (token + skew) / VEC;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const int v = k == 0 ? of_t : 0, id = v * VEC - skew + lane;
      if (v < v0 || v >= v1 || (k == 1 && (skew == 0 || of_t == 0))) continue;
      if (lane < VEC && id >= 0 && id < token) before += element<VEC>(src, id) == xt;
    }
  }

  // ---- the CTA's sums
  s = join_lanes(s, 32, c);
  if constexpr (kRank) before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) {
    sh.part[warp] = s;
    sh.before[warp] = before;
  }
  if (tid == 0) sh.n_max = sh.n_hit = sh.n_cand = 0, sh.bound = 1;
  if (tid < kMaxTop) sh.top[tid] = 0;

  // ---- the CTA's alternatives
  const int k = p.topk;
  if (k > 0) {
    // The k-th largest of the threads' maxima. At least k of them reach the least of the warps' (k / kWarps)-th largest;
    // those that do find their places by counting.
    const uint32_t key = order_of(my_top);
    uint32_t rest = key, low = 0;
#pragma unroll 1
    for (int i = 0; i < k; i += kWarps) {
      low = __reduce_max_sync(0xffffffffu, rest);
      if (lane == __ffs(__ballot_sync(0xffffffffu, rest == low)) - 1) rest = 0;
    }
    if (lane == 0) sh.low[warp] = low;
    __syncthreads();
    low = sh.low[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) low = min(low, sh.low[w]);
    if (key >= max(low, 1u)) sh.maxima[atomicAdd(&sh.n_max, 1)] = key;
    __syncthreads();
    const int n_max = sh.n_max;
    if (tid < n_max) {
      const uint32_t mine = sh.maxima[tid];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < n_max; ++j) r += sh.maxima[j] > mine || (sh.maxima[j] == mine && j < tid);
      if (r == k - 1) sh.bound = mine;
    }
    __syncthreads();
    const uint32_t bound = sh.bound;  // (1 where fewer than k threads have seen anything above -infinity)
#pragma unroll 1
    for (int q = 0; q < seg; ++q)
      if (order_of(sh.seg[q * kThreads + tid]) >= bound) {
        const int at = atomicAdd(&sh.n_hit, 1);
        if (at < kList) sh.hit[at] = (uint16_t)(q * kThreads + tid);
      }
    __syncthreads();
    const int n_hit = min(sh.n_hit, kList), per = per_seg * kUnroll * VEC;
    bool many = sh.n_hit > kList;
#pragma unroll 1
    for (int i = tid; i < n_hit * per && !many; i += kThreads) {
      const unsigned h = (unsigned)i / (unsigned)per, j = (unsigned)i - h * per, hit = sh.hit[h];
      const int v = v0 + (int)((hit / kThreads * per_seg + j / (kUnroll * VEC)) * kTurnPieces +
                               (j / VEC % kUnroll) * kThreads + hit % kThreads);
      const int id = v * VEC - skew + (int)(j % VEC);
      if (v >= v1 || id < 0 || id >= V) continue;
      const float x = element<VEC>(src, id);
      if (order_of(x) >= bound) {
        const int at = atomicAdd(&sh.n_cand, 1);
        if (at < kList) sh.cand[at] = key_of(x, id);
      }
    }
    __syncthreads();
    const int n_cand = sh.n_cand;
    many |= n_cand > kList;
    if (!many) {
#pragma unroll 1
      for (int i = tid; i < n_cand; i += kThreads) {
        const uint64_t mine = sh.cand[i];
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < n_cand; ++j) r += sh.cand[j] > mine;
        if (r < k) sh.top[r] = mine;  // keys are distinct
      }
    } else {
      // so many equal logits at the bound that the list does not hold them: one alternative after the other
      uint64_t last = ~0ull;
#pragma unroll 1
      for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
#pragma unroll 1
        for (int v = v0 + tid; v < v1; v += kThreads) {
#pragma unroll 1
          for (int id = max(0, v * VEC - skew); id < min(V, (v + 1) * VEC - skew); ++id) {
            const uint64_t q = key_of(element<VEC>(src, id), id);
            if (q < last && q > best) best = q;
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, (uint64_t)__shfl_xor_sync(0xffffffffu, best, o));
        if (lane == 0) sh.best[warp] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) best = max(best, sh.best[w]);
        if (tid == 0) sh.top[j] = best;
        last = best;
        __syncthreads();
        if (best == 0) break;
      }
    }
  }
  __syncthreads();

  // ---- the cluster's, in its first CTA
  {
    Shared* first = split > 1 ? cluster.map_shared_rank(&sh, 0) : &sh;
    if (split > 1) cluster_wait();
    if (warp == 0) {
      const Stat all = join_lanes(lane < kWarps ? sh.part[lane] : Stat{-INFINITY, 0.f, 0.f, 0.f}, kWarps, c);
      const int n = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.before[lane] : 0);
      if (lane == 0) {
        first->stat[part] = all;
        first->count[part] = n;
      }
    } else if (tid < 32 + k) {
      first->all[part * kMaxTop + tid - 32] = sh.top[tid - 32];
    }
  }
  if (split > 1) {
    cluster_arrive();
    if (part != 0) return;
    cluster_wait();
  } else {
    __syncthreads();
  }
  const Stat all = join_lanes(sh.stat[lane & (split - 1)], split, c);
  const float log_z = log_of(all);
  if (warp == 0) {
    const int n = __reduce_add_sync(0xffffffffu, lane < split ? sh.count[lane] : 0);
    if (lane == 0) {
      if (p.logprob != nullptr) p.logprob[e] = known ? fmaf(xt - all.m, p.inv_t, -log_z) : 0.f;
      if (kRank) p.rank[e] = known ? n + 1 : -1;
      if (kEntropy) p.entropy[e] = fmaf(-all.w / all.z, kLn2, log_z);
    }
  }
  auto write = [&](int at, uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    const float x = __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
    if (p.top_ids != nullptr) p.top_ids[(long)e * k + at] = key == 0 ? -1 : (int)~(uint32_t)key;
    if (p.top_lp != nullptr) p.top_lp[(long)e * k + at] = key == 0 ? -INFINITY : fmaf(x - all.m, p.inv_t, -log_z);
  };
  if (tid < split * kMaxTop && tid % kMaxTop < k) {
    // the CTAs' lists: an alternative's place is the number of larger ones (keys are distinct); places that no
    // alternative takes come behind, in the order of the lists' empty places
    const uint64_t mine = sh.all[tid];
    int r = 0;
#pragma unroll 1
    for (int q = 0; q < split; ++q)
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        const uint64_t other = sh.all[q * kMaxTop + j];
        r += other > mine || (other == mine && q * kMaxTop + j < tid);
      }
    if (r < k) write(r, mine);
  }
}

}  // namespace lp

// CTAs of a row: as many as fill the GPU's places (four an SM) with the rows that there may be, each with 4096
// elements at least. (Twice as many: 160 fp32 rows of 288 places 48 us instead of 31.)
static int split_of(long rows, int vocab) {
  int s = 1;
  while (s < lp::kMaxSplit && rows * s < 4L * sm_count() && vocab / (2 * s) >= 4096) s *= 2;
  return s;
}

int launch_token_logprobs(int dtype, const void* logits, long row_stride, int vocab, const int32_t* tokens,
                          const int32_t* path, const int32_t* accept_len, const int32_t* qo, int batch, int cap,
                          int total, float temperature, int topk, float* logprob, int32_t* rank, float* entropy,
                          int32_t* top_ids, float* top_lp, int32_t* status, cudaStream_t stream) {
  using namespace lp;
  const int e = dtype == SPEC_F32 ? 4 : 2;
  const Params p{static_cast<const uint8_t*>(logits), row_stride * e, vocab, tokens, path, accept_len, qo, batch, cap,
                 total, 1.0f / temperature, top_ids != nullptr || top_lp != nullptr ? topk : 0, logprob, rank, entropy,
                 top_ids, top_lp, status};
  const long rows = (long)batch * cap;
  const int split = split_of(rows, vocab);
  if (rows * split > 0x7FFFFFFFL) return SPEC_ERR_UNSUPPORTED;
  const bool r = rank != nullptr, h = entropy != nullptr;
  const auto kernel = e == 4 ? (r ? h ? token_logprobs_kernel<4, true, true> : token_logprobs_kernel<4, true, false>
                                  : h ? token_logprobs_kernel<4, false, true> : token_logprobs_kernel<4, false, false>)
                             : (r ? h ? token_logprobs_kernel<8, true, true> : token_logprobs_kernel<8, true, false>
                                  : h ? token_logprobs_kernel<8, false, true> : token_logprobs_kernel<8, false, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * split));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
