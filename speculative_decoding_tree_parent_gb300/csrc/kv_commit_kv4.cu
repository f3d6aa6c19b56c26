// K-COMMIT into the 4-bit paged cache (kv4.cuh): bf16 rows quantised as they are written.
//
// Every 16 elements x of a row share a scale: with a the largest finite |x| and f the head's
// kv_scale, s = e4m3(a / (6 f)), at least 2^-9 and at most 448, so that the largest element meets E2M1's
// largest value, 6; an element's code is e2m1(x / (s f)). Groups lie within one token, so a
// row is written once and never again (a scale shared by tokens would have to grow as they arrive).
//
// Bound: latency on an accepted path (sizes and path -> rows -> codes), on a prompt chunk the bf16 rows' bytes and the
// issue of instructions. GB300: one path of 4 tokens 8.2 us, 32 chunks of 512 tokens, 8 heads, 33 us (2.6 TB/s of rows and
// records; with a division for every element 10.2 and 49). Every CTA checks the whole path of its sequence, a load of the page
// table a row, which is nothing for a chunk but grows with the square of a long prompt: 8192 rows of one sequence 40 us, of
// eight 127, 65536 of one 470. The rows' pointers are taken out of the arguments by an index known at run time, for which
// each thread keeps a copy of the arguments in local memory (120 bytes).
// Layout: a CTA per (sequence, touched page, share of the KV heads); of its 256 threads half take K, half V, each one
// group of one token. K's codes go out from the thread that made them; V's stand token by token
// inside a byte, so they are turned through shared memory and each thread writes the 16 tokens of an
// element, the page's other tokens kept. No two CTAs write the same page and head.
#include <algorithm>

#include "kv4.cuh"
#include "tc_host.cuh"
#include "tc_math.cuh"

namespace specv {

using namespace kv4;

struct Commit4Args {
  const __nv_bfloat16* tree[2];  // K, V rows [T][hkv][128]
  const float* kv_scale;         // [2][hkv] or nullptr
  const int32_t* path;
  int path_cap;
  const int32_t* accept_len;
  const int32_t* qo;
  const int32_t* page_table;
  int max_pages, num_pages;
  const int32_t* prefix_len;
  int32_t* seq_len_out;
  uint8_t* pool;  // [num_pages][hkv][2304]
  int batch, total, hkv;
  int32_t* status;
};

__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint16_t c;
  asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u16.u8 %0, t; }" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}
// e2m1(x / d) of two elements (bf16 bits in a word), a byte, the low element low; NaN gives 0
__device__ __forceinline__ uint32_t code2(uint32_t w, float d) {
  const float lo = __fdiv_rn(__uint_as_float(w << 16), d), hi = __fdiv_rn(__uint_as_float(w & 0xFFFF0000u), d);
  return e2m1x2(lo == lo ? lo : 0.f, hi == hi ? hi : 0.f);
}
// The same for finite x with |x / d| < 16 and d >= 2^-59, without a division for every element: with r = 1 / d rounded and
// y = x r, y + (x - y d) r is the quotient but for 2^-46 of it before it is rounded (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990). The code of the rounded quotient changes only halfway between a
// midpoint of E2M1 and its neighbours in fp32, and of all x / d (x with 8 bits, d with 24) but one kind none comes nearer to
// such a place than 2^-33; the one, a power of two over the largest significand, comes out right. The sign is x's, zero's too.
__device__ __forceinline__ uint32_t code2_near(uint32_t w, float2 d_neg, float2 r) {
  const float2 x = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  const float2 y = fmul2(x, r), q = ffma2(ffma2(y, d_neg, x), r, y);
  return e2m1x2(copysignf(q.x, x.x), copysignf(q.y, x.y));
}

// A group's 16 codes (element i in nibble i) and its scale code, 0x7F (NaN) where an element is NaN.
__device__ __forceinline__ uint2 quantise(const uint4 (&x)[2], float f, uint32_t& scale) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  bool nan = false;
  const bool all_finite = top < 0x7F80u;
  if (!all_finite) {  // an infinity or NaN: the largest among the others
    top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t v = (w[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
      if (v < 0x7F80u) top = max(top, v);
      nan |= v > 0x7F80u;
    }
  }
  const float t = fminf(fmaxf(__fdiv_rn(__uint_as_float(top << 16), 6.f * f), 0.001953125f), 448.f);
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(t));
  const float d = float2_of(half2_of_scales(c)).x * f;
  scale = nan ? 0x7Fu : (c & 0xFFu);
  uint2 codes = make_uint2(0, 0);
  if (all_finite && t < 448.f) {  // (t >= a / (6 f) and the scale is t * 2/3 at least: |x / d| <= 9)
    const float r = __frcp_rn(d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      codes.x |= code2_near(w[i], make_float2(-d, -d), make_float2(r, r)) << (8 * i);
      codes.y |= code2_near(w[4 + i], make_float2(-d, -d), make_float2(r, r)) << (8 * i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      codes.x |= code2(w[i], d) << (8 * i);
      codes.y |= code2(w[4 + i], d) << (8 * i);
    }
  }
  return codes;
}

constexpr int kC4Threads = 256;
constexpr int kTurn = kDim * 8 + kGroups * 8;  // V's codes of a page, 8 bytes of padding a group (bank conflicts)

// Four nibbles (16 bits) -> the low halves of four bytes.
__device__ __forceinline__ uint32_t spread(uint32_t x) {
  x = (x | (x << 8)) & 0x00FF00FFu;
  return (x | (x << 4)) & 0x0F0F0F0Fu;
}

// kMany: the grid has fewer places than the path may have pages.
template <bool kMany>
__global__ void __launch_bounds__(kC4Threads) kv_commit_kv4_kernel(const Commit4Args p) {
  // (batch and pages share the grid's x extent: y would end at 65535 pages)
  const int b = blockIdx.x % (unsigned)p.batch, nth = blockIdx.x / (unsigned)p.batch;
  const int half = threadIdx.x >> 7, tid = threadIdx.x & 127, r = tid >> 3, grp = tid & 7;  // 0: K, 1: V; token, group
  __shared__ __align__(16) uint8_t s_v[2][kTurn];  // V's codes of a page, of every other head
  pdl_wait();
  const int base = ld(p.qo + b), n = ld(p.qo + b + 1) - base;
  const int P = ld(p.prefix_len + b), L = ld(p.accept_len + b);
  const int32_t* path = p.path + (size_t)b * p.path_cap;
  const int32_t* table = p.page_table + (size_t)b * p.max_pages;
  const bool lead = nth == 0 && blockIdx.y == 0;
  if (L < 0 || L >= p.path_cap || L >= n || base < 0 || n > p.total - base || P < 0 || P > 0x7FFFFFFF - p.path_cap) {
    if (lead && threadIdx.x == 0) report(p.status, SPEC_ERR_INDEX);
    return;
  }
  bool checked = false;
  int turn = 0;
  for (long at = P / kPage + (long)nth; at * kPage <= (long)P + L; at += gridDim.x / (unsigned)p.batch) {
    const int lp = (int)at;
    // the page's rows [r0, r1) take the path's nodes from r0 - shift on; the others stay
    const int shift = P - lp * kPage;
    const int r0 = max(shift, 0), r1 = min(kPage, shift + L + 1);
    long from = -1;  // this thread's piece (head 0), -1: not a new row, or a bad node, which is not followed
    if (r >= r0 && r < r1) {
      const int node = ld(path + r - shift);
      if (node >= 0 && node < n) from = (long)(base + node) * p.hkv * kDim + kGroup * grp;
    }
    auto load = [&](int g, uint4 (&x)[2]) {
      x[0] = x[1] = make_uint4(0, 0, 0, 0);
      if (from < 0) return;
      const uint4* src = reinterpret_cast<const uint4*>(p.tree[half] + from + (long)g * kDim);
      x[0] = ld(src);
      x[1] = ld(src + 1);
    };
    // the first head's rows are on their way while the sequence is checked
    uint4 x[2];
    load(blockIdx.y, x);
    if (!checked) {
      int bad = 0;
      for (int i = threadIdx.x; i <= L; i += kC4Threads) {
        const int node = ld(path + i);
        const int q = (P + i) / kPage;
        if (node < 0 || node >= n || (i == 0 && node != 0)) bad = SPEC_ERR_INDEX;
        else if (q >= p.max_pages) bad = SPEC_ERR_CAPACITY;
        else {
          const int page = ld(table + q);
          if (page < 0 || page >= p.num_pages) bad = SPEC_ERR_PAGE;
        }
        if (bad) break;
      }
      if (bad && lead) report(p.status, bad);
      if (__syncthreads_or(bad)) return;
      checked = true;
    }
    const size_t page = (size_t)ld(table + lp);
    const uint64_t fresh = (~0ull >> (64 - 4 * (r1 - r0))) << (4 * r0);  // the new tokens' nibbles of an element
    for (int g = blockIdx.y; g < p.hkv; g += gridDim.y, turn ^= 1) {
      uint8_t* rec = p.pool + (page * p.hkv + g) * kRecord;
      uint4 y[2];  // the next head's rows, while this one's become codes
      if (g + gridDim.y < p.hkv) load(g + gridDim.y, y);
      uint32_t scale;
      uint2 c = quantise(x, head_scale(p.kv_scale, half, p.hkv, g), scale);
      const bool mine = r >= r0 && r < r1;
      if (half == 0) {
        if (mine) {
          *reinterpret_cast<uint2*>(rec + k_at(r, grp)) = c;
          rec[kOffKs + r * kGroups + grp] = (uint8_t)scale;
        }
      } else {
        // the pair of tokens r, r ^ 1 (8 lanes apart): the even one's thread joins elements 0 .. 7,
        // the odd one's 8 .. 15, two tokens a byte
        const bool odd = (r & 1) != 0;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? c.x : c.y, 8);
        const uint32_t lo = odd ? got : c.x, hi = odd ? c.y : got;
        const uint32_t w[2] = {spread(lo & 0xFFFFu) | (spread(hi & 0xFFFFu) << 4),
                               spread(lo >> 16) | (spread(hi >> 16) << 4)};
        uint8_t* to = s_v[turn] + (grp * kGroup + (odd ? 8 : 0)) * 8 + grp * 8 + (r >> 1);
#pragma unroll
        for (int k = 0; k < 8; ++k) to[8 * k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
        if (mine) rec[kOffVs + grp * kPage + r] = (uint8_t)scale;
        asm volatile("bar.sync 1, 128;" ::: "memory");  // (V's warps; the buffer of two heads ago has been read)
        uint64_t v = *reinterpret_cast<const uint64_t*>(s_v[turn] + tid * 8 + (tid >> 4) * 8);
        uint64_t* dst = reinterpret_cast<uint64_t*>(rec + kOffV) + tid;
        if (fresh != ~0ull) v = (v & fresh) | (*dst & ~fresh);
        *dst = v;
      }
      x[0] = y[0];
      x[1] = y[1];
    }
    if (!kMany) break;
  }
  if (lead && threadIdx.x == 0 && p.seq_len_out != nullptr) p.seq_len_out[b] = P + L + 1;
}

int launch_kv_commit_kv4(const void* k_tree, const void* v_tree, const int32_t* path, int path_cap,
                         const int32_t* accept_len, const int32_t* qo, const int32_t* page_table, int max_pages,
                         int num_pages, const int32_t* prefix_len, int32_t* seq_len_out, uint8_t* pool,
                         const float* kv_scale, int batch, int total_nodes, int hkv, int32_t* status,
                         cudaStream_t stream) {
  const Commit4Args p{{static_cast<const __nv_bfloat16*>(k_tree), static_cast<const __nv_bfloat16*>(v_tree)}, kv_scale,
                      path, path_cap, accept_len, qo, page_table, max_pages, num_pages, prefix_len, seq_len_out, pool,
                      batch, total_nodes, hkv, status};
  // most rows a path has (its nodes are the sequence's rows), and most pages that they touch
  const long most = path_cap < total_nodes ? path_cap : total_nodes > 1 ? total_nodes : 1;
  const long all = (most + kPage - 2) / kPage + 1;
  // A path may be much shorter than path_cap allows, and a CTA without a page is not free: the grid
  // holds the longest tree's pages, or as many as leave every head a CTA at 16 CTAs an SM, and a CTA
  // takes further pages in turn.
  const long tree = (kMaxTreeNodes + kPage - 2) / kPage + 1, room = 16L * sm_count() / batch / hkv;
  const long pages = std::min(all, std::max(tree, room));
  if (batch * pages > 0x7FFFFFFFL) return SPEC_ERR_UNSUPPORTED;
  const long share = 16L * sm_count() / (batch * pages);
  const dim3 grid((unsigned)(batch * pages), (unsigned)(share < 1 ? 1 : share < hkv ? share : hkv)), block(kC4Threads);
  const auto kernel = pages < all ? kv_commit_kv4_kernel<true> : kv_commit_kv4_kernel<false>;
  if (launch_pdl(kernel, grid, block, 0, stream, p) != cudaSuccess) return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
