// K-COMMIT into an 8-bit paged cache with a scale per (page, KV head), for K and for V.
//
// A page's scale s is a power of two, the smallest with max|x| <= 448 s over the rows written
// to it, so an element's code is e4m3(x / s) with an exact division. Rows that arrive later
// can only raise s; the page's older codes are then rewritten as e4m3(code * s_old / s), a
// shift of their exponent that loses nothing but bits falling below E4M3's smallest step
// (2^-9 of the new scale). E4M3 is a floating format, so a scale up to twice what max|x|
// needs costs no precision, only one binade of its range.
//
// Bound: latency on an accepted path (sizes and path -> rows -> maximum -> stores), HBM on a
// prompt chunk (bf16 rows read once, codes written once).
// Layout: a CTA per (sequence, touched page or several, share of the KV heads), half its threads for K, half for V;
// a thread keeps its 16-element pieces of the page in registers from the maximum to the
// store. No two CTAs write the same page and head, so nothing is exchanged between them; each
// makes the sequence's checks itself and comes to the same verdict.
#include <algorithm>

#include "common.cuh"
#include "tc_host.cuh"

namespace specv {

constexpr int kQcHalf = 128;  // threads for K, and for V

struct CommitP8Args {
  const __nv_bfloat16* tree[2];  // K, V rows [T][hkv][d]
  const int32_t* path;
  int path_cap;
  const int32_t* accept_len;
  const int32_t* qo;
  const int32_t* page_table;
  int max_pages, num_pages, page_size;
  const int32_t* prefix_len;
  int32_t* seq_len_out;
  uint8_t* pool[2];   // K, V codes [num_pages][hkv][page_size][d]
  float* kv_scale;    // [num_pages][hkv][2]
  int batch, total, hkv, d;  // total: tree rows
  int32_t* status;
};

// Largest finite magnitude (bf16 bits) among sixteen elements; infinities and NaN do not count.
__device__ __forceinline__ uint32_t top16(const uint4& u, const uint4& v) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t m = 0;  // of the low and of the high halves
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  if (m >= 0x7F80u) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = (w[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
      if (x < 0x7F80u) m = max(m, x);
    }
  }
  return m;
}

// e4m3(x * r), ties to even, beyond +-448 saturated, NaN kept; x4 in byte order
__device__ __forceinline__ uint32_t code4(float x0, float x1, float x2, float x3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Sixteen codes e4m3(x / s). Scales written here are powers of two, and then the product with
// r = 1 / s is exactly the quotient; a scale that came with the page may be any number (r = 0).
__device__ __forceinline__ uint32_t code4(uint32_t a, uint32_t b, float r) {
  return code4(__uint_as_float(a << 16) * r, __uint_as_float(a & 0xFFFF0000u) * r, __uint_as_float(b << 16) * r,
               __uint_as_float(b & 0xFFFF0000u) * r);
}
__device__ __noinline__ uint32_t code4_div(float x0, float x1, float x2, float x3, float s) {
  return code4(__fdiv_rn(x0, s), __fdiv_rn(x1, s), __fdiv_rn(x2, s), __fdiv_rn(x3, s));
}
__device__ __forceinline__ uint32_t code4_div(uint32_t a, uint32_t b, float s) {
  return code4_div(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16),
                   __uint_as_float(b & 0xFFFF0000u), s);
}
// 1 / s for a power of two s (in [2^-50, 2^50]), else 0.
__device__ __forceinline__ float exact_inverse(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x7FFFFFu) == 0 ? __uint_as_float(0x7F000000u - u) : 0.f;
}

// The smallest power of two s in [2^-50, 2^50] with x <= 448 s (x >= 0 given by its bf16 bits;
// 448 = 1.75 * 2^8, so a fraction up to 1.75 keeps x's own exponent less 8).
__device__ __forceinline__ float scale_for(uint32_t bits) {
  if (bits == 0) return kPageScaleMin;
  const int e = (int)(bits >> 7) - 127 - 8 + ((bits & 0x7Fu) > 0x60u ? 1 : 0);
  return exp2f((float)max(-kPageScaleExp, min(kPageScaleExp, e)));
}

// kPer: 16-element pieces of a page and head that a thread holds; kMany: the grid has fewer places
// than the path may have pages. (32 chunks of about 500 rows: 23.7 us without the loop, 25.8 with it;
// an accepted path takes as long either way.)
template <int kPer, bool kMany>
__global__ void __launch_bounds__(2 * kQcHalf, !kMany ? 0 : kPer == 1 ? 5 : kPer == 2 ? 3 : 2) kv_commit_kv8p_kernel(const CommitP8Args p) {
  // (batch and pages share the grid's x extent: y would end at 65535 pages)
  const int b = blockIdx.x % (unsigned)p.batch, nth = blockIdx.x / (unsigned)p.batch;
  const int half = threadIdx.x / kQcHalf, tid = threadIdx.x % kQcHalf;  // 0: K, 1: V
  __shared__ uint32_t s_top[2][2][kQcHalf / 32];  // [head of a pair][half][warp]
  pdl_wait();
  const int base = ld(p.qo + b), n = ld(p.qo + b + 1) - base;
  const int P = ld(p.prefix_len + b), L = ld(p.accept_len + b);
  const int ps = p.page_size;
  const int32_t* path = p.path + (size_t)b * p.path_cap;
  const int32_t* table = p.page_table + (size_t)b * p.max_pages;
  const bool lead = nth == 0 && blockIdx.y == 0;
  if (L < 0 || L >= p.path_cap || L >= n || base < 0 || n > p.total - base || P < 0 || P > 0x7FFFFFFF - p.path_cap) {
    if (lead && threadIdx.x == 0) report(p.status, SPEC_ERR_INDEX);
    return;
  }
  const int pieces = p.d >> 4;
  bool checked = false;
  int turn = 0;
  for (long at = P / ps + (long)nth; at * ps <= (long)P + L; at += gridDim.x / (unsigned)p.batch) {
    const int lp = (int)at;
    // the page's rows [r0, r1) take the path's nodes from r0 - shift on; rows below r0 are older
    const int shift = P - lp * ps;  // > 0 on the first page where it starts inside
    const int r0 = max(shift, 0), r1 = min(ps, shift + L + 1);
    // where this thread's new pieces come from (head 0), -1: an older row, none, or a bad node, which
    // is not followed
    long from[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + i * kQcHalf, r = e / pieces;
      from[i] = -1;
      if (r < r0 || r >= r1) continue;
      const int node = ld(path + r - shift);
      if (node >= 0 && node < n) from[i] = (long)(base + node) * p.hkv * p.d + 16 * (e - r * pieces);
    }
    auto load = [&](int g, uint4 (&x)[kPer][2]) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        if (from[i] < 0) continue;
        const uint4* src = reinterpret_cast<const uint4*>(p.tree[half] + from[i] + (long)g * p.d);
        x[i][0] = ld(src);
        x[i][1] = ld(src + 1);
      }
    };
    // the first head's rows are on their way while the sequence is checked
    uint4 x[kPer][2];
    load(blockIdx.y, x);
    if (!checked) {
      int bad = 0;
      for (int i = threadIdx.x; i <= L; i += 2 * kQcHalf) {
        const int node = ld(path + i);
        const int q = (P + i) / ps;
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
    for (int g = blockIdx.y; g < p.hkv; g += gridDim.y, turn ^= 1) {
      const size_t unit = page * p.hkv + g;
      float* sp = p.kv_scale + unit * 2 + half;
      const float old = r0 > 0 ? *sp : 0.f;  // (read by every thread before the barrier, written after it)
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = max(top, top16(x[i][0], x[i][1]));
      top = __reduce_max_sync(0xffffffffu, top);
      if ((tid & 31) == 0) s_top[turn][half][tid >> 5] = top;
      // the next head's rows, while this one's are joined, turned into codes and stored
      uint4 y[kPer][2];
      if (g + gridDim.y < p.hkv) load(g + gridDim.y, y);
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kQcHalf / 32; ++w) top = max(top, s_top[turn][half][w]);
      uint8_t* codes = p.pool[half] + unit * ps * p.d;
      float now = scale_for(top);
      float was = now;
      if (r0 > 0) {
        was = page_scale(old);
        now = fmaxf(now, was);
      }
      const float inv = exact_inverse(now);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = tid + i * kQcHalf, r = e / pieces;
        if (r >= r1) continue;
        uint4* dst = reinterpret_cast<uint4*>(codes) + e;  // rows are contiguous: piece e of the page
        if (r >= r0) {
          *dst = inv != 0.f ? make_uint4(code4(x[i][0].x, x[i][0].y, inv), code4(x[i][0].z, x[i][0].w, inv),
                                         code4(x[i][1].x, x[i][1].y, inv), code4(x[i][1].z, x[i][1].w, inv))
                            : make_uint4(code4_div(x[i][0].x, x[i][0].y, now), code4_div(x[i][0].z, x[i][0].w, now),
                                         code4_div(x[i][1].x, x[i][1].y, now), code4_div(x[i][1].z, x[i][1].w, now));
        } else if (now != was) {
          const uint4 c = *dst;
          const uint32_t in[4] = {c.x, c.y, c.z, c.w};
          uint32_t out[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 v = e4m3x4_to_f32(in[k]);
            out[k] = inv != 0.f ? code4(v.x * was * inv, v.y * was * inv, v.z * was * inv, v.w * was * inv)
                                : code4_div(v.x * was, v.y * was, v.z * was, v.w * was, now);
          }
          *dst = make_uint4(out[0], out[1], out[2], out[3]);
        }
      }
      if (tid == 0) *sp = now;
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i][0] = y[i][0], x[i][1] = y[i][1];
    }
    if (!kMany) break;
  }
  if (lead && threadIdx.x == 0 && p.seq_len_out != nullptr) p.seq_len_out[b] = P + L + 1;
}

// Pieces of a (page, head) a thread can hold: page_size * d <= 4 * 128 * 16 elements.
bool commit_kv8p_shape(int page_size, int d) {
  return page_size >= 1 && d >= 16 && d % 16 == 0 && (long)page_size * d <= 4L * kQcHalf * 16;
}

int launch_kv_commit_kv8p(const void* k_tree, const void* v_tree, const int32_t* path, int path_cap,
                          const int32_t* accept_len, const int32_t* qo, const int32_t* page_table, int max_pages,
                          int num_pages, int page_size, const int32_t* prefix_len, int32_t* seq_len_out,
                          uint8_t* k_pool, uint8_t* v_pool, float* kv_scale, int batch, int total_nodes, int hkv,
                          int d, int32_t* status, cudaStream_t stream) {
  const CommitP8Args p{{static_cast<const __nv_bfloat16*>(k_tree), static_cast<const __nv_bfloat16*>(v_tree)},
                       path, path_cap, accept_len, qo, page_table, max_pages, num_pages, page_size, prefix_len,
                       seq_len_out, {k_pool, v_pool}, kv_scale, batch, total_nodes, hkv, d, status};
  // most rows a path has (its nodes are the sequence's rows), and most pages that they touch
  const long most = path_cap < total_nodes ? path_cap : total_nodes > 1 ? total_nodes : 1;
  const long all = (most + page_size - 2) / page_size + 1;
  // a CTA per head while they stand on the GPU at once (its longest chain is then the shortest),
  // else as many heads a CTA as make it so: the checks and the chain before the rows are then made
  // once for several heads, and a head's rows are loaded under the one before it (32 sequences of
  // about 500 rows, 8 heads: a CTA per head 39 us; at most 8, 16, 32 CTAs an SM: 26.8, 24.8, 28.8)
  // A path may be much shorter than path_cap allows, and a CTA without a page costs about a
  // microsecond of its place: the grid holds the longest tree's pages, or as many as leave every head
  // a CTA at 16 CTAs an SM, and a CTA takes further pages in turn (with room for 131,072 rows: 32
  // chunks of 500 rows 36 us, 54 with a CTA for every page; 4 paths of 4 rows 9 and 15)
  const long tree = (kMaxTreeNodes + page_size - 2) / page_size + 1, room = 16L * sm_count() / batch / hkv;
  const long pages = std::min(all, std::max(tree, room));
  if (batch * pages > 0x7FFFFFFFL) return SPEC_ERR_UNSUPPORTED;
  const long share = 16L * sm_count() / (batch * pages);
  const dim3 grid((unsigned)(batch * pages), (unsigned)(share < 1 ? 1 : share < hkv ? share : hkv)), block(2 * kQcHalf);
  const int per = ceil_div(page_size * (d / 16), kQcHalf);
  const auto kernel = pages < all ? (per <= 1   ? kv_commit_kv8p_kernel<1, true>
                                     : per <= 2 ? kv_commit_kv8p_kernel<2, true>
                                                : kv_commit_kv8p_kernel<4, true>)
                                  : (per <= 1   ? kv_commit_kv8p_kernel<1, false>
                                     : per <= 2 ? kv_commit_kv8p_kernel<2, false>
                                                : kv_commit_kv8p_kernel<4, false>);
  const cudaError_t e = launch_pdl(kernel, grid, block, 0, stream, p);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
