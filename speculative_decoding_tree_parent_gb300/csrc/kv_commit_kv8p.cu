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
// Layout: one CTA per (sequence, touched page, KV head), half its threads for K, half for V;
// a thread keeps its 16-element pieces of the page in registers from the maximum to the
// store. No two CTAs write the same page and head, so nothing is exchanged between them; each
// makes the sequence's checks itself and comes to the same verdict.
#include "common.cuh"

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
  int hkv, d;
  int32_t* status;
};

// Largest finite magnitude (bf16 bits) among eight elements; infinities and NaN do not count.
__device__ __forceinline__ uint32_t top8(const uint4& u) {
  uint32_t m = 0;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    if (lo < 0x7F80u) m = max(m, lo);
    if (hi < 0x7F80u) m = max(m, hi);
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
__device__ __forceinline__ uint32_t code4(uint32_t a, uint32_t b, float s) {
  return code4(__fdiv_rn(__uint_as_float(a << 16), s), __fdiv_rn(__uint_as_float(a & 0xFFFF0000u), s),
               __fdiv_rn(__uint_as_float(b << 16), s), __fdiv_rn(__uint_as_float(b & 0xFFFF0000u), s));
}

// The smallest power of two s in [2^-50, 2^50] with x <= 448 s (x >= 0 given by its bf16 bits;
// 448 = 1.75 * 2^8, so a fraction up to 1.75 keeps x's own exponent less 8).
__device__ __forceinline__ float scale_for(uint32_t bits) {
  if (bits == 0) return kPageScaleMin;
  const int e = (int)(bits >> 7) - 127 - 8 + ((bits & 0x7Fu) > 0x60u ? 1 : 0);
  return exp2f((float)max(-kPageScaleExp, min(kPageScaleExp, e)));
}

// kPer: 16-element pieces of a page and head that a thread holds
template <int kPer>
__global__ void __launch_bounds__(2 * kQcHalf) kv_commit_kv8p_kernel(const CommitP8Args p) {
  const int b = blockIdx.x, g = blockIdx.z;
  const int half = threadIdx.x / kQcHalf, tid = threadIdx.x % kQcHalf;  // 0: K, 1: V
  __shared__ uint32_t s_top[2][kQcHalf / 32];
  pdl_wait();
  const int base = __ldg(p.qo + b), n = __ldg(p.qo + b + 1) - base;
  const int P = __ldg(p.prefix_len + b), L = __ldg(p.accept_len + b);
  const int ps = p.page_size;
  const int32_t* path = p.path + (size_t)b * p.path_cap;
  const int32_t* table = p.page_table + (size_t)b * p.max_pages;
  const bool lead = blockIdx.y == 0 && g == 0;
  if (L < 0 || L >= p.path_cap || L >= n || P < 0 || P > 0x7FFFFFFF - p.path_cap) {
    if (lead && threadIdx.x == 0) report(p.status, SPEC_ERR_INDEX);
    return;
  }
  const int lp = P / ps + (int)blockIdx.y;
  if ((long long)lp * ps > (long long)P + L) return;  // the path ends before this page
  // the page's rows [r0, r1) take the path's nodes from r0 - shift on; rows below r0 are older
  const int shift = P - lp * ps;  // > 0 on the first page where it starts inside
  const int r0 = max(shift, 0), r1 = min(ps, shift + L + 1);
  const int pieces = p.d >> 4;
  // this thread's new rows, loaded while the sequence is checked (a bad node is not followed)
  uint4 x[kPer][2];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid + i * kQcHalf, r = e / pieces;
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (r < r0 || r >= r1) continue;
    const int node = __ldg(path + r - shift);
    if (node < 0 || node >= n) continue;
    const uint4* src = reinterpret_cast<const uint4*>(p.tree[half] + ((size_t)(base + node) * p.hkv + g) * p.d) +
                       2 * (e - r * pieces);
    x[i][0] = __ldg(src);
    x[i][1] = __ldg(src + 1);
  }
  int bad = 0;
  for (int i = threadIdx.x; i <= L; i += 2 * kQcHalf) {
    const int node = __ldg(path + i);
    const int q = (P + i) / ps;
    if (node < 0 || node >= n || (i == 0 && node != 0)) bad = SPEC_ERR_INDEX;
    else if (q >= p.max_pages) bad = SPEC_ERR_CAPACITY;
    else {
      const int page = __ldg(table + q);
      if (page < 0 || page >= p.num_pages) bad = SPEC_ERR_PAGE;
    }
    if (bad) break;
  }
  if (bad && lead) report(p.status, bad);
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = max(top, max(top8(x[i][0]), top8(x[i][1])));
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) s_top[half][tid >> 5] = top;
  if (__syncthreads_or(bad)) return;
#pragma unroll
  for (int w = 0; w < kQcHalf / 32; ++w) top = max(top, s_top[half][w]);
  const size_t unit = (size_t)__ldg(table + lp) * p.hkv + g;
  float* sp = p.kv_scale + unit * 2 + half;
  uint8_t* codes = p.pool[half] + unit * ps * p.d;
  float now = scale_for(top);
  float was = now;
  if (r0 > 0) {
    was = page_scale(*sp);
    now = fmaxf(now, was);
  }
  __syncthreads();  // every thread has read the old scale
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid + i * kQcHalf, r = e / pieces;
    if (r >= r1) continue;
    uint4* dst = reinterpret_cast<uint4*>(codes) + e;  // rows are contiguous: piece e of the page
    if (r >= r0) {
      *dst = make_uint4(code4(x[i][0].x, x[i][0].y, now), code4(x[i][0].z, x[i][0].w, now),
                        code4(x[i][1].x, x[i][1].y, now), code4(x[i][1].z, x[i][1].w, now));
    } else if (now != was) {
      const uint4 c = *dst;
      const uint32_t in[4] = {c.x, c.y, c.z, c.w};
      uint32_t out[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = e4m3x4_to_f32(in[k]);
        out[k] = code4(__fdiv_rn(v.x * was, now), __fdiv_rn(v.y * was, now), __fdiv_rn(v.z * was, now),
                       __fdiv_rn(v.w * was, now));
      }
      *dst = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
  if (tid == 0) *sp = now;
  if (lead && threadIdx.x == 0 && p.seq_len_out != nullptr) p.seq_len_out[b] = P + L + 1;
}

// Pieces of a (page, head) a thread can hold: page_size * d <= 4 * 128 * 16 elements.
bool commit_kv8p_shape(int page_size, int d) {
  return page_size >= 1 && d >= 16 && d % 16 == 0 && (long)page_size * d <= 4L * kQcHalf * 16;
}

int launch_kv_commit_kv8p(const void* k_tree, const void* v_tree, const int32_t* path, int path_cap,
                          const int32_t* accept_len, const int32_t* qo, const int32_t* page_table, int max_pages,
                          int num_pages, int page_size, const int32_t* prefix_len, int32_t* seq_len_out,
                          uint8_t* k_pool, uint8_t* v_pool, float* kv_scale, int batch, int hkv, int d,
                          int32_t* status, cudaStream_t stream) {
  const CommitP8Args p{{static_cast<const __nv_bfloat16*>(k_tree), static_cast<const __nv_bfloat16*>(v_tree)},
                       path, path_cap, accept_len, qo, page_table, max_pages, num_pages, page_size, prefix_len,
                       seq_len_out, {k_pool, v_pool}, kv_scale, hkv, d, status};
  // most pages a path of path_cap nodes touches; a tree holds at most kMaxTreeNodes nodes
  const int most = path_cap < kMaxTreeNodes ? path_cap : kMaxTreeNodes;
  const dim3 grid(batch, ceil_div(most - 1, page_size) + 1, hkv), block(2 * kQcHalf);
  const int per = ceil_div(page_size * (d / 16), kQcHalf);
  const cudaError_t e = per <= 1   ? launch_pdl(kv_commit_kv8p_kernel<1>, grid, block, 0, stream, p)
                        : per <= 2 ? launch_pdl(kv_commit_kv8p_kernel<2>, grid, block, 0, stream, p)
                                   : launch_pdl(kv_commit_kv8p_kernel<4>, grid, block, 0, stream, p);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
