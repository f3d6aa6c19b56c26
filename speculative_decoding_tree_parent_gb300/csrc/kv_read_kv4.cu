// Rows of the 4-bit paged cache (kv4.cuh) brought back in bf16: code * group scale * the head's scale.
// The first product is exact in fp16; the second is rounded to fp32, then once to bf16.
//
// Bound: HBM, 512 bytes written for 144 read (a token of a head, K and V). GB300: 4 tokens 6.1 us, 32 sequences of 512
// tokens, 8 heads, 23 us; of 8191 tokens 235 us (5.8 TB/s).
// Layout: a CTA per (sequence, page, share of the KV heads). Half of its 256 threads take K, a group of
// one token each, and store its 32 bytes as they come; half take V, one element of the
// page's 16 tokens each, turned through shared memory into rows. Eight CTAs an SM (32 registers; what spills is the judges'): 32
// sequences of 4096 tokens, one call among others, 117 us; six (40 registers) 131. The halves' loops stand apart: one loop
// with both in it 133.
#include "kv4.cuh"
#include "tc_host.cuh"

namespace specv {

using namespace kv4;

struct Read4Args {
  const uint8_t* pool;
  const float* kv_scale;
  const int32_t* page_table;
  int max_pages, num_pages;
  const int32_t* first;
  const int32_t* qo;
  __nv_bfloat16* out[2];  // [total][hkv][128]
  int batch, total, hkv, places;
  int32_t* status;
};

constexpr int kR4Threads = 256;
constexpr int kPad = kDim + 8;  // a turned row of V in shared memory (16 bytes of padding: bank conflicts)

// Two fp16 values times f, as two bf16.
__device__ __forceinline__ uint32_t scaled(uint32_t h, float f) {
  const float2 v = float2_of(h);
  const __nv_bfloat162 o = __floats2bfloat162_rn(v.x * f, v.y * f);
  return *reinterpret_cast<const uint32_t*>(&o);
}

// What sequence b asks for: n rows from slot `at` on, to rows from `base` on. none: its numbers are out of range, its rows are
// left as they were.
struct Run {
  int base, n, at;
  bool none;
  __device__ __forceinline__ int pages() const { return none || n == 0 ? 0 : ((at + n - 1) >> 4) - (at >> 4) + 1; }
};
__device__ __forceinline__ bool outside(const Read4Args& p, int base, int end) { return base < 0 || end < base || end > p.total; }
__device__ __forceinline__ Run run_of(const Read4Args& p, int b) {
  const int base = ld(p.qo + b), end = ld(p.qo + b + 1), at = ld(p.first + b);
  const bool none = outside(p, base, end) || at < 0 || at > 0x7FFFFFFF - (end - base);
  return Run{base, none ? 0 : end - base, at, none};
}

using TurnedRows = uint16_t[2][kPage * kPad];  // V's rows of a page, of every other head

// The i-th page of sequence b's run.
__device__ __forceinline__ void read_page(const Read4Args& p, int b, const Run& run, int i, TurnedRows& s_v) {
  const int half = threadIdx.x >> 7, tid = threadIdx.x & 127, r = tid >> 3, grp = tid & 7;
  const int base = run.base, n = run.n, at = run.at;
  const int lp = (at >> 4) + i;
  const int shift = at - lp * kPage;  // the page's rows [r0, r1) are output rows from base + r0 - shift on
  const int r0 = max(shift, 0), r1 = min(kPage, shift + n);
  int page = -1;
  if (lp < p.max_pages) page = ld(p.page_table + (size_t)b * p.max_pages + lp);
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(p.status, lp < p.max_pages ? SPEC_ERR_PAGE : SPEC_ERR_CAPACITY);
    page = -1;  // its rows are zeros
  }
  const long row0 = (long)base - shift;  // output row of the page's row 0
  const uint8_t* rec = p.pool + ((size_t)max(page, 0) * p.hkv + blockIdx.y) * kRecord;
  if (half == 0) {
    if (r < r0 || r >= r1) return;
    for (int g = blockIdx.y; g < p.hkv; g += gridDim.y, rec += gridDim.y * (size_t)kRecord) {
      const float f = page < 0 ? 0.f : head_scale(p.kv_scale, 0, p.hkv, g);
      const uint2 c = page < 0 ? make_uint2(0, 0) : ld(reinterpret_cast<const uint2*>(rec + k_at(r, grp)));
      const uint32_t s = half2_of_scale(page < 0 ? 0u : ld(rec + kOffKs + r * kGroups + grp));
      uint4* dst = reinterpret_cast<uint4*>(p.out[0] + ((row0 + r) * p.hkv + g) * kDim + grp * kGroup);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t w = k == 0 ? c.x : c.y;
        dst[k] = make_uint4(scaled(hmul2(half2_of_codes<0>(w), s), f), scaled(hmul2(half2_of_codes<1>(w), s), f),
                            scaled(hmul2(half2_of_codes<2>(w), s), f), scaled(hmul2(half2_of_codes<3>(w), s), f));
      }
    }
  } else {
    int turn = 0;
    for (int g = blockIdx.y; g < p.hkv; g += gridDim.y, turn ^= 1, rec += gridDim.y * (size_t)kRecord) {
      const float f = page < 0 ? 0.f : head_scale(p.kv_scale, 1, p.hkv, g);
      const uint2 c = page < 0 ? make_uint2(0, 0) : ld(reinterpret_cast<const uint2*>(rec + kOffV) + tid);
      const uint4 sc = page < 0 ? make_uint4(0, 0, 0, 0) : ld(reinterpret_cast<const uint4*>(rec + kOffVs) + (tid >> 4));
      const uint32_t sw[4] = {sc.x, sc.y, sc.z, sc.w};
      uint16_t* to = s_v[turn] + tid;
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // tokens 2k, 2k + 1
        const uint32_t w = k < 4 ? c.x : c.y;
        const uint32_t h = (k & 3) == 0   ? half2_of_codes<0>(w)
                           : (k & 3) == 1 ? half2_of_codes<1>(w)
                           : (k & 3) == 2 ? half2_of_codes<2>(w)
                                          : half2_of_codes<3>(w);
        const uint32_t o = scaled(hmul2(h, half2_of_scales((uint16_t)(sw[k >> 1] >> (16 * (k & 1))))), f);
        to[(2 * k) * kPad] = (uint16_t)o;
        to[(2 * k + 1) * kPad] = (uint16_t)(o >> 16);
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");  // (V's warps; the buffer of two heads ago has been read)
      if (r < r0 || r >= r1) continue;
      const uint4* src = reinterpret_cast<const uint4*>(s_v[turn] + r * kPad + grp * kGroup);
      uint4* dst = reinterpret_cast<uint4*>(p.out[1] + ((row0 + r) * p.hkv + g) * kDim + grp * kGroup);
      dst[0] = src[0];
      dst[1] = src[1];
    }
  }
}

// CTAs (of each share of the heads) behind the places, which judge all ranges. Pages find their CTAs while the ranges rise and lie
// within the rows; where they do not, a place may find another sequence than its own, and these CTAs write all rows of all
// sequences that are in range, a group of 16 elements of K or V a thread at a time. (A sum over the batch in each CTA, which
// finds pages whatever the ranges, took 18 us instead of 10 for 1024 short sequences.)
constexpr unsigned kJudges = 64;

__device__ __forceinline__ void judge(const Read4Args& p) {
  const unsigned place = blockIdx.x - p.places, judges = gridDim.x - p.places;
  bool wrong = false;
  for (int b = threadIdx.x; b < p.batch; b += kR4Threads) {
    wrong |= outside(p, ld(p.qo + b), ld(p.qo + b + 1));
    if (place == 0 && blockIdx.y == 0 && run_of(p, b).none) report(p.status, SPEC_ERR_INDEX);
  }
  if (!__syncthreads_or(wrong)) return;
#pragma unroll 1
  for (int b = 0; b < p.batch; ++b) {
    const Run run = run_of(p, b);
#pragma unroll 1
    for (long j = (long)place * kR4Threads + threadIdx.x; j < 2L * kGroups * run.n; j += (long)judges * kR4Threads) {
      const int grp = (int)(j & (kGroups - 1)), half = (int)(j / kGroups & 1), i = (int)(j / (2 * kGroups));
      const int lp = (run.at + i) / kPage, r = (run.at + i) % kPage;
      int page = -1;
      if (lp < p.max_pages) page = ld(p.page_table + (size_t)b * p.max_pages + lp);
      const bool good = page >= 0 && page < p.num_pages;
      if (!good) report(p.status, lp < p.max_pages ? SPEC_ERR_PAGE : SPEC_ERR_CAPACITY);
#pragma unroll 1
      for (int g = blockIdx.y; g < p.hkv; g += gridDim.y) {
        const uint8_t* rec = p.pool + ((size_t)(good ? page : 0) * p.hkv + g) * kRecord;
        const float f = good ? head_scale(p.kv_scale, half, p.hkv, g) : 0.f;
        const uint32_t s = half2_of_scale(good ? ld(rec + (half == 0 ? kOffKs + r * kGroups + grp : kOffVs + grp * kPage + r)) : 0u);
        __nv_bfloat16* dst = (half == 0 ? p.out[0] : p.out[1]) + (((long)run.base + i) * p.hkv + g) * kDim + grp * kGroup;
#pragma unroll 1
        for (int e = 0; e < kGroup; ++e) {
          const uint32_t two = !good ? 0u : ld(rec + (half == 0 ? k_at(r, grp) + e / 2 : kOffV + (grp * kGroup + e) * 8 + r / 2));
          const uint32_t v = scaled(hmul2(half2_of_codes<0>(two), s), f);
          dst[e] = __ushort_as_bfloat16((uint16_t)(((half == 0 ? e : r) & 1) ? v >> 16 : v));
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kR4Threads, 8) kv_read_kv4_kernel(const Read4Args p) {
  __shared__ __align__(16) TurnedRows s_v;
  pdl_wait();
  // Sequence b's pages stand at places qo[b] / 16 + 2 b and on: they touch at most n / 16 + 2 pages, so
  // the places of two sequences never meet, and a CTA finds its own by bisection.
  const int u = blockIdx.x;
  if (u >= p.places) {
    judge(p);
    return;
  }
  int lo = 0, hi = p.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((ld(p.qo + mid) >> 4) + 2 * mid <= u) lo = mid; else hi = mid - 1;
  }
  const Run run = run_of(p, lo);
  const int i = u - (run.base >> 4) - 2 * lo;
  if (i >= 0 && i < run.pages()) read_page(p, lo, run, i, s_v);
}

int launch_kv_read_kv4(const uint8_t* pool, const float* kv_scale, const int32_t* page_table, int max_pages,
                       int num_pages, const int32_t* first, const int32_t* qo, int batch, int total, int hkv,
                       void* k_out, void* v_out, int32_t* status, cudaStream_t stream) {
  const long places = (long)total / kPage + 2L * batch;
  const long judges = places < kJudges ? places : kJudges;
  if (places + judges > 0x7FFFFFFFL) return SPEC_ERR_UNSUPPORTED;
  const Read4Args p{pool, kv_scale, page_table, max_pages, num_pages, first, qo,
                    {static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out)}, batch, total, hkv,
                    (int)places, status};
  const long share = 16L * sm_count() / places;
  const dim3 grid((unsigned)(places + judges), (unsigned)(share < 1 ? 1 : share < hkv ? share : hkv));
  if (launch_pdl(kv_read_kv4_kernel, grid, dim3(kR4Threads), 0, stream, p) != cudaSuccess) return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
