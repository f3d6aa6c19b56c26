// Page-table rows grown (or shrunk) to the sequences' lengths, and the step's slot map.
//
// The lengths of a speculative step stay on the device (the commit writes seq_len there), so
// the pages of the next step have to be given out there too. Sequence b needs
//   need = ceil((seq_len[b] + n_b) / page_size) pages   (n_b = its nodes of this step)
// and holds held[b]; what it lacks comes off a stack of free pages, what it no longer needs
// (only where asked) goes back onto it. The result is a function of the inputs alone: with
// exclusive sums over the sequences, G_b of the pages asked for and R_b of those returned,
// and n1 = n_free + sum of the returned,
//   returned page k of b      -> place n_free + R_b + k of the stack,
//   page j granted to b       <- place n1 - 1 - (G_b + j),   granted while G_b + grow_b <= n1.
//
// Every CTA makes both sums itself (a few loads and one scan), so no CTA waits for another:
// nothing one CTA writes is read by another. Grants read places below n_free, or returned
// pages straight from the rows that give them up (the ends of shrinking rows, which nobody
// writes); returned pages are written to places from n_free on; grants go to the entries past
// a growing row's end. Only the two counters could be overwritten too early where they are
// updated in place: where there is one CTA it writes them at its end, else a second kernel does,
// which starts after the first has ended.
// Bound: latency for a step; the 8-byte slots' stores for a batch of prompts.
#include "common.cuh"
#include "page_stack.cuh"

namespace specv {

constexpr int kPageThreads = 512;
constexpr int kPageMaxBatch = 4096;
constexpr int kPagePer = kPageMaxBatch / kPageThreads;
constexpr int kPageTok = 4;  // slots a thread writes at a time: a 32-byte sector

struct PageArgs {
  const int32_t* seq_len;
  const int32_t* qo;
  const int32_t* held;
  int32_t* page_table;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* held_out;
  int32_t* n_free_out;
  long long* slot_map;
  int batch, total_nodes, max_pages, num_pages, page_size, shrink;
  int32_t* status;
};

// What sequence b asks for (grow) and gives back (back); a sequence with bad or too long
// sizes does neither (*code says which).
struct PageWant {
  int grow, back;
};
__device__ __forceinline__ PageWant page_want(const PageArgs& p, int b, int* code) {
  const int len = ld(p.seq_len + b), n = ld(p.qo + b + 1) - ld(p.qo + b), held = ld(p.held + b);
  *code = 0;
  if (len < 0 || n < 0 || held < 0 || held > p.max_pages) {
    *code = SPEC_ERR_INDEX;
    return PageWant{0, 0};
  }
  const long long need = ((long long)len + n + p.page_size - 1) / p.page_size;
  if (need > p.max_pages) {
    *code = SPEC_ERR_CAPACITY;
    return PageWant{0, 0};
  }
  return PageWant{need > held ? (int)need - held : 0, p.shrink && need < held ? held - (int)need : 0};
}

// The sequence that owns row t: the last b with qo[b] <= t.
__device__ __forceinline__ int page_seq_of(const int32_t* qo, int batch, int t) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ld(qo + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct PagePlan {
  int grow[kPageMaxBatch], back[kPageMaxBatch];  // inclusive sums over the sequences
  int wg[kPageThreads / 32], wb[kPageThreads / 32];
};

// Inclusive sums of grow and back over the batch (the whole CTA); the totals fit 32 bits
// (at most batch * max_pages entries of one table, checked on the host).
__device__ __forceinline__ void page_plan(const PageArgs& p, PagePlan& s, bool tell) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = ceil_div(p.batch, kPageThreads);
  int g[kPagePer], r[kPagePer], sg = 0, sr = 0;
#pragma unroll
  for (int i = 0; i < kPagePer; ++i) {
    g[i] = r[i] = 0;
    const int b = tid * per + i;
    if (i < per && b < p.batch) {
      int code;
      const PageWant w = page_want(p, b, &code);
      if (code != 0 && tell) report(p.status, code);
      g[i] = w.grow;
      r[i] = w.back;
    }
    sg += g[i];
    sr += r[i];
    g[i] = sg;
    r[i] = sr;
  }
  int xg = sg, xr = sr;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, xg, o), c = __shfl_up_sync(0xffffffffu, xr, o);
    if (lane >= o) {
      xg += a;
      xr += c;
    }
  }
  if (lane == 31) {
    s.wg[warp] = xg;
    s.wb[warp] = xr;
  }
  __syncthreads();
  int bg = xg - sg, br = xr - sr;
  for (int w = 0; w < warp; ++w) {
    bg += s.wg[w];
    br += s.wb[w];
  }
#pragma unroll
  for (int i = 0; i < kPagePer; ++i) {
    const int b = tid * per + i;
    if (i < per && b < p.batch) {
      s.grow[b] = bg + g[i];
      s.back[b] = br + r[i];
    }
  }
  __syncthreads();
}

// First b with sums[b] > x (sums rise; x < sums[batch - 1]).
__device__ __forceinline__ int page_owner(const int* sums, int batch, int x) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int page_returned(const PageArgs& p, const PagePlan& s, int r) {
  const int b = page_owner(s.back, p.batch, r);
  // row b gives up its last back_b entries, in order
  return __ldcg(p.page_table + (size_t)b * p.max_pages + ld(p.held + b) - (s.back[b] - r));
}

__device__ __forceinline__ int page_granted(const PageArgs& p, const PagePlan& s, int n0, int n1, int x) {
  const int at = n1 - 1 - x;
  return at < n0 ? __ldcg(p.free_pages + at) : page_returned(p, s, at - n0);
}

// Pages granted: whole sequences in order, while they last.
__device__ __forceinline__ int page_grants(const PagePlan& s, int batch, int n1) {
  if (s.grow[batch - 1] <= n1) return s.grow[batch - 1];
  const int b = page_owner(s.grow, batch, n1);
  return b > 0 ? s.grow[b - 1] : 0;
}

// A sequence for the slot map: pages [0, keeps) stand in its row, [held, ends) are granted now,
// from place `from` of the grants on. len -1: sizes that name no page.
struct PageSeq {
  int len, held, keeps, ends, from;
};
__device__ __forceinline__ PageSeq page_seq(const PageArgs& p, const PagePlan& s, int b, bool sane, int granted) {
  PageSeq q{ld(p.seq_len + b), ld(p.held + b), 0, 0, b > 0 ? s.grow[b - 1] : 0};
  if (q.held < 0 || q.held > p.max_pages) q.len = -1;
  q.keeps = sane ? q.held - (s.back[b] - (b > 0 ? s.back[b - 1] : 0)) : q.held;
  // (a sequence grows or shrinks, not both: held = keeps where anything is granted)
  q.ends = sane && s.grow[b] <= granted && s.grow[b] > q.from ? q.held + s.grow[b] - q.from : q.keeps;
  return q;
}

// The counters after the call.
__device__ __forceinline__ void page_count(const PageArgs& p, const PagePlan& s, int n0, bool sane, int granted) {
  for (int b = threadIdx.x; b < p.batch; b += kPageThreads) {
    const int g0 = b > 0 ? s.grow[b - 1] : 0, r0 = b > 0 ? s.back[b - 1] : 0;
    int now = p.held[b];
    if (sane) now += (s.grow[b] <= granted ? s.grow[b] - g0 : 0) - (s.back[b] - r0);
    p.held_out[b] = now;
  }
  if (threadIdx.x == 0) *p.n_free_out = sane ? n0 + s.back[p.batch - 1] - granted : n0;
}

__global__ void __launch_bounds__(kPageThreads) page_table_kernel(const PageArgs p) {
  __shared__ PagePlan s;
  // Signals early to its own second kernel alone (which waits, and does not signal): the table is
  // an input that a later kernel may read before its wait, where the caller lets it.
  if (gridDim.x > 1) pdl_trigger();
  pdl_wait();
  const int n0 = ld(p.n_free);
  page_plan(p, s, blockIdx.x == 0);
  const int asked = s.grow[p.batch - 1], back = s.back[p.batch - 1];
  const bool sane = page_stack_holds(n0, back, p.num_pages);  // else the stack is not what it should be: nothing moves
  const int n1 = sane ? n0 + back : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (!sane) report(p.status, SPEC_ERR_CAPACITY);
    else if (asked > n1) report(p.status, SPEC_ERR_CAPACITY);
  }
  const int step = gridDim.x * kPageThreads, first = blockIdx.x * kPageThreads + threadIdx.x;
  const int granted = sane ? page_grants(s, p.batch, n1) : 0;
  if (sane) {
    for (int x = first; x < granted; x += step) {
      const int b = page_owner(s.grow, p.batch, x);
      const int j = x - (b > 0 ? s.grow[b - 1] : 0);
      const int page = page_granted(p, s, n0, n1, x);
      if (page < 0 || page >= p.num_pages) report(p.status, SPEC_ERR_PAGE);
      p.page_table[(size_t)b * p.max_pages + ld(p.held + b) + j] = page;
    }
    for (int r = first; r < back - granted; r += step) p.free_pages[n0 + r] = page_returned(p, s, r);
  }
  if (p.slot_map != nullptr) {
    const int last = min(p.total_nodes, ld(p.qo + p.batch));  // rows behind the last sequence stay as they are
    for (long at0 = (long)first * kPageTok; at0 < last; at0 += (long)step * kPageTok) {
      const int t0 = (int)at0;
      long long slots[kPageTok];
      int b = page_seq_of(p.qo, p.batch, t0);
      int lo = ld(p.qo + b), hi = ld(p.qo + b + 1);
      PageSeq q = page_seq(p, s, b, sane, granted);
      unsigned at_page = 0xFFFFFFFFu;
      int page = -1;
#pragma unroll
      for (int k = 0; k < kPageTok; ++k) {
        const int t = t0 + k;
        slots[k] = -1;
        if (at0 + k >= last) continue;
        while (t >= hi && b + 1 < p.batch) {  // the next sequence that has nodes
          ++b;
          lo = hi;
          hi = ld(p.qo + b + 1);
          if (t < hi) q = page_seq(p, s, b, sane, granted);
          at_page = 0xFFFFFFFFu;
        }
        if (q.len < 0 || t < lo) continue;
        const unsigned at = (unsigned)q.len + (unsigned)(t - lo), lp = at / (unsigned)p.page_size;
        if (lp != at_page) {
          at_page = lp;
          page = -1;
          if (lp < (unsigned)q.keeps) page = __ldcg(p.page_table + (size_t)b * p.max_pages + lp);
          else if (lp < (unsigned)q.ends) page = page_granted(p, s, n0, n1, q.from + (int)lp - q.held);
          if (lp < (unsigned)q.ends && (page < 0 || page >= p.num_pages)) {
            if (lp < (unsigned)q.keeps) report(p.status, SPEC_ERR_PAGE);
            page = -1;
          }
        }
        if (page >= 0) slots[k] = (long long)page * p.page_size + (at - lp * (unsigned)p.page_size);
      }
      if (at0 + kPageTok <= last && (reinterpret_cast<uintptr_t>(p.slot_map) & 15) == 0) {
        longlong2* dst = reinterpret_cast<longlong2*>(p.slot_map + t0);
#pragma unroll
        for (int k = 0; k < kPageTok / 2; ++k) dst[k] = make_longlong2(slots[2 * k], slots[2 * k + 1]);
      } else {
#pragma unroll
        for (int k = 0; k < kPageTok; ++k)
          if (at0 + k < last) p.slot_map[at0 + k] = slots[k];
      }
    }
  }
  if (gridDim.x == 1) {
    __syncthreads();  // every read of the counters
    page_count(p, s, n0, sane, granted);
  }
}

__global__ void __launch_bounds__(kPageThreads) page_count_kernel(const PageArgs p) {
  __shared__ PagePlan s;
  pdl_wait();  // the kernel before has read the counters that this one may overwrite
  const int n0 = ld(p.n_free);
  page_plan(p, s, false);
  const bool sane = page_stack_holds(n0, s.back[p.batch - 1], p.num_pages);
  page_count(p, s, n0, sane, sane ? page_grants(s, p.batch, n0 + s.back[p.batch - 1]) : 0);
}

int launch_page_table(const int32_t* seq_len, const int32_t* qo, const int32_t* held, int32_t* page_table,
                      int max_pages, int32_t* free_pages, int num_pages, const int32_t* n_free, int page_size,
                      int shrink, int batch, int total_nodes, int32_t* held_out, int32_t* n_free_out,
                      long long* slot_map, int32_t* status, cudaStream_t stream) {
  const PageArgs p{seq_len,  qo,    held,        page_table, free_pages, n_free,    held_out, n_free_out,
                   slot_map, batch, total_nodes, max_pages,  num_pages,  page_size, shrink,   status};
  const int slots = slot_map != nullptr ? ceil_div(total_nodes, kPageTok) : 0;
  const int ctas = ceil_div(slots > batch ? slots : batch, kPageThreads);
  if (launch_pdl(page_table_kernel, dim3(ctas < 608 ? ctas : 608), dim3(kPageThreads), 0, stream, p) != cudaSuccess)
    return SPEC_ERR_CUDA;
  if (ctas > 1 && launch_pdl(page_count_kernel, dim3(1), dim3(kPageThreads), 0, stream, p) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

int page_table_max_batch() { return kPageMaxBatch; }

}  // namespace specv
