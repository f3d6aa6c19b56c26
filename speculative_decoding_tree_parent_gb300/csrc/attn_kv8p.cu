// Tree-verify attention over an 8-bit paged cache with a scale per (page, KV head).
//
// Row (node i of sequence b, query head h, g = h / (hq / hkv)), over the prefix keys j (page
// and row of slot j) and the tree nodes that row's mask bits name:
//   s_j = sm_scale * q . (k_code_j * ks[page_j][g]),   tree: q . k_j
//   out = sum_j 2^((s_j - m) log2 e) v_j / sum_j 2^((s_j - m) log2 e),  v_j = v_code_j * vs
// One warp per row, one pass over the keys with the running maximum and sum.
#include "attn_common.cuh"

namespace specv {

struct Kv8pArgs {
  const __nv_bfloat16* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float2* kv_scale;
  const int32_t* page_table;
  int max_pages, num_pages;
  const int32_t* prefix_len;
  const __nv_bfloat16* k_tree;
  const __nv_bfloat16* v_tree;
  const uint64_t* mask;
  int mask_words;
  const int32_t* qo;
  int batch, total_nodes, hq, hkv;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  int32_t* status;
};

__device__ __forceinline__ float4 bf16x4(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

__global__ void __launch_bounds__(256) attn_kv8p_kernel(const Kv8pArgs p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(row / p.hq), h = (int)(row - (long)t * p.hq);
  if (t >= p.total_nodes || t >= __ldg(p.qo + p.batch)) return;
  const int b = seq_of_row(p.qo, p.batch, t);
  const int base = __ldg(p.qo + b), N = __ldg(p.qo + b + 1) - base, P = __ldg(p.prefix_len + b);
  if (N > p.mask_words * 64 || P < 0 || P > p.max_pages * 16) {
    if (lane == 0) report(p.status, SPEC_ERR_CAPACITY);
    return;
  }
  const int g = h / (p.hq / p.hkv);
  const float4 q = bf16x4(p.q + row * 128 + 4 * lane);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto key = [&](float4 k, float4 v, float ks, float vs) {
    float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2 * ks;
    const float mx = fmaxf(m, s);
    const float a = mx == -INFINITY ? 1.f : exp2f(m - mx), w = mx == -INFINITY ? 0.f : exp2f(s - mx);
    l = l * a + w;
    const float wv = w * vs;
    o = make_float4(o.x * a + wv * v.x, o.y * a + wv * v.y, o.z * a + wv * v.z, o.w * a + wv * v.w);
    m = mx;
  };
  for (int j = 0; j < P; ++j) {
    const int page = __ldg(p.page_table + (size_t)b * p.max_pages + (j >> 4));
    if (page < 0 || page >= p.num_pages) {
      report(p.status, SPEC_ERR_PAGE);
      key(make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f), 1.f, 1.f);
      continue;
    }
    const size_t unit = (size_t)page * p.hkv + g;
    const float2 sc = __ldg(p.kv_scale + unit);
    const size_t at = (unit * 16 + (j & 15)) * 128 + 4 * lane;
    key(e4m3x4_to_f32(__ldg(reinterpret_cast<const uint32_t*>(p.k_pool + at))),
        e4m3x4_to_f32(__ldg(reinterpret_cast<const uint32_t*>(p.v_pool + at))), page_scale(sc.x), page_scale(sc.y));
  }
  const uint64_t* mrow = p.mask + (size_t)t * p.mask_words;
  for (int j = 0; j < N; ++j) {
    if (!((__ldg(mrow + (j >> 6)) >> (j & 63)) & 1)) continue;
    const size_t at = ((size_t)(base + j) * p.hkv + g) * 128 + 4 * lane;
    key(bf16x4(p.k_tree + at), bf16x4(p.v_tree + at), 1.f, 1.f);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), c = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.out + row * 128 + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
  if (lane == 0 && p.lse != nullptr) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

size_t attn_kv8p_ws_bytes(int, int, int, int, int) { return 0; }

int launch_attn_kv8p(const void* q, const uint8_t* k_pool, const uint8_t* v_pool, const float* kv_scale, int num_pages,
                     const int32_t* page_table, int max_pages, const int32_t* prefix_len, int max_prefix,
                     const void* k_tree, const void* v_tree, const uint64_t* mask, const int32_t* qo, int batch,
                     int total_nodes, int max_nodes, int hq, int hkv, float sm_scale, void* out, float* lse, void* ws,
                     int32_t* status, cudaStream_t stream) {
  (void)max_prefix;
  (void)ws;
  const Kv8pArgs p{static_cast<const __nv_bfloat16*>(q), k_pool, v_pool, reinterpret_cast<const float2*>(kv_scale),
                   page_table, max_pages, num_pages, prefix_len, static_cast<const __nv_bfloat16*>(k_tree),
                   static_cast<const __nv_bfloat16*>(v_tree), mask, (max_nodes + 63) >> 6, qo, batch, total_nodes, hq,
                   hkv, sm_scale * kLog2e, static_cast<__nv_bfloat16*>(out), lse, status};
  const long rows = (long)total_nodes * hq;
  if (launch_pdl(attn_kv8p_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, stream, p) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
