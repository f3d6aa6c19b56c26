// Norm and rotation of the tree's queries and keys, before the attention reads them.
//
// For node t of sequence b, at position pos = prefix_len[b] + depth[t] (the node's place in the
// sequence were its path accepted), and every query and key head x of d elements:
//   y = x / sqrt(mean(x^2) + eps) * w            (skipped where no weight is given)
//   (u, v) -> (u c - v s, v c + u s)             for the rot / 2 pairs, c = cos, s = sin of the
//                                                position's table row; elements past rot pass
// in fp32, rounded once on output; value heads are copied.
//
// Bound: HBM on a prompt chunk (each element is read and written once, a few operations each),
// latency on a tree (a chain of three loads: the sequence's bounds, the position's table row,
// then the store; the heads' own loads are in flight meanwhile).
// Layout: a thread holds the eight pairs 8j .. 8j+7 of a head as two chunks of eight elements
// (both halves of the split form, or two adjacent chunks of the interleaved form), so a pair
// never leaves its thread, every access is 16 bytes, and the norm needs log2(d / 16) shuffles.
// A CTA takes one node and up to 12 warps' worth of its heads.
#include "common.cuh"

namespace specv {

constexpr int kRopeMaxWarps = 12;

struct RopeArgs {
  const void* q_in;
  const void* k_in;
  const void* v_in;
  long q_stride, k_stride, v_stride;  // elements between nodes
  const void* q_weight;
  const void* k_weight;
  float eps;
  const float* cos_sin;  // [max_pos][rot]: rot / 2 cosines, then rot / 2 sines
  int max_pos, rot;
  const int32_t* prefix_len;
  const int32_t* depth;  // nullptr: node i of a sequence is i tokens past its prefix
  const int32_t* qo;
  int batch, hq, hkv, d;
  void* q_out;
  void* k_out;
  void* v_out;
  int32_t* status;
};

struct Eight {
  float x[8];
};

__device__ __forceinline__ Eight load8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ Eight load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.x[2 * i] = __uint_as_float(w[i] << 16);
    r.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}
__device__ __forceinline__ void store8(float* p, const Eight& v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Eight& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x[2 * i], v.x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// LPH: lanes per head, the power of two that holds d / 16
template <typename T, int LPH, bool kInterleaved>
__global__ void __launch_bounds__(kRopeMaxWarps * 32) qk_norm_rope_kernel(const RopeArgs p) {
  pdl_wait();
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane & (LPH - 1);
  const int head = (blockIdx.y * (blockDim.x >> 5) + warp) * (32 / LPH) + lane / LPH;
  const int heads = p.hq + p.hkv + (p.v_in != nullptr ? p.hkv : 0);
  const bool mine = head < heads && 16 * j < p.d;
  const int part = head < p.hq ? 0 : head < p.hq + p.hkv ? 1 : 2;  // query, key, value
  const bool turns = part < 2 && 16 * j < p.rot;
  // the thread's two chunks (element offsets): the pairs 8j .. 8j+7, or 16 elements past rot
  int ca = 16 * j, cb = 16 * j + 8;
  if (!kInterleaved && 16 * j < p.rot) {
    ca = 8 * j;
    cb = 8 * j + p.rot / 2;
  }
  Eight a{}, b{};
  const T* in = nullptr;
  if (mine) {
    const long row = part == 0 ? t * p.q_stride + (long)head * p.d
                     : part == 1 ? t * p.k_stride + (long)(head - p.hq) * p.d
                                 : t * p.v_stride + (long)(head - p.hq - p.hkv) * p.d;
    in = static_cast<const T*>(part == 0 ? p.q_in : part == 1 ? p.k_in : p.v_in) + row;
    a = load8(in + ca);
    b = load8(in + cb);
  }
  // the node's sequence: every lane tests its own sequences, one of them owns the node
  const int dep = p.depth != nullptr ? __ldg(p.depth + t) : 0;
  int pos = 0, owned = 0;
  for (int s = lane; s < p.batch; s += 32) {
    const int lo = __ldg(p.qo + s), hi = __ldg(p.qo + s + 1), len = __ldg(p.prefix_len + s);
    if (t >= lo && t < hi) {
      pos = len + (p.depth != nullptr ? dep : t - lo);
      owned = len < 0 || dep < 0 ? -1 : 1;
    }
  }
  const unsigned who = __ballot_sync(0xffffffffu, owned != 0);
  if (who == 0) return;  // a row behind the last sequence: left as it is
  const int src = __ffs(who) - 1;
  pos = __shfl_sync(0xffffffffu, pos, src);
  owned = __shfl_sync(0xffffffffu, owned, src);
  if (owned < 0 || (p.rot > 0 && (pos < 0 || pos >= p.max_pos))) {
    if (threadIdx.x == 0) report(p.status, SPEC_ERR_INDEX);
    return;
  }
  Eight c{}, s{};
  if (mine && turns) {
    const float* tab = p.cos_sin + (size_t)pos * p.rot + 8 * j;
    c = load8(tab);
    s = load8(tab + p.rot / 2);
  }
  const void* wp = part == 0 ? p.q_weight : part == 1 ? p.k_weight : nullptr;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += a.x[i] * a.x[i] + b.x[i] * b.x[i];
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (!mine) return;
  if (wp != nullptr) {
    const float r = rsqrtf(ss / (float)p.d + p.eps);
    const T* w = static_cast<const T*>(wp);
    const Eight wa = load8(w + ca), wb = load8(w + cb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a.x[i] = a.x[i] * r * wa.x[i];
      b.x[i] = b.x[i] * r * wb.x[i];
    }
  }
  if (turns) {
    if (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = a.x[2 * i], v = a.x[2 * i + 1];
        a.x[2 * i] = u * c.x[i] - v * s.x[i];
        a.x[2 * i + 1] = v * c.x[i] + u * s.x[i];
        const float u2 = b.x[2 * i], v2 = b.x[2 * i + 1];
        b.x[2 * i] = u2 * c.x[4 + i] - v2 * s.x[4 + i];
        b.x[2 * i + 1] = v2 * c.x[4 + i] + u2 * s.x[4 + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = a.x[i], v = b.x[i];
        a.x[i] = u * c.x[i] - v * s.x[i];
        b.x[i] = v * c.x[i] + u * s.x[i];
      }
    }
  }
  T* out = part == 0 ? static_cast<T*>(p.q_out) + ((size_t)t * p.hq + head) * p.d
           : part == 1 ? static_cast<T*>(p.k_out) + ((size_t)t * p.hkv + head - p.hq) * p.d
                       : static_cast<T*>(p.v_out) + ((size_t)t * p.hkv + head - p.hq - p.hkv) * p.d;
  store8(out + ca, a);
  store8(out + cb, b);
}

template <typename T, int LPH>
static cudaError_t launch_rope(const RopeArgs& p, bool interleaved, int total_nodes, cudaStream_t stream) {
  const int heads = p.hq + p.hkv + (p.v_in != nullptr ? p.hkv : 0);
  const int warps = ceil_div(heads, 32 / LPH);
  const int y = ceil_div(warps, kRopeMaxWarps);
  const dim3 grid(total_nodes, y), block(ceil_div(warps, y) * 32);
  return interleaved ? launch_pdl(qk_norm_rope_kernel<T, LPH, true>, grid, block, 0, stream, p)
                     : launch_pdl(qk_norm_rope_kernel<T, LPH, false>, grid, block, 0, stream, p);
}

template <typename T>
static cudaError_t launch_rope_d(const RopeArgs& p, bool interleaved, int total_nodes, cudaStream_t stream) {
  const int l = p.d / 16;
  if (l <= 4) return launch_rope<T, 4>(p, interleaved, total_nodes, stream);
  if (l <= 8) return launch_rope<T, 8>(p, interleaved, total_nodes, stream);
  if (l <= 16) return launch_rope<T, 16>(p, interleaved, total_nodes, stream);
  return launch_rope<T, 32>(p, interleaved, total_nodes, stream);
}

int launch_qk_norm_rope(int dtype, const void* q_in, long q_stride, const void* k_in, long k_stride, const void* v_in,
                        long v_stride, const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
                        int max_pos, int rot, bool interleaved, const int32_t* prefix_len, const int32_t* depth,
                        const int32_t* qo, int batch, int total_nodes, int hq, int hkv, int d, void* q_out,
                        void* k_out, void* v_out, int32_t* status, cudaStream_t stream) {
  const RopeArgs p{q_in, k_in,  v_in,       q_stride, k_stride, v_stride, q_weight, k_weight, eps,   cos_sin, max_pos,
                   rot,  prefix_len, depth, qo,       batch,    hq,       hkv,      d,        q_out, k_out,   v_out,
                   status};
  const cudaError_t e = dtype == SPEC_F32 ? launch_rope_d<float>(p, interleaved, total_nodes, stream)
                                          : launch_rope_d<__nv_bfloat16>(p, interleaved, total_nodes, stream);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
