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
// Layout: a thread holds two chunks of eight elements of a head, so chosen that a pair never
// leaves its thread and neighbouring lanes touch neighbouring 16 bytes (halves of the head for
// adjacent pairs, halves of the rotated part for split ones), and the norm needs log2(d / 16)
// shuffles. A CTA has up to 10 warps' worth of heads and a run of nodes; the grid is 768 threads an SM. The rows come through shared memory by asynchronous copies, 8 / sizeof(T) nodes
// ahead, each thread reading back what it copied: 40 KB in flight a CTA, which registers cannot
// hold (one node a CTA, in registers: 118 us on 10,000 nodes of 64 + 16 heads of 128 in bf16; a
// run of nodes, the next in registers: 99; so: 76, 5.5 TB/s read and written). A node's weights
// and its sequence stay with the thread from node to node.
#include "common.cuh"
#include "tc_host.cuh"
#include "tc_math.cuh"

namespace specv {

constexpr int kRopeMaxWarps = 10;
// Threads an SM that the grid is made for. (At the kernel's 96 registers an SM holds 640: two blocks of
// 320 threads, as for 64 + 16 heads of 128, all stand at once; of smaller blocks the last ones wait for
// a place, 32 + 16 heads of 128 in bf16: 72 us for 10,000 tokens, 1.9 times their bytes' time.)
constexpr int kRopeThreads = 768;

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
  int batch, total, hq, hkv, d;
  void* q_out;
  void* k_out;
  void* v_out;
  int32_t* status;
};

struct Eight {
  float x[8];
};

// Eight elements as they lie in memory, widened only when they are used.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
};
__device__ __forceinline__ Raw<float> load_raw(const float* p) {
  return Raw<float>{reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
}
__device__ __forceinline__ Raw<__nv_bfloat16> load_raw(const __nv_bfloat16* p) {
  return Raw<__nv_bfloat16>{*reinterpret_cast<const uint4*>(p)};
}
// The same into shared memory, asynchronously.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async(Raw<float>* dst, const float* src) {
  copy16(&dst->a, src);
  copy16(&dst->b, src + 4);
}
__device__ __forceinline__ void copy_async(Raw<__nv_bfloat16>* dst, const __nv_bfloat16* src) { copy16(&dst->u, src); }
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ Eight widen(const Raw<float>& r) {
  return Eight{{r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w}};
}
__device__ __forceinline__ Eight widen(const Raw<__nv_bfloat16>& r) {
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e.x[2 * i] = __uint_as_float(w[i] << 16);
    e.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return e;
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
__global__ void __launch_bounds__(kRopeMaxWarps * 32, 2) qk_norm_rope_kernel(const RopeArgs p) {
  constexpr int kStages = 8 / (int)sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane & (LPH - 1);
  const int head = (blockIdx.y * (blockDim.x >> 5) + warp) * (32 / LPH) + lane / LPH;
  const int heads = p.hq + p.hkv + (p.v_in != nullptr ? p.hkv : 0);
  const bool mine = head < heads && 16 * j < p.d;
  const int part = head < p.hq ? 0 : head < p.hq + p.hkv ? 1 : 2;  // query, key, value
  const int at = part == 0 ? head : part == 1 ? head - p.hq : head - p.hq - p.hkv;
  const bool turns = mine && part < 2 && (kInterleaved ? 8 * j : 16 * j) < p.rot;
  // the thread's two chunks (element offsets): of the head's halves where pairs are adjacent, else
  // of the rotated part's halves or of the rest's
  int ca = 8 * j, cb = 8 * j + p.d / 2;
  if (!kInterleaved) {
    const bool rest = 16 * j >= p.rot;
    ca = rest ? p.rot / 2 + 8 * j : 8 * j;
    cb = rest ? ca + (p.d - p.rot) / 2 : ca + p.rot / 2;
  }
  const long stride = part == 0 ? p.q_stride : part == 1 ? p.k_stride : p.v_stride;
  const T* in = static_cast<const T*>(part == 0 ? p.q_in : part == 1 ? p.k_in : p.v_in) + (long)at * p.d;
  T* out = static_cast<T*>(part == 0 ? p.q_out : part == 1 ? p.k_out : p.v_out) + (size_t)at * p.d;
  const size_t out_stride = (size_t)(part == 0 ? p.hq : p.hkv) * p.d;
  const T* weight = static_cast<const T*>(part == 0 ? p.q_weight : part == 1 ? p.k_weight : nullptr);

  pdl_wait();
  Raw<T> wa{}, wb{};  // the head's weights stay with the thread
  if (mine && weight != nullptr) {
    wa = load_raw(weight + ca);
    wb = load_raw(weight + cb);
  }
  // The node's position, -1 where there is nothing to do (a row behind the last sequence is left as
  // it is). Its sequence is looked for only when the one before has ended: every lane tests its own
  // sequences, one of them owns the node.
  int lo = 0, hi = 0, len = 0;
  auto locate = [&](int t) -> int {
    const int dep = p.depth != nullptr ? ld(p.depth + t) : 0;
    if (t < lo || t >= hi) {
      int mlo = 0, mhi = 0, mlen = 0;
      for (int s = lane; s < p.batch; s += 32) {
        const int a = ld(p.qo + s), b = ld(p.qo + s + 1), l = ld(p.prefix_len + s);
        if (t >= a && t < b) mlo = a, mhi = b, mlen = l;
      }
      const unsigned who = __ballot_sync(0xffffffffu, mhi > mlo);
      if (who == 0) return -1;
      const int src = __ffs(who) - 1;
      lo = __shfl_sync(0xffffffffu, mlo, src);
      hi = __shfl_sync(0xffffffffu, mhi, src);
      len = __shfl_sync(0xffffffffu, mlen, src);
    }
    const int pos = len + (p.depth != nullptr ? dep : t - lo);
    if (len < 0 || dep < 0 || (p.rot > 0 && (pos < 0 || pos >= p.max_pos))) {
      if (threadIdx.x == 0) report(p.status, SPEC_ERR_INDEX);
      return -1;
    }
    return pos;
  };
  // four cosines and sines for the chunk at `at`
  auto load_turns = [](const float* tab, int rot, int at, Eight& c, Eight& s, int to) {
    const float4 x = *reinterpret_cast<const float4*>(tab + at / 2);
    const float4 y = *reinterpret_cast<const float4*>(tab + (rot + at) / 2);
    c.x[to] = x.x, c.x[to + 1] = x.y, c.x[to + 2] = x.z, c.x[to + 3] = x.w;
    s.x[to] = y.x, s.x[to + 1] = y.y, s.x[to + 2] = y.z, s.x[to + 3] = y.w;
  };
  auto turns_of = [&](int pos, Eight& c, Eight& s) {
    if (!turns || pos < 0) return;
    const float* tab = p.cos_sin + (size_t)pos * p.rot;
    if (!kInterleaved) {
      c = widen(load_raw(tab + 8 * j));
      s = widen(load_raw(tab + p.rot / 2 + 8 * j));
    } else {
      load_turns(tab, p.rot, ca, c, s, 0);
      if (cb < p.rot) load_turns(tab, p.rot, cb, c, s, 4);
    }
  };
  // A CTA has a run of nodes; the next ones' rows, and the next one's position and cosines, are on
  // their way while this one's are worked on.
  int t = (int)((long)blockIdx.x * p.total / gridDim.x);
  const int end = (int)((long)(blockIdx.x + 1) * p.total / gridDim.x);
  if (t >= end) return;
  in += t * stride;
  out += t * out_stride;
  // (each thread reads back only what it copied itself: no barrier)
  __shared__ Raw<T> ring[kStages][2][kRopeMaxWarps * 32];
  int fetched = t, slot = 0, from = 0;
  auto fetch = [&]() {
    if (mine && fetched < end) {
      copy_async(&ring[slot][0][threadIdx.x], in + ca);
      copy_async(&ring[slot][1][threadIdx.x], in + cb);
    }
    copy_commit();
    in += stride;
    ++fetched;
    slot = slot + 1 < kStages ? slot + 1 : 0;
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch();
  int pos = locate(t);
  Eight c{}, s{};
  turns_of(pos, c, s);
  while (true) {
    const int tn = t + 1;
    fetch();
    const int next = tn < end ? locate(tn) : -1;
    Eight nc{}, ns{};
    turns_of(next, nc, ns);
    copy_wait<kStages - 1>();
    if (pos >= 0) {
      Eight a{}, b{};
      if (mine) {
        a = widen(ring[from][0][threadIdx.x]);
        b = widen(ring[from][1][threadIdx.x]);
      }
      float2 sq = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        sq = ffma2(make_float2(a.x[i], a.x[i + 1]), make_float2(a.x[i], a.x[i + 1]), sq);
        sq = ffma2(make_float2(b.x[i], b.x[i + 1]), make_float2(b.x[i], b.x[i + 1]), sq);
      }
      float ss = sq.x + sq.y;
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (weight != nullptr) {
        const float r = rsqrtf(ss / (float)p.d + p.eps);
        const Eight u = widen(wa), v = widen(wb);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 r2 = make_float2(r, r);
          const float2 y = fmul2(fmul2(make_float2(a.x[i], a.x[i + 1]), r2), make_float2(u.x[i], u.x[i + 1]));
          const float2 z = fmul2(fmul2(make_float2(b.x[i], b.x[i + 1]), r2), make_float2(v.x[i], v.x[i + 1]));
          a.x[i] = y.x, a.x[i + 1] = y.y, b.x[i] = z.x, b.x[i + 1] = z.y;
        }
      }
      if (turns) {
        if (kInterleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = a.x[2 * i], v = a.x[2 * i + 1];
            a.x[2 * i] = u * c.x[i] - v * s.x[i];
            a.x[2 * i + 1] = v * c.x[i] + u * s.x[i];
            if (cb >= p.rot) continue;
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
      if (mine) {
        store8(out + ca, a);
        store8(out + cb, b);
      }
    }
    if (tn >= end) return;
    out += out_stride;
    t = tn;
    pos = next;
    from = from + 1 < kStages ? from + 1 : 0;
    c = nc;
    s = ns;
  }
}

template <typename T, int LPH>
static cudaError_t launch_rope(const RopeArgs& p, bool interleaved, int total_nodes, cudaStream_t stream) {
  const int heads = p.hq + p.hkv + (p.v_in != nullptr ? p.hkv : 0);
  const int warps = ceil_div(heads, 32 / LPH);
  const int y = ceil_div(warps, kRopeMaxWarps);
  const dim3 block(ceil_div(warps, y) * 32);
  // kRopeThreads an SM, each CTA with its share of the nodes
  const int resident = ceil_div(sm_count() * (kRopeThreads / (int)block.x), y);
  const dim3 grid(total_nodes < resident ? total_nodes : resident, y);
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
                   rot,  prefix_len, depth, qo,       batch,    total_nodes, hq,       hkv,      d,        q_out, k_out,   v_out,
                   status};
  const cudaError_t e = dtype == SPEC_F32 ? launch_rope_d<float>(p, interleaved, total_nodes, stream)
                                          : launch_rope_d<__nv_bfloat16>(p, interleaved, total_nodes, stream);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
