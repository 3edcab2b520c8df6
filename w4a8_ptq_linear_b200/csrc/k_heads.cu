// Norm of every query and key head and the rotation of its position, in one pass.
//
//     n = norm(x) * weight + bias                    over the head's D elements
//     (u, v) -> (u c - v s, u s + v c)               pairs i < rot / 2, (c, s) = angle[pos][i]
//
// A group of G = 4, 8, 16 or 32 lanes holds one head, eight consecutive elements to a lane (one
// 16-byte load and store). The sums of the norm are a butterfly over the group's lanes; a pair
// (2i, 2i + 1) lies in one lane, a pair (i, i + rot / 2) in two lanes rot / 16 apart, which
// exchange their elements by shuffles. Everything is float32, rounded to bf16 once.
#include <cuda_bf16.h>

#include <algorithm>

#include "oq_internal.h"

namespace oq {
namespace {

struct HeadParams {
  HeadIo q, k;
  int64_t seq;
  int64_t tokens;
  int D, norm, rope, rot;
  int cq, ck;                 // chunks of U heads: queries, keys
  float eps, inv_d;
  const float* cos;
  const float* sin;
  int64_t n_pos;
  const int32_t* positions;
  int64_t pos_bs;
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// U heads of one token to a group.
template <typename TIN, int G, int U>
__global__ void __launch_bounds__(256) k_heads(const HeadParams p) {
  const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G;
  const int nch = p.cq + p.ck;
  int64_t t = item / nch;
  int c = (int)(item - t * nch);
  const bool live = t < p.tokens;   // the last block's spare groups follow along to the shuffles
  if (!live) t = 0, c = 0;
  const bool is_q = c < p.cq;
  const HeadIo& io = is_q ? p.q : p.k;
  const int h0 = (is_q ? c : c - p.cq) * U;
  const int64_t b = t / p.seq, s = t - b * p.seq;
  const int lg = threadIdx.x & (G - 1), e0 = lg * 8;
  const bool on = e0 < p.D;

  float x[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[u][j] = 0.f;
    if (on && live && h0 + u < io.heads)
      load8(reinterpret_cast<const TIN*>(io.in) + b * io.si[0] + s * io.si[1] +
                (int64_t)(h0 + u) * io.si[2] + e0, x[u]);
  }
  float w[8], bs[8], cs[8] = {}, sn[8] = {};
#pragma unroll
  for (int j = 0; j < 8; ++j) { w[j] = 1.f; bs[j] = 0.f; }
  if (on && io.weight) load8(io.weight + e0, w);
  if (on && io.bias) load8(io.bias + e0, bs);
  const int half = p.rot / 2;
  bool turn = false;   // this lane's elements are rotated
  if (p.rope != OQ_ROPE_NONE && e0 < p.rot) {
    const int64_t pos = p.positions ? (int64_t)p.positions[b * p.pos_bs + s] : s;
    turn = pos >= 0;
    if (pos >= p.n_pos) {
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = sn[j] = __int_as_float(0x7fc00000);
    } else if (pos >= 0) {
      if (p.rope == OQ_ROPE_PAIRS) {
        const float4 a = *reinterpret_cast<const float4*>(p.cos + pos * half + e0 / 2);
        const float4 d = *reinterpret_cast<const float4*>(p.sin + pos * half + e0 / 2);
        cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
        sn[0] = d.x; sn[1] = d.y; sn[2] = d.z; sn[3] = d.w;
      } else {
        const int i0 = e0 < half ? e0 : e0 - half;
        load8(p.cos + pos * half + i0, cs);
        load8(p.sin + pos * half + i0, sn);
      }
    }
  }
  // the lane that holds the other half of this lane's pairs (halves), and this lane's sign:
  // u c - v s below half, v c + u s above
  const int lane = threadIdx.x & 31;
  const int mate = e0 < half ? lane + half / 8 : e0 < p.rot ? lane - half / 8 : lane;
  const float sgn = e0 < half ? -1.f : 1.f;

#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (p.norm == OQ_NORM_LAYER) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m += x[u][j];
      m = group_sum<G>(m) * p.inv_d;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[u][j] = on ? x[u][j] - m : 0.f;
    }
    float r = 1.f;
    if (p.norm != OQ_NORM_NONE) {
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) q = fmaf(x[u][j], x[u][j], q);
      r = rsqrtf(fmaf(group_sum<G>(q), p.inv_d, p.eps));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[u][j] = fmaf(x[u][j] * r, w[j], bs[j]);
    float y[8];
    if (p.rope == OQ_ROPE_PAIRS) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = x[u][2 * j], d = x[u][2 * j + 1];
        y[2 * j] = turn ? a * cs[j] - d * sn[j] : a;
        y[2 * j + 1] = turn ? a * sn[j] + d * cs[j] : d;
      }
    } else if (p.rope == OQ_ROPE_HALVES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float o = __shfl_sync(0xffffffffu, x[u][j], mate);
        y[j] = turn ? x[u][j] * cs[j] + sgn * o * sn[j] : x[u][j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = x[u][j];
    }
    if (on && live && h0 + u < io.heads) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(io.out) + b * io.so[0] +
                                s * io.so[1] + (int64_t)(h0 + u) * io.so[2] + e0) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <typename TIN, int G>
oq_status run(HeadParams& p, cudaStream_t s) {
  constexpr int U = 1;
  p.cq = (p.q.heads + U - 1) / U;
  p.ck = (p.k.heads + U - 1) / U;
  const int64_t blocks = (p.tokens * (p.cq + p.ck) * G + 255) / 256;
  if (blocks > 0x7FFFFFFF)
    return fail(OQ_ERR_INVALID_ARG, "too many heads in one call: split the batch");
  k_heads<TIN, G, U><<<(unsigned)blocks, 256, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? OQ_OK : cuda_fail(e, "launch heads");
}

template <typename TIN>
oq_status run_g(HeadParams& p, cudaStream_t s) {
  if (p.D <= 32) return run<TIN, 4>(p, s);
  if (p.D <= 64) return run<TIN, 8>(p, s);
  if (p.D <= 128) return run<TIN, 16>(p, s);
  return run<TIN, 32>(p, s);
}

}  // namespace

oq_status launch_heads(const HeadArgs& a, cudaStream_t s) {
  if (a.batch == 0 || a.seq == 0) return OQ_OK;
  HeadParams p{};
  p.q = a.q;
  p.k = a.k;
  p.seq = a.seq;
  p.tokens = a.batch * a.seq;
  p.D = a.head_dim;
  p.norm = a.norm;
  p.rope = a.rope;
  p.rot = a.rope == OQ_ROPE_NONE ? 0 : a.rot_dim;
  p.eps = a.eps;
  p.inv_d = 1.f / (float)a.head_dim;
  p.cos = a.cos;
  p.sin = a.sin;
  p.n_pos = a.n_pos;
  p.positions = a.positions;
  p.pos_bs = a.pos_batch_stride;
  return a.in_f32 ? run_g<float>(p, s) : run_g<__nv_bfloat16>(p, s);
}

}  // namespace oq
