// Norm of every query and key head and the rotation of its position, in one pass.
//
//     n = norm(x) * weight + bias                    over the head's D elements
//     (u, v) -> (u c - v s, u s + v c)               pairs i < rot / 2, (c, s) = angle[pos][i]
//
// A group of G = 4, 8, 16 or 32 lanes holds one head, eight consecutive elements to a lane (one
// 16-byte load and store). The sums of the norm are a butterfly over the group's lanes; a pair
// (2i, 2i + 1) lies in one lane, a pair (i, i + rot / 2) in two lanes rot / 16 apart, which
// exchange their elements, as they were read, by shuffles. Weight, bias, angle and sign are folded
// into three factors per element, once for the heads of a group. Everything is float32, rounded to
// bf16 once.
//
// Bound by HBM: 2 x 8192 tokens x (32 + 8) heads of 128, 340 MB, take 57 us (6.0 TB/s, 91 % of the
// measured copy rate; 4096 x 60 heads of 64: 13.6 us). What that needs is bytes in flight and few
// instructions: the elements come by cp.async into slots of shared memory that only their own
// thread reads (three stages of two heads to a group, no registers held), the factors are made once
// for up to 32 heads, and the pairing is a template parameter. A head to a group with everything in
// registers took 157 us, four heads 93, the slots 65, the pairing as a branch 61.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "oq_internal.h"

namespace oq {
namespace {

constexpr int HT = 128;   // threads
constexpr int HB = 7;     // blocks to an SM

struct HeadParams {
  HeadIo q, k;
  int64_t seq;
  int64_t tokens;
  int D, norm, rope, rot;
  int chunk_q, chunk_k;       // heads of a chunk
  int cq, ck;                 // chunks of a token
  bool dependent;             // begin beside the launch before (float input)
  bool small;                 // items (tokens x chunks) within 31 bits
  float eps, inv_d;
  const float* cos;
  const float* sin;
  int64_t n_pos;
  const int32_t* positions;
  int64_t pos_bs;
};

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
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

// Eight elements of one head on their way from global memory to a slot of shared memory that only
// their own thread reads, and from there as pairs, and those of another lane.
__device__ __forceinline__ void async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <typename TIN>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  static constexpr int kBytes = 16;
  uint4 v;
  static __device__ __forceinline__ void send(uint32_t slot, const __nv_bfloat16* p) {
    async16(slot, p);
  }
  __device__ __forceinline__ void take(const uint8_t* slot) {
    v = *reinterpret_cast<const uint4*>(slot);
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
    x[0] = unpack2(v.x); x[1] = unpack2(v.y); x[2] = unpack2(v.z); x[3] = unpack2(v.w);
  }
  __device__ __forceinline__ void get_from(int lane, bool take, float2 (&x)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t o = __shfl_sync(0xffffffffu, w[j], lane);
      x[j] = unpack2(take ? o : 0u);
    }
  }
};
template <>
struct Raw<float> {
  static constexpr int kBytes = 32;
  float4 v[2];
  static __device__ __forceinline__ void send(uint32_t slot, const float* p) {
    async16(slot, p);
    async16(slot + 16, p + 4);
  }
  __device__ __forceinline__ void take(const uint8_t* slot) {
    v[0] = *reinterpret_cast<const float4*>(slot);
    v[1] = *reinterpret_cast<const float4*>(slot + 16);
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
    x[0] = make_float2(v[0].x, v[0].y); x[1] = make_float2(v[0].z, v[0].w);
    x[2] = make_float2(v[1].x, v[1].y); x[3] = make_float2(v[1].z, v[1].w);
  }
  __device__ __forceinline__ void get_from(int lane, bool take, float2 (&x)[4]) const {
    get(x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = __shfl_sync(0xffffffffu, x[j].x, lane);
      const float b = __shfl_sync(0xffffffffu, x[j].y, lane);
      x[j] = take ? make_float2(a, b) : make_float2(0.f, 0.f);
    }
  }
};

// A chunk of one token's heads to a group, U at a time: the factors are made once for them, and a
// round's loads are in flight while the round before is computed.
template <typename TIN, int G, int U, int NS, bool HALVES>
__global__ void __launch_bounds__(HT, HB) k_heads(const HeadParams p) {
  constexpr int SB = Raw<TIN>::kBytes;
  __shared__ __align__(16) uint8_t s_slot[NS][U][HT][SB];
  // Items: every token's query chunks, then every token's key chunks, so that a warp's groups make
  // as many rounds.
  uint64_t item = ((uint64_t)blockIdx.x * HT + threadIdx.x) / G;
  const uint64_t nq = (uint64_t)p.tokens * (uint32_t)p.cq;
  const bool is_q = item < nq;
  if (!is_q) item -= nq;
  const uint32_t nch = (uint32_t)max(is_q ? p.cq : p.ck, 1);
  int64_t t;
  int c;
  if (p.small) {   // 32-bit division where the items allow it
    t = (uint32_t)item / nch;
    c = (int)((uint32_t)item - (uint32_t)t * nch);
  } else {
    t = (int64_t)(item / nch);
    c = (int)(item - (uint64_t)t * nch);
  }
  const HeadIo& io = is_q ? p.q : p.k;
  const int chunk = is_q ? p.chunk_q : p.chunk_k;
  // the last block's spare groups follow along to the shuffles
  const bool live = t < p.tokens && (is_q ? p.cq : p.ck) > 0;
  if (!live) t = 0, c = 0;
  const int h0 = c * chunk;
  const int h1 = live ? min(io.heads, h0 + chunk) : h0;   // this group's heads [h0, h1)
  const int64_t b = (uint32_t)t / (uint32_t)p.seq, s = t - b * p.seq;   // tokens < 2^31
  const int lg = threadIdx.x & (G - 1), e0 = lg * 8;
  const bool on = e0 < p.D;
  int64_t pos = s;   // read ahead of everything that waits for it
  if (p.positions) pos = p.positions[b * p.pos_bs + s];
  const int rounds = __reduce_max_sync(0xffffffffu, (h1 - h0 + U - 1) / U);   // of the warp

  const TIN* src = reinterpret_cast<const TIN*>(io.in) + b * io.si[0] + s * io.si[1] +
                   (int64_t)h0 * io.si[2] + e0;   // of the next heads to fetch
  const uint32_t slot0 = (uint32_t)__cvta_generic_to_shared(s_slot[0][0][threadIdx.x]);
  if (!on) {   // lanes past the head: zeros that no load replaces (they enter the group's sums)
#pragma unroll
    for (int i = 0; i < NS * U * SB / 16; ++i)
      *reinterpret_cast<uint4*>(&s_slot[i / (U * SB / 16)][i / (SB / 16) % U][threadIdx.x][16 * (i % (SB / 16))]) =
          make_uint4(0u, 0u, 0u, 0u);
  }
  // U heads into stage st; an empty group where there are none, so that the groups can be counted
  auto fetch = [&](int st, int h) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (on && h + u < h1)
        Raw<TIN>::send(slot0 + (uint32_t)((st * U + u) * HT * SB), src + u * io.si[2]);
    src += U * io.si[2];
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Float input comes from a GEMM that this grid may begin beside: the factors, which do not, are
  // made first. Else the elements are asked for first.
  constexpr bool kAfter = std::is_same<TIN, float>::value;
  if constexpr (!kAfter) {
#pragma unroll
    for (int st = 0; st < NS; ++st) fetch(st, h0 + st * U);
  }
  // Element x of a pair whose other element is o becomes r (x A + o B) + C, r the norm's factor:
  // A = w c, B = -/+ w_o s, C = b c -/+ b_o s (o, w_o, b_o of the other element); A = w, B = 0,
  // C = b, o = 0 where nothing is turned, so that an infinity stays in its element.
  float2 A[4], B[4], C[4];
  const int half = p.rot / 2;
  constexpr bool pairs = !HALVES;   // or nothing is turned
  bool turn = false;   // this lane's elements are turned
  int eo = e0;         // where the other elements lie (halves)
  {
    float w[8], bs[8], c[8], sn[8] = {}, wo[8], bo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) { w[j] = c[j] = wo[j] = 1.f; bs[j] = bo[j] = 0.f; }
    if (on && io.weight) load8(io.weight + e0, w);
    if (on && io.bias) load8(io.bias + e0, bs);
    if (p.rope != OQ_ROPE_NONE && e0 < p.rot) {
      turn = pos >= 0;
      if (!pairs) eo = e0 < half ? e0 + half : e0 - half;
      if (pos >= p.n_pos) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = sn[j] = __int_as_float(0x7fc00000);
      } else if (turn && pairs) {
        const float4 a = *reinterpret_cast<const float4*>(p.cos + pos * half + e0 / 2);
        const float4 d = *reinterpret_cast<const float4*>(p.sin + pos * half + e0 / 2);
        c[0] = c[1] = a.x; c[2] = c[3] = a.y; c[4] = c[5] = a.z; c[6] = c[7] = a.w;
        sn[0] = -d.x; sn[1] = d.x; sn[2] = -d.y; sn[3] = d.y;
        sn[4] = -d.z; sn[5] = d.z; sn[6] = -d.w; sn[7] = d.w;
      } else if (turn) {
        const int i0 = e0 < half ? e0 : e0 - half;
        load8(p.cos + pos * half + i0, c);
        load8(p.sin + pos * half + i0, sn);
        if (e0 < half) {
#pragma unroll
          for (int j = 0; j < 8; ++j) sn[j] = -sn[j];
        }
      }
      if (turn && !pairs && io.weight) load8(io.weight + eo, wo);
      if (turn && !pairs && io.bias) load8(io.bias + eo, bo);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if (pairs) {   // the other element is the neighbour
        wo[j] = w[j + 1]; wo[j + 1] = w[j];
        bo[j] = bs[j + 1]; bo[j + 1] = bs[j];
      }
      A[j / 2] = make_float2(w[j] * c[j], w[j + 1] * c[j + 1]);
      B[j / 2] = make_float2(wo[j] * sn[j], wo[j + 1] * sn[j + 1]);
      C[j / 2] = make_float2(bs[j] * c[j] + bo[j] * sn[j], bs[j + 1] * c[j + 1] + bo[j + 1] * sn[j + 1]);
    }
  }
  const int mate = (threadIdx.x & 31) + (eo - e0) / 8;
  if constexpr (kAfter) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
    for (int st = 0; st < NS; ++st) fetch(st, h0 + st * U);
  }

  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(io.out) + b * io.so[0] + s * io.so[1] +
                       (int64_t)h0 * io.so[2] + e0;
  int h = h0, st = 0;
  for (int i = 0; i < rounds; ++i, h += U) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");   // this stage's has landed
    Raw<TIN> cur[U];
#pragma unroll
    for (int u = 0; u < U; ++u) cur[u].take(s_slot[st][u][threadIdx.x]);   // past the last head: unused
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 x[4], o[4];
      cur[u].get(x);
      if constexpr (HALVES) {
        cur[u].get_from(mate, turn, o);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = turn ? make_float2(x[j].y, x[j].x) : make_float2(0.f, 0.f);
      }
      if (p.norm == OQ_NORM_LAYER) {
        float2 m2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) m2 = __fadd2_rn(m2, x[j]);
        const float m = -group_sum<G>(m2.x + m2.y) * p.inv_d;
        // lanes past the head stay zero
        const float2 mx = on ? make_float2(m, m) : make_float2(0.f, 0.f);
        const float2 mo = turn ? mx : make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = __fadd2_rn(x[j], mx);
          o[j] = __fadd2_rn(o[j], mo);
        }
      }
      float r = 1.f;
      if (p.norm != OQ_NORM_NONE) {
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) q = __ffma2_rn(x[j], x[j], q);
        r = rsqrtf(fmaf(group_sum<G>(q.x + q.y), p.inv_d, p.eps));
      }
      const float2 r2 = make_float2(r, r);
      uint32_t out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = __ffma2_rn(r2, __ffma2_rn(x[j], A[j], __fmul2_rn(o[j], B[j])), C[j]);
        const __nv_bfloat162 v = __float22bfloat162_rn(y);
        out[j] = *reinterpret_cast<const uint32_t*>(&v);
      }
      if (on && h + u < h1)
        *reinterpret_cast<uint4*>(dst + u * io.so[2]) =
            make_uint4(out[0], out[1], out[2], out[3]);
    }
    dst += U * io.so[2];
    fetch(st, h + NS * U);   // this thread has read its slots
    st = st + 1 == NS ? 0 : st + 1;
  }
}

template <typename TIN, int G, int U, int NS, bool HALVES>
oq_status run_u(HeadParams& p, int chunk, cudaStream_t s) {
  auto cut = [&](int heads, int& chunks, int& size) {   // into chunks of about the same size
    chunks = (heads + chunk - 1) / chunk;
    size = chunks ? (heads + chunks - 1) / chunks : 1;
  };
  cut(p.q.heads, p.cq, p.chunk_q);
  cut(p.k.heads, p.ck, p.chunk_k);
  const int64_t items = p.tokens * (p.cq + p.ck), blocks = (items * G + HT - 1) / HT;
  if (blocks > 0x7FFFFFFF)
    return fail(OQ_ERR_INVALID_ARG, "too many heads in one call: split the batch");
  p.small = items + HT < (int64_t)0x7FFFFFFF;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(HT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = std::is_same<TIN, float>::value && p.dependent ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_heads<TIN, G, U, NS, HALVES>, p);
  return e == cudaSuccess ? OQ_OK : cuda_fail(e, "launch heads");
}

template <typename TIN, int G, bool HALVES>
oq_status run(HeadParams& p, cudaStream_t s) {
  // Chunks of at most 32 heads, and so long that they occupy about half of the groups that the device
  // holds at once: a group starts slowly (position, angle, factors, the first loads, one after the
  // other), then streams with three stages in flight, of which half the groups have enough. Measured
  // against one chunk to every group, and two: 3 x 777 tokens x 24 heads of 96 8.1 us, 9.5, 11.5;
  // 1024 x 40 of 128 6.8, 8.1, 10.1; 4096 x 60 of 64 13.6, 14.5, 15.9; 512 x 32 of 256 6.0, 8.2, 13.6;
  // 4096 x 40 of 128 17.0, 16.0, 18.7; 2 x 8192 x 40 56.9 all (32 heads everywhere). Below a head to a
  // group, one head each.
  const int64_t heads = p.tokens * (p.q.heads + p.k.heads), groups = (int64_t)device_sms() * HB * HT / G;
  if (heads <= groups) return run_u<TIN, G, 1, 1, HALVES>(p, 1, s);
  return run_u<TIN, G, 2, 3, HALVES>(p, (int)std::min<int64_t>(2 * heads / groups, 32), s);
}

template <typename TIN, int G>
oq_status run_rope(HeadParams& p, cudaStream_t s) {
  return p.rope == OQ_ROPE_HALVES ? run<TIN, G, true>(p, s) : run<TIN, G, false>(p, s);
}

template <typename TIN>
oq_status run_g(HeadParams& p, cudaStream_t s) {
  if (p.D <= 32) return run_rope<TIN, 4>(p, s);
  if (p.D <= 64) return run_rope<TIN, 8>(p, s);
  if (p.D <= 128) return run_rope<TIN, 16>(p, s);
  return run_rope<TIN, 32>(p, s);
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
  p.dependent = a.dependent;
  return a.in_f32 ? run_g<float>(p, s) : run_g<__nv_bfloat16>(p, s);
}

}  // namespace oq
