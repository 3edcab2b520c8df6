// W8A8 GEMM: int8 activations against int8 weights, exact int32 sums, the dequant epilogue of
// the INT4 GEMMs.
//
//     acc[t, o] = sum_k a[t, k] w[o, k]
//     y[t, o]   = bf16( alpha_t s_o acc + (mean_t w1_o + b_o) )
//
// A plain tiled kernel: 64 tokens x 64 channels per block, 64 bytes of K at a time through
// shared memory, four-way byte dot products.
#include <cuda_bf16.h>

#include <algorithm>

#include "oq_internal.h"

namespace oq {
namespace {

constexpr int BT = 64, BO = 64, BKB = 64;

struct W8Params {
  const int8_t* a;
  const int8_t* w;
  const float* a_scale;
  const float* mean;
  const float* w_scale;
  const float* w_rowsum;
  const __nv_bfloat16* bias;
  int64_t T;
  int K, N, out_acc, n_head;
  void* out;
  float* head;
};

__device__ __forceinline__ void store_one(const W8Params& p, int64_t t, int o, int acc) {
  if (p.out_acc) {
    reinterpret_cast<int32_t*>(p.out)[t * p.N + o] = acc;
    return;
  }
  const float c = __fmaf_rn(p.mean ? p.mean[t] : 0.f, p.mean ? p.w_rowsum[o] : 0.f,
                            p.bias ? __bfloat162float(p.bias[o]) : 0.f);
  const float y = __fmaf_rn((float)acc, __fmul_rn(p.a_scale[t], p.w_scale[o]), c);
  if (o < p.n_head)
    p.head[t * p.n_head + o] = y;
  else
    reinterpret_cast<__nv_bfloat16*>(p.out)[t * p.N + o] = __float2bfloat16_rn(y);
}

__global__ void __launch_bounds__(256) k_gemm_w8_plain(const W8Params p) {
  __shared__ int sa[BT][BKB / 4 + 1], sw[BO][BKB / 4 + 1];
  const int64_t t0 = (int64_t)blockIdx.y * BT;
  const int o0 = blockIdx.x * BO;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += BKB) {
    for (int i = threadIdx.x; i < BT * BKB / 4; i += 256) {
      const int r = i / (BKB / 4), c = i % (BKB / 4);
      const int k = k0 + 4 * c;
      sa[r][c] = (t0 + r < p.T && k < p.K)
                     ? *reinterpret_cast<const int*>(p.a + (t0 + r) * p.K + k) : 0;
      sw[r][c] = (o0 + r < p.N && k < p.K)
                     ? *reinterpret_cast<const int*>(p.w + (int64_t)(o0 + r) * p.K + k) : 0;
    }
    __syncthreads();
    for (int c = 0; c < BKB / 4; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __dp4a(sa[ty + 16 * i][c], sw[tx + 16 * j][c], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + ty + 16 * i;
      const int o = o0 + tx + 16 * j;
      if (t < p.T && o < p.N) store_one(p, t, o, acc[i][j]);
    }
}

}  // namespace

oq_status launch_gemm_w8(const GemmW8Args& g, cudaStream_t s) {
  if (g.T == 0) return OQ_OK;
  W8Params p{g.a, g.w, g.a_scale, g.mean, g.w_scale, g.w_rowsum,
             reinterpret_cast<const __nv_bfloat16*>(g.bias), g.T, (int)g.K, (int)g.N, g.out_acc,
             (int)g.n_head, g.out, g.head};
  // token tiles past the grid's y limit run in further launches
  for (int64_t t0 = 0; t0 < g.T; t0 += (int64_t)65535 * BT) {
    const int64_t n = std::min<int64_t>(g.T - t0, (int64_t)65535 * BT);
    W8Params q = p;
    q.a = p.a + t0 * p.K;
    q.a_scale = p.a_scale + t0;
    q.mean = p.mean ? p.mean + t0 : nullptr;
    q.T = n;
    q.out = static_cast<uint8_t*>(p.out) + (size_t)t0 * p.N * (p.out_acc ? 4 : 2);
    q.head = p.head ? p.head + t0 * p.n_head : nullptr;
    k_gemm_w8_plain<<<dim3((unsigned)((g.N + BO - 1) / BO), (unsigned)((n + BT - 1) / BT)), 256,
                      0, s>>>(q);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "launch gemm_w8");
  }
  return OQ_OK;
}

}  // namespace oq
