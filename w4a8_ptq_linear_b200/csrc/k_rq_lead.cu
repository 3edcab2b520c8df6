// The INT8 rotate-quantize in front of a GEMM that may start beside it: the two-token body of the
// standalone kernel (rq_device.cuh, the same result bit for bit), in a kernel that lets its
// dependent launch begin at once. The W8A8 GEMM then sets up, and fetches weights, while the
// tokens are rotated, and waits for this grid to end (griddepcontrol.wait) before it reads a code.
#include <cuda_bf16.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <new>
#include <tuple>

#include "oq_internal.h"
#include "ptx.cuh"

#include "rq_device.cuh"

namespace oq {
namespace {

template <int HLOG2, int ROUNDS>
__global__ void __launch_bounds__(256, 2) k_rq_lead(const RqParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  rq_pair_body<HLOG2, ROUNDS, kRqInt8>(p, smem, (int)blockIdx.x, (int)gridDim.x, (int)blockDim.x,
                                       false);
}

template <int R>
const void* lead_kernel(int hlog2) {
  switch (hlog2) {
    case 0: return reinterpret_cast<const void*>(&k_rq_lead<0, R>);
    case 1: return reinterpret_cast<const void*>(&k_rq_lead<1, R>);
    case 2: return reinterpret_cast<const void*>(&k_rq_lead<2, R>);
    case 3: return reinterpret_cast<const void*>(&k_rq_lead<3, R>);
    case 4: return reinterpret_cast<const void*>(&k_rq_lead<4, R>);
    case 5: return reinterpret_cast<const void*>(&k_rq_lead<5, R>);
    case 6: return reinterpret_cast<const void*>(&k_rq_lead<6, R>);
    case 7: return reinterpret_cast<const void*>(&k_rq_lead<7, R>);
    case 8: return reinterpret_cast<const void*>(&k_rq_lead<8, R>);
    case 9: return reinterpret_cast<const void*>(&k_rq_lead<9, R>);
    default: return reinterpret_cast<const void*>(&k_rq_lead<10, R>);
  }
}

}  // namespace

oq_status launch_rotate_quant_lead(const RqArgs& a, cudaStream_t s) try {
  if (a.mode != kRqInt8 || a.d > kRqPairMaxD)
    return fail(OQ_ERR_UNSUPPORTED, "leading rotate-quantize: INT8 absmax, d <= %d", kRqPairMaxD);
  if (a.T == 0) return OQ_OK;
  RqParams p;
  int threads = 0;
  size_t smem = 0;
  oq_status st = rq_pair_setup(a, p, threads, smem);
  if (st != OQ_OK) return st;
  int hlog2 = 0;
  while ((1 << hlog2) < a.h) ++hlog2;
  const void* fn = a.rounds == 1 ? lead_kernel<1>(hlog2) : lead_kernel<2>(hlog2);
  // blocks that are resident at once, per (device, kernel, width)
  int resident = 0;
  {
    static std::mutex mu;
    static std::map<std::tuple<int, const void*, int>, int> kept;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lock(mu);
    int& n = kept[std::make_tuple(dev, fn, a.d)];
    if (n == 0) {
      e = allow_max_dynamic_smem(fn);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(rq_lead)");
      int per_sm = 0;
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, threads, smem);
      if (e != cudaSuccess) return cuda_fail(e, "occupancy(rq_lead)");
      n = std::max(per_sm, 1) * device_sms();
    }
    resident = n;
  }
  const unsigned grid = (unsigned)std::min<int64_t>((a.T + 1) / 2, resident);
  void* args[] = {&p};
  const cudaError_t e = cudaLaunchKernel(fn, dim3(grid), dim3((unsigned)threads), args, smem, s);
  return e == cudaSuccess ? OQ_OK : cuda_fail(e, "launch rq_lead");
} catch (const std::bad_alloc&) {   // of the kept launch shapes
  return fail(OQ_ERR_NOMEM, "host allocation");
}

}  // namespace oq
