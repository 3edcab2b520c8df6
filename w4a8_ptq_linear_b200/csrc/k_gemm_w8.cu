// W8A8 GEMM: int8 activations against int8 weights, exact int32 sums, the dequant epilogue of
// the INT4 GEMMs.
//
//     acc[t, o] = sum_k a[t, k] w[o, k]
//     y[t, o]   = bf16( alpha_t s_o acc + (mean_t w1_o + b_o) )
//
// Every shape of the kernel takes the same float steps (fma(acc, alpha s, fma(mean, w1, b))), so a
// token's result does not depend on how many tokens it comes with.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>
#include <vector>

#include "oq_internal.h"
#include "ptx.cuh"

namespace oq {

bool tma_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner,
                uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                CUtensorMapSwizzle sw);

namespace {

struct W8Params {
  const int8_t* a;
  const int8_t* w;
  const float* a_scale;
  const float* mean;
  const float* w_scale;
  const float* w_rowsum;
  const __nv_bfloat16* bias;
  int T, K, N, out_acc, n_head;
  void* out;
  float* head;
  unsigned long long* err;
  unsigned long long limit_ns;
};

// ---- tiles on CTA pairs ----------------------------------------------------------------------
// D[t, o] on tcgen05 (kind::i8, cta_group::2): 256 tokens are the M rows, up to 256 channels the
// N columns, so that a thread of the epilogue holds one token's row of the accumulator: its scale
// and mean are two registers, the channels' constants are broadcast from shared memory, and
// sums over a row stay in the thread.
//
// One persistent CTA pair per two SMs. Both operands come by TMA, K-major, 128 bytes of K to a
// block; two producer threads, one to an operand (one thread's TMA reads from L2 run at about
// 32 bytes a clock, a full tile needs 64 per CTA). TMEM holds two accumulators of 256 columns, so a
// tile's epilogue runs under the next tile's MMAs.
//
// What bounds it: a 256 x 256 tile reads 64 KB per 128 bytes of K for 2 * 256 * 256 * 128 operations,
// 64 bytes a clock and SM at the tensor pipe's full rate, which is about what L2 delivers.
//
// Schedule: a pair takes a contiguous range of the (token block, channel chunk) space, cut into
// tiles of at most 256 channels. A tile costs its chunks and, whatever its width, the 128 token rows
// of each CTA, so the ranges are chosen by a cost of chunks plus a fixed part per tile.
constexpr int TM = 128;                    // tokens per CTA
constexpr int TN = 256;                    // channels per tile at most
constexpr int CH = 32;                     // channels per chunk
constexpr int SK = 6;                      // stages of one 128-byte K block
constexpr int AB = TM * 128;               // activation bytes of a stage
constexpr int BB = (TN / 2) * 128;         // weight bytes of a stage (this CTA's half)
constexpr int BBOX = 64;                   // weight rows of one TMA load
constexpr int NEPI = 256;                  // epilogue threads, two warps to a TMEM lane quarter
constexpr int NTHR = 128 + NEPI;
constexpr int STG = 32 * 64;               // staging tile: 32 tokens x 64 bytes
constexpr int OFF_B = SK * AB;
constexpr int OFF_STG = OFF_B + SK * BB;
constexpr int OFF_COL = OFF_STG + (NEPI / 32) * STG;   // [2][3][TN] floats
constexpr int OFF_BAR = OFF_COL + 2 * 3 * TN * 4;
constexpr int NBAR = 2 * SK + 5;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int SMEM = OFF_MISC + 16 + 1024;
constexpr int kMaxUnits = 96;              // CTA pairs at most
static_assert(SMEM <= 232448, "shared memory");

struct TileParams {
  W8Params w;
  int npm;                                 // chunks of a token block
  int sched[kMaxUnits + 1];                // pair u: chunks [sched[u], sched[u + 1])
};

// The tiles of one pair's range; every role walks the same sequence.
struct Tiles {
  int npm, maxch, cur, end;
  __device__ Tiles(const TileParams& p, int unit, int maxch_)
      : npm(p.npm), maxch(maxch_), cur(p.sched[unit]), end(p.sched[unit + 1]) {}
  // token block m, first chunk c0, number of chunks n
  __device__ bool next(int& m, int& c0, int& n) {
    if (cur >= end) return false;
    m = cur / npm;
    c0 = cur - m * npm;
    const int left = min(end, (m + 1) * npm) - cur;
    const int cuts = (left + maxch - 1) / maxch;
    n = (left + cuts - 1) / cuts;
    cur += n;
    return true;
  }
};

// y of two neighbouring channels: c = fma(mean, w1, b), y = fma(acc, alpha s, c)
__device__ __forceinline__ float2 dequant2(int a0, int a1, float alpha, float mean, float2 s,
                                           float2 w1, float2 b) {
  const float2 c = __ffma2_rn(make_float2(mean, mean), w1, b);
  return __ffma2_rn(make_float2((float)a0, (float)a1),
                    __fmul2_rn(make_float2(alpha, alpha), s), c);
}

__global__ void __launch_bounds__(NTHR, 1)
    k_gemm_w8(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_h,
              const __grid_constant__ TileParams tp) {
  const W8Params& p = tp.w;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* s_col = reinterpret_cast<float*>(smem + OFF_COL);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* s_misc = reinterpret_cast<uint32_t*>(smem + OFF_MISC);   // TMEM base, abort, decisions
  volatile uint32_t* s_abort = s_misc + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = dev::cluster_ctarank();
  const int unit = (int)blockIdx.x / 2;
  const int nkb = (p.K + 127) / 128;
  auto bar = [&](int i) { return dev::smem_u32(&bars[i]); };
  auto full_bar = [&](int s) { return bar(s); };
  auto free_bar = [&](int s) { return bar(SK + s); };
  auto tfull_bar = [&](int b) { return bar(2 * SK + b); };
  auto tempty_bar = [&](int b) { return bar(2 * SK + 2 + b); };
  const uint32_t drain_bar = bar(2 * SK + 4);
  auto lead = [&](uint32_t a) { return dev::map_to_cta(a, 0); };
  auto give_up = [&]() { *s_abort = 1; };

  if (tid == 0) {
    for (int s = 0; s < SK; ++s) {
      dev::mbar_init(full_bar(s), 2);     // the leader's two producers (and the bytes of both CTAs)
      dev::mbar_init(free_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      dev::mbar_init(tfull_bar(b), 1);
      dev::mbar_init(tempty_bar(b), 2 * (NEPI / 32));
    }
    dev::mbar_init(drain_bar, 1);
    s_misc[1] = 0;
    dev::fence_mbar_init_cluster();
  }
  if (warp == 0 && lane == 0) dev::prefetch_tmap(&tm_a);
  if (warp == 2 && lane == 0) dev::prefetch_tmap(&tm_b);
  if (warp == 1) {
    dev::tmem_alloc_pair(dev::smem_u32(&s_misc[0]), 2 * TN);
    dev::tmem_relinquish_pair();
  }
  dev::tc_fence_before();
  dev::cluster_sync();   // barrier inits of both CTAs visible before any remote arrive
  dev::tc_fence_after();
  const uint32_t tmem = s_misc[0];
  Tiles it(tp, unit, TN / CH);
  int m, c0, nch;

  if (warp == 0 || warp == 2) {
    // ---------------- producers: warp 0 the tokens, warp 2 the weights ----------------
    if (lane == 0) {
      const bool tok = warp == 0;
      uint32_t j = 0;
      bool ok = true;
      while (ok && it.next(m, c0, nch)) {
        const int rows = nch * CH / 2;                      // this CTA's weight rows
        const int boxes = tok ? 1 : (rows + BBOX - 1) / BBOX;
        const uint32_t bytes = tok ? 2u * AB : 2u * boxes * BBOX * 128u;   // of both CTAs
        const int row0 = tok ? (2 * m + (int)rank) * TM : c0 * CH + (int)rank * rows;
        for (int kb = 0; kb < nkb; ++kb, ++j) {
          const int s = j % SK;
          if (!dev::mbar_wait(free_bar(s), ((j / SK) & 1u) ^ 1u, p.err, kSiteGemmEmpty,
                              p.limit_ns) || *s_abort) {
            give_up();
            ok = false;
            break;
          }
          if (rank == 0) dev::mbar_arrive_expect_tx(full_bar(s), bytes);
          if (tok)
            dev::tma_load_2d_pair(dev::smem_u32(smem + s * AB), &tm_a, kb * 128, row0,
                                  lead(full_bar(s)));
          else
            for (int i = 0; i < boxes; ++i)
              dev::tma_load_2d_pair(dev::smem_u32(smem + OFF_B + s * BB + i * BBOX * 128), &tm_b,
                                    kb * 128, row0 + i * BBOX, lead(full_bar(s)));
        }
      }
      // Every stage this thread filled has been read by its MMAs before the CTA ends (their
      // arrivals on the free barriers, too, have landed); after an abort the bytes in flight
      // cannot be told apart, so the leader waits for the stages' own completion.
      for (uint32_t i = (j >= (uint32_t)SK ? j - SK : 0); i < j; ++i) {
        if (ok)
          dev::mbar_wait(free_bar(i % SK), (i / SK) & 1u, p.err, kSiteGemmDrain, p.limit_ns);
        else if (rank == 0)
          dev::mbar_wait(full_bar(i % SK), (i / SK) & 1u, p.err, kSiteGemmDrain, p.limit_ns);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (the leader's lane 0) ----------------
    if (lane == 0 && rank == 0) {
      uint32_t j = 0, n = 0;
      bool ok = true, issued = false;
      for (; ok && it.next(m, c0, nch); ++n) {
        const uint32_t idesc = dev::idesc_i8(2 * TM, nch * CH);
        const int b = n & 1;
        if (!dev::mbar_wait(tempty_bar(b), ((n >> 1) & 1u) ^ 1u, p.err, kSiteGemmAccum,
                            p.limit_ns) || *s_abort) {
          give_up();
          ok = false;
          break;
        }
        dev::tc_fence_after();
        const uint32_t dt = tmem + (uint32_t)(b * TN);
        for (int kb = 0; kb < nkb; ++kb, ++j) {
          const int s = j % SK;
          if (!dev::mbar_wait(full_bar(s), (j / SK) & 1u, p.err, kSiteGemmFull, p.limit_ns)) {
            give_up();
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t sa = dev::smem_u32(smem + s * AB), sb = dev::smem_u32(smem + OFF_B + s * BB);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            dev::mma_i8_pair(dt, dev::sdesc_sw128(sa + kk * 32), dev::sdesc_sw128(sb + kk * 32),
                             idesc, (kb | kk) != 0);
          issued = true;
          dev::mma_commit_pair(free_bar(s));
        }
        if (!ok) break;
        dev::mma_commit_pair(tfull_bar(b));
      }
      if (!ok && issued) {   // wait for the MMAs in flight before TMEM is freed
        dev::mma_commit_pair(drain_bar);
        dev::mbar_wait(drain_bar, 0, p.err, kSiteGemmDrain, p.limit_ns);
      }
    }
  } else if (warp >= 4) {
    // ---------------- epilogue: a lane holds a token ----------------
    const int etid = tid - 128, q = warp & 3, half = (warp - 4) >> 2;
    uint8_t* stg = smem + OFF_STG + (warp - 4) * STG;
    uint32_t n = 0;
    bool ok = true;
    for (; ok && it.next(m, c0, nch); ++n) {
      const int b = n & 1, ncols = nch * CH, o0 = c0 * CH;
      const int tw = (2 * m + (int)rank) * TM + q * 32, t = tw + lane;   // tokens of the warp
      float* col = s_col + b * 3 * TN;
      for (int i = etid; i < ncols; i += NEPI) {
        const int o = o0 + i;
        const bool in = o < p.N;
        col[i] = in ? p.w_scale[o] : 0.f;
        col[TN + i] = in && p.mean ? p.w_rowsum[o] : 0.f;
        col[2 * TN + i] = in && p.bias ? __bfloat162float(p.bias[o]) : 0.f;
      }
      const float alpha = t < p.T ? p.a_scale[t] : 0.f;
      const float mean = t < p.T && p.mean ? p.mean[t] : 0.f;
      // one thread waits and decides for all, so that every warp meets the same barriers; the
      // constants and the decision have two slots, so that the writes for the next tile cannot
      // meet a reader of this one
      if (etid == 0) {
        const bool ready = dev::mbar_wait(tfull_bar(b), (n >> 1) & 1u, p.err, kSiteGemmAccum,
                                          p.limit_ns) && !*s_abort;
        if (!ready) give_up();
        s_misc[2 + b] = ready ? 1u : 0u;
      }
      dev::named_bar(1, NEPI);
      ok = *reinterpret_cast<volatile uint32_t*>(&s_misc[2 + b]) != 0;
      dev::tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * TN);
#pragma unroll 1
      for (int c = half; ok && c < nch; c += 2) {
        uint32_t r[32];
        dev::tmem_ld32(acc + (uint32_t)(c * 32), r);
        dev::tmem_wait_ld();
        const int o = o0 + c * 32;
        if (tw >= p.T || o >= p.N) continue;
        // 64-byte rows of the staging tile: 16-byte chunk i of row l at i ^ ((l >> 1) & 3)
        auto put = [&](int piece, const uint32_t (&v)[4]) {
          *reinterpret_cast<uint4*>(stg + lane * 64 + ((piece ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(v[0], v[1], v[2], v[3]);
        };
        auto begin = [&]() {   // the store before has read its values
          if (lane == 0) dev::bulk_wait_all_read();
          __syncwarp();
        };
        auto send = [&](const CUtensorMap* map, int x) {
          dev::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            dev::tma_store_2d(map, dev::smem_u32(stg), x, tw);
            dev::bulk_commit();
          }
        };
        if (p.out_acc) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            begin();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              put(i, {r[h * 16 + 4 * i], r[h * 16 + 4 * i + 1], r[h * 16 + 4 * i + 2],
                      r[h * 16 + 4 * i + 3]});
            send(&tm_y, o + h * 16);
          }
          continue;
        }
        const float2* cs = reinterpret_cast<const float2*>(col + c * 32);
        float2 y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          y[i] = dequant2((int)r[2 * i], (int)r[2 * i + 1], alpha, mean, cs[i], cs[TN / 2 + i],
                          cs[TN + i]);
        auto pack = [&](int i) {
          const __nv_bfloat162 v = __float22bfloat162_rn(y[i]);
          return *reinterpret_cast<const uint32_t*>(&v);
        };
        if (o >= p.n_head) {
          begin();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            put(i, {pack(4 * i), pack(4 * i + 1), pack(4 * i + 2), pack(4 * i + 3)});
          send(&tm_y, o);
        } else {
          // float32 columns, 16 to a store; n_head % 16 == 0, so each half is one kind
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int oh = o + h * 16;
            if (oh < p.n_head) {
              begin();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                put(i, {__float_as_uint(y[h * 8 + 2 * i].x), __float_as_uint(y[h * 8 + 2 * i].y),
                        __float_as_uint(y[h * 8 + 2 * i + 1].x),
                        __float_as_uint(y[h * 8 + 2 * i + 1].y)});
              send(&tm_h, oh);
            } else if (t < p.T && oh < p.N) {
              uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) +
                                                    (int64_t)t * p.N + oh);
              dst[0] = make_uint4(pack(h * 8), pack(h * 8 + 1), pack(h * 8 + 2), pack(h * 8 + 3));
              dst[1] = make_uint4(pack(h * 8 + 4), pack(h * 8 + 5), pack(h * 8 + 6),
                                  pack(h * 8 + 7));
            }
          }
        }
      }
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive_cluster(lead(tempty_bar(b)));
    }
    if (lane == 0) dev::bulk_wait_all();
  }

  __syncwarp();
  dev::tc_fence_before();
  dev::cluster_sync();   // no MMA, remote arrive or TMEM access of either CTA is still pending
  if (warp == 1) {
    dev::tc_fence_after();
    dev::tmem_dealloc_pair(tmem, 2 * TN);
  }
}

// Ranges of the flattened (token block, chunk) space: the largest cost over the pairs, chunks plus
// kTileCost for every tile of at most maxch chunks inside one token block, is made as small as
// possible: bisection on the bound, each pair taking as much as the bound allows. kTileCost = 8
// chunks: a tile reads its token rows whatever its width, as many bytes as 8 chunks of weights.
// Kept per shape; a space of very many chunks is cut evenly (its tail is short beside it).
constexpr int kTileCost = 8;

bool make_schedule(int64_t blocks, int npm, int units, int maxch, int* out) {
  const int64_t total = blocks * npm;
  if (total > 0x7FFFFFFF) return false;
  if (total > (1 << 18)) {
    for (int u = 0; u <= units; ++u) out[u] = (int)(total * u / units);
    return true;
  }
  static std::mutex mu;
  static std::map<std::tuple<int, int, int, int>, std::vector<int>> kept;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple((int)blocks, npm, units, maxch);
  auto found = kept.find(key);
  if (found == kept.end()) {
    std::vector<int> v((size_t)units + 1);
    auto fits = [&](int64_t bound) {
      int64_t pos = 0;
      for (int u = 0; u < units; ++u) {
        v[(size_t)u] = (int)pos;
        int64_t left = bound;
        while (pos < total) {
          // whole tiles of the rest of this token block, then a part of one
          const int64_t run = std::min<int64_t>(npm - pos % npm, maxch);
          const int64_t take = std::min<int64_t>(run, left - kTileCost);
          if (take < 1) break;
          pos += take;
          left -= take + kTileCost;
          if (take < run) break;
        }
      }
      v[(size_t)units] = (int)total;
      return pos >= total;
    };
    int64_t lo = 1 + kTileCost, hi = total * (1 + kTileCost);
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (fits(mid)) hi = mid; else lo = mid + 1;
    }
    fits(lo);
    found = kept.emplace(key, std::move(v)).first;
  }
  std::copy(found->second.begin(), found->second.end(), out);
  return true;
}

// CTA pairs that are resident at once, per kernel and device (0 if the query fails).
int resident_pairs(const void* kern, int smem, int threads) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, int> kept;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  auto found = kept.find({kern, dev});
  if (found != kept.end()) return found->second;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2u * (unsigned)std::max(sms, 1));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  kept[{kern, dev}] = n;
  return n;
}

oq_status run_tiles(const W8Params& w, cudaStream_t s) {
  CUtensorMap ta, tb, ty, th;
  std::memset(&th, 0, sizeof(th));
  const uint64_t K = (uint64_t)w.K, N = (uint64_t)w.N, T = (uint64_t)w.T;
  bool ok = tma_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.a, K, T, K, 128, TM,
                       CU_TENSOR_MAP_SWIZZLE_128B) &&
            tma_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.w, K, N, K, 128, BBOX,
                       CU_TENSOR_MAP_SWIZZLE_128B);
  if (w.out_acc)
    ok = ok && tma_map_2d(&ty, CU_TENSOR_MAP_DATA_TYPE_INT32, w.out, N, T, N * 4, 16, 32,
                          CU_TENSOR_MAP_SWIZZLE_64B);
  else
    ok = ok && tma_map_2d(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.out, N, T, N * 2, 32, 32,
                          CU_TENSOR_MAP_SWIZZLE_64B);
  if (w.n_head)
    ok = ok && tma_map_2d(&th, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, w.head, (uint64_t)w.n_head, T,
                          (uint64_t)w.n_head * 4, 16, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (!ok) return fail(OQ_ERR_CUDA, "cuTensorMapEncodeTiled failed or unavailable");
  const auto kern = &k_gemm_w8;
  cudaError_t e = allow_max_dynamic_smem(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(gemm_w8)");
  int units = resident_pairs(reinterpret_cast<const void*>(kern), SMEM, NTHR);
  if (units <= 0) return fail(OQ_ERR_UNSUPPORTED, "gemm_w8: no CTA pair fits on this device");
  TileParams p;
  p.w = w;
  p.npm = (w.N + CH - 1) / CH;
  const int64_t blocks = ((int64_t)w.T + 2 * TM - 1) / (2 * TM);
  units = (int)std::min<int64_t>(std::min(units, kMaxUnits), blocks * p.npm);
  if (!make_schedule(blocks, p.npm, units, TN / CH, p.sched))
    return fail(OQ_ERR_INVALID_ARG, "gemm_w8: T x d_out too large for one call");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2u * (unsigned)units);
  cfg.blockDim = dim3(NTHR);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, ta, tb, ty, th, p);
  return e == cudaSuccess ? OQ_OK : cuda_fail(e, "launch gemm_w8");
}

}  // namespace

oq_status launch_gemm_w8(const GemmW8Args& g, cudaStream_t s) {
  if (g.T == 0) return OQ_OK;
  W8Params p{};
  p.a = g.a; p.w = g.w; p.a_scale = g.a_scale; p.mean = g.mean; p.w_scale = g.w_scale;
  p.w_rowsum = g.w_rowsum; p.bias = reinterpret_cast<const __nv_bfloat16*>(g.bias);
  p.T = (int)g.T; p.K = (int)g.K; p.N = (int)g.N; p.out_acc = g.out_acc;
  p.n_head = (int)g.n_head; p.out = g.out; p.head = g.head;
  p.err = device_error_word();
  if (!p.err) return fail(OQ_ERR_CUDA, "device error word unavailable");
  p.limit_ns = kWaitLimitNs;
  return run_tiles(p, s);
}

}  // namespace oq
