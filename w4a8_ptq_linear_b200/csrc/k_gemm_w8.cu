// W8A8 GEMM: int8 activations against int8 weights, exact int32 sums, the dequant epilogue of
// the INT4 GEMMs.
//
//     acc[t, o] = sum_k a[t, k] w[o, k]
//     y[t, o]   = bf16( alpha_t s_o acc + (mean_t w1_o + b_o) )
//
// Every shape of the kernel takes the same float steps (fma(acc, alpha s, fma(mean, w1, b))), so a
// token's result does not depend on how many tokens it comes with. That ends where heads are formed
// behind the product: each shape adds a head's squares in the order in which it holds them, so a normed
// head's last bits may depend on the shape, and so on the number of tokens.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <new>
#include <tuple>

#include "kept.h"
#include "oq_internal.h"
#include "ptx.cuh"
#include "split_shape.h"

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
  bool wide;                // out is 32-byte aligned (its rows are: N % 16 == 0)
  void* out;
  float* head;
  bool dependent;           // launched beside the kernel that writes a, a_scale and mean
  unsigned long long* err;
  unsigned long long limit_ns;
};

// The launch before (whose results a, a_scale and mean may be) has ended and its writes are visible;
// at once where the launch is an ordinary one.
__device__ __forceinline__ void dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// A launch that waits for this grid may begin beside it.
__device__ __forceinline__ void dependents_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A walk over the stages of a ring. One thread issues a role's steps, so its own instructions are on
// the critical path: without a division for the stage and the phase of each step the few-token product
// took 8.3 us instead of 8.8 (16 x 4096 x 4096).
struct Ring {
  int st = 0;
  uint32_t phase = 0;
  bool alone = false;   // the launch before has ended
  __device__ __forceinline__ void next(int n) {
    if (++st == n) {
      st = 0;
      phase ^= 1u;
    }
  }
};

// Wait for a stage's barrier; false (and the CTA's abort flag set) when the wait gave up or another
// role has. The flag is looked at only where the stage was not ready, and the limit starts only when
// the launch before has ended, for whose tokens the stage may be waiting.
__device__ __forceinline__ bool ring_wait(Ring& rg, uint32_t bar, uint32_t parity,
                                          volatile uint32_t* abort, const W8Params& p,
                                          uint32_t site) {
  if (dev::mbar_try_wait(bar, parity)) return true;
  if (!rg.alone) {
    dependency_wait();
    rg.alone = true;
  }
  if (*abort == 0u && dev::mbar_wait(bar, parity, p.err, site, p.limit_ns)) return true;
  *abort = 1u;
  return false;
}

// ---- tiles on CTA pairs ----------------------------------------------------------------------
// D[t, o] on tcgen05 (kind::i8, cta_group::2): 256 tokens are the M rows, up to 256 channels the
// N columns, so that a thread of the epilogue holds one token's row of the accumulator: its scale
// and mean are two registers, the channels' constants are broadcast from shared memory, and
// sums over a row stay in the thread.
//
// One persistent CTA pair per two SMs. Both operands come by TMA, K-major, 128 bytes of K to a
// block; two producer threads, one to an operand. TMEM holds two accumulators of 256 columns, so a
// tile's epilogue runs under the next tile's MMAs; it writes 32-byte sectors from registers.
//
// What bounds it is L2 and shared memory together. A full tile brings 64 KB per 128 bytes of K
// through L2, writes them to shared memory and reads them again for the MMAs: at the tensor pipe's
// full rate 64 bytes a clock and SM from L2 and all 128 of shared memory. Measured at 4096 x 4096 x
// 12288, parts left out in a copy of the kernel: MMAs alone 102 us (4.05 POPS), loads alone 127,
// both 132, with the epilogue's arithmetic 139, whole 140 to 142 us (2.9 POPS, 68 % of the kind::i8 peak
// loop of 4.3; a library product of the same operands to int32 takes 137 to 141). Under the power cap of
// a long run 160 to 170 us (the library 158). Hence stages of two K blocks (one commit for eight
// MMAs; of one block 167 us where two took 155), no staging of the output in shared memory, constants
// read from it only where they count.
//
// Schedule: tiles in waves, one to a pair, down the token blocks of a group first, so that the
// tiles in flight share their weights and the group's activations stay in L2 (contiguous ranges of
// tiles for each pair kept all weights live at once: 154 us where waves took 146). What does not
// fill a wave is cut into narrower tiles, one to a pair.
constexpr int TM = 128;                    // tokens per CTA
constexpr int TN = 256;                    // channels per tile at most
constexpr int CH = 64;                     // channels per chunk, where no heads are formed
constexpr int KS = 2;                      // 128-byte K blocks per stage
constexpr int SK = 3;                      // stages
constexpr int AK = TM * 128;               // activation bytes of a K block
constexpr int BK = (TN / 2) * 128;         // weight bytes of a K block (this CTA's half)
constexpr int AB = KS * AK, BB = KS * BK;  // of a stage
constexpr int BBOX = 64;                   // weight rows of one TMA load
constexpr int NEPI = 256;                  // epilogue threads, two warps to a TMEM lane quarter
constexpr int NTHR = 128 + NEPI;
constexpr int OFF_B = SK * AB;
constexpr int OFF_COL = OFF_B + SK * BB;   // [2][3][TN] floats
constexpr int OFF_HEAD = OFF_COL + 2 * 3 * TN * 4;   // [4][TN] floats: q, k weights, q, k biases
constexpr int OFF_BAR = OFF_HEAD + 4 * TN * 4;
constexpr int NBAR = 2 * SK + 5;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int SMEM = OFF_MISC + 16 + 1024;
static_assert(SMEM <= 232448, "shared memory");

// Heads formed in an epilogue (columns o < w.n_head): the parameters of HeadArgs
struct TileHeads {
  int D, nq, norm, rope, rot;              // nq: query columns
  float eps, inv_d;
  const float *qw, *qb, *kw, *kb, *cos, *sin;
  int64_t n_pos, pos_bs;
  int seq;
  const int32_t* positions;
};

struct TileParams {
  W8Params w;
  TileHeads h;
  int cw, maxch;                           // channels of a chunk, chunks of a tile at most
  int npm;                                 // chunks of a token block
  int blocks, ncol, gm;                    // token blocks, tiles of a block, blocks of a group
  int total, full;                         // tiles; those run whole
  int split;                               // parts that each of the others is cut into
};

// The tiles of one pair, the same sequence in every role: pair u takes tiles u, u + units, ...
// whole, as long as there is one for every pair, then at most one part of a remaining tile.
struct Tiles {
  const TileParams& p;
  int idx, units;
  __device__ Tiles(const TileParams& p_, int unit, int units_) : p(p_), idx(unit), units(units_) {}
  // token block m, first chunk c0, number of chunks n
  __device__ bool next(int& m, int& c0, int& n) {
    int tile = idx, part = 0;
    const bool whole = idx < p.full;
    if (!whole) {
      tile = p.full + (idx - p.full) / p.split;
      part = (idx - p.full) % p.split;
    }
    if (tile >= p.total) return false;
    idx += units;
    const int g = tile / (p.gm * p.ncol), r = tile - g * p.gm * p.ncol;
    const int rows = min(p.gm, p.blocks - g * p.gm);
    const int col = r / rows;
    m = g * p.gm + r - col * rows;
    c0 = (int)((int64_t)col * p.npm / p.ncol);
    n = (int)((int64_t)(col + 1) * p.npm / p.ncol) - c0;
    if (!whole) {
      const int a = part * n / p.split, b = (part + 1) * n / p.split;
      c0 += a;
      n = b - a;
    }
    return n > 0;
  }
};

// 32 bytes from registers; `wide`: the address is a multiple of 32
__device__ __forceinline__ void store32(void* dst, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    uint4* d = reinterpret_cast<uint4*>(dst);
    d[0] = make_uint4(v[0], v[1], v[2], v[3]);
    d[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ uint32_t pack2(float2 y) {
  const __nv_bfloat162 v = __float22bfloat162_rn(y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// y of a token's NF neighbouring channels: c = fma(mean, w1, b), y = fma(acc, alpha s, c). The
// channels' constants lie at col (scales), col + TN (row sums) and col + 2 TN (biases), the last
// two read only where they count: shared memory is what the mainloop is short of.
template <int NF>
__device__ __forceinline__ void dequant(const uint32_t (&r)[NF], float alpha, float mean,
                                        const float* col, bool has_mean, bool has_bias,
                                        float2 (&y)[NF / 2]) {
  const float4* cs = reinterpret_cast<const float4*>(col);
  const float2 al = make_float2(alpha, alpha), mn = make_float2(mean, mean);
#pragma unroll
  for (int i = 0; i < NF / 4; ++i) {
    float4 w4 = make_float4(0.f, 0.f, 0.f, 0.f), b4 = w4;
    const float4 s4 = cs[i];
    if (has_mean) w4 = cs[TN / 4 + i];
    if (has_bias) b4 = cs[TN / 2 + i];
    const float2 c0 = __ffma2_rn(mn, make_float2(w4.x, w4.y), make_float2(b4.x, b4.y));
    const float2 c1 = __ffma2_rn(mn, make_float2(w4.z, w4.w), make_float2(b4.z, b4.w));
    y[2 * i] = __ffma2_rn(make_float2((float)(int)r[4 * i], (float)(int)r[4 * i + 1]),
                          __fmul2_rn(al, make_float2(s4.x, s4.y)), c0);
    y[2 * i + 1] = __ffma2_rn(make_float2((float)(int)r[4 * i + 2], (float)(int)r[4 * i + 3]),
                              __fmul2_rn(al, make_float2(s4.z, s4.w)), c1);
  }
}

// The bf16 results of 16 channels
__device__ __forceinline__ void store_bf16x16(const W8Params& p, int t, int o, const float2* y) {
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = pack2(y[i]);
  store32(reinterpret_cast<__nv_bfloat16*>(p.out) + (int64_t)t * p.N + o, v, p.wide);
}

// One query or key head of the warp's 32 tokens, a token to a lane, from its D accumulator columns
// at `acc`: norm, weight, bias, rotation. The sums of the norm need no exchange. The first pass puts
// the float32 values back in TMEM in the sums' place, and the later ones (squares about the mean,
// result) read them from there: shared memory, which the channels' constants come from, is what
// the mainloop is short of. D and rot are multiples of 32. The angles of the next 16 pairs are on
// their way while 16 are turned.
__device__ __forceinline__ void head_epilogue(const TileParams& tp, uint32_t acc, const float* col,
                                              const float* s_head, int t, int o, float alpha,
                                              float mean, int64_t pos) {
  const W8Params& p = tp.w;
  const TileHeads& h = tp.h;
  const bool row = t < p.T;
  const bool is_q = o < h.nq;
  const float* wt = s_head + (is_q ? 0 : TN);
  const float* bs = s_head + (is_q ? 2 * TN : 3 * TN);
  const bool has_wt = (is_q ? h.qw : h.kw) != nullptr, has_bs = (is_q ? h.qb : h.kb) != nullptr;
  const int half = h.rot / 2;
  const bool turn = row && pos >= 0, lost = pos >= h.n_pos;
  float4 cs[4], sn[4];
  auto angles = [&](int i) {   // of pairs i .. i + 15
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (turn && !lost && i < half) {
        cs[j] = __ldg(reinterpret_cast<const float4*>(h.cos + pos * half + i) + j);
        sn[j] = __ldg(reinterpret_cast<const float4*>(h.sin + pos * half + i) + j);
      } else {
        const float n = __int_as_float(0x7fc00000);   // a position past the table, or unused
        cs[j] = sn[j] = make_float4(n, n, n, n);
      }
    }
  };
  angles(0);

  float2 sum = make_float2(0.f, 0.f), sq = sum;
  const bool layer = h.norm == OQ_NORM_LAYER;
  uint32_t v[32];
  float2 y[16];
  auto floats = [](const uint32_t (&q)[32], int i) {   // columns 2 i, 2 i + 1
    return make_float2(__uint_as_float(q[2 * i]), __uint_as_float(q[2 * i + 1]));
  };
#pragma unroll 1
  for (int c = 0; c < h.D; c += 32) {
    __syncwarp();
    dev::tmem_ld32(acc + (uint32_t)c, v);
    dev::tmem_wait_ld();
    dequant<32>(v, alpha, mean, col + c, p.mean != nullptr, p.bias != nullptr, y);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      sum = __fadd2_rn(sum, y[i]);
      sq = __ffma2_rn(y[i], y[i], sq);
      v[2 * i] = __float_as_uint(y[i].x);
      v[2 * i + 1] = __float_as_uint(y[i].y);
    }
    dev::tmem_st32(acc + (uint32_t)c, v);
  }
  dev::tmem_wait_st();
  const float m = layer ? (sum.x + sum.y) * h.inv_d : 0.f;
  const float2 neg = make_float2(-m, -m);
  if (layer) {
    sq = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int c = 0; c < h.D; c += 32) {
      dev::tmem_ld32(acc + (uint32_t)c, v);
      dev::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 d = __fadd2_rn(floats(v, i), neg);
        sq = __ffma2_rn(d, d, sq);
      }
    }
  }
  const float r = h.norm == OQ_NORM_NONE ? 1.f : rsqrtf(fmaf(sq.x + sq.y, h.inv_d, h.eps));
  const float2 r2 = make_float2(r, r);
  // n pairs of columns x from column c on: norm, weight, bias
  auto normed = [&](float2* x, int n, int c) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      if (i >= n) break;
      float4 w4 = make_float4(1.f, 1.f, 1.f, 1.f), b4 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (has_wt) w4 = *reinterpret_cast<const float4*>(wt + c + 2 * i);
      if (has_bs) b4 = *reinterpret_cast<const float4*>(bs + c + 2 * i);
      x[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(x[i], neg), r2), make_float2(w4.x, w4.y),
                        make_float2(b4.x, b4.y));
      x[i + 1] = __ffma2_rn(__fmul2_rn(__fadd2_rn(x[i + 1], neg), r2), make_float2(w4.z, w4.w),
                            make_float2(b4.z, b4.w));
    }
  };
  if (h.rope == OQ_ROPE_HALVES) {
#pragma unroll 1
    for (int i = 0; i < half; i += 16) {
      __syncwarp();   // the lanes' ways part below; TMEM is read by the whole warp
      uint32_t a[16], d[16];
      dev::tmem_ld16(acc + (uint32_t)i, a);
      dev::tmem_ld16(acc + (uint32_t)(i + half), d);
      dev::tmem_wait_ld();
      float2 u[8], w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = make_float2(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]));
        w[j] = make_float2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]));
      }
      normed(u, 8, i);
      normed(w, 8, i + half);
      if (turn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 c4 = cs[j / 2], s4 = sn[j / 2];
          const float2 c2 = j & 1 ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
          const float2 s2 = j & 1 ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
          const float2 ru = __ffma2_rn(u[j], c2, __fmul2_rn(make_float2(-w[j].x, -w[j].y), s2));
          w[j] = __ffma2_rn(w[j], c2, __fmul2_rn(u[j], s2));
          u[j] = ru;
        }
      }
      angles(i + 16);
      if (row) {
        store_bf16x16(p, t, o + i, u);
        store_bf16x16(p, t, o + i + half, w);
      }
    }
  } else {
#pragma unroll 1
    for (int c = 0; c < h.rot; c += 32) {
      __syncwarp();
      dev::tmem_ld32(acc + (uint32_t)c, v);
      dev::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] = floats(v, j);
      normed(y, 16, c);
      if (turn) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 n = y[j];
          const float4 c4 = cs[j / 4], s4 = sn[j / 4];
          const float cc = j % 4 == 0 ? c4.x : j % 4 == 1 ? c4.y : j % 4 == 2 ? c4.z : c4.w;
          const float ss = j % 4 == 0 ? s4.x : j % 4 == 1 ? s4.y : j % 4 == 2 ? s4.z : s4.w;
          y[j] = make_float2(n.x * cc - n.y * ss, n.x * ss + n.y * cc);
        }
      }
      angles((c + 32) / 2);
      if (row) {
        store_bf16x16(p, t, o + c, y);
        store_bf16x16(p, t, o + c + 16, y + 8);
      }
    }
  }
#pragma unroll 1
  for (int c = h.rot; c < h.D; c += 32) {   // elements that no rotation reaches
    __syncwarp();
    dev::tmem_ld32(acc + (uint32_t)c, v);
    dev::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] = floats(v, j);
    normed(y, 16, c);
    if (row) {
      store_bf16x16(p, t, o + c, y);
      store_bf16x16(p, t, o + c + 16, y + 8);
    }
  }
}

// HEADS: query and key heads are formed in the epilogue (tp.h); tiles then hold whole heads.
template <bool HEADS>
__global__ void __launch_bounds__(NTHR, 1)
    k_gemm_w8(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ TileParams tp) {
  const W8Params& p = tp.w;
  dependents_begin();
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
  const int nst = (nkb + KS - 1) / KS;   // stages of a tile
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
  if constexpr (HEADS) {
    float* s_head = reinterpret_cast<float*>(smem + OFF_HEAD);
    for (int i = tid; i < tp.h.D; i += NTHR) {
      s_head[i] = tp.h.qw ? tp.h.qw[i] : 1.f;
      s_head[TN + i] = tp.h.kw ? tp.h.kw[i] : 1.f;
      s_head[2 * TN + i] = tp.h.qb ? tp.h.qb[i] : 0.f;
      s_head[3 * TN + i] = tp.h.kb ? tp.h.kb[i] : 0.f;
    }
  }
  __syncwarp();   // the lanes' ways parted above; what follows is for whole warps
  if (warp == 1) {
    dev::tmem_alloc_pair(dev::smem_u32(&s_misc[0]), 2 * TN);
    dev::tmem_relinquish_pair();
  }
  dev::tc_fence_before();
  dev::cluster_sync();   // barrier inits of both CTAs visible before any remote arrive
  dev::tc_fence_after();
  const uint32_t tmem = s_misc[0];
  const int cw = HEADS ? tp.cw : CH;   // channels of a chunk
  Tiles it(tp, unit, (int)gridDim.x / 2);
  int m, c0, nch;

  if (warp == 0 || warp == 2) {
    // ---------------- producers: warp 0 the tokens, warp 2 the weights ----------------
    if (warp == 0) dependency_wait();   // the weights do not come from the launch before
    if (lane == 0) {
      const bool tok = warp == 0;
      uint32_t j = 0;
      Ring rg;
      bool ok = true;
      while (ok && it.next(m, c0, nch)) {
        const int rows = nch * cw / 2;                      // this CTA's weight rows
        const int boxes = tok ? 1 : (rows + BBOX - 1) / BBOX;
        const uint32_t block_bytes = tok ? 2u * AK : 2u * boxes * BBOX * 128u;   // of both CTAs
        const int row0 = tok ? (2 * m + (int)rank) * TM : c0 * cw + (int)rank * rows;
        for (int st = 0; st < nst; ++st, ++j, rg.next(SK)) {
          const int s = rg.st, nk = min(KS, nkb - st * KS);
          if (!ring_wait(rg, free_bar(s), rg.phase ^ 1u, s_abort, p, kSiteGemmEmpty)) {
            ok = false;
            break;
          }
          if (rank == 0) dev::mbar_arrive_expect_tx(full_bar(s), (uint32_t)nk * block_bytes);
          for (int u = 0; u < nk; ++u) {
            const int k = (st * KS + u) * 128;
            if (tok)
              dev::tma_load_2d_pair(dev::smem_u32(smem + s * AB + u * AK), &tm_a, k, row0,
                                    lead(full_bar(s)));
            else
              for (int i = 0; i < boxes; ++i)
                dev::tma_load_2d_pair(dev::smem_u32(smem + OFF_B + s * BB + u * BK + i * BBOX * 128),
                                      &tm_b, k, row0 + i * BBOX, lead(full_bar(s)));
          }
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
      const uint64_t da = dev::sdesc_sw128(dev::smem_u32(smem));
      const uint64_t db = dev::sdesc_sw128(dev::smem_u32(smem) + OFF_B);
      uint32_t n = 0;
      Ring rg;
      bool ok = true, issued = false;
      for (; ok && it.next(m, c0, nch); ++n) {
        const uint32_t idesc = dev::idesc_i8(2 * TM, nch * cw);
        const int b = n & 1;
        if (!ring_wait(rg, tempty_bar(b), ((n >> 1) & 1u) ^ 1u, s_abort, p, kSiteGemmAccum)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        const uint32_t dt = tmem + (uint32_t)(b * TN);
        for (int st = 0; st < nst; ++st, rg.next(SK)) {
          const int s = rg.st, nk = min(KS, nkb - st * KS);
          if (!ring_wait(rg, full_bar(s), rg.phase, s_abort, p, kSiteGemmFull)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint64_t sa = da + (uint64_t)(s * AB >> 4), sb = db + (uint64_t)(s * BB >> 4);
#pragma unroll
          for (int u = 0; u < KS; ++u) {
            if (u >= nk) break;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              dev::mma_i8_pair(dt, sa + (u * AK >> 4) + 2 * kk, sb + (u * BK >> 4) + 2 * kk, idesc,
                               (st | u | kk) != 0);
          }
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
    dependency_wait();   // scales, means, and the output's earlier readers
    const int etid = tid - 128, q = warp & 3, half = (warp - 4) >> 2;
    uint32_t n = 0;
    bool ok = true;
    for (; ok && it.next(m, c0, nch); ++n) {
      const int b = n & 1, ncols = nch * cw, o0 = c0 * cw;
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
      __syncwarp();
      dev::named_bar(1, NEPI);
      ok = *reinterpret_cast<volatile uint32_t*>(&s_misc[2 + b]) != 0;
      dev::tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * TN);
      // Heads: a chunk is a head or, behind them, as many plain columns; the two warps of a lane
      // quarter take chunks in turn. Else they take 32 columns in turn.
      int first = half, step = 2, last = ncols / 32, pieces = 0;
      int64_t pos = -1;
      if constexpr (HEADS) {
        first = 0, last = 0;
        if (t < p.T) {
          const int bt = t / tp.h.seq, st = t - bt * tp.h.seq;
          pos = tp.h.positions ? (int64_t)tp.h.positions[bt * tp.h.pos_bs + st] : st;
        }
        pieces = nch;
      }
#pragma unroll 1
      for (int ch = half; HEADS ? ok && ch < pieces : ch == half; ch += 2) {
        if constexpr (HEADS) {
          if (tw >= p.T || o0 + ch * cw >= p.N) continue;   // warp-uniform
          if (o0 + ch * cw < p.n_head) {
            head_epilogue(tp, acc + (uint32_t)(ch * cw), col + ch * cw,
                          reinterpret_cast<const float*>(smem + OFF_HEAD), t, o0 + ch * cw, alpha,
                          mean, pos);
            continue;
          }
          first = ch * cw / 32, step = 1, last = (ch + 1) * cw / 32;
        }
#pragma unroll 1
        for (int c = first; ok && c < last; c += step) {
          uint32_t r[32];
          __syncwarp();   // lanes of missing tokens have gone ahead; TMEM is read by the whole warp
          dev::tmem_ld32(acc + (uint32_t)(c * 32), r);
          dev::tmem_wait_ld();
          const int o = o0 + c * 32;
          if (t >= p.T || o >= p.N) continue;
          const bool two = o + 16 < p.N;        // N % 16 == 0: sixteen or all of the channels
          if (!HEADS && p.out_acc) {
            int32_t* dst = reinterpret_cast<int32_t*>(p.out) + (int64_t)t * p.N + o;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < 2 || two) store32(dst + 8 * i, r + 8 * i, p.wide);
            continue;
          }
          float2 y[16];
          dequant<32>(r, alpha, mean, col + c * 32, p.mean != nullptr, p.bias != nullptr, y);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int oh = o + h * 16;
            if (h && !two) break;
            if (!HEADS && oh < p.n_head) {   // n_head % 16 == 0
              float* dst = p.head + (int64_t)t * p.n_head + oh;
              store32(dst, reinterpret_cast<const uint32_t*>(y + h * 8), true);
              store32(dst + 8, reinterpret_cast<const uint32_t*>(y + h * 8 + 4), true);
            } else {
              store_bf16x16(p, t, oh, y + h * 8);
            }
          }
        }
      }
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive_cluster(lead(tempty_bar(b)));
    }
  }

  __syncwarp();
  dev::tc_fence_before();
  dev::cluster_sync();   // no MMA, remote arrive or TMEM access of either CTA is still pending
  if (warp == 1) {
    dev::tc_fence_after();
    dev::tmem_dealloc_pair(tmem, 2 * TN);
  }
}

// Clusters that are resident at once, per device and launch shape (-1 if the query fails).
int resident_clusters(const void* kern, int cluster, int smem, int threads) {
  static Kept<std::tuple<int, const void*, int, int>, int> kept;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  const bool known = kept.get(std::make_tuple(dev, kern, cluster, smem), &n, [&](int* clusters) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(cluster * device_sms()));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(clusters, kern, &cfg) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
  });
  return known ? n : -1;
}

// Launch with an optional cluster, beside the launch before where `dependent`.
template <typename... P, typename... A>
cudaError_t launch_beside(void (*kern)(P...), unsigned grid, unsigned threads, size_t smem,
                          unsigned cluster, bool dependent, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

TileHeads head_params(const HeadArgs& a) {
  TileHeads h{};
  h.D = a.head_dim; h.nq = a.q.heads * a.head_dim;
  h.norm = a.norm; h.rope = a.rope;
  h.rot = a.rope == OQ_ROPE_NONE ? 0 : a.rot_dim;
  h.eps = a.eps; h.inv_d = 1.f / (float)a.head_dim;
  h.qw = a.q.weight; h.qb = a.q.bias;
  h.kw = a.k.weight; h.kb = a.k.bias;
  h.cos = a.cos; h.sin = a.sin; h.n_pos = a.n_pos;
  h.positions = a.positions; h.pos_bs = a.pos_batch_stride;
  h.seq = (int)a.seq;
  return h;
}

oq_status run_tiles(const W8Params& w, const HeadArgs* heads, cudaStream_t s) {
  CUtensorMap ta, tb;
  const uint64_t K = (uint64_t)w.K, N = (uint64_t)w.N, T = (uint64_t)w.T;
  const bool ok = tma_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.a, K, T, K, 128, TM,
                             CU_TENSOR_MAP_SWIZZLE_128B) &&
                  tma_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.w, K, N, K, 128, BBOX,
                             CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return fail(OQ_ERR_CUDA, "cuTensorMapEncodeTiled failed or unavailable");
  const auto kern = heads ? &k_gemm_w8<true> : &k_gemm_w8<false>;
  cudaError_t e = allow_max_dynamic_smem(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(gemm_w8)");
  int units = resident_clusters(reinterpret_cast<const void*>(kern), 2, SMEM, NTHR);
  if (units < 0) return fail(OQ_ERR_CUDA, "gemm_w8: the occupancy query failed");
  if (units == 0) return fail(OQ_ERR_UNSUPPORTED, "gemm_w8: no CTA pair fits on this device");
  TileParams p{};
  p.w = w;
  p.cw = CH;
  if (heads) {
    p.cw = heads->head_dim;
    p.h = head_params(*heads);
  }
  p.maxch = TN / p.cw;
  p.npm = (w.N + p.cw - 1) / p.cw;
  const int64_t blocks = ((int64_t)w.T + 2 * TM - 1) / (2 * TM);
  p.ncol = (p.npm + p.maxch - 1) / p.maxch;
  if (blocks * p.ncol > 0x3FFFFFFF)
    return fail(OQ_ERR_INVALID_ARG, "gemm_w8: T x d_out too large for one call");
  p.blocks = (int)blocks;
  p.total = (int)blocks * p.ncol;
  // a group's activations take a quarter of L2 at most
  p.gm = (int)std::max<int64_t>(1, std::min<int64_t>(blocks, (32 << 20) / (2 * TM * (int64_t)w.K)));
  p.full = p.total / units * units;
  const int rest = p.total - p.full;
  p.split = rest ? std::min(units / rest, p.maxch) : 1;
  if (p.full == 0) units = rest * p.split;
  e = launch_beside(kern, 2u * (unsigned)units, NTHR, SMEM, 2, w.dependent, s, ta, tb, p);
  return e == cudaSuccess ? OQ_OK : cuda_fail(e, "launch gemm_w8");
}

// ---- few tokens ------------------------------------------------------------------------------
// Up to 32 tokens: bound by the weights' bytes (4096 x 4096: 16.8 MB, 2.6 us of HBM) and by latency, so
// nothing is staged (one token 5.4 us where tiles take 19.9; 4096 x 12288 10.6 us or 4.7 TB/s; with every
// call's weights from HBM). A block takes 16 channels and all of K: its eight warps read the weight rows
// straight into registers, all loads of a warp in flight together, and feed mma.sync (m16n8k32,
// weights as the 16 rows, tokens as the 8 columns); their sums meet in shared memory.
//
// Operand layout: lane (g = lane / 4, i = lane % 4) reads 32 bytes, k = 128 s + 32 i ..., of the weight rows g
// and g + 8 and of token g. An MMA adds products over its 32 k in any order, as long as both
// operands have the same one, so each 8 bytes a lane holds serve as its share of one MMA: four
// MMAs per 128 bytes, no shuffles, whole 128-byte lines from every row.
constexpr int kRowTokens = 32;             // tokens at most: four groups of the MMA's columns
constexpr int kHeadRowTokens = 16;         // tokens at most with heads
constexpr int RT = 256;                    // threads
constexpr int RW = RT / 32;

struct Line { uint32_t v[8]; };

// 32 bytes, zeros past the end of the row or of the rows. All loads are volatile: weights are asked
// for before dependency_wait() and codes after it, in the order written.
__device__ __forceinline__ Line load32(const int8_t* p, bool in, bool wide) {
  Line l;
  if (!in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) l.v[i] = 0u;
  } else if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(l.v[0]), "=r"(l.v[1]), "=r"(l.v[2]), "=r"(l.v[3]), "=r"(l.v[4]),
                   "=r"(l.v[5]), "=r"(l.v[6]), "=r"(l.v[7])
                 : "l"(p));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(l.v[4 * h]), "=r"(l.v[4 * h + 1]), "=r"(l.v[4 * h + 2]),
                     "=r"(l.v[4 * h + 3])
                   : "l"(p + 16 * h));
  }
  return l;
}

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct RowParams {
  W8Params w;
  TileHeads h;             // heads formed by the blocks of a cluster
  bool wide_a, wide_w;     // the codes' bases are 32-byte aligned (their rows are: K % 32 == 0)
};

// what the epilogue needs of one output, read before the weights arrive
struct OutConst { float alpha, mean, s, w1, b; };
__device__ __forceinline__ OutConst out_const(const W8Params& p, int t, int o) {
  OutConst c;
  c.alpha = p.a_scale[t];
  c.mean = p.mean ? p.mean[t] : 0.f;
  c.s = p.w_scale[o];
  c.w1 = p.mean ? p.w_rowsum[o] : 0.f;
  c.b = p.bias ? __bfloat162float(p.bias[o]) : 0.f;
  return c;
}
__device__ __forceinline__ float out_value(int sum, const OutConst& c) {
  return __fmaf_rn((float)sum, __fmul_rn(c.alpha, c.s), __fmaf_rn(c.mean, c.w1, c.b));
}
__device__ __forceinline__ void store_bf16(const W8Params& p, int t, int o, float y) {
  reinterpret_cast<__nv_bfloat16*>(p.out)[(int64_t)t * p.N + o] = __float2bfloat16_rn(y);
}
// a float in the shared memory of CTA `rank` of the cluster, at this CTA's address `mine`
__device__ __forceinline__ float cluster_float(const float* mine, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];"
               : "=f"(v)
               : "r"(dev::map_to_cta(dev::smem_u32(mine), (uint32_t)rank))
               : "memory");
  return v;
}
// sum over the 16 lanes that hold a token's 16 channels
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Heads of D <= 128 elements for few tokens: the D / 16 blocks that hold a head's channels are a
// cluster. Each block's values and partial sums (of values, of squares) lie in its shared memory,
// and every block reads the others'. Thread: channel oc of tokens tid / 16 + 16 e, y[e] its values.
template <int NO, int MT>
__device__ __forceinline__ void cluster_heads(const RowParams& rp, int o0, const float (&y)[NO],
                                              const int64_t (&pos)[NO], const float (&cs)[NO],
                                              const float (&sn)[NO], float (*s_y)[17],
                                              float (*s_stat)[MT]) {
  const W8Params& p = rp.w;
  const TileHeads& h = rp.h;
  const int tid = threadIdx.x, oc = tid & 15, C = h.D / 16, half = h.rot / 2;
  const int rank = (int)dev::cluster_ctarank(), el = rank * 16 + oc;
  const bool is_q = o0 < h.nq, layer = h.norm == OQ_NORM_LAYER;
  const float* wt = is_q ? h.qw : h.kw;
  const float* bs = is_q ? h.qb : h.kb;
  const bool in_rot = el < h.rot;
  const int other = h.rope == OQ_ROPE_PAIRS ? el ^ 1 : el < half ? el + half : el - half;
  const float wv = wt ? wt[el] : 1.f, bv = bs ? bs[el] : 0.f;
  const float wo = wt && in_rot ? wt[other] : 1.f, bo = bs && in_rot ? bs[other] : 0.f;
  float m[NO], q[NO];
#pragma unroll
  for (int e = 0; e < NO; ++e) {
    const int t = (tid >> 4) + 16 * e;
    const float part = half_warp_sum(layer ? y[e] : y[e] * y[e]);
    if (t < MT) {
      s_y[t][oc] = y[e];
      if (oc == 0) s_stat[0][t] = part;
    }
    m[e] = 0.f;
  }
  __syncwarp();   // the cluster's barrier is for whole warps, whose lanes parted at the stores
  dev::cluster_sync();
#pragma unroll
  for (int e = 0; e < NO; ++e) {
    const int t = min((tid >> 4) + 16 * e, MT - 1);
    q[e] = 0.f;
    for (int r = 0; r < C; ++r) q[e] += cluster_float(&s_stat[0][t], r);
  }
  if (layer) {
#pragma unroll
    for (int e = 0; e < NO; ++e) {
      const int t = (tid >> 4) + 16 * e;
      m[e] = q[e] * h.inv_d;
      const float part = half_warp_sum((y[e] - m[e]) * (y[e] - m[e]));
      if (oc == 0 && t < MT) s_stat[1][t] = part;
    }
    __syncwarp();
    dev::cluster_sync();
#pragma unroll
    for (int e = 0; e < NO; ++e) {
      const int t = min((tid >> 4) + 16 * e, MT - 1);
      q[e] = 0.f;
      for (int r = 0; r < C; ++r) q[e] += cluster_float(&s_stat[1][t], r);
    }
  }
#pragma unroll
  for (int e = 0; e < NO; ++e) {
    const int t = (tid >> 4) + 16 * e;
    if (t >= p.T) break;
    const float r = h.norm == OQ_NORM_NONE ? 1.f : rsqrtf(fmaf(q[e], h.inv_d, h.eps));
    const float n = fmaf((y[e] - m[e]) * r, wv, bv);
    float out = n;
    if (in_rot && pos[e] >= 0) {
      const float no = fmaf((cluster_float(&s_y[t][other & 15], other >> 4) - m[e]) * r, wo, bo);
      const bool low = h.rope == OQ_ROPE_PAIRS ? !(el & 1) : el < half;
      out = low ? n * cs[e] - no * sn[e] : n * cs[e] + no * sn[e];
    }
    store_bf16(p, t, o0 + oc, out);
  }
  __syncwarp();
  dev::cluster_sync();   // no block leaves while another still reads its values
}

// Position and angle of this thread's elements; they do not come from the launch before.
template <int NO>
__device__ __forceinline__ void row_angles(const RowParams& rp, int64_t (&pos)[NO], float (&cs)[NO],
                                           float (&sn)[NO]) {
  const TileHeads& h = rp.h;
  const int half = h.rot / 2;
  const int el = (int)dev::cluster_ctarank() * 16 + ((int)threadIdx.x & 15);
  const int i = h.rope == OQ_ROPE_PAIRS ? el / 2 : el < half ? el : el - half;
#pragma unroll
  for (int e = 0; e < NO; ++e) {
    const int t = ((int)threadIdx.x >> 4) + 16 * e;
    pos[e] = -1;
    cs[e] = sn[e] = __int_as_float(0x7fc00000);   // a position past the table
    if (t < rp.w.T && el < h.rot) {
      const int b = t / h.seq, s = t - b * h.seq;
      pos[e] = h.positions ? (int64_t)h.positions[b * h.pos_bs + s] : s;
      if (pos[e] >= 0 && pos[e] < h.n_pos) {
        cs[e] = h.cos[pos[e] * half + i];
        sn[e] = h.sin[pos[e] * half + i];
      }
    }
  }
}

// NT groups of eight tokens; RU 128-byte segments of a warp in flight; blocks for RB to an SM.
// HEADS: a cluster's blocks form a head (cluster_heads).
template <int NT, int RU, int RB, bool HEADS>
__global__ void __launch_bounds__(RT, RB) k_gemm_w8_rows(const __grid_constant__ RowParams rp) {
  const W8Params& p = rp.w;
  __shared__ int s_part[RW][NT * 8][17];   // [warp][token][channel], one word of padding
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, i = lane & 3;
  const int o0 = (int)blockIdx.x * 16;
  const int segs = (p.K + 127) / 128;
  const int8_t* w0 = p.w + (int64_t)(o0 + g) * p.K + 32 * i;
  const int8_t* w1 = w0 + (int64_t)8 * p.K;
  const int8_t* a0 = p.a + (int64_t)g * p.K + 32 * i;
  // this thread's outputs: channel tid % 16 of tokens tid / 16, tid / 16 + 16; their constants are
  // read ahead where there are registers for them
  constexpr int NO = NT > 2 ? 2 : 1;
  const int oc = tid & 15;
  OutConst c0 = {};
  dependents_begin();
  if (HEADS && o0 >= p.N) return;   // the last cluster's spare blocks, behind all heads
  const bool head = HEADS && o0 < p.n_head;   // the same for a cluster's blocks
  int64_t pos[NO];
  float cs[NO], sn[NO];
  bool waited = false;
  int acc[NT][4] = {};
  for (int s0 = warp; s0 < segs; s0 += RW * RU) {
    Line wr[RU][2], x[RU][NT];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int k = (s0 + u * RW) * 128;
      const bool in = k + 32 * i < p.K;   // N % 16 == 0: the channels are all there
      wr[u][0] = load32(w0 + k, in, rp.wide_w);
      wr[u][1] = load32(w1 + k, in, rp.wide_w);
    }
    if (!waited) {   // the first weights are on their way
      if (head) row_angles<NO>(rp, pos, cs, sn);
      dependency_wait();
      waited = true;
      if (NO == 1 && (tid >> 4) < p.T) c0 = out_const(p, tid >> 4, o0 + oc);
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int k = (s0 + u * RW) * 128;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        x[u][n] = load32(a0 + (int64_t)(n * 8) * p.K + k, k + 32 * i < p.K && n * 8 + g < p.T,
                         rp.wide_a);
    }
#pragma unroll
    for (int u = 0; u < RU; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          mma_s8(acc[n], wr[u][0].v[j], wr[u][1].v[j], wr[u][0].v[j + 1], wr[u][1].v[j + 1],
                 x[u][n].v[j], x[u][n].v[j + 1]);
  }
  if (!waited) {   // a warp without a segment
    if (head) row_angles<NO>(rp, pos, cs, sn);
    dependency_wait();
    if (NO == 1 && (tid >> 4) < p.T) c0 = out_const(p, tid >> 4, o0 + oc);
  }
  // channels g and g + 8 of tokens 2 i and 2 i + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    s_part[warp][n * 8 + 2 * i][g] = acc[n][0];
    s_part[warp][n * 8 + 2 * i + 1][g] = acc[n][1];
    s_part[warp][n * 8 + 2 * i][g + 8] = acc[n][2];
    s_part[warp][n * 8 + 2 * i + 1][g + 8] = acc[n][3];
  }
  __syncthreads();
  float y[NO] = {};
#pragma unroll
  for (int e = 0; e < NO; ++e) {
    const int t = (tid >> 4) + 16 * e, o = o0 + oc;
    if (t >= p.T) break;   // T <= 8 NT
    int sum = 0;
#pragma unroll
    for (int q = 0; q < RW; ++q) sum += s_part[q][t][oc];
    if (!HEADS && p.out_acc) {
      reinterpret_cast<int32_t*>(p.out)[(int64_t)t * p.N + o] = sum;
      continue;
    }
    y[e] = out_value(sum, NO == 1 ? c0 : out_const(p, t, o));
    if (!HEADS && o < p.n_head)
      p.head[(int64_t)t * p.n_head + o] = y[e];
    else if (!head)
      store_bf16(p, t, o, y[e]);
  }
  if constexpr (HEADS) {
    __shared__ float s_y[NT * 8][17], s_stat[2][NT * 8];
    __syncwarp();
    if (head) cluster_heads<NO, NT * 8>(rp, o0, y, pos, cs, sn, s_y, s_stat);
  }
}

template <int NT, bool HEADS>
cudaError_t launch_rows(const RowParams& p, cudaStream_t s) {
  // More segments in flight where a warp has them (K >= 4096) and the blocks are at most two waves
  // of two to an SM; else more blocks to an SM. Measured, one token: 4096 x 4096 5.4 us against
  // 5.9, 12288 x 4096 10.9 against 11.8; the other way 4096 x 12288 10.6 against 12.3, 1920 x 5760
  // (8 tokens) 4.6 against 6.0. 16 tokens: 4096 x 4096 6.4 against 7.0; the other way
  // 4096 x 12288 13.5 against 14.6, 1920 x 5760 (24 tokens) 6.2 against 7.8.
  const unsigned cluster = HEADS ? (unsigned)p.h.D / 16u : 1u;
  const unsigned grid = ((unsigned)(p.w.N / 16) + cluster - 1) / cluster * cluster;
  constexpr int D = NT == 1 ? 2 : 1;
  // Clusters (heads) want the room: 4096 -> 6144, one token, 9.9 us with the rotation in front against 13.2.
  if constexpr (!HEADS)
    if (p.w.K >= 4096 && grid <= 2u * 2u * (unsigned)device_sms())
      return launch_beside(k_gemm_w8_rows<NT, 2 * D, 2, false>, grid, RT, 0, cluster, p.w.dependent,
                           s, p);
  return launch_beside(k_gemm_w8_rows<NT, D, 3, HEADS>, grid, RT, 0, cluster, p.w.dependent, s, p);
}

oq_status run_rows(const W8Params& w, const HeadArgs* heads, cudaStream_t s) {
  RowParams p{};
  p.w = w;
  p.wide_a = (reinterpret_cast<uintptr_t>(w.a) & 31u) == 0;
  p.wide_w = (reinterpret_cast<uintptr_t>(w.w) & 31u) == 0;
  cudaError_t e;
  if (heads) {
    p.h = head_params(*heads);
    e = w.T <= 8 ? launch_rows<1, true>(p, s) : launch_rows<2, true>(p, s);
  } else {
    e = w.T <= 8    ? launch_rows<1, false>(p, s)
        : w.T <= 16 ? launch_rows<2, false>(p, s)
        : w.T <= 24 ? launch_rows<3, false>(p, s)
                    : launch_rows<4, false>(p, s);
  }
  return e == cudaSuccess ? OQ_OK : cuda_fail(e, "launch gemm_w8_rows");
}

// ---- a few dozen to a few hundred tokens -----------------------------------------------------
// Up to 256 tokens the weights' bytes still bound the product, and a tile for every 256 channels leaves
// most SMs idle, so K is split too: a cluster of S CTAs owns 128 channels, CTA r its K blocks
// [r ks, (r + 1) ks). All tokens at once: channels are the MMA's 128 rows (cta_group::1), tokens
// its columns. Weights and tokens stream through a ring of TMA stages, weights by one thread and
// tokens by another; the int32 partial sums go from TMEM to shared memory, and after a cluster
// barrier CTA r adds its share of the tokens from all S CTAs through distributed shared memory.
// Whole numbers add exactly in any order, so the result is that of the other shapes bit for bit.
// 40 x 4096 x 4096 9.5 us, 128 x 4096 x 12288 18.2, 256 x 12288 x 4096 21.8; a CTA's start, the barriers
// and the end are 6 to 10 us of that, a K block 0.36 us.
constexpr int PT = 256;                    // threads
constexpr int PM = kSplitChannels;         // channels of a cluster
constexpr int PWB = PM * 128;              // weight bytes of a K block
constexpr int kSplitTokens = kGemmW8FewTokens;   // tokens at most
static_assert(kSplitTail == 256 + 12 * kSplitTokens, "barriers, scales, means, positions");

struct SplitParams {
  W8Params w;
  TileHeads h;                             // heads formed in the epilogue (HEADS)
  int npad, tcols, ks, nkb, ns, off_bar;   // of SplitShape
};

// Heads of D elements, D a divisor of 128, in the epilogue of the split: a lane holds four channels (o
// ... o + 3) of one token, D / 4 neighbouring lanes a head. The token is the warp's.
struct LaneHead {
  float4 wv, bv;
  int el;         // first element of this lane in its head
  bool head;
};
__device__ __forceinline__ LaneHead lane_head(const SplitParams& sp, int o) {
  const TileHeads& h = sp.h;
  LaneHead l;
  l.head = o < sp.w.n_head;
  l.el = o % h.D;
  const float* wt = o < h.nq ? h.qw : h.kw;
  const float* bs = o < h.nq ? h.qb : h.kb;
  l.wv = l.head && wt ? *reinterpret_cast<const float4*>(wt + l.el) : make_float4(1.f, 1.f, 1.f, 1.f);
  l.bv = l.head && bs ? *reinterpret_cast<const float4*>(bs + l.el) : make_float4(0.f, 0.f, 0.f, 0.f);
  return l;
}
// the angle of a token at position pos for the lane's channels: cosines, and sines with their signs
struct LaneAngle {
  float4 c, s;
  bool turn;
};
__device__ __forceinline__ LaneAngle lane_angle(const SplitParams& sp, const LaneHead& l, int pos) {
  const TileHeads& h = sp.h;
  const int half = h.rot / 2;
  const bool low = l.el < half;
  LaneAngle a;
  a.turn = l.head && l.el < h.rot && pos >= 0;
  const float nan = __int_as_float(0x7fc00000);   // a position past the table
  a.c = a.s = make_float4(nan, nan, nan, nan);
  if (a.turn && pos < h.n_pos) {
    if (h.rope == OQ_ROPE_PAIRS) {
      const float2 c2 = *reinterpret_cast<const float2*>(h.cos + (int64_t)pos * half + l.el / 2);
      const float2 s2 = *reinterpret_cast<const float2*>(h.sin + (int64_t)pos * half + l.el / 2);
      a.c = make_float4(c2.x, c2.x, c2.y, c2.y);
      a.s = make_float4(-s2.x, s2.x, -s2.y, s2.y);
    } else {
      const int i = low ? l.el : l.el - half;
      a.c = *reinterpret_cast<const float4*>(h.cos + (int64_t)pos * half + i);
      a.s = *reinterpret_cast<const float4*>(h.sin + (int64_t)pos * half + i);
      if (low) a.s = make_float4(-a.s.x, -a.s.y, -a.s.z, -a.s.w);
    }
  }
  return a;
}
// The values of the lane's channels of TU tokens, step by step for all of them (the steps of one wait
// for each other's shuffles); y stays where the lane holds no head.
template <int TU>
__device__ __forceinline__ void lane_heads(const SplitParams& sp, const LaneHead& l,
                                           const LaneAngle (&a)[TU], int lane, float4 (&y)[TU]) {
  const TileHeads& h = sp.h;
  const int lanes = h.D / 4, half = h.rot / 2;
  auto group_sums = [&](float (&v)[TU]) {
    for (int m = lanes / 2; m > 0; m >>= 1) {
#pragma unroll
      for (int u = 0; u < TU; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], m);
    }
  };
  float4 n[TU];
  float q[TU], r[TU];
#pragma unroll
  for (int u = 0; u < TU; ++u) {
    n[u] = y[u];
    q[u] = (y[u].x + y[u].y) + (y[u].z + y[u].w);
  }
  if (h.norm == OQ_NORM_LAYER) {
    group_sums(q);
#pragma unroll
    for (int u = 0; u < TU; ++u) {
      const float m = q[u] * h.inv_d;
      n[u] = make_float4(y[u].x - m, y[u].y - m, y[u].z - m, y[u].w - m);
    }
  }
#pragma unroll
  for (int u = 0; u < TU; ++u) {
    q[u] = fmaf(n[u].x, n[u].x, n[u].y * n[u].y) + fmaf(n[u].z, n[u].z, n[u].w * n[u].w);
    r[u] = 1.f;
  }
  if (h.norm != OQ_NORM_NONE) {
    group_sums(q);
#pragma unroll
    for (int u = 0; u < TU; ++u) r[u] = rsqrtf(fmaf(q[u], h.inv_d, h.eps));
  }
  // the other half's lanes
  const int mate = l.el >= h.rot ? lane : l.el < half ? lane + half / 4 : lane - half / 4;
#pragma unroll
  for (int u = 0; u < TU; ++u) {
    n[u] = make_float4(fmaf(n[u].x * r[u], l.wv.x, l.bv.x), fmaf(n[u].y * r[u], l.wv.y, l.bv.y),
                       fmaf(n[u].z * r[u], l.wv.z, l.bv.z), fmaf(n[u].w * r[u], l.wv.w, l.bv.w));
    float4 o = make_float4(n[u].y, n[u].x, n[u].w, n[u].z);
    if (h.rope != OQ_ROPE_PAIRS) {
      o.x = __shfl_sync(0xffffffffu, n[u].x, mate);
      o.y = __shfl_sync(0xffffffffu, n[u].y, mate);
      o.z = __shfl_sync(0xffffffffu, n[u].z, mate);
      o.w = __shfl_sync(0xffffffffu, n[u].w, mate);
    }
    if (!l.head) continue;
    y[u] = n[u];
    if (a[u].turn)
      y[u] = make_float4(fmaf(n[u].x, a[u].c.x, o.x * a[u].s.x), fmaf(n[u].y, a[u].c.y, o.y * a[u].s.y),
                         fmaf(n[u].z, a[u].c.z, o.z * a[u].s.z), fmaf(n[u].w, a[u].c.w, o.w * a[u].s.w));
  }
}

template <bool HEADS>
__global__ void __launch_bounds__(PT)
    k_gemm_w8_split(const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_a,
                    const __grid_constant__ SplitParams sp) {
  const W8Params& p = sp.w;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + sp.off_bar);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 2 * kRingMax + 1);   // TMEM base, abort
  volatile uint32_t* s_abort = misc + 1;
  float2* s_tok = reinterpret_cast<float2*>(smem + sp.off_bar + 256);
  int* s_pos = reinterpret_cast<int*>(s_tok + kSplitTokens);   // HEADS: the tokens' positions
  dependents_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = (int)dev::cluster_nctarank(), r = (int)dev::cluster_ctarank();
  const int o0 = ((int)blockIdx.x / S) * PM;
  const int kb0 = r * sp.ks, nk = max(0, min(sp.nkb, kb0 + sp.ks) - kb0);
  const int ns = sp.ns, xb = sp.npad * 128, stage = PWB + xb;
  auto full = [&](int st) { return dev::smem_u32(&bars[st]); };
  auto free_bar = [&](int st) { return dev::smem_u32(&bars[kRingMax + st]); };
  const uint32_t done = dev::smem_u32(&bars[2 * kRingMax]);

  if (tid == 0) {
    for (int st = 0; st < ns; ++st) {
      dev::mbar_init(full(st), 2);
      dev::mbar_init(free_bar(st), 1);
    }
    dev::mbar_init(done, 1);
    misc[1] = 0u;
    dev::fence_mbar_init();
    dev::prefetch_tmap(&tm_w);
    dev::prefetch_tmap(&tm_a);
  }
  if (warp == 1) {
    dev::tmem_alloc(dev::smem_u32(&misc[0]), (uint32_t)sp.tcols);
    dev::tmem_relinquish();
  }
  // this CTA's share of the tokens; this lane's four channels. What does not come from the launch before
  // is read before dependency_wait(), while that runs (0.2 us of 13).
  const int per = (p.T + S - 1) / S, t0 = min(p.T, r * per), t1 = min(p.T, t0 + per);
  const int o = o0 + lane * 4;
  const bool has = o < p.N;   // N % 16 == 0: the four channels lie all inside or all outside
  float2 cs[2], cw[2], cb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    cs[i] = has ? make_float2(p.w_scale[o + 2 * i], p.w_scale[o + 2 * i + 1]) : make_float2(0.f, 0.f);
    cw[i] = has && p.mean ? make_float2(p.w_rowsum[o + 2 * i], p.w_rowsum[o + 2 * i + 1])
                          : make_float2(0.f, 0.f);
    cb[i] = has && p.bias ? make_float2(__bfloat162float(p.bias[o + 2 * i]),
                                        __bfloat162float(p.bias[o + 2 * i + 1]))
                          : make_float2(0.f, 0.f);
  }
  LaneHead lh = {};
  if constexpr (HEADS) lh = lane_head(sp, o);
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem = misc[0];

  int issued = 0;   // stages this thread filled (the producers)
  if (warp == 0 || warp == 2) {
    // ---------------- producers: warp 0 the weights, warp 2 the tokens ----------------
    if (warp == 2) dependency_wait();   // the weights do not come from the launch before
    if (lane == 0) {
      const uint32_t first = dev::smem_u32(smem) + (warp == 0 ? 0u : (uint32_t)PWB);
      const uint32_t bytes = warp == 0 ? (uint32_t)PWB : (uint32_t)xb;
      const CUtensorMap* map = warp == 0 ? &tm_w : &tm_a;
      const int row = warp == 0 ? o0 : 0;
      Ring rg;
      for (int k = 0; k < nk; ++k, rg.next(ns)) {
        if (k >= ns && !ring_wait(rg, free_bar(rg.st), rg.phase ^ 1u, s_abort, p, kSiteGemmEmpty)) break;
        dev::mbar_arrive_expect_tx(full(rg.st), bytes);
        dev::tma_load_2d(first + (uint32_t)(rg.st * stage), map, (kb0 + k) * 128, row, full(rg.st));
        issued = k + 1;
      }
    }
    __syncwarp();
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMA issuer ----------------
    const uint32_t idesc = dev::idesc_i8(PM, sp.npad);
    const uint64_t dw = dev::sdesc_sw128(dev::smem_u32(smem));
    const uint64_t dx = dev::sdesc_sw128(dev::smem_u32(smem) + PWB);
    Ring rg;
    for (int k = 0; k < nk; ++k, rg.next(ns)) {
      if (!ring_wait(rg, full(rg.st), rg.phase, s_abort, p, kSiteGemmFull)) break;
      dev::tc_fence_after();
      const uint64_t at = (uint64_t)((uint32_t)(rg.st * stage) >> 4);   // of the stage, 16-byte units
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        dev::mma_i8(tmem, dw + at + 2 * kk, dx + at + 2 * kk, idesc, (k | kk) != 0);
      dev::mma_commit(free_bar(rg.st));
    }
    dev::mma_commit(done);   // arrives once every MMA issued above has completed
  }
  if constexpr (HEADS)
    for (int t = t0 + tid; t < t1; t += PT) {
      const int b = t / sp.h.seq, st = t - b * sp.h.seq;
      s_pos[t - t0] = sp.h.positions ? sp.h.positions[b * sp.h.pos_bs + st] : st;
    }
  if (warp != 2) dependency_wait();
  for (int t = t0 + tid; t < t1; t += PT)
    s_tok[t - t0] = make_float2(p.a_scale[t], p.mean ? p.mean[t] : 0.f);

  // ---- partial sums: TMEM -> shared memory, int32 [token][128 channels] ----
  {
    bool ok = true;
    if (lane == 0) ok = dev::mbar_wait(done, 0, p.err, kSiteGemmAccum, p.limit_ns);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0 && nk > 0 && *s_abort == 0u;
    dev::tc_fence_after();
    int32_t* part = reinterpret_cast<int32_t*>(smem);   // the stages are consumed
    const int q = warp & 3;
    for (int c = warp >> 2; c < sp.npad / 16; c += 2) {
      uint32_t v[16];
      dev::tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(c * 16), v);
      dev::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c * 16 + j) * PM + q * 32 + lane] = ok ? (int32_t)v[j] : 0;
    }
  }
  dev::tc_fence_before();
  __syncwarp();
  dev::cluster_sync();   // every CTA's partial sums and token scales are in place

  // ---- sum over the cluster and epilogue: a warp takes a token's 128 channels ----
  {
    const uint32_t mine = dev::smem_u32(smem) + (uint32_t)lane * 16u;
    constexpr int TU = 2;   // tokens of a warp whose loads are in flight together
    for (int tb = t0 + warp; tb < t1; tb += TU * (PT / 32)) {
      int4 sum[TU];
#pragma unroll
      for (int u = 0; u < TU; ++u) sum[u] = make_int4(0, 0, 0, 0);
      LaneAngle angle[TU];
      if constexpr (HEADS) {
#pragma unroll
        for (int u = 0; u < TU; ++u)
          angle[u] = lane_angle(sp, lh, s_pos[min(tb + u * (PT / 32), t1 - 1) - t0]);
      }
#pragma unroll
      for (int sr = 0; sr < kSplitMax; ++sr) {
        if (sr >= S) break;
        const uint32_t peer = dev::map_to_cta(mine, (uint32_t)sr);
#pragma unroll
        for (int u = 0; u < TU; ++u) {
          const int t = tb + u * (PT / 32);
          if (t < t1) {
            const uint4 v = dev::ld_cluster_v4(peer + (uint32_t)t * (PM * 4));
            sum[u].x += (int)v.x; sum[u].y += (int)v.y;
            sum[u].z += (int)v.z; sum[u].w += (int)v.w;
          }
        }
      }
      float4 y[TU];
#pragma unroll
      for (int u = 0; u < TU; ++u) {
        const int t = tb + u * (PT / 32);
        const float2 tk = s_tok[min(t, t1 - 1) - t0];
        const float2 al = make_float2(tk.x, tk.x), mn = make_float2(tk.y, tk.y);
        const float2 y0 = __ffma2_rn(make_float2((float)sum[u].x, (float)sum[u].y),
                                     __fmul2_rn(al, cs[0]), __ffma2_rn(mn, cw[0], cb[0]));
        const float2 y1 = __ffma2_rn(make_float2((float)sum[u].z, (float)sum[u].w),
                                     __fmul2_rn(al, cs[1]), __ffma2_rn(mn, cw[1], cb[1]));
        y[u] = make_float4(y0.x, y0.y, y1.x, y1.y);
      }
      if constexpr (HEADS) lane_heads<TU>(sp, lh, angle, lane, y);
#pragma unroll
      for (int u = 0; u < TU; ++u) {
        const int t = tb + u * (PT / 32);
        if (t >= t1 || !has) continue;
        if (!HEADS && p.out_acc)
          *reinterpret_cast<int4*>(reinterpret_cast<int32_t*>(p.out) + (int64_t)t * p.N + o) = sum[u];
        else if (!HEADS && o < p.n_head)
          *reinterpret_cast<float4*>(p.head + (int64_t)t * p.n_head + o) = y[u];
        else
          *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + (int64_t)t * p.N + o) =
              make_uint2(pack2(make_float2(y[u].x, y[u].y)), pack2(make_float2(y[u].z, y[u].w)));
      }
    }
  }
  __syncwarp();
  dev::cluster_sync();   // no CTA leaves while another still reads its partial sums

  // after an abort, loads already issued may still land: wait for them (bounded)
  if (lane == 0 && (warp == 0 || warp == 2) && *s_abort != 0u)
    for (int k = max(0, issued - ns); k < issued; ++k)
      dev::mbar_wait(full(k % ns), (uint32_t)(k / ns) & 1u, p.err, kSiteGemmDrain, p.limit_ns);
  __syncwarp();
  if (warp == 1) {
    dev::tc_fence_after();
    dev::tmem_dealloc(tmem, (uint32_t)sp.tcols);
  }
}

// How a product is split, and what it is expected to take (see "which shape" below).
struct SplitPlan {
  int S = 0;
  SplitShape shape;
  double us = 1e30;
};

SplitPlan plan_split(const W8Params& w) {
  const int npad = (w.T + 15) / 16 * 16, nkb = (w.K + 127) / 128, tiles = (w.N + PM - 1) / PM;
  const void* kern = reinterpret_cast<const void*>(&k_gemm_w8_split<false>);
  static Kept<std::tuple<int, int, int, int>, SplitPlan> kept;
  SplitPlan plan;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || allow_max_dynamic_smem(kern) != cudaSuccess) return plan;
  kept.get(std::make_tuple(dev, npad, nkb, tiles), &plan, [&](SplitPlan* best) {
    const double sms = device_sms();
    bool known = true;
    for (int S = 1; S <= kSplitMax; ++S) {
      SplitPlan c;
      c.S = S;
      c.shape = split_shape(w.T, w.K, S);
      if (c.shape.ks == 0) continue;   // a CTA would have nothing to do
      const int resident = resident_clusters(kern, S, c.shape.smem, PT);
      known = known && resident >= 0;
      if (resident <= 0) continue;     // does not launch here, or could not be asked now
      // Clusters that run at once: two CTAs to an SM where their shared memory allows, and about a
      // tenth less than the SMs would hold where a cluster's CTAs have to find room together (the
      // occupancy query counts one CTA to an SM; 192 CTAs in pairs ran faster than 96 alone).
      const double slots = split_ctas_per_sm(c.shape) * sms;
      const int fit = std::max(1, (int)(S == 1 ? slots : 0.9 * slots / S));
      // Fitted to measurements (one block of K of a CTA: 0.36 us and more with the tokens; two CTAs
      // on an SM share its rate; a CTA's start and end: 5.6 us and 0.02 a token; a wave of clusters
      // that does not fit waits for the one before)
      const int waves = (tiles + fit - 1) / fit;
      const double share = std::max(1.0, std::min(tiles, fit) * S / sms);
      c.us = waves * (5.6 + 0.02 * npad + share * c.shape.ks * (0.36 + 0.0004 * npad) + 0.2 * S);
      if (c.us < best->us) *best = c;
    }
    return known;
  });
  return plan;
}

oq_status run_split(const W8Params& w, const SplitPlan& plan, const HeadArgs* heads,
                    cudaStream_t s) {
  SplitParams p{};
  p.w = w;
  if (heads) p.h = head_params(*heads);
  const SplitShape& c = plan.shape;
  p.npad = c.npad; p.tcols = c.tcols; p.nkb = c.nkb; p.ks = c.ks; p.ns = c.ns; p.off_bar = c.off_bar;
  CUtensorMap tw, ta;
  const uint64_t K = (uint64_t)w.K, N = (uint64_t)w.N, T = (uint64_t)w.T;
  if (!tma_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.w, K, N, K, 128, PM,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tma_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.a, K, T, K, 128, (uint32_t)p.npad,
                  CU_TENSOR_MAP_SWIZZLE_128B))
    return fail(OQ_ERR_CUDA, "cuTensorMapEncodeTiled failed or unavailable");
  const int tiles = (w.N + PM - 1) / PM;
  const auto kern = heads ? &k_gemm_w8_split<true> : &k_gemm_w8_split<false>;
  cudaError_t e = allow_max_dynamic_smem(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(gemm_w8_split)");
  e = launch_beside(kern, (unsigned)(tiles * plan.S), PT, (size_t)c.smem, (unsigned)plan.S,
                    w.dependent, s, tw, ta, p);
  return e == cudaSuccess ? OQ_OK : cuda_fail(e, "launch gemm_w8_split");
}

// ---- which shape -------------------------------------------------------------------------------
// All three give the product's same bits, so the choice is one of time alone (of formed heads the last
// bits may differ), by estimates (us) fitted to measurements on this device. Rows: the weights at the
// HBM rate, and the tokens once for every 16 channels at the L2 rate. Tiles: 128 bytes of K of a tile,
// by its width. Measured against estimate: rows 1 x 4096 x 4096 5.4 (5.0), 32 x 4096 x 12288 17.1 (18.1);
// split 40 x 4096 x 4096 9.5 (10.4), 128 x 4096 x 12288 18.2 (17.2), 256 x 12288 x 4096 21.8 (22.6);
// tiles 256 x 4096 x 12288 20.8 (21.2), 256 x 4096 x 4096 14.6 (15.0).
double rows_us(const W8Params& w) {
  const double bytes = (double)w.N * w.K;
  return 2.2 + bytes / 6.2e6 + bytes * w.T / 16 / 13e6;
}
double tiles_us(const W8Params& w, int cw) {   // cw: channels of a chunk, as run_tiles cuts tiles
  const int maxch = TN / cw, npm = (w.N + cw - 1) / cw;
  const int ncol = (npm + maxch - 1) / maxch;   // T <= 256: one token block
  const int units = std::max(device_sms() / 2, 1);
  const int split = std::max(1, std::min(units / ncol, maxch)), waves = (ncol + units - 1) / units;
  return 6.8 + waves * ((w.K + 127) / 128) * (0.19 + 0.00102 * cw * maxch / split);
}

}  // namespace

namespace {
bool tiles_form(int head_dim, int rope, int rot_dim) {
  return head_dim % 32 == 0 && (rope == OQ_ROPE_NONE || rot_dim % 32 == 0);
}
}  // namespace

// Forming the heads saves a launch, about 3 us of the host's time. On the GPU, with the rotation in
// front, against the head kernel behind: 4096 -> 6144 with 1 token 9.9 us against 11.2, 16 tokens 11.9
// against 13.8, 32 tokens 13.0 against 15.6, 64 tokens 14.0 against 15.4; 1920 -> 5760 with 24 tokens
// 11.5 against 11.3, 128 tokens 16.4 against 15.5.
bool gemm_w8_forms_heads(int64_t T, int head_dim, int rope, int rot_dim) {
  if (T <= kHeadRowTokens) return head_dim <= 128;    // a cluster of at most eight blocks
  if (T <= kSplitTokens) return PM % head_dim == 0;   // whole heads in a cluster's channels
  return tiles_form(head_dim, rope, rot_dim);
}

oq_status launch_gemm_w8(const GemmW8Args& g, cudaStream_t s) try {
  if (g.T == 0) return OQ_OK;
  W8Params p{};
  p.a = g.a; p.w = g.w; p.a_scale = g.a_scale; p.mean = g.mean; p.w_scale = g.w_scale;
  p.w_rowsum = g.w_rowsum; p.bias = reinterpret_cast<const __nv_bfloat16*>(g.bias);
  p.T = (int)g.T; p.K = (int)g.K; p.N = (int)g.N; p.out_acc = g.out_acc;
  p.n_head = (int)g.n_head; p.out = g.out; p.head = g.head; p.dependent = g.dependent;
  p.wide = (reinterpret_cast<uintptr_t>(g.out) & 31u) == 0;
  p.err = device_error_word();
  if (!p.err) return fail(OQ_ERR_CUDA, "device error word unavailable");
  p.limit_ns = kWaitLimitNs;
  if (g.T > kSplitTokens) return run_tiles(p, g.heads, s);
  // with heads: rows up to 16 tokens (a cluster of up to eight blocks each), then the split
  if (g.heads && g.T <= kHeadRowTokens) return run_rows(p, g.heads, s);
  const SplitPlan split = plan_split(p);
  if (!g.heads && g.T <= kRowTokens && rows_us(p) <= split.us) return run_rows(p, nullptr, s);
  const bool tiles = !g.heads || tiles_form(g.heads->head_dim, g.heads->rope, g.heads->rot_dim);
  // A split's CTA that is alone on its SM has nothing to run under its heads' epilogue: 1.2 us. Split
  // against tiles, with the rotation: 200 tokens 4096 -> 4608 22.3 us, 23.3; 256 tokens 25.4, 24.1;
  // 64 tokens 512 -> 768 10.9, 12.2 (heads of 128, of which two make a tile).
  const double alone = g.heads && split_ctas_per_sm(split.shape) == 1 ? 1.2 : 0.0;
  if (split.S > 0 &&
      (!tiles || split.us + alone <= tiles_us(p, g.heads ? g.heads->head_dim : CH)))
    return run_split(p, split, g.heads, s);
  if (tiles) return run_tiles(p, g.heads, s);
  return fail(OQ_ERR_UNSUPPORTED, "gemm_w8: no cluster fits on this device");
} catch (const std::bad_alloc&) {   // of the kept launch shapes
  return fail(OQ_ERR_NOMEM, "host allocation");
}

}  // namespace oq
