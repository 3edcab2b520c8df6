// How the split-K W8A8 GEMM (k_gemm_w8.cu) lays out its shared memory. Host arithmetic alone.
#pragma once

#include <algorithm>

namespace oq {

constexpr int kSplitChannels = 128;        // channels of a cluster (the MMA's rows)
constexpr int kSplitMax = 8;               // CTAs of a cluster at most (portable size)
constexpr int kRingMax = 12;               // stages at most
constexpr int kSplitTail = 256 + 12 * 256; // barriers; scale, mean and position of 256 tokens

constexpr int kSmemOfSm = 228 * 1024;      // shared memory of an SM,
constexpr int kSmemOfBlock = 1024;         // of which every block takes this much for itself
constexpr int kTmemOfSm = 512;             // tensor memory columns of an SM

struct SplitShape {
  int npad = 0;      // tokens, rounded up to 16 (the MMA's columns)
  int tcols = 0;     // TMEM columns: a power of two >= 32
  int nkb = 0;       // K blocks of 128 bytes,
  int ks = 0;        // of one CTA,
  int ns = 0;        // and stages of its ring
  int off_bar = 0;   // ring and partial sums lie in front of the barriers
  int need = 0;      // shared memory that is used,
  int smem = 0;      // and asked for
};

// CTAs to an SM that the estimate of a split's time counts on: two within 112 KB each. (With the few
// KB more that an SM has, 16 x 4096 x 12288 was split, 14.4 us, where rows take 13.7.)
inline int split_ctas_per_sm(const SplitShape& c) { return c.need <= 112 * 1024 ? 2 : 1; }

// T tokens, K bytes of K, over S CTAs; ks = 0 where a CTA would have nothing to do.
//
// Ring: as deep as the CTA has blocks, within half an SM's shared memory where the partial sums
// leave room for two CTAs, else within all of it; at least as large as the partial sums.
//
// A CTA asks for at least the share of its SM's shared memory that it takes of the tensor memory.
// Its tcgen05.alloc would otherwise wait, without a limit, for another CTA's columns (three CTAs
// of 256, five of 128), and that one may belong to a cluster, of a call on another stream, whose
// other CTAs wait for columns held by this cluster. With the shares no mix of these CTAs is
// resident that has not its columns too. The library's other kernels with tensor memory leave no
// more registers (or shared memory) on an SM than CTAs for the columns they leave.
inline SplitShape split_shape(int T, int K, int S) {
  SplitShape c;
  c.npad = (T + 15) / 16 * 16;
  c.tcols = 32;
  while (c.tcols < c.npad) c.tcols *= 2;
  c.nkb = (K + 127) / 128;
  const int ks = (c.nkb + S - 1) / S;
  if ((S - 1) * ks >= c.nkb) return c;
  const int stage = (kSplitChannels + c.npad) * 128;
  const int room = c.npad <= 192 ? 108 * 1024 : 216 * 1024;
  c.ks = ks;
  c.ns = std::min(std::min(ks, kRingMax), room / stage);
  c.off_bar = (std::max(c.ns * stage, c.npad * kSplitChannels * 4) + 1023) / 1024 * 1024;
  c.need = c.off_bar + kSplitTail + 1024;   // 1024: the base is aligned in the kernel
  c.smem = std::max(c.need, c.tcols * (kSmemOfSm / kTmemOfSm) - kSmemOfBlock);
  return c;
}

}  // namespace oq
