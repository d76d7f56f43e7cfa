// scan_launch.hpp -- arguments and tiling of the selective-scan kernels
// (scan_fwd.hpp, scan_bwd.hpp, scan.hip), shared by the C ABI (checks,
// workspace queries) and the launchers so that the two always agree.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dsc {

// Tensors as in include/dsc.h; a null pointer is an absent optional one.
// *_row: elements from one token of a tensor to the next.
struct ScanArgs {
  const void *x, *delta, *Bm, *Cm, *w, *cb, *z, *conv0, *dy;
  const float *A, *Dk, *dtb, *h0;
  const int32_t *pos;
  void *y, *convT;                       // forward, decode
  float *hT;
  void *dx, *ddelta, *dBm, *dCm, *dw, *dcb, *dz;  // backward
  float *dA, *dDk, *ddtb;
  float *ws;
  int64_t B, T, D;
  int N, G, W;                           // W == 0: no convolution
  int64_t x_row, delta_row, z_row, b_row, c_row;
  bool bc_vec;  // four values of Bm or Cm are one aligned access
  bool bf16, residual, act;
  void *stream;
};

// Channels of a backward workgroup, one a lane.
constexpr int kScanCh = 64;

// N states in groups of ns, rounded up to a power of two: the forward's groups
// side by side in a wave, the waves of a backward workgroup.
inline int scan_waves(int N, int ns = 4) {
  int nw = 1;
  while (nw * ns < N) nw *= 2;
  return nw;
}

// Waves of a forward workgroup, by the groups that a channel's states lie in: a
// workgroup has 64 channels, or 32 from eight groups on.
constexpr int scan_fwd_waves(int gr) { return gr <= 4 ? gr : gr / 2; }

// Chunks of the time axis are whole numbers of kScanTile tokens, which every
// forward tile divides.
constexpr int kScanTile = 64;
constexpr int kCUs = 256;

// The forward's tiling.
struct ScanPlan {
  int ns, nw;    // states of a group, groups of a channel
  int nblk;      // channel blocks of one group of B and C
  int64_t cols;  // B * G * nblk: workgroups when the time axis is whole
  int tc;        // tokens of one chunk of the time axis (a multiple of the tile)
  int nc;        // chunks; more than one: a first pass leaves each chunk's end state
  // workspace, in floats from its start
  size_t hend;   // (B, nc, D, ns nw) states that the chunks end in, started from zero
  size_t sdt;    // (B, nc, D) sums of the step sizes
  size_t total;
};

// Two rules, by the waves a SIMD (m) that whole rows in groups of four states
// would give; both sides measured in bf16, T = 4096, D = 1536, N = 16:
// - the time axis is cut where m <= 0.4, into chunks that make three waves a
//   SIMD: a cut call runs the recurrence twice, once for the chunks' end states
//   without the output.  m = 0.38: 214 us cut, 278 whole; m = 0.47: 288 and
//   278.  It takes five tiles at least: 3 x 777 x 1032 fp32 takes 60 us in six
//   chunks, 74 in four and whole.
// - whole rows take groups of two states, and so twice the waves, while those
//   are at most three a SIMD.  m = 0.94: 431 us with two, 497 with four; m =
//   1.5: 580 and 680; m = 1.97: 782 and 681; m = 3: 1111 and 930.
inline ScanPlan scan_plan(int64_t B, int64_t T, int64_t D, int G, int N) {
  ScanPlan p{};
  const int64_t dg = D / G;
  auto block = [&p, B, G, N, dg](int ns) {
    p.ns = ns;
    p.nw = scan_waves(N, ns);
    const int cb = 64 / p.nw * scan_fwd_waves(p.nw);
    p.nblk = (int)((dg + cb - 1) / cb);
    p.cols = B * G * p.nblk;
  };
  block(4);
  const int64_t tiles = (T + kScanTile - 1) / kScanTile;
  const int64_t waves = p.cols * scan_fwd_waves(p.nw), simds = 4 * kCUs;
  int64_t nc = 1;
  if (waves > 0 && waves * 5 <= simds * 2 && tiles >= 5) {
    nc = 3 * simds / waves;
    if (nc > tiles) nc = tiles;
    if (nc > 64) nc = 64;
  } else if (N > 2 && N <= 32 && waves * 2 <= simds * 3) {
    block(2);
  }
  const int64_t per = tiles > 0 ? (tiles + nc - 1) / nc : 1;
  p.tc = (int)(per * kScanTile);
  p.nc = (int)(tiles > 0 ? (tiles + per - 1) / per : 1);
  size_t at = 0;
  auto take = [&at](size_t n) {
    const size_t o = at;
    at += (n + 15) / 16 * 16;  // 64-byte steps
    return o;
  };
  if (p.nc > 1) {
    p.hend = take((size_t)B * p.nc * D * (p.ns * p.nw));
    p.sdt = take((size_t)B * p.nc * D);
  }
  p.total = B > 0 && T > 0 ? at : 0;
  return p;
}

// Widest convolution, and the per-channel sums of the backward besides dA:
// dDk, ddt_bias, dcb and a row for each tap.
constexpr int kScanMaxW = 8;
constexpr int kScanParV = 3 + kScanMaxW;

// Tokens of a backward tile, whose states a lane keeps in registers: 64 of
// them, or 32 for one or two waves, whose threads prepare more of a tile each.
// 8 x 2048 x 1536, N = 8, two waves: 498 us (bf16) and 490 us (fp32) with tiles
// of 8 tokens, 748 and 1202 us with 16.
constexpr int scan_bwd_tile(int ns, int nw) { return ns == 8 || nw <= 2 ? 8 : 16; }

// Workgroups of the backward's main launch that a CU holds at once, by its
// registers and LDS.
constexpr int scan_bwd_resident(bool bf16, int nw, int W) {
  const bool full = !bf16 && W > 4;  // fp32 with more than four taps: above 256 registers
  return nw >= 8 ? 1 : nw == 4 ? (full ? 1 : 2) : nw == 2 ? (full ? 2 : 4) : 4;
}

// Chunks of the backward's time axis for `cols` columns of workgroups.  k chunks
// of n tiles each take cols k / slots rounds of resident workgroups, rounded up,
// and a round takes the time of n tiles; in a cut call of one tile more, for
// starting and for what the chunks hand on, and of a twentieth of a tile for every
// chunk, whose states each workgroup folds.  The least of that product, among the
// k that rounding leaves as they are.  Measured at 40 sizes with 1 to 64 chunks:
// 1.1 % above the best of them in the mean, 14 % at most (74 us against 65).
// N = 16, bf16: 8 x 4096 x 1536 (0.38 rounds whole) 1292 us in eight, 1409 in five,
// 2436 whole; 8 x 2048 x 1088 (0.27) 523 in eleven, 542 in seven, 573 in eight;
// 24 x 2048 x 1536 (1.13) 1902 in eight, 1998 in five, 2517 whole; 32 x 2048 x 1536
// (1.5) 2529 in two, 2549 whole, 2522 in eight; 1 x 4096 x 512 114 in 64, 123 in 32.
inline int64_t scan_bwd_chunks(int64_t cols, int64_t slots, int64_t tiles) {
  int64_t best = 1;
  double least = 0.0;
  for (int64_t k = 1; k <= 64 && k <= tiles; ++k) {
    const int64_t n = (tiles + k - 1) / k;
    if ((tiles + n - 1) / n != k) continue;
    const int64_t rounds = (cols * k + slots - 1) / slots;
    const double t = (double)rounds * ((double)n + (k > 1 ? 1.0 + 0.05 * (double)k : 0.0));
    if (k == 1 || t < least) {
      least = t;
      best = k;
    }
  }
  return best;
}

// Tiling of the backward and its workspace, in floats from the start.
struct ScanBwdPlan {
  int ns, nw, nblk, tc, nc, tiles;
  int64_t cols;
  size_t ck, cum, hend, qend, sdt, dbc, pA, pV, tail, head, total;
};

inline ScanBwdPlan scan_bwd_plan(int64_t B, int64_t T, int64_t D, int G, int N, int W,
                                 bool bf16) {
  ScanBwdPlan p{};
  // 16 waves of four states would have 128 registers each, too few
  p.ns = N > 32 ? 8 : 4;
  p.nw = scan_waves(N, p.ns);
  const int64_t dg = D / G;
  p.nblk = (int)((dg + kScanCh - 1) / kScanCh);
  p.cols = B * G * p.nblk;
  const int tile = scan_bwd_tile(p.ns, p.nw);
  const int64_t tiles = (T + tile - 1) / tile;
  const int64_t nc = scan_bwd_chunks(p.cols, (int64_t)kCUs * scan_bwd_resident(bf16, p.nw, W),
                                     tiles);
  const int64_t per = tiles > 0 ? (tiles + nc - 1) / nc : 1;
  p.tc = (int)(per * tile);
  p.nc = (int)(tiles > 0 ? (tiles + per - 1) / per : 1);
  p.tiles = (int)tiles;
  size_t at = 0;
  auto take = [&at](size_t n) {
    const size_t o = at;
    at += (n + 15) / 16 * 16;  // 64-byte steps
    return o;
  };
  const size_t rows = (size_t)B * tiles, parts = (size_t)B * p.nc, d = (size_t)D, np = p.ns * p.nw;
  p.ck = take(rows * d * np);
  p.cum = take(rows * d);
  if (p.nc > 1) {
    p.hend = take(parts * d * np);
    p.qend = take(parts * d * np);
    p.sdt = take(parts * d);
    p.tail = take(parts * (kScanMaxW - 1) * d);
    p.head = take(parts * (kScanMaxW - 1) * d);
  }
  p.dbc = take((size_t)G * p.nblk * B * T * 2 * np);
  p.pA = take(parts * d * np);
  p.pV = take(parts * kScanParV * d);
  p.total = B > 0 && T > 0 ? at : 0;
  return p;
}

hipError_t scan_fwd_launch(const ScanArgs &a);
hipError_t scan_bwd_launch(const ScanArgs &a);
hipError_t scan_decode_launch(const ScanArgs &a);

}  // namespace dsc
