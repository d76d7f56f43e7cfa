// scan_bwd.hip -- dispatch of the selective-scan backward (scan_bwd.hpp) and the
// kernel that adds its partial sums.
#include "scan_device.hpp"

namespace dsc {

constexpr int kScanFinThreads = 256;

// Adds the partials, in order, in one launch of four kinds of workgroups:
//   dC, dB of a token over its group's channel blocks;
//   dA, and the other parameters, over sequences and chunks;
//   dx of the last W - 1 tokens of each chunk but the last: the main kernel's
//   sum over its own tokens, and the next chunk's first ones.
struct ScanFin {
  int64_t bc, dA, dV, seam;  // workgroups of each kind
  int np;
  int64_t parts;
};

template <typename E>
__global__ __launch_bounds__(kScanFinThreads) void scan_bwd_finish_kernel(ScanBwdP p, ScanFin f) {
  const ScanArgs &a = p.a;
  int64_t blk = (int64_t)blockIdx.x + p.first;
  const int64_t BT = a.B * a.T;
  if (blk < f.bc) {
    int64_t i = blk * kScanFinThreads + threadIdx.x;
    const int64_t per = 2 * (int64_t)a.G * a.N;
    if (i >= BT * per) return;
    const int64_t row = i / per;
    int e = (int)(i - row * per);
    const bool isB = e >= a.G * a.N;
    if (isB) e -= a.G * a.N;
    const int g = e / a.N, n = e % a.N;
    const float *q = p.ws.dbc + ((int64_t)g * p.nblk * BT + row) * 2 * f.np + (isB ? f.np : 0) + n;
    const int64_t step = BT * 2 * f.np;
    float v = 0.0f;
#pragma unroll 4
    for (int k = 0; k < p.nblk; ++k) v += q[k * step];
    E *o = isB ? (E *)a.dBm : (E *)a.dCm;
    st_elem<E>(o + row * a.G * a.N + e, v);
    return;
  }
  blk -= f.bc;
  if (blk < f.dA) {
    const int64_t i = blk * kScanFinThreads + threadIdx.x;
    if (i >= a.D * a.N) return;
    const int64_t c = i / a.N, n = i - c * a.N;
    float v = 0.0f;
#pragma unroll 4
    for (int64_t k = 0; k < f.parts; ++k) v += p.ws.pA[(k * a.D + c) * f.np + n];
    a.dA[i] = v;
    return;
  }
  blk -= f.dA;
  if (blk < f.dV) {
    const int64_t i = blk * kScanFinThreads + threadIdx.x;
    if (i >= a.D * (3 + a.W)) return;
    const int k = (int)(i / a.D);
    const int64_t c = i - k * a.D;
    float v = 0.0f;
#pragma unroll 4
    for (int64_t r = 0; r < f.parts; ++r) v += p.ws.pV[(r * kScanParV + k) * a.D + c];
    if (k == 0) {
      if (a.dDk) a.dDk[c] = v;
    } else if (k == 1) {
      if (a.ddtb) a.ddtb[c] = v;
    } else if (k == 2) {
      if (a.dcb) st_elem<E>((E *)a.dcb + c, v);
    } else {
      st_elem<E>((E *)a.dw + c * a.W + (k - 3), v);
    }
    return;
  }
  blk -= f.dV;
  {
    int64_t i = blk * kScanFinThreads + threadIdx.x;
    const int S = a.W - 1;  // at least 1 where there are such workgroups
    if (i >= a.B * (p.nc - 1) * S * a.D) return;
    const int64_t c = i % a.D;
    i /= a.D;
    const int from_end = (int)(i % S);
    i /= S;
    const int chunk = (int)(i % (p.nc - 1));
    const int64_t b = i / (p.nc - 1);
    const int64_t t1 = (int64_t)(chunk + 1) * p.tc, t = t1 - 1 - from_end;
    const int64_t part = b * p.nc + chunk;
    constexpr int HALO = kScanMaxW - 1;
    float dx = p.ws.tail[(part * HALO + from_end) * a.D + c];
    for (int k = from_end + 1; k < a.W; ++k) {
      if (t + k >= a.T) break;
      if (a.pos && k > a.pos[b * a.T + t + k]) continue;
      dx = fmaf(to_f32<E>(((const E *)a.w)[c * a.W + k]),
                p.ws.head[((part + 1) * HALO + (k - from_end - 1)) * a.D + c], dx);
    }
    st_elem<E>((E *)a.dx + (b * a.T + t) * a.D + c, dx);
  }
}

// instantiated in scan_bwd_{bf16,f32}.hip
template <typename E, int NS, int NW> hipError_t scan_bwd_nw(const ScanBwdP &, int64_t);

template <typename E> static hipError_t bwd(const ScanArgs &a) {
  const ScanBwdPlan pl = scan_bwd_plan(a.B, a.T, a.D, a.G, a.N, a.W, a.bf16);
  ScanBwdP p{};
  p.a = a;
  p.dg = (int)(a.D / a.G);
  p.nblk = pl.nblk;
  p.nc = pl.nc;
  p.tc = pl.tc;
  p.tiles = pl.tiles;
  float *w = a.ws;
  p.ws = ScanBwdWs{w + pl.ck,  w + pl.cum, w + pl.hend, w + pl.qend, w + pl.sdt,
                   w + pl.dbc, w + pl.pA,  w + pl.pV,   w + pl.tail, w + pl.head};
  const bool any = a.B > 0 && a.T > 0;
  hipError_t e = hipSuccess;
  if (any) {
    const int64_t groups = pl.cols * pl.nc;
    if (pl.ns == 8) {
      e = scan_bwd_nw<E, 8, 8>(p, groups);
    } else {
      switch (pl.nw) {
        case 1: e = scan_bwd_nw<E, 4, 1>(p, groups); break;
        case 2: e = scan_bwd_nw<E, 4, 2>(p, groups); break;
        case 4: e = scan_bwd_nw<E, 4, 4>(p, groups); break;
        default: e = scan_bwd_nw<E, 4, 8>(p, groups); break;
      }
    }
    if (e != hipSuccess) return e;
  }
  auto blocks = [](int64_t n) { return (n + kScanFinThreads - 1) / kScanFinThreads; };
  ScanFin f{};
  f.bc = blocks(a.B * a.T * 2 * a.G * a.N);
  f.dA = blocks(a.D * a.N);
  f.dV = blocks(a.D * (3 + a.W));
  f.seam = any && a.W > 1 ? blocks(a.B * (pl.nc - 1) * (a.W - 1) * a.D) : 0;
  f.np = pl.ns * pl.nw;
  f.parts = any ? a.B * pl.nc : 0;
  return launch_slices(f.bc + f.dA + f.dV + f.seam, kScanFinThreads,
                       [&](uint32_t first, dim3 grid) {
    p.first = first;
    hipLaunchKernelGGL((scan_bwd_finish_kernel<E>), grid, dim3(kScanFinThreads), 0,
                       (hipStream_t)a.stream, p, f);
  });
}

hipError_t scan_bwd_launch(const ScanArgs &a) { return a.bf16 ? bwd<bf16>(a) : bwd<float>(a); }

}  // namespace dsc
