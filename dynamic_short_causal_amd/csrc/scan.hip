// scan.hip -- dispatch of the selective-scan kernels and the one-token step.
#include "scan_device.hpp"

namespace dsc {

template <typename E, int NS, int NW> hipError_t scan_fwd_nw(const ScanP &, int64_t);

template <typename E> static hipError_t fwd(const ScanArgs &a) {
  if (a.B == 0 || a.T == 0) return hipSuccess;
  const ScanPlan pl = scan_plan(a.B, a.T, a.D, a.G, a.N);
  const ScanP p{a, a.ws + pl.hend, a.ws + pl.sdt, (int)(a.D / a.G), pl.nblk, pl.nc, pl.tc, 0};
  const int64_t groups = pl.cols * pl.nc;
  if (pl.ns == 2) {
    switch (pl.nw) {
      case 2: return scan_fwd_nw<E, 2, 2>(p, groups);
      case 4: return scan_fwd_nw<E, 2, 4>(p, groups);
      case 8: return scan_fwd_nw<E, 2, 8>(p, groups);
      default: return scan_fwd_nw<E, 2, 16>(p, groups);
    }
  }
  switch (pl.nw) {
    case 1: return scan_fwd_nw<E, 4, 1>(p, groups);
    case 2: return scan_fwd_nw<E, 4, 2>(p, groups);
    case 4: return scan_fwd_nw<E, 4, 4>(p, groups);
    case 8: return scan_fwd_nw<E, 4, 8>(p, groups);
    default: return scan_fwd_nw<E, 4, 16>(p, groups);
  }
}

hipError_t scan_fwd_launch(const ScanArgs &a) { return a.bf16 ? fwd<bf16>(a) : fwd<float>(a); }

// ---------------------------------------------------------------------------
// One token: h = exp(dt A) h + dt u B, y = (C h + Dk u) silu(z), the states h
// (B, D, N) and the convolution's inputs conv (B, W-1, D) in place.
//
// The states' bytes decide: 8 N a channel against 20 of everything else (W = 4,
// bf16).
// A wave takes 64 channels of a sequence.  For the states, L lanes share a
// channel, four states each: a wave's access is 1 KiB in one piece, 64 / L
// channels, and it makes L of them.  For everything else a lane has one channel
// of its own, the one of the L that its place among them names, so that the
// convolution, the step and the gate are computed once a channel and reach the
// other lanes by a broadcast among L neighbours; the sums come back the same way.
// ---------------------------------------------------------------------------
//
// The states are read and written past the caches, which nothing reads them
// from again before they are pushed out: 256 sequences x 6144 channels, 16
// states, in new memory each time, 76 us without and 60 us with that.
// Workgroups of 16 waves, where they give every CU one, walk memory in larger
// pieces: 55 us, 4.2 TB/s (a plain copy: 5.2 TB/s); 1024 sequences 228 and
// 193 us.  The bytes bound it.
constexpr int kScanDecWaves = 4, kScanDecManyWaves = 16;

// v of the lane at place i of the L neighbours
template <int L> __device__ __forceinline__ float spread(float v, int i) {
  if constexpr (L == 1) return v;
  else if constexpr (L == 2) return i == 0 ? dpp<0xa0>(v) : dpp<0xf5>(v);
  else if constexpr (L == 4)
    return i == 0 ? dpp<0x00>(v) : i == 1 ? dpp<0x55>(v) : i == 2 ? dpp<0xaa>(v) : dpp<0xff>(v);
  else return __shfl(v, ((int)threadIdx.x & (64 - L)) + i);
}
// the sum over the L neighbours, in each of them
template <int L> __device__ __forceinline__ float join(float v) {
  if constexpr (L > 1) v += dpp<0xb1>(v);
  if constexpr (L > 2) v += dpp<0x4e>(v);
  if constexpr (L > 4) v += dpp<0x141>(v);
  if constexpr (L > 8) v += dpp<0x140>(v);
  return v;
}

template <typename E, int L, bool ONE>
__global__ __launch_bounds__(kScanDecManyWaves * 64) void scan_decode_kernel(ScanArgs a,
                                                                            uint32_t first) {
  constexpr int NS = 4, WT = kScanMaxW, CP = 64 / L, LB = L < 4 ? L : 4;
  const int lane = (int)threadIdx.x & 63, q = lane % L, n0 = q * NS;
  const int64_t wid = ((int64_t)blockIdx.x + first) * (blockDim.x >> 6) + (threadIdx.x >> 6);
  const int64_t cols = (a.D + 63) / 64, b = wid / cols, c0 = (wid - b * cols) * 64;
  if (b >= a.B) return;  // whole waves; nothing is shared between them
  const int have = a.N - n0, S = a.W - 1;
  const bool whole = (a.N % 4) == 0 && have > 0;  // rows of states are whole 16-byte vectors
  const bool whole_A = whole && ((uintptr_t)a.A & 15) == 0;
  const int64_t cg = a.D / a.G;
  const int64_t co = c0 + q * CP + lane / L;  // the lane's own channel
  const bool mine = co < a.D;
  const int64_t c = mine ? co : a.D - 1;  // channels past the last are read as the last
  const E xr = ((const E *)a.x)[b * a.x_row + c];
  const float dl = to_f32<E>(((const E *)a.delta)[b * a.delta_row + c]);
  const E zr = a.z ? ((const E *)a.z)[b * a.z_row + c] : E{};
  E *cp = (E *)a.convT + b * S * a.D + c;
  E cv[WT - 1];
  float taps[WT];
#pragma unroll
  for (int k = 1; k < WT; ++k) {
    cv[k - 1] = E{};
    if (k < a.W) cv[k - 1] = cp[(int64_t)(S - k) * a.D];
  }
#pragma unroll
  for (int k = 0; k < WT; ++k) {
    taps[k] = a.W == 0 && k == 0 ? 1.0f : 0.0f;
    if (k < a.W) taps[k] = to_f32<E>(((const E *)a.w)[c * a.W + k]);
  }
  const float cb = a.cb ? to_f32<E>(((const E *)a.cb)[c]) : 0.0f;
  const float dtb = a.dtb ? a.dtb[c] : 0.0f, dk = a.Dk ? a.Dk[c] : 0.0f;

  auto bc = [&](const void *m, int64_t row, int64_t ch, float (&v)[NS]) {
    const E *p = (const E *)m + b * row + (ONE ? c0 : ch) / cg * a.N + n0;
    if (a.bc_vec && have > 0) {
      unpack_row<E, NS>(ld_row<E, NS>(p), v);
    } else {
#pragma unroll
      for (int j = 0; j < NS; ++j) v[j] = j < have ? to_f32<E>(p[j]) : 0.0f;
    }
  };
  float u = 0.0f, dt = 0.0f, z = 0.0f, o = 0.0f;
#pragma unroll 1
  for (int i0 = 0; i0 < L; i0 += LB) {
    // the states of LB accesses and what meets them, before they are needed
    float h[LB][NS], A2[LB][NS], Bv[ONE ? 1 : LB][NS], Cv[ONE ? 1 : LB][NS];
    float *hp[LB];
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int64_t chan = c0 + (i0 + i) * CP + lane / L, ch = chan < a.D ? chan : a.D - 1;
      hp[i] = a.hT + (b * a.D + ch) * a.N + n0;
      const float *Ap = a.A + ch * a.N + n0;
      if (whole) {
        const uint4 v = ld16nt(hp[i]);
        h[i][0] = __uint_as_float(v.x); h[i][1] = __uint_as_float(v.y);
        h[i][2] = __uint_as_float(v.z); h[i][3] = __uint_as_float(v.w);
      } else {
#pragma unroll
        for (int j = 0; j < NS; ++j) h[i][j] = j < have ? hp[i][j] : 0.0f;
      }
      if (!ONE || i == 0) {
        bc(a.Bm, a.b_row, ch, Bv[ONE ? 0 : i]);
        bc(a.Cm, a.c_row, ch, Cv[ONE ? 0 : i]);
      }
      if (whole_A) {
        ld_lds<NS>(Ap, A2[i]);
      } else {
#pragma unroll
        for (int j = 0; j < NS; ++j) A2[i][j] = j < have ? Ap[j] : 0.0f;
      }
    }
    if (i0 == 0) {
      float v = fmaf(taps[0], to_f32<E>(xr), cb);
#pragma unroll
      for (int k = 1; k < WT; ++k)
        if (k < a.W) v = fmaf(taps[k], to_f32<E>(cv[k - 1]), v);
      u = a.act ? silu_f(v) : v;
      if (a.residual) u += to_f32<E>(xr);
      dt = softplus_f(dl + dtb);
      z = a.z ? silu_f(to_f32<E>(zr)) : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const float dti = spread<L>(dt, i0 + i), dui = spread<L>(dt * u, i0 + i);
      float p = 0.0f;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        h[i][j] = fmaf(__builtin_amdgcn_exp2f(dti * (A2[i][j] * kLog2e)), h[i][j],
                       dui * Bv[ONE ? 0 : i][j]);
        // past N: zero times an infinite dt u would reach the sum
        h[i][j] = j < have ? h[i][j] : 0.0f;
        p = fmaf(Cv[ONE ? 0 : i][j], h[i][j], p);
      }
      p = join<L>(p);
      o = q == i0 + i ? p : o;
      if (c0 + (i0 + i) * CP + lane / L < a.D) {
        if (whole) {
          st16nt(hp[i], make_uint4(__float_as_uint(h[i][0]), __float_as_uint(h[i][1]),
                                   __float_as_uint(h[i][2]), __float_as_uint(h[i][3])));
        } else {
#pragma unroll
          for (int j = 0; j < NS; ++j)
            if (j < have) hp[i][j] = h[i][j];
        }
      }
    }
  }
  if (mine) {
    ((E *)a.y)[b * a.D + c] = to_elem<E>((a.Dk ? fmaf(dk, u, o) : o) * z);
#pragma unroll
    for (int k = 2; k < WT; ++k)  // the inputs slide by one token
      if (k < a.W) cp[(int64_t)(S - k) * a.D] = cv[k - 2];
    if (a.W > 1) cp[(int64_t)(S - 1) * a.D] = xr;
  }
}

template <typename E, int L, bool ONE> static hipError_t dec(const ScanArgs &a) {
  const int64_t n = a.B * ((a.D + 63) / 64);
  const int wv = n >= (int64_t)kScanDecManyWaves * kCUs ? kScanDecManyWaves : kScanDecWaves;
  return launch_slices((n + wv - 1) / wv, wv * 64, [&](uint32_t first, dim3 grid) {
    hipLaunchKernelGGL((scan_decode_kernel<E, L, ONE>), grid, dim3(wv * 64), 0,
                       (hipStream_t)a.stream, a, first);
  });
}

template <typename E, bool ONE> static hipError_t dec_l(const ScanArgs &a) {
  switch (scan_waves(a.N)) {
    case 1: return dec<E, 1, ONE>(a);
    case 2: return dec<E, 2, ONE>(a);
    case 4: return dec<E, 4, ONE>(a);
    case 8: return dec<E, 8, ONE>(a);
    default: return dec<E, 16, ONE>(a);
  }
}

template <typename E> static hipError_t dec_g(const ScanArgs &a) {
  if (a.B == 0) return hipSuccess;
  // every wave's 64 channels in one group: B and C are loaded once for them
  return a.G == 1 || a.D / a.G % 64 == 0 ? dec_l<E, true>(a) : dec_l<E, false>(a);
}

hipError_t scan_decode_launch(const ScanArgs &a) {
  return a.bf16 ? dec_g<bf16>(a) : dec_g<float>(a);
}

}  // namespace dsc
