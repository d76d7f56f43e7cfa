// scan_fwd.hpp -- forward of the selective state-space scan with its short
// causal convolution, gfx950.
//
//   s = cb + sum_k w[:,k] x[t-k],  u = act(s) + rho x,  dt = softplus(delta + dt_bias)
//   h[t] = exp(dt A) h[t-1] + dt u B[t],  p = C[t] h[t] + Dk u,  y = p silu(z)
//
// A wave owns 64 / GR channels of one sequence (or of one chunk of it), their
// states in GR groups of NS side by side in its lanes, in registers.  The time
// axis passes in tiles, through a part of LDS that the wave has for itself:
//   prepare  a lane loads x, delta, z of the next tile, four channels at a time
//            (one tile ahead, in registers), forms u and dt, and leaves dt and
//            dt u in LDS;
//   scan     every lane walks the tile's tokens with its NS states; after GR
//            tokens the groups exchange their parts of C h, so that each ends
//            up with one token's sum;
//   finish   the lanes of the preparation add Dk u, gate, and store.
// B and C, as fp32, are all that the waves of a workgroup share: two buffers,
// one barrier a tile.  With the states of a channel in different waves instead,
// and three barriers, 16 x 4096 tokens of 1536 channels took 717 us, not 580.
//
// One state update is two products, two fused multiply-adds and an exponential,
// 24.5 cycles of a SIMD's issue; the preparation, the exchange and the loop add
// as much again.  The issue of vector instructions bounds the kernel: 16 x 4096
// x 1536, N = 16, bf16 takes 584 us, of which the state updates' own
// instructions are 251 us and the 0.8 GB moved 157 us.  It issues 9.8 instructions
// an update there, with two states a lane; with four, 8.7, but whole rows of that
// size then leave the SIMDs unevenly filled (scan_plan).
//
// A call with few channels and a long axis cuts the axis into chunks: a first
// launch (SUM) leaves the state that each chunk ends in when it starts from
// zero, and the sum of its step sizes, whose product with A is the logarithm
// of the chunk's whole decay.  Every workgroup of the second launch folds the
// chunks before its own, in order, and scans.
#pragma once

#include <type_traits>

#include "scan_device.hpp"

namespace dsc {

// Shape of a workgroup: WV waves of CP channels, whose states lie in GR groups
// of NS side by side in the wave; tiles of TT tokens, of which a lane prepares
// NI consecutive ones of PV of its wave's channels.
template <int NS_, int GR_> struct ScanGeo {
  static constexpr int NS = NS_, GR = GR_, CP = 64 / GR;
  static constexpr int WV = scan_fwd_waves(GR), CB = CP * WV, TH = 64 * WV;
  static constexpr int TT = GR <= 2 ? 16 : GR == 4 ? 32 : 64;
  static constexpr int per = TT * CP / 64;
  static constexpr int PV = CP < 4 ? CP : 4, NI = per / PV, NV = CP / PV;
  static_assert(NI * PV * 64 == TT * CP, "whole items");
};

// Orders a wave's LDS accesses: other lanes have written what is read next.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sums of GR registers over the GR groups of a wave; the lanes of group g
// return that of register g.
template <int GR> __device__ __forceinline__ float join_groups(const float (&v)[GR]) {
  if constexpr (GR == 1) {
    return v[0];
  } else {
    float r[GR / 2];
#pragma unroll
    for (int i = 0; i < GR / 2; ++i) r[i] = add_swap32(v[i], v[i + GR / 2]);
    if constexpr (GR == 2) {
      return r[0];
    } else {
      float s[GR / 4];
#pragma unroll
      for (int i = 0; i < GR / 4; ++i) s[i] = add_swap16(r[i], r[i + GR / 4]);
      if constexpr (GR == 4) {
        return s[0];
      } else {
        const bool b3 = (threadIdx.x & 8) != 0;
        float t[GR / 8];
#pragma unroll
        for (int i = 0; i < GR / 8; ++i)
          t[i] = (b3 ? s[i + GR / 8] : s[i]) + dpp<0x128>(b3 ? s[i] : s[i + GR / 8]);  // row_ror:8
        if constexpr (GR == 8) {
          return t[0];
        } else {
          const bool b2 = (threadIdx.x & 4) != 0;
          // the lane four away: mirrored in its half row, then in its quad
          return (b2 ? t[1] : t[0]) + dpp<0x1b>(dpp<0x141>(b2 ? t[0] : t[1]));
        }
      }
    }
  }
}

template <typename E, int NS, int GR, int WM, bool SUM>
__global__ __launch_bounds__(64 * scan_fwd_waves(GR))
    __attribute__((amdgpu_waves_per_eu(sizeof(E) == 2 && NS == 2 && WM <= 4 ? 3 : 2))) void scan_fwd_kernel(ScanP p) {
  typedef ScanGeo<NS, GR> Geo;
  constexpr int TT = Geo::TT, PV = Geo::PV, NI = Geo::NI, CP = Geo::CP, CB = Geo::CB;
  constexpr int WV = Geo::WV, TH = Geo::TH, NV = Geo::NV;
  constexpr int GT = 2;                 // tokens whose operands are loaded together
  constexpr int UB = GR < 4 ? 4 : GR;   // tokens of one round of the loop
  constexpr int Np = NS * GR, BR = 2 * Np;
  __shared__ __align__(16) E s_w[WM][CB];
  __shared__ __align__(16) float s_par[3][CB];
  __shared__ __align__(16) float s_dt[WV][TT + GT][CP];  // two more rows: see the loop's loads
  __shared__ __align__(16) float s_du[WV][TT + GT][CP];  // then the sums of C h
  __shared__ __align__(16) float s_bc[2][(TT + GT) * BR];
  const ScanArgs &a = p.a;
  const ScanWhere at = scan_where(blockIdx.x + p.first, a.G, p.dg, p.nblk, p.nc, CB);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int T = (int)a.T;
  const int t0 = at.chunk * p.tc, t1 = min(T, t0 + p.tc);
  const bool gate = !SUM && a.z != nullptr, packed = a.pos != nullptr;

  ld_filter<E, WM, CB>(a, at.c0, at.nch, TH, s_w);

  // the recurrence's lane: channel c, states n0 .. n0 + NS - 1.  Places past N hold
  // copies of the first states, and a state's places have a part of its C each: an
  // empty state, with zeros for B and C, would make an infinite input undefined,
  // and to clear it at every token took 456 us instead of 430 (8 x 4096 x 1536,
  // N = 12, bf16).
  const int ch = lane % CP, grp = lane / CP, n0 = grp * NS, have = a.N - n0;
  const int c = at.c0 + wave * CP + ch;
  const bool mine = wave * CP + ch < at.nch;
  float A2[NS], h[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    A2[j] = mine ? a.A[(int64_t)c * a.N + copy_of(n0 + j, a.N)] * kLog2e : 0.0f;
    h[j] = 0.0f;
  }
  if constexpr (!SUM) {
    if (a.h0 && mine) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
        h[j] = a.h0[((int64_t)at.b * a.D + c) * a.N + copy_of(n0 + j, a.N)];
    }
    if (mine) {
      // the chunks before this one, in order; a negative sum marks a chunk
      // that a document starts in, which keeps nothing of the state before it
      for (int q = 0; q < at.chunk; ++q) {
        const int64_t row = ((int64_t)at.b * p.nc + q) * a.D + c;
        const float sd = p.sdt[row];
        float ev[NS];
        ld_lds<NS>(p.hend + row * Np + n0, ev);
#pragma unroll
        for (int j = 0; j < NS; ++j)
          h[j] = sd < 0.0f ? ev[j] : fmaf(__builtin_amdgcn_exp2f(A2[j] * sd), h[j], ev[j]);
      }
    }
  }
  float sum_dt = 0.0f;
  bool fresh = false;  // a document started in this chunk

  // the lane's items: tokens r0 .. r0 + NI - 1 of the tile, channels v0 .. of the wave
  const int v0 = lane % NV * PV, r0 = lane / NV * NI;
  const int w0 = wave * CP + v0;  // in the workgroup's block
  const bool prep = w0 < at.nch;
  // the convolution's and the step's bias and Dk of the block's channels
  for (int i = threadIdx.x; i < CB; i += TH) {
    const bool on = i < at.nch;
    s_par[0][i] = on && a.cb ? to_f32<E>(((const E *)a.cb)[at.c0 + i]) : 0.0f;
    s_par[1][i] = on && a.dtb ? a.dtb[at.c0 + i] : 0.0f;
    s_par[2][i] = on && a.Dk ? a.Dk[at.c0 + i] : 0.0f;
  }
  // what u is held to where Dk multiplies it: without Dk an infinite u adds nothing.
  // (An undefined u has made the sum undefined.)  A select on the pointer would
  // take the one register more that the kernel for N = 16 does not have.
  __shared__ float s_most;
  if (threadIdx.x == 0) s_most = a.Dk ? __builtin_inff() : 0.0f;
  ScanRaw<E, PV, NI, WM> raw;
  BcRaw<E, NS, GR, TT, TH> bcr;
  const ScanOff off = scan_off(a, r0, w0);
  if (prep) ld_tile<E, PV, NI, WM, TT>(a, at.b, t0, r0, t1, at.c0, w0, off, gate, raw);
  ld_bc<E, NS, GR, TT, TH, true>(a, at.b, at.g, t0, t1, bcr);
  __syncthreads();

  int buf = 0;
  for (int tv = t0; tv < t1; tv += TT, buf ^= 1) {
    const int t = __builtin_amdgcn_readfirstlane(tv);
    float u[NI][PV];
    RowBits<E, PV> zr[NI];
    if (prep) {
      float cb[PV], dtb[PV];
      ld_lds<PV>(&s_par[0][w0], cb);
      ld_lds<PV>(&s_par[1][w0], dtb);
      conv_tile<E, PV, NI, WM, CB>(raw, a.W, packed, s_w, w0, cb, u);
      if (a.act) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < PV; ++j) u[i][j] = silu_f(u[i][j]);
      }
      if (a.residual) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          float x0[PV];
          unpack_row<E, PV>(raw.x[i + WM - 1], x0);
#pragma unroll
          for (int j = 0; j < PV; ++j) u[i][j] += x0[j];
        }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float dl[PV], dt[PV], du[PV];
        unpack_row<E, PV>(raw.dl[i], dl);
#pragma unroll
        for (int j = 0; j < PV; ++j) {
          dt[j] = softplus_f(dl[j] + dtb[j]);
          du[j] = dt[j] * u[i][j];
        }
        if (t + TT > t1) {  // a token past the end leaves the state as it is
          const bool in = t + r0 + i < t1;
#pragma unroll
          for (int j = 0; j < PV; ++j) {
            dt[j] = in ? dt[j] : 0.0f;
            du[j] = in ? du[j] : 0.0f;
          }
        }
        st_lds<PV>(&s_dt[wave][r0 + i][v0], dt);
        st_lds<PV>(&s_du[wave][r0 + i][v0], du);
        zr[i] = raw.z[i];
      }
    }
    // stored before the next tile's loads are issued: the wait for these values
    // would be a wait for those, too
    st_bc<E, NS, GR, TT, TH, true>(bcr, s_bc[buf], a.N);
    if (t + TT < t1) {
      ld_bc<E, NS, GR, TT, TH, true>(a, at.b, at.g, t + TT, t1, bcr);
      if (prep)
        ld_tile<E, PV, NI, WM, TT>(a, at.b, t + TT, r0, t1, at.c0, w0, off, gate, raw);
    }
    // tokens of the tile that start a document
    uint64_t starts = 0;
    if (packed) {
      const int tt = t + lane;
      starts = __ballot(lane < TT && tt < t1 && a.pos[(int64_t)at.b * T + min(tt, t1 - 1)] == 0);
    }
    // the only thing that the waves share is the tile's B and C; the other
    // buffer holds those of the tile that a wave may still be scanning
    __syncthreads();
    auto scan_tile = [&](auto starts_t) {
      constexpr bool STARTS = decltype(starts_t)::value;
      // a group's operands are loaded while the group before it is scanned
      struct Group {
        float bc[GT][SUM ? NS : 2 * NS], dt[GT], du[GT];
      } gr[2];
      const float *bcl = s_bc[buf] + grp * 2 * NS;
      const float *dtl = &s_dt[wave][0][ch];
      float *dul = &s_du[wave][0][ch];
      auto ld_group = [&](int g0, Group &g) {
#pragma unroll
        for (int i = 0; i < GT; ++i) {
          ld_lds<SUM ? NS : 2 * NS>(bcl + (g0 + i) * BR, g.bc[i]);
          g.dt[i] = dtl[(g0 + i) * CP];
          g.du[i] = dul[(g0 + i) * CP];
        }
      };
      auto scan_group = [&](int g0, const Group &g, float *acc) {
#pragma unroll
        for (int i = 0; i < GT; ++i) {
          const bool start = STARTS && (starts >> (g0 + i) & 1);
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            const float e = __builtin_amdgcn_exp2f(g.dt[i] * A2[j]);
            h[j] = fmaf(e, start ? 0.0f : h[j], g.du[i] * g.bc[i][j]);
            if constexpr (!SUM) sum = fmaf(g.bc[i][SUM ? 0 : NS + j], h[j], sum);
          }
          if constexpr (SUM) sum_dt += g.dt[i];
          else acc[i] = sum;
        }
      };
      ld_group(0, gr[0]);
#pragma unroll 1
      for (int g0 = 0; g0 < TT; g0 += UB) {
        float acc[UB];
#pragma unroll
        for (int k = 0; k < UB; k += 2 * GT) {
          ld_group(g0 + k + GT, gr[1]);
          scan_group(g0 + k, gr[0], acc + k);
          if constexpr (NS == 4) __builtin_amdgcn_sched_barrier(0);
          // past the tile's end: the next rows of LDS, which nothing uses
          ld_group(g0 + k + 2 * GT, gr[0]);
          scan_group(g0 + k + GT, gr[1], acc + k + GT);
          if constexpr (NS == 4) __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!SUM) {
          // the place of a token's dt u, which every lane has read, takes its sum
#pragma unroll
          for (int k = 0; k < UB; k += GR) {
            float v[GR];
#pragma unroll
            for (int i = 0; i < GR; ++i) v[i] = acc[k + i];
            dul[(g0 + k + grp) * CP] = join_groups<GR>(v);
          }
        }
      }
    };
    if (starts) scan_tile(std::true_type{});
    else scan_tile(std::false_type{});
    fresh |= starts != 0;
    wave_sync();
    if constexpr (!SUM) {
      if (prep) {
        float dk[PV];
        ld_lds<PV>(&s_par[2][w0], dk);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (t + r0 + i < t1) {
            float o[PV];
            ld_lds<PV>(&s_du[wave][r0 + i][v0], o);
            const float most = s_most;
#pragma unroll
            for (int j = 0; j < PV; ++j)
              o[j] = fmaf(dk[j], __builtin_amdgcn_fmed3f(u[i][j], -most, most), o[j]);
            if (gate) {
              float zv[PV];
              unpack_row<E, PV>(zr[i], zv);
#pragma unroll
              for (int j = 0; j < PV; ++j) o[j] *= silu_f(zv[j]);
            }
            st_at<E, PV>((E *)a.y + ((int64_t)at.b * T + t + i) * a.D + at.c0, off.d, o);
          }
        }
      }
      wave_sync();
    }
  }

  if constexpr (SUM) {
    if (mine) {
      const int64_t row = ((int64_t)at.b * p.nc + at.chunk) * a.D + c;
      st_lds<NS>(p.hend + row * Np + n0, h);
      if (grp == 0) p.sdt[row] = fresh ? -1.0f : sum_dt;
    }
  } else if (at.chunk == p.nc - 1) {
    if (a.hT && mine) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
        if (j < have) a.hT[((int64_t)at.b * a.D + c) * a.N + n0 + j] = h[j];
    }
    if (a.convT) {
      // the last W - 1 inputs, oldest first
      const int S = a.W - 1;
      for (int i = threadIdx.x; i < S * CB; i += TH) {
        const int j = i / CB, k = i % CB, tt = T - S + j;
        if (k >= at.nch) continue;
        E v{};
        if (tt >= 0)
          v = ((const E *)a.x)[((int64_t)at.b * T + tt) * a.x_row + at.c0 + k];
        else if (a.conv0)
          v = ((const E *)a.conv0)[((int64_t)at.b * S + tt + S) * a.D + at.c0 + k];
        ((E *)a.convT)[((int64_t)at.b * S + j) * a.D + at.c0 + k] = v;
      }
    }
  }
}

template <typename E, int NS, int GR, int WM>
static hipError_t scan_fwd_run(const ScanP &p, int64_t groups) {
  hipStream_t s = (hipStream_t)p.a.stream;
  constexpr int TH = ScanGeo<NS, GR>::TH;
  ScanP q = p;
  if (p.nc > 1) {
    const hipError_t e = launch_slices(groups, TH, [&](uint32_t first, dim3 grid) {
      q.first = first;
      hipLaunchKernelGGL((scan_fwd_kernel<E, NS, GR, WM, true>), grid, dim3(TH), 0, s, q);
    });
    if (e != hipSuccess) return e;
  }
  return launch_slices(groups, TH, [&](uint32_t first, dim3 grid) {
    q.first = first;
    hipLaunchKernelGGL((scan_fwd_kernel<E, NS, GR, WM, false>), grid, dim3(TH), 0, s, q);
  });
}

template <typename E, int NS, int GR>
hipError_t scan_fwd_nw(const ScanP &p, int64_t groups) {
  return p.a.W <= 4 ? scan_fwd_run<E, NS, GR, 4>(p, groups)
                    : scan_fwd_run<E, NS, GR, 8>(p, groups);
}

}  // namespace dsc
