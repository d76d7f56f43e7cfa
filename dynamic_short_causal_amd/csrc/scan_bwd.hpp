// scan_bwd.hpp -- backward of the selective state-space scan, gfx950.
//
// With dp = dy silu(z) and q[t] = dL/dh[t]:
//   q[t]  = C[t] dp[t] + exp(dt[t+1] A) q[t+1]
//   dC[t,n] = sum_c dp h,  dB[t,n] = sum_c q dt u          (over a group's channels)
//   r     = q exp(dt A) h[t-1],  dA += dt r,  S = sum_n A r,  e = sum_n q B
//   ddt   = u e + S,  ddelta = ddt sigmoid(delta + dt_bias)
//   du    = dt e + Dk dp,  ds = du act'(s),  dx = rho du + transposed convolution of ds
//   dz    = dy p silu'(z),  p = sum_n C h + Dk u
//
// Stored, the states would be N fp32 values against one activation, so they are
// formed again from the inputs.  Two launches over workgroups of 64 channels,
// one a lane, and N / 4 waves of four states each (N > 32: eight waves of
// eight states, since 16 waves would have 128 registers each):
//   sums  walks each chunk of the time axis from a zero state and leaves the
//         state and the summed step sizes at every tile's start and at the
//         chunk's end.  exp(A times the summed steps) is the decay since the
//         chunk's start, so the true state at a tile's start is the stored one
//         plus that decay times the state that enters the chunk.  Where the
//         axis is cut it also leaves what the chunk hands back to the tokens
//         before it, sum_t exp(A sum of steps to t) C[t] dp[t].
//   main  walks the tiles of each chunk backwards: the tile's states go into
//         registers, then the recurrence of q runs over them.
// Both prepare a tile four channels a thread, from rows that were loaded while
// the tile before was scanned.  The sums over a group's channels are taken over
// the 64 lanes by exchanging halves of two registers at a time, eight values a
// token together, and leave one fp32 partial per channel block; the parameters'
// gradients stay in the preparing threads' registers and leave one per chunk.
// A last launch adds the partials in a fixed order.
//
// The issue of vector instructions and the waits of two waves a SIMD for each
// other's barriers and LDS bound it: main issues 30 instructions a state
// update, 20 of them in the two recurrences (the exponential of a step twice,
// 4.5 for the sums over channels), and keeps the vector units 80 % busy.  8 x
// 4096 x 1536, N = 16, bf16: 1.28 ms, of which sums 0.32, main 0.95 and the last
// launch 0.02; the 0.7 GB of tensors take 137 us.  Tiles of eight tokens would
// allow three waves a SIMD, but store and read twice the states: 8 x 2048 x
// 1536 bf16 790 us against 708.
#pragma once

#include <type_traits>

#include "scan_device.hpp"

namespace dsc {

// Shape of a workgroup: NW waves of NS states, tiles of TT tokens, of which a
// thread prepares NI consecutive ones of PV channels.
template <int NS_, int NW_> struct BwdGeo {
  static constexpr int NS = NS_, NW = NW_, TT = scan_bwd_tile(NS, NW), Np = NS * NW;
  static constexpr int per = TT / NW;                 // channel-tokens a thread
  static constexpr int PV = per < 4 ? per : 4, NI = per / PV;
  static constexpr int NV = kScanCh / PV;             // threads of a token row
  static constexpr int NR = TT / NI;                  // such rows
};

// What a thread computes of its tokens before the recurrence.
template <int NI, int PV> struct BwdTok {
  float s[NI][PV], u[NI][PV], v[NI][PV], dt[NI][PV], dp[NI][PV];
};

template <typename E, int PV, int NI, int WM>
__device__ __forceinline__ void prepare(const ScanArgs &a, const ScanRaw<E, PV, NI, WM> &r,
                                        const RowBits<E, PV> (&dyr)[NI], const E (&w)[WM][kScanCh],
                                        const float (&par)[3][kScanCh], int v0, int t, int t1, bool full, bool want_dp,
                                        BwdTok<NI, PV> &o) {
  float cb[PV], dtb[PV];
  ld_lds<PV>(&par[0][v0], cb);
  ld_lds<PV>(&par[1][v0], dtb);
  conv_tile<E, PV, NI, WM, kScanCh>(r, a.W, a.pos != nullptr, w, v0, cb, o.s);
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < PV; ++j) o.u[i][j] = o.s[i][j];
  if (a.act) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < PV; ++j) o.u[i][j] = silu_f(o.s[i][j]);
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float x0[PV];
      unpack_row<E, PV>(r.x[i + WM - 1], x0);
#pragma unroll
      for (int j = 0; j < PV; ++j) o.u[i][j] += x0[j];
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float dl[PV];
    unpack_row<E, PV>(r.dl[i], dl);
#pragma unroll
    for (int j = 0; j < PV; ++j) {
      o.v[i][j] = dl[j] + dtb[j];
      o.dt[i][j] = softplus_f(o.v[i][j]);
    }
    if (want_dp) {
      unpack_row<E, PV>(dyr[i], o.dp[i]);
      if (a.z) {
        float z[PV];
        unpack_row<E, PV>(r.z[i], z);
#pragma unroll
        for (int j = 0; j < PV; ++j) o.dp[i][j] *= silu_f(z[j]);
      }
    }
    if (!full) {  // a token past the end changes nothing
      const bool in = t + i < t1;
#pragma unroll
      for (int j = 0; j < PV; ++j) {
        o.dt[i][j] = in ? o.dt[i][j] : 0.0f;
        o.dp[i][j] = in ? o.dp[i][j] : 0.0f;
        o.u[i][j] = in ? o.u[i][j] : 0.0f;
      }
    }
  }
}

// The convolution's and the step's bias and Dk of the block's channels, in LDS:
// in registers all the while they would cost a wave of occupancy.
template <typename E>
__device__ __forceinline__ void ld_params(const ScanArgs &a, int c0, int nch, int threads,
                                          float (&par)[3][kScanCh]) {
  for (int i = threadIdx.x; i < kScanCh; i += threads) {
    const bool on = i < nch;
    par[0][i] = on && a.cb ? to_f32<E>(((const E *)a.cb)[c0 + i]) : 0.0f;
    par[1][i] = on && a.dtb ? a.dtb[c0 + i] : 0.0f;
    par[2][i] = on && a.Dk ? a.Dk[c0 + i] : 0.0f;
  }
}

template <typename E, int PV, int NI>
__device__ __forceinline__ void ld_dy(const ScanArgs &a, int b, int t, int r0, int t1, int c0,
                                      const ScanOff &off, RowBits<E, PV> (&o)[NI]) {
  const E *p = (const E *)a.dy + ((int64_t)b * a.T + t) * a.D + c0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    o[i] = zero_row<E, PV>();
    if (t + r0 + i < t1) o[i] = ld_at<E, PV>(p + i * a.D, off.d);
  }
}

// Sums of eight registers over the wave's lanes; lane l returns that of
// register l / 8.  Each exchange halves the registers: lanes 0-31 keep one of a
// pair and lanes 32-63 the other, then the rows of 16, then the halves of a row.
__device__ __forceinline__ float sum8(const float *v, bool upper) {
  float r[4], s[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = add_swap32(v[i], v[i + 4]);
#pragma unroll
  for (int i = 0; i < 2; ++i) s[i] = add_swap16(r[i], r[i + 2]);
  // upper: the lane lies in the upper half of its row of 16
  float t = (upper ? s[1] : s[0]) + dpp<0x128>(upper ? s[0] : s[1]);  // row_ror:8
  t += dpp<0xb1>(t);   // quad_perm 1,0,3,2
  t += dpp<0x4e>(t);   // quad_perm 2,3,0,1
  t += dpp<0x141>(t);  // row_half_mirror
  return t;
}

// The tile's tokens that start a document.
__device__ __forceinline__ uint32_t tile_starts(const ScanArgs &a, int b, int t, int t1, int TT,
                                                int lane) {
  const int tt = t + lane;
  return (uint32_t)__ballot(lane < TT && tt < t1 && a.pos[(int64_t)b * a.T + min(tt, t1 - 1)] == 0);
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------
template <typename E, int NS, int NW, int WM, bool PACKED, bool CUT>
__global__ __launch_bounds__(64 * NW) void scan_bwd_sums_kernel(ScanBwdP p) {
  typedef BwdGeo<NS, NW> Geo;
  constexpr int TT = Geo::TT, Np = Geo::Np, PV = Geo::PV, NI = Geo::NI;
  constexpr int GT = 2, BR = 2 * NS * NW;
  __shared__ __align__(16) E s_w[WM][kScanCh];
  __shared__ __align__(16) float s_par[3][kScanCh];
  __shared__ __align__(16) float s_dt[TT][kScanCh], s_du[TT][kScanCh];
  __shared__ __align__(16) float s_dp[CUT ? TT : 1][kScanCh];
  __shared__ __align__(16) float s_bc[TT * BR];
  const ScanArgs &a = p.a;
  const ScanWhere at = scan_where(blockIdx.x + p.first, a.G, p.dg, p.nblk, p.nc);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = at.chunk * p.tc, t1 = min((int)a.T, t0 + p.tc);
  const int n0 = wave * NS, have = a.N - n0;
  const bool mine = lane < at.nch;
  const int64_t c = at.c0 + (mine ? lane : 0);
  const bool want_z = CUT && a.z != nullptr;
  ld_filter<E, WM, kScanCh>(a, at.c0, at.nch, 64 * NW, s_w);
  ld_params<E>(a, at.c0, at.nch, 64 * NW, s_par);
  float A2[NS], h[NS], pr[NS], qe[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    A2[j] = mine && j < have ? a.A[c * a.N + n0 + j] * kLog2e : 0.0f;
    h[j] = qe[j] = 0.0f;
    pr[j] = 1.0f;
  }
  float cum = 0.0f;
  bool fresh = false;
  const int v0 = (int)threadIdx.x % Geo::NV * PV, r0 = (int)threadIdx.x / Geo::NV * NI;
  const bool prep = r0 < TT && v0 < at.nch;
  ScanRaw<E, PV, NI, WM> raw;
  RowBits<E, PV> dyr[NI];
  BcRaw<E, NS, NW, TT> bcr;
  const ScanOff off = scan_off(a, r0, v0);
  if (prep) {
    ld_tile<E, PV, NI, WM, TT>(a, at.b, t0, r0, t1, at.c0, v0, off, want_z, raw);
    if constexpr (CUT) ld_dy<E, PV, NI>(a, at.b, t0, r0, t1, at.c0, off, dyr);
  }
  ld_bc<E, NS, NW, TT>(a, at.b, at.g, t0, t1, bcr);
  // channels that the block does not have stay zero
  for (int i = threadIdx.x; i < TT * kScanCh; i += 64 * NW) {
    (&s_dt[0][0])[i] = (&s_du[0][0])[i] = 0.0f;
    if constexpr (CUT) (&s_dp[0][0])[i] = 0.0f;
  }
  __syncthreads();
  for (int tv = t0; tv < t1; tv += TT) {
    const int t = __builtin_amdgcn_readfirstlane(tv);
    if (prep) {
      BwdTok<NI, PV> k;
      prepare<E, PV, NI, WM>(a, raw, dyr, s_w, s_par, v0, t + r0, t1, t + TT <= t1, CUT, k);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float du[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) du[j] = k.dt[i][j] * k.u[i][j];
        st_lds<PV>(&s_dt[r0 + i][v0], k.dt[i]);
        st_lds<PV>(&s_du[r0 + i][v0], du);
        if constexpr (CUT) st_lds<PV>(&s_dp[r0 + i][v0], k.dp[i]);
      }
    }
    st_bc<E, NS, NW, TT>(bcr, s_bc);
    if (t + TT < t1) {
      ld_bc<E, NS, NW, TT>(a, at.b, at.g, t + TT, t1, bcr);
      if (prep) {
        ld_tile<E, PV, NI, WM, TT>(a, at.b, t + TT, r0, t1, at.c0, v0, off, want_z, raw);
        if constexpr (CUT) ld_dy<E, PV, NI>(a, at.b, t + TT, r0, t1, at.c0, off, dyr);
      }
    }
    uint32_t starts = 0;
    if constexpr (PACKED) starts = tile_starts(a, at.b, t, t1, TT, lane);
    // the tile's start, as reached from a zero state at the chunk's start
    const int64_t row = ((int64_t)at.b * p.tiles + t / TT) * a.D + c;
    if (mine) {
      st_lds<NS>(p.ws.ck + row * Np + n0, h);
      if (wave == 0) p.ws.cum[row] = fresh ? -1.0f : cum;
    }
    __syncthreads();
    if (have > 0) {
      struct Group {
        float bc[GT][CUT ? 2 * NS : NS], dt[GT], du[GT], dp[GT];
      } gr[2];
      auto load = [&](int g0, Group &g) {
#pragma unroll
        for (int i = 0; i < GT; ++i) {
          ld_lds<CUT ? 2 * NS : NS>(s_bc + (g0 + i) * BR + wave * 2 * NS, g.bc[i]);
          g.dt[i] = s_dt[g0 + i][lane];
          g.du[i] = s_du[g0 + i][lane];
          g.dp[i] = CUT ? s_dp[CUT ? g0 + i : 0][lane] : 0.0f;
        }
      };
      // the tile's tokens before the chunk's first start of a document
      const int first = fresh ? 0 : starts ? __builtin_ctz(starts) : TT;
      fresh |= starts != 0;
      auto walk = [&](int g0, const Group &g) {
#pragma unroll
        for (int i = 0; i < GT; ++i) {
          const bool start = PACKED && (starts >> (g0 + i) & 1);
          // nothing of a document that starts in the chunk goes to the tokens
          // before the chunk: left out, since its values may be infinite
          const bool before = !PACKED || g0 + i < first;
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            const float e = __builtin_amdgcn_exp2f(g.dt[i] * A2[j]);
            h[j] = fmaf(e, start ? 0.0f : h[j], g.du[i] * g.bc[i][j]);
            if constexpr (CUT) {
              pr[j] *= e;
              const float more = fmaf(pr[j], g.dp[i] * g.bc[i][CUT ? NS + j : 0], qe[j]);
              qe[j] = before ? more : qe[j];
            }
          }
          cum += g.dt[i];
        }
      };
      load(0, gr[0]);
#pragma unroll 1
      for (int g0 = 0; g0 < TT; g0 += 2 * GT) {
        load(g0 + GT, gr[1]);
        walk(g0, gr[0]);
        if (g0 + 2 * GT < TT) load(g0 + 2 * GT, gr[0]);
        walk(g0 + GT, gr[1]);
      }
    }
    __syncthreads();
  }
  if constexpr (CUT) {
    if (mine) {
      const int64_t row = ((int64_t)at.b * p.nc + at.chunk) * a.D + c;
      st_lds<NS>(p.ws.hend + row * Np + n0, h);
      st_lds<NS>(p.ws.qend + row * Np + n0, qe);
      if (wave == 0) p.ws.sdt[row] = fresh ? -1.0f : cum;
    }
  }
}

// ---------------------------------------------------------------------------
// main
// ---------------------------------------------------------------------------
// Two workgroups of four waves a CU, that is 256 registers a wave: 8 x 2048 x
// 1536, N = 16, fp32 takes 684 us so and 932 us with one workgroup, bf16 with
// eight taps 733 and 1031 us.  fp32 with eight taps does not fit: 1110 us with
// the rest in memory, 1052 us with one workgroup.
constexpr int scan_bwd_occupancy(int esize, int nw, int wm) {
  return nw == 4 ? scan_bwd_resident(esize == 2, nw, wm) : 1;
}
// Those that fit only without the addresses and values that can be had again
// where they are used.  The compiler would put 60 to 100 bytes a lane into memory
// instead: 711 and 768 us for the two above.  bf16 with four taps has room for
// all: 1272 us at 8 x 4096 x 1536, 1301 us without them.
constexpr bool scan_bwd_tight(int esize, int nw, int wm) {
  return scan_bwd_occupancy(esize, nw, wm) == 2 && (esize == 4 || wm > 4);
}

// v, where tight as a value that the compiler does not know to be the same in
// every tile: it forms the addresses that depend on it where they are used,
// instead of keeping them in registers (two an address) through the recurrences.
template <bool TIGHT> __device__ __forceinline__ int in_loop(int v) {
  if constexpr (TIGHT) asm volatile("" : "+v"(v));
  return v;
}

// RAGGED: N is not a multiple of NS.  The states past N then stay zero, which dt u
// or dp times their zero B or C do not where they are infinite.  In the same kernel
// the selects for that would cost a whole N 1 %: 8 x 4096 x 1536, N = 16, bf16.
template <typename E, int NS, int NW, int WM, bool PACKED, bool RAGGED>
__global__ __launch_bounds__(64 * NW)
    __attribute__((amdgpu_waves_per_eu(scan_bwd_occupancy(sizeof(E), NW, WM))))
    void scan_bwd_kernel(ScanBwdP p) {
  typedef BwdGeo<NS, NW> Geo;
  constexpr int TT = Geo::TT, Np = Geo::Np, PV = Geo::PV, NI = Geo::NI;
  constexpr int NV = Geo::NV, NR = Geo::NR, BR = 2 * NS * NW;
  constexpr int HALO = kScanMaxW - 1, KA = 3 + WM;
  constexpr bool TIGHT = scan_bwd_tight(sizeof(E), NW, WM);
  __shared__ __align__(16) E s_w[WM][kScanCh];
  __shared__ __align__(16) float s_par[3][kScanCh];
  __shared__ __align__(16) float s_dt[TT][kScanCh], s_du[TT][kScanCh], s_dp[TT][kScanCh];
  // the waves' parts of sum C h, of e and of S; at the end, the threads' sums
  __shared__ __align__(16) float s_part[3][NW][TT][kScanCh];
  // ds of the tile and of the tile after it, by turns
  __shared__ __align__(16) float s_ds[2][TT][kScanCh];
  // rows four values apart from a multiple of the banks
  constexpr int DB = 2 * Np + 4;
  __shared__ float s_dbc[TT][DB];
  __shared__ __align__(16) float s_bc[TT * BR];
  static_assert(TT > HALO && TT % 8 == 0, "the rows after a tile lie in one tile");
  const ScanArgs &a = p.a;
  const ScanWhere at = scan_where(blockIdx.x + p.first, a.G, p.dg, p.nblk, p.nc);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int T = (int)a.T;
  const int t0 = at.chunk * p.tc, t1 = min(T, t0 + p.tc);
  const int n0 = wave * NS, have = a.N - n0;
  const bool mine = lane < at.nch, upper = (lane & 8) != 0;
  const int64_t c = at.c0 + (mine ? lane : 0);
  const bool gate = a.z != nullptr;
  ld_filter<E, WM, kScanCh>(a, at.c0, at.nch, 64 * NW, s_w);
  ld_params<E>(a, at.c0, at.nch, 64 * NW, s_par);
  float A2[NS], hin[NS], q[NS], dA[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    A2[j] = mine && j < have ? a.A[c * a.N + n0 + j] * kLog2e : 0.0f;
    hin[j] = q[j] = dA[j] = 0.0f;
  }
  if (mine && p.nc > 1) {
    // what enters the chunk from before, and from after it
    auto fold = [&](int k, const float *ends, float (&s)[NS]) {
      const int64_t row = ((int64_t)at.b * p.nc + k) * a.D + c;
      const float sd = p.ws.sdt[row];
      float ev[NS];
      ld_lds<NS>(ends + row * Np + n0, ev);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        s[j] = sd < 0.0f ? ev[j] : fmaf(__builtin_amdgcn_exp2f(A2[j] * sd), s[j], ev[j]);
    };
    for (int k = 0; k < at.chunk; ++k) fold(k, p.ws.hend, hin);
    for (int k = p.nc - 1; k > at.chunk; --k) fold(k, p.ws.qend, q);
  }
  const int v0 = (int)threadIdx.x % NV * PV, r0 = (int)threadIdx.x / NV * NI;
  const bool prep = r0 < TT && v0 < at.nch;
  // sums over the thread's tokens for dDk, ddt_bias, dcb and dw
  float acc[KA][PV];
#pragma unroll
  for (int j = 0; j < PV; ++j) {
#pragma unroll
    for (int k = 0; k < KA; ++k) acc[k][j] = 0.0f;
  }
  // channels that the block does not have, and the rows after the chunk, stay zero
  for (int i = threadIdx.x; i < TT * kScanCh; i += 64 * NW) {
    (&s_dt[0][0])[i] = (&s_du[0][0])[i] = (&s_dp[0][0])[i] = 0.0f;
    (&s_ds[0][0][0])[i] = (&s_ds[1][0][0])[i] = 0.0f;
  }
  for (int i = threadIdx.x; i < TT * DB; i += 64 * NW) (&s_dbc[0][0])[i] = 0.0f;
  if (have <= 0) {
    for (int i = 0; i < TT; ++i)
      s_part[0][wave][i][lane] = s_part[1][wave][i][lane] = s_part[2][wave][i][lane] = 0.0f;
  }
  const int nt = (t1 - t0 + TT - 1) / TT;
  ScanRaw<E, PV, NI, WM> nxt;
  RowBits<E, PV> dyn[NI];
  BcRaw<E, NS, NW, TT> bcr;
  const ScanOff off = scan_off(a, r0, v0);
  float hn[NS], cumn = 0.0f;  // the tile's start as the sums kernel left it
  auto ahead = [&](int t) {
    ld_bc<E, NS, NW, TT>(a, at.b, at.g, t, t1, bcr, in_loop<TIGHT>((int)threadIdx.x));
    const int64_t row = ((int64_t)at.b * p.tiles + t / TT) * a.D + in_loop<TIGHT>((int)c);
    ld_lds<NS>(p.ws.ck + row * Np + n0, hn);
    if (p.nc > 1) cumn = p.ws.cum[row];
    if (prep) {
      const int ro = in_loop<TIGHT>(r0), vo = in_loop<TIGHT>(v0);
      ld_tile<E, PV, NI, WM, TT>(a, at.b, t, ro, t1, at.c0, vo, off, gate, nxt);
      ld_dy<E, PV, NI>(a, at.b, t, ro, t1, at.c0, off, dyn);
    }
  };
  ahead(t0 + (nt - 1) * TT);
  __syncthreads();
  for (int ti = nt - 1; ti >= 0; --ti) {
    const int t = __builtin_amdgcn_readfirstlane(t0 + ti * TT), par = ti & 1;
    BwdTok<NI, PV> k;
    ScanRaw<E, PV, NI, WM> raw;
    RowBits<E, PV> dyr[NI];
    if (prep) {
      raw = nxt;
#pragma unroll
      for (int i = 0; i < NI; ++i) dyr[i] = dyn[i];
      prepare<E, PV, NI, WM>(a, raw, dyr, s_w, s_par, v0, t + r0, t1, t + TT <= t1, true,
                             k);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float du[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) du[j] = k.dt[i][j] * k.u[i][j];
        st_lds<PV>(&s_dt[r0 + i][v0], k.dt[i]);
        st_lds<PV>(&s_du[r0 + i][v0], du);
        st_lds<PV>(&s_dp[r0 + i][v0], k.dp[i]);
      }
    }
    st_bc<E, NS, NW, TT>(bcr, s_bc);
    // the state that enters the tile
    float hs[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      hs[j] = hn[j];
      if (p.nc > 1 && cumn >= 0.0f)
        hs[j] = fmaf(__builtin_amdgcn_exp2f(A2[j] * cumn), hin[j], hs[j]);
    }
    if (ti > 0) ahead(t - TT);
    uint32_t starts = 0;
    if constexpr (PACKED) starts = tile_starts(a, at.b, t, t1, TT, lane);
    __syncthreads();
    if (have > 0) {
      if constexpr (RAGGED) {
#pragma unroll
        for (int j = 0; j < NS; ++j) hs[j] = j < have ? hs[j] : 0.0f;
      }
      // the tile's states, then q through them backwards
      float hist[TT][NS];
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const float dtv = s_dt[i][lane], duv = s_du[i][lane];
        float bc[2 * NS];
        ld_lds<2 * NS>(s_bc + i * BR + wave * 2 * NS, bc);
        const bool start = PACKED && (starts >> i & 1);
        float o = 0.0f;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const float hp = i ? hist[i > 0 ? i - 1 : 0][j] : hs[j];
          hist[i][j] = fmaf(__builtin_amdgcn_exp2f(dtv * A2[j]), start ? 0.0f : hp, duv * bc[j]);
          if constexpr (RAGGED) hist[i][j] = j < have ? hist[i][j] : 0.0f;
          o = fmaf(bc[NS + j], hist[i][j], o);
        }
        s_part[0][wave][i][lane] = o;
        if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
      float tot[NS / 4] = {};
#pragma unroll
      for (int i = TT - 1; i >= 0; --i) {
        const float dtv = s_dt[i][lane], duv = s_du[i][lane], dpv = s_dp[i][lane];
        float bc[2 * NS], sums[2 * NS], e = 0.0f, ss = 0.0f;
        ld_lds<2 * NS>(s_bc + i * BR + wave * 2 * NS, bc);
        const bool start = PACKED && (starts >> i & 1);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const float hp = i ? hist[i > 0 ? i - 1 : 0][j] : hs[j];
          q[j] = fmaf(bc[NS + j], dpv, q[j]);
          if constexpr (RAGGED) q[j] = j < have ? q[j] : 0.0f;
          sums[j] = dpv * hist[i][j];
          sums[NS + j] = q[j] * duv;
          e = fmaf(q[j], bc[j], e);
          const float qa = q[j] * __builtin_amdgcn_exp2f(dtv * A2[j]);
          q[j] = start || (RAGGED && j >= have) ? 0.0f : qa;
          const float r = start ? 0.0f : q[j] * hp;
          dA[j] = fmaf(r, dtv, dA[j]);
          ss = fmaf(r, A2[j], ss);
        }
        // keeps the compiler from moving all of a tile's sums of dA to its
        // end, with every r in a register until then
#pragma unroll
        for (int j = 0; j < NS; ++j) asm volatile("" : "+v"(dA[j]));
        s_part[1][wave][i][lane] = e;
        s_part[2][wave][i][lane] = ss;
        // lane 8 k + (i mod 8) keeps token i's sum k of each eight
#pragma unroll
        for (int m = 0; m < NS / 4; ++m) {
          const float sum = sum8(&sums[8 * m], upper);
          tot[m] = (lane & 7) == (i & 7) ? sum : tot[m];
          if ((i & 7) == 0) {
            // the sums are dC of the wave's states, then dB of them
            const int k = 8 * m + (lane >> 3);
            s_dbc[i + (lane & 7)][(k < NS ? 0 : Np) + n0 + k % NS] = tot[m];
          }
        }
      }
    }
    __syncthreads();
    const int64_t tokn = (int64_t)at.b * T + t;
    // the tile's parts of dC and dB
    {
      const int64_t col = (int64_t)(blockIdx.x + p.first) % (a.G * p.nblk);
      float *o = p.ws.dbc + (col * a.B * T + tokn) * (2 * Np);
      const int n = min(TT, t1 - t) * 2 * Np;
      for (int i = threadIdx.x; i < n; i += 64 * NW) o[i] = s_dbc[i / (2 * Np)][i % (2 * Np)];
    }
    float du[NI][PV], ds[NI][PV];
    if (prep) {
      float dk[PV];
      ld_lds<PV>(&s_par[2][v0], dk);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float sum[3][PV];
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          ld_lds<PV>(&s_part[m][0][r0 + i][v0], sum[m]);
#pragma unroll 4
          for (int wv = 1; wv < NW; ++wv) {
            float o[PV];
            ld_lds<PV>(&s_part[m][wv][r0 + i][v0], o);
#pragma unroll
            for (int j = 0; j < PV; ++j) sum[m][j] += o[j];
          }
        }
        const bool on = t + r0 + i < t1;
        const int64_t n = (tokn + i) * a.D + at.c0;
        if constexpr (TIGHT) {
          ld_lds<PV>(&s_dt[r0 + i][v0], k.dt[i]);
          ld_lds<PV>(&s_dp[r0 + i][v0], k.dp[i]);
        }
        float ddelta[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) {
          // sum[2] holds A log2(e) r
          const float ddt = fmaf(k.u[i][j], sum[1][j], sum[2][j] * 0.6931471805599453f);
          ddelta[j] = on ? ddt * sigmoid_f(k.v[i][j]) : 0.0f;
          du[i][j] = on ? fmaf(k.dt[i][j], sum[1][j], a.Dk ? dk[j] * k.dp[i][j] : 0.0f) : 0.0f;
          ds[i][j] = du[i][j];
        }
        if (a.act && on) {
#pragma unroll
          for (int j = 0; j < PV; ++j) ds[i][j] *= silu_grad_f(k.s[i][j]);
        }
        st_lds<PV>(&s_ds[par][r0 + i][v0], ds[i]);
        if (on) {
          st_at<E, PV>((E *)a.ddelta + n, off.d, ddelta);
          if (gate) {
            float z[PV], dz[PV];
            unpack_row<E, PV>(raw.z[i], z);
            unpack_row<E, PV>(dyr[i], dz);
#pragma unroll
            for (int j = 0; j < PV; ++j)
              dz[j] *= (a.Dk ? fmaf(dk[j], k.u[i][j], sum[0][j]) : sum[0][j]) * silu_grad_f(z[j]);
            st_at<E, PV>((E *)a.dz + n, off.d, dz);
          }
#pragma unroll
          for (int j = 0; j < PV; ++j) {
            acc[0][j] = fmaf(k.dp[i][j], k.u[i][j], acc[0][j]);
            acc[1][j] += ddelta[j];
            acc[2][j] += ds[i][j];
          }
#pragma unroll
          for (int m = 0; m < WM; ++m) {
            if (m < a.W && (m == 0 || !PACKED || m <= raw.pos[i])) {
              float x[PV];
              unpack_row<E, PV>(raw.x[i + WM - 1 - m], x);
#pragma unroll
              for (int j = 0; j < PV; ++j) acc[3 + m][j] = fmaf(ds[i][j], x[j], acc[3 + m][j]);
            }
          }
        }
      }
    }
    __syncthreads();
    // dx[t] = rho du[t] + sum_k w[k] ds[t+k]: the rows after the tile are the
    // first ones of the tile done before it.  At a cut of the axis they belong
    // to another workgroup: the sum so far goes to `tail`, the chunk's first
    // rows of ds to `head`, and a later kernel adds the rest.
    const bool inner = t + TT + WM - 1 <= t1;  // all rows that the tile reads exist
    if (prep) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = r0 + i, tt = t + r;
        if (!inner && tt >= t1) continue;
        float dx[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) dx[j] = a.residual ? du[i][j] : 0.0f;
#pragma unroll
        for (int m = 0; m < WM; ++m) {
          if (m > 0 && (m >= a.W || (!inner && tt + m >= t1))) continue;
          if (PACKED && m > 0 && m > a.pos[tokn + r + m]) continue;
          float w[PV], o[PV];
          unpack_row<E, PV>(ld_row<E, PV>(&s_w[m][v0]), w);
          ld_lds<PV>(r + m < TT ? &s_ds[par][r + m][v0] : &s_ds[par ^ 1][r + m - TT][v0], o);
#pragma unroll
          for (int j = 0; j < PV; ++j) dx[j] = fmaf(w[j], o[j], dx[j]);
        }
        const int from_end = t1 - 1 - tt;
        const int64_t edge = ((int64_t)at.b * p.nc + at.chunk) * HALO;
        const int64_t cv = at.c0 + in_loop<TIGHT>(v0);
        if (t1 < T && from_end < a.W - 1)
          st_row<float, PV>(p.ws.tail + (edge + from_end) * a.D + cv, dx);
        else
          st_at<E, PV>((E *)a.dx + (tokn + i) * a.D + at.c0, off.d, dx);
        if (at.chunk > 0 && tt - t0 < a.W - 1)
          st_row<float, PV>(p.ws.head + (edge + tt - t0) * a.D + cv, ds[i]);
      }
    }
  }

  // the parameters' gradients of this chunk: dA by its waves, the others summed
  // over the threads of a channel, in the rows' order
  const int64_t part = (int64_t)at.b * p.nc + at.chunk;
  if (mine) st_lds<NS>(p.ws.pA + (part * a.D + c) * Np + n0, dA);
  float (*buf)[kScanCh] = &s_part[0][0][0];
#pragma unroll
  for (int m = 0; m < KA; ++m) {
    __syncthreads();
    if (r0 < TT) st_lds<PV>(&buf[r0 / NI][v0], acc[m]);
    __syncthreads();
    if (wave == 0 && mine) {
      float v = 0.0f;
      for (int i = 0; i < NR; ++i) v += buf[i][lane];
      p.ws.pV[(part * kScanParV + m) * a.D + c] = v;
    }
  }
}

template <typename E, int NS, int NW, int WM, bool PACKED>
static hipError_t scan_bwd_run(const ScanBwdP &p, int64_t groups) {
  hipStream_t s = (hipStream_t)p.a.stream;
  constexpr int TH = 64 * NW;
  ScanBwdP q = p;
  const hipError_t e = launch_slices(groups, TH, [&](uint32_t first, dim3 grid) {
    q.first = first;
    if (p.nc > 1)
      hipLaunchKernelGGL((scan_bwd_sums_kernel<E, NS, NW, WM, PACKED, true>), grid, dim3(TH), 0,
                         s, q);
    else
      hipLaunchKernelGGL((scan_bwd_sums_kernel<E, NS, NW, WM, PACKED, false>), grid, dim3(TH), 0,
                         s, q);
  });
  if (e != hipSuccess) return e;
  return launch_slices(groups, TH, [&](uint32_t first, dim3 grid) {
    q.first = first;
    if (p.a.N % NS)
      hipLaunchKernelGGL((scan_bwd_kernel<E, NS, NW, WM, PACKED, true>), grid, dim3(TH), 0, s, q);
    else
      hipLaunchKernelGGL((scan_bwd_kernel<E, NS, NW, WM, PACKED, false>), grid, dim3(TH), 0, s, q);
  });
}

template <typename E, int NS, int NW> hipError_t scan_bwd_nw(const ScanBwdP &p, int64_t groups) {
  if (p.a.W <= 4)
    return p.a.pos ? scan_bwd_run<E, NS, NW, 4, true>(p, groups)
                   : scan_bwd_run<E, NS, NW, 4, false>(p, groups);
  return p.a.pos ? scan_bwd_run<E, NS, NW, 8, true>(p, groups)
                 : scan_bwd_run<E, NS, NW, 8, false>(p, groups);
}

}  // namespace dsc
