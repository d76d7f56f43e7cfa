// scan_device.hpp -- device helpers of the selective-scan kernels.
#pragma once

#include "dsc_device.hpp"
#include "grid_slices.hpp"
#include "scan_launch.hpp"

namespace dsc {

constexpr float kLog2e = 1.4426950408889634f;

// log(1 + e^v) = max(v, 0) + log1p(e^-|v|), the logarithm as
// 2 atanh(s), s = e / (2 + e) <= 1/3: atanh(s) / s as a polynomial in s^2,
// fitted on [0, 1/9] for the smallest relative error (8e-9).  The result keeps
// single precision's relative error also where it is small.
__device__ __forceinline__ float softplus_f(float v) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
  const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
  const float q = s * s;
  float r = fmaf(q, 0.1408916711807251f, 0.13980300724506378f);
  r = fmaf(q, r, 0.20012454688549042f);
  r = fmaf(q, r, 0.3333315849304199f);
  r = fmaf(q, r, 1.0f);
  return fmaf(2.0f * s, r, fmaxf(v, 0.0f));
}

// Kernel parameters: ScanArgs with the tiling.
struct ScanP {
  ScanArgs a;
  float *hend, *sdt;
  int dg, nblk, nc, tc;
  uint32_t first;  // the launch's first workgroup among all
};

// Workspace of a backward call, in floats.
struct ScanBwdWs {
  float *ck, *cum;          // tile starts: (B, tiles, D, Np), (B, tiles, D)
  float *hend, *qend, *sdt; // chunks: (B, nc, D, Np) twice, (B, nc, D)
  float *dbc;               // (G nblk, B T, 2 Np): dC then dB of a channel block
  float *pA, *pV;           // (B nc, D, Np), (B nc, kScanParV, D)
  float *tail, *head;       // (B nc, 7, D) twice: see the convolution's seam below
};

// Parameters of the backward kernels.
struct ScanBwdP {
  ScanArgs a;
  ScanBwdWs ws;
  int dg, nblk, nc, tc, tiles;
  uint32_t first;
};

// V consecutive floats of LDS, aligned to their size (16 bytes at most)
template <int V>
__device__ __forceinline__ void ld_lds(const float *p, float (&o)[V]) {
  unpack_row<float, V>(ld_row<float, V>(p), o);
}
template <int V>
__device__ __forceinline__ void st_lds(float *p, const float (&o)[V]) {
  st_row<float, V>(p, o);
}

// Where a workgroup works: sequence b, chunk of the time axis, group g of B and
// C, channels c0 .. c0 + nch - 1.  Channel blocks are numbered fastest, so the
// workgroups in flight cover whole token rows.
struct ScanWhere {
  int b, chunk, g, c0, nch;
};
__device__ __forceinline__ ScanWhere scan_where(unsigned id, int G, int dg, int nblk, int nc,
                                                int ch = kScanCh) {
  ScanWhere w;
  const unsigned per = (unsigned)(G * nblk);
  const unsigned col = id % per;
  id /= per;
  w.chunk = (int)(id % (unsigned)nc);
  w.b = (int)(id / (unsigned)nc);
  w.g = (int)(col / (unsigned)nblk);
  const int blk = (int)(col % (unsigned)nblk);
  w.c0 = w.g * dg + blk * ch;
  w.nch = min(ch, dg - blk * ch);
  return w;
}

// One element of a parameter row stored as E, and one value as stored in E.
template <typename E> __device__ __forceinline__ float to_f32(E v) {
  if constexpr (sizeof(E) == 2) return __uint_as_float((uint32_t)v << 16);
  else return v;
}
template <typename E> __device__ __forceinline__ E to_elem(float v) {
  if constexpr (sizeof(E) == 2) return (E)(pack_bf16x2(v, 0.0f) & 0xffffu);
  else return v;
}
template <typename E> __device__ __forceinline__ void st_elem(E *p, float v) {
  *p = to_elem<E>(v);
}

// A pointer that is the same in every lane, as a scalar address.
__device__ __forceinline__ uint64_t uniform_addr(const void *p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (uint64_t)hi << 32 | lo;
}
// N consecutive values at a lane's offset from a base that is the same for all
// lanes: the base goes into scalar registers, so that the access costs no
// vector instruction for its address.  The bytes of the offset fit 32 bits.
template <int BYTES> struct MemWord;
template <> struct MemWord<2> { typedef uint16_t type; };
template <> struct MemWord<4> { typedef uint32_t type; };
template <> struct MemWord<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct MemWord<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <typename E, int N>
using global_word = typename MemWord<N * (int)sizeof(E)>::type __attribute__((address_space(1)));
template <typename E, int N>
__device__ __forceinline__ global_word<E, N> *word_at(const E *base, uint32_t off) {
  typedef char __attribute__((address_space(1))) gchar;
  gchar *p = (gchar *)(uintptr_t)uniform_addr(base);
  return (global_word<E, N> *)(p + off * (uint32_t)sizeof(E));
}
template <typename E, int N>
__device__ __forceinline__ RowBits<E, N> ld_at(const E *base, uint32_t off) {
  RowBits<E, N> r;
  const auto v = *word_at<E, N>(base, off);
  constexpr int bytes = N * (int)sizeof(E);
  if constexpr (bytes <= 4) {
    r.d[0] = v;
  } else {
#pragma unroll
    for (int i = 0; i < bytes / 4; ++i) r.d[i] = v[i];
  }
  return r;
}
template <typename E, int N>
__device__ __forceinline__ void st_at(E *base, uint32_t off, const float (&o)[N]) {
  constexpr int bytes = N * (int)sizeof(E);
  uint32_t d[(bytes + 3) / 4];
#pragma unroll
  for (int i = 0; i < (bytes + 3) / 4; ++i) {
    if constexpr (sizeof(E) == 4) d[i] = __float_as_uint(o[i]);
    else d[i] = pack_bf16x2(o[2 * i], 2 * i + 1 < N ? o[2 * i + 1 < N ? 2 * i + 1 : 0] : 0.0f);
  }
  typename MemWord<bytes>::type v;
  if constexpr (bytes <= 4) {
    v = (typename MemWord<bytes>::type)d[0];
  } else {
#pragma unroll
    for (int i = 0; i < bytes / 4; ++i) v[i] = d[i];
  }
  *word_at<E, N>(base, off) = v;
}

// ---- B and C of a tile ------------------------------------------------------
// In LDS as fp32: [token][group] runs of 2 NS, the B of a group's NS states, then
// their C; tokens past the end are zero.  States past N are zero, too, or with
// COPY further copies of the first ones, among which a state's C is shared out.
// The lanes of a group
// (in the backward a whole wave) read the same run, a broadcast, in order with
// their other LDS reads.  Scalar loads
// from memory were measured instead: unpacking and addressing took as many
// issue slots as the arithmetic, and with an fp32 copy made beforehand their
// waits (a scalar load's is for all in flight) cost what that saved.
// Each of TH threads loads QN consecutive values of B or of C of one token.
template <int NS, int NW, int TT, int TH> struct BcGeo {
  static constexpr int row = 2 * NS * NW;                   // floats of a token
  static constexpr int n = TT * row / TH;                   // values a thread
  static constexpr int QN = n < NS ? n : NS;                // in runs of QN ...
  static constexpr int NQ = n / QN;                         // ... NQ of them
  static_assert(n * TH == TT * row && NQ * QN == n && NS % QN == 0, "whole runs");
};

template <typename E, int NS, int NW, int TT, int TH = 64 * NW> struct BcRaw {
  RowBits<E, BcGeo<NS, NW, TT, TH>::QN> q[BcGeo<NS, NW, TT, TH>::NQ];
};

// Where run k of thread tid goes: token, B or C, first state, place in LDS.
template <int NS, int NW, int TT, int TH>
__device__ __forceinline__ void bc_at(int tid, int k, int &row, int &which, int &n0, int &at) {
  typedef BcGeo<NS, NW, TT, TH> G;
  at = (tid + k * TH) * G::QN;
  row = at / G::row;
  const int r = at % G::row, group = r / (2 * NS), i = r % (2 * NS);
  which = i / NS;
  n0 = group * NS + i % NS;
}

// The state that place n < Np stands for, where places past N hold copies: Np is
// below 2 N, or four (N = 1), so a state has one, two or four places.
__device__ __forceinline__ int copy_of(int n, int N) { return n < N ? n : n % N; }

template <typename E, int NS, int NW, int TT, int TH = 64 * NW, bool COPY = false>
__device__ __forceinline__ void ld_bc(const ScanArgs &a, int b, int g, int t, int t1,
                                      BcRaw<E, NS, NW, TT, TH> &o, int tid = (int)threadIdx.x) {
  typedef BcGeo<NS, NW, TT, TH> G;
#pragma unroll
  for (int k = 0; k < G::NQ; ++k) {
    auto &r = o.q[k];
#pragma unroll
    for (int i = 0; i < RowBits<E, G::QN>::dwords; ++i) r.d[i] = 0u;
    int row, which, n0, at;
    bc_at<NS, NW, TT, TH>(tid, k, row, which, n0, at);
    if (t + row >= t1) continue;
    if constexpr (COPY) {
      // a run of four states with N a multiple of four: all its own, or all copies
      if (a.bc_vec && n0 >= a.N) n0 -= a.N;
    } else if (n0 >= a.N) {
      continue;
    }
    const int64_t tok = (int64_t)b * a.T + t + row;
    const E *p = (which ? (const E *)a.Cm + tok * a.c_row : (const E *)a.Bm + tok * a.b_row) +
                 g * a.N;
    if (a.bc_vec) {
      r = ld_row<E, G::QN>(p + n0);
    } else {
#pragma unroll
      for (int j = 0; j < G::QN; ++j)
        if (COPY || n0 + j < a.N) {
          const E v = p[COPY ? copy_of(n0 + j, a.N) : n0 + j];
          if constexpr (sizeof(E) == 2) r.d[j >> 1] |= (uint32_t)v << (16 * (j & 1));
          else r.d[j] = __float_as_uint(v);
        }
    }
  }
}

template <typename E, int NS, int NW, int TT, int TH = 64 * NW, bool COPY = false>
__device__ __forceinline__ void st_bc(const BcRaw<E, NS, NW, TT, TH> &o, float *s_bc, int N = 0) {
  typedef BcGeo<NS, NW, TT, TH> G;
#pragma unroll
  for (int k = 0; k < G::NQ; ++k) {
    int row, which, n0, at;
    bc_at<NS, NW, TT, TH>((int)threadIdx.x, k, row, which, n0, at);
    float v[G::QN];
    unpack_row<E, G::QN>(o.q[k], v);
    if constexpr (COPY) {
      if (N < NS * NW && which) {
        const float part = N == 1 ? 0.25f : 0.5f;  // exact
#pragma unroll
        for (int j = 0; j < G::QN; ++j)
          if (n0 + j >= N || n0 + j + N < NS * NW) v[j] *= part;
      }
    }
    st_row<float, G::QN>(s_bc + at, v);
  }
}

// ---- the convolution's taps ---------------------------------------------------
// In LDS, in the type they are stored in; without a convolution (W == 0) tap 0
// is one, which leaves x as it is.
template <typename E, int WM, int CB>
__device__ __forceinline__ void ld_filter(const ScanArgs &a, int c0, int nch, int threads,
                                          E (&par)[WM][CB]) {
  const E *w = (const E *)a.w;
  for (int i = threadIdx.x; i < WM * CB; i += threads) {
    const int k = i / CB, ch = i % CB;
    E v{};
    if (a.W == 0) v = to_elem<E>(k == 0 ? 1.0f : 0.0f);
    else if (ch < nch && k < a.W) v = w[(int64_t)(c0 + ch) * a.W + k];
    par[k][ch] = v;
  }
}

// ---- preparation of a tile -------------------------------------------------
// A thread takes NI consecutive tokens of PV consecutive channels.  Raw holds
// what it loads for one tile: the tokens' x with the WM - 1 rows before them,
// the step inputs, the gates and, on packed rows, the positions.
template <typename E, int PV, int NI, int WM> struct ScanRaw {
  RowBits<E, PV> x[NI + WM - 1], dl[NI], z[NI];
  int pos[NI];
};

template <typename E, int PV> __device__ __forceinline__ RowBits<E, PV> zero_row() {
  RowBits<E, PV> r;
#pragma unroll
  for (int i = 0; i < RowBits<E, PV>::dwords; ++i) r.d[i] = 0u;
  return r;
}

// Row t of x; rows before the sequence lie in conv0 or are zero.
template <typename E, int PV>
__device__ __forceinline__ RowBits<E, PV> ld_x(const ScanArgs &a, int b, int t, int64_t c) {
  if (t >= 0) return ld_row<E, PV>((const E *)a.x + ((int64_t)b * a.T + t) * a.x_row + c);
  const int j = t + a.W - 1;
  if (a.conv0 && j >= 0)
    return ld_row<E, PV>((const E *)a.conv0 + ((int64_t)b * (a.W - 1) + j) * a.D + c);
  return zero_row<E, PV>();
}

// A thread's offsets from a tile's first row, in elements, one a row distance.
struct ScanOff {
  uint32_t x, dl, z, d;  // d: dense rows of D
};
__device__ __forceinline__ ScanOff scan_off(const ScanArgs &a, int r0, int v0) {
  return ScanOff{(uint32_t)r0 * (uint32_t)a.x_row + v0, (uint32_t)r0 * (uint32_t)a.delta_row + v0,
                 (uint32_t)r0 * (uint32_t)a.z_row + v0, (uint32_t)r0 * (uint32_t)a.D + v0};
}

// Tokens t + r0 .. t + r0 + NI - 1 of the tile at t, channels c0 + v0 on; those
// from t1 on are not loaded.
template <typename E, int PV, int NI, int WM, int TT>
__device__ __forceinline__ void ld_tile(const ScanArgs &a, int b, int t, int r0, int t1, int c0,
                                        int v0, const ScanOff &off, bool want_z,
                                        ScanRaw<E, PV, NI, WM> &r) {
  if (t >= WM - 1 && t + TT <= t1) {  // every row exists
    const int64_t n = (int64_t)b * a.T + t;
    const E *xp = (const E *)a.x + (n - (WM - 1)) * a.x_row + c0;
    const E *dp = (const E *)a.delta + n * a.delta_row + c0;
#pragma unroll
    for (int i = 0; i < NI + WM - 1; ++i) r.x[i] = ld_at<E, PV>(xp + i * a.x_row, off.x);
#pragma unroll
    for (int i = 0; i < NI; ++i) r.dl[i] = ld_at<E, PV>(dp + i * a.delta_row, off.dl);
    if (want_z) {
      const E *zp = (const E *)a.z + n * a.z_row + c0;
#pragma unroll
      for (int i = 0; i < NI; ++i) r.z[i] = ld_at<E, PV>(zp + i * a.z_row, off.z);
    }
  } else {
    const int64_t n0 = (int64_t)b * a.T + t + r0, c = c0 + v0;
#pragma unroll
    for (int i = 0; i < NI + WM - 1; ++i) {
      const int tt = t + r0 + i - (WM - 1);
      r.x[i] = tt < t1 ? ld_x<E, PV>(a, b, tt, c) : zero_row<E, PV>();
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      r.dl[i] = r.z[i] = zero_row<E, PV>();
      if (t + r0 + i < t1) {
        r.dl[i] = ld_row<E, PV>((const E *)a.delta + (n0 + i) * a.delta_row + c);
        if (want_z) r.z[i] = ld_row<E, PV>((const E *)a.z + (n0 + i) * a.z_row + c);
      }
    }
  }
  if (a.pos) {
    const int64_t n0 = (int64_t)b * a.T + t + r0;
#pragma unroll
    for (int i = 0; i < NI; ++i) r.pos[i] = t + r0 + i < t1 ? a.pos[n0 + i] : WM;
  }
}

// The convolution of the thread's tokens before its activation, for the
// thread's channels at column v0 of the block.  A tap that the filter does not
// have, or that would reach into another document, is dropped, not multiplied
// by zero: the value there may be infinite.
template <typename E, int PV, int NI, int WM, int CB>
__device__ __forceinline__ void conv_tile(const ScanRaw<E, PV, NI, WM> &r, int W, bool packed,
                                          const E (&par)[WM][CB], int v0,
                                          const float (&cb)[PV], float (&s)[NI][PV]) {
  float x[NI + WM - 1][PV];
#pragma unroll
  for (int i = 0; i < NI + WM - 1; ++i) unpack_row<E, PV>(r.x[i], x[i]);
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < PV; ++j) s[i][j] = cb[j];
  auto tap = [&](int k, bool drop) {
    float w[PV];
    unpack_row<E, PV>(ld_row<E, PV>(&par[k][v0]), w);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool out = drop && k > r.pos[i];
#pragma unroll
      for (int j = 0; j < PV; ++j)
        s[i][j] = fmaf(w[j], out ? 0.0f : x[i + WM - 1 - k][j], s[i][j]);
    }
  };
  if (!packed && W == WM) {
#pragma unroll
    for (int k = 0; k < WM; ++k) tap(k, false);
  } else {
    tap(0, false);
#pragma unroll
    for (int k = 1; k < WM; ++k)
      if (k < W) tap(k, packed);
  }
}

}  // namespace dsc
