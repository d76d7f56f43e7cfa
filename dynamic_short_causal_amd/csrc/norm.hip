// norm.hip -- layer norm over the last axis, forward and backward, gfx950.
//
//   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),  g = dy w,  xhat = (x - mean) rstd
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// Both directions move their bytes once (x in, y out; x, dy in, dx out) and are
// bound by that.  A row stays in the registers of the threads that read it, so
// the variance is the mean of the centred squares, not a difference of large
// sums.  Rows too long for that are read again from the caches.  Measured:
// forward 16384 x 6144 bf16 69 us, 5.8 TB/s; backward 16384 x 2048 bf16 41 us,
// 4.9 TB/s (37 us and 4 us for the sums of the partials), 999 x 8192 fp32 27 us.
#include "dsc_device.hpp"
#include "grid_slices.hpp"
#include "norm_launch.hpp"

namespace dsc {

constexpr int kLnThreads = 256;

// Sum over the TPR threads of a row (64: one wave; 256: the workgroup, through
// LDS, in the waves' order; `slot` alternates so that one barrier is enough).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[kLnThreads / 64], int slot) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[slot][0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v += red[slot][i];
  }
  return v;
}

template <typename E> __device__ __forceinline__ void ld_vec(const void *p, int64_t c, float none,
                                                             float (&o)[Vw<E>::n]) {
  if (p) {
    unpack<E>(ld16((const E *)p + c), o);
  } else {
#pragma unroll
    for (int i = 0; i < Vw<E>::n; ++i) o[i] = none;
  }
}

// ---------------------------------------------------------------------------
// Forward, VPT vectors of a row a thread, TPR threads a row
// ---------------------------------------------------------------------------
template <typename E, int TPR, int VPT>
__global__ __launch_bounds__(kLnThreads) void ln_fwd_kernel(LnArgs a, uint32_t first) {
  constexpr int V = Vw<E>::n;
  __shared__ float red[2][kLnThreads / 64];
  const int tid = (int)threadIdx.x % TPR;
  const int64_t m = ((int64_t)blockIdx.x + first) * (kLnThreads / TPR) + threadIdx.x / TPR;
  if (TPR == 64 && m >= a.M) return;  // whole waves; a workgroup's single row always exists
  const int nvec = (int)(a.D / V);
  const E *x = (const E *)a.x + m * a.D;
  uint4 r[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * TPR;
    r[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < nvec) r[i] = ld16nt(x + (int64_t)v * V);
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float f[V], q = 0.0f;
    unpack<E>(r[i], f);
#pragma unroll
    for (int j = 0; j < V; ++j) q += f[j];
    s += q;
  }
  const float mean = row_sum<TPR>(s, red, 0) / (float)a.D;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (tid + i * TPR < nvec) {
      float f[V], q = 0.0f;
      unpack<E>(r[i], f);
#pragma unroll
      for (int j = 0; j < V; ++j) q = fmaf(f[j] - mean, f[j] - mean, q);
      s += q;
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, red, 1) / (float)a.D + a.eps);
  E *y = (E *)a.y + m * a.D;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * TPR;
    if (v < nvec) {
      float f[V], w[V], b[V];
      unpack<E>(r[i], f);
      ld_vec<E>(a.w, (int64_t)v * V, 1.0f, w);
      ld_vec<E>(a.b, (int64_t)v * V, 0.0f, b);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = fmaf((f[j] - mean) * rstd, w[j], b[j]);
      st16nt(y + (int64_t)v * V, pack<E>(f));
    }
  }
  if (tid == 0) {
    a.mean[m] = mean;
    a.rstd[m] = rstd;
  }
}

// Rows longer than the registers: one workgroup a row, three readings.
template <typename E>
__global__ __launch_bounds__(kLnThreads) void ln_fwd_long_kernel(LnArgs a) {
  constexpr int V = Vw<E>::n;
  __shared__ float red[2][kLnThreads / 64];
  const int64_t m = blockIdx.x, nvec = a.D / V;
  const E *x = (const E *)a.x + m * a.D;
  E *y = (E *)a.y + m * a.D;
  float s = 0.0f;
  for (int64_t v = threadIdx.x; v < nvec; v += kLnThreads) {
    float f[V], q = 0.0f;
    unpack<E>(ld16(x + v * V), f);
#pragma unroll
    for (int j = 0; j < V; ++j) q += f[j];
    s += q;
  }
  const float mean = row_sum<kLnThreads>(s, red, 0) / (float)a.D;
  s = 0.0f;
  for (int64_t v = threadIdx.x; v < nvec; v += kLnThreads) {
    float f[V], q = 0.0f;
    unpack<E>(ld16(x + v * V), f);
#pragma unroll
    for (int j = 0; j < V; ++j) q = fmaf(f[j] - mean, f[j] - mean, q);
    s += q;
  }
  const float rstd = 1.0f / sqrtf(row_sum<kLnThreads>(s, red, 1) / (float)a.D + a.eps);
  for (int64_t v = threadIdx.x; v < nvec; v += kLnThreads) {
    float f[V], w[V], b[V];
    unpack<E>(ld16(x + v * V), f);
    ld_vec<E>(a.w, v * V, 1.0f, w);
    ld_vec<E>(a.b, v * V, 0.0f, b);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = fmaf((f[j] - mean) * rstd, w[j], b[j]);
    st16(y + v * V, pack<E>(f));
  }
  if (threadIdx.x == 0) {
    a.mean[m] = mean;
    a.rstd[m] = rstd;
  }
}

// ---------------------------------------------------------------------------
// Backward, long rows.  A workgroup of TH threads takes rows blockIdx.x, + gridDim.x, ...;
// a thread keeps the same VPT vectors of every row, so its shares of dw and db
// stay in registers until its last row.  R rows pass at once, one barrier for
// both sums of all of them, and with AHEAD the next rows are loaded meanwhile.
// ---------------------------------------------------------------------------
template <typename E, int TH, int VPT, int R, bool AHEAD>
__global__ __launch_bounds__(TH) void ln_bwd_kernel(LnArgs a) {
  constexpr int V = Vw<E>::n, NWV = TH / 64;
  __shared__ float red[2][2 * R][NWV];
  const int tid = (int)threadIdx.x;
  const int nvec = (int)(a.D / V);
  float dw[VPT][V], db[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) { dw[i][j] = 0.0f; db[i][j] = 0.0f; }
  const int64_t step = gridDim.x;
  int slot = 0;
  uint4 xn[R][VPT], gn[R][VPT];
  float mn[R], rn[R];
  auto load = [&](int64_t m0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t m = m0 + r * step;
      const bool on = m < a.M;
      mn[r] = on ? a.mean_in[m] : 0.0f;
      rn[r] = on ? a.rstd_in[m] : 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * TH;
        xn[r][i] = gn[r][i] = make_uint4(0u, 0u, 0u, 0u);
        if (on && v < nvec) {
          xn[r][i] = ld16nt((const E *)a.x + m * a.D + (int64_t)v * V);
          gn[r][i] = ld16nt((const E *)a.dy + m * a.D + (int64_t)v * V);
        }
      }
    }
  };
  if constexpr (AHEAD) load(blockIdx.x);
  for (int64_t m0 = blockIdx.x; m0 < a.M; m0 += step * R, slot ^= 1) {
    if constexpr (!AHEAD) load(m0);
    uint4 xr[R][VPT], gr[R][VPT];
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = mn[r];
      rstd[r] = rn[r];
#pragma unroll
      for (int i = 0; i < VPT; ++i) { xr[r][i] = xn[r][i]; gr[r][i] = gn[r][i]; }
    }
    if constexpr (AHEAD) load(m0 + step * R);
    float s1[R], s2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) { s1[r] = 0.0f; s2[r] = 0.0f; }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * TH;
      float w[V];
      ld_vec<E>(v < nvec ? a.w : nullptr, (int64_t)v * V, 1.0f, w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x[V], g[V];
        unpack<E>(xr[r][i], x);
        unpack<E>(gr[r][i], g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (x[j] - mean[r]) * rstd[r];
          dw[i][j] = fmaf(g[j], xh, dw[i][j]);
          db[i][j] += g[j];
          const float gw = g[j] * w[j];
          s1[r] += gw;
          s2[r] = fmaf(gw, xh, s2[r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s1[r] = wave_sum(s1[r]);
      s2[r] = wave_sum(s2[r]);
      if ((tid & 63) == 0) {
        red[slot][2 * r][tid >> 6] = s1[r];
        red[slot][2 * r + 1][tid >> 6] = s2[r];
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s1[r] = red[slot][2 * r][0];
      s2[r] = red[slot][2 * r + 1][0];
#pragma unroll
      for (int i = 1; i < NWV; ++i) {
        s1[r] += red[slot][2 * r][i];
        s2[r] += red[slot][2 * r + 1][i];
      }
      s1[r] /= (float)a.D;
      s2[r] /= (float)a.D;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * TH;
      if (v < nvec) {
        float w[V];
        ld_vec<E>(a.w, (int64_t)v * V, 1.0f, w);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int64_t m = m0 + r * step;
          if (m < a.M) {
            float x[V], g[V];
            unpack<E>(xr[r][i], x);
            unpack<E>(gr[r][i], g);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const float xh = (x[j] - mean[r]) * rstd[r];
              x[j] = rstd[r] * (g[j] * w[j] - s1[r] - xh * s2[r]);
            }
            st16nt((E *)a.dx + m * a.D + (int64_t)v * V, pack<E>(x));
          }
        }
      }
    }
  }
  if (a.ws) {
    float *row = a.ws + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * TH;
      if (v < nvec) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          *reinterpret_cast<float4 *>(row + (int64_t)v * V + j) =
              make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
          *reinterpret_cast<float4 *>(row + a.D + (int64_t)v * V + j) =
              make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
        }
      }
    }
  }
}

// Backward, short rows: a wave a row, VPT vectors a lane, so that nothing waits
// for another wave until the workgroup's sums of dw and db are added at the end.
// 16384 x 2048 bf16, side by side when the form was chosen: 45 us, and 54 us with a
// workgroup a row.
template <typename E, int VPT>
__global__ __launch_bounds__(kLnBwdWaves * 64) void ln_bwd_wave_kernel(LnArgs a) {
  constexpr int V = Vw<E>::n;
  __shared__ __align__(16) float red[kLnBwdWaves / 2][2 * VPT * V][64];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int nvec = (int)(a.D / V);
  float w[VPT][V], dw[VPT][V], db[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = lane + i * 64;
    ld_vec<E>(v < nvec ? a.w : nullptr, (int64_t)v * V, 1.0f, w[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) { dw[i][j] = 0.0f; db[i][j] = 0.0f; }
  }
  const int64_t step = (int64_t)gridDim.x * kLnBwdWaves;
  uint4 xn[VPT], gn[VPT];
  float mn, rn;
  auto load = [&](int64_t m) {
    const bool on = m < a.M;
    mn = on ? a.mean_in[m] : 0.0f;
    rn = on ? a.rstd_in[m] : 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = lane + i * 64;
      xn[i] = gn[i] = make_uint4(0u, 0u, 0u, 0u);
      if (on && v < nvec) {
        xn[i] = ld16nt((const E *)a.x + m * a.D + (int64_t)v * V);
        gn[i] = ld16nt((const E *)a.dy + m * a.D + (int64_t)v * V);
      }
    }
  };
  int64_t m = (int64_t)blockIdx.x * kLnBwdWaves + wave;
  load(m);
  for (; m < a.M; m += step) {
    uint4 xr[VPT], gr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) { xr[i] = xn[i]; gr[i] = gn[i]; }
    const float mean = mn, rstd = rn;
    load(m + step);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float x[V], g[V];
      unpack<E>(xr[i], x);
      unpack<E>(gr[i], g);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = (x[j] - mean) * rstd, gw = g[j] * w[i][j];
        dw[i][j] = fmaf(g[j], xh, dw[i][j]);
        db[i][j] += g[j];
        s1 += gw;
        s2 = fmaf(gw, xh, s2);
      }
    }
    s1 = wave_sum(s1) / (float)a.D;
    s2 = wave_sum(s2) / (float)a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = lane + i * 64;
      float x[V], g[V];
      unpack<E>(xr[i], x);
      unpack<E>(gr[i], g);
#pragma unroll
      for (int j = 0; j < V; ++j)
        x[j] = rstd * (g[j] * w[i][j] - s1 - (x[j] - mean) * rstd * s2);
      if (v < nvec) st16nt((E *)a.dx + m * a.D + (int64_t)v * V, pack<E>(x));
    }
  }
  if (!a.ws) return;
  // the waves' sums, halved in number with each round
#pragma unroll
  for (int half = kLnBwdWaves / 2; half > 0; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          red[wave - half][2 * (i * V + j)][lane] = dw[i][j];
          red[wave - half][2 * (i * V + j) + 1][lane] = db[i][j];
        }
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          dw[i][j] += red[wave][2 * (i * V + j)][lane];
          db[i][j] += red[wave][2 * (i * V + j) + 1][lane];
        }
    }
    __syncthreads();
  }
  if (wave == 0) {
    float *row = a.ws + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = lane + i * 64;
      if (v < nvec) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          *reinterpret_cast<float4 *>(row + (int64_t)v * V + j) =
              make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
          *reinterpret_cast<float4 *>(row + a.D + (int64_t)v * V + j) =
              make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
        }
      }
    }
  }
}

// Rows longer than the registers: dx with two readings of a row; dw and db by
// the next kernel.
template <typename E>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_long_kernel(LnArgs a) {
  constexpr int V = Vw<E>::n;
  __shared__ float red[2][kLnThreads / 64];
  const int64_t m = blockIdx.x, nvec = a.D / V;
  const E *x = (const E *)a.x + m * a.D, *dy = (const E *)a.dy + m * a.D;
  const float mean = a.mean_in[m], rstd = a.rstd_in[m];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t v = threadIdx.x; v < nvec; v += kLnThreads) {
    float f[V], g[V], w[V];
    unpack<E>(ld16(x + v * V), f);
    unpack<E>(ld16(dy + v * V), g);
    ld_vec<E>(a.w, v * V, 1.0f, w);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float gw = g[j] * w[j];
      s1 += gw;
      s2 = fmaf(gw, (f[j] - mean) * rstd, s2);
    }
  }
  s1 = row_sum<kLnThreads>(s1, red, 0) / (float)a.D;
  s2 = row_sum<kLnThreads>(s2, red, 1) / (float)a.D;
  for (int64_t v = threadIdx.x; v < nvec; v += kLnThreads) {
    float f[V], g[V], w[V];
    unpack<E>(ld16(x + v * V), f);
    unpack<E>(ld16(dy + v * V), g);
    ld_vec<E>(a.w, v * V, 1.0f, w);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = rstd * (g[j] * w[j] - s1 - (f[j] - mean) * rstd * s2);
    st16((E *)a.dx + m * a.D + v * V, pack<E>(f));
  }
}

// Sums of dw and db of one column vector over rows blockIdx.y, + gridDim.y, ...
template <typename E>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_long_cols_kernel(LnArgs a) {
  constexpr int V = Vw<E>::n;
  const int64_t v = (int64_t)blockIdx.x * kLnThreads + threadIdx.x;
  if (v >= a.D / V) return;
  float dw[V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) { dw[j] = 0.0f; db[j] = 0.0f; }
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    float f[V], g[V];
    unpack<E>(ld16((const E *)a.x + m * a.D + v * V), f);
    unpack<E>(ld16((const E *)a.dy + m * a.D + v * V), g);
    const float mean = a.mean_in[m], rstd = a.rstd_in[m];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      dw[j] = fmaf(g[j], (f[j] - mean) * rstd, dw[j]);
      db[j] += g[j];
    }
  }
  float *row = a.ws + (int64_t)blockIdx.y * 2 * a.D + v * V;
#pragma unroll
  for (int j = 0; j < V; ++j) { row[j] = dw[j]; row[a.D + j] = db[j]; }
}

// dw and db: the sums of the workspace's `parts` rows of 2 D values.  A
// workgroup takes 32 columns; 8 threads of four columns each make a row of it,
// 32 rows at a time, whose sums are added in order at the end.
template <typename E>
__global__ __launch_bounds__(256) void ln_reduce_kernel(LnArgs a, int64_t parts, uint32_t first) {
  __shared__ __align__(16) float red[32][32];
  const int q = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int64_t col = ((int64_t)blockIdx.x + first) * 32 + q * 4, cols = 2 * a.D;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < cols) {
#pragma unroll 8
    for (int64_t p = g; p < parts; p += 32) {
      const float4 v = *reinterpret_cast<const float4 *>(a.ws + p * cols + col);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  *reinterpret_cast<float4 *>(&red[g][q * 4]) = s;
  __syncthreads();
  const int64_t c = ((int64_t)blockIdx.x + first) * 32 + threadIdx.x;
  if (threadIdx.x < 32 && c < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][threadIdx.x];
    E *o = c < a.D ? (E *)a.dw + c : (E *)a.db + (c - a.D);
    if constexpr (sizeof(E) == 2) *o = (E)(pack_bf16x2(t, 0.0f) & 0xffffu);
    else *o = t;
  }
}

// ---------------------------------------------------------------------------
// Host-side launchers
// ---------------------------------------------------------------------------
// A wave a row from this many rows on (four waves a SIMD), if that is at most
// four vectors a lane; otherwise a row gets a whole workgroup, so that few rows
// still use the chip and long ones leave registers for more waves.  Measured,
// wave against workgroup: 16384 x 2048 bf16 27 and 39 us, 65536 x 512 fp32 46
// and 105 us; 16384 x 4096 bf16 50 and 47 us, 16384 x 8192 bf16 106 and 93 us.
constexpr int64_t kLnWaveRows = 4 * 4 * 256;
constexpr int64_t kLnWaveVecs = 4 * 64;

template <typename E, int TPR, int VPT> static hipError_t ln_fwd_go(const LnArgs &a) {
  constexpr int rows = kLnThreads / TPR;
  return launch_slices((a.M + rows - 1) / rows, kLnThreads, [&](uint32_t first, dim3 grid) {
    hipLaunchKernelGGL((ln_fwd_kernel<E, TPR, VPT>), grid, dim3(kLnThreads), 0,
                       (hipStream_t)a.stream, a, first);
  });
}

template <typename E, int TPR> static hipError_t ln_fwd_vpt(const LnArgs &a, int64_t vpt) {
  if (vpt <= 1) return ln_fwd_go<E, TPR, 1>(a);
  if (vpt <= 2) return ln_fwd_go<E, TPR, 2>(a);
  if (vpt <= 3) return ln_fwd_go<E, TPR, 3>(a);
  if constexpr (TPR > 64) {
    if (vpt > 8) return ln_fwd_go<E, TPR, 16>(a);
    if (vpt > 6) return ln_fwd_go<E, TPR, 8>(a);
    if (vpt > 4) return ln_fwd_go<E, TPR, 6>(a);
  }
  return ln_fwd_go<E, TPR, 4>(a);
}

template <typename E> static hipError_t ln_fwd(const LnArgs &a) {
  if (a.M == 0) return hipSuccess;
  const int64_t nvec = a.D / Vw<E>::n;
  if (nvec <= kLnWaveVecs && (a.M >= kLnWaveRows || nvec <= 64))
    return ln_fwd_vpt<E, 64>(a, (nvec + 63) / 64);
  if (nvec <= kLnThreads * 16) return ln_fwd_vpt<E, kLnThreads>(a, (nvec + 255) / 256);
  hipLaunchKernelGGL((ln_fwd_long_kernel<E>), dim3((unsigned)a.M), dim3(kLnThreads), 0,
                     (hipStream_t)a.stream, a);
  return hipGetLastError();
}

template <typename E, int TH, int VPT, int R, bool AHEAD>
static hipError_t ln_bwd_go(const LnArgs &a) {
  hipLaunchKernelGGL((ln_bwd_kernel<E, TH, VPT, R, AHEAD>), dim3((unsigned)ln_bwd_groups(a.M, a.D, a.bf16)),
                     dim3(TH), 0, (hipStream_t)a.stream, a);
  return hipGetLastError();
}

template <typename E, int VPT> static hipError_t ln_bwd_wave_go(const LnArgs &a) {
  hipLaunchKernelGGL((ln_bwd_wave_kernel<E, VPT>),
                     dim3((unsigned)ln_bwd_groups(a.M, a.D, a.bf16)), dim3(kLnBwdWaves * 64), 0,
                     (hipStream_t)a.stream, a);
  return hipGetLastError();
}

template <typename E> static hipError_t ln_bwd(const LnArgs &a) {
  const int64_t nvec = a.D / Vw<E>::n;
  hipError_t e = hipSuccess;
  if (a.M > 0) {
    if (nvec <= 64) e = ln_bwd_wave_go<E, 1>(a);
    else if (nvec <= 128) e = ln_bwd_wave_go<E, 2>(a);
    else if (nvec <= 256) e = ln_bwd_wave_go<E, 4>(a);
    else if (nvec <= 512) e = ln_bwd_go<E, 512, 1, 2, true>(a);
    else if (nvec <= 768) e = ln_bwd_go<E, 768, 1, 2, true>(a);
    else if (nvec <= 1024) e = ln_bwd_go<E, 1024, 1, 1, true>(a);
    else if (nvec <= 2048) e = ln_bwd_go<E, 1024, 2, 1, true>(a);
    // with the next row loaded ahead it would not fit 128 registers: 16384 x
    // 16384 fp32 takes 630 us so, 691 us with it, 1219 us by the kernel for
    // any length
    else if (nvec <= 4096 && !a.bf16) e = ln_bwd_go<float, 1024, 4, 1, false>(a);
    else {
      hipLaunchKernelGGL((ln_bwd_long_kernel<E>), dim3((unsigned)a.M), dim3(kLnThreads), 0,
                         (hipStream_t)a.stream, a);
      e = hipGetLastError();
      if (e == hipSuccess && a.ws) {
        hipLaunchKernelGGL((ln_bwd_long_cols_kernel<E>),
                           dim3((unsigned)((nvec + kLnThreads - 1) / kLnThreads),
                                (unsigned)ln_bwd_groups(a.M, a.D, a.bf16)),
                           dim3(kLnThreads), 0, (hipStream_t)a.stream, a);
        e = hipGetLastError();
      }
    }
    if (e != hipSuccess) return e;
  }
  if (!a.dw) return hipSuccess;
  return launch_slices((2 * a.D + 31) / 32, 256, [&](uint32_t first, dim3 grid) {
    hipLaunchKernelGGL((ln_reduce_kernel<E>), grid, dim3(256), 0, (hipStream_t)a.stream, a,
                       ln_bwd_groups(a.M, a.D, a.bf16), first);
  });
}

hipError_t ln_fwd_launch(const LnArgs &a) { return a.bf16 ? ln_fwd<bf16>(a) : ln_fwd<float>(a); }
hipError_t ln_bwd_launch(const LnArgs &a) { return a.bf16 ? ln_bwd<bf16>(a) : ln_bwd<float>(a); }

}  // namespace dsc
