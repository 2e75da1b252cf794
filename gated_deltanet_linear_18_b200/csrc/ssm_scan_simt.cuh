// The selective scan on CUDA cores, token by token, in fp32: every type and shape.
//   D_t = softplus(dt_t + dt_bias)   S_t = exp(-D_t exp(A_log)) S_{t-1} + D_t B_t x_t^T
//   y_t = (S_t^T C_t + D x_t) SiLU(z_t)
//
// A CTA owns PT columns of one (sequence, head): 128 threads as PT columns x NG groups of N / NG state rows,
// the state in registers.  Tokens come in tiles through shared memory (B and C as rows that a warp
// reads at few addresses); the next tile is loaded into registers while this one is computed, and the NG
// partial read-outs of a tile are added at its end.  It is the fp32 path and the one for shapes and row distances
// without a tensor-core kernel.  A CTA walks its sequence token by token, so that few sequences and heads leave most SMs
// idle (12 CTAs below) and the time is tokens x 0.1 to 0.2 us; the recurrence would allow to cut the tokens into segments as
// the tensor-core kernel does, which this kernel does not.  Measured, 2 x 333 tokens of 6 heads of 16 x 32 with gates:
// 35 us through the binding, 33 of the kernel; 38 with the gate's values loaded when they are needed, 52 with every tile
// loaded only when its turn came.  At model size: 8192 tokens of 64 heads of 128 x 64 with gates, 1.73 ms in fp32 and
// 1.83 in bf16; of 16 x 64, 0.91 ms in bf16; 4 x 2048 tokens of 48 heads of 128 x 128, 1.50 ms in fp32.
#pragma once

#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

constexpr int kSimtThreads = 128;

template <int N, int P, typename T>
__global__ void __launch_bounds__(kSimtThreads) scan_simt_kernel(const ScanArgs a) {
  constexpr int PT = P < 32 ? P : 32;
  constexpr int NG = kSimtThreads / PT;
  constexpr int NR = N / NG;
  constexpr int kTile = N >= 128 ? 16 : 32;                     // tokens: 16 B and C values a thread at most
  constexpr int kNB = (kTile * N + kSimtThreads - 1) / kSimtThreads, kNX = kTile * PT / kSimtThreads;
  static_assert(N % NG == 0 && kTile * N % kSimtThreads == 0 && kTile * PT % kSimtThreads == 0, "tiles divide");
  const int nblk = P / PT;
  const int pb = blockIdx.x % nblk, h = blockIdx.x / nblk, seq = blockIdx.y;
  const int g = h / (a.H / a.G);
  const RowSpan sp = row_span(a.cu, seq, a.T, a.max_len);
  const int tid = threadIdx.x, col = tid % PT, ng = tid / PT;
  const int p0 = pb * PT;

  __shared__ __align__(16) float sB[kTile][N];
  __shared__ __align__(16) float sC[kTile][N];
  __shared__ float sx[kTile][PT];
  __shared__ float s_step[kTile], s_fade[kTile];
  __shared__ float part[kTile][NG][PT];

  const T* __restrict__ x = static_cast<const T*>(a.x) + (long)h * P + p0;
  const T* __restrict__ dt = static_cast<const T*>(a.dt) + h;
  const T* __restrict__ Bm = static_cast<const T*>(a.B) + (long)g * N;
  const T* __restrict__ Cm = static_cast<const T*>(a.C) + (long)g * N;
  const T* __restrict__ z = a.z ? static_cast<const T*>(a.z) + (long)h * P + p0 : nullptr;
  T* __restrict__ y = static_cast<T*>(a.y) + (long)h * P + p0;
  const float rate = decay_rate(a.A_log[h]);
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const float skip = a.D ? a.D[h] : 0.f;

  const long sbase = ((long)seq * a.H + h) * N * P + p0 + col;
  float S[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) S[i] = a.S0 ? a.S0[sbase + (long)(ng * NR + i) * P] : 0.f;

  T rb[kNB], rc[kNB], rx[kNX], rt;               // the next tile, as loaded
  T rz[kNX];                                     // this tile's gate values
  auto fetch = [&](int t0) {
    const int nt = min(kTile, sp.len - t0);
#pragma unroll
    for (int k = 0; k < kNB; ++k) {
      const int i = tid + k * kSimtThreads, t = i / N, n = i % N;
      if (t < nt) {
        const long r = sp.row0 + t0 + t;
        rb[k] = Bm[r * a.ldb + n];
        rc[k] = Cm[r * a.ldc + n];
      }
    }
#pragma unroll
    for (int k = 0; k < kNX; ++k) {
      const int i = tid + k * kSimtThreads, t = i / PT, p = i % PT;
      if (t < nt) rx[k] = x[(sp.row0 + t0 + t) * a.ldx + p];
    }
    if (tid < nt) rt = dt[(sp.row0 + t0 + tid) * a.lddt];
  };
  fetch(0);
  for (int t0 = 0; t0 < sp.len; t0 += kTile) {
    const int nt = min(kTile, sp.len - t0);
    __syncthreads();                             // the tile before has been read
#pragma unroll
    for (int k = 0; k < kNB; ++k) {
      const int i = tid + k * kSimtThreads, t = i / N, n = i % N;
      if (t < nt) {
        sB[t][n] = to_f(rb[k]);
        sC[t][n] = to_f(rc[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kNX; ++k) {
      const int i = tid + k * kSimtThreads, t = i / PT, p = i % PT;
      if (t < nt) sx[t][p] = to_f(rx[k]);
    }
    if (tid < nt) {
      const float step = softplus(to_f(rt) + bias);
      s_step[tid] = step;
      s_fade[tid] = expf(step * rate);
    }
    __syncthreads();
    if (z) {
#pragma unroll
      for (int k = 0; k < kNX; ++k) {
        const int i = tid + k * kSimtThreads, t = i / PT, p = i % PT;
        if (t < nt) rz[k] = z[(sp.row0 + t0 + t) * a.ldz + p];
      }
    }
    fetch(t0 + kTile);
    auto token = [&](int t) {
      const float fade = s_fade[t], xd = sx[t][col] * s_step[t];
      float acc = 0.f;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        S[i] = fmaf(fade, S[i], xd * sB[t][ng * NR + i]);
        acc = fmaf(S[i], sC[t][ng * NR + i], acc);
      }
      part[t][ng][col] = acc;
    };
    int t = 0;
    for (; t + 4 <= nt; t += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) token(t + i);
    }
    for (; t < nt; ++t) token(t);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kNX; ++k) {
      const int i = tid + k * kSimtThreads, t = i / PT, p = i % PT;
      if (t < nt) {
        float o = skip * sx[t][p];
#pragma unroll
        for (int q = 0; q < NG; ++q) o += part[t][q][p];
        if (z) o *= silu(to_f(rz[k]));
        y[(sp.row0 + t0 + t) * ((long)a.H * P) + p] = from_f<T>(o);
      }
    }
  }
  if (a.S_T) {
#pragma unroll
    for (int i = 0; i < NR; ++i) a.S_T[sbase + (long)(ng * NR + i) * P] = S[i];
  }
}

}  // namespace ssm
}  // namespace gdn
