// One token of the state space block for n sequences: the short convolution over a carried
// three-row history, SiLU, the time step, the state update in place and the gated read-out
//   x, B, C = SiLU(conv4([history; row]))        D_t = softplus(dt + dt_bias)
//   S <- exp(-D_t exp(A_log)) S + D_t B x^T       y = (S^T C + D x) SiLU(z)
// in one kernel, everything between the row and y in fp32.
//
// Bound by HBM: the state crosses it once each way (8 N P bytes per head) and is most of the
// traffic.  One CTA per (sequence, head), the layout of the delta rule's decode step: thread t owns
// four columns (one float4) of the rows rg, rg + RG, ..., all of whose loads are issued before the
// convolution is computed, so that the row's work hides under them.  The heads of a group each
// recompute its B and C (8 N values against 8 N P bytes of state); the group's first head moves
// their history on.  Measured, bf16: 256 sequences of 48 heads of 128 x 128 in 262 us = 6.3 TB/s, the rate
// of a copy; one of 64 heads of 128 x 64 in 3.9 us, the latency of its loads and sums.
#pragma once

#include "decode.cuh"
#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

struct StepArgs {
  const void *u, *dt, *z;               // [n, H P + 2 G N], [n, H], [n, H, P] or null
  long ldu, lddt, ldz;
  const void* hist_in;                  // [n, 3, H P + 2 G N]
  void* hist_out;
  const float *w, *bias, *A_log, *D, *dt_bias;
  float* S;                             // [n, H, N, P]
  void* y;                              // [n, H, P]
  int H, G;
};

template <int N, int P, typename T>
__global__ void __launch_bounds__(DecodeShape<N, P>::NT) step_kernel(const StepArgs a) {
  using Sh = DecodeShape<N, P>;
  constexpr int CG = Sh::CG, NT = Sh::NT, RG = Sh::RG, RPT = Sh::RPT;
  const long nh = blockIdx.x;
  const int h = (int)(nh % a.H);
  const long n = nh / a.H;
  const int hpg = a.H / a.G, g = h / hpg;
  const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
  const int C = a.H * P + 2 * a.G * N;

  __shared__ __align__(16) float sx[P];
  __shared__ __align__(16) float sB[N];
  __shared__ __align__(16) float sC[N];
  __shared__ __align__(16) float red[RG][P + 4];

  float4* Sh4 = reinterpret_cast<float4*>(a.S + nh * (long)N * P);
  float4 m[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) m[r] = Sh4[(rg + r * RG) * CG + cg];

  const T* __restrict__ row = static_cast<const T*>(a.u) + n * a.ldu;
  const T* __restrict__ hin = static_cast<const T*>(a.hist_in) + n * 3L * C;
  T* __restrict__ hout = static_cast<T*>(a.hist_out) + n * 3L * C;
  auto conv = [&](int c, bool write) -> float {
    const T u0 = hin[c], u1 = hin[(long)C + c], u2 = hin[2L * C + c], u3 = row[c];
    const float* w = a.w + 4L * c;
    float acc = a.bias ? a.bias[c] : 0.f;
    acc = fmaf(w[0], to_f(u0), acc);
    acc = fmaf(w[1], to_f(u1), acc);
    acc = fmaf(w[2], to_f(u2), acc);
    acc = fmaf(w[3], to_f(u3), acc);
    if (write) {
      hout[c] = u1;
      hout[(long)C + c] = u2;
      hout[2L * C + c] = u3;
    }
    return silu(acc);
  };
  const bool writer = h % hpg == 0;
  for (int i = tid; i < P + 2 * N; i += NT) {
    if (i < P) {
      sx[i] = conv(h * P + i, true);
    } else if (i < P + N) {
      sB[i - P] = conv(a.H * P + g * N + i - P, writer);
    } else {
      sC[i - P - N] = conv(a.H * P + (a.G + g) * N + i - P - N, writer);
    }
  }
  const float step = softplus(to_f(static_cast<const T*>(a.dt)[n * a.lddt + h]) +
                              (a.dt_bias ? a.dt_bias[h] : 0.f));
  const float fade = expf(step * decay_rate(a.A_log[h]));
  __syncthreads();
  float4 xd = *reinterpret_cast<const float4*>(&sx[cg * 4]);
  xd.x *= step; xd.y *= step; xd.z *= step; xd.w *= step;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int i = rg + r * RG;
    const float b = sB[i], c = sC[i];
    float4 s = m[r];
    s.x = fmaf(fade, s.x, b * xd.x); s.y = fmaf(fade, s.y, b * xd.y);
    s.z = fmaf(fade, s.z, b * xd.z); s.w = fmaf(fade, s.w, b * xd.w);
    Sh4[i * CG + cg] = s;
    acc.x = fmaf(c, s.x, acc.x); acc.y = fmaf(c, s.y, acc.y);
    acc.z = fmaf(c, s.z, acc.z); acc.w = fmaf(c, s.w, acc.w);
  }
  *reinterpret_cast<float4*>(&red[rg][cg * 4]) = acc;
  __syncthreads();
  if (tid < P) {
    float o = a.D ? a.D[h] * sx[tid] : 0.f;
#pragma unroll
    for (int q = 0; q < RG; ++q) o += red[q][tid];
    if (a.z) o *= silu(to_f(static_cast<const T*>(a.z)[n * a.ldz + (long)h * P + tid]));
    static_cast<T*>(a.y)[nh * P + tid] = from_f<T>(o);
  }
}

}  // namespace ssm
}  // namespace gdn
