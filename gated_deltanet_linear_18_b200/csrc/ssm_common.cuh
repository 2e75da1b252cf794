// What the state space kernels share: arguments of the scan and the time step's arithmetic.
#pragma once

#include "common.cuh"

namespace gdn {
namespace ssm {

// log(1 + e^v) without overflow; the accurate functions: one value per (token, head).
__device__ __forceinline__ float softplus(float v) {
  return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}
// -exp(A_log), finite however large A_log is (a step of 0 then still leaves the state alone)
__device__ __forceinline__ float decay_rate(float a_log) {
  const float e = expf(a_log);
  return -(e > 3.402823466e38f ? 3.402823466e38f : e);
}
// 1 / (1 + e^-v) from the hardware's 2^x and reciprocal (each within 2^-22; below 2^-126 it is 0)
__device__ __forceinline__ float sigmoid(float v) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }

// One call of the scan.  Token tensors have `ld*` values between tokens; inside a token's row the
// heads (groups) follow one another without gaps.
struct ScanArgs {
  const void *x, *dt, *B, *C, *z;       // [rows, H, P], [rows, H], [rows, G, N] twice, [rows, H, P]
  long ldx, lddt, ldb, ldc, ldz;
  const float *A_log, *D, *dt_bias;     // [H]; D, dt_bias may be null
  const float* S0;                      // [nseq, H, N, P] or null
  void* y;                              // [rows, H, P], no gaps
  float* S_T;                           // [nseq, H, N, P] or null
  const int* cu;                        // null: nseq sequences of T rows
  int nseq, T, max_len, H, G;
};

}  // namespace ssm
}  // namespace gdn
