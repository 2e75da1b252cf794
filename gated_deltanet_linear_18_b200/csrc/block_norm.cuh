// The norms before and after a block, fused with the block's gate and its residual scale:
//   n  = RMSNorm(y) w_post            (y: the block's output; n = y without w_post)
//   h' = h + s (.) SiLU(z) (.) n      (h: the residual stream; s, z may be missing: 1)
//   x  = RMSNorm(h') w_pre            (the next block's input; not written without w_pre)
// with RMSNorm(v) = v / sqrt(mean(v^2) + eps), everything in fp32 from the loads to the final
// rounding (x is the norm of h' before its rounding).  Backward, with v' the gradient of v:
//   a  = h'' + r (w_pre x' - h' r^2 mean(w_pre x' h')),  r = 1 / sqrt(mean(h'^2) + eps)   (= dh)
//   dz = a s n SiLU'(z),  ds = sum_rows a SiLU(z) n,  n' = a s SiLU(z)
//   dy = q (w_post n' - y q^2 mean(w_post n' y)),  q = 1 / sqrt(mean(y^2) + eps)
//   dw_post = sum_rows n' y q,  dw_pre = sum_rows x' h' r
//
// Bound by HBM.  A persistent CTA walks rows: the row's arrays arrive in shared memory by bulk
// asynchronous copies a stage or more ahead (one mbarrier per stage), so the loads of the next
// rows run under the two block-wide reductions of this one; a thread owns the same 8 K columns in
// every row, so the fp32 vectors (and the backward's three column sums) stay in registers and are
// read (written) once per CTA.  The column sums of the CTAs are added by a second kernel in a fixed
// order, so the results are reproducible bit for bit.  Rows whose width is not a multiple of 8
// values, or whose tensors are not 16-byte aligned, take the loop kernels at the end.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace bn {

constexpr uint64_t kWaitCycles = 4000000000ull;   // bounded waits: about 2 s

struct FwdArgs {
  const void *y, *h, *z;
  const float *w_post, *w_pre, *scale;
  void *h_out, *x;
  long rows;
  int D;
  float eps;
};
struct BwdArgs {
  const void *y, *h, *z, *dh_in, *dx;     // h: the residual after the block
  const float *w_post, *w_pre, *scale;
  void *dy, *dh, *dz;
  float* part;                            // [CTAs, 3, D]: dw_post, dw_pre, dscale
  long rows;
  int D;
  float eps;
};

__device__ __forceinline__ float sigm(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// 8 consecutive values
template <typename T> __device__ __forceinline__ void ld8(const T* p, float (&f)[8]);
template <> __device__ __forceinline__ void ld8<float>(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <>
__device__ __forceinline__ void ld8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
template <typename T> __device__ __forceinline__ void st8(T* p, const float (&f)[8]);
template <> __device__ __forceinline__ void st8<float>(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
template <>
__device__ __forceinline__ void st8<__nv_bfloat16>(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = tc::pack_bf16(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// Sum over the CTA; one barrier: `red` (32 floats) must not be in use by an earlier call that some
// thread may still read, so callers alternate between two.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  const int warps = (blockDim.x + 31) >> 5;
  if (warps == 1) {
    __syncthreads();
    return v;
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

// The row stages: `n` arrays of a row each, `bytes[i]` long, at `at[i]` in a stage; `off`: the same
// places by the array's role (a missing array has none).
struct Ring {
  const char* src[5];
  uint32_t bytes[5], at[5], off[5];
  uint32_t stage_bytes;
  int n, stages;
};

// ---------------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------------
template <typename T, typename TH, int K, int MAXT>
__global__ void __launch_bounds__(MAXT) fwd_kernel(const FwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[4];
  __shared__ float red[3][32];
  __shared__ int abort_word;
  const int tid = threadIdx.x, nt = blockDim.x;
  const uint32_t sb = tc::smem_u32(smem);
  volatile int* abort_flag = &abort_word;
  if (tid == 0) {
    abort_word = 0;
    for (int i = 0; i < ring.stages; ++i) tc::mbar_init(tc::smem_u32(&full[i]), 1);
    tc::fence_barrier_init();
  }
  __syncthreads();
  const long row0 = blockIdx.x, step = gridDim.x;
  const long mine = row0 < a.rows ? (a.rows - row0 + step - 1) / step : 0;
  auto issue = [&](long i) {             // this CTA's i-th row into its stage (one thread)
    const int st = (int)(i % ring.stages);
    const uint32_t bar = tc::smem_u32(&full[st]), dst = sb + st * ring.stage_bytes;
    tc::mbar_arrive_expect_tx(bar, ring.stage_bytes);
    const long r = row0 + i * step;
    for (int k = 0; k < ring.n; ++k)
      tc::bulk_load(dst + ring.at[k], ring.src[k] + r * (long)ring.bytes[k], ring.bytes[k], bar);
  };
  if (tid == 0)
    for (long i = 0; i < ring.stages && i < mine; ++i) issue(i);

  float wp[K][8], wn[K][8], sc[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * nt + tid) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) wp[k][e] = sc[k][e] = wn[k][e] = 1.f;
    if (c < a.D) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (a.w_post) wp[k][e] = a.w_post[c + e];
        if (a.w_pre) wn[k][e] = a.w_pre[c + e];
        if (a.scale) sc[k][e] = a.scale[c + e];
      }
    }
  }
  const float invD = 1.0f / (float)a.D;
  for (long i = 0; i < mine; ++i) {
    const int st = (int)(i % ring.stages);
    const long r = row0 + i * step;
    const unsigned char* base = smem + (long)st * ring.stage_bytes;
    const T* sy = reinterpret_cast<const T*>(base + ring.off[0]);
    const TH* sh = reinterpret_cast<const TH*>(base + ring.off[1]);
    const T* sz = reinterpret_cast<const T*>(base + ring.off[2]);
    tc::mbar_wait(tc::smem_u32(&full[st]), (uint32_t)(i / ring.stages) & 1u, abort_flag, kWaitCycles);
    float v[K][8];
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + tid) * 8;
      if (c < a.D) ld8<T>(sy + c, v[k]);
      else for (int e = 0; e < 8; ++e) v[k][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(v[k][e], v[k][e], q);
    }
    float ry = 1.f;
    // without the second norm's barrier the next row's sums go to the other buffer
    if (a.w_post) ry = rsqrtf(fmaf(block_sum(q, red[a.w_pre ? 0 : (int)(i & 1)]), invD, a.eps));
    else __syncthreads();
    // every thread has left the previous row's stage: refill it
    if (ring.stages > 1 && tid == 0 && i > 0 && i - 1 + ring.stages < mine) issue(i - 1 + ring.stages);
    q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + tid) * 8;
      float hv[8];
      if (c < a.D) ld8<TH>(sh + c, hv);
      else for (int e = 0; e < 8; ++e) hv[e] = 0.f;
      if (a.z) {
        float zv[8];
        if (c < a.D) ld8<T>(sz + c, zv);
        else for (int e = 0; e < 8; ++e) zv[e] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] *= zv[e] * sigm(zv[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[k][e] = fmaf(v[k][e] * ry, wp[k][e] * sc[k][e], hv[e]);
        q = fmaf(v[k][e], v[k][e], q);
      }
      if (c < a.D) st8<TH>(static_cast<TH*>(a.h_out) + r * a.D + c, v[k]);
    }
    if (a.w_pre) {
      const float rh = rsqrtf(fmaf(block_sum(q, red[2]), invD, a.eps));
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * nt + tid) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] *= rh * wn[k][e];
        if (c < a.D) st8<T>(static_cast<T*>(a.x) + r * a.D + c, v[k]);
      }
    }
    if (ring.stages == 1) {
      __syncthreads();
      if (tid == 0 && i + 1 < mine) issue(i + 1);
    }
  }
  __syncthreads();
  if (tid == 0 && abort_word) record_error(kErrTimeout);
}

// ---------------------------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------------------------
template <typename T, typename TH, int K, int MAXT>
__global__ void __launch_bounds__(MAXT) bwd_kernel(const BwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[4];
  __shared__ float red[4][32];
  __shared__ int abort_word;
  const int tid = threadIdx.x, nt = blockDim.x;
  const uint32_t sb = tc::smem_u32(smem);
  volatile int* abort_flag = &abort_word;
  if (tid == 0) {
    abort_word = 0;
    for (int i = 0; i < ring.stages; ++i) tc::mbar_init(tc::smem_u32(&full[i]), 1);
    tc::fence_barrier_init();
  }
  __syncthreads();
  const long row0 = blockIdx.x, step = gridDim.x;
  const long mine = row0 < a.rows ? (a.rows - row0 + step - 1) / step : 0;
  auto issue = [&](long i) {
    const int st = (int)(i % ring.stages);
    const uint32_t bar = tc::smem_u32(&full[st]), dst = sb + st * ring.stage_bytes;
    tc::mbar_arrive_expect_tx(bar, ring.stage_bytes);
    const long r = row0 + i * step;
    for (int k = 0; k < ring.n; ++k)
      tc::bulk_load(dst + ring.at[k], ring.src[k] + r * (long)ring.bytes[k], ring.bytes[k], bar);
  };
  if (tid == 0)
    for (long i = 0; i < ring.stages && i < mine; ++i) issue(i);

  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  // the three vectors and their gradients' sums over this CTA's rows
  float wp[K][8], wn[K][8], sc[K][8], gp[K][8], gn[K][8], gs[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * nt + tid) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      wp[k][e] = wn[k][e] = sc[k][e] = 1.f;
      gp[k][e] = gn[k][e] = gs[k][e] = 0.f;
      if (c < a.D) {
        if (post) wp[k][e] = a.w_post[c + e];
        if (pre) wn[k][e] = a.w_pre[c + e];
        if (a.scale) sc[k][e] = a.scale[c + e];
      }
    }
  }
  const float invD = 1.0f / (float)a.D;
  for (long i = 0; i < mine; ++i) {
    const int st = (int)(i % ring.stages);
    const long r = row0 + i * step;
    const unsigned char* base = smem + (long)st * ring.stage_bytes;
    const T* sy = reinterpret_cast<const T*>(base + ring.off[0]);
    const TH* sh = reinterpret_cast<const TH*>(base + ring.off[1]);
    const T* sz = reinterpret_cast<const T*>(base + ring.off[2]);
    const TH* sg = reinterpret_cast<const TH*>(base + ring.off[3]);
    const T* sx = reinterpret_cast<const T*>(base + ring.off[4]);
    tc::mbar_wait(tc::smem_u32(&full[st]), (uint32_t)(i / ring.stages) & 1u, abort_flag, kWaitCycles);
    // the three sums that do not need dh: y^2, h'^2, w_pre x' h'
    float qy = 0.f, qh = 0.f, qx = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + tid) * 8;
      if (c < a.D) {
        float f[8];
        if (post) {
          ld8<T>(sy + c, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) qy = fmaf(f[e], f[e], qy);
        }
        if (pre) {
          float d[8];
          ld8<TH>(sh + c, f);
          ld8<T>(sx + c, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            qh = fmaf(f[e], f[e], qh);
            qx = fmaf(f[e] * wn[k][e], d[e], qx);
          }
        }
      }
    }
    qy = warp_sum(qy);
    qh = warp_sum(qh);
    qx = warp_sum(qx);
    const int warps = (nt + 31) >> 5, lane = tid & 31;
    if (lane == 0) {
      red[0][tid >> 5] = qy;
      red[1][tid >> 5] = qh;
      red[2][tid >> 5] = qx;
    }
    __syncthreads();
    if (ring.stages > 1 && tid == 0 && i > 0 && i - 1 + ring.stages < mine) issue(i - 1 + ring.stages);
    qy = warp_sum(lane < warps ? red[0][lane] : 0.f);
    qh = warp_sum(lane < warps ? red[1][lane] : 0.f);
    qx = warp_sum(lane < warps ? red[2][lane] : 0.f);
    const float ry = post ? rsqrtf(fmaf(qy, invD, a.eps)) : 1.f;
    const float rh = pre ? rsqrtf(fmaf(qh, invD, a.eps)) : 0.f;
    const float mx = rh * rh * qx * invD;
    float u[K][8];                       // n' w_post: what dy starts from
    float qd = 0.f;                      // w_post n' y
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + tid) * 8;
      if (c < a.D) {
        float yv[8], dh[8], f[8];
        ld8<T>(sy + c, yv);
        if (a.dh_in) ld8<TH>(sg + c, dh);
        else for (int e = 0; e < 8; ++e) dh[e] = 0.f;
        if (pre) {
          float d[8];
          ld8<TH>(sh + c, f);
          ld8<T>(sx + c, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            gn[k][e] = fmaf(d[e] * rh, f[e], gn[k][e]);
            dh[e] = fmaf(rh, fmaf(d[e], wn[k][e], -f[e] * mx), dh[e]);
          }
        }
        st8<TH>(static_cast<TH*>(a.dh) + r * a.D + c, dh);
        if (a.z) {
          float zv[8], dz[8];
          ld8<T>(sz + c, zv);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float s = sigm(zv[e]), gate = zv[e] * s;
            const float yr = yv[e] * ry, as = dh[e] * sc[k][e];
            const float n = yr * wp[k][e];
            gs[k][e] = fmaf(dh[e] * gate, n, gs[k][e]);
            dz[e] = as * n * s * fmaf(zv[e], 1.f - s, 1.f);
            const float dn = as * gate;
            gp[k][e] = fmaf(dn, yr, gp[k][e]);
            u[k][e] = dn * wp[k][e];
            qd = fmaf(u[k][e], yv[e], qd);
          }
          st8<T>(static_cast<T*>(a.dz) + r * a.D + c, dz);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float yr = yv[e] * ry, dn = dh[e] * sc[k][e];
            gs[k][e] = fmaf(dh[e], yr * wp[k][e], gs[k][e]);
            gp[k][e] = fmaf(dn, yr, gp[k][e]);
            u[k][e] = dn * wp[k][e];
            qd = fmaf(u[k][e], yv[e], qd);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[k][e] = 0.f;
      }
    }
    float my = 0.f;
    if (post) my = ry * ry * block_sum(qd, red[3]) * invD;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + tid) * 8;
      if (c < a.D) {
        if (post) {
          float yv[8];
          ld8<T>(sy + c, yv);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[k][e] = ry * fmaf(-yv[e], my, u[k][e]);
        }
        st8<T>(static_cast<T*>(a.dy) + r * a.D + c, u[k]);
      }
    }
    if (!post || ring.stages == 1) {      // red[0..2] and the stage are used again
      __syncthreads();
      if (ring.stages == 1 && tid == 0 && i + 1 < mine) issue(i + 1);
    }
  }
  float* part = a.part + (long)blockIdx.x * 3 * a.D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * nt + tid) * 8;
    if (c < a.D) {
      if (post) st8<float>(part + c, gp[k]);
      if (pre) st8<float>(part + (long)a.D + c, gn[k]);
      if (a.scale) st8<float>(part + 2L * a.D + c, gs[k]);
    }
  }
  __syncthreads();
  if (tid == 0 && abort_word) record_error(kErrTimeout);
}

// Column sums of the CTAs' parts, in a fixed order: 32 columns x 16 slices of the CTAs per block,
// then the 16 slices.  blockIdx.y: which of the three vectors.
__global__ void __launch_bounds__(512) column_sum_kernel(const float* __restrict__ part, int ctas, int D,
                                                         float* dw_post, float* dw_pre, float* dscale) {
  __shared__ float s[16][33];
  float* out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dw_pre : dscale;
  if (!out) return;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < D) {
    const float* p = part + (long)blockIdx.y * D + c;
#pragma unroll 4
    for (int i = slice; i < ctas; i += 16) v += p[(long)i * 3 * D];
  }
  s[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && c < D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][lane];
    out[c] = t;
  }
}

// ---------------------------------------------------------------------------------------------
// any width and alignment: the row is read again in each pass (from L1 / L2)
// ---------------------------------------------------------------------------------------------
constexpr int kLoopThreads = 256;

template <typename T, typename TH>
__global__ void __launch_bounds__(kLoopThreads) fwd_loop_kernel(const FwdArgs a) {
  __shared__ float red[2][32];
  const int tid = threadIdx.x;
  const float invD = 1.0f / (float)a.D;
  for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* y = static_cast<const T*>(a.y) + r * a.D;
    const TH* h = static_cast<const TH*>(a.h) + r * a.D;
    const T* z = a.z ? static_cast<const T*>(a.z) + r * a.D : nullptr;
    TH* ho = static_cast<TH*>(a.h_out) + r * a.D;
    float q = 0.f, ry = 1.f;
    if (a.w_post) {
      for (int c = tid; c < a.D; c += kLoopThreads) {
        const float v = to_f(y[c]);
        q = fmaf(v, v, q);
      }
      ry = rsqrtf(fmaf(block_sum(q, red[0]), invD, a.eps));
    }
    auto after = [&](int c) -> float {
      float v = to_f(y[c]) * ry;
      if (a.w_post) v *= a.w_post[c];
      if (a.scale) v *= a.scale[c];
      if (z) {
        const float zv = to_f(z[c]);
        v *= zv * sigm(zv);
      }
      return to_f(h[c]) + v;
    };
    q = 0.f;
    for (int c = tid; c < a.D; c += kLoopThreads) {
      const float v = after(c);
      ho[c] = from_f<TH>(v);
      q = fmaf(v, v, q);
    }
    if (a.w_pre) {
      const float rh = rsqrtf(fmaf(block_sum(q, red[1]), invD, a.eps));
      T* x = static_cast<T*>(a.x) + r * a.D;
      for (int c = tid; c < a.D; c += kLoopThreads) x[c] = from_f<T>(after(c) * rh * a.w_pre[c]);
    }
    __syncthreads();
  }
}

// The column sums are kept in this CTA's part of the workspace: column c belongs to one thread.
template <typename T, typename TH>
__global__ void __launch_bounds__(kLoopThreads) bwd_loop_kernel(const BwdArgs a) {
  __shared__ float red[4][32];
  const int tid = threadIdx.x;
  const float invD = 1.0f / (float)a.D;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  float* gp = a.part + (long)blockIdx.x * 3 * a.D;
  float *gn = gp + a.D, *gs = gn + a.D;
  for (int c = tid; c < a.D; c += kLoopThreads) gp[c] = gn[c] = gs[c] = 0.f;
  for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* y = static_cast<const T*>(a.y) + r * a.D;
    const TH* h = static_cast<const TH*>(a.h) + r * a.D;
    const T* z = a.z ? static_cast<const T*>(a.z) + r * a.D : nullptr;
    const TH* g = a.dh_in ? static_cast<const TH*>(a.dh_in) + r * a.D : nullptr;
    const T* dx = pre ? static_cast<const T*>(a.dx) + r * a.D : nullptr;
    TH* dho = static_cast<TH*>(a.dh) + r * a.D;
    T* dyo = static_cast<T*>(a.dy) + r * a.D;
    T* dzo = z ? static_cast<T*>(a.dz) + r * a.D : nullptr;
    float ry = 1.f, rh = 0.f, mx = 0.f;
    if (post) {
      float q = 0.f;
      for (int c = tid; c < a.D; c += kLoopThreads) {
        const float v = to_f(y[c]);
        q = fmaf(v, v, q);
      }
      ry = rsqrtf(fmaf(block_sum(q, red[0]), invD, a.eps));
    }
    if (pre) {
      float q = 0.f, p = 0.f;
      for (int c = tid; c < a.D; c += kLoopThreads) {
        const float v = to_f(h[c]);
        q = fmaf(v, v, q);
        p = fmaf(v * a.w_pre[c], to_f(dx[c]), p);
      }
      rh = rsqrtf(fmaf(block_sum(q, red[1]), invD, a.eps));
      mx = rh * rh * block_sum(p, red[2]) * invD;
    }
    // the residual's gradient and n' w_post of column c (without the norm's projection)
    auto grads = [&](int c, float& dh, float& yr, float& dn) {
      dh = g ? to_f(g[c]) : 0.f;
      if (pre) dh = fmaf(rh, fmaf(to_f(dx[c]), a.w_pre[c], -to_f(h[c]) * mx), dh);
      yr = to_f(y[c]) * ry;
      dn = a.scale ? dh * a.scale[c] : dh;
      if (z) {
        const float zv = to_f(z[c]);
        dn *= zv * sigm(zv);
      }
    };
    float qd = 0.f;
    for (int c = tid; c < a.D; c += kLoopThreads) {
      float dh, yr, dn;
      grads(c, dh, yr, dn);
      const float w = post ? a.w_post[c] : 1.f, n = yr * w;
      dho[c] = from_f<TH>(dh);
      float gate = 1.f;
      if (z) {
        const float zv = to_f(z[c]), s = sigm(zv);
        gate = zv * s;
        dzo[c] = from_f<T>(dh * (a.scale ? a.scale[c] : 1.f) * n * s * fmaf(zv, 1.f - s, 1.f));
      }
      gp[c] = fmaf(dn, yr, gp[c]);
      gs[c] = fmaf(dh * gate, n, gs[c]);
      if (pre) gn[c] = fmaf(to_f(dx[c]) * rh, to_f(h[c]), gn[c]);
      if (post) qd = fmaf(dn * w, to_f(y[c]), qd);
      else dyo[c] = from_f<T>(dn);
    }
    if (post) {
      const float my = ry * ry * block_sum(qd, red[3]) * invD;
      for (int c = tid; c < a.D; c += kLoopThreads) {
        float dh, yr, dn;
        grads(c, dh, yr, dn);
        dyo[c] = from_f<T>(ry * fmaf(-to_f(y[c]), my, dn * a.w_post[c]));
      }
    }
    __syncthreads();
  }
}

}  // namespace bn
}  // namespace gdn
