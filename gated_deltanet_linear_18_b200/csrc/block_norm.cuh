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
// s and w_post meet one column sum A = sum_rows a SiLU(z) y q only: dw_post = s A, ds = w_post A.
//
// Bound by HBM.  One persistent CTA an SM, cut into groups of threads that walk rows of their own:
// a row's arrays arrive in shared memory by bulk asynchronous copies a stage or more ahead (one
// mbarrier per stage), and while one group waits for its block-wide sums another computes.  The fp32
// vectors (w_post s, w_pre) sit in shared memory, read from HBM once per CTA; a thread owns the same
// 8 K columns in every row, so the backward's two column sums stay in registers.  The sums of the
// groups are added by a second kernel in a fixed order: reproducible bit for bit.  Rows whose width
// is not a multiple of 8 values or above 8192, whose tensors are not 16-byte aligned, or that do not fit
// shared memory beside the two vectors (the fp32 backward's five arrays above 7896 columns), take the loop
// kernels at the end.
// Measured, 8192 x 6144 bf16, gate and both vectors: forward 100 us = 5.0 TB/s (a copy: 6.45), backward 203 us = 4.0
// TB/s.  The backward is short of warps: its 158 registers a thread (40 of raw values, 32 of column sums, 16 of
// sigmoids) leave 12 an SM, which issue in 43 % of the cycles and wait for the row's sums in between.  With
// two syncs a row it took 214 us, with a row a CTA, read again in each pass, 240 (the forward so: 181).
// 8192 rows in other types, gate and vectors, forward and backward in us (TB/s): fp32 residual, 6144 wide 132 (5.3) and 245
// (4.5), 8192 wide 198 (4.8) and 392 (3.8); fp32, 4096 wide 132 (5.1) and 243 (4.4), 6144 wide 196 (5.1) and 395 (4.1), 8192
// wide 317 (4.2) and, in the loop kernel, 1672 (1.3).
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
  float* part;                            // [parts, 2, D]: A, dw_pre
  long rows;
  int D;
  float eps;
};

// 1 / (1 + e^-v) from the hardware's 2^x and reciprocal (each within 2^-22)
__device__ __forceinline__ float sigm(float v) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// 8 consecutive values as loaded, and as four pairs for the paired fp32 instructions
template <typename T> struct Piece8;
template <> struct Piece8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(f2_t (&f)[4]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pk2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const f2_t (&f)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x, y;
      up2(f[i], x, y);
      u[i] = tc::pack_bf16(x, y);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <> struct Piece8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(f2_t (&f)[4]) const {
    f[0] = pk2(a.x, a.y);
    f[1] = pk2(a.z, a.w);
    f[2] = pk2(b.x, b.y);
    f[3] = pk2(b.z, b.w);
  }
  static __device__ __forceinline__ void store(float* p, const f2_t (&f)[4]) {
    float4 o[2];
    up2(f[0], o[0].x, o[0].y);
    up2(f[1], o[0].z, o[0].w);
    up2(f[2], o[1].x, o[1].y);
    up2(f[3], o[1].z, o[1].w);
    reinterpret_cast<float4*>(p)[0] = o[0];
    reinterpret_cast<float4*>(p)[1] = o[1];
  }
};
__device__ __forceinline__ void ldv(const float* p, f2_t (&f)[4]) {   // 8 values of a vector
  Piece8<float> v;
  v.load(p);
  v.get(f);
}

constexpr int kMaxGroups = 12, kMaxStages = 4;

// A call's rows over the grid: `groups` groups of `nt` threads a CTA; group g of CTA b takes rows g gridDim.x + b,
// then every (groups gridDim.x)-th.  The row stages: `n` arrays of a row each, `bytes[i]` long, at `at[i]` in a
// stage; `off`: the same places by the array's role (a missing array has none).
struct Ring {
  const char* src[5];
  uint32_t bytes[5], at[5], off[5];
  uint32_t stage_bytes;
  int n, stages, groups, nt;
};

__device__ __forceinline__ void group_sync(int g, int nt) {
  if (nt == 32) __syncwarp();
  else tc::named_bar(1 + g, nt);
}

// What both directions share: the barriers, the vectors in shared memory, and a group's row walk.
struct Walk {
  uint64_t* full;                // this group's stage barriers
  unsigned char* stage0;         // this group's stages
  int g, t;                      // group; thread in it
  long row0, step, mine;         // first row, distance, number of rows
  int st;                        // the present row's stage and its barrier's parity (counted, not divided)
  uint32_t phase;
  volatile int* abort_flag;

  // `vec`: dynamic shared memory, [2][D] floats (w_post s, w_pre) and then the groups' stages
  __device__ __forceinline__ void init(const Ring& ring, unsigned char* smem, uint64_t (*bars)[kMaxStages], int* abort_word,
                                       const float* w_post, const float* scale, const float* w_pre, int D, long rows) {
    abort_flag = abort_word;
    g = threadIdx.x / ring.nt;
    t = threadIdx.x % ring.nt;
    full = bars[g];
    stage0 = smem + 8L * D + (long)g * ring.stages * ring.stage_bytes;
    if (threadIdx.x == 0) {
      *abort_word = 0;
      for (int i = 0; i < ring.groups; ++i)
        for (int j = 0; j < ring.stages; ++j) tc::mbar_init(tc::smem_u32(&bars[i][j]), 1);
      tc::fence_barrier_init();
    }
    row0 = (long)g * gridDim.x + blockIdx.x;
    step = (long)ring.groups * gridDim.x;
    mine = row0 < rows ? (rows - row0 + step - 1) / step : 0;
    st = 0;
    phase = 0;
    __syncthreads();
    if (t == 0)
      for (int i = 0; i < ring.stages && i < mine; ++i) issue(ring, i, i);
    float* v = reinterpret_cast<float*>(smem);
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      v[c] = (w_post ? w_post[c] : 1.f) * (scale ? scale[c] : 1.f);
      v[D + c] = w_pre ? w_pre[c] : 1.f;
    }
    __syncthreads();
  }
  __device__ __forceinline__ void issue(const Ring& ring, long i, int to) const {   // row i into stage `to` (one thread)
    const uint32_t bar = tc::smem_u32(&full[to]), dst = tc::smem_u32(stage0) + to * ring.stage_bytes;
    tc::mbar_arrive_expect_tx(bar, ring.stage_bytes);
    const long r = row0 + i * step;
    for (int k = 0; k < ring.n; ++k)
      tc::bulk_load(dst + ring.at[k], ring.src[k] + r * (long)ring.bytes[k], ring.bytes[k], bar);
  }
  __device__ __forceinline__ const unsigned char* wait(const Ring& ring) const {
    tc::mbar_wait(tc::smem_u32(&full[st]), phase, abort_flag, kWaitCycles);
    return stage0 + (uint32_t)st * ring.stage_bytes;
  }
  // after the first group-wide sync of row i: every thread holds the row in registers, its stage is free
  __device__ __forceinline__ void refill(const Ring& ring, long i) {
    if (t == 0 && i + ring.stages < mine) issue(ring, i + ring.stages, st);
    if (++st == ring.stages) {
      st = 0;
      phase ^= 1u;
    }
  }
};

// Sum over the group; one sync.  `red` (32 floats) must not be in use by an earlier call that some
// thread may still read.
__device__ __forceinline__ float group_sum(float v, float* red, int g, int t, int nt) {
  v = warp_sum(v);
  if (nt == 32) {
    __syncwarp();
    return v;
  }
  if ((t & 31) == 0) red[t >> 5] = v;
  group_sync(g, nt);
  return warp_sum((t & 31) < (nt >> 5) ? red[t & 31] : 0.f);
}
// Six sums over the group; one sync.  In a warp, eight values (two of them zeros) take nine shuffles: with each of the
// first three steps a lane gives half of its values away, so that lane 4 i ends with the sum of v[i].  Then each warp adds
// the warps' parts, four lanes a value.  red: [warps][8] floats.
__device__ __forceinline__ void group_sum6(float (&v)[6], float* red, int g, int t, int nt) {
  const int lane = t & 31;
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  const float w[8] = {v[0], v[1], v[2], v[3], v[4], v[5], 0.f, 0.f};
  float x4[4], x2[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) x4[i] = (b4 ? w[i + 4] : w[i]) + __shfl_xor_sync(0xffffffffu, b4 ? w[i] : w[i + 4], 16);
#pragma unroll
  for (int i = 0; i < 2; ++i) x2[i] = (b3 ? x4[i + 2] : x4[i]) + __shfl_xor_sync(0xffffffffu, b3 ? x4[i] : x4[i + 2], 8);
  float x = (b2 ? x2[1] : x2[0]) + __shfl_xor_sync(0xffffffffu, b2 ? x2[0] : x2[1], 4);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  if (nt == 32) {
    __syncwarp();
  } else {
    if ((lane & 3) == 0) red[(t >> 5) * 8 + (lane >> 2)] = x;
    group_sync(g, nt);
    x = 0.f;
    for (int i = lane & 3; i < (nt >> 5); i += 4) x += red[i * 8 + (lane >> 2)];
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, x, 4 * i);
}

// ---------------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------------
template <typename T, typename TH, int K, int MAXT>
__global__ void __launch_bounds__(MAXT) fwd_kernel(const FwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[kMaxGroups][kMaxStages];
  __shared__ float red[kMaxGroups][3][32];
  __shared__ int abort_word;
  Walk w;
  w.init(ring, smem, bars, &abort_word, a.w_post, a.scale, a.w_pre, a.D, a.rows);
  const float* sw = reinterpret_cast<const float*>(smem);
  const float* wn = sw + a.D;
  const int nt = ring.nt, t = w.t, g = w.g;
  const float invD = 1.0f / (float)a.D;
#pragma unroll 1
  for (long i = 0; i < w.mine; ++i) {
    const long at = (w.row0 + i * w.step) * a.D;
    const unsigned char* base = w.wait(ring);
    const T* sy = reinterpret_cast<const T*>(base + ring.off[0]);
    const TH* sh = reinterpret_cast<const TH*>(base + ring.off[1]);
    const T* sz = reinterpret_cast<const T*>(base + ring.off[2]);
    Piece8<TH> hv[K];
    Piece8<T> zv[K];
    f2_t v[K][4];
    f2_t q2 = 0;                       // (+0, +0)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + t) * 8;
      Piece8<T> y;
      y.zero();
      hv[k].zero();
      zv[k].zero();
      if (c < a.D) {
        y.load(sy + c);
        hv[k].load(sh + c);
        if (a.z) zv[k].load(sz + c);
      }
      y.get(v[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) q2 = fma2(v[k][e], v[k][e], q2);
    }
    float ry = 1.f;
    // without the second norm's sync the next row's sums go to the other buffer
    if (a.w_post) ry = rsqrtf(fmaf(group_sum(hsum2(q2), red[g][a.w_pre ? 0 : (int)(i & 1)], g, t, nt), invD, a.eps));
    else group_sync(g, nt);
    w.refill(ring, i);
    const f2_t ry2 = splat2(ry);
    q2 = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + t) * 8;
      if (c < a.D) {
        f2_t f[4], u[4];
        if (a.z) {
          zv[k].get(f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float z0, z1;
            up2(f[e], z0, z1);
            v[k][e] = mul2(v[k][e], mul2(f[e], pk2(sigm(z0), sigm(z1))));
          }
        }
        ldv(sw + c, u);
        hv[k].get(f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[k][e] = fma2(mul2(v[k][e], ry2), u[e], f[e]);
          q2 = fma2(v[k][e], v[k][e], q2);
        }
        Piece8<TH>::store(static_cast<TH*>(a.h_out) + at + c, v[k]);
      }
    }
    if (a.w_pre) {
      const f2_t rh2 = splat2(rsqrtf(fmaf(group_sum(hsum2(q2), red[g][2], g, t, nt), invD, a.eps)));
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * nt + t) * 8;
        if (c < a.D) {
          f2_t u[4];
          ldv(wn + c, u);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[k][e] = mul2(v[k][e], mul2(rh2, u[e]));
          Piece8<T>::store(static_cast<T*>(a.x) + at + c, v[k]);
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && abort_word) record_error(kErrTimeout);
}

// ---------------------------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------------------------
// One sync a row: mean(w_post n' y), which needs dh, is linear in the row's scalars,
//   sum w_post n' y = sum g h'' + r sum g w_pre x' - r (r^2 mean(w_pre x' h')) sum g h',  g = s SiLU(z) w_post y,
// so all six sums are taken in one go before any output is formed.
template <typename T, typename TH, int K, int MAXT>
__global__ void __launch_bounds__(MAXT) bwd_kernel(const BwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[kMaxGroups][kMaxStages];
  __shared__ float red[2][256];          // [warps][8], a group's at its first warp; rows alternate
  __shared__ int abort_word;
  Walk w;
  w.init(ring, smem, bars, &abort_word, a.w_post, a.scale, a.w_pre, a.D, a.rows);
  const float* sw = reinterpret_cast<const float*>(smem);
  const float* wn = sw + a.D;
  const int nt = ring.nt, t = w.t, g = w.g;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  f2_t ga[K][4], gn[K][4];               // the column sums A and dw_pre over this group's rows
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) ga[k][e] = gn[k][e] = 0;
  const float invD = 1.0f / (float)a.D;
  const f2_t one = splat2(1.f), minus = splat2(-1.f);
#pragma unroll 1
  for (long i = 0; i < w.mine; ++i) {
    const long at = (w.row0 + i * w.step) * a.D;
    const unsigned char* base = w.wait(ring);
    Piece8<T> yv[K], zv[K], dx[K];
    Piece8<TH> hv[K], dh[K];
    f2_t sg[K][4];                       // sigmoid(z)
    f2_t q[6] = {0, 0, 0, 0, 0, 0};      // y^2, h'^2, w_pre x' h', and the sums of g h'', g w_pre x', g h'
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + t) * 8;
      yv[k].zero();
      zv[k].zero();
      dx[k].zero();
      hv[k].zero();
      dh[k].zero();
#pragma unroll
      for (int e = 0; e < 4; ++e) sg[k][e] = 0;
      if (c < a.D) {
        f2_t y[4], gv[4], f[4];
        yv[k].load(reinterpret_cast<const T*>(base + ring.off[0]) + c);
        yv[k].get(y);
        ldv(sw + c, gv);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q[0] = fma2(y[e], y[e], q[0]);
          gv[e] = mul2(gv[e], y[e]);
        }
        if (a.z) {
          zv[k].load(reinterpret_cast<const T*>(base + ring.off[2]) + c);
          zv[k].get(f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float z0, z1;
            up2(f[e], z0, z1);
            sg[k][e] = pk2(sigm(z0), sigm(z1));
            gv[e] = mul2(gv[e], mul2(f[e], sg[k][e]));
          }
        }
        if (a.dh_in) {
          dh[k].load(reinterpret_cast<const TH*>(base + ring.off[3]) + c);
          dh[k].get(f);
#pragma unroll
          for (int e = 0; e < 4; ++e) q[3] = fma2(gv[e], f[e], q[3]);
        }
        if (pre) {
          hv[k].load(reinterpret_cast<const TH*>(base + ring.off[1]) + c);
          dx[k].load(reinterpret_cast<const T*>(base + ring.off[4]) + c);
          f2_t d[4], u[4];
          hv[k].get(f);
          dx[k].get(d);
          ldv(wn + c, u);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f2_t wx = mul2(u[e], d[e]);
            q[1] = fma2(f[e], f[e], q[1]);
            q[2] = fma2(wx, f[e], q[2]);
            q[4] = fma2(gv[e], wx, q[4]);
            q[5] = fma2(gv[e], f[e], q[5]);
          }
        }
      }
    }
    float s[6];
#pragma unroll
    for (int e = 0; e < 6; ++e) s[e] = hsum2(q[e]);
    group_sum6(s, red[i & 1] + g * (nt >> 5) * 8, g, t, nt);
    w.refill(ring, i);
    const float ry = post ? rsqrtf(fmaf(s[0], invD, a.eps)) : 1.f;
    const float rh = pre ? rsqrtf(fmaf(s[1], invD, a.eps)) : 0.f;
    const float mx = rh * rh * s[2] * invD;
    const float qd = fmaf(rh, fmaf(-mx, s[5], s[4]), s[3]);
    const f2_t ry2 = splat2(ry), rh2 = splat2(rh), mx2 = splat2(-mx);
    const f2_t my2 = splat2(post ? -ry * ry * ry * qd * invD : 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * nt + t) * 8;
      if (c < a.D) {
        f2_t d[4], y[4], f[4], v[4];
        dh[k].get(d);
        if (pre) {
          hv[k].get(f);
          dx[k].get(v);
          ldv(wn + c, y);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            gn[k][e] = fma2(mul2(v[e], rh2), f[e], gn[k][e]);
            d[e] = fma2(rh2, fma2(v[e], y[e], mul2(f[e], mx2)), d[e]);
          }
        }
        Piece8<TH>::store(static_cast<TH*>(a.dh) + at + c, d);
        yv[k].get(y);
        ldv(sw + c, v);
        if (a.z) {
          f2_t z[4];
          zv[k].get(z);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f2_t gate = mul2(z[e], sg[k][e]), yr = mul2(y[e], ry2), as = mul2(d[e], v[e]);
            f[e] = mul2(mul2(as, yr), mul2(sg[k][e], fma2(z[e], fma2(sg[k][e], minus, one), one)));
            ga[k][e] = fma2(mul2(d[e], gate), yr, ga[k][e]);
            d[e] = fma2(y[e], my2, mul2(mul2(as, gate), ry2));
          }
          Piece8<T>::store(static_cast<T*>(a.dz) + at + c, f);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ga[k][e] = fma2(d[e], mul2(y[e], ry2), ga[k][e]);
            d[e] = fma2(y[e], my2, mul2(mul2(d[e], v[e]), ry2));
          }
        }
        Piece8<T>::store(static_cast<T*>(a.dy) + at + c, d);
      }
    }
  }
  float* part = a.part + ((long)blockIdx.x * ring.groups + g) * 2 * a.D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * nt + t) * 8;
    if (c < a.D) {
      Piece8<float>::store(part + c, ga[k]);
      Piece8<float>::store(part + a.D + c, gn[k]);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && abort_word) record_error(kErrTimeout);
}

// Column sums of the parts, in a fixed order: 32 columns x 16 slices of the parts per block, then
// the 16 slices.  blockIdx.y: A (giving dw_post and dscale) or dw_pre.
__global__ void __launch_bounds__(512) column_sum_kernel(const float* __restrict__ part, int parts, int D,
                                                         const float* __restrict__ w_post, const float* __restrict__ scale,
                                                         float* dw_post, float* dw_pre, float* dscale) {
  __shared__ float s[16][33];
  if (blockIdx.y == 0 ? !dw_post && !dscale : !dw_pre) return;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < D) {
    const float* p = part + (long)blockIdx.y * D + c;
#pragma unroll 4
    for (int i = slice; i < parts; i += 16) v += p[(long)i * 2 * D];
  }
  s[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && c < D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][lane];
    if (blockIdx.y == 1) {
      dw_pre[c] = t;
    } else {
      if (dw_post) dw_post[c] = t * (scale ? scale[c] : 1.f);
      if (dscale) dscale[c] = t * (w_post ? w_post[c] : 1.f);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// any width and alignment: the row is read again in each pass (from L1 / L2)
// ---------------------------------------------------------------------------------------------
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
  float* ga = a.part + (long)blockIdx.x * 2 * a.D;
  float* gn = ga + a.D;
  for (int c = tid; c < a.D; c += kLoopThreads) ga[c] = gn[c] = 0.f;
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
      ga[c] = fmaf(dh * gate, yr, ga[c]);
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
