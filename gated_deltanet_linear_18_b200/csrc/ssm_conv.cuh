// Short causal convolution of the state space block: per channel c
//   out_t = SiLU(bias[c] + sum_{j=0..3} w[c][j] u_{t-3+j})
// with the three rows before the sequence taken from a carried history (zeros without one), and
// the last three raw rows written out as the history after the call.
//
// Each raw row is read once and each result written once.  In bf16 neither the special functions (two a value, 52 % of
// their pipe) nor the issue slots (60 %) are full: with 16 warps an SM, what is left is latency.  One thread owns VEC neighbouring channels (16 bytes) and a tile of consecutive rows: its taps
// and the three-row window stay in registers, and the next kConvBatch rows are loaded while the present
// ones are computed.  A tile is as long as one wave of CTAs allows, since a thread's 5 VEC taps and biases
// are as many bytes as ten rows of bf16.  Only the window's three rows are read twice.
// Measured, 16384 x 6144: bf16 88-90 us = 4.5 TB/s (a copy: 6.45), 161 with tiles of 32 rows; fp32 175 us = 4.6 TB/s.  Rows ahead and CTAs an SM: 2 and 4 95 us, 2 and 5 104, 4 and 5 125, 8 and 3 92; 8-byte
// pieces with twice the warps 104; a branch for four rows of one sequence, without the question of each
// row's sequence, 107 (it spills).
#pragma once

#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

constexpr int kConvThreads = 128;
constexpr int kConvBatch = 4;       // rows loaded ahead

// Rows [a, b) of sequence s, clamped like row_span; the same for dense and packed tensors.
__device__ __forceinline__ void seq_rows(const int* __restrict__ cu, int s, int T, int max_len,
                                         long& a, long& b) {
  const RowSpan sp = row_span(cu, s, T, max_len);
  a = sp.row0;
  b = sp.row0 + sp.len;
}

// The last sequence whose first row is at most r (packed offsets are non-decreasing), so that
// empty sequences before it are passed over.
__device__ __forceinline__ int seq_of_row(const int* __restrict__ cu, int nseq, int T, long r) {
  if (!cu) return (int)(r / T);
  int lo = 0, hi = nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long)cu[mid] <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// VEC neighbouring channels of a row as loaded, and as pairs for the paired fp32 instructions (a single channel
// leaves the second of its pair unused).
template <typename T, int VEC> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(f2_t (&f)[4]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pk2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const f2_t (&f)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      up2(f[i], a, b);
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <> struct Piece<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(f2_t (&f)[2]) const {
    f[0] = pk2(v.x, v.y);
    f[1] = pk2(v.z, v.w);
  }
  static __device__ __forceinline__ void store(float* p, const f2_t (&f)[2]) {
    float4 o;
    up2(f[0], o.x, o.y);
    up2(f[1], o.z, o.w);
    *reinterpret_cast<float4*>(p) = o;
  }
};
template <typename T> struct Piece<T, 1> {   // any alignment
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void get(f2_t (&f)[1]) const { f[0] = pk2(to_f(v), 0.f); }
  static __device__ __forceinline__ void store(T* p, const f2_t (&f)[1]) {
    float a, b;
    up2(f[0], a, b);
    *p = from_f<T>(a);
  }
};

struct ConvArgs {
  const void* x;        // [rows, C], rows ldx values apart
  long ldx;
  const float *w, *bias;
  const void* hist_in;  // [nseq, 3, C] or null
  void *out, *hist_out; // [rows, C]; [nseq, 3, C] or null
  const int* cu;        // null: nseq sequences of T rows
  int nseq, T, max_len, C;
  int tile;             // rows of a thread, a multiple of kConvBatch
  int w_vec;            // w and bias allow 16-byte loads
};

// grid (row tiles + 1, channel blocks): the last row tile hands the history of sequences without
// rows on.
template <typename T, int VEC>
__global__ void __launch_bounds__(kConvThreads) conv_kernel(const ConvArgs a) {
  const int c = (blockIdx.y * kConvThreads + threadIdx.x) * VEC;
  if (c >= a.C) return;
  using Pc = Piece<T, VEC>;
  constexpr int NP = (VEC + 1) / 2;
  const T* __restrict__ x = static_cast<const T*>(a.x) + c;
  const T* __restrict__ hin = a.hist_in ? static_cast<const T*>(a.hist_in) + c : nullptr;
  T* __restrict__ hout = a.hist_out ? static_cast<T*>(a.hist_out) + c : nullptr;
  T* __restrict__ out = static_cast<T*>(a.out) + c;
  const long C = a.C;

  if (blockIdx.x == gridDim.x - 1) {
    if (!hout) return;
    for (int s = 0; s < a.nseq; ++s) {
      long r0, r1;
      seq_rows(a.cu, s, a.T, a.max_len, r0, r1);
      if (r1 > r0) continue;
      for (int i = 0; i < 3; ++i) {
        f2_t f[NP] = {};
        if (hin) {
          Pc p;
          p.load(hin + (3L * s + i) * C);
          p.get(f);
        }
        Pc::store(hout + (3L * s + i) * C, f);
      }
    }
    return;
  }

  const long rows = a.cu ? (long)a.T : (long)a.nseq * a.T;
  long first = (long)blockIdx.x * a.tile;
  const long last = min(first + a.tile, rows);
  int s = seq_of_row(a.cu, a.nseq, a.T, first);
  long r0, r1;
  seq_rows(a.cu, s, a.T, a.max_len, r0, r1);
  first = max(first, r0);              // rows before the first sequence are in none
  if (first >= last) return;

  f2_t w[4][NP], b[NP];
  {
    float ws[4][2 * NP] = {}, bs[2 * NP] = {};
    if (VEC > 1 && a.w_vec) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(a.w + 4L * (c + i));
        ws[0][i] = v.x; ws[1][i] = v.y; ws[2][i] = v.z; ws[3][i] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) ws[j][i] = a.w[4L * (c + i) + j];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) bs[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      b[i] = pk2(bs[2 * i], bs[2 * i + 1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j][i] = pk2(ws[j][2 * i], ws[j][2 * i + 1]);
    }
  }
  // window: the raw rows t-3, t-2, t-1
  f2_t w0[NP], w1[NP], w2[NP];
  auto prev = [&](long r, int back, f2_t (&f)[NP]) {   // the raw row `back` rows before row r
    const long t = r - back;
    Pc p;
    if (t >= r0) {
      p.load(x + t * a.ldx);
      p.get(f);
    } else if (hin && r0 - t <= 3) {
      p.load(hin + (3L * s + 3 - (r0 - t)) * C);
      p.get(f);
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) f[i] = 0;
    }
  };
  prev(first, 3, w0);
  prev(first, 2, w1);
  prev(first, 1, w2);

  Pc next[kConvBatch];
  auto fetch = [&](long base) {
#pragma unroll
    for (int i = 0; i < kConvBatch; ++i)
      if (base + i < last) next[i].load(x + (base + i) * a.ldx);
  };
  fetch(first);
#pragma unroll 1
  for (long base = first; base < last; base += kConvBatch) {
    Pc now[kConvBatch];
#pragma unroll
    for (int i = 0; i < kConvBatch; ++i) now[i] = next[i];
    fetch(base + kConvBatch);
#pragma unroll
    for (int i = 0; i < kConvBatch; ++i) {
      const long r = base + i;
      if (r < last) {
        if (r >= r1) {               // the next sequence with rows (rows in none are left alone)
          while (r >= r1 && s + 1 < a.nseq) {
            long n0, n1;
            seq_rows(a.cu, s + 1, a.T, a.max_len, n0, n1);
            if (n0 > r) break;
            ++s;
            r0 = n0;
            r1 = n1;
          }
          prev(r, 3, w0);
          prev(r, 2, w1);
          prev(r, 1, w2);
        }
        f2_t u[NP], o[NP];
        now[i].get(u);
        if (r >= r0 && r < r1) {
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            f2_t acc = fma2(w[0][e], w0[e], b[e]);
            acc = fma2(w[1][e], w1[e], acc);
            acc = fma2(w[2][e], w2[e], acc);
            acc = fma2(w[3][e], u[e], acc);
            float s0, s1;
            up2(acc, s0, s1);
            o[e] = mul2(acc, pk2(sigmoid(s0), VEC > 1 ? sigmoid(s1) : 0.f));
          }
          Pc::store(out + r * C, o);
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          w0[e] = w1[e];
          w1[e] = w2[e];
          w2[e] = u[e];
        }
        if (hout && r == r1 - 1) {
          Pc::store(hout + (3L * s + 0) * C, w0);
          Pc::store(hout + (3L * s + 1) * C, w1);
          Pc::store(hout + (3L * s + 2) * C, w2);
        }
      }
    }
  }
}

}  // namespace ssm
}  // namespace gdn
