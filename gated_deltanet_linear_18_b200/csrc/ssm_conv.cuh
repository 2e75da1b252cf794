// Short causal convolution of the state space block: per channel c
//   out_t = SiLU(bias[c] + sum_{j=0..3} w[c][j] u_{t-3+j})
// with the three rows before the sequence taken from a carried history (zeros without one), and
// the last three raw rows written out as the history after the call.
//
// Bound by HBM: each raw row is read once and each result written once (the 12 operations and two
// special-function calls per value stay below that).  One thread owns VEC neighbouring channels
// (16 bytes) and R consecutive rows: its taps and the three-row window stay in registers, and the
// loads of kConvBatch rows are issued together before any of them is used.  Only the window's
// three rows are read twice (3 / R more reads, from L2).
#pragma once

#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

constexpr int kConvThreads = 128;
constexpr int kConvBatch = 8;       // rows whose loads are in flight together

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

template <typename T, int VEC> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <> struct Piece<float, 4> {
  float4 v;
  __device__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
  static __device__ void store(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <typename T> struct Piece<T, 1> {   // any alignment
  T v;
  __device__ void load(const T* p) { v = *p; }
  __device__ void get(float (&f)[1]) const { f[0] = to_f(v); }
  static __device__ void store(T* p, const float (&f)[1]) { *p = from_f<T>(f[0]); }
};

struct ConvArgs {
  const void* x;        // [rows, C], rows ldx values apart
  long ldx;
  const float *w, *bias;
  const void* hist_in;  // [nseq, 3, C] or null
  void *out, *hist_out; // [rows, C]; [nseq, 3, C] or null
  const int* cu;        // null: nseq sequences of T rows
  int nseq, T, max_len, C;
};

// grid (row tiles + 1, channel blocks): the last row tile hands the history of sequences without
// rows on.
template <typename T, int VEC, int R>
__global__ void __launch_bounds__(kConvThreads) conv_kernel(const ConvArgs a) {
  const int c = (blockIdx.y * kConvThreads + threadIdx.x) * VEC;
  if (c >= a.C) return;
  using Pc = Piece<T, VEC>;
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
        float f[VEC] = {};
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
  const long first = (long)blockIdx.x * R;
  const long last = min(first + R, rows);
  int s = seq_of_row(a.cu, a.nseq, a.T, first);
  long r0, r1;
  seq_rows(a.cu, s, a.T, a.max_len, r0, r1);

  float w[4][VEC], b[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    b[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j][i] = a.w[4L * (c + i) + j];
  }
  // window: the raw rows t-3, t-2, t-1
  float w0[VEC], w1[VEC], w2[VEC];
  auto prev = [&](long r, int back, float (&f)[VEC]) {   // the raw row `back` rows before row r
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
      for (int i = 0; i < VEC; ++i) f[i] = 0.f;
    }
  };
  prev(first, 3, w0);
  prev(first, 2, w1);
  prev(first, 1, w2);

  for (long base = first; base < last; base += kConvBatch) {
    Pc rowv[kConvBatch];
#pragma unroll
    for (int i = 0; i < kConvBatch; ++i)
      if (base + i < last) rowv[i].load(x + (base + i) * a.ldx);
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
        float u[VEC], o[VEC];
        rowv[i].get(u);
        if (r >= r0 && r < r1) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float acc = fmaf(w[0][e], w0[e], b[e]);
            acc = fmaf(w[1][e], w1[e], acc);
            acc = fmaf(w[2][e], w2[e], acc);
            acc = fmaf(w[3][e], u[e], acc);
            o[e] = silu(acc);
          }
          Pc::store(out + r * C, o);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
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
