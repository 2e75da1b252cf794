// C ABI of the norms around a block (declared in include/gdn.h): argument checks, kernel choice
// and launches.
#include <algorithm>

#include "gdn.h"
#include "block_norm.cuh"

using namespace gdn;

namespace {

constexpr int kSms = 148;
constexpr uint32_t kStageBytes = 200 * 1024;   // shared memory of an SM given to row stages

bool elem_aligned(const void* p, size_t el) { return (reinterpret_cast<uintptr_t>(p) & (el - 1)) == 0; }
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// How a width is walked: `k` pieces of 8 columns a thread, `threads` threads, `ctas` per SM.
struct Shape {
  int k, threads, ctas;
};
// One piece a thread up to 2048 columns, two up to 8192 (512 threads); enough CTAs on an SM to
// give it about 512 threads.
Shape shape_of(int D) {
  const int nv = D / 8, k = nv <= 256 ? 1 : 2;
  const int threads = ((nv + k - 1) / k + 31) / 32 * 32;
  return Shape{k, threads, std::max(1, std::min(8, 512 / threads))};
}
bool ring_fits(int D, uint32_t row_bytes) {
  return D % 8 == 0 && D <= 8192 && row_bytes <= kStageBytes / shape_of(D).ctas;
}
// CTAs of the backward: as many as run at once, at most one per row; the loop kernel's walk four a SM.
long bwd_ctas(long rows, int D) {
  const int per = D % 8 == 0 && D <= 8192 ? shape_of(D).ctas : 4;
  return std::min<long>(rows, (long)kSms * per);
}

void ring_add(bn::Ring& r, int i, const void* p, uint32_t bytes) {
  r.off[i] = r.stage_bytes;
  if (!p) return;
  r.src[r.n] = static_cast<const char*>(p);
  r.bytes[r.n] = bytes;
  r.at[r.n] = r.stage_bytes;
  r.stage_bytes += bytes;
  ++r.n;
}

template <typename Kern, typename Args>
gdn_status launch_ring(Kern kern, const Args& a, bn::Ring ring, const Shape& s, long ctas, cudaStream_t st) {
  ring.stages = (int)std::min<uint32_t>(4, kStageBytes / s.ctas / ring.stage_bytes);
  const uint32_t smem = ring.stages * ring.stage_bytes;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return GDN_ERR_CUDA;
  kern<<<(unsigned)ctas, s.threads, smem, st>>>(a, ring);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, typename TH>
gdn_status fwd(const bn::FwdArgs& a, bool vec, cudaStream_t st) {
  bn::Ring ring{};
  const uint32_t bt = (uint32_t)a.D * sizeof(T), bh = (uint32_t)a.D * sizeof(TH);
  if (vec) {
    ring_add(ring, 0, a.y, bt);
    ring_add(ring, 1, a.h, bh);
    ring_add(ring, 2, a.z, bt);
  }
  if (!vec || !ring_fits(a.D, ring.stage_bytes)) {
    bn::fwd_loop_kernel<T, TH><<<(unsigned)std::min<long>(a.rows, kSms * 8), bn::kLoopThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  }
  const Shape s = shape_of(a.D);
  const long ctas = std::min<long>(a.rows, (long)kSms * s.ctas);
  if (s.k == 1) return launch_ring(bn::fwd_kernel<T, TH, 1, 256>, a, ring, s, ctas, st);
  if (s.threads <= 384) return launch_ring(bn::fwd_kernel<T, TH, 2, 384>, a, ring, s, ctas, st);
  return launch_ring(bn::fwd_kernel<T, TH, 2, 512>, a, ring, s, ctas, st);
}

template <typename T, typename TH>
gdn_status bwd(const bn::BwdArgs& a, bool vec, float* dw_post, float* dw_pre, float* dscale, cudaStream_t st) {
  bn::Ring ring{};
  const uint32_t bt = (uint32_t)a.D * sizeof(T), bh = (uint32_t)a.D * sizeof(TH);
  if (vec) {
    ring_add(ring, 0, a.y, bt);
    ring_add(ring, 1, a.w_pre ? a.h : nullptr, bh);
    ring_add(ring, 2, a.z, bt);
    ring_add(ring, 3, a.dh_in, bh);
    ring_add(ring, 4, a.w_pre ? a.dx : nullptr, bt);
  }
  const long ctas = bwd_ctas(a.rows, a.D);
  gdn_status s = GDN_OK;
  if (!vec || !ring_fits(a.D, ring.stage_bytes)) {
    bn::bwd_loop_kernel<T, TH><<<(unsigned)ctas, bn::kLoopThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) s = GDN_ERR_CUDA;
  } else {
    const Shape sh = shape_of(a.D);
    s = sh.k == 1 ? launch_ring(bn::bwd_kernel<T, TH, 1, 256>, a, ring, sh, ctas, st)
        : sh.threads <= 384 ? launch_ring(bn::bwd_kernel<T, TH, 2, 384>, a, ring, sh, ctas, st)
                            : launch_ring(bn::bwd_kernel<T, TH, 2, 512>, a, ring, sh, ctas, st);
  }
  if (s != GDN_OK) return s;
  if (!dw_post && !dw_pre && !dscale) return GDN_OK;
  bn::column_sum_kernel<<<dim3((unsigned)((a.D + 31) / 32), 3), 512, 0, st>>>(a.part, (int)ctas, a.D, dw_post,
                                                                             dw_pre, dscale);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status check_types(gdn_dtype t, gdn_dtype h) {
  if ((t != GDN_F32 && t != GDN_BF16) || (h != GDN_F32 && h != GDN_BF16)) return GDN_ERR_INVALID_ARG;
  return t == GDN_F32 && h == GDN_BF16 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

}  // namespace

namespace gdn {
// gdn_check_error's share of this translation unit: reads and clears its error word.
bool norm_take_error(unsigned int* word) {
  const unsigned int zero = 0;
  *word = 0;
  if (cudaMemcpyFromSymbol(word, g_error_word, sizeof(*word)) != cudaSuccess) return false;
  return *word == 0 || cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero)) == cudaSuccess;
}
}  // namespace gdn

extern "C" {

gdn_status gdn_block_norm(const void* y, const void* h, const void* z, const float* w_post, const float* w_pre,
                          const float* res_scale, void* h_out, void* x, long long rows, int D, float eps,
                          gdn_dtype dtype, gdn_dtype h_dtype, gdn_stream_t stream) {
  if (rows < 0 || D <= 0 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  const gdn_status s = check_types(dtype, h_dtype);
  if (s != GDN_OK) return s;
  if (rows == 0) return GDN_OK;
  if ((w_pre == nullptr) != (x == nullptr)) return GDN_ERR_INVALID_ARG;
  const size_t et = dtype == GDN_F32 ? 4 : 2, eh = h_dtype == GDN_F32 ? 4 : 2;
  if (!y || !h || !h_out || h_out == h || h_out == y || (x && (x == y || x == h || x == z)) || (z && z == h_out))
    return GDN_ERR_INVALID_ARG;
  if (!elem_aligned(y, et) || !elem_aligned(h, eh) || !elem_aligned(z, et) || !elem_aligned(h_out, eh) ||
      !elem_aligned(x, et) || !elem_aligned(w_post, 4) || !elem_aligned(w_pre, 4) || !elem_aligned(res_scale, 4))
    return GDN_ERR_INVALID_ARG;
  const bool vec = D % 8 == 0 && al16(y) && al16(h) && al16(z) && al16(h_out) && al16(x);
  const bn::FwdArgs a{y, h, z, w_post, w_pre, res_scale, h_out, x, (long)rows, D, eps};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == GDN_F32) return fwd<float, float>(a, vec, st);
  if (h_dtype == GDN_F32) return fwd<__nv_bfloat16, float>(a, vec, st);
  return fwd<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
}

size_t gdn_block_norm_bwd_workspace_bytes(long long rows, int D) {
  if (rows <= 0 || D <= 0) return 0;
  return (size_t)bwd_ctas(rows, D) * 3 * D * sizeof(float);
}

gdn_status gdn_block_norm_bwd(const void* y, const void* h_out, const void* z, const void* dh_out, const void* dx,
                              const float* w_post, const float* w_pre, const float* res_scale, void* dy, void* dh,
                              void* dz, float* dw_post, float* dw_pre, float* dres_scale, void* workspace,
                              size_t workspace_bytes, long long rows, int D, float eps, gdn_dtype dtype,
                              gdn_dtype h_dtype, gdn_stream_t stream) {
  if (rows < 0 || D <= 0 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  const gdn_status s = check_types(dtype, h_dtype);
  if (s != GDN_OK) return s;
  if ((w_post == nullptr) != (dw_post == nullptr) || (w_pre == nullptr) != (dw_pre == nullptr) ||
      (res_scale == nullptr) != (dres_scale == nullptr) || (z == nullptr) != (dz == nullptr))
    return GDN_ERR_INVALID_ARG;
  if (!elem_aligned(w_post, 4) || !elem_aligned(w_pre, 4) || !elem_aligned(res_scale, 4) ||
      !elem_aligned(dw_post, 4) || !elem_aligned(dw_pre, 4) || !elem_aligned(dres_scale, 4))
    return GDN_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {
    for (float* g : {dw_post, dw_pre, dres_scale})
      if (g && cudaMemsetAsync(g, 0, (size_t)D * sizeof(float), st) != cudaSuccess) return GDN_ERR_CUDA;
    return GDN_OK;
  }
  if (!y || !dy || !dh || (w_pre && (!h_out || !dx)) || (!w_pre && !dh_out)) return GDN_ERR_INVALID_ARG;
  const size_t et = dtype == GDN_F32 ? 4 : 2, eh = h_dtype == GDN_F32 ? 4 : 2;
  const void* in_t[] = {y, z, dx};
  const void* in_h[] = {h_out, dh_out};
  const void* outs[] = {dy, dh, dz};
  bool vec = D % 8 == 0;
  for (const void* p : in_t) {
    if (!elem_aligned(p, et)) return GDN_ERR_INVALID_ARG;
    vec = vec && al16(p);
    for (const void* o : outs)
      if (p && p == o) return GDN_ERR_INVALID_ARG;
  }
  for (const void* p : in_h) {
    if (!elem_aligned(p, eh)) return GDN_ERR_INVALID_ARG;
    vec = vec && al16(p);
    for (const void* o : outs)
      if (p && p == o) return GDN_ERR_INVALID_ARG;
  }
  if (!elem_aligned(dy, et) || !elem_aligned(dh, eh) || !elem_aligned(dz, et)) return GDN_ERR_INVALID_ARG;
  vec = vec && al16(dy) && al16(dh) && al16(dz);
  if (!workspace || !al16(workspace) || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < gdn_block_norm_bwd_workspace_bytes(rows, D))
    return GDN_ERR_INVALID_ARG;
  const bn::BwdArgs a{y, w_pre ? h_out : nullptr, z, dh_out, w_pre ? dx : nullptr, w_post, w_pre, res_scale, dy, dh, dz,
                      static_cast<float*>(workspace), (long)rows, D, eps};
  if (dtype == GDN_F32) return bwd<float, float>(a, vec, dw_post, dw_pre, dres_scale, st);
  if (h_dtype == GDN_F32) return bwd<__nv_bfloat16, float>(a, vec, dw_post, dw_pre, dres_scale, st);
  return bwd<__nv_bfloat16, __nv_bfloat16>(a, vec, dw_post, dw_pre, dres_scale, st);
}

}  // extern "C"
