// C ABI of the norms around a block (declared in include/gdn.h): argument checks, kernel choice
// and launches.
#include <algorithm>

#include "gdn.h"
#include "block_norm.cuh"

using namespace gdn;

namespace {

constexpr int kSms = 148;
constexpr uint32_t kSmem = 216 * 1024;   // shared memory of a CTA given to vectors and row stages

bool elem_aligned(const void* p, size_t el) { return (reinterpret_cast<uintptr_t>(p) & (el - 1)) == 0; }
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// How a width is walked: `k` pieces of 8 columns a thread, groups of `nt` threads, `groups` a CTA and
// `stages` row stages a group.
struct Shape {
  int k, nt, groups, stages;
};
// One piece a thread up to 2048 columns, two above (8192 x 6144 bf16: the forward 100 us with two, 111 with three or
// four; the backward 203 with two in 384 threads, 218 with one in 768).  As many groups as make 768 threads (512 where
// the backward's two pieces need 128 registers), fewer where a row stage for each does not fit beside the vectors.
// groups = 0: the width is not walked.
int pieces(int D) { return D <= 2048 ? 1 : 2; }
int group_threads(int D) {
  const int k = pieces(D);
  return ((D / 8 + k - 1) / k + 31) / 32 * 32;
}
int most_groups(int D, bool backward) {
  return std::max(1, std::min(bn::kMaxGroups, (backward && pieces(D) == 2 ? 512 : 768) / group_threads(D)));
}
Shape shape_of(int D, uint32_t row_bytes, bool backward) {
  if (D % 8 != 0 || D > 8192) return Shape{0, 0, 0, 0};
  const uint32_t room = kSmem - 8u * D;
  int groups = most_groups(D, backward);
  while (groups > 1 && room / (groups * row_bytes) < 1) --groups;
  const int stages = (int)std::min<uint32_t>(bn::kMaxStages, room / (groups * row_bytes));
  return stages < 1 ? Shape{0, 0, 0, 0} : Shape{pieces(D), group_threads(D), groups, stages};
}
// Parts of the backward's column sums that the workspace holds: the most of its two kernels, each of which
// writes one a group or CTA.
constexpr int kLoopCtas = kSms * 4;
long bwd_parts(long rows, int D) {
  const long walked = D % 8 == 0 && D <= 8192 ? std::min<long>(rows, kSms) * most_groups(D, true) : 0;
  return std::max(walked, std::min<long>(rows, kLoopCtas));
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

template <auto kern, typename Args>
gdn_status launch_ring(const Args& a, bn::Ring ring, const Shape& s, cudaStream_t st) {
  ring.stages = s.stages;
  ring.groups = s.groups;
  ring.nt = s.nt;
  const uint32_t smem = 8u * a.D + s.groups * s.stages * ring.stage_bytes;
  if (!allow_smem<kern, (int)kSmem>()) return GDN_ERR_CUDA;
  kern<<<(unsigned)std::min<long>(a.rows, kSms), s.groups * s.nt, smem, st>>>(a, ring);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, typename TH>
gdn_status fwd(const bn::FwdArgs& a, bool vec, cudaStream_t st) {
  bn::Ring ring{};
  const uint32_t bt = (uint32_t)a.D * sizeof(T), bh = (uint32_t)a.D * sizeof(TH);
  Shape s{0, 0, 0, 0};
  if (vec) {
    ring_add(ring, 0, a.y, bt);
    ring_add(ring, 1, a.h, bh);
    ring_add(ring, 2, a.z, bt);
    s = shape_of(a.D, ring.stage_bytes, false);
  }
  if (s.groups == 0) {
    bn::fwd_loop_kernel<T, TH><<<(unsigned)std::min<long>(a.rows, kSms * 8), bn::kLoopThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  }
  if (s.k == 1) return launch_ring<bn::fwd_kernel<T, TH, 1, 768>>(a, ring, s, st);
  return launch_ring<bn::fwd_kernel<T, TH, 2, 768>>(a, ring, s, st);
}

template <typename T, typename TH>
gdn_status bwd(const bn::BwdArgs& a, bool vec, float* dw_post, float* dw_pre, float* dscale, cudaStream_t st) {
  bn::Ring ring{};
  const uint32_t bt = (uint32_t)a.D * sizeof(T), bh = (uint32_t)a.D * sizeof(TH);
  Shape sh{0, 0, 0, 0};
  if (vec) {
    ring_add(ring, 0, a.y, bt);
    ring_add(ring, 1, a.w_pre ? a.h : nullptr, bh);
    ring_add(ring, 2, a.z, bt);
    ring_add(ring, 3, a.dh_in, bh);
    ring_add(ring, 4, a.w_pre ? a.dx : nullptr, bt);
    sh = shape_of(a.D, ring.stage_bytes, true);
  }
  gdn_status s = GDN_OK;
  long parts;
  if (sh.groups == 0) {
    parts = std::min<long>(a.rows, kLoopCtas);
    bn::bwd_loop_kernel<T, TH><<<(unsigned)parts, bn::kLoopThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) s = GDN_ERR_CUDA;
  } else {
    parts = std::min<long>(a.rows, kSms) * sh.groups;
    s = sh.k == 1 ? launch_ring<bn::bwd_kernel<T, TH, 1, 768>>(a, ring, sh, st)
        : sh.groups * sh.nt <= 384 ? launch_ring<bn::bwd_kernel<T, TH, 2, 384>>(a, ring, sh, st)
                                   : launch_ring<bn::bwd_kernel<T, TH, 2, 512>>(a, ring, sh, st);
  }
  if (s != GDN_OK) return s;
  if (!dw_post && !dw_pre && !dscale) return GDN_OK;
  bn::column_sum_kernel<<<dim3((unsigned)((a.D + 31) / 32), 2), 512, 0, st>>>(a.part, (int)parts, a.D, a.w_post, a.scale,
                                                                             dw_post, dw_pre, dscale);
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
  return (size_t)bwd_parts(rows, D) * 2 * D * sizeof(float);
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
