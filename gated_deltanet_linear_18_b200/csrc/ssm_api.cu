// C ABI of the state space block (declared in include/gdn.h): argument checks, kernel choice and
// launches of the short convolution, the prompt scan and the token step.
#include <algorithm>

#include "gdn.h"
#include "ssm_conv.cuh"
#include "ssm_scan_simt.cuh"
#include "ssm_scan_tc.cuh"
#include "ssm_step.cuh"

using namespace gdn;

namespace {

using bf = __nv_bfloat16;

constexpr int kMostPacked = 1 << 30;   // rows of a packed call: a row and the tile or chunk behind it fit in 32 bits

bool valid_dtype(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }
bool supported_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
size_t elem(gdn_dtype t) { return t == GDN_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
gdn_status launch_status() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// ---------------------------------------------------------------------------------------------
// convolution
// ---------------------------------------------------------------------------------------------
template <typename T, int VEC>
gdn_status conv_launch(ssm::ConvArgs a, cudaStream_t st) {
  const long rows = a.cu ? (long)a.T : (long)a.nseq * a.T;
  const long per = (long)ssm::kConvThreads * VEC, blocks = (a.C + per - 1) / per;
  if (blocks > 65535) return GDN_ERR_UNSUPPORTED;
  // one wave of four CTAs an SM (128 registers), at least eight rows a thread
  const long wave = 148L * 4 / blocks;
  long tile = wave > 0 ? (rows + wave - 1) / wave : rows;
  tile = (std::max(8L, tile) + ssm::kConvBatch - 1) / ssm::kConvBatch * ssm::kConvBatch;
  tile = std::min(tile, 4096L);
  const long tiles = (rows + tile - 1) / tile + 1;
  if (tiles > 0x7fffffffL) return GDN_ERR_UNSUPPORTED;
  a.tile = (int)tile;
  a.w_vec = aligned(a.w, 16) && aligned(a.bias, 16);
  ssm::conv_kernel<T, VEC><<<dim3((unsigned)tiles, (unsigned)blocks), ssm::kConvThreads, 0, st>>>(a);
  return launch_status();
}

gdn_status conv_call(const void* x, long long ldx, const float* w, const float* bias, const void* hist_in, void* out,
                     void* hist_out, const int* cu, int nseq, int T, int max_len, int C, gdn_dtype dtype,
                     gdn_stream_t stream) {
  if (nseq < 0 || T < 0 || max_len < 0 || C <= 0 || !valid_dtype(dtype)) return GDN_ERR_INVALID_ARG;
  const long rows = cu ? (long)T : (long)nseq * T;
  if (cu && T > kMostPacked) return GDN_ERR_UNSUPPORTED;
  if (cu) max_len = std::min(max_len, T);
  if (nseq == 0 || (rows == 0 && !hist_out)) return GDN_OK;
  const size_t el = elem(dtype);
  if (rows > 0 && (!x || !out || !w || ldx < C)) return GDN_ERR_INVALID_ARG;
  if (!aligned(x, el) || !aligned(out, el) || !aligned(hist_in, el) || !aligned(hist_out, el) || !aligned(w, 4) ||
      !aligned(bias, 4))
    return GDN_ERR_INVALID_ARG;
  if ((hist_out && hist_out == hist_in) || (rows > 0 && out == x)) return GDN_ERR_INVALID_ARG;
  const int v = dtype == GDN_F32 ? 4 : 8;
  const bool vec = C % v == 0 && ldx % v == 0 && aligned(x, 16) && aligned(out, 16) && aligned(hist_in, 16) &&
                   aligned(hist_out, 16);
  const ssm::ConvArgs a{x, (long)ldx, w, bias, hist_in, out, hist_out, cu, nseq, T, max_len, C, 0, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == GDN_F32) return vec ? conv_launch<float, 4>(a, st) : conv_launch<float, 1>(a, st);
  return vec ? conv_launch<bf, 8>(a, st) : conv_launch<bf, 1>(a, st);
}

// ---------------------------------------------------------------------------------------------
// scan
// ---------------------------------------------------------------------------------------------
template <int N, int P, typename T>
gdn_status simt_launch(const ssm::ScanArgs& a, cudaStream_t st) {
  ssm::scan_simt_kernel<N, P, T>
      <<<dim3((unsigned)(a.H * (P < 32 ? 1 : P / 32)), (unsigned)a.nseq), ssm::kSimtThreads, 0, st>>>(a);
  return launch_status();
}
template <typename T, int N>
gdn_status simt_p(int P, const ssm::ScanArgs& a, cudaStream_t st) {
  switch (P) {
    case 16: return simt_launch<N, 16, T>(a, st);
    case 32: return simt_launch<N, 32, T>(a, st);
    case 64: return simt_launch<N, 64, T>(a, st);
    default: return simt_launch<N, 128, T>(a, st);
  }
}
template <typename T>
gdn_status simt_scan(int N, int P, const ssm::ScanArgs& a, cudaStream_t st) {
  switch (N) {
    case 16: return simt_p<T, 16>(P, a, st);
    case 32: return simt_p<T, 32>(P, a, st);
    case 64: return simt_p<T, 64>(P, a, st);
    default: return simt_p<T, 128>(P, a, st);
  }
}

gdn_status check_heads(int H, int G, int P, int N) {
  if (H <= 0 || G <= 0 || P <= 0 || N <= 0 || H % G != 0) return GDN_ERR_INVALID_ARG;
  if (!supported_dim(P) || !supported_dim(N) || H > 65535) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// total: rows of a packed call; -1: not known, or not packed
size_t scan_workspace(int nseq, int max_len, long total, int H, int G, int P, int N, gdn_dtype dtype) {
  if (nseq <= 0 || max_len <= 0 || dtype != GDN_BF16 || !ssm::tcs::supported(P, N)) return 0;
  return ssm::tcs::space(nseq, max_len, total, H, G, P, N).bytes;
}

gdn_status scan_call(ssm::ScanArgs a, int P, int N, void* workspace, size_t workspace_bytes, gdn_dtype dtype,
                     gdn_stream_t stream) {
  if (a.nseq < 0 || a.T < 0 || a.max_len < 0 || !valid_dtype(dtype)) return GDN_ERR_INVALID_ARG;
  const gdn_status s = check_heads(a.H, a.G, P, N);
  if (s != GDN_OK) return s;
  if (a.nseq == 0) return GDN_OK;
  if (a.nseq > 65535) return GDN_ERR_UNSUPPORTED;
  const long rows = a.cu ? (long)a.T : (long)a.nseq * a.T;
  if (a.cu && a.T > kMostPacked) return GDN_ERR_UNSUPPORTED;
  const size_t el = elem(dtype);
  if (!a.A_log || !aligned(a.A_log, 4) || !aligned(a.D, 4) || !aligned(a.dt_bias, 4) || !aligned(a.S0, 16) ||
      !aligned(a.S_T, 16) || (a.S_T && a.S_T == a.S0))
    return GDN_ERR_INVALID_ARG;
  const long HP = (long)a.H * P, GN = (long)a.G * N;
  if (rows > 0) {
    if (!a.x || !a.dt || !a.B || !a.C || !a.y) return GDN_ERR_INVALID_ARG;
    if (a.ldx < HP || a.lddt < a.H || a.ldb < GN || a.ldc < GN || (a.z && a.ldz < HP)) return GDN_ERR_INVALID_ARG;
    const void* in[] = {a.x, a.dt, a.B, a.C, a.z};
    for (const void* p : in)
      if (!aligned(p, el) || p == a.y) return GDN_ERR_INVALID_ARG;
    if (!aligned(a.y, 16)) return GDN_ERR_INVALID_ARG;
  }
  if (a.cu) a.max_len = std::min(a.max_len, a.T);
  const size_t need = scan_workspace(a.nseq, a.max_len, a.cu ? rows : -1L, a.H, a.G, P, N, dtype);
  if (need && rows > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return GDN_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const void* tiles[] = {a.x, a.B, a.C, a.z};
  bool tc = dtype == GDN_BF16 && ssm::tcs::supported(P, N) && rows > 0 && rows <= 0x7fffffffL - 2 * ssm::tcs::L &&
            a.max_len > 0 && a.max_len <= 65535 * ssm::tcs::L && a.ldx % 8 == 0 && a.ldb % 8 == 0 && a.ldc % 8 == 0 &&
            (!a.z || a.ldz % 8 == 0);
  for (const void* p : tiles) tc = tc && aligned(p, 16);
  if (tc) {
    if (P == 64) return (gdn_status)(N == 64 ? ssm::tcs::launch_np<64, 64>(a, workspace, st)
                                             : ssm::tcs::launch_np<128, 64>(a, workspace, st));
    return (gdn_status)(N == 64 ? ssm::tcs::launch_np<64, 128>(a, workspace, st)
                                : ssm::tcs::launch_np<128, 128>(a, workspace, st));
  }
  return dtype == GDN_F32 ? simt_scan<float>(N, P, a, st) : simt_scan<bf>(N, P, a, st);
}

// ---------------------------------------------------------------------------------------------
// token step
// ---------------------------------------------------------------------------------------------
template <int N, int P, typename T>
gdn_status step_launch(const ssm::StepArgs& a, int n, cudaStream_t st) {
  ssm::step_kernel<N, P, T><<<(unsigned)((long)n * a.H), DecodeShape<N, P>::NT, 0, st>>>(a);
  return launch_status();
}
template <typename T, int N>
gdn_status step_p(int P, const ssm::StepArgs& a, int n, cudaStream_t st) {
  switch (P) {
    case 16: return step_launch<N, 16, T>(a, n, st);
    case 32: return step_launch<N, 32, T>(a, n, st);
    case 64: return step_launch<N, 64, T>(a, n, st);
    default: return step_launch<N, 128, T>(a, n, st);
  }
}
template <typename T>
gdn_status step_n(int N, int P, const ssm::StepArgs& a, int n, cudaStream_t st) {
  switch (N) {
    case 16: return step_p<T, 16>(P, a, n, st);
    case 32: return step_p<T, 32>(P, a, n, st);
    case 64: return step_p<T, 64>(P, a, n, st);
    default: return step_p<T, 128>(P, a, n, st);
  }
}

}  // namespace

namespace gdn {
// gdn_check_error's share of this translation unit: reads and clears its error word.
bool ssm_take_error(unsigned int* word) {
  const unsigned int zero = 0;
  *word = 0;
  if (cudaMemcpyFromSymbol(word, g_error_word, sizeof(*word)) != cudaSuccess) return false;
  return *word == 0 || cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero)) == cudaSuccess;
}
}  // namespace gdn

extern "C" {

gdn_status gdn_ssm_conv(const void* x, long long ldx, const float* w, const float* bias, const void* hist_in,
                        void* out, void* hist_out, int B, int T, int C, gdn_dtype dtype, gdn_stream_t stream) {
  return conv_call(x, ldx, w, bias, hist_in, out, hist_out, nullptr, B, T, T, C, dtype, stream);
}

gdn_status gdn_ssm_conv_varlen(const void* x, long long ldx, const float* w, const float* bias,
                               const int* cu_seqlens, int nseq, int max_seqlen, const void* hist_in, void* out,
                               void* hist_out, int total_T, int C, gdn_dtype dtype, gdn_stream_t stream) {
  if (!cu_seqlens || !aligned(cu_seqlens, 4)) return GDN_ERR_INVALID_ARG;
  return conv_call(x, ldx, w, bias, hist_in, out, hist_out, cu_seqlens, nseq, total_T, max_seqlen, C, dtype, stream);
}

size_t gdn_ssm_scan_workspace_bytes(int nseq, int max_seqlen, int H, int G, int P, int N, gdn_dtype dtype) {
  if (!valid_dtype(dtype) || check_heads(H, G, P, N) != GDN_OK) return 0;
  return scan_workspace(nseq, max_seqlen, -1L, H, G, P, N, dtype);
}

size_t gdn_ssm_scan_varlen_workspace_bytes(int nseq, int max_seqlen, int total_T, int H, int G, int P, int N,
                                           gdn_dtype dtype) {
  if (total_T < 0 || !valid_dtype(dtype) || check_heads(H, G, P, N) != GDN_OK) return 0;
  return scan_workspace(nseq, std::min(max_seqlen, total_T), total_T, H, G, P, N, dtype);
}

gdn_status gdn_ssm_scan(const void* x, long long ldx, const void* dt, long long lddt, const void* Bm, long long ldb,
                        const void* Cm, long long ldc, const void* z, long long ldz, const float* A_log,
                        const float* D, const float* dt_bias, const float* S0, void* y, float* S_T, void* workspace,
                        size_t workspace_bytes, int B, int T, int H, int G, int P, int N, gdn_dtype dtype,
                        gdn_stream_t stream) {
  return scan_call(ssm::ScanArgs{x, dt, Bm, Cm, z, (long)ldx, (long)lddt, (long)ldb, (long)ldc, (long)ldz, A_log, D,
                                 dt_bias, S0, y, S_T, nullptr, B, T, T, H, G},
                   P, N, workspace, workspace_bytes, dtype, stream);
}

gdn_status gdn_ssm_scan_varlen(const void* x, long long ldx, const void* dt, long long lddt, const void* Bm,
                               long long ldb, const void* Cm, long long ldc, const void* z, long long ldz,
                               const float* A_log, const float* D, const float* dt_bias, const int* cu_seqlens,
                               int nseq, int max_seqlen, const float* S0, void* y, float* S_T, void* workspace,
                               size_t workspace_bytes, int total_T, int H, int G, int P, int N, gdn_dtype dtype,
                               gdn_stream_t stream) {
  if (!cu_seqlens || !aligned(cu_seqlens, 4)) return GDN_ERR_INVALID_ARG;
  return scan_call(ssm::ScanArgs{x, dt, Bm, Cm, z, (long)ldx, (long)lddt, (long)ldb, (long)ldc, (long)ldz, A_log, D,
                                 dt_bias, S0, y, S_T, cu_seqlens, nseq, total_T, max_seqlen, H, G},
                   P, N, workspace, workspace_bytes, dtype, stream);
}

gdn_status gdn_ssm_step(const void* u, long long ldu, const void* dt, long long lddt, const void* z, long long ldz,
                        const void* hist_in, void* hist_out, const float* w, const float* bias, const float* A_log,
                        const float* D, const float* dt_bias, float* S, void* y, int n, int H, int G, int P, int N,
                        gdn_dtype dtype, gdn_stream_t stream) {
  if (n < 0 || !valid_dtype(dtype)) return GDN_ERR_INVALID_ARG;
  const gdn_status s = check_heads(H, G, P, N);
  if (s != GDN_OK) return s;
  if (n == 0) return GDN_OK;
  if ((long)n * H > 0x7fffffffL) return GDN_ERR_UNSUPPORTED;
  const long HP = (long)H * P, C = HP + 2L * G * N;
  if (C > 0x7fffffffL) return GDN_ERR_UNSUPPORTED;
  const size_t el = elem(dtype);
  if (!u || !dt || !hist_in || !hist_out || hist_in == hist_out || !w || !A_log || !S || !y || ldu < C || lddt < H ||
      (z && ldz < HP))
    return GDN_ERR_INVALID_ARG;
  // every head's CTA reads its group's rows of u and hist_in while others write
  if (y == u || y == dt || y == z || y == hist_in || y == hist_out || y == S || hist_out == u) return GDN_ERR_INVALID_ARG;
  const void* ts[] = {u, dt, z, hist_in, hist_out, y};
  for (const void* p : ts)
    if (!aligned(p, el)) return GDN_ERR_INVALID_ARG;
  const void* fs[] = {w, bias, A_log, D, dt_bias};
  for (const void* p : fs)
    if (!aligned(p, 4)) return GDN_ERR_INVALID_ARG;
  if (!aligned(S, 16)) return GDN_ERR_INVALID_ARG;
  const ssm::StepArgs a{u, dt, z, (long)ldu, (long)lddt, (long)ldz, hist_in, hist_out, w, bias, A_log, D, dt_bias,
                        S, y, H, G};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == GDN_F32 ? step_n<float>(N, P, a, n, st) : step_n<bf>(N, P, a, n, st);
}

}  // extern "C"
