// The selective scan on the tensor cores (bf16; P, N in {64, 128}), in chunks of L = 128 tokens.
//
// With a_t = -D_t exp(A_log) (D_t the time step), c_t = a_1 + .. + a_t inside the chunk and S the state
// before it, the recurrence S_t = exp(a_t) S_{t-1} + D_t B_t x_t^T, y_t = S_t^T C_t + D x_t unrolls to
//   y_t = exp(c_t) S^T C_t + sum_{s <= t} (C_t . B_s) exp(c_t - c_s) D_s x_s + D x_t
//   S'  = exp(c_L) S + sum_s B_s (exp(c_L - c_s) D_s x_s)^T
// every exponent at most 0: nothing overflows however fast a head decays.  As matrix products, for the
// 128 columns hp that a CTA owns (two heads of 64 columns or one of 128, of one group):
//   G  [t, s]  = C B^T                      (shared by the CTA's heads)
//   Yi [t, hp] = C S
//   P_h[t, s]  = G exp(c_t - c_s) D_s, s <= t: formed from G in registers, back to TMEM as bf16
//   Ya [t, hp] = P_h X_h                    (P from TMEM, the raw x tile as the other operand)
//   U  [hp, n] = X'^T B,  X' = exp(c_L - c_s) D_s x_s as three bf16 terms (24 bits: the fp32 state
//                         keeps fp32 accuracy; B and x are exact)
// and y = exp(c_t) Yi + Ya + D x, S' = exp(c_L) S + U in fp32 registers; the state's copy that Yi reads is
// rounded to bf16 once a chunk, P once.
//
// Decays are never formed as differences of long sums: a chunk is four blocks of 32 tokens (a warp's lanes).
// c_t - c_s inside a block is the difference of that block's prefix sums, across blocks it is
// prefix(t) + whole blocks between + suffix(s), each a sum of its own, so that exponents near 0, the ones
// that matter, keep their relative accuracy.  Across blocks P's factor is a product of a row's and a
// column's exponential (both at most 1), so only the diagonal 32 x 32 blocks need one exponential each.
//
// Roles (10 warps): warps 0-7 form operands and epilogues, warp 8 moves tiles (TMA), warp 9 issues the
// MMAs.  x tiles are loaded a chunk ahead; y goes back through the x tile's memory by a TMA store.
// B and C, which the heads of a group share, come from L2.
//
// A sequence may be cut into segments that run side by side: a first launch (kOut = false) leaves
// each segment's own final state and its total decay in the workspace, and the second starts every
// segment from the states before it, combined in order (the result does not depend on timing).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ssm_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace ssm {
namespace tcs {

constexpr int L = 128;                        // tokens of a chunk
constexpr int kWorkers = 256;                 // threads of the eight worker warps
constexpr int kThreads = kWorkers + 64;
constexpr uint64_t kBudget = 4000000000ull;   // wait budget in SM cycles (about 2 s)
constexpr uint32_t kTile = L * 128;           // bytes of a [128 rows, 64 bf16] tile
using bf16_t = __nv_bfloat16;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
  ScanArgs a;
  float* ws;                    // segment states, then segment decays (segments > 1)
  int seg_chunks, segments;     // chunks of a segment; segments of the longest sequence
  int z_vec;                    // z's rows allow 16-byte loads
};

// Vectors of a chunk (two, by the chunk's parity): u, w, e [2 heads][128]; (prefix, step) [2][128] pairs;
// block sums [2][4]; decay [2].
constexpr uint32_t kVec = (2 * 128 * 5 + 16) * 4;

// Shared memory: x tiles (two chunks), B, C, the state operand, X' staging, vectors, barriers.
template <int N, bool kOut> struct Layout {
  static constexpr uint32_t NB = N / 64;
  static constexpr uint32_t x = 0;                                  // [2][2] tiles
  static constexpr uint32_t b = 4 * kTile;
  static constexpr uint32_t c = b + NB * kTile;                     // kOut only
  static constexpr uint32_t s = c + (kOut ? NB * kTile : 0);
  static constexpr uint32_t xw = s + (kOut ? NB * kTile : 0);       // [stages][3 terms][2] half tiles
  static constexpr uint32_t xw_stage = 6 * kTile / 2;
  static constexpr uint32_t vec = xw + (kOut ? 1 : 2) * xw_stage;
  static constexpr uint32_t bars = vec + 2 * kVec;
  static constexpr uint32_t bytes = bars + 256;
  static constexpr uint32_t alloc = bytes + 1024;                   // the base is rounded up to 1024
  static_assert(alloc <= 232448, "shared memory of a CTA");
};

enum Bar { XF = 0, BF = 2, CF, GD, CFREE, U0, YA, U1, XT, PR, SR, YR, DRAIN, kBars };

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc]: lane = row of A, two bf16 of K per 32-bit column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

template <int N, int P, bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
scan_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mb,
            const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap my, const Args k) {
  using Lay = Layout<N, kOut>;
  constexpr int NH = 128 / P;                 // heads of this CTA
  constexpr int NB = N / 64;
  constexpr int NR = N / 2;                   // state columns of a worker thread
  constexpr uint32_t TG = 0, TYI = 128, TYA = 256, TU = 384;
  const ScanArgs& a = k.a;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = tc::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int hpg = a.H / a.G, pairs = (hpg + NH - 1) / NH;
  const int g = blockIdx.x / pairs, pr = blockIdx.x % pairs;
  const int h0 = g * hpg + pr * NH;
  const int heads = min(NH, hpg - pr * NH);   // 1 where a group's last pair has one head only
  const int seg = blockIdx.y, seq = blockIdx.z;
  const RowSpan sp = row_span(a.cu, seq, a.T, a.max_len);
  const int chunks = (sp.len + L - 1) / L;
  const int ch0 = seg * k.seg_chunks;
  const int nc = min(k.seg_chunks, chunks - ch0);
  const bool last = ch0 + nc >= chunks;       // this segment ends the sequence
  if (seg > 0 && nc <= 0) return;
  if (!kOut && (last || nc <= 0)) return;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::bars + kBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::bars + kBars * 8 + 8);
  auto bar = [&](int i) { return sb + Lay::bars + 8u * i; };
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool workers = i == XT || i == PR || i == SR || i == YR;
      tc::mbar_init(tc::smem_u32(&bars[i]), workers ? kWorkers : 1);
    }
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 9) tc::tmem_alloc(tc::smem_u32(tmem_slot), 512);
  if (NH == 2 && heads == 1) {                // the missing head's x tiles: zeros, never loaded
    for (int i = tid; i < 2 * (int)kTile / 16; i += kThreads) {
      const int buf = i / ((int)kTile / 16), o = i % ((int)kTile / 16);
      tc::st_shared_v4(sb + Lay::x + (2 * buf + 1) * kTile + o * 16, 0, 0, 0, 0);
    }
    tc::fence_proxy_async_smem();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](int b, int phase) { tc::mbar_wait(bar(b), (uint32_t)phase & 1u, abort_flag, kBudget); };

  if (warp == 8) {
    // ----------------------------------- tiles -----------------------------------------------
    if (lane == 0 && nc > 0) {
      const int row = (int)(sp.row0 + (long)ch0 * L);
      auto load_x = [&](int c) {
        const uint32_t dst = sb + Lay::x + (c & 1) * 2 * kTile;
        tc::mbar_arrive_expect_tx(bar(XF + (c & 1)), (NH == 2 && heads == 1 ? 1 : 2) * kTile);
        tma_load_2d(dst, &mx, bar(XF + (c & 1)), h0 * P, row + c * L);
        if (NH == 1 || heads == 2) tma_load_2d(dst + kTile, &mx, bar(XF + (c & 1)), h0 * P + 64, row + c * L);
      };
      auto load_n = [&](uint32_t dst, const CUtensorMap* m, int b, int c) {
        tc::mbar_arrive_expect_tx(bar(b), NB * kTile);
        for (int i = 0; i < NB; ++i) tma_load_2d(dst + i * kTile, m, bar(b), g * N + i * 64, row + c * L);
      };
      int xs = 0, bs = 0, cs = 0;             // loads issued
      load_x(xs++);
      load_n(sb + Lay::b, &mb, BF, bs++);
      if (kOut) load_n(sb + Lay::c, &mc, CF, cs++);
      if (nc > 1) load_x(xs++);
      for (int c = 0; c < nc && !*abort_flag; ++c) {
        const bool more = c + 1 < nc;
        if (kOut) {
          if (more) {
            wait(CFREE, c);
            load_n(sb + Lay::c, &mc, CF, cs++);
          }
          wait(YR, c);
          if (sp.len - (ch0 + c) * L >= L) {
            const uint32_t src = sb + Lay::x + (c & 1) * 2 * kTile;
            tma_store_2d(&my, src, h0 * P, row + c * L);
            if (NH == 1 || heads == 2) tma_store_2d(&my, src + kTile, h0 * P + 64, row + c * L);
            tc::bulk_commit();
          }
        }
        wait(U1, c);
        if (more) load_n(sb + Lay::b, &mb, BF, bs++);
        if (c + 2 < nc) {
          if (kOut) tc::bulk_wait_read_all();
          load_x(xs++);
        }
      }
      // every load issued lands, and every store has read its source, before the CTA can leave
      volatile int never = 0;
      if (kOut) tc::bulk_wait_all();
      for (int i = max(0, xs - 2); i < xs; ++i) tc::mbar_wait(bar(XF + (i & 1)), (i >> 1) & 1, &never, kBudget / 4);
      tc::mbar_wait(bar(BF), (bs - 1) & 1, &never, kBudget / 4);
      if (kOut) tc::mbar_wait(bar(CF), (cs - 1) & 1, &never, kBudget / 4);
    }
  } else if (warp == 9) {
    // ----------------------------------- MMAs ------------------------------------------------
    if (lane == 0 && nc > 0) {
      constexpr uint32_t ID_G = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t ID_YA = tc::idesc_bf16(128, P, false, true);
      constexpr uint32_t ID_U = tc::idesc_bf16(128, N, true, true);
      const uint64_t dc = tc::sdesc_sw128(sb + Lay::c, 16, 1024);          // C, K = n
      const uint64_t db = tc::sdesc_sw128(sb + Lay::b, 16, 1024);          // B, K = n
      const uint64_t dbt = tc::sdesc_sw128(sb + Lay::b, kTile, 1024);      // B, K = t
      const uint64_t ds = tc::sdesc_sw128(sb + Lay::s, 16, 1024);          // S^T, K = n
      for (int c = 0; c < nc; ++c) {
        const uint64_t dx = tc::sdesc_sw128(sb + Lay::x + (c & 1) * 2 * kTile, kTile, 1024);
        wait(BF, c);
        if (kOut) {
          wait(CF, c);
          tc::tc_fence_after();
#pragma unroll
          for (int i = 0; i < NB * 4; ++i) {
            const uint32_t o = (i >> 2) * kTile + (i & 3) * 32;
            tc::mma_bf16(tmem + TG, tc::desc_adv(dc, o), tc::desc_adv(db, o), ID_G, i > 0);
          }
          tc::mma_commit(bar(GD));
          wait(SR, c);
          tc::tc_fence_after();
#pragma unroll
          for (int i = 0; i < NB * 4; ++i) {
            const uint32_t o = (i >> 2) * kTile + (i & 3) * 32;
            tc::mma_bf16(tmem + TYI, tc::desc_adv(dc, o), tc::desc_adv(ds, o), ID_G, i > 0);
          }
          tc::mma_commit(bar(CFREE));
        }
        // half `hf` of the chunk's tokens: 4 steps of 16 for each of the three terms
        auto issue_u = [&](int hf) {
          const uint64_t dw =
              tc::sdesc_sw128(sb + Lay::xw + (kOut ? 0 : hf) * Lay::xw_stage, kTile / 2, 1024);
#pragma unroll
          for (int i = 0; i < 12; ++i)
            tc::mma_bf16(tmem + TU, tc::desc_adv(dw, (i >> 2) * kTile + (i & 3) * 2048),
                         tc::desc_adv(dbt, hf * (kTile / 2) + (i & 3) * 2048), ID_U, hf > 0 || i > 0);
        };
        wait(XT, 0);
        tc::tc_fence_after();
        issue_u(0);
        tc::mma_commit(bar(U0));
        if (kOut) {
          wait(PR, c);
          tc::tc_fence_after();
#pragma unroll
          for (int hs = 0; hs < NH; ++hs)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mma_bf16_ta(tmem + TYA + hs * 64, tmem + TG + 32 * (i >> 1) + 16 * hs + 8 * (i & 1),
                          tc::desc_adv(dx, hs * kTile + i * 2048), ID_YA, i > 0);
          tc::mma_commit(bar(YA));
        }
        wait(XT, 1);
        tc::tc_fence_after();
        issue_u(1);
        tc::mma_commit(bar(U1));
      }
      tc::mma_commit(bar(DRAIN));
      volatile int never = 0;
      tc::mbar_wait(bar(DRAIN), 0, &never, kBudget / 4);
    }
  } else {
    // ----------------------------------- workers ---------------------------------------------
    const int q = warp & 3, wg = warp >> 2;          // lane quadrant; half of the columns
    const int t = tid & 127;                         // the row (of tokens, or of hp) of this thread
    const uint32_t tlane = tmem + ((uint32_t)(32 * q) << 16);
    const int vh = NH == 2 ? wg : 0;                 // the head whose vectors this thread forms
    const bool vec_on = NH == 2 ? wg < heads : wg == 0;
    const int sh = NH == 2 ? (t >> 6) : 0;           // the head of state row t
    const int p = NH == 2 ? (t & 63) : t;
    const bool s_on = sh < heads;
    const int n0 = wg * NR;
    float rate = 0.f, bias = 0.f;
    if (vec_on) {
      rate = -expf(a.A_log[h0 + vh]) * kLog2e;
      bias = a.dt_bias ? a.dt_bias[h0 + vh] : 0.f;
    }
    const bool y_on = NH == 1 || wg < heads;
    const float skip = kOut && a.D && y_on ? a.D[h0 + (NH == 2 ? wg : 0)] : 0.f;

    // ---- the state before this segment
    float S[NR];
    const long HNP = (long)a.H * N * P;
    const long srow = ((long)(h0 + sh) * N + n0) * P + p;    // state rows n0 .. n0 + NR - 1, column p
    const float* wseg = k.ws + (long)seq * (k.segments - 1) * HNP + srow;
    const float* wdec = k.ws + (long)a.nseq * (k.segments - 1) * HNP + (long)seq * (k.segments - 1) * a.H + h0 + sh;
#pragma unroll
    for (int i = 0; i < NR; ++i) S[i] = 0.f;
    if (s_on) {
      if (seg == 0) {
        if (a.S0) {
#pragma unroll
          for (int i = 0; i < NR; ++i) S[i] = a.S0[seq * HNP + srow + (long)i * P];
        }
      } else if (kOut) {
        for (int j = 0; j < seg; ++j) {
          const float d = wdec[(long)j * a.H];
#pragma unroll
          for (int i = 0; i < NR; ++i) S[i] = fmaf(d, S[i], wseg[j * HNP + (long)i * P]);
        }
      }
    }
    float seg_decay = 1.f;
    auto publish_state = [&]() {               // the copy that the next chunk's Yi reads
#pragma unroll
      for (int j = 0; j < NR / 8; ++j) {
        const uint32_t chunk = N == 128 ? j : wg * 4 + j;
        tc::st_shared_v4(sb + Lay::s + (N == 128 ? wg * kTile : 0) + tc::sw128(t, chunk),
                         tc::pack_bf16(S[8 * j], S[8 * j + 1]), tc::pack_bf16(S[8 * j + 2], S[8 * j + 3]),
                         tc::pack_bf16(S[8 * j + 4], S[8 * j + 5]), tc::pack_bf16(S[8 * j + 6], S[8 * j + 7]));
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      tc::mbar_arrive(bar(SR));
    };
    if (kOut && nc > 0) publish_state();

    const bf16_t* dtp = static_cast<const bf16_t*>(a.dt) + h0 + vh;
    auto load_dt = [&](int c) -> float {
      const int at = (ch0 + c) * L + t;
      return vec_on && c < nc && at < sp.len ? __bfloat162float(dtp[(sp.row0 + at) * a.lddt]) : 0.f;
    };
    float raw = load_dt(0);
    for (int c = 0; c < nc; ++c) {
      const int valid = min(L, sp.len - (ch0 + c) * L);
      const long row = sp.row0 + (long)(ch0 + c) * L;
      float* vec = reinterpret_cast<float*>(smem + Lay::vec + (c & 1) * kVec);
      float* u_ = vec;                          // [2][128] D_s exp(suffix in its block)
      float* w_ = vec + 256;                    // [2][128] D_s exp(suffix in the chunk)
      float* e_ = vec + 512;                    // [2][128] exp(prefix in the chunk)
      float2* pd = reinterpret_cast<float2*>(vec + 768);   // [2][128] (prefix in its block, D_s)
      float* tot = vec + 1280;                  // [2][4] block sums
      float* dec = tot + 8;                     // [2] exp(sum of the chunk)
      // ---- 1. the chunk's decays, in base-2 logarithms
      if (NH == 2 || wg == 0) {
        const bool live = vec_on && t < valid;
        const float step = live ? softplus(raw + bias) : 0.f;
        const float la = live ? step * rate : 0.f;
        float pre = la, suf = la;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float up = __shfl_up_sync(0xffffffffu, pre, o);
          const float dn = __shfl_down_sync(0xffffffffu, suf, o);
          if (lane >= o) pre += up;
          if (lane < 32 - o) suf += dn;
        }
        suf = __shfl_down_sync(0xffffffffu, suf, 1);         // the sum over the tokens after this one
        if (lane == 31) {
          suf = 0.f;
          tot[vh * 4 + q] = pre;
        }
        pd[vh * 128 + t] = make_float2(pre, step);
        u_[vh * 128 + t] = step * tc::ex2(suf);
        tc::named_bar(1 + vh, 128);
        const float t0 = tot[vh * 4], t1 = tot[vh * 4 + 1], t2 = tot[vh * 4 + 2], t3 = tot[vh * 4 + 3];
        const float before = q == 0 ? 0.f : q == 1 ? t0 : q == 2 ? t0 + t1 : t0 + t1 + t2;
        const float after = q == 3 ? 0.f : q == 2 ? t3 : q == 1 ? t2 + t3 : t1 + t2 + t3;
        w_[vh * 128 + t] = step * tc::ex2(suf + after);
        e_[vh * 128 + t] = tc::ex2(pre + before);
        if (t == 0) dec[vh] = tc::ex2(t0 + t1 + t2 + t3);
      }
      raw = load_dt(c + 1);
      wait(XF + (c & 1), c >> 1);
      const uint32_t xt = sb + Lay::x + (c & 1) * 2 * kTile;
      if (valid < L) {       // rows behind the sequence reach no product: another sequence's, maybe NaN
        wait(BF, c);
        if (kOut) wait(GD, c);             // G reads the same B tile
        for (int i = tid; i < (L - valid) * 8 * (2 + NB); i += kWorkers) {
          const int j = i & 7, tile = (i >> 3) % (2 + NB), r = valid + (i >> 3) / (2 + NB);
          tc::st_shared_v4((tile < 2 ? xt + tile * kTile : sb + Lay::b + (tile - 2) * kTile) + tc::sw128(r, j), 0, 0, 0, 0);
        }
      }
      tc::named_bar(3, kWorkers);
      // ---- 2. X' of half `hf` of the tokens, in three terms
      auto weigh = [&](int hf) {
        const uint32_t dst = sb + Lay::xw + (kOut ? 0 : hf) * Lay::xw_stage;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int id = tid + kWorkers * i;
          const int j = id & 7, r = (id >> 3) & 63, tile = id >> 9;
          const uint4 v = tc::ld_shared_v4(xt + tile * kTile + tc::sw128(hf * 64 + r, j));
          const float w = w_[(NH == 2 ? tile : 0) * 128 + hf * 64 + r];
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t o0[4], o1[4], o2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f0 = tc::bf16lo(in[e]) * w, f1 = tc::bf16hi(in[e]) * w;
            o0[e] = tc::pack_bf16(f0, f1);
            const float g0 = f0 - tc::bf16lo(o0[e]), g1 = f1 - tc::bf16hi(o0[e]);
            o1[e] = tc::pack_bf16(g0, g1);
            o2[e] = tc::pack_bf16(g0 - tc::bf16lo(o1[e]), g1 - tc::bf16hi(o1[e]));
          }
          const uint32_t at = dst + tile * (kTile / 2) + tc::sw128(r, j);
          tc::st_shared_v4(at, o0[0], o0[1], o0[2], o0[3]);
          tc::st_shared_v4(at + kTile, o1[0], o1[1], o1[2], o1[3]);
          tc::st_shared_v4(at + 2 * kTile, o2[0], o2[1], o2[2], o2[3]);
        }
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(bar(XT));
      };
      weigh(0);
      if constexpr (kOut) {
        // ---- 3. P from G, block of 32 columns by block
        wait(GD, c);
        tc::tc_fence_after();
#pragma unroll
        for (int bi = 0; bi < 2; ++bi) {
          const int b = 2 * wg + bi;
          float G[32];
          if (b <= q) {
            tc::tmem_ld32(tlane + TG + 32 * b, G);
            tc::tmem_wait_ld();
          }
#pragma unroll
          for (int hs = 0; hs < NH; ++hs) {
            uint32_t o[16];
            if (b > q) {
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = 0;
            } else if (b < q) {
              float mid = pd[hs * 128 + t].x;
              for (int i = b + 1; i < q; ++i) mid += tot[hs * 4 + i];
              const float r = tc::ex2(mid);
              const float4* u4 = reinterpret_cast<const float4*>(u_ + hs * 128 + 32 * b);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 uu = u4[i];
                o[2 * i] = tc::pack_bf16(G[4 * i] * (uu.x * r), G[4 * i + 1] * (uu.y * r));
                o[2 * i + 1] = tc::pack_bf16(G[4 * i + 2] * (uu.z * r), G[4 * i + 3] * (uu.w * r));
              }
            } else {
              const float mine = pd[hs * 128 + t].x;
              const float4* p4 = reinterpret_cast<const float4*>(pd + hs * 128 + 32 * b);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float4 v = p4[i];                 // (prefix, step) of columns 2 i and 2 i + 1
                const float f0 = 2 * i <= lane ? G[2 * i] * (v.y * tc::ex2(mine - v.x)) : 0.f;
                const float f1 = 2 * i + 1 <= lane ? G[2 * i + 1] * (v.w * tc::ex2(mine - v.z)) : 0.f;
                o[i] = tc::pack_bf16(f0, f1);
              }
            }
            tmem_st16(tlane + TG + 32 * b + 16 * hs, o);
          }
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        tc::mbar_arrive(bar(PR));
      }
      uint4 zr[8];
      if constexpr (kOut) {
        // the gate's values, needed in step 5
        if (a.z && y_on && t < valid) {
          const bf16_t* zp = static_cast<const bf16_t*>(a.z) + (row + t) * a.ldz + (long)h0 * P + wg * 64;
          if (k.z_vec) {
#pragma unroll
            for (int j = 0; j < 8; ++j) zr[j] = reinterpret_cast<const uint4*>(zp)[j];
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] = (uint32_t)__bfloat16_as_ushort(zp[8 * j + 2 * e]) |
                       ((uint32_t)__bfloat16_as_ushort(zp[8 * j + 2 * e + 1]) << 16);
              zr[j] = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        wait(U0, c);                       // the staging of the first half is free again
      }
      // ---- 4. the second half
      weigh(1);
      if constexpr (kOut) {
        // ---- 5. y, in place of x
        wait(YA, c);
        tc::tc_fence_after();
        tc::named_bar(3, kWorkers);        // every thread has read the x tile in step 4
        const float e = e_[(NH == 2 ? wg : 0) * 128 + t];
        bf16_t* yp = static_cast<bf16_t*>(a.y) + (row + t) * ((long)a.H * P) + (long)h0 * P + wg * 64;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float yi[32], ya[32];
          tc::tmem_ld32(tlane + TYI + 64 * wg + 32 * hf, yi);
          tc::tmem_ld32(tlane + TYA + 64 * wg + 32 * hf, ya);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t at = xt + wg * kTile + tc::sw128(t, 4 * hf + j);
            const uint4 xv = tc::ld_shared_v4(at);
            const uint32_t xi[4] = {xv.x, xv.y, xv.z, xv.w};
            const uint4 z4 = zr[4 * hf + j];
            const uint32_t zi[4] = {z4.x, z4.y, z4.z, z4.w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int cidx = 8 * j + 2 * i;
              float f0 = fmaf(e, yi[cidx], fmaf(skip, tc::bf16lo(xi[i]), ya[cidx]));
              float f1 = fmaf(e, yi[cidx + 1], fmaf(skip, tc::bf16hi(xi[i]), ya[cidx + 1]));
              if (a.z) {
                f0 *= silu(tc::bf16lo(zi[i]));
                f1 *= silu(tc::bf16hi(zi[i]));
              }
              o[i] = tc::pack_bf16(f0, f1);
            }
            if (!y_on) continue;
            if (valid == L) tc::st_shared_v4(at, o[0], o[1], o[2], o[3]);
            else if (t < valid)
              *reinterpret_cast<uint4*>(yp + 32 * hf + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(bar(YR));
      }
      // ---- 6. the state
      wait(U1, c);
      tc::tc_fence_after();
      const float d = dec[sh];
      seg_decay *= d;
#pragma unroll
      for (int i = 0; i < NR / 32; ++i) {
        float U[32];
        tc::tmem_ld32(tlane + TU + n0 + 32 * i, U);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) S[32 * i + j] = fmaf(d, S[32 * i + j], U[j]);
      }
      if (kOut) {
        if (c + 1 < nc) publish_state();
      } else {
        tc::tc_fence_before();             // U has been read before this thread's next X' lets U0 run again
      }
    }
    // ---- the state after this segment
    if (s_on) {
      if constexpr (kOut) {
        if (last && a.S_T) {
#pragma unroll
          for (int i = 0; i < NR; ++i) a.S_T[seq * HNP + srow + (long)i * P] = S[i];
        }
      } else {
        float* out = const_cast<float*>(wseg) + seg * HNP;
#pragma unroll
        for (int i = 0; i < NR; ++i) out[(long)i * P] = S[i];
        if (p == 0 && wg == 0) const_cast<float*>(wdec)[(long)seg * a.H] = seg_decay;
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc::tc_fence_after();
    tc::tmem_relinquish();
    tc::tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && *abort_flag) record_error(kErrTimeout);
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}
// [rows, cols] bf16, rows ld values apart, boxes of 64 columns x 128 rows, 128-byte swizzle; rows
// past the end load as zeros and are not stored.
inline bool make_map(CUtensorMap* m, const void* base, long rows, long cols, long ld) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)L}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool supported(int P, int N) { return (P == 64 || P == 128) && (N == 64 || N == 128); }
inline int columns(int H, int G, int P) {       // CTAs of one sequence and segment
  const int nh = 128 / P;
  return G * ((H / G + nh - 1) / nh);
}
// Segments of the longest sequence, a rule on sizes alone (so that the workspace can be sized without
// a device): one while the sequences and columns fill the SMs, else as many as still fit into one wave, none
// shorter than four chunks (a segment costs the first launch and the combination, about two chunks' time).
inline int segments(int nseq, int max_len, int H, int G, int P) {
  const long ctas = (long)nseq * columns(H, G, P);
  const int chunks = (max_len + L - 1) / L;
  const long fit = 148 / (ctas > 0 ? ctas : 1);
  const int s = (int)(fit < chunks / 4 ? fit : chunks / 4);
  return s < 2 ? 1 : s;
}
inline size_t workspace(int nseq, int max_len, int H, int G, int P, int N) {
  const size_t s = (size_t)segments(nseq, max_len, H, G, P) - 1;
  return (size_t)nseq * s * H * ((size_t)N * P + 1) * sizeof(float);
}

template <int N, int P>
int launch_np(const ScanArgs& a, void* ws, cudaStream_t st) {
  const long rows = a.cu ? (long)a.T : (long)a.nseq * a.T;
  Args k{a, static_cast<float*>(ws), 0, segments(a.nseq, a.max_len, a.H, a.G, P), 0};
  const int chunks = (a.max_len + L - 1) / L;
  k.seg_chunks = chunks > 0 ? (chunks + k.segments - 1) / k.segments : 1;
  k.z_vec = a.z && a.ldz % 8 == 0 && (reinterpret_cast<uintptr_t>(a.z) & 15u) == 0;
  CUtensorMap mx, mb, mc, my;
  if (!make_map(&mx, a.x, rows, (long)a.H * P, a.ldx) || !make_map(&mb, a.B, rows, (long)a.G * N, a.ldb) ||
      !make_map(&mc, a.C, rows, (long)a.G * N, a.ldc) || !make_map(&my, a.y, rows, (long)a.H * P, (long)a.H * P))
    return GDN_ERR_CUDA;
  const dim3 grid((unsigned)columns(a.H, a.G, P), (unsigned)k.segments, (unsigned)a.nseq);
  if (k.segments > 1) {
    auto first = scan_kernel<N, P, false>;
    if (cudaFuncSetAttribute(first, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<N, false>::alloc) != cudaSuccess)
      return GDN_ERR_CUDA;
    first<<<dim3(grid.x, grid.y - 1, grid.z), kThreads, Layout<N, false>::alloc, st>>>(mx, mb, mc, my, k);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  }
  auto kern = scan_kernel<N, P, true>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<N, true>::alloc) != cudaSuccess)
    return GDN_ERR_CUDA;
  kern<<<grid, kThreads, Layout<N, true>::alloc, st>>>(mx, mb, mc, my, k);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace tcs
}  // namespace ssm
}  // namespace gdn
