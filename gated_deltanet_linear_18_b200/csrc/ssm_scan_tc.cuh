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
// and y = exp(c_t) Yi + Ya + D x, S' = exp(c_L) S + U in fp32 registers.  Two roundings to bf16 are chosen: of the state's
// copy that Yi reads, once a chunk, and of P, once (2^-8 of each term at most).  They reach y only, never the state, and y is
// rounded to bf16 itself: its error against fp64 is 1.84e-3 to 1.91e-3 of its norm on the prompts below, 1.66e-3 of which
// that last rounding makes.  A second term for each, as X' has, would double the MMAs of Yi and Ya and needs 128 columns of
// TMEM and up to 32 KB of shared memory that the CTA does not have.
//
// Decays are never formed as differences of long sums: a chunk is four blocks of 32 tokens (a warp's lanes).
// c_t - c_s inside a block is the difference of that block's prefix sums, across blocks it is
// prefix(t) + whole blocks between + suffix(s), each a sum of its own, so that exponents near 0, the ones
// that matter, keep their relative accuracy.  Across blocks P's factor is a product of a row's and a
// column's exponential (both at most 1), so only the diagonal 32 x 32 blocks need one exponential each.
//
// Roles: five warpgroups that run ahead of one another as far as the tiles and accumulators allow.
//   warp 0 loads B, C and the chunks' decay vectors, warp 2 loads x tiles and stores y, warp 3 issues the MMAs of U in
//     four quarters of 32 tokens, warp 1 those of G, Yi and Ya;
//   warpgroup 1 forms X';
//   warpgroup 2 forms P and keeps the state in registers (a thread a row hp of S^T);
//   warpgroups 3 and 4 form y, 64 columns each, in place of x in its tile, which leaves by a TMA store.
// B and C, which the heads of a group share, come from L2.
//
// The decay vectors (five numbers a token and head) come from a small kernel before: formed here they kept one warp busy
// with 1000 instructions a chunk.
//
// One CTA an SM stays and takes one item after another (a sequence's columns, or a segment of them) from a counter;
// the roles go on into the next item while others finish the last, so that a short sequence costs little more than its
// chunks: a CTA for each item spent 14 us beside its chunks on filling and draining the pipeline.
//
// A sequence's columns may be cut into segments that run side by side: a first launch (kOut = false) leaves each
// segment's own final state and its total decay in the workspace, and the second starts every segment from the
// states before it, combined in order (the result does not depend on timing).  That is done for the (sequence,
// column) pairs that do not fill a wave of the SMs: 192 of them run as 148 whole ones and 44 in three segments.
//
// Measured (bf16, inputs that are not in L2): 8192 tokens of 64 heads of 128 x 64, gated, 139-147 us (decays 8, first launch
// about 37, the rest the second); 4 x 2048 tokens of 48 heads of 128 x 128, 124-131 us (114 with the inputs in L2); a ragged
// batch of 32 prompts of 64 heads, gated, 157-164 us.  A chunk takes about 5 us.  352 KB of MMA operands and about as much
// of tiles pass through shared memory in it (2.9 us at 128 bytes a cycle); the rest is what the roles wait for one
// another.  Counted for 128 x 128: the tensor pipe is active in 39 % of the cycles, the issue slots in 47 %; per issued
// instruction a warp waits 4.7 cycles for loads, barriers and TMEM (long scoreboard), 1.3 for shared memory and 0.6 for
// instructions.  The kernels with outputs and N = 128 spill 160 bytes.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ssm_common.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace ssm {
namespace tcs {

constexpr int L = 128;                        // tokens of a chunk
constexpr int kThreads = 640;
constexpr uint32_t kPolls = 1u << 24;         // polls of a barrier before a wait gives up (half a second or more)
constexpr uint32_t kTile = L * 128;           // bytes of a [128 rows, 64 bf16] tile
using bf16_t = __nv_bfloat16;
constexpr float kLog2e = 1.4426950408889634f;

// Where the chunks of a sequence have their records, `n` in all for a column.  Each sequence has room for the longest
// one's `chunks`; or, where a packed call's rows make that fewer, sequence s starts at record (its first row) / L + s:
// behind the last one of every sequence before it, since floor(len / L) + 1 >= ceil(len / L), and below total / L + nseq.
struct Records {
  long n;
  int chunks, by_rows;
  __host__ __device__ long first(int seq, long row0) const { return by_rows ? row0 / L + seq : (long)seq * chunks; }
};
inline Records records_of(int nseq, int max_len, long total) {     // total < 0: not known, or not packed
  const int chunks = max_len / L + (max_len % L != 0);
  const long each = (long)nseq * chunks, by_rows = total / L + nseq;
  return total >= 0 && by_rows < each ? Records{by_rows, chunks, 1} : Records{each, chunks, 0};
}

struct Args {
  ScanArgs a;
  int* next;                    // the next item of each launch (set by the decay kernel)
  float* ws;                    // [pairs cut][segments - 1] of a state [N][128] and two decays
  const float* vecs;            // decay vectors: [columns][records.n] records of kVec bytes
  Records records;
  int columns, whole;           // pair = sequence * columns + column; the first `whole` pairs are not cut
  int seg_chunks, segments;     // the others: chunks of a segment, segments of the longest sequence
  int items;                    // of this launch
};

constexpr uint32_t kSlot = 6 * kTile / 4;      // X' of 32 tokens: three terms, two 64-column quarter tiles each
// The decay vectors of a chunk of two heads (exponents in base 2): u [2][128] D_s exp(suffix in its block), w [2][128]
// D_s exp(suffix in the chunk), e [2][128] exp(prefix in the chunk), prefix in its block [2][128], the same less
// log2 D_s [2][128], block sums [2][4], exp(chunk's sum) [2].
constexpr uint32_t kVec = (2 * 128 * 5 + 16) * 4;
constexpr int VU = 0, VW = 256, VE = 512, VP = 768, VT = 1280, VD = 1288;

// Shared memory.  With the outputs: x tiles of two chunks, B, C, the state operand, two slots of X' (32 tokens
// each), vectors, barriers.  Without: x and B of two chunks, X'.
template <int N, bool kOut> struct Layout {
  static constexpr uint32_t NB = N / 64;
  static constexpr uint32_t x = 0;                                  // [2][2] tiles
  static constexpr uint32_t b = 4 * kTile;                          // [1 or 2][NB] tiles
  static constexpr uint32_t c = b + (kOut ? 1 : 2) * NB * kTile;
  static constexpr uint32_t s = c + (kOut ? NB * kTile : 0);
  static constexpr uint32_t xw = s + (kOut ? NB * kTile : 0);       // [2 slots][3 terms][2] quarter tiles
  static constexpr uint32_t vec = xw + 2 * kSlot;
  static constexpr int kVecs = kOut ? 3 : 4;                        // chunks whose vectors are here
  static constexpr uint32_t bars = vec + kVecs * kVec;
  static constexpr uint32_t queue = bars + 320;                     // [4] items of 32 bytes
  static constexpr uint32_t bytes = queue + 4 * 32;
  static constexpr uint32_t alloc = bytes + 1024;                   // the base is rounded up to 1024
  static_assert(alloc <= 232448, "shared memory of a CTA");
};

// Barriers.  By TMA: XF (two x tiles), BF (B's four quarters; without outputs two buffers), CF, VR (three or four
// vector slots).  By warp 0: IQ (four items).  By MMA commits: UQ (the two X' slots read), U1 (U complete), BE (the same parts of
// B read by U), BX (two: U complete and so x's tile read for X'), GD (G), YI, YA.  By the threads of the warpgroups: XT
// (two X' slots staged), PR (P), UR (U is in registers; without outputs two, by
// place), SR (the state operand), YR (two: y in its tile, Yi and Ya read).
// A wait names a phase by its parity alone, so each one below stands where the phase after the awaited
// one cannot have completed: what completes that needs something this waiter has yet to do.  For the same
// reason YR and BX are kept by tile and only warp 3 waits for XT.  Copies complete in any order (B and C of a chunk from
// L2 may be there before its vectors), so every role that reads the vectors waits for VR itself, in vectors(); a slot's
// next copy is issued only after all of them have read this one.
// log2 of a time step (0 gives -infinity: that token's weight is 0)
__device__ __forceinline__ float log2_step(float v) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

enum Bar {
  XF = 0, BF = 2, CF = BF + 4, UQ, U1 = UQ + 2, BE, BX = BE + 4, GD = BX + 2, YI, YA, VR, IQ = VR + 4, DRAIN = IQ + 4,
  XT, PR = XT + 2, UR, SR = UR + 2, YR, kBars = YR + 2
};

// Bounded wait in few instructions (there are many of them, and the roles' code has to stay in the instruction
// cache): gives up after kPolls polls, or as soon as another thread has; the caller goes on with what is there and
// the kernel reports it at its end.
__device__ __forceinline__ void bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (uint32_t n = 0; !tc::mbar_try_wait(bar, parity); ++n)
    if (n == kPolls || *abort_flag) {
      *abort_flag = 1;
      break;
    }
}

// Rows `valid` .. 127 of `tiles` tiles to zeros, by 128 threads.
__device__ __forceinline__ void zero_rows(uint32_t tile0, int tiles, int valid, int t) {
#pragma unroll 1
  for (int i = t; i < (L - valid) * 8 * tiles; i += 128) {
    const int j = i & 7, tl = (i >> 3) % tiles, r = valid + (i >> 3) / tiles;
    tc::st_shared_v4(tile0 + tl * kTile + tc::sw128(r, j), 0, 0, 0, 0);
  }
}

template <int kRegs> __device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs> __device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const void* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0),
               "r"(c1)
               : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
// The MMAs, run by a whole warp and issued by its `leader` lane: the descriptors then stay in uniform registers, where
// an MMA issued from a branch of one thread moves each of them there first.  D[tmem] (+)= A * B; A from shared memory, or
// from tmem (lane = row, two bf16 of K per 32-bit column).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// The launches of a call overlap: each one lets the next be placed as soon as its own CTAs all run, and the next sets
// its barriers and TMEM up before it waits for the launch before to have completed (which has waited likewise).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The decay vectors of every chunk: grid (blocks of kDecayCols columns, records as y + z gridDim.y: the chunks of sequence z
// where records are not by rows), 128 threads for each of a column's heads, a token a thread and a block of 32 tokens a
// warp.  The columns of a block share the sectors of a token's dt row, all loaded before the first is used.  It also sets
// the item counters of the launches that follow, and hands the state of a sequence without tokens on.
// (8192 x 64 heads: 139 us with two or four columns, 141 with eight; ragged batch 162, 160 and 161.)
constexpr int kDecayCols = 4;
template <int NH>
__global__ void __launch_bounds__(128 * NH) decay_kernel(const ScanArgs a, const Records rec, float* __restrict__ vecs, int* next,
                                                         int2 first, int N, int cols) {
  launch_dependents();
  const int hpg = a.H / a.G, pairs = (hpg + NH - 1) / NH;
  const long record = (long)blockIdx.z * gridDim.y + blockIdx.y;
  int seq = blockIdx.z;
  if (rec.by_rows) {                       // the last sequence that starts at this record or before
    seq = 0;
    for (int hi = a.nseq - 1; seq < hi;) {
      const int mid = (seq + hi + 1) >> 1;
      if (rec.first(mid, row_span(a.cu, mid, a.T, a.max_len).row0) <= record) seq = mid; else hi = mid - 1;
    }
  }
  const RowSpan sp = row_span(a.cu, seq, a.T, a.max_len);
  const int c = rec.by_rows ? (int)(record - rec.first(seq, sp.row0)) : (int)blockIdx.y;
  const int hs = threadIdx.x >> 7, t = threadIdx.x & 127, q = t >> 5, lane = t & 31;
  if (blockIdx.x + blockIdx.y + blockIdx.z == 0 && threadIdx.x == 0) {
    next[0] = first.x;
    next[1] = first.y;
  }
  const int col0 = blockIdx.x * kDecayCols, ncol = min(kDecayCols, cols - col0);
  // head of this thread in column col0 + i, or -1
  auto head = [&](int i) {
    const int g = (col0 + i) / pairs, in = ((col0 + i) % pairs) * NH + hs;
    return i < ncol && in < hpg ? g * hpg + in : -1;
  };
  if (record >= rec.n || c < 0 || (long)c * L >= sp.len) {       // (c < 0: offsets that decrease)
    if (sp.len == 0 && c == 0 && a.S_T) {
      for (int i = 0; i < ncol; ++i) {
        const int h = head(i);
        if (h < 0) continue;
        const int n = N * (128 / NH);
        const long at = ((long)seq * a.H + h) * n;
        for (int j = t; j < n; j += 128) a.S_T[at + j] = a.S0 ? a.S0[at + j] : 0.f;
      }
    }
    return;
  }
  const bool row_on = c * L + t < sp.len;
  const bf16_t* dt = static_cast<const bf16_t*>(a.dt) + (sp.row0 + c * L + t) * a.lddt;
  bf16_t raw[kDecayCols];
#pragma unroll
  for (int i = 0; i < kDecayCols; ++i) {
    const int h = head(i);
    if (row_on && h >= 0) raw[i] = dt[h];
  }
  __shared__ float4 tot[kDecayCols][NH];
  float step[kDecayCols], pre[kDecayCols], suf[kDecayCols];
#pragma unroll
  for (int i = 0; i < kDecayCols; ++i) {
    const int h = head(i);
    const bool live = row_on && h >= 0;
    step[i] = live ? softplus(__bfloat162float(raw[i]) + (a.dt_bias ? a.dt_bias[h] : 0.f)) : 0.f;
    // A factor below 2^-128 is 0 wherever its exponent goes into a power; held there, it leaves the sums it is part of
    // as accurate as their other terms are large.
    const float v = live ? step[i] * decay_rate(a.A_log[h]) * kLog2e : 0.f;
    pre[i] = suf[i] = v < -128.f ? -128.f : v;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < kDecayCols; ++i) {
      const float up = __shfl_up_sync(0xffffffffu, pre[i], o);
      const float dn = __shfl_down_sync(0xffffffffu, suf[i], o);
      if (lane >= o) pre[i] += up;
      if (lane < 32 - o) suf[i] += dn;
    }
  }
#pragma unroll
  for (int i = 0; i < kDecayCols; ++i) {
    suf[i] = __shfl_down_sync(0xffffffffu, suf[i], 1);   // the sum over the tokens after this one
    if (lane == 31) {
      suf[i] = 0.f;
      reinterpret_cast<float*>(&tot[i][hs])[q] = pre[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kDecayCols; ++i) {
    if (i >= ncol) break;
    float* vec = vecs + ((col0 + i) * rec.n + record) * (kVec / 4);
    const float4 s4 = tot[i][hs];
    const float before = q == 0 ? 0.f : q == 1 ? s4.x : q == 2 ? s4.x + s4.y : s4.x + s4.y + s4.z;
    const float after = q == 3 ? 0.f : q == 2 ? s4.w : q == 1 ? s4.z + s4.w : s4.y + s4.z + s4.w;
    const int at = hs * 128 + t;
    vec[VU + at] = step[i] * tc::ex2(suf[i]);
    vec[VW + at] = step[i] * tc::ex2(suf[i] + after);
    vec[VE + at] = tc::ex2(pre[i] + before);
    vec[VP + at] = pre[i];
    vec[VP + 256 + at] = pre[i] - log2_step(step[i]);
    if (t == 0) {
      *reinterpret_cast<float4*>(vec + VT + hs * 4) = s4;
      vec[VD + hs] = tc::ex2(s4.x + s4.y + s4.z + s4.w);
    }
  }
}

template <int N, int P, bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
scan_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mb,
            const __grid_constant__ CUtensorMap mbq, const __grid_constant__ CUtensorMap mc,
            const __grid_constant__ CUtensorMap my, const Args k) {
  using Lay = Layout<N, kOut>;
  constexpr int NH = 128 / P;                 // heads of this CTA
  constexpr int NB = N / 64;
  constexpr uint32_t TG = 0, TYI = 128, TYA = 256, TU = kOut ? 384 : 0;
  constexpr uint32_t kTmem = kOut ? 512 : 256;   // (without outputs U has two places)
  const ScanArgs& a = k.a;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = tc::smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (known to be uniform)
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::bars + kBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::bars + kBars * 8 + 8);
  static_assert(kBars * 8 + 12 <= 320, "barriers");
  auto bar = [&](int i) { return sb + Lay::bars + 8u * i; };
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) tc::mbar_init(tc::smem_u32(&bars[i]), i == DRAIN ? (kOut ? 2 : 1) : i >= YR ? 256 : i >= XT ? 128 : 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tc::smem_u32(tmem_slot), kTmem);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  dependency_wait();         // what the launch before wrote is read from here on
  if (!kOut) launch_dependents();
  auto wait = [&](int b, int phase) { bounded_wait(bar(b), (uint32_t)phase & 1u, abort_flag); };
  const int wg = warp >> 2, q = warp & 3;                 // warpgroup; lane quadrant
  const int t = tid & 127;                                // a token's (or hp's) row
  const uint32_t tlane = tmem + ((uint32_t)(32 * q) << 16);
  constexpr int kV = Lay::kVecs;
  // The decay vectors of chunk cc, once their copy has landed.
  auto vectors = [&](int cc) {
    wait(VR + cc % kV, cc / kV);
    return reinterpret_cast<const float*>(smem + Lay::vec + (cc % kV) * kVec);
  };
  // The n-th item of this CTA, for every role but warp 0, which writes it.  Four slots: warp 0 writes item n + 4 when
  // the last chunk of item n + 3 is being loaded, and so after every role has done with chunks three before that.
  struct Item {
    int nc, row0, rows, h0, heads, seg, g, seq, pair;     // chunks (0: no more); first row, tokens from it to the end
  };
  auto item = [&](int n) {
    wait(IQ + (n & 3), n >> 2);
    const int4* r = reinterpret_cast<const int4*>(smem + Lay::queue + (n & 3) * 32);
    const int4 u = r[0], v = r[1];
    return Item{*abort_flag ? 0 : u.x, u.y, u.z, u.w, v.x & 255, v.x >> 8, v.y, v.z, v.w};
  };
  // In every role cc counts this CTA's chunks over all items (phases and buffers go by it), c those of the item.

  if (wg == 0) {
    regs_dec<56>();          // 56 + 72 + 192 + 2 x 80: the registers of five threads at launch (96 each)
    volatile int never = 0;
    if (warp == 0 && lane == 0) {
      // --------------------- items, B, C and the decay vectors -----------------------------------
      const int hpg = a.H / a.G, pairs = (hpg + NH - 1) / NH, per = kOut ? k.segments : k.segments - 1;
      auto load_n = [&](uint32_t dst, const CUtensorMap* m, int b, int col, int row) {
        tc::mbar_arrive_expect_tx(bar(b), NB * kTile);
#pragma unroll 1
        for (int i = 0; i < NB; ++i) tma_load_2d(dst + i * kTile, m, bar(b), col + i * 64, row);
      };
      int cc = 0, n = 0;
#pragma unroll 1
      for (int id = blockIdx.x; id < k.items && !*abort_flag; id = atomicAdd(k.next + (kOut ? 1 : 0), 1)) {
        // the whole pairs first, then the segments of each of the others
        const int cutb = id - (kOut ? k.whole : 0);
        const bool cut = cutb >= 0;
        const int pair = cut ? k.whole + cutb / per : id, seg = cut ? cutb % per : 0;
        const int seq = pair / k.columns, col = pair % k.columns;
        const int g = col / pairs, pr = col % pairs;
        const RowSpan sp = row_span(a.cu, seq, a.T, a.max_len);
        const int ch0 = seg * k.seg_chunks, rows = sp.len - ch0 * L, chunks = (rows + L - 1) / L;
        const int nc = cut ? min(k.seg_chunks, chunks) : chunks;
        if (rows <= 0 || (!kOut && nc == chunks)) continue;       // (without outputs: nor a sequence's last segment)
        const int row0 = (int)(sp.row0 + (long)ch0 * L);
        int4* r = reinterpret_cast<int4*>(smem + Lay::queue + (n & 3) * 32);
        r[0] = make_int4(nc, row0, rows, g * hpg + pr * NH);
        r[1] = make_int4(min(NH, hpg - pr * NH) | seg << 8, g, seq, pair);
        tc::mbar_arrive(bar(IQ + (n & 3)));
        ++n;
        if (a.S0 && seg == 0) {                    // the item's state into L2: warpgroup 2 waits for it
          const float* s0 = a.S0 + ((long)seq * a.H + g * hpg + pr * NH) * N * P;
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(s0), "r"(min(NH, hpg - pr * NH) * N * P * 4)
                       : "memory");
        }
        const float* src = k.vecs + (col * k.records.n + k.records.first(seq, sp.row0) + ch0) * (kVec / 4);
#pragma unroll 1
        for (int c = 0; c < nc && !*abort_flag; ++c, ++cc) {
          // the vectors' slot held chunk cc - kV's, which every role is through with: this thread has seen (with outputs)
          // Yi of cc - 2, issued after y and the state of cc - 3, or U of cc - 2, issued after the state of cc - 4
          if (!kOut && cc >= 2) wait(BE + (cc & 1), (cc >> 1) - 1);
          tc::mbar_arrive_expect_tx(bar(VR + cc % kV), kVec);
          tc::bulk_load(sb + Lay::vec + (cc % kV) * kVec, src + (long)c * (kVec / 4), kVec, bar(VR + cc % kV));
          const int row = row0 + c * L;
          if constexpr (kOut) {
            // There is room for one B tile: a quarter of the next one takes its place as soon as U and G have read that
            // quarter, so that U does not wait for a whole tile.
            if (cc > 0) wait(GD, cc - 1);
#pragma unroll 1
            for (int qd = 0; qd < 4; ++qd) {
              if (cc > 0) wait(BE + qd, cc - 1);
              tc::mbar_arrive_expect_tx(bar(BF + qd), NB * (kTile / 4));
#pragma unroll 1
              for (int i = 0; i < NB; ++i)
                tma_load_2d(sb + Lay::b + i * kTile + qd * (kTile / 4), &mbq, bar(BF + qd), g * N + i * 64, row + qd * 32);
            }
            if (cc > 0) wait(YI, cc - 1);
            load_n(sb + Lay::c, &mc, CF, g * N, row);
          } else {
            load_n(sb + Lay::b + (cc & 1) * NB * kTile, &mb, BF + (cc & 1), g * N, row);
          }
        }
      }
      reinterpret_cast<int4*>(smem + Lay::queue + (n & 3) * 32)[0] = make_int4(0, 0, 0, 0);
      tc::mbar_arrive(bar(IQ + (n & 3)));
      // every load issued lands before the CTA can leave
      if (cc > 0) {
        if (kOut) {
          for (int qd = 0; qd < 4; ++qd) bounded_wait(bar(BF + qd), (cc - 1) & 1, &never);
          bounded_wait(bar(CF), (cc - 1) & 1, &never);
        } else {
          for (int i = max(0, cc - 2); i < cc; ++i) bounded_wait(bar(BF + (i & 1)), (i >> 1) & 1, &never);
        }
        for (int i = max(0, cc - kV); i < cc; ++i) bounded_wait(bar(VR + i % kV), (i / kV) & 1, &never);
      }
    } else if (warp == 2 && lane == 0) {
      // --------------------------------- x and y -----------------------------------------------
      int cc = 0;
      int4 y1 = make_int4(0, 0, 0, 0), y2 = y1;           // y of the last two chunks: (row, column, second tile, whole)
      auto store_y = [&](int4 y, int at) {
        wait(YR + (at & 1), at >> 1);
        if (y.w) {
          const uint32_t src = sb + Lay::x + (at & 1) * 2 * kTile;
          tma_store_2d(&my, src, y.y, y.x);
          if (y.z) tma_store_2d(&my, src + kTile, y.y + 64, y.x);
          tc::bulk_commit();
        }
      };
#pragma unroll 1
      for (int n = 0;; ++n) {
        const Item it = item(n);
        if (it.nc == 0) break;
#pragma unroll 1
        for (int c = 0; c < it.nc && !*abort_flag; ++c, ++cc) {
          const int row = it.row0 + c * L, col = it.h0 * P;
          // a missing second head's tile gets the first one's x: it reaches no row or column that is kept
          const int col1 = NH == 1 || it.heads == 2 ? col + 64 : col;
          if (cc >= 2) {                      // into L2 while the tile is in use: the load then takes half the time
            tma_prefetch_2d(&mx, col, row);
            tma_prefetch_2d(&mx, col1, row);
            if constexpr (kOut) {
              store_y(y2, cc - 2);
              tc::bulk_wait_read_all();
            } else {
              wait(BX + (cc & 1), (cc >> 1) - 1);         // X' of chunk cc - 2 is staged
            }
          }
          const uint32_t dst = sb + Lay::x + (cc & 1) * 2 * kTile, b = bar(XF + (cc & 1));
          tc::mbar_arrive_expect_tx(b, 2 * kTile);
          tma_load_2d(dst, &mx, b, col, row);
          tma_load_2d(dst + kTile, &mx, b, col1, row);
          y2 = y1;
          y1 = make_int4(row, col, NH == 1 || it.heads == 2, it.rows - c * L >= L);
        }
      }
      if (kOut) {
        if (cc >= 2) store_y(y2, cc - 2);
        if (cc >= 1) store_y(y1, cc - 1);
        tc::bulk_wait_all();                  // every store has read its source before the CTA can leave
      }
      for (int i = max(0, cc - 2); i < cc; ++i) bounded_wait(bar(XF + (i & 1)), (i >> 1) & 1, &never);
    } else if (warp == 3) {
      // ----------------------------------- MMAs of U -------------------------------------------
      const uint32_t leader = elect();
      constexpr uint32_t ID_U = tc::idesc_bf16(128, N, true, true);
      const uint64_t dxw = tc::sdesc_sw128(sb + Lay::xw, kTile / 4, 1024);                      // X', K = t
      const uint64_t db0 = tc::sdesc_sw128(sb + Lay::b, kTile, 1024);                           // B, K = t
      int cc = 0;
#pragma unroll 1
      for (int n = 0;; ++n) {
        const int nc = item(n).nc;
        if (nc == 0) break;
#pragma unroll 1
        for (int c = 0; c < nc; ++c, ++cc) {
          const int bbuf = kOut ? 0 : cc & 1;
          const uint64_t dbt = tc::desc_adv(db0, bbuf * NB * kTile);
          if (!kOut) wait(BF + bbuf, cc >> 1);
          if (kOut && cc > 0) wait(UR, cc - 1);
          if (!kOut && cc > 1) wait(UR + bbuf, (cc >> 1) - 1);
          const uint32_t tu = tmem + TU + bbuf * 128;
          // a quarter of the chunk's tokens: 2 steps of 16 for each of the three terms
#pragma unroll 1
          for (int qd = 0; qd < 4; ++qd) {
            if (kOut) wait(BF + qd, cc);
            wait(XT + (qd & 1), 2 * cc + (qd >> 1));
            tc::tc_fence_after();
            const uint64_t dw = tc::desc_adv(dxw, (qd & 1) * kSlot), dq = tc::desc_adv(dbt, qd * (kTile / 4));
#pragma unroll
            for (int i = 0; i < 6; ++i)
              mma_ss(tu, tc::desc_adv(dw, (i >> 1) * (kTile / 2) + (i & 1) * 2048), tc::desc_adv(dq, (i & 1) * 2048),
                     ID_U, qd + i > 0, leader);
            commit(bar(UQ + (qd & 1)), leader);
            if (kOut) commit(bar(BE + qd), leader);
          }
          if (kOut) commit(bar(U1), leader);
          commit(bar(BX + (cc & 1)), leader);
          if (!kOut) commit(bar(BE + bbuf), leader);
        }
      }
      commit(bar(DRAIN), leader);
      bounded_wait(bar(DRAIN), 0, &never);
    } else if (kOut && warp == 1) {
      // ----------------------------------- MMAs of G, Yi, Ya -----------------------------------
      const uint32_t leader = elect();
      constexpr uint32_t ID_G = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t ID_YA = tc::idesc_bf16(128, P, false, true);
      const uint64_t dc = tc::sdesc_sw128(sb + Lay::c, 16, 1024);          // C, K = n
      const uint64_t db = tc::sdesc_sw128(sb + Lay::b, 16, 1024);          // B, K = n
      const uint64_t ds = tc::sdesc_sw128(sb + Lay::s, 16, 1024);          // S^T, K = n
      const uint64_t dx0 = tc::sdesc_sw128(sb + Lay::x, kTile, 1024);      // x, K = t
      int cc = 0;
#pragma unroll 1
      for (int n = 0;; ++n) {
        const int nc = item(n).nc;
        if (nc == 0) break;
#pragma unroll 1
        for (int c = 0; c < nc; ++c, ++cc) {
#pragma unroll 1
          for (int qd = 0; qd < 4; ++qd) wait(BF + qd, cc);
          wait(CF, cc);
          // G = C B^T, then Yi = C S
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {
            if (w) {
              wait(SR, cc);
              if (cc > 0) wait(YR + ((cc - 1) & 1), (cc - 1) >> 1);
            }
            tc::tc_fence_after();
            const uint64_t dn = w ? ds : db;
#pragma unroll 1
            for (int m = 0; m < NB; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_ss(tmem + (w ? TYI : TG), tc::desc_adv(dc, m * kTile + i * 32), tc::desc_adv(dn, m * kTile + i * 32),
                       ID_G, m + i > 0, leader);
            commit(bar(w ? YI : GD), leader);
          }
          wait(XF + (cc & 1), cc >> 1);
          wait(PR, cc);
          tc::tc_fence_after();
          const uint64_t dx = tc::desc_adv(dx0, (cc & 1) * 2 * kTile);
#pragma unroll 1
          for (int hs = 0; hs < NH; ++hs)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mma_ts(tmem + TYA + hs * 64, tmem + TG + 32 * (i >> 1) + 16 * hs + 8 * (i & 1),
                     tc::desc_adv(dx, hs * kTile + i * 2048), ID_YA, i > 0, leader);
          commit(bar(YA), leader);
        }
      }
      commit(bar(DRAIN), leader);
      bounded_wait(bar(DRAIN), 0, &never);
    }
  } else if (wg == 1 || (!kOut && wg == 3)) {
    // ------------------------- X' (without outputs: every other quarter each) --------------------
    regs_dec<72>();
    // this thread's four 16-byte pieces of a quarter: rows (t + 128 i) / 16, piece t % 16 of 16
    const int j = t & 7, tile = (t >> 3) & 1, r0 = t >> 4;
    constexpr int kStep = kOut ? 1 : 2;           // quarters from one of this warpgroup's to its next
    int cc = 0;
#pragma unroll 1
    for (int n = 0;; ++n) {
      const Item it = item(n);
      if (it.nc == 0) break;
#pragma unroll 1
      for (int c = 0; c < it.nc; ++c, ++cc) {
        const int valid = min(L, it.rows - c * L);
        const float* vec = vectors(cc);
        wait(XF + (cc & 1), cc >> 1);
        if (kOut && valid < L) {   // rows behind the sequence reach no product: another sequence's, maybe NaN
          // (G may be reading B meanwhile: it yields columns s >= valid, which no row t < valid keeps)
          for (int i = 0; i < 4; ++i) wait(BF + i, cc);
          zero_rows(sb + Lay::b, NB, valid, t);
        }
#pragma unroll 1
        for (int qd = wg == 1 ? 0 : 1; qd < 4; qd += kStep) {
          const int slot = qd & 1, use = 2 * cc + (qd >> 1);
          if (use > 0) wait(UQ + slot, use - 1);          // the slot is free again
          // three bf16 terms that add up to the fp32 product
          const uint32_t from = sb + Lay::x + ((cc & 1) * 2 + tile) * kTile + qd * (kTile / 4);
          const uint32_t dst = sb + Lay::xw + slot * kSlot + tile * (kTile / 4);
          const float* w_ = vec + VW + (NH == 2 ? tile : 0) * 128 + qd * 32;
#pragma unroll 2
          for (int r = r0; r < 32; r += 8) {
            uint4 xv = tc::ld_shared_v4(from + tc::sw128(r, j));
            if (qd * 32 + r >= valid) xv = make_uint4(0, 0, 0, 0);
            const float w = w_[r];
            const uint64_t ww = tc::f2(w, w);
            const uint32_t in[4] = {xv.x, xv.y, xv.z, xv.w};
            uint32_t o0[4], o1[4], o2[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t f = tc::mul2(tc::f2(tc::bf16lo(in[e]), tc::bf16hi(in[e])), ww);
              float f0, f1;
              tc::f2_get(f, f0, f1);
              o0[e] = tc::pack_bf16(f0, f1);
              const uint64_t g2 = tc::sub2(f, tc::f2(tc::bf16lo(o0[e]), tc::bf16hi(o0[e])));
              tc::f2_get(g2, f0, f1);
              o1[e] = tc::pack_bf16(f0, f1);
              tc::f2_get(tc::sub2(g2, tc::f2(tc::bf16lo(o1[e]), tc::bf16hi(o1[e]))), f0, f1);
              o2[e] = tc::pack_bf16(f0, f1);
            }
            const uint32_t at = dst + tc::sw128(r, j);
            tc::st_shared_v4(at, o0[0], o0[1], o0[2], o0[3]);
            tc::st_shared_v4(at + kTile / 2, o1[0], o1[1], o1[2], o1[3]);
            tc::st_shared_v4(at + kTile, o2[0], o2[1], o2[2], o2[3]);
          }
          tc::fence_proxy_async_smem();
          tc::mbar_arrive(bar(XT + slot));
        }
      }
    }
  } else if (wg == 2) {
    // ----------------------------------- P and the state -----------------------------------------
    regs_inc<192>();
    const int sh = NH == 2 ? (t >> 6) : 0;           // the head of state row t
    const int p = NH == 2 ? (t & 63) : t;
    const long HNP = (long)a.H * N * P;
    constexpr int kRec = N * 128 + 2;                // a segment's record
    uint64_t S[N / 2];                               // row (sh, p) of S^T, in pairs
    auto packed = [&](int i) {
      float f0, f1;
      tc::f2_get(S[i], f0, f1);
      return tc::pack_bf16(f0, f1);
    };
    int cc = 0;
#pragma unroll 1
    for (int n = 0;; ++n) {
      const Item it = item(n);
      if (it.nc == 0) break;
      const bool s_on = sh < it.heads;
      const long srow = (long)it.seq * HNP + (long)(it.h0 + sh) * N * P + p;
      float* wseg = k.ws + (long)(it.pair - k.whole) * (k.segments - 1) * kRec + t;
      // the state before: S0, or those of the segments before, in order
      const float* from0 = it.seg == 0 ? (a.S0 ? a.S0 + srow : nullptr) : wseg;
      const int step = it.seg == 0 ? P : 128;        // distance of two state rows there
      const bool some = s_on && from0 != nullptr && (kOut || it.seg == 0);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) S[i] = 0;
      if (some) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) S[i] = tc::f2(from0[2 * i * step], from0[(2 * i + 1) * step]);
      }
      if (kOut && some && it.seg > 1) {
#pragma unroll
        for (int i0 = 0; i0 < N / 2; i0 += 16) {     // 32 columns at a time: the rest of S is in registers
#pragma unroll 1
          for (int s = 1; s < it.seg; ++s) {
            const float* from = wseg + (long)s * kRec;
            const float d = from[N * 128 + sh - t];
            const uint64_t dd = tc::f2(d, d);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              S[i0 + i] = tc::fma2(dd, S[i0 + i], tc::f2(from[2 * (i0 + i) * 128], from[(2 * (i0 + i) + 1) * 128]));
          }
        }
      }
      float seg_decay = 1.f;
#pragma unroll 1
      for (int c = 0; c < it.nc; ++c, ++cc) {
        if constexpr (kOut) {
          // ---- the copy of S that this chunk's Yi reads, once the one before has read its own
          if (cc > 0) wait(YI, cc - 1);
#pragma unroll
          for (int i = 0; i < N / 8; ++i)
            tc::st_shared_v4(sb + Lay::s + (i >> 3) * kTile + tc::sw128(t, i & 7), packed(4 * i), packed(4 * i + 1),
                             packed(4 * i + 2), packed(4 * i + 3));
          tc::fence_proxy_async_smem();
          tc::mbar_arrive(bar(SR));
        }
        const float* vec = vectors(cc);
        if constexpr (kOut) {
          // ---- P from G
          wait(GD, cc);
          tc::tc_fence_after();
          float mid[NH], mine[NH];
#pragma unroll
          for (int hs = 0; hs < NH; ++hs) mid[hs] = mine[hs] = vec[VP + hs * 128 + t];
#pragma unroll 1
          for (int b = 3; b >= 0; --b) {
            const uint32_t at = tlane + TG + 32 * b;
            if (b > q) {                             // after every token of these rows
              uint32_t o[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = 0;
              tmem_st16(at, o);
              if (NH == 2) tmem_st16(at + 16, o);
              continue;
            }
            float G[32];
            tc::tmem_ld32(at, G);
            tc::tmem_wait_ld();
#pragma unroll 1
            for (int hs = 0; hs < NH; ++hs) {
              uint32_t o[16];
              if (b < q) {
                const float r = tc::ex2(hs ? mid[NH - 1] : mid[0]);
                const uint64_t rr = tc::f2(r, r);
                const float4* u4 = reinterpret_cast<const float4*>(vec + VU + hs * 128 + 32 * b);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float4 u = u4[i];
                  float f0, f1;
                  tc::f2_get(tc::mul2(tc::f2(G[4 * i], G[4 * i + 1]), tc::mul2(tc::f2(u.x, u.y), rr)), f0, f1);
                  o[2 * i] = tc::pack_bf16(f0, f1);
                  tc::f2_get(tc::mul2(tc::f2(G[4 * i + 2], G[4 * i + 3]), tc::mul2(tc::f2(u.z, u.w), rr)), f0, f1);
                  o[2 * i + 1] = tc::pack_bf16(f0, f1);
                }
              } else {
                const float m = hs ? mine[NH - 1] : mine[0];
                const float4* p4 = reinterpret_cast<const float4*>(vec + VP + 256 + hs * 128 + 32 * b);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float4 v = p4[i];            // prefix - log2 D of columns 4 i .. 4 i + 3
                  const float f0 = 4 * i <= lane ? G[4 * i] * tc::ex2(m - v.x) : 0.f;
                  const float f1 = 4 * i + 1 <= lane ? G[4 * i + 1] * tc::ex2(m - v.y) : 0.f;
                  const float f2 = 4 * i + 2 <= lane ? G[4 * i + 2] * tc::ex2(m - v.z) : 0.f;
                  const float f3 = 4 * i + 3 <= lane ? G[4 * i + 3] * tc::ex2(m - v.w) : 0.f;
                  o[2 * i] = tc::pack_bf16(f0, f1);
                  o[2 * i + 1] = tc::pack_bf16(f2, f3);
                }
              }
              tmem_st16(at + 16 * hs, o);
            }
            if (b < q) {                             // the blocks between: whole
#pragma unroll
              for (int hs = 0; hs < NH; ++hs) mid[hs] += vec[VT + hs * 4 + b];
            }
          }
          tc::tmem_wait_st();
          const int valid = min(L, it.rows - c * L);
          if (valid < L) {                           // nor do x's rows behind the sequence reach Ya
            wait(XF + (cc & 1), cc >> 1);
            zero_rows(sb + Lay::x + (cc & 1) * 2 * kTile, 2, valid, t);
            tc::fence_proxy_async_smem();
          }
          tc::tc_fence_before();
          tc::mbar_arrive(bar(PR));
        }
        // ---- S' = exp(c_L) S + U
        if (kOut) wait(U1, cc);
        else wait(BX + (cc & 1), cc >> 1);           // (U runs up to two chunks ahead: kept by place)
        tc::tc_fence_after();
        const uint32_t tu = tlane + TU + (kOut ? 0 : (cc & 1) * 128);
        const float d = vec[VD + sh];
        seg_decay *= d;
        const uint64_t dd = tc::f2(d, d);
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {
          float U[32];
          tc::tmem_ld32(tu + 32 * i, U);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) S[16 * i + e] = tc::fma2(dd, S[16 * i + e], tc::f2(U[2 * e], U[2 * e + 1]));
        }
        tc::tc_fence_before();
        tc::mbar_arrive(bar(UR + (kOut ? 0 : cc & 1)));
      }
      // ---- the state after this item
      if (s_on) {
        if constexpr (kOut) {
          if (it.rows <= it.nc * L && a.S_T) {       // it ends its sequence
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
              float f0, f1;
              tc::f2_get(S[i], f0, f1);
              a.S_T[srow + (long)(2 * i) * P] = f0;
              a.S_T[srow + (long)(2 * i + 1) * P] = f1;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            float f0, f1;
            tc::f2_get(S[i], f0, f1);
            wseg[(long)it.seg * kRec + (2 * i) * 128] = f0;
            wseg[(long)it.seg * kRec + (2 * i + 1) * 128] = f1;
          }
          if (p == 0) wseg[(long)it.seg * kRec + N * 128 + sh - t] = seg_decay;
        }
      }
    }
  } else {
    // ------------------------------------------- y -----------------------------------------------
    regs_dec<80>();
    if constexpr (kOut) {
      const int half = wg - 3;                       // this warpgroup's 64 columns
      const int hs = NH == 2 ? half : 0;             // their head
      const bool gated = a.z != nullptr;
      int cc = 0;
#pragma unroll 1
      for (int n = 0;; ++n) {
        const Item it = item(n);
        if (it.nc == 0) break;
        const bool y_on = hs < it.heads;
        const float skip = a.D && y_on ? a.D[it.h0 + hs] : 0.f;
        const uint64_t skip2 = tc::f2(skip, skip);
        const long col = (long)it.h0 * P + 64 * half;
#pragma unroll 1
        for (int c = 0; c < it.nc; ++c, ++cc) {
          const int valid = min(L, it.rows - c * L);
          const long row = (long)it.row0 + c * L + t;
          const uint32_t xt = sb + Lay::x + (cc & 1) * 2 * kTile;
          const bf16_t* zp = gated ? static_cast<const bf16_t*>(a.z) + row * a.ldz + col : nullptr;
          bf16_t* yp = static_cast<bf16_t*>(a.y) + row * ((long)a.H * P) + col;
          // the gate's values of 16 columns (piece i of this warpgroup's four)
          auto load_z = [&](int i, uint4 (&zr)[2]) {
            const bool on = gated && t < valid && y_on;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              zr[e] = make_uint4(0, 0, 0, 0);
              if (!on) continue;
              zr[e] = *reinterpret_cast<const uint4*>(zp + 16 * i + 8 * e);
            }
          };
          uint4 za[2], zb[2];                        // this piece's and the next one's
          load_z(0, za);
          load_z(1, zb);
          if (gated && y_on && (c + 1) * L + t < it.rows && c + 1 < it.nc)     // the next chunk's into L2
            asm volatile("prefetch.global.L2 [%0];" ::"l"(zp + L * a.ldz));
          wait(XF + (cc & 1), cc >> 1);
          wait(BX + (cc & 1), cc >> 1);              // warpgroup 1 has read x's tile: y may take its place
          wait(YA, cc);
          tc::tc_fence_after();
          const float e = vectors(cc)[VE + hs * 128 + t];
          const uint64_t e2 = tc::f2(e, e);
#pragma unroll 1
          for (int i = 0; i < 4 && y_on; ++i) {
            float yi[16], ya[16];
            tmem_ld16(tlane + TYI + 64 * half + 16 * i, yi);
            tmem_ld16(tlane + TYA + 64 * half + 16 * i, ya);
            const uint32_t at0 = xt + half * kTile + tc::sw128(t, 2 * i), at1 = xt + half * kTile + tc::sw128(t, 2 * i + 1);
            const uint4 xq[2] = {tc::ld_shared_v4(at0), tc::ld_shared_v4(at1)};
            tc::tmem_wait_ld();
            uint32_t o[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t xi[4] = {xq[m].x, xq[m].y, xq[m].z, xq[m].w};
              const uint32_t zi[4] = {za[m].x, za[m].y, za[m].z, za[m].w};
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const int at = 8 * m + 2 * f;
                uint64_t y2 = tc::fma2(skip2, tc::f2(tc::bf16lo(xi[f]), tc::bf16hi(xi[f])), tc::f2(ya[at], ya[at + 1]));
                y2 = tc::fma2(e2, tc::f2(yi[at], yi[at + 1]), y2);
                if (gated) {
                  const float z0 = tc::bf16lo(zi[f]), z1 = tc::bf16hi(zi[f]);
                  y2 = tc::mul2(y2, tc::mul2(tc::f2(z0, z1), tc::f2(sigmoid(z0), sigmoid(z1))));
                }
                float f0, f1;
                tc::f2_get(y2, f0, f1);
                o[m][f] = tc::pack_bf16(f0, f1);
              }
            }
            if (valid == L) {
              tc::st_shared_v4(at0, o[0][0], o[0][1], o[0][2], o[0][3]);
              tc::st_shared_v4(at1, o[1][0], o[1][1], o[1][2], o[1][3]);
            } else if (t < valid) {
              uint4* to = reinterpret_cast<uint4*>(yp + 16 * i);
              to[0] = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
              to[1] = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
            }
            za[0] = zb[0];                           // loaded a piece ago
            za[1] = zb[1];
            if (i < 2) load_z(i + 2, zb);
          }
          tc::tc_fence_before();
          tc::fence_proxy_async_smem();
          tc::mbar_arrive(bar(YR + (cc & 1)));
        }
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_relinquish();
    tc::tmem_dealloc(tmem, kTmem);
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
// [rows, cols] bf16, rows ld values apart, boxes of 64 columns x box_rows, 128-byte swizzle; rows
// past the end load as zeros and are not stored.
inline bool make_map(CUtensorMap* m, const void* base, long rows, long cols, long ld, int box_rows = L) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool supported(int P, int N) { return (P == 64 || P == 128) && (N == 64 || N == 128); }
inline int columns(int H, int G, int P) {       // CTAs of one sequence and segment
  const int nh = 128 / P;
  return G * ((H / G + nh - 1) / nh);
}
// How the pairs are cut, a rule on sizes alone (so that the workspace can be sized without a device).  Of n pairs
// floor(n / 148) full waves run whole; the rest r is cut into as many segments as fill one more wave, none shorter than
// four chunks (a segment costs the first launch and the combination, about two chunks' time).  4 x 48 pairs of 16
// chunks (inputs in L2): 132 us whole in two waves, of which the second has 44 CTAs, and 123 cut when that was compared; 114
// now.  From five waves on nothing is cut.
struct Cut {
  int whole, segments;
};
inline Cut cut(int nseq, int max_len, int H, int G, int P) {
  const long n = (long)nseq * columns(H, G, P), rest = n % 148;
  const int chunks = max_len / L + (max_len % L != 0);
  if (rest == 0 || n > 148 * 5) return Cut{(int)n, 1};
  const long s = 148 / rest < chunks / 4 ? 148 / rest : chunks / 4;
  return s < 2 ? Cut{(int)n, 1} : Cut{(int)(n - rest), (int)s};
}
// The workspace: the item counters (256 bytes), segment states and decays, the decay vectors (total: rows of a packed
// call, -1 where that is not known).
struct Space {
  size_t vecs, bytes;
};
inline Space space(int nseq, int max_len, long total, int H, int G, int P, int N) {
  const Cut c = cut(nseq, max_len, H, G, P);
  const size_t cols = (size_t)columns(H, G, P), pairs = nseq * cols;
  const size_t states = ((pairs - c.whole) * (c.segments - 1) * (N * 128 + 2) * sizeof(float) + 255) / 256 * 256;
  return Space{256 + states, 256 + states + cols * records_of(nseq, max_len, total).n * kVec};
}

// A launch that may be placed before the one before it in its stream has completed.
template <auto kern, int smem, typename... A>
bool launch_after(int ctas, cudaStream_t st, const A&... args) {
  if (!allow_smem<kern, smem>()) return false;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)ctas);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  cudaLaunchKernelEx(&c, kern, args...);
  return cudaGetLastError() == cudaSuccess;
}

template <int N, int P>
int launch_np(const ScanArgs& a, void* ws, cudaStream_t st) {
  constexpr int NH = 128 / P;
  const long rows = a.cu ? (long)a.T : (long)a.nseq * a.T;
  const long total = a.cu ? (long)a.T : -1L;
  const Records rec = records_of(a.nseq, a.max_len, total);
  const Cut ct = cut(a.nseq, a.max_len, a.H, a.G, P);
  const int cols = columns(a.H, a.G, P);
  const long pairs = (long)a.nseq * cols, rest = pairs - ct.whole;
  float* vecs = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + space(a.nseq, a.max_len, total, a.H, a.G, P, N).vecs);
  int* next = static_cast<int*>(ws);
  Args k{a, next, reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256), vecs, rec, cols, ct.whole,
         (rec.chunks + ct.segments - 1) / ct.segments, ct.segments, 0};
  const long cut_items = rest * (ct.segments - 1), items = ct.whole + rest * ct.segments;
  if (items > 0x3fffffffL) return GDN_ERR_UNSUPPORTED;
  // records over y and z (by rows there are 2^23 + nseq at most, otherwise nseq of at most 65535 chunks each)
  const long gy = rec.by_rows ? (rec.n < 65535 ? rec.n : 65535) : rec.chunks, gz = (rec.n + gy - 1) / gy;
  const int2 ctas = make_int2((int)(cut_items < 148 ? cut_items : 148), (int)(items < 148 ? items : 148));
  CUtensorMap mx, mb, mbq, mc, my;
  if (!make_map(&mx, a.x, rows, (long)a.H * P, a.ldx) || !make_map(&mb, a.B, rows, (long)a.G * N, a.ldb) ||
      !make_map(&mbq, a.B, rows, (long)a.G * N, a.ldb, L / 4) || !make_map(&mc, a.C, rows, (long)a.G * N, a.ldc) || !make_map(&my, a.y, rows, (long)a.H * P, (long)a.H * P))
    return GDN_ERR_CUDA;
  decay_kernel<NH><<<dim3((unsigned)((cols + kDecayCols - 1) / kDecayCols), (unsigned)gy, (unsigned)gz), 128 * NH, 0, st>>>(
      a, rec, vecs, next, ctas, N, cols);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  if (rest > 0) {
    k.items = (int)cut_items;
    if (!launch_after<scan_kernel<N, P, false>, (int)Layout<N, false>::alloc>(ctas.x, st, mx, mb, mbq, mc, my, k))
      return GDN_ERR_CUDA;
  }
  k.items = (int)items;
  return launch_after<scan_kernel<N, P, true>, (int)Layout<N, true>::alloc>(ctas.y, st, mx, mb, mbq, mc, my, k)
             ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace tcs
}  // namespace ssm
}  // namespace gdn
