// What the two kernels of the gated delta rule in blocks share: the records of
// the blocks' solutions in the workspace, and where a slot's tokens lie.
//
// With g the sum of the log decays from the block's first token on, i, j its
// tokens and S0 the state that enters it:
//     (1 + A) U = beta (X - e^g K S0^T),  A_ij = beta_i e^(g_i - g_j) k_i k_j (j < i)
//     Y = scale (e^g Q S0^T + M U),       M_ij = e^(g_i - g_j) q_i k_j     (j <= i)
//     S = e^g_end S0 + U^T e^(g_end - g) K
// A record holds, for one block and head, T = (1 + A)^-1 beta and scale M as
// matrix-core operands, and the decays. T is 16 bits or more (two bf16 terms);
// M one bf16, or two for fp32 io.
#pragma once

#include "delta.h"
#include "mfma_common.h"

namespace ssd {

constexpr int kTriFrags = 6;  // 16 x 32 operands of a lower triangle of 64 x 64: those of its 32 x 32 blocks
constexpr int kFragBytes = 1024;
// Operand of rows 32 kk + .. (half h of them) and columns 32 ks + .., ks <= kk.
constexpr int tri_frag(int kk, int h, int ks) { return kk == 0 ? h : 2 + 2 * h + ks; }

template <int TERMS> struct DeltaRecord {  // TERMS: of the io type's operands
  static constexpr int T_hi = 0, T_lo = kTriFrags * kFragBytes, M = 2 * kTriFrags * kFragBytes,
                       decays = M + TERMS * kTriFrags * kFragBytes,  // e^g [64], e^(g_end - g) [64]
                       bytes = decays + 512;
};

// Tokens of a slot: n (0: the slot is empty) from token t0 of batch row `row`.
struct DeltaSlot {
  int64_t row, t0;
  int n;
};
__device__ __forceinline__ int64_t delta_first_slot(const DeltaArgs& a, int64_t s) {
  return seq_offset(a.cu, s, a.L) / kDeltaBlock + s;
}
// (by a whole wave)
__device__ __forceinline__ DeltaSlot delta_slot(const DeltaArgs& a, int64_t slot) {
  DeltaSlot r;
  if (a.cu == nullptr) {
    const int64_t nc = (a.L + kDeltaBlock - 1) / kDeltaBlock;
    r.row = slot / nc;
    r.t0 = (slot - r.row * nc) * kDeltaBlock;
    r.n = (int)(a.L - r.t0 < kDeltaBlock ? a.L - r.t0 : kDeltaBlock);
    return r;
  }
  // the last sequence whose slots begin at or before this one
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, n = a.nseq;
  while (n > 1) {
    const int64_t step = (n + 63) / 64;
    const int64_t i = lo + lane * step;
    const bool le = lane * step < n && delta_first_slot(a, i) <= slot;
    const uint64_t m = __ballot(le);
    const int k = m == 0 ? 0 : 63 - __builtin_clzll(m);
    const int64_t left = n - k * step;
    lo += k * step;
    n = left < step ? left : step;
  }
  const int64_t first = seq_offset(a.cu, lo, a.L), last = seq_offset(a.cu, lo + 1, a.L);
  const int64_t c = slot - delta_first_slot(a, lo);
  r.row = 0;
  r.t0 = first + c * kDeltaBlock;
  const int64_t left = last - r.t0;
  r.n = c < 0 || left < 1 ? 0 : (int)(left < kDeltaBlock ? left : kDeltaBlock);
  return r;
}

// Eight consecutive elements from column n on of a row of N (zeros behind it,
// or all zeros), as they lie in memory.
template <typename TIO> struct Raw8;
template <> struct Raw8<__hip_bfloat16> { uint4 v; };
template <> struct Raw8<float> { uint4 v, w; };
template <typename TIO>
__device__ __forceinline__ Raw8<TIO> load8(const TIO* row, int n, int N, bool there) {
  Raw8<TIO> r;
  if (N % 8 == 0) {
    const bool in = there && n < N;
    const TIO* p = row + (in ? n : 0);
    __builtin_memcpy(&r, p, sizeof(r));
    r.v = in ? r.v : make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(TIO) == 4) r.w = in ? r.w : make_uint4(0, 0, 0, 0);
  } else {
    const int nn = !there || n >= N ? 0 : N - n < 8 ? N - n : 8;
    if (nn == 8) {
      __builtin_memcpy(&r, row + n, sizeof(r));
    } else {
      Pack<TIO, 8> p;
#pragma unroll
      for (int i = 0; i < 8; ++i) p.v[i] = i < nn ? reinterpret_cast<const typename Elem<TIO>::raw*>(row)[n + i] : 0;
      __builtin_memcpy(&r, &p, sizeof(r));
    }
  }
  return r;
}

// fp32 values as a bf16 and the bf16 of what it leaves. (An infinity leaves a NaN.)
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  lo = pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi));
}
__device__ __forceinline__ void split8(const float (&f)[8], uint4& hi, uint4& lo) {
  split2(f[0], f[1], hi.x, lo.x);
  split2(f[2], f[3], hi.y, lo.y);
  split2(f[4], f[5], hi.z, lo.z);
  split2(f[6], f[7], hi.w, lo.w);
}
__device__ __forceinline__ void split_raw(const Raw8<float>& r, uint4& hi, uint4& lo) {
  const float f[8] = {__uint_as_float(r.v.x), __uint_as_float(r.v.y), __uint_as_float(r.v.z), __uint_as_float(r.v.w),
                      __uint_as_float(r.w.x), __uint_as_float(r.w.y), __uint_as_float(r.w.z), __uint_as_float(r.w.w)};
  split8(f, hi, lo);
}

}  // namespace ssd
