// What the two kernels of the gated delta rule in blocks share: the records of
// the blocks' solutions in the workspace, and where a slot's tokens lie.
//
// With g the sum of the log decays from the block's first token on, i, j its
// tokens and S0 the state that enters it:
//     (1 + A) U = beta (X - e^g K S0^T),  A_ij = beta_i e^(g_i - g_j) k_i k_j (j < i)
//     Y = scale (e^g Q S0^T + M U),       M_ij = e^(g_i - g_j) q_i k_j     (j <= i)
//     S = e^g_end S0 + U^T e^(g_end - g) K
// A record holds, for one block and head, T = (1 + A)^-1 beta and scale M as
// matrix-core operands, and the decays.
//
// Operands of the matrix cores are bf16, so an fp32 value enters a product as a sum
// of terms: itself rounded, what that leaves rounded, and so on. Terms:
//   io     B and C: 1 with bf16 io (exact), 3 with fp32 io
//   state  S, R, T, U' (all that reaches a state): 2 with bf16 io (off by 2^-16),
//          3 with fp32 io (off by 2^-24)
//   y      S, U, M in y's own products: 1 with bf16 io, beside y's rounding; 3
// With bf16 io more terms are more matrix instructions of the chain, which bounds the walk,
// and at N = 128, P > 64 neither its registers nor the LDS has room for them. Smaller instances
// have (146 to 199 of 256 registers); they take the same terms, so that what a result is off by does not
// hang on P and N. Measured errors, 2-norm, against 64 bits: y 2.8e-3 (its own rounding 1.7e-3), states
// 3.6e-6 to 5.4e-6; where one key fills a block, so that y is a small difference of its solutions,
// y up to 1.9e-2 (fp32 io 5.7e-6), states 7.9e-5.
#pragma once

#include "delta.h"
#include "mfma_common.h"

namespace ssd {

template <typename TIO> struct DeltaTerms {
  static constexpr bool wide = sizeof(TIO) == 4;
  static constexpr int io = wide ? 3 : 1, state = wide ? 3 : 2, y = wide ? 3 : 1;
};

constexpr int kTriFrags = 6;  // 16 x 32 operands of a lower triangle of 64 x 64: those of its 32 x 32 blocks
constexpr int kFragBytes = 1024;
// Operand of rows 32 kk + .. (half h of them) and columns 32 ks + .., ks <= kk.
constexpr int tri_frag(int kk, int h, int ks) { return kk == 0 ? h : 2 + 2 * h + ks; }

template <typename TIO> struct DeltaRecord {
  static constexpr int T = 0, M = T + DeltaTerms<TIO>::state * kTriFrags * kFragBytes,
                       decays = M + DeltaTerms<TIO>::y * kTriFrags * kFragBytes,  // e^g [64], e^(g_end - g) [64]
                       bytes = decays + 512;
};

// fp32 values as terms, packed in pairs.
template <int T> __device__ __forceinline__ void split2(float a, float b, uint32_t (&w)[T]) {
#pragma unroll
  for (int i = 0; i < T; ++i) {
    w[i] = pack_bf16x2(a, b);
    if (i + 1 < T) a -= bf16_lo(w[i]), b -= bf16_hi(w[i]);
  }
}
// Operand of T terms.
template <int T> struct Terms { bf16x8_t v[T]; };
template <int T> __device__ __forceinline__ Terms<T> split8(const float (&f)[8]) {
  uint32_t w[4][T];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2<T>(f[2 * i], f[2 * i + 1], w[i]);
  Terms<T> r;
#pragma unroll
  for (int i = 0; i < T; ++i) r.v[i] = as_bf16x8(make_uint4(w[0][i], w[1][i], w[2][i], w[3][i]));
  return r;
}
// acc += A B, one of its pairs of terms (all that are as large as the longer
// operand's last): a caller spreads them over accumulators.
constexpr int term_pairs(int ta, int tb) {
  int n = 0;
  for (int i = 0; i < ta; ++i)
    for (int j = 0; j < tb; ++j) n += i + j < (ta > tb ? ta : tb);
  return n;
}
template <int TA, int TB> __device__ __forceinline__ void mul_pair(f32x4_t& acc, const Terms<TA>& a, const Terms<TB>& b, int pair) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
      if (i + j < (TA > TB ? TA : TB)) {
        if (n == pair) acc = mfma_16x16x32(a.v[i], b.v[j], acc);
        ++n;
      }
}

// A slot of `unit` tokens: its sequence, the index of that among those in blocks,
// which of the sequence's slots it is, the sequence's tokens [first, last), of
// batch row `row`, and the slot's own: from t0 up to t1 (t1 <= t0: the slot is empty).
struct DeltaSlot {
  int64_t seq, index, part, row, first, last, t0, t1;
};
// Of a packed stream: the sequence that is the i-th in blocks, -1 behind the last; where it begins.
__device__ __forceinline__ int64_t delta_seq(const DeltaArgs& a, int64_t i) { return a.longs != nullptr ? a.longs[i] : i; }
__device__ __forceinline__ int64_t delta_begin(const DeltaArgs& a, int64_t seq) { return seq < 0 ? a.L : seq_offset(a.cu, seq, a.L); }
// (Tokens, slots and units are below 2^31: their quotients are taken in 32 bits.)
__device__ __forceinline__ int64_t delta_first_slot(const DeltaArgs& a, int64_t i, uint32_t unit) {
  return a.cu != nullptr ? (uint32_t)delta_begin(a, delta_seq(a, i)) / unit + i : i * (((uint32_t)a.L + unit - 1) / unit);
}
// (by a whole wave)
__device__ __forceinline__ DeltaSlot delta_slot(const DeltaArgs& a, uint32_t slot, uint32_t unit) {
  DeltaSlot r;
  if (a.cu == nullptr) {
    const uint32_t nc = ((uint32_t)a.L + unit - 1) / unit;
    r.seq = r.index = r.row = slot / nc;
    r.first = 0, r.last = a.L;
  } else {
    // the last sequence whose slots begin at or before this one
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, n = a.upto > 0 ? (uint32_t)a.L / (uint32_t)(a.upto + 1) : a.nseq;
    while (n > 1) {
      const int64_t step = (n + 63) / 64;
      const int64_t i = lo + lane * step;
      const bool le = lane * step < n && delta_first_slot(a, i, unit) <= (int64_t)slot;
      const uint64_t m = __ballot(le);
      const int k = m == 0 ? 0 : 63 - __builtin_clzll(m);
      const int64_t left = n - k * step;
      lo += k * step;
      n = left < step ? left : step;
    }
    r.seq = delta_seq(a, lo), r.index = lo, r.row = 0;
    r.first = delta_begin(a, r.seq), r.last = delta_begin(a, r.seq < 0 ? r.seq : r.seq + 1);
  }
  r.part = (int64_t)slot - delta_first_slot(a, r.index, unit);
  r.t0 = r.first + r.part * unit;
  r.t1 = r.t0 + unit < r.last ? r.t0 + unit : r.last;
  if (r.part < 0) r.t1 = r.t0;  // (before the first sequence)
  return r;
}

// What a workgroup walks: a sequence, or (a.seg != 0) one of the sequences' segments.
// PASS 0: from the states that enter them. PASS 1: over segments, what becomes of a
// state of zeros (rows p) and, with values of zero, of the unit states (rows P + n),
// see delta_join. False: nothing to walk.
template <int PASS> __device__ __forceinline__ bool delta_piece(const DeltaArgs& a, int64_t piece, DeltaSlot& sl) {
  if (a.seg != 0) {
    sl = delta_slot(a, (uint32_t)piece, (uint32_t)a.seg);
    if (sl.part < 0 || (sl.part > 0 && sl.t1 <= sl.t0)) return false;
    return PASS == 0 || sl.t1 < sl.last;  // nothing begins behind the last one
  }
  sl.seq = sl.index = piece, sl.part = 0, sl.row = a.cu != nullptr ? 0 : piece;
  if (a.longs != nullptr) {
    sl.seq = a.longs[piece];
    if (sl.seq < 0) return false;
  }
  sl.t0 = sl.first = a.cu != nullptr ? seq_offset(a.cu, sl.seq, a.L) : 0;
  sl.t1 = sl.last = a.cu != nullptr ? seq_offset(a.cu, sl.seq + 1, a.L) : a.L;
  return true;
}

// Where the 16-byte piece c of row t lies in K's and Q's tile in LDS: c with these
// bits flipped.
template <int NP> __device__ __forceinline__ int k_swz(int t) {
  return NP >= 128 ? ((t & 3) << 2) | ((t >> 3) & 3) : NP == 64 ? ((t & 2) << 1) | ((t >> 3) & 3) : (t >> 3) & 3;
}

// One matrix product, then V ordinary instructions, M times: what runs beside what.
template <int M, int V> __device__ __forceinline__ void spread() {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x2, V, 0);
  }
}

// Rows of a block's tokens through a buffer descriptor: what lies behind the
// block's last row reads as zeros, and so does an offset of kNowhere. Pieces of
// eight elements; where N is no multiple of eight (WHOLE false) the last piece of
// a row ends with it and is moved into place after the load.
constexpr uint32_t kNowhere = 0x7ffffff0u;
template <typename TIO> struct Piece;
template <> struct Piece<__hip_bfloat16> { uint4 v; };
template <> struct Piece<float> { uint4 v, w; };
template <typename TIO>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t block_rows(const TIO* first, int64_t token, int n, int N) {
  return buffer_range(const_cast<TIO*>(first), (uint32_t)((n - 1) * token + N) * (uint32_t)sizeof(TIO));
}
__device__ __forceinline__ uint4 buffer_ld16(__amdgpu_buffer_rsrc_t rows, uint32_t off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rows, (int)off, 0, 0));
}
// Byte offset of the piece from column c on within its row, and how many
// elements it is moved by.
template <typename TIO, bool WHOLE>
__device__ __forceinline__ uint32_t piece_at(int c, int N, int& moved, int len = 8) {
  moved = 0;
  if (c >= N) return kNowhere;
  if (!WHOLE && c + len > N) moved = c + len - N;
  return (uint32_t)(c - moved) * (uint32_t)sizeof(TIO);
}
// row: its byte offset
template <typename TIO> __device__ __forceinline__ Piece<TIO> load_piece(__amdgpu_buffer_rsrc_t rows, uint32_t row, uint32_t at) {
  const uint32_t off = at == kNowhere ? kNowhere : row + at;
  Piece<TIO> r;
  r.v = buffer_ld16(rows, off);
  if constexpr (sizeof(TIO) == 4) r.w = buffer_ld16(rows, off + 16);
  return r;
}
// W words down by `moved` elements (fewer than W words'), zeros behind.
template <typename TIO, int W> __device__ __forceinline__ void move_down(uint32_t (&w)[W], int moved) {
  int words = moved;
  if constexpr (sizeof(TIO) == 2) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t above = i + 1 < W ? w[i + 1] : 0u;
      w[i] = moved & 1 ? (w[i] >> 16) | (above << 16) : w[i];
    }
    words = moved / 2;
  }
#pragma unroll
  for (int s = 1; s < W; s *= 2)
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = words & s ? (i + s < W ? w[i + s] : 0u) : w[i];
}
template <typename TIO, bool WHOLE> __device__ __forceinline__ void move_piece(Piece<TIO>& p, int moved) {
  if constexpr (!WHOLE) {
    constexpr int W = sizeof(Piece<TIO>) / 4;
    uint32_t w[W];
    __builtin_memcpy(w, &p, sizeof(p));
    move_down<TIO, W>(w, moved);
    __builtin_memcpy(&p, w, sizeof(p));
  }
}

template <int T> __device__ __forceinline__ Terms<T> split_piece(const Piece<float>& r) {
  const float f[8] = {__uint_as_float(r.v.x), __uint_as_float(r.v.y), __uint_as_float(r.v.z), __uint_as_float(r.v.w),
                      __uint_as_float(r.w.x), __uint_as_float(r.w.y), __uint_as_float(r.w.z), __uint_as_float(r.w.w)};
  return split8<T>(f);
}

// Nothing is moved across by the compiler: no memory access by any of its passes,
// nothing at all by the scheduler.
__device__ __forceinline__ void hold() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace ssd
