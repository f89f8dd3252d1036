// The gated delta rule in blocks, first kernel: for every block of 64 tokens
// and head, the solution T = (1 + A)^-1 beta of its triangular system and its
// scores M (delta_blocks.h), as operands for the second kernel.
//
// One wave to a block and head; nothing is shared, so there is no barrier.
// The products with K run on the matrix cores (only the tiles on and below the
// diagonal), operands straight from memory and all on their way at once, rows
// numbered 8 (r / 4) + 4 h + r % 4 in a pair of tiles h: the pair then leaves
// eight consecutive columns j of a row i in a lane, M's operands as they stand, and
// A in 16-byte writes. The decays' exponents g_i - g_j are
// differences of sums in 64 bits: in 32, one token that decays by e^-300 would cost
// the tokens behind it five digits. The inverse is taken in fp32 in three
// steps: the four 16 x 16 blocks of the diagonal by substitution, a column to a
// lane; then T10 = -T11 A10 T00 for the two pairs of them, and once more for the
// two halves, as products of fp32 matrix instructions, whose result in
// registers is the right operand of the next as it stands.
//
// Bound by memory, two waves a SIMD covering it poorly: 8192 blocks of N = 128, bf16 (74 MB in
// from memory, 152 MB of records out) 65 us; without the stores 45, without the
// loads 42, without both 33. Three waves a SIMD spill and took 67.
#include "delta_blocks.h"

namespace ssd {
namespace {

constexpr int kWaves = 4;
// The matrix's rows of 16-blocks 0 .. i: floats from one row to the next, and where
// the first of them lies.
constexpr int pitch(int i) { return 16 * (i + 1) + 4; }
constexpr int base(int i) { return i == 0 ? 0 : base(i - 1) + 16 * pitch(i - 1); }
// a token's log2 decay: exp2 of either end is 0 or infinity by far, and a sum of 64 keeps its digits
constexpr float kMostDecay = 1024.f;

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
// The value of another lane of the wave (DPP), 0 where there is none.
template <int CTRL, int ROWS> __device__ __forceinline__ double from_lane(double v) {
  const int2 w = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_update_dpp(0, w.x, CTRL, ROWS, 0xf, false),
                                              __builtin_amdgcn_update_dpp(0, w.y, CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ f32x4_t ld4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }
// D += A B of 16 x 16 each: a = A[r][4 g ..], b = B[4 g ..][r]
__device__ __forceinline__ f32x4_t mul16(const f32x4_t& a, const f32x4_t& b, f32x4_t d) {
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], d, 0, 0, 0);
  return d;
}

// The same of 16 x 32 and 32 x 16: fp32 io by fp32 instructions, one of every
// piece's elements each.
__device__ __forceinline__ f32x4_t product(const Piece<__hip_bfloat16>& a, const Piece<__hip_bfloat16>& b, const f32x4_t& d) {
  return mfma_16x16x32(as_bf16x8(a.v), as_bf16x8(b.v), d);
}
__device__ __forceinline__ f32x4_t product(const Piece<float>& a, const Piece<float>& b, f32x4_t d) {
  d = mul16(__builtin_bit_cast(f32x4_t, a.v), __builtin_bit_cast(f32x4_t, b.v), d);
  return mul16(__builtin_bit_cast(f32x4_t, a.w), __builtin_bit_cast(f32x4_t, b.w), d);
}

template <typename TIO, typename TDT, int NP, bool WHOLE>
__global__ __launch_bounds__(64 * kWaves, sizeof(TIO) == 2 && NP <= 128 ? 2 : 1) void delta_solve_kernel(const DeltaArgs a, uint32_t tasks) {
  constexpr int KS = NP / 32;
  constexpr int TT = DeltaTerms<TIO>::state, MT = DeltaTerms<TIO>::y;
  using Rec = DeltaRecord<TIO>;
  using RD = typename Elem<TDT>::raw;
  struct Shared {
    float m[base(4)];
    double g[64];
    float beta[64];
  };
  __shared__ __align__(16) Shared shared[kWaves];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const uint32_t task = blockIdx.x * kWaves + wave;  // (below 2^31)
  if (task >= tasks) return;
  const uint32_t slot = task / (uint32_t)a.H;
  const int h = (int)(task - slot * a.H);
  const DeltaSlot at = delta_slot(a, slot, kDeltaBlock);
  if (at.t1 <= at.t0) return;
  const int n = (int)(at.t1 - at.t0);
  Shared& sh = shared[wave];
  float* m = sh.m;
  char* rec = a.ws + (int64_t)task * Rec::bytes;

  // columns 32 ks + 8 g .. of a row
  const int grp = (int)((uint32_t)h / ((uint32_t)a.H / (uint32_t)a.G));
  const TIO* Bp = static_cast<const TIO*>(a.B) + at.row * a.bs.batch + at.t0 * a.bs.token + (int64_t)grp * a.N;
  const TIO* Cp = static_cast<const TIO*>(a.C) + at.row * a.cs.batch + at.t0 * a.cs.token + (int64_t)grp * a.N;
  uint32_t col[KS];
  int moved[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) col[ks] = piece_at<TIO, WHOLE>(32 * ks + 8 * g, a.N, moved[ks]);
  auto rows = [&](__amdgpu_buffer_rsrc_t from, int64_t token, int t, Piece<TIO>(&v)[KS]) {
    const uint32_t row = (uint32_t)(t * (int)token) * (uint32_t)sizeof(TIO);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) v[ks] = load_piece<TIO>(from, row, col[ks]);
  };
  auto placed = [&](Piece<TIO>(&v)[KS]) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) move_piece<TIO, WHOLE>(v[ks], moved[ks]);
  };
  const __amdgpu_buffer_rsrc_t Br = block_rows(Bp, a.bs.token, n, a.N), Cr = block_rows(Cp, a.cs.token, n, a.N);
  const bool there = lane < n;
  const int64_t token = at.t0 + (there ? lane : 0);
  const RD dt = static_cast<const RD*>(a.dt)[at.row * a.ds.batch + token * a.ds.token + h];
  const RD be = static_cast<const RD*>(a.beta)[at.row * a.es.batch + token * a.es.token + h];
  const float bias = a.dto.bias != nullptr ? a.dto.bias[h] : 0.f, Ah = a.A[h];
  // tile (kk, hh): rows 32 kk + 8 (r / 4) + 4 hh + r % 4
  Piece<TIO> k[2][2][KS], q[2][2][KS];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) rows(Br, a.bs.token, 32 * kk + 8 * (r / 4) + 4 * hh + r % 4, k[kk][hh]);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) rows(Cr, a.cs.token, 32 * kk + 8 * (r / 4) + 4 * hh + r % 4, q[kk][hh]);
  }
  hold();

  // a lane to a token: beta, and the sum of the log2 decays
  {
    const float l = clamped(delta_log2_decay(Elem<TDT>::f32(dt), bias, Ah, a.dto), -kMostDecay, kMostDecay);
    double sum = there ? (double)l : 0.0;
    sum += from_lane<0x111, 0xf>(sum);  // 1, 2, 4 and 8 lanes below, in rows of 16
    sum += from_lane<0x112, 0xf>(sum);
    sum += from_lane<0x114, 0xf>(sum);
    sum += from_lane<0x118, 0xf>(sum);
    sum += from_lane<0x142, 0xa>(sum);  // the end of the row below
    sum += from_lane<0x143, 0xc>(sum);  // the end of the lower half
    const int2 w = __builtin_bit_cast(int2, sum);
    const double end = __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(w.x, 63), __builtin_amdgcn_readlane(w.y, 63)));
    sh.g[lane] = sum;
    sh.beta[lane] = there ? delta_beta(Elem<TDT>::f32(be), a.sigmoid) : 0.f;
    float* dec = reinterpret_cast<float*>(rec + Rec::decays);
    dec[lane] = __builtin_amdgcn_exp2f((float)sum);
    dec[64 + lane] = __builtin_amdgcn_exp2f((float)(end - sum));
  }
  wave_sync();

  // tiles (kk, hh) against (kc, hc): rows j = 32 kk + 8 g + 4 hh + e, column i
#pragma unroll
  for (int kc = 0; kc < 2; ++kc) {
#pragma unroll
    for (int hc = 0; hc < 2; ++hc) placed(k[kc][hc]), placed(q[kc][hc]);
#pragma unroll
    for (int hc = 0; hc < 2; ++hc) {
      const int in = 8 * (r / 4) + 4 * hc + r % 4, i = 32 * kc + in;
      const bool lower = in >= 16;
      const double gi = sh.g[i];
      const float beta = sh.beta[i];
      // (row i of the matrix has room up to its own 16-block)
      float* row = m + (lower ? base(2 * kc + 1) + (in - 16) * pitch(2 * kc + 1) : base(2 * kc) + in * pitch(2 * kc));
#pragma unroll
      for (int kk = 0; kk <= kc; ++kk) {
        float f[8];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          f32x4_t ka = {0.f, 0.f, 0.f, 0.f}, qa = ka;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            ka = product(k[kk][hh][ks], k[kc][hc][ks], ka);
            qa = product(k[kk][hh][ks], q[kc][hc][ks], qa);
          }
          const int j = 32 * kk + 8 * g + 4 * hh;
          f32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float dec = __builtin_amdgcn_exp2f((float)(gi - sh.g[j + e]));
            v[e] = kk < kc || j + e < i ? beta * dec * ka[e] : 0.f;
            f[4 * hh + e] = kk < kc || j + e <= i ? a.scale * dec * qa[e] : 0.f;
          }
          if (kk < kc || lower || g < 2) *reinterpret_cast<f32x4_t*>(row + j) = v;
        }
        const Terms<MT> v = split8<MT>(f);
#pragma unroll
        for (int e = 0; e < MT; ++e)
          st16(rec + Rec::M + (e * kTriFrags + tri_frag(kc, hc, kk)) * kFragBytes + 16 * lane, __builtin_bit_cast(uint4, v.v[e]));
      }
    }
  }
  wave_sync();

  // the blocks of the diagonal: column r of block g
  float x[16];
  {
    const int dp = 16 * (g + 1) + 4;                     // pitch(g)
    const float* d = m + 128 * g * (g + 1) + 64 * g + 16 * g;  // base(g), and the block's column
    // (rows are read ahead, in two parts)
    auto part = [&](auto first, auto last) {
      constexpr int F = first, L = last;
      f32x4_t row[L - F][(L + 2) / 4];
#pragma unroll
      for (int i = F; i < L; ++i)
#pragma unroll
        for (int j = 0; j < i; j += 4) row[i - F][j / 4] = ld4(d + i * dp + j);
      hold();
#pragma unroll
      for (int i = F; i < L; ++i) {
        float v = i == r ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) v = fmaf(-row[i - F][j / 4][j % 4], x[j], v);
        x[i] = v;
      }
      hold();
    };
    part(std::integral_constant<int, 0>{}, std::integral_constant<int, 9>{});
    part(std::integral_constant<int, 9>{}, std::integral_constant<int, 16>{});
  }
  wave_sync();
  {
    const int dp = 16 * (g + 1) + 4;
    float* d = m + 128 * g * (g + 1) + 64 * g + 16 * g + r;
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i * dp] = x[i];
  }
  wave_sync();

  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  auto left = [&](int i, int j) { return ld4(m + base(i) + r * pitch(i) + 16 * j + 4 * g); };
  auto right = [&](int i, int j) {
    f32x4_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = m[base(i) + (4 * g + e) * pitch(i) + 16 * j + r];
    return v;
  };
  auto put = [&](int i, int j, const f32x4_t& v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) m[base(i) + (4 * g + e) * pitch(i) + 16 * j + r] = -v[e];
  };
  f32x4_t b10;
  {
    const f32x4_t y0 = mul16(left(1, 0), right(0, 0), zero), y1 = mul16(left(3, 2), right(2, 2), zero);
    const f32x4_t t0 = mul16(left(1, 1), y0, zero), t1 = mul16(left(3, 3), y1, zero);
    b10 = -t0;
    wave_sync();
    put(1, 0, t0);
    put(3, 2, t1);
    wave_sync();
  }
  {
    f32x4_t y[2][2];
    const f32x4_t b00 = right(0, 0), b11 = right(1, 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4_t l0 = left(2 + i, 0), l1 = left(2 + i, 1);
      y[i][0] = mul16(l1, b10, mul16(l0, b00, zero));
      y[i][1] = mul16(l1, b11, zero);
    }
    const f32x4_t a22 = left(2, 2), a32 = left(3, 2), a33 = left(3, 3);
    f32x4_t t[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      t[0][j] = mul16(a22, y[0][j], zero);
      t[1][j] = mul16(a33, y[1][j], mul16(a32, y[0][j], zero));
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) put(2 + i, j, t[i][j]);
    wave_sync();
  }

  // T beta: the operands' rows are 32 kk + 8 (r / 4) + 4 h + r % 4. Right of the
  // diagonal's blocks 0 and 2 are zeros, for which there is no room.
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
      for (int ks = 0; ks <= kk; ++ks) {
        const int in = 8 * (r / 4) + 4 * hh + r % 4;
        const bool lower = in >= 16;
        const int at = (lower ? base(2 * kk + 1) + (in - 16) * pitch(2 * kk + 1) : base(2 * kk) + in * pitch(2 * kk)) + 32 * ks + 8 * g;
        const bool none = ks == kk && !lower && g >= 2;
        const float* from = m + (none ? 0 : at);
        const f32x4_t lo = ld4(from), hi = ld4(from + 4);
        const f32x4_t b0 = ld4(sh.beta + 32 * ks + 8 * g), b1 = ld4(sh.beta + 32 * ks + 8 * g + 4);
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = none ? 0.f : lo[e] * b0[e], f[4 + e] = none ? 0.f : hi[e] * b1[e];
        const Terms<TT> v = split8<TT>(f);
#pragma unroll
        for (int e = 0; e < TT; ++e)
          st16(rec + Rec::T + (e * kTriFrags + tri_frag(kk, hh, ks)) * kFragBytes + 16 * lane, __builtin_bit_cast(uint4, v.v[e]));
      }
}

template <typename TIO, typename TDT>
hipError_t launch_io(const DeltaArgs& a, hipStream_t s) {
  const uint32_t tasks = (uint32_t)(delta_slots(a) * a.H);
  const dim3 grid((unsigned)delta_solve_groups(a));
  auto go = [&](auto whole, auto other) {
    if (a.N % 8 == 0) whole<<<grid, 64 * kWaves, 0, s>>>(a, tasks);
    else other<<<grid, 64 * kWaves, 0, s>>>(a, tasks);
  };
  if (a.N <= 32) go(delta_solve_kernel<TIO, TDT, 32, true>, delta_solve_kernel<TIO, TDT, 32, false>);
  else if (a.N <= 64) go(delta_solve_kernel<TIO, TDT, 64, true>, delta_solve_kernel<TIO, TDT, 64, false>);
  else if (a.N <= 128) go(delta_solve_kernel<TIO, TDT, 128, true>, delta_solve_kernel<TIO, TDT, 128, false>);
  else if constexpr (sizeof(TIO) == 2) go(delta_solve_kernel<TIO, TDT, 256, true>, delta_solve_kernel<TIO, TDT, 256, false>);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

int64_t delta_solve_groups(const DeltaArgs& a) { return (delta_slots(a) * a.H + kWaves - 1) / kWaves; }

hipError_t launch_delta_solve(const DeltaArgs& a, int io, int dt, hipStream_t s) {
  if (io == kF32) return launch_io<float, float>(a, s);
  if (dt == kF32) return launch_io<__hip_bfloat16, float>(a, s);
  return launch_io<__hip_bfloat16, __hip_bfloat16>(a, s);
}

}  // namespace ssd
