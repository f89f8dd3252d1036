// The gated delta rule in segments: the states that enter them. A segment makes
// of the state S that enters it S M + B, with M [N, N] what becomes of the unit
// states and B [P, N] of a state of zeros (the rows that the first walk left). So, in
// turn over a sequence's segments, S <- S M + B.
//
// A workgroup keeps 16 rows of a head's S in LDS and goes over the segments, a
// wave a quarter of the columns; fp32 matrix instructions, since nothing may be
// lost that the walks keep. Bound by the latency of M and B (64 KB and more a
// segment, from the caches), so the next segment's are on their way, all at
// once, while a segment is joined: 8 segments of 32 heads, P = N = 128 32 us, where loads
// at their use took 195.
#include "delta_blocks.h"

namespace ssd {
namespace {

constexpr int kThreads = 256, kRows = 16;

template <int NP>
__global__ __launch_bounds__(kThreads) void delta_join_kernel(const DeltaArgs a, uint32_t blocks_p) {
  constexpr int PITCH = NP + 4;
  constexpr int CT = (NP / 16 + 3) / 4;  // 16-column tiles of a wave
  __shared__ __align__(16) float s[kRows * PITCH];
  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, g = lane / 16, r = lane % 16;
  const uint32_t sh = blockIdx.x / blocks_p;
  const int pb = (int)(blockIdx.x - sh * blocks_p);
  const int64_t seq = sh / (uint32_t)a.H;
  const int h = (int)(sh - (uint32_t)seq * a.H);
  const int p0 = pb * kRows;
  const int64_t base = delta_first_slot(a, seq, a.seg);
  const int64_t first = a.cu != nullptr ? seq_offset(a.cu, seq, a.L) : 0, last = a.cu != nullptr ? seq_offset(a.cu, seq + 1, a.L) : a.L;
  const int64_t parts = last - first > a.seg ? (last - first + a.seg - 1) / a.seg : 1;

  for (int q = tid; q < kRows * NP; q += kThreads) {
    const int p = q / NP, n = q % NP;
    const bool in = p0 + p < a.P && n < a.N;
    const float v = in && a.init != nullptr ? a.init[((seq * a.H + h) * a.P + p0 + p) * a.N + n] : 0.f;
    s[p * PITCH + n] = v;
    if (in) a.enter[((base * a.H + h) * a.P + p0 + p) * a.N + n] = v;
  }
  // operand of columns 16 (wave + 4 c) + r, rows 16 k + 4 g + e; and B
  constexpr int KT = NP / 16, KS = KT < 8 ? KT : 8;  // rows' tiles, of them at a time
  struct Next {
    float m[KS][CT][4], b[CT][4];
  } next;
  auto load = [&](int64_t j, int k0) {
    const float* B = a.ends + ((base + j) * a.H + h) * (int64_t)(a.P + a.N) * a.N;
    const float* M = B + (int64_t)a.P * a.N;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int n = 16 * (wave + 4 * c) + r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int m = 16 * (k0 + k) + 4 * g + e;
          next.m[k][c][e] = m < a.N && n < a.N ? M[(int64_t)m * a.N + n] : 0.f;
        }
        const int p = p0 + 4 * g + e;
        if (k0 == 0) next.b[c][e] = p < a.P && n < a.N ? B[(int64_t)p * a.N + n] : 0.f;
      }
    }
  };
  if (parts > 1) load(0, 0);
  for (int64_t j = 0; j + 1 < parts; ++j) {
    __syncthreads();
    f32x4_t d[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) d[c] = f32x4_t{next.b[c][0], next.b[c][1], next.b[c][2], next.b[c][3]};
#pragma unroll
    for (int k0 = 0; k0 < KT; k0 += KS) {
      const Next now = next;
      if (k0 + KS < KT) load(j, k0 + KS);
      else if (j + 2 < parts) load(j + 1, 0);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(s + r * PITCH + 16 * (k0 + k) + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < CT; ++c) d[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], now.m[k][c][e], d[c], 0, 0, 0);
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int n = 16 * (wave + 4 * c) + r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = 4 * g + e;
        if (n >= NP) continue;
        s[p * PITCH + n] = d[c][e];
        if (p0 + p < a.P && n < a.N) a.enter[(((base + j + 1) * a.H + h) * a.P + p0 + p) * a.N + n] = d[c][e];
      }
    }
  }
}

}  // namespace

int64_t delta_join_groups(const DeltaArgs& a) { return a.seqs() * a.H * ((a.P + kRows - 1) / kRows); }

hipError_t launch_delta_join(const DeltaArgs& a, hipStream_t s) {
  const uint32_t blocks_p = (a.P + kRows - 1) / kRows;
  const dim3 grid((unsigned)delta_join_groups(a));
  if (a.N <= 32) delta_join_kernel<32><<<grid, kThreads, 0, s>>>(a, blocks_p);
  else if (a.N <= 64) delta_join_kernel<64><<<grid, kThreads, 0, s>>>(a, blocks_p);
  else if (a.N <= 128) delta_join_kernel<128><<<grid, kThreads, 0, s>>>(a, blocks_p);
  else delta_join_kernel<256><<<grid, kThreads, 0, s>>>(a, blocks_p);
  return hipGetLastError();
}

}  // namespace ssd
