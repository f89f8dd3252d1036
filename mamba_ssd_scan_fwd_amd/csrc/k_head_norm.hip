// Norm of each head of queries and keys, and the rotation of its first R
// channels by the token's position:
//     v = x / sqrt(mean(x^2) + eps) w   (or sum in place of mean)
//     (v_a, v_b) <- (v_a cos - v_b sin, v_b cos + v_a sin),  angle = pos * freq[i]
// (a, b) = (i, i + R / 2) or (2 i, 2 i + 1).
//
// One pass over memory: a team of T lanes holds a head in registers, M packs of
// V consecutive channels to a lane, sums its squares by DPP, and exchanges the
// halves of the pairs through LDS, where the wave's lanes need no barrier. A
// wave takes one token: its 64 lanes compute one angle each (product and
// reduction to a turn in 64 bits, so that positions in the millions keep the
// angle's digits; sine and cosine of the reduced angle in fp32), and all heads of the token use
// them. Queries and keys are one launch.
#include "delta.h"

namespace ssd {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

template <typename TIO, int T, int M, bool WHOLE>
__global__ __launch_bounds__(kThreads) void head_norm_kernel(const HeadNormArgs a) {
  constexpr int V = 16 / sizeof(TIO), TEAMS = 64 / T, DP = T * M * V;  // DP: channels that a team has room for
  __shared__ float2 turns[kWaves][kHeadNormMaxDim / 2];  // cos, sin of this wave's token
  __shared__ __align__(16) float swap[kWaves][TEAMS][DP];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, team = lane / T, sub = lane % T;
  const int heads = a.heads[0] + a.heads[1];
  const int parts = (heads + a.per - 1) / a.per;  // waves to a token
  const int half = a.R / 2;
  const float inv = a.l2 ? 1.f : 1.f / (float)a.D;

  // This lane's packs: first channel, and which of its elements count. WHOLE:
  // heads of V channels and more; the last pack of a head ends with it, and where
  // it overlaps the one before (skip > 0) both write the same values. Otherwise
  // the one pack of a small head, of which nn elements are there.
  int at[M], nn[M], skip[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int c = (m * T + sub) * V, from = WHOLE && c + V > a.D ? a.D - V : c;
    nn[m] = c >= a.D ? 0 : a.D - from < V ? a.D - from : V;
    skip[m] = c - from;
    at[m] = nn[m] > 0 ? from : 0;
  }

  const int64_t tasks = a.batch * a.rows * parts;
  for (int64_t task = (int64_t)blockIdx.x * kWaves + wave; task < tasks; task += (int64_t)gridDim.x * kWaves) {
    const int64_t token = task / parts;
    const int h0 = (int)(task % parts) * a.per;
    const int h1 = h0 + a.per < heads ? h0 + a.per : heads;
    const int64_t b = token / a.rows, t = token - b * a.rows;
    if (half > 0) {
      const double pos = (double)a.pos[token];
      for (int i = lane; i < half; i += 64) {
        const double rev = pos * ((double)a.freq[i] * 0.15915494309189533577);  // turns
        float sn, cs;
        sincospif(2.f * (float)(rev - rint(rev)), &sn, &cs);
        turns[wave][i] = make_float2(cs, sn);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    for (int hb = h0; hb < h1; hb += TEAMS) {
      const bool live = hb + team < h1;
      const int hh = live ? hb + team : h1 - 1;
      const int which = hh >= a.heads[0];
      const int h = which ? hh - a.heads[0] : hh;
      const TIO* xp = static_cast<const TIO*>(a.in[which]) + b * a.st[which].batch + t * a.st[which].token + (int64_t)h * a.D;
      const float* w = a.w[which];
      float v[M][V], sq = 0.f;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const Pack<TIO, V> x = load_pack<TIO, V, !WHOLE>(xp + at[m], nn[m]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[m][i] = Elem<TIO>::f32(x.v[i]);
          if (i < nn[m] && i >= skip[m]) sq = fmaf(v[m][i], v[m][i], sq);
        }
      }
      const float var = team_sum<T>(sq) * inv + a.eps;
      // one Newton step on the hardware's reciprocal root (1 ulp); it takes a
      // subnormal for 0, so small ones go in times 2^64
      const bool small = var < 0x1p-100f;
      const float vs = small ? var * 0x1p64f : var;
      float rs = __builtin_amdgcn_rsqf(vs);
      rs = vs > 0.f && vs < 1e38f ? rs * fmaf(-0.5f * vs * rs, rs, 1.5f) : rs;
      if (small) rs *= 0x1p32f;
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[m][i] *= rs;
          if (w != nullptr) v[m][i] *= w[at[m] + (i < nn[m] ? i : 0)];
        }
      if (half > 0) {
        float* line = swap[wave][team];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i < nn[m]) line[at[m] + i] = v[m][i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int c = at[m] + i;
            if (i < nn[m] && c < a.R) {
              const bool second = a.pairs ? c & 1 : c >= half;
              const float2 cs = turns[wave][a.pairs ? c / 2 : second ? c - half : c];
              const float other = line[a.pairs ? c ^ 1 : second ? c - half : c + half];
              v[m][i] = second ? fmaf(v[m][i], cs.x, other * cs.y) : fmaf(v[m][i], cs.x, -other * cs.y);
            }
          }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      TIO* op = static_cast<TIO*>(a.out[which]) + (token * a.heads[which] + h) * a.D;
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (live && nn[m] > 0) store_pack<TIO, V, !WHOLE>(op + at[m], v[m], nn[m]);
    }
  }
}

template <typename TIO>
hipError_t launch_io(const HeadNormArgs& args, hipStream_t s) {
  HeadNormArgs a = args;
  constexpr int V = 16 / sizeof(TIO);
  const int packs = (a.D + V - 1) / V, heads = a.heads[0] + a.heads[1];
  const int64_t tokens = a.batch * a.rows;
  auto go = [&](auto kern, int team) {
    // all heads of a token to a wave where the tokens alone fill the card,
    // otherwise fewer, down to one head to a team
    const int teams = 64 / team;
    const int64_t full = (int64_t)device_cu_count() * 16;
    int64_t parts = (full + tokens - 1) / tokens;
    int64_t per = (heads + parts - 1) / parts;
    per = (per + teams - 1) / teams * teams;
    a.per = (int)per;
    const int64_t tasks = tokens * ((heads + per - 1) / per);
    int64_t blocks = (tasks + kWaves - 1) / kWaves;
    if (blocks > full) blocks = full;
    kern<<<dim3((unsigned)blocks), kThreads, 0, s>>>(a);
    return hipGetLastError();
  };
  if (a.D < V) return go(head_norm_kernel<TIO, 8, 1, false>, 8);
  if (packs <= 8) return go(head_norm_kernel<TIO, 8, 1, true>, 8);
  if (packs <= 16) return go(head_norm_kernel<TIO, 16, 1, true>, 16);
  if (packs <= 32) return go(head_norm_kernel<TIO, 32, 1, true>, 32);
  if (packs <= 64) return go(head_norm_kernel<TIO, 64, 1, true>, 64);
  if constexpr (V == 4) return go(head_norm_kernel<TIO, 64, 2, true>, 64);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_head_norm(const HeadNormArgs& a, int io, hipStream_t s) {
  return io == kBF16 ? launch_io<__hip_bfloat16>(a, s) : launch_io<float>(a, s);
}

}  // namespace ssd
