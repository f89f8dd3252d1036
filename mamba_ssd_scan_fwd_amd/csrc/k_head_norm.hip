// Norm of each head of queries and keys, and the rotation of its first R
// channels by the token's position:
//     v = x / sqrt(mean(x^2) + eps) w   (or sum in place of mean)
//     (v_a, v_b) <- (v_a cos - v_b sin, v_b cos + v_a sin),  angle = pos * freq[i]
// (a, b) = (i, i + R / 2) or (2 i, 2 i + 1).
//
// One pass over memory: a team of T lanes holds a head in registers, M packs of
// V consecutive channels to a lane, and sums its squares by DPP. A
// wave takes one token: its 64 lanes compute one angle each (product and
// reduction to a turn in 64 bits, so that positions in the millions keep the
// angle's digits; sine and cosine of the reduced angle in fp32), each lane takes
// those of its channels into registers, and all heads of the token are turned by them. Queries
// and keys are one launch.
//
// The other half of a pair lies in the same lane (neighbouring channels), in lane
// ^ T / 2 where all channels of a head that fills the team are turned (DPP or one
// exchange of rows), or anywhere: through LDS, where the wave's lanes need no
// barrier.
#include "delta.h"

namespace ssd {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

enum Exchange { kNone, kSameLane, kHalfTeam, kAnywhere };

// The value of lane ^ T / 2.
template <int T> __device__ __forceinline__ float half_team(float v) {
  if constexpr (T == 8) return dpp_f32<0x141>(dpp_f32<0x1B>(v));  // mirrored in 4, then in 8
  if constexpr (T == 16) return dpp_f32<0x128>(v);                // turned by 8 in 16
  const uint32_t u = __float_as_uint(v);
  if constexpr (T == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __uint_as_float(threadIdx.x & 16 ? r[0] : r[1]);
  }
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(threadIdx.x & 32 ? r[0] : r[1]);
}

template <typename TIO, int T, int M, bool WHOLE, Exchange X>
__global__ __launch_bounds__(kThreads) void head_norm_kernel(const HeadNormArgs a) {
  constexpr int V = 16 / sizeof(TIO), TEAMS = 64 / T, DP = T * M * V;  // DP: channels that a team has room for
  __shared__ float2 turns[X != kNone ? kWaves : 1][X != kNone ? kHeadNormMaxDim / 2 : 1];  // cos, sin of this wave's token
  __shared__ __align__(16) float line_[X == kAnywhere ? kWaves : 1][X == kAnywhere ? TEAMS : 1][X == kAnywhere ? DP : 1];
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
  float w[2][M][V];
  const bool weighted = a.w[0] != nullptr || a.w[1] != nullptr;
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int m = 0; m < M; ++m)
      {
#pragma unroll
        for (int i = 0; i < V; ++i) w[x][m][i] = 1.f;
        if (!weighted) continue;
        const Pack<float, V> p = load_pack<float, V, !WHOLE>((a.w[x] != nullptr ? a.w[x] : a.w[1 - x]) + at[m], nn[m]);
#pragma unroll
        for (int i = 0; i < V; ++i) w[x][m][i] = a.w[x] != nullptr ? p.v[i] : 1.f;
      }

  const int64_t tasks = a.batch * a.rows * parts;
  for (int64_t task = (int64_t)blockIdx.x * kWaves + wave; task < tasks; task += (int64_t)gridDim.x * kWaves) {
    const int64_t token = parts == 1 ? task : task / parts;
    const int h0 = (int)(task - token * parts) * a.per;
    const int h1 = h0 + a.per < heads ? h0 + a.per : heads;
    const int64_t b = a.batch == 1 ? 0 : token / a.rows, t = token - b * a.rows;
    auto load = [&](int hb, Pack<TIO, V>(&x)[M]) {
      const int hh = hb + team < h1 ? hb + team : h1 - 1;
      const int which = hh >= a.heads[0];
      const TIO* xp = static_cast<const TIO*>(a.in[which]) + b * a.st[which].batch + t * a.st[which].token +
                      (int64_t)(which ? hh - a.heads[0] : hh) * a.D;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        if (WHOLE && a.stream) x[m] = load_stream<TIO, V>(xp + at[m]);
        else x[m] = load_pack<TIO, V, !WHOLE>(xp + at[m], nn[m]);
      }
    };
    Pack<TIO, V> next[M];
    load(h0, next);
    // what this lane's channels are multiplied with, and the others of their pairs
    float cs[X != kNone ? M : 1][V], sn[X != kNone ? M : 1][V];
    if constexpr (X != kNone) {
      const double pos = (double)a.pos[token];
      for (int i = lane; i < half; i += 64) {
        const double rev = pos * ((double)a.freq[i] * 0.15915494309189533577);  // turns
        float s, c;
        sincospif(2.f * (float)(rev - rint(rev)), &s, &c);
        turns[wave][i] = make_float2(c, s);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = at[m] + i;
          const bool second = a.pairs ? c & 1 : c >= half;
          const bool turned = i < nn[m] && c < a.R;
          const float2 f = turns[wave][!turned ? 0 : a.pairs ? c / 2 : second ? c - half : c];
          cs[m][i] = f.x;
          sn[m][i] = second ? f.y : -f.y;
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    for (int hb = h0; hb < h1; hb += TEAMS) {
      const bool live = hb + team < h1;
      const int hh = live ? hb + team : h1 - 1;
      const int which = hh >= a.heads[0];
      Pack<TIO, V> x[M];
#pragma unroll
      for (int m = 0; m < M; ++m) x[m] = next[m];
      if (hb + TEAMS < h1) load(hb + TEAMS, next);
      float v[M][V], sq = 0.f;
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[m][i] = Elem<TIO>::f32(x[m].v[i]);
          if (i < nn[m] && i >= skip[m]) sq = fmaf(v[m][i], v[m][i], sq);
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
        for (int i = 0; i < V; ++i) v[m][i] = v[m][i] * rs * (which ? w[1][m][i] : w[0][m][i]);
      if constexpr (X != kNone) {
        float other[M][V];
        if constexpr (X == kSameLane) {
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < V; ++i) other[m][i] = v[m][i ^ 1];
        } else if constexpr (X == kHalfTeam) {
#pragma unroll
          for (int i = 0; i < V; ++i) other[0][i] = half_team<T>(v[0][i]);
        } else {
          float* line = line_[wave][team];
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
              const bool turned = i < nn[m] && c < a.R;
              other[m][i] = line[!turned ? 0 : a.pairs ? c ^ 1 : c >= half ? c - half : c + half];
            }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float turned = fmaf(v[m][i], cs[m][i], other[m][i] * sn[m][i]);
            // (half a team: every channel is turned)
            v[m][i] = X == kHalfTeam || at[m] + i < a.R ? turned : v[m][i];
          }
      }
      TIO* op = static_cast<TIO*>(a.out[which]) + (token * a.heads[which] + (which ? hh - a.heads[0] : hh)) * a.D;
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (live && nn[m] > 0) store_pack<TIO, V, !WHOLE>(op + at[m], v[m], nn[m]);
    }
  }
}

template <typename TIO>
hipError_t launch_io(const HeadNormArgs& args, hipStream_t s) {
  HeadNormArgs a = args;
  // as in the group norm: inputs and outputs beyond half the memory-side cache are
  // read past it, which leaves it to the outputs (335 MB 78 -> 72 us)
  a.stream = a.batch * a.rows * (a.heads[0] + a.heads[1]) * a.D * (int64_t)sizeof(TIO) * 2 > kMemorySideCache / 2;
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
  auto team = [&](auto lanes, auto packs_each, auto whole) {
    constexpr int T = decltype(lanes)::value, M = decltype(packs_each)::value;
    constexpr bool W = decltype(whole)::value;
    if (a.R == 0) return go(head_norm_kernel<TIO, T, M, W, kNone>, T);
    if constexpr (W) {
      if (a.pairs && a.D % 2 == 0) return go(head_norm_kernel<TIO, T, M, W, kSameLane>, T);
      if constexpr (M == 1)
        if (!a.pairs && a.R == a.D && a.D == T * V) return go(head_norm_kernel<TIO, T, M, W, kHalfTeam>, T);
    }
    return go(head_norm_kernel<TIO, T, M, W, kAnywhere>, T);
  };
  using std::integral_constant;
  constexpr integral_constant<int, 1> one{};
  if (a.D < V) return team(integral_constant<int, 8>{}, one, std::false_type{});
  if (packs <= 8) return team(integral_constant<int, 8>{}, one, std::true_type{});
  if (packs <= 16) return team(integral_constant<int, 16>{}, one, std::true_type{});
  if (packs <= 32) return team(integral_constant<int, 32>{}, one, std::true_type{});
  if (packs <= 64) return team(integral_constant<int, 64>{}, one, std::true_type{});
  if constexpr (V == 4) return team(integral_constant<int, 64>{}, integral_constant<int, 2>{}, std::true_type{});
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_head_norm(const HeadNormArgs& a, int io, hipStream_t s) {
  return io == kBF16 ? launch_io<__hip_bfloat16>(a, s) : launch_io<float>(a, s);
}

}  // namespace ssd
