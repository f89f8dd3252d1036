// Group norm over the channels of each token (channels last), with the gate
// of the layer around the scan. For every row and group of S = C / G channels:
//     v = x silu(z) where the gate comes first, else x
//     mu = mean(v) if centred, else 0;   var = mean((v - mu)^2)
//     o = (v - mu) / sqrt(var + eps) * w + bias
//     o = o silu(z) where the gate comes last;  or silu(o)
//
// One pass over memory: a team of lanes holds a group's channels in registers
// (M packs of V consecutive ones to a lane), so the mean and the squares
// around it are both taken from registers, in fp32. A team keeps its group
// and walks over rows, with its weights in registers and the next row's loads
// issued before the current row is reduced (not in the 1024-lane teams of the
// largest groups: 128 registers a lane hold the row and nothing beside it).
// Teams up to a wave reduce by lane exchanges; larger groups take a
// workgroup, which exchanges its waves' sums through LDS.
//
// Bound by memory: 16384 x 4096 bf16 with gate 67 us, 6.0 TB/s; 1001 x 8192 fp32 in
// 128 groups 18.2 us, 5.4 TB/s. Groups of 4096 channels: a workgroup of 256 lanes
// 82 us (weights still loaded one by one), 128 lanes 96, one wave 151.
#include "selective.h"

namespace ssd {
namespace {

template <typename TIO, int V, int M, bool WHOLE, int T, bool Z>
__global__ __launch_bounds__(T > 64 ? T : 256) void group_norm_kernel(const GroupNormArgs a) {
  constexpr int THREADS = T > 64 ? T : 256;
  constexpr int TEAMS = THREADS / T;  // teams per workgroup
  constexpr int WAVES = THREADS / 64;
  __shared__ float part[2][T > 64 ? WAVES : 1];
  const int S = a.C / a.G;
  const int lane = threadIdx.x % T;
  const int64_t team = (int64_t)blockIdx.x * TEAMS + threadIdx.x / T;
  const int64_t nteams = (int64_t)gridDim.x * TEAMS;  // a multiple of G (launch)
  const int g = (int)(team % a.G);
  const int64_t step = nteams / a.G;
  const int64_t rows = a.batch * a.rows;
  const float inv = 1.f / (float)S;
  int par = 0;

  // This lane's packs: first channel, and which of its elements count. WHOLE:
  // groups of V channels and more; the last pack of a group ends with it, and
  // where it overlaps the one before (skip > 0) both write the same values.
  // Otherwise the one pack of a small group, of which nn elements are there.
  int at[M], nn[M], skip[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int c = (m * T + lane) * V, from = WHOLE && c + V > S ? S - V : c;
    nn[m] = c >= S ? 0 : S - from < V ? S - from : V;
    skip[m] = c - from;
    at[m] = g * S + (nn[m] > 0 ? from : 0);
  }
  auto counts = [&](int m, int v) { return v < nn[m] && v >= skip[m]; };
  constexpr bool HOLD = T < 1024;
  // weights and offsets of pack m (any valid address stands in for none)
  auto weights = [&](int m, float (&w)[V], float (&bias)[V]) {
    const Pack<float, V> wp = load_pack<float, V, !WHOLE>(a.w != nullptr ? a.w + at[m] : a.bias + at[m], nn[m]);
    const Pack<float, V> bp = load_pack<float, V, !WHOLE>(a.bias != nullptr ? a.bias + at[m] : a.w + at[m], nn[m]);
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = a.w != nullptr ? wp.v[v] : 1.f, bias[v] = a.bias != nullptr ? bp.v[v] : 0.f;
  };
  const bool affine = a.w != nullptr || a.bias != nullptr;
  float w[HOLD ? M : 1][V], bias[HOLD ? M : 1][V];
  if constexpr (HOLD) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int v = 0; v < V; ++v) w[m][v] = 1.f, bias[m][v] = 0.f;
      if (affine) weights(m, w[m], bias[m]);
    }
  }

  Pack<TIO, V> xn[M], zn[Z ? M : 1];
  auto fetch = [&](int64_t r) {
    const int64_t b = r / a.rows, t = r - b * a.rows;
    const TIO* xp = static_cast<const TIO*>(a.x) + b * a.xs.batch + t * a.xs.token;
    const TIO* zp = static_cast<const TIO*>(a.z) + b * a.zs.batch + t * a.zs.token;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (WHOLE && a.stream) {
        xn[m] = load_stream<TIO, V>(xp + at[m]);
        if constexpr (Z) zn[m] = load_stream<TIO, V>(zp + at[m]);
      } else {
        xn[m] = load_pack<TIO, V, !WHOLE>(xp + at[m], nn[m]);
        if constexpr (Z) zn[m] = load_pack<TIO, V, !WHOLE>(zp + at[m], nn[m]);
      }
    }
  };
  auto team_sum = [&](float v) {
#pragma unroll
    for (int off = (T > 64 ? 64 : T) / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    if constexpr (T > 64) {
      // two buffers: the next sum's writes meet no reader of this one
      par ^= 1;
      if ((threadIdx.x & 63) == 0) part[par][threadIdx.x / 64] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) v += part[par][i];
    }
    return v;
  };

  int64_t r = team / a.G;
  // (all lanes of a workgroup-wide team share r, so its barriers are met by all)
  if (r >= rows) return;
  fetch(r);
  for (; r < rows; r += step) {
    float x[M][V];
    Pack<TIO, V> zc[Z ? M : 1];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if constexpr (Z) zc[m] = zn[m];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[m][v] = Elem<TIO>::f32(xn[m].v[v]);
        if constexpr (Z) {
          if (a.gate_first) x[m][v] *= silu_f32(Elem<TIO>::f32(zc[m].v[v]));
        }
      }
    }
    if (HOLD && r + step < rows) fetch(r + step);
    float mu = 0.f;
    if (a.center) {
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (counts(m, v)) mu += x[m][v];
      mu = team_sum(mu) * inv;
    }
    float sq = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[m][v] -= mu;
        if (counts(m, v)) sq = fmaf(x[m][v], x[m][v], sq);
      }
    const float var = team_sum(sq) * inv + a.eps;
    // one Newton step on the hardware's reciprocal root (1 ulp); it takes a
    // subnormal for 0, so small ones go in times 2^64
    const bool small = var < 0x1p-100f;
    const float vs = small ? var * 0x1p64f : var;
    float rs = __builtin_amdgcn_rsqf(vs);
    rs = vs > 0.f && vs < 1e38f ? rs * fmaf(-0.5f * vs * rs, rs, 1.5f) : rs;
    if (small) rs *= 0x1p32f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float o[V], wv[V], ov[V];
      if constexpr (!HOLD) {
#pragma unroll
        for (int v = 0; v < V; ++v) wv[v] = 1.f, ov[v] = 0.f;
        if (affine) weights(m, wv, ov);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (HOLD) o[v] = fmaf(x[m][v] * rs, w[m][v], bias[m][v]);
        else o[v] = fmaf(x[m][v] * rs, wv[v], ov[v]);
        if constexpr (Z) {
          if (!a.gate_first) o[v] *= silu_f32(Elem<TIO>::f32(zc[m].v[v]));
        } else {
          if (a.silu) o[v] = silu_f32(o[v]);
        }
      }
      if (nn[m] > 0) store_pack<TIO, V, !WHOLE>(static_cast<TIO*>(a.out) + r * a.C + at[m], o, nn[m]);
    }
    if (!HOLD && r + step < rows) fetch(r + step);
  }
}

template <typename TIO, bool Z>
hipError_t launch_z(const GroupNormArgs& a, hipStream_t s) {
  constexpr int V = 16 / sizeof(TIO);
  const int64_t S = a.C / a.G, packs = (S + V - 1) / V, rows = a.batch * a.rows;
  auto go = [&](auto kern, int team) {
    const int threads = team > 64 ? team : 256, per = threads / team;
    // teams for all rows and groups, but no more than fill the card, and a
    // whole number of rows' worth: a team keeps its group
    int64_t want = rows * a.G;
    const int64_t full = (int64_t)device_cu_count() * (2048 / team);
    int64_t teams = want < full ? want : full;
    // smallest number of workgroups that is a multiple of G / gcd(G, per)
    int64_t x = a.G, y = per;
    while (y != 0) {
      const int64_t t = x % y;
      x = y;
      y = t;
    }
    const int64_t unit = a.G / x;
    int64_t blocks = ((teams + per - 1) / per + unit - 1) / unit * unit;
    kern<<<dim3((unsigned)blocks), threads, 0, s>>>(a);
    return hipGetLastError();
  };
  if (S < V) return go(group_norm_kernel<TIO, V, 1, false, 8, Z>, 8);
  if (packs <= 8) return go(group_norm_kernel<TIO, V, 1, true, 8, Z>, 8);
  if (packs <= 16) return go(group_norm_kernel<TIO, V, 1, true, 16, Z>, 16);
  if (packs <= 32) return go(group_norm_kernel<TIO, V, 1, true, 32, Z>, 32);
  if (packs <= 64) return go(group_norm_kernel<TIO, V, 1, true, 64, Z>, 64);
  if (packs <= 128) return go(group_norm_kernel<TIO, V, 2, true, 64, Z>, 64);
  if (packs <= 256) return go(group_norm_kernel<TIO, V, 1, true, 256, Z>, 256);
  if (packs <= 512) return go(group_norm_kernel<TIO, V, 2, true, 256, Z>, 256);
  if (packs <= 1024) return go(group_norm_kernel<TIO, V, 4, true, 256, Z>, 256);
  constexpr int M = (int)(kGroupNormMaxGroup / 1024 / V);
  return go(group_norm_kernel<TIO, V, M, true, 1024, Z>, 1024);
}

template <typename TIO>
hipError_t launch_io(const GroupNormArgs& args, hipStream_t s) {
  GroupNormArgs a = args;
  // Inputs and output beyond half the memory-side cache: the inputs are read past
  // it (non-temporal), which leaves it to the output, 192 MB 40 -> 35 us, 384 MB
  // 79 -> 67, 768 MB 157 -> 152. Smaller ones are better off in it (96 MB 20.8 us,
  // past it 21.6; 19.4 and 21.0 where the inputs lie there already).
  a.stream = a.batch * a.rows * a.C * (int64_t)sizeof(TIO) * (a.z != nullptr ? 3 : 2) > kMemorySideCache / 2;
  return a.z != nullptr ? launch_z<TIO, true>(a, s) : launch_z<TIO, false>(a, s);
}

}  // namespace

hipError_t launch_group_norm(const GroupNormArgs& a, int io, hipStream_t s) {
  return io == kBF16 ? launch_io<__hip_bfloat16>(a, s) : launch_io<float>(a, s);
}

}  // namespace ssd
