// The gated delta rule over prompts, token after token:
//     a = exp(pre(dt) A);  u = beta (x - a S k);  S <- a S + u k^T;  y = scale S q
// batched or packed. The rows of a head's state do not meet, so a team of
// padded N / 4 lanes keeps R of them in registers, four columns to a lane, for
// the whole sequence; S k and S q are reduced side by side (y = scale (a S q +
// u (k q))). The next kAhead tokens' rows are loaded while the present ones are
// worked on. Decays and betas are taken by a lane for a token, 64 tokens at once: by
// every lane for every token they were half of all instructions.
//
// Bound by a wave's instructions and their latency, some 800 cycles a token of one
// sequence of 32 heads, P = N = 128 (0.38 us), 1.6 us a token of eight of them (two waves a SIMD).
// For prompts of a few tokens, which the blocks' two kernels do not repay, for the
// short ones of a pack, and for sizes that have no blocks (P or N below 8; fp32 of N above
// 128, whose three terms of K and Q do not fit the LDS: 16384 tokens of 16 heads of 128 x 256 7.1 ms,
// 8 x 2048 3.7 ms).
#include "delta.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;

template <typename TIO, int R> struct Token {
  Pack<TIO, 4> k, q;
  typename Elem<TIO>::raw x[R];
};

template <typename TIO, typename TDT, int NP, bool VEC, int R>
__global__ __launch_bounds__(kThreads) void delta_walk_kernel(const DeltaArgs a, uint32_t blocks_p) {
  constexpr int LPR = NP / 4;
  constexpr int TEAMS = kThreads / LPR;
  using RX = typename Elem<TIO>::raw;
  using RD = typename Elem<TDT>::raw;
  const int tid = threadIdx.x, sub = tid % LPR, team = tid / LPR;
  const uint32_t sh = blockIdx.x / blocks_p;
  const int pb = (int)(blockIdx.x - sh * blocks_p);
  const int64_t seq = sh / (uint32_t)a.H;
  const int h = (int)(sh - (uint32_t)seq * a.H);
  const int g = h / (a.H / a.G);
  const int n0 = 4 * sub;
  const int nn = a.N - n0 < 0 ? 0 : a.N - n0 > 4 ? 4 : a.N - n0;
  const int nc = nn > 0 ? n0 : 0;

  const int64_t row = a.cu != nullptr ? 0 : seq;  // batch row
  int64_t first = 0, last = a.L;
  if (a.cu != nullptr) first = seq_offset(a.cu, seq, a.L), last = seq_offset(a.cu, seq + 1, a.L);
  if (a.upto > 0 && last - first > a.upto) return;  // (in blocks)
  const TIO* xp = static_cast<const TIO*>(a.x) + row * a.xs.batch;
  const TIO* Bp = static_cast<const TIO*>(a.B) + row * a.bs.batch + (int64_t)g * a.N + nc;
  const TIO* Cp = static_cast<const TIO*>(a.C) + row * a.cs.batch + (int64_t)g * a.N + nc;
  const RD* dp = static_cast<const RD*>(a.dt) + row * a.ds.batch + h;
  const RD* ep = static_cast<const RD*>(a.beta) + row * a.es.batch + h;
  RX* yp = static_cast<RX*>(a.y) + (row * a.L * a.H + h) * a.P;
  const float bias = a.dto.bias != nullptr ? a.dto.bias[h] : 0.f, Ah = a.A[h];

  int p[R];
  bool mine[R];
  float S[R][4];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int pr = (pb * R + k) * TEAMS + team;
    mine[k] = pr < a.P;
    p[k] = mine[k] ? pr : a.P - 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) S[k][i] = 0.f;
    if (a.init != nullptr) {
      const Pack<float, 4> v = load_pack<float, 4, !VEC>(a.init + ((seq * a.H + h) * a.P + p[k]) * a.N + nc, nn);
#pragma unroll
      for (int i = 0; i < 4; ++i) S[k][i] = i < nn ? v.v[i] : 0.f;
    }
  }
  auto load = [&](Token<TIO, R>(&v)[kAhead], int64_t t0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t t = t0 + j < last ? t0 + j : last - 1;
      v[j].k = load_pack<TIO, 4, !VEC>(Bp + t * a.bs.token, nn);
      v[j].q = load_pack<TIO, 4, !VEC>(Cp + t * a.cs.token, nn);
#pragma unroll
      for (int k = 0; k < R; ++k) v[j].x[k] = reinterpret_cast<const RX*>(xp)[t * a.xs.token + (int64_t)h * a.P + p[k]];
    }
  };
  Token<TIO, R> next[kAhead];
  if (first < last) load(next, first);
  // decay and beta of token `from` + lane
  float decays = 0.f, betas = 0.f;
  auto gates = [&](int64_t from) {
    const int64_t t = from + (tid & 63) < last ? from + (tid & 63) : last - 1;
    decays = __builtin_amdgcn_exp2f(delta_log2_decay(Elem<TDT>::f32(dp[t * a.ds.token]), bias, Ah, a.dto));
    betas = delta_beta(Elem<TDT>::f32(ep[t * a.es.token]), a.sigmoid);
  };
  auto of_lane = [](float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); };
  for (int64_t t0 = first; t0 < last; t0 += kAhead) {
    const int at = (int)(t0 - first) & 63;  // (kAhead divides 64)
    if (at == 0) gates(t0);
    Token<TIO, R> cur[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) cur[j] = next[j];
    if (t0 + kAhead < last) load(next, t0 + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (t0 + j >= last) break;
      const float dec = of_lane(decays, at + j), beta = of_lane(betas, at + j);
      float kf[4], qf[4], kq = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kf[i] = i < nn ? Elem<TIO>::f32(cur[j].k.v[i]) : 0.f;
        qf[i] = i < nn ? Elem<TIO>::f32(cur[j].q.v[i]) : 0.f;
        kq = fmaf(kf[i], qf[i], kq);
      }
      kq = team_sum<LPR>(kq);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          S[k][i] *= dec;
          sk = fmaf(S[k][i], kf[i], sk);
          sq = fmaf(S[k][i], qf[i], sq);
        }
        sk = team_sum<LPR>(sk);
        sq = team_sum<LPR>(sq);
        const float u = beta * (Elem<TIO>::f32(cur[j].x[k]) - sk);
#pragma unroll
        for (int i = 0; i < 4; ++i) S[k][i] = fmaf(u, kf[i], S[k][i]);
        if (sub == 0 && mine[k])
          yp[(t0 + j) * a.H * a.P + p[k]] = Elem<TIO>::bits(a.scale * fmaf(u, kq, sq));
      }
    }
  }
  if (a.final_state != nullptr && nn > 0) {
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (mine[k]) store_pack<float, 4, !VEC>(a.final_state + ((seq * a.H + h) * a.P + p[k]) * a.N + n0, S[k], nn);
  }
}

constexpr int kRows = 2;  // rows of the state to a team

// Workgroups to a head's P rows.
uint32_t blocks_of(const DeltaArgs& a) {
  const int rows = kRows * kThreads / (selective_padded_states(a.N) / 4);
  return (a.P + rows - 1) / rows;
}

template <typename TIO, typename TDT, int NP>
hipError_t launch_np(const DeltaArgs& a, hipStream_t s) {
  const uint32_t blocks_p = blocks_of(a);
  const dim3 grid((unsigned)(a.seqs() * a.H * blocks_p));
  if (a.N % 4 == 0) delta_walk_kernel<TIO, TDT, NP, true, kRows><<<grid, kThreads, 0, s>>>(a, blocks_p);
  else delta_walk_kernel<TIO, TDT, NP, false, kRows><<<grid, kThreads, 0, s>>>(a, blocks_p);
  return hipGetLastError();
}

template <typename TIO, typename TDT>
hipError_t launch_io(const DeltaArgs& a, hipStream_t s) {
  switch (selective_padded_states(a.N)) {
    case 16: return launch_np<TIO, TDT, 16>(a, s);
    case 32: return launch_np<TIO, TDT, 32>(a, s);
    case 64: return launch_np<TIO, TDT, 64>(a, s);
    case 128: return launch_np<TIO, TDT, 128>(a, s);
    default: return launch_np<TIO, TDT, 256>(a, s);
  }
}

}  // namespace

bool delta_walk_fits(const DeltaArgs& a) { return grid_fits(a.seqs() * a.H * blocks_of(a), kThreads); }

hipError_t launch_delta_walk(const DeltaArgs& a, int io, int dt, hipStream_t s) {
  if (io == kF32) return launch_io<float, float>(a, s);
  if (dt == kF32) return launch_io<__hip_bfloat16, float>(a, s);
  return launch_io<__hip_bfloat16, __hip_bfloat16>(a, s);
}

}  // namespace ssd
