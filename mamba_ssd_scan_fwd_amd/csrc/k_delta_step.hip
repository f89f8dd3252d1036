// The gated delta rule at one token: a step of every sequence of a batch, the
// states kept in a pool of slots between calls.
//     a = exp(pre(dt) A);  u = beta (x - a S k);  S <- a S + u k^T;  y = scale S q
// with y = scale (a S q + u (k q)), so that the sums over the state's columns,
// S k and S q, are both taken of the state as it was read, side by side.
//
// Streaming: the fp32 states are read once and written once, which is nearly
// all the traffic. Four consecutive columns to a lane, padded N / 4 lanes to a
// row of the state, which reduce by DPP; R rows to a team, all of whose loads
// are issued before the first is used, so that k and q are read once for R
// rows. Measured: 256 rows of 32 heads, P = N = 128 (1.08 GB) 182 us, 5.9 TB/s, what the memory
// gives for updates in place; 37 rows of 32 heads, P = N = 64 8.5 us; one row 3.7 us, a launch's
// and a round of dependent reads' (slot, state).
//
// A row whose slot is negative or behind the pool is padding: nothing is
// read or written for it. Where a slot is named twice the first row has it
// and the later ones are treated as padding, so no two rows write one state.
#include <type_traits>

#include "delta.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

template <typename TIO, typename TDT, int NP, bool VEC, int R>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(const DeltaStepArgs a, uint32_t blocks_p) {
  constexpr int LPR = NP / 4;             // lanes per row of the state
  constexpr int TEAMS = kThreads / LPR;
  const int tid = threadIdx.x, sub = tid % LPR, team = tid / LPR;
  const uint32_t rh = blockIdx.x / blocks_p;
  const int pb = (int)(blockIdx.x - rh * blocks_p);
  const int64_t r = rh / (uint32_t)a.H;
  const int h = (int)(rh - (uint32_t)r * a.H);
  const int g = h / (a.H / a.G);
  const int n0 = 4 * sub;
  const int nn = a.N - n0 < 0 ? 0 : a.N - n0 > 4 ? 4 : a.N - n0;  // columns this lane holds
  const int nc = nn > 0 ? n0 : 0;                                 // an address inside the row for the others
  using RX = typename Elem<TIO>::raw;
  using RD = typename Elem<TDT>::raw;

  int64_t slot = a.slots != nullptr ? a.slots[r] : r;
  if (slot < 0 || slot >= a.nslots) slot = -1;
  const int64_t from = slot < 0 ? 0 : slot;
  int p[R];
  bool mine[R];
  Pack<float, 4> S[R];
  RX xv[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int row = (pb * R + k) * TEAMS + team;
    mine[k] = row < a.P;
    p[k] = mine[k] ? row : a.P - 1;
    const float* sp = a.state + ((from * a.H + h) * a.P + p[k]) * a.N + nc;
    if (VEC && a.stream) S[k] = load_stream<float, 4>(sp);
    else S[k] = load_pack<float, 4, !VEC>(sp, nn);
    xv[k] = reinterpret_cast<const RX*>(a.x)[r * a.xs + (int64_t)h * a.P + p[k]];
  }
  const Pack<TIO, 4> kp = load_pack<TIO, 4, !VEC>(static_cast<const TIO*>(a.B) + r * a.bs + (int64_t)g * a.N + nc, nn);
  const Pack<TIO, 4> qp = load_pack<TIO, 4, !VEC>(static_cast<const TIO*>(a.C) + r * a.cs + (int64_t)g * a.N + nc, nn);
  const float dt = Elem<TDT>::f32(reinterpret_cast<const RD*>(a.dt)[r * a.ds + h]);
  const float be = Elem<TDT>::f32(reinterpret_cast<const RD*>(a.beta)[r * a.es + h]);
  const float bias = a.dto.bias != nullptr ? a.dto.bias[h] : 0.f;
  const float Ah = a.A[h];
  if (a.slots != nullptr && (repeated_slots<1, kThreads>(a.slots, r, a.batch) & 1)) slot = -1;

  const float dec = __builtin_amdgcn_exp2f(delta_log2_decay(dt, bias, Ah, a.dto));
  const float beta = delta_beta(be, a.sigmoid);
  float kf[4], qf[4], kq = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    kf[i] = i < nn ? Elem<TIO>::f32(kp.v[i]) : 0.f;
    qf[i] = i < nn ? Elem<TIO>::f32(qp.v[i]) : 0.f;
    kq = fmaf(kf[i], qf[i], kq);
  }
  kq = team_sum<LPR>(kq);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    float sk = 0.f, sq = 0.f, s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = i < nn ? dec * S[k].v[i] : 0.f;
      sk = fmaf(s[i], kf[i], sk);
      sq = fmaf(s[i], qf[i], sq);
    }
    sk = team_sum<LPR>(sk);
    sq = team_sum<LPR>(sq);
    const float u = beta * (Elem<TIO>::f32(xv[k]) - sk);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = fmaf(u, kf[i], s[i]);
    if (slot >= 0 && mine[k]) {
      float* sp = a.state + ((slot * a.H + h) * a.P + p[k]) * a.N + n0;
      if (nn > 0) {
        if (VEC && a.stream) store_stream<float, 4>(sp, s);
        else store_pack<float, 4, !VEC>(sp, s, nn);
      }
      if (sub == 0)
        reinterpret_cast<RX*>(a.y)[(r * a.H + h) * a.P + p[k]] = Elem<TIO>::bits(a.scale * fmaf(u, kq, sq));
    }
  }
}

template <typename TIO, typename TDT, int NP>
hipError_t launch_np(const DeltaStepArgs& args, hipStream_t s) {
  DeltaStepArgs a = args;
  // past the caches as in the selective step: a layer's states are next used a
  // token later, behind those of all other layers
  a.stream = a.batch * a.H * a.P * a.N * (int64_t)sizeof(float) >= kMemorySideCache / 4;
  constexpr int TEAMS = kThreads / (NP / 4);
  auto go = [&](auto kern, int rows) {
    const uint32_t blocks_p = (a.P + TEAMS * rows - 1) / (TEAMS * rows);
    if (!grid_fits(a.batch * a.H * blocks_p, kThreads)) return hipErrorInvalidConfiguration;
    kern<<<dim3((unsigned)(a.batch * a.H * blocks_p)), kThreads, 0, s>>>(a, blocks_p);
    return hipGetLastError();
  };
  // Several rows a team where the teams are more than the card holds at once: fewer, longer
  // requests for each start of a workgroup. Rows a team 1 / 2 / 4: 37 rows of 32 heads, P = N = 64 12.7 / 9.2 / 8.5 us; 30 rows
  // of 32 heads, P = N = 128 32.2 / 26.6 / 23.2; past the caches, 256 of these 238 / 182 / 194; below
  // 2048 workgroups no difference. No team is left without a row for it.
  int rows = a.batch * a.H * ((a.P + TEAMS - 1) / TEAMS) < 2048 ? 1 : a.stream ? 2 : 4;
  while (rows > 1 && TEAMS * rows / 2 >= a.P) rows /= 2;
  auto pick = [&](auto vec) {
    constexpr bool V = decltype(vec)::value;
    if (rows == 4) return go(delta_step_kernel<TIO, TDT, NP, V, 4>, 4);
    if (rows == 2) return go(delta_step_kernel<TIO, TDT, NP, V, 2>, 2);
    return go(delta_step_kernel<TIO, TDT, NP, V, 1>, 1);
  };
  return a.N % 4 == 0 ? pick(std::true_type{}) : pick(std::false_type{});
}

template <typename TIO, typename TDT>
hipError_t launch_io(const DeltaStepArgs& a, hipStream_t s) {
  switch (selective_padded_states(a.N)) {
    case 16: return launch_np<TIO, TDT, 16>(a, s);
    case 32: return launch_np<TIO, TDT, 32>(a, s);
    case 64: return launch_np<TIO, TDT, 64>(a, s);
    case 128: return launch_np<TIO, TDT, 128>(a, s);
    default: return launch_np<TIO, TDT, 256>(a, s);
  }
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, int io, int dt, hipStream_t s) {
  if (io == kF32) return launch_io<float, float>(a, s);
  if (dt == kF32) return launch_io<__hip_bfloat16, float>(a, s);
  return launch_io<__hip_bfloat16, __hip_bfloat16>(a, s);
}

}  // namespace ssd
