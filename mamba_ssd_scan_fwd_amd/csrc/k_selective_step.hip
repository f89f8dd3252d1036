// The selective scan at one token: a step of every sequence of a batch, the
// states kept in a pool of slots between calls.
//     d = pre(dt[e]);  h[n] <- exp(d A[e][n]) h[n] + d x[e] B[g][n]
//     y[e] = (sum_n h[n] C[g][n] + D[e] x[e]) * silu(z[e])
//
// Streaming: the fp32 states are read once and written once, which is nearly
// all the traffic. Four consecutive states to a lane (one 16-byte access
// where N is a multiple of 4), padded N / 4 lanes to a channel; a workgroup keeps its
// channels' A for up to kRows rows of the batch, since A is as large as one
// row's state and would otherwise double what L2 has to deliver. All rows'
// loads are issued before the first is used. B and C in one access each took
// the kernel from 82 to 57 us (256 rows of 8192 channels): element by element
// they were half of all load instructions. Rows a workgroup: 1 68 us, 2 59, 4 57,
// 8 60. With the states past the cache (below) 51 us, 5.5 TB/s of 6.0 that an
// update in place reaches; one row of 4096 channels 3.1 us.
//
// A row whose slot is negative or behind the pool is padding: nothing is
// read or written for it. Where a slot is named twice the first row has it
// and the later ones are treated as padding, so no two rows write one state.
#include "selective.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

template <typename TIO, typename TDT, int NP, bool VEC, int R>
__global__ __launch_bounds__(kThreads) void selective_step_kernel(const SelectiveStepArgs a) {
  constexpr int LPC = NP / 4;  // lanes per channel
  const int tid = threadIdx.x;
  const int sub = tid % LPC;
  const int ch = blockIdx.x * (kThreads / LPC) + tid / LPC;
  const bool mine = ch < a.E;
  const int e = mine ? ch : a.E - 1;
  const int g = e / (a.E / a.G);
  const int64_t row0 = (int64_t)blockIdx.y * R;
  const int n0 = 4 * sub;
  const int nn = a.N - n0 < 0 ? 0 : a.N - n0 > 4 ? 4 : a.N - n0;  // states this lane holds
  const int nc = nn > 0 ? n0 : 0;                                 // an address inside the row for the others

  Pack<float, 4> Av = load_pack<float, 4, !VEC>(a.A + (int64_t)e * a.N + nc, nn);
  const float bias = a.dto.bias != nullptr ? a.dto.bias[e] : 0.f;
  const float Dv = a.D != nullptr ? a.D[e] : 0.f;

  Pack<float, 4> h[R];
  Pack<TIO, 4> bv[R], cv[R];
  typename Elem<TIO>::raw xv[R], zv[R];
  typename Elem<TDT>::raw dv[R];
  int64_t slot[R];
  const TIO* zp = static_cast<const TIO*>(a.z != nullptr ? a.z : a.x);
  const int64_t zs = a.z != nullptr ? a.zs : a.xs;
  using RX = typename Elem<TIO>::raw;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t r = row0 + k < a.batch ? row0 + k : a.batch - 1;
    slot[k] = a.slots != nullptr ? a.slots[r] : r;
    if (row0 + k >= a.batch || slot[k] < 0 || slot[k] >= a.nslots) slot[k] = -1;
    const int64_t from = slot[k] < 0 ? 0 : slot[k];
    const float* hp = a.state + (from * a.E + e) * a.N + nc;
    if (VEC && a.stream) h[k] = load_stream<float, 4>(hp);
    else h[k] = load_pack<float, 4, !VEC>(hp, nn);
    bv[k] = load_pack<TIO, 4, !VEC>(static_cast<const TIO*>(a.B) + r * a.bs + (int64_t)g * a.N + nc, nn);
    cv[k] = load_pack<TIO, 4, !VEC>(static_cast<const TIO*>(a.C) + r * a.cs + (int64_t)g * a.N + nc, nn);
    xv[k] = reinterpret_cast<const RX*>(a.x)[r * a.xs + e];
    dv[k] = reinterpret_cast<const typename Elem<TDT>::raw*>(a.dt)[r * a.ds + e];
    zv[k] = reinterpret_cast<const RX*>(zp)[r * zs + e];
  }
  if (a.slots != nullptr) {
    const uint32_t again = repeated_slots<R, kThreads>(a.slots, row0, a.batch);
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (again >> k & 1) slot[k] = -1;
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const float d = step_size(Elem<TDT>::f32(dv[k]), bias, a.dto);
    const float x = Elem<TIO>::f32(xv[k]), u = d * x;
    float hn[4], p = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float dec = __builtin_amdgcn_exp2f(d * log2_decay(Av.v[i]));
      hn[i] = fmaf(dec, h[k].v[i], u * Elem<TIO>::f32(bv[k].v[i]));
      if (i < nn) p = fmaf(hn[i], Elem<TIO>::f32(cv[k].v[i]), p);
    }
#pragma unroll
    for (int off = LPC / 2; off > 0; off >>= 1) p += __shfl_xor(p, off, LPC);
    if (slot[k] >= 0 && mine) {
      float* hp = a.state + (slot[k] * a.E + e) * a.N + n0;
      if (nn > 0) {
        if (VEC && a.stream) store_stream<float, 4>(hp, hn);
        else store_pack<float, 4, !VEC>(hp, hn, nn);
      }
      if (sub == 0) {
        float y = fmaf(Dv, x, p);
        if (a.z != nullptr) y *= silu_f32(Elem<TIO>::f32(zv[k]));
        reinterpret_cast<RX*>(a.y)[(row0 + k) * a.E + e] = Elem<TIO>::bits(y);
      }
    }
  }
}

template <typename TIO, typename TDT, int NP>
hipError_t launch_np(const SelectiveStepArgs& args, hipStream_t s) {
  SelectiveStepArgs a = args;
  // A layer's states are next used a token later, behind those of all other
  // layers. From a quarter of the memory-side cache on they are not kept in it
  // (non-temporal): 256 rows of 8192 x 16 (128 MiB), three layers in turn, 57 ->
  // 52 us, 128 rows of twelve layers 31 -> 28 us. That costs a program of one
  // layer, whose states would stay there (44 -> 52, 24 -> 27 us), and from 64
  // rows down it would cost three layers too (13.8 -> 15.7 us).
  a.stream = a.batch * a.E * a.N * (int64_t)sizeof(float) >= kMemorySideCache / 4;
  const unsigned gx = (unsigned)((a.E + kThreads / (NP / 4) - 1) / (kThreads / (NP / 4)));
  const bool vec = a.N % 4 == 0;  // no lane holds part of four states
  auto go = [&](auto kern, int rows) {
    kern<<<dim3(gx, (unsigned)((a.batch + rows - 1) / rows)), kThreads, 0, s>>>(a);
    return hipGetLastError();
  };
  // several rows a workgroup once that still leaves the card full
  const bool many = (int64_t)gx * a.batch >= 4 * 2048;
  if (vec) return many ? go(selective_step_kernel<TIO, TDT, NP, true, 4>, 4) : go(selective_step_kernel<TIO, TDT, NP, true, 1>, 1);
  return go(selective_step_kernel<TIO, TDT, NP, false, 1>, 1);
}

template <typename TIO, typename TDT>
hipError_t launch_io(const SelectiveStepArgs& a, hipStream_t s) {
  switch (selective_padded_states(a.N)) {
    case 16: return launch_np<TIO, TDT, 16>(a, s);
    case 32: return launch_np<TIO, TDT, 32>(a, s);
    case 64: return launch_np<TIO, TDT, 64>(a, s);
    case 128: return launch_np<TIO, TDT, 128>(a, s);
    default: return launch_np<TIO, TDT, 256>(a, s);
  }
}

}  // namespace

hipError_t launch_selective_step(const SelectiveStepArgs& a, int io, int dt, hipStream_t s) {
  if (io == kF32) return launch_io<float, float>(a, s);
  if (dt == kF32) return launch_io<__hip_bfloat16, float>(a, s);
  return launch_io<__hip_bfloat16, __hip_bfloat16>(a, s);
}

}  // namespace ssd
