// The selective scan: the recurrence with a decay of its own for every
// channel and state (the diagonal transition that the SSD form replaces by one
// scalar per head). Per batch row or packed sequence, channel e of B/C group g:
//     d_t       = pre(dt_t[e])                            (bias, softplus, clamp)
//     h_t[n]    = exp(d_t A[e][n]) h_{t-1}[n] + d_t x_t[e] B_t[g][n]
//     y_t[e]    = (sum_n h_t[n] C_t[g][n] + D[e] x_t[e]) * silu(z_t[e])
//
// A product with the decays of every (e, n) has no matrix form over tokens, so
// this is vector work: per token, channel and state one exp2, two products
// and two fused adds. Memory (x, dt, z and y once) stays well below that.
//
// Layout: four lanes share a channel, each holding a quarter of its states in
// registers for the whole walk over the tokens; a workgroup of four waves
// takes 64 channels of one group, so a token's row of a bf16 array is one
// 128-byte line. Tokens go in groups of four: lane q of the quad loads x, dt
// and z of token 4i + q and computes its softplus, dt x, gate and store alone
// (nothing is done four times), and the four tokens' dt and dt x reach the
// quad by DPP broadcasts. The four partial sums of y are exchanged in one
// transposing reduction (three adds), which leaves token 4i + q's sum in lane
// q. B and C are the same for all channels of a group: they are converted to
// fp32 once per tile into LDS (two buffers, one barrier a tile), whence the
// four quarters read 16 bytes each, without bank conflicts.
//
// The time axis: where batch rows and channels are too few waves for the
// card, the tokens are cut into segments. A first launch walks each segment
// but the last from a zero state (or the initial state) and leaves its end
// state and its sum of d; the second walks every segment again with its
// output, from the state folded together from the segments before:
//     h <- exp(A sum_j d) h + end_j.
// That doubles most of the arithmetic, so it is done only below a wave count
// (selective_scan_segments). No workgroup waits for another.
//
// Packed sequences use the same segments of the packed stream; a segment's
// walk is a list of runs, one for each sequence with tokens in it, each
// beginning from its own state, so nothing of one sequence meets another.
#include "selective.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kChannels = 64;  // channels per workgroup

// One lane of the quad's value in all four (DPP quad_perm [j, j, j, j]).
template <int J> __device__ __forceinline__ float quad_bcast(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), J * 0x55, 0xf, 0xf, true));
}
// Lane q ^ X of the quad (X = 1: [1, 0, 3, 2], X = 2: [2, 3, 0, 1]).
template <int X> __device__ __forceinline__ float quad_xor(float v) {
  constexpr int ctrl = X == 1 ? 0xB1 : 0x4E;
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, true));
}

template <typename T> __device__ __forceinline__ typename Elem<T>::raw load_raw(const T* p, uint32_t off) {
  return *reinterpret_cast<const typename Elem<T>::raw*>(reinterpret_cast<const char*>(p) + off);
}

// Tokens per tile (a multiple of 4): the unrolled tile has tokens * states / 4
// state updates, kept within the instruction cache.
constexpr int tile_tokens(int np) { return np <= 32 ? 32 : np == 64 ? 16 : np == 128 ? 8 : 4; }

// OUT: the walk that writes y and the final states; otherwise the walk that
// leaves the segments' end states.
template <typename TIO, typename TDT, int NP, bool OUT>
__global__ __launch_bounds__(kThreads) void selective_scan_kernel(const SelectiveArgs a) {
  constexpr int SPL = NP / 4;  // states per lane: n = 16 i + 4 q + k
  constexpr int TT = tile_tokens(NP);
  constexpr int GR = TT / 4;   // groups of four tokens per tile
  constexpr int ROW = OUT ? 2 * NP : NP;  // LDS row of a token: B, then C
  constexpr int PER = TT * NP / kThreads;  // elements of B (and of C) a thread stages
  __shared__ float4 bc4[2][TT * ROW / 4];

  const int tid = threadIdx.x;
  const int q = tid & 3;
  const int g = blockIdx.x / a.tiles;
  const int cg = (blockIdx.x % a.tiles) * kChannels + tid / 4;
  const bool mine = cg < a.epg;
  const int e = g * a.epg + (mine ? cg : a.epg - 1);
  const int64_t b = blockIdx.z;
  const int seg = blockIdx.y;
  const int64_t s0 = (int64_t)seg * a.seg_len;
  const int64_t s1 = s0 + a.seg_len < a.L ? s0 + a.seg_len : a.L;

  const TIO* xb = static_cast<const TIO*>(a.x) + b * a.xs.batch;
  const TDT* db = static_cast<const TDT*>(a.dt) + b * a.ds.batch;
  const TIO* zb = OUT && a.z != nullptr ? static_cast<const TIO*>(a.z) + b * a.zs.batch : xb;
  const int64_t zt = OUT && a.z != nullptr ? a.zs.token : a.xs.token;
  const TIO* Bb = static_cast<const TIO*>(a.B) + b * a.bs.batch + (int64_t)g * a.N;
  const TIO* Cb = static_cast<const TIO*>(a.C) + b * a.cs.batch + (int64_t)g * a.N;
  TIO* yb = static_cast<TIO*>(a.y) + b * a.L * a.E;
  // this lane's place in the rows of a group of four tokens, in bytes
  const uint32_t xo = (uint32_t)((q * a.xs.token + e) * sizeof(TIO));
  const uint32_t dof = (uint32_t)((q * a.ds.token + e) * sizeof(TDT));
  const uint32_t zo = (uint32_t)((q * zt + e) * sizeof(TIO));
  const uint32_t yo = (uint32_t)(((int64_t)q * a.E + e) * sizeof(TIO));

  float A2[SPL], h[SPL];
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    const int n = (s / 4) * 16 + q * 4 + s % 4;
    A2[s] = n < a.N ? a.A[(int64_t)e * a.N + n] * kLog2e : 0.f;
  }
  const float bias = a.dto.bias != nullptr ? a.dto.bias[e] : 0.f;
  const float Dv = OUT && a.D != nullptr ? a.D[e] : 0.f;
  float dsum = 0.f;

  auto load_state = [&](const float* src, int64_t row) {  // [row, E, N], or zeros
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      const int n = (s / 4) * 16 + q * 4 + s % 4;
      h[s] = src != nullptr && n < a.N ? src[(row * a.E + e) * a.N + n] : 0.f;
    }
  };
  auto store_state = [&](float* dst, int64_t row) {
    if (!mine) return;
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
      const int n = (s / 4) * 16 + q * 4 + s % 4;
      if (n < a.N) dst[(row * a.E + e) * a.N + n] = h[s];
    }
  };
  // workspace states: [batch, segment, E, NP]
  auto ws_at = [&](float* base, int64_t j, int i) {
    return reinterpret_cast<float4*>(base + (((b * a.nseg + j) * a.E + e) * NP + i * 16 + q * 4));
  };
  auto ws_store = [&](float* base) {
    if (!mine) return;
#pragma unroll
    for (int i = 0; i < SPL / 4; ++i) *ws_at(base, seg, i) = make_float4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
  };

  int buf = 0;
  using RX = typename Elem<TIO>::raw;
  using RD = typename Elem<TDT>::raw;

  // One run: tokens [r0, r1) of one sequence, h updated over them.
  auto walk = [&](int64_t r0, int64_t r1) {
    RX bn[PER], cn[OUT ? PER : 1];
    RX xn[GR], zn[OUT ? GR : 1];
    RD dn[GR];
    // loads of the tile at t0, all from addresses inside the run
    auto fetch = [&](int64_t t0) {
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int el = tid + k * kThreads, n = el % NP;
        int64_t t = t0 + el / NP;
        t = t < r1 ? t : r1 - 1;
        const int nn = n < a.N ? n : a.N - 1;
        bn[k] = *reinterpret_cast<const RX*>(Bb + t * a.bs.token + nn);
        if constexpr (OUT) cn[k] = *reinterpret_cast<const RX*>(Cb + t * a.cs.token + nn);
      }
      if (t0 + TT <= r1) {
#pragma unroll
        for (int i = 0; i < GR; ++i) {
          dn[i] = load_raw(db + (t0 + 4 * i) * a.ds.token, dof);
          xn[i] = load_raw(xb + (t0 + 4 * i) * a.xs.token, xo);
          if constexpr (OUT) zn[i] = load_raw(zb + (t0 + 4 * i) * zt, zo);
        }
      } else {
#pragma unroll
        for (int i = 0; i < GR; ++i) {
          int64_t t = t0 + 4 * i + q;
          t = t < r1 ? t : r1 - 1;
          dn[i] = load_raw(db + t * a.ds.token + e, 0);
          xn[i] = load_raw(xb + t * a.xs.token + e, 0);
          if constexpr (OUT) zn[i] = load_raw(zb + t * zt + e, 0);
        }
      }
    };
    // B and C into the other buffer (zeros behind the run and behind N)
    auto stage = [&](int64_t t0) {
      float* dst = reinterpret_cast<float*>(bc4[buf]);
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int el = tid + k * kThreads, n = el % NP, tk = el / NP;
        const bool in = n < a.N && t0 + tk < r1;
        dst[tk * ROW + n] = in ? Elem<TIO>::f32(bn[k]) : 0.f;
        if constexpr (OUT) dst[tk * ROW + NP + n] = in ? Elem<TIO>::f32(cn[k]) : 0.f;
      }
    };

    fetch(r0);
    for (int64_t t0 = r0; t0 < r1; t0 += TT) {
      buf ^= 1;
      stage(t0);
      RX xc[GR], zc[OUT ? GR : 1];
      RD dc[GR];
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        xc[i] = xn[i];
        dc[i] = dn[i];
        if constexpr (OUT) zc[i] = zn[i];
      }
      __syncthreads();
      if (t0 + TT < r1) fetch(t0 + TT);
      const float4* row = bc4[buf] + q;
      const int left = (int)(r1 - t0 < TT ? r1 - t0 : TT);
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        const bool in = 4 * i + q < left;
        // tokens behind the run: a step of zero leaves the state as it is
        const float dv = in ? step_size(Elem<TDT>::f32(dc[i]), bias, a.dto) : 0.f;
        const float xv = in ? Elem<TIO>::f32(xc[i]) : 0.f;
        const float uv = dv * xv;
        float acc[4];
        auto token = [&](auto jc) {
          constexpr int j = decltype(jc)::value;
          const float d = quad_bcast<j>(dv), u = quad_bcast<j>(uv);
          const float4* rj = row + (4 * i + j) * (ROW / 4);
          float p = 0.f;
#pragma unroll
          for (int v = 0; v < SPL / 4; ++v) {
            const float4 bv = rj[4 * v];
            float4 cv = make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (OUT) cv = rj[NP / 4 + 4 * v];
            const float bb[4] = {bv.x, bv.y, bv.z, bv.w}, cc[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int s = 4 * v + k;
              h[s] = fmaf(__builtin_amdgcn_exp2f(d * A2[s]), h[s], u * bb[k]);
              if constexpr (OUT) p = fmaf(h[s], cc[k], p);
            }
          }
          acc[j] = p;
        };
        token(std::integral_constant<int, 0>{});
        token(std::integral_constant<int, 1>{});
        token(std::integral_constant<int, 2>{});
        token(std::integral_constant<int, 3>{});
        if constexpr (OUT) {
          // sum over the quad, transposed: lane q ends with token q's
          const bool o1 = q & 1, o2 = q & 2;
          const float k0 = o1 ? acc[1] : acc[0], m0 = o1 ? acc[0] : acc[1];
          const float k1 = o1 ? acc[3] : acc[2], m1 = o1 ? acc[2] : acc[3];
          const float v0 = k0 + quad_xor<1>(m0), v1 = k1 + quad_xor<1>(m1);
          float yv = (o2 ? v1 : v0) + quad_xor<2>(o2 ? v0 : v1);
          yv = fmaf(Dv, xv, yv);
          if (a.z != nullptr) yv *= silu_f32(Elem<TIO>::f32(zc[i]));
          if (in && mine)
            *reinterpret_cast<RX*>(reinterpret_cast<char*>(yb + (t0 + 4 * i) * a.E) + yo) = Elem<TIO>::bits(yv);
        } else {
          dsum += dv;
        }
      }
    }
  };

  if constexpr (!OUT) {
    // the run that reaches the segment's end and goes on behind it
    int64_t row = b, first = 0, last = a.L;
    if (a.cu != nullptr) {
      row = seq_of(a.cu, a.nseq, a.L, s1 - 1);
      if (row >= a.nseq) return;
      first = seq_offset(a.cu, row, a.L);
      last = seq_offset(a.cu, row + 1, a.L);
    }
    if (last <= s1) return;
    const bool starts = first >= s0;
    if (starts) {
      load_state(a.init, row);
      if (a.init_copy != nullptr) ws_store(a.init_copy);
    } else {
      load_state(nullptr, 0);
    }
    walk(starts ? first : s0, s1);
    ws_store(a.ends);
    dsum += quad_xor<1>(dsum);
    dsum += quad_xor<2>(dsum);
    if (mine && q == 0) a.dsums[(b * a.nseg + seg) * a.E + e] = dsum;
  } else {
    // the state that enters at the segment's start, for a sequence that
    // began in segment j0
    auto enter = [&](int64_t j0) {
#pragma unroll
      for (int i = 0; i < SPL / 4; ++i) {
        const float4 v = *ws_at(a.ends, j0, i);
        h[4 * i] = v.x, h[4 * i + 1] = v.y, h[4 * i + 2] = v.z, h[4 * i + 3] = v.w;
      }
      for (int64_t j = j0 + 1; j < seg; ++j) {
        const float ds = a.dsums[(b * a.nseg + j) * a.E + e];
#pragma unroll
        for (int i = 0; i < SPL / 4; ++i) {
          const float4 v = *ws_at(a.ends, j, i);
          const float vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            h[4 * i + k] = fmaf(__builtin_amdgcn_exp2f(ds * A2[4 * i + k]), h[4 * i + k], vv[k]);
        }
      }
    };
    auto begin = [&](int64_t row, bool goes_on) {
      if (goes_on && a.init_copy != nullptr) {
        // the final state of this sequence may be written over its initial
        // state by another workgroup of this launch: take the kept copy
#pragma unroll
        for (int i = 0; i < SPL / 4; ++i) {
          const float4 v = *ws_at(a.init_copy, seg, i);
          h[4 * i] = v.x, h[4 * i + 1] = v.y, h[4 * i + 2] = v.z, h[4 * i + 3] = v.w;
        }
      } else {
        load_state(a.init, row);
      }
    };
    if (a.cu == nullptr) {
      if (seg == 0) begin(b, a.L > s1); else enter(0);
      walk(s0, s1);
      if (s1 == a.L && a.final_state != nullptr) store_state(a.final_state, b);
    } else {
      int64_t row = seq_of(a.cu, a.nseq, a.L, s0);
      int64_t pos = s0;
      while (pos < s1 && row < a.nseq) {
        const int64_t first = seq_offset(a.cu, row, a.L), last = seq_offset(a.cu, row + 1, a.L);
        if (last > pos && first <= pos) {
          const int64_t r1 = last < s1 ? last : s1;
          if (first < s0) enter(first / a.seg_len); else begin(row, last > s1);
          walk(pos, r1);
          if (last <= s1 && a.final_state != nullptr) store_state(a.final_state, row);
          pos = r1;
        }
        ++row;
      }
      // sequences without tokens keep their state: this segment's share of them
      if (a.final_state != nullptr) {
        const int lane = tid & 63;
        for (int64_t r = (int64_t)seg * 64; r < a.nseq; r += (int64_t)a.nseg * 64) {
          const int64_t i = r + lane < a.nseq ? r + lane : a.nseq - 1;
          uint64_t empty = __ballot(r + lane < a.nseq && seq_offset(a.cu, i + 1, a.L) <= seq_offset(a.cu, i, a.L));
          while (empty != 0) {
            const int k = __builtin_ctzll(empty);
            empty &= empty - 1;
            load_state(a.init, r + k);
            store_state(a.final_state, r + k);
          }
        }
      }
    }
  }
}

template <typename TIO, typename TDT, int NP>
hipError_t launch_np(const SelectiveArgs& a, int64_t batch, hipStream_t s) {
  const unsigned tiles = (unsigned)(a.tiles * (a.E / a.epg));
  if (a.nseg > 1) {
    selective_scan_kernel<TIO, TDT, NP, false><<<dim3(tiles, (unsigned)(a.nseg - 1), (unsigned)batch), kThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  selective_scan_kernel<TIO, TDT, NP, true><<<dim3(tiles, (unsigned)a.nseg, (unsigned)batch), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename TIO, typename TDT>
hipError_t launch_io(const SelectiveArgs& a, int64_t batch, hipStream_t s) {
  switch (selective_padded_states(a.N)) {
    case 16: return launch_np<TIO, TDT, 16>(a, batch, s);
    case 32: return launch_np<TIO, TDT, 32>(a, batch, s);
    case 64: return launch_np<TIO, TDT, 64>(a, batch, s);
    case 128: return launch_np<TIO, TDT, 128>(a, batch, s);
    default: return launch_np<TIO, TDT, 256>(a, batch, s);
  }
}

}  // namespace

SelectiveCut selective_scan_segments(int64_t batch, int64_t L, int64_t E, int64_t G, int64_t nseq) {
  const int64_t tiles = (E / G + kChannels - 1) / kChannels * G;
  const int64_t waves = tiles * 4 * batch;
  // one wave a SIMD keeps the vector units busy enough that walking the
  // tokens twice would cost more; below that, aim at two waves a SIMD
  const int64_t full = 1024;
  int64_t want = waves >= full ? 1 : (2 * full + waves - 1) / waves;
  int64_t len = (L + want - 1) / want;
  if (nseq > 0 && 4 * L / nseq < len) len = 4 * L / nseq;
  if (len < 64) len = 64;
  len = (len + 31) / 32 * 32;
  SelectiveCut c;
  c.nseg = (L + len - 1) / len;
  if (c.nseg > 65535) {
    len = ((L + 65534) / 65535 + 31) / 32 * 32;
    c.nseg = (L + len - 1) / len;
  }
  c.len = len;
  return c;
}

hipError_t launch_selective_scan(const SelectiveArgs& args, int io, int dt, int64_t batch, hipStream_t s) {
  SelectiveArgs a = args;
  a.epg = (int)(a.E / a.G);
  a.tiles = (a.epg + kChannels - 1) / kChannels;
  if (io == kF32) return launch_io<float, float>(a, batch, s);
  if (dt == kF32) return launch_io<__hip_bfloat16, float>(a, batch, s);
  return launch_io<__hip_bfloat16, __hip_bfloat16>(a, batch, s);
}

}  // namespace ssd
