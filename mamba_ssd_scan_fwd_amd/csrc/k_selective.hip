// The selective scan: the recurrence with a decay of its own for every
// channel and state (the diagonal transition that the SSD form replaces by one
// scalar per head). Per batch row or packed sequence, channel e of B/C group g:
//     d_t       = pre(dt_t[e])                            (bias, softplus, clamp)
//     h_t[n]    = exp(d_t A[e][n]) h_{t-1}[n] + d_t x_t[e] B_t[g][n]
//     y_t[e]    = (sum_n h_t[n] C_t[g][n] + D[e] x_t[e]) * silu(z_t[e])
//
// A product with the decays of every (e, n) has no matrix form over tokens, so
// this is vector work: per token, channel and state one exp2, two products
// and two fused adds: for 64 lanes 4 x 4 + 8 = 24 cycles of a SIMD (a wave's
// exp2 takes 8 cycles and keeps other waves' arithmetic waiting, measured).
// Memory (x, dt, z and y once) stays well below that.
//
// Layout: four lanes share a channel, each holding a quarter of its states in
// registers for the whole walk over the tokens; a workgroup of four waves
// takes 64 channels of one group, so a token's row of a bf16 array is one
// 128-byte line. Tokens go in groups of four: lane q of the quad takes x, dt
// and z of token 4i + q and computes its softplus, dt x and gate alone (nothing
// is done four times), and the four tokens' dt and dt x reach the quad by DPP
// broadcasts. The four partial sums of y are exchanged in one transposing
// reduction (three adds), which leaves token 4i + q's sum in lane q.
//
// Tiles of 32 tokens (fewer with more states) go through LDS, two buffers and
// one barrier a tile: x, dt and z as they are, in 16-byte accesses, and B and
// C, the same for all channels of a group, converted to fp32, whence the four
// quarters read 16 bytes each. The next tile's loads are issued at the start of
// a tile and written to LDS before y is stored, so that no wait for a load is
// also a wait for a store.
//
// Measured (8 x 2048 tokens, 4096 channels, 16 states, bf16, gate): 264 us;
// the vector units busy 86% of the time; 30 instructions a token and wave, of which
// the 20 above are the states' and 9 the step sizes, gates and moves. The
// arithmetic of the 20 alone takes about 180 us, a copy of the same bytes 100.
//
// The time axis: where batch rows and channels are too few waves for the
// card, the tokens are cut into segments. A first launch walks each segment
// but the last from a zero state (or the initial state) and leaves its end
// state and its sum of d; the second walks every segment again with its
// output, from the state folded together from the segments before:
//     h <- exp(A sum_j d) h + end_j.
// That doubles most of the arithmetic, so it is done only below a wave count
// (selective_scan_cut). No workgroup waits for another.
//
// Packed sequences use the same segments of the packed stream; a segment's
// walk is a list of runs, one for each sequence with tokens in it, each
// beginning from its own state, so nothing of one sequence meets another.
#include "selective.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kChannels = 64;  // channels per workgroup
// Elements from one token to the next in LDS: a quarter row more than its
// channels, so the four tokens that a wave reads at once lie in other banks.
constexpr int kPitch = kChannels + 16;

// One lane of the quad's value in all four (DPP quad_perm [j, j, j, j]).
template <int J> __device__ __forceinline__ float quad_bcast(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), J * 0x55, 0xf, 0xf, true));
}
// j is a constant wherever this is called, once the loops are unrolled.
__device__ __forceinline__ float quad_bcast_of(int j, float v) {
  return j == 0 ? quad_bcast<0>(v) : j == 1 ? quad_bcast<1>(v) : j == 2 ? quad_bcast<2>(v) : quad_bcast<3>(v);
}
// Lane q ^ X of the quad (X = 1: [1, 0, 3, 2], X = 2: [2, 3, 0, 1]).
template <int X> __device__ __forceinline__ float quad_xor(float v) {
  constexpr int ctrl = X == 1 ? 0xB1 : 0x4E;
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, true));
}

// V consecutive elements in 32-bit words, as they lie in memory. (Words, not
// elements: 16-bit values that come from two branches would be unpacked, and
// so waited for, right behind the loads.)
template <typename T, int V> struct Words {
  static constexpr int BYTES = V * (int)sizeof(T);
  static constexpr int N = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t w[N];
  __device__ __forceinline__ float f32(int k) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
    else return __uint_as_float(k % 2 == 0 ? w[k / 2] << 16 : w[k / 2] & 0xffff0000u);
  }
  // to V elements in LDS, aligned to them (up to 16 bytes)
  __device__ __forceinline__ void put(typename Elem<T>::raw* at) const {
    if constexpr (BYTES == 2) *at = (typename Elem<T>::raw)w[0];
    else *reinterpret_cast<Pack<float, N>*>(at) = __builtin_bit_cast(Pack<float, N>, *this);
  }
};

// Elements at `row` (of the wave) + `off` bytes from p, of which n are there
// (at least one; the first stands in for the others), in accesses of up to
// 16 bytes, at any address, where WHOLE says that all are.
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void load_row(Words<T, V>& r, const T* p, uint64_t row, uint32_t off, int n) {
  using W = Words<T, V>;
  const char* at = reinterpret_cast<const char*>(p) + row + off;
  if constexpr (W::BYTES == 2) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(at);
  } else if constexpr (WHOLE) {
    // (a vector, not memcpy: that may keep r in memory, in LDS or scratch)
    typedef uint32_t Vec __attribute__((ext_vector_type(W::N), aligned(sizeof(T))));
    const Vec v = *reinterpret_cast<const Vec*>(at);
#pragma unroll
    for (int k = 0; k < W::N; ++k) r.w[k] = v[k];
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < V; ++k) r.w[k] = reinterpret_cast<const uint32_t*>(at)[k < n ? k : 0];
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      const uint16_t* e = reinterpret_cast<const uint16_t*>(at);
      r.w[k] = e[2 * k < n ? 2 * k : 0] | (uint32_t)e[2 * k + 1 < n ? 2 * k + 1 : 0] << 16;
    }
  }
}

// Moves a byte offset of the whole wave on. The empty asm keeps it in its
// registers: as a function of the loop count it would be recomputed with
// 64-bit products on every tile.
__device__ __forceinline__ void advance(uint64_t& off, uint32_t bytes) {
  off += bytes;
  asm volatile("" : "+s"(off));
}

// Tokens per tile (a multiple of 4): the unrolled tile has tokens * states / 4
// state updates, kept within the instruction cache.
constexpr int tile_tokens(int np) { return np <= 32 ? 32 : np == 64 ? 16 : np == 128 ? 8 : 4; }

// OUT: the walk that writes y and the final states; otherwise the walk that
// leaves the segments' end states.
// The first walk's waves: what LDS lets stand on a SIMD (16 states in 16-bit
// types: 16384 tokens of 4096 channels 453 us in all with the four that the
// compiler's registers would leave, 433 with five).
template <typename TIO, typename TDT, int NP, bool OUT>
__global__ __launch_bounds__(kThreads, !OUT && NP == 16 && sizeof(TIO) + sizeof(TDT) == 4 ? 5 : 1) void selective_scan_kernel(const SelectiveArgs a) {
  constexpr int SPL = NP / 4;  // states per lane: n = 16 i + 4 q + k
  constexpr int TT = tile_tokens(NP);
  constexpr int GR = TT / 4;   // groups of four tokens per tile
  constexpr int VU = SPL / 4;  // units of four states per lane and token
  constexpr int ROW = OUT ? 2 * NP : NP;  // LDS row of a token: B, then C
  constexpr int PER = TT * NP / kThreads;         // states of B (and of C) a thread stages
  constexpr int PK = TT * kChannels / kThreads;   // channels of one token it stages of x, dt and z
  using RX = typename Elem<TIO>::raw;
  using RD = typename Elem<TDT>::raw;
  __shared__ float4 bc4[2][TT * ROW / 4];
  __shared__ __attribute__((aligned(16))) RX xl[2][TT * kPitch];
  __shared__ __attribute__((aligned(16))) RX zl[OUT ? 2 : 1][OUT ? TT * kPitch : 1];
  __shared__ __attribute__((aligned(16))) RD dl[2][TT * kPitch];

  const int tid = threadIdx.x;
  const int q = tid & 3;
  const int g = blockIdx.x / a.tiles;
  // Where a group does not end with a pack, its last workgroup moves back to end
  // with it, so that its packs are whole too: the channels that it shares with the one before are computed
  // by both and written by that one alone (8 x 2048 tokens of 4095 channels:
  // 369 us element by element, 293 moved). Where the final state lies over the
  // initial one, the shared channels may start from what the other has already
  // written; nothing of theirs leaves the workgroup.
  const int ch = (blockIdx.x % a.tiles) * kChannels;
  const int shared = a.epg % PK != 0 && a.epg >= kChannels && ch + kChannels > a.epg ? ch + kChannels - a.epg : 0;
  const int ch0 = ch - shared;
  const int cg = ch0 + tid / 4;
  const bool mine = cg < a.epg && tid / 4 >= shared;
  const int e = g * a.epg + (cg < a.epg ? cg : a.epg - 1);
  const int64_t b = blockIdx.z;
  // the piece of the time axis this workgroup begins with, and its tokens:
  // one piece, or with output a segment of them
  const int seg = OUT ? blockIdx.y * a.cut.pieces : blockIdx.y;
  const int64_t s0 = (int64_t)seg * a.cut.len, want = (int64_t)a.cut.len * (OUT ? a.cut.pieces : 1);
  const int64_t s1 = s0 + want < a.L ? s0 + want : a.L;

  const TIO* xb = static_cast<const TIO*>(a.x) + b * a.xs.batch + (int64_t)g * a.epg;
  const TDT* db = static_cast<const TDT*>(a.dt) + b * a.ds.batch + (int64_t)g * a.epg;
  const TIO* zb = OUT && a.z != nullptr ? static_cast<const TIO*>(a.z) + b * a.zs.batch + (int64_t)g * a.epg : xb;
  const int64_t zt = OUT && a.z != nullptr ? a.zs.token : a.xs.token;
  const TIO* Bb = static_cast<const TIO*>(a.B) + b * a.bs.batch + (int64_t)g * a.N;
  const TIO* Cb = static_cast<const TIO*>(a.C) + b * a.cs.batch + (int64_t)g * a.N;
  TIO* yb = static_cast<TIO*>(a.y) + b * a.L * a.E + (int64_t)g * a.epg;
  // row strides in bytes
  const uint32_t xs = (uint32_t)(a.xs.token * sizeof(TIO)), ds = (uint32_t)(a.ds.token * sizeof(TDT));
  const uint32_t zs = (uint32_t)(zt * sizeof(TIO));
  const uint32_t bs = (uint32_t)(a.bs.token * sizeof(TIO)), cs = (uint32_t)(a.cs.token * sizeof(TIO));
  const uint32_t ys = (uint32_t)(a.E * sizeof(TIO));
  const bool o1 = q & 1, o2 = q & 2;

  float A2[SPL], h[SPL];
#pragma unroll
  for (int s = 0; s < SPL; ++s) {
    const int n = (s / 4) * 16 + q * 4 + s % 4;
    // (finite, also for the steps of zero behind a run's end)
    A2[s] = n < a.N ? log2_decay(a.A[(int64_t)e * a.N + n]) : 0.f;
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
    return reinterpret_cast<float4*>(base + (((b * a.cut.n + j) * a.E + e) * NP + i * 16 + q * 4));
  };
  auto ws_store = [&](float* base) {
    if (!mine) return;
#pragma unroll
    for (int i = 0; i < SPL / 4; ++i) *ws_at(base, seg, i) = make_float4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
  };

  // whether all of this workgroup's packs of x, dt, z and y, and of B and C, are whole
  const bool whole = (a.epg % PK == 0 || a.epg >= kChannels) && a.N >= PER;
  if (whole && a.N < NP) {  // what whole packs leave out stays zero
    for (int i = tid; i < 2 * TT * ROW / 4; i += kThreads) (&bc4[0][0])[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  }
  int buf = 0;
  const int wave_slot = __builtin_amdgcn_s_getreg(4 | 0 << 6 | 3 << 11);  // HW_ID: wave of its SIMD

  // One run: tokens [r0, r1) of one sequence, h updated over them. WHOLE: all
  // packs are whole; MOVED: the workgroup writes its channels from `shared` on.
  // Each is a walk of its own, not a branch inside of one: where two fetches
  // meet, the loads are waited for, and a choice at y's store keeps it from
  // overlapping (8 x 2048 tokens, 4096 channels: 284 us with the fetch chosen
  // in the walk, 278 with the store, 264 with neither).
  auto walk_as = [&](auto whole_of, auto moved_of, int64_t r0, int64_t r1) {
    constexpr bool WHOLE = decltype(whole_of)::value, MOVED = decltype(moved_of)::value;
    // what this thread stages: states bn0.. of token btk, channels xc0.. of
    // token xtk (the group's first where it has none there). WHOLE: a pack of
    // B or C that reaches behind N moves back to end with it; what two packs
    // share they both write, alike.
    const int btk = tid * PER / NP, bp = tid * PER % NP;
    const int bn0 = WHOLE && bp > a.N - PER ? a.N - PER : bp;
    const int xtk = tid * PK / kChannels, xc0 = tid * PK % kChannels;
    const int there = a.epg - ch0 - xc0;
    const int xn0 = there > 0 ? ch0 + xc0 : 0, xnn = there > 0 ? there : 1;
    Words<TIO, PER> bn, cn;
    Words<TIO, PK> xn, zn;
    Words<TDT, PK> dn;
    // the next tile's rows, and the tokens left from there on
    uint64_t xr = r0 * xs, dr = r0 * ds, zr = r0 * zs, br = r0 * bs, cr = r0 * cs, yr = r0 * ys;
    int left = (int)(r1 - r0);
    // loads of the next tile, all from addresses inside the run
    auto fetch = [&](int left) {
      const int bt = btk < left ? btk : left - 1, xt = xtk < left ? xtk : left - 1;
      const int nb = bn0 < a.N ? bn0 : 0, nbn = a.N - nb;
      load_row<WHOLE>(dn, db, dr, __umul24(xt, ds) + (uint32_t)(xn0 * sizeof(TDT)), xnn);
      load_row<WHOLE>(xn, xb, xr, __umul24(xt, xs) + (uint32_t)(xn0 * sizeof(TIO)), xnn);
      if constexpr (OUT) load_row<WHOLE>(zn, zb, zr, __umul24(xt, zs) + (uint32_t)(xn0 * sizeof(TIO)), xnn);
      load_row<WHOLE>(bn, Bb, br, __umul24(bt, bs) + (uint32_t)(nb * sizeof(TIO)), nbn);
      if constexpr (OUT) load_row<WHOLE>(cn, Cb, cr, __umul24(bt, cs) + (uint32_t)(nb * sizeof(TIO)), nbn);
      advance(xr, TT * xs);
      advance(dr, TT * ds);
      advance(br, TT * bs);
      if constexpr (OUT) {
        advance(zr, TT * zs);
        advance(cr, TT * cs);
      }
    };
    // into a buffer: B and C in fp32 (zeros behind the run and behind
    // N), the rest as it is
    auto stage = [&](int left, int buf) {
      float* dst = reinterpret_cast<float*>(bc4[buf]) + btk * ROW + bn0;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const bool in = (WHOLE || bn0 + k < a.N) && btk < left;
        dst[k] = in ? bn.f32(k) : 0.f;
        if constexpr (OUT) dst[NP + k] = in ? cn.f32(k) : 0.f;
      }
      const int at = xtk * kPitch + xc0;
      xn.put(xl[buf] + at);
      dn.put(dl[buf] + at);
      if constexpr (OUT) zn.put(zl[buf] + at);
    };

    // NG groups of four tokens from group i0 of the tile on. TAIL: the run may
    // end among them; behind it a step of zero leaves the state as it is.
    auto groups = [&](auto ng, auto tail, auto more, int i0) {
      constexpr int NG = decltype(ng)::value;
      constexpr bool TAIL = decltype(tail)::value, MORE = decltype(more)::value;
      const int at0 = (4 * i0 + q) * kPitch + tid / 4;
      RX* xq = xl[buf] + at0;
      const RD* dq = dl[buf] + at0;
      float dv[NG], xv[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        dv[i] = Elem<TDT>::f32(dq[4 * i * kPitch]) + bias;
        xv[i] = Elem<TIO>::f32(xq[4 * i * kPitch]);
      }
      if (a.dto.softplus) {
#pragma unroll
        for (int i = 0; i < NG; ++i) dv[i] = softplus_f32(dv[i]);
      }
      if (a.dto.clamp) {
#pragma unroll
        for (int i = 0; i < NG; ++i) dv[i] = clamped(dv[i], a.dto.lo, a.dto.hi);
      }
      if constexpr (TAIL) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const bool in = 4 * (i0 + i) + q < left;
          dv[i] = in ? dv[i] : 0.f;
          xv[i] = in ? xv[i] : 0.f;
        }
      }
      const float4* row = bc4[buf] + 4 * i0 * (ROW / 4) + q;
      float yv[OUT ? NG : 1], uv[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        uv[i] = dv[i] * xv[i];
        if constexpr (OUT) yv[i] = Dv * xv[i];
        else dsum += dv[i];
      }
      // Four states of one token make a unit. A unit's B and C are read two
      // units ahead and its decays computed one ahead, so neither LDS nor the
      // exp2 is waited for; the scheduling barrier keeps the compiler from
      // moving them back to their use.
      float4 bq[3], cq[OUT ? 3 : 1];
      float dec[2][4], acc[4];
      auto read = [&](int w) {
        const int at = (w / VU) * (ROW / 4) + 4 * (w % VU);
        bq[w % 3] = row[at];
        if constexpr (OUT) cq[w % 3] = row[at + NP / 4];
      };
      auto decay = [&](int w) {
        const int tk = w / VU, v = w % VU;
        const float d = quad_bcast_of(tk % 4, dv[tk / 4]);
#pragma unroll
        for (int k = 0; k < 4; ++k) dec[w % 2][k] = __builtin_amdgcn_exp2f(d * A2[4 * v + k]);
      };
      read(0);
      if (4 * NG * VU > 1) read(1);
      decay(0);
#pragma unroll
      for (int w = 0; w < 4 * NG * VU; ++w) {
        const int tk = w / VU, v = w % VU, i = tk / 4, j = tk % 4;
        if (w + 2 < 4 * NG * VU) read(w + 2);
        if (w + 1 < 4 * NG * VU) decay(w + 1);
        const float u = quad_bcast_of(j, uv[i]);
        const float4 bv = bq[w % 3], cv = cq[OUT ? w % 3 : 0];
        const float bb[4] = {bv.x, bv.y, bv.z, bv.w}, cc[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int s = 4 * v + k;
          h[s] = fmaf(dec[w % 2][k], h[s], u * bb[k]);
          if constexpr (OUT) acc[j] = s == 0 ? h[s] * cc[k] : fmaf(h[s], cc[k], acc[j]);
        }
        if (OUT && j == 3 && v == VU - 1) {
          // sum over the quad, transposed: lane q ends with token q's
          const float k0 = o1 ? acc[1] : acc[0], m0 = o1 ? acc[0] : acc[1];
          const float k1 = o1 ? acc[3] : acc[2], m1 = o1 ? acc[2] : acc[3];
          const float v0 = k0 + quad_xor<1>(m0), v1 = k1 + quad_xor<1>(m1);
          yv[i] += (o2 ? v1 : v0) + quad_xor<2>(o2 ? v0 : v1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // (the states are final here: without a use of them the compiler would
      // move the whole computation behind the next branch, out of its order)
#pragma unroll
      for (int s = 0; s < SPL; ++s) asm volatile("" : "+v"(h[s]));
      // the next tile's loads are all that is in flight here; y's stores, below,
      // then have the whole of the next tile to land
      if constexpr (MORE) stage(left - TT, buf ^ 1);
      if constexpr (OUT) {
        if (a.z != nullptr) {
          const RX* zq = zl[buf] + at0;
#pragma unroll
          for (int i = 0; i < NG; ++i) yv[i] *= silu_f32(Elem<TIO>::f32(zq[4 * i * kPitch]));
        }
        // y takes the places of x, which no other lane reads
#pragma unroll
        for (int i = 0; i < NG; ++i) xq[4 * i * kPitch] = Elem<TIO>::bits(yv[i]);
      }
    };

    auto take_turns = [&] {
      // The older of two waves on a SIMD would otherwise run at its own pace
      // and leave the other to finish alone, at half of the SIMD's rate. They
      // take turns instead, by the clock: every 2^15 cycles (8 x 2048 tokens,
      // 4096 channels, when it took 276: no turns 297 us, a turn a tile 283, 2^19
      // 295; short runs want them no longer: packed 143, 143, 142, 150 us).
      if (((uint32_t)(__builtin_amdgcn_s_memtime() >> 15) ^ wave_slot) & 1) __builtin_amdgcn_s_setprio(2);
      else __builtin_amdgcn_s_setprio(0);
    };
    auto write_y = [&] {
      if constexpr (OUT) {
        // each lane writes PK channels of a token of its wave's 16
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const int ytk = (tid & 63) * PK / 16, yc0 = (tid / 64) * 16 + (tid & 63) * PK % 16;
        const Pack<TIO, PK> out = *reinterpret_cast<const Pack<TIO, PK>*>(xl[buf] + ytk * kPitch + yc0);
        const int yn = a.epg - ch0 - yc0;
        if (ytk < left && yn > 0) {
          RX* to = reinterpret_cast<RX*>(reinterpret_cast<char*>(yb) + yr + (ytk * ys + (uint32_t)((ch0 + yc0) * sizeof(TIO))));
          if (WHOLE && (!MOVED || yc0 >= shared)) {
            __builtin_memcpy(to, &out, sizeof(out));
          } else {
#pragma unroll
            for (int k = 0; k < PK; ++k)
              if (k < yn && yc0 + k >= shared) to[k] = out.v[k];
          }
        }
        advance(yr, TT * ys);
      }
    };

    // (the last tile stands by itself: the others fetch and stage without asking)
    const std::integral_constant<int, GR> tile{};
    const std::true_type yes{};
    const std::false_type no{};
    fetch(left);
    buf ^= 1;
    stage(left, buf);
    __syncthreads();
    for (; left > TT; left -= TT) {
      take_turns();
      fetch(left - TT);
      groups(tile, no, yes, 0);
      write_y();
      __syncthreads();
      buf ^= 1;
    }
    take_turns();
    if (left == TT) {
      groups(tile, no, no, 0);
    } else {
      for (int i = 0; 4 * i < left; ++i) groups(std::integral_constant<int, 1>{}, yes, no, i);
    }
    write_y();
  };

  auto walk = [&](int64_t r0, int64_t r1) {
    const std::true_type yes{};
    const std::false_type no{};
    if (!whole) walk_as(no, no, r0, r1);
    else if (OUT && shared != 0) walk_as(yes, yes, r0, r1);
    else walk_as(yes, no, r0, r1);
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
    int64_t r0;
    if (!passing_run(first, last, s0, s1, r0)) return;
    const bool starts = first >= s0;
    if (starts) {
      load_state(a.init, row);
      if (a.init_copy != nullptr) ws_store(a.init_copy);
    } else {
      load_state(nullptr, 0);
    }
    walk(r0, s1);
    ws_store(a.ends);
    dsum += quad_xor<1>(dsum);
    dsum += quad_xor<2>(dsum);
    if (mine && q == 0) a.dsums[(b * a.cut.n + seg) * a.E + e] = dsum;
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
        const float ds = a.dsums[(b * a.cut.n + j) * a.E + e];
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
    auto begin = [&](int64_t row, int64_t piece, bool goes_on) {
      if (goes_on && a.init_copy != nullptr) {
        // the final state of this sequence may be written over its initial
        // state by another workgroup of this launch: take the kept copy
#pragma unroll
        for (int i = 0; i < SPL / 4; ++i) {
          const float4 v = *ws_at(a.init_copy, piece, i);
          h[4 * i] = v.x, h[4 * i + 1] = v.y, h[4 * i + 2] = v.z, h[4 * i + 3] = v.w;
        }
      } else {
        load_state(a.init, row);
      }
    };
    // batched: one sequence, the batch row's
    const bool packed = a.cu != nullptr;
    int64_t row = packed ? seq_of(a.cu, a.nseq, a.L, s0) : b;
    const int64_t rows = packed ? a.nseq : b + 1;
    for (int64_t pos = s0; pos < s1 && row < rows; ++row) {
      const int64_t first = packed ? seq_offset(a.cu, row, a.L) : 0;
      const int64_t last = packed ? seq_offset(a.cu, row + 1, a.L) : a.L;
      int64_t r0, r1;
      if (first >= s1) break;
      if (!next_run(first, last, pos, s1, r0, r1)) continue;
      if (first < s0) enter(first / a.cut.len); else begin(row, first / a.cut.len, last > s1);
      walk(r0, r1);
      if (last <= s1 && a.final_state != nullptr) store_state(a.final_state, row);
      pos = r1;
    }
    if (packed && a.final_state != nullptr) {
      // sequences without tokens keep their state: this segment's share of them
      const int lane = tid & 63;
      for (int64_t r = (int64_t)blockIdx.y * 64; r < a.nseq; r += (int64_t)gridDim.y * 64) {
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

template <typename TIO, typename TDT, int NP>
hipError_t launch_np(const SelectiveArgs& a, int64_t batch, hipStream_t s) {
  const unsigned tiles = (unsigned)(a.tiles * (a.E / a.epg));
  const int segments = (a.cut.n + a.cut.pieces - 1) / a.cut.pieces;
  if (segments > 1) {
    selective_scan_kernel<TIO, TDT, NP, false>
        <<<dim3(tiles, (unsigned)((segments - 1) * a.cut.pieces), (unsigned)batch), kThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  selective_scan_kernel<TIO, TDT, NP, true><<<dim3(tiles, (unsigned)segments, (unsigned)batch), kThreads, 0, s>>>(a);
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

SelectiveCut selective_scan_cut(int64_t batch, int64_t L, int64_t E, int64_t G, int64_t nseq) {
  const int64_t tiles = (E / G + kChannels - 1) / kChannels * G;
  const int64_t waves = tiles * 4 * batch;
  // As many segments as two waves a SIMD allow (with more than 128 states the
  // output walk's registers leave one, and its segments run in two rounds; the
  // rule does not tell these apart): one walk takes the same time
  // for 1025 waves as for 2048, and for 1 as for 1024. 4096 tokens of 4096
  // channels, batch 2 (512 waves): 392 us in one walk, 224 in four segments;
  // batch 4: 395 and 371 in two; batch 6: 534 and, as two, 619.
  const int64_t full = 2048;
  const int64_t want = 2 * waves > full ? 1 : full / waves;
  int64_t len = (L + want - 1) / want;
  if (nseq > 0) {
    // a run's start is waited for: about four runs to a segment, as far as
    // eight times the segments go (they bound the workspace)
    const int64_t runs = 4 * L / nseq, least = (len + 7) / 8;
    if (runs < len) len = runs > least ? runs : least;
  }
  if (len < 64) len = 64;
  if (len >= L) return SelectiveCut{1, L, 1};
  // The first walk needs half the registers of the second, so it has room for
  // more waves: a quarter of a segment each (16384 tokens of 4096 channels 462
  // -> 434 us). Packed sequences keep whole segments: every piece may end in
  // the middle of a run (37 sequences in 8197 tokens 139 us, in two pieces 150).
  // Narrow layers of long prompts have pieces by the hundred, and the fold over
  // them is a load's latency each: 32768 tokens of 64 channels (1024 pieces) 309
  // us, of 512 (256 pieces) 180.
  int64_t pieces = nseq > 0 ? 1 : 4;
  int64_t unit = 32 * pieces;  // whole tiles
  len = (len + unit - 1) / unit * unit;
  while (L > len * 16384) len *= 2;  // pieces along grid.y
  if (len >= L) return SelectiveCut{1, L, 1};
  len /= pieces;
  return SelectiveCut{(int)((L + len - 1) / len), len, (int)pieces};
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
