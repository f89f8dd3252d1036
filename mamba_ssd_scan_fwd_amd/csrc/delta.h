// Internal declarations of the gated delta rule and of the norm of heads. Not
// part of the public ABI.
#pragma once

#include "selective.h"

namespace ssd {

// ---- gated delta rule ----------------------------------------------------------
constexpr int kDeltaMaxDim = 256;  // P, N

struct DeltaArgs {
  const void *x, *dt, *beta, *B, *C;
  const float *A, *init;           // init nullable
  void* y;
  float* final_state;              // nullable
  Stride xs, ds, es, bs, cs;       // of x, dt, beta, B, C
  int64_t batch, L;                // packed: 1 and the tokens of the stream
  int H, P, N, G;
  const int32_t* cu;               // packed: sequence offsets [nseq + 1], else nullptr
  int64_t nseq;
  DtOpts dto;
  int sigmoid;
  float scale;
  // in blocks (set at launch)
  char* ws;                        // workspace: the blocks' records
  int64_t upto;                    // packed, not 0: sequences of more tokens go in blocks, the others token after token
  int32_t* longs;                  // workspace, then: which those are, in order, -1 behind the last; else nullptr
  int64_t seg;                     // tokens of a segment; 0: sequences in one piece
  float *ends, *enter;             // workspace: segments' ends and entering states
  int64_t seqs() const { return nseq > 0 ? nseq : batch; }
};
// The recurrence token after token. Whether its launch can be counted (grid_fits):
// a call's plan asks, here and below, before anything is launched.
bool delta_walk_fits(const DeltaArgs& a);
hipError_t launch_delta_walk(const DeltaArgs& a, int io, int dt, hipStream_t s);

// In blocks of kDeltaBlock tokens. A sequence's blocks begin with it; the blocks
// of all sequences lie behind one another in slots, sequence s of a packed
// stream from slot offset / kDeltaBlock + s on (so that nobody has to sum the
// sequences' block counts; a few slots stay empty).
constexpr int kDeltaBlock = 64;
// Sequences that go in blocks: all, or as many as can have more than a.upto tokens.
inline int64_t delta_seqs_in_blocks(const DeltaArgs& a) { return a.upto > 0 ? a.L / (a.upto + 1) : a.seqs(); }
// (Segments, of several blocks, have slots of the same kind.)
inline int64_t delta_slots(const DeltaArgs& a, int64_t unit = kDeltaBlock) {
  return a.nseq > 0 ? a.L / unit + delta_seqs_in_blocks(a) : a.batch * ((a.L + unit - 1) / unit);
}
// Whether any of the call goes in blocks; sets a.upto.
bool delta_blocks_apply(DeltaArgs& a, int io);
int64_t delta_blocks_workspace(DeltaArgs& a, int io);  // in bytes; sets a.seg
// Whether every launch of the form in blocks can be counted, by whichever walk the
// rows' addresses and strides will choose. (a.seg is set.)
bool delta_blocks_fit(const DeltaArgs& a, int io);
hipError_t launch_delta_blocks(const DeltaArgs& a, int io, int dt, hipStream_t s);
// The kernels of the form in blocks: their workgroups, and launches.
int64_t delta_solve_groups(const DeltaArgs& a);
hipError_t launch_delta_solve(const DeltaArgs& a, int io, int dt, hipStream_t s);
bool delta_chain_applies(const DeltaArgs& a, int io);
int64_t delta_chain_groups(const DeltaArgs& a, int pass);
hipError_t launch_delta_chain(const DeltaArgs& a, int pass, hipStream_t s);
int64_t delta_join_groups(const DeltaArgs& a);
hipError_t launch_delta_join(const DeltaArgs& a, hipStream_t s);
// What the walks over blocks divide among their workgroups: rows of the state (with
// the unit states' in pass 1), and sequences or segments.
inline int delta_rows(const DeltaArgs& a, int pass) { return pass == 1 ? a.P + a.N : a.P; }
inline int64_t delta_pieces(const DeltaArgs& a) { return a.seg != 0 ? delta_slots(a, a.seg) : delta_seqs_in_blocks(a); }

struct DeltaStepArgs {
  const void *x, *dt, *beta, *B, *C;  // one token per row
  const float* A;
  float* state;                       // [nslots, H, P, N]
  const int32_t* slots;               // [batch], nullable: row b uses slot b
  int64_t nslots;
  void* y;
  int64_t xs, ds, es, bs, cs;         // elements from one row to the next
  int64_t batch;
  int H, P, N, G;
  DtOpts dto;
  int sigmoid;
  float scale;
  bool stream;                        // states past the memory-side cache (set at launch)
};
hipError_t launch_delta_step(const DeltaStepArgs& a, int io, int dt, hipStream_t s);

// ---- norm of heads -------------------------------------------------------------
constexpr int kHeadNormMaxDim = 512;

struct HeadNormArgs {
  const void* in[2];               // q, k (nullable with no heads)
  const float* w[2];               // [D], nullable
  void* out[2];
  Stride st[2];
  int heads[2];
  int64_t batch, rows;
  int D, R;                        // channels of a head, of them rotated
  const int32_t* pos;              // [batch, rows]
  const float* freq;               // [R / 2]
  int l2, pairs;
  float eps;
  int per;                         // heads a wave takes of a token (set at launch)
  bool stream;                     // read past the memory-side cache (set at launch)
};
hipError_t launch_head_norm(const HeadNormArgs& a, int io, hipStream_t s);

// Whether a launch's threads can be counted (in 32 bits).
inline bool grid_fits(int64_t groups, int threads) { return groups < (int64_t(1) << 32) / threads; }

#ifdef __HIPCC__
// Sum over teams of T lanes (a power of two, aligned), in all of them: DPP
// within 16 lanes, then exchanges of rows and of halves of the wave. All lanes
// take part.
template <int CTRL> __device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int T> __device__ __forceinline__ float team_sum(float v) {
  static_assert(T >= 1 && T <= 64, "lanes of a team");
  if constexpr (T >= 2) v += dpp_f32<0xB1>(v);   // quad: lane ^ 1
  if constexpr (T >= 4) v += dpp_f32<0x4E>(v);   // quad: lane ^ 2
  if constexpr (T >= 8) v += dpp_f32<0x141>(v);  // mirrored in 8
  if constexpr (T >= 16) v += dpp_f32<0x140>(v); // mirrored in 16
  if constexpr (T >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (T >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// log2 of a token's decay, finite (a NaN stays one), and its beta.
__device__ __forceinline__ float delta_log2_decay(float dt, float bias, float A, const DtOpts& o) {
  return clamped(step_size(dt, bias, o) * log2_decay(A), -FLT_MAX, FLT_MAX);
}
__device__ __forceinline__ float delta_beta(float v, int sigmoid) {
  return sigmoid ? __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e)) : v;
}
#endif

}  // namespace ssd
