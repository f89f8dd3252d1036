// Internal declarations of the layer operators around the scan: selective
// scan and step, short convolution and its step, group norm. Not part of the
// public ABI.
#pragma once

#include <cfloat>
#include <type_traits>

#include "packed_runs.h"
#include "ssd_internal.h"

namespace ssd {

// Elements from one token to the next and from one batch row to the next.
struct Stride {
  int64_t token, batch;
};

// ---- selective scan ----------------------------------------------------------
// The cut of the time axis: n pieces of len tokens, `pieces` of them to a
// segment of the second walk. n = 1: one walk over all tokens.
struct SelectiveCut {
  int n;
  int64_t len;
  int pieces;
};
SelectiveCut selective_scan_cut(int64_t batch, int64_t L, int64_t E, int64_t G, int64_t nseq);

struct SelectiveArgs {
  const void *x, *dt, *B, *C, *z;  // z nullable
  const float *A, *D, *init;       // D, init nullable
  void* y;
  float* final_state;              // nullable
  Stride xs, ds, bs, cs, zs;
  int64_t L;                       // tokens per batch row, or of the packed stream
  int E, N, G;
  const int32_t* cu;               // packed: sequence offsets [nseq + 1], else nullptr
  int64_t nseq;
  DtOpts dto;
  SelectiveCut cut;
  // the workspace when cut.n > 1
  float* ends;       // [batch, cut.n, E, padded N]: the pieces' end states
  float* dsums;      // [batch, cut.n, E]: their sums of dt
  float* init_copy;  // as ends: initial states that the final states overwrite, else nullptr
  int epg, tiles;    // channels per group, workgroups per group (set at launch)
};
// States per channel as the kernels hold them: the next of 16, 32, .. 256.
inline int selective_padded_states(int64_t N) {
  int np = 16;
  while (np < N) np *= 2;
  return np;
}
hipError_t launch_selective_scan(const SelectiveArgs& a, int io, int dt, int64_t batch, hipStream_t s);

// The recurrence at one token, states in slots.
struct SelectiveStepArgs {
  const void *x, *dt, *B, *C, *z;  // z nullable; one token per row
  const float *A, *D;              // D nullable
  float* state;                    // [nslots, E, N]
  const int32_t* slots;            // [batch], nullable: row b uses slot b
  int64_t nslots;
  void* y;
  int64_t xs, ds, bs, cs, zs;      // elements from one row to the next
  int64_t batch;
  int E, N, G;
  DtOpts dto;
  bool stream;                     // states past the memory-side cache (set at launch)
};
hipError_t launch_selective_step(const SelectiveStepArgs& a, int io, int dt, hipStream_t s);

// ---- short causal convolution ------------------------------------------------
// Up to three dense outputs share the channels in order (x | B | C); a plain
// convolution has one.
struct Conv1dArgs {
  const void* x;
  const float *w, *bias;           // [CH, K], [CH] (nullable)
  const float* state_in;           // [batch or nseq, CH, K - 1], nullable
  float* state_out;                // likewise, nullable
  void* out[3];
  int width[3];                    // channels of each output
  Stride xs;
  int64_t L;
  int CH;
  int silu;
  const int32_t* cu;               // packed: sequence offsets [nseq + 1], else nullptr
  int64_t nseq;
  int tile;                        // tokens per workgroup (set at launch)
};
hipError_t launch_conv1d(const Conv1dArgs& a, int io, int K, int64_t batch, hipStream_t s);

struct Conv1dStepArgs {
  const void* x;
  const float *w, *bias;
  float* state;                    // [nslots, CH, K - 1]
  const int32_t* slots;            // [batch], nullable: row b uses slot b
  int64_t nslots;
  void* out[3];
  int width[3];
  int64_t xs;                      // elements from one row to the next
  int64_t batch;
  int CH;
  int silu;
};
hipError_t launch_conv1d_step(const Conv1dStepArgs& a, int io, int K, hipStream_t s);

// ---- group norm ----------------------------------------------------------------
struct GroupNormArgs {
  const void *x, *z;               // z nullable
  const float *w, *bias;           // [C], nullable
  void* out;                       // dense [batch, rows, C]
  Stride xs, zs;                   // "token" = from one row to the next
  int64_t batch, rows;
  int C, G;
  float eps;
  int center, gate_first, silu;
  bool stream;                     // read past the memory-side cache (set at launch)
};
constexpr int64_t kGroupNormMaxGroup = 16384;  // channels per group
hipError_t launch_group_norm(const GroupNormArgs& a, int io, hipStream_t s);

constexpr int64_t kMemorySideCache = int64_t(256) << 20;  // bytes, on MI355X

#ifdef __HIPCC__
// ---- device helpers --------------------------------------------------------------

constexpr float kLog2e = 1.44269504088896340736f;

// z * sigmoid(z), with the hardware's exp2 and reciprocal (about 1 ulp each)
__device__ __forceinline__ float silu_f32(float z) {
  return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// log(1 + e^v) from the hardware's log2 and exp2. w = 1 + e is rounded; what
// the rounding lost, c, is added to first order as c / w, so the result keeps its
// relative accuracy where e is small (dt near 0.001 is the usual range). v
// itself above 20, as dt_pre does.
__device__ __forceinline__ float softplus_f32(float v) {
  const float e = __builtin_amdgcn_exp2f(v * kLog2e);
  const float w = 1.f + e;
  const float c = e - (w - 1.f);
  const float r = fmaf(__builtin_amdgcn_logf(w), 0.69314718055994530942f, c * __builtin_amdgcn_rcpf(w));
  return v > 20.f ? v : r;
}
// v within [lo, hi]; a NaN stays one (fminf and fmaxf would make it lo).
__device__ __forceinline__ float clamped(float v, float lo, float hi) {
  v = v < lo ? lo : v;
  return v > hi ? hi : v;
}
// A decay for exp2, finite (log2(e) times the lowest values is not): a step of
// zero then leaves the state as it is.
__device__ __forceinline__ float log2_decay(float A) { return clamped(A * kLog2e, -FLT_MAX, FLT_MAX); }
__device__ __forceinline__ float step_size(float v, float bias, const DtOpts& o) {
  v += bias;
  if (o.softplus) v = softplus_f32(v);
  if (o.clamp) v = clamped(v, o.lo, o.hi);
  return v;
}

// fp32 to bf16, to nearest even, by the hardware's conversion
__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// One element as it lies in memory, kept so until it is used.
template <typename T> struct Elem;
template <> struct Elem<float> {
  using raw = float;
  static __device__ __forceinline__ float f32(float v) { return v; }
  static __device__ __forceinline__ float bits(float v) { return v; }
};
template <> struct Elem<__hip_bfloat16> {
  using raw = uint16_t;
  static __device__ __forceinline__ float f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t bits(float v) { return bf16_bits(v); }
};

// V consecutive elements (a power of two).
template <typename T, int V> struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Pack {
  typename Elem<T>::raw v[V];
};
// A pack from or to memory that is aligned to its elements only, in accesses of
// up to 16 bytes (the hardware takes them at any address). PART: n of its V
// elements are there; the first stands in for the others.
template <typename T, int V, bool PART = false>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p, int n = V) {
  Pack<T, V> r;
  if (!PART || n >= V) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
    using R = typename Elem<T>::raw;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = reinterpret_cast<const R*>(p)[i < n ? i : 0];
  }
  return r;
}
template <typename T, int V, bool PART = false>
__device__ __forceinline__ void store_pack(T* p, const float (&f)[V], int n = V) {
  using R = typename Elem<T>::raw;
  if (!PART || n >= V) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = Elem<T>::bits(f[i]);
    __builtin_memcpy(p, &r, sizeof(r));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) reinterpret_cast<R*>(p)[i] = Elem<T>::bits(f[i]);
  }
}

// The same for packs that are not expected to be used again soon: past the
// caches (non-temporal).
typedef uint32_t u32x4_unaligned __attribute__((ext_vector_type(4), aligned(2)));
template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_stream(const T* p) {
  static_assert(sizeof(Pack<T, V>) == 16, "one 16-byte access");
  const u32x4_unaligned v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_unaligned*>(p));
  return __builtin_bit_cast(Pack<T, V>, v);
}
template <typename T, int V> __device__ __forceinline__ void store_stream(T* p, const float (&f)[V]) {
  Pack<T, V> r;
  static_assert(sizeof(r) == 16, "one 16-byte access");
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = Elem<T>::bits(f[i]);
  u32x4_unaligned v;
  __builtin_memcpy(&v, &r, 16);
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4_unaligned*>(p));
}

// Offset i of a packed batch, clamped into [0, T].
__device__ __forceinline__ int64_t seq_offset(const int32_t* cu, int64_t i, int64_t T) {
  const int64_t v = cu[i];
  return v < 0 ? 0 : v > T ? T : v;
}
// Largest s in [0, S] with cu[s] <= t (0 if there is none), by the whole
// wave: 64 candidates a step.
__device__ __forceinline__ int64_t seq_of(const int32_t* cu, int64_t S, int64_t T, int64_t t) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, n = S + 1;  // candidates lo .. lo + n - 1
  while (n > 1) {
    const int64_t step = (n + 63) / 64;
    const int64_t i = lo + lane * step;
    const bool le = lane * step < n && seq_offset(cu, i < S ? i : S, T) <= t;
    const uint64_t m = __ballot(le);
    const int k = m == 0 ? 0 : 63 - __builtin_clzll(m);  // the last candidate that is <= t
    const int64_t left = n - k * step;
    lo += k * step;
    n = left < step ? left : step;
  }
  return lo;
}

// Whether an earlier row of a batch names the same slot (its slot is then
// that row's alone): bit k for row row0 + k. Called by all threads of a
// workgroup; R <= 32.
template <int R, int THREADS>
__device__ __forceinline__ uint32_t repeated_slots(const int32_t* slots, int64_t row0, int64_t batch) {
  int32_t want[R];
#pragma unroll
  for (int k = 0; k < R; ++k) want[k] = row0 + k < batch ? slots[row0 + k] : -1;
  const int64_t end = row0 + R - 1 < batch ? row0 + R - 1 : batch - 1;  // the last row needs those before it
  uint32_t hit = 0;
  for (int64_t i = threadIdx.x; i < end; i += THREADS) {
    const int32_t v = slots[i];
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (i < row0 + k && v == want[k]) hit |= 1u << k;
  }
  __shared__ uint32_t all;
  if (threadIdx.x == 0) all = 0;
  __syncthreads();
  if (hit != 0) atomicOr(&all, hit);
  __syncthreads();
  return all;
}
#endif

}  // namespace ssd
