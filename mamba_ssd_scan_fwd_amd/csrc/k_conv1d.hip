// The short causal convolution for any channel count, strided rows and packed
// sequences, and its single-token step.
//     y[t][ch] = act(bias[ch] + sum_{k<K} w[ch][k] in[t - (K-1) + k][ch])
// where in[] before a sequence's first token is its carried state.
//
// Prompts: each thread owns V consecutive channels (16 bytes of a row, at any
// address; one where outputs share such a pack) and walks a tile of tokens with the K - 1 inputs before
// it in registers, kU tokens' loads in flight ahead of the ones in use. Each
// input is read once, plus K - 1 rows at the start of a tile, and the work
// per element is far below what the memory traffic costs. Eight bf16 channels and
// four tokens ahead: 8 x 2048 x 4096 47 us (5.7 TB/s; a copy of the same bytes
// takes 50); eight tokens ahead leave two waves a SIMD (55 -> 51 us, with scalar
// weight loads). 8197 packed tokens of 4352 channels: 34 us, 4.2 TB/s, the
// start of each run (offsets, carried state, first rows) being waited for.
//
// Packed sequences cut the packed stream into the same tiles: a tile is a
// list of runs, one for each sequence with tokens in it, and a run starts
// from its own sequence's inputs or carried state.
#include "selective.h"

namespace ssd {
namespace {

constexpr int kThreads = 64;
constexpr int kU = 4;  // tokens whose loads are issued together

// The output that holds channel ch: its base for row 0 and its row length.
// (V channels never straddle outputs: the widths are multiples of V.)
template <typename TIO>
__device__ __forceinline__ TIO* output_of(void* const (&out)[3], const int (&width)[3], int ch, int& stride) {
  int o = 0;
  if (ch >= width[0]) {
    ch -= width[0];
    o = 1;
    if (ch >= width[1]) {
      ch -= width[1];
      o = 2;
    }
  }
  stride = width[o];
  return static_cast<TIO*>(out[o]) + ch;
}

// STREAM: the inputs are read past the memory-side cache.
template <typename TIO, int K, int V, bool STREAM>
__global__ __launch_bounds__(kThreads) void conv1d_kernel(const Conv1dArgs a) {
  constexpr int H = K > 1 ? K - 1 : 1;
  const int ch = V * (blockIdx.x * kThreads + threadIdx.x);
  const bool mine = ch < a.CH;
  // (the last pack ends with the channels; where it overlaps the one before,
  // both write the same values)
  const int cc = !mine ? 0 : ch + V <= a.CH ? ch : a.CH - V;
  const int64_t b = blockIdx.z;
  const int64_t t0 = (int64_t)blockIdx.y * a.tile;
  const int64_t t1 = t0 + a.tile < a.L ? t0 + a.tile : a.L;
  const TIO* in = static_cast<const TIO*>(a.x) + b * a.xs.batch + cc;
  int os;
  TIO* out = output_of<TIO>(a.out, a.width, cc, os);
  out += b * a.L * os;

  // The V channels' weights, and their carried states, are blocks of K V and
  // (K - 1) V consecutive floats, channel by channel, taken V at a time.
  float w[K][V], bias[V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Pack<float, V> p = load_pack<float, V>(a.w + cc * K + k * V);
#pragma unroll
    for (int v = 0; v < V; ++v) w[(k * V + v) % K][(k * V + v) / K] = p.v[v];
  }
  {
    const Pack<float, V> p = load_pack<float, V>(a.bias != nullptr ? a.bias + cc : a.w);
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = a.bias != nullptr ? p.v[v] : 0.f;
  }
  // the K - 1 inputs that row's carried state holds (zeros without one)
  auto carried = [&](int64_t row, float (&f)[H][V]) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      Pack<float, V> p = {};
      if (a.state_in != nullptr) p = load_pack<float, V>(a.state_in + (row * a.CH + cc) * H + j * V);
#pragma unroll
      for (int v = 0; v < V; ++v) f[(j * V + v) % H][(j * V + v) / H] = p.v[v];
    }
  };
  auto keep = [&](int64_t row, const float (&hist)[H][V]) {
    if (!mine) return;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      float f[V];
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = hist[(j * V + v) % H][(j * V + v) / H];
      store_pack<float, V>(a.state_out + (row * a.CH + cc) * H + j * V, f);
    }
  };

  // V inputs of token t
  auto input = [&](int64_t t) {
    const TIO* p = in + t * a.xs.token;
    if constexpr (STREAM) return load_stream<TIO, V>(p);
    else return load_pack<TIO, V>(p);
  };

  // Tokens [r0, r1) of the sequence `row` that began at `first`.
  auto walk = [&](int64_t row, int64_t first, int64_t r0, int64_t r1, bool ends) {
    // (all loads first: the tokens before r0, or the run's first in their place)
    Pack<TIO, V> nxt[kU], before[H];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      nxt[u] = input(r0 + u < r1 ? r0 + u : r1 - 1);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int64_t t = r0 - (K - 1) + j;
      before[j] = input(t >= first ? t : r0);
    }
    float hist[H][V];
    // of the carried state, inputs r0 - first .. K - 2 still lie before r0
    const int64_t d = r0 - first;
    if (d < K - 1) {
      float old[H][V];
      carried(row, old);
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          hist[j][v] = Elem<TIO>::f32(before[j].v[v]);
#pragma unroll
          for (int i = j; i < K - 1; ++i)
            if (j + d == i) hist[j][v] = old[i][v];
        }
    } else {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) hist[j][v] = Elem<TIO>::f32(before[j].v[v]);
    }
    for (int64_t tb = r0; tb < r1; tb += kU) {
      Pack<TIO, V> cur[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) cur[u] = nxt[u];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t t = tb + kU + u;
        nxt[u] = input(t < r1 ? t : r1 - 1);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (tb + u < r1) {
          float z[V];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float now = Elem<TIO>::f32(cur[u].v[v]);
            z[v] = bias[v];
#pragma unroll
            for (int k = 0; k < K - 1; ++k) z[v] = fmaf(w[k][v], hist[k][v], z[v]);
            z[v] = fmaf(w[K - 1][v], now, z[v]);
            if (a.silu) z[v] = silu_f32(z[v]);
#pragma unroll
            for (int k = 0; k + 1 < K - 1; ++k) hist[k][v] = hist[k + 1][v];
            hist[H - 1][v] = now;
          }
          if (mine) store_pack<TIO, V>(out + (tb + u) * os, z);
        }
      }
    }
    if (ends && a.state_out != nullptr) keep(row, hist);
  };

  if (a.cu == nullptr) {
    walk(b, 0, t0, t1, t1 == a.L);
    return;
  }
  int64_t row = seq_of(a.cu, a.nseq, a.L, t0), pos = t0;
  while (pos < t1 && row < a.nseq) {
    const int64_t first = seq_offset(a.cu, row, a.L), last = seq_offset(a.cu, row + 1, a.L);
    int64_t r0, r1;
    if (first >= t1) break;
    if (next_run(first, last, pos, t1, r0, r1)) {
      walk(row, first, r0, r1, last <= t1);
      pos = r1;
    }
    ++row;
  }
  // sequences without tokens keep their state: this tile's share of them
  if (a.state_out != nullptr) {
    const int lane = threadIdx.x & 63;
    for (int64_t r = (int64_t)blockIdx.y * 64; r < a.nseq; r += (int64_t)gridDim.y * 64) {
      const int64_t i = r + lane < a.nseq ? r + lane : a.nseq - 1;
      uint64_t empty = __ballot(r + lane < a.nseq && seq_offset(a.cu, i + 1, a.L) <= seq_offset(a.cu, i, a.L));
      while (empty != 0) {
        const int k = __builtin_ctzll(empty);
        empty &= empty - 1;
        float hist[H][V];
        carried(r + k, hist);
        keep(r + k, hist);
      }
    }
  }
}

// One token per row: V channels to a thread, their K - 1 old inputs read and
// written as one block of V (K - 1) floats. Rows without a slot of their own
// (negative, behind the pool, or named by an earlier row) are padding. 256 rows
// of 8192 channels: 13.0 us, 4.5 TB/s (rows a workgroup: 1 13.5, 2 13.0, 4 13.6, 8
// 14.3); one row of 4352 channels 2.8 us.
constexpr int kStepThreads = 256;

// PART: the last thread of a row has fewer than V channels.
template <typename TIO, int K, int V, int R, bool PART>
__global__ __launch_bounds__(kStepThreads) void conv1d_step_kernel(const Conv1dStepArgs a) {
  constexpr int H = K > 1 ? K - 1 : 1;
  const int ch = V * (blockIdx.x * kStepThreads + threadIdx.x);
  const bool mine = ch < a.CH;
  const int cc = mine ? ch : 0;
  const int n = a.CH - cc < V ? a.CH - cc : V;  // channels there: fewer at the end of a row
  // V of the n K weights or n H inputs of a lane's channels, from the j V-th on
  auto block = [&](const float* p, int per, int j) {
    const int there = n * per - j * V;
    return load_pack<float, V, PART>(PART && there <= 0 ? p : p + j * V, there);
  };
  const int64_t row0 = (int64_t)blockIdx.y * R;
  int os;
  TIO* out = output_of<TIO>(a.out, a.width, cc, os);

  Pack<float, V> w[K], bias;
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = block(a.w + cc * K, K, k);
  bias = load_pack<float, V, PART>(a.bias != nullptr ? a.bias + cc : a.w + cc * K, n);
  Pack<float, V> old[R][H];
  Pack<TIO, V> xv[R];
  int64_t slot[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = row0 + r < a.batch ? row0 + r : a.batch - 1;
    slot[r] = a.slots != nullptr ? a.slots[row] : row;
    if (row0 + r >= a.batch || slot[r] < 0 || slot[r] >= a.nslots) slot[r] = -1;
    const int64_t from = slot[r] < 0 ? 0 : slot[r];
    if constexpr (K > 1) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        old[r][j] = block(a.state + (from * a.CH + cc) * H, H, j);
    }
    xv[r] = load_pack<TIO, V, PART>(static_cast<const TIO*>(a.x) + row * a.xs + cc, n);
  }
  if (a.slots != nullptr) {
    const uint32_t again = repeated_slots<R, kStepThreads>(a.slots, row0, a.batch);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (again >> r & 1) slot[r] = -1;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (slot[r] < 0 || !mine) continue;
    float z[V], kept[H][V];  // element i of a block is channel i / H, input i % H
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float now = Elem<TIO>::f32(xv[r].v[v]);
      z[v] = a.bias != nullptr ? bias.v[v] : 0.f;
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {
        const int i = v * H + k, j = v * K + k;
        z[v] = fmaf(w[j / V].v[j % V], old[r][i / V].v[i % V], z[v]);
        const int n = v * H + k + 1;
        kept[i / V][i % V] = k + 1 < K - 1 ? old[r][(k + 1 < K - 1 ? n : i) / V].v[(k + 1 < K - 1 ? n : i) % V] : now;
      }
      const int j = v * K + K - 1;
      z[v] = fmaf(w[j / V].v[j % V], now, z[v]);
      if (a.silu) z[v] = silu_f32(z[v]);
    }
    if constexpr (K > 1) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        store_pack<float, V, PART>(a.state + (slot[r] * a.CH + cc) * H + j * V, kept[j], n * H - j * V);
    }
    store_pack<TIO, V, PART>(out + (row0 + r) * os, z, n);
  }
}

// Whether no V consecutive channels from a multiple of V on, nor the last V,
// belong to two outputs.
template <int V, typename Args> bool whole_packs(const Args& a) {
  int last = 2;
  while (last > 0 && a.width[last] == 0) --last;
  for (int i = 0; i < last; ++i)
    if (a.width[i] % V) return false;
  return a.width[last] >= V;
}

template <typename TIO, int K>
hipError_t launch_conv_k(const Conv1dArgs& args, int64_t batch, hipStream_t s) {
  constexpr int W = 16 / sizeof(TIO);
  Conv1dArgs a = args;
  const bool vec = whole_packs<W>(a);
  const int64_t gx = (a.CH + kThreads * (vec ? W : 1) - 1) / (kThreads * (vec ? W : 1));
  // short tiles while they are needed to fill the card, then long ones, whose
  // K - 1 repeated rows weigh less
  int64_t tile = 64;
  while (tile > 8 && gx * batch * ((a.L + tile - 1) / tile) < 2048) tile /= 2;
  // Where the input would drive the output, which the next operator reads, out
  // of the memory-side cache, it is read past the cache (non-temporal): 128 MiB of
  // both 27.7 -> 26.9 us, 256 MiB 56 -> 48 us. Smaller ones may lie there
  // themselves (64 MiB: 14.8 us, past it 16.8), and an output as large as the
  // cache is lost either way (512 MiB: 111 us, past it 114).
  const int64_t out_bytes = batch * a.L * a.CH * (int64_t)sizeof(TIO);
  const bool stream = 2 * out_bytes >= kMemorySideCache / 2 && out_bytes < kMemorySideCache;
  if ((a.L + tile - 1) / tile > 65535) tile = (a.L + 65534) / 65535;
  a.tile = (int)tile;
  const dim3 grid((unsigned)gx, (unsigned)((a.L + tile - 1) / tile), (unsigned)batch);
  if (vec && stream) conv1d_kernel<TIO, K, W, true><<<grid, kThreads, 0, s>>>(a);
  else if (vec) conv1d_kernel<TIO, K, W, false><<<grid, kThreads, 0, s>>>(a);
  else conv1d_kernel<TIO, K, 1, false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename TIO, int K>
hipError_t launch_step_k(const Conv1dStepArgs& a, hipStream_t s) {
  const bool vec = whole_packs<4>(a);
  const int64_t gx = (a.CH + kStepThreads * (vec ? 4 : 1) - 1) / (kStepThreads * (vec ? 4 : 1));
  auto go = [&](auto kern, int rows) {
    kern<<<dim3((unsigned)gx, (unsigned)((a.batch + rows - 1) / rows)), kStepThreads, 0, s>>>(a);
    return hipGetLastError();
  };
  if (!vec) return go(conv1d_step_kernel<TIO, K, 1, 1, false>, 1);
  if (a.CH % 4 != 0) return go(conv1d_step_kernel<TIO, K, 4, 1, true>, 1);
  // several rows a workgroup share the weights once that leaves the card full
  return gx * a.batch >= 4 * 512 ? go(conv1d_step_kernel<TIO, K, 4, 2, false>, 2) : go(conv1d_step_kernel<TIO, K, 4, 1, false>, 1);
}

}  // namespace

hipError_t launch_conv1d(const Conv1dArgs& a, int io, int K, int64_t batch, hipStream_t s) {
  auto with = [&](auto t) {
    using T = decltype(t);
    switch (K) {
      case 1: return launch_conv_k<T, 1>(a, batch, s);
      case 2: return launch_conv_k<T, 2>(a, batch, s);
      case 3: return launch_conv_k<T, 3>(a, batch, s);
      default: return launch_conv_k<T, 4>(a, batch, s);
    }
  };
  return io == kBF16 ? with(__hip_bfloat16{}) : with(float{});
}

hipError_t launch_conv1d_step(const Conv1dStepArgs& a, int io, int K, hipStream_t s) {
  auto with = [&](auto t) {
    using T = decltype(t);
    switch (K) {
      case 1: return launch_step_k<T, 1>(a, s);
      case 2: return launch_step_k<T, 2>(a, s);
      case 3: return launch_step_k<T, 3>(a, s);
      default: return launch_step_k<T, 4>(a, s);
    }
  };
  return io == kBF16 ? with(__hip_bfloat16{}) : with(float{});
}

}  // namespace ssd
