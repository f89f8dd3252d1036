// The gated delta rule in blocks, second kernel: the walk over a sequence's
// blocks of 64 tokens (delta_blocks.h has the formulas and what the first
// kernel left), batched or packed.
//
// The state's rows p do not meet, so a wave keeps 16 of them, transposed
// (S^T [N, 16] in accumulators), for the whole sequence, and nothing of the chain
//     R = X - e^g K S0^T;  U = T R;  S^T <- e^g_end S^T + K^T (e^(g_end - g) U)
// leaves its registers: a product's result, four consecutive rows of a column to a
// lane, is the next product's right operand as it stands once the rows of a
// pair of result tiles are numbered 8 (r / 4) + 4 h + r % 4 (r the row, h the tile).
// The left operands (K by rows and by columns, Q, T, M) are shared by the
// workgroup's four waves through LDS, its 16-byte pieces permuted so that the
// reads by rows and the transposing ones meet few bank conflicts.
//
// Aligned bf16 rows go from memory straight to the LDS (DMA), the next block's while a
// block is worked on: K, which a block needs first and last, into a second tile, what
// else into its own place once it has been read. So two workgroups fit a compute
// unit, and one's products run beside the other's roundings and waits: with 32 rows a
// wave and one workgroup a block of 128 rows took 8600 cycles (each wave's
// instructions one after the other), with all of the LDS once and the whole load waited
// for 8400, of which 3900 were that wait. Other rows go through registers, where odd ones are put
// in order and fp32 is split into terms.
//
// S, R and U' = e^(g_end - g) U are held in fp32. As operands they are terms
// (delta_blocks.h).
#include <type_traits>

#include "delta_blocks.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;  // rows p of a workgroup

template <typename TIO, int NP, bool DMA> struct Layout {
  static constexpr int IO = DeltaTerms<TIO>::io;
  static constexpr int tile = 64 * NP * 2;  // K or Q, one term
  static constexpr int xrow = kCols * (int)sizeof(TIO);
  static constexpr int K = 0, Q = (DMA ? 2 : IO) * tile, rec = Q + IO * tile,
                       X = rec + (DeltaRecord<TIO>::bytes + 1023) / 1024 * 1024, bytes = X + 64 * xrow;
};

// Where the 16-byte piece c of row t lies in K's and Q's and in (bf16) X's tile: c
// with these bits flipped.
template <int NP> __device__ __forceinline__ int k_swz(int t) {
  return NP >= 128 ? ((t & 3) << 2) | ((t >> 3) & 3) : NP == 64 ? ((t & 2) << 1) | ((t >> 3) & 3) : (t >> 3) & 3;
}
__device__ __forceinline__ int x_swz(int t) { return (t & 2) | ((t >> 1) & 4); }

// One matrix product, then V ordinary instructions, M times: what runs beside what.
template <int M, int V> __device__ __forceinline__ void spread() {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x2, V, 0);
  }
}

// PASS 0: over sequences, or over their segments from the states that enter
// them. PASS 1: over segments, what becomes of a state of zeros (rows p) and, with
// values of zero, of the unit states (rows P + n): see delta_join.
template <typename TIO, int NP, bool DMA, bool WHOLE, int PASS>
__global__ __launch_bounds__(kThreads, DMA && NP <= 128 ? 2 : 1) void delta_blocks_kernel(const DeltaArgs a, uint32_t blocks_p) {
  using L = Layout<TIO, NP, DMA>;
  using Rec = DeltaRecord<TIO>;
  constexpr int IO = DeltaTerms<TIO>::io, ST = DeltaTerms<TIO>::state, YT = DeltaTerms<TIO>::y;
  constexpr int KN = NP / 32;          // 32-column groups of N
  constexpr int PACKS = NP / 8;        // 16-byte pieces to a row of K
  constexpr int XP = 16 / (int)sizeof(TIO), XPACKS = kCols / XP;
  constexpr int CK = 64 * PACKS / kThreads, CR = (Rec::bytes / 16 + kThreads - 1) / kThreads, CX = 64 * XPACKS / kThreads;
  constexpr int SZ = (int)sizeof(TIO);
  static_assert(!DMA || (IO == 1 && WHOLE), "rows as they lie");
  static_assert(L::bytes <= 160 * 1024, "LDS of a compute unit");
  __shared__ __align__(16) unsigned char lds[L::bytes];
  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, g = lane / 16, r = lane % 16;

  // (32-bit divisions: those of 64 bits took a microsecond each)
  const uint32_t bid = (uint32_t)xcd_local_order(blockIdx.x, gridDim.x);
  const uint32_t sh = bid / blocks_p;
  const int pb = (int)(bid - sh * blocks_p);
  const int64_t piece = sh / (uint32_t)a.H;
  const int h = (int)(sh - (uint32_t)piece * a.H);
  const int p0 = pb * kCols, pw = p0 + 16 * wave, p = pw + r;  // this wave's rows, this lane's

  // the tokens: of a sequence, or of one of its segments
  DeltaSlot sl;
  if (a.seg != 0) {
    sl = delta_slot(a, (uint32_t)piece, (uint32_t)a.seg);
    if (sl.part < 0 || (sl.part > 0 && sl.t1 <= sl.t0)) return;
    if (PASS == 1 && sl.t1 >= sl.last) return;  // nothing begins behind the last one
  } else {
    sl.seq = piece, sl.row = a.cu != nullptr ? 0 : piece;
    sl.t0 = a.cu != nullptr ? seq_offset(a.cu, piece, a.L) : 0;
    sl.t1 = sl.last = a.cu != nullptr ? seq_offset(a.cu, piece + 1, a.L) : a.L;
    sl.first = sl.t0;
  }
  const int64_t row = sl.row, first = sl.t0, last = sl.t1;
  int64_t slot = delta_first_slot(a, sl.seq, kDeltaBlock) + (first - sl.first) / kDeltaBlock;
  const int rows_p = PASS == 1 ? a.P + a.N : a.P;  // rows in all
  const int64_t grp = (uint32_t)h / ((uint32_t)a.H / (uint32_t)a.G);
  const TIO* Xp = static_cast<const TIO*>(a.x) + row * a.xs.batch + (int64_t)h * a.P;
  const TIO* Bp = static_cast<const TIO*>(a.B) + row * a.bs.batch + grp * a.N;
  const TIO* Cp = static_cast<const TIO*>(a.C) + row * a.cs.batch + grp * a.N;
  TIO* Yp = static_cast<TIO*>(a.y) + (row * a.L * a.H + h) * a.P;
  const int HP = a.H * a.P;

  // ---- rows into LDS
  struct Rows {
    __amdgpu_buffer_rsrc_t B, C, X, R;
  };
  auto rows_of = [&](int64_t t0, int64_t sl) {
    const int n = (int)(last - t0 < 64 ? last - t0 : 64);
    return Rows{block_rows(Bp + t0 * a.bs.token, a.bs.token, n, a.N), block_rows(Cp + t0 * a.cs.token, a.cs.token, n, a.N),
                block_rows(Xp + t0 * a.xs.token, a.xs.token, n, a.P), buffer_range(a.ws + (sl * a.H + h) * Rec::bytes, Rec::bytes)};
  };
  // by DMA: piece c of the LDS holds the row's piece c with the tile's bits flipped
  struct Words {
    v4i32_t B, C, X, R;
    int ktile;
  } to;
  bool more = false;
  auto aim = [&](int64_t t0, int64_t sl, int ktile) {
    const int n = (int)(last - t0 < 64 ? last - t0 : 64);
    to.B = buffer_words(Bp + t0 * a.bs.token, (uint32_t)((n - 1) * a.bs.token + a.N) * SZ);
    to.C = buffer_words(Cp + t0 * a.cs.token, (uint32_t)((n - 1) * a.cs.token + a.N) * SZ);
    to.X = buffer_words(Xp + t0 * a.xs.token, (uint32_t)((n - 1) * a.xs.token + a.P) * SZ);
    to.R = buffer_words(a.ws + (sl * a.H + h) * Rec::bytes, Rec::bytes);
    to.ktile = ktile;
  };
  const uint32_t here = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds + wave * 1024;
  auto send_rows = [&](const v4i32_t& words, int64_t token, uint32_t at, int j) {
    const int t = (j * kThreads + tid) / PACKS, n = 8 * ((tid % PACKS) ^ k_swz<NP>(t));
    dma16(words, here + at + j * kThreads * 16, n < a.N ? (uint32_t)(t * (int)token + n) * SZ : kNowhere);
  };
  auto send_k = [&](int j) { send_rows(to.B, a.bs.token, L::K + to.ktile * L::tile, j); };
  auto send_q_x = [&] {
    if constexpr (PASS == 0) {
#pragma unroll
      for (int j = 0; j < CK; ++j) send_rows(to.C, a.cs.token, L::Q, j);
    }
#pragma unroll
    for (int j = 0; j < CX; ++j) {
      const int t = (j * kThreads + tid) / XPACKS, c = p0 + 8 * ((tid % XPACKS) ^ x_swz(t));
      dma16(to.X, here + L::X + j * kThreads * 16, c < a.P ? (uint32_t)(t * (int)a.xs.token + c) * SZ : kNowhere);
    }
  };
  auto send_record = [&] {
#pragma unroll
    for (int j = 0; j < CR; ++j)
      if (j * 4 + wave < (Rec::bytes + 1023) / 1024) dma16(to.R, here + L::rec + j * kThreads * 16, 16 * (j * kThreads + tid));
  };
  // through registers
  Piece<TIO> kq[2][DMA ? 1 : CK];
  uint4 rc[DMA ? 1 : CR], xv[DMA ? 1 : CX];
  int kmoved, xmoved;
  const int kc = tid % PACKS, xc = tid % XPACKS;  // this thread's piece of a row
  const uint32_t kcol = piece_at<TIO, WHOLE>(8 * kc, a.N, kmoved);
  const uint32_t xcol = piece_at<TIO, WHOLE>(p0 + XP * xc, a.P, xmoved, XP);
  auto fetch = [&](int64_t t0, int64_t sl) {
    if constexpr (!DMA) {
      const Rows from = rows_of(t0, sl);
#pragma unroll
      for (int j = 0; j < CK; ++j) {
        const int t = (j * kThreads + tid) / PACKS;
        kq[0][j] = load_piece<TIO>(from.B, (uint32_t)(t * (int)a.bs.token) * SZ, kcol);
        kq[1][j] = load_piece<TIO>(from.C, (uint32_t)(t * (int)a.cs.token) * SZ, kcol);
      }
#pragma unroll
      for (int j = 0; j < CR; ++j) rc[j] = buffer_ld16(from.R, 16 * (j * kThreads + tid));
#pragma unroll
      for (int j = 0; j < CX; ++j) {
        const int t = (j * kThreads + tid) / XPACKS;
        xv[j] = buffer_ld16(from.X, xcol == kNowhere ? kNowhere : (uint32_t)(t * (int)a.xs.token) * SZ + xcol);
      }
    }
  };
  auto stage = [&] {
    if constexpr (!DMA) {
#pragma unroll
      for (int j = 0; j < CK; ++j) {
        const int t = (j * kThreads + tid) / PACKS;
        unsigned char* kd = lds + L::K + t * (NP * 2) + 16 * (kc ^ k_swz<NP>(t));
        unsigned char* qd = lds + L::Q + t * (NP * 2) + 16 * (kc ^ k_swz<NP>(t));
        move_piece<TIO, WHOLE>(kq[0][j], kmoved);
        move_piece<TIO, WHOLE>(kq[1][j], kmoved);
        if constexpr (IO > 1) {
          const Terms<IO> k = split_piece<IO>(kq[0][j]), q = split_piece<IO>(kq[1][j]);
#pragma unroll
          for (int i = 0; i < IO; ++i) {
            st16(kd + i * L::tile, __builtin_bit_cast(uint4, k.v[i]));
            st16(qd + i * L::tile, __builtin_bit_cast(uint4, q.v[i]));
          }
        } else {
          st16(kd, kq[0][j].v), st16(qd, kq[1][j].v);
        }
      }
#pragma unroll
      for (int j = 0; j < CR; ++j) {
        const int q = j * kThreads + tid;
        if (q < Rec::bytes / 16) st16(lds + L::rec + 16 * q, rc[j]);
      }
#pragma unroll
      for (int j = 0; j < CX; ++j) {
        const int t = (j * kThreads + tid) / XPACKS;
        if constexpr (!WHOLE) {
          uint32_t w[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
          move_down<TIO, 4>(w, xmoved);
          xv[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if constexpr (SZ == 4) st16(lds + L::X + t * L::xrow + ((16 * xc + 64 * ((t >> 3) & 3)) & 255), xv[j]);
        else st16(lds + L::X + t * L::xrow + 16 * (xc ^ x_swz(t)), xv[j]);
      }
    }
  };

  // ---- this lane's operands in LDS
  const int rt = 8 * (r / 4) + r % 4;  // its row of a pair of tiles
  const int ta = r / 4, tb = r % 4;    // its row and piece of a transposing read
  const int kat = rt * (NP * 2), tat = L::K + (8 * g + ta) * (NP * 2);
  const int kf = k_swz<NP>(rt), tf = k_swz<NP>(8 * g + ta);

  if (first < last) {
    if constexpr (DMA) {
      aim(first, slot, 0);
#pragma unroll
      for (int j = 0; j < CK; ++j) send_k(j);
      send_q_x();
      send_record();
    } else {
      fetch(first, slot);
    }
  }

  // S^T: tile (kn, hh) rows 32 kn + 8 g + 4 hh .., column p
  f32x4_t S[KN][2];
  Terms<ST> Sv[KN];
  const int64_t states = (a.seg != 0 ? piece : sl.seq) * a.H + h;
  const float* init = PASS == 1 ? nullptr : a.seg != 0 ? a.enter : a.init;
  auto state_at = [&](int64_t of) { return (of * rows_p + (p < rows_p ? p : 0)) * a.N; };
  auto split_tiles = [&](auto terms, const f32x4_t& t0, const f32x4_t& t1) {
    const float f[8] = {t0[0], t0[1], t0[2], t0[3], t1[0], t1[1], t1[2], t1[3]};
    return split8<decltype(terms)::value>(f);
  };
  constexpr std::integral_constant<int, ST> st_terms{};
  constexpr std::integral_constant<int, YT> y_terms{};
#pragma unroll
  for (int kn = 0; kn < KN; ++kn) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      S[kn][hh] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      const int n = 32 * kn + 8 * g + 4 * hh;
      if (init != nullptr && p < a.P && n < a.N) {
        const Pack<float, 4> v = load_pack<float, 4, true>(init + state_at(states) + n, a.N - n);
#pragma unroll
        for (int i = 0; i < 4; ++i) S[kn][hh][i] = n + i < a.N ? v.v[i] : 0.f;
      }
      if constexpr (PASS == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) S[kn][hh][i] = p - a.P == n + i ? 1.f : 0.f;
      }
    }
    Sv[kn] = split_tiles(st_terms, S[kn][0], S[kn][1]);
  }

  const bool live = pw < rows_p;
  int ktile = 0;
  for (int64_t t0 = first; t0 < last; t0 += 64, ++slot) {
    more = t0 + 64 < last;
    if constexpr (DMA) {
      // this block's rows are there (the last block's four stores are younger)
      if (PASS == 0 && live && t0 != first) vm_wait<4>();
      else vm_wait<0>();
      __syncthreads();
      if (more) aim(t0 + 64, slot + 1, ktile ^ 1);
    } else {
      __syncthreads();  // the last block's operands have been read
      stage();
      __syncthreads();
      if (more) fetch(t0 + 64, slot + 1);
    }
    // The places of Q and X, and later of the record, are free for the next block's.
    auto free_q_x = [&] {
      if constexpr (DMA) {
        __syncthreads();
        if (more) send_q_x();
      }
    };
    auto free_record = [&] {
      if constexpr (DMA) {
        __syncthreads();
        if (more) send_record();
      }
    };
    if (!live) {
      if constexpr (DMA) {
        if (more) {
#pragma unroll
          for (int j = 0; j < CK; ++j) send_k(j);
        }
        ktile ^= 1;
      }
      free_q_x();
      free_record();
      continue;
    }
    const unsigned char* at = lds;
    const unsigned char* ktiles = lds + L::K + (DMA ? ktile * L::tile : 0);
    if constexpr (DMA) ktile ^= 1;
    const int n = (int)(last - t0 < 64 ? last - t0 : 64);

    const float* eg = reinterpret_cast<const float*>(at + L::rec + Rec::decays);
    const float* ed = eg + 64;
    auto by_rows = [&](const unsigned char* from, int i, int kn) {  // rows of tile i, columns 32 kn ..
      Terms<IO> v;
#pragma unroll
      for (int e = 0; e < IO; ++e)
        v.v[e] = as_bf16x8(ld16(from + kat + e * L::tile + (32 * (i / 2) + 4 * (i % 2)) * (NP * 2) + 16 * ((4 * kn + g) ^ kf)));
      return v;
    };
    auto kfrag = [&](int i, int kn) { return by_rows(ktiles, i, kn); };
    auto qfrag = [&](int i, int kn) { return by_rows(at + L::Q, i, kn); };
    auto ktfrag = [&](int hh, int kk, int kn) {  // tile hh of columns 32 kn .., rows 32 kk ..
      Terms<IO> v;
#pragma unroll
      for (int e = 0; e < IO; ++e) {
        const unsigned char* s = ktiles + tat + e * L::tile + 32 * kk * (NP * 2) + 16 * ((4 * kn + tb) ^ tf) + 8 * hh;
        const uint2 lo = lds_tr8(s), hi = lds_tr8(s + 4 * (NP * 2));
        v.v[e] = as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
      }
      return v;
    };
    auto tri = [&](auto terms, int from, int i) {
      Terms<decltype(terms)::value> v;
#pragma unroll
      for (int e = 0; e < decltype(terms)::value; ++e)
        v.v[e] = as_bf16x8(ld16(at + L::rec + 16 * lane + from + (e * kTriFrags + i) * kFragBytes));
      return v;
    };
    auto of_y = [&](const Terms<ST>& s) {
      Terms<YT> v;
#pragma unroll
      for (int e = 0; e < YT; ++e) v.v[e] = s.v[e];
      return v;
    };

    // Operands are read a group ahead of the products that use them, and the
    // order is held: the compiler by itself reads each right before its use and
    // waits for it.
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    const float end = eg[63];
    f32x4_t R[4], O[4], e[4];
    float xw[4][4];
    uint2 xr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) R[i] = O[i] = zero;
    Terms<IO> f[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[0][i] = kfrag(i, 0);

    // K S0^T (rows t, column p); beside it S^T e^g_end
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      if (kn + 1 < KN) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[(kn + 1) % 2][i] = kfrag(i, kn + 1);
      } else {
#pragma unroll
        for (int i = 0; i < 4 && PASS == 0; ++i) f[(kn + 1) % 2][i] = qfrag(i, 0);
        // X by columns, and the decays
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tr = 32 * (i / 2) + 8 * g + 4 * (i % 2);
          e[i] = *reinterpret_cast<const f32x4_t*>(eg + tr);
          if constexpr (SZ == 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              xw[i][k] = *reinterpret_cast<const float*>(at + L::X + (tr + k) * L::xrow + ((4 * (16 * wave + r) + 64 * g) & 255));
          } else {
            const int t = tr + ta;
            xr[i] = lds_tr8(at + L::X + t * L::xrow + 16 * ((2 * wave + tb / 2) ^ x_swz(t)) + 8 * (tb & 1));
          }
        }
      }
      hold();
#pragma unroll
      for (int pair = 0; pair < term_pairs(IO, ST); ++pair)
#pragma unroll
        for (int i = 0; i < 4; ++i) mul_pair(R[i], f[kn % 2][i], Sv[kn], pair);
#pragma unroll
      for (int i = 0; i < 8; ++i) S[kn][i / 4][i % 4] *= end;
      spread<4 * term_pairs(IO, ST), 1>();
      hold();
      if constexpr (DMA) {
        if (more) {
#pragma unroll
          for (int j = 0; j < CK; ++j)
            if (j * KN / CK == kn) send_k(j);
        }
      }
    }
    // S0 Q^T (rows p, column t); beside it R = X - e^g K S0^T
    Terms<ST> Rv[2];
    Terms<ST> tm[kTriFrags];
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      if (PASS == 0 && kn + 1 < KN) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[(KN + kn + 1) % 2][i] = qfrag(i, kn + 1);
      }
#pragma unroll
      for (int i = 0; i < kTriFrags; ++i)
        if (i * KN / kTriFrags == kn) tm[i] = tri(st_terms, Rec::T, i);
      hold();
#pragma unroll
      for (int pair = 0; pair < term_pairs(YT, IO) && PASS == 0; ++pair)
#pragma unroll
        for (int i = 0; i < 4; ++i) mul_pair(O[i], of_y(Sv[kn]), f[(KN + kn) % 2][i], pair);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        if (kk * KN / 2 != kn) continue;
#pragma unroll
        for (int i = 2 * kk; i < 2 * kk + 2; ++i) {
          if constexpr (SZ == 2) {
            xw[i][0] = bf16_lo(xr[i].x), xw[i][1] = bf16_hi(xr[i].x);
            xw[i][2] = bf16_lo(xr[i].y), xw[i][3] = bf16_hi(xr[i].y);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) R[i][k] = fmaf(-e[i][k], R[i][k], xw[i][k]);
        }
        Rv[kk] = split_tiles(st_terms, R[2 * kk], R[2 * kk + 1]);
      }
      spread<4 * term_pairs(YT, IO), 2>();
      hold();
    }
    free_q_x();
    // U = T R; beside it O e^g
    f32x4_t U[4], d[4];
    float er[4];
    Terms<YT> mf[kTriFrags], Uy[2];
#pragma unroll
    for (int i = 0; i < 4 && PASS == 0; ++i) er[i] = eg[32 * (i / 2) + 4 * (i % 2) + rt];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<const f32x4_t*>(ed + 32 * (i / 2) + 8 * g + 4 * (i % 2));
    hold();
#pragma unroll
    for (int i = 0; i < 4; ++i) U[i] = zero;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int pair = 0; pair < term_pairs(ST, ST); ++pair)
#pragma unroll
        for (int i = 2 * ks; i < 4; ++i) mul_pair(U[i], tm[tri_frag(i / 2, i % 2, ks)], Rv[ks], pair);
#pragma unroll
    for (int i = 0; i < 4 && PASS == 0; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) O[i][k] *= a.scale * er[i];
    spread<6 * term_pairs(ST, ST), 2>();
    hold();
#pragma unroll
    for (int i = 0; i < kTriFrags && PASS == 0; ++i) mf[i] = tri(y_terms, Rec::M, i);
    hold();
    // operands of y, and U' = e^(g_end - g) U
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      if constexpr (PASS == 0) Uy[kk] = split_tiles(y_terms, U[2 * kk], U[2 * kk + 1]);
#pragma unroll
      for (int i = 2 * kk; i < 2 * kk + 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) U[i][k] *= d[i][k];
      Rv[kk] = split_tiles(st_terms, U[2 * kk], U[2 * kk + 1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[0][i] = ktfrag(i % 2, i / 2, 0);
    hold();
    // + U^T (scale M)^T
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int pair = 0; pair < term_pairs(YT, YT) && PASS == 0; ++pair)
#pragma unroll
        for (int i = 2 * ks; i < 4; ++i) mul_pair(O[i], Uy[ks], mf[tri_frag(i / 2, i % 2, ks)], pair);
    hold();
    free_record();
    // y: rows pw + 4 g .. of a lane at token 32 (i / 2) + 4 (i % 2) + rt
    auto put_y = [&] {
      const __amdgpu_buffer_rsrc_t Yr = buffer_range(Yp + t0 * HP, (uint32_t)((n - 1) * HP + a.P) * SZ);
      const int pr = pw + 4 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t off = (uint32_t)((32 * (i / 2) + 4 * (i % 2) + rt) * HP + pr) * SZ;
        if constexpr (WHOLE) {
          const uint32_t where = pr < a.P ? off : kNowhere;
          if constexpr (SZ == 4) buffer_st16(__builtin_bit_cast(uint4, O[i]), Yr, where);
          else buffer_st8(make_uint2(pack_bf16x2(O[i][0], O[i][1]), pack_bf16x2(O[i][2], O[i][3])), Yr, where);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t where = pr + k < a.P ? off + k * SZ : kNowhere;
            if constexpr (SZ == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(O[i][k]), Yr, (int)where, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b16(bf16_bits(O[i][k]), Yr, (int)where, 0, 0);
          }
        }
      }
    };
    // S^T += K^T U'; beside it the terms of the group before, and y
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      if (kn + 1 < KN) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[(kn + 1) % 2][i] = ktfrag(i % 2, i / 2, kn + 1);
      }
      hold();
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int pair = 0; pair < term_pairs(IO, ST); ++pair)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) mul_pair(S[kn][hh], f[kn % 2][2 * kk + hh], Rv[kk], pair);
      if (kn > 0) Sv[kn - 1] = split_tiles(st_terms, S[kn - 1][0], S[kn - 1][1]);
      spread<4 * term_pairs(IO, ST), 2>();
      hold();
      if (PASS == 0 && kn == 0) put_y();
    }
    Sv[KN - 1] = split_tiles(st_terms, S[KN - 1][0], S[KN - 1][1]);
  }

  float* out = PASS == 1 ? a.ends : sl.t1 >= sl.last ? a.final_state : nullptr;
  if (out == nullptr || p >= rows_p) return;
#pragma unroll
  for (int kn = 0; kn < KN; ++kn)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int n = 32 * kn + 8 * g + 4 * hh;
      const float v[4] = {S[kn][hh][0], S[kn][hh][1], S[kn][hh][2], S[kn][hh][3]};
      if (n < a.N) store_pack<float, 4, true>(out + state_at(PASS == 1 ? states : sl.seq * a.H + h) + n, v, a.N - n);
    }
}

template <typename TIO, int NP, int PASS>
hipError_t launch_pass(const DeltaArgs& a, hipStream_t s) {
  const int rows_p = PASS == 1 ? a.P + a.N : a.P;
  const uint32_t blocks_p = (rows_p + kCols - 1) / kCols;
  const int64_t pieces = a.seg != 0 ? delta_slots(a, a.seg) : a.seqs();
  auto go = [&](auto kern) {
    kern<<<dim3((unsigned)(pieces * a.H * blocks_p)), kThreads, 0, s>>>(a, blocks_p);
    return hipGetLastError();
  };
  const bool whole = a.N % 8 == 0 && a.P % (16 / sizeof(TIO)) == 0;
  if constexpr (sizeof(TIO) == 2) {
    auto lies = [](const void* p, const Stride& st) {
      return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(st.token * 2) | (uintptr_t)(st.batch * 2)) % 16 == 0;
    };
    if (whole && lies(a.x, a.xs) && lies(a.B, a.bs) && lies(a.C, a.cs)) return go(delta_blocks_kernel<TIO, NP, true, true, PASS>);
    return go(delta_blocks_kernel<TIO, NP, false, false, PASS>);
  } else {
    return whole ? go(delta_blocks_kernel<TIO, NP, false, true, PASS>) : go(delta_blocks_kernel<TIO, NP, false, false, PASS>);
  }
}

template <typename TIO, int NP>
hipError_t launch_np(const DeltaArgs& a, hipStream_t s) {
  if (a.seg != 0) {
    hipError_t e = launch_pass<TIO, NP, 1>(a, s);
    if (e == hipSuccess) e = launch_delta_join(a, s);
    if (e != hipSuccess) return e;
  }
  return launch_pass<TIO, NP, 0>(a, s);
}

template <typename TIO>
hipError_t launch_io(const DeltaArgs& a, hipStream_t s) {
  if (a.N <= 32) return launch_np<TIO, 32>(a, s);
  if (a.N <= 64) return launch_np<TIO, 64>(a, s);
  if (a.N <= 128) return launch_np<TIO, 128>(a, s);
  if constexpr (sizeof(TIO) == 2) return launch_np<TIO, 256>(a, s);
  return hipErrorInvalidValue;
}

// Tokens of a segment, 0 where sequences are walked in one piece. A sequence's
// blocks depend on one another; where all rows, heads and columns give fewer workgroups
// than the card has compute units, the time axis is cut: a first walk gives what each segment
// makes of any state (P + N rows instead of P, without y, about 3/4 of a block's time
// a row), the states are joined in turn, and the segments are walked side by side.
// In quarters of a block's time on a compute unit; a join takes about a block's.
// Of packed sequences only the number is known here: the stream is taken for so many
// of four times their mean length.
int64_t delta_segment(const DeltaArgs& a, int io) {
  int64_t tokens = a.L, seqs = a.batch;
  if (a.nseq > 0) tokens = 4 * ((a.L + a.nseq - 1) / a.nseq) < a.L ? 4 * ((a.L + a.nseq - 1) / a.nseq) : a.L, seqs = (a.L + tokens - 1) / tokens;
  const int64_t wgs = seqs * a.H * ((a.P + kCols - 1) / kCols), first = seqs * a.H * ((a.P + a.N + kCols - 1) / kCols);
  const int64_t blocks = (tokens + kDeltaBlock - 1) / kDeltaBlock, cus = io == kBF16 && a.N <= 128 ? 512 : 256;  // workgroups at once
  auto turns = [&](int64_t w) { return (w + cus - 1) / cus; };
  int64_t best = turns(wgs) * blocks * 4, cut = 0;
  for (int64_t n = 2; n <= 64 && n * 4 <= blocks; ++n) {
    const int64_t len = (blocks + n - 1) / n;
    const int64_t t = turns(wgs * n) * len * 4 + turns(first * (n - 1)) * len * 3 + n * 4 + 12;
    if (t < best) best = t, cut = len;
  }
  return cut * kDeltaBlock;
}

size_t record_bytes(int io) { return io == kBF16 ? DeltaRecord<__hip_bfloat16>::bytes : DeltaRecord<float>::bytes; }

}  // namespace

bool delta_blocks_apply(const DeltaArgs& a, int io) {
  return (io == kBF16 || a.N <= 128) && a.L >= 16 && a.N >= 8 && a.P >= 8;
}

int64_t delta_blocks_workspace(DeltaArgs& a, int io) {
  const int64_t records = delta_slots(a) * a.H * (int64_t)record_bytes(io);
  a.seg = delta_segment(a, io);
  if (a.seg == 0) return records;
  const int64_t states = delta_slots(a, a.seg) * a.H;
  return records + states * (2 * a.P + a.N) * a.N * (int64_t)sizeof(float);
}

hipError_t launch_delta_blocks(const DeltaArgs& args, int io, int dt, hipStream_t s) {
  DeltaArgs a = args;
  if (a.seg != 0) {
    const int64_t states = delta_slots(a, a.seg) * a.H;
    a.ends = reinterpret_cast<float*>(a.ws + delta_slots(a) * a.H * (int64_t)record_bytes(io));
    a.enter = a.ends + states * (a.P + a.N) * a.N;
  }
  const hipError_t e = launch_delta_solve(a, io, dt, s);
  if (e != hipSuccess) return e;
  return io == kBF16 ? launch_io<__hip_bfloat16>(a, s) : launch_io<float>(a, s);
}

}  // namespace ssd
