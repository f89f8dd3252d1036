// The gated delta rule in blocks, the walk over a sequence's blocks of 64 tokens for
// aligned bf16 rows (delta_blocks.h has the formulas, and what the first kernel left;
// k_delta_blocks.hip takes all other rows).
//
// Two kinds of waves. The state's rows p do not meet, so each of four waves keeps 16 PT of
// them, transposed (S^T [N, 16] in accumulators), for the whole sequence, and nothing of the chain
//     R = X - e^g K S0^T;  U = T R;  S^T <- e^g_end S^T + K^T (e^(g_end - g) U)
// leaves its registers: a product's result, four consecutive rows of a column to a
// lane, is the next product's right operand as it stands once the rows of a
// pair of result tiles are numbered 8 (r / 4) + 4 h + r % 4 (r the row, h the tile).
// A partner of each on the same SIMD is handed S0 and U through LDS, makes y of
// them, and brings the next block's rows to the LDS (DMA), so that the chain's
// own instructions are all that a block's time is made of.
//
// The left operands (K by rows and by columns, Q, T, M) are shared by the
// workgroup through LDS, its 16-byte pieces permuted so that the reads by rows and
// the transposing ones meet few bank conflicts. All but T have two places, so that
// the next block's have a block's time to arrive; U takes the place of the X that it came from,
// and T, which a block needs last, is refilled once it has been read.
//
// Measured: 8 sequences of 2048 tokens, 32 heads, P = N = 128: 118 us, 3.4 us a block
// (8400 cycles). Bound by the chain's instructions: 164 matrix and some 560 others a wave
// and block, which alone take 6600 cycles; the rest is the partner's share of the
// SIMD and of the LDS. The register-staged walk of one kind of waves took 158 us.
#include <type_traits>

#include "delta_blocks.h"

namespace ssd {
namespace {

using T16 = __hip_bfloat16;
constexpr int kChainWaves = 4, kThreads = 128 * kChainWaves;
constexpr int ST = DeltaTerms<T16>::state;  // 2
using Rec = DeltaRecord<T16>;

template <int NP, int PT, int PASS> struct Layout {
  static constexpr int cols = 64 * PT;  // rows p of a workgroup
  static constexpr int tile = 64 * NP * 2, xrow = 2 * cols, mbytes = kTriFrags * kFragBytes;
  static constexpr int K = 0, X = 2 * tile, T = X + 2 * 64 * xrow, decays = T + Rec::M, all = decays + 2048;  // of both passes
  static constexpr int Q = all, M = Q + 2 * tile, S0 = M + 2 * mbytes, y = S0 + cols * NP * 2;
  static constexpr int bytes = PASS == 0 ? y : all;
};
template <int PT> __device__ __forceinline__ int x_swz(int t) { return PT == 2 ? (t & 3) << 2 : (t & 2) | ((t >> 1) & 4); }

// PASS as in k_delta_blocks.hip.
template <int NP, int PT, int PASS>
__global__ __launch_bounds__(kThreads) void delta_chain_kernel(const DeltaArgs a, uint32_t blocks_p) {
  using L = Layout<NP, PT, PASS>;
  constexpr int KN = NP / 32;            // 32-column groups of N
  constexpr int PACKS = NP / 8;          // 16-byte pieces to a row of K
  constexpr int XPACKS = L::cols / 8;
  constexpr int CK = 64 * PACKS / 256, CX = 64 * XPACKS / 256;
  static_assert(L::bytes <= 160 * 1024, "LDS of a compute unit");
  __shared__ __align__(16) unsigned char lds[L::bytes];
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  // (known to be the same in all lanes: the two kinds' barriers are then behind branches of the whole wave)
  const int any_wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x / 64), wave = any_wave % kChainWaves;
  const bool chain = any_wave < kChainWaves;

  // (32-bit divisions: those of 64 bits took a microsecond each)
  const uint32_t bid = (uint32_t)xcd_local_order(blockIdx.x, gridDim.x);
  const uint32_t sh = bid / blocks_p;
  const int pb = (int)(bid - sh * blocks_p);
  const int64_t piece = sh / (uint32_t)a.H;
  const int h = (int)(sh - (uint32_t)piece * a.H);
  DeltaSlot sl;
  if (!delta_piece<PASS>(a, piece, sl)) return;
  const int64_t first = sl.t0, last = sl.t1;
  int64_t slot = delta_first_slot(a, sl.index, kDeltaBlock) + (first - sl.first) / kDeltaBlock;
  const int rows_p = PASS == 1 ? a.P + a.N : a.P;  // rows in all
  const int p0 = pb * L::cols, pw = p0 + 16 * PT * wave;
  const bool live = pw < rows_p;
  const int rt = 8 * (r / 4) + r % 4;  // this lane's row of a pair of tiles
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  // 16 x 32 operands that one wave wrote or the first kernel did, lane after lane
  auto frag = [&](int at, int i) { return as_bf16x8(ld16(lds + at + i * kFragBytes + 16 * lane)); };
  // rows of tile i of a pair, columns 32 kn ..
  const int kat = rt * (NP * 2), kf = k_swz<NP>(rt);
  auto by_rows = [&](int at, int i, int kn) {
    return as_bf16x8(ld16(lds + at + kat + (32 * (i / 2) + 4 * (i % 2)) * (NP * 2) + 16 * ((4 * kn + g) ^ kf)));
  };

  // U's piece i of this lane, in the place of this wave's columns of X
  auto u_place = [&](int half, int i) {
    const int u = i * 64 + lane, t = u / (2 * PT);
    return L::X + half * 64 * L::xrow + t * L::xrow + 16 * ((2 * PT * wave + u % (2 * PT)) ^ x_swz<PT>(t));
  };

  if (!chain) {
    // ---- rows to LDS, and y
    const int64_t grp = (uint32_t)h / ((uint32_t)a.H / (uint32_t)a.G);
    const T16* Xp = static_cast<const T16*>(a.x) + sl.row * a.xs.batch + (int64_t)h * a.P;
    const T16* Bp = static_cast<const T16*>(a.B) + sl.row * a.bs.batch + grp * a.N;
    const T16* Cp = static_cast<const T16*>(a.C) + sl.row * a.cs.batch + grp * a.N;
    T16* Yp = static_cast<T16*>(a.y) + (sl.row * a.L * a.H + h) * a.P;
    const int HP = a.H * a.P, tid = threadIdx.x - 64 * kChainWaves;
    const uint32_t here = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds + wave * 1024;
    v4i32_t Bw, Cw, Xw, Rw;
    auto aim = [&](int64_t t0, int64_t s) {
      const int n = (int)(last - t0 < 64 ? last - t0 : 64);
      Bw = buffer_words(Bp + t0 * a.bs.token, (uint32_t)((n - 1) * a.bs.token + a.N) * 2);
      Cw = buffer_words(Cp + t0 * a.cs.token, (uint32_t)((n - 1) * a.cs.token + a.N) * 2);
      Xw = buffer_words(Xp + t0 * a.xs.token, (uint32_t)((n - 1) * a.xs.token + a.P) * 2);
      Rw = buffer_words(a.ws + (s * a.H + h) * Rec::bytes, Rec::bytes);
    };
    // piece c of the LDS holds the row's piece c with the tile's bits flipped
    auto send_rows = [&](const v4i32_t& words, int64_t token, uint32_t at) {
#pragma unroll
      for (int j = 0; j < CK; ++j) {
        const int t = (j * 256 + tid) / PACKS, n = 8 * ((tid % PACKS) ^ k_swz<NP>(t));
        dma16(words, here + at + j * 4096, n < a.N ? (uint32_t)(t * (int)token + n) * 2 : kNowhere);
      }
    };
    auto send_record = [&](uint32_t from, uint32_t to, int bytes) {
#pragma unroll
      for (int j = 0; j < (bytes + 4095) / 4096; ++j)
        if (j * 4 + wave < (bytes + 1023) / 1024) dma16(Rw, here + to + j * 4096, from + j * 4096 + wave * 1024 + 16 * lane);
    };
    auto send_rest = [&](int half) {
      send_rows(Bw, a.bs.token, L::K + half * L::tile);
#pragma unroll
      for (int j = 0; j < CX; ++j) {
        const int t = (j * 256 + tid) / XPACKS, c = p0 + 8 * ((tid % XPACKS) ^ x_swz<PT>(t));
        dma16(Xw, here + L::X + half * 64 * L::xrow + j * 4096, c < a.P ? (uint32_t)(t * (int)a.xs.token + c) * 2 : kNowhere);
      }
      // (the second half of the instruction's 1024 bytes lies behind the record and reads as zeros)
      if (wave == 0) dma16(Rw, here + L::decays + half * 1024, Rec::decays + 16 * lane);
      if constexpr (PASS == 0) {
        send_rows(Cw, a.cs.token, L::Q + half * L::tile);
        send_record(Rec::M, L::M + half * L::mbytes, L::mbytes);
      }
    };
    auto send_t = [&] { send_record(Rec::T, L::T, Rec::M); };
    int half = 0;
    if (first < last) {
      aim(first, slot);
      send_rest(0);
      send_t();
    }
    for (int64_t t0 = first; t0 < last; t0 += 64, ++slot, half ^= 1) {
      const bool more = t0 + 64 < last;
      // this block's rows are there (the last block's four stores are younger)
      if (PASS == 0 && live && t0 != first) vm_wait<4>();
      else vm_wait<0>();
      __syncthreads();
      if (more) {
        aim(t0 + 64, slot + 1);
        send_rest(half ^ 1);
      }
      f32x4_t O[PT][4];
      if constexpr (PASS == 0) {
        if (live) {
          // S0 Q^T (rows p, column t) scale e^g
          bf16x8_t q[2][4], s[2][PT];
          auto group = [&](int b, int kn) {
#pragma unroll
            for (int i = 0; i < 4; ++i) q[b][i] = by_rows(L::Q + half * L::tile, i, kn);
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) s[b][pt] = frag(L::S0 + wave * KN * PT * kFragBytes, kn * PT + pt);
          };
#pragma unroll
          for (int pt = 0; pt < PT; ++pt)
#pragma unroll
            for (int i = 0; i < 4; ++i) O[pt][i] = zero;
          group(0, 0);
#pragma unroll
          for (int kn = 0; kn < KN; ++kn) {
            if (kn + 1 < KN) group((kn + 1) % 2, kn + 1);
            hold();
#pragma unroll
            for (int pt = 0; pt < PT; ++pt)
#pragma unroll
              for (int i = 0; i < 4; ++i) O[pt][i] = mfma_16x16x32(s[kn % 2][pt], q[kn % 2][i], O[pt][i]);
            hold();
          }
          const float* eg = reinterpret_cast<const float*>(lds + L::decays + half * 1024);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = a.scale * eg[32 * (i / 2) + 4 * (i % 2) + rt];
#pragma unroll
            for (int pt = 0; pt < PT; ++pt)
#pragma unroll
              for (int k = 0; k < 4; ++k) O[pt][i][k] *= e;
          }
        }
      }
      __syncthreads();  // T has been read, U is there
      if (more) send_t();
      if constexpr (PASS == 0) {
        if (!live) continue;
        // + U^T (scale M)^T
        bf16x8_t m[kTriFrags], u[PT][2];
#pragma unroll
        for (int i = 0; i < kTriFrags; ++i) m[i] = frag(L::M + half * L::mbytes, i);
#pragma unroll
        for (int pt = 0; pt < PT; ++pt)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) u[pt][ks] = as_bf16x8(ld16(lds + u_place(half, pt * 2 + ks)));
        hold();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int i = 2 * ks; i < 4; ++i)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) O[pt][i] = mfma_16x16x32(u[pt][ks], m[tri_frag(i / 2, i % 2, ks)], O[pt][i]);
        // rows pw + 4 PT g .. of a lane at token 32 (i / 2) + 4 (i % 2) + rt
        const int n = (int)(last - t0 < 64 ? last - t0 : 64), pr = pw + 4 * PT * g;
        const __amdgpu_buffer_rsrc_t Yr = buffer_range(Yp + t0 * HP, (uint32_t)((n - 1) * HP + a.P) * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t to = pr < a.P ? (uint32_t)((32 * (i / 2) + 4 * (i % 2) + rt) * HP + pr) * 2 : kNowhere;
          const uint2 lo = make_uint2(pack_bf16x2(O[0][i][0], O[0][i][1]), pack_bf16x2(O[0][i][2], O[0][i][3]));
          if constexpr (PT == 2)
            buffer_st16(make_uint4(lo.x, lo.y, pack_bf16x2(O[1][i][0], O[1][i][1]), pack_bf16x2(O[1][i][2], O[1][i][3])), Yr, to);
          else
            buffer_st8(lo, Yr, to);
        }
      }
    }
    return;
  }

  if (!live) {
    for (int64_t t0 = first; t0 < last; t0 += 64) {
      __syncthreads();
      __syncthreads();
    }
    return;
  }

  // ---- the chain. Column r of tile pt:
  auto column = [&](int pt) { return PT == 2 ? pw + rt + 4 * pt : pw + r; };
  // S^T: tile (pt, kn, hh) rows 32 kn + 8 g + 4 hh .., column `column(pt)`
  f32x4_t S[PT][KN][2];
  Terms<ST> Sv[PT][KN];
  const int64_t states = (a.seg != 0 ? piece : sl.seq) * a.H + h;
  const float* init = PASS == 1 ? nullptr : a.seg != 0 ? a.enter : a.init;
  auto state_at = [&](int pt, int64_t of) { return (of * rows_p + (column(pt) < rows_p ? column(pt) : 0)) * a.N; };
  auto split_tiles = [&](const f32x4_t& t0, const f32x4_t& t1) {
    const float f[8] = {t0[0], t0[1], t0[2], t0[3], t1[0], t1[1], t1[2], t1[3]};
    return split8<ST>(f);
  };
  auto hand_over_s = [&](int kn, int pt) {
    if constexpr (PASS == 0)
      st16(lds + L::S0 + (wave * KN * PT + kn * PT + pt) * kFragBytes + 16 * lane, __builtin_bit_cast(uint4, Sv[pt][kn].v[0]));
  };
#pragma unroll
  for (int pt = 0; pt < PT; ++pt)
#pragma unroll
    for (int kn = 0; kn < KN; ++kn)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        S[pt][kn][hh] = zero;
        const int n = 32 * kn + 8 * g + 4 * hh;
        if (init != nullptr && column(pt) < a.P && n < a.N) {  // (N is a multiple of 8)
          const Pack<float, 4> v = load_pack<float, 4>(init + state_at(pt, states) + n);
          S[pt][kn][hh] = f32x4_t{v.v[0], v.v[1], v.v[2], v.v[3]};
        }
        if constexpr (PASS == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) S[pt][kn][hh][i] = column(pt) - a.P == n + i ? 1.f : 0.f;
        }
      }
#pragma unroll
  for (int pt = 0; pt < PT; ++pt)
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      Sv[pt][kn] = split_tiles(S[pt][kn][0], S[pt][kn][1]);
      hand_over_s(kn, pt);
    }

  const int ta = r / 4, tb = r % 4;  // this lane's row and piece of a transposing read
  const int tat = (8 * g + ta) * (NP * 2), tf = k_swz<NP>(8 * g + ta);
  int half = 0;
  for (int64_t t0 = first; t0 < last; t0 += 64, half ^= 1) {
    __syncthreads();
    const float* eg = reinterpret_cast<const float*>(lds + L::decays + half * 1024);
    const int k_at = L::K + half * L::tile;
    auto ktfrag = [&](int hh, int kk, int kn) {  // tile hh of columns 32 kn .., rows 32 kk ..
      const unsigned char* s = lds + k_at + tat + 32 * kk * (NP * 2) + 16 * ((4 * kn + tb) ^ tf) + 8 * hh;
      const uint2 lo = lds_tr8(s), hi = lds_tr8(s + 4 * (NP * 2));
      return as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
    };
    // Operands are read a group ahead of the products that use them, and the
    // order is held: the compiler by itself reads each right before its use and
    // waits for it.
    bf16x8_t f[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[0][i] = by_rows(k_at, i, 0);
    const float end = eg[63];
    f32x4_t R[PT][4], e[4], d[4];
    uint2 xr[PT][4];
    bf16x8_t tm[ST][kTriFrags];
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int i = 0; i < 4; ++i) R[pt][i] = zero;
    // K S0^T (rows t, column p); beside it S^T e^g_end
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      if (kn + 1 < KN) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[(kn + 1) % 2][i] = by_rows(k_at, i, kn + 1);
      } else {
        // X by columns, and the decays
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tr = 32 * (i / 2) + 8 * g + 4 * (i % 2), t = tr + ta;
          e[i] = *reinterpret_cast<const f32x4_t*>(eg + tr);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            const int c = PT == 2 ? 4 * wave + tb : 2 * wave + tb / 2;
            xr[pt][i] = lds_tr8(lds + L::X + half * 64 * L::xrow + t * L::xrow + 16 * (c ^ x_swz<PT>(t)) + 8 * (PT == 2 ? pt : tb & 1));
          }
        }
      }
      hold();
#pragma unroll
      for (int term = 0; term < ST; ++term)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) R[pt][i] = mfma_16x16x32(f[kn % 2][i], Sv[pt][kn].v[term], R[pt][i]);
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int i = 0; i < 8; ++i) S[pt][kn][i / 4][i % 4] *= end;
      spread<4 * PT * ST, 1>();
      hold();
    }
    // R = X - e^g K S0^T
#pragma unroll
    for (int i = 0; i < kTriFrags; ++i)
#pragma unroll
      for (int term = 0; term < ST; ++term) tm[term][i] = frag(L::T + term * kTriFrags * kFragBytes, i);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<const f32x4_t*>(eg + 64 + 32 * (i / 2) + 8 * g + 4 * (i % 2));
    hold();
    Terms<ST> Rv[PT][2];
    f32x4_t U[PT][4];
    auto turn_r = [&](int pt, int kk) {
#pragma unroll
      for (int i = 2 * kk; i < 2 * kk + 2; ++i) {
        const float x[4] = {bf16_lo(xr[pt][i].x), bf16_hi(xr[pt][i].x), bf16_lo(xr[pt][i].y), bf16_hi(xr[pt][i].y)};
#pragma unroll
        for (int k = 0; k < 4; ++k) R[pt][i][k] = fmaf(-e[i][k], R[pt][i][k], x[k]);
      }
      Rv[pt][kk] = split_tiles(R[pt][2 * kk], R[pt][2 * kk + 1]);
    };
    // U = T R; beside it the next of R
    auto times_t = [&](int pt, int ks) {
#pragma unroll
      for (int pair = 0; pair < 3; ++pair)
#pragma unroll
        for (int i = 2 * ks; i < 4; ++i)
          U[pt][i] = mfma_16x16x32(tm[pair == 2][tri_frag(i / 2, i % 2, ks)], Rv[pt][ks].v[pair == 1], U[pt][i]);
    };
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int i = 0; i < 4; ++i) U[pt][i] = zero;
    turn_r(0, 0);
    hold();
#pragma unroll
    for (int step = 0; step < 2 * PT; ++step) {
      times_t(step / 2, step % 2);
      if (step + 1 < 2 * PT) turn_r((step + 1) / 2, (step + 1) % 2);
      spread<12, 3>();
      hold();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[0][i] = ktfrag(i % 2, i / 2, 0);
    // U for y, and U' = e^(g_end - g) U
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const f32x4_t &u0 = U[pt][2 * kk], &u1 = U[pt][2 * kk + 1];
        if constexpr (PASS == 0)
          st16(lds + u_place(half, pt * 2 + kk), make_uint4(pack_bf16x2(u0[0], u0[1]), pack_bf16x2(u0[2], u0[3]),
                                                            pack_bf16x2(u1[0], u1[1]), pack_bf16x2(u1[2], u1[3])));
      }
    __syncthreads();  // T has been read, U is there
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int i = 2 * kk; i < 2 * kk + 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) U[pt][i][k] *= d[i][k];
        Rv[pt][kk] = split_tiles(U[pt][2 * kk], U[pt][2 * kk + 1]);
      }
    // S^T += K^T U'; beside it the terms of the group before
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
        for (int term = 0; term < ST; ++term)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) S[pt][kn][hh] = mfma_16x16x32(f[kn % 2][2 * kk + hh], Rv[pt][kk].v[term], S[pt][kn][hh]);
      if (kn > 0) {
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) Sv[pt][kn - 1] = split_tiles(S[pt][kn - 1][0], S[pt][kn - 1][1]);
      }
      spread<4 * PT * ST, 3>();
      hold();
    }
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) Sv[pt][KN - 1] = split_tiles(S[pt][KN - 1][0], S[pt][KN - 1][1]);
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int kn = 0; kn < KN; ++kn) hand_over_s(kn, pt);
  }

  float* out = PASS == 1 ? a.ends : sl.t1 >= sl.last ? a.final_state : nullptr;
  if (out == nullptr) return;
#pragma unroll
  for (int pt = 0; pt < PT; ++pt)
#pragma unroll
    for (int kn = 0; kn < KN; ++kn)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int n = 32 * kn + 8 * g + 4 * hh;
        const float v[4] = {S[pt][kn][hh][0], S[pt][kn][hh][1], S[pt][kn][hh][2], S[pt][kn][hh][3]};
        if (column(pt) < rows_p && n < a.N) store_pack<float, 4>(out + state_at(pt, PASS == 1 ? states : sl.seq * a.H + h) + n, v);
      }
}

// Workgroups to a head's rows: of 128 of them, of 64 where there are no more.
uint32_t blocks_of(const DeltaArgs& a, int pass) { return (delta_rows(a, pass) + 127) / 128; }

template <int NP, int PASS> hipError_t launch_np(const DeltaArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)delta_chain_groups(a, PASS));
  const uint32_t blocks_p = blocks_of(a, PASS);
  if (delta_rows(a, PASS) > 64) delta_chain_kernel<NP, 2, PASS><<<grid, kThreads, 0, s>>>(a, blocks_p);
  else delta_chain_kernel<NP, 1, PASS><<<grid, kThreads, 0, s>>>(a, blocks_p);
  return hipGetLastError();
}

}  // namespace

bool delta_chain_applies(const DeltaArgs& a, int io) {
  auto lies = [](const void* p, const Stride& st) {
    return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(st.token * 2) | (uintptr_t)(st.batch * 2)) % 16 == 0;
  };
  return io == kBF16 && a.N <= 128 && a.N % 8 == 0 && a.P % 8 == 0 && lies(a.x, a.xs) && lies(a.B, a.bs) && lies(a.C, a.cs);
}

int64_t delta_chain_groups(const DeltaArgs& a, int pass) { return delta_pieces(a) * a.H * blocks_of(a, pass); }

hipError_t launch_delta_chain(const DeltaArgs& a, int pass, hipStream_t s) {
  if (a.N <= 32) return pass == 1 ? launch_np<32, 1>(a, s) : launch_np<32, 0>(a, s);
  if (a.N <= 64) return pass == 1 ? launch_np<64, 1>(a, s) : launch_np<64, 0>(a, s);
  return pass == 1 ? launch_np<128, 1>(a, s) : launch_np<128, 0>(a, s);
}

}  // namespace ssd
