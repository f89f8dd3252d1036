// The gated delta rule in blocks, the walk over a sequence's blocks for rows that
// k_delta_chain.hip does not take: fp32, states of more than 128 columns, odd sizes
// and rows that are not aligned. (And the choice between them.)
//
// The same products in the same layouts. Each of four waves keeps 16 rows of the state.
// The next block's rows are loaded into registers while a block is worked on; on the way
// from there to the LDS odd rows are put in order and fp32 is split into terms.
//
// Where a workgroup has a compute unit to itself by its LDS (fp32 of N 33 to 64, bf16 of
// N > 128), and for fp32 of N <= 32, where two would fit, each wave has a partner, which brings
// the rows and makes y, as in k_delta_chain.hip: handed S0's terms and U in fp32. Elsewhere (bf16 of
// N <= 128, two workgroups and more to a compute unit, and fp32 of N > 64, no LDS left for S0 and
// U) the wave does it all. Measured without / with partners, both kernels: 3 sequences of 1001
// tokens, 32 heads, P = N = 64, fp32 118 / 102 us (the walk 85 / 69), of N = 32 87 / 74; 16384 tokens of
// 16 heads, P = 128, N = 256, bf16 716 / 617.
// Of their 256 registers the instances with partners spill, fp32 of N 33 to 64, 5 (18 at odd sizes), and
// those without, fp32 of N > 64 at odd sizes, 8.
//
// S, R and U' = e^(g_end - g) U are held in fp32. As operands they are terms
// (delta_blocks.h).
//
// Of the 69 us, 4.3 a block (10 000 cycles): rows to LDS 2400, K S0^T, R and U 3200 beside the
// partner's 4400 (half of them the issue of its loads), U' and the state 2800. Later or
// split issue of the loads, and terms made ahead of the LDS's turn, took 71 to 79.
#include <type_traits>

#include "delta_blocks.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;  // of the waves of either kind
constexpr int kCols = 64;  // rows p of a workgroup

template <typename TIO, int NP> struct Layout {
  static constexpr int IO = DeltaTerms<TIO>::io;
  static constexpr int tile = 64 * NP * 2;  // K or Q, one term
  static constexpr int xrow = kCols * (int)sizeof(TIO);
  static constexpr int K = 0, Q = IO * tile, rec = Q + IO * tile,
                       X = rec + (DeltaRecord<TIO>::bytes + 1023) / 1024 * 1024, bytes = X + 64 * xrow;
  // handed to the partners
  static constexpr int S0 = bytes, U = S0 + DeltaTerms<TIO>::y * kCols * NP * 2, two = U + 64 * kCols * 4;
};

// Likewise in (bf16) X's tile.
__device__ __forceinline__ int x_swz(int t) { return (t & 2) | ((t >> 1) & 4); }

// PASS: see delta_piece.
template <typename TIO, int NP, bool WHOLE, int PASS, bool TWO>
__global__ __launch_bounds__(TWO ? 2 * kThreads : kThreads) void delta_blocks_kernel(const DeltaArgs a, uint32_t blocks_p) {
  using L = Layout<TIO, NP>;
  using Rec = DeltaRecord<TIO>;
  constexpr int IO = DeltaTerms<TIO>::io, ST = DeltaTerms<TIO>::state, YT = DeltaTerms<TIO>::y;
  constexpr int KN = NP / 32;          // 32-column groups of N
  constexpr int PACKS = NP / 8;        // 16-byte pieces to a row of K
  constexpr int XP = 16 / (int)sizeof(TIO), XPACKS = kCols / XP;
  constexpr int CK = 64 * PACKS / kThreads, CR = (Rec::bytes / 16 + kThreads - 1) / kThreads, CX = 64 * XPACKS / kThreads;
  constexpr int SZ = (int)sizeof(TIO);
  constexpr bool Y = PASS == 0 && !TWO;  // whether the chain's waves make y
  constexpr int BYTES = TWO && PASS == 0 ? L::two : L::bytes;
  static_assert(BYTES <= 160 * 1024, "LDS of a compute unit");
  __shared__ __align__(16) unsigned char lds[BYTES];
  // (known to be the same in all lanes: the two kinds' barriers are then behind branches of the whole wave)
  const int any_wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x / 64), wave = any_wave % 4;
  const bool chain = !TWO || any_wave < 4;
  const int tid = threadIdx.x % kThreads, lane = tid % 64, g = lane / 16, r = lane % 16;

  // (32-bit divisions: those of 64 bits took a microsecond each)
  const uint32_t bid = (uint32_t)xcd_local_order(blockIdx.x, gridDim.x);
  const uint32_t sh = bid / blocks_p;
  const int pb = (int)(bid - sh * blocks_p);
  const int64_t piece = sh / (uint32_t)a.H;
  const int h = (int)(sh - (uint32_t)piece * a.H);
  const int p0 = pb * kCols, pw = p0 + 16 * wave, p = pw + r;  // this wave's rows, this lane's

  DeltaSlot sl;
  if (!delta_piece<PASS>(a, piece, sl)) return;
  const int64_t row = sl.row, first = sl.t0, last = sl.t1;
  int64_t slot = delta_first_slot(a, sl.index, kDeltaBlock) + (first - sl.first) / kDeltaBlock;
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
  Piece<TIO> kq[2][CK];
  uint4 rc[CR], xv[CX];
  int kmoved, xmoved;
  const int kc = tid % PACKS, xc = tid % XPACKS;  // this thread's piece of a row
  const uint32_t kcol = piece_at<TIO, WHOLE>(8 * kc, a.N, kmoved);
  const uint32_t xcol = piece_at<TIO, WHOLE>(p0 + XP * xc, a.P, xmoved, XP);
  auto fetch = [&](int64_t t0, int64_t sl) {
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
  };
  auto stage = [&] {
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
  };

  // ---- this lane's operands in LDS
  const int rt = 8 * (r / 4) + r % 4;  // its row of a pair of tiles
  const int ta = r / 4, tb = r % 4;    // its row and piece of a transposing read
  const int kat = rt * (NP * 2), tat = L::K + (8 * g + ta) * (NP * 2);
  const int kf = k_swz<NP>(rt), tf = k_swz<NP>(8 * g + ta);

  const bool live = pw < rows_p;
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  auto split_tiles = [&](auto terms, const f32x4_t& t0, const f32x4_t& t1) {
    const float f[8] = {t0[0], t0[1], t0[2], t0[3], t1[0], t1[1], t1[2], t1[3]};
    return split8<decltype(terms)::value>(f);
  };
  constexpr std::integral_constant<int, ST> st_terms{};
  constexpr std::integral_constant<int, YT> y_terms{};
  const float* eg = reinterpret_cast<const float*>(lds + L::rec + Rec::decays);
  const float* ed = eg + 64;
  auto by_rows = [&](const unsigned char* from, int i, int kn) {  // rows of tile i, columns 32 kn ..
    Terms<IO> v;
#pragma unroll
    for (int e = 0; e < IO; ++e)
      v.v[e] = as_bf16x8(ld16(from + kat + e * L::tile + (32 * (i / 2) + 4 * (i % 2)) * (NP * 2) + 16 * ((4 * kn + g) ^ kf)));
    return v;
  };
  auto kfrag = [&](int i, int kn) { return by_rows(lds + L::K, i, kn); };
  auto qfrag = [&](int i, int kn) { return by_rows(lds + L::Q, i, kn); };
  auto ktfrag = [&](int hh, int kk, int kn) {  // tile hh of columns 32 kn .., rows 32 kk ..
    Terms<IO> v;
#pragma unroll
    for (int e = 0; e < IO; ++e) {
      const unsigned char* s = lds + L::K + tat + e * L::tile + 32 * kk * (NP * 2) + 16 * ((4 * kn + tb) ^ tf) + 8 * hh;
      const uint2 lo = lds_tr8(s), hi = lds_tr8(s + 4 * (NP * 2));
      v.v[e] = as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
    }
    return v;
  };
  auto tri = [&](auto terms, int from, int i) {
    Terms<decltype(terms)::value> v;
#pragma unroll
    for (int e = 0; e < decltype(terms)::value; ++e)
      v.v[e] = as_bf16x8(ld16(lds + L::rec + 16 * lane + from + (e * kTriFrags + i) * kFragBytes));
    return v;
  };
  // y of the block from t0 on: rows pw + 4 g .. of a lane at token 32 (i / 2) + 4 (i % 2) + rt
  auto put_y = [&](const f32x4_t (&O)[4], int64_t t0) {
    const int n = (int)(last - t0 < 64 ? last - t0 : 64);
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
  unsigned char* const s_place = lds + L::S0 + wave * KN * YT * kFragBytes + 16 * lane;
  unsigned char* const u_place = lds + L::U + wave * 4096 + 16 * lane;

  if constexpr (TWO) {
    if (!chain) {
      // ---- the partners: rows to LDS, and y
      if (first < last) fetch(first, slot);
      for (int64_t t0 = first; t0 < last; t0 += 64, ++slot) {
        __syncthreads();  // the last block's operands have been read
        stage();
        __syncthreads();
        if (t0 + 64 < last) fetch(t0 + 64, slot + 1);
        f32x4_t O[4];
        if constexpr (PASS == 0) {
          // S0 Q^T (rows p, column t) scale e^g
          Terms<IO> q[2][4];
          Terms<YT> s[2];
          auto group = [&](int b, int kn) {
#pragma unroll
            for (int i = 0; i < 4; ++i) q[b][i] = qfrag(i, kn);
#pragma unroll
            for (int e = 0; e < YT; ++e) s[b].v[e] = as_bf16x8(ld16(s_place + (kn * YT + e) * kFragBytes));
          };
#pragma unroll
          for (int i = 0; i < 4; ++i) O[i] = zero;
          group(0, 0);
#pragma unroll
          for (int kn = 0; kn < KN; ++kn) {
            if (kn + 1 < KN) group((kn + 1) % 2, kn + 1);
            hold();
#pragma unroll
            for (int pair = 0; pair < term_pairs(YT, IO); ++pair)
#pragma unroll
              for (int i = 0; i < 4; ++i) mul_pair(O[i], s[kn % 2], q[kn % 2][i], pair);
            hold();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = a.scale * eg[32 * (i / 2) + 4 * (i % 2) + rt];
#pragma unroll
            for (int k = 0; k < 4; ++k) O[i][k] *= e;
          }
        }
        __syncthreads();  // U is there
        if constexpr (PASS == 0) {
          // + U^T (scale M)^T
          Terms<YT> mf[kTriFrags], Uy[2];
          f32x4_t U[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) U[i] = *reinterpret_cast<const f32x4_t*>(u_place + i * 1024);
#pragma unroll
          for (int i = 0; i < kTriFrags; ++i) mf[i] = tri(y_terms, Rec::M, i);
          hold();
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) Uy[kk] = split_tiles(y_terms, U[2 * kk], U[2 * kk + 1]);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int pair = 0; pair < term_pairs(YT, YT); ++pair)
#pragma unroll
              for (int i = 2 * ks; i < 4; ++i) mul_pair(O[i], Uy[ks], mf[tri_frag(i / 2, i % 2, ks)], pair);
          // (a wave without rows reads what no wave wrote and stores nothing)
          put_y(O, t0);
        }
      }
      return;
    }
    if (!live) {
      for (int64_t t0 = first; t0 < last; t0 += 64) {
        __syncthreads();
        __syncthreads();
        __syncthreads();
      }
      return;
    }
  } else {
    if (first < last) fetch(first, slot);
  }

  // S^T: tile (kn, hh) rows 32 kn + 8 g + 4 hh .., column p
  f32x4_t S[KN][2];
  Terms<ST> Sv[KN];
  const int64_t states = (a.seg != 0 ? piece : sl.seq) * a.H + h;
  const float* init = PASS == 1 ? nullptr : a.seg != 0 ? a.enter : a.init;
  auto state_at = [&](int64_t of) { return (of * rows_p + (p < rows_p ? p : 0)) * a.N; };
#pragma unroll
  for (int kn = 0; kn < KN; ++kn) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      S[kn][hh] = zero;
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
  auto hand_over_s = [&] {
#pragma unroll
    for (int kn = 0; kn < KN && TWO && PASS == 0; ++kn)
#pragma unroll
      for (int e = 0; e < YT; ++e) st16(s_place + (kn * YT + e) * kFragBytes, __builtin_bit_cast(uint4, Sv[kn].v[e]));
  };
  hand_over_s();

  for (int64_t t0 = first; t0 < last; t0 += 64, ++slot) {
    __syncthreads();  // the last block's operands have been read
    if constexpr (!TWO) stage();
    __syncthreads();
    if constexpr (!TWO) {
      if (t0 + 64 < last) fetch(t0 + 64, slot + 1);
      if (!live) continue;
    }

    auto of_y = [&](const Terms<ST>& s) {
      Terms<YT> v;
#pragma unroll
      for (int e = 0; e < YT; ++e) v.v[e] = s.v[e];
      return v;
    };

    // Operands are read a group ahead of the products that use them, and the
    // order is held: the compiler by itself reads each right before its use and
    // waits for it.
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
        for (int i = 0; i < 4 && Y; ++i) f[(kn + 1) % 2][i] = qfrag(i, 0);
        // X by columns, and the decays
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tr = 32 * (i / 2) + 8 * g + 4 * (i % 2);
          e[i] = *reinterpret_cast<const f32x4_t*>(eg + tr);
          if constexpr (SZ == 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              xw[i][k] = *reinterpret_cast<const float*>(lds + L::X + (tr + k) * L::xrow + ((4 * (16 * wave + r) + 64 * g) & 255));
          } else {
            const int t = tr + ta;
            xr[i] = lds_tr8(lds + L::X + t * L::xrow + 16 * ((2 * wave + tb / 2) ^ x_swz(t)) + 8 * (tb & 1));
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
    }
    // S0 Q^T (rows p, column t); beside it R = X - e^g K S0^T
    Terms<ST> Rv[2];
    Terms<ST> tm[kTriFrags];
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      if (Y && kn + 1 < KN) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[(KN + kn + 1) % 2][i] = qfrag(i, kn + 1);
      }
#pragma unroll
      for (int i = 0; i < kTriFrags; ++i)
        if (i * KN / kTriFrags == kn) tm[i] = tri(st_terms, Rec::T, i);
      hold();
#pragma unroll
      for (int pair = 0; pair < term_pairs(YT, IO) && Y; ++pair)
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
    // U = T R; beside it O e^g
    f32x4_t U[4], d[4];
    float er[4];
    Terms<YT> mf[kTriFrags], Uy[2];
#pragma unroll
    for (int i = 0; i < 4 && Y; ++i) er[i] = eg[32 * (i / 2) + 4 * (i % 2) + rt];
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
    for (int i = 0; i < 4 && Y; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) O[i][k] *= a.scale * er[i];
    spread<6 * term_pairs(ST, ST), 2>();
    hold();
#pragma unroll
    for (int i = 0; i < kTriFrags && Y; ++i) mf[i] = tri(y_terms, Rec::M, i);
    if constexpr (TWO) {
#pragma unroll
      for (int i = 0; i < 4 && PASS == 0; ++i) *reinterpret_cast<f32x4_t*>(u_place + i * 1024) = U[i];
      __syncthreads();  // U is there
    }
    hold();
    // operands of y, and U' = e^(g_end - g) U
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      if constexpr (Y) Uy[kk] = split_tiles(y_terms, U[2 * kk], U[2 * kk + 1]);
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
      for (int pair = 0; pair < term_pairs(YT, YT) && Y; ++pair)
#pragma unroll
        for (int i = 2 * ks; i < 4; ++i) mul_pair(O[i], Uy[ks], mf[tri_frag(i / 2, i % 2, ks)], pair);
    hold();
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
      if (Y && kn == 0) put_y(O, t0);
    }
    Sv[KN - 1] = split_tiles(st_terms, S[KN - 1][0], S[KN - 1][1]);
    hand_over_s();
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

uint32_t blocks_of(const DeltaArgs& a, int pass) { return (delta_rows(a, pass) + kCols - 1) / kCols; }
int64_t groups_of(const DeltaArgs& a, int pass) { return delta_pieces(a) * a.H * blocks_of(a, pass); }

template <typename TIO, int NP, int PASS>
hipError_t launch_pass(const DeltaArgs& a, hipStream_t s) {
  const uint32_t blocks_p = blocks_of(a, PASS);
  // Waves of two kinds (the file's head has the sizes and both sides' times).
  constexpr bool TWO = sizeof(TIO) == 4 ? NP <= 64 : NP == 256;
  constexpr int threads = TWO ? 2 * kThreads : kThreads;
  auto go = [&](auto kern) {
    kern<<<dim3((unsigned)groups_of(a, PASS)), threads, 0, s>>>(a, blocks_p);
    return hipGetLastError();
  };
  const bool whole = a.N % 8 == 0 && a.P % (16 / sizeof(TIO)) == 0;
  return whole ? go(delta_blocks_kernel<TIO, NP, true, PASS, TWO>) : go(delta_blocks_kernel<TIO, NP, false, PASS, TWO>);
}

template <typename TIO, int PASS>
hipError_t launch_io(const DeltaArgs& a, hipStream_t s) {
  if (a.N <= 32) return launch_pass<TIO, 32, PASS>(a, s);
  if (a.N <= 64) return launch_pass<TIO, 64, PASS>(a, s);
  if (a.N <= 128) return launch_pass<TIO, 128, PASS>(a, s);
  if constexpr (sizeof(TIO) == 2) return launch_pass<TIO, 256, PASS>(a, s);
  return hipErrorInvalidValue;
}

template <int PASS> hipError_t launch_walk(const DeltaArgs& a, int io, hipStream_t s) {
  if (delta_chain_applies(a, io)) return launch_delta_chain(a, PASS, s);
  return io == kBF16 ? launch_io<__hip_bfloat16, PASS>(a, s) : launch_io<float, PASS>(a, s);
}

// Tokens of a segment, 0 where sequences are walked in one piece. A sequence's
// blocks depend on one another; where all rows, heads and columns give fewer workgroups
// than the card has compute units, the time axis is cut: a first walk gives what each segment
// makes of any state (P + N rows instead of P, without y, about 3/4 of a block's time
// a row), the states are joined in turn, and the segments are walked side by side.
// In quarters of a block's time on a compute unit; a join takes about a block's.
// Of packed sequences only the number is known here: the stream is taken for so many
// of four times their mean length. A pack of one long sequence and many short ones is then
// not cut: 16384 tokens and 36 sequences of one, 32 heads, P = N = 128, 816 us, where the prompt alone
// takes 395. Cut as if one sequence could be all of the stream (with states of sequences of one
// segment read where they lie) it took 1178, 16 sequences of 512 113 -> 131 and 200 of 40 338 -> 536:
// the other sequences' workgroups that find nothing to do cost more than the cut gives.
int64_t delta_segment(const DeltaArgs& a, int io) {
  int64_t tokens = a.L, seqs = a.batch;
  if (a.nseq > 0) tokens = 4 * ((a.L + a.nseq - 1) / a.nseq) < a.L ? 4 * ((a.L + a.nseq - 1) / a.nseq) : a.L, seqs = (a.L + tokens - 1) / tokens;
  const bool pairs = io == kBF16 && a.N <= 128;  // of 64 columns, in the walk for aligned rows
  const int64_t cols = pairs && a.P > 64 ? 128 : 64, cols1 = pairs ? 128 : 64;
  const int64_t wgs = seqs * a.H * ((a.P + cols - 1) / cols), first = seqs * a.H * ((a.P + a.N + cols1 - 1) / cols1);
  const int64_t blocks = (tokens + kDeltaBlock - 1) / kDeltaBlock, cus = 256;
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

// Which of a packed stream's sequences have more than a.upto tokens: one workgroup
// goes over the offsets.
constexpr int kPick = 1024, kEach = 4;  // threads, and sequences of each at a time
__global__ __launch_bounds__(kPick) void delta_pick_kernel(const DeltaArgs a, int64_t room) {
  __shared__ int counts[kPick / 64];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  int64_t found = 0;
  for (int64_t s0 = 0; s0 < a.nseq; s0 += kPick * kEach) {
    // (a wave's sequences lie behind one another, a lane's 64 apart)
    const int64_t mine = s0 + wave * (64 * kEach) + lane;
    uint64_t is_long[kEach];
    int n = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int64_t s = mine + 64 * k;
      is_long[k] = __ballot(s < a.nseq && seq_offset(a.cu, s + 1, a.L) - seq_offset(a.cu, s, a.L) > a.upto);
      n += __popcll(is_long[k]);
    }
    if (lane == 0) counts[wave] = n;
    __syncthreads();
    int64_t at = found;
#pragma unroll
    for (int w = 0; w < kPick / 64; ++w) {
      if (w < wave) at += counts[w];
      found += counts[w];
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int64_t i = at + __popcll(is_long[k] & ((uint64_t(1) << lane) - 1));
      // (offsets that do not rise may have more than there is room for)
      if ((is_long[k] >> lane & 1) != 0 && i < room) a.longs[i] = (int32_t)(mine + 64 * k);
      at += __popcll(is_long[k]);
    }
    __syncthreads();
  }
  for (int64_t i = found + threadIdx.x; i < room; i += kPick) a.longs[i] = -1;
}

// What either form takes, in microseconds, by a fit to 446 measured calls: 2 to 32 heads of 8 x 8 to
// 128 x 256, 3 to 16 384 sequences of 1 to 2048 tokens, even ones and one long among ones of a
// token (root mean square of the error: the walk's 17%, the blocks' 10 to 14%). The walk: the tokens of the
// longest sequence in turn, or, where the card is full, all tokens' updates and the states, in and
// out. The blocks: two launches and the blocks of the longest sequence in turn, or a record
// and a block's products for every block and head.
struct Times {
  double start, token, full;       // token after token
  double latency, block, records;  // in blocks
  double walk(double longest) const { return start + (full > token * longest ? full : token * longest); }
  double blocks(double longest) const {
    const double turn = latency + block * longest / kDeltaBlock;
    return turn > records ? turn : records;
  }
};
Times times_of(const DeltaArgs& a, int io) {
  const bool packed = a.nseq > 0, odd = a.N % 4 != 0;
  const bool chain = io == kBF16 && a.N <= 128 && a.N % 8 == 0 && a.P % 8 == 0;
  const double state = (double)a.P * a.N, tokens = (double)a.batch * a.L;
  const double blocks = packed ? (double)(a.L / kDeltaBlock + a.nseq) : (double)a.batch * ((a.L + kDeltaBlock - 1) / kDeltaBlock);
  const double update = state > 2000 ? state * 3e-7 : 6e-4;
  Times t;
  const double search = packed ? 2 : 0;  // for a slot's sequence
  t.start = 5, t.token = odd ? 0.75 : 0.27 + 8.5e-4 * a.N;
  t.full = a.H * (tokens * (odd ? 2.7 : 1.) * update + a.seqs() * state * 2e-6);
  if (chain) {
    t.latency = search + 6.5 + 0.078 * a.N, t.block = 0.63 + 0.016 * a.N, t.records = 11 + blocks * a.H * (0.013 + 1.6e-6 * state);
  } else if (io != kBF16) {
    t.latency = search + 7.4 + 0.255 * a.N, t.block = 0.85 + 0.041 * a.N, t.records = 15 + blocks * a.H * (0.025 + 5.2e-6 * state);
  } else {
    t.latency = search + 11.3 + 0.062 * a.N, t.block = 2.5 + 0.013 * a.N, t.records = 14 + blocks * a.H * (0.0033 + 5e-6 * state);
  }
  return t;
}

}  // namespace

// The form that takes less: of the 446 calls the batched ones take 1.00 of the faster form's time in the
// geometric mean. Of packed sequences the host knows the mean length alone, and takes the
// longest for twice that. Where token after token is then the faster one, and there are tokens
// enough for a sequence that it would be slow for, the choice is made sequence by
// sequence where the lengths are known: those that take longer token after token than in
// blocks, were they alone, go in blocks, at the price of three launches (9 us) that find
// nothing to do where there are none. Measured, all token after token / all in blocks / each
// in its own form: 2048 tokens and 255 sequences of one, fp32, 8 heads of 64 x 64 659 / 162 / 170, bf16, 16 heads of
// 128 x 256 1643 / 956 / 509; 256 sequences of 4 tokens, fp32, 8 heads of 64 x 64 28 / 110 / 36, 2 heads of
// 32 x 32 7.3 / 31 / 16.5.
bool delta_blocks_apply(DeltaArgs& a, int io) {
  a.upto = 0;
  if ((io != kBF16 && a.N > 128) || a.N < 8 || a.P < 8) return false;
  const Times t = times_of(a, io);
  const double mean2 = a.nseq > 0 ? 2. * a.L / a.nseq : (double)a.L, longest = mean2 < a.L ? mean2 : (double)a.L;
  const double walk = t.walk(longest), blocks = t.blocks(longest), launches = 8;
  if (blocks < walk) return true;
  const int64_t upto = (int64_t)((t.latency + launches - t.start) / (t.token - t.block / kDeltaBlock));
  if (a.nseq == 0 || a.L <= 4 * upto) return false;
  if (blocks > walk + launches) a.upto = upto;
  return true;
}

int64_t delta_blocks_workspace(DeltaArgs& a, int io) {
  const int64_t records = delta_slots(a) * a.H * (int64_t)record_bytes(io);
  if (a.upto > 0) return records + delta_seqs_in_blocks(a) * (int64_t)sizeof(int32_t);
  a.seg = delta_segment(a, io);
  if (a.seg == 0) return records;
  const int64_t states = delta_slots(a, a.seg) * a.H;
  return records + states * (2 * a.P + a.N) * a.N * (int64_t)sizeof(float);
}

bool delta_blocks_fit(const DeltaArgs& a, int io) {
  // (twice kThreads: as with partners)
  auto walks = [&](int pass) {
    return grid_fits(groups_of(a, pass), 2 * kThreads) && (io != kBF16 || grid_fits(delta_chain_groups(a, pass), 2 * kThreads));
  };
  if (a.upto > 0 && !delta_walk_fits(a)) return false;
  return grid_fits(delta_solve_groups(a), kThreads) && walks(0) && (a.seg == 0 || (walks(1) && grid_fits(delta_join_groups(a), kThreads)));
}

hipError_t launch_delta_blocks(const DeltaArgs& args, int io, int dt, hipStream_t s) {
  DeltaArgs a = args;
  if (a.seg != 0) {
    const int64_t states = delta_slots(a, a.seg) * a.H;
    a.ends = reinterpret_cast<float*>(a.ws + delta_slots(a) * a.H * (int64_t)record_bytes(io));
    a.enter = a.ends + states * (a.P + a.N) * a.N;
  }
  if (a.upto > 0) {
    a.longs = reinterpret_cast<int32_t*>(a.ws + delta_slots(a) * a.H * (int64_t)record_bytes(io));
    delta_pick_kernel<<<1, kPick, 0, s>>>(a, delta_seqs_in_blocks(a));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipError_t e = launch_delta_solve(a, io, dt, s);
  if (e == hipSuccess && a.seg != 0) {
    e = launch_walk<1>(a, io, s);
    if (e == hipSuccess) e = launch_delta_join(a, s);
  }
  if (e == hipSuccess) e = launch_walk<0>(a, io, s);
  return e == hipSuccess && a.upto > 0 ? launch_delta_walk(a, io, dt, s) : e;
}

}  // namespace ssd
