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
// reads by rows and the transposing ones meet few bank conflicts; the next
// block's are loaded into registers while a block is worked on.
//
// Roundings. S, R and U' = e^(g_end - g) U are held in fp32 and enter the
// products as two bf16 terms (2^-16; K is exact with bf16 io and two terms with
// fp32 io), so that states keep fp32's use over thousands of tokens. y's own
// products take one bf16 term of S, U and M with bf16 io, beside y's rounding.
#include "delta_blocks.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;  // rows p of a workgroup

template <typename TIO, int NP> struct BlockLds {
  static constexpr int TERMS = sizeof(TIO) == 4 ? 2 : 1;
  static constexpr int tile = 64 * NP * 2;  // K or Q, one term
  static constexpr int K = 0, Q = TERMS * tile, rec = 2 * TERMS * tile, X = rec + DeltaRecord<TERMS>::bytes,
                       bytes = X + 64 * kCols * (int)sizeof(TIO);
};

// Where the 16-byte piece c of row t lies in K's and in Q's tile.
template <int NP> __device__ __forceinline__ int k_swz(int t) {
  return NP >= 128 ? ((t & 3) << 2) | ((t >> 3) & 3) : NP == 64 ? ((t & 2) << 1) | ((t >> 3) & 3) : (t >> 3) & 3;
}
template <int NP> __device__ __forceinline__ int q_swz(int t) {
  return NP >= 128 ? ((t & 3) << 2) | ((t >> 2) & 3) : NP == 64 ? ((t & 2) << 1) | ((t >> 2) & 3) : (t >> 2) & 3;
}
__device__ __forceinline__ int x_swz(int t) { return (t & 2) | ((t >> 1) & 4); }

// Nothing but ordinary arithmetic is moved across.
__device__ __forceinline__ void hold() { __builtin_amdgcn_sched_barrier(0x6); }

template <typename TIO, int NP, bool WHOLE, int TERMS = BlockLds<TIO, NP>::TERMS>
__global__ __launch_bounds__(kThreads, NP <= 128 && TERMS == 1 ? 2 : 1) void delta_blocks_kernel(const DeltaArgs a, int blocks_p) {
  using L = BlockLds<TIO, NP>;
  using Rec = DeltaRecord<TERMS>;
  constexpr int KN = NP / 32;          // 32-column groups of N
  constexpr int PACKS = NP / 8;        // 16-byte pieces to a row
  constexpr int CK = 64 * PACKS / kThreads, CR = (Rec::bytes / 16 + kThreads - 1) / kThreads,
                CX = 64 * kCols * (int)sizeof(TIO) / 16 / kThreads, XP = 16 / (int)sizeof(TIO);
  __shared__ __align__(16) unsigned char lds[L::bytes];
  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, g = lane / 16, r = lane % 16;

  const int64_t bid = xcd_local_order(blockIdx.x, gridDim.x);
  const int pb = (int)(bid % blocks_p);
  const int64_t sh = bid / blocks_p;
  const int h = (int)(sh % a.H);
  const int64_t seq = sh / a.H;
  const int p0 = pb * kCols, pw = p0 + 16 * wave, p = pw + r;

  int64_t row = seq, first = 0, last = a.L, slot = seq * ((a.L + kDeltaBlock - 1) / kDeltaBlock);
  if (a.cu != nullptr) {
    row = 0, first = seq_offset(a.cu, seq, a.L), last = seq_offset(a.cu, seq + 1, a.L);
    slot = delta_first_slot(a, seq);
  }
  const int64_t grp = h / (a.H / a.G);
  const TIO* Xp = static_cast<const TIO*>(a.x) + row * a.xs.batch + (int64_t)h * a.P;
  const TIO* Bp = static_cast<const TIO*>(a.B) + row * a.bs.batch + grp * a.N;
  const TIO* Cp = static_cast<const TIO*>(a.C) + row * a.cs.batch + grp * a.N;
  TIO* Yp = static_cast<TIO*>(a.y) + (row * a.L * a.H + h) * a.P;

  // S^T: tile (kn, hh) rows 32 kn + 8 g + 4 hh .., column p
  f32x4_t S[KN][2];
  const int64_t state = (seq * a.H + h) * (int64_t)a.P + (p < a.P ? p : 0);
#pragma unroll
  for (int kn = 0; kn < KN; ++kn)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      S[kn][hh] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      const int n = 32 * kn + 8 * g + 4 * hh;
      if (a.init != nullptr && p < a.P && n < a.N) {
        const Pack<float, 4> v = load_pack<float, 4, true>(a.init + state * a.N + n, a.N - n);
#pragma unroll
        for (int i = 0; i < 4; ++i) S[kn][hh][i] = n + i < a.N ? v.v[i] : 0.f;
      }
    }

  // the next block on its way
  Piece<TIO> kq[2][CK];
  uint4 rc[CR], xv[CX];
  int kmoved, xmoved;
  const int kc = tid % PACKS, xc = tid % (kCols / XP);  // this thread's piece of a row
  const uint32_t kcol = piece_at<TIO, WHOLE>(8 * kc, a.N, kmoved);
  const uint32_t xcol = piece_at<TIO, WHOLE>(p0 + XP * xc, a.P, xmoved, XP);
  auto fetch = [&](int64_t t0, int64_t sl) {
    const int n = (int)(last - t0 < 64 ? last - t0 : 64);
    const __amdgpu_buffer_rsrc_t Br = block_rows(Bp + t0 * a.bs.token, a.bs.token, n, a.N),
                                 Cr = block_rows(Cp + t0 * a.cs.token, a.cs.token, n, a.N),
                                 Xr = block_rows(Xp + t0 * a.xs.token, a.xs.token, n, a.P),
                                 Rr = buffer_range(a.ws + (sl * a.H + h) * Rec::bytes, Rec::bytes);
#pragma unroll
    for (int j = 0; j < CK; ++j) {
      const int t = (j * kThreads + tid) / PACKS;
      kq[0][j] = load_piece<TIO>(Br, (uint32_t)(t * (int)a.bs.token) * (uint32_t)sizeof(TIO), kcol);
      kq[1][j] = load_piece<TIO>(Cr, (uint32_t)(t * (int)a.cs.token) * (uint32_t)sizeof(TIO), kcol);
    }
#pragma unroll
    for (int j = 0; j < CR; ++j) rc[j] = buffer_ld16(Rr, 16 * (j * kThreads + tid));
#pragma unroll
    for (int j = 0; j < CX; ++j) {
      const int t = (j * kThreads + tid) / (kCols / XP);
      const uint32_t off = (uint32_t)(t * (int)a.xs.token) * (uint32_t)sizeof(TIO) + xcol;
      xv[j] = buffer_ld16(Xr, xcol == kNowhere ? kNowhere : off);
    }
  };
  auto stage = [&] {
#pragma unroll
    for (int j = 0; j < CK; ++j) {
      const int t = (j * kThreads + tid) / PACKS, c = kc;
      move_piece<TIO, WHOLE>(kq[0][j], kmoved);
      move_piece<TIO, WHOLE>(kq[1][j], kmoved);
      unsigned char* kd = lds + L::K + t * (NP * 2) + 16 * (c ^ k_swz<NP>(t));
      unsigned char* qd = lds + L::Q + t * (NP * 2) + 16 * (c ^ q_swz<NP>(t));
      if constexpr (TERMS == 2) {
        uint4 hi, lo;
        split_piece(kq[0][j], hi, lo);
        st16(kd, hi), st16(kd + L::tile, lo);
        split_piece(kq[1][j], hi, lo);
        st16(qd, hi), st16(qd + L::tile, lo);
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
      const int t = (j * kThreads + tid) / (kCols / XP), c = xc;
      if constexpr (!WHOLE) {
        uint32_t w[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
        move_down<TIO, 4>(w, xmoved);
        xv[j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if constexpr (TERMS == 2) st16(lds + L::X + t * 256 + ((16 * c + 64 * ((t >> 3) & 3)) & 255), xv[j]);
      else st16(lds + L::X + t * 128 + 16 * (c ^ x_swz(t)), xv[j]);
    }
  };

  // this lane's operands in LDS
  const int rt = 8 * (r / 4) + r % 4;  // its row of a pair of tiles
  const int ta = r / 4, tb = r % 4;    // its row and piece of a transposing read
  const unsigned char* kbase = lds + L::K + rt * (NP * 2);
  const unsigned char* qbase = lds + L::Q + r * (NP * 2);
  const unsigned char* tbase = lds + L::K + (8 * g + ta) * (NP * 2);
  const int kf = k_swz<NP>(rt), qf = q_swz<NP>(r), tf = k_swz<NP>(8 * g + ta);
  const unsigned char* rec = lds + L::rec + 16 * lane;
  const float* eg = reinterpret_cast<const float*>(lds + L::rec + Rec::decays);
  const float* ed = eg + 64;
  auto kfrag = [&](int kk, int hh, int kn, int term) {
    return as_bf16x8(ld16(kbase + term * L::tile + (32 * kk + 4 * hh) * (NP * 2) + 16 * ((4 * kn + g) ^ kf)));
  };
  auto qfrag = [&](int tt, int kn, int term) {
    return as_bf16x8(ld16(qbase + term * L::tile + 16 * tt * (NP * 2) + 16 * ((4 * kn + g) ^ qf)));
  };
  auto ktfrag = [&](int kn, int hh, int kk, int term) {
    const unsigned char* s = tbase + term * L::tile + 32 * kk * (NP * 2) + 16 * ((4 * kn + tb) ^ tf) + 8 * hh;
    const uint2 lo = lds_tr8(s), hi = lds_tr8(s + 4 * (NP * 2));
    return as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
  };
  auto frag = [&](int at, int i) { return as_bf16x8(ld16(rec + at + i * kFragBytes)); };
  auto split_tiles = [&](const f32x4_t& t0, const f32x4_t& t1, bf16x8_t& hi, bf16x8_t& lo) {
    const float f[8] = {t0[0], t0[1], t0[2], t0[3], t1[0], t1[1], t1[2], t1[3]};
    uint4 vh, vl;
    split8(f, vh, vl);
    hi = as_bf16x8(vh), lo = as_bf16x8(vl);
  };

  bf16x8_t Sh[KN], Sl[KN];
#pragma unroll
  for (int kn = 0; kn < KN; ++kn) split_tiles(S[kn][0], S[kn][1], Sh[kn], Sl[kn]);

  const bool live = pw < a.P;
  if (first < last) fetch(first, slot);
  for (int64_t t0 = first; t0 < last; t0 += 64, ++slot) {
    __syncthreads();  // the last block's operands have been read
    stage();
    __syncthreads();
    if (t0 + 64 < last) fetch(t0 + 64, slot + 1);
    if (!live) continue;
    const int n = (int)(last - t0 < 64 ? last - t0 : 64);

    // Operands are read a group ahead of the products that use them, and the
    // order is held (hold()): the compiler by itself reads each right before its
    // use and waits for it.
    bf16x8_t f[2][4][TERMS];
    auto k_group = [&](bf16x8_t (&v)[4][TERMS], int kn) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < TERMS; ++e) v[i][e] = kfrag(i / 2, i % 2, kn, e);
    };
    auto q_group = [&](bf16x8_t (&v)[4][TERMS], int kn) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < TERMS; ++e) v[i][e] = qfrag(i, kn, e);
    };
    auto kt_group = [&](bf16x8_t (&v)[4][TERMS], int kn) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < TERMS; ++e) v[i][e] = ktfrag(kn, i % 2, i / 2, e);
    };
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};

    // K S0^T (rows t, column p) and S0 Q^T (rows p, column t)
    f32x4_t R[2][2] = {{zero, zero}, {zero, zero}}, O[4] = {zero, zero, zero, zero}, e[2][2];
    float x[2][2][4];
    uint2 xr[2][2];
    k_group(f[0], 0);
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      if (kn + 1 < KN) k_group(f[(kn + 1) % 2], kn + 1);
      else q_group(f[(kn + 1) % 2], 0);
      hold();
      auto& k = f[kn % 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) R[i / 2][i % 2] = mfma_16x16x32(k[i][0], Sh[kn], R[i / 2][i % 2]);
#pragma unroll
      for (int i = 0; i < 4; ++i) R[i / 2][i % 2] = mfma_16x16x32(k[i][0], Sl[kn], R[i / 2][i % 2]);
      if constexpr (TERMS == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) R[i / 2][i % 2] = mfma_16x16x32(k[i][1], Sh[kn], R[i / 2][i % 2]);
      }
      hold();
    }
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      if (kn + 1 < KN) {
        q_group(f[(KN + kn + 1) % 2], kn + 1);
      } else {
        // X by columns, and the decays
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            e[kk][hh] = *reinterpret_cast<const f32x4_t*>(eg + 32 * kk + 8 * g + 4 * hh);
            if constexpr (TERMS == 2) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[kk][hh][i] = *reinterpret_cast<const float*>(lds + L::X + (32 * kk + 8 * g + 4 * hh + i) * 256 +
                                                               ((4 * (16 * wave + r) + 64 * g) & 255));
            } else {
              const int t = 32 * kk + 8 * g + 4 * hh + ta;
              xr[kk][hh] = lds_tr8(lds + L::X + t * 128 + 16 * ((2 * wave + tb / 2) ^ x_swz(t)) + 8 * (tb & 1));
            }
          }
      }
      hold();
      auto& q = f[(KN + kn) % 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) O[i] = mfma_16x16x32(Sh[kn], q[i][0], O[i]);
      if constexpr (TERMS == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) O[i] = mfma_16x16x32(Sl[kn], q[i][0], O[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) O[i] = mfma_16x16x32(Sh[kn], q[i][1], O[i]);
      }
      hold();
    }
    // R = X - e^g K S0^T
    bf16x8_t th[kTriFrags], tl[kTriFrags];
#pragma unroll
    for (int i = 0; i < 2; ++i) th[i] = frag(Rec::T_hi, i), tl[i] = frag(Rec::T_lo, i);
    hold();
    bf16x8_t Rh[2], Rl[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        if constexpr (TERMS == 1) {
          const uint2 v = xr[kk][hh];
          x[kk][hh][0] = bf16_lo(v.x), x[kk][hh][1] = bf16_hi(v.x), x[kk][hh][2] = bf16_lo(v.y), x[kk][hh][3] = bf16_hi(v.y);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) R[kk][hh][i] = fmaf(-e[kk][hh][i], R[kk][hh][i], x[kk][hh][i]);
      }
      split_tiles(R[kk][0], R[kk][1], Rh[kk], Rl[kk]);
    }
    // U = T R
#pragma unroll
    for (int i = 2; i < kTriFrags; ++i) th[i] = frag(Rec::T_hi, i), tl[i] = frag(Rec::T_lo, i);
    hold();
    f32x4_t U[2][2] = {{zero, zero}, {zero, zero}};
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) U[0][hh] = mfma_16x16x32(th[hh], Rh[0], U[0][hh]);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) U[0][hh] = mfma_16x16x32(th[hh], Rl[0], U[0][hh]);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) U[0][hh] = mfma_16x16x32(tl[hh], Rh[0], U[0][hh]);
    hold();
    bf16x8_t mf[kTriFrags][TERMS];
    f32x4_t d[2][2];
    float er[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i / 2][i % 2] = *reinterpret_cast<const f32x4_t*>(ed + 32 * (i / 2) + 8 * g + 4 * (i % 2));
      er[i] = eg[16 * i + r];
    }
    const float end = eg[63];
    hold();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) U[1][hh] = mfma_16x16x32(th[tri_frag(1, hh, ks)], Rh[ks], U[1][hh]);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) U[1][hh] = mfma_16x16x32(th[tri_frag(1, hh, ks)], Rl[ks], U[1][hh]);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) U[1][hh] = mfma_16x16x32(tl[tri_frag(1, hh, ks)], Rh[ks], U[1][hh]);
    }
#pragma unroll
    for (int i = 0; i < kTriFrags; ++i)
#pragma unroll
      for (int k = 0; k < TERMS; ++k) mf[i][k] = frag(Rec::M, i + k * kTriFrags);
    hold();
    // Y^T = scale e^g S0 Q^T + U^T (scale M)^T, and U' = e^(g_end - g) U
    bf16x8_t Uh[2], Ul[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      if constexpr (TERMS == 2) {
        split_tiles(U[kk][0], U[kk][1], Uh[kk], Ul[kk]);
      } else {
        Uh[kk] = as_bf16x8(make_uint4(pack_bf16x2(U[kk][0][0], U[kk][0][1]), pack_bf16x2(U[kk][0][2], U[kk][0][3]),
                                      pack_bf16x2(U[kk][1][0], U[kk][1][1]), pack_bf16x2(U[kk][1][2], U[kk][1][3])));
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int i = 0; i < 4; ++i) U[kk][hh][i] *= d[kk][hh][i];
      split_tiles(U[kk][0], U[kk][1], Rh[kk], Rl[kk]);
    }
    kt_group(f[0], 0);
    hold();
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) O[tt][i] *= a.scale * er[tt];
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int tt = 2 * ks; tt < 4; ++tt) {
        const auto& mm = mf[tri_frag(tt / 2, tt % 2, ks)];
        O[tt] = mfma_16x16x32(Uh[ks], mm[0], O[tt]);
        if constexpr (TERMS == 2) {
          O[tt] = mfma_16x16x32(Ul[ks], mm[0], O[tt]);
          O[tt] = mfma_16x16x32(Uh[ks], mm[1], O[tt]);
        }
      }
    hold();
    // S^T <- e^g_end S^T + K^T U'
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) {
      if (kn + 1 < KN) kt_group(f[(kn + 1) % 2], kn + 1);
      hold();
      auto& k = f[kn % 2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[kn][hh][i] *= end;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) S[kn][hh] = mfma_16x16x32(k[2 * kk + hh][0], Rh[kk], S[kn][hh]);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) S[kn][hh] = mfma_16x16x32(k[2 * kk + hh][0], Rl[kk], S[kn][hh]);
        if constexpr (TERMS == 2) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) S[kn][hh] = mfma_16x16x32(k[2 * kk + hh][1], Rh[kk], S[kn][hh]);
        }
      }
      hold();
    }
#pragma unroll
    for (int kn = 0; kn < KN; ++kn) split_tiles(S[kn][0], S[kn][1], Sh[kn], Sl[kn]);
    // rows pw + 4 g .., column t = 16 tt + r
    const int pr = pw + 4 * g, pn = a.P - pr;
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      const int t = 16 * tt + r;
      if (t < n && pn > 0) {
        const float f[4] = {O[tt][0], O[tt][1], O[tt][2], O[tt][3]};
        store_pack<TIO, 4, true>(Yp + (t0 + t) * a.H * a.P + pr, f, pn);
      }
    }
  }

  if (a.final_state == nullptr || p >= a.P) return;
#pragma unroll
  for (int kn = 0; kn < KN; ++kn)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int n = 32 * kn + 8 * g + 4 * hh;
      const float f[4] = {S[kn][hh][0], S[kn][hh][1], S[kn][hh][2], S[kn][hh][3]};
      if (n < a.N) store_pack<float, 4, true>(a.final_state + state * a.N + n, f, a.N - n);
    }
}

template <typename TIO, int NP>
hipError_t launch_np(const DeltaArgs& a, hipStream_t s) {
  using L = BlockLds<TIO, NP>;
  static_assert(L::bytes <= 160 * 1024, "LDS of a compute unit");
  const int blocks_p = (a.P + kCols - 1) / kCols;
  const dim3 grid((unsigned)(a.seqs() * a.H * blocks_p));
  if (a.N % 8 == 0 && a.P % (16 / sizeof(TIO)) == 0) delta_blocks_kernel<TIO, NP, true><<<grid, kThreads, 0, s>>>(a, blocks_p);
  else delta_blocks_kernel<TIO, NP, false><<<grid, kThreads, 0, s>>>(a, blocks_p);
  return hipGetLastError();
}

template <typename TIO>
hipError_t launch_io(const DeltaArgs& a, hipStream_t s) {
  if (a.N <= 32) return launch_np<TIO, 32>(a, s);
  if (a.N <= 64) return launch_np<TIO, 64>(a, s);
  if (a.N <= 128) return launch_np<TIO, 128>(a, s);
  if constexpr (sizeof(TIO) == 2) return launch_np<TIO, 256>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace

bool delta_blocks_apply(const DeltaArgs& a, int io) {
  return (io == kBF16 || a.N <= 128) && a.L >= 16 && a.N >= 8 && a.P >= 8;
}
size_t delta_blocks_workspace(const DeltaArgs& a, int io) {
  return size_t(delta_slots(a)) * a.H * (io == kBF16 ? DeltaRecord<1>::bytes : DeltaRecord<2>::bytes);
}

hipError_t launch_delta_blocks(const DeltaArgs& a, int io, int dt, hipStream_t s) {
  const hipError_t e = launch_delta_solve(a, io, dt, s);
  if (e != hipSuccess) return e;
  return io == kBF16 ? launch_io<__hip_bfloat16>(a, s) : launch_io<float>(a, s);
}

}  // namespace ssd
