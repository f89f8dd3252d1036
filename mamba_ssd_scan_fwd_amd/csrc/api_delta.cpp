// C ABI of the gated delta rule and of the norm of heads. Argument validation
// and launch only; no HIP call is made before every argument is checked.
#include <cstdint>

#include "delta.h"
#include "layer_checks.h"

namespace ssd {
namespace {

struct DeltaPlan {
  DeltaArgs a;
  int io, dt;
  int64_t x_ext, dt_ext, e_ext, b_ext, c_ext;  // extents in elements
  bool blocks;                                 // in blocks, or token after token
  size_t total;                                // workspace
};

// nseq 0: batched.
ssd_status_t plan_delta(const ssd_delta_desc_t* d, int64_t nseq, DeltaPlan* p) {
  if (d == nullptr) return SSD_ERR_NULL_POINTER;
  if (d->batch < 1 || d->seqlen < 1 || d->nheads < 1 || d->headdim < 1 || d->dstate < 1 || d->ngroups < 1)
    return SSD_ERR_BAD_SHAPE;
  if (d->nheads > 65535 || d->nheads % d->ngroups != 0) return SSD_ERR_BAD_SHAPE;
  if (d->batch >= kMaxRows || d->seqlen >= kMaxRows || nseq >= kMaxRows) return SSD_ERR_BAD_SHAPE;
  if (d->headdim > kDeltaMaxDim || d->dstate > kDeltaMaxDim) return SSD_ERR_UNSUPPORTED;
  if (!io_of(d->io_dtype, &p->io) || !io_of(d->dt_dtype, &p->dt)) return SSD_ERR_UNSUPPORTED;
  if (p->dt != kF32 && p->dt != p->io) return SSD_ERR_UNSUPPORTED;
  if (d->dt_clamp && !(d->dt_min <= d->dt_max)) return SSD_ERR_BAD_SHAPE;
  if (!aligned(d->dt_bias, 4)) return SSD_ERR_ALIGNMENT;
  const int64_t H = d->nheads, HP = H * d->headdim, GN = d->ngroups * d->dstate;
  if (HP > kMaxChannels || GN > kMaxChannels) return SSD_ERR_BAD_SHAPE;
  DeltaArgs& a = p->a;
  if (!resolve(d->x_stride, d->batch, d->seqlen, HP, &a.xs, &p->x_ext) ||
      !resolve(d->dt_stride, d->batch, d->seqlen, H, &a.ds, &p->dt_ext) ||
      !resolve(d->beta_stride, d->batch, d->seqlen, H, &a.es, &p->e_ext) ||
      !resolve(d->B_stride, d->batch, d->seqlen, GN, &a.bs, &p->b_ext) ||
      !resolve(d->C_stride, d->batch, d->seqlen, GN, &a.cs, &p->c_ext))
    return SSD_ERR_BAD_SHAPE;
  const int64_t rows = nseq > d->batch ? nseq : d->batch;
  if (rows > kMaxElems / (HP * d->dstate)) return SSD_ERR_BAD_SHAPE;
  // a workgroup per row, head and, at the finest, row of the state: a grid's limit
  if (rows > (kMaxRows - 1) / HP) return SSD_ERR_BAD_SHAPE;
  a.batch = d->batch, a.L = d->seqlen;
  a.H = (int)H, a.P = (int)d->headdim, a.N = (int)d->dstate, a.G = (int)d->ngroups;
  a.nseq = nseq;
  a.dto = DtOpts{d->dt_bias, d->dt_softplus != 0, d->dt_clamp != 0, d->dt_min, d->dt_max};
  a.sigmoid = d->beta_sigmoid != 0;
  a.scale = d->scale;
  a.seg = a.upto = 0;
  a.longs = nullptr;
  return SSD_OK;
}

// The prompt form: the way it is walked (token after token too where the form in
// blocks has more workgroups than can be launched), and the workspace that needs.
ssd_status_t plan_rule(const ssd_delta_desc_t* d, int64_t nseq, DeltaPlan* p) {
  const ssd_status_t st = plan_delta(d, nseq, p);
  if (st != SSD_OK) return st;
  p->blocks = false;
  p->total = 0;
  if (delta_blocks_apply(p->a, p->io)) {
    const int64_t bytes = delta_blocks_workspace(p->a, p->io);
    p->blocks = bytes <= kMaxElems && delta_blocks_fit(p->a, p->io);
    if (p->blocks) p->total = size_t(bytes);
    else p->a.upto = 0;
  }
  return p->blocks || delta_walk_fits(p->a) ? SSD_OK : SSD_ERR_BAD_SHAPE;
}

ssd_status_t run_rule(DeltaPlan& p, const int32_t* cu, const void* x, const void* dt, const float* A, const void* B,
                      const void* C, const void* beta, const float* init, void* y, float* final_state, void* workspace,
                      size_t workspace_bytes, hipStream_t s) {
  DeltaArgs& a = p.a;
  const size_t io = bytes_of(p.io), dts = bytes_of(p.dt);
  if (!x || !dt || !A || !B || !C || !beta || !y) return SSD_ERR_NULL_POINTER;
  if (!aligned(x, io) || !aligned(dt, dts) || !aligned(A, 4) || !aligned(B, io) || !aligned(C, io) ||
      !aligned(beta, dts) || !aligned(init, 4) || !aligned(y, io) || !aligned(final_state, 4) || !aligned(cu, 4) ||
      !aligned(workspace, kWsAlign))
    return SSD_ERR_ALIGNMENT;
  if (workspace != nullptr && workspace_bytes < p.total) return SSD_ERR_WORKSPACE;
  const size_t st_bytes = size_t(a.seqs() * a.H * a.P * a.N) * sizeof(float);
  const Range in[] = {range_of(x, size_t(p.x_ext) * io),     range_of(dt, size_t(p.dt_ext) * dts),
                      range_of(beta, size_t(p.e_ext) * dts), range_of(A, size_t(a.H) * sizeof(float)),
                      range_of(B, size_t(p.b_ext) * io),     range_of(C, size_t(p.c_ext) * io),
                      range_of(cu, cu != nullptr ? size_t(a.nseq + 1) * sizeof(int32_t) : 0),
                      range_of(a.dto.bias, size_t(a.H) * sizeof(float))};
  const Range ri = range_of(init, st_bytes), rf = range_of(final_state, st_bytes);
  const Range ry = range_of(y, size_t(a.batch * a.L * a.H * a.P) * io);
  const Range rw = range_of(workspace, p.total);
  if (overlaps_any(ry, in) || overlaps_any(rf, in) || overlaps_any(rw, in)) return SSD_ERR_ALIAS;
  if (overlap(ry, ri) || overlap(ry, rf) || overlap(ry, rw) || overlap(rw, ri) || overlap(rw, rf)) return SSD_ERR_ALIAS;
  if (overlap(rf, ri) && rf.lo != ri.lo) return SSD_ERR_ALIAS;  // the same array or none of it
  a.x = x, a.dt = dt, a.A = A, a.B = B, a.C = C, a.beta = beta, a.init = init, a.y = y, a.final_state = final_state;
  a.cu = cu;
  if (!p.blocks) return from_hip(launch_delta_walk(a, p.io, p.dt, s));
  void* w = workspace;
  if (w == nullptr && hipMallocAsync(&w, p.total, s) != hipSuccess) return SSD_ERR_HIP;
  a.ws = static_cast<char*>(w);
  hipError_t e = launch_delta_blocks(a, p.io, p.dt, s);
  if (workspace == nullptr) {
    const hipError_t fe = hipFreeAsync(w, s);
    if (e == hipSuccess) e = fe;
  }
  return from_hip(e);
}

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status_t ssd_delta_rule_workspace_bytes(const ssd_delta_desc_t* desc, int64_t num_seqs, size_t* bytes) {
  if (bytes == nullptr) return SSD_ERR_NULL_POINTER;
  if (num_seqs < 0) return SSD_ERR_BAD_SHAPE;
  ssd::DeltaPlan p;
  const ssd_status_t st = ssd::plan_rule(desc, num_seqs, &p);
  if (st != SSD_OK) return st;
  if (num_seqs > 0 && desc->batch != 1) return SSD_ERR_BAD_SHAPE;
  *bytes = p.total;
  return SSD_OK;
}

ssd_status_t ssd_delta_rule(const ssd_delta_desc_t* desc, const void* x, const void* dt, const float* A, const void* B,
                            const void* C, const void* beta, const float* init_state, void* y, float* final_state,
                            void* workspace, size_t workspace_bytes, void* stream) {
  ssd::DeltaPlan p;
  const ssd_status_t st = ssd::plan_rule(desc, 0, &p);
  if (st != SSD_OK) return st;
  return ssd::run_rule(p, nullptr, x, dt, A, B, C, beta, init_state, y, final_state, workspace, workspace_bytes,
                       static_cast<hipStream_t>(stream));
}

ssd_status_t ssd_delta_rule_varlen(const ssd_delta_desc_t* desc, const int32_t* cu_seqlens, int64_t num_seqs,
                                   const void* x, const void* dt, const float* A, const void* B, const void* C,
                                   const void* beta, const float* init_states, void* y, float* final_states,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  ssd::DeltaPlan p;
  if (num_seqs < 1) return desc == nullptr ? SSD_ERR_NULL_POINTER : SSD_ERR_BAD_SHAPE;
  const ssd_status_t st = ssd::plan_rule(desc, num_seqs, &p);
  if (st != SSD_OK) return st;
  if (desc->batch != 1) return SSD_ERR_BAD_SHAPE;
  if (cu_seqlens == nullptr) return SSD_ERR_NULL_POINTER;
  return ssd::run_rule(p, cu_seqlens, x, dt, A, B, C, beta, init_states, y, final_states, workspace, workspace_bytes,
                       static_cast<hipStream_t>(stream));
}

ssd_status_t ssd_delta_step(const ssd_delta_desc_t* desc, const void* x, const void* dt, const float* A, const void* B,
                            const void* C, const void* beta, float* state, const int32_t* state_slots,
                            int64_t num_slots, void* y, void* stream) {
  using namespace ssd;
  DeltaPlan p;
  const ssd_status_t st = plan_delta(desc, 0, &p);
  if (st != SSD_OK) return st;
  if (desc->seqlen != 1 || num_slots < 1 || num_slots >= kMaxRows) return SSD_ERR_BAD_SHAPE;
  if (state_slots == nullptr && num_slots < desc->batch) return SSD_ERR_BAD_SHAPE;
  const DeltaArgs& a = p.a;
  const int64_t HPN = (int64_t)a.H * a.P * a.N;
  if (num_slots > kMaxElems / HPN) return SSD_ERR_BAD_SHAPE;
  if (!x || !dt || !A || !B || !C || !beta || !state || !y) return SSD_ERR_NULL_POINTER;
  const size_t io = bytes_of(p.io), dts = bytes_of(p.dt);
  if (!aligned(x, io) || !aligned(dt, dts) || !aligned(A, 4) || !aligned(B, io) || !aligned(C, io) ||
      !aligned(beta, dts) || !aligned(state, 4) || !aligned(state_slots, 4) || !aligned(y, io))
    return SSD_ERR_ALIGNMENT;
  const Range in[] = {range_of(x, size_t(p.x_ext) * io),     range_of(dt, size_t(p.dt_ext) * dts),
                      range_of(beta, size_t(p.e_ext) * dts), range_of(A, size_t(a.H) * sizeof(float)),
                      range_of(B, size_t(p.b_ext) * io),     range_of(C, size_t(p.c_ext) * io),
                      range_of(state_slots, size_t(a.batch) * sizeof(int32_t)),
                      range_of(a.dto.bias, size_t(a.H) * sizeof(float))};
  const Range rs = range_of(state, size_t(num_slots * HPN) * sizeof(float));
  const Range ry = range_of(y, size_t(a.batch * a.H * a.P) * io);
  if (overlaps_any(rs, in) || overlaps_any(ry, in) || overlap(rs, ry)) return SSD_ERR_ALIAS;
  DeltaStepArgs r{};
  r.x = x, r.dt = dt, r.beta = beta, r.B = B, r.C = C, r.A = A, r.state = state, r.slots = state_slots, r.y = y;
  r.nslots = num_slots;
  r.xs = a.xs.batch, r.ds = a.ds.batch, r.es = a.es.batch, r.bs = a.bs.batch, r.cs = a.cs.batch;
  r.batch = a.batch;
  r.H = a.H, r.P = a.P, r.N = a.N, r.G = a.G;
  r.dto = a.dto;
  r.sigmoid = a.sigmoid;
  r.scale = a.scale;
  const hipError_t e = launch_delta_step(r, p.io, p.dt, static_cast<hipStream_t>(stream));
  // a launch of too many threads is one of too many rows
  return e == hipErrorInvalidConfiguration ? SSD_ERR_BAD_SHAPE : from_hip(e);
}

ssd_status_t ssd_head_norm(const ssd_head_norm_desc_t* desc, const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const int32_t* positions, const float* inv_freq, void* q_out,
                           void* k_out, void* stream) {
  using namespace ssd;
  if (desc == nullptr) return SSD_ERR_NULL_POINTER;
  const ssd_head_norm_desc_t& d = *desc;
  int io;
  if (d.batch < 1 || d.rows < 1 || d.q_heads < 1 || d.k_heads < 0 || d.headdim < 1) return SSD_ERR_BAD_SHAPE;
  if (d.batch >= kMaxRows || d.rows >= kMaxRows || !(d.eps >= 0.f)) return SSD_ERR_BAD_SHAPE;
  if (d.rot < 0 || d.rot > d.headdim || d.rot % 2 != 0) return SSD_ERR_BAD_SHAPE;
  if (!io_of(d.io_dtype, &io) || d.headdim > kHeadNormMaxDim) return SSD_ERR_UNSUPPORTED;
  if (d.q_heads > kMaxChannels / d.headdim || d.k_heads > kMaxChannels / d.headdim) return SSD_ERR_BAD_SHAPE;
  const int64_t wq = d.q_heads * d.headdim, wk = d.k_heads * d.headdim;
  HeadNormArgs a{};
  int64_t q_ext, k_ext = 0;
  if (!resolve(d.q_stride, d.batch, d.rows, wq, &a.st[0], &q_ext)) return SSD_ERR_BAD_SHAPE;
  if (wk > 0 && !resolve(d.k_stride, d.batch, d.rows, wk, &a.st[1], &k_ext)) return SSD_ERR_BAD_SHAPE;
  if (!q || !q_out || (wk > 0 && (!k || !k_out))) return SSD_ERR_NULL_POINTER;
  if (d.rot > 0 && (!positions || !inv_freq)) return SSD_ERR_NULL_POINTER;
  const size_t eb = bytes_of(io);
  if (wk == 0) k = nullptr, k_out = nullptr, k_weight = nullptr;
  if (d.rot == 0) positions = nullptr, inv_freq = nullptr;
  if (!aligned(q, eb) || !aligned(k, eb) || !aligned(q_out, eb) || !aligned(k_out, eb) || !aligned(q_weight, 4) ||
      !aligned(k_weight, 4) || !aligned(positions, 4) || !aligned(inv_freq, 4))
    return SSD_ERR_ALIGNMENT;
  const int64_t tokens = d.batch * d.rows;
  const Range in[] = {range_of(q, size_t(q_ext) * eb), range_of(k, size_t(k_ext) * eb),
                      range_of(q_weight, size_t(d.headdim) * sizeof(float)),
                      range_of(k_weight, size_t(d.headdim) * sizeof(float)),
                      range_of(positions, size_t(tokens) * sizeof(int32_t)),
                      range_of(inv_freq, size_t(d.rot / 2) * sizeof(float))};
  const Range oq = range_of(q_out, size_t(tokens * wq) * eb), ok = range_of(k_out, size_t(tokens * wk) * eb);
  if (overlaps_any(oq, in) || overlaps_any(ok, in) || overlap(oq, ok)) return SSD_ERR_ALIAS;
  a.in[0] = q, a.in[1] = k, a.w[0] = q_weight, a.w[1] = k_weight, a.out[0] = q_out, a.out[1] = k_out;
  a.heads[0] = (int)d.q_heads, a.heads[1] = (int)d.k_heads;
  a.batch = d.batch, a.rows = d.rows;
  a.D = (int)d.headdim, a.R = (int)d.rot;
  a.pos = positions, a.freq = inv_freq;
  a.l2 = d.l2 != 0, a.pairs = d.pairs != 0;
  a.eps = d.eps;
  return from_hip(launch_head_norm(a, io, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
