// C ABI of the layer operators around the SSD scan: selective scan and step,
// short convolution and its step, group norm. Argument validation and launch
// only; as in api.cpp no HIP call is made before every argument is checked.
#include <cstdint>

#include "layer_checks.h"

namespace ssd {
namespace {

struct SelectivePlan {
  SelectiveArgs a;
  int io, dt;
  int64_t batch;
  int64_t x_ext, dt_ext, z_ext, b_ext, c_ext;  // extents in elements
  SelectiveCut cut;
  size_t ends_off, dsums_off, copy_off, total;  // workspace
};

// rows: tokens per batch row (packed: of the stream); nseq 0: batched.
ssd_status_t plan_selective(const ssd_selective_desc_t* d, int64_t nseq, SelectivePlan* p) {
  if (d == nullptr) return SSD_ERR_NULL_POINTER;
  if (d->batch < 1 || d->seqlen < 1 || d->channels < 1 || d->dstate < 1 || d->ngroups < 1) return SSD_ERR_BAD_SHAPE;
  if (d->channels > kMaxChannels || d->channels % d->ngroups != 0) return SSD_ERR_BAD_SHAPE;
  if (d->batch >= kMaxRows || d->seqlen >= kMaxRows || nseq >= kMaxRows) return SSD_ERR_BAD_SHAPE;
  if (d->dstate > 256 || !io_of(d->io_dtype, &p->io) || !io_of(d->dt_dtype, &p->dt)) return SSD_ERR_UNSUPPORTED;
  if (p->dt != kF32 && p->dt != p->io) return SSD_ERR_UNSUPPORTED;
  if (d->dt_clamp && !(d->dt_min <= d->dt_max)) return SSD_ERR_BAD_SHAPE;
  if (!aligned(d->dt_bias, 4)) return SSD_ERR_ALIGNMENT;
  SelectiveArgs& a = p->a;
  const int64_t E = d->channels, GN = d->ngroups * d->dstate;
  if (!resolve(d->x_stride, d->batch, d->seqlen, E, &a.xs, &p->x_ext) ||
      !resolve(d->dt_stride, d->batch, d->seqlen, E, &a.ds, &p->dt_ext) ||
      !resolve(d->z_stride, d->batch, d->seqlen, E, &a.zs, &p->z_ext) ||
      !resolve(d->B_stride, d->batch, d->seqlen, GN, &a.bs, &p->b_ext) ||
      !resolve(d->C_stride, d->batch, d->seqlen, GN, &a.cs, &p->c_ext))
    return SSD_ERR_BAD_SHAPE;
  const int64_t rows = nseq > d->batch ? nseq : d->batch;
  if (rows > kMaxElems / (E * d->dstate)) return SSD_ERR_BAD_SHAPE;
  p->batch = d->batch;
  a.L = d->seqlen;
  a.E = (int)E;
  a.N = (int)d->dstate;
  a.G = (int)d->ngroups;
  a.nseq = nseq;
  a.dto = DtOpts{d->dt_bias, d->dt_softplus != 0, d->dt_clamp != 0, d->dt_min, d->dt_max};
  return SSD_OK;
}

// The prompt form: the cut of the time axis and the workspace it needs.
ssd_status_t plan_scan(const ssd_selective_desc_t* d, int64_t nseq, SelectivePlan* p) {
  const ssd_status_t st = plan_selective(d, nseq, p);
  if (st != SSD_OK) return st;
  if (d->batch > kMaxGridZ) return SSD_ERR_BAD_SHAPE;
  const SelectiveCut c = selective_scan_cut(d->batch, d->seqlen, d->channels, d->ngroups, nseq);
  p->cut = c;
  p->ends_off = p->dsums_off = p->copy_off = p->total = 0;
  if (c.n > 1) {
    const int64_t per = d->channels * selective_padded_states(d->dstate);
    if (d->batch * c.n > kMaxElems / per) return SSD_ERR_BAD_SHAPE;
    const size_t ends = size_t(d->batch * c.n * per) * sizeof(float);
    p->dsums_off = align_up(ends, kWsAlign);
    p->copy_off = align_up(p->dsums_off + size_t(d->batch * c.n * d->channels) * sizeof(float), kWsAlign);
    p->total = p->copy_off + align_up(ends, kWsAlign);
  }
  return SSD_OK;
}

ssd_status_t run_scan(SelectivePlan& p, const int32_t* cu, const void* x, const void* dt, const float* A,
                      const void* B, const void* C, const float* D, const void* z, const float* init, void* y,
                      float* final_state, void* workspace, size_t workspace_bytes, hipStream_t s) {
  SelectiveArgs& a = p.a;
  const size_t io = bytes_of(p.io), dts = bytes_of(p.dt);
  if (!x || !dt || !A || !B || !C || !y) return SSD_ERR_NULL_POINTER;
  if (!aligned(x, io) || !aligned(dt, dts) || !aligned(A, 4) || !aligned(B, io) || !aligned(C, io) ||
      !aligned(D, 4) || !aligned(z, io) || !aligned(init, 4) || !aligned(y, io) || !aligned(final_state, 4) ||
      !aligned(cu, 4) || !aligned(workspace, kWsAlign))
    return SSD_ERR_ALIGNMENT;
  if (workspace != nullptr && workspace_bytes < p.total) return SSD_ERR_WORKSPACE;
  const int64_t E = a.E, N = a.N, nstates = a.nseq > 0 ? a.nseq : p.batch;
  const size_t st_bytes = size_t(nstates * E * N) * sizeof(float);
  const Range in[] = {range_of(x, size_t(p.x_ext) * io),
                      range_of(dt, size_t(p.dt_ext) * dts),
                      range_of(A, size_t(E * N) * sizeof(float)),
                      range_of(B, size_t(p.b_ext) * io),
                      range_of(C, size_t(p.c_ext) * io),
                      range_of(D, size_t(E) * sizeof(float)),
                      range_of(z, size_t(p.z_ext) * io),
                      range_of(cu, cu != nullptr ? size_t(a.nseq + 1) * sizeof(int32_t) : 0),
                      range_of(a.dto.bias, size_t(E) * sizeof(float))};
  const Range ri = range_of(init, st_bytes), rf = range_of(final_state, st_bytes);
  const Range ry = range_of(y, size_t(p.batch * a.L * E) * io);
  const Range rw = range_of(workspace, p.total);
  if (overlaps_any(ry, in) || overlaps_any(rf, in) || overlaps_any(rw, in)) return SSD_ERR_ALIAS;
  if (overlap(ry, ri) || overlap(ry, rf) || overlap(ry, rw) || overlap(rw, ri) || overlap(rw, rf)) return SSD_ERR_ALIAS;
  if (overlap(rf, ri) && rf.lo != ri.lo) return SSD_ERR_ALIAS;  // the same array or none of it

  void* w = workspace;
  bool owned = false;
  if (w == nullptr && p.total > 0) {
    if (hipMallocAsync(&w, p.total, s) != hipSuccess) return SSD_ERR_HIP;
    owned = true;
  }
  a.x = x, a.dt = dt, a.B = B, a.C = C, a.z = z, a.A = A, a.D = D, a.init = init, a.y = y;
  a.final_state = final_state;
  a.cu = cu;
  a.cut = p.cut;
  char* wc = static_cast<char*>(w);
  a.ends = reinterpret_cast<float*>(wc + p.ends_off);
  a.dsums = reinterpret_cast<float*>(wc + p.dsums_off);
  a.init_copy = init != nullptr && init == final_state && a.cut.n > 1 ? reinterpret_cast<float*>(wc + p.copy_off) : nullptr;
  hipError_t e = launch_selective_scan(a, p.io, p.dt, p.batch, s);
  if (owned) {
    const hipError_t fe = hipFreeAsync(w, s);
    if (e == hipSuccess) e = fe;
  }
  return from_hip(e);
}

// Checks shared by the two convolutions; extent of the input in elements.
ssd_status_t check_conv(const ssd_conv1d_desc_t* d, int* io, Stride* xs, int64_t* extent, int (*width)[3]) {
  if (d == nullptr) return SSD_ERR_NULL_POINTER;
  if (d->batch < 1 || d->seqlen < 1 || d->channels < 1 || d->channels > kMaxChannels) return SSD_ERR_BAD_SHAPE;
  if (d->batch >= kMaxRows || d->seqlen >= kMaxRows) return SSD_ERR_BAD_SHAPE;
  if (d->conv_width < 1 || d->conv_width > 4 || !io_of(d->io_dtype, io)) return SSD_ERR_UNSUPPORTED;
  if (!resolve(d->x_stride, d->batch, d->seqlen, d->channels, xs, extent)) return SSD_ERR_BAD_SHAPE;
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) {
    const int64_t w = d->out_channels[i];
    if (w < 0 || w > d->channels) return SSD_ERR_BAD_SHAPE;
    (*width)[i] = (int)w;
    sum += w;
  }
  return sum == d->channels && d->out_channels[0] > 0 ? SSD_OK : SSD_ERR_BAD_SHAPE;
}

// Pointer checks of the outputs: given and aligned where they have channels.
ssd_status_t check_outputs(void* const (&out)[3], const int (&width)[3], size_t io) {
  for (int i = 0; i < 3; ++i) {
    if (width[i] > 0 && out[i] == nullptr) return SSD_ERR_NULL_POINTER;
    if (!aligned(out[i], io)) return SSD_ERR_ALIGNMENT;
  }
  return SSD_OK;
}

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status_t ssd_selective_scan_workspace_bytes(const ssd_selective_desc_t* desc, int64_t num_seqs, size_t* bytes) {
  if (bytes == nullptr) return SSD_ERR_NULL_POINTER;
  if (num_seqs < 0) return SSD_ERR_BAD_SHAPE;
  ssd::SelectivePlan p;
  const ssd_status_t st = ssd::plan_scan(desc, num_seqs, &p);
  if (st != SSD_OK) return st;
  if (num_seqs > 0 && desc->batch != 1) return SSD_ERR_BAD_SHAPE;
  *bytes = p.total;
  return SSD_OK;
}

ssd_status_t ssd_selective_scan(const ssd_selective_desc_t* desc, const void* x, const void* dt, const float* A,
                                const void* B, const void* C, const float* D, const void* z, const float* init_state,
                                void* y, float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  ssd::SelectivePlan p;
  const ssd_status_t st = ssd::plan_scan(desc, 0, &p);
  if (st != SSD_OK) return st;
  return ssd::run_scan(p, nullptr, x, dt, A, B, C, D, z, init_state, y, final_state, workspace, workspace_bytes,
                       static_cast<hipStream_t>(stream));
}

ssd_status_t ssd_selective_scan_varlen(const ssd_selective_desc_t* desc, const int32_t* cu_seqlens, int64_t num_seqs,
                                       const void* x, const void* dt, const float* A, const void* B, const void* C,
                                       const float* D, const void* z, const float* init_states, void* y,
                                       float* final_states, void* workspace, size_t workspace_bytes, void* stream) {
  ssd::SelectivePlan p;
  if (num_seqs < 1) return desc == nullptr ? SSD_ERR_NULL_POINTER : SSD_ERR_BAD_SHAPE;
  const ssd_status_t st = ssd::plan_scan(desc, num_seqs, &p);
  if (st != SSD_OK) return st;
  if (desc->batch != 1) return SSD_ERR_BAD_SHAPE;
  if (cu_seqlens == nullptr) return SSD_ERR_NULL_POINTER;
  return ssd::run_scan(p, cu_seqlens, x, dt, A, B, C, D, z, init_states, y, final_states, workspace, workspace_bytes,
                       static_cast<hipStream_t>(stream));
}

ssd_status_t ssd_selective_step(const ssd_selective_desc_t* desc, const void* x, const void* dt, const float* A,
                                const void* B, const void* C, const float* D, const void* z, float* state,
                                const int32_t* state_slots, int64_t num_slots, void* y, void* stream) {
  using namespace ssd;
  SelectivePlan p;
  const ssd_status_t st = plan_selective(desc, 0, &p);
  if (st != SSD_OK) return st;
  if (desc->seqlen != 1 || num_slots < 1 || num_slots >= kMaxRows) return SSD_ERR_BAD_SHAPE;
  if (state_slots == nullptr && num_slots < desc->batch) return SSD_ERR_BAD_SHAPE;
  if (desc->batch > kMaxGridZ) return SSD_ERR_BAD_SHAPE;
  const int64_t E = desc->channels, N = desc->dstate;
  if (num_slots > kMaxElems / (E * N)) return SSD_ERR_BAD_SHAPE;
  if (!x || !dt || !A || !B || !C || !state || !y) return SSD_ERR_NULL_POINTER;
  const size_t io = bytes_of(p.io), dts = bytes_of(p.dt);
  if (!aligned(x, io) || !aligned(dt, dts) || !aligned(A, 4) || !aligned(B, io) || !aligned(C, io) ||
      !aligned(D, 4) || !aligned(z, io) || !aligned(state, 4) || !aligned(state_slots, 4) || !aligned(y, io))
    return SSD_ERR_ALIGNMENT;
  const Range in[] = {range_of(x, size_t(p.x_ext) * io),
                      range_of(dt, size_t(p.dt_ext) * dts),
                      range_of(A, size_t(E * N) * sizeof(float)),
                      range_of(B, size_t(p.b_ext) * io),
                      range_of(C, size_t(p.c_ext) * io),
                      range_of(D, size_t(E) * sizeof(float)),
                      range_of(z, size_t(p.z_ext) * io),
                      range_of(state_slots, size_t(desc->batch) * sizeof(int32_t)),
                      range_of(p.a.dto.bias, size_t(E) * sizeof(float))};
  const Range rs = range_of(state, size_t(num_slots * E * N) * sizeof(float));
  const Range ry = range_of(y, size_t(desc->batch * E) * io);
  if (overlaps_any(rs, in) || overlaps_any(ry, in) || overlap(rs, ry)) return SSD_ERR_ALIAS;
  SelectiveStepArgs a{};
  a.x = x, a.dt = dt, a.B = B, a.C = C, a.z = z, a.A = A, a.D = D, a.state = state, a.y = y;
  a.slots = state_slots;
  a.nslots = num_slots;
  a.xs = p.a.xs.batch, a.ds = p.a.ds.batch, a.bs = p.a.bs.batch, a.cs = p.a.cs.batch, a.zs = p.a.zs.batch;
  a.batch = desc->batch;
  a.E = (int)E, a.N = (int)N, a.G = (int)desc->ngroups;
  a.dto = p.a.dto;
  return from_hip(launch_selective_step(a, p.io, p.dt, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_conv1d(const ssd_conv1d_desc_t* desc, const int32_t* cu_seqlens, int64_t num_seqs, const void* x,
                        const float* weight, const float* bias, const float* conv_state_in, float* conv_state_out,
                        void* out, void* out_b, void* out_c, void* stream) {
  using namespace ssd;
  Conv1dArgs a{};
  int io;
  int64_t ext;
  ssd_status_t st = check_conv(desc, &io, &a.xs, &ext, &a.width);
  if (st != SSD_OK) return st;
  if (cu_seqlens != nullptr ? (num_seqs < 1 || num_seqs >= kMaxRows || desc->batch != 1) : num_seqs != 0)
    return SSD_ERR_BAD_SHAPE;
  if (desc->batch > kMaxGridZ) return SSD_ERR_BAD_SHAPE;
  const int64_t CH = desc->channels, km1 = desc->conv_width - 1;
  const int64_t nstates = cu_seqlens != nullptr ? num_seqs : desc->batch;
  if (nstates > kMaxElems / (CH * 4)) return SSD_ERR_BAD_SHAPE;
  if (!x || !weight) return SSD_ERR_NULL_POINTER;
  a.out[0] = out, a.out[1] = out_b, a.out[2] = out_c;
  const size_t eb = bytes_of(io);
  st = check_outputs(a.out, a.width, eb);
  if (st != SSD_OK) return st;
  if (!aligned(x, eb) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(conv_state_in, 4) ||
      !aligned(conv_state_out, 4) || !aligned(cu_seqlens, 4))
    return SSD_ERR_ALIGNMENT;
  const size_t state_bytes = size_t(nstates * CH * km1) * sizeof(float);
  const Range in[] = {range_of(x, size_t(ext) * eb), range_of(weight, size_t(CH * desc->conv_width) * sizeof(float)),
                      range_of(bias, size_t(CH) * sizeof(float)), range_of(conv_state_in, state_bytes),
                      range_of(cu_seqlens, cu_seqlens != nullptr ? size_t(num_seqs + 1) * sizeof(int32_t) : 0)};
  const Range outs[] = {range_of(out, size_t(desc->batch * desc->seqlen * a.width[0]) * eb),
                        range_of(out_b, size_t(desc->batch * desc->seqlen * a.width[1]) * eb),
                        range_of(out_c, size_t(desc->batch * desc->seqlen * a.width[2]) * eb),
                        range_of(conv_state_out, state_bytes)};
  for (int i = 0; i < 4; ++i) {
    if (overlaps_any(outs[i], in)) return SSD_ERR_ALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return SSD_ERR_ALIAS;
  }
  a.x = x, a.w = weight, a.bias = bias, a.state_in = conv_state_in, a.state_out = conv_state_out;
  a.L = desc->seqlen;
  a.CH = (int)CH;
  a.silu = desc->silu != 0;
  a.cu = cu_seqlens;
  a.nseq = num_seqs;
  return from_hip(launch_conv1d(a, io, desc->conv_width, desc->batch, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_conv1d_step(const ssd_conv1d_desc_t* desc, const void* x, const float* weight, const float* bias,
                             float* conv_state, const int32_t* state_slots, int64_t num_slots, void* out,
                             void* out_b, void* out_c, void* stream) {
  using namespace ssd;
  Conv1dStepArgs a{};
  int io;
  int64_t ext;
  Stride xs;
  ssd_status_t st = check_conv(desc, &io, &xs, &ext, &a.width);
  if (st != SSD_OK) return st;
  if (desc->seqlen != 1 || num_slots < 1 || num_slots >= kMaxRows) return SSD_ERR_BAD_SHAPE;
  if (state_slots == nullptr && num_slots < desc->batch) return SSD_ERR_BAD_SHAPE;
  if (desc->batch > kMaxGridZ) return SSD_ERR_BAD_SHAPE;
  const int64_t CH = desc->channels, km1 = desc->conv_width - 1;
  if (num_slots > kMaxElems / (CH * 4)) return SSD_ERR_BAD_SHAPE;
  if (!x || !weight || (km1 > 0 && !conv_state)) return SSD_ERR_NULL_POINTER;
  a.out[0] = out, a.out[1] = out_b, a.out[2] = out_c;
  const size_t eb = bytes_of(io);
  st = check_outputs(a.out, a.width, eb);
  if (st != SSD_OK) return st;
  if (!aligned(x, eb) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(conv_state, 4) || !aligned(state_slots, 4))
    return SSD_ERR_ALIGNMENT;
  const Range in[] = {range_of(x, size_t(ext) * eb), range_of(weight, size_t(CH * desc->conv_width) * sizeof(float)),
                      range_of(bias, size_t(CH) * sizeof(float)),
                      range_of(state_slots, size_t(desc->batch) * sizeof(int32_t))};
  const Range outs[] = {range_of(out, size_t(desc->batch * a.width[0]) * eb),
                        range_of(out_b, size_t(desc->batch * a.width[1]) * eb),
                        range_of(out_c, size_t(desc->batch * a.width[2]) * eb),
                        range_of(conv_state, size_t(num_slots * CH * km1) * sizeof(float))};
  for (int i = 0; i < 4; ++i) {
    if (overlaps_any(outs[i], in)) return SSD_ERR_ALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return SSD_ERR_ALIAS;
  }
  a.x = x, a.w = weight, a.bias = bias, a.state = conv_state, a.slots = state_slots;
  a.nslots = num_slots;
  a.xs = xs.batch;
  a.batch = desc->batch;
  a.CH = (int)CH;
  a.silu = desc->silu != 0;
  return from_hip(launch_conv1d_step(a, io, desc->conv_width, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_group_norm(const ssd_group_norm_desc_t* desc, const void* x, const float* weight, const float* bias,
                            const void* z, void* out, void* stream) {
  using namespace ssd;
  if (desc == nullptr) return SSD_ERR_NULL_POINTER;
  const ssd_group_norm_desc_t& d = *desc;
  int io;
  if (d.batch < 1 || d.rows < 1 || d.channels < 1 || d.ngroups < 1 || d.channels > kMaxChannels) return SSD_ERR_BAD_SHAPE;
  if (d.batch >= kMaxRows || d.rows >= kMaxRows || d.channels % d.ngroups != 0 || !(d.eps >= 0.f)) return SSD_ERR_BAD_SHAPE;
  if (!io_of(d.io_dtype, &io) || d.channels / d.ngroups > kGroupNormMaxGroup) return SSD_ERR_UNSUPPORTED;
  if (z != nullptr && d.silu) return SSD_ERR_UNSUPPORTED;  // one activation: the gate's or the result's
  GroupNormArgs a{};
  int64_t x_ext, z_ext;
  if (!resolve(d.x_stride, d.batch, d.rows, d.channels, &a.xs, &x_ext) ||
      !resolve(d.z_stride, d.batch, d.rows, d.channels, &a.zs, &z_ext))
    return SSD_ERR_BAD_SHAPE;
  if (!x || !out) return SSD_ERR_NULL_POINTER;
  const size_t eb = bytes_of(io);
  if (!aligned(x, eb) || !aligned(z, eb) || !aligned(out, eb) || !aligned(weight, 4) || !aligned(bias, 4))
    return SSD_ERR_ALIGNMENT;
  const Range in[] = {range_of(x, size_t(x_ext) * eb), range_of(z, size_t(z_ext) * eb),
                      range_of(weight, size_t(d.channels) * sizeof(float)),
                      range_of(bias, size_t(d.channels) * sizeof(float))};
  if (overlaps_any(range_of(out, size_t(d.batch * d.rows * d.channels) * eb), in)) return SSD_ERR_ALIAS;
  a.x = x, a.z = z, a.w = weight, a.bias = bias, a.out = out;
  a.batch = d.batch, a.rows = d.rows;
  a.C = (int)d.channels, a.G = (int)d.ngroups;
  a.eps = d.eps;
  a.center = d.center != 0, a.gate_first = d.gate_first != 0, a.silu = d.silu != 0;
  return from_hip(launch_group_norm(a, io, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
