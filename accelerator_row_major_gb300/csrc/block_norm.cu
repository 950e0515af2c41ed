// The norms at a block's ends and their gradients: entry points, their checks
// and what the kernels (block_norm_kernels.cuh) are given.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/gemm_f32_block.h"
#include "block_norm.h"
#include "launch.h"
#include "workspace.h"

namespace gemm_f32_impl {

namespace {

constexpr int kMostWidth = INT_MAX - 1024;   // a step beyond the last column stays within an int

size_t type_size(int type) { return type == GEMM_F32_TYPE_F32 ? 4 : 2; }

bool aligned_to(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

bool matrix_ok(const void* p, long long ld, int width, size_t size) { return p && aligned_to(p, size) && ld >= width; }

size_t matrix_bytes(long long rows, int width, long long ld, size_t size) {
  return rows > 0 ? (static_cast<size_t>(rows - 1) * ld + width) * size : 0;
}

// An element's address within its matrix fits in 63 bits.
bool addressable(long long rows, long long ld) { return rows == 0 || ld <= LLONG_MAX / 8 / rows; }

struct Matrix {
  const void* p;
  long long ld;
};

RowSource source(const void* p, long long ld, int size, const RowPlan& plan) {
  RowSource m = {};
  if (!p) return m;
  m.p = static_cast<const char*>(p);
  m.ld = ld * size;
  m.size = size;
  m.end = m.p + matrix_bytes(plan.rows, plan.width, ld, size);
  return m;
}

// Bytes of 8-bit rows, all of which may be read.
RowSource saved_source(const void* p, long long ld, bool exponents, const RowPlan& plan) {
  RowSource m = {};
  if (!p) return m;
  m.p = static_cast<const char*>(p);
  m.ld = ld;
  m.size = exponents ? 0 : 1;
  m.end = m.p + plan.rows * ld;
  return m;
}

// Whether rows start on 16-byte boundaries and hold whole vectors.
bool vector_rows(const void* p, long long ld, int width, size_t size) {
  return aligned_to(p, 16) && ld * size % 16 == 0 && width * size % 16 == 0;
}

// What both entry points ask of the block's description.
bool block_ok(const gemm_f32_block_t* b) {
  if (!b) return false;
  if (b->type != GEMM_F32_TYPE_F32 && b->type != GEMM_F32_TYPE_BF16) return false;
  if (b->weight_type != GEMM_F32_TYPE_F32 && b->weight_type != b->type) return false;
  if (b->norm != GEMM_F32_NORM_LAYER && b->norm != GEMM_F32_NORM_RMS) return false;
  if ((b->post != 0 && b->post != 1) || b->rows < 0 || b->width < 1 || b->width > kMostWidth) return false;
  if (!std::isfinite(b->residual_scale) || !std::isfinite(b->branch_scale)) return false;
  if (b->norm == GEMM_F32_NORM_RMS && (b->bias || b->post_bias)) return false;
  if (!b->post && (b->post_weight || b->post_bias)) return false;
  const size_t es = type_size(b->type), ws = type_size(b->weight_type);
  if (!aligned_to(b->weight, ws) || !aligned_to(b->bias, ws) || !aligned_to(b->post_weight, ws) ||
      !aligned_to(b->post_bias, ws))
    return false;
  if (b->gate) {
    if (b->ld_gate == 0) return aligned_to(b->gate, ws);
    return matrix_ok(b->gate, b->ld_gate, b->width, es) && addressable(b->rows, b->ld_gate);
  }
  return true;
}

int gate_of(const gemm_f32_block_t& b) { return !b.gate ? kNoGate : b.ld_gate == 0 ? kChannelGate : kElementGate; }

// The vectors that the kernels keep; returns how many.
int vectors_of(const gemm_f32_block_t& b, bool forward, VectorArgs& v) {
  const void* const p[kVectors] = {b.weight, b.bias, b.post_weight, b.post_bias, b.gate};
  const int gate = gate_of(b);
  // the bias of the norm of h does not enter its gradient, that of the
  // branch's norm only through the gate's
  const bool there[kVectors] = {true, forward && b.bias, b.post != 0, b.post_bias && (forward || gate != kNoGate),
                                gate == kChannelGate};
  int n = 0;
  for (int i = 0; i < kVectors; ++i) {
    v.p[i] = there[i] ? p[i] : nullptr;
    v.slot[i] = there[i] ? n++ : -1;
  }
  v.f32 = b.weight_type == GEMM_F32_TYPE_F32;
  return n;
}

// An output that is one of the matrices itself, with the same stride, or
// apart from all of them; and apart from `others`, further outputs, and from
// 8-bit rows.
bool output_fits(const Matrix& out, const Matrix* in, int n_in, const Matrix* others, int n_others, long long rows,
                 int width, size_t size) {
  const size_t bytes = matrix_bytes(rows, width, out.ld, size);
  for (int i = 0; i < n_in; ++i) {
    if (!in[i].p || (out.p == in[i].p && out.ld == in[i].ld)) continue;
    if (ranges_overlap(out.p, bytes, in[i].p, matrix_bytes(rows, width, in[i].ld, size))) return false;
  }
  for (int i = 0; i < n_others; ++i)
    if (others[i].p && ranges_overlap(out.p, bytes, others[i].p, matrix_bytes(rows, width, others[i].ld, size)))
      return false;
  return true;
}

// Rows as they are, or in 8 bits.
bool rows_ok(const gemm_f32_rows_t* r, long long rows, int width, size_t size) {
  if (!r) return false;
  if (!r->codes) return matrix_ok(r->data, r->ld, width, size) && addressable(rows, r->ld);
  return r->exponents && aligned_to(r->codes, 16) && aligned_to(r->exponents, 16) && r->ld_codes % 16 == 0 &&
         r->ld_exponents % 16 == 0 && r->ld_codes >= (width + 31LL) / 32 * 32 && r->ld_exponents >= (width + 31LL) / 32 &&
         addressable(rows, r->ld_codes) && addressable(rows, r->ld_exponents);
}

bool apart_from_saved(const Matrix& out, const gemm_f32_rows_t* r, long long rows, int width, size_t size) {
  if (!out.p || !r || !r->codes) return true;
  const size_t bytes = matrix_bytes(rows, width, out.ld, size);
  return !ranges_overlap(out.p, bytes, r->codes, static_cast<size_t>(rows) * r->ld_codes) &&
         !ranges_overlap(out.p, bytes, r->exponents, static_cast<size_t>(rows) * r->ld_exponents);
}

RowPlan plan_of(const gemm_f32_block_t& b) {
  RowPlan plan = {};
  plan.width = b.width;
  plan.rows = b.rows;
  return plan;
}

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" int gemm_f32_block_norm(const gemm_f32_block_t* block, const void* branch, long long ld_branch,
                                   const void* residual, long long ld_residual, void* y, long long ldy, void* h,
                                   long long ldh, float* stats, gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!block_ok(block) || !std::isfinite(block->eps) || block->eps < 0.0f) return GEMM_F32_EINVAL;
  if (block->rows == 0) return GEMM_F32_OK;
  const gemm_f32_block_t& b = *block;
  const size_t es = type_size(b.type);
  const Matrix in[3] = {{branch, ld_branch}, {residual, ld_residual}, {b.ld_gate ? b.gate : nullptr, b.ld_gate}};
  const Matrix out[2] = {{y, ldy}, {h, ldh}};
  for (int i = 0; i < 2; ++i)
    if (!matrix_ok(in[i].p, in[i].ld, b.width, es) || !addressable(b.rows, in[i].ld)) return GEMM_F32_EINVAL;
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && !h) continue;
    if (!matrix_ok(out[i].p, out[i].ld, b.width, es) || !addressable(b.rows, out[i].ld)) return GEMM_F32_EINVAL;
    if (!output_fits(out[i], in, 3, out + 1, i == 0 ? 1 : 0, b.rows, b.width, es)) return GEMM_F32_EINVAL;
  }
  if (!aligned_to(stats, 4)) return GEMM_F32_EINVAL;
  BlockArgs a = {};
  int device = 0, num_sms = 0;
  if (!current_device(&device, &num_sms, &a.err)) return GEMM_F32_EDEVICE;
  a.plan = plan_of(b);
  bool aligned = true;
  for (int i = 0; i < 3; ++i) {
    a.in[i] = source(in[i].p, in[i].ld, static_cast<int>(es), a.plan);
    aligned = aligned && (!in[i].p || vector_rows(in[i].p, in[i].ld, b.width, es));
  }
  for (int i = 0; i < 2; ++i) aligned = aligned && (!out[i].p || vector_rows(out[i].p, out[i].ld, b.width, es));
  const int vectors = vectors_of(b, true, a.vectors);
  a.rms = b.norm == GEMM_F32_NORM_RMS;
  a.post = b.post;
  a.gate = gate_of(b);
  a.eps = b.eps;
  a.alpha = b.residual_scale;
  a.beta = b.branch_scale;
  a.y = {y, ldy};
  a.h = {h, ldh};
  a.stats = stats;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
  const char* kernel = "none";
  int launches = 0;
  const BlockLaunch l = {vectors, aligned, b.weight_type == GEMM_F32_TYPE_F32, device, num_sms, stream, &launches, &kernel};
  const int rc = b.type == GEMM_F32_TYPE_F32 ? block_norm_f32(a, l) : block_norm_bf16(a, l);
  if (rc == GEMM_F32_OK) note_launches(launches, kernel);
  return rc;
}

extern "C" int gemm_f32_block_norm_grad(const gemm_f32_block_t* block, const void* dy, long long lddy, const void* dh,
                                        long long lddh, const gemm_f32_rows_t* h, const gemm_f32_rows_t* branch,
                                        const float* stats, void* dbranch, long long ld_dbranch, void* dresidual,
                                        long long ld_dresidual, void* dgate, long long ld_dgate, void* dweight,
                                        void* dbias, void* dpost_weight, void* dpost_bias,
                                        gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!block_ok(block)) return GEMM_F32_EINVAL;
  const gemm_f32_block_t& b = *block;
  const size_t es = type_size(b.type), ws = type_size(b.weight_type);
  const int gate = gate_of(b);
  const bool needs_branch = b.post || gate != kNoGate;
  if (b.norm == GEMM_F32_NORM_RMS && (dbias || dpost_bias)) return GEMM_F32_EINVAL;
  if ((!b.post && (dpost_weight || dpost_bias)) || (gate == kNoGate && dgate)) return GEMM_F32_EINVAL;
  void* const vectors_out[kSums] = {dweight, dbias, gate == kChannelGate ? dgate : nullptr, dpost_weight, dpost_bias};
  for (void* v : vectors_out)
    if (!aligned_to(v, ws)) return GEMM_F32_EINVAL;
  const Matrix out[3] = {{dbranch, ld_dbranch}, {dresidual, ld_dresidual}, {gate == kElementGate ? dgate : nullptr, ld_dgate}};
  if (b.rows > 0) {
    if (!matrix_ok(dy, lddy, b.width, es) || !addressable(b.rows, lddy)) return GEMM_F32_EINVAL;
    if (dh && (!matrix_ok(dh, lddh, b.width, es) || !addressable(b.rows, lddh))) return GEMM_F32_EINVAL;
    if (!rows_ok(h, b.rows, b.width, es) || (needs_branch && !rows_ok(branch, b.rows, b.width, es))) return GEMM_F32_EINVAL;
    if (!stats || !aligned_to(stats, 4)) return GEMM_F32_EINVAL;
    const gemm_f32_rows_t* const used = needs_branch ? branch : nullptr;
    const Matrix in[5] = {{dy, lddy}, {dh, lddh}, {h->codes ? nullptr : h->data, h->ld},
                          {used && !used->codes ? used->data : nullptr, used ? used->ld : 0},
                          {gate == kElementGate ? b.gate : nullptr, b.ld_gate}};
    for (int i = 0; i < 3; ++i) {
      if (!out[i].p) continue;
      if (!matrix_ok(out[i].p, out[i].ld, b.width, es) || !addressable(b.rows, out[i].ld)) return GEMM_F32_EINVAL;
      if (!output_fits(out[i], in, 5, out + i + 1, 2 - i, b.rows, b.width, es)) return GEMM_F32_EINVAL;
      if (!apart_from_saved(out[i], h, b.rows, b.width, es) || !apart_from_saved(out[i], used, b.rows, b.width, es))
        return GEMM_F32_EINVAL;
    }
  }
  bool wanted = false;
  for (void* v : vectors_out) wanted = wanted || v;
  if (!wanted && (b.rows == 0 || !(out[0].p || out[1].p || out[2].p))) return GEMM_F32_OK;
  BlockGradArgs a = {};
  int device = 0, num_sms = 0;
  if (!current_device(&device, &num_sms, &a.err)) return GEMM_F32_EDEVICE;
  a.plan = plan_of(b);
  bool aligned = true;
  if (b.rows > 0) {
    const int size = static_cast<int>(es);
    auto add = [&](int i, const void* p, long long ld) {
      a.in[i] = source(p, ld, size, a.plan);
      aligned = aligned && (!p || vector_rows(p, ld, b.width, es));
    };
    auto add_rows = [&](int i, int exponents, const gemm_f32_rows_t* r) {
      if (!r->codes) return add(i, r->data, r->ld);
      a.in[i] = saved_source(r->codes, r->ld_codes, false, a.plan);
      a.in[exponents] = saved_source(r->exponents, r->ld_exponents, true, a.plan);
    };
    add(kGradDy, dy, lddy);
    add(kGradDh, dh, lddh);
    add_rows(kGradH, kGradHExponents, h);
    if (needs_branch) add_rows(kGradBranch, kGradBranchExponents, branch);
    if (gate == kElementGate) add(kGradGate, b.gate, b.ld_gate);
    for (const Matrix& o : out) aligned = aligned && (!o.p || vector_rows(o.p, o.ld, b.width, es));
    // codes alone are always on boundaries, but the vectors are those of whole rows
    aligned = aligned && b.width * es % 16 == 0;
  }
  const int vectors = vectors_of(b, false, a.vectors);
  a.rms = b.norm == GEMM_F32_NORM_RMS;
  a.post = b.post;
  a.gate = gate;
  a.branch = needs_branch;
  a.alpha = b.residual_scale;
  a.beta = b.branch_scale;
  a.stats = stats;
  a.dbranch = {const_cast<void*>(out[0].p), out[0].ld};
  a.dresidual = {const_cast<void*>(out[1].p), out[1].ld};
  a.dgate = {const_cast<void*>(out[2].p), out[2].ld};
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
  int launches = 0;
  const char* kernel = "none";
  const WorkspaceCall call;
  const BlockLaunch l = {vectors, aligned, b.weight_type == GEMM_F32_TYPE_F32, device, num_sms, stream, &launches, &kernel};
  const int rc = b.type == GEMM_F32_TYPE_F32 ? block_norm_grad_f32(a, vectors_out, l) : block_norm_grad_bf16(a, vectors_out, l);
  if (rc == GEMM_F32_OK) note_launches(launches, kernel);
  return rc;
}
