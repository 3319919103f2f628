// api_layers.cu -- the C ABI of the operators around the scan (declared in
// include/ssmscan.h): argument validation and launch.  Every argument error is
// found here, before anything is enqueued, and is returned as an ssm_status.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "api_util.h"
#include "layers.h"
#include "ssd.h"
#include "ssmscan.h"

namespace {

using ssm::aligned;
using ssm::current_device_for;
using ssm::elem_size;
using ssm::mul_ok;

constexpr int64_t kMaxElements = int64_t(1) << 60;  // byte offsets then fit in int64

bool known(ssm_dtype t) { return t == SSM_F32 || t == SSM_BF16; }

ssm_status status_of(cudaError_t e) { return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

// Sizes and strides of a convolution; x is read up to (batch - 1) and
// (seqlen - 1) strides in.
ssm_status check_conv(const ssm_conv_shapes* s, ssm_dtype dtype) {
  if (s == nullptr) return SSM_ERR_NULL;
  if (!known(dtype)) return SSM_ERR_UNSUPPORTED;
  if (s->batch < 1 || s->seqlen < 1 || s->dim < 1 || s->width < 1) return SSM_ERR_SHAPE;
  if (!ssm::conv_supported_width(s->width) || (s->silu != 0 && s->silu != 1))
    return SSM_ERR_UNSUPPORTED;
  int64_t bl, n, span_b, span_t;
  if (!mul_ok(s->batch, s->seqlen, &bl) || !mul_ok(bl, s->dim, &n) || n > kMaxElements ||
      !mul_ok(s->batch, s->width, &span_b) || !mul_ok(span_b, s->dim, &span_b) ||
      span_b > kMaxElements)
    return SSM_ERR_SHAPE;
  if (s->x_batch_stride < 0 || s->x_step_stride < 0 ||
      !mul_ok(s->batch, s->x_batch_stride, &span_b) ||
      !mul_ok(s->seqlen, s->x_step_stride, &span_t) || span_b > kMaxElements ||
      span_t > kMaxElements)
    return SSM_ERR_SHAPE;
  return SSM_OK;
}

ssm::ConvParams conv_params(const void* x, const float* weight, const float* bias,
                            const int32_t* valid_len, const void* state0, void* y,
                            void* out_final, const ssm_conv_shapes& s) {
  ssm::ConvParams p;
  p.x = x; p.x_batch = s.x_batch_stride; p.x_step = s.x_step_stride;
  p.weight = weight; p.bias = bias; p.valid_len = valid_len; p.state0 = state0;
  p.y = y; p.out_final = out_final;
  p.batch = s.batch; p.seqlen = s.seqlen; p.dim = s.dim;
  p.width = static_cast<int>(s.width); p.silu = s.silu;
  return p;
}

ssm_status check_norm(const ssm_norm_shapes* s) {
  if (s == nullptr) return SSM_ERR_NULL;
  if (!known(s->dtype) || !known(s->residual_dtype)) return SSM_ERR_UNSUPPORTED;
  if (s->rows < 1 || s->dim < 1) return SSM_ERR_SHAPE;
  if (!(s->eps >= 0.f) || isinf(s->eps)) return SSM_ERR_SHAPE;
  if (s->dim > ssm::kNormMaxDim || (s->rms != 0 && s->rms != 1) ||
      (s->residual_dtype != s->dtype && s->residual_dtype != SSM_F32))
    return SSM_ERR_UNSUPPORTED;
  int64_t n;
  if (!mul_ok(s->rows, s->dim, &n) || n > kMaxElements) return SSM_ERR_SHAPE;
  return SSM_OK;
}

ssm_status check_xent(const ssm_xent_shapes* s) {
  if (s == nullptr) return SSM_ERR_NULL;
  if (s->tokens < 1 || s->vocab < 1 || s->dim < 1) return SSM_ERR_SHAPE;
  const int64_t lim = int64_t(1) << 30;  // rows are addressed by 32-bit copy coordinates
  int64_t n;
  if (s->tokens > lim || s->vocab > lim || s->dim > lim || !mul_ok(s->tokens, s->vocab, &n) ||
      n > kMaxElements / 16)
    return SSM_ERR_SHAPE;
  return s->dim % 8 == 0 ? SSM_OK : SSM_ERR_UNSUPPORTED;  // copies start on 16-byte boundaries
}

// A tensor read with these strides: its span stays addressable.
bool span_ok(int64_t batch, int64_t batch_stride, int64_t seqlen, int64_t step_stride) {
  int64_t b, t;
  return batch_stride >= 0 && step_stride >= 0 && mul_ok(batch, batch_stride, &b) &&
         mul_ok(seqlen, step_stride, &t) && b <= kMaxElements && t <= kMaxElements;
}

ssm_status check_recur(const ssm_recur_shapes* s, ssm_dtype dtype) {
  if (s == nullptr) return SSM_ERR_NULL;
  if (!known(dtype)) return SSM_ERR_UNSUPPORTED;
  if (s->batch < 1 || s->seqlen < 1 || s->dim < 1) return SSM_ERR_SHAPE;
  int64_t n, units;
  if (!mul_ok(s->batch, s->seqlen, &n) || !mul_ok(n, s->dim, &n) || n > kMaxElements)
    return SSM_ERR_SHAPE;
  // the grid: a CTA per (batch row, 32 channels)
  if (!mul_ok(s->batch, s->dim / 32 + 1, &units) || units > INT32_MAX) return SSM_ERR_SHAPE;
  if (!span_ok(s->batch, s->gate_batch_stride, s->seqlen, s->gate_step_stride) ||
      !span_ok(s->batch, s->value_batch_stride, s->seqlen, s->value_step_stride))
    return SSM_ERR_SHAPE;
  return SSM_OK;
}

ssm::RecurParams recur_params(const void* gate, const void* value, const float* floor,
                              const int32_t* valid_len, const ssm_recur_shapes& s) {
  ssm::RecurParams p = {};
  p.gate = gate; p.value = value; p.floor = floor; p.valid_len = valid_len;
  p.gate_batch = s.gate_batch_stride; p.gate_step = s.gate_step_stride;
  p.value_batch = s.value_batch_stride; p.value_step = s.value_step_stride;
  p.batch = s.batch; p.seqlen = s.seqlen; p.dim = s.dim;
  return p;
}

ssm_status check_embed(const ssm_embed_shapes* s) {
  if (s == nullptr) return SSM_ERR_NULL;
  if (!known(s->dtype) || !known(s->io_dtype)) return SSM_ERR_UNSUPPORTED;
  if (s->tokens < 1 || s->vocab < 1 || s->dim < 1) return SSM_ERR_SHAPE;
  if (!isfinite(s->scale)) return SSM_ERR_SHAPE;
  if (s->io_dtype != s->dtype && s->io_dtype != SSM_F32) return SSM_ERR_UNSUPPORTED;
  const int64_t lim = int64_t(1) << 30;  // ids and tokens are kept in 32 bits
  int64_t n;
  if (s->tokens > lim || s->vocab > lim || !mul_ok(s->vocab, s->dim, &n) || n > kMaxElements)
    return SSM_ERR_SHAPE;
  // the grid of the sums: a warp per 8 tokens and 128 columns at most
  if (!mul_ok(s->tokens / 8 + 1, s->dim / 128 + 1, &n) || n > INT32_MAX) return SSM_ERR_SHAPE;
  return SSM_OK;
}

ssm::XentParams xent_params(const void* h, const void* weight, const int64_t* targets,
                            const ssm_xent_shapes& s, void* workspace) {
  ssm::XentParams p = {};
  p.h = h; p.weight = weight; p.targets = targets; p.ignore_index = s.ignore_index;
  p.shape = {s.tokens, s.vocab, s.dim};
  p.workspace = workspace;
  return p;
}

ssm_status check_distill(const ssm_distill_shapes* s) {
  if (s == nullptr) return SSM_ERR_NULL;
  const ssm_xent_shapes x = {s->tokens, s->vocab, s->dim, 0};
  const ssm_status st = check_xent(&x);
  if (st != SSM_OK) return st;
  if (!known(s->teacher_dtype)) return SSM_ERR_UNSUPPORTED;
  // a subnormal one has no reciprocal, or none that log2(e) can scale
  if (s->top < 1 || !(s->temperature >= FLT_MIN) || isinf(s->temperature)) return SSM_ERR_SHAPE;
  return s->top <= ssm::kDistillMaxTop ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

ssm::DistillParams distill_params(const void* h, const void* weight, const int64_t* ids,
                                  const void* logits, const ssm_distill_shapes& s,
                                  void* workspace) {
  ssm::DistillParams d = {};
  d.xent = xent_params(h, weight, nullptr, {s.tokens, s.vocab, s.dim, 0}, workspace);
  d.ids = ids; d.logits = logits; d.logits_bf16 = s.teacher_dtype == SSM_BF16;
  d.top = static_cast<int>(s.top); d.ignore_index = s.ignore_index;
  d.temperature = s.temperature;
  return d;
}

}  // namespace

extern "C" {

ssm_status ssm_conv_fwd(const void* x, const float* weight, const float* bias,
                        const int32_t* valid_len, const void* state0, void* out_y,
                        void* out_final, const ssm_conv_shapes* shapes, ssm_dtype dtype,
                        cudaStream_t stream) {
  ssm_status st = check_conv(shapes, dtype);
  if (st != SSM_OK) return st;
  if (!x || !weight || !out_y) return SSM_ERR_NULL;
  const size_t es = elem_size(dtype);
  if (!aligned(x, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(valid_len, 4) ||
      !aligned(state0, es) || !aligned(out_y, es) || !aligned(out_final, es))
    return SSM_ERR_ALIGN;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  unsigned* err = ssm::stream::error_word();
  if (!err) return SSM_ERR_CUDA;
  return status_of(ssm::launch_conv_fwd(
      conv_params(x, weight, bias, valid_len, state0, out_y, out_final, *shapes),
      dtype == SSM_BF16, err, stream));
}

size_t ssm_conv_bwd_workspace_bytes(const ssm_conv_shapes* shapes) {
  if (check_conv(shapes, SSM_F32) != SSM_OK) return 0;
  const int64_t parts = ssm::conv_bwd_partials(shapes->batch, shapes->seqlen, shapes->dim,
                                                static_cast<int>(shapes->width));
  return static_cast<size_t>(parts) * (shapes->width + 1) * shapes->dim * sizeof(float);
}

ssm_status ssm_conv_bwd(const void* x, const float* weight, const float* bias,
                        const int32_t* valid_len, const void* state0, const void* dy, void* dx,
                        float* dweight, float* dbias, void* dstate0, void* workspace,
                        size_t workspace_bytes, const ssm_conv_shapes* shapes, ssm_dtype dtype,
                        cudaStream_t stream) {
  ssm_status st = check_conv(shapes, dtype);
  if (st != SSM_OK) return st;
  if (!x || !weight || !dy || !dx || !dweight || !workspace) return SSM_ERR_NULL;
  const size_t es = elem_size(dtype);
  if (!aligned(x, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(valid_len, 4) ||
      !aligned(state0, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(dweight, 4) ||
      !aligned(dbias, 4) || !aligned(dstate0, es) || !aligned(workspace, 16))
    return SSM_ERR_ALIGN;
  if (workspace_bytes < ssm_conv_bwd_workspace_bytes(shapes)) return SSM_ERR_SHAPE;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::ConvBwdParams q;
  q.fwd = conv_params(x, weight, bias, valid_len, state0, nullptr, nullptr, *shapes);
  q.dy = dy; q.dx = dx; q.dstate0 = dstate0; q.dweight = dweight; q.dbias = dbias;
  q.partial = static_cast<float*>(workspace);
  unsigned* err = ssm::stream::error_word();
  if (!err) return SSM_ERR_CUDA;
  return status_of(ssm::launch_conv_bwd(q, dtype == SSM_BF16, err, stream));
}

ssm_status ssm_conv_step(const void* x, const float* weight, const float* bias, void* state,
                         void* out_y, const ssm_conv_shapes* shapes, ssm_dtype dtype,
                         cudaStream_t stream) {
  ssm_status st = check_conv(shapes, dtype);
  if (st != SSM_OK) return st;
  if (shapes->seqlen != 1) return SSM_ERR_SHAPE;
  if (!x || !weight || !state || !out_y) return SSM_ERR_NULL;
  const size_t es = elem_size(dtype);
  if (!aligned(x, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(state, es) ||
      !aligned(out_y, es))
    return SSM_ERR_ALIGN;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::ConvStepParams p;
  p.x = x; p.x_batch = shapes->x_batch_stride; p.weight = weight; p.bias = bias;
  p.state = state; p.y = out_y; p.batch = shapes->batch; p.dim = shapes->dim;
  p.width = static_cast<int>(shapes->width); p.silu = shapes->silu;
  return status_of(ssm::launch_conv_step(p, dtype == SSM_BF16, stream));
}

ssm_status ssm_norm_fwd(const void* x, const void* residual, const float* weight,
                        const float* bias, void* out_y, void* out_r, float* out_stats,
                        const ssm_norm_shapes* shapes, cudaStream_t stream) {
  ssm_status st = check_norm(shapes);
  if (st != SSM_OK) return st;
  const ssm_norm_shapes& s = *shapes;
  if (!x || !weight || !out_y || (residual != nullptr) != (out_r != nullptr)) return SSM_ERR_NULL;
  if (!residual && s.residual_dtype != s.dtype) return SSM_ERR_UNSUPPORTED;
  const size_t es = elem_size(s.dtype), rs = elem_size(s.residual_dtype);
  if (!aligned(x, es) || !aligned(residual, rs) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(out_y, es) || !aligned(out_r, rs) || !aligned(out_stats, 4))
    return SSM_ERR_ALIGN;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::NormParams p;
  p.x = x; p.residual = residual; p.weight = weight; p.bias = bias;
  p.y = out_y; p.r = out_r; p.stats = out_stats;
  p.rows = s.rows; p.dim = s.dim; p.rms = s.rms; p.eps = s.eps;
  return status_of(ssm::launch_norm_fwd(p, s.dtype == SSM_BF16, s.residual_dtype == SSM_BF16,
                                        stream));
}

size_t ssm_norm_bwd_workspace_bytes(const ssm_norm_shapes* shapes) {
  if (check_norm(shapes) != SSM_OK) return 0;
  return static_cast<size_t>(ssm::norm_bwd_partials(shapes->rows, shapes->dim)) * 2 *
         shapes->dim * sizeof(float);
}

ssm_status ssm_norm_bwd(const void* r, const float* weight, const float* stats, const void* dy,
                        const void* dr, void* dx, void* dresidual, float* dweight, float* dbias,
                        void* workspace, size_t workspace_bytes, const ssm_norm_shapes* shapes,
                        cudaStream_t stream) {
  ssm_status st = check_norm(shapes);
  if (st != SSM_OK) return st;
  const ssm_norm_shapes& s = *shapes;
  if (!r || !weight || !stats || !dy || !dx || !dweight || !workspace) return SSM_ERR_NULL;
  const size_t es = elem_size(s.dtype), rs = elem_size(s.residual_dtype);
  if (!aligned(r, rs) || !aligned(weight, 4) || !aligned(stats, 4) || !aligned(dy, es) ||
      !aligned(dr, rs) || !aligned(dx, es) || !aligned(dresidual, rs) || !aligned(dweight, 4) ||
      !aligned(dbias, 4) || !aligned(workspace, 16))
    return SSM_ERR_ALIGN;
  if (workspace_bytes < ssm_norm_bwd_workspace_bytes(shapes)) return SSM_ERR_SHAPE;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::NormBwdParams p;
  p.r = r; p.weight = weight; p.stats = stats; p.dy = dy; p.dr = dr; p.dx = dx;
  p.dresidual = dresidual; p.dweight = dweight; p.dbias = dbias;
  p.partial = static_cast<float*>(workspace);
  p.rows = s.rows; p.dim = s.dim; p.rms = s.rms;
  return status_of(ssm::launch_norm_bwd(p, s.dtype == SSM_BF16, s.residual_dtype == SSM_BF16,
                                        stream));
}

size_t ssm_xent_workspace_bytes(const ssm_xent_shapes* shapes, int backward) {
  if (check_xent(shapes) != SSM_OK) return 0;
  return ssm::xent_workspace_bytes({shapes->tokens, shapes->vocab, shapes->dim}, backward != 0);
}

ssm_status ssm_xent_fwd(const void* h, const void* weight, const int64_t* targets, float* out_loss,
                        float* out_lse, void* workspace, size_t workspace_bytes,
                        const ssm_xent_shapes* shapes, ssm_dtype dtype, cudaStream_t stream) {
  ssm_status st = check_xent(shapes);
  if (st != SSM_OK) return st;
  if (dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (!h || !weight || !targets || !out_loss || !out_lse || !workspace) return SSM_ERR_NULL;
  if (!aligned(h, 16) || !aligned(weight, 16) || !aligned(targets, 8) || !aligned(out_loss, 4) ||
      !aligned(out_lse, 4) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (workspace_bytes < ssm_xent_workspace_bytes(shapes, 0)) return SSM_ERR_SHAPE;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::XentParams p = xent_params(h, weight, targets, *shapes, workspace);
  if (!(p.err = ssm::stream::error_word())) return SSM_ERR_CUDA;
  p.loss = out_loss; p.lse = out_lse;
  return status_of(ssm::launch_xent_fwd(p, stream));
}

ssm_status ssm_xent_bwd(const void* h, const void* weight, const int64_t* targets,
                        const float* lse, const float* dloss, void* dh, void* dweight,
                        void* workspace, size_t workspace_bytes, const ssm_xent_shapes* shapes,
                        ssm_dtype dtype, cudaStream_t stream) {
  ssm_status st = check_xent(shapes);
  if (st != SSM_OK) return st;
  if (dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (!h || !weight || !targets || !lse || !dloss || !dh || !dweight || !workspace)
    return SSM_ERR_NULL;
  if (!aligned(h, 16) || !aligned(weight, 16) || !aligned(targets, 8) || !aligned(lse, 4) ||
      !aligned(dloss, 4) || !aligned(dh, 16) || !aligned(dweight, 16) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (workspace_bytes < ssm_xent_workspace_bytes(shapes, 1)) return SSM_ERR_SHAPE;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::XentParams p = xent_params(h, weight, targets, *shapes, workspace);
  if (!(p.err = ssm::stream::error_word())) return SSM_ERR_CUDA;
  p.lse_in = lse; p.dloss = dloss; p.dh = dh; p.dweight = dweight;
  return status_of(ssm::launch_xent_bwd(p, stream));
}

size_t ssm_distill_workspace_bytes(const ssm_distill_shapes* shapes, int backward) {
  if (check_distill(shapes) != SSM_OK) return 0;
  return ssm::distill_workspace_bytes({shapes->tokens, shapes->vocab, shapes->dim},
                                      static_cast<int>(shapes->top), backward != 0);
}

ssm_status ssm_distill_fwd(const void* h, const void* weight, const int64_t* ids,
                           const void* logits, float* out_loss, float* out_lse, void* workspace,
                           size_t workspace_bytes, const ssm_distill_shapes* shapes,
                           ssm_dtype dtype, cudaStream_t stream) {
  ssm_status st = check_distill(shapes);
  if (st != SSM_OK) return st;
  if (dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (!h || !weight || !ids || !logits || !out_loss || !out_lse || !workspace) return SSM_ERR_NULL;
  if (!aligned(h, 16) || !aligned(weight, 16) || !aligned(ids, 8) ||
      !aligned(logits, elem_size(shapes->teacher_dtype)) || !aligned(out_loss, 4) ||
      !aligned(out_lse, 4) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (workspace_bytes < ssm_distill_workspace_bytes(shapes, 0)) return SSM_ERR_SHAPE;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::DistillParams d = distill_params(h, weight, ids, logits, *shapes, workspace);
  if (!(d.xent.err = ssm::stream::error_word())) return SSM_ERR_CUDA;
  d.xent.loss = out_loss; d.xent.lse = out_lse;
  return status_of(ssm::launch_distill_fwd(d, stream));
}

ssm_status ssm_distill_bwd(const void* h, const void* weight, const int64_t* ids,
                           const void* logits, const float* lse, const float* dloss, void* dh,
                           void* dweight, void* workspace, size_t workspace_bytes,
                           const ssm_distill_shapes* shapes, ssm_dtype dtype, cudaStream_t stream) {
  ssm_status st = check_distill(shapes);
  if (st != SSM_OK) return st;
  if (dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (!h || !weight || !ids || !logits || !lse || !dloss || !dh || !dweight || !workspace)
    return SSM_ERR_NULL;
  if (!aligned(h, 16) || !aligned(weight, 16) || !aligned(ids, 8) ||
      !aligned(logits, elem_size(shapes->teacher_dtype)) || !aligned(lse, 4) ||
      !aligned(dloss, 4) || !aligned(dh, 16) || !aligned(dweight, 16) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (workspace_bytes < ssm_distill_workspace_bytes(shapes, 1)) return SSM_ERR_SHAPE;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::DistillParams d = distill_params(h, weight, ids, logits, *shapes, workspace);
  if (!(d.xent.err = ssm::stream::error_word())) return SSM_ERR_CUDA;
  d.xent.lse_in = lse; d.xent.dloss = dloss; d.xent.dh = dh; d.xent.dweight = dweight;
  return status_of(ssm::launch_distill_bwd(d, stream));
}

ssm_status ssm_recur_fwd(const void* gate, const void* value, const float* floor,
                         const int32_t* valid_len, const float* state0, void* out_y,
                         float* out_final, float* out_states, const ssm_recur_shapes* shapes,
                         ssm_dtype dtype, cudaStream_t stream) {
  ssm_status st = check_recur(shapes, dtype);
  if (st != SSM_OK) return st;
  if (!gate || !value || !out_y) return SSM_ERR_NULL;
  const size_t es = elem_size(dtype);
  if (!aligned(gate, es) || !aligned(value, es) || !aligned(floor, 4) || !aligned(valid_len, 4) ||
      !aligned(state0, 4) || !aligned(out_y, es) || !aligned(out_final, 4) ||
      !aligned(out_states, 4))
    return SSM_ERR_ALIGN;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::RecurParams p = recur_params(gate, value, floor, valid_len, *shapes);
  p.state0 = state0; p.y = out_y; p.out_final = out_final; p.states = out_states;
  unsigned* err = ssm::stream::error_word();
  if (!err) return SSM_ERR_CUDA;
  return status_of(ssm::launch_recur_fwd(p, dtype == SSM_BF16, err, stream));
}

size_t ssm_recur_bwd_workspace_bytes(const ssm_recur_shapes* shapes) {
  if (check_recur(shapes, SSM_F32) != SSM_OK) return 0;
  return static_cast<size_t>(ssm::recur_bwd_partials(shapes->batch)) * shapes->dim * sizeof(float);
}

int64_t ssm_recur_chunks(const ssm_recur_shapes* shapes) {
  if (check_recur(shapes, SSM_F32) != SSM_OK) return 0;
  return (shapes->seqlen + ssm::kRecurChunk - 1) / ssm::kRecurChunk;
}

ssm_status ssm_recur_bwd(const void* gate, const void* value, const float* floor,
                         const int32_t* valid_len, const float* states, const void* dy,
                         const float* dfinal, void* dgate, void* dvalue, float* dfloor,
                         float* dstate0, void* workspace, size_t workspace_bytes,
                         const ssm_recur_shapes* shapes, ssm_dtype dtype, cudaStream_t stream) {
  ssm_status st = check_recur(shapes, dtype);
  if (st != SSM_OK) return st;
  if (!gate || !value || !states || !dy || !dgate || !dvalue || (dfloor && !workspace))
    return SSM_ERR_NULL;
  const size_t es = elem_size(dtype);
  if (!aligned(gate, es) || !aligned(value, es) || !aligned(floor, 4) || !aligned(valid_len, 4) ||
      !aligned(states, 4) || !aligned(dy, es) || !aligned(dfinal, 4) || !aligned(dgate, es) ||
      !aligned(dvalue, es) || !aligned(dfloor, 4) || !aligned(dstate0, 4) ||
      !aligned(workspace, 16))
    return SSM_ERR_ALIGN;
  if (dfloor && workspace_bytes < ssm_recur_bwd_workspace_bytes(shapes)) return SSM_ERR_SHAPE;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::RecurBwdParams q;
  q.fwd = recur_params(gate, value, floor, valid_len, *shapes);
  q.states = states; q.dy = dy; q.dfinal = dfinal; q.dgate = dgate; q.dvalue = dvalue;
  q.dfloor = dfloor; q.dstate0 = dstate0; q.partial = static_cast<float*>(workspace);
  unsigned* err = ssm::stream::error_word();
  if (!err) return SSM_ERR_CUDA;
  return status_of(ssm::launch_recur_bwd(q, dtype == SSM_BF16, err, stream));
}

ssm_status ssm_recur_step(const void* gate, const void* value, const float* floor, float* state,
                          void* out_y, const ssm_recur_shapes* shapes, ssm_dtype dtype,
                          cudaStream_t stream) {
  ssm_status st = check_recur(shapes, dtype);
  if (st != SSM_OK) return st;
  if (shapes->seqlen != 1) return SSM_ERR_SHAPE;
  if (!gate || !value || !state || !out_y) return SSM_ERR_NULL;
  const size_t es = elem_size(dtype);
  if (!aligned(gate, es) || !aligned(value, es) || !aligned(floor, 4) || !aligned(state, 4) ||
      !aligned(out_y, es))
    return SSM_ERR_ALIGN;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::RecurParams p = recur_params(gate, value, floor, nullptr, *shapes);
  p.y = out_y; p.out_final = state;
  return status_of(ssm::launch_recur_step(p, dtype == SSM_BF16, stream));
}

ssm_status ssm_embed_fwd(const int64_t* ids, const void* weight, void* out_y,
                         const ssm_embed_shapes* shapes, cudaStream_t stream) {
  ssm_status st = check_embed(shapes);
  if (st != SSM_OK) return st;
  const ssm_embed_shapes& s = *shapes;
  if (!ids || !weight || !out_y) return SSM_ERR_NULL;
  if (!aligned(ids, 8) || !aligned(weight, elem_size(s.dtype)) ||
      !aligned(out_y, elem_size(s.io_dtype)))
    return SSM_ERR_ALIGN;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::EmbedParams p;
  p.ids = ids; p.weight = weight; p.y = out_y;
  p.tokens = s.tokens; p.vocab = s.vocab; p.dim = s.dim;
  p.ignore = s.ignore_index; p.scale = s.scale;
  return status_of(ssm::launch_embed_fwd(p, s.dtype == SSM_BF16, s.io_dtype == SSM_BF16, stream));
}

size_t ssm_embed_bwd_workspace_bytes(const ssm_embed_shapes* shapes) {
  if (check_embed(shapes) != SSM_OK) return 0;
  return ssm::embed_bwd_workspace_bytes(shapes->tokens, shapes->dim, shapes->dtype == SSM_BF16);
}

ssm_status ssm_embed_bwd(const int64_t* ids, const void* dy, void* dweight, int add,
                         void* workspace, size_t workspace_bytes, const ssm_embed_shapes* shapes,
                         cudaStream_t stream) {
  ssm_status st = check_embed(shapes);
  if (st != SSM_OK) return st;
  const ssm_embed_shapes& s = *shapes;
  if (add != 0 && add != 1) return SSM_ERR_UNSUPPORTED;
  if (!ids || !dy || !dweight || !workspace) return SSM_ERR_NULL;
  if (!aligned(ids, 8) || !aligned(dy, elem_size(s.io_dtype)) ||
      !aligned(dweight, elem_size(s.dtype)) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (workspace_bytes < ssm_embed_bwd_workspace_bytes(shapes)) return SSM_ERR_SHAPE;
  int dev = 0;
  if ((st = current_device_for(stream, &dev)) != SSM_OK) return st;
  ssm::EmbedBwdParams p;
  p.ids = ids; p.dy = dy; p.dweight = dweight; p.add = add != 0;
  p.tokens = s.tokens; p.vocab = s.vocab; p.dim = s.dim;
  p.ignore = s.ignore_index; p.scale = s.scale; p.workspace = workspace;
  return status_of(ssm::launch_embed_bwd(p, s.dtype == SSM_BF16, s.io_dtype == SSM_BF16, stream));
}

}  // extern "C"
