// api_layers.cu -- the C ABI of the operators around the scan (declared in
// include/ssmscan.h): argument validation and launch.  Every argument error is
// found here, before anything is enqueued, and is returned as an ssm_status.
#include <cuda_runtime.h>
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

ssm::XentParams xent_params(const void* h, const void* weight, const int64_t* targets,
                            const ssm_xent_shapes& s, void* workspace) {
  ssm::XentParams p = {};
  p.h = h; p.weight = weight; p.targets = targets; p.ignore_index = s.ignore_index;
  p.shape = {s.tokens, s.vocab, s.dim};
  p.workspace = workspace;
  return p;
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

}  // extern "C"
