// layers.h -- parameters and launchers of the operators around the scan: the
// short causal convolution, the norm of the residual stream and the softmax
// cross entropy over the vocabulary.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

// Bits of the sticky device error word that the bounded waits of these operators
// set, one each.  The scan's kernels have 1 (STREAM and the tiled backward), 2 and 4
// (SSD form) and 8 (STREAM-TM).
constexpr unsigned kErrConvWait = 16u;
constexpr unsigned kErrXentWait = 32u;

// ---- short causal convolution (kernel_conv.cu) ------------------------------
struct ConvParams {
  const void* x;             // [batch, seqlen, dim], channels contiguous
  int64_t x_batch, x_step;   // strides of x in elements
  const float* weight;       // [dim, width]
  const float* bias;         // nullable, [dim]
  const int32_t* valid_len;  // nullable, [batch]
  const void* state0;        // nullable, [batch, width - 1, dim]: the steps before the first
  void* y;                   // [batch, seqlen, dim]
  void* out_final;           // nullable, [batch, width - 1, dim]
  int64_t batch, seqlen, dim;
  int width, silu;
};

struct ConvBwdParams {
  ConvParams fwd;       // y, out_final unused
  const void* dy;       // [batch, seqlen, dim]
  void* dx;             // [batch, seqlen, dim]
  void* dstate0;        // nullable, [batch, width - 1, dim]
  float* dweight;       // [dim, width]
  float* dbias;         // nullable, [dim]
  float* partial;       // workspace: [conv_bwd_partials, width + 1, dim]
};

struct ConvStepParams {
  const void* x;        // [batch, dim]
  int64_t x_batch;      // stride of x in elements
  const float* weight;
  const float* bias;
  void* state;          // [batch, width - 1, dim], advanced in place
  void* y;              // [batch, dim]
  int64_t batch, dim;
  int width, silu;
};

inline bool conv_supported_width(int64_t k) { return k >= 2 && k <= 4; }
// `err`: the sticky error word of the bounded waits.
cudaError_t launch_conv_fwd(const ConvParams& p, bool bf16, unsigned* err, cudaStream_t s);
int64_t conv_bwd_partials(int64_t batch, int64_t seqlen, int64_t dim, int width);
cudaError_t launch_conv_bwd(const ConvBwdParams& p, bool bf16, unsigned* err, cudaStream_t s);
// The forms whose rows are staged by TMA (kernel_conv_tma.cu), and whether a
// call's tensors allow it.
bool conv_tma_ok(const ConvParams& p, bool bf16);
bool conv_bwd_tma_ok(const ConvBwdParams& p, bool bf16);
int64_t conv_bwd_tma_partials(int64_t batch, int64_t seqlen, int64_t dim, int width);
cudaError_t launch_conv_fwd_tma(const ConvParams& p, bool bf16, unsigned* err, cudaStream_t s);
cudaError_t launch_conv_bwd_tma(const ConvBwdParams& p, bool bf16, unsigned* err, int* parts,
                                cudaStream_t s);
cudaError_t launch_conv_step(const ConvStepParams& p, bool bf16, cudaStream_t s);

// ---- norm of the residual stream (kernel_norm.cu) ----------------------------
constexpr int64_t kNormMaxDim = 8192;  // a row is held in the registers of one CTA
struct NormParams {
  const void* x;         // [rows, dim], I/O type
  const void* residual;  // nullable, [rows, dim], residual type
  const float* weight;   // [dim]
  const float* bias;     // nullable, [dim]
  void* y;               // [rows, dim], I/O type
  void* r;               // [rows, dim], residual type; written when residual is given
  float* stats;          // nullable, [2, rows]: mean, reciprocal standard deviation
  int64_t rows, dim;
  int rms;
  float eps;
};

struct NormBwdParams {
  const void* r;         // [rows, dim]: what was normalised, residual type
  const float* weight;
  const float* stats;    // [2, rows]
  const void* dy;        // [rows, dim], I/O type
  const void* dr;        // nullable, [rows, dim], residual type
  void* dx;              // [rows, dim], I/O type
  void* dresidual;       // nullable, [rows, dim], residual type
  float* dweight;        // [dim]
  float* dbias;          // nullable, [dim]
  float* partial;        // workspace: [norm_bwd_partials, 2, dim]
  int64_t rows, dim;
  int rms;
};

cudaError_t launch_norm_fwd(const NormParams& p, bool bf16, bool residual_bf16, cudaStream_t s);
int64_t norm_bwd_partials(int64_t rows, int64_t dim);
cudaError_t launch_norm_bwd(const NormBwdParams& p, bool bf16, bool residual_bf16, cudaStream_t s);

// ---- softmax cross entropy over the vocabulary (kernel_xent.cu) ----------------
struct XentShape {
  int64_t tokens, vocab, dim;
};

struct XentParams {
  const void* h;            // [tokens, dim] bf16
  const void* weight;       // [vocab, dim] bf16
  const int64_t* targets;   // [tokens]
  int64_t ignore_index;
  XentShape shape;
  void* workspace;
  unsigned int* err;        // sticky error word of the bounded waits
  // forward
  float* loss;              // [tokens]
  float* lse;               // [tokens]
  // backward
  const float* lse_in;      // [tokens]
  const float* dloss;       // [tokens]
  void* dh;                 // [tokens, dim] bf16
  void* dweight;            // [vocab, dim] bf16
};

size_t xent_workspace_bytes(const XentShape& s, bool backward);
cudaError_t launch_xent_fwd(const XentParams& p, cudaStream_t s);
cudaError_t launch_xent_bwd(const XentParams& p, cudaStream_t s);

}  // namespace ssm
