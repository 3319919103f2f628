// kernel_norm.cu -- the norm of the residual stream, with the addition that
// precedes it, and its backward.
//
//   r = x + residual (stored in the residual's type; r = x without one)
//   y = (r - mean(r)) rstd w + b,   rstd = 1 / sqrt(var(r) + eps)
// or, as the root-mean-square form, mean = 0 and var = mean(r^2).  The norm is
// taken of r as stored, so that the backward, which reads r again, sees the
// values that were normalised.  Statistics are fp32: the mean first, then the
// centred squares, both from registers.
//
// With xhat = (r - mean) rstd and g = dy w, the backward is
//   dr_total = rstd (g - mean(g) - xhat mean(g xhat)) + dr
//   dw = sum over rows of dy xhat,   db = sum over rows of dy
// (mean(g) only with a mean).  dr is the gradient that arrives along the
// residual stream; dr_total is the gradient of x and of the residual.
//
// Bound by HBM: every tensor is moved once.  A row is held in registers by
// `tpr` threads (a power of two), NV groups of VEC elements each.  The backward
// keeps CTAs resident and walks rows, so that every thread sums dw and db of
// its own columns in registers; the CTAs' sums are written once and added by a
// second kernel in a fixed order (no atomics).
#include "common.cuh"
#include "layers.h"
#include "pdl.cuh"
#include "vec.cuh"

namespace ssm {
namespace {

constexpr int kSms = 152;
constexpr int kBwdPer = 8;  // backward: elements of a row per thread, up to 512 threads; then twice as many
constexpr int kBwdWarpsPerSm = 20;  // backward: what the registers are shared out for
__host__ __device__ constexpr int bwd_ctas_per_sm(int threads) {
  return kBwdWarpsPerSm * 32 / threads;
}

// Sum of v over the tpr threads of the row (a part of a warp, or whole warps,
// whose sums meet in `red`, one slot per warp).  Every thread of the CTA takes
// part.
__device__ __forceinline__ float row_sum(float v, int tpr, float* red) {
#pragma unroll
  for (int m = 16; m >= 1; m /= 2) {
    const float o = __shfl_xor_sync(0xffffffffu, v, m);
    v += m < tpr ? o : 0.f;
  }
  if (tpr <= 32) return v;
  const int wpr = tpr >> 5;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  const int first = warp & ~(wpr - 1);
  float a = 0.f;
  for (int i = 0; i < wpr; ++i) a += red[first + i];
  return a;
}

// Group i of a thread's columns starts at column (i tpr + lane) VEC.  Loads past
// the row's end are made at its last group instead, and their values dropped,
// so that no load waits on a branch.
template <int VEC>
__device__ __forceinline__ int clamped(int c, int dim) {
  return c < dim ? c : dim - VEC;
}

template <typename TX, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(VEC * NV == 8 ? 1024 : 512)
    norm_fwd_kernel(const NormParams p, int tpr) {
  __shared__ float red[2][32];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const int lane = threadIdx.x & (tpr - 1);
  const bool on = row < p.rows;
  const int dim = static_cast<int>(p.dim);
  const int64_t at = (on ? row : p.rows - 1) * p.dim;  // groups without a row write nothing
  const TX* x = static_cast<const TX*>(p.x) + at;
  float f[NV][VEC];
  Raw<TX, VEC> xr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    xr[i] = raw_load<TX, VEC>(x + clamped<VEC>((i * tpr + lane) * VEC, dim));
  if (p.residual) {
    const TR* res = static_cast<const TR*>(p.residual) + at;
    TR* out = static_cast<TR*>(p.r) + at;
    Raw<TR, VEC> rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      rr[i] = raw_load_rw<TR, VEC>(res + clamped<VEC>((i * tpr + lane) * VEC, dim));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * VEC;
      float g[VEC];
      widen<VEC>(xr[i], f[i]);
      widen<VEC>(rr[i], g);
#pragma unroll
      for (int v = 0; v < VEC; ++v) f[i][v] += g[v];
      Raw<TR, VEC> o;
      narrow<VEC>(f[i], o);
      if (on && c < dim) raw_store<TR, VEC>(out + c, o);
      widen<VEC>(o, f[i]);  // as stored
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) widen<VEC>(xr[i], f[i]);
  }
  const float inv = 1.f / static_cast<float>(dim);
  float mean = 0.f;
  if (!p.rms) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * tpr + lane) * VEC < dim;
#pragma unroll
      for (int v = 0; v < VEC; ++v) a += in ? f[i][v] : 0.f;
    }
    mean = row_sum(a, tpr, red[0]) * inv;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = (i * tpr + lane) * VEC < dim;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      f[i][v] -= mean;
      q = fmaf(in ? f[i][v] : 0.f, f[i][v], q);
    }
  }
  const float rstd = rsqrtf(row_sum(q, tpr, red[1]) * inv + p.eps);
  if (!on) return;
  if (p.stats && lane == 0) {
    p.stats[row] = mean;
    p.stats[p.rows + row] = rstd;
  }
  TX* y = static_cast<TX*>(p.y) + at;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[VEC];
    load_f<float, VEC>(p.weight + clamped<VEC>((i * tpr + lane) * VEC, dim), w);
#pragma unroll
    for (int v = 0; v < VEC; ++v) f[i][v] *= rstd * w[v];
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float b[VEC];
      load_f<float, VEC>(p.bias + clamped<VEC>((i * tpr + lane) * VEC, dim), b);
#pragma unroll
      for (int v = 0; v < VEC; ++v) f[i][v] += b[v];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * VEC;
    if (c < dim) store_f<TX, VEC>(y + c, f[i]);
  }
}

// A row's operands of one thread, as loaded.
template <typename TX, typename TR, int VEC, int NV>
struct RowRaw {
  Raw<TR, VEC> r[NV], dr[NV];
  Raw<TX, VEC> dy[NV];
  float mean, rstd;
};

// The loads of the next row are in flight while a row is reduced and written.
template <typename TX, typename TR, int VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, bwd_ctas_per_sm(THREADS))
    norm_bwd_kernel(const NormBwdParams p, int tpr) {
  __shared__ float2 red[2][32];
  __shared__ float acc[THREADS * VEC];
  const int wpr = tpr >> 5, groups = THREADS / tpr;
  const int group = threadIdx.x / tpr, lane = threadIdx.x & (tpr - 1);
  const int dim = static_cast<int>(p.dim);
  const float inv = 1.f / static_cast<float>(dim);
  const bool has_dr = p.dr != nullptr;
  constexpr bool kHoldW = NV * VEC == kBwdPer;  // wider rows read the weight again per row
  float w[kHoldW ? NV : 1][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (kHoldW)
      load_f<float, VEC>(p.weight + clamped<VEC>((i * tpr + lane) * VEC, dim), w[i]);
#pragma unroll
    for (int v = 0; v < VEC; ++v) dw[i][v] = db[i][v] = 0.f;
  }
  release_next();
  const auto load = [&](RowRaw<TX, TR, VEC, NV>& x, int64_t row) {
    if (row >= p.rows) return;
    const int64_t at = row * p.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t o = at + clamped<VEC>((i * tpr + lane) * VEC, dim);
      x.r[i] = raw_load<TR, VEC>(static_cast<const TR*>(p.r) + o);
      x.dy[i] = raw_load<TX, VEC>(static_cast<const TX*>(p.dy) + o);
    }
    if (has_dr) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        x.dr[i] = raw_load<TR, VEC>(static_cast<const TR*>(p.dr) + at +
                                    clamped<VEC>((i * tpr + lane) * VEC, dim));
    }
    x.mean = p.rms ? 0.f : __ldg(p.stats + row);
    x.rstd = __ldg(p.stats + p.rows + row);
  };
  int buf = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  RowRaw<TX, TR, VEC, NV> next = {};
  load(next, static_cast<int64_t>(blockIdx.x) * groups + group);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < p.rows; base += step) {
    const int64_t row = base + group;
    const bool on = row < p.rows;
    const int64_t at = row * p.dim;
    const float mean = next.mean, rstd = next.rstd;
    float xh[NV][VEC], g[NV][VEC];
    Raw<TR, VEC> er[NV];
    float2 a = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = on && (i * tpr + lane) * VEC < dim;
      widen<VEC>(next.r[i], xh[i]);
      widen<VEC>(next.dy[i], g[i]);
      er[i] = next.dr[i];
      float wi[VEC];
      if constexpr (kHoldW) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) wi[v] = w[i][v];
      } else {
        load_f<float, VEC>(p.weight + clamped<VEC>((i * tpr + lane) * VEC, dim), wi);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        xh[i][v] = in ? (xh[i][v] - mean) * rstd : 0.f;
        g[i][v] = in ? g[i][v] : 0.f;
        db[i][v] += g[i][v];
        dw[i][v] = fmaf(g[i][v], xh[i][v], dw[i][v]);
        g[i][v] *= wi[v];
        a.x += g[i][v];
        a.y = fmaf(g[i][v], xh[i][v], a.y);
      }
    }
    load(next, row + step);
#pragma unroll
    for (int m = 16; m >= 1; m /= 2) {
      const float ox = __shfl_xor_sync(0xffffffffu, a.x, m);
      const float oy = __shfl_xor_sync(0xffffffffu, a.y, m);
      a.x += m < tpr ? ox : 0.f;
      a.y += m < tpr ? oy : 0.f;
    }
    if (wpr > 1) {  // two buffers: a row's sums are read before the buffer's next writes
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) red[buf][warp] = a;
      __syncthreads();
      const int first = warp & ~(wpr - 1);
      a = make_float2(0.f, 0.f);
      for (int i = 0; i < wpr; ++i) {
        a.x += red[buf][first + i].x;
        a.y += red[buf][first + i].y;
      }
      buf ^= 1;
    }
    const float mg = p.rms ? 0.f : a.x * inv, mx = a.y * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * VEC;
      float o[VEC], e[VEC];
      widen<VEC>(er[i], e);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        o[v] = rstd * (g[i][v] - mg - xh[i][v] * mx);
        o[v] = has_dr ? o[v] + e[v] : o[v];
      }
      if (on && c < dim) {
        store_f<TX, VEC>(static_cast<TX*>(p.dx) + at + c, o);
        if (p.dresidual) store_f<TR, VEC>(static_cast<TR*>(p.dresidual) + at + c, o);
      }
    }
  }
  // the row groups' sums, added in the order of the groups
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[threadIdx.x * VEC + v] = k == 0 ? dw[i][v] : db[i][v];
      __syncthreads();
      const int wide = tpr * VEC;
      for (int j = threadIdx.x; j < wide; j += THREADS) {
        const int c = i * wide + j;
        float s = 0.f;
        for (int u = 0; u < groups; ++u) s += acc[u * wide + j];
        if (c >= dim) continue;
        if (gridDim.x > 1)
          p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + k) * p.dim + c] = s;
        else if (k == 0)  // the only CTA: its sums are the result
          p.dweight[c] = s;
        else if (p.dbias)
          p.dbias[c] = s;
      }
    }
  }
}

// dw and db: the sums of the CTAs' partial sums, 32 warps to 32 columns.
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float* partial, float* dweight,
                                                            float* dbias, int64_t dim, int parts) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int k = blockIdx.y;
  wait_previous();
  float a = 0.f;
  if (d < dim) {
#pragma unroll 8
    for (int j = wy; j < parts; j += 32) a += partial[(static_cast<int64_t>(j) * 2 + k) * dim + d];
  }
  red[lane][wy] = a;
  __syncthreads();
  float v = red[wy][lane];  // warp wy joins column wy
#pragma unroll
  for (int m = 16; m >= 1; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + wy;
  if (lane == 0 && o < dim) (k == 0 ? dweight : dbias)[o] = v;
}

bool fits(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Threads per row, a power of two: at most `per` elements of the row per thread.
int threads_per_row(int64_t dim, int per) {
  int t = 8;
  while (int64_t(t) * per < dim) t *= 2;
  return t;
}

// Rows are held 8 elements per thread where there are few of them (a row's
// latency counts), else 16 (fewer threads to synchronise per row).
template <typename TX, typename TR, int VEC>
cudaError_t norm_fwd_v(const NormParams& p, cudaStream_t s) {
  const int per = p.rows < 4 * kSms ? 8 : 16;
  const int tpr = threads_per_row(p.dim, per);
  const int threads = tpr > 128 ? tpr : 128;
  const int64_t rpb = threads / tpr, blocks = (p.rows + rpb - 1) / rpb;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(blocks);
  if (per == 8)
    norm_fwd_kernel<TX, TR, VEC, 8 / VEC><<<g, threads, 0, s>>>(p, tpr);
  else
    norm_fwd_kernel<TX, TR, VEC, 16 / VEC><<<g, threads, 0, s>>>(p, tpr);
  return cudaGetLastError();
}

template <typename TX, typename TR>
cudaError_t norm_fwd_t(const NormParams& p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(TX);
  const bool vec = p.dim % V == 0 && fits(p.x, 16) && fits(p.y, 16) && fits(p.residual, 16) &&
                   fits(p.r, 16) && fits(p.weight, 16) && fits(p.bias, 16);
  return vec ? norm_fwd_v<TX, TR, V>(p, s) : norm_fwd_v<TX, TR, 1>(p, s);
}

int bwd_threads(int64_t dim) {
  const int t = threads_per_row(dim, kBwdPer);
  return t < 512 ? t : 512;
}

int64_t bwd_ctas(int64_t rows, int tpr) {
  const int threads = tpr > 128 ? tpr : 128;
  const int64_t groups = threads / tpr, need = (rows + groups - 1) / groups;
  if (need <= 4) return 1;  // a few rows in turn cost less than a second kernel for the sums
  const int64_t most = int64_t(kSms) * bwd_ctas_per_sm(threads);
  return need < most ? need : most;
}

template <typename TX, typename TR, int VEC>
cudaError_t norm_bwd_v(const NormBwdParams& p, cudaStream_t s) {
  constexpr int NV = kBwdPer / VEC;
  const int tpr = bwd_threads(p.dim);
  const unsigned g = static_cast<unsigned>(bwd_ctas(p.rows, tpr));
  if (p.dim > kBwdPer * 512)
    norm_bwd_kernel<TX, TR, VEC, 2 * NV, 512><<<g, 512, 0, s>>>(p, tpr);
  else if (tpr == 512)
    norm_bwd_kernel<TX, TR, VEC, NV, 512><<<g, 512, 0, s>>>(p, tpr);
  else if (tpr == 256)
    norm_bwd_kernel<TX, TR, VEC, NV, 256><<<g, 256, 0, s>>>(p, tpr);
  else
    norm_bwd_kernel<TX, TR, VEC, NV, 128><<<g, 128, 0, s>>>(p, tpr);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || g == 1) return e;
  return launch_after(norm_bwd_sum_kernel,
                      dim3(static_cast<unsigned>((p.dim + 31) / 32), p.dbias ? 2 : 1), 1024, 0, s,
                      p.partial, p.dweight, p.dbias, p.dim, static_cast<int>(g));
}

template <typename TX, typename TR>
cudaError_t norm_bwd_t(const NormBwdParams& p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(TX);
  const bool vec = p.dim % V == 0 && fits(p.r, 16) && fits(p.dy, 16) && fits(p.dr, 16) &&
                   fits(p.dx, 16) && fits(p.dresidual, 16) && fits(p.weight, 16);
  return vec ? norm_bwd_v<TX, TR, V>(p, s) : norm_bwd_v<TX, TR, 1>(p, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormParams& p, bool bf16, bool residual_bf16, cudaStream_t s) {
  if (p.dim > kNormMaxDim) return cudaErrorInvalidValue;
  if (!bf16) return norm_fwd_t<float, float>(p, s);
  return residual_bf16 ? norm_fwd_t<__nv_bfloat16, __nv_bfloat16>(p, s)
                       : norm_fwd_t<__nv_bfloat16, float>(p, s);
}

int64_t norm_bwd_partials(int64_t rows, int64_t dim) {
  return bwd_ctas(rows, bwd_threads(dim));
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, bool bf16, bool residual_bf16,
                            cudaStream_t s) {
  if (p.dim > kNormMaxDim) return cudaErrorInvalidValue;
  if (!bf16) return norm_bwd_t<float, float>(p, s);
  return residual_bf16 ? norm_bwd_t<__nv_bfloat16, __nv_bfloat16>(p, s)
                       : norm_bwd_t<__nv_bfloat16, float>(p, s);
}

}  // namespace ssm
