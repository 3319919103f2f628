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

// Sum of v over the tpr threads of the row (tpr >= 32: whole warps; the warp
// sums meet in `red`, one slot per warp).  Every thread of the CTA takes part.
__device__ __forceinline__ float row_sum(float v, int wpr, float* red) {
#pragma unroll
  for (int m = 16; m >= 1; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (wpr == 1) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  const int first = warp & ~(wpr - 1);
  float a = 0.f;
  for (int i = 0; i < wpr; ++i) a += red[first + i];
  return a;
}

template <typename TX, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormParams p, int tpr) {
  __shared__ float red[2][32];
  const int wpr = tpr >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const int lane = threadIdx.x & (tpr - 1);
  const bool on = row < p.rows;
  const int dim = static_cast<int>(p.dim);
  const int64_t at = row * p.dim;
  float f[NV][VEC];
  if (on) {
    Raw<TX, VEC> xr[NV];
    Raw<TR, VEC> rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * VEC;
      if (c < dim) {
        xr[i] = raw_load<TX, VEC>(static_cast<const TX*>(p.x) + at + c);
        if (p.residual) rr[i] = raw_load_rw<TR, VEC>(static_cast<const TR*>(p.residual) + at + c);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * VEC;
      if (c < dim) {
        widen<VEC>(xr[i], f[i]);
        if (p.residual) {
          float g[VEC];
          widen<VEC>(rr[i], g);
#pragma unroll
          for (int v = 0; v < VEC; ++v) f[i][v] += g[v];
          Raw<TR, VEC> o;
          narrow<VEC>(f[i], o);
          raw_store<TR, VEC>(static_cast<TR*>(p.r) + at + c, o);
          widen<VEC>(o, f[i]);  // as stored
        }
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) f[i][v] = 0.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) f[i][v] = 0.f;
  }
  const float inv = 1.f / static_cast<float>(dim);
  float mean = 0.f;
  if (!p.rms) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) a += f[i][v];
    mean = row_sum(a, wpr, red[0]) * inv;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * tpr + lane) * VEC < dim) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        f[i][v] -= mean;
        q = fmaf(f[i][v], f[i][v], q);
      }
    }
  }
  const float rstd = rsqrtf(row_sum(q, wpr, red[1]) * inv + p.eps);
  if (!on) return;
  if (p.stats && lane == 0) {
    p.stats[row] = mean;
    p.stats[p.rows + row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * VEC;
    if (c < dim) {
      float w[VEC], b[VEC];
      load_f<float, VEC>(p.weight + c, w);
      if (p.bias) load_f<float, VEC>(p.bias + c, b);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        f[i][v] *= rstd * w[v];
        if (p.bias) f[i][v] += b[v];
      }
      store_f<TX, VEC>(static_cast<TX*>(p.y) + at + c, f[i]);
    }
  }
}

template <typename TX, typename TR, int VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(const NormBwdParams p, int tpr) {
  __shared__ float2 red[2][32];
  __shared__ float acc[THREADS * VEC];
  const int wpr = tpr >> 5, groups = THREADS / tpr;
  const int group = threadIdx.x / tpr, lane = threadIdx.x & (tpr - 1);
  const int dim = static_cast<int>(p.dim);
  const float inv = 1.f / static_cast<float>(dim);
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * VEC;
#pragma unroll
    for (int v = 0; v < VEC; ++v) w[i][v] = dw[i][v] = db[i][v] = 0.f;
    if (c < dim) load_f<float, VEC>(p.weight + c, w[i]);
  }
  release_next();
  int buf = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < p.rows; base += step) {
    const int64_t row = base + group;
    const bool on = row < p.rows;
    const int64_t at = row * p.dim;
    float xh[NV][VEC], g[NV][VEC];
    Raw<TR, VEC> rr[NV], er[NV];
    Raw<TX, VEC> gr[NV];
    float mean = 0.f, rstd = 0.f;
    if (on) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + lane) * VEC;
        if (c < dim) {
          rr[i] = raw_load<TR, VEC>(static_cast<const TR*>(p.r) + at + c);
          gr[i] = raw_load<TX, VEC>(static_cast<const TX*>(p.dy) + at + c);
          if (p.dr) er[i] = raw_load<TR, VEC>(static_cast<const TR*>(p.dr) + at + c);
        }
      }
      mean = p.rms ? 0.f : __ldg(p.stats + row);
      rstd = __ldg(p.stats + p.rows + row);
    }
    float2 a = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on && (i * tpr + lane) * VEC < dim) {
        widen<VEC>(rr[i], xh[i]);
        widen<VEC>(gr[i], g[i]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          xh[i][v] = (xh[i][v] - mean) * rstd;
          db[i][v] += g[i][v];
          dw[i][v] = fmaf(g[i][v], xh[i][v], dw[i][v]);
          g[i][v] *= w[i][v];
          a.x += g[i][v];
          a.y = fmaf(g[i][v], xh[i][v], a.y);
        }
      }
    }
#pragma unroll
    for (int m = 16; m >= 1; m /= 2) {
      a.x += __shfl_xor_sync(0xffffffffu, a.x, m);
      a.y += __shfl_xor_sync(0xffffffffu, a.y, m);
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
    if (on) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + lane) * VEC;
        if (c < dim) {
          float o[VEC], e[VEC];
#pragma unroll
          for (int v = 0; v < VEC; ++v) o[v] = rstd * (g[i][v] - mg - xh[i][v] * mx);
          if (p.dr) {
            widen<VEC>(er[i], e);
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[v] += e[v];
          }
          if (p.dx) store_f<TX, VEC>(static_cast<TX*>(p.dx) + at + c, o);
          if (p.dresidual) store_f<TR, VEC>(static_cast<TR*>(p.dresidual) + at + c, o);
        }
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
        if (c < dim) p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + k) * p.dim + c] = s;
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

// Threads per row, whole warps: at most `per` elements of the row per thread.
int threads_per_row(int64_t dim, int per) {
  int t = 32;
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

constexpr int kBwdPer = 8;       // elements of a row per thread: 1024 threads hold kNormMaxDim
constexpr int kBwdThreads = 256; // threads per CTA, for rows of up to that many threads
constexpr int kBwdCtasPerSm = 4;

int64_t bwd_ctas(int64_t rows, int tpr) {
  const int threads = tpr > kBwdThreads ? tpr : kBwdThreads;
  const int64_t groups = threads / tpr, need = (rows + groups - 1) / groups;
  const int64_t most = int64_t(kSms) * kBwdCtasPerSm * kBwdThreads / threads;
  return need < most ? need : most;
}

template <typename TX, typename TR, int VEC>
cudaError_t norm_bwd_v(const NormBwdParams& p, cudaStream_t s) {
  constexpr int NV = kBwdPer / VEC;
  const int tpr = threads_per_row(p.dim, kBwdPer);
  const unsigned g = static_cast<unsigned>(bwd_ctas(p.rows, tpr));
  switch (tpr) {
    case 512: norm_bwd_kernel<TX, TR, VEC, NV, 512><<<g, 512, 0, s>>>(p, tpr); break;
    case 1024: norm_bwd_kernel<TX, TR, VEC, NV, 1024><<<g, 1024, 0, s>>>(p, tpr); break;
    default: norm_bwd_kernel<TX, TR, VEC, NV, kBwdThreads><<<g, kBwdThreads, 0, s>>>(p, tpr);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
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
  return bwd_ctas(rows, threads_per_row(dim, kBwdPer));
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, bool bf16, bool residual_bf16,
                            cudaStream_t s) {
  if (p.dim > kNormMaxDim) return cudaErrorInvalidValue;
  if (!bf16) return norm_bwd_t<float, float>(p, s);
  return residual_bf16 ? norm_bwd_t<__nv_bfloat16, __nv_bfloat16>(p, s)
                       : norm_bwd_t<__nv_bfloat16, float>(p, s);
}

}  // namespace ssm
