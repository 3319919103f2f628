// kernel_conv.cu -- the short causal convolution in front of the scan: every
// channel is filtered along time with its own `width` (2 to 4) taps,
//   pre[t] = bias + sum_k w[k] x[t - (width - 1) + k],   y = silu(pre) or pre,
// the steps before the first taken from a carried state (zeros without one).
// Steps past valid_len give y = 0, whatever x holds there.
//
// Bound by HBM: each element is read and written once, for `width` fused
// multiply-adds and one MUFU pair.  A thread holds VEC channels with their taps
// in registers and walks along time with the last width - 1 rows in registers,
// so a row is loaded once.  A sequence is cut into chunks of steps for
// parallelism; a chunk re-reads the width - 1 rows before it.  Tensors whose
// rows start on 16-byte boundaries take the TMA-staged kernels
// (kernel_conv_tma.cu); the kernels here take any other (odd widths, odd
// offsets, strides that are no multiples) one channel per thread with U rows in flight.  Training step bf16
// 4 x 2000 x 513: 19.8 us, against 18.5 us for 512 channels staged by TMA.
//
// The backward, with dpre = dy silu'(pre) (pre formed again from x) and 0 past
// valid_len:
//   dx[t] = sum_k w[k] dpre[t + (width - 1) - k],
//   dw[k] = sum_{b,t} dpre[t] x[t - (width - 1) + k],   dbias = sum_{b,t} dpre[t].
// The same walk, with the last width values of dpre in registers too and
// width - 1 steps run past the chunk's end.  dw and dbias are summed per
// thread, then over the threads of the CTA in a fixed order, then over the
// CTAs by a second kernel: no atomics, so the sums do not depend on timing.
#include "conv.cuh"
#include "pdl.cuh"

namespace ssm {
namespace {

constexpr int kConvThreads = 256;
constexpr int kSms = 152;

constexpr int U = 8;         // rows in flight per thread
constexpr int kFwdCtas = 3, kBwdCtas = 2;  // resident CTAs per SM

// Steps per chunk.  A thread's time is its number of chunks times their length
// and the `halo` steps a chunk adds; short chunks spread the work evenly, long
// ones add less.
int chunk_steps(int64_t batch, int64_t seqlen, int64_t dim, int ctas_per_sm, int halo) {
  const int64_t slots = int64_t(kSms) * ctas_per_sm * kConvThreads;
  int best = 64;
  int64_t least = INT64_MAX;
  for (int tc : {64, 48, 32, 24, 16, 8}) {
    const int64_t per = (batch * ((seqlen + tc - 1) / tc) * dim + slots - 1) / slots;
    if (per * (tc + halo) < least) {
      least = per * (tc + halo);
      best = tc;
    }
  }
  return best;
}

// Channels per CTA (a power of two): a warp along the channels where
// there are enough of them.
int lanes_log2(int64_t dim) { return dim >= 32 ? 5 : dim >= 16 ? 4 : 3; }

struct ConvGrid {
  int tc, lx;
  int64_t chunks, gx, gy;
};

ConvGrid conv_grid(int64_t batch, int64_t seqlen, int64_t dim, int ctas_per_sm, int halo) {
  ConvGrid g;
  g.tc = chunk_steps(batch, seqlen, dim, ctas_per_sm, halo);
  g.lx = lanes_log2(dim);
  g.chunks = (seqlen + g.tc - 1) / g.tc;
  const int64_t ty = kConvThreads >> g.lx;
  g.gx = (dim + (int64_t(1) << g.lx) - 1) >> g.lx;
  const int64_t need = (batch * g.chunks + ty - 1) / ty;
  const int64_t most = (int64_t(kSms) * ctas_per_sm + g.gx - 1) / g.gx;
  g.gy = need < most ? need : most;
  return g;
}

template <typename T, int K>
__global__ void __launch_bounds__(kConvThreads, kFwdCtas)
    conv_fwd_kernel(const ConvParams p, int tc, int lx, int64_t chunks) {
  constexpr int VEC = 1;  // channels per thread
  const int64_t d0 = (static_cast<int64_t>(blockIdx.x) << lx) + (threadIdx.x & ((1 << lx) - 1));
  if (d0 >= p.dim) return;
  const int64_t ty = kConvThreads >> lx, items = p.batch * chunks;
  float w[K][VEC], bv[VEC];
  load_taps<K, VEC>(p.weight, p.bias, d0, w, bv);
  for (int64_t it = blockIdx.y * ty + (threadIdx.x >> lx); it < items; it += gridDim.y * ty) {
    const int64_t b = it / chunks, c = it - b * chunks;
    const int64_t t0 = c * tc;
    const int64_t vl = conv_valid(p, b);
    const int n = static_cast<int>(p.seqlen - t0 < tc ? p.seqlen - t0 : tc);  // steps of the chunk
    const int nv = static_cast<int>(vl - t0 < 0 ? 0 : vl - t0 < n ? vl - t0 : n);  // valid ones
    const T* xb = static_cast<const T*>(p.x) + b * p.x_batch + d0;
    T* y = static_cast<T*>(p.y) + (b * p.seqlen + t0) * p.dim + d0;
    if (nv > 0) {
      const T* x = xb + t0 * p.x_step;
      float win[K - 1][VEC];
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
        widen<VEC>(t0 > 0 ? raw_load<T, VEC>(x - (K - 1 - k) * p.x_step)
                          : state_row<T, K, VEC>(p.state0, b, p.dim, d0, k),
                   win[k]);
      auto emit = [&](const Raw<T, VEC>& raw) {
        float cur[VEC], pre[VEC];
        widen<VEC>(raw, cur);
        taps<K, VEC>(w, bv, win, cur, pre);
        if (p.silu) apply_silu<VEC>(pre);
        store_f<T, VEC>(y, pre);
        y += p.dim;
        push<K, VEC>(win, cur);
      };
      int i = 0;
      for (; i + U <= nv; i += U) {  // U rows in flight
        Raw<T, VEC> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          raw[u] = raw_load<T, VEC>(x);
          x += p.x_step;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) emit(raw[u]);
      }
#pragma unroll 1
      for (; i < nv; ++i, x += p.x_step) emit(raw_load<T, VEC>(x));
    }
    Raw<T, VEC> z;
    raw_zero<T, VEC>(z);
    for (int i = nv; i < n; ++i, y += p.dim) raw_store<T, VEC>(y, z);
    if (c == 0 && p.out_final != nullptr) {
      T* fb = static_cast<T*>(p.out_final) + b * (K - 1) * p.dim + d0;
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {
        const int64_t t = vl - (K - 1) + k;
        raw_store<T, VEC>(fb + k * p.dim,
                          t >= 0 ? raw_load<T, VEC>(xb + t * p.x_step)
                                 : state_row<T, K, VEC>(p.state0, b, p.dim, d0,
                                                        static_cast<int>(t) + K - 1));
      }
    }
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(kConvThreads, kBwdCtas)
    conv_bwd_kernel(const ConvBwdParams q, int tc, int lx, int64_t chunks) {
  constexpr int VEC = 1;  // channels per thread
  const ConvParams& p = q.fwd;
  const int tx = threadIdx.x & ((1 << lx) - 1);
  const int64_t d0 = (static_cast<int64_t>(blockIdx.x) << lx) + tx;
  const bool on = d0 < p.dim;
  const int ty = kConvThreads >> lx;
  const int64_t items = on ? p.batch * chunks : 0;
  release_next();
  float w[K][VEC], bv[VEC], dw[K][VEC], db[VEC] = {0.f};
#pragma unroll
  for (int k = 0; k < K; ++k) dw[k][0] = 0.f;
  if (on) load_taps<K, VEC>(p.weight, p.bias, d0, w, bv);
  for (int64_t it = static_cast<int64_t>(blockIdx.y) * ty + (threadIdx.x >> lx); it < items;
       it += static_cast<int64_t>(gridDim.y) * ty) {
    const int64_t b = it / chunks, c = it - b * chunks;
    const int64_t t0 = c * tc;
    const int64_t vl = conv_valid(p, b);
    const int n = static_cast<int>(p.seqlen - t0 < tc ? p.seqlen - t0 : tc);  // steps of the chunk
    // steps from the chunk's first that have a dpre; dx[n - 1] needs dpre up to n + K - 2
    const int nl = static_cast<int>(vl - t0 < 0 ? 0 : vl - t0 < n + K - 1 ? vl - t0 : n + K - 1);
    const T* x = static_cast<const T*>(p.x) + b * p.x_batch + t0 * p.x_step + d0;
    const T* gy = static_cast<const T*>(q.dy) + (b * p.seqlen + t0) * p.dim + d0;
    // dx of step i - (K - 1), written at step i
    T* o = static_cast<T*>(q.dx) + (b * p.seqlen + t0 - (K - 1)) * p.dim + d0;
    float win[K - 1][VEC], dp[K - 1][VEC];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      win[k][0] = dp[k][0] = 0.f;
      if (nl > 0)
        widen<VEC>(t0 > 0 ? raw_load<T, VEC>(x - (K - 1 - k) * p.x_step)
                          : state_row<T, K, VEC>(p.state0, b, p.dim, d0, k),
                   win[k]);
    }
    // dx from the window of dpre and the step's own
    auto emit = [&](int i, const float(&g)[VEC]) {
      float a[VEC];
      dx_taps<K, VEC>(w, dp, g, a);
      if (i >= K - 1)
        store_f<T, VEC>(o, a);
      else if (c == 0 && q.dstate0)
        store_f<T, VEC>(static_cast<T*>(q.dstate0) + (b * (K - 1) + i) * p.dim + d0, a);
      o += p.dim;
      push<K, VEC>(dp, g);
    };
    auto step = [&](int i, const Raw<T, VEC>& xr, const Raw<T, VEC>& gr) {
      float cur[VEC], g[VEC];
      widen<VEC>(xr, cur);
      widen<VEC>(gr, g);
      if (p.silu) {
        float pre[VEC];
        taps<K, VEC>(w, bv, win, cur, pre);
        apply_dsilu<VEC>(pre, g);
      }
      if (i < n) add_dw<K, VEC>(dw, db, g, win, cur);
      emit(i, g);
      push<K, VEC>(win, cur);
    };
    int i = 0;
    for (; i + U <= nl; i += U) {  // U rows of x and of dy in flight
      Raw<T, VEC> xr[U], gr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xr[u] = raw_load<T, VEC>(x);
        gr[u] = raw_load<T, VEC>(gy);
        x += p.x_step;
        gy += p.dim;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) step(i + u, xr[u], gr[u]);
    }
#pragma unroll 1
    for (; i < nl; ++i, x += p.x_step, gy += p.dim)
      step(i, raw_load<T, VEC>(x), raw_load<T, VEC>(gy));
    const float none[VEC] = {0.f};
#pragma unroll 1
    for (; i < n + K - 1; ++i) emit(i, none);
  }

  // sums over the CTA's time slots: quantity k < K is tap k, quantity K the bias
  __shared__ float red[kConvThreads];
  const int wide = 1 << lx;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    __syncthreads();
    red[threadIdx.x] = k < K ? dw[k < K ? k : 0][0] : db[0];
    __syncthreads();
    for (int i = threadIdx.x; i < wide; i += kConvThreads) {
      const int64_t d = (static_cast<int64_t>(blockIdx.x) << lx) + i;
      float a = 0.f;
      for (int j = 0; j < ty; ++j) a += red[j * wide + i];
      if (d >= p.dim) continue;
      if (gridDim.y > 1)
        q.partial[(static_cast<int64_t>(blockIdx.y) * (K + 1) + k) * p.dim + d] = a;
      else if (k < K)  // the channels' only CTA: its sums are the result
        q.dweight[d * K + k] = a;
      else if (q.dbias)
        q.dbias[d] = a;
    }
  }
}

// dweight[d][k] and dbias[d]: the sums of the CTAs' partial sums, 32 warps to 32
// channels.
__global__ void __launch_bounds__(1024) conv_bwd_sum_kernel(const float* partial, float* dweight,
                                                            float* dbias, int64_t dim, int width,
                                                            int parts) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int k = blockIdx.y;
  wait_previous();
  float a = 0.f;
  if (d < dim) {
#pragma unroll 8
    for (int j = wy; j < parts; j += 32)
      a += partial[(static_cast<int64_t>(j) * (width + 1) + k) * dim + d];
  }
  red[lane][wy] = a;
  __syncthreads();
  float v = red[wy][lane];  // warp wy joins channel wy
#pragma unroll
  for (int m = 16; m >= 1; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + wy;
  if (lane == 0 && o < dim) {
    if (k < width)
      dweight[o * width + k] = v;
    else
      dbias[o] = v;
  }
}

// One step for R batch rows per thread: the taps are read once for all of them.
template <typename T, int K, int VEC, int R>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvStepParams p, int64_t cvs) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t b0 = i / cvs * R, d0 = (i - i / cvs * cvs) * VEC;
  if (b0 >= p.batch) return;
  Raw<T, VEC> win[R][K];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t b = b0 + r < p.batch ? b0 + r : p.batch - 1;  // past the last: read, not written
    const T* st = static_cast<const T*>(p.state) + b * (K - 1) * p.dim + d0;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) win[r][k] = raw_load_rw<T, VEC>(st + k * p.dim);
    win[r][K - 1] = raw_load<T, VEC>(static_cast<const T*>(p.x) + b * p.x_batch + d0);
  }
  float w[K][VEC], bv[VEC];
  load_taps<K, VEC>(p.weight, p.bias, d0, w, bv);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (b0 + r >= p.batch) break;
    T* st = static_cast<T*>(p.state) + (b0 + r) * (K - 1) * p.dim + d0;
    float f[K - 1][VEC], cur[VEC], pre[VEC];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      widen<VEC>(win[r][k], f[k]);
      raw_store<T, VEC>(st + k * p.dim, win[r][k + 1]);
    }
    widen<VEC>(win[r][K - 1], cur);
    taps<K, VEC>(w, bv, f, cur, pre);
    if (p.silu) apply_silu<VEC>(pre);
    store_f<T, VEC>(static_cast<T*>(p.y) + (b0 + r) * p.dim + d0, pre);
  }
}

bool fits(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename T, int K>
cudaError_t conv_fwd_k(const ConvParams& p, cudaStream_t s) {
  const ConvGrid g = conv_grid(p.batch, p.seqlen, p.dim, kFwdCtas, 2);
  conv_fwd_kernel<T, K><<<dim3(g.gx, g.gy), kConvThreads, 0, s>>>(p, g.tc, g.lx, g.chunks);
  return cudaGetLastError();
}

template <typename T, int K>
cudaError_t conv_bwd_k(const ConvBwdParams& q, int* parts, cudaStream_t s) {
  const ConvParams& p = q.fwd;
  const ConvGrid g = conv_grid(p.batch, p.seqlen, p.dim, kBwdCtas, 4);
  conv_bwd_kernel<T, K><<<dim3(g.gx, g.gy), kConvThreads, 0, s>>>(q, g.tc, g.lx, g.chunks);
  *parts = static_cast<int>(g.gy);
  return cudaGetLastError();
}

template <typename T, int K, int VEC, int R>
cudaError_t conv_step_r(const ConvStepParams& p, cudaStream_t s) {
  constexpr int64_t threads = 128;
  const int64_t cvs = p.dim / VEC, rows = (p.batch + R - 1) / R;
  const int64_t blocks = (rows * cvs + threads - 1) / threads;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  conv_step_kernel<T, K, VEC, R><<<static_cast<unsigned>(blocks), threads, 0, s>>>(p, cvs);
  return cudaGetLastError();
}

// Four rows share a thread's taps where that leaves every SM two CTAs' worth of
// threads: a thread's taps are 2.5 times the bytes of a bf16 row's state and x.
// Batch 1024 x 2048, width 4: bf16 6.7 us with four rows, 9.9 us with two, 13.2
// us with one; fp32 9.9, 9.5 and 11.0 us.
template <typename T, int K>
cudaError_t conv_step_k(const ConvStepParams& p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  constexpr int R = 4;
  const bool vec = p.dim % V == 0 && (p.x_batch * sizeof(T)) % 16 == 0 && fits(p.x, 16) &&
                   fits(p.y, 16) && fits(p.state, 16) && fits(p.weight, 16);
  if (!vec) return conv_step_r<T, K, 1, 1>(p, s);
  const bool many = p.batch * (p.dim / V) >= int64_t(kSms) * 256 * R;
  return many ? conv_step_r<T, K, V, R>(p, s) : conv_step_r<T, K, V, 1>(p, s);
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvParams& p, bool bf16, unsigned* err, cudaStream_t s) {
  if (conv_tma_ok(p, bf16)) return launch_conv_fwd_tma(p, bf16, err, s);
  switch (p.width) {
    case 2: return bf16 ? conv_fwd_k<__nv_bfloat16, 2>(p, s) : conv_fwd_k<float, 2>(p, s);
    case 3: return bf16 ? conv_fwd_k<__nv_bfloat16, 3>(p, s) : conv_fwd_k<float, 3>(p, s);
    case 4: return bf16 ? conv_fwd_k<__nv_bfloat16, 4>(p, s) : conv_fwd_k<float, 4>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

// The most partial sums any form of the backward writes.
int64_t conv_bwd_partials(int64_t batch, int64_t seqlen, int64_t dim, int width) {
  const int64_t a = conv_grid(batch, seqlen, dim, kBwdCtas, 4).gy;
  const int64_t b = conv_bwd_tma_partials(batch, seqlen, dim, width);
  return a > b ? a : b;
}

cudaError_t launch_conv_bwd(const ConvBwdParams& q, bool bf16, unsigned* err, cudaStream_t s) {
  const int width = q.fwd.width;
  int parts = 0;
  cudaError_t e = cudaErrorInvalidValue;
  if (conv_bwd_tma_ok(q, bf16)) {
    e = launch_conv_bwd_tma(q, bf16, err, &parts, s);
  } else {
    switch (width) {
      case 2: e = bf16 ? conv_bwd_k<__nv_bfloat16, 2>(q, &parts, s) : conv_bwd_k<float, 2>(q, &parts, s); break;
      case 3: e = bf16 ? conv_bwd_k<__nv_bfloat16, 3>(q, &parts, s) : conv_bwd_k<float, 3>(q, &parts, s); break;
      case 4: e = bf16 ? conv_bwd_k<__nv_bfloat16, 4>(q, &parts, s) : conv_bwd_k<float, 4>(q, &parts, s); break;
      default: break;
    }
  }
  if (e != cudaSuccess || parts == 1) return e;
  return launch_after(conv_bwd_sum_kernel,
                      dim3(static_cast<unsigned>((q.fwd.dim + 31) / 32), q.dbias ? width + 1 : width),
                      1024, 0, s, q.partial, q.dweight, q.dbias, q.fwd.dim, width, parts);
}

cudaError_t launch_conv_step(const ConvStepParams& p, bool bf16, cudaStream_t s) {
  switch (p.width) {
    case 2: return bf16 ? conv_step_k<__nv_bfloat16, 2>(p, s) : conv_step_k<float, 2>(p, s);
    case 3: return bf16 ? conv_step_k<__nv_bfloat16, 3>(p, s) : conv_step_k<float, 3>(p, s);
    case 4: return bf16 ? conv_step_k<__nv_bfloat16, 4>(p, s) : conv_step_k<float, 4>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ssm
