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
// `tpr` threads, NV groups of VEC elements each.  The backward
// keeps CTAs resident and walks rows, so that every thread sums dw and db of
// its own columns in registers; the CTAs' sums are written once and added by a
// second kernel in a fixed order (no atomics).
#include <type_traits>

#include "common.cuh"
#include "layers.h"
#include "pdl.cuh"
#include "vec.cuh"

namespace ssm {
namespace {

constexpr int kSms = 152;
constexpr int kBwdPer = 8;  // backward: elements of a row per thread, up to 512 threads
// Backward: CTAs of up to `threads` that the registers of an SM are shared out
// for: 20 warps, and 24 where small CTAs hold their operands in 16 bits (`narrow`).
// Training steps of 1024 bf16 columns 100 us with 24 warps, 103 us with 20; of
// 1536 with an fp32 stream 428 and 413 us.
__host__ __device__ constexpr int bwd_ctas_per_sm(int threads, bool narrow) {
  return (narrow && threads <= 192 ? 24 : 20) * 32 / threads;
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
  const int first = warp / wpr * wpr;
  float a = 0.f;
  for (int i = 0; i < wpr; ++i) a += red[first + i];
  return a;
}

// A thread's columns: NV groups of VEC, group i from column (i tpr + lane) VEC.
// Rows whose length is not a multiple of VEC start off the access boundary; with
// SHIFT their groups start `shift` columns earlier, on it, and reach into the
// rows before and after, whose elements are read (but past the tensor's end) and
// dropped.  shift = row dim mod VEC, as tensors start on a boundary.
template <int VEC, bool SHIFT>
struct Cols {
  int dim, shift;
  bool last;  // the tensor ends within a group of the row's end: nothing is read past it
  __device__ __forceinline__ Cols(int dim_, int64_t row, int64_t rows) : dim(dim_), shift(0) {
    if (SHIFT) shift = static_cast<int>(row % VEC) * (dim % VEC) % VEC;
    set_row(row, rows);
  }
  // Another row of the same shift.
  __device__ __forceinline__ void set_row(int64_t row, int64_t rows) {
    last = SHIFT && (rows - 1 - row) * dim < VEC;
  }
  __device__ __forceinline__ int at(int group) const { return group * VEC - shift; }
  __device__ __forceinline__ bool whole(int c) const {
    return SHIFT ? c >= 0 && c + VEC <= dim : c < dim;
  }
  // f(v, whether column c + v is the row's), for the elements of a group: by
  // selects on the group, or (BRANCH, and with a shift) without any in the groups
  // inside the row.
  template <bool BRANCH = SHIFT, typename F>
  __device__ __forceinline__ void each(int c, F&& f) const {
    if constexpr (!BRANCH) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) f(v, c < dim);
    } else if (whole(c)) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) f(v, std::true_type());
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) f(v, SHIFT && c + v >= 0 && c + v < dim);
    }
  }
  // Loads of groups past the row's end are made at its last group instead, and
  // their values dropped, so that no load waits on a branch.
  template <typename T, bool RW = false>
  __device__ __forceinline__ Raw<T, VEC> load(const T* row, int c) const {
    const int end = SHIFT ? (dim + shift - 1) / VEC * VEC - shift : dim - VEC;
    c = c < dim ? c : end;
    if constexpr (SHIFT) {
      if (last && c + VEC > dim) {
        Raw<T, VEC> r;
        float f[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) f[v] = c + v < dim ? static_cast<float>(row[c + v]) : 0.f;
        narrow<VEC>(f, r);
        return r;
      }
    }
    if constexpr (RW) return raw_load_rw<T, VEC>(row + c);
    else return raw_load<T, VEC>(row + c);
  }
  // The weight's (or bias's) values of a group; they start on a boundary only
  // without a shift.
  __device__ __forceinline__ void load_w(const float* w, int c, float (&f)[VEC]) const {
    if constexpr (SHIFT) {
      each(c, [&](int v, auto in) { f[v] = in ? __ldg(w + (c + v)) : 0.f; });
    } else {
      load_f<float, VEC>(w + (c < dim ? c : dim - VEC), f);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int c, const float (&f)[VEC]) const {
    if (whole(c)) {
      store_f<T, VEC>(row + c, f);
    } else if constexpr (SHIFT) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float one[1] = {f[v]};
        if (c + v >= 0 && c + v < dim) store_f<T, 1>(row + c + v, one);
      }
    }
  }
};

template <typename TX, typename TR, int VEC, int NV, bool SHIFT>
__global__ void __launch_bounds__(VEC * NV == 8 ? 1024 : 512)
    norm_fwd_kernel(const NormParams p, int tpr) {
  __shared__ float red[2][32];
  const int group = threadIdx.x / tpr, lane = threadIdx.x - group * tpr;
  int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + group;
  const bool on = row < p.rows;
  row = on ? row : p.rows - 1;  // groups without a row write nothing
  const int dim = static_cast<int>(p.dim);
  const int64_t at = row * p.dim;
  const Cols<VEC, SHIFT> cols(dim, row, p.rows);
  const TX* x = static_cast<const TX*>(p.x) + at;
  float f[NV][VEC];
  Raw<TX, VEC> xr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) xr[i] = cols.load(x, cols.at(i * tpr + lane));
  if (p.residual) {
    const TR* res = static_cast<const TR*>(p.residual) + at;
    TR* out = static_cast<TR*>(p.r) + at;
    Raw<TR, VEC> rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      rr[i] = cols.template load<TR, true>(res, cols.at(i * tpr + lane));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[VEC];
      widen<VEC>(xr[i], f[i]);
      widen<VEC>(rr[i], g);
#pragma unroll
      for (int v = 0; v < VEC; ++v) f[i][v] += g[v];
      Raw<TR, VEC> o;
      narrow<VEC>(f[i], o);
      widen<VEC>(o, f[i]);  // as stored
      if (on) cols.store(out, cols.at(i * tpr + lane), f[i]);
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
      const int c = cols.at(i * tpr + lane);
      cols.each(c, [&](int v, auto in) { a += in ? f[i][v] : 0.f; });
    }
    mean = row_sum(a, tpr, red[0]) * inv;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = cols.at(i * tpr + lane);
    if constexpr (SHIFT) {
      cols.each(c, [&](int v, auto in) {
        f[i][v] -= mean;
        const float own = in ? f[i][v] : 0.f;  // what is dropped may be another row's NaN
        q = fmaf(own, own, q);
      });
    } else {  // a group is the row's, or dropped, as a whole
      float s = q;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        f[i][v] -= mean;
        s = fmaf(f[i][v], f[i][v], s);
      }
      q = c < dim ? s : q;
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
    cols.load_w(p.weight, cols.at(i * tpr + lane), w);
#pragma unroll
    for (int v = 0; v < VEC; ++v) f[i][v] *= rstd * w[v];
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float b[VEC];
      cols.load_w(p.bias, cols.at(i * tpr + lane), b);
#pragma unroll
      for (int v = 0; v < VEC; ++v) f[i][v] += b[v];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) cols.store(y, cols.at(i * tpr + lane), f[i]);
}

// A row's operands of one thread, as loaded.
template <typename TX, typename TR, int VEC, int NV>
struct RowRaw {
  Raw<TR, VEC> r[NV], dr[NV];
  Raw<TX, VEC> dy[NV];
  float mean, rstd;
};

// The loads of the next row are in flight while a row is reduced and written.
// With SHIFT a group of threads takes rows of one shift only (the launch makes
// the rows' stride a multiple of VEC), so that its columns stay its own.
template <typename TX, typename TR, int VEC, int NV, int THREADS, bool SHIFT>
__global__ void __launch_bounds__(THREADS, bwd_ctas_per_sm(THREADS, sizeof(TR) == 2))
    norm_bwd_kernel(const NormBwdParams p, int tpr) {
  __shared__ float2 red[2][32];
  __shared__ float acc[THREADS * VEC * NV];
  const int wpr = tpr >> 5, groups = blockDim.x / tpr;
  const int group = threadIdx.x / tpr, lane = threadIdx.x - group * tpr;
  const int dim = static_cast<int>(p.dim);
  const float inv = 1.f / static_cast<float>(dim);
  const bool has_dr = p.dr != nullptr;
  constexpr bool kHoldW = NV * VEC == kBwdPer;  // wider rows read the weight again per row
  float w[kHoldW ? NV : 1][VEC], dw[NV][VEC], db[NV][VEC];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups + group;
  const Cols<VEC, SHIFT> own(dim, row0, p.rows);  // the shift of the group's rows
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (kHoldW) own.load_w(p.weight, own.at(i * tpr + lane), w[i]);
#pragma unroll
    for (int v = 0; v < VEC; ++v) dw[i][v] = db[i][v] = 0.f;
  }
  release_next();
  const auto load = [&](RowRaw<TX, TR, VEC, NV>& x, int64_t row) {
    if (row >= p.rows) return;
    const int64_t at = row * p.dim;
    Cols<VEC, SHIFT> cols = own;
    cols.set_row(row, p.rows);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = cols.at(i * tpr + lane);
      x.r[i] = cols.load(static_cast<const TR*>(p.r) + at, c);
      x.dy[i] = cols.load(static_cast<const TX*>(p.dy) + at, c);
    }
    if (has_dr) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        x.dr[i] = cols.load(static_cast<const TR*>(p.dr) + at, cols.at(i * tpr + lane));
    }
    x.mean = p.rms ? 0.f : __ldg(p.stats + row);
    x.rstd = __ldg(p.stats + p.rows + row);
  };
  int buf = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  RowRaw<TX, TR, VEC, NV> next = {};
  load(next, row0);
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
      const int c = own.at(i * tpr + lane);
      widen<VEC>(next.r[i], xh[i]);
      widen<VEC>(next.dy[i], g[i]);
      er[i] = next.dr[i];
      float wi[VEC];
      if constexpr (kHoldW) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) wi[v] = w[i][v];
      } else {
        own.load_w(p.weight, c, wi);
      }
      constexpr bool kBranch = SHIFT || !kHoldW;  // fewer registers live at once
      if (!kBranch || on) {
        own.template each<kBranch>(c, [&](int v, auto here) {
          const bool in = here && (kBranch || on);
          xh[i][v] = in ? (xh[i][v] - mean) * rstd : 0.f;
          g[i][v] = in ? g[i][v] : 0.f;
          db[i][v] += g[i][v];
          dw[i][v] = fmaf(g[i][v], xh[i][v], dw[i][v]);
          g[i][v] *= wi[v];
          a.x += g[i][v];
          a.y = fmaf(g[i][v], xh[i][v], a.y);
        });
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
      const int first = group * wpr;
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
      const int c = own.at(i * tpr + lane);
      float o[VEC], e[VEC];
      widen<VEC>(er[i], e);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        o[v] = rstd * (g[i][v] - mg - xh[i][v] * mx);
        o[v] = has_dr ? o[v] + e[v] : o[v];
      }
      if (on) {
        own.store(static_cast<TX*>(p.dx) + at, c, o);
        if (p.dresidual) own.store(static_cast<TR*>(p.dresidual) + at, c, o);
      }
    }
  }
  // the row groups' sums, added in the order of the groups
  const int span = tpr * VEC * NV;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        acc[group * span + (i * tpr + lane) * VEC + v] = k == 0 ? dw[i][v] : db[i][v];
    __syncthreads();
    for (int c = threadIdx.x; c < dim; c += blockDim.x) {
      float s = 0.f;
      for (int u = 0; u < groups; ++u) {
        const Cols<VEC, SHIFT> theirs(dim, row0 - group + u, p.rows);
        s += acc[u * span + c + theirs.shift];
      }
      if (gridDim.x > 1)
        p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + k) * p.dim + c] = s;
      else if (k == 0)  // the only CTA: its sums are the result
        p.dweight[c] = s;
      else if (p.dbias)
        p.dbias[c] = s;
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

// Threads per row: at most `per` elements of the row per thread.  Parts of a warp
// and pairs of warps share CTAs of 128 threads; wider rows take a CTA of their
// own of as many warps as they need.
int threads_per_row(int64_t dim, int per) {
  int t = 8;
  while (int64_t(t) * per < dim && t < 64) t *= 2;
  if (int64_t(t) * per < dim) t = static_cast<int>((dim + 32 * per - 1) / (32 * per)) * 32;
  return t;
}
int cta_threads(int tpr) { return tpr > 64 ? tpr : 128; }

// Columns that a row's groups span.
int64_t span_of(int64_t dim, int vec, bool shift) { return shift ? dim + vec - 1 : dim; }

// Rows are held 8 elements per thread where there are few of them (a row's
// latency counts), else 16 (fewer threads to synchronise per row).
template <typename TX, typename TR, int VEC, bool SHIFT>
cudaError_t norm_fwd_v(const NormParams& p, cudaStream_t s) {
  const int per = p.rows < 4 * kSms ? 8 : 16;
  const int tpr = threads_per_row(span_of(p.dim, VEC, SHIFT), per);
  const int threads = cta_threads(tpr);
  const int64_t rpb = threads / tpr, blocks = (p.rows + rpb - 1) / rpb;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(blocks);
  if (per == 8)
    norm_fwd_kernel<TX, TR, VEC, 8 / VEC, SHIFT><<<g, threads, 0, s>>>(p, tpr);
  else
    norm_fwd_kernel<TX, TR, VEC, 16 / VEC, SHIFT><<<g, threads, 0, s>>>(p, tpr);
  return cudaGetLastError();
}

// How a call's rows are accessed: in whole groups, in shifted groups (rows that
// do not start on a boundary, tensors that do), or element by element.
enum class Access { kWhole, kShift, kSingle };
Access access_of(int64_t dim, int vec, bool aligned) {
  if (!aligned) return Access::kSingle;
  if (dim % vec == 0) return Access::kWhole;
  return span_of(dim, vec, true) <= kNormMaxDim ? Access::kShift : Access::kSingle;
}

template <typename TX, typename TR>
cudaError_t norm_fwd_t(const NormParams& p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(TX);
  const bool aligned = fits(p.x, 16) && fits(p.y, 16) && fits(p.residual, 16) && fits(p.r, 16) &&
                       fits(p.weight, 16) && fits(p.bias, 16);
  switch (access_of(p.dim, V, aligned)) {
    case Access::kWhole: return norm_fwd_v<TX, TR, V, false>(p, s);
    case Access::kShift: return norm_fwd_v<TX, TR, V, true>(p, s);
    default: return norm_fwd_v<TX, TR, 1, false>(p, s);
  }
}

// The backward's rows: kBwdPer elements per thread up to 512 threads, else twice
// as many.
int bwd_threads(int64_t span) {
  return threads_per_row(span, span <= kBwdPer * 512 ? kBwdPer : 2 * kBwdPer);
}

// The bound on a CTA's threads that its kernel is compiled for.
int bwd_bound(int64_t span, int tpr) {
  if (span > kBwdPer * 512) return 512;
  for (int t : {128, 192, 256, 320})
    if (cta_threads(tpr) <= t) return t;
  return 512;
}

int64_t bwd_ctas(int64_t rows, int64_t span, bool narrow) {
  const int tpr = bwd_threads(span);
  const int64_t groups = cta_threads(tpr) / tpr, need = (rows + groups - 1) / groups;
  if (need <= 4) return 1;  // a few rows in turn cost less than a second kernel for the sums
  const int64_t most = int64_t(kSms) * bwd_ctas_per_sm(bwd_bound(span, tpr), narrow);
  return need < most ? need : most;
}

template <typename TX, typename TR, int VEC, bool SHIFT>
cudaError_t norm_bwd_v(const NormBwdParams& p, cudaStream_t s) {
  constexpr int NV = kBwdPer / VEC;
  const int64_t span = span_of(p.dim, VEC, SHIFT);
  const int tpr = bwd_threads(span), threads = cta_threads(tpr);
  unsigned g = static_cast<unsigned>(bwd_ctas(p.rows, span, sizeof(TR) == 2));
  if (SHIFT) g = (g + VEC - 1) / VEC * VEC;  // the rows' stride a multiple of VEC
  if (span > kBwdPer * 512) {
    norm_bwd_kernel<TX, TR, VEC, 2 * NV, 512, SHIFT><<<g, threads, 0, s>>>(p, tpr);
  } else {
    switch (bwd_bound(span, tpr)) {
      case 128: norm_bwd_kernel<TX, TR, VEC, NV, 128, SHIFT><<<g, threads, 0, s>>>(p, tpr); break;
      case 192: norm_bwd_kernel<TX, TR, VEC, NV, 192, SHIFT><<<g, threads, 0, s>>>(p, tpr); break;
      case 256: norm_bwd_kernel<TX, TR, VEC, NV, 256, SHIFT><<<g, threads, 0, s>>>(p, tpr); break;
      case 320: norm_bwd_kernel<TX, TR, VEC, NV, 320, SHIFT><<<g, threads, 0, s>>>(p, tpr); break;
      default: norm_bwd_kernel<TX, TR, VEC, NV, 512, SHIFT><<<g, threads, 0, s>>>(p, tpr);
    }
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || g == 1) return e;
  return launch_after(norm_bwd_sum_kernel,
                      dim3(static_cast<unsigned>((p.dim + 31) / 32), p.dbias ? 2 : 1), 1024, 0, s,
                      p.partial, p.dweight, p.dbias, p.dim, static_cast<int>(g));
}

template <typename TX, typename TR>
cudaError_t norm_bwd_t(const NormBwdParams& p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(TX);
  const bool aligned = fits(p.r, 16) && fits(p.dy, 16) && fits(p.dr, 16) && fits(p.dx, 16) &&
                       fits(p.dresidual, 16) && fits(p.weight, 16);
  switch (access_of(p.dim, V, aligned)) {
    case Access::kWhole: return norm_bwd_v<TX, TR, V, false>(p, s);
    case Access::kShift: return norm_bwd_v<TX, TR, V, true>(p, s);
    default: return norm_bwd_v<TX, TR, 1, false>(p, s);
  }
}

}  // namespace

cudaError_t launch_norm_fwd(const NormParams& p, bool bf16, bool residual_bf16, cudaStream_t s) {
  if (p.dim > kNormMaxDim) return cudaErrorInvalidValue;
  if (!bf16) return norm_fwd_t<float, float>(p, s);
  return residual_bf16 ? norm_fwd_t<__nv_bfloat16, __nv_bfloat16>(p, s)
                       : norm_fwd_t<__nv_bfloat16, float>(p, s);
}

// The most CTAs any form of the backward launches.
int64_t norm_bwd_partials(int64_t rows, int64_t dim) {
  int64_t most = bwd_ctas(rows, dim, true);
  for (int vec : {4, 8}) {
    if (dim % vec == 0) continue;
    const int64_t n = (bwd_ctas(rows, span_of(dim, vec, true), true) + vec - 1) / vec * vec;
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, bool bf16, bool residual_bf16,
                            cudaStream_t s) {
  if (p.dim > kNormMaxDim) return cudaErrorInvalidValue;
  if (!bf16) return norm_bwd_t<float, float>(p, s);
  return residual_bf16 ? norm_bwd_t<__nv_bfloat16, __nv_bfloat16>(p, s)
                       : norm_bwd_t<__nv_bfloat16, float>(p, s);
}

}  // namespace ssm
