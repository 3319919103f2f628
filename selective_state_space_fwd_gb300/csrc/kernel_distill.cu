// kernel_distill.cu -- distillation from a teacher's top logits: per token the
// divergence of the student's softmax over the vocabulary, whose logits
// S = h W^T are never kept, from the teacher's over its few entries (i_k, z_k),
//   q = softmax_k(z / T),   p = softmax_v(S / T),
//   loss[t] = sum_k q_k (log q_k - log p[i_k]),
//   G[t,v] = dloss[t] / T (p[v] - sum_{k: i_k = v} q_k),   dh = G W,   dW = G^T h.
//
// The scheme and its products are the cross entropy's (kernel_xent.cu), with a list
// of entries in the place of one target.  A first kernel turns each token's entries
// into probabilities and sorts them by id, a warp per token; an epilogue's thread then
// finds the first entry of its tile by bisection, while the tile's products still
// run, and meets the others in the order of the columns: the forward keeps their
// logits, the backward takes their probabilities from G before it is rounded, so
// that p - q keeps its digits where the student has come close.  The rest of the
// loss is formed by the kernel that joins the tiles.
//
// Measured on GB300: values of 4096 tokens x 50257 x 1536, 64 entries, 385 us in a graph
// (1.64 PFLOP/s; the cross entropy of the same sizes 367), with gradients 8192 x 65536 x
// 2048, 32 entries, 5.13 ms (1.71 PFLOP/s), both at the power limit; 1000 tokens, half of
// them without entries, x 32001 x 768, 16 entries, 128 us: uneven last tiles and the
// ends of nine short launches.
#include "xent_core.cuh"

namespace ssm {
namespace {

constexpr int kPrepWarps = 4;
constexpr int64_t kNone = INT64_MIN;  // target of a token without entries

struct PrepArgs {
  const int64_t* ids;
  const void* logits;
  int top;
  int padded;       // the least power of two that holds them
  int64_t tokens, vocab, ignore;
  float inv_temp;
  uint2* entries;
  int64_t* targets;  // the likeliest entry's id; -1 if an id is outside the vocabulary
};

template <typename T>
__global__ void __launch_bounds__(kPrepWarps * 32) distill_prep_kernel(const PrepArgs p) {
  extern __shared__ uint2 prep_mem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kPrepWarps + warp;
  release_next();
  if (t >= p.tokens) return;
  uint2* list = prep_mem + warp * p.padded;
  float top = -INFINITY, best = 0.f;
  int at = INT32_MAX;  // the likeliest entry's place
  bool bad = false;
  for (int k = lane; k < p.padded; k += 32) {
    uint2 e = make_uint2(kNoEntry, 0);
    if (k < p.top) {
      const int64_t id = __ldg(p.ids + t * p.top + k);
      const float z = IO<T>::load(p.logits, t * p.top + k);
      if (id != p.ignore && z != -INFINITY) {
        const bool in = id >= 0 && id < p.vocab;
        bad |= !in;
        e = make_uint2(in ? static_cast<uint32_t>(id) : kNoEntry, __float_as_uint(z));
        top = fmaxf(top, z);
        if (at == INT32_MAX || z > best) {
          best = z;
          at = k;
        }
      }
    }
    list[k] = e;
  }
  bad = __any_sync(0xffffffffu, bad);
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float z = __shfl_xor_sync(0xffffffffu, best, o);
    const int k = __shfl_xor_sync(0xffffffffu, at, o);
    if (k != INT32_MAX && (at == INT32_MAX || z > best || (z == best && k < at))) {
      best = z;
      at = k;
    }
  }
  __syncwarp();
  if (lane == 0)
    p.targets[t] = at == INT32_MAX ? kNone : bad ? -1 : static_cast<int64_t>(list[at].x);
  __syncwarp();
  float sum = 0.f;
  for (int k = lane; k < p.top; k += 32) {
    if (list[k].x == kNoEntry) continue;
    const float e = expf((__uint_as_float(list[k].y) - top) * p.inv_temp);
    list[k].y = __float_as_uint(e);
    sum += e;
  }
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  for (int k = lane; k < p.top; k += 32)
    if (list[k].x != kNoEntry) list[k].y = __float_as_uint(__uint_as_float(list[k].y) / sum);
  __syncwarp();
  // by id: a bitonic network over the padded list
  for (int width = 2; width <= p.padded; width *= 2)
    for (int step = width / 2; step >= 1; step /= 2) {
      for (int i = lane; i < p.padded / 2; i += 32) {
        const int a = 2 * i - (i & (step - 1)), b = a + step;
        const uint2 x = list[a], y = list[b];
        const bool above = x.x > y.x || (x.x == y.x && x.y > y.y);
        if (above == ((a & width) == 0)) {
          list[a] = y;
          list[b] = x;
        }
      }
      __syncwarp();
    }
  uint2* out = p.entries + t * (p.top + kEntryPad);
  for (int k = lane; k < p.top + kEntryPad; k += 32)
    out[k] = k < p.top ? list[k] : make_uint2(kNoEntry, 0);
}

// Joins the tiles of a row, as the cross entropy does, and adds up its entries: a
// CTA takes 32 rows, first 32 lanes per tile of a row, then a warp per row.
__global__ void __launch_bounds__(1024) distill_join_kernel(const GemmArgs p, int tiles,
                                                            float* loss, float* lse) {
  __shared__ float2 red[32][33];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  wait_previous();
  const float unit = kLog2e * p.inv_temp;
  const int rows = rows_of(p);
  float m = -INFINITY, l = 0.f;
  if (r < rows) {
    const float2* q = p.part + r;
    for (int i = wy; i < tiles; i += 128) {
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = i + 32 * j < tiles ? q[(i + 32 * j) * p.part_pitch] : make_float2(-INFINITY, 0.f);
      join(m, l, v, unit);
    }
  }
  red[lane][wy] = make_float2(m, l);
  __syncthreads();
  const float2 v = red[wy][lane];
  m = v.x;
  l = v.y;
  join_lanes(m, l, unit);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + wy;
  if (row >= rows) return;
  const int64_t t = p.count ? p.idx[row] : row;
  const float s = logf(l);  // l >= 1: the maximum's own term
  // log p of an entry from its logit's difference to the maximum, which keeps its
  // digits where the logits are large
  const uint2* list = p.entries + t * (p.top + kEntryPad);
  float sum = 0.f;
  for (int k = lane; k < p.top; k += 32) {
    const uint2 e = __ldg(list + k);
    const float q = __uint_as_float(e.y);
    if (e.x == kNoEntry || q == 0.f) continue;
    sum += q * (logf(q) + (s + (m - p.entry_logit[t * p.top + k]) * p.inv_temp));
  }
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    const int64_t target = p.targets[t];
    lse[t] = target == kNone ? 0.f : fmaf(m, p.inv_temp, s);
    loss[t] = target == kNone ? 0.f : target < 0 ? NAN : sum;
  }
}

struct Extra {
  size_t entries, targets, logits, total;
};

// Behind the cross entropy's workspace.
Extra extra_of(const XentShape& z, const Layout& l, int top, bool backward) {
  Extra x;
  size_t off = l.total;
  const auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  x.entries = take(sizeof(uint2) * z.tokens * (top + kEntryPad));
  x.targets = take(8 * z.tokens);
  x.logits = backward ? 0 : take(sizeof(float) * z.tokens * top);
  x.total = off;
  return x;
}

// The tokens' entries, and the arguments that point at them.
cudaError_t prepare(const DistillParams& d, const Extra& x, char* ws, XentParams* p,
                    cudaStream_t s) {
  *p = d.xent;
  p->targets = reinterpret_cast<int64_t*>(ws + x.targets);
  p->ignore_index = kNone;
  PrepArgs a = {};
  a.ids = d.ids;
  a.logits = d.logits;
  a.top = d.top;
  a.padded = 1;
  while (a.padded < d.top) a.padded *= 2;
  a.tokens = p->shape.tokens;
  a.vocab = p->shape.vocab;
  a.ignore = d.ignore_index;
  a.inv_temp = 1.f / d.temperature;
  a.entries = reinterpret_cast<uint2*>(ws + x.entries);
  a.targets = reinterpret_cast<int64_t*>(ws + x.targets);
  const unsigned ctas = static_cast<unsigned>((a.tokens + kPrepWarps - 1) / kPrepWarps);
  const size_t smem = sizeof(uint2) * kPrepWarps * a.padded;
  if (d.logits_bf16)
    distill_prep_kernel<__nv_bfloat16><<<ctas, kPrepWarps * 32, smem, s>>>(a);
  else
    distill_prep_kernel<float><<<ctas, kPrepWarps * 32, smem, s>>>(a);
  return cudaGetLastError();
}

GemmArgs soft_args(const DistillParams& d, const XentParams& p, const Layout& l, const Extra& x,
                   const GatherArgs& g, char* ws) {
  GemmArgs a = gemm_args(p, l, ws);
  a.idx = g.idx;
  a.entries = reinterpret_cast<const uint2*>(ws + x.entries);
  a.top = d.top;
  a.inv_temp = 1.f / d.temperature;
  a.gain = 1.f / d.temperature;
  return a;
}

}  // namespace

size_t distill_workspace_bytes(const XentShape& s, int top, bool backward) {
  return extra_of(s, layout_of(s, backward), top, backward).total;
}

cudaError_t launch_distill_fwd(const DistillParams& d, cudaStream_t s) {
  const XentShape& z = d.xent.shape;
  const Layout l = layout_of(z, false);
  const Extra x = extra_of(z, l, d.top, false);
  char* ws = static_cast<char*>(d.xent.workspace);
  XentParams p;
  GatherArgs g;
  cudaError_t e = prepare(d, x, ws, &p, s);
  if (e != cudaSuccess) return e;
  g = gather_args(p, l, ws);
  g.loss = p.loss;
  g.lse_out = p.lse;
  GemmArgs a = soft_args(d, p, l, x, g, ws);
  a.v0 = 0;
  a.vp = static_cast<int>(z.vocab);
  a.part = reinterpret_cast<float2*>(ws + l.part);
  a.part_pitch = l.tpad;
  a.entry_logit = reinterpret_cast<float*>(ws + x.logits);
  Maps maps = {};
  if (!map_bf16_sw128(&maps.b, p.weight, z.dim, z.vocab, z.dim, kHalfTile) ||
      !map_bf16_sw128(&maps.h, p.h, z.dim, z.tokens, z.dim, kHalfTile) ||
      !map_bf16_sw128(&maps.a, g.rows, z.dim, l.tpad, z.dim, kHalfTile))
    return cudaErrorInvalidValue;
  // leaving tokens out saves nothing while all of them fit one row of tiles
  if (z.tokens <= kTile)
    a.count = nullptr;
  else if ((e = gather(g, true, s)) != cudaSuccess)
    return e;
  e = z.dim > kRange * kBk ? gemm<kRangeLse>(maps, a, s) : gemm<kSoftLse>(maps, a, s);
  if (e != cudaSuccess) return e;
  return launch_after(distill_join_kernel, static_cast<unsigned>((z.tokens + 31) / 32), 1024, 0, s,
                      a, ceil_div(z.vocab, kTile), p.loss, p.lse);
}

cudaError_t launch_distill_bwd(const DistillParams& d, cudaStream_t s) {
  const XentShape& z = d.xent.shape;
  const Layout l = layout_of(z, true);
  const Extra x = extra_of(z, l, d.top, true);
  char* ws = static_cast<char*>(d.xent.workspace);
  XentParams p;
  const cudaError_t e = prepare(d, x, ws, &p, s);
  if (e != cudaSuccess) return e;
  const GatherArgs g = gather_args(p, l, ws);
  return backward<kSoftGrad>(p, g, soft_args(d, p, l, x, g, ws), l, ws, s);
}

}  // namespace ssm
