// kernel_xent.cu -- softmax cross entropy over a large vocabulary, from the
// hidden states and the output embedding, without keeping the logits.
//
// With S = h W^T (tokens x vocabulary), per token t with target c:
//   lse[t]  = log sum_v exp(S[t,v]),   loss[t] = lse[t] - S[t,c]
//   G[t,v]  = dloss[t] (exp(S[t,v] - lse[t]) - [v = c])
//   dh = G W,   dW = G^T h.
// Tokens whose target is ignored take no part: the others' rows of h are
// gathered first, which also keeps whatever the ignored rows hold (NaN, say)
// out of dW.
//
// The forward multiplies tile by tile; a tile's epilogue reduces each row to
// the maximum and the sum of exponentials of its 256 columns (and picks the
// target's logit out), so that only a 64th of the logits' size is written; a
// second kernel joins the tiles of a row.  The backward forms G again in
// pieces of the vocabulary: one launch writes a piece of G (bf16; the products
// take bf16 operands), a second multiplies it with W into dh and with h into
// dW, both kinds of tile in one launch.  dh is summed over the pieces in fp32.
// 8 T V D operations with the gradients; the tensor cores bound it.
//
// Where all tokens have the same dloss (a mean), G is formed without it and the
// results are multiplied by it in fp32: rounded into G it would be off by up to
// 2^-8 in the same direction for every token, as p - 1 at the target is nearly
// -1.  What rounding takes from a token's G at the target is kept in fp32 and
// put back into its dh.  With a dloss per token dW keeps the rounding of G, which
// falls either way: 2.4e-3 off in all, against 1.7e-3 for its own rounding alone.
//
// Products: 256 x 256 tiles on pairs of CTAs (umma_pair.cuh), operands by TMA
// in 64-wide, 128-byte swizzled boxes through a ring of kStages stages, fp32
// accumulators in tensor memory, two of them so that the epilogue of a tile
// runs under the products of the next.  Per CTA: warp 0 copies, warp 1 (of the
// even CTA) issues products, warps 2 to 5 run the epilogue, a thread per row.
// Clusters are persistent and take tiles in turn.
//
// Measured on GB300: values of 4096 tokens x 50257 x 1536 in 350 to 379 us in a
// loop, 1.71 PFLOP/s, 326 in a short run; with gradients, 8192 x 65536 x 2048
// in 5.17 ms, 1.70 PFLOP/s (the power limit: a cuBLAS loop sustains 1.75), 1000
// tokens, half of them ignored, x 32001 x 768 in 112 us, 0.88 PFLOP/s (short
// launches: fill, drain and uneven last tiles).  Eight epilogue warps instead of four, and 4 or 5 stages instead
// of 6, measured no better on these.
#include "xent_core.cuh"

namespace ssm {
namespace {

// ---- few tokens ---------------------------------------------------------------
// With up to kFewMost tokens the forward only streams W: it is the A operand
// here (128 rows of the vocabulary per tile and CTA) and the tokens, padded to N
// rows, the B operand, so that nearly all bytes in flight are W's.  Thread r of
// the epilogue holds row r of a tile and keeps a running (maximum, sum) per
// token over the CTA's tiles; the threads' pairs are joined once, at the end.
// With a vocabulary of 32768 x 1024 (67 MB, 9.9 us of HBM): 1 token 19.8 us, 32
// tokens 20.8 us.  The 256 x 256 tiles take 25.8 us for 1 token, 20.4 us for 33 and
// 19.3 us for 64, which took 25.3 us here with N = 64.
constexpr int kFewMost = 32;

template <int N>
struct Few {
  static constexpr uint32_t kA = kHalfTile * kBk * 2, kB = N * kBk * 2, kStageF = kA + kB;
  static constexpr int kStagesF = 200 * 1024 / kStageF;
  static constexpr uint32_t kBarsF = kStagesF * kStageF;
  static constexpr uint32_t kSmemF = kBarsF + 512 + 1024;
  static constexpr uint32_t kCols = 2 * N < 32 ? 32 : 2 * N;  // two accumulators of N columns
  static_assert(kSmemF <= 227 * 1024 && kStageF % 1024 == 0 && 16 * kStagesF + 48 <= 512, "layout");
  static_assert(N * 128 * sizeof(float2) <= kBarsF, "the pairs fit the ring");
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
    xent_few_kernel(const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_h, const GemmArgs p) {
  using F = Few<N>;
  constexpr int S = F::kStagesF;
  extern __shared__ unsigned char sm_raw[];
  __shared__ int tgt_s[N];
  const uint32_t raw = umma::smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t bars = base + F::kBarsF;
  const auto full = [&](int s) { return bars + 8 * s; };
  const auto empty = [&](int s) { return bars + 8 * (S + s); };
  const auto acc_full = [&](int b) { return bars + 8 * (2 * S + b); };
  const auto acc_empty = [&](int b) { return bars + 8 * (2 * S + 2 + b); };
  const uint32_t slot = bars + 8 * (2 * S + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = ceil_div(p.vocab, kHalfTile), kt = ceil_div(p.dim, kBk);
  const int first = blockIdx.x, step = gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      umma::mbar_init(full(s), 1);
      umma::mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      umma::mbar_init(acc_full(b), 1);
      umma::mbar_init(acc_empty(b), kEpilogueWarps);
    }
  }
  if (warp == 1) umma::tmem_alloc(slot, F::kCols);
  wait_previous();
  release_next();
  if (threadIdx.x < N) tgt_s[threadIdx.x] = target_of(p, threadIdx.x);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  uint32_t tm;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tm) : "r"(slot) : "memory");

  bool bad = false;
  if (warp == 0 && lane == 0) {
    int s = 0, used = 0;
    uint32_t ph = 1;
    for (int t = first; t < tiles && !bad; t += step) {
      for (int k = 0; k < kt; ++k) {
        if (!pair::mbar_wait(empty(s), ph, kWaitNs)) {
          bad = true;
          break;
        }
        const uint32_t a = base + s * F::kStageF;
        umma::mbar_expect_tx(full(s), F::kStageF);
        umma::tma_load_2d(a, &map_w, k * kBk, t * kHalfTile, full(s));
        umma::tma_load_2d(a + F::kA, &map_h, k * kBk, 0, full(s));
        if (used < S) ++used;
        if (++s == S) { s = 0; ph ^= 1; }
      }
    }
    // every copy has landed, and been read, once its stage is free again
    for (int i = 0; i < used; ++i) {
      if (--s < 0) { s = S - 1; ph ^= 1; }
    }
    for (int i = 0; i < used; ++i) {
      if (!pair::mbar_wait(empty(s), ph ^ 1, kWaitNs)) {
        bad = true;
        break;
      }
      if (++s == S) { s = 0; ph ^= 1; }
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t id = umma::idesc_bf16(kHalfTile, N, false, false);
    int s = 0, n = 0;
    uint32_t ph = 0;
    for (int t = first; t < tiles && !bad; t += step, ++n) {
      const int b = n & 1;
      if (!pair::mbar_wait(acc_empty(b), ((n >> 1) & 1) ^ 1, kWaitNs)) {
        bad = true;
        break;
      }
      umma::fence_after_sync();
      for (int k = 0; k < kt; ++k) {
        if (!pair::mbar_wait(full(s), ph, kWaitNs)) {
          bad = true;
          break;
        }
        umma::fence_after_sync();
        const uint32_t a = base + s * F::kStageF;
#pragma unroll
        for (int j = 0; j < kBk / 16; ++j)
          umma::mma_bf16(tm + b * N, desc(a, j, false), desc(a + F::kA, j, false), id, k > 0 || j > 0);
        umma::mma_commit(empty(s));
        if (++s == S) { s = 0; ph ^= 1; }
      }
      if (!bad) umma::mma_commit(acc_full(b));
    }
  } else if (warp >= 2) {
    const int q = warp & 3, row = q * 32 + lane;
    float m[N], l[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.f;
    }
    int n = 0;
    for (int t = first; t < tiles && !bad; t += step, ++n) {
      const int b = n & 1;
      if (!pair::mbar_wait(acc_full(b), (n >> 1) & 1, kWaitNs)) bad = true;
      if (__any_sync(0xffffffffu, bad)) {
        bad = true;
        break;
      }
      umma::fence_after_sync();
      const int64_t v = static_cast<int64_t>(t) * kHalfTile + row;
      const bool in = v < p.vocab;
#pragma unroll
      for (int c = 0; c < N; c += 16) {
        uint32_t r[16];
        __syncwarp();
        tmem_ld16(tm + b * N + c + (static_cast<uint32_t>(q * 32) << 16), r);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = __uint_as_float(r[j]);
          if (in && tgt_s[c + j] == v) p.target_logit[c + j] = x;
          // one exponential: of the distance between the maximum so far and x
          const float d = x - m[c + j], e = ex2(-fabsf(d) * kLog2e);
          if (in && x != -INFINITY) {
            l[c + j] = d > 0.f ? fmaf(l[c + j], e, 1.f) : l[c + j] + e;
            m[c + j] = fmaxf(m[c + j], x);
          }
        }
      }
      umma::fence_before_sync();
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(acc_empty(b));
    }
    // the 128 threads' pairs, token by token, in the ring's memory: the last
    // accumulator was complete, so every operand has been read
    float2* pairs = reinterpret_cast<float2*>(sm_raw + (base - raw));
#pragma unroll
    for (int j = 0; j < N; ++j) pairs[j * 128 + row] = make_float2(m[j], l[j]);
    asm volatile("bar.sync 1, 128;" ::: "memory");
    for (int j = q; j < N; j += 4) {
      float a = -INFINITY, z = 0.f;
      float2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = pairs[j * 128 + i * 32 + lane];
      join(a, z, v);
      join_lanes(a, z);
      if (lane == 0) p.part[static_cast<int64_t>(blockIdx.x) * p.part_pitch + j] = make_float2(a, z);
    }
  }
  if (bad) atomicOr(p.err, kErrXentWait);
  __syncwarp();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == 1) umma::tmem_dealloc(tm, F::kCols);
}

// ---- joining the tiles of a row --------------------------------------------------
// A warp row per 32 tokens, 32 of them sharing the tiles.
__global__ void __launch_bounds__(1024) xent_join_kernel(const GemmArgs p, int64_t ignore,
                                                         const int* idx, int tiles, float* loss,
                                                         float* lse) {
  __shared__ float2 red[32][33];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  wait_previous();
  const bool on = r < rows_of(p);
  float m = -INFINITY, l = 0.f;
  if (on) {
    const float2* q = p.part + r;
    for (int i = wy; i < tiles; i += 128) {
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = i + 32 * j < tiles ? q[(i + 32 * j) * p.part_pitch] : make_float2(-INFINITY, 0.f);
      join(m, l, v);
    }
  }
  red[lane][wy] = make_float2(m, l);
  __syncthreads();
  // warp wy joins token wy's 32 pairs
  const float2 v = red[wy][lane];
  m = v.x;
  l = v.y;
  join_lanes(m, l);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + wy;
  if (lane == 0 && row < rows_of(p)) {
    const int64_t t = idx ? idx[row] : row;
    const bool none = !p.count && p.targets[t] == ignore;
    const float s = logf(l);  // l >= 1: the maximum's own term
    lse[t] = none ? 0.f : m + s;
    // of the difference to the maximum: a certain token's loss, far below an ulp of
    // lse, keeps its digits and is never negative
    loss[t] = none ? 0.f : target_of(p, row) >= 0 ? s + (m - p.target_logit[row]) : NAN;
  }
}

template <int N>
cudaError_t few(const XentShape& z, const void* h, const CUtensorMap& map_w, const GemmArgs& a,
                int ctas, cudaStream_t s) {
  CUtensorMap map_h;
  if (!map_bf16_sw128(&map_h, h, z.dim, z.tokens, z.dim, N)) return cudaErrorInvalidValue;
  auto* k = xent_few_kernel<N>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(Few<N>::kSmemF));
  if (e != cudaSuccess) return e;
  return launch_after(k, ctas, kThreads, Few<N>::kSmemF, s, map_w, map_h, a);
}

}  // namespace

size_t xent_workspace_bytes(const XentShape& s, bool backward) { return layout_of(s, backward).total; }

cudaError_t launch_xent_fwd(const XentParams& p, cudaStream_t s) {
  const XentShape& z = p.shape;
  const Layout l = layout_of(z, false);
  char* ws = static_cast<char*>(p.workspace);
  GemmArgs a = gemm_args(p, l, ws);
  a.v0 = 0;
  a.vp = static_cast<int>(z.vocab);
  a.part = reinterpret_cast<float2*>(ws + l.part);
  a.part_pitch = l.tpad;
  a.target_logit = reinterpret_cast<float*>(ws + l.target_logit);
  GatherArgs g = gather_args(p, l, ws);
  g.loss = p.loss;
  g.lse_out = p.lse;
  Maps maps = {};
  if (!map_bf16_sw128(&maps.b, p.weight, z.dim, z.vocab, z.dim, kHalfTile))
    return cudaErrorInvalidValue;
  cudaError_t e;
  int parts = ceil_div(z.vocab, kTile);
  // leaving ignored tokens out saves nothing while all of them fit one row of tiles
  const bool direct = z.tokens <= kTile;
  if (direct) a.count = nullptr;
  if (z.tokens <= kFewMost) {
    parts = ceil_div(z.vocab, kHalfTile);
    parts = parts < kSms ? parts : kSms;
    e = z.tokens <= 16 ? few<16>(z, p.h, maps.b, a, parts, s)
                       : few<32>(z, p.h, maps.b, a, parts, s);
  } else {
    if (!map_bf16_sw128(&maps.h, p.h, z.dim, z.tokens, z.dim, kHalfTile))
      return cudaErrorInvalidValue;
    if (!direct) {
      if (!map_bf16_sw128(&maps.a, g.rows, z.dim, l.tpad, z.dim, kHalfTile))
        return cudaErrorInvalidValue;
      if ((e = gather(g, false, s)) != cudaSuccess) return e;
    }
    e = gemm<kLse>(maps, a, s);
  }
  if (e != cudaSuccess) return e;
  return launch_after(xent_join_kernel, static_cast<unsigned>((z.tokens + 31) / 32), 1024, 0, s, a,
                      p.ignore_index, direct ? nullptr : g.idx, parts, p.loss, p.lse);
}

cudaError_t launch_xent_bwd(const XentParams& p, cudaStream_t s) {
  const Layout l = layout_of(p.shape, true);
  char* ws = static_cast<char*>(p.workspace);
  return backward<kGrad>(p, gather_args(p, l, ws), gemm_args(p, l, ws), l, ws, s);
}

}  // namespace ssm
