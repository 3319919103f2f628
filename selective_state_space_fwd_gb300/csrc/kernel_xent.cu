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
#include <cuda.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "layers.h"
#include "pdl.cuh"
#include "ssd.h"
#include "tma_map.h"
#include "umma_pair.cuh"

namespace ssm {
namespace {

constexpr int kSms = 152;
constexpr int kClusters = kSms / 2;
constexpr int kTile = 256;               // rows and columns of a tile of the pair
constexpr int kHalfTile = 128;           // rows of A, and of B, that a CTA holds
constexpr int kBk = 64;                  // K per stage
constexpr int kStages = 6;
constexpr uint32_t kOperand = kHalfTile * kBk * 2;  // 16 KB: a CTA's A or B of a stage
constexpr uint32_t kStage = 2 * kOperand;
constexpr uint32_t kBox = 32 * 128;      // 4 KB: a warp's 32 rows of 128 bytes on their way out
constexpr uint32_t kOut = kStages * kStage;  // two boxes per epilogue warp
constexpr uint32_t kBars = kOut + 4 * 2 * kBox;
constexpr uint32_t kSmem = kBars + 256 + 1024;  // ring, boxes, barriers, alignment slack
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
constexpr int kThreads = 192;
constexpr int kEpilogueWarps = 4;
constexpr uint64_t kWaitNs = 2000000000ull;  // a wait gives up after 2 s
// Most bytes of one piece of G, which has at least one tile of columns (from 2^20
// tokens on the larger).
constexpr int64_t kPieceBytes = int64_t(512) << 20;

// The dloss that all kept tokens share, or 1 with `shared` 0.
struct Common {
  int shared;
  float dloss;
};

enum Mode { kLse = 0, kGrad = 1, kProducts = 2 };

struct GemmArgs {
  const int* count;       // rows kept; null: every token is a row
  const Common* common;   // the tokens' dloss, if it is one
  const int* target;      // [rows] column of the target, -1 for none
  const int64_t* targets;  // the tokens' targets, used without `count`
  int64_t tokens;
  const float* lse;       // [rows], kGrad
  const float* scale;     // [rows] dloss, kGrad
  float* lost;            // [rows] what rounding took from G at the target (kGrad writes it)
  const __nv_bfloat16* weight;  // [vocab][dim]
  int64_t vocab, dim;
  int64_t v0;             // first column of the piece
  int vp;                 // columns of the piece
  int kv_whole;           // kProducts: stages of a whole piece's columns
  float2* part;           // kLse: [tiles of columns][part_pitch] maximum, sum of exp(logit - maximum)
  int64_t part_pitch;
  float* target_logit;    // kLse: [rows]
  float* dh;              // kProducts: [splits][rows, whole tiles][dim] partial sums
  bool add;               // kProducts: add to dh (a later piece) rather than store
  unsigned* err;
};

// Operand maps: kLse and kGrad use a = the gathered rows of h and b = W in boxes
// of 128 rows; kProducts uses a = G (128-row boxes) and b = W (64-row boxes) for
// dh, at = G and bt = the rows of h (64-row boxes) for dW.  h is the same as
// the rows' map, over h itself: with no token ignored nothing is gathered.
// Results leave in boxes of 32 rows: g = the piece of G (kGrad), dw and dh
// (kProducts).
struct Maps {
  CUtensorMap a, b, at, bt, h, g, dw, dh;
};

// Whether the products read h itself: no token is ignored, and there is a whole
// tile of them.
__device__ __forceinline__ bool rows_in_place(int64_t rows, int64_t tokens) {
  return rows == tokens && tokens >= kTile;
}
__device__ __forceinline__ int rows_of(const GemmArgs& p) {
  return p.count ? *p.count : static_cast<int>(p.tokens);
}
__device__ __forceinline__ int target_of(const GemmArgs& p, int64_t row) {
  if (p.count) return p.target[row];
  if (row >= p.tokens) return -1;
  const int64_t t = p.targets[row];
  return t >= 0 && t < p.vocab ? static_cast<int>(t) : -1;
}

__host__ __device__ inline int ceil_div(int64_t a, int64_t b) {
  return static_cast<int>((a + b - 1) / b);
}

// The dh tiles' reduction over the vocabulary is split into ranges where there
// are fewer tiles than clusters.  Every piece takes the split of a whole one
// (kv stages), so that all pieces add into the same partial sums.
__host__ __device__ inline int dh_splits(int mt, int nt, int kv) {
  const int tiles = mt * nt > 0 ? mt * nt : 1;
  int s = kClusters / tiles;
  if (s < 1) s = 1;
  return s < kv ? s : kv;
}

// One tile of work: its position, its range of K in stages and its kind.
struct Unit {
  int m, n, k0, k1, split;
  bool dw;
};

// The units of one cluster, in order: its dh tiles, then its dW tiles.  Tiles are
// dealt out in turn; where the dh tiles do not come out even, the clusters with
// one fewer take the dW tiles that make up for it first.
template <int MODE>
struct Work {
  int rows, mt, nt, vt, kv, kt, splits;
  int ndh, ndw;              // units of either kind (kLse and kGrad: all are "dh")
  int cluster, clusters;
  int heavy, light, ahead;   // clusters with a dh unit more, without, dW units these take first
  __device__ Work(const GemmArgs& p, int c, int n) : cluster(c), clusters(n) {
    rows = rows_of(p);
    mt = ceil_div(rows, kTile);
    vt = ceil_div(p.vp, kTile);
    nt = MODE == kProducts ? ceil_div(p.dim, kTile) : vt;
    kv = ceil_div(p.vp, kBk);
    kt = MODE == kProducts ? ceil_div(rows, kBk) : ceil_div(p.dim, kBk);
    splits = MODE == kProducts ? dh_splits(mt, nt, p.kv_whole) : 1;
    ndh = mt * nt * splits;
    ndw = MODE == kProducts ? vt * nt : 0;
    heavy = ndh % clusters;
    light = clusters - heavy;
    ahead = 0;
    if (MODE == kProducts && heavy > 0 && kt > 0) {
      ahead = kv / splits / kt;
      if (ahead > ndw / light) ahead = ndw / light;
    }
  }
  // The cluster's i-th unit; false past its last.
  __device__ bool at(int i, Unit* r) const {
    const int u = cluster + i * clusters;
    if (u < ndh) {
      r->split = 0; r->dw = false; r->k0 = 0; r->k1 = kt;
      if (MODE != kProducts) {
        r->m = u % mt; r->n = u / mt;
        return true;
      }
      const int q = u / nt;
      r->n = u % nt; r->m = q % mt; r->split = q / mt;
      r->k0 = static_cast<int>(static_cast<int64_t>(kv) * r->split / splits);
      r->k1 = static_cast<int>(static_cast<int64_t>(kv) * (r->split + 1) / splits);
      return true;
    }
    if (MODE != kProducts) return false;
    int j = i - (ndh / clusters + (cluster < heavy ? 1 : 0)), w;
    if (cluster >= heavy && j < ahead) {
      w = cluster - heavy + j * light;
    } else {
      if (cluster >= heavy) j -= ahead;
      w = ahead * light + cluster + j * clusters;
    }
    if (w >= ndw) return false;
    r->n = w % nt; r->m = w / nt; r->split = 0; r->dw = true; r->k0 = 0; r->k1 = kt;
    return true;
  }
};

// K-major operand of 128 rows: K step j (16 elements) is 32 bytes further in
// the 128-byte rows; 8-row groups 1024 bytes apart.  MN-major operand in two
// boxes of 64 x 64: K step j is 16 rows further; the boxes are 8192 bytes
// apart, 8-row groups 1024.
__device__ __forceinline__ uint64_t desc(uint32_t tile, int j, bool mn) {
  const uint64_t sw128 = uint64_t(2) << 61;
  return sw128 | (mn ? umma::smem_desc(tile + j * 2048, 8192, 1024)
                     : umma::smem_desc(tile + j * 32, 16, 1024));
}

// A box of 32 rows x 128 bytes in shared memory, a row per lane, leaves by one
// copy (or one elementwise addition) of the warp.  Two boxes alternate: a box is
// written again once the copy before the last has read it.
struct OutBox {
  uint32_t base;
  int n;
  __device__ __forceinline__ void open() {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
  }
  __device__ __forceinline__ void put(int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const int lane = threadIdx.x & 31;
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                     base + (n & 1) * kBox + lane * 128 + ((chunk ^ (lane & 7)) << 4)),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
  }
  __device__ __forceinline__ void send(const CUtensorMap* map, int x, int y, bool add) {
    umma::fence_smem_to_async();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      const uint32_t box = base + (n & 1) * kBox;
      if (add)
        asm volatile(
            "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];"
            ::"l"(map), "r"(x), "r"(y), "r"(box)
            : "memory");
      else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                     ::"l"(map), "r"(x), "r"(y), "r"(box)
                     : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    ++n;
  }
  __device__ __forceinline__ void drain() {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Softmax statistics are kept in the logits' own units, so that a maximum is a
// logit, not the rounding of one, and exp(v - max) is taken of the rounded
// difference: never above 1, and 0 for a logit that a mask has put far below the
// others, or at -infinity.  (exp2(v log2(e) - max') with a fused product and a
// rounded max' is infinite where max' is off by more than 128: for logits past
// 10^9.)

// What exponents are taken from: the maximum, or 0 while all there is is
// -infinity, whose exponentials are then 0.
__device__ __forceinline__ float origin(float m) { return m == -INFINITY ? 0.f : m; }

// v = exp(v - from).
__device__ __forceinline__ void exponentials(float (&v)[32], float from) {
  float a[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) a[j] = -from;
  vadd<32>(v, v, a);
  vscale<32>(v, v, kLog2e);
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = ex2(v[j]);
}

// The epilogue of one thread: row `row` of the tile, whose 256 columns are the
// TMEM columns from `acc`.
__device__ __forceinline__ void epilogue_lse(const GemmArgs& p, uint32_t acc, int64_t row, int n,
                                             int tgt) {
  const int c0 = n * kTile;
  const int cols = p.vp - c0 < kTile ? p.vp - c0 : kTile;
  const int rel = tgt - c0;  // the target's column in this tile, if it is in it
  float m = -INFINITY, l = 0.f;
  for (int c = 0; c < cols; c += 32) {
    uint32_t r[32];
    __syncwarp();
    umma::tmem_ld32_async(acc + c, r);
    umma::tmem_wait_ld(r);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
    if (c + 32 > cols) {  // columns past the vocabulary
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = c + j < cols ? v[j] : -INFINITY;
    }
    if (static_cast<unsigned>(rel - c) < 32u) {
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) t = c + j == rel ? v[j] : t;
      p.target_logit[row] = t;
    }
    float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int j = 4; j < 32; ++j) top[j & 3] = fmaxf(top[j & 3], v[j]);
    const float nm = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
    const float from = origin(nm);
    exponentials(v, from);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j & 3] += v[j];
    l = fmaf(l, ex2((m - from) * kLog2e), (s[0] + s[1]) + (s[2] + s[3]));
    m = nm;
  }
  p.part[static_cast<int64_t>(n) * p.part_pitch + row] = make_float2(m, l);
}

__device__ __forceinline__ void epilogue_grad(const GemmArgs& p, const Maps& maps, OutBox& out,
                                              uint32_t acc, int64_t row, int n, int tgt,
                                              float lse, float scale, bool kept) {
  const int row0 = static_cast<int>(row) - static_cast<int>(threadIdx.x & 31);
  const int c0 = n * kTile;
  const int cols = p.vp - c0 < kTile ? p.vp - c0 : kTile;
  const int64_t t64 = static_cast<int64_t>(tgt) - p.v0 - c0;
  const int rel = t64 >= 0 && t64 < kTile ? static_cast<int>(t64) : -1;
  for (int c = 0; c < kTile; c += 64) {
    uint32_t r[2][32];
    __syncwarp();
    umma::tmem_ld32_async(acc + c, r[0]);
    umma::tmem_ld32_async(acc + c + 32, r[1]);
    out.open();
    umma::tmem_wait_ld(r[0]);
    umma::tmem_wait_ld(r[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b = c + 32 * h;
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[h][j]);
      exponentials(v, lse);
      if (static_cast<unsigned>(rel - b) < 32u) {
        float at = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          v[j] -= b + j == rel ? 1.f : 0.f;
          at = b + j == rel ? v[j] * scale : at;
        }
        p.lost[row] = at - __bfloat162float(__float2bfloat16_rn(at));
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= scale;
      if (!kept) {  // zeros, whatever the products of no token's row gave (0 inf = NaN)
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
      }
      if (b + 32 > cols) {  // columns past the vocabulary take no part in dh
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = b + j < cols ? v[j] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        out.put(4 * h + k, pack2(v[8 * k], v[8 * k + 1]), pack2(v[8 * k + 2], v[8 * k + 3]),
                pack2(v[8 * k + 4], v[8 * k + 5]), pack2(v[8 * k + 6], v[8 * k + 7]));
    }
    out.send(&maps.g, c0 + c, row0, false);
  }
}

// `row`: the warp's first row in the tile.
__device__ __forceinline__ void epilogue_products(const GemmArgs& p, const Maps& maps, OutBox& out,
                                                  uint32_t acc, const Unit& u, int row, int rows,
                                                  int mt, bool empty, float common) {
  const int c0 = u.n * kTile;
  const int cols = p.dim - c0 < kTile ? static_cast<int>(p.dim - c0) : kTile;
  const int64_t y = u.dw ? p.v0 + static_cast<int64_t>(u.m) * kTile + row
                         : (static_cast<int64_t>(u.split) * mt + u.m) * kTile + row;
  // nothing to write, or to add
  if (u.dw ? y >= p.vocab : u.m * kTile + row >= rows || (empty && p.add)) return;
  const int width = u.dw ? 64 : 32;
  for (int c = 0; c < cols; c += width) {
    uint32_t r[2][32];
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (empty) {
#pragma unroll
        for (int j = 0; j < 32; ++j) r[h][j] = 0u;
      } else if (h == 0 || u.dw) {
        umma::tmem_ld32_async(acc + c + 32 * h, r[h]);
      }
    }
    out.open();
    umma::tmem_wait_ld(r[0]);
    umma::tmem_wait_ld(r[1]);
    if (u.dw) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack2(__uint_as_float(r[h][8 * k + 2 * i]) * common,
                         __uint_as_float(r[h][8 * k + 2 * i + 1]) * common);
          out.put(4 * h + k, w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        out.put(k, r[0][4 * k], r[0][4 * k + 1], r[0][4 * k + 2], r[0][4 * k + 3]);
    }
    out.send(u.dw ? &maps.dw : &maps.dh, c0 + c, static_cast<int>(y), !u.dw && p.add);
  }
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    xent_gemm_kernel(const __grid_constant__ Maps maps, const GemmArgs p) {
  extern __shared__ unsigned char sm_raw[];
  const uint32_t base = (umma::smem_u32(sm_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + kBars;
  const auto full = [&](int s) { return bars + 8 * s; };
  const auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  const auto acc_full = [&](int b) { return bars + 8 * (2 * kStages + b); };
  const auto acc_empty = [&](int b) { return bars + 8 * (2 * kStages + 2 + b); };
  const uint32_t slot = bars + 8 * (2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = pair::cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      umma::mbar_init(full(s), 1);
      umma::mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      umma::mbar_init(acc_full(b), 1);
      umma::mbar_init(acc_empty(b), 2 * kEpilogueWarps);
    }
  }
  if (warp == 1) pair::tmem_alloc(slot, 512);
  umma::fence_before_sync();
  __syncthreads();
  pair::cluster_sync();
  umma::fence_after_sync();
  uint32_t tm;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tm) : "r"(slot) : "memory");
  wait_previous();
  release_next();
  const Work<MODE> work(p, blockIdx.x >> 1, gridDim.x >> 1);

  bool bad = false;
  if (warp == 0 && lane == 0) {
    // ---- copies: this CTA's halves of A and B, announced on the even CTA's barrier
    int s = 0;
    uint32_t ph = 1;
    int used = 0;  // stages that hold a copy, at most kStages
    const bool all = p.count == nullptr || rows_in_place(rows_of(p), p.tokens);
    const CUtensorMap* ma_map = MODE != kProducts && all ? &maps.h : &maps.a;
    const CUtensorMap* bt_map = all ? &maps.h : &maps.bt;
    Unit t;
    for (int i = 0; !bad && work.at(i, &t); ++i) {
      const int ma = t.m * kTile + rank * kHalfTile, nb = t.n * kTile + rank * kHalfTile;
      const int v0 = static_cast<int>(p.v0);
      for (int k = t.k0; k < t.k1; ++k) {
        if (!pair::mbar_wait(empty(s), ph, kWaitNs)) {
          bad = true;
          break;
        }
        const uint32_t a = base + s * kStage, b = a + kOperand;
        const uint32_t bar = pair::map_to(full(s), 0);
        if (rank == 0) umma::mbar_expect_tx(full(s), 2 * kStage);
        if (MODE != kProducts) {
          pair::tma_load_2d(a, ma_map, k * kBk, ma, bar);
          pair::tma_load_2d(b, &maps.b, k * kBk, v0 + nb, bar);
        } else if (!t.dw) {
          pair::tma_load_2d(a, &maps.a, k * kBk, ma, bar);
          pair::tma_load_2d(b, &maps.b, nb, v0 + k * kBk, bar);
          pair::tma_load_2d(b + kOperand / 2, &maps.b, nb + 64, v0 + k * kBk, bar);
        } else {
          pair::tma_load_2d(a, &maps.at, ma, k * kBk, bar);
          pair::tma_load_2d(a + kOperand / 2, &maps.at, ma + 64, k * kBk, bar);
          pair::tma_load_2d(b, bt_map, nb, k * kBk, bar);
          pair::tma_load_2d(b + kOperand / 2, bt_map, nb + 64, k * kBk, bar);
        }
        if (used < kStages) ++used;
        if (++s == kStages) { s = 0; ph ^= 1; }
      }
    }
    // every copy has landed, and been read, once its stage is free again
    for (int i = 0; i < used; ++i) {
      if (--s < 0) { s = kStages - 1; ph ^= 1; }
    }
    for (int i = 0; i < used; ++i) {
      if (!pair::mbar_wait(empty(s), ph ^ 1, kWaitNs)) {
        bad = true;  // far longer than any copy takes has passed
        break;
      }
      if (++s == kStages) { s = 0; ph ^= 1; }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- products
    int s = 0, n = 0;
    uint32_t ph = 0;
    Unit t;
    for (; !bad && work.at(n, &t); ++n) {
      const int b = n & 1;
      const bool a_mn = t.dw, b_mn = MODE == kProducts;
      const uint32_t id = umma::idesc_bf16(kTile, kTile, a_mn, b_mn);
      if (!pair::mbar_wait(acc_empty(b), ((n >> 1) & 1) ^ 1, kWaitNs)) {
        bad = true;
        break;
      }
      umma::fence_after_sync();
      for (int k = t.k0; k < t.k1; ++k) {
        if (!pair::mbar_wait(full(s), ph, kWaitNs)) {
          bad = true;
          break;
        }
        umma::fence_after_sync();
        const uint32_t at = base + s * kStage, bt = at + kOperand;
#pragma unroll
        for (int j = 0; j < kBk / 16; ++j)
          pair::mma_bf16(tm + b * kTile, desc(at, j, a_mn), desc(bt, j, b_mn), id,
                         k > t.k0 || j > 0);
        pair::mma_commit(empty(s));
        if (++s == kStages) { s = 0; ph ^= 1; }
      }
      if (!bad) pair::mma_commit(acc_full(b));
    }
  } else if (warp >= 2) {
    // ---- epilogue: warp w reads TMEM lanes 32 (w mod 4) ..
    const int q = warp & 3;
    const int row = static_cast<int>(rank) * kHalfTile + q * 32 + lane;
    OutBox out = {base + kOut + (warp - 2) * 2 * kBox, 0};
    const float common = MODE == kProducts ? p.common->dloss : 1.f;
    const bool shared = MODE == kGrad && p.common->shared;
    Unit t;
    for (int n = 0; !bad && work.at(n, &t); ++n) {
      const int b = n & 1;
      const int64_t r = static_cast<int64_t>(t.m) * kTile + row;
      int tgt = -1;
      float lse = 0.f, scale = 0.f;
      if (MODE != kProducts) tgt = target_of(p, r);
      if (MODE == kGrad) {
        lse = p.lse[r];
        scale = shared ? 1.f : p.scale[r];
      }
      if (!pair::mbar_wait(acc_full(b), (n >> 1) & 1, kWaitNs)) bad = true;
      if (__any_sync(0xffffffffu, bad)) {
        bad = true;
        break;
      }
      umma::fence_after_sync();
      const uint32_t acc = tm + b * kTile + (static_cast<uint32_t>(q * 32) << 16);
      if (MODE == kLse) epilogue_lse(p, acc, r, t.n, tgt);
      // rows of G past the last kept one are read up to a whole stage of dW's products
      if (MODE == kGrad && r - lane < (work.rows + kBk - 1) / kBk * kBk)
        epilogue_grad(p, maps, out, acc, r, t.n, tgt, lse, scale, r < work.rows);
      if (MODE == kProducts)
        epilogue_products(p, maps, out, acc, t, row - lane, work.rows, work.mt, t.k1 <= t.k0,
                          common);
      __syncwarp();
      umma::fence_before_sync();
      __syncwarp();
      if (lane == 0) pair::mbar_arrive(pair::map_to(acc_empty(b), 0));
    }
    out.drain();
  }
  if (bad) atomicOr(p.err, kErrXentWait);
  __syncwarp();
  umma::fence_before_sync();
  __syncthreads();
  pair::cluster_sync();  // the peer's barriers and operands stay until both are done
  umma::fence_after_sync();
  if (warp == 1) pair::tmem_dealloc(tm, 512);
}

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

// (maximum, sum) pairs of a softmax's denominator joined with (m, l): the maximum
// of all first, then the sums, each scaled to it once.
template <int N>
__device__ __forceinline__ void join(float& m, float& l, const float2 (&v)[N]) {
  float top = m;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, v[i].x);
  const float from = origin(top);
  l *= ex2((m - from) * kLog2e);
#pragma unroll
  for (int i = 0; i < N; ++i) l = fmaf(v[i].y, ex2((v[i].x - from) * kLog2e), l);
  m = top;
}
// The pairs of a warp's lanes, joined in every lane.
__device__ __forceinline__ void join_lanes(float& m, float& l) {
  float top = m;
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  l *= ex2((m - origin(top)) * kLog2e);
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
  m = top;
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

// ---- gathering the kept tokens --------------------------------------------------
constexpr int kGatherThreads = 256;

// Tokens per CTA: few, for the copy's sake, while there are at most four CTAs
// per SM (each reads all the targets).
int gather_tokens(int64_t tokens) {
  int64_t per = 16;
  while ((tokens + per - 1) / per > 4 * kSms) per *= 2;
  return static_cast<int>(per);
}

struct GatherArgs {
  const __nv_bfloat16* h;
  const int64_t* targets;
  int64_t ignore;
  int64_t tokens, vocab, dim;
  int* count;
  int* idx;            // [rows] token of the row
  int* target;         // [rows]
  __nv_bfloat16* rows;  // [rows][dim], written only where a token is ignored
  int per;             // tokens per CTA
  // forward: zeroed for ignored tokens
  float* loss;
  float* lse_out;
  // backward: gathered, and dh zeroed for ignored tokens
  const float* lse;
  const float* dloss;
  float* lse_rows;
  float* scale;
  Common* common;
  __nv_bfloat16* dh;
};

// Every CTA counts the kept tokens before its own (the targets are a few bytes
// per token), so one launch places them all, in order.
__global__ void __launch_bounds__(kGatherThreads) xent_gather_kernel(const GatherArgs p) {
  constexpr int kWarps = kGatherThreads / 32;
  __shared__ int before_n[kWarps], total_n[kWarps], warp_n[kWarps];
  __shared__ unsigned low_n[kWarps], high_n[kWarps];
  __shared__ int src[kGatherThreads], gone[kGatherThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.per;
  release_next();
  int before = 0, total = 0;
#pragma unroll 8
  for (int64_t t = tid; t < p.tokens; t += kGatherThreads) {
    const int keep = __ldg(p.targets + t) != p.ignore;
    total += keep;
    before += t < t0 ? keep : 0;
  }
  unsigned low = 0xffffffffu, high = 0u;  // of the bits of the kept tokens' dloss
  if (p.common && blockIdx.x == 0) {
#pragma unroll 8
    for (int64_t t = tid; t < p.tokens; t += kGatherThreads) {
      const int64_t tg = __ldg(p.targets + t);
      const unsigned dloss = __float_as_uint(__ldg(p.dloss + t));
      // a target outside the vocabulary counts as a dloss of its own
      const unsigned bits = tg >= 0 && tg < p.vocab ? dloss : 0xffffffffu;
      const bool keep = tg != p.ignore;
      low = keep && bits < low ? bits : low;
      high = keep && bits > high ? bits : high;
    }
  }
  for (int m = 16; m >= 1; m /= 2) {
    before += __shfl_xor_sync(0xffffffffu, before, m);
    total += __shfl_xor_sync(0xffffffffu, total, m);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    before_n[warp] = before;
    total_n[warp] = total;
    low_n[warp] = low;
    high_n[warp] = high;
  }
  __syncthreads();
  before = total = 0;
  for (int w = 0; w < kWarps; ++w) {
    before += before_n[w];
    total += total_n[w];
  }
  const bool all = rows_in_place(total, p.tokens);
  const int vec = static_cast<int>(p.dim / 8);
  const int64_t t1 = t0 + p.per < p.tokens ? t0 + p.per : p.tokens;
  for (int64_t c0 = t0; c0 < t1; c0 += kGatherThreads) {
    const int64_t t = c0 + tid;
    const bool in = t < t1;
    const int64_t tg = in ? __ldg(p.targets + t) : p.ignore;
    const bool keep = in && tg != p.ignore;
    const unsigned votes = __ballot_sync(0xffffffffu, keep);
    __syncthreads();  // the lists of the chunk before have been read
    if (lane == 0) warp_n[warp] = __popc(votes);
    __syncthreads();
    int rank = __popc(votes & ((1u << lane) - 1)), kept = 0;
    for (int w = 0; w < kWarps; ++w) {
      rank += w < warp ? warp_n[w] : 0;
      kept += warp_n[w];
    }
    if (keep) {
      const int64_t r = before + rank;
      const bool fine = tg >= 0 && tg < p.vocab;
      src[rank] = static_cast<int>(t);
      p.idx[r] = static_cast<int>(t);
      p.target[r] = fine ? static_cast<int>(tg) : -1;
      if (p.scale) {
        p.lse_rows[r] = p.lse[t];
        p.scale[r] = fine ? p.dloss[t] : NAN;
      }
    } else if (in) {
      gone[tid - rank] = static_cast<int>(t);  // `rank` kept tokens come before it
      if (p.loss) {
        p.loss[t] = 0.f;
        p.lse_out[t] = 0.f;
      }
    }
    if (!all) {
      __syncthreads();
      const int n = kept * vec;
#pragma unroll 4
      for (int i = tid; i < n; i += kGatherThreads) {
        const int r = i / vec, c = i - r * vec;
        reinterpret_cast<uint4*>(p.rows + (static_cast<int64_t>(before) + r) * p.dim)[c] =
            __ldg(reinterpret_cast<const uint4*>(p.h + src[r] * p.dim) + c);
      }
      const int absent = p.dh ? (static_cast<int>(t1 - c0 < kGatherThreads ? t1 - c0 : kGatherThreads) - kept) * vec : 0;
      for (int i = tid; i < absent; i += kGatherThreads) {
        const int r = i / vec, c = i - r * vec;
        reinterpret_cast<uint4*>(p.dh + gone[r] * p.dim)[c] = make_uint4(0, 0, 0, 0);
      }
    }
    before += kept;
  }
  if (blockIdx.x == 0 && tid == 0) {
    *p.count = total;
    if (p.common) {
      for (int w = 0; w < kWarps; ++w) {
        low = low_n[w] < low ? low_n[w] : low;
        high = high_n[w] > high ? high_n[w] : high;
      }
      const bool shared = low == high && low != ~0u;
      p.common->shared = shared;
      p.common->dloss = shared ? __uint_as_float(low) : 1.f;
    }
  }
  // past the kept rows: no target up to a whole tile, and zeros up to a whole
  // stage of the products that sum over rows
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kGatherThreads + tid;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGatherThreads;
  const int64_t end = (static_cast<int64_t>(total) + kTile - 1) / kTile * kTile;
  for (int64_t r = total + first; r < end; r += step) {
    p.target[r] = -1;
    if (p.scale) p.lse_rows[r] = p.scale[r] = 0.f;
  }
  if (!all) {
    const int64_t zeros = ((static_cast<int64_t>(total) + kBk - 1) / kBk * kBk - total) * vec;
    for (int64_t i = first; i < zeros; i += step)
      reinterpret_cast<uint4*>(p.rows + static_cast<int64_t>(total) * p.dim)[i] =
          make_uint4(0, 0, 0, 0);
  }
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

// dh of a token: the sum of the splits' partial sums and of what rounding took
// from G at the target, rounded once.
__global__ void __launch_bounds__(256) xent_dh_kernel(const GemmArgs p, const int* idx,
                                                      __nv_bfloat16* dh) {
  wait_previous();
  const int rows = rows_of(p), mt = ceil_div(rows, kTile);
  const int splits = dh_splits(mt, ceil_div(p.dim, kTile), p.kv_whole);
  const int vec = static_cast<int>(p.dim / 4);
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256, n = static_cast<int64_t>(rows) * vec;
  const int64_t plane = static_cast<int64_t>(mt) * kTile * p.dim;
  const float common = p.common->dloss;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
    const int64_t r = i / vec, c = (i - r * vec) * 4;
    const float* q = p.dh + r * p.dim + c;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
      const float4 a = *reinterpret_cast<const float4*>(q + s * plane);
      v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
    }
    if (const int t = p.target[r]; t >= 0) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.weight + t * p.dim + c));
      const float lost = p.lost[r];
      v.x = fmaf(lost, __uint_as_float(w.x << 16), v.x);
      v.y = fmaf(lost, __uint_as_float(w.x & 0xffff0000u), v.y);
      v.z = fmaf(lost, __uint_as_float(w.y << 16), v.z);
      v.w = fmaf(lost, __uint_as_float(w.y & 0xffff0000u), v.w);
    }
    *reinterpret_cast<uint2*>(dh + idx[r] * p.dim + c) =
        make_uint2(pack2(v.x * common, v.y * common), pack2(v.z * common, v.w * common));
  }
}

// ---- workspace and launches -------------------------------------------------------
struct Layout {
  size_t count, idx, target, target_logit, lse, scale, lost, rows, part, g, dh, total;
  int64_t tpad, piece, pieces, dh_rows;
};

Layout layout_of(const XentShape& s, bool backward) {
  Layout l;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  l.tpad = (s.tokens + kTile - 1) / kTile * kTile;
  const int64_t vpad = (s.vocab + kTile - 1) / kTile * kTile;
  int64_t piece = kPieceBytes / (2 * l.tpad) / kTile * kTile;
  piece = piece < kTile ? kTile : piece;
  // equal pieces, in whole tiles
  l.pieces = (vpad + piece - 1) / piece;
  l.piece = ((vpad / kTile + l.pieces - 1) / l.pieces) * kTile;
  l.pieces = (vpad + l.piece - 1) / l.piece;
  l.count = take(256);
  l.idx = take(4 * l.tpad);
  l.target = take(4 * l.tpad);
  l.rows = take(2 * l.tpad * s.dim);
  l.target_logit = l.part = l.lse = l.scale = l.lost = l.g = l.dh = 0;
  l.dh_rows = 0;
  if (!backward) {
    l.target_logit = take(4 * l.tpad);
    // a row per tile of columns; per CTA with few tokens
    const int64_t parts = vpad / kTile > kSms ? vpad / kTile : kSms;
    l.part = take(sizeof(float2) * parts * l.tpad);
  } else {
    l.lse = take(4 * l.tpad);
    l.scale = take(4 * l.tpad);
    l.lost = take(4 * l.tpad);
    l.g = take(2 * l.tpad * l.piece);
    // splits x rows: with fewer tiles than clusters the splits fill the clusters
    const int64_t nt = (s.dim + kTile - 1) / kTile;
    l.dh_rows = l.tpad + ((kClusters + nt - 1) / nt) * kTile;
    l.dh = take(4 * l.dh_rows * s.dim);
  }
  l.total = off;
  return l;
}

template <int MODE>
cudaError_t gemm(const Maps& maps, const GemmArgs& a, cudaStream_t s) {
  auto* k = xent_gemm_kernel<MODE>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  return launch_after(k, 2 * kClusters, kThreads, kSmem, s, maps, a);
}

cudaError_t gather(const GatherArgs& g, cudaStream_t s) {
  const int64_t ctas = (g.tokens + g.per - 1) / g.per;
  xent_gather_kernel<<<static_cast<unsigned>(ctas), kGatherThreads, 0, s>>>(g);
  return cudaGetLastError();
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

GatherArgs gather_args(const XentParams& p, const Layout& l, char* ws) {
  GatherArgs g = {};
  g.h = static_cast<const __nv_bfloat16*>(p.h);
  g.targets = p.targets;
  g.ignore = p.ignore_index;
  g.tokens = p.shape.tokens; g.vocab = p.shape.vocab; g.dim = p.shape.dim;
  g.count = reinterpret_cast<int*>(ws + l.count);
  g.idx = reinterpret_cast<int*>(ws + l.idx);
  g.target = reinterpret_cast<int*>(ws + l.target);
  g.rows = reinterpret_cast<__nv_bfloat16*>(ws + l.rows);
  g.per = gather_tokens(p.shape.tokens);
  return g;
}

GemmArgs gemm_args(const XentParams& p, const Layout& l, char* ws) {
  GemmArgs a = {};
  a.count = reinterpret_cast<int*>(ws + l.count);
  a.target = reinterpret_cast<int*>(ws + l.target);
  a.targets = p.targets;
  a.tokens = p.shape.tokens;
  a.vocab = p.shape.vocab; a.dim = p.shape.dim;
  a.err = p.err;
  return a;
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
      if ((e = gather(g, s)) != cudaSuccess) return e;
    }
    e = gemm<kLse>(maps, a, s);
  }
  if (e != cudaSuccess) return e;
  return launch_after(xent_join_kernel, static_cast<unsigned>((z.tokens + 31) / 32), 1024, 0, s, a,
                      p.ignore_index, direct ? nullptr : g.idx, parts, p.loss, p.lse);
}

cudaError_t launch_xent_bwd(const XentParams& p, cudaStream_t s) {
  const XentShape& z = p.shape;
  const Layout l = layout_of(z, true);
  char* ws = static_cast<char*>(p.workspace);
  GatherArgs g = gather_args(p, l, ws);
  g.lse = p.lse_in;
  g.dloss = p.dloss;
  g.lse_rows = reinterpret_cast<float*>(ws + l.lse);
  g.scale = reinterpret_cast<float*>(ws + l.scale);
  g.common = reinterpret_cast<Common*>(ws + l.count + 64);  // `count` holds 256 bytes
  g.dh = static_cast<__nv_bfloat16*>(p.dh);
  GemmArgs a = gemm_args(p, l, ws);
  a.lse = g.lse_rows;
  a.scale = g.scale;
  a.common = g.common;
  a.lost = reinterpret_cast<float*>(ws + l.lost);
  a.weight = static_cast<const __nv_bfloat16*>(p.weight);
  void* piece = ws + l.g;
  a.dh = reinterpret_cast<float*>(ws + l.dh);
  a.kv_whole = ceil_div(l.piece, kBk);
  Maps in = {}, out = {};
  if (!map_bf16_sw128(&in.a, g.rows, z.dim, l.tpad, z.dim, kHalfTile) ||
      !map_bf16_sw128(&in.h, p.h, z.dim, z.tokens, z.dim, kHalfTile) ||
      !map_bf16_sw128(&in.b, p.weight, z.dim, z.vocab, z.dim, kHalfTile) ||
      !map_bf16_sw128(&in.g, piece, l.piece, l.tpad, l.piece, 32) ||
      !map_bf16_sw128(&out.dw, p.dweight, z.dim, z.vocab, z.dim, 32) ||
      !map_f32_sw128(&out.dh, a.dh, z.dim, l.dh_rows, z.dim, 32) ||
      !map_bf16_sw128(&out.a, piece, l.piece, l.tpad, l.piece, kHalfTile) ||
      !map_bf16_sw128(&out.b, p.weight, z.dim, z.vocab, z.dim, kBk) ||
      !map_bf16_sw128(&out.at, piece, l.piece, l.tpad, l.piece, kBk) ||
      !map_bf16_sw128(&out.bt, g.rows, z.dim, l.tpad, z.dim, kBk) ||
      !map_bf16_sw128(&out.h, p.h, z.dim, z.tokens, z.dim, kBk))
    return cudaErrorInvalidValue;
  cudaError_t e = gather(g, s);
  if (e != cudaSuccess) return e;
  for (int64_t i = 0; i < l.pieces; ++i) {
    a.v0 = i * l.piece;
    a.vp = static_cast<int>(z.vocab - a.v0 < l.piece ? z.vocab - a.v0 : l.piece);
    a.add = i > 0;
    if ((e = gemm<kGrad>(in, a, s)) != cudaSuccess) return e;
    if ((e = gemm<kProducts>(out, a, s)) != cudaSuccess) return e;
  }
  return launch_after(xent_dh_kernel, 4 * kSms, 256, 0, s, a, g.idx,
                      static_cast<__nv_bfloat16*>(p.dh));
}

}  // namespace ssm
