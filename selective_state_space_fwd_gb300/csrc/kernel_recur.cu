// kernel_recur.cu -- the gated linear recurrence along time (formulas in
// recur.cuh): prompts with valid lengths and a carried state, every gradient,
// single steps in place.
//
// Work split: a CTA owns 32 x VEC channels (128 bytes of a row) of one batch row
// and walks its time in tiles of kTile steps.  Each of its warps folds kSteps
// consecutive steps of the tile, lane by lane, into the stretch's map; the
// maps meet in shared memory, every thread composes those before its own with
// the carried state, and the warp's outputs follow from the state that enters it.
// The next tile's rows are loaded while a tile is folded.  While the
// GPU holds more, a cluster of R of them shares the time of its channels, each
// taking every R-th tile: the tiles' maps then go to all of the cluster's shared
// memories, one barrier of the cluster per round.  No step is read twice, and no
// CTA waits for one that might not run.
//
// Backward, from the last tile to the first, with l_t = dL/dh_t:
//   l_t = dy_t + a_{t+1} l_{t+1},   dv = b l,   dg = l (h_{t-1} - v) b sigmoid(g),
//   dfloor = sum l (h_{t-1} - v) sigmoid(-g).
// What enters a tile from its past is the state that the forward kept there (one
// per kTile steps); the states inside are formed again.  The same maps carry
// m = a l backwards: m -> e' + P m, with the same P.  dfloor is summed per
// thread, over the warps and, by a second kernel, over the CTAs, in a fixed order.
//
// Tensors whose rows start on 16-byte boundaries take kernel_recur_tma.cu; the kernels
// here read rows directly, two bf16 channels per lane where both lie on 4 bytes and one
// otherwise.  Bound by the latency of the loads that 16 warps per SM have in flight:
// fp32 8 x 4096 x 1025 forward 91 us (4.4 TB/s), backward 180 us (3.7 TB/s), bf16
// 8 x 4096 x 1026 91 and 155 us; with 1024 channels staged by TMA 63 and 103, 47 and 65.
//
// A single step is bound by its launch: bf16 1024 x 2048 in 4.4 us, of which its bytes
// take 4.3.
#include "cluster.cuh"
#include "f32x2.cuh"
#include "pdl.cuh"
#include "recur.cuh"
#include "umma_pair.cuh"
#include "vec.cuh"

namespace ssm {
namespace {

using recur::Cell;

constexpr int kWarps = 8;
constexpr int kSteps = 8;                  // per warp and tile
constexpr int kTile = kWarps * kSteps;     // steps of a tile, and between kept states
static_assert(kTile == kRecurChunk, "the states that the backward starts from");
constexpr int kThreads = kWarps * 32;

// Where a thread stands.
template <int VEC>
struct Place {
  int warp, lane;
  uint32_t rank, size;   // in the cluster
  int64_t b, d;          // batch row, first channel
  bool on;               // d < dim
  __device__ __forceinline__ Place(int64_t dim, uint32_t r) : size(r) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    const int64_t groups = (dim + 32 * VEC - 1) / (32 * VEC);
    const int64_t unit = blockIdx.x / r;
    rank = blockIdx.x - static_cast<unsigned>(unit) * r;
    b = unit / groups;
    d = (unit - b * groups) * (32 * VEC) + lane * VEC;
    on = d < dim;
  }
};

// kSteps rows of a strided tensor from step t0 on, 0 past step `end` and past the
// last channel.
template <typename T, int VEC>
__device__ __forceinline__ void load_rows(typename Cell<T, VEC>::Word (&w)[kSteps], const T* row,
                                          int64_t step, int64_t t0, int64_t end, bool on) {
  using Word = typename Cell<T, VEC>::Word;
  const T* q = row + t0 * step;
  if (t0 + kSteps <= end) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      w[s] = on ? __ldg(reinterpret_cast<const Word*>(q + s * step)) : Word(0);
  } else {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      w[s] = on && t0 + s < end ? __ldg(reinterpret_cast<const Word*>(q + s * step)) : Word(0);
  }
}

// kSteps rows of a contiguous [.., dim] tensor, up to step `end`.
template <typename T, int VEC>
__device__ __forceinline__ void store_rows(const typename Cell<T, VEC>::Word (&w)[kSteps], T* row,
                                           int64_t dim, int64_t t0, int64_t end, bool on) {
  using Word = typename Cell<T, VEC>::Word;
  T* q = row + t0 * dim;
  if (!on) return;
  if (t0 + kSteps <= end) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) *reinterpret_cast<Word*>(q + s * dim) = w[s];
  } else {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (t0 + s < end) *reinterpret_cast<Word*>(q + s * dim) = w[s];
  }
}

// Stretches one after the other: (P, e) per channel in `all`, 1 - P in `rest`.
template <int VEC>
__device__ __forceinline__ void none(float (&all)[2 * VEC], float (&rest)[VEC]) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    all[2 * v] = 1.f;
    all[2 * v + 1] = rest[v] = 0.f;
  }
}
// ... and then one of which c is kept, from which e comes; a channel's are so far apart.
template <int VEC>
__device__ __forceinline__ void then(float (&all)[2 * VEC], float (&rest)[VEC], const float* c,
                                     int c_step, const float* e, int e_step) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const float P = recur::product(c[v * c_step]);
    all[2 * v] *= P;
    rest[v] = fmaf(P, rest[v], recur::remainder(c[v * c_step]));
    all[2 * v + 1] = fmaf(P, all[2 * v + 1], e[v * e_step]);
  }
}
template <int VEC>
__device__ __forceinline__ void keep_all(float (&all)[2 * VEC], const float (&rest)[VEC]) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) all[2 * v] = recur::kept(all[2 * v], rest[v]);
}

// The maps of the tiles that the cluster's CTAs hold in a round, sent to all of
// them; `slots` alternates so that one barrier per round is enough.
template <int N>
__device__ __forceinline__ void share(float (*slots)[32][N], const Place<N / 2>& at,
                                      const float (&v)[N]) {
  if (at.warp == 0) {
    const uint32_t mine = umma::smem_u32(&slots[at.rank][at.lane][0]);
    for (uint32_t r = 0; r < at.size; ++r) {
      const uint32_t to = pair::map_to(mine, r);
#pragma unroll
      for (int i = 0; i < N; i += 2)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to + 4 * i), "f"(v[i]),
                     "f"(v[i + 1])
                     : "memory");
    }
  }
  pair::cluster_sync();
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2) recur_fwd_kernel(const RecurParams p, uint32_t size) {
  using Word = typename Cell<T, VEC>::Word;
  constexpr int N = 2 * VEC;  // floats of a map: P as it is kept, and e, per channel
  __shared__ __align__(16) float maps[2][kWarps][32][N];
  __shared__ __align__(16) float tiles_s[2][kMaxCluster][32][N];
  const Place<VEC> at(p.dim, size);
  const int64_t len = recur::valid_of(p.valid_len, at.b, p.seqlen);
  const int64_t tiles = (p.seqlen + kTile - 1) / kTile, live = (len + kTile - 1) / kTile;
  const int64_t rounds = (live + size - 1) / size;
  const int64_t d = at.on ? at.d : 0;
  const T* gate = static_cast<const T*>(p.gate) + at.b * p.gate_batch + d;
  const T* value = static_cast<const T*>(p.value) + at.b * p.value_batch + d;
  T* y = static_cast<T*>(p.y) + at.b * p.seqlen * p.dim + d;
  float* states = p.states ? p.states + at.b * tiles * p.dim + d : nullptr;
  const int inside = at.warp * kSteps;

  recur::Floor<VEC> floor;
  float x[VEC];  // the state that enters the round
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    floor.set(v, p.floor ? __ldg(p.floor + d + v) : 0.f);
    // before the first barrier, and not as a constant: out_final may be the same memory
    x[v] = p.state0 ? p.state0[at.b * p.dim + d + v] : 0.f;
  }
  Word gw[kSteps], vw[kSteps];
  int64_t t0 = static_cast<int64_t>(at.rank) * kTile + inside;
  load_rows<T, VEC>(gw, gate, p.gate_step, t0, len, at.on);
  load_rows<T, VEC>(vw, value, p.value_step, t0, len, at.on);
  if (size > 1) pair::cluster_sync();  // all of the cluster has started
  for (int64_t i = 0; i < rounds; ++i, t0 += static_cast<int64_t>(size) * kTile) {
    float a[kSteps][VEC], u[kSteps][VEC];  // u: b v
    float hl[VEC], pl[VEC], ql[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      hl[v] = ql[v] = 0.f;
      pl[v] = 1.f;
    }
    const int64_t left = len - t0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float g[VEC], open[VEC], b[VEC];
      Cell<T, VEC>::get(gw[s], g);
      Cell<T, VEC>::get(vw[s], u[s]);
      recur::gates<T>(g, floor, open, b, a[s]);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        u[s][v] *= b[v];
        if (s >= left) {
          a[s][v] = 1.f;
          b[v] = u[s][v] = 0.f;
        }
        hl[v] = fmaf(a[s][v], hl[v], u[s][v]);
        ql[v] = fmaf(a[s][v], ql[v], b[v]);
        pl[v] *= a[s][v];
      }
    }
    const int64_t next = t0 + static_cast<int64_t>(size) * kTile;
    load_rows<T, VEC>(gw, gate, p.gate_step, next, len, at.on);
    load_rows<T, VEC>(vw, value, p.value_step, next, len, at.on);
    const int k = i & 1;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      maps[k][at.warp][at.lane][2 * v] = recur::kept(pl[v], ql[v]);
      maps[k][at.warp][at.lane][2 * v + 1] = hl[v];
    }
    __syncthreads();
    float xt[VEC];  // the state that enters this CTA's tile
    if (size > 1) {
      float all[N], rest[VEC];
      none<VEC>(all, rest);
      if (at.warp == 0) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          then<VEC>(all, rest, maps[k][w][at.lane], 2, maps[k][w][at.lane] + 1, 2);
        keep_all<VEC>(all, rest);
      }
      share<N>(tiles_s[k], at, all);
      for (uint32_t r = 0; r < size; ++r)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if (r == at.rank) xt[v] = x[v];
          x[v] = recur::through(tiles_s[k][r][at.lane][2 * v], x[v], tiles_s[k][r][at.lane][2 * v + 1]);
        }
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) xt[v] = x[v];
    }
    float in[VEC], out[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) in[v] = out[v] = xt[v];
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (w == at.warp) in[v] = out[v];
        out[v] = recur::through(maps[k][w][at.lane][2 * v], out[v], maps[k][w][at.lane][2 * v + 1]);
      }
    if (size == 1) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) x[v] = out[v];
    }
    if (states && at.warp == 0 && at.on && t0 < p.seqlen) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) states[t0 / kTile * p.dim + v] = xt[v];
    }
    Word yw[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float f[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        in[v] = fmaf(a[s][v], in[v], u[s][v]);
        f[v] = s < left ? in[v] : 0.f;
      }
      yw[s] = Cell<T, VEC>::put(f);
    }
    store_rows<T, VEC>(yw, y, p.dim, t0, p.seqlen, at.on);
  }
  // x is the last valid step's state
  if (p.out_final && at.rank == 0 && at.warp == 0 && at.on) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) p.out_final[at.b * p.dim + d + v] = x[v];
  }
  // past the valid steps: tiles that no round has covered
  Word zero[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) zero[s] = Word(0);
  for (; t0 - inside < p.seqlen; t0 += static_cast<int64_t>(size) * kTile) {
    store_rows<T, VEC>(zero, y, p.dim, t0, p.seqlen, at.on);
    if (states && at.warp == 0 && at.on) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) states[t0 / kTile * p.dim + v] = x[v];
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2)
    recur_bwd_kernel(const RecurBwdParams q, uint32_t size) {
  using Word = typename Cell<T, VEC>::Word;
  constexpr int N = 2 * VEC;
  const RecurParams& p = q.fwd;
  __shared__ __align__(16) float past[2][kWarps][32][N];         // (P, e) of the states
  __shared__ __align__(16) float coming[2][kWarps][32][VEC];     // e' of m
  __shared__ __align__(16) float tiles_s[2][kMaxCluster][32][N];  // (P, e') of the tiles
  const Place<VEC> at(p.dim, size);
  const int64_t len = recur::valid_of(p.valid_len, at.b, p.seqlen);
  const int64_t tiles = (p.seqlen + kTile - 1) / kTile, live = (len + kTile - 1) / kTile;
  const int64_t rounds = (live + size - 1) / size;
  const int64_t d = at.on ? at.d : 0;
  const T* gate = static_cast<const T*>(p.gate) + at.b * p.gate_batch + d;
  const T* value = static_cast<const T*>(p.value) + at.b * p.value_batch + d;
  const int64_t base = at.b * p.seqlen * p.dim + d;
  const T* dy = static_cast<const T*>(q.dy) + base;
  T* dgate = static_cast<T*>(q.dgate) + base;
  T* dvalue = static_cast<T*>(q.dvalue) + base;
  const float* states = q.states + at.b * tiles * p.dim + d;
  const int inside = at.warp * kSteps;

  recur::Floor<VEC> floor;
  float m[VEC], dfloor[VEC];  // m: a l of the step after the round's last; half of dfloor
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    floor.set(v, p.floor ? __ldg(p.floor + d + v) : 0.f);
    m[v] = q.dfinal ? __ldg(q.dfinal + at.b * p.dim + d + v) : 0.f;
    dfloor[v] = 0.f;
  }
  if (size > 1) pair::cluster_sync();  // all of the cluster has started
  for (int64_t i = 0; i < rounds; ++i) {
    const int64_t tile = live - 1 - i * size - at.rank;  // negative: none is left
    const int64_t t0 = tile * kTile + inside;
    const int64_t end = tile < 0 ? t0 : len;
    const int64_t left = end - t0;
    Word gw[kSteps], vw[kSteps], yw[kSteps];
    load_rows<T, VEC>(gw, gate, p.gate_step, t0, end, at.on);
    load_rows<T, VEC>(vw, value, p.value_step, t0, end, at.on);
    load_rows<T, VEC>(yw, dy, p.dim, t0, end, at.on);
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = tile < 0 ? 0.f : __ldg(states + tile * p.dim + v);
    float open[kSteps][VEC], hold[kSteps][VEC], a[kSteps][VEC], u[kSteps][VEC];
    float pl[VEC], ql[VEC], hl[VEC], ml[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      ql[v] = hl[v] = ml[v] = 0.f;
      pl[v] = 1.f;
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float g[VEC], b[VEC];
      Cell<T, VEC>::get(gw[s], g);
      Cell<T, VEC>::get(vw[s], u[s]);
      recur::gates<T>(g, floor, open[s], b, a[s]);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        hold[s][v] = recur::holding(g[v], open[s][v]);
        if (s >= left) {
          open[s][v] = b[v] = 0.f;
          a[s][v] = 1.f;
        }
        hl[v] = fmaf(a[s][v], hl[v], b[v] * u[s][v]);
        ql[v] = fmaf(a[s][v], ql[v], b[v]);
        pl[v] *= a[s][v];
      }
    }
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
      float l[VEC];
      Cell<T, VEC>::get(yw[s], l);
#pragma unroll
      for (int v = 0; v < VEC; ++v) ml[v] = a[s][v] * (l[v] + ml[v]);
    }
    const int k = i & 1;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      past[k][at.warp][at.lane][2 * v] = recur::kept(pl[v], ql[v]);
      past[k][at.warp][at.lane][2 * v + 1] = hl[v];
      coming[k][at.warp][at.lane][v] = ml[v];
    }
    __syncthreads();
    float mt[VEC];  // what enters the tile from the steps after it
    if (size > 1) {
      float all[N], rest[VEC];
      none<VEC>(all, rest);
      if (at.warp == 0) {
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w)
          then<VEC>(all, rest, past[k][w][at.lane], 2, coming[k][w][at.lane], 1);
        keep_all<VEC>(all, rest);
      }
      share<N>(tiles_s[k], at, all);
      for (uint32_t r = 0; r < size; ++r)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if (r == at.rank) mt[v] = m[v];
          m[v] = recur::through(tiles_s[k][r][at.lane][2 * v], m[v], tiles_s[k][r][at.lane][2 * v + 1]);
        }
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) mt[v] = m[v];
    }
    float mi[VEC];
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (w < at.warp)
          h[v] = recur::through(past[k][w][at.lane][2 * v], h[v], past[k][w][at.lane][2 * v + 1]);
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (w == at.warp) mi[v] = mt[v];
        mt[v] = recur::through(past[k][w][at.lane][2 * v], mt[v], coming[k][w][at.lane][v]);
      }
    if (size == 1) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) m[v] = mt[v];
    }
    // the distance of the state before a step to its value, in the value's place
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float in = floor.half[v] * open[s][v] * u[s][v];
        u[s][v] = h[v] - u[s][v];
        h[v] = fmaf(a[s][v], h[v], in);
      }
    float some[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) some[v] = 0.f;
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
      float dv[VEC], dg[VEC], l[VEC];
      Cell<T, VEC>::get(yw[s], l);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float b = floor.half[v] * open[s][v], lam = l[v] + mi[v];
        mi[v] = a[s][v] * lam;
        dv[v] = b * lam;
        const float w = lam * u[s][v];
        dg[v] = w * (b * hold[s][v]);
        some[v] = fmaf(w, open[s][v], some[v]);
      }
      if (s >= left) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) dv[v] = dg[v] = 0.f;
      }
      vw[s] = Cell<T, VEC>::put(dv);
      gw[s] = Cell<T, VEC>::put(dg);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) dfloor[v] += some[v];
    const int64_t stop = tile < 0 ? t0 : p.seqlen;
    store_rows<T, VEC>(vw, dvalue, p.dim, t0, stop, at.on);
    store_rows<T, VEC>(gw, dgate, p.dim, t0, stop, at.on);
  }
  if (q.dstate0 && at.rank == 0 && at.warp == 0 && at.on) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) q.dstate0[at.b * p.dim + d + v] = m[v];
  }
  Word zero[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) zero[s] = Word(0);
  for (int64_t tile = live + at.rank; tile < tiles; tile += size) {
    store_rows<T, VEC>(zero, dvalue, p.dim, tile * kTile + inside, p.seqlen, at.on);
    store_rows<T, VEC>(zero, dgate, p.dim, tile * kTile + inside, p.seqlen, at.on);
  }
  if (q.dfloor) {
    __syncthreads();
    float* sums = &past[0][0][0][0];  // [warp][lane][VEC]
#pragma unroll
    for (int v = 0; v < VEC; ++v) sums[(at.warp * 32 + at.lane) * VEC + v] = dfloor[v];
    __syncthreads();
    if (at.warp == 0 && at.on) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        float t = 0.f;
        for (int w = 0; w < kWarps; ++w) t += sums[(w * 32 + at.lane) * VEC + v];
        q.partial[(at.b * size + at.rank) * p.dim + d + v] = 0.5f * t;
      }
    }
  }
}

// dfloor: the sum of `rows` partial sums per channel; 8 threads share a channel.
__global__ void __launch_bounds__(256) recur_floor_kernel(const float* partial, int64_t rows,
                                                          int64_t dim, float* dfloor) {
  __shared__ float part[8][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  wait_previous();
  float t = 0.f;
  if (d < dim) {
#pragma unroll 8
    for (int64_t r = w; r < rows; r += 8) t += partial[r * dim + d];
  }
  part[w][lane] = t;
  __syncthreads();
  if (w == 0 && d < dim) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += part[i][lane];
    dfloor[d] = t;
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256) recur_step_kernel(const RecurParams p) {
  const int64_t vecs = p.dim / VEC;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t b = i / vecs, d = (i - b * vecs) * VEC;
  if (b >= p.batch) return;
  float g[VEC], u[VEC], h[VEC], f[VEC], open[VEC], in[VEC], a[VEC];
  recur::Floor<VEC> floor;
  load_f<T, VEC>(static_cast<const T*>(p.gate) + b * p.gate_batch + d, g);
  load_f<T, VEC>(static_cast<const T*>(p.value) + b * p.value_batch + d, u);
  widen<VEC>(raw_load_rw<float, VEC>(p.out_final + b * p.dim + d), h);
  if (p.floor) {
    load_f<float, VEC>(p.floor + d, f);
  } else {
#pragma unroll
    for (int v = 0; v < VEC; ++v) f[v] = 0.f;
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) floor.set(v, f[v]);
  recur::gates<T>(g, floor, open, in, a);
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    h[v] = recur::through(recur::kept(a[v], in[v]), h[v], in[v] * u[v]);
  store_f<float, VEC>(p.out_final + b * p.dim + d, h);
  store_f<T, VEC>(static_cast<T*>(p.y) + b * p.dim + d, h);
}

// Whether rows of 2 bf16 channels can be read in one access.
bool pairs(const RecurParams& p) {
  return p.dim % 2 == 0 && p.gate_batch % 2 == 0 && p.gate_step % 2 == 0 &&
         p.value_batch % 2 == 0 && p.value_step % 2 == 0 &&
         (reinterpret_cast<uintptr_t>(p.gate) | reinterpret_cast<uintptr_t>(p.value) |
          reinterpret_cast<uintptr_t>(p.y)) % 4 == 0;
}

// CTAs that share the time of a channel group: a power of two, doubled while all clusters
// run at once and every CTA has a tile (fp32 1 x 65536 x 601, 19 groups, forward: 8 CTAs
// 269 us, 16, some of them after the others, 289 us).
template <auto KERNEL>
int cluster_of(const RecurParams& p, int64_t units) {
  const int64_t tiles = (p.seqlen + kTile - 1) / kTile;
  int i = 0;
  while (i < 4 && (int64_t(2) << i) <= tiles && units <= resident_clusters<KERNEL>(i + 1, kThreads, 0))
    ++i;
  return 1 << i;
}

// `lanes`: channels of a CTA; *size: the CTAs of a cluster.
template <auto KERNEL, typename A>
cudaError_t launch(const RecurParams& p, int lanes, const A& args, int* size, cudaStream_t s) {
  const int64_t units = p.batch * ((p.dim + lanes - 1) / lanes);
  *size = cluster_of<KERNEL>(p, units);
  if (*size > kPortableCluster) {
    const cudaError_t e = allow_large_clusters(reinterpret_cast<const void*>(KERNEL));
    if (e != cudaSuccess) return e;
  }
  const ClusterLaunch l(units, *size, kThreads, 0, s);
  return cudaLaunchKernelEx(&l.cfg, KERNEL, args, static_cast<uint32_t>(*size));
}

}  // namespace

int64_t recur_bwd_partials(int64_t batch) { return batch * kMaxCluster; }

cudaError_t launch_recur_fwd(const RecurParams& p, bool bf16, unsigned* err, cudaStream_t s) {
  if (recur_tma_ok(p, bf16)) return launch_recur_fwd_tma(p, bf16, err, s);
  int size;
  if (!bf16) return launch<recur_fwd_kernel<float, 1>>(p, 32, p, &size, s);
  return pairs(p) ? launch<recur_fwd_kernel<__nv_bfloat16, 2>>(p, 64, p, &size, s)
                  : launch<recur_fwd_kernel<__nv_bfloat16, 1>>(p, 32, p, &size, s);
}

cudaError_t launch_recur_bwd(const RecurBwdParams& q, bool bf16, unsigned* err, cudaStream_t s) {
  const RecurParams& p = q.fwd;
  const bool two = bf16 && pairs(p) &&
                   (reinterpret_cast<uintptr_t>(q.dy) | reinterpret_cast<uintptr_t>(q.dgate) |
                    reinterpret_cast<uintptr_t>(q.dvalue)) % 4 == 0;
  int size;
  cudaError_t e;
  if (recur_bwd_tma_ok(q, bf16))
    e = launch_recur_bwd_tma(q, bf16, err, &size, s);
  else if (!bf16)
    e = launch<recur_bwd_kernel<float, 1>>(p, 32, q, &size, s);
  else
    e = two ? launch<recur_bwd_kernel<__nv_bfloat16, 2>>(p, 64, q, &size, s)
            : launch<recur_bwd_kernel<__nv_bfloat16, 1>>(p, 32, q, &size, s);
  if (e != cudaSuccess || !q.dfloor) return e;
  return launch_after(recur_floor_kernel, static_cast<unsigned>((p.dim + 31) / 32), 256, 0, s,
                      q.partial, p.batch * size, p.dim, q.dfloor);
}

cudaError_t launch_recur_step(const RecurParams& p, bool bf16, cudaStream_t s) {
  const auto wide = [&](int vec, size_t bytes) {
    return p.dim % vec == 0 && p.gate_batch % vec == 0 && p.value_batch % vec == 0 &&
           (reinterpret_cast<uintptr_t>(p.gate) | reinterpret_cast<uintptr_t>(p.value) |
            reinterpret_cast<uintptr_t>(p.y)) % bytes == 0 &&
           (reinterpret_cast<uintptr_t>(p.out_final) | reinterpret_cast<uintptr_t>(p.floor)) % 16 == 0;
  };
  const auto go = [&](auto* kernel, int vec) {
    const int64_t n = p.batch * (p.dim / vec);
    kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(p);
    return cudaGetLastError();
  };
  if (!bf16) return wide(4, 16) ? go(recur_step_kernel<float, 4>, 4) : go(recur_step_kernel<float, 1>, 1);
  return wide(8, 16) ? go(recur_step_kernel<__nv_bfloat16, 8>, 8)
                     : go(recur_step_kernel<__nv_bfloat16, 1>, 1);
}

}  // namespace ssm
