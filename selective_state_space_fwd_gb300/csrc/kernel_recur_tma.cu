// kernel_recur_tma.cu -- the gated linear recurrence (recur.cuh has the formulas,
// kernel_recur.cu the split of the work) with its rows staged by TMA, for tensors
// whose rows start on 16-byte boundaries and whose strides a tensor map takes
// (axes_of).
//
// A CTA of W warps owns 128 bytes of channels of a batch row and walks its time in
// tiles of W x kSteps steps, a warp folding kSteps of them.  The tiles of gate and
// value (and dy) arrive in a ring of slots; a slot is free again when all warps
// have taken its rows into registers, which the tile's one barrier, for the warps'
// maps, tells.  Results leave through shared memory, a box per warp.  Masked steps
// are rewritten in the slot as closed gates, so that the loops need no masks.
//
// Two passes over a warp's steps, from registers: the first folds them into the
// stretch's map, the second runs them from the state that enters.  Keeping the outputs
// from a state of 0 and adding the state's share instead costs as many instructions,
// and where a channel forgets within a stretch it leaves an error of the size of the
// state before it.
//
// Measured on GB300, forward and backward: fp32 8 x 4096 x 1024 63 and 103 us (6.4 and
// 6.5 TB/s), bound by HBM; bf16 47 and 65 us (4.3 and 5.1) and 2 x 32768 x 2048 in clusters
// of 4 167 and 264 us (4.8 and 5.1): 53 and 49 % of the issue slots with four and two
// warps per scheduler, which wait for their own dependent steps; bf16 prompts 32 x 2048 x 1536
// with valid lengths 70 us forward; fp32 1 x 65536 x 256 in clusters of 16, 128 CTAs in all,
// 59 and 116 us (3.4 and 2.9 TB/s): a round of a cluster takes 1.8 us, the latency of its
// dependent steps.  With h + b (v - h) for a h + b v and a product P alone, which loses a
// small a and a long memory's digits, these took 62 and 101, 39 and 59, 132 and 233, 68, 49 and 107
// us; the choices of shapes below were measured with that.  With the cluster's own barrier in
// place of the exchange the last took 106 and 219 us, and with all of a round's latency in the
// open 92 us forward.
#include <cuda.h>

#include "cluster.cuh"
#include "f32x2.cuh"
#include "pdl.cuh"
#include "recur.cuh"
#include "tma_map.h"
#include "umma_pair.cuh"

namespace ssm {
namespace {

using recur::rcp;

constexpr int kSms = 152;
constexpr int kSteps = 16;                       // per warp and tile
constexpr uint32_t kRow = 128;                   // bytes of a step's channels
constexpr uint32_t kBox = kSteps * kRow;         // of a warp's rows
constexpr uint64_t kWaitNs = 2000000000ull;

template <typename T> struct Of;
template <> struct Of<float> { static constexpr int kVec = 1; };
template <> struct Of<__nv_bfloat16> { static constexpr int kVec = 2; };

__device__ __forceinline__ uint32_t lds(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void unpack(uint32_t w, float (&f)[1]) { f[0] = __uint_as_float(w); }
__device__ __forceinline__ void unpack(uint32_t w, float (&f)[2]) {
  f[0] = __uint_as_float(w << 16);
  f[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack(const float (&f)[1]) { return __float_as_uint(f[0]); }
__device__ __forceinline__ uint32_t pack(const float (&f)[2]) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The words of a closed gate (+infinity).
template <typename T> __device__ __forceinline__ uint32_t closed() {
  return sizeof(T) == 4 ? 0x7f800000u : 0x7f807f80u;
}

// d = a - b.
template <int V>
__device__ __forceinline__ void minus(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  float m[V];
#pragma unroll
  for (int v = 0; v < V; ++v) m[v] = -1.f;
  vfma<V>(d, b, m, a);
}
// Waits for a phase of an mbarrier that this CTA alone arrives on; false after kWaitNs.
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (;;) {
    if (umma::mbar_wait(bar, parity, 64)) return true;
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t0 == 0) t0 = t;
    else if (t - t0 > kWaitNs) return false;
  }
}

// A lane's 2 V floats in shared memory: P as it is kept, and e, of its channels.
template <int V> struct alignas(8 * V) Map {
  float p[V], e[V];
  // The state (or what goes back) that leaves when x enters.
  __device__ __forceinline__ void through(float (&x)[V]) const {
    float d[V], k[V];
    vfma<V>(d, x, p, e);
#pragma unroll
    for (int v = 0; v < V; ++v) k[v] = recur::is_rest(p[v]);
    vfma<V>(x, x, k, d);
  }
};
// Steps or stretches, one after the other.
template <int V> struct Fold {
  float p[V], q[V], e[V];
  __device__ __forceinline__ Fold() {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = 1.f;
      q[v] = e[v] = 0.f;
    }
  }
  __device__ __forceinline__ void then(const float (&a)[V], const float (&b)[V], const float (&add)[V]) {
    vmul<V>(p, a, p);
    vfma<V>(q, a, q, b);
    vfma<V>(e, a, e, add);
  }
  __device__ __forceinline__ void then(const Map<V>& m) {
    float a[V], b[V], k[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      k[v] = recur::is_rest(m.p[v]);
      b[v] = 1.f;
    }
    vadd<V>(a, m.p, k);  // P
    minus<V>(b, b, k);
    minus<V>(b, b, m.p);  // 1 - P
    then(a, b, m.e);
  }
  __device__ __forceinline__ Map<V> map() const {
    Map<V> m;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m.p[v] = recur::kept(p[v], q[v]);
      m.e[v] = e[v];
    }
    return m;
  }
};

// Axes of a [batch, seqlen, dim] tensor's map beyond the channels.
struct Axes {
  bool ok, time_last;
  int64_t inner, outer;
};

// Tiles in shared memory.  With 3 (in fewer CTAs per SM) the measured shapes took as
// long or longer.
constexpr int kSlots = 2;

struct TmaArgs {
  uint32_t size;               // CTAs of a cluster
  bool gate_last, value_last;  // the maps' axes are (channel, batch, time)
  unsigned* err;
};

// NT tensors' tiles, each in a slot: they are used in turn, and loaded again when
// their rows have been taken.
template <int W, int NT>
struct Ring {
  static constexpr uint32_t kTileBytes = W * kBox;
  static constexpr uint32_t kSlot = NT * kTileBytes;
  uint32_t base, bars;
  int at, phase;  // the slot in use, and its barrier's parity
  __device__ __forceinline__ uint32_t slot() const { return base + at * kSlot; }
  __device__ __forceinline__ void init() const {
    if (threadIdx.x == 0)
      for (int s = 0; s < kSlots; ++s) umma::mbar_init(bars + 8 * s, 1);
  }
  __device__ __forceinline__ void load(int s, const CUtensorMap* const (&map)[NT],
                                       const bool (&last)[NT], int x, int t, int b) const {
    const uint32_t bar = bars + 8 * s;
    umma::mbar_expect_tx(bar, kSlot);
#pragma unroll
    for (int i = 0; i < NT; ++i)
      umma::tma_load_3d(base + s * kSlot + i * kTileBytes, map[i], x, last[i] ? b : t,
                        last[i] ? t : b, bar);
  }
  __device__ __forceinline__ bool wait() const { return pair::mbar_wait(bars + 8 * at, phase, kWaitNs); }
  __device__ __forceinline__ void next() {
    if (++at == kSlots) {
      at = 0;
      phase ^= 1;
    }
  }
  // The copy of round i, which nothing has waited for, has landed.
  __device__ __forceinline__ void drain(int i) const {
    pair::mbar_wait(bars + 8 * (i % kSlots), (i / kSlots) & 1, kWaitNs);
  }
};

__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t box, int x, int t, int b) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   map),
               "r"(x), "r"(t), "r"(b), "r"(box)
               : "memory");
}
__device__ __forceinline__ void commit_stores() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The warp's boxes have been read by the copies before.
__device__ __forceinline__ void boxes_free() {
  if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

// The maps of a round's tiles meet in every CTA of the cluster: each sends its tile's to
// all (itself too), and the bytes arrive on the receiver's mbarrier, so that no CTA
// waits for more than the maps.  A CTA sends round i + 1 before it reads
// round i (it folds the next tile meanwhile), but after it has read round i - 1, for
// which all had sent theirs, after reading round i - 3: four buffers are enough.
constexpr int kBuffers = 4;
template <int V>
struct Exchange {
  Map<V> (*slots)[32];  // [kBuffers][size][32]
  uint32_t bars, rank, size;
  __device__ __forceinline__ void init() const {
    if (threadIdx.x == 0)
      for (int k = 0; k < kBuffers; ++k) umma::mbar_init(bars + 8 * k, 1);
  }
  // To the CTAs from `first` on, a `step` apart; 0 is among one warp's.
  __device__ __forceinline__ void send(int i, const Map<V>& m, uint32_t first, uint32_t step) const {
    const int lane = threadIdx.x & 31, k = i % kBuffers;
    const uint32_t bar = bars + 8 * k;
    if (first == 0 && lane == 0) umma::mbar_expect_tx(bar, size * 32 * sizeof(Map<V>));
    const uint32_t mine = umma::smem_u32(&slots[k * size + rank][lane]);
    for (uint32_t r = first; r < size; r += step) {
      const uint32_t to = pair::map_to(mine, r), on = pair::map_to(bar, r);
      if constexpr (V == 1)
        asm volatile(
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(to),
            "r"(__float_as_uint(m.p[0])), "r"(__float_as_uint(m.e[0])), "r"(on)
            : "memory");
      else
        asm volatile(
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
            "r"(__float_as_uint(m.p[0])), "r"(__float_as_uint(m.p[1])),
            "r"(__float_as_uint(m.e[0])), "r"(__float_as_uint(m.e[1])), "r"(on)
            : "memory");
    }
  }
  __device__ __forceinline__ bool wait(int i) const {
    return pair::mbar_wait(bars + 8 * (i % kBuffers), (i / kBuffers) & 1, kWaitNs);
  }
  // The maps of the last rounds, which nothing may have waited for, have landed.
  __device__ __forceinline__ void drain(int rounds) const {
    for (int i = rounds > kBuffers ? rounds - kBuffers : 0; i < rounds; ++i) wait(i);
  }
  // x through the tiles of round i; `in` is what enters this CTA's.
  template <int N>
  __device__ __forceinline__ void some(const Map<V> (*at)[32], uint32_t r, float (&x)[V],
                                       float (&in)[V]) const {
    Map<V> m[N];
#pragma unroll
    for (int j = 0; j < N; ++j) m[j] = at[r + j][threadIdx.x & 31];
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) in[v] = r + j == rank ? x[v] : in[v];
      m[j].through(x);
    }
  }
  __device__ __forceinline__ void pass(int i, float (&x)[V], float (&in)[V]) const {
    const Map<V>(*at)[32] = slots + (i % kBuffers) * size;
    if (size == 2) return some<2>(at, 0, x, in);
    if (size == 4) return some<4>(at, 0, x, in);
    for (uint32_t r = 0; r < size; r += 8) some<8>(at, r, x, in);
  }
};

// What the warps of a CTA and the two beside them that deal with the cluster hand
// over: every warp's map of a round, and the state that enters the CTA's tile.  Two barriers of each are enough: a warp gives the map of round i + 2
// after it has taken the state of round i, which both helpers' parts in round i precede.
template <int V>
struct Handover {
  uint32_t bars;
  float (*state)[32][V];  // [2][32]
  __device__ __forceinline__ void init(int warps) const {
    if (threadIdx.x == 0)
      for (int k = 0; k < 2; ++k) {
        umma::mbar_init(bars + 8 * k, warps);
        umma::mbar_init(bars + 16 + 8 * k, 1);
      }
  }
  __device__ __forceinline__ void arrive(uint32_t bar) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) umma::mbar_arrive(bar);
  }
  __device__ __forceinline__ void map_given(int i) const { arrive(bars + 8 * (i & 1)); }
  __device__ __forceinline__ bool maps(int i) const { return wait_here(bars + 8 * (i & 1), (i >> 1) & 1); }
  __device__ __forceinline__ void publish(int i, const float (&x)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) state[i & 1][threadIdx.x & 31][v] = x[v];
    arrive(bars + 16 + 8 * (i & 1));
  }
  __device__ __forceinline__ bool take(int i, float (&x)[V]) const {
    const bool ok = wait_here(bars + 16 + 8 * (i & 1), (i >> 1) & 1);
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = state[i & 1][threadIdx.x & 31][v];
    return ok;
  }
};

// Where a CTA stands.
template <typename T>
struct Place {
  static constexpr int V = Of<T>::kVec;
  int warp, lane, x0, len, seqlen;
  uint32_t rank, size;
  int64_t b, d;  // batch row; the lane's first channel (0 past the last)
  bool on;       // d < dim
  __device__ __forceinline__ Place(const RecurParams& p, uint32_t n) : size(n) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    const int64_t groups = (p.dim * sizeof(T) + kRow - 1) / kRow;
    const int64_t unit = blockIdx.x / n;
    rank = blockIdx.x - static_cast<uint32_t>(unit) * n;
    b = unit / groups;
    x0 = static_cast<int>(unit - b * groups) * 32 * V;
    if (p.valid_len && p.batch <= 32) b = recur::by_length(p.valid_len, p.batch, p.seqlen, b);
    d = x0 + lane * V;
    on = d < p.dim;
    if (!on) d = 0;
    len = static_cast<int>(recur::valid_of(p.valid_len, b, p.seqlen));
    seqlen = static_cast<int>(p.seqlen);
  }
};

// Shared memory: barriers, maps, NO boxes per warp on their way out, the slots of NT
// tensors' tiles, and the cluster's buffers.
template <typename T, int W, int NT, int NO, int MAPS>
struct Mem {
  static constexpr int V = Of<T>::kVec;
  static constexpr uint32_t kBars = 0, kShared = 8 * kSlots;  // the cluster's barriers
  static constexpr uint32_t kHand = kShared + 8 * kBuffers, kState = 128;  // the helpers'
  static constexpr uint32_t kMaps = kState + 2 * 32 * V * sizeof(float);
  static constexpr uint32_t kOut = kMaps + MAPS;
  static constexpr uint32_t kIn = kOut + NO * W * kBox;
  static constexpr uint32_t kTiles = kIn + kSlots * NT * W * kBox;
  static_assert(kHand + 32 <= kState && MAPS % 128 == 0, "layout");
  static uint32_t bytes(int size) {
    const uint32_t tile = 32 * static_cast<uint32_t>(sizeof(Map<V>));
    return kTiles + (size > 1 ? kBuffers * size * tile : 0) + 128;
  }
};

// ---- forward ------------------------------------------------------------------
constexpr int kFwdMaps = 4;  // rounds whose warps' maps are kept
template <typename T, int W>
using FwdMem = Mem<T, W, 2, 1, kFwdMaps * W * 32 * sizeof(Map<Of<T>::kVec>)>;

// A warp's steps of a tile: a and b v.
template <int V> struct Steps { float a[kSteps][V], u[kSteps][V]; };

// Reads the rows at `at` (of the gate; the value's are `far` bytes on) and folds them.
template <typename T, int V>
__device__ __forceinline__ Map<V> fold(Steps<V>& t, uint32_t at, uint32_t far, int left,
                                       const recur::Floor<V>& floor) {
  Fold<V> m;
  if (left <= 0) return m.map();
  if (left < kSteps) {  // closed gates past the valid steps
    for (int s = left; s < kSteps; ++s) {
      sts(at + s * kRow, closed<T>());
      sts(at + far + s * kRow, 0u);
    }
    umma::fence_smem_to_async();
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    float g[V], open[V], b[V];
    unpack(lds(at + s * kRow), g);
    unpack(lds(at + far + s * kRow), t.u[s]);
    recur::gates<T>(g, floor, open, b, t.a[s]);
    vmul<V>(t.u[s], b, t.u[s]);
    m.then(t.a[s], b, t.u[s]);
  }
  return m.map();
}

// CLUSTER: a cluster shares the time.  With one channel per lane the next round's tile
// is folded while the maps of this one travel, and two warps beside the others take the
// exchange: one loads tiles and sends the CTA's map, one takes the maps of all and hands
// the state that enters on (fp32 1 x 65536 x 256: 49 us, with the exchange in all warps
// 59 us).  With two channels that takes registers that other CTAs hide the way with
// (bf16 2 x 32768 x 2048 141 us with the two warps, 132 us without).
template <typename T, bool CLUSTER>
constexpr int kHelpers = CLUSTER && Of<T>::kVec == 1 ? 2 : 0;

template <typename T, int W, bool CLUSTER>
__global__ void __launch_bounds__((W + kHelpers<T, CLUSTER>) * 32, W == 8 ? 2 : 4)
    recur_fwd_tma_kernel(const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap mv,
                         const __grid_constant__ CUtensorMap my, const RecurParams p, const TmaArgs a) {
  using M = FwdMem<T, W>;
  constexpr int V = M::V, kTile = W * kSteps;
  extern __shared__ unsigned char raw[];
  const uint32_t raw_at = umma::smem_u32(raw), pad = (128u - raw_at % 128u) % 128u;
  unsigned char* mem = raw + pad;
  const uint32_t base = raw_at + pad;
  Map<V>(*maps)[W][32] = reinterpret_cast<Map<V>(*)[W][32]>(mem + M::kMaps);
  constexpr bool kAhead = kHelpers<T, CLUSTER> > 0;
  Ring<W, 2> ring = {base + M::kIn, base + M::kBars, 0, 0};
  const Place<T> at(p, CLUSTER ? a.size : 1);
  const int warp = at.warp, lane = at.lane, len = at.len, size = static_cast<int>(at.size);
  const Exchange<V> cluster = {reinterpret_cast<Map<V>(*)[32]>(mem + M::kTiles),
                               base + M::kShared, at.rank, at.size};
  const Handover<V> hand = {base + M::kHand, reinterpret_cast<float(*)[32][V]>(mem + M::kState)};
  const int live = (len + kTile - 1) / kTile, rounds = (live + size - 1) / size;
  const CUtensorMap* const in_map[2] = {&mg, &mv};
  const bool last[2] = {a.gate_last, a.value_last};
  const auto tile_of = [&](int i) { return i * size + static_cast<int>(at.rank); };
  const auto load = [&](int i, int slot) {  // the tile of round i
    if (i < rounds && tile_of(i) < live)
      ring.load(slot, in_map, last, at.x0, tile_of(i) * kTile, static_cast<int>(at.b));
  };
  ring.init();
  if (CLUSTER) cluster.init();
  if (kAhead) hand.init(W);
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 0; i < kSlots; ++i) load(i, i);
  recur::Floor<V> floor;
  float x[V];  // the state that enters the round
#pragma unroll
  for (int v = 0; v < V; ++v) {
    floor.set(v, p.floor ? __ldg(p.floor + at.d + v) : 0.f);
    // before the first barrier, and not as a constant: out_final may be the same memory
    x[v] = p.state0 && (!kAhead || warp > W) ? p.state0[at.b * p.dim + at.d + v] : 0.f;
  }
  float* states = p.states
      ? p.states + at.b * ((p.seqlen + kRecurChunk - 1) / kRecurChunk) * p.dim + at.d
      : nullptr;
  const uint32_t out = base + M::kOut + warp * kBox;
  bool bad = false;
  if (CLUSTER) pair::cluster_sync();  // all of the cluster has started, its barriers too

  // past the valid steps: tiles that no round has covered
  const int64_t rest = static_cast<int64_t>(tile_of(rounds)) * kTile;
  const auto ends = [&]() {  // one warp per CTA; x: what leaves the valid steps
    if (!at.on) return;
    if (p.out_final && at.rank == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.out_final[at.b * p.dim + at.d + v] = x[v];
    }
    if (!states) return;
    for (int64_t t = rest; t < at.seqlen; t += static_cast<int64_t>(size) * kTile)
      for (int64_t c = t; c < t + kTile && c < at.seqlen; c += kRecurChunk)
#pragma unroll
        for (int v = 0; v < V; ++v) states[c / kRecurChunk * p.dim + v] = x[v];
  };
  const auto of_tile = [&](int i) {
    Fold<V> all;
#pragma unroll
    for (int w = 0; w < W; ++w) all.then(maps[i % kFwdMaps][w][lane]);
    return all.map();
  };
  // folds the tile of round i and publishes its map
  const auto first_half = [&](Steps<V>& t, int i) {
    if (tile_of(i) < live && !bad && !ring.wait()) bad = true;
    maps[i % kFwdMaps][warp][lane] =
        fold<T, V>(t, ring.slot() + warp * kBox + lane * 4, W * kBox,
                   len - tile_of(i) * kTile - warp * kSteps, floor);
    if (kAhead) {
      hand.map_given(i);
    } else {
      __syncthreads();
      if (threadIdx.x == 0) load(i + kSlots, ring.at);
      if (CLUSTER && warp < size) cluster.send(i, of_tile(i), warp, W);
    }
    ring.next();
  };
  if (kAhead && warp == W) {
    for (int i = 0; i < rounds; ++i) {
      if (!bad && !hand.maps(i)) bad = true;
      if (lane == 0) load(i + kSlots, i % kSlots);
      cluster.send(i, of_tile(i), 0, 1);
    }
  } else if (kAhead && warp > W) {
    for (int i = 0; i < rounds; ++i) {
      float in[V];
      if (!bad && !(hand.maps(i) && cluster.wait(i))) bad = true;
      cluster.pass(i, x, in);
      hand.publish(i, in);
    }
    ends();
  } else {
    Steps<V> now, next;
    if (kAhead && rounds > 0) first_half(now, 0);
    for (int i = 0; i < rounds; ++i) {
      if (!kAhead) first_half(now, i);
      if (kAhead && i + 1 < rounds) first_half(next, i + 1);
      float in[V];
      if (CLUSTER) {
        if (kAhead) {
          if (!bad && !hand.take(i, in)) bad = true;
        } else {
          if (!bad && !cluster.wait(i)) bad = true;
          cluster.pass(i, x, in);
        }
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
          if (w < warp) maps[i % kFwdMaps][w][lane].through(in);
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (w == warp) {
#pragma unroll
            for (int v = 0; v < V; ++v) in[v] = x[v];
          }
          maps[i % kFwdMaps][w][lane].through(x);
        }
      }
      const int t0 = tile_of(i) * kTile + warp * kSteps, left = len - t0;
      if (t0 < at.seqlen) {
        if (states && at.on && t0 % kRecurChunk == 0) {
#pragma unroll
          for (int v = 0; v < V; ++v) states[t0 / kRecurChunk * p.dim + v] = in[v];
        }
        boxes_free();
        if (left > 0) {
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            vfma<V>(in, now.a[s], in, now.u[s]);
            sts(out + s * kRow + lane * 4, pack(in));
          }
        }
        if (left < kSteps) {
          for (int s = left < 0 ? 0 : left; s < kSteps; ++s) sts(out + s * kRow + lane * 4, 0u);
        }
        umma::fence_smem_to_async();
        __syncwarp();
        if (lane == 0) {
          store_box(&my, out, at.x0, t0, static_cast<int>(at.b));
          commit_stores();
        }
      }
      if (kAhead) now = next;
    }
    if (!kAhead && warp == 0) ends();
    if (rest < at.seqlen) {
      boxes_free();
      for (int s = 0; s < kSteps; ++s) sts(out + s * kRow + lane * 4, 0u);
      umma::fence_smem_to_async();
      __syncwarp();
      if (lane == 0) {
        for (int64_t t = rest + warp * kSteps; t < at.seqlen; t += static_cast<int64_t>(size) * kTile) {
          store_box(&my, out, at.x0, static_cast<int>(t), static_cast<int>(at.b));
          commit_stores();
        }
      }
    }
    boxes_free();
  }
  if (bad) {
    // tiles and maps that were not waited for land before the CTA ends
    for (int i = rounds > kSlots ? rounds - kSlots : 0; i < rounds; ++i)
      if (tile_of(i) < live) ring.drain(i);
    if (CLUSTER) cluster.drain(rounds);
    atomicOr(a.err, kErrRecurWait);
  }
  if (CLUSTER) pair::cluster_sync();  // no map is on its way to a CTA that has ended
}

// ---- backward -----------------------------------------------------------------
template <typename T, int W>
using BwdMem = Mem<T, W, 3, 2, 2 * W * 32 * (sizeof(Map<Of<T>::kVec>) + 4 * Of<T>::kVec)>;

template <typename T, int W, bool CLUSTER>
__global__ void __launch_bounds__(W * 32)
    recur_bwd_tma_kernel(const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap mv,
                         const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mdg,
                         const __grid_constant__ CUtensorMap mdv, const RecurBwdParams q,
                         const TmaArgs a) {
  using M = BwdMem<T, W>;
  constexpr int V = M::V, kTile = W * kSteps;
  const RecurParams& p = q.fwd;
  extern __shared__ unsigned char raw[];
  const uint32_t raw_at = umma::smem_u32(raw), pad = (128u - raw_at % 128u) % 128u;
  unsigned char* mem = raw + pad;
  const uint32_t base = raw_at + pad;
  Map<V>(*past)[W][32] = reinterpret_cast<Map<V>(*)[W][32]>(mem + M::kMaps);
  float(*coming)[W][32][V] = reinterpret_cast<float(*)[W][32][V]>(past + 2);
  Ring<W, 3> ring = {base + M::kIn, base + M::kBars, 0, 0};
  const Place<T> at(p, CLUSTER ? a.size : 1);
  const int warp = at.warp, lane = at.lane, len = at.len, size = static_cast<int>(at.size);
  const Exchange<V> cluster = {reinterpret_cast<Map<V>(*)[32]>(mem + M::kTiles),
                               base + M::kShared, at.rank, at.size};
  const int live = (len + kTile - 1) / kTile, rounds = (live + size - 1) / size;
  const CUtensorMap* const in_map[3] = {&mg, &mv, &my};
  const bool last[3] = {a.gate_last, a.value_last, false};
  const auto tile_of = [&](int i) { return live - 1 - i * size - static_cast<int>(at.rank); };
  const auto load = [&](int i, int slot) {
    if (i < rounds && tile_of(i) >= 0)
      ring.load(slot, in_map, last, at.x0, tile_of(i) * kTile, static_cast<int>(at.b));
  };
  ring.init();
  if (CLUSTER) cluster.init();
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 0; i < kSlots; ++i) load(i, i);
  recur::Floor<V> floor;
  float m[V], dfloor[V];  // m: a l of the step after the round's last; half of dfloor
#pragma unroll
  for (int v = 0; v < V; ++v) {
    floor.set(v, p.floor ? __ldg(p.floor + at.d + v) : 0.f);
    m[v] = q.dfinal ? __ldg(q.dfinal + at.b * p.dim + at.d + v) : 0.f;
    dfloor[v] = 0.f;
  }
  const float* states =
      q.states + at.b * ((p.seqlen + kRecurChunk - 1) / kRecurChunk) * p.dim + at.d;
  const uint32_t out = base + M::kOut + warp * 2 * kBox;
  bool bad = false;
  if (CLUSTER) pair::cluster_sync();  // all of the cluster has started, its barriers too
  for (int i = 0; i < rounds; ++i) {
    const int tile = tile_of(i);
    const bool here = tile >= 0;  // else none is left
    const int t0 = tile * kTile + warp * kSteps;
    const int left = here ? len - t0 : 0;
    const uint32_t row = ring.slot() + warp * kBox + lane * 4;
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = here ? __ldg(states + static_cast<int64_t>(tile) * (kTile / kRecurChunk) * p.dim + v) : 0.f;
    if (here && !bad && !ring.wait()) bad = true;
    if (left > 0 && left < kSteps) {
      for (int s = left; s < kSteps; ++s) {
        sts(row + s * kRow, closed<T>());
        sts(row + W * kBox + s * kRow, 0u);
        sts(row + 2 * W * kBox + s * kRow, 0u);
      }
      umma::fence_smem_to_async();
    }
    // dy stays in its own words: with two channels per lane registers are short
    float open[kSteps][V], hold[kSteps][V], decay[kSteps][V], u[kSteps][V];
    uint32_t l[kSteps];
    Fold<V> fold;
    float ml[V];
#pragma unroll
    for (int v = 0; v < V; ++v) ml[v] = 0.f;
    if (left > 0) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        float e[V], b[V];
        unpack(lds(row + s * kRow), e);
        unpack(lds(row + W * kBox + s * kRow), u[s]);
        l[s] = lds(row + 2 * W * kBox + s * kRow);
        recur::gates<T>(e, floor, open[s], b, decay[s]);
#pragma unroll
        for (int v = 0; v < V; ++v) hold[s][v] = recur::holding(e[v], open[s][v]);
        float in[V];
        vmul<V>(in, b, u[s]);
        fold.then(decay[s], b, in);
      }
#pragma unroll
      for (int s = kSteps - 1; s >= 0; --s) {
        float lam[V];
        unpack(l[s], lam);
        vadd<V>(lam, ml, lam);
        vmul<V>(ml, decay[s], lam);
      }
    }
    const int k = i & 1;
    past[k][warp][lane] = fold.map();
#pragma unroll
    for (int v = 0; v < V; ++v) coming[k][warp][lane][v] = ml[v];
    __syncthreads();
    if (threadIdx.x == 0) load(i + kSlots, ring.at);
    ring.next();
    const auto back = [&](int w) {  // the warp's map of what goes back
      Map<V> r;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        r.p[v] = past[k][w][lane].p[v];
        r.e[v] = coming[k][w][lane][v];
      }
      return r;
    };
    float mi[V];
    if (CLUSTER) {
      if (warp < size) {
        Fold<V> all;
#pragma unroll
        for (int w = W - 1; w >= 0; --w) all.then(back(w));
        cluster.send(i, all.map(), warp, W);
      }
      if (!bad && !cluster.wait(i)) bad = true;
      cluster.pass(i, m, mi);
#pragma unroll
      for (int w = W - 1; w > 0; --w)
        if (w > warp) back(w).through(mi);
    } else {
#pragma unroll
      for (int w = W - 1; w >= 0; --w) {
        if (w == warp) {
#pragma unroll
          for (int v = 0; v < V; ++v) mi[v] = m[v];
        }
        back(w).through(m);
      }
    }
#pragma unroll
    for (int w = 0; w < W - 1; ++w)
      if (w < warp) past[k][w][lane].through(h);
    boxes_free();
    if (left > 0) {
      // the distance of the state before a step to its value, in the value's place
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        float b[V];
        vmul<V>(b, floor.half, open[s]);
        vmul<V>(b, b, u[s]);
        minus<V>(u[s], h, u[s]);
        vfma<V>(h, decay[s], h, b);
      }
      float some[V];
#pragma unroll
      for (int v = 0; v < V; ++v) some[v] = 0.f;
#pragma unroll
      for (int s = kSteps - 1; s >= 0; --s) {
        float b[V], lam[V], o[V];
        unpack(l[s], lam);
        vmul<V>(b, floor.half, open[s]);
        vadd<V>(lam, mi, lam);
        vmul<V>(mi, decay[s], lam);
        vmul<V>(o, b, lam);
        sts(out + s * kRow + lane * 4, pack(o));
        vmul<V>(lam, lam, u[s]);
        vfma<V>(some, lam, open[s], some);
        vmul<V>(b, b, hold[s]);
        vmul<V>(o, lam, b);
        sts(out + kBox + s * kRow + lane * 4, pack(o));
      }
#pragma unroll
      for (int v = 0; v < V; ++v) dfloor[v] += some[v];
    }
    if (left < kSteps) {
      for (int s = left < 0 ? 0 : left; s < kSteps; ++s) {
        sts(out + s * kRow + lane * 4, 0u);
        sts(out + kBox + s * kRow + lane * 4, 0u);
      }
    }
    umma::fence_smem_to_async();
    __syncwarp();
    if (lane == 0 && here && t0 < at.seqlen) {
      store_box(&mdv, out, at.x0, t0, static_cast<int>(at.b));
      store_box(&mdg, out + kBox, at.x0, t0, static_cast<int>(at.b));
      commit_stores();
    }
  }
  if (q.dstate0 && at.rank == 0 && warp == 0 && at.on) {
#pragma unroll
    for (int v = 0; v < V; ++v) q.dstate0[at.b * p.dim + at.d + v] = m[v];
  }
  const int64_t rest = static_cast<int64_t>(live + static_cast<int>(at.rank)) * kTile;
  if (rest < at.seqlen) {
    boxes_free();
    for (int s = 0; s < kSteps; ++s) sts(out + s * kRow + lane * 4, 0u);
    umma::fence_smem_to_async();
    __syncwarp();
    if (lane == 0) {
      for (int64_t t = rest + warp * kSteps; t < at.seqlen; t += static_cast<int64_t>(size) * kTile) {
        store_box(&mdv, out, at.x0, static_cast<int>(t), static_cast<int>(at.b));
        store_box(&mdg, out, at.x0, static_cast<int>(t), static_cast<int>(at.b));
        commit_stores();
      }
    }
  }
  boxes_free();
  if (q.dfloor) {
    __syncthreads();
    float* sums = &coming[0][0][0][0];
#pragma unroll
    for (int v = 0; v < V; ++v) sums[(warp * 32 + lane) * V + v] = dfloor[v];
    __syncthreads();
    if (warp == 0 && at.on) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float t = 0.f;
        for (int w = 0; w < W; ++w) t += sums[(w * 32 + lane) * V + v];
        q.partial[(at.b * size + at.rank) * p.dim + at.d + v] = 0.5f * t;
      }
    }
  }
  if (bad) {
    // as in the forward
    for (int i = rounds > kSlots ? rounds - kSlots : 0; i < rounds; ++i)
      if (tile_of(i) >= 0) ring.drain(i);
    if (CLUSTER) cluster.drain(rounds);
    atomicOr(a.err, kErrRecurWait);
  }
  if (CLUSTER) pair::cluster_sync();  // no map is on its way to a CTA that has ended
}

// The axes in the order of their strides, as a tensor map wants them: each stride
// a multiple of the one before.
Axes axes_of(const RecurParams& p, int64_t batch_stride, int64_t step_stride) {
  Axes a;
  if (p.batch == 1) {
    a.time_last = false;
    a.inner = p.seqlen > 1 ? step_stride : p.dim;
    a.outer = a.inner * p.seqlen;
  } else if (p.seqlen == 1) {
    a.time_last = true;
    a.inner = batch_stride;
    a.outer = batch_stride * p.batch;
  } else {
    a.time_last = batch_stride < step_stride;
    a.inner = a.time_last ? batch_stride : step_stride;
    a.outer = a.time_last ? step_stride : batch_stride;
  }
  a.ok = a.inner >= p.dim && a.outer % a.inner == 0;
  return a;
}

bool map_of(CUtensorMap* m, bool bf16, const void* base, const RecurParams& p, const Axes& a, int rows) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const unsigned es = bf16 ? 2 : 4;
  const cuuint64_t time = static_cast<cuuint64_t>(p.seqlen), batch = static_cast<cuuint64_t>(p.batch);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.dim), a.time_last ? batch : time,
                              a.time_last ? time : batch};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.inner) * es,
                                 static_cast<cuuint64_t>(a.outer) * es};
  const cuuint32_t n = static_cast<cuuint32_t>(rows);
  const cuuint32_t box[3] = {kRow / es, a.time_last ? 1 : n, a.time_last ? n : 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Axes dense(const RecurParams& p) { return {true, false, p.dim, p.seqlen * p.dim}; }

bool fits(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int64_t units_of(const RecurParams& p, bool bf16) {
  const int64_t lanes = bf16 ? 64 : 32;
  return p.batch * ((p.dim + lanes - 1) / lanes);
}

template <auto KERNEL, typename MEM>
cudaError_t allow(int sizes) {
  cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(MEM::bytes(sizes)));
  if (e == cudaSuccess && sizes > kPortableCluster)
    e = allow_large_clusters(reinterpret_cast<const void*>(KERNEL));
  return e;
}

// CTAs that share the time of a channel group: doubled while all clusters run at
// once and every CTA has a tile.  (bf16 2 x 32768 x 2048, 64 groups, forward: 2 CTAs
// 195 us, 4 135 us, 8, half of them waiting for the others to end, 220 us.)
template <auto KERNEL, typename MEM, int W, int THREADS>
int cluster_of(const RecurParams& p, int64_t units) {
  const int64_t tiles = (p.seqlen + W * kSteps - 1) / (W * kSteps);
  int i = 0;
  while (i < 4 && (int64_t(2) << i) <= tiles &&
         units <= resident_clusters<KERNEL>(i + 1, THREADS, MEM::bytes(2 << i)))
    ++i;
  return 1 << i;
}

template <auto KERNEL, typename MEM, int THREADS, typename... A>
cudaError_t go(const RecurParams& p, bool bf16, int size, cudaStream_t s, const A&... args) {
  const cudaError_t e = allow<KERNEL, MEM>(size > 1 ? kMaxCluster : 1);
  if (e != cudaSuccess) return e;
  const ClusterLaunch l(units_of(p, bf16), size, THREADS, MEM::bytes(size), s);
  return cudaLaunchKernelEx(&l.cfg, KERNEL, args...);
}

// Warps per CTA.  Forward: 8 (fp32 8 x 4096 x 1024 62 us, with 4 68 us; bf16 40 and
// 55 us).  Backward: 8 with two channels per lane and 4 otherwise (bf16 59 and 73 us,
// fp32 106 and 101 us), but 4 in clusters (bf16 2 x 32768 x 2048 235 and 271 us).
// Short sequences take as few warps as hold them (bf16 1024 x 16 x 768 with 8 and 8:
// 100 and 249 us).
template <typename T, int W>
cudaError_t fwd(const RecurParams& p, unsigned* err, cudaStream_t s) {
  constexpr bool bf16 = sizeof(T) == 2;
  using M = FwdMem<T, W>;
  const Axes g = axes_of(p, p.gate_batch, p.gate_step), v = axes_of(p, p.value_batch, p.value_step);
  CUtensorMap mg, mv, my;
  if (!map_of(&mg, bf16, p.gate, p, g, W * kSteps) || !map_of(&mv, bf16, p.value, p, v, W * kSteps) ||
      !map_of(&my, bf16, p.y, p, dense(p), kSteps))
    return cudaErrorInvalidValue;
  TmaArgs a = {1, g.time_last, v.time_last, err};
  if constexpr (W == 8) {
    constexpr auto shared = recur_fwd_tma_kernel<T, W, true>;
    const cudaError_t e = allow<shared, M>(kMaxCluster);
    if (e != cudaSuccess) return e;
    constexpr int threads = (W + kHelpers<T, true>) * 32;
    const int size = cluster_of<shared, M, W, threads>(p, units_of(p, bf16));
    a.size = static_cast<uint32_t>(size);
    if (size > 1) return go<shared, M, threads>(p, bf16, size, s, mg, mv, my, p, a);
  }
  return go<recur_fwd_tma_kernel<T, W, false>, M, W * 32>(p, bf16, 1, s, mg, mv, my, p, a);
}

template <typename T>
cudaError_t fwd_any(const RecurParams& p, unsigned* err, cudaStream_t s) {
  if (p.seqlen <= kSteps) return fwd<T, 1>(p, err, s);
  return p.seqlen <= 4 * kSteps ? fwd<T, 4>(p, err, s) : fwd<T, 8>(p, err, s);
}

template <typename T, int W, bool CLUSTER>
cudaError_t bwd(const RecurBwdParams& q, int size, unsigned* err, cudaStream_t s) {
  constexpr bool bf16 = sizeof(T) == 2;
  const RecurParams& p = q.fwd;
  const Axes g = axes_of(p, p.gate_batch, p.gate_step), v = axes_of(p, p.value_batch, p.value_step);
  CUtensorMap mg, mv, my, mdg, mdv;
  if (!map_of(&mg, bf16, p.gate, p, g, W * kSteps) || !map_of(&mv, bf16, p.value, p, v, W * kSteps) ||
      !map_of(&my, bf16, q.dy, p, dense(p), W * kSteps) ||
      !map_of(&mdg, bf16, q.dgate, p, dense(p), kSteps) ||
      !map_of(&mdv, bf16, q.dvalue, p, dense(p), kSteps))
    return cudaErrorInvalidValue;
  const TmaArgs a = {static_cast<uint32_t>(size), g.time_last, v.time_last, err};
  return go<recur_bwd_tma_kernel<T, W, CLUSTER>, BwdMem<T, W>, W * 32>(p, bf16, size, s, mg, mv, my, mdg,
                                                                  mdv, q, a);
}

template <typename T>
cudaError_t bwd_any(const RecurBwdParams& q, unsigned* err, int* size, cudaStream_t s) {
  constexpr bool bf16 = sizeof(T) == 2;
  *size = 1;
  if (q.fwd.seqlen <= kSteps) return bwd<T, 1, false>(q, 1, err, s);
  if (q.fwd.seqlen <= 4 * kSteps) return bwd<T, 4, false>(q, 1, err, s);
  const int64_t units = units_of(q.fwd, bf16);
  constexpr auto shared = recur_bwd_tma_kernel<T, 4, true>;
  const cudaError_t e = allow<shared, BwdMem<T, 4>>(kMaxCluster);
  if (e != cudaSuccess) return e;
  // With two channels per lane one CTA per group from half of the SMs on (bf16 5 x 4096
  // x 1024, 80 groups: 55 us, in clusters of two 59 us; fp32 4 x 4096 x 1024, 128
  // groups: 68 and 56 us).
  *size = bf16 && 2 * units >= kSms ? 1 : cluster_of<shared, BwdMem<T, 4>, 4, 128>(q.fwd, units);
  if (*size > 1) return bwd<T, 4, true>(q, *size, err, s);
  return bwd<T, bf16 ? 8 : 4, false>(q, 1, err, s);
}

}  // namespace

bool recur_tma_ok(const RecurParams& p, bool bf16) {
  const int64_t es = bf16 ? 2 : 4;
  const int64_t lim = int64_t(1) << 30, far = int64_t(1) << 38;
  for (const Axes& a : {axes_of(p, p.gate_batch, p.gate_step), axes_of(p, p.value_batch, p.value_step)})
    if (!a.ok || (a.inner * es) % 16 != 0 || a.outer >= far) return false;
  return (p.dim * es) % 16 == 0 && p.dim <= lim && p.seqlen <= lim && p.batch <= lim &&
         p.seqlen * p.dim < far && fits(p.gate) && fits(p.value) && fits(p.y);
}
bool recur_bwd_tma_ok(const RecurBwdParams& q, bool bf16) {
  return recur_tma_ok(q.fwd, bf16) && fits(q.dy) && fits(q.dgate) && fits(q.dvalue);
}

cudaError_t launch_recur_fwd_tma(const RecurParams& p, bool bf16, unsigned* err, cudaStream_t s) {
  return bf16 ? fwd_any<__nv_bfloat16>(p, err, s) : fwd_any<float>(p, err, s);
}

cudaError_t launch_recur_bwd_tma(const RecurBwdParams& q, bool bf16, unsigned* err, int* parts,
                                 cudaStream_t s) {
  return bf16 ? bwd_any<__nv_bfloat16>(q, err, parts, s) : bwd_any<float>(q, err, parts, s);
}

}  // namespace ssm
