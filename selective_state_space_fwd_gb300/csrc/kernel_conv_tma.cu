// kernel_conv_tma.cu -- the short causal convolution (conv.cuh has the
// formulas) with its rows staged by TMA, for tensors whose rows start on 16-byte
// boundaries and whose strides a tensor map takes (axes_of).
//
// Work split: a warp owns a slab of 256 bytes of channels (8 bytes per lane) and
// walks pieces of sequences, a piece after another: boxes of kRows steps x 256
// bytes arrive in the warp's own ring of stages, so that the copies of the next
// boxes are in flight while a box is filtered, and no CTA barrier is needed.  A
// piece of tc steps reads the width - 1 steps before it again (and in the
// backward the width - 1 after it), which its first box covers: steps before
// the sequence arrive as zeros.  tc makes the steps of a piece whole boxes.
//
// Bound by HBM.  Measured on GB300, width 4 with silu: fp32 8 x 4096 x 1024
// forward 47.1 us, 5.7 TB/s, forward and backward 120 us, 5.6 TB/s, with x
// time-major 119 us (one launch alone, ncu: 40.0 and 62.0 us, 6.7 and 6.5 TB/s);
// bf16 8 x 4096 x 1024 forward 23.4 us, 5.7 TB/s; bf16 prompts 32 x 2048 x 1536
// with valid lengths 61 us.
#include <cuda.h>

#include <type_traits>

#include "conv.cuh"
#include "pdl.cuh"
#include "tma_map.h"
#include "umma_pair.cuh"

namespace ssm {
namespace {

constexpr int kSms = 152;
constexpr int kRows = 16;           // steps per box
constexpr int kWarps = 4;           // warps per CTA
constexpr uint32_t kRowBytes = 256;  // of a slab
constexpr uint32_t kBoxBytes = kRows * kRowBytes;
constexpr uint64_t kWaitNs = 2000000000ull;

// Stages per warp and CTAs per SM.  Measured on bf16 8 x 4096 x 1024 (forward)
// and 8 x 2048 x 2048 (training step): boxes of 16 steps 23.7 and 64.5 us, of 8
// steps 26.0 and 69.6 us; in the backward 3 stages and 2 CTAs 68.0 us.
constexpr int kFwdStages = 2, kFwdCtas = 6;
constexpr int kBwdStages = 2, kBwdCtas = 3;
constexpr uint32_t kFwdSmem = kWarps * kFwdStages * kBoxBytes;
static_assert(kFwdSmem <= 48 * 1024, "within the default limit");
constexpr uint32_t kBwdSmem = kWarps * kBwdStages * 2 * kBoxBytes;

struct Pieces {
  int tc;           // steps per piece
  int segs;         // pieces per batch row
  int slabs;        // slabs of channels
  int64_t items;    // pieces of a slab: batch x segs
  bool time_last;   // x's map has the axes (channel, batch, time), not (channel, time, batch)
};

// One piece of one batch row.
struct Piece {
  int64_t b, t0, vl;
  int n;       // its steps
  int live;    // steps from t0 that are computed: valid ones, with `after` steps past the piece
  int boxes;   // boxes to copy
};

__device__ __forceinline__ Piece piece_at(const ConvParams& p, const Pieces& q, int64_t it, int K,
                                          int after) {
  Piece r;
  // the same stretch of every batch row, then the next: with valid lengths all
  // warps then have about as many live pieces
  const int64_t seg = it / p.batch;
  r.b = it - seg * p.batch;
  r.t0 = seg * q.tc;
  r.vl = conv_valid(p, r.b);
  r.n = static_cast<int>(p.seqlen - r.t0 < q.tc ? p.seqlen - r.t0 : q.tc);
  const int64_t left = r.vl - r.t0;
  r.live = static_cast<int>(left < 0 ? 0 : left < r.n + after ? left : r.n + after);
  r.boxes = r.live > 0 ? (r.live + K - 1 + kRows - 1) / kRows : 0;
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> lds_row(uint32_t addr) {
  Raw<T, VEC> r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(addr));
  return r;
}

// The warp's ring of boxes, filled in the order in which the pieces use them.
// NT tensors (x, or x and dy) per stage.
template <int NT, int STAGES>
struct Ring {
  uint32_t base, bars;
  const CUtensorMap* map[NT];
  int x;                 // first channel of the slab
  int64_t it, step;      // load cursor: piece, and the distance to the warp's next
  Piece piece;
  int box;
  int filled, used;      // boxes issued and consumed

  __device__ __forceinline__ void load(const ConvParams& p, const Pieces& q, int K, int after) {
    while (it < q.items && box >= piece.boxes) {  // the next piece that has boxes
      it += step;
      box = 0;
      if (it < q.items) piece = piece_at(p, q, it, K, after);
    }
    if (it >= q.items) return;
    if ((threadIdx.x & 31) == 0) {
      const int s = filled % STAGES;
      const uint32_t bar = bars + 8 * s;
      umma::mbar_expect_tx(bar, NT * kBoxBytes);
      const int t = static_cast<int>(piece.t0) - (K - 1) + box * kRows;
      const int b = static_cast<int>(piece.b);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const bool swap = i == 0 && q.time_last;
        umma::tma_load_3d(base + (s * NT + i) * kBoxBytes, map[i], x, swap ? b : t, swap ? t : b,
                          bar);
      }
    }
    ++box;
    ++filled;
  }
  // Waits for the next box; false when the wait gave up.
  __device__ __forceinline__ bool wait() {
    return pair::mbar_wait(bars + 8 * (used % STAGES), (used / STAGES) & 1, kWaitNs);
  }
  __device__ __forceinline__ uint32_t at() const {
    return base + (used % STAGES) * NT * kBoxBytes;
  }
  // For a warp that gives up: its copies land before it ends.
  __device__ __forceinline__ void drain() {
    for (; used < filled; ++used) wait();
  }
};

template <typename T, int K>
__global__ void __launch_bounds__(kWarps * 32, kFwdCtas)
    conv_fwd_tma_kernel(const __grid_constant__ CUtensorMap mx, const ConvParams p, const Pieces q,
                        unsigned* err) {
  constexpr int VEC = 8 / sizeof(T);
  extern __shared__ __align__(128) unsigned char ring_mem[];
  __shared__ __align__(8) uint64_t bar_mem[kWarps * kFwdStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slab = blockIdx.x % q.slabs;
  Ring<1, kFwdStages> ring;
  ring.base = umma::smem_u32(ring_mem) + warp * kFwdStages * kBoxBytes;
  ring.bars = umma::smem_u32(bar_mem) + warp * kFwdStages * 8;
  ring.map[0] = &mx;
  ring.x = slab * 32 * VEC;
  ring.it = static_cast<int64_t>(blockIdx.x / q.slabs) * kWarps + warp;
  ring.step = static_cast<int64_t>(gridDim.x / q.slabs) * kWarps;
  ring.box = ring.filled = ring.used = 0;
  if (lane == 0)
    for (int s = 0; s < kFwdStages; ++s) umma::mbar_init(ring.bars + 8 * s, 1);
  __syncwarp();
  const int64_t first = ring.it, step = ring.step;
  if (first < q.items) ring.piece = piece_at(p, q, first, K, 0);
  for (int s = 0; s < kFwdStages; ++s) ring.load(p, q, K, 0);

  const int64_t d0 = ring.x + lane * VEC;
  const bool on = d0 < p.dim;
  float w[K][VEC], bv[VEC];
  load_taps<K, VEC>(p.weight, p.bias, on ? d0 : 0, w, bv);
  bool bad = false;
  for (int64_t it = first; it < q.items && !bad; it += step) {
    const Piece c = piece_at(p, q, it, K, 0);
    T* y = static_cast<T*>(p.y) + (c.b * p.seqlen + c.t0) * p.dim + d0;
    float win[K - 1][VEC];
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
#pragma unroll
      for (int v = 0; v < VEC; ++v) win[k][v] = 0.f;
    // a whole box; the first of a piece starts with the width - 1 steps before it
    auto whole = [&](uint32_t at, auto first_box) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float cur[VEC], pre[VEC];
        widen<VEC>(lds_row<T, VEC>(at + r * kRowBytes), cur);
        if (!first_box.value || r >= K - 1) {
          taps<K, VEC>(w, bv, win, cur, pre);
          if (p.silu) apply_silu<VEC>(pre);
          if (on) store_f<T, VEC>(y, pre);
          y += p.dim;
        }
        push<K, VEC>(win, cur);
      }
    };
    const bool given = c.t0 == 0 && p.state0 != nullptr;  // the steps before are the state's
    for (int j = 0; j < c.boxes; ++j) {
      if (__any_sync(0xffffffffu, !ring.wait())) {
        bad = true;
        break;
      }
      const uint32_t at = ring.at() + lane * 8;
      const int s0 = j * kRows - (K - 1);  // the step of the box's first row, from t0
      if (s0 + kRows <= c.live && j > 0) {
        whole(at, std::false_type());
      } else if (s0 + kRows <= c.live && !given) {
        whole(at, std::true_type());
      } else {
#pragma unroll 1
        for (int r = 0; r < kRows; ++r) {
          const int s = s0 + r;
          if (s >= c.live) break;
          float cur[VEC], pre[VEC];
          if (s < 0 && given && on)
            widen<VEC>(state_row<T, K, VEC>(p.state0, c.b, p.dim, d0, s + K - 1), cur);
          else
            widen<VEC>(lds_row<T, VEC>(at + r * kRowBytes), cur);
          if (s >= 0) {
            taps<K, VEC>(w, bv, win, cur, pre);
            if (p.silu) apply_silu<VEC>(pre);
            if (on) store_f<T, VEC>(y, pre);
            y += p.dim;
          }
          push<K, VEC>(win, cur);
        }
      }
      __syncwarp();  // the box has been read
      ++ring.used;
      ring.load(p, q, K, 0);
    }
    if (bad || !on) continue;
    Raw<T, VEC> z;
    raw_zero<T, VEC>(z);
    for (int s = c.live; s < c.n; ++s, y += p.dim) raw_store<T, VEC>(y, z);
    if (c.t0 == 0 && p.out_final != nullptr) {
      T* fb = static_cast<T*>(p.out_final) + c.b * (K - 1) * p.dim + d0;
      const T* xb = static_cast<const T*>(p.x) + c.b * p.x_batch + d0;
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {
        const int64_t t = c.vl - (K - 1) + k;
        raw_store<T, VEC>(fb + k * p.dim,
                          t >= 0 ? raw_load<T, VEC>(xb + t * p.x_step)
                                 : state_row<T, K, VEC>(p.state0, c.b, p.dim, d0,
                                                        static_cast<int>(t) + K - 1));
      }
    }
  }
  if (bad) {
    if (lane == 0) atomicOr(err, kErrConvWait);
    ring.drain();
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(kWarps * 32, kBwdCtas)
    conv_bwd_tma_kernel(const __grid_constant__ CUtensorMap mx,
                        const __grid_constant__ CUtensorMap mg, const ConvBwdParams bp,
                        const Pieces q, unsigned* err) {
  constexpr int VEC = 8 / sizeof(T);
  const ConvParams& p = bp.fwd;
  extern __shared__ __align__(128) unsigned char ring_mem[];
  __shared__ __align__(8) uint64_t bar_mem[kWarps * kBwdStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slab = blockIdx.x % q.slabs;
  Ring<2, kBwdStages> ring;
  ring.base = umma::smem_u32(ring_mem) + warp * kBwdStages * 2 * kBoxBytes;
  ring.bars = umma::smem_u32(bar_mem) + warp * kBwdStages * 8;
  ring.map[0] = &mx;
  ring.map[1] = &mg;
  ring.x = slab * 32 * VEC;
  ring.it = static_cast<int64_t>(blockIdx.x / q.slabs) * kWarps + warp;
  ring.step = static_cast<int64_t>(gridDim.x / q.slabs) * kWarps;
  ring.box = ring.filled = ring.used = 0;
  if (lane == 0)
    for (int s = 0; s < kBwdStages; ++s) umma::mbar_init(ring.bars + 8 * s, 1);
  __syncwarp();
  const int64_t first = ring.it, step = ring.step;
  if (first < q.items) ring.piece = piece_at(p, q, first, K, K - 1);
  for (int s = 0; s < kBwdStages; ++s) ring.load(p, q, K, K - 1);
  release_next();

  const int64_t d0 = ring.x + lane * VEC;
  const bool on = d0 < p.dim;
  float w[K][VEC], bv[VEC], dw[K][VEC], db[VEC];
  load_taps<K, VEC>(p.weight, p.bias, on ? d0 : 0, w, bv);
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][v] = 0.f;
  }
  bool bad = false;
  for (int64_t it = first; it < q.items && !bad; it += step) {
    const Piece c = piece_at(p, q, it, K, K - 1);
    // dx of step s - (K - 1) is complete, and written, at step s
    T* o = static_cast<T*>(bp.dx) + (c.b * p.seqlen + c.t0) * p.dim + d0;
    T* state = c.t0 == 0 && bp.dstate0
                   ? static_cast<T*>(bp.dstate0) + c.b * (K - 1) * p.dim + d0
                   : nullptr;
    float win[K - 1][VEC], dp[K - 1][VEC];
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
#pragma unroll
      for (int v = 0; v < VEC; ++v) win[k][v] = dp[k][v] = 0.f;
    auto emit = [&](int s, const float(&g)[VEC]) {
      float a[VEC];
      dx_taps<K, VEC>(w, dp, g, a);
      if (s >= K - 1) {
        if (on) store_f<T, VEC>(o, a);
        o += p.dim;
      } else if (state != nullptr && on) {
        store_f<T, VEC>(state + s * p.dim, a);
      }
      push<K, VEC>(dp, g);
    };
    // a whole box; the first of a piece starts with the width - 1 steps before
    // it, whose dx belongs to the piece before, and the last of a whole piece
    // ends with the width - 1 steps after it, which the next piece sums
    auto whole = [&](uint32_t at, auto first_box, auto last_box) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float cur[VEC], g[VEC], pre[VEC], a[VEC];
        widen<VEC>(lds_row<T, VEC>(at + r * kRowBytes), cur);
        if (!first_box.value || r >= K - 1) {
          widen<VEC>(lds_row<T, VEC>(at + kBoxBytes + r * kRowBytes), g);
          if (p.silu) {
            taps<K, VEC>(w, bv, win, cur, pre);
            apply_dsilu<VEC>(pre, g);
          }
          if (!last_box.value || r < kRows - (K - 1)) add_dw<K, VEC>(dw, db, g, win, cur);
          if (!first_box.value || r >= 2 * (K - 1)) {
            dx_taps<K, VEC>(w, dp, g, a);
            if (on) store_f<T, VEC>(o, a);
            o += p.dim;
          }
          push<K, VEC>(dp, g);
        }
        push<K, VEC>(win, cur);
      }
    };
    const bool given = c.t0 == 0 && p.state0 != nullptr;  // the steps before are the state's
    int s = 0;  // steps done
    for (int j = 0; j < c.boxes; ++j) {
      if (__any_sync(0xffffffffu, !ring.wait())) {
        bad = true;
        break;
      }
      const uint32_t at = ring.at() + lane * 8;
      const int s0 = j * kRows - (K - 1);
      const bool all = s0 + kRows <= c.live;
      if (all && j > 0 && s0 + kRows <= c.n) {
        whole(at, std::false_type(), std::false_type());
        s = s0 + kRows;
      } else if (all && j > 0 && s0 + kRows == c.n + K - 1) {
        whole(at, std::false_type(), std::true_type());
        s = s0 + kRows;
      } else if (all && j == 0 && s0 + kRows <= c.n && !given && state == nullptr) {
        whole(at, std::true_type(), std::false_type());
        s = s0 + kRows;
      } else {
#pragma unroll 1
        for (int r = 0; r < kRows; ++r) {
          const int t = s0 + r;
          if (t >= c.live) break;
          float cur[VEC], g[VEC], pre[VEC];
          if (t < 0 && given && on)
            widen<VEC>(state_row<T, K, VEC>(p.state0, c.b, p.dim, d0, t + K - 1), cur);
          else
            widen<VEC>(lds_row<T, VEC>(at + r * kRowBytes), cur);
          if (t >= 0) {
            widen<VEC>(lds_row<T, VEC>(at + kBoxBytes + r * kRowBytes), g);
            if (p.silu) {
              taps<K, VEC>(w, bv, win, cur, pre);
              apply_dsilu<VEC>(pre, g);
            }
            if (t < c.n) add_dw<K, VEC>(dw, db, g, win, cur);
            emit(t, g);
            s = t + 1;
          }
          push<K, VEC>(win, cur);
        }
      }
      __syncwarp();  // the box has been read
      ++ring.used;
      ring.load(p, q, K, K - 1);
    }
    if (bad) continue;
    float none[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) none[v] = 0.f;
#pragma unroll 1
    for (; s < c.n + K - 1; ++s) emit(s, none);  // steps past valid_len: dpre is 0
  }
  if (bad) {
    if (lane == 0) atomicOr(err, kErrConvWait);
    ring.drain();
  }

  // sums over the CTA's warps (the ring's memory: every box has been read)
  float* red = reinterpret_cast<float*>(ring_mem);
  constexpr int kWide = 32 * VEC;
  static_assert(kWarps * (K + 1) * kWide * 4 <= kBwdSmem, "fits the ring");
  __syncthreads();
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      red[(warp * (K + 1) + k) * kWide + lane * VEC + v] = k < K ? dw[k < K ? k : 0][v] : db[v];
  __syncthreads();
  for (int i = threadIdx.x; i < (K + 1) * kWide; i += kWarps * 32) {
    const int k = i / kWide, c = i - k * kWide;
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) a += red[(j * (K + 1) + k) * kWide + c];
    const int64_t d = ring.x + c;
    if (d >= p.dim) continue;
    if (gridDim.x > q.slabs)
      bp.partial[(static_cast<int64_t>(blockIdx.x / q.slabs) * (K + 1) + k) * p.dim + d] = a;
    else if (k < K)  // the slab's only CTA: its sums are the result
      bp.dweight[d * K + k] = a;
    else if (bp.dbias)
      bp.dbias[d] = a;
  }
}

// Pieces of whole boxes, with `halo` steps around them: the longest piece for
// which the slowest warp has least to do, and up to 8 boxes with valid lengths
// (`masked`), so that a warp has several pieces, live and masked ones (bf16 32 x
// 2048 x 1536: 60.5 us against 64.2 us with up to 16).  Only the first piece of a sequence
// may reach into the state, so a piece has at least width - 1 steps.  `rows`:
// CTAs per slab.  With `alone`, work that a slab's four warps finish in a piece
// of up to four boxes each goes to one CTA, whose sums need no second kernel.
Pieces make_pieces(const ConvParams& p, int vec, int ctas, int halo, bool masked, bool alone,
                   int* rows) {
  Pieces q = {};
  q.slabs = static_cast<int>((p.dim + 32 * vec - 1) / (32 * vec));
  const int64_t most = int64_t(kSms) * ctas / q.slabs > 0 ? int64_t(kSms) * ctas / q.slabs : 1;
  int64_t least = INT64_MAX;
  q.tc = 0;
  for (int n = masked ? 8 : 16; n >= 1; --n) {
    const int tc = n * kRows - halo;
    if (tc < p.width - 1) break;
    const int64_t items = p.batch * ((p.seqlen + tc - 1) / tc);
    const int64_t cost = (items + most * kWarps - 1) / (most * kWarps) * (n + 1);
    if (cost < least) {
      least = cost;
      q.tc = tc;
    }
  }
  for (int n = 1; alone && n <= 4; ++n) {
    const int tc = n * kRows - halo;
    if (tc >= p.width - 1 && p.batch * ((p.seqlen + tc - 1) / tc) <= kWarps) {
      q.tc = tc;
      break;
    }
  }
  q.segs = static_cast<int>((p.seqlen + q.tc - 1) / q.tc);
  q.items = p.batch * q.segs;
  const int64_t need = (q.items + kWarps - 1) / kWarps;
  *rows = static_cast<int>(need < most ? need : most);
  return q;
}

// A [batch, seqlen, dim] tensor's axes in the order in which a tensor map takes
// them: every stride a multiple of the one before, and the first no less than a
// row of channels.  An axis of one element goes last, whatever its stride.
struct Axes {
  bool ok, time_last;
  int64_t inner, outer;  // strides in elements
};

Axes axes_of(const ConvParams& p, int64_t batch_stride, int64_t step_stride) {
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

// The same, copied in boxes of kRows steps x 256 bytes.
bool conv_map(CUtensorMap* m, bool bf16, const void* base, const ConvParams& p, const Axes& a) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const unsigned size = bf16 ? 2 : 4;
  const cuuint64_t time = static_cast<cuuint64_t>(p.seqlen), batch = static_cast<cuuint64_t>(p.batch);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.dim), a.time_last ? batch : time,
                              a.time_last ? time : batch};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.inner) * size,
                                 static_cast<cuuint64_t>(a.outer) * size};
  const cuuint32_t rows = kRows;
  const cuuint32_t box[3] = {kRowBytes / size, a.time_last ? 1 : rows, a.time_last ? rows : 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool fits(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename T, int K>
cudaError_t fwd_k(const ConvParams& p, unsigned* err, cudaStream_t s) {
  int rows;
  Pieces q = make_pieces(p, 8 / sizeof(T), kFwdCtas, K - 1, p.valid_len != nullptr, false, &rows);
  const Axes ax = axes_of(p, p.x_batch, p.x_step);
  q.time_last = ax.time_last;
  CUtensorMap mx;
  if (!conv_map(&mx, sizeof(T) == 2, p.x, p, ax)) return cudaErrorInvalidValue;
  conv_fwd_tma_kernel<T, K><<<q.slabs * rows, kWarps * 32, kFwdSmem, s>>>(mx, p, q, err);
  return cudaGetLastError();
}

template <typename T, int K>
cudaError_t bwd_k(const ConvBwdParams& b, unsigned* err, int* parts, cudaStream_t s) {
  const ConvParams& p = b.fwd;
  int rows;
  Pieces q = make_pieces(p, 8 / sizeof(T), kBwdCtas, 2 * (K - 1), p.valid_len != nullptr, true,
                         &rows);
  const Axes ax = axes_of(p, p.x_batch, p.x_step);
  q.time_last = ax.time_last;
  const Axes ag = {true, false, p.dim, p.seqlen * p.dim};
  CUtensorMap mx, mg;
  if (!conv_map(&mx, sizeof(T) == 2, p.x, p, ax) || !conv_map(&mg, sizeof(T) == 2, b.dy, p, ag))
    return cudaErrorInvalidValue;
  auto* k = conv_bwd_tma_kernel<T, K>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kBwdSmem));
  if (e != cudaSuccess) return e;
  k<<<q.slabs * rows, kWarps * 32, kBwdSmem, s>>>(mx, mg, b, q, err);
  *parts = rows;
  return cudaGetLastError();
}

}  // namespace

bool conv_tma_ok(const ConvParams& p, bool bf16) {
  const int64_t es = bf16 ? 2 : 4;
  const int64_t lim = int64_t(1) << 30, stride = int64_t(1) << 38;
  const Axes a = axes_of(p, p.x_batch, p.x_step);
  return a.ok && (p.dim * es) % 16 == 0 && (a.inner * es) % 16 == 0 && a.outer < stride &&
         p.dim <= lim && p.seqlen <= lim && p.batch <= lim && p.seqlen * p.dim < stride &&
         fits(p.x, 16) && fits(p.weight, 16) && fits(p.y, 8) && fits(p.state0, 8) &&
         fits(p.out_final, 8);
}
bool conv_bwd_tma_ok(const ConvBwdParams& b, bool bf16) {
  return conv_tma_ok(b.fwd, bf16) && fits(b.dy, 16) && fits(b.dx, 8) && fits(b.dstate0, 8);
}

int64_t conv_bwd_tma_partials(int64_t batch, int64_t seqlen, int64_t dim, int width) {
  ConvParams p = {};
  p.batch = batch; p.seqlen = seqlen; p.dim = dim; p.width = width;
  int most = 0;
  for (int vec : {2, 4})
    for (bool masked : {false, true}) {
      int rows;
      make_pieces(p, vec, kBwdCtas, 2 * (width - 1), masked, true, &rows);
      most = rows > most ? rows : most;
    }
  return most;
}

cudaError_t launch_conv_fwd_tma(const ConvParams& p, bool bf16, unsigned* err, cudaStream_t s) {
  switch (p.width) {
    case 2: return bf16 ? fwd_k<__nv_bfloat16, 2>(p, err, s) : fwd_k<float, 2>(p, err, s);
    case 3: return bf16 ? fwd_k<__nv_bfloat16, 3>(p, err, s) : fwd_k<float, 3>(p, err, s);
    case 4: return bf16 ? fwd_k<__nv_bfloat16, 4>(p, err, s) : fwd_k<float, 4>(p, err, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_conv_bwd_tma(const ConvBwdParams& b, bool bf16, unsigned* err, int* parts,
                                cudaStream_t s) {
  switch (b.fwd.width) {
    case 2: return bf16 ? bwd_k<__nv_bfloat16, 2>(b, err, parts, s) : bwd_k<float, 2>(b, err, parts, s);
    case 3: return bf16 ? bwd_k<__nv_bfloat16, 3>(b, err, parts, s) : bwd_k<float, 3>(b, err, parts, s);
    case 4: return bf16 ? bwd_k<__nv_bfloat16, 4>(b, err, parts, s) : bwd_k<float, 4>(b, err, parts, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ssm
