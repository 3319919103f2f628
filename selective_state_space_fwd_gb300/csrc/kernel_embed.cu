// kernel_embed.cu -- the embedding lookup, y[t] = scale W[ids[t]], and the
// gradient of its weight, dW[v] = scale sum_{t: ids[t] = v} dy[t].
//
// The lookup is a copy of rows, bound by HBM.
//
// The gradient adds the rows of equal tokens in the order of the tokens, without
// atomics, so that equal inputs give equal bits.  Three launches:
// 1. The tokens are sorted by id, stably (least significant digits first, kDigits
//    values at a time), by one cluster of kSortCtas CTAs whose counts meet in
//    shared memory; the other clusters of the same launch fill dW with zeros, which
//    takes longer wherever dW is more than a few MB.
// 2. The sorted tokens are cut into windows.  A warp takes a window for a slab of
//    columns, adds the rows of each run of equal ids in fp32 and writes the runs
//    that lie in the window.  A run that another window shares leaves a partial
//    sum: `head` where it began before the window, `tail` where it began in it.
// 3. A warp per window and slab adds a tail and the heads that follow, in order.
// A frequent token is thus summed by many warps; reads and writes are dy once, dW
// once, and per window two rows of fp32.
#include <cuda_bf16.h>

#include "common.cuh"
#include "layers.h"
#include "pdl.cuh"
#include "umma_pair.cuh"
#include "vec.cuh"

namespace ssm {
namespace {

constexpr int kSms = 152;

// ---- lookup ---------------------------------------------------------------------
constexpr int kLookThreads = 256;

// A warp copies a stretch of 32 x VEC x U columns of a token's row.
template <typename W, typename O, int VEC, int U>
__global__ void __launch_bounds__(kLookThreads) embed_fwd_kernel(const EmbedParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t per = (p.dim + 32 * VEC * U - 1) / (32 * VEC * U), units = p.tokens * per;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kLookThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kLookThreads / 32) + (threadIdx.x >> 5);
       u < units; u += step) {
    const int64_t t = u / per, c0 = (u - t * per) * (32 * VEC * U) + lane * VEC;
    const int64_t id = __ldg(p.ids + t);
    const bool in = id >= 0 && id < p.vocab && id != p.ignore;
    const float other = id == p.ignore ? 0.f : NAN;
    const W* row = static_cast<const W*>(p.weight) + (in ? id : 0) * p.dim;
    Raw<W, VEC> r[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = c0 + i * 32 * VEC;
      if (in && c < p.dim) r[i] = raw_load<W, VEC>(row + c);
      else raw_zero(r[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = c0 + i * 32 * VEC;
      float f[VEC];
      widen<VEC>(r[i], f);
#pragma unroll
      for (int v = 0; v < VEC; ++v) f[v] = in ? f[v] * p.scale : other;
      if (c < p.dim) store_f<O, VEC>(static_cast<O*>(p.y) + t * p.dim + c, f);
    }
  }
}

// ---- sorting the tokens, and zeros ------------------------------------------------
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kRounds = 8;                             // keys per thread and tile
constexpr int kSortTile = kSortThreads * kRounds;
constexpr uint32_t kSortSmem = (kSortWarps + 2) * kDigits * 4;

struct SortArgs {
  const int64_t* ids;
  int64_t tokens, vocab, ignore;
  uint2 *even, *odd;     // (id, token): what even and odd passes write
  int passes, bits;    // digits and their width
  uint4* zeros;        // the part of dW that is filled in 16-byte stores
  int64_t nzeros;
  char* edge[2];       // what lies before and after it
  int nedge[2];
};

__device__ __forceinline__ uint32_t read_remote(uint32_t addr, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(pair::map_to(addr, rank)) : "memory");
  return v;
}

// The keys of a thread: a warp takes consecutive ones of the tile, round by round.
struct Keys {
  uint2 key[kRounds];        // (id, token); the token is kNone where there is none
  uint32_t place[kRounds];   // among the warp's keys of the same digit
  int rounds;

  static constexpr uint32_t kNone = 0xffffffffu;
  __device__ __forceinline__ bool is(int r) const { return r < rounds && key[r].y != kNone; }

  __device__ __forceinline__ void load(const SortArgs& p, int pass, int64_t t0, int64_t end) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = end - t0 < kSortTile ? end - t0 : kSortTile;
    rounds = static_cast<int>((n + kSortThreads - 1) / kSortThreads);
    const uint2* from = pass & 1 ? p.even : p.odd;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int64_t i = t0 + (warp * rounds + r) * 32 + lane;
      key[r] = make_uint2(0, kNone);
      if (r < rounds && i < end) {
        if (pass == 0) {
          const int64_t id = __ldg(p.ids + i);
          const bool kept = id >= 0 && id < p.vocab && id != p.ignore;
          key[r] = make_uint2(static_cast<uint32_t>(kept ? id : p.vocab), static_cast<uint32_t>(i));
        } else {
          key[r] = __ldcg(from + i);
        }
      }
    }
  }
  // The lanes whose key of round r has the same digit as this lane's.
  __device__ __forceinline__ uint32_t peers(int r, uint32_t digit) const {
    return __match_any_sync(0xffffffffu, is(r) ? digit : kDigits);
  }
  // Ranks the keys; whist[warp] is left with the number of each digit.
  __device__ __forceinline__ void rank(uint32_t (*whist)[kDigits], int shift, uint32_t mask) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads) whist[0][i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      place[r] = 0;
      if (r < rounds) {
        const uint32_t digit = (key[r].x >> shift) & mask, same = peers(r, digit);
        const uint32_t before = __popc(same & ((1u << lane) - 1)), seen = whist[warp][digit];
        place[r] = seen + before;
        __syncwarp();
        if (is(r) && before == 0) whist[warp][digit] = seen + __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();
  }
};

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const SortArgs p) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  release_next();
  if (blockIdx.x >= kSortCtas) {
    const int64_t first = static_cast<int64_t>(blockIdx.x - kSortCtas) * kSortThreads + tid;
    const int64_t step = static_cast<int64_t>(gridDim.x - kSortCtas) * kSortThreads;
#pragma unroll 4
    for (int64_t i = first; i < p.nzeros; i += step) p.zeros[i] = make_uint4(0, 0, 0, 0);
    if (first < p.nedge[0]) p.edge[0][first] = 0;
    if (first < p.nedge[1]) p.edge[1][first] = 0;
    return;
  }
  extern __shared__ __align__(16) uint32_t sort_mem[];
  uint32_t(*whist)[kDigits] = reinterpret_cast<uint32_t(*)[kDigits]>(sort_mem);
  uint32_t* hist = sort_mem + kSortWarps * kDigits;
  uint32_t* base = hist + kDigits;
  __shared__ uint32_t sums[kSortWarps];
  const uint32_t rank = pair::cluster_rank();
  const int64_t per = (p.tokens + 32 * kSortCtas - 1) / (32 * kSortCtas) * 32;
  const int64_t k0 = rank * per < p.tokens ? rank * per : p.tokens;
  const int64_t k1 = k0 + per < p.tokens ? k0 + per : p.tokens;
  const bool one = k1 - k0 <= kSortTile;  // the keys stay in registers between count and move
  Keys k;
  if (one) k.load(p, 0, k0, k1);

  for (int pass = 0; pass < p.passes; ++pass) {
    uint2* to = pass & 1 ? p.odd : p.even;
    const int shift = pass * p.bits;
    const uint32_t mask = (1u << p.bits) - 1;
    if (tid < kDigits) hist[tid] = 0;
    __syncthreads();
    if (one) {
      if (pass > 0) k.load(p, pass, k0, k1);
      k.rank(whist, shift, mask);
      if (tid < kDigits) {
        uint32_t n = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) n += whist[w][tid];
        hist[tid] = n;
      }
    } else {
      for (int64_t t0 = k0; t0 < k1; t0 += kSortTile) {
        k.load(p, pass, t0, k1);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
          const uint32_t digit = (k.key[r].x >> shift) & mask, same = k.peers(r, digit);
          if (k.is(r) && (same & ((1u << lane) - 1)) == 0) atomicAdd(hist + digit, __popc(same));
        }
      }
    }
    pair::cluster_sync();
    // where this CTA's keys of a digit go: after the lower digits of all CTAs and
    // the same digit of the CTAs before
    uint32_t total = 0, below = 0;
    if (tid < kDigits) {
      const uint32_t at = umma::smem_u32(hist + tid);
#pragma unroll
      for (uint32_t q = 0; q < kSortCtas; ++q) {
        const uint32_t n = read_remote(at, q);
        total += n;
        below += q < rank ? n : 0;
      }
    }
    uint32_t sum = total;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += n;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    if (tid < kDigits) {
      uint32_t start = sum - total + below;
      for (int w = 0; w < warp; ++w) start += sums[w];
      base[tid] = start;
    }
    for (int64_t t0 = k0; t0 < k1; t0 += kSortTile) {
      if (!one) {
        k.load(p, pass, t0, k1);
        k.rank(whist, shift, mask);
      }
      if (tid < kDigits) {
        uint32_t at = base[tid];
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
          const uint32_t n = whist[w][tid];
          whist[w][tid] = at;
          at += n;
        }
        base[tid] = at;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
        if (k.is(r)) to[whist[warp][(k.key[r].x >> shift) & mask] + k.place[r]] = k.key[r];
      __syncthreads();
    }
    pair::cluster_sync();
  }
}

// ---- sums -------------------------------------------------------------------------
constexpr int kSumThreads = 128;

struct SumArgs {
  const uint2* sorted;
  const void* dy;
  void* dweight;
  float* part;          // [windows][2][dim]: head, tail
  int64_t tokens, vocab, dim, windows;
  int window;           // tokens per window
  int slabs;
  float scale;
  bool add;
};

// A lane's columns of a slab: G groups of VEC, a warp's width apart.
template <int VEC> struct Slab {
  static constexpr int kGroups = VEC == 1 ? 4 : 1;
  static constexpr int kWidth = 32 * VEC * kGroups;
};

template <typename W, int VEC, int G>
__device__ __forceinline__ void write_row(const SumArgs& p, int64_t id, int64_t c0,
                                          const float (&acc)[G][VEC]) {
  W* row = static_cast<W*>(p.dweight) + id * p.dim;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c = c0 + g * 32 * VEC;
    if (c >= p.dim) continue;
    float f[VEC];
    if (p.add) widen<VEC>(raw_load_rw<W, VEC>(row + c), f);
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      f[v] = p.add ? fmaf(acc[g][v], p.scale, f[v]) : acc[g][v] * p.scale;
    store_f<W, VEC>(row + c, f);
  }
}

template <int VEC, int G>
__device__ __forceinline__ void write_part(const SumArgs& p, int64_t slot, int64_t c0,
                                           const float (&acc)[G][VEC]) {
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c = c0 + g * 32 * VEC;
    if (c < p.dim) store_f<float, VEC>(p.part + slot * p.dim + c, acc[g]);
  }
}

template <typename W, typename O, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumArgs p) {
  constexpr int G = Slab<VEC>::kGroups;
  constexpr int kAhead = 8;
  const int lane = threadIdx.x & 31;
  wait_previous();
  release_next();
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (kSumThreads / 32) + (threadIdx.x >> 5);
  const int64_t w = u / p.slabs;
  if (w >= p.windows) return;
  const int64_t c0 = (u - w * p.slabs) * Slab<VEC>::kWidth + lane * VEC;
  const int64_t i0 = w * p.window;
  const int64_t i1 = i0 + p.window < p.tokens ? i0 + p.window : p.tokens;
  const O* dy = static_cast<const O*>(p.dy);
  float acc[G][VEC];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[g][v] = 0.f;
  bool head = i0 > 0 && __ldg(p.sorted + i0 - 1).x == __ldg(p.sorted + i0).x;
  for (int64_t j = i0; j < i1; j += 32) {
    const int n = i1 - j < 32 ? static_cast<int>(i1 - j) : 32;
    uint2 k = make_uint2(0xffffffffu, 0);
    if (lane < n) k = __ldg(p.sorted + j + lane);
    // the key after each: the next lane's, or the next group's first
    uint32_t after = __shfl_down_sync(0xffffffffu, k.x, 1);
    if (lane == n - 1) after = j + n < p.tokens ? __ldg(p.sorted + j + n).x : 0xffffffffu;
    const unsigned ends = __ballot_sync(0xffffffffu, lane < n && after != k.x);
    if (__shfl_sync(0xffffffffu, k.x, 0) >= p.vocab) return;  // from here on none is kept
    for (int s = 0; s < n; s += kAhead) {
      Raw<O, VEC> r[kAhead][G];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int src = s + a < n ? s + a : 0;
        const uint32_t id = __shfl_sync(0xffffffffu, k.x, src);
        const int64_t row = __shfl_sync(0xffffffffu, k.y, src);
        const bool in = s + a < n && id < p.vocab;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int64_t c = c0 + g * 32 * VEC;
          if (in && c < p.dim) r[a][g] = raw_load<O, VEC>(dy + row * p.dim + c);
          else raw_zero(r[a][g]);
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (s + a >= n) break;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float f[VEC];
          widen<VEC>(r[a][g], f);
#pragma unroll
          for (int v = 0; v < VEC; ++v) acc[g][v] += f[v];
        }
        const bool end = (ends >> (s + a)) & 1, last = j + s + a + 1 == i1;
        if (end || last) {
          const uint32_t id = __shfl_sync(0xffffffffu, k.x, s + a);
          if (id < p.vocab) {
            if (head) write_part<VEC, G>(p, 2 * w, c0, acc);
            else if (end) write_row<W, VEC, G>(p, id, c0, acc);
            else write_part<VEC, G>(p, 2 * w + 1, c0, acc);
          }
          head = false;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int v = 0; v < VEC; ++v) acc[g][v] = 0.f;
        }
      }
    }
  }
}

template <typename W, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const SumArgs p) {
  constexpr int G = Slab<VEC>::kGroups;
  const int lane = threadIdx.x & 31;
  wait_previous();
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (kSumThreads / 32) + (threadIdx.x >> 5);
  const int64_t w = u / p.slabs;
  if (w + 1 >= p.windows) return;
  const int64_t i1 = (w + 1) * p.window;
  const uint32_t id = __ldg(p.sorted + i1 - 1).x;
  // the window's last run began in it and goes on
  if (id >= p.vocab || __ldg(p.sorted + i1).x != id) return;
  const int64_t i0 = w * p.window;
  if (i0 > 0 && __ldg(p.sorted + i0).x == id && __ldg(p.sorted + i0 - 1).x == id) return;
  const int64_t c0 = (u - w * p.slabs) * Slab<VEC>::kWidth + lane * VEC;
  float acc[G][VEC];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c = c0 + g * 32 * VEC;
    if (c < p.dim) load_f<float, VEC>(p.part + (2 * w + 1) * p.dim + c, acc[g]);
  }
  for (int64_t j = w + 1;;) {
    const int64_t mine = j + lane;
    const bool goes = mine < p.windows && __ldg(p.sorted + mine * p.window).x == id;
    const unsigned stop = ~__ballot_sync(0xffffffffu, goes);
    const int n = stop ? __ffs(stop) - 1 : 32;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int64_t c = c0 + g * 32 * VEC;
        if (c >= p.dim) continue;
        float f[VEC];
        load_f<float, VEC>(p.part + 2 * (j + i) * p.dim + c, f);
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[g][v] += f[v];
      }
    }
    j += n;
    if (n < 32) break;
  }
  write_row<W, VEC, G>(p, id, c0, acc);
}

// ---- sizes and launches -------------------------------------------------------------
struct Layout {
  size_t buf[2], part, total;
  int64_t windows;
  int window;
};

// Tokens per window: as many as leave about 16 warps per SM, each over 256 columns.
Layout layout_of(int64_t tokens, int64_t dim) {
  Layout l;
  const int64_t slabs = (dim + 255) / 256;
  l.window = 8;
  while (l.window < 128 && (tokens / (2 * l.window)) * slabs >= 16 * kSms) l.window *= 2;
  l.windows = (tokens + l.window - 1) / l.window;
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  l.buf[0] = take(8 * tokens);
  l.buf[1] = take(8 * tokens);
  l.part = take(sizeof(float) * 2 * l.windows * dim);
  l.total = off;
  return l;
}

bool rows_of(const void* p, int64_t dim, size_t elem, int vec) {
  return dim % vec == 0 && reinterpret_cast<uintptr_t>(p) % (elem * vec < 16 ? elem * vec : 16) == 0;
}

template <typename W, typename O, int VEC, int U>
cudaError_t look(const EmbedParams& p, cudaStream_t s) {
  const int64_t units = p.tokens * ((p.dim + 32 * VEC * U - 1) / (32 * VEC * U));
  const int64_t ctas = (units + kLookThreads / 32 - 1) / (kLookThreads / 32);
  const int64_t most = int64_t(kSms) * 64;
  embed_fwd_kernel<W, O, VEC, U><<<static_cast<unsigned>(ctas < most ? ctas : most), kLookThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename W, typename O, int VEC>
cudaError_t sum(const SumArgs& a, cudaStream_t s) {
  SumArgs b = a;
  b.slabs = static_cast<int>((a.dim + Slab<VEC>::kWidth - 1) / Slab<VEC>::kWidth);
  const int64_t ctas = (a.windows * b.slabs + kSumThreads / 32 - 1) / (kSumThreads / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_after(embed_sum_kernel<W, O, VEC>, static_cast<unsigned>(ctas), kSumThreads, 0, s, b);
  if (e != cudaSuccess) return e;
  return launch_after(embed_join_kernel<W, VEC>, static_cast<unsigned>(ctas), kSumThreads, 0, s, b);
}

}  // namespace

size_t embed_bwd_workspace_bytes(int64_t tokens, int64_t dim) { return layout_of(tokens, dim).total; }

cudaError_t launch_embed_fwd(const EmbedParams& p, bool bf16, bool io_bf16, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const auto wide = [&](int vec) {
    return rows_of(p.weight, p.dim, bf16 ? 2 : 4, vec) && rows_of(p.y, p.dim, io_bf16 ? 2 : 4, vec);
  };
  if (!bf16) return wide(4) ? look<float, float, 4, 2>(p, s) : look<float, float, 1, 4>(p, s);
  if (io_bf16) return wide(8) ? look<bf, bf, 8, 2>(p, s) : look<bf, bf, 1, 4>(p, s);
  return wide(8) ? look<bf, float, 8, 1>(p, s) : look<bf, float, 1, 4>(p, s);
}

cudaError_t launch_embed_bwd(const EmbedBwdParams& p, bool bf16, bool io_bf16, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const Layout l = layout_of(p.tokens, p.dim);
  char* ws = static_cast<char*>(p.workspace);
  SortArgs a = {};
  a.ids = p.ids;
  a.tokens = p.tokens; a.vocab = p.vocab; a.ignore = p.ignore;
  a.even = reinterpret_cast<uint2*>(ws + l.buf[0]);
  a.odd = reinterpret_cast<uint2*>(ws + l.buf[1]);
  int bits = 1;
  while ((p.vocab >> bits) > 0) ++bits;  // ids, and `vocab` for the tokens that are left out
  a.passes = (bits + kDigitBits - 1) / kDigitBits;
  a.bits = (bits + a.passes - 1) / a.passes;
  int fill = 0;
  if (!p.add) {
    char* begin = static_cast<char*>(p.dweight);
    const size_t bytes = static_cast<size_t>(p.vocab) * p.dim * (bf16 ? 2 : 4);
    size_t before = (16 - reinterpret_cast<uintptr_t>(begin) % 16) % 16;
    if (before > bytes) before = bytes;
    a.zeros = reinterpret_cast<uint4*>(begin + before);
    a.nzeros = static_cast<int64_t>((bytes - before) / 16);
    a.edge[0] = begin;
    a.nedge[0] = static_cast<int>(before);
    a.edge[1] = begin + before + a.nzeros * 16;
    a.nedge[1] = static_cast<int>(bytes - before - a.nzeros * 16);
    const int64_t need = (a.nzeros / kSortThreads + 1 + kSortCtas - 1) / kSortCtas;
    const int64_t most = kSms / kSortCtas - 1;
    fill = static_cast<int>(need < most ? need : most) * kSortCtas;
  }
  cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSortSmem));
  if (e != cudaSuccess) return e;
  embed_sort_kernel<<<kSortCtas + fill, kSortThreads, kSortSmem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  SumArgs b = {};
  b.sorted = a.passes & 1 ? a.even : a.odd;
  b.dy = p.dy; b.dweight = p.dweight;
  b.part = reinterpret_cast<float*>(ws + l.part);
  b.tokens = p.tokens; b.vocab = p.vocab; b.dim = p.dim;
  b.windows = l.windows; b.window = l.window;
  b.scale = p.scale; b.add = p.add;
  const auto wide = [&](int vec) {
    return rows_of(p.dweight, p.dim, bf16 ? 2 : 4, vec) && rows_of(p.dy, p.dim, io_bf16 ? 2 : 4, vec);
  };
  if (!bf16) return wide(4) ? sum<float, float, 4>(b, s) : sum<float, float, 1>(b, s);
  if (io_bf16) return wide(8) ? sum<bf, bf, 8>(b, s) : sum<bf, bf, 1>(b, s);
  return wide(8) ? sum<bf, float, 8>(b, s) : sum<bf, float, 1>(b, s);
}

}  // namespace ssm
