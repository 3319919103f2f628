// kernel_embed.cu -- the embedding lookup, y[t] = scale W[ids[t]], and the
// gradient of its weight, dW[v] = scale sum_{t: ids[t] = v} dy[t].
//
// The lookup is a copy of rows, bound by HBM: 65536 tokens x 2048 in bf16, 16,000 rows
// of the weight among them, 56 us (6.0 TB/s).
//
// The gradient adds the rows of equal tokens in the order of the tokens, without
// atomics, so that equal inputs give equal bits:
// 1. The tokens are sorted by id, stably (least significant digits first, kDigits
//    values at a time), by one cluster whose counts meet in shared memory; few tokens
//    are placed by counting instead.  dW is filled with zeros meanwhile.
// 2. The sorted tokens are cut into windows.  A warp takes a window for a slab of
//    columns, adds the rows of each run of equal ids in fp32 and writes the runs
//    that lie in the window.  A run that another window shares leaves a partial
//    sum: `head` where it began before the window, `tail` where it began in it.
// 3. A CTA per window and slab adds a tail and the heads that follow, in order.
// A frequent token is thus summed by many warps; reads and writes are dy once, dW
// once, and per window two rows of fp32.
//
// Measured on GB300, ids with a frequency that falls with their rank: 65536 tokens x 2048
// onto a bf16 gradient 102 us, of which the sort 21 (16 SMs, the latency of its barriers
// and scattered stores), the sums 73 (5.1 TB/s) and the heads 9; as a whole gradient of
// 65536 rows 131 us; fp32 5001 x 1536 of 32001 rows 45 us, 27.5 of which are the zeros;
// with 1537 columns, one element per access, 53 us; 8 tokens onto a gradient 6 us.  Code
// that runs once or twice per warp is fetched at its own cost: with 8 rows ahead instead
// of 4, and 4 columns per lane instead of 2 off a boundary, 8 tokens took 45 us as a
// whole gradient, not 38.
#include <cuda_bf16.h>

#include "cluster.cuh"
#include "common.cuh"
#include "f32x2.cuh"
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
constexpr int kSortCtas = kMaxCluster;                 // at most
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kRounds = 4;                             // keys per thread and tile
constexpr int kSortTile = kSortThreads * kRounds;
static_assert(kSortTile <= 65536, "places within a tile are kept in 16 bits");

struct SortArgs {
  const int64_t* ids;
  int64_t tokens, vocab, ignore;
  uint2 *even, *odd;     // (id, token): what even and odd passes write
  int passes, bits;      // digits and their width
  uint32_t ctas;         // of the cluster
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
  // Ranks the keys; counts[warp] is left with the number of each digit.
  __device__ __forceinline__ void rank(uint16_t (*counts)[kDigits], int shift, uint32_t mask) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint4* clear = reinterpret_cast<uint4*>(counts[warp]);
#pragma unroll
    for (int i = 0; i < kDigits / 8; i += 32) clear[i + lane] = make_uint4(0, 0, 0, 0);
    __syncwarp();
    uint32_t same[kRounds];  // first, so that the rounds' searches overlap
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      same[r] = r < rounds ? peers(r, (key[r].x >> shift) & mask) : 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      place[r] = 0;
      if (r < rounds) {
        const uint32_t digit = (key[r].x >> shift) & mask;
        const uint32_t before = __popc(same[r] & ((1u << lane) - 1)), seen = counts[warp][digit];
        place[r] = seen + before;
        __syncwarp();
        if (is(r) && before == 0) counts[warp][digit] = static_cast<uint16_t>(seen + __popc(same[r]));
        __syncwarp();
      }
    }
    __syncthreads();
  }
};

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const SortArgs p) {
  __shared__ __align__(16) uint16_t counts[kSortWarps][kDigits];
  __shared__ uint32_t hist[kDigits], base[kDigits], sums[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  release_next();
  const uint32_t rank = pair::cluster_rank();
  const int64_t per = (p.tokens + 32 * p.ctas - 1) / (32 * p.ctas) * 32;
  const int64_t k0 = rank * per < p.tokens ? rank * per : p.tokens;
  const int64_t k1 = k0 + per < p.tokens ? k0 + per : p.tokens;
  const bool one = k1 - k0 <= kSortTile;  // the keys stay in registers between count and move
  Keys k;
  if (one) k.load(p, 0, k0, k1);

  for (int pass = 0; pass < p.passes; ++pass) {
    uint2* to = pass & 1 ? p.odd : p.even;
    const int shift = pass * p.bits;
    const uint32_t mask = (1u << p.bits) - 1;
    if (one) {
      if (pass > 0) k.load(p, pass, k0, k1);
      k.rank(counts, shift, mask);
      if (tid < kDigits) {
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
          const uint32_t c = counts[w][tid];
          counts[w][tid] = static_cast<uint16_t>(n);  // those of the warps before
          n += c;
        }
        hist[tid] = n;
      }
    } else {
      if (tid < kDigits) hist[tid] = 0;
      __syncthreads();
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
        const uint32_t n = q < p.ctas ? read_remote(at, q) : 0;
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
    __syncthreads();
    for (int64_t t0 = k0; t0 < k1; t0 += kSortTile) {
      uint32_t n = 0;
      if (!one) {
        k.load(p, pass, t0, k1);
        k.rank(counts, shift, mask);
        if (tid < kDigits) {
#pragma unroll
          for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = counts[w][tid];
            counts[w][tid] = static_cast<uint16_t>(n);
            n += c;
          }
        }
        __syncthreads();
      }
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        if (!k.is(r)) continue;
        const uint32_t digit = (k.key[r].x >> shift) & mask;
        to[base[digit] + counts[warp][digit] + k.place[r]] = k.key[r];
      }
      __syncthreads();
      if (!one && tid < kDigits) base[tid] += n;
      if (!one) __syncthreads();
    }
    pair::cluster_sync();
  }
}

// Few tokens are placed by counting, all SMs at once and without passes: a CTA takes
// kRankTokens of them, one per lane, and its warps share the tokens that each is
// compared with.  T^2 comparisons: 8192 tokens 5 us, where the passes' latencies alone
// are 12 us.
constexpr int kRankMost = 8192, kRankTokens = 32, kRankWarps = 16;
__global__ void __launch_bounds__(kRankWarps * 32) embed_rank_kernel(const SortArgs p) {
  __shared__ __align__(16) uint32_t ids[kRankMost];
  __shared__ uint32_t part[kRankWarps][kRankTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = static_cast<int>(p.tokens), i0 = blockIdx.x * kRankTokens, i = i0 + lane;
  release_next();
#pragma unroll 8
  for (int t = threadIdx.x; t < n; t += kRankWarps * 32) {
    const int64_t id = __ldg(p.ids + t);
    const bool kept = id >= 0 && id < p.vocab && id != p.ignore;
    ids[t] = static_cast<uint32_t>(kept ? id : p.vocab);
  }
  const int pad = (n + 3) / 4 * 4;
  if (threadIdx.x < pad - n) ids[n + threadIdx.x] = 0x7fffffffu;  // before nothing
  __syncthreads();
  const uint32_t mine = i < n ? ids[i] : 0;
  // those of an equal id count where they come before: the CTA's own tokens one by one,
  // the others in groups of four
  uint32_t count = 0;
  const auto groups = [&](int from, int to, uint32_t below) {
#pragma unroll 4
    for (int j = from + warp * 4; j < to; j += kRankWarps * 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(ids + j);
      // k < below: the difference's sign, as neither reaches 2^31
      count += ((k.x - below) >> 31) + ((k.y - below) >> 31);
      count += ((k.z - below) >> 31) + ((k.w - below) >> 31);
    }
  };
  groups(0, i0, mine + 1);
  groups(i0 + kRankTokens, pad, mine);
  if (warp == 0) {
    const int own = n - i0 < kRankTokens ? n - i0 : kRankTokens;
    for (int j = 0; j < own; ++j) {
      const uint32_t k = ids[i0 + j];
      count += k < mine || (k == mine && j < lane);
    }
  }
  part[warp][lane] = count;
  __syncthreads();
  if (warp == 0 && i < n) {
    uint32_t place = 0;
#pragma unroll
    for (int w = 0; w < kRankWarps; ++w) place += part[w][lane];
    p.even[place] = make_uint2(mine, static_cast<uint32_t>(i));
  }
}

// Zeros over `bytes` bytes at `begin`.  It runs beside the sort, which it does not
// depend on, but ends after it, so that what follows has both.  It writes before it waits:
// the sort (or embed_rank_kernel) is launched in plain stream order, so that all work before
// it, which may still use those bytes, is done.  (Filling only the rows
// without tokens, beside the sums, gained nothing: the sums' few dependent loads wait
// behind its stores.)
constexpr int kFillThreads = 256;
__global__ void __launch_bounds__(kFillThreads) embed_fill_kernel(char* begin, int64_t bytes) {
  release_next();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kFillThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kFillThreads;
  int64_t before = (16 - reinterpret_cast<uintptr_t>(begin) % 16) % 16;
  if (before > bytes) before = bytes;
  const int64_t n = (bytes - before) / 16, after = bytes - before - 16 * n;
  uint4* body = reinterpret_cast<uint4*>(begin + before);
#pragma unroll 8
  for (int64_t i = first; i < n; i += step) body[i] = make_uint4(0, 0, 0, 0);
  if (first < before) begin[first] = 0;
  if (first < after) begin[before + 16 * n + first] = 0;
  wait_previous();
}

// ---- sums -------------------------------------------------------------------------
constexpr int kSumThreads = 128;

struct SumArgs {
  const uint2* sorted;
  const void* dy;
  void* dweight;
  float* part;          // [windows][2][dim]: head, tail
  int64_t tokens, vocab, dim;
  int64_t windows;      // of the CTAs
  int window;           // tokens per warp
  int slabs;
  float scale;
};

// A lane's columns of a slab: G groups of VEC, a warp's width apart.
template <int VEC> struct Slab {
  static constexpr int kGroups = VEC == 1 ? 2 : 1;
  static constexpr int kWidth = 32 * VEC * kGroups;
};

// A lane's columns of dW's row as it is, for `add`.
template <typename W, int VEC, int G>
__device__ __forceinline__ void there(const SumArgs& p, int64_t id, int64_t c0, Raw<W, VEC> (&r)[G]) {
  const W* row = static_cast<const W*>(p.dweight) + id * p.dim;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c = c0 + g * 32 * VEC;
    if (c < p.dim) r[g] = raw_load_rw<W, VEC>(row + c);
    else raw_zero(r[g]);
  }
}

template <typename W, int VEC, int G, bool ADD>
__device__ __forceinline__ void write_row(const SumArgs& p, int64_t id, int64_t c0,
                                          const float (&acc)[G][VEC], const Raw<W, VEC> (&old)[G]) {
  W* row = static_cast<W*>(p.dweight) + id * p.dim;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c = c0 + g * 32 * VEC;
    if (c >= p.dim) continue;
    float f[VEC], by[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) by[v] = p.scale;
    if (ADD) {
      widen<VEC>(old[g], f);
      vfma<VEC>(f, acc[g], by, f);
    } else {
      vmul<VEC>(f, acc[g], by);
    }
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

// A CTA's warps take consecutive windows of one slab.  What a run leaves in a warp, its
// head where it began in an earlier window and its tail where it goes on, meets in
// shared memory; only what leaves the CTA's windows is joined by the next kernel.
constexpr int kSumWarps = kSumThreads / 32;
template <typename W, typename O, int VEC, bool ADD>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumArgs p) {
  constexpr int G = Slab<VEC>::kGroups;
  constexpr int kAhead = 4;
  __shared__ float part[kSumWarps][2][G * VEC][32];
  __shared__ uint32_t tail_id[kSumWarps];
  __shared__ unsigned char has_tail[kSumWarps], whole[kSumWarps];
  release_next();
  wait_previous();
  const int64_t unit = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t set = unit / p.slabs, w = set * kSumWarps + warp;
  const int64_t c0 = (unit - set * p.slabs) * Slab<VEC>::kWidth + lane * VEC;
  const int64_t i0 = w * p.window;
  const int64_t i1 = i0 + p.window < p.tokens ? i0 + p.window : p.tokens;
  const O* dy = static_cast<const O*>(p.dy);
  float acc[G][VEC];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[g][v] = 0.f;
  const auto keep = [&](int which) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int v = 0; v < VEC; ++v) part[warp][which][g * VEC + v][lane] = acc[g][v];
  };
  const bool begun = i0 > 0 && i0 < i1 && __ldg(p.sorted + i0 - 1).x == __ldg(p.sorted + i0).x;
  bool head = begun, goes = false;  // the run in hand began before; the last one goes on
  uint32_t last_id = 0xffffffffu;
  for (int64_t j = i0; j < i1; j += 32) {
    const int n = i1 - j < 32 ? static_cast<int>(i1 - j) : 32;
    uint2 k = make_uint2(0xffffffffu, 0);
    if (lane < n) k = __ldg(p.sorted + j + lane);
    // the key after each: the next lane's, or the next group's first
    uint32_t after = __shfl_down_sync(0xffffffffu, k.x, 1);
    if (lane == n - 1) after = j + n < p.tokens ? __ldg(p.sorted + j + n).x : 0xffffffffu;
    const unsigned ends = __ballot_sync(0xffffffffu, lane < n && after != k.x);
    if (__shfl_sync(0xffffffffu, k.x, 0) >= p.vocab) break;  // from here on none is kept
    for (int s = 0; s < n; s += kAhead) {
      Raw<O, VEC> r[kAhead][G];
      Raw<W, VEC> old[ADD ? kAhead : 1][G];
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
        // a row of dW that a run ends at, before its sum is known
        if (ADD && in && ((ends >> src) & 1)) there<W, VEC, G>(p, id, c0, old[a]);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (s + a >= n) break;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float f[VEC];
          widen<VEC>(r[a][g], f);
          vadd<VEC>(acc[g], acc[g], f);
        }
        const bool end = (ends >> (s + a)) & 1, last = j + s + a + 1 == i1;
        if (end || last) {
          const uint32_t id = __shfl_sync(0xffffffffu, k.x, s + a);
          if (id < p.vocab) {
            if (head) keep(0);
            else if (end) write_row<W, VEC, G, ADD>(p, id, c0, acc, old[ADD ? a : 0]);
            else keep(1);
            goes = !end;
            last_id = id;
          }
          if (!end) break;
          head = false;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int v = 0; v < VEC; ++v) acc[g][v] = 0.f;
        }
      }
    }
  }
  if (lane == 0) {
    has_tail[warp] = goes && !head;
    whole[warp] = goes && head;  // one run, from before the window to after it
    tail_id[warp] = last_id;
  }
  __syncthreads();
  const auto add = [&](int of) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[g][v] += part[of][0][g * VEC + v][lane];
  };
  const auto take = [&](int which) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[g][v] = part[warp][which][g * VEC + v][lane];
  };
  if (warp == 0 && begun) {  // a run from before the CTA's windows
    take(0);
    for (int of = 0; of + 1 < kSumWarps && whole[of]; ++of) add(of + 1);
    write_part<VEC, G>(p, 2 * set, c0, acc);
  }
  if (has_tail[warp]) {  // a run that began here: the heads that follow are its own
    const uint32_t id = tail_id[warp];
    take(1);
    int of = warp + 1;
    bool open = true;
    for (; of < kSumWarps && open; ++of) {
      add(of);
      open = whole[of];
    }
    if (open) {
      write_part<VEC, G>(p, 2 * set + 1, c0, acc);
    } else {
      Raw<W, VEC> old[G];
      if (ADD) there<W, VEC, G>(p, id, c0, old);
      write_row<W, VEC, G, ADD>(p, id, c0, acc, old);
    }
  }
}

// A CTA takes the run that its windows' last tokens began, for one slab; its warps
// share the heads.
template <typename W, int VEC, bool ADD>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const SumArgs p) {
  constexpr int G = Slab<VEC>::kGroups;
  __shared__ float part[kSumWarps][G * VEC][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_previous();
  const int64_t set = blockIdx.x / p.slabs, width = static_cast<int64_t>(p.window) * kSumWarps;
  const int64_t i0 = set * width, i1 = i0 + width;
  if (set + 1 >= p.windows) return;
  const uint32_t id = __ldg(p.sorted + i1 - 1).x, next = __ldg(p.sorted + i1).x;
  const uint32_t first = __ldg(p.sorted + i0).x, before = i0 > 0 ? __ldg(p.sorted + i0 - 1).x : ~id;
  // the last run goes on, and began in these windows
  if (id >= p.vocab || next != id || (first == id && before == id)) return;
  const int64_t c0 = (blockIdx.x - set * p.slabs) * Slab<VEC>::kWidth + lane * VEC;
  int64_t n = 0;  // heads
  for (unsigned stop = 0; !stop;) {
    const int64_t j = set + 1 + n + lane;
    stop = ~__ballot_sync(0xffffffffu, j < p.windows && __ldg(p.sorted + j * width).x == id);
    n += stop ? __ffs(stop) - 1 : 32;
  }
  const int64_t share = (n + kSumWarps - 1) / kSumWarps;
  const int64_t h0 = warp * share, h1 = h0 + share < n ? h0 + share : n;
  float acc[G][VEC];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[g][v] = 0.f;
  const auto add = [&](int64_t slot) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t c = c0 + g * 32 * VEC;
      if (c >= p.dim) continue;
      float f[VEC];
      load_f<float, VEC>(p.part + slot * p.dim + c, f);
      vadd<VEC>(acc[g], acc[g], f);
    }
  };
  if (warp == 0) add(2 * set + 1);  // the tail
#pragma unroll 4
  for (int64_t h = h0; h < h1; ++h) add(2 * (set + 1 + h));
  if (warp > 0) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int v = 0; v < VEC; ++v) part[warp][g * VEC + v][lane] = acc[g][v];
  }
  __syncthreads();
  if (warp > 0) return;
  Raw<W, VEC> old[G];
  if (ADD) there<W, VEC, G>(p, id, c0, old);
  for (int w = 1; w < kSumWarps; ++w) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[g][v] += part[w][g * VEC + v][lane];
  }
  write_row<W, VEC, G, ADD>(p, id, c0, acc, old);
}

// ---- sizes and launches -------------------------------------------------------------
struct Layout {
  size_t buf[2], part, total;
  int64_t windows;
  int window;
};

// Tokens per warp: the most, up to 32, that leave 16 warps per SM (long windows
// leave fewer partial sums).  They are counted by the slabs of tensors on a boundary, even
// where a call's are not: the windows fix the order of the sums.
Layout layout_of(int64_t tokens, int64_t dim, bool bf16) {
  Layout l;
  const int vec = bf16 ? 8 : 4;
  const int width = dim % vec != 0 ? Slab<1>::kWidth : bf16 ? Slab<8>::kWidth : Slab<4>::kWidth;
  const int64_t slabs = (dim + width - 1) / width;
  l.window = 8;
  while (l.window < 32 && tokens / (2 * l.window) * slabs >= 16 * kSms) l.window *= 2;
  l.windows = (tokens + l.window * kSumWarps - 1) / (l.window * kSumWarps);
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

template <typename W, typename O, int VEC, bool ADD>
cudaError_t sum(SumArgs a, cudaStream_t s) {
  a.slabs = static_cast<int>((a.dim + Slab<VEC>::kWidth - 1) / Slab<VEC>::kWidth);
  const int64_t units = a.windows * a.slabs;
  const cudaError_t e = launch_after(embed_sum_kernel<W, O, VEC, ADD>,
                                     static_cast<unsigned>(units), kSumThreads, 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_after(embed_join_kernel<W, VEC, ADD>, static_cast<unsigned>(units), kSumThreads, 0, s, a);
}

// Launched in plain stream order: embed_fill_kernel counts on it.
// Sorts with one thread per token, but in at most kSortCtas CTAs (8 where the GPU has
// no room for a larger cluster).
cudaError_t sort(SortArgs& a, cudaStream_t s) {
  a.ctas = 1;
  while (a.ctas < kSortCtas && a.ctas * kSortThreads < a.tokens) a.ctas *= 2;
  if (a.ctas > kPortableCluster) {
    if (resident_clusters<embed_sort_kernel>(4, kSortThreads, 0) < 1) {
      a.ctas = kPortableCluster;
    } else {
      const cudaError_t e = allow_large_clusters(reinterpret_cast<const void*>(embed_sort_kernel));
      if (e != cudaSuccess) return e;
    }
  }
  const ClusterLaunch l(1, static_cast<int>(a.ctas), kSortThreads, 0, s);
  return cudaLaunchKernelEx(&l.cfg, embed_sort_kernel, a);
}

}  // namespace

size_t embed_bwd_workspace_bytes(int64_t tokens, int64_t dim, bool bf16) {
  return layout_of(tokens, dim, bf16).total;
}

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
  const int most = bf16 ? 8 : 4;
  const bool wide = rows_of(p.dweight, p.dim, bf16 ? 2 : 4, most) &&
                    rows_of(p.dy, p.dim, io_bf16 ? 2 : 4, most);
  const Layout l = layout_of(p.tokens, p.dim, bf16);
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
  cudaError_t e;
  if (p.tokens <= kRankMost) {
    a.passes = 1;
    const int64_t ctas = (p.tokens + kRankTokens - 1) / kRankTokens;
    // in plain stream order too
    embed_rank_kernel<<<static_cast<unsigned>(ctas), kRankWarps * 32, 0, s>>>(a);
    e = cudaGetLastError();
  } else {
    e = sort(a, s);
  }
  if (e != cudaSuccess) return e;
  if (!p.add) {
    const int64_t bytes = p.vocab * p.dim * (bf16 ? 2 : 4);
    const int64_t need = bytes / (16 * kFillThreads) + 1, most = int64_t(kSms) * 8;
    e = launch_after(embed_fill_kernel, static_cast<unsigned>(need < most ? need : most),
                     kFillThreads, 0, s, static_cast<char*>(p.dweight), bytes);
    if (e != cudaSuccess) return e;
  }
  SumArgs b = {};
  b.sorted = a.passes & 1 ? a.even : a.odd;
  b.dy = p.dy; b.dweight = p.dweight;
  b.part = reinterpret_cast<float*>(ws + l.part);
  b.tokens = p.tokens; b.vocab = p.vocab; b.dim = p.dim;
  b.windows = l.windows; b.window = l.window;
  b.scale = p.scale;
  const auto pick = [&](auto* onto, auto* fresh) { return p.add ? onto(b, s) : fresh(b, s); };
  if (!bf16)
    return wide ? pick(sum<float, float, 4, true>, sum<float, float, 4, false>)
                : pick(sum<float, float, 1, true>, sum<float, float, 1, false>);
  if (io_bf16)
    return wide ? pick(sum<bf, bf, 8, true>, sum<bf, bf, 8, false>)
                : pick(sum<bf, bf, 1, true>, sum<bf, bf, 1, false>);
  return wide ? pick(sum<bf, float, 8, true>, sum<bf, float, 8, false>)
              : pick(sum<bf, float, 1, true>, sum<bf, float, 1, false>);
}

}  // namespace ssm
