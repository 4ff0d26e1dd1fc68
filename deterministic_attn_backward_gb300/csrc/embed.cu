// embed.cu -- the embedding lookup and its gradient.
//
//   forward   out_t = scale * W[id_t]
//   gradient  dW_v  = scale * sum over t with id_t = v of dOut_t
//
// Both are bandwidth-bound: the forward reads the named rows and writes one
// row a token, the gradient reads one row a token and writes (dense) every row
// of the table or (accumulating) the named ones.
//
// The gradient's sums are taken in a fixed order, as the attention backward's
// dQ is: the tokens of a row in ascending order, in f32, by segments whose
// bounds depend on their number alone, the segments' sums in ascending order.
// So the bits do not depend on the grid or on which CTA ran first.  Integer
// atomics only hand out places; no float is added atomically.
//
// For few tokens one launch does it all (grad_few_kernel).  Beyond:
//   zero      clears the counts (dense: of all rows; accumulating: of the
//             rows the tokens name, so that it costs nothing in the table's
//             size) and the cursors
//   count     per token: how many tokens its row has so far (any order)
//   alloc     per row that has tokens: a run of places in the token list, and
//             its work items, one for every segment of the run
//   place     the tokens into their rows' runs: those of up to 32 tokens in any
//             order, the others ascending.  Dense: the rows without a token
//             are zeroed by the same launch, so that the writes (most of the
//             traffic of a large table) cover the latency of the rest.
//   sum       adds the rows of dOut of each run or segment, a warp each; where
//             there is much to read in long rows, streams them, in the order of
//             the runs, through rings in shared memory.  The short runs' tokens
//             are sorted on the way
//   join      adds the sums of a long run's segments
// Each of these launches may start while the one before it ends.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "dab.h"
#include "host.h"
#include "vec.cuh"

namespace dab {
namespace {

constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr uint32_t kDetailToken = 0x05000000u;  // a token outside the table
constexpr int kSegment = 32;                    // tokens of a segment, up to kSegment^2 tokens a run
constexpr int kSortRun = 8192;                  // runs up to this are sorted in shared memory

// Up to kFewTokens tokens, and as long as a search of all of them for every token
// and piece of a row takes at most kFewSteps, one launch does it all.  One launch
// against several, bf16 rows added to 1000 of f32, frequencies as 1 / rank: 1024
// tokens of width 2048 12.1 us against 15.1, at the bound 2048 of 512 14.2 against
// 15.3 (f32 rows 16.9 against 16.2); beyond it 2048 of 1024 17.0 against 15.9, but
// 1500 of 1024 12.5 against 15.3 and 1024 of 4096 16.3 against 17.7.
constexpr int kFewTokens = 2048;
constexpr long long kFewSteps = 1ll << 23;
// Up to this many tokens, long runs are gathered by walking all tokens, a CTA for
// each run; beyond, they are scattered and sorted by a launch of their own.  Walking
// against sorting, 65536 tokens of width 64, frequencies as 1 / rank: 40 us against
// 46 (1000 rows), 51 against 55 (131072).  How many long runs there are is known on
// the device only, so the rule cannot look at it: 1638 rows named evenly, more long
// runs than CTAs, take 73 us for 41.
constexpr long long kWalkTokens = 65536;

// Cursors, in the header's padding: short runs' places and short runs share one
// 64-bit word (pad[0], pad[1]), long runs and their segments another (pad[2],
// pad[3]).  Short runs take places from the front of the token list, one after
// the other in the order of their items, long runs from its back.  kCurOutside
// is set when a token is outside the table; the last launch reports it, because
// an error in the status word ends the waits of the launches before.
enum : int { kCurPlace = 0, kCurShort = 1, kCurRun = 2, kCurLong = 3, kCurBack = 4, kCurUnit = 5, kCurOutside = 6,
             kCursors = 7 };

// A short run (up to kSegment tokens): its row, and where its tokens are; or a
// segment of a long run: its run, and where its tokens are.  Segment s of all
// long runs' has its sum at partial[s].
struct Item {
  uint32_t owner, start, len, pad;
};
struct Run {  // a long run: its row, its first segment, its tokens and where they are
  uint32_t row, first, tokens, start;
};

__device__ __forceinline__ long long token(const void* ids, int wide, long long t) {
  return wide ? static_cast<const long long*>(ids)[t] : (long long)static_cast<const int*>(ids)[t];
}

// Tokens of a segment of a run of c: kSegment, or for long runs the power of
// two next to sqrt(c), so that the segments and their sums are equally many.
__device__ __forceinline__ uint32_t segment_len(uint32_t c) {
  uint32_t s = kSegment;
  while ((unsigned long long)s * s < c) s *= 2;
  return s;
}

// ------------------------------------------------------------------ forward
// A CTA takes `group` consecutive tokens; thread = VEC elements of a row, two to
// four of them in flight (f32 to bf16 rows of 16 KB: 76 us with two vectors of
// eight, 80 with four, 86 with four of four elements, 32768 tokens).
template <typename TI, typename TO, int VEC, typename Id>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const Id* __restrict__ ids,
                                                        const TI* __restrict__ table, TO* __restrict__ out,
                                                        long long n, long long rows, int width, int group,
                                                        float scale, WsHeader* __restrict__ hdr) {
  const long long t0 = (long long)blockIdx.x * group;
  const int here = (int)min((long long)group, n - t0);
  const int vecs = width / VEC;
  const int total = here * vecs;
  constexpr int kFly = VEC == 8 ? 2 : 4;
  for (int i0 = threadIdx.x; i0 < total; i0 += kFly * 256) {
    // no load depends on a condition (past the end: the last vector again;
    // outside the table: its first row), or each would wait for the other
    typename Row<TI, VEC>::Raw raw[kFly];
    bool ok[kFly];
    int at[kFly], col[kFly];
    Id id[kFly];
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      const int i = min(i0 + u * 256, total - 1);
      at[u] = i / vecs;
      col[u] = (i - at[u] * vecs) * VEC;
      id[u] = ids[t0 + at[u]];
    }
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      ok[u] = id[u] >= 0 && id[u] < rows;
      raw[u] = Row<TI, VEC>::load(table + (size_t)(ok[u] ? id[u] : 0) * width + col[u]);
    }
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      if (i0 + u * 256 >= total) continue;
      float v[VEC];
      if (ok[u]) {
        Row<TI, VEC>::unpack(raw[u], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] *= scale;
      } else {
        if (hdr != nullptr && col[u] == 0) raise_error(hdr, kStatusBounds, kDetailToken);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = 0.f;
      }
      Row<TO, VEC>::store(out + (size_t)(t0 + at[u]) * width + col[u], v);
    }
  }
}

// A table without rows: every token is outside it.
__global__ void __launch_bounds__(256) embed_none_kernel(uint8_t* __restrict__ out, size_t bytes,
                                                         WsHeader* __restrict__ hdr) {
  const size_t tid = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (tid == 0 && hdr != nullptr) raise_error(hdr, kStatusBounds, kDetailToken);
  for (size_t i = tid; i < bytes; i += (size_t)gridDim.x * 256) out[i] = 0;
}

// ----------------------------------------------------------------- gradient
struct GradParams {
  const void* ids;
  int wide;
  long long n, rows, padding;
  int width, pieces;  // pieces: parts of a row that one warp sums
  int accumulate;
  float scale;
  WsHeader* hdr;
  uint32_t *count, *start;        // [rows]
  uint32_t *key, *slot, *list;    // [n]; key: the token's row or kNone
  Item *shorts, *longs;           // short runs, and the segments of long ones
  Run* runs;                      // long runs
  float* partial;                 // [segments][width]
};

// The row of token t, or kNone when it has no gradient.
__device__ __forceinline__ uint32_t grad_row(const GradParams& p, long long t, bool& outside) {
  const long long id = token(p.ids, p.wide, t);
  outside = id < 0 || id >= p.rows;
  return (outside || id == p.padding) ? kNone : (uint32_t)id;
}

__global__ void __launch_bounds__(256) grad_zero_kernel(const GradParams p) {
  grid_launch_dependents();
  const long long tid = (long long)blockIdx.x * 256 + threadIdx.x, all = (long long)gridDim.x * 256;
  if (tid == 0) {
    p.hdr->status = 0u;
    p.hdr->detail = 0u;
  }
  if (tid < kCursors) p.hdr->pad[tid] = 0u;
  if (p.accumulate) {
    for (long long t = tid; t < p.n; t += all) {
      bool outside;
      const uint32_t v = grad_row(p, t, outside);
      if (v != kNone) p.count[v] = 0u;
    }
  } else {
    for (long long v = tid; v < p.rows; v += all) p.count[v] = 0u;
  }
}

// A CTA counts the tokens of a row among its own in a small table first, so that
// a row that many tokens name takes one atomic a CTA (one each and the L2
// handles them one by one).  Rows that find their entry taken count directly.
constexpr int kCountEach = 2;
constexpr int kCountTable = 1024;
__global__ void __launch_bounds__(256) grad_count_kernel(const GradParams p) {
  __shared__ uint32_t key[kCountTable], num[kCountTable];
  grid_launch_dependents();
  const long long t0 = (long long)blockIdx.x * (256 * kCountEach) + threadIdx.x;
  uint32_t v[kCountEach], local[kCountEach], base[kCountEach];
  int entry[kCountEach];
  bool claimed[kCountEach], outside = false;
#pragma unroll
  for (int i = 0; i < kCountEach; ++i) {
    const long long t = t0 + i * 256;
    bool out = false;
    v[i] = t < p.n ? grad_row(p, t, out) : kNone;
    outside |= out;
  }
#pragma unroll
  for (int i = threadIdx.x; i < kCountTable; i += 256) {
    key[i] = kNone;
    num[i] = 0u;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCountEach; ++i) {
    entry[i] = -1;
    claimed[i] = false;
    if (v[i] == kNone) continue;
    const int h = (int)((v[i] * 2654435761u) >> 22);
    const uint32_t had = atomicCAS(&key[h], kNone, v[i]);
    claimed[i] = had == kNone;
    if (claimed[i] || had == v[i]) {
      entry[i] = h;
      local[i] = atomicAdd(&num[h], 1u);
    }
  }
  __syncthreads();
  grid_wait();
  if (outside) p.hdr->pad[kCurOutside] = 1u;
  // the thread that claimed an entry counts it, beside the rows without one
#pragma unroll
  for (int i = 0; i < kCountEach; ++i)
    if (v[i] != kNone && (claimed[i] || entry[i] < 0)) base[i] = atomicAdd(&p.count[v[i]], claimed[i] ? num[entry[i]] : 1u);
#pragma unroll
  for (int i = 0; i < kCountEach; ++i)
    if (claimed[i]) num[entry[i]] = base[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCountEach; ++i) {
    const long long t = t0 + i * 256;
    if (t >= p.n) continue;
    p.key[t] = v[i];
    if (v[i] != kNone) p.slot[t] = entry[i] >= 0 ? num[entry[i]] + local[i] : base[i];
  }
}

// Exclusive sum over the warp, and its total.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x, int lane, uint32_t& total) {
  uint32_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  return s - x;
}

// The token that took a row's first place makes the row's run.  The places and
// the short runs of a CTA take one atomic together, the long runs of a warp two.
__global__ void __launch_bounds__(256) grad_alloc_kernel(const GradParams p) {
  __shared__ uint32_t sums[2][8];
  __shared__ uint32_t base[2];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  const uint32_t v = t < p.n ? p.key[t] : kNone;
  const uint32_t slot = t < p.n ? p.slot[t] : kNone;
  const bool first = v != kNone && slot == 0u;
  const uint32_t c = first ? p.count[v] : 0u;
  const bool longer = c > (uint32_t)kSegment, brief = first && !longer;
  const uint32_t len = segment_len(c), segs = longer ? (c + len - 1) / len : 0u;
  uint32_t all, all_runs, all_segs, all_back;
  uint32_t start = warp_scan(brief ? c : 0u, lane, all);
  if (lane == 0) sums[0][warp] = all;
  uint32_t item = warp_scan(brief ? 1u : 0u, lane, all);
  if (lane == 0) sums[1][warp] = all;
  uint32_t run = warp_scan(longer ? 1u : 0u, lane, all_runs), seg = warp_scan(segs, lane, all_segs);
  uint32_t back = warp_scan(longer ? c : 0u, lane, all_back);
  unsigned long long got = 0;
  uint32_t got_back = 0;
  if (lane == 0 && all_runs != 0) {
    got = atomicAdd(reinterpret_cast<unsigned long long*>(&p.hdr->pad[kCurRun]),
                    (unsigned long long)all_runs | (unsigned long long)all_segs << 32);
    got_back = atomicAdd(&p.hdr->pad[kCurBack], all_back);
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t a_all, b_all;
    const uint32_t a = warp_scan(lane < 8 ? sums[0][lane] : 0u, lane, a_all);
    const uint32_t b = warp_scan(lane < 8 ? sums[1][lane] : 0u, lane, b_all);
    if (lane < 8) {
      sums[0][lane] = a;
      sums[1][lane] = b;
    }
    if (lane == 0 && a_all != 0) {
      const unsigned long long x = atomicAdd(reinterpret_cast<unsigned long long*>(&p.hdr->pad[kCurPlace]),
                                             (unsigned long long)a_all | (unsigned long long)b_all << 32);
      base[0] = (uint32_t)x;
      base[1] = (uint32_t)(x >> 32);
    }
  }
  __syncthreads();
  if (brief) {
    start += base[0] + sums[0][warp];
    p.start[v] = start;
    p.shorts[item + base[1] + sums[1][warp]] = Item{v, start, c, 0u};
  }
  got = __shfl_sync(0xffffffffu, got, 0);
  got_back = __shfl_sync(0xffffffffu, got_back, 0);
  if (!longer) return;
  start = (uint32_t)p.n - (got_back + back + c);
  p.start[v] = start;
  run += (uint32_t)got;
  seg += (uint32_t)(got >> 32);
  p.runs[run] = Run{v, seg, c, start};
  for (uint32_t s = 0; s < segs; ++s) p.longs[seg + s] = Item{run, start + s * len, min(len, c - s * len), 0u};
}

// A run's tokens in ascending order into its places, by walking all tokens and
// keeping those of its row: eight a thread and step, the next step's loads in
// flight.  (n reads from the L2: 1.3 us per 8192 tokens.)
__device__ __forceinline__ void walk_run(const GradParams& p, uint32_t row, uint32_t start, uint32_t* warp_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint4 none = make_uint4(kNone, kNone, kNone, kNone);
  const uint4* keys = reinterpret_cast<const uint4*>(p.key);
  const long long quads = p.n / 4;  // whole ones; the rest of the tokens is handled below
  auto fetch = [&](long long t0, uint4 (&k)[2]) {
    const long long q = t0 / 4 + tid * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k[i] = none;
      if (q + i < quads) {
        k[i] = __ldcg(keys + q + i);
      } else if (q + i == quads) {
        const long long t = quads * 4;
        if (t < p.n) k[i].x = __ldcg(p.key + t);
        if (t + 1 < p.n) k[i].y = __ldcg(p.key + t + 1);
        if (t + 2 < p.n) k[i].z = __ldcg(p.key + t + 2);
      }
    }
  };
  uint4 next[2];
  fetch(0, next);
  uint32_t kept = 0;
  for (long long t0 = 0; t0 < p.n; t0 += 1024 * 8) {
    const uint32_t k[8] = {next[0].x, next[0].y, next[0].z, next[0].w, next[1].x, next[1].y, next[1].z, next[1].w};
    if (t0 + 1024 * 8 < p.n) fetch(t0 + 1024 * 8, next);
    uint32_t hit = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) hit |= (k[e] == row ? 1u : 0u) << e;
    uint32_t total, all;
    uint32_t at = warp_scan((uint32_t)__popc(hit), lane, total);
    if (lane == 0) warp_sum[warp] = total;
    __syncthreads();
    const uint32_t before = warp_scan(warp_sum[lane], lane, all);
    at += kept + __shfl_sync(0xffffffffu, before, warp);
    kept += all;
    __syncthreads();
    while (hit) {
      const int e = __ffs(hit) - 1;
      hit &= hit - 1;
      p.list[start + at++] = (uint32_t)(t0 + tid * 8 + e);
    }
  }
}

// Zeros a row, with the widest stores its length allows.
template <typename TO>
__device__ __forceinline__ void zero_row(TO* dst, int width, int lane) {
  constexpr int kWide = 16 / sizeof(TO);
  if (width % kWide == 0) {
    uint4* q = reinterpret_cast<uint4*>(dst);
#pragma unroll 4
    for (int i = lane; i < width / kWide; i += 32) q[i] = make_uint4(0u, 0u, 0u, 0u);
  } else {
#pragma unroll 4
    for (int i = lane; i < width; i += 32) dst[i] = TO(0.f);
  }
}

// The rows without a token, zeroed (dense gradients): a warp takes every
// `warps`-th row, the counts of 32 of them at a time.
template <typename TO>
__device__ __forceinline__ void zero_rows(const GradParams& p, TO* grad) {
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  const long long warp = (long long)(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  for (long long v0 = warp; v0 < p.rows; v0 += 32 * warps) {
    const long long mine = v0 + lane * warps;
    uint32_t todo = __ballot_sync(0xffffffffu, mine < p.rows && p.count[mine] == 0u);
    while (todo) {
      const int k = __ffs(todo) - 1;
      todo &= todo - 1;
      zero_row(grad + (size_t)(v0 + k * warps) * p.width, p.width, lane);
    }
  }
}

// Tokens into the runs, and zeros into the rows that have none.  walk: long
// runs are gathered in order here; otherwise all tokens are scattered, and
// grad_order_kernel sorts the long runs.
template <typename TO>
__global__ void __launch_bounds__(1024, 2) grad_place_kernel(const GradParams p, TO* __restrict__ grad, int walk) {
  __shared__ uint32_t warp_sum[32];
  grid_launch_dependents();
  grid_wait();
  if (walk) {
    const uint32_t n_long = p.hdr->pad[kCurRun];
    for (uint32_t r = blockIdx.x; r < n_long; r += gridDim.x) {
      const Run run = p.runs[r];
      walk_run(p, run.row, run.start, warp_sum);
    }
  }
  const long long all = (long long)gridDim.x * 1024;
  for (long long t = (long long)blockIdx.x * 1024 + threadIdx.x; t < p.n; t += all) {
    const uint32_t v = p.key[t];
    if (v == kNone || (walk && p.count[v] > (uint32_t)kSegment)) continue;
    p.list[p.start[v] + p.slot[t]] = (uint32_t)t;
  }
  if (!p.accumulate) zero_rows(p, grad);
}

// Whether a run of c tokens (of n in all) is sorted sooner by a bitonic sort in
// shared memory than by walking all tokens.  A step of the sort takes 0.1 us up
// to 2048 tokens and with their number beyond; 8192 tokens of the walk 1.3 us.
__device__ __forceinline__ bool sort_run(uint32_t c, long long n, uint32_t& size) {
  int log = 6;
  while ((1u << log) < c) ++log;
  size = 1u << log;
  const long long steps = (long long)(log * (log + 1) / 2) * (size > 2048 ? size / 2048 : 1);
  return c <= (uint32_t)kSortRun && steps <= 13 * ((n + 8191) / 8192);
}

// Long runs of scattered tokens into ascending order (more than kWalkTokens
// tokens).
__global__ void __launch_bounds__(1024) grad_order_kernel(const GradParams p) {
  __shared__ uint32_t key[kSortRun];
  __shared__ uint32_t warp_sum[32];
  grid_launch_dependents();
  grid_wait();
  const int tid = threadIdx.x;
  const uint32_t n_long = p.hdr->pad[kCurRun];
  for (uint32_t r = blockIdx.x; r < n_long; r += gridDim.x) {
    const Run run = p.runs[r];
    const uint32_t start = run.start, c = run.tokens;
    uint32_t size;
    if (!sort_run(c, p.n, size)) {
      walk_run(p, run.row, start, warp_sum);
      continue;
    }
    for (uint32_t i = tid; i < size; i += 1024) key[i] = i < c ? p.list[start + i] : kNone;
    __syncthreads();
    for (uint32_t k = 2; k <= size; k *= 2) {
      for (uint32_t j = k / 2; j > 0; j /= 2) {
        for (uint32_t i = tid; i < size / 2; i += 1024) {
          const uint32_t a = 2 * i - (i & (j - 1)), b = a + j;
          const uint32_t x = key[a], y = key[b];
          if ((x > y) == ((a & k) == 0)) {
            key[a] = y;
            key[b] = x;
          }
        }
        __syncthreads();
      }
    }
    for (uint32_t i = tid; i < c; i += 1024) p.list[start + i] = key[i];
    __syncthreads();
  }
}

template <typename TO, int VEC>
__device__ __forceinline__ void write_row(const GradParams& p, TO* grad, uint32_t row, int col, float (&v)[VEC]) {
  TO* dst = grad + (size_t)row * p.width + col;
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] *= p.scale;
  if (p.accumulate) {
    float old[VEC];
    Row<TO, VEC>::unpack(Row<TO, VEC>::load(dst), old);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] += old[e];
  }
  Row<TO, VEC>::store(dst, v);
}

// Adds kRows rows, list(k0), list(k0 + 1), ..., in that order: all loads, then
// the sums.  No load depends on a condition (a lane behind the row's end reads
// its last elements), or each would wait for the one before it.
template <typename TI, int VEC, int NV, int kRows, typename F>
__device__ __forceinline__ void add_batch(const TI* __restrict__ dout, int width, const int (&col)[NV], int k0, F&& list,
                                          float (&acc)[NV][VEC]) {
  typename Row<TI, VEC>::Raw raw[kRows][NV];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const TI* row = dout + (size_t)list(k0 + k) * width;
#pragma unroll
    for (int x = 0; x < NV; ++x) raw[k][x] = Row<TI, VEC>::load(row + col[x]);
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
#pragma unroll
    for (int x = 0; x < NV; ++x) {
      float f[VEC];
      Row<TI, VEC>::unpack(raw[k][x], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[x][e] += f[e];
    }
  }
}

// Adds rows list(0), list(1), ... list(m - 1) of dout, in that order, to acc:
// a lane's vectors of columns col0, col0 + 32 * VEC, ...; up to kFly rows in
// flight.
template <typename TI, int VEC, int NV, int kFly, typename F>
__device__ __forceinline__ void add_rows(const TI* __restrict__ dout, int width, int col0, int m, F&& list,
                                         float (&acc)[NV][VEC]) {
  int col[NV];
#pragma unroll
  for (int x = 0; x < NV; ++x) col[x] = min(col0 + x * 32 * VEC, width - VEC);
  int k = 0;
#pragma unroll 1
  for (; k + kFly <= m; k += kFly) add_batch<TI, VEC, NV, kFly>(dout, width, col, k, list, acc);
  if constexpr (kFly > 8) {
    if (k + 8 <= m) {
      add_batch<TI, VEC, NV, 8>(dout, width, col, k, list, acc);
      k += 8;
    }
  }
  if constexpr (kFly > 4) {
    if (k + 4 <= m) {
      add_batch<TI, VEC, NV, 4>(dout, width, col, k, list, acc);
      k += 4;
    }
  }
  if (k + 2 <= m) {
    add_batch<TI, VEC, NV, 2>(dout, width, col, k, list, acc);
    k += 2;
  }
  if (k < m) add_batch<TI, VEC, NV, 1>(dout, width, col, k, list, acc);
}

template <int NV, int VEC>
__device__ __forceinline__ void clear(float (&acc)[NV][VEC]) {
#pragma unroll
  for (int x = 0; x < NV; ++x)
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[x][e] = 0.f;
}

// The k-th smallest of a warp's `m` first values (all different) in lane k.
__device__ __forceinline__ uint32_t warp_sort(uint32_t t, int m, int lane) {
  int rank = 0;
  for (int k = 0; k < m; ++k) rank += __shfl_sync(0xffffffffu, t, k) < t ? 1 : 0;
  uint32_t sorted = t;
  for (int k = 0; k < m; ++k) {
    const uint32_t tk = __shfl_sync(0xffffffffu, t, k);
    if (__shfl_sync(0xffffffffu, rank, k) == lane) sorted = tk;
  }
  return sorted;
}

// The sums of runs and segments, any width: one warp per item and piece of the
// row (NV vectors of VEC elements per lane), long runs' segments first.  128
// bytes a lane in flight (64: up to a quarter slower where runs are long; 256:
// a tenth where they are short).
template <typename TI, typename TO, int VEC, int NV>
__global__ void __launch_bounds__(256) grad_sum_kernel(const GradParams p, const TI* __restrict__ dout,
                                                       TO* __restrict__ grad) {
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x & 31;
  const unsigned long long warp = ((unsigned long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  const unsigned long long warps = (unsigned long long)gridDim.x * 8;
  constexpr int kLaneBytes = NV * VEC * (int)sizeof(TI), kFly = kLaneBytes < 16 ? 8 : 128 / kLaneBytes;
  const uint32_t n_long = p.hdr->pad[kCurLong];
  const unsigned long long total = (unsigned long long)(n_long + p.hdr->pad[kCurShort]) * p.pieces;
  auto fetch = [&](unsigned long long w) {
    const uint32_t i = (uint32_t)(w / (uint32_t)p.pieces);
    return w >= total ? Item{0u, 0u, 0u, 0u} : i < n_long ? p.longs[i] : p.shorts[i - n_long];
  };
  auto tokens = [&](const Item& x) { return (uint32_t)lane < x.len ? p.list[x.start + lane] : kNone; };
  // the item after the next one and the next one's tokens are on their way while
  // an item's rows are added
  Item it = fetch(warp), it1 = fetch(warp + warps);
  uint32_t t = tokens(it);
  for (unsigned long long w = warp; w < total; w += warps) {
    const uint32_t t1 = tokens(it1);
    const Item it2 = fetch(w + 2 * warps);
    const uint32_t i = (uint32_t)(w / (uint32_t)p.pieces);
    const int piece = (int)(w - (unsigned long long)i * p.pieces);
    const int col0 = piece * (32 * VEC * NV) + lane * VEC;
    float acc[NV][VEC];
    clear(acc);
    for (uint32_t i0 = 0; i0 < it.len; i0 += 32) {
      const int m = (int)min(32u, it.len - i0);
      uint32_t ahead = kNone;
      if (i0 + 32 + (uint32_t)lane < it.len) ahead = p.list[it.start + i0 + 32 + lane];
      if (i >= n_long && m > 1) t = warp_sort(t, m, lane);
      add_rows<TI, VEC, NV, kFly>(dout, p.width, col0, m, [&](int k) { return __shfl_sync(0xffffffffu, t, k & 31); }, acc);
      t = ahead;
    }
#pragma unroll
    for (int x = 0; x < NV; ++x) {
      const int col = col0 + x * 32 * VEC;
      if (col >= p.width) continue;
      if (i >= n_long) write_row<TO, VEC>(p, grad, it.owner, col, acc[x]);
      else Row<float, VEC>::store(p.partial + (size_t)i * p.width + col, acc[x]);
    }
    it = it1;
    it1 = it2;
    t = t1;
  }
}

// The same for much to read in long rows, as a stream.  A CTA takes a piece of
// the row's columns (16 a lane) of a segment or of kGroup short runs at a time,
// whichever is next.  Warp 0 reads the items and their tokens ahead,
// sorts the short runs' and copies the named rows' pieces, one bulk copy each,
// into a ring of stages of a few rows; the other warps add the rows of a stage
// once they are all there, and write a row after its last token.  So the
// ring's 48 KB a CTA (192 KB an SM; 44 KB hold the card's bandwidth at a
// microsecond's latency) stay in flight across runs of any length, where a warp
// per run waited for its item, tokens and rows in turn.  Stages of several rows,
// because a wait, the row's record and the release cost a warp 40 instructions:
// once a row they bound the kernel.
constexpr int kGroup = 4;
constexpr int kRingBytes = 49152;
constexpr int kLaneColumns = 16;
constexpr int kMaxStages = 32;
constexpr int kStageRows = 4;  // at most
constexpr uint32_t kMetaLast = 1u << 31, kMetaPartial = 1u << 30, kMetaNone = 1u << 29;  // beside the piece

struct StreamSmem {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint2 meta[kMaxStages][kStageRows];
  uint32_t tokens[kGroup * kSegment], sorted[kGroup * kSegment];
  int end[kMaxStages];
  int abort;
};

// Rows of a stage: four, or fewer where rows are so long that the ring would have
// under four stages.
__host__ __device__ constexpr int stage_rows(int slot_bytes) {
  return kRingBytes / slot_bytes >= 4 * kStageRows ? kStageRows : kStageRows / 2;
}

template <typename TI, typename TO, int VEC, int kWarps>
__global__ void __launch_bounds__(32 * (kWarps + 1), 4) grad_stream_kernel(const GradParams p,
                                                                           const TI* __restrict__ dout,
                                                                           TO* __restrict__ grad) {
  constexpr int kPiece = kWarps * 32 * kLaneColumns;
  constexpr int kSlot = kPiece * (int)sizeof(TI);
  constexpr int kRows = stage_rows(kSlot);
  constexpr int kStages = kRingBytes / kSlot / kRows < kMaxStages ? kRingBytes / kSlot / kRows : kMaxStages;
  // rows issued at a time, one a lane: half the ring, while the other half is added
  constexpr int kStep = kStages / 2 * kRows < 32 ? kStages / 2 * kRows : 32;
  static_assert(kStep % kRows == 0 && kStages >= 2, "ring");
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  StreamSmem* sh = reinterpret_cast<StreamSmem*>(smem + kRingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh->full[i], kRows);
      mbar_init(&sh->empty[i], kWarps);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_launch_dependents();
  grid_wait();
  constexpr unsigned long long kTimeout = 2000000000ull;
  const WaitCtl wc{&sh->abort, p.hdr, kTimeout};

  if (warp == 0) {
    const uint32_t n_long = p.hdr->pad[kCurLong], n_short = p.hdr->pad[kCurShort];
    const uint32_t pieces = (uint32_t)p.pieces;
    const unsigned long long units = (unsigned long long)(n_long + (n_short + kGroup - 1) / kGroup) * pieces;
    const bool prefetch = p.accumulate && p.width * sizeof(TO) % 16 == 0;
    int stage0 = 0;      // the next stage to fill
    uint32_t turn0 = 0;  // how often that one was filled
    bool ok = true;
    // Copies m <= kStep rows, a lane each, into the next stages, kRows a stage;
    // the rows that the last one lacks arrive empty.
    auto issue = [&](uint32_t token, uint32_t dest, uint32_t flags, int m, uint32_t piece) {
      const int used = (m + kRows - 1) / kRows;
      int stage = stage0 + lane / kRows;
      uint32_t turn = turn0;
      if (stage >= kStages) {
        stage -= kStages;
        ++turn;
      }
      const bool part = lane < used * kRows;
      bool mine = true;
      if (part && turn != 0) mine = mbar_wait(&sh->empty[stage], (turn - 1) & 1, wc, 1);
      if (!__all_sync(0xffffffffu, mine)) return false;
      if (part) {
        const int slot = lane % kRows;
        sh->meta[stage][slot] = make_uint2(dest, lane < m ? flags | piece : kMetaNone);
        if (slot == 0) sh->end[stage] = 0;
        if (lane < m) {
          const uint32_t col = piece * (uint32_t)kPiece;
          const uint32_t bytes = min((uint32_t)kPiece, (uint32_t)p.width - col) * (uint32_t)sizeof(TI);
          mbar_arrive_expect_tx(&sh->full[stage], bytes);
          bulk_load(ring + (stage * kRows + slot) * kSlot, dout + (size_t)token * p.width + col, bytes, &sh->full[stage]);
          // accumulating: the row that this token is the last of will be read
          if (prefetch && (flags & (kMetaLast | kMetaPartial)) == kMetaLast)
            bulk_prefetch(grad + (size_t)dest * p.width + col, bytes / (uint32_t)sizeof(TI) * (uint32_t)sizeof(TO));
        } else {
          mbar_arrive(&sh->full[stage]);
        }
      }
      stage0 += used;
      if (stage0 >= kStages) {
        stage0 -= kStages;
        ++turn0;
      }
      return true;
    };
    // The next unit; a unit: lane g its g-th short run, or every lane its segment.
    auto take = [&]() {
      uint32_t u = 0;
      if (lane == 0) u = atomicAdd(&p.hdr->pad[kCurUnit], 1u);
      return (unsigned long long)__shfl_sync(0xffffffffu, u, 0);
    };
    auto item_of = [&](unsigned long long u) { return (uint32_t)u / pieces; };
    auto fetch = [&](unsigned long long u) {
      if (u >= units) return Item{0u, 0u, 0u, 0u};
      const uint32_t i = item_of(u);
      if (i < n_long) return p.longs[i];
      const uint32_t k = (i - n_long) * kGroup + (uint32_t)lane;
      return lane < kGroup && k < n_short ? p.shorts[k] : Item{0u, 0u, 0u, 0u};
    };
    // its first 32 tokens (those of a group's runs lie one after the other)
    auto first_tokens = [&](const Item& x, bool is_long) {
      const uint32_t start = __shfl_sync(0xffffffffu, x.start, 0);
      uint32_t count = x.len;
      if (!is_long) count = __reduce_add_sync(0xffffffffu, x.len);
      return (uint32_t)lane < count ? p.list[start + (uint32_t)lane] : 0u;
    };
    // Three units under way: while the rows of u are copied, the tokens of u1 and
    // the items of u2 are on their way, and the number of the one after is asked
    // for.  A CTA's first two are its own.
    unsigned long long u = blockIdx.x, u1 = u + gridDim.x, u2 = take() + 2 * gridDim.x;
    Item it = fetch(u), it1 = fetch(u1);
    uint32_t t = first_tokens(it, item_of(u) < n_long);
    while (ok && u < units) {
      const uint32_t t1 = first_tokens(it1, item_of(u1) < n_long);
      const Item it2 = fetch(u2);
      const unsigned long long u3 = u2 < units ? take() + 2 * gridDim.x : u2;
      const uint32_t i = item_of(u), piece = (uint32_t)u - i * pieces;
      if (i < n_long) {
        for (uint32_t x0 = 0; ok && x0 < it.len; x0 += 32) {
          uint32_t ahead = 0;
          if (x0 + 32 + (uint32_t)lane < it.len) ahead = p.list[it.start + x0 + 32 + (uint32_t)lane];
          const int here = (int)min(32u, it.len - x0);
          for (int y = 0; ok && y < here; y += kStep) {
            const int m = min(kStep, here - y);
            const uint32_t tok = __shfl_sync(0xffffffffu, t, (y + lane) & 31);
            ok = issue(tok, i, kMetaPartial | (x0 + (uint32_t)(y + lane) + 1 == it.len ? kMetaLast : 0u), m, piece);
          }
          t = ahead;
        }
      } else {
        const uint32_t first = __shfl_sync(0xffffffffu, it.start, 0);
        const int count = (int)__reduce_add_sync(0xffffffffu, it.len);
        __syncwarp();
        if (lane < count) sh->tokens[lane] = t;
        for (int x = lane + 32; x < count; x += 32) sh->tokens[x] = p.list[first + (uint32_t)x];
        __syncwarp();
        // each token to its place in the order of its run's tokens
        for (int x0 = 0; x0 < count; x0 += 32) {
          const uint32_t x = (uint32_t)(x0 + lane);
          uint32_t a = 0, len = 0;
#pragma unroll
          for (int g = 0; g < kGroup; ++g) {
            const uint32_t ga = __shfl_sync(0xffffffffu, it.start, g) - first, gl = __shfl_sync(0xffffffffu, it.len, g);
            if (gl != 0 && x >= ga) {
              a = ga;
              len = gl;
            }
          }
          if (x < (uint32_t)count) {
            const uint32_t mine = sh->tokens[x];
            uint32_t rank = 0;
            for (uint32_t y = 0; y < len; ++y) rank += sh->tokens[a + y] < mine ? 1u : 0u;
            sh->sorted[a + rank] = mine;
          }
        }
        __syncwarp();
        for (int x0 = 0; ok && x0 < count; x0 += kStep) {
          const uint32_t x = (uint32_t)(x0 + lane);
          const int m = min(kStep, count - x0);
          uint32_t dest = 0, flags = 0;
#pragma unroll
          for (int g = 0; g < kGroup; ++g) {
            const uint32_t ga = __shfl_sync(0xffffffffu, it.start, g) - first, gl = __shfl_sync(0xffffffffu, it.len, g);
            const uint32_t owner = __shfl_sync(0xffffffffu, it.owner, g);
            if (gl != 0 && x >= ga) {
              dest = owner;
              flags = x + 1 == ga + gl ? kMetaLast : 0u;
            }
          }
          ok = issue(lane < m ? sh->sorted[x] : 0u, dest, flags, m, piece);
        }
      }
      u = u1;
      u1 = u2;
      u2 = u3;
      it = it1;
      it1 = it2;
      t = t1;
    }
    if (lane == 0) {
      // every copy lands before the CTA may exit; then the end
      for (int s = 0; s < kStages; ++s) {
        const uint32_t turns = turn0 + (s < stage0 ? 1u : 0u);  // how often stage s was filled
        if (turns != 0) drain_wait(&sh->full[s], (turns - 1) & 1, p.hdr, kTimeout, 21);
      }
      if (ok && (turn0 == 0 || mbar_wait(&sh->empty[stage0], (turn0 - 1) & 1, wc, 2))) {
        sh->end[stage0] = 1;
        for (int r = 0; r < kRows; ++r) mbar_arrive(&sh->full[stage0]);
      }
    }
  } else {
    constexpr int kNv = kLaneColumns / VEC;
    const uint32_t col_in = (uint32_t)((warp - 1) * 32 * kLaneColumns + lane * VEC);  // + 32 * VEC * x
    float acc[kNv][VEC];
    clear(acc);
    int stage = 0;
    uint32_t parity = 0;
    while (warp_wait(&sh->full[stage], parity, wc, 3)) {
      if (sh->end[stage]) break;
      const TI* src = reinterpret_cast<const TI*>(ring + stage * kRows * kSlot) + col_in;
      uint2 meta[kRows];
      typename Row<TI, VEC>::Raw raw[kRows][kNv];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        meta[r] = sh->meta[stage][r];
#pragma unroll
        for (int x = 0; x < kNv; ++x) raw[r][x] = Row<TI, VEC>::load(src + r * kPiece + x * 32 * VEC);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (meta[r].y & kMetaNone) break;  // so are the rows after it
#pragma unroll
        for (int x = 0; x < kNv; ++x) {
          float f[VEC];
          Row<TI, VEC>::unpack(raw[r][x], f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[x][e] += f[e];
        }
        if (meta[r].y & kMetaLast) {
          const uint32_t col = (meta[r].y & 0xFFFFFFu) * (uint32_t)kPiece + col_in;
#pragma unroll
          for (int x = 0; x < kNv; ++x) {
            if (col + x * 32 * VEC < (uint32_t)p.width) {
              if (meta[r].y & kMetaPartial)
                Row<float, VEC>::store(p.partial + (size_t)meta[r].x * p.width + col + x * 32 * VEC, acc[x]);
              else
                write_row<TO, VEC>(p, grad, meta[r].x, (int)(col + x * 32 * VEC), acc[x]);
            }
          }
          clear(acc);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->empty[stage]);
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1;
      }
    }
  }
}

// Adds the sums of a long run's segments, in order: one warp per run and piece of
// 32 * VEC columns, sixteen sums in flight.
template <typename TO, int VEC>
__global__ void __launch_bounds__(256) grad_join_kernel(const GradParams p, TO* __restrict__ grad) {
  grid_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.hdr->pad[kCurOutside] != 0u)
    raise_error(p.hdr, kStatusBounds, kDetailToken);
  const int lane = threadIdx.x & 31;
  const unsigned long long warp = ((unsigned long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  const unsigned long long warps = (unsigned long long)gridDim.x * 8;
  const uint32_t pieces = (uint32_t)(p.width + 32 * VEC - 1) / (32 * VEC);
  const unsigned long long total = (unsigned long long)p.hdr->pad[kCurRun] * pieces;
  for (unsigned long long w = warp; w < total; w += warps) {
    const uint32_t r = (uint32_t)(w / pieces);
    const int col = (int)(w - (unsigned long long)r * pieces) * (32 * VEC) + lane * VEC;
    const Run run = p.runs[r];
    const uint32_t len = segment_len(run.tokens), segs = (run.tokens + len - 1) / len;
    float acc[1][VEC];
    clear(acc);
    add_rows<float, VEC, 1, 16>(p.partial + (size_t)run.first * p.width, p.width, col, (int)segs,
                               [&](int k) { return (uint32_t)k; }, acc);
    if (col < p.width) write_row<TO, VEC>(p, grad, run.row, col, acc[0]);
  }
}

// Up to kFewTokens tokens: every CTA holds all their rows in shared memory, so
// nothing is counted or sorted.  A warp takes a token and a piece of its row;
// if no earlier token names the row, it finds the row's tokens by walking them
// and adds them.  Rows of more than two segments it leaves to the CTA,
// whose warps take a segment each and add the segments' sums in order.  Dense:
// then its share of the rows, zeroed where no token names them.  CTA 0 alone
// reports, so the status needs no reset.
template <typename TI, typename TO, int VEC, int NV>
__global__ void __launch_bounds__(256, 3) grad_few_kernel(const GradParams p, const TI* __restrict__ dout,
                                                          TO* __restrict__ grad) {
  constexpr int kFly = sizeof(TI) == 2 ? 8 : 4;
  constexpr int kPiece = 32 * VEC * NV, kFlags = 2048, kEach = kFewTokens / 256, kOwn = 2 * kSegment;
  __shared__ __align__(16) uint32_t row[kFewTokens];
  __shared__ uint16_t list[kFewTokens];
  __shared__ float part[8][kPiece];
  __shared__ uint8_t named[kFlags];
  __shared__ uint16_t mine[8][kOwn];  // a warp's tokens of its row
  __shared__ int left[8];                 // the token of a row left to the CTA by each warp, or -1
  __shared__ uint32_t sums[8];
  const int n = (int)p.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  {
    uint32_t v[kEach];
    bool outside = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      bool out = false;
      v[e] = e * 256 + tid < n ? grad_row(p, e * 256 + tid, out) : kNone;
      outside |= out;
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) row[e * 256 + tid] = v[e];  // kNone behind the last token
    outside = __syncthreads_or(outside);
    if (blockIdx.x == 0 && tid == 0) {
      p.hdr->status = outside ? kStatusBounds : 0u;
      p.hdr->detail = outside ? kDetailToken : 0u;
    }
  }

  const int units = n * p.pieces, step = (int)gridDim.x * 8;
  for (int u0 = (int)blockIdx.x * 8; u0 < units; u0 += step) {
    // neighbouring warps: other tokens, so that the pieces of a row with many
    // tokens lie in different CTAs
    const int u = u0 + warp, piece = u / n, t = u - piece * n;
    const uint32_t v = u < units ? row[t] : kNone;
    int leave = -1;
    if (v != kNone) {
      int c = 0;
      for (int b = 0; b < n && c <= kOwn; b += 128) {
        // 128 tokens a step, four consecutive ones a lane
        const uint4 r = *reinterpret_cast<const uint4*>(&row[b + 4 * lane]);
        const uint32_t hit = (r.x == v ? 1u : 0u) | (r.y == v ? 2u : 0u) | (r.z == v ? 4u : 0u) | (r.w == v ? 8u : 0u);
        const uint32_t lanes = __ballot_sync(0xffffffffu, hit != 0u);
        if (lanes == 0) continue;
        const int lead = __ffs(lanes) - 1;
        if (c == 0 && b + 4 * lead + __ffs(__shfl_sync(0xffffffffu, hit, lead)) - 1 != t) {
          c = -1;  // an earlier token names the row
          break;
        }
        uint32_t found;
        int at = c + (int)warp_scan((uint32_t)__popc(hit), lane, found);
        for (uint32_t h = hit; h != 0; h &= h - 1, ++at)
          if (at < kOwn) mine[warp][at] = (uint16_t)(b + 4 * lane + __ffs(h) - 1);
        c += (int)found;
      }
      __syncwarp();
      if (c > kOwn) {
        leave = t;
      } else if (c > 0) {
        // one segment, or two and their sum
        const uint32_t t0 = mine[warp][lane], t1 = mine[warp][kSegment + lane];
        const int col0 = piece * kPiece + lane * VEC;
        float acc[NV][VEC];
        clear(acc);
        add_rows<TI, VEC, NV, kFly>(dout, p.width, col0, min(c, kSegment),
                                    [&](int k) { return __shfl_sync(0xffffffffu, t0, k & 31); }, acc);
        if (c > kSegment) {
          float more[NV][VEC];
          clear(more);
          add_rows<TI, VEC, NV, kFly>(dout, p.width, col0, c - kSegment,
                                      [&](int k) { return __shfl_sync(0xffffffffu, t1, k & 31); }, more);
#pragma unroll
          for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[x][e] += more[x][e];
        }
#pragma unroll
        for (int x = 0; x < NV; ++x)
          if (col0 + x * 32 * VEC < p.width) write_row<TO, VEC>(p, grad, v, col0 + x * 32 * VEC, acc[x]);
      }
      __syncwarp();
    }
    if (lane == 0) left[warp] = leave;
    if (!__syncthreads_or(leave >= 0)) continue;
    for (int l = 0; l < 8; ++l) {
      if (left[l] < 0) continue;  // the same in every thread
      const uint32_t v2 = row[left[l]];
      const int pc = (u0 + l) / n;
      // the row's tokens, ascending: kEach consecutive ones a thread
      uint32_t hit = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) hit |= (row[tid * kEach + e] == v2 ? 1u : 0u) << e;
      uint32_t total;
      uint32_t at = warp_scan((uint32_t)__popc(hit), lane, total);
      if (lane == 0) sums[warp] = total;
      __syncthreads();
      int c = 0;
      for (int w = 0; w < 8; ++w) {
        if (w < warp) at += sums[w];
        c += (int)sums[w];
      }
      while (hit) {
        const int e = __ffs(hit) - 1;
        hit &= hit - 1;
        list[at++] = (uint16_t)(tid * kEach + e);
      }
      __syncthreads();
      // eight segments a round; each thread keeps its columns of the row's sum
      constexpr int kCols = (kPiece + 255) / 256;
      const int len = (int)segment_len((uint32_t)c);
      float sum[kCols];
#pragma unroll
      for (int x = 0; x < kCols; ++x) sum[x] = 0.f;
      for (int r0 = 0; r0 < c; r0 += 8 * len) {
        const int first = r0 + warp * len, m = min(len, c - first);
        float acc[NV][VEC];
        clear(acc);
        if (m > 0)
          add_rows<TI, VEC, NV, kFly>(dout, p.width, pc * kPiece + lane * VEC, m,
                                [&](int k) { return (uint32_t)list[min(first + k, c - 1)]; }, acc);
#pragma unroll
        for (int x = 0; x < NV; ++x)
#pragma unroll
          for (int e = 0; e < VEC; ++e) part[warp][x * 32 * VEC + lane * VEC + e] = acc[x][e];
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kCols; ++x) {
          const int col = x * 256 + tid;
          if (col >= kPiece) continue;
          for (int w = 0; w < 8 && r0 + w * len < c; ++w) sum[x] += part[w][col];
        }
        __syncthreads();
      }
#pragma unroll
      for (int x = 0; x < kCols; ++x) {
        const int col = x * 256 + tid;
        float one[1] = {sum[x]};
        if (col < kPiece && pc * kPiece + col < p.width) write_row<TO, 1>(p, grad, v2, pc * kPiece + col, one);
      }
    }
    __syncthreads();
  }

  // dense: this CTA's share of the rows, where no token names them
  if (!p.accumulate) {
    const long long v0 = (long long)blockIdx.x * p.rows / gridDim.x;
    const long long v1 = (long long)(blockIdx.x + 1) * p.rows / gridDim.x;
    for (long long b = v0; b < v1; b += kFlags) {
      const int here = (int)min((long long)kFlags, v1 - b);
      for (int i = tid; i < here; i += 256) named[i] = 0;
      __syncthreads();
      for (int t = tid; t < n; t += 256) {
        const long long i = (long long)row[t] - b;
        if (row[t] != kNone && i >= 0 && i < here) named[i] = 1;
      }
      __syncthreads();
      for (int i = warp; i < here; i += 8)
        if (!named[i]) zero_row(grad + (size_t)(b + i) * p.width, p.width, lane);
      __syncthreads();
    }
  }
}

// Elements a lane takes at a time: eight where rows of eight are whole 16 (bf16)
// or 32 (f32) bytes on both sides.
int vec_of(int width, bool wide_rows) {
  return width % 8 == 0 && wide_rows ? 8 : width % 4 == 0 ? 4 : width % 2 == 0 ? 2 : 1;
}
bool wide_tensor(const void* p, int type) { return type == DAB_BF16 || is_aligned(p, 32); }

template <typename T>
using Plain = std::conditional_t<std::is_same<T, WideF32>::value, float, T>;
template <typename T>
using Wide = std::conditional_t<std::is_same<T, float>::value, WideF32, T>;

constexpr int kNv8 = 1, kNv4 = 2, kNv2 = 4, kNv1 = 4;  // vectors of a lane, by the elements of one
int piece_of(int vec) { return 32 * (vec == 8 ? 8 * kNv8 : vec == 4 ? 4 * kNv4 : vec == 2 ? 2 * kNv2 : kNv1); }

constexpr int kMaxWidth = 1 << 24;

struct GradLayout {
  size_t count, start, key, slot, list, shorts, longs, runs, partial, total;
};

// At most n short runs and n / 33 long ones; a long run of c tokens has at most
// c / 32 + 1 < c / 16 segments.  For few tokens only the header is used, but the
// sizes do not drop there.
bool grad_layout(long long n, long long rows, int width, GradLayout* L) {
  if (n < 0 || rows < 0 || width < 0 || n >= (1ll << 31) || rows >= (1ll << 31) || width > kMaxWidth) return false;
  const size_t N = (size_t)n, V = (size_t)rows;
  const size_t longs = N / (kSegment + 1) + 1, segments = N / (kSegment / 2) + 1;
  size_t off = 256;
  auto place = [&](size_t bytes) {
    const size_t at = off;
    off = round_up_to(off + bytes, 256);
    return at;
  };
  L->count = place(4 * V);
  L->start = place(4 * V);
  L->key = place(4 * N);
  L->slot = place(4 * N);
  L->list = place(4 * N);
  L->shorts = place(sizeof(Item) * N);
  L->longs = place(sizeof(Item) * segments);
  L->runs = place(sizeof(Run) * longs);
  L->partial = place(4 * (size_t)width * segments);
  L->total = off;
  return true;
}

bool float_type(int t) { return t == DAB_BF16 || t == DAB_F32; }
bool index_type(int t) { return t == DAB_I32 || t == DAB_I64; }

template <typename TI, typename TO, typename Id>
cudaError_t launch_embed_fwd(const void* ids, const void* table, void* out, long long n, long long rows, int width,
                             float scale, WsHeader* hdr, bool wide_rows, cudaStream_t stream) {
  // enough tokens a CTA for the vectors a thread has in flight, one at least
  const int vec = vec_of(width, wide_rows), vecs = width / vec;
  long long group = (vec == 8 ? 512 : 1024) / vecs;
  if (group < 1) group = 1;
  const unsigned grid = (unsigned)((n + group - 1) / group);
  auto run = [&](auto kernel) {
    return launch(kernel, grid, 256, stream, false, ids, table, out, n, rows, width, (int)group, scale, hdr);
  };
  switch (vec) {
    case 8: return run(embed_fwd_kernel<Wide<TI>, Wide<TO>, 8, Id>);
    case 4: return run(embed_fwd_kernel<TI, TO, 4, Id>);
    case 2: return run(embed_fwd_kernel<TI, TO, 2, Id>);
  }
  return run(embed_fwd_kernel<TI, TO, 1, Id>);
}

// Whether rows of so many bytes are summed by the stream.  It starts 6 us later
// than a warp per run does, and its copies, which an SM issues one after the
// other, take some 45 ns each.  Whole gradients, the stream against a warp per
// run, bf16 rows added to f32 ones, frequencies as 1 / rank: at 32 MB 8192 of 4 KB
// 42.5 us against 39.2 (dense 67.6 against 70.2) and 32768 of 1 KB 51.1 against
// 43.8; beyond, 16384 of 4 KB into bf16 51.7 against 53.7 (dense 53.7 against 60.8),
// 65536 of them into 131072 rows 160 against 175, where rows are shorter 32768 of 2
// KB 61.9 against 59.1 and 65536 of 1 KB 74.4 against 67.3.
bool streams(long long row_bytes, long long n) {
  return row_bytes % 16 == 0 && row_bytes >= 1024 && row_bytes * n > (1 << 25);
}

template <typename TI, typename TO, int VEC, int NV>
cudaError_t launch_grad(const GradParams& p, const void* dout, void* grad, int sms, cudaStream_t stream) {
  const TI* d = static_cast<const TI*>(dout);
  TO* g = static_cast<TO*>(grad);
  auto ctas = [&](long long work, long long most) {
    return (unsigned)(work < 1 ? 1 : work < most ? work : most);
  };
  const long long warps = p.n * p.pieces, dense_rows = p.accumulate ? 0 : p.rows;
  if (p.n <= kFewTokens && p.n * warps <= kFewSteps)
    return launch(grad_few_kernel<TI, TO, VEC, NV>, ctas((std::max(warps, dense_rows) + 7) / 8, sms * 3), 256, stream,
                  false, p, d, g);
  cudaError_t e = launch(grad_zero_kernel, ctas(((p.accumulate ? p.n : p.rows) + 255) / 256, sms * 8), 256, stream,
                         false, p);
  if (e == cudaSuccess)
    e = launch(grad_count_kernel, (unsigned)((p.n + 256 * kCountEach - 1) / (256 * kCountEach)), 256, stream, true, p);
  if (e == cudaSuccess) e = launch(grad_alloc_kernel, (unsigned)((p.n + 255) / 256), 256, stream, true, p);
  const int walk = p.n <= kWalkTokens ? 1 : 0;
  if (e == cudaSuccess) e = launch(grad_place_kernel<TO>, (unsigned)(2 * sms), 1024, stream, true, p, g, walk);
  if (e == cudaSuccess && !walk) e = launch(grad_order_kernel, (unsigned)(2 * sms), 1024, stream, true, p);
  if constexpr (VEC >= 4) {
    if (e == cudaSuccess && streams((long long)p.width * sizeof(TI), p.n)) {
      auto stream_rows = [&](auto kernel, int threads, std::atomic<uint64_t>& sized) {
        constexpr int kBytes = kRingBytes + (int)sizeof(StreamSmem);
        GradParams q = p;
        const int piece = (threads - 32) * kLaneColumns;
        q.pieces = (p.width + piece - 1) / piece;
        const cudaError_t x = allow_smem(reinterpret_cast<const void*>(kernel), kBytes, sized);
        if (x != cudaSuccess) return x;
        return launch_smem(kernel, (unsigned)(4 * sms), (unsigned)threads, kBytes, stream, true, q,
                           d, g);
      };
      static std::atomic<uint64_t> sized1{0}, sized2{0};
      e = p.width > 32 * kLaneColumns ? stream_rows(grad_stream_kernel<TI, TO, VEC, 2>, 96, sized2)
                                      : stream_rows(grad_stream_kernel<TI, TO, VEC, 1>, 64, sized1);
      if (e == cudaSuccess)
        e = launch(grad_join_kernel<Plain<TO>, 4>, (unsigned)(4 * sms), 256, stream, true, p,
                   static_cast<Plain<TO>*>(grad));
      return e;
    }
  }
  if (e == cudaSuccess)
    e = launch(grad_sum_kernel<TI, TO, VEC, NV>, ctas((warps + 7) / 8, sms * 8), 256, stream, true, p, d, g);
  if (e == cudaSuccess)
    e = launch(grad_join_kernel<Plain<TO>, (VEC > 4 ? 4 : VEC)>, (unsigned)(4 * sms), 256, stream, true, p,
               static_cast<Plain<TO>*>(grad));
  return e;
}

template <typename TI, typename TO>
cudaError_t launch_grad(const GradParams& p, const void* dout, void* grad, bool wide_rows, int sms,
                        cudaStream_t stream) {
  // eight elements a lane of bf16 rows into either type; of f32 rows four (the
  // stream reads them from shared memory 16 bytes at a time)
  constexpr bool kWide = sizeof(TI) == 2;
  switch (vec_of(p.width, kWide && wide_rows)) {
    case 8: return launch_grad<TI, std::conditional_t<kWide, Wide<TO>, TO>, kWide ? 8 : 4, kWide ? kNv8 : kNv4>(p, dout, grad, sms, stream);
    case 4: return launch_grad<TI, TO, 4, kNv4>(p, dout, grad, sms, stream);
    case 2: return launch_grad<TI, TO, 2, kNv2>(p, dout, grad, sms, stream);
  }
  return launch_grad<TI, TO, 1, kNv1>(p, dout, grad, sms, stream);
}

}  // namespace
}  // namespace dab

using namespace dab;

extern "C" dab_status_t dab_embed_fwd(const void* ids, dab_dtype_t ids_type, const void* table,
                                      dab_dtype_t table_type, void* out, dab_dtype_t out_type, int64_t n,
                                      int64_t rows, int width, float scale, void* workspace, size_t ws_bytes,
                                      cudaStream_t stream) {
  GradLayout L;
  if (!index_type(ids_type) || !float_type(table_type) || !float_type(out_type)) return DAB_ERR_INVALID_ARG;
  if (!grad_layout(n, rows, width, &L)) return DAB_ERR_INVALID_ARG;
  if (workspace != nullptr && (ws_bytes < 256 || !is_aligned(workspace, 16))) return DAB_ERR_WORKSPACE;
  const bool nothing = n == 0 || width == 0;
  if (!nothing && (!is_aligned(ids, ids_type == DAB_I64 ? 8 : 4) || !is_aligned(out, 16) ||
                   (rows > 0 && !is_aligned(table, 16))))
    return DAB_ERR_INVALID_ARG;
  if (!device_ready(nullptr)) return DAB_ERR_UNSUPPORTED;
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  cudaError_t e = cudaSuccess;
  if (hdr != nullptr && (e = cudaMemsetAsync(hdr, 0, 16, stream)) != cudaSuccess)
    return record_cuda_error(e, "status reset");
  if (nothing) return DAB_OK;
  const bool wide_rows = wide_tensor(table, table_type) && wide_tensor(out, out_type);
  auto with = [&](auto ti, auto to) {
    using TI = decltype(ti);
    using TO = decltype(to);
    return ids_type == DAB_I64
               ? launch_embed_fwd<TI, TO, long long>(ids, table, out, n, rows, width, scale, hdr, wide_rows, stream)
               : launch_embed_fwd<TI, TO, int>(ids, table, out, n, rows, width, scale, hdr, wide_rows, stream);
  };
  const __nv_bfloat16 h{};
  if (rows == 0)
    e = launch(embed_none_kernel, 256u, 256u, stream, false, out, (size_t)n * width * (out_type == DAB_F32 ? 4 : 2), hdr);
  else if (table_type == DAB_BF16) e = out_type == DAB_BF16 ? with(h, h) : with(h, 0.f);
  else e = out_type == DAB_BF16 ? with(0.f, h) : with(0.f, 0.f);
  return e == cudaSuccess ? DAB_OK : record_cuda_error(e, "embedding lookup launch");
}

extern "C" size_t dab_embed_bwd_workspace_size(int64_t n, int64_t rows, int width) {
  GradLayout L;
  return grad_layout(n, rows, width, &L) ? L.total : 0;
}

extern "C" dab_status_t dab_embed_bwd(const void* ids, dab_dtype_t ids_type, const void* dout,
                                      dab_dtype_t dout_type, void* grad, dab_dtype_t grad_type, int64_t n,
                                      int64_t rows, int width, float scale, int64_t padding, int accumulate,
                                      void* workspace, size_t ws_bytes, cudaStream_t stream) {
  GradLayout L;
  if (!index_type(ids_type) || !float_type(dout_type) || !float_type(grad_type)) return DAB_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return DAB_ERR_INVALID_ARG;
  if (!grad_layout(n, rows, width, &L)) return DAB_ERR_INVALID_ARG;
  // the tokens are read whatever the width, for those outside the table
  if (n > 0 && !is_aligned(ids, ids_type == DAB_I64 ? 8 : 4)) return DAB_ERR_INVALID_ARG;
  if (n > 0 && width > 0 && !is_aligned(dout, 16)) return DAB_ERR_INVALID_ARG;
  if (rows > 0 && width > 0 && !is_aligned(grad, 16)) return DAB_ERR_INVALID_ARG;
  if (!is_aligned(workspace, 16) || ws_bytes < L.total) return DAB_ERR_WORKSPACE;
  int sms = 0;
  if (!device_ready(&sms)) return DAB_ERR_UNSUPPORTED;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  GradParams p;
  p.ids = ids;
  p.wide = ids_type == DAB_I64 ? 1 : 0;
  p.n = n;
  p.rows = rows;
  p.padding = padding;
  p.width = width;
  const bool wide_rows = wide_tensor(grad, grad_type);
  const int piece = piece_of(vec_of(width, dout_type == DAB_BF16 && wide_rows));
  p.pieces = (width + piece - 1) / piece;
  p.accumulate = accumulate;
  p.scale = scale;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.count = reinterpret_cast<uint32_t*>(ws + L.count);
  p.start = reinterpret_cast<uint32_t*>(ws + L.start);
  p.key = reinterpret_cast<uint32_t*>(ws + L.key);
  p.slot = reinterpret_cast<uint32_t*>(ws + L.slot);
  p.list = reinterpret_cast<uint32_t*>(ws + L.list);
  p.shorts = reinterpret_cast<Item*>(ws + L.shorts);
  p.longs = reinterpret_cast<Item*>(ws + L.longs);
  p.runs = reinterpret_cast<Run*>(ws + L.runs);
  p.partial = reinterpret_cast<float*>(ws + L.partial);
  cudaError_t e;
  if (dout_type == DAB_BF16 && grad_type == DAB_BF16)
    e = launch_grad<__nv_bfloat16, __nv_bfloat16>(p, dout, grad, wide_rows, sms, stream);
  else if (dout_type == DAB_BF16)
    e = launch_grad<__nv_bfloat16, float>(p, dout, grad, wide_rows, sms, stream);
  else if (grad_type == DAB_BF16)
    e = launch_grad<float, __nv_bfloat16>(p, dout, grad, wide_rows, sms, stream);
  else
    e = launch_grad<float, float>(p, dout, grad, wide_rows, sms, stream);
  return e == cudaSuccess ? DAB_OK : record_cuda_error(e, "embedding gradient launch");
}
