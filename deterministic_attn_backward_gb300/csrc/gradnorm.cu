// gradnorm.cu -- the global 2-norm of many gradient tensors, and clipping.
//
//   norm = sqrt(sum over all tensors of g^2)
//   g'   = g * min(1, max_norm / (norm + 1e-6))
//
// Bandwidth-bound: the norm needs every gradient before the first can be
// scaled, so clipping reads twice and writes once; what the second pass finds
// in the L2 it need not read from memory, and it walks the elements backwards
// to find as much there as it can.
//
// Every tensor is cut into cells of kCell elements.  Eight consecutive cells of
// the list are a batch (the cells that do not fill a last round of batches are
// shared out evenly), and CTA s of kCtas takes the batches s, s +
// kCtas, ...: balanced whatever the tensors' sizes, all CTAs at neighbouring
// addresses at a time (a contiguous share for each was 8 % slower), and the
// bits depend on the list alone, not on the grid or the device.  A thread adds
// the squares of a batch in f32 (eight sums of at most eight terms), and from
// there on every sum (a thread's batches, a CTA's threads, the CTAs) is a pair
// of floats that keeps the rounding errors, added in a fixed order.  The scaling
// pass's CTAs each add the CTAs' sums themselves, so there is no launch between
// the two passes.  f32 squares leave the type's range for |g| above 2^63 or far below
// 2^-63: a CTA whose sum came out infinite or tiny adds once more with its
// elements scaled by a power of two, so the norm is right over the whole range
// of the types.
//
// Tensors that are not aligned to 16 bytes (views into a flat buffer) are read and
// written element by element: 118 MB in 32 tensors take 56 us aligned, 71 in f32 at
// 4 bytes off and 176 to 190 in bf16 at 2 to 8 bytes off; the norm alone 21, 25 and 40.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>
#include <type_traits>

#include "common.cuh"
#include "dab.h"
#include "host.h"
#include "vec.cuh"

namespace dab {
namespace {

constexpr int kThreads = 256;
constexpr int kCell = kThreads * 8;  // elements; a thread takes eight at a time
constexpr int kBatch = 8;            // cells of a batch, at most
constexpr int kCtas = 608;           // four on each of GB300's 152 SMs (a constant: the bits do not follow the device)

// The tensors of one launch, in the kernel's parameters: nothing is copied to
// the device, and a captured launch holds them.  `first` is the tensor's first
// cell within the launch.
template <int N>
struct Table {
  const void* src[N];
  void* dst[N];
  unsigned long long numel[N];  // top bit: f32
  uint32_t first[N + 1];
  uint32_t full;  // batches of kBatch cells: whole rounds of kCtas
  uint32_t rest;  // cells of the batches after them
  int count;
  bool in_place;  // all of them
};
constexpr int kSmall = 64, kLarge = 1000;
constexpr unsigned long long kF32 = 1ull << 63;
static_assert(sizeof(Table<kLarge>) < 32000, "kernel parameters");

// The tensor that cell c belongs to.
template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, uint32_t c) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int N>
__host__ __device__ __forceinline__ uint32_t batches_of(const Table<N>& t) {
  const uint32_t left = t.first[t.count] - t.full * kBatch;
  return t.full + (left != 0 ? (left + t.rest - 1) / t.rest : 0u);
}

// The first cell of batch b.
template <int N>
__device__ __forceinline__ uint32_t batch_edge(const Table<N>& t, uint32_t b) {
  const uint32_t whole = min(b, t.full);
  return min(whole * kBatch + (b - whole) * t.rest, t.first[t.count]);
}

// A thread's eight elements of a cell, in 16-byte pieces that are contiguous
// over the warp.  Past the tensor's end they are 0.
template <typename T>
struct Eight {
  static constexpr int kEach = 16 / sizeof(T);          // elements of a piece
  static constexpr int kPieces = 8 / kEach;
  uint4 raw[kPieces];

  static __device__ __forceinline__ unsigned long long place(unsigned long long cell, int i) {
    return cell * kCell + i * (kThreads * kEach) + threadIdx.x * kEach;
  }
  // a whole cell of a 16-byte aligned tensor
  __device__ __forceinline__ void load(const T* src, unsigned long long cell) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) raw[i] = *reinterpret_cast<const uint4*>(src + place(cell, i));
  }
  __device__ __forceinline__ void store(T* dst, unsigned long long cell, float f) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4*>(dst + place(cell, i)) = scaled(i, f);
  }
  // element by element: the last cell, or a tensor that is not aligned (the
  // same elements for the same thread, so the same sum)
  __device__ __forceinline__ void load_each(const T* src, unsigned long long cell, unsigned long long n) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const unsigned long long at = place(cell, i);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          w[j] = at + j < n ? __float_as_uint(src[at + j]) : 0u;
        } else {
          const uint16_t* s16 = reinterpret_cast<const uint16_t*>(src);
          const uint32_t lo = at + 2 * j < n ? s16[at + 2 * j] : 0u, hi = at + 2 * j + 1 < n ? s16[at + 2 * j + 1] : 0u;
          w[j] = lo | hi << 16;
        }
      }
      raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void store_each(T* dst, unsigned long long cell, unsigned long long n, float f) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const unsigned long long at = place(cell, i);
      const uint4 r = scaled(i, f);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (at + j >= n) break;
        if constexpr (sizeof(T) == 4) dst[at + j] = __uint_as_float(w[j]);
        else reinterpret_cast<uint16_t*>(dst)[at + j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
      }
    }
  }
  __device__ __forceinline__ void unpack(int i, float (&v)[kEach]) const {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        v[j] = __uint_as_float(w[j]);
      } else {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
  // piece i times f, in T again
  __device__ __forceinline__ uint4 scaled(int i, float f) const {
    float v[kEach];
    unpack(i, v);
    if constexpr (sizeof(T) == 4)
      return make_uint4(__float_as_uint(v[0] * f), __float_as_uint(v[1] * f), __float_as_uint(v[2] * f),
                        __float_as_uint(v[3] * f));
    else
      return make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f),
                        pack_bf16x2(v[4] * f, v[5] * f), pack_bf16x2(v[6] * f, v[7] * f));
  }
  // the squares of the elements (kScaled: mul times them), added to s; bits that
  // are set when an element is not zero
  template <bool kScaled>
  __device__ __forceinline__ uint32_t squares(float mul, float (&s)[8]) const {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      any |= raw[i].x | raw[i].y | raw[i].z | raw[i].w;
      float v[kEach];
      unpack(i, v);
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const float y = kScaled ? v[j] * mul : v[j];
        s[i * kEach + j] = fmaf(y, y, s[i * kEach + j]);
      }
    }
    return any & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
  }
};

// Cells of a tensor in flight a thread: 128 bytes.
template <typename T>
constexpr int kFly = 16 / sizeof(T);

// How many of `cells` cells from `cell` on are whole and aligned.
template <typename T>
__device__ __forceinline__ uint32_t whole_cells(uint32_t cell, uint32_t cells, unsigned long long n, uintptr_t at) {
  if ((at & 15u) != 0) return 0;
  const unsigned long long last = n / kCell;  // whole cells of the tensor
  return last >= (unsigned long long)cell + cells ? cells : (uint32_t)(last > cell ? last - cell : 0);
}

// A float sum and the rounding errors of its additions.  (Not double: an
// addition of doubles holds an SM for 16 cycles a warp, and the threads' sums of
// four CTAs took 3 us.)
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float x_lo = 0.f) {
    const float s = hi + x, b = s - hi;
    lo = (lo + x_lo) + ((hi - (s - b)) + (x - b));
    hi = s;
  }
  // hi alone when it is infinite: its errors are none
  __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

// The threads' sums, added: the lanes of a warp, then the warps.  (Adding two
// pairs gives the same bits either way round, so all threads hold the same.)
__device__ __forceinline__ Pair block_sum(Pair v, Pair* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, v.hi, o), lo = __shfl_xor_sync(0xffffffffu, v.lo, o);
    v.add(hi, lo);
  }
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  Pair w[kThreads / 32];
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) w[i] = sh[i];
#pragma unroll
  for (int o = 1; o < kThreads / 32; o *= 2)
#pragma unroll
    for (int i = 0; i < kThreads / 32; i += 2 * o) w[i].add(w[i + o].hi, w[i + o].lo);
  __syncthreads();
  return w[0];
}

// A CTA's sum: (hi + lo) * 2^up, up being 160, 0 or -160 (also of a sum of 0).
struct __align__(16) Sum {
  float hi, lo;
  int up, unused;
};

// The squares of (mul * element) of `cells` (at most kBatch) cells of one
// tensor, added to the thread's sum; `any` gathers whether an element is not
// zero.
template <typename T, bool kScaled>
__device__ __forceinline__ void squares(const T* src, uint32_t cell, unsigned long long n, uint32_t cells, float mul,
                                        Pair& sum, uint32_t& any) {
  const uint32_t whole = whole_cells<T>(cell, cells, n, reinterpret_cast<uintptr_t>(src));
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.f;
  uint32_t k0 = 0;
  auto some = [&](auto count) {
    constexpr int kCount = decltype(count)::value;
    Eight<T> x[kCount];
#pragma unroll
    for (int k = 0; k < kCount; ++k) x[k].load(src, cell + k0 + k);
#pragma unroll
    for (int k = 0; k < kCount; ++k) any |= x[k].template squares<kScaled>(mul, s);
    k0 += kCount;
  };
  while (k0 + kFly<T> <= whole) some(std::integral_constant<int, kFly<T>>{});
  if (kFly<T> > 4 && k0 + 4 <= whole) some(std::integral_constant<int, 4>{});
  if (k0 + 2 <= whole) some(std::integral_constant<int, 2>{});
  if (k0 < whole) some(std::integral_constant<int, 1>{});
#pragma unroll 1
  for (; k0 < cells; ++k0) {
    Eight<T> x;
    x.load_each(src, cell + k0, n);
    any |= x.template squares<kScaled>(mul, s);
  }
  sum.add(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
}

template <bool kScaled, int N>
__device__ __forceinline__ Pair cta_squares(const Table<N>& t, float mul, uint32_t& any, Pair* sh) {
  const uint32_t batches = batches_of(t);
  Pair sum;
  for (uint32_t b = blockIdx.x; b < batches; b += gridDim.x) {
    uint32_t c0 = batch_edge(t, b);
    const uint32_t c1 = batch_edge(t, b + 1);
    for (int k = tensor_of(t, c0); c0 < c1; ++k) {
      const uint32_t end = min(t.first[k + 1], c1);
      const unsigned long long n = t.numel[k] & ~kF32;
      const uint32_t cell = c0 - t.first[k];
      if (t.numel[k] & kF32) squares<float, kScaled>(static_cast<const float*>(t.src[k]), cell, n, end - c0, mul, sum, any);
      else squares<__nv_bfloat16, kScaled>(static_cast<const __nv_bfloat16*>(t.src[k]), cell, n, end - c0, mul, sum, any);
      c0 = end;
    }
  }
  return block_sum(sum, sh);
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) grad_squares_kernel(const __grid_constant__ Table<N> t,
                                                                   Sum* __restrict__ sums) {
  __shared__ Pair sh[kThreads / 32];
  grid_launch_dependents();
  uint32_t any = 0;
  Pair s = cta_squares<false>(t, 1.f, any, sh);
  const bool big = isinf(s.hi), tiny = s.hi < 0x1p-60f;
  if ((big || tiny) && __syncthreads_or(any != 0u)) s = cta_squares<true>(t, big ? 0x1p-80f : 0x1p80f, any, sh);
  if (threadIdx.x == 0) sums[blockIdx.x] = Sum{s.hi, s.lo, big ? 160 : tiny ? -160 : 0, 0};
}

// sqrt of the sum of `n` sums, in every thread of the CTA.  All are brought to
// the largest `up` among them (what is lost of the smaller is below 2^-60 of it);
// those of 160 and 0 are divided by 2^20 first, so that the total of up to 2^20
// stays in range.
__device__ __forceinline__ float total_norm(const Sum* sums, int n, Pair* sh) {
  constexpr int kEach = 3;
  auto fetch = [&](int j) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(sums + min(j, n - 1)));
    return Sum{j < n ? x.x : 0.f, j < n ? x.y : 0.f, j < n ? __float_as_int(x.z) : -160, 0};
  };
  Sum mine[kEach];  // of the first kEach * kThreads
  bool big = false, some = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) mine[i] = n > 0 ? fetch(threadIdx.x + i * kThreads) : Sum{0.f, 0.f, -160, 0};
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    big |= mine[i].up > 0;
    some |= mine[i].up == 0;
  }
  for (int j = threadIdx.x + kEach * kThreads; j < n; j += kThreads) {
    const int up = fetch(j).up;
    big |= up > 0;
    some |= up == 0;
  }
  big = __syncthreads_or(big);
  some = __syncthreads_or(some);
  // 2^(half of the sum's exponent in the total's units)
  auto half = [&](int up) {
    if (big) return up > 0 ? 0x1p-10f : up == 0 ? 0x1p-90f : 0.f;
    if (some) return up == 0 ? 0x1p-10f : 0x1p-90f;
    return 1.f;
  };
  Pair v;
  auto add = [&](const Sum& x) {
    const float f = half(x.up);
    v.add(x.hi * f * f, x.lo * f * f);
  };
#pragma unroll
  for (int i = 0; i < kEach; ++i) add(mine[i]);
  for (int j = threadIdx.x + kEach * kThreads; j < n; j += kThreads) add(fetch(j));
  return sqrtf(block_sum(v, sh).value()) * (big ? 0x1p90f : some ? 0x1p10f : 0x1p-80f);
}

// These kernels have no device-side error to report: the last launch of a call
// leaves the workspace's status clear, for whoever reads it.
__device__ __forceinline__ void clear_status(WsHeader* hdr) {
  hdr->status = 0u;
  hdr->detail = 0u;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const Sum* __restrict__ sums, int n,
                                                             float* __restrict__ norm, WsHeader* __restrict__ hdr) {
  __shared__ Pair sh[kThreads / 32];
  grid_wait();
  const float v = total_norm(sums, n, sh);
  if (threadIdx.x == 0) {
    *norm = v;
    clear_status(hdr);
  }
}

// Scales `cells` (at most kBatch) cells of a tensor.
template <typename T>
__device__ __forceinline__ void scale_cells(const T* src, T* dst, unsigned long long n, uint32_t cell, uint32_t cells,
                                            float f) {
  const uint32_t whole =
      whole_cells<T>(cell, cells, n, reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst));
  uint32_t k0 = 0;
  auto some = [&](auto count) {
    constexpr int kCount = decltype(count)::value;
    Eight<T> x[kCount];
#pragma unroll
    for (int k = 0; k < kCount; ++k) x[k].load(src, cell + k0 + k);
#pragma unroll
    for (int k = 0; k < kCount; ++k) x[k].store(dst, cell + k0 + k, f);
    k0 += kCount;
  };
  while (k0 + kFly<T> <= whole) some(std::integral_constant<int, kFly<T>>{});
  if (kFly<T> > 4 && k0 + 4 <= whole) some(std::integral_constant<int, 4>{});
  if (k0 + 2 <= whole) some(std::integral_constant<int, 2>{});
  if (k0 < whole) some(std::integral_constant<int, 1>{});
#pragma unroll 1
  for (; k0 < cells; ++k0) {
    Eight<T> x;
    x.load_each(src, cell + k0, n);
    x.store_each(dst, cell + k0, n, f);
  }
}

// `sums`: the sums to add for the norm, or null when `given` holds it already.
template <int N>
__global__ void __launch_bounds__(kThreads, 4) grad_scale_kernel(const __grid_constant__ Table<N> t,
                                                                 const Sum* __restrict__ sums, int n_sums,
                                                                 const float* given, float* norm, float max_norm,
                                                                 WsHeader* __restrict__ hdr) {
  __shared__ Pair sh[kThreads / 32];
  const uint32_t batches = batches_of(t);
  grid_wait();
  const float v = sums != nullptr ? total_norm(sums, n_sums, sh) : *given;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *norm = v;
    clear_status(hdr);
  }
  const float q = max_norm / (v + 1e-6f);
  const float f = q >= 1.f ? 1.f : q;  // a norm that is no number makes the gradients none
  if (f == 1.f && t.in_place) return;  // x * 1 is x (walking the batches took 10 us for 512 MB)
  for (uint32_t b = blockIdx.x; b < batches; b += gridDim.x) {
    uint32_t c0 = batch_edge(t, batches - 1 - b);
    const uint32_t c1 = batch_edge(t, batches - b);
    for (int k = tensor_of(t, c0); c0 < c1; ++k) {
      const uint32_t end = min(t.first[k + 1], c1);
      const unsigned long long n = t.numel[k] & ~kF32;
      const uint32_t cell = c0 - t.first[k];
      if (f != 1.f || t.src[k] != t.dst[k]) {  // a list of both kinds
        if (t.numel[k] & kF32)
          scale_cells<float>(static_cast<const float*>(t.src[k]), static_cast<float*>(t.dst[k]), n, cell, end - c0, f);
        else
          scale_cells<__nv_bfloat16>(static_cast<const __nv_bfloat16*>(t.src[k]),
                                     static_cast<__nv_bfloat16*>(t.dst[k]), n, cell, end - c0, f);
      }
      c0 = end;
    }
  }
}

long long cells_of(const dab_grad_t& g) { return (g.numel + kCell - 1) / kCell; }

// The sums of a list: kCtas for every launch of at most kLarge tensors (more
// than needed when a launch has fewer cells).
int sums_of(int count) { return kCtas * std::max(1, (count + kLarge - 1) / kLarge); }

// Checks the list; the number of its cells.
bool check_list(const dab_grad_t* grads, int count, bool write, long long* cells) {
  *cells = 0;
  if (count < 0 || count > 1000000 || (count > 0 && grads == nullptr)) return false;
  for (int k = 0; k < count; ++k) {
    const dab_grad_t& g = grads[k];
    if (g.numel < 0 || g.numel >= (1ll << 46) || (g.dtype != DAB_BF16 && g.dtype != DAB_F32)) return false;
    if (g.numel == 0) continue;
    const size_t a = g.dtype == DAB_F32 ? 4 : 2;
    if (!is_aligned(g.src, a) || (write && !is_aligned(g.dst, a))) return false;
    *cells += cells_of(g);
    if (*cells >= (1ll << 31)) return false;
  }
  return true;
}

// Whether a destination shares memory with another entry's, or with a source
// other than its own as a whole.  (Scaling twice, or reading what another CTA
// has written, would depend on which ran first.)
enum class Overlap { kNone, kSome, kNoMemory };
Overlap overlaps(const dab_grad_t* grads, int count) {
  struct Span {
    uintptr_t lo, hi;
    bool dst;
  };
  Span stack[256];
  Span* s = stack;
  if (2 * (long long)count > 256) {
    s = new (std::nothrow) Span[2 * (size_t)count];
    if (s == nullptr) return Overlap::kNoMemory;
  }
  int n = 0;
  for (int k = 0; k < count; ++k) {
    const dab_grad_t& g = grads[k];
    if (g.numel == 0) continue;
    const size_t bytes = (size_t)g.numel * (g.dtype == DAB_F32 ? 4 : 2);
    const uintptr_t a = reinterpret_cast<uintptr_t>(g.src), b = reinterpret_cast<uintptr_t>(g.dst);
    s[n++] = Span{b, b + bytes, true};
    if (a != b) s[n++] = Span{a, a + bytes, false};
  }
  std::sort(s, s + n, [](const Span& x, const Span& y) { return x.lo < y.lo; });
  uintptr_t any_hi = 0, dst_hi = 0;  // ends of all spans so far, and of the written ones
  bool bad = false;
  for (int i = 0; i < n && !bad; ++i) {
    bad = s[i].lo < (s[i].dst ? any_hi : dst_hi);
    any_hi = std::max(any_hi, s[i].hi);
    if (s[i].dst) dst_hi = std::max(dst_hi, s[i].hi);
  }
  if (s != stack) delete[] s;
  return bad ? Overlap::kSome : Overlap::kNone;
}

constexpr size_t kOffSums = 256;
size_t norm_workspace(int count) { return round_up_to(kOffSums + sizeof(Sum) * (size_t)sums_of(count), 256); }

template <int N>
void fill(Table<N>* t, const dab_grad_t* grads, int from, int to) {
  uint32_t at = 0;
  int n = 0;
  t->in_place = true;
  for (int k = from; k < to; ++k) {
    const dab_grad_t& g = grads[k];
    if (g.numel == 0) continue;
    t->in_place = t->in_place && g.src == g.dst;
    t->src[n] = g.src;
    t->dst[n] = g.dst;
    t->numel[n] = (unsigned long long)g.numel | (g.dtype == DAB_F32 ? kF32 : 0ull);
    t->first[n++] = at;
    at += (uint32_t)cells_of(g);
  }
  t->first[n] = at;
  t->count = n;
  t->full = at / (kCtas * kBatch) * kCtas;
  t->rest = std::max(1u, (at - t->full * kBatch + kCtas - 1) / kCtas);
}

// The CTAs of a table's launch.
template <int N>
unsigned ctas_of(const Table<N>& t) {
  return std::min(batches_of(t), (uint32_t)kCtas);
}

template <int N>
cudaError_t norm_pass(const dab_grad_t* grads, int count, Sum* sums, int* n_sums, cudaStream_t stream) {
  *n_sums = 0;
  cudaError_t e = cudaSuccess;
  for (int k = 0; k < count && e == cudaSuccess; k += N) {
    Table<N> t;
    fill(&t, grads, k, std::min(count, k + N));
    if (t.count == 0) continue;
    e = launch(grad_squares_kernel<N>, ctas_of(t), kThreads, stream, false, t, sums + *n_sums);
    *n_sums += (int)ctas_of(t);
  }
  return e;
}

template <int N>
cudaError_t clip_pass(const dab_grad_t* grads, int count, float max_norm, const float* given, float* norm,
                      Sum* sums, WsHeader* hdr, cudaStream_t stream) {
  int n_sums = 0;
  cudaError_t e = cudaSuccess;
  if (given == nullptr && (e = norm_pass<N>(grads, count, sums, &n_sums, stream)) != cudaSuccess) return e;
  const Sum* add = given != nullptr ? nullptr : sums;
  bool first = true;  // of the scaling launches: it may start while the last norm launch ends
  for (int k = (count - 1) / N * N; k >= 0 && e == cudaSuccess; k -= N) {
    Table<N> t;
    fill(&t, grads, k, std::min(count, k + N));
    if (t.count == 0) continue;
    e = launch(grad_scale_kernel<N>, ctas_of(t), kThreads, stream, first && given == nullptr, t, add, n_sums, given,
               norm, max_norm, hdr);
    first = false;
  }
  return e;
}

}  // namespace
}  // namespace dab

using namespace dab;

extern "C" size_t dab_grad_workspace_size(const dab_grad_t* grads, int count) {
  long long cells = 0;
  return check_list(grads, count, false, &cells) ? norm_workspace(count) : 0;
}

extern "C" dab_status_t dab_grad_norm(const dab_grad_t* grads, int count, float* norm, void* workspace,
                                      size_t ws_bytes, cudaStream_t stream) {
  long long cells = 0;
  if (!check_list(grads, count, false, &cells) || !is_aligned(norm, 4)) return DAB_ERR_INVALID_ARG;
  if (!is_aligned(workspace, 16) || ws_bytes < norm_workspace(count)) return DAB_ERR_WORKSPACE;
  if (!device_ready(nullptr)) return DAB_ERR_UNSUPPORTED;
  Sum* sums = reinterpret_cast<Sum*>(static_cast<uint8_t*>(workspace) + kOffSums);
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  int n_sums = 0;
  cudaError_t e = count <= kSmall ? norm_pass<kSmall>(grads, count, sums, &n_sums, stream)
                                  : norm_pass<kLarge>(grads, count, sums, &n_sums, stream);
  if (e == cudaSuccess)
    e = launch(grad_norm_kernel, 1, kThreads, stream, n_sums > 0, (const Sum*)sums, n_sums, norm, hdr);
  return e == cudaSuccess ? DAB_OK : record_cuda_error(e, "gradient norm launch");
}

extern "C" dab_status_t dab_grad_clip(const dab_grad_t* grads, int count, float max_norm, const float* given,
                                      float* norm, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  long long cells = 0;
  if (!check_list(grads, count, true, &cells) || !is_aligned(norm, 4)) return DAB_ERR_INVALID_ARG;
  if (given != nullptr && !is_aligned(given, 4)) return DAB_ERR_INVALID_ARG;
  if (!(max_norm >= 0.f)) return DAB_ERR_INVALID_ARG;
  const Overlap o = overlaps(grads, count);
  if (o != Overlap::kNone) return o == Overlap::kSome ? DAB_ERR_INVALID_ARG : DAB_ERR_UNSUPPORTED;
  if (!is_aligned(workspace, 16) || ws_bytes < norm_workspace(count)) return DAB_ERR_WORKSPACE;
  if (!device_ready(nullptr)) return DAB_ERR_UNSUPPORTED;
  Sum* sums = reinterpret_cast<Sum*>(static_cast<uint8_t*>(workspace) + kOffSums);
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  cudaError_t e;
  if (cells == 0) {  // nothing to scale: only the norm is written
    if (given == nullptr) {
      e = launch(grad_norm_kernel, 1, kThreads, stream, false, (const Sum*)sums, 0, norm, hdr);
    } else {
      e = cudaMemsetAsync(hdr, 0, 8, stream);
      if (e == cudaSuccess && given != norm)
        e = cudaMemcpyAsync(norm, given, sizeof(float), cudaMemcpyDeviceToDevice, stream);
    }
  } else {
    e = count <= kSmall ? clip_pass<kSmall>(grads, count, max_norm, given, norm, sums, hdr, stream)
                        : clip_pass<kLarge>(grads, count, max_norm, given, norm, sums, hdr, stream);
  }
  return e == cudaSuccess ? DAB_OK : record_cuda_error(e, "gradient clip launch");
}
