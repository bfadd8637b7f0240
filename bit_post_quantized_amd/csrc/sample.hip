// One token per row of logits: temperature, top-k, top-p and min-p, drawn with a given number.
//
// Every weight is a whole number, w = rne(2^40 exp((z - zmax) / temperature)), so sums are exact in
// 64 bits and may be formed in any order, by atomics too: the result is one for all launch shapes.
// (The exponential is in fp64, 2^-50 of itself off, so a weight is hardly ever a unit off.)
//
// The limits keep the first elements in the order of falling logits, lower indices first among equal
// ones: with the 64-bit keys (logit's ordered bits, ~index), all different, that is "key >= cut", and
// nothing needs to be sorted.  Four launches over (chunk of the vocabulary, row):
//   max     the chunk's largest logit; clears what the next one adds to
//   mass    the weights: without limits the chunk's sum, else 2048 bins over (zmax - z) / temperature,
//           counts where top-k is on, sums where only top-p is
//   gather  from the bins, the one that the limit falls into; the chunk's elements that may be cut go
//           to the row's list (top-k: all down to that bin; top-p: that bin's, and the sum of what lies
//           above it is kept per chunk)
//   draw    a workgroup per row: the cut by bins over the list's keys, narrowed until a bin has one
//           element; the chunk in which the drawn number falls; the element in it
// A list that would not fit (many equal logits, a top-k of thousands) is not used: `draw` then narrows
// over the row itself, more slowly.
#include "decoder_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {
namespace {

typedef unsigned long long u64;

constexpr int kUnitBits = 40;
constexpr double kSpan = 28.5;        // exp(-28.5) 2^40 rounds to 0
constexpr int kBins = 2048;
constexpr int kCap = 2048;            // elements of a row's list
constexpr int kMaxChunk = 16384, kMinChunk = 1024;
constexpr int kMaxChunks = 512;       // of a row
constexpr int kThreads = 256, kDrawThreads = 1024;
constexpr uint32_t kNanKey = 0xFFFFFFFFu, kNoneKey = 0x007FFFFFu;  // -infinity's

struct Entry {
  u64 key;
  u64 w;
};

struct Sizes {
  int chunks, chunk;   // of a row; elements of a chunk
};

Sizes sizes(int rows, int vocab) {
  // about four workgroups per CU, chunks of 1024 to 16384 elements
  int chunks = (1024 + rows - 1) / rows;
  const int most = (vocab + kMinChunk - 1) / kMinChunk, least = (vocab + kMaxChunk - 1) / kMaxChunk;
  if (chunks > most) chunks = most;
  if (chunks > kMaxChunks) chunks = kMaxChunks;
  if (chunks < least) chunks = least;
  int chunk = (vocab + chunks - 1) / chunks;
  chunk = (chunk + 7) / 8 * 8;
  return {(vocab + chunk - 1) / chunk, chunk};
}

// The workspace: per row and chunk a maximum and a sum, per row the bins, the list and its length.
struct Space {
  uint32_t* top;     // [rows, chunks]
  u64* sum;          // [rows, chunks]
  u64* bins;         // [rows, kBins]
  Entry* list;       // [rows, kCap]
  uint32_t* length;  // [rows]
};

size_t place(Space& s, void* ws, int rows, int chunks) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = p ? p + at : nullptr;
    at += (bytes + 15) / 16 * 16;
    return q;
  };
  const size_t r = rows;
  s.list = reinterpret_cast<Entry*>(take(r * kCap * sizeof(Entry)));
  s.bins = reinterpret_cast<u64*>(take(r * kBins * 8));
  s.sum = reinterpret_cast<u64*>(take(r * chunks * 8));
  s.top = reinterpret_cast<uint32_t*>(take(r * chunks * 4));
  s.length = reinterpret_cast<uint32_t*>(take(r * 4));
  return at;
}

// ---------------------------------------------------------------- values
template <typename T>
__device__ __forceinline__ float logit(const T* p, int64_t i) {
  return (float)p[i];
}

// ordered bits: greater floats have greater keys; both zeros the same
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ u64 full_key(float z, int i) { return (u64)order_key(z) << 32 | (uint32_t)~i; }

struct Row {
  double zmax, inv;       // largest logit, 1 / temperature
  uint32_t top;           // its key
  bool greedy, by_count, by_mass;
  int k;
  double p, least_w;      // top-p; min-p in units of the weights

  __device__ __forceinline__ bool limited() const { return by_count || by_mass; }

  // (z - zmax) / temperature; far below where the weight is 0
  __device__ __forceinline__ double arg(float z) const {
    if (!(z > -__builtin_inff())) return -1e30;
    if (top == 0xFF800000u) return z == __builtin_inff() ? 0.0 : -1e30;
    return ((double)z - zmax) * inv;
  }
};

__device__ __forceinline__ int bin_of(double x) {   // x in [-kSpan, 0]
  return min(kBins - 1, (int)((float)-x * (float)(kBins / kSpan)));
}

// rne(2^40 exp(x)), x in [-kSpan, 0]: x = n ln 2 + r, exp(r) by its series to r^12 (|r| < 0.347: the rest
// is under 2^-52), and the whole number out of the sum with 2^52, whose last bit is 1.
__device__ __forceinline__ u64 weight(double x) {
  const double n = rint(x * 1.4426950408889634074);
  const double r = __builtin_fma(-n, 0.69314718055994530942, x);
  double e = 1.0 / 479001600.0;
  e = __builtin_fma(e, r, 1.0 / 39916800.0);
  e = __builtin_fma(e, r, 1.0 / 3628800.0);
  e = __builtin_fma(e, r, 1.0 / 362880.0);
  e = __builtin_fma(e, r, 1.0 / 40320.0);
  e = __builtin_fma(e, r, 1.0 / 5040.0);
  e = __builtin_fma(e, r, 1.0 / 720.0);
  e = __builtin_fma(e, r, 1.0 / 120.0);
  e = __builtin_fma(e, r, 1.0 / 24.0);
  e = __builtin_fma(e, r, 1.0 / 6.0);
  e = __builtin_fma(e, r, 0.5);
  e = __builtin_fma(e, r, 1.0);
  e = __builtin_fma(e, r, 1.0);
  const double v = ldexp(e, (int)n + kUnitBits) + 0x1p52;
  return (u64)__double_as_longlong(v) & 0xFFFFFFFFFFFFFull;
}
__device__ __forceinline__ u64 weight_of(const Row& R, float z) {
  const double x = R.arg(z);
  return x < -kSpan ? 0 : weight(x);
}

// ---------------------------------------------------------------- workgroup sums
template <int T>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t* slots) {
  for (int d = 32; d; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  for (int i = 0; i < T / 64; ++i) v = max(v, slots[i]);
  return v;
}

// Sum of v over the threads before this one; `all` is the whole sum.
template <int T>
__device__ __forceinline__ u64 group_scan(u64 v, u64* slots, u64& all) {
  const u64 mine = (u64)wave_scan((long long)v);
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 63) slots[w] = mine;
  __syncthreads();
  u64 before = 0;
  all = 0;
  for (int i = 0; i < T / 64; ++i) {
    const u64 s = slots[i];
    if (i < w) before += s;
    all += s;
  }
  return before + mine - v;
}

// The row's settings, the same in every workgroup of the row.  T threads.
template <int T>
__device__ __forceinline__ Row row_of(const SampleRows& a, const Space& s, int chunks, int row, uint32_t* slots) {
  uint32_t top = 0;
  for (int c = threadIdx.x; c < chunks; c += T) top = max(top, s.top[(size_t)row * chunks + c]);
  Row R;
  R.top = group_max<T>(top, slots);
  R.zmax = (double)key_value(R.top);
  const float t = a.temperature[row];
  R.greedy = !(t > 0.0f);
  R.inv = 1.0 / (double)t;
  R.k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.0f;
  R.p = p;
  R.by_count = R.k > 0;
  R.by_mass = p < 1.0f;
  const float m = a.min_p ? a.min_p[row] : 0.0f;
  R.least_w = m > 0.0f ? (double)fminf(m, 1.0f) * 0x1p40 : 0.0;
  return R;
}

// whether the limit lies at or before what sums up to `through`
__device__ __forceinline__ bool crossed(bool by_count, u64 through, int k, double least) {
  return by_count ? through >= (u64)k : !((double)through < least);
}

// ---------------------------------------------------------------- launches
template <typename T>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(SampleRows a, Space s, Sizes z) {
  __shared__ uint32_t slots[kThreads / 64];
  const int row = blockIdx.y, c = blockIdx.x;
  if (a.top_k || a.top_p)
    for (int b = c * kThreads + threadIdx.x; b < kBins; b += gridDim.x * kThreads) s.bins[(size_t)row * kBins + b] = 0;
  if (c == 0 && threadIdx.x == 0) s.length[row] = 0;
  const T* p = reinterpret_cast<const T*>(a.logits) + row * a.stride;
  const int end = min(a.vocab, (c + 1) * z.chunk);
  uint32_t top = 0;
#pragma unroll 8
  for (int i = c * z.chunk + threadIdx.x; i < end; i += kThreads) {
    const float v = logit(p, i);
    top = max(top, v != v ? kNanKey : order_key(v));
  }
  top = group_max<kThreads>(top, slots);
  if (threadIdx.x == 0) s.top[(size_t)row * z.chunks + c] = top;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_mass_kernel(SampleRows a, Space s, Sizes z) {
  __shared__ u64 bins[kBins];
  __shared__ u64 sums[kThreads / 64];
  __shared__ uint32_t slots[kThreads / 64];
  const int row = blockIdx.y, c = blockIdx.x;
  const Row R = row_of<kThreads>(a, s, z.chunks, row, slots);
  if (R.greedy || R.top == kNanKey || R.top <= kNoneKey) return;
  const T* p = reinterpret_cast<const T*>(a.logits) + row * a.stride;
  const int end = min(a.vocab, (c + 1) * z.chunk);
  if (!R.limited()) {
    u64 sum = 0, all;
#pragma unroll 4
    for (int i = c * z.chunk + threadIdx.x; i < end; i += kThreads) {
      const u64 w = weight_of(R, logit(p, i));
      if ((double)w >= R.least_w) sum += w;
    }
    group_scan<kThreads>(sum, sums, all);
    if (threadIdx.x == 0) s.sum[(size_t)row * z.chunks + c] = all;
    return;
  }
  for (int b = threadIdx.x; b < kBins; b += kThreads) bins[b] = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = c * z.chunk + threadIdx.x; i < end; i += kThreads) {
    const double x = R.arg(logit(p, i));
    if (x >= -kSpan) {
      const u64 w = weight(x);
      if (w) atomicAdd(&bins[bin_of(x)], R.by_count ? 1ull : w);
    }
  }
  __syncthreads();
  // what lies behind this chunk's own k-th element cannot hold the row's
  u64 seen = 0, all;
  constexpr int kPer = kBins / kThreads;
  for (int j = 0; j < kPer; ++j) seen += bins[threadIdx.x * kPer + j];
  seen = group_scan<kThreads>(seen, sums, all);
  for (int j = 0; j < kPer; ++j) {
    const int b = threadIdx.x * kPer + j;
    const u64 n = bins[b];
    if (n && !(R.by_count && seen >= (u64)R.k)) atomicAdd(&s.bins[(size_t)row * kBins + b], n);
    seen += n;
  }
}

// The first of kBins bins through which the limit is reached (kBins where none is), and what stands
// before it, `base` and the bins in front of it.  T threads; sums has T / 64 + 1 places.
template <int T>
__device__ __forceinline__ int first_crossing(const u64* bins, bool by_count, int k, double least, u64 base, u64* sums,
                                              int* found, u64& before) {
  constexpr int kPer = kBins / T;
  u64 n[kPer], mine = 0, all;
#pragma unroll
  for (int j = 0; j < kPer; ++j) mine += n[j] = bins[threadIdx.x * kPer + j];
  if (threadIdx.x == 0) *found = kBins;
  u64 through = base + group_scan<T>(mine, sums, all), in_front = 0;
  int b = kBins;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (b == kBins && n[j] && crossed(by_count, through + n[j], k, least)) {
      b = threadIdx.x * kPer + j;
      in_front = through;
    }
    through += n[j];
  }
  if (b < kBins) atomicMin(found, b);
  __syncthreads();
  const int first = *found;
  if (b == first && b < kBins) sums[T / 64] = in_front;
  __syncthreads();
  before = sums[T / 64];
  __syncthreads();
  return first;
}

// The bin that the row's limit falls into; top-p's share of the row's sum.
template <int T>
__device__ __forceinline__ int limit_bin(const Row& R, const u64* bins, u64* sums, int* found, double& least,
                                         u64& before) {
  least = 0.0;
  if (!R.by_count) {
    u64 mine = 0, all;
    for (int b = threadIdx.x; b < kBins; b += T) mine += bins[b];
    group_scan<T>(mine, sums, all);
    least = R.p * (double)all;
  }
  return first_crossing<T>(bins, R.by_count, R.k, least, 0, sums, found, before);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_gather_kernel(SampleRows a, Space s, Sizes z) {
  __shared__ u64 sums[kThreads / 64 + 1];
  __shared__ uint32_t slots[kThreads / 64];
  __shared__ int found;
  const int row = blockIdx.y, c = blockIdx.x;
  const Row R = row_of<kThreads>(a, s, z.chunks, row, slots);
  if (R.greedy || R.top == kNanKey || R.top <= kNoneKey || !R.limited()) return;
  double least;
  u64 above;
  const int cut = limit_bin<kThreads>(R, s.bins + (size_t)row * kBins, sums, &found, least, above);
  const T* p = reinterpret_cast<const T*>(a.logits) + row * a.stride;
  const int end = min(a.vocab, (c + 1) * z.chunk);
  u64 sum = 0, all;
#pragma unroll 4
  for (int i = c * z.chunk + threadIdx.x; i < end; i += kThreads) {
    const float v = logit(p, i);
    const double x = R.arg(v);
    if (x < -kSpan) continue;
    const int b = bin_of(x);
    if (b > cut) continue;
    const u64 w = weight(x);
    if (!w) continue;
    if (R.by_count || b == cut) {
      const uint32_t at = atomicAdd(&s.length[row], 1u);
      if (at < (uint32_t)kCap) s.list[(size_t)row * kCap + at] = Entry{full_key(v, i), w};
    } else if ((double)w >= R.least_w) {
      sum += w;
    }
  }
  group_scan<kThreads>(sum, sums, all);
  if (threadIdx.x == 0) s.sum[(size_t)row * z.chunks + c] = all;
}

// ---------------------------------------------------------------- draw
// The elements that a limit is looked for among: the row's list, or the row itself.
template <typename T>
struct Source {
  const Entry* list;   // NULL: the row
  const T* logits;
  const Row* R;
  int n;

  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (list) {
      for (int i = threadIdx.x; i < n; i += kDrawThreads) f(list[i].key, list[i].w);
    } else {
      for (int i = threadIdx.x; i < n; i += kDrawThreads) {
        const float v = logit(logits, i);
        const u64 w = weight_of(*R, v);
        if (w) f(full_key(v, i), w);
      }
    }
  }
};

struct DrawSpace {
  u64 bins[kBins];
  uint32_t count[kBins];
  u64 sums[kDrawThreads / 64 + 1];
  u64 chunk[kMaxChunks];
  u64 lo, hi;
  uint32_t slots[kDrawThreads / 64];
  int found;
};

// The smallest key that stays, where those stay that come, from the greatest key down, before the
// limit; `base` comes before all of them.  Only keys >= floor are looked at.  0 where all stay.
template <typename T>
__device__ u64 find_cut(const Source<T>& src, DrawSpace& L, bool by_count, int k, double least, u64 base, u64 floor) {
  if (threadIdx.x == 0) L.lo = ~0ull, L.hi = 0;
  __syncthreads();
  u64 lo = ~0ull, hi = 0;
  src.each([&](u64 key, u64) {
    if (key >= floor) lo = min(lo, key), hi = max(hi, key);
  });
  if (lo <= hi) {
    atomicMin(&L.lo, lo);
    atomicMax(&L.hi, hi);
  }
  __syncthreads();
  lo = L.lo;
  hi = L.hi;
  if (lo > hi) return floor;
  for (;;) {
    const u64 range = hi - lo;
    const int bits = 64 - (range ? __clzll((long long)range) : 64), shift = bits > 11 ? bits - 11 : 0;
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kDrawThreads) L.bins[b] = 0, L.count[b] = 0;
    if (threadIdx.x == 0) L.found = kBins;
    __syncthreads();
    src.each([&](u64 key, u64 w) {
      if (key >= lo && key <= hi) {
        const int b = (int)((hi - key) >> shift);
        atomicAdd(&L.bins[b], by_count ? 1ull : w);
        atomicAdd(&L.count[b], 1u);
      }
    });
    __syncthreads();
    u64 before;
    const int b = first_crossing<kDrawThreads>(L.bins, by_count, k, least, base, L.sums, &L.found, before);
    if (b == kBins) return floor;   // never reached: all stay
    base = before;
    const uint32_t here = L.count[b];
    hi -= (u64)b << shift;
    const u64 width = (1ull << shift) - 1;
    lo = hi - lo > width ? hi - width : lo;
    if (here == 1 || shift == 0) return lo;
  }
}

template <typename T>
__global__ __launch_bounds__(kDrawThreads) void sample_draw_kernel(SampleRows a, Space s, Sizes z) {
  __shared__ DrawSpace L;
  const int row = blockIdx.x, tid = threadIdx.x;
  const Row R = row_of<kDrawThreads>(a, s, z.chunks, row, L.slots);
  const T* p = reinterpret_cast<const T*>(a.logits) + row * a.stride;
  if (R.top == kNanKey || R.top <= kNoneKey) {
    if (tid == 0) {
      a.tokens[row] = -1;
      if (a.share) a.share[row] = 0.0f;
    }
    return;
  }
  const uint32_t* tops = s.top + (size_t)row * z.chunks;
  if (R.greedy) {
    // the first chunk with the largest logit, then the first element in it
    if (tid == 0) L.found = z.chunks;
    __syncthreads();
    for (int c = tid; c < z.chunks; c += kDrawThreads)
      if (tops[c] == R.top) atomicMin(&L.found, c);
    __syncthreads();
    const int c = L.found, end = min(a.vocab, (c + 1) * z.chunk);
    __syncthreads();
    if (tid == 0) L.found = a.vocab;
    __syncthreads();
    for (int i = c * z.chunk + tid; i < end; i += kDrawThreads)
      if (order_key(logit(p, i)) == R.top) {
        atomicMin(&L.found, i);
        break;
      }
    __syncthreads();
    if (tid == 0) {
      a.tokens[row] = L.found;
      if (a.share) a.share[row] = 1.0f;
    }
    return;
  }

  // ---- the cut
  u64 cut = 0;
  Source<T> src{nullptr, p, &R, a.vocab};
  if (R.limited()) {
    const uint32_t length = s.length[row];
    const bool listed = length <= (uint32_t)kCap;
    if (listed) {
      src.list = s.list + (size_t)row * kCap;
      src.n = (int)length;
    }
    if (R.by_count) {
      cut = find_cut(src, L, true, R.k, 0.0, 0, 0);
      if (R.by_mass) {
        u64 mass = 0, all;
        src.each([&](u64 key, u64 w) {
          if (key >= cut) mass += w;
        });
        group_scan<kDrawThreads>(mass, L.sums, all);
        cut = find_cut(src, L, false, 0, R.p * (double)all, 0, cut);
      }
    } else {
      double least;
      u64 above;
      (void)limit_bin<kDrawThreads>(R, s.bins + (size_t)row * kBins, L.sums, &L.found, least, above);
      cut = find_cut(src, L, false, 0, least, listed ? above : 0, 0);
    }
    // ---- the chunks' sums: what lies above the list for certain, and what of the list stays
    const bool part = listed && !R.by_count;
    __syncthreads();
    for (int c = tid; c < z.chunks; c += kDrawThreads) L.chunk[c] = part ? s.sum[(size_t)row * z.chunks + c] : 0;
    __syncthreads();
    src.each([&](u64 key, u64 w) {
      if (key >= cut && (double)w >= R.least_w) atomicAdd(&L.chunk[(uint32_t)~key / (uint32_t)z.chunk], w);
    });
  } else {
    for (int c = tid; c < z.chunks; c += kDrawThreads) L.chunk[c] = s.sum[(size_t)row * z.chunks + c];
  }
  __syncthreads();

  // ---- the chunk that the number falls into
  u64 total;
  const u64 mine = tid < z.chunks ? L.chunk[tid] : 0;
  u64 before = group_scan<kDrawThreads>(mine, L.sums, total);
  const float u = a.uniform[row];
  const double part = (double)total * (double)(u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f);
  u64 at = (u64)floor(part);
  if (at > total - 1) at = total - 1;
  if (mine && before <= at && at < before + mine) {
    L.found = tid;
    L.lo = before;
  }
  __syncthreads();
  const int c = L.found;
  const u64 start = L.lo;

  // ---- the element in it: neighbouring elements per thread, in order
  const int first = c * z.chunk, end = min(a.vocab, first + z.chunk);
  const int per = (z.chunk + kDrawThreads - 1) / kDrawThreads;
  auto kept = [&](int i) {
    const float v = logit(p, i);
    const u64 w = weight_of(R, v);
    return full_key(v, i) >= cut && (double)w >= R.least_w ? w : 0;
  };
  u64 sum = 0, all;
  for (int i = first + tid * per; i < min(end, first + (tid + 1) * per); ++i) sum += kept(i);
  before = start + group_scan<kDrawThreads>(sum, L.sums, all);
  if (sum && before <= at && at < before + sum)
    for (int i = first + tid * per;; ++i) {
      const u64 w = kept(i);
      if (at < before + w) {
        a.tokens[row] = i;
        if (a.share) a.share[row] = (float)((double)w / (double)total);
        break;
      }
      before += w;
    }
}

template <typename T>
hipError_t launch(const SampleRows& a, hipStream_t st) {
  const Sizes z = sizes(a.rows, a.vocab);
  Space s;
  place(s, a.ws, a.rows, z.chunks);
  const dim3 grid(z.chunks, a.rows);
  hipLaunchKernelGGL((sample_max_kernel<T>), grid, dim3(kThreads), 0, st, a, s, z);
  hipLaunchKernelGGL((sample_mass_kernel<T>), grid, dim3(kThreads), 0, st, a, s, z);
  if (a.top_k || a.top_p) hipLaunchKernelGGL((sample_gather_kernel<T>), grid, dim3(kThreads), 0, st, a, s, z);
  hipLaunchKernelGGL((sample_draw_kernel<T>), dim3(a.rows), dim3(kDrawThreads), 0, st, a, s, z);
  return hipGetLastError();
}

}  // namespace

size_t sample_workspace_bytes(int rows, int vocab) {
  Space s;
  return place(s, nullptr, rows, sizes(rows, vocab).chunks);
}

hipError_t launch_sample(const SampleRows& a, int logits_fp32, hipStream_t stream) {
  return logits_fp32 ? launch<float>(a, stream) : launch<__bf16>(a, stream);
}

}  // namespace svdq
