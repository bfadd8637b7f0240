// One token per row of logits: temperature, top-k, top-p and min-p, drawn with a given number.
//
// Every weight is a whole number, w = rne(2^40 exp((z - zmax) / temperature)), so sums are exact in
// 64 bits and may be formed in any order, by atomics too: the result is one for all launch shapes.
// (The exponential is in fp64, 2^-50 of itself off, so a weight is hardly ever a unit off.)
//
// The limits keep the first elements in the order of falling logits, lower indices first among equal
// ones: with the 64-bit keys (logit's ordered bits, ~index), all different, that is "key >= cut", and
// nothing needs to be sorted.  Launches over (chunk of the vocabulary, row):
//   max     largest logits of up to 512 parts of the row
//   mass    top-k: the k-th largest part holds an element that k - 1 others reach or pass, so the k first are among
//           the elements that reach it: hardly more than k, which go to the row's list with their weights.
//           Only top-p: 2048 bins of the weights over (zmax - z) / temperature, per chunk.
//           No limit: the weights' sum per chunk
//   gather  only top-p: the elements of the bin that the limit falls into go to the row's list
//   draw    a workgroup per row.  Top-k: everything from the list.  Otherwise the cut from the list, the
//           chunk in which the drawn number falls, and the element in it
// A list that would not fit is not used: `draw` then narrows down the cut by bins over the row itself, which takes 6 to
// 20 times as long.  That is so for a top-k of more than the row's parts with a maximum above -infinity (512 at
// most; a mask that leaves fewer than k tokens is such a row), for a limit among thousands of equal logits, and for
// more than kCap elements in the one bin (1/72 of the temperature wide) that the limit of top-p alone falls into.
//
// Bound by the chain of launches and exchanges, not by bytes: 64 rows of 131072 in fp32 (33 MB, 6.5 us of a copy)
// take 15 us at temperature 0, 26 - 29 without a limit, 19 - 21 with top-k and 47 - 63 with top-p alone; one row 13 - 16,
// 27 - 30 with top-p alone; 300 rows of 32001 in bf16 36 and 56.  Searched by one workgroup each, 64 rows of 131072 and one:
// a top-k of 1000 264 and 233, of 50 where a mask leaves 40 tokens 126 and 106, among equal logits 299 and 281, top-p among
// equal logits 467 and 413, top-p 0.5 of logits of spread 1 at temperature 6 357 and 308.
#include "decoder_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {
namespace {

typedef unsigned long long u64;

constexpr int kUnitBits = 40;
constexpr double kSpan = 28.5;        // exp(-28.5) 2^40 rounds to 0
constexpr int kBins = 2048, kCoarse = 64, kFine = kBins / kCoarse;
constexpr int kCap = 4096;            // elements of a row's list
constexpr int kPairs = 256;           // as many are compared each with each
constexpr int kParts = 512;           // of a row, at most
constexpr int kMaxChunks = 64;        // of a row
constexpr int kThreads = 512;
constexpr int kApart = 32;
// pieces of 16 bytes that a thread loads before it knows the settings
template <typename T>
constexpr int kAhead = sizeof(T) == 4 ? 2 : 1;
constexpr uint32_t kNanKey = 0xFFFFFFFFu, kNoneKey = 0x007FFFFFu;  // -infinity's

struct Sizes {
  int chunks, chunk;   // of a row; elements of a chunk
  int parts;           // of a chunk: a power of two
};

Sizes sizes(int rows, int vocab) {
  // four workgroups per CU, as many as run at once, of 2048 elements or more
  int chunks = rows < 1024 ? 1024 / rows : 1;
  const int most = (vocab + 2047) / 2048;
  if (chunks > most) chunks = most;
  if (chunks > kMaxChunks) chunks = kMaxChunks;
  int chunk = (vocab + chunks - 1) / chunks;
  chunk = (chunk + 3) / 4 * 4;
  chunks = (vocab + chunk - 1) / chunk;
  int parts = kParts;
  while (parts * chunks > kParts) parts /= 2;
  return {chunks, chunk, parts};
}

// The workspace of `rows` rows: per chunk its parts' maxima, a sum, the bins and the sums of each kFine of
// them; per row the list and its length.
struct Space {
  uint32_t* top;     // [rows, chunks, parts]
  u64* sum;          // [rows, chunks]
  u64* bins;         // [rows, chunks, kBins]
  u64* coarse;       // [rows, chunks, kCoarse]
  u64* list;         // [rows, kCap], keys
  uint32_t* length;  // [rows, kApart]: a cache line each, many workgroups add to them
};

size_t place(Space& s, void* ws, int rows, const Sizes& z) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = p ? p + at : nullptr;
    at += (bytes + 15) / 16 * 16;
    return q;
  };
  const size_t r = rows, c = r * z.chunks;
  s.list = reinterpret_cast<u64*>(take(r * kCap * 8));
  s.bins = reinterpret_cast<u64*>(take(c * kBins * 8));
  s.coarse = reinterpret_cast<u64*>(take(c * kCoarse * 8));
  s.sum = reinterpret_cast<u64*>(take(c * 8));
  s.top = reinterpret_cast<uint32_t*>(take(c * z.parts * 4));
  s.length = reinterpret_cast<uint32_t*>(take(r * kApart * 4));
  return at;
}

// Rows that are done at a time: their chunks' bins are 16 KB each.
int batch(int rows, const Sizes& z) {
  const int most = 4096 / z.chunks;
  return rows < most ? rows : most;
}

// ---------------------------------------------------------------- values
// The elements [begin, end) of a row, 16 bytes of neighbours per thread at a time (of any alignment).  `U`
// such pieces are loaded when the object is made, so that they are under way while other things are waited
// for; then f(element, index) for all.
template <int U, typename T>
struct Elements {
  static constexpr int E = 16 / sizeof(T);
  struct __attribute__((packed, aligned(sizeof(T)))) Piece {
    T v[E];
  };
  const T* p;
  int begin, end;
  Piece q[U];

  __device__ __forceinline__ Elements(const T* row, int first, int last) : p(row), begin(first), end(last) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = begin + E * (threadIdx.x + u * kThreads);
      if (i + E <= end) q[u] = *reinterpret_cast<const Piece*>(p + i);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = begin + E * (threadIdx.x + u * kThreads);
      if (i + E <= end) {
#pragma unroll
        for (int e = 0; e < E; ++e) f((float)q[u].v[e], i + e);
      } else {
        for (int j = i; j < end; ++j) f((float)p[j], j);
      }
    }
#pragma unroll 1
    for (int i = begin + E * (threadIdx.x + U * kThreads); i < end; i += E * kThreads) {
      if (i + E <= end) {
        const Piece more = *reinterpret_cast<const Piece*>(p + i);
#pragma unroll
        for (int e = 0; e < E; ++e) f((float)more.v[e], i + e);
      } else {
        for (int j = i; j < end; ++j) f((float)p[j], j);
      }
    }
  }
};

// ordered bits: greater floats have greater keys; both zeros the same
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ u64 full_key(float z, int i) { return (u64)order_key(z) << 32 | (uint32_t)~i; }
__device__ __forceinline__ int index_of(u64 key) { return (int)~(uint32_t)key; }

struct Row {
  double zmax, inv;       // largest logit, 1 / temperature
  uint32_t top;           // its key
  bool greedy, by_count, by_mass;
  int k;
  double p;               // top-p
  u64 least_w;            // min-p in units of the weights, the next whole number

  __device__ __forceinline__ bool limited() const { return by_count || by_mass; }

  // (z - zmax) / temperature, <= 0; far below 0 where the weight is 0
  __device__ __forceinline__ double arg(float z) const { return fmin(((double)z - zmax) * inv, 0.0); }
};

__device__ __forceinline__ int bin_of(double x) {   // x in [-kSpan, 0]
  return min(kBins - 1, (int)((float)-x * (float)(kBins / kSpan)));
}

// rne(2^40 exp(x)), x in [-kSpan, 0]: x = n ln 2 + r, exp(r) by its series to r^12 (|r| < 0.347: the rest
// is under 2^-52).  n is rounded by an addition in whose sum it is the low bits, the power of two is added to
// the exponent, and the whole number is read out of the sum with 2^52, whose last bit is 1.
__device__ __forceinline__ double fma_scalar(double a, double b, double c) {   // a b + c, c in scalar registers
  double d;   // (left to itself the compiler copies c into the sum's registers first, for each element)
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
  return d;
}
__device__ __forceinline__ u64 weight(double x) {
  constexpr double kRound = 0x1.8p52;
  const double t = __builtin_fma(x, 1.4426950408889634074, kRound);
  const double r = __builtin_fma(-(t - kRound), 0.69314718055994530942, x);
  double e = fma_scalar(r, 1.0 / 479001600.0, 1.0 / 39916800.0);
  e = fma_scalar(e, r, 1.0 / 3628800.0);
  e = fma_scalar(e, r, 1.0 / 362880.0);
  e = fma_scalar(e, r, 1.0 / 40320.0);
  e = fma_scalar(e, r, 1.0 / 5040.0);
  e = fma_scalar(e, r, 1.0 / 720.0);
  e = fma_scalar(e, r, 1.0 / 120.0);
  e = fma_scalar(e, r, 1.0 / 24.0);
  e = fma_scalar(e, r, 1.0 / 6.0);
  e = __builtin_fma(e, r, 0.5);
  e = __builtin_fma(e, r, 1.0);
  e = __builtin_fma(e, r, 1.0);
  const int n = (int)__double_as_longlong(t) + kUnitBits;   // (the sum's low word)
  const double scaled = __longlong_as_double(__double_as_longlong(e) + ((long long)n << 52));
  return (u64)__double_as_longlong(scaled + 0x1p52) & 0xFFFFFFFFFFFFFull;
}
__device__ __forceinline__ u64 weight_of(const Row& R, float z) {
  const double x = R.arg(z);
  return x >= -kSpan ? weight(x) : 0;
}
__device__ __forceinline__ u64 weight_of(const Row& R, u64 key) { return weight_of(R, key_value((uint32_t)(key >> 32))); }

// ---------------------------------------------------------------- workgroup sums
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

__device__ __forceinline__ u64 wave_max64(u64 v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = max(v, (u64)__shfl_xor((long long)v, d));
  return v;
}

// Sum of v over the threads before this one; `all` is the whole sum.  `slots` has kThreads / 64 places.
__device__ __forceinline__ u64 group_scan(u64 v, u64* slots, u64& all) {
  const u64 mine = (u64)wave_scan((long long)v);
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 63) slots[w] = mine;
  __syncthreads();
  u64 before = 0;
  all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) {
    const u64 s = slots[i];
    if (i < w) before += s;
    all += s;
  }
  return before + mine - v;
}
__device__ __forceinline__ u64 group_sum(u64 v, u64* slots) {
  u64 all;
  group_scan(v, slots, all);
  return all;
}

// What a workgroup shares of its row: the parts' maxima, and room to agree on one.
struct Shared {
  uint32_t tops[kParts], most[kThreads / 64], least;
  u64 coarse[kThreads / 64][kCoarse];
};

// The row's settings, the same in every workgroup of the row.
__device__ __forceinline__ Row row_of(const SampleRows& a, const Space& s, const Sizes& z, int row, Shared& L) {
  static_assert(kThreads == kParts, "a part for each thread");
  const int n = z.chunks * z.parts, t = threadIdx.x;
  const uint32_t mine = t < n ? s.top[(size_t)row * n + t] : 0u;
  const float temperature = a.temperature[row];
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.0f;
  const float m = a.min_p ? a.min_p[row] : 0.0f;
  L.tops[t] = mine;
  const uint32_t most = wave_max(mine);
  if ((t & 63) == 0) L.most[t >> 6] = most;
  __syncthreads();
  Row R;
  R.top = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) R.top = max(R.top, L.most[i]);
  R.greedy = !(temperature > 0.0f);
  // (an infinite temperature: so small that no difference is seen, but -infinity is)
  R.zmax = (double)key_value(R.top);
  R.inv = fmax(1.0 / (double)temperature, 1e-300);
  // (where the largest is +infinity, a border between it and all finite logits)
  if (R.top == 0xFF800000u) R.zmax = 1e39, R.inv = 1.0;
  R.k = k;
  R.p = p;
  R.by_count = k > 0;
  R.by_mass = p < 1.0f;
  R.least_w = m > 0.0f ? (u64)ceil((double)fminf(m, 1.0f) * 0x1p40) : 0;
  return R;
}

// What the k-th largest of a wave's 512 values reaches, and hardly more do: the 13 leading bits in which
// the values (those that are not 0; `top` is the largest) differ, bit by bit.  0 where there are fewer than k.
__device__ __forceinline__ uint32_t kth_largest(const uint32_t (&v)[8], uint32_t top, int k) {
  uint32_t low = top;
  int n = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (v[i]) low = min(low, v[i]);
    n += __popcll(__ballot(v[i] != 0u));
  }
  if (n < k) return 0u;
  for (int d = 32; d; d >>= 1) low = min(low, (uint32_t)__shfl_xor((int)low, d));
  const int bits = __builtin_amdgcn_readfirstlane(32 - __clz((int)(low ^ top | 1u)));
  uint32_t found = __builtin_amdgcn_readfirstlane(bits < 32 ? top >> bits << bits : 0u);
#pragma unroll 1
  for (int bit = bits - 1; bit >= max(bits - 13, 0); --bit) {
    const uint32_t trial = found | 1u << bit;
    n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) n += __popcll(__ballot(v[i] >= trial));
    if (n >= k) found = trial;
  }
  return found;
}

// whether the limit lies at or before what sums up to `through`
__device__ __forceinline__ bool crossed(bool by_count, u64 through, int k, double least) {
  return by_count ? through >= (u64)k : !((double)through < least);
}

// ---------------------------------------------------------------- launches
template <typename T>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(SampleRows a, Space s, Sizes z) {
  const int row = blockIdx.y, c = blockIdx.x, t = threadIdx.x;
  if (c == 0 && t == 0) s.length[(size_t)row * kApart] = 0;
  const T* p = reinterpret_cast<const T*>(a.logits) + row * a.stride;
  uint32_t top = 0;
  const Elements<4, T> elements(p, c * z.chunk, min(a.vocab, (c + 1) * z.chunk));
  elements.each([&](float v, int) { top = max(top, v != v ? kNanKey : order_key(v)); });
  // a part: what neighbouring threads (at most a wave) have read, of those that have something to read
  int live = kThreads;
  while (live > z.parts && (live / 2) * (16 / (int)sizeof(T)) >= z.chunk) live /= 2;
  const int group = live / z.parts;
  for (int d = 1; d < group; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if (t < live && t % group == 0) s.top[((size_t)row * z.chunks + c) * z.parts + t / group] = top;
}

// Elements for a row's list, gathered in LDS first (2048 of a chunk: a chunk with more makes the list too
// long).
constexpr int kOfChunk = 2048;
struct Gathered {
  u64 key[kOfChunk];
  uint32_t count, place;
};
__device__ __forceinline__ void gather(Gathered& L, float v, int i) {
  const uint32_t at = atomicAdd(&L.count, 1u);
  if (at < (uint32_t)kOfChunk) L.key[at] = full_key(v, i);
}
// (a length over kCap says that the list is not whole)
__device__ __forceinline__ void append(Gathered& L, const Space& s, int row) {
  __syncthreads();
  const uint32_t n = L.count;
  if (threadIdx.x == 0) L.place = n ? atomicAdd(&s.length[(size_t)row * kApart], n > (uint32_t)kOfChunk ? kCap + 1u : n) : 0u;
  __syncthreads();
  const uint32_t first = L.place;
  for (uint32_t i = threadIdx.x; i < min(n, (uint32_t)kOfChunk); i += kThreads)
    if (first + i < (uint32_t)kCap) s.list[(size_t)row * kCap + first + i] = L.key[i];
}

template <typename T>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(8))) void sample_mass_kernel(SampleRows a, Space s, Sizes z) {
  __shared__ union {
    u64 bins[kBins];
    Gathered list;
  } L;
  __shared__ u64 sums[kThreads / 64];
  __shared__ Shared S;
  const int row = blockIdx.y, c = blockIdx.x, t = threadIdx.x;
  const T* p = reinterpret_cast<const T*>(a.logits) + row * a.stride;
  const Elements<kAhead<T>, T> elements(p, c * z.chunk, min(a.vocab, (c + 1) * z.chunk));
  const Row R = row_of(a, s, z, row, S);
  if (R.greedy || R.top == kNanKey || R.top <= kNoneKey) return;
  const size_t at = (size_t)row * z.chunks + c;
  if (R.by_count) {
    if (t < 64) {
      uint32_t tops[kParts / 64];
#pragma unroll
      for (int i = 0; i < kParts / 64; ++i) tops[i] = S.tops[64 * i + t];
      const uint32_t least = kth_largest(tops, R.top, R.k);
      if (t == 0) S.least = least, L.list.count = 0;
    }
    __syncthreads();
    const uint32_t least = S.least;
    elements.each([&](float v, int i) {
      if (order_key(v) >= least) gather(L.list, v, i);
    });
    append(L.list, s, row);
    return;
  }
  if (!R.by_mass) {
    u64 sum = 0;
    elements.each([&](float v, int) {
      const u64 w = weight_of(R, v);
      sum += w >= R.least_w ? w : 0;
    });
    sum = group_sum(sum, sums);
    if (t == 0) s.sum[at] = sum;
    return;
  }
  for (int b = t; b < kBins; b += kThreads) L.bins[b] = 0;
  __syncthreads();
  elements.each([&](float v, int) {
    const double x = R.arg(v);
    if (x >= -kSpan) atomicAdd(&L.bins[bin_of(x)], weight(x));
  });
  __syncthreads();
  constexpr int kPer = kBins / kThreads;   // (kFine / kPer = 8 threads have a coarse bin)
  u64 sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const u64 n = L.bins[t * kPer + j];
    s.bins[at * kBins + t * kPer + j] = n;
    sum += n;
  }
  for (int d = 1; d < kFine / kPer; d <<= 1) sum += (u64)__shfl_xor((long long)sum, d);
  if (t % (kFine / kPer) == 0) s.coarse[at * kCoarse + t / (kFine / kPer)] = sum;
}

// Of a row's bins: those before `lo` stay whole, those behind `hi` go, the elements from lo to hi are looked
// at; what stands before lo, and top-p's share of the row's sum.  The same in every thread.
struct Limit {
  int lo, hi;
  u64 before;
  double least;
};
__device__ __forceinline__ Limit limit_of(const Row& R, const Space& s, const Sizes& z, int row, Shared& L) {
  constexpr int kWaves = kThreads / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // sums over the chunks, each wave an eighth of them (`live`: lanes with a bin), in every wave
  auto over_chunks = [&](const u64* first, size_t stride, bool live) {
    u64 sum = 0;
    if (live) {
#pragma unroll
      for (int i = 0; i < kMaxChunks / kWaves; ++i)
        if (wave + i * kWaves < z.chunks) sum += first[(size_t)(wave + i * kWaves) * stride];
    }
    __syncthreads();
    L.coarse[wave][lane] = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) sum += L.coarse[i][lane];
    return sum;
  };
  u64 mine = over_chunks(s.coarse + (size_t)row * z.chunks * kCoarse + lane, kCoarse, true);
  const u64 coarse_sum = mine, coarse_through = (u64)wave_scan((long long)mine);
  const u64 all = (u64)__shfl((long long)coarse_through, 63);
  // the sums of the bins of coarse bin cb, and what stands before each
  auto fine = [&](int cb, u64& before) {
    const u64 sum = over_chunks(s.bins + (size_t)row * z.chunks * kBins + cb * kFine + lane, kBins, lane < kFine);
    before = (u64)__shfl((long long)(coarse_through - coarse_sum), cb) + (u64)wave_scan((long long)sum) - sum;
    return sum;
  };
  Limit f{kBins, kBins, all, R.p * (double)all};
  u64 over = __ballot(mine && !((double)coarse_through < f.least));
  if (over) {
    const int cb = __ffsll((unsigned long long)over) - 1;
    u64 before;
    mine = fine(cb, before);
    over = __ballot(mine && !((double)(before + mine) < f.least));
    const int b = __ffsll((unsigned long long)over) - 1;   // (there is one: the coarse bin reaches the limit)
    f.lo = f.hi = cb * kFine + b;
    f.before = (u64)__shfl((long long)before, b);
  }
  if (R.least_w > 0) {
    // min-p's border, where what rounds up to least_w begins (so x > log(2^-41) > -kSpan): nearly always in one bin
    const double x = log(((double)R.least_w - 0.5) * 0x1p-40);
    f.hi = min(f.hi, bin_of(fmax(x - 1e-6, -kSpan)));
    const int m = bin_of(fmin(x + 1e-6, 0.0));
    if (m < f.lo) {
      f.lo = m;
      u64 before;
      fine(f.lo / kFine, before);
      f.before = (u64)__shfl((long long)before, f.lo % kFine);
    }
  }
  return f;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_gather_kernel(SampleRows a, Space s, Sizes z) {
  constexpr int kPieces = 64 / 16 * sizeof(T) / 4;   // (16 elements)
  __shared__ Gathered L;
  __shared__ Shared S;
  const int row = blockIdx.y, c = blockIdx.x;
  if (a.top_k && a.top_k[row] > 0) return;
  const T* p = reinterpret_cast<const T*>(a.logits) + row * a.stride;
  const Elements<kPieces, T> elements(p, c * z.chunk, min(a.vocab, (c + 1) * z.chunk));
  const Row R = row_of(a, s, z, row, S);
  if (R.greedy || R.top == kNanKey || R.top <= kNoneKey || !R.by_mass) return;
  const Limit f = limit_of(R, s, z, row, S);
  if (f.lo == kBins) return;
  if (threadIdx.x == 0) L.count = 0;
  __syncthreads();
  // (a first look in fp32, with room for what its roundings and the bins' are off: nearly all end there)
  const double bin = kSpan / kBins / R.inv;
  const float below = nextafterf((float)(R.zmax - (f.hi + 1.01) * bin), -__builtin_inff());
  const float above = nextafterf((float)(R.zmax - (f.lo - 0.01) * bin), __builtin_inff());
  elements.each([&](float v, int i) {
    if (!(v >= below && v <= above)) return;
    const double x = R.arg(v);
    if (x < -kSpan) return;
    const int b = bin_of(x);
    if (b >= f.lo && b <= f.hi) gather(L, v, i);
  });
  append(L, s, row);
}

// ---------------------------------------------------------------- draw
struct DrawSpace {
  struct {
    u64 key, w;
  } pair[kPairs];
  u64 list[kCap];
  u64 bins[kBins];
  uint32_t count[kBins];
  u64 sums[kThreads / 64];
  u64 chunk[kMaxChunks];
  u64 round[4][kThreads / 64];
  u64 lo, hi, before;
  int found, several;
};

// The elements that a limit is looked for among: the row's list (in LDS), or (list NULL) the row itself.
template <typename T>
struct Among {
  static constexpr int kPieces = 2, kAtOnce = kPieces * Elements<1, T>::E * kThreads;
  const T* logits;
  const u64* list;
  int n;

  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (list)
      for (int i = threadIdx.x; i < n; i += kThreads) f(list[i]);
    else
#pragma unroll 1
      for (int first = 0; first < n; first += kAtOnce) {
        const Elements<kPieces, T> elements(logits, first, min(n, first + kAtOnce));
        elements.each([&](float v, int i) { f(full_key(v, i)); });
      }
  }
};

// The smallest key that stays, where those stay that come, from the greatest key down, before the limit,
// with `base` before all of them; `floor` where all that are >= floor stay (others are not looked at).
// Bins over the keys, narrowed until the limit's bin has one element.
template <typename T>
__device__ __forceinline__ u64 find_cut(const Among<T>& among, const Row& R, DrawSpace& L, bool by_count, double least,
                                     u64 base, u64 floor) {
  if (threadIdx.x == 0) L.lo = ~0ull, L.hi = 0;
  __syncthreads();
  u64 lo = ~0ull, hi = 0;
  among.each([&](u64 key) {
    if (key >= floor && weight_of(R, key)) lo = min(lo, key), hi = max(hi, key);
  });
  lo = ~wave_max64(~lo);
  hi = wave_max64(hi);
  if ((threadIdx.x & 63) == 0) {
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
    for (int b = threadIdx.x; b < kBins; b += kThreads) L.bins[b] = 0, L.count[b] = 0;
    if (threadIdx.x == 0) L.found = kBins;
    __syncthreads();
    among.each([&](u64 key) {
      if (key < lo || key > hi) return;
      const u64 w = weight_of(R, key);
      if (!w) return;
      const int b = (int)((hi - key) >> shift);
      atomicAdd(&L.bins[b], by_count ? 1ull : w);
      atomicAdd(&L.count[b], 1u);
    });
    __syncthreads();
    // the first bin through which the limit is reached, and what stands before it
    constexpr int kPer = kBins / kThreads;
    u64 n[kPer], mine = 0, all;
#pragma unroll
    for (int j = 0; j < kPer; ++j) mine += n[j] = L.bins[threadIdx.x * kPer + j];
    u64 through = base + group_scan(mine, L.sums, all), in_front = 0;
    int first = kBins;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (first == kBins && n[j] && crossed(by_count, through + n[j], R.k, least)) {
        first = threadIdx.x * kPer + j;
        in_front = through;
      }
      through += n[j];
    }
    if (first < kBins) atomicMin(&L.found, first);
    __syncthreads();
    const int b = L.found;
    if (b == kBins) return floor;   // never reached: all stay
    if (first == b) L.before = in_front;
    __syncthreads();
    base = L.before;
    const uint32_t here = L.count[b];
    hi -= (u64)b << shift;
    const u64 width = (1ull << shift) - 1;
    lo = hi - lo > width ? hi - width : lo;
    if (here == 1 || shift == 0) return lo;
  }
}

// The same where the list holds the elements of the bins f.lo to f.hi and the limit is one of mass: these bins
// are divided into kThreads, and in the one that the limit falls into few elements are left, which are
// compared each with each.  False where they are not few.
__device__ __forceinline__ bool cut_of_bins(const Row& R, const Limit& f, DrawSpace& L, int n, u64& cut) {
  constexpr int kAtOnce = 128;   // so few are compared without the bins
  const int t = threadIdx.x;
  int m = n;
  u64 in_front = f.before;
  cut = 0;
  if (t == 0) L.lo = ~0ull;
  if (n <= kAtOnce) {
    if (n == 0) return true;
    if (t < n) L.pair[t] = {L.list[t], weight_of(R, L.list[t])};
    __syncthreads();
  } else {
    L.bins[t] = 0;
    if (t == 0) L.found = kBins, L.several = 0;
    __syncthreads();
    const float first = (float)f.lo, scale = (float)kThreads / (float)(f.hi + 1 - f.lo);
    auto part_of = [&](u64 key) {   // (monotone, as bin_of is)
      const float b = (float)-R.arg(key_value((uint32_t)(key >> 32))) * (float)(kBins / kSpan);
      return max(0, min(kThreads - 1, (int)((b - first) * scale)));
    };
#pragma unroll 1
    for (int i = t; i < n; i += kThreads) {
      const u64 key = L.list[i];
      atomicAdd(&L.bins[part_of(key)], weight_of(R, key));
    }
    __syncthreads();
    const u64 mine = L.bins[t];
    u64 all;
    const u64 before = f.before + group_scan(mine, L.sums, all);
    const bool here = mine && !((double)(before + mine) < f.least) && ((double)before < f.least || before == 0);
    if (here) L.found = t, L.before = before;
    __syncthreads();
    const int b = L.found;
    if (b == kBins) return true;   // not reached: all stay
    in_front = L.before;
#pragma unroll 1
    for (int i = t; i < n; i += kThreads) {
      const u64 key = L.list[i];
      if (part_of(key) == b) {
        const int place = atomicAdd(&L.several, 1);
        if (place < kPairs) L.pair[place] = {key, weight_of(R, key)};
      }
    }
    __syncthreads();
    m = L.several;
    if (m > kPairs) return false;
  }
  int split = kThreads / kPairs;   // threads of an element: neighbours, a power of two
  while (split < 64 && 2 * split * m <= kThreads) split *= 2;
  const int i = t / split;
  u64 key = 0, mass = 0;
  if (i < m) {
    key = L.pair[i].key;
#pragma unroll 2
    for (int j = t % split; j < m; j += split) mass += L.pair[j].key > key ? L.pair[j].w : 0;
  }
  for (int d = 1; d < split; d <<= 1) mass += (u64)__shfl_xor((long long)mass, d);
  in_front += mass;
  const bool stays = i < m && ((double)in_front < f.least || in_front == 0);
  const u64 lowest = ~wave_max64(stays ? ~key : 0);
  if ((t & 63) == 0 && lowest != ~0ull) atomicMin(&L.lo, lowest);
  __syncthreads();
  cut = L.lo;
  return true;
}

// The number that is drawn, of a sum of `total`.
__device__ __forceinline__ u64 drawn(float u, u64 total) {
  const u64 at = (u64)floor((double)total * (double)(u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f));
  return at < total - 1 ? at : total - 1;
}
__device__ __forceinline__ void give(const SampleRows& a, int row, int token, u64 w, u64 total) {
  a.tokens[row] = token;
  if (a.share) a.share[row] = (float)((double)w / (double)total);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(SampleRows a, Space s, Sizes z) {
  __shared__ DrawSpace L;
  __shared__ Shared S;
  const int row = blockIdx.x, tid = threadIdx.x;
  // (asked for before the settings are there)
  const float number = a.uniform[row];
  const uint32_t length = s.length[(size_t)row * kApart];
  const u64 chunk_sum = tid < z.chunks ? s.sum[(size_t)row * z.chunks + tid] : 0;
  const Row R = row_of(a, s, z, row, S);
  const T* p = reinterpret_cast<const T*>(a.logits) + row * a.stride;
  if (R.top == kNanKey || R.top <= kNoneKey) {
    if (tid == 0) {
      a.tokens[row] = -1;
      if (a.share) a.share[row] = 0.0f;
    }
    return;
  }
  if (R.greedy) {
    // the first chunk with the largest logit, then the first element in it
    if (tid == 0) L.found = kParts;
    __syncthreads();
    if (S.tops[tid] == R.top) atomicMin(&L.found, tid);
    __syncthreads();
    const int c = L.found / z.parts;
    __syncthreads();
    if (tid == 0) L.found = a.vocab;
    __syncthreads();
    int least = a.vocab;
    const Elements<kAhead<T>, T> elements(p, c * z.chunk, min(a.vocab, (c + 1) * z.chunk));
    elements.each([&](float v, int i) {
      if (order_key(v) == R.top) least = min(least, i);
    });
    if (least < a.vocab) atomicMin(&L.found, least);
    __syncthreads();
    if (tid == 0) {
      a.tokens[row] = L.found;
      if (a.share) a.share[row] = 1.0f;
    }
    return;
  }

  u64 cut = 0;
  Limit f{0, 0, 0, 0.0};
  const bool listed = length <= (uint32_t)kCap;
  const int n = listed ? (int)length : a.vocab;
  if (R.limited() && listed && !R.by_count) f = limit_of(R, s, z, row, S);
  if (R.limited() && listed) {
    for (int i = tid; i < n; i += kThreads) L.list[i] = s.list[(size_t)row * kCap + i];
  }
  const Among<T> among{p, listed ? L.list : nullptr, n};
  __syncthreads();
  if (R.by_count && n <= kPairs && listed) {
    // ---- a short list: for each element what comes before it; threads share an element where there are few
    if (tid < n) L.pair[tid] = {L.list[tid], weight_of(R, L.list[tid])};
    double least = 0.0;
    __syncthreads();
    int split = kThreads / kPairs;   // threads of an element: neighbours, a power of two
    while (split < 64 && 2 * split * n <= kThreads) split *= 2;
    const int i = tid / split, part = tid % split;
    const bool first = part == 0;    // (one thread of an element counts it)
    u64 key = 0, w = 0, mass = 0;
    int rank = 0;
    if (i < n) key = L.pair[i].key, w = L.pair[i].w;
#pragma unroll 4
    for (int j = part; j < n; j += split) {
      const auto e = L.pair[j];
      const bool before = e.key > key;
      mass += before ? e.w : 0;
      rank += before;
    }
    for (int d = 1; d < split; d <<= 1) {
      mass += (u64)__shfl_xor((long long)mass, d);
      rank += __shfl_xor(rank, d);
    }
    if (R.by_mass) least = R.p * (double)group_sum(first && rank < R.k ? w : 0, L.sums);
    if (!(rank < R.k && (!R.by_mass || rank == 0 || (double)mass < least) && w >= R.least_w)) w = 0;
    const u64 total = group_sum(first ? w : 0, L.sums), at = drawn(number, total);
    if (first && i < n) L.pair[i].w = w;
    __syncthreads();
    // the weights of lower indices: those with a greater lower half of the key
    u64 start = 0;
#pragma unroll 4
    for (int j = part; j < n; j += split) {
      const auto e = L.pair[j];
      start += (uint32_t)e.key > (uint32_t)key ? e.w : 0;
    }
    for (int d = 1; d < split; d <<= 1) start += (u64)__shfl_xor((long long)start, d);
    if (first && w && start <= at && at < start + w) give(a, row, index_of(key), w, total);
    return;
  } else if (!(R.by_mass && !R.by_count && listed && cut_of_bins(R, f, L, n, cut)) && R.limited()) {
#pragma unroll 1
    for (int by_count = 1; by_count >= 0; --by_count) {   // top-k first
      if (!(by_count ? R.by_count : R.by_mass)) continue;
      double least = f.least;
      if (!by_count && (R.by_count || !listed)) {
        u64 sum = 0;
        among.each([&](u64 key) { sum += key >= cut ? weight_of(R, key) : 0; });
        least = R.p * (double)group_sum(sum, L.sums);
      }
      cut = find_cut(among, R, L, by_count, least, listed ? f.before : 0, cut);
    }
  }

  // ---- the chunks' sums of what stays
  __syncthreads();
  if (tid < kMaxChunks) L.chunk[tid] = R.limited() ? 0 : chunk_sum;
  __syncthreads();
  if (R.limited()) {
    if (listed && !R.by_count) {
      // the bins that stay whole, a wave per chunk
      const int cb = f.lo / kFine, lane = tid & 63;
      for (int c = tid >> 6; c < z.chunks; c += kThreads / 64) {
        const size_t at = (size_t)row * z.chunks + c;
        u64 sum = lane < cb ? s.coarse[at * kCoarse + lane] : 0;
        if (f.lo < kBins && lane < f.lo % kFine) sum += s.bins[at * kBins + cb * kFine + lane];
        sum = (u64)wave_scan((long long)sum);
        if (lane == 63) L.chunk[c] = sum;
      }
      __syncthreads();
    }
    // (a list of top-k holds everything that stays, and f no bin then)
    among.each([&](u64 key) {
      const u64 w = key >= cut ? weight_of(R, key) : 0;
      if (w && w >= R.least_w) atomicAdd(&L.chunk[(uint32_t)index_of(key) / (uint32_t)z.chunk], w);
    });
  }
  __syncthreads();

  // ---- the chunk that the number falls into
  u64 total;
  const u64 mine = tid < z.chunks ? L.chunk[tid] : 0;
  u64 before = group_scan(mine, L.sums, total);
  const u64 at = drawn(number, total);
  if (mine && before <= at && at < before + mine) {
    L.found = tid;
    L.lo = before;
  }
  __syncthreads();
  const int c = L.found;
  const u64 start = L.lo;

  // ---- the element in it, in rounds of kRound pieces of 16 bytes per thread: the pieces' sums by wave, then
  //      the wave that the number falls into, its lane, and the element
  constexpr int kWaves = kThreads / 64, kRound = 4, E = 16 / sizeof(T);
  const int wave = tid >> 6, lane = tid & 63;
  u64 in_front = start;
  auto kept = [&](float v, int i) {
    const u64 w = full_key(v, i) >= cut ? weight_of(R, v) : 0;
    return w >= R.least_w ? w : 0;
  };
  const int end = min(a.vocab, (c + 1) * z.chunk);
  for (int first = c * z.chunk; first < end; first += kRound * kThreads * E) {
    typename Elements<1, T>::Piece q[kRound];
    u64 through[kRound];
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      const int i = first + E * (u * kThreads + tid);
#pragma unroll
      for (int e = 0; e < E; ++e) q[u].v[e] = (T)(-__builtin_inff());
      if (first + E * u * kThreads >= end) continue;   // (none for any thread)
      if (i + E <= end) {
        q[u] = *reinterpret_cast<const typename Elements<1, T>::Piece*>(p + i);
      } else {
        for (int e = 0; e < E; ++e)
          if (i + e < end) q[u].v[e] = p[i + e];
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      u64 sum = 0;
      if (first + E * u * kThreads < end) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum += kept((float)q[u].v[e], first + E * (u * kThreads + tid) + e);
      }
      through[u] = (u64)wave_scan((long long)sum);
      if (lane == 63) L.round[u][wave] = through[u];
    }
    __syncthreads();
    // (every wave for itself: lane l has the l-th of the sums)
    const u64 mine = lane < kRound * kWaves ? L.round[lane / kWaves][lane % kWaves] : 0;
    const u64 upto = in_front + (u64)wave_scan((long long)mine);
    const u64 hit = __ballot(at < upto);
    if (hit) {
      const int x = __ffsll((unsigned long long)hit) - 1;
      const u64 from = (u64)__shfl((long long)(upto - mine), x);
#pragma unroll
      for (int u = 0; u < kRound; ++u)
        if (x == u * kWaves + wave) {
          // (before this lane's piece: the sum of the lanes in front)
          u64 before = (u64)__shfl_up((long long)through[u], 1);
          before = from + (lane ? before : 0);
          if (before <= at && at < from + through[u]) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const int i = first + E * (u * kThreads + tid) + e;
              const u64 w = kept((float)q[u].v[e], i);
              if (w && before <= at && at < before + w) give(a, row, i, w, total);
              before += w;
            }
          }
        }
      break;
    }
    in_front = (u64)__shfl((long long)upto, 63);
  }
}

template <typename T>
hipError_t launch(const SampleRows& all, hipStream_t st) {
  const Sizes z = sizes(all.rows, all.vocab);
  const int most = batch(all.rows, z);
  Space s;
  place(s, all.ws, most, z);
  for (int first = 0; first < all.rows; first += most) {
    SampleRows a = all;
    a.rows = all.rows - first < most ? all.rows - first : most;
    a.logits = reinterpret_cast<const T*>(all.logits) + first * all.stride;
    a.temperature += first;
    a.uniform += first;
    if (a.top_k) a.top_k += first;
    if (a.top_p) a.top_p += first;
    if (a.min_p) a.min_p += first;
    a.tokens += first;
    if (a.share) a.share += first;
    const dim3 grid(z.chunks, a.rows);
    hipLaunchKernelGGL((sample_max_kernel<T>), grid, dim3(kThreads), 0, st, a, s, z);
    hipLaunchKernelGGL((sample_mass_kernel<T>), grid, dim3(kThreads), 0, st, a, s, z);
    if (a.top_p) hipLaunchKernelGGL((sample_gather_kernel<T>), grid, dim3(kThreads), 0, st, a, s, z);
    hipLaunchKernelGGL((sample_draw_kernel<T>), dim3(a.rows), dim3(kThreads), 0, st, a, s, z);
  }
  return hipGetLastError();
}

}  // namespace

size_t sample_workspace_bytes(int rows, int vocab) {
  Space s;
  const Sizes z = sizes(rows, vocab);
  return place(s, nullptr, batch(rows, z), z);
}

hipError_t launch_sample(const SampleRows& a, int logits_fp32, hipStream_t stream) {
  return logits_fp32 ? launch<float>(a, stream) : launch<__bf16>(a, stream);
}

}  // namespace svdq
