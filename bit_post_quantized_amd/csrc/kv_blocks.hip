// The paged KV cache held in 8 bits with a scale for each block of tokens and head: block tables
// and slot maps, the append and the read-back (svdq_serve.h has the layouts and rules; VARC "INT8
// KV cache quantization": the codes of a cache that decoding keeps growing).
#include "serve_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {

// ------------------------------------------------------------------------------ block tables
// One launch.  Every workgroup scans the lengths of all requests (a few KB, from L2) in chunks of
// its threads, and handles one range of kPlanRows rows: a thread finds its row's request among
// those the scan left in LDS, takes the block from the table or, for a block the step adds, from
// the free list, and writes the table entry if it is the block's first row.  Workgroup 0 also
// writes what there is one of per request.  So no workgroup waits for another, and the launch is
// latency: 5.2 us for 8 requests of a row, 5.8 for 1000 with 65536 rows together (three block scans
// per 1024 requests, and loads that depend on each other; 6.5 and 7.2 with shuffles in the scans).
constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 1024;

__device__ __forceinline__ int clamp0(int x) { return x < 0 ? 0 : x; }

// Adds what the waves before have (`total`: of this wave, in its last lane); sum: of all.  One barrier:
// two scans that follow each other take different `lds`.
__device__ __forceinline__ long long waves_before(long long total, long long* lds, long long& sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 63) lds[wave] = total;
  __syncthreads();
  long long before = 0;
  sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    const long long x = lds[w];
    if (w < wave) before += x;
    sum += x;
  }
  return before;
}

// Inclusive sums of one value per thread over the workgroup, in 64 bits.
__device__ __forceinline__ long long block_scan(long long v, long long* lds, long long& sum) {
  v = wave_scan(v);
  return v + waves_before(v, lds, sum);
}

__global__ __launch_bounds__(kPlanThreads) void kv_block_plan_kernel(
    const int32_t* __restrict__ ctx, const int32_t* __restrict__ add, int requests,
    int32_t* __restrict__ tables, int width, int shift, const int32_t* __restrict__ free_blocks,
    int capacity, const int32_t* __restrict__ free_count, int32_t* __restrict__ cu,
    int32_t* __restrict__ seq, int rows, int32_t* __restrict__ positions,
    int64_t* __restrict__ slots, int32_t* __restrict__ status, int32_t* __restrict__ free_out) {
  __shared__ long long scan_lds[3][kPlanThreads / 64];
  // the requests with rows in this workgroup's range, in order: at most one per row
  __shared__ int s_first[kPlanRows], s_ctx[kPlanRows], s_take[kPlanRows], s_req[kPlanRows];
  const int tid = threadIdx.x, bs = 1 << shift;
  const long long row0 = (long long)blockIdx.x * kPlanRows;
  const int row1 = (int)(row0 + kPlanRows < rows ? row0 + kPlanRows : rows);
  const int have = min(clamp0(free_count[0]), capacity);
  const bool head = blockIdx.x == 0;
  long long cu_base = 0, need_base = 0, taken = 0;
  int found = 0;  // requests in LDS so far (the same in every thread)

  for (int b0 = 0; b0 < requests; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int c = b < requests ? clamp0(ctx[b]) : 0;
    const int n = b < requests ? clamp0(add[b]) : 0;
    long long sum;
    const long long cu1 = cu_base + block_scan(n, scan_lds[0], sum), first = cu1 - n;
    cu_base += sum;
    const long long end = ((long long)c + n + bs - 1) >> shift;
    const int held = (int)(((long long)c + bs - 1) >> shift);
    int st = end > width ? 2 : cu1 > rows ? 3 : 0;
    const long long need = st ? 0 : end - held;
    const long long incl = need_base + block_scan(need, scan_lds[1], sum);
    need_base += sum;
    if (need > 0 && incl > have) st = 1;
    // blocks really taken: the prefix up to the first request that did not get its blocks
    if (st == 0 && need > 0 && incl > taken) taken = incl;
    if (head && b < requests) {
      cu[b + 1] = (int)(cu1 > 0x7FFFFFFFLL ? 0x7FFFFFFFLL : cu1);
      seq[b] = st ? c : c + n;
      status[b] = st;
    }
    // this range's requests (those with rows in it): compacted into LDS in order
    const bool mine = n > 0 && first < row1 && cu1 > row0;
    const uint64_t all = __ballot(mine);
    const int at = __popcll(all & ((1ull << (tid & 63)) - 1)) + (int)waves_before(__popcll(all), scan_lds[2], sum);
    if (mine) {
      const int i = found + at;  // < kPlanRows: each has a row of its own in the range
      s_first[i] = (int)first;
      s_ctx[i] = c;
      s_take[i] = st ? -1 : (int)(incl - need);
      s_req[i] = b;
    }
    found += (int)sum;
    if (!head && cu_base >= row1) break;  // (uniform: later requests have no row here)
  }
  if (head) {
    // the largest `taken` of any thread
    for (int o = 1; o < 64; o <<= 1) {
      const long long u = __shfl_xor(taken, o);
      taken = u > taken ? u : taken;
    }
    if ((tid & 63) == 0) scan_lds[0][tid >> 6] = taken;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kPlanThreads / 64; ++w) taken = scan_lds[0][w] > taken ? scan_lds[0][w] : taken;
      free_out[0] = have - (int)taken;
      cu[0] = 0;
    }
  }
  __syncthreads();

  for (long long t = row0 + tid; t < row1; t += kPlanThreads) {
    // the last request that begins at or before row t; rows behind the last request find none
    int lo = 0, hi = found;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] <= t) lo = mid + 1; else hi = mid;
    }
    int pos = 0;
    long long slot = -1;
    if (lo > 0 && t < cu_base) {
      const int i = lo - 1, b = s_req[i], c = s_ctx[i], take = s_take[i];
      const long long p = (long long)c + (t - s_first[i]);
      pos = (int)(p > 0x7FFFFFFFLL ? 0x7FFFFFFFLL : p);
      if (take >= 0) {  // the table holds every position of the request
        const int blk = pos >> shift, held = (int)(((long long)c + bs - 1) >> shift);
        int32_t* entry = tables + (size_t)b * width + blk;
        int id;
        if (blk < held) {
          id = *entry;
        } else {
          id = free_blocks[have - 1 - (take + blk - held)];
          if ((pos & (bs - 1)) == 0) *entry = id;
        }
        slot = id < 0 ? -1 : (long long)id * bs + (pos & (bs - 1));
      }
    }
    positions[t] = pos;
    slots[t] = slot;
  }
}

hipError_t launch_kv_block_plan(const int32_t* ctx, const int32_t* add, int requests,
                                int32_t* tables, int width, int bs, const int32_t* free_blocks,
                                int capacity, const int32_t* free_count, int32_t* cu,
                                int32_t* seq, int rows, int32_t* positions, int64_t* slots,
                                int32_t* status, int32_t* free_out, hipStream_t stream) {
  const int grid = rows > 0 ? (rows + kPlanRows - 1) / kPlanRows : 1;
  hipLaunchKernelGGL(kv_block_plan_kernel, dim3(grid), dim3(kPlanThreads), 0, stream, ctx, add,
                     requests, tables, width, __builtin_ctz(bs), free_blocks, capacity,
                     free_count, cu, seq, rows, positions, slots, status, free_out);
  return hipGetLastError();
}

// One workgroup per request (and one more for the count): it scans the finished requests before
// its own, then moves its blocks to the free list.
__global__ __launch_bounds__(kPlanThreads) void kv_block_release_kernel(
    const int32_t* __restrict__ seq, const uint8_t* __restrict__ done, int requests,
    int32_t* __restrict__ tables, int width, int shift, int32_t* __restrict__ free_blocks,
    int capacity, const int32_t* __restrict__ free_count, int32_t* __restrict__ seq_out,
    int32_t* __restrict__ free_out) {
  __shared__ long long scan_lds[2][kPlanThreads / 64];
  const int me = blockIdx.x, tid = threadIdx.x, bs = 1 << shift;
  const int have = min(clamp0(free_count[0]), capacity);
  const bool last = me == requests, mine = !last && done[me];
  if (!last && tid == 0) seq_out[me] = mine ? 0 : seq[me];
  if (!last && !mine) return;
  long long before = 0;
  int par = 0;
  for (int b0 = 0; b0 < me; b0 += kPlanThreads, par ^= 1) {
    const int b = b0 + tid;
    long long v = 0, sum;
    if (b < me && done[b]) {
      v = ((long long)clamp0(seq[b]) + bs - 1) >> shift;
      if (v > width) v = width;
    }
    waves_before(wave_scan(v), scan_lds[par], sum);
    before += sum;
  }
  if (last) {
    if (tid == 0) {
      const long long n = (long long)have + before;
      free_out[0] = (int)(n < capacity ? n : capacity);
    }
    return;
  }
  long long mineb = ((long long)clamp0(seq[me]) + bs - 1) >> shift;
  if (mineb > width) mineb = width;
  for (int j = tid; j < width; j += kPlanThreads) {
    int32_t* entry = tables + (size_t)me * width + j;
    if (j < mineb) {
      const long long at = (long long)have + before + j;
      if (at < capacity) free_blocks[at] = *entry;
    }
    *entry = -1;
  }
}

hipError_t launch_kv_block_release(const int32_t* seq, const uint8_t* done, int requests,
                                   int32_t* tables, int width, int bs, int32_t* free_blocks,
                                   int capacity, const int32_t* free_count, int32_t* seq_out,
                                   int32_t* free_out, hipStream_t stream) {
  hipLaunchKernelGGL(kv_block_release_kernel, dim3(requests + 1), dim3(kPlanThreads), 0, stream,
                     seq, done, requests, tables, width, __builtin_ctz(bs), free_blocks, capacity,
                     free_count, seq_out, free_out);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------ append
// A run is the rows of one block: it begins at a row whose predecessor is not the slot before it,
// or at a block's first slot, and goes on while the slots ascend inside the block.  One workgroup
// per (window of rows, head) writes the runs that begin in its window, K's and V's rows together.
// Every wave finds them by itself: a lane looks at one row, and the rows where a run breaks are
// three 64-bit masks.
//  - Short runs (up to kShort rows: decoding) go to groups of D / 8 lanes, one run to a group, all
//    at once.
//  - A long run (a prompt's block) takes the whole workgroup: its rows are read once, 8 channels
//    and 4 consecutive rows to a thread and step, all loads before the largest magnitude is known;
//    K's codes are stored as they are, V's go through LDS to become rows of tokens.
// 20000 rows of 8 x 128 (82 MB in, 41 MB out) take 33 to 35 us, 3.6 TB/s: the loads alone 21, the
// coding 2 of the rest.  Measured: non-temporal stores 3 us less, but the read of the codes that
// follows takes 3 us more; K and V in workgroups of their own the same; a clamp and float conversions in
// the coding 14 us more.
constexpr int kAppendThreads = 256;
constexpr int kShort = 4;

// Rows of a window: a block's worth (at most 64) where that makes enough workgroups, so that a
// prompt's window begins a run; less for few rows, where a window's short runs would queue up.
inline int append_window(int rows, int heads, int bs) {
  int w = bs < 64 ? bs : 64;
  while (w > 16 && (long long)(rows / w) * heads < 1024) w /= 2;
  return w;
}

// What turns a value into a code + 128 under the block scale s: the correctly rounded quotient
// (div_rn) plus 1.5 2^23 + 128, whose low byte is then the code to the nearest even.  s is amax / 127
// rounded, by 2^-24 of it or, among the subnormal numbers, by 2^-150 of 2^-140 at least, so |x / s| is
// at most 127 (1 + 2^-10) < 127.5 and no code needs a clamp.  The correction step needs a normal
// reciprocal, so a scale below 2^-80 and its values are taken 2^64 times larger (exact, the quotient is
// the same).  s = 0: every value of the block is 0, and so is every quotient by 1.  A scale that is NaN
// or infinite gives the values `times` 0, and their codes 0, by the same branch.
struct Coder {
  float s, rcp, times;  // values times that (1: none)
};

__device__ __forceinline__ Coder coder_of(float s) {
  const bool tiny = s < 0x1p-80f, finite = s < __builtin_inff();
  Coder k;
  k.times = tiny ? 0x1p64f : finite ? 1.0f : 0.0f;
  k.s = s == 0.0f || !finite ? 1.0f : tiny ? s * 0x1p64f : s;
  k.rcp = 1.0f / k.s;
  return k;
}

// The larger of two scales; a NaN stays one.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ uint32_t kv_code_bits(float x, Coder k) {
  return __float_as_uint(div_rn(x, k.s, k.rcp) + 12583040.0f);
}

// Eight bf16 of a 16-byte load as fp32.
__device__ __forceinline__ void bf16x8(v4u w, float* x) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(ws[e] << 16);
    x[2 * e + 1] = __uint_as_float(ws[e] & 0xFFFF0000u);
  }
}

// Largest magnitudes as bf16 bits without the sign, two to a dword (they order like integers, infinity
// and then NaN last).
typedef uint16_t v2s __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2s, a), __builtin_bit_cast(v2s, b)));
}

__device__ __forceinline__ uint32_t amax8(v4u w, uint32_t amax) {
#pragma unroll
  for (int e = 0; e < 4; ++e) amax = pk_max(amax, w[e] & 0x7FFF7FFFu);
  return amax;
}

// ... over the lanes that differ in the bits below `lanes`, as fp32 in every one of them.
__device__ __forceinline__ float amax_lanes(uint32_t amax, int lanes) {
  amax = pk_max(amax, amax >> 16);
  for (int o = 1; o < lanes; o <<= 1) amax = pk_max(amax, __shfl_xor(amax, o));
  return __uint_as_float(amax << 16);
}

// Codes of one row's 8 channels (byte e: channel e).
__device__ __forceinline__ v2u codes8(v4u w, Coder k) {
  float x[8];
  bf16x8(w, x);
  if (k.times != 1.0f)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = k.times == 0.0f ? 0.0f : x[e] * k.times;
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = kv_code_bits(x[e], k);
  // the low bytes of four words -> one dword
  auto low4 = [](const uint32_t* v) {
    const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(v[3], v[2], 0x04000C0Cu);
    return lo | hi;
  };
  return v2u{low4(b), low4(b + 4)};
}

// The first `n` bytes of a dword of codes under a grown scale; the others as they are.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio, int n) {
  uint32_t r = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float c = (float)((w >> (8 * e)) & 0xFFu);
    r = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_rintf((c - 128.0f) * ratio) + 128.0f, e, r);
  }
  const uint32_t keep = n >= 4 ? 0u : ~0u << (8 * n);
  return (r & ~keep) | (w & keep);
}

// ... and of the first `n` bytes of 16.
__device__ __forceinline__ v4u rescale16(v4u w, float ratio, int n) {
  return v4u{rescale4(w.x, ratio, max(n, 0)), rescale4(w.y, ratio, max(n - 4, 0)),
             rescale4(w.z, ratio, max(n - 8, 0)), rescale4(w.w, ratio, max(n - 12, 0))};
}

// The codes of a block's first `off` tokens under a grown scale: K's rows or V's rows of tokens, the
// 16-byte pieces i, i + step, ... of them, AHEAD loads in flight.  (One token each to 64 x 8 blocks of
// 127 that all grow: 42 us, 135 with a dword at a time; without growth 6.)
template <int D, bool V, int AHEAD>
__device__ __forceinline__ void rescale_block(uint8_t* codes, int bs, int off, float ratio, int i, int step) {
  const int per = (off + 15) / 16, all = V ? D * per : off * D / 16;  // V: pieces of a channel
  for (; i < all; i += AHEAD * step) {
    v4u* p[AHEAD];
    v4u w[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int at = min(i + u * step, all - 1);
      p[u] = reinterpret_cast<v4u*>(V ? codes + (size_t)(at / per) * bs + 16 * (at % per) : codes + 16 * at);
      w[u] = *p[u];
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (i + u * step < all) *p[u] = rescale16(w[u], ratio, V ? off - 16 * ((i + u * step) % per) : 16);
  }
}

// STEPS: of 4 rows per group of lanes, for the longest run.
template <int D, int STEPS>
__global__ __launch_bounds__(kAppendThreads) void kv_block_append_kernel(
    const uint16_t* __restrict__ kx, const uint16_t* __restrict__ vx, int64_t k_stride,
    int64_t v_stride, const int64_t* __restrict__ slots, int rows, int shift, int window,
    BlockCacheView c) {
  constexpr int TPR = D / 8;                       // lanes per row, 8 channels each
  constexpr int GROUPS = kAppendThreads / TPR;
  constexpr int PITCH = 4 * GROUPS * STEPS + 4;    // of a channel's tokens in LDS, bytes
  __shared__ float wmax[2][kAppendThreads / 64];
  __shared__ __attribute__((aligned(16))) uint8_t vt[D * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // head fastest: the workgroups that run together read whole rows between them
  const int h = blockIdx.x % c.heads, bs = 1 << shift;
  const int part = tid % TPR, group = tid / TPR;
  kx += (size_t)h * D + 8 * part;
  vx += (size_t)h * D + 8 * part;
  const int64_t limit = (int64_t)c.num_blocks << shift;
  const int row0 = (int)(blockIdx.x / c.heads) * window;

  // rows row0 + 0 .. 191: where a run (or a row without a token) begins
  uint64_t brk[3], lead = 0;
  int64_t first64 = -1;  // slot of row row0 + lane
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const int t = row0 + 64 * q + lane, at = min(t, rows - 1);
    const int64_t s = slots[at], before = slots[max(at - 1, 0)];
    const bool valid = t < rows && s >= 0 && s < limit;
    brk[q] = __ballot(!valid || (s & (bs - 1)) == 0 || at == 0 || before != s - 1);
    if (q == 0) {
      lead = __ballot(valid && lane < window) & brk[0];
      first64 = s;
    }
  }
  auto length = [&](int i) {  // rows of the run that begins at row0 + i
    const uint64_t m = i < 63 ? brk[0] >> (i + 1) : 0;
    if (m) return __builtin_ctzll(m) + 1;
    if (brk[1]) return 64 + __builtin_ctzll(brk[1]) - i;
    return 128 + (brk[2] ? __builtin_ctzll(brk[2]) : 64) - i;
  };
  uint64_t shorts = 0;
  for (uint64_t m = lead; m; m &= m - 1) {
    const int i = __builtin_ctzll(m);
    if (length(i) <= kShort) shorts |= 1ull << i;
  }

  // ---- long runs, the whole workgroup
  for (uint64_t m = lead & ~shorts; m; m &= m - 1) {
    const int i0 = __builtin_ctzll(m), n = length(i0), t = row0 + i0;
    const int64_t slot = __shfl(first64, i0);
    const int off = (int)(slot & (bs - 1));
    const size_t bh = (size_t)(slot >> shift) * c.heads + h;
    uint8_t* const kc = c.k_codes + bh * bs * D;
    uint8_t* const vc = c.v_codes + bh * bs * D;
    v4u wk[STEPS][4], wv[STEPS][4];
#pragma unroll
    for (int p = 0; p < STEPS; ++p)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // (rows past the run read its last one)
        const size_t at = (size_t)(t + min(4 * (group + GROUPS * p) + r, n - 1));
        wk[p][r] = *reinterpret_cast<const v4u*>(kx + at * k_stride);
        wv[p][r] = *reinterpret_cast<const v4u*>(vx + at * v_stride);
      }
    const float k_old = off == 0 ? 0.0f : c.k_scale[bh], v_old = off == 0 ? 0.0f : c.v_scale[bh];
    uint32_t k_top = 0, v_top = 0;
#pragma unroll
    for (int p = 0; p < STEPS; ++p)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        k_top = amax8(wk[p][r], k_top);
        v_top = amax8(wv[p][r], v_top);
      }
    float ka = amax_lanes(k_top, 64), va = amax_lanes(v_top, 64);
    if (lane == 0) {
      wmax[0][wave] = ka;
      wmax[1][wave] = va;
    }
    __syncthreads();  // (also: every thread has read the old scales)
#pragma unroll
    for (int q = 0; q < kAppendThreads / 64; ++q) {
      ka = larger(ka, wmax[0][q]);
      va = larger(va, wmax[1][q]);
    }
    const float ks = larger(k_old, ka / 127.0f), vs = larger(v_old, va / 127.0f);
    const Coder kk = coder_of(ks), vk = coder_of(vs);
    if (tid == 0) {
      c.k_scale[bh] = ks;
      c.v_scale[bh] = vs;
    }
    if (off > 0 && ks > k_old) rescale_block<D, false, 1>(kc, bs, off, k_old / ks, tid, kAppendThreads);
    if (off > 0 && vs > v_old) rescale_block<D, true, 1>(vc, bs, off, v_old / vs, tid, kAppendThreads);
#pragma unroll
    for (int p = 0; p < STEPS; ++p) {
      const int i = 4 * (group + GROUPS * p);
      if (i >= n) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const v2u q = codes8(wk[p][r], kk);
        if (i + r < n) *reinterpret_cast<v2u*>(kc + (size_t)(off + i + r) * D + 8 * part) = q;
      }
      // four tokens of each of 8 channels as a dword: bytes e of q[0..3]
      v2u q[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) q[r] = codes8(wv[p][r], vk);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t lo_sel = 0x0C0C0400u + 0x0101u * (e & 3), hi_sel = 0x04000C0Cu + 0x01010000u * (e & 3);
        const uint32_t lo = e < 4 ? __builtin_amdgcn_perm(q[1].x, q[0].x, lo_sel) : __builtin_amdgcn_perm(q[1].y, q[0].y, lo_sel);
        const uint32_t hi = e < 4 ? __builtin_amdgcn_perm(q[3].x, q[2].x, hi_sel) : __builtin_amdgcn_perm(q[3].y, q[2].y, hi_sel);
        *reinterpret_cast<uint32_t*>(&vt[(8 * part + e) * PITCH + i]) = lo | hi;
      }
    }
    __syncthreads();  // (the earlier tokens' rescaled pieces are written before bytes in them)
    // V's rows of tokens to the block: 16 bytes at a time where a chunk is whole and in step with
    // LDS (off a multiple of 4), else its bytes
    const int c0 = off >> 4, c1 = (off + n + 15) >> 4, nc = c1 - c0;
    for (int i = tid; i < D * nc; i += kAppendThreads) {
      const int d = i / nc, ch = c0 + i % nc;
      const int lo = max(off, 16 * ch), hi = min(off + n, 16 * ch + 16);
      const uint8_t* from = &vt[d * PITCH + lo - off];
      uint8_t* to = vc + (size_t)d * bs + lo;
      if (hi - lo == 16 && (off & 3) == 0) {
        const uint32_t* f4 = reinterpret_cast<const uint32_t*>(from);
        *reinterpret_cast<v4u*>(to) = v4u{f4[0], f4[1], f4[2], f4[3]};
      } else {
        for (int b = 0; b < hi - lo; ++b) to[b] = from[b];
      }
    }
    __syncthreads();  // (wmax and vt before the next run)
  }

  // ---- short runs, one to a group of lanes
  for (int k = group; k < __popcll(shorts); k += GROUPS) {
    uint64_t m = shorts;
    for (int q = 0; q < k; ++q) m &= m - 1;
    const int i0 = __builtin_ctzll(m), n = length(i0), t = row0 + i0;
    const int64_t slot = slots[t];
    const int off = (int)(slot & (bs - 1));
    const size_t bh = (size_t)(slot >> shift) * c.heads + h;
    uint8_t* const kc = c.k_codes + bh * bs * D;
    uint8_t* const vc = c.v_codes + bh * bs * D;
    v4u wk[kShort], wv[kShort];
#pragma unroll
    for (int r = 0; r < kShort; ++r) {
      wk[r] = *reinterpret_cast<const v4u*>(kx + (size_t)(t + min(r, n - 1)) * k_stride);
      wv[r] = *reinterpret_cast<const v4u*>(vx + (size_t)(t + min(r, n - 1)) * v_stride);
    }
    const float k_old = off == 0 ? 0.0f : c.k_scale[bh], v_old = off == 0 ? 0.0f : c.v_scale[bh];
    uint32_t k_top = 0, v_top = 0;
#pragma unroll
    for (int r = 0; r < kShort; ++r) {
      k_top = amax8(wk[r], k_top);
      v_top = amax8(wv[r], v_top);
    }
    const float ks = larger(k_old, amax_lanes(k_top, TPR) / 127.0f);
    const float vs = larger(v_old, amax_lanes(v_top, TPR) / 127.0f);
    const Coder kk = coder_of(ks), vk = coder_of(vs);
    if (part == 0) {  // (the group's lanes have read them: they are one wave's)
      c.k_scale[bh] = ks;
      c.v_scale[bh] = vs;
    }
    // (a lane rescales the pieces that it writes codes into: its own channels' rows of V)
    if (off > 0 && ks > k_old) rescale_block<D, false, 4>(kc, bs, off, k_old / ks, part, TPR);
    if (off > 0 && vs > v_old) {
      const float ratio = v_old / vs;
#pragma unroll 1
      for (int i = 0; i < 2 * ((off + 15) / 16); ++i) {  // 16 tokens of four channels at a time
        v4u* const p = reinterpret_cast<v4u*>(vc + (size_t)(8 * part + 4 * (i & 1)) * bs + 16 * (i >> 1));
        const int n = off - 16 * (i >> 1);
        v4u w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = p[e * bs / 16];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e * bs / 16] = rescale16(w[e], ratio, n);
      }
    }
#pragma unroll
    for (int r = 0; r < kShort; ++r)
      if (r < n) {
        *reinterpret_cast<v2u*>(kc + (size_t)(off + r) * D + 8 * part) = codes8(wk[r], kk);
        const v2u q = codes8(wv[r], vk);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          vc[(size_t)(8 * part + e) * bs + off + r] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
      }
  }
}

hipError_t launch_kv_block_append(const uint16_t* k, const uint16_t* v, int64_t k_stride,
                                  int64_t v_stride, const int64_t* slots, int rows,
                                  const BlockCacheView& c, hipStream_t stream) {
  const int window = append_window(rows, c.heads, c.bs);
  const dim3 grid((unsigned)((rows + window - 1) / window * c.heads));
  const int shift = __builtin_ctz(c.bs);
#define SVDQ_APPEND(D, STEPS)                                                                       \
  hipLaunchKernelGGL((kv_block_append_kernel<D, STEPS>), grid, dim3(kAppendThreads), 0, stream, k, v, \
                     k_stride, v_stride, slots, rows, shift, window, c)
  if (c.dim == 64) SVDQ_APPEND(64, 1);
  else if (c.bs <= 64) SVDQ_APPEND(128, 1);
  else SVDQ_APPEND(128, 2);
#undef SVDQ_APPEND
  return hipGetLastError();
}

// -------------------------------------------------------------------------------------- read
// One workgroup per (window of 64 rows, head, K or V), head fastest, so that the workgroups that run
// together write whole rows between them.  K: a thread per 8 channels of a row.  V: a thread per
// channel and 16 rows at a time; where these are 16 slots in a row from a multiple of 16 on, save
// those without a token, their codes are one 16-byte load, otherwise a byte per row; the values go
// through LDS to become rows of channels.  20000 rows of 8 x 128 (41 MB in, 82 MB out): 22 us,
// 5.6 TB/s, with the codes still in L2 from the append.
constexpr int kReadRows = 64;

template <int D>
__global__ __launch_bounds__(256) void kv_block_read_kernel(const int64_t* __restrict__ slots,
                                                            int rows, int shift, BlockCacheView c,
                                                            uint16_t* __restrict__ k_out,
                                                            uint16_t* __restrict__ v_out) {
  constexpr int TPR = D / 8, W = kReadRows, PER = 256 / TPR;
  __shared__ __attribute__((aligned(16))) uint16_t vt[W][D + 8];
  const int tid = threadIdx.x, bs = 1 << shift;
  const int h = blockIdx.x % c.heads, is_v = blockIdx.x / c.heads & 1;
  const int window = blockIdx.x / c.heads >> 1;
  const int64_t limit = (int64_t)c.num_blocks << shift;
  const int row0 = window * W, part = tid % TPR, lane = tid & 63;
  auto block_head = [&](int64_t slot) { return (size_t)(slot >> shift) * c.heads + h; };
  // Every wave holds the window's 64 slots, a row to a lane, and which rows have a token.
  const int64_t slot = slots[min(row0 + lane, rows - 1)];
  const uint64_t live = __ballot(row0 + lane < rows && slot >= 0 && slot < limit);
  // (c - 128 is exact, so the product rounds once; 128 s, for an FMA, may be past the largest number)
  auto value = [](uint32_t byte, float scale) { return ((float)byte - 128.0f) * scale; };
  if (!is_v) {
    v2u w[W / PER];
    float s[W / PER];
#pragma unroll
    for (int p = 0; p < W / PER; ++p) {  // (rows without a token read slot 0's)
      const int i = tid / TPR + PER * p;
      const int64_t si = __shfl(slot, i), at = live >> i & 1 ? si : 0;
      const size_t bh = block_head(at);
      s[p] = c.k_scale[bh];
      w[p] = *reinterpret_cast<const v2u*>(c.k_codes + (bh * bs + (at & (bs - 1))) * D + 8 * part);
    }
#pragma unroll
    for (int p = 0; p < W / PER; ++p) {
      const int i = tid / TPR + PER * p;
      if (!(live >> i & 1)) continue;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = value(((e < 4 ? w[p].x : w[p].y) >> (8 * (e & 3))) & 0xFFu, s[p]);
      *reinterpret_cast<v8bf*>(k_out + ((size_t)(row0 + i) * c.heads + h) * D + 8 * part) = to_bf16x8(x);
    }
    return;
  }
  // where row i - (i mod 16) would be if a lane's 16 rows ran on from it, against the first's
  const int here = (int)(live >> (lane & 48)) & 0xFFFF;
  const int64_t base = slot - (lane & 15), lead = __shfl(base, (lane & 48) + (here ? __builtin_ctz(here) : 0));
  const uint64_t odd = __ballot((live >> lane & 1) && (base != lead || (base & 15) != 0));
  constexpr int PARTS = W * D / (16 * 256);  // 16-row parts of the window to a thread
  const int d = tid % D;
  v4u w[PARTS];
  float s[PARTS];
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    const int i0 = __builtin_amdgcn_readfirstlane(16 * (tid / D + 256 / D * q));
    const int64_t first = __shfl(lead, i0);
    const bool run = (live >> i0 & 0xFFFF) && !(odd >> i0 & 0xFFFF);
    const int64_t at = run ? first : 0;
    const size_t bh = block_head(at);
    s[q] = c.v_scale[bh];
    w[q] = *reinterpret_cast<const v4u*>(c.v_codes + (bh * D + d) * bs + (at & (bs - 1)));
  }
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    const int i0 = __builtin_amdgcn_readfirstlane(16 * (tid / D + 256 / D * q));
    float x[16];
    if (!(odd >> i0 & 0xFFFF)) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        x[i] = value((w[q][i >> 2] >> (8 * (i & 3))) & 0xFFu, s[q]);
    } else {
      uint8_t b[16];
      float t[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int64_t si = __shfl(slot, i0 + i), at = live >> (i0 + i) & 1 ? si : 0;
        const size_t bh = block_head(at);
        b[i] = c.v_codes[(bh * D + d) * bs + (at & (bs - 1))];
        t[i] = c.v_scale[bh];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = value(b[i], t[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      const v4u u = __builtin_bit_cast(v4u, to_bf16x8(x + i));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        vt[i0 + i + 2 * e][d] = (uint16_t)u[e];
        vt[i0 + i + 2 * e + 1][d] = (uint16_t)(u[e] >> 16);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < W / PER; ++p) {
    const int i = tid / TPR + PER * p;
    if (live >> i & 1)
      *reinterpret_cast<v4u*>(v_out + ((size_t)(row0 + i) * c.heads + h) * D + 8 * part) =
          *reinterpret_cast<const v4u*>(&vt[i][8 * part]);
  }
}

hipError_t launch_kv_block_read(const int64_t* slots, int rows, const BlockCacheView& c,
                                uint16_t* k_out, uint16_t* v_out, hipStream_t stream) {
  const int grid = (rows + kReadRows - 1) / kReadRows * c.heads * 2;
  const int shift = __builtin_ctz(c.bs);
  if (c.dim == 128)
    hipLaunchKernelGGL(kv_block_read_kernel<128>, dim3((unsigned)grid), dim3(256), 0, stream,
                       slots, rows, shift, c, k_out, v_out);
  else
    hipLaunchKernelGGL(kv_block_read_kernel<64>, dim3((unsigned)grid), dim3(256), 0, stream, slots,
                       rows, shift, c, k_out, v_out);
  return hipGetLastError();
}

}  // namespace svdq
