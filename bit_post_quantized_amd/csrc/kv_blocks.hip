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
// latency: two block scans per 1024 requests.
constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 1024;

__device__ __forceinline__ int clamp0(int x) { return x < 0 ? 0 : x; }

// Inclusive sums of one value per thread over the workgroup, in 64 bits; total in `sum`.
__device__ __forceinline__ long long block_scan(long long v, long long* lds, long long& sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const long long u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // (the previous scan's readers are done with lds)
  if (lane == 63) lds[wave] = v;
  __syncthreads();
  long long before = 0;
  sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    const long long x = lds[w];
    if (w < wave) before += x;
    sum += x;
  }
  return v + before;
}

__global__ __launch_bounds__(kPlanThreads) void kv_block_plan_kernel(
    const int32_t* __restrict__ ctx, const int32_t* __restrict__ add, int requests,
    int32_t* __restrict__ tables, int width, int shift, const int32_t* __restrict__ free_blocks,
    int capacity, const int32_t* __restrict__ free_count, int32_t* __restrict__ cu,
    int32_t* __restrict__ seq, int rows, int32_t* __restrict__ positions,
    int64_t* __restrict__ slots, int32_t* __restrict__ status, int32_t* __restrict__ free_out) {
  __shared__ long long scan_lds[kPlanThreads / 64];
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
    const long long cu1 = cu_base + block_scan(n, scan_lds, sum), first = cu1 - n;
    cu_base += sum;
    const long long end = ((long long)c + n + bs - 1) >> shift;
    const int held = (int)(((long long)c + bs - 1) >> shift);
    int st = end > width ? 2 : cu1 > rows ? 3 : 0;
    const long long need = st ? 0 : end - held;
    const long long incl = need_base + block_scan(need, scan_lds, sum);
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
    const long long at = block_scan(mine ? 1 : 0, scan_lds, sum) - 1;
    if (mine) {
      const int i = found + (int)at;  // < kPlanRows: each has a row of its own in the range
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
    __syncthreads();
    if ((tid & 63) == 0) scan_lds[tid >> 6] = taken;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kPlanThreads / 64; ++w) taken = scan_lds[w] > taken ? scan_lds[w] : taken;
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
  __shared__ long long scan_lds[kPlanThreads / 64];
  const int me = blockIdx.x, tid = threadIdx.x, bs = 1 << shift;
  const int have = min(clamp0(free_count[0]), capacity);
  const bool last = me == requests, mine = !last && done[me];
  if (!last && tid == 0) seq_out[me] = mine ? 0 : seq[me];
  if (!last && !mine) return;
  long long before = 0;
  for (int b0 = 0; b0 < me; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long v = 0, sum;
    if (b < me && done[b]) {
      v = ((long long)clamp0(seq[b]) + bs - 1) >> shift;
      if (v > width) v = width;
    }
    block_scan(v, scan_lds, sum);
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
// per (tile of kAppendTile rows, head, K or V) handles the runs that begin in its tile, one after
// the other: amax over the run, the scale, the old codes where it grew, the new codes.
constexpr int kAppendThreads = 256;
constexpr int kAppendTile = 4;

// One value -> code + 128, for s != 0 and rcp = fl32(1 / s).  The correction-step quotient needs a
// normal reciprocal; below 2^-100 the division itself is used.
__device__ __forceinline__ uint32_t kv_code(float x, float s, float rcp) {
  const float t = s >= 0x1p-100f ? rne_quotient(x, s, rcp) : __builtin_rintf(x / s);
  return (uint32_t)(int)(__builtin_amdgcn_fmed3f(t, -127.0f, 127.0f) + 128.0f);
}

template <int D>
__global__ __launch_bounds__(kAppendThreads) void kv_block_append_kernel(
    const uint16_t* __restrict__ kx, const uint16_t* __restrict__ vx, int64_t k_stride,
    int64_t v_stride, const int64_t* __restrict__ slots, int rows, int shift, BlockCacheView c) {
  constexpr int TPR = D / 8;                     // threads per token row, 8 channels each
  constexpr int PER = kAppendThreads / TPR;      // tokens per pass
  __shared__ float wmax[kAppendThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.y, is_v = blockIdx.z, bs = 1 << shift;
  const uint16_t* x = is_v ? vx : kx;
  const int64_t stride = is_v ? v_stride : k_stride;
  const int64_t limit = (int64_t)c.num_blocks << shift;
  const int row0 = blockIdx.x * kAppendTile;
  for (int t = row0; t < min(row0 + kAppendTile, rows); ++t) {
    const int64_t slot = slots[t];
    if (slot < 0 || slot >= limit) continue;
    const int off = (int)(slot & (bs - 1));
    if (off != 0 && t > 0 && slots[t - 1] == slot - 1) continue;  // inside a run
    int n = 1;
    while (off + n < bs && t + n < rows && slots[t + n] == slot + n) ++n;
    const size_t bh = (size_t)(slot >> shift) * c.heads + h;
    uint8_t* codes = (is_v ? c.v_codes : c.k_codes) + bh * bs * D;
    float* scale = (is_v ? c.v_scale : c.k_scale) + bh;
    const int part = tid % TPR, first = tid / TPR;
    float amax = 0.0f;
    for (int i = first; i < n; i += PER) {
      const v4u w = *reinterpret_cast<const v4u*>(x + (size_t)(t + i) * stride + (size_t)h * D + 8 * part);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        amax = __builtin_fmaxf(amax, __builtin_fabsf(__uint_as_float(ws[e] << 16)));
        amax = __builtin_fmaxf(amax, __builtin_fabsf(__uint_as_float(ws[e] & 0xFFFF0000u)));
      }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o));
    __syncthreads();
    if (lane == 0) wmax[wave] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 64; ++w) amax = __builtin_fmaxf(amax, wmax[w]);
    const float old = off == 0 ? 0.0f : *scale;
    const float s = __builtin_fmaxf(old, amax / 127.0f);
    __syncthreads();  // (every thread has read the old scale)
    if (tid == 0) *scale = s;
    if (off > 0 && s > old) {
      const float ratio = old / s;
      for (int i = tid; i < off * D; i += kAppendThreads) {
        const int at = is_v ? (i / off) * bs + i % off : i;
        codes[at] = (uint8_t)(int)(__builtin_rintf(((float)codes[at] - 128.0f) * ratio) + 128.0f);
      }
    }
    const float s1 = s == 0.0f ? 1.0f : s, rcp = 1.0f / s1;
    for (int i = first; i < n; i += PER) {
      const v4u w = *reinterpret_cast<const v4u*>(x + (size_t)(t + i) * stride + (size_t)h * D + 8 * part);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = __uint_as_float(e & 1 ? ws[e >> 1] & 0xFFFF0000u : ws[e >> 1] << 16);
        const uint32_t q = s == 0.0f ? 128u : kv_code(f, s1, rcp);
        const int d = 8 * part + e;
        codes[is_v ? d * bs + off + i : (off + i) * D + d] = (uint8_t)q;
      }
    }
  }
}

hipError_t launch_kv_block_append(const uint16_t* k, const uint16_t* v, int64_t k_stride,
                                  int64_t v_stride, const int64_t* slots, int rows,
                                  const BlockCacheView& c, hipStream_t stream) {
  const dim3 grid((rows + kAppendTile - 1) / kAppendTile, c.heads, 2);
  const int shift = __builtin_ctz(c.bs);
  if (c.dim == 128)
    hipLaunchKernelGGL(kv_block_append_kernel<128>, grid, dim3(kAppendThreads), 0, stream, k, v,
                       k_stride, v_stride, slots, rows, shift, c);
  else
    hipLaunchKernelGGL(kv_block_append_kernel<64>, grid, dim3(kAppendThreads), 0, stream, k, v,
                       k_stride, v_stride, slots, rows, shift, c);
  return hipGetLastError();
}

// -------------------------------------------------------------------------------------- read
// One thread per (row, head, 8 channels).
template <int D>
__global__ __launch_bounds__(256) void kv_block_read_kernel(const int64_t* __restrict__ slots,
                                                            int rows, int shift, BlockCacheView c,
                                                            uint16_t* __restrict__ k_out,
                                                            uint16_t* __restrict__ v_out) {
  constexpr int TPR = D / 8;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int part = (int)(i % TPR);
  const long long rh = i / TPR;
  const int h = (int)(rh % c.heads), bs = 1 << shift;
  const long long t = rh / c.heads;
  if (t >= rows) return;
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= ((int64_t)c.num_blocks << shift)) return;
  const int off = (int)(slot & (bs - 1));
  const size_t bh = (size_t)(slot >> shift) * c.heads + h;
  const size_t out = ((size_t)t * c.heads + h) * D + 8 * part;
  const float ks = c.k_scale[bh], vs = c.v_scale[bh];
  const v2u kw = *reinterpret_cast<const v2u*>(c.k_codes + (bh * bs + off) * D + 8 * part);
  const uint8_t* vp = c.v_codes + (bh * D + 8 * part) * bs + off;
  float kf[8], vf[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    kf[e] = ((float)(((e < 4 ? kw.x : kw.y) >> (8 * (e & 3))) & 0xFFu) - 128.0f) * ks;
    vf[e] = ((float)vp[(size_t)e * bs] - 128.0f) * vs;
  }
  *reinterpret_cast<v4u*>(k_out + out) = v4u{pack2_bf16(kf[0], kf[1]), pack2_bf16(kf[2], kf[3]),
                                             pack2_bf16(kf[4], kf[5]), pack2_bf16(kf[6], kf[7])};
  *reinterpret_cast<v4u*>(v_out + out) = v4u{pack2_bf16(vf[0], vf[1]), pack2_bf16(vf[2], vf[3]),
                                             pack2_bf16(vf[4], vf[5]), pack2_bf16(vf[6], vf[7])};
}

hipError_t launch_kv_block_read(const int64_t* slots, int rows, const BlockCacheView& c,
                                uint16_t* k_out, uint16_t* v_out, hipStream_t stream) {
  const long long threads = (long long)rows * c.heads * (c.dim / 8);
  const long long grid = (threads + 255) / 256;
  if (grid > 0x7FFFFFFFLL) return hipErrorInvalidConfiguration;
  const int shift = __builtin_ctz(c.bs);
  if (c.dim == 128)
    hipLaunchKernelGGL(kv_block_read_kernel<128>, dim3((unsigned)grid), dim3(256), 0, stream,
                       slots, rows, shift, c, k_out, v_out);
  else
    hipLaunchKernelGGL(kv_block_read_kernel<64>, dim3((unsigned)grid), dim3(256), 0, stream,
                       slots, rows, shift, c, k_out, v_out);
  return hipGetLastError();
}

}  // namespace svdq
