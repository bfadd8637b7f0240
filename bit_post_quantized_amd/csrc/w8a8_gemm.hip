// Product of 8-bit integers with a scale for each row and column.
//
//   Y[m, n] = sx[m] sw[n] sum_k qx[m, k] qw[n, k] + bias[n]
//
// The sums are int32 and exact, so they may be divided over waves and workgroups in any way.  The weight is
// the first operand of the matrix instruction (rows of the result) and X the second (columns): a lane then
// holds four neighbouring columns of Y in one row.  Few rows, v_mfma_i32_16x16x64_i8:
//   operand: lane l has row l % 16, k = 16 (l / 16) .. + 15 of 64;
//   result:  lane l has column l % 16 (a row of X), rows 4 (l / 16) + e (columns of Y);
// more rows, v_mfma_i32_32x32x32_i8:
//   operand: lane l has row l % 32, k = 16 (l / 32) .. + 15 of 32;
//   result:  lane l has column l % 32, rows 8 (e / 4) + 4 (l / 32) + e % 4.
// (A loop of nothing but matrix instructions on random codes reaches 3410 TOPS with 32x32x32 and 3040 with
// 16x16x64, 4970 on zeros: what the card's power allows, not what the instruction takes.)
//
// Up to 64 rows the weight is read once, and memory bounds it: 40 x 8192 x 28672 (M, K, N) 44 us, 5.4 TB/s, 64 x
// 8192 x 28672 45, 64 x 4096 x 131072 98, 1 x 8192 x 28672 38 (partly from the last cache), 1 x 4096 x 4096 6.
// Many rows are bound by power
// where they fill the device (8192 x 8192 x 12288 660 - 760 us from card to card, 2170 - 2500 TOPS; 530 on zeros)
// and by the loads from L2 where they do not (500 x 12288 x 4096 36 - 40 us; 2000 x 8192 x 4096 65).  Rows of Y that do not
// begin at pieces of 16 bytes are stored element by element: 2000 x 4096 x 12287 133 us, x 12288 105; 8192 x 8192 x 12287
// 806, x 12288 695; 500 x 4096 x 4095 18.9, x 4096 15.6.
#include "decoder_launch.hpp"
#include "svdq_device.hpp"
#include "w8a8_plan.hpp"

namespace svdq {
namespace {

using namespace w8a8;

typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kUnit = 1024;  // 16 columns x 64 k of the container

__device__ __forceinline__ v4i mfma(v4i w, v4i x, v4i acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0);
}

// A value that is the same in every lane, in scalar registers (a buffer's base and size have to be).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <typename P>
__device__ __forceinline__ P* uniform(P* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<P*>((uint64_t)hi << 32 | lo);
}

struct Output {
  const float* sx;
  const float* sw;
  const uint16_t* bias;
  void* Y;
  int M, N;
};

// Four neighbouring columns n .. n + 3 of row m (m < M).
template <bool F32>
__device__ __forceinline__ void store4(const Output& o, int m, int n, v4i acc) {
  const float sx = o.sx[m];
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = min(n + e, o.N - 1);
    y[e] = ((float)acc[e] * sx) * o.sw[c];
    if (o.bias) y[e] += bf16_bits_to_float(o.bias[c]);
  }
  const size_t at = (size_t)m * o.N + n;
  if (n + 3 < o.N && (o.N & 3) == 0) {
    if constexpr (F32) {
      reinterpret_cast<v4f*>(o.Y)[at >> 2] = v4f{y[0], y[1], y[2], y[3]};
    } else {
      v2u w;
      w.x = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{y[0], y[1]}), v2bf));
      w.y = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{y[2], y[3]}), v2bf));
      reinterpret_cast<v2u*>(o.Y)[at >> 2] = w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < o.N) {
        if constexpr (F32) reinterpret_cast<float*>(o.Y)[at + e] = y[e];
        else reinterpret_cast<__bf16*>(o.Y)[at + e] = (__bf16)y[e];
      }
  }
}

// ---------------------------------------------------------------- container
__global__ __launch_bounds__(256) void w8a8_pack_kernel(const int8_t* codes, int N, int K,
                                                        int8_t* container, int64_t pieces) {
  const int G = K / 64;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
    const int l = (int)(i & 63);
    const int64_t unit = i >> 6;
    const int64_t t = unit / G;
    const int u = (int)(unit - t * G);
    const int64_t n = 16 * t + (l & 15);
    v4i v = {0, 0, 0, 0};
    if (n < N) v = *reinterpret_cast<const v4i*>(codes + n * K + 64 * u + 16 * (l >> 4));
    reinterpret_cast<v4i*>(container)[i] = v;
  }
}

#define SVDQ_LDS(p) ((__attribute__((address_space(3))) void*)(p))

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// 16 bytes per lane from base + offset (0 past the buffer's end) to `to` + 16 lane of LDS
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t base, uint8_t* to, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, SVDQ_LDS(to), 16, offset, 0, 0, 0);
}

// the same with 4, and with 2 bytes (a dword each), to `to` + 4 lane
__device__ __forceinline__ void load_to_lds4(__amdgpu_buffer_rsrc_t base, uint8_t* to, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, SVDQ_LDS(to), 4, offset, 0, 0, 0);
}
__device__ __forceinline__ void load_to_lds2(__amdgpu_buffer_rsrc_t base, uint8_t* to, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, SVDQ_LDS(to), 2, offset, 0, 0, 0);
}
// 16 bytes per lane, none past the buffer's end
__device__ __forceinline__ void store_16(__amdgpu_buffer_rsrc_t base, v4u v, uint32_t offset) {
  __builtin_amdgcn_raw_buffer_store_b128(v, base, offset, 0, 0);
}

// s_waitcnt vmcnt(0) lgkmcnt(0): the loads into LDS have landed, the reads from it are done
#define SVDQ_WAIT_LDS() SVDQ_WAIT_LDS_AND(0)
// the same but for the n newest loads; the loads alone
#define SVDQ_WAIT_LDS_AND(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | (7 << 4))
#define SVDQ_WAIT_LOADS(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8))

// ---------------------------------------------------------------- few rows
// A workgroup has CT tiles of 16 columns and all of K, dealt unit by unit to its waves; each wave
// keeps RT x CT accumulators and the waves' sums meet in LDS.  The weights are read once, in whole
// units; X comes from L2.
//
// An operand of X is 16 rows with 64 bytes each, and the memory unit takes four neighbouring lanes at a
// time: read straight into registers, where four neighbours are four rows, X costs four times what its
// bytes do.  So rows are read piece by piece (four lanes a row) into LDS of the wave's own, and the
// operand from there (the pieces of a row exchanged as for many rows); U units of both operands are on
// their way while U are computed.
template <int RT, int CT, int WAVES, int U, bool F32>
__global__ __launch_bounds__(64 * WAVES) void w8a8_few_kernel(const int8_t* __restrict__ qx,
                                                              const int8_t* __restrict__ container,
                                                              int K, Output o) {
  constexpr int TILES = RT * CT, CHUNK = TILES < 4 ? TILES : 4;  // tiles exchanged at a time
  constexpr int kSet = U * RT * 1024;                            // X of U units
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  v4i(*parts)[CHUNK][64] = reinterpret_cast<v4i(*)[CHUNK][64]>(lds);   // (behind the loop)
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = K / 64, tiles = (o.N + 15) / 16, t0 = blockIdx.x * CT;
  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(qx, o.M * K);          // (rows past M: zeros)
  uint8_t* mine = lds + wave * 2 * kSet;
  uint32_t x_off[RT];
  const int8_t* w[CT];
#pragma unroll
  for (int r = 0; r < RT; ++r) x_off[r] = (uint32_t)(16 * r + (lane >> 2)) * K + 16 * ((lane & 3) ^ (lane >> 4));
#pragma unroll
  for (int c = 0; c < CT; ++c)
    w[c] = container + (size_t)min(t0 + c, tiles - 1) * G * kUnit + lane * 16;
  const int x_at = (lane & 15) * 64 + 16 * ((lane >> 4) ^ ((lane >> 2) & 3));
  v4i acc[CT][RT] = {};
  const int units = (G - wave + WAVES - 1) / WAVES, steps = (units + U - 1) / U;   // (0 for a wave without any)
  auto issue = [&](int s, v4i (&wf)[U][CT]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = min(wave + (s * U + i) * WAVES, G - 1);   // (past the end: read again, not used)
#pragma unroll
      for (int r = 0; r < RT; ++r) load_to_lds(rx, mine + (s & 1) * kSet + (i * RT + r) * 1024, x_off[r] + 64 * u);
#pragma unroll
      for (int c = 0; c < CT; ++c)
        wf[i][c] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(w[c] + (size_t)u * kUnit));
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto compute = [&](int s, const v4i (&wf)[U][CT]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (s * U + i < units) {
        v4i xf[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
          xf[r] = *reinterpret_cast<const v4i*>(mine + (s & 1) * kSet + (i * RT + r) * 1024 + x_at);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[c][r] = mfma(wf[i][c], xf[r], acc[c][r]);
      }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int kAhead = U * (RT + CT);   // loads of a step
  v4i wa[U][CT], wb[U][CT];
  // (a wait for all but the newest step's loads: what is computed has landed, in LDS too)
  if (steps > 0) issue(0, wa);
  int s = 0;
  for (; s + 1 < steps; s += 2) {
    issue(s + 1, wb);
    SVDQ_WAIT_LOADS(kAhead);
    asm volatile("" ::: "memory");
    compute(s, wa);
    if (s + 2 < steps) {
      issue(s + 2, wa);
      SVDQ_WAIT_LOADS(kAhead);
    } else {
      SVDQ_WAIT_LOADS(0);
    }
    asm volatile("" ::: "memory");
    compute(s + 1, wb);
  }
  if (s < steps) {
    SVDQ_WAIT_LOADS(0);
    asm volatile("" ::: "memory");
    compute(s, wa);
  }
  __syncthreads();   // (X's place is taken by the sums)
#pragma unroll
  for (int first = 0; first < TILES; first += CHUNK) {
    if (first) __syncthreads();
#pragma unroll
    for (int i = 0; i < CHUNK; ++i)
      if (first + i < TILES) parts[wave][i][lane] = acc[(first + i) / RT][(first + i) % RT];
    __syncthreads();
    for (int i = wave; i < CHUNK; i += WAVES) {
      const int tile = first + i;
      if (tile < TILES) {
        v4i sum = parts[0][i][lane];
#pragma unroll
        for (int p = 1; p < WAVES; ++p) sum += parts[p][i][lane];
        const int m = 16 * (tile % RT) + (lane & 15), n = 16 * (t0 + tile / RT) + 4 * (lane >> 4);
        if (m < o.M && n < o.N) store4<F32>(o, m, n, sum);
      }
    }
  }
}

// ---------------------------------------------------------------- many rows
// Tiles of 64 RT x 64 WN by 2 x WN waves of 32 RT x 64, persistent workgroups that go from tile to tile.
// K in units of 64, four of them in LDS: one stream of units that runs on over the tiles, so that the next
// tile's first units are on their way while a tile is stored.  A step computes a unit in halves of k: during
// the first the operands of the second are read from LDS; then a barrier (unit u + 1 has landed, unit u is
// read: its place takes u + 4); during the second those of the next unit.  The order of matrix instructions,
// reads and loads is the written one.
//
// KS groups of 2 x WN waves take every KS-th unit each, with places of their own: a tile of few waves has one on
// a SIMD, which waits for LDS and for its products in turn.  Their sums meet in LDS before the store.
//
// With K divided (`split` shares of a tile, in a row) the shares' sums go to `partial`, [split][M][pitch].
constexpr int kPlaces = 4;      // units in LDS
constexpr int kScratch = 4096;  // LDS of a wave, for scales and stores
enum { kBf16, kFp32, kPartial };

struct Problem {
  const int8_t* qx;
  const int8_t* container;
  int M, N, K, split;
  const float* sx;
  const float* sw;
  const uint16_t* bias;
  void* Y;   // or the partial sums
};

// Item `l` of nx x ny tiles times `split` shares, in the order of xcd_tile_order: workgroup l runs on XCD
// l % 8, and each XCD has a run of items, those of the first share first and, in bands of 8 row tiles, the
// row tile fastest, so that neighbours have their weights, and then their rows, in one L2.
struct Item {
  int mt, nt, share, first, end;   // the tile, and the share's units
};
__device__ __forceinline__ Item item_at(int l, int nx, int ny, int split, int G) {
  constexpr int kBand = 8;
  const int tiles = nx * ny, items = tiles * split, i8 = items / 8 * 8;
  if (l < i8) l = (l % 8) * (items / 8) + l / 8;
  const int share = l / tiles;
  l -= share * tiles;
  const int b = l / (kBand * nx), rows = min(ny - b * kBand, kBand), within = l - b * kBand * nx;
  return {uniform(b * kBand + within % rows), uniform(within / rows), uniform(share), uniform((int)((int64_t)G * share / split)),
          uniform((int)((int64_t)G * (share + 1) / split))};
}

// What a group's loads bring next: a unit of an item (a share of a tile), every KS-th from the group's own on, and
// where it goes.  All of it is uniform.
template <int TM, int TN, int KS>
struct Stream {
  const int8_t* ax;
  const int8_t* bw;
  int item, unit, end, place, group;
  int a_left, b_left;   // bytes to the end of the operand, 0 behind the last item

  // (units are as many for every group: past the item's last, W's are zeros)
  __device__ __forceinline__ int w_bytes() const { return KS == 1 || unit < end ? b_left : 0; }

  __device__ __forceinline__ void start(const Problem& p, int items, int nx, int ny) {
    a_left = b_left = 0;
    unit = group;
    end = 1;
    if (item >= items) return;
    const int G = p.K / 64;
    const Item i = item_at(item, nx, ny, p.split, G);
    unit = i.first + group;
    end = i.end;
    ax = p.qx + (size_t)i.mt * TM * p.K + unit * 64;
    bw = p.container + ((size_t)i.nt * (TN / 16) * G + unit) * kUnit;
    a_left = min(p.M - i.mt * TM, TM) * p.K - unit * 64;
    b_left = min((p.N + 15) / 16 - i.nt * (TN / 16), TN / 16) * G * kUnit - unit * kUnit;
  }
  __device__ __forceinline__ void advance(const Problem& p, int items, int nx, int ny) {
    place = (place + 1) & (kPlaces - 1);
    ax += 64 * KS;
    bw += kUnit * KS;
    a_left = max(a_left - 64 * KS, 0);
    b_left = max(b_left - kUnit * KS, 0);
    unit += KS;
    if (unit - group >= end) {
      item += gridDim.x;
      start(p, items, nx, ny);
    }
  }
};

template <int RT, int WN, int KS, int OUT>
__global__ __launch_bounds__(128 * WN * KS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void w8a8_tile_kernel(Problem p) {
  constexpr int TM = 64 * RT, TN = 64 * WN, WAVES = 2 * WN, kA = TM * 64, kStage = kA + TN * 64;
  constexpr int kLoadsA = TM / 16 / WAVES, kLoadsB = TN / 16 / WAVES, kLoads = kLoadsA + kLoadsB;  // of a wave
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = KS == 1 ? 0 : all_waves / WAVES, wave = all_waves - group * WAVES;   // (a group's waves)
  const int wm = wave / WN, wn = wave % WN;
  uint8_t* ring = lds + group * kPlaces * kStage;
  const int G = p.K / 64;
  const int nx = (p.N + TN - 1) / TN, ny = (p.M + TM - 1) / TM, items = nx * ny * p.split;

  // ---- the stream of units.  X: rows of 64 bytes as in memory, a load has 16 of them; their four pieces of
  //      16 bytes are exchanged (slot s of row r holds piece s ^ (r / 4) % 4), so that an operand's read, the
  //      same piece of 32 rows, meets every bank equally.  W: units of the container as they are.
  uint32_t a_off[kLoadsA], b_off[kLoadsB];
#pragma unroll
  for (int j = 0; j < kLoadsA; ++j)
    a_off[j] = (uint32_t)(16 * (WAVES * j + wave) + (lane >> 2)) * p.K + 16 * ((lane & 3) ^ (lane >> 4));
#pragma unroll
  for (int j = 0; j < kLoadsB; ++j) b_off[j] = (uint32_t)(WAVES * j + wave) * G * kUnit + lane * 16;
  Stream<TM, TN, KS> next;
  next.item = blockIdx.x;
  next.group = group;
  next.place = 0;
  next.start(p, items, nx, ny);
  auto issue = [&](int j) __attribute__((always_inline)) {
    uint8_t* st = ring + next.place * kStage;
    if (j < kLoadsA) load_to_lds(buffer_rsrc(next.ax, next.a_left), st + (WAVES * j + wave) * 1024, a_off[j < kLoadsA ? j : 0]);
    else load_to_lds(buffer_rsrc(next.bw, next.w_bytes()), st + kA + (WAVES * (j - kLoadsA) + wave) * 1024,
                     b_off[j < kLoadsA ? 0 : j - kLoadsA]);
  };

  // ---- operands from LDS: lane l has row l % 32 at k = 16 (l / 32) .. + 15 of 32
  const int a0 = (wm * 32 * RT + (lane & 31)) * 64 + 16 * ((lane >> 5) ^ ((lane >> 2) & 3));
  const int b0 = kA + (wn * 4 + ((lane >> 4) & 1)) * kUnit + ((lane & 15) + 16 * (lane >> 5)) * 16;
  struct Frag {
    v4i x[RT], w[2];
  };
  auto read = [&](const uint8_t* st, int h, int r, Frag& f) __attribute__((always_inline)) {
    if (r < 2) f.w[r] = *reinterpret_cast<const v4i*>(st + b0 + 512 * h + r * 2 * kUnit);
    else if (r < RT + 2) f.x[r - 2] = *reinterpret_cast<const v4i*>(st + (a0 ^ (32 * h)) + (r - 2) * 2048);
  };
  v16i acc[RT][2] = {};
  auto product = [&](int i, int j, const Frag& f) __attribute__((always_inline)) {
    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[j], f.x[i], acc[i][j], 0, 0, 0);
  };

  // ---- a tile's scales, into the wave's scratch: sx of its rows, sw and bias of its 64 columns
  constexpr int kScaleLoads = OUT == kPartial ? 0 : 3 + (RT > 2);
  uint8_t* scratch = lds + KS * kPlaces * kStage + all_waves * kScratch;
  auto issue_scales = [&](int m0, int n0, int lane) __attribute__((always_inline)) {
    const int rows = uniform(max(min(p.M - m0, 32 * RT), 0)), columns = uniform(max(min(p.N - n0, 64), 0));
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(uniform(p.sx + min(m0, p.M)), rows * 4);
    const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(uniform(p.sw + min(n0, p.N)), columns * 4);
    load_to_lds4(rx, scratch, lane * 4);
    if constexpr (RT > 2) load_to_lds4(rx, scratch + 256, 256 + lane * 4);
    load_to_lds4(rw, scratch + 512, lane * 4);
    // (without a bias something as long is loaded, so that the loads in flight can be counted)
    if (p.bias) load_to_lds2(buffer_rsrc(uniform(p.bias + min(n0, p.N)), columns * 2), scratch + 768, lane * 2);
    else load_to_lds4(rw, scratch + 768, lane * 4);
  };

#pragma unroll
  for (int u = 0; u < kPlaces; ++u) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) issue(j);
    next.advance(p, items, nx, ny);
  }
  Frag f0, f1;
  static_assert((kPlaces - 1) * kLoads < 64, "loads that can be counted");
  SVDQ_WAIT_LOADS((kPlaces - 1) * kLoads);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int r = 0; r < RT + 2; ++r) read(ring, 0, r, f0);

  constexpr int kSize = OUT == kBf16 ? 2 : 4, kPer = 16 / kSize;   // bytes; columns of a piece of 16 bytes
  constexpr int kPasses = OUT == kBf16 ? 1 : 2;                    // of a wave's 64 columns
  constexpr int kStores = 4 * RT * kPasses;                        // of a tile, per wave
  constexpr int kBehind = (kPlaces - 2) * kLoads + kScaleLoads + kStores;
  constexpr int kPair = (kLoads + RT - 1) / RT, kReads = (RT + 2 + RT - 1) / RT;  // behind two matrix instructions
  const int64_t pitch = OUT == kPartial ? (p.N + 15) / 16 * 16 : p.N;
  const bool whole = pitch % kPer == 0;                            // Y's rows begin at pieces
  int at = 0;                                                      // the place that is computed
  int units_before = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const Item it = item_at(item, nx, ny, p.split, G);
    const int units = (it.end - it.first + KS - 1) / KS, m0 = it.mt * TM + wm * 32 * RT, n0 = it.nt * TN + wn * 64;
    // a tile's first steps follow the stores of the one before, and wait for units that were sent for
    // earlier than these
    int behind = group == 0 && whole && units_before >= kPlaces && units >= kPlaces ? 3 : 0;
    units_before = units;
    // (kept from the compiler, which would compute the addresses of the store before the loop and keep them
    // in registers that it does not have)
    int lane_ = lane;
    asm volatile("" : "+v"(lane_));
    if constexpr (OUT != kPartial)
      if (group == 0) issue_scales(m0, n0, lane_);
    for (int u = 0; u < units; ++u) {
      const uint8_t* st = ring + at * kStage;
      at = (at + 1) & (kPlaces - 1);
      const uint8_t* after = ring + at * kStage;
#pragma unroll
      for (int c = 0; c < RT; ++c) {
        product(c, c & 1, f0);
        product(c, 1 - (c & 1), f0);
#pragma unroll
        for (int r = 0; r < kReads; ++r) read(st, 1, kReads * c + r, f1);
        __builtin_amdgcn_sched_barrier(0);
      }
      // the next unit has landed for every wave, and every wave has read this one
      if (behind > 0) {
        --behind;
        SVDQ_WAIT_LDS_AND(kBehind < 63 ? kBehind : 63);
      } else {
        SVDQ_WAIT_LDS_AND((kPlaces - 2) * kLoads);
      }
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < RT; ++c) {
        product(c, c & 1, f1);
        product(c, 1 - (c & 1), f1);
#pragma unroll
        for (int r = 0; r < kReads; ++r) read(after, 0, kReads * c + r, f0);
#pragma unroll
        for (int j = 0; j < kPair; ++j)
          if (kPair * c + j < kLoads) issue(kPair * c + j);
        __builtin_amdgcn_sched_barrier(0);
      }
      next.advance(p, items, nx, ny);
      asm volatile("" ::: "memory");
    }

    if constexpr (KS > 1) {
      // ---- the groups' sums meet in the first: 32 x 32 at a time, through the second's scratch
      static_assert(KS == 2, "one group gives, one takes");
      v4i* give = reinterpret_cast<v4i*>(lds + KS * kPlaces * kStage + (WAVES + wave) * kScratch) + lane;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (group == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              give[64 * e] = v4i{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
          }
          SVDQ_WAIT_LDS_AND(63);
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          if (group == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const v4i v = give[64 * e];
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[i][j][4 * e + q] += v[q];
            }
          }
          SVDQ_WAIT_LDS_AND(63);
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
    }
    if (group == 0) {
    // ---- the tile's store.  A matrix instruction leaves four columns of one row in a lane; stored from
    //      there, a store would touch 32 rows with 16 bytes each.  A wave turns 32 rows at a time over in
    //      its scratch (4-byte results: 32 columns of them) and stores rows of 128 bytes; the pieces of a
    //      row are exchanged by the row.
    asm volatile("" : "+v"(lane_));
    float sx[RT];
    v4f sw[2][4];
    v2u bias[2][4];   // packed as they are
    if constexpr (OUT != kPartial) {
      if (units < kPlaces) SVDQ_WAIT_LOADS(0);   // (so few steps have not waited for the scales)
#pragma unroll
      for (int i = 0; i < RT; ++i) sx[i] = *reinterpret_cast<const float*>(scratch + (32 * i + (lane_ & 31)) * 4);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 32 * j + 8 * e + 4 * (lane_ >> 5);
          sw[j][e] = *reinterpret_cast<const v4f*>(scratch + 512 + c * 4);
          const v4u b = *reinterpret_cast<const v4u*>(scratch + 768 + c * 4);
          bias[j][e] = v2u{b.x | b.y << 16, b.z | b.w << 16};
        }
    }
    uint8_t* base = reinterpret_cast<uint8_t*>(p.Y) + (size_t)it.share * p.M * pitch * kSize;
    uint8_t* to = scratch + (lane_ & 31) * 128;
    const int r8 = lane_ >> 3, p8 = lane_ & 7;   // row and piece of a store's lane
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int m = m0 + 32 * i;
      const __amdgpu_buffer_rsrc_t ry =
          buffer_rsrc(uniform(base + ((size_t)min(m, p.M) * pitch + min(n0, p.N)) * kSize), 0x7FFFFFFF);
#pragma unroll
      for (int half = 0; half < kPasses; ++half) {
#pragma unroll
        for (int j = kPasses == 2 ? half : 0; j < (kPasses == 2 ? half + 1 : 2); ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const v4i sum = {acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
            if constexpr (OUT == kPartial) {
              *reinterpret_cast<v4i*>(to + 16 * ((2 * e + (lane_ >> 5)) ^ (lane_ & 7))) = sum;
            } else {
              float y[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                y[q] = ((float)sum[q] * sx[i]) * sw[j][e][q];
                const uint32_t b = bias[j][e][q >> 1];
                if (p.bias) y[q] += __uint_as_float(q & 1 ? b & 0xFFFF0000u : b << 16);
              }
              if constexpr (OUT == kFp32) {
                *reinterpret_cast<v4f*>(to + 16 * ((2 * e + (lane_ >> 5)) ^ (lane_ & 7))) = v4f{y[0], y[1], y[2], y[3]};
              } else {
                v2u w;
                w.x = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{y[0], y[1]}), v2bf));
                w.y = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{y[2], y[3]}), v2bf));
                *reinterpret_cast<v2u*>(to + 16 * ((4 * j + e) ^ (lane_ & 7)) + 8 * (lane_ >> 5)) = w;
              }
            }
          }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int r = 8 * g + r8, n = n0 + 32 * half + p8 * kPer;
          const v4u v = *reinterpret_cast<const v4u*>(scratch + r * 128 + 16 * (p8 ^ (r & 7)));
          if (whole) {   // (past the end of Y: past the buffer's)
            store_16(ry, v, m + r < p.M && n < p.N ? (uint32_t)(r * pitch + 32 * half + p8 * kPer) * kSize : ~0u);
          } else if (m + r < p.M) {
#pragma unroll
            for (int q = 0; q < kPer; ++q)
              if (n + q < p.N) {
                if constexpr (kSize == 4) reinterpret_cast<uint32_t*>(base)[(size_t)(m + r) * pitch + n + q] = v[q];
                else reinterpret_cast<uint16_t*>(base)[(size_t)(m + r) * pitch + n + q] = (uint16_t)(v[q / 2] >> (16 * (q & 1)));
              }
          }
        }
      }
    }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = v16i{};
  }
  SVDQ_WAIT_LOADS(0);   // (the loads past the end bring nothing, but write to LDS)
}

// Y from the partial sums of `split` workgroups.
template <bool F32>
__global__ __launch_bounds__(256) void w8a8_join_kernel(const int32_t* __restrict__ partial, int split, Output o) {
  const int64_t pitch = (o.N + 15) / 16 * 16, quads = pitch / 4, all = quads * o.M;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int m = (int)(i / quads), n = (int)(i - m * quads) * 4;
    if (n >= o.N) continue;
    v4i sum = {0, 0, 0, 0};
    for (int s = 0; s < split; ++s)
      sum += *reinterpret_cast<const v4i*>(partial + ((int64_t)s * o.M + m) * pitch + n);
    store4<F32>(o, m, n, sum);
  }
}

// ---------------------------------------------------------------- launches
template <int RT, int CT, int WAVES, int U>
hipError_t launch_few(const int8_t* qx, const int8_t* container, int K, const Output& o, int f32, hipStream_t st) {
  constexpr int kX = WAVES * 2 * U * RT * 1024, kParts = WAVES * (RT * CT < 4 ? RT * CT : 4) * 1024;
  constexpr int kLds = kX > kParts ? kX : kParts;
  const dim3 grid(((o.N + 15) / 16 + CT - 1) / CT), block(64 * WAVES);
  const void* fn = f32 ? reinterpret_cast<const void*>(w8a8_few_kernel<RT, CT, WAVES, U, true>)
                       : reinterpret_cast<const void*>(w8a8_few_kernel<RT, CT, WAVES, U, false>);
  if (kLds > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  if (f32) hipLaunchKernelGGL((w8a8_few_kernel<RT, CT, WAVES, U, true>), grid, block, kLds, st, qx, container, K, o);
  else hipLaunchKernelGGL((w8a8_few_kernel<RT, CT, WAVES, U, false>), grid, block, kLds, st, qx, container, K, o);
  return hipGetLastError();
}

template <int RT>
hipError_t launch_few_rows(const int8_t* qx, const int8_t* container, int K, const Output& o, int f32, hipStream_t st) {
  const int columns = few_columns(RT, (o.N + 15) / 16, K);
  if constexpr (RT == 1)
    if (columns == 2) return launch_few<1, 2, 8, 2>(qx, container, K, o, f32, st);
  if (columns == 4) return launch_few<RT, 4, 8, 2>(qx, container, K, o, f32, st);
  if constexpr (RT > 1)
    if (columns == 2) return launch_few<RT, 2, 8, 2>(qx, container, K, o, f32, st);
  return launch_few<RT, 1, 8, RT <= 2 ? 4 : 2>(qx, container, K, o, f32, st);
}

template <int RT, int WN, int KS, int OUT>
hipError_t launch_tile(const Problem& p, hipStream_t st) {
  constexpr int kLds = KS * (kPlaces * (RT + WN) * 4096 + 2 * WN * kScratch);
  constexpr int kPerCu = 160 * 1024 / kLds;
  // more than the default 64 KB of LDS
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(w8a8_tile_kernel<RT, WN, KS, OUT>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  const int64_t items = (int64_t)((p.N + 64 * WN - 1) / (64 * WN)) * ((p.M + 64 * RT - 1) / (64 * RT)) * p.split;
  const int grid = items < kCus * kPerCu ? (int)items : kCus * kPerCu;
  hipLaunchKernelGGL((w8a8_tile_kernel<RT, WN, KS, OUT>), dim3(grid), dim3(128 * WN * KS), kLds, st, p);
  return hipGetLastError();
}

template <int RT, int WN, int KS>
hipError_t launch_many(const Problem& problem, int out_fp32, const Output& o, int32_t* ws, hipStream_t st) {
  Problem p = problem;
  if (p.split == 1) return out_fp32 ? launch_tile<RT, WN, KS, kFp32>(p, st) : launch_tile<RT, WN, KS, kBf16>(p, st);
  p.Y = ws;
  const hipError_t e = launch_tile<RT, WN, KS, kPartial>(p, st);
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)((o.N + 15) / 16) * 4 * o.M, blocks = (quads + 255) / 256;
  const dim3 grid((int)(blocks < 4096 ? blocks : 4096));
  if (out_fp32) hipLaunchKernelGGL((w8a8_join_kernel<true>), grid, dim3(256), 0, st, ws, p.split, o);
  else hipLaunchKernelGGL((w8a8_join_kernel<false>), grid, dim3(256), 0, st, ws, p.split, o);
  return hipGetLastError();
}

}  // namespace

size_t w8a8_container_bytes(int N, int K) { return (size_t)((N + 15) / 16) * (K / 64) * kUnit; }

hipError_t launch_w8a8_pack(const int8_t* codes, int N, int K, int8_t* container, hipStream_t stream) {
  const int64_t pieces = (int64_t)(w8a8_container_bytes(N, K) / 16), blocks = (pieces + 255) / 256;
  hipLaunchKernelGGL(w8a8_pack_kernel, dim3((int)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256), 0, stream,
                     codes, N, K, container, pieces);
  return hipGetLastError();
}

size_t w8a8_workspace_bytes(int M, int N, int K) {
  const Plan p = plan(M, N, K);
  return p.split > 1 ? (size_t)p.split * M * ((N + 15) / 16 * 16) * 4 : 0;
}

hipError_t launch_w8a8_gemm(const int8_t* qx, const float* sx, const int8_t* container, const float* sw,
                            const uint16_t* bias, int M, int N, int K, void* Y, int out_fp32, void* workspace,
                            hipStream_t stream) {
  const Output o{sx, sw, bias, Y, M, N};
  const Plan p = plan(M, N, K);
  if (p.rt == 0) {
    switch ((M + 15) / 16) {
      case 1: return launch_few_rows<1>(qx, container, K, o, out_fp32, stream);
      case 2: return launch_few_rows<2>(qx, container, K, o, out_fp32, stream);
      case 3: return launch_few_rows<3>(qx, container, K, o, out_fp32, stream);
      default: return launch_few_rows<4>(qx, container, K, o, out_fp32, stream);
    }
  }
  const Problem q{qx, container, M, N, K, p.split, sx, sw, bias, Y};
  int32_t* ws = static_cast<int32_t*>(workspace);
  if (p.rt == 4) return launch_many<4, 4, 1>(q, out_fp32, o, ws, stream);
  if (p.rt == 1) return launch_many<1, 2, 2>(q, out_fp32, o, ws, stream);
  return p.wn == 4 ? launch_many<2, 4, 1>(q, out_fp32, o, ws, stream) : launch_many<2, 2, 1>(q, out_fp32, o, ws, stream);
}

}  // namespace svdq
