// The linear layer on few rows: INT4 weights, 16-bit activations, fp32 sums.
//
//     Y[m, n] = sum_g s_w[g, n] sum_{k in g} X^[m, k] q[n, k] + sum_j T[m, j] L2[j, n] + bias[n],
//     X^ = fl32(X inv_lambda),  T = X^ L1
//
// With few rows the weights are read once and used M times, so the floor is their N K / 2 bytes.
// The products run on v_mfma_f32_16x16x32_f16: a code is an exact fp16, and an activation enters
// as an fp16 after a power-of-two scale per (row, 8 groups) (11 significant bits, for bf16 output)
// or as the fp16 pair hi + lo (22 bits, for fp32 output); products of 11 x 4 bits are exact and
// the sums are the matrix unit's fp32.
//  1. w4a16_prep_kernel: X^ in the matrix operand's order, its scales, and T's partial sums over
//     slices of K (bf16 MFMA on X^ split into three bf16, which keeps all 24 bits).
//  2. w4a16_kernel: persistent workgroups of 8 waves that split K, or a part of it; a wave keeps
//     its part of X^ in registers and walks over tiles of 16 columns, with the next tiles' weights
//     in flight while it computes the current one's.  A lane turns 16 nibbles of one column into fp16 per group,
//     one fp32 FMA per output and group applies the weight scale, the low-rank product is one more
//     matrix step per 32 ranks, and the waves meet in LDS once per tile.
// The weights come in a container of the matrix operand's order (svdq_pack_w4a16): in [N, K/2] a
// wave's load takes 32 bytes of each of 16 rows, and the scales one 2-byte load per group.
//  3. w4a16_sum_kernel, where K was cut over workgroups: the sum of their shares.
//
// Measured (kernel times): 1 row, 4096 x 131072: 45 us, 6.3 TB/s of weights, the memory's rate.
// 1 row, 4096 x 4096, rank 32: 4.9 + 6.7 us, of which the weights' bytes are 1.7: two launches and
// the latency of each one's first loads.  8 rows, 4096 x 12288: 4.9 + 10.7 us (bytes 4.9).  24 fp32
// rows, 12288 x 4096, rank 48: 7.0 + 18.4 + 3.9 us, without the branch 4.7 + 14.9 + 4.0: the workgroups
// of the first share of K add up all of T and do the branch, the others do none of it; of the rest
// about 5 us are the instructions' issue and 5 the weights' bytes, at two waves to a SIMD that wait for
// them on 6 or 7 tiles.  64 rows, 4096 x 12288, rank 32: 5.5 + 19.5 + 4.5 us, without 4.2 + 17.3 + 4.0.
#include "serve_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kFragBytes = 2048;     // of X^: one (row tile, group), 16 rows x 64 k of fp16
constexpr int kMaxSlices = 32;       // of K, in the preparing kernel
constexpr int kWaves = 8;            // of the main kernel
constexpr int kSeg = 8;              // groups that share an activation scale; of one container unit

// Container unit (column tile t, segment s), at (t segments + s) kUnit bytes: for each of 4 pairs
// of groups 64 lanes x 16 bytes (lane l: column 16 t + l % 16, k = 16 (l / 16) .. + 15 of either
// group, 8 bytes of nibbles each), then fp16 scales [16 columns][8 groups].  Columns past N and
// groups past K / 64 hold code 0 and scale 0.
constexpr int kUnitCodes = 4096, kUnit = kUnitCodes + 256;

__host__ __device__ inline int w4a16_segments(int K) { return (K / kGroup + kSeg - 1) / kSeg; }

size_t w4a16_container_bytes(int N, int K) {
  return (size_t)((N + 15) / 16) * w4a16_segments(K) * kUnit;
}

// One thread per lane of a unit.
__global__ __launch_bounds__(256) void w4a16_pack_kernel(const uint8_t* __restrict__ wq,
                                                         const uint16_t* __restrict__ w_scales,
                                                         int N, int K, long long units,
                                                         uint8_t* __restrict__ out) {
  const long long unit = (long long)blockIdx.x * 4 + threadIdx.x / 64;
  if (unit >= units) return;
  const int G = K / kGroup, segs = w4a16_segments(K);
  const int lane = threadIdx.x & 63, j = lane >> 4, seg = (int)(unit % segs);
  const long long n = unit / segs * 16 + (lane & 15);
  uint8_t* u = out + (size_t)unit * kUnit;
  uint16_t s[kSeg];
#pragma unroll
  for (int p = 0; p < kSeg / 2; ++p) {
    v2u w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int g = seg * kSeg + 2 * p + e;
      const bool live = n < N && g < G;
      w[e] = live ? *reinterpret_cast<const v2u*>(wq + (size_t)n * (K / 2) + (size_t)g * 32 + 8 * j) : v2u{0u, 0u};
      s[2 * p + e] = live ? w_scales[(size_t)g * N + n] : (uint16_t)0;
    }
    reinterpret_cast<v4u*>(u)[p * 64 + lane] = v4u{w[0].x, w[0].y, w[1].x, w[1].y};
  }
  if (j == 0)
    reinterpret_cast<v4u*>(u + kUnitCodes)[lane] =
        v4u{s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16, s[4] | (uint32_t)s[5] << 16,
            s[6] | (uint32_t)s[7] << 16};
}

hipError_t launch_w4a16_pack(const uint8_t* wq, const uint16_t* w_scales, int N, int K,
                             uint8_t* container, hipStream_t stream) {
  const long long units = (long long)((N + 15) / 16) * w4a16_segments(K);
  hipLaunchKernelGGL(w4a16_pack_kernel, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, stream,
                     wq, w_scales, N, K, units, container);
  return hipGetLastError();
}

// Row tiles: 16 rows each, or for fp32 output 8 rows, hi parts in matrix rows 0..7 and lo parts
// in rows 8..15.
__host__ __device__ inline int w4a16_rows_per_tile(int out_fp32) { return out_fp32 ? 8 : 16; }

inline int w4a16_tiles(int M, int out_fp32) {
  const int rpt = w4a16_rows_per_tile(out_fp32);
  return (M + rpt - 1) / rpt;
}

// Slices of K for T's partial sums: one segment (a group per wave) to a preparing workgroup, as far
// as summing the partials again in every workgroup of the main kernel stays cheap.
inline int w4a16_slices(int K) {
  const int s = w4a16_segments(K);
  return s < kMaxSlices ? s : kMaxSlices;
}

// Up to 4 row tiles share a pass over the weights (64 bf16 rows, 32 fp32 rows).  What a wave holds
// of X^ is 8 registers per row tile and group, so more row tiles mean fewer groups to a chunk.
constexpr int kMaxTiles = 4;
constexpr int groups_per_wave(int tiles) { return tiles <= 2 ? 8 : 4; }

// (Three row tiles with 2 groups and two workgroups to a CU: 32.6 us against 28.2 for 24 fp32 rows,
// 12288 x 4096, rank 48.)

// How a pass is cut.  One persistent workgroup per CU.  Where K is more than a workgroup's waves
// hold of X^, it is cut into chunks.  With one row tile a workgroup walks over them all and reads X^
// again (12288 x 4096, rank 32: 1 row 16.1 us, cut 18.3; 16 rows 18.7, cut 20.3); with more, where
// that is most of what it reads, the workgroups of a column tile take one chunk each and their sums
// go through memory, shares (64 rows 29 us, read again 39).
struct W4a16Pass {
  int rows, shares, grid;
  bool loop;
};

inline W4a16Pass w4a16_pass(int M, int N, int K, int tile0, int tiles, int out_fp32) {
  const int rpt = w4a16_rows_per_tile(out_fp32);
  const int mt = tiles - tile0 < kMaxTiles ? tiles - tile0 : kMaxTiles;
  const int per = kWaves * groups_per_wave(mt), chunks = (K / kGroup + per - 1) / per;
  W4a16Pass p;
  p.rows = M - tile0 * rpt < mt * rpt ? M - tile0 * rpt : mt * rpt;
  p.loop = chunks > 1 && mt == 1;
  p.shares = p.loop ? 1 : chunks;
  // a multiple of 8, for the XCDs
  const int run = ((N + 15) / 16 + 7) / 8, most = 32 / p.shares < 1 ? 1 : 32 / p.shares;
  p.grid = 8 * p.shares * (run < most ? run : most);
  return p;
}

struct W4a16Ws {
  size_t frags, scales, parts, partial, bytes;  // byte offsets and the total
};

inline W4a16Ws w4a16_layout(int M, int N, int K, int r, int out_fp32) {
  const size_t tiles = w4a16_tiles(M, out_fp32), G = K / kGroup;
  W4a16Ws w;
  w.frags = 0;
  w.scales = tiles * G * kFragBytes;
  w.parts = w.scales + tiles * w4a16_segments(K) * 16 * sizeof(float);
  w.partial = w.parts + (size_t)w4a16_slices(K) * M * r * sizeof(float);
  w.partial = (w.partial + 15) / 16 * 16;
  size_t most = 0;
  for (int t = 0; t < (int)tiles; t += kMaxTiles) {
    const W4a16Pass p = w4a16_pass(M, N, K, t, (int)tiles, out_fp32);
    const size_t need = p.shares == 1 ? 0 : (size_t)p.shares * p.rows * ((N + 15) / 16 * 16) * sizeof(float);
    most = need > most ? need : most;
  }
  w.bytes = w.partial + most;
  return w;
}

size_t w4a16_workspace_bytes(int M, int N, int K, int r, int out_fp32) {
  return w4a16_layout(M, N, K, r, out_fp32).bytes;
}

// Eight packed nibbles -> eight exact fp16 codes, in the order k0 k4 k1 k5 k2 k6 k3 k7.  A nibble
// with its bit 3 flipped is c + 8; in the mantissa of 1024 it makes 1024 + (c + 8), or from bits
// 4..7 1024 + 16 (c + 8), and one packed fp16 operation takes the offset (and the 16) away,
// exactly.  Mask, flip and exponent are one three-operand bit operation, (w & mask) ^ constant.
__device__ __forceinline__ v8h unpack8_f16(uint32_t w) {
  constexpr int kAndXor = 0x6A;  // (a & b) ^ c
  const uint32_t v = w >> 8;
  const v2h six = {(_Float16)0.0625f, (_Float16)0.0625f};
  const v2h off0 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
  const v2h off4 = {(_Float16)-72.0f, (_Float16)-72.0f};
  const v2h a = __builtin_bit_cast(v2h, __builtin_amdgcn_bitop3_b32(w, 0x000F000Fu, 0x64086408u, kAndXor)) + off0;
  const v2h b = __builtin_elementwise_fma(
      __builtin_bit_cast(v2h, __builtin_amdgcn_bitop3_b32(w, 0x00F000F0u, 0x64806480u, kAndXor)), six, off4);
  const v2h c = __builtin_bit_cast(v2h, __builtin_amdgcn_bitop3_b32(v, 0x000F000Fu, 0x64086408u, kAndXor)) + off0;
  const v2h d = __builtin_elementwise_fma(
      __builtin_bit_cast(v2h, __builtin_amdgcn_bitop3_b32(v, 0x00F000F0u, 0x64806480u, kAndXor)), six, off4);
  return v8h{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ v4f mfma_f16(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma_bf16(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Eight fp32 -> TERMS bf16 operands that add up to them (8 bits each).
template <int TERMS>
__device__ __forceinline__ void split_bf16(const float* x, v8bf* out) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i];
#pragma unroll
  for (int c = 0; c < TERMS; ++c) {
    out[c] = to_bf16x8(y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] -= (float)out[c][i];
  }
}

// One workgroup per (slice of K, row tile); a segment of 8 groups at a time, a group to a wave; the
// waves share their rows' largest magnitudes in LDS.  Lane (row l % 16, j = l / 16) holds
// k = 64 g + 16 j .. + 15.  RT >= r / 16 rank tiles.
template <int RT>
__global__ __launch_bounds__(kSeg * 64) void w4a16_prep_kernel(
    const uint16_t* __restrict__ X, const float* __restrict__ inv_lambda,
    const uint16_t* __restrict__ L1p, int M, int K, int r, int out_fp32, v8h* __restrict__ frags,
    float* __restrict__ scales, float* __restrict__ parts) {
  __shared__ float red[RT ? RT : 1][kSeg][16][17];
  __shared__ float top[2][kSeg][16];
  const int G = K / kGroup, segs = w4a16_segments(K);
  const int slices = gridDim.x, slice = blockIdx.x, tile = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int mr = lane & 15, j = lane >> 4;
  const int rpt = w4a16_rows_per_tile(out_fp32);
  const int row = tile * rpt + (mr & (rpt - 1));
  const bool live = row < M, low = out_fp32 && mr >= 8;
  const int s0 = (int)((long long)segs * slice / slices), s1 = (int)((long long)segs * (slice + 1) / slices);

  v4f t[RT ? RT : 1];
#pragma unroll
  for (int i = 0; i < RT; ++i) t[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  int par = 0;
  for (int seg = s0; seg < s1; ++seg, par ^= 1) {
    const bool mine = seg * kSeg + wave < G;  // (the others read the last group and store nothing)
    const int g = min(seg * kSeg + wave, G - 1), k0 = g * kGroup + 16 * j;
    v8bf b[RT ? RT : 1][2];
    // the rank rows' loads first: they do not wait for X (rows past r - 1 read row r - 1, unused)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        b[i][s] = *reinterpret_cast<const v8bf*>(L1p + (size_t)min(16 * i + mr, r - 1) * K + k0 + 8 * s);
    const v4u* xp = reinterpret_cast<const v4u*>(X + (size_t)min(row, M - 1) * K + k0);
    const v4u w0 = xp[0], w1 = xp[1];
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    const v4f* lp = reinterpret_cast<const v4f*>(inv_lambda + k0);
    float x[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4f l = lp[i];
      x[4 * i] = __uint_as_float(w[2 * i] << 16) * l.x;
      x[4 * i + 1] = __uint_as_float(w[2 * i] & 0xFFFF0000u) * l.y;
      x[4 * i + 2] = __uint_as_float(w[2 * i + 1] << 16) * l.z;
      x[4 * i + 3] = __uint_as_float(w[2 * i + 1] & 0xFFFF0000u) * l.w;
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (!live || !mine) x[i] = 0.0f;
      amax = __builtin_fmaxf(amax, __builtin_fabsf(x[i]));
    }
    amax = __builtin_fmaxf(amax, __shfl_xor(amax, 16));
    amax = __builtin_fmaxf(amax, __shfl_xor(amax, 32));
    if (j == 0) top[par][wave][mr] = amax;
    __syncthreads();  // (the next round's buffer is the other one)
#pragma unroll
    for (int q = 0; q < kSeg; ++q) amax = __builtin_fmaxf(amax, top[par][q][mr]);
    // 2^e with amax 2^-e in [2^10, 2^11) (e clamped so that both powers are normal; 0 keeps e = 0)
    int e = (int)(__float_as_uint(amax) >> 23) - 127 - 10;
    e = amax == 0.0f ? 0 : max(e, -126);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    _Float16 h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = x[i] * down;
      const _Float16 hi = (_Float16)y;
      h[i] = low ? (_Float16)(y - (float)hi) : hi;
    }
    if (mine) {
      const size_t base = ((size_t)tile * G + g) * 128;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        v8h f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = h[8 * s + (i >> 1) + ((i & 1) << 2)];
        frags[base + s * 64 + lane] = f;
      }
      if (j == 0 && wave == 0) scales[((size_t)tile * segs + seg) * 16 + mr] = up;
    }

    if constexpr (RT > 0) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        v8bf p[3];
        split_bf16<3>(x + 8 * s, p);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int c = 0; c < 3; ++c) t[i] = mfma_bf16(p[c], b[i][s], t[i]);
      }
    }
  }

  // T's partial of this slice: the waves' sums meet in LDS
  if constexpr (RT > 0) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) red[i][wave][4 * j + q][mr] = t[i][q];
    __syncthreads();
    for (int o = threadIdx.x; o < RT * 256; o += kSeg * 64) {
      const int i = o >> 8, m = (o >> 4) & 15, c = o & 15, out = tile * rpt + m;
      if (m < rpt && out < M && 16 * i + c < r) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kSeg; ++w) s += red[i][w][m][c];
        parts[((size_t)slice * M + out) * r + 16 * i + c] = s;
      }
    }
  }
}

// What one wave holds of a (column tile, chunk of K): GPW groups of codes and their scales (fp16
// pairs), and the ranks it adds; and of X^, MT row tiles of the same groups.
template <int GPW>
struct Weights {
  v4u w[GPW / 2];
  uint32_t s[GPW / 2];
  v8bf l2;
};

template <int MT, int GPW>
struct Rows {
  v8h a[MT][GPW][2];
  v4f up[MT];  // the scales of its rows 4 j + i: a wave's groups lie in one segment
};

// MT row tiles; a chunk of K is kWaves * GPW groups, GPW to a wave.  HOLD: K is one chunk, and the
// wave's X^ stays in registers for all its column tiles; otherwise it is read again per chunk, a
// chunk ahead.  STAGES - 1 steps of weights are in flight.  RANK: there is a low-rank branch.
template <int MT, int GPW, bool HOLD, bool FP32, bool RANK>
__global__ __launch_bounds__(kWaves * 64, 1) void w4a16_kernel(
    const v8h* __restrict__ frags, const float* __restrict__ scales,
    const float* __restrict__ parts, int slices, const uint8_t* __restrict__ container,
    const uint16_t* __restrict__ L2p, const uint16_t* __restrict__ bias, int M, int N, int K,
    int r, int tile0, int tiles, int shares, float* __restrict__ partial, void* __restrict__ Y) {
  constexpr int RPT = FP32 ? 8 : 16;
  constexpr int TERMS = FP32 ? 3 : 2;  // bf16 terms of T: 24 or 16 bits
  __shared__ __attribute__((aligned(16))) float red[2][kWaves][MT * 16][17];
  __shared__ v8bf t_lds[RANK ? MT : 1][4][TERMS][64];
  static_assert(kSeg % GPW == 0 && GPW % 2 == 0, "a wave's groups are pairs of one segment");
  const int G = K / kGroup, segs = w4a16_segments(K);
  const int chunks = (G + kWaves * GPW - 1) / (kWaves * GPW);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, j = lane >> 4;
  const int row0 = tile0 * RPT, rows = min(M - row0, MT * RPT);
  const int steps = RANK ? (r + 31) / 32 : 0;  // matrix steps of the low-rank product, one to a wave

  // Column tiles of this workgroup; each XCD (workgroups go to the 8 round-robin) takes a
  // contiguous run of them.  HOLD: a workgroup has one chunk, and 'shares' of them share a tile.
  const int all = (N + 15) / 16, run = (all + 7) / 8, per = gridDim.x / 8 / shares;
  const int first = (blockIdx.x & 7) * run, end = min(first + run, all);
  const int share = HOLD ? (int)(blockIdx.x >> 3) % shares : 0;
  int tile = first + (int)(blockIdx.x >> 3) / shares, chunk = share;
  if (tile >= end) return;

  auto load_x = [&](int ch, Rows<MT, GPW>& x) {
    const int g0 = (ch * kWaves + wave) * GPW;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      // (a row tile past the last and a group past the last read the last one's; neither counts)
      const int tt = min(tile0 + t, tiles - 1);
      // rows past the last are not stored, so they may be the last one's: fewer bytes to read
      const int most = min(RPT, M - tt * RPT) - 1;
      const int at = 16 * j + (FP32 ? (c & 8) + min(c & 7, most) : min(c, most));
#pragma unroll
      for (int u = 0; u < GPW; ++u) {
        const v8h* f = frags + ((size_t)tt * G + min(g0 + u, G - 1)) * 128;
        x.a[t][u][0] = f[at];
        x.a[t][u][1] = f[64 + at];
      }
      x.up[t] = reinterpret_cast<const v4f*>(scales + ((size_t)tt * segs + min(g0 / kSeg, segs - 1)) * 16)[j];
    }
  };
  // Loads without branches, so that the next step's are all in flight while this one's are waited
  // for; a step that is not there (spread = 0) reads one address.
  auto load_w = [&](int t, int ch, int spread, Weights<GPW>& w) {
    const int g0 = (ch * kWaves + wave) * GPW, seg = min(g0 / kSeg, segs - 1);
    const uint8_t* u = container + ((size_t)t * segs + seg) * kUnit;
    const uint8_t* codes = u + (g0 % kSeg) * 512 + lane * 16 * spread;
#pragma unroll
    for (int p = 0; p < GPW / 2; ++p) w.w[p] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(codes + p * 1024));
    const uint32_t* sp = reinterpret_cast<const uint32_t*>(u + kUnitCodes + (g0 % kSeg) * 2 + c * 16 * spread);
#pragma unroll
    for (int p = 0; p < GPW / 2; ++p) w.s[p] = sp[p];
    if constexpr (RANK) {
      // (a wave that adds no ranks reads one address)
      const bool adds = share == 0 && wave < steps;
      const int n = adds ? min(t * 16 + c, N - 1) : 0, k = adds ? min(32 * wave + 8 * j, r - 8) : 0;
      w.l2 = *reinterpret_cast<const v8bf*>(L2p + (size_t)n * r + k);
    }
  };
  // the (tile, chunk) after one
  auto after = [&](int& t, int& ch) {
    const bool wrap = HOLD || ch + 1 >= chunks;
    t += wrap ? per : 0;
    ch = HOLD ? share : wrap ? 0 : ch + 1;
  };

  constexpr int STAGES = HOLD && !(MT == 2 && GPW == 8) ? 3 : 2;  // (as far as the registers go)
  Weights<GPW> wa, wb, wc;
  Rows<MT, GPW> xa, xb;
  int tile2 = tile, chunk2 = chunk;  // what the next load reads
  auto load_next = [&](Weights<GPW>& w, Rows<MT, GPW>& x) {
    const bool there = tile2 < end;
    load_w(there ? tile2 : tile, chunk2, there, w);
    if (!HOLD) load_x(chunk2, x);
    after(tile2, chunk2);
  };
  if (HOLD) load_x(share, xa);
  load_next(wa, xa);
  if (STAGES == 3) load_next(wb, xa);
  auto barrier = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };
  // T (its slices' sum) as the low-rank product's operand; ranks past r and lo rows are 0.  All
  // threads add, four elements of every fold-th slice each, eight loads in flight; then a wave splits
  // a (row tile, matrix step) into its bf16 terms.
  if (RANK && share == 0) {
    static_assert(sizeof(red) >= MT * 16 * 128 * 4, "the sums fit where the waves meet");
    v4f* sums = reinterpret_cast<v4f*>(&red[0][0][0][0]);
    const int quads = rows * r / 4, fold = max(1, min(kWaves * 64 / quads, slices));
    for (int i = threadIdx.x; i < quads * fold; i += kWaves * 64) {
      const int from = i / quads, at = i % quads;
      const v4f* pp = reinterpret_cast<const v4f*>(parts + (size_t)row0 * r) + at;
      v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int q = from; q < slices; q += 8 * fold) {
        v4f v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = pp[(size_t)min(q + e * fold, slices - 1) * (M * r / 4)];
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] += q + e * fold < slices ? v[e][k] : 0.0f;
      }
      sums[i] = x;
    }
    barrier();
    for (int task = wave; task < MT * steps; task += kWaves) {
      const int t = task / steps, st = task % steps, m = t * RPT + c, k = 32 * st + 8 * j;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
      if (c < RPT && m < rows && k < r)
        for (int p = 0; p < fold; ++p) {
          const v4f* q = sums + p * quads + (m * r + k) / 4;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] += q[i >> 2][i & 3];
        }
      v8bf p[TERMS];
      split_bf16<TERMS>(x, p);
#pragma unroll
      for (int i = 0; i < TERMS; ++i) t_lds[t][st][i][lane] = p[i];
    }
    barrier();
  }

  int par = 0;
  v4f acc[MT];
  // One (tile, chunk): loads ahead, this one's products; false after the last.
  auto step = [&](Weights<GPW>& w, Weights<GPW>& wn, Rows<MT, GPW>& x, Rows<MT, GPW>& xn) {
    load_next(wn, xn);
    if (HOLD || chunk == 0) {
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (RANK && share == 0 && wave < steps) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < TERMS; ++i) acc[t] = mfma_bf16(t_lds[t][wave][i][lane], w.l2, acc[t]);
      }
    }
    v4f part[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) part[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < GPW; ++u) {
      const v4u q = w.w[u / 2];
      const v8h b0 = unpack8_f16(u & 1 ? q.z : q.x), b1 = unpack8_f16(u & 1 ? q.w : q.y);
      const float sw = half_bits_to_float((uint16_t)(u & 1 ? w.s[u / 2] >> 16 : w.s[u / 2]));
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        v4f p = mfma_f16(x.a[t][u][0], b0, v4f{0.0f, 0.0f, 0.0f, 0.0f});
        p = mfma_f16(x.a[t][u][1], b1, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) part[t][i] = __builtin_fmaf(p[i], sw, part[t][i]);
      }
    }
    const bool counts = (chunk * kWaves + wave) * GPW < G;
    const bool last = HOLD || chunk + 1 == chunks;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(part[t][i], counts ? x.up[t][i] : 0.0f, acc[t][i]);
    if (last) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[par][wave][t * 16 + 4 * j + i][c] = acc[t][i];
      barrier();
      for (int i = threadIdx.x; i < rows * 16; i += kWaves * 64) {
        const int m = i >> 4, col = i & 15, nn = tile * 16 + col;
        if (nn < N) {
          const int rr = FP32 ? (m >> 3) * 16 + (m & 7) : m;
          float y = 0.0f;
#pragma unroll
          for (int q = 0; q < kWaves; ++q) {
            y += red[par][q][rr][col];
            if (FP32) y += red[par][q][rr + 8][col];
          }
          if (HOLD && shares > 1) {
            partial[((size_t)share * rows + m) * (all * 16) + nn] = y;
            continue;
          }
          if (bias) y += bf16_bits_to_float(bias[nn]);
          const size_t at = (size_t)(row0 + m) * N + nn;
          if (FP32) {
            static_cast<float*>(Y)[at] = y;
          } else {
            static_cast<uint16_t*>(Y)[at] = float_to_bf16_bits(y);
          }
        }
      }
      par ^= 1;  // (the next tile's barrier separates these reads from the buffer's next writes)
    }
    after(tile, chunk);
    return tile < end;
  };
  if constexpr (STAGES == 3) {
    while (step(wa, wc, xa, xa) && step(wb, wa, xa, xa) && step(wc, wb, xa, xa)) {
    }
  } else {
    while (step(wa, wb, xa, xb) && step(wb, wa, xb, xa)) {
    }
  }
}

// Adds the shares of a pass and the bias; a thread has four columns of a row.
template <bool FP32>
__global__ __launch_bounds__(256) void w4a16_sum_kernel(const float* __restrict__ partial, int shares,
                                                        const uint16_t* __restrict__ bias, int rows,
                                                        int row0, int N, void* __restrict__ Y) {
  const int quads = (N + 15) / 16 * 4, at = blockIdx.x * 256 + threadIdx.x;
  if (at >= rows * quads) return;
  const int m = at / quads, n = at % quads * 4;
  v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int q = 0; q < shares; q += 4) {
    v4f v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      v[u] = reinterpret_cast<const v4f*>(partial)[(size_t)min(q + u, shares - 1) * rows * quads + at];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += q + u < shares ? v[u][i] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < N) {
      const float z = bias ? y[i] + bf16_bits_to_float(bias[n + i]) : y[i];
      const size_t to = (size_t)(row0 + m) * N + n + i;
      if (FP32) {
        static_cast<float*>(Y)[to] = z;
      } else {
        static_cast<uint16_t*>(Y)[to] = float_to_bf16_bits(z);
      }
    }
}

struct W4a16Call {
  const v8h* frags;
  const float* scales;
  const float* parts;
  int slices;
  const uint8_t* container;
  const uint16_t* L2p;
  const uint16_t* bias;
  int M, N, K, r, tiles;
  float* partial;
  void* Y;
  hipStream_t stream;
};

template <int MT, int GPW, bool FP32, bool RANK>
static hipError_t launch_main(const W4a16Call& a, int tile0) {
  const W4a16Pass p = w4a16_pass(a.M, a.N, a.K, tile0, a.tiles, FP32);
#define SVDQ_MAIN(HOLD)                                                                            \
  hipLaunchKernelGGL((w4a16_kernel<MT, GPW, HOLD, FP32, RANK>), dim3(p.grid), dim3(kWaves * 64),   \
                     0, a.stream, a.frags, a.scales, a.parts, a.slices, a.container, a.L2p,        \
                     a.bias, a.M, a.N, a.K, a.r, tile0, a.tiles, p.shares, a.partial, a.Y)
  if constexpr (MT == 1) {
    if (p.loop) SVDQ_MAIN(false);
    else SVDQ_MAIN(true);
  } else {
    SVDQ_MAIN(true);
  }
#undef SVDQ_MAIN
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.shares == 1) return e;
  const long long threads = (long long)p.rows * ((a.N + 15) / 16 * 4);
  hipLaunchKernelGGL(w4a16_sum_kernel<FP32>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, a.stream,
                     a.partial, p.shares, a.bias, p.rows, tile0 * w4a16_rows_per_tile(FP32), a.N, a.Y);
  return hipGetLastError();
}

template <bool FP32, bool RANK>
static hipError_t launch_tiles(const W4a16Call& a) {
  for (int t = 0; t < a.tiles; t += kMaxTiles) {
    const int left = a.tiles - t;
    const hipError_t e = left >= 4   ? launch_main<4, groups_per_wave(4), FP32, RANK>(a, t)
                         : left == 3 ? launch_main<3, groups_per_wave(3), FP32, RANK>(a, t)
                         : left == 2 ? launch_main<2, groups_per_wave(2), FP32, RANK>(a, t)
                                     : launch_main<1, groups_per_wave(1), FP32, RANK>(a, t);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_w4a16_gemv(const uint16_t* X, const float* inv_lambda, const uint16_t* L1p,
                             const uint8_t* container, const uint16_t* L2p, const uint16_t* bias,
                             int M, int N, int K, int r, void* Y, int out_fp32, void* workspace,
                             hipStream_t stream) {
  const W4a16Ws w = w4a16_layout(M, N, K, r, out_fp32);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  v8h* frags = reinterpret_cast<v8h*>(base + w.frags);
  float* scales = reinterpret_cast<float*>(base + w.scales);
  float* parts = reinterpret_cast<float*>(base + w.parts);
  const int tiles = w4a16_tiles(M, out_fp32), slices = w4a16_slices(K);
  const dim3 grid(slices, tiles);
#define SVDQ_PREP(RT)                                                                            \
  hipLaunchKernelGGL(w4a16_prep_kernel<RT>, grid, dim3(kSeg * 64), 0, stream, X, inv_lambda,     \
                     L1p, M, K, r, out_fp32, frags, scales, parts)
  if (r == 0) SVDQ_PREP(0);
  else if (r <= 32) SVDQ_PREP(2);
  else if (r <= 64) SVDQ_PREP(4);
  else SVDQ_PREP(8);
#undef SVDQ_PREP
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const W4a16Call a{frags, scales, parts, slices, container, L2p, bias, M, N, K, r, tiles, reinterpret_cast<float*>(base + w.partial), Y, stream};
  if (out_fp32) return r ? launch_tiles<true, true>(a) : launch_tiles<true, false>(a);
  return r ? launch_tiles<false, true>(a) : launch_tiles<false, false>(a);
}

}  // namespace svdq
