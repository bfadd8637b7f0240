// The linear layer on few rows: INT4 weights, 16-bit activations, fp32 sums.
//
//     Y[m, n] = sum_g s_w[g, n] sum_{k in g} X^[m, k] q[n, k] + sum_j T[m, j] L2[j, n] + bias[n],
//     X^ = fl32(X inv_lambda),  T = X^ L1
//
// With few rows the weights are read once and used M times, so the floor is their N K / 2 bytes.
// The products run on v_mfma_f32_16x16x32_f16: a code is an exact fp16, and an activation enters
// as an fp16 after a power-of-two scale per (row, group) (11 significant bits, for bf16 output) or
// as the fp16 pair hi + lo (22 bits, for fp32 output); products of 11 x 4 bits are exact and the
// sums are the matrix unit's fp32.
//  1. w4a16_prep_kernel: X^ in the matrix operand's order, its scales, and T's partial sums over
//     slices of K (bf16 MFMA on X^ split into three bf16, which keeps all 24 bits).
//  2. w4a16_kernel: one workgroup per 16 columns; its waves split K, each lane turns 16 nibbles of
//     one column into fp16 per group, one fp32 FMA per output and group applies the two scales,
//     and the waves meet in LDS, where the low-rank product and the bias join.
#include "serve_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kFragBytes = 2048;     // one (row tile, group): 16 rows x 64 k of fp16
constexpr int kPrepWaves = 4;
constexpr int kMaxSlices = 16;

// Row tiles: 16 rows each, or for fp32 output 8 rows, hi parts in matrix rows 0..7 and lo parts
// in rows 8..15.
__host__ __device__ inline int w4a16_rows_per_tile(int out_fp32) { return out_fp32 ? 8 : 16; }

inline int w4a16_tiles(int M, int out_fp32) {
  const int rpt = w4a16_rows_per_tile(out_fp32);
  return (M + rpt - 1) / rpt;
}

// Slices of K for T's partial sums: enough workgroups to be short, few enough that summing the
// partials again in every workgroup of the main kernel (32 KB) stays cheap.
inline int w4a16_slices(int M, int K, int r) {
  const int G = K / kGroup;
  int s = (G + kPrepWaves - 1) / kPrepWaves;
  if (s > kMaxSlices) s = kMaxSlices;
  while (s > 1 && (long long)s * M * r * 4 > 32768) --s;
  return s;
}

struct W4a16Ws {
  size_t frags, scales, parts, bytes;  // byte offsets and the total
};

inline W4a16Ws w4a16_layout(int M, int K, int r, int out_fp32) {
  const size_t tiles = w4a16_tiles(M, out_fp32), G = K / kGroup;
  W4a16Ws w;
  w.frags = 0;
  w.scales = tiles * G * kFragBytes;
  w.parts = w.scales + tiles * G * 16 * sizeof(float);
  w.bytes = w.parts + (size_t)w4a16_slices(M, K, r) * M * r * sizeof(float);
  return w;
}

size_t w4a16_workspace_bytes(int M, int K, int r, int out_fp32) {
  return w4a16_layout(M, K, r, out_fp32).bytes;
}

// The matrix operand's k order inside a lane's 8: the order in which unpack8_f16 yields them.
__device__ __forceinline__ int frag_k(int i) { return (i >> 1) + ((i & 1) << 2); }

// Eight packed nibbles -> eight exact fp16 codes, in the order k0 k4 k1 k5 k2 k6 k3 k7.  After the
// flip of bit 3 a nibble holds c + 8; or-ed into the mantissa of 1024 it makes 1024 + (c + 8), or
// from bits 4..7 1024 + 16 (c + 8), and one packed fp16 operation takes the offset (and the 16)
// away, exactly.
__device__ __forceinline__ v8h unpack8_f16(uint32_t w) {
  const uint32_t u = w ^ 0x88888888u, v = u >> 8;
  const v2h six = {(_Float16)0.0625f, (_Float16)0.0625f};
  const v2h off0 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
  const v2h off4 = {(_Float16)-72.0f, (_Float16)-72.0f};
  const v2h a = __builtin_bit_cast(v2h, (u & 0x000F000Fu) | 0x64006400u) + off0;
  const v2h b = __builtin_elementwise_fma(__builtin_bit_cast(v2h, (u & 0x00F000F0u) | 0x64006400u), six, off4);
  const v2h c = __builtin_bit_cast(v2h, (v & 0x000F000Fu) | 0x64006400u) + off0;
  const v2h d = __builtin_elementwise_fma(__builtin_bit_cast(v2h, (v & 0x00F000F0u) | 0x64006400u), six, off4);
  return v8h{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ v4f mfma_f16(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma_bf16(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One workgroup per (slice of K, row tile); a wave takes every kPrepWaves-th group of the slice.
// Lane (row l % 16, j = l / 16) holds k = 64 g + 16 j .. + 15.
__global__ __launch_bounds__(kPrepWaves * 64) void w4a16_prep_kernel(
    const uint16_t* __restrict__ X, const float* __restrict__ inv_lambda,
    const uint16_t* __restrict__ L1p, int M, int K, int r, int out_fp32, v8h* __restrict__ frags,
    float* __restrict__ scales, float* __restrict__ parts) {
  __shared__ float red[kPrepWaves][16][17];
  const int G = K / kGroup, slices = gridDim.x, slice = blockIdx.x, tile = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int mr = lane & 15, j = lane >> 4;
  const int rpt = w4a16_rows_per_tile(out_fp32);
  const int row = tile * rpt + (mr & (rpt - 1));
  const bool live = row < M, low = out_fp32 && mr >= 8;
  const int g0 = (int)((long long)G * slice / slices), g1 = (int)((long long)G * (slice + 1) / slices);
  const int ranks = r / 16;

  v4f t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  for (int g = g0 + wave; g < g1; g += kPrepWaves) {
    const int k0 = g * kGroup + 16 * j;
    float x[16];
    float amax = 0.0f;
    if (live) {
      const v4u* xp = reinterpret_cast<const v4u*>(X + (size_t)row * K + k0);
      const v4u w0 = xp[0], w1 = xp[1];
      const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      const v4f* lp = reinterpret_cast<const v4f*>(inv_lambda + k0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4f l = lp[i];
        x[4 * i] = __uint_as_float(w[2 * i] << 16) * l.x;
        x[4 * i + 1] = __uint_as_float(w[2 * i] & 0xFFFF0000u) * l.y;
        x[4 * i + 2] = __uint_as_float(w[2 * i + 1] << 16) * l.z;
        x[4 * i + 3] = __uint_as_float(w[2 * i + 1] & 0xFFFF0000u) * l.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(x[i]));
    amax = __builtin_fmaxf(amax, __shfl_xor(amax, 16));
    amax = __builtin_fmaxf(amax, __shfl_xor(amax, 32));
    // 2^e with amax 2^-e in [2^10, 2^11) (e clamped so that both powers are normal; 0 keeps e = 0)
    int e = (int)(__float_as_uint(amax) >> 23) - 127 - 10;
    e = amax == 0.0f ? 0 : max(e, -110);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    _Float16 h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = x[i] * down;
      const _Float16 hi = (_Float16)y;
      h[i] = low ? (_Float16)(y - (float)hi) : hi;
    }
    const size_t base = ((size_t)tile * G + g) * 128;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      v8h f;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = h[8 * s + (i >> 1) + ((i & 1) << 2)];
      frags[base + s * 64 + lane] = f;
    }
    if (j == 0) scales[((size_t)tile * G + g) * 16 + mr] = up;

    if (ranks) {
      // X^ = p0 + p1 + p2, each a bf16 (8 bits at a time)
      v8bf p[3][2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[8 * s + i];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          p[c][s] = to_bf16x8(y);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] -= (float)p[c][s][i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i < ranks) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const v8bf b = *reinterpret_cast<const v8bf*>(L1p + (size_t)(16 * i + mr) * K + k0 + 8 * s);
#pragma unroll
            for (int c = 0; c < 3; ++c) t[i] = mfma_bf16(p[c][s], b, t[i]);
          }
        }
      }
    }
  }

  // T's partial of this slice: the waves' sums meet in LDS, one tile of 16 ranks after the other
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < ranks) {
#pragma unroll
      for (int q = 0; q < 4; ++q) red[wave][4 * j + q][mr] = t[i][q];
      __syncthreads();
      const int m = threadIdx.x >> 4, c = threadIdx.x & 15, out = tile * rpt + m;
      if (m < rpt && out < M) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kPrepWaves; ++w) s += red[w][m][c];
        parts[((size_t)slice * M + out) * r + 16 * i + c] = s;
      }
      __syncthreads();
    }
  }
}

// MT row tiles, WAVES waves that split K.  LDS: the waves' sums, T and the columns' L2 rows.
template <int MT, int WAVES, bool FP32>
__global__ __launch_bounds__(WAVES * 64) void w4a16_kernel(
    const v8h* __restrict__ frags, const float* __restrict__ scales,
    const float* __restrict__ parts, int slices, const uint8_t* __restrict__ wq,
    const uint16_t* __restrict__ w_scales, const uint16_t* __restrict__ L2p,
    const uint16_t* __restrict__ bias, int M, int N, int K, int r, int tile0,
    int tiles, void* __restrict__ Y) {
  constexpr int RPT = FP32 ? 8 : 16;
  constexpr int UNROLL = 4;
  extern __shared__ float lds[];
  float* red = lds;                           // [WAVES][MT * 16][17]
  float* Ts = lds + WAVES * MT * 16 * 17;     // [rows of these tiles][r]
  const int G = K / kGroup;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, j = lane >> 4;
  const int n0 = blockIdx.x * 16, n = min(n0 + c, N - 1);
  const int g0 = (int)((long long)G * wave / WAVES), g1 = (int)((long long)G * (wave + 1) / WAVES);
  const int row0 = tile0 * RPT, rows = min(M - row0, MT * RPT);

  v4f acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const uint8_t* wp = wq + (size_t)n * (K / 2) + 8 * j;
  const uint16_t* sp = w_scales + n;

  for (int g = g0; g < g1; g += UNROLL) {
    v2u w[UNROLL];
    uint16_t s[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int gu = min(g + u, g1 - 1);
      w[u] = *reinterpret_cast<const v2u*>(wp + (size_t)gu * 32);
      s[u] = sp[(size_t)gu * N];
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (g + u < g1) {
        const v8h b0 = unpack8_f16(w[u].x), b1 = unpack8_f16(w[u].y);
        const float sw = half_bits_to_float(s[u]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          // (a tile past the last reads the last one's operands; its results are not stored)
          const size_t at = (size_t)min(tile0 + t, tiles - 1) * G + g + u;
          const v8h a0 = frags[at * 128 + lane], a1 = frags[at * 128 + 64 + lane];
          const v4f up = *reinterpret_cast<const v4f*>(scales + at * 16 + 4 * j);
          v4f p = mfma_f16(a0, b0, v4f{0.0f, 0.0f, 0.0f, 0.0f});
          p = mfma_f16(a1, b1, p);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(p[i], sw * up[i], acc[t][i]);
        }
      }
    }
  }

#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[(wave * MT * 16 + t * 16 + 4 * j + i) * 17 + c] = acc[t][i];
  for (int i = threadIdx.x; i < rows * r; i += WAVES * 64) {
    float s = 0.0f;
    for (int q = 0; q < slices; ++q) s += parts[((size_t)q * M + row0) * r + i];
    Ts[i] = s;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * 16; i += WAVES * 64) {
    const int m = i >> 4, col = i & 15, nn = n0 + col;
    if (nn >= N) continue;
    const int rr = FP32 ? (m >> 3) * 16 + (m & 7) : m;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      y += red[(w * MT * 16 + rr) * 17 + col];
      if (FP32) y += red[(w * MT * 16 + rr + 8) * 17 + col];
    }
    if (r) {
      const v4u* lp = reinterpret_cast<const v4u*>(L2p + (size_t)nn * r);
      float z = 0.0f;
      for (int q = 0; q < r / 8; ++q) {
        const v4u l = lp[q];
        const float* tp = Ts + m * r + 8 * q;
        const uint32_t lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          z = __builtin_fmaf(tp[2 * p], __uint_as_float(lw[p] << 16), z);
          z = __builtin_fmaf(tp[2 * p + 1], __uint_as_float(lw[p] & 0xFFFF0000u), z);
        }
      }
      y += z;
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

template <int MT, int WAVES, bool FP32>
static hipError_t launch_main(const v8h* frags, const float* scales, const float* parts,
                              int slices, const uint8_t* wq, const uint16_t* w_scales,
                              const uint16_t* L2p, const uint16_t* bias, int M, int N, int K,
                              int r, int tile0, int tiles, void* Y, hipStream_t stream) {
  const int rows = min(M - tile0 * (FP32 ? 8 : 16), MT * (FP32 ? 8 : 16));
  const size_t lds = ((size_t)WAVES * MT * 16 * 17 + (size_t)rows * r) * sizeof(float);
  hipLaunchKernelGGL((w4a16_kernel<MT, WAVES, FP32>), dim3((N + 15) / 16), dim3(WAVES * 64), lds,
                     stream, frags, scales, parts, slices, wq, w_scales, L2p, bias, M, N, K, r,
                     tile0, tiles, Y);
  return hipGetLastError();
}

template <bool FP32>
static hipError_t launch_tiles(const v8h* frags, const float* scales, const float* parts,
                               int slices, const uint8_t* wq, const uint16_t* w_scales,
                               const uint16_t* L2p, const uint16_t* bias, int M, int N, int K,
                               int r, int tiles, void* Y, hipStream_t stream) {
  // up to 4 row tiles share a pass over the weights (64 bf16 rows, 32 fp32 rows)
  for (int t = 0; t < tiles; t += 4) {
    const int left = tiles - t;
    hipError_t e;
    if (left >= 3)
      e = launch_main<4, 4, FP32>(frags, scales, parts, slices, wq, w_scales, L2p, bias, M, N, K, r, t, tiles, Y, stream);
    else if (left == 2)
      e = launch_main<2, 8, FP32>(frags, scales, parts, slices, wq, w_scales, L2p, bias, M, N, K, r, t, tiles, Y, stream);
    else
      e = launch_main<1, 8, FP32>(frags, scales, parts, slices, wq, w_scales, L2p, bias, M, N, K, r, t, tiles, Y, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_w4a16_gemv(const uint16_t* X, const float* inv_lambda, const uint16_t* L1p,
                             const uint8_t* wq, const uint16_t* w_scales, const uint16_t* L2p,
                             const uint16_t* bias, int M, int N, int K, int r, void* Y,
                             int out_fp32, void* workspace, hipStream_t stream) {
  const W4a16Ws w = w4a16_layout(M, K, r, out_fp32);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  v8h* frags = reinterpret_cast<v8h*>(base + w.frags);
  float* scales = reinterpret_cast<float*>(base + w.scales);
  float* parts = reinterpret_cast<float*>(base + w.parts);
  const int tiles = w4a16_tiles(M, out_fp32), slices = w4a16_slices(M, K, r);
  hipLaunchKernelGGL(w4a16_prep_kernel, dim3(slices, tiles), dim3(kPrepWaves * 64), 0, stream, X,
                     inv_lambda, L1p, M, K, r, out_fp32, frags, scales, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (out_fp32)
    return launch_tiles<true>(frags, scales, parts, slices, wq, w_scales, L2p, bias, M, N, K, r,
                              tiles, Y, stream);
  return launch_tiles<false>(frags, scales, parts, slices, wq, w_scales, L2p, bias, M, N, K, r,
                             tiles, Y, stream);
}

}  // namespace svdq
