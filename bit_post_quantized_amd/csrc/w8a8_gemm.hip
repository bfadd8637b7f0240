// Product of 8-bit integers with a scale for each row and column.
//
//   Y[m, n] = sx[m] sw[n] sum_k qx[m, k] qw[n, k] + bias[n]
//
// The sums are int32 on v_mfma_i32_16x16x64_i8 and exact, so they may be divided over waves and
// workgroups in any way.  The weight is the first operand (rows of the result) and X the second
// (columns): a lane then holds four neighbouring columns of Y in one row.
//   operand: lane l has row l % 16, k = 16 (l / 16) .. + 15 of 64;
//   result:  lane l has column l % 16 (a row of X), rows 4 (l / 16) + e (columns of Y).
#include "decoder_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {
namespace {

constexpr int kUnit = 1024;  // 16 columns x 64 k of the container

__device__ __forceinline__ v4i mfma(v4i w, v4i x, v4i acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0);
}

template <int N>
struct Count {
  static constexpr int value = N;
};

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

// ---------------------------------------------------------------- few rows
// A workgroup has CT tiles of 16 columns and all of K, dealt unit by unit to its waves; each wave
// keeps RT x CT accumulators and the waves' sums meet in LDS.  The weights are read once, in whole
// units; X comes from L2.
template <int RT, int CT, int WAVES, bool F32>
__global__ __launch_bounds__(64 * WAVES) void w8a8_few_kernel(const int8_t* __restrict__ qx,
                                                              const int8_t* __restrict__ container,
                                                              int K, Output o) {
  constexpr int TILES = RT * CT, CHUNK = TILES < 4 ? TILES : 4;  // tiles exchanged at a time
  __shared__ v4i parts[WAVES][CHUNK][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = K / 64, tiles = (o.N + 15) / 16, t0 = blockIdx.x * CT;
  const int8_t* x[RT];
  const int8_t* w[CT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    x[r] = qx + (size_t)min(16 * r + (lane & 15), o.M - 1) * K + 16 * (lane >> 4);
#pragma unroll
  for (int c = 0; c < CT; ++c)
    w[c] = container + (size_t)min(t0 + c, tiles - 1) * G * kUnit + lane * 16;
  v4i acc[CT][RT] = {};
  // U units at a time, so that their loads are in flight together (a loop around matrix instructions is
  // not unrolled by the compiler)
  auto step = [&](int u, auto count) {
    constexpr int U = decltype(count)::value;
    v4i wf[U][CT], xf[U][RT];
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int c = 0; c < CT; ++c)
        wf[i][c] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(w[c] + (size_t)(u + i * WAVES) * kUnit));
#pragma unroll
      for (int r = 0; r < RT; ++r) xf[i][r] = *reinterpret_cast<const v4i*>(x[r] + 64 * (u + i * WAVES));
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[c][r] = mfma(wf[i][c], xf[i][r], acc[c][r]);
  };
  constexpr int U = RT * CT > 4 ? 2 : 4;
  int u = wave;
  for (; u + (U - 1) * WAVES < G; u += U * WAVES) step(u, Count<U>());
  for (; u < G; u += WAVES) step(u, Count<1>());
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
#define SVDQ_LDS(p) ((__attribute__((address_space(3))) void*)(p))

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// 16 bytes per lane from base + offset (0 past the buffer's end) to `to` + 16 lane of LDS
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t base, uint8_t* to, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, SVDQ_LDS(to), 16, offset, 0, 0, 0);
}

// s_waitcnt vmcnt(0) lgkmcnt(0): the loads into LDS have landed, the reads from it are done
#define SVDQ_WAIT_LDS() __builtin_amdgcn_s_waitcnt(7 << 4)

// A workgroup has a TM x TN tile of Y and WM x WN waves; K in stages of 128, two of them in LDS, filled
// by loads that go straight there: while one is computed the next is on its way.
//   X stage: rows of 128 bytes as in memory, their eight pieces of 16 bytes exchanged by the row
//     (slot p of row r holds piece p ^ (r % 8)): a load of 64 lanes then reads eight whole rows, and an
//     operand's read, 16 rows of the same piece, meets every bank equally.
//   W stage: units of the container as they are, each an operand.
// Reads past the last row or tile of columns are cut off by the buffers' sizes and give 0.
template <int TM, int TN, int WM, int WN, bool F32>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2)))
void w8a8_tile_kernel(const int8_t* __restrict__ qx, const int8_t* __restrict__ container, int K,
                      Output o, int split, int32_t* __restrict__ partial) {
  constexpr int WAVES = WM * WN, kA = TM * 128, kB = TN * 128, kStage = kA + kB;
  constexpr int RT = TM / WM / 16, CT = TN / WN / 16;   // tiles of a wave
  constexpr int kLoadsA = kA / 1024 / WAVES, kLoadsB = kB / 1024 / WAVES;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int G = K / 64, S = (G + 1) / 2, tiles = (o.N + 15) / 16;
  int mt, nt;
  xcd_tile_order(8, mt, nt);
  const int m0 = mt * TM, n0 = nt * TN;
  const int s0 = (int)((int64_t)S * blockIdx.z / split), s1 = (int)((int64_t)S * (blockIdx.z + 1) / split);

  const int8_t* ax = qx + (size_t)m0 * K;
  const int8_t* bw = container + (size_t)(n0 / 16) * G * kUnit;
  const int a_bytes = min(o.M - m0, TM) * K, b_bytes = min(tiles - n0 / 16, TN / 16) * G * kUnit;
  uint32_t a_off[kLoadsA], b_off[kLoadsB];
#pragma unroll
  for (int j = 0; j < kLoadsA; ++j) {
    const int r = 8 * (j * WAVES + wave) + lane / 8;
    a_off[j] = (uint32_t)r * K + 16 * ((lane & 7) ^ (r & 7));
  }
#pragma unroll
  for (int j = 0; j < kLoadsB; ++j) {
    const int i = j * WAVES + wave;
    b_off[j] = (uint32_t)(i / 2) * G * kUnit + (i & 1) * kUnit + lane * 16;
  }
  auto issue = [&](int s) {
    uint8_t* st = lds + (s & 1) * kStage;
    const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(ax + s * 128, a_bytes - s * 128);
    const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(bw + (size_t)s * 2 * kUnit, b_bytes - s * 2 * kUnit);
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j)
      load_to_lds(ra, st + (j * WAVES + wave) * 1024, a_off[j]);
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j)
      load_to_lds(rb, st + kA + (j * WAVES + wave) * 1024, b_off[j]);
  };

  v4i acc[RT][CT] = {};
  const int a_row = (wm * RT * 16 + (lane & 15)) * 128;
  const int a_piece = lane >> 4, a_turn = lane & 7;
  const int b_at = kA + wn * CT * 2 * kUnit + lane * 16;
  auto unit = [&](const uint8_t* st, int u) {
    v4i xf[RT], wf[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) wf[c] = *reinterpret_cast<const v4i*>(st + b_at + (2 * c + u) * kUnit);
#pragma unroll
    for (int r = 0; r < RT; ++r)
      xf[r] = *reinterpret_cast<const v4i*>(st + a_row + r * 16 * 128 + 16 * ((4 * u + a_piece) ^ a_turn));
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[r][c] = mfma(wf[c], xf[r], acc[r][c]);
  };
  if (s0 < s1) issue(s0);
  for (int s = s0; s < s1; ++s) {
    // stage s has landed for every wave, and every wave has read stage s - 1
    SVDQ_WAIT_LDS();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (s + 1 < s1) issue(s + 1);
    const uint8_t* st = lds + (s & 1) * kStage;
    unit(st, 0);
    if (2 * s + 1 < G) unit(st, 1);   // (an odd number of units: the last stage has one)
    asm volatile("" ::: "memory");
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int m = m0 + (wm * RT + r) * 16 + (lane & 15);
    if (m < o.M) {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int n = n0 + (wn * CT + c) * 16 + 4 * (lane >> 4);
        if (n < o.N) {
          if (split == 1) {
            store4<F32>(o, m, n, acc[r][c]);
          } else {
            // (partials have rows of whole tiles, so that four columns are one store)
            const size_t pitch = (size_t)tiles * 16;
            *reinterpret_cast<v4i*>(partial + ((size_t)blockIdx.z * o.M + m) * pitch + n) = acc[r][c];
          }
        }
      }
    }
  }
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

// ---------------------------------------------------------------- choice
constexpr int kFewRows = 64;
constexpr int kCus = 256;

struct Plan {
  int tile;    // 0: few rows
  int split;
};

Plan plan(int M, int N, int K) {
  if (M <= kFewRows) return {0, 1};
  const int64_t big = (int64_t)((M + 255) / 256) * ((N + 255) / 256);
  if (big >= kCus) return {256, 1};
  // tiles of 128, K divided where they are fewer than two per CU and a share keeps 4 stages
  const int64_t small = (int64_t)((M + 127) / 128) * ((N + 127) / 128);
  const int S = (K / 64 + 1) / 2;
  int64_t split = 2 * kCus / small;
  if (split > S / 4) split = S / 4;
  return {128, split < 1 ? 1 : (int)split};
}

template <int RT, int CT, int WAVES>
void launch_few(const int8_t* qx, const int8_t* container, int K, const Output& o, int f32, hipStream_t st) {
  const dim3 grid(((o.N + 15) / 16 + CT - 1) / CT), block(64 * WAVES);
  if (f32) hipLaunchKernelGGL((w8a8_few_kernel<RT, CT, WAVES, true>), grid, block, 0, st, qx, container, K, o);
  else hipLaunchKernelGGL((w8a8_few_kernel<RT, CT, WAVES, false>), grid, block, 0, st, qx, container, K, o);
}

template <int RT>
void launch_few_rows(const int8_t* qx, const int8_t* container, int K, const Output& o, int f32, hipStream_t st) {
  const int tiles = (o.N + 15) / 16;
  if (tiles >= 4 * 2 * kCus) launch_few<RT, 4, 8>(qx, container, K, o, f32, st);
  else if (tiles >= 2 * 2 * kCus) launch_few<RT, 2, 8>(qx, container, K, o, f32, st);
  else launch_few<RT, 1, 16>(qx, container, K, o, f32, st);
}

template <int T, int WM, int WN, bool F32>
hipError_t launch_tile(const int8_t* qx, const int8_t* container, int K, const Output& o, int split, int32_t* ws,
                 hipStream_t st) {
  constexpr int kLds = 2 * 2 * T * 128;
  // two stages need more than the default 64 KB of LDS
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(w8a8_tile_kernel<T, T, WM, WN, F32>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  const dim3 grid((o.N + T - 1) / T, (o.M + T - 1) / T, split);
  hipLaunchKernelGGL((w8a8_tile_kernel<T, T, WM, WN, F32>), grid, dim3(64 * WM * WN), kLds, st, qx, container, K, o,
                     split, ws);
  return hipGetLastError();
}

template <bool F32>
hipError_t launch_many(const int8_t* qx, const int8_t* container, int K, const Output& o, const Plan& p, int32_t* ws,
                 hipStream_t st) {
  if (p.tile == 256) return launch_tile<256, 2, 4, F32>(qx, container, K, o, 1, ws, st);
  const hipError_t e = launch_tile<128, 2, 2, F32>(qx, container, K, o, p.split, ws, st);
  if (e != hipSuccess) return e;
  if (p.split > 1) {
    const int64_t quads = (int64_t)((o.N + 15) / 16) * 4 * o.M, blocks = (quads + 255) / 256;
    hipLaunchKernelGGL((w8a8_join_kernel<F32>), dim3((int)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, ws,
                       p.split, o);
  }
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
  if (p.tile == 0) {
    switch ((M + 15) / 16) {
      case 1: launch_few_rows<1>(qx, container, K, o, out_fp32, stream); break;
      case 2: launch_few_rows<2>(qx, container, K, o, out_fp32, stream); break;
      case 3: launch_few_rows<3>(qx, container, K, o, out_fp32, stream); break;
      default: launch_few_rows<4>(qx, container, K, o, out_fp32, stream); break;
    }
  } else if (out_fp32) {
    return launch_many<true>(qx, container, K, o, p, static_cast<int32_t*>(workspace), stream);
  } else {
    return launch_many<false>(qx, container, K, o, p, static_cast<int32_t*>(workspace), stream);
  }
  return hipGetLastError();
}

}  // namespace svdq
