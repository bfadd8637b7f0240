// Root-mean-square norm of rows with the residual's addition, to bf16 or to 8 bits with a scale for
// each row, and the 8 bits without the norm.
//
//   h = fl32(x + residual),  g = fl32(h gamma),  y = fl32(g rstd),
//   rstd = 1 / sqrt(sum h^2 / K + eps),  s = fl32(max |y| / 127),  c = rne(fl32(y / s)).
//
// Rounding is monotone, so max |y| = fl32(rstd max |g|) exactly, and one exchange between the waves
// carries both the sum of squares and max |g|: the row is read once, held in registers, and written
// once.  The maximum runs over the magnitudes' bits as whole numbers, in which a NaN is the largest.
//
// Where the sum of squares, or max |g|, leaves the middle of fp32's range (a row of zeros, of values
// past 2^60 or under 2^-50, or one with a NaN or an infinity), the row is scaled by a power of two that
// brings its largest |h| to [1, 2), and the exchange is made again: every row then has its 24 bits.
//
// Bound by memory: 16384 rows of 8192, bf16 with a residual to 8 bits, move 940 MB in 193 - 212 us (4.4 - 4.9 TB/s,
// where torch's copy of 1 GiB reaches 5.1 - 5.2 and one in runs of 16 KiB 6.2), to bf16 1074 MB in 197 (5.4), all of it
// in fp32 to bf16 1879 MB in 360 (5.2); 4096 x 8192 to 8 bits 52 - 57 us, in fp32 to bf16 92; 16384 x 4096 88.  Without the
// norm 16384 x 8192 take 77 us (5.2 TB/s), in fp32 111.  Rows that are read twice, 2048 x 32768: to bf16 135 us (4.0 TB/s of
// one reading), to 8 bits 127, in fp32 239, without the norm 51.  Up to a few hundred rows a call costs what its launch costs.
#include "decoder_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {
namespace {

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0u, v, CTRL, ROWS, 0xF, false);
}

// Sum of a (>= 0 or NaN) and maximum of m over the wave, in every lane.
__device__ __forceinline__ void wave_sum_max(float& a, uint32_t& m) {
#define SVDQ_STEP(CTRL, ROWS)                                   \
  a += __uint_as_float(dpp0<CTRL, ROWS>(__float_as_uint(a)));   \
  m = max(m, dpp0<CTRL, ROWS>(m));
  SVDQ_STEP(0x111, 0xF)
  SVDQ_STEP(0x112, 0xF)
  SVDQ_STEP(0x114, 0xF)
  SVDQ_STEP(0x118, 0xF)
  SVDQ_STEP(0x142, 0xA)
  SVDQ_STEP(0x143, 0xC)
#undef SVDQ_STEP
  a = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(a), 63));
  m = __builtin_amdgcn_readlane(m, 63);
}

// The same over the WAVES waves of a row; `slot` has WAVES places, and the caller uses another one
// for the next exchange (so one barrier is enough).
template <int WAVES>
__device__ __forceinline__ void row_sum_max(float& a, uint32_t& m, float2* slot) {
  wave_sum_max(a, m);
  if constexpr (WAVES > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) slot[w] = make_float2(a, __uint_as_float(m));
    __syncthreads();
    a = 0.0f;
    m = 0u;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const float2 p = slot[i];
      a += p.x;
      m = max(m, __float_as_uint(p.y));
    }
  }
}

// Eight values.  Rows are read and written once: past the caches (NT), where there are more of them than
// stay there; gamma is not.
template <bool NT, typename T>
__device__ __forceinline__ T fetch(const T* p) {
  return NT ? __builtin_nontemporal_load(p) : *p;
}
template <bool NT, typename T>
__device__ __forceinline__ void put(T* p, T v) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool NT, typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    const v4f a = fetch<NT>(reinterpret_cast<const v4f*>(p)), b = fetch<NT>(reinterpret_cast<const v4f*>(p) + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const v4u a = fetch<NT>(reinterpret_cast<const v4u*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

template <bool NT, typename T>
__device__ __forceinline__ void store8(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    put<NT>(reinterpret_cast<v4f*>(p), v4f{v[0], v[1], v[2], v[3]});
    put<NT>(reinterpret_cast<v4f*>(p) + 1, v4f{v[4], v[5], v[6], v[7]});
  } else {
    put<NT>(reinterpret_cast<v4u*>(p), __builtin_bit_cast(v4u, to_bf16x8(v)));   // (a NaN stays one)
  }
}

// Eight codes rne(fl32(y / s)) in [-127, 127]; 0 where s is 0 or not finite.
__device__ __forceinline__ v2u codes8(const float* y, float s, float rcp) {
  uint32_t b[8];
  if (s >= 0x1p-100f && s < __builtin_inff()) {
    // |y| <= 127 s (1 + 2^-23), so the quotient rounds to at most 127; it is rounded to a whole number by the
    // sum with 1.5 2^23, whose low byte is the code
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(div_rn(y[i], s, rcp) + 12582912.0f);
  } else {
    // (a scale that is hardly a normal number has no exact reciprocal: divide)
    const bool live = s > 0.0f && s < __builtin_inff();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = live ? y[i] / s : 0.0f;
      b[i] = (uint32_t)(int)fminf(fmaxf(__builtin_rintf(q), -127.0f), 127.0f);
    }
  }
  v2u w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000C0Cu);
    w[i] = lo | hi;
  }
  return w;
}

__device__ __forceinline__ bool ordinary(float a, uint32_t m) {
  // (comparisons with a NaN are false)
  return a >= 0x1p-96f && a <= 0x1p126f && m >= 0x0D800000u /* 2^-100 */ && m <= 0x7E800000u /* 2^126 */;
}

// 1 / sqrt(a / K + eps) for a row scaled by 2^-e, as a factor on the scaled row; in fp64, where
// neither end is near.  A row of zeros stays one, with eps 0 too.
__device__ __forceinline__ float scaled_rstd(float a, int K, float eps, int e) {
  return a == 0.0f ? 0.0f : (float)(1.0 / sqrt((double)a / K + ldexp((double)eps, -2 * e)));
}

// exponent that brings the largest |h| to [1, 2); 0 where it is zero or not finite
__device__ __forceinline__ int row_exponent(uint32_t m) {
  if (m == 0u || m >= 0x7F800000u) return 0;
  int e;
  (void)frexpf(__uint_as_float(m), &e);
  return e - 1;
}

// One row (or one of ROWS of a workgroup, a wave each) in registers: V pieces of 8 per thread.
template <typename X, typename R, int WAVES, int ROWS, int V, bool NT>
__global__ __launch_bounds__(64 * WAVES * ROWS) void norm_rows_kernel(NormRows a) {
  constexpr int T = 64 * WAVES;
  __shared__ float2 slots[2][WAVES];
  const int t = ROWS > 1 ? threadIdx.x & 63 : threadIdx.x;
  const int K = a.K;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x >> 6 : 0); row < a.M;
       row += (int64_t)gridDim.x * ROWS) {
    float h[V][8], g[V][8];
    const X* x = reinterpret_cast<const X*>(a.x) + row * a.x_stride;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = 8 * (v * T + t);
      if (k < K) {
        load8<NT>(x + k, h[v]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = 0.0f;
      }
    }
    if constexpr (sizeof(R) > 1) {
      const R* r = reinterpret_cast<const R*>(a.residual) + row * K;
      R* ro = reinterpret_cast<R*>(a.residual_out);
      float d[V][8];
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (8 * (v * T + t) < K) load8<NT>(r + 8 * (v * T + t), d[v]);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (8 * (v * T + t) < K) {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] += d[v][i];
          if (ro) store8<NT>(ro + row * K + 8 * (v * T + t), h[v]);
        }
    }
    float ss = 0.0f;
    uint32_t top = 0u;
    auto fold = [&]() {
      ss = 0.0f;
      top = 0u;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (8 * (v * T + t) < K) {
          if (a.gamma) {
            load8<false>(a.gamma + 8 * (v * T + t), g[v]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[v][i] = 1.0f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = __builtin_fmaf(h[v][i], h[v][i], ss);
            g[v][i] *= h[v][i];
            top = max(top, __float_as_uint(g[v][i]) & 0x7FFFFFFFu);
          }
        }
    };
    fold();
    row_sum_max<WAVES>(ss, top, slots[0]);
    float rstd = 1.0f;
    if (a.norm) {
      if (ordinary(ss, top)) {
        rstd = 1.0f / sqrtf(ss / (float)K + a.eps);
      } else {
        uint32_t hm = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) hm = max(hm, __float_as_uint(h[v][i]) & 0x7FFFFFFFu);
        float none = 0.0f;
        row_sum_max<WAVES>(none, hm, slots[1]);
        const int e = row_exponent(hm);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] = ldexpf(h[v][i], -e);
        fold();
        row_sum_max<WAVES>(ss, top, slots[0]);
        rstd = scaled_rstd(ss, K, a.eps, e);
      }
    }
    const float s = a.norm ? (__uint_as_float(top) * rstd) / 127.0f : __uint_as_float(top) / 127.0f;
    const float rcp = 1.0f / s;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = 8 * (v * T + t);
      if (k < K) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[v][i] *= rstd;
        if (a.y) store8<NT>(reinterpret_cast<__bf16*>(a.y) + row * K + k, g[v]);
        if (a.codes) put<NT>(reinterpret_cast<v2u*>(a.codes + row * K + k), codes8(g[v], s, rcp));
      }
    }
    if (a.codes && t == 0) a.scales[row] = s;
    if constexpr (WAVES > 1) __syncthreads();  // the slots are free for the next row
  }
}

// Rows too long for registers: read once for the sum and the maximum and once more to be written, between
// them a third time where the row is scaled.
template <typename X, typename R>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormRows a) {
  constexpr int WAVES = 16, T = 1024;
  constexpr bool NT = false;   // (rows are read again)
  __shared__ float2 slots[2][WAVES];
  const int t = threadIdx.x, K = a.K;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const X* x = reinterpret_cast<const X*>(a.x) + row * a.x_stride;
    auto load_h = [&](int k, float* h) {
      load8<NT>(x + k, h);
      if constexpr (sizeof(R) > 1) {
        float d[8];
        load8<NT>(reinterpret_cast<const R*>(a.residual) + row * K + k, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += d[i];
      }
    };
    auto load_g = [&](int k, float* g) {
      if (a.gamma) {
        load8<false>(a.gamma + k, g);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = 1.0f;
      }
    };
    int e = 0;
    float ss = 0.0f;
    uint32_t top = 0u, hm = 0u;
    auto fold = [&]() {
      ss = 0.0f;
      top = 0u;
      for (int k = 8 * t; k < K; k += 8 * T) {
        float h[8], g[8];
        load_h(k, h);
        load_g(k, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          hm = max(hm, __float_as_uint(h[i]) & 0x7FFFFFFFu);
          const float v = ldexpf(h[i], -e);
          ss = __builtin_fmaf(v, v, ss);
          top = max(top, __float_as_uint(g[i] * v) & 0x7FFFFFFFu);
        }
      }
      row_sum_max<WAVES>(ss, top, slots[0]);
    };
    fold();
    float rstd = 1.0f;
    if (a.norm) {
      if (ordinary(ss, top)) {
        rstd = 1.0f / sqrtf(ss / (float)K + a.eps);
      } else {
        float none = 0.0f;
        row_sum_max<WAVES>(none, hm, slots[1]);
        e = row_exponent(hm);
        fold();
        rstd = scaled_rstd(ss, K, a.eps, e);
      }
    }
    const float s = a.norm ? (__uint_as_float(top) * rstd) / 127.0f : __uint_as_float(top) / 127.0f;
    const float rcp = 1.0f / s;
    for (int k = 8 * t; k < K; k += 8 * T) {
      float h[8], g[8];
      load_h(k, h);
      load_g(k, g);
      if constexpr (sizeof(R) > 1)   // (residual_out may be residual: these eight are read by now)
        if (a.residual_out) store8<NT>(reinterpret_cast<R*>(a.residual_out) + row * K + k, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = (g[i] * ldexpf(h[i], -e)) * rstd;
      if (a.y) store8<NT>(reinterpret_cast<__bf16*>(a.y) + row * K + k, g);
      if (a.codes) put<NT>(reinterpret_cast<v2u*>(a.codes + row * K + k), codes8(g, s, rcp));
    }
    if (a.codes && t == 0) a.scales[row] = s;
    __syncthreads();
  }
}

struct None {};   // no residual (one byte)

constexpr int kMaxGrid = 1 << 20;  // workgroups of a launch (at most 1024 threads each: < 2^32)

template <typename X, typename R, int WAVES, int ROWS, int V, bool NT>
void launch_one(const NormRows& a, hipStream_t st) {
  const int64_t groups = (a.M + (int64_t)ROWS - 1) / ROWS;
  const int grid = (int)(groups < kMaxGrid ? groups : kMaxGrid);
  hipLaunchKernelGGL((norm_rows_kernel<X, R, WAVES, ROWS, V, NT>), dim3(grid), dim3(64 * WAVES * ROWS),
                     0, st, a);
}

template <typename X, typename R, bool NT>
hipError_t launch_typed(const NormRows& a, hipStream_t st) {
  const int K = a.K;
  // A row in registers: 16 elements per thread, so that a CU has 16 waves or more (16384 x 8192 to 8 bits with
  // 32 elements 234 us, 217 with 16), 8 where that needs no second wave.
  if (K <= 512) launch_one<X, R, 1, 4, 1, NT>(a, st);
  else if (K <= 1024) launch_one<X, R, 1, 4, 2, NT>(a, st);
  else if (K <= 2048) launch_one<X, R, 4, 1, 1, NT>(a, st);
  else if (K <= 4096) launch_one<X, R, 4, 1, 2, NT>(a, st);
  else if (K <= 8192) launch_one<X, R, 8, 1, 2, NT>(a, st);
  else if (K <= 16384) launch_one<X, R, 16, 1, 2, NT>(a, st);
  else
    hipLaunchKernelGGL((norm_long_kernel<X, R>), dim3(a.M < kMaxGrid ? a.M : kMaxGrid), dim3(1024),
                       0, st, a);
  return hipGetLastError();
}

template <typename X>
hipError_t launch_residual(const NormRows& a, int residual_fp32, hipStream_t st) {
  // Past the caches where the call moves more than the last of them holds (256 MB): 16384 x 8192 in bf16 with
  // a residual to 8 bits 217 -> 212 us, to bf16 211 -> 199, 16384 x 4096 94 -> 88; the smaller 4096 x 5120 to bf16
  // would take 44 instead of 43, 1000 x 8192 16.4 instead of 14.5.
  const int64_t moved = (int64_t)a.M * a.K * ((int)sizeof(X) + (a.residual ? (residual_fp32 ? 4 : 2) : 0) +
                                              (a.residual_out ? (residual_fp32 ? 4 : 2) : 0) + (a.y ? 2 : 0) + (a.codes ? 1 : 0));
  const bool nt = moved >= (256ll << 20);
  if (!a.residual) return nt ? launch_typed<X, None, true>(a, st) : launch_typed<X, None, false>(a, st);
  if (residual_fp32) return nt ? launch_typed<X, float, true>(a, st) : launch_typed<X, float, false>(a, st);
  return nt ? launch_typed<X, __bf16, true>(a, st) : launch_typed<X, __bf16, false>(a, st);
}

}  // namespace

hipError_t launch_norm_rows(const NormRows& a, int x_fp32, int residual_fp32, hipStream_t stream) {
  return x_fp32 ? launch_residual<float>(a, residual_fp32, stream)
                : launch_residual<__bf16>(a, residual_fp32, stream);
}

}  // namespace svdq
