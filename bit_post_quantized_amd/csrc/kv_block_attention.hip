// Attention of ragged rows over the block cache held in 8 bits (svdq_serve.h has the layouts).
//
//     out[i, h] = softmax_t(sm_scale q[i, h] . K[t, h']) V[t, h'],  K = (c_k - 128) s_k, V likewise
//
// One pass over the codes with a running maximum and sum.  The query rows of one request that
// share a cached head (rows x heads / kv_heads of them) fill the columns of the matrix
// instructions, 16 to a tile, against 64 tokens at a time:
//     S^T [64 tokens x 16 rows] = codes_K [64 x D] Q^T,     O^T [D x 16] += codes_V^T [D x 64] P^T
// on v_mfma_f32_16x16x32_f16.  Codes are exact fp16; a query enters as its bf16 bits scaled by a
// power of two per row, which fp16 holds exactly down to 2^-22 of the row's largest; a weight
// enters PV as fp16 (11 bits).  A block's scale multiplies whole tiles, so it is applied to scores
// and weights and never to codes.  The K rows go to the matrix rows in such an order that a lane's
// scores are those of consecutive tokens of one row: its P is then the second product's operand as
// it stands, and 8 or 16 of its scores share one pair of scales.
//
// Two kernels.  Few rows (one or two tiles: decoding) are bound by the codes' bytes: every wave
// walks over tokens of its own, straight from memory to registers, and the waves meet at the end; the
// workgroups take equal shares of the batch's tokens.  More rows (drafts, prompts) are bound by the
// softmax's vector work: the waves share the tokens, whose codes become fp16 once, in LDS, and own their
// rows; with few workgroups the tokens are split over more of them (chunks).  Where a row's tokens went
// to several workgroups, a second launch joins their maxima, sums and outputs.
//
// Measured (kernel times).  64 requests of up to 8192 tokens, 32 heads to 8 of 128: 128 us, 5.3 TB/s of
// codes, and 4.7 for the join (139 and none with a workgroup per request and head).  1 x 10240 tokens, 32
// heads: 21 us and 4; the bytes are 15 at 5.5 TB/s.  2 x 5 rows, 32 heads to 4, before up to 131071
// tokens: 49 us and 7; the bytes are 40.  4 prompts of 475 to 1000 rows, 24 heads to 8 of 64, before up
// to 4096 tokens: 89 us, 450 TFLOP/s: a wave's tile of 16 rows x 64 tokens is 195 vector
// instructions (counted, unpacking and all else among them), 16 of them exponentials at a quarter of
// the rate, against 16 matrix ones, and the longest request's 64 tiles follow each other at 1.1 to 1.3 us.  4096 rows, 32 heads to 8 of 128,
// before 8192 tokens, the whole call: 434 us, 950 TFLOP/s.
#include "serve_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kTile = 64;         // tokens per step
constexpr int kWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;
// Weights are held 2^10 too large (the sum too, so it cancels): an fp16 weight then keeps its 11
// bits down to 2^-24 of the row's largest and something of it to 2^-34, however long the row.  The
// running maximum follows a new one only when that is 2^4 ahead, so a weight stays below 2^15.
constexpr float kShift = 10.0f, kLazy = 4.0f;

// Four codes + 128 (bytes) -> four exact fp16: a byte in the mantissa of 1024 is 1024 + c + 128.
__device__ __forceinline__ void codes4_f16(uint32_t w, v2h& lo, v2h& hi) {
  const v2h off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  lo = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off;
  hi = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off;
}

// Sixteen codes -> the operands of two matrix steps, eight codes each in order.
__device__ __forceinline__ void codes16_f16(v4u w, v8h& a, v8h& b) {
  v2h x[8];
  codes4_f16(w.x, x[0], x[1]);
  codes4_f16(w.y, x[2], x[3]);
  codes4_f16(w.z, x[4], x[5]);
  codes4_f16(w.w, x[6], x[7]);
  a = v8h{x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
  b = v8h{x[4].x, x[4].y, x[5].x, x[5].y, x[6].x, x[6].y, x[7].x, x[7].y};
}

__device__ __forceinline__ v4f mfma16(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The largest of the four lanes l % 16 + 16 {0, 1, 2, 3}, in all of them.
__device__ __forceinline__ float max_quads(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __builtin_elementwise_maximum(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_elementwise_maximum(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The IEEE maximum (a NaN stays one): the form that needs no canonical operands.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

__device__ __forceinline__ float sum_quads(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// The rows and tokens of a workgroup that takes `span` rows (row x head, head fastest) from
// group * span on.
struct Range {
  int row0, n, vrows, len, hg;
  int hidden;  // tokens behind the first row's last (a request's rows past the batch's count here)
  __device__ __forceinline__ Range(const BlockAttention& a, int b) {
    row0 = min(max(a.cu[b], 0), a.rows);
    const int end = max(a.cu[b + 1], row0);
    n = min(end, a.rows) - row0;
    hg = a.heads / a.cache.heads;
    vrows = min(n, a.max_rows) * hg;
    len = min(max(a.seq[b], 0), a.width << __builtin_ctz(a.cache.bs));
    hidden = end - row0 - 1;
  }
  // tokens that row vr sees
  __device__ __forceinline__ int limit(const BlockAttention& a, int vr) const {
    return a.causal ? min(len, max(len - hidden + vr / hg, 0)) : len;
  }
  __device__ __forceinline__ size_t out_row(const BlockAttention& a, int h, int vr) const {
    return (size_t)(row0 + vr / hg) * a.heads + h * hg + vr % hg;
  }
};

__device__ __forceinline__ long long uniform(long long x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (long long)((uint64_t)hi << 32 | lo);
}

// The batch as one row of units, units(range) to a request: the request that holds unit target(all) of
// all of them, and the units before it.  Every workgroup adds the lengths up by itself.  False: no unit
// (target < 0).
template <int THREADS, class Units, class Target>
__device__ __forceinline__ bool locate(const BlockAttention& a, Units units, Target target, int& b,
                                       long long& before, long long& all) {
  __shared__ long long sums[THREADS / 64], s_before;
  __shared__ int s_b;
  const int tid = threadIdx.x, wave = tid >> 6;
  const int each = (a.requests + THREADS - 1) / THREADS, b0 = tid * each;
  long long mine = 0;
  for (int k = 0; k < each && b0 + k < a.requests; ++k) mine += units(Range(a, b0 + k));
  long long at = wave_scan(mine);
  if ((tid & 63) == 63) sums[wave] = at;
  __syncthreads();
  at -= mine;
  all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) at += sums[w];
    all += sums[w];
  }
  all = uniform(all);
  const long long u = target(all);
  if (u < 0) return false;
  if (at <= u && u < at + mine)
    for (int k = 0;; ++k) {  // (ends: u lies in one of this thread's requests)
      const int n = units(Range(a, b0 + k));
      if (u < at + n) {
        s_b = b0 + k;
        s_before = at;
        break;
      }
      at += n;
    }
  __syncthreads();
  b = __builtin_amdgcn_readfirstlane(s_b);
  before = uniform(s_before);
  return true;
}

// 16 (SEG of 64 channels) of a query's channels per lane as fp16, scaled by a power of two that
// puts the row's largest into [2^8, 2^9); returns what turns a code product into a log2 score
// (never negative: the query takes the sign of sm_scale).
template <int SEG>
__device__ __forceinline__ float scale_query(const BlockAttention& a, float (*x)[16]) {
  float amax = 0.0f;
#pragma unroll
  for (int s = 0; s < SEG; ++s)
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = __builtin_fmaxf(amax, __builtin_fabsf(x[s][e]));
  amax = max_quads(amax);
  int e2 = (int)(__float_as_uint(amax) >> 23) - 127 - 8;
  e2 = amax == 0.0f ? 0 : max(e2, -110);
  const float down = __builtin_copysignf(__uint_as_float((uint32_t)(127 - e2) << 23), a.sm_scale);
#pragma unroll
  for (int s = 0; s < SEG; ++s)
#pragma unroll
    for (int e = 0; e < 16; ++e) x[s][e] *= down;
  return __builtin_fabsf(a.sm_scale) * kLog2e * __uint_as_float((uint32_t)(127 + e2) << 23);
}

__device__ __forceinline__ void bf16x16(const uint16_t* p0, const uint16_t* p1, float* x) {
  const v4u w0 = *reinterpret_cast<const v4u*>(p0), w1 = *reinterpret_cast<const v4u*>(p1);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = __uint_as_float(e & 1 ? w0[e >> 1] & 0xFFFF0000u : w0[e >> 1] << 16);
    x[8 + e] = __uint_as_float(e & 1 ? w1[e >> 1] & 0xFFFF0000u : w1[e >> 1] << 16);
  }
}

// The scales of a lane's two runs of tokens, and how far its row sees into each: of run g's 8
// scores sc[2 g], sc[2 g + 1] those of tokens below seen[g].
struct Runs {
  float ks[2], lv[2], ivs[2];
};

// A weight carries its block's V scale vs, and the sum takes it out again in units of 2^-unit: it holds
// weights times 2^unit / vs.  The unit is a wave's own and follows the largest scale that the wave has
// met, at most 2^20 behind; a smaller scale than 2^(unit - 80), zero among them, counts as that (its
// codes then add 127 2^-80 of the largest scale at most, and it sets no maximum that matters).  So a term
// of the sum lies between 2^-20 and 2^80 times its weight, whatever normal or subnormal numbers the
// scales are; the exponential, logarithm and reciprocal see normal numbers only.  Where a new unit would
// take a sum past 2^100 (a row of tiny scales beside one that sees the large ones), the row's maximum
// rises instead: its n weights of up to 2^14 then give less than n 2^-86 of the largest value.
constexpr int kFirstUnit = -126, kLastUnit = 126;
constexpr float kLeastScale = 0x1p-80f;
constexpr float kFullSum = 100.0f;  // log2

__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The largest of a wave's values, in every lane.
__device__ __forceinline__ uint32_t max_wave(uint32_t x) {
#define SVDQ_ROTATED(CTRL) (uint32_t) __builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false)
  x = max(x, SVDQ_ROTATED(0x121));  // within rows of 16 lanes by 1, 2, 4 and 8
  x = max(x, SVDQ_ROTATED(0x122));
  x = max(x, SVDQ_ROTATED(0x124));
  x = max(x, SVDQ_ROTATED(0x128));
#undef SVDQ_ROTATED
  const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  x = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

// A unit, with what goes by it ready (each is worth several scalar instructions per tile otherwise).
struct Unit {
  int e;
  float power;         // 2^e
  uint32_t low, span;  // the normal numbers from 2^(e - 80) to 2^(e + 20)
  __device__ __forceinline__ explicit Unit(int unit)
      : e(unit), power(power2(unit)), low((uint32_t)(max(unit - 80, -126) + 127) << 23),
        span(((uint32_t)(min(unit + 20, 127) + 127) << 23) - low) {}
};

// What a lane's V scale is to weights (log2) and to the sum.
struct VScale {
  float log2, inverse;
};

// ... where every scale of the wave is near the unit,
__device__ __forceinline__ bool all_near(float vs, const Unit& unit) {
  return __all(__float_as_uint(vs) - unit.low < unit.span);
}

__device__ __forceinline__ VScale near_scale(float vs, const Unit& unit) {
  return VScale{__builtin_amdgcn_logf(vs), __builtin_amdgcn_rcpf(vs) * unit.power};
}

// ... and of any scale, after the unit has followed the wave's.
__device__ __forceinline__ VScale any_scale(float vs, Unit& unit) {
  const uint32_t bits = __float_as_uint(vs);
  const int top = (int)(__builtin_amdgcn_readfirstlane(max_wave(bits < 0x7F800000u ? bits : 0u)) >> 23) - 127;
  unit = Unit(top >= unit.e + 20 ? min(top, kLastUnit) : unit.e);
  const float in_units = __builtin_elementwise_maximum(vs * power2(-unit.e), kLeastScale);  // (NaN stays one)
  // (the inverse is a number where the scale is not: it is multiplied by the weights of rows that do not
  // see the block, which are 0)
  return VScale{__builtin_amdgcn_logf(in_units) + (float)unit.e,
                __builtin_amdgcn_rcpf(__builtin_fmaxf(in_units, kLeastScale))};
}

// How far a sum goes past 2^100 where its maximum is 2^x times the whole's and its unit `up` below the
// whole's, and the sum on the whole's terms.  (The two go together: a scale that raises the unit raises
// the maximum too, where its score is not far behind.)
__device__ __forceinline__ float over_full(float l, float x, float up) {
  return x + up + (float)((int)(__float_as_uint(l) >> 23) - 127) - kFullSum;
}
__device__ __forceinline__ float sum_on(float l, float x, float up) {
  return l * __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(x + up, 126.0f));  // (0 stays 0)
}

// One softmax step of RT tiles of rows: the lane's 16 code products of each become weights (pf, the
// second product's operand), and m, l, o follow.  A weight is 2^(score + log2 vs), so the codes of V
// stay codes.  The sums' unit rises by `up` (uniform).  The tiles of rows go through it together, with
// one branch for all: each is a chain of dependent operations, and two chains fill each other's gaps.
template <int RT, int DT>
__device__ __forceinline__ void softmax_step(v4f (*sc)[4], const float* fac, const Runs& r, int up, bool masked,
                                             const int (*seen)[2], float* m, float* l, v4f (*o)[DT],
                                             v8h (*pf)[2]) {
  float f[RT][2], add[2] = {r.lv[0], r.lv[1]}, mx[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    f[q][0] = fac[q] * r.ks[0];
    f[q][1] = fac[q] * r.ks[1];
  }
  if (masked) {  // (uniform) the products become scores here
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      float x = -__builtin_inff();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = __builtin_fmaf(sc[q][t][i], f[q][t >> 1], add[t >> 1]);
          sc[q][t][i] = 4 * (t & 1) + i < seen[q][t >> 1] ? y : -__builtin_inff();
        }
        x = max3(max3(x, sc[q][t][0], sc[q][t][1]), sc[q][t][2], sc[q][t][3]);
      }
      mx[q] = x;
      f[q][0] = f[q][1] = 1.0f;
    }
    add[0] = add[1] = 0.0f;
  } else {
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      float x[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const v4f a = sc[q][2 * g], b = sc[q][2 * g + 1];
        x[g] = max3(max3(__builtin_elementwise_maximum(a[0], a[1]), a[2], a[3]), b[0], b[1]);
        x[g] = max3(x[g], b[2], b[3]);
        x[g] = __builtin_fmaf(x[g], f[q][g], add[g]);
      }
      mx[q] = __builtin_elementwise_maximum(x[0], x[1]);
    }
  }
  bool ahead = false;
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    mx[q] = max_quads(mx[q]);
    ahead = ahead || mx[q] > m[q] + kLazy;
  }
  if (__any(ahead) || up) {
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      float mn = __builtin_fmaxf(m[q], mx[q]), x = mn == -__builtin_inff() ? 0.0f : m[q] - mn;
      if (__builtin_expect(up, 0)) {
        const float over = __builtin_fmaxf(over_full(max_quads(l[q]), x, up), 0.0f);
        mn += over;
        x -= over;
      }
      const float alpha = __builtin_amdgcn_exp2f(x);
      m[q] = mn;
      l[q] = sum_on(l[q], x, up);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[q][d][i] *= alpha;
    }
  }
  float c[RT][2], sum[RT][2];
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      c[q][g] = add[g] + kShift - (m[q] == -__builtin_inff() ? 0.0f : m[q]);
      sum[q][g] = 0.0f;
    }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int i = 0; i < 4; i += 2)
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const float f0 = f[q][t >> 1], c0 = c[q][t >> 1];
        const v2f x = {__builtin_amdgcn_exp2f(__builtin_fmaf(sc[q][t][i], f0, c0)),
                       __builtin_amdgcn_exp2f(__builtin_fmaf(sc[q][t][i + 1], f0, c0))};
        sum[q][t >> 1] += x.x + x.y;  // (in fp32: a run of small V scale counts in the sum all the same)
        const v2h p = __builtin_convertvector(x, v2h);
        pf[q][t >> 1][4 * (t & 1) + i] = p.x;
        pf[q][t >> 1][4 * (t & 1) + i + 1] = p.y;
      }
#pragma unroll
  for (int q = 0; q < RT; ++q)
    l[q] = __builtin_fmaf(sum[q][1], r.ivs[1], __builtin_fmaf(sum[q][0], r.ivs[0], l[q]));
}

// ------------------------------------------------------------------------------------ few rows
// RT tiles of 16 rows.  A wave's lane (c = l % 16, j = l / 16) scores tokens 16 j .. + 15 of its
// tile for row c: K's row of matrix row 4 j' + i of product t is token 16 j' + 4 t + i.  The next
// tile's codes are in flight while this one's are used.
//
// shares = 0: a workgroup has one request's cached head.  Otherwise the batch's tokens, in units of
// kUnit, are one row per cached head, and a workgroup takes an equal share of it: the end of one
// request, some whole ones, the beginning of another.  Each workgroup adds up the units itself, from the
// lengths.  What it has of a request is a segment, kept in the workspace unless that is all of it; segment
// (share w, request b) is number w + b of its head, since one of the two grows from each to the next.
// The request's first and the number of its segments go to the workspace's beginning.
constexpr int kUnit = kWaves * kTile;

__device__ __forceinline__ int units_of(const BlockAttention& a, const Range& rg) {
  return rg.vrows == 0 ? 0 : max(1, (rg.limit(a, rg.vrows - 1) + kUnit - 1) / kUnit);
}

__host__ __device__ inline size_t table_floats(int requests) { return ((size_t)requests * 2 + 3) / 4 * 4; }

template <int D, int RT>
__global__ __launch_bounds__(kWaves * 64, 2) void kv_block_attention_kernel(BlockAttention a, int shares,
                                                                            int seg_rows) {
  constexpr int SEG = D / 64, DT = D / 16;
  __shared__ float o_lds[kWaves][16][D + 4];
  __shared__ float m_lds[kWaves][16], l_lds[kWaves][16], unit_lds[kWaves][16], f_lds[kWaves][16], up_lds[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, j = lane >> 4;
  const int KV = a.cache.heads, shift = __builtin_ctz(a.cache.bs);
  const int h = blockIdx.x % KV, share = blockIdx.x / KV;
  int b = share;
  long long before = 0, u0 = 0, u1 = 0, all = 0;  // units before request b, of this share, of the batch
  if (shares &&
      !locate<kWaves * 64>(
          a, [&](const Range& rg) { return units_of(a, rg); },
          [&](long long all) {
            if (shares > all) shares = (int)all;  // (so that none is empty)
            if (share >= shares) return -1ll;
            u1 = all * (share + 1) / shares;
            return u0 = all * share / shares;
          },
          b, before, all))
    return;

  auto segment = [&](const Range& rg, int t0, int t1, float* seg) {
    const int32_t* table = a.tables + (size_t)b * a.width;

    // the table's entries for this lane's K rows (16 tokens from base + 16 (c / 4)) and for its 16
    // scores and V columns (from base + 16 j); they are looked at one step later, so that the loads
    // stay in flight meanwhile
    struct Pages {
      int k, v;
    };
    auto load_pages = [&](int base) {
      return Pages{table[min(base + 16 * (c >> 2), t1 - 1) >> shift], table[min(base + 16 * j, t1 - 1) >> shift]};
    };
    struct Codes {
      v4u k[4][SEG], v[DT];
      float ks, vs;
      bool there;  // this lane's 16 tokens
    };
    const int mask = a.cache.bs - 1;
    auto load_codes = [&](int base, Pages p, Codes& w) {
      // a block of no token, or outside the pool, is read as block 0 and left out
      const bool k_there = base + 16 * (c >> 2) < t1 && (unsigned)p.k < (unsigned)a.cache.num_blocks;
      w.there = base + 16 * j < t1 && (unsigned)p.v < (unsigned)a.cache.num_blocks;
      p.k = k_there ? p.k : 0;
      p.v = w.there ? p.v : 0;
      const size_t bk = (size_t)p.k * KV + h, bv = (size_t)p.v * KV + h;
      const int tk = (base + 16 * (c >> 2)) & mask, tv = (base + 16 * j) & mask;
      const uint8_t* kp = a.cache.k_codes + (bk * a.cache.bs + tk + (c & 3)) * D + 16 * j;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int s = 0; s < SEG; ++s) w.k[t][s] = *reinterpret_cast<const v4u*>(kp + 4 * t * D + 64 * s);
      const uint8_t* vp = a.cache.v_codes + (bv * D + c) * a.cache.bs + tv;
#pragma unroll
      for (int d = 0; d < DT; ++d) w.v[d] = *reinterpret_cast<const v4u*>(vp + (size_t)16 * d * a.cache.bs);
      w.ks = a.cache.k_scale[bv];
      w.vs = a.cache.v_scale[bv];
    };

    v8h qf[RT][SEG][2];
    float fac[RT], m[RT], l[RT];
    int limit[RT];
    v4f o[RT][DT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int vr = min(16 * t + c, rg.vrows - 1);
      limit[t] = rg.limit(a, vr);
      const uint16_t* qp = a.q + (size_t)(rg.row0 + vr / rg.hg) * a.q_stride + (size_t)(h * rg.hg + vr % rg.hg) * D + 16 * j;
      float x[SEG][16];
#pragma unroll
      for (int s = 0; s < SEG; ++s) bf16x16(qp + 64 * s, qp + 64 * s + 8, x[s]);
      fac[t] = scale_query<SEG>(a, x);
#pragma unroll
      for (int s = 0; s < SEG; ++s)
#pragma unroll
        for (int e = 0; e < 16; ++e) qf[t][s][e >> 3][e & 7] = (_Float16)x[s][e];
      m[t] = -__builtin_inff();
      l[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[t][d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }

    constexpr int STEP = kUnit;
    Unit unit(kFirstUnit);
    auto step = [&](int base, const Codes& w) {
      v4f sc[RT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        v8h ka[SEG][2];
#pragma unroll
        for (int s = 0; s < SEG; ++s) codes16_f16(w.k[t][s], ka[s][0], ka[s][1]);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int s = 0; s < SEG; ++s) {
            x = mfma16(ka[s][0], qf[q][s][0], x);
            x = mfma16(ka[s][1], qf[q][s][1], x);
          }
          sc[q][t] = x;
        }
      }
      Runs r;  // (here: the scales are the last loads of a tile)
      const int was = unit.e;
      const float x = w.there ? w.vs : unit.power;
      VScale vs = near_scale(x, unit);
      if (__builtin_expect(!all_near(x, unit), 0)) vs = any_scale(x, unit);
      r.ks[0] = r.ks[1] = w.there ? w.ks : 0.0f;
      r.lv[0] = r.lv[1] = vs.log2;
      r.ivs[0] = r.ivs[1] = vs.inverse;
      v8h pf[RT][2];
      int seen[RT][2];
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const int n = w.there ? limit[q] - (base + 16 * j) : 0;  // of this lane's 16 tokens
        seen[q][0] = n;
        seen[q][1] = n - 8;
      }
      softmax_step<RT, DT>(sc, fac, r, unit.e - was, true, seen, m, l, o, pf);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        v8h va, vb;
        codes16_f16(w.v[d], va, vb);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          o[q][d] = mfma16(va, pf[q][0], o[q][d]);
          o[q][d] = mfma16(vb, pf[q][1], o[q][d]);
        }
      }
    };
    int base = t0 + wave * kTile;
    if (base < t1) {
      // pages two steps ahead, codes one (past the last tile block 0 is read, unused)
      Pages p = load_pages(base);
      Codes wa, wb;
      load_codes(base, p, wa);
      p = load_pages(base + STEP);
      for (;;) {
        load_codes(base + STEP, p, wb);
        p = load_pages(base + 2 * STEP);
        step(base, wa);
        base += STEP;
        if (base >= t1) break;
        load_codes(base + STEP, p, wa);
        p = load_pages(base + 2 * STEP);
        step(base, wb);
        base += STEP;
        if (base >= t1) break;
      }
    }

    // ---- the waves meet, one tile of 16 rows after the other.  The first wave, a lane to each wave's row,
    // turns their maxima, units and sums into factors of their outputs (a wave that saw no token of a
    // row has maximum -inf and the least unit).
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const float ls = sum_quads(l[q]);
      __syncthreads();
      if (j == 0) {
        m_lds[wave][c] = m[q];
        l_lds[wave][c] = ls;
        unit_lds[wave][c] = m[q] == -__builtin_inff() ? kFirstUnit : unit.e;
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<v4f*>(&o_lds[wave][c][16 * d + 4 * j]) = o[q][d];
      __syncthreads();
      if (wave == 0) {
        const float mw = m_lds[j][c], uw = unit_lds[j][c], lw = l_lds[j][c];
        const float mm = max_quads(mw), top = max_quads(uw), off = mm == -__builtin_inff() ? 0.0f : mm;
        const float over = max_quads(__builtin_fmaxf(over_full(lw, mw - off, top - uw), 0.0f));
        const float x = mw - off - over, sum = sum_quads(sum_on(lw, x, top - uw));
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        // (the outputs' last factor, 2^top, goes by itself: both may be far from 1)
        f_lds[j][c] = __builtin_amdgcn_exp2f(x) * (seg ? 1.0f : inv);
        if (j == 0) {
          up_lds[c] = power2((int)top);
          if (seg && 16 * q + c < rg.vrows)
            *reinterpret_cast<v4f*>(seg + (size_t)(16 * q + c) * (D + 4)) = v4f{mm + over, sum, top, 0.0f};
        }
      }
      __syncthreads();
      for (int e = threadIdx.x; e < 16 * D; e += kWaves * 64) {
        const int row = e / D, d = e % D, vr = 16 * q + row;
        if (vr >= rg.vrows) continue;
        float out = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) out = __builtin_fmaf(o_lds[w][row][d], f_lds[w][row], out);
        if (seg) seg[(size_t)vr * (D + 4) + 4 + d] = out;
        else a.out[rg.out_row(a, h, vr) * D + d] = float_to_bf16_bits(out * up_lds[row]);
      }
    }
  };
  if (!shares) {
    const Range rg(a, b);
    if (rg.vrows > 0) segment(rg, 0, rg.limit(a, rg.vrows - 1), nullptr);
    return;
  }
  float* const segs = a.ws + table_floats(a.requests) + (size_t)h * (gridDim.x / KV + a.requests) * seg_rows * (D + 4);
  for (; before < u1; ++b) {
    const Range rg(a, b);
    const int n = units_of(a, rg);
    if (n == 0) continue;
    const int s0 = (int)max(u0 - before, 0ll), s1 = (int)min(u1 - before, (long long)n);
    if (s0 == 0 && h == 0 && threadIdx.x == 0) {
      int32_t* const info = reinterpret_cast<int32_t*>(a.ws) + 2 * (size_t)b;
      info[0] = share;
      info[1] = (int)(((before + n) * shares - 1) / all) - share + 1;
    }
    segment(rg, s0 * kUnit, min(s1 * kUnit, rg.limit(a, rg.vrows - 1)),
            s1 - s0 == n ? nullptr : segs + (size_t)(share + b) * seg_rows * (D + 4));
    before += n;
  }
}

// ----------------------------------------------------------------------------------- more rows
// A workgroup takes 16 RT rows per wave and walks over its tokens with them, 64 at a time.
// Their codes come a tile or two ahead, 16 bytes per thread and load, and become fp16 in LDS: for eight
// waves a tile ahead (double buffered, one barrier per tile: 80 against 88 us for 4096 rows of 12 heads of
// 64), for four in one buffer, whose two barriers cost less than more workgroups on the CU gain (66
// against 71 us for 2 x 5 rows of 32 heads of 128 before 131071 tokens, 95 against 109 for 64 x 34 rows
// of 12 heads of 64 before 4096).  K lies there as [token][D], V as [channel][token], the 16-byte slots
// of both permuted within the row so that the 16 lanes which read a matrix operand, or write 16
// pieces, meet 16 different bank groups.  Lane (c, j) scores tokens 32 g + 8 j .. + 7 (g = 0, 1) for
// row c: K's row of matrix row 4 j' + i of product t = 2 g + e is token 32 g + 8 j' + 4 e + i.
template <int D>
struct TileLds {
  uint16_t k[kTile][D];
  uint16_t v[D][kTile];
};

template <int D>
__device__ __forceinline__ int k_slot(int token, int slot) {
  return D == 64 ? slot ^ ((token >> 3 & 3) * 2 | (token >> 1 & 1)) : slot ^ ((token >> 3 & 3) * 4 | (token & 3));
}

__device__ __forceinline__ int v_slot(int d, int slot) { return slot ^ (d >> 1 & 7); }

template <int D, int RT, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 512 / (WAVES * 64)) void kv_block_attention_rows_kernel(
    BlockAttention a, int chunks, int groups, int chunk_tokens) {
  constexpr int DT = D / 16, STEPS = D / 32, THREADS = 64 * WAVES, ITEMS = 8 * D / THREADS;
  constexpr int BUFS = WAVES == 8 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) TileLds<D> lds[BUFS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, j = lane >> 4;
  const int KV = a.cache.heads, shift = __builtin_ctz(a.cache.bs);
  // From the linear id: cached head fastest (the workgroups of one run of blocks read neighbouring memory,
  // and with 8 heads an XCD keeps to one), then the rows, those that see most tokens first, then the
  // request and its chunk of tokens, only those that there are.  (Chunks without tokens between the others
  // leave their places in the order of CUs empty: 326 us against 148 for 64 requests of 5 rows and 4096
  // tokens with one of four chunks alive.)
  constexpr int ROWS = 16 * RT * WAVES;
  unsigned id = blockIdx.x;
  const int h = id % KV;
  id /= KV;
  const int vr0 = (groups - 1 - (int)(id % groups)) * ROWS;
  int b = id / groups, chunk = 0;
  if (chunks > 1) {
    long long before = 0, all = 0;
    const int item = b;
    if (!locate<THREADS>(
            a,
            [&](const Range& rg) {
              return rg.vrows == 0 ? 0 : min(max(1, (rg.limit(a, rg.vrows - 1) + chunk_tokens - 1) / chunk_tokens), chunks);
            },
            [&](long long all) { return item < all ? (long long)item : -1ll; }, b, before, all))
      return;
    chunk = item - (int)before;
  }
  const Range rg(a, b);
  if (vr0 >= rg.vrows) return;
  const int top = rg.limit(a, min(vr0 + ROWS, rg.vrows) - 1);
  const int t0 = chunk * chunk_tokens, t1 = min(t0 + chunk_tokens, top);
  if (chunks > 1 && t0 >= t1) return;
  const int32_t* table = a.tables + (size_t)b * a.width;

  // The four 16-token parts of a tile: lane l holds the table's entry for part l % 4 and the part's
  // scales; readlane makes them uniform where they are used.  The entry is looked at one step
  // later, so that the load stays in flight meanwhile; -1: a block of no token, or outside the pool.
  auto load_page = [&](int base) {
    const uint32_t at = (uint32_t)(max(min(base + 16 * (lane & 3), t1 - 1), 0) >> shift);
    return *reinterpret_cast<const int32_t*>(reinterpret_cast<const char*>(table) + 4u * at);
  };
  auto checked = [&](int base, int page) {
    return base + 16 * (lane & 3) < t1 && (unsigned)page < (unsigned)a.cache.num_blocks ? page : -1;
  };
  struct Parts {
    int page;
    float ks, vs;
  };
  auto load_parts = [&](int page) {  // (a cache has at most 2^30 scales, so 32 bits hold their offsets)
    const uint32_t at = 4u * ((uint32_t)max(page, 0) * KV + h);
    return Parts{page, *reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.cache.k_scale) + at),
                 *reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.cache.v_scale) + at)};
  };
  // this lane's runs of a tile, tokens 32 g + 8 j .. + 7, lie in part 2 g + j / 2
  struct Tile {
    Runs r;
    uint32_t there;  // bit k: part k is there (uniform)
    float vs;        // of part l % 4
    int unit;        // that r goes by, where all scales are near it (uniform)
  };
  Unit unit(kFirstUnit);  // of this wave's sums
  auto spread = [&](const VScale& vs, Runs& r) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      r.lv[g] = __shfl(vs.log2, 2 * g + (j >> 1));
      r.ivs[g] = __shfl(vs.inverse, 2 * g + (j >> 1));
    }
  };
  auto tile_of = [&](const Parts& p) {
    const bool there = p.page >= 0;
    const float ks = there ? p.ks : 0.0f;
    Tile t;
    t.there = (uint32_t)__ballot(there) & 15u;
    t.vs = there ? p.vs : unit.power;
    t.unit = all_near(t.vs, unit) ? unit.e : kFirstUnit - 1;
    spread(near_scale(t.vs, unit), t.r);
#pragma unroll
    for (int g = 0; g < 2; ++g) t.r.ks[g] = __shfl(ks, 2 * g + (j >> 1));
    return t;
  };
  // A tile's codes are 4 D pieces of 16 bytes each for K and V, ITEMS of them to a thread.  K: a
  // wave takes 16 tokens or fewer of one part, so the block is uniform; V: a thread takes 16 tokens
  // of one channel in part tid % 4, the one whose table entry its lane holds.
  struct Codes {
    v4u x[ITEMS];
  };
  const int mask = a.cache.bs - 1;
  const uint32_t block_bytes = (uint32_t)KV * a.cache.bs * D;
  auto is_k = [&](int i) { return ITEMS == 1 ? wave < WAVES / 2 : i < ITEMS / 2; };
  auto piece = [&](int i) { return tid + THREADS * i - (is_k(i) ? 0 : 4 * D); };
  uint32_t off[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int x = piece(i), token = x / (D / 16);
    off[i] = (uint32_t)h * a.cache.bs * D +
             (is_k(i) ? (token & mask) * D + 16 * (x % (D / 16)) : x / 4 * a.cache.bs + (16 * (x & 3) & mask));
  }
  auto load_codes = [&](int base, int pages, Codes& w) {
    const int in = base & mask;  // (a tile begins inside a block of 128 only)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int part = ((wave * 64 + THREADS * i) / (D / 16) >> 4) & 3;
      const uint32_t uniform = (uint32_t)max(__builtin_amdgcn_readlane(pages, part), 0);
      const uint32_t page = is_k(i) ? uniform : (uint32_t)max(pages, 0);
      const uint8_t* codes = is_k(i) ? a.cache.k_codes + in * D : a.cache.v_codes + in;
      w.x[i] = *reinterpret_cast<const v4u*>(codes + (uint64_t)page * block_bytes + off[i]);
    }
  };
  auto store_codes = [&](const Codes& w, TileLds<D>& to) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int x = piece(i), token = x / (D / 16), col = x % (D / 16);
      v8h lo, hi;
      codes16_f16(w.x[i], lo, hi);
      uint16_t* at = is_k(i) ? &to.k[token][8 * k_slot<D>(token, 2 * col)] : &to.v[x / 4][8 * v_slot(x / 4, 2 * (x & 3))];
      uint16_t* next = is_k(i) ? &to.k[token][8 * k_slot<D>(token, 2 * col + 1)] : &to.v[x / 4][8 * v_slot(x / 4, 2 * (x & 3) + 1)];
      *reinterpret_cast<v8h*>(at) = lo;
      *reinterpret_cast<v8h*>(next) = hi;
    }
  };

  v8h qf[RT][STEPS];
  float fac[RT], m[RT], l[RT];
  int limit[RT];
  v4f o[RT][DT];
  const int first = vr0 + 16 * RT * wave;
  // what the wave's first and last row see (a wave without rows only helps to load)
  const int low = rg.limit(a, min(first, rg.vrows - 1));
  const int high = first < rg.vrows ? rg.limit(a, min(first + 16 * RT, rg.vrows) - 1) : 0;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int vr = min(first + 16 * t + c, rg.vrows - 1);
    limit[t] = rg.limit(a, vr);
    const uint16_t* qp = a.q + (size_t)(rg.row0 + vr / rg.hg) * a.q_stride + (size_t)(h * rg.hg + vr % rg.hg) * D + 8 * j;
    float x[STEPS / 2][16];
#pragma unroll
    for (int s = 0; s < STEPS / 2; ++s) bf16x16(qp + 64 * s, qp + 64 * s + 32, x[s]);
    fac[t] = scale_query<STEPS / 2>(a, x);
#pragma unroll
    for (int s = 0; s < STEPS / 2; ++s)
#pragma unroll
      for (int e = 0; e < 16; ++e) qf[t][2 * s + (e >> 3)][e & 7] = (_Float16)x[s][e];
    m[t] = -__builtin_inff();
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[t][d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // K's slot of step s is the same for every token of this lane's matrix row
  const int token0 = 8 * (c >> 2) + (c & 3);
  int k_at[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) k_at[s] = token0 * D + 8 * k_slot<D>(token0, 4 * s + j);
  const int va_at = c * kTile + 8 * v_slot(c, j), vb_at = c * kTile + 8 * v_slot(c, 4 + j);
  auto products = [&](int base, Tile& tl, const TileLds<D>& in) {
    const int was = unit.e;
    if (__builtin_expect(tl.unit != was, 0)) spread(any_scale(tl.vs, unit), tl.r);
    v4f sc[RT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const v8h ka = *reinterpret_cast<const v8h*>(&in.k[0][0] + k_at[s] + (32 * (t >> 1) + 4 * (t & 1)) * D);
#pragma unroll
        for (int q = 0; q < RT; ++q) sc[q][t] = mfma16(ka, qf[q][s], s ? sc[q][t] : v4f{0.0f, 0.0f, 0.0f, 0.0f});
      }
    }
    const bool masked = tl.there != 15u || base + kTile > low;  // (uniform)
    v8h pf[RT][2];
    int seen[RT][2];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const int n = limit[q] - (base + 8 * j);
      seen[q][0] = tl.there >> (j >> 1) & 1 ? n : 0;
      seen[q][1] = tl.there >> (2 + (j >> 1)) & 1 ? n - 32 : 0;
    }
    softmax_step<RT, DT>(sc, fac, tl.r, unit.e - was, masked, seen, m, l, o, pf);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const v8h va = *reinterpret_cast<const v8h*>(&in.v[16 * d][0] + va_at);
      const v8h vb = *reinterpret_cast<const v8h*>(&in.v[16 * d][0] + vb_at);
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        o[q][d] = mfma16(va, pf[q][0], o[q][d]);
        o[q][d] = mfma16(vb, pf[q][1], o[q][d]);
      }
    }
  };
  auto barrier = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };

  if (t0 < t1) {
    // tile by tile: pages two or three ahead, codes and scales one or two, fp16 in LDS (past the
    // last tile block 0 is read, unused)
    int page = checked(t0, load_page(t0));
    Codes w;
    load_codes(t0, page, w);
    // (loads in the loop's own order: what the loop waits for is the later of both orders)
    __builtin_amdgcn_sched_barrier(0);
    Parts p = load_parts(page);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (BUFS == 2) {
      page = checked(t0 + kTile, load_page(t0 + kTile));
      store_codes(w, lds[0]);
      Tile now = tile_of(p);
      load_codes(t0 + kTile, page, w);
      p = load_parts(page);
      page = load_page(t0 + 2 * kTile);
      barrier();
      int buf = 0;
      for (int base = t0; base < t1; base += kTile, buf ^= 1) {
        store_codes(w, lds[buf ^ 1]);
        const Parts was = p;
        page = checked(base + 2 * kTile, page);
        load_codes(base + 2 * kTile, page, w);
        p = load_parts(page);
        page = load_page(base + 3 * kTile);
        Tile next = tile_of(was);
        if (base < high) products(base, now, lds[buf]);
        now = next;
        barrier();
      }
    } else {
      page = load_page(t0 + kTile);
      for (int base = t0; base < t1; base += kTile) {
        store_codes(w, lds[0]);
        Tile now = tile_of(p);
        page = checked(base + kTile, page);
        load_codes(base + kTile, page, w);
        p = load_parts(page);
        page = load_page(base + 2 * kTile);
        barrier();
        // (a wave with products goes before those of other workgroups that still unpack codes: 4% at 4096
        // rows before 8192 tokens, 107 against 116 us for 64 x 5 rows before 4096, but 77
        // against 74 for 4 x 1024 rows; with two buffers 85 against 80 for 12 heads, so not there)
        __builtin_amdgcn_s_setprio(1);
        if (base < high) products(base, now, lds[0]);
        __builtin_amdgcn_s_setprio(0);
        barrier();
      }
    }
  }

#pragma unroll
  for (int q = 0; q < RT; ++q) {
    const int vr = first + 16 * q + c;
    const float sum = sum_quads(l[q]);
    if (vr >= rg.vrows) continue;
    const size_t at = rg.out_row(a, h, vr);
    if (chunks == 1) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum, up = unit.power;
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *reinterpret_cast<v2u*>(a.out + at * D + 16 * d + 4 * j) =
            v2u{pack2_bf16(o[q][d][0] * inv * up, o[q][d][1] * inv * up),
                pack2_bf16(o[q][d][2] * inv * up, o[q][d][3] * inv * up)};
    } else {
      float* ws = a.ws + (at * chunks + chunk) * (D + 4);
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<v4f*>(ws + 4 + 16 * d + 4 * j) = o[q][d];
      if (j == 0) *reinterpret_cast<v4f*>(ws) = v4f{m[q], sum, (float)(m[q] == -__builtin_inff() ? kFirstUnit : unit.e), 0.0f};
    }
  }
}

// --------------------------------------------------------------------------------------- join
constexpr int kJoinThreads = 256;

// How a batch is cut (split_of).
struct Cut {
  int shares, seg_rows;             // few rows: workgroups per cached head (0: not cut), rows of a segment
  int chunks, chunk_tokens, span;   // more rows: chunks of tokens, rows per workgroup
};

// The parts of row i, head h of request b, `used` of them `stride` floats apart; used < 0: its output
// is written already.
struct Parts {
  const float* first;
  size_t stride;
  int used;
};

template <int D>
__device__ __forceinline__ Parts parts_of(const BlockAttention& a, const Cut& cut, const Range& rg, int b, int i,
                                          int h) {
  const int vr = i * rg.hg + h % rg.hg;
  if (cut.shares) {
    const v2u info = reinterpret_cast<const v2u*>(a.ws)[b];
    const size_t seg = (size_t)(h / rg.hg) * (cut.shares + a.requests) + info.x + b;
    return Parts{a.ws + table_floats(a.requests) + (seg * cut.seg_rows + vr) * (D + 4),
                 (size_t)cut.seg_rows * (D + 4), info.y == 1 ? -1 : (int)info.y};
  }
  // the chunks below the tokens that the last row of its workgroup sees
  const int top = rg.limit(a, min((vr / cut.span + 1) * cut.span, rg.vrows) - 1);
  return Parts{a.ws + ((size_t)(rg.row0 + i) * a.heads + h) * cut.chunks * (D + 4), D + 4,
               min((top + cut.chunk_tokens - 1) / cut.chunk_tokens, cut.chunks)};
}

// Joins a few parts of many rows: a lane adds four channels of a (row, head), part by part.  (A
// workgroup per (row, head), as below, takes 110 us more than this for 2 chunks of 2950 rows x 24 heads.)
constexpr int kFewParts = 16;

template <int D>
__global__ __launch_bounds__(kJoinThreads) void kv_block_join_kernel(BlockAttention a, Cut cut, unsigned joins) {
  constexpr int LANES = D / 4;
  const int lane = threadIdx.x & (LANES - 1);
  unsigned id = blockIdx.x * (kJoinThreads / LANES) + threadIdx.x / LANES;
  if (id >= joins) return;
  const int h = id % a.heads;
  id /= a.heads;
  const int i = id % a.max_rows, b = id / a.max_rows;
  const Range rg(a, b);
  if (i >= rg.n) return;
  const Parts p = parts_of<D>(a, cut, rg, b, i, h);
  if (p.used < 0) return;
  float m = -__builtin_inff(), sum = 0.0f, unit = kFirstUnit;
  v4f out = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < p.used; k += 4) {
    v4f ms[4];  // maximum, sum, unit
    v4f v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // (past the last part, that again)
      const float* ws = p.first + min(k + u, p.used - 1) * p.stride;
      ms[u] = *reinterpret_cast<const v4f*>(ws);
      v[u] = *reinterpret_cast<const v4f*>(ws + 4 + 4 * lane);
    }
    float mn = m, top = unit;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      mn = __builtin_fmaxf(mn, ms[u].x);
      top = __builtin_fmaxf(top, ms[u].z);
    }
    const float off0 = mn == -__builtin_inff() ? 0.0f : mn;
    float over = __builtin_fmaxf(over_full(sum, m - off0, top - unit), 0.0f);
#pragma unroll
    for (int u = 0; u < 4; ++u) over = __builtin_fmaxf(over, over_full(ms[u].y, ms[u].x - off0, top - ms[u].z));
    mn += over;
    const float off = off0 + over, alpha = __builtin_amdgcn_exp2f(m - off);
    sum = sum_on(sum, m - off, top - unit);
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] *= alpha;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float x = k + u < p.used ? ms[u].x - off : -__builtin_inff(), f = __builtin_amdgcn_exp2f(x);
      sum += sum_on(ms[u].y, x, top - ms[u].z);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = __builtin_fmaf(v[u][e], f, out[e]);
    }
    m = mn;
    unit = top;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum, up = power2((int)unit);
  *reinterpret_cast<v2u*>(a.out + ((size_t)(rg.row0 + i) * a.heads + h) * D + 4 * lane) =
      v2u{pack2_bf16(out[0] * inv * up, out[1] * inv * up), pack2_bf16(out[2] * inv * up, out[3] * inv * up)};
}

// Joins more parts of few rows, one (row, head) per workgroup (a lane of the kernel above would add
// them one after the other).  256 threads: the parts' weights 2^(m_k - M) go through
// LDS, then a thread adds four channels of every PARTS-th one, eight loads in flight (96 chunks of
// 320 rows x heads of 128: 8.7 us with one channel to a thread).
constexpr int kMaxParts = 1024;

template <int D>
__global__ __launch_bounds__(kJoinThreads) void kv_block_combine_kernel(BlockAttention a, Cut cut) {
  constexpr int PARTS = kJoinThreads / (D / 4);
  __shared__ float f_lds[kMaxParts];
  __shared__ float red[3][kJoinThreads / 64];
  __shared__ __attribute__((aligned(16))) float o_lds[PARTS][D];
  unsigned id = blockIdx.x;
  const int h = id % a.heads;
  id /= a.heads;
  const int i = id % a.max_rows, b = id / a.max_rows;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Range rg(a, b);
  if (i >= rg.n) return;
  const Parts p = parts_of<D>(a, cut, rg, b, i, h);
  const int used = p.used;
  if (used < 0) return;
  // four parts to a thread at most: their maxima, sums and units
  float m[kMaxParts / kJoinThreads], s[kMaxParts / kJoinThreads], un[kMaxParts / kJoinThreads];
  float mm = -__builtin_inff(), top = kFirstUnit;
#pragma unroll
  for (int q = 0; q < kMaxParts / kJoinThreads; ++q) {
    const int k = tid + kJoinThreads * q;
    const v4f ms = *reinterpret_cast<const v4f*>(p.first + max(min(k, used - 1), 0) * p.stride);
    m[q] = k < used ? ms.x : -__builtin_inff();
    s[q] = k < used ? ms.y : 0.0f;
    un[q] = k < used ? ms.z : (float)kFirstUnit;
    mm = __builtin_fmaxf(mm, m[q]);
    top = __builtin_fmaxf(top, un[q]);
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    mm = __builtin_fmaxf(mm, __shfl_xor(mm, x));
    top = __builtin_fmaxf(top, __shfl_xor(top, x));
  }
  if (lane == 0) {
    red[0][wave] = mm;
    red[2][wave] = top;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 64; ++w) {
    mm = __builtin_fmaxf(mm, red[0][w]);
    top = __builtin_fmaxf(top, red[2][w]);
  }
  const float off = mm == -__builtin_inff() ? 0.0f : mm;
  float sum = 0.0f;
#pragma unroll
  for (int q = 0; q < kMaxParts / kJoinThreads; ++q) {
    const int k = tid + kJoinThreads * q;
    if (k < used) f_lds[k] = __builtin_amdgcn_exp2f(m[q] - off);
    const float up = top - un[q], over = __builtin_fmaxf(over_full(s[q], m[q] - off, up), 0.0f);
    sum += sum_on(s[q], m[q] - off - over, up);  // (as far as it counts: the sum stays finite)
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
  if (lane == 0) red[1][wave] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 64; ++w) sum += red[1][w];
  const int d = 4 * (tid % (D / 4)), part = tid / (D / 4);
  v4f out = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = part; k < used; k += 8 * PARTS) {
    v4f v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      v[u] = *reinterpret_cast<const v4f*>(p.first + min(k + u * PARTS, used - 1) * p.stride + 4 + d);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k + u * PARTS < used) {
        const float f = f_lds[k + u * PARTS];
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = __builtin_fmaf(v[u][e], f, out[e]);
      }
  }
  *reinterpret_cast<v4f*>(&o_lds[part][d]) = out;
  __syncthreads();
  if (tid < D) {
    float o = 0.0f;
#pragma unroll
    for (int q = 0; q < PARTS; ++q) o += o_lds[q][tid];
    a.out[((size_t)(rg.row0 + i) * a.heads + h) * D + tid] = float_to_bf16_bits(sum == 0.0f ? 0.0f : o / sum * power2((int)top));
  }
}

// How a batch is cut, from sizes the host knows (lengths are the device's).  The kernel is one for the
// whole call, by the most rows that any request has: one prompt among decoding requests takes them all
// through the kernel of more rows, so a program calls once for each kind.
//  - Up to 16 query rows per cached head (32 at 64 channels): the few-rows kernel; more would spill.
//    Above, a workgroup takes 64 rows, or 128 if there are more: at 64 channels in eight waves of 16 (4
//    prompts of 475..1000 rows 85 us, 97 in four of 32: more waves hide the softmax's latency), at 128
//    in four waves of 32 (13% at 4096 rows before 8192 tokens: an LDS read feeds two products).
//  - Few rows: equal shares for 256 workgroups, up to 512 where there are as many requests (one request
//    of 32768 tokens, 8 heads: 174 us uncut, 22.1 by 256, 24.1 by 512).  A join costs 5 us, so only
//    where uncut workgroups leave CUs idle for longer (1.3 us a unit; 24 requests of 2048, 8 heads: 12.4
//    us uncut, 17.5 cut), or where the table has room for a request that goes on long after the others
//    (64 requests, 8 heads, one of 16384 tokens and 200 in the others: 85 us uncut, 30 cut; 500 in all:
//    17, 22); the room must be more where the requests alone fill the chip twice.
//  - More rows: cut so that the workgroups fit the chip at once, if the tiles saved (1.2 us each) take
//    longer than the join (6 us and its bytes at 4 TB/s): 2 x 5 rows before 131071 tokens 91 us in 32
//    chunks, 60 in 96; 2 prompts of 1024 rows, 12 heads: 22.7 us uncut, 30 in two.  Up to 64 rows
//    (drafts) under a table of more than 4096 tokens: chunks of 4096, or larger ones so that there are
//    at most as many as a join of few rows takes (64 requests of 5 rows, 8 heads, one of 32768 tokens and
//    300 in the others: 603 us uncut, 101 cut; 500 in all: 20, 28).  For prompts the parts would be too
//    many bytes.
struct Split {
  bool few;
  int rt, groups;
  Cut cut;
  bool joins() const { return few ? cut.shares > 0 : cut.chunks > 1; }
};

static Split split_of(int requests, int rows, int max_rows, int heads, int kv_heads, int dim, int width, int bs) {
  Split s;
  const long long vrows = (long long)max_rows * (heads / kv_heads);
  s.few = vrows <= (dim == 64 ? 32 : 16);
  s.rt = s.few ? (vrows > 16 ? 2 : 1) : (vrows > 64 ? 2 : 1);
  s.cut = Cut{0, s.few ? (int)vrows : 0, 1, 0, (s.few ? 16 : 64) * s.rt};
  s.groups = (int)((vrows + s.cut.span - 1) / s.cut.span);
  const long long natural = (long long)requests * kv_heads * s.groups;
  const long long tokens = (long long)width * bs;
  const long long uneven = natural < 1024 ? 4096 : 16384;  // of more tokens one request may outlast the others
  if (s.few) {
    const long long units = (tokens + kUnit - 1) / kUnit, idle = natural < 256 ? 256 - natural : 0;
    const bool cut = tokens > uneven || units * idle * 1300 > 256 * 6000;  // ns
    if (cut && requests <= 4096 && natural <= 16384) {
      const int least = 256 / kv_heads, most = 512 / kv_heads;
      const int shares = requests < least ? least : requests < most ? requests : most;
      s.cut.shares = shares > 1 ? shares : 1;
    }
    return s;
  }
  const int unit = 4 * kTile;
  long long chunks = (s.rt == 1 ? 768 : 512) / natural;
  const long long most = (tokens + unit - 1) / unit;
  if (chunks > most) chunks = most;
  if (chunks > kMaxParts) chunks = kMaxParts;
  const long long room = s.rt == 1 && tokens > uneven ? 8192 / natural : 1, capped = (tokens + 4095) / 4096;
  long long least = capped < room ? capped : room;
  if (least > kMaxParts) least = kMaxParts;  // (then a chunk has more tokens)
  if (chunks < least) {
    chunks = least;
  } else if (chunks > 1) {
    long long joins = (long long)requests * max_rows;
    joins = (joins < rows ? joins : rows) * heads;
    const long long saved = tokens / kTile * (chunks - 1) / chunks * 1200;  // ns
    if (saved < 6000 + joins * chunks * (dim + 4) * 8 / 4000) chunks = 1;
  }
  if (chunks < 1 || requests > 4096) chunks = 1;
  long long per = (tokens + chunks - 1) / chunks;
  per = (per + unit - 1) / unit * unit;
  s.cut.chunk_tokens = (int)per;
  s.cut.chunks = (int)((tokens + per - 1) / per);
  return s;
}

// A launch has fewer than 2^32 threads: with 512 to a workgroup there is room for 2^23.  (What is cut
// has fewer workgroups than that, and fewer joins.)
bool kv_block_attention_fits(int requests, int max_rows, int heads, int kv_heads, int dim) {
  const long long groups = split_of(1, 0, max_rows, heads, kv_heads, dim, 1, 16).groups;
  return requests * groups * kv_heads < 1 << 23;
}

size_t kv_block_attention_ws_bytes(int requests, int rows, int max_rows, int heads, int kv_heads,
                                   int dim, int width, int bs) {
  if (requests <= 0 || rows <= 0) return 0;
  const Split s = split_of(requests, rows, max_rows, heads, kv_heads, dim, width, bs);
  if (!s.joins()) return 0;
  const size_t parts = s.few ? (size_t)kv_heads * (s.cut.shares + requests) * s.cut.seg_rows
                             : (size_t)rows * heads * s.cut.chunks;
  return (parts * (dim + 4) + (s.few ? table_floats(requests) : 0)) * sizeof(float);
}

template <int D>
static hipError_t launch(const BlockAttention& a, hipStream_t stream) {
  const Split s = split_of(a.requests, a.rows, a.max_rows, a.heads, a.cache.heads, D, a.width, a.cache.bs);
  const dim3 few((unsigned)a.cache.heads * (s.cut.shares ? s.cut.shares : a.requests));
  const dim3 more((unsigned)(a.requests * s.groups * s.cut.chunks * a.cache.heads));
#define SVDQ_ATTEND(GRID, WAVES, KERNEL, ...) \
  hipLaunchKernelGGL(KERNEL, GRID, dim3(WAVES * 64), 0, stream, a, __VA_ARGS__)
  if (s.few && s.rt == 1) SVDQ_ATTEND(few, kWaves, (kv_block_attention_kernel<D, 1>), s.cut.shares, s.cut.seg_rows);
  else if (s.few)  // (128 channels: never)
    SVDQ_ATTEND(few, kWaves, (kv_block_attention_kernel<D, (D == 64 ? 2 : 1)>), s.cut.shares, s.cut.seg_rows);
  else if (s.rt == 1)
    SVDQ_ATTEND(more, 4, (kv_block_attention_rows_kernel<D, 1, 4>), s.cut.chunks, s.groups, s.cut.chunk_tokens);
  else if constexpr (D == 64)
    SVDQ_ATTEND(more, 8, (kv_block_attention_rows_kernel<D, 1, 8>), s.cut.chunks, s.groups, s.cut.chunk_tokens);
  else
    SVDQ_ATTEND(more, 4, (kv_block_attention_rows_kernel<D, 2, 4>), s.cut.chunks, s.groups, s.cut.chunk_tokens);
#undef SVDQ_ATTEND
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !s.joins()) return e;
  const unsigned joins = (unsigned)(a.requests * a.max_rows * a.heads);
  // Many rows have few parts each, most of them (64 requests of up to 8192 tokens x 32 heads: 130.5 us by
  // lanes, 132.5 by workgroups; with one request of 60 parts 28, 25.7).
  if ((s.few ? s.cut.shares : s.cut.chunks) <= kFewParts || joins >= 1024) {
    const unsigned each = kJoinThreads / (D / 4);
    hipLaunchKernelGGL(kv_block_join_kernel<D>, dim3((joins + each - 1) / each), dim3(kJoinThreads), 0, stream, a,
                       s.cut, joins);
  } else {
    hipLaunchKernelGGL(kv_block_combine_kernel<D>, dim3(joins), dim3(kJoinThreads), 0, stream, a, s.cut);
  }
  return hipGetLastError();
}

hipError_t launch_kv_block_attention(const BlockAttention& a, hipStream_t stream) {
  return a.cache.dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace svdq
