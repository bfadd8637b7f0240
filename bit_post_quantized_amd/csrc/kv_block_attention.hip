// Attention of ragged rows over the block cache held in 8 bits (svdq_serve.h has the layouts).
//
//     out[i, h] = softmax_t(sm_scale q[i, h] . K[t, h']) V[t, h'],  K = (c_k - 128) s_k, V likewise
//
// One pass over the codes with a running maximum and sum.  The query rows of one request that
// share a cached head (rows x heads / kv_heads of them) fill the columns of the matrix
// instructions, 16 to a tile; a wave takes 64 tokens at a time:
//     S^T [64 tokens x 16 rows] = codes_K [64 x D] Q^T,     O^T [D x 16] += codes_V^T [D x 64] P^T
// on v_mfma_f32_16x16x32_f16.  Codes are exact fp16; a query enters as its bf16 bits scaled by a
// power of two per row, which fp16 holds exactly down to 2^-22 of the row's largest; a weight
// enters PV as fp16 (11 bits).  A block's scale multiplies whole tiles, so it is applied to scores
// and weights and never to codes.  The K rows go to the matrix rows in such an order that a
// lane's 16 scores are those of 16 consecutive tokens of one row: its P is then the second
// product's operand as it stands, and it shares one block, hence one pair of scales.
//
// With few rows the tokens are split over workgroups (chunks), and kv_block_combine_kernel joins
// the chunks' maxima, sums and outputs.
#include "serve_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kTile = 64;         // tokens per wave step
constexpr int kWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;
// Weights are held 2^14 too large (the sum too, so it cancels): an fp16 weight then keeps its 11
// bits down to 2^-28 of the row's largest and something of it to 2^-38, however long the row.
constexpr float kShift = 14.0f;

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

// What one workgroup works on, from its linear id: cached head fastest (the workgroups of one
// run of blocks read neighbouring memory), then the chunk, the row group, the request.
struct Work {
  int h, chunk, group, b;
};

__device__ __forceinline__ Work work_of(int kv_heads, int chunks, int groups) {
  Work w;
  unsigned id = blockIdx.x;
  w.h = id % kv_heads;
  id /= kv_heads;
  w.chunk = id % chunks;
  id /= chunks;
  w.group = id % groups;
  w.b = id / groups;
  return w;
}

// RT tiles of 16 rows.
template <int D, int RT>
__global__ __launch_bounds__(kWaves * 64, 2) void kv_block_attention_kernel(BlockAttention a,
                                                                            int chunks, int groups,
                                                                            int chunk_tokens) {
  constexpr int SEG = D / 64, DT = D / 16;
  __shared__ float o_lds[kWaves][16][D + 4];
  __shared__ float m_lds[kWaves][16], l_lds[kWaves][16];
  const Work wk = work_of(a.cache.heads, chunks, groups);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, j = lane >> 4;
  const int KV = a.cache.heads, hg = a.heads / KV, shift = __builtin_ctz(a.cache.bs);
  const int row0 = min(max(a.cu[wk.b], 0), a.rows), row1 = min(max(a.cu[wk.b + 1], row0), a.rows);
  const int n = row1 - row0;
  const int vr0 = wk.group * 16 * RT;               // first row (row x head) of this workgroup
  const int vrows = min(n, a.max_rows) * hg;
  if (vr0 >= vrows) return;
  const int len = min(max(a.seq[wk.b], 0), a.width << shift);
  // rows in [vr0, vr0 + 16 RT) see at most `top` tokens
  const int last = min(vr0 + 16 * RT, vrows) - 1;
  const int top = a.causal ? min(len, max(len - n + last / hg + 1, 0)) : len;
  const int t0 = wk.chunk * chunk_tokens, t1 = min(t0 + chunk_tokens, top);
  if (chunks > 1 && t0 >= t1) return;               // (the combine knows which chunks there are)
  const int32_t* table = a.tables + (size_t)wk.b * a.width;

  v8h qf[RT][SEG][2];
  float fac[RT];
  int limit[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int vr = min(vr0 + 16 * t + c, vrows - 1), i = vr / hg;
    limit[t] = a.causal ? min(len, max(len - n + i + 1, 0)) : len;
    const uint16_t* qp = a.q + (size_t)(row0 + i) * a.q_stride + (size_t)(wk.h * hg + vr % hg) * D + 16 * j;
    float x[SEG][16];
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < SEG; ++s) {
      const v4u w0 = *reinterpret_cast<const v4u*>(qp + 64 * s), w1 = *reinterpret_cast<const v4u*>(qp + 64 * s + 8);
      const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[s][e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
        amax = __builtin_fmaxf(amax, __builtin_fabsf(x[s][e]));
      }
    }
    amax = __builtin_fmaxf(amax, __shfl_xor(amax, 16));
    amax = __builtin_fmaxf(amax, __shfl_xor(amax, 32));
    int e2 = (int)(__float_as_uint(amax) >> 23) - 127 - 8;  // amax 2^-e2 in [2^8, 2^9)
    e2 = amax == 0.0f ? 0 : max(e2, -110);
    const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
    fac[t] = a.sm_scale * kLog2e * __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
    for (int s = 0; s < SEG; ++s)
#pragma unroll
      for (int e = 0; e < 16; ++e) qf[t][s][e >> 3][e & 7] = (_Float16)(x[s][e] * down);
  }

  v4f o[RT][DT];
  float m[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = -__builtin_inff();
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[t][d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }

  for (int base = t0 + wave * kTile; base < t1; base += kWaves * kTile) {
    // the blocks of this lane's K rows (16 tokens from base + 16 (c / 4)) and of its 16 scores and
    // V columns (from base + 16 j); -1 where there are none
    const int tk = base + 16 * (c >> 2), tv = base + 16 * j;
    int pk = tk < t1 ? table[tk >> shift] : -1, pv = tv < t1 ? table[tv >> shift] : -1;
    if ((unsigned)pk >= (unsigned)a.cache.num_blocks) pk = -1;
    if ((unsigned)pv >= (unsigned)a.cache.num_blocks) pv = -1;
    const size_t bk = (size_t)max(pk, 0) * KV + wk.h, bv = (size_t)max(pv, 0) * KV + wk.h;
    const int mask = a.cache.bs - 1;
    v4u kw[4][SEG], vw[DT];
    const uint8_t* kp = a.cache.k_codes + (bk * a.cache.bs + (tk & mask) + (c & 3)) * D + 16 * j;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int s = 0; s < SEG; ++s) kw[t][s] = *reinterpret_cast<const v4u*>(kp + 4 * t * D + 64 * s);
    const uint8_t* vp = a.cache.v_codes + (bv * D + c) * a.cache.bs + (tv & mask);
#pragma unroll
    for (int d = 0; d < DT; ++d) vw[d] = *reinterpret_cast<const v4u*>(vp + (size_t)16 * d * a.cache.bs);
    float ks = 0.0f, vs = 1.0f;
    if (pv >= 0) {
      ks = a.cache.k_scale[bv];
      vs = a.cache.v_scale[bv];
    }
    // A weight carries its block's V scale: it is 2^(score + log2 vs), and the sum takes vs out
    // again.  A zero scale belongs to codes that are all zero, so any scale serves.
    if (vs == 0.0f) vs = 1.0f;
    const float lv = __builtin_amdgcn_logf(vs), ivs = 1.0f / vs;

    v4f sc[RT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v8h ka[SEG][2];
#pragma unroll
      for (int s = 0; s < SEG; ++s) codes16_f16(kw[t][s], ka[s][0], ka[s][1]);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < SEG; ++s) {
          x = mfma16(ka[s][0], qf[r][s][0], x);
          x = mfma16(ka[s][1], qf[r][s][1], x);
        }
        sc[r][t] = x;
      }
    }
    v8h pf[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float f = fac[r] * ks;
      const int seen = pv >= 0 ? limit[r] - tv : 0;  // of this lane's 16 tokens
      float mx = -__builtin_inff();
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = __builtin_fmaf(sc[r][t][i], f, lv);
          sc[r][t][i] = 4 * t + i < seen ? x : -__builtin_inff();
          mx = __builtin_fmaxf(mx, sc[r][t][i]);
        }
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16));
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32));
      const float mn = __builtin_fmaxf(m[r], mx);
      const float off = (mn == -__builtin_inff() ? 0.0f : mn) - kShift;
      const float alpha = __builtin_amdgcn_exp2f(m[r] - (off + kShift));
      m[r] = mn;
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(sc[r][t][i] - off);
          sum += p;
          pf[r][t >> 1][4 * (t & 1) + i] = (_Float16)p;
        }
      l[r] = __builtin_fmaf(l[r], alpha, sum * ivs);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[r][d][i] *= alpha;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      v8h va, vb;
      codes16_f16(vw[d], va, vb);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        o[r][d] = mfma16(va, pf[r][0], o[r][d]);
        o[r][d] = mfma16(vb, pf[r][1], o[r][d]);
      }
    }
  }

  // ---- the waves meet, one tile of 16 rows after the other
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float ls = l[r];
    ls += __shfl_xor(ls, 16);
    ls += __shfl_xor(ls, 32);
    __syncthreads();
    if (j == 0) {
      m_lds[wave][c] = m[r];
      l_lds[wave][c] = ls;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) *reinterpret_cast<v4f*>(&o_lds[wave][c][16 * d + 4 * j]) = o[r][d];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * D; e += kWaves * 64) {
      const int row = e / D, d = e % D, vr = vr0 + 16 * r + row;
      if (vr >= vrows) continue;
      float mm = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mm = __builtin_fmaxf(mm, m_lds[w][row]);
      const float off = mm == -__builtin_inff() ? 0.0f : mm;
      float sum = 0.0f, out = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(m_lds[w][row] - off);
        sum = __builtin_fmaf(l_lds[w][row], f, sum);
        out = __builtin_fmaf(o_lds[w][row][d], f, out);
      }
      const size_t at = (size_t)(row0 + vr / hg) * a.heads + wk.h * hg + vr % hg;
      if (chunks == 1) {
        a.out[at * D + d] = float_to_bf16_bits(sum == 0.0f ? 0.0f : out / sum);
      } else {
        float* ws = a.ws + (at * chunks + wk.chunk) * (D + 2);
        ws[2 + d] = out;
        if (d == 0) {
          ws[0] = mm;
          ws[1] = sum;
        }
      }
    }
  }
}

// Joins the chunks of one (row, head): D threads, each one channel.
template <int D>
__global__ __launch_bounds__(D) void kv_block_combine_kernel(BlockAttention a, int chunks,
                                                             int chunk_tokens, int span) {
  const int hg = a.heads / a.cache.heads, shift = __builtin_ctz(a.cache.bs);
  unsigned id = blockIdx.x;
  const int h = id % a.heads;
  id /= a.heads;
  const int i = id % a.max_rows, b = id / a.max_rows;
  const int row0 = min(max(a.cu[b], 0), a.rows), row1 = min(max(a.cu[b + 1], row0), a.rows);
  const int n = row1 - row0;
  if (i >= n) return;
  const int len = min(max(a.seq[b], 0), a.width << shift);
  // the chunks that the workgroup of this row's group wrote: those below the tokens its last row sees
  const int vrows = min(n, a.max_rows) * hg, vr = i * hg + h % hg;
  const int last = min((vr / span + 1) * span, vrows) - 1;
  const int top = a.causal ? min(len, max(len - n + last / hg + 1, 0)) : len;
  const int used = min((top + chunk_tokens - 1) / chunk_tokens, chunks);
  const size_t at = (size_t)(row0 + i) * a.heads + h;
  const float* ws = a.ws + at * chunks * (D + 2);
  float mm = -__builtin_inff();
  for (int k = 0; k < used; ++k) mm = __builtin_fmaxf(mm, ws[(size_t)k * (D + 2)]);
  const float off = mm == -__builtin_inff() ? 0.0f : mm;
  float sum = 0.0f, out = 0.0f;
  for (int k = 0; k < used; ++k) {
    const float* p = ws + (size_t)k * (D + 2);
    const float f = __builtin_amdgcn_exp2f(p[0] - off);
    sum = __builtin_fmaf(p[1], f, sum);
    out = __builtin_fmaf(p[2 + threadIdx.x], f, out);
  }
  a.out[at * D + threadIdx.x] = float_to_bf16_bits(sum == 0.0f ? 0.0f : out / sum);
}

// How a call is split, from its sizes alone.
struct Split {
  int rt, groups, chunks, chunk_tokens;
};

static Split split_of(int requests, int max_rows, int heads, int kv_heads, int width, int bs) {
  Split s;
  const long long vrows = (long long)max_rows * (heads / kv_heads);
  s.rt = vrows > 16 ? 2 : 1;
  s.groups = (int)((vrows + 16 * s.rt - 1) / (16 * s.rt));
  const long long natural = (long long)requests * kv_heads * s.groups;
  const long long tokens = (long long)width * bs;
  const long long want = (1024 + natural - 1) / natural;              // workgroups for 256 CUs
  const long long most = (tokens + kWaves * kTile - 1) / (kWaves * kTile);
  long long chunks = want < most ? want : most;
  if (chunks < 1) chunks = 1;
  long long per = (tokens + chunks - 1) / chunks;
  per = (per + kWaves * kTile - 1) / (kWaves * kTile) * (kWaves * kTile);
  s.chunk_tokens = (int)per;
  s.chunks = (int)((tokens + per - 1) / per);
  return s;
}

size_t kv_block_attention_ws_bytes(int requests, int rows, int max_rows, int heads, int kv_heads,
                                   int dim, int width, int bs) {
  if (requests <= 0 || rows <= 0) return 0;
  const Split s = split_of(requests, max_rows, heads, kv_heads, width, bs);
  return s.chunks == 1 ? 0 : (size_t)rows * heads * s.chunks * (dim + 2) * sizeof(float);
}

template <int D>
static hipError_t launch(const BlockAttention& a, hipStream_t stream) {
  const Split s = split_of(a.requests, a.max_rows, a.heads, a.cache.heads, a.width, a.cache.bs);
  const long long grid = (long long)a.requests * s.groups * s.chunks * a.cache.heads;
  const long long joins = (long long)a.requests * a.max_rows * a.heads;
  if (grid > 0x7FFFFFFFLL || (s.chunks > 1 && joins > 0x7FFFFFFFLL)) return hipErrorInvalidConfiguration;
  if (s.rt == 1)
    hipLaunchKernelGGL((kv_block_attention_kernel<D, 1>), dim3((unsigned)grid), dim3(kWaves * 64), 0, stream, a,
                       s.chunks, s.groups, s.chunk_tokens);
  else
    hipLaunchKernelGGL((kv_block_attention_kernel<D, 2>), dim3((unsigned)grid), dim3(kWaves * 64), 0, stream, a,
                       s.chunks, s.groups, s.chunk_tokens);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || s.chunks == 1) return e;
  hipLaunchKernelGGL(kv_block_combine_kernel<D>, dim3((unsigned)joins), dim3(D), 0, stream, a, s.chunks,
                     s.chunk_tokens, 16 * s.rt);
  return hipGetLastError();
}

hipError_t launch_kv_block_attention(const BlockAttention& a, hipStream_t stream) {
  return a.cache.dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace svdq
