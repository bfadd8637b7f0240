// Rotary positions on the heads of q and k.
//
// A pair's angle is position * frequency: at position 2^20 an fp32 product is off by a sixteenth of a
// radian, so it is formed in fp64, in half turns, and its whole turns are taken off there; what is
// left, in [-1, 1] half turns, goes through fp32 sines and cosines.  They are the same for all heads
// of a row, so a workgroup computes a row's pairs once into LDS, and its threads then turn the heads:
// each takes 8 channels and, in the half layout, the 8 that they are paired with.
//
// Bound by memory: 20000 rows of 24 + 8 heads of 128 in bf16, 328 MB, in 64 us into other tensors (5.1 TB/s) and 67 in place
// (4.9) for whole heads in halves, 68 (4.8) for neighbours; half of each in place 36.5 (4.5).  64 rows take a launch's 4.
#include "decoder_launch.hpp"
#include "svdq_device.hpp"

namespace svdq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGrid = 1 << 20;  // workgroups of a launch: fewer than 2^32 threads

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    const v4f a = reinterpret_cast<const v4f*>(p)[0], b = reinterpret_cast<const v4f*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const v4u a = *reinterpret_cast<const v4u*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

template <typename X, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeRows a, int group, int per_head) {
  extern __shared__ float2 turns[];  // [group][rot / 2]: (cos, sin) times scale
  const int half = a.rot / 2, per_row = (a.heads[0] + a.heads[1]) * per_head;
  for (int64_t row0 = (int64_t)blockIdx.x * group; row0 < a.rows; row0 += (int64_t)gridDim.x * group) {
    const int rows = (int)min((int64_t)group, a.rows - row0);
    for (int i = threadIdx.x; i < rows * half; i += kThreads) {
      const int r = i / half;
      const double t = (double)a.positions[row0 + r] * (a.freqs[i - r * half] * 0.31830988618379067154);
      float sn, cs;
      sincospif((float)(t - 2.0 * rint(0.5 * t)), &sn, &cs);
      turns[i] = make_float2(cs * a.scale, sn * a.scale);
    }
    __syncthreads();
    // an item, of per_row of a row, heads of q first: 8 channels, turned or only copied, and in the half
    // layout the 8 that they are paired with; the same one of several rows at a time, all loaded first
    const int half8 = half / 8;
    for (int j = threadIdx.x; j < per_row; j += kThreads) {
      const int h = j / per_head, p = j - h * per_head;
      const int which = h >= a.heads[0];
      const int head = which ? h - a.heads[0] : h;
      const X* in = reinterpret_cast<const X*>(a.in[which]) + row0 * a.in_stride[which] + head * a.dim;
      __bf16* out = reinterpret_cast<__bf16*>(a.out[which]) + row0 * a.out_stride[which] + head * a.dim;
      // (half layout: the first of the pairs' channels, or one that is copied)
      const bool turned = INTERLEAVED ? 8 * p < a.rot : p < half8;
      const int c = INTERLEAVED || turned ? 8 * p : a.rot + 8 * (p - half8);
      constexpr int kRows = INTERLEAVED ? 4 : 2;   // (16 channels of each in the half layout)
      for (int r0 = 0; r0 < rows; r0 += kRows) {
        float u[kRows][8], v[kRows][8];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (r0 + r < rows) {
            load8(in + (r0 + r) * a.in_stride[which] + c, u[r]);
            if (!INTERLEAVED && turned) load8(in + (r0 + r) * a.in_stride[which] + c + half, v[r]);
          }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (r0 + r < rows) {
            __bf16* to = out + (r0 + r) * a.out_stride[which] + c;
            const float2* cs = turns + (r0 + r) * half + (INTERLEAVED ? 4 * p : 8 * p);
            if (INTERLEAVED && turned) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 t = cs[e];
                const float x = u[r][2 * e], y = u[r][2 * e + 1];
                u[r][2 * e] = x * t.x - y * t.y;
                u[r][2 * e + 1] = x * t.y + y * t.x;
              }
            }
            if (!INTERLEAVED && turned) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 t = cs[e];
                const float x = u[r][e], y = v[r][e];
                u[r][e] = x * t.x - y * t.y;
                v[r][e] = x * t.y + y * t.x;
              }
              *reinterpret_cast<v8bf*>(to + half) = to_bf16x8(v[r]);
            }
            *reinterpret_cast<v8bf*>(to) = to_bf16x8(u[r]);
          }
      }
    }
    __syncthreads();  // the next rows' pairs take these ones' place
  }
}

template <typename X, bool INTERLEAVED>
void launch(const RopeRows& a, hipStream_t st) {
  const int half = a.rot / 2;
  // rows of a workgroup: one while that fills the device, else as many as its threads have pairs
  int group = 1;
  while (group < 8 && 2 * group * half <= kThreads && a.rows >= 4096 * group) group *= 2;
  // (in place, the channels behind rot_dim are where they belong)
  const bool in_place = a.in[0] == a.out[0] && (a.heads[1] == 0 || a.in[1] == a.out[1]);
  const int rest = in_place ? 0 : (a.dim - a.rot) / 8, per_head = (INTERLEAVED ? a.rot / 8 : half / 8) + rest;
  hipLaunchKernelGGL((rope_kernel<X, INTERLEAVED>), dim3(min((a.rows + group - 1) / group, kMaxGrid)), dim3(kThreads),
                     group * half * sizeof(float2), st, a, group, per_head);
}

}  // namespace

hipError_t launch_rope(const RopeRows& a, int x_fp32, hipStream_t stream) {
  if (x_fp32) a.interleaved ? launch<float, true>(a, stream) : launch<float, false>(a, stream);
  else a.interleaved ? launch<__bf16, true>(a, stream) : launch<__bf16, false>(a, stream);
  return hipGetLastError();
}

}  // namespace svdq
