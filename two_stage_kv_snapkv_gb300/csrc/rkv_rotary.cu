// Rotary positions of queries and keys.
//
//   y_u = s (x_u cos a - x_v sin a),  y_v = s (x_v cos a + x_u sin a),  a = position * f_i
// An angle is kept in turns as a 64-bit fraction: position * turns_i modulo 2^64 is exact, so
// a far position loses nothing, and its upper 32 bits, as a signed part of a turn, go to
// sincospif.
//
// Bound by its bytes (two read, two written a channel).  A head's 128 channels are eight
// items of 32 bytes: a pair item (8 channels of each half, or 16 neighbouring ones: eight
// angles either way) or 16 channels to copy.  A thread has one item of one token, computes its
// eight sines and cosines once and takes eight heads with them, four of them in flight.
// Measured: 16384 tokens of 32 + 8 heads (336 MB) 53.6 us, 6.3 TB/s, 93 % of a plain copy's rate;
// a step of 64 tokens 4.2 us.
#include "rkv_device.cuh"
#include "rkv_internal.h"

namespace rkv {
namespace {

constexpr int kRoThreads = 256;

struct RotaryParams {
  uint64_t turns[64];
  const rkv_bf16* in[2];  // queries, keys
  rkv_bf16* out[2];
  int64_t is[2][3], os[2][3];
  const int32_t* positions;
  int heads[2];
  int T, rot, interleaved, per_token, inverse, per;  // per: heads of a thread
  long long tokens;
  float amplitude;
};

struct Item {
  uint4 a, b;
};

__device__ __forceinline__ void rotate2(uint32_t& a, uint32_t& b, const float* c, const float* s) {
  const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  a = pack_bf16x2(a0 * c[0] - b0 * s[0], a1 * c[1] - b1 * s[1]);
  b = pack_bf16x2(b0 * c[0] + a0 * s[0], b1 * c[1] + a1 * s[1]);
}
// Neighbours: the two channels of a word are a pair.
__device__ __forceinline__ void rotate1(uint32_t& x, float c, float s) {
  const float a = bf16_lo(x), b = bf16_hi(x);
  x = pack_bf16x2(a * c - b * s, b * c + a * s);
}

__global__ void __launch_bounds__(kRoThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  const int j = threadIdx.x & 7;  // the item
  const long long tok = (long long)blockIdx.x * (kRoThreads / 8) + (threadIdx.x >> 3);
  if (tok >= p.tokens) return;
  const int b = (int)(tok / p.T), t = (int)(tok - (long long)b * p.T);
  const bool turn = j < p.rot / 16;
  float c[8], s[8];
  if (turn) {
    const int32_t pos = p.per_token ? p.positions[tok] : (int32_t)((uint32_t)p.positions[b] + (uint32_t)t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t at = (uint64_t)(int64_t)pos * p.turns[8 * j + i];
      sincospif((float)(int32_t)(at >> 32) * 4.656612873077393e-10f, &s[i], &c[i]);  // 2^-31: half turns
      c[i] *= p.amplitude;
      s[i] *= p.inverse ? -p.amplitude : p.amplitude;
    }
  }
  // the item's two 16-byte pieces
  const bool halves = turn && !p.interleaved;
  const int at_a = halves ? 8 * j : 16 * j, at_b = halves ? p.rot / 2 + 8 * j : 16 * j + 8;
  const int all = p.heads[0] + p.heads[1], h0 = blockIdx.y * p.per, h1 = min(all, h0 + p.per);
  for (int h = h0; h < h1; h += 4) {
    Item x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (h + e < h1) {
        const int w = h + e >= p.heads[0], hh = h + e - (w ? p.heads[0] : 0);
        const rkv_bf16* src = p.in[w] + b * p.is[w][0] + hh * p.is[w][1] + t * p.is[w][2];
        x[e].a = *reinterpret_cast<const uint4*>(src + at_a);
        x[e].b = *reinterpret_cast<const uint4*>(src + at_b);
      }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (h + e < h1) {
        const int w = h + e >= p.heads[0], hh = h + e - (w ? p.heads[0] : 0);
        if (halves) {
          rotate2(x[e].a.x, x[e].b.x, c, s);
          rotate2(x[e].a.y, x[e].b.y, c + 2, s + 2);
          rotate2(x[e].a.z, x[e].b.z, c + 4, s + 4);
          rotate2(x[e].a.w, x[e].b.w, c + 6, s + 6);
        } else if (turn) {
          rotate1(x[e].a.x, c[0], s[0]);
          rotate1(x[e].a.y, c[1], s[1]);
          rotate1(x[e].a.z, c[2], s[2]);
          rotate1(x[e].a.w, c[3], s[3]);
          rotate1(x[e].b.x, c[4], s[4]);
          rotate1(x[e].b.y, c[5], s[5]);
          rotate1(x[e].b.z, c[6], s[6]);
          rotate1(x[e].b.w, c[7], s[7]);
        }
        rkv_bf16* dst = p.out[w] + b * p.os[w][0] + hh * p.os[w][1] + t * p.os[w][2];
        *reinterpret_cast<uint4*>(dst + at_a) = x[e].a;
        *reinterpret_cast<uint4*>(dst + at_b) = x[e].b;
      }
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  RotaryParams p;
  for (int i = 0; i < 64; ++i) p.turns[i] = a.plan.turns[i];
  for (int i = 0; i < 3; ++i) {
    p.is[0][i] = a.q_strides[i];
    p.os[0][i] = a.q_out_strides[i];
    p.is[1][i] = a.k ? a.k_strides[i] : 0;
    p.os[1][i] = a.k ? a.k_out_strides[i] : 0;
  }
  p.in[0] = a.q;
  p.in[1] = a.k;
  p.out[0] = a.q_out;
  p.out[1] = a.k_out;
  p.positions = a.positions;
  p.heads[0] = a.Hq;
  p.heads[1] = a.k ? a.Hkv : 0;
  p.T = a.T;
  p.rot = a.plan.rot_dim;
  p.interleaved = a.plan.interleaved;
  p.per_token = a.per_token;
  p.inverse = a.inverse;
  p.tokens = (long long)a.B * a.T;
  p.amplitude = a.plan.amplitude;
  const int all = p.heads[0] + p.heads[1];
  p.per = 8;
  const dim3 grid((unsigned)((p.tokens + kRoThreads / 8 - 1) / (kRoThreads / 8)), (all + p.per - 1) / p.per);
  launch_begin(K_ROTARY, s);
  rotary_kernel<<<grid, kRoThreads, 0, s>>>(p);
  launch_end(K_ROTARY, s);
  return cudaGetLastError();
}

}  // namespace rkv
