// What the kernels of the attention over the 8-bit cache share (rkv_q8_attend.cu, rkv_q8_tiles.cu).
#pragma once

#include "rkv_attend.cuh"
#include "rkv_causal.cuh"
#include "rkv_internal.h"
#include "rkv_q8.cuh"

namespace rkv {

struct Q8Params {
  CUtensorMap tmk, tmv;  // the codes as [rows][128] bytes, a page's (or half a 64-token page's) rows to a box
  const rkv_bf16* q;     // [B][Hq][T][128]
  const float *k_scale, *v_scale;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* row_len;  // null: T rows everywhere
  int32_t* err;
  rkv_bf16* out;
  float* lse;      // may be null
  float* part_o;   // [2 N][tile rows][128]
  float2* part_ml; // [2 N][tile rows]
  int B, Hq, Hkv, G, gshift, T, P, pshift, max_pages, num_phys, N;
  int join_tiles;  // q8_join: row tiles of a unit with T rows
  float scale_log2;
};

constexpr float kSlack = 8.f;        // a weight's exponent may lie this far above the maximum it refers to
constexpr float kUnit = 128.f;       // 2^7: a weight of 2^8 becomes 2^15 in fp16

__device__ __forceinline__ int checked_len(const Q8Params& p, int b) {
  const int n = p.seq_len[b];
  if (n < 0 || n > p.max_pages * p.P) {
    flag_error(p.err, RKV_DEVERR_CAPACITY);
    return 0;
  }
  return n;
}
__device__ __forceinline__ int checked_rows(const Q8Params& p, int b) {
  const int m = p.row_len ? p.row_len[b] : p.T;
  if (m < 0 || m > p.T) {
    flag_error(p.err, RKV_DEVERR_TREE);
    return 0;
  }
  return m;
}
__device__ __forceinline__ size_t out_row(const Q8Params& p, int b, int g, int r) {
  return ((size_t)b * p.Hq + g * p.G + (r & (p.G - 1))) * p.T + (r >> p.gshift);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 .. 127

// More than 24 query rows a KV head, on the fifth-generation tensor cores: the parts of split
// units for q8_join, or the results.  wide: 256 rows to a tile, else 128.
constexpr int kQtKeysShift = 7, kQtPad = 4;
template <int kRowsShift>
using TileLine = CausalLine<kRowsShift, kQtKeysShift, kQtPad>;
cudaError_t launch_q8_tiles(const Q8Params& p, bool wide, bool int8, cudaStream_t s);

}  // namespace rkv
