// The flat split (rkv_flat.cuh) for rows that see a part of the keys each.
//
// Sequence b's m rows (positions n - m .. n - 1 of its n tokens, G heads each) go in tiles of
// kRows = s G query rows; tile i's last row sees
//   vis(i) = min(n, n - m + (i + 1) s)
// keys, in ceil(vis / kKeys) pieces (and kPad empty ones) for each of the KV heads.  A tile
// that sees nothing has none.  How many pieces lie before tile k is a closed form, so a
// place on the line is found by bisection, with nothing stored but n, m and each sequence's
// start.
#pragma once

#include "rkv_flat.cuh"

namespace rkv {

// sum of floor((a + j s) / keys) over j < count; s = 2^sshift, keys = 2^kshift, a >= 0
__device__ __forceinline__ long long floors_before(long long a, int sshift, int kshift, long long count) {
  if (sshift >= kshift) return count * (a >> kshift) + ((count * (count - 1) / 2) << (sshift - kshift));
  const int rshift = kshift - sshift;  // floor((a + j s) / keys) = floor((floor(a / s) + j) / r), r = 2^rshift
  const long long x0 = a >> sshift, x1 = x0 + count;
  auto upto = [&](long long x) {  // sum of floor(j / r) over j < x
    const long long u = x >> rshift, w = x & ((1LL << rshift) - 1);
    return ((u * (u - 1) / 2) << rshift) + u * w;
  };
  return upto(x1) - upto(x0);
}

// A run and the rows that it belongs to: KV head, row tile, tokens and rows of its sequence.
struct CausalRun : FlatRun {
  int g, rt, n, m;
};

template <int kRowsShift, int kKeysShift, int kPadPieces>
struct CausalLine {
  static constexpr int kKeys = 1 << kKeysShift, kPad = kPadPieces, kRows = 1 << kRowsShift;
  long long base[RKV_MAX_BATCH + 1];

  static __device__ __forceinline__ int tiles(int m, int gshift) {
    const int sshift = kRowsShift - gshift;
    return (m + (1 << sshift) - 1) >> sshift;
  }
  // pieces of tile i of a KV head, the empty ones included
  static __device__ __forceinline__ int per(int n, int m, int gshift, int i) {
    const int end = (i + 1) << (kRowsShift - gshift);
    const int vis = end >= m ? n : n - m + end;
    return vis > 0 ? ((vis + kKeys - 1) >> kKeysShift) + kPad : 0;
  }
  // pieces of the tiles before tile k of a KV head
  static __device__ __forceinline__ long long before(int n, int m, int gshift, int k) {
    if (k == 0 || n == 0) return 0;
    const int sshift = kRowsShift - gshift, last = tiles(m, gshift) - 1, c = n - m;
    const int i0 = c < 0 ? (-c) >> sshift : 0;  // the first tile that sees anything
    if (k <= i0) return 0;
    const int inner = min(k, last) - i0;  // of these, tiles that end before the last row
    long long sum = 0;
    if (inner > 0)
      sum = floors_before((long long)c + ((long long)(i0 + 1) << sshift) + kKeys - 1, sshift, kKeysShift, inner) +
            (long long)inner * kPad;
    if (k > last) sum += ((n + kKeys - 1) >> kKeysShift) + kPad;
    return sum;
  }
  // len(b), rows(b): tokens and rows of a sequence, asked for by the first warp; ends with a
  // block barrier
  template <class Len, class Rows>
  __device__ __forceinline__ void build(int B, int Hkv, int gshift, Len len, Rows rows) {
    flat_scan(base, B, [&](int b) {
      const int m = rows(b);
      return m > 0 ? before(len(b), m, gshift, tiles(m, gshift)) * Hkv : 0LL;
    });
  }
  // the next run of a share at or behind x
  template <class Len, class Rows>
  __device__ __forceinline__ bool next(int B, int Hkv, int gshift, Len len, Rows rows, long long x, long long x0,
                                       long long x1, CausalRun& r) const {
    for (; x < x1; x = r.next) {
      int lo = 0, hi = B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= x) lo = mid; else hi = mid - 1;
      }
      r.b = lo;
      r.n = len(lo);
      r.m = rows(lo);
      const long long off = x - base[lo];
      int a = 0, z = tiles(r.m, gshift) - 1;
      while (a < z) {  // the last tile whose pieces begin at or before off
        const int mid = (a + z + 1) >> 1;
        if (before(r.n, r.m, gshift, mid) * Hkv <= off) a = mid; else z = mid - 1;
      }
      const int pieces = per(r.n, r.m, gshift, a);
      const uint32_t in = (uint32_t)(off - before(r.n, r.m, gshift, a) * Hkv);
      r.rt = a;
      r.g = (int)(in / (uint32_t)pieces);
      r.unit = 0;
      r.first = x == x0;
      r.x = x;
      if (flat_part(r, (int)(in - (uint32_t)r.g * (uint32_t)pieces), x1 - x, pieces, kPad)) return true;
    }
    return false;
  }
  // where unit (b, tile i, KV head g) of a sequence of n tokens and m rows begins on the line
  __device__ __forceinline__ long long at(int b, int n, int m, int Hkv, int gshift, int i, int g) const {
    return base[b] + before(n, m, gshift, i) * Hkv + (long long)g * per(n, m, gshift, i);
  }
};

// The same with the sequences' lengths beside it, read once.
template <class Line>
struct LineLengths : Line {
  int n[RKV_MAX_BATCH], m[RKV_MAX_BATCH];
  template <class Len, class Rows>
  __device__ __forceinline__ void build(int B, int Hkv, int gshift, Len len, Rows rows) {
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
      n[b] = len(b);
      m[b] = rows(b);
    }
    __syncthreads();
    Line::build(B, Hkv, gshift, [&](int b) { return n[b]; }, [&](int b) { return m[b]; });
  }
  __device__ __forceinline__ bool next(int B, int Hkv, int gshift, long long x, long long x0, long long x1, CausalRun& r) const {
    return Line::next(B, Hkv, gshift, [&](int b) { return n[b]; }, [&](int b) { return m[b]; }, x, x0, x1, r);
  }
  __device__ __forceinline__ long long at(int b, int Hkv, int gshift, int i, int g) const {
    return Line::at(b, n[b], m[b], Hkv, gshift, i, g);
  }
};

}  // namespace rkv
