// A flat split of ragged units over a grid, from lengths that only the device knows.
//
// Every sequence b holds `per_unit(b)` pieces of work (key chunks, token blocks) for each
// of its `units(b)` units (KV heads, row tiles).  All units' pieces in order (b major)
// form one line of `total` pieces and CTA i of N takes [i total / N, (i + 1) total / N):
// the grid is sized without the lengths, and no CTA carries more than one piece above
// the mean.  A unit's first `pad` pieces are empty: they stand for what starting and ending
// a run costs, so that a CTA with many short units gets fewer pieces.  Each CTA rebuilds
// the table (one load a sequence and a warp scan, about a microsecond).
#pragma once

#include "rkv_device.cuh"

namespace rkv {

struct FlatTable {
  long long base[RKV_MAX_BATCH + 1];  // pieces before sequence b
  int n[RKV_MAX_BATCH];               // tokens of sequence b (0 when its length is not usable)
  int t[RKV_MAX_BATCH];               // query rows (nodes) of sequence b
  int per[RKV_MAX_BATCH];             // pieces of each of its units, the empty ones included
  int units[RKV_MAX_BATCH];           // its units
  int pad;                            // empty pieces of a unit
};

// base[b] = sum of size(0 .. b - 1), base[B] the total: the first warp's scan; ends with a
// block barrier.
template <class Size>
__device__ __forceinline__ void flat_scan(long long* base, int B, Size size) {
  const int lane = threadIdx.x;
  if (lane < 32) {
    const int each = (B + 31) / 32;
    long long s = 0, only = 0;
    for (int j = 0; j < each; ++j)
      if (lane * each + j < B) s += (only = size(lane * each + j));
    long long incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      if (o < B) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
    }
    long long at = incl - s;
    for (int j = 0; j < each; ++j) {
      const int b = lane * each + j;
      if (b < B) {
        base[b] = at;
        at += each == 1 ? only : size(b);
        if (b == B - 1) base[B] = at;
      }
    }
  }
  __syncthreads();
}

// len(b) -> tokens, rows(b) -> nodes, per(n, t) -> pieces a unit (without the empty ones),
// units(t) -> units.
// Called by every thread of the block (at least 32); ends with a block barrier.
template <class Len, class Rows, class Per, class Units>
__device__ __forceinline__ void flat_build(FlatTable& ft, int B, int pad, Len len, Rows rows, Per per, Units units) {
  const int tid = threadIdx.x;
  if (tid == 0) ft.pad = pad;
  for (int b = tid; b < B; b += blockDim.x) {
    ft.n[b] = len(b);
    ft.t[b] = rows(b);
    const int real = per(ft.n[b], ft.t[b]);
    ft.per[b] = real > 0 ? real + pad : 0;
    ft.units[b] = units(ft.t[b]);
  }
  __syncthreads();
  flat_scan(ft.base, B, [&](int b) { return (long long)ft.per[b] * ft.units[b]; });
}

// CTAs that take part: no more than there are pieces, so that no share is empty and every
// CTA between a unit's first and last holds a part of it.
__device__ __forceinline__ int flat_ctas(long long total, int N) { return (int)min((long long)N, total); }
// 32-bit divisions where the operands allow it: a 64-bit one costs about a hundred
// instructions.  N is at most kMaxSms + 1 < 2^10.
__device__ __forceinline__ long long flat_first(long long total, int i, int N) {
  if (total < (1 << 20)) return (uint32_t)total * (uint32_t)i / (uint32_t)N;
  return total * i / N;
}
// The CTA whose share holds piece x.
__device__ __forceinline__ int flat_cta(long long x, long long total, int N) {
  if (total < (1 << 20)) return (int)(((uint32_t)(x + 1) * (uint32_t)N - 1) / (uint32_t)total);
  return (int)(((x + 1) * N - 1) / total);
}
// The sequence that holds piece x (0 <= x < base[B]).
__device__ __forceinline__ int flat_seq(const FlatTable& ft, int B, long long x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ft.base[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Walks the pieces of a share a run at a time: a run is the share's part of one unit.
struct FlatRun {
  int b, unit;           // sequence, unit inside it
  int lo, hi;            // the run's pieces of the unit, without the empty ones; lo < hi
  int whole;             // the run is the whole unit
  int first;             // the run starts the share
  long long x, next;     // the run's first piece on the line, and the one behind its last
};
// Part [off, off + room) of a unit of `per` pieces as a run; false: only empty pieces.
__device__ __forceinline__ bool flat_part(FlatRun& r, int off, long long room, int per, int pad) {
  const int end = (int)min((long long)per, off + room);
  r.next = r.x + (end - off);
  r.lo = max(off - pad, 0);
  r.hi = end - pad;
  r.whole = r.lo == 0 && end == per;
  return r.hi > r.lo;
}
__device__ __forceinline__ bool flat_run(const FlatTable& ft, int B, long long x, long long x0, long long x1, FlatRun& r) {
  for (; x < x1; x = r.next) {
    r.b = flat_seq(ft, B, x);
    const int per = ft.per[r.b];
    const long long off = x - ft.base[r.b];
    r.unit = off < (1LL << 31) ? (int)((uint32_t)off / (uint32_t)per) : (int)(off / per);
    r.first = x == x0;
    r.x = x;
    if (flat_part(r, (int)(off - (long long)r.unit * per), x1 - x, per, ft.pad)) return true;
  }
  return false;
}

}  // namespace rkv
