// Accumulated attention weights of the cached tokens, and the eviction by them.
//
//   accum_rows   acc_t += sum over the group's heads and the given rows i of
//                [t <= n - m + i] exp(scale q_i . k_t - lse_i): the m rows are the
//                cache's last m positions, lse_i what their attention left behind.
//   evict        keeps, per (sequence, KV head), the `recent` last tokens and the
//                heaviest of the others, in order, in this or another cache.
#include "rkv_flat.cuh"
#include "rkv_internal.h"
#include "rkv_select.cuh"

namespace rkv {
namespace {

// ---------------------------------------------------------------------------
// accum_rows: transposed logits, keys as the MMA's M and query rows as its N, so that a
// key's sum over the rows is a private loop and a shuffle over four lanes.  Only K is
// read, 4 KB for a 16-key chunk, and every position has one writer: no atomics, the
// same sums in the same order every time.  The bytes of K bound it: 24 rows over the ragged
// batch of 16 x 8K .. 32K (685 MB) take 121 us, 5.7 TB/s, 83 % of a plain copy's rate; the
// rest is the chain of a chunk (copy, product, exponential, sum) in too few warps.
constexpr int kRwKeys = 16;
constexpr int kRwPad = 16;  // what a run costs, in chunks
constexpr int kRwStageBytes = 4096;
constexpr int kRwBlock = 64;  // query rows staged at a time, at most
constexpr int kRwSmem = 1024 + 48 * kRwStageBytes + kRwBlock * 256;

struct RowsParams {
  CUtensorMap tmk;     // the key pool as [rows][128] bf16, 128-byte swizzled boxes of 64 channels
  CUtensorMap tmq;     // q the same, boxes of nq rows (accum_tiles)
  const rkv_bf16* q;   // [B][Hq][T][128]
  const float* lse;    // [B][Hq][T]
  const int32_t* row_len;
  const int32_t* row_ids;
  const int32_t* page_table;
  const int32_t* seq_len;
  int32_t* err;
  float* acc;
  float* part;         // accum_tiles: [2 N][256] sums of the units' parts
  int B, Hq, Hkv, G, gshift, T, ids_stride, P, pshift, max_pages, num_phys, acc_stride, N, nq;
  float scale, scale_log2;
};

// Rows of sequence b that are taken (0 when the count or the length is not usable).
__device__ __forceinline__ int rows_of(const RowsParams& p, int b, int n) {
  const int most = p.row_ids ? p.ids_stride : p.T;
  const int m = p.row_len ? p.row_len[b] : most;
  if (m < 0 || m > most || m > n) {
    flag_error(p.err, RKV_DEVERR_TREE);
    return 0;
  }
  return m;
}
__device__ __forceinline__ int rows_cache_len(const RowsParams& p, int b) {
  const int n = p.seq_len[b];
  if (n < 0 || n > p.max_pages * p.P) {
    flag_error(p.err, RKV_DEVERR_CAPACITY);
    return 0;
  }
  return n;
}

// kR16: 16-row groups of a block; the block's rows stay in registers as B fragments.
// Up to two groups leave room for 16 warps with three stages each, which hide the chain
// of a chunk (load, product, exponential, sum) better than eight warps with six.
template <int kR16>
struct RowsShape {
  static constexpr int kWarps = kR16 <= 2 ? 16 : 8;
  static constexpr int kStages = 48 / kWarps;
};
template <int kR16>
__global__ void __launch_bounds__(RowsShape<kR16>::kWarps * 32, 1)
    accum_rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int kBlock = kR16 * 16;
  constexpr int kRwWarps = RowsShape<kR16>::kWarps, kRwStages = RowsShape<kR16>::kStages, kRwThreads = kRwWarps * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ FlatTable ft;
  __shared__ uint64_t full_b[kRwWarps][kRwStages];
  __shared__ float ls[kBlock];  // base-2 log-sum-exp of the staged rows, +inf: weighs nothing
  __shared__ int last[kBlock];  // last position a staged row sees
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* base = align1024(smem);
  uint8_t* ring = base + warp * kRwStages * kRwStageBytes;
  uint8_t* qs = base + kRwWarps * kRwStages * kRwStageBytes;
  if (lane == 0) {
    for (int s = 0; s < kRwStages; ++s) mbar_init(&full_b[warp][s], 1);
    fence_mbar_init();
  }
  flat_build(
      ft, p.B, kRwPad, [&](int b) { return rows_cache_len(p, b); }, [&](int b) { return rows_of(p, b, rows_cache_len(p, b)); },
      [&](int n, int m) { return m > 0 ? (n + kRwKeys - 1) / kRwKeys : 0; }, [&](int) { return p.Hkv; });
  const long long total = ft.base[p.B];
  const int N = flat_ctas(total, p.N);
  if (blockIdx.x >= N) return;
  const long long x0 = flat_first(total, blockIdx.x, N), x1 = flat_first(total, blockIdx.x + 1, N);
  int fetched = 0, used = 0;
  bool dead = false;
  uint32_t skipped = 0;
  FlatRun r;
  for (long long x = x0; flat_run(ft, p.B, x, x0, x1, r); x = r.next) {
    const int b = r.b, g = r.unit, n = ft.n[b], m = ft.t[b], rows = m * p.G;
    int ids = -1, ids_at = 0;  // page ids of this warp's chunks ids_at + 8 lane
    auto load_ids = [&](int c) {
      ids_at = c;
      const int mine = c + lane * kRwWarps;
      ids = mine < r.hi ? p.page_table[(size_t)b * p.max_pages + ((mine * kRwKeys) >> p.pshift)] : -1;
    };
    auto fetch = [&](int c) {
      const int s = fetched % kRwStages, t0 = c * kRwKeys;
      if (c >= ids_at + 32 * kRwWarps) load_ids(c);
      const int phys = __shfl_sync(0xffffffffu, ids, (c - ids_at) / kRwWarps);
      if (phys >= 0 && phys < p.num_phys) {
        skipped &= ~(1u << s);
        if (lane == 0) {
          const int row = (phys * p.Hkv + g) * p.P + (t0 & (p.P - 1));
          uint8_t* st = ring + s * kRwStageBytes;
          mbar_arrive_expect_tx(&full_b[warp][s], kRwStageBytes);
          tma_load_2d(st, &p.tmk, 0, row, &full_b[warp][s]);
          tma_load_2d(st + 2048, &p.tmk, 64, row, &full_b[warp][s]);
        }
      } else {
        skipped |= 1u << s;
        if (lane == 0) {
          flag_error(p.err, RKV_DEVERR_PAGE_ID);
          mbar_arrive(&full_b[warp][s]);
        }
      }
      ++fetched;
    };
    for (int blk = 0; blk < rows; blk += kBlock) {
      const int live = min(kBlock, rows - blk);
      int fc = r.lo + warp;
      load_ids(fc);
      for (int s = 0; s < kRwStages && fc < r.hi && !dead; ++s, fc += kRwWarps) fetch(fc);
      // the block's query rows (row = i G + head), swizzled as the boxes are
      for (int e = tid; e < kBlock * 16; e += kRwThreads) {
        const int row = e >> 4, piece = e & 15;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < live) {
          const int i = (blk + row) >> p.gshift, h = (blk + row) & (p.G - 1);
          const int id = p.row_ids ? p.row_ids[(size_t)b * p.ids_stride + i] : i;
          const bool ok = id >= 0 && id < p.T;
          const size_t at = ((size_t)b * p.Hq + g * p.G + h) * p.T + (ok ? id : 0);
          if (ok) v = reinterpret_cast<const uint4*>(p.q + at * 128)[piece];
          if (piece == 0) {
            if (!ok) flag_error(p.err, RKV_DEVERR_TREE);
            const float l = ok ? p.lse[at] * 1.4426950408889634f : INFINITY;
            ls[row] = l == -INFINITY ? INFINITY : l;
            last[row] = n - m + i;
          }
        } else if (piece == 0) {
          ls[row] = INFINITY;
          last[row] = -1;
        }
        *reinterpret_cast<uint4*>(qs + (piece >> 3) * (kBlock * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4)) = v;
      }
      __syncthreads();
      uint32_t qf[kR16][8][4];
      float lr[kR16][4];
      {
        const uint32_t qb = smem_u32(qs);
        const int rr = ((lane >> 4) << 3) + (lane & 7), sub = (lane >> 3) & 1;
#pragma unroll
        for (int q = 0; q < kR16; ++q) {
          const int row = q * 16 + rr;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int piece = k * 2 + sub;
            ldsm_x4(qf[q][k][0], qf[q][k][1], qf[q][k][2], qf[q][k][3],
                    qb + (piece >> 3) * (kBlock * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) lr[q][e] = ls[q * 16 + (e >> 1) * 8 + (lane & 3) * 2 + (e & 1)];
        }
      }
      // the sums of the next chunk's positions, loaded a chunk ahead of their use
      float* const sums = p.acc + ((size_t)b * p.Hkv + g) * p.acc_stride + (lane >> 2);
      const bool adds = (lane & 3) == 0;
      auto sum_at = [&](int c, int o) {
        const int t = c * kRwKeys + o;
        return adds && c < r.hi && t + (lane >> 2) < n ? sums[t] : 0.f;
      };
      float next0 = sum_at(r.lo + warp, 0), next1 = sum_at(r.lo + warp, 8);
      for (int c = r.lo + warp; c < r.hi; c += kRwWarps) {
        const int s = used % kRwStages;
        const float old0 = next0, old1 = next1;
        next0 = sum_at(c + kRwWarps, 0);
        next1 = sum_at(c + kRwWarps, 8);
        const bool late = !dead && !mbar_wait(&full_b[warp][s], (uint32_t)((used / kRwStages) & 1));
        if (__any_sync(0xffffffffu, late)) {
          if (lane == 0) flag_error(p.err, RKV_DEVERR_TIMEOUT);
          dead = true;
        }
        if (dead) break;
        const bool take = !((skipped >> s) & 1u);
        const uint32_t ks = smem_u32(ring + s * kRwStageBytes);
        float z[kR16][2][4];
#pragma unroll
        for (int q = 0; q < kR16; ++q)
#pragma unroll
          for (int e = 0; e < 8; ++e) z[q][e >> 2][e & 3] = 0.f;
        {
          const int key = (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int piece = k * 2 + (lane >> 4);
            uint32_t a0, a1, a2, a3;
            ldsm_x4(a0, a1, a2, a3, ks + (piece >> 3) * 2048 + key * 128 + (((piece & 7) ^ (key & 7)) << 4));
#pragma unroll
            for (int q = 0; q < kR16; ++q) {
              mma_16816(z[q][0], a0, a1, a2, a3, qf[q][k][0], qf[q][k][1]);
              mma_16816(z[q][1], a0, a1, a2, a3, qf[q][k][2], qf[q][k][3]);
            }
          }
        }
        ++used;
        __syncwarp();  // every lane has read the stage
        if (fc < r.hi) {
          fetch(fc);
          fc += kRwWarps;
        }
        if (!take) continue;
        const int t0 = c * kRwKeys + (lane >> 2), t1 = t0 + 8;
        float w0 = 0.f, w1 = 0.f;
        const bool all = (c + 1) * kRwKeys <= n - m + 1;  // every row sees the whole chunk
#pragma unroll
        for (int q = 0; q < kR16; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float e0 = ex2_approx(fmaf(z[q][e >> 1][e & 1], p.scale_log2, -lr[q][e]));
            const float e1 = ex2_approx(fmaf(z[q][e >> 1][2 + (e & 1)], p.scale_log2, -lr[q][e]));
            if (all) {
              w0 += e0;
              w1 += e1;
            } else {
              const int seen = last[q * 16 + (e >> 1) * 8 + (lane & 3) * 2 + (e & 1)];
              w0 += t0 <= seen ? e0 : 0.f;
              w1 += t1 <= seen ? e1 : 0.f;
            }
          }
        w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
        w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
        if (adds) {
          if (t0 < n) sums[c * kRwKeys] = old0 + w0;
          if (t1 < n) sums[c * kRwKeys + 8] = old1 + w1;
        }
      }
      __syncthreads();  // the staged rows are free
    }
  }
  if (dead)
    for (int i = used; i < fetched; ++i) mbar_wait(&full_b[warp][i % kRwStages], (uint32_t)((i / kRwStages) & 1));
}

// ---------------------------------------------------------------------------
// accum_tiles: many rows (a prompt's or a chunk's), on the fifth-generation tensor cores.
//
// S^T = K Q^T with the keys on the TMEM lanes: a thread owns a key, and its sum over the
// rows is a private loop over columns, as in the window scoring of the prefill.  A unit is
// 256 keys of a KV head (two 128-key MMAs share each query tile of nq rows, so that a tile
// read from L2 feeds twice the products); its pieces are the (head, row tile) pairs that
// see it, and all units' pieces form one line that is split evenly over the SMs: the
// causal triangle needs no balancing of its own.  A unit split between CTAs leaves its
// parts in the workspace and accum_join adds them in order.
// The log-sum-exps come off inside the product: a 17th group of 16 channels holds 1, 1, 1
// for every key and, for row i, -lse_i / scale as three bf16 terms (24 bits), so the
// accumulator is (z - lse) / scale and the sum a product, an exponential and an addition
// per cell.  The three terms keep an lse to 2^-24, as its product with log2 e does in
// accum_rows; the sums of 16K rows come out within 5e-7 of the 64-bit ones.  (Read from
// shared memory instead, 16 loads a warp and tile, the sums of a tile took 2619 clocks
// beside running products, which use all of its bandwidth, and 1244 alone.)
// Per piece 2 x 128 x nq x 144 multiply-adds and 256 nq exponentials; at nq = 128 the
// products take 1152 clocks of an SM and the exponentials 1024 at 32 a clock: two
// accumulators a key tile keep both busy.  Measured: 16K rows x 32 heads 845 us, 1.3 PFLOP/s
// of the triangle's products (without exponentials 764, with a third of the products 776,
// with neither 580, with loads of the accumulators alone 775: products, loads and sums share
// the tensor memory's ports and the issue slots, near the card's power limit).
//   warps 0-15: sums (warps 4 w .. 4 w + 3: key tile w / 2, column half w % 2);
//   warp 16: TMA;  warp 17: MMA issue;  warps 18, 19: the rows' log-sum-exps.
constexpr int kAmKeys = 256;
constexpr int kAmThreads = 640;
constexpr int kAmQ = 4;           // query tiles in the ring
constexpr int kAmExtra = 128 * 32;  // 128 rows x 16 channels of the extra product
constexpr int kAmSmem = 1024 + 6 * 32768 + (1 + kAmQ) * kAmExtra;

struct TilesTable {
  long long base[RKV_MAX_BATCH + 1];
  int n[RKV_MAX_BATCH], m[RKV_MAX_BATCH];
};

// The units of one KV head: n tokens, m rows at positions c0 = n - m ...; unit j (keys
// 256 j ...) is seen by row tiles f(j) .. RT - 1 of every head.
struct HeadShape {
  int RT, J0, jz, units, G;
  __device__ __forceinline__ HeadShape(int n, int m, int nq, int G_) : G(G_) {
    RT = (m + nq - 1) / nq;
    const int c0 = n - m;
    J0 = (c0 + 127) / 128;  // nq < 128 means one row tile: f is 0 throughout
    if (RT == 1) J0 = 1 << 28;
    jz = J0 / 2 + 1;        // the first unit that some row tile does not see
    units = m > 0 ? (n + kAmKeys - 1) / kAmKeys : 0;
  }
  __device__ __forceinline__ int first(int j) const { return max(0, 2 * j - J0); }
  __device__ __forceinline__ int pieces(int j) const { return G * (RT - first(j)); }
  __device__ __forceinline__ long long before(int j) const {  // pieces of units 0 .. j - 1
    long long c = (long long)j * RT;
    if (j > jz) c -= (long long)(j - jz) * (jz + j - 1) - (long long)J0 * (j - jz);
    return c * G;
  }
};

struct TilesRun {
  int b, g, j, lo, hi, f, width;  // pieces lo .. hi of unit j; width = row tiles of a head that see it
  long long x, ux;                // the run's first piece, the unit's first piece
  int whole, first;
};

// The run that holds piece x, found from nothing (two 64-bit divisions and two searches).
__device__ __forceinline__ bool tiles_find(const RowsParams& p, const TilesTable& tt, int nq, long long x, long long x0,
                                           long long x1, TilesRun& r) {
  if (x >= x1) return false;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tt.base[mid] <= x) lo = mid; else hi = mid - 1;
  }
  r.b = lo;
  const HeadShape h(tt.n[lo], tt.m[lo], nq, p.G);
  const long long each = h.before(h.units), off = x - tt.base[lo];
  r.g = (int)(off / each);
  const long long in = off - r.g * each;
  int a = 0, z = h.units - 1;
  while (a < z) {
    const int mid = (a + z + 1) >> 1;
    if (h.before(mid) <= in) a = mid; else z = mid - 1;
  }
  r.j = a;
  r.f = h.first(a);
  r.width = h.RT - r.f;
  const int count = h.pieces(a);
  r.lo = (int)(in - h.before(a));
  r.hi = (int)min((long long)count, r.lo + (x1 - x));
  r.whole = r.lo == 0 && r.hi == count;
  r.first = x == x0;
  r.x = x;
  r.ux = x - r.lo;
  return true;
}

// The run behind r: the next unit of the head, of the next head or sequence.
__device__ __forceinline__ bool tiles_next(const RowsParams& p, const TilesTable& tt, int nq, long long x1, TilesRun& r) {
  r.x += r.hi - r.lo;
  if (r.x >= x1) return false;
  if (++r.j * kAmKeys >= tt.n[r.b]) {
    r.j = 0;
    if (++r.g == p.Hkv) {
      r.g = 0;
      do ++r.b;
      while (tt.m[r.b] == 0);  // there is one: pieces are left
    }
  }
  const HeadShape h(tt.n[r.b], tt.m[r.b], nq, p.G);
  r.f = h.first(r.j);
  r.width = h.RT - r.f;
  const int count = h.pieces(r.j);
  r.lo = 0;
  r.hi = (int)min((long long)count, x1 - r.x);
  r.whole = r.hi == count;
  r.first = 0;
  r.ux = r.x;
  return true;
}

__device__ __forceinline__ void tiles_table(const RowsParams& p, TilesTable& tt) {
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int n = rows_cache_len(p, b);
    tt.n[b] = n;
    tt.m[b] = rows_of(p, b, n);
  }
  __syncthreads();
  flat_scan(tt.base, p.B, [&](int b) {
    const HeadShape h(tt.n[b], tt.m[b], p.nq, p.G);
    return p.Hkv * h.before(h.units);
  });
}

// kQRows (nq): 128 with one unit's keys (64 KB) resident and four 32 KB query tiles in
// flight, a unit then having many pieces; 64 (T <= 64: a piece per head) with two units'
// keys and four 16 KB tiles.
template <int kQRows>
__global__ void __launch_bounds__(kAmThreads, 1) accum_tiles_kernel(const __grid_constant__ RowsParams p) {
  constexpr int KS = kQRows == 128 ? 1 : 2, QB = kQRows * 256;
  static_assert(KS * 65536 + kAmQ * QB == 6 * 32768, "the rings fill the shared memory");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ TilesTable tt;
  __shared__ uint64_t kfull[KS], kempty[KS], qfull[kAmQ], qempty[kAmQ];
  __shared__ uint64_t sfull[2][2], sempty[2][2], hsum, drained;  // [buffer][key tile]
  __shared__ float half_s[2][2][128];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* ks = align1024(smem);
  uint8_t* qs = ks + KS * 65536;
  uint8_t* ones = ks + 6 * 32768;        // the extra channels of every key
  uint8_t* bias = ones + kAmExtra;       // and of the rows of the query tiles in the ring
  for (int i = tid; i < (1 + kAmQ) * kAmExtra / 16; i += kAmThreads) {
    // rows of 8 to a core matrix, the two core matrices of a row 128 bytes apart
    const bool one = i < kAmExtra / 16 && ((i >> 3) & 1) == 0;
    reinterpret_cast<uint4*>(ones)[i] = one ? make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (tid == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < kAmQ; ++i) {
      mbar_init(&qfull[i], 1 + 32);  // the copy and the lanes that write the log-sum-exps
      mbar_init(&qempty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i >> 1][i & 1], 1);
      mbar_init(&sempty[i >> 1][i & 1], 256);
    }
    mbar_init(&hsum, 512);
    mbar_init(&drained, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  tiles_table(p, tt);
  tc_fence_after();
  grid_launch_dependents();
  const uint32_t tmem = tmem_base;
  constexpr int nq = kQRows;
  const long long total = tt.base[p.B];
  const int N = flat_ctas(total, p.N);
  const bool works = (int)blockIdx.x < N;
  const long long x0 = works ? flat_first(total, blockIdx.x, N) : 0, x1 = works ? flat_first(total, blockIdx.x + 1, N) : 0;
  auto wait = [&](uint64_t* bar, int phase) {
    const bool late = !mbar_wait_role(bar, (uint32_t)(phase & 1), &abort_flag);
    if (__any_sync(0xffffffffu, late)) {
      flag_error(p.err, RKV_DEVERR_TIMEOUT);
      abort_flag = 1;
      return false;
    }
    return true;
  };
  auto wait_one = [&](uint64_t* bar, int phase) {  // a single lane's
    if (mbar_wait_role(bar, (uint32_t)(phase & 1), &abort_flag)) return true;
    flag_error(p.err, RKV_DEVERR_TIMEOUT);
    abort_flag = 1;
    return false;
  };
  TilesRun r;
  int units = 0, tiles = 0;  // units and query tiles loaded (16), used (17), read (others)
  bool ok = true;

  if (warp < 16) {
    const int wg = warp >> 2, kt = wg >> 1, half = wg & 1, key = kt * 128 + (tid & 127);
    constexpr int cols = nq >> 1;
    const int c0 = half * cols;  // this warp's columns
    const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kt * 128 + c0;
    const float sl = p.scale_log2;
    for (bool more = tiles_find(p, tt, nq, x0, x0, x1, r); ok && more; more = tiles_next(p, tt, nq, x1, r)) {
      const int n = tt.n[r.b], m = tt.m[r.b], t = r.j * kAmKeys + key;
      float sum = 0.f;
      int rt = r.f + (r.lo > 0 ? r.lo % r.width : 0);
      for (int o = r.lo; o < r.hi; ++o) {
        const int buf = tiles & 1, i0 = rt * nq;
        if (++rt == r.f + r.width) rt = r.f;
        if (!(ok = wait(&sfull[buf][kt], tiles / 2))) break;
        tc_fence_after();
        uint32_t va[2][32];
        tc_ld32(mine + buf * 256, va[0]);
        if (cols > 32) tc_ld32(mine + buf * 256 + 32, va[1]);
        // the columns this key's sum takes: rows i >= t - (n - m) (causal) and i < m
        const int jmin = t - (n - m) - i0, jmax = m - i0;
        const bool all = __all_sync(0xffffffffu, jmin <= c0 && jmax >= c0 + cols);
        float s0 = 0.f, s1 = 0.f;
        tc_ld_wait();
#pragma unroll
        for (int c = 0; c < cols; c += 32) {
          uint32_t(&v)[32] = va[c / 32];
          tc_ld_done(v);
          if (all) {
            float u0 = 0.f, u1 = 0.f;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {  // scalar on purpose: the packed product measured half as fast
              s0 += ex2_approx(__uint_as_float(v[j]) * sl);
              s1 += ex2_approx(__uint_as_float(v[j + 1]) * sl);
              u0 += ex2_approx(__uint_as_float(v[j + 2]) * sl);
              u1 += ex2_approx(__uint_as_float(v[j + 3]) * sl);
            }
            s0 += u0;
            s1 += u1;
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int col = c0 + c + j;
              const float e = ex2_approx(__uint_as_float(v[j]) * sl);
              s0 += col >= jmin && col < jmax ? e : 0.f;
            }
          }
        }
        sum += s0 + s1;  // tile by tile: a sum of thousands of rows keeps its small terms
        tc_fence_before();
        mbar_arrive(&sempty[buf][kt]);
        ++tiles;
      }
      if (!ok) break;
      // the two halves of the columns meet (in turn in two places: one barrier a unit)
      if (half) half_s[units & 1][kt][tid & 127] = sum;
      mbar_arrive(&hsum);
      if (!(ok = wait(&hsum, units))) break;
      if (!half) {
        sum += half_s[units & 1][kt][tid & 127];
        if (r.whole) {
          if (t < n) {
            const int phys = p.page_table[(size_t)r.b * p.max_pages + (t >> p.pshift)];
            if (phys >= 0 && phys < p.num_phys) p.acc[((size_t)r.b * p.Hkv + r.g) * p.acc_stride + t] += sum;
          }
        } else {
          p.part[(2 * (size_t)blockIdx.x + (r.first ? 0 : 1)) * kAmKeys + key] = sum;
        }
      }
      ++units;
    }
  } else {
    if (warp == 16) {
      if (elect_lane()) {  // one lane: a copy issued from converged code costs 90 clocks
        const int pages = kAmKeys >> p.pshift, box = p.P * 128;
        for (bool more = tiles_find(p, tt, nq, x0, x0, x1, r); ok && more; more = tiles_next(p, tt, nq, x1, r)) {
          const int n = tt.n[r.b], s = units % KS;
          // the unit's page ids: the table's rows are whole groups of eight
          int ids[16];
          const int* at = p.page_table + (size_t)r.b * p.max_pages + r.j * pages;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            int4 id = make_int4(-1, -1, -1, -1);
            if (4 * q < pages && (r.j * pages + 4 * q) * p.P < n) id = *reinterpret_cast<const int4*>(at + 4 * q);
            ids[4 * q] = id.x;
            ids[4 * q + 1] = id.y;
            ids[4 * q + 2] = id.z;
            ids[4 * q + 3] = id.w;
          }
          uint32_t have = 0;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < pages && (r.j * pages + j) * p.P < n) {
              if (ids[j] >= 0 && ids[j] < p.num_phys) have |= 1u << j;
              else flag_error(p.err, RKV_DEVERR_PAGE_ID);
            }
          if (units >= KS && !(ok = wait_one(&kempty[s], units / KS - 1))) break;
          if (have) mbar_arrive_expect_tx(&kfull[s], __popc(have) * 2 * box);
          else mbar_arrive(&kfull[s]);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if ((have >> j) & 1u) {
              const int in = j * p.P, row = (ids[j] * p.Hkv + r.g) * p.P;  // row of the unit's 256, of the pool
              uint8_t* to = ks + s * 65536 + (in >> 7) * 32768 + (in & 127) * 128;
              tma_load_2d(to, &p.tmk, 0, row, &kfull[s]);
              tma_load_2d(to + 16384, &p.tmk, 64, row, &kfull[s]);
            }
          ++units;
          int h = r.lo > 0 ? r.lo / r.width : 0, rt = r.f + r.lo - h * r.width;
          for (int o = r.lo; o < r.hi; ++o) {
            const int t = tiles % kAmQ;
            if (tiles >= kAmQ && !(ok = wait_one(&qempty[t], tiles / kAmQ - 1))) break;
            const int row = (r.b * p.Hq + r.g * p.G + h) * p.T + rt * nq;
            mbar_arrive_expect_tx(&qfull[t], nq * 256);
            tma_load_2d(qs + t * QB, &p.tmq, 0, row, &qfull[t]);
            tma_load_2d(qs + t * QB + QB / 2, &p.tmq, 64, row, &qfull[t]);
            ++tiles;
            if (++rt == r.f + r.width) {
              rt = r.f;
              ++h;
            }
          }
        }
      }
    } else if (warp == 17) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, nq);
      const bool lead = elect_lane();
      const uint32_t klo = sw128_kmajor_lo(smem_u32(ks)), qlo = sw128_kmajor_lo(smem_u32(qs));
      const uint32_t onelo = plain_kmajor_lo(smem_u32(ones)), biaslo = plain_kmajor_lo(smem_u32(bias));
      // The waits stand where products are still queued: inside a unit a query tile is waited
      // for before the second key tile of the one before it is issued.  (Not across units: the
      // next unit's keys, and its query tiles behind them, wait for this unit's products.)
      for (bool more = tiles_find(p, tt, nq, x0, x0, x1, r); ok && more; more = tiles_next(p, tt, nq, x1, r)) {
        const int s = units % KS;
        if (!(ok = wait(&kfull[s], units / KS))) break;
        ++units;
        if (!(ok = wait(&qfull[tiles % kAmQ], tiles / kAmQ))) break;
        for (int o = r.lo; o < r.hi; ++o) {
          const int t = tiles % kAmQ, d = tiles & 1;
          const uint32_t q = qlo + t * (QB >> 4);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (w == 1 && o + 1 < r.hi && !(ok = wait(&qfull[(tiles + 1) % kAmQ], (tiles + 1) / kAmQ))) break;
            if (tiles >= 2 && !(ok = wait(&sempty[d][w], tiles / 2 - 1))) break;
            tc_fence_after();
            const uint32_t to = tmem + d * 256 + w * 128, key = klo + s * (65536 >> 4) + w * (32768 >> 4);
            tc_mma_ss<false>(lead, to, key, q, idesc);
#pragma unroll
            for (int k = 1; k < 8; ++k) {
              const uint32_t in = (k & 3) * 32;
              tc_mma_ss<true>(lead, to, key + (((k >> 2) * 16384 + in) >> 4), q + (((k >> 2) * (QB / 2) + in) >> 4), idesc);
            }
            tc_mma_ss<true, kPlainDescHi>(lead, to, onelo, biaslo + t * (kAmExtra >> 4), idesc);
            tc_commit_if(lead, &sfull[d][w]);
          }
          if (!ok) break;
          tc_commit_if(lead, &qempty[t]);
          tc_commit_if(lead && o + 1 == r.hi, &kempty[s]);
          __syncwarp();
          ++tiles;
        }
      }
      if (ok) {  // the last releases land before the CTA may exit
        for (int i = max(0, tiles - kAmQ); i < tiles; ++i) mbar_wait(&qempty[i % kAmQ], (uint32_t)((i / kAmQ) & 1));
        for (int i = max(0, units - KS); i < units; ++i) mbar_wait(&kempty[i % KS], (uint32_t)((i / KS) & 1));
      }
    } else {
      // two warps take the query tiles in turn; a tile's log-sum-exps are loaded while the
      // one before it (of this warp) is still being written
      const float inv = 1.f / p.scale;
      int before = 0;  // tiles of the runs before
      for (bool more = tiles_find(p, tt, nq, x0, x0, x1, r); ok && more; more = tiles_next(p, tt, nq, x1, r)) {
        const int m = tt.m[r.b];
        int o = r.lo + ((before + warp) & 1);  // warp 18 takes the even tiles of the CTA
        int h = o / r.width, rt = r.f + o - h * r.width;
        auto load = [&](float(&v)[4]) {
          const int i0 = rt * nq;
          const float* src = p.lse + ((size_t)r.b * p.Hq + r.g * p.G + h) * p.T + i0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = o < r.hi && lane + 32 * e < min(nq, m - i0) ? src[lane + 32 * e] : -INFINITY;
        };
        float next[4];
        load(next);
        while (o < r.hi) {
          const int tile = before + o - r.lo, t = tile % kAmQ;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = next[e];
          o += 2;
          rt += 2;
          while (rt >= r.f + r.width) {
            rt -= r.width;
            ++h;
          }
          load(next);
          // -lse / scale in three bf16 terms.  At most 3e38, which bf16 holds: times the smallest
          // scale that is 3e8, and no weight of a row that far off is but 0 or infinite.  A row
          // that weighs nothing takes the lowest.
          uint2 w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a = v[e] == -INFINITY ? -3e38f : -v[e] * inv;
            a = a > 3e38f ? 3e38f : (a < -3e38f ? -3e38f : a);  // a NaN stays one
            const float hi = __bfloat162float(__float2bfloat16_rn(a)), r1 = a - hi;
            const float mid = __bfloat162float(__float2bfloat16_rn(r1));
            w[e] = make_uint2(pack_bf16x2(hi, mid), pack_bf16x2(r1 - mid, 0.f));
          }
          if (tile >= kAmQ && !(ok = wait(&qempty[t], tile / kAmQ - 1))) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = lane + 32 * e;
            if (row < nq) *reinterpret_cast<uint2*>(bias + t * kAmExtra + (row >> 3) * 256 + (row & 7) * 16) = w[e];
          }
          fence_proxy_async_smem();
          mbar_arrive(&qfull[t]);
        }
        before += r.hi - r.lo;
      }
    }
  }

  // teardown: after a timeout, wait (bounded) for the copies and products still in flight
  tc_fence_before();
  __syncthreads();
  if (abort_flag) {
    if (warp == 16) {  // the lane that issued them; the others have none
      for (int i = max(0, tiles - kAmQ); i < tiles; ++i) mbar_wait(&qfull[i % kAmQ], (uint32_t)((i / kAmQ) & 1));
      for (int i = max(0, units - KS); i < units; ++i) mbar_wait(&kfull[i % KS], (uint32_t)((i / KS) & 1));
    }
    if (warp == 17) {  // a tile given up between its two key tiles has one product that no phase counts
      tc_commit_if(elect_lane(), &drained);
      mbar_wait(&drained, 0);
    }
    __syncthreads();
  }
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the parts of the units that were split between CTAs, in the CTAs' order.  grid N,
// 256 threads (keys): CTA c joins the unit that starts in c's share and ends behind it.
__global__ void __launch_bounds__(kAmKeys) accum_join_kernel(const __grid_constant__ RowsParams p) {
  __shared__ TilesTable tt;
  tiles_table(p, tt);
  grid_dependency_wait();
  const long long total = tt.base[p.B];
  const int N = flat_ctas(total, p.N), c = blockIdx.x;
  if (c >= N) return;
  const long long x0 = flat_first(total, c, N), x1 = flat_first(total, c + 1, N);
  TilesRun r;
  tiles_find(p, tt, p.nq, x1 - 1, x0, total, r);
  const long long end = r.x + (r.hi - r.lo);  // the unit's end
  if (r.ux < x0 || end <= x1) return;
  const int last = flat_cta(end - 1, total, N), t = r.j * kAmKeys + threadIdx.x;
  float sum = 0.f;
  for (int i = c; i <= last; ++i)
    sum += p.part[(2 * (size_t)i + (flat_first(total, i, N) >= r.ux ? 0 : 1)) * kAmKeys + threadIdx.x];
  if (t < tt.n[r.b]) {
    const int phys = p.page_table[(size_t)r.b * p.max_pages + (t >> p.pshift)];
    if (phys >= 0 && phys < p.num_phys) p.acc[((size_t)r.b * p.Hkv + r.g) * p.acc_stride + t] += sum;
  }
}

// ---------------------------------------------------------------------------
// evict
// Positions that one CTA selects from by itself: 1000, 2000 and 4096 of them took 10.0, 11.2
// and 12.4 us, a cluster 12.5, 14.9 and 14.7.
constexpr int kSelectOne = 8192;

struct EvictParams {
  rkv_cache src, dst;
  int in_place;
  const float* acc;
  float* dst_acc;
  int acc_stride, dst_acc_stride, recent, kept_stride, stage_stride;
  int32_t* kept;        // [B][Hkv][kept_stride]
  int32_t* count;       // [B] tokens kept (workspace); -1: not touched
  rkv_bf16* stage_k;    // in place: [B][Hkv][stage_stride][128], else null
  rkv_bf16* stage_v;
  float* stage_acc;     // [B][Hkv][stage_stride]
  int cgroup;
  int32_t keep[RKV_MAX_BATCH];
};

__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = p.src.seq_len[b];
  return n < 0 || n > p.src.max_pages * p.src.page_size ? 0 : n;
}

// Kept positions, ascending.  A cluster of C CTAs per unit, grid (C, B*Hkv).  33 us for the
// ragged batch (clusters of 1, 4 and 8: 45, 42, 85); cluster barriers and passes over
// shared memory, not bytes.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t skeys[];
  __shared__ union {
    SelectSmem cluster;
    TopkSmem<kSelectThreads> block;
  } ss;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int unit = blockIdx.y, b = unit / p.src.Hkv, tid = threadIdx.x;
  const int n = evict_len(p, b), keep = p.keep[b];
  int32_t* out = p.kept + (size_t)unit * p.kept_stride;
  if (rank == 0 && tid == 0 && unit % p.src.Hkv == 0) {
    const bool usable = n == p.src.seq_len[b];
    if (!usable) flag_error(p.src.error_word, RKV_DEVERR_CAPACITY);
    p.count[b] = usable || !p.in_place ? min(n, keep) : -1;  // in place: left as it is
  }
  if (n <= keep) {  // the same branch in every CTA of the cluster
    for (int i = rank * kSelectThreads + tid; i < n; i += C * kSelectThreads) out[i] = i;
    return;
  }
  const int recent = p.recent, Lp = n - recent, k = keep - recent;  // recent <= keep < n
  if (rank == 0)
    for (int i = tid; i < recent; i += kSelectThreads) out[k + i] = Lp + i;
  if (k == 0) return;
  const float* acc = p.acc + (size_t)unit * p.acc_stride;
  // a NaN counts as the heaviest, and both zeros as one
  auto load = [&](int t) {
    const float v = acc[t];
    return v != v ? __int_as_float(0x7fffffff) : v + 0.f;
  };
  if (C > 1) {
    cluster_select(Lp, k, load, out, skeys, ss.cluster);
    return;
  }
  // one CTA: the same select over the block, without the cluster's barriers
  for (int i0 = tid; i0 < Lp; i0 += 8 * kSelectThreads) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i0 + j * kSelectThreads < Lp ? load(i0 + j * kSelectThreads) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j * kSelectThreads < Lp) skeys[i0 + j * kSelectThreads] = float_key(v[j]);
  }
  __syncthreads();
  topk_adaptive_fn<kSelectThreads>(Lp, k, [&](int i) { return skeys[i]; }, ss.block, [&](int at, int i) { out[at] = i; });
}

// Row i of a unit's kept list in the source cache; null when its page id is out of range.
__device__ __forceinline__ bool evict_source(const EvictParams& p, int b, int g, int t, size_t& row) {
  const int P = p.src.page_size;
  const int phys = p.src.page_table[(size_t)b * p.src.max_pages + t / P];
  if (phys < 0 || phys >= p.src.num_phys_pages) {
    flag_error(p.src.error_word, RKV_DEVERR_PAGE_ID);
    return false;
  }
  row = (((size_t)phys * p.src.Hkv + g) * P + t % P) * 128;
  return true;
}

// In place only: the rows that move, into the workspace, before any page is written.
// grid (ceil(max keep / 64), Hkv, B), 256 threads: 16 rows x 16 pieces of 16 bytes.
__global__ void __launch_bounds__(256) evict_stage_kernel(const __grid_constant__ EvictParams p) {
  const int b = blockIdx.z, g = blockIdx.y, n = p.count[b];
  const size_t unit = (size_t)b * p.src.Hkv + g;
  const int piece = threadIdx.x & 15;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = blockIdx.x * 64 + j * 16 + (threadIdx.x >> 4);
    if (i >= n) continue;
    const int t = p.kept[unit * p.kept_stride + i];
    if (t == i) continue;
    const size_t to = unit * p.stage_stride + i;
    size_t row;
    if (evict_source(p, b, g, t, row)) {
      reinterpret_cast<uint4*>(p.stage_k + to * 128)[piece] = reinterpret_cast<const uint4*>(p.src.k_pages + row)[piece];
      reinterpret_cast<uint4*>(p.stage_v + to * 128)[piece] = reinterpret_cast<const uint4*>(p.src.v_pages + row)[piece];
    }
    if (piece == 0) p.stage_acc[to] = p.acc[unit * p.acc_stride + t];
  }
}

// Kept rows into the destination's pages, their summaries, their weights (zero behind
// them) and the new lengths.  grid (ceil(max keep / (cgroup P)), Hkv, B), 128 threads: a
// CTA fills cgroup <= 8 consecutive pages; thread t moves 16-byte piece t % 16 of rows
// t / 16, t / 16 + 8, ... and keeps their max / min, which a shuffle and a pass over the
// four warps combine into the page's column of a [channel][8 pages] tile, so that with
// groups of eight a channel's summaries go out as one 16-byte store.  The bytes bound it:
// the ragged batch cut to 8192 tokens moves 1.04 GB in 173 us, 6.0 TB/s, 88 % of a plain
// copy's rate.
template <int kRows>  // rows per thread: page size / 8
__global__ void __launch_bounds__(128) evict_compact_kernel(const __grid_constant__ EvictParams p) {
  constexpr int P = 8 * kRows;
  __shared__ float red[2][4][128];
  __shared__ int32_t idx[8 * P];
  __shared__ __align__(16) uint16_t tile[2][128][8];
  const int b = blockIdx.z, g = blockIdx.y, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const size_t unit = (size_t)b * p.src.Hkv + g;
  const int n = p.count[b];
  const int pg0 = blockIdx.x * p.cgroup;
  if (n < 0) return;
  if (blockIdx.x == 0 && g == 0 && tid == 0) p.dst.seq_len[b] = n;
  // the weights behind the kept ones start again at zero
  for (int t = n + blockIdx.x * 128 + tid; t < p.dst_acc_stride; t += gridDim.x * 128)
    p.dst_acc[unit * p.dst_acc_stride + t] = 0.f;
  if (pg0 * P >= n) return;
  const int npg = min(p.cgroup, (n + P - 1) / P - pg0);
  const int r_end = min(p.cgroup * P, n - pg0 * P);
  const int32_t* kept = p.kept + unit * p.kept_stride + (size_t)pg0 * P;
  for (int r = tid; r < r_end; r += 128) {
    const int t = kept[r], i = pg0 * P + r;
    idx[r] = t;
    if (!p.in_place)
      p.dst_acc[unit * p.dst_acc_stride + i] = p.acc[unit * p.acc_stride + t];
    else if (t != i)
      p.dst_acc[unit * p.dst_acc_stride + i] = p.stage_acc[unit * p.stage_stride + i];
  }
  __syncthreads();
  const int piece = tid & 15, rg = tid >> 4;
  for (int q = 0; q < npg; ++q) {
    const int pg = pg0 + q;
    const int phys = p.dst.page_table[(size_t)b * p.dst.max_pages + pg];
    const bool page_ok = phys >= 0 && phys < p.dst.num_phys_pages;
    if (!page_ok && tid == 0) flag_error(p.dst.error_word, RKV_DEVERR_PAGE_ID);
    const int cnt = min(P, n - pg * P);
    const size_t dst0 = (((size_t)(page_ok ? phys : 0) * p.dst.Hkv + g) * P) * 128 + piece * 8;
    uint4 kv[kRows], vv[kRows];
    bool have[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = rg + 8 * j, i = pg * P + r;
      have[j] = r < cnt;
      kv[j] = make_uint4(0, 0, 0, 0);
      vv[j] = make_uint4(0, 0, 0, 0);
      if (!have[j]) continue;
      const int t = idx[q * P + r];
      size_t row;
      have[j] = evict_source(p, b, g, t, row);  // a row that cannot be read was not staged either
      if (!have[j]) continue;
      const bool moved = p.in_place && t != i;
      if (moved) row = (unit * p.stage_stride + i) * 128;
      kv[j] = *reinterpret_cast<const uint4*>((moved ? p.stage_k : p.src.k_pages) + row + piece * 8);
      vv[j] = *reinterpret_cast<const uint4*>((moved ? p.stage_v : p.src.v_pages) + row + piece * 8);
    }
    float mx[8], mn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mx[e] = -INFINITY;
      mn[e] = INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (!have[j]) continue;
      const int r = rg + 8 * j;
      if (page_ok) {
        *reinterpret_cast<uint4*>(p.dst.k_pages + dst0 + (size_t)r * 128) = kv[j];
        *reinterpret_cast<uint4*>(p.dst.v_pages + dst0 + (size_t)r * 128) = vv[j];
      }
      const uint32_t w4[4] = {kv[j].x, kv[j].y, kv[j].z, kv[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a0 = bf16_lo(w4[e]), a1 = bf16_hi(w4[e]);
        mx[2 * e] = fmaxf(mx[2 * e], a0);
        mx[2 * e + 1] = fmaxf(mx[2 * e + 1], a1);
        mn[2 * e] = fminf(mn[2 * e], a0);
        mn[2 * e + 1] = fminf(mn[2 * e + 1], a1);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // lanes l and l ^ 16 hold the same piece
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
      mn[e] = fminf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], 16));
    }
    if (lane < 16) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        red[0][warp][piece * 8 + e] = mx[e];
        red[1][warp][piece * 8 + e] = mn[e];
      }
    }
    __syncthreads();
    const float M = fmaxf(fmaxf(red[0][0][tid], red[0][1][tid]), fmaxf(red[0][2][tid], red[0][3][tid]));
    const float m = fminf(fminf(red[1][0][tid], red[1][1][tid]), fminf(red[1][2][tid], red[1][3][tid]));
    // the values came from bf16 bit patterns, so the top 16 bits are exact
    tile[0][tid][q] = (uint16_t)(__float_as_uint(M) >> 16);
    tile[1][tid][q] = (uint16_t)(__float_as_uint(m) >> 16);
    __syncthreads();  // red is reused by the next page
  }
  const size_t row = (unit * 128 + tid) * p.dst.max_pages + pg0;
  if (npg == 8) {  // cgroup == 8: 16-byte aligned (max_pages is a multiple of 8)
    *reinterpret_cast<uint4*>(p.dst.kmax + row) = *reinterpret_cast<const uint4*>(&tile[0][tid][0]);
    *reinterpret_cast<uint4*>(p.dst.kmin + row) = *reinterpret_cast<const uint4*>(&tile[1][tid][0]);
  } else {
    for (int q = 0; q < npg; ++q) {
      p.dst.kmax[row + q] = tile[0][tid][q];
      p.dst.kmin[row + q] = tile[1][tid][q];
    }
  }
}

}  // namespace

size_t accum_rows_ws_bytes(int, int, int, int, int, int) { return (size_t)2 * kMaxSms * kAmKeys * 4; }

cudaError_t launch_accum_rows(const AccumRowsArgs& a, cudaStream_t s) {
  const rkv_cache& c = a.cache;
  RowsParams p;
  // Up to two staged blocks of 64 rows of a KV head go to accum_rows (30 rows x 4 heads, 1 x
  // 16K tokens: 26 us against 34 with the join; 32 x 4, 4 x 16K: 78 against 74; 48 x 4: 112
  // against 75); so do rows picked by id, which only it gathers.
  const bool tiles = !a.row_ids && (long long)a.T * (a.Hq / c.Hkv) > 2 * kRwBlock;
  p.nq = a.T > 64 ? 128 : 64;
  bool ok = encode_rows_map(&p.tmk, c.k_pages, (uint64_t)c.num_phys_pages * c.Hkv * c.page_size,
                            tiles ? (uint32_t)c.page_size : (uint32_t)kRwKeys);
  if (tiles) ok = ok && encode_rows_map(&p.tmq, a.q, (uint64_t)c.B * a.Hq * a.T, (uint32_t)p.nq);
  if (!ok) {
    set_last_error("cuTensorMapEncodeTiled failed for the cache's pages or the queries");
    return cudaErrorInvalidValue;
  }
  p.q = a.q;
  p.lse = a.lse;
  p.row_len = a.row_len;
  p.row_ids = a.row_ids;
  p.page_table = c.page_table;
  p.seq_len = c.seq_len;
  p.err = c.error_word;
  p.acc = a.acc;
  p.B = c.B;
  p.Hq = a.Hq;
  p.Hkv = c.Hkv;
  p.G = a.Hq / c.Hkv;
  p.gshift = log2_int(p.G);
  p.T = a.T;
  p.ids_stride = a.ids_stride;
  p.P = c.page_size;
  p.pshift = log2_int(c.page_size);
  p.max_pages = c.max_pages;
  p.num_phys = c.num_phys_pages;
  p.acc_stride = a.acc_stride;
  p.N = num_sms();
  p.scale = a.scale;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  if (p.N > kMaxSms) p.N = kMaxSms;
  p.part = static_cast<float*>(a.ws);
  cudaError_t e;
  if (tiles) {
    static SmemOptIn opt[2];
    void (*kernel)(RowsParams) = p.nq == 128 ? accum_tiles_kernel<128> : accum_tiles_kernel<64>;
    if ((e = opt[p.nq == 128].raise(reinterpret_cast<const void*>(kernel), kAmSmem)) != cudaSuccess) return e;
    launch_begin(K_ACCUM_TILES, s);
    kernel<<<p.N, kAmThreads, kAmSmem, s>>>(p);
    launch_end(K_ACCUM_TILES, s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_dependent(accum_join_kernel, dim3(p.N), kAmKeys, K_ACCUM_JOIN, s, p);
  }
  const long long most = (long long)(a.row_ids ? a.ids_stride : a.T) * p.G;
  void (*kernel)(RowsParams) = most <= 16 ? accum_rows_kernel<1> : (most <= 32 ? accum_rows_kernel<2> : accum_rows_kernel<4>);
  static SmemOptIn opt[3];
  if ((e = opt[most <= 16 ? 0 : (most <= 32 ? 1 : 2)].raise(reinterpret_cast<const void*>(kernel), kRwSmem)) != cudaSuccess)
    return e;
  launch_begin(K_ACCUM_ROWS, s);
  kernel<<<p.N, most <= 32 ? RowsShape<2>::kWarps * 32 : RowsShape<4>::kWarps * 32, kRwSmem, s>>>(p);
  launch_end(K_ACCUM_ROWS, s);
  return cudaGetLastError();
}

int evict_max_tokens() { return kSelectMaxCluster * kSelectSliceMax; }

size_t evict_ws_bytes(int B, int Hkv, int max_keep, bool in_place) {
  size_t n = align256((size_t)B * 4);
  if (in_place) {
    const size_t rows = (size_t)B * Hkv * max_keep;
    n += 2 * align256(rows * 256) + align256(rows * 4);
  }
  return n;
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const rkv_cache& c = a.cache;
  EvictParams p;
  p.src = c;
  p.dst = a.dst;
  p.in_place = a.in_place;
  p.acc = a.acc;
  p.dst_acc = a.dst_acc;
  p.acc_stride = a.acc_stride;
  p.dst_acc_stride = a.dst_acc_stride;
  p.recent = a.recent;
  p.kept = a.kept_idx;
  p.kept_stride = a.kept_stride;
  int keep_max = 1;
  for (int b = 0; b < c.B; ++b) {
    p.keep[b] = a.keep[b];
    keep_max = a.keep[b] > keep_max ? a.keep[b] : keep_max;
  }
  uint8_t* w = static_cast<uint8_t*>(a.ws);
  p.count = reinterpret_cast<int32_t*>(w);
  w += align256((size_t)c.B * 4);
  p.stage_k = p.stage_v = nullptr;
  p.stage_acc = nullptr;
  p.stage_stride = keep_max;
  const size_t rows = (size_t)c.B * c.Hkv * keep_max;
  if (a.in_place) {
    p.stage_k = reinterpret_cast<rkv_bf16*>(w);
    w += align256(rows * 256);
    p.stage_v = reinterpret_cast<rkv_bf16*>(w);
    w += align256(rows * 256);
    p.stage_acc = reinterpret_cast<float*>(w);
  }
  // select: one CTA up to 8192 positions; about 4096 positions a CTA beyond, clusters of up to
  // 8 while the units leave SMs idle and of 2 once they cover them, wide enough for the
  // slices to fit
  const int units = c.B * c.Hkv, cap = c.max_pages * c.page_size;
  int C = cap <= kSelectOne ? 1 : (cap + 4095) / 4096;
  const int by_units = num_sms() / units > 2 ? num_sms() / units : 2;
  const int by_smem = (cap + kSelectSliceMax - 1) / kSelectSliceMax;
  C = C < by_units ? C : by_units;
  C = C > by_smem ? C : by_smem;
  C = C > kSelectMaxCluster ? kSelectMaxCluster : C;
  static SmemOptIn opt;
  cudaError_t e = opt.raise(reinterpret_cast<const void*>(evict_select_kernel), kSelectSliceMax * 4);
  if (e != cudaSuccess) return e;
  {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, (unsigned)units, 1);
    cfg.blockDim = dim3(kSelectThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)((cap + C - 1) / C) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    launch_begin(K_EVICT_SELECT, s);
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
    launch_end(K_EVICT_SELECT, s);
    if (e != cudaSuccess) return e;
  }
  if (a.in_place) {
    launch_begin(K_EVICT_STAGE, s);
    evict_stage_kernel<<<dim3((keep_max + 63) / 64, c.Hkv, c.B), 256, 0, s>>>(p);
    launch_end(K_EVICT_STAGE, s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int P = c.page_size;
  p.cgroup = 8;
  while (p.cgroup > 1 && (long)((keep_max + p.cgroup * P - 1) / (p.cgroup * P)) * units < 16L * num_sms()) p.cgroup /= 2;
  const dim3 grid((keep_max + p.cgroup * P - 1) / (p.cgroup * P), c.Hkv, c.B);
  launch_begin(K_EVICT_COMPACT, s);
  if (P == 16)
    evict_compact_kernel<2><<<grid, 128, 0, s>>>(p);
  else if (P == 32)
    evict_compact_kernel<4><<<grid, 128, 0, s>>>(p);
  else
    evict_compact_kernel<8><<<grid, 128, 0, s>>>(p);
  launch_end(K_EVICT_COMPACT, s);
  return cudaGetLastError();
}

}  // namespace rkv
