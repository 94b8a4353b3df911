// Dense attention of a few query rows over the paged cache: the one-token step that
// keeps count of every position's weight, and the tree of drafted tokens.
//
// For unit (sequence b, KV head g), query rows r = t G + h (node t, head h of the group),
// keys j = the cache's n tokens and, for a tree, the drafted nodes row t may see:
//   z_rj = scale q_r . k_j,  out_r = sum_j exp(z_rj) v_j / sum_j exp(z_rj),
//   lse_r = log sum_j exp(z_rj),  acc_j += sum_r exp(z_rj - lse_r)   (one token only)
// A row that sees nothing has out = 0 and lse = -inf.
//
// attend_rows: 16 query rows against 16-key chunks.  A chunk's K and V are 8 KB for 16 x
// 16 x 128 x 2 multiply-adds, so the cache's bytes bound it: all units' chunks form one
// line that is split evenly over one CTA per SM (rkv_flat.cuh); a CTA's eight warps take
// a run's chunks in turn, each with its own three-stage TMA ring (192 KB in flight per SM
// keep HBM busy), its own running maximum, sum and fp32 output, and meet once per run.  A
// run that is a whole unit is final; the parts of a split unit go to the workspace and
// attend_combine joins them.  Measured: 16 x 20000 tokens, 8 KV heads (1.31 GB) 209 us,
// 6.3 TB/s, 92 % of a plain copy's rate; with the logits kept, the ragged batch of 16 x 8K
// .. 32K (1.22 GB) 210 us.
#include <cooperative_groups.h>

#include "rkv_flat.cuh"
#include "rkv_internal.h"

namespace rkv {
namespace {

constexpr int kArRows = 16;                       // query rows of a tile (the MMA's M)
constexpr int kArKeys = 16;                       // keys of a chunk
constexpr int kArWarps = 8;
constexpr int kArThreads = kArWarps * 32;
constexpr int kArStages = 3;
constexpr int kArStageBytes = 4 * 2048;           // K, V: two 16 x 64 boxes each
constexpr int kArMergeRows = 4;                   // rows of every warp that meet at a time
constexpr int kArMergeFloats = kArWarps * kArMergeRows * 128;
constexpr int kArSmem = 1024 + kArWarps * kArStages * kArStageBytes + kArMergeFloats * 4;
constexpr int kArPad = 16, kAtPad = 4;           // what a run costs, in chunks of 16 and tiles of 128 keys
// Running maximum of a row that saw nothing: no logit lies below it, and differences with
// it are never inf - inf.
constexpr float kNoMax = -3.402823466e+38f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWeighTokens = 2048;                // tokens of a weighing block, eight a thread

struct AttendParams {
  CUtensorMap tmk, tmv;    // the page pools as [rows][128] bf16, 16-row x 64-channel boxes (the tiled
                           // kernel: a page's rows)
  CUtensorMap tmkt, tmvt;  // the tree's keys and values, the same boxes (the tiled kernel: 128 rows)
  const rkv_bf16* q;       // [B][Hq][T][128]
  const uint32_t* mask;    // [B][T][words], null: no tree
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* tree_len;  // null: T nodes everywhere
  int32_t* err;
  rkv_bf16* out;            // [B][Hq][T][128]
  float* lse;               // [B][Hq][T], may be null
  float* part_o;            // [2 N][tile rows][128]
  float2* part_ml;          // [2 N][tile rows]
  float2* row_ml;           // [B][Hkv][G]: final (m, l) of a one-token step, for the weights
  float* z;                 // [B][Hkv][G][zstride] base-2 scaled logits of a one-token step, or null
  float* acc;               // [B][Hkv][acc_stride]
  int B, Hq, Hkv, G, gshift, T, words, P, pshift, max_pages, num_phys, zstride, acc_stride, N;
  int row_tiles;            // attend_units: 16-row tiles of a KV head
  float scale_log2;
};

__device__ __forceinline__ int checked_len(const AttendParams& p, int b) {
  const int n = p.seq_len[b];
  if (n < 0 || n > p.max_pages * p.P) {
    flag_error(p.err, RKV_DEVERR_CAPACITY);
    return 0;
  }
  return n;
}
__device__ __forceinline__ int checked_nodes(const AttendParams& p, int b) {
  const int t = p.tree_len ? p.tree_len[b] : p.T;
  if (t < 0 || t > p.T) {
    flag_error(p.err, RKV_DEVERR_TREE);
    return 0;
  }
  return t;
}

// Empty pieces of a unit: a run's start and end in chunks and tiles.
template <int kKeys>
__device__ __forceinline__ constexpr int pad_of() { return kKeys == kArKeys ? kArPad : kAtPad; }

template <int kRows, int kKeys>
__device__ __forceinline__ void build_table(const AttendParams& p, FlatTable& ft) {
  flat_build(
      ft, p.B, pad_of<kKeys>(), [&](int b) { return checked_len(p, b); }, [&](int b) { return checked_nodes(p, b); },
      [&](int n, int t) { return (n + kKeys - 1) / kKeys + (p.mask ? (t + kKeys - 1) / kKeys : 0); },
      [&](int t) { return p.Hkv * ((t * p.G + kRows - 1) / kRows); });
}

// Rows 16 rt .. of unit (b, g): node and head of row r.
__device__ __forceinline__ size_t out_row(const AttendParams& p, int b, int g, int r) {
  return ((size_t)b * p.Hq + g * p.G + (r & (p.G - 1))) * p.T + (r >> p.gshift);
}

// A row's results from its maximum m and sum l.  l = 0: it saw nothing, and nothing is what it
// weighs; a NaN among its logits has left l a NaN, which stays one.
__device__ __forceinline__ float inverse_of(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }
// What turns base-2 logits into weights, 2^(z - m) / l: not 2^(z - log-sum-exp), whose sum
// m + log2 l keeps nothing of l once m is past 2^24.
__device__ __forceinline__ float2 norm_of(float m, float l) { return make_float2(m, inverse_of(l)); }

// A warp's share of a 16-row tile: the queries as A fragments (eight steps of 16
// channels), the running maximum, sum and fp32 output of fragment rows r0 = lane / 4 and
// r1 = r0 + 8 of the tile.
struct RowTile {
  uint32_t qa[8][4];
  float o[16][4];
  float m0, m1, l0, l1;
  int b, r0, r1, rows, nc, n, nodes;  // rows: live query rows of the KV head; nc: cache chunks

  __device__ __forceinline__ void start(const AttendParams& p, int b_, int g, int rt, int n_, int nodes_) {
    const int lane = threadIdx.x & 31;
    b = b_;
    n = n_;
    nodes = nodes_;
    rows = nodes * p.G;
    nc = (n + kArKeys - 1) / kArKeys;
    r0 = rt * kArRows + (lane >> 2);
    r1 = r0 + 8;
    const uint32_t* q0 = reinterpret_cast<const uint32_t*>(p.q + out_row(p, b, g, r0) * 128);
    const uint32_t* q1 = reinterpret_cast<const uint32_t*>(p.q + out_row(p, b, g, r1) * 128);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      qa[k][0] = r0 < rows ? q0[k * 8 + (lane & 3)] : 0u;
      qa[k][1] = r1 < rows ? q1[k * 8 + (lane & 3)] : 0u;
      qa[k][2] = r0 < rows ? q0[k * 8 + 4 + (lane & 3)] : 0u;
      qa[k][3] = r1 < rows ? q1[k * 8 + 4 + (lane & 3)] : 0u;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    m0 = m1 = kNoMax;
    l0 = l1 = 0.f;
  }

  // One chunk, K and V in st (its copy has landed).  save(z, col): base-2 logits of row r0
  // at columns col, col + 1 of the chunk, -inf where masked.
  template <class Save>
  __device__ __forceinline__ void step(const AttendParams& p, uint8_t* st, int c, Save save) {
    const int lane = threadIdx.x & 31, qc = (lane & 3) * 2;
    const int left = c < nc ? n - c * kArKeys : nodes - (c - nc) * kArKeys;  // keys of the chunk from here on
    if (left < kArKeys) {  // what lies behind the last key may be anything: 0 x NaN is not 0
      for (int i = lane; i < 2 * (kArKeys - left) * 8; i += 32) {
        const int half = i & 1, rest = i >> 1;
        *reinterpret_cast<uint4*>(st + 4096 + half * 2048 + (left + (rest >> 3)) * 128 + (rest & 7) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    const uint32_t ks = smem_u32(st), vs = ks + 4096;
    float z[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    {
      const int key = ((lane >> 4) << 3) + (lane & 7), sub = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int piece = k * 2 + sub;
        uint32_t b0, b1, b2, b3;
        ldsm_x4(b0, b1, b2, b3, ks + (piece >> 3) * 2048 + key * 128 + (((piece & 7) ^ (key & 7)) << 4));
        mma_16816(z[0], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b0, b1);
        mma_16816(z[1], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b2, b3);
      }
    }
    // base-2 logits; masked ones -inf
    uint32_t see0 = left >= kArKeys ? 0xffffu : (1u << left) - 1u, see1 = see0;
    if (c >= nc) {
      const int j0 = (c - nc) * kArKeys;
      const uint32_t* mk = p.mask + (size_t)b * p.T * p.words + (j0 >> 5);
      see0 &= r0 < rows ? mk[(size_t)(r0 >> p.gshift) * p.words] >> (j0 & 31) : 0u;
      see1 &= r1 < rows ? mk[(size_t)(r1 >> p.gshift) * p.words] >> (j0 & 31) : 0u;
    }
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = h * 8 + qc + e;
        z[h][e] = (see0 >> col) & 1u ? z[h][e] * p.scale_log2 : -INFINITY;
        z[h][2 + e] = (see1 >> col) & 1u ? z[h][2 + e] * p.scale_log2 : -INFINITY;
        mx0 = fmaxf(mx0, z[h][e]);
        mx1 = fmaxf(mx1, z[h][2 + e]);
      }
    save(make_float2(z[0][0], z[0][1]), qc);
    save(make_float2(z[1][0], z[1][1]), qc + 8);
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
    const float f0 = ex2_approx(m0 - n0), f1 = ex2_approx(m1 - n1);
    m0 = n0;
    m1 = n1;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        z[h][e] = ex2_approx(z[h][e] - n0);
        z[h][2 + e] = ex2_approx(z[h][2 + e] - n1);
        s0 += z[h][e];
        s1 += z[h][2 + e];
      }
    l0 = l0 * f0 + s0;  // this thread's columns; the four lanes of a row add up at the end
    l1 = l1 * f1 + s1;
    if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][0] *= f0;
        o[j][1] *= f0;
        o[j][2] *= f1;
        o[j][3] *= f1;
      }
    }
    // The weights enter the second product as bf16 (off by at most 2^-8 of each, as
    // the values they multiply and the output are); their sum stays unrounded.
    const uint32_t a0 = pack_bf16x2(z[0][0], z[0][1]), a1 = pack_bf16x2(z[0][2], z[0][3]);
    const uint32_t a2 = pack_bf16x2(z[1][0], z[1][1]), a3 = pack_bf16x2(z[1][2], z[1][3]);
    const int key = (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int piece = j * 2 + (lane >> 4);
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(b0, b1, b2, b3, vs + (piece >> 3) * 2048 + key * 128 + (((piece & 7) ^ (key & 7)) << 4));
      mma_16816(o[2 * j], a0, a1, a2, a3, b0, b1);
      mma_16816(o[2 * j + 1], a0, a1, a2, a3, b2, b3);
    }
  }

  // The four lanes of a row add their sums up.
  __device__ __forceinline__ void finish() {
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  }
};

__global__ void __launch_bounds__(kArThreads, 1) attend_rows_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ FlatTable ft;
  __shared__ uint64_t full_b[kArWarps][kArStages];
  __shared__ float wm[kArWarps][kArRows], wl[kArWarps][kArRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* base = align1024(smem);
  uint8_t* ring = base + warp * kArStages * kArStageBytes;
  float* merge = reinterpret_cast<float*>(base + kArWarps * kArStages * kArStageBytes);
  if (lane == 0) {
    for (int s = 0; s < kArStages; ++s) mbar_init(&full_b[warp][s], 1);
    fence_mbar_init();
  }
  build_table<kArRows, kArKeys>(p, ft);
  grid_launch_dependents();
  const long long total = ft.base[p.B];
  const int N = flat_ctas(total, p.N);
  if (blockIdx.x >= N) return;
  const long long x0 = flat_first(total, blockIdx.x, N), x1 = flat_first(total, blockIdx.x + 1, N);

  // this warp's chunks of a run: lo + warp, lo + warp + 8, ...  The fetch side walks the
  // runs ahead of the compute side.
  FlatRun fr;
  long long fx = x0;
  bool more = flat_run(ft, p.B, fx, x0, x1, fr);
  int fc = fr.lo + warp;
  auto settle = [&]() {  // the next chunk to fetch, past runs in which this warp has none left
    while (more && fc >= fr.hi) {
      fx = fr.next;
      more = flat_run(ft, p.B, fx, x0, x1, fr);
      if (more) fc = fr.lo + warp;
    }
  };
  settle();
  // page ids of the run's next 32 chunks of this warp, one a lane: a load per 32 chunks
  // instead of one, with its latency, in front of every copy
  int ids = 0, ids_at = -1;  // ids: for chunks ids_at + 8 lane of the fetch run
  long long ids_x = -1;
  const uint64_t policy = l2_policy(p.T * p.G <= kArRows);  // one row tile: nobody reads the cache again
  int fetched = 0, used = 0;
  bool dead = false;
  // the stages of this ring that hold no copy: a page id out of range (its keys are skipped)
  uint32_t skipped = 0;
  auto fetch = [&]() {
    if (!more) return;
    const int s = fetched % kArStages;
    const int g = fr.unit % p.Hkv;
    const int nc = (ft.n[fr.b] + kArKeys - 1) / kArKeys;
    bool ok = true;
    int row;
    if (fc < nc) {
      const int t0 = fc * kArKeys;
      if (ids_x != fr.x || fc >= ids_at + 32 * kArWarps) {
        ids_x = fr.x;
        ids_at = fc;
        const int c = fc + lane * kArWarps;
        ids = c < min(fr.hi, nc) ? p.page_table[(size_t)fr.b * p.max_pages + ((c * kArKeys) >> p.pshift)] : -1;
      }
      const int phys = __shfl_sync(0xffffffffu, ids, (fc - ids_at) / kArWarps);
      ok = phys >= 0 && phys < p.num_phys;
      row = (phys * p.Hkv + g) * p.P + (t0 & (p.P - 1));
    } else {
      row = (fr.b * p.Hkv + g) * p.T + (fc - nc) * kArKeys;
    }
    if (ok) {
      skipped &= ~(1u << s);
      if (lane == 0) {
        const CUtensorMap* mk = fc < nc ? &p.tmk : &p.tmkt;
        const CUtensorMap* mv = fc < nc ? &p.tmv : &p.tmvt;
        uint8_t* st = ring + s * kArStageBytes;
        uint64_t* bar = &full_b[warp][s];
        mbar_arrive_expect_tx(bar, kArStageBytes);
        tma_load_2d_hint(st, mk, 0, row, bar, policy);
        tma_load_2d_hint(st + 2048, mk, 64, row, bar, policy);
        tma_load_2d_hint(st + 4096, mv, 0, row, bar, policy);
        tma_load_2d_hint(st + 6144, mv, 64, row, bar, policy);
      }
    } else {
      skipped |= 1u << s;
      if (lane == 0) {
        flag_error(p.err, RKV_DEVERR_PAGE_ID);
        mbar_arrive(&full_b[warp][s]);
      }
    }
    ++fetched;
    fc += kArWarps;
    settle();
  };
  for (int s = 0; s < kArStages; ++s) fetch();

  const int qr = lane >> 2, qc = (lane & 3) * 2;  // fragment row and column pair
  FlatRun cr;
  RowTile tile;
  for (long long x = x0; flat_run(ft, p.B, x, x0, x1, cr); x = cr.next) {
    const int b = cr.b, g = cr.unit % p.Hkv, rt = cr.unit / p.Hkv;
    tile.start(p, b, g, rt, ft.n[b], ft.t[b]);
    const int rows = tile.rows;
    float* const zu = p.z + ((size_t)(b * p.Hkv + g) * p.G) * p.zstride;
    for (int c = cr.lo + warp; c < cr.hi; c += kArWarps) {
      const int s = used % kArStages;
      const bool late = !dead && !mbar_wait(&full_b[warp][s], (uint32_t)((used / kArStages) & 1));
      if (__any_sync(0xffffffffu, late)) {
        if (lane == 0) flag_error(p.err, RKV_DEVERR_TIMEOUT);
        dead = true;
      }
      if (!dead && !((skipped >> s) & 1u)) {
        tile.step(p, ring + s * kArStageBytes, c, [&](float2 z, int col) {
          if (p.z && tile.r0 < rows)
            *reinterpret_cast<float2*>(zu + (size_t)tile.r0 * p.zstride + (size_t)c * kArKeys + col) = z;
        });
      } else if (p.z) {  // nothing was read: the positions weigh nothing
        for (int i = lane; i < rows * kArKeys; i += 32)
          zu[(size_t)(i / kArKeys) * p.zstride + (size_t)c * kArKeys + i % kArKeys] = -INFINITY;
      }
      ++used;
      __syncwarp();  // every lane has read the stage
      if (!dead) fetch();
    }

    tile.finish();
    if ((lane & 3) == 0) {
      wm[warp][qr] = tile.m0;
      wl[warp][qr] = tile.l0;
      wm[warp][qr + 8] = tile.m1;
      wl[warp][qr + 8] = tile.l1;
    }
    // the warps meet, four rows at a time: thread = (row, two channels)
    const int live = min(kArRows, rows - rt * kArRows);
    const size_t slot = 2 * (size_t)blockIdx.x + (cr.first ? 0 : 1);
#pragma unroll
    for (int quarter = 0; quarter < 4; ++quarter) {
      if (quarter * kArMergeRows >= live) break;
      if ((qr >> 2) == (quarter & 1)) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          *reinterpret_cast<float2*>(merge + (warp * kArMergeRows + (qr & 3)) * 128 + j * 8 + qc) =
              make_float2(tile.o[j][(quarter >> 1) * 2], tile.o[j][(quarter >> 1) * 2 + 1]);
      }
      __syncthreads();
      const int sub = tid >> 6, d = (tid & 63) * 2, row = quarter * kArMergeRows + sub, r = rt * kArRows + row;
      if (row < live) {
        float M = kNoMax, L = 0.f, ax = 0.f, ay = 0.f;
#pragma unroll
        for (int w = 0; w < kArWarps; ++w) M = fmaxf(M, wm[w][row]);
#pragma unroll
        for (int w = 0; w < kArWarps; ++w) {
          const float f = ex2_approx(wm[w][row] - M);
          const float2 v = *reinterpret_cast<const float2*>(merge + (w * kArMergeRows + sub) * 128 + d);
          L += wl[w][row] * f;
          ax += v.x * f;
          ay += v.y * f;
        }
        if (cr.whole) {
          const float inv = inverse_of(L);
          const size_t orow = out_row(p, b, g, r);
          *reinterpret_cast<uint32_t*>(p.out + orow * 128 + d) = pack_bf16x2(ax * inv, ay * inv);
          if (d == 0) {
            if (p.lse) p.lse[orow] = lse_of(M, L);
            if (p.z) p.row_ml[((size_t)b * p.Hkv + g) * p.G + r] = make_float2(M, L);
          }
        } else {
          *reinterpret_cast<float2*>(p.part_o + (slot * kArRows + row) * 128 + d) = make_float2(ax, ay);
          if (d == 0) p.part_ml[slot * kArRows + row] = make_float2(M, L);
        }
      }
      __syncthreads();  // the merge buffer (and, after the last rows, wm and wl) are free
    }
  }
  // after a timeout: wait (bounded) for what this warp still has in flight
  if (dead)
    for (int i = used; i < fetched; ++i) mbar_wait(&full_b[warp][i % kArStages], (uint32_t)((i / kArStages) & 1));
}

// ---------------------------------------------------------------------------
// attend_units: the same tile for small caches, where launches and latencies count: one
// cluster of C CTAs per (sequence, KV head, row tile), each with an equal part of the
// unit's chunks, two stages a warp.  The parts meet through distributed shared memory, so
// there is one launch and no workspace; with weights, the logits stay in shared memory
// until the log-sum-exps are known.  kWarps 8 for clusters of four and eight, 4 (three CTAs
// an SM) for smaller ones.
constexpr int kAuStages = 2;
constexpr int kMaxUnitTokens = 1536 + kArKeys;  // tokens of a CTA whose logits it keeps
template <int kWarps>
struct UnitsShape {
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRing = kWarps * kAuStages * kArStageBytes;  // then the warps' outputs
  static constexpr int kPart = kArRows * 128 * 4;                   // the CTA's output
  static_assert(kWarps * kArRows * 128 * 4 <= kRing, "the warps' outputs take the ring's place");
  static constexpr int smem(int z_tokens, int G) { return 1024 + kRing + kPart + z_tokens * G * 4; }
};

template <int kWarps>
__global__ void __launch_bounds__(UnitsShape<kWarps>::kThreads) attend_units_kernel(const __grid_constant__ AttendParams p) {
  using Sh = UnitsShape<kWarps>;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full_b[kWarps][kAuStages];
  __shared__ float wm[kWarps][kArRows], wl[kWarps][kArRows];
  __shared__ float2 part_ml[kArRows];  // this CTA's (m, l), read by the cluster
  __shared__ float2 norm[8];  // a head's maximum and 1 / sum
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  uint8_t* base = align1024(smem);
  uint8_t* ring = base + warp * kAuStages * kArStageBytes;
  float* merge = reinterpret_cast<float*>(base);
  float* part_o = reinterpret_cast<float*>(base + Sh::kRing);
  float* zs = part_o + kArRows * 128;  // [G][tokens of this CTA]
  const int units = p.Hkv * p.row_tiles, b = blockIdx.y / units, unit = blockIdx.y % units;
  const int g = unit % p.Hkv, rt = unit / p.Hkv;
  if (lane == 0) {
    for (int s = 0; s < kAuStages; ++s) mbar_init(&full_b[warp][s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int n = checked_len(p, b), nodes = checked_nodes(p, b);
  const int live = min(kArRows, nodes * p.G - rt * kArRows);
  if (live <= 0) return;  // the same in every CTA of the cluster
  const int nc = (n + kArKeys - 1) / kArKeys, chunks = nc + (p.mask ? (nodes + kArKeys - 1) / kArKeys : 0);
  const int lo = (int)((long long)chunks * rank / C), hi = (int)((long long)chunks * (rank + 1) / C);
  int ids = -1, ids_at = lo + warp;
  auto load_ids = [&](int c) {
    ids_at = c;
    const int mine = c + lane * kWarps;
    ids = mine < min(hi, nc) ? p.page_table[(size_t)b * p.max_pages + ((mine * kArKeys) >> p.pshift)] : -1;
  };
  load_ids(lo + warp);
  int fetched = 0, used = 0;
  bool dead = false;
  uint32_t skipped = 0;
  auto fetch = [&](int c) {
    const int s = fetched % kAuStages;
    bool ok = true;
    int row;
    if (c < nc) {
      if (c >= ids_at + 32 * kWarps) load_ids(c);
      const int phys = __shfl_sync(0xffffffffu, ids, (c - ids_at) / kWarps);
      ok = phys >= 0 && phys < p.num_phys;
      row = (phys * p.Hkv + g) * p.P + ((c * kArKeys) & (p.P - 1));
    } else {
      row = (b * p.Hkv + g) * p.T + (c - nc) * kArKeys;
    }
    if (ok) {
      skipped &= ~(1u << s);
      if (lane == 0) {
        const CUtensorMap* mk = c < nc ? &p.tmk : &p.tmkt;
        const CUtensorMap* mv = c < nc ? &p.tmv : &p.tmvt;
        uint8_t* st = ring + s * kArStageBytes;
        uint64_t* bar = &full_b[warp][s];
        mbar_arrive_expect_tx(bar, kArStageBytes);
        tma_load_2d(st, mk, 0, row, bar);
        tma_load_2d(st + 2048, mk, 64, row, bar);
        tma_load_2d(st + 4096, mv, 0, row, bar);
        tma_load_2d(st + 6144, mv, 64, row, bar);
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
  int fc = lo + warp;
  for (int s = 0; s < kAuStages && fc < hi; ++s, fc += kWarps) fetch(fc);
  RowTile tile;
  tile.start(p, b, g, rt, n, nodes);
  const int tokens = (hi - lo) * kArKeys;
  for (int c = lo + warp; c < hi; c += kWarps) {
    const int s = used % kAuStages;
    const bool late = !dead && !mbar_wait(&full_b[warp][s], (uint32_t)((used / kAuStages) & 1));
    if (__any_sync(0xffffffffu, late)) {
      if (lane == 0) flag_error(p.err, RKV_DEVERR_TIMEOUT);
      dead = true;
    }
    if (!dead && !((skipped >> s) & 1u)) {
      tile.step(p, ring + s * kArStageBytes, c, [&](float2 z, int col) {
        if (p.acc && tile.r0 < p.G) *reinterpret_cast<float2*>(zs + tile.r0 * tokens + (c - lo) * kArKeys + col) = z;
      });
    } else if (p.acc) {
      for (int i = lane; i < p.G * kArKeys; i += 32)
        zs[(i / kArKeys) * tokens + (c - lo) * kArKeys + i % kArKeys] = -INFINITY;
    }
    ++used;
    __syncwarp();
    if (fc < hi && !dead) {
      fetch(fc);
      fc += kWarps;
    }
  }
  if (dead)
    for (int i = used; i < fetched; ++i) mbar_wait(&full_b[warp][i % kAuStages], (uint32_t)((i / kAuStages) & 1));
  tile.finish();
  const int qr = lane >> 2, qc = (lane & 3) * 2;
  if ((lane & 3) == 0) {
    wm[warp][qr] = tile.m0;
    wl[warp][qr] = tile.l0;
    wm[warp][qr + 8] = tile.m1;
    wl[warp][qr + 8] = tile.l1;
  }
  __syncthreads();  // every warp is done with its ring: the outputs take its place
#pragma unroll
  for (int half = 0; half < 2; ++half)
    if (half * 8 < live) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        *reinterpret_cast<float2*>(merge + (warp * kArRows + half * 8 + qr) * 128 + j * 8 + qc) =
            make_float2(tile.o[j][half * 2], tile.o[j][half * 2 + 1]);
    }
  __syncthreads();
  for (int i = tid; i < live * 64; i += Sh::kThreads) {
    const int row = i >> 6, d = (i & 63) * 2;
    float M = kNoMax, L = 0.f, ax = 0.f, ay = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w][row]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2_approx(wm[w][row] - M);
      const float2 v = *reinterpret_cast<const float2*>(merge + (w * kArRows + row) * 128 + d);
      L += wl[w][row] * f;
      ax += v.x * f;
      ay += v.y * f;
    }
    *reinterpret_cast<float2*>(part_o + row * 128 + d) = make_float2(ax, ay);
    if (d == 0) part_ml[row] = make_float2(M, L);
  }
  cluster.sync();  // every CTA's part is in place
  // rows of the output in turn over the cluster: thread = (row, two channels), eight parts'
  // reads in flight
  for (int i = tid; i < live * 64; i += Sh::kThreads) {
    const int row = i >> 6, d = (i & 63) * 2;
    if (row % C != rank) continue;
    float2 ml[8], v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < C) {
        ml[c] = *cluster.map_shared_rank(&part_ml[row], c);
        v[c] = *cluster.map_shared_rank(reinterpret_cast<float2*>(part_o + row * 128 + d), c);
      }
    float M = kNoMax, L = 0.f, ax = 0.f, ay = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < C) M = fmaxf(M, ml[c].x);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < C) {
        const float f = ex2_approx(ml[c].x - M);
        L += ml[c].y * f;
        ax += v[c].x * f;
        ay += v[c].y * f;
      }
    const float inv = inverse_of(L);
    const size_t orow = out_row(p, b, g, rt * kArRows + row);
    *reinterpret_cast<uint32_t*>(p.out + orow * 128 + d) = pack_bf16x2(ax * inv, ay * inv);
    if (d == 0 && p.lse) p.lse[orow] = lse_of(M, L);
  }
  if (p.acc) {  // one token: its rows are the group's heads
    {
      for (int h = warp; h < p.G; h += kWarps) {
        float2 ml = lane < C ? *cluster.map_shared_rank(&part_ml[h], lane) : make_float2(kNoMax, 0.f);
        float M = ml.x;
#pragma unroll
        for (int o = 4; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = ml.y * ex2_approx(ml.x - M);
#pragma unroll
        for (int o = 4; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0) norm[h] = norm_of(M, L);
      }
    }
    __syncthreads();
    float* a = p.acc + ((size_t)b * p.Hkv + g) * p.acc_stride + (size_t)lo * kArKeys;
    for (int t = tid; t < tokens; t += Sh::kThreads) {
      if (lo * kArKeys + t >= n) break;
      float w = 0.f;
      for (int h = 0; h < p.G; ++h) w += ex2_approx(zs[h * tokens + t] - norm[h].x) * norm[h].y;
      a[t] += w;
    }
  }
  cluster.sync();  // no CTA leaves while another still reads its shared memory
}

// Where the parts of a split unit lie: CTA c's at slot 2 c, but the first CTA's at 2 c + 1
// when its share began before the unit.
struct PartSlots {
  int c0, c1, late;
  __device__ __forceinline__ PartSlots(long long ux, int per, int pad, long long total, int N)
      : c0(flat_cta(ux + pad, total, N)), c1(flat_cta(ux + per - 1, total, N)), late(flat_first(total, c0, N) < ux) {}
  __device__ __forceinline__ size_t operator[](int c) const { return 2 * (size_t)c + (c == c0 ? late : 0); }
};

// Final (m, l) of one row of a split unit: the lanes of a warp take its parts.
template <int kRows>
__device__ __forceinline__ float2 join_ml(const AttendParams& p, const PartSlots& ps, int row, int lane) {
  float M = kNoMax, L = 0.f;
  for (int c = ps.c0 + lane; c <= ps.c1; c += 32) {
    const float2 ml = p.part_ml[ps[c] * kRows + row];
    const float to = fmaxf(M, ml.x);
    L = L * ex2_approx(M - to) + ml.y * ex2_approx(ml.x - to);
    M = to;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m = __shfl_xor_sync(0xffffffffu, M, o), l = __shfl_xor_sync(0xffffffffu, L, o), to = fmaxf(M, m);
    L = L * ex2_approx(M - to) + l * ex2_approx(m - to);
    M = to;
  }
  return make_float2(M, L);
}

// Joins the parts of the split units: one warp a row, four channels a lane, four parts'
// loads in flight.  256 threads, eight rows of the line of all rows at a time.
template <int kRows, int kKeys>
__device__ __forceinline__ void combine_row(const AttendParams& p, const FlatTable& ft, int b, int idx, int lane) {
  const long long total = ft.base[p.B];
  const int N = flat_ctas(total, p.N);
  const int t = ft.t[b], per = ft.per[b];
  const int rows = t * p.G;  // query rows of a unit's KV head
  if (idx >= rows * p.Hkv) return;
  const int g = idx / rows, r = idx - g * rows, rt = r / kRows, row = r % kRows;
  const size_t orow = out_row(p, b, g, r);
  uint2* out = reinterpret_cast<uint2*>(p.out + orow * 128) + lane;
  if (per == 0) {  // nothing to see: no token cached and no tree
    *out = make_uint2(0u, 0u);
    if (lane == 0 && p.lse) p.lse[orow] = -INFINITY;
    return;
  }
  const PartSlots ps(ft.base[b] + (long long)(rt * p.Hkv + g) * per, per, ft.pad, total, N);
  if (ps.c0 == ps.c1) return;  // final already
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = kNoMax, L = 0.f;
  for (int c = ps.c0; c <= ps.c1; c += 4) {
    float4 v[4];
    float2 ml[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = c + j <= ps.c1;
      const size_t at = ps[in ? c + j : c] * kRows + row;  // behind the last part: the first again, unweighted
      ml[j] = p.part_ml[at];
      v[j] = reinterpret_cast<const float4*>(p.part_o + at * 128)[lane];
      if (!in) ml[j] = make_float2(kNoMax, 0.f);
    }
    const float to = fmaxf(M, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
    const float f = ex2_approx(M - to);
    M = to;
    L *= f;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float w = c + j <= ps.c1 ? ex2_approx(ml[j].x - M) : 0.f;
      L += ml[j].y * w;
      o.x += v[j].x * w;
      o.y += v[j].y * w;
      o.z += v[j].z * w;
      o.w += v[j].w * w;
    }
  }
  const float inv = inverse_of(L);
  *out = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (lane == 0 && p.lse) p.lse[orow] = lse_of(M, L);
}

template <int kRows, int kKeys>
__global__ void __launch_bounds__(256, 4) attend_combine_kernel(const __grid_constant__ AttendParams p) {
  __shared__ FlatTable ft;
  build_table<kRows, kKeys>(p, ft);  // lengths only: they were final before the parts' kernel began
  grid_dependency_wait();
  const long long each = (long long)p.Hq * p.T, rows = each * p.B;
  for (long long x = blockIdx.x * 8 + (threadIdx.x >> 5); x < rows; x += gridDim.x * 8)
    combine_row<kRows, kKeys>(p, ft, (int)(x / each), (int)(x % each), threadIdx.x & 31);
}

// The end of a one-token step (19 us for the ragged batch, of which the join of a tree's
// rows alone takes 8): the first CTAs join the rows as attend_combine does, the
// others add the weights, acc_j += sum_h 2^(z_hj - m_h) / l_h, over blocks of
// kWeighTokens tokens of a (sequence, KV head), eight tokens a thread; each block joins its
// heads' (m, l) for itself.  The logits were written a moment ago and mostly lie in L2.
__global__ void __launch_bounds__(256, 4) attend_weigh_kernel(const __grid_constant__ AttendParams p) {
  __shared__ FlatTable ft;
  __shared__ float2 norm[8];  // a head's maximum and 1 / sum
  __shared__ long long wbase[RKV_MAX_BATCH + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  build_table<kArRows, kArKeys>(p, ft);
  flat_scan(wbase, p.B, [&](int b) { return (long long)p.Hkv * ((ft.n[b] + kWeighTokens - 1) / kWeighTokens); });
  grid_dependency_wait();
  const int joins = p.B * ((p.Hq + 7) / 8);
  if ((int)blockIdx.x < joins) {
    const int per_b = (p.Hq + 7) / 8;
    combine_row<kArRows, kArKeys>(p, ft, blockIdx.x / per_b, (blockIdx.x % per_b) * 8 + warp, lane);
    return;
  }
  const long long total = ft.base[p.B];
  const int N = flat_ctas(total, p.N);
  for (long long x = blockIdx.x - joins; x < wbase[p.B]; x += gridDim.x - joins) {
    int b = 0, hi = p.B - 1;
    while (b < hi) {
      const int mid = (b + hi + 1) >> 1;
      if (wbase[mid] <= x) b = mid; else hi = mid - 1;
    }
    const int n = ft.n[b], blocks = (n + kWeighTokens - 1) / kWeighTokens;
    const int g = (int)((x - wbase[b]) / blocks), blk = (int)((x - wbase[b]) % blocks);
    const size_t unit = (size_t)b * p.Hkv + g;
    if (warp < p.G) {
      const PartSlots ps(ft.base[b] + (long long)g * ft.per[b], ft.per[b], ft.pad, total, N);
      const float2 ml = ps.c0 == ps.c1 ? p.row_ml[unit * p.G + warp] : join_ml<kArRows>(p, ps, warp, lane);
      if (lane == 0) norm[warp] = norm_of(ml.x, ml.y);
    }
    __syncthreads();
    // two quads of tokens a thread; positions behind n hold -inf up to the chunk's end and
    // are not read beyond it
    const int t[2] = {blk * kWeighTokens + tid * 4, blk * kWeighTokens + kWeighTokens / 2 + tid * 4};
    float4 w[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    const float* zu = p.z + unit * p.G * p.zstride;
#pragma unroll 4
    for (int h = 0; h < p.G; ++h) {
      const float base = norm[h].x, inv = norm[h].y;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (t[q] < n) {
          const float4 z = *reinterpret_cast<const float4*>(zu + (size_t)h * p.zstride + t[q]);
          w[q].x += ex2_approx(z.x - base) * inv;
          w[q].y += ex2_approx(z.y - base) * inv;
          w[q].z += ex2_approx(z.z - base) * inv;
          w[q].w += ex2_approx(z.w - base) * inv;
        }
    }
    float* a = p.acc + unit * p.acc_stride;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float e[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t[q] + i < n) a[t[q] + i] += e[i];
    }
    __syncthreads();  // norm is free
  }
}

// ---------------------------------------------------------------------------
// attend_tiles: 17 query rows and more, on the fifth-generation tensor cores.
//
// Two row slots of 128 rows work in turn on 128-key tiles: while a slot's four warps turn
// its logits into weights, the tensor cores run the other slot's products.
//   S = Q K^T   128 x 128 x 128, both operands in shared memory, S in TMEM;
//   P           bf16, written back over S's columns (thread = row = TMEM lane);
//   O += P V    128 x 128 x 128, P from TMEM, V from shared memory, O in TMEM.
// kWide: a unit's tile is 256 rows, the slots hold different rows and both use every key
// tile, so the cache is read once for 256 rows.  Otherwise the tile is 128 rows and the
// slots take alternate key tiles of the same rows, each with its own maximum, sum and O,
// and join them at the end of a run.  K and V of a key tile are 64 KB, 128 keys x 128
// channels x 256 rows x 4 = 16.8 MFLOP: at the card's rates the bytes take 1.4 us of an
// SM's share and the products 1.1 us, so the wide form sits near both roofs and the narrow
// one on the bytes alone.  Measured, 8 x 64K tokens, 8 KV heads (2.15 GB): 32 rows 314 us,
// 6.8 TB/s, a plain copy's rate; 256 rows 406 us, 5.3 TB/s and 1.36 PFLOP/s, with the card
// at its power limit and the SM clock down to 1.55 .. 1.75 GHz.  (Taking out the exponentials
// or most of the second product changed that by under 7 %.)
//   warps 0-3, 4-7: softmax of slot 0, 1;  warps 8, 10: TMA of K, V;  warp 9: MMA issue;  11: idle.
// The running maximum that the weights refer to moves only when a row's new maximum is
// above it by more than 8 (base 2): weights then stay below 2^8 and O is rescaled, a TMEM
// round trip of 64 KB, a few times a run instead of every tile.
// Ring entries are 32 KB, a tile's K or V; order and phases are the same formula on the TMA
// and the MMA side.  Every wait is bounded; one that runs out flags RKV_DEVERR_TIMEOUT and
// stops every role.
constexpr int kAtKeys = 128;
constexpr int kAtThreads = 384;
// Registers: 384 threads start with 168 each; the softmax warps take 208 and the third
// warpgroup (TMA, MMA, an idle warp) keeps 88: 256 x 208 + 128 x 88 = 384 x 168.
constexpr int kAtSoftRegs = 208, kAtIssueRegs = 88;
static_assert(256 * kAtSoftRegs + 128 * kAtIssueRegs == 384 * 168, "the split must be what the block was launched with");
constexpr int kAtEntry = 128 * 256;
constexpr float kAtSlack = 8.f;
// A weight's exponent is z sl - m as one fused multiply-add, in which m is rounded and z sl is
// not.  The difference, at most 2^-24 of m, is the same for the whole row and cancels, while
// it is no more than 64.  A row whose maximum lies beyond this has distinct logits at least
// 64 apart, so that only ties with the maximum count: it takes the power of two below sl,
// whose product with the maximum is exact.  The choice is made where the maximum moves: 266 us
// for the ragged batch of 63 nodes against 264 without it, 280 with a test in every tile.
constexpr float kAtFar = 1073741824.f;
// The tiled kernel's table: only the line's offsets; a run's lengths are read again.
struct SlimRun : FlatRun {
  int n, t;
};
template <bool kWide>
struct TileShape {
  static constexpr int kRows = kWide ? 256 : 128;
  static constexpr int kQBytes = kRows * 256;
  static constexpr int kEntries = 5;
  // Everything lies in dynamic shared memory, declared with the swizzle atom's 1024-byte
  // alignment: queries and ring fill 224 of the 227 KB in the wide form, with no room to
  // round an address up.
  struct Shared {
    uint8_t q[kQBytes];
    uint8_t ring[kEntries * kAtEntry];
    long long base[RKV_MAX_BATCH + 1];
    uint64_t full[kEntries], empty[kEntries], s[2], p[2], o[2], qf[2], out[2], ml, drained;
    uint32_t groups[kEntries];  // a K entry's 16-key groups that were loaded (page ids in range)
    uint32_t sgroups[2];        // the same for the tile whose logits a slot holds
    uint32_t tmem_base;
    int abort_flag;
    SlimRun first;  // the share's first run, worked out once
    bool any;       // there is one
    long long x0, x1;
    float2 ml_s[kWide ? 1 : 2][kWide ? 1 : 128];
  };
  static constexpr int kSmem = sizeof(Shared);
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

// Pieces of a unit, the empty ones included.
template <int kRows, int kKeys>
__device__ __forceinline__ int pieces_of(const AttendParams& p, int n, int t) {
  const int real = (n + kKeys - 1) / kKeys + (p.mask ? (t + kKeys - 1) / kKeys : 0);
  return real > 0 ? real + pad_of<kKeys>() : 0;
}
template <int kRows, int kKeys>
__device__ __forceinline__ bool slim_run(const AttendParams& p, const long long* base, long long x, long long x0,
                                         long long x1, SlimRun& r) {
  for (; x < x1; x = r.next) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (base[mid] <= x) lo = mid; else hi = mid - 1;
    }
    r.b = lo;
    r.n = checked_len(p, lo);
    r.t = checked_nodes(p, lo);
    const int per = pieces_of<kRows, kKeys>(p, r.n, r.t);
    const long long off = x - base[lo];
    r.unit = off < (1LL << 31) ? (int)((uint32_t)off / (uint32_t)per) : (int)(off / per);
    r.first = x == x0;
    r.x = x;
    if (flat_part(r, (int)(off - (long long)r.unit * per), x1 - x, per, pad_of<kKeys>())) return true;
  }
  return false;
}

template <bool kWide>
__global__ void __launch_bounds__(kAtThreads, 1) attend_tiles_kernel(const __grid_constant__ AttendParams p) {
  using Sh = TileShape<kWide>;
  constexpr int E = Sh::kEntries, R = Sh::kRows;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  typename Sh::Shared& sh = *reinterpret_cast<typename Sh::Shared*>(dyn_smem);
  uint64_t *const full_b = sh.full, *const empty_b = sh.empty, *const s_b = sh.s, *const p_b = sh.p, *const o_b = sh.o,
                  *const q_b = sh.qf;
  uint64_t* const ml_b = &sh.ml;
  uint32_t *const groups = sh.groups, *const sgroups = sh.sgroups;
  volatile int& abort_flag = *const_cast<volatile int*>(&sh.abort_flag);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* const qs = sh.q;
  uint8_t* const ring = sh.ring;
  if (tid == 0) {
    for (int e = 0; e < E; ++e) {
      mbar_init(&full_b[e], 1);
      mbar_init(&empty_b[e], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_b[s], 2);    // the issuing thread and its commit
      mbar_init(&p_b[s], 128);
      mbar_init(&o_b[s], 1);
      mbar_init(&q_b[s], kWide ? 128 : 256);
      mbar_init(&sh.out[s], kWide ? 128 : 256);
    }
    mbar_init(ml_b, 256);
    mbar_init(&sh.drained, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (tid == 32) {
    prefetch_map(&p.tmk);
    prefetch_map(&p.tmv);
  }
  if (warp == 9) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  flat_scan(sh.base, p.B, [&](int b) {  // ends with a block barrier
    const int t = checked_nodes(p, b);
    return (long long)pieces_of<R, kAtKeys>(p, checked_len(p, b), t) * p.Hkv * ((t * p.G + R - 1) / R);
  });
  tc_fence_after();
  grid_launch_dependents();
  const uint32_t tmem = sh.tmem_base;
  if (tid == 0) {  // one thread: twelve warps dividing at once took twice as long
    const long long total = sh.base[p.B];
    const int N = flat_ctas(total, p.N);
    const bool works = (int)blockIdx.x < N;
    sh.x0 = works ? flat_first(total, blockIdx.x, N) : 0;
    sh.x1 = works ? flat_first(total, blockIdx.x + 1, N) : 0;
    sh.any = slim_run<R, kAtKeys>(p, sh.base, sh.x0, sh.x0, sh.x1, sh.first);
  }
  __syncthreads();
  const long long x0 = sh.x0, x1 = sh.x1;
  auto next_run = [&](long long x, SlimRun& r) {
    if (x != x0) return slim_run<R, kAtKeys>(p, sh.base, x, x0, x1, r);
    r = sh.first;
    return sh.any;
  };
  auto give_up = [&]() {
    flag_error(p.err, RKV_DEVERR_TIMEOUT);
    abort_flag = 1;
  };
  int loaded = 0;  // one past the last ring entry filled (warps 8, 10) or used (warp 9)
  SlimRun r;

  if (warp < 8) {
    setmaxnreg_inc<kAtSoftRegs>();
    const int slot = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), mine = lanes + slot * 256;
    const float sl = p.scale_log2;
    int seen_s = 0, run = 0, done[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {
      const bool late = !mbar_wait_role(bar, (uint32_t)(phase & 1), &abort_flag);
      if (__any_sync(0xffffffffu, late)) {  // warp-uniform: the TMEM accesses are .aligned
        give_up();
        return false;
      }
      return true;
    };
    for (long long x = x0; ok && next_run(x, r); x = r.next) {
      const int b = r.b, g = r.unit % p.Hkv, rt = r.unit / p.Hkv;
      const int n = r.n, nodes = r.t, rows = nodes * p.G, nc = (n + kAtKeys - 1) / kAtKeys, nt = r.hi - r.lo;
      const bool idle = kWide && slot == 1 && rows - rt * R <= 128;
      // the query rows, swizzled as TMA would store them, over the last run's staged outputs
      if (run > 0 && !(ok = wait(&sh.out[kWide ? slot : 0], run - 1))) break;
      {
        constexpr int kPer = kWide ? 128 : 64;  // rows this slot's warps load
        const int q0 = kWide ? 0 : slot * 64;
        uint8_t* dst = qs + (kWide ? slot * (128 * 256) : 0);
        const int piece = row & 15;
        uint4 v[kPer / 8];  // all loads in flight together
#pragma unroll
        for (int j = 0; j < kPer / 8; ++j) {
          const int rr = rt * R + (kWide ? slot * 128 : 0) + q0 + (row >> 4) + j * 8;
          v[j] = make_uint4(0, 0, 0, 0);
          if (rr < rows) v[j] = reinterpret_cast<const uint4*>(p.q + out_row(p, b, g, rr) * 128)[piece];
        }
#pragma unroll
        for (int j = 0; j < kPer / 8; ++j) {
          const int i = q0 + (row >> 4) + j * 8;
          *reinterpret_cast<uint4*>(dst + (piece >> 3) * (128 * 128) + i * 128 + (((piece & 7) ^ (i & 7)) << 4)) = v[j];
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_b[kWide ? slot : 0]);
      }
      const int my = rt * R + (kWide ? slot * 128 : 0) + row;  // this thread's query row
      float m = kNoMax, l = 0.f;
      float ref = m, ref_sl = sl;  // what the weights' exponents are taken with: z ref_sl - ref
      auto set_ref = [&](float raw) {
        const bool far = fabsf(m) > kAtFar && m != kNoMax;
        ref_sl = far ? __uint_as_float(__float_as_uint(sl) & 0x7f800000u) : sl;
        ref = far ? raw * ref_sl : m;
      };
      if (!idle) {
        for (int i = kWide ? 0 : slot; i < nt; i += kWide ? 1 : 2) {
          if (!(ok = wait(&s_b[slot], seen_s++))) break;
          tc_fence_after();
          const int tile = r.lo + i;
          const uint32_t gr = sgroups[slot];
          const int left = tile < nc ? n - tile * kAtKeys : nodes - (tile - nc) * kAtKeys;
          const bool all = tile < nc && left >= kAtKeys && gr == 0xffu;
          uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
          if (!all) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int k = left - w * 32;
              see[w] = k >= 32 ? ~0u : (k <= 0 ? 0u : (1u << k) - 1u);
              if (!((gr >> (2 * w)) & 1u)) see[w] &= 0xffff0000u;
              if (!((gr >> (2 * w + 1)) & 1u)) see[w] &= 0x0000ffffu;
            }
            if (tile >= nc) {
              const int w0 = (tile - nc) * 4;
              const uint32_t* mk = p.mask + ((size_t)b * p.T + (my < rows ? my >> p.gshift : 0)) * p.words + w0;
#pragma unroll
              for (int w = 0; w < 4; ++w) see[w] &= w0 + w < p.words ? mk[w] : 0u;
            }
          }
          uint32_t v[4][32];
          float mx = -INFINITY, mx1 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) tc_ld32(mine + c * 32, v[c]);
          tc_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tc_ld_done(v[c]);
            if (!all) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((see[c] >> j) & 1u)) v[c][j] = 0xff800000u;  // -inf
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              mx = max3(mx, __uint_as_float(v[c][j]), __uint_as_float(v[c][j + 1]));
              mx1 = max3(mx1, __uint_as_float(v[c][j + 2]), __uint_as_float(v[c][j + 3]));
            }
          }
          const float raw = fmaxf(mx, mx1);
          mx = raw * sl;  // sl > 0
          const bool first = i < (kWide ? 1 : 2);
          if (first) {
            m = fmaxf(kNoMax, mx);
            set_ref(raw);
          } else if (__any_sync(0xffffffffu, mx > m + kAtSlack)) {
            // this slot's earlier products are complete: its logits were issued after them
            const float to = fmaxf(m, mx), f = ex2_approx(m - to);
            if (mx > m) {
              m = to;
              set_ref(raw);
            }
            l *= f;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tc_ld32_wait(mine + 128 + c * 32, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tc_st32_wait(mine + 128 + c * 32, o);
            }
          }
          float s0 = 0.f, s1 = 0.f, u0 = 0.f, u1 = 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int cc = c * 2 + (j >> 4), jj = (j & 15) * 2;
              const float ax = ex2_approx(fmaf(__uint_as_float(v[cc][jj]), ref_sl, -ref));
              const float ay = ex2_approx(fmaf(__uint_as_float(v[cc][jj + 1]), ref_sl, -ref));
              (j & 1 ? u0 : s0) += ax;
              (j & 1 ? u1 : s1) += ay;
              // bf16 weights (off by at most 2^-8 of each, as V is); their sum stays unrounded
              pk[j] = pack_bf16x2(ax, ay);
            }
            tc_st32(mine + c * 32, pk);
          }
          tc_st_wait();
          l += (s0 + s1) + (u0 + u1);
          tc_fence_before();
          mbar_arrive(&p_b[slot]);
        }
      }
      if (!ok) break;
      // the run's end: out = O / l (whole unit) or the part (m, l, O)
      const bool has[2] = {true, kWide ? true : nt > 1};
      float f0 = 1.f, f1 = 0.f;
      if (kWide) {
        if (!(ok = wait(&o_b[slot], done[slot]++))) break;
      } else {
        sh.ml_s[slot][row] = make_float2(m, l);
        mbar_arrive(ml_b);
        if (!(ok = wait(ml_b, run))) break;
        if (!(ok = wait(&o_b[0], done[0]++))) break;
        if (has[1] && !(ok = wait(&o_b[1], done[1]++))) break;
        const float2 a = sh.ml_s[0][row], c = has[1] ? sh.ml_s[1][row] : make_float2(kNoMax, 0.f);
        m = fmaxf(a.x, c.x);
        f0 = ex2_approx(a.x - m);
        f1 = ex2_approx(c.x - m);
        l = a.y * f0 + c.y * f1;
      }
      ++run;
      tc_fence_after();
      if (!idle) {
        const bool live = my < rows;
        const float inv = r.whole ? inverse_of(l) : 1.f;
        const size_t orow = live ? out_row(p, b, g, my) : 0;
        const size_t prow = (2 * (size_t)blockIdx.x + (r.first ? 0 : 1)) * R + (kWide ? slot * 128 : 0) + row;
        // kWide: all 128 channels of this slot's row; else 64 channels of both slots' O.  32
        // channels of the warp's 32 rows at a time go through the query tile's memory (its
        // products are done), so that the stores are whole 128-byte (bf16: 64-byte) pieces
        // of rows and not 16 bytes of 32 rows each.
        constexpr int kChunks = kWide ? 4 : 2;
        uint8_t* const stage = qs + slot * (kWide ? 32768 : 16384) + (warp & 3) * 4096;
        const int row0 = rt * R + (kWide ? slot * 128 : 0) + (warp & 3) * 32;  // the warp's first query row
        const size_t prow0 = prow - lane;
#pragma unroll 1
        for (int cc = 0; cc < kChunks; ++cc) {
          const int c = kWide ? cc : slot * 2 + cc;
          uint32_t o[32];
          tc_ld32_wait(kWide ? mine + 128 + c * 32 : lanes + 128 + c * 32, o);
          if (!kWide) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f0);
            if (has[1]) {
              uint32_t o1[32];
              tc_ld32_wait(lanes + 256 + 128 + c * 32, o1);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                o[j] = __float_as_uint(fmaf(__uint_as_float(o1[j]), f1, __uint_as_float(o[j])));
            }
          }
          __syncwarp();  // the staged piece before this one is read
          if (r.whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(o[j * 8 + 2 * e]) * inv, __uint_as_float(o[j * 8 + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = k * 8 + (lane >> 2), j = lane & 3;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + i * 64 + ((j ^ ((i >> 1) & 3)) << 4));
              if (row0 + i < rows)
                reinterpret_cast<uint4*>(p.out + out_row(p, b, g, row0 + i) * 128 + c * 32)[j] = v;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                  make_uint4(o[j * 4], o[j * 4 + 1], o[j * 4 + 2], o[j * 4 + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int i = k * 4 + (lane >> 3), j = lane & 7;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + i * 128 + ((j ^ (i & 7)) << 4));
              if (row0 + i < rows) reinterpret_cast<uint4*>(p.part_o + (prow0 + i) * 128 + c * 32)[j] = v;
            }
          }
        }
        if (live && (kWide || slot == 0)) {
          if (!r.whole) p.part_ml[prow] = make_float2(m, l);
          else if (p.lse) p.lse[orow] = lse_of(m, l);
        }
        tc_fence_before();  // O is read before the next run's queries let its products start
      }
      mbar_arrive(&sh.out[kWide ? slot : 0]);  // this thread has read what it staged
    }
  } else {
    setmaxnreg_dec<kAtIssueRegs>();
    if (warp == 8 || warp == 10) {
      // warp 8 fetches K, warp 10 V; entry of K_i / V_i among a run's 2 nt entries:
      // wide K_i 2 i, V_i 2 i + 1; narrow K_0, then K_(i+1) and V_i for every i
      const bool v = warp == 10;
      const CUtensorMap* map = v ? &p.tmv : &p.tmk;
      const CUtensorMap* tmap = v ? &p.tmvt : &p.tmkt;
      const bool lead = elect_lane();
      const int pages = kAtKeys >> p.pshift, box = p.P * 128;  // pages of a tile, bytes of a box
      // one row tile: nobody reads the cache again (the wide form measured 267 us with this
      // and 255 without, 63 nodes over the ragged batch; the narrow one 33 against 37)
      const uint64_t policy = l2_policy(!kWide && p.T * p.G <= R);
      int before = 0;                                          // entries of the runs before
      bool ok = true;
      for (long long x = x0; ok && next_run(x, r); x = r.next) {
        const int b = r.b, g = r.unit % p.Hkv, n = r.n, nc = (n + kAtKeys - 1) / kAtKeys, nt = r.hi - r.lo;
        // lane j: page id of the tile's page j, -1: none; loaded a tile ahead and judged only
        // when it is used, so that the load's latency stays off the ring
        auto page_of = [&](int tile) {
          const int pg = tile * pages + lane;
          return tile < nc && lane < pages && pg * p.P < n ? p.page_table[(size_t)b * p.max_pages + pg] : -1;
        };
        int next = page_of(r.lo);
        for (int i = 0; i < nt; ++i) {
          const int tile = r.lo + i;
          int phys = next;
          next = i + 1 < nt ? page_of(tile + 1) : -1;
          const int at = before + (kWide ? 2 * i + v : (v ? (i + 1 < nt ? 2 * i + 2 : 2 * nt - 1) : (i > 0 ? 2 * i - 1 : 0)));
          const int e = at % E;
          const bool late = at >= E && !mbar_wait_role(&empty_b[e], (uint32_t)((at / E - 1) & 1), &abort_flag);
          if (__any_sync(0xffffffffu, late)) {
            give_up();
            ok = false;
            break;
          }
          uint8_t* const st = ring + e * kAtEntry;
          const uint32_t st32 = smem_u32(st), bar32 = smem_u32(&full_b[e]);
          if (tile < nc) {
            if (phys < 0 || phys >= p.num_phys) {
              if (lane < pages && (tile * pages + lane) * p.P < n) flag_error(p.err, RKV_DEVERR_PAGE_ID);
              phys = -1;
            }
            const uint32_t have = __ballot_sync(0xffffffffu, phys >= 0);
            if (lead) {
              if (!v) {
                uint32_t gr = 0;  // a page is P / 16 groups
                for (int j = 0; j < pages; ++j)
                  if ((have >> j) & 1u) gr |= ((1u << (p.P >> 4)) - 1u) << (j * (p.P >> 4));
                groups[e] = gr;
              }
              if (have) mbar_arrive_expect_tx(&full_b[e], __popc(have) * 2 * box);
              else mbar_arrive(&full_b[e]);
            }
            __syncwarp();
            int row[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) row[j] = (__shfl_sync(0xffffffffu, phys, j) * p.Hkv + g) * p.P;
            if (kWide) {
              // The wide form is bound by the products and the card's power: boxes issued from
              // converged code, 90 clocks each, measured 406 us against 429 from one lane.
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                tma_load_2d_if(lead && ((have >> j) & 1u), st32 + j * box, map, 0, row[j], bar32);
                tma_load_2d_if(lead && ((have >> j) & 1u), st32 + kAtEntry / 2 + j * box, map, 64, row[j], bar32);
              }
            } else if (lead) {  // the narrow one by the copies: 320 us from one lane against 364 (8 nodes, 8 x 64K)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if ((have >> j) & 1u) {
                  tma_load_2d_hint(st + j * box, map, 0, row[j], &full_b[e], policy);
                  tma_load_2d_hint(st + kAtEntry / 2 + j * box, map, 64, row[j], &full_b[e], policy);
                }
            }
          } else {
            const int row = (b * p.Hkv + g) * p.T + (tile - nc) * kAtKeys;
            if (lead) {
              if (!v) groups[e] = 0xffu;
              mbar_arrive_expect_tx(&full_b[e], kAtEntry);
            }
            __syncwarp();
            if (lead) {
              tma_load_2d(st, tmap, 0, row, &full_b[e]);
              tma_load_2d(st + kAtEntry / 2, tmap, 64, row, &full_b[e]);
            }
          }
          loaded = at + 1;
        }
        before += 2 * nt;
      }
    } else if (warp == 9) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128), idesc_o = idesc_s | kIdescBNMajor;
      const uint32_t q32 = smem_u32(qs), ring32 = smem_u32(ring);
      int seen_p[2] = {0, 0}, runs[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        const bool late = !mbar_wait_role(bar, (uint32_t)(phase & 1), &abort_flag);
        if (__any_sync(0xffffffffu, late)) {
          give_up();
          return false;
        }
        return true;
      };
      const bool lead = elect_lane();
      const uint32_t qlo = sw128_kmajor_lo(q32), klo = sw128_kmajor_lo(ring32), vlo = sw128_nmajor_lo(ring32, kAtEntry / 2);
      // S of `slot` from the K entry e (its copy has landed)
      auto mma_s = [&](int slot, int e, bool release) {
        tc_fence_after();
        if (lead) sgroups[slot] = groups[e];
        const uint32_t d = tmem + slot * 256, qa = qlo + (kWide ? slot * (128 * 256 >> 4) : 0), ka = klo + e * (kAtEntry >> 4);
        tc_mma_ss<false>(lead, d, qa, ka, idesc_s);
#pragma unroll
        for (int k = 1; k < 8; ++k) {
          const uint32_t off = ((k >> 2) * (kAtEntry / 2) + (k & 3) * 32) >> 4;
          tc_mma_ss<true>(lead, d, qa + off, ka + off, idesc_s);
        }
        tc_commit_if(lead && release, &empty_b[e]);
        tc_commit_if(lead, &s_b[slot]);
        if (lead) mbar_arrive(&s_b[slot]);
        __syncwarp();
      };
      // O += P V once the slot's weights are there (handed over in two halves, the issuing
      // warp waited twice and the other slot with it: 480 us against 410 for 64 nodes, 8 x 64K)
      auto mma_o = [&](int slot, int e, bool first, bool last, bool release) {
        if (!(ok = wait(&p_b[slot], seen_p[slot]++))) return;
        tc_fence_after();
        const uint32_t d = tmem + slot * 256 + 128, pa = tmem + slot * 256, va = vlo + e * (kAtEntry >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_ts(lead, d, pa + k * 8, va + (k * 2048 >> 4), idesc_o, (first && k == 0) ? 0u : 1u);
        tc_commit_if(lead && release, &empty_b[e]);
        tc_commit_if(lead && last, &o_b[slot]);
      };
      for (long long x = x0; ok && next_run(x, r); x = r.next) {
        const int n = r.n, nodes = r.t, nc = (n + kAtKeys - 1) / kAtKeys, nt = r.hi - r.lo;
        const bool two = kWide && nodes * p.G - (r.unit / p.Hkv) * R > 128;  // slot 1 has rows
        // keys of a tile that may hold anything (behind the end, on a bad page) have weight 0,
        // and 0 x NaN is not 0: their V rows are cleared first
        auto clean_v = [&](int tile, int e, uint32_t gr) {
          const int left = tile < nc ? n - tile * kAtKeys : nodes - (tile - nc) * kAtKeys;
          if (left >= kAtKeys && gr == 0xffu) return;
          for (int i = lane; i < 128 * 16; i += 32) {
            const int row = i >> 4;
            if (row < left && ((gr >> (row >> 4)) & 1u)) continue;
            *reinterpret_cast<uint4*>(ring + e * kAtEntry + ((i >> 3) & 1) * (kAtEntry / 2) + row * 128 + (i & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        };
        auto take = [&]() {  // the next ring entry, landed
          const int e = loaded % E;
          ok = wait(&full_b[e], loaded / E);
          ++loaded;
          return e;
        };
        ok = wait(&q_b[0], runs[0]++);
        if (kWide && ok) ok = wait(&q_b[1], runs[1]++);
        if (!ok) break;
        if (kWide) {
          int ek = take();
          if (!ok) break;
          uint32_t gr = groups[ek];
          mma_s(0, ek, !two);
          if (two) mma_s(1, ek, true);
          for (int i = 0; i < nt; ++i) {
            const int ev = take();
            if (!ok) break;
            clean_v(r.lo + i, ev, gr);
            const bool last = i + 1 == nt;
            mma_o(0, ev, i == 0, last, !two);
            if (!ok) break;
            if (kWide) tc_commit_if(lead && last && !two, &o_b[1]);  // keeps an idle slot in step
            int en = 0;
            if (!last) {
              en = take();
              if (!ok) break;
              gr = groups[en];
              mma_s(0, en, !two);
            }
            if (two) {
              mma_o(1, ev, i == 0, last, true);
              if (!ok) break;
              if (!last) mma_s(1, en, true);
            }
          }
        } else {
          uint32_t gr[2];
          const int e0 = take();
          if (!ok) break;
          gr[0] = groups[e0];
          mma_s(0, e0, true);
          for (int i = 0; i < nt; ++i) {
            // order of the entries: K_0, then K_(i+1) and V_i for every i
            const int slot = i & 1;
            int en = 0;
            uint32_t gn = 0;
            if (i + 1 < nt) {
              en = take();
              if (!ok) break;
              gn = groups[en];
              if (i == 0) mma_s(1, en, true);
            }
            // tile i + 1's logits go where tile i - 1's weights lay: its product was issued before
            if (i + 1 < nt && i > 0) mma_s(slot ^ 1, en, true);
            const int ev = take();
            if (!ok) break;
            clean_v(r.lo + i, ev, gr[slot]);
            if (i + 1 < nt) gr[slot ^ 1] = gn;
            mma_o(slot, ev, i < 2, i + 2 >= nt, true);
            if (!ok) break;
          }
        }
      }
      // the last entries' releases land before the CTA may exit
      if (ok)
        for (int i = loaded > E ? loaded - E : 0; i < loaded; ++i) mbar_wait(&empty_b[i % E], (uint32_t)((i / E) & 1));
    }
  }

  // teardown: after a timeout, wait (bounded) for the copies and products still in flight
  tc_fence_before();
  __syncthreads();
  if (abort_flag) {
    if ((warp == 8 || warp == 10) && lane == 0)
      for (int i = loaded > E ? loaded - E : 0; i < loaded; ++i) mbar_wait(&full_b[i % E], (uint32_t)((i / E) & 1));
    if (warp == 9) {  // everything this lane issued before the commit has completed when it arrives
      tc_commit_if(elect_lane(), &sh.drained);
      mbar_wait(&sh.drained, 0);
    }
    __syncthreads();
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// How many rows of a unit share a pass over the cache: 16 (mma.sync), 128 or 256 (tcgen05).
int tile_rows(int T, int G) { return T * G <= kArRows ? kArRows : (T * G <= 128 ? 128 : 256); }

cudaError_t fill_params(const AttendArgs& a, AttendParams& p, int rows) {
  const uint32_t box = rows == kArRows ? kArKeys : (uint32_t)a.cache.page_size;
  const uint32_t tbox = rows == kArRows ? kArKeys : kAtKeys;
  const rkv_cache& c = a.cache;
  const uint64_t prows = (uint64_t)c.num_phys_pages * c.Hkv * c.page_size;
  bool ok = encode_rows_map(&p.tmk, c.k_pages, prows, box) && encode_rows_map(&p.tmv, c.v_pages, prows, box);
  p.tmkt = p.tmk;
  p.tmvt = p.tmv;
  if (a.mask) {
    const uint64_t trows = (uint64_t)c.B * c.Hkv * a.T;
    ok = ok && encode_rows_map(&p.tmkt, a.k_tree, trows, tbox) && encode_rows_map(&p.tmvt, a.v_tree, trows, tbox);
  }
  if (!ok) {
    set_last_error("cuTensorMapEncodeTiled failed for the cache's pages or the tree");
    return cudaErrorInvalidValue;
  }
  p.q = a.q;
  p.mask = a.mask;
  p.page_table = c.page_table;
  p.seq_len = c.seq_len;
  p.tree_len = a.tree_len;
  p.err = c.error_word;
  p.out = a.out;
  p.lse = a.lse;
  p.acc = a.acc;
  p.acc_stride = a.acc_stride;
  p.B = c.B;
  p.Hq = a.Hq;
  p.Hkv = c.Hkv;
  p.G = a.Hq / c.Hkv;
  p.gshift = log2_int(p.G);
  p.T = a.T;
  p.words = (a.T + 31) / 32;
  p.P = c.page_size;
  p.pshift = log2_int(c.page_size);
  p.max_pages = c.max_pages;
  p.num_phys = c.num_phys_pages;
  p.zstride = c.max_pages * c.page_size;
  p.z = nullptr;
  p.row_ml = nullptr;
  p.part_o = nullptr;
  p.part_ml = nullptr;
  p.row_tiles = 0;
  p.N = num_sms();
  p.scale_log2 = a.scale * 1.4426950408889634f;
  return cudaSuccess;
}

}  // namespace

size_t attend_ws_bytes(int B, int Hq, int Hkv, int T, int max_pages, int page_size, bool weights) {
  const size_t rows = (size_t)2 * kMaxSms * tile_rows(T, Hq / Hkv > 0 ? Hq / Hkv : 1);
  size_t n = align256(rows * 128 * 4) + align256(rows * 8);
  if (weights) n += align256((size_t)B * Hq * 8) + align256((size_t)B * Hq * max_pages * page_size * 4);
  return n;
}

// Whether attend_units takes the call, with clusters of how many CTAs (0: it does not).
// The host knows the caches' capacity, not their lengths.  One wave of clusters (a CTA an
// SM; with four warps three) against the line split over all SMs plus the join, one token,
// 8 KV heads, us: 1 x 515 tokens 7.3 (C = 8) against 11.3, 1 x 2563 10.0 against 12.1, 1 x
// 8192 16.5 against 15.1; 4 x 4096 16.4 (C = 4) against 20.5; 16 x 600 13.1 (C = 2, four
// warps) against 16.8, 16 x 4000 57.4 against 55.5; 64 x 300 25.4 (C = 1) against 32.4, 64
// x 2000 110 against 99.  Two row tiles, 2 KV heads, 515 tokens: 9.4 against 11.3 on the
// tensor-core tiles; 32 units of four row tiles no longer gain.
int units_cluster(const AttendArgs& a) {
  const rkv_cache& c = a.cache;
  const int tiles = (a.T * (a.Hq / c.Hkv) + kArRows - 1) / kArRows, cap = c.max_pages * c.page_size;
  const long long units = (long long)c.B * c.Hkv * tiles;
  if (units > 65535 || (tiles > 1 && units > 8)) return 0;
  const int C = units <= 9 ? 8 : (units <= 36 ? 4 : (units <= 300 ? 2 : 1));
  return cap <= C * (C == 8 ? 1024 : (C == 4 ? 1536 : 512)) ? C : 0;
}

cudaError_t launch_units(const AttendArgs& a, AttendParams& p, int C, cudaStream_t s) {
  const rkv_cache& c = a.cache;
  p.row_tiles = (a.T * p.G + kArRows - 1) / kArRows;
  const int cap = (c.max_pages * c.page_size) / kArKeys + (a.mask ? (a.T + kArKeys - 1) / kArKeys : 0);
  const int z_tokens = a.acc ? (cap + C - 1) / C * kArKeys : 0;
  const bool four = C <= 2;
  const int smem = four ? UnitsShape<4>::smem(z_tokens, p.G) : UnitsShape<8>::smem(z_tokens, p.G);
  void (*kernel)(AttendParams) = four ? attend_units_kernel<4> : attend_units_kernel<8>;
  static SmemOptIn opt[2];
  cudaError_t e = opt[four].raise(reinterpret_cast<const void*>(kernel), UnitsShape<8>::smem(kMaxUnitTokens, 8));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, (unsigned)(c.B * c.Hkv * p.row_tiles));
  cfg.blockDim = dim3(four ? UnitsShape<4>::kThreads : UnitsShape<8>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  launch_begin(K_ATTEND_UNITS, s);
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  launch_end(K_ATTEND_UNITS, s);
  return e;
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  AttendParams p;
  const rkv_cache& c = a.cache;
  const int C = units_cluster(a);
  cudaError_t e = fill_params(a, p, C > 0 ? kArRows : tile_rows(a.T, a.Hq / c.Hkv));
  if (e != cudaSuccess) return e;
  if (p.N > kMaxSms) p.N = kMaxSms;
  if (C > 0) return launch_units(a, p, C, s);
  const int tile = tile_rows(a.T, p.G);
  const size_t rows = (size_t)2 * kMaxSms * tile;
  uint8_t* w = static_cast<uint8_t*>(a.ws);
  p.part_o = reinterpret_cast<float*>(w);
  w += align256(rows * 128 * 4);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += align256(rows * 8);
  p.row_ml = nullptr;
  p.z = nullptr;
  if (a.acc) {
    p.row_ml = reinterpret_cast<float2*>(w);
    w += align256((size_t)c.B * a.Hq * 8);
    p.z = reinterpret_cast<float*>(w);
  }
  const long long jrows = ((long long)c.B * a.Hq * a.T + 7) / 8, jmost = 8LL * p.N;
  const dim3 jgrid((unsigned)(jrows < jmost ? jrows : jmost));
  if (tile > kArRows) {
    const bool wide = tile == 256;
    static SmemOptIn opt[2];
    const int smem = wide ? TileShape<true>::kSmem : TileShape<false>::kSmem;
    const void* f = wide ? reinterpret_cast<const void*>(attend_tiles_kernel<true>)
                         : reinterpret_cast<const void*>(attend_tiles_kernel<false>);
    if ((e = opt[wide].raise(f, smem)) != cudaSuccess) return e;
    launch_begin(K_ATTEND_TILES, s);
    if (wide)
      attend_tiles_kernel<true><<<p.N, kAtThreads, smem, s>>>(p);
    else
      attend_tiles_kernel<false><<<p.N, kAtThreads, smem, s>>>(p);
    launch_end(K_ATTEND_TILES, s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return wide ? launch_dependent(attend_combine_kernel<256, kAtKeys>, jgrid, 256, K_ATTEND_COMBINE, s, p)
                : launch_dependent(attend_combine_kernel<128, kAtKeys>, jgrid, 256, K_ATTEND_COMBINE, s, p);
  }
  static SmemOptIn opt;
  if ((e = opt.raise(reinterpret_cast<const void*>(attend_rows_kernel), kArSmem)) != cudaSuccess) return e;
  launch_begin(K_ATTEND_ROWS, s);
  attend_rows_kernel<<<p.N, kArThreads, kArSmem, s>>>(p);
  launch_end(K_ATTEND_ROWS, s);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (!a.acc)
    return launch_dependent(attend_combine_kernel<kArRows, kArKeys>, jgrid, 256, K_ATTEND_COMBINE, s, p);
  const int joins = c.B * ((a.Hq + 7) / 8);
  const long long blocks = (long long)c.B * c.Hkv * ((p.zstride + kWeighTokens - 1) / kWeighTokens);
  const long long most = 8LL * p.N;
  return launch_dependent(attend_weigh_kernel, dim3(joins + (unsigned)(blocks < most ? blocks : most)), 256,
                          K_ATTEND_WEIGH, s, p);
}

}  // namespace rkv
