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
// attend_combine joins them.
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
constexpr float kNoMax = -1e30f;                  // running maximum of a row that saw nothing
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWeighTokens = 1024;                // tokens of a weighing block

struct AttendParams {
  CUtensorMap tmk, tmv;    // the page pools as [rows][128] bf16, 16-row x 64-channel boxes
  CUtensorMap tmkt, tmvt;  // the tree's keys and values, the same boxes (T > 0 nodes given)
  const rkv_bf16* q;       // [B][Hq][T][128]
  const uint32_t* mask;    // [B][T][words], null: no tree
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* tree_len;  // null: T nodes everywhere
  int32_t* err;
  rkv_bf16* out;            // [B][Hq][T][128]
  float* lse;               // [B][Hq][T], may be null
  float* part_o;            // [2 N][16][128]
  float2* part_ml;          // [2 N][16]
  float2* row_ml;           // [B][Hkv][G]: final (m, l) of a one-token step, for the weights
  float* z;                 // [B][Hkv][G][zstride] base-2 scaled logits of a one-token step, or null
  float* acc;               // [B][Hkv][acc_stride]
  int B, Hq, Hkv, G, gshift, T, words, P, pshift, max_pages, num_phys, zstride, acc_stride, N;
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

__device__ __forceinline__ void build_rows_table(const AttendParams& p, FlatTable& ft) {
  flat_build(
      ft, p.B, [&](int b) { return checked_len(p, b); }, [&](int b) { return checked_nodes(p, b); },
      [&](int n, int t) { return (n + kArKeys - 1) / kArKeys + (p.mask ? (t + kArKeys - 1) / kArKeys : 0); },
      [&](int t) { return p.Hkv * ((t * p.G + kArRows - 1) / kArRows); });
}

// Rows 16 rt .. of unit (b, g): node and head of row r.
__device__ __forceinline__ size_t out_row(const AttendParams& p, int b, int g, int r) {
  return ((size_t)b * p.Hq + g * p.G + (r & (p.G - 1))) * p.T + (r >> p.gshift);
}

__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY; }

__global__ void __launch_bounds__(kArThreads, 1) attend_rows_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ FlatTable ft;
  __shared__ uint64_t full_b[kArWarps][kArStages];
  __shared__ float wm[kArWarps][kArRows], wl[kArWarps][kArRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* base = align1024(smem);
  uint8_t* ring = base + warp * kArStages * kArStageBytes;
  float* merge = reinterpret_cast<float*>(base + kArWarps * kArStages * kArStageBytes);
  if (lane == 0)
    for (int s = 0; s < kArStages; ++s) mbar_init(&full_b[warp][s], 1);
  if (tid == 0) fence_mbar_init();
  build_rows_table(p, ft);
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
      fx = fr.x + (fr.hi - fr.lo);
      more = flat_run(ft, p.B, fx, x0, x1, fr);
      if (more) fc = fr.lo + warp;
    }
  };
  settle();
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
      const int phys = p.page_table[(size_t)fr.b * p.max_pages + (t0 >> p.pshift)];
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
    fc += kArWarps;
    settle();
  };
  for (int s = 0; s < kArStages; ++s) fetch();

  const int qr = lane >> 2, qc = (lane & 3) * 2;  // fragment row and column pair
  FlatRun cr;
  for (long long x = x0; flat_run(ft, p.B, x, x0, x1, cr); x = cr.x + (cr.hi - cr.lo)) {
    const int b = cr.b, g = cr.unit % p.Hkv, rt = cr.unit / p.Hkv;
    const int n = ft.n[b], nodes = ft.t[b], rows = nodes * p.G;
    const int nc = (n + kArKeys - 1) / kArKeys;
    const int r0 = rt * kArRows + qr, r1 = r0 + 8;
    // the tile's queries as A fragments, eight steps of 16 channels
    uint32_t qa[8][4];
    {
      const uint32_t* q0 = reinterpret_cast<const uint32_t*>(p.q + out_row(p, b, g, r0) * 128);
      const uint32_t* q1 = reinterpret_cast<const uint32_t*>(p.q + out_row(p, b, g, r1) * 128);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        qa[k][0] = r0 < rows ? q0[k * 8 + (lane & 3)] : 0u;
        qa[k][1] = r1 < rows ? q1[k * 8 + (lane & 3)] : 0u;
        qa[k][2] = r0 < rows ? q0[k * 8 + 4 + (lane & 3)] : 0u;
        qa[k][3] = r1 < rows ? q1[k * 8 + 4 + (lane & 3)] : 0u;
      }
    }
    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m0 = kNoMax, m1 = kNoMax, l0 = 0.f, l1 = 0.f;

    for (int c = cr.lo + warp; c < cr.hi; c += kArWarps) {
      const int s = used % kArStages;
      const bool late = !dead && !mbar_wait(&full_b[warp][s], (uint32_t)((used / kArStages) & 1));
      if (__any_sync(0xffffffffu, late)) {
        if (lane == 0) flag_error(p.err, RKV_DEVERR_TIMEOUT);
        dead = true;
      }
      const bool take = !dead && !((skipped >> s) & 1u);
      const int left = c < nc ? n - c * kArKeys : nodes - (c - nc) * kArKeys;  // keys of the chunk from here on
      if (take) {
        uint8_t* st = ring + s * kArStageBytes;
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
        if (p.z) {  // the logits, for the weights (positions behind n hold -inf)
          const size_t zb = ((size_t)(b * p.Hkv + g) * p.G) * p.zstride + (size_t)c * kArKeys + qc;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (r0 < rows)
              *reinterpret_cast<float2*>(p.z + zb + (size_t)r0 * p.zstride + h * 8) = make_float2(z[h][0], z[h][1]);
        }
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
        // The weights enter the second product as bf16 (off by at most 2^-9 of each, as
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
      } else if (p.z) {  // nothing was read: the positions weigh nothing
        for (int i = lane; i < rows * kArKeys; i += 32)
          p.z[((size_t)(b * p.Hkv + g) * p.G + i / kArKeys) * p.zstride + (size_t)c * kArKeys + i % kArKeys] = -INFINITY;
      }
      ++used;
      __syncwarp();  // every lane has read the stage
      if (!dead) fetch();
    }

    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if ((lane & 3) == 0) {
      wm[warp][qr] = m0;
      wl[warp][qr] = l0;
      wm[warp][qr + 8] = m1;
      wl[warp][qr + 8] = l1;
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
              make_float2(o[j][(quarter >> 1) * 2], o[j][(quarter >> 1) * 2 + 1]);
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
          const float inv = L > 0.f ? 1.f / L : 0.f;
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

// Slot of CTA c's part of the unit whose chunks start at ux.
__device__ __forceinline__ size_t part_slot(long long ux, long long total, int c, int N) {
  return 2 * (size_t)c + (flat_first(total, c, N) >= ux ? 0 : 1);
}

// Joins the parts of the split units.  One CTA of 128 threads per (row tile x KV head,
// sequence), thread = channel; it reads the parts (L2 resident) once.
__global__ void __launch_bounds__(128) attend_combine_kernel(const __grid_constant__ AttendParams p) {
  __shared__ FlatTable ft;
  grid_dependency_wait();
  build_rows_table(p, ft);
  const long long total = ft.base[p.B];
  const int N = flat_ctas(total, p.N);
  const int d = threadIdx.x;
  const int b = blockIdx.y;
  for (int unit = blockIdx.x; unit < ft.units[b]; unit += gridDim.x) {
    const int g = unit % p.Hkv, rt = unit / p.Hkv;
    const int live = min(kArRows, ft.t[b] * p.G - rt * kArRows);
    const int per = ft.per[b];
    if (per == 0) {  // nothing to see: no token cached and no tree
      for (int r = 0; r < live; ++r) {
        const size_t orow = out_row(p, b, g, rt * kArRows + r);
        p.out[orow * 128 + d] = 0;
        if (d == 0 && p.lse) p.lse[orow] = -INFINITY;
      }
      continue;
    }
    const long long ux = ft.base[b] + (long long)unit * per;
    const int c0 = flat_cta(ux, total, N), c1 = flat_cta(ux + per - 1, total, N);
    if (c0 == c1) continue;  // final already
    for (int r = 0; r < live; ++r) {
      float M = kNoMax;
      for (int c = c0; c <= c1; ++c) M = fmaxf(M, p.part_ml[part_slot(ux, total, c, N) * kArRows + r].x);
      float L = 0.f, o = 0.f;
      for (int c = c0; c <= c1; ++c) {
        const size_t at = part_slot(ux, total, c, N) * kArRows + r;
        const float2 ml = p.part_ml[at];
        const float f = ex2_approx(ml.x - M);
        L += ml.y * f;
        o += p.part_o[at * 128 + d] * f;
      }
      const size_t orow = out_row(p, b, g, rt * kArRows + r);
      const __nv_bfloat16 v = __float2bfloat16_rn(L > 0.f ? o / L : 0.f);
      p.out[orow * 128 + d] = *reinterpret_cast<const rkv_bf16*>(&v);
      if (d == 0) {
        if (p.lse) p.lse[orow] = lse_of(M, L);
        if (p.z) p.row_ml[((size_t)b * p.Hkv + g) * p.G + r] = make_float2(M, L);
      }
    }
  }
}

// The weights of a one-token step: acc_j += sum_h 2^(z_hj - m_h) / l_h.  Blocks of
// kWeighTokens tokens of a (sequence, KV head), 256 threads with four tokens each; the
// logits were written a moment ago and mostly still lie in L2.
__global__ void __launch_bounds__(256) attend_weigh_kernel(const __grid_constant__ AttendParams p) {
  __shared__ FlatTable ft;
  grid_dependency_wait();
  flat_build(
      ft, p.B, [&](int b) { return checked_len(p, b); }, [&](int) { return 1; },
      [&](int n, int) { return (n + kWeighTokens - 1) / kWeighTokens; }, [&](int) { return p.Hkv; });
  const long long total = ft.base[p.B];
  for (long long x = blockIdx.x; x < total; x += gridDim.x) {
    const int b = flat_seq(ft, p.B, x);
    const long long off = x - ft.base[b];
    const int g = (int)(off / ft.per[b]), blk = (int)(off % ft.per[b]);
    const size_t unit = (size_t)b * p.Hkv + g;
    const int t = blk * kWeighTokens + threadIdx.x * 4, n = ft.n[b];
    if (t >= n) continue;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int h = 0; h < p.G; ++h) {
      const float2 ml = p.row_ml[unit * p.G + h];
      const float base = ml.x + log2f(ml.y);
      const float4 z = *reinterpret_cast<const float4*>(p.z + (unit * p.G + h) * p.zstride + t);
      w[0] += ex2_approx(z.x - base);
      w[1] += ex2_approx(z.y - base);
      w[2] += ex2_approx(z.z - base);
      w[3] += ex2_approx(z.w - base);
    }
    float* a = p.acc + unit * p.acc_stride + t;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (t + e < n) a[e] += w[e];
  }
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <class K, class P>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, int kind, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  launch_begin(kind, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  launch_end(kind, s);
  return e;
}

int log2_int(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

cudaError_t fill_params(const AttendArgs& a, AttendParams& p) {
  const rkv_cache& c = a.cache;
  const uint64_t rows = (uint64_t)c.num_phys_pages * c.Hkv * c.page_size;
  bool ok = encode_rows_map(&p.tmk, c.k_pages, rows, kArKeys) && encode_rows_map(&p.tmv, c.v_pages, rows, kArKeys);
  p.tmkt = p.tmk;
  p.tmvt = p.tmv;
  if (a.mask) {
    const uint64_t trows = (uint64_t)c.B * c.Hkv * a.T;
    ok = ok && encode_rows_map(&p.tmkt, a.k_tree, trows, kArKeys) && encode_rows_map(&p.tmvt, a.v_tree, trows, kArKeys);
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
  p.N = num_sms();
  p.scale_log2 = a.scale * 1.4426950408889634f;
  return cudaSuccess;
}

}  // namespace

size_t attend_ws_bytes(int B, int Hq, int Hkv, int T, int max_pages, int page_size, bool weights) {
  (void)Hkv;
  (void)T;
  size_t n = align256((size_t)2 * kMaxSms * kArRows * 128 * 4) + align256((size_t)2 * kMaxSms * kArRows * 8);
  if (weights) n += align256((size_t)B * Hq * 8) + align256((size_t)B * Hq * max_pages * page_size * 4);
  return n;
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  AttendParams p;
  const rkv_cache& c = a.cache;
  cudaError_t e = fill_params(a, p);
  if (e != cudaSuccess) return e;
  if (p.N > kMaxSms) p.N = kMaxSms;
  uint8_t* w = static_cast<uint8_t*>(a.ws);
  p.part_o = reinterpret_cast<float*>(w);
  w += align256((size_t)2 * kMaxSms * kArRows * 128 * 4);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += align256((size_t)2 * kMaxSms * kArRows * 8);
  p.row_ml = nullptr;
  p.z = nullptr;
  if (a.acc) {
    p.row_ml = reinterpret_cast<float2*>(w);
    w += align256((size_t)c.B * a.Hq * 8);
    p.z = reinterpret_cast<float*>(w);
  }
  static SmemOptIn opt;
  if ((e = opt.raise(reinterpret_cast<const void*>(attend_rows_kernel), kArSmem)) != cudaSuccess) return e;
  launch_begin(K_ATTEND_ROWS, s);
  attend_rows_kernel<<<p.N, kArThreads, kArSmem, s>>>(p);
  launch_end(K_ATTEND_ROWS, s);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int units = c.Hkv * ((a.T * p.G + kArRows - 1) / kArRows);
  e = launch_dependent(attend_combine_kernel, dim3(units < 65536 ? units : 65535, c.B), 128, K_ATTEND_COMBINE, s, p);
  if (e != cudaSuccess || !a.acc) return e;
  const long long blocks = (long long)c.B * c.Hkv * ((p.zstride + kWeighTokens - 1) / kWeighTokens);
  const long long most = 8LL * p.N;
  return launch_dependent(attend_weigh_kernel, dim3((unsigned)(blocks < most ? blocks : most)), 256, K_ATTEND_WEIGH, s, p);
}

}  // namespace rkv
