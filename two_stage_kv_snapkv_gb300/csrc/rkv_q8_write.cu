// The write side of the 8-bit cache: new tokens, or a whole bf16 cache, rounded to codes with
// one power of two a page and KV head.
//
//   scale = 2^ceil(log2(max |x| / largest code)),  code = round(x / scale)
// A page that holds tokens already keeps the larger of its scale and the new rows'; where it
// grows, the old codes are rounded again to it (dividing by a power of two is exact, so only
// codes that fall below the smallest step change their value).
//
// Bound by its bytes: two read and one written a value.  A warp takes up to 16 rows of a page
// in registers (a row's 256 bytes are 16 lanes' 16-byte loads, two rows at a time, so K and V
// are 16 loads in flight a lane), finds their largest magnitude and rounds them: every value
// is read once.  A page's 16-row pieces are neighbouring warps of a CTA and meet in shared
// memory for the maximum.  Measured: prompts of up to 16384 tokens of 8 sequences (574 MB) 95 us,
// 6.0 TB/s; a bf16 cache of 16 x up to 9675 tokens (545 MB) 88 us, 6.2 TB/s, 91 % of a plain copy's
// rate (108 and 103 with CTAs that are not all resident at once); one token of 64 sequences 4.4 us.
#include "rkv_internal.h"
#include "rkv_flat.cuh"
#include "rkv_q8.cuh"

namespace rkv {
namespace {

struct Q8WriteParams {
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;
  const int32_t* page_table;
  int32_t* seq_len;
  int32_t* sync;
  int32_t* err;
  // rkv_q8_append: rows with strides
  const rkv_bf16 *k_new, *v_new;
  int64_t ks[3], vs[3];
  const int32_t* new_len;
  int T;
  // rkv_q8_load: another cache's pages
  const rkv_bf16 *k_pages, *v_pages;
  const int32_t* src_table;
  const int32_t* src_len;
  int src_pages, src_phys;
  int B, Hkv, P, pshift, max_pages, num_phys;
};

// The pair of 16-bit magnitudes' maximum, and whether a value is not finite (0x7f80 and above).
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) { return __vmaxu2(m, x & 0x7fff7fffu); }

// Eight bf16 values divided by a power of two, as codes.
template <int kFormat>
__device__ __forceinline__ uint2 encode8(uint4 x, float inv) {
  return make_uint2(
      encode4<kFormat>(bf16_lo(x.x) * inv, bf16_hi(x.x) * inv, bf16_lo(x.y) * inv, bf16_hi(x.y) * inv),
      encode4<kFormat>(bf16_lo(x.z) * inv, bf16_hi(x.z) * inv, bf16_lo(x.w) * inv, bf16_hi(x.w) * inv));
}

__device__ __forceinline__ uint32_t finite2(uint32_t x) {  // values that are not finite become 0
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

// Old codes of a row (16 lanes, eight each) rounded to a larger scale; f = old / new.
template <int kFormat>
__device__ __forceinline__ void recode8(uint8_t* at, float f) {
  uint2 w = *reinterpret_cast<uint2*>(at);
  uint32_t* v[2] = {&w.x, &w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    decode4<kFormat>(*v[i], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    *v[i] = encode4<kFormat>(a.x * f, a.y * f, b.x * f, b.y * f);
  }
  *reinterpret_cast<uint2*>(at) = w;
}

// A warp's piece of a page of KV head g: the page's rows [r0, r1) (at most 16, none when r0 >=
// r1) are new, rows [0, held) were there before the call; src(r, v) is where row r's 256 bytes
// of K or V are.  The kPieces warps that share a page all get here, with their slot `top`
// zeroed.  A page that cannot be written (`phys` out of range) is read all the same, so that
// no load waits for the table's.
template <int kFormat, int kPieces, class Src>
__device__ __forceinline__ void write_rows(const Q8WriteParams& p, int phys, int g, int r0, int r1, int held, Src src,
                                           uint32_t* top) {
  const int lane = threadIdx.x & 31, sub = lane >> 4, piece = lane & 15;
  uint4 x[2][8];
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 2 * i + sub;
      x[v][i] = r < r1 ? *(reinterpret_cast<const uint4*>(src(r, v)) + piece) : make_uint4(0, 0, 0, 0);
    }
  const bool ok = phys >= 0 && phys < p.num_phys;
  if (!ok && lane == 0) flag_error(p.err, RKV_DEVERR_PAGE_ID);
  const size_t unit = (size_t)(ok ? phys : 0) * p.Hkv + g;
  auto largest = [&](int v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      m = max_abs2(max_abs2(max_abs2(max_abs2(m, x[v][i].x), x[v][i].y), x[v][i].z), x[v][i].w);
    return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  };
  uint32_t most[2] = {largest(0), largest(1)};
  if (kPieces > 1) {
    if (lane < 2) atomicMax(&top[lane], lane ? most[1] : most[0]);
    __syncthreads();
    most[0] = top[0];
    most[1] = top[1];
  }
  const bool broken = most[0] >= 0x7f80u || most[1] >= 0x7f80u;
  if (broken) {  // a NaN or an infinity: both scales become NaN, the codes mean nothing
#pragma unroll
    for (int v = 0; v < 2; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[v][i] = make_uint4(finite2(x[v][i].x), finite2(x[v][i].y), finite2(x[v][i].z), finite2(x[v][i].w));
      most[v] = largest(v);
    }
  }
  const bool first = r0 == held && r0 < r1;  // of the page's pieces: it has what all share to write
  float s[2], was[2] = {0.f, 0.f};
  if (held > 0 && ok) {
    was[0] = p.k_scale[unit];
    was[1] = p.v_scale[unit];
  }
  const bool gone = broken || was[0] != was[0] || was[1] != was[1];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint8_t* const codes = (v ? p.v_codes : p.k_codes) + unit * p.P * 128;
    s[v] = scale_of<kFormat>(most[v] << 16);
    if (held > 0) {
      if (was[v] >= s[v]) {
        s[v] = was[v];
      } else if (first && ok && !gone) {
        const float f = was[v] * inverse_scale(s[v]);
        for (int r = sub; r < held; r += 2) recode8<kFormat>(codes + r * 128 + piece * 8, f);
      }
    }
    const float inv = inverse_scale(s[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 2 * i + sub;
      if (r < r1 && ok) *reinterpret_cast<uint2*>(codes + r * 128 + piece * 8) = encode8<kFormat>(x[v][i], inv);
    }
  }
  if (kPieces > 1) __syncthreads(); else __syncwarp();  // the old scales have been read
  if (first && ok && lane < 2) (lane ? p.v_scale : p.k_scale)[unit] = gone ? __uint_as_float(0x7fffffffu) : (lane ? s[1] : s[0]);
}

// New rows of sequence b: false when it is left as it is.
__device__ __forceinline__ bool new_rows(const Q8WriteParams& p, int b, bool flags, int& n, int& m) {
  n = p.seq_len[b];
  m = p.new_len ? p.new_len[b] : p.T;
  int bad = 0;
  if (m < 0 || m > p.T) bad = RKV_DEVERR_TREE;
  else if (n < 0 || (long long)n + m > (long long)p.max_pages * p.P) bad = RKV_DEVERR_CAPACITY;
  if (bad && flags) flag_error(p.err, bad);
  return bad == 0;
}

struct NewRows {  // row r of the page whose first row is new row `at` (which may lie before the rows)
  const rkv_bf16 *k, *v;
  int64_t ks, vs;
  __device__ __forceinline__ NewRows(const Q8WriteParams& p, int b, int g, int at)
      : k(p.k_new + b * p.ks[0] + g * p.ks[1] + at * p.ks[2]),
        v(p.v_new + b * p.vs[0] + g * p.vs[1] + at * p.vs[2]),
        ks(p.ks[2]),
        vs(p.vs[2]) {}
  __device__ __forceinline__ const rkv_bf16* operator()(int r, int which) const { return which ? v + r * vs : k + r * ks; }
};

// At most 16 new tokens (a decode step): a warp for each KV head and touched page, of which a
// sequence has at most two; its CTAs count themselves in sync[b] and the last one moves the
// length on.
constexpr int kWrWarps = 8;
constexpr int kWrSmall = 16;
constexpr int kWrCtas = 2;  // of an SM, all resident: 16 loads in flight a lane take 128 registers

template <int kFormat>
__global__ void __launch_bounds__(kWrWarps * 32) q8_append_small_kernel(const __grid_constant__ Q8WriteParams p) {
  const int b = blockIdx.y, warp = threadIdx.x >> 5;
  int n, m;
  if (!new_rows(p, b, blockIdx.x == 0 && threadIdx.x == 0, n, m)) return;  // the same in all of its CTAs
  const int pages = p.T > 1 ? 2 : 1, u = blockIdx.x * kWrWarps + warp;
  const int g = u / pages, pg = (n >> p.pshift) + u % pages, lo = pg << p.pshift;
  const int r0 = max(n - lo, 0), r1 = min(n + m - lo, p.P);
  if (g < p.Hkv && r0 < r1)
    write_rows<kFormat, 1>(p, p.page_table[(size_t)b * p.max_pages + pg], g, r0, r1, r0, NewRows(p, b, g, lo - n),
                           nullptr);
  __syncthreads();  // every warp has read the old length
  if (threadIdx.x == 0 && m > 0) {
    bool last = gridDim.x == 1;
    if (!last) {
      __threadfence();
      last = atomicAdd(&p.sync[b], 1) == (int)gridDim.x - 1;
      if (last) p.sync[b] = 0;
    }
    if (last) p.seq_len[b] = n + m;
  }
}

// Any number of tokens: the touched pages of all sequences and KV heads form one line (KV head
// after KV head, each with its pages in order), which the grid's CTAs take eight warps' worth
// at a time.
struct WriteLine {
  long long base[RKV_MAX_BATCH + 1];
  int n[RKV_MAX_BATCH], m[RKV_MAX_BATCH];  // tokens before the call, new ones
  uint32_t top[kWrWarps][2];
  int last;
};

template <int kFormat, int kPieces, bool kLoad>
__global__ void __launch_bounds__(kWrWarps * 32, kWrCtas) q8_write_kernel(const __grid_constant__ Q8WriteParams p) {
  constexpr int kPages = kWrWarps / kPieces;  // pages of a CTA at a time
  __shared__ WriteLine line;
  const int tid = threadIdx.x, warp = tid >> 5, slot = warp / kPieces;
  for (int b = tid; b < p.B; b += kWrWarps * 32) {
    int n = 0, m = 0;
    bool ok;
    if (kLoad) {
      m = p.src_len[b];
      ok = m >= 0 && m <= min(p.max_pages, p.src_pages) * p.P;
      if (!ok && blockIdx.x == 0) flag_error(p.err, RKV_DEVERR_CAPACITY);
    } else {
      ok = new_rows(p, b, blockIdx.x == 0, n, m);
    }
    line.n[b] = n;
    line.m[b] = ok ? m : 0;
  }
  if (tid < kWrWarps * 2) line.top[tid >> 1][tid & 1] = 0u;
  __syncthreads();
  auto touched = [&](int b) {
    return line.m[b] > 0 ? ((line.n[b] + line.m[b] - 1) >> p.pshift) - (line.n[b] >> p.pshift) + 1 : 0;
  };
  flat_scan(line.base, p.B, [&](int b) { return (long long)touched(b) * p.Hkv; });
  const long long total = line.base[p.B];
  for (long long x0 = (long long)blockIdx.x * kPages; x0 < total; x0 += (long long)gridDim.x * kPages) {
    const long long x = x0 + slot;
    int r0 = 0, r1 = 0, held = 0, phys = 0, g = 0, b = 0, pg = 0;
    if (x < total) {
      int hi = p.B - 1;
      while (b < hi) {
        const int mid = (b + hi + 1) >> 1;
        if (line.base[mid] <= x) b = mid; else hi = mid - 1;
      }
      const int n = line.n[b], m = line.m[b], pages = touched(b), off = (int)(x - line.base[b]);
      g = off / pages;
      pg = (n >> p.pshift) + off % pages;
      const int lo = pg << p.pshift;
      phys = p.page_table[(size_t)b * p.max_pages + pg];
      held = max(n - lo, 0);
      r0 = max(held, (warp % kPieces) * 16);
      r1 = min(min(n + m - lo, p.P), (warp % kPieces) * 16 + 16);
    }
    if (kLoad) {
      const int from = x < total ? p.src_table[(size_t)b * p.src_pages + pg] : 0;
      const bool there = from >= 0 && from < p.src_phys;
      const size_t row0 = ((size_t)(there ? from : 0) * p.Hkv + g) * p.P * 128;
      write_rows<kFormat, kPieces>(
          p, phys, g, r0, there ? r1 : r0, held,
          [&](int r, int v) { return (v ? p.v_pages : p.k_pages) + row0 + (size_t)r * 128; }, line.top[slot]);
      // a page that cannot be read: what its tokens would be is not known
      if (!there && (tid & 31) < 2 && warp % kPieces == 0) {
        flag_error(p.err, RKV_DEVERR_PAGE_ID);
        if (phys >= 0 && phys < p.num_phys)
          ((tid & 1) ? p.v_scale : p.k_scale)[(size_t)phys * p.Hkv + g] = __uint_as_float(0x7fffffffu);
      }
    } else {
      const int lo = (pg << p.pshift) - line.n[b];
      write_rows<kFormat, kPieces>(p, phys, g, r0, r1, held, NewRows(p, b, g, lo), line.top[slot]);
    }
    if (kPieces > 1) {
      if (tid < kWrWarps * 2) line.top[tid >> 1][tid & 1] = 0u;  // read before write_rows' last barrier
      __syncthreads();
    }
  }
  __syncthreads();  // every thread of this CTA has read the old lengths
  if (tid == 0) {
    __threadfence();
    line.last = atomicAdd(&p.sync[0], 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (line.last) {
    for (int b = tid; b < p.B; b += kWrWarps * 32)
      if (kLoad || line.m[b] > 0) p.seq_len[b] = line.n[b] + line.m[b];
    if (tid == 0) p.sync[0] = 0;
  }
}

Q8WriteParams cache_params(const rkv_cache8& c) {
  Q8WriteParams p = {};
  p.k_codes = c.k_codes;
  p.v_codes = c.v_codes;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.page_table = c.page_table;
  p.seq_len = c.seq_len;
  p.sync = c.sync;
  p.err = c.error_word;
  p.B = c.B;
  p.Hkv = c.Hkv;
  p.P = c.page_size;
  p.pshift = log2_int(c.page_size);
  p.max_pages = c.max_pages;
  p.num_phys = c.num_phys_pages;
  return p;
}

template <int kFormat, bool kLoad>
cudaError_t launch_line(const Q8WriteParams& p, long long most_pages, int kind, cudaStream_t s) {
  const int pieces = p.P / 16;
  const long long units = (long long)p.B * p.Hkv * most_pages, ctas = (units * pieces + kWrWarps - 1) / kWrWarps;
  const long long most = (long long)kWrCtas * num_sms();
  const unsigned grid = (unsigned)(ctas < most ? ctas : most);
  void (*kernel)(Q8WriteParams) = pieces == 1   ? q8_write_kernel<kFormat, 1, kLoad>
                                  : pieces == 2 ? q8_write_kernel<kFormat, 2, kLoad>
                                                : q8_write_kernel<kFormat, 4, kLoad>;
  launch_begin(kind, s);
  kernel<<<grid, kWrWarps * 32, 0, s>>>(p);
  launch_end(kind, s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendArgs& a, cudaStream_t s) {
  Q8WriteParams p = cache_params(a.cache);
  p.k_new = a.k_new;
  p.v_new = a.v_new;
  for (int i = 0; i < 3; ++i) {
    p.ks[i] = a.k_strides[i];
    p.vs[i] = a.v_strides[i];
  }
  p.T = a.T;
  p.new_len = a.new_len;
  const bool int8 = a.cache.format == RKV_Q8_INT8;
  if (a.T <= kWrSmall) {
    const int units = p.Hkv * (a.T > 1 ? 2 : 1);
    const dim3 grid((units + kWrWarps - 1) / kWrWarps, p.B);
    launch_begin(K_Q8_APPEND, s);
    if (int8) q8_append_small_kernel<RKV_Q8_INT8><<<grid, kWrWarps * 32, 0, s>>>(p);
    else q8_append_small_kernel<RKV_Q8_E4M3><<<grid, kWrWarps * 32, 0, s>>>(p);
    launch_end(K_Q8_APPEND, s);
    return cudaGetLastError();
  }
  const long long pages = (a.T + p.P - 1) / p.P + 1;
  return int8 ? launch_line<RKV_Q8_INT8, false>(p, pages, K_Q8_APPEND, s)
              : launch_line<RKV_Q8_E4M3, false>(p, pages, K_Q8_APPEND, s);
}

cudaError_t launch_q8_load(const Q8LoadArgs& a, cudaStream_t s) {
  Q8WriteParams p = cache_params(a.cache);
  p.k_pages = a.src.k_pages;
  p.v_pages = a.src.v_pages;
  p.src_table = a.src.page_table;
  p.src_len = a.src.seq_len;
  p.src_pages = a.src.max_pages;
  p.src_phys = a.src.num_phys_pages;
  const long long pages = p.max_pages < p.src_pages ? p.max_pages : p.src_pages;
  return a.cache.format == RKV_Q8_INT8 ? launch_line<RKV_Q8_INT8, true>(p, pages, K_Q8_LOAD, s)
                                       : launch_line<RKV_Q8_E4M3, true>(p, pages, K_Q8_LOAD, s);
}

}  // namespace rkv
