// Internal launcher interface between the C-ABI layer (rkv_api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "rkv.h"

namespace rkv {

// Kinds of kernel, for launch counting and the optional per-kernel timing.
enum KernelKind {
  K_APPEND_SMALL = 0,
  K_APPEND_PAGES,
  K_APPEND_ADVANCE,
  K_SNAP_STATS,
  K_SNAP_STATS_COMBINE,
  K_SNAP_COLSUM,
  K_SNAP_POOL,
  K_SNAP_SELECT,
  K_SNAP_COMPACT,
  K_HSA_SCORE,
  K_HSA_TOPK,
  K_HSA_ATTEND,
  K_HSA_COMBINE,
  K_HSA_STEP,
  K_RECALL,
  K_CHUNK_GATHER,
  K_SPARQ_SCORE,
  K_SPARQ_TOPK,
  K_SPARQ_ATTEND,
  K_WAIT_SELFTEST,
  K_SPARQ_KEYS_SYNC,
  K_ATTEND_ROWS,
  K_ATTEND_TILES,
  K_ATTEND_UNITS,
  K_ATTEND_COMBINE,
  K_ATTEND_WEIGH,
  K_TREE_COMMIT,
  K_ACCUM_ROWS,
  K_ACCUM_TILES,
  K_ACCUM_JOIN,
  K_EVICT_SELECT,
  K_EVICT_STAGE,
  K_EVICT_COMPACT,
  K_NUM_KINDS
};
const char* kernel_name(int kind);

// Launch bookkeeping: counting and, when enabled, event brackets on `stream`.
void launch_begin(int kind, cudaStream_t stream);
void launch_end(int kind, cudaStream_t stream);
int num_sms();
// SMs a workspace is laid out for (a grid never has more CTAs per SM slot than this).
constexpr int kMaxSms = 256;
// Raises a kernel's dynamic shared memory limit, once for each device it runs on.
struct SmemOptIn {
  std::atomic<uint64_t> done{0};
  cudaError_t raise(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
};
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int log2_int(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}
// A launch that may start while the kernel before it on `s` ends (it must wait for it with
// griddepcontrol.wait before reading what that kernel wrote).
template <class Params>
cudaError_t launch_dependent(void (*kernel)(Params), dim3 grid, int threads, int kind, cudaStream_t s,
                             const Params& p) {
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
// Sets the message rkv_last_error() returns on this thread.
void set_last_error(const char* msg);

// A [rows][128] bf16 array as a 2-D tensor map of box_rows x 64-element boxes with
// 128-byte swizzle (a box row is 128 B; its 16-byte pieces are XOR-ed with row % 8).
// False when the driver's encoder is unavailable or rejects the map.
bool encode_rows_map(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows);

// --------------------------------------------------------------- cache append
cudaError_t launch_append(const rkv_cache& c, const rkv_bf16* k_new, const rkv_bf16* v_new,
                          int n_new, cudaStream_t s);

// --------------------------------------------------------------- prefill
struct PrefillArgs {
  const rkv_bf16* q_win;
  const rkv_bf16* k;
  const rkv_bf16* v;
  int B, Hq, Hkv, G, w, Lmax;
  const int32_t* prompt_len;   // host [B]
  const int32_t* keep1;        // host [B]
  const int32_t* pool_kernel;  // host [B]
  float scale;
  rkv_cache cache;
  int32_t* kept_idx;
  int kept_stride;
  float* pooled_out;  // may be null
  void* ws;
  size_t ws_bytes;
};
size_t prefill_ws_bytes(int B, int Hq, int Hkv, int w, int Lmax);
cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t s);

// Chunked prefill: the held survivors plus one chunk, re-evicted to keep1.
struct PrefillChunkArgs {
  const rkv_bf16* q_win;    // [B][Hq][w][128]: the chunk's last w queries
  const rkv_bf16* k_chunk;  // [B][Hkv][chunk_max][128]
  const rkv_bf16* v_chunk;
  int Hq, w, chunk_max;
  const int32_t* chunk_len;   // host [B]
  const int32_t* held_len;    // host [B]
  const int32_t* keep1;       // host [B]
  const int32_t* pool_kernel; // host [B]
  float scale;
  rkv_cache cache;
  int32_t* kept_idx;
  int kept_stride;
  void* ws;
  size_t ws_bytes;
};
size_t prefill_chunk_ws_bytes(int B, int Hq, int Hkv, int w, int Lc);
cudaError_t launch_prefill_chunk(const PrefillChunkArgs& a, cudaStream_t s);

// --------------------------------------------------------------- decode
enum DecodePath { DECODE_AUTO = 0, DECODE_SPLIT = 1, DECODE_FUSED = 2 };
struct DecodeArgs {
  rkv_cache cache;
  const rkv_bf16* q;
  const rkv_bf16* k_new;  // null: no append (rkv_decode_hsa)
  const rkv_bf16* v_new;
  int mode;               // DecodePath
  int Hq, G;
  const int32_t* k1;  // host [B]
  const int32_t* k2;  // host [B]
  float scale;
  float* out;
  int32_t* sel_channels;
  int32_t* sel_pages;
  int sel_pages_stride;
  void* ws;
  size_t ws_bytes;
  void* keys_t = nullptr;  // token path: the channel-major key copy, or null
};
size_t decode_ws_bytes(int B, int Hq, int Hkv, int max_pages);
// Token path (SparQ-only): k2 counts tokens; k_new must be null.
size_t sparq_ws_bytes(int B, int Hq, int Hkv, int max_pages, int page_size);
int sparq_max_tokens();
size_t sparq_keys_bytes(int B, int Hkv, int max_pages, int page_size);
cudaError_t launch_sparq(const DecodeArgs& a, cudaStream_t s);
bool decode_fused_ok(const rkv_cache& c);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);

// --------------------------------------------------------------- dense rows: tree and weights
struct AttendArgs {
  rkv_cache cache;
  const rkv_bf16* q;  // [B][Hq][T][128]
  int Hq, T;
  const rkv_bf16* k_tree;  // [B][Hkv][T][128] (mask given)
  const rkv_bf16* v_tree;
  const uint32_t* mask;     // [B][T][ceil(T/32)], null: the cache alone
  const int32_t* tree_len;  // device [B] or null
  float scale;
  rkv_bf16* out;
  float* lse;  // may be null
  float* acc;  // [B][Hkv][acc_stride] (T == 1, no mask) or null
  int acc_stride;
  void* ws;
};
size_t attend_ws_bytes(int B, int Hq, int Hkv, int T, int max_pages, int page_size, bool weights);
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s);

struct CommitArgs {
  rkv_cache cache;
  const rkv_bf16* k_tree;
  const rkv_bf16* v_tree;
  int T;
  const int32_t* path;  // device [B][path_stride]
  int path_stride;
  const int32_t* path_len;  // device [B]
};
cudaError_t launch_commit(const CommitArgs& a, cudaStream_t s);

struct AccumRowsArgs {
  rkv_cache cache;
  const rkv_bf16* q;  // [B][Hq][T][128]
  const float* lse;   // [B][Hq][T]
  int Hq, T;
  const int32_t* row_len;  // device [B] or null
  const int32_t* row_ids;  // device [B][ids_stride] or null
  int ids_stride;
  float scale;
  float* acc;
  int acc_stride;
  void* ws;
};
size_t accum_rows_ws_bytes(int B, int Hq, int Hkv, int T, int max_pages, int page_size);
cudaError_t launch_accum_rows(const AccumRowsArgs& a, cudaStream_t s);

struct EvictArgs {
  rkv_cache cache, dst;
  bool in_place;
  const float* acc;
  int acc_stride;
  float* dst_acc;
  int dst_acc_stride;
  const int32_t* keep;  // host [B]
  int recent;
  int32_t* kept_idx;
  int kept_stride;
  void* ws;
};
int evict_max_tokens();
size_t evict_ws_bytes(int B, int Hkv, int max_keep, bool in_place);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);

// --------------------------------------------------------------- diagnostics
struct RecallArgs {
  rkv_cache cache;
  const rkv_bf16* q;
  int Hq;
  const int32_t* sel_pages;
  int sel_pages_stride;
  const int32_t* k_tokens;  // host [B]
  float scale;
  float* recall;
  float* mass;  // may be null
};
int recall_max_tokens();
cudaError_t launch_recall(const RecallArgs& a, cudaStream_t s);

// One CTA that waits, for at most limit_ns, on an mbarrier nothing arrives on, and
// flags RKV_DEVERR_TIMEOUT in err when the wait runs out (the failure path's test).
cudaError_t launch_wait_selftest(int32_t* err, uint64_t limit_ns, cudaStream_t s);

}  // namespace rkv
