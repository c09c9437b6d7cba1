// Host-side plumbing of the paged-cache operators: launch descriptors shared
// by the C ABI (fa_paged_api.cu) and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_internal.h"
#include "fa_paged.h"

namespace fa {

constexpr int kMinScaleExp = -110, kMaxScaleExp = 119;   // E4M3 rows: exponent of the scale

// A paged cache and the sequences in it, as every kernel gets them.
struct PagedSeqs {
  const int* block_table;   // [B, max_pages]
  const int* seq_lens;      // [B] (nullptr for the read-back, whose lengths are cu's)
  const int* cu;            // [B + 1] or nullptr: Sn new tokens each
  int B, Hkv, Sn;           // packed: Sn = rows of the packed arrays
  int num_pages, page_shift, max_pages;
};

struct CacheParams {
  PagedSeqs s;
  const void* k;            // packed or dense rows (written by the read-back)
  const void* v;
  void* k_pages;
  void* v_pages;
  uint8_t* k_scale;         // nullptr: BF16 pages
  uint8_t* v_scale;
  int D;
  int rows;                 // rows of k and v
};

struct RopeParams {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const int* positions;
  int tokens, Hq, Hkv, D;   // Hkv = 0 without keys
  int axes, pairs;          // rotary pairs R
  int interleaved, inverse;
  int tb;                   // tokens per thread block
  unsigned long long turn[64];   // turns per position of each pair, as a fraction of 2^64
  unsigned char axis[64];
};

// Most drafted tokens of a sequence.
constexpr int kMaxTree = FA_MAX_TREE;

struct TreeParams {
  const int* parents;
  uint32_t* mask;           // `words` of each token
  int* depth;
  const int* cu;            // [B + 1] or nullptr: Sn tokens each
  int B, Sn, max_q, words;  // packed: Sn = rows of the packed arrays
};

struct WeighParams {
  PagedSeqs s;
  const void* q;
  const float* lse;
  const void* k_pages;
  const uint8_t* k_scale;   // nullptr: BF16 pages
  float* sums;              // [num_pages, Hkv, page_size]
  int Hq, group, D;         // group = Hq / Hkv
  int causal;
  int max_q;
  float scale, decay;
  int held;                 // a barrier that never completes (fa_diag_cache_weights), or -1
  unsigned long long wait_limit_ns;
};

struct SelectParams {
  PagedSeqs s;              // cu = nullptr
  const float* sums;        // [num_pages, Hkv, page_size]
  int* index;               // [B, Hkv, keep]
  int* kept;                // [B]
  int keep, first, recent;
  int cached;               // tokens of a thread block in shared memory
};

struct KeepParams {
  PagedSeqs s;              // seq_lens = cu = nullptr
  void* k_pages;
  void* v_pages;
  uint8_t* k_scale;         // nullptr: BF16 pages
  uint8_t* v_scale;
  float* sums;              // or nullptr
  const int* index;         // [B, heads, most]
  const int* counts;        // [B]
  const int* start;         // [B] or nullptr: 0
  int D, heads, most;       // heads: Hkv or 1
};

struct PagedAttnParams {
  PagedSeqs s;
  const void* q;
  void* o;
  float* lse;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  int Hq, group;            // group = Hq / Hkv
  int causal;
  const uint32_t* tree;     // masks of drafted tokens, tree_words of each new token; or nullptr
  int tree_words;
  int max_q;
  float scale_log2;         // scale * log2(e)
  float* part;              // workspace: partial results
  int num_ctas;             // persistent thread blocks
  unsigned long long wait_limit_ns;
};

struct PagedAttnLaunch {
  PagedAttnParams p;
  const void* k_pages;
  const void* v_pages;
  int D;
  bool fp8;
  int num_sms;
};

// 3-D tensor map over pages [num_pages * Hkv, page_size, D]: boxes of box_rows
// tokens by 128 bytes of D (64 where a row has no more), swizzled by that
// width.
fa_status make_tmap_pages(CUtensorMap* map, const void* base, long long page_heads, int page_size, int D, bool fp8,
                          int box_rows);

// 3-D tensor map over rows [rows, heads, D] of BF16: boxes of box_rows rows by
// `group` heads by 64 columns, 128-byte swizzle.
fa_status make_tmap_rows_group(CUtensorMap* map, const void* base, int rows, int heads, int D, int group,
                               int box_rows);

fa_status device_info(int* num_sms);

// Persistent thread blocks of the attention kernels: one per SM, at most this
// many, so that the workspace's size is known without a device.
constexpr int kMaxCtas = 160;

// Most rows of one sequence and key/value head that the decode kernel takes.
constexpr int kDecodeRows(int D) { return D == 64 ? 32 : 16; }
size_t paged_decode_workspace(int D);
size_t paged_chunk_workspace(int D);

// Launches a kernel that may start while the one before it in the stream still
// runs; it executes griddepcontrol.wait before its first access to global memory.
// Back to back: rope of 16,384 tokens 43.3 -> 40.9 us, cache writes and read-back 2 us
// less each, a decoding step of three calls in a graph 17.5 -> 16.6 us.
template <class... P, class... A>
fa_status launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream,
                            const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status launch_cache_weights(const WeighParams& p, int num_sms, cudaStream_t stream);
// How many of its barriers WeighParams::held may name.
int weigh_barriers(int D);
fa_status launch_cache_select(const SelectParams& p, int num_sms, cudaStream_t stream);
fa_status launch_cache_keep(const KeepParams& p, int num_sms, cudaStream_t stream);
fa_status launch_tree_mask(const TreeParams& p, cudaStream_t stream);
fa_status launch_rope(const RopeParams& p, int num_sms, cudaStream_t stream);
fa_status launch_cache_write(const CacheParams& p, int num_sms, cudaStream_t stream);
fa_status launch_cache_read(const CacheParams& p, int num_sms, cudaStream_t stream);
fa_status launch_paged_decode(const PagedAttnLaunch& L, cudaStream_t stream);
fa_status launch_paged_chunk(const PagedAttnLaunch& L, cudaStream_t stream);

fa_status weigh_take_device_error();
fa_status evict_take_device_error();
fa_status tree_take_device_error();
fa_status cache_take_device_error();
fa_status paged_decode_take_device_error();
fa_status paged_chunk_take_device_error();

}  // namespace fa
