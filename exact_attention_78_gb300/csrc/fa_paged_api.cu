// C ABI of the paged-cache operators (include/fa_paged.h): argument
// validation and dispatch.  No device memory is allocated here.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa_diag.h"
#include "fa_paged.h"
#include "paged_internal.h"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxGroup = 128;      // query heads per key/value head
constexpr int kMaxHkv = 4096;       // (the cache kernels' row arithmetic)
constexpr int kMinPage = 16, kMaxPage = 1024;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }

// What every call with a cache checks; fills `s`.
fa_status check_cache(const void* k_pages, const void* v_pages, const void* k_scale, const void* v_scale, int B,
                      int Hkv, int Sn, int D, int num_pages, int page_size, int max_pages, const int* block_table,
                      const int* seq_lens, const int* cu, PagedSeqs* s) {
  if (!k_pages || !v_pages || !block_table || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu, 4))
    return FA_ERR_INVALID_ARG;
  if ((k_scale == nullptr) != (v_scale == nullptr) || !aligned(k_scale, 16) || !aligned(v_scale, 16))
    return FA_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || Sn <= 0 || num_pages <= 0 || max_pages <= 0) return FA_ERR_INVALID_ARG;
  if (page_size <= 0 || (page_size & (page_size - 1)) != 0) return FA_ERR_INVALID_ARG;
  if (page_size < kMinPage || page_size > kMaxPage) return FA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (Hkv > kMaxHkv) return FA_ERR_UNSUPPORTED;
  if (B > kMaxPackedSeqs || (long long)max_pages * page_size > (1ll << 30)) return FA_ERR_UNSUPPORTED;
  // (page, head) pairs and rows of the new tokens fit 32-bit indices
  if ((long long)num_pages * Hkv > INT32_MAX) return FA_ERR_UNSUPPORTED;
  if ((cu ? (long long)Sn : (long long)B * Sn) > INT32_MAX - 512) return FA_ERR_UNSUPPORTED;
  s->block_table = block_table;
  s->seq_lens = seq_lens;
  s->cu = cu;
  s->B = B;
  s->Hkv = Hkv;
  s->Sn = Sn;
  s->num_pages = num_pages;
  s->max_pages = max_pages;
  s->page_shift = 0;
  while ((1 << s->page_shift) < page_size) ++s->page_shift;
  return FA_OK;
}

// Whether a call takes the decode kernel: up to kDecodeRows rows of one sequence
// and key/value head; else the chunk kernel.  64 sequences of 4096 keys, 32/8
// heads, decode against chunk kernel: 16 rows 177 / 186 us (D = 128 BF16), 127 /
// 222 (E4M3), 97 / 167 and 103 / 185 (D = 64); 32 rows, whose accumulators do not fit
// the registers at D = 128, 412 / 186 and 370 / 222, but 128 / 168 and 145 / 186
// (D = 64).
bool takes_decode(int Hq, int Hkv, int Sn, int D, bool packed, int max_q) {
  return (long long)(packed ? max_q : Sn) * (Hq / Hkv) <= kDecodeRows(D);
}

bool attn_shape_ok(int B, int Hq, int Hkv, int Sn, int D, bool packed, int max_q, fa_status* why) {
  *why = FA_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sn <= 0 || Hq % Hkv != 0) return false;
  if (packed && (max_q <= 0 || max_q > Sn)) return false;
  *why = FA_ERR_UNSUPPORTED;
  if (Hkv > kMaxHkv || Hq / Hkv > kMaxGroup || (D != 64 && D != 128) || B > kMaxPackedSeqs) return false;
  if ((packed ? (long long)Sn : (long long)B * Sn) > INT32_MAX - 512) return false;
  if ((long long)(packed ? max_q : Sn) * (Hq / Hkv) > INT32_MAX - 512) return false;
  return true;
}

size_t workspace_size(int B, int Hq, int Hkv, int Sn, int D, bool packed, int max_q) {
  return takes_decode(Hq, Hkv, Sn, D, packed, max_q) ? paged_decode_workspace(D) : paged_chunk_workspace(D);
}

// `tree`: masks of drafted tokens, or nullptr.
fa_status fwd_paged(const void* q, const void* k_pages, const void* v_pages, const void* k_scale,
                    const void* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int Sn, int D, int num_pages,
                    int page_size, int max_pages, int causal, const uint32_t* tree, float scale,
                    const int* block_table, const int* seq_lens, const int* cu_seqlens, int max_q, void* workspace,
                    size_t workspace_bytes, unsigned long long wait_limit_ns, fa_stream_t stream) {
  try {
    PagedAttnLaunch L{};
    if (!q || !o || !lse || !seq_lens || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16))
      return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    // (a factor of -inf, masked scores, has to be a normal number)
    if (!(scale > 0.0f) || !std::isnormal(scale * kLog2e)) return FA_ERR_INVALID_ARG;
    fa_status st;
    if (!attn_shape_ok(B, Hq, Hkv, Sn, D, cu_seqlens != nullptr, max_q, &st)) return st;
    if (tree && (cu_seqlens ? max_q : Sn) > kMaxTree) return FA_ERR_UNSUPPORTED;
    st = check_cache(k_pages, v_pages, k_scale, v_scale, B, Hkv, Sn, D, num_pages, page_size, max_pages, block_table,
                     seq_lens, cu_seqlens, &L.p.s);
    if (st != FA_OK) return st;
    const size_t need = workspace_size(B, Hq, Hkv, Sn, D, cu_seqlens != nullptr, max_q);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return FA_ERR_WORKSPACE;
    if ((st = device_info(&L.num_sms)) != FA_OK) return st;
    L.p.q = q;
    L.p.o = o;
    L.p.lse = lse;
    L.p.k_scale = static_cast<const uint8_t*>(k_scale);
    L.p.v_scale = static_cast<const uint8_t*>(v_scale);
    L.p.Hq = Hq;
    L.p.group = Hq / Hkv;
    L.p.causal = causal;
    L.p.max_q = cu_seqlens ? max_q : Sn;
    L.p.tree = tree;
    L.p.tree_words = tree ? (L.p.max_q + 31) / 32 : 0;
    L.p.scale_log2 = scale * kLog2e;
    L.p.part = static_cast<float*>(workspace);
    L.p.num_ctas = L.num_sms < kMaxCtas ? L.num_sms : kMaxCtas;
    L.p.wait_limit_ns = wait_limit_ns;
    L.k_pages = k_pages;
    L.v_pages = v_pages;
    L.D = D;
    L.fp8 = k_scale != nullptr;
    const bool decode = takes_decode(Hq, Hkv, Sn, D, cu_seqlens != nullptr, max_q);
    return (decode ? launch_paged_decode : launch_paged_chunk)(L, reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return FA_ERR_CUDA;
  }
}

fa_status cache_weights(const void* q, const float* lse, const void* k_pages, const void* k_scale, float* sums, int B,
                        int Hq, int Hkv, int Sn, int D, int num_pages, int page_size, int max_pages, int causal,
                        float scale, float decay, const int* block_table, const int* seq_lens, const int* cu_seqlens,
                        int max_q, unsigned long long wait_limit_ns, int held, fa_stream_t stream) {
  try {
    WeighParams p{};
    if (!q || !lse || !sums || !seq_lens || !aligned(q, 16) || !aligned(lse, 16) || !aligned(sums, 16))
      return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !std::isnormal(scale) || !(decay >= 0.0f) || !std::isfinite(decay)) return FA_ERR_INVALID_ARG;
    fa_status st;
    if (!attn_shape_ok(B, Hq, Hkv, Sn, D, cu_seqlens != nullptr, max_q, &st)) return st;
    // (no values here: the keys stand in for their check)
    st = check_cache(k_pages, k_pages, k_scale, k_scale, B, Hkv, Sn, D, num_pages, page_size, max_pages, block_table,
                     seq_lens, cu_seqlens, &p.s);
    if (st != FA_OK) return st;
    int num_sms = 0;
    if ((st = device_info(&num_sms)) != FA_OK) return st;
    p.q = q;
    p.lse = lse;
    p.k_pages = k_pages;
    p.k_scale = static_cast<const uint8_t*>(k_scale);
    p.sums = sums;
    p.Hq = Hq;
    p.group = Hq / Hkv;
    p.D = D;
    p.causal = causal;
    p.max_q = cu_seqlens ? max_q : Sn;
    p.scale = scale;
    p.decay = decay;
    p.wait_limit_ns = wait_limit_ns;
    p.held = held;
    return launch_cache_weights(p, num_sms, reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return FA_ERR_CUDA;
  }
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_rope(const void* q, const void* k, void* q_out, void* k_out, int tokens, int Hq, int Hkv, int D,
                  const int* positions, int axes, const int* sections, double base, int restart, int interleaved,
                  int inverse, fa_stream_t stream) {
  try {
    if (!q || !q_out || !positions || !sections || (k == nullptr) != (k_out == nullptr)) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(positions, 4))
      return FA_ERR_INVALID_ARG;
    if (tokens <= 0 || Hq <= 0 || (k && Hkv <= 0) || axes < 1 || axes > 4) return FA_ERR_INVALID_ARG;
    if (!(base >= 1.0) || !std::isfinite(base)) return FA_ERR_INVALID_ARG;
    if ((restart | interleaved | inverse) & ~1) return FA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    long long pairs = 0;
    for (int a = 0; a < axes; ++a) {
      if (sections[a] < 1) return FA_ERR_INVALID_ARG;
      pairs += sections[a];
    }
    if (pairs > D / 2) return FA_ERR_INVALID_ARG;
    // the largest loop index of a thread block: 4 tokens of 16 pieces per head
    if ((long long)Hq + (k ? Hkv : 0) > (1 << 20)) return FA_ERR_UNSUPPORTED;
    if (tokens > INT32_MAX - 512) return FA_ERR_UNSUPPORTED;      // (the grid's size and the last block's tokens)
    int num_sms = 0;
    fa_status st = device_info(&num_sms);
    if (st != FA_OK) return st;
    RopeParams p{};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.positions = positions;
    p.tokens = tokens;
    p.Hq = Hq;
    p.Hkv = k ? Hkv : 0;
    p.D = D;
    p.axes = axes;
    p.pairs = (int)pairs;
    p.interleaved = interleaved;
    p.inverse = inverse;
    // Frequencies base^-x as 2^-y, y = x log2 base.  y is rounded by 2^-52 of
    // itself, which moves 2^-y by less than 2^-53; against 60 digits the turns
    // are off by 2^-55 at most.
    const double log2_base = std::log2(base);
    int i = 0;
    for (int a = 0; a < axes; ++a)
      for (int j = 0; j < sections[a]; ++j, ++i) {
        const double f = std::exp2(-log2_base * (restart ? (double)j / sections[a] : (double)i / (double)pairs));
        // turns per position, its whole turns dropped, as a fraction of 2^64.
        // The division by two pi in double is good to 2^-53 of the frequency;
        // a long double would not be the same on both host architectures.
        constexpr double kTwo32 = 4294967296.0;
        double t = f / 6.283185307179586476925;
        t -= std::floor(t);
        const double hi = std::floor(t * kTwo32), lo = (t * kTwo32 - hi) * kTwo32;
        p.turn[i] = ((unsigned long long)hi << 32) + (unsigned long long)lo;
        p.axis[i] = (unsigned char)a;
      }
    return launch_rope(p, num_sms, reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return FA_ERR_CUDA;
  }
}

fa_status fa_cache_write(const void* k, const void* v, void* k_pages, void* v_pages, void* k_scale, void* v_scale,
                         int B, int Hkv, int Sn, int D, int num_pages, int page_size, int max_pages,
                         const int* block_table, const int* seq_lens, const int* cu_seqlens, fa_stream_t stream) {
  try {
    CacheParams p{};
    if (!k || !v || !seq_lens || !aligned(k, 16) || !aligned(v, 16)) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(k_pages, v_pages, k_scale, v_scale, B, Hkv, Sn, D, num_pages, page_size, max_pages,
                               block_table, seq_lens, cu_seqlens, &p.s);
    if (st != FA_OK) return st;
    int num_sms = 0;
    if ((st = device_info(&num_sms)) != FA_OK) return st;
    p.k = k;
    p.v = v;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scale = static_cast<uint8_t*>(k_scale);
    p.v_scale = static_cast<uint8_t*>(v_scale);
    p.D = D;
    p.rows = cu_seqlens ? Sn : B * Sn;
    return launch_cache_write(p, num_sms, reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return FA_ERR_CUDA;
  }
}

fa_status fa_cache_read(const void* k_pages, const void* v_pages, const void* k_scale, const void* v_scale, void* k,
                        void* v, int B, int Hkv, int total, int D, int num_pages, int page_size, int max_pages,
                        const int* block_table, const int* cu_seqlens, fa_stream_t stream) {
  try {
    CacheParams p{};
    if (!k || !v || !cu_seqlens || !aligned(k, 16) || !aligned(v, 16)) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(k_pages, v_pages, k_scale, v_scale, B, Hkv, total, D, num_pages, page_size, max_pages,
                               block_table, nullptr, cu_seqlens, &p.s);
    if (st != FA_OK) return st;
    int num_sms = 0;
    if ((st = device_info(&num_sms)) != FA_OK) return st;
    p.k = k;
    p.v = v;
    p.k_pages = const_cast<void*>(k_pages);
    p.v_pages = const_cast<void*>(v_pages);
    p.k_scale = static_cast<uint8_t*>(const_cast<void*>(k_scale));
    p.v_scale = static_cast<uint8_t*>(const_cast<void*>(v_scale));
    p.D = D;
    p.rows = total;
    return launch_cache_read(p, num_sms, reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return FA_ERR_CUDA;
  }
}

size_t fa_fwd_paged_workspace_size(int B, int Hq, int Hkv, int Sn, int D, int packed, int max_q) {
  fa_status why;
  if ((packed != 0 && packed != 1) || !attn_shape_ok(B, Hq, Hkv, Sn, D, packed != 0, max_q, &why)) return 0;
  return workspace_size(B, Hq, Hkv, Sn, D, packed != 0, max_q);
}

fa_status fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages, const void* k_scale,
                       const void* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int Sn, int D, int num_pages,
                       int page_size, int max_pages, int causal, float scale, const int* block_table,
                       const int* seq_lens, const int* cu_seqlens, int max_q, void* workspace, size_t workspace_bytes,
                       fa_stream_t stream) {
  return fwd_paged(q, k_pages, v_pages, k_scale, v_scale, o, lse, B, Hq, Hkv, Sn, D, num_pages, page_size, max_pages,
                   causal, nullptr, scale, block_table, seq_lens, cu_seqlens, max_q, workspace, workspace_bytes,
                   kDefaultWaitLimitNs, stream);
}

fa_status fa_fwd_paged_tree(const void* q, const void* k_pages, const void* v_pages, const void* k_scale,
                            const void* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int Sn, int D,
                            int num_pages, int page_size, int max_pages, const unsigned* tree, float scale,
                            const int* block_table, const int* seq_lens, const int* cu_seqlens, int max_q,
                            void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (!tree || !aligned(tree, 4)) return FA_ERR_INVALID_ARG;
  return fwd_paged(q, k_pages, v_pages, k_scale, v_scale, o, lse, B, Hq, Hkv, Sn, D, num_pages, page_size, max_pages,
                   0, tree, scale, block_table, seq_lens, cu_seqlens, max_q, workspace, workspace_bytes,
                   kDefaultWaitLimitNs, stream);
}

fa_status fa_tree_mask(const int* parents, unsigned* mask, int* depth, int B, int Sn, const int* cu_seqlens, int max_q,
                       fa_stream_t stream) {
  try {
    if (!parents || !mask || !depth || !aligned(parents, 4) || !aligned(mask, 4) || !aligned(depth, 4) ||
        !aligned(cu_seqlens, 4))
      return FA_ERR_INVALID_ARG;
    if (B <= 0 || Sn <= 0 || (cu_seqlens && (max_q <= 0 || max_q > Sn))) return FA_ERR_INVALID_ARG;
    TreeParams p{};
    p.max_q = cu_seqlens ? max_q : Sn;
    if (p.max_q > kMaxTree || B > kMaxPackedSeqs || Sn > INT32_MAX - 512) return FA_ERR_UNSUPPORTED;
    int num_sms = 0;
    fa_status st = device_info(&num_sms);
    if (st != FA_OK) return st;
    p.parents = parents;
    p.mask = mask;
    p.depth = depth;
    p.cu = cu_seqlens;
    p.B = B;
    p.Sn = Sn;
    p.words = (p.max_q + 31) / 32;
    return launch_tree_mask(p, reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return FA_ERR_CUDA;
  }
}

fa_status fa_cache_weights(const void* q, const float* lse, const void* k_pages, const void* k_scale, float* sums, int B,
                           int Hq, int Hkv, int Sn, int D, int num_pages, int page_size, int max_pages, int causal,
                           float scale, float decay, const int* block_table, const int* seq_lens, const int* cu_seqlens,
                           int max_q, fa_stream_t stream) {
  return cache_weights(q, lse, k_pages, k_scale, sums, B, Hq, Hkv, Sn, D, num_pages, page_size, max_pages, causal, scale,
                       decay, block_table, seq_lens, cu_seqlens, max_q, kDefaultWaitLimitNs, -1, stream);
}

fa_status fa_cache_select(const float* sums, int* index, int* kept, int B, int Hkv, int num_pages, int page_size,
                          int max_pages, int keep, int first, int recent, const int* block_table, const int* seq_lens,
                          fa_stream_t stream) {
  try {
    SelectParams p{};
    if (!sums || !index || !kept || !seq_lens || !aligned(sums, 16) || !aligned(index, 4) || !aligned(kept, 4))
      return FA_ERR_INVALID_ARG;
    if (keep <= 0 || first < 0 || recent < 0 || first > keep || recent > keep - first) return FA_ERR_INVALID_ARG;
    // (sums have no pages of their own: the checks of the table and the sizes are the pages')
    fa_status st = check_cache(sums, sums, nullptr, nullptr, B, Hkv, 1, 64, num_pages, page_size, max_pages, block_table,
                               seq_lens, nullptr, &p.s);
    if (st != FA_OK) return st;
    if (keep > 1 << 30) return FA_ERR_UNSUPPORTED;
    int num_sms = 0;
    if ((st = device_info(&num_sms)) != FA_OK) return st;
    p.sums = sums;
    p.index = index;
    p.kept = kept;
    p.keep = keep;
    p.first = first;
    p.recent = recent;
    return launch_cache_select(p, num_sms, reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return FA_ERR_CUDA;
  }
}

fa_status fa_cache_keep(void* k_pages, void* v_pages, void* k_scale, void* v_scale, float* sums, int B, int Hkv, int D,
                        int num_pages, int page_size, int max_pages, const int* block_table, const int* index,
                        int heads, int most, const int* counts, const int* start, fa_stream_t stream) {
  try {
    KeepParams p{};
    if (!index || !counts || !aligned(sums, 16) || !aligned(index, 4) || !aligned(counts, 4) || !aligned(start, 4))
      return FA_ERR_INVALID_ARG;
    if (most <= 0 || (heads != 1 && heads != Hkv)) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(k_pages, v_pages, k_scale, v_scale, B, Hkv, 1, D, num_pages, page_size, max_pages,
                               block_table, nullptr, nullptr, &p.s);
    if (st != FA_OK) return st;
    if (most > 1 << 30) return FA_ERR_UNSUPPORTED;
    int num_sms = 0;
    if ((st = device_info(&num_sms)) != FA_OK) return st;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scale = static_cast<uint8_t*>(k_scale);
    p.v_scale = static_cast<uint8_t*>(v_scale);
    p.sums = sums;
    p.index = index;
    p.counts = counts;
    p.start = start;
    p.D = D;
    p.heads = heads;
    p.most = most;
    return launch_cache_keep(p, num_sms, reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return FA_ERR_CUDA;
  }
}

fa_status fa_diag_fwd_paged(const void* q, const void* k_pages, const void* v_pages, const void* k_scale,
                            const void* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int Sn, int D,
                            int num_pages, int page_size, int max_pages, int causal, float scale,
                            const int* block_table, const int* seq_lens, const int* cu_seqlens, int max_q,
                            void* workspace, size_t workspace_bytes, unsigned long long wait_limit_ns,
                            fa_stream_t stream) {
  if (wait_limit_ns == 0 || wait_limit_ns > 10000000000ull) return FA_ERR_INVALID_ARG;
  return fwd_paged(q, k_pages, v_pages, k_scale, v_scale, o, lse, B, Hq, Hkv, Sn, D, num_pages, page_size, max_pages,
                   causal, nullptr, scale, block_table, seq_lens, cu_seqlens, max_q, workspace, workspace_bytes,
                   wait_limit_ns, stream);
}

fa_status fa_diag_cache_weights(const void* q, const float* lse, const void* k_pages, const void* k_scale, float* sums,
                                int B, int Hq, int Hkv, int Sn, int D, int num_pages, int page_size, int max_pages,
                                int causal, float scale, float decay, const int* block_table, const int* seq_lens,
                                const int* cu_seqlens, int max_q, unsigned long long wait_limit_ns, int held,
                                fa_stream_t stream) {
  if (wait_limit_ns == 0 || wait_limit_ns > 10000000000ull) return FA_ERR_INVALID_ARG;
  if (held < -1 || held >= weigh_barriers(D)) return FA_ERR_INVALID_ARG;
  return cache_weights(q, lse, k_pages, k_scale, sums, B, Hq, Hkv, Sn, D, num_pages, page_size, max_pages, causal, scale,
                       decay, block_table, seq_lens, cu_seqlens, max_q, wait_limit_ns, held, stream);
}

}  // extern "C"
