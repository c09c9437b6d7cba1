// Writes of new keys and values into the pages of a cache, quantised to E4M3
// on the way or copied as BF16, and the read-back into packed rows.
//
// Both move rows of D values, one token of one head each, and do little
// arithmetic, so HBM bounds them.  A thread block takes consecutive tokens, some
// 128 rows of keys and values, and looks each token's page and slot up once for
// the 2 Hkv rows that share them.  D / 16 lanes take a row, 16 values each (8
// of BF16 pages' read-back), and have several rows in flight.  The rows' own
// loads do not wait for the lookup.
#include <cuda_runtime.h>

#include "paged.cuh"

namespace fa {
namespace cache {

__device__ DeviceError g_err;

using paged::find_sequence;
using paged::record_bad_input;

constexpr int kThreads = 256;
constexpr int kMaxTb = 64;     // tokens per thread block
constexpr int kMinRows = 128;  // rows of a thread block, where there are enough

enum Site { kSiteOffsets = 1, kSitePage };

// Where the block's tokens are: page, or -1 for a row that is skipped, -2 for
// one that reads as zeros (a read-back's bad page); slot in the page.
struct Slots {
  int page[kMaxTb];
  int slot[kMaxTb];
};

// kWrite: a cache write, whose tokens are the last ones of their sequences;
// else a read-back, which counts from the first.  A warp does 32 tokens: it
// searches for the first one's sequence together, and each lane goes on from
// there to its own.
template <bool kWrite>
FA_DEV void find_slots(const PagedSeqs& s, int rows, int tb, Slots& out) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tok0 = blockIdx.x * tb;
  if (warp * 32 >= tb || tok0 + warp * 32 >= rows) return;
  const int i = tok0 + threadIdx.x;
  const int capacity = s.max_pages << s.page_shift;
  int b, pos = -1;
  bool mine = true, good;             // the row belongs to a sequence; its offsets and length keep to the rules
  if (s.cu) {
    b = find_sequence(s.cu, s.B, tok0 + warp * 32, lane);
    if ((int)threadIdx.x >= tb || i >= rows) return;
    while (b < s.B && s.cu[b + 1] <= i) ++b;
    mine = b < s.B;
    if (mine) {
      const int first = s.cu[b], end = s.cu[b + 1];
      const int len = kWrite ? s.seq_lens[b] : end - first;
      good = first >= 0 && i >= first && end <= rows && (b > 0 || first == 0) && len >= 0 && len <= capacity;
      if (good) pos = kWrite ? len - (end - i) : i - first;
    }
  } else {
    if ((int)threadIdx.x >= tb || i >= rows) return;
    b = i / s.Sn;
    const int len = s.seq_lens[b];
    good = len >= 0 && len <= capacity;
    if (good) pos = len - (s.Sn - (i - b * s.Sn));
  }
  int page = -1;
  if (pos >= 0) {                     // below the capacity: a token lies before its sequence's end
    page = s.block_table[(size_t)b * s.max_pages + (pos >> s.page_shift)];
    if (page < 0 || page >= s.num_pages) {
      record_bad_input(&g_err, kSitePage);
      page = kWrite ? -1 : -2;
    }
  }
  if (mine && !good) record_bad_input(&g_err, kSiteOffsets);
  out.page[threadIdx.x] = page;
  out.slot[threadIdx.x] = pos & ((1 << s.page_shift) - 1);
}

// Row r of a block's: token in the block, keys or values, head.
struct Row {
  int tok, which, head;
};
FA_DEV Row row_of(int r, int Hkv, float inv) {      // inv = 1 / (2 Hkv)
  Row x;
  x.tok = (int)(((float)r + 0.5f) * inv);           // exact: r < 2^20
  const int h = r - x.tok * 2 * Hkv;
  x.which = h >= Hkv;
  x.head = h - x.which * Hkv;
  return x;
}

// The rules that no single row shows (first offset, order) are checked by the
// first block, for the report only.
FA_DEV void report_sequences(const PagedSeqs& s) {
  if (blockIdx.x == 0) {
    const bool ok = paged::sequences_ok(s, s.Sn);
    if (!ok && threadIdx.x == 0) record_bad_input(&g_err, kSiteOffsets);
  }
}

// A word of two BF16 values as two E4M3 codes; f = 2^-e.
FA_DEV uint32_t codes_of(uint32_t w, float f) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(h)
      : "f"(__uint_as_float(w & 0xFFFF0000u) * f), "f"(__uint_as_float(w << 16) * f));      // exact products
  return h;
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads) write_kernel(const CacheParams p, int tb) {
  constexpr int kLanes = D / 16;
  constexpr int kGroups = kThreads / kLanes;
  constexpr int kUnroll = kMinRows / kGroups;
  __shared__ Slots slots;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int Hkv = p.s.Hkv;
  const float inv = 1.0f / (float)(2 * Hkv);
  const int tok0 = blockIdx.x * tb;
  const int n = min(tb, p.rows - tok0) * 2 * Hkv;    // rows of this block

  overlap_launches();
  // (n >= 2 Hkv > 0, and every thread makes the same number of steps)
  for (int r0 = 0; r0 < n; r0 += kUnroll * kGroups) {
    uint4 x[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kGroups + group;
      if (r >= n) continue;
      const Row w = row_of(r, Hkv, inv);
      const uint4* src = static_cast<const uint4*>(w.which ? p.v : p.k) +
                         ((size_t)(tok0 + w.tok) * Hkv + w.head) * (D / 8) + 2 * lane;
      x[u][0] = src[0];
      x[u][1] = src[1];
    }
    if (r0 == 0) {
      find_slots<true>(p.s, p.rows, tb, slots);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kGroups + group;
      if (r >= n) continue;
      const Row w = row_of(r, Hkv, inv);
      const int page = slots.page[w.tok];
      // a row's lanes sit in one warp, and each group of lanes goes its own way
      if (page < 0) continue;
      const size_t row = ((size_t)page * Hkv + w.head << p.s.page_shift) + slots.slot[w.tok];
      void* pages = w.which ? p.v_pages : p.k_pages;
      if (!kFp8) {
        uint4* to = static_cast<uint4*>(pages) + row * (D / 8) + 2 * lane;
        to[0] = x[u][0];
        to[1] = x[u][1];
        continue;
      }
      const uint32_t v[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
      uint32_t m2 = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m2 = paged::max_bf16x2(m2, v[i] & 0x7FFF7FFFu);
      uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
      const uint32_t mask = ((1u << kLanes) - 1) << (threadIdx.x % 32 / kLanes * kLanes);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d /= 2) m = max(m, __shfl_xor_sync(mask, m, d));
      // amax = (1 + f / 128) 2^(E - 127), and 448 = 1.75 * 2^8
      int e = (int)(m >> 7) - 127 - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
      e = min(max(e, kMinScaleExp), kMaxScaleExp);
      const bool bad = m >= 0x7F80u;
      const float f = __uint_as_float((uint32_t)(127 - e) << 23);
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = bad ? 0u : codes_of(v[2 * i], f) | codes_of(v[2 * i + 1], f) << 16;
      static_cast<uint4*>(pages)[row * (D / 16) + lane] = make_uint4(c[0], c[1], c[2], c[3]);
      if (lane == 0) (w.which ? p.v_scale : p.k_scale)[row] = bad ? 255 : (uint8_t)(e + 127);
    }
  }
  report_sequences(p.s);
}

// 16 bytes of a row as they lie in the cache are 16 codes (32 bytes of
// output) or 8 BF16 values.
template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads) read_kernel(const CacheParams p, int tb) {
  constexpr int kLanes = kFp8 ? D / 16 : D / 8;
  constexpr int kGroups = kThreads / kLanes;
  constexpr int kUnroll = 4;
  __shared__ Slots slots;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int Hkv = p.s.Hkv;
  const float inv = 1.0f / (float)(2 * Hkv);
  const int tok0 = blockIdx.x * tb;
  const int n = min(tb, p.rows - tok0) * 2 * Hkv;
  overlap_launches();
  find_slots<false>(p.s, p.rows, tb, slots);
  __syncthreads();
  for (int r0 = 0; r0 < n; r0 += kUnroll * kGroups) {
    uint4 x[kUnroll];
    uint32_t scale[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kGroups + group;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      scale[u] = 127;
      if (r >= n) continue;
      const Row w = row_of(r, Hkv, inv);
      const int page = slots.page[w.tok];
      if (page < 0) continue;
      const size_t row = ((size_t)page * Hkv + w.head << p.s.page_shift) + slots.slot[w.tok];
      x[u] = static_cast<const uint4*>(w.which ? p.v_pages : p.k_pages)[row * kLanes + lane];
      if (kFp8) scale[u] = (w.which ? p.v_scale : p.k_scale)[row];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kGroups + group;
      if (r >= n) continue;
      const Row w = row_of(r, Hkv, inv);
      if (slots.page[w.tok] == -1) continue;
      uint4* dst = static_cast<uint4*>(const_cast<void*>(w.which ? p.v : p.k)) +
                   ((size_t)(tok0 + w.tok) * Hkv + w.head) * (D / 8);
      if (!kFp8) {
        dst[lane] = x[u];
        continue;
      }
      // 2^e as a BF16 pair; every product is exact (a code times 2^e is a
      // normal BF16 for every e that a write makes)
      const uint32_t f = scale[u] == 255u ? 0x7FC07FC0u : scale[u] << 7 | scale[u] << 23;
      const uint32_t v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t even = paged::mul_bf16x2(paged::e4m3_even(v[i]), f);
        const uint32_t odd = paged::mul_bf16x2(paged::e4m3_odd(v[i]), f);
        y[2 * i] = __byte_perm(even, odd, 0x5410);
        y[2 * i + 1] = __byte_perm(even, odd, 0x7632);
      }
      dst[2 * lane] = make_uint4(y[0], y[1], y[2], y[3]);
      dst[2 * lane + 1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
  report_sequences(p.s);
}

// Tokens per thread block: enough for kMinRows rows, fewer while that would
// leave SMs without a block.  (18,000 ragged tokens of 8 heads, E4M3: 128 rows
// 19.0 us, 256 rows 23.4 us; one head, 165,000 tokens: 16.1 and 20.0 us, and 39 us
// with 8 tokens a block, whose lookups then cost more than their rows.)
int tokens_per_block(int rows, int Hkv, int num_sms) {
  int tb = 1;
  while (tb < kMaxTb && 2 * Hkv * tb < kMinRows && (long long)rows > (long long)num_sms * 2 * tb) tb *= 2;
  return tb;
}

template <int D>
fa_status launch_write_d(const CacheParams& p, int num_sms, cudaStream_t stream) {
  const int tb = tokens_per_block(p.rows, p.s.Hkv, num_sms);
  const int grid = (p.rows + tb - 1) / tb;
  auto kernel = p.k_scale ? write_kernel<D, true> : write_kernel<D, false>;
  return launch_overlapped(kernel, dim3(grid), kThreads, 0, stream, p, tb);
}

template <int D>
fa_status launch_read_d(const CacheParams& p, int num_sms, cudaStream_t stream) {
  const int tb = tokens_per_block(p.rows, p.s.Hkv, num_sms);
  const int grid = (p.rows + tb - 1) / tb;
  auto kernel = p.k_scale ? read_kernel<D, true> : read_kernel<D, false>;
  return launch_overlapped(kernel, dim3(grid), kThreads, 0, stream, p, tb);
}

}  // namespace cache

fa_status launch_cache_write(const CacheParams& p, int num_sms, cudaStream_t stream) {
  return p.D == 128 ? cache::launch_write_d<128>(p, num_sms, stream) : cache::launch_write_d<64>(p, num_sms, stream);
}

fa_status launch_cache_read(const CacheParams& p, int num_sms, cudaStream_t stream) {
  return p.D == 128 ? cache::launch_read_d<128>(p, num_sms, stream) : cache::launch_read_d<64>(p, num_sms, stream);
}

fa_status cache_take_device_error() {
  DeviceError e{0, 0};
  if (cudaMemcpyFromSymbol(&e, cache::g_err, sizeof(e)) != cudaSuccess) return FA_ERR_CUDA;
  if (e.status != 0) {
    const DeviceError z{0, 0};
    if (cudaMemcpyToSymbol(cache::g_err, &z, sizeof(z)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return static_cast<fa_status>(e.status);
}

}  // namespace fa
