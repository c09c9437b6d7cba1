// Writes of new keys and values into the pages of a cache, quantised to E4M3
// on the way or copied as BF16, and the read-back into packed rows.
//
// Both move rows of D values, one token of one head each, and do next to no
// arithmetic, so HBM bounds them.  A thread block takes a few consecutive
// tokens (`tb`) and all their heads, keys and values: its warps first look up
// each token's page and slot, once for the 2 Hkv rows that share them, then
// D / 8 lanes take a row, 16 bytes of BF16 each.  Four rows are in flight per
// lane.  The rows' own loads do not wait for the lookup.
#include <cuda_runtime.h>

#include "paged.cuh"

namespace fa {
namespace cache {

__device__ DeviceError g_err;

using paged::find_sequence;
using paged::record_bad_input;

constexpr int kThreads = 256;
constexpr int kMaxTb = 8;      // tokens per thread block: one per warp
constexpr int kUnroll = 4;     // rows in flight per lane

enum Site { kSiteOffsets = 1, kSitePage };

// Page and slot of each of the block's tokens, or page -1 for a row that is
// skipped, into shared memory.  `written`: a cache write, whose tokens are the
// last ones of their sequences; else a read-back, which counts from the first
// and takes a bad page as zeros (page -2).
struct Slots {
  int page[kMaxTb];
  int slot[kMaxTb];
};

template <bool kWrite>
FA_DEV void find_slots(const PagedSeqs& s, int rows, int tb, Slots& out) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int i = blockIdx.x * tb + warp;
  if (warp >= tb || i >= rows) return;
  int b, pos = -1;
  bool mine = true, good = true;      // the row belongs to a sequence; its offsets keep to the rules
  if (s.cu) {
    b = find_sequence(s.cu, s.B, i, lane);
    mine = b < s.B;
    if (mine) {
      const int first = s.cu[b], end = s.cu[b + 1];
      good = first >= 0 && i >= first && i < end;
      pos = kWrite ? s.seq_lens[b] - (end - i) : i - first;
      good = good && (!kWrite || s.seq_lens[b] >= 0);
    }
  } else {
    b = i / s.Sn;
    pos = s.seq_lens[b] - (s.Sn - (i - b * s.Sn));
    good = s.seq_lens[b] >= 0;
  }
  good = good && (pos >> s.page_shift) < s.max_pages;
  int page = -1;
  if (mine && good && pos >= 0) {
    page = s.block_table[(size_t)b * s.max_pages + (pos >> s.page_shift)];
    if (page < 0 || page >= s.num_pages) {
      if (lane == 0) record_bad_input(&g_err, kSitePage);
      page = kWrite ? -1 : -2;
    }
  }
  if (mine && !good && lane == 0) record_bad_input(&g_err, kSiteOffsets);
  if (lane == 0) {
    out.page[warp] = page;
    out.slot[warp] = pos & ((1 << s.page_shift) - 1);
  }
}

// The rules that no single row shows (first offset, order) are checked by the
// first block, for the report only.
FA_DEV void report_sequences(const PagedSeqs& s) {
  if (blockIdx.x == 0) {
    const bool ok = paged::sequences_ok(s, s.Sn);
    if (!ok && threadIdx.x == 0) record_bad_input(&g_err, kSiteOffsets);
  }
}

// 8 BF16 values of a row as 8 E4M3 codes; f = 2^-e.
FA_DEV uint2 codes_of(const uint4& x, float f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16) * f, hi = __uint_as_float(w[i] & 0xFFFF0000u) * f;   // exact
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
    c[i] = h;
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads) write_kernel(const CacheParams p, int tb) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kThreads / kLanes;
  __shared__ Slots slots;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int Hkv = p.s.Hkv;
  const int tok0 = blockIdx.x * tb;
  const int n = min(tb, p.rows - tok0) * 2 * Hkv;    // rows of this block
  const uint4* src[2] = {static_cast<const uint4*>(p.k), static_cast<const uint4*>(p.v)};

  // (n >= 2 Hkv > 0, and every thread makes the same number of steps)
  for (int r0 = 0; r0 < n; r0 += kUnroll * kGroups) {
    uint4 x[kUnroll];
    int tok[kUnroll], head[kUnroll], which[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kGroups + group;
      tok[u] = r / (2 * Hkv);
      const int h = r - tok[u] * 2 * Hkv;
      which[u] = h >= Hkv;
      head[u] = h - which[u] * Hkv;
      if (r < n) x[u] = src[which[u]][((size_t)(tok0 + tok[u]) * Hkv + head[u]) * kLanes + lane];
    }
    if (r0 == 0) {
      find_slots<true>(p.s, p.rows, tb, slots);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kGroups + group;
      // a row's lanes sit in one warp, and each group of lanes goes its own way
      if (r >= n || slots.page[tok[u]] < 0) continue;
      const size_t row = ((size_t)slots.page[tok[u]] * Hkv + head[u] << p.s.page_shift) + slots.slot[tok[u]];
      void* pages = which[u] ? p.v_pages : p.k_pages;
      if (!kFp8) {
        static_cast<uint4*>(pages)[row * kLanes + lane] = x[u];
        continue;
      }
      uint32_t m = 0;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      const uint32_t mask = (kLanes == 32 ? 0xFFFFFFFFu : (1u << kLanes) - 1) << (threadIdx.x % 32 / kLanes * kLanes);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d /= 2) m = max(m, __shfl_xor_sync(mask, m, d));
      // amax = (1 + f / 128) 2^(E - 127), and 448 = 1.75 * 2^8
      int e = (int)(m >> 7) - 127 - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
      e = min(max(e, kMinScaleExp), kMaxScaleExp);
      const bool bad = m >= 0x7F80u;
      uint2 c = codes_of(x[u], __uint_as_float((uint32_t)(127 - e) << 23));
      if (bad) c = make_uint2(0u, 0u);
      static_cast<uint2*>(pages)[row * kLanes + lane] = c;
      if (lane == 0) (which[u] ? p.v_scale : p.k_scale)[row] = bad ? 255 : (uint8_t)(e + 127);
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
  __shared__ Slots slots;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int Hkv = p.s.Hkv;
  const int tok0 = blockIdx.x * tb;
  const int n = min(tb, p.rows - tok0) * 2 * Hkv;
  uint4* dst[2] = {static_cast<uint4*>(const_cast<void*>(p.k)), static_cast<uint4*>(const_cast<void*>(p.v))};
  find_slots<false>(p.s, p.rows, tb, slots);
  __syncthreads();
  for (int r0 = 0; r0 < n; r0 += kUnroll * kGroups) {
    uint4 x[kUnroll];
    uint32_t scale[kUnroll];
    int tok[kUnroll], head[kUnroll], which[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kGroups + group;
      tok[u] = r / (2 * Hkv);
      const int h = r - tok[u] * 2 * Hkv;
      which[u] = h >= Hkv;
      head[u] = h - which[u] * Hkv;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      scale[u] = 127;
      if (r < n && slots.page[tok[u]] >= 0) {
        const size_t row = ((size_t)slots.page[tok[u]] * Hkv + head[u] << p.s.page_shift) + slots.slot[tok[u]];
        x[u] = static_cast<const uint4*>(which[u] ? p.v_pages : p.k_pages)[row * kLanes + lane];
        if (kFp8) scale[u] = (which[u] ? p.v_scale : p.k_scale)[row];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kGroups + group;
      if (r >= n || slots.page[tok[u]] == -1) continue;
      const size_t row = (size_t)(tok0 + tok[u]) * Hkv + head[u];
      if (!kFp8) {
        dst[which[u]][row * kLanes + lane] = x[u];
        continue;
      }
      // 2^e as a BF16 pair; every product is exact (a code times 2^e is a
      // normal BF16 for every e that a write makes)
      const uint32_t f = scale[u] == 255u ? 0x7FC07FC0u : scale[u] << 7 | scale[u] << 23;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t even = paged::mul_bf16x2(paged::e4m3_even(w[i]), f);
        const uint32_t odd = paged::mul_bf16x2(paged::e4m3_odd(w[i]), f);
        y[2 * i] = __byte_perm(even, odd, 0x5410);
        y[2 * i + 1] = __byte_perm(even, odd, 0x7632);
      }
      uint4* to = dst[which[u]] + (row * kLanes + lane) * 2;
      to[0] = make_uint4(y[0], y[1], y[2], y[3]);
      to[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
  report_sequences(p.s);
}

// Tokens per thread block: one while that still leaves SMs without a block,
// more where a block's lookup is better shared.
int tokens_per_block(int rows, int num_sms) {
  int tb = 1;
  while (tb < kMaxTb && (long long)rows >= (long long)num_sms * 4 * tb) tb *= 2;
  return tb;
}

template <int D>
fa_status launch_write_d(const CacheParams& p, int num_sms, cudaStream_t stream) {
  const int tb = tokens_per_block(p.rows, num_sms);
  const int grid = (p.rows + tb - 1) / tb;
  if (p.k_scale)
    write_kernel<D, true><<<grid, kThreads, 0, stream>>>(p, tb);
  else
    write_kernel<D, false><<<grid, kThreads, 0, stream>>>(p, tb);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
fa_status launch_read_d(const CacheParams& p, int num_sms, cudaStream_t stream) {
  const int tb = tokens_per_block(p.rows, num_sms);
  const int grid = (p.rows + tb - 1) / tb;
  if (p.k_scale)
    read_kernel<D, true><<<grid, kThreads, 0, stream>>>(p, tb);
  else
    read_kernel<D, false><<<grid, kThreads, 0, stream>>>(p, tb);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
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
