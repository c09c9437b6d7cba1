// Eviction from a paged cache: which tokens each key/value head keeps, by the sums of
// the attention weights that they got, and the move of the kept rows to the front,
// in place.
#include <cuda_runtime.h>

#include "paged.cuh"

namespace fa {
namespace evict {

__device__ DeviceError g_err;

using paged::record_bad_input;

enum Site { kSiteLength = 1, kSitePage, kSiteCount, kSiteList };

constexpr int kMaxCluster = 8;       // the largest portable one

FA_DEV uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
FA_DEV uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
FA_DEV uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Row (slot of a head) of a token; -1 where its page is none.
FA_DEV long long row_of(const PagedSeqs& s, int b, int head, int tok) {
  const int page = s.block_table[(size_t)b * s.max_pages + (tok >> s.page_shift)];
  if (page < 0 || page >= s.num_pages) {
    record_bad_input(&g_err, kSitePage);
    return -1;
  }
  return ((long long)page * s.Hkv + head << s.page_shift) + (tok & ((1 << s.page_shift) - 1));
}

// ------------------------------------------------------------------ select --
// The k-th largest of a head's sums by their bits, 11, 11 and 10 at a time: a
// histogram of the candidates, and from its top down the bin in which the k-th
// lies.  A cluster takes a (sequence, head), each of its blocks a stretch of the
// tokens, which stay in shared memory, and every block adds up the histograms of all
// (reading the others' shared memory), so that all know the bin with one barrier a
// round and nothing goes through global memory.  Then each block counts what
// it keeps, and writes it in order.
//
// It reads four bytes a key, little: what takes the time is the chain of loads and
// barriers.

constexpr int kThreads = 512;
constexpr int kBins = 2048;
FA_DEV int bits_of(int round) { return round == 2 ? 10 : 11; }
FA_DEV int shift_of(int round) { return round == 0 ? 21 : round == 1 ? 10 : 0; }
constexpr int kMostCached = 49152;         // tokens of a block in shared memory; the others are read again

// Floats in an order that unsigned integers have; a NaN is above all numbers.
FA_DEV uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);       // (-0 is 0)
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFEu;
  return u >> 31 ? ~u : u | 0x80000000u;
}
constexpr uint32_t kProtected = 0xFFFFFFFFu;

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* hist = smem;                              // [3][kBins]
  uint32_t* cached = smem + 3 * kBins;
  __shared__ uint32_t warp_sum[kThreads / 32];
  __shared__ uint32_t found[3];                       // bin, how many candidates lie above it
  __shared__ uint32_t counts[2];                      // this block's: above the threshold, equal to it
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int C = (int)cluster_size(), rank = (int)cluster_ctarank();
  const int unit = blockIdx.x / C, b = unit / p.s.Hkv, head = unit - b * p.s.Hkv;
  for (int i = tid; i < 3 * kBins; i += kThreads) hist[i] = 0u;
  overlap_launches();

  const int capacity = p.s.max_pages << p.s.page_shift;
  int L = p.s.seq_lens[b];
  if (L < 0 || L > capacity) {
    if (tid == 0) record_bad_input(&g_err, kSiteLength);
    L = 0;
  }
  const int kept = min(L, p.keep);
  int* out = p.index + (size_t)unit * p.keep;
  if (head == 0 && rank == 0 && tid == 0) p.kept[b] = kept;
  if (L <= p.keep) {                                  // all of them (the whole cluster comes here)
    for (int i = rank * kThreads + tid; i < p.keep; i += C * kThreads) out[i] = i < L ? i : -1;
    return;
  }

  const int each = ((L + C - 1) / C + 3) / 4 * 4;     // tokens of a block
  const int t0 = min(L, rank * each), n = min(L, t0 + each) - t0;
  // tokens go four at a time, which lie in one page (i a multiple of 4)
  auto load = [&](int i) -> uint4 {
    const int t = t0 + i;
    const long long row = row_of(p.s, b, head, t);
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row >= 0) x = *reinterpret_cast<const float4*>(p.sums + row);
    const int end = L - p.recent;
    return make_uint4(t < p.first || t >= end ? kProtected : ordered(x.x),
                      t + 1 < p.first || t + 1 >= end ? kProtected : ordered(x.y),
                      t + 2 < p.first || t + 2 >= end ? kProtected : ordered(x.z),
                      t + 3 < p.first || t + 3 >= end ? kProtected : ordered(x.w));
  };
  auto keys_at = [&](int i) -> uint4 {
    return i < p.cached ? *reinterpret_cast<const uint4*>(cached + i) : load(i);
  };
  __syncthreads();
#pragma unroll 4
  for (int i = 4 * tid; i < n; i += 4 * kThreads) {
    const uint4 x = load(i);
    if (i < p.cached) *reinterpret_cast<uint4*>(cached + i) = x;
    atomicAdd(&hist[x.x >> shift_of(0)], 1u);
    if (i + 1 < n) atomicAdd(&hist[x.y >> shift_of(0)], 1u);
    if (i + 2 < n) atomicAdd(&hist[x.z >> shift_of(0)], 1u);
    if (i + 3 < n) atomicAdd(&hist[x.w >> shift_of(0)], 1u);
  }

  uint32_t prefix = 0u, need = (uint32_t)p.keep;      // of the candidates, whose bits so far are `prefix`
  uint32_t above = 0u;                                // of this block, over the threshold
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    uint32_t* h = hist + round * kBins;
    if (round > 0) {
      const int shift = shift_of(round), bits = bits_of(round);
      for (int i = 4 * tid; i < n; i += 4 * kThreads) {
        const uint4 x = keys_at(i);
        const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + k < n && key[k] >> shift >> bits == prefix) atomicAdd(&h[key[k] >> shift & ((1u << bits) - 1u)], 1u);
      }
    }
    cluster_sync();
    // thread t adds up bins 4 t ... 4 t + 3 of all blocks; bins run from the top down
    const int bin0 = kBins - 4 - 4 * tid;
    uint4 sum = make_uint4(0u, 0u, 0u, 0u);
    for (int r = 0; r < C; ++r) {
      const uint4 x = ld_cluster_v4(mapa_shared(smem_u32(h + bin0), r));
      sum.x += x.x;
      sum.y += x.y;
      sum.z += x.z;
      sum.w += x.w;
    }
    const uint32_t own = sum.x + sum.y + sum.z + sum.w;
    uint32_t incl = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - own;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    if (before < need && before + own >= need) {      // one thread
      const uint32_t v[4] = {sum.w, sum.z, sum.y, sum.x};
      int k = 0;
      while (before + v[k] < need) before += v[k++];
      found[0] = (uint32_t)(bin0 + 3 - k);
      found[1] = before;
    }
    __syncthreads();
    const uint32_t bin = found[0];
    need -= found[1];
    // this block's own candidates above the bin
    uint32_t mine = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) mine += bin0 + k > (int)bin ? h[bin0 + k] : 0u;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) warp_sum[warp] = mine;             // (read above ahead of the barrier)
    prefix = round == 0 ? bin : prefix << bits_of(round) | bin;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) above += warp_sum[w];
    __syncthreads();
  }

  // Kept: the tokens above the threshold, and the first `need` of those at it.
  const uint32_t threshold = prefix;
  if (tid == 0) {
    counts[0] = above;
    counts[1] = hist[2 * kBins + (threshold & (kBins / 2 - 1))];
  }
  cluster_sync();
  uint32_t over = 0u, equal = 0u;                     // in the blocks before this one, and on the way
  for (int r = 0; r < rank; ++r) {
    over += ld_cluster_u32(mapa_shared(smem_u32(&counts[0]), r));
    equal += ld_cluster_u32(mapa_shared(smem_u32(&counts[1]), r));
  }
  for (int i0 = 0; i0 < n; i0 += 4 * kThreads) {
    const int i = i0 + 4 * tid;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (i < n) x = keys_at(i);
    const uint32_t key[4] = {x.x, x.y, x.z, x.w};
    uint32_t own = 0u;                                // above: low half, equal: high half
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) own += key[k] > threshold ? 1u : key[k] == threshold ? 0x10000u : 0u;
    uint32_t incl = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - own, all = 0u;
    for (int w = 0; w < kThreads / 32; ++w) {
      const uint32_t x = warp_sum[w];
      before += w < warp ? x : 0u;
      all += x;
    }
    uint32_t a = over + (before & 0xFFFFu), e = equal + (before >> 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k >= n || key[k] < threshold) continue;
      const uint32_t at = a + min(e, need);
      const bool more = key[k] > threshold;
      // (below `keep`, unless the sums change meanwhile)
      if ((more || e < need) && at < (uint32_t)p.keep) out[at] = t0 + i + k;
      a += more;
      e += !more;
    }
    over += all & 0xFFFFu;
    equal += all >> 16;
    __syncthreads();
  }
  cluster_sync();                                     // the others may still read this block's counts
}

// -------------------------------------------------------------------- keep --
// Rows i of a list move from slot index[i] to slot start + i, index ascending, so
// index[i] >= start + i: with the rows taken in order, a row's new slot is behind
// all that are still to be read, and the move can be in place.  A tile of rows is
// read into registers, a barrier shows that it has been read by all, and while it
// is written the next is on its way: what that reads lies behind all of this tile's
// new slots.  Where there are fewer lists than would fill the SMs a cluster takes a
// list, its blocks the parts of a tile.  Keys and values go apart.

constexpr int kMoveThreads = 256;
constexpr int kUnroll = 4;

template <int D, bool kFp8>
__global__ void __launch_bounds__(kMoveThreads, 4) keep_kernel(const KeepParams p) {
  constexpr int kLanes = D * (kFp8 ? 1 : 2) / 16;                    // of a row
  constexpr int kGroups = kMoveThreads / kLanes;
  constexpr int kRows = kUnroll * kGroups;                           // of a block's part of a tile
  constexpr int kEach = (kRows + kMoveThreads - 1) / kMoveThreads;   // rows whose numbers a thread looks up
  struct Move {
    long long from, to;      // rows; from < 0: none
  };
  __shared__ Move moves[3][kRows];      // of a tile that is written, one that is read, one that is looked up
  __shared__ int bad;
  const int tid = threadIdx.x;
  const int C = (int)cluster_size(), rank = (int)cluster_ctarank();
  const int unit = blockIdx.x / C, list = unit / 2, which = unit % 2;
  const int b = list / p.s.Hkv, head = list - b * p.s.Hkv;
  if (tid == 0) bad = 0;
  overlap_launches();
  const int capacity = p.s.max_pages << p.s.page_shift;
  const int count = p.counts[b], start = p.start ? p.start[b] : 0;
  if (count < 0 || count > p.most || start < 0) {                    // (the whole cluster)
    if (tid == 0) record_bad_input(&g_err, kSiteCount);
    return;
  }
  const int* index = p.index + ((size_t)b * p.heads + (p.heads == 1 ? 0 : head)) * p.most;

  // ascending, from `start` on, and within the table; each block looks at a share
  bool ok = true;
#pragma unroll 4
  for (int i = rank * kMoveThreads + tid; i < count; i += C * kMoveThreads) {
    const int x = index[i];
    ok = ok && x >= start && x < capacity && (i == 0 || index[i - 1] < x);
  }
  ok = __syncthreads_and(ok);
  if (C > 1) {
    cluster_sync();                                                  // every `bad` is 0
    if (!ok && tid < C) st_cluster_u32(mapa_shared(smem_u32(&bad), tid), 1u);
    cluster_sync();
    ok = *reinterpret_cast<volatile int*>(&bad) == 0;
  }
  if (!ok) {
    if (tid == 0) record_bad_input(&g_err, kSiteList);
    return;
  }

  const int lane = tid % kLanes, group = tid / kLanes;
  uint4* pages = static_cast<uint4*>(which ? p.v_pages : p.k_pages);
  uint8_t* scales = which ? p.v_scale : p.k_scale;
  float* sums = which ? nullptr : p.sums;
  const int tile = C * kRows, tiles = (count + tile - 1) / tile;
  auto look_up = [&](int t) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int r = e * kMoveThreads + tid;
      if (r >= kRows) break;
      const long long i = (long long)t * tile + rank * kRows + r;
      Move m{-1, -1};
      if (i < count) {
        const int from = index[i], to = start + (int)i;
        if (from != to) {
          m.from = row_of(p.s, b, head, from);
          m.to = row_of(p.s, b, head, to);
          if (m.to < 0) m.from = -1;
        }
      }
      moves[t % 3][r] = m;
    }
  };
  uint4 x[kUnroll];
  uint8_t scale[kEach];
  float sum[kEach];
  auto read = [&](int t, uint4 (&y)[kUnroll], uint8_t (&sc)[kEach], float (&su)[kEach]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long from = moves[t % 3][u * kGroups + group].from;
      if (from >= 0) y[u] = pages[from * kLanes + lane];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int r = e * kMoveThreads + tid;
      if (r >= kRows) break;
      const long long from = moves[t % 3][r].from;
      if (from < 0) continue;
      if (kFp8) sc[e] = scales[from];
      if (sums) su[e] = sums[from];
    }
  };
  if (tiles == 0) return;
  look_up(0);
  __syncthreads();
  read(0, x, scale, sum);
#pragma unroll 1
  for (int t = 0; t < tiles; ++t) {
    uint4 next[kUnroll];
    uint8_t next_scale[kEach];
    float next_sum[kEach];
    if (t + 1 < tiles) look_up(t + 1);
    if (C > 1)
      cluster_sync();
    else
      __syncthreads();
    if (t + 1 < tiles) read(t + 1, next, next_scale, next_sum);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const Move m = moves[t % 3][u * kGroups + group];
      if (m.from >= 0) pages[m.to * kLanes + lane] = x[u];
      x[u] = next[u];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int r = e * kMoveThreads + tid;
      if (r >= kRows) break;
      const Move m = moves[t % 3][r];
      if (m.from >= 0) {
        if (kFp8) scales[m.to] = scale[e];
        if (sums) sums[m.to] = sum[e];
      }
      scale[e] = next_scale[e];
      sum[e] = next_sum[e];
    }
  }
}

// Launches `units` clusters of C blocks; see launch_overlapped().
template <class P>
fa_status launch_clusters(void (*kernel)(P), int units, int C, int threads, int smem, cudaStream_t stream,
                          const P& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(units * C);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool kFp8>
fa_status launch_keep(const KeepParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kRows = kUnroll * kMoveThreads / (D * (kFp8 ? 1 : 2) / 16);
  const long long units = 2ll * p.s.B * p.s.Hkv;
  int C = 1;
  while (C < kMaxCluster && units * C * 2 <= 3ll * num_sms && (long long)kRows * C < p.most) C *= 2;
  return launch_clusters(keep_kernel<D, kFp8>, (int)units, C, kMoveThreads, 0, stream, p);
}

}  // namespace evict

fa_status launch_cache_select(const SelectParams& in, int num_sms, cudaStream_t stream) {
  SelectParams p = in;
  const int capacity = p.s.max_pages << p.s.page_shift;
  const long long units = (long long)p.s.B * p.s.Hkv;
  int C = 1;
  while (C < evict::kMaxCluster && units * C * 2 <= 4ll * num_sms && 1024 * C < capacity) C *= 2;
  const int each = ((capacity + C - 1) / C + 3) / 4 * 4;
  p.cached = each < evict::kMostCached ? each : evict::kMostCached;
  const int most = (3 * evict::kBins + evict::kMostCached) * 4;
  const fa_status st = prepare_kernel(reinterpret_cast<const void*>(evict::select_kernel), most);
  if (st != FA_OK) return st;
  return evict::launch_clusters(evict::select_kernel, (int)units, C, evict::kThreads,
                                (3 * evict::kBins + p.cached) * 4, stream, p);
}

fa_status launch_cache_keep(const KeepParams& p, int num_sms, cudaStream_t stream) {
  if (p.D == 128)
    return p.k_scale ? evict::launch_keep<128, true>(p, num_sms, stream)
                     : evict::launch_keep<128, false>(p, num_sms, stream);
  return p.k_scale ? evict::launch_keep<64, true>(p, num_sms, stream) : evict::launch_keep<64, false>(p, num_sms, stream);
}

fa_status evict_take_device_error() {
  DeviceError e{0, 0};
  if (cudaMemcpyFromSymbol(&e, evict::g_err, sizeof(e)) != cudaSuccess) return FA_ERR_CUDA;
  if (e.status != 0) {
    const DeviceError z{0, 0};
    if (cudaMemcpyToSymbol(evict::g_err, &z, sizeof(z)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return static_cast<fa_status>(e.status);
}

}  // namespace fa
