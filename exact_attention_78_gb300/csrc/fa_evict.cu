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
constexpr int kMaxSelect = 16;       // blocks of a selection's cluster

FA_DEV uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
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
// lies.  A thread block takes a (sequence, head), whose tokens stay in shared memory;
// where there are fewer of those than SMs, a cluster does, each of its blocks a stretch
// of the tokens, and its blocks add up their histograms by reading one another's shared
// memory.  They share the bins out: reading all of every histogram, 8 KB, in each block
// took 20,000 cycles a round with 16 blocks.  Then each block counts what it keeps, and
// writes it in order.
//
// It reads four bytes a key, little: what takes the time is the chain of loads and
// barriers, and the instructions for each token of the few SMs that take part.

constexpr int kBins = 2048;
constexpr int kGroups = kBins / 32;        // of bins that a warp adds up
static_assert(kGroups == 64, "two groups a lane");
FA_DEV int bits_of(int round) { return round == 2 ? 10 : 11; }
FA_DEV int shift_of(int round) { return round == 0 ? 21 : round == 1 ? 10 : 0; }
constexpr int kShort = 2048;               // tokens of a table whose heads take the smallest blocks
constexpr int kMostCached = 49152;         // tokens of a block in shared memory; the others are read again

// Floats in an order that unsigned integers have; a NaN is above all numbers.  Nothing
// comes out below 0x007FFFFF, which is -inf.
FA_DEV uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);       // (-0 is 0)
  const uint32_t key = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
  return (u & 0x7FFFFFFFu) > 0x7F800000u ? 0xFFFFFFFEu : key;
}
constexpr uint32_t kProtected = 0xFFFFFFFFu, kNoToken = 0u;

// Inclusive sums over the lanes.
FA_DEV uint32_t scan(uint32_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* hist = smem;                              // [3][kBins]
  uint32_t* cached = smem + 3 * kBins;
  __shared__ uint32_t total[kBins], group_total[kGroups];      // of this block's share of the bins, over all blocks
  __shared__ uint32_t warp_over[kWarps], warp_equal[kWarps];   // above the threshold, equal to it
  __shared__ uint32_t found[2];                       // bin, how many candidates lie above it
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
  int* out = p.index + (size_t)unit * p.keep;
  if (head == 0 && rank == 0 && tid == 0) p.kept[b] = min(L, p.keep);
  if (L <= p.keep) {                                  // all of them (the whole cluster comes here)
    for (int i = rank * kThreads + tid; i < p.keep; i += C * kThreads) out[i] = i < L ? i : -1;
    return;
  }

  const int each = ((L + C - 1) / C + 3) / 4 * 4;     // tokens of a block
  const int t0 = min(L, rank * each), n = min(L, t0 + each) - t0;
  // A warp has a stretch of the block's tokens, 128 at a time, four a lane, which lie
  // in one page.
  const int stretch = (each + 128 * kWarps - 1) / (128 * kWarps) * 128;
  const int i0 = min(n, warp * stretch), i1 = min(n, i0 + stretch);
  const int last = L - p.recent;                      // the first protected one at the end
  auto load = [&](int i) -> uint4 {
    const int t = t0 + i;
    const long long row = row_of(p.s, b, head, t);
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row >= 0) x = *reinterpret_cast<const float4*>(p.sums + row);
    uint4 y = make_uint4(ordered(x.x), ordered(x.y), ordered(x.z), ordered(x.w));
    if (t < p.first || t + 3 >= last || i + 3 >= n) {
      auto key = [&](int k, uint32_t v) {
        return i + k >= n ? kNoToken : t + k < p.first || t + k >= last ? kProtected : v;
      };
      y = make_uint4(key(0, y.x), key(1, y.y), key(2, y.z), key(3, y.w));
    }
    return y;
  };
  auto sync_all = [&]() {
    if (C > 1) cluster_sync(); else __syncthreads();
  };
  auto keys_at = [&](int i) -> uint4 {
    return i < p.cached ? *reinterpret_cast<const uint4*>(cached + i) : load(i);
  };
  __syncthreads();
#pragma unroll 1
  for (int j = i0; j < i1; j += 512) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = j + 128 * u + 4 * lane;
      x[u] = make_uint4(kNoToken, kNoToken, kNoToken, kNoToken);
      if (i < i1) x[u] = load(i);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = j + 128 * u + 4 * lane;
      if (j + 128 * u >= i1) break;                   // (the whole warp)
      if (i < i1 && i < p.cached) *reinterpret_cast<uint4*>(cached + i) = x[u];
      const uint32_t bin[4] = {x[u].x >> shift_of(0), x[u].y >> shift_of(0), x[u].z >> shift_of(0), x[u].w >> shift_of(0)};
      // tokens that are all alike (protected ones, zeros) would be counted one by one
      const uint32_t lead = __shfl_sync(0xffffffffu, bin[0], 0);
      if (__all_sync(0xffffffffu, bin[0] == lead && bin[1] == lead && bin[2] == lead && bin[3] == lead)) {
        if (lane == 0) atomicAdd(&hist[lead], 128u);
      } else {      // (what is no token goes to bin 0, where no token is)
#pragma unroll
        for (int k = 0; k < 4; ++k) atomicAdd(&hist[bin[k]], 1u);
      }
    }
  }
  uint32_t prefix = 0u, need = (uint32_t)p.keep;      // of the candidates, whose bits so far are `prefix`
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    uint32_t* h = hist + round * kBins;
    if (round > 0) {
      const int shift = shift_of(round), bits = bits_of(round);
      const uint32_t low = (1u << bits) - 1u;
#pragma unroll 4
      for (int j = i0 + 4 * lane; j < i1; j += 128) {
        const uint4 x = keys_at(j);
        const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (key[k] >> shift >> bits == prefix) atomicAdd(&h[key[k] >> shift & low], 1u);
      }
    }
    sync_all();
    // this block's share: bins [rank * share, + share), 32 a warp
    const int share = kBins / C, per = kGroups / C, shift_per = __ffs(per) - 1;      // (powers of two)
    for (int g = warp; g < per; g += kWarps) {
      uint32_t sum = 0u;
      if (C == 1) {
        sum = h[g * 32 + lane];
      } else {
        const uint32_t from = smem_u32(h + rank * share + g * 32 + lane);
        uint32_t x[kMaxSelect];
#pragma unroll
        for (int r = 0; r < kMaxSelect; ++r) x[r] = r < C ? ld_cluster_u32(mapa_shared(from, r)) : 0u;
#pragma unroll
        for (int r = 0; r < kMaxSelect; ++r) sum += x[r];
      }
      if (C > 1) total[g * 32 + lane] = sum;
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == 0) group_total[g] = sum;
    }
    sync_all();
    if (warp == 0) {
      // the group, then the bin in it, from the top down
      auto group_of = [&](int g) {
        return C == 1 ? group_total[g] : ld_cluster_u32(mapa_shared(smem_u32(group_total + (g & (per - 1))), g >> shift_per));
      };
      const uint32_t v0 = group_of(63 - 2 * lane), v1 = group_of(62 - 2 * lane);
      uint32_t above = scan(v0 + v1, lane) - v0 - v1;
      uint32_t mine = __ballot_sync(0xffffffffu, above < need && above + v0 + v1 >= need);
      int at = mine ? __ffs(mine) - 1 : 0;
      const bool second = above + v0 < need;
      const int group = __shfl_sync(0xffffffffu, second ? 62 - 2 * lane : 63 - 2 * lane, at);
      const uint32_t base = __shfl_sync(0xffffffffu, second ? above + v0 : above, at);
      const uint32_t v =
          C == 1 ? h[group * 32 + 31 - lane]
                 : ld_cluster_u32(mapa_shared(smem_u32(total + (group & (per - 1)) * 32 + 31 - lane), group >> shift_per));
      above = base + scan(v, lane) - v;
      mine = __ballot_sync(0xffffffffu, above < need && above + v >= need);
      at = mine ? __ffs(mine) - 1 : 0;
      if (lane == at) {
        found[0] = (uint32_t)(group * 32 + 31 - lane);
        found[1] = above;
      }
    }
    __syncthreads();
    need -= found[1];
    prefix = round == 0 ? found[0] : prefix << bits_of(round) | found[0];
  }

  // Kept: the tokens above the threshold, and the first `need` of those at it.
  const uint32_t threshold = prefix;
  uint32_t over = 0u, equal = 0u;                     // in the blocks and warps before, and on the way
#pragma unroll 2
  for (int i = i0 + 4 * lane; i < i1; i += 128) {
    const uint4 x = keys_at(i);
    over += (x.x > threshold) + (x.y > threshold) + (x.z > threshold) + (x.w > threshold);
    equal += (x.x == threshold) + (x.y == threshold) + (x.z == threshold) + (x.w == threshold);
  }
  over = __reduce_add_sync(0xffffffffu, over);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    warp_over[warp] = over;
    warp_equal[warp] = equal;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t o = lane < kWarps ? warp_over[lane] : 0u, e = lane < kWarps ? warp_equal[lane] : 0u;
    const uint32_t so = scan(o, lane), se = scan(e, lane);
    if (lane < kWarps) {
      warp_over[lane] = so - o;
      warp_equal[lane] = se - e;
    }
    if (lane == 31) {
      counts[0] = so;
      counts[1] = se;
    }
  }
  sync_all();
  over = warp_over[warp];
  equal = warp_equal[warp];
  for (int r = 0; r < rank; ++r) {
    over += ld_cluster_u32(mapa_shared(smem_u32(&counts[0]), r));
    equal += ld_cluster_u32(mapa_shared(smem_u32(&counts[1]), r));
  }
  const uint32_t below = (1u << lane) - 1u;
  // (places are below `keep`, unless the sums change meanwhile)
#pragma unroll 2
  for (int j = i0; j < i1; j += 128) {
    const int i = j + 4 * lane;
    uint4 x = make_uint4(kNoToken, kNoToken, kNoToken, kNoToken);
    if (i < i1) x = keys_at(i);
    const uint32_t key[4] = {x.x, x.y, x.z, x.w};
    uint32_t a = over;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t more = __ballot_sync(0xffffffffu, key[k] > threshold);
      a += __popc(more & below);
      over += __popc(more);
    }
    if (!__any_sync(0xffffffffu, key[0] == threshold || key[1] == threshold || key[2] == threshold || key[3] == threshold)) {
      uint32_t to = a + min(equal, need);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (key[k] <= threshold) continue;
        if (to < (uint32_t)p.keep) out[to] = t0 + i + k;
        ++to;
      }
      continue;
    }
    uint32_t e = equal;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t same = __ballot_sync(0xffffffffu, key[k] == threshold);
      e += __popc(same & below);
      equal += __popc(same);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool up = key[k] > threshold, at = key[k] == threshold;
      const uint32_t to = a + min(e, need);
      if ((up || (at && e < need)) && to < (uint32_t)p.keep) out[to] = t0 + i + k;
      a += up;
      e += at;
    }
  }
  sync_all();                                         // the others may still read this block's counts
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
  // Where a tile's rows lie, step by step, each with the loads of the step before
  // behind it: the tokens, their old and new pages, the rows.
  struct Tokens {
    int from, to;            // the same: stays, or none
  };
  struct Pages {
    int from, to;
  };
  auto tokens = [&](int t, Tokens (&x)[kEach]) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int r = e * kMoveThreads + tid;
      const long long i = (long long)t * tile + rank * kRows + r;
      x[e].from = x[e].to = -1;
      if (r < kRows && i < count) {
        x[e].to = start + (int)i;
        x[e].from = index[i];
      }
    }
  };
  const int* table = p.s.block_table + (size_t)b * p.s.max_pages;
  auto pages_of = [&](const Tokens (&x)[kEach], Pages (&y)[kEach]) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (x[e].from == x[e].to) continue;
      y[e].from = table[x[e].from >> p.s.page_shift];
      y[e].to = table[x[e].to >> p.s.page_shift];
    }
  };
  auto row = [&](int page, int tok) -> long long {
    return ((long long)page * p.s.Hkv + head << p.s.page_shift) + (tok & ((1 << p.s.page_shift) - 1));
  };
  auto place = [&](int t, const Tokens (&x)[kEach], const Pages (&y)[kEach]) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int r = e * kMoveThreads + tid;
      if (r >= kRows) break;
      Move m{-1, -1};
      if (x[e].from != x[e].to) {
        if ((unsigned)y[e].from < (unsigned)p.s.num_pages && (unsigned)y[e].to < (unsigned)p.s.num_pages)
          m = Move{row(y[e].from, x[e].from), row(y[e].to, x[e].to)};
        else
          record_bad_input(&g_err, kSitePage);
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
  Tokens one[kEach], two[kEach];     // of the tiles one and two further on than the one that is read
  Pages pages_one[kEach];
  tokens(0, one);
  tokens(1, two);
  pages_of(one, pages_one);
  place(0, one, pages_one);
  pages_of(two, pages_one);
#pragma unroll
  for (int e = 0; e < kEach; ++e) one[e] = two[e];
  tokens(2, two);
  __syncthreads();
  read(0, x, scale, sum);
#pragma unroll 1
  for (int t = 0; t < tiles; ++t) {
    uint4 next[kUnroll];
    uint8_t next_scale[kEach];
    float next_sum[kEach];
    if (t + 1 < tiles) {
      place(t + 1, one, pages_one);
      pages_of(two, pages_one);
#pragma unroll
      for (int e = 0; e < kEach; ++e) one[e] = two[e];
      tokens(t + 3, two);
    }
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

// How many clusters of C blocks the device holds at once.
bool clusters_at_once(const void* kernel, int C, int threads, int smem, int* most) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(most, kernel, &cfg) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
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

namespace evict {

template <int kThreads>
fa_status launch_select(const SelectParams& in, int C, cudaStream_t stream) {
  SelectParams p = in;
  const int capacity = p.s.max_pages << p.s.page_shift;
  const long long units = (long long)p.s.B * p.s.Hkv;
  auto kernel = select_kernel<kThreads>;
  const void* func = reinterpret_cast<const void*>(kernel);
  const fa_status st = prepare_kernel(func, (3 * kBins + kMostCached) * 4);
  if (st != FA_OK) return st;
  // clusters of more than 8 blocks have to be asked for (on each device), and whether
  // they are to be had depends on the chip's parts
  if (C > kMaxCluster && cudaFuncSetAttribute(func, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
    cudaGetLastError();
    C = kMaxCluster;
  }
  for (;; C /= 2) {
    const int each = ((capacity + C - 1) / C + 3) / 4 * 4;
    p.cached = each < kMostCached ? each : kMostCached;
    const int smem = (3 * kBins + p.cached) * 4;
    int most = 1;
    if (C > kMaxCluster && clusters_at_once(func, C, kThreads, smem, &most) && most == 0) continue;
    return launch_clusters(kernel, (int)units, C, kThreads, smem, stream, p);
  }
}

}  // namespace evict

// A block of its own for each head where those fill the SMs, else a cluster, but no more
// blocks than have some thousand tokens each.  (24 x 8 heads, up to 12,000 tokens: 17 us,
// with two blocks 5 more; 4 heads of 200,001: 16 blocks 18 us, 8 blocks 26.)
// More heads than two blocks an SM take smaller ones, of which an SM holds more: 800
// heads of 1253 tokens each 39 / 18 / 16.5 us with 1024 / 512 / 256 threads, 512 of 4000
// 30 / 18.3 / 14.6; 160 of 4000 15 / 12.3 / 12.8, 192 of 12,000 22 / 16.6 / 19.6 (of random
// lengths up to 12,000: 17 with 1024).
//   The lengths are on the device, so all of this, and a block's shared memory, goes by the
// table's width.  Under a table for 65,536 tokens instead of one as wide as the longest
// sequence: 24 x 8 heads up to 12,000 tokens 17 us as before, 100 x 8 heads up to 1253
// 13.8 -> 30, 8 heads of one sequence of 12,000 10.8 -> 26.
fa_status launch_cache_select(const SelectParams& p, int num_sms, cudaStream_t stream) {
  const int capacity = p.s.max_pages << p.s.page_shift;
  const long long units = (long long)p.s.B * p.s.Hkv;
  int C = 1;
  while (C < evict::kMaxSelect && units * C * 2 <= num_sms && 4096 * C < capacity) C *= 2;
  if (units <= 2ll * num_sms) return evict::launch_select<1024>(p, C, stream);
  return capacity <= evict::kShort ? evict::launch_select<256>(p, 1, stream) : evict::launch_select<512>(p, 1, stream);
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
