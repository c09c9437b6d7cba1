// Sums of the attention weights that the keys of a paged cache get, one for each key
// and key/value head:
//
//   sums[t] = decay sums[t] + sum over the rows r that see key t of exp(scale q_r k_t - lse_r),
//
// a row being a new token and a query head of the group.  A key's sum is one thread's
// (or four lanes'), which adds its rows up in a fixed order: nothing is added
// atomically, and results repeat bit by bit.
#include <cuda_runtime.h>

#include "paged.cuh"
#include "softmax_math.cuh"

namespace fa {
namespace weigh {

__device__ DeviceError g_err;

constexpr float kLog2e = 1.4426950408889634f;

enum Site { kSiteSeqs = 1, kSitePage, kSiteKEmpty, kSiteKFull, kSiteQEmpty, kSiteQFull, kSiteSEmpty, kSiteSFull,
            kSiteLseEmpty, kSiteLseFull };

FA_DEV size_t lse_at(const WeighParams& p, int b, int q0, int head, int tok) {
  return p.s.cu ? (size_t)head * p.s.Sn + q0 + tok : ((size_t)b * p.Hq + head) * p.s.Sn + tok;
}
// A row that saw no key has an LSE of -inf, and gives no key a weight.
FA_DEV float lse_of(float x) { return x == -INFINITY ? INFINITY : x; }

// The slot of the key's sum; -1 in a bad page.
FA_DEV long long slot_of(const WeighParams& p, int b, int head, int key) {
  const int page = p.s.block_table[(size_t)b * p.s.max_pages + (key >> p.s.page_shift)];
  if (page < 0 || page >= p.s.num_pages) {
    paged::record_bad_input(&g_err, kSitePage);
    return -1;
  }
  return ((long long)page * p.s.Hkv + head << p.s.page_shift) + (key & ((1 << p.s.page_shift) - 1));
}

// ---------------------------------------------------------------- few rows --
// A step of single tokens reads every key once and computes little with it, so HBM
// bounds it.  The keys are the M side of mma.sync products, 16 a tile, the rows the N
// side, 8 a tile.  A product's sum may take its elements in any order, so each
// lane's share of a key is whole pieces of 16 bytes, which the lane itself copies from
// global memory ahead of their use, into its own places of a ring in shared memory:
// a warp is on its own, with no barrier but its own lanes', and some 150 KB an SM are
// under way.  All tiles of all (sequence, head) units form one line, of which every
// warp takes an equal stretch.  (STEP_FIGURES)
//
// E4M3 codes become FP16, and the queries too, by a power of two of each row's own
// (as in the decode kernel of the attention); keys' scales go to the scores in FP32.

constexpr int kStepThreads = 512;
constexpr int kStepWarps = kStepThreads / 32;
constexpr int kStepKeys = 16;
constexpr int kStepRows = 32;        // most rows of a sequence and key/value head here

FA_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
FA_DEV void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two E4M3 codes (the lower half of w) as FP16, exactly.
FA_DEV uint32_t e4m3_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}
FA_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 bytes from global to shared memory, past the L1 cache.
FA_DEV void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(reinterpret_cast<uint64_t>(from)) : "memory");
}
FA_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
FA_DEV void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, bool kFp8>
struct StepLayout {
  static constexpr int kPieces = D * (kFp8 ? 1 : 2) / 64;     // of 16 bytes of a key that a lane has
  static constexpr int kTile = kStepKeys * kPieces * 64;
  // behind a stage's keys: their scales, their sums so far, their row
  static constexpr int kScales = kTile, kOld = kTile + 16, kRow = kTile + 80;
  static constexpr int kStage = kTile + 128;
  static constexpr int kRing = 212992;
  static constexpr int kFit = kRing / (kStepWarps * kStage);
  static constexpr int kDepth = kFit < 8 ? kFit : 8;
  static constexpr int kBytes = kStepWarps * kDepth * kStage;
};

// A walk over a warp's stretch of the line, tile by tile.
struct Walk {
  paged::SeqRows q;
  int b, head, k, tiles;      // tile k of `tiles` of a unit
  long long left;             // tiles from here on
  // To the next tile; whether it is another unit's.
  FA_DEV bool next(const WeighParams& p) {
    --left;
    if (++k < tiles || left == 0) return false;
    k = 0;
    if (++head == p.s.Hkv) {
      head = 0;
      do {
        ++b;                  // (one with tiles follows)
        q = paged::rows_of(p.s, b);
        tiles = q.n > 0 ? (q.L + kStepKeys - 1) / kStepKeys : 0;
      } while (tiles == 0);
    }
    return true;
  }
};

template <int D, bool kFp8, int kTiles>
__global__ void __launch_bounds__(kStepThreads, 1) step_kernel(const WeighParams p) {
  using Lay = StepLayout<D, kFp8>;
  constexpr int kPieces = Lay::kPieces;
  constexpr int kWords = kFp8 ? 2 * kPieces : kPieces;        // of 16 bytes of a row of Q
  extern __shared__ __align__(128) uint8_t ring_raw[];
  __shared__ long long pre[kMaxPackedSeqs + 1];
  __shared__ long long work_sums[2 * kStepWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int c = lane % 4, g = lane / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool ok = paged::prefix_sequences(
      p.s, p.max_q,
      [&](const paged::SeqRows& r) {
        return paged::Work{(long long)p.s.Hkv * ((r.L + kStepKeys - 1) / kStepKeys), 0, 0};
      },
      pre, nullptr, work_sums);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) paged::record_bad_input(&g_err, kSiteSeqs);
    return;
  }
  const long long total = pre[p.s.B];
  const int warps = gridDim.x * kStepWarps, id = warp * gridDim.x + blockIdx.x;
  const long long t0 = paged::div64(total * id, warps);
  Walk at;
  at.left = paged::div64(total * (id + 1), warps) - t0;
  if (at.left == 0) return;
  {
    int lo = 0, hi = p.s.B - 1;      // last b with pre[b] <= t0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= t0) lo = mid; else hi = mid - 1;
    }
    at.b = lo;
    at.q = paged::rows_of(p.s, lo);
    at.tiles = (at.q.L + kStepKeys - 1) / kStepKeys;
    at.head = (int)paged::div64(t0 - pre[lo], at.tiles);
    at.k = (int)(t0 - pre[lo] - (long long)at.head * at.tiles);
  }

  uint8_t* ring = ring_raw + warp * Lay::kDepth * Lay::kStage;
  Walk ahead = at;                                     // the tile that is copied next
  int held = -64, pages = -1;                          // its unit's pages [held, held + 32), one a lane
  auto copy = [&](int stage) {
    if (ahead.left > 0) {
      const int key0 = ahead.k * kStepKeys, page_at = key0 >> p.s.page_shift;
      if (page_at >= held + 32 || page_at < held) {
        held = page_at;
        pages = held + lane <= (ahead.q.L - 1) >> p.s.page_shift
                    ? p.s.block_table[(size_t)ahead.b * p.s.max_pages + held + lane]
                    : -1;
      }
      const int page = __shfl_sync(0xffffffffu, pages, page_at - held);
      uint8_t* to = ring + stage * Lay::kStage;
      long long row = -1;
      if (page < 0 || page >= p.s.num_pages) {
        paged::record_bad_input(&g_err, kSitePage);
      } else {
        row = ((long long)page * p.s.Hkv + ahead.head << p.s.page_shift) + (key0 & ((1 << p.s.page_shift) - 1));
        const uint32_t mine = smem_u32(to) + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4* src = static_cast<const uint4*>(p.k_pages) + (row + g + 8 * h) * (4 * kPieces) + c;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) copy16(mine + (h * kPieces + i) * 512, src + 4 * i);
        }
        if (lane < 4) copy16(smem_u32(to) + Lay::kOld + lane * 16, p.sums + row + 4 * lane);
        if (kFp8 && lane == 4) copy16(smem_u32(to) + Lay::kScales, p.k_scale + row);
      }
      if (lane == 0) *reinterpret_cast<long long*>(to + Lay::kRow) = row;
      if (ahead.next(p)) held = -64;
    }
    copy_commit();
  };
#pragma unroll 1
  for (int i = 0; i < Lay::kDepth; ++i) copy(i);

  const int least_exp = 14 + max(0, 127 - (int)(__float_as_uint(p.scale) >> 23));
  int stage = 0;
  bool fresh = true;                                   // a unit begins
  uint4 qf[kTiles][kWords];                            // row 8 n + g, as the keys' pieces lie
  float row_scale[kTiles][2], lse[kTiles][2];          // of rows 8 n + 2 c + e
  int lim[kTiles][2];                                  // keys that they see
#pragma unroll 1
  while (at.left > 0) {
    const int past = at.q.L - at.q.n;
    if (fresh) {
      const int rows = at.q.n * p.group;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const int r = 8 * n + g, tok = r / p.group;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(p.q) +
            ((size_t)(at.q.q0 + tok) * p.Hq + at.head * p.group + r - tok * p.group) * D);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          qf[n][i] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows) qf[n][i] = src[kFp8 ? 8 * (i / 2) + 2 * c + i % 2 : 4 * i + c];
        }
      }
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        float scale = p.scale;
        if (kFp8) {
          uint32_t top = 0u;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const uint32_t v[4] = {qf[n][i].x, qf[n][i].y, qf[n][i].z, qf[n][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(v[j] & 0x7FFFu, (v[j] >> 16) & 0x7FFFu));
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = max((int)(top >> 7), least_exp) - 127;
          const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
          scale *= __uint_as_float((uint32_t)(127 - 13 + e) << 23);
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            uint32_t v[4] = {qf[n][i].x, qf[n][i].y, qf[n][i].z, qf[n][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[j] = pack_f16x2(__uint_as_float(v[j] << 16) * up, __uint_as_float(v[j] & 0xFFFF0000u) * up);
            qf[n][i] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * n + 2 * c + e, tk = row / p.group;
          row_scale[n][e] = kFp8 ? __shfl_sync(0xffffffffu, scale, (2 * c + e) * 4) : scale;
          lim[n][e] = row >= rows ? 0 : p.causal ? past + tk + 1 : at.q.L;
          lse[n][e] =
              row >= rows ? 0.0f : lse_of(p.lse[lse_at(p, at.b, at.q.q0, at.head * p.group + row - tk * p.group, tk)]);
        }
      }
    }
    copy_wait<Lay::kDepth - 1>();
    __syncwarp();                                      // the other lanes' copies are here too
    const uint8_t* from = ring + stage * Lay::kStage;
    const int key0 = at.k * kStepKeys;
    float fac[2] = {1.0f, 1.0f};
    if (kFp8) {
      fac[0] = paged::scale_value(from[Lay::kScales + g]);
      fac[1] = paged::scale_value(from[Lay::kScales + g + 8]);
    }
    float s[kTiles][4];                                // [2 h + e]: key g + 8 h, row 8 n + 2 c + e
#pragma unroll
    for (int n = 0; n < kTiles; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(from + i * 512 + lane * 16);
      const uint4 y = *reinterpret_cast<const uint4*>(from + (kPieces + i) * 512 + lane * 16);
      if (!kFp8) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          mma16816(s[n], x.x, y.x, x.y, y.y, qf[n][i].x, qf[n][i].y);
          mma16816(s[n], x.z, y.z, x.w, y.w, qf[n][i].z, qf[n][i].w);
        }
      } else {
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = e4m3_f16x2(xs[j]), a1 = e4m3_f16x2(ys[j]);
          const uint32_t a2 = e4m3_f16x2(xs[j] >> 16), a3 = e4m3_f16x2(ys[j] >> 16);
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            const uint4 qw = qf[n][kFp8 ? 2 * i + j / 2 : 0];
            mma16816_f16(s[n], a0, a1, a2, a3, j % 2 ? qw.z : qw.x, j % 2 ? qw.w : qw.y);
          }
        }
      }
    }
    float w[2] = {0.0f, 0.0f};                         // of keys g, g + 8
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // taken from the LSE before it goes to log2 units: the difference is small
        // where the weight is large, and so is its rounding
        float x = kFp8 ? s[n][e] * fac[e >> 1] : s[n][e];
        x = fmaf(x, row_scale[n][e & 1], -lse[n][e & 1]) * kLog2e;
        w[e >> 1] += key0 + g + 8 * (e >> 1) < lim[n][e & 1] ? ex2_mufu(x) : 0.0f;
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] += __shfl_xor_sync(0xffffffffu, w[h], 1);
      w[h] += __shfl_xor_sync(0xffffffffu, w[h], 2);
    }
    const long long row = *reinterpret_cast<const long long*>(from + Lay::kRow);
    const int in = g + 8 * c;                          // lanes with c < 2 write a key's sum
    if (c < 2 && key0 + in < at.q.L && row >= 0) {
      const float old = *reinterpret_cast<const float*>(from + Lay::kOld + 4 * in);
      p.sums[row + in] = (p.decay != 0.0f && key0 + in < past ? p.decay * old : 0.0f) + (c ? w[1] : w[0]);
    }
    __syncwarp();                                      // every lane is done with the stage
    copy(stage);
    stage = stage + 1 == Lay::kDepth ? 0 : stage + 1;
    fresh = at.next(p);
  }
}

template <int D, bool kFp8>
fa_status launch_step(const WeighParams& p, int num_sms, cudaStream_t stream) {
  const long long rows = (long long)p.max_q * p.group;
  auto kernel = rows <= 8 ? step_kernel<D, kFp8, 1> : rows <= 16 ? step_kernel<D, kFp8, 2> : step_kernel<D, kFp8, 4>;
  constexpr int kBytes = StepLayout<D, kFp8>::kBytes;
  const fa_status st = prepare_kernel(reinterpret_cast<const void*>(kernel), kBytes);
  if (st != FA_OK) return st;
  return launch_overlapped(kernel, dim3(num_sms), kStepThreads, kBytes, stream, p);
}

// --------------------------------------------------------------- many rows --
// S^T = K Q^T on tcgen05: 256 keys of a unit (two tiles of 128, the M side, one key a
// lane of tensor memory), the rows 128 at a time (N).  A thread has a key, reads its
// scores out of tensor memory and adds their exponentials up: no row statistics, no
// second product, nothing between the threads.  Both operands' tiles are read by all
// units of a head (Q) or tiles of rows (K), from L2.  What bounds it is the
// exponential, 16 a clock and SM.
//
// Warps: 0-3 and 4-7 exponentials of the first and second 128 keys, 8 loads (Q; K of
// BF16 pages), 9 MMA issue, 10 the rows' LSE, 11-14 widening (E4M3 pages: codes and
// scale to BF16, exactly, once per unit).
//
// Tensor memory: scores of the first keys at columns 0 and 128, of the second at 256
// and 384.

constexpr int kBM = 128, kBN = 128;
constexpr int kUnitKeys = 2 * kBM;
constexpr int kLses = 4;

template <int D, bool kFp8>
struct Layout {
  static constexpr int kThreads = kFp8 ? 480 : 352;
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = 128 * 128;             // 128 rows by 64 columns
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kQStages = D == 128 ? 2 : 4;
  static constexpr int kK = 0;                              // [2][two tiles]
  static constexpr int kQ = kK + 4 * kTileBytes;
  static constexpr int kLse = kQ + kQStages * kTileBytes;   // [kLses][kBN]
  static constexpr int kPre = kLse + kLses * kBN * 4;       // prefix of units, [B + 1], 64 bits
  static constexpr int kSums = kPre + (kMaxPackedSeqs + 1) * 8;
  static constexpr int kBars = kSums + 32 * 16;
  static constexpr int kNumBars = 4 + 2 * kQStages + 8 + 2 * kLses;
  static constexpr int kMisc = kBars + kNumBars * 8;
  static constexpr int kBytes = kMisc + 64 + kSmemAlignSlack;
  static_assert(kBytes <= 232448, "dynamic shared memory above the 227 KB per-CTA limit");
};

template <int D, bool kFp8>
struct Shared {
  using L = Layout<D, kFp8>;
  uint8_t* base;
  uint32_t sbase;
  FA_DEV uint32_t bar(int i) const { return sbase + L::kBars + 8 * i; }
  FA_DEV uint32_t k_full(int i) const { return bar(i); }
  FA_DEV uint32_t k_empty(int i) const { return bar(2 + i); }
  FA_DEV uint32_t q_full(int i) const { return bar(4 + i); }
  FA_DEV uint32_t q_empty(int i) const { return bar(4 + L::kQStages + i); }
  FA_DEV uint32_t s_full(int m, int i) const { return bar(4 + 2 * L::kQStages + 2 * m + i); }
  FA_DEV uint32_t s_empty(int m, int i) const { return bar(8 + 2 * L::kQStages + 2 * m + i); }
  FA_DEV uint32_t lse_full(int i) const { return bar(12 + 2 * L::kQStages + i); }
  FA_DEV uint32_t lse_empty(int i) const { return bar(12 + 2 * L::kQStages + kLses + i); }
  FA_DEV const long long* pre() const { return reinterpret_cast<const long long*>(base + L::kPre); }
  FA_DEV float* lse(int i) const { return reinterpret_cast<float*>(base + L::kLse) + i * kBN; }
  FA_DEV uint32_t abort() const { return sbase + L::kMisc + 4; }
  FA_DEV uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(base + L::kMisc); }
  FA_DEV bool wait(uint32_t b, uint32_t parity, int site, const WeighParams& p) const {
    return paged::wait_warp(b, parity, abort(), &g_err, site, p.wait_limit_ns);
  }
  // For waits that last as long as a unit, whose rows may be many (the other roles
  // wait for a tile at a time, and give up first if nothing moves).
  FA_DEV bool wait_long(uint32_t b, uint32_t parity, int site, const WeighParams& p) const {
#pragma unroll 1
    for (int i = 0; i < (1 << 27) && !mbar_try_wait(b, parity) && !ld_shared_volatile(abort()); ++i) __nanosleep(100);
    return wait(b, parity, site, p);
  }
};

// A place in a ring of N.
template <int N>
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  FA_DEV void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1;
    }
  }
};

// 256 keys of a (sequence, head), and the tiles of rows that see some of them.
struct Unit {
  int b, head, key0;
  int n, past, q0, L;
  int tile0, tiles;      // of tt tokens each
  FA_DEV bool two() const { return key0 + kBM < L; }
};
FA_DEV int units_of(int L) { return (L + kUnitKeys - 1) / kUnitKeys; }
FA_DEV Unit unit_at(const WeighParams& p, const long long* pre, long long u) {
  int lo = 0, hi = p.s.B - 1;      // last b with pre[b] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid; else hi = mid - 1;
  }
  const paged::SeqRows r = paged::rows_of(p.s, lo);
  Unit w;
  w.b = lo;
  const int block = (int)paged::div64(u - pre[lo], p.s.Hkv);      // the first keys, which most rows see, come first
  w.head = (int)(u - pre[lo] - (long long)block * p.s.Hkv);
  w.key0 = block * kUnitKeys;
  w.n = r.n;
  w.L = r.L;
  w.past = r.L - r.n;
  w.q0 = r.q0;
  const int tt = kBN / p.group;
  w.tile0 = p.causal ? max(0, w.key0 - w.past) / tt : 0;          // (the first key is seen by the last row at least)
  w.tiles = (w.n + tt - 1) / tt - w.tile0;
  return w;
}

// Q tiles, and the keys of BF16 pages.
template <int D, bool kFp8>
__device__ void load_role(const Shared<D, kFp8>& sh, const CUtensorMap* tq, const CUtensorMap* tk, const WeighParams& p,
                          long long units) {
  using L = Layout<D, kFp8>;
  const int lane = threadIdx.x % 32;
  const int tt = kBN / p.group;
  const int box = min(1 << p.s.page_shift, kBM);
  Ring<2> kr;
  Ring<L::kQStages> qr;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit w = unit_at(p, sh.pre(), u);
    if (!kFp8) {
      if (!sh.wait(sh.k_empty(kr.i), kr.phase ^ 1, kSiteKEmpty, p)) return;
      const int keys = min(kUnitKeys, w.L - w.key0), boxes = (keys + box - 1) / box;
      if (lane == 0) mbar_arrive_expect_tx(sh.k_full(kr.i), boxes * box * 2 * D);
      __syncwarp();
      // each lane issues its own box of 64 columns
      const int i = lane / L::kChunks, c = lane % L::kChunks;
      for (int x = i; x < boxes; x += 32 / L::kChunks) {
        const int key = w.key0 + x * box;
        const int page = p.s.block_table[(size_t)w.b * p.s.max_pages + (key >> p.s.page_shift)];
        const bool bad = page < 0 || page >= p.s.num_pages;
        if (bad) paged::record_bad_input(&g_err, kSitePage);
        tma_load_3d(sh.sbase + L::kK + (2 * kr.i + x * box / kBM) * L::kTileBytes + c * L::kChunkBytes + x * box % kBM * 128,
                    tk, sh.k_full(kr.i), c * 64, key & ((1 << p.s.page_shift) - 1),
                    bad ? -1 : page * p.s.Hkv + w.head);          // -1: reads as zeros
      }
      __syncwarp();
      kr.next();
    }
    for (int t = 0; t < w.tiles; ++t) {
      if (!sh.wait(sh.q_empty(qr.i), qr.phase ^ 1, kSiteQEmpty, p)) return;
      if (lane == 0) {
        mbar_arrive_expect_tx(sh.q_full(qr.i), tt * p.group * D * 2);
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
          tma_load_3d(sh.sbase + L::kQ + qr.i * L::kTileBytes + c * L::kChunkBytes, tq, sh.q_full(qr.i), c * 64,
                      w.head * p.group, w.q0 + (w.tile0 + t) * tt);
      }
      __syncwarp();
      qr.next();
    }
  }
}

// The rows' LSE, 128 floats a tile.
template <int D, bool kFp8>
__device__ void lse_role(const Shared<D, kFp8>& sh, const WeighParams& p, long long units) {
  const int lane = threadIdx.x % 32;
  const int tt = kBN / p.group;
  Ring<kLses> r;
  int tok[kBN / 32], head[kBN / 32];
#pragma unroll
  for (int i = 0; i < kBN / 32; ++i) {
    tok[i] = (lane + 32 * i) / p.group;
    head[i] = lane + 32 * i - tok[i] * p.group;
  }
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit w = unit_at(p, sh.pre(), u);
    for (int t = 0; t < w.tiles; ++t) {
      float x[kBN / 32];
      const int tok0 = (w.tile0 + t) * tt;
#pragma unroll
      for (int i = 0; i < kBN / 32; ++i) {
        x[i] = 0.0f;
        if (tok[i] < tt && tok0 + tok[i] < w.n)
          x[i] = lse_of(p.lse[lse_at(p, w.b, w.q0, w.head * p.group + head[i], tok0 + tok[i])]);
      }
      if (!sh.wait(sh.lse_empty(r.i), r.phase ^ 1, kSiteLseEmpty, p)) return;
#pragma unroll
      for (int i = 0; i < kBN / 32; ++i) sh.lse(r.i)[lane + 32 * i] = -x[i];
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.lse_full(r.i));
      r.next();
    }
  }
}

// E4M3 pages: four warps make the unit's keys BF16, which holds a code times its
// power of two exactly.  Rows behind the sequence's end are left as they were: each
// is a lane of the product of its own.
template <int D>
__device__ void widen_role(const Shared<D, true>& sh, const WeighParams& p, long long units) {
  using L = Layout<D, true>;
  constexpr int kLanes = D / 16;                  // of a row
  constexpr int kRows = 128 / kLanes;             // at a time
  constexpr int kUnroll = 4;
  const int thread = threadIdx.x - 352;
  const int piece = thread % kLanes, row0 = thread / kLanes;
  Ring<2> r;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit w = unit_at(p, sh.pre(), u);
    const int keys = min(kUnitKeys, w.L - w.key0);
    if (!sh.wait_long(sh.k_empty(r.i), r.phase ^ 1, kSiteKEmpty, p)) return;
#pragma unroll 1
    for (int i0 = row0; i0 < keys; i0 += kRows * kUnroll) {
      uint4 x[kUnroll];
      uint32_t byte[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + k * kRows;
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        byte[k] = 127u;
        if (i >= keys) continue;
        const long long row = slot_of(p, w.b, w.head, w.key0 + i);
        if (row < 0) continue;
        x[k] = static_cast<const uint4*>(p.k_pages)[row * kLanes + piece];
        byte[k] = p.k_scale[row];
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + k * kRows;
        if (i >= keys) continue;
        const uint32_t f = byte[k] == 255u ? 0x7FC07FC0u : byte[k] << 7 | byte[k] << 23;
        const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        uint32_t y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t even = paged::mul_bf16x2(paged::e4m3_even(v[j]), f);
          const uint32_t odd = paged::mul_bf16x2(paged::e4m3_odd(v[j]), f);
          y[2 * j] = __byte_perm(even, odd, 0x5410);
          y[2 * j + 1] = __byte_perm(even, odd, 0x7632);
        }
        const int m = i % kBM;
        uint8_t* to = sh.base + L::kK + (2 * r.i + i / kBM) * L::kTileBytes + piece / 4 * L::kChunkBytes + m * 128;
        const int c = piece % 4 * 2;
        *reinterpret_cast<uint4*>(to + ((c ^ (m & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(to + (((c + 1) ^ (m & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(sh.k_full(r.i));
    r.next();
  }
}

// MMA issue (a converged warp, one elected lane).
template <int D, bool kFp8>
__device__ void mma_role(const Shared<D, kFp8>& sh, const uint32_t tmem, const WeighParams& p, long long units) {
  using L = Layout<D, kFp8>;
  constexpr uint32_t kId = idesc_bf16_f32(kBM, kBN, false, false);
  Ring<2> kr, sr[2];
  Ring<L::kQStages> qr;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit w = unit_at(p, sh.pre(), u);
    const int tiles = __shfl_sync(0xffffffffu, w.tiles, 0);
    const bool two = __shfl_sync(0xffffffffu, (int)w.two(), 0) != 0;
    // (the keys of a unit are on their way while the one before is worked on, but E4M3's
    // may be waited for as long as a unit takes)
    if (!sh.wait_long(sh.k_full(kr.i), kr.phase, kSiteKFull, p)) return;
    tc_fence_after();
    for (int t = 0; t < tiles; ++t) {
      if (!sh.wait(sh.q_full(qr.i), qr.phase, kSiteQFull, p)) return;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (m == 1 && !two) break;
        if (!sh.wait(sh.s_empty(m, sr[m].i), sr[m].phase ^ 1, kSiteSEmpty, p)) return;
        tc_fence_after();
        const uint64_t da = sdesc_sw128(sh.sbase + L::kK + (2 * kr.i + m) * L::kTileBytes, 16, 1024);
        const uint64_t db = sdesc_sw128(sh.sbase + L::kQ + qr.i * L::kTileBytes, 16, 1024);
        const uint32_t d = tmem + m * 256 + sr[m].i * 128;
        mma_ss_w<0, 0>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 0u);
        mma_ss_w<2, 2>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 1u);
        mma_ss_w<4, 4>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 1u);
        mma_ss_w<6, 6>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 1u);
        if (D == 128) {
          constexpr uint32_t kC = L::kChunkBytes / 16;
          mma_ss_w<kC, kC>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 1u);
          mma_ss_w<kC + 2, kC + 2>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 1u);
          mma_ss_w<kC + 4, kC + 4>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 1u);
          mma_ss_w<kC + 6, kC + 6>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 1u);
        }
        mma_commit_w(sh.s_full(m, sr[m].i));
        sr[m].next();
      }
      mma_commit_w(sh.q_empty(qr.i));
      qr.next();
    }
    mma_commit_w(sh.k_empty(kr.i));
    kr.next();
  }
}

// 32 scores of a key: their exponentials added to sum2; kMasked: those of columns
// [lo, hi) alone.
template <bool kMasked>
FA_DEV void add_weights(const uint32_t (&x)[32], const float* nlse, float scale, int lo, int hi, uint64_t (&sum2)[2]) {
  const uint64_t scale2 = pk2(scale, scale), log2e2 = pk2(kLog2e, kLog2e);
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(nlse + i);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // taken from the LSE before it goes to log2 units: the difference is small where
      // the weight is large, and so is its rounding
      const uint64_t s2 = pk2(__uint_as_float(x[i + 2 * h]), __uint_as_float(x[i + 2 * h + 1]));
      float a, b;
      up2(mul2(fma2(s2, scale2, h ? pk2(l.z, l.w) : pk2(l.x, l.y)), log2e2), a, b);
      if (kMasked) {
        const int c = i + 2 * h;
        if (c < lo || c >= hi) a = -INFINITY;
        if (c + 1 < lo || c + 1 >= hi) b = -INFINITY;
      }
      sum2[h] = add2(sum2[h], pk2(ex2_mufu(a), ex2_mufu(b)));
    }
  }
}

// Exponentials and sums of 128 keys of each unit, a thread a key.
template <int D, bool kFp8>
__device__ void sum_role(const int m, const Shared<D, kFp8>& sh, const uint32_t tmem, const WeighParams& p,
                         long long units) {
  const int lane = threadIdx.x % 32, wq = threadIdx.x / 32 % 4;
  const int tt = kBN / p.group;
  Ring<2> sr;
  Ring<kLses> lr;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit w = unit_at(p, sh.pre(), u);
    const int key = w.key0 + m * kBM + wq * 32 + lane;
    const bool active = m == 0 || w.two();
    long long slot = -1;
    float old = 0.0f;
    if (key < w.L) {
      slot = slot_of(p, w.b, w.head, key);
      if (slot >= 0 && p.decay != 0.0f && key < w.past) old = p.sums[slot];
    }
    uint64_t total2[2] = {0ull, 0ull};
    for (int t = 0; t < w.tiles; ++t) {
      const int tok0 = (w.tile0 + t) * tt;
      const int hi = min(tt, w.n - tok0) * p.group;                                   // columns with a row
      const int lo = p.causal ? max(0, key - w.past - tok0) * p.group : 0;            // first one that sees the key
      if (!sh.wait_long(sh.lse_full(lr.i), lr.phase, kSiteLseFull, p)) return;
      if (active) {
        if (!sh.wait(sh.s_full(m, sr.i), sr.phase, kSiteSFull, p)) return;
        tc_fence_after();
        const uint32_t tm = tmem + (uint32_t(wq * 32) << 16) + m * 256 + sr.i * 128;
        const float* nlse = sh.lse(lr.i);
        const bool plain = __all_sync(0xffffffffu, lo == 0 && hi == kBN);
        uint64_t sum2[2] = {0ull, 0ull};
        uint32_t xa[32], xb[32];
        tmem_ld32(tm, xa);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = 64 * half;
          tmem_ld_wait();
          tmem_ld_fence(xa);
          tmem_ld32(tm + c + 32, xb);
          if (plain)
            add_weights<false>(xa, nlse + c, p.scale, 0, 0, sum2);
          else
            add_weights<true>(xa, nlse + c, p.scale, lo - c, hi - c, sum2);
          tmem_ld_wait();
          tmem_ld_fence(xb);
          if (half == 0) {
            tmem_ld32(tm + 64, xa);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sh.s_empty(m, sr.i));
          }
          if (plain)
            add_weights<false>(xb, nlse + c + 32, p.scale, 0, 0, sum2);
          else
            add_weights<true>(xb, nlse + c + 32, p.scale, lo - c - 32, hi - c - 32, sum2);
        }
        total2[0] = add2(total2[0], sum2[0]);
        total2[1] = add2(total2[1], sum2[1]);
        sr.next();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.lse_empty(lr.i));
      lr.next();
    }
    if (slot >= 0) {
      float a, b;
      up2(add2(total2[0], total2[1]), a, b);
      p.sums[slot] = p.decay * old + (a + b);
    }
  }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(Layout<D, kFp8>::kThreads, 1)
    block_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const WeighParams p) {
  using L = Layout<D, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32;
  Shared<D, kFp8> sh;
  sh.base = smem;
  sh.sbase = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(sh.k_full(i), kFp8 ? 4 : 1);      // one arrival per widening warp
      mbar_init(sh.k_empty(i), 1);
      for (int m = 0; m < 2; ++m) {
        mbar_init(sh.s_full(m, i), 1);
        mbar_init(sh.s_empty(m, i), 4);
      }
    }
    for (int i = 0; i < L::kQStages; ++i) {
      mbar_init(sh.q_full(i), 1);
      mbar_init(sh.q_empty(i), 1);
    }
    for (int i = 0; i < kLses; ++i) {
      mbar_init(sh.lse_full(i), 1);
      mbar_init(sh.lse_empty(i), 8);
    }
    st_shared(sh.abort(), 0);
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    if (!kFp8) tma_prefetch_desc(&tm_k);
  }
  if (warp == 9) {
    tmem_alloc(sh.tmem_slot(), 512);
    tmem_relinquish();
  }
  const bool ok = paged::prefix_sequences(
      p.s, p.max_q,
      [&](const paged::SeqRows& r) { return paged::Work{(long long)p.s.Hkv * units_of(r.L), 0, 0}; },
      reinterpret_cast<long long*>(smem + L::kPre), nullptr, reinterpret_cast<long long*>(smem + L::kSums));
  if (!ok && blockIdx.x == 0 && threadIdx.x == 0) paged::record_bad_input(&g_err, kSiteSeqs);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sh.tmem_slot();
  const long long units = ok ? sh.pre()[p.s.B] : 0;

  if (warp < 8) {
    sum_role<D, kFp8>(warp / 4, sh, tmem, p, units);
  } else if (warp == 8) {
    load_role<D, kFp8>(sh, &tm_q, &tm_k, p, units);
  } else if (warp == 9) {
    mma_role<D, kFp8>(sh, tmem, p, units);
  } else if (warp == 10) {
    lse_role<D, kFp8>(sh, p, units);
  } else {
    if constexpr (kFp8) widen_role<D>(sh, p, units);
  }

  // after a give-up, copies and MMAs in flight land before the memory they target is
  // released
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    if (ld_shared_volatile(sh.abort())) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
      __syncwarp();
    }
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kFp8>
fa_status launch_blocks(const WeighParams& p, int num_sms, cudaStream_t stream) {
  using L = Layout<D, kFp8>;
  const int page_size = 1 << p.s.page_shift;
  CUtensorMap tq, tk{};
  fa_status st;
  const int rows = p.s.cu ? p.s.Sn : p.s.B * p.s.Sn;
  if ((st = make_tmap_rows_group(&tq, p.q, rows, p.Hq, D, p.group, kBN / p.group)) != FA_OK) return st;
  if (!kFp8 && (st = make_tmap_pages(&tk, p.k_pages, (long long)p.s.num_pages * p.s.Hkv, page_size, D, false,
                                     page_size < kBM ? page_size : kBM)) != FA_OK)
    return st;
  auto kernel = block_kernel<D, kFp8>;
  if ((st = prepare_kernel(reinterpret_cast<const void*>(kernel), L::kBytes)) != FA_OK) return st;
  kernel<<<num_sms, L::kThreads, L::kBytes, stream>>>(tq, tk, p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool kFp8>
fa_status launch(const WeighParams& p, int num_sms, cudaStream_t stream) {
  return (long long)p.max_q * p.group <= kStepRows ? launch_step<D, kFp8>(p, num_sms, stream)
                                                    : launch_blocks<D, kFp8>(p, num_sms, stream);
}

}  // namespace weigh

fa_status launch_cache_weights(const WeighParams& p, int num_sms, cudaStream_t stream) {
  if (p.D == 128)
    return p.k_scale ? weigh::launch<128, true>(p, num_sms, stream) : weigh::launch<128, false>(p, num_sms, stream);
  return p.k_scale ? weigh::launch<64, true>(p, num_sms, stream) : weigh::launch<64, false>(p, num_sms, stream);
}

fa_status weigh_take_device_error() {
  DeviceError e{0, 0};
  if (cudaMemcpyFromSymbol(&e, weigh::g_err, sizeof(e)) != cudaSuccess) return FA_ERR_CUDA;
  if (e.status != 0) {
    const DeviceError z{0, 0};
    if (cudaMemcpyToSymbol(weigh::g_err, &z, sizeof(z)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return static_cast<fa_status>(e.status);
}

}  // namespace fa
