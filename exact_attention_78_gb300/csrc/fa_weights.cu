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
            kSiteLseEmpty, kSiteStep, kSiteUnitEmpty, kSiteUnitFull,
            kSitePart };

FA_DEV size_t lse_at(const WeighParams& p, int b, int q0, int head, int tok) {
  return p.s.cu ? (size_t)head * p.s.Sn + q0 + tok : ((size_t)b * p.Hq + head) * p.s.Sn + tok;
}
// A row that saw no key has an LSE of -inf, and gives no key a weight.  (With finite
// queries: a score of NaN or infinity stays NaN.  fwd_paged gives no such row that sees a key; a look at
// each row's LSE beside its score took 3% (2048 tokens over 32,768 keys) to 12% more time.)
FA_DEV float lse_of(float x) { return x == -INFINITY ? INFINITY : x; }

// The barrier's phase waits for bytes that nobody brings (fa_diag_cache_weights).
FA_DEV void hold(uint32_t bar) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], 16;" ::"r"(bar) : "memory");
}

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
// side, 8 a tile.  A product's sum may take its elements in any order, so each lane's
// share of a key is whole pieces of 16 bytes.  A head's rows of a page lie in one
// piece, so that one bulk copy brings a tile of keys; each warp has a ring of its
// own in shared memory and is on its own, and some 150 KB an SM are under way.  All
// tiles of all (sequence, head) units form one line, of which every warp takes an equal
// stretch.  (64 sequences of random lengths up to 4096 keys, 2229 on average, 8 heads, D = 128,
// 4 rows: E4M3 32 us of the bytes' 23, BF16 52 of 45.
// Every lane loading its own pieces into registers, 64 ragged sequences up to 8192
// E4M3 keys took 73 us; copying them to shared memory 60; so 57.)
//
// E4M3 codes become FP16, and the queries too, by a power of two of each row's own
// (as in the decode kernel of the attention); keys' scales go to the scores in FP32.  A
// product is brought back by its row's power of two, with that of `scale`, before it
// meets the key's: that is where queries and keys far from one cancel, and the other
// way round products of 2^30 pass FP32's range with keys from 2^98 on.  Powers of two
// round nothing; the rest of `scale`, 1 to 2, goes along with the key's.

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

template <int D, bool kFp8, int kTiles>
struct StepLayout {
  static constexpr int kWarps = kTiles == 4 && D == 128 ? 8 : 16;      // (32 rows of Q in registers)
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPieces = D * (kFp8 ? 1 : 2) / 64;     // of 16 bytes of a key that a lane has
  static constexpr int kRowBytes = 64 * kPieces;
  static constexpr int kTile = 16 * kRowBytes;
  // Tiles of a stage: two where they are small, which halves what goes with a stage.
  static constexpr int kHalves = D == 128 && !kFp8 ? 1 : 2;
  static constexpr int kKeys = 16 * kHalves;
  // behind the keys: their sums so far, their scales, the halves' rows
  static constexpr int kOld = kHalves * kTile, kScales = kOld + kHalves * 64, kRows = kScales + kHalves * 16;
  static constexpr int kStage = (kRows + kHalves * 8 + 127) / 128 * 128;
  static constexpr int kRing = 212992;
  static constexpr int kFit = kRing / (kWarps * kStage);
  static constexpr int kDepth = kFit < 6 ? kFit : 6;
  static constexpr int kBars = kWarps * kDepth * kStage;  // [warp][stage]
  static constexpr int kMisc = kBars + kWarps * kDepth * 8;
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kHalfBytes = kTile + 64 + (kFp8 ? 16 : 0);
};

// A walk over a warp's stretch of the line, tile by tile.
struct Walk {
  paged::SeqRows q;
  int b, head, k, tiles;      // tile k of `tiles` of a unit
  long long left;             // tiles from here on
  // To the next tile; whether it is another unit's.
  template <int kKeys>
  FA_DEV bool next(const WeighParams& p) {
    --left;
    if (++k < tiles || left == 0) return false;
    k = 0;
    if (++head == p.s.Hkv) {
      head = 0;
      do {
        ++b;                  // (one with tiles follows)
        q = paged::rows_of(p.s, b);
        tiles = q.n > 0 ? (q.L + kKeys - 1) / kKeys : 0;
      } while (tiles == 0);
    }
    return true;
  }
};

template <int D, bool kFp8, int kTiles>
__global__ void __launch_bounds__(StepLayout<D, kFp8, kTiles>::kThreads, 1) step_kernel(const WeighParams p) {
  using Lay = StepLayout<D, kFp8, kTiles>;
  constexpr int kPieces = Lay::kPieces, kHalves = Lay::kHalves, kKeys = Lay::kKeys;
  constexpr int kWords = kFp8 ? 2 * kPieces : kPieces;        // of 16 bytes of a row of Q
  // The tensor cores cut a running sum off where FP32 would round it, so a score is the
  // sum of kParts shorter ones that are added, and rounded, outside them.  Error of
  // the sums over 65,536 BF16 keys, D = 128, against 64 bits: one token, 8 heads
  // 8.7e-7 as one sum, 5.2e-7 as two, 4.1e-7 as four; 32 rows 8.4e-7 and 3.7e-7.  Four cost
  // nothing at 8 rows (52 us for 64 sequences up to 4096 keys, 2229 on average); two cost
  // 64 -> 70 us at 32, four spill.
  constexpr int kParts = kTiles == 1 ? 4 : 2;
  extern __shared__ __align__(128) uint8_t ring_raw[];
  __shared__ long long pre[kMaxPackedSeqs + 1];
  __shared__ long long work_sums[2 * Lay::kWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int c = lane % 4, g = lane / 4;
  const uint32_t bars = smem_u32(ring_raw) + Lay::kBars + warp * Lay::kDepth * 8, abort = smem_u32(ring_raw) + Lay::kMisc;
  if (lane < Lay::kDepth) mbar_init(bars + 8 * lane, 1);
  if (lane < Lay::kDepth && lane == p.held) hold(bars + 8 * lane);
  if (threadIdx.x == 0) st_shared(abort, 0);
  fence_barrier_init();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool ok = paged::prefix_sequences(
      p.s, p.max_q,
      [&](const paged::SeqRows& r) {
        return paged::Work{(long long)p.s.Hkv * ((r.L + kKeys - 1) / kKeys), 0, 0};
      },
      pre, nullptr, work_sums);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) paged::record_bad_input(&g_err, kSiteSeqs);
    return;
  }
  const long long total = pre[p.s.B];
  const int warps = gridDim.x * Lay::kWarps, id = warp * gridDim.x + blockIdx.x;
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
    at.tiles = (at.q.L + kKeys - 1) / kKeys;
    at.head = (int)paged::div64(t0 - pre[lo], at.tiles);
    at.k = (int)(t0 - pre[lo] - (long long)at.head * at.tiles);
  }

  uint8_t* ring = ring_raw + warp * Lay::kDepth * Lay::kStage;
  Walk ahead = at;                                     // the tile that is copied next
  int held = -64, pages = -1;                          // its unit's pages [held, held + 32), one a lane
  // what a lane copies of a stage: a half's keys, sums or scales
  const int half = lane / 3, what = lane % 3;
  const uint32_t copy_to = what == 0 ? half * Lay::kTile : what == 1 ? Lay::kOld + half * 64 : Lay::kScales + half * 16;
  const char* copy_from = what == 0 ? static_cast<const char*>(p.k_pages)
                          : what == 1 ? reinterpret_cast<const char*>(p.sums)
                                      : reinterpret_cast<const char*>(p.k_scale);
  const uint32_t copy_row = what == 0 ? Lay::kRowBytes : what == 1 ? 4 : 1;      // bytes of a key
  const bool copies = lane < 3 * kHalves && (kFp8 || what != 2);
  auto copy = [&](int stage) {
    if (ahead.left == 0) return;
    const int key0 = ahead.k * kKeys, page_at = key0 >> p.s.page_shift;
    if (page_at >= held + 31 || page_at < held) {      // (two pages at most)
      held = page_at;
      pages = held + lane <= (ahead.q.L - 1) >> p.s.page_shift
                  ? p.s.block_table[(size_t)ahead.b * p.s.max_pages + held + lane]
                  : -1;
    }
    const int key = key0 + 16 * half;
    const int page = __shfl_sync(0xffffffffu, pages, (key >> p.s.page_shift) - held);
    const bool mine = copies && key < ahead.q.L;
    const bool good = mine && (unsigned)page < (unsigned)p.s.num_pages;
    if (mine && !good) paged::record_bad_input(&g_err, kSitePage);
    const long long row = ((long long)page * p.s.Hkv + ahead.head << p.s.page_shift) + (key & ((1 << p.s.page_shift) - 1));
    uint8_t* to = ring + stage * Lay::kStage;
    if (copies && what == 0) *reinterpret_cast<long long*>(to + Lay::kRows + 8 * half) = good ? row : -1;
    const int halves = __popc(__ballot_sync(0xffffffffu, good && what == 0));
    if (lane == 0) mbar_arrive_expect_tx(bars + 8 * stage, halves * Lay::kHalfBytes);
    __syncwarp();
    if (good) bulk_load(smem_u32(to) + copy_to, copy_from + row * copy_row, 16 * copy_row, bars + 8 * stage);
    if (ahead.next<kKeys>(p)) held = -64;
  };
#pragma unroll 1
  for (int i = 0; i < Lay::kDepth; ++i) copy(i);

  const int least_exp = 14 + max(0, 127 - (int)(__float_as_uint(p.scale) >> 23));
  const float scale_pow = __uint_as_float(__float_as_uint(p.scale) & 0x7F800000u);
  const uint32_t scale_rest = __float_as_uint(p.scale) & 0x007FFFFFu;      // (p.scale is a normal number)
  int stage = 0;
  uint32_t phase = 0;
  bool fresh = true;                                   // a unit begins
  uint4 qf[kTiles][kWords];                            // row 8 n + g, as the keys' pieces lie
  float row_scale[kTiles][2], nlse[kTiles][2];         // of rows 8 n + 2 c + e
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
        float scale = kFp8 ? scale_pow : p.scale;
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
          nlse[n][e] =
              row >= rows ? 0.0f : -lse_of(p.lse[lse_at(p, at.b, at.q.q0, at.head * p.group + row - tk * p.group, tk)]);
        }
      }
    }
    if (!paged::wait_warp(bars + 8 * stage, phase, abort, &g_err, kSiteStep, p.wait_limit_ns)) {
      // what is under way lands before the memory that it targets is released
      const uint64_t w0 = globaltimer_ns();
      while (globaltimer_ns() - w0 < 2000000ull) __nanosleep(1000);
      return;
    }
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
      const uint8_t* from = ring + stage * Lay::kStage + half * Lay::kTile + g * Lay::kRowBytes + c * 16;
      const uint8_t* stats = ring + stage * Lay::kStage;
      const int key0 = at.k * kKeys + 16 * half;
      // [2 h + e]: key g + 8 h, row 8 n + 2 c + e
      float part[kTiles][kParts][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < kParts; ++i) part[n][i][0] = part[n][i][1] = part[n][i][2] = part[n][i][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(from + i * 64);
        const uint4 y = *reinterpret_cast<const uint4*>(from + 8 * Lay::kRowBytes + i * 64);
        if (!kFp8) {
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            mma16816(part[n][2 * i % kParts], x.x, y.x, x.y, y.y, qf[n][i].x, qf[n][i].y);
            mma16816(part[n][(2 * i + 1) % kParts], x.z, y.z, x.w, y.w, qf[n][i].z, qf[n][i].w);
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
              mma16816_f16(part[n][j % kParts], a0, a1, a2, a3, j % 2 ? qw.z : qw.x, j % 2 ? qw.w : qw.y);
            }
          }
        }
      }
      float s[kTiles][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = part[n][0][e];
#pragma unroll
          for (int i = 1; i < kParts; ++i) s[n][e] += part[n][i][e];
        }
      float w[2];                                      // of keys g, g + 8
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (a row that stands for NaN has codes of zero and the byte 255, which is
        // infinity or NaN here: its scores are NaN)
        const float fac =
            kFp8 ? __uint_as_float((uint32_t)stats[Lay::kScales + 16 * half + g + 8 * h] << 23 | scale_rest) : 1.0f;
        uint64_t sum2 = 0ull;
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          // taken from the LSE before it goes to log2 units: the difference is small
          // where the weight is large, and so is its rounding
          const uint64_t s2 = pk2(s[n][2 * h], s[n][2 * h + 1]), row2 = pk2(row_scale[n][0], row_scale[n][1]);
          const uint64_t nlse2 = pk2(nlse[n][0], nlse[n][1]);
          const uint64_t x2 =
              mul2(kFp8 ? fma2(mul2(s2, row2), pk2(fac, fac), nlse2) : fma2(s2, row2, nlse2), pk2(kLog2e, kLog2e));
          float x0, x1;
          up2(x2, x0, x1);
          const int key = key0 + g + 8 * h;
          sum2 = add2(sum2, pk2(key < lim[n][0] ? ex2_mufu(x0) : 0.0f, key < lim[n][1] ? ex2_mufu(x1) : 0.0f));
        }
        float a, b;
        up2(sum2, a, b);
        w[h] = a + b;
      }
      // over the four lanes of a key; lanes with an odd c end up with key g + 8, the
      // others with key g
      float sum = c & 1 ? w[1] : w[0];
      sum += __shfl_xor_sync(0xffffffffu, c & 1 ? w[0] : w[1], 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const long long row = *reinterpret_cast<const long long*>(stats + Lay::kRows + 8 * half);
      const int in = g + 8 * c;                        // lanes with c < 2 write a key's sum
      if (c < 2 && key0 + in < at.q.L && row >= 0) {
        const float old = *reinterpret_cast<const float*>(stats + Lay::kOld + 64 * half + 4 * in);
        p.sums[row + in] = fmaf(p.decay, p.decay != 0.0f && key0 + in < past ? old : 0.0f, sum);
      }
    }
    __syncwarp();                                      // every lane is done with the stage
    copy(stage);
    if (++stage == Lay::kDepth) {
      stage = 0;
      phase ^= 1;
    }
    fresh = at.next<kKeys>(p);
  }
}

template <int D, bool kFp8, int kTiles>
fa_status launch_tiles(const WeighParams& p, int num_sms, cudaStream_t stream) {
  using Lay = StepLayout<D, kFp8, kTiles>;
  auto kernel = step_kernel<D, kFp8, kTiles>;
  const fa_status st = prepare_kernel(reinterpret_cast<const void*>(kernel), Lay::kBytes);
  if (st != FA_OK) return st;
  return launch_overlapped(kernel, dim3(num_sms), Lay::kThreads, Lay::kBytes, stream, p);
}

template <int D, bool kFp8>
fa_status launch_step(const WeighParams& p, int num_sms, cudaStream_t stream) {
  const long long rows = (long long)p.max_q * p.group;
  return rows <= 8    ? launch_tiles<D, kFp8, 1>(p, num_sms, stream)
         : rows <= 16 ? launch_tiles<D, kFp8, 2>(p, num_sms, stream)
                      : launch_tiles<D, kFp8, 4>(p, num_sms, stream);
}

// --------------------------------------------------------------- many rows --
// S^T = K Q^T on tcgen05: 256 keys of a unit (two tiles of 128, the M side, one key a
// lane of tensor memory), the rows 128 at a time (N).  A thread has a key and half of a
// tile's rows, reads their scores out of tensor memory and adds their exponentials up:
// no row statistics, no second product.  Both operands' tiles are read by all units
// of a head (Q) or tiles of rows (K), from L2.
//
// 2048 tokens over 32,768 BF16 keys, 32/8 heads: 433 us, of which the products take 281 at
// cuBLAS's rate and the exponentials 230 (452 where a tile that is not full, or not seen
// whole by all keys of a warp, was masked throughout); each set of warps waits for scores a tenth of
// the time, the products' warp a third of it for room.  (One set of eight warps 597 us;
// two that took tiles in turn 510; a share of the exponentials as polynomials on the
// FMA pipe, 1 / 2 / 4 of 8 pairs, 549 / 594 / 728 instead.)  With few rows a unit's fixed
// work bounds it: 32 sequences of random lengths up to 4096 keys, 128 rows each, BF16 39 us
// of the bytes' 24, E4M3 72 of 13, where the widening takes as long as two tiles of rows.
// A score is one sum in the tensor cores, which cut it off where FP32 would round it:
// relative error of the sums against 64 bits 1.4e-7 to 4.6e-7 for that call, D = 128 (the plain
// form in FP32 4e-8 to 7e-8); 64 tokens over 8192 keys 0.9e-7 to 8e-7, D = 64 0.6e-7 to 1.7e-7.
//
// Warps: 0-15 exponentials (8 m + 4 j on: keys m, rows j of a tile), 16 loads (Q; K of
// BF16 pages), 17 MMA issue, 18 the rows' LSE, 19 units (works out the next ones, looks
// their pages up and has their old sums copied, ahead of the others), 20-27 widening
// (E4M3 pages: codes and scale to BF16, once per unit; see key_exp).
//
// Tensor memory: scores of the first keys at columns 0 and 128, tile by tile in turn, of
// the second at 256 and 384.

constexpr int kBM = 128, kBN = 128;
constexpr int kUnitKeys = 2 * kBM;
constexpr int kUnits = 6;

// 256 keys of a (sequence, head), and the tiles of rows that see some of them, as the
// roles get them.
struct Unit {
  int b, head, key0;     // b < 0: no more work
  int n, past, q0, L;
  int tile0, tiles;      // of tt tokens each
  int pad[3];
  long long row[kUnitKeys / 16];      // of every 16 keys' first; -1: behind the end, or in a bad page
  float old[kUnitKeys];
  float part[kUnitKeys];              // what the second set of warps has added up
  FA_DEV bool two() const { return key0 + kBM < L; }
};

template <int D, bool kFp8>
struct Layout {
  static constexpr int kWideners = kFp8 ? 8 : 0;
  static constexpr int kThreads = 640 + 32 * kWideners;
  static constexpr int kReaders = 19 + kWideners;           // warps that take units
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = 128 * 128;             // 128 rows by 64 columns
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kQStages = D == 128 ? 2 : 4;
  static constexpr int kK = 0;                              // [2][two tiles]
  static constexpr int kQ = kK + 4 * kTileBytes;
  static constexpr int kLse = kQ + kQStages * kTileBytes;   // [2][kBN]
  static constexpr int kUnitRing = kLse + 2 * kBN * 4;
  static constexpr int kPre = kUnitRing + kUnits * (int)sizeof(Unit);      // prefix of units, [B + 1], 64 bits
  static constexpr int kSums = kPre + (kMaxPackedSeqs + 1) * 8;
  static constexpr int kBars = kSums + 32 * 16;
  static constexpr int kTileBars = 4 + 2 * kQStages + 8 + 2;      // somebody waits for each with a limit
  static constexpr int kNumBars = kTileBars + 4 * kUnits;
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
  // scores are complete, and the rows' LSE is here
  FA_DEV uint32_t s_full(int m, int i) const { return bar(4 + 2 * L::kQStages + 2 * m + i); }
  FA_DEV uint32_t s_empty(int m, int i) const { return bar(8 + 2 * L::kQStages + 2 * m + i); }
  FA_DEV uint32_t lse_empty(int i) const { return bar(12 + 2 * L::kQStages + i); }
  FA_DEV uint32_t unit_full(int i) const { return bar(14 + 2 * L::kQStages + i); }
  FA_DEV uint32_t unit_empty(int i) const { return bar(14 + 2 * L::kQStages + kUnits + i); }
  FA_DEV uint32_t part_full(int i, int m) const { return bar(14 + 2 * L::kQStages + 2 * kUnits + 2 * i + m); }
  FA_DEV Unit* unit(int i) const { return reinterpret_cast<Unit*>(base + L::kUnitRing) + i; }
  FA_DEV const long long* pre() const { return reinterpret_cast<const long long*>(base + L::kPre); }
  FA_DEV float* lse(int i) const { return reinterpret_cast<float*>(base + L::kLse) + i * kBN; }
  FA_DEV uint32_t abort() const { return sbase + L::kMisc + 4; }
  FA_DEV uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(base + L::kMisc); }
  FA_DEV bool wait(uint32_t b, uint32_t parity, int site, const WeighParams& p) const {
    return paged::wait_warp(b, parity, abort(), &g_err, site, p.wait_limit_ns);
  }
  // For waits that last as long as a unit, whose rows may be many (the other roles
  // wait for a tile at a time, and give up first if nothing moves).
  FA_DEV bool wait_long(uint32_t b, uint32_t parity, int site, const WeighParams& p, bool sleeps = true) const {
#pragma unroll 1
    for (int i = 0; i < (1 << 27) && !mbar_try_wait(b, parity) && !ld_shared_volatile(abort()); ++i)
      if (sleeps) __nanosleep(100);
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

FA_DEV int units_of(int L) { return (L + kUnitKeys - 1) / kUnitKeys; }

// Works out this thread block's units, every gridDim.x-th, two at a time, half a warp
// each.
template <int D, bool kFp8>
__device__ void unit_role(const Shared<D, kFp8>& sh, const WeighParams& p, long long units) {
  const int lane = threadIdx.x % 32, half = lane / 16, in = lane % 16;
  const int tt = kBN / p.group;
  const long long* pre = sh.pre();
  Ring<kUnits> r;
  for (long long u0 = blockIdx.x;; u0 += 2 * gridDim.x) {
    Ring<kUnits> next = r;
    next.next();
    const int i = half ? next.i : r.i;
    const long long u = u0 + half * gridDim.x;
    const bool some = u < units;
    int lo = 0;                      // last b with pre[b] <= u
    if (some) {
      int hi = p.s.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= u) lo = mid; else hi = mid - 1;
      }
    }
    __syncwarp();
    const paged::SeqRows q = paged::rows_of(p.s, lo);
    const int block = some ? (int)paged::div64(u - pre[lo], p.s.Hkv) : 0;      // the first keys, which most rows see, come first
    const int head = some ? (int)(u - pre[lo] - (long long)block * p.s.Hkv) : 0;
    const int key = block * kUnitKeys + 16 * in, past = q.L - q.n;
    const long long row = some && key < q.L ? slot_of(p, lo, head, key) : -1;
    const uint32_t good = __ballot_sync(0xffffffffu, row >= 0);
    if (!sh.wait_long(sh.unit_empty(r.i), r.phase ^ 1, kSiteUnitEmpty, p)) return;
    if (!sh.wait_long(sh.unit_empty(next.i), next.phase ^ 1, kSiteUnitEmpty, p)) return;
    Unit* to = sh.unit(i);
    to->row[in] = row;
    __syncwarp();                    // the rows are written
    if (in == 0) {
      to->b = some ? lo : -1;
      to->head = head;
      to->key0 = block * kUnitKeys;
      to->n = q.n;
      to->past = past;
      to->q0 = q.q0;
      to->L = q.L;
      const int tile0 = p.causal ? max(0, block * kUnitKeys - past) / tt : 0;      // (the last row at least sees the first key)
      to->tile0 = tile0;
      to->tiles = (q.n + tt - 1) / tt - tile0;
      mbar_arrive_expect_tx(sh.unit_full(i), __popc(good >> 16 * half & 0xFFFFu) * 64);
    }
    __syncwarp();
    if (row >= 0) bulk_load(smem_u32(to->old + 16 * in), p.sums + row, 64, sh.unit_full(i));
    if (u0 + gridDim.x >= units) return;      // one of them said that there are no more
    r = next;
    r.next();
  }
}

// Takes units out of the ring.
template <int D, bool kFp8>
struct UnitReader {
  const Shared<D, kFp8>& sh;
  const WeighParams& p;
  Ring<kUnits> r;
  FA_DEV UnitReader(const Shared<D, kFp8>& s, const WeighParams& q) : sh(s), p(q) {}
  // The next one; nullptr at the end of the work or after a give-up.  The whole warp
  // calls it, and done() when it no longer needs the unit.
  FA_DEV const Unit* next(bool sleeps = true) {
    if (!sh.wait_long(sh.unit_full(r.i), r.phase, kSiteUnitFull, p, sleeps)) return nullptr;
    const Unit* w = sh.unit(r.i);
    return w->b < 0 ? nullptr : w;
  }
  FA_DEV void done() {
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(sh.unit_empty(r.i));
    r.next();
  }
};
FA_DEV int all_same(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Q tiles, and the keys of BF16 pages.
template <int D, bool kFp8>
__device__ void load_role(const Shared<D, kFp8>& sh, const CUtensorMap* tq, const CUtensorMap* tk, const WeighParams& p) {
  using L = Layout<D, kFp8>;
  const int lane = threadIdx.x % 32;
  const int tt = kBN / p.group;
  const int box = min(1 << p.s.page_shift, kBM);
  Ring<2> kr;
  Ring<L::kQStages> qr;
  UnitReader<D, kFp8> in(sh, p);
  while (const Unit* w = in.next()) {
    const int tiles = all_same(w->tiles), head = all_same(w->head), q0 = all_same(w->q0 + w->tile0 * tt);
    if (!kFp8) {
      if (!sh.wait(sh.k_empty(kr.i), kr.phase ^ 1, kSiteKEmpty, p)) return;
      const int keys = min(kUnitKeys, w->L - w->key0), boxes = (keys + box - 1) / box;
      if (lane == 0) mbar_arrive_expect_tx(sh.k_full(kr.i), boxes * box * 2 * D);
      __syncwarp();
      // each lane issues its own box of 64 columns
      const int c = lane % L::kChunks;
      for (int x = lane / L::kChunks; x < boxes; x += 32 / L::kChunks) {
        const int row0 = x * box;
        const long long row = w->row[row0 / 16];
        tma_load_3d(sh.sbase + L::kK + (2 * kr.i + row0 / kBM) * L::kTileBytes + c * L::kChunkBytes + row0 % kBM * 128, tk,
                    sh.k_full(kr.i), c * 64, row < 0 ? 0 : (int)(row & ((1 << p.s.page_shift) - 1)),
                    row < 0 ? -1 : (int)(row >> p.s.page_shift));          // -1: reads as zeros
      }
      __syncwarp();
      kr.next();
    }
    in.done();
    for (int t = 0; t < tiles; ++t) {
      if (!sh.wait(sh.q_empty(qr.i), qr.phase ^ 1, kSiteQEmpty, p)) return;
      if (lane == 0) {
        mbar_arrive_expect_tx(sh.q_full(qr.i), tt * p.group * D * 2);
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
          tma_load_3d(sh.sbase + L::kQ + qr.i * L::kTileBytes + c * L::kChunkBytes, tq, sh.q_full(qr.i), c * 64,
                      head * p.group, q0 + t * tt);
      }
      __syncwarp();
      qr.next();
    }
  }
}

// The rows' LSE, negative, 128 floats a tile.  They are loaded kAhead tiles before their
// turn, also over the units' borders: one tile at a time, with the loads' latency
// each time, this warp took 2300 cycles a tile and held up all others.
template <int D, bool kFp8>
__device__ void lse_role(const Shared<D, kFp8>& sh, const WeighParams& p) {
  constexpr int kAhead = 2;
  // With tile k on its way, and each unit a tile, this warp waits for unit k + kAhead.
  // That comes together with one more, whose slot has to be that of a unit before k.
  static_assert(kAhead + 1 - kUnits <= -1, "a tile waits for a unit that waits for it");
  constexpr int kEach = kBN / 32;
  const int lane = threadIdx.x % 32;
  const int tt = kBN / p.group;
  int tok[kEach], head[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    tok[i] = (lane + 32 * i) / p.group;
    head[i] = lane + 32 * i - tok[i] * p.group;
  }
  UnitReader<D, kFp8> in(sh, p);
  // the unit whose tiles are loaded, and the next tile's first token
  int b = 0, q0 = 0, head0 = 0, n = 0, tok0 = 0;
  bool two = false, more = true;
  float x[kAhead + 1][kEach];
  int kind[kAhead + 1];      // 0: no tile; 1: of a unit of up to 128 keys; 2: of more
  auto load = [&](float (&y)[kEach]) -> int {
    if (more && tok0 >= n) {
      const Unit* u = in.next(false);
      more = u != nullptr;
      if (more) {
        b = u->b;
        q0 = u->q0;
        head0 = u->head * p.group;
        n = u->n;
        two = u->two();
        tok0 = u->tile0 * tt;
        in.done();
      }
    }
    if (!more) return 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      y[i] = INFINITY;      // (of a column without a row)
      if (tok[i] < tt && tok0 + tok[i] < n) y[i] = p.lse[lse_at(p, b, q0, head0 + head[i], tok0 + tok[i])];
    }
    tok0 += tt;
    return two ? 2 : 1;
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) kind[k] = load(x[k]);
  Ring<2> r;
  for (;;) {
    kind[kAhead] = load(x[kAhead]);
    if (kind[0] == 0) return;
    if (!sh.wait(sh.lse_empty(r.i), r.phase ^ 1, kSiteLseEmpty, p)) return;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sh.lse(r.i)[lane + 32 * i] = -lse_of(x[0][i]);
    __syncwarp();
    if (lane < kind[0]) mbar_arrive(sh.s_full(lane, r.i));
    r.next();
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      kind[k] = kind[k + 1];
#pragma unroll
      for (int i = 0; i < kEach; ++i) x[k][i] = x[k + 1][i];
    }
  }
}

// What keys of E4M3 pages are held times: 2^key_exp.  With a scale below 2^-110 products
// pass FP32's range where scores are ordinary, so what the scale lies below that goes to
// the keys.  All but those below 2^-110 stay exact, and what is cut off of these moves
// no score by more than 2^-100: each element by 2^-134, times queries, times 2^-109 at most.
FA_DEV int key_exp(float scale) { return min(0, (int)(__float_as_uint(scale) >> 23) - (127 - 110)); }

// E4M3 pages: eight warps make the unit's keys BF16, which holds a code times its
// power of two exactly.  Rows behind the sequence's end are left as they were: each
// is a lane of the product of its own.
template <int D>
__device__ void widen_role(const Shared<D, true>& sh, const WeighParams& p) {
  using L = Layout<D, true>;
  constexpr int kLanes = D / 16;                  // of a row
  constexpr int kRows = 32 * L::kWideners / kLanes;         // at a time
  constexpr int kUnroll = D == 128 ? 8 : 4;                 // a unit's 256
  static_assert(kRows * kUnroll == kUnitKeys, "a unit at a time");
  const int thread = threadIdx.x - 640;
  const int piece = thread % kLanes, row0 = thread / kLanes;
  const uint32_t up = (127 + 120 + key_exp(p.scale)) * 0x00800080u;      // a code's exponent (see e4m3_even_raw), twice
  Ring<2> r;
  UnitReader<D, true> in(sh, p);
  while (const Unit* w = in.next()) {
    const int keys = min(kUnitKeys, w->L - w->key0);
    uint4 x[kUnroll];
    uint32_t byte[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = row0 + k * kRows;
      x[k] = make_uint4(0u, 0u, 0u, 0u);
      byte[k] = 127u;
      const long long row = w->row[i / 16];
      if (row < 0) continue;
      x[k] = static_cast<const uint4*>(p.k_pages)[(row + i % 16) * kLanes + piece];
      byte[k] = p.k_scale[row + i % 16];
    }
    // (the codes are on their way while the products still read what was there before)
    if (!sh.wait_long(sh.k_empty(r.i), r.phase ^ 1, kSiteKEmpty, p, false)) return;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = row0 + k * kRows;
      if (i >= keys) continue;
      const uint32_t f = byte[k] == 255u ? 0x7FC07FC0u : byte[k] << 7 | byte[k] << 23;
      const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      uint32_t y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t even = paged::mul_bf16x2(paged::mul_bf16x2(paged::e4m3_even_raw(v[j]), up), f);
        const uint32_t odd = paged::mul_bf16x2(paged::mul_bf16x2(paged::e4m3_odd_raw(v[j]), up), f);
        y[2 * j] = __byte_perm(even, odd, 0x5410);
        y[2 * j + 1] = __byte_perm(even, odd, 0x7632);
      }
      const int m = i % kBM;
      uint8_t* to = sh.base + L::kK + (2 * r.i + i / kBM) * L::kTileBytes + piece / 4 * L::kChunkBytes + m * 128;
      const int c = piece % 4 * 2;
      *reinterpret_cast<uint4*>(to + ((c ^ (m & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(to + (((c + 1) ^ (m & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(sh.k_full(r.i));
    in.done();
    r.next();
  }
}

// MMA issue (a converged warp, one elected lane).  Tiles are numbered through; tile i
// takes score buffer i mod 2 of either 128 keys, which a unit with no more than 128
// leaves out for the second.
template <int D, bool kFp8>
__device__ void mma_role(const Shared<D, kFp8>& sh, const uint32_t tmem, const WeighParams& p) {
  using L = Layout<D, kFp8>;
  constexpr uint32_t kId = idesc_bf16_f32(kBM, kBN, false, false);
  Ring<2> kr;
  Ring<L::kQStages> qr;
  int j = 0;
  uint32_t phase = 0;      // bit 2 m + j: of a score buffer
  UnitReader<D, kFp8> in(sh, p);
  while (const Unit* w = in.next(false)) {
    const int tiles = all_same(w->tiles);
    const bool two = all_same((int)w->two()) != 0;
    in.done();
    if (!sh.wait(sh.k_full(kr.i), kr.phase, kSiteKFull, p)) return;
    tc_fence_after();
    for (int t = 0; t < tiles; ++t, j ^= 1) {
      if (!sh.wait(sh.q_full(qr.i), qr.phase, kSiteQFull, p)) return;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (m == 1 && !two) break;
        const int i = 2 * m + j;
        if (!sh.wait(sh.s_empty(m, j), (phase >> i & 1) ^ 1, kSiteSEmpty, p)) return;
        phase ^= 1u << i;
        tc_fence_after();
        const uint64_t da = sdesc_sw128(sh.sbase + L::kK + (2 * kr.i + m) * L::kTileBytes, 16, 1024);
        const uint64_t db = sdesc_sw128(sh.sbase + L::kQ + qr.i * L::kTileBytes, 16, 1024);
        const uint32_t d = tmem + i * 128;
        paged::mma4_ss<0>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 0u);
        if (D == 128)
          paged::mma4_ss<L::kChunkBytes / 16>(d, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kId, 1u);
        mma_commit_w(sh.s_full(m, j));
      }
      mma_commit_w(sh.q_empty(qr.i));
      qr.next();
    }
    mma_commit_w(sh.k_empty(kr.i));
    kr.next();
  }
}

// 32 lanes x 16 consecutive columns of tensor memory; the wait for them, which
// what uses them is tied to.
FA_DEV void load_scores(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
FA_DEV void scores_here(uint32_t (&r)[16]) {
  tmem_ld_wait();
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Scores of a key: their exponentials added to sum2; kMasked: those of columns [lo, hi)
// alone.
template <bool kMasked, int kCols>
FA_DEV void add_weights(const uint32_t (&x)[kCols], const float* nlse, float scale, int lo, int hi, uint64_t (&sum2)[2]) {
  const uint64_t scale2 = pk2(scale, scale), log2e2 = pk2(kLog2e, kLog2e);
#pragma unroll
  for (int i = 0; i < kCols; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(nlse + i);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // taken from the LSE before it goes to log2 units: the difference is small where
      // the weight is large, and so is its rounding
      const uint64_t s2 = pk2(__uint_as_float(x[i + 2 * h]), __uint_as_float(x[i + 2 * h + 1]));
      const uint64_t x2 = mul2(fma2(s2, scale2, h ? pk2(l.z, l.w) : pk2(l.x, l.y)), log2e2);
      float a, b;
      up2(x2, a, b);
      if (kMasked) {
        const int c = i + 2 * h;
        if (c < lo || c >= hi) a = -INFINITY;
        if (c + 1 < lo || c + 1 >= hi) b = -INFINITY;
      }
      sum2[h] = add2(sum2[h], pk2(ex2_mufu(a), ex2_mufu(b)));
    }
  }
}

// Exponentials and sums: 128 keys of each unit, a thread a key, over columns 64 j on of
// each tile.
template <int D, bool kFp8>
__device__ void sum_role(const int m, const int j, const Shared<D, kFp8>& sh, const uint32_t tmem, const WeighParams& p) {
  constexpr int kCols = 16;      // of scores in registers, twice
  const int lane = threadIdx.x % 32, wq = threadIdx.x / 32 % 4;
  const int tt = kBN / p.group;
  const int in_unit = m * kBM + wq * 32 + lane;
  const float scale = kFp8 ? p.scale * __uint_as_float((uint32_t)(127 - key_exp(p.scale)) << 23) : p.scale;
  const uint32_t tm0 = tmem + (uint32_t(wq * 32) << 16) + m * 256 + j * 64;
  uint32_t tile = 0;             // numbered through
  uint32_t phase = 0;            // bit i: of score buffer i
  UnitReader<D, kFp8> in(sh, p);
  while (const Unit* w = in.next(false)) {
    const int tiles = all_same(w->tiles);
    const bool active = m == 0 || all_same((int)w->two()) != 0;
    const int past_key = w->key0 + in_unit - w->past;      // the first token that sees the key
    const int n = w->n;
    int tok0 = w->tile0 * tt;
    uint64_t total2[2] = {0ull, 0ull};
    for (int t = 0; t < tiles; ++t, tok0 += tt, ++tile) {
      const int i = tile & 1;
      if (!active) {      // goes along with the first keys
        if (!sh.wait_long(sh.s_full(0, i), tile >> 1 & 1, kSiteSFull, p)) return;
      } else {
        const int hi = min(tt, n - tok0) * p.group - 64 * j;                             // columns with a row
        const int lo = p.causal ? max(0, past_key - tok0) * p.group - 64 * j : 0;        // first one that sees the key
        const uint32_t tm = tm0 + i * 128;
        const float* nlse = sh.lse(i) + 64 * j;
        // Columns that are no row's in any tile (the group does not divide 128) have queries
        // of zero and an LSE of infinity; in a tile that is not full they are other rows'.
        const bool seen = __all_sync(0xffffffffu, lo <= 0), plain = seen && hi >= min(64, tt * p.group - 64 * j);
        uint64_t sum2[2] = {0ull, 0ull};
        uint32_t xa[kCols], xb[kCols];
        if (!sh.wait(sh.s_full(m, i), phase >> i & 1, kSiteSFull, p)) return;
        phase ^= 1u << i;
        tc_fence_after();
        // the buffer's last columns are here
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sh.s_empty(m, i));
        };
        if (plain) {
          load_scores(tm, xa);
#pragma unroll
          for (int c = 0; c < 64; c += 2 * kCols) {
            scores_here(xa);
            load_scores(tm + c + kCols, xb);
            add_weights<false>(xa, nlse + c, scale, 0, 0, sum2);
            scores_here(xb);
            if (c + 2 * kCols < 64) load_scores(tm + c + 2 * kCols, xa); else release();
            add_weights<false>(xb, nlse + c + kCols, scale, 0, 0, sum2);
          }
        } else if (hi <= 0) {
          release();
        } else {
          load_scores(tm, xa);
#pragma unroll 1
          for (int c = 0; c < 64; c += kCols) {
            scores_here(xa);
            if (seen && c + kCols <= hi)
              add_weights<false>(xa, nlse + c, scale, 0, 0, sum2);
            else
              add_weights<true>(xa, nlse + c, scale, lo - c, hi - c, sum2);
            if (c + kCols < min(hi, 64)) {
              load_scores(tm + c + kCols, xa);
            } else {
              release();
              break;
            }
          }
        }
        total2[0] = add2(total2[0], sum2[0]);
        total2[1] = add2(total2[1], sum2[1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.lse_empty(i));
    }
    float a, b;
    up2(add2(total2[0], total2[1]), a, b);
    const int slot = in.r.i;
    if (j == 1) {
      sh.unit(slot)->part[in_unit] = a + b;
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.part_full(slot, m));
    } else {
      if (!sh.wait_long(sh.part_full(slot, m), in.r.phase, kSitePart, p, false)) return;
      const long long row = w->row[in_unit / 16];
      if (row >= 0 && w->key0 + in_unit < w->L)
        p.sums[row + in_unit % 16] =
            fmaf(p.decay, p.decay != 0.0f && past_key < 0 ? w->old[in_unit] : 0.0f, a + b + w->part[in_unit]);
    }
    in.done();
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
      mbar_init(sh.k_full(i), kFp8 ? L::kWideners : 1);      // one arrival per widening warp
      mbar_init(sh.k_empty(i), 1);
      for (int m = 0; m < 2; ++m) {
        mbar_init(sh.s_full(m, i), 2);
        mbar_init(sh.s_empty(m, i), 8);
      }
    }
    for (int i = 0; i < L::kQStages; ++i) {
      mbar_init(sh.q_full(i), 1);
      mbar_init(sh.q_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(sh.lse_empty(i), 16);
    if (p.held >= 0) hold(sh.bar(p.held));
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(sh.unit_full(i), 1);
      mbar_init(sh.unit_empty(i), L::kReaders);
      mbar_init(sh.part_full(i, 0), 4);
      mbar_init(sh.part_full(i, 1), 4);
    }
    st_shared(sh.abort(), 0);
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    if (!kFp8) tma_prefetch_desc(&tm_k);
  }
  // rows of Q's tiles that no box fills
  const int rows = kBN / p.group * p.group;
  for (int i = threadIdx.x; i < (kBN - rows) * 8 * L::kChunks * L::kQStages; i += L::kThreads) {
    const int chunk = i / ((kBN - rows) * 8), at = i - chunk * (kBN - rows) * 8;
    *reinterpret_cast<uint4*>(smem + L::kQ + chunk * L::kChunkBytes + rows * 128 + at * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == 17) {
    tmem_alloc(sh.tmem_slot(), 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");      // nothing global before this
  const bool ok = paged::prefix_sequences(
      p.s, p.max_q,
      [&](const paged::SeqRows& r) { return paged::Work{(long long)p.s.Hkv * units_of(r.L), 0, 0}; },
      reinterpret_cast<long long*>(smem + L::kPre), nullptr, reinterpret_cast<long long*>(smem + L::kSums));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!ok && blockIdx.x == 0 && threadIdx.x == 0) paged::record_bad_input(&g_err, kSiteSeqs);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sh.tmem_slot();
  const long long units = ok ? sh.pre()[p.s.B] : 0;

  if (warp < 16) {
    sum_role<D, kFp8>(warp / 8, warp / 4 % 2, sh, tmem, p);
  } else if (warp == 16) {
    load_role<D, kFp8>(sh, &tm_q, &tm_k, p);
  } else if (warp == 17) {
    mma_role<D, kFp8>(sh, tmem, p);
  } else if (warp == 18) {
    lse_role<D, kFp8>(sh, p);
  } else if (warp == 19) {
    unit_role<D, kFp8>(sh, p, units);
  } else {
    if constexpr (kFp8) widen_role<D>(sh, p);
  }

  // after a give-up, copies and MMAs in flight land before the memory they target is
  // released
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
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
  return launch_overlapped(kernel, dim3(num_sms), L::kThreads, L::kBytes, stream, tq, tk, p);
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

int weigh_barriers(int D) {
  return D == 128 ? weigh::Layout<128, false>::kTileBars : weigh::Layout<64, false>::kTileBars;
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
