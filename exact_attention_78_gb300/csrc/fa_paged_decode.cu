// Attention of a few new tokens over a paged cache (a decoding step).
//
//   O = softmax(scale q K^T [+ causal or tree mask]) V, LSE, per row of q.
//
// A step reads every sequence's keys and values once and computes little with
// them, so HBM bounds it: the design keeps loads in flight and splits the keys
// evenly over the SMs.
//
//   * Rows.  The query heads of one key/value head, for up to 16 rows (32 at
//     D = 64) of (new token, head of the group), share the keys that a warp
//     loads.  They are the N side of the products, 8 rows an mma.sync tile, and
//     keys (for S^T = K Q^T) and columns of V (for O^T = V^T P^T) the M side:
//     with 8 rows or fewer, the usual case, that halves the products and the
//     softmax against rows on the M side, whose tiles are 16 high.  (tcgen05
//     tiles have at least 64 rows on M and their accumulators are a trip through
//     tensor memory away; with so few rows the warp-level instruction leaves
//     the tensor cores 8 to 14% busy.)
//   * Work.  The key blocks of all (sequence, key/value head) units, and a
//     constant for each unit's start and end, form one line, and thread block c
//     takes the c-th of `grid` equal stretches of it.  A unit cut by a border
//     leaves partial results in the workspace, at most two per thread block, and
//     the combine kernel joins them.  Sequences of any mixture of lengths load all
//     SMs alike.
//   * Pipeline.  One warp looks up the pages of the stretch's blocks, 32 at a
//     time and on into the next units.  The other warps take the blocks in turn
//     and each refills by TMA the slots of the ring in shared memory that it
//     empties (the pages' rows, swizzled for ldmatrix), every lane with a load of
//     its own: a single thread issues one in some 150 cycles, too slow to feed an
//     SM alone (313 us for 64 x 4096 BF16 keys).  At a unit's end they leave
//     their softmax states in shared memory and go on; the warp that looks pages
//     up merges them in between.
//   * E4M3 pages are widened in registers on the way to the tensor cores, to
//     FP16, which holds every code and which one instruction makes of a pair (to
//     BF16 it takes five).  The queries become FP16 by a power of two of each
//     row's own, which loses nothing of note: a row's largest value is below 2^14
//     then, and what lies below 2^-30 of it is rounded, by 2^-38 of it at most.
//     The keys' scales go to the scores in FP32, the values' to the weights.
//   * The launch overlaps the end of the kernel before it in the stream: barriers
//     are set up before griddepcontrol.wait (a call over a few keys, behind another:
//     13.3 -> 11.0 us on the GPU).
//   * The running maximum is lazy: it moves, and the sums and O are rescaled,
//     only when a row's scores pass it by more than 8 log2 units.
#include <cuda_runtime.h>

#include "paged.cuh"
#include "softmax_math.cuh"

namespace fa {
namespace pdec {

__device__ DeviceError g_err;

constexpr float kThreshold = 8.0f;   // lazy rescaling, log2 units
// E4M3: weights are taken times 2^6 to FP16.  With the threshold they stay
// below 2^14, and keep FP16's full precision down to 2^-20 of the maximum.
constexpr int kWeightUp = 6;

enum Site { kSiteSeqs = 1, kSitePage, kSiteFull, kSitePlaced, kSiteTaken, kSiteMerged };

// Layout of the workspace: per slot the rows' unnormalised outputs, then per
// slot and row the maximum (log2 units) and the two sums.
template <int D, int kRows>
struct Part {
  static constexpr int kSlotFloats = kRows * D;
  static constexpr int kStat = 4;
  FA_DEV static float* out(float* ws, int slot) { return ws + (size_t)slot * kSlotFloats; }
  FA_DEV static float* stat(float* ws, int slot) {
    return ws + (size_t)2 * kMaxCtas * kSlotFloats + (size_t)slot * kRows * kStat;
  }
  FA_DEV static paged::Join* join(float* ws, int c) {
    return reinterpret_cast<paged::Join*>(stat(ws, 2 * kMaxCtas)) + c;
  }
  static constexpr size_t bytes() {
    return (size_t)2 * kMaxCtas * (kSlotFloats + kRows * kStat) * sizeof(float) + kMaxCtas * sizeof(paged::Join);
  }
};

// kTiles: tiles of 8 rows.  11 computing warps with up to 168 registers hide
// more latency than 7; with more than one tile they would spill.
template <int D, bool kFp8, int kTiles>
struct Layout {
  static constexpr int kWarps = kTiles == 1 ? 11 : 7;       // with the looking-up one, a multiple of 4
  static constexpr int kThreads = (kWarps + 1) * 32;         // and the warp that looks up pages
  static constexpr int kRows = 8 * kTiles;
  // Keys of a block, at most two pages: stages of 8 KB of keys and values (4 KB
  // for E4M3 at D = 64) keep enough bytes in flight with few stages.
  static constexpr int kKeys = D == 128 && !kFp8 ? 16 : 32;
  static constexpr int kTile = kKeys * D * (kFp8 ? 1 : 2);        // keys or values of a block
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRingBytes = 184320;
  static constexpr int kSlots = kRingBytes / (kWarps * kStage) * kWarps;   // of the ring; warp w takes those = w mod kWarps
  static constexpr int kBatches = 4;                              // of 32 looked-up blocks
  static constexpr int kPitch = D + 4;                            // floats of a merge row
  static constexpr int kRound = kTiles == 1 ? 4 : 8;              // rows that are merged at a time
  static constexpr int kMergeFloats = kWarps * kRound * kPitch;   // a round's outputs of all warps
  static constexpr int kRing = 0;
  static constexpr int kScales = kRing + kSlots * kStage;   // E4M3: scale bytes of a stage's keys, values
  static constexpr int kFactors = kScales + (kFp8 ? kSlots * 2 * kKeys : 0);   // a block's, as floats
  static constexpr int kMerge = kFactors + (kFp8 ? kWarps * 2 * kKeys * 4 : 0);
  static constexpr int kStats = kMerge + kMergeFloats * 4;        // m, l, lr of [row in round][warp]
  static constexpr int kPre = (kStats + 3 * kWarps * kRound * 4 + 7) / 8 * 8;   // prefix of blocks, [B + 1]
  static constexpr int kBars = kPre + (kMaxPackedSeqs + 1) * 8 + 8;
  static constexpr int kPlaces = (kBars + kSlots * 8 + 2 * kBatches * 8 + 16 + 15) / 16 * 16;   // where blocks lie
  static constexpr int kMisc = kPlaces + kBatches * 32 * 16;
  static constexpr int kBytes = kMisc + 64 + kSmemAlignSlack;
  static_assert(kBytes <= 232448, "dynamic shared memory above the 227 KB per-CTA limit");
  // places are looked up to 64 behind the last block, and asked for up to kSlots
  static_assert(kSlots <= 64, "slots whose places nobody looks up");
};

// ------------------------------------------------------------ the work line --

using Seq = paged::SeqRows;
FA_DEV Seq seq_of(const PagedSeqs& s, int b) { return paged::rows_of(s, b); }
// Blocks of a unit: at least one, so that rows without a key are written too.
FA_DEV int blocks_of(int L, int keys) { return max(1, (L + keys - 1) / keys); }
// What a unit takes on the line besides its blocks: starting and merging it.  (64
// ragged sequences up to 8192 E4M3 keys, 8 heads: counted as nothing, 111 us, since
// a stretch of short sequences has up to 16 units, the average 4; as 14 blocks 99,
// 20 100.)
constexpr int kUnitCost = 14;

// Prefix sums of the sequences' blocks into pre[0 .. B]; returns their total,
// 0 when the sequences break the rules.  All threads of the block.
template <int kKeys>
FA_DEV long long build_line(const PagedAttnParams& p, long long* pre, long long* warp_sums) {
  const bool ok = paged::prefix_sequences(
      p.s, p.max_q,
      [&](const Seq& q) { return paged::Work{(long long)p.s.Hkv * (blocks_of(q.L, kKeys) + kUnitCost), 0, 0}; },
      pre, nullptr, warp_sums);
  if (ok) return pre[p.s.B];
  if (blockIdx.x == 0 && threadIdx.x == 0) paged::record_bad_input(&g_err, kSiteSeqs);
  return 0;
}

// Thread blocks that share the line: no more than leave each 8 key blocks.
FA_DEV int active_ctas(long long total, int ctas) {
  const long long most = (total + 7) / 8;
  return most < ctas ? (int)most : ctas;
}
// First block of stretch c of G.
FA_DEV long long stretch(long long total, int c, int G) { return paged::div64(total * c, G); }

// A walk over the segments (the stretch's share of one unit) of [t0, t1).  A
// border behind a unit's blocks, in what starting and merging it counts, leaves
// the unit whole.
template <int kKeys>
struct Walk {
  int b, head;
  Seq s;
  int nblk;          // blocks of the unit
  int kb, count;     // the segment: blocks [kb, kb + count)
  long long start;   // the unit's first place on the line
  long long t1;

  FA_DEV void load(const PagedAttnParams& p) {
    s = seq_of(p.s, b);
    nblk = blocks_of(s.L, kKeys);
  }
  FA_DEV void begin(const PagedAttnParams& p, const long long* pre, long long t0, long long end) {
    int lo = 0, hi = p.s.B - 1;      // last b with pre[b] <= t0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= t0) lo = mid; else hi = mid - 1;
    }
    b = lo;
    t1 = end;
    load(p);
    const long long r = t0 - pre[b];
    const long long unit = paged::div64(r, nblk + kUnitCost);
    kb = (int)(r - unit * (nblk + kUnitCost));
    start = t0 - kb;
    head = (int)unit;
    cut();
    if (kb >= nblk) next(p);
  }
  FA_DEV void cut() { count = (int)min((long long)(nblk - kb), t1 - start - kb); }
  FA_DEV bool more() const { return start + kb < t1; }
  FA_DEV void next(const PagedAttnParams& p) {
    start += nblk + kUnitCost;
    kb = 0;
    if (start >= t1) return;
    if (++head == p.s.Hkv) {
      head = 0;
      do ++b; while (b < p.s.B - 1 && seq_of(p.s, b).n == 0);
      load(p);
    }
    cut();
  }
  // Rows (token, head of the group) of the unit.
  FA_DEV int rows(const PagedAttnParams& p) const { return s.n * p.group; }
  // Blocks of the segment with keys, all of which the last token sees.
  FA_DEV int visible() const { return min(count, max(0, (s.L + kKeys - 1) / kKeys - kb)); }
};

// ----------------------------------------------------------- instructions --

FA_DEV void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
FA_DEV void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
FA_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

FA_DEV void mma16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Transposes an 8 x 8 matrix of 16-bit values over the warp: lane 4 r + c holds
// row r, columns 2 c and 2 c + 1.
FA_DEV uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Shared-memory address of 16-byte piece `c` of row `r` of a tile at `base`.
// BF16: 64-column chunks of 128-byte rows, 128-byte swizzle.  E4M3: rows of D
// bytes, swizzled by their width.
template <int D, bool kFp8, int kKeys>
FA_DEV uint32_t piece(uint32_t base, int r, int c) {
  if (!kFp8) return base + (c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  if (D == 128) return base + r * 128 + ((c ^ (r & 7)) << 4);
  return base + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// ---------------------------------------------------------------- kernel --

// Whether a phase is complete, without waiting; one answer for the whole warp.
FA_DEV bool test_warp(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, done != 0);
}

// Joins the states that the computing warps left of rows [r0, r0 + kRound) of a
// segment: final when it is the whole unit, else into the workspace.  One warp.
template <int D, bool kFp8, int kTiles>
FA_DEV void merge_rows(const PagedAttnParams& p, const Walk<Layout<D, kFp8, kTiles>::kKeys>& at, int r0,
                       const float* buf, float* stats) {
  using L = Layout<D, kFp8, kTiles>;
  using W = Part<D, L::kRows>;
  constexpr int kWarps = L::kWarps;
  const int lane = threadIdx.x % 32;
  const int rows = min(L::kRound, at.rows(p) - r0);
  const bool whole = at.kb == 0 && at.count == at.nblk;
  // a stretch begins in a cut unit at most once, and ends in one at most once
  const int slot = 2 * blockIdx.x + (at.kb > 0 ? 0 : 1);
  float* st_m = stats;
  const float* st_l = st_m + kWarps * L::kRound;
  float* st_lr = stats + 2 * kWarps * L::kRound;
  if (lane < rows) {
    float f[kWarps], mt = -INFINITY, lt = 0.0f, lrt = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = st_m[lane * kWarps + w];
      mt = fmaxf(mt, f[w]);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = mt == -INFINITY ? 1.0f : ex2_mufu(f[w] - mt);
      lt += st_l[lane * kWarps + w] * f[w];
      lrt += st_lr[lane * kWarps + w] * f[w];
    }
    const float inv = !whole ? 1.0f : lrt == 0.0f ? 0.0f : 1.0f / lrt;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) st_m[lane * kWarps + w] = f[w] * inv;       // from here on the warps' factors
    st_lr[lane * kWarps] = lt;                                                   // and the row's sum
    if (whole) {
      const int row = r0 + lane, t = row / p.group, head = at.head * p.group + row - t * p.group;
      const size_t li = p.s.cu ? (size_t)head * p.s.Sn + at.s.q0 + t : ((size_t)at.b * p.Hq + head) * p.s.Sn + t;
      p.lse[li] = lt == 0.0f ? -INFINITY : (mt + log2f(lt)) * 0.693147180559945309f;
    } else {
      *reinterpret_cast<float4*>(W::stat(p.part, slot) + (r0 + lane) * W::kStat) = make_float4(mt, lt, lrt, 0.0f);
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < rows * (D / 4); i += 32) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(buf + (w * L::kRound + r) * L::kPitch + d);
      const float f = st_m[r * kWarps + w];
      y.x += x.x * f;
      y.y += x.y * f;
      y.z += x.z * f;
      y.w += x.w * f;
    }
    // a row that sees none of the keys is zero, whatever their values made of its zeros
    if (st_lr[r * kWarps] == 0.0f) y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (whole) {
      const int row = r0 + r, t = row / p.group, head = at.head * p.group + row - t * p.group;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + ((size_t)(at.s.q0 + t) * p.Hq + head) * D + d) =
          make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    } else {
      *reinterpret_cast<float4*>(W::out(p.part, slot) + (r0 + r) * D + d) = y;
    }
  }
}

// kTree: the new tokens are drafted ones, each of which sees the keys before them and
// those of them that its mask names.  A mask is one word: a sequence has no more
// than 32 rows here.
template <int D, bool kFp8, int kTiles, bool kTree>
__global__ void __launch_bounds__(Layout<D, kFp8, kTiles>::kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const PagedAttnParams p) {
  using L = Layout<D, kFp8, kTiles>;
  using W = Part<D, L::kRows>;
  constexpr int kWarps = L::kWarps;
  constexpr int kKeys = L::kKeys;
  constexpr int kGroups = kKeys / 16;
  constexpr int kSteps = D / 16;      // 16-wide steps along D
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int c = lane % 4, g = lane / 4;       // column pair and row of the fragments
  long long* pre = reinterpret_cast<long long*>(smem + L::kPre);
  float* merge = reinterpret_cast<float*>(smem + L::kMerge);
  float* stats = reinterpret_cast<float*>(smem + L::kStats);
  const uint32_t abort = sbase + L::kMisc;
  // barriers: a slot is loaded; a batch of places is looked up, is used up; the
  // merge rows are written, are free
  const uint32_t full = sbase + L::kBars, placed = full + 8 * L::kSlots, taken = placed + 8 * L::kBatches;
  const uint32_t written = taken + 8 * L::kBatches, merged = written + 8;
  int4* places = reinterpret_cast<int4*>(smem + L::kPlaces);

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kSlots + L::kBatches; ++i) mbar_init(full + 8 * i, 1);
    for (int i = 0; i < L::kBatches; ++i) mbar_init(taken + 8 * i, 32);
    mbar_init(written, kWarps);
    mbar_init(merged, 1);
    st_shared(abort, 0);
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");      // nothing global before this
  const long long total = build_line<kKeys>(p, pre, reinterpret_cast<long long*>(merge));
  __syncthreads();
  const int G = active_ctas(total, gridDim.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if ((int)blockIdx.x >= G) {
    if (threadIdx.x == 0) W::join(p.part, blockIdx.x)->parts = 0;
    return;
  }
  const long long t0 = stretch(total, blockIdx.x, G), t1 = stretch(total, blockIdx.x + 1, G);

  // The stretch's visible blocks are numbered through; block q goes through ring
  // slot q mod kSlots.
  Walk<kKeys> at;
  at.begin(p, pre, t0, t1);

  const int box_shift = min(p.s.page_shift, kKeys == 32 ? 5 : 4);    // rows of a box
  const int two = kKeys >> box_shift == 2;                            // two boxes a block, else one
  constexpr int kEnd = -2;                                             // in place of a page: no more blocks

  if (warp == kWarps) {
    // ---- says what there is to join at the border before this stretch
    if (lane == 0) {
      const int c = blockIdx.x;
      paged::Join j{0, at.b, at.head, 0, at.s.n, at.s.q0, {0, 0}};
      if (at.kb > 0 && stretch(total, c - 1, G) <= at.start) {       // the unit's first cut
        j.parts = 2;
        while (c + j.parts - 1 < G && stretch(total, c + j.parts - 1, G) < at.start + at.nblk) ++j.parts;
      }
      *W::join(p.part, c) = j;
    }
    // ---- looks up where blocks lie, (page, head) and row of the block's boxes,
    // and merges the states that the other warps leave at a unit's end, whichever
    // can be done
    Walk<kKeys> mine = at;
    int r0 = 0;                        // of the rows to merge next
    uint32_t round = 0, batch = 0;
    int i = 0, vis = at.visible(), past = 0;
    bool have = false;                 // a batch that waits for its place
    int4 place;
    uint64_t idle = 0;                 // since when nothing could be done
    for (uint32_t it = 1;; ++it) {
      bool did = false;
      if (past < 2 || have) {          // until a whole batch lies behind the end
        if (!have) {
          place = make_int4(kEnd, kEnd, 0, 0);
          if (!at.more()) ++past;
          for (int filled = 0; filled < 32 && at.more();) {
            const int take = min(32 - filled, vis - i);
            if (lane >= filled && lane < filled + take) {
              int ph[2] = {-1, -1}, off[2] = {0, 0};      // -1: outside the tensor maps, reads as zeros
              for (int j = 0; j <= two; ++j) {
                const int key = (at.kb + i + lane - filled) * kKeys + (j << box_shift);
                if (key >= at.s.L) break;
                const int page = p.s.block_table[(size_t)at.b * p.s.max_pages + (key >> p.s.page_shift)];
                if (page < 0 || page >= p.s.num_pages)
                  paged::record_bad_input(&g_err, kSitePage);
                else
                  ph[j] = page * p.s.Hkv + at.head;
                off[j] = key & ((1 << p.s.page_shift) - 1);
              }
              place = make_int4(ph[0], ph[1], off[0], off[1]);
            }
            filled += take;
            i += take;
            if (i == vis) {
              at.next(p);
              i = 0;
              vis = at.more() ? at.visible() : 0;
            }
          }
          have = true;
        }
        const int b = batch % L::kBatches;
        if (test_warp(taken + 8 * b, (batch / L::kBatches & 1) ^ 1)) {
          places[b * 32 + lane] = place;
          __syncwarp();
          if (lane == 0) mbar_arrive(placed + 8 * b);
          ++batch;
          have = false;
          did = true;
        }
      }
      if (mine.more()) {
        if (test_warp(written, round & 1)) {
          merge_rows<D, kFp8, kTiles>(p, mine, r0, merge, stats);
          __syncwarp();
          if (lane == 0) mbar_arrive(merged);
          ++round;
          r0 += L::kRound;
          if (r0 >= mine.rows(p)) {
            r0 = 0;
            mine.next(p);
          }
          did = true;
        }
      } else if (past == 2 && !have) {
        break;
      }
      if (did) {
        idle = 0;
        continue;
      }
      __nanosleep(40);
      if ((it & 15u) == 0u) {
        const uint64_t now = globaltimer_ns();
        if (idle == 0) idle = now;
        const bool late = now - idle > p.wait_limit_ns;
        if (__any_sync(0xffffffffu, late)) {
          if (lane == 0) {
            if (atomicCAS(&g_err.status, 0, FA_ERR_TIMEOUT) == 0) atomicExch(&g_err.site, kSiteTaken);
            st_shared(abort, 1);
          }
          break;
        }
        if (__any_sync(0xffffffffu, ld_shared_volatile(abort) != 0)) break;
      }
    }
    return;
  }

  // Loads block q into its slot.  The whole warp calls it.
  auto load = [&](uint32_t q) {
    const int b = q / 32 % L::kBatches;
    if (!paged::wait_warp(placed + 8 * b, q / (32 * L::kBatches) & 1, abort, &g_err, kSitePlaced, p.wait_limit_ns)) return;
    const int4 place = places[q % (32 * L::kBatches)];
    __syncwarp();
    if (lane == 0) mbar_arrive(taken + 8 * b);
    if (place.x == kEnd) return;
    const uint32_t slot = q % L::kSlots, bar = full + 8 * slot;
    if (lane == 0) mbar_arrive_expect_tx(bar, 2 * L::kTile + (kFp8 ? 2 * kKeys : 0));
    __syncwarp();
    // each lane issues its own load: keys or values, 64-column chunk, box
    constexpr int kParts = kFp8 ? 2 : D / 32;
    const int j = lane / kParts, which = lane & 1, h = lane % kParts / 2;
    if (j <= two) {
      const int ph = j ? place.y : place.x, off = j ? place.w : place.z;
      tma_load_3d(sbase + L::kRing + slot * L::kStage + which * L::kTile + h * kKeys * 128 +
                      (j << box_shift) * (kFp8 ? D : 128),
                  which ? &tm_v : &tm_k, bar, h * 64, off, ph);
      if (kFp8)
        bulk_load(sbase + L::kScales + slot * 2 * kKeys + which * kKeys + (j << box_shift),
                  ph < 0 ? paged::g_no_scales : (which ? p.v_scale : p.k_scale) + ((size_t)ph << p.s.page_shift) + off,
                  1 << box_shift, bar);
    }
    __syncwarp();
  };
#pragma unroll 1
  for (int q = warp; q < L::kSlots; q += kWarps) load(q);

  // Q of a segment as B fragments: row 8 n + g in tile n, d = 16 s + 2 c,
  // + 1 and + 8, + 9.  E4M3: four consecutive values at 16 s + 4 c instead, which
  // is how a word of four codes of a key lies in its fragment.
  uint32_t qf[kTiles][kSteps][2];
  const float inv_group = 1.0f / (float)p.group;
  // token of a row: exact for the small numbers here.  Where registers are shortest it
  // is worked out for each unit anew (64 x 4096 E4M3 keys, 32 rows at D = 64: 145 us
  // with the tokens kept, 143 so; BF16 124 and 126).
  auto token_of = [&](int row) {
    if (kFp8 && kTiles == 4) asm volatile("" : "+r"(row));
    return (int)(((float)row + 0.5f) * inv_group);
  };
  auto load_q = [&](const Walk<kKeys>& w) {
    const int rows = w.rows(p);
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int r = 8 * n + g;
      const bool valid = r < rows;
      const int t = token_of(r), j = r - t * p.group;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
                                 ((size_t)(w.s.q0 + t) * p.Hq + w.head * p.group + j) * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint2 x = make_uint2(0u, 0u);
        if (valid) {
          if (kFp8) {
            x = *reinterpret_cast<const uint2*>(src + 16 * s + 4 * c);
          } else {
            x.x = *reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * c);
            x.y = *reinterpret_cast<const uint32_t*>(src + 16 * s + 8 + 2 * c);
          }
        }
        qf[n][s][0] = x.x;
        qf[n][s][1] = x.y;
      }
    }
  };
  load_q(at);

  // E4M3: a row of Q is taken times 2^(13 - e), and its scores times 2^(e - 13)
  // and the scale.  e is -113 at least, where every BF16 number is exact in FP16,
  // and large enough to keep that product normal: a small scale leaves fewer bits to
  // rows of small queries, which moves no score by more than 2^-15.
  const int least_exp = 14 + max(0, 127 - (int)(__float_as_uint(p.scale_log2) >> 23));
  uint32_t q0 = 0;        // number of the segment's first block
  uint32_t round = 0;     // of merging
  bool lost = false;      // a wait ran out: no more results
  while (at.more()) {
    const int rows = at.rows(p);
    const int vis = at.visible();
    // rows 8 n + 2 c + e, whose scores this lane gets:
    int row_lim[kTiles][2];          // keys that they see (a tree's: the keys before it)
    uint32_t row_bits[kTiles][2];    // and of the tree
    float row_scale[kTiles][2];      // what their scores are multiplied by, for log2 units
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      float scale = p.scale_log2;
      if (kFp8) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) top = max(top, max(qf[n][s][k] & 0x7FFFu, (qf[n][s][k] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max((int)(top >> 7), least_exp) - 127;     // of the largest value
        const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);     // e <= 128
        scale *= __uint_as_float((uint32_t)(127 - 13 + e) << 23);            // normal
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w = qf[n][s][k];
            qf[n][s][k] = pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row_scale[n][e] = kFp8 ? __shfl_sync(0xffffffffu, scale, (2 * c + e) * 4) : scale;
        const int row = 8 * n + 2 * c + e;
        if (kTree) {
          const int past = at.s.L - at.s.n, t = token_of(row);
          row_lim[n][e] = past;
          row_bits[n][e] = row >= rows || past + t < 0 ? 0u : paged::tree_bits(p.tree + at.s.q0 + t, 0, at.s.n);
        } else {
          row_lim[n][e] = row >= rows ? 0 : p.causal ? at.s.L - at.s.n + token_of(row) + 1 : at.s.L;
        }
      }
    }
    // O^T: columns of V on the rows, rows of Q on the columns (2 c, 2 c + 1 here)
    float acc[kTiles][kSteps][4];
    float m[kTiles][2], l[kTiles][2];
    float ones[kTiles][4];      // BF16: sums of the weights as the product takes them
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ones[n][e] = 0.0f;
#pragma unroll
        for (int d = 0; d < kSteps; ++d) acc[n][d][e] = 0.0f;
      }
    }
    int v_top = 0;      // E4M3: the largest scale byte of a value so far; acc counts in 2^(v_top - 127 - kWeightUp)

#pragma unroll 1
    for (int i = (warp + kWarps - q0 % kWarps) % kWarps; i < vis && !lost; i += kWarps) {
      const uint32_t slot = (q0 + i) % L::kSlots;
      if (!paged::wait_warp(full + 8 * slot, (q0 + i) / L::kSlots & 1, abort, &g_err, kSiteFull, p.wait_limit_ns)) {
        lost = true;
        break;
      }
      const uint32_t kt = sbase + L::kRing + slot * L::kStage, vt = kt + L::kTile;
      const int key0 = (at.kb + i) * kKeys;
      float2* factor = reinterpret_cast<float2*>(smem + L::kFactors) + warp * kKeys;     // of a key and its value
      if (kFp8) {
        // lane i: the factors of key i.  Values' scales are taken relative to
        // the largest so far.
        const uint8_t* bytes = smem + L::kScales + slot * 2 * kKeys;
        const bool mine = key0 + lane < at.s.L;          // behind the end: anything
        const uint32_t kb = bytes[lane], vb = mine ? bytes[kKeys + lane] : 0u;
        const int block_top = __reduce_max_sync(0xffffffffu, vb == 255u ? 0u : vb);
        if (block_top > v_top) {
          if (v_top > 0) {
            const float f = __uint_as_float((uint32_t)max(v_top - block_top + 127, 0) << 23);
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
              for (int d = 0; d < kSteps; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][d][e] *= f;
          }
          v_top = block_top;
        }
        factor[lane] = make_float2(paged::scale_value(kb),
                                   vb == 255u ? __int_as_float(0x7FC00000)
                                              : __uint_as_float((uint32_t)max((int)vb - v_top + kWeightUp + 127, 0) << 23));
        __syncwarp();
      }
      // S^T of 16-key groups: s[n][j][2 h + e] is key 16 j + g + 8 h, row 8 n + 2 c + e
      float s[kTiles][kGroups][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int j = 0; j < kGroups; ++j) s[n][j][0] = s[n][j][1] = s[n][j][2] = s[n][j][3] = 0.0f;
#pragma unroll
      for (int st = 0; st < kSteps; st += kFp8 ? 2 : 1)
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          uint32_t b[4];
          if (!kFp8) {
            // keys 0-7, 8-15 of the group at piece 2 st, then at 2 st + 1
            ldsm4(piece<D, kFp8, kKeys>(kt, 16 * j + (lane & 15), 2 * st + (lane >> 4)), b);
#pragma unroll
            for (int n = 0; n < kTiles; ++n) mma16816(s[n][j], b, qf[n][st][0], qf[n][st][1]);
          } else {
            // keys 0-7, 8-15 of the group at piece st, then at st + 1
            ldsm4(piece<D, kFp8, kKeys>(kt, 16 * j + (lane & 15), st + (lane >> 4)), b);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {e4m3_f16x2(b[2 * k]), e4m3_f16x2(b[2 * k + 1]), e4m3_f16x2(b[2 * k] >> 16),
                                     e4m3_f16x2(b[2 * k + 1] >> 16)};
#pragma unroll
              for (int n = 0; n < kTiles; ++n) mma16816_f16(s[n][j], a, qf[n][st + k][0], qf[n][st + k][1]);
            }
          }
        }
      float2 fac[kGroups][2];
#pragma unroll
      for (int j = 0; j < kGroups; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) fac[j][h] = kFp8 ? factor[16 * j + 8 * h + g] : make_float2(1.0f, 1.0f);
      // Behind the sequence's end values may be NaN or infinite, which a weight
      // of zero would not cancel: they are cleared below.
      const int n_left = at.s.L - key0;
      const bool ragged = n_left < kKeys;
      // a block that the first token sees whole needs no mask
      const bool masked = key0 + kKeys > (kTree ? at.s.L - at.s.n : p.causal ? at.s.L - at.s.n + 1 : at.s.L);
      uint32_t pb[kTiles][kGroups][2];        // P^T as B fragments
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = s[n][j][e] * row_scale[n][e & 1];
            if (kFp8) x *= fac[j][e >> 1].x;
            const int behind = key0 + 16 * j + 8 * (e >> 1) + g - row_lim[n][e & 1];
            if (masked && behind >= 0 && !(kTree && behind < 32 && (row_bits[n][e & 1] >> behind & 1))) x = -INFINITY;
            s[n][j][e] = x;
          }
          mx[0] = max3(mx[0], s[n][j][0], s[n][j][2]);
          mx[1] = max3(mx[1], s[n][j][1], s[n][j][3]);
        }
        if (__any_sync(0xffffffffu, mx[0] > m[n][0] + kThreshold || mx[1] > m[n][1] + kThreshold)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d *= 2) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], d));
            const float top = fmaxf(m[n][e], mx[e]);
            const float f = top == -INFINITY ? 1.0f : ex2_mufu(m[n][e] - top);      // 0 from a maximum of -inf
            m[n][e] = top;
            l[n][e] *= f;
            ones[n][e] *= f;
#pragma unroll
            for (int d = 0; d < kSteps; ++d) {
              acc[n][d][e] *= f;
              acc[n][d][2 + e] *= f;
            }
          }
        }
        const float use[2] = {m[n][0] == -INFINITY ? 0.0f : m[n][0], m[n][1] == -INFINITY ? 0.0f : m[n][1]};
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float e0 = ex2_mufu(s[n][j][2 * h] - use[0]), e1 = ex2_mufu(s[n][j][2 * h + 1] - use[1]);
            l[n][0] += e0;
            l[n][1] += e1;
            pb[n][j][h] = transpose8x8(kFp8 ? pack_f16x2(e0 * fac[j][h].y, e1 * fac[j][h].y) : pack_bf16x2(e0, e1));
          }
      }
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};      // keys 2 c, 2 c + 1 and 2 c + 8, 2 c + 9
        if (ragged) {
          const int k = n_left - 16 * j - 2 * c;
          keep[0] = (k > 0 ? 0x0000FFFFu : 0u) | (k > 1 ? 0xFFFF0000u : 0u);
          keep[1] = (k > 8 ? 0x0000FFFFu : 0u) | (k > 9 ? 0xFFFF0000u : 0u);
        }
        if (!kFp8) {
          // the weights' sum as they are rounded, for the division, so that the
          // weights used add up to one: a product with ones
          const uint32_t one[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
          for (int n = 0; n < kTiles; ++n) mma16816(ones[n], one, pb[n][j][0], pb[n][j][1]);
#pragma unroll
          for (int d = 0; d < kSteps; ++d) {
            // keys 0-7 at pieces 2 d and 2 d + 1, then keys 8-15
            uint32_t b[4];
            ldsm4_t(piece<D, kFp8, kKeys>(vt, 16 * j + (lane & 7) + (lane >> 4) * 8, 2 * d + ((lane >> 3) & 1)), b);
            if (ragged) {
#pragma unroll
              for (int e = 0; e < 4; ++e) b[e] &= keep[e >> 1];
            }
#pragma unroll
            for (int n = 0; n < kTiles; ++n) mma16816(acc[n][d], b, pb[n][j][0], pb[n][j][1]);
          }
        } else {
          // a word holds D columns 2 g and 2 g + 1 of two keys: the even bytes
          // are row g of the tile, the odd bytes row g + 8
#pragma unroll
          for (int d = 0; d < kSteps; d += 2) {
            // keys 0-7, 8-15 at piece d, then at d + 1
            uint32_t b[4];
            ldsm4_t(piece<D, kFp8, kKeys>(vt, 16 * j + (lane & 15), d + (lane >> 4)), b);
            if (ragged) {
#pragma unroll
              for (int e = 0; e < 4; ++e) b[e] &= keep[e & 1];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = __byte_perm(b[e], 0u, 0x3120);     // even bytes, odd bytes
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {e4m3_f16x2(b[2 * k]), e4m3_f16x2(b[2 * k] >> 16), e4m3_f16x2(b[2 * k + 1]),
                                     e4m3_f16x2(b[2 * k + 1] >> 16)};
#pragma unroll
              for (int n = 0; n < kTiles; ++n) mma16816_f16(acc[n][d + k], a, pb[n][j][0], pb[n][j][1]);
            }
          }
        }
      }
      __syncwarp();       // every lane is done with the slot
      load(q0 + i + L::kSlots);
    }
    q0 += vis;

    // the next segment's queries come while this one is finished
    Walk<kKeys> after = at;
    after.next(p);
    if (after.more()) load_q(after);
    // Long units end together: warps that drift apart refill the ring out of turn.
    // (64 ragged E4M3 sequences up to 8192 keys: 97.6 us, without 101; 256 of 300
    // keys 61.7, without 58.)  A warp that has given up still walks along to here.
    if (vis >= 4 * kWarps) named_barrier(1, kWarps * 32);

    // Every warp leaves its rows and their statistics, kRound rows at a time, for
    // the merging warp, and goes on with the next unit.  (With the merging done by
    // all of them behind a barrier they waited for one another at every unit's end:
    // 256 sequences of 300 keys, 8 heads, E4M3 67 us.)
    // acc's unit; an empty share has none
    const float unit = kFp8 && v_top > 0 ? __uint_as_float((uint32_t)max(v_top - kWeightUp, 0) << 23) : 1.0f;
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
#pragma unroll 1
    for (int r0 = 0; r0 < rows && !lost; r0 += L::kRound, ++round) {
      if (!paged::wait_warp(merged, round & 1 ^ 1, abort, &g_err, kSiteMerged, p.wait_limit_ns)) {
        lost = true;
        break;
      }
      float* st_m = stats;
      float* st_l = st_m + kWarps * L::kRound;
      float* st_lr = st_l + kWarps * L::kRound;
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * n + 2 * c + e - r0;
          if (row < 0 || row >= min(L::kRound, rows - r0)) continue;
          if (g == 0) {
            st_m[row * kWarps + warp] = m[n][e];
            st_l[row * kWarps + warp] = l[n][e];
            // FP16 weights (E4M3 pages) are off by 2^-11 of themselves at most, an
            // eighth of O's own rounding, and O divided by the sum of the FP32 ones by
            // 2^-11 of the weighted mean of |v|; with their own sum that bound would
            // be no smaller (only values all alike would come out as they are)
            st_lr[row * kWarps + warp] = kFp8 ? l[n][e] : ones[n][e];
          }
          float* to = merge + (warp * L::kRound + row) * L::kPitch;
#pragma unroll
          for (int d = 0; d < kSteps; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) to[16 * d + (kFp8 ? 2 * g + h : 8 * h + g)] = acc[n][d][2 * h + e] * unit;
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(written);
    }
    at = after;
  }

  // After a give-up, loads already in flight land before the shared memory they
  // target is released.
  if (ld_shared_volatile(abort)) {
    const uint64_t w0 = globaltimer_ns();
    while (globaltimer_ns() - w0 < 2000000ull) __nanosleep(1000);
  }
}

// Joins the partial results of the units that borders between thread blocks
// cut: block (x, y) looks at border x + 1 and does rows [8 y, 8 y + 8) of the
// unit whose first cut that border is.  One long sequence has parts of every
// thread block: their statistics and rows are loaded together, not one after
// the other.
constexpr int kJoinThreads = 256, kJoinRows = 8;
template <int D, int kRows>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const PagedAttnParams p) {
  using W = Part<D, kRows>;
  __shared__ float st_m[kMaxCtas + 1][kJoinRows], st_l[kMaxCtas + 1][kJoinRows], st_lr[kMaxCtas + 1][kJoinRows];
  __shared__ float inv[kJoinRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = blockIdx.x + 1;
  const int row0 = blockIdx.y * kJoinRows;
  const int r = threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;
  // Which slots the parts are in is known before how many there are; the first two
  // are loaded along with that (they hold anything where nothing is joined).
  constexpr int kAhead = 2;
  auto stat_of = [&](int k, int row) {
    return *reinterpret_cast<const float4*>(W::stat(p.part, paged::join_slot(c, k)) + (row0 + row) * W::kStat);
  };
  auto part_of = [&](int k) {
    return *reinterpret_cast<const float4*>(W::out(p.part, paged::join_slot(c, k)) + (row0 + r) * D + d);
  };
  const paged::Join j = *W::join(p.part, c);
  float4 st0, x0[kAhead];
  if (threadIdx.x < kAhead * kJoinRows) st0 = stat_of(threadIdx.x / kJoinRows, threadIdx.x % kJoinRows);
  if (r < kJoinRows) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) x0[k] = part_of(k);
  }
  const int rows = j.parts == 0 ? 0 : min(kJoinRows, j.n * p.group - row0);
  if (rows <= 0) return;
  for (int i = threadIdx.x; i < j.parts * kJoinRows; i += kJoinThreads) {
    const int k = i / kJoinRows, row = i % kJoinRows;
    if (row >= rows) continue;
    const float4 st = k < kAhead ? st0 : stat_of(k, row);
    st_m[k][row] = st.x;
    st_l[k][row] = st.y;
    st_lr[k][row] = st.z;
  }
  __syncthreads();
  if ((int)threadIdx.x < rows) {
    const int row = threadIdx.x;
    float mt = -INFINITY, lt = 0.0f, lrt = 0.0f;
    for (int k = 0; k < j.parts; ++k) mt = fmaxf(mt, st_m[k][row]);
    for (int k = 0; k < j.parts; ++k) {
      const float f = mt == -INFINITY ? 1.0f : ex2_mufu(st_m[k][row] - mt);
      st_m[k][row] = f;                            // from here on the part's factor
      lt += st_l[k][row] * f;
      lrt += st_lr[k][row] * f;
    }
    inv[row] = lrt == 0.0f ? 0.0f : 1.0f / lrt;
    const int tk = (row0 + row) / p.group, head = j.head * p.group + row0 + row - tk * p.group;
    const size_t li = p.s.cu ? (size_t)head * p.s.Sn + j.q0 + tk : ((size_t)j.b * p.Hq + head) * p.s.Sn + tk;
    p.lse[li] = lt == 0.0f ? -INFINITY : (mt + log2f(lt)) * 0.693147180559945309f;
  }
  __syncthreads();
  if (r >= rows) return;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float4& x, float f) {
    y.x += x.x * f;
    y.y += x.y * f;
    y.z += x.z * f;
    y.w += x.w * f;
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) add(x0[k], st_m[k][r]);      // (a join has two parts or more)
#pragma unroll 8
  for (int k = kAhead; k < j.parts; ++k) add(part_of(k), st_m[k][r]);
  const int tk = (row0 + r) / p.group, head = j.head * p.group + row0 + r - tk * p.group;
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + ((size_t)(j.q0 + tk) * p.Hq + head) * D + d) =
      make_uint2(pack_bf16x2(y.x * inv[r], y.y * inv[r]), pack_bf16x2(y.z * inv[r], y.w * inv[r]));
}

template <int D, bool kFp8, int kTiles, bool kTree>
fa_status launch_inst(const PagedAttnLaunch& L, cudaStream_t stream) {
  using Lay = Layout<D, kFp8, kTiles>;
  const int page_size = 1 << L.p.s.page_shift;
  const long long page_heads = (long long)L.p.s.num_pages * L.p.s.Hkv;
  const int box = page_size < Lay::kKeys ? page_size : Lay::kKeys;
  CUtensorMap tk, tv;
  fa_status st;
  if ((st = make_tmap_pages(&tk, L.k_pages, page_heads, page_size, D, kFp8, box)) != FA_OK) return st;
  if ((st = make_tmap_pages(&tv, L.v_pages, page_heads, page_size, D, kFp8, box)) != FA_OK) return st;
  auto kern = decode_kernel<D, kFp8, kTiles, kTree>;
  if ((st = prepare_kernel(reinterpret_cast<const void*>(kern), Lay::kBytes)) != FA_OK) return st;
  const int ctas = L.p.num_ctas;
  if ((st = launch_overlapped(kern, dim3(ctas), Lay::kThreads, Lay::kBytes, stream, tk, tv, L.p)) != FA_OK) return st;
  if (ctas == 1) return FA_OK;
  return launch_overlapped(combine_kernel<D, Lay::kRows>, dim3(ctas - 1, Lay::kRows / kJoinRows), kJoinThreads, 0, stream,
                           L.p);
}

// As few tiles of 8 rows as hold a sequence's rows.
template <int D, bool kFp8, bool kTree>
fa_status launch_tiles(const PagedAttnLaunch& L, cudaStream_t stream) {
  const long long rows = (long long)L.p.max_q * L.p.group;
  if (rows <= 8) return launch_inst<D, kFp8, 1, kTree>(L, stream);
  if constexpr (kDecodeRows(D) > 16) {
    if (rows > 16) return launch_inst<D, kFp8, 4, kTree>(L, stream);
  }
  return launch_inst<D, kFp8, 2, kTree>(L, stream);
}

template <bool kTree>
fa_status launch_pages(const PagedAttnLaunch& L, cudaStream_t stream) {
  if (L.D == 128) return L.fp8 ? launch_tiles<128, true, kTree>(L, stream) : launch_tiles<128, false, kTree>(L, stream);
  return L.fp8 ? launch_tiles<64, true, kTree>(L, stream) : launch_tiles<64, false, kTree>(L, stream);
}

}  // namespace pdec

size_t paged_decode_workspace(int D) {
  return D == 128 ? pdec::Part<128, kDecodeRows(128)>::bytes() : pdec::Part<64, kDecodeRows(64)>::bytes();
}

fa_status launch_paged_decode(const PagedAttnLaunch& L, cudaStream_t stream) {
  return L.p.tree ? pdec::launch_pages<true>(L, stream) : pdec::launch_pages<false>(L, stream);
}

fa_status paged_decode_take_device_error() {
  DeviceError e{0, 0};
  if (cudaMemcpyFromSymbol(&e, pdec::g_err, sizeof(e)) != cudaSuccess) return FA_ERR_CUDA;
  if (e.status != 0) {
    const DeviceError z{0, 0};
    if (cudaMemcpyToSymbol(pdec::g_err, &z, sizeof(z)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return static_cast<fa_status>(e.status);
}

}  // namespace fa
