// Attention of chunks of new tokens over a paged cache, on tcgen05.
//
//   O = softmax(scale q K^T [+ causal mask]) V, LSE, per row of q.
//
// A tile is up to 128 rows of (new token, query head of one key/value head's
// group), so grouped heads share the key and value tiles they read; a unit is
// a pair of tiles of one (sequence, key/value head), worked on in turn: while
// one tile's softmax runs, the tensor cores compute the other's products.
//
//   * Keys and values come in blocks of 128 from pages of 16 to 1024 tokens,
//     one TMA box per page (or per 128 rows of it), into a ring of shared
//     memory tiles.  Rows behind the sequence's end hold anything: as keys
//     they are masked, as values they are cleared before the product, since a
//     weight of zero would not cancel a NaN.
//   * E4M3 pages go through a second ring: eight warps widen each tile once per
//     unit, to FP16, which one conversion per pair of codes makes (BF16 takes
//     five instructions: 668 us for 512 tokens over 32K keys, 76/19 heads).  A
//     segment's largest key scale and largest value scale are taken out of the
//     tiles; what that leaves is a power of two of at most 1 per row, exact down
//     to 2^-15 (FP16's subnormals: below, bits of a code are rounded off, 2^-25 of
//     what the largest scale stands for).  The queries become FP16 by a power of
//     two of each row's own, which with the keys' scale goes to the scores in
//     FP32; the values' goes to O at the end.
//   * Work.  Whole rounds of units, one per thread block, run in lockstep
//     from the first key on, so that the pairs of a head share its keys in L2.
//     The units left over are a line, of their keys and a constant for each
//     one's start and end, that is cut into equal stretches (at the key block
//     before each border), one per thread block; parts of a cut unit are joined
//     by the combine kernel.  A few long chunks thus load all SMs.  A scheduler
//     warp works out each thread block's segments and hands them to the other
//     warps through a small ring.
//
// Warps: 0-3 and 4-7 softmax of tile 0 and 1 (a thread per row), 8-11
// correction and epilogue, 12 loads, 13 MMA issue, 14 clearing of values
// behind the end (BF16 pages), 15 scheduler, 16-23 widening (E4M3 pages).
// Registers: BF16 256 x 192 + 128 x 80 + 128 x 48 = 65,536 = 512 x 128;
// E4M3 256 x 128 + 128 x 72 + 128 x 56 + 256 x 48 = 61,440 = 768 x 80.
//
// Tensor memory (512 columns): [0, 128) S of tile 0, its P as BF16 pairs in
// the first 64; [128, 256) tile 1; [256, 256 + D) O of tile 0; the next D
// columns O of tile 1.
#include <cuda_runtime.h>

#include "paged.cuh"
#include "softmax_math.cuh"

namespace fa {
namespace pchunk {

__device__ DeviceError g_err;

constexpr int kBM = 128;      // rows of a tile
constexpr int kBN = 128;      // keys of a block
constexpr float kThreshold = 8.0f;   // lazy rescaling, log2 units
// E4M3: weights are taken times 2^7 to FP16.  With the threshold they stay at
// most 2^15, and keep FP16's full precision down to 2^-21 of the maximum.
constexpr float kWeightUp = 7.0f;
constexpr int kMinStretch = 2 * kBN;  // keys: shorter stretches cost more to join than they save
// What a unit takes on the line besides its keys: its start (queries, the first
// scores) and its epilogue, when the tensor cores wait.  (12 ragged E4M3
// sequences, 1 to 500 tokens over up to 9000 keys: as nothing 123 us, as one block
// 119, 4 110, 8 115; others 138 -> 99, 119 -> 72.)
constexpr int kUnitCost = 4 * kBN;

enum Site {
  kSiteSeqs = 1, kSitePage, kSiteSegFull, kSiteSegEmpty, kSiteQEmpty, kSiteKvEmpty, kSiteKvFull, kSiteQFull, kSiteS,
  kSiteP, kSiteO, kSiteLanded, kSiteRaw, kSiteQReady, kSiteTops
};

// Workspace: per slot (two per thread block) both tiles' unnormalised rows, then
// per slot and row maximum and sums.  The rows lie in pieces of 8 columns,
// [D / 8][row][8], so that a warp, which holds a row a lane, stores whole lines.
template <int D>
struct Part {
  static constexpr int kRows = 2 * kBM;
  static constexpr int kStat = 4;
  FA_DEV static float* out(float* ws, int slot) { return ws + (size_t)slot * kRows * D; }
  FA_DEV static int piece(int i, int row) { return (i * kRows + row) * 8; }
  FA_DEV static float* stat(float* ws, int slot) {
    return ws + (size_t)2 * kMaxCtas * kRows * D + (size_t)slot * kRows * kStat;
  }
  FA_DEV static paged::Join* join(float* ws, int c) {
    return reinterpret_cast<paged::Join*>(stat(ws, 2 * kMaxCtas)) + c;
  }
  static constexpr size_t bytes() {
    return (size_t)2 * kMaxCtas * kRows * (D + kStat) * sizeof(float) + kMaxCtas * sizeof(paged::Join);
  }
};

// A segment: blocks [kb, kb + count) of a unit, as the roles get it.
struct Seg {
  int b, head, tok0;     // tok0: the pair's first new token; b < 0: no more work
  int kb, count;
  int n, L, q0;
  int slot;              // partial results go here; -1: the unit is whole
  int pad[3];
};
constexpr int kSegs = 4;

template <int D, bool kFp8>
struct Layout {
  static constexpr int kThreads = kFp8 ? 768 : 512;
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = kBM * D * 2;
  static constexpr int kChunkBytes = kBM * 128;
  static constexpr int kStages = D == 128 ? (kFp8 ? 3 : 4) : 6;
  static constexpr int kRawBytes = kBN * D;                  // an E4M3 tile
  static constexpr int kRaws = kFp8 ? 3 : 0;
  static constexpr int kReaders = kFp8 ? 22 : 15;            // warps that take segments
  static constexpr int kQ = 0;
  static constexpr int kKV = kQ + 2 * kTileBytes;
  static constexpr int kRaw = kKV + kStages * kTileBytes;
  static constexpr int kRawScale = kRaw + kRaws * kRawBytes;
  static constexpr int kStats = kRawScale + kRaws * kBN;     // scale, l, m (and lr) of [2][128]
  // E4M3.  Of four segments in turn: the warps' largest scale bytes of keys and
  // values (the widening warps are up to two segments ahead of the products, and
  // those one ahead of the epilogue).
  static constexpr int kTops = kStats + (kFp8 ? 3 : 4) * 2 * kBM * 4;
  static constexpr int kKPre = kTops + (kFp8 ? 4 * 8 * 2 * 4 : 0);     // key prefix [B + 1], 64 bits
  static constexpr int kUPre = kKPre + (kMaxPackedSeqs + 1) * 8;   // unit prefix [B + 1], longest unit
  static constexpr int kSums = (kUPre + (kMaxPackedSeqs + 2) * 4 + 7) / 8 * 8;
  static constexpr int kSegRing = (kSums + 32 * 16 + 15) / 16 * 16;
  static constexpr int kBars = kSegRing + kSegs * (int)sizeof(Seg);
  static constexpr int kNumBars = 2 + 2 * kStages + 10 + 2 * kSegs + (kFp8 ? 2 * kRaws + 2 : kStages);
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
  FA_DEV uint32_t q_full() const { return bar(0); }
  FA_DEV uint32_t q_empty() const { return bar(1); }
  FA_DEV uint32_t kv_full(int s) const { return bar(2 + s); }
  FA_DEV uint32_t kv_empty(int s) const { return bar(2 + L::kStages + s); }
  FA_DEV uint32_t s_full(int t) const { return bar(2 + 2 * L::kStages + t); }
  FA_DEV uint32_t p_lo(int t) const { return bar(4 + 2 * L::kStages + t); }
  FA_DEV uint32_t p_hi(int t) const { return bar(6 + 2 * L::kStages + t); }
  FA_DEV uint32_t o_ready(int t) const { return bar(8 + 2 * L::kStages + t); }
  FA_DEV uint32_t o_full(int t) const { return bar(10 + 2 * L::kStages + t); }
  FA_DEV uint32_t seg_full(int s) const { return bar(12 + 2 * L::kStages + s); }
  FA_DEV uint32_t seg_empty(int s) const { return bar(12 + 2 * L::kStages + kSegs + s); }
  // BF16: a value tile with rows to clear has landed (the clearing warp then
  // fills kv_full).  One per stage, so that it cannot run a phase ahead.
  FA_DEV uint32_t v_landed(int s) const { return bar(12 + 2 * L::kStages + 2 * kSegs + s); }
  FA_DEV uint32_t raw_full(int s) const { return bar(12 + 2 * L::kStages + 2 * kSegs + s); }
  FA_DEV uint32_t raw_empty(int s) const { return bar(12 + 2 * L::kStages + 2 * kSegs + L::kRaws + s); }
  FA_DEV uint32_t q_ready() const { return bar(12 + 2 * L::kStages + 2 * kSegs + 2 * L::kRaws); }   // E4M3: Q is FP16
  FA_DEV uint32_t tops_full() const { return bar(13 + 2 * L::kStages + 2 * kSegs + 2 * L::kRaws); }
  // E4M3, of segment number seg: largest scale bytes (all widening warps have
  // written theirs).
  FA_DEV int* tops(uint32_t seg) const { return reinterpret_cast<int*>(base + L::kTops) + (seg & 3) * 16; }
  FA_DEV int key_top(uint32_t seg) const { return top_of(tops(seg)); }
  FA_DEV int value_top(uint32_t seg) const { return top_of(tops(seg) + 8); }
  FA_DEV static int top_of(const int* t) {
    const int4 a = *reinterpret_cast<const int4*>(t), b = *reinterpret_cast<const int4*>(t + 4);
    return max(max(max(a.x, a.y), max(a.z, a.w)), max(max(b.x, b.y), max(b.z, b.w)));
  }
  FA_DEV uint32_t abort() const { return sbase + L::kMisc + 4; }
  FA_DEV uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(base + L::kMisc); }
  FA_DEV int* warp_flag() const { return reinterpret_cast<int*>(base + L::kMisc + 8); }
  FA_DEV float* st_scale() const { return reinterpret_cast<float*>(base + L::kStats); }
  FA_DEV float* st_l() const { return st_scale() + 2 * kBM; }
  FA_DEV float* st_m() const { return st_l() + 2 * kBM; }
  FA_DEV float* st_lr() const { return kFp8 ? st_l() : st_m() + 2 * kBM; }      // E4M3: one sum for both
  FA_DEV volatile Seg* segs() const { return reinterpret_cast<volatile Seg*>(base + L::kSegRing); }
  FA_DEV bool wait(uint32_t b, uint32_t parity, int site, const PagedAttnParams& p) const {
    return paged::wait_warp(b, parity, abort(), &g_err, site, p.wait_limit_ns);
  }
  // For waits that last as long as a segment (some seconds over 2^30 keys; the
  // other roles wait for a block at a time, and give up first if nothing moves).
  // Roles that are not in a hurry sleep between looks, off the issue slots.
  FA_DEV bool wait_long(uint32_t b, uint32_t parity, int site, const PagedAttnParams& p, bool sleeps = true) const {
#pragma unroll 1
    for (int i = 0; i < (1 << 27) && !mbar_try_wait(b, parity) && !ld_shared_volatile(abort()); ++i)
      if (sleeps) __nanosleep(200);
    return wait(b, parity, site, p);
  }
};

// ------------------------------------------------------------- units, line --

FA_DEV int tile_tokens(int group) { return kBM / group; }

// A sequence's pairs of tiles and the keys that they see.
struct Seq {
  int n, L, q0;
  int pairs, t2;      // pairs of tiles, tokens of a pair
  bool causal;
  // Keys of a pair: at least one, so that rows without a key are written too.
  FA_DEV int keys(int pair) const { return max(1, causal ? min(L, L - n + (pair + 1) * t2) : L); }
  FA_DEV int blocks(int pair) const { return (keys(pair) + kBN - 1) / kBN; }
  // What the pairs [0, p) take on the line: their keys, and kUnitCost each.
  FA_DEV long long prefix(int p) const { return keys_before(p) + (long long)p * kUnitCost; }
  FA_DEV long long keys_before(int p) const {
    if (!causal) return (long long)p * max(1, L);
    const long long last = p == pairs ? keys(pairs - 1) : 0;  // the one whose end the sequence's end cuts
    if (p == pairs) --p;
    const int e0 = L - n + t2;                                // of pair 0
    const int none = e0 <= 0 ? min(p, -e0 / t2 + 1) : 0;      // pairs that see no key
    return last + none + (long long)(p - none) * e0 +
           ((long long)p * (p - 1) - (long long)none * (none - 1)) / 2 * t2;
  }
  FA_DEV long long total() const { return prefix(pairs); }
  // Pairs run from the last (the longest under a mask) to the first: keys of
  // the i units before unit i of a head, all of which have `total`.
  FA_DEV long long before(int i, long long total) const { return total - prefix(pairs - i); }
};
FA_DEV Seq seq_from(const PagedAttnParams& p, const paged::SeqRows& rows) {
  Seq r;
  r.L = rows.L;
  r.n = rows.n;
  r.q0 = rows.q0;
  r.t2 = 2 * tile_tokens(p.group);
  r.pairs = (r.n + r.t2 - 1) / r.t2;
  r.causal = p.causal != 0;
  return r;
}
FA_DEV Seq seq_of(const PagedAttnParams& p, int b) { return seq_from(p, paged::rows_of(p.s, b)); }

// The work of a call: prefix tables over the sequences and where the whole
// rounds end.
struct Line {
  const long long* kpre;
  const int* upre;
  int units;          // all units
  int whole;          // units of the whole rounds
  long long t0, t1;   // the keys of the others
  int G;              // stretches that they are cut into
  FA_DEV long long stretch(int c) const { return t0 + paged::div64((t1 - t0) * c, G); }
};

// Last b in [0, B) with table[b] <= x.
template <class T>
FA_DEV int last_at_most(const T* table, int B, T x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Builds the tables; all threads of the block.  No units when the sequences
// break the rules.
FA_DEV Line build_line(const PagedAttnParams& p, long long* kpre, int* upre, long long* sums, int ctas) {
  Line line{kpre, upre, 0, 0, 0, 0, 0};
  const bool ok = paged::prefix_sequences(
      p.s, p.max_q,
      [&](const paged::SeqRows& rows) {
        const Seq s = seq_from(p, rows);
        return paged::Work{s.total() * p.s.Hkv, s.pairs * p.s.Hkv, s.keys(s.pairs - 1) + kUnitCost};
      },
      kpre, upre, sums);
  if (!ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) paged::record_bad_input(&g_err, kSiteSeqs);
    return line;
  }
  const int carry_u = upre[p.s.B];
  line.units = carry_u;
  line.t1 = kpre[p.s.B];
  // Whole rounds need units of about one length; else everything is cut.  (4
  // prompts of 4096 tokens, where units under the mask are of all lengths: 317 us
  // in rounds, 275 us cut; 512 tokens over 32K keys, 76/19 heads: 442 us in a round,
  // 483 us cut.)  A last round that is nearly full is not worth cutting.
  const int rest = carry_u < ctas ? carry_u : carry_u % ctas;
  const bool alike = (long long)upre[p.s.B + 1] * carry_u * 4 <= line.t1 * 5;
  line.whole = !alike ? 0 : rest * 10 >= ctas * 9 ? carry_u : carry_u - rest;
  if (line.whole == 0) {
    line.t0 = 0;
  } else if (line.whole < carry_u) {
    const int b = last_at_most(upre, p.s.B, line.whole);
    const Seq s = seq_of(p, b);
    const int r = line.whole - upre[b], head = r / s.pairs;
    const long long total = s.total();
    line.t0 = kpre[b] + head * total + s.before(r - head * s.pairs, total);
  } else {
    line.t0 = line.t1;
  }
  const long long most = (line.t1 - line.t0 + kMinStretch - 1) / kMinStretch;
  line.G = most < ctas ? (int)most : ctas;
  return line;
}

// A place on the line, at a key block: block kb of unit i of a head (pair
// pairs - 1 - i).
struct Place {
  int b, head, i, kb;
  long long start;    // the unit's first position
};
// The last one at or before position t < t1; kb may be the unit's blocks (t lies
// in its cost: the unit stays whole).  One warp, converged.
FA_DEV Place find_place(const PagedAttnParams& p, const Line& line, long long t) {
  Place w;
  w.b = last_at_most(line.kpre, p.s.B, t);
  const Seq s = seq_of(p, w.b);
  const long long per_head = s.total();
  long long r = t - line.kpre[w.b];
  w.head = (int)paged::div64(r, per_head);
  r -= w.head * per_head;
  const int lane = threadIdx.x % 32;
  int lo = 0, size = s.pairs;       // the unit is in [lo, lo + size)
  while (size > 1) {
    const int step = (size + 31) / 32, at = lo + lane * step;
    const bool in = at < lo + size && s.before(at, per_head) <= r;
    const int k = __popc(__ballot_sync(0xffffffffu, in)) - 1;
    size = min(step, size - k * step);
    lo += k * step;
  }
  w.i = lo;
  w.start = t - r + s.before(lo, per_head);
  w.kb = min((int)((t - w.start) / kBN), s.blocks(s.pairs - 1 - lo));
  return w;
}

// ------------------------------------------------------------------ roles --

FA_DEV int all_same(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Takes the next segment out of the ring; false at the end of the work or
// after a give-up.
template <int D, bool kFp8>
struct SegReader {
  const Shared<D, kFp8>& sh;
  const PagedAttnParams& p;
  int i = 0;
  uint32_t phase = 0;
  FA_DEV SegReader(const Shared<D, kFp8>& s, const PagedAttnParams& q) : sh(s), p(q) {}
  // The whole warp calls it.  `idle`: had nothing to do with the segments before, and
  // may be here as long before the next as one lasts.
  FA_DEV bool next(Seg& w, bool idle = false, bool sleeps = true) {
    if (!(idle ? sh.wait_long(sh.seg_full(i), phase, kSiteSegFull, p, sleeps)
               : sh.wait(sh.seg_full(i), phase, kSiteSegFull, p)))
      return false;
    const volatile Seg& r = sh.segs()[i];
    // a value that comes out of a shuffle is known to be the same in all lanes,
    // so that what depends on it (loops, ring positions, MMA descriptors) stays
    // in uniform registers; with plain loads the MMA warp alone took half as
    // long again
    w.b = all_same(r.b);
    w.head = all_same(r.head);
    w.tok0 = all_same(r.tok0);
    w.kb = all_same(r.kb);
    w.count = all_same(r.count);
    w.n = all_same(r.n);
    w.L = all_same(r.L);
    w.q0 = all_same(r.q0);
    w.slot = all_same(r.slot);
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(sh.seg_empty(i));
    if (++i == kSegs) {
      i = 0;
      phase ^= 1;
    }
    return w.b >= 0;
  }
};

// Key blocks of the segment that tile t sees.
FA_DEV int tile_blocks(const Seg& w, int t, int tt, bool causal) {
  const int tok = w.tok0 + t * tt;
  if (tok >= w.n) return 0;
  const int end = causal ? min(w.L, w.L - w.n + min(tok + tt, w.n)) : w.L;
  return min(w.count, max(0, (end + kBN - 1) / kBN - w.kb));
}

template <int D, bool kFp8>
__device__ void scheduler_role(const Shared<D, kFp8>& sh, const PagedAttnParams& p, const Line& line) {
  const int lane = threadIdx.x % 32;
  const int G = gridDim.x, c = blockIdx.x;
  int slot_i = 0;
  uint32_t phase = 1;
  auto put = [&](int b, int head, int pair, int kb, int count, const Seq& s, int slot) -> bool {
    if (!sh.wait_long(sh.seg_empty(slot_i), phase, kSiteSegEmpty, p)) return false;
    if (lane == 0) {
      volatile Seg& r = sh.segs()[slot_i];
      r.b = b;
      r.head = head;
      r.tok0 = pair * s.t2;
      r.kb = kb;
      r.count = count;
      r.n = s.n;
      r.L = s.L;
      r.q0 = s.q0;
      r.slot = slot;
      mbar_arrive(sh.seg_full(slot_i));
    }
    __syncwarp();
    if (++slot_i == kSegs) {
      slot_i = 0;
      phase ^= 1;
    }
    return true;
  };
  for (int u = c; u < line.whole; u += G) {
    const int b = last_at_most(line.upre, p.s.B, u);
    const Seq s = seq_of(p, b);
    const int r = u - line.upre[b], head = r / s.pairs;
    const int pair = s.pairs - 1 - (r - head * s.pairs);
    if (!put(b, head, pair, 0, s.blocks(pair), s, -1)) return;
  }
  paged::Join join{};
  if (c < line.G) {
    Place w = find_place(p, line, line.stretch(c));
    const bool to_end = c + 1 == line.G;
    const Place z = to_end ? Place{} : find_place(p, line, line.stretch(c + 1));
    Seq s = seq_of(p, w.b);
    const int pair = s.pairs - 1 - w.i, nblk = s.blocks(pair);
    if (w.kb > 0 && w.kb < nblk) {
      // the unit is cut here: if for the first time, its parts are joined
      if (line.stretch(c - 1) < w.start + kBN) {
        const long long end = w.start + (long long)nblk * kBN;
        join = paged::Join{2, w.b, w.head, pair * s.t2, s.n, s.q0, {0, 0}};
        while (c + join.parts - 1 < line.G && line.stretch(c + join.parts - 1) < end) ++join.parts;
      }
    }
    // from place w to place z
    for (;;) {
      const int pair = s.pairs - 1 - w.i, nblk = s.blocks(pair);
      const bool last = !to_end && w.b == z.b && w.head == z.head && w.i == z.i;
      const int end = last ? z.kb : nblk;
      if (end > w.kb) {
        const int slot = w.kb > 0 ? 2 * c : end < nblk ? 2 * c + 1 : -1;
        if (!put(w.b, w.head, pair, w.kb, end - w.kb, s, slot)) return;
      }
      if (last) break;
      w.kb = 0;
      if (++w.i == s.pairs) {
        w.i = 0;
        if (++w.head == p.s.Hkv) {
          w.head = 0;
          do {
            if (++w.b == p.s.B) break;
            s = seq_of(p, w.b);
          } while (s.n == 0);
          if (w.b == p.s.B) break;
        }
      }
    }
  }
  if (lane == 0) *Part<D>::join(p.part, c) = join;
  Seq none{};
  put(-1, 0, 0, 0, 0, none, -1);
}

// Loads: Q of both tiles once per segment, then the key and value blocks in
// turn.  The whole warp runs along; lane 0 issues, the lanes hold the numbers
// of the next 32 pages.
template <int D, bool kFp8>
__device__ void load_role(const Shared<D, kFp8>& sh, const CUtensorMap* tq, const CUtensorMap* tk,
                          const CUtensorMap* tv, const PagedAttnParams& p) {
  using L = Layout<D, kFp8>;
  const int lane = threadIdx.x % 32;
  const int tt = tile_tokens(p.group);
  const int box = min(1 << p.s.page_shift, kBN);          // rows of a box
  constexpr int kRing = kFp8 ? L::kRaws : L::kStages;
  SegReader<D, kFp8> in(sh, p);
  Seg w;
  uint32_t uit = 0;
  int stage = 0;
  uint32_t phase = 1;
  while (in.next(w)) {
    const int n0 = tile_blocks(w, 0, tt, p.causal), n1 = tile_blocks(w, 1, tt, p.causal);
    const int n = max(n0, n1);
    if (n == 0) continue;
    if (!sh.wait(sh.q_empty(), (uit & 1) ^ 1, kSiteQEmpty, p)) return;
    if (lane == 0) {
      mbar_arrive_expect_tx(sh.q_full(), 2 * tt * p.group * D * 2);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
          tma_load_3d(sh.sbase + L::kQ + t * L::kTileBytes + c * L::kChunkBytes, tq, sh.q_full(), c * 64,
                      w.head * p.group, w.q0 + w.tok0 + t * tt);
    }
    ++uit;
    const int* table = p.s.block_table + (size_t)w.b * p.s.max_pages;
    const int last_page = (w.L - 1) >> p.s.page_shift;
    int held = -64, pages = -1;                            // pages[held .. held + 32) one per lane
    for (int j = 0; j < n; ++j) {
      const int key0 = (w.kb + j) * kBN;
      const int boxes = (min(kBN, w.L - key0) + box - 1) / box;   // that hold a key of the sequence
      const int page0 = key0 >> p.s.page_shift;
      if (page0 < held || page0 + boxes > held + 32) {
        held = page0;
        pages = -1;
        if (held + lane <= last_page) {
          pages = table[held + lane];
          if (pages < 0 || pages >= p.s.num_pages) {
            if (held + lane <= (min(w.L, (w.kb + n) * kBN) - 1) >> p.s.page_shift)
              paged::record_bad_input(&g_err, kSitePage);
            pages = -1;
          }
        }
      }
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        const bool clear = !kFp8 && which && w.L - key0 < kBN;
        const uint32_t full = kFp8 ? sh.raw_full(stage) : clear ? sh.v_landed(stage) : sh.kv_full(stage);
        if (!sh.wait(kFp8 ? sh.raw_empty(stage) : sh.kv_empty(stage), phase, kSiteKvEmpty, p)) return;
        if (lane == 0) mbar_arrive_expect_tx(full, boxes * box * (kFp8 ? D + 1 : 2 * D));
        __syncwarp();
        const CUtensorMap* map = which ? tv : tk;
        const uint32_t dst = sh.sbase + (kFp8 ? L::kRaw + stage * L::kRawBytes : L::kKV + stage * L::kTileBytes);
        // each lane issues its own box
        constexpr int kParts = kFp8 ? 1 : L::kChunks;
        const int i = lane / kParts, c = lane % kParts;
        const int page = __shfl_sync(0xffffffffu, pages, (page0 + i - held) & 31);
        if (i < boxes) {
          const int off = (key0 + i * box) & ((1 << p.s.page_shift) - 1);
          const int ph = page < 0 ? -1 : page * p.s.Hkv + w.head;    // -1: reads as zeros
          if (kFp8) {
            tma_load_3d(dst + i * box * D, map, full, 0, off, ph);
            bulk_load(sh.sbase + L::kRawScale + stage * kBN + i * box,
                      ph < 0 ? paged::g_no_scales : (which ? p.v_scale : p.k_scale) + ((size_t)ph << p.s.page_shift) + off,
                      box, full);
          } else {
            tma_load_3d(dst + c * L::kChunkBytes + i * box * 128, map, full, c * 64, off, ph);
          }
        }
        __syncwarp();
        if (++stage == kRing) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  }
}

// BF16 pages: value rows behind the sequence's end, in its last block, are
// cleared between the load and the product.
template <int D>
__device__ void clean_role(const Shared<D, false>& sh, const PagedAttnParams& p) {
  using L = Layout<D, false>;
  const int lane = threadIdx.x % 32;
  const int tt = tile_tokens(p.group);
  SegReader<D, false> in(sh, p);
  Seg w;
  uint32_t tiles = 0;      // tiles that went through the ring
  uint32_t parity = 0;     // of each stage's v_landed
  while (in.next(w, true)) {
    const int n = max(tile_blocks(w, 0, tt, p.causal), tile_blocks(w, 1, tt, p.causal));
    const int rows = w.L - (w.kb + n - 1) * kBN;
    if (n > 0 && rows < kBN) {
      const int stage = (tiles + 2 * n - 1) % L::kStages;
      if (!sh.wait_long(sh.v_landed(stage), (parity >> stage) & 1, kSiteLanded, p)) return;
      parity ^= 1u << stage;
      uint8_t* tile = sh.base + L::kKV + stage * L::kTileBytes;
      for (int c = 0; c < L::kChunks; ++c)
        for (int i = rows * 8 + lane; i < kBN * 8; i += 32)
          *reinterpret_cast<uint4*>(tile + c * L::kChunkBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.kv_full(stage));
    }
    tiles += 2 * n;
  }
}

FA_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes (the lower half of w) as FP16, exactly, times f.
FA_DEV uint32_t widened(uint32_t w, uint32_t f) {
  uint32_t r;
  asm("{\n\t.reg .b32 h;\n\tcvt.rn.f16x2.e4m3x2 h, %1;\n\tmul.rn.f16x2 %0, h, %2;\n\t}"
      : "=r"(r)
      : "h"((uint16_t)w), "r"(f));
  return r;
}
// 2^d, d <= 0, as FP16 twice; zero below its range.
FA_DEV uint32_t power_f16x2(int d) {
  const uint32_t h = d >= -14 ? (uint32_t)(15 + d) << 10 : d >= -24 ? 1u << (24 + d) : 0u;
  return h | h << 16;
}

// The largest scale bytes (of finite rows) among the segment's keys and values,
// left in `tops`; the eight widening warps, 16 keys a thread at a time.
template <int D>
FA_DEV void find_tops(const PagedAttnParams& p, const Seg& w, int blocks, int* tops) {
  const int lane = threadIdx.x % 32, thread = threadIdx.x - 512;
  const int first = w.kb * kBN, end = min(w.L, (w.kb + blocks) * kBN);
  const int* table = p.s.block_table + (size_t)w.b * p.s.max_pages;
  uint32_t top[2] = {0u, 0u};                        // per byte
#pragma unroll 4
  for (int key = first + 16 * thread; key < end; key += 16 * 256) {
    const int page = table[key >> p.s.page_shift];
    if (page < 0 || page >= p.s.num_pages) continue;
    const size_t row = ((size_t)page * p.s.Hkv + w.head << p.s.page_shift) + (key & ((1 << p.s.page_shift) - 1));
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint4 x = *reinterpret_cast<const uint4*>((which ? p.v_scale : p.k_scale) + row);
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int left = end - key - 4 * i;          // bytes of the word that count
        const uint32_t on = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        top[which] = __vmaxu4(top[which], v[i] & on & ~__vcmpeq4(v[i], 0xFFFFFFFFu));
      }
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint32_t m = max(max(top[which] & 255u, (top[which] >> 8) & 255u), max((top[which] >> 16) & 255u, top[which] >> 24));
    const int all = __reduce_max_sync(0xffffffffu, (int)m);
    if (lane == 0) tops[8 * which + thread / 32] = all;
  }
}

// E4M3 pages: eight warps widen the tiles, four the keys and four the values, a
// piece of 16 codes at a time, into the swizzled FP16 tiles that the products
// read.  Rows behind the sequence's end come out as zeros.
template <int D>
__device__ void widen_role(const Shared<D, true>& sh, const PagedAttnParams& p) {
  using L = Layout<D, true>;
  // A step is a warp's 32 pieces of 16 codes.  The eight lanes that load and
  // store together touch all banks: at D = 128 they are four pieces of rows r
  // and r ^ 5 (the 128-byte swizzle puts the halves of a raw row apart by bit 2
  // of its number, the even and odd pieces of a wide row by bit 0), a step
  // rows {0, 5, 1, 4} or {2, 7, 3, 6} of eight; at D = 64 two neighbouring rows.
  constexpr int kSteps = D / 16;
  constexpr int kGroups = D == 128 ? 1 : 2;          // of eight rows, in two steps
  constexpr int kDown = 8 * kGroups * D;             // raw bytes
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 % 4;
  const bool values = threadIdx.x >= 640;
  const int tt = tile_tokens(p.group);
  int row[2], from[2], to[2][2];                     // in the warp's 32 rows; offsets of the tiles
#pragma unroll
  for (int odd = 0; odd < 2; ++odd) {
    const int piece = D == 128 ? lane & 3 | lane >> 1 & 4 : lane & 3;
    row[odd] = D == 128 ? (2 * odd + (lane >> 4)) ^ (lane & 4 ? 5 : 0) : 8 * odd + (lane >> 2);
    const int r = warp * 32 + row[odd];
    from[odd] = D == 128 ? r * 128 + ((piece ^ (r & 7)) << 4) : r * 64 + ((piece ^ ((r >> 1) & 3)) << 4);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      to[odd][s] = (piece / 4) * L::kChunkBytes + r * 128 + (((2 * (piece % 4) + s) ^ (r & 7)) << 4);
  }
  SegReader<D, true> in(sh, p);
  Seg w;
  uint32_t at = values ? 1 : 0;                      // tile in the order of the loads: keys even, values odd
  uint32_t seg = 0;
  while (in.next(w)) {
    const int n = max(tile_blocks(w, 0, tt, p.causal), tile_blocks(w, 1, tt, p.causal));
    if (n == 0) continue;
    // The eight warps wait for one another's largest scales on an mbarrier, which
    // gives up with the rest of the block: a barrier of the hardware's would hold
    // the ones that come to it after the others have given up and left.
    find_tops<D>(p, w, n, sh.tops(seg));
    if (lane == 0) mbar_arrive(sh.tops_full());
    if (!sh.wait(sh.tops_full(), seg & 1, kSiteTops, p)) return;
    const int top = values ? sh.value_top(seg) : sh.key_top(seg);
    ++seg;
#pragma unroll 1
    for (int j = 0; j < n; ++j, at += 2) {
      const int rows = w.L - (w.kb + j) * kBN;
      const int raw = at % L::kRaws, stage = at % L::kStages;
      if (!sh.wait(sh.raw_full(raw), (at / L::kRaws) & 1, kSiteRaw, p)) return;
      if (!sh.wait(sh.kv_empty(stage), (at / L::kStages & 1) ^ 1, kSiteKvEmpty, p)) return;
      const uint8_t* src = sh.base + L::kRaw + raw * L::kRawBytes;
      uint8_t* dst = sh.base + L::kKV + stage * L::kTileBytes;
      // lane l holds the factor of row 32 warp + l
      const int byte = sh.base[L::kRawScale + raw * kBN + warp * 32 + lane];
      const uint32_t f = byte == 255 ? 0x7E007E00u : power_f16x2(byte - top);
      const bool ragged = rows < kBN;
#pragma unroll 4
      for (int i = 0; i < kSteps; ++i) {
        // rows of a step repeat every two steps, 8 rows (1024 bytes) further
        const int odd = i & 1, down = i >> 1;
        const int r = row[odd] + down * 8 * kGroups;
        uint4 x = *reinterpret_cast<const uint4*>(src + from[odd] + down * kDown);
        const uint32_t fr = __shfl_sync(0xffffffffu, f, r);
        if (ragged && warp * 32 + r >= rows) x = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t fz = ragged && warp * 32 + r >= rows ? 0u : fr;
        *reinterpret_cast<uint4*>(dst + to[odd][0] + down * 1024 * kGroups) =
            make_uint4(widened(x.x, fz), widened(x.x >> 16, fz), widened(x.y, fz), widened(x.y >> 16, fz));
        *reinterpret_cast<uint4*>(dst + to[odd][1] + down * 1024 * kGroups) =
            make_uint4(widened(x.z, fz), widened(x.z >> 16, fz), widened(x.w, fz), widened(x.w >> 16, fz));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sh.kv_full(stage));
        mbar_arrive(sh.raw_empty(raw));
      }
    }
  }
}

// Masks the columns >= lim of a row's scores, in tensor memory: only the blocks
// at the edge of the mask come here, and a rolled loop over tensor memory costs
// the others less (in code to fetch) than predicates on 128 registers.
FA_DEV void mask_scores(uint32_t tm_s, int lim) {
#pragma unroll 1
  for (int c = 0; c < kBN; c += 32) {
    uint32_t x[32];
    tmem_ld32(tm_s + c, x);
    tmem_ld_wait();
    tmem_ld_fence(x);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c + i >= lim) x[i] = __float_as_uint(-INFINITY);
    tmem_st32(tm_s + c, x);
  }
  tmem_st_wait();
}
FA_DEV float max32(const uint32_t (&x)[32]) {
  float m = __uint_as_float(x[0]);
#pragma unroll
  for (int i = 1; i < 31; i += 2) m = max3(m, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
  return fmaxf(m, __uint_as_float(x[31]));
}

// A row's weights and sums, 32 scores at a time.
template <bool kFp16>
struct RowSums {
  uint64_t scale2, negm2;      // pairs of scale, -maximum (FP16: + kWeightUp)
  uint64_t e2[2];              // sums of the FP32 weights (LSE); a NaN among the scores passes into them
  uint64_t r2[2];              // BF16: and of the weights as they are rounded for the product, for the division.
                               // FP16 weights are off by 2^-11 of themselves at most, an eighth of O's own
                               // rounding: with a sum of their own O's bound would be no smaller
  FA_DEV void begin(float scale, float m) {
    scale2 = pk2(scale, scale);
    const float b = kFp16 ? kWeightUp - m : -m;
    negm2 = pk2(b, b);
    e2[0] = e2[1] = r2[0] = r2[1] = 0ull;
  }
  FA_DEV void weights(const uint32_t (&x)[32], uint32_t* pk) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint64_t x2 = fma2(pk2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), scale2, negm2);
      float x0, x1;
      up2(x2, x0, x1);
      const float e0 = ex2_mufu(x0), e1 = ex2_mufu(x1);
      const uint32_t pp = kFp16 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
      pk[i / 2] = pp;
      e2[(i / 2) & 1] = add2(e2[(i / 2) & 1], pk2(e0, e1));
      if (!kFp16)
        r2[(i / 2) & 1] = add2(r2[(i / 2) & 1], pk2(__uint_as_float(pp << 16), __uint_as_float(pp & 0xFFFF0000u)));
    }
  }
  FA_DEV void totals(float& e, float& r) const {
    float a, b;
    up2(add2(e2[0], e2[1]), a, b);
    e = a + b;
    if (kFp16) {
      r = e;
    } else {
      up2(add2(r2[0], r2[1]), a, b);
      r = a + b;
    }
  }
};

// Row r of tile t of Q, in place, to FP16 by a power of two of its own: 2^(13 - e),
// below 2^14 then; returns e.  At 2^126, the most, every BF16 number is exact in FP16.
template <int D>
FA_DEV int narrow_row(const Shared<D, true>& sh, int t, int r) {
  using L = Layout<D, true>;
  uint8_t* row = sh.base + L::kQ + t * L::kTileBytes + r * 128;
  uint4 x[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)     // (in an order in which eight neighbouring rows touch all banks)
    x[i] = *reinterpret_cast<const uint4*>(row + (i / 8) * L::kChunkBytes + (((i ^ r) & 7) << 4));
  uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    m[0] = paged::max_bf16x2(m[0], x[i].x & 0x7FFF7FFFu);
    m[1] = paged::max_bf16x2(m[1], x[i].y & 0x7FFF7FFFu);
    m[2] = paged::max_bf16x2(m[2], x[i].z & 0x7FFF7FFFu);
    m[3] = paged::max_bf16x2(m[3], x[i].w & 0x7FFF7FFFu);
  }
  m[0] = paged::max_bf16x2(paged::max_bf16x2(m[0], m[1]), paged::max_bf16x2(m[2], m[3]));
  const int e = max((int)(max(m[0] & 0xFFFFu, m[0] >> 16) >> 7), 14) - 127;       // of the largest value, -113 at least
  const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = pack_f16x2(__uint_as_float(v[k] << 16) * up, __uint_as_float(v[k] & 0xFFFF0000u) * up);
    *reinterpret_cast<uint4*>(row + (i / 8) * L::kChunkBytes + (((i ^ r) & 7) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
  }
  return e;
}

// Softmax of tile t: one thread per row.  The scores are read from tensor memory
// twice, for the maximum and for the exponentials, 32 columns at a time with
// the next 32 on their way.  The rolled loops keep the code small: with a
// block's 128 scores in registers and everything unrolled, the warps of the
// other roles found their code pushed out of the instruction cache each time
// (chunk of 512 tokens over 32K keys, 76 heads: 489 us, rolled 446 us).
template <int D, bool kFp8>
__device__ void softmax_role(const int t, const Shared<D, kFp8>& sh, const uint32_t tmem, const PagedAttnParams& p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int wq = warp & 3;
  const int r_in_tile = wq * 32 + lane;
  const uint32_t tm_s = tmem + (uint32_t(wq * 32) << 16) + uint32_t(t * kBN);
  float sl2 = p.scale_log2;
  const int tt = tile_tokens(p.group);
  const int my_tok = r_in_tile / p.group;
  SegReader<D, kFp8> in(sh, p);
  Seg w;
  uint32_t sit = 0, seg = 0;
  bool idle = false;       // the segment before had no block of this tile
  while (in.next(w, idle, false)) {
    const int nt = tile_blocks(w, t, tt, p.causal);
    int q_exp = 0;
    if constexpr (kFp8) {
      // Both tiles' warps take every segment's Q, also when theirs has no block,
      // so that neither falls two phases behind.
      if (max(nt, tile_blocks(w, t ^ 1, tt, p.causal)) > 0) {
        if (!(idle ? sh.wait_long(sh.q_full(), seg & 1, kSiteQFull, p, false)
                   : sh.wait(sh.q_full(), seg & 1, kSiteQFull, p)))
          return;
        if (nt > 0) q_exp = narrow_row<D>(sh, t, r_in_tile);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.q_ready());
        ++seg;
      }
    }
    idle = nt == 0;
    if (idle) continue;
    const int tok = w.tok0 + t * tt;
    const int lim_first = p.causal ? w.L - w.n + tok + 1 : w.L;                  // of the tile's first row
    const int lim_row = p.causal ? min(w.L, lim_first + my_tok) : w.L;
    // rows of the tile that are no token's hold anything: they must not cause
    // rescaling
    const bool live = my_tok < tt && tok + my_tok < w.n;
    float m_run = -INFINITY, l_run = 0.0f, lr_run = 0.0f;
    RowSums<kFp8> sums;
    // The new running maximum from the block's; returns the factor for what
    // was summed so far.  Lazy: a maximum that grew by less than the threshold
    // stays.
    auto move_max = [&](float m_blk, bool first, bool& rescaled) -> float {
      rescaled = false;
      if (first) {
        m_run = m_blk;
      } else if (m_blk - m_run > kThreshold) {
        const float f = ex2_mufu(m_run - m_blk);
        m_run = m_blk;
        rescaled = true;
        return f;
      }
      return 1.0f;
    };
    // The first half of P is in place: the factor goes along.
    auto give_lo = [&](float factor, bool rescaled) {
      sh.st_scale()[t * kBM + r_in_tile] = factor;
      const unsigned any = __any_sync(0xffffffffu, rescaled && live);
      if (lane == 0) sh.warp_flag()[t * 4 + wq] = any ? 1 : 0;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(sh.p_lo(t));
    };
    for (int j = 0; j < nt; ++j, ++sit) {
      if (!sh.wait(sh.s_full(t), sit & 1, kSiteS, p)) return;
      tc_fence_after();
      if (kFp8 && j == 0) {
        // the scores' unit, 2^-236 to 2^234: of the row of Q, and of the segment's
        // keys.  Its halves are floats, and both move the scale the same way, so
        // that only the product's own size counts.  That is normal and finite at
        // least: a masked score is -inf times this, which zero would make NaN, and a
        // score of zero stays one (below 2^-126 every score, 2^31 at most, is zero
        // to the exponentials).
        const int top = sh.key_top(seg - 1);
        const int unit = q_exp - 13 + (top > 0 ? top - 127 : 0), half = unit / 2;
        sl2 = p.scale_log2 * __uint_as_float((uint32_t)(half + 127) << 23) *
              __uint_as_float((uint32_t)(unit - half + 127) << 23);
        sl2 = fminf(fmaxf(sl2, 1.17549435e-38f), 3.40282347e38f);
      }
      const int kv0 = (w.kb + j) * kBN;
      const bool need_mask = kv0 + kBN > lim_first;
      const int lim = lim_row - kv0;            // columns >= lim are masked
      bool rescaled;
      float factor, m_blk, e, r;
      if (need_mask) mask_scores(tm_s, lim);
      uint32_t xa[32], xb[32], pk[16];
      m_blk = -INFINITY;
      tmem_ld32(tm_s, xa);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        tmem_ld_wait();
        tmem_ld_fence(xa);
        tmem_ld32(tm_s + 64 * half + 32, xb);
        m_blk = fmaxf(m_blk, max32(xa));
        tmem_ld_wait();
        tmem_ld_fence(xb);
        tmem_ld32(tm_s + (half ? 0 : 64), xa);       // at the end: the first columns again
        m_blk = fmaxf(m_blk, max32(xb));
      }
      m_blk *= sl2;
      factor = move_max(m_blk, j == 0, rescaled);
      sums.begin(sl2, m_run == -INFINITY ? 0.0f : m_run);
      // P goes over columns of S whose scores have been read
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        tmem_ld_wait();
        tmem_ld_fence(xa);
        tmem_ld32(tm_s + 64 * half + 32, xb);
        sums.weights(xa, pk);
        tmem_st16(tm_s + 32 * half, pk);
        tmem_ld_wait();
        tmem_ld_fence(xb);
        if (half == 0) tmem_ld32(tm_s + 64, xa);
        sums.weights(xb, pk);
        tmem_st16(tm_s + 32 * half + 16, pk);
        if (half == 0) give_lo(factor, rescaled);
      }
      sums.totals(e, r);
      l_run = l_run * factor + e;
      lr_run = lr_run * factor + r;
      tmem_st_wait();
      if (j == nt - 1) {
        sh.st_l()[t * kBM + r_in_tile] = kFp8 ? l_run * 0.0078125f : l_run;        // 2^-kWeightUp
        sh.st_lr()[t * kBM + r_in_tile] = kFp8 ? lr_run * 0.0078125f : lr_run;
        sh.st_m()[t * kBM + r_in_tile] = m_run;
      }
      tc_fence_before();
      mbar_arrive(sh.p_hi(t));
    }
  }
}

// Correction: rescales O in tensor memory when a row's maximum moved, and
// writes the segment's rows: O / l in BF16 and LSE of a whole unit, else the
// unnormalised row and its statistics.
template <int D, bool kFp8>
__device__ void correction_role(const Shared<D, kFp8>& sh, const uint32_t tmem, const PagedAttnParams& p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int wq = warp & 3;
  const int r_in_tile = wq * 32 + lane;
  const uint32_t lane_off = uint32_t(wq * 32) << 16;
  const int tt = tile_tokens(p.group);
  const int my_tok = r_in_tile / p.group, my_head = r_in_tile - my_tok * p.group;
  SegReader<D, kFp8> in(sh, p);
  Seg w;
  uint32_t sit = 0;      // phase bits of the two tiles
  uint32_t uit[2] = {0u, 0u}, seg = 0;
  while (in.next(w)) {
    const int nts[2] = {tile_blocks(w, 0, tt, p.causal), tile_blocks(w, 1, tt, p.causal)};
    const int n = max(nts[0], nts[1]);
    if (kFp8 && n > 0) ++seg;
    float unit = 1.0f;       // of O
    float fin_l[2] = {0.0f, 0.0f}, fin_lr[2] = {0.0f, 0.0f}, fin_m[2] = {-INFINITY, -INFINITY};
    for (int j = 0; j < n; ++j) {
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        if (j >= (t ? nts[1] : nts[0])) continue;
        const uint32_t ph = (sit >> t) & 1;
        sit ^= 1u << t;
        if (!sh.wait(sh.p_lo(t), ph, kSiteP, p)) return;
        tc_fence_after();
        if (j > 0 && sh.warp_flag()[t * 4 + wq]) {
          const float f = sh.st_scale()[t * kBM + r_in_tile];
          const uint64_t f2 = pk2(f, f);
          const uint32_t tm_o = tmem + lane_off + uint32_t(256 + t * D);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            tmem_ld32(tm_o + c * 32, r);
            tmem_ld_wait();
            tmem_ld_fence(r);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float y0, y1;
              up2(mul2(pk2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), f2), y0, y1);
              r[i] = __float_as_uint(y0);
              r[i + 1] = __float_as_uint(y1);
            }
            tmem_st32(tm_o + c * 32, r);
          }
          tmem_st_wait();
        }
        // the statistics come with the second half of the last block's P; they
        // are taken before O is released, after which the next segment's
        // softmax may overwrite them
        if (j == (t ? nts[1] : nts[0]) - 1) {
          if (!sh.wait(sh.p_hi(t), ph, kSiteP, p)) return;
          const float a = sh.st_l()[t * kBM + r_in_tile], b = sh.st_lr()[t * kBM + r_in_tile];
          const float c = sh.st_m()[t * kBM + r_in_tile];
          (t ? fin_l[1] : fin_l[0]) = a;
          (t ? fin_lr[1] : fin_lr[0]) = b;
          (t ? fin_m[1] : fin_m[0]) = c;
        }
        tc_fence_before();
        mbar_arrive(sh.o_ready(t));
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int tok = w.tok0 + t * tt + my_tok;
      const bool valid = my_tok < tt && tok < w.n;
      const bool has = nts[t] > 0;
      if (has) {
        if (!sh.wait(sh.o_full(t), uit[t] & 1, kSiteO, p)) return;
        ++uit[t];
        tc_fence_after();
      }
      const float l = fin_l[t], lr = fin_lr[t], m = fin_m[t];
      if (kFp8 && has) {
        const int top = sh.value_top(seg - 1);
        unit = top > 0 ? __uint_as_float((uint32_t)max(top - (int)kWeightUp, 0) << 23) : 1.0f;   // 2^(top - 127 - kWeightUp)
      }
      const float inv = w.slot >= 0 ? unit : lr == 0.0f ? 0.0f : unit / lr;
      const int head = w.head * p.group + my_head;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + ((size_t)(w.q0 + tok) * p.Hq + head) * D;
      float* part = Part<D>::out(p.part, max(w.slot, 0));
      const uint32_t tm_o = tmem + lane_off + uint32_t(256 + t * D);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        if (has) {
          tmem_ld32(tm_o + c * 32, r);
          tmem_ld_wait();
          tmem_ld_fence(r);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        if (l == 0.0f) {     // sees none of the keys: zero, whatever their values made of its zeros
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        if (valid && w.slot >= 0) {
          if (kFp8) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * inv);
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) st_global_v8(part + Part<D>::piece(4 * c + v, t * kBM + r_in_tile), r + v * 8);
        } else if (valid) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
          // 32 bytes a store where O is aligned so
          if ((reinterpret_cast<uintptr_t>(p.o) & 31) == 0) {
            st_global_v8(dst + c * 32, pk);
            st_global_v8(dst + c * 32 + 16, pk + 8);
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              reinterpret_cast<uint4*>(dst)[c * 4 + v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
          }
        }
      }
      if (valid) {
        if (w.slot >= 0) {
          *reinterpret_cast<float4*>(Part<D>::stat(p.part, w.slot) + (t * kBM + r_in_tile) * Part<D>::kStat) =
              make_float4(m, l, lr, 0.0f);
        } else {
          const size_t li = p.s.cu ? (size_t)head * p.s.Sn + w.q0 + tok : ((size_t)w.b * p.Hq + head) * p.s.Sn + tok;
          p.lse[li] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        }
      }
      if (has) tc_fence_before();
    }
  }
}

// Four MMAs in one piece of PTX, issued by one elected lane of the (converged)
// warp: one election instead of four, and only the operands' base words live
// across it.  Offsets are in units of 16 bytes (descriptors) or TMEM columns.
// The first MMA accumulates if acc != 0, the others always do.
// D[tmem] (+)= A[smem] B[smem]: steps k at offset + 2 k in both operands.
template <uint32_t OFF>
FA_DEV void mma4_ss(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b32 al, bl;\n\t.reg .b64 ad, bd;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "add.u32 al, %1, %7;\n\tadd.u32 bl, %3, %7;\n\tmov.b64 ad, {al, %2};\n\tmov.b64 bd, {bl, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, p;\n\t"
      "add.u32 al, %1, %7 + 2;\n\tadd.u32 bl, %3, %7 + 2;\n\tmov.b64 ad, {al, %2};\n\tmov.b64 bd, {bl, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, 1;\n\t"
      "add.u32 al, %1, %7 + 4;\n\tadd.u32 bl, %3, %7 + 4;\n\tmov.b64 ad, {al, %2};\n\tmov.b64 bd, {bl, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, 1;\n\t"
      "add.u32 al, %1, %7 + 6;\n\tadd.u32 bl, %3, %7 + 6;\n\tmov.b64 ad, {al, %2};\n\tmov.b64 bd, {bl, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, 1;\n\t}\n" ::"r"(d),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc), "n"(OFF)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A at 8 columns, B at 128 units per step.
template <uint32_t FIRST>
FA_DEV void mma4_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b32 at, bl;\n\t.reg .b64 bd;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "add.u32 at, %1, %6 * 8;\n\tadd.u32 bl, %2, %6 * 128;\n\tmov.b64 bd, {bl, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [at], bd, %4, p;\n\t"
      "add.u32 at, %1, %6 * 8 + 8;\n\tadd.u32 bl, %2, %6 * 128 + 128;\n\tmov.b64 bd, {bl, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [at], bd, %4, 1;\n\t"
      "add.u32 at, %1, %6 * 8 + 16;\n\tadd.u32 bl, %2, %6 * 128 + 256;\n\tmov.b64 bd, {bl, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [at], bd, %4, 1;\n\t"
      "add.u32 at, %1, %6 * 8 + 24;\n\tadd.u32 bl, %2, %6 * 128 + 384;\n\tmov.b64 bd, {bl, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [at], bd, %4, 1;\n\t}\n" ::"r"(d),
      "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc), "n"(FIRST)
      : "memory");
}

// MMA issue (a converged warp, one elected lane): S of both tiles for the first
// block, then per block and tile PV(j), S(j + 1).  S(j + 1) overwrites the
// columns of P(j) only after PV(j) was issued; MMAs of one thread run in order.
// One copy of each product's code serves both tiles and the first block: this
// warp comes by once in some thousand cycles, in between the softmax warps'
// long code has pushed its own out of the instruction cache, and with six
// unrolled copies fetching it took longer than the products.
template <int D, bool kFp8>
__device__ void mma_role(const Shared<D, kFp8>& sh, const uint32_t tmem, const PagedAttnParams& p) {
  using L = Layout<D, kFp8>;
  // E4M3: both operands of both products are FP16 (format 0 in place of BF16's 1)
  constexpr uint32_t kFormats = kFp8 ? (1u << 7) | (1u << 10) : 0u;
  constexpr uint32_t kIdS = idesc_bf16_f32(kBM, kBN, false, false) & ~kFormats;
  constexpr uint32_t kIdPV = idesc_bf16_f32(kBM, D, false, true) & ~kFormats;
  const int tt = tile_tokens(p.group);
  uint32_t uit = 0;
  uint32_t sit = 0;      // phase bits of the two tiles
  int stage = 0;
  uint32_t phase = 0;
  // S_t = Q_t K^T in K steps of 16: step k reads 64-element chunk k / 4 at byte
  // offset 32 (k % 4) of its rows.
  auto issue_s = [&](int t, int st) {
    const uint64_t da = sdesc_sw128(sh.sbase + L::kQ + t * L::kTileBytes, 16, 1024);
    const uint64_t db = sdesc_sw128(sh.sbase + L::kKV + st * L::kTileBytes, 16, 1024);
    mma4_ss<0>(tmem + t * kBN, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kIdS, 0u);
    if (D == 128)
      mma4_ss<L::kChunkBytes / 16>(tmem + t * kBN, desc_lo(da), desc_hi(da), desc_lo(db), desc_hi(db), kIdS, 1u);
    mma_commit_w(sh.s_full(t));
  };
  // O_t (+)= P_t V in K steps of 16 keys: TMEM columns 8 k.. of P, key rows
  // 16 k.. (2048 bytes further) of V.
  auto issue_pv = [&](int t, int st, bool acc, uint32_t ph) -> bool {
    const uint64_t db = sdesc_sw128(sh.sbase + L::kKV + st * L::kTileBytes, L::kChunkBytes, 1024);
    mma4_ts<0>(tmem + 256 + t * D, tmem + t * kBN, desc_lo(db), desc_hi(db), kIdPV, acc ? 1u : 0u);
    if (!sh.wait(sh.p_hi(t), ph, kSiteP, p)) return false;
    tc_fence_after();
    mma4_ts<4>(tmem + 256 + t * D, tmem + t * kBN, desc_lo(db), desc_hi(db), kIdPV, 1u);
    return true;
  };
  struct Pos {
    int stage;
    uint32_t phase;
  };
  auto take = [&]() {
    const Pos r{stage, phase};
    if (++stage == L::kStages) {
      stage = 0;
      phase ^= 1;
    }
    return r;
  };
  auto ready = [&](Pos r) -> bool {
    if (!sh.wait(sh.kv_full(r.stage), r.phase, kSiteKvFull, p)) return false;
    tc_fence_after();
    return true;
  };
  SegReader<D, kFp8> in(sh, p);
  Seg w;
  while (in.next(w)) {
    const int n0 = tile_blocks(w, 0, tt, p.causal), n1 = tile_blocks(w, 1, tt, p.causal);
    const int n = max(n0, n1);
    if (n == 0) continue;
    if (!sh.wait(kFp8 ? sh.q_ready() : sh.q_full(), uit & 1, kSiteQFull, p)) return;
    tc_fence_after();
    Pos kp = take(), vp{0, 0u};
    if (!ready(kp)) return;
#pragma unroll 1
    for (int j = -1; j < n; ++j) {
      const bool more = j + 1 < n;
      bool k_ready = j < 0;
      if (j >= 0) {
        vp = take();
        if (!ready(vp)) return;
        if (more) kp = take();
      }
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int nt = t ? n1 : n0;
        if (j >= nt) continue;
        if (j >= 0) {
          const uint32_t ph = (sit >> t) & 1;
          sit ^= 1u << t;
          if (!sh.wait(sh.o_ready(t), ph, kSiteO, p)) return;
          tc_fence_after();
          if (!issue_pv(t, vp.stage, j > 0, ph)) return;
          if (t == 1 || j >= n1) mma_commit_w(sh.kv_empty(vp.stage));
        }
        if (j + 1 < nt) {
          if (!k_ready && !ready(kp)) return;
          k_ready = true;
          issue_s(t, kp.stage);
        } else if (j >= 0) {
          mma_commit_w(sh.o_full(t));
        }
      }
      if (more) {
        mma_commit_w(sh.kv_empty(kp.stage));
        if (j + 1 == n - 1) mma_commit_w(sh.q_empty());
      }
    }
    ++uit;
  }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(Layout<D, kFp8>::kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const PagedAttnParams p) {
  using L = Layout<D, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32;
  Shared<D, kFp8> sh;
  sh.base = smem;
  sh.sbase = smem_u32(smem);

  if (threadIdx.x == 0) {
    mbar_init(sh.q_full(), 1);
    mbar_init(sh.q_empty(), 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(sh.kv_full(s), kFp8 ? 4 : 1);      // one arrival per widening warp
      mbar_init(sh.kv_empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(sh.s_full(t), 1);
      mbar_init(sh.p_lo(t), kBM);
      mbar_init(sh.p_hi(t), kBM);
      mbar_init(sh.o_ready(t), kBM);
      mbar_init(sh.o_full(t), 1);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(sh.seg_full(s), 1);
      mbar_init(sh.seg_empty(s), L::kReaders);
    }
    for (int s = 0; s < (kFp8 ? 0 : L::kStages); ++s) mbar_init(sh.v_landed(s), 1);
    if (kFp8) {
      mbar_init(sh.q_ready(), 8);
      mbar_init(sh.tops_full(), 8);
    }
    for (int s = 0; s < L::kRaws; ++s) {
      mbar_init(sh.raw_full(s), 1);
      mbar_init(sh.raw_empty(s), 4);
    }
    st_shared(sh.abort(), 0);
    Part<D>::join(p.part, blockIdx.x)->parts = 0;      // the scheduler's to fill; after a give-up it stays
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 13) {
    tmem_alloc(sh.tmem_slot(), 512);
    tmem_relinquish();
  }
  const Line line = build_line(p, reinterpret_cast<long long*>(smem + L::kKPre), reinterpret_cast<int*>(smem + L::kUPre),
                               reinterpret_cast<long long*>(smem + L::kSums), gridDim.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sh.tmem_slot();

  if (warp < 8) {
    reg_alloc<kFp8 ? 128 : 192>();
    softmax_role<D, kFp8>(warp / 4, sh, tmem, p);
  } else if (warp < 12) {
    reg_dealloc<kFp8 ? 72 : 80>();
    correction_role<D, kFp8>(sh, tmem, p);
  } else if (warp < 16) {
    reg_dealloc<kFp8 ? 56 : 48>();
    if (warp == 12) {
      load_role<D, kFp8>(sh, &tm_q, &tm_k, &tm_v, p);
    } else if (warp == 13) {
      mma_role<D, kFp8>(sh, tmem, p);
    } else if (warp == 14) {
      if constexpr (!kFp8) clean_role<D>(sh, p);
    } else {
      scheduler_role<D, kFp8>(sh, p, line);
    }
  } else {
    if constexpr (kFp8) {
      reg_dealloc<48>();
      widen_role<D>(sh, p);
    }
  }

  // After a give-up, copies and MMAs in flight land before the memory they target is
  // released: one warp stays for that, when all roles have ended.  (With every warp
  // staying, ahead of the barrier, those of 48 registers among them, a give-up over
  // E4M3 pages ended in a launch failure.)
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    if (ld_shared_volatile(sh.abort())) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
      __syncwarp();
    }
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the units that borders between stretches cut: block
// (x, y) does rows [32 y, 32 y + 32) of the unit whose first cut is border x + 1.
constexpr int kJoinThreads = 256, kJoinRows = 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const PagedAttnParams p) {
  __shared__ float fac[kMaxCtas + 1][kJoinRows];
  __shared__ float inv[kJoinRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = blockIdx.x + 1;
  const int row0 = blockIdx.y * kJoinRows;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  // 16 bytes a thread at a time, as they lie in the workspace; the rows are put
  // together in shared memory
  constexpr int kEach = kJoinRows * (D / 4) / kJoinThreads;
  const int r = threadIdx.x / 2 % kJoinRows, half = threadIdx.x % 2;
  const int piece0 = threadIdx.x / (2 * kJoinRows);
  constexpr int kPieces = kJoinThreads / (2 * kJoinRows);        // at a time
  auto stat_of = [&](int k) {
    return *reinterpret_cast<const float4*>(Part<D>::stat(p.part, paged::join_slot(c, k)) + (row0 + lane) * Part<D>::kStat);
  };
  auto part_of = [&](int k, int e) {
    return *reinterpret_cast<const float4*>(Part<D>::out(p.part, paged::join_slot(c, k)) +
                                            Part<D>::piece(piece0 + e * kPieces, row0 + r) + half * 4);
  };
  // Which slots the parts are in is known before how many there are; the first two
  // are loaded along with that (they hold anything where nothing is joined).
  constexpr int kAhead = 2;
  const paged::Join j = *Part<D>::join(p.part, c);
  float4 st0[kAhead], x0[kAhead][kEach];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    st0[k] = stat_of(k);
#pragma unroll
    for (int e = 0; e < kEach; ++e) x0[k][e] = part_of(k, e);
  }
  const int tt = tile_tokens(p.group);
  const int tok0 = j.row0 + row0 / kBM * tt;                // of the rows' tile
  if (j.parts == 0 || tok0 >= j.n) return;
  // The parts' factors, one row a lane: 2^(maximum - the row's largest).
  if (warp == 0) {
    float mt = fmaxf(st0[0].x, st0[1].x), lt = 0.0f, lrt = 0.0f;
#pragma unroll 4
    for (int k = kAhead; k < j.parts; ++k) mt = fmaxf(mt, stat_of(k).x);
    auto take = [&](int k, const float4& st) {
      const float f = mt == -INFINITY ? 1.0f : ex2_mufu(st.x - mt);
      fac[k][lane] = f;
      lt += st.y * f;
      lrt += st.z * f;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) take(k, st0[k]);
#pragma unroll 4
    for (int k = kAhead; k < j.parts; ++k) take(k, stat_of(k));
    inv[lane] = lrt == 0.0f ? 0.0f : 1.0f / lrt;
    const int in_tile = (row0 + lane) % kBM, tk = in_tile / p.group;
    const int tok = tok0 + tk;
    if (tk < tt && tok < j.n) {
      const int head = j.head * p.group + in_tile - tk * p.group;
      const size_t li = p.s.cu ? (size_t)head * p.s.Sn + j.q0 + tok : ((size_t)j.b * p.Hq + head) * p.s.Sn + tok;
      p.lse[li] = lt == 0.0f ? -INFINITY : (mt + log2f(lt)) * 0.693147180559945309f;
    }
  }
  __syncthreads();
  // (rows that no part wrote hold anything, and are not stored)
  float4 y[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) y[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](int e, const float4& x, float f) {
    y[e].x += x.x * f;
    y[e].y += x.y * f;
    y[e].z += x.z * f;
    y[e].w += x.w * f;
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
#pragma unroll
    for (int e = 0; e < kEach; ++e) add(e, x0[k][e], fac[k][r]);
#pragma unroll 2
  for (int k = kAhead; k < j.parts; ++k) {
    const float f = fac[k][r];
#pragma unroll
    for (int e = 0; e < kEach; ++e) add(e, part_of(k, e), f);
  }
  __shared__ uint2 rows[kJoinRows][D / 4 + 1];
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    rows[r][2 * (piece0 + e * kPieces) + half] =
        make_uint2(pack_bf16x2(y[e].x * inv[r], y[e].y * inv[r]), pack_bf16x2(y[e].z * inv[r], y[e].w * inv[r]));
  __syncthreads();
  for (int i = threadIdx.x; i < kJoinRows * (D / 4); i += kJoinThreads) {
    const int row = i / (D / 4), d = i % (D / 4);
    const int in_tile = (row0 + row) % kBM, tk = in_tile / p.group;
    const int tok = tok0 + tk;
    if (tk >= tt || tok >= j.n) continue;
    const int head = j.head * p.group + in_tile - tk * p.group;
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + ((size_t)(j.q0 + tok) * p.Hq + head) * D)[d] = rows[row][d];
  }
}

template <int D, bool kFp8>
fa_status launch_inst(const PagedAttnLaunch& L, cudaStream_t stream) {
  using Lay = Layout<D, kFp8>;
  const PagedSeqs& s = L.p.s;
  const int page_size = 1 << s.page_shift;
  const long long page_heads = (long long)s.num_pages * s.Hkv;
  const int box = page_size < kBN ? page_size : kBN;
  CUtensorMap tq, tk, tv;
  fa_status st;
  const int rows = s.cu ? s.Sn : s.B * s.Sn;
  if ((st = make_tmap_rows_group(&tq, L.p.q, rows, L.p.Hq, D, L.p.group, kBM / L.p.group)) != FA_OK) return st;
  if ((st = make_tmap_pages(&tk, L.k_pages, page_heads, page_size, D, kFp8, box)) != FA_OK) return st;
  if ((st = make_tmap_pages(&tv, L.v_pages, page_heads, page_size, D, kFp8, box)) != FA_OK) return st;
  auto kern = chunk_kernel<D, kFp8>;
  if ((st = prepare_kernel(reinterpret_cast<const void*>(kern), Lay::kBytes)) != FA_OK) return st;
  // (Not overlapped with the kernel before it, unlike the decode kernel: small calls
  // would gain 2 us, but blocks then land on whichever SMs are free, away from
  // those that share their keys: 16 x 512 E4M3 tokens over 4096 keys 476 -> 497 us.)
  const int ctas = L.p.num_ctas;
  kern<<<ctas, Lay::kThreads, Lay::kBytes, stream>>>(tq, tk, tv, L.p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (ctas == 1) return FA_OK;
  return launch_overlapped(combine_kernel<D>, dim3(ctas - 1, 2 * kBM / kJoinRows), kJoinThreads, 0, stream, L.p);
}

}  // namespace pchunk

size_t paged_chunk_workspace(int D) { return D == 128 ? pchunk::Part<128>::bytes() : pchunk::Part<64>::bytes(); }

fa_status launch_paged_chunk(const PagedAttnLaunch& L, cudaStream_t stream) {
  if (L.D == 128) return L.fp8 ? pchunk::launch_inst<128, true>(L, stream) : pchunk::launch_inst<128, false>(L, stream);
  return L.fp8 ? pchunk::launch_inst<64, true>(L, stream) : pchunk::launch_inst<64, false>(L, stream);
}

fa_status paged_chunk_take_device_error() {
  DeviceError e{0, 0};
  if (cudaMemcpyFromSymbol(&e, pchunk::g_err, sizeof(e)) != cudaSuccess) return FA_ERR_CUDA;
  if (e.status != 0) {
    const DeviceError z{0, 0};
    if (cudaMemcpyToSymbol(pchunk::g_err, &z, sizeof(z)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return static_cast<fa_status>(e.status);
}

}  // namespace fa
