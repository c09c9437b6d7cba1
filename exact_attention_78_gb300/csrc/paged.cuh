// Device code shared by the paged-cache kernels: which sequence and position a
// new token has, E4M3 rows and their scales.
#pragma once

#include "paged_internal.h"
#include "ptx.cuh"

namespace fa {

// In a kernel started by launch_overlapped(), ahead of its first access to global
// memory: lets the next such launch start once all blocks are here, and waits for
// the end of the kernel before.
FA_DEV void overlap_launches() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

namespace paged {

FA_DEV void record_bad_input(DeviceError* err, int site) {
  if (atomicCAS(&err->status, 0, FA_ERR_INVALID_ARG) == 0) atomicExch(&err->site, site);
}

// A bounded wait of a whole warp, whose lanes all get one answer: a lane that
// gave up alone would leave the others waiting for it at the next __syncwarp.
FA_DEV bool wait_warp(uint32_t bar, uint32_t parity, uint32_t abort, DeviceError* err, int site, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort, err, site, limit_ns));
}

// Scale bytes of the rows of a bad page, which reads as zeros (one box at most).
static __device__ const __align__(128) uint8_t g_no_scales[128] = {};

// The sequence that packed row i belongs to: the number of b in [1, B] with
// cu[b] <= i (B where i lies behind the last sequence).  One warp searches for
// one row, 32 offsets a step: two steps of independent loads for up to 1024
// sequences, where a binary search takes ten dependent ones.
FA_DEV int find_sequence(const int* __restrict__ cu, int B, int i, int lane) {
  const int step = (B + 31) / 32;
  // shares of `step` offsets whose last one is still <= i, then the rest one by one
  const int last = (lane + 1) * step;
  const int full = __popc(__ballot_sync(0xffffffffu, last <= B && cu[min(last, B)] <= i));
  if (step == 1) return full;
  const int b = full * step + 1 + lane;                     // step <= 32
  return full * step + __popc(__ballot_sync(0xffffffffu, lane < step && b <= B && cu[min(b, B)] <= i));
}

// Whether the offsets and lengths of all sequences keep to the rules.  Every
// thread of the block calls it; the answer is the same in all of them.
// max_new: the most new tokens that a sequence may have (packed).
FA_DEV bool sequences_ok(const PagedSeqs& s, int max_new) {
  bool ok = true;
  const int capacity = s.max_pages << s.page_shift;
  for (int b = threadIdx.x; b < s.B; b += blockDim.x) {
    if (s.seq_lens) ok = ok && s.seq_lens[b] >= 0 && s.seq_lens[b] <= capacity;
    if (s.cu) {
      const int a = s.cu[b], e = s.cu[b + 1];
      ok = ok && a >= 0 && e >= a && e <= s.Sn && e - a <= max_new && (b > 0 || a == 0);
      if (!s.seq_lens) ok = ok && e - a <= capacity;
    }
  }
  return __syncthreads_and(ok);
}

// New tokens, keys and first row of sequence b.
struct SeqRows {
  int n, L, q0;
};
FA_DEV SeqRows rows_of(const PagedSeqs& s, int b) {
  SeqRows r;
  r.L = s.seq_lens[b];
  if (s.cu) {
    r.q0 = s.cu[b];
    r.n = s.cu[b + 1] - r.q0;
  } else {
    r.q0 = b * s.Sn;
    r.n = s.Sn;
  }
  return r;
}

// Checks the sequences' offsets and lengths, and sums up their work: `work`
// gives a sequence's, whose prefix sums go to bpre and (if given) upre, [B + 1],
// and the longest unit of all to upre[B + 1].  All threads of the block; false,
// in all of them, when the rules are broken.  Both attention kernels start with
// this, so one pass and two barriers have to do: the loads, the sums within
// warps and the check share the first.  `sums`: two values per warp.
struct Work {
  long long blocks;      // of keys (decode kernel), or keys (chunk kernel)
  int units;
  int longest;           // unit
};
template <class F>
FA_DEV bool prefix_sequences(const PagedSeqs& s, int max_new, F work, long long* bpre, int* upre, long long* sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int capacity = s.max_pages << s.page_shift;
  Work carry{0, 0, 0};
  int ok = 1;
  for (int b0 = 0; b0 < s.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const int warps = (min(s.B - b0, (int)blockDim.x) + 31) / 32;      // with a sequence
    Work own{0, 0, 0}, incl;
    if (b < s.B) {
      const SeqRows r = rows_of(s, b);
      bool fine = r.L >= 0 && r.L <= capacity;
      if (s.cu) fine = fine && r.q0 >= 0 && r.n >= 0 && r.n <= max_new && r.q0 <= s.Sn - r.n && (b > 0 || r.q0 == 0);
      if (fine && r.n > 0) own = work(r);
      ok = ok && fine;
    }
    incl = own;
    if (warp < warps) {
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const long long ob = __shfl_up_sync(0xffffffffu, incl.blocks, d);
        const int ou = __shfl_up_sync(0xffffffffu, incl.units, d);
        if (lane >= d) {
          incl.blocks += ob;
          incl.units += ou;
        }
      }
      const int longest = __reduce_max_sync(0xffffffffu, own.longest);
      if (lane == 31) {
        sums[2 * warp] = incl.blocks;
        sums[2 * warp + 1] = (long long)longest << 32 | (unsigned)incl.units;
      }
    }
    ok = __syncthreads_and(ok);
    Work before = carry;
    for (int w = 0; w < warps; ++w) {
      const long long sb = sums[2 * w];
      const int su = (int)sums[2 * w + 1];
      if (w < warp) {
        before.blocks += sb;
        before.units += su;
      }
      carry.blocks += sb;
      carry.units += su;
      carry.longest = max(carry.longest, (int)(sums[2 * w + 1] >> 32));
    }
    if (b < s.B) {
      bpre[b] = before.blocks + incl.blocks - own.blocks;
      if (upre) upre[b] = before.units + incl.units - own.units;
    }
    if (b0 + (int)blockDim.x >= s.B && threadIdx.x == 0) {
      bpre[s.B] = carry.blocks;
      if (upre) {
        upre[s.B] = carry.units;
        upre[s.B + 1] = carry.longest;
      }
    }
    __syncthreads();
  }
  return ok;
}

// Bits o ... o + 31 of a drafted token's mask `row` in a tree of n (nullptr: sees
// none of the tree), the keys before the tree, o < 0, as ones.
FA_DEV uint32_t tree_bits(const uint32_t* __restrict__ row, int o, int n) {
  const int q = o >> 5, r = o & 31;
  const uint32_t lo = q < 0 ? 0xFFFFFFFFu : row && 32 * q < n ? row[q] : 0u;
  const uint32_t hi = r && row && 32 * (q + 1) < n ? row[q + 1] : 0u;      // (o > -32: q + 1 >= 0)
  const uint32_t bits = __funnelshift_r(lo, hi, r);
  const int left = n - o;                                                  // a row's last bits mean nothing
  return left >= 32 ? bits : left <= 0 ? 0u : bits & ((1u << left) - 1u);
}

// a / b for a >= 0, b > 0: 64-bit division takes some hundred instructions, and
// the numbers here mostly fit 32 bits.
FA_DEV long long div64(long long a, long long b) {
  if ((unsigned long long)(a | b) >> 32 == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

// What the kernels that join partial results need to know of border c between
// thread blocks c - 1 and c.  Thread block c of the main kernel, which knows the
// place, leaves it behind for them: working it out again took as long as the
// joining.
struct Join {
  int parts;       // of the unit whose first cut this border is (two or more); 0: none
  int b, head;
  int row0;        // chunk kernel: the unit's first token; decode kernel: 0
  int n, q0;       // the sequence's new tokens and their first row
  int pad[2];
};
// A thread block's slots: 2 c for the part that begins at the border before it,
// 2 c + 1 for the one that ends at the border behind it (and began at its unit's
// start).  The slot of part k:
FA_DEV int join_slot(int c, int k) { return k == 0 ? 2 * c - 1 : 2 * (c + k - 1); }

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

// 2^e of a scale byte; NaN for the byte of a row without a finite scale.
FA_DEV float scale_value(uint32_t byte) {
  return byte == 255u ? __int_as_float(0x7FC00000) : __uint_as_float(byte << 23);
}

// E4M3 codes to BF16, exactly but for a factor of 2^-120: sign, exponent and
// mantissa move to their places in a BF16, whose exponent then reads 120 too
// low (subnormal codes become subnormal BF16, in the same proportion).  One
// word of four codes gives two pairs, of codes 0 and 2 and of codes 1 and 3.
// Three logic instructions a pair; there is no direct conversion, and the one
// through FP16 and FP32 takes five.
FA_DEV uint32_t e4m3_even_raw(uint32_t w) { return ((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u); }
FA_DEV uint32_t e4m3_odd_raw(uint32_t w) { return ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u); }
// Product of BF16 pairs (subnormals kept).
FA_DEV uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Larger of two BF16 pairs, element by element; NaN if either is.
FA_DEV uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kTwo120 = 0x7B807B80u;   // 2^120 twice
FA_DEV uint32_t e4m3_even(uint32_t w) { return mul_bf16x2(e4m3_even_raw(w), kTwo120); }
FA_DEV uint32_t e4m3_odd(uint32_t w) { return mul_bf16x2(e4m3_odd_raw(w), kTwo120); }

}  // namespace paged
}  // namespace fa
