// Rotary positions with several axes, on queries and keys in one launch.
//
// Each rotary pair (x_a, x_b) of a row turns by position * frequency:
//   y_a = x_a cos - x_b sin,   y_b = x_b cos + x_a sin.
// The angle is taken in turns: a pair's frequency is a 64-bit fraction of a
// turn per position, and the product with the position, modulo 2^64, is the
// angle's fraction of a turn with no range reduction to lose bits in (FP32
// angles are off by 0.01 rad at position 200,000).  Its upper 32 bits go to
// sincospif.
//
// HBM bounds the kernel at training sizes (a row is read once and written
// once), so each angle is computed once per token, into shared memory, for all
// heads of q and k, and rows move in 16-byte pieces, several in flight per
// thread; the first ones are on their way while the angles are computed.
#include <cuda_runtime.h>

#include "paged.cuh"

namespace fa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxTb = 4;      // tokens per thread block

FA_DEV float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
FA_DEV float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// kHalf: pairs (i, i + R), R a multiple of 8, so that a 16-byte piece of
// first elements has its partners in one other aligned piece and a thread
// turns both.  kAdjacent: pairs (2 i, 2 i + 1), inside one piece.  kAny: pairs
// (i, i + R) at any R: a thread's piece meets its partners one by one, in the
// row's copy in shared memory.  16,384 tokens x 32 heads, D = 128: kHalf 41.1 us at
// R = 64 (6.5 TB/s), kAny 70, 92, 88 and 73 us at R = 63, 60, 44 and 20, kAdjacent 48.
enum Layout { kHalf, kAdjacent, kAny };

// 16-byte pieces that one thread loads and stores at a time.
struct Piece {
  uint4 a, b;      // b: the partners' (kHalf)
};

template <int D, Layout kLayout>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPieces = D / 8;                // of a row
  constexpr int kPer = kLayout == kAdjacent ? 4 : 8;        // pairs of a piece
  constexpr int kUnroll = kLayout == kHalf ? 2 : 4;
  // cos, sin of each token's pairs, pair i at (i mod kPer) (pairs / kPer) +
  // i / kPer: lanes with neighbouring pieces read neighbouring entries
  constexpr int kStride = D / 2 / kPer;
  __shared__ float2 cs[kMaxTb][D / 2];
  __shared__ uint4 copy[kLayout == kAny ? kThreads : 1];
  const int R = p.pairs;
  const int tok0 = blockIdx.x * p.tb;
  const int ntok = min(p.tb, p.tokens - tok0);

  // A thread does one piece of every step's row: piece j (kHalf: and j + R / 8;
  // the pieces from 2 R / 8 on are copied).
  const int half = R / 8;
  const int work = kLayout == kHalf ? kPieces - half : kPieces;
  const int step = kThreads / work;             // rows a step
  const int first = threadIdx.x / work;
  int j = threadIdx.x - first * work;
  const bool turns = kLayout != kHalf || j < half;
  if (!turns) j += half;
  const int nq = ntok * p.Hq, n = nq + ntok * p.Hkv;        // rows of q, of both
  const uint4* q = static_cast<const uint4*>(p.q) + (size_t)tok0 * p.Hq * kPieces;
  const uint4* k = static_cast<const uint4*>(p.k) + (size_t)tok0 * p.Hkv * kPieces;
  uint4* q_out = static_cast<uint4*>(p.q_out) + (size_t)tok0 * p.Hq * kPieces;
  uint4* k_out = static_cast<uint4*>(p.k_out) + (size_t)tok0 * p.Hkv * kPieces;

  auto load = [&](int r0, Piece (&x)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + first + u * step;
      if (first >= step || r >= n) continue;
      const uint4* src = (r < nq ? q + (size_t)r * kPieces : k + (size_t)(r - nq) * kPieces) + j;
      x[u].a = src[0];
      if (kLayout == kHalf && turns) x[u].b = src[half];
    }
  };
  overlap_launches();
  Piece x[kUnroll];
  load(0, x);

  for (int i = threadIdx.x; i < ntok * R; i += kThreads) {
    const int t = i / R, pair = i - t * R;
    const long long pos = p.positions[(size_t)p.axis[pair] * p.tokens + tok0 + t];
    const unsigned long long frac = (unsigned long long)pos * p.turn[pair];
    float s, c;
    sincospif((float)(int)(frac >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    cs[t][pair % kPer * kStride + pair / kPer] = make_float2(c, p.inverse ? -s : s);
  }
  __syncthreads();

  for (int r0 = 0; r0 < n; r0 += kUnroll * step) {
    if (r0 > 0) load(r0, x);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + first + u * step;
      const bool on = first < step && r < n;
      if (kLayout == kAny) {
        // (a row's lanes, 8 or 16 from a multiple of that on, sit in one warp; in
        // place, a thread stores over no piece but its own, which it has loaded)
        __syncwarp();
        if (on) copy[threadIdx.x] = x[u].a;
        __syncwarp();
      }
      if (!on) continue;
      const int in = r < nq ? r : r - nq, heads = r < nq ? p.Hq : p.Hkv;
      const int t = (in >= heads) + (in >= 2 * heads) + (in >= 3 * heads);       // kMaxTb is 4
      uint4* dst = (r < nq ? q_out + (size_t)r * kPieces : k_out + (size_t)in * kPieces) + j;
      const uint32_t a[4] = {x[u].a.x, x[u].a.y, x[u].a.z, x[u].a.w};
      if constexpr (kLayout == kHalf) {
        if (!turns) {
          *dst = x[u].a;
          continue;
        }
        const uint32_t b[4] = {x[u].b.x, x[u].b.y, x[u].b.z, x[u].b.w};
        uint32_t ya[4], yb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 c0 = cs[t][2 * e * kStride + j], c1 = cs[t][(2 * e + 1) * kStride + j];
          const float a0 = lo_of(a[e]), a1 = hi_of(a[e]), b0 = lo_of(b[e]), b1 = hi_of(b[e]);
          ya[e] = pack_bf16x2(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
          yb[e] = pack_bf16x2(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
        }
        dst[0] = make_uint4(ya[0], ya[1], ya[2], ya[3]);
        dst[half] = make_uint4(yb[0], yb[1], yb[2], yb[3]);
      } else if constexpr (kLayout == kAdjacent) {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = a[e];
          if (4 * j + e < R) {
            const float2 cc = cs[t][e * kStride + j];
            const float a0 = lo_of(a[e]), b0 = hi_of(a[e]);
            y[e] = pack_bf16x2(a0 * cc.x - b0 * cc.y, b0 * cc.x + a0 * cc.y);
          }
        }
        *dst = make_uint4(y[0], y[1], y[2], y[3]);
      } else {
        const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(copy + first * kPieces);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = 8 * j + e;
          const float own = e & 1 ? hi_of(a[e / 2]) : lo_of(a[e / 2]);
          y[e] = own;
          if (i < 2 * R) {
            const int pair = i < R ? i : i - R;
            const float other = __bfloat162float(row[i < R ? i + R : pair]);
            const float2 cc = cs[t][pair % kPer * kStride + pair / kPer];
            y[e] = own * cc.x + (i < R ? -other : other) * cc.y;
          }
        }
        *dst = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                          pack_bf16x2(y[6], y[7]));
      }
    }
  }
}

template <int D>
fa_status launch_d(RopeParams p, int num_sms, cudaStream_t stream) {
  // one token per block while that does not fill the SMs
  p.tb = 1;
  while (p.tb < kMaxTb && (long long)p.tokens >= (long long)num_sms * 4 * p.tb) p.tb *= 2;
  const int grid = (p.tokens + p.tb - 1) / p.tb;
  auto kernel = p.interleaved ? rope_kernel<D, kAdjacent> : p.pairs % 8 == 0 ? rope_kernel<D, kHalf> : rope_kernel<D, kAny>;
  return launch_overlapped(kernel, dim3(grid), kThreads, 0, stream, p);
}

}  // namespace rope

fa_status launch_rope(const RopeParams& p, int num_sms, cudaStream_t stream) {
  return p.D == 128 ? rope::launch_d<128>(p, num_sms, stream) : rope::launch_d<64>(p, num_sms, stream);
}

}  // namespace fa
