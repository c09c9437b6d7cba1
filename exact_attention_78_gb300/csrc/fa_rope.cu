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
// heads of q and k, and rows move in 16-byte pieces.
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
// (i, i + R) at any R: a thread's piece meets its partners one by one.
enum Layout { kHalf, kAdjacent, kAny };

template <int D, Layout kLayout>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[kMaxTb * (D / 2)];      // cos, sin of each token's pairs
  const int R = p.pairs;
  const int tok0 = blockIdx.x * p.tb;
  const int ntok = min(p.tb, p.tokens - tok0);
  for (int i = threadIdx.x; i < ntok * R; i += kThreads) {
    const int t = i / R, pair = i - t * R;
    const long long pos = p.positions[(size_t)p.axis[pair] * p.tokens + tok0 + t];
    const unsigned long long frac = (unsigned long long)pos * p.turn[pair];
    float s, c;
    sincospif((float)(int)(frac >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    cs[t * (D / 2) + pair] = make_float2(c, p.inverse ? -s : s);
  }
  __syncthreads();

  const int heads = p.Hq + p.Hkv;
  // 16-byte pieces of a row; kHalf: the thread of piece j < R / 8 also does
  // piece j + R / 8, and the pieces from 2 R / 8 on are copied
  constexpr int kPieces = D / 8;
  const int half = R / 8;
  const int work = kLayout == kHalf ? kPieces - half : kPieces;
  for (int i = threadIdx.x; i < ntok * heads * work; i += kThreads) {
    const int row = i / work;
    int j = i - row * work;
    const int t = row / heads, h = row - t * heads;
    const bool is_k = h >= p.Hq;
    const size_t at = ((size_t)(tok0 + t) * (is_k ? p.Hkv : p.Hq) + (is_k ? h - p.Hq : h)) * D;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_k ? p.k : p.q) + at;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_k ? p.k_out : p.q_out) + at;
    const float2* c = cs + t * (D / 2);
    if constexpr (kLayout == kHalf) {
      if (j >= half) {
        j += half;
        reinterpret_cast<uint4*>(dst)[j] = reinterpret_cast<const uint4*>(src)[j];
        continue;
      }
      const uint4 a4 = reinterpret_cast<const uint4*>(src)[j], b4 = reinterpret_cast<const uint4*>(src)[j + half];
      const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
      uint32_t ya[4], yb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 c0 = c[8 * j + 2 * e], c1 = c[8 * j + 2 * e + 1];
        const float a0 = lo_of(a[e]), a1 = hi_of(a[e]), b0 = lo_of(b[e]), b1 = hi_of(b[e]);
        ya[e] = pack_bf16x2(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
        yb[e] = pack_bf16x2(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
      }
      reinterpret_cast<uint4*>(dst)[j] = make_uint4(ya[0], ya[1], ya[2], ya[3]);
      reinterpret_cast<uint4*>(dst)[j + half] = make_uint4(yb[0], yb[1], yb[2], yb[3]);
    } else if constexpr (kLayout == kAdjacent) {
      const uint4 x4 = reinterpret_cast<const uint4*>(src)[j];
      const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int pair = 4 * j + e;
        y[e] = x[e];
        if (pair < R) {
          const float2 cc = c[pair];
          const float a0 = lo_of(x[e]), b0 = hi_of(x[e]);
          y[e] = pack_bf16x2(a0 * cc.x - b0 * cc.y, b0 * cc.x + a0 * cc.y);
        }
      }
      reinterpret_cast<uint4*>(dst)[j] = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  if constexpr (kLayout == kAny) {
    // A row's D / 8 lanes take a piece each; partners come from the row's copy
    // in shared memory, so that the rows may be turned in place.
    __shared__ float rows[kThreads * 8];
    const int lane = threadIdx.x % kPieces, group = threadIdx.x / kPieces;
    constexpr int kGroups = kThreads / kPieces;
    float* mine = rows + group * D;
    for (int r0 = 0; r0 < ntok * heads; r0 += kGroups) {
      const int row = r0 + group;
      const bool on = row < ntok * heads;
      const int t = row / heads, h = row - t * heads;
      const bool is_k = h >= p.Hq;
      const size_t at = ((size_t)(tok0 + t) * (is_k ? p.Hkv : p.Hq) + (is_k ? h - p.Hq : h)) * D;
      if (on) {
        const uint4 x4 = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(is_k ? p.k : p.q) + at)[lane];
        const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mine[8 * lane + 2 * e] = lo_of(x[e]);
          mine[8 * lane + 2 * e + 1] = hi_of(x[e]);
        }
      }
      __syncwarp();
      if (on) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = 8 * lane + e;
          y[e] = mine[i];
          if (i < 2 * R) {
            const float2 cc = cs[t * (D / 2) + (i < R ? i : i - R)];
            y[e] = i < R ? mine[i] * cc.x - mine[i + R] * cc.y : mine[i] * cc.x + mine[i - R] * cc.y;
          }
        }
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_k ? p.k_out : p.q_out) + at)[lane] =
            make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                       pack_bf16x2(y[6], y[7]));
      }
      __syncwarp();
    }
  }
}

template <int D>
fa_status launch_d(RopeParams p, int num_sms, cudaStream_t stream) {
  // one token per block while that does not fill the SMs
  p.tb = 1;
  while (p.tb < kMaxTb && (long long)p.tokens >= (long long)num_sms * 4 * p.tb) p.tb *= 2;
  const int grid = (p.tokens + p.tb - 1) / p.tb;
  if (p.interleaved)
    rope_kernel<D, kAdjacent><<<grid, kThreads, 0, stream>>>(p);
  else if (p.pairs % 8 == 0)
    rope_kernel<D, kHalf><<<grid, kThreads, 0, stream>>>(p);
  else
    rope_kernel<D, kAny><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace rope

fa_status launch_rope(const RopeParams& p, int num_sms, cudaStream_t stream) {
  return p.D == 128 ? rope::launch_d<128>(p, num_sms, stream) : rope::launch_d<64>(p, num_sms, stream);
}

}  // namespace fa
