// Masks and depths of trees of drafted tokens, from their parents.
//
// Bit j of token i's mask: j is i or an ancestor of it.  depth(i): how many proper
// ancestors it has.
//
// A tree has some tens of tokens, so the call is a launch, two round trips to
// memory and what depends on one another in between.  A block takes a sequence, a
// warp 32 tokens, one word of the masks.  The ancestors within the word come by
// doubling the step in five shuffles; since a parent comes before its child, the
// lowest of them is the last, and its parent, in an earlier word, is where the way up
// goes on.  Each thread then walks up a word at a time, and writes its mask's words
// on the way.  (256 packed trees of up to 200 tokens: 3.2 us on the GPU, a call 14;
// walking from parent to parent a call took 23.  One tree of 25: 1.1 us and 11.)
#include <cuda_runtime.h>

#include "paged.cuh"

namespace fa {
namespace tree {

__device__ DeviceError g_err;

enum Site { kSiteOffsets = 1, kSiteParent };

__global__ void __launch_bounds__(kMaxTree) mask_kernel(const TreeParams p) {
  __shared__ uint32_t within[kMaxTree];      // ancestors in a token's own word, itself among them
  __shared__ int above[kMaxTree];            // where the way up leaves the word; -1: nowhere
  overlap_launches();
  const int b = blockIdx.x, i = threadIdx.x, lane = i % 32;
  int q0 = b * p.Sn, n = p.Sn;
  if (p.cu) {
    q0 = p.cu[b];
    n = p.cu[b + 1] - q0;
    if (q0 < 0 || n < 0 || n > p.max_q || q0 > p.Sn - n || (b == 0 && q0 != 0)) {
      if (i == 0) paged::record_bad_input(&g_err, kSiteOffsets);
      return;
    }
  }
  int parent = -1;
  if (i < n) {
    parent = p.parents[(size_t)q0 + i];
    if (parent < -1 || parent >= i) {      // a token without a place in the tree stands alone
      paged::record_bad_input(&g_err, kSiteParent);
      parent = -1;
    }
  }
  uint32_t bits = 1u << lane;
  int at = parent >= i - lane ? parent & 31 : lane;      // 1, 2, 4, ... steps up, as far as the word goes
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    bits |= __shfl_sync(0xffffffffu, bits, at);
    at = __shfl_sync(0xffffffffu, at, at);
  }
  int up = __shfl_sync(0xffffffffu, parent, __ffs(bits) - 1);
  within[i] = bits;
  above[i] = up;
  __syncthreads();
  if (i >= n) return;
  uint32_t* row = p.mask + ((size_t)q0 + i) * p.words;
  int depth = -1;
  int w = p.words - 1;
  for (; w > i >> 5; --w) row[w] = 0u;
  for (;;) {
    row[w--] = bits;
    depth += __popc(bits);
    if (up < 0) break;
    for (; w > up >> 5; --w) row[w] = 0u;
    bits = within[up];
    up = above[up];
  }
  for (; w >= 0; --w) row[w] = 0u;
  p.depth[(size_t)q0 + i] = depth;
}

}  // namespace tree

fa_status launch_tree_mask(const TreeParams& p, cudaStream_t stream) {
  return launch_overlapped(tree::mask_kernel, dim3(p.B), (p.max_q + 31) / 32 * 32, 0, stream, p);
}

fa_status tree_take_device_error() {
  DeviceError e{0, 0};
  if (cudaMemcpyFromSymbol(&e, tree::g_err, sizeof(e)) != cudaSuccess) return FA_ERR_CUDA;
  if (e.status != 0) {
    const DeviceError z{0, 0};
    if (cudaMemcpyToSymbol(tree::g_err, &z, sizeof(z)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return static_cast<fa_status>(e.status);
}

}  // namespace fa
