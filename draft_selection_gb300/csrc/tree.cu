// Trees of drafted tokens: what each node sees, and the path of the target's
// tokens through the tree (include/dfl2.h).  A few integers per node: both are
// bound by the latency of their dependent steps (3.3 and 3.0 us for a chain of 17, 3.7 and
// 3.6 for 64 trees of 33 nodes; ncu, caches flushed), about 2 us of which is a launch.
#include <cuda_runtime.h>

#include "cache.cuh"

namespace dfl2 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kNodesPerLane = kMaxTree / 32;

struct MaskArgs {
  const int32_t* parents;
  const int32_t* count;
  uint32_t* mask;
  int32_t* depth;
  int T, W;
  uint32_t* err;
};

// One CTA a tree, a thread a node: up the chain of parents in shared memory, a
// bit at a time, about 30 cycles a step (a tree of 33 nodes is rarely deeper than 20).
__global__ void __launch_bounds__(kMaxTree) tree_mask_kernel(const __grid_constant__ MaskArgs a) {
  __shared__ int16_t par[kMaxTree];
  __shared__ uint32_t bits[kMaxTree][kMaxTree / 32 + 1];  // +1: rows on different banks
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x, i = threadIdx.x;
  int p = i < a.T ? a.parents[static_cast<int64_t>(b) * a.T + i] : -1;  // beside the count
  const int n = a.count ? max(0, min(a.T, a.count[b])) : a.T;
  if (i < n) {
    if (p < -1 || p >= i) {
      record_error(a.err, kDevErrBadIndex);
      p = -1;
    }
    par[i] = static_cast<int16_t>(p);
  }
  if (i < a.T)
    for (int w = 0; w < a.W; ++w) bits[i][w] = 0;
  __syncthreads();
  if (i < a.T) {
    int up = -1;
    if (i < n)
      for (int j = i; j >= 0; j = par[j]) {
        bits[i][j >> 5] |= 1u << (j & 31);
        ++up;
      }
    if (a.depth) a.depth[static_cast<int64_t>(b) * a.T + i] = max(0, up);
  }
  __syncthreads();
  uint32_t* out = a.mask + static_cast<int64_t>(b) * a.T * a.W;
  for (int x = i; x < a.T * a.W; x += blockDim.x) out[x] = bits[x / a.W][x % a.W];
}

struct AcceptArgs {
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* target;
  const int32_t* count;
  int32_t* path;
  int32_t* n_path;
  int32_t* next;
  int B, T;
};

// One warp a tree, each lane up to eight nodes in registers: a step down is one
// comparison per node, a warp-wide minimum and a shuffle.  A child's number is above its
// parent's, so there are at most T steps whatever the parents hold.
__global__ void __launch_bounds__(128) tree_accept_kernel(const __grid_constant__ AcceptArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= a.B) return;
  const int64_t at = static_cast<int64_t>(b) * a.T;
  int tok[kNodesPerLane], par[kNodesPerLane], tgt[kNodesPerLane];
#pragma unroll
  for (int j = 0; j < kNodesPerLane; ++j) {  // all loads at once, the count's beside them
    const int i = lane + 32 * j;
    tok[j] = i < a.T ? a.tokens[at + i] : 0;
    par[j] = i < a.T ? a.parents[at + i] : -2;
    tgt[j] = i < a.T ? a.target[at + i] : -1;
  }
  const int n = a.count ? max(0, min(a.T, a.count[b])) : a.T;
#pragma unroll
  for (int j = 0; j < kNodesPerLane; ++j)
    if (lane + 32 * j >= n) par[j] = -2;
  int cur = 0, len = 0, want = -1;
  if (n > 0) {
    while (true) {
      int x = tgt[0];
#pragma unroll
      for (int j = 1; j < kNodesPerLane; ++j)
        if (j == cur >> 5) x = tgt[j];
      want = __shfl_sync(kAll, x, cur & 31);
      if (lane == 0) a.path[at + len] = cur;
      ++len;
      unsigned child = 0x7fffffffu;
#pragma unroll
      for (int j = kNodesPerLane - 1; j >= 0; --j) {
        const int i = lane + 32 * j;
        if (par[j] == cur && tok[j] == want && i > cur) child = i;
      }
      child = __reduce_min_sync(kAll, child);
      if (child == 0x7fffffffu) break;
      cur = static_cast<int>(child);
    }
  }
  for (int i = len + lane; i < a.T; i += 32) a.path[at + i] = -1;
  if (lane == 0) {
    a.n_path[b] = len;
    a.next[b] = want;
  }
}

dfl2_status check_tree(int B, int T) {
  if (B < 1 || T < 1)
    return report_errorf(DFL2_ERR_INVALID_ARG, "B=%d and T=%d must be >= 1", B, T);
  if (B > kMaxBatch || T > kMaxTree)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "B=%d, T=%d: at most %d trees of %d nodes", B, T,
                         kMaxBatch, kMaxTree);
  return DFL2_OK;
}

}  // namespace
}  // namespace dfl2

#define DFL2_TRY(expr)              \
  do {                              \
    dfl2_status _st = (expr);       \
    if (_st != DFL2_OK) return _st; \
  } while (0)

extern "C" {

dfl2_status dfl2_tree_mask(const int32_t* parents, int B, int T, const int32_t* count,
                           uint32_t* mask, int32_t* depth, dfl2_stream stream) {
  const dfl2::PtrArg ptrs[] = {{parents, "parents", 4}, {count, "count", 4, true},
                               {mask, "mask", 4}, {depth, "depth", 4, true}};
  DFL2_TRY(dfl2::check_tree(B, T));
  DFL2_TRY(dfl2::check_args_host(ptrs, 4));
  DFL2_TRY(dfl2::check_args_device(ptrs, 4));
  const dfl2::MaskArgs a{parents, count, mask, depth, T, (T + 31) / 32, dfl2::device_error_word()};
  const cudaError_t e = dfl2::launch_k(dfl2::tree_mask_kernel, dim3(B), dim3((T + 31) / 32 * 32), 0,
                                       reinterpret_cast<cudaStream_t>(stream), true, a);
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "tree mask launch");
}

dfl2_status dfl2_tree_accept(const int32_t* tokens, const int32_t* parents,
                             const int32_t* target, int B, int T, const int32_t* count,
                             int32_t* path, int32_t* n_path, int32_t* next_token,
                             dfl2_stream stream) {
  const dfl2::PtrArg ptrs[] = {{tokens, "tokens", 4}, {parents, "parents", 4},
                               {target, "target", 4}, {count, "count", 4, true},
                               {path, "path", 4}, {n_path, "n_path", 4},
                               {next_token, "next_token", 4}};
  DFL2_TRY(dfl2::check_tree(B, T));
  DFL2_TRY(dfl2::check_args_host(ptrs, 7));
  DFL2_TRY(dfl2::check_args_device(ptrs, 7));
  const dfl2::AcceptArgs a{tokens, parents, target, count, path, n_path, next_token, B, T};
  const cudaError_t e =
      dfl2::launch_k(dfl2::tree_accept_kernel, dim3((B + 3) / 4), dim3(128), 0,
                     reinterpret_cast<cudaStream_t>(stream), true, a);
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "tree accept launch");
}

}  // extern "C"
