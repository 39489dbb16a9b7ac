// tree_masks.cu -- which drafted tokens see which, from the parent of each (no counterpart
// in the sources).
//
// A draft's ancestors are found by walking its parents, which are lower and lower: the
// words of its mask are filled from the highest one down, and leave two at a time.  A
// request's parents are in shared memory (32 clocks a step, where global memory would take
// 800), one CTA per request, one thread per draft; drafts are some tens, their depth below
// ten.  Bound by the launch and two dependent round trips (row_start, then parents and ctx_rows
// together): 1024 requests of 1 to 250 drafts 3.6 us (5.2 with 128 threads, contexts after
// the parents and single words).
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kTreeThreads = 256, kMaxWords = 16;

__global__ void __launch_bounds__(kTreeThreads) tree_masks_kernel(const __grid_constant__ TreeMasksArgs a) {
  __shared__ int16_t s_parent[kMaxWords * 64];
  __shared__ int32_t s_ctx[kMaxWords * 64];
  pdl_wait();
  const int32_t T = static_cast<int32_t>(a.T), b = blockIdx.x;
  auto none = [&](int32_t t) {
    for (int w = 0; w < a.words; ++w) a.mask[static_cast<int64_t>(t) * a.words + w] = 0;
    if (a.positions) a.positions[t] = -1;
  };
  if (b >= a.B) {  // what lies behind the last request, spread over the remaining CTAs
    const int32_t end = a.B ? min(max(a.row_start[a.B], 0), T) : 0;
    for (int64_t t = end + static_cast<int64_t>(b - a.B) * kTreeThreads + threadIdx.x; t < T;
         t += static_cast<int64_t>(gridDim.x - a.B) * kTreeThreads)
      none(static_cast<int32_t>(t));
    return;
  }
  const int32_t t0 = min(max(a.row_start[b], 0), T), t1 = min(max(a.row_start[b + 1], 0), T);
  const int32_t n = t1 - t0, most = a.words * 64, used = min(n, most);
  for (int32_t i = threadIdx.x; i < used; i += kTreeThreads) {
    int32_t p = a.parents[t0 + i];
    const int32_t ctx = a.ctx_rows ? a.ctx_rows[t0 + i] : 0;
    s_ctx[i] = ctx;
    if (p < -1 || p >= i) {
      if (ctx >= 0) flag_error(a.err, CKV_DEVERR_PLAN);  // padding has no parent
      p = -1;
    }
    s_parent[i] = static_cast<int16_t>(p);
  }
  __syncthreads();
  const bool pairs = a.words % 2 == 0 && reinterpret_cast<uintptr_t>(a.mask) % 16 == 0;
  for (int32_t i = threadIdx.x; i < n; i += kTreeThreads) {
    const int32_t t = t0 + i, ctx = i < most ? s_ctx[i] : -1;
    if (ctx < 0) {
      if (i >= most && !(a.ctx_rows && a.ctx_rows[t] < 0)) flag_error(a.err, CKV_DEVERR_PLAN);
      none(t);
      continue;
    }
    uint64_t* to = a.mask + static_cast<int64_t>(t) * a.words;
    int32_t depth = 0, p = i;
    auto word = [&](int w) {
      uint64_t m = 0;
      while (p >= w * 64) {  // p is below (w + 1) * 64
        m |= 1ull << (p & 63);
        p = s_parent[p];
        ++depth;
      }
      return m;
    };
    if (pairs) {
      for (int w = a.words - 2; w >= 0; w -= 2) {
        const uint64_t high = word(w + 1);
        *reinterpret_cast<ulonglong2*>(to + w) = make_ulonglong2(word(w), high);
      }
    } else {
      for (int w = a.words - 1; w >= 0; --w) to[w] = word(w);
    }
    if (a.positions) a.positions[t] = ctx + depth - 1;
  }
}

}  // namespace

cudaError_t launch_tree_masks(const TreeMasksArgs& a, bool use_pdl, cudaStream_t s) {
  // rows behind the last request are few (a padded step); their number is not known here
  const int64_t tail = (a.T + 16 * kTreeThreads - 1) / (16 * kTreeThreads);
  return launch_ex(tree_masks_kernel, dim3(static_cast<unsigned>(a.B + (tail < 152 ? tail : 152))), dim3(kTreeThreads), 0, use_pdl, s, a);
}

}  // namespace ckv
