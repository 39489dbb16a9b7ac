// kv_attention.cuh -- what a token of ckv_kv_attention sees, and where its rows are.
#pragma once

#include <cmath>
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr float kKvLn2 = 0.69314718055994531f;

// The rows that a token sees: j < c and (j >= low or j < first), and of the drafts from row c on those
// whose bit is set.  c < 0: a token that is left as it is.
struct Seen {
  int32_t c, low, first;
  int32_t end;  // one past the last row seen
};

__device__ __forceinline__ Seen seen_by(const KvAttentionArgs& a, int32_t t) {
  Seen s;
  s.c = a.ctx_rows[t];
  s.end = s.c;
  if (s.c > a.max_rows) {
    flag_error(a.err, CKV_DEVERR_SEQ_LEN);
    s.c = s.end = a.max_rows;
  }
  int32_t n = 0;
  if (a.words > 0 && s.c >= 0) {
    for (int w = 0; w < a.words; ++w) {
      const uint64_t m = a.mask[static_cast<int64_t>(t) * a.words + w];
      n += __popcll(m);
      if (m) s.end = s.c + w * 64 + 64 - __clzll(static_cast<long long>(m));
    }
    if (s.end > a.max_rows) {
      flag_error(a.err, CKV_DEVERR_SEQ_LEN);
      s.end = a.max_rows;
    }
  }
  s.low = a.window > 0 ? min(max(s.c + n - a.window, 0), max(s.c, 0)) : 0;
  s.first = min(a.first, s.low);
  return s;
}

__device__ __forceinline__ int32_t kv_start_of(const KvAttentionArgs& a, int32_t b) {
  return min(max(a.row_start[b], 0), static_cast<int32_t>(a.T));
}

}  // namespace
}  // namespace ckv
