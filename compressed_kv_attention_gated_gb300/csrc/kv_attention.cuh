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

// The (token, head of a group) rows of a request are cut into tiles of R.  Tiles begin anew with every
// request: request b's first tile is (r_b + b (R - g)) / R with r_b the rows before it and g =
// gcd(G, R), which all r_b and R are multiples of.  That leaves it ceil(rows / R) tiles at least,
// and none over where tokens are whole tiles.
__host__ __device__ inline int kv_tile_pad(int G, int R) {
  const int g = G & -G;  // R is a power of two
  return g < R ? R - g : 0;
}

// Which request and rows a tile has.
struct KvTile {
  int32_t b, tok0, ntok;  // the request, and its ragged rows
  int32_t base, rows;     // first row of the tile in the request, and how many (<= 0: none)
};

// By one converged warp.
__device__ __forceinline__ KvTile kv_find_tile(const KvAttentionArgs& a, int32_t tile, int R) {
  const int lane = threadIdx.x & 31;
  const int64_t pad = kv_tile_pad(a.G, R);
  int lo = 0, n = a.B;  // the request is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && (kv_start_of(a, i) * static_cast<int64_t>(a.G) + i * pad) / R <= tile;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  KvTile t;
  t.b = lo;
  t.tok0 = kv_start_of(a, lo);
  t.ntok = kv_start_of(a, lo + 1) - t.tok0;
  const int64_t base = (tile - (t.tok0 * static_cast<int64_t>(a.G) + lo * pad) / R) * R, left = static_cast<int64_t>(t.ntok) * a.G - base;
  t.rows = base < 0 || left <= 0 ? 0 : static_cast<int32_t>(left < R ? left : R);  // base < 0: row_start does not begin with 0
  t.base = static_cast<int32_t>(base);
  return t;
}

}  // namespace
}  // namespace ckv
