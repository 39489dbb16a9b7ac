// step_maps.cu -- block tables and slot maps of one serving step, from request
// lengths on the device (no counterpart in the sources; the arrays are those
// that the pooled, c128 and 4-bit calls take).
//
// Request b with s_b positions after the step and n_b new ones:
//   first ragged row      start_b = sum_{i<b} n_i
//   pages held before     f_b = ceil(floor((s_b - n_b) / P) / ps)
//   pages taken           t_b = ceil(floor(s_b / P) / ps) - f_b
//   index in the free list c + sum_{i<b} t_i
// Token i of request b has position s_b - n_b + i; it closes chunk row r =
// pos / P when (pos + 1) % P == 0, which lies in page r / ps of the request.
// The token that closes the first row of a taken page writes the page's table
// entry (pages are taken for rows that close in this step, so every taken page
// has such a token; for tokens past num_tokens the scan does it), and every
// token of a taken page derives the page id from the free list itself: no CTA
// waits for another's table entries.
//
// Every CTA scans the lengths of all requests into shared memory (12 bytes per
// request), so one launch does it all; then the tokens are spread over the
// grid.  Bound: launch and two dependent round trips for a decode step, the
// 28-32 bytes written per token for a long prompt.  Measured (GB300): 512 requests
// x 4 tokens 3.9 us, 64 requests of 1 to 8192 tokens 5.1 us (7.3 MB).
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kMapThreads = 1024;

// Block-wide exclusive scan of two values per thread.
struct Pair {
  uint32_t a, b;
};
__device__ __forceinline__ Pair block_exclusive_scan(Pair v, Pair* s_warp, Pair& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pair x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t ya = __shfl_up_sync(0xFFFFFFFFu, x.a, o), yb = __shfl_up_sync(0xFFFFFFFFu, x.b, o);
    if (lane >= o) {
      x.a += ya;
      x.b += yb;
    }
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  // every warp scans the 32 warps' totals (kMapThreads / 32 == 32) for itself
  Pair w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t ya = __shfl_up_sync(0xFFFFFFFFu, w.a, o), yb = __shfl_up_sync(0xFFFFFFFFu, w.b, o);
    if (lane >= o) {
      w.a += ya;
      w.b += yb;
    }
  }
  total.a = __shfl_sync(0xFFFFFFFFu, w.a, 31);
  total.b = __shfl_sync(0xFFFFFFFFu, w.b, 31);
  const uint32_t pa = __shfl_sync(0xFFFFFFFFu, w.a, max(warp - 1, 0)), pb = __shfl_sync(0xFFFFFFFFu, w.b, max(warp - 1, 0));
  return Pair{(warp > 0 ? pa : 0u) + x.a - v.a, (warp > 0 ? pb : 0u) + x.b - v.b};
}

// Largest b in [0, B) with pre[b] <= e (pre is non-decreasing, pre[0] = 0).
__device__ __forceinline__ int find_request(const int32_t* pre, int B, int32_t e) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= e) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The cursor after `taken` pages: never past the list, and a bad one stays put.
__device__ __forceinline__ int32_t next_cursor(int32_t c, int64_t taken, int64_t num_free) {
  if (c < 0 || c >= num_free) return c;
  return static_cast<int32_t>(min(c + taken, num_free));
}

constexpr uint32_t kNarrow = 1u << 21;

template <bool kWide>
__global__ void __launch_bounds__(kMapThreads) step_maps_kernel(const __grid_constant__ StepMapsArgs a) {
  extern __shared__ __align__(16) int32_t s_maps[];
  int32_t* s_start = s_maps;         // first ragged row [B], clamped to num_tokens
  int32_t* s_first = s_start + a.B;  // position of ragged row 0 if it were the request's: (s - n) - start
  int32_t* s_free = s_first + a.B;   // free-list index of the request's page number 0: c + taken before - pages held
  __shared__ Pair s_warp[2][32];  // by turns: a scan's totals may still be read when the next one begins

  pdl_wait();
  const uint32_t P = a.P, ps = a.page_size;
  const int32_t c0 = a.cursor[0];
  const bool lead = blockIdx.x == 0;
  uint32_t flags = 0;
  // tokens and pages of the requests so far; 1024 requests are summed in 32 bits at a time
  int64_t tokens = 0, pages = 0;
  int turn = 0;
  for (int base = 0; base < a.B; base += kMapThreads) {
    const int b = base + threadIdx.x;
    int32_t n = 0, s = 0, held = 0, need = 0;
    if (b < a.B) {
      s = a.seq_lens[b];
      n = a.query_lens[b];
      if (n < 0 || s < n) {
        flags |= CKV_DEVERR_SEQ_LEN;
        n = s = 0;
      }
      held = ((static_cast<uint32_t>(s - n) / P) + ps - 1u) / ps;
      need = ((static_cast<uint32_t>(s) / P) + ps - 1u) / ps;
      if (need > a.max_pages) {
        flags |= n > 0 ? CKV_DEVERR_PAGES : 0u;
        need = a.max_pages;
        held = min(held, need);
      }
    }
    // Counts below 2^21 are summed as they are.  When the call's limits are below that, larger
    // counts mean "past the limit" wherever they end; else the upper 16 bits go in a scan of their own.
    const uint32_t take = static_cast<uint32_t>(need - held);
    Pair total;
    int64_t before_tokens, before_pages, add_tokens, add_pages;
    if constexpr (!kWide) {
      const Pair at = block_exclusive_scan(Pair{min(static_cast<uint32_t>(n), kNarrow), min(take, kNarrow)}, s_warp[turn], total);
      turn ^= 1;
      before_tokens = at.a, before_pages = at.b, add_tokens = total.a, add_pages = total.b;
    } else {
      const Pair lo = block_exclusive_scan(Pair{n & 0xFFFFu, take & 0xFFFFu}, s_warp[turn], total);
      turn ^= 1;
      Pair total_hi;
      const Pair hi = block_exclusive_scan(Pair{static_cast<uint32_t>(n) >> 16, take >> 16}, s_warp[turn], total_hi);
      turn ^= 1;
      before_tokens = lo.a + (static_cast<int64_t>(hi.a) << 16), before_pages = lo.b + (static_cast<int64_t>(hi.b) << 16);
      add_tokens = total.a + (static_cast<int64_t>(total_hi.a) << 16), add_pages = total.b + (static_cast<int64_t>(total_hi.b) << 16);
    }
    if (b < a.B) {
      const int64_t start = min(tokens + before_tokens, static_cast<int64_t>(a.num_tokens));
      s_start[b] = static_cast<int32_t>(start);
      s_first[b] = static_cast<int32_t>((s - n) - start);
      // clamped: any index at or past num_free is past the list
      const int64_t f = min(c0 + pages + before_pages, a.num_free);
      s_free[b] = static_cast<int32_t>(f - held);
      // Tokens past num_tokens are dropped, their pages are taken all the same (a call with more
      // room takes the same ones): entered here, as no token does it.
      if (lead && c0 >= 0 && tokens + before_tokens + n > a.num_tokens) {
        for (int32_t pg = held; pg < need && f + (pg - held) < a.num_free; ++pg) {
          const int64_t closes = (static_cast<int64_t>(pg) * ps + 1) * P - 1;  // position that closes the page's first row
          if (tokens + before_tokens + closes - (s - n) >= a.num_tokens)
            a.block_table[b * a.table_stride + pg] = a.free_pages[f + (pg - held)];
        }
      }
      if (lead && a.row_start) a.row_start[b] = static_cast<int32_t>(start);
    }
    tokens += add_tokens;
    pages += add_pages;
  }
  __syncthreads();
  const int32_t live = static_cast<int32_t>(min(tokens, static_cast<int64_t>(a.num_tokens)));
  if (lead && threadIdx.x == 0) {
    if (a.row_start) a.row_start[a.B] = live;
    if (tokens > a.num_tokens) flags |= CKV_DEVERR_PLAN;
    if (pages > 0 && (c0 < 0 || c0 + pages > a.num_free)) flags |= CKV_DEVERR_PAGES;
    if (a.cursor_out != a.cursor) a.cursor_out[0] = next_cursor(c0, pages, a.num_free);
  }
  if (lead && flags) flag_error(a.err, flags);
  flags = 0;

  // unsigned: num_tokens goes to 2^31 - 1, and the step past the last token would leave 32 signed bits
  const uint32_t stride = gridDim.x * kMapThreads, places = a.num_tokens;
  for (uint32_t i = blockIdx.x * kMapThreads + threadIdx.x; i < places; i += stride) {
    int32_t pos = -1, req = -1, ctx = -1, rpos = -1, tail = -1, loc32 = -1;
    int64_t loc = -1;
    if (i < static_cast<uint32_t>(live)) {
      req = find_request(s_start, a.B, static_cast<int32_t>(i));
      pos = s_first[req] + static_cast<int32_t>(i);
      const uint32_t row = static_cast<uint32_t>(pos) / P;
      const uint32_t slot = static_cast<uint32_t>(pos) - row * P;
      ctx = static_cast<int32_t>(row);
      if (slot == P - 1u) {
        ctx += 1;
        rpos = pos - static_cast<int32_t>(P - 1u);
        const uint32_t pg = row / ps, r = row - pg * ps;
        // pages held before the step: those of the rows closed before its first token
        const uint32_t first = static_cast<uint32_t>(s_first[req] + s_start[req]);
        const uint32_t held = (first / P + ps - 1u) / ps;
        int32_t id = -1;
        if (pg < static_cast<uint32_t>(a.max_pages)) {
          int32_t* entry = a.block_table + req * a.table_stride + pg;
          if (pg >= held) {
            const int64_t f = static_cast<int64_t>(s_free[req]) + pg;
            if (f >= 0 && f < a.num_free && c0 >= 0) id = a.free_pages[f];
            if (r == 0) *entry = id;
          } else {
            id = *entry;
          }
          if (id < 0) flags |= CKV_DEVERR_PAGES;
        }
        if (id >= 0) {
          loc = static_cast<int64_t>(id) * ps + r;
          if (loc <= INT32_MAX) loc32 = static_cast<int32_t>(loc);
          else if (a.slot_mapping) flags |= CKV_DEVERR_CACHE_LOC;
        }
      }
      if (a.tail_slots) {
        const int32_t blk = a.tail_blocks[req];
        if (blk >= 0) {
          const int64_t t = static_cast<int64_t>(blk) * P + slot;
          if (t <= INT32_MAX) tail = static_cast<int32_t>(t);
          else flags |= CKV_DEVERR_TAIL_BLOCK;
        }
      }
    }
    if (a.positions) a.positions[i] = pos;
    if (a.batch_ids) a.batch_ids[i] = req;
    if (a.slot_mapping) a.slot_mapping[i] = loc32;
    if (a.cache_loc) a.cache_loc[i] = loc;
    if (a.tail_slots) a.tail_slots[i] = tail;
    if (a.row_positions) a.row_positions[i] = rpos;
    if (a.ctx_rows) a.ctx_rows[i] = ctx;
  }
  if (flags) flag_error(a.err, flags);

  if (a.cursor_out == a.cursor) {
    // in place: the CTA that arrives last (every CTA has read the cursor by
    // then) moves it and leaves the arrival count at 0 again
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      const int32_t arrived = atomicAdd(a.cursor + 1, 1);
      if (arrived == static_cast<int32_t>(gridDim.x) - 1) {
        a.cursor[0] = next_cursor(c0, pages, a.num_free);
        a.cursor[1] = 0;
      }
    }
  }
}

template <bool kWide>
cudaError_t launch(const StepMapsArgs& a, bool use_pdl, cudaStream_t s) {
  // sized for the largest B the entry point accepts (8192 requests, 96 KB)
  cudaError_t e = set_max_smem_once<step_maps_kernel<kWide>>(8192 * 3 * sizeof(int32_t));
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int64_t want = (static_cast<int64_t>(a.num_tokens) + kMapThreads - 1) / kMapThreads;
  const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : (want > sms ? sms : want));
  return launch_ex(step_maps_kernel<kWide>, dim3(grid), dim3(kMapThreads), static_cast<size_t>(a.B) * 3 * sizeof(int32_t), use_pdl, s,
                   a);
}

}  // namespace

cudaError_t launch_step_maps(const StepMapsArgs& a, bool use_pdl, cudaStream_t s) {
  const bool narrow = static_cast<uint32_t>(a.num_tokens) < kNarrow && a.num_free < kNarrow;
  return narrow ? launch<false>(a, use_pdl, s) : launch<true>(a, use_pdl, s);
}

}  // namespace ckv
