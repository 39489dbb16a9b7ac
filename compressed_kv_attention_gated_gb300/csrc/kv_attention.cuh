// kv_attention.cuh -- what the two forms of ckv_kv_attention share: what a token sees, jobs
// (tiles of rows with the keys that their tokens see together), and the copying of queries,
// keys and values into shared memory.
#pragma once

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ckv_device.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"
#include "ckv_tcgen05.cuh"

namespace ckv {

// How a call is cut up (kv_attention.cu).
struct KvPlan {
  int R;       // rows of a tile: 16, 32 or 64 (keys on the M side), 128 or 256 (rows on the M side)
  int tiles;   // bound of the number of tiles
  int splits;  // ranges of keys
  int chunk;   // keys of a range (a multiple of kKvKeys); the last range takes all that are left: more, if a tile's contexts lie apart
  int heads;   // key heads whose jobs a CTA takes together
  bool sorted; // requests with the longest contexts first, by kv_order_kernel
};
// CTAs of the launch: a tile, a range of keys and p.heads key heads each.
inline int64_t kv_jobs(const KvPlan& p, int32_t KH) { return static_cast<int64_t>(p.tiles) * p.splits * ((KH + p.heads - 1) / p.heads); }
cudaError_t launch_kv_attention_few(const KvAttentionArgs& a, const KvPlan& p, bool use_pdl, cudaStream_t s);

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
// request: request b's first tile is (r_b + m (R - g)) / R with r_b the rows before it, g =
// gcd(G, R), which all r_b and R are multiples of, and m the lesser of b and the tokens before it, which
// grows by one at least with every request that has tokens.  That leaves it ceil(rows / R) tiles at
// least, and none over where tokens are whole tiles; and there are no more tiles than the tokens can
// fill, however many requests have none (a CTA that passes over an empty one takes 1.6 us for it, and
// its other warps wait for two seconds at most).
__host__ __device__ inline int kv_tile_pad(int G, int R) {
  const int g = G & -G;  // R is a power of two
  return g < R ? R - g : 0;
}

__device__ __forceinline__ int32_t kv_page_of(const KvAttentionArgs& a, int32_t key) {
  return a.page_shift >= 0 ? key >> a.page_shift : key / a.cache.page_size;
}
__device__ __forceinline__ bool kv_page_there(const KvAttentionArgs& a, int32_t page) { return page >= 0 && page < a.cache.num_pages; }

__device__ __forceinline__ int32_t kv_first_tile(const KvAttentionArgs& a, int32_t b, int32_t tok0, int64_t pad, int R) {
  return static_cast<int32_t>((tok0 * static_cast<int64_t>(a.G) + min(b, tok0) * pad) / R);
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
  const int32_t* first_tile = a.order + a.B;  // of request order[i], the i-th; where there is an order
  int lo = 0, n = a.B;  // the request is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && (a.order ? first_tile[i] : kv_first_tile(a, i, kv_start_of(a, i), pad, R)) <= tile;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  KvTile t;
  t.b = a.order ? a.order[lo] : lo;
  t.tok0 = kv_start_of(a, t.b);
  t.ntok = kv_start_of(a, t.b + 1) - t.tok0;
  // with an order, a request's last tile, which sees most, comes first
  const int64_t i = a.order ? first_tile[lo + 1] - 1 - tile : tile - kv_first_tile(a, lo, t.tok0, pad, R);
  const int64_t base = i * R, left = static_cast<int64_t>(t.ntok) * a.G - base;
  t.rows = base < 0 || left <= 0 ? 0 : static_cast<int32_t>(left < R ? left : R);  // base < 0: row_start does not begin with 0
  t.base = static_cast<int32_t>(base);
  return t;
}

constexpr int kKvKeys = 128, kKvUnit = 32768;  // keys of a tile; bytes of a unit
constexpr int kKvMaxRing = 6;                  // places of the ring
constexpr int kKvShort = 2;                    // tiles of keys of a job behind which the next one is taken at once
constexpr float kKvJump = 16.f;                // log2 of the largest weight over its reference

struct Job {
  KvTile tile;
  int32_t kh, split;
  int32_t first, low;  // the list of keys: rows 0 .. first - 1, then low, low + 1, ...
  int32_t v0, v1;      // of the list
  int32_t n;           // tiles of keys
  int32_t two;         // each softmax group has a tile of rows of its own
  int32_t missing;     // pages are not there: the softmax has to look (where L::kFindMissing; else it always does)
  int32_t live;        // 0: no more jobs
};

// Barriers of both forms.  Uses of a barrier are numbered from 0 over the whole kernel, so that everyone
// counts alike.
struct KvCommon {
  uint64_t full[kKvMaxRing], empty[kKvMaxRing];  // of a unit of the ring: 128 copying threads; the products that read it
  uint64_t q_full[2], q_empty[2];                // of a slot of queries, alike
  uint64_t s_full[2], p_full[2];                 // of a buffer of scores: the products; the softmax warps that made weights of it
  uint64_t o_full[2];                            // every product of a job: once per job with keys
  uint64_t pv_done[2];                           // second products of a tile of keys
  uint64_t job_full[2], job_empty[2];
  uint64_t wanted;                               // a job behind a long one, by the first copying warp
  uint64_t taken;                                // the answer to take_job()
  uint64_t drain;
  alignas(16) uint64_t answer[2];
  uint32_t tmem;
  Job job[2];
};

__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool b_mn_major) { return idesc_f16(n, false, b_mn_major) | (1u << 7) | (1u << 10); }

// Wait for use `n` of a barrier, by a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t n) { return __all_sync(0xFFFFFFFFu, mbar_wait_near(bar, n & 1u)); }

// ---------------------------------------------------------------------- jobs
// The first job of CTA `id` (of p.heads), by one converged warp; rows <= 0 when there is nothing to do in it.
template <typename L>
__device__ __forceinline__ Job make_job(const KvAttentionArgs& a, const KvPlan& p, int64_t id) {
  const int lane = threadIdx.x & 31;
  Job j;
  const int32_t groups = (a.KH + p.heads - 1) / p.heads;
  j.kh = static_cast<int32_t>(id % groups) * p.heads;
  id /= groups;
  j.split = static_cast<int32_t>(id % p.splits);
  j.tile = kv_find_tile(a, static_cast<int32_t>(id / p.splits), L::kRows);
  j.live = 1;
  j.two = L::kRows == 256 && j.tile.rows > 128;
  j.first = j.low = j.v0 = j.v1 = j.n = j.missing = 0;
  if (j.tile.rows <= 0) return j;
  // what its tokens see together
  const int32_t t0 = j.tile.tok0 + j.tile.base / a.G, t1 = j.tile.tok0 + (j.tile.base + j.tile.rows - 1) / a.G;
  int32_t low = INT32_MAX, end = -1;
  for (int32_t t = t0 + lane; t <= t1; t += 32) {
    const Seen s = seen_by(a, t);
    if (s.c < 0) continue;
    end = max(end, s.end);
    if (s.end > 0) low = min(low, s.low);  // a token that sees nothing does not widen the list
  }
  low = __reduce_min_sync(0xFFFFFFFFu, low);
  end = __reduce_max_sync(0xFFFFFFFFu, end);
  if (end < 0) j.tile.rows = 0;  // every token is left as it is
  end = max(end, 0);
  j.low = min(low, end);
  j.first = min(a.first, j.low);
  const int32_t count = end - j.low + j.first;
  j.v0 = static_cast<int32_t>(min(static_cast<int64_t>(j.split) * p.chunk, static_cast<int64_t>(count)));
  j.v1 = j.split == p.splits - 1 ? count : min(count, j.v0 + p.chunk);
  j.n = (j.v1 - j.v0 + kKvKeys - 1) / kKvKeys;
  if (j.n == 0 || !L::kFindMissing) return j;
  // the pages of its keys: rows v0 .. first - 1, then those from the list's second part
  const int32_t* table = a.table + static_cast<int64_t>(j.tile.b) * a.table_stride;
  bool lost = false;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int32_t k0 = part ? j.low + max(j.v0 - j.first, 0) : j.v0, k1 = part ? j.low + j.v1 - j.first : min(j.v1, j.first);
    if (k0 >= k1) continue;
    const int32_t p0 = kv_page_of(a, k0), p1 = kv_page_of(a, k1 - 1);
#pragma unroll 4
    for (int32_t p = p0 + lane; p <= p1; p += 32) lost |= !kv_page_there(a, table[p]);
  }
  j.missing = __any_sync(0xFFFFFFFFu, lost);
  return j;
}

// A job of a CTA that has not begun, which then never does: the launch has a CTA for each job, and CTAs that are
// there take what is left, so that none waits for another's long jobs.  -1: there is none (and none may be asked for
// again).  By one converged warp; false when the answer does not come.
__device__ __forceinline__ bool take_job(KvCommon& sm, uint32_t use, int64_t& id) {
  if ((threadIdx.x & 31) == 0) {
    fence_proxy_async_smem();  // the last answer has been read
    mbar_arrive_expect_tx(&sm.taken, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_u32(sm.answer)),
                 "r"(smem_u32(&sm.taken))
                 : "memory");
  }
  __syncwarp();
  if (!warp_wait(&sm.taken, use)) return false;
  const uint64_t lo = sm.answer[0], hi = sm.answer[1];
  uint32_t got, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n mov.b128 r, {%2, %3};\n clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
      : "=r"(got), "=r"(x)
      : "l"(lo), "l"(hi));
  __syncwarp();
  id = got ? static_cast<int64_t>(x) : -1;
  return true;
}

// The planning warp: jobs that have something to do, one after the other; more(job, i) adds what a form wants to
// know of the job in place i.
template <typename L, typename F>
__device__ __forceinline__ bool plan_jobs(const KvAttentionArgs& a, const KvPlan& p, KvCommon& sm, F&& more) {
  const int lane = threadIdx.x & 31;
  uint32_t use = 0, asked = 0, wanted = 0;
  for (int64_t id = blockIdx.x;;) {
    Job j;
    j.live = 0;
    if (id >= 0) j = make_job<L>(a, p, id);
    if (j.live && j.tile.rows <= 0) j.kh = a.KH;
    for (const int32_t last = j.live ? min(j.kh + p.heads, a.KH) : 1; j.live ? j.kh < last : true; ++j.kh) {
      if (use >= 2 && !warp_wait(&sm.job_empty[use & 1], (use >> 1) - 1)) return false;
      if (j.live) more(j, use & 1);
      if (lane == 0) sm.job[use & 1] = j;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.job_full[use & 1]);
      if (!j.live) return true;
      ++use;
      // the next one follows a long one when the copies of this one come to their end
      if (j.n > kKvShort && !warp_wait(&sm.wanted, wanted++)) return false;
    }
    if (!take_job(sm, asked++, id)) return false;
  }
}

// Four warps: queries, keys and values of the jobs, unit by unit, as many ahead as the ring has places.
// A unit is 128 rows x 256 bytes, 32 of the rows by each warp, 16 lanes to a row; every thread's copies
// arrive at the unit's barrier by themselves.  A lane holds the place of one row, from which the others
// get it by a shuffle; places are counted in KvSide::unit bytes, so that they have 32 bits.
template <typename L>
__device__ __forceinline__ bool copy_jobs(const KvAttentionArgs& a, KvCommon& sm, uint8_t* smem) {
  const int lane = threadIdx.x & 31, cw = (threadIdx.x >> 5) - L::kCopyWarp, x = lane & 15, upper = lane >> 4;
  constexpr bool kLate = L::kRows == 256;
  uint32_t unit = 0, q_use = 0;
  auto arrive = [](uint64_t* bar) { asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory"); };
  auto copy16 = [](uint32_t to, const uint8_t* from, uint32_t bytes) {  // zeros behind `bytes`
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
  };
  // where this lane's piece of row 2 i + upper of the warp goes, from the beginning of the unit
  uint32_t piece[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = cw * 32 + 2 * i + upper;
    piece[i] = (x >> 3) * 16384 + r * 128 + (((x & 7) ^ (r & 7)) * 16);
  }
  // the warp's rows of a unit, at `at` (one per lane; only those in `on` are there)
  auto copy_rows = [&](uint32_t to, const uint8_t* from, uint32_t at, uint32_t step, uint32_t on) {
#pragma unroll
    for (int i0 = 0; i0 < 16; i0 += 8) {
      // the shuffles first: the compiler keeps their order with the copies, each of which would wait for its own
      uint32_t r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = __shfl_sync(0xFFFFFFFFu, at, 2 * (i0 + i) + upper);
      if (on == 0xFFFFFFFFu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) copy16(to + piece[i % 4] + ((i0 + i) / 4) * 1024, from + static_cast<uint64_t>(r[i]) * step, 16);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          copy16(to + piece[i % 4] + ((i0 + i) / 4) * 1024, from + static_cast<uint64_t>(r[i]) * step, (on >> (2 * (i0 + i) + upper)) & 1 ? 16 : 0);
      }
    }
  };
  const uint32_t ring = smem_u32(smem) + L::kUnits;
  auto has_place = [&](uint32_t c) { return c < L::kRing || warp_wait(&sm.empty[c % L::kRing], c / L::kRing - 1); };
  auto copy_unit = [&](const uint16_t* from, uint32_t at, uint32_t step, uint32_t on) {
    if (!has_place(unit)) return false;
    copy_rows(ring + unit % L::kRing * kKvUnit, reinterpret_cast<const uint8_t*>(from + x * 8), at, step, on);
    arrive(&sm.full[unit % L::kRing]);
    ++unit;
    return true;
  };
  bool ok = true;
#pragma unroll 1
  for (uint32_t job_use = 0;; ++job_use) {
    ok = warp_wait(&sm.job_full[job_use & 1], job_use >> 1);
    if (!ok) break;
    const Job job = sm.job[job_use & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.job_empty[job_use & 1]);
    if (!job.live) break;
    if (job.n == 0) continue;
    const bool two = L::kRows == 256 && job.two;
    const int32_t* table = a.table + static_cast<int64_t>(job.tile.b) * a.table_stride;
    // the row of the cache in this lane's place of a tile, -1: none; and its page
    auto key_of = [&](int j) {
      const int32_t v = job.v0 + j * kKvKeys + cw * 32 + lane;
      return j >= job.n || v >= job.v1 ? -1 : v < job.first ? v : job.low + v - job.first;
    };
    int32_t key = key_of(0), page = key >= 0 ? table[kv_page_of(a, key)] : 0;
    auto queries = [&]() {
      for (int w = 0; w < (two ? 2 : 1); ++w, ++q_use) {
        const uint32_t slot = q_use % L::kQSlots;
        if (q_use >= L::kQSlots && !warp_wait(&sm.q_empty[slot], q_use / L::kQSlots - 1)) return false;
        constexpr int kMine = L::kQRows / 4;  // rows of this warp
        const int32_t i = w * 128 + cw * kMine + lane, r = job.tile.base + i;
        int64_t off = -1;
        if (lane < kMine && i < job.tile.rows) {
          const int32_t tok = r / a.G;
          off = (job.tile.tok0 + tok) * a.q_st + (job.kh * a.G + r - tok * a.G) * a.q_sh;
        }
        const uint32_t to = smem_u32(smem) + slot * L::kQSlot;
#pragma unroll 1
        for (int u = 0; u < L::kKU; ++u) {
#pragma unroll
          for (int k = 0; k < kMine / 2; ++k) {
            const int rr = cw * kMine + 2 * k + upper;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, 2 * k + upper);
            copy16(to + (u * 2 + (x >> 3)) * L::kQBlock + rr * 128 + (((x & 7) ^ (rr & 7)) * 16),
                   reinterpret_cast<const uint8_t*>(a.q + (o >= 0 ? o : 0) + u * 128 + x * 8), o >= 0 ? 16 : 0);
          }
        }
        arrive(&sm.q_full[slot]);
      }
      return true;
    };
    uint32_t v_at = 0, v_on = 0;
#pragma unroll 1
    for (int j = 0; j <= job.n && ok; ++j) {
      if (job.n > kKvShort && j == job.n - 2 && cw == 0 && lane == 0) mbar_arrive(&sm.wanted);
      uint32_t next_at = 0, on = 0;
      if (j < job.n) {
        uint32_t k_at = 0;
        const bool there = key >= 0 && kv_page_there(a, page);
        if (there) {
          const uint32_t row = key - kv_page_of(a, key) * a.cache.page_size;
          k_at = page * a.k_side.page + row * a.k_side.row + job.kh * a.k_side.head;
          next_at = page * a.v_side.page + row * a.v_side.row + job.kh * a.v_side.head;
        }
        on = __ballot_sync(0xFFFFFFFFu, there);
        key = key_of(j + 1);
        page = key >= 0 ? table[kv_page_of(a, key)] : 0;
        for (int u = 0; u < L::kKU && ok; ++u) {
          // Two tiles of queries come behind the first unit, whose place is free before theirs; otherwise their place is
          // free first, and a unit behind could have to wait for what is made of them.
          if (!kLate && j == 0 && u == 0) ok = queries();
          ok = ok && copy_unit(a.cache.k + u * 128, k_at, a.k_side.unit, on);
          if (kLate && j == 0 && u == 0) ok = ok && queries();
        }
      }
      if (a.same) continue;  // the keys' units are the values'
      if (two ? j < job.n : j > 0) {
        for (int u = 0; u < L::kKU && ok; ++u)
          ok = copy_unit(a.cache.v + u * 128, two ? next_at : v_at, a.v_side.unit, two ? on : v_on);
      }
      v_at = next_at;
      v_on = on;
    }
    if (!ok) break;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  return ok;
}

}  // namespace
}  // namespace ckv
