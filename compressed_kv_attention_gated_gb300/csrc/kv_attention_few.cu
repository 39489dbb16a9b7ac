// kv_attention_few.cu -- attention over the uncompressed paged cache with the keys on the M
// side of both products, for tiles of at most 64 (token, head) rows that share a key head
// (kv_attention.cu holds the other form and the formulas):
//   S^T [128 keys x R]     = K [128 x D] Q^T [D x R]
//   O^T [D channels x R]  += V^T [D x 128] P^T [128 x R]        R = 16, 32 or 64
// M is 128 whatever the number of rows, so that few rows cost few columns, and a thread of the softmax
// has one key of half of the rows: 8 to 32 exponentials per 128 keys.  A row's maximum is spread
// over 128 threads; weights are taken against a reference, the largest score of the tile that set it,
// and only when some weight exceeds 2^16 the true maxima are formed again and O and the sums
// rescaled.  The two groups of four softmax warps have half of the rows each and nothing to tell one
// another.  P goes through shared memory (rows of 128 bytes, 128-byte swizzle).
//
// Roles, jobs and the ring of units are those of the other form.  Where one row of the cache is key and
// value, its units stay for the second product.
//
// Bound by HBM with grouped heads (every row of the window is read once for its heads): 256 tokens x 64 heads over
// 1024 rows of 8 key heads, D = 128, 165 us, 98% of the copy rate.  At D = 512 with 64 rows queries (64 KB), P and one
// tile of keys fill shared memory, and the next tile's keys wait for the second product of this one: 1024 tokens x
// 64 heads over 128 rows 59 us (4.5 TB/s), 8000 over 128 rows 327 us.  With more keys the copies of a tile (256 KB, keys and
// values) and its products still take turns: 8000 tokens over 4096 rows 5175 us, 830 TFLOP/s, the tensor cores busy 34%
// of the time and 10 TB/s from L2, half of what the copies reach alone.
#include "kv_attention.cuh"

namespace ckv {
namespace {

// What a job's rows see, by the planning warp.
template <int R>
struct FewRows {
  alignas(16) int32_t c[R], low[R], first[R];
  int32_t end[R], flat[R], t[R];  // flat: (token, head) index, -1: none
  int32_t c_min, low_max;         // of rows that are there
};

template <int R>
struct FewSmall : KvCommon {
  FewRows<R> rows[2];
  alignas(16) float ref[R];    // references of the weights, log2 units
  alignas(16) float keep[R];   // what a move of the references leaves of sums and outputs
  alignas(16) float scale[R];  // of the output
  float part[4][R];
};

template <int D_, int R>
struct FewLayout {
  static constexpr int D = D_;
  static constexpr int kRows = R;
  static constexpr int kMmaWarp = 8, kPlanWarp = 9, kCopyWarp = 12, kThreads = 512;  // behind the softmax's eight
  static constexpr int kKU = D / 128;  // units of a tile's keys, and of its values
  static constexpr int kQRows = R;
  static constexpr bool kFindMissing = false;  // a softmax thread looks up the page of its key while it waits
  static constexpr int kQBlock = R * 128;
  static constexpr int kQSlot = kQBlock * (D / 64);
  static constexpr int kQSlots = kQSlot <= 16384 ? 2 : 1;
  static constexpr int kP = kQSlots * kQSlot;                // P: 128 keys x 128 bytes
  static constexpr int kPBufs = D == 512 && R == 64 ? 1 : 2;
  static constexpr int kUnits = kP + kPBufs * kKvKeys * 128;
  static constexpr int kMost = (227 * 1024 - static_cast<int>(sizeof(FewSmall<R>)) - kUnits) / kKvUnit;
  static constexpr int kRing = kMost < kKvMaxRing ? kMost : kKvMaxRing;
  static constexpr int kSmall = kUnits + kRing * kKvUnit;
  static constexpr int kCols = R / 2;                        // rows (columns of S^T) of a softmax thread
  static constexpr int kTmemO = 0, kTmemS = 256;             // O^T: R columns per 128 channels; S^T: two buffers of 64
  static_assert(kRing >= kKU, "a tile's units");
};

template <int D, int R>
constexpr int few_smem_bytes() {
  return FewLayout<D, R>::kSmall + static_cast<int>(sizeof(FewSmall<R>));
}

// The four softmax warps of group w meet; true when p holds for one of the 128 threads.
__device__ __forceinline__ void group_barrier(int w) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + w) : "memory"); }
__device__ __forceinline__ bool group_any(int w, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(1 + w)
      : "memory");
  return r != 0;
}

template <int n>
__device__ __forceinline__ void load_row(const float* p, float (&v)[n]) {
#pragma unroll
  for (int i = 0; i < n; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(p + i);
    v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
  }
}

template <int D, int R>
__device__ __forceinline__ bool few_soft(const KvAttentionArgs& a, const KvPlan& p, FewSmall<R>& sm, uint8_t* smem, uint32_t tmem) {
  using L = FewLayout<D, R>;
  constexpr int kCols = L::kCols;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, w = warp >> 2, place = threadIdx.x & 127;
  const int c0 = w * kCols;
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const float c = a.softmax_scale * kLog2e;
  uint32_t tile = 0, o_use = 0;  // tiles of keys and jobs with keys so far
  bool ok = true;                // exits are taken by the four warps of a group together
#pragma unroll 1
  for (uint32_t job_use = 0;; ++job_use) {
    ok = ok && mbar_wait_near(&sm.job_full[job_use & 1], (job_use >> 1) & 1);
    if (group_any(w, !ok)) return false;
    const Job& job = sm.job[job_use & 1];
    const FewRows<R>& rows = sm.rows[job_use & 1];
    if (!job.live) return true;
    const int32_t n = job.n, v0 = job.v0, v1 = job.v1, head0 = job.first, low0 = job.low;
    const int32_t* table = a.table + static_cast<int64_t>(job.tile.b) * a.table_stride;
    float l[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) l[i] = 0.f;
    if (n == 0 && place < kCols) sm.ref[c0 + place] = kNegBig;
#pragma unroll 1
    for (int j = 0; j < n; ++j, ++tile) {
      const int buf = tile & 1;
      // the key of the thread's place, which rows may see it
      const int32_t v = v0 + j * kKvKeys, k0 = low0 + v - head0;  // first place; its row, were it none of the first ones
      const int32_t key = v + place < head0 ? v + place : k0 + place;
      const bool gone = v + place < v1 && !kv_page_there(a, table[kv_page_of(a, key)]), there = v + place < v1 && !gone;
      ok = mbar_wait_near(&sm.s_full[buf], (tile >> 1) & 1) && ok;  // a wait that ran out before is not forgotten
      __syncwarp();
      tc_fence_after();
      const uint32_t at_s = tmem + lanes + L::kTmemS + buf * 64 + c0;
      const bool whole = v + kKvKeys <= v1 && k0 + kKvKeys <= rows.c_min && (v >= head0 ? k0 : low0) >= rows.low_max;
      const bool masks = __any_sync(0xFFFFFFFFu, gone) || !whole;
      // scores over the references in log2 units, -infinity for what a row does not see
      uint32_t seen = ~0u;
      if (masks) {
        seen = 0;
#pragma unroll
        for (int i = 0; i < kCols; i += 4) {
          const int4 cc = *reinterpret_cast<const int4*>(&rows.c[c0 + i]), lo = *reinterpret_cast<const int4*>(&rows.low[c0 + i]),
                     fi = *reinterpret_cast<const int4*>(&rows.first[c0 + i]);
          seen |= (key < cc.x && (key >= lo.x || key < fi.x) ? 1u : 0u) << i;
          seen |= (key < cc.y && (key >= lo.y || key < fi.y) ? 2u : 0u) << i;
          seen |= (key < cc.z && (key >= lo.z || key < fi.z) ? 4u : 0u) << i;
          seen |= (key < cc.w && (key >= lo.w || key < fi.w) ? 8u : 0u) << i;
        }
        if (a.words > 0) {
#pragma unroll 1
          for (int i = 0; i < kCols; ++i) {
            const int32_t d = key - rows.c[c0 + i];
            if (d >= 0 && key < rows.end[c0 + i])
              seen |= static_cast<uint32_t>((a.mask[static_cast<int64_t>(rows.t[c0 + i]) * a.words + (d >> 6)] >> (d & 63)) & 1) << i;
          }
        }
        if (v + place >= v1) seen = 0;
        if (gone && seen) flag_error(a.err, CKV_DEVERR_CACHE_LOC);
        if (!there) seen = 0;
      }
      auto read_scores = [&](float (&z)[kCols]) {
        tmem_ld<kCols>(at_s, z);
#pragma unroll
        for (int i = 0; i < kCols; ++i) z[i] *= c;
        if (masks) {
#pragma unroll
          for (int i = 0; i < kCols; ++i) z[i] = (seen >> i) & 1 ? z[i] : -INFINITY;
        }
      };
      auto over_refs = [&](float (&z)[kCols]) {
        float f[kCols], over = -INFINITY;
        load_row<kCols>(&sm.ref[c0], f);
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          z[i] -= f[i];
          over = fmaxf(over, z[i]);
        }
        return over;
      };
      float z[kCols];
      read_scores(z);
      // a job's first tile sets the references (nothing is lost where that was not to be known)
      if (j == 0 || group_any(w, !ok || over_refs(z) > kKvJump)) {
        // new references: the largest score so far of each row
        if (j > 0) read_scores(z);
        const float top = reduce_columns<kCols, true>(z, lane);
        constexpr int kShare = 32 / kCols;  // lanes that hold the same row's result
        if (lane % kShare == 0) sm.part[quad][c0 + lane / kShare] = top;
        if (group_any(w, !ok)) return false;
        if (place < kCols) {
          const int r = c0 + place;
          const float old = j == 0 ? kNegBig : sm.ref[r];
          const float now = fmaxf(fmaxf(fmaxf(sm.part[0][r], sm.part[1][r]), fmaxf(sm.part[2][r], sm.part[3][r])), old);
          sm.keep[r] = fast_exp2(old - now);
          sm.ref[r] = now;
        }
        group_barrier(w);
        if (j > 0) {
          load_row<kCols>(&sm.keep[c0], z);
#pragma unroll
          for (int i = 0; i < kCols; ++i) l[i] *= z[i];
          ok = mbar_wait_near(&sm.pv_done[0], (tile - 1) & 1) && ok;
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int u = 0; u < L::kKU; ++u) {
#pragma unroll
            for (int i = 0; i < kCols; i += 8) {
              float o[8];
              const uint32_t at = tmem + lanes + L::kTmemO + u * R + c0 + i;
              tmem_ld<8>(at, o);
#pragma unroll
              for (int x = 0; x < 8; ++x) o[x] *= z[i + x];
              tmem_st8(at, o);
            }
          }
          tc_wait_st();
        }
        read_scores(z);
        over_refs(z);
      }
      // weights, rounded to bf16, as row `place` of P
      if (L::kPBufs == 1 && tile > 0) ok = mbar_wait_near(&sm.pv_done[0], (tile - 1) & 1) && ok;  // its last use is over
      uint8_t* row = smem + L::kP + (L::kPBufs == 2 ? buf : 0) * (kKvKeys * 128) + place * 128;
#pragma unroll
      for (int i = 0; i < kCols; i += 8) {
        uint32_t x[4];
#pragma unroll
        for (int y = 0; y < 8; y += 2) {
          const float p0 = fast_exp2(z[i + y]), p1 = fast_exp2(z[i + y + 1]);
          l[i + y] += p0;
          l[i + y + 1] += p1;
          x[y / 2] = pack_bf16x2_rn(p0, p1);
        }
        *reinterpret_cast<uint4*>(row + ((((c0 + i) / 8) ^ (place & 7)) * 16)) = make_uint4(x[0], x[1], x[2], x[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[buf]);
    }
    // ------------------------------------------------------------------ output
    const float sum = reduce_columns<kCols, false>(l, lane);
    constexpr int kShare = 32 / kCols;
    if (lane % kShare == 0) sm.part[quad][c0 + lane / kShare] = sum;
    group_barrier(w);
    const bool split = p.splits > 1;
    const int64_t all_rows = a.T * a.H, range = split ? job.split * all_rows : 0;
    float* part_out = static_cast<float*>(a.workspace);
    if (place < kCols) {
      const int r = c0 + place;
      const int32_t flat = rows.flat[r];
      float all = (sm.part[0][r] + sm.part[1][r]) + (sm.part[2][r] + sm.part[3][r]), m = sm.ref[r], keep = 1.f, sink = -INFINITY;
      const bool none = all == 0.f;
      if (a.sink && !split && flat >= 0) {
        sink = a.sink[flat % a.H];
        const float s = sink * kLog2e, high = fmaxf(none ? kNegBig : m, s);
        keep = none ? 0.f : fast_exp2(m - high);
        all = (none ? 0.f : all * keep) + (s == high ? 1.f : fast_exp2(s - high));
        m = high;
      }
      sm.scale[r] = none ? 0.f : keep / all;
      if (flat >= 0) {
        // nothing at all: no sink, or one that is -infinity in log2 units
        const float lse = all == 0.f ? sink : (m + log2f(all)) * kKvLn2;
        if (split) part_out[p.splits * all_rows * D + range + flat] = lse;
        else if (a.lse) a.lse[flat] = lse;
      }
    }
    group_barrier(w);
    load_row<kCols>(&sm.scale[c0], l);
    if (n > 0) {
      ok = mbar_wait_near(&sm.o_full[0], o_use & 1) && ok;
      ++o_use;
      __syncwarp();
      tc_fence_after();
    }
#pragma unroll 1
    for (int u = 0; u < L::kKU; ++u) {
      float o[kCols];
      if (n > 0) {
        tmem_ld<kCols>(tmem + lanes + L::kTmemO + u * R + c0, o);
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) o[i] = 0.f;
      }
      const int ch = u * 128 + quad * 32 + lane;
      if (split) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const int32_t flat = rows.flat[c0 + i];
          if (flat >= 0) part_out[(range + flat) * D + ch] = o[i] * l[i];
        }
      } else {
        // Through the group's own pieces of P, whose last product is done (the other group may be a job ahead and writing
        // its own), so that rows leave in 16-byte pieces.  Neighbouring lanes (channels) trade halves: the even one has
        // both channels of row i, the odd one of row i + 1.
        // Piece y of the group's row r is piece r / 8 of its own in row at = r % 8 * 16 + (y, by 4 further on in odd rows) of P.
        const int odd = lane & 1, to = odd * 16 + ((quad * 4 + lane / 8) ^ (odd * 4));
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
          const float o0 = o[i] * l[i], o1 = o[i + 1] * l[i + 1];
          const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? o0 : o1, 1);
          *reinterpret_cast<uint32_t*>(smem + L::kP + (i % 8 * 16 + to) * 128 + ((c0 / 8 + i / 8) ^ (to & 7)) * 16 + lane % 8 / 2 * 4) =
              odd ? pack_bf16x2_rn(got, o1) : pack_bf16x2_rn(o0, got);
        }
        group_barrier(w);
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          const int at = place ^ (place / 16 % 2 * 4);
          const int32_t flat = rows.flat[c0 + i * 8 + place / 16];
          if (flat >= 0)
            *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(flat) * D + u * 128 + place % 16 * 8) =
                *reinterpret_cast<const uint4*>(smem + L::kP + at * 128 + ((c0 / 8 + i) ^ (at & 7)) * 16);
        }
        group_barrier(w);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.job_empty[job_use & 1]);
  }
}

// One thread: the products, in the order of their units.
template <int D, int R>
__device__ __forceinline__ bool few_mma(const KvAttentionArgs& a, FewSmall<R>& sm, uint32_t base, uint32_t tmem) {
  using L = FewLayout<D, R>;
  constexpr uint32_t kIdescS = idesc_bf16(R, false), kIdescO = idesc_bf16(R, true) | (1u << 15);
  uint32_t unit = 0, q_use = 0, tile = 0;
  auto wait = [](uint64_t* bar, uint32_t n) { return mbar_wait_near(bar, n & 1u); };
  auto unit_there = [&](uint32_t c) {
    const bool ok = wait(&sm.full[c % L::kRing], c / L::kRing);
    fence_proxy_async_smem();  // the copies are ordinary writes of other threads, done when the barrier says so
    tc_fence_after();
    return ok;
  };
#pragma unroll 1
  for (uint32_t job_use = 0;; ++job_use) {
    if (!wait(&sm.job_full[job_use & 1], job_use >> 1)) return false;
    const Job& job = sm.job[job_use & 1];
    if (!job.live) return true;
    const int n = job.n;
    mbar_arrive(&sm.job_empty[job_use & 1]);
    if (n == 0) continue;
    const uint32_t slot = q_use % L::kQSlots, unit0 = unit;
    if (!wait(&sm.q_full[slot], q_use / L::kQSlots)) return false;
    auto tile_scores = [&](int j) {
      const uint32_t buf = (tile + j) & 1;
      uint32_t c = a.same ? unit0 + j * L::kKU : unit;
      for (int u = 0; u < L::kKU; ++u, ++c) {
        if (!unit_there(c)) return false;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const uint64_t da = smem_desc_sw128(base + L::kUnits + (c % L::kRing) * kKvUnit + (s / 4) * 16384 + (s % 4) * 32, 16, 1024);
          const uint64_t db = smem_desc_sw128(base + slot * L::kQSlot + (u * 2 + s / 4) * L::kQBlock + (s % 4) * 32, 16, 1024);
          mma_f16_ss(tmem + L::kTmemS + buf * 64, da, db, kIdescS, u > 0 || s > 0);
        }
        if (!a.same) tc_commit(&sm.empty[c % L::kRing]);
      }
      if (!a.same) unit = c;
      tc_commit(&sm.s_full[buf]);
      if (j == n - 1) tc_commit(&sm.q_empty[slot]);
      return true;
    };
    // where a row is key and value, the next tile's units have a place beside this one's only in part of the rings
    const bool ahead = !a.same || L::kRing >= 2 * L::kKU;
    if (!tile_scores(0) || (ahead && n > 1 && !tile_scores(1))) return false;
    for (int j = 0; j < n; ++j) {
      const uint32_t buf = (tile + j) & 1;
      if (!wait(&sm.p_full[buf], (tile + j) >> 1)) return false;
      tc_fence_after();
      uint32_t c = a.same ? unit0 + j * L::kKU : unit;
      for (int u = 0; u < L::kKU; ++u, ++c) {
        if (!a.same && !unit_there(c)) return false;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const uint64_t da = smem_desc_sw128(base + L::kUnits + (c % L::kRing) * kKvUnit + s * 2048, 16384, 1024);
          const uint64_t db = smem_desc_sw128(base + L::kP + (L::kPBufs == 2 ? buf : 0) * (kKvKeys * 128) + s * 2048, 16384, 1024);
          mma_f16_ss(tmem + L::kTmemO + u * R, da, db, kIdescO, j > 0 || s > 0);
        }
        tc_commit(&sm.empty[c % L::kRing]);
      }
      if (!a.same) unit = c;
      tc_commit(&sm.pv_done[0]);
      const int next = j + (ahead ? 2 : 1);
      if (next < n && !tile_scores(next)) return false;
    }
    if (a.same) unit = unit0 + n * L::kKU;
    tc_commit(&sm.o_full[0]);
    tile += n;
    ++q_use;
  }
}

template <int D, int R>
__global__ void __launch_bounds__((FewLayout<D, R>::kThreads), 1)
    kv_attention_few_kernel(const __grid_constant__ KvAttentionArgs a, const __grid_constant__ KvPlan p) {
  using L = FewLayout<D, R>;
  // no static shared memory: the dynamic one begins on the swizzle's 1024 bytes (checked below)
  extern __shared__ __align__(1024) uint8_t smem[];
  FewSmall<R>& sm = *reinterpret_cast<FewSmall<R>*>(smem + L::kSmall);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023u) {
    pdl_wait();  // whoever follows in the stream counts on what came before having ended
    if (threadIdx.x == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
    return;
  }
  if (warp == L::kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < L::kRing; ++i) {
        mbar_init(&sm.full[i], 128);
        mbar_init(&sm.empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.q_full[i], 128);
        mbar_init(&sm.q_empty[i], 1);
        mbar_init(&sm.s_full[i], 1);
        mbar_init(&sm.p_full[i], 8);
        mbar_init(&sm.o_full[i], 1);
        mbar_init(&sm.pv_done[i], 1);
        mbar_init(&sm.job_full[i], 1);
        mbar_init(&sm.job_empty[i], 13);
      }
      mbar_init(&sm.wanted, 1);
      mbar_init(&sm.taken, 1);
      mbar_init(&sm.drain, 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc<512>(&sm.tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  pdl_wait();

  bool ok = true;
  if (warp < L::kMmaWarp) {
    ok = few_soft<D, R>(a, p, sm, smem, tmem);
    tc_fence_before();
  } else if (warp == L::kMmaWarp) {
    if (elect_one()) {
      ok = few_mma<D, R>(a, sm, smem_u32(smem), tmem);
      // the end of every product: tensor memory may be given back
      tc_commit(&sm.drain);
      ok = mbar_wait_near(&sm.drain, 0) && ok;
      if (!ok) flag_error(a.err, CKV_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == L::kPlanWarp) {
    ok = plan_jobs<L>(a, p, sm, [&](const Job& j, uint32_t i) {
      FewRows<R>& rows = sm.rows[i];
      int32_t c_min = INT32_MAX, low_max = 0;
      for (int r = lane; r < R; r += 32) {
        Seen s{0, 0, 0, 0};
        int32_t flat = -1, t = 0;
        if (r < j.tile.rows) {
          const int32_t row = j.tile.base + r, tok = row / a.G;
          t = j.tile.tok0 + tok;
          const Seen x = seen_by(a, t);
          if (x.c >= 0) {
            s = x;
            flat = t * a.H + j.kh * a.G + row - tok * a.G;
            c_min = min(c_min, s.c);
            low_max = max(low_max, s.low);
          }
        }
        rows.c[r] = s.c;
        rows.low[r] = s.low;
        rows.first[r] = s.first;
        rows.end[r] = s.end;
        rows.flat[r] = flat;
        rows.t[r] = t;
      }
      c_min = __reduce_min_sync(0xFFFFFFFFu, c_min);
      low_max = __reduce_max_sync(0xFFFFFFFFu, low_max);
      if (lane == 0) {
        rows.c_min = c_min;
        rows.low_max = low_max;
      }
    });
  } else if (warp >= L::kCopyWarp) {
    ok = copy_jobs<L>(a, sm, smem);
  }
  if (!ok && lane == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
  pdl_trigger();
  __syncthreads();
  if (warp == L::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

template <int D, int R>
cudaError_t launch(const KvAttentionArgs& a, const KvPlan& p, bool use_pdl, cudaStream_t s) {
  static_assert(few_smem_bytes<D, R>() <= 227 * 1024, "shared memory");
  cudaError_t e;
  if ((e = set_max_smem_once<kv_attention_few_kernel<D, R>>(few_smem_bytes<D, R>())) != cudaSuccess) return e;
  KvAttentionArgs b = a;
  const ckv_kv_cache& c = a.cache;
  // Units that stay keep the next tile's out of a ring that has no more places than one tile has units (D = 512, 64 rows):
  // there only jobs of one tile keep them (1024 tokens x 64 heads: 128 keys 65 us against 72, 1024 keys 256 against 242).
  b.same = c.k == c.v && c.k_stride_page == c.v_stride_page && c.k_stride_row == c.v_stride_row && c.k_stride_head == c.v_stride_head &&
           (FewLayout<D, R>::kRing > FewLayout<D, R>::kKU || p.chunk <= kKvKeys);
  return launch_ex(kv_attention_few_kernel<D, R>, dim3(static_cast<unsigned>(kv_jobs(p, a.KH))), dim3(FewLayout<D, R>::kThreads), few_smem_bytes<D, R>(),
                   use_pdl, s, b, p);
}

template <int D>
cudaError_t launch_d(const KvAttentionArgs& a, const KvPlan& p, bool use_pdl, cudaStream_t s) {
  return p.R == 16 ? launch<D, 16>(a, p, use_pdl, s) : p.R == 32 ? launch<D, 32>(a, p, use_pdl, s) : launch<D, 64>(a, p, use_pdl, s);
}

}  // namespace

cudaError_t launch_kv_attention_few(const KvAttentionArgs& a, const KvPlan& p, bool use_pdl, cudaStream_t s) {
  return a.cache.D == 128 ? launch_d<128>(a, p, use_pdl, s) : a.cache.D == 256 ? launch_d<256>(a, p, use_pdl, s) : launch_d<512>(a, p, use_pdl, s);
}

}  // namespace ckv
