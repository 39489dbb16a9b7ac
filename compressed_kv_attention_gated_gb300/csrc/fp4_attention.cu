// fp4_attention.cu -- attention over the 4-bit paged cache (no counterpart in
// the sources; the format is in ckv_fp4.cuh).  Every cache row is key and
// value of all heads:
//   z_j = scale <q, k_j>,  lse = log(sum_j e^z_j [+ e^sink]),  out = sum_j e^(z_j - lse) k_j.
//
// The (token, head) rows of a request are cut into tiles of R rows (16, 32 or
// 64); a CTA takes one tile and a range of cache rows, 128 at a time, and runs
// both products on the tensor cores with the cache rows as the M side:
//   S^T [128 keys x R]     = K [128 x D] Q^T [D x R]
//   O^T [D channels x R]  += K^T [D x 128] P^T [128 x R]
// so one decoded tile of K in shared memory (fp16, 128-byte swizzle) serves as
// A of both, K-major for the first and MN-major for the second, M is always 128
// whatever the number of heads, and O (D x R) fits tensor memory.
//
// Exactness: a decoded value is code * scale (2 + 4 significant bits, 2^-10 ..
// 2688), exact in fp16; cache_scale goes into the factor of the scores and of
// the output.  A query row is scaled by a power of two to fp16's top, which
// keeps its 8 bits for every channel above 2^-28 of its largest.  Scores, sums
// and outputs are fp32.  Only the weights are rounded, to fp16 (2^-11).
//
// Softmax: in S^T a thread holds one key for R/2 rows, so a row's maximum is
// spread over 128 threads.  It is not formed per tile: weights are taken
// against a reference that is the maximum of the tile that set it, and only
// when some score exceeds its reference by more than 2^8 (weights up to 256 are
// harmless in fp16 and fp32) the CTA forms the true maxima and rescales O and
// the sums.  Sums stay per thread until the end.
//
// Roles: 8 softmax warps (also query load and output), 1 warp that issues the
// MMAs, 8 warps that load and decode cache rows into a ring of four units of
// 128 keys x 128 channels.  With D < 512 the ring holds more than a tile, and
// the scores of the next tile are computed under the softmax of this one.
//
// Long rows of few tiles are split over CTAs (blockIdx.y), whose partial
// outputs (fp32) and references a second kernel joins in a fixed order.
#include <cmath>
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_fp4.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"
#include "ckv_tcgen05.cuh"

namespace ckv {
namespace {

constexpr int kKeys = 128;       // cache rows per tile
constexpr int kRing = 4;         // units of 128 keys x 128 channels
constexpr int kUnitBytes = 32768;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarps = 8;
constexpr int kThreads = (kSoftWarps + 1 + kLoadWarps) * 32;
constexpr float kJump = 8.f;     // log2 of the largest weight before the reference moves
constexpr float kLn2 = 0.69314718055994531f;

struct SplitPlan {
  int R;        // rows per tile
  int tiles;    // bound of the number of tiles
  int splits;   // ranges of cache rows per tile
  int chunk;    // cache rows per range (multiple of kKeys)
};

SplitPlan plan_splits(int64_t T, int32_t B, int32_t H, int64_t max_rows) {
  SplitPlan p;
  const int64_t rows = (T + B - 1) / B * H;  // of an average request
  p.R = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  p.tiles = static_cast<int>(T * H / p.R + B);
  const int64_t busy = (T * H + p.R - 1) / p.R;
  const int64_t most = (max_rows + kKeys - 1) / kKeys;
  int64_t s = 152 / (busy < 1 ? 1 : busy);
  s = s < 1 ? 1 : s > most ? most : s;
  p.chunk = static_cast<int>(((max_rows + s - 1) / s + kKeys - 1) / kKeys * kKeys);
  p.splits = static_cast<int>((max_rows + p.chunk - 1) / p.chunk);
  return p;
}

// Which request and rows a tile has.  Request b's tiles start at
// floor(row_start[b] * H / R) + b: increasing, and never fewer than it needs.
struct Tile {
  int32_t tok0, ntok;  // the request's ragged rows
  int32_t b;
  int32_t base, rows;  // first (token, head) row of the tile in the request, and how many (<= 0: none)
};

__device__ __forceinline__ int32_t start_of(const Fp4AttentionArgs& a, int32_t b) {
  return min(max(a.row_start[b], 0), static_cast<int32_t>(a.T));
}

// By one converged warp.
__device__ __forceinline__ Tile find_tile(const Fp4AttentionArgs& a, int32_t tile, int R) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.B;  // the request is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && start_of(a, i) * static_cast<int64_t>(a.H) / R + i <= tile;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  Tile t;
  t.b = lo;
  t.tok0 = start_of(a, lo);
  t.ntok = start_of(a, lo + 1) - t.tok0;
  t.base = (tile - static_cast<int32_t>(t.tok0 * static_cast<int64_t>(a.H) / R + lo)) * R;
  t.rows = t.base < 0 ? 0 : min(R, t.ntok * a.H - t.base);  // base < 0: row_start does not begin with 0
  return t;
}

template <int D, int R>
struct Layout {
  static constexpr int kUnits = D / 128;
  static constexpr bool kAhead = kUnits < kRing;            // scores of the next tile under this one's softmax
  static constexpr int kBufs = kAhead ? 2 : 1;              // of S and of P
  static constexpr int kCols = R / 2;                       // rows (columns of S^T) of a softmax thread
  static constexpr int kQ = kRing * kUnitBytes;             // Q: D/64 blocks of R rows x 128 bytes
  static constexpr int kP = kQ + (D / 64) * R * 128;        // P: 128 keys x 128 bytes
  static constexpr int kSmall = kP + kBufs * kKeys * 128;
  static constexpr int kTmemO = 0, kTmemS = kUnits * R;
  static constexpr int kTmemUsed = kTmemS + kBufs * R;
  static constexpr int kTmem = kTmemUsed <= 32 ? 32 : kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kTmemUsed <= 512, "tensor memory");
};

template <int R>
struct Small {
  uint64_t full[kRing], empty[kRing], s_full[2], p_full[2], q_full, o_done, drain;
  uint32_t tmem;
  int32_t abort;
  Tile tile;
  int32_t ctx_max, ctx_min;
  float c[R];      // score factor: softmax_scale * log2(e) * cache_scale / the row's power of two
  float ref[R];    // reference of the weights, log2 units
  int32_t ctx[R];  // cache rows that the row sees (0: a row without a token)
  int32_t out[R];  // flat (token, head) index, -1: none
  float keep[R];   // what a move of the references leaves of sums and outputs
  float part[4][R];
  uint8_t bad[4][kKeys];  // keys of a tile that are not there (ring over tiles)
};

template <int D, int R>
constexpr int smem_bytes() {
  return Layout<D, R>::kSmall + static_cast<int>(sizeof(Small<R>)) + 1024;  // 1024: alignment of the swizzled tiles
}

// Reduce n values per lane over the warp's lanes; afterwards lane l holds the
// result of value (l * n / 32): halves the values while lanes differ in a bit.
template <int n, bool kMax>
__device__ __forceinline__ float reduce_columns(float (&v)[n], int lane) {
  int width = n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (width > 1) {
      const int half = width / 2;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        if (i < half) {
          const float mine = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
          const float got = __shfl_xor_sync(0xFFFFFFFFu, send, o);
          v[i] = kMax ? fmaxf(mine, got) : mine + got;
        }
      }
      width = half;
    } else {
      const float got = __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
      v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
    }
  }
  return v[0];
}

__device__ __forceinline__ void soft_barrier() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 256, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}
static_assert(kSoftWarps * 32 == 256, "the softmax warps' named barrier");

// 8 codes (one 32-bit word) times their block's scale -> 8 fp16 values.
__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 s) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>((w >> (8 * i)) & 0xFFu), __NV_E2M1);
    const __half2 p = __hmul2(__half2(h), s);
    r[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1) fp4_attention_kernel(const __grid_constant__ Fp4AttentionArgs a, int chunk,
                                                                    int page_shift) {
  using L = Layout<D, R>;
  extern __shared__ uint8_t s_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Small<R>& sm = *reinterpret_cast<Small<R>*>(smem + L::kSmall);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == kMmaWarp) {
    tmem_alloc<L::kTmem>(&sm.tmem);
    if (lane == 0) {
      for (int i = 0; i < kRing; ++i) {
        mbar_init(&sm.full[i], kLoadWarps);
        mbar_init(&sm.empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.s_full[i], 1);
        mbar_init(&sm.p_full[i], kSoftWarps);
      }
      mbar_init(&sm.q_full, kSoftWarps);
      mbar_init(&sm.o_done, 1);
      mbar_init(&sm.drain, 1);
      sm.abort = 0;
      fence_mbar_init();
    }
  }
  pdl_wait();
  if (warp == 0) {
    const Tile t = find_tile(a, blockIdx.x, R);
    if (lane == 0) {
      sm.tile = t;
      sm.ctx_max = -1;
      sm.ctx_min = INT32_MAX;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Tile tile = sm.tile;
  const uint32_t tmem = sm.tmem;
  if (threadIdx.x < R) {
    const int r = threadIdx.x;
    int ctx = -1;
    int32_t flat = -1;
    if (r < tile.rows) {
      const int t = tile.tok0 + (tile.base + r) / a.H;
      ctx = a.ctx_rows[t];
      if (ctx > a.max_rows) {
        flag_error(a.err, CKV_DEVERR_SEQ_LEN);
        ctx = a.max_rows;
      }
      if (ctx >= 0) flat = tile.tok0 * a.H + tile.base + r;
    }
    sm.ctx[r] = max(ctx, 0);
    sm.out[r] = flat;
    sm.ref[r] = kNegBig;
    const uint32_t in_warp = R < 32 ? (1u << (R & 31)) - 1u : 0xFFFFFFFFu;
    const int top = __reduce_max_sync(in_warp, ctx);
    const int low = __reduce_min_sync(in_warp, ctx < 0 ? INT32_MAX : ctx);
    if (lane == 0) {
      atomicMax(&sm.ctx_max, top);
      atomicMin(&sm.ctx_min, low);
    }
  }
  __syncthreads();
  const int ctx_max = sm.ctx_max, ctx_min = sm.ctx_min;
  const int k_first = blockIdx.y * chunk;
  const int k_last = min(ctx_max, k_first + chunk);
  const bool split = ctx_max > chunk;  // several CTAs share the tile
  const int n = k_last > k_first ? (k_last - k_first + kKeys - 1) / kKeys : 0;
  // nothing to add: only the first range answers for rows that see nothing
  const bool idle = n == 0 && (blockIdx.y > 0 || ctx_max < 0);

  if (!idle && warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    const int quad = warp & 3, half = warp >> 2;
    const int col0 = half * L::kCols;
    // queries: a warp takes every eighth row, scales it and stores it as fp16
#pragma unroll 1
    for (int r = warp; r < R && n > 0; r += kSoftWarps) {
      constexpr int kC = D / 32;  // channels of a lane, 4, 8 or 16 neighbours
      float v[kC];
      const int32_t flat = sm.out[r];
      if (flat >= 0) {
        const int32_t t = flat / a.H, h = flat - t * a.H;
        const uint16_t* q = a.q + t * a.q_st + h * a.q_sh + lane * kC;
        if constexpr (kC == 4) {
          const uint2 w = *reinterpret_cast<const uint2*>(q);
          v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
        } else {
#pragma unroll
          for (int i = 0; i < kC; i += 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(q + i);
            v[i] = bf16_lo(w.x), v[i + 1] = bf16_hi(w.x), v[i + 2] = bf16_lo(w.y), v[i + 3] = bf16_hi(w.y);
            v[i + 4] = bf16_lo(w.z), v[i + 5] = bf16_hi(w.z), v[i + 6] = bf16_lo(w.w), v[i + 7] = bf16_hi(w.w);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kC; ++i) v[i] = 0.f;
      }
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < kC; ++i) am = fmaxf(am, fabsf(v[i]));
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(am));
      // power of two that brings the largest channel to [2^14, 2^15); 1 for a row of zeros or with an infinity
      const int e = static_cast<int>(top >> 23);
      const int se = top == 0u || e == 255 ? 127 : min(127 + 14 + 127 - e, 253);
      const float up = __uint_as_float(static_cast<uint32_t>(se) << 23);
      if (lane == 0) sm.c[r] = a.softmax_scale * kLog2e * a.g * __uint_as_float(static_cast<uint32_t>(254 - se) << 23);
      uint32_t w[kC / 2];
#pragma unroll
      for (int i = 0; i < kC; i += 2) {
        const __half2 p = __floats2half2_rn(v[i] * up, v[i + 1] * up);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
      }
      const int ch = lane * kC;
      uint8_t* row = smem + L::kQ + (ch / 64) * (R * 128) + r * 128;
      if constexpr (kC == 4) {
        *reinterpret_cast<uint2*>(row + ((((ch % 64) / 8) ^ (r & 7)) * 16) + (ch % 8) * 2) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int i = 0; i < kC; i += 8)
          *reinterpret_cast<uint4*>(row + ((((ch + i) % 64) / 8) ^ (r & 7)) * 16) =
              make_uint4(w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
    soft_barrier();  // every row's factor is there

    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    float l[L::kCols];
#pragma unroll
    for (int i = 0; i < L::kCols; ++i) l[i] = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int buf = L::kAhead ? j & 1 : 0;
      const int key = k_first + j * kKeys + quad * 32 + lane;
      const int unit0 = j * L::kUnits;
      // the decoding warps' note on missing keys, then the scores
      ok = mbar_wait(&sm.full[unit0 % kRing], (unit0 / kRing) & 1) && mbar_wait(&sm.s_full[j & 1], (j >> 1) & 1);
      if (!ok) atomicExch(&sm.abort, 1);
      __syncwarp();
      tc_fence_after();
      const bool gone = sm.bad[j & 3][quad * 32 + lane] != 0;
      const bool masks = gone || key - lane + 32 > ctx_min;
      const uint32_t at_s = tmem + lanes + L::kTmemS + buf * R + col0;
      // scores in log2 units over the rows' references, -infinity for keys that a row does not see
      float z[L::kCols];
      tmem_ld<L::kCols>(at_s, z);
      float over = -INFINITY;
#pragma unroll
      for (int i = 0; i < L::kCols; ++i) {
        z[i] = fmaf(z[i], sm.c[col0 + i], -sm.ref[col0 + i]);
        if (masks) z[i] = !gone && key < sm.ctx[col0 + i] ? z[i] : -INFINITY;
        over = fmaxf(over, z[i]);
      }
      ok = ok && *reinterpret_cast<volatile int32_t*>(&sm.abort) == 0;
      if (soft_any(over > kJump || !ok)) {
        ok = !soft_any(!ok);
        if (!ok) break;
        // new references: the largest score so far of each row
        tmem_ld<L::kCols>(at_s, z);
#pragma unroll
        for (int i = 0; i < L::kCols; ++i) {
          z[i] *= sm.c[col0 + i];
          if (masks) z[i] = !gone && key < sm.ctx[col0 + i] ? z[i] : -INFINITY;
        }
        const float top = reduce_columns<L::kCols, true>(z, lane);
        constexpr int kShare = 32 / L::kCols;  // lanes that hold the same row's result
        if (lane % kShare == 0) sm.part[quad][col0 + lane / kShare] = top;
        soft_barrier();
        if (threadIdx.x < R) {
          const int r = threadIdx.x;
          const float old = sm.ref[r];
          const float now = fmaxf(fmaxf(fmaxf(sm.part[0][r], sm.part[1][r]), fmaxf(sm.part[2][r], sm.part[3][r])), old);
          sm.keep[r] = fast_exp2(old - now);
          sm.ref[r] = now;
        }
        soft_barrier();
#pragma unroll
        for (int i = 0; i < L::kCols; ++i) l[i] *= sm.keep[col0 + i];
        if (j > 0) {
          ok = mbar_wait(&sm.o_done, (j - 1) & 1);
          if (!ok) atomicExch(&sm.abort, 1);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int u = 0; u < L::kUnits; ++u) {
#pragma unroll
            for (int i = 0; i < L::kCols; i += 8) {
              float o[8];
              const uint32_t at = tmem + lanes + L::kTmemO + u * R + col0 + i;
              tmem_ld<8>(at, o);
#pragma unroll
              for (int x = 0; x < 8; ++x) o[x] *= sm.keep[col0 + i + x];
              tmem_st8(at, o);
            }
          }
          tc_wait_st();
        }
        tmem_ld<L::kCols>(at_s, z);
#pragma unroll
        for (int i = 0; i < L::kCols; ++i) {
          z[i] = fmaf(z[i], sm.c[col0 + i], -sm.ref[col0 + i]);
          if (masks) z[i] = !gone && key < sm.ctx[col0 + i] ? z[i] : -INFINITY;
        }
      }
      // weights, rounded to fp16, as row `key` of P
      uint8_t* row = smem + L::kP + buf * (kKeys * 128) + (quad * 32 + lane) * 128;
#pragma unroll
      for (int i = 0; i < L::kCols; i += 8) {
        uint32_t w[4];
#pragma unroll
        for (int x = 0; x < 8; x += 2) {
          const float p0 = fast_exp2(z[i + x]), p1 = fast_exp2(z[i + x + 1]);
          l[i + x] += p0;
          l[i + x + 1] += p1;
          const __half2 h = __floats2half2_rn(p0, p1);
          w[x / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(row + ((((col0 + i) / 8) ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[j & 1]);
    }
    // --------------------------------------------------------------- output
    if (n > 0 && ok) {
      ok = mbar_wait(&sm.o_done, (n - 1) & 1);
      __syncwarp();
      tc_fence_after();
    }
    if (!ok && lane == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
    const float sum = reduce_columns<L::kCols, false>(l, lane);
    constexpr int kShare = 32 / L::kCols;
    soft_barrier();
    if (lane % kShare == 0) sm.part[quad][col0 + lane / kShare] = sum;
    soft_barrier();
    float* ws = static_cast<float*>(a.workspace);
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * gridDim.y + blockIdx.y;
    if (threadIdx.x < R) {
      const int r = threadIdx.x;
      const float total = sm.part[0][r] + sm.part[1][r] + sm.part[2][r] + sm.part[3][r];
      const int32_t flat = sm.out[r];
      if (split) {
        float* ml = ws + static_cast<int64_t>(gridDim.x) * gridDim.y * R * D + slot * R * 2;
        ml[r] = sm.ref[r];
        ml[R + r] = total;
      } else {
        float m = sm.ref[r], all = total;
        if (a.sink && flat >= 0) {
          const float s = a.sink[flat % a.H] * kLog2e;
          const float top = fmaxf(m, s);
          const float keep = fast_exp2(m - top);  // 0 where no key was seen
          all = (total == 0.f ? 0.f : total * keep) + (s == top ? 1.f : fast_exp2(s - top));
          sm.c[r] = all == 0.f ? 0.f : keep * a.g / all;
          m = top;
        } else {
          sm.c[r] = all == 0.f ? 0.f : a.g / all;
        }
        if (a.lse && flat >= 0) a.lse[flat] = all == 0.f ? -INFINITY : (m + log2f(all)) * kLn2;
      }
    }
    soft_barrier();
#pragma unroll 1
    for (int u = 0; u < L::kUnits; ++u) {
      float o[L::kCols];
      if (n > 0) {
        tmem_ld<L::kCols>(tmem + lanes + L::kTmemO + u * R + col0, o);
      } else {
#pragma unroll
        for (int i = 0; i < L::kCols; ++i) o[i] = 0.f;
      }
      const int ch = u * 128 + quad * 32 + lane;
      if (split) {
#pragma unroll
        for (int i = 0; i < L::kCols; ++i) ws[(slot * R + col0 + i) * D + ch] = o[i];
      } else {
#pragma unroll
        for (int i = 0; i < L::kCols; i += 2) {
          // neighbouring lanes (channels) trade halves: the even one writes both channels of row i, the odd one of row i + 1
          const float v0 = n > 0 ? o[i] * sm.c[col0 + i] : 0.f, v1 = n > 0 ? o[i + 1] * sm.c[col0 + i + 1] : 0.f;
          const float got = __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? v0 : v1, 1);
          const int32_t flat = sm.out[col0 + i + (lane & 1)];
          const uint32_t w = lane & 1 ? pack_bf16x2_rn(got, v1) : pack_bf16x2_rn(v0, got);
          if (flat >= 0) *reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(flat) * D + (ch & ~1)) = w;
        }
      }
    }
    tc_fence_before();
  } else if (!idle && warp == kMmaWarp && n > 0) {
    // ------------------------------------------------------------ tensor cores
    if (elect_one()) {
      constexpr uint32_t kIdescS = idesc_f16(R, false, false), kIdescO = idesc_f16(R, true, true);
      const uint32_t base = smem_u32(smem);
      bool ok = mbar_wait(&sm.q_full, 0);
      auto scores = [&](int j) {
        const uint32_t d = tmem + L::kTmemS + (L::kAhead ? j & 1 : 0) * R;
        for (int u = 0; u < L::kUnits && ok; ++u) {
          const int c = j * L::kUnits + u;
          ok = mbar_wait(&sm.full[c % kRing], (c / kRing) & 1);
          tc_fence_after();
          if (!ok) break;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint64_t da = smem_desc_sw128(base + (c % kRing) * kUnitBytes + (s / 4) * 16384 + (s % 4) * 32, 16, 1024);
            const uint64_t db = smem_desc_sw128(base + L::kQ + (u * 2 + s / 4) * (R * 128) + (s % 4) * 32, 16, 1024);
            mma_f16_ss(d, da, db, kIdescS, u > 0 || s > 0);
          }
        }
        tc_commit(&sm.s_full[j & 1]);
      };
      if (ok) scores(0);
      for (int j = 0; j < n && ok; ++j) {
        if (L::kAhead && j + 1 < n) scores(j + 1);
        ok = ok && mbar_wait(&sm.p_full[j & 1], (j >> 1) & 1);
        tc_fence_after();
        if (!ok) break;
        const uint32_t p = base + L::kP + (L::kAhead ? j & 1 : 0) * (kKeys * 128);
        for (int u = 0; u < L::kUnits; ++u) {
          const int c = j * L::kUnits + u;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint64_t da = smem_desc_sw128(base + (c % kRing) * kUnitBytes + s * 2048, 16384, 1024);
            const uint64_t db = smem_desc_sw128(p + s * 2048, 16384, 1024);
            mma_f16_ss(tmem + L::kTmemO + u * R, da, db, kIdescO, j > 0 || s > 0);
          }
          tc_commit(&sm.empty[c % kRing]);
        }
        tc_commit(&sm.o_done);
        if (!L::kAhead && j + 1 < n) scores(j + 1);
      }
      if (!ok) atomicExch(&sm.abort, 1);
      // tensor memory is given back only when no MMA writes it any more
      tc_commit(&sm.drain);
      if (!mbar_wait(&sm.drain, 0) || !ok) flag_error(a.err, CKV_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (!idle && warp > kMmaWarp && n > 0) {
    // ------------------------------------------------------- load and decode
    const int tid = threadIdx.x - (kMmaWarp + 1) * 32;
    const int key = tid >> 1, part = tid & 1;  // 64 channels of a unit: 32 code bytes, 4 scale bytes
    const int32_t* table = a.table + static_cast<int64_t>(tile.b) * a.table_stride;
    const int64_t page_bytes = fp4_page_bytes<D>(a.page_size);
    struct Unit {
      uint4 c[2];
      uint32_t s;
    };
    Unit reg[kRing];
    const uint8_t *codes = nullptr, *scales = nullptr;
    bool there = false, bad = false;
    // where the key's row of tile j is
    auto locate = [&](int j) {
      const int k = k_first + j * kKeys + key;
      there = false;
      bad = false;
      if (k < k_last) {
        const int pg = page_shift >= 0 ? k >> page_shift : k / a.page_size;
        const int row = k - pg * a.page_size;
        const int32_t page = table[pg];
        if (page >= 0 && page < a.num_pages) {
          const uint8_t* p = a.cache + page * page_bytes;
          codes = p + static_cast<int64_t>(row) * (D / 2) + part * 32;
          scales = p + static_cast<int64_t>(a.page_size) * (D / 2) + static_cast<int64_t>(row) * (D / 16) + part * 4;
          there = true;
        } else {
          bad = true;
          if (part == 0) flag_error(a.err, CKV_DEVERR_CACHE_LOC);
        }
      }
    };
    auto load = [&](Unit& x, int u) {
      x.c[0] = x.c[1] = make_uint4(0, 0, 0, 0);
      x.s = 0;
      if (there) {
        x.c[0] = *reinterpret_cast<const uint4*>(codes + u * 64);
        x.c[1] = *reinterpret_cast<const uint4*>(codes + u * 64 + 16);
        x.s = *reinterpret_cast<const uint32_t*>(scales + u * 8);
      }
    };
    const int total = n * L::kUnits;
    bool was_bad[kRing];
#pragma unroll
    for (int c = 0; c < kRing; ++c) {
      if (c % L::kUnits == 0 && c < total) locate(c / L::kUnits);
      if (c < total) load(reg[c], c % L::kUnits);
      was_bad[c] = bad;
    }
    bool ok = true;
#pragma unroll 1
    for (int c0 = 0; c0 < total && ok; c0 += kRing) {
#pragma unroll
      for (int i = 0; i < kRing; ++i) {
        const int c = c0 + i;
        if (c < total && ok) {
          if (c >= kRing) ok = mbar_wait(&sm.empty[i], ((c / kRing) - 1) & 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (ok) {
            uint8_t* unit = smem + i * kUnitBytes + part * 16384 + key * 128;
            const uint32_t word[8] = {reg[i].c[0].x, reg[i].c[0].y, reg[i].c[0].z, reg[i].c[0].w,
                                      reg[i].c[1].x, reg[i].c[1].y, reg[i].c[1].z, reg[i].c[1].w};
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              const __half_raw sr = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>((reg[i].s >> (8 * (w / 2))) & 0xFFu), __NV_E4M3);
              *reinterpret_cast<uint4*>(unit + ((w ^ (key & 7)) * 16)) = decode8(word[w], __half2half2(__half(sr)));
            }
            if (c % L::kUnits == 0 && part == 0) sm.bad[(c / L::kUnits) & 3][key] = was_bad[i] ? 1 : 0;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.full[i]);
            const int next = c + kRing;
            if (next < total) {
              if (next % L::kUnits == 0) locate(next / L::kUnits);
              load(reg[i], next % L::kUnits);
              was_bad[i] = bad;
            }
          }
        }
      }
    }
    if (!ok) {
      atomicExch(&sm.abort, 1);
      if (lane == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
    }
  }
  pdl_trigger();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<L::kTmem>(tmem);
  }
}

// Joins the ranges of a tile: one warp per row, in the order of the ranges.
template <int D, int R>
__global__ void __launch_bounds__(128) fp4_join_kernel(const __grid_constant__ Fp4AttentionArgs a, int chunk, int splits) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const Tile t = find_tile(a, blockIdx.x, R);
  if (t.rows <= 0) return;
  int ctx_max = 0;
  for (int i = lane; i < R; i += 32)
    if (i < t.rows) ctx_max = max(ctx_max, min(a.ctx_rows[t.tok0 + (t.base + i) / a.H], a.max_rows));
  ctx_max = __reduce_max_sync(0xFFFFFFFFu, ctx_max);
  const int used = (ctx_max + chunk - 1) / chunk;
  const int r = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (used <= 1 || r >= t.rows) return;
  if (a.ctx_rows[t.tok0 + (t.base + r) / a.H] < 0) return;
  const float* ws = static_cast<const float*>(a.workspace);
  const int64_t slot0 = static_cast<int64_t>(blockIdx.x) * splits;
  const float* ml = ws + static_cast<int64_t>(gridDim.x) * splits * R * D + slot0 * R * 2;
  const int64_t flat = static_cast<int64_t>(t.tok0) * a.H + t.base + r;
  float m = kNegBig;
  for (int s = lane; s < used; s += 32) m = fmaxf(m, ml[s * 2 * R + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float all = 0.f;
  if (a.sink) {
    const float s = a.sink[flat % a.H] * kLog2e;
    m = fmaxf(m, s);
    all = s == m ? 1.f : fast_exp2(s - m);
  }
  float acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  for (int s = 0; s < used; ++s) {
    const float l = ml[s * 2 * R + R + r];
    const float w = fast_exp2(ml[s * 2 * R + r] - m);
    all += l == 0.f ? 0.f : l * w;
    const float4* o = reinterpret_cast<const float4*>(ws + ((slot0 + s) * R + r) * D);
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const float4 v = o[i * 32 + lane];
      acc[4 * i] = fmaf(v.x, w, acc[4 * i]);
      acc[4 * i + 1] = fmaf(v.y, w, acc[4 * i + 1]);
      acc[4 * i + 2] = fmaf(v.z, w, acc[4 * i + 2]);
      acc[4 * i + 3] = fmaf(v.w, w, acc[4 * i + 3]);
    }
  }
  const float inv = all == 0.f ? 0.f : a.g / all;
#pragma unroll
  for (int i = 0; i < D / 128; ++i)
    *reinterpret_cast<uint2*>(a.out + flat * D + i * 128 + lane * 4) =
        make_uint2(pack_bf16x2_rn(acc[4 * i] * inv, acc[4 * i + 1] * inv), pack_bf16x2_rn(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv));
  if (lane == 0 && a.lse) a.lse[flat] = all == 0.f ? -INFINITY : (m + log2f(all)) * kLn2;
}

template <int D, int R>
cudaError_t launch(const Fp4AttentionArgs& a, const SplitPlan& p, bool use_pdl, cudaStream_t s) {
  cudaError_t e = set_max_smem_once<fp4_attention_kernel<D, R>>(smem_bytes<D, R>());
  if (e != cudaSuccess) return e;
  int shift = -1;
  if ((a.page_size & (a.page_size - 1)) == 0)
    for (shift = 0; (1 << shift) != a.page_size;) ++shift;
  e = launch_ex(fp4_attention_kernel<D, R>, dim3(p.tiles, p.splits), dim3(kThreads), smem_bytes<D, R>(), use_pdl, s, a, p.chunk,
                shift);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_ex(fp4_join_kernel<D, R>, dim3(p.tiles, R / 4), dim3(128), 0, true, s, a, p.chunk, p.splits);
}

template <int D>
cudaError_t launch_d(const Fp4AttentionArgs& a, const SplitPlan& p, bool use_pdl, cudaStream_t s) {
  return p.R == 16 ? launch<D, 16>(a, p, use_pdl, s) : p.R == 32 ? launch<D, 32>(a, p, use_pdl, s) : launch<D, 64>(a, p, use_pdl, s);
}

}  // namespace

int64_t fp4_attention_workspace(int64_t T, int32_t B, int32_t H, int32_t D, int64_t max_rows) {
  const SplitPlan p = plan_splits(T, B, H, max_rows);
  return p.splits == 1 ? 0 : static_cast<int64_t>(p.tiles) * p.splits * p.R * (D + 2) * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_fp4_attention(const Fp4AttentionArgs& a, int D, bool use_pdl, cudaStream_t s) {
  const SplitPlan p = plan_splits(a.T, a.B, a.H, a.max_rows);
  return D == 128 ? launch_d<128>(a, p, use_pdl, s) : D == 256 ? launch_d<256>(a, p, use_pdl, s) : launch_d<512>(a, p, use_pdl, s);
}

}  // namespace ckv
