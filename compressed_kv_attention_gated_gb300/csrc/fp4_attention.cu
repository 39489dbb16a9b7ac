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
// Warpgroups (4 warps) 0 and 1: softmax; 2: its first warp issues the MMAs; 3 and 4: load and decode.
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 12, kLoadWarps = 8;
constexpr int kThreads = (kLoadWarp + kLoadWarps) * 32;
// Registers per thread: 96 at launch (640 x 96 = 61,440), then 256 x 120 + 128 x 64 + 256 x 88 = 61,440.
constexpr int kSoftRegs = 120, kMmaRegs = 64, kLoadRegs = 88;
static_assert(256 * kSoftRegs + 128 * kMmaRegs + 256 * kLoadRegs <= kThreads * 96, "registers of the launch");
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
  static constexpr int kOutPitch = D * 2 + 64;              // output rows on their way out: two rows of 64 bytes hit all banks
  static_assert(R * kOutPitch <= kRing * kUnitBytes, "output staging");
  static constexpr int kTmemO = 0, kTmemS = kUnits * R;
  static constexpr int kTmemK = kTmemS + kBufs * R;         // decoded units as A of the first product, 64 columns each
  static constexpr int kSlots = kTmemK + 4 * 64 <= 512 ? 4 : 3;
  static constexpr int kTmemUsed = kTmemK + kSlots * 64;
  static constexpr int kTmem = kTmemUsed <= 32 ? 32 : kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kTmemUsed <= 512, "tensor memory");
};

template <int R>
struct Small {
  uint64_t full[kRing], empty[kRing], a_free[4], s_full[2], p_full[2], q_full, o_done, drain;
  uint32_t tmem;
  int32_t abort;
  Tile tile;
  int32_t ctx_max, ctx_min;
  alignas(16) float c[R];  // score factor: softmax_scale * log2(e) * cache_scale / the row's power of two
  alignas(16) float ref[R];  // reference of the weights, log2 units
  alignas(16) int32_t ctx[R];  // cache rows that the row sees (0: a row without a token)
  int64_t q[R];    // where the row's query begins, elements
  int32_t out[R];  // flat (token, head) index, -1: none
  float sink[R];   // log2 units, -infinity without
  alignas(16) float keep[R];  // what a move of the references leaves of sums and outputs
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

// Columns of a per-row array, 16 bytes at a time.  They are read in one go before
// anything is stored: the compiler may not move a load over a store that could alias.
template <int n>
__device__ __forceinline__ void load_cols(const float* p, float (&v)[n]) {
#pragma unroll
  for (int i = 0; i < n; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(p + i);
    v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
  }
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

// Decoding on the integer and fp16 pipes (a hardware conversion of two codes
// runs at an eighth of their rate).  A code's exponent and mantissa bits at bits
// 11..9 of an fp16 are its value * 2^-14 (a subnormal code lands on a subnormal),
// an e4m3's bits shifted up by 7 its value * 2^-8; the scale is brought to
// scale * 2^7 (at most 57344), so that the product is value * 2^-7: at least
// 2^-17 with 6 significant bits, exact in fp16.  Every byte decodes to a finite
// number.  The left shifts are multiplications by kernel parameters, which the
// multiplier pipe does beside the logic pipe.  Codes come out in pairs (i, i + 4) of the word's eight.
constexpr float kUnscale = 128.f;

struct Shifts {
  uint32_t by[6];  // 2^9, 2^12, 2^5, 2^8, 2^1, 2^4
};

__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 s, const Shifts& k) {
  const uint32_t m[4] = {((w * k.by[0]) & 0x0E000E00u) | ((w * k.by[1]) & 0x80008000u),
                         ((w * k.by[2]) & 0x0E000E00u) | ((w * k.by[3]) & 0x80008000u),
                         ((w * k.by[4]) & 0x0E000E00u) | ((w * k.by[5]) & 0x80008000u), ((w >> 3) & 0x0E000E00u) | (w & 0x80008000u)};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&m[i]), s);
    r[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Four e4m3 bytes, each twice in a register, times 2^7.
__device__ __forceinline__ void decode_scales(uint32_t b, __half2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = b >> (8 * i);  // bytes i and i + 2 in the low byte of each half
    const uint32_t m = ((x & 0x007F007Fu) << 7) | ((x & 0x00800080u) << 8);
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&m), __float2half2_rn(32768.f));
    s[i] = __low2half2(v);
    s[i + 2] = __high2half2(v);
  }
}

// Where channel c of a row is kept in the decoded tile (and so in Q and O): the
// eight channels of a word in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ constexpr int channel_of(int place) {
  return (place & ~7) | ((place & 1) << 2) | ((place >> 1) & 3);
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1) fp4_attention_kernel(const __grid_constant__ Fp4AttentionArgs a, int chunk,
                                                                    int page_shift, const __grid_constant__ Shifts shifts) {
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
        mbar_init(&sm.a_free[i], 1);
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
      if (ctx >= 0) {
        flat = tile.tok0 * a.H + tile.base + r;
        sm.q[r] = t * a.q_st + (flat - t * a.H) * a.q_sh;
      }
    }
    sm.ctx[r] = max(ctx, 0);
    sm.out[r] = flat;
    sm.ref[r] = kNegBig;
    sm.sink[r] = a.sink && flat >= 0 ? a.sink[flat % a.H] * kLog2e : -INFINITY;
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

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    if (!idle) {
    // ------------------------------------------------------------- softmax
    const int quad = warp & 3, half = warp >> 2;
    const int col0 = half * L::kCols;
    // queries: a warp takes R/8 rows, a lane eight channels of a row (16 at D = 512); all
    // loads are issued before the first is used
    if (n > 0) {
      constexpr int kC = D == 512 ? 16 : 8;     // channels of a lane
      constexpr int kSpan = D / kC;             // lanes of a row
      constexpr int kLoads = R / kSoftWarps * kSpan / 32;
      constexpr int kBatch = kLoads < 8 ? kLoads : 8;  // rows in flight (registers)
      const int sub = lane / kSpan, ch = lane % kSpan * kC;
      static_assert(kLoads >= 1 && kLoads % kBatch == 0, "");
#pragma unroll 1
      for (int i0 = 0; i0 < kLoads; i0 += kBatch) {
      uint4 raw[kBatch][kC / 8];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = warp * (R / kSoftWarps) + (i0 + i) * (32 / kSpan) + sub;
        const bool on = sm.out[r] >= 0;
        const uint4* q = reinterpret_cast<const uint4*>(a.q + sm.q[r] + ch);
#pragma unroll
        for (int x = 0; x < kC / 8; ++x) raw[i][x] = on ? q[x] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = warp * (R / kSoftWarps) + (i0 + i) * (32 / kSpan) + sub;
        uint32_t am = 0;  // the largest magnitude: bf16 bits order like the values
#pragma unroll
        for (int x = 0; x < kC / 8; ++x) {
          const uint32_t w[4] = {raw[i][x].x, raw[i][x].y, raw[i][x].z, raw[i][x].w};
#pragma unroll
          for (int y = 0; y < 4; ++y) am = __vmaxu2(am, w[y] & 0x7FFF7FFFu);
        }
        am = max(am >> 16, am & 0xFFFFu);
#pragma unroll
        for (int o = 1; o < kSpan; o <<= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
        // power of two that brings the largest channel to [2^14, 2^15); 1 for a row of zeros or with an infinity or NaN
        const int e = static_cast<int>(am >> 7);
        const int se = am == 0u || e == 255 ? 127 : min(127 + 14 + 127 - e, 253);
        const float up = __uint_as_float(static_cast<uint32_t>(se) << 23);
        if (lane % kSpan == 0)
          sm.c[r] = a.softmax_scale * kLog2e * kUnscale * a.g * __uint_as_float(static_cast<uint32_t>(254 - se) << 23);
        uint8_t* row = smem + L::kQ + (ch / 64) * (R * 128) + r * 128;
#pragma unroll
        for (int x = 0; x < kC / 8; ++x) {
          const uint32_t w[4] = {raw[i][x].x, raw[i][x].y, raw[i][x].z, raw[i][x].w};
          uint32_t v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {  // channels y and y + 4 of the eight
            const float lo = y & 1 ? bf16_hi(w[y / 2]) : bf16_lo(w[y / 2]), hi = y & 1 ? bf16_hi(w[2 + y / 2]) : bf16_lo(w[2 + y / 2]);
            const __half2 p = __floats2half2_rn(lo * up, hi * up);
            v[y] = *reinterpret_cast<const uint32_t*>(&p);
          }
          *reinterpret_cast<uint4*>(row + ((((ch % 64) / 8 + x) ^ (r & 7)) * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
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
      // scores in log2 units, -infinity for keys that a row does not see
      auto read_scores = [&](float (&z)[L::kCols]) {
        tmem_ld<L::kCols>(at_s, z);
#pragma unroll
        for (int i = 0; i < L::kCols; i += 4) {
          const float4 c = *reinterpret_cast<const float4*>(&sm.c[col0 + i]);
          z[i] *= c.x, z[i + 1] *= c.y, z[i + 2] *= c.z, z[i + 3] *= c.w;
        }
        if (masks) {
#pragma unroll
          for (int i = 0; i < L::kCols; i += 4) {
            const int4 x = *reinterpret_cast<const int4*>(&sm.ctx[col0 + i]);
            z[i] = !gone && key < x.x ? z[i] : -INFINITY;
            z[i + 1] = !gone && key < x.y ? z[i + 1] : -INFINITY;
            z[i + 2] = !gone && key < x.z ? z[i + 2] : -INFINITY;
            z[i + 3] = !gone && key < x.w ? z[i + 3] : -INFINITY;
          }
        }
      };
      auto over_refs = [&](float (&z)[L::kCols]) {
        float over = -INFINITY;
#pragma unroll
        for (int i = 0; i < L::kCols; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&sm.ref[col0 + i]);
          z[i] -= f.x, z[i + 1] -= f.y, z[i + 2] -= f.z, z[i + 3] -= f.w;
          over = fmaxf(over, fmaxf(fmaxf(z[i], z[i + 1]), fmaxf(z[i + 2], z[i + 3])));
        }
        return over;
      };
      float z[L::kCols];
      read_scores(z);
      const float over = over_refs(z);
      ok = ok && *reinterpret_cast<volatile int32_t*>(&sm.abort) == 0;
      if (soft_any(over > kJump || !ok)) {
        ok = !soft_any(!ok);
        if (!ok) break;
        // new references: the largest score so far of each row
        read_scores(z);
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
        if (j > 0) {
          load_cols<L::kCols>(&sm.keep[col0], z);
#pragma unroll
          for (int i = 0; i < L::kCols; ++i) l[i] *= z[i];
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
              for (int x = 0; x < 8; ++x) o[x] *= z[i + x];
              tmem_st8(at, o);
            }
          }
          tc_wait_st();
        }
        read_scores(z);
        over_refs(z);
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
        if (a.sink) {
          const float s = sm.sink[r];
          const float top = fmaxf(m, s);
          const float keep = fast_exp2(m - top);  // 0 where no key was seen
          all = (total == 0.f ? 0.f : total * keep) + (s == top ? 1.f : fast_exp2(s - top));
          sm.c[r] = all == 0.f ? 0.f : keep * kUnscale * a.g / all;
          m = top;
        } else {
          sm.c[r] = all == 0.f ? 0.f : kUnscale * a.g / all;
        }
        if (a.lse && flat >= 0) a.lse[flat] = all == 0.f ? -INFINITY : (m + log2f(all)) * kLn2;
      }
    }
    soft_barrier();
    load_cols<L::kCols>(&sm.c[col0], l);
#pragma unroll 1
    for (int u = 0; u < L::kUnits; ++u) {
      float o[L::kCols];
      if (n > 0) {
        tmem_ld<L::kCols>(tmem + lanes + L::kTmemO + u * R + col0, o);
      } else {
#pragma unroll
        for (int i = 0; i < L::kCols; ++i) o[i] = 0.f;
      }
      const int ch = u * 128 + channel_of(quad * 32 + lane);
      if (split) {
#pragma unroll
        for (int i = 0; i < L::kCols; ++i) ws[(slot * R + col0 + i) * D + ch] = o[i];
      } else {
        // through shared memory (the ring is free) so that rows leave in 16-byte pieces; lanes
        // with channels 2c and 2c + 1 (two apart) trade halves: one has both channels of row i, the other of row i + 1
        const bool odd = lane & 2;
        uint8_t* to = smem + (col0 + (odd ? 1 : 0)) * L::kOutPitch + (ch & ~1) * 2;
#pragma unroll
        for (int i = 0; i < L::kCols; i += 2) {
          const float v0 = o[i] * l[i], v1 = o[i + 1] * l[i + 1];
          const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 2);
          *reinterpret_cast<uint32_t*>(to + i * L::kOutPitch) = odd ? pack_bf16x2_rn(got, v1) : pack_bf16x2_rn(v0, got);
        }
      }
    }
    if (!split) {
      soft_barrier();
      constexpr int kRowLanes = D / 8;  // 16-byte pieces of a row
#pragma unroll 4
      for (int i = threadIdx.x; i < R * kRowLanes; i += kSoftWarps * 32) {
        const int r = i / kRowLanes, x = i % kRowLanes;
        const int32_t flat = sm.out[r];
        if (flat >= 0)
          *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(flat) * D + x * 8) =
              *reinterpret_cast<const uint4*>(smem + r * L::kOutPitch + x * 16);
      }
    }
    tc_fence_before();
    }
  } else if (warp < kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == kMmaWarp && n > 0) {
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
            const uint64_t db = smem_desc_sw128(base + L::kQ + (u * 2 + s / 4) * (R * 128) + (s % 4) * 32, 16, 1024);
            mma_f16_ts(d, tmem + L::kTmemK + (c % L::kSlots) * 64 + s * 8, db, kIdescS, u > 0 || s > 0);
          }
          tc_commit(&sm.a_free[c % L::kSlots]);
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
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    if (n > 0) {
    // ------------------------------------------------------- load and decode
    // a thread has 64 channels of a unit's 128 for one key, that of its lane of tensor memory;
    // neighbouring lanes have neighbouring keys, whose 16-byte chunks the swizzle spreads over all banks
    const int quad = warp & 3, key = quad * 32 + lane, part = (warp - kLoadWarp) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int32_t* table = a.table + static_cast<int64_t>(tile.b) * a.table_stride;
    const int64_t page_bytes = fp4_page_bytes<D>(a.page_size);
    struct Unit {
      uint4 c[2];  // 64 codes
      uint32_t s;  // 4 scales
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
      x.s = there ? *reinterpret_cast<const uint32_t*>(scales + u * 8) : 0u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.c[i] = make_uint4(0, 0, 0, 0);
        if (there) x.c[i] = *reinterpret_cast<const uint4*>(codes + u * 64 + i * 16);
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
          if (c >= L::kSlots) ok = mbar_wait(&sm.a_free[c % L::kSlots], ((c / L::kSlots) - 1) & 1);
          if (c >= kRing) ok = ok && mbar_wait(&sm.empty[i], ((c / kRing) - 1) & 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (ok) {
            tc_fence_after();
            uint8_t* unit = smem + i * kUnitBytes + part * 16384 + key * 128;
            const uint32_t a_tile = tmem + lanes + L::kTmemK + (c % L::kSlots) * 64 + part * 32;
            __half2 sc[4];
            decode_scales(reg[i].s, sc);
#pragma unroll
            for (int b = 0; b < 4; ++b) {  // blocks of 16 channels
              const uint4 x = reg[i].c[b / 2];
              const uint4 lo = decode8(b & 1 ? x.z : x.x, sc[b], shifts), hi = decode8(b & 1 ? x.w : x.y, sc[b], shifts);
              *reinterpret_cast<uint4*>(unit + (((2 * b) ^ (key & 7)) * 16)) = lo;
              *reinterpret_cast<uint4*>(unit + (((2 * b + 1) ^ (key & 7)) * 16)) = hi;
              tmem_st8(a_tile + b * 8, lo, hi);
            }
            if (c % L::kUnits == 0 && part == 0) sm.bad[(c / L::kUnits) & 3][key] = was_bad[i] ? 1 : 0;
            tc_wait_st();
            tc_fence_before();
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
  const float inv = all == 0.f ? 0.f : kUnscale * a.g / all;
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
                shift, Shifts{{1u << 9, 1u << 12, 1u << 5, 1u << 8, 1u << 1, 1u << 4}});
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
