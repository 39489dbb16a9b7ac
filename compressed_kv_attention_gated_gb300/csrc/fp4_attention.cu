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
// so that M is always 128 whatever the number of heads, and O (D x R) fits tensor
// memory.  A cache row is decoded once, to fp16, into tensor memory (a lane per key,
// A of the first product) and into shared memory (128-byte swizzle, MN-major A of
// the second); P goes through shared memory as an MN-major B.
//
// Exactness: a decoded value is code * scale (2 + 4 significant bits, 2^-10 ..
// 2688), exact in fp16; cache_scale goes into the factor of the scores and of
// the output.  A query row is scaled by a power of two to fp16's top, which
// keeps its 8 bits for every channel above 2^-28 of its largest.  Scores, sums
// and outputs are fp32.  Only the weights are rounded, to fp16: by 2^-11 of their
// value, and those below 2^-21 of the row's largest by 2^-32 of that.
//
// Softmax: in S^T a thread holds one key for R/2 rows, so a row's maximum is
// spread over 128 threads.  It is not formed per tile: weights are taken
// against a reference that is 2^7 below the largest of the tile that set it, and
// only when some weight exceeds 2^15 (fp16 goes to 65504) the CTA forms the true
// maxima and rescales O and the sums.  Sums stay per thread until the end.
//
// Roles: 8 softmax warps (also query load and output), 1 warp that issues the
// MMAs, 1 that brings the next CTA's first bytes to L2, and groups of 4 warps that
// load and decode cache rows into a ring of four units of 128 keys x 128 channels:
// two groups, three at D = 512.  With D < 512 the ring holds more than a tile, and
// the scores of the next tile are computed under the softmax of this one.
//
// Long rows of few tiles are split over CTAs (blockIdx.y), whose partial
// outputs (fp32) and references a second kernel joins in a fixed order.
//
// What bounds it (D = 512, R = 64, 128 keys, 8 k clocks): softmax 2.7 k, then the
// second product 2.0 k, and what is left of the next tile's decoding (its units
// come free with the second product) and first product, 3 k; the products read
// 256 KB of shared memory per tile and the decoding writes 128 KB (3.1 k at 128
// bytes per clock).  Around its tiles a CTA spends about 18 k clocks (setup 3 k,
// queries 8.5 k, output 5 k), which one CTA per SM cannot hide.  Measured (GB300):
// 1024 requests x 64 heads x 512 rows on average 206 us (334 TFLOP/s), 512 requests
// x 16 heads x 922-1024 rows 104 us, one request of 16 heads over 131,072 rows 32 us.
// Slower forms: decoding in two groups (237 us for the first of these, when three
// took 230), in four at R <= 32 (116 us for the second, when three took 110; at
// D = 256 80 us, when two took 68); output straight from registers (211 us, when 206);
// on a prompt that took 1.70 ms: K as A of both products from shared memory
// (1.80 ms), decoding twice so that the scores run ahead of the second product (2.21 ms).
#include "fp4_attention.cuh"

namespace ckv {
namespace {

// Warpgroups (4 warps) 0 and 1: softmax; 2: its first warp issues the MMAs; 3 and 4: load and decode.
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 12;
// Registers per thread at launch: 640 x 96 or (D = 512) 768 x 80, 61,440 both; then 256 x 112 +
// 128 x 64 and 256 x 96 or 384 x 64, the same.  All kernels of this form but <128, 16> spill
// (6 to 42 bytes stored, 2 to 110 loaded per thread).
constexpr int kSoftRegs = 112, kMmaRegs = 64;
template <int D, int R>
struct Layout {
  static constexpr int kUnits = D / 128;
  static constexpr int kGroups = D == 512 ? 3 : 2;          // groups of four decoding warps
  static constexpr int kThreads = (kLoadWarp + kGroups * 4) * 32;
  static constexpr int kLoadRegs = D == 512 ? 64 : 96;
  static_assert(256 * kSoftRegs + 128 * kMmaRegs + kGroups * 128 * kLoadRegs <= kThreads * (D == 512 ? 80 : 96), "registers");
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
  uint32_t bad[4][4];  // a bit per key of a tile whose page is not there (ring over tiles)
};

template <int D, int R>
constexpr int smem_bytes() {
  return Layout<D, R>::kSmall + static_cast<int>(sizeof(Small<R>)) + 1024;  // 1024: alignment of the swizzled tiles
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

template <int D, int R>
__global__ void __launch_bounds__((Layout<D, R>::kThreads), 1) fp4_attention_kernel(const __grid_constant__ Fp4AttentionArgs a, int chunk,
                                                                    int page_shift) {
  using L = Layout<D, R>;
  extern __shared__ uint8_t s_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Small<R>& sm = *reinterpret_cast<Small<R>*>(smem + L::kSmall);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == kMmaWarp && lane == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.full[i], 4);
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
  pdl_wait();
  if (warp == 0) {
    const Tile t = find_tile(a, blockIdx.x, R);
    if (lane == 0) {
      sm.tile = t;
      sm.ctx_max = -1;
      sm.ctx_min = INT32_MAX;
    }
  }
  __syncthreads();
  const Tile tile = sm.tile;
  if (tile.rows <= 0) return;  // more tiles than rows need
  if (warp == kMmaWarp) tmem_alloc<L::kTmem>(&sm.tmem);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
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
      if (n > 0) load_queries<D, R, R / kSoftWarps>(a, warp * (R / kSoftWarps), sm.out, sm.q, sm.c, smem + L::kQ);
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
        const int last = (j + 1) * L::kUnits - 1;
        // the decoding warps' note on missing keys, then the scores
        ok = mbar_wait_near(&sm.full[last % kRing], (last / kRing) & 1) && mbar_wait_near(&sm.s_full[j & 1], (j >> 1) & 1);
        if (!ok) atomicExch(&sm.abort, 1);
        __syncwarp();
        tc_fence_after();
        const bool gone = (sm.bad[j & 3][quad] >> lane) & 1;
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
          // new references: kTop below the largest score so far of each row
          read_scores(z);
          const float top = reduce_columns<L::kCols, true>(z, lane);
          constexpr int kShare = 32 / L::kCols;  // lanes that hold the same row's result
          if (lane % kShare == 0) sm.part[quad][col0 + lane / kShare] = top;
          soft_barrier();
          if (threadIdx.x < R) {
            const int r = threadIdx.x;
            const float old = sm.ref[r];
            const float high = fmaxf(fmaxf(sm.part[0][r], sm.part[1][r]), fmaxf(sm.part[2][r], sm.part[3][r]));
            const float now = fmaxf(high - kTop, old);
            sm.keep[r] = fast_exp2(old - now);
            sm.ref[r] = now;
          }
          soft_barrier();
          if (j > 0) {
            load_cols<L::kCols>(&sm.keep[col0], z);
#pragma unroll
            for (int i = 0; i < L::kCols; ++i) l[i] *= z[i];
            ok = mbar_wait_near(&sm.o_done, (j - 1) & 1);
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
      // the rows' factors while the last products still run
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
            sm.c[r] = all == 0.f ? 0.f : keep * a.g / all;
            m = top;
          } else {
            sm.c[r] = all == 0.f ? 0.f : a.g / all;
          }
          // nothing at all: no sink, or one that is -infinity in log2 units
          if (a.lse && flat >= 0) a.lse[flat] = all == 0.f ? a.sink ? a.sink[flat % a.H] : -INFINITY : (m + log2f(all)) * kLn2;
        }
      }
      soft_barrier();
      load_cols<L::kCols>(&sm.c[col0], l);
      if (n > 0 && ok) {
        // not o_done: a warp that has not waited for tile n - 2 could take its phase for the last one's
        ok = mbar_wait_near(&sm.drain, 0);
        __syncwarp();
        tc_fence_after();
      }
      if (!ok && lane == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
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
          // through shared memory (the ring is free) so that rows leave in 16-byte pieces; neighbouring
          // lanes (channels) trade halves: the even one has both channels of row i, the odd one of row i + 1
          const bool odd = lane & 1;
          uint8_t* to = smem + (col0 + (odd ? 1 : 0)) * L::kOutPitch + (ch & ~1) * 2;
#pragma unroll
          for (int i = 0; i < L::kCols; i += 2) {
            const float v0 = o[i] * l[i], v1 = o[i + 1] * l[i + 1];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 1);
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
        bool ok = mbar_wait_near(&sm.q_full, 0);
        auto scores = [&](int j) {
          const uint32_t d = tmem + L::kTmemS + (L::kAhead ? j & 1 : 0) * R;
          for (int u = 0; u < L::kUnits && ok; ++u) {
            const int c = j * L::kUnits + u;
            ok = mbar_wait_near(&sm.full[c % kRing], (c / kRing) & 1);
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
          ok = ok && mbar_wait_near(&sm.p_full[j & 1], (j >> 1) & 1);
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
        // the end of every MMA: the output may be read, and tensor memory given back
        tc_commit(&sm.drain);
        if (!mbar_wait_near(&sm.drain, 0) || !ok) flag_error(a.err, CKV_DEVERR_TIMEOUT);
      }
      __syncwarp();
    } else if (warp == kMmaWarp + 1 && n > 0 && gridDim.y == 1) {
      // The CTA that follows on this SM takes about the tile that lies a wave of CTAs (one per SM)
      // ahead; all SMs begin and end their tiles at much the same time, and its queries and first
      // keys would come from memory in that crowd.  Bring them to L2 now.
      if (__all_sync(0xFFFFFFFFu, mbar_wait_near(&sm.q_full, 0))) prefetch_tile<D>(a, blockIdx.x + kSMs, gridDim.x, R, page_shift);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kLoadRegs));
    if (n > 0) {
      // ------------------------------------------------------- load and decode
      const bool ok = load_units<D, true, L::kSlots, kRing, L::kGroups>(a, tile, threadIdx.x - kLoadWarp * 32, k_first, k_last, page_shift, 0,
                                                            smem, tmem + L::kTmemK, sm.full, sm.empty, sm.a_free, sm.bad);
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

template <int D, int R>
cudaError_t launch(const Fp4AttentionArgs& a, const Fp4Plan& p, bool use_pdl, cudaStream_t s) {
  cudaError_t e = set_max_smem_once<fp4_attention_kernel<D, R>>(smem_bytes<D, R>());
  if (e != cudaSuccess) return e;
  e = launch_ex(fp4_attention_kernel<D, R>, dim3(p.tiles, p.splits), dim3(Layout<D, R>::kThreads), smem_bytes<D, R>(), use_pdl, s, a,
                p.chunk, page_shift_of(a.page_size));
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_join<D, R, 1>(a, p, s);
}

template <int D>
cudaError_t launch_d(const Fp4AttentionArgs& a, const Fp4Plan& p, bool use_pdl, cudaStream_t s) {
  if constexpr (D == 512) {
    if (p.R == 64) return launch<D, 64>(a, p, use_pdl, s);
  }
  return p.R == 16 ? launch<D, 16>(a, p, use_pdl, s) : launch<D, 32>(a, p, use_pdl, s);
}

// Rows per tile, and into how many ranges of cache rows a tile is split: the count that a model of
// the time finds best.  A CTA costs a few microseconds around its tiles, a tile of 128 rows what D
// asks for; CTAs run in waves over the 152 SMs; split tiles write and read fp32 partials and need
// a second launch.  Lengths are known on the host by their bound only, so ranges are of equal size,
// and of 2^17 rows at most: the tensor cores add to the accumulator four products at a time and cut
// each sum off towards 0 (by 2^-23 of it at most), so over n rows of like weights an output loses up
// to n 2^-26 of its value.  Measured on channels that are constant: 2^17 rows 7.4e-4, 2^21 1.3e-2 (a
// bf16 output's half step is 3.9e-3).
// Against counts from 1 to 152 on 48 shapes the model's took at most 5% more than the best for all
// but three (13%).
// Rows per tile follow those of an average request: 128 are the M side of the rows form, with two
// CTAs per tile at D = 512, where 64 rows take the form here (256 requests x 64 heads x 922-1024
// rows 95 us, when the rows form took 156) and 80 the other (159 us, when this one took 174).  Below D = 512 the
// rows form's border is where this form's R = 64 would begin: 512 x 4 tokens x 32 heads at D = 128
// went from 149 to 82 us with it.
Fp4Plan plan_fp4(int64_t T, int32_t B, int32_t H, int32_t D, int64_t max_rows) {
  Fp4Plan p;
  const int64_t rows = (T + B - 1) / B * H;  // of an average request
  p.R = rows <= 16 ? 16 : rows <= 32 ? 32 : D == 512 && rows <= 64 ? 64 : 128;
  p.tiles = static_cast<int>((T * H + static_cast<int64_t>(B) * fp4_tile_pad(H, p.R)) / p.R);
  int64_t busy = (T * H + p.R - 1) / p.R;
  busy = busy < T && busy < B ? (T < B ? T : B) : busy;
  const int64_t most = (max_rows + kKeys - 1) / kKeys;
  const int halves = fp4_row_halves(D, p.R);
  busy *= halves;
  const double around = D == 512 ? 8.0 : 6.0;
  const double tile = D == 512 ? (halves == 2 ? 2.2 : p.R == 64 ? 3.5 : 2.5) : D == 256 ? (p.R == 128 ? 1.4 : 1.2) : p.R == 128 ? 1.0 : 0.6;
  double best = 0;
  const int64_t first = (max_rows + kFp4MaxRange - 1) / kFp4MaxRange;  // <= kFp4MaxSplits: the callers' bound of max_rows
  int64_t best_s = first;
  for (int64_t s = first; s <= most && s <= kFp4MaxSplits; ++s) {
    const int64_t waves = (busy * s + 151) / 152;
    double us = waves * (around + tile * static_cast<double>((most + s - 1) / s));
    if (s > 1) us += 2.0 + 0.02 * static_cast<double>(s) + 2.0 * static_cast<double>(busy / halves * s) * p.R * D * 4 / 4e6;
    if (s == first || us < best) {
      best = us;
      best_s = s;
    }
  }
  p.chunk = static_cast<int>((most + best_s - 1) / best_s * kKeys);
  p.splits = static_cast<int>((max_rows + p.chunk - 1) / p.chunk);
  return p;
}

}  // namespace

int64_t fp4_attention_workspace(int64_t T, int32_t B, int32_t H, int32_t D, int64_t max_rows) {
  const Fp4Plan p = plan_fp4(T, B, H, D, max_rows);
  const int64_t row = static_cast<int64_t>(sizeof(float)) * (D + 2 * fp4_row_halves(D, p.R));
  return p.splits == 1 ? 0 : static_cast<int64_t>(p.tiles) * p.splits * p.R * row;
}

cudaError_t launch_fp4_attention(const Fp4AttentionArgs& a, int D, bool use_pdl, cudaStream_t s) {
  const Fp4Plan p = plan_fp4(a.T, a.B, a.H, D, a.max_rows);
  if (p.R == 128) return launch_fp4_attention_rows(a, p, D, use_pdl, s);
  return D == 128 ? launch_d<128>(a, p, use_pdl, s) : D == 256 ? launch_d<256>(a, p, use_pdl, s) : launch_d<512>(a, p, use_pdl, s);
}

}  // namespace ckv
