// fp4_attention_rows.cu -- attention over the 4-bit paged cache with the (token,
// head) rows on the M side of both products, for requests with more than 32 rows
// (64 at D = 512; fp4_attention.cu holds the other form and the formulas):
//   S [128 rows x 128 keys]   = Q [128 x D] K^T
//   O [128 rows x D]         += P [128 x 128 keys] K
// A thread owns 64 keys of a row of S (two warps share 32 rows): maximum and sum
// need one other thread at most, and the weights go back to tensor memory as A of
// the second product.  Per 128 keys the 8 softmax warps evaluate 128 x 128
// exponentials, half as long as the products take (1,024 clocks at D = 128).
//
// As in the other form a row's weights are taken against a reference that moves
// only when a weight exceeds 2^15; here that is the affair of two warps.
//
// At D = 512 the accumulator would fill tensor memory, so two CTAs share a tile:
// both form the scores and the softmax, each multiplies with its half of the
// channels.  A key is decoded twice per 128 rows, as often as in the other form
// (once per 64), but a product step has twice the rows.  Queries take 128 KB of
// shared memory there and the ring has three places; only the units of the CTA's
// own half stay for the second product, so they come last in a tile.
//
// What bounds it: neither the tensor cores (30% of the active cycles at D = 128) nor
// the exponentials (15%).  With D = 128 128 keys take 0.9-1.2 us where their products
// take 0.5, and a CTA 7 us besides them, of which one CTA per SM hides nothing (456
// requests x 4 tokens x 32 heads, three CTAs on each SM: 27.7 us over 128 rows, 52.0
// over 1024, 73.2 over 2048); requests of different lengths leave SMs idle at the
// launch's end.  With D = 512 the chain of a tile (5.5 k clocks), as the ring has no place for the next tile's units before the second
// product gives them back: softmax 1.6 k, second product 0.8 k, decoding of three
// units by a group each and scores 3 k.  Around its tiles a CTA of D = 512 spends 18 k
// clocks: queries 10 k, output 4 k, first tile.
// Measured (GB300): 512 requests x 4 tokens x 32 heads at D = 128, 0-2048 rows 61 us
// (560 TFLOP/s); D = 512, a prompt of 8750 tokens x 64 heads over 200-1024 rows
// 1.36-1.39 ms (510 TFLOP/s; with two decoding groups 1.49 ms, when three took 1.39,
// with queries through registers 1.58 ms, when copies took 1.49; the other form
// 1.70 ms).  Slower: D = 128 with two CTAs of 9 warps per SM (109 us, when one took
// 82), 16 softmax warps (63.7 us, when 8 took 61.4), and four lanes per key in the
// decoding's loads (65.3 us, when one took 64.2; at D = 512 1.37 ms, when one took 1.39).
#include "fp4_attention.cuh"

namespace ckv {
namespace {

// Warpgroups 0 and 1: softmax; 2: its first warp issues the MMAs; 3 and 4: load and decode.
constexpr int kRowMmaWarp = 8, kRowLoadWarp = 12;
// Registers per thread at launch: 640 x 96 or (D = 512) 768 x 80, 61,440 both; then 256 x 112 +
// 128 x 64 and 256 x 96 or 384 x 64, the same.
constexpr int kRowSoftRegs = 112, kRowMmaRegs = 64;

template <int D>
struct RowLayout {
  static constexpr int kUnits = D / 128;
  static constexpr int kHalves = fp4_row_halves(D, 128);
  static constexpr int kDV = D / kHalves;            // channels of the output that a CTA has
  static constexpr int kKept = kDV / 128;            // a tile's last units, of which they are
  static constexpr int kRingN = D == 512 ? 3 : 4;
  // groups of four decoding warps; at D = 512 one for each place of the ring: what a tile waits for is
  // the decoding of the units whose places its predecessor's second product gives back
  static constexpr int kGroups = D == 512 ? 3 : 2;
  static constexpr int kThreads = (kRowLoadWarp + kGroups * 4) * 32;
  static constexpr int kLoadRegs = D == 512 ? 64 : 96;
  static_assert(256 * kRowSoftRegs + 128 * kRowMmaRegs + kGroups * 128 * kLoadRegs <= kThreads * (D == 512 ? 80 : 96),
                "registers of the launch");
  static constexpr int kSBufs = D == 128 ? 2 : 1;
  static constexpr int kQ = kRingN * kUnitBytes;     // Q: D/64 blocks of 128 rows x 128 bytes
  static constexpr int kSmall = kQ + (D / 64) * 128 * 128;
  static constexpr int kTmemO = 0, kTmemS = kDV, kTmemP = kDV + kSBufs * 128;  // P: two buffers of 64 columns
  static_assert(kTmemP + 2 * 64 <= 512, "tensor memory");
  static constexpr int kOutPitch = kDV * 2 + 16;     // output rows on their way out, over the ring and Q
  static constexpr int kPartPitch = kDV * 4 + 16;    // the same of fp32 partials
  static_assert(128 * kPartPitch <= kSmall, "output staging");
};

struct RowSmall {
  uint64_t full[4], empty[4], s_full[2], s_read, p_full[2], q_full, o_done, drain;
  uint32_t tmem;
  int32_t abort;
  Tile tile;
  int32_t ctx_max;
  alignas(16) uint32_t bad[4][4];
  float c[128];      // score factors
  int32_t out[128];  // flat (token, head) index, -1: none
  union {
    int64_t q[128];      // where the rows' queries begin, elements (until they are loaded)
    float part[2][128];  // what the two warps of a row tell each other
  };
};

template <int D>
constexpr int row_smem_bytes() {
  return RowLayout<D>::kSmall + static_cast<int>(sizeof(RowSmall));
}
static_assert(row_smem_bytes<512>() <= 227 * 1024, "shared memory");

// The two warps of 32 rows (quad q) meet; true when p holds for one of the 64 threads.
__device__ __forceinline__ void pair_barrier(int quad) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + quad) : "memory"); }
__device__ __forceinline__ bool pair_any(int quad, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(1 + quad)
      : "memory");
  return r != 0;
}

// 16 packed columns of the warp's lanes.
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(RowLayout<D>::kThreads, 1)
    fp4_attention_rows_kernel(const __grid_constant__ Fp4AttentionArgs a, int chunk, int page_shift) {
  using L = RowLayout<D>;
  // no static shared memory: the dynamic one begins on the swizzle's 1024 bytes (checked below)
  extern __shared__ __align__(1024) uint8_t smem[];
  RowSmall& sm = *reinterpret_cast<RowSmall*>(smem + L::kSmall);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the CTA's half of the channels, and the unit that a tile begins with: the units of that half come last
  const int half_v = L::kHalves == 2 ? blockIdx.x & 1 : 0, turn = L::kHalves == 2 && half_v == 0 ? 2 : 0;
  const uint32_t index = blockIdx.x / L::kHalves, tiles = gridDim.x / L::kHalves;
  if (smem_u32(smem) & 1023u) {
    pdl_wait();  // whoever follows in the stream counts on what came before having ended
    if (threadIdx.x == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
    return;
  }

  if (warp == kRowMmaWarp && lane == 0) {
    for (int i = 0; i < L::kRingN; ++i) {
      mbar_init(&sm.full[i], 4);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 8);
    }
    mbar_init(&sm.s_read, 8);
    mbar_init(&sm.q_full, 8);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 0) {
    const Tile t = find_tile(a, index, 128);
    if (lane == 0) {
      sm.tile = t;
      sm.ctx_max = -1;
    }
  }
  __syncthreads();
  const Tile tile = sm.tile;
  if (tile.rows <= 0) return;  // more tiles than rows need
  if (warp == kRowMmaWarp) tmem_alloc<512>(&sm.tmem);
  int32_t my_ctx = -1, my_flat = -1;  // of softmax thread t: row t % 128
  if (threadIdx.x < 256) {
    const int r = threadIdx.x & 127;
    if (r < tile.rows) {
      const int t = tile.tok0 + (tile.base + r) / a.H;
      my_ctx = a.ctx_rows[t];
      if (my_ctx > a.max_rows) {
        flag_error(a.err, CKV_DEVERR_SEQ_LEN);
        my_ctx = a.max_rows;
      }
      if (my_ctx >= 0) {
        my_flat = tile.tok0 * a.H + tile.base + r;
        sm.q[r] = t * a.q_st + (my_flat - t * a.H) * a.q_sh;
      }
    }
    sm.out[r] = my_flat;
    const int top = __reduce_max_sync(0xFFFFFFFFu, my_ctx);
    if (lane == 0) atomicMax(&sm.ctx_max, top);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int ctx_max = sm.ctx_max;
  const int k_first = blockIdx.y * chunk;
  const int k_last = min(ctx_max, k_first + chunk);
  const bool split = ctx_max > chunk;  // several CTAs share the tile
  const int n = k_last > k_first ? (k_last - k_first + kKeys - 1) / kKeys : 0;
  // nothing to add: only the first range answers for rows that see nothing
  const bool idle = n == 0 && (blockIdx.y > 0 || ctx_max < 0);

  if (warp < kRowMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowSoftRegs));
    if (!idle) {
      const int quad = warp & 3, half = warp >> 2, row = threadIdx.x & 127;
      // ----------------------------------------------------------- queries
      if (n > 0) {
        if constexpr (D == 512)
          copy_queries<D, 128, 16>(a, warp * 16, sm.out, sm.q, sm.c, smem + L::kQ);
        else
          load_queries<D, 128, 16>(a, warp * 16, sm.out, sm.q, sm.c, smem + L::kQ);
      }
      fence_proxy_async_smem();
      asm volatile("barrier.cta.sync 5, 256;" ::: "memory");  // every row's factor is there
      if (lane == 0) mbar_arrive(&sm.q_full);

      // ----------------------------------------------------------- softmax
      const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
      const float c = n > 0 ? sm.c[row] : 0.f;
      float ref = kNegBig, l = 0.f;  // the reference is the same in both threads of a row, the sum each one's own
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int buf = L::kSBufs == 2 ? j & 1 : 0;
        const int last = (j + 1) * L::kUnits - 1;
        // the scores, then (there by now) the decoding warps' note on missing keys
        ok = mbar_wait_near(&sm.s_full[j & 1], (j >> 1) & 1) && mbar_wait_near(&sm.full[last % L::kRingN], (last / L::kRingN) & 1);
        if (!ok) atomicExch(&sm.abort, 1);
        __syncwarp();
        tc_fence_after();
        float z[2][32];
#pragma unroll
        for (int i = 0; i < 2; ++i) tmem_ld<32>(tmem + lanes + L::kTmemS + buf * 128 + half * 64 + i * 32, z[i]);
        if (L::kSBufs == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.s_read);
        }
        // log2 units over the row's reference; a row that has seen no key yet has none
        const bool unset = ref == kNegBig;
        const float shift = unset ? 0.f : ref;
#pragma unroll
        for (int i = 0; i < 64; ++i) z[i / 32][i % 32] = fmaf(z[i / 32][i % 32], c, -shift);
        const int left = my_ctx - (k_first + j * kKeys + half * 64);  // keys of the thread's that the row sees
        const uint2 gone = *reinterpret_cast<const uint2*>(&sm.bad[j & 3][half * 2]);
        if (__any_sync(0xFFFFFFFFu, left < 64)) {
#pragma unroll
          for (int i = 0; i < 64; ++i) z[i / 32][i % 32] = i < left ? z[i / 32][i % 32] : -INFINITY;
        }
        if (gone.x | gone.y) {
#pragma unroll
          for (int i = 0; i < 64; ++i) z[i / 32][i % 32] = ((i < 32 ? gone.x : gone.y) >> (i % 32)) & 1 ? -INFINITY : z[i / 32][i % 32];
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 64; ++i) top[i % 4] = fmaxf(top[i % 4], z[i / 32][i % 32]);
        float over = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        ok = ok && *reinterpret_cast<volatile int32_t*>(&sm.abort) == 0;
        if (pair_any(quad, over > kJump || (unset && over > -INFINITY) || !ok)) {
          ok = !pair_any(quad, !ok);
          if (!ok) break;
          // the reference goes to kTop below the largest score so far
          sm.part[half][row] = over;
          pair_barrier(quad);
          over = fmaxf(over, sm.part[half ^ 1][row]);
          pair_barrier(quad);  // read, before it is written again
          const float d = unset ? over - kTop : fmaxf(over - kTop, 0.f);
          const bool move = d > -INFINITY;
          const float by = move ? d : 0.f;
          const float keep = unset ? 0.f : fast_exp2(-by);
          l *= keep;
          ref = move ? shift + by : ref;
#pragma unroll
          for (int i = 0; i < 64; ++i) z[i / 32][i % 32] -= by;
          if (j > 0) {
            ok = mbar_wait_near(&sm.o_done, (j - 1) & 1);
            if (!ok) atomicExch(&sm.abort, 1);
            __syncwarp();
            tc_fence_after();
            const float k = unset ? 1.f : keep;  // an unset row's output is 0
#pragma unroll 1
            for (int i = half * (L::kDV / 2); i < (half + 1) * (L::kDV / 2); i += 16) {
              float o[16];
              tmem_ld<16>(tmem + lanes + L::kTmemO + i, o);
              uint32_t v[16];
#pragma unroll
              for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(o[x] * k);
              tmem_st16(tmem + lanes + L::kTmemO + i, v);
            }
          }
        }
        // weights, rounded to fp16, as A of the second product
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t v[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const float p0 = fast_exp2(z[i][x]), p1 = fast_exp2(z[i][x + 1]);
            part[x % 4] += p0;
            part[x % 4 + 1] += p1;
            const __half2 h = __floats2half2_rn(p0, p1);
            v[x / 2] = *reinterpret_cast<const uint32_t*>(&h);
          }
          tmem_st16(tmem + lanes + L::kTmemP + (j & 1) * 64 + half * 32 + i * 16, v);
        }
        l += (part[0] + part[1]) + (part[2] + part[3]);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[j & 1]);
      }
      // ------------------------------------------------------------ output
      pair_barrier(quad);
      sm.part[half][row] = l;
      pair_barrier(quad);
      l += sm.part[half ^ 1][row];
      float* ws = static_cast<float*>(a.workspace);
      const int64_t slot = static_cast<int64_t>(index) * gridDim.y + blockIdx.y;
      float scale = 1.f;
      if (split) {
        if (half == 0) {
          float* ml = ws + static_cast<int64_t>(tiles) * gridDim.y * 128 * D + (slot * L::kHalves + half_v) * 128 * 2;
          ml[row] = ref;
          ml[128 + row] = l;
        }
      } else {
        float m = ref, all = l, keep = 1.f;
        if (a.sink && my_flat >= 0) {
          const float s = a.sink[my_flat % a.H] * kLog2e;
          const float high = fmaxf(m, s);
          keep = fast_exp2(m - high);  // 0 where no key was seen
          all = (l == 0.f ? 0.f : l * keep) + (s == high ? 1.f : fast_exp2(s - high));
          m = high;
        }
        scale = all == 0.f ? 0.f : keep * a.g / all;
        // nothing at all: no sink, or one that is -infinity in log2 units
        if (a.lse && my_flat >= 0 && half == 0 && half_v == 0)
          a.lse[my_flat] = all == 0.f ? a.sink ? a.sink[my_flat % a.H] : -INFINITY : (m + log2f(all)) * kLn2;
      }
      if (n > 0 && ok) {
        // not o_done: a warp that has not waited for tile n - 2 could take its phase for the last one's
        ok = mbar_wait_near(&sm.drain, 0);
        __syncwarp();
        tc_fence_after();
      }
      if (!ok && lane == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
#pragma unroll 1
      for (int i = half * (L::kDV / 2); i < (half + 1) * (L::kDV / 2); i += 32) {
        float o[32];
        if (n > 0) {
          tmem_ld<32>(tmem + lanes + L::kTmemO + i, o);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.f;
        }
        if (split) {
          uint8_t* to = smem + row * L::kPartPitch + i * 4;
#pragma unroll
          for (int x = 0; x < 32; x += 4) *reinterpret_cast<float4*>(to + x * 4) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
        } else {
          uint8_t* to = smem + row * L::kOutPitch + i * 2;
#pragma unroll
          for (int x = 0; x < 32; x += 8)
            *reinterpret_cast<uint4*>(to + x * 2) =
                make_uint4(pack_bf16x2_rn(o[x] * scale, o[x + 1] * scale), pack_bf16x2_rn(o[x + 2] * scale, o[x + 3] * scale),
                           pack_bf16x2_rn(o[x + 4] * scale, o[x + 5] * scale), pack_bf16x2_rn(o[x + 6] * scale, o[x + 7] * scale));
        }
      }
      // a warp takes out what it brought, its rows' half, in 16-byte pieces
      __syncwarp();
      const int piece = split ? L::kDV / 8 : L::kDV / 16, pitch = split ? L::kPartPitch : L::kOutPitch;
      uint8_t* to = split ? reinterpret_cast<uint8_t*>(ws + slot * 128 * D) : reinterpret_cast<uint8_t*>(a.out);
      const int whole = 2 * piece * L::kHalves, first = 2 * piece * half_v;  // of the row, in pieces
#pragma unroll 4
      for (int i = lane; i < 32 * piece; i += 32) {
        const int r = quad * 32 + i / piece, x = half * piece + i % piece;
        const int32_t flat = sm.out[r];
        if (flat >= 0)
          *reinterpret_cast<uint4*>(to + (static_cast<int64_t>(split ? r : flat) * whole + first + x) * 16) =
              *reinterpret_cast<const uint4*>(smem + r * pitch + x * 16);
      }
      tc_fence_before();
    }
  } else if (warp < kRowLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRowMmaRegs));
    if (warp == kRowMmaWarp && n > 0) {
      // ------------------------------------------------------- tensor cores
      if (elect_one()) {
        constexpr uint32_t kIdescS = idesc_f16(128, false, false), kIdescO = idesc_f16(128, false, true);
        const uint32_t base = smem_u32(smem);
        bool ok = mbar_wait_near(&sm.q_full, 0);
        // Scores run ahead of the last tile's second product as far as the ring goes: all of them, or
        // (kept units fill all places but one) the first unit's.  Units are given back in their order:
        // a place's users are of both groups, whose waits tell its phases apart by that.
        constexpr int kEarly = L::kRingN < 2 * L::kKept ? 1 : L::kUnits;
        // units i0 .. i1 - 1 of tile j's scores; a unit that the second product does not need is free after them
        auto scores = [&](int j, int i0, int i1) {
          const uint32_t d = tmem + L::kTmemS + (L::kSBufs == 2 ? j & 1 : 0) * 128;
          for (int i = i0; i < i1 && ok; ++i) {
            const int c = j * L::kUnits + i, u = (i + turn) % L::kUnits;
            ok = mbar_wait_near(&sm.full[c % L::kRingN], (c / L::kRingN) & 1);
            tc_fence_after();
            if (!ok) break;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
              const uint64_t da = smem_desc_sw128(base + L::kQ + (u * 2 + s / 4) * (128 * 128) + (s % 4) * 32, 16, 1024);
              const uint64_t db = smem_desc_sw128(base + (c % L::kRingN) * kUnitBytes + (s / 4) * 16384 + (s % 4) * 32, 16, 1024);
              mma_f16_ss(d, da, db, kIdescS, i > 0 || s > 0);
            }
            if (i < L::kUnits - L::kKept && (kEarly == L::kUnits || i > 0)) tc_commit(&sm.empty[c % L::kRingN]);
          }
          if (i1 == L::kUnits) tc_commit(&sm.s_full[j & 1]);
        };
        if (ok) {
          scores(0, 0, kEarly);
          if (kEarly < L::kUnits) {
            tc_commit(&sm.empty[0]);
            scores(0, kEarly, L::kUnits);
          }
        }
        for (int j = 0; j < n && ok; ++j) {
          if (j + 1 < n) {
            if (L::kSBufs == 1) ok = mbar_wait_near(&sm.s_read, j & 1);  // with two buffers the weights of tile j - 1 said so
            tc_fence_after();
            if (ok) scores(j + 1, 0, kEarly);
          }
          ok = ok && mbar_wait_near(&sm.p_full[j & 1], (j >> 1) & 1);
          tc_fence_after();
          if (!ok) break;
          for (int i = L::kUnits - L::kKept; i < L::kUnits; ++i) {
            const int c = j * L::kUnits + i;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
              const uint64_t db = smem_desc_sw128(base + (c % L::kRingN) * kUnitBytes + s * 2048, 16384, 1024);
              mma_f16_ts(tmem + L::kTmemO + (i - (L::kUnits - L::kKept)) * 128, tmem + L::kTmemP + (j & 1) * 64 + s * 8, db, kIdescO,
                         j > 0 || s > 0);
            }
            tc_commit(&sm.empty[c % L::kRingN]);
          }
          tc_commit(&sm.o_done);
          if (kEarly < L::kUnits && j + 1 < n) {
            tc_commit(&sm.empty[(j + 1) * L::kUnits % L::kRingN]);
            scores(j + 1, kEarly, L::kUnits);
          }
        }
        if (!ok) atomicExch(&sm.abort, 1);
        // the end of every MMA: the output may be read, and tensor memory given back
        tc_commit(&sm.drain);
        if (!mbar_wait_near(&sm.drain, 0) || !ok) flag_error(a.err, CKV_DEVERR_TIMEOUT);
      }
      __syncwarp();
    } else if (warp == kRowMmaWarp + 1 && n > 0 && half_v == 0) {
      // as in the other form: what the CTA that follows on this SM begins with, to L2
      if (__all_sync(0xFFFFFFFFu, mbar_wait_near(&sm.q_full, 0)))
        prefetch_tile<D>(a, index + kSMs / L::kHalves, tiles, 128, page_shift);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kLoadRegs));
    if (n > 0) {
      const bool ok = load_units<D, false, 1, L::kRingN, L::kGroups>(a, tile, threadIdx.x - kRowLoadWarp * 32, k_first, k_last, page_shift,
                                                         turn, smem, 0u, sm.full, sm.empty, nullptr, sm.bad);
      if (!ok) {
        atomicExch(&sm.abort, 1);
        if (lane == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
      }
    }
  }
  pdl_trigger();
  __syncthreads();
  if (warp == kRowMmaWarp) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

template <int D>
cudaError_t launch(const Fp4AttentionArgs& a, const Fp4Plan& p, bool use_pdl, cudaStream_t s) {
  cudaError_t e = set_max_smem_once<fp4_attention_rows_kernel<D>>(row_smem_bytes<D>());
  if (e != cudaSuccess) return e;
  e = launch_ex(fp4_attention_rows_kernel<D>, dim3(p.tiles * RowLayout<D>::kHalves, p.splits), dim3(RowLayout<D>::kThreads), row_smem_bytes<D>(),
                use_pdl, s, a, p.chunk, page_shift_of(a.page_size));
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_join<D, 128, RowLayout<D>::kHalves>(a, p, s);
}

}  // namespace

cudaError_t launch_fp4_attention_rows(const Fp4AttentionArgs& a, const Fp4Plan& p, int D, bool use_pdl, cudaStream_t s) {
  return D == 128 ? launch<128>(a, p, use_pdl, s) : D == 256 ? launch<256>(a, p, use_pdl, s) : launch<512>(a, p, use_pdl, s);
}

}  // namespace ckv
