// fp4_attention.cuh -- what the two forms of the 4-bit attention share: tiles of
// (token, head) rows, the decoding of cache rows into shared (and tensor) memory,
// and the joining of split ranges.
#pragma once

#include <cmath>
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_fp4.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"
#include "ckv_tcgen05.cuh"

namespace ckv {

constexpr int kSMs = 152;        // of a GB300
constexpr int kKeys = 128;       // cache rows per tile
constexpr int kRing = 4;         // units of 128 keys x 128 channels
constexpr int kUnitBytes = 32768;
// log2 of a row's largest weight when its reference is set, and before it moves (2^8 over that): as
// high as fp16 goes, so that weights keep their 11 bits down to 2^-21 of the largest one's and below
// that are off by 2^-32 of it at most.  With a reference at the largest score itself, 131,071 keys of
// weight 2^-25.1, 0.36% of their row together, were lost whole.
constexpr float kTop = 7.f, kJump = 15.f;
constexpr float kLn2 = 0.69314718055994531f;

// How a call is cut up (fp4_attention.cu).
struct Fp4Plan {
  int R;        // (token, head) rows per tile: 16, 32, 64 (keys on the M side) or 128 (rows on the M side)
  int tiles;    // bound of the number of tiles
  int splits;   // ranges of cache rows per tile
  int chunk;    // cache rows per range (multiple of kKeys)
};
// CTAs that share a tile and a range, each with as many of the channels: with rows on the M side
// the accumulator of 512 channels would fill tensor memory.
constexpr int fp4_row_halves(int D, int R) { return D == 512 && R == 128 ? 2 : 1; }
cudaError_t launch_fp4_attention_rows(const Fp4AttentionArgs& a, const Fp4Plan& p, int D, bool use_pdl, cudaStream_t s);

namespace {

// Which request and rows a tile has.
struct Tile {
  int32_t tok0, ntok;  // the request's ragged rows
  int32_t b;
  int32_t base, rows;  // first (token, head) row of the tile in the request, and how many (<= 0: none)
};

__device__ __forceinline__ int32_t start_of(const Fp4AttentionArgs& a, int32_t b) {
  return min(max(a.row_start[b], 0), static_cast<int32_t>(a.T));
}

// Tiles begin anew with every request: request b's first tile is (r_b + b (R - g)) / R with r_b
// the (token, head) rows before it and g = gcd(H, R), which all r_b and R are multiples of.  That
// leaves it ceil(rows / R) tiles at least, and none over where tokens are whole tiles.
__host__ __device__ inline int fp4_tile_pad(int H, int R) {
  const int g = H & -H;  // R is a power of two
  return g < R ? R - g : 0;
}

// By one converged warp.
__device__ __forceinline__ Tile find_tile(const Fp4AttentionArgs& a, int32_t tile, int R) {
  const int lane = threadIdx.x & 31;
  const int64_t pad = fp4_tile_pad(a.H, R);
  int lo = 0, n = a.B;  // the request is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && (start_of(a, i) * static_cast<int64_t>(a.H) + i * pad) / R <= tile;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  Tile t;
  t.b = lo;
  t.tok0 = start_of(a, lo);
  t.ntok = start_of(a, lo + 1) - t.tok0;
  t.base = (tile - static_cast<int32_t>((t.tok0 * static_cast<int64_t>(a.H) + lo * pad) / R)) * R;
  t.rows = t.base < 0 ? 0 : min(R, t.ntok * a.H - t.base);  // base < 0: row_start does not begin with 0
  return t;
}

// Decoding: the hardware converts two codes to two fp16, which the block's scale then
// multiplies.  A value has 2 + 4 significant bits and lies in 2^-10 .. 2688: exact.
// An e4m3's bits shifted up by 7 are an fp16 of 2^-8 of its value, for every byte (0x7F
// is 480): every byte of a cache decodes to a finite number.
__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 s) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), s);
    r[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// log2 of a page size that is a power of two, else -1
inline int page_shift_of(int32_t page_size) {
  if (page_size & (page_size - 1)) return -1;
  int s = 0;
  while ((1 << s) != page_size) ++s;
  return s;
}

// Four e4m3 bytes, each twice in a register.
__device__ __forceinline__ void decode_scales(uint32_t b, __half2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = b >> (8 * i);  // bytes i and i + 2 in the low byte of each half
    const uint32_t m = ((x & 0x007F007Fu) << 7) | ((x & 0x00800080u) << 8);
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&m), __float2half2_rn(256.f));
    s[i] = __low2half2(v);
    s[i + 2] = __high2half2(v);
  }
}

// Queries.  A row is scaled by a power of two that brings its largest magnitude (its
// bf16 bits) to [2^14, 2^15); by 1 when it is zero, infinite or NaN.  Returns the
// power's biased exponent.
__device__ __forceinline__ int query_exponent(uint32_t am) {
  const int e = static_cast<int>(am >> 7);
  return am == 0u || e == 255 ? 127 : min(127 + 14 + 127 - e, 253);
}

// Eight bf16 channels times `up`, as fp16.
__device__ __forceinline__ uint4 query8(uint4 raw, float up) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t v[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const __half2 p = __floats2half2_rn(bf16_lo(w[y]) * up, bf16_hi(w[y]) * up);
    v[y] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// The largest magnitude of a lane's channels: bf16 bits order like the values.
template <int n>
__device__ __forceinline__ uint32_t query_magnitude(const uint4 (&raw)[n]) {
  uint32_t two = 0;  // of the low halves and of the high ones
#pragma unroll
  for (int x = 0; x < n; ++x) {
    const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
    for (int y = 0; y < 4; ++y) two = __vmaxu2(two, w[y] & 0x7FFF7FFFu);
  }
  return max(two & 0xFFFFu, two >> 16);
}

// A warp's kRows queries, from row0 on, as fp16 in blocks of R rows x 128 bytes (128-byte swizzle)
// from `to` on, with the factors of their scores in c.  Rows with out < 0 are zeros.  A lane has
// eight channels of a row (16 at D = 512); a batch's loads are issued before the first is used.
template <int D, int R, int kRows>
__device__ __forceinline__ void load_queries(const Fp4AttentionArgs& a, int row0, const int32_t* out, const int64_t* from, float* c,
                                             uint8_t* to) {
  constexpr int kX = D == 512 ? 2 : 1;           // 16-byte pieces of a lane
  constexpr int kSpan = D / 8 / kX;              // lanes of a row
  constexpr int kLoads = kRows * kSpan / 32;
  constexpr int kBatch = kLoads < 8 ? kLoads : 8;  // rows in flight (registers)
  static_assert(kLoads >= 1 && kLoads % kBatch == 0, "");
  const int lane = threadIdx.x & 31, sub = lane / kSpan, ch = lane % kSpan * kX * 8;
#pragma unroll 1
  for (int i0 = 0; i0 < kLoads; i0 += kBatch) {
    uint4 raw[kBatch][kX];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = row0 + (i0 + i) * (32 / kSpan) + sub;
      const bool on = out[r] >= 0;
      const uint4* q = reinterpret_cast<const uint4*>(a.q + from[r] + ch);
#pragma unroll
      for (int x = 0; x < kX; ++x) raw[i][x] = on ? q[x] : make_uint4(0, 0, 0, 0);
    }
    uint32_t am[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) am[i] = query_magnitude(raw[i]);
    if constexpr (kSpan == 32) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) am[i] = __reduce_max_sync(0xFFFFFFFFu, am[i]);
    } else {
#pragma unroll
      for (int o = 1; o < kSpan; o <<= 1) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) am[i] = max(am[i], __shfl_xor_sync(0xFFFFFFFFu, am[i], o));
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = row0 + (i0 + i) * (32 / kSpan) + sub;
      const int se = query_exponent(am[i]);
      const float up = __uint_as_float(static_cast<uint32_t>(se) << 23);
      if (lane % kSpan == 0) c[r] = a.softmax_scale * kLog2e * a.g * __uint_as_float(static_cast<uint32_t>(254 - se) << 23);
      uint8_t* row = to + (ch / 64) * (R * 128) + r * 128;
#pragma unroll
      for (int x = 0; x < kX; ++x) *reinterpret_cast<uint4*>(row + ((((ch % 64) / 8 + x) ^ (r & 7)) * 16)) = query8(raw[i][x], up);
    }
  }
}

__device__ __forceinline__ void copies_wait(int left) {
  switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

// The same for more rows than registers hold (128 x 512 channels: 10 k clocks against 12.5 k in four
// batches; with one batch the registers win): all are copied to their places as bf16 and scaled
// there by the lanes that copied them.
template <int D, int R, int kRows>
__device__ __forceinline__ void copy_queries(const Fp4AttentionArgs& a, int row0, const int32_t* out, const int64_t* from, float* c,
                                             uint8_t* to) {
  constexpr int kX = D / 256, kGroups = 4, kDeep = kRows / kGroups;  // 16-byte pieces of a lane; rows that are scaled together
  static_assert(D % 256 == 0 && kRows % kGroups == 0, "");
  const int lane = threadIdx.x & 31;
  auto place = [&](int r, int x) {
    const int p = lane + x * 32;
    return to + (p / 8) * (R * 128) + r * 128 + ((p % 8) ^ (r & 7)) * 16;
  };
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int r = row0 + g * kDeep + i;
      const bool on = out[r] >= 0;
      const uint16_t* q = on ? a.q + from[r] : a.q;
#pragma unroll
      for (int x = 0; x < kX; ++x)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(place(r, x))), "l"(q + (lane + x * 32) * 8),
                     "r"(on ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    copies_wait(kGroups - 1 - g);
    uint4 raw[kDeep][kX];
    uint32_t am[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
#pragma unroll
      for (int x = 0; x < kX; ++x) raw[i][x] = *reinterpret_cast<const uint4*>(place(row0 + g * kDeep + i, x));
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) am[i] = __reduce_max_sync(0xFFFFFFFFu, query_magnitude(raw[i]));
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int r = row0 + g * kDeep + i;
      const int se = query_exponent(am[i]);
      const float up = __uint_as_float(static_cast<uint32_t>(se) << 23);
      if (lane == 0) c[r] = a.softmax_scale * kLog2e * a.g * __uint_as_float(static_cast<uint32_t>(254 - se) << 23);
#pragma unroll
      for (int x = 0; x < kX; ++x) *reinterpret_cast<uint4*>(place(r, x)) = query8(raw[i][x], up);
    }
  }
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

// The work of kGroups x 4 warps (tid from 0): cache rows k_first .. k_last - 1 of the tile's
// request, 128 at a time and 128 channels at a time, through the ring of units.
// A unit is two blocks of 128 keys x 64 channels of fp16, 128 bytes per key, with
// the 128-byte swizzle; with kCopy it also goes to tensor memory (a lane per
// key, 64 columns, slot c % kSlots from column tmem_k on).  The groups of 4 warps
// take units by turns: one's waits and fences lie under the others' decoding.
//   full[c % kRingN]   one arrival per warp of the group (4) when unit c is there
//   empty[c % kRingN]  completed when both products are done with it
//   a_free[c % kSlots] completed when the first product is done with it (only waited for where
//                      kSlots < kRingN, and there a tile is kRingN units: the other waits imply it)
//   bad[tile & 3]      a bit per key whose page is not there, written with the tile's last unit
// Units are given back in their order: a place may be used by several groups, and a
// group tells the phases of its barriers apart because the unit before last there is
// older than one that it has seen given back.  A tile's units come in channel order from unit `turn` on.  Rows that are not there are
// zeros.  False when a wait ran out.
template <int D, bool kCopy, int kSlots, int kRingN, int kGroups>
__device__ __forceinline__ bool load_units(const Fp4AttentionArgs& a, const Tile& tile, int tid, int k_first, int k_last, int page_shift,
                                           int turn, uint8_t* ring, uint32_t tmem_k, uint64_t* full, uint64_t* empty,
                                           uint64_t* a_free, uint32_t (*bad)[4]) {
  constexpr int kUnits = D / 128, kAhead = kGroups == 2 ? 4 : kGroups;
  constexpr int kDeep = kAhead / kGroups;  // units of a group in registers: loads run this far ahead
  static_assert(!kCopy || kSlots == kRingN || kUnits == kRingN, "waits");
  // a thread has one key's 128 channels of a unit, that of its lane of tensor memory; neighbouring
  // lanes have neighbouring keys, whose 16-byte chunks the swizzle spreads over all banks
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, key = quad * 32 + lane, group = tid >> 7;
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const int32_t* table = a.table + static_cast<int64_t>(tile.b) * a.table_stride;
  const int64_t page_bytes = fp4_page_bytes<D>(a.page_size);
  struct Unit {
    uint4 c[4];  // 128 codes
    uint2 s;     // 8 scales
    uint32_t gone;
  };
  Unit reg[kDeep];
  const uint8_t *codes = nullptr, *scales = nullptr;
  bool there = false;
  uint32_t gone = 0;  // the warp's keys without a page
  // where the key's row of tile j is
  auto locate = [&](int j) {
    const int k = k_first + j * kKeys + key;
    there = false;
    bool missing = false;
    if (k < k_last) {
      const int pg = page_shift >= 0 ? k >> page_shift : k / a.page_size;
      const int row = k - pg * a.page_size;
      const int32_t page = table[pg];
      if (page >= 0 && page < a.num_pages) {
        const uint8_t* p = a.cache + page * page_bytes;
        codes = p + static_cast<int64_t>(row) * (D / 2);
        scales = p + static_cast<int64_t>(a.page_size) * (D / 2) + static_cast<int64_t>(row) * (D / 16);
        there = true;
      } else {
        missing = true;
        flag_error(a.err, CKV_DEVERR_CACHE_LOC);
      }
    }
    gone = __ballot_sync(0xFFFFFFFFu, missing);
  };
  const int total = k_last > k_first ? (k_last - k_first + kKeys - 1) / kKeys * kUnits : 0;
  auto fetch = [&](Unit& x, int c) {
    if (c < total) {
      // the group's first unit of a tile
      if (kUnits <= kGroups || c % kUnits < kGroups) locate(c / kUnits);
      const int u = (c + turn) % kUnits;
      x.gone = gone;
      x.s = make_uint2(0, 0);
      if (there) x.s = *reinterpret_cast<const uint2*>(scales + u * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x.c[i] = make_uint4(0, 0, 0, 0);
        if (there) x.c[i] = *reinterpret_cast<const uint4*>(codes + u * 64 + i * 16);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kDeep; ++i) fetch(reg[i], group + i * kGroups);
  bool ok = true;
#pragma unroll 1
  for (int c0 = group; c0 < total && ok; c0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int c = c0 + i * kGroups, slot = kRingN == kAhead ? group + i * kGroups : c % kRingN;
      if (c < total && ok) {
        // the ring's last unit in this place has served both products
        if (c >= kRingN) ok = mbar_wait_near(&empty[slot], ((c / kRingN) - 1) & 1);
        if (kCopy && kSlots < kRingN && slot >= kSlots) ok = ok && mbar_wait_near(&a_free[c % kSlots], ((c / kSlots) - 1) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) {
          if (kCopy) tc_fence_after();
#pragma unroll
          for (int p = 0; p < 2; ++p) {  // blocks of 64 channels
            uint8_t* unit = ring + slot * kUnitBytes + p * 16384 + key * 128;
            const uint32_t a_tile = tmem_k + lanes + (c % kSlots) * 64 + p * 32;
            __half2 sc[4];
            decode_scales(p ? reg[i].s.y : reg[i].s.x, sc);
#pragma unroll
            for (int b = 0; b < 4; ++b) {  // blocks of 16 channels
              const uint4 x = reg[i].c[p * 2 + b / 2];
              const uint4 lo = decode8(b & 1 ? x.z : x.x, sc[b]), hi = decode8(b & 1 ? x.w : x.y, sc[b]);
              *reinterpret_cast<uint4*>(unit + (((2 * b) ^ (key & 7)) * 16)) = lo;
              *reinterpret_cast<uint4*>(unit + (((2 * b + 1) ^ (key & 7)) * 16)) = hi;
              if (kCopy) tmem_st8(a_tile + b * 8, lo, hi);
            }
          }
          if (c % kUnits == kUnits - 1 && lane == 0) bad[(c / kUnits) & 3][quad] = reg[i].gone;
          if (kCopy) {
            tc_wait_st();
            tc_fence_before();
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[slot]);
          fetch(reg[i], c + kAhead);
        }
      }
    }
  }
  return ok;
}

// Queries and first cache rows of a tile, to L2.  By one converged warp.
template <int D>
__device__ __forceinline__ void prefetch_tile(const Fp4AttentionArgs& a, uint32_t index, uint32_t tiles, int R, int page_shift) {
  const int lane = threadIdx.x & 31;
  if (index >= tiles) return;
  const Tile tile = find_tile(a, index, R);
  if (tile.rows <= 0) return;
  auto line = [](const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); };
  constexpr int kLines = D * 2 / 128;  // of a query row
  for (int i = lane; i < tile.rows * kLines; i += 32) {
    const int r = i / kLines, t = tile.tok0 + (tile.base + r) / a.H, h = tile.base + r - (t - tile.tok0) * a.H;
    line(a.q + t * a.q_st + h * a.q_sh + i % kLines * 64);
  }
  const int seen = min(min(a.ctx_rows[tile.tok0 + tile.base / a.H], a.max_rows), kKeys);
  const int32_t* table = a.table + static_cast<int64_t>(tile.b) * a.table_stride;
  const int64_t page_bytes = fp4_page_bytes<D>(a.page_size);
  for (int k = lane; k < seen; k += 32) {
    const int pg = page_shift >= 0 ? k >> page_shift : k / a.page_size;
    const int32_t page = table[pg];
    if (page < 0 || page >= a.num_pages) continue;
    const uint8_t* p = a.cache + page * page_bytes;
    const int64_t row = k - pg * a.page_size;
#pragma unroll
    for (int x = 0; x < D / 2; x += 64) line(p + row * (D / 2) + x);
    line(p + static_cast<int64_t>(a.page_size) * (D / 2) + row * (D / 16));
  }
}

// Joins the ranges of a tile, in their order: one warp per row and 128 channels, since few rows
// over many ranges would wait for one load after the other.  One request of 64 heads over 8192 rows
// at D = 512 takes 38.9 us with a warp per row, 25.0 us so, and 18.5 us with 16 loads in flight
// instead of what 32 registers hold.  With few ranges many warps hide the latency instead (kFew:
// 600 tokens x 16 heads over 2048 rows in two ranges at D = 128, 28.1 -> 23.0 us).  With kHalves
// == 2 two CTAs shared a range, each with half of the channels and with references and sums of
// its own.
constexpr int kFewSplits = 4;
template <int D, int R, int kHalves, bool kFew>
__global__ void __launch_bounds__(128, kFew ? 12 : 4) fp4_join_kernel(const __grid_constant__ Fp4AttentionArgs a, int chunk, int splits) {
  constexpr int kParts = D / 128, kDeep = kFew ? kFewSplits : 16;  // loads in flight (the second bound leaves them registers)
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const Tile t = find_tile(a, blockIdx.x, R);
  if (t.rows <= 0) return;
  int ctx_max = 0;
  for (int i = lane; i < R; i += 32)
    if (i < t.rows) ctx_max = max(ctx_max, min(a.ctx_rows[t.tok0 + (t.base + i) / a.H], a.max_rows));
  ctx_max = __reduce_max_sync(0xFFFFFFFFu, ctx_max);
  const int used = (ctx_max + chunk - 1) / chunk;
  const int work = blockIdx.y * 4 + (threadIdx.x >> 5), r = work / kParts, part = work % kParts;
  if (used <= 1 || r >= t.rows) return;
  if (a.ctx_rows[t.tok0 + (t.base + r) / a.H] < 0) return;
  const float* ws = static_cast<const float*>(a.workspace);
  const int64_t slot0 = static_cast<int64_t>(blockIdx.x) * splits;
  const int half = part / (kParts / kHalves);
  const float* ml = ws + static_cast<int64_t>(gridDim.x) * splits * R * D + (slot0 * kHalves + half) * R * 2 + r;
  const int64_t flat = static_cast<int64_t>(t.tok0) * a.H + t.base + r;
  // a lane has the references and sums of ranges lane, lane + 32, ...
  constexpr int kOwn = kFew ? 1 : kFp4MaxSplits / 32;
  float ref[kOwn], l[kOwn], m = kNegBig;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int s = lane + i * 32;
    ref[i] = s < used ? ml[s * kHalves * 2 * R] : kNegBig;
    l[i] = s < used ? ml[s * kHalves * 2 * R + R] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i) m = fmaxf(m, ref[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float sink = a.sink ? a.sink[flat % a.H] * kLog2e : -INFINITY;
  if (a.sink) m = fmaxf(m, sink);
  float w[kOwn], all = 0.f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    w[i] = fast_exp2(ref[i] - m);
    all += l[i] == 0.f ? 0.f : l[i] * w[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  if (a.sink) all += sink == m ? 1.f : fast_exp2(sink - m);
  const float4* o = reinterpret_cast<const float4*>(ws + (slot0 * R + r) * D + part * 128) + lane;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    for (int s0 = j * 32; s0 < min(used, j * 32 + 32); s0 += kDeep) {
      float4 v[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i)
        v[i] = s0 + i < used ? o[static_cast<int64_t>(s0 + i) * (R * D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const float x = __shfl_sync(0xFFFFFFFFu, w[j], (s0 + i) % 32);
        acc[0] = fmaf(v[i].x, x, acc[0]);
        acc[1] = fmaf(v[i].y, x, acc[1]);
        acc[2] = fmaf(v[i].z, x, acc[2]);
        acc[3] = fmaf(v[i].w, x, acc[3]);
      }
    }
  }
  const float inv = all == 0.f ? 0.f : a.g / all;
  *reinterpret_cast<uint2*>(a.out + flat * D + part * 128 + lane * 4) =
      make_uint2(pack_bf16x2_rn(acc[0] * inv, acc[1] * inv), pack_bf16x2_rn(acc[2] * inv, acc[3] * inv));
  if (part == 0 && lane == 0 && a.lse) a.lse[flat] = all == 0.f ? -INFINITY : (m + log2f(all)) * kLn2;
}

template <int D, int R, int kHalves>
cudaError_t launch_join(const Fp4AttentionArgs& a, const Fp4Plan& p, cudaStream_t s) {
  const dim3 grid(p.tiles, R * (D / 128) / 4);
  return p.splits <= kFewSplits ? launch_ex(fp4_join_kernel<D, R, kHalves, true>, grid, dim3(128), 0, true, s, a, p.chunk, p.splits)
                                : launch_ex(fp4_join_kernel<D, R, kHalves, false>, grid, dim3(128), 0, true, s, a, p.chunk, p.splits);
}

}  // namespace
}  // namespace ckv
