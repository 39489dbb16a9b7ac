// fp4_rows.cu -- rows to and from the 4-bit paged cache (no counterpart in the
// sources; the format is in ckv_fp4.cuh).
//
// store: per block of 16 channels  scale = e4m3(min(absmax / (6 g), 448)),
//        code = e2m1(x / (scale g)), nearest even, saturating.
// load:  value = code * scale * g.
//
// g is a power of two, so 6 g and scale * g are exact, and a correctly rounded
// quotient lies on the same side of every rounding border as the exact one (a
// border times scale * g is a float, and the float next to it is off by more
// than half a step of the quotient): the codes are those of exact arithmetic.
// The quotients of a block share their divisor: its correctly rounded reciprocal,
// and per quotient one Newton step on the remainder (Markstein's method: the result
// is the correctly rounded quotient).
//
// Bound by HBM (2-4 bytes in and 9/16 out per channel, or the reverse) when there
// are many rows.  Measured (GB300): 65,536 rows of 128 channels, bf16, 6.7 us a call
// (3.2 TB/s): launch, two round trips and about 3 us of instructions; two blocks
// per thread with their loads in flight together gained 1%.  One
// thread per block of 16 channels: D/16 neighbouring threads write a row's D/2
// code bytes (8 each) and D/16 scale bytes.
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_fp4.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kRowThreads = 256;

template <int D, bool kF32>
__global__ void __launch_bounds__(kRowThreads) fp4_store_kernel(const __grid_constant__ Fp4RowsArgs a) {
  constexpr int kBlocks = D / kFp4Block;
  pdl_wait();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t r = id / kBlocks;
  const int blk = static_cast<int>(id % kBlocks);
  if (r >= a.n) return;
  const int64_t loc = a.loc[r];
  if (loc < 0) return;
  int64_t page;
  int32_t row;
  split_location(loc, a.page_size, a.page_shift, page, row);
  if (page >= a.num_pages) {
    if (blk == 0) flag_error(a.err, CKV_DEVERR_CACHE_LOC);
    return;
  }
  float x[kFp4Block];
  if constexpr (kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.rows) + r * a.stride + blk * kFp4Block);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = p[i];
      x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.rows) + r * a.stride + blk * kFp4Block);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 w = p[i];
      x[8 * i] = bf16_lo(w.x), x[8 * i + 1] = bf16_hi(w.x), x[8 * i + 2] = bf16_lo(w.y), x[8 * i + 3] = bf16_hi(w.y);
      x[8 * i + 4] = bf16_lo(w.z), x[8 * i + 5] = bf16_hi(w.z), x[8 * i + 6] = bf16_lo(w.w), x[8 * i + 7] = bf16_hi(w.w);
    }
  }
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < kFp4Block; ++i) am = fmaxf(am, fabsf(x[i]));
  const uint32_t sc = __nv_cvt_float_to_fp8(fminf(__fdiv_rn(am, 6.f * a.g), 448.f), __NV_SATFINITE, __NV_E4M3);
  uint32_t lo = 0, hi = 0;
  if (sc != 0) {
    const float f = e4m3_to_float(sc) * a.g, inv = __frcp_rn(f);
    // a saturated scale leaves quotients of any size: beyond 8 every one saturates (a NaN becomes finite here)
    const float most = 8.f * f;
#pragma unroll
    for (int i = 0; i < kFp4Block; ++i) {
      const float y = fminf(fmaxf(x[i], -most), most), q = y * inv;
      x[i] = copysignf(fmaf(fmaf(-q, f, y), inv, q), y);  // the step turns -0 into 0
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = make_float2(x[2 * i], x[2 * i + 1]), v = make_float2(x[8 + 2 * i], x[9 + 2 * i]);
      lo |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(u, __NV_E2M1, cudaRoundNearest)) << (8 * i);
      hi |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest)) << (8 * i);
    }
  }
  uint8_t* base = a.cache + page * fp4_page_bytes<D>(a.page_size);
  *reinterpret_cast<uint2*>(base + static_cast<int64_t>(row) * (D / 2) + blk * 8) = make_uint2(lo, hi);
  base[static_cast<int64_t>(a.page_size) * (D / 2) + static_cast<int64_t>(row) * kBlocks + blk] = static_cast<uint8_t>(sc);
}

template <int D, bool kF32>
__global__ void __launch_bounds__(kRowThreads) fp4_load_kernel(const __grid_constant__ Fp4RowsArgs a) {
  constexpr int kBlocks = D / kFp4Block;
  pdl_wait();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t r = id / kBlocks;
  const int blk = static_cast<int>(id % kBlocks);
  if (r >= a.n) return;
  const int64_t loc = a.loc[r];
  if (loc < 0) return;
  int64_t page;
  int32_t row;
  split_location(loc, a.page_size, a.page_shift, page, row);
  if (page >= a.num_pages) {
    if (blk == 0) flag_error(a.err, CKV_DEVERR_CACHE_LOC);
    return;
  }
  const uint8_t* base = a.cache + page * fp4_page_bytes<D>(a.page_size);
  const uint2 c = *reinterpret_cast<const uint2*>(base + static_cast<int64_t>(row) * (D / 2) + blk * 8);
  const float f =
      e4m3_to_float(base[static_cast<int64_t>(a.page_size) * (D / 2) + static_cast<int64_t>(row) * kBlocks + blk]) * a.g;
  float x[kFp4Block];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = e2m1x2_to_float2((c.x >> (8 * i)) & 0xFFu), v = e2m1x2_to_float2((c.y >> (8 * i)) & 0xFFu);
    x[2 * i] = u.x * f, x[2 * i + 1] = u.y * f, x[8 + 2 * i] = v.x * f, x[9 + 2 * i] = v.y * f;
  }
  if constexpr (kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out) + r * a.stride + blk * kFp4Block);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + r * a.stride + blk * kFp4Block);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      p[i] = make_uint4(pack_bf16x2_rn(x[8 * i], x[8 * i + 1]), pack_bf16x2_rn(x[8 * i + 2], x[8 * i + 3]),
                        pack_bf16x2_rn(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2_rn(x[8 * i + 6], x[8 * i + 7]));
  }
}

template <int D, bool kF32>
cudaError_t launch(const Fp4RowsArgs& a, bool store, bool use_pdl, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.n * (D / kFp4Block) + kRowThreads - 1) / kRowThreads);
  return store ? launch_ex(fp4_store_kernel<D, kF32>, dim3(grid), dim3(kRowThreads), 0, use_pdl, s, a)
               : launch_ex(fp4_load_kernel<D, kF32>, dim3(grid), dim3(kRowThreads), 0, use_pdl, s, a);
}

template <int D>
cudaError_t launch_d(const Fp4RowsArgs& a, int dtype, bool store, bool use_pdl, cudaStream_t s) {
  return dtype == CKV_F32 ? launch<D, true>(a, store, use_pdl, s) : launch<D, false>(a, store, use_pdl, s);
}

cudaError_t launch_any(const Fp4RowsArgs& a, int D, int dtype, bool store, bool use_pdl, cudaStream_t s) {
  return D == 128   ? launch_d<128>(a, dtype, store, use_pdl, s)
         : D == 256 ? launch_d<256>(a, dtype, store, use_pdl, s)
                    : launch_d<512>(a, dtype, store, use_pdl, s);
}

}  // namespace

cudaError_t launch_fp4_store(const Fp4RowsArgs& a, int D, int dtype, bool use_pdl, cudaStream_t s) {
  return launch_any(a, D, dtype, true, use_pdl, s);
}
cudaError_t launch_fp4_load(const Fp4RowsArgs& a, int D, int dtype, bool use_pdl, cudaStream_t s) {
  return launch_any(a, D, dtype, false, use_pdl, s);
}

}  // namespace ckv
