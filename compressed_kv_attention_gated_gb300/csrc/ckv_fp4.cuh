// ckv_fp4.cuh -- the 4-bit row format: blocks of 16 channels as FP4-e2m1 codes
// with one FP8-e4m3 scale, in a paged cache (per page: page_size rows of D/2
// code bytes, then page_size rows of D/16 scale bytes).
#pragma once

#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "ckv_device.cuh"

namespace ckv {

constexpr int kFp4Block = 16;

// Page and row of a cache location >= 0 (a shift when the page size is a power
// of two: the 64-bit division is a long instruction sequence).
__device__ __forceinline__ void split_location(int64_t loc, int32_t page_size, int32_t page_shift, int64_t& page,
                                               int32_t& row) {
  if (page_shift >= 0) {
    page = loc >> page_shift;
    row = static_cast<int32_t>(loc) & (page_size - 1);
  } else {
    page = loc / page_size;
    row = static_cast<int32_t>(loc - page * page_size);
  }
}

template <int D>
__device__ __forceinline__ int64_t fp4_page_bytes(int32_t page_size) {
  return static_cast<int64_t>(page_size) * (D / 2 + D / kFp4Block);
}

__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
  return __half2float(__half(h));
}

// Two e2m1 codes (low half: first) as floats.
__device__ __forceinline__ float2 e2m1x2_to_float2(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
  return __half22float2(__half2(h));
}

}  // namespace ckv
