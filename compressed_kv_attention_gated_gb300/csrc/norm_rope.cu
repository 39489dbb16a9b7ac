// norm_rope.cu -- root-mean-square norm of every head's vector and the rotation
// of its position in one pass (no counterpart in the sources).
//
//   y = x * rsqrt(mean(x^2) + eps) * w,  then pairs (a, b) of the rotated span
//   become (a c - b s, b c + a s); fp32 throughout, one rounding to the output.
//
// Bound by HBM: D values in, D values out, a few FMAs each.  One warp per
// (token, head) row; a lane owns 8 neighbouring channels per 256 (4 at D =
// 128), so a row is read and written in 16-byte (8-byte) accesses, 512 (256)
// consecutive bytes per warp.  The rotation's partner channel sits in another
// lane when pairs are halves of the span: the normalised row then goes through
// the warp's own row in shared memory, which serves any even span and offset.
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kNormThreads = 256;

template <int N>
__device__ __forceinline__ void load_row(const void* p, int dtype, int64_t at, float* v) {
  if (dtype == CKV_F32) {
    const float* r = static_cast<const float*>(p) + at;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(r + i);
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
  } else {
    const uint16_t* r = static_cast<const uint16_t*>(p) + at;
    if constexpr (N == 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(r);
      v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
      v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(r);
      v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    }
  }
}

template <int N>
__device__ __forceinline__ void store_row(void* p, int dtype, int64_t at, const float* v) {
  if (dtype == CKV_F32) {
    float* r = static_cast<float*>(p) + at;
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(r + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    uint16_t* r = static_cast<uint16_t*>(p) + at;
    if constexpr (N == 8) {
      *reinterpret_cast<uint4*>(r) = make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                                                pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
    } else {
      *reinterpret_cast<uint2*>(r) = make_uint2(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kVec = D == 128 ? 4 : 8;        // neighbouring channels of a lane
  constexpr int kGroups = D / (32 * kVec);      // groups of them per lane
  __shared__ float s_rows[kNormThreads / 32][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_row = s_rows[warp];
  pdl_wait();
  const int64_t rows_q = a.set[0].tokens * a.set[0].heads;
  const int64_t rows = rows_q + a.set[1].tokens * a.set[1].heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kNormThreads / 32);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kNormThreads / 32) + warp; r < rows; r += step) {
    const ckv_norm_rows& m = r < rows_q ? a.set[0] : a.set[1];
    const int64_t i = r < rows_q ? r : r - rows_q;
    const int64_t t = i / m.heads;
    const int64_t h = i - t * m.heads;
    const int32_t pos = m.positions[t];
    if (pos < 0) continue;
    if (a.rope_dim > 0 && pos >= a.num_positions) {
      if (lane == 0 && h == 0) flag_error(a.err, CKV_DEVERR_SEQ_LEN);
      continue;
    }
    float v[kGroups][kVec];
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      load_row<kVec>(m.x, m.dtype, t * m.stride_t + h * m.stride_h + g * 32 * kVec + lane * kVec, v[g]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) sum = fmaf(v[g][j], v[g][j], sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float inv = 1.f / sqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int c = g * 32 * kVec + lane * kVec + j;
        v[g][j] *= inv;
        if (m.weight) v[g][j] *= __ldg(m.weight + c);
        s_row[c] = v[g][j];
      }
    }
    if (a.rope_dim > 0) {
      __syncwarp();
      const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rope_dim;
      const int half = a.rope_dim >> 1;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const int c = g * 32 * kVec + lane * kVec + j;
          const int k = c - a.rope_offset;
          if (k >= 0 && k < a.rope_dim) {
            const bool second = a.interleaved ? (k & 1) : k >= half;
            const int p = a.interleaved ? k >> 1 : (second ? k - half : k);
            const int mate = a.interleaved ? (c ^ 1) : (second ? c - half : c + half);
            const float co = __ldg(cs + p), si = __ldg(cs + half + p);
            v[g][j] = second ? v[g][j] * co + s_row[mate] * si : v[g][j] * co - s_row[mate] * si;
          }
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      store_row<kVec>(m.out, m.out_dtype, t * m.out_stride_t + h * m.out_stride_h + g * 32 * kVec + lane * kVec, v[g]);
    __syncwarp();
  }
}

template <int D>
cudaError_t launch_d(const NormRopeArgs& a, bool use_pdl, cudaStream_t s) {
  const int64_t rows = a.set[0].tokens * a.set[0].heads + a.set[1].tokens * a.set[1].heads;
  const int64_t want = (rows + kNormThreads / 32 - 1) / (kNormThreads / 32);
  const unsigned grid = static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20));
  return launch_ex(norm_rope_kernel<D>, dim3(grid), dim3(kNormThreads), 0, use_pdl, s, a);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int D, bool use_pdl, cudaStream_t s) {
  return D == 128 ? launch_d<128>(a, use_pdl, s) : D == 256 ? launch_d<256>(a, use_pdl, s) : launch_d<512>(a, use_pdl, s);
}

}  // namespace ckv
