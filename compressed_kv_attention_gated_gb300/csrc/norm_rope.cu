// norm_rope.cu -- root-mean-square norm of every head's vector and the rotation
// of its position in one pass (no counterpart in the sources).
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then pairs (a, b) of the rotated span
//   become (a c - b s, b c + a s); fp32 throughout, one rounding to the output.
//
// Bound by HBM: D values in, D values out, a few FMAs each.  A lane owns eight
// neighbouring channels (two such groups at D = 512), so every access is 16
// bytes per lane; a row takes 32 lanes (16 at D = 128, two rows to a warp).
// Warps stay resident and walk over the rows: the next row and its position
// are on their way while a row is worked on, and weights stay in registers.
//
// The rotation's partner is in the same lane when pairs are neighbours, and in
// another one when they are halves of the span: the normalised row then goes
// through the warp's row in shared memory.  Spans and offsets that are not whole
// groups of eight channels (16 for halves) take a channel-by-channel path.
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormBlocks = 4;  // per SM

enum Rotation { kNone, kPairs, kHalves, kAny };

// A lane's channels of one row as they come from memory, and where they belong.
template <int kGroups>
struct Fetched {
  uint4 raw[kGroups * 2];  // fp32: 8 words per group; bf16: the first 4
  int64_t out;             // element offset of the row's output
  int32_t pos;             // < 0: nothing to do
  int32_t set;
};

__device__ __forceinline__ float4 as_float4(uint4 w) {
  return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
}

template <int D, Rotation kRot>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kLanes = D >= 256 ? 32 : D / 8;   // of a row
  constexpr int kRows = 32 / kLanes;              // rows of a warp
  constexpr int kGroups = D / (kLanes * 8);
  constexpr bool kStage = kRot == kHalves || kRot == kAny;
  __shared__ __align__(16) float s_rows[kStage ? kNormThreads / 32 * kRows : 1][kStage ? D : 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / kLanes, sl = lane % kLanes;
  float* s_row = s_rows[kStage ? warp * kRows + sub : 0];
  pdl_wait();
  const uint32_t rows_q = static_cast<uint32_t>(a.set[0].tokens * a.set[0].heads);
  const uint32_t rows = rows_q + static_cast<uint32_t>(a.set[1].tokens * a.set[1].heads);
  const uint32_t step = gridDim.x * (kNormThreads / 32) * kRows;

  auto fetch = [&](Fetched<kGroups>& f, uint32_t r) {
    f.pos = -1;
    if (r >= rows) return;
    f.set = r >= rows_q;
    const ckv_norm_rows& m = a.set[f.set];
    const uint32_t i = f.set ? r - rows_q : r;
    const uint32_t t = i / static_cast<uint32_t>(m.heads), h = i - t * static_cast<uint32_t>(m.heads);
    f.out = t * m.out_stride_t + h * m.out_stride_h;
    f.pos = m.positions[t];
    const int64_t in = t * m.stride_t + h * m.stride_h + sl * 8;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (m.dtype == CKV_F32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(m.x) + in + g * 256);
        f.raw[2 * g] = p[0];
        f.raw[2 * g + 1] = p[1];
      } else {
        f.raw[2 * g] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(m.x) + in + g * 256);
      }
    }
  };

  float w[kGroups][8];
  int w_set = -1;
  uint32_t base = (blockIdx.x * (kNormThreads / 32) + warp) * kRows;
  Fetched<kGroups> next;
  fetch(next, base + sub);
  for (; base < rows; base += step) {
    const Fetched<kGroups> f = next;
    if (base + step < rows) fetch(next, base + step + sub);
    const ckv_norm_rows& m = a.set[f.pos >= 0 ? f.set : 0];
    bool on = f.pos >= 0;
    if (kRot != kNone && on && f.pos >= a.num_positions) {
      if (sl == 0) flag_error(a.err, CKV_DEVERR_SEQ_LEN);
      on = false;
    }
    float v[kGroups][8];
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (m.dtype == CKV_F32) {
        const float4 x = as_float4(f.raw[2 * g]), y = as_float4(f.raw[2 * g + 1]);
        v[g][0] = x.x, v[g][1] = x.y, v[g][2] = x.z, v[g][3] = x.w;
        v[g][4] = y.x, v[g][5] = y.y, v[g][6] = y.z, v[g][7] = y.w;
      } else {
        const uint4 x = f.raw[2 * g];
        v[g][0] = bf16_lo(x.x), v[g][1] = bf16_hi(x.x), v[g][2] = bf16_lo(x.y), v[g][3] = bf16_hi(x.y);
        v[g][4] = bf16_lo(x.z), v[g][5] = bf16_hi(x.z), v[g][6] = bf16_lo(x.w), v[g][7] = bf16_hi(x.w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[g][j], v[g][j], sum);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float inv = 1.f / sqrtf(sum * (1.f / D) + a.eps);
    if (on && w_set != f.set) {
      w_set = f.set;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const float4 x = m.weight ? *reinterpret_cast<const float4*>(m.weight + g * 256 + sl * 8 + j) : make_float4(1.f, 1.f, 1.f, 1.f);
          w[g][j] = x.x, w[g][j + 1] = x.y, w[g][j + 2] = x.z, w[g][j + 3] = x.w;
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[g][j] *= inv * w[g][j];
      if constexpr (kStage) {
        float4* s = reinterpret_cast<float4*>(s_row + g * 256 + sl * 8);
        s[0] = make_float4(v[g][0], v[g][1], v[g][2], v[g][3]);
        s[1] = make_float4(v[g][4], v[g][5], v[g][6], v[g][7]);
      }
    }
    if constexpr (kStage) __syncwarp();
    if (kRot != kNone && on) {
      const float* cs = a.cos_sin + static_cast<int64_t>(f.pos) * a.rope_dim;
      const int half = a.rope_dim >> 1;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int c0 = g * 256 + sl * 8, k0 = c0 - a.rope_offset;
        if constexpr (kRot == kPairs) {
          if (k0 >= 0 && k0 < a.rope_dim) {
            const float4 co = __ldg(reinterpret_cast<const float4*>(cs + k0 / 2)), si = __ldg(reinterpret_cast<const float4*>(cs + half + k0 / 2));
            const float c[4] = {co.x, co.y, co.z, co.w}, s[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x = v[g][2 * j], y = v[g][2 * j + 1];
              v[g][2 * j] = x * c[j] - y * s[j];
              v[g][2 * j + 1] = y * c[j] + x * s[j];
            }
          }
        } else if constexpr (kRot == kHalves) {
          if (k0 >= 0 && k0 < a.rope_dim) {
            const bool second = k0 >= half;
            const int p = second ? k0 - half : k0;
            const float* mate = s_row + (second ? c0 - half : c0 + half);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
              const float4 co = __ldg(reinterpret_cast<const float4*>(cs + p + j)), si = __ldg(reinterpret_cast<const float4*>(cs + half + p + j));
              const float4 o = *reinterpret_cast<const float4*>(mate + j);
              const float c[4] = {co.x, co.y, co.z, co.w}, s[4] = {si.x, si.y, si.z, si.w}, z[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x = v[g][j + i];
                v[g][j + i] = second ? x * c[i] + z[i] * s[i] : x * c[i] - z[i] * s[i];
              }
            }
          }
        } else if constexpr (kRot == kAny) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = c0 + j, k = k0 + j;
            if (k >= 0 && k < a.rope_dim) {
              const bool second = a.interleaved ? (k & 1) : k >= half;
              const int p = a.interleaved ? k >> 1 : (second ? k - half : k);
              const int mate = a.interleaved ? (second ? c - 1 : c + 1) : (second ? c - half : c + half);
              const float co = __ldg(cs + p), si = __ldg(cs + half + p);
              v[g][j] = second ? v[g][j] * co + s_row[mate] * si : v[g][j] * co - s_row[mate] * si;
            }
          }
        }
      }
    }
    if (on) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int64_t at = f.out + g * 256 + sl * 8;
        if (m.out_dtype == CKV_F32) {
          float4* p = reinterpret_cast<float4*>(static_cast<float*>(m.out) + at);
          p[0] = make_float4(v[g][0], v[g][1], v[g][2], v[g][3]);
          p[1] = make_float4(v[g][4], v[g][5], v[g][6], v[g][7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(m.out) + at) =
              make_uint4(pack_bf16x2_rn(v[g][0], v[g][1]), pack_bf16x2_rn(v[g][2], v[g][3]),
                         pack_bf16x2_rn(v[g][4], v[g][5]), pack_bf16x2_rn(v[g][6], v[g][7]));
        }
      }
    }
    if constexpr (kStage) __syncwarp();
  }
}

template <int D, Rotation kRot>
cudaError_t launch_rot(const NormRopeArgs& a, bool use_pdl, cudaStream_t s) {
  constexpr int kPerBlock = kNormThreads / 32 * (D >= 256 ? 1 : 256 / D);
  const int64_t rows = a.set[0].tokens * a.set[0].heads + a.set[1].tokens * a.set[1].heads;
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int64_t want = (rows + kPerBlock - 1) / kPerBlock, most = static_cast<int64_t>(sms) * kNormBlocks;
  return launch_ex(norm_rope_kernel<D, kRot>, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kNormThreads), 0, use_pdl,
                   s, a);
}

template <int D>
cudaError_t launch_d(const NormRopeArgs& a, bool use_pdl, cudaStream_t s) {
  if (a.rope_dim == 0) return launch_rot<D, kNone>(a, use_pdl, s);
  // whole groups of eight channels, and cos | sin rows that 16-byte loads can start in
  const bool whole = a.rope_offset % 8 == 0 && a.rope_dim % (a.interleaved ? 8 : 16) == 0 &&
                     reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0;
  if (!whole) return launch_rot<D, kAny>(a, use_pdl, s);
  return a.interleaved ? launch_rot<D, kPairs>(a, use_pdl, s) : launch_rot<D, kHalves>(a, use_pdl, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int D, bool use_pdl, cudaStream_t s) {
  return D == 128 ? launch_d<128>(a, use_pdl, s) : D == 256 ? launch_d<256>(a, use_pdl, s) : launch_d<512>(a, use_pdl, s);
}

}  // namespace ckv
