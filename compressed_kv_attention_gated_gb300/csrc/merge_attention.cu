// merge_attention.cu -- one attention from those over several sets of rows (no counterpart in
// the sources):  lse = log(sum_i e^lse_i),  out = sum_i e^(lse_i - lse) out_i.
//
// Bound by HBM: every part is read once, the result written once.  A row takes D/8 lanes
// (at most 32) with eight channels each; the loads of all parts are issued before the
// weights, which need the parts' lse, are formed.
#include <cmath>
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kMergeThreads = 256;
constexpr float kLn2 = 0.69314718055994531f;

template <int D, int kParts, bool kF32, bool kOutF32>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ MergeArgs a) {
  constexpr int kLanes = D >= 256 ? 32 : D / 8, kGroups = D / (kLanes * 8);
  pdl_wait();
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * kMergeThreads + threadIdx.x) / kLanes;
  const int sl = threadIdx.x % kLanes;
  const bool on = r < a.rows && (!a.positions || a.positions[r / a.H] >= 0);
  float s[kParts];
  uint4 raw[kParts][kGroups][kF32 ? 2 : 1];
  if (on) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      s[i] = -INFINITY;
      if (i < a.n) {
        s[i] = a.part[i].lse[r];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const int64_t at = r * D + (g * 32 + sl) * 8;
#pragma unroll
          for (int x = 0; x < (kF32 ? 2 : 1); ++x)
            raw[i][g][x] = kF32 ? *reinterpret_cast<const uint4*>(static_cast<const float*>(a.part[i].out) + at + x * 4)
                                : *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.part[i].out) + at);
        }
      }
    }
  }
  __syncwarp();  // the result may lie over a part: every lane has read its row's lse
  if (!on) return;
  float top = s[0];
#pragma unroll
  for (int i = 1; i < kParts; ++i) top = fmaxf(top, s[i]);
  const float safe = top == -INFINITY ? 0.f : top;
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    s[i] = s[i] == safe ? 1.f : fast_exp2((s[i] - safe) * kLog2e);  // infinity less infinity is no number
    all += s[i];
  }
  const float inv = all == 0.f ? 0.f : 1.f / all;
  if (a.lse && sl == 0) a.lse[r] = all == 0.f ? -INFINITY : safe + log2f(all) * kLn2;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      if (i < a.n && s[i] != 0.f) {
        const float w = s[i] * inv;
        const uint4 x = raw[i][g][0], y = raw[i][g][kF32 ? 1 : 0];
        float v[8];
        if constexpr (kF32) {
          v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y), v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
          v[4] = __uint_as_float(y.x), v[5] = __uint_as_float(y.y), v[6] = __uint_as_float(y.z), v[7] = __uint_as_float(y.w);
        } else {
          v[0] = bf16_lo(x.x), v[1] = bf16_hi(x.x), v[2] = bf16_lo(x.y), v[3] = bf16_hi(x.y);
          v[4] = bf16_lo(x.z), v[5] = bf16_hi(x.z), v[6] = bf16_lo(x.w), v[7] = bf16_hi(x.w);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fmaf(v[j], w, o[j]);
      }
    }
    const int64_t at = r * D + (g * 32 + sl) * 8;
    if constexpr (kOutF32) {
      float* to = static_cast<float*>(a.out) + at;
      *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<float4*>(to + 4) = make_float4(o[4], o[5], o[6], o[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) =
          make_uint4(pack_bf16x2_rn(o[0], o[1]), pack_bf16x2_rn(o[2], o[3]), pack_bf16x2_rn(o[4], o[5]), pack_bf16x2_rn(o[6], o[7]));
    }
  }
}

template <int D, int kParts, bool kF32, bool kOutF32>
cudaError_t launch(const MergeArgs& a, bool use_pdl, cudaStream_t s) {
  constexpr int kRows = kMergeThreads / (D >= 256 ? 32 : D / 8);  // of a CTA
  return launch_ex(merge_kernel<D, kParts, kF32, kOutF32>, dim3(static_cast<unsigned>((a.rows + kRows - 1) / kRows)), dim3(kMergeThreads), 0,
                   use_pdl, s, a);
}

template <int D, bool kF32, bool kOutF32>
cudaError_t launch_n(const MergeArgs& a, bool use_pdl, cudaStream_t s) {
  if (a.n <= 2) return launch<D, 2, kF32, kOutF32>(a, use_pdl, s);
  if (a.n <= 4) return launch<D, 4, kF32, kOutF32>(a, use_pdl, s);
  return launch<D, 8, kF32, kOutF32>(a, use_pdl, s);
}

template <int D>
cudaError_t launch_d(const MergeArgs& a, int dtype, int out_dtype, bool use_pdl, cudaStream_t s) {
  if (dtype == CKV_F32)
    return out_dtype == CKV_F32 ? launch_n<D, true, true>(a, use_pdl, s) : launch_n<D, true, false>(a, use_pdl, s);
  return out_dtype == CKV_F32 ? launch_n<D, false, true>(a, use_pdl, s) : launch_n<D, false, false>(a, use_pdl, s);
}

}  // namespace

cudaError_t launch_merge_attention(const MergeArgs& a, int D, int dtype, int out_dtype, bool use_pdl, cudaStream_t s) {
  return D == 128   ? launch_d<128>(a, dtype, out_dtype, use_pdl, s)
         : D == 256 ? launch_d<256>(a, dtype, out_dtype, use_pdl, s)
                    : launch_d<512>(a, dtype, out_dtype, use_pdl, s);
}

}  // namespace ckv
