// fp4_attention.cu -- attention over the 4-bit paged cache (no counterpart in
// the sources; the format is in ckv_fp4.cuh).  Every cache row is key and
// value of all heads:
//   z_j = scale <q, k_j>,  lse = log(sum_j e^z_j [+ e^sink]),  out = sum_j e^(z_j - lse) k_j.
//
// One warp per (token, head): a lane holds D/32 channels of the query and of
// the output, and the running maximum and sum of the softmax.
#include <cmath>
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_fp4.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kAttnThreads = 128;

template <int D>
__global__ void __launch_bounds__(kAttnThreads) fp4_attention_kernel(const __grid_constant__ Fp4AttentionArgs a) {
  constexpr int kC = D / 32;  // channels of a lane
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * (kAttnThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = id / a.H;
  const int h = static_cast<int>(id - t * a.H);
  if (t >= a.T || t >= a.row_start[a.B]) return;
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.row_start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  int ctx = a.ctx_rows[t];
  if (ctx < 0) return;
  if (ctx > a.max_rows) {
    if (lane == 0) flag_error(a.err, CKV_DEVERR_SEQ_LEN);
    ctx = a.max_rows;
  }
  float q[kC], o[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.q_st + h * a.q_sh + lane * kC + i]) << 16);
    o[i] = 0.f;
  }
  const float zs = a.softmax_scale * kLog2e;
  float m = -INFINITY, l = 0.f;
  if (a.sink) {
    m = a.sink[h] * kLog2e;
    l = m > -INFINITY ? 1.f : 0.f;
  }
  const int32_t* table = a.table + static_cast<int64_t>(lo) * a.table_stride;
  for (int j = 0; j < ctx; ++j) {
    const int32_t page = table[j / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) flag_error(a.err, CKV_DEVERR_CACHE_LOC);
      continue;
    }
    const uint8_t* base = a.cache + page * fp4_page_bytes<D>(a.page_size);
    const int64_t row = j % a.page_size;
    const float f = e4m3_to_float(base[static_cast<int64_t>(a.page_size) * (D / 2) + row * (D / kFp4Block) + lane * kC / kFp4Block]) * a.g;
    float k[kC], z = 0.f;
#pragma unroll
    for (int i = 0; i < kC; i += 2) {
      const float2 u = e2m1x2_to_float2(base[row * (D / 2) + (lane * kC + i) / 2]);
      k[i] = u.x * f, k[i + 1] = u.y * f;
      z = fmaf(q[i], k[i], fmaf(q[i + 1], k[i + 1], z));
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
    z *= zs;
    const float top = fmaxf(m, z);
    const float keep = m > -INFINITY ? fast_exp2(m - top) : 0.f, p = fast_exp2(z - top);
    l = fmaf(l, keep, p);
    m = top;
#pragma unroll
    for (int i = 0; i < kC; ++i) o[i] = fmaf(o[i], keep, p * k[i]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
#pragma unroll
  for (int i = 0; i < kC; i += 2)
    *reinterpret_cast<uint32_t*>(a.out + (t * a.H + h) * D + lane * kC + i) = pack_bf16x2_rn(o[i] * inv, o[i + 1] * inv);
  if (lane == 0 && a.lse) a.lse[t * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int D>
cudaError_t launch_d(const Fp4AttentionArgs& a, bool use_pdl, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.T * a.H + kAttnThreads / 32 - 1) / (kAttnThreads / 32));
  return launch_ex(fp4_attention_kernel<D>, dim3(grid), dim3(kAttnThreads), 0, use_pdl, s, a);
}

}  // namespace

int64_t fp4_attention_workspace(int64_t, int32_t, int32_t, int32_t, int64_t) { return 0; }

cudaError_t launch_fp4_attention(const Fp4AttentionArgs& a, int D, bool use_pdl, cudaStream_t s) {
  return D == 128 ? launch_d<128>(a, use_pdl, s) : D == 256 ? launch_d<256>(a, use_pdl, s) : launch_d<512>(a, use_pdl, s);
}

}  // namespace ckv
