// kv_append.cu -- keys (rotated) and values of new tokens into a paged bf16 cache, and
// the rotation of their queries, in one pass (no counterpart in the sources).
//
//   pairs (a, b) of the rotated span become (a c - b s, b c + a s), fp32, one rounding.
//
// Bound by HBM: every row is read once and written once.  A lane owns eight channels
// (two such groups at D = 512), a row takes 32 lanes (16 at D = 128, two rows to a
// warp); a warp takes a token and some of its heads, queries, keys and values alike, so that
// position, location and angles are loaded once for all of them.  Both channels of a
// pair belong to one lane: eight neighbours when pairs are neighbours, four and their four
// partners when they are halves of the span.  Halves that are not whole groups of four
// channels read their partners one by one (from L1: the row has just been read).
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_fp4.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kAppendThreads = 256;
constexpr uint32_t kAppendShare = 16;  // heads of a token that a warp takes at most
enum Turn { kNone, kPairs, kHalves, kOddHalves };

// CTAs of an SM, and of the grid: as many as registers allow without spilling much (64 of a thread with four).  A grid of more
// goes in waves, the last of them hardly filled, and long units leave SMs waiting at the end: 8191 tokens x 48 heads 40.6 us
// with 64 heads to a warp and eight CTAs per SM, 33.7 so; 4000 x 65 of 512 channels 158 and 102.
template <int D, Turn kTurn, bool kF32>
__host__ __device__ constexpr int append_ctas() {
  return kTurn == kOddHalves ? (D == 512 ? 1 : 2) : D == 512 && !kF32 ? 3 : 4;
}

__device__ __forceinline__ float value_at(const void* x, int64_t i, bool f32) {
  return f32 ? static_cast<const float*>(x)[i] : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(x)[i]) << 16);
}

template <int D, Turn kTurn, bool kF32>
__global__ void __launch_bounds__(kAppendThreads, (append_ctas<D, kTurn, kF32>())) kv_append_kernel(const __grid_constant__ KvAppendArgs a, uint32_t share) {
  constexpr int kLanes = D >= 256 ? 32 : D / 8;  // of a row
  constexpr int kRows = 32 / kLanes;             // rows of a warp
  constexpr int kGroups = D / (kLanes * 8);
  constexpr int kBatch = (D == 512 ? 2 : 4) / (kF32 ? 2 : 1);  // rows of a lane in flight
  const int lane = threadIdx.x & 31, sl = lane % kLanes, sub = lane / kLanes;
  const int half = a.rope_dim >> 1;
  int base[kGroups][2];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int q = g * 32 + sl;  // of D/8
    base[g][0] = q * 8;
    base[g][1] = q * 8 + 4;
    if constexpr (kTurn == kHalves) {
      if (q * 8 < a.rope_dim) {
        base[g][0] = a.rope_offset + q * 4;
        base[g][1] = a.rope_offset + half + q * 4;
      } else {  // the channels around the span, four by four
        const int c = q * 8 - a.rope_dim;
        base[g][0] = c < a.rope_offset ? c : c + a.rope_dim;
        base[g][1] = c + 4 < a.rope_offset ? c + 4 : c + 4 + a.rope_dim;
      }
    }
  }
  pdl_wait();
  const uint32_t hq = a.set[0].heads, hk = hq + a.set[1].heads, heads = hk + a.set[2].heads;
  const uint32_t per = (heads + share - 1) / share, units = static_cast<uint32_t>(a.T) * per;
  const uint32_t stride = gridDim.x * (kAppendThreads / 32);
  uint32_t u = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  int64_t next_loc = 0;  // of the next unit's token: known when it begins
  int32_t next_pos = 0;
  if (u < units) {
    next_loc = a.loc[u / per];
    next_pos = a.positions ? a.positions[u / per] : 0;
  }
  for (; u < units; u += stride) {
    const uint32_t t = u / per, h0 = (u - t * per) * share, h1 = min(h0 + share, heads);
    const int64_t loc = next_loc;
    const int32_t pos = next_pos;
    if (u + stride < units) {
      next_loc = a.loc[(u + stride) / per];
      next_pos = a.positions ? a.positions[(u + stride) / per] : 0;
    }
    if (pos < 0) continue;
    if (kTurn != kNone && pos >= a.num_positions) {
      if (lane == 0) flag_error(a.err, CKV_DEVERR_SEQ_LEN);
      continue;
    }
    bool stored = loc >= 0;
    int64_t page = 0;
    int32_t row = 0;
    if (stored) {
      split_location(loc, a.cache.page_size, a.page_shift, page, row);
      if (page >= a.cache.num_pages) {
        stored = false;
        if (lane == 0) flag_error(a.err, CKV_DEVERR_CACHE_LOC);
      }
    }
    // angles of the lane's pairs, (1, 0) outside the span
    float co[kGroups][kTurn == kOddHalves ? 8 : 4], si[kGroups][kTurn == kOddHalves ? 8 : 4];
    int mate[kGroups][kTurn == kOddHalves ? 8 : 1];
    bool turns[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rope_dim;
      turns[g] = false;
      if constexpr (kTurn == kPairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = base[g][0] + 2 * j - a.rope_offset;
          const bool in = k >= 0 && k < a.rope_dim;
          turns[g] |= in;
          co[g][j] = in ? cs[k >> 1] : 1.f;
          si[g][j] = in ? cs[half + (k >> 1)] : 0.f;
        }
      } else if constexpr (kTurn == kHalves) {
        turns[g] = (g * 32 + sl) * 8 < a.rope_dim;
        float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turns[g]) {
          const int p = base[g][0] - a.rope_offset;
          c4 = *reinterpret_cast<const float4*>(cs + p);
          s4 = *reinterpret_cast<const float4*>(cs + half + p);
        }
        co[g][0] = c4.x, co[g][1] = c4.y, co[g][2] = c4.z, co[g][3] = c4.w;
        si[g][0] = s4.x, si[g][1] = s4.y, si[g][2] = s4.z, si[g][3] = s4.w;
      } else if constexpr (kTurn == kOddHalves) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = base[g][0] + j, k = c - a.rope_offset;
          const bool in = k >= 0 && k < a.rope_dim, second = k >= half;
          const int p = second ? k - half : k;
          turns[g] |= in;
          mate[g][j] = !in ? -1 : second ? c - half : c + half;
          co[g][j] = in ? cs[p] : 1.f;
          si[g][j] = !in ? 0.f : second ? cs[half + p] : -cs[half + p];
        }
      }
    }
    for (uint32_t h = h0; h < h1; h += kBatch * kRows) {
      uint4 raw[kBatch][kGroups][kF32 ? 2 : 1];
      float other[kBatch][kGroups][kTurn == kOddHalves ? 8 : 1];
      uint16_t* to[kBatch];
      bool turned[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const uint32_t hh = h + b * kRows + sub;
        const int set = hh < hq ? 0 : hh < hk ? 1 : 2;
        const uint32_t i = hh - (set == 0 ? 0 : set == 1 ? hq : hk);
        to[b] = nullptr;
        turned[b] = set < 2;
        if (hh < h1) {
          if (set == 0) to[b] = a.q_out + t * a.qo_st + i * a.qo_sh;
          else if (!stored) to[b] = nullptr;
          else if (set == 1) to[b] = a.cache.k + page * a.cache.k_stride_page + row * a.cache.k_stride_row + i * a.cache.k_stride_head;
          else to[b] = a.cache.v + page * a.cache.v_stride_page + row * a.cache.v_stride_row + i * a.cache.v_stride_head;
        }
        const ckv_kv_rows& m = a.set[set];
        const int64_t in = static_cast<int64_t>(t) * m.stride_t + i * m.stride_h;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          raw[b][g][0] = raw[b][g][kF32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
          if (to[b]) {
            if constexpr (kF32) {
#pragma unroll
              for (int x = 0; x < 2; ++x) raw[b][g][x] = *reinterpret_cast<const uint4*>(static_cast<const float*>(m.x) + in + base[g][x]);
            } else if constexpr (kTurn == kHalves) {
              const uint2 lo = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(m.x) + in + base[g][0]);
              const uint2 hi = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(m.x) + in + base[g][1]);
              raw[b][g][0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
              raw[b][g][0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(m.x) + in + base[g][0]);
            }
          }
          if constexpr (kTurn == kOddHalves) {
#pragma unroll
            for (int j = 0; j < 8; ++j) other[b][g][j] = to[b] && turned[b] && mate[g][j] >= 0 ? value_at(m.x, in + mate[g][j], kF32) : 0.f;
          }
        }
      }
      // queries may be rotated in place: their partners' values are read by now
      if constexpr (kTurn == kOddHalves) __syncwarp();
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          float v[8];
          const uint4 x = raw[b][g][0], y = raw[b][g][kF32 ? 1 : 0];
          if constexpr (kF32) {
            v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y), v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
            v[4] = __uint_as_float(y.x), v[5] = __uint_as_float(y.y), v[6] = __uint_as_float(y.z), v[7] = __uint_as_float(y.w);
          } else {
            v[0] = bf16_lo(x.x), v[1] = bf16_hi(x.x), v[2] = bf16_lo(x.y), v[3] = bf16_hi(x.y);
            v[4] = bf16_lo(x.z), v[5] = bf16_hi(x.z), v[6] = bf16_lo(x.w), v[7] = bf16_hi(x.w);
          }
          if (turned[b] && turns[g]) {
            if constexpr (kTurn == kPairs) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float p = v[2 * j], q = v[2 * j + 1];
                const int k = base[g][0] + 2 * j - a.rope_offset;
                if (k >= 0 && k < a.rope_dim) {  // a pair outside stays what it is, infinite or not
                  v[2 * j] = fmaf(p, co[g][j], -(q * si[g][j]));
                  v[2 * j + 1] = fmaf(q, co[g][j], p * si[g][j]);
                }
              }
            } else if constexpr (kTurn == kHalves) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float p = v[j], q = v[4 + j];
                v[j] = fmaf(p, co[g][j], -(q * si[g][j]));
                v[4 + j] = fmaf(q, co[g][j], p * si[g][j]);
              }
            } else if constexpr (kTurn == kOddHalves) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (mate[g][j] >= 0) v[j] = fmaf(v[j], co[g][j], other[b][g][j] * si[g][j]);
            }
          }
          if (to[b]) {
            const uint4 o = make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
            if constexpr (kTurn == kHalves) {
              *reinterpret_cast<uint2*>(to[b] + base[g][0]) = make_uint2(o.x, o.y);
              *reinterpret_cast<uint2*>(to[b] + base[g][1]) = make_uint2(o.z, o.w);
            } else {
              *reinterpret_cast<uint4*>(to[b] + base[g][0]) = o;
            }
          }
        }
      }
    }
  }
}

template <int D, Turn kTurn, bool kF32>
cudaError_t launch(const KvAppendArgs& a, bool use_pdl, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // as many heads of a token to a warp as leaves every resident warp two units
  const int64_t heads = static_cast<int64_t>(a.set[0].heads) + a.set[1].heads + a.set[2].heads;
  const int64_t most = static_cast<int64_t>(sms) * append_ctas<D, kTurn, kF32>();
  int64_t units = 0;
  uint32_t share = kAppendShare;
  for (;; share /= 2) {
    units = a.T * ((heads + share - 1) / share);
    if (units >= 2 * (kAppendThreads / 32) * most || share == 1) break;
  }
  const int64_t want = (units + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  return launch_ex(kv_append_kernel<D, kTurn, kF32>, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kAppendThreads), 0,
                   use_pdl, s, a, share);
}

template <int D, bool kF32>
cudaError_t launch_d(const KvAppendArgs& a, bool use_pdl, cudaStream_t s) {
  if (a.rope_dim == 0) return launch<D, kNone, kF32>(a, use_pdl, s);
  if (a.interleaved) return launch<D, kPairs, kF32>(a, use_pdl, s);
  // halves of whole groups of four channels, and cos | sin rows that 16-byte loads can start in
  const bool whole = a.rope_offset % 4 == 0 && a.rope_dim % 8 == 0 && reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0;
  return whole ? launch<D, kHalves, kF32>(a, use_pdl, s) : launch<D, kOddHalves, kF32>(a, use_pdl, s);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, int D, int dtype, bool use_pdl, cudaStream_t s) {
  if (dtype == CKV_F32)
    return D == 128 ? launch_d<128, true>(a, use_pdl, s) : D == 256 ? launch_d<256, true>(a, use_pdl, s) : launch_d<512, true>(a, use_pdl, s);
  return D == 128 ? launch_d<128, false>(a, use_pdl, s) : D == 256 ? launch_d<256, false>(a, use_pdl, s) : launch_d<512, false>(a, use_pdl, s);
}

}  // namespace ckv
