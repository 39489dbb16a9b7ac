// kv_append.cu -- keys (rotated) and values of new tokens into a paged bf16 cache, and
// the rotation of their queries, in one pass (no counterpart in the sources).
//
//   pairs (a, b) of the rotated span become (a c - b s, b c + a s), fp32, one rounding.
//
// Bound by HBM: every row is read once and written once.  A row takes 32 lanes (16 at D = 128, two
// rows to a warp); a warp takes a token and some of its heads, queries, keys and values alike, so that
// position, location and angles are loaded once for all of them.  Both channels of a pair belong to
// one lane.  Where pairs are neighbours it has pieces of eight channels.  Where they are halves of the
// span it has pieces of W channels and their W partners, lanes side by side, and those around the span
// by twos; W = 4 where the span and its half begin on such a piece, 2 where the half does, otherwise 1
// (8191 tokens x 48 heads of 128 channels: 34, 40 and 78 us; eight neighbours to a lane with their partners
// read one by one took 112).
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_fp4.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kAppendThreads = 256;
constexpr uint32_t kAppendShare = 16;  // heads of a token that a warp takes at most
enum Turn { kNone, kPairs, kHalves4, kHalves2, kHalves1 };

// CTAs of an SM, and of the grid: as many as registers allow without spilling much (64 of a thread with four).  A grid of more
// goes in waves, the last of them hardly filled, and long units leave SMs waiting at the end: 8191 tokens x 48 heads 40.6 us
// with 64 heads to a warp and eight CTAs per SM, 33.7 so; 4000 x 65 of 512 channels 158 and 102.
template <int D, Turn kTurn, bool kF32>
__host__ __device__ constexpr int append_ctas() {
  return kTurn == kHalves1 ? 2 : D == 512 && !kF32 ? 3 : 4;
}

// kBytes bytes of one lane, as many words.
template <int kBytes>
__device__ __forceinline__ void load_piece(const uint8_t* p, uint32_t* x) {
  if constexpr (kBytes >= 16) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      const uint4 w = reinterpret_cast<const uint4*>(p)[i];
      x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
    }
  } else if constexpr (kBytes == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    x[0] = w.x, x[1] = w.y;
  } else if constexpr (kBytes == 4) {
    x[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    x[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}

// W values to bf16.
template <int W>
__device__ __forceinline__ void store_piece(uint16_t* p, const float* v) {
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
  else if constexpr (W == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]));
  else if constexpr (W == 2) *reinterpret_cast<uint32_t*>(p) = pack_bf16x2_rn(v[0], v[1]);
  else *p = static_cast<uint16_t>(pack_bf16x2_rn(v[0], 0.f));
}

template <int D, Turn kTurn, bool kF32>
__global__ void __launch_bounds__(kAppendThreads, (append_ctas<D, kTurn, kF32>())) kv_append_kernel(const __grid_constant__ KvAppendArgs a, uint32_t share) {
  constexpr int kLanes = D >= 256 ? 32 : D / 8;  // of a row
  constexpr int kRows = 32 / kLanes;             // rows of a warp
  constexpr bool kHalves = kTurn >= kHalves4;
  constexpr int W = kTurn == kHalves1 ? 1 : kTurn == kHalves2 ? 2 : kTurn == kHalves4 ? 4 : 8;
  constexpr int N = D / kLanes / W;              // pieces of a lane; with halves, 2 n and 2 n + 1 belong together
  constexpr int kES = kF32 ? 4 : 2, kWords = W * kES >= 4 ? W * kES / 4 : 1;
  constexpr int kAngles = kHalves ? W : 4;       // of two pieces, or of one with pairs of neighbours
  constexpr int kBatch = (D == 512 ? 2 : 4) / (kF32 ? 2 : 1);  // rows of a lane in flight
  const int lane = threadIdx.x & 31, sl = lane % kLanes, sub = lane / kLanes;
  const int half = a.rope_dim >> 1;
  int base[N];
#pragma unroll
  for (int n = 0; n < N; n += kHalves ? 2 : 1) {
    if constexpr (kHalves) {
      const int c = (n / 2 * kLanes + sl) * W;
      if (c < half) {
        base[n] = a.rope_offset + c;
        base[n + 1] = a.rope_offset + half + c;
      } else {  // the channels around the span, by twos
        const int d = 2 * (c - half);
        base[n] = d < a.rope_offset ? d : d + a.rope_dim;
        base[n + 1] = d + W < a.rope_offset ? d + W : d + W + a.rope_dim;
      }
    } else {
      base[n] = (n * kLanes + sl) * 8;
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
    float co[N][kAngles], si[N][kAngles];
    bool turns[N];
#pragma unroll
    for (int n = 0; n < N; n += kHalves ? 2 : 1) {
      const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rope_dim;
      turns[n] = false;
      if constexpr (kTurn == kPairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = base[n] + 2 * j - a.rope_offset;
          const bool in = k >= 0 && k < a.rope_dim;
          turns[n] |= in;
          co[n][j] = in ? cs[k >> 1] : 1.f;
          si[n][j] = in ? cs[half + (k >> 1)] : 0.f;
        }
      } else if constexpr (kHalves) {
        const int c = (n / 2 * kLanes + sl) * W;
        turns[n] = c < half;
        if (turns[n]) {
          load_piece<4 * W>(reinterpret_cast<const uint8_t*>(cs + c), reinterpret_cast<uint32_t*>(co[n]));
          load_piece<4 * W>(reinterpret_cast<const uint8_t*>(cs + half + c), reinterpret_cast<uint32_t*>(si[n]));
        }
      }
    }
    for (uint32_t h = h0; h < h1; h += kBatch * kRows) {
      uint32_t raw[kBatch][N][kWords];
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
        const uint8_t* in = static_cast<const uint8_t*>(m.x) + (static_cast<int64_t>(t) * m.stride_t + i * m.stride_h) * kES;
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
          for (int x = 0; x < kWords; ++x) raw[b][n][x] = 0;
          if (to[b]) load_piece<W * kES>(in + base[n] * kES, raw[b][n]);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float v[N][W];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int j = 0; j < W; ++j)
            v[n][j] = kF32 ? __uint_as_float(raw[b][n][j * kES / 4]) : j % 2 ? bf16_hi(raw[b][n][j / 2]) : bf16_lo(raw[b][n][j / 2]);
#pragma unroll
        for (int n = 0; n < N; n += kHalves ? 2 : 1) {
          if (kTurn == kNone || !turned[b] || !turns[n]) continue;
          if constexpr (kTurn == kPairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float p = v[n][2 * j], q = v[n][2 * j + 1];
              const int k = base[n] + 2 * j - a.rope_offset;
              if (k >= 0 && k < a.rope_dim) {  // a pair outside stays what it is, infinite or not
                v[n][2 * j] = fmaf(p, co[n][j], -(q * si[n][j]));
                v[n][2 * j + 1] = fmaf(q, co[n][j], p * si[n][j]);
              }
            }
          } else if constexpr (kHalves) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
              const float p = v[n][j], q = v[n + 1][j];
              v[n][j] = fmaf(p, co[n][j], -(q * si[n][j]));
              v[n + 1][j] = fmaf(q, co[n][j], p * si[n][j]);
            }
          }
        }
        if (to[b]) {
#pragma unroll
          for (int n = 0; n < N; ++n) store_piece<W>(to[b] + base[n], v[n]);
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
  // Pieces as wide as the span's place, its half and the rows of angles allow; spans begin on even channels.
  const uintptr_t angles = reinterpret_cast<uintptr_t>(a.cos_sin);
  if (a.rope_offset % 4 == 0 && a.rope_dim % 8 == 0 && angles % 16 == 0) return launch<D, kHalves4, kF32>(a, use_pdl, s);
  if (a.rope_dim % 4 == 0 && angles % 8 == 0) return launch<D, kHalves2, kF32>(a, use_pdl, s);
  return launch<D, kHalves1, kF32>(a, use_pdl, s);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, int D, int dtype, bool use_pdl, cudaStream_t s) {
  if (dtype == CKV_F32)
    return D == 128 ? launch_d<128, true>(a, use_pdl, s) : D == 256 ? launch_d<256, true>(a, use_pdl, s) : launch_d<512, true>(a, use_pdl, s);
  return D == 128 ? launch_d<128, false>(a, use_pdl, s) : D == 256 ? launch_d<256, false>(a, use_pdl, s) : launch_d<512, false>(a, use_pdl, s);
}

}  // namespace ckv
