// norm_rope.cu -- root-mean-square norm of every head's vector and the rotation
// of its position in one pass (no counterpart in the sources).
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then pairs (a, b) of the rotated span
//   become (a c - b s, b c + a s); fp32 throughout, one rounding to the output.
//
// Bound by HBM: D values in, D values out, a few FMAs each.  A lane owns eight
// channels (two such groups at D = 512), a row takes 32 lanes (16 at D = 128, two
// rows to a warp).  A warp takes a token and some of its heads: position, angles
// and weights are loaded once for all of them, and the next rows are on their way
// (2 KB per warp) while a batch of rows is worked on, whose sums are formed side by
// side so that the shuffles' latencies overlap.
//
// Both channels of a rotated pair belong to one lane: eight neighbours when pairs
// are neighbours (16-byte accesses), and when they are halves of the span, four
// of the first half and their four partners (8-byte accesses at bf16, still 256
// bytes in a row per warp).  Halves that do not consist of whole groups of four
// channels exchange partners through shared memory (word (c mod 8) * D/8 + c / 8 for
// channel c: a lane's eight words and its partners' lie in different banks).
//
// Measured (GB300, L2 cold, 6.8 TB/s copy peak): 8192 tokens x 64 heads of 512,
// bf16: 175-177 us (a copy of the same bytes 167), 65,536 x 24 of 128: 142-146 us
// (copy 125).  Loading the angles per row instead of per token: 205-273 and 179-198.
#include <cstdint>

#include "ckv_device.cuh"
#include "ckv_launch.h"
#include "ckv_launch_util.cuh"

namespace ckv {
namespace {

constexpr int kNormThreads = 256;
constexpr uint32_t kNormShare = 32;  // heads of a token that a warp takes at most
enum Rotation { kNone, kPairs, kHalves, kOddHalves };

// Blocks per SM: two, because 128 registers hold everything.  (With three and a few
// spilled registers 8192 x 64 rows of 512 took 220-257 us instead of 173-177.)
constexpr int kNormBlocks = 2;

// Two fp32 values for the packed instructions (each half an ordinary IEEE operation).
struct Two {
  uint64_t v;
  __device__ __forceinline__ Two() {}
  __device__ __forceinline__ Two(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ void get(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

__device__ __forceinline__ void widen(uint4 x, uint4 y, bool f32, Two (&v)[4]) {
  if (f32) {
    v[0] = Two(__uint_as_float(x.x), __uint_as_float(x.y)), v[1] = Two(__uint_as_float(x.z), __uint_as_float(x.w));
    v[2] = Two(__uint_as_float(y.x), __uint_as_float(y.y)), v[3] = Two(__uint_as_float(y.z), __uint_as_float(y.w));
  } else {
    v[0] = Two(bf16_lo(x.x), bf16_hi(x.x)), v[1] = Two(bf16_lo(x.y), bf16_hi(x.y));
    v[2] = Two(bf16_lo(x.z), bf16_hi(x.z)), v[3] = Two(bf16_lo(x.w), bf16_hi(x.w));
  }
}

template <bool kSplit>
__device__ __forceinline__ void store_row(const ckv_norm_rows& m, int64_t at, const int (&base)[2], const float (&v)[8]) {
  if (m.out_dtype == CKV_F32) {
    float* o = static_cast<float*>(m.out) + at;
    *reinterpret_cast<float4*>(o + base[0]) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(o + base[1]) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint16_t* o = static_cast<uint16_t*>(m.out) + at;
    const uint4 x = make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
    if constexpr (kSplit) {
      *reinterpret_cast<uint2*>(o + base[0]) = make_uint2(x.x, x.y);
      *reinterpret_cast<uint2*>(o + base[1]) = make_uint2(x.z, x.w);
    } else {
      *reinterpret_cast<uint4*>(o + base[0]) = x;
    }
  }
}

// Heads h0 .. h1 - 1 of token t of one set, by one warp.  The lane's channels are
// base[g][0] + 0..3 and base[g][1] + 0..3.
template <int D, Rotation kRot, bool kF32>
__device__ __forceinline__ void norm_heads(const NormRopeArgs& a, const ckv_norm_rows& m, uint32_t t, uint32_t h0, uint32_t h1,
                                           float* s_row) {
  constexpr int kLanes = D >= 256 ? 32 : D / 8;  // of a row
  constexpr int kRows = 32 / kLanes;             // rows of a warp
  constexpr int kGroups = D / (kLanes * 8);
  constexpr int kMost = (D == 512 ? 2 : 4) / (kRot == kOddHalves ? 2 : 1) / (kF32 ? 2 : 1);
  constexpr int kBatch = kMost < 1 ? 1 : kMost;  // rows of a lane in work, and as many in flight (registers)
  const int sl = (threadIdx.x & 31) % kLanes, sub = (threadIdx.x & 31) / kLanes;
  const int half = a.rope_dim >> 1;
  int base[kGroups][2];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int q = g * 32 + sl;  // of D/8
    base[g][0] = q * 8;
    base[g][1] = q * 8 + 4;
    if constexpr (kRot == kHalves) {
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
  struct Rows {
    uint4 raw[kBatch][kGroups][kF32 ? 2 : 1];
  };
  const int64_t in0 = static_cast<int64_t>(t) * m.stride_t;
  auto load = [&](Rows& x, uint32_t h) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const uint32_t hh = h + b * kRows + sub;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        x.raw[b][g][0] = x.raw[b][g][kF32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
        if (hh < h1) {
          const int64_t in = in0 + hh * m.stride_h;
          if constexpr (kF32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              x.raw[b][g][i] = *reinterpret_cast<const uint4*>(static_cast<const float*>(m.x) + in + base[g][i]);
          } else if constexpr (kRot == kHalves) {
            const uint2 lo = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(m.x) + in + base[g][0]);
            const uint2 hi = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(m.x) + in + base[g][1]);
            x.raw[b][g][0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          } else {
            x.raw[b][g][0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(m.x) + in + base[g][0]);
          }
        }
      }
    }
  };
  const int32_t pos = m.positions[t];
  Rows cur, next;
  load(cur, h0);
  if (pos < 0) return;
  if (kRot != kNone && pos >= a.num_positions) {
    if (sl == 0) flag_error(a.err, CKV_DEVERR_SEQ_LEN);
    return;
  }
  const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rope_dim;
  // angles of the lane's pairs, and which of them lie in the span (a bit each; the others stay as they are)
  uint32_t in_span[kGroups];
  constexpr int kA = kRot == kOddHalves ? 4 : 2;
  Two c2[kGroups][kA], s2[kGroups][kA], w[kGroups][4];
  int mate[kGroups][kRot == kOddHalves ? 8 : 1];  // where the partner of each channel lies in s_row
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    in_span[g] = 0;
    if constexpr (kRot == kPairs) {
      float co[4], si[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = base[g][0] + 2 * j - a.rope_offset;
        const bool in = k >= 0 && k < a.rope_dim;
        in_span[g] |= in ? 1u << j : 0u;
        co[j] = in ? cs[k >> 1] : 1.f;
        si[j] = in ? cs[half + (k >> 1)] : 0.f;
      }
      c2[g][0] = Two(co[0], co[1]), c2[g][1] = Two(co[2], co[3]);
      s2[g][0] = Two(si[0], si[1]), s2[g][1] = Two(si[2], si[3]);
    } else if constexpr (kRot == kHalves) {
      float4 co = make_float4(1.f, 1.f, 1.f, 1.f), si = make_float4(0.f, 0.f, 0.f, 0.f);
      if ((g * 32 + sl) * 8 < a.rope_dim) {
        const int p = base[g][0] - a.rope_offset;
        in_span[g] = 1;
        co = *reinterpret_cast<const float4*>(cs + p);
        si = *reinterpret_cast<const float4*>(cs + half + p);
      }
      c2[g][0] = Two(co.x, co.y), c2[g][1] = Two(co.z, co.w);
      s2[g][0] = Two(si.x, si.y), s2[g][1] = Two(si.z, si.w);
    } else if constexpr (kRot == kOddHalves) {
      float co[8], si[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = base[g][0] + j, k = c - a.rope_offset;
        const bool in = k >= 0 && k < a.rope_dim, second = k >= half;
        const int p = second ? k - half : k, o = !in ? c : second ? c - half : c + half;
        co[j] = in ? cs[p] : 1.f;
        si[j] = !in ? 0.f : second ? cs[half + p] : -cs[half + p];
        mate[g][j] = (o & 7) * (D / 8) + (o >> 3);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c2[g][j] = Two(co[2 * j], co[2 * j + 1]);
        s2[g][j] = Two(si[2 * j], si[2 * j + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = m.weight ? *reinterpret_cast<const float4*>(m.weight + base[g][i]) : make_float4(1.f, 1.f, 1.f, 1.f);
      w[g][2 * i] = Two(f.x, f.y);
      w[g][2 * i + 1] = Two(f.z, f.w);
    }
  }
  const int64_t out0 = static_cast<int64_t>(t) * m.out_stride_t;
  for (uint32_t h = h0; h < h1; h += kBatch * kRows) {
    if (h + kBatch * kRows < h1) load(next, h + kBatch * kRows);
    float inv[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      Two sum(0.f, 0.f);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        Two v[4];
        widen(cur.raw[b][g][0], cur.raw[b][g][kF32 ? 1 : 0], kF32, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = fma(v[j], v[j], sum);
      }
      float lo, hi;
      sum.get(lo, hi);
      inv[b] = lo + hi;
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) inv[b] += __shfl_xor_sync(0xFFFFFFFFu, inv[b], o);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) inv[b] = rsqrtf(inv[b] * (1.f / D) + a.eps);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const uint32_t hh = h + b * kRows + sub;
      const int64_t out = out0 + hh * m.out_stride_h;
      const Two scale(inv[b], inv[b]);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        Two z[4];
        widen(cur.raw[b][g][0], cur.raw[b][g][kF32 ? 1 : 0], kF32, z);
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = mul(mul(z[j], scale), w[g][j]);
        if (kRot == kPairs && in_span[g]) {  // z[j] = (x, y): (x, y) c + (-y, x) s
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x, y, c[2], si[2];
            z[j].get(x, y);
            c2[g][j >> 1].get(c[0], c[1]);
            s2[g][j >> 1].get(si[0], si[1]);
            const Two turned = fma(z[j], Two(c[j & 1], c[j & 1]), mul(Two(-y, x), Two(si[j & 1], si[j & 1])));
            if ((in_span[g] >> j) & 1) z[j] = turned;
          }
        } else if (kRot == kHalves && in_span[g]) {  // z[j], z[2 + j] = two x and their two y
          const Two minus(-1.f, -1.f);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const Two x = z[j], y = z[2 + j];
            z[j] = fma(x, c2[g][j], mul(mul(y, minus), s2[g][j]));
            z[2 + j] = fma(y, c2[g][j], mul(x, s2[g][j]));
          }
        }
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j].get(v[2 * j], v[2 * j + 1]);
        if constexpr (kRot == kOddHalves) {
#pragma unroll
          for (int j = 0; j < 8; ++j) s_row[j * (D / 8) + (base[g][0] >> 3)] = v[j];
        } else if (hh < h1) {
          store_row<kRot == kHalves>(m, out, base[g], v);
        }
      }
      if constexpr (kRot == kOddHalves) {
        __syncwarp();
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int own = base[g][0] >> 3;
            const Two x(s_row[2 * j * (D / 8) + own], s_row[(2 * j + 1) * (D / 8) + own]);
            const Two o(s_row[mate[g][2 * j]], s_row[mate[g][2 * j + 1]]);
            fma(x, c2[g][j], mul(o, s2[g][j])).get(v[2 * j], v[2 * j + 1]);
          }
          if (hh < h1) store_row<false>(m, out, base[g], v);
        }
        __syncwarp();
      }
    }
    cur = next;
  }
}

template <int D, Rotation kRot>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a, uint32_t share) {
  constexpr int kRows = D >= 256 ? 1 : 256 / D;  // of a warp
  __shared__ float s_rows[kRot == kOddHalves ? kNormThreads / 32 * kRows : 1][kRot == kOddHalves ? D : 1];
  const int warp = threadIdx.x >> 5, sub = (threadIdx.x & 31) / (32 / kRows);
  float* s_row = s_rows[kRot == kOddHalves ? warp * kRows + sub : 0];
  pdl_wait();
  // a unit is `share` heads of a token
  const uint32_t per_q = (a.set[0].heads + share - 1) / share, per_k = (a.set[1].heads + share - 1) / share;
  const uint32_t units_q = static_cast<uint32_t>(a.set[0].tokens) * per_q;
  const uint32_t units = units_q + static_cast<uint32_t>(a.set[1].tokens) * per_k;
  const uint32_t step = gridDim.x * (kNormThreads / 32);
  for (uint32_t u = blockIdx.x * (kNormThreads / 32) + warp; u < units; u += step) {
    const ckv_norm_rows& m = a.set[u >= units_q];
    const uint32_t i = u < units_q ? u : u - units_q, per = u < units_q ? per_q : per_k;
    const uint32_t t = i / per, h0 = (i - t * per) * share, h1 = min(h0 + share, static_cast<uint32_t>(m.heads));
    if (m.dtype == CKV_F32) norm_heads<D, kRot, true>(a, m, t, h0, h1, s_row);
    else norm_heads<D, kRot, false>(a, m, t, h0, h1, s_row);
  }
}

template <int D, Rotation kRot>
cudaError_t launch_rot(const NormRopeArgs& a, bool use_pdl, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int64_t most = static_cast<int64_t>(sms) * kNormBlocks;
  // as many heads of a token to a warp as leaves every resident warp two units
  int64_t units = 0;
  uint32_t share = kNormShare;
  for (; share >= 1; share /= 2) {
    units = 0;
    for (const ckv_norm_rows& m : a.set) units += m.tokens * ((m.heads + share - 1) / share);
    if (units >= 2 * most * (kNormThreads / 32) || share == 1) break;
  }
  const int64_t want = (units + kNormThreads / 32 - 1) / (kNormThreads / 32);
  return launch_ex(norm_rope_kernel<D, kRot>, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kNormThreads), 0, use_pdl, s,
                   a, share);
}

template <int D>
cudaError_t launch_d(const NormRopeArgs& a, bool use_pdl, cudaStream_t s) {
  if (a.rope_dim == 0) return launch_rot<D, kNone>(a, use_pdl, s);
  if (a.interleaved) return launch_rot<D, kPairs>(a, use_pdl, s);
  // halves of whole groups of four channels, and cos | sin rows that 16-byte loads can start in
  const bool whole = a.rope_offset % 4 == 0 && a.rope_dim % 8 == 0 && reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0;
  return whole ? launch_rot<D, kHalves>(a, use_pdl, s) : launch_rot<D, kOddHalves>(a, use_pdl, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int D, bool use_pdl, cudaStream_t s) {
  return D == 128 ? launch_d<128>(a, use_pdl, s) : D == 256 ? launch_d<256>(a, use_pdl, s) : launch_d<512>(a, use_pdl, s);
}

}  // namespace ckv
