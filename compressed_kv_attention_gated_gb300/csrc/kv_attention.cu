// kv_attention.cu -- attention over the uncompressed paged cache (no counterpart in the
// sources).
#include "kv_attention.cuh"

namespace ckv {
namespace {

constexpr int kWarps = 4, kHeads = 4;  // query heads that a warp works on together

// One CTA per token and key head, its warps taking the rows by turns.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_attention_kernel(const __grid_constant__ KvAttentionArgs a) {
  constexpr int kCh = D / 32;  // channels of a lane
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ __align__(16) float s_o[kWarps][kHeads][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t t = blockIdx.x, kh = blockIdx.y;
  pdl_wait();
  int32_t b = 0;
  for (int32_t n = a.B; n > 1;) {
    const int32_t step = (n + 31) / 32, i = lane * step;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, i < n && kv_start_of(a, b + i) <= t);
    const int32_t last = m ? 31 - __clz(m) : 0;
    b += last * step;
    n = min(step, n - last * step);
  }
  if (t >= kv_start_of(a, b + 1) || t < kv_start_of(a, b)) return;
  const Seen s = seen_by(a, t);
  if (s.c < 0) return;
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.table_stride;
  for (int g0 = 0; g0 < a.G; g0 += kHeads) {
    float q[kHeads][kCh], o[kHeads][kCh], m[kHeads], l[kHeads];
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
      const uint16_t* from = a.q + t * a.q_st + (kh * a.G + min(g0 + g, a.G - 1)) * a.q_sh + lane * kCh;
#pragma unroll
      for (int x = 0; x < kCh; ++x) {
        q[g][x] = __uint_as_float(static_cast<uint32_t>(from[x]) << 16);
        o[g][x] = 0.f;
      }
      m[g] = kNegBig;
      l[g] = 0.f;
    }
    for (int32_t i = warp; i < s.end - s.low + s.first; i += kWarps) {
      const int32_t j = i < s.first ? i : s.low + i - s.first;
      if (j >= s.c && !((a.mask[static_cast<int64_t>(t) * a.words + (j - s.c) / 64] >> ((j - s.c) & 63)) & 1)) continue;
      const int32_t pg = a.page_shift >= 0 ? j >> a.page_shift : j / a.cache.page_size, row = j - pg * a.cache.page_size;
      const int32_t page = table[pg];
      if (page < 0 || page >= a.cache.num_pages) {
        if (lane == 0) flag_error(a.err, CKV_DEVERR_CACHE_LOC);
        continue;
      }
      const uint16_t* k = a.cache.k + page * a.cache.k_stride_page + row * a.cache.k_stride_row + kh * a.cache.k_stride_head + lane * kCh;
      const uint16_t* v = a.cache.v + page * a.cache.v_stride_page + row * a.cache.v_stride_row + kh * a.cache.v_stride_head + lane * kCh;
      float kv[kCh], z[kHeads];
#pragma unroll
      for (int x = 0; x < kCh; ++x) kv[x] = __uint_as_float(static_cast<uint32_t>(k[x]) << 16);
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        z[g] = 0.f;
#pragma unroll
        for (int x = 0; x < kCh; ++x) z[g] = fmaf(q[g][x], kv[x], z[g]);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
#pragma unroll
        for (int g = 0; g < kHeads; ++g) z[g] += __shfl_xor_sync(0xFFFFFFFFu, z[g], d);
      }
#pragma unroll
      for (int x = 0; x < kCh; ++x) kv[x] = __uint_as_float(static_cast<uint32_t>(v[x]) << 16);
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        const float y = z[g] * (a.softmax_scale * kLog2e), top = fmaxf(m[g], y);
        const float keep = fast_exp2(m[g] - top), w = fast_exp2(y - top);
        m[g] = top;
        l[g] = l[g] * keep + w;
#pragma unroll
        for (int x = 0; x < kCh; ++x) o[g][x] = fmaf(w, kv[x], o[g][x] * keep);
      }
    }
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
      if (lane == 0) s_m[warp][g] = m[g], s_l[warp][g] = l[g];
#pragma unroll
      for (int x = 0; x < kCh; ++x) s_o[warp][g][lane * kCh + x] = o[g][x];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kHeads * D; i += kWarps * 32) {
      const int g = i / D, ch = i % D;
      if (g0 + g < a.G) {
        const int h = kh * a.G + g0 + g;
        float top = a.sink ? a.sink[h] * kLog2e : kNegBig, all = 0.f, acc = 0.f;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_l[w][g] > 0.f ? s_m[w][g] : kNegBig);
        for (int w = 0; w < kWarps; ++w) {
          if (s_l[w][g] == 0.f) continue;
          const float x = fast_exp2(s_m[w][g] - top);
          all += s_l[w][g] * x;
          acc += s_o[w][g][ch] * x;
        }
        if (a.sink) all += fast_exp2(a.sink[h] * kLog2e - top);
        const int64_t flat = static_cast<int64_t>(t) * a.H + h;
        a.out[flat * D + ch] = __bfloat16_as_ushort(__float2bfloat16_rn(all == 0.f ? 0.f : acc / all));
        if (a.lse && ch == 0) a.lse[flat] = all == 0.f ? -INFINITY : (top + log2f(all)) * kKvLn2;
      }
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t launch(const KvAttentionArgs& a, bool use_pdl, cudaStream_t s) {
  return launch_ex(kv_attention_kernel<D>, dim3(static_cast<unsigned>(a.T), a.KH), dim3(kWarps * 32), 0, use_pdl, s, a);
}

}  // namespace

int64_t kv_attention_workspace(int64_t, int32_t, int32_t, int32_t, int32_t, int64_t, int32_t, int32_t, int32_t) { return 0; }

cudaError_t launch_kv_attention(const KvAttentionArgs& a, bool use_pdl, cudaStream_t s) {
  return a.cache.D == 128 ? launch<128>(a, use_pdl, s) : a.cache.D == 256 ? launch<256>(a, use_pdl, s) : launch<512>(a, use_pdl, s);
}

}  // namespace ckv
