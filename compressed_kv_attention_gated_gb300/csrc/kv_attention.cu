// kv_attention.cu -- attention over the uncompressed paged cache (no counterpart in the
// sources):
//   z_j = scale <q, k_j>,  lse = log(sum_j e^z_j [+ e^sink]),  out = sum_j e^(z_j - lse) v_j
// over the rows j that a token sees: those of its window, the first ones, its drafts.
//
// The (token, head) rows that share a key head are cut into tiles, the M side of both products, which
// run on the tensor cores:
//   S [128 rows x 128 keys] = Q [128 x D] K^T        O [128 rows x D] += P [128 x 128 keys] V
// This is the form for more than 64 rows to a request and key head at D = 128 and 256; fewer, and
// D = 512, are in kv_attention_few.cu.  A tile's keys are the rows that any of its tokens sees: the
// first ones, then those from the lowest window to the last row, cut into 128s as one list, so that a
// window of 128 is one tile of keys wherever it begins.  What single tokens do not see of it is masked.
//
// A job is a tile of rows with its keys (or a range of them); the launch has a CTA for each, and those
// that are resident, one per SM, take over the others (take_job()).  Roles of a CTA: softmax warps, 8 with a
// thread per row of S at D = 128, 16 at D = 256; one thread that issues the products, two at D = 128; one warp that looks up the
// jobs ahead of the others; 4 that copy queries, keys and values (cp.async, 16 bytes at a time: pages
// begin anywhere in a tile and rows have any stride; TMA's gathered rows took 88 clocks per 512 bytes)
// into a ring of units of 128 rows x 128 channels, across the jobs, so that memory is busy while a job
// ends.
//
// D = 128: each group of four softmax warps has its own S and O, and a thread that issues its products.
// With more than 128 rows it has a tile of its own, and keys and values serve both; otherwise the groups
// take the tiles of keys by turns and join their outputs in the end.  One group's softmax runs under the
// other's products, and tiles of keys go through in halves.  D = 256: O has room for one tile; the groups
// take tiles of keys by turns and share it and the references of its rows.
//
// Softmax: weights are taken against a reference, the maximum of the tile that set it, which moves only
// when a weight exceeds 2^16 (D = 128: the sum of a half's); then O is rescaled.  The weights are rounded to
// bf16, the type of the values that they multiply (by 2^-8 of their value at most); sums are of unrounded
// ones, in fp32, as are scores and outputs.
//
// Few tiles with many keys are split into ranges of keys; their results (fp32, and lse) go through
// the workspace and are joined by a second kernel in a fixed order.
//
// Measured: 9 prompts of 600 to 3000 tokens x 32 heads (8 key heads, D = 128, window 1024) 286 us, 965 TFLOP/s
// without the masked parts; 128 drafts of 40 to 64 tokens over up to 4096 rows 255 us (247 to 272 from run to run), 4.75 TB/s.  The tensor cores are
// busy 49 and 53% of the time, instructions issue in 44 and 40% of the cycles, exponentials take 24%.  A softmax warp of the
// prompts spends, of 39 k clocks on a job of 9 tiles of keys, 10 on exponentials and their rounding, 8 on scaling and
// masks, 4.4 waiting for scores, 3 on the output, 4 on the next job's rows and on sums, and about 5 on getting its
// instructions: loops are not unrolled for that.  Twice as many softmax warps (16 rows to a warp, four lanes to a row)
// take as long (304 us when this took 290), with whole tiles of scores to a product longer (335).
#include <algorithm>

#include "kv_attention.cuh"

namespace ckv {
namespace {

constexpr float kKvMost = 65536.f;  // D = 128: sum of a tile's weights from which on the reference moves

template <int D_>
struct KvLayout {
  static constexpr int D = D_;
  static constexpr int kRows = D == 128 ? 256 : 128;    // of a job
  static constexpr int kSoftWarps = D == 128 ? 8 : 16;
  static constexpr int kMmaWarp = kSoftWarps, kPlanWarp = kSoftWarps + 1, kMmaWarp2 = kSoftWarps + 2, kCopyWarp = kSoftWarps + 4;
  static constexpr int kThreads = (kSoftWarps + 8) * 32;
  // registers per thread: 512 x 128 at launch, then 256 x 192 + 256 x 64; 768 x 80, then 512 x 88 + 256 x 64, the same
  static constexpr int kSoftRegs = D == 128 ? 192 : 88, kOtherRegs = 64;
  static constexpr int kKU = D / 128;                   // units of a tile's keys, and of its values
  static constexpr bool kFindMissing = true;            // pages that are not there, by the planning warp
  static constexpr int kQRows = 128;                    // of a slot of queries
  static constexpr int kQBlock = kQRows * 128;          // 64 channels of them
  static constexpr int kQSlot = kQBlock * (D / 64);
  static constexpr int kQSlots = D == 128 ? 2 : 1;
  static constexpr int kRing = 5;
  static constexpr int kUnits = kQSlots * kQSlot;  // where the ring begins, behind the queries
  static constexpr int kSmall = kUnits + kRing * kKvUnit;
  static constexpr int kTmemO = 0, kTmemS = 256;  // O: 256 columns; S: two buffers of 128, P over the first half of each
};

// Beside the common ones (o_full[w] and pv_done[w] are group w's; at D = 256 s_full[w] and p_full[w] too, p_full of 8 warps):
template <int D>
struct KvSmall : KvCommon {
  uint64_t decided[2][8];         // D = 256: warp i of group w knows the references under which its tile is taken
  uint64_t half_s[2][2], half_p[2][2];  // D = 128: scores and weights of group w, by halves of a tile of keys (4 warps)
  uint64_t met;                   // both groups have got there: all softmax warps, twice per job of shared rows
  float ref[D == 128 ? 2 : 1][128];  // references of shared rows (each group's own at D = 128)
  float sum[2][128];
};

template <int D>
constexpr int kv_smem_bytes() {
  return KvLayout<D>::kSmall + static_cast<int>(sizeof(KvSmall<D>));
}
static_assert(kv_smem_bytes<128>() <= 227 * 1024 && kv_smem_bytes<256>() <= 227 * 1024, "shared memory");

// 32 columns of the warp's lanes; the values are there after tc_wait_ld() and settled32().
__device__ __forceinline__ void tmem_ld32_async(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr));
}
// Arithmetic on loaded values may not be moved over the wait: here they change as far as the compiler knows.
__device__ __forceinline__ void settled32(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
               "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
  asm volatile("" : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
               "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void kv_tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Bits x0 .. x1 - 1 of a 32-bit word (any of them outside it).
__device__ __forceinline__ uint32_t bits_between(int32_t x0, int32_t x1) {
  const int32_t lo = max(x0, 0);
  uint32_t m;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(lo), "r"(max(x1 - lo, 0)));
  return m;
}

// Two fp32 values for the packed instructions (each half an ordinary IEEE operation).
__device__ __forceinline__ void fma2(float& x, float& y, uint64_t scale, uint64_t shift) {
  asm("{\n .reg .b64 v;\n mov.b64 v, {%0, %1};\n fma.rn.f32x2 v, v, %2, %3;\n mov.b64 {%0, %1}, v;\n}\n" : "+f"(x), "+f"(y) : "l"(scale), "l"(shift));
}
__device__ __forceinline__ void add2(float& x, float& y, float p, float q) {
  asm("{\n .reg .b64 v, w;\n mov.b64 v, {%0, %1};\n mov.b64 w, {%2, %3};\n add.rn.f32x2 v, v, w;\n mov.b64 {%0, %1}, v;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(p), "f"(q));
}
__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %1};" : "=l"(v) : "f"(x));
  return v;
}

// A softmax thread's row: what it sees, in places of the job's list of keys.
struct SoftRow {
  int32_t flat, t;         // (token, head) index, -1: none; token
  int32_t a1, b0, b1, b2;  // places 0 .. a1 - 1 and b0 .. b1 - 1, and of the drafts' from b1 to b2 - 1 those with a bit
};

__device__ __forceinline__ SoftRow soft_row(const KvAttentionArgs& a, const Job& job, int32_t i) {
  SoftRow x{-1, 0, 0, 0, 0, 0};
  if (i < job.tile.rows) {
    const int32_t r = job.tile.base + i, tok = r / a.G;
    x.t = job.tile.tok0 + tok;
    const Seen s = seen_by(a, x.t);
    if (s.c >= 0) {
      x.flat = x.t * a.H + job.kh * a.G + r - tok * a.G;
      const int32_t at = job.first - job.low;  // a row's place over its number, behind the first rows
      x.a1 = s.first > job.low ? s.first + at : min(job.first, s.c);
      x.b0 = max(s.low + at, job.first);
      x.b1 = s.c + at;
      x.b2 = s.end + at;
    }
  }
  return x;
}

// The spans of n keys from place v0 on that every row of the warp sees whole: the first a of them, and those from b0
// to b1 - 1.  (Rows without a token do not count.)
struct WholeSpans {
  int32_t a, b0, b1;
  __device__ __forceinline__ bool operator()(int32_t i) const { return i < a || (i >= b0 && i < b1); }
};
template <int n>
__device__ __forceinline__ WholeSpans whole_spans(const SoftRow& x, const SoftRow& y, int32_t v0, int32_t v1, bool missing) {  // two rows a thread
  auto least = [&](int32_t p, int32_t q) { return __reduce_min_sync(0xFFFFFFFFu, min(x.flat >= 0 ? p : INT32_MAX, y.flat >= 0 ? q : INT32_MAX)); };
  const int32_t a1 = min(least(x.a1, y.a1), v1) - v0, b1 = min(least(x.b1, y.b1), v1) - v0;
  const int32_t b0 = __reduce_max_sync(0xFFFFFFFFu, max(x.flat >= 0 ? x.b0 : 0, y.flat >= 0 ? y.b0 : 0)) - v0;
  return missing ? WholeSpans{0, 0, 0} : WholeSpans{a1 / n, b0 > 0 ? (b0 + n - 1) / n : 0, b1 / n};
}

// Which of n keys (places v .. v + n - 1, v1 the list's end) the row sees, a bit each.
template <int n>
__device__ __forceinline__ void tile_bits(const KvAttentionArgs& a, const SoftRow& x, const Job& job, int32_t v, int32_t v1, bool missing,
                                          uint32_t (&bits)[n / 32]) {
#pragma unroll
  for (int i = 0; i < n / 32; ++i) {
    const int32_t y = v + i * 32;
    uint32_t m = bits_between(0, min(x.a1, v1) - y) | bits_between(x.b0 - y, min(x.b1, v1) - y);
    if (a.words > 0 && y + 32 > x.b1 && y < x.b2) {  // 32 bits of the drafts' mask, from bit y - b1 on
      const int32_t d = y - x.b1, at = d >> 5;       // rounded down
      const uint32_t* words = reinterpret_cast<const uint32_t*>(a.mask + static_cast<int64_t>(x.t) * a.words);
      const uint32_t lo = at >= 0 && at < 2 * a.words ? words[at] : 0u, hi = at + 1 >= 0 && at + 1 < 2 * a.words ? words[at + 1] : 0u;
      m |= __funnelshift_r(lo, hi, d & 31) & bits_between(0, min(x.b2, v1) - y);
    }
    bits[i] = m;
  }
  if (missing) {  // keys whose page is not there, a lane each
    const int32_t* table = a.table + static_cast<int64_t>(job.tile.b) * a.table_stride;
    uint32_t missed = 0;
#pragma unroll
    for (int i = 0; i < n / 32; ++i) {
      const int32_t y = v + i * 32 + (threadIdx.x & 31), key = y < job.first ? y : job.low + y - job.first;
      const uint32_t gone = __ballot_sync(0xFFFFFFFFu, y < v1 && !kv_page_there(a, table[kv_page_of(a, key)]));
      missed |= bits[i] & gone;
      bits[i] &= ~gone;
    }
    if (missed && x.flat >= 0) flag_error(a.err, CKV_DEVERR_CACHE_LOC);
  }
}

template <int n>
__device__ __forceinline__ float largest(const float* z) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < n; ++i) top[i % 4] = fmaxf(top[i % 4], z[i]);
  return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}

// n scores of the row in log2 units over its reference; -infinity for what it does not see.
template <int n>
__device__ __forceinline__ void over_reference(float* z, uint64_t scale, uint64_t shift, bool masks, const uint32_t* bits) {
#pragma unroll
  for (int i = 0; i < n; i += 2) fma2(z[i], z[i + 1], scale, shift);
  if (__builtin_expect(masks, 0)) {
#pragma unroll
    for (int i = 0; i < n; ++i) z[i] = (bits[i / 32] >> (i % 32)) & 1 ? z[i] : -INFINITY;
  }
}

// Their weights, rounded to bf16, to tensor memory as A of the second product; returns the sum.
template <int n>
__device__ __forceinline__ float weights(const float* z, uint32_t at) {
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
  for (int i = 0; i < n / 32; ++i) {
    uint32_t x[16];
#pragma unroll
    for (int y = 0; y < 32; y += 4) {
      const float p0 = fast_exp2(z[i * 32 + y]), p1 = fast_exp2(z[i * 32 + y + 1]);
      const float p2 = fast_exp2(z[i * 32 + y + 2]), p3 = fast_exp2(z[i * 32 + y + 3]);
      add2(s0, s1, p0, p1);
      add2(s2, s3, p2, p3);
      x[y / 2] = pack_bf16x2_rn(p0, p1);
      x[y / 2 + 1] = pack_bf16x2_rn(p2, p3);
    }
    kv_tmem_st16(at + i * 16, x);
  }
  return (s0 + s1) + (s2 + s3);
}

// Columns of O times what a move of the rows' references leaves.
template <int kColumns>
__device__ __forceinline__ void rescale(uint32_t at, float keep) {
#pragma unroll 1
  for (int i = 0; i < kColumns; i += 16) {
    float o[16];
    tmem_ld<16>(at + i, o);
    uint32_t x[16];
#pragma unroll
    for (int y = 0; y < 16; ++y) x[y] = __float_as_uint(o[y] * keep);
    kv_tmem_st16(at + i, x);
  }
  tc_wait_st();
}

// Sum and reference of a row -> the scale of its output; stores lse (of the range when the row is split).
__device__ __forceinline__ float finish_row(const KvAttentionArgs& a, const KvPlan& p, int D, int32_t range, int32_t flat, float all, float m, bool tell) {
  const bool none = all == 0.f, split = p.splits > 1;
  float keep = 1.f, sink = -INFINITY;
  if (a.sink && !split && flat >= 0) {
    sink = a.sink[flat % a.H];
    const float s = sink * kLog2e, high = fmaxf(none ? kNegBig : m, s);
    keep = none ? 0.f : fast_exp2(m - high);
    all = (none ? 0.f : all * keep) + (s == high ? 1.f : fast_exp2(s - high));
    m = high;
  }
  if (flat >= 0 && tell) {
    // nothing at all: no sink, or one that is -infinity in log2 units
    const float lse = all == 0.f ? sink : (m + log2f(all)) * kKvLn2;
    if (split) static_cast<float*>(a.workspace)[a.T * a.H * (p.splits * D + static_cast<int64_t>(range)) + flat] = lse;
    else if (a.lse) a.lse[flat] = lse;
  }
  return none ? 0.f : keep / all;
}

// 32 channels from `ch` on of a row, in whole sectors where its beginning allows that.
__device__ __forceinline__ void put_row(const KvAttentionArgs& a, const KvPlan& p, int D, int32_t range, int32_t flat, int ch, const float (&o)[32]) {
  if (flat < 0) return;
  if (p.splits > 1) {
    float4* to = reinterpret_cast<float4*>(static_cast<float*>(a.workspace) + (a.T * a.H * static_cast<int64_t>(range) + flat) * D + ch);
#pragma unroll
    for (int x = 0; x < 8; ++x) to[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
    return;
  }
  uint32_t x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = pack_bf16x2_rn(o[2 * i], o[2 * i + 1]);
  uint16_t* to = a.out + static_cast<int64_t>(flat) * D + ch;
  if (reinterpret_cast<uintptr_t>(a.out) % 32 == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + i * 16), "r"(x[8 * i]), "r"(x[8 * i + 1]), "r"(x[8 * i + 2]),
                   "r"(x[8 * i + 3]), "r"(x[8 * i + 4]), "r"(x[8 * i + 5]), "r"(x[8 * i + 6]), "r"(x[8 * i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(to + i * 8) = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}

// The part of the softmax warps at D = 128: every group has an output of its own.
__device__ __forceinline__ bool soft_apart(const KvAttentionArgs& a, const KvPlan& p, KvSmall<128>& sm, uint32_t tmem) {
  using L = KvLayout<128>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, w = warp >> 2, row = threadIdx.x & 127;
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t at_s = tmem + lanes + L::kTmemS + w * 128, at_o = tmem + lanes + L::kTmemO + w * 128;
  const uint64_t scale = twice(a.softmax_scale * kLog2e);
  uint32_t use = 0, met_use = 0;    // tiles of keys of the group, ...
  uint32_t o_use[2] = {0, 0};       // jobs in which a group had a tile of keys
#pragma unroll 1
  for (uint32_t job_use = 0;; ++job_use) {
    if (!warp_wait(&sm.job_full[job_use & 1], job_use >> 1)) return false;
    const Job& job = sm.job[job_use & 1];
    if (!job.live) return true;
    const bool two = job.two;  // a tile of rows of its own; otherwise the groups take tiles of keys of the same rows by turns
    const int32_t n = job.n, v0 = job.v0, v1 = job.v1, range = job.split;
    const bool missing = job.missing;
    const SoftRow x = soft_row(a, job, (two ? w * 128 : 0) + row);
    const bool any = __any_sync(0xFFFFFFFFu, x.flat >= 0);
    const WholeSpans whole = whole_spans<64>(x, x, v0, v1, missing);
    float ref = x.flat >= 0 ? kNegBig : 0.f, l = 0.f;  // a row that has seen no key yet has no reference
    uint64_t shift = twice(0.f);                       // -ref, or 0 without one
    bool unset = any;                                  // some row of the warp may have none
    const int j0 = two ? 0 : w, step = two ? 1 : 2;
    // a tile of keys goes through in halves, each with a buffer of scores of its own, so that there are always
    // scores to work on while the products of the other half run
    auto half = [&](int j, int h) {
      uint32_t bits[2];
      const bool masks = any && !whole(2 * j + h);
      bool some = any;  // of the warp's rows see some of the keys
      if (__builtin_expect(masks, 0)) {
        tile_bits<64>(a, x, job, v0 + j * kKvKeys + h * 64, v1, missing, bits);
        some = __any_sync(0xFFFFFFFFu, bits[0] | bits[1]);
      }
      const uint32_t at = at_s + h * 64;
      if (!warp_wait(&sm.half_s[w][h], use)) return false;
      tc_fence_after();
      if (__builtin_expect(any && !some, 0)) {
        uint32_t none[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) none[i] = 0;
        kv_tmem_st16(at, none);
        kv_tmem_st16(at + 16, none);
        tc_wait_st();
      } else if (any) {
        float z[64];
        tmem_ld32_async(at, z);
        tmem_ld32_async(at + 32, z + 32);
        tc_wait_ld();
        settled32(z);
        settled32(z + 32);
        over_reference<64>(z, scale, shift, masks, bits);
        if (__builtin_expect(unset, 0)) {  // the output of a row without a reference is 0: the reference is just set
          const float top = ref == kNegBig ? largest<64>(z) : -INFINITY;
          if (top > -INFINITY) {
            ref = top;
            shift = twice(-top);
#pragma unroll
            for (int i = 0; i < 64; ++i) z[i] -= top;
          }
          unset = __any_sync(0xFFFFFFFFu, ref == kNegBig);
        }
        // weights under the reference as it is; when a row's sum shows that it has grown too old, once more
        float sum = weights<64>(z, at);
        while (__builtin_expect(__any_sync(0xFFFFFFFFu, sum > kKvMost), 0)) {
          const float by = sum > kKvMost ? largest<64>(z) : 0.f, keep = fast_exp2(-by);
          if (sum > kKvMost) {
            ref += by;
            shift = twice(-ref);
          }
          l *= keep;
#pragma unroll
          for (int i = 0; i < 64; ++i) z[i] -= by;
          if (j > j0 || h > 0) {  // the products of the half before
            if (h == 0 && !warp_wait(&sm.half_s[w][1], use)) return false;
            // they came before the scores that were made next: this half's, the next tile's first, or none
            if (h == 1 && !(j + step < n ? warp_wait(&sm.half_s[w][0], use + 1) : warp_wait(&sm.pv_done[w], o_use[w]))) return false;
            tc_fence_after();
            rescale<128>(at_o, keep);
          }
          tc_wait_st();
          sum = weights<64>(z, at);
        }
        l += sum;
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.half_p[w][h]);
      return true;
    };
    for (int j = j0, h = 0; j < n;) {
      if (!half(j, h)) return false;
      j += h ? step : 0;
      use += h;
      h ^= 1;
    }
    // ------------------------------------------------------------------ output
    float all = l, m = ref, mine = 1.f, other = 0.f;  // shares of the two outputs
    if (!two) {
      sm.sum[w][row] = l;
      sm.ref[w][row] = ref;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.met);
      if (!warp_wait(&sm.met, met_use++)) return false;
      const float l1 = sm.sum[w ^ 1][row], m1 = sm.ref[w ^ 1][row];
      m = fmaxf(l == 0.f ? kNegBig : ref, l1 == 0.f ? kNegBig : m1);
      mine = l == 0.f ? 0.f : fast_exp2(ref - m);
      other = l1 == 0.f ? 0.f : fast_exp2(m1 - m);
      all = l * mine + l1 * other;
    }
    const float share = finish_row(a, p, 128, range, x.flat, all, m, two || w == 0);
    mine *= share;
    other *= share;
    // a group without a tile of keys has no products to wait for, and its thread for them could be a job ahead
    if (n > j0 && !warp_wait(&sm.o_full[w], o_use[w])) return false;
    if (!two && n > (w ^ 1) && !warp_wait(&sm.o_full[w ^ 1], o_use[w ^ 1])) return false;
    for (int g = 0; g < 2; ++g) o_use[g] += n > (two ? 0 : g);
    tc_fence_after();
    if (any) {
#pragma unroll 1
      for (int i = two ? 0 : w * 64; i < (two ? 128 : w * 64 + 64); i += 32) {
        float o[32];
        if (n > j0) {
          tmem_ld<32>(at_o + i, o);
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] *= mine;
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0.f;
        }
        if (!two && n > (w ^ 1)) {
          float o1[32];
          tmem_ld<32>(tmem + lanes + L::kTmemO + (w ^ 1) * 128 + i, o1);
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = fmaf(o1[y], other, o[y]);
        }
        put_row(a, p, 128, range, x.flat, i, o);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sm.job_empty[job_use & 1]);
      if (!two) mbar_arrive(&sm.met);
    }
    if (!two && !warp_wait(&sm.met, met_use++)) return false;  // both outputs and the sums are read
  }
}

// 16 lanes of tensor memory, in pieces of 8 columns: a thread has two neighbouring columns, 2 (lane % 4), of rows lane / 4
// and lane / 4 + 8 in each piece (registers 4 i, 4 i + 1 and 4 i + 2, 4 i + 3).
__device__ __forceinline__ void tmem_ld16x64(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr));
  tc_wait_ld();
  settled32(v);
}
__device__ __forceinline__ void tmem_ld16x16(uint32_t addr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
  tc_wait_ld();
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}
__device__ __forceinline__ void tmem_st16x16(uint32_t addr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
// The same rows of 32 columns, in pieces of 4: column lane % 4 of both rows.
__device__ __forceinline__ void tmem_st16x32(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Over the four lanes that have a row.
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
  return x + __shfl_xor_sync(0xFFFFFFFFu, x, 2);
}
// Weights of both rows to tensor memory, rounded to bf16; their sums are added.
__device__ __forceinline__ void weights16(const float* z, uint32_t at, float (&sum)[2]) {
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  uint32_t x[16];
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float p0 = fast_exp2(z[i]), p1 = fast_exp2(z[i + 1]), p2 = fast_exp2(z[i + 2]), p3 = fast_exp2(z[i + 3]);
    add2(s0, s1, p0, p1);
    add2(s2, s3, p2, p3);
    x[i / 2] = pack_bf16x2_rn(p0, p1);
    x[i / 2 + 1] = pack_bf16x2_rn(p2, p3);
  }
  tmem_st16x32(at, x);
  sum[0] = s0 + s1;
  sum[1] = s2 + s3;
}

// Four lanes trade the four words that each has: word i of lane j becomes word j of lane i.
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[4], int lane) {
#pragma unroll
  for (int b = 1; b < 4; b *= 2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & b) continue;
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, lane & b ? x[k] : x[k | b], b);
      if (lane & b) x[k] = got;
      else x[k | b] = got;
    }
  }
}

// 64 channels from `ch` on of a row, which four lanes have (o as of tmem_ld16x64, r: 0 or 1), times `share`.
__device__ __forceinline__ void put_row16(const KvAttentionArgs& a, const KvPlan& p, int D, int32_t range, int32_t flat, int ch, const float (&o)[32], int r,
                                          float share, int lane) {
  if (p.splits > 1) {
    float* to = static_cast<float*>(a.workspace) + (a.T * a.H * static_cast<int64_t>(range) + flat) * D + ch + lane % 4 * 2;
    if (flat >= 0) {
#pragma unroll
      for (int y = 0; y < 8; ++y) *reinterpret_cast<float2*>(to + y * 8) = make_float2(o[4 * y + 2 * r] * share, o[4 * y + 2 * r + 1] * share);
    }
    return;
  }
#pragma unroll
  for (int y = 0; y < 8; y += 4) {  // 32 channels: a lane gets eight that follow each other
    uint32_t x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = pack_bf16x2_rn(o[4 * (y + k) + 2 * r] * share, o[4 * (y + k) + 2 * r + 1] * share);
    quad_transpose(x, lane);
    if (flat >= 0)
      *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(flat) * D + ch + y * 8 + lane % 4 * 8) = make_uint4(x[0], x[1], x[2], x[3]);
  }
}

// Columns of O times what a move of the rows' references leaves.
template <int kColumns>
__device__ __forceinline__ void rescale16(uint32_t at, const float (&keep)[2]) {
#pragma unroll 1
  for (int i = 0; i < kColumns; i += 16) {
    float o[8];
    tmem_ld16x16(at + i, o);
#pragma unroll
    for (int y = 0; y < 8; ++y) o[y] *= keep[y / 2 % 2];
    tmem_st16x16(at + i, o);
  }
  tc_wait_st();
}

// The part of the softmax warps at D = 256: the two groups of eight take tiles of keys by turns and share the output.  Products
// of a group's next tile come behind those of its last one, so its time counts twice over, and it has eight warps: 16 rows to
// a warp, four lanes to a row (8000 tokens x 64 heads over 128 rows 242 us, 32 heads over 1024 rows 310 us; with a row to a
// thread 284 and 321).
__device__ __forceinline__ bool soft_shared(const KvAttentionArgs& a, const KvPlan& p, KvSmall<256>& sm, uint32_t tmem) {
  constexpr int D = 256;
  using L = KvLayout<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = (warp >> 2) & 1, part = (warp & 3) * 2 + (warp >> 3);
  const int row = part * 16 + lane / 4;  // and row + 8
  const uint32_t lanes = static_cast<uint32_t>(part * 16) << 16;
  const uint32_t at_s = tmem + lanes + L::kTmemS + w * 128, at_o = tmem + lanes + L::kTmemO;
  const uint64_t scale = twice(a.softmax_scale * kLog2e);
  uint32_t s_use = 0, o_use = 0, met_use = 0;
  uint32_t other_tiles = 0;  // of the other group so far
#pragma unroll 1
  for (uint32_t job_use = 0;; ++job_use) {
    if (!warp_wait(&sm.job_full[job_use & 1], job_use >> 1)) return false;
    const Job& job = sm.job[job_use & 1];
    if (!job.live) return true;
    const int32_t n = job.n, v0 = job.v0, v1 = job.v1;
    const bool missing = job.missing;
    const SoftRow x[2] = {soft_row(a, job, row), soft_row(a, job, row + 8)};
    const bool any = __any_sync(0xFFFFFFFFu, x[0].flat >= 0 || x[1].flat >= 0);
    const WholeSpans whole = whole_spans<128>(x[0], x[1], v0, v1, missing);
    float ref[2], l[2] = {0.f, 0.f};  // a row that has seen no key yet has no reference
#pragma unroll
    for (int r = 0; r < 2; ++r) ref[r] = x[r].flat >= 0 ? kNegBig : 0.f;
#pragma unroll 1
    for (int j = w; j < n; j += 2) {
      uint32_t bits[2][4];
      const bool masks = any && !whole(j);
      if (masks) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          tile_bits<128>(a, x[r], job, v0 + j * kKvKeys, v1, missing, bits[r]);
#pragma unroll
          for (int i = 0; i < 4; ++i) bits[r][i] >>= lane % 4 * 2;
        }
      }
      if (!warp_wait(&sm.s_full[w], s_use++)) return false;
      tc_fence_after();
      if (any) {
        // scores of half of the tile in log2 units less `less`, -infinity for what a row does not see
        auto scores = [&](int h, float (&z)[32], float less0, float less1) {
          tmem_ld16x64(at_s + h * 64, z);
          const uint64_t s0 = twice(-less0), s1 = twice(-less1);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            fma2(z[i], z[i + 1], scale, s0);
            fma2(z[i + 2], z[i + 3], scale, s1);
          }
          if (__builtin_expect(masks, 0)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t b0 = h ? bits[r][2] : bits[r][0], b1 = h ? bits[r][3] : bits[r][1];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t two = (i < 4 ? b0 : b1) >> (i % 4 * 8);
                if (!(two & 1)) z[4 * i + 2 * r] = -INFINITY;
                if (!(two & 2)) z[4 * i + 2 * r + 1] = -INFINITY;
              }
            }
          }
        };
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float z[32];
          scores(h, z, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            top[0] = fmaxf(top[0], fmaxf(z[i], z[i + 1]));
            top[1] = fmaxf(top[1], fmaxf(z[i + 2], z[i + 3]));
          }
        }
        const uint32_t others = other_tiles + (j + 1) / 2;                                // tiles of the other group before this one
        if (j > 0 && !warp_wait(&sm.decided[w ^ 1][part], others - 1)) return false;  // the references as it left them
        float keep[2];
        bool moves = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = quad_max(top[r]);
          if (j > 0) {
            const float now = sm.ref[0][row + 8 * r];
            if (now != ref[r]) {
              l[r] = l[r] == 0.f ? 0.f : l[r] * fast_exp2(ref[r] - now);
              ref[r] = now;
            }
          }
          const bool unset = ref[r] == kNegBig;
          moves |= unset ? top[r] > -INFINITY : top[r] - ref[r] > kKvJump;
        }
        if (__any_sync(0xFFFFFFFFu, moves)) {  // references go to the largest scores so far
          bool rescales = false;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const bool unset = ref[r] == kNegBig;
            const float now = fmaxf(ref[r], top[r]);
            keep[r] = unset ? 1.f : fast_exp2(ref[r] - now);  // an unset row's output is 0
            l[r] *= keep[r];
            ref[r] = now;
            rescales |= keep[r] != 1.f;
          }
          if (j > 0 && __any_sync(0xFFFFFFFFu, rescales)) {
            if (!warp_wait(&sm.pv_done[w ^ 1], others - 1)) return false;  // the products of the tile before
            tc_fence_after();
            rescale16<D>(at_o, keep);
          }
        }
        if (lane % 4 == 0) {
          sm.ref[0][row] = ref[0];
          sm.ref[0][row + 8] = ref[1];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.decided[w][part]);
        const float less[2] = {ref[0] == kNegBig ? 0.f : ref[0], ref[1] == kNegBig ? 0.f : ref[1]};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float z[32], sum[2];
          scores(h, z, less[0], less[1]);
          weights16(z, at_s + h * 32, sum);
          l[0] += sum[0];
          l[1] += sum[1];
        }
        tc_wait_st();
      } else if (lane == 0) {
        mbar_arrive(&sm.decided[w][part]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[w]);
    }
    // ------------------------------------------------------------------ output
    other_tiles += (n + w) / 2;
    float share[2] = {ref[0], ref[1]};
    if (n > 0) {  // both sums against the references that O has in the end: the last tile's
      if (((n - 1) & 1) != w && !warp_wait(&sm.decided[w ^ 1][part], other_tiles - 1)) return false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        share[r] = any ? sm.ref[0][row + 8 * r] : 0.f;
        l[r] = l[r] == 0.f ? 0.f : l[r] * fast_exp2(ref[r] - share[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] = quad_sum(l[r]);
      if (lane % 4 == 0) sm.sum[w][row + 8 * r] = l[r];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.met);
    if (!warp_wait(&sm.met, met_use++)) return false;
#pragma unroll
    for (int r = 0; r < 2; ++r)
      share[r] = finish_row(a, p, D, job.split, x[r].flat, l[r] + sm.sum[w ^ 1][row + 8 * r], share[r], w == 0 && lane % 4 == 0);
    if (n > 0) {
      if (!warp_wait(&sm.o_full[w], o_use++)) return false;
      tc_fence_after();
    }
    if (any) {
#pragma unroll 1
      for (int i = w * (D / 2); i < (w + 1) * (D / 2); i += 64) {
        float o[32];
        if (n > 0) {
          tmem_ld16x64(at_o + i, o);
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) put_row16(a, p, D, job.split, x[r].flat, i, o, r, n > 0 ? share[r] : 0.f, lane);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sm.job_empty[job_use & 1]);
      mbar_arrive(&sm.met);
    }
    if (!warp_wait(&sm.met, met_use++)) return false;  // O and the sums are read
  }
}

// Descriptors and products of a tile's keys: kN of them at a time in the scores.
template <int D, int kN>
struct Products {
  using L = KvLayout<D>;
  static constexpr uint32_t kIdescS = idesc_bf16(kN, false), kIdescO = idesc_bf16(128, true);
  KvCommon& sm;
  uint64_t k_major, mn_major;  // descriptors of operands at the beginning of shared memory; places are added in 16 bytes
  uint32_t tmem;
  __device__ __forceinline__ Products(KvCommon& c, uint32_t base, uint32_t t)
      : sm(c), k_major(smem_desc_sw128(base, 16, 1024)), mn_major(smem_desc_sw128(base, kKvUnit / 2, 1024)), tmem(t) {}
  static __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t n) { return mbar_wait_near(bar, n & 1u); }
  static __device__ __forceinline__ uint64_t place_of(uint32_t c) { return static_cast<uint64_t>((L::kUnits + c % L::kRing * kKvUnit) >> 4); }
  __device__ __forceinline__ bool unit_there(uint32_t c) const {
    const bool ok = wait(&sm.full[c % L::kRing], c / L::kRing);
    fence_proxy_async_smem();  // the copies are ordinary writes of other threads, done when the barrier says so
    tc_fence_after();
    return ok;
  }
  // scores of group w with keys kN h ... of unit c: queries in slot q, channels 128 u ...
  __device__ __forceinline__ void scores(int w, uint32_t q, uint32_t c, int u, int h) const {
    const uint64_t da = k_major + ((q * L::kQSlot + u * 2 * L::kQBlock) >> 4), db = k_major + place_of(c) + ((h * kN * 128) >> 4);
    const uint32_t to = tmem + L::kTmemS + w * 128 + h * kN;
#pragma unroll
    for (int s = 0; s < 8; ++s)
      mma_f16_ss(to, da + (((s / 4) * L::kQBlock + (s % 4) * 32) >> 4), db + (((s / 4) * (kKvUnit / 2) + (s % 4) * 32) >> 4), kIdescS, u > 0 || s > 0);
  }
  // weights of group w (of their half h) with unit c, into 128 columns of the output; 16 keys a step
  __device__ __forceinline__ void values(int w, uint32_t column, uint32_t c, bool more, int h) const {
    const uint64_t db = mn_major + place_of(c) + ((h * kN * 128) >> 4);
    const uint32_t from = tmem + L::kTmemS + w * 128 + h * kN;
#pragma unroll
    for (int s = 0; s < kN / 16; ++s) mma_f16_ts(tmem + L::kTmemO + column, from + s * 8, db + (s * 2048 >> 4), kIdescO, more || s > 0);
  }
};

// D = 128: one thread for each softmax group issues that group's products, so that one's waits and fences lie under
// the other's products.  Both go through all units and queries, and a place is given back when both are through with
// it: a thread that left out what the other uses could not tell the phases of the barriers apart.
__device__ __forceinline__ bool mma_apart(KvSmall<128>& sm, uint32_t base, uint32_t tmem, int w) {
  using L = KvLayout<128>;
  const Products<128, 64> mma(sm, base, tmem);
  uint32_t unit = 0, next = 0, q_use = 0, p_use = 0;  // next: the first unit that has not been waited for
#pragma unroll 1
  for (uint32_t job_use = 0;; ++job_use) {
    if (!mma.wait(&sm.job_full[job_use & 1], job_use >> 1)) return false;
    const Job& job = sm.job[job_use & 1];
    if (!job.live) return true;
    const int n = job.n;
    const bool two = job.two;
    mbar_arrive(&sm.job_empty[job_use & 1]);
    if (n == 0) continue;
    // tiles of keys of the group, and where its queries are
    const int j0 = two ? 0 : w, step = two ? 1 : 2;
    const uint32_t q = q_use + (two ? w : 0), slot = q & 1;
    auto keys_of = [&](int j) { return unit + (two || j == 0 ? 2 * j : 2 * j - 1); };
    auto values_of = [&](int j) { return unit + (two ? 2 * j + 1 : min(j + 2, n) + j); };
    // units up to c - 1, which the other thread uses
    auto pass_to = [&](uint32_t c) {
      for (; next < c; ++next) {
        if (!mma.wait(&sm.full[next % L::kRing], next / L::kRing)) return false;
        mbar_arrive(&sm.empty[next % L::kRing]);
      }
      return true;
    };
    auto own_unit = [&](uint32_t c) {
      const bool ok = pass_to(c) && mma.unit_there(c);
      next = c + 1;
      return ok;
    };
    auto pass_queries = [&](uint32_t i) {
      if (!mma.wait(&sm.q_full[i & 1], i >> 1)) return false;
      mbar_arrive(&sm.q_empty[i & 1]);
      return true;
    };
    if (j0 < n) {
      if (!mma.wait(&sm.q_full[slot], q >> 1) || !own_unit(keys_of(j0))) return false;
      for (int h = 0; h < 2; ++h) {
        mma.scores(w, slot, keys_of(j0), 0, h);
        tc_commit(&sm.half_s[w][h]);
      }
      tc_commit(&sm.empty[keys_of(j0) % L::kRing]);
      if (j0 + step >= n) tc_commit(&sm.q_empty[slot]);  // used for the last time
      if (two && !pass_queries(q_use + (w ^ 1))) return false;
    } else if (!pass_queries(q)) {
      return false;
    }
    for (int j = j0; j < n; j += step, ++p_use) {
      const bool more = j + step < n;
      const uint32_t v = values_of(j), k = keys_of(j + step);
      if (!own_unit(v)) return false;
      for (int h = 0; h < 2; ++h) {
        if (!mma.wait(&sm.half_p[w][h], p_use)) return false;
        tc_fence_after();
        mma.values(w, w * 128, v, j > j0 || h > 0, h);
        if (more) {
          if (h == 0 && !own_unit(k)) return false;
          mma.scores(w, slot, k, 0, h);
          tc_commit(&sm.half_s[w][h]);
        } else if (h == 0) {
          tc_commit(&sm.pv_done[w]);
        }
      }
      tc_commit(&sm.empty[v % L::kRing]);
      if (more) {
        tc_commit(&sm.empty[k % L::kRing]);
        if (j + 2 * step >= n) tc_commit(&sm.q_empty[slot]);
      }
    }
    if (j0 < n) tc_commit(&sm.o_full[w]);
    unit += 2 * n;
    if (!pass_to(unit)) return false;
    q_use += two ? 2 : 1;
  }
}

// D = 256: one thread issues the products, in the order of their units.
__device__ __forceinline__ bool mma_shared(KvSmall<256>& sm, uint32_t base, uint32_t tmem) {
  constexpr int D = 256;
  using L = KvLayout<D>;
  const Products<D, 128> mma(sm, base, tmem);
  uint32_t unit = 0, q_use = 0, p_use[2] = {0, 0};
#pragma unroll 1
  for (uint32_t job_use = 0;; ++job_use) {
    if (!mma.wait(&sm.job_full[job_use & 1], job_use >> 1)) return false;
    const Job& job = sm.job[job_use & 1];
    if (!job.live) return true;
    const int n = job.n;
    mbar_arrive(&sm.job_empty[job_use & 1]);
    if (n == 0) continue;
    const uint32_t slot = q_use % L::kQSlots;
    if (!mma.wait(&sm.q_full[slot], q_use / L::kQSlots)) return false;
    auto tile_scores = [&](int j) {
      for (int u = 0; u < L::kKU; ++u, ++unit) {
        if (!mma.unit_there(unit)) return false;
        mma.scores(j & 1, slot, unit, u, 0);
        tc_commit(&sm.empty[unit % L::kRing]);
      }
      tc_commit(&sm.s_full[j & 1]);
      if (j == n - 1) tc_commit(&sm.q_empty[slot]);
      return true;
    };
    if (!tile_scores(0) || (n > 1 && !tile_scores(1))) return false;
    for (int j = 0; j < n; ++j) {
      if (!mma.wait(&sm.p_full[j & 1], p_use[j & 1]++)) return false;
      tc_fence_after();
      for (int u = 0; u < L::kKU; ++u, ++unit) {
        if (!mma.unit_there(unit)) return false;
        mma.values(j & 1, u * 128, unit, j > 0, 0);
        tc_commit(&sm.empty[unit % L::kRing]);
      }
      tc_commit(&sm.pv_done[j & 1]);
      if (j + 2 < n && !tile_scores(j + 2)) return false;
    }
    tc_commit(&sm.o_full[0]);
    tc_commit(&sm.o_full[1]);
    ++q_use;
  }
}

template <int D>
__global__ void __launch_bounds__(KvLayout<D>::kThreads, 1)
    kv_attention_kernel(const __grid_constant__ KvAttentionArgs a, const __grid_constant__ KvPlan p) {
  using L = KvLayout<D>;
  // no static shared memory: the dynamic one begins on the swizzle's 1024 bytes (checked below)
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kIssuers = D == 128 ? 2 : 1;  // threads that issue products
  KvSmall<D>& sm = *reinterpret_cast<KvSmall<D>*>(smem + L::kSmall);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023u) {
    pdl_wait();  // whoever follows in the stream counts on what came before having ended
    if (threadIdx.x == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
    return;
  }
  if (warp == L::kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < L::kRing; ++i) {
        mbar_init(&sm.full[i], 128);
        mbar_init(&sm.empty[i], kIssuers);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.q_full[i], 128);
        mbar_init(&sm.q_empty[i], kIssuers);
        if constexpr (D == 128) {
          for (int h = 0; h < 2; ++h) {
            mbar_init(&sm.half_s[i][h], 1);
            mbar_init(&sm.half_p[i][h], 4);
          }
        } else {
          mbar_init(&sm.s_full[i], 1);
          mbar_init(&sm.p_full[i], 8);
          for (int x = 0; x < 8; ++x) mbar_init(&sm.decided[i][x], 1);
        }
        mbar_init(&sm.o_full[i], 1);
        mbar_init(&sm.pv_done[i], 1);
        mbar_init(&sm.job_full[i], 1);
        mbar_init(&sm.job_empty[i], L::kSoftWarps + 4 + kIssuers);
      }
      mbar_init(&sm.met, L::kSoftWarps);
      mbar_init(&sm.wanted, 1);
      mbar_init(&sm.taken, 1);
      mbar_init(&sm.drain, kIssuers);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc<512>(&sm.tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  pdl_wait();

  bool ok = true;
  if (warp < L::kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoftRegs));
    if constexpr (D == 128) ok = soft_apart(a, p, sm, tmem);
    else ok = soft_shared(a, p, sm, tmem);
    tc_fence_before();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kOtherRegs));
    if (warp == L::kMmaWarp || (D == 128 && warp == L::kMmaWarp2)) {
      if (elect_one()) {
        if constexpr (D == 128) ok = mma_apart(sm, smem_u32(smem), tmem, warp != L::kMmaWarp);
        else ok = mma_shared(sm, smem_u32(smem), tmem);
        // the end of every product: tensor memory may be given back
        tc_commit(&sm.drain);
        ok = mbar_wait_near(&sm.drain, 0) && ok;
        if (!ok) flag_error(a.err, CKV_DEVERR_TIMEOUT);
      }
      __syncwarp();
    } else if (warp == L::kPlanWarp) {
      ok = plan_jobs<L>(a, p, sm, [](const Job&, uint32_t) {});
    } else if (warp >= L::kCopyWarp) {
      ok = copy_jobs<L>(a, sm, smem);
    }
  }
  if (!ok && lane == 0) flag_error(a.err, CKV_DEVERR_TIMEOUT);
  pdl_trigger();
  __syncthreads();
  if (warp == L::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

// Without a window jobs are as long as the contexts, and a long one that begins last leaves the other SMs waiting: requests
// are put in the order of their last tokens' contexts, the longest first (and their tiles from the last one on).  That takes
// a kernel of its own and longer lookups, which few or short jobs do not earn back.  With contexts of up to 4096 rows, not
// sorted and sorted: 256 tokens x 64 heads of 512 channels (2 jobs to an SM) 180 and 142 us, x 32 heads of 256 (7) 330 and
// 315, 128 drafts of 40 to 64 (7) 267 and 257; x 64 heads of 128 (14) 319 and 324, 1000 tokens x 32 heads (7) 185 and 196; up
// to 1024 rows, 256 tokens x 32 heads of 256 109 and 113.  One CTA ranks the requests, a thread each: more than its 256
// are taken as they come, however few their jobs.
constexpr int kOrderRequests = 256, kOrderTiles = 20, kOrderJobs = 152 * 8;

__global__ void __launch_bounds__(kOrderRequests) kv_order_kernel(const __grid_constant__ KvAttentionArgs a, int R) {
  __shared__ __align__(16) uint32_t key[kOrderRequests];
  __shared__ int32_t count[kOrderRequests], total[32];
  pdl_wait();
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5;
  int32_t tiles = 0, len = 0;
  if (b < a.B) {
    const int32_t t0 = kv_start_of(a, b), n = kv_start_of(a, b + 1) - t0;
    if (n > 0) {
      tiles = static_cast<int32_t>((static_cast<int64_t>(n) * a.G + R - 1) / R);
      len = min(max(a.ctx_rows[t0 + n - 1], 0), a.max_rows);
    }
  }
  // contexts in steps of 16 rows (21 bits hold the largest), then the lower request: all keys are different
  key[b] = b < a.B ? static_cast<uint32_t>(len) >> 4 << 10 | static_cast<uint32_t>(kOrderRequests - 1 - b) : 0u;
  __syncthreads();
  int rank = 0;
  const uint32_t mine = key[b];
  for (int i = 0; i < (a.B + 3) / 4; ++i) {
    const uint4 k = reinterpret_cast<const uint4*>(key)[i];
    rank += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
  }
  int32_t* order = static_cast<int32_t*>(a.workspace);
  if (b < a.B) {
    order[rank] = b;
    count[rank] = tiles;
  }
  __syncthreads();
  const int32_t own = b < a.B ? count[b] : 0;
  int32_t sum = own;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) total[warp] = sum;
  __syncthreads();
  for (int i = 0; i < warp; ++i) sum += total[i];
  if (b < a.B) {
    if (b == 0) order[a.B] = 0;
    order[a.B + 1 + b] = sum;
  }
  pdl_trigger();
}

// Joins the ranges of a row, in their order: one warp per row and 128 channels.
template <int D, bool kFew>
__global__ void __launch_bounds__(128, kFew ? 12 : 4) kv_join_kernel(const __grid_constant__ KvAttentionArgs a, int splits) {
  constexpr int kParts = D / 128, kDeep = kFew ? 4 : 16, kOwn = kFew ? 1 : kKvMaxSplits / 32;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const int64_t work = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5), flat = work / kParts, rows = a.T * a.H;
  const int part = static_cast<int>(work % kParts);
  if (flat >= rows) return;
  const int32_t t = static_cast<int32_t>(flat / a.H);
  if (a.ctx_rows[t] < 0 || t < kv_start_of(a, 0) || t >= kv_start_of(a, a.B)) return;
  const float* ws = static_cast<const float*>(a.workspace);
  const float* part_lse = ws + splits * rows * D + flat;
  float lse[kOwn], m = -INFINITY;  // of ranges lane, lane + 32, ...
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int s = lane + i * 32;
    lse[i] = s < splits ? part_lse[s * rows] : -INFINITY;
    m = fmaxf(m, lse[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float sink = a.sink ? a.sink[flat % a.H] : -INFINITY;
  m = fmaxf(m, sink);
  const float safe = m == -INFINITY ? 0.f : m;
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    lse[i] = fast_exp2((lse[i] - safe) * kLog2e);  // its weight from here on
    all += lse[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  if (a.sink) all += sink == safe ? 1.f : fast_exp2((sink - safe) * kLog2e);  // safe: one of -infinity counts for nothing
  const float4* o = reinterpret_cast<const float4*>(ws + flat * D + part * 128) + lane;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    for (int s0 = j * 32; s0 < min(splits, j * 32 + 32); s0 += kDeep) {
      float4 v[kDeep];
      float x[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        x[i] = __shfl_sync(0xFFFFFFFFu, lse[j], (s0 + i) % 32);
        v[i] = s0 + i < splits && x[i] != 0.f ? o[(s0 + i) * (rows * D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        if (s0 + i >= splits) x[i] = 0.f;
        acc[0] = fmaf(v[i].x, x[i], acc[0]);
        acc[1] = fmaf(v[i].y, x[i], acc[1]);
        acc[2] = fmaf(v[i].z, x[i], acc[2]);
        acc[3] = fmaf(v[i].w, x[i], acc[3]);
      }
    }
  }
  const float inv = all == 0.f ? 0.f : 1.f / all;
  *reinterpret_cast<uint2*>(a.out + flat * D + part * 128 + lane * 4) =
      make_uint2(pack_bf16x2_rn(acc[0] * inv, acc[1] * inv), pack_bf16x2_rn(acc[2] * inv, acc[3] * inv));
  if (part == 0 && lane == 0 && a.lse) a.lse[flat] = all == 0.f ? -INFINITY : safe + log2f(all) * kKvLn2;
}

// Rows of tiles, and into how many ranges of keys a tile is split: the count that a model of the time
// finds best.  CTAs take their jobs one after the other.  Lengths are known on the host by their
// bound only, so ranges are of equal size, and of 2^17 keys at most (the tensor cores cut each sum
// off towards 0: fp4_attention.cu has the figures).  With a window that holds where a tile's tokens have
// contexts next to one another, as tokens of a request do; where they are apart the last range has all
// that the span leaves out, of which a token sees its window at most.
KvPlan plan_kv(int64_t T, int32_t B, int32_t H, int32_t KH, int32_t D, int64_t max_rows, int32_t window, int32_t first, int32_t words) {
  KvPlan p;
  const int G = H / KH;
  const int64_t rows = (T + B - 1) / B * G;  // of an average request and key head
  // At D = 512 a tile of 128 rows has no place in tensor memory beside its scores, and two CTAs that form them both for half
  // of the channels each take longer than tiles of 64 rows (8000 tokens x 64 heads, windows of 128 to 4096 rows: 698 against
  // 336 us, 1659 against 1323, 3211 against 2965).  Below it, longer tiles win (D = 256, 32 heads, 4096: 631 against 942).
  const int R = p.R = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 || D == 512 ? 64 : D == 128 ? 256 : 128;
  const int64_t pad = kv_tile_pad(G, R);
  p.tiles = static_cast<int>((T * G + std::min<int64_t>(T, B) * pad) / R);
  int64_t busy = (T * G + R - 1) / R;
  busy = busy < T && busy < B ? (T < B ? T : B) : busy;
  busy *= KH;
  // keys that a tile's tokens, `tokens` at most, see together when they follow each other
  int64_t span = max_rows;
  const int g = G & -G, tokens = (G - std::min(g, R) + R + G - 1) / G;
  if (window > 0) span = std::min<int64_t>(max_rows, static_cast<int64_t>(window) + first + tokens - 1 + 64 * words);
  const int64_t most = (span + kKvKeys - 1) / kKvKeys;
  const double around = 2.0, tile = D == 512 ? 2.0 : D == 256 ? 1.2 : 0.8;
  const int64_t least = (span + kKvMaxRange - 1) / kKvMaxRange;  // <= kKvMaxSplits: the callers' bound of max_rows
  int64_t best_s = least;
  double best = 0;
  for (int64_t s = least; s <= most && s <= kKvMaxSplits; ++s) {
    if (s > least && p.tiles * s * KH > INT32_MAX) break;  // CTAs of a grid
    const int64_t waves = (busy * s + 151) / 152;
    double us = static_cast<double>(waves) * (around + tile * static_cast<double>((most + s - 1) / s));
    if (s > 1) us += 2.5 + 0.02 * static_cast<double>(s) + 2.0 * static_cast<double>(T * H * s) * D * 4 / 4e6;
    if (s == least || us < best) {
      best = us;
      best_s = s;
    }
  }
  p.chunk = static_cast<int>((most + best_s - 1) / best_s * kKvKeys);
  p.splits = static_cast<int>((span + p.chunk - 1) / p.chunk);
  // What a job is about is looked up once for several key heads where jobs are short (a lookup takes 4 us, a tile of keys
  // 1.5) and leave each SM six CTAs all the same: 1024 requests x 64 heads over 128 rows 209 -> 158 us.
  p.heads = 1;
  const int64_t ctas = static_cast<int64_t>(p.tiles) * p.splits * KH;
  p.sorted = window == 0 && p.splits == 1 && B > 1 && B <= kOrderRequests && most >= kOrderTiles && busy > 152 && busy <= kOrderJobs;
  while (p.heads < KH && p.heads * ((p.chunk < span ? p.chunk : span) + kKvKeys - 1) / kKvKeys < 8 && ctas / (2 * p.heads) >= 152 * 6) p.heads *= 2;
  return p;
}

// Warps that ask for more registers than the CTA has would wait for ever: the registers of its launch have to be as counted.
template <int D>
cudaError_t check_registers_once() {
  static const cudaError_t result = [] {
    using L = KvLayout<D>;
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, kv_attention_kernel<D>);
    if (e != cudaSuccess) return e;
    const int need = L::kSoftWarps * 32 * L::kSoftRegs + (L::kThreads - L::kSoftWarps * 32) * L::kOtherRegs;
    return attr.numRegs * L::kThreads >= need ? cudaSuccess : cudaErrorInvalidConfiguration;
  }();
  return result;
}

template <int D>
cudaError_t launch(const KvAttentionArgs& a, const KvPlan& p, bool use_pdl, cudaStream_t s) {
  cudaError_t e;
  if ((e = check_registers_once<D>()) != cudaSuccess) return e;
  if ((e = set_max_smem_once<kv_attention_kernel<D>>(kv_smem_bytes<D>())) != cudaSuccess) return e;
  return launch_ex(kv_attention_kernel<D>, dim3(static_cast<unsigned>(kv_jobs(p, a.KH))), dim3(KvLayout<D>::kThreads), kv_smem_bytes<D>(), use_pdl,
                   s, a, p);
}

template <int D>
cudaError_t launch_join(const KvAttentionArgs& a, const KvPlan& p, cudaStream_t s) {
  const int64_t ctas = (a.T * a.H * (D / 128) + 3) / 4;
  return p.splits <= 4 ? launch_ex(kv_join_kernel<D, true>, dim3(static_cast<unsigned>(ctas)), dim3(128), 0, true, s, a, p.splits)
                       : launch_ex(kv_join_kernel<D, false>, dim3(static_cast<unsigned>(ctas)), dim3(128), 0, true, s, a, p.splits);
}

template <int D>
cudaError_t launch_d(const KvAttentionArgs& args, bool use_pdl, cudaStream_t s) {
  const KvPlan p = plan_kv(args.T, args.B, args.H, args.KH, D, args.max_rows, args.window, args.first, args.words);
  if (p.tiles == 0) return cudaSuccess;
  cudaError_t e;
  KvAttentionArgs a = args;
  if (p.sorted) {
    a.order = static_cast<const int32_t*>(a.workspace);
    if ((e = launch_ex(kv_order_kernel, dim3(1), dim3(kOrderRequests), 0, use_pdl, s, a, p.R)) != cudaSuccess) return e;
    use_pdl = true;  // behind a kernel of this call
  }
  if constexpr (D == 512) e = launch_kv_attention_few(a, p, use_pdl, s);
  else e = p.R <= 64 ? launch_kv_attention_few(a, p, use_pdl, s) : launch<D>(a, p, use_pdl, s);
  return e != cudaSuccess || p.splits == 1 ? e : launch_join<D>(a, p, s);
}

}  // namespace

int64_t kv_attention_workspace(int64_t T, int32_t B, int32_t H, int32_t KH, int32_t D, int64_t max_rows, int32_t window, int32_t first_rows,
                               int32_t words) {
  const KvPlan p = plan_kv(T, B, H, KH, D, max_rows, window, window > 0 ? first_rows : 0, words);
  if (kv_jobs(p, KH) > INT32_MAX) return -1;  // more CTAs than a grid has
  if (p.sorted) return (2 * static_cast<int64_t>(B) + 1) * static_cast<int64_t>(sizeof(int32_t));
  return p.splits == 1 ? 0 : static_cast<int64_t>(p.splits) * T * H * (D + 1) * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, bool use_pdl, cudaStream_t s) {
  return a.cache.D == 128 ? launch_d<128>(a, use_pdl, s) : a.cache.D == 256 ? launch_d<256>(a, use_pdl, s) : launch_d<512>(a, use_pdl, s);
}

}  // namespace ckv
