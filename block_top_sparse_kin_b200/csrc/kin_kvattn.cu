// kin_kvattn.cu -- split-K flash-decode over a KV cache of either format
// (bf16 rows, or 4-bit rows: kin_kv4.cu), over the kept blocks or over every
// block, optionally adding each token's attention weight to a running sum.
//
// Math, for the query heads j of a pair (b, KV head h):
//   z_jt = scale q_j . K_t,  out_j = sum_t e^(z_jt - M) V_t / sum_t e^(z_jt - M),
//   acc_t += sum_j e^(z_jt - lse_j),
// in the running-maximum form with base-2 logits, chunks of the kept blocks
// merged by their log-sum-exp (the pair's last chunk to finish merges, counted
// with an atomic; nothing spins).  With 4-bit rows K_t = (ks_tg c_td), V_t =
// (vs_tg c_td), g the group of 32 channels, c an integer in [-7, 7]:
//   q . K_t = sum_g ks_tg (q_g . c_tg)       one product per group, scaled after
//   sum_t p_t V_td = sum_t (p_t vs_tg) c_td  the scale goes to the weight
// so the codes enter the matrix instructions exactly and no row is rounded.
//
// A decode group has at most 8 heads, so the products are mma.sync m16n8k16
// tiles of 16 tokens by 8 heads, fed per warp by a ring of asynchronous
// copies, 3 CTAs of 4 warps on an SM.  The bytes, 144 (4 bit) or 512 (bf16) a
// token and pair, bound bf16 rows: 32 x 8 pairs, 4096 of 32768 tokens each, 4
// heads: 87 us, 6.2 TB/s.  4-bit rows are bounded by what a tile costs the
// SM: the same batch 41.7 us, 3.6 TB/s; 261 instructions a tile by one warp,
// 102 of them for the logic unit (64 unpack its 4096 codes) and 84 multiply-
// adds.  No unit is over half busy and half of the issue slots are empty: 12
// warps an SM, each one dependent chain from the copies to the sums.  Measured
// on the way there: nibbles through one conversion for two, 66 us; as fp16
// subnormals, with no conversion, 49; two tiles a step, which share the
// maximum, the copies' waits and the query loads, and even ranges, 41; codes
// placed so that light tokens keep their bits and scales watched, 41.7.  16
// warps of 128 registers, one tile a step: 45 for 42.
#include <type_traits>

#include "kin_internal.cuh"

namespace kin {

namespace {

#define kNegInf (-__int_as_float(0x7f800000))

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
static_assert(kThreads == kHeadDim, "a thread has one output channel, and 16 threads a query head");
constexpr int kRowPad = kHeadDim + 4;
constexpr int kHalfBox = 16 * 64 * 2;

template <bool kInt4>
struct Ring {
  // tiles of 16 tokens that a warp takes at a step
  static constexpr int kStep = kInt4 ? 2 : 1;
  // bf16: K0 K1 V0 V1 half tiles of 16 rows x 64 channels.  4 bit: 16 rows of
  // 64 bytes of key codes, of value codes, then 16 x 4 scales of each.
  static constexpr int kTileBytes = kInt4 ? 2 * 16 * kCodeBytes + 2 * 16 * kGroups * 2 : 4 * kHalfBox;
  static constexpr int kStageBytes = kStep * kTileBytes;
  static constexpr int kStages = kInt4 ? 3 : 2;
  // 4 bit, per warp and tile behind the ring: the tile's key scales as fp32
  // [16][4] and its value scales as fp16 pairs [8 token pairs][4]
  static constexpr int kScaleBytes = kInt4 ? 256 + 128 : 0;
  static constexpr int kWarpBytes = kStages * kStageBytes + kStep * kScaleBytes;
  static constexpr int kPipe = kWarps * kWarpBytes;
  static constexpr int kComb = kWarps * kMaxGroup * kRowPad * 4;
  static constexpr int kSmem = (kPipe > kComb ? kPipe : kComb) + 1024;
};

// Rows are read once: their lines leave L2 before the logits and partials do.
// 32 x 8 pairs of 4096 tokens, against copies without the hint: bf16 rows 86.9
// us for 89.2, 4-bit rows 42.2 for 43.9; with weights 53.6 for 55.0 (4 bit) and
// 102.7 for 103.3 (bf16), three caches in turn (one build, 1% slower than the
// last).  Called on one cache again and again, bf16 with weights takes 95 for
// 103.
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ void cp_async16_once(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(src_bytes),
               "l"(policy)
               : "memory");
}

__device__ __forceinline__ void cp_async8_once(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
  asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], 8, %2, %3;" ::"r"(dst), "l"(src), "r"(src_bytes),
               "l"(policy)
               : "memory");
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B, from zero
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma_bf16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t part_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ unsigned count_chunk(uint32_t* counter) {
  unsigned v;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(counter) : "memory");
  return v;
}

// 2^x to 2^-22, results below 2^-126 as zero: a weight that small adds nothing
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ void sts64(uint32_t a, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Zero the bf16 halves of a V^T fragment register whose token is invalid.
__device__ __forceinline__ uint32_t tok_mask(int t, int nvalid) {
  return (t < nvalid ? 0x0000FFFFu : 0u) | (t + 1 < nvalid ? 0xFFFF0000u : 0u);
}

// A head's weights are 2^(z - r) with a reference r that follows the running
// maximum m of its logits loosely: r = m - lead, and m moves (all sums are
// then rescaled) only when a logit passes m + kSlack.  So a tile usually
// costs no reduction over its tokens.  4 bit: weights reach 2^15, near the top
// of fp16's range.  bf16: weights stay below 2^-22 and a pair attends to at
// most 2^22 tokens (32768 blocks of 128), so no sum of weights passes 1, in a
// warp or over the ranges, and values of any magnitude average without
// overflow; from 2^-80 down they come near the end of fp32.
constexpr float kSlack = 8.f;
template <bool kInt4>
constexpr float kLead = kInt4 ? 7.f : -kSlack - 22.f;

// The sums of a warp: O^T fragments, and for its two head columns the maximum
// logit followed, before the scaling to base 2 (raw), the reference and the
// weights' sum.
struct Acc {
  float o[8][4];
  float sums[4];  // 4 bit: row G < 4 holds the weights' sums p vs of group G
  float m[2], thr[2], r[2], l[2];
};

// The weights p of N tiles from their raw logits s (rows tq, tq + 8; heads ta,
// ta + 1; -inf where there is no token); sl2: base-2 scale of the two heads.
template <bool kInt4, int N>
__device__ __forceinline__ void weigh(Acc& a, const float (&s)[N][4], const float (&sl2)[2], float (&p)[N][4]) {
  float x[2] = {fmaxf(s[0][0], s[0][2]), fmaxf(s[0][1], s[0][3])};
#pragma unroll
  for (int h = 1; h < N; ++h) {
    x[0] = fmaxf(x[0], fmaxf(s[h][0], s[h][2]));
    x[1] = fmaxf(x[1], fmaxf(s[h][1], s[h][3]));
  }
  if (__any_sync(0xffffffffu, x[0] > a.thr[0] || x[1] > a.thr[1])) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], off));
      x[1] = fmaxf(x[1], __shfl_xor_sync(0xffffffffu, x[1], off));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float mn = fmaxf(a.m[j], x[j]);
      const float al = mn == a.m[j] ? 1.f : exp2_approx((a.m[j] - mn) * sl2[j]);
      a.m[j] = mn;
      a.thr[j] = mn + __fdividef(kSlack, sl2[j]);
      a.r[j] = mn * sl2[j] - kLead<kInt4>;
      a.l[j] *= al;
      a.sums[j] *= al;
      a.sums[2 + j] *= al;
#pragma unroll
      for (int dm = 0; dm < 8; ++dm) {
        a.o[dm][j] *= al;
        a.o[dm][2 + j] *= al;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < N; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[h][i] = exp2_approx(fmaf(s[h][i], sl2[i & 1], -a.r[i & 1]));
      a.l[i & 1] += p[h][i];
    }
  }
}

}  // namespace

constexpr uint32_t kPartial = 0x80000000u;

// Tile i of a warp, in its CTA's range: steps are dealt to the warps in turn.
template <int kStep>
__device__ __forceinline__ int warp_tile(int warp, int i) {
  return (warp + kWarps * (i / kStep)) * kStep + i % kStep;
}

template <bool kInt4, bool kAcc>
__global__ void __launch_bounds__(kThreads, kKvCtasPerSm) kv_attn_kernel(KvAttnParams p) {
  using R = Ring<kInt4>;
  constexpr int kStages = R::kStages, kStep = R::kStep;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float s_m[kWarps][kMaxGroup], s_l[kWarps][kMaxGroup];
  __shared__ int s_last;
  constexpr int kMaxMergeWeights = R::kPipe / (4 * kPartStride);
  __shared__ float s_mr[kMaxGroup], s_den[kMaxGroup], s_inv[kMaxGroup], s_a[kMaxGroup], s_w[kMaxMergeWeights];
  __shared__ float s_ww[kWarps][kMaxGroup], s_cm[kMaxGroup], s_cden[kMaxGroup];
  // per warp: its tiles' rows (kPartial: less than 16 of them valid) and valid rows
  __shared__ __align__(8) uint32_t s_rows[kWarps][64];
  __shared__ uint8_t s_valid[kWarps][64];
  // 4 bit: the group's queries in fp16, per group of channels -8 times their sum, the logits' scales
  __shared__ __align__(16) uint32_t s_q[kInt4 ? kMaxGroup * 64 : 4];
  __shared__ float s_off[kMaxGroup][4], s_sl2[kMaxGroup];

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = p.g, bs = p.bs, Lcap = p.kv.Lcap;
  pdl_wait();  // the selection comes from the select kernels
  // No early launch_dependents: the next grid's CTAs would take what room this
  // one leaves on each SM and so lie unevenly (296 CTAs of 128 tiles, launched
  // back to back: 29.5 us a call with it, 23.4 without).
  const int lbs = 31 - __clz(bs), ltpb = lbs - 4;  // log2 of a block's tokens and of its tiles
  const int c = lane & 3, tq = lane >> 2, ta = 2 * c;

  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * R::kWarpBytes);
  const uint32_t scales = ring + kStages * R::kStageBytes;
  const uint32_t rows_s = smem_u32(s_rows[warp]);
  // 4 bit: a row's 4 pieces of 16 bytes of codes lie in token order, pieces 2
  // and 3 swapped with 0 and 1 in every second pair of rows: both the keys'
  // 16-byte reads (two rows of different parity in 8 lanes) and the values'
  // 8-byte reads (four rows, both parities, both orders, in 16 lanes) are then
  // free of bank conflicts, with the tokens' order below
  const uint32_t code_dst = ring + tq * 64 + ((c ^ (tq & 2)) << 4);
  const uint32_t scale_dst = ring + 2048 + lane * 8;
  // k slots 2c, 2c + 1, 2c + 8, 2c + 9 of the second product are tokens c, 4 +
  // (c ^ 1), 8 + c and 12 + (c ^ 1) of the tile: so is the order of its rows
  const int t0 = kInt4 ? ((tq & 1) ? 4 + ((tq >> 1) ^ 1) : tq >> 1) : tq, t1 = t0 + 8;

  // This CTA's range of the (pair, kept block) slots, cut at pair boundaries:
  // blocks [j0, j1) of one pair at a time.
  const int hi_slot = min((int)(blockIdx.x + 1) * p.per, p.slots);
  for (int at = blockIdx.x * p.per; at < hi_slot;) {
  const int pair = at / p.stride;
  int j0 = at - pair * p.stride, j1 = min(p.k, hi_slot - pair * p.stride), per = p.per;
  at = (pair + 1) * p.stride;
  const int b = pair / p.Hkv, h = pair - b * p.Hkv;
  const int L = __ldg(p.seq_lens + b);
  if (p.fit) {  // dense, every CTA resident: the pair's CTAs share what its length has
    const int blocks = L < 1 || L > Lcap ? 0 : (L + bs - 1) >> lbs;
    per = min(p.per, max((blocks + p.max_chunks - 1) / p.max_chunks, p.fit));
    j0 = ((int)blockIdx.x - pair * p.max_chunks) * per;
    j1 = min(p.k, j0 + per);
  }
  const int64_t qh0 = (int64_t)b * p.Hq + (int64_t)h * g;
  // lane l's tiles l and l + 32 of this warp (steps warp, warp + W, .. of the
  // range, kStep tiles each): their block indices are requested before the
  // length and count, whose round trip they would follow
  int blk[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int j = j0 + (warp_tile<kStep>(warp, lane + 32 * r) >> ltpb);
    blk[r] = j;
    if (p.sel_idx) blk[r] = j < j1 ? __ldg(p.sel_idx + (int64_t)pair * p.k_row + j) : -1;
  }
  // 4 bit: thread t's 8 query channels, 8 (t % 16) .. of head t / 16
  uint4 qw = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (kInt4) {
    if ((tid >> 4) < g) qw = __ldg(reinterpret_cast<const uint4*>(p.q + (qh0 + (tid >> 4)) * kHeadDim) + (tid & 15));
  }
  const bool bad_len = L < 1 || L > Lcap;
  const int nb = bad_len ? 0 : (L + bs - 1) >> lbs;
  int cnt = p.sel_idx ? __ldg(p.sel_cnt + pair) : nb;
  if (bad_len) cnt = 0;
  if (cnt > p.k) cnt = p.k;
  if (cnt <= 0) {  // nothing to attend to: out = 0, lse = -inf
    if (j0 == 0) {
      for (int d = tid; d < g * kHeadDim; d += kThreads) p.out[qh0 * kHeadDim + d] = __float2bfloat16_rn(0.f);
      if (tid < g) {
        if (p.lse) p.lse[qh0 + tid] = kNegInf;
        if (kAcc) p.lse2[qh0 + tid] = kNegInf;
      }
      if (bad_len && tid == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
    }
    continue;
  }
  const int ntiles = (min(j1, cnt) - j0) << ltpb;
  if (ntiles <= 0) continue;
  // the pair's ranges that hold a kept block, and this one's place among them
  const int first_cta = pair * p.stride / p.per;
  const int nchunks = p.fit ? (cnt + per - 1) / per : (pair * p.stride + cnt - 1) / p.per - first_cta + 1;
  const int chunk = blockIdx.x - first_cta;

  // the warp's tiles' first rows (a cache of 2^31 rows is larger than the
  // memory); a tile of less than 16 rows is marked and their number kept aside
  const int n_w = warp * kStep < ntiles ? (ntiles - 1 - warp * kStep) / (kWarps * kStep) + 1 : 0;  // steps
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int tile = warp_tile<kStep>(warp, lane + 32 * r);
    uint32_t row = 0u;
    int nv = 0;
    if (tile < ntiles) {
      const int tok = (blk[r] << lbs) + ((tile & ((1 << ltpb) - 1)) << 4);
      const bool there = blk[r] >= 0 && blk[r] < nb;
      bool good = there && tok < L;
      if (good) {
        if (p.kv.pages.table) {
          const int page = __ldg(p.kv.pages.table + (int64_t)b * p.kv.pages.max_blocks + blk[r]);
          good = page >= 0 && page < p.kv.pages.num_pages;
          row = ((uint32_t)(page * p.Hkv + h) << lbs) + (tok & (bs - 1));
        } else {
          row = (uint32_t)pair * (uint32_t)Lcap + (uint32_t)tok;
        }
      }
      if (!there || (tok < L && !good)) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
      if (good) nv = min(kTileTokens, L - tok);
      if (!good) row = 0u;
    }
    s_rows[warp][lane + 32 * r] = row | (nv < kTileTokens ? kPartial : 0u);
    s_valid[warp][lane + 32 * r] = (uint8_t)nv;
  }
  __syncwarp();

  const uint64_t once = read_once_policy();
  auto issue_tile = [&](int nt, uint32_t row, uint32_t slot) {  // slot: byte offset of the tile's place in the ring
    if (row < kPartial) {
      if constexpr (kInt4) {
        const uint8_t* ks = p.kv.k + (uint64_t)row * kCodeBytes + lane * 16;
        const uint8_t* vs = p.kv.v + (uint64_t)row * kCodeBytes + lane * 16;
        const uint16_t* ss = (lane < 16 ? p.kv.ks : p.kv.vs) + ((uint64_t)row + (lane & 15)) * kGroups;
        cp_async16_once(code_dst + slot, ks, 16u, once);
        cp_async16_once(code_dst + slot + 512, ks + 512, 16u, once);
        cp_async16_once(code_dst + slot + 1024, vs, 16u, once);
        cp_async16_once(code_dst + slot + 1536, vs + 512, 16u, once);
        cp_async8_once(scale_dst + slot, ss, 8u, once);
      } else {
        const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(p.kv.k) + (uint64_t)row * kHeadDim;
        const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.kv.v) + (uint64_t)row * kHeadDim;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int piece = lane + 32 * i;
          const int r = piece >> 4, cc = piece & 15;
          const uint32_t off = ring + slot + (uint32_t)((cc >> 3) * kHalfBox + r * 128 + (((cc & 7) ^ (r & 7)) << 4));
          cp_async16_once(off, k + piece * 8, 16u, once);
          cp_async16_once(off + 2 * kHalfBox, v + piece * 8, 16u, once);
        }
      }
    } else {  // rows behind the length: zeros, nothing read (the address stays on a valid row)
      const int nv = s_valid[warp][nt];
      row &= ~kPartial;
      if constexpr (kInt4) {
        // a tile without any row: its scales become zeros, its codes may be
        // anything (every nibble is a finite number and its weight is zero)
        if (nv > 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = tq + 8 * i;
            const int64_t from = (int64_t)row * kCodeBytes + lane * 16 + (t < nv ? 512 * i : -tq * 64);
            cp_async16_once(code_dst + slot + 512 * i, p.kv.k + from, t < nv ? 16u : 0u, once);
            cp_async16_once(code_dst + slot + 1024 + 512 * i, p.kv.v + from, t < nv ? 16u : 0u, once);
          }
        }
        const int t = lane & 15;
        cp_async8_once(scale_dst + slot, (lane < 16 ? p.kv.ks : p.kv.vs) + ((uint64_t)row + (t < nv ? t : 0)) * kGroups,
                       t < nv ? 8u : 0u, once);
      } else if (nv > 0) {
        const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(p.kv.k) + (uint64_t)row * kHeadDim;
        const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.kv.v) + (uint64_t)row * kHeadDim;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int piece = lane + 32 * i;
          const int r = piece >> 4, cc = piece & 15;
          const uint32_t off = ring + slot + (uint32_t)((cc >> 3) * kHalfBox + r * 128 + (((cc & 7) ^ (r & 7)) << 4));
          const int src = (r < nv ? r : 0) * kHeadDim + cc * 8;
          const uint32_t bytes = r < nv ? 16u : 0u;
          cp_async16_once(off, k + src, bytes, once);
          cp_async16_once(off + 2 * kHalfBox, v + src, bytes, once);
        }
      }
    }
  };
  auto issue = [&](int st, uint32_t slot) {
    if (st < n_w) {
      if constexpr (kStep == 2) {
        const uint2 r = lds64(rows_s + st * 8);
        issue_tile(2 * st, r.x, slot);
        issue_tile(2 * st + 1, r.y, slot + R::kTileBytes);
      } else {
        issue_tile(st, lds32(rows_s + st * 4), slot);
      }
    }
    cp_async_commit();  // one group per step, empty or not
  };
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) issue(i, i * R::kStageBytes);

  // Queries.  4 bit: key nibbles enter the first product as the fp16 numbers
  // n 2^-24 (bits 0..3 of a half) and n 2^-20 (bits 4..7): one AND for two, no
  // conversion.  So q is fp16 too, each head scaled by a power of two to a
  // largest magnitude in [2^14, 2^15), the channels met by n 2^-20 by 2^-4
  // more: its 8 bits are kept exactly down to 2^-31 of that, or 2^-27.  The
  // instruction keeps 25 bits below the exponents of the largest query and of
  // 2^-14 (as in the second product, below), so a channel's product loses less
  // than 2^-15 of the largest |q| of its group: with one channel 64 times the
  // others the lse is off by 7e-5, at like magnitudes by 1e-6.  A nibble is c +
  // 8: each group's sum is short of -8 times its sum of q, and the logit of -8 sum_g
  // ks_g sum q_g: one product of the scales with that sum in three bf16 parts
  // (24 bits), k slots 0..3 the high parts of groups 0..3, 4..7 the middle,
  // 8..11 the low ones.
  uint32_t qf[8][2];  // bf16: B fragments, head tq
  uint32_t off_b[2] = {0u, 0u};
  float sl2[2] = {p.scale_log2, p.scale_log2};  // base-2 scale of the raw logits of heads ta and ta + 1
  const uint32_t q_s = smem_u32(s_q) + tq * 256 + c * 16;
  if constexpr (kInt4) {
    uint32_t mx = max_u16x2(max_u16x2(qw.x & 0x7FFF7FFFu, qw.y & 0x7FFF7FFFu), max_u16x2(qw.z & 0x7FFF7FFFu, qw.w & 0x7FFF7FFFu));
    mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const uint32_t e = mx >> 7;  // biased exponent of the head's largest magnitude
    const uint32_t fe = e == 255u || mx == 0u ? 127u : min(268u - e, 254u);
    const float f = __uint_as_float(fe << 23);  // 2^(fe - 127)
    const float x0 = lo_f(qw.x) * f, x1 = hi_f(qw.x) * f, x4 = lo_f(qw.z) * f, x5 = hi_f(qw.z) * f;
    const float x2 = lo_f(qw.y) * f, x3 = hi_f(qw.y) * f, x6 = lo_f(qw.w) * f, x7 = hi_f(qw.w) * f;
    float sum = ((x0 + x1) + (x2 + x3)) + ((x4 + x5) + (x6 + x7));
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);  // over the group's 4 threads
    const int hd = tid >> 4, x = tid & 15;  // channels 32 (x / 4) + 8 (x % 4) ..
    *reinterpret_cast<uint4*>(s_q + hd * 64 + x * 4) =
        make_uint4(pack_f16x2(x0, x1), pack_f16x2(x2 * 0x1p-4f, x3 * 0x1p-4f), pack_f16x2(x4, x5), pack_f16x2(x6 * 0x1p-4f, x7 * 0x1p-4f));
    if ((x & 3) == 0) s_off[hd][x >> 2] = sum * -0x1p-21f;  // -8 * 2^-24
    // 2^24 / f; infinity where q passes 2^118 and it overflows: the outputs are then not finite
    if (x == 0) s_sl2[hd] = p.scale_log2 * __uint_as_float(min(278u - fe, 255u) << 23);
    __syncthreads();
    sl2[0] = s_sl2[ta];
    sl2[1] = s_sl2[ta + 1];
    const float p0 = s_off[tq][2 * (c & 1)], p1 = s_off[tq][2 * (c & 1) + 1];
    const uint32_t hi = pack_bf16x2(p0, p1);
    const float m0 = p0 - lo_f(hi), m1 = p1 - hi_f(hi);
    const uint32_t mid = pack_bf16x2(m0, m1);
    off_b[0] = c < 2 ? hi : mid;
    off_b[1] = c < 2 ? pack_bf16x2(m0 - lo_f(mid), m1 - hi_f(mid)) : 0u;
  } else {
    const uint32_t* q32 = reinterpret_cast<const uint32_t*>(p.q + (qh0 + (tq < g ? tq : 0)) * kHeadDim);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      qf[kk][0] = tq < g ? __ldg(q32 + kk * 8 + c) : 0u;
      qf[kk][1] = tq < g ? __ldg(q32 + kk * 8 + 4 + c) : 0u;
    }
  }

  Acc a;
#pragma unroll
  for (int dm = 0; dm < 8; ++dm) a.o[dm][0] = a.o[dm][1] = a.o[dm][2] = a.o[dm][3] = 0.f;
  a.sums[0] = a.sums[1] = a.sums[2] = a.sums[3] = 0.f;
  a.m[0] = a.m[1] = a.thr[0] = a.thr[1] = a.r[0] = a.r[1] = kNegInf;
  a.l[0] = a.l[1] = 0.f;
  // 4 bit: the second product's weights p vs are fp16 (11 bits; a bf16 weight
  // would cost as much accuracy as the final rounding): p, and vs divided by
  // vn, a power of two above the group's largest scale in this warp so far (at
  // least 2^-100; lane l keeps the vn of group l % 4).  That holds while every
  // scale is at least 2^-10 vn: vs / vn is then exact, the heaviest token has p
  // >= 2^7, so the weights' sum is at least 2^-3 vn, and what fp16's least step
  // takes from the small weights of a warp's 1024 tokens, at most 2 * 2^-25 vn
  // each, is 2^-11 of it.  From the first step with a smaller scale on (a row
  // of zeros has none) the warp forms its weights in fp32 and each step has
  // factors of its own (below).  least: a bound below the scales of the
  // lane's tokens, looked after when a step leaves [2^-8 vn, vn).
  constexpr float kFlat = 0x1p-8f, kWide = 0x1p-10f;
  constexpr uint32_t kFlat16 = 0x1C001C00u;  // kFlat in fp16; 0x2000 above it is 1
  uint32_t vn_bits = 27u << 23;
  float least = __int_as_float(0x7f800000);
  bool v_nan = false;
  uint32_t slot = 0;

  // Step st of the warp.  False, with nothing added: the scales have come to lie
  // too far apart for this form of it, the step is taken again in the wide one.
  auto step = [&](auto wide, int st) {
    constexpr bool kWideStep = decltype(wide)::value;
    cp_async_wait<kStages - 1>();
    __syncwarp();
    int nv[kStep];
    uint32_t part = lds32(rows_s + st * kStep * 4);
    if constexpr (kStep == 2) part |= lds32(rows_s + st * 8 + 4);
    part &= kPartial;
    bool some = true;
#pragma unroll
    for (int h = 0; h < kStep; ++h) nv[h] = kTileTokens;
    if (part) {
      some = false;
#pragma unroll
      for (int h = 0; h < kStep; ++h) {
        nv[h] = s_valid[warp][st * kStep + h];
        some |= nv[h] > 0;
      }
    }
    if (some) {
      const uint32_t base = ring + slot;
      float s[kStep][4], pr[kStep][4];
      if constexpr (kInt4) {
        // the scales, each unpacked once for the warp: lane l the key scales of
        // token l / 2, groups 2 (l % 2) and the next; and group l % 4's value
        // scales of a token pair of the second product's slots
        const int tp = (tq & 3) + 8 * (tq >> 2), tp2 = tp ^ 5;  // ((tp & 3) ^ 1) + 4
        float v[kStep][2];
        uint32_t vx[kStep], off = 0u;
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
          const uint32_t kw = lds32(base + h * R::kTileBytes + 2048 + lane * 4);
          v[h][0] = __uint_as_float(lds16(base + h * R::kTileBytes + 2176 + tp * 8 + c * 2) << 16);
          v[h][1] = __uint_as_float(lds16(base + h * R::kTileBytes + 2176 + tp2 * 8 + c * 2) << 16);
          sts64(scales + h * R::kScaleBytes + lane * 8, lo_f(kw), hi_f(kw));
          const float inv_vn = __uint_as_float((254u << 23) - vn_bits);
          vx[h] = pack_f16x2(v[h][0] * inv_vn, v[h][1] * inv_vn);
          off |= vx[h] - kFlat16;  // NaN too is behind 1; a borrow comes only from a half that is off
        }
        if (__any_sync(0xffffffffu, (off & 0xE000E000u) != 0u)) {
          // a scale that is not finite makes its group NaN whatever its
          // weight: noted here, and kept out of the products
          const float vn = __uint_as_float(vn_bits);
          uint32_t mb = 0u;
          if (st > 0) least = fminf(least, vn * kFlat);  // the steps that did not come here
#pragma unroll
          for (int h = 0; h < kStep; ++h) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if ((i ? tp2 : tp) < nv[h]) least = fminf(least, v[h][i]);
              if (!(v[h][i] < 0x1p127f)) {
                v_nan = true;
                v[h][i] = 0.f;
              }
              if (v[h][i] > 0.f) mb = max(mb, __float_as_uint(v[h][i]));
            }
          }
          // a larger one moves the group's sums to a power of two with some room above it
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, off));
          const uint32_t e = mb >= vn_bits ? min((mb >> 23) + 3u, 253u) : vn_bits >> 23;
          const float down = vn * __uint_as_float((254u - e) << 23);
          vn_bits = e << 23;
          const float mine = __shfl_sync(0xffffffffu, down, tq & 3);
#pragma unroll
          for (int i = 0; i < 4; ++i) a.sums[i] *= mine;
#pragma unroll
          for (int dm = 0; dm < 8; ++dm) {
            const float dg = __shfl_sync(0xffffffffu, down, dm >> 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) a.o[dm][i] *= dg;
          }
          if (!kWideStep && __any_sync(0xffffffffu, least < __uint_as_float(vn_bits) * kWide)) return false;
#pragma unroll
          for (int h = 0; h < kStep; ++h) {
            const float inv_vn = __uint_as_float((254u << 23) - vn_bits);
            vx[h] = pack_f16x2(v[h][0] * inv_vn, v[h][1] * inv_vn);
          }
        }
#pragma unroll
        for (int h = 0; h < kStep; ++h) sts32(scales + h * R::kScaleBytes + 256 + lane * 4, vx[h]);
        __syncwarp();
        uint4 wa[kStep], wb[kStep], sa[kStep], sb[kStep];
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
          const uint32_t tb = base + h * R::kTileBytes, ka = tb + t0 * 64 + ((c ^ (t0 & 2)) << 4);
          wa[h] = lds128(ka);
          wb[h] = lds128(ka + 512);
          sa[h] = lds128(scales + h * R::kScaleBytes + t0 * 16);
          sb[h] = lds128(scales + h * R::kScaleBytes + t1 * 16);
          const uint32_t ra = lds32(tb + 2048 + t0 * 8 + (c & 1) * 4), rb = lds32(tb + 2048 + t1 * 8 + (c & 1) * 4);
          mma_bf16_new(s[h], ra, rb, ra, rb, off_b[0], off_b[1]);
        }
#pragma unroll
        for (int G = 0; G < 4; ++G) {
          const uint4 q = lds128(q_s + G * 64);
          float d[kStep][4];
          uint32_t ha[kStep], hb[kStep];
#pragma unroll
          for (int h = 0; h < kStep; ++h) {
            const uint32_t ka = part_of(wa[h], G), kb = part_of(wb[h], G);
            // the upper bytes of both halves, by the multiplier: the logic
            // unit is the busiest here
            ha[h] = __umulhi(ka, p.two24);
            hb[h] = __umulhi(kb, p.two24);
            mma_f16_new(d[h], ka & 0x000F000Fu, kb & 0x000F000Fu, ka & 0x00F000F0u, kb & 0x00F000F0u, q.x, q.y);
          }
#pragma unroll
          for (int h = 0; h < kStep; ++h)
            mma_f16_16816(d[h], ha[h] & 0x000F000Fu, hb[h] & 0x000F000Fu, ha[h] & 0x00F000F0u, hb[h] & 0x00F000F0u, q.z, q.w);
#pragma unroll
          for (int h = 0; h < kStep; ++h) {
            const float fa = __uint_as_float(part_of(sa[h], G)), fb = __uint_as_float(part_of(sb[h], G));
            s[h][0] = fmaf(fa, d[h][0], s[h][0]);
            s[h][1] = fmaf(fa, d[h][1], s[h][1]);
            s[h][2] = fmaf(fb, d[h][2], s[h][2]);
            s[h][3] = fmaf(fb, d[h][3], s[h][3]);
          }
        }
      } else {
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
        const int kr = lane & 15, khi = lane >> 4;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t box = base + (kk < 4 ? 0u : (uint32_t)kHalfBox);
          const int ch = (kk & 3) * 2 + khi;
          uint32_t a0, a1, a2, a3;
          ldmatrix_x4(box + kr * 128 + ((ch ^ (kr & 7)) << 4), a0, a1, a2, a3);
          if (kk & 1)
            mma_bf16_16816(sb, a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
          else
            mma_bf16_16816(sa, a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[0][i] = sa[i] + sb[i];
      }
      if (part) {
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
          if (t0 >= nv[h]) s[h][0] = s[h][1] = kNegInf;
          if (t1 >= nv[h]) s[h][2] = s[h][3] = kNegInf;
        }
      }
      if constexpr (kAcc) {  // the logits of the tiles, for the weights once lse is known
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
          if (nv[h] > 0) {
            const int tile = (warp + kWarps * st) * kStep + h;
            const int64_t slot0 = ((int64_t)pair * p.k << lbs) + (int64_t)((j0 << ltpb) + tile) * kTileTokens;
            float* z0 = p.z + (slot0 + t0) * g + ta;
            float* z1 = p.z + (slot0 + t1) * g + ta;
            if (!(g & 1)) {
              if (ta < g) {
                *reinterpret_cast<float2*>(z0) = make_float2(s[h][0] * sl2[0], s[h][1] * sl2[1]);
                *reinterpret_cast<float2*>(z1) = make_float2(s[h][2] * sl2[0], s[h][3] * sl2[1]);
              }
            } else {
              if (ta < g) {
                z0[0] = s[h][0] * sl2[0];
                z1[0] = s[h][2] * sl2[0];
              }
              if (ta + 1 < g) {
                z0[1] = s[h][1] * sl2[1];
                z1[1] = s[h][3] * sl2[1];
              }
            }
          }
        }
      }
      weigh<kInt4>(a, s, sl2, pr);
      if constexpr (kWideStep) {
        // Scales far apart, so a token that weighs nothing must not set the
        // others' factor, nor one head's tokens another's: the products p vs /
        // vn in fp32, and per head and group of this step a power of two that
        // takes the largest of them to [2^14, 2^15) before they become fp16.
        // The step's sums start from zero, every code as n 2^-18, and join the
        // running ones in fp32, whose range ends 2^80 below vn.
        // 32 x 8 pairs of 4096 tokens, every 64th with a scale of 10^-4: 57.3 us,
        // every step being of this kind, 41.7 without.
#pragma unroll
        for (int G = 0; G < 4; ++G) {
          const float inv = __shfl_sync(0xffffffffu, __uint_as_float((254u << 23) - vn_bits), G);
          float w[kStep][4], top[2] = {0.f, 0.f};
#pragma unroll
          for (int h = 0; h < kStep; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float vs = __uint_as_float(lds16(base + h * R::kTileBytes + 2176 + (i < 2 ? t0 : t1) * 8 + G * 2) << 16);
              w[h][i] = pr[h][i] * (vs < 0x1p127f ? vs * inv : 0.f);  // not finite: noted above
              top[i & 1] = fmaxf(top[i & 1], w[h][i]);
            }
          }
          float up[2], down[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], off));
            const uint32_t e = max(__float_as_uint(top[j]) >> 23, 15u);  // biased exponent; 255 (not finite) at most
            up[j] = __uint_as_float((268u - e) << 23);
            down[j] = __uint_as_float((e - 14u) << 23);
          }
          float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f}, ds[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < kStep; ++h) {
            const uint32_t p0 = movmatrix_trans(pack_f16x2(w[h][0] * up[0], w[h][1] * up[1]));
            const uint32_t p1 = movmatrix_trans(pack_f16x2(w[h][2] * up[0], w[h][3] * up[1]));
            const uint32_t sel = (G & 1) ? 0x7632u : 0x5410u;
            uint32_t x[4];  // value codes, as below
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = 4 * i + ((i & 1) ? c ^ 1 : c);
              x[i] = lds32(base + h * R::kTileBytes + 1024 + t * 64 + (((tq >> 1) ^ (t & 2)) << 4) + (tq & 1) * 8 + (G >> 1) * 4);
            }
            const uint32_t u01 = __byte_perm(x[0], x[1], sel), u23 = __byte_perm(x[2], x[3], sel);
            const uint32_t one = tq == G ? 0x3C003C00u : 0u;
            mma_f16_16816(d0, (u01 << 6) & 0x03C003C0u, (u01 << 2) & 0x03C003C0u, (u23 << 6) & 0x03C003C0u,
                          (u23 << 2) & 0x03C003C0u, p0, p1);
            mma_f16_16816(d1, (u01 >> 2) & 0x03C003C0u, (u01 >> 6) & 0x03C003C0u, (u23 >> 2) & 0x03C003C0u,
                          (u23 >> 6) & 0x03C003C0u, p0, p1);
            mma_f16_16816(ds, one, 0u, one, 0u, p0, p1);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = down[j] * 0x1p-6f;
            a.o[2 * G][j] = fmaf(d0[j], down[j], a.o[2 * G][j]);
            a.o[2 * G][2 + j] = fmaf(fmaf(d0[2 + j], 16.f, d0[j]), f, a.o[2 * G][2 + j]);
            a.o[2 * G + 1][j] = fmaf(d1[j], down[j], a.o[2 * G + 1][j]);
            a.o[2 * G + 1][2 + j] = fmaf(fmaf(d1[2 + j], 16.f, d1[j]), f, a.o[2 * G + 1][2 + j]);
            a.sums[j] = fmaf(ds[j], down[j], a.sums[j]);
          }
        }
      } else if constexpr (kInt4) {
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
          const uint32_t tb = base + h * R::kTileBytes, sc = scales + h * R::kScaleBytes + 256;
          const uint32_t p0 = movmatrix_trans(pack_f16x2(pr[h][0], pr[h][1]));
          const uint32_t p1 = movmatrix_trans(pack_f16x2(pr[h][2], pr[h][3]));
          const uint4 va = lds128(sc + c * 16), vb = lds128(sc + 64 + c * 16);
          const uint32_t pb[4][2] = {{hmul2(p0, va.x), hmul2(p1, vb.x)}, {hmul2(p0, va.y), hmul2(p1, vb.y)},
                                     {hmul2(p0, va.z), hmul2(p1, vb.z)}, {hmul2(p0, va.w), hmul2(p1, vb.w)}};
          // value codes: the lane's 4 channels of each group, of its 4 tokens.
          // Two tokens' halfwords side by side; of a byte of each, the low
          // nibbles (n 2^-18) for one channel, and both (n 2^-24 + n' 2^-20)
          // for the next, whose sum the first channel's comes off at the end.
          // So does 8 times the weights' sum, taken by a product with a row of
          // ones for each group (a warp's tiles are few enough for the
          // difference to keep its bits).
          // The instruction lines its products up by the operands' exponents
          // and keeps 25 bits below the largest (measured); a subnormal's is
          // that of 2^-14, so where a code stands decides what is left of the
          // light tokens beside a heavy one.  n 2^-18 keeps them down to 2^-21
          // of its weight, n 2^-24 would to 2^-15: where the heavy code is 0 the
          // output was then off by up to 2^-12 of a step.  32 x 8 pairs of 4096
          // tokens take 0.8 us more for it.
          uint2 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 4 * i + ((i & 1) ? c ^ 1 : c);
            x[i] = lds64(tb + 1024 + t * 64 + (((tq >> 1) ^ (t & 2)) << 4) + (tq & 1) * 8);
          }
#pragma unroll
          for (int G = 0; G < 4; ++G) {
            const uint32_t sel = (G & 1) ? 0x7632u : 0x5410u;
            const uint32_t u01 = __byte_perm(G < 2 ? x[0].x : x[0].y, G < 2 ? x[1].x : x[1].y, sel);
            const uint32_t u23 = __byte_perm(G < 2 ? x[2].x : x[2].y, G < 2 ? x[3].x : x[3].y, sel);
            const uint32_t l01 = u01 & 0x00FF00FFu, l23 = u23 & 0x00FF00FFu;
            const uint32_t h01 = __byte_perm(u01, 0u, 0x4341), h23 = __byte_perm(u23, 0u, 0x4341);
            const uint32_t one = tq == G ? 0x3C003C00u : 0u;
            mma_f16_16816(a.o[2 * G], (u01 << 6) & 0x03C003C0u, l01, (u23 << 6) & 0x03C003C0u, l23, pb[G][0], pb[G][1]);
            mma_f16_16816(a.o[2 * G + 1], (h01 << 6) & 0x03C003C0u, h01, (h23 << 6) & 0x03C003C0u, h23, pb[G][0], pb[G][1]);
            mma_f16_16816(a.sums, one, 0u, one, 0u, pb[G][0], pb[G][1]);
          }
        }
      } else {
        // weights as the sum of two bf16 numbers (16 bits): a single bf16
        // weight would cost as much accuracy as the final rounding
        const uint32_t h0 = pack_bf16x2(pr[0][0], pr[0][1]), h1 = pack_bf16x2(pr[0][2], pr[0][3]);
        const uint32_t pb0 = movmatrix_trans(h0), pb1 = movmatrix_trans(h1);
        const uint32_t pl0 = movmatrix_trans(pack_bf16x2(pr[0][0] - lo_f(h0), pr[0][1] - hi_f(h0)));
        const uint32_t pl1 = movmatrix_trans(pack_bf16x2(pr[0][2] - lo_f(h1), pr[0][3] - hi_f(h1)));
        const uint32_t mlo = tok_mask(ta, nv[0]), mhi = tok_mask(ta + 8, nv[0]);
        const int vt = (lane & 7) + ((lane >> 4) << 3), vsel = (lane >> 3) & 1;
#pragma unroll
        for (int dm = 0; dm < 8; ++dm) {
          const int d0 = dm * 16 + vsel * 8;
          const uint32_t box = base + 2u * kHalfBox + (d0 < 64 ? 0u : (uint32_t)kHalfBox);
          const int ch = (d0 & 63) >> 3;
          uint32_t a0, a1, a2, a3;
          ldmatrix_x4_trans(box + vt * 128 + ((ch ^ (vt & 7)) << 4), a0, a1, a2, a3);
          if (part) {
            a0 &= mlo;
            a1 &= mlo;
            a2 &= mhi;
            a3 &= mhi;
          }
          mma_bf16_16816(a.o[dm], a0, a1, a2, a3, pb0, pb1);
          mma_bf16_16816(a.o[dm], a0, a1, a2, a3, pl0, pl1);
        }
      }
    }
    __syncwarp();
    issue(st + kStages, slot);
    slot = slot == (kStages - 1) * R::kStageBytes ? 0u : slot + R::kStageBytes;
    return true;
  };
  int st = 0;
  while (st < n_w && step(std::false_type{}, st)) ++st;
  // A loop of its own: in the other's it would cost that one 3% where it is
  // never taken (24 x 8 pairs of 16384 tokens: 108.3 us, 112 in one loop).
  if constexpr (kInt4) {
    for (; st < n_w; ++st) step(std::true_type{}, st);
  }
  cp_async_wait<0>();

#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    a.l[0] += __shfl_xor_sync(0xffffffffu, a.l[0], off);
    a.l[1] += __shfl_xor_sync(0xffffffffu, a.l[1], off);
  }
  __syncthreads();  // every warp is done with its ring; the combine area reuses it
  float* comb = reinterpret_cast<float*>(smem);  // [warp][head][kRowPad]
  {
    float* w0 = comb + ((warp * kMaxGroup) + ta) * kRowPad;
    if constexpr (kInt4) {
      // o[2G + e][i]: channels 32 G + 4 tq + 2 e (and, with it, the next), head
      // ta + (i & 1); the weights' sums of group G sit in the lanes of row G
      const uint32_t nans = __ballot_sync(0xffffffffu, v_nan);  // lanes l = c (mod 4): group c
      const float mine = (nans & (0x11111111u << c)) ? __int_as_float(0x7FFFFFFF) : __uint_as_float(vn_bits);
#pragma unroll
      for (int G = 0; G < 4; ++G) {
        const float vn = __shfl_sync(0xffffffffu, mine, G);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float off = -8.f * __shfl_sync(0xffffffffu, a.sums[j], G * 4 + c);
          const float x0 = a.o[2 * G][j] * 0x1p18f, x2 = a.o[2 * G + 1][j] * 0x1p18f;
          const float x1 = fmaf(a.o[2 * G][2 + j], 0x1p20f, x0 * -0x1p-4f), x3 = fmaf(a.o[2 * G + 1][2 + j], 0x1p20f, x2 * -0x1p-4f);
          *reinterpret_cast<float4*>(w0 + j * kRowPad + 32 * G + 4 * tq) =
              make_float4((x0 + off) * vn, (x1 + off) * vn, (x2 + off) * vn, (x3 + off) * vn);
        }
      }
    } else {
#pragma unroll
      for (int dm = 0; dm < 8; ++dm) {
        const int d = dm * 16 + tq;
        w0[d] = a.o[dm][0];
        w0[kRowPad + d] = a.o[dm][1];
        w0[d + 8] = a.o[dm][2];
        w0[kRowPad + d + 8] = a.o[dm][3];
      }
    }
  }
  if (lane < 4) {
    s_m[warp][2 * lane] = a.r[0];
    s_m[warp][2 * lane + 1] = a.r[1];
    s_l[warp][2 * lane] = a.l[0];
    s_l[warp][2 * lane + 1] = a.l[1];
  }
  __syncthreads();
  auto write_lse = [&](int j, float den, float M) {
    // in the sum's own units: M + lead is the reference logit
    const float l2 = den == 0.f ? kNegInf : (M + kLead<kInt4>) + log2f(den * (kInt4 ? 0x1p-7f : 0x1p30f));
    if (p.lse) p.lse[qh0 + j] = l2 * 0.6931471805599453f;
    if (kAcc) p.lse2[qh0 + j] = l2;
    s_inv[j] = den == 0.f ? 0.f : __frcp_rn(den);
  };
  if (tid < g) {  // per head: the maximum over the warps, each warp's weight, the sum
    const int j = tid;
    float M = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][j]);
    float den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      // a warp without a token (its sum is zero) weighs nothing; a NaN sum stays one
      const float e = s_l[w][j] == 0.f ? 0.f : exp2f(s_m[w][j] - M);
      s_ww[w][j] = e;
      den += e * s_l[w][j];
    }
    s_cm[j] = M;
    s_cden[j] = den;
    if (nchunks == 1) write_lse(j, den, M);
  }
  __syncthreads();
  auto combined = [&](int j) {
    float num = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) num += s_ww[w][j] * comb[(w * kMaxGroup + j) * kRowPad + tid];
    return num;
  };
  auto finish = [&](int j, float num) { p.out[(qh0 + j) * kHeadDim + tid] = __float2bfloat16_rn(num * s_inv[j]); };
  if (nchunks == 1) {
#pragma unroll 2
    for (int j = 0; j < g; ++j) finish(j, combined(j));
    __syncthreads();  // the next pair's ring takes the combine area
    continue;
  }

  // this chunk's partial; the pair's last chunk merges all of them
  float* part = p.partials + ((int64_t)pair * p.max_chunks + chunk) * g * kPartStride;
#pragma unroll 1
  for (int j = 0; j < g; ++j) {
    part[j * kPartStride + tid] = combined(j);
    if (tid == 0) {
      part[j * kPartStride + kHeadDim] = s_cm[j];
      part[j * kPartStride + kHeadDim + 1] = s_cden[j];
    }
  }
  // the barrier orders every thread's partial before thread 0's release, its
  // acquire (of the other chunks' releases) before what the others read
  __syncthreads();
  if (tid == 0) s_last = (count_chunk(&p.counters[pair]) == (unsigned)(nchunks - 1));
  __syncthreads();
  if (!s_last) continue;
  if (tid == 0) p.counters[pair] = 0u;  // ready for the next call
  // The partials are staged in shared memory, a batch of chunks at a time;
  // thread j < g folds head j's maxima and sums and leaves one weight per
  // (chunk, head); every thread folds its output channel.
  const int rec = g * kPartStride;
  const int per_batch = R::kPipe / (4 * rec);
  const float4* src4 = reinterpret_cast<const float4*>(p.partials + (int64_t)pair * p.max_chunks * rec);
  const float* stage = reinterpret_cast<const float*>(smem);
  const uint32_t stage_s = smem_u32(smem);
  float num[kMaxGroup];
#pragma unroll
  for (int j = 0; j < kMaxGroup; ++j) num[j] = 0.f;
  if (tid < g) {
    s_mr[tid] = kNegInf;
    s_den[tid] = 0.f;
  }
  for (int cb = 0; cb < nchunks; cb += per_batch) {
    const int nbat = min(per_batch, nchunks - cb);
    const int n4 = nbat * rec / 4;
    const float4* s4 = src4 + (int64_t)cb * (rec / 4);
    for (int i = tid; i < n4; i += kThreads) cp_async16(stage_s + 16u * (uint32_t)i, s4 + i, 16u);
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    if (tid < g) {
      const int j = tid;
      float Mb = kNegInf;
#pragma unroll 4
      for (int cc = 0; cc < nbat; ++cc) Mb = fmaxf(Mb, stage[(cc * g + j) * kPartStride + kHeadDim]);
      const float Mr = s_mr[j];
      const float Mn = fmaxf(Mr, Mb);
      const float al = s_den[j] == 0.f ? 0.f : exp2f(Mr - Mn);
      float dd = s_den[j] * al;
#pragma unroll 4
      for (int cc = 0; cc < nbat; ++cc) {
        const float* r = stage + (cc * g + j) * kPartStride;
        const float e = r[kHeadDim + 1] == 0.f ? 0.f : exp2f(r[kHeadDim] - Mn);
        s_w[cc * g + j] = e;
        dd += e * r[kHeadDim + 1];
      }
      s_a[j] = al;
      s_mr[j] = Mn;
      s_den[j] = dd;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxGroup; ++j)
      if (j < g) num[j] *= s_a[j];
#pragma unroll 2
    for (int cc = 0; cc < nbat; ++cc) {
      const float* rc = stage + cc * g * kPartStride + tid;
#pragma unroll
      for (int j = 0; j < kMaxGroup; ++j)
        if (j < g) num[j] += s_w[cc * g + j] * rc[j * kPartStride];
    }
    __syncthreads();  // the next batch overwrites the staging area and the weights
  }
  if (tid < g) write_lse(tid, s_den[tid], s_mr[tid]);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMaxGroup; ++j)
    if (j < g) finish(j, num[j]);
  }
}

// The weights of the attended tokens, once every lse is known: one thread per
// four consecutive tokens of a kept block adds sum_j 2^(z_j - lse2_j) to each
// one's running sum.  A kept token has one slot, so the addition is an atomic
// only where a block is listed twice (it then counts twice).  The logits come
// from L2; four tokens a thread keep one wave's worth of them in flight.
template <int G>
__global__ void __launch_bounds__(256) kv_weights_kernel(KvAttnParams p) {
  pdl_wait();
  const int lbs = 31 - __clz(p.bs), quads = p.k << (lbs - 2);  // of a pair
  const int ctas = (quads + 255) >> 8;
  const int pair = blockIdx.x / ctas;
  const int i = (blockIdx.x - pair * ctas) * 256 + threadIdx.x, j = i >> (lbs - 2);
  const int b = pair / p.Hkv, h = pair - b * p.Hkv;
  if (j >= p.k) return;
  const int blk = p.sel_idx ? __ldg(p.sel_idx + (int64_t)pair * p.k_row + j) : j;
  const int L = __ldg(p.seq_lens + b);
  const int cnt = p.sel_idx ? __ldg(p.sel_cnt + pair) : p.k;
  float z[4 * G], l[G];
  const float4* z4 = reinterpret_cast<const float4*>(p.z + (((int64_t)pair * p.k << lbs) + 4 * (int64_t)i) * G);
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const float4 v = __ldcg(z4 + q);
    z[4 * q] = v.x;
    z[4 * q + 1] = v.y;
    z[4 * q + 2] = v.z;
    z[4 * q + 3] = v.w;
    l[q] = __ldcg(p.lse2 + (int64_t)b * p.Hq + (int64_t)h * G + q);
  }
  if (j >= cnt || L < 1 || L > p.kv.Lcap || blk < 0 || blk >= (L + p.bs - 1) >> lbs) return;
  if (p.kv.pages.table) {  // a bad page: nothing was attended
    const int page = __ldg(p.kv.pages.table + (int64_t)b * p.kv.pages.max_blocks + blk);
    if (page < 0 || page >= p.kv.pages.num_pages) return;
  }
  const int t0 = (blk << lbs) + ((4 * i) & (p.bs - 1));
  float* acc = p.acc + (int64_t)pair * p.kv.Lcap + t0;
  float w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    w[u] = 0.f;
#pragma unroll
    for (int q = 0; q < G; ++q) w[u] += exp2f(z[u * G + q] - l[q]);
  }
  if (t0 + 4 <= L && (reinterpret_cast<uintptr_t>(acc) & 15u) == 0) {  // one 16-byte reduction in place of four
    atomicAdd(reinterpret_cast<float4*>(acc), make_float4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (t0 + u < L) atomicAdd(acc + u, w[u]);
  }
}

static cudaError_t launch_kv_weights(const KvAttnParams& p, cudaStream_t s) {
  const int64_t quads = (int64_t)p.k * p.bs / 4;
  const dim3 grid((unsigned)((int64_t)p.B * p.Hkv * ((quads + 255) / 256))), block(256);
  switch (p.g) {
    case 1: return launch_pdl(kv_weights_kernel<1>, grid, block, 0, s, p);
    case 2: return launch_pdl(kv_weights_kernel<2>, grid, block, 0, s, p);
    case 3: return launch_pdl(kv_weights_kernel<3>, grid, block, 0, s, p);
    case 4: return launch_pdl(kv_weights_kernel<4>, grid, block, 0, s, p);
    case 5: return launch_pdl(kv_weights_kernel<5>, grid, block, 0, s, p);
    case 6: return launch_pdl(kv_weights_kernel<6>, grid, block, 0, s, p);
    case 7: return launch_pdl(kv_weights_kernel<7>, grid, block, 0, s, p);
    default: return launch_pdl(kv_weights_kernel<8>, grid, block, 0, s, p);
  }
}

template <bool kInt4, bool kAcc>
static cudaError_t launch_kv_attn_as(const KvAttnParams& p, cudaStream_t s) {
  const auto kernel = kv_attn_kernel<kInt4, kAcc>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), 16 + 2 * kInt4 + kAcc, Ring<kInt4>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3((unsigned)((p.slots + p.per - 1) / p.per)), dim3(kThreads), Ring<kInt4>::kSmem, s, p);
  return e != cudaSuccess || !kAcc ? e : launch_kv_weights(p, s);
}

cudaError_t launch_kv_attn(const KvAttnParams& p, cudaStream_t s) {
  if (p.kv.int4) return p.acc ? launch_kv_attn_as<true, true>(p, s) : launch_kv_attn_as<true, false>(p, s);
  return p.acc ? launch_kv_attn_as<false, true>(p, s) : launch_kv_attn_as<false, false>(p, s);
}

}  // namespace kin
