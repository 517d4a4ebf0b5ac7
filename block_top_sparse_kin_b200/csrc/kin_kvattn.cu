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
// Bounded by HBM: 144 bytes (4 bit) or 512 bytes (bf16) a token and pair
// against 4 g D flops.  A decode group has at most 8 heads, so the products
// are mma.sync m16n8k16 tiles of 16 tokens by 8 heads, fed per warp by a
// ring of asynchronous copies.
#include "kin_internal.cuh"

namespace kin {

namespace {

#define kNegInf (-__int_as_float(0x7f800000))

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRowPad = kHeadDim + 4;
constexpr int kHalfBox = 16 * 64 * 2;

template <bool kInt4>
struct Ring {
  // bf16: K0 K1 V0 V1 half tiles of 16 rows x 64 channels.  4 bit: 16 rows of
  // 64 bytes of key codes, of value codes, then 16 x 4 scales of each.
  static constexpr int kStageBytes = kInt4 ? 2 * 16 * kCodeBytes + 2 * 16 * kGroups * 2 : 4 * kHalfBox;
  static constexpr int kStages = kInt4 ? 4 : 2;
  static constexpr int kPipe = kWarps * kStages * kStageBytes;
  static constexpr int kComb = kWarps * kMaxGroup * kRowPad * 4;
  static constexpr int kSmem = (kPipe > kComb ? kPipe : kComb) + 1024;
};

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
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

// The product sums' state of a warp: O^T fragments, running maximum and sum
// of its two head columns.
struct Acc {
  float o[8][4];
  float m0, m1, l0, l1;
};

// Running maximum over the tile and the tile's weights; rescales the sums
// when some maximum grew (then the whole warp does).  s holds the base-2
// logits (rows tq, tq + 8; heads ta, ta + 1), -inf where there is no token.
__device__ __forceinline__ void online_softmax(Acc& a, const float (&s)[4], float (&p)[4]) {
  float x0 = fmaxf(s[0], s[2]), x1 = fmaxf(s[1], s[3]);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
  }
  const float mn0 = fmaxf(a.m0, x0), mn1 = fmaxf(a.m1, x1);
  if (__any_sync(0xffffffffu, mn0 != a.m0 || mn1 != a.m1)) {
    const float al0 = exp2f(a.m0 - mn0), al1 = exp2f(a.m1 - mn1);
    a.l0 *= al0;
    a.l1 *= al1;
#pragma unroll
    for (int dm = 0; dm < 8; ++dm) {
      a.o[dm][0] *= al0;
      a.o[dm][1] *= al1;
      a.o[dm][2] *= al0;
      a.o[dm][3] *= al1;
    }
    a.m0 = mn0;
    a.m1 = mn1;
  }
  p[0] = exp2f(s[0] - a.m0);
  p[1] = exp2f(s[1] - a.m1);
  p[2] = exp2f(s[2] - a.m0);
  p[3] = exp2f(s[3] - a.m1);
  a.l0 += p[0] + p[2];
  a.l1 += p[1] + p[3];
}

}  // namespace

template <bool kInt4, bool kAcc>
__global__ void __launch_bounds__(kThreads, kInt4 ? 4 : 3) kv_attn_kernel(KvAttnParams p) {
  using R = Ring<kInt4>;
  constexpr int kStages = R::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float s_m[kWarps][kMaxGroup], s_l[kWarps][kMaxGroup];
  __shared__ int s_last;
  constexpr int kMaxMergeWeights = R::kPipe / (4 * kPartStride);
  __shared__ float s_mr[kMaxGroup], s_den[kMaxGroup], s_a[kMaxGroup], s_w[kMaxMergeWeights];
  __shared__ float s_ww[kWarps][kMaxGroup], s_cm[kMaxGroup], s_cden[kMaxGroup];

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = p.g, bs = p.bs, Lcap = p.kv.Lcap;
  pdl_wait();  // the selection comes from the select kernels
  pdl_trigger_early();
  const int tpb = bs / kTileTokens;
  const int64_t pair = blockIdx.x / p.max_chunks;
  const int chunk = (int)(blockIdx.x - pair * p.max_chunks);
  // lane l's tile of this warp (tile warp + W l of the chunk): its block index
  // is requested before the length and count, whose round trip it would follow
  int blk = -1;
  {
    const int t = warp + kWarps * lane;
    const int j = chunk * p.chunk_blocks + t / tpb;
    if (t < p.chunk_blocks * tpb && j < p.k) blk = p.sel_idx ? __ldg(p.sel_idx + pair * p.k_row + j) : j;
  }
  const int b = (int)(pair / p.Hkv), h = (int)(pair - (int64_t)b * p.Hkv);
  const int L = __ldg(p.seq_lens + b);
  const bool bad_len = L < 1 || L > Lcap;
  const int nb = bad_len ? 0 : (L + bs - 1) / bs;
  int cnt = p.sel_idx ? __ldg(p.sel_cnt + pair) : nb;
  if (bad_len) cnt = 0;
  if (cnt > p.k) cnt = p.k;
  const int nchunks = cnt > 0 ? (cnt + p.chunk_blocks - 1) / p.chunk_blocks : 0;
  const int j0 = chunk * p.chunk_blocks;
  const int ntiles = chunk < nchunks ? (min(j0 + p.chunk_blocks, cnt) - j0) * tpb : 0;
  const int64_t qh0 = (int64_t)b * p.Hq + (int64_t)h * g;
  if (cnt <= 0) {  // nothing to attend to: out = 0, lse = -inf
    if (chunk == 0) {
      for (int j = 0; j < g; ++j) p.out[(qh0 + j) * kHeadDim + tid] = __float2bfloat16_rn(0.f);
      if (tid < g) {
        if (p.lse) p.lse[qh0 + tid] = kNegInf;
        if (kAcc) p.lse2[qh0 + tid] = kNegInf;
      }
      if (bad_len && tid == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
    }
    return;
  }
  if (ntiles == 0) return;

  // this warp's tiles t = warp + W n; lane n holds tile n's row and valid rows
  const int n_w = warp < ntiles ? (ntiles - 1 - warp) / kWarps + 1 : 0;
  int64_t my_row = 0;
  int my_nvalid = 0;
  if (lane < n_w) {
    const int t = warp + kWarps * lane;
    const int tok = blk * bs + (t % tpb) * kTileTokens;
    int64_t row = -1;
    if (blk >= 0 && blk < nb && tok < L) row = kv_row(p.kv.pages, b, h, p.Hkv, Lcap, bs, tok);
    if (blk < 0 || blk >= nb || (tok < L && row < 0)) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
    my_nvalid = row < 0 ? 0 : min(kTileTokens, L - tok);
    my_row = row < 0 ? 0 : row;
  }

  // Q fragments (B operand): head n = lane / 4; channels by the tile's order
  uint32_t qf[8][2];
  const int n = lane >> 2, c = lane & 3;
  {
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(p.q + (qh0 + (n < g ? n : 0)) * kHeadDim);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      if constexpr (kInt4) {  // k slots 2c.. of step 2G + e: channels 32 G + 8 c + 4 e ..
        const int w = (kk >> 1) * 16 + 4 * c + 2 * (kk & 1);
        qf[kk][0] = n < g ? __ldg(qrow + w) : 0u;
        qf[kk][1] = n < g ? __ldg(qrow + w + 1) : 0u;
      } else {
        qf[kk][0] = n < g ? __ldg(qrow + kk * 8 + c) : 0u;
        qf[kk][1] = n < g ? __ldg(qrow + kk * 8 + 4 + c) : 0u;
      }
    }
  }

  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kStages * R::kStageBytes);
  auto issue = [&](int nt) {
    const int64_t row = (int64_t)(((uint64_t)(uint32_t)__shfl_sync(0xffffffffu, (int)(my_row >> 32), nt & 31) << 32) |
                                  (uint32_t)__shfl_sync(0xffffffffu, (int)(uint32_t)my_row, nt & 31));
    const int nv = __shfl_sync(0xffffffffu, my_nvalid, nt & 31);
    if (nt < n_w && nv > 0) {
      const uint32_t base = ring + (uint32_t)((nt % kStages) * R::kStageBytes);
      if constexpr (kInt4) {
        // 64 pieces of 16 bytes of key codes and of value codes.  Key row i of
        // the tile holds token (i & 8) + 4 (i & 1) + (i & 7) / 2, so that the
        // tile's k slots 2c, 2c + 1 of the second product are tokens c, c + 4
        // (and 8 + c, 12 + c); the value rows stay in token order, their
        // pieces 2 and 3 swapped with 0 and 1 in every second pair of rows.
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = (lane >> 2) + 8 * i, col = lane & 3;
          const int kr = (t & 8) | ((t & 3) << 1) | ((t >> 2) & 1);
          const int64_t src = (row + (t < nv ? t : 0)) * kCodeBytes + col * 16;
          const uint32_t bytes = t < nv ? 16u : 0u;
          cp_async16(base + kr * 64 + col * 16, p.kv.k + src, bytes);
          cp_async16(base + 1024 + t * 64 + ((col ^ (t & 2)) << 4), p.kv.v + src, bytes);
        }
        const int t = lane & 15;
        const uint16_t* sc = (lane < 16 ? p.kv.ks : p.kv.vs) + (row + (t < nv ? t : 0)) * kGroups;
        cp_async8(base + 2048 + lane * 8, sc, t < nv ? 8u : 0u);
      } else {
        const int64_t off0 = row * kHeadDim;
        const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(p.kv.k);
        const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.kv.v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int piece = lane + 32 * i;
          const int r = piece >> 4, cc = piece & 15;
          const uint32_t off = (uint32_t)((cc >> 3) * kHalfBox + r * 128 + (((cc & 7) ^ (r & 7)) << 4));
          const int64_t src = off0 + (int64_t)(r < nv ? r : 0) * kHeadDim + cc * 8;
          const uint32_t bytes = r < nv ? 16u : 0u;
          cp_async16(base + off, k + src, bytes);
          cp_async16(base + 2 * kHalfBox + off, v + src, bytes);
        }
      }
    }
    cp_async_commit();  // one group per tile, empty or not
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) issue(i);

  Acc a;
#pragma unroll
  for (int dm = 0; dm < 8; ++dm) a.o[dm][0] = a.o[dm][1] = a.o[dm][2] = a.o[dm][3] = 0.f;
  a.m0 = a.m1 = kNegInf;
  a.l0 = a.l1 = 0.f;
  const float sl2 = p.scale_log2;
  const int tq = lane >> 2, ta = 2 * c;

  // 4 bit: the codes enter the first product as 24 + c (16 + nibble, one
  // shift and one logic operation for two); each group's sum starts at -24
  // times the sum of its query channels, from a product with ones.
  float qs[4][2];
  // the second product's weights p vs are held in fp16 (11 bits; a bf16 weight
  // would cost as much accuracy as the final rounding), scaled by 2^14 / vn,
  // vn a power of two above the warp's largest value scale so far
  uint32_t vn_bits = 27u << 23;  // 2^-100
  float kf = 0x1p114f;
  if constexpr (kInt4) {
#pragma unroll
    for (int G = 0; G < 4; ++G) {
      float one[4] = {0.f, 0.f, 0.f, 0.f};
      mma_bf16_16816(one, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, qf[2 * G][0], qf[2 * G][1]);
      mma_bf16_16816(one, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, qf[2 * G + 1][0], qf[2 * G + 1][1]);
      qs[G][0] = -24.f * one[0];
      qs[G][1] = -24.f * one[1];
    }
  }

  for (int nt = 0; nt < n_w; ++nt) {
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const int nvalid = __shfl_sync(0xffffffffu, my_nvalid, nt & 31);
    if (nvalid > 0) {
      const uint32_t base = ring + (uint32_t)((nt % kStages) * R::kStageBytes);
      float s[4], pr[4];
      int t0, t1;  // the tokens of this lane's logits
      if constexpr (kInt4) {
        const uint4 wa = lds128(base + lane * 16), wb = lds128(base + 512 + lane * 16);
        const uint32_t ka[4] = {wa.x, wa.y, wa.z, wa.w}, kb[4] = {wb.x, wb.y, wb.z, wb.w};
        t0 = ((tq & 1) << 2) | (tq >> 1);
        t1 = t0 + 8;
        const uint2 sa = lds64(base + 2048 + t0 * 8), sb = lds64(base + 2048 + t1 * 8);
        s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
        for (int G = 0; G < 4; ++G) {
          auto pair_of = [](uint32_t w, int i) {
            const uint32_t x = i == 0 ? w << 3 : w >> (4 * i - 3);
            return (x & 0x00780078u) | 0x41804180u;
          };
          float d[4] = {qs[G][0], qs[G][1], qs[G][0], qs[G][1]};
          mma_bf16_16816(d, pair_of(ka[G], 0), pair_of(kb[G], 0), pair_of(ka[G], 1), pair_of(kb[G], 1), qf[2 * G][0],
                         qf[2 * G][1]);
          mma_bf16_16816(d, pair_of(ka[G], 2), pair_of(kb[G], 2), pair_of(ka[G], 3), pair_of(kb[G], 3),
                         qf[2 * G + 1][0], qf[2 * G + 1][1]);
          const uint32_t wsa = G < 2 ? sa.x : sa.y, wsb = G < 2 ? sb.x : sb.y;
          const float fa = (G & 1) ? hi_f(wsa) : lo_f(wsa), fb = (G & 1) ? hi_f(wsb) : lo_f(wsb);
          s[0] = fmaf(fa, d[0], s[0]);
          s[1] = fmaf(fa, d[1], s[1]);
          s[2] = fmaf(fb, d[2], s[2]);
          s[3] = fmaf(fb, d[3], s[3]);
        }
      } else {
        t0 = tq;
        t1 = tq + 8;
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
        for (int i = 0; i < 4; ++i) s[i] = sa[i] + sb[i];
      }
      const bool v0 = t0 < nvalid, v1 = t1 < nvalid;
      s[0] = v0 ? s[0] * sl2 : kNegInf;
      s[1] = v0 ? s[1] * sl2 : kNegInf;
      s[2] = v1 ? s[2] * sl2 : kNegInf;
      s[3] = v1 ? s[3] * sl2 : kNegInf;
      if constexpr (kAcc) {  // the logits of the tile, for the weights once lse is known
        const int64_t slot = pair * p.k * bs + (int64_t)(j0 * tpb + warp + kWarps * nt) * kTileTokens;
        float* z0 = p.z + (slot + t0) * g + ta;
        float* z1 = p.z + (slot + t1) * g + ta;
        if (ta < g) {
          z0[0] = s[0];
          z1[0] = s[2];
        }
        if (ta + 1 < g) {
          z0[1] = s[1];
          z1[1] = s[3];
        }
      }
      online_softmax(a, s, pr);
      if constexpr (kInt4) {
        const uint2 sa = lds64(base + 2048 + 128 + t0 * 8), sb = lds64(base + 2048 + 128 + t1 * 8);
        float fa[4] = {lo_f(sa.x), hi_f(sa.x), lo_f(sa.y), hi_f(sa.y)};
        float fb[4] = {lo_f(sb.x), hi_f(sb.x), lo_f(sb.y), hi_f(sb.y)};
        // fmaxf drops NaN scales: they reach the output through the weights
        const float mx = fmaxf(fmaxf(fmaxf(fa[0], fa[1]), fmaxf(fa[2], fa[3])),
                               fmaxf(fmaxf(fb[0], fb[1]), fmaxf(fb[2], fb[3])));
        const uint32_t mb = __reduce_max_sync(0xffffffffu, mx > 0.f ? __float_as_uint(mx) : 0u);
        if (mb >= vn_bits) {  // warp-uniform: a larger scale, the sums move to its power of two
          const uint32_t e = min((mb >> 23) + 1u, 253u);
          const float down = __uint_as_float(vn_bits) * __uint_as_float((254u - e) << 23);  // old vn / new vn
#pragma unroll
          for (int dm = 0; dm < 8; ++dm) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a.o[dm][i] *= down;
          }
          vn_bits = e << 23;
          kf = __uint_as_float((254u - e) << 23) * 0x1p14f;
        }
        float pk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pk[i] = pr[i] * kf;
        uint32_t pb[4][2];
#pragma unroll
        for (int G = 0; G < 4; ++G) {
          pb[G][0] = movmatrix_trans(pack_f16x2(pk[0] * fa[G], pk[1] * fa[G]));
          pb[G][1] = movmatrix_trans(pack_f16x2(pk[2] * fb[G], pk[3] * fb[G]));
        }
        // value codes: tokens c, c + 4, c + 8, c + 12; lane's 4 channels of
        // each group.  Two tokens' halfwords side by side, then a nibble of
        // each as 1024 + n (or 1024 + 16 n) in fp16, brought to n - 8 exactly.
        uint2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = c + 4 * i;
          x[i] = lds64(base + 1024 + t * 64 + (((tq >> 1) ^ (t & 2)) << 4) + (tq & 1) * 8);
        }
#pragma unroll
        for (int G = 0; G < 4; ++G) {
          const uint32_t sel = (G & 1) ? 0x7632u : 0x5410u;
          const uint32_t u01 = __byte_perm(G < 2 ? x[0].x : x[0].y, G < 2 ? x[1].x : x[1].y, sel);
          const uint32_t u23 = __byte_perm(G < 2 ? x[2].x : x[2].y, G < 2 ? x[3].x : x[3].y, sel);
          auto nib = [](uint32_t u, int i) {
            const uint32_t v = i & 2 ? u >> 8 : u;
            return (i & 1) ? hfma2((v & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u)   // x / 16 - 72
                           : hfma2((v & 0x000F000Fu) | 0x64006400u, 0x3C003C00u, 0xE408E408u);  // x - 1032
          };
          mma_f16_16816(a.o[2 * G], nib(u01, 0), nib(u01, 1), nib(u23, 0), nib(u23, 1), pb[G][0], pb[G][1]);
          mma_f16_16816(a.o[2 * G + 1], nib(u01, 2), nib(u01, 3), nib(u23, 2), nib(u23, 3), pb[G][0], pb[G][1]);
        }
      } else {
        // weights as the sum of two bf16 numbers (16 bits): a single bf16
        // weight would cost as much accuracy as the final rounding
        const uint32_t h0 = pack_bf16x2(pr[0], pr[1]), h1 = pack_bf16x2(pr[2], pr[3]);
        const uint32_t pb0 = movmatrix_trans(h0), pb1 = movmatrix_trans(h1);
        const uint32_t pl0 = movmatrix_trans(pack_bf16x2(pr[0] - lo_f(h0), pr[1] - hi_f(h0)));
        const uint32_t pl1 = movmatrix_trans(pack_bf16x2(pr[2] - lo_f(h1), pr[3] - hi_f(h1)));
        const uint32_t mlo = tok_mask(ta, nvalid), mhi = tok_mask(ta + 8, nvalid);
        const int vt = (lane & 7) + ((lane >> 4) << 3), vsel = (lane >> 3) & 1;
#pragma unroll
        for (int dm = 0; dm < 8; ++dm) {
          const int d0 = dm * 16 + vsel * 8;
          const uint32_t box = base + 2u * kHalfBox + (d0 < 64 ? 0u : (uint32_t)kHalfBox);
          const int ch = (d0 & 63) >> 3;
          uint32_t a0, a1, a2, a3;
          ldmatrix_x4_trans(box + vt * 128 + ((ch ^ (vt & 7)) << 4), a0, a1, a2, a3);
          if (nvalid < kTileTokens) {
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
    issue(nt + kStages);
  }
  cp_async_wait<0>();

#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    a.l0 += __shfl_xor_sync(0xffffffffu, a.l0, off);
    a.l1 += __shfl_xor_sync(0xffffffffu, a.l1, off);
  }
  __syncthreads();  // every warp is done with its ring; the combine area reuses it
  float* comb = reinterpret_cast<float*>(smem);  // [warp][head][kRowPad]
  {
    float* w0 = comb + ((warp * kMaxGroup) + ta) * kRowPad;
    if constexpr (kInt4) {
      // o[2G + e][..]: channel 32 G + 4 tq + 2 e (+ 1), heads ta and ta + 1
      const float back = __uint_as_float(vn_bits) * 0x1p-14f;
#pragma unroll
      for (int dm = 0; dm < 8; ++dm) {
        const int d = (dm >> 1) * 32 + 4 * tq + 2 * (dm & 1);
        w0[d] = a.o[dm][0] * back;
        w0[kRowPad + d] = a.o[dm][1] * back;
        w0[d + 1] = a.o[dm][2] * back;
        w0[kRowPad + d + 1] = a.o[dm][3] * back;
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
    s_m[warp][2 * lane] = a.m0;
    s_m[warp][2 * lane + 1] = a.m1;
    s_l[warp][2 * lane] = a.l0;
    s_l[warp][2 * lane + 1] = a.l1;
  }
  __syncthreads();
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
  }
  __syncthreads();
  const int d = tid;
  auto combined = [&](int j) {
    float num = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) num += s_ww[w][j] * comb[(w * kMaxGroup + j) * kRowPad + d];
    return num;
  };
  auto finish = [&](int j, float num, float den, float M) {
    p.out[(qh0 + j) * kHeadDim + d] = __float2bfloat16_rn(den == 0.f ? 0.f : num / den);
    if (d == 0) {
      const float l2 = den == 0.f ? kNegInf : M + log2f(den);
      if (p.lse) p.lse[qh0 + j] = l2 * 0.6931471805599453f;
      if (kAcc) p.lse2[qh0 + j] = l2;
    }
  };
  if (nchunks == 1) {
    for (int j = 0; j < g; ++j) finish(j, combined(j), s_cden[j], s_cm[j]);
    return;
  }

  // this chunk's partial; the pair's last chunk merges all of them
  float* part = p.partials + (pair * p.max_chunks + chunk) * (int64_t)g * kPartStride;
  for (int j = 0; j < g; ++j) {
    part[j * kPartStride + d] = combined(j);
    if (d == 0) {
      part[j * kPartStride + kHeadDim] = s_cm[j];
      part[j * kPartStride + kHeadDim + 1] = s_cden[j];
    }
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) s_last = (atomicAdd(&p.counters[pair], 1u) == (unsigned)(nchunks - 1));
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (tid == 0) p.counters[pair] = 0u;  // ready for the next call
  // The partials are staged in shared memory, a batch of chunks at a time;
  // thread j < g folds head j's maxima and sums and leaves one weight per
  // (chunk, head); every thread folds its output channel.
  const int rec = g * kPartStride;
  const int per_batch = R::kPipe / (4 * rec);
  const float4* src4 = reinterpret_cast<const float4*>(p.partials + pair * p.max_chunks * (int64_t)rec);
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
      for (int cc = 0; cc < nbat; ++cc) Mb = fmaxf(Mb, stage[(cc * g + j) * kPartStride + kHeadDim]);
      const float Mr = s_mr[j];
      const float Mn = fmaxf(Mr, Mb);
      const float al = s_den[j] == 0.f ? 0.f : exp2f(Mr - Mn);
      float dd = s_den[j] * al;
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
    for (int cc = 0; cc < nbat; ++cc) {
      const float* rc = stage + cc * g * kPartStride + d;
#pragma unroll
      for (int j = 0; j < kMaxGroup; ++j)
        if (j < g) num[j] += s_w[cc * g + j] * rc[j * kPartStride];
    }
    __syncthreads();  // the next batch overwrites the staging area and the weights
  }
#pragma unroll
  for (int j = 0; j < kMaxGroup; ++j)
    if (j < g) finish(j, num[j], s_den[j], s_mr[j]);
}

// The weights of the attended tokens, once every lse is known: one thread per
// (pair, slot of the kept blocks) adds sum_j 2^(z_j - lse2_j) to its token's
// running sum.  Each kept token has one slot, so the addition is an atomic
// only where an index is listed twice (it then counts twice).
__global__ void __launch_bounds__(256) kv_weights_kernel(KvAttnParams p) {
  pdl_wait();
  pdl_trigger_early();
  const int per = p.k * p.bs;
  const int ctas = (per + 255) / 256;  // per pair
  const int64_t pair = blockIdx.x / ctas;
  const int i = (int)(blockIdx.x - pair * ctas) * 256 + threadIdx.x;
  if (i >= per) return;
  const int b = (int)(pair / p.Hkv), h = (int)(pair - (int64_t)b * p.Hkv);
  const int L = __ldg(p.seq_lens + b);
  if (L < 1 || L > p.kv.Lcap) return;
  const int nb = (L + p.bs - 1) / p.bs;
  const int j = i / p.bs;
  const int cnt = p.sel_idx ? __ldg(p.sel_cnt + pair) : nb;
  if (j >= cnt) return;
  const int blk = p.sel_idx ? __ldg(p.sel_idx + pair * p.k_row + j) : j;
  const int t = blk * p.bs + (i - j * p.bs);
  if (blk < 0 || blk >= nb || t >= L) return;
  if (kv_row(p.kv.pages, b, h, p.Hkv, p.kv.Lcap, p.bs, t) < 0) return;  // a bad page: nothing was attended
  const float* z = p.z + (pair * per + i) * p.g;
  const float* l = p.lse2 + (int64_t)b * p.Hq + (int64_t)h * p.g;
  float w = 0.f;
  for (int q = 0; q < p.g; ++q) w += exp2f(z[q] - l[q]);
  atomicAdd(p.acc + pair * p.kv.Lcap + t, w);
}

template <bool kInt4, bool kAcc>
static cudaError_t launch_kv_attn_as(const KvAttnParams& p, cudaStream_t s) {
  const auto kernel = kv_attn_kernel<kInt4, kAcc>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), 16 + 2 * kInt4 + kAcc, Ring<kInt4>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = (int64_t)p.B * p.Hkv;
  e = launch_pdl(kernel, dim3((unsigned)(pairs * p.max_chunks)), dim3(kThreads), Ring<kInt4>::kSmem, s, p);
  if (e != cudaSuccess || !kAcc) return e;
  const int64_t per = (int64_t)p.k * p.bs;
  return launch_pdl(kv_weights_kernel, dim3((unsigned)(pairs * ((per + 255) / 256))), dim3(256), 0, s, p);
}

cudaError_t launch_kv_attn(const KvAttnParams& p, cudaStream_t s) {
  if (p.kv.int4) return p.acc ? launch_kv_attn_as<true, true>(p, s) : launch_kv_attn_as<true, false>(p, s);
  return p.acc ? launch_kv_attn_as<false, true>(p, s) : launch_kv_attn_as<false, false>(p, s);
}

}  // namespace kin
