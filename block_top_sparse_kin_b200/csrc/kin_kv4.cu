// kin_kv4.cu -- the KV cache held in 4 bits: store (a prefilled bf16 cache),
// append (the new tokens of a step) and load (rows back as bf16).
//
// Math, per row (a token's key or value of one KV head) and group of 32
// channels: a = max |x|, s = bf16(a / 7), c = clamp(rne(x / s), -7, 7), held
// as the nibble c + 8; the group stands for c s (exact in fp32: a 4-bit
// integer times an 8-bit significand).  A group that holds NaN or an infinity
// gets s = NaN and c = 0, so it stands for NaN; s = 0 gives c = 0.  Block
// means are the fp32 sums, in token order, of the keys' held values divided
// by the row count: what the attention reads, so an append and a store of the
// same tokens leave the same means, bit for bit.
//
// The nibbles' order suits the attention's fragments (kin_kvattn.cu): a key
// row is 16 words, word 4c + g holding channels 32g + 8c .. + 7 (even ones in
// nibbles 0..3, odd ones in 4..7); a value row is 32 halfwords, halfword
// 4r + g holding channels 32g + 4r .. + 3.
//
// Layout of the work: one warp per block (16 to 128 tokens); its lower half
// holds the key row, its upper half the value row, lane x of a half 8
// channels (one 16-byte load of bf16), so a group is 4 lanes and its maximum
// two shuffles.  Both are streams bounded by HBM.
#include "kin_internal.cuh"

namespace kin {

namespace {

constexpr int kKvThreads = 128;
constexpr int kKvWarps = kKvThreads / 32;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 8 channels of a group in 4 bits: w = the bf16 pairs of this lane.  Returns
// the scale's bits (the same in the group's 4 lanes) and the codes c[i] as
// numbers.
//
// The rounding is exact with one reciprocal.  x has an 8-bit significand S
// and a midpoint (c + 1/2) s a product of an odd number 2c + 1 <= 13 and an
// 8-bit one, so a quotient x / s that is not a midpoint is at least 2^-11
// away from one (2^-8 of 1/2, 2^-10 of 3/2, 2^-11 of 5/2 and 7/2, 2^-12 of
// 9/2 to 13/2).  x times the rounded reciprocal, added to 1.5 * 2^11 in one
// rounding, is the quotient to 2^-13 + 2^-21 on a grid of 2^-12: at a midpoint
// exactly there, elsewhere on its side of it.  The second addition rounds
// that to a whole number, half to even, and the third leaves it.  A normal
// scale is a / 7 to 2^-9, so no quotient reaches 7.5.
__device__ __forceinline__ uint32_t encode8(const uint4& w, float (&c)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = max_u16x2(max_u16x2(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu), max_u16x2(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu));
  m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = max(m & 0xFFFFu, m >> 16);
  // a NaN's bits are above infinity's, so the integer maximum keeps it
  const uint32_t s = m < 0x7F80u ? (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(__uint_as_float(m << 16), 7.0f)))
                                 : 0x7FC0u;
  const float sf = __uint_as_float(s << 16);
  constexpr float kGrid = 0x1.8p11f, kWhole = 0x1.8p23f - 0x1.8p11f;
  if (sf >= 0x1p-100f) {
    const float inv = __frcp_rn(sf);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = (i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]);
      c[i] = __fsub_rn(__fadd_rn(__fmaf_rn(x, inv, kGrid), kWhole), 12582912.f);
    }
  } else {
    // a scale of zero, or NaN: every code is 0.  A tiny one: x and s are first
    // scaled by 2^100 (exact), since 1 / s overflows below 2^-126; a subnormal
    // scale may be rounded by half, so the quotient is cut at 7.
    const bool some = sf > 0.f;
    const float inv = some ? __frcp_rn(sf * 0x1p100f) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = some ? ((i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1])) * 0x1p100f : 0.f;
      const float y = fminf(fmaxf(x * inv, -7.f), 7.f);
      c[i] = __fsub_rn(__fadd_rn(__fadd_rn(y, kGrid), kWhole), 12582912.f);
    }
  }
  return s;
}

// Four codes as the nibbles c + 8 of the low half of a word: the number
// sum 16^i (c_i + 8) < 2^16, exact, read off behind 2^23.
__device__ __forceinline__ uint32_t nibbles4(float c0, float c1, float c2, float c3) {
  const float n = fmaf(fmaf(fmaf(c3, 16.f, c2), 16.f, c1), 16.f, c0);
  return __float_as_uint(n + (8388608.f + 34952.f));  // 8 * 0x1111
}

// Nibble i of w as a number: behind 2^23, less 2^23 and the offset.
__device__ __forceinline__ float code_of(uint32_t w, int i) {
  return __uint_as_float(((w >> (4 * i)) & 15u) | 0x4B000000u) - 8388616.f;
}

// Values of a key word: channel e of the word times s.
__device__ __forceinline__ void key_values(uint32_t w, float s, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = code_of(w, (e >> 1) + 4 * (e & 1)) * s;
}

// Lane x of a half holds 8 channels 32g + 8c ..: g = x / 4, c = x % 4.
// Writes a row's codes and scales; half 0 a key row, half 1 a value row.
__device__ __forceinline__ void write_row(const KvView& kv, int half, int x, int64_t row, const float (&n)[8], uint32_t s) {
  const int g = x >> 2, c = x & 3;
  if (half == 0) {
    *reinterpret_cast<uint32_t*>(kv.k + row * kCodeBytes + (4 * c + g) * 4) =
        __byte_perm(nibbles4(n[0], n[2], n[4], n[6]), nibbles4(n[1], n[3], n[5], n[7]), 0x5410);
    if (c == 0) kv.ks[row * kGroups + g] = (uint16_t)s;
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(kv.v + row * kCodeBytes);
    o[8 * c + g] = (uint16_t)nibbles4(n[0], n[1], n[2], n[3]);
    o[8 * c + 4 + g] = (uint16_t)nibbles4(n[4], n[5], n[6], n[7]);
    if (c == 0) kv.vs[row * kGroups + g] = (uint16_t)s;
  }
}

}  // namespace

// The key half's block sum as a mean row: lane l of the warp takes channels
// 4l .. 4l + 3 from lane l / 2 and stores them in the layout the flag names.
__device__ __forceinline__ void store_half_mean(void* means, int flag, int64_t rows, int64_t row, int lane,
                                                const float (&acc)[8], float count) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __shfl_sync(0xffffffffu, acc[i], lane >> 1);
    const float hi = __shfl_sync(0xffffffffu, acc[4 + i], lane >> 1);
    m[i] = __fdiv_rn((lane & 1) ? hi : lo, count);
  }
  store_mean(means, flag, rows, row, lane, make_float4(m[0], m[1], m[2], m[3]));
}

constexpr int kWriteRows = 8;  // bf16 rows in flight per lane
constexpr int kHeldRows = 16;  // 4-bit rows in flight per lane

// One warp per (pair, block): rows below the old length come from the cache
// (append; keys only, for the mean), the others are quantised and written.
__global__ void __launch_bounds__(kKvThreads) kv4_write_kernel(Kv4WriteParams p) {
  pdl_wait();
  pdl_trigger_early();
  const int lane = threadIdx.x & 31, half = lane >> 4, x = lane & 15;
  const int64_t unit = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  const int64_t pair = unit / p.span;
  const int j = (int)(unit - pair * p.span);
  if (pair >= (int64_t)p.B * p.Hkv) return;
  const int b = (int)(pair / p.Hkv), h = (int)(pair - (int64_t)b * p.Hkv);
  const int Lcap = p.dst.Lcap, bs = p.bs;
  const int len = __ldg(p.seq_lens + b);
  const int L0 = p.append ? len : 0;                                  // rows already held
  const int64_t L1w = p.append ? (int64_t)len + p.n_new : (int64_t)len;
  if (len < 0 || L1w > Lcap) {
    if (lane == 0 && j == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
    // the length stays as it was
    if (p.append && h == 0 && j == 0 && lane == 0 && p.new_lens && p.new_lens != p.seq_lens) p.new_lens[b] = len;
    return;
  }
  const int L1 = (int)L1w;
  if (p.append && h == 0 && j == 0 && lane == 0 && p.new_lens && p.new_lens != p.seq_lens) p.new_lens[b] = L1;
  const int i = L0 / bs + j;
  const int t0 = i * bs, t1 = min(t0 + bs, L1);
  if (t0 >= t1) return;
  const int64_t row0 = kv_row(p.dst.pages, b, h, p.Hkv, Lcap, bs, t0);  // a block's rows are contiguous
  const int tn = max(t0, L0);                                          // first new row
  int64_t src0;                                                        // source row of token tn
  if (p.append)
    src0 = pair * p.n_new + (tn - L0);
  else
    src0 = kv_row(p.src_pages, b, h, p.Hkv, Lcap, bs, t0);
  if (row0 < 0 || src0 < 0) {  // a page index outside its pool: the block is left as it was
    if (lane == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
    return;
  }
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  const int g = x >> 2, c = x & 3;
  if (p.means && half == 0) {  // held keys of the block, in token order
    for (int t = t0; t < tn; t += kHeldRows) {
      uint32_t w[kHeldRows];
      uint16_t s[kHeldRows];
#pragma unroll
      for (int u = 0; u < kHeldRows; ++u) {
        const int64_t row = row0 + min(t + u, tn - 1) - t0;
        w[u] = *reinterpret_cast<const uint32_t*>(p.dst.k + row * kCodeBytes + (4 * c + g) * 4);
        s[u] = p.dst.ks[row * kGroups + g];
      }
#pragma unroll
      for (int u = 0; u < kHeldRows; ++u) {
        if (t + u < tn) {
          float v[8];
          key_values(w[u], __uint_as_float((uint32_t)s[u] << 16), v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += v[e];
        }
      }
    }
  }
  __syncwarp();
  const uint8_t* src = (half ? p.v_src : p.k_src) + src0 * (kHeadDim * 2) + x * 16;
  for (int t = tn; t < t1; t += kWriteRows) {
    uint4 w[kWriteRows];
#pragma unroll
    for (int u = 0; u < kWriteRows; ++u)
      w[u] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)(min(t + u, t1 - 1) - tn) * (kHeadDim * 2)));
#pragma unroll
    for (int u = 0; u < kWriteRows; ++u) {
      if (t + u < t1) {  // warp-uniform
        float n[8];
        const uint32_t s = encode8(w[u], n);
        write_row(p.dst, half, x, row0 + (t + u - t0), n, s);
        const float sf = __uint_as_float(s << 16);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(n[e], sf, acc[e]);  // the product is exact
      }
    }
  }
  if (p.means) {
    const int64_t mrow = means_row_index(p.dst.pages, p.means_per_page, b, h, p.Hkv, p.nbcap, i);
    if (mrow >= 0) store_half_mean(p.means, p.means_flag, p.mean_rows, mrow, lane, acc, (float)(t1 - t0));
  }
}

// In-place advance of the lengths, after every CTA of the write has read them.
__global__ void __launch_bounds__(256) kv4_advance_kernel(int32_t* lens, int B, int n_new, int Lcap) {
  pdl_wait();
  pdl_trigger_early();
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= B) return;
  const int len = lens[b];
  if (len >= 0 && (int64_t)len + n_new <= Lcap) lens[b] = len + n_new;
}

cudaError_t launch_kv4_write(const Kv4WriteParams& p, cudaStream_t s) {
  const int64_t units = (int64_t)p.B * p.Hkv * p.span;
  cudaError_t e = launch_pdl(kv4_write_kernel, dim3((unsigned)((units + kKvWarps - 1) / kKvWarps)), dim3(kKvThreads), 0, s, p);
  if (e != cudaSuccess || !p.append || p.new_lens != p.seq_lens) return e;
  return launch_pdl(kv4_advance_kernel, dim3((p.B + 255) / 256), dim3(256), 0, s, p.new_lens, p.B, p.n_new, p.dst.Lcap);
}

constexpr int kLoadRows = 8;  // rows per warp

// Rows back as bf16: one warp per kLoadRows consecutive output rows of a
// pair, lower half keys, upper half values.
__global__ void __launch_bounds__(kKvThreads) kv4_load_kernel(Kv4LoadParams p) {
  pdl_wait();
  pdl_trigger_early();
  const int lane = threadIdx.x & 31, half = lane >> 4, x = lane & 15;
  const int per = (p.n + kLoadRows - 1) / kLoadRows;
  const int64_t unit = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  const int64_t pair = unit / per;
  const int r0 = (int)(unit - pair * per) * kLoadRows;
  if (pair >= (int64_t)p.B * p.Hkv) return;
  const int b = (int)(pair / p.Hkv), h = (int)(pair - (int64_t)b * p.Hkv);
  int L = __ldg(p.seq_lens + b);
  const int start = p.starts ? __ldg(p.starts + b) : 0;
  if (L < 0 || L > p.src.Lcap || start < 0) {
    if (lane == 0 && r0 == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
    L = 0;  // zeros
  }
  const int g = x >> 2, c = x & 3;
  uint32_t w[kLoadRows];
  uint16_t s[kLoadRows];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kLoadRows; ++u) {
    w[u] = 0x88888888u;
    s[u] = 0;
    const int64_t t = (int64_t)start + r0 + u;
    if (r0 + u < p.n && t < L) {
      const int64_t row = kv_row(p.src.pages, b, h, p.Hkv, p.src.Lcap, p.bs, (int)t);
      if (row >= 0) {
        if (half == 0) {
          w[u] = __ldg(reinterpret_cast<const uint32_t*>(p.src.k + row * kCodeBytes + (4 * c + g) * 4));
          s[u] = __ldg(p.src.ks + row * kGroups + g);
        } else {
          const uint16_t* o = reinterpret_cast<const uint16_t*>(p.src.v + row * kCodeBytes);
          w[u] = (uint32_t)__ldg(o + 8 * c + g) | ((uint32_t)__ldg(o + 8 * c + 4 + g) << 16);
          s[u] = __ldg(p.src.vs + row * kGroups + g);
        }
      } else {
        bad = true;
      }
    }
  }
  if (bad && x == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
  __nv_bfloat16* out = half ? p.v_out : p.k_out;
#pragma unroll
  for (int u = 0; u < kLoadRows; ++u) {
    if (r0 + u < p.n) {
      const float sf = __uint_as_float((uint32_t)s[u] << 16);
      float v[8];
      if (half == 0) {
        key_values(w[u], sf, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = code_of(w[u], e) * sf;
      }
      // the product has up to 11 significant bits: one rounding to bf16
      uint4 o;
      o.x = pack_bf16x2(v[0], v[1]);
      o.y = pack_bf16x2(v[2], v[3]);
      o.z = pack_bf16x2(v[4], v[5]);
      o.w = pack_bf16x2(v[6], v[7]);
      reinterpret_cast<uint4*>(out)[(pair * p.n + r0 + u) * 16 + x] = o;
    }
  }
}

cudaError_t launch_kv4_load(const Kv4LoadParams& p, cudaStream_t s) {
  const int64_t units = (int64_t)p.B * p.Hkv * ((p.n + kLoadRows - 1) / kLoadRows);
  return launch_pdl(kv4_load_kernel, dim3((unsigned)((units + kKvWarps - 1) / kKvWarps)), dim3(kKvThreads), 0, s, p);
}

// ------------------------------------------------------------- eviction: move
// One warp per (pair, destination block): the kept tokens' rows, scales and
// weights move to their new places (ascending, so blocks keep the time order)
// and the block's mean is taken on the way.  Destination weights behind the
// kept tokens become zero, so tokens appended later start at nothing.  Rows
// are gathered, 8 in flight per lane.
template <bool kInt4>
__global__ void __launch_bounds__(kKvThreads) evict_move_kernel(EvictParams p) {
  pdl_wait();
  pdl_trigger_early();
  const int lane = threadIdx.x & 31, half = lane >> 4, x = lane & 15;
  const int64_t unit = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  const int64_t pair = unit / p.nbcap_dst;
  const int i = (int)(unit - pair * p.nbcap_dst);
  if (pair >= (int64_t)p.B * p.Hkv) return;
  const int b = (int)(pair / p.Hkv), h = (int)(pair - (int64_t)b * p.Hkv);
  const int bs = p.bs;
  const int m = __ldg(p.dst_lens + b);  // written by the select kernel: min(L, n_keep), 0 for a bad length
  const int t0 = i * bs, t1 = min(t0 + bs, m);
  const int32_t* sel = p.sel + pair * p.n_keep;
  if (p.dst_acc) {
    const int end = min(t0 + bs, p.dst.Lcap);
    for (int t = t0 + lane; t < end; t += 32)
      p.dst_acc[pair * p.dst.Lcap + t] = t < t1 ? __ldg(p.acc + pair * p.src.Lcap + __ldg(sel + t)) : 0.f;
  }
  if (t0 >= t1) return;
  const int64_t to0 = kv_row(p.dst.pages, b, h, p.Hkv, p.dst.Lcap, bs, t0);
  if (to0 < 0) {
    if (lane == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
    return;
  }
  const int g = x >> 2, c = x & 3;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  bool bad = false;
  for (int tb = t0; tb < t1; tb += 32) {
    int64_t my = -1;  // lane's source row
    if (tb + lane < t1) {
      my = kv_row(p.src.pages, b, h, p.Hkv, p.src.Lcap, bs, __ldg(sel + tb + lane));
      bad |= my < 0;
    }
    const int n = min(32, t1 - tb);
    for (int u0 = 0; u0 < n; u0 += 8) {
      uint4 w[8];
      uint16_t s[8];
      int64_t from[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int src_lane = (u0 + u) & 31;
        from[u] = (int64_t)(((uint64_t)(uint32_t)__shfl_sync(0xffffffffu, (int)(my >> 32), src_lane) << 32) |
                            (uint32_t)__shfl_sync(0xffffffffu, (int)(uint32_t)my, src_lane));
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        s[u] = 0;
        if (u0 + u < n && from[u] >= 0) {
          if constexpr (kInt4) {
            const uint8_t* codes = half ? p.src.v : p.src.k;
            w[u].x = __ldg(reinterpret_cast<const uint32_t*>(codes + from[u] * kCodeBytes + (4 * c + g) * 4));
            s[u] = __ldg((half ? p.src.vs : p.src.ks) + from[u] * kGroups + g);
          } else {
            w[u] = __ldg(reinterpret_cast<const uint4*>((half ? p.src.v : p.src.k) + from[u] * (kHeadDim * 2) + x * 16));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (u0 + u < n && from[u] >= 0) {
          const int64_t to = to0 + (tb - t0) + u0 + u;
          float v[8];
          if constexpr (kInt4) {
            uint8_t* codes = half ? p.dst.v : p.dst.k;
            *reinterpret_cast<uint32_t*>(codes + to * kCodeBytes + (4 * c + g) * 4) = w[u].x;
            if (c == 0) (half ? p.dst.vs : p.dst.ks)[to * kGroups + g] = s[u];
            key_values(w[u].x, __uint_as_float((uint32_t)s[u] << 16), v);
          } else {
            *reinterpret_cast<uint4*>((half ? p.dst.v : p.dst.k) + to * (kHeadDim * 2) + x * 16) = w[u];
            v[0] = bf16_lo(w[u].x);
            v[1] = bf16_hi(w[u].x);
            v[2] = bf16_lo(w[u].y);
            v[3] = bf16_hi(w[u].y);
            v[4] = bf16_lo(w[u].z);
            v[5] = bf16_hi(w[u].z);
            v[6] = bf16_lo(w[u].w);
            v[7] = bf16_hi(w[u].w);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += v[e];
        }
      }
    }
  }
  if (bad) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);  // the row is left as it was
  if (p.means) {
    const int64_t mrow = means_row_index(p.dst.pages, p.means_per_page, b, h, p.Hkv, p.nbcap_dst, i);
    if (mrow >= 0) store_half_mean(p.means, p.means_flag, p.mean_rows, mrow, lane, acc, (float)(t1 - t0));
  }
}

cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t s) {
  const int64_t units = (int64_t)p.B * p.Hkv * p.nbcap_dst;
  const dim3 grid((unsigned)((units + kKvWarps - 1) / kKvWarps));
  return p.src.int4 ? launch_pdl(evict_move_kernel<true>, grid, dim3(kKvThreads), 0, s, p)
                    : launch_pdl(evict_move_kernel<false>, grid, dim3(kKvThreads), 0, s, p);
}

}  // namespace kin
