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
// Layout of the work: half a warp holds a row, lane x of it 8 channels (one
// 16-byte load of bf16), so a group is 4 lanes and its maximum two shuffles.
// A warp has keys or values, never both (their orders would cost it both
// paths), and to store, two consecutive blocks, one each half: a lane adds up
// its 8 channels of a block's mean on the way.  Reading back and the bf16 move
// are streams bounded by HBM: 1M tokens read back in 108 us (6.4 TB/s), 512K
// bf16 tokens moved in 87 us (6.0 TB/s).  The store is bounded by its
// instructions, 122 a token: 1M tokens in 150 us (4.7 TB/s), where its bytes
// would take 110.  Short stores and appends are bounded by their round trips
// to memory, 4 rows of a block at a time (333 tokens to 32 pairs: 15 us).
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

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kGrid = 0x1.8p11f, kWhole = 0x1.8p23f - 0x1.8p11f;  // see encode8

struct Codes8 {
  float c[8];
};

// encode8's codes where the scale is below 2^-100, zero or NaN: zero and NaN
// give codes of 0.  Otherwise x and s are first scaled by 2^100 (exact), since
// 1 / s overflows below 2^-126; a subnormal scale may be rounded by half, so
// the quotient is cut at 7.  Its own function: inlined, it would double the
// code of the paths that run.
__device__ __noinline__ Codes8 encode8_tiny(uint4 w, float sf) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  const bool some = sf > 0.f;
  const float inv = some ? __frcp_rn(sf * 0x1p100f) : 0.f;
  Codes8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = some ? ((i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1])) * 0x1p100f : 0.f;
    const float y = fminf(fmaxf(x * inv, -7.f), 7.f);
    r.c[i] = __fsub_rn(__fadd_rn(__fadd_rn(y, kGrid), kWhole), 12582912.f);
  }
  return r;
}

// 8 channels of a group in 4 bits: w = the bf16 pairs of this lane.  Returns
// the scale's bits (the same in the group's 4 lanes) and the codes c[i] as
// numbers.
//
// The rounding is exact with one reciprocal.  x and s have significands X, S <
// 2^8, and a midpoint is m / 2, m odd, so a quotient x / s = 2^n X / S that is
// not a midpoint is at least 2^-9 away from it: by a whole number over 2 S, or
// over 2^-n S, which is at most 2 X near a midpoint, where n < -1.  x times
// the rounded reciprocal, added to 1.5 * 2^11 in one rounding, is the quotient
// to 2^-13 + 2^-20 on a grid of 2^-12: at a midpoint exactly there, elsewhere
// on its side of it.  The second addition rounds
// that to a whole number, half to even, and the third leaves it.  A normal
// scale is a / 7 to 2^-9, so no quotient reaches 7.5.  The scale itself: a / 7
// is never a midpoint of bf16 (7 times an odd 9-bit number has 11 bits, a has
// 8) and at least 2^-12 away from one, so a times the rounded 1 / 7 serves.
__device__ __forceinline__ uint32_t encode8(const uint4& w, float (&c)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = max_u16x2(max_u16x2(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu), max_u16x2(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu));
  m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = max(m & 0xFFFFu, m >> 16);
  // a NaN's bits are above infinity's, so the integer maximum keeps it
  const uint32_t s = m < 0x7F80u ? (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(m << 16) * 0x1.24924ap-3f))
                                 : 0x7FC0u;
  const float sf = __uint_as_float(s << 16);
  if (sf >= 0x1p-100f) {
    const float inv = rcp_approx(sf);  // to 2^-23
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = (i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]);
      c[i] = __fsub_rn(__fadd_rn(__fmaf_rn(x, inv, kGrid), kWhole), 12582912.f);
    }
  } else {
    const Codes8 t = encode8_tiny(w, sf);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = t.c[i];
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

}  // namespace

// A block's mean row from the half warp `half` that holds its sums: lane l of
// the warp takes channels 4l .. 4l + 3 from lane l / 2 of that half.
__device__ __forceinline__ void store_half_mean(void* means, int flag, int64_t rows, int64_t row, int lane, int half,
                                                const float (&acc)[8], float count) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __shfl_sync(0xffffffffu, acc[i], 16 * half + (lane >> 1));
    const float hi = __shfl_sync(0xffffffffu, acc[4 + i], 16 * half + (lane >> 1));
    m[i] = __fdiv_rn((lane & 1) ? hi : lo, count);
  }
  store_mean(means, flag, rows, row, lane, make_float4(m[0], m[1], m[2], m[3]));
}

constexpr int kWriteRows = 4;  // bf16 rows a lane takes at a time, the next ones in flight
constexpr int kHeldRows = 16;  // 4-bit rows in flight per lane

// Keys (kKeys) or values of two consecutive blocks of a pair, one each half of
// the warp: rows below the old length come from the cache (append; keys only,
// for the mean), the others are quantised and written.
template <bool kKeys>
__device__ __forceinline__ void write_blocks(const Kv4WriteParams& p, int64_t pair, int j, int lane) {
  const int half = lane >> 4, x = lane & 15, g = x >> 2, c = x & 3;
  const int b = (int)(pair / p.Hkv), h = (int)(pair - (int64_t)b * p.Hkv);
  const int Lcap = p.dst.Lcap, bs = p.bs;
  const int len = __ldg(p.seq_lens + b);
  const int L0 = p.append ? len : 0;                                  // rows already held
  const int64_t L1w = p.append ? (int64_t)len + p.n_new : (int64_t)len;
  const bool bad = len < 0 || L1w > Lcap;
  const int L1 = bad ? 0 : (int)L1w;
  if (kKeys && h == 0 && j == 0 && lane == 0) {  // a sequence that does not fit keeps its length
    if (p.append && p.new_lens != p.seq_lens) p.new_lens[b] = bad ? len : L1;
    if (bad) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
  }
  if (bad) return;
  const int i = L0 / bs + j + half;
  const int t0 = i * bs, tn = max(t0, L0);  // tn: the first new row
  int t1 = j + half < p.span ? min(t0 + bs, L1) : t0;
  int64_t row0 = 0, src0 = 0;               // a block's rows are contiguous, so are the new ones
  if (t0 < t1) {
    row0 = kv_row(p.dst.pages, b, h, p.Hkv, Lcap, bs, t0);
    src0 = p.append ? pair * p.n_new + (tn - L0) : kv_row(p.src_pages, b, h, p.Hkv, Lcap, bs, t0);
    if (row0 < 0 || src0 < 0) {  // a page index outside its pool: the block is left as it was
      if (kKeys) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
      t1 = t0;
      row0 = src0 = 0;  // a half without rows reads row 0 beside the other's
    }
  }
  const int held = t0 < t1 ? tn - t0 : 0, fresh = t0 < t1 ? t1 - tn : 0;
  const int most = max(fresh, __shfl_xor_sync(0xffffffffu, fresh, 16));
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  if (kKeys && p.means) {  // held keys of the block, in token order
    const uint8_t* codes = p.dst.k + row0 * kCodeBytes + (4 * c + g) * 4;
    const uint16_t* sc = p.dst.ks + row0 * kGroups + g;
    for (int r = 0; r < held; r += kHeldRows) {
      uint32_t w[kHeldRows];
      uint16_t s[kHeldRows];
#pragma unroll
      for (int u = 0; u < kHeldRows; ++u) {
        const int64_t row = min(r + u, held - 1);
        w[u] = *reinterpret_cast<const uint32_t*>(codes + row * kCodeBytes);
        s[u] = sc[row * kGroups];
      }
#pragma unroll
      for (int u = 0; u < kHeldRows; ++u) {
        if (r + u < held) {
          float v[8];
          key_values(w[u], __uint_as_float((uint32_t)s[u] << 16), v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += v[e];
        }
      }
    }
    __syncwarp();
  }
  const uint8_t* src = (kKeys ? p.k_src : p.v_src) + src0 * (kHeadDim * 2) + x * 16;
  uint8_t* to = (kKeys ? p.dst.k : p.dst.v) + (row0 + held) * kCodeBytes + (kKeys ? (4 * c + g) * 4 : (8 * c + g) * 2);
  uint16_t* to_s = (kKeys ? p.dst.ks : p.dst.vs) + (row0 + held) * kGroups + g;
  uint4 w[kWriteRows], next[kWriteRows];
  auto fetch = [&](int r, uint4(&to)[kWriteRows]) {  // rows r .. of the new ones, the last one where there are no more
#pragma unroll
    for (int u = 0; u < kWriteRows; ++u)
      to[u] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)max(min(r + u, fresh - 1), 0) * (kHeadDim * 2)));
  };
  if (most > 0) fetch(0, next);
  for (int r = 0; r < most; r += kWriteRows) {
#pragma unroll
    for (int u = 0; u < kWriteRows; ++u) w[u] = next[u];
    if (r + kWriteRows < most) fetch(r + kWriteRows, next);
#pragma unroll
    for (int u = 0; u < kWriteRows; ++u) {
      if (r + u < most) {  // warp-uniform
        float n[8];
        const uint32_t s = encode8(w[u], n);
        if (r + u < fresh) {
          if (kKeys) {
            *reinterpret_cast<uint32_t*>(to + (r + u) * kCodeBytes) =
                __byte_perm(nibbles4(n[0], n[2], n[4], n[6]), nibbles4(n[1], n[3], n[5], n[7]), 0x5410);
            const float sf = __uint_as_float(s << 16);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(n[e], sf, acc[e]);  // the product is exact
          } else {
            *reinterpret_cast<uint16_t*>(to + (r + u) * kCodeBytes) = (uint16_t)nibbles4(n[0], n[1], n[2], n[3]);
            *reinterpret_cast<uint16_t*>(to + (r + u) * kCodeBytes + 8) = (uint16_t)nibbles4(n[4], n[5], n[6], n[7]);
          }
          if (c == 0) to_s[(r + u) * kGroups] = (uint16_t)s;
        }
      }
    }
  }
  if (kKeys && p.means) {
    const int rows = held + fresh;
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {
      const int n = __shfl_sync(0xffffffffu, rows, 16 * hb);
      if (n > 0) {
        const int64_t mrow = means_row_index(p.dst.pages, p.means_per_page, b, h, p.Hkv, p.nbcap, L0 / bs + j + hb);
        store_half_mean(p.means, p.means_flag, p.mean_rows, mrow, lane, hb, acc, (float)n);
      }
    }
  }
}

__global__ void __launch_bounds__(kKvThreads) kv4_write_kernel(Kv4WriteParams p) {
  pdl_wait();
  pdl_trigger_early();
  const int lane = threadIdx.x & 31, per = (p.span + 1) / 2;  // units of a pair, for keys and for values
  const int64_t unit = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  const int64_t of = unit >> 1, pair = of / per;
  if (pair >= (int64_t)p.B * p.Hkv) return;
  const int j = 2 * (int)(of - pair * per);
  if (unit & 1)
    write_blocks<false>(p, pair, j, lane);
  else
    write_blocks<true>(p, pair, j, lane);
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
  const int64_t units = 2 * (int64_t)p.B * p.Hkv * ((p.span + 1) / 2);
  cudaError_t e = launch_pdl(kv4_write_kernel, dim3((unsigned)((units + kKvWarps - 1) / kKvWarps)), dim3(kKvThreads), 0, s, p);
  if (e != cudaSuccess || !p.append || p.new_lens != p.seq_lens) return e;
  return launch_pdl(kv4_advance_kernel, dim3((p.B + 255) / 256), dim3(256), 0, s, p.new_lens, p.B, p.n_new, p.dst.Lcap);
}

constexpr int kLoadRows = 8;  // rows of a half warp

__device__ __forceinline__ uint32_t hadd2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("{.reg .b32 one; mov.b32 one, 0x3F803F80; fma.rn.bf16x2 %0, %1, one, %2;}" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("{.reg .b32 zero; mov.b32 zero, 0x80008000; fma.rn.bf16x2 %0, %1, %2, zero;}" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Rows back as bf16: a warp has keys (kKeys) or values of 16 consecutive
// output rows of a pair, a half 8 of them.  A nibble n becomes the bf16 number
// 128 + n by one logic operation for two, less 136 the code, exact; its
// product with the scale is rounded once.
template <bool kKeys>
__device__ __forceinline__ void load_rows(const Kv4LoadParams& p, int64_t pair, int unit, int lane) {
  const int half = lane >> 4, x = lane & 15, g = x >> 2, c = x & 3;
  const int b = (int)(pair / p.Hkv), h = (int)(pair - (int64_t)b * p.Hkv);
  const int r0 = unit * 2 * kLoadRows + half * kLoadRows;
  int L = __ldg(p.seq_lens + b);
  const int start = p.starts ? __ldg(p.starts + b) : 0;
  if (L < 0 || L > p.src.Lcap || start < 0) {
    if (kKeys && unit == 0 && lane == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
    L = 0;  // zeros
  }
  const int rows = min(kLoadRows, p.n - r0);
  const int live = (int)max((int64_t)0, min((int64_t)rows, (int64_t)L - start - r0));  // rows below the length
  // the rows: up to the block's end from one place, then from another (a block
  // holds 16 at least); every load goes out, at row 0 where there is none
  const int lbs = 31 - __clz(p.bs), t = live > 0 ? start + r0 : 0, cross = p.bs - (t & (p.bs - 1));
  int64_t first = 0, second = 0;
  bool good1 = false, good2 = false;
  if (live > 0) {
    first = kv_row(p.src.pages, b, h, p.Hkv, p.src.Lcap, p.bs, t);
    good1 = good2 = first >= 0;
    second = first;
    if (p.src.pages.table && cross < live) {
      second = kv_row(p.src.pages, b, h, p.Hkv, p.src.Lcap, p.bs, ((t >> lbs) + 1) << lbs) - cross;
      good2 = second + cross >= 0;
    }
    if (!(good1 && good2) && x == 0) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
  }
  uint32_t w[kLoadRows], s[kLoadRows];
#pragma unroll
  for (int u = 0; u < kLoadRows; ++u) {
    const bool there = u < live && (u < cross ? good1 : good2);
    const int64_t row = there ? (u < cross ? first : second) + u : 0;
    if (kKeys) {
      w[u] = __ldg(reinterpret_cast<const uint32_t*>(p.src.k + row * kCodeBytes + (4 * c + g) * 4));
      s[u] = __ldg(p.src.ks + row * kGroups + g);
    } else {
      const uint16_t* o = reinterpret_cast<const uint16_t*>(p.src.v + row * kCodeBytes) + 8 * c + g;
      w[u] = (uint32_t)__ldg(o) | ((uint32_t)__ldg(o + 4) << 16);
      s[u] = __ldg(p.src.vs + row * kGroups + g);
    }
    if (!there) {  // a zero
      w[u] = 0x88888888u;
      s[u] = 0u;
    }
  }
  uint4* out = reinterpret_cast<uint4*>(kKeys ? p.k_out : p.v_out) + (pair * p.n + r0) * 16 + x;
#pragma unroll
  for (int u = 0; u < kLoadRows; ++u) {
    if (u < rows) {
      const uint32_t s2 = s[u] * 0x10001u;
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t y;
        if (kKeys) {  // channels 2i, 2i + 1 in nibbles i, i + 4
          y = w[u] >> (4 * i);
        } else {  // in nibbles 2i, 2i + 1
          const uint32_t v = w[u] >> (8 * i);
          y = (v & 0xFu) | (v << 12);
        }
        o[i] = hmul2_bf16(hadd2_bf16((y & 0x000F000Fu) | 0x43004300u, 0xC308C308u), s2);
      }
      out[u * 16] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

__global__ void __launch_bounds__(kKvThreads) kv4_load_kernel(Kv4LoadParams p) {
  pdl_wait();
  pdl_trigger_early();
  const int lane = threadIdx.x & 31, per = (p.n + 2 * kLoadRows - 1) / (2 * kLoadRows);
  const int64_t unit = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  const int64_t of = unit >> 1, pair = of / per;
  if (pair >= (int64_t)p.B * p.Hkv) return;
  if (unit & 1)
    load_rows<false>(p, pair, (int)(of - pair * per), lane);
  else
    load_rows<true>(p, pair, (int)(of - pair * per), lane);
}

cudaError_t launch_kv4_load(const Kv4LoadParams& p, cudaStream_t s) {
  const int64_t units = 2 * (int64_t)p.B * p.Hkv * ((p.n + 2 * kLoadRows - 1) / (2 * kLoadRows));
  return launch_pdl(kv4_load_kernel, dim3((unsigned)((units + kKvWarps - 1) / kKvWarps)), dim3(kKvThreads), 0, s, p);
}

// ------------------------------------------------------------- eviction: move
// The kept tokens' rows, scales and weights move to their new places
// (ascending, so blocks keep the time order) and the blocks' means are taken
// on the way.  A warp has keys or values of two consecutive destination
// blocks, one each half; rows are gathered, 8 in flight per lane (16 of
// 4 bits cost more in registers than they hid).  Destination
// weights behind the kept tokens become zero, so tokens appended later start
// at nothing.
template <bool kInt4, bool kKeys>
__device__ __forceinline__ void move_blocks(const EvictParams& p, int64_t pair, int i0, int lane) {
  constexpr uint32_t kNone = 0xFFFFFFFFu;
  constexpr int kFly = 8;  // rows in flight per lane
  const int half = lane >> 4, x = lane & 15, g = x >> 2, c = x & 3;
  const int b = (int)(pair / p.Hkv), h = (int)(pair - (int64_t)b * p.Hkv);
  const int bs = p.bs, lbs = 31 - __clz(bs);
  const int m = __ldg(p.dst_lens + b);  // written by the select kernel: min(L, n_keep), 0 for a bad length
  const int i = i0 + half, t0 = i << lbs;
  int n = max(0, min(bs, m - t0));  // this half's rows
  const int32_t* sel = p.sel + pair * p.n_keep + t0;
  if (kKeys && p.dst_acc) {
    const int end = min(bs, p.dst.Lcap - t0);
    for (int r = x; r < end; r += 16)
      p.dst_acc[pair * p.dst.Lcap + t0 + r] = r < n ? __ldg(p.acc + pair * p.src.Lcap + __ldg(sel + r)) : 0.f;
  }
  int64_t to0 = 0;
  if (n > 0) {
    to0 = kv_row(p.dst.pages, b, h, p.Hkv, p.dst.Lcap, bs, t0);
    if (to0 < 0) {
      if (kKeys) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);
      n = 0;
      to0 = 0;
    }
  }
  const int most = max(n, __shfl_xor_sync(0xffffffffu, n, 16));
  // a lane's bytes of a row: 16 of a bf16 row; of a 4-bit row the key word of
  // its 8 channels or the x-th value word, and its group's scale
  const int at = kInt4 ? (kKeys ? (4 * c + g) * 4 : x * 4) : x * 16;
  constexpr int kRow = kInt4 ? kCodeBytes : kHeadDim * 2;
  const uint8_t* src = (kKeys ? p.src.k : p.src.v) + at;
  uint8_t* dst = (kKeys ? p.dst.k : p.dst.v) + to0 * kRow + at;
  const uint16_t* src_s = (kKeys ? p.src.ks : p.src.vs) + g;
  uint16_t* dst_s = (kKeys ? p.dst.ks : p.dst.vs) + to0 * kGroups + g;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  bool bad = false;
  for (int r0 = 0; r0 < most; r0 += 16) {
    uint32_t my = kNone;  // lane's source row (a cache of 2^32 rows is larger than the memory)
    if (r0 + x < n) {
      const int t = __ldg(sel + r0 + x);
      if (p.src.pages.table) {
        const int page = __ldg(p.src.pages.table + (int64_t)b * p.src.pages.max_blocks + (t >> lbs));
        if (page >= 0 && page < p.src.pages.num_pages)
          my = ((uint32_t)(page * p.Hkv + h) << lbs) + (t & (bs - 1));
        else
          bad = true;
      } else {
        my = (uint32_t)pair * (uint32_t)p.src.Lcap + (uint32_t)t;
      }
    }
#pragma unroll
    for (int u0 = 0; u0 < 16; u0 += kFly) {
      if (r0 + u0 >= most) break;  // warp-uniform
      uint4 w[kFly];
      uint32_t s[kFly], from[kFly];
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        from[u] = __shfl_sync(0xffffffffu, my, 16 * half + u0 + u);
        const uint64_t row = from[u] != kNone ? from[u] : 0u;  // every load goes out, row 0 in place of none
        if constexpr (kInt4) {
          w[u].x = __ldg(reinterpret_cast<const uint32_t*>(src + row * kRow));
          s[u] = __ldg(src_s + row * kGroups);
        } else {
          w[u] = __ldg(reinterpret_cast<const uint4*>(src + row * kRow));
        }
      }
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        if (from[u] != kNone) {
          const int r = r0 + u0 + u;
          if constexpr (kInt4) {
            *reinterpret_cast<uint32_t*>(dst + r * kRow) = w[u].x;
            if (c == 0) dst_s[r * kGroups] = (uint16_t)s[u];
          } else {
            *reinterpret_cast<uint4*>(dst + r * kRow) = w[u];
          }
          if constexpr (kKeys) {
            if constexpr (kInt4) {
              float v[8];
              key_values(w[u].x, __uint_as_float(s[u] << 16), v);
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[e] += v[e];
            } else {
              acc[0] += bf16_lo(w[u].x);
              acc[1] += bf16_hi(w[u].x);
              acc[2] += bf16_lo(w[u].y);
              acc[3] += bf16_hi(w[u].y);
              acc[4] += bf16_lo(w[u].z);
              acc[5] += bf16_hi(w[u].z);
              acc[6] += bf16_lo(w[u].w);
              acc[7] += bf16_hi(w[u].w);
            }
          }
        }
      }
    }
  }
  if (kKeys && bad) set_status(p.dev_status, KIN_ERR_DEVICE_DATA);  // the row is left as it was
  if (kKeys && p.means) {
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {
      const int rows = __shfl_sync(0xffffffffu, n, 16 * hb);
      if (rows > 0) {
        const int64_t mrow = means_row_index(p.dst.pages, p.means_per_page, b, h, p.Hkv, p.nbcap_dst, i0 + hb);
        store_half_mean(p.means, p.means_flag, p.mean_rows, mrow, lane, hb, acc, (float)rows);
      }
    }
  }
}

template <bool kInt4>
__global__ void __launch_bounds__(kKvThreads) evict_move_kernel(EvictParams p) {
  pdl_wait();
  pdl_trigger_early();
  const int lane = threadIdx.x & 31, per = (p.nbcap_dst + 1) / 2;
  const int64_t unit = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  const int64_t of = unit >> 1, pair = of / per;
  if (pair >= (int64_t)p.B * p.Hkv) return;
  const int i0 = 2 * (int)(of - pair * per);
  if (unit & 1)
    move_blocks<kInt4, false>(p, pair, i0, lane);
  else
    move_blocks<kInt4, true>(p, pair, i0, lane);
}

cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t s) {
  const int64_t units = 2 * (int64_t)p.B * p.Hkv * ((p.nbcap_dst + 1) / 2);
  const dim3 grid((unsigned)((units + kKvWarps - 1) / kKvWarps));
  return p.src.int4 ? launch_pdl(evict_move_kernel<true>, grid, dim3(kKvThreads), 0, s, p)
                    : launch_pdl(evict_move_kernel<false>, grid, dim3(kKvThreads), 0, s, p);
}

}  // namespace kin
