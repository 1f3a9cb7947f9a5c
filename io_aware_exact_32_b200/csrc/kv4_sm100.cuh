// 4-bit key/value cache: rows quantised as they are written, and read back.
//
// Format.  The d channels of a token's head vector form groups of 32.  A group has
//     step = bf16(max |x| / 7),   code = clamp(round_half_even(x / step), -7, 7) + 8   (4 bits),
// and stands for step * (code - 8); a group of zeros has step 0 and codes 8, a group with an infinity or
// NaN has step NaN.  One bf16 step per 32 codes: 4.5 bits per channel.
//
// Code order in a row, chosen for the decode kernel's matrix-instruction operands (decode_window_sm100.cuh),
// which read a group's codes without crossing lanes: a group's channels are cut into units (8 channels for K,
// 4 for V), unit u of group g sits at unit position u * (d / 32) + g, a unit's first channel in its lowest
// nibble.
//
// Both kernels only move bytes, 2.56 a channel.  At 6.5 TB/s an SM moves 23 a clock (at 1.9 GHz), 9 channels, for which it
// can issue 14 lane-instructions each.  So a thread takes 16 channels of a row (two lanes a group), so that what is done
// once a row, a group or a thread is shared by as many channels as its registers hold, and packed fp32 pairs do the
// arithmetic.  With 8 channels a thread a prompt of B4 H8 T2048..4096 d128 took 39 us, write and read back; so it takes
// 32 to 34 us, each way about 17 us for 8.8 us of bytes.  Per channel the write then issues 14.2 and the read 12.6
// lane-instructions, those of the threads of rows past the sequences' ends among them: about what the bytes leave time for
// if no slot stayed empty, and 63 to 65% of the slots (52 to 62% of the ALU) are used.  Each row is read and written in
// whole 32-byte sectors.
#pragma once

#include "sm100_ptx.cuh"

namespace fa {

constexpr int kKv4Group = 32;

struct Kv4RowsParams {
  const __nv_bfloat16* x[2];  // write: new K, V rows [B, Hkv, T, d]
  __nv_bfloat16* out[2];      // read: K, V rows [B, Hkv, T, d]
  uint8_t* codes[2];          // [B, Hkv, Lmax, d / 2]
  __nv_bfloat16* steps[2];    // [B, Hkv, Lmax, d / 32]
  const int* starts;          // [B] position of each sequence's first row, or null (0)
  const int* lens;            // [B] rows of each sequence, or null (T)
  unsigned rows;              // B * Hkv * T
  int Hkv, T, Lmax;
};

// Walks a thread's rows of [B, Hkv, T]: row(): the cache row of the current one, or -1 where it lies past the
// sequence's rows or outside the cache (or past all rows).
struct Kv4Walk {
  const Kv4RowsParams& p;
  unsigned r, bh;
  int t, start, len;

  __device__ __forceinline__ Kv4Walk(const Kv4RowsParams& params, unsigned row0) : p(params), r(row0) {
    bh = r / (unsigned)p.T;
    t = (int)(r - bh * p.T);
    sequence();
  }
  __device__ __forceinline__ void sequence() {
    if (r >= p.rows) return;
    const int b = (int)(bh / (unsigned)p.Hkv);
    start = p.starts ? __ldg(p.starts + b) : 0;
    len = p.lens ? min(__ldg(p.lens + b), p.T) : p.T;
  }
  __device__ __forceinline__ long long row() const {
    if (r >= p.rows || t >= len) return -1;
    const long long pos = (long long)start + t;
    return pos < 0 || pos >= p.Lmax ? -1 : (long long)bh * p.Lmax + pos;
  }
  __device__ __forceinline__ void advance(int by) {
    r += by;
    t += by;
    if (t >= p.T) {
      const unsigned over = (unsigned)t / (unsigned)p.T;
      bh += over;
      t -= (int)over * p.T;
      sequence();
    }
  }
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest magnitude of 16 channels, from their bf16 words' sign-free bits (which order like the magnitudes, with
// infinities and NaN on top), in both halves.
__device__ __forceinline__ uint32_t kv4_max(const uint4 (&v)[2]) {
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu),
                             __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu)));
  return __vmaxu2(m, (m >> 16) | (m << 16));
}

// Bits of 1.5 * 2^23 + (code of x in a group of the given step), for pairs of quotients q = x / step that are good to
// 2^-20.  x and step have 8 significant bits each, so x / step is a tie (n + 1/2) exactly or at least 2^-10 away from
// one: rounding q to a multiple of 2^-11 first (adding and taking away 1.5 * 2^12) restores the ties, and adding
// 1.5 * 2^23 + 8 then rounds half to even.
__device__ __forceinline__ uint2 kv4_code_bits(float2 q) {
  const float2 a = fadd2(fadd2(q, make_float2(6144.f, 6144.f)), make_float2(-6144.f, -6144.f));
  const float2 c = fadd2(a, make_float2(12582920.f, 12582920.f));
  return make_uint2(__float_as_uint(c.x), __float_as_uint(c.y));
}
// Eight codes, the first in the lowest nibble, from their kv4_code_bits: the constant part of the bits comes off at
// the end (mod 2^32).
__device__ __forceinline__ uint32_t kv4_pack(const uint2 (&c)[4]) {
  uint32_t acc = c[3].y;
  acc = acc * 16u + c[3].x;
#pragma unroll
  for (int k = 2; k >= 0; --k) {
    acc = acc * 16u + c[k].y;
    acc = acc * 16u + c[k].x;
  }
  return acc - 0x4b400000u * 0x11111111u;
}

// Eight codes of the channels in v, for a group whose step has the reciprocal inv.
__device__ __forceinline__ uint32_t kv4_codes8(const uint4& v, float inv) {
  const uint32_t word[4] = {v.x, v.y, v.z, v.w};
  uint2 c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = kv4_code_bits(fmul2(make_float2(bf16lo_to_f32(word[k]), bf16hi_to_f32(word[k])), make_float2(inv, inv)));
  return kv4_pack(c);
}
// The same for steps down to 0, rounded to few bits or to none: quotients by division, clamped.
__device__ __noinline__ uint32_t kv4_codes8_tiny(uint4 v, float step) {
  const uint32_t word[4] = {v.x, v.y, v.z, v.w};
  auto q = [&](float y) { return step > 0.f ? fminf(fmaxf(__fdiv_rn(y, step), -7.f), 7.f) : 0.f; };
  uint2 c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = kv4_code_bits(make_float2(q(bf16lo_to_f32(word[k])), q(bf16hi_to_f32(word[k]))));
  return kv4_pack(c);
}

// R rows per thread, whose loads are in flight together: 2 where that still leaves every SM two blocks, else 1 (4 rows:
// 63 registers, the prompt above 35.5 us).
template <int D, int R>
__global__ void __launch_bounds__(256) fa_kv4_write_kernel(const Kv4RowsParams p) {
  constexpr int TPR = D / 16;  // threads per row
  constexpr int NG = D / kKv4Group;
  const int which = blockIdx.y;  // 0: K, 1: V
  const __nv_bfloat16* x = which ? p.x[1] : p.x[0];
  uint8_t* out = which ? p.codes[1] : p.codes[0];
  __nv_bfloat16* steps = which ? p.steps[1] : p.steps[0];
  const unsigned r0 = blockIdx.x * (256u / TPR * R) + threadIdx.x / TPR;
  const int i = threadIdx.x % TPR;
  const int w = i / 2, h = i % 2;  // group, and its half that this thread has
  // The thread's two words of a row: K, units 2 h and 2 h + 1 of its group; V (units 4 h .. 4 h + 3), those two words
  // of its group and its neighbour's that fall to it: an even group's thread has units 4 h, 4 h + 1, an odd one's the
  // other two.
  const int at0 = which == 0 ? 2 * h * NG + w : ((4 * h + 2 * (w & 1)) * NG + (w & ~1)) / 2;
  const int at1 = at0 + (which == 0 ? NG : NG / 2);
  long long dst[R];
  uint4 val[R][2];
  Kv4Walk walk(p, r0);
#pragma unroll
  for (int n = 0; n < R; ++n) {
    if (n > 0) walk.advance(256 / TPR);
    dst[n] = walk.row();
    val[n][0] = val[n][1] = make_uint4(0u, 0u, 0u, 0u);
    if (dst[n] >= 0) {
      const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)(r0 + n * (256u / TPR)) * D + 16 * i);
      val[n][0] = __ldcs(src);
      val[n][1] = __ldcs(src + 1);
    }
  }
#pragma unroll
  for (int n = 0; n < R; ++n) {
    if (__all_sync(0xffffffffu, dst[n] < 0)) continue;
    uint32_t amax = kv4_max(val[n]);
    amax = __vmaxu2(amax, __shfl_xor_sync(0xffffffffu, amax, 1)) & 0xffffu;
    // amax / 7 is never within 2^-12 of a bf16 tie (amax has 8 bits), so the fp32 product rounds like the quotient.
    __nv_bfloat16 step = __float2bfloat16(__uint_as_float(amax << 16) * (1.f / 7.f));
    const float s = __bfloat162float(step);
    uint32_t c0, c1;
    if (amax >= 0x7f80u) {
      step = __ushort_as_bfloat16((unsigned short)0x7fff);
      c0 = c1 = 0x88888888u;
    } else if (s >= 0x1p-100f) {  // |x / step| < 7.03: no clamp
      const float inv = rcp_approx(s);
      c0 = kv4_codes8(val[n][0], inv);
      c1 = kv4_codes8(val[n][1], inv);
    } else {
      c0 = kv4_codes8_tiny(val[n][0], s);
      c1 = kv4_codes8_tiny(val[n][1], s);
    }
    if (which == 1) {
      // Lanes of neighbouring groups trade the codes that fall to the other.
      const uint32_t got = __shfl_xor_sync(0xffffffffu, (w & 1) ? c0 : c1, 2);
      const uint32_t lo = (w & 1) ? got : c0, hi = (w & 1) ? c1 : got;
      c0 = __byte_perm(lo, hi, 0x5410);
      c1 = __byte_perm(lo, hi, 0x7632);
    }
    if (dst[n] < 0) continue;
    uint32_t* row = reinterpret_cast<uint32_t*>(out + dst[n] * (D / 2));
    row[at0] = c0;
    row[at1] = c1;
    if (h == 0) steps[dst[n] * NG + w] = step;
  }
}

template <int D, int R>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(const Kv4RowsParams p) {
  constexpr int TPR = D / 16;
  constexpr int NG = D / kKv4Group;
  const int which = blockIdx.y;
  const uint8_t* in = which ? p.codes[1] : p.codes[0];
  const __nv_bfloat16* steps = which ? p.steps[1] : p.steps[0];
  __nv_bfloat16* out = which ? p.out[1] : p.out[0];
  const unsigned r0 = blockIdx.x * (256u / TPR * R) + threadIdx.x / TPR;
  const int i = threadIdx.x % TPR;
  const int w = i / 2, h = i % 2;
  const int at0 = which == 0 ? 2 * h * NG + w : ((4 * h + 2 * (w & 1)) * NG + (w & ~1)) / 2;  // as in the write
  const int at1 = at0 + (which == 0 ? NG : NG / 2);
  bool live[R];
  uint32_t word[R][2];
  float st[R];
  Kv4Walk walk(p, r0);
#pragma unroll
  for (int n = 0; n < R; ++n) {
    if (n > 0) walk.advance(256 / TPR);
    const long long src = walk.row();
    live[n] = src >= 0;
    word[n][0] = word[n][1] = 0u;
    st[n] = 0.f;
    if (live[n]) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(in + src * (D / 2));
      word[n][0] = row[at0];
      word[n][1] = row[at1];
      st[n] = __bfloat162float(steps[src * NG + w]);
    }
  }
#pragma unroll
  for (int n = 0; n < R; ++n) {
    if (__all_sync(0xffffffffu, !live[n])) continue;
    uint32_t c[2] = {word[n][0], word[n][1]};
    if (which == 1) {
      const uint32_t lo = __byte_perm(c[0], c[1], 0x5410), hi = __byte_perm(c[0], c[1], 0x7632);  // even, odd group's
      const uint32_t got = __shfl_xor_sync(0xffffffffu, (w & 1) ? lo : hi, 2);
      c[0] = (w & 1) ? got : lo;
      c[1] = (w & 1) ? hi : got;
    }
    if (!live[n]) continue;
    uint4* dst = reinterpret_cast<uint4*>(out + (size_t)(r0 + n * (256u / TPR)) * D + 16 * i);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // code - 8 from the low bits of 2^23 + code; step * (code - 8) is exact in fp32; one rounding to bf16.
      auto with = [&](int k) { return __uint_as_float(((c[b] >> (4 * k)) & 0xfu) | 0x4b000000u); };
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 y = fmul2(fadd2(make_float2(with(2 * k), with(2 * k + 1)), make_float2(-8388616.f, -8388616.f)),
                               make_float2(st[n], st[n]));
        o[k] = pack_bf16x2(y.x, y.y);
      }
      __stcs(dst + b, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

}  // namespace fa
