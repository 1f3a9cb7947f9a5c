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
// Both kernels move bytes and nothing else (2 d bytes one way, 9 d / 16 the other): a thread holds 8 channels
// (16 bytes of bf16), four lanes a group, and each row is read and written in full 32-byte sectors.
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
  long long rows;             // B * Hkv * T
  int Hkv, T, Lmax;
};

// Cache row of row `r` of the [B, Hkv, T] rows, or -1 where it lies past the sequence's rows or outside the
// cache.
__device__ __forceinline__ long long kv4_cache_row(const Kv4RowsParams& p, long long r) {
  const long long bh = r / p.T;
  const int t = (int)(r - bh * p.T);
  const int b = (int)(bh / p.Hkv);
  const long long pos = (p.starts ? (long long)__ldg(p.starts + b) : 0ll) + t;
  if (t >= (p.lens ? __ldg(p.lens + b) : p.T) || pos < 0 || pos >= p.Lmax) return -1;
  return bh * p.Lmax + pos;
}

// The largest magnitude of a group, from its bf16 words' sign-free bits (which order like the magnitudes, with
// infinities and NaN on top), over the group's four lanes.
__device__ __forceinline__ uint32_t kv4_group_max(const uint4& v) {
  uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return max(m & 0xffffu, m >> 16);
}

// Code of x in a group of the given step (inv = 1 / step).  x and step have 8 significant bits each, so
// x / step is a tie (n + 1/2) exactly or at least 2^-10 away from one: rounding the product x * inv to a
// multiple of 2^-11 first (adding and taking away 1.5 * 2^12) restores the ties that the rounding of inv lost,
// and round_half_even then agrees with the exact quotient.
__device__ __forceinline__ uint32_t kv4_code(float x, float inv) {
  const float q = __fadd_rn(__fadd_rn(x * inv, 6144.f), -6144.f);
  const float n = fminf(fmaxf(rintf(q), -7.f), 7.f);
  return __float_as_uint(n + 12582920.f) & 0xfu;  // 1.5 * 2^23 + 8: the sum's low bits are n + 8
}

template <int D>
__global__ void __launch_bounds__(256) fa_kv4_write_kernel(const Kv4RowsParams p) {
  constexpr int TPR = D / 8;  // threads per row
  constexpr int NG = D / kKv4Group;
  const int which = blockIdx.y;  // 0: K, 1: V
  const long long r = (blockIdx.x * 256ll + threadIdx.x) / TPR;
  const int i = threadIdx.x % TPR;
  const int w = i / 4, u = i % 4;  // group, and the thread's place in it
  const long long dst = r < p.rows ? kv4_cache_row(p, r) : -1;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (dst >= 0) v = *reinterpret_cast<const uint4*>((which ? p.x[1] : p.x[0]) + r * D + 8 * i);
  const uint32_t amax = kv4_group_max(v);
  __nv_bfloat16 step = __float2bfloat16(__fdiv_rn(__uint_as_float(amax << 16), 7.f));
  const float s = __bfloat162float(step);
  const uint32_t word[4] = {v.x, v.y, v.z, v.w};
  uint32_t codes = 0;
  if (amax >= 0x7f80u) {
    step = __ushort_as_bfloat16((unsigned short)0x7fff);
    codes = 0x88888888u;
  } else if (s >= 0x1p-100f) {
    const float inv = __fdiv_rn(1.f, s);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      codes |= (kv4_code(bf16lo_to_f32(word[k]), inv) << (8 * k)) | (kv4_code(bf16hi_to_f32(word[k]), inv) << (8 * k + 4));
  } else {
    // Steps whose reciprocal is out of range, and 0: the quotients by division.
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = (k & 1) ? bf16hi_to_f32(word[k / 2]) : bf16lo_to_f32(word[k / 2]);
      codes |= kv4_code(s > 0.f ? __fdiv_rn(x, s) : 0.f, 1.f) << (4 * k);
    }
  }
  // V: the thread's two units (4 codes each) lie d / 32 half-words apart; lanes of neighbouring groups trade
  // halves so that each stores one word.
  const uint32_t give = (w & 1) ? codes & 0xffffu : codes >> 16;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
  if (dst < 0) return;
  uint32_t* row = reinterpret_cast<uint32_t*>((which ? p.codes[1] : p.codes[0]) + dst * (D / 2));
  if (which == 0)
    row[u * NG + w] = codes;
  else if (w & 1)
    row[((2 * u + 1) * NG + w - 1) / 2] = got | (codes & 0xffff0000u);
  else
    row[(2 * u * NG + w) / 2] = (codes & 0xffffu) | (got << 16);
  if (u == 0) (which ? p.steps[1] : p.steps[0])[dst * NG + w] = step;
}

template <int D>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(const Kv4RowsParams p) {
  constexpr int TPR = D / 8;
  constexpr int NG = D / kKv4Group;
  const int which = blockIdx.y;
  const long long r = (blockIdx.x * 256ll + threadIdx.x) / TPR;
  const int i = threadIdx.x % TPR;
  const int w = i / 4, u = i % 4;
  const long long src = r < p.rows ? kv4_cache_row(p, r) : -1;
  uint32_t codes = 0;
  float s = 0.f;
  if (src >= 0) {
    const uint32_t* row = reinterpret_cast<const uint32_t*>((which ? p.codes[1] : p.codes[0]) + src * (D / 2));
    codes = which == 0 ? row[u * NG + w] : row[(w & 1) ? ((2 * u + 1) * NG + w - 1) / 2 : (2 * u * NG + w) / 2];
    s = __bfloat162float((which ? p.steps[1] : p.steps[0])[src * NG + w]);
  }
  const uint32_t give = (w & 1) ? codes & 0xffffu : codes >> 16;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
  if (src < 0) return;
  if (which == 1) codes = (w & 1) ? got | (codes & 0xffff0000u) : (codes & 0xffffu) | (got << 16);
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)  // step * (code - 8) is exact in fp32; one rounding to bf16
    o[k] = pack_bf16x2(s * (float)((int)((codes >> (8 * k)) & 0xfu) - 8), s * (float)((int)((codes >> (8 * k + 4)) & 0xfu) - 8));
  *reinterpret_cast<uint4*>((which ? p.out[1] : p.out[0]) + r * D + 8 * i) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace fa
