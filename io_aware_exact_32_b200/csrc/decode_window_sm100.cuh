// Single-token attention with a sliding window, sinks and shared key/value heads, over a bf16 cache or a 4-bit
// cache (format: kv4_sm100.cuh).
//
// Sequence b's query sits at position L - 1 and sees the keys [max(0, L - window), L) and [0, sinks).  These
// are numbered 0 .. n - 1 (the sinks first); the list is cut into S equal parts (multiples of 64 keys), one CTA
// each, whose (m, l, O~) partials a second kernel merges with the two-block identity of the online softmax.  No
// other cache row is read.
//
// Bound: HBM (each cache byte serves at most 8 query heads here).  What the 4-bit form costs instead is
// instructions: at 6.5 TB/s an SM receives 46 codes a clock and issues 128 lane-instructions, so a code
// may cost at most 2.7 of them.  Hence, per warp and tile of 16 keys:
//  * both products run on mma.sync m16n8k16 with the cache as the 16-row operand and 8 query heads as the
//    8 columns (S = K q: rows are keys; O^T = V^T p: rows are channels), so a code is unpacked once for up to 8
//    heads, and loads go from global memory straight into the operand registers;
//  * a code is not converted: (word & 0x000f000f) is a pair of fp16 numbers c * 2^-24 (subnormal, exact in
//    the tensor core), (word & 0x00f000f0) one of c * 2^-20, whose factor 16 goes into q or the output.
//    5 instructions for 8 codes;
//  * K steps multiply the fp32 sums of their group; the -8 of (code - 8) is the sums' starting value;
//  * V steps multiply the weights, p * step in fp16 (11 bits; 2^-11 relative), transposed between the two
//    products by movmatrix; the -8 is a product of the same rounded weights with a constant row.
// fp16 range: q is scaled by a power of two per head so that its largest entry is in [2^14, 2^15); the
// running maximum is that of x + log2(step) (a power-of-two bound of the key's largest V step), so
// p * step stays below 2^15 whatever the steps.  The stale maximum is kept until a score outgrows it by 2^8.
// The bf16 form is the same with bf16 products; there p = hi + lo in two bf16 terms (16 bits), since its
// instruction budget is 3.5 times larger.
#pragma once

#include <cuda_fp16.h>

#include "kv4_sm100.cuh"

namespace fa {

constexpr int kDwWarps = 4;
constexpr int kDwTile = 16;                     // keys per warp tile
constexpr int kDwStep = kDwWarps * kDwTile;     // keys per CTA step

struct DecWinParams {
  const __nv_bfloat16* q;         // [B, H, d]
  const void* k;                  // bf16 rows or codes, [B, Hkv, Lmax, ...]
  const void* v;
  const __nv_bfloat16* k_steps;   // 4-bit cache only
  const __nv_bfloat16* v_steps;
  const int* seqlens;
  float* part_o;                  // [B * H * S, D] (S > 1)
  float* part_ml;                 // [B * H * S, 2]
  __nv_bfloat16* o;               // [B, H, D] (S == 1)
  float* lse;                     // [B, H] or null (S == 1)
  int Lmax, H, Hkv, group, hblocks, S;  // hblocks = ceil(group / 8)
  int window, sinks;
  float scale_log2;
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit entries (lane 4 r + c holds entries (r, 2 c) and (r, 2 c + 1)) transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// N consecutive 32-bit words (N = 1, 2 or a multiple of 4) from a 4 N-byte aligned address (16 at most).
template <int N>
__device__ __forceinline__ void ldg_words(uint32_t (&dst)[N], const void* src) {
  if constexpr (N == 1) {
    dst[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
  } else if constexpr (N == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
    dst[0] = x.x;
    dst[1] = x.y;
  } else {
    static_assert(N == 4, "16 bytes");
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
    dst[0] = x.x;
    dst[1] = x.y;
    dst[2] = x.z;
    dst[3] = x.w;
  }
}

// A warp's tile of 16 keys in registers.  Lane 4 g + t holds, of the K rows g and g + 8, the t-th quarter, and of
// the V rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9, the g-th eighth: the operand layout of the two products.
template <int D, bool Q4>
struct DwTile;

template <int D>
struct DwTile<D, true> {
  static constexpr int NG = D / kKv4Group;
  uint32_t k[2][NG];       // unit t of every group (8 codes each)
  uint32_t v[4][NG / 2];   // unit g of every group (4 codes each)
  uint32_t ks[2][NG / 2];  // steps of K rows g, g + 8 (bf16 pairs)
  uint32_t vs[2][NG / 2];  // steps of V rows g, g + 8

  // row(i): cache row (from the head's first) of list entry i.
  template <typename Row>
  __device__ __forceinline__ void load(const DecWinParams& p, size_t head_row, int g, int t, Row row) {
    const uint8_t* kc = static_cast<const uint8_t*>(p.k);
    const uint8_t* vc = static_cast<const uint8_t*>(p.v);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const size_t at = head_row + row(g + 8 * r);
      ldg_words<NG>(k[r], kc + at * (D / 2) + 4 * NG * t);
      ldg_words<NG / 2>(ks[r], p.k_steps + at * NG);
      ldg_words<NG / 2>(vs[r], p.v_steps + at * NG);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const size_t at = head_row + row(2 * t + (r & 1) + 8 * (r >> 1));
      ldg_words<NG / 2>(v[r], vc + at * (D / 2) + 2 * NG * g);
    }
  }
};

template <int D>
struct DwTile<D, false> {
  uint32_t k[2][D / 32][4];  // 16-byte chunks 4 c + t
  uint32_t v[4][D / 64][4];  // 16-byte chunks 8 c + g

  template <typename Row>
  __device__ __forceinline__ void load(const DecWinParams& p, size_t head_row, int g, int t, Row row) {
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(p.k);
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(p.v);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const size_t at = head_row + row(g + 8 * r);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) ldg_words<4>(k[r][c], kc + at * D + 8 * (4 * c + t));
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const size_t at = head_row + row(2 * t + (r & 1) + 8 * (r >> 1));
#pragma unroll
      for (int c = 0; c < D / 64; ++c) ldg_words<4>(v[r][c], vc + at * D + 8 * (8 * c + g));
    }
  }
};

// A warp's running state: 8 heads (columns); this lane keeps the maxima and (its keys' part of) the sums of
// heads 2 t and 2 t + 1, and O^T accumulators of two channels each per 16-channel tile.
template <int D, bool Q4>
struct DwState;

template <int D>
struct DwState<D, true> {
  static constexpr int NG = D / kKv4Group;
  uint32_t qf[NG][4];    // q of head g: fp16 pairs in the order of the unpacked K codes
  float c0[NG][2];       // -8 * 2^-24 * (sum of the group's q), heads 2 t, 2 t + 1
  float fx[2];           // what turns step-weighted sums into scores (log2 units)
  float m[2], l[2];
  float acc[NG][2][4];   // group, channels 4 g' + {0, 1} / {2, 3}
  float sum[4];          // row w of the tile: 2^-24 * sum of the rounded weights of group w

  __device__ __forceinline__ void init(const DecWinParams& p, const __nv_bfloat16* q, bool live, int g, int t) {
    float x[NG][8];
    float mx = 0.f;
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      uint32_t raw[4] = {0u, 0u, 0u, 0u};
      if (live) ldg_words<4>(raw, q + kKv4Group * w + 8 * t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[w][2 * i] = bf16lo_to_f32(raw[i]);
        x[w][2 * i + 1] = bf16hi_to_f32(raw[i]);
        mx = fmaxf(mx, fmaxf(fabsf(x[w][2 * i]), fabsf(x[w][2 * i + 1])));
      }
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // Power of two that brings the largest |q| to [2^14, 2^15); its exponent is kept inside fp32's normal range.
    const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 126);
    const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
    const float back = p.scale_log2 * __uint_as_float((uint32_t)(e - 14 + 127) << 23) * 16777216.f;
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[w][i] = __half2float(__float2half_rn(x[w][i] * up));
        s += x[w][i];
      }
      // K words unpack to code pairs (0, 4), 16 (1, 5), (2, 6), 16 (3, 7).
      qf[w][0] = pack_f16x2(x[w][0], x[w][4]);
      qf[w][1] = pack_f16x2(x[w][1] * 0.0625f, x[w][5] * 0.0625f);
      qf[w][2] = pack_f16x2(x[w][2], x[w][6]);
      qf[w][3] = pack_f16x2(x[w][3] * 0.0625f, x[w][7] * 0.0625f);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s *= -8.f / 16777216.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) c0[w][h] = __shfl_sync(0xffffffffu, s, 4 * (2 * t + h));
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[w][b][i] = 0.f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fx[h] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + h));
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = 0.f;
  }

  __device__ __forceinline__ void step(const DwTile<D, true>& x, bool ok0, bool ok1, int g) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      const uint32_t a = x.k[0][w], b = x.k[1][w];
      float d[4];
      mma_f16_16816(d, a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u, qf[w][0], qf[w][1],
                    c0[w][0], c0[w][1], c0[w][0], c0[w][1]);
      const uint32_t a8 = a >> 8, b8 = b >> 8;
      mma_f16_16816(d, a8 & 0x000f000fu, b8 & 0x000f000fu, a8 & 0x00f000f0u, b8 & 0x00f000f0u, qf[w][2], qf[w][3],
                    d[0], d[1], d[2], d[3]);
      const float s0 = (w & 1) ? bf16hi_to_f32(x.ks[0][w / 2]) : bf16lo_to_f32(x.ks[0][w / 2]);
      const float s1 = (w & 1) ? bf16hi_to_f32(x.ks[1][w / 2]) : bf16lo_to_f32(x.ks[1][w / 2]);
      s[0] = fmaf(s0, d[0], s[0]);
      s[1] = fmaf(s0, d[1], s[1]);
      s[2] = fmaf(s1, d[2], s[2]);
      s[3] = fmaf(s1, d[3], s[3]);
    }
    // Scores in log2 units; a key past the list has none.  e: log2 of a power of two above the key's V steps
    // (not below 2^-60, which keeps the sums in range where V is all but zero).
    float e[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t mx = x.vs[r][0];
      if constexpr (NG == 4) mx = __vmaxu2(mx, x.vs[r][1]);
      mx = max(mx & 0xffffu, mx >> 16);
      e[r] = fmaxf((float)((int)(mx >> 7) - 126), -60.f);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = ok0 ? s[h] * fx[h] : -INFINITY;
      s[2 + h] = ok1 ? s[2 + h] * fx[h] : -INFINITY;
    }
    const float y0 = fmaxf(s[0] + e[0], s[2] + e[1]), y1 = fmaxf(s[1] + e[0], s[3] + e[1]);
    if (__any_sync(0xffffffffu, y0 > m[0] + 14.f || y1 > m[1] + 14.f)) {
      float y[2] = {y0, y1};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) y[h] = fmaxf(y[h], __shfl_xor_sync(0xffffffffu, y[h], off));
        const float mn = fmaxf(m[h], y[h] - 6.f);
        const float f = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - mn);
        m[h] = mn;
        l[h] *= f;
#pragma unroll
        for (int w = 0; w < NG; ++w)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            acc[w][b][h] *= f;
            acc[w][b][2 + h] *= f;
          }
        sum[h] *= f;
      }
    }
    float pr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pr[i] = ex2_approx(s[i] - m[i & 1]);
    l[0] += pr[0] + pr[2];
    l[1] += pr[1] + pr[3];
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      float s0 = (w & 1) ? bf16hi_to_f32(x.vs[0][w / 2]) : bf16lo_to_f32(x.vs[0][w / 2]);
      float s1 = (w & 1) ? bf16hi_to_f32(x.vs[1][w / 2]) : bf16lo_to_f32(x.vs[1][w / 2]);
      const uint32_t b0 = movmatrix_trans(pack_f16x2(pr[0] * s0, pr[1] * s0));
      const uint32_t b1 = movmatrix_trans(pack_f16x2(pr[2] * s1, pr[3] * s1));
      const uint32_t sel = (w & 1) ? 0x7632u : 0x5410u;
      const uint32_t lo = __byte_perm(x.v[0][w / 2], x.v[1][w / 2], sel);
      const uint32_t hi = __byte_perm(x.v[2][w / 2], x.v[3][w / 2], sel);
      const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
      mma_f16_16816(acc[w][0], lo & 0x000f000fu, lo & 0x00f000f0u, hi & 0x000f000fu, hi & 0x00f000f0u, b0, b1,
                    acc[w][0][0], acc[w][0][1], acc[w][0][2], acc[w][0][3]);
      mma_f16_16816(acc[w][1], lo8 & 0x000f000fu, lo8 & 0x00f000f0u, hi8 & 0x000f000fu, hi8 & 0x00f000f0u, b0, b1,
                    acc[w][1][0], acc[w][1][1], acc[w][1][2], acc[w][1][3]);
      const uint32_t one = g == w ? 0x00010001u : 0u;
      mma_f16_16816(sum, one, 0u, one, 0u, b0, b1, sum[0], sum[1], sum[2], sum[3]);
    }
  }

  // O~ of this lane's channels: put(channel, head column, value).
  template <typename Put>
  __device__ __forceinline__ void finish(int g, int t, Put put) {
#pragma unroll
    for (int w = 0; w < NG; ++w)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float off = -8.f * __shfl_sync(0xffffffffu, sum[h], 4 * w + t);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int ch = kKv4Group * w + 4 * g + 2 * b;
          put(ch, 2 * t + h, (acc[w][b][h] + off) * 16777216.f);
          put(ch + 1, 2 * t + h, (acc[w][b][2 + h] * 0.0625f + off) * 16777216.f);
        }
      }
  }
};

template <int D>
struct DwState<D, false> {
  uint32_t qf[D / 32][4];  // q of head g, channels 8 (4 c + t) ..
  float fx;
  float m[2], l[2];
  float acc[D / 64][4][4];  // chunk 8 c + g, word: its two channels

  __device__ __forceinline__ void init(const DecWinParams& p, const __nv_bfloat16* q, bool live, int g, int t) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[c][i] = 0u;
      if (live) ldg_words<4>(qf[c], q + 8 * (4 * c + t));
    }
    fx = p.scale_log2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[c][j][i] = 0.f;
  }

  __device__ __forceinline__ void step(const DwTile<D, false>& x, bool ok0, bool ok1, int g) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      mma_bf16_16816(s, x.k[0][c][0], x.k[1][c][0], x.k[0][c][1], x.k[1][c][1], qf[c][0], qf[c][1]);
      mma_bf16_16816(s, x.k[0][c][2], x.k[1][c][2], x.k[0][c][3], x.k[1][c][3], qf[c][2], qf[c][3]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = ok0 ? s[h] * fx : -INFINITY;
      s[2 + h] = ok1 ? s[2 + h] * fx : -INFINITY;
    }
    const float y0 = fmaxf(s[0], s[2]), y1 = fmaxf(s[1], s[3]);
    if (__any_sync(0xffffffffu, y0 > m[0] + 8.f || y1 > m[1] + 8.f)) {
      float y[2] = {y0, y1};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) y[h] = fmaxf(y[h], __shfl_xor_sync(0xffffffffu, y[h], off));
        const float mn = fmaxf(m[h], y[h]);
        const float f = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - mn);
        m[h] = mn;
        l[h] *= f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[c][j][h] *= f;
            acc[c][j][2 + h] *= f;
          }
      }
    }
    float pr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pr[i] = ex2_approx(s[i] - m[i & 1]);
    l[0] += pr[0] + pr[2];
    l[1] += pr[1] + pr[3];
    const uint32_t h0 = pack_bf16x2(pr[0], pr[1]), h1 = pack_bf16x2(pr[2], pr[3]);
    const uint32_t r0 = pack_bf16x2(pr[0] - bf16lo_to_f32(h0), pr[1] - bf16hi_to_f32(h0));
    const uint32_t r1 = pack_bf16x2(pr[2] - bf16lo_to_f32(h1), pr[3] - bf16hi_to_f32(h1));
    const uint32_t b0 = movmatrix_trans(h0), b1 = movmatrix_trans(h1);
    const uint32_t d0 = movmatrix_trans(r0), d1 = movmatrix_trans(r1);
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = __byte_perm(x.v[0][c][j], x.v[1][c][j], 0x5410), a1 = __byte_perm(x.v[0][c][j], x.v[1][c][j], 0x7632);
        const uint32_t a2 = __byte_perm(x.v[2][c][j], x.v[3][c][j], 0x5410), a3 = __byte_perm(x.v[2][c][j], x.v[3][c][j], 0x7632);
        mma_bf16_16816(acc[c][j], a0, a1, a2, a3, b0, b1);
        mma_bf16_16816(acc[c][j], a0, a1, a2, a3, d0, d1);
      }
  }

  template <typename Put>
  __device__ __forceinline__ void finish(int g, int t, Put put) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ch = 8 * (8 * c + g) + 2 * j;
          put(ch, 2 * t + h, acc[c][j][h]);
          put(ch + 1, 2 * t + h, acc[c][j][2 + h]);
        }
  }
};

template <int D, bool Q4>
__global__ void __launch_bounds__(32 * kDwWarps) fa_decode_window_kernel(const DecWinParams p) {
  __shared__ float sm_o[kDwWarps][8][D + 4];
  __shared__ float sm_ml[kDwWarps][8][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int s_idx = blockIdx.x % p.S;
  int unit = blockIdx.x / p.S;
  const int hb = unit % p.hblocks;
  unit /= p.hblocks;  // b * Hkv + key/value head
  const int b = unit / p.Hkv;
  const int h0 = hb * 8;                      // first head of the group's 8
  const int nh = min(8, p.group - h0);
  const size_t head0 = (size_t)unit * p.group + h0;  // b * H + first query head

  const int L = min(max(p.seqlens[b], 0), p.Lmax);
  const int lo = max(0, L - p.window);  // first key of the window
  const int ns = min(p.sinks, lo);      // sinks before it
  const int n = ns + L - lo;
  const int chunk = ((n + p.S - 1) / p.S + kDwStep - 1) / kDwStep * kDwStep;
  const long long begin = (long long)chunk * s_idx;
  const int i0 = (int)min(begin, (long long)n), i1 = (int)min(begin + chunk, (long long)n);

  DwState<D, Q4> st;
  st.init(p, p.q + (head0 + min(g, nh - 1)) * D, g < nh, g, t);
  const size_t head_row = (size_t)unit * p.Lmax;
  const int jump = lo - ns;
  for (int i = i0 + warp * kDwTile; i < i1; i += kDwStep) {
    DwTile<D, Q4> x;
    // Entries past the end repeat the last one (a key the query sees); their weights are 0.
    x.load(p, head_row, g, t, [&](int r) -> size_t {
      const int k = min(i + r, i1 - 1);
      return (size_t)(k + (k >= ns ? jump : 0));
    });
    st.step(x, i + g < i1, i + g + 8 < i1, g);
  }
  // The warps' states meet in shared memory.
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) st.l[h] += __shfl_xor_sync(0xffffffffu, st.l[h], off);
  st.finish(g, t, [&](int ch, int head, float val) { sm_o[warp][head][ch] = val; });
  if (g == 0)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sm_ml[warp][2 * t + h][0] = st.m[h];
      sm_ml[warp][2 * t + h][1] = st.l[h];
    }
  __syncthreads();
  for (int idx = threadIdx.x; idx < nh * D; idx += 32 * kDwWarps) {
    const int h = idx / D, ch = idx % D;
    float mt = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDwWarps; ++w) mt = fmaxf(mt, sm_ml[w][h][0]);
    float o = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kDwWarps; ++w) {
      const float lw = sm_ml[w][h][1];
      if (lw != 0.f) {  // 0: no key (a NaN sum goes on as one)
        const float f = ex2_approx(sm_ml[w][h][0] - mt);
        o = fmaf(f, sm_o[w][h][ch], o);
        l = fmaf(f, lw, l);
      }
    }
    const size_t head = head0 + h;
    if (p.S == 1) {
      p.o[head * D + ch] = __float2bfloat16(l != 0.f ? o / l : 0.f);
      if (ch == 0 && p.lse) p.lse[head] = l != 0.f ? (mt + log2f(l)) * 0.6931471805599453f : -INFINITY;
    } else {
      p.part_o[(head * p.S + s_idx) * D + ch] = o;
      if (ch == 0) {
        p.part_ml[2 * (head * p.S + s_idx)] = l != l ? 0.f : mt;
        p.part_ml[2 * (head * p.S + s_idx) + 1] = l;
      }
    }
  }
}

}  // namespace fa
