// Single-token attention with a sliding window, sinks and shared key/value heads, over a bf16 cache or a 4-bit
// cache (format: kv4_sm100.cuh).
//
// Sequence b's query sits at position L - 1 and sees the keys [max(0, L - window), L) and [0, sinks).  These
// are numbered 0 .. n - 1 (the sinks first); no other cache row is read.  A unit is a sequence's keys under one
// key/value head and up to 8 of its query heads.  CTAs work on parts of units, and where a unit has several, a second
// kernel merges their (m, l, O~) or (m, l, O) partials with the two-block identity of the online softmax:
//  * bf16 cache: parts of at most 1024 keys, which the hardware deals out (the pass is bound by memory, whose
//    speed differs from SM to SM);
//  * 4-bit cache: one wave of CTAs, each with an equal share of the list of all units' steps, whose loads run
//    ahead across the ends of units (the pass is bound by instructions, and starting and ending a part costs as
//    much as 500 keys).
//
// Bound: HBM (each cache byte serves at most 8 query heads here).  What the 4-bit form costs instead is
// instructions: at 6.5 TB/s an SM receives 41 codes a clock (at 1.9 GHz) and issues 128 lane-instructions, so a code
// may cost at most 3.1 of them.  Measured, both kernels of a call: bf16 B32 H32/8 L1024..8192 window 4096 82 us
// (5.5 TB/s of visible rows), B1 H32/32 L8192 window 1024 14 us (launches and one pass's latency); 4 bits B32 H32/8
// L1024..8192 51 to 56 us (3.0 to 3.3 TB/s; the issue slots are 48% and the ALU 40% busy, three CTAs of four warps an
// SM do not fill more of the gaps, four spill), B1 H16/4 L65536 22 us.
// Hence, per warp and tile of 16 keys:
//  * both products run on mma.sync m16n8k16 with the cache as the 16-row operand and 8 query heads as the
//    8 columns (S = K q: rows are keys; O^T = V^T p: rows are channels), so a code is unpacked once for up to 8
//    heads, and loads go from global memory straight into the operand registers;
//  * a K code is not converted: (word & 0x000f000f) is a pair of fp16 numbers c * 2^-24 (subnormal, exact in
//    the tensor core), (word & 0x00f000f0) one of c * 2^-20, whose factor 16 goes into q: 5 instructions for
//    8 codes.  The steps multiply the fp32 sums of their group, and the -8 of (code - 8) is the sums'
//    starting value;
//  * a V code becomes code - 8 (or 16 times that) by or-ing 1024 and subtracting, 9 instructions for 8: its sums
//    run over the whole cache, and subnormal codes with the -8 taken off at the end left a bias of 1e-5 of
//    8 step (the tensor core aligns products by their exponent fields) that is 3e-3 of the output at 65536
//    keys;
//  * V steps multiply the weights, p * step in fp16 (11 bits; 2^-11 relative), transposed between the two
//    products by movmatrix.
// Ranges: q is scaled by a power of two per head so that its largest entry is in [2^14, 2^15).  The weights' base m is an
// integer, kMargin above the maximum it was set at, so that weights are at most 1 until a score outgrows that maximum by
// 2^kMargin and m moves; the sums l and the LSE see nothing of V.  p * step enters fp16 in units of its own per head and
// group, a power of two, of which the largest product of the warp's keys so far has 2^kFine or more (what fp16's end
// takes off any product is then below 2^-28 of that largest one, and of a channel 2^-25, as in an fp32 sum) and no
// product has 2^16; unit and accumulators change when a step comes that does not fit.  Heads, groups and keys of any
// sizes so leave each other's bits alone.  Parts hold O, normalised by their own l, so that no sum outgrows the values it
// averages: V may use all of bf16's range.  One unit for all heads and groups, tied to the largest step, lost a group
// 2^-28 the size of another; its calls took 51.6 us (B32 H32/8 L1024..8192), 22.6 us (B1 H16/4 L65536) and 39.0 us (the
// first with d = 64) where these take 52.3, 22.6 and 40.0 (calls in a row), and 56.0 where the rows' sizes are spread as
// exp(1.5 N(0, 1)) (these 61.6: the general way in refit).  It hangs on the short way for a part's first keys: with a test
// of every product for the end of fp16's range the first of these took 61 to 67 us (registers), with the general way for
// the first keys 58.
// The bf16 form is the same with bf16 products; there p = hi + lo in two bf16 terms (16 bits), since its
// instruction budget is 3.5 times larger.
#pragma once

#include <cuda_fp16.h>

#include "kv4_sm100.cuh"

namespace fa {

constexpr int kDwWarps = 4;
constexpr int kDwTile = 16;   // keys per matrix-instruction tile
constexpr int kDwHeads = 8;   // query heads per pass over a unit's keys

struct DecWinParams {
  const __nv_bfloat16* q;         // [B, H, d]
  const void* k;                  // bf16 rows or codes, [B, Hkv, Lmax, ...]
  const void* v;
  const __nv_bfloat16* k_steps;   // 4-bit cache only
  const __nv_bfloat16* v_steps;
  const int* seqlens;
  float* part_o;                  // partials: bf16 O~ [B * H, S, D], 4 bits O [2 grid, 8, D]
  float* part_ml;                 // their (m, l): the same without D, 2
  __nv_bfloat16* o;               // [B, H, D]
  float* lse;                     // [B, H] or null
  int B, Lmax, H, Hkv, group, hblocks;  // hblocks = ceil(group / 8)
  int S, min_chunk;                  // bf16: parts per unit, at most; keys in a part, at least
  int grid;                          // 4 bits: CTAs
  int window, sinks;
  float scale_log2;
};

// What a sequence's query sees.
struct DwKeys {
  int n, ns, jump;  // keys; sinks before the window; list entry e >= ns is cache row e + jump
};
__device__ __forceinline__ DwKeys dw_keys(const DecWinParams& p, int b) {
  DwKeys k;
  const int L = min(max(__ldg(p.seqlens + b), 0), p.Lmax);
  const int lo = max(0, L - p.window);
  k.ns = min(p.sinks, lo);
  k.n = k.ns + L - lo;
  k.jump = lo - k.ns;
  return k;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (a & m) | k in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t k) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(m), "r"(k));
  return d;
}
// Differences of fp16 pairs.
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
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

// N consecutive 32-bit words (N = 1, 2 or 4) from a 4 N-byte aligned address.
template <int N, typename Src>
__device__ __forceinline__ void load_words(uint32_t (&dst)[N], const Src* src) {  // read-only data
  static_assert(N == 1 || N == 2 || N == 4, "4, 8 or 16 bytes");
  if constexpr (N == 1) {
    dst[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
  } else if constexpr (N == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
    dst[0] = x.x;
    dst[1] = x.y;
  } else {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
    dst[0] = x.x;
    dst[1] = x.y;
    dst[2] = x.z;
    dst[3] = x.w;
  }
}
// N consecutive words from shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&dst)[N], const uint8_t* src) {
  if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(src);
    dst[0] = x.x;
    dst[1] = x.y;
  } else {
    static_assert(N == 4, "8 or 16 bytes");
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    dst[0] = x.x;
    dst[1] = x.y;
    dst[2] = x.z;
    dst[3] = x.w;
  }
}

// A tile of 16 keys.  Lane 4 g + t works on, of the K rows g and g + 8, the t-th quarter, and of the V rows 2 t,
// 2 t + 1, 2 t + 8, 2 t + 9, the g-th eighth: the operand layout of the two products.  Base: where the lane's parts
// of a unit's rows g (K, steps) and 2 t (V) lie (a unit's rows span at most 2^32 bytes).  Loads name the tile's
// first row and `at`, the distance of tile row r from it: r itself, or where a step is cut by the list's jump or end
// the row of each entry.
struct DwRows {
  __device__ __forceinline__ int operator()(int r) const { return r; }
};

// bf16 rows in registers.
template <int D, bool Q4>
struct DwTile {
  static_assert(!Q4, "bf16 rows");
  // 168 registers; four CTAs at 128 spill (1.15x).
  static constexpr int NT = 1, STEP = kDwWarps * kDwTile, CTAS = 3;
  uint32_t k[2][D / 32][4];       // 16-byte chunks 4 c + t
  uint32_t v[4][D / 64][4];       // 16-byte chunks 8 c + g

  struct Base {
    const uint8_t *k, *v;
    __device__ __forceinline__ void set(const DecWinParams& p, size_t row, int g, int t) {
      k = static_cast<const uint8_t*>(p.k) + (row + g) * (2 * D) + 16 * t;
      v = static_cast<const uint8_t*>(p.v) + (row + 2 * t) * (2 * D) + 16 * g;
    }
  };
  template <typename At>
  __device__ __forceinline__ void load_k(const Base& base, uint32_t row, int g, int, At at) {
    const uint8_t* kc = base.k + row * (2u * D);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) load_words<4>(k[r][c], kc + (long long)(at(g + 8 * r) - g) * (2 * D) + 64 * c);
  }
  template <typename At>
  __device__ __forceinline__ void load_v(const Base& base, uint32_t row, int, int t, At at) {
    const uint8_t* vc = base.v + row * (2u * D);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        load_words<4>(v[r][c], vc + (long long)(at(2 * t + (r & 1) + 8 * (r >> 1)) - 2 * t) * (2 * D) + 128 * c);
  }
};

// Codes and steps.
template <int D>
struct DwTile<D, true> {
  static constexpr int NG = D / kKv4Group;
  // Two tiles at a time, whose chains of dependent instructions fill each other's gaps.
  static constexpr int NT = 2, STEP = kDwWarps * kDwTile * NT, CTAS = 3;
  uint32_t k[2][NG];       // unit t of every group (8 codes each)
  uint32_t ks[2][NG / 2];  // steps of K rows g, g + 8 (bf16 pairs)
  uint32_t v[4][NG / 2];   // unit g of every group (4 codes each)
  uint32_t vs[2][NG / 2];  // steps of V rows g, g + 8

  struct Base {
    const uint8_t *k, *v, *ks, *vs;
    __device__ __forceinline__ void set(const DecWinParams& p, size_t row, int g, int t) {
      k = static_cast<const uint8_t*>(p.k) + (row + g) * (D / 2) + 4 * NG * t;
      v = static_cast<const uint8_t*>(p.v) + (row + 2 * t) * (D / 2) + 2 * NG * g;
      ks = reinterpret_cast<const uint8_t*>(p.k_steps + (row + g) * NG);
      vs = reinterpret_cast<const uint8_t*>(p.v_steps + (row + g) * NG);
    }
  };
  // Tile n of the rows from `row` on (n a constant, so that it ends up in the loads' immediate offsets).
  template <typename At>
  __device__ __forceinline__ void load_k(const Base& base, uint32_t row, int n, int g, int, At at) {
    const uint8_t *kc = base.k + row * (D / 2) + n * (kDwTile * D / 2);
    const uint8_t *st = base.ks + row * (2 * NG) + n * (kDwTile * 2 * NG);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const long long d = at(g + 8 * r) - g;
      load_words<NG>(k[r], kc + d * (D / 2));
      load_words<NG / 2>(ks[r], st + d * (2 * NG));
    }
  }
  template <typename At>
  __device__ __forceinline__ void load_v(const Base& base, uint32_t row, int n, int g, int t, At at) {
    const uint8_t *vc = base.v + row * (D / 2) + n * (kDwTile * D / 2);
    const uint8_t *st = base.vs + row * (2 * NG) + n * (kDwTile * 2 * NG);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      load_words<NG / 2>(v[r], vc + (long long)(at(2 * t + (r & 1) + 8 * (r >> 1)) - 2 * t) * (D / 2));
#pragma unroll
    for (int r = 0; r < 2; ++r) load_words<NG / 2>(vs[r], st + (long long)(at(g + 8 * r) - g) * (2 * NG));
  }
};

// A warp's running state: 8 heads (columns); this lane keeps the maxima and (its keys' part of) the sums of
// heads 2 t and 2 t + 1, and O^T accumulators of two channels each per 16-channel tile.
template <int D, bool Q4>
struct DwState;

template <int D>
struct DwState<D, true> {
  static constexpr int NG = D / kKv4Group;
  // The queries' operands, in shared memory, the same for all warps (by lane): q of head g as fp16 pairs in the order
  // of the unpacked K codes (16 bytes a group), -8 * 2^-24 * (sum of the group's q) of heads 2 t, 2 t + 1 (8 bytes
  // a group), and what turns their step-weighted sums into scores in log2 units (8 bytes).
  static constexpr int Q_BYTES = 32 * (NG * 24 + 8);
  float fx[2];
  float m[2], l[2];      // weights are 2^(score - m), l their sum
  float top[2];          // scores up to here (m, in units of fx) need no new m
  uint32_t vtop[NG / 2]; // steps of each group up to here (bf16 pairs) need no new units
  // Shared memory of the warp, 4 w + t, heads 2 t and 2 t + 1: the factors (1 / unit) of group w's products weight * step
  // for fp16, and lower bounds of the largest product so far.
  float4* unit;
  float acc[NG][2][4];   // group, channels 4 g + {0, 1} / {2, 3}, in those units; the odd channels times 16

  // By one warp, q being head g's row (live: there is one).
  static __device__ __forceinline__ void prepare(const DecWinParams& p, const __nv_bfloat16* q, bool live, int g, int t,
                                                 uint8_t* sm_q) {
    const int lane = 4 * g + t;
    float x[NG][8];
    float mx = 0.f;
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      uint32_t raw[4] = {0u, 0u, 0u, 0u};
      if (live) load_words<4>(raw, q + kKv4Group * w + 8 * t);
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
    const float back = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(e - 14 + 127) << 23) * 16777216.f, 1e-37f);
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[w][i] = __half2float(__float2half_rn(x[w][i] * up));
        s += x[w][i];
      }
      // K words unpack to code pairs (0, 4), 16 (1, 5), (2, 6), 16 (3, 7).
      reinterpret_cast<uint4*>(sm_q)[32 * w + lane] =
          make_uint4(pack_f16x2(x[w][0], x[w][4]), pack_f16x2(x[w][1] * 0.0625f, x[w][5] * 0.0625f),
                     pack_f16x2(x[w][2], x[w][6]), pack_f16x2(x[w][3] * 0.0625f, x[w][7] * 0.0625f));
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s *= -8.f / 16777216.f;
      const float s0 = __shfl_sync(0xffffffffu, s, 8 * t), s1 = __shfl_sync(0xffffffffu, s, 8 * t + 4);
      reinterpret_cast<float2*>(sm_q + NG * 512)[32 * w + lane] = make_float2(s0, s1);
    }
    const float f0 = __shfl_sync(0xffffffffu, back, 8 * t), f1 = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    reinterpret_cast<float2*>(sm_q + NG * 768)[lane] = make_float2(f0, f1);
  }
  // By every warp, once the operands are there.
  __device__ __forceinline__ void start(const uint8_t* sm_q, float4* units, int lane) {
    unit = units;
    if (lane < 4 * NG) unit[lane] = make_float4(pow2(kFinest), pow2(kFinest), 0.f, 0.f);
    __syncwarp();
    const float2 f = reinterpret_cast<const float2*>(sm_q + NG * 768)[lane];
    fx[0] = f.x;
    fx[1] = f.y;
#pragma unroll
    for (int w = 0; w < NG; ++w)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[w][b][i] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m[h] = top[h] = -INFINITY;
      l[h] = 0.f;
    }
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) vtop[w] = 0u;
  }

  // Scores of keys g (s[.][0], s[.][1]) and g + 8 of N tiles for heads 2 t and 2 t + 1, in units of fx.
  template <int N>
  __device__ __forceinline__ void scores(const DwTile<D, true> (&x)[N], const uint8_t* sm_q, int lane,
                                         float (&s)[N][4]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      uint32_t qf[4];
      lds_words<4>(qf, sm_q + 16 * (32 * w + lane));
      const float2 c0 = *reinterpret_cast<const float2*>(sm_q + NG * 512 + 8 * (32 * w + lane));
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint32_t a = x[n].k[0][w], b = x[n].k[1][w];
        float d[4] = {c0.x, c0.y, c0.x, c0.y};
        mma_f16_16816(d, a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u, qf[0], qf[1]);
        const uint32_t a8 = a >> 8, b8 = b >> 8;
        mma_f16_16816(d, a8 & 0x000f000fu, b8 & 0x000f000fu, a8 & 0x00f000f0u, b8 & 0x00f000f0u, qf[2], qf[3]);
        const float s0 = (w & 1) ? bf16hi_to_f32(x[n].ks[0][w / 2]) : bf16lo_to_f32(x[n].ks[0][w / 2]);
        const float s1 = (w & 1) ? bf16hi_to_f32(x[n].ks[1][w / 2]) : bf16lo_to_f32(x[n].ks[1][w / 2]);
        s[n][0] = fmaf(s0, d[0], s[n][0]);
        s[n][1] = fmaf(s0, d[1], s[n][1]);
        s[n][2] = fmaf(s1, d[2], s[n][2]);
        s[n][3] = fmaf(s1, d[3], s[n][3]);
      }
    }
  }

  static constexpr int kFinest = 126;  // exponent of the largest factor
  // m starts kMargin above the largest score; the largest product of a head and group has 2^kFine units or more.  A wide
  // margin moves m more rarely and leaves the steps less room: with kMargin 6 and 8, B32 H32/8 L1024..8192 takes 51.7
  // and 51.7 us, queries 4 times as large 55.1 and 54.3, rows' sizes spread as exp(1.5 N(0, 1)) 61.3 and 67.0 (kFine 5,
  // kMargin 6: 67).
  static constexpr int kMargin = 6, kFine = 3;
  // 2^e (0 below fp32's normal range).
  static __device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(e + 127) << 23); }
  static __device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }  // x >= 0
  // Makes room before the weights of N tiles are formed, where a score is above top or a step above vtop.
  template <int N>
  __device__ __forceinline__ void raise(const DwTile<D, true> (&x)[N], const float (&s)[N][4], int g, int t) {
    float y[2] = {-INFINITY, -INFINITY};
    uint32_t mx[NG / 2], over = 0u;
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) mx[w] = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) mx[w] = __vmaxu2(mx[w], __vmaxu2(x[i].vs[0][w], x[i].vs[1][w]));
#pragma unroll
      for (int h = 0; h < 2; ++h) y[h] = fmaxf(y[h], fmaxf(s[i][h], s[i][2 + h]));
    }
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) over |= __vmaxu2(mx[w], vtop[w]) ^ vtop[w];
    if (!__any_sync(0xffffffffu, over != 0u || y[0] > top[0] || y[1] > top[1])) return;

    uint32_t mn[NG / 2];
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) {
      mn[w] = x[0].vs[0][w];
#pragma unroll
      for (int i = 0; i < N; ++i) mn[w] = __vminu2(mn[w], __vminu2(x[i].vs[0][w], x[i].vs[1][w]));
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) y[h] = fmaxf(y[h], __shfl_xor_sync(0xffffffffu, y[h], off));
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) mn[w] = __vminu2(mn[w], __shfl_xor_sync(0xffffffffu, mn[w], off));
    }
    int up[2];
    bool moved[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      moved[h] = y[h] > top[h];
      const float mnew = moved[h] ? fmaxf(m[h], ceilf(y[h] * fx[h]) + kMargin) : m[h];
      up[h] = m[h] == -INFINITY ? 0 : (int)fminf(mnew - m[h], 512.f);  // from nothing: no sums yet
      m[h] = mnew;
      const float q = mnew * rcp_approx(fx[h]);
      top[h] = fmaf(fabsf(q), -0x1p-20f, q);  // below m / fx: no weight is above 1
      l[h] *= pow2(-up[h]);
    }
    if (vtop[0] == 0u) {
      // The first keys.  Every head's largest product is 2^-(kMargin + 1) of the smallest step or more: made 2^kFine
      // units, if that leaves room for weights of 1 at the largest step.
      constexpr uint32_t room = 15 - kFine - kMargin - 1;  // exponents between them
      uint32_t vt[NG / 2];
      over = 0u;
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) {
        vt[w] = (mn[w] & 0x7f807f80u) + ((room << 7) + 0x7fu) * 0x10001u;
        over |= __vmaxu2(mx[w], vt[w]) ^ vt[w];
      }
      if (!__any_sync(0xffffffffu, over != 0u)) {
        __syncwarp();  // all lanes have read the old ones
#pragma unroll
        for (int w = 0; w < NG; ++w) {
          const int field = (int)(((w & 1) ? mn[w / 2] >> 16 : mn[w / 2] & 0xffffu) >> 7);
          const float f = pow2(min(kFine + kMargin + 1 + 127 - field, kFinest)), run = pow2(field - 127 - kMargin - 1);
          if (g == 0) unit[4 * w + t] = make_float4(f, f, run, run);
        }
#pragma unroll
        for (int w = 0; w < NG / 2; ++w) vtop[w] = vt[w];
        __syncwarp();
        return;
      }
    }
    refit(x, s, mx, mn, up, moved, g, t);
  }

  // The units in general.  For each head and group a lower bound of the largest product so far is kept; where the steps'
  // own unit would leave it less than kFine units, the products themselves are looked at.
  template <int N>
  __device__ __forceinline__ void refit(const DwTile<D, true> (&x)[N], const float (&s)[N][4], uint32_t (&mx)[NG / 2],
                                        const uint32_t (&mn)[NG / 2], const int (&up)[2], const bool (&moved)[2], int g,
                                        int t) {
#pragma unroll
    for (int w = 0; w < NG / 2; ++w)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) mx[w] = __vmaxu2(mx[w], __shfl_xor_sync(0xffffffffu, mx[w], off));
    float pr[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[n][i] = ex2_approx(fmaf(s[n][i], fx[i & 1], -m[i & 1]));
    uint32_t finest[NG / 2];  // exponents + 127 of groups 2 w, 2 w + 1, of all heads
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      const float4 old = unit[4 * w + t];
      const int field = (int)(((w & 1) ? mx[w / 2] >> 16 : mx[w / 2] & 0xffffu) >> 7);
      const int least = (int)(((w & 1) ? mn[w / 2] >> 16 : mn[w / 2] & 0xffffu) >> 7);
      const int own = 14 + 127 - field;
      int e[2] = {exponent(old.x) + up[0], exponent(old.y) + up[1]};
      float run[2] = {old.z * pow2(-up[0]), old.w * pow2(-up[1])};
      bool look = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (moved[h]) run[h] = fmaxf(run[h], pow2(least - 127 - kMargin - 1));
        look |= own < min(e[h], kFinest) && kFine - exponent(run[h]) > own;
      }
      if (__any_sync(0xffffffffu, look)) {
        float most[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t st = x[n].vs[i / 2][w / 2];
            most[i & 1] = fmaxf(most[i & 1], pr[n][i] * ((w & 1) ? bf16hi_to_f32(st) : bf16lo_to_f32(st)));
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) most[h] = fmaxf(most[h], __shfl_xor_sync(0xffffffffu, most[h], off));
          run[h] = fmaxf(run[h], most[h]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int to = min(min(e[h], kFinest), max(own, kFine - exponent(run[h])));
        const float c = pow2(to - e[h]);  // (old sums shrink by 2^up, and count 2^up as many of the units that shrank so)
        e[h] = to;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          acc[w][b][h] *= c;
          acc[w][b][2 + h] *= c;
        }
      }
      __syncwarp();  // all lanes have read the old ones
      if (g == 0) unit[4 * w + t] = make_float4(pow2(e[0]), pow2(e[1]), run[0], run[1]);
      const uint32_t ex = (uint32_t)(max(e[0], e[1]) + 127);
      finest[w / 2] = (w & 1) ? finest[w / 2] | ex << 16 : ex;
    }
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) {
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) finest[w] = __vmaxu2(finest[w], __shfl_xor_sync(0xffffffffu, finest[w], off));
      // The largest bf16 below 2^16 units, at most that of exponent 127 (NaN: such steps come here always).
      vtop[w] = (__vminu2(0x010d010du - finest[w], 0x00fe00feu) << 7) | 0x007f007fu;
    }
    __syncwarp();
  }

  __device__ __forceinline__ void accumulate(const DwTile<D, true>& x, const float (&s)[4], int t) {
    float pr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pr[i] = ex2_approx(fmaf(s[i], fx[i & 1], -m[i & 1]));
    l[0] += pr[0] + pr[2];
    l[1] += pr[1] + pr[3];
    auto lo4 = [](uint32_t c) { return f16x2_sub(and_or(c, 0x000f000fu, 0x64006400u), 0x64086408u); };  // code - 8
    auto hi4 = [](uint32_t c) { return f16x2_sub(and_or(c, 0x00f000f0u, 0x64006400u), 0x64806480u); };  // 16 (code - 8)
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      const float s0 = (w & 1) ? bf16hi_to_f32(x.vs[0][w / 2]) : bf16lo_to_f32(x.vs[0][w / 2]);
      const float s1 = (w & 1) ? bf16hi_to_f32(x.vs[1][w / 2]) : bf16lo_to_f32(x.vs[1][w / 2]);
      // The unit first: at most 2^126, and a weight of 0 stays one whatever the step.
      const float2 f = *reinterpret_cast<const float2*>(unit + 4 * w + t);
      const float2 p0 = fmul2(make_float2(pr[0], pr[1]), f), p1 = fmul2(make_float2(pr[2], pr[3]), f);
      const uint32_t b0 = movmatrix_trans(pack_f16x2(p0.x * s0, p0.y * s0));
      const uint32_t b1 = movmatrix_trans(pack_f16x2(p1.x * s1, p1.y * s1));
      const uint32_t sel = (w & 1) ? 0x7632u : 0x5410u;
      const uint32_t lo = __byte_perm(x.v[0][w / 2], x.v[1][w / 2], sel);
      const uint32_t hi = __byte_perm(x.v[2][w / 2], x.v[3][w / 2], sel);
      const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
      mma_f16_16816(acc[w][0], lo4(lo), hi4(lo), lo4(hi), hi4(hi), b0, b1);
      mma_f16_16816(acc[w][1], lo4(lo8), hi4(lo8), lo4(hi8), hi4(hi8), b0, b1);
    }
  }

  // O = O~ / l of this lane's channels (l summed over the keys; 0 without a key): put(channel, head column, value).
  template <typename Put>
  __device__ __forceinline__ void finish(int g, int t, Put put) {
    const float inv[2] = {l[0] == 0.f ? 0.f : rcp_approx(l[0]), l[1] == 0.f ? 0.f : rcp_approx(l[1])};
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      const float2 f = *reinterpret_cast<const float2*>(unit + 4 * w + t);
      const float back[2] = {pow2(-exponent(f.x)), pow2(-exponent(f.y))};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int ch = kKv4Group * w + 4 * g + 2 * b;
          put(ch, 2 * t + h, acc[w][b][h] * inv[h] * back[h]);
          put(ch + 1, 2 * t + h, acc[w][b][2 + h] * 0.0625f * inv[h] * back[h]);
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
      if (live) load_words<4>(qf[c], q + 8 * (4 * c + t));
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

  __device__ __forceinline__ void scores(const DwTile<D, false>& x, float (&s)[4]) {
    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of dependent products
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      mma_bf16_16816(a, x.k[0][c][0], x.k[1][c][0], x.k[0][c][1], x.k[1][c][1], qf[c][0], qf[c][1]);
      mma_bf16_16816(b, x.k[0][c][2], x.k[1][c][2], x.k[0][c][3], x.k[1][c][3], qf[c][2], qf[c][3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = (a[i] + b[i]) * fx;
  }

  template <int N>
  __device__ __forceinline__ void raise(const DwTile<D, false> (&)[N], const float (&s)[N][4]) {
    float y[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) y[h] = fmaxf(y[h], fmaxf(s[i][h], s[i][2 + h]));
    if (__any_sync(0xffffffffu, y[0] > m[0] + 8.f || y[1] > m[1] + 8.f)) {
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
  }

  __device__ __forceinline__ void accumulate(const DwTile<D, false>& x, const float (&s)[4]) {
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

// Where the warps' states meet at the end of a part of a unit.
template <int D>
struct DwMeet {
  float o[kDwWarps][kDwHeads][D + 4];
  float ml[kDwWarps][kDwHeads][2];

  // The warp's state; l still spread over the lanes' keys.
  template <typename State>
  __device__ __forceinline__ void put(State& st, int warp, int g, int t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) st.l[h] += __shfl_xor_sync(0xffffffffu, st.l[h], off);
    st.finish(g, t, [&](int ch, int head, float val) { o[warp][head][ch] = val; });
    if (g == 0)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ml[warp][2 * t + h][0] = st.m[h];
        ml[warp][2 * t + h][1] = st.l[h];
      }
  }
  // After a barrier: the CTA's result for heads head0 ..., the outputs themselves if this part was the whole unit (done),
  // else the partials row(h).  MEANS: the warps have put O, else O~, and the partials are in the same form.
  template <bool MEANS, typename Row>
  __device__ __forceinline__ void write(const DecWinParams& p, size_t head0, int nh, bool done, Row row) {
    for (int idx = threadIdx.x; idx < nh * D; idx += 32 * kDwWarps) {
      const int h = idx / D, ch = idx % D;
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDwWarps; ++w) mt = fmaxf(mt, ml[w][h][0]);
      float v = 0.f, l = 0.f;
      if constexpr (MEANS) {  // shares of at most 1 in all, so that no sum outgrows O
        float f[kDwWarps];
#pragma unroll
        for (int w = 0; w < kDwWarps; ++w) {
          const float lw = ml[w][h][1];
          f[w] = lw != 0.f ? ex2_approx(ml[w][h][0] - mt) * lw : 0.f;  // 0: no key (a NaN sum goes on as one)
          l += f[w];
        }
        const float inv = rcp_approx(l);
#pragma unroll
        for (int w = 0; w < kDwWarps; ++w) v = fmaf(f[w] * inv, o[w][h][ch], v);
      } else {
#pragma unroll
        for (int w = 0; w < kDwWarps; ++w) {
          const float lw = ml[w][h][1];
          if (lw != 0.f) {  // as above
            const float f = ex2_approx(ml[w][h][0] - mt);
            v = fmaf(f, o[w][h][ch], v);
            l = fmaf(f, lw, l);
          }
        }
      }
      if (done) {
        p.o[(head0 + h) * D + ch] = __float2bfloat16(MEANS ? v : v / l);
        if (ch == 0 && p.lse) p.lse[head0 + h] = (mt + log2f(l)) * 0.6931471805599453f;
      } else {
        const size_t part = row(h);
        p.part_o[part * D + ch] = v;
        if (ch == 0) {
          p.part_ml[2 * part] = l != l ? 0.f : mt;
          p.part_ml[2 * part + 1] = l;
        }
      }
    }
  }
};

// Merges `parts` > 1 partials, rows row(0 ...), of one (batch, head) by a CTA of NW warps: each takes every
// NW-th partial, a lane D / 32 channels.  NW = 16 where a unit may have more than 16 partials (those of a long sequence
// then come in one or two rounds of loads), else 4 (a batch's merges then run in one wave; with 16 warps that of
// B32 H32 took 11 us more).  MEANS: the partials are O, else O~.
template <int D, int NW, bool MEANS, typename Row>
__device__ __forceinline__ void dw_merge(const DecWinParams& p, int parts, Row row) {
  constexpr int PER = D / 32;
  __shared__ float sm_o[NW][D], sm_ml[NW][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  // A warp's partials warp + NW i, 32 of them a round: their (m, l) one to a lane, then their rows.
  for (int c = warp; c < parts; c += 32 * NW) {
    const int n = min(32, (parts - 1 - c) / NW + 1);
    const float2 x = lane < n ? ml[row(c + NW * lane)] : make_float2(-INFINITY, 0.f);
    float mx = x.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    mx = fmaxf(m, mx);
    float f = ex2_approx(m - mx);  // 0 at first
    m = mx;
    l *= f;
    float w = ex2_approx(x.x - m);
    if constexpr (MEANS) {  // l is the warp's, acc the mean so far
      w *= x.y;
      float sum = w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      sum += l;
      const float inv = rcp_approx(sum);
      f = l * inv;
      w *= inv;
      l = sum;
    } else {
      l = fmaf(w, x.y, l);  // this lane's part
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= f;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* src = p.part_o + row(c + NW * i) * D + lane * PER;
      if constexpr (PER == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(wi, v.x, acc[0]);
        acc[1] = fmaf(wi, v.y, acc[1]);
        acc[2] = fmaf(wi, v.z, acc[2]);
        acc[3] = fmaf(wi, v.w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(wi, v.x, acc[0]);
        acc[1] = fmaf(wi, v.y, acc[1]);
      }
    }
  }
  if constexpr (!MEANS) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) sm_o[warp][lane * PER + e] = acc[e];
  if (lane == 0) {
    sm_ml[warp][0] = m;
    sm_ml[warp][1] = l;
  }
  __syncthreads();
  if (threadIdx.x >= D) return;
  float mt = -INFINITY, os = 0.f, ls = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) mt = fmaxf(mt, sm_ml[w][0]);
  if constexpr (MEANS) {
#pragma unroll
    for (int w = 0; w < NW; ++w) ls = fmaf(ex2_approx(sm_ml[w][0] - mt), sm_ml[w][1], ls);
    const float inv = rcp_approx(ls);
#pragma unroll
    for (int w = 0; w < NW; ++w)
      os = fmaf(ex2_approx(sm_ml[w][0] - mt) * sm_ml[w][1] * inv, sm_o[w][threadIdx.x], os);
  } else {
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ex2_approx(sm_ml[w][0] - mt);
      os = fmaf(f, sm_o[w][threadIdx.x], os);
      ls = fmaf(f, sm_ml[w][1], ls);
    }
    os /= ls;
  }
  p.o[(size_t)blockIdx.x * D + threadIdx.x] = __float2bfloat16(os);
  if (p.lse && threadIdx.x == 0) p.lse[blockIdx.x] = (mt + log2f(ls)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------------------------
// bf16 cache: one part of one unit per CTA.
// ---------------------------------------------------------------------------------------------
// Keys per part: an equal S-th of the unit's in whole steps, or the smallest part.
__device__ __forceinline__ int dw_chunk(const DecWinParams& p, int n) {
  constexpr int STEP = DwTile<128, false>::STEP;
  const int even = (int)(((unsigned)n + p.S - 1) / p.S);
  return max(p.min_chunk, (even + STEP - 1) / STEP * STEP);
}

template <int D>
__global__ void __launch_bounds__(32 * kDwWarps, (DwTile<D, false>::CTAS)) fa_decode_window_kernel(const DecWinParams p) {
  using Tile = DwTile<D, false>;
  constexpr int STEP = Tile::STEP;
  __shared__ DwMeet<D> meet;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int s_idx = blockIdx.x % p.S;
  int unit = blockIdx.x / p.S;
  const int hb = unit % p.hblocks;
  unit /= p.hblocks;  // b * Hkv + key/value head
  const int h0 = hb * kDwHeads, nh = min(kDwHeads, p.group - h0);
  const size_t head0 = (size_t)unit * p.group + h0;  // b * H + first query head
  const DwKeys keys = dw_keys(p, unit / p.Hkv);
  const int chunk = dw_chunk(p, keys.n);
  const long long begin = (long long)chunk * s_idx;
  if (begin >= keys.n) {  // nothing of this sequence is left (n = 0: the first part's CTA writes the outputs)
    if (s_idx == 0)
      for (int idx = threadIdx.x; idx < nh * D; idx += 32 * kDwWarps) {
        p.o[head0 * D + idx] = __float2bfloat16(0.f);
        if (p.lse && idx < nh) p.lse[head0 + idx] = -INFINITY;
      }
    grid_launch_next();
    return;
  }
  const int i0 = (int)begin, i1 = min(i0 + chunk, keys.n), ns = keys.ns, jump = keys.jump;

  typename Tile::Base base;
  base.set(p, (size_t)unit * p.Lmax, g, t);
  // The warp's tile of the step at list entry i.  A whole step on one side of the jump is consecutive cache rows
  // (the test is the same for all warps); elsewhere each row is found by itself, entries past the end repeating the
  // last one (a key the query sees; their weights are 0).
  const int w0 = warp * kDwTile;
  auto whole = [&](int i) { return i + STEP <= i1 && (i >= ns || i + STEP <= ns); };
  auto row0 = [&](int i) -> uint32_t { return i + w0 + (i >= ns ? jump : 0); };
  auto row_of = [&](int i) {
    return [=](int r) -> int {
      const int e = min(i + w0 + r, i1 - 1);
      return e + (e >= ns ? jump : 0);
    };
  };
  Tile x[1];
  auto load_k = [&](int i) {
    if (whole(i)) x[0].load_k(base, row0(i), g, t, DwRows());
    else x[0].load_k(base, 0, g, t, row_of(i));
  };
  auto load_v = [&](int i) {
    if (whole(i)) x[0].load_v(base, row0(i), g, t, DwRows());
    else x[0].load_v(base, 0, g, t, row_of(i));
  };
  load_k(i0);
  load_v(i0);
  DwState<D, false> st;
  st.init(p, p.q + (head0 + min(g, nh - 1)) * D, g < nh, g, t);
  // K of the next step is on its way from the moment this one's scores are done, V from this one's products on.
#pragma unroll 1
  for (int i = i0; i < i1; i += STEP) {
    float s[1][4];
    st.scores(x[0], s[0]);
    const bool more = i + STEP < i1;
    if (more) load_k(i + STEP);
    if (i + STEP > i1) {  // scores past the list's end do not count
      const int e = i + w0 + g;
      if (e >= i1) s[0][0] = s[0][1] = -INFINITY;
      if (e + 8 >= i1) s[0][2] = s[0][3] = -INFINITY;
      if (i + w0 >= i1) break;  // the warp's tile lies past it altogether
    }
    st.raise(x, s);
    st.accumulate(x[0], s[0]);
    if (more) load_v(i + STEP);
  }
  // The merge may be launched: it waits for this grid's end before it reads.
  grid_launch_next();
  meet.put(st, warp, g, t);
  __syncthreads();
  meet.template write<false>(p, head0, nh, keys.n <= chunk, [&](int h) { return (head0 + h) * p.S + s_idx; });
}

// One (batch, head) per CTA; launched while the partials' kernel still runs, it waits for that kernel's end.  A head of
// one part, or without any key, is left alone.
template <int D, int NW>
__global__ void __launch_bounds__(32 * NW) fa_decode_window_merge_kernel(const DecWinParams p) {
  const int n = dw_keys(p, blockIdx.x / p.H).n, chunk = dw_chunk(p, n);
  grid_wait_prior();  // by every CTA: this grid ends after the partials' does
  const int parts = (n + chunk - 1) / chunk;
  if (parts > 1) dw_merge<D, NW, false>(p, parts, [&](int c) { return (size_t)blockIdx.x * p.S + c; });
}

// ---------------------------------------------------------------------------------------------
// 4-bit cache: equal shares of the list of all units' steps.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ int dw4_steps(int n) {
  constexpr int STEP = DwTile<128, true>::STEP;
  return (n + STEP - 1) / STEP;
}
// Steps per CTA when `total` steps (of all units; below 2^31, checked by the host) are shared out.
__device__ __forceinline__ int dw4_share(const DecWinParams& p, int total) {
  return max(1, (int)(((long long)total + p.grid - 1) / p.grid));
}

// A place in the list of steps.
struct Dw4Place {
  int b, in_seq, step, steps;  // sequence, its unit (key/value head, head block), the unit's step and steps
  DwKeys keys;

  __device__ __forceinline__ void set_seq(const DecWinParams& p, int seq) {
    b = seq;
    keys = dw_keys(p, b);
    steps = dw4_steps(keys.n);
  }
  // To the next unit that has a step (there is one).
  __device__ __forceinline__ void next_unit(const DecWinParams& p) {
    step = 0;
    if (++in_seq == p.Hkv * p.hblocks) {
      in_seq = 0;
      do set_seq(p, b + 1);
      while (steps == 0);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(32 * kDwWarps, (DwTile<D, true>::CTAS)) fa_decode_kv4_kernel(const DecWinParams p) {
  using Tile = DwTile<D, true>;
  using State = DwState<D, true>;
  constexpr int NT = Tile::NT, STEP = Tile::STEP;
  __shared__ DwMeet<D> meet;
  __shared__ __align__(16) uint8_t sm_q[State::Q_BYTES];
  __shared__ float4 sm_unit[kDwWarps][4 * State::NG];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int per_seq = p.Hkv * p.hblocks;  // units of a sequence

  // This CTA's share [begin, end) of the list of steps, and the place where it begins.
  int mine = lane < p.B ? dw4_steps(dw_keys(p, lane).n) : 0;
  int sum = mine;
  for (int i = lane + 32; i < p.B; i += 32) sum += dw4_steps(dw_keys(p, i).n);
  const int total = __reduce_add_sync(0xffffffffu, sum) * per_seq;
  const int share = dw4_share(p, total);
  const int begin = (int)min((long long)share * blockIdx.x, (long long)total);
  const int end = (int)min((long long)begin + share, (long long)total);
  if (begin < end) {
    Dw4Place at;
    int first = 0;  // steps before the sequence
    for (int base = 0;; base += 32) {
      if (base > 0) mine = base + lane < p.B ? dw4_steps(dw_keys(p, base + lane).n) : 0;
      int incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, first + incl * per_seq > begin);
      if (past) {  // at the last 32 sequences at the latest: begin < total
        const int l = __ffs(past) - 1;
        at.set_seq(p, base + l);
        first += __shfl_sync(0xffffffffu, incl - mine, l) * per_seq;
        break;
      }
      first += __shfl_sync(0xffffffffu, incl, 31) * per_seq;
    }
    at.in_seq = (begin - first) / at.steps;
    at.step = begin - first - at.in_seq * at.steps;

    // The loads run a step ahead of the work, across the ends of units.  A step's tile rows as in the bf16 kernel.
    Dw4Place ahead = at;
    int to_load = end - begin;
    typename Tile::Base base;
    auto set_base = [&]() { base.set(p, (size_t)(ahead.b * p.Hkv + ahead.in_seq / p.hblocks) * p.Lmax, g, t); };
    set_base();
    const int w0 = warp * (kDwTile * NT);
    Tile x[NT];
    auto whole = [&]() {
      const int i = ahead.step * STEP;
      return i + STEP <= ahead.keys.n && (i >= ahead.keys.ns || i + STEP <= ahead.keys.ns);
    };
    auto row0 = [&]() -> uint32_t {
      const int i = ahead.step * STEP;
      return i + w0 + (i >= ahead.keys.ns ? ahead.keys.jump : 0);
    };
    auto row_of = [&](int r) -> int {
      const int e = min(ahead.step * STEP + w0 + r, ahead.keys.n - 1);
      return e + (e >= ahead.keys.ns ? ahead.keys.jump : 0);
    };
    auto load_k = [&]() {
      if (to_load <= 0) return;
      if (whole()) {
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n].load_k(base, row0(), n, g, t, DwRows());
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n].load_k(base, 0, 0, g, t, [&](int r) { return row_of(kDwTile * n + r); });
      }
    };
    auto load_v = [&]() {  // and on to the next step
      if (to_load <= 0) return;
      if (whole()) {
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n].load_v(base, row0(), n, g, t, DwRows());
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n].load_v(base, 0, 0, g, t, [&](int r) { return row_of(kDwTile * n + r); });
      }
      if (--to_load > 0 && ++ahead.step == ahead.steps) {
        ahead.next_unit(p);
        set_base();
      }
    };
    load_k();
    load_v();
    State st;
    int seg0 = begin;  // first step of the segment (this CTA's part of a unit)
#pragma unroll 1
    for (int j = begin; j < end; ++j) {
      if (j == seg0) {
        if (warp == 0) {
          const int h0 = at.in_seq % p.hblocks * kDwHeads, nh = min(kDwHeads, p.group - h0);
          const size_t head0 = (size_t)(at.b * p.Hkv + at.in_seq / p.hblocks) * p.group + h0;
          State::prepare(p, p.q + (head0 + min(g, nh - 1)) * D, g < nh, g, t, sm_q);
        }
        __syncthreads();  // also: the last segment's states have been read
        st.start(sm_q, sm_unit[warp], lane);
      }
      float s[NT][4];
      st.scores(x, sm_q, lane, s);
      load_k();
      const int i = at.step * STEP;
      bool some = true;
      if (i + STEP > at.keys.n) {  // scores past the list's end do not count
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int e = i + w0 + kDwTile * n + g;
          if (e >= at.keys.n) s[n][0] = s[n][1] = -INFINITY;
          if (e + 8 >= at.keys.n) s[n][2] = s[n][3] = -INFINITY;
        }
        some = i + w0 < at.keys.n;
      }
      if (some) {
        st.raise(x, s, g, t);
#pragma unroll
        for (int n = 0; n < NT; ++n) st.accumulate(x[n], s[n], t);
      }
      load_v();
      ++at.step;
      if (at.step < at.steps && j + 1 < end) continue;

      const int h0 = at.in_seq % p.hblocks * kDwHeads, nh = min(kDwHeads, p.group - h0);
      const size_t head0 = (size_t)(at.b * p.Hkv + at.in_seq / p.hblocks) * p.group + h0;  // b * H + first query head
      meet.put(st, warp, g, t);
      __syncthreads();
      const size_t part = (2 * (size_t)blockIdx.x + (seg0 == begin ? 0 : 1)) * kDwHeads;
      meet.template write<true>(p, head0, nh, j + 1 - seg0 == at.steps, [&](int h) { return part + h; });
      seg0 = j + 1;
      if (j + 1 < end) at.next_unit(p);
    }
  }
  // The merge may be launched: it waits for this grid's end before it reads.
  grid_launch_next();
}

// As fa_decode_window_merge_kernel; a head without any key gets O = 0 and LSE = -inf here.
template <int D, int NW>
__global__ void __launch_bounds__(32 * NW) fa_decode_kv4_merge_kernel(const DecWinParams p) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.H, head = blockIdx.x % p.H;
  const int per_seq = p.Hkv * p.hblocks;
  int all = 0, before = 0;  // steps of all sequences, of those before b
  for (int i = lane; i < p.B; i += 32) {
    const int s = dw4_steps(dw_keys(p, i).n);
    all += s;
    before += i < b ? s : 0;
  }
  const int steps = dw4_steps(dw_keys(p, b).n);
  const int share = dw4_share(p, __reduce_add_sync(0xffffffffu, all) * per_seq);
  const int in_group = head % p.group;
  const int unit0 = __reduce_add_sync(0xffffffffu, before) * per_seq +
                    (head / p.group * p.hblocks + in_group / kDwHeads) * steps;
  grid_wait_prior();  // by every CTA: this grid ends after the partials' does
  if (steps == 0) {
    if (threadIdx.x < D) p.o[(size_t)blockIdx.x * D + threadIdx.x] = __float2bfloat16(0.f);
    if (threadIdx.x == 0 && p.lse) p.lse[blockIdx.x] = -INFINITY;
    return;
  }
  const int c0 = unit0 / share, parts = (unit0 + steps - 1) / share - c0 + 1;
  // The partial of share c0 + i is in its first slot if the share begins inside the unit, else in its last.
  if (parts > 1)
    dw_merge<D, NW, true>(p, parts, [&](int i) -> size_t {
      return (2 * (size_t)(c0 + i) + ((long long)(c0 + i) * share < unit0 ? 1 : 0)) * kDwHeads + in_group % kDwHeads;
    });
}

}  // namespace fa
