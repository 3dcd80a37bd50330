// Microscaled 4-bit quantisation (MXFP4) and its read-back.
//
// A block of 32 elements along the product's contraction axis shares a power
// of two: with amax = m 2^e, 1 <= m < 2, the scale is 2^(e - 2 + [m > 1.5]),
// at least 2^-127, the smallest one with amax / scale <= 6. Six is e2m1's
// largest value, so nothing saturates, which stochastic rounding needs to be
// unbiased. Elements go to the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} (ties to
// the even code), or up or down at random in proportion to the distance. A
// block that holds an infinity or a NaN gets the scale 0xff (NaN).
//
// quantize: persistent blocks take 128 x 128 tiles, read each once (cp.async,
// the next tiles in flight while one is coded) and write both orientations
// from shared memory, each with its whole 512-byte scale tile. A thread codes
// whole blocks, along a row or down a column. Dropout is applied in the row
// pass, which writes the masked values back for the column pass; the blend of the
// parameters with their average is formed while the tile is filled.
//
// Bound by instructions, at 58-66 % of the issue slots: 16384 x 2560 bf16 to both
// orientations 24 us (its bytes 20), with dropout 47, stochastic 90; fp32 38 (33)
// and 101. The blend of 768 x 50304 runs at the memory's rate, 44 us.
#include "dtype_io.cuh"
#include "lowbit.cuh"
#include "philox.cuh"

namespace muon {

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Scale byte of a block and the factor that brings its values to e2m1's
// range (an exact power of two; 0 for a block that stands for NaN).
__device__ __forceinline__ uint32_t block_scale(float amax, float& inv) {
  const uint32_t b = __float_as_uint(amax) & 0x7FFFFFFFu;
  if (b >= 0x7F800000u) {
    inv = 0.0f;
    return 255u;
  }
  const int e = static_cast<int>(b >> 23) - 2 + ((b & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  const uint32_t byte = e > 0 ? static_cast<uint32_t>(e) : 0u;
  inv = __uint_as_float((254u - byte) << 23);
  return byte;
}

// The codes of eight values already in e2m1's range, the first in the low bits.
__device__ __forceinline__ uint32_t pack8_e2m1(const float (&y)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}

// Stochastic codes of eight values with |y| <= 6: between the neighbours of
// |y|, up when the 16-bit number u plus one half is below the fraction times
// 2^16. With E = max(0, exponent of y), the gap is 2^(E - 1), the code of the
// lower neighbour floor(|y| 2^(1 - E)) + 2 E, and the one wanted
// ceil((|y| 2^(17 - E) - (u + 1/2)) 2^-16) + 2 E. The difference has the exact
// sign, and is exact where it is near a multiple of 2^16 (a multiple of 2^-7
// below 2^18), so the ceiling, taken by adding 1.5 * 2^23 with rounding
// upwards, is that of the exact value.
__device__ __forceinline__ uint32_t pack8_stochastic(const float (&y)[8], const uint4& u) {
  const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u16 = (j & 1) ? uu[j >> 1] >> 16 : uu[j >> 1] & 0xFFFFu;
    const float half_up = __uint_as_float(0x4B000000u | u16) - 8388607.5f;        // u16 + 1/2
    const uint32_t e = __float_as_uint(fmaxf(fabsf(y[j]), 1.0f)) & 0x7F800000u;
    const float k = __uint_as_float(0x48000000u + 0x3F800000u - e);               // 2^(17 - E)
    const float d = fmaf(fabsf(y[j]), k, -half_up);
    const uint32_t c = __float_as_uint(__fmaf_ru(d, 1.0f / 65536.0f, 12582912.0f));
    // 1.5 * 2^23 has the bits 0x4B400000, E is (e >> 23) - 127
    const uint32_t code = c + (e >> 22) - (0x4B400000u + 254u) + ((__float_as_uint(y[j]) >> 28) & 8u);
    w |= code << (4 * j);
  }
  return w;
}

// Per half, the larger magnitude (NaN if either is); its sign means nothing.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Both halves of w as fp32, times those of f (exact where f's are powers of
// two; adding -0 keeps the sign of a zero). One instruction each, and not on
// the pipe that the conversions and maxima keep busy.
__device__ __forceinline__ float2 mul_bf16x2_f32(uint32_t w, uint32_t f) {
  float2 r;
  asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %2;\n\tmov.b32 {c, d}, %3;\n\t"
      "fma.rn.f32.bf16 %0, a, c, 0f80000000;\n\tfma.rn.f32.bf16 %1, b, d, 0f80000000;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(w), "r"(f));
  return r;
}

// A power of two (or 0) as bf16, its upper half word.
__device__ __forceinline__ uint32_t bf16_bits(float pow2) { return __float_as_uint(pow2) >> 16; }

enum QuantSrc : int { kSrcBf16 = 0, kSrcF32 = 1, kSrcBlendBf16 = 2, kSrcBlendF32 = 3 };

// How a source is staged: threads per block, tiles in flight per block, blocks
// per SM (the tile is kept as bf16 for a bf16 source, else as fp32).
template <int kSrc>
struct QuantConfig {
  static constexpr bool kBf16 = kSrc == kSrcBf16 || kSrc == kSrcBlendBf16;
  static constexpr bool kBlend = kSrc >= kSrcBlendBf16;
  static constexpr bool kHalf = kSrc == kSrcBf16;
  static constexpr int kThreads = kHalf ? 256 : 512;
  static constexpr int kStages = kBlend ? 1 : kHalf ? 2 : 3;
  static constexpr int kBlocks = kBlend ? 2 : kHalf ? 3 : 1;
  static constexpr int kRowBytes = kMxTile * (kHalf ? 2 : 4);
  static constexpr int kTileBytes = kMxTile * kRowBytes;
  static constexpr int blocks(bool stoch) { return kHalf && stoch ? 2 : kBlocks; }   // registers
  static constexpr int kSmem = kStages * kTileBytes + 4 * kMxTileBytes;
};

__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool exists) {
  const int n = exists ? 16 : 0;   // the rest of the 16 bytes is zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}

// Position (in 16-byte groups of the row) of 16-byte group g of a tile row: a
// warp of the column pass reads 32 (bf16: 2 per word) values of 8 neighbouring
// words in four row blocks, which this spreads over all 32 banks.
__device__ __forceinline__ int swizzled_group(int row, int g) { return g ^ ((row >> 5) * 2); }

struct QuantTile {
  int mat, r0, c0;
  long long at;     // scale tile of `q` (row tile, column tile); at_t: of `qt`
  long long at_t;
};

__device__ __forceinline__ QuantTile quant_tile(const QuantParams& p, int t) {
  const int per_mat = p.tiles_r * p.tiles_c;
  QuantTile x;
  x.mat = fdiv(t, p.fd_tiles);
  const int u = t - x.mat * per_mat;
  const int tr = fdiv(u, p.fd_tiles_c), tc = u - tr * p.tiles_c;
  x.r0 = tr * kMxTile;
  x.c0 = tc * kMxTile;
  x.at = t;
  x.at_t = static_cast<long long>(x.mat) * per_mat + static_cast<long long>(tc) * p.tiles_r + tr;
  return x;
}

__device__ __forceinline__ void copy4_async(void* dst, const void* src, bool exists) {
  const int n = exists ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}

// Byte offset of element `col` in a tile row.
template <bool kHalf>
__device__ __forceinline__ int tile_offset(int lr, int col) {
  constexpr int kPer = kHalf ? 8 : 4, kElt = kHalf ? 2 : 4;
  return 16 * swizzled_group(lr, col / kPer) + (col % kPer) * kElt;
}

// Copies a tile to shared memory; what lies outside the matrix becomes zero.
// Asynchronously in 16-byte pieces where rows start on 16-byte boundaries, in
// 4-byte pieces where they start on 4-byte boundaries, else (bf16, odd length)
// through registers. The blend is formed here, with readout_blend's roundings.
template <int kSrc>
__device__ __forceinline__ void fill_tile(const QuantParams& p, uint8_t* tile, const QuantTile& T) {
  using C = QuantConfig<kSrc>;
  constexpr int kElt = C::kBf16 ? 2 : 4;
  const int tid = threadIdx.x;
  const long long first = (static_cast<long long>(T.mat) * p.rows + T.r0) * p.cols + T.c0;
  const int rows = p.rows - T.r0, cols = p.cols - T.c0;   // from the tile's corner on
  if constexpr (!C::kBlend) {
    const uint8_t* src = static_cast<const uint8_t*>(p.x) + first * kElt;
    if (p.cols % 8 == 0) {
      constexpr int kPer = 16 / kElt, kGroups = kMxTile / kPer, kStep = C::kThreads / kGroups;
      const int g = tid % kGroups, r = tid / kGroups;
      const bool in = g * kPer < cols;
      const uint8_t* at = src + (static_cast<long long>(r) * p.cols + g * kPer) * kElt;
      const long long step = static_cast<long long>(kStep) * p.cols * kElt;
#pragma unroll
      for (int i = 0; i < kMxTile / kStep; ++i) {
        const int lr = r + i * kStep;
        const bool exists = in && lr < rows;
        copy16_async(tile + lr * C::kRowBytes + 16 * swizzled_group(lr, g), exists ? at : p.x, exists);
        at += step;
      }
      return;
    }
    constexpr int kPer = 4 / kElt;
    if (p.cols % kPer == 0) {
      constexpr int kWords = kMxTile / kPer, kStep = C::kThreads / kWords;
      const int c = tid % kWords * kPer, r = tid / kWords;
      const bool in = c < cols;
      const uint8_t* at = src + (static_cast<long long>(r) * p.cols + c) * kElt;
      const long long step = static_cast<long long>(kStep) * p.cols * kElt;
#pragma unroll 8
      for (int i = 0; i < kMxTile / kStep; ++i) {
        const int lr = r + i * kStep;
        const bool exists = in && lr < rows;
        copy4_async(tile + lr * C::kRowBytes + tile_offset<C::kHalf>(lr, c), exists ? at : p.x, exists);
        at += step;
      }
      return;
    }
  } else if (p.cols % 8 == 0) {   // four averages and four parameters at a time
    constexpr int kGroups = kMxTile / 4, kStep = C::kThreads / kGroups;
    const int g = tid % kGroups, r = tid / kGroups;
    const bool in = g * 4 < cols;
    constexpr int kEach = kMxTile / kStep;
    float4 m[kEach];
    uint4 th[kEach];   // four parameters: fp32, or bf16 in x and y
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int lr = r + i * kStep;
      const long long e = first + static_cast<long long>(lr) * p.cols + g * 4;
      m[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      th[i] = make_uint4(0u, 0u, 0u, 0u);
      if (in && lr < rows) {
        m[i] = *reinterpret_cast<const float4*>(p.ema + e);
        if (C::kBf16) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.x) + e);
          th[i].x = w.x;
          th[i].y = w.y;
        } else {
          th[i] = *reinterpret_cast<const uint4*>(static_cast<const float*>(p.x) + e);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int lr = r + i * kStep;
      const float4 t = C::kBf16 ? make_float4(bf16_lo_f(th[i].x), bf16_hi_f(th[i].x), bf16_lo_f(th[i].y),
                                              bf16_hi_f(th[i].y))
                                : make_float4(__uint_as_float(th[i].x), __uint_as_float(th[i].y),
                                              __uint_as_float(th[i].z), __uint_as_float(th[i].w));
      float4 v;
      v.x = fmaf(p.w_final, t.x, __fmul_rn(p.w_ema, m[i].x));
      v.y = fmaf(p.w_final, t.y, __fmul_rn(p.w_ema, m[i].y));
      v.z = fmaf(p.w_final, t.z, __fmul_rn(p.w_ema, m[i].z));
      v.w = fmaf(p.w_final, t.w, __fmul_rn(p.w_ema, m[i].w));
      *reinterpret_cast<float4*>(tile + lr * C::kRowBytes + 16 * swizzled_group(lr, g)) = v;
    }
    return;
  }
  constexpr int kStep = C::kThreads / kMxTile;
  const int c = tid % kMxTile, r = tid / kMxTile;
#pragma unroll 8
  for (int i = 0; i < kMxTile / kStep; ++i) {
    const int lr = r + i * kStep;
    const long long e = first + static_cast<long long>(lr) * p.cols + c;
    float v = 0.0f;
    if (c < cols && lr < rows) {
      v = load1t<C::kBf16>(p.x, e);
      if constexpr (C::kBlend) v = fmaf(p.w_final, v, __fmul_rn(p.w_ema, p.ema[e]));
    }
    uint8_t* at = tile + lr * C::kRowBytes + tile_offset<C::kHalf>(lr, c);
    if constexpr (C::kHalf)
      *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(v);   // exact: v is a bf16 value
    else
      *reinterpret_cast<float*>(at) = v;
  }
}

// Largest magnitude of 32 fp32 values (NaN if any is).
__device__ __forceinline__ float amax32(const uint32_t (&w)[32]) {
  float m[2] = {fabsf(__uint_as_float(w[0])), fabsf(__uint_as_float(w[1]))};
#pragma unroll
  for (int i = 2; i < 32; i += 2)
    m[(i >> 1) & 1] = max_nan(m[(i >> 1) & 1], fabsf(__uint_as_float(w[i])), fabsf(__uint_as_float(w[i + 1])));
  return max_nan(m[0], m[1]);
}

// Rows: a thread codes one block of 32 columns. It reads the block's four
// groups of 8 elements in an order that differs between neighbouring lanes
// (group j is the block's j ^ order), so that their loads fall into different
// banks, and puts the four words of codes back in order at the end.
template <int kSrc, bool kDrop, bool kStoch>
__device__ __forceinline__ void code_rows(const QuantParams& p, uint8_t* tile, uint8_t* srow, const QuantTile& T,
                                          const RngKey& key) {
  using C = QuantConfig<kSrc>;
  constexpr int kWords = C::kHalf ? 16 : 32, kPer = kWords / 4;   // 32-bit words per block and per group
  const int tid = threadIdx.x, blk = tid & 3;
  const float mul = kDrop ? p.scale : 1.0f;
  const uint32_t threshold_hi = p.threshold << 16;
  const int block = (T.c0 >> 5) + blk;
  const int rows = block < p.blocks_c ? p.rows - T.r0 : 0;
  const uint32_t grow0 = static_cast<uint32_t>(T.mat) * static_cast<uint32_t>(p.rows) + static_cast<uint32_t>(T.r0);
#pragma unroll
  for (int i = 0; i < kMxTile * 4 / C::kThreads; ++i) {
    const int lr = (tid >> 2) + i * (C::kThreads / 4);
    const uint32_t order = static_cast<uint32_t>((blk >> 1) | ((lr & 1) << 1));
    uint8_t* row = tile + lr * C::kRowBytes;
    uint32_t w[kWords];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int g8 = blk * 4 + static_cast<int>(j ^ order);
#pragma unroll
      for (int h = 0; h < kPer / 4; ++h) {
        const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * swizzled_group(lr, C::kHalf ? g8 : 2 * g8 + h));
        w[j * kPer + 4 * h] = x.x; w[j * kPer + 4 * h + 1] = x.y;
        w[j * kPer + 4 * h + 2] = x.z; w[j * kPer + 4 * h + 3] = x.w;
      }
    }
    uint32_t group[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      group[j] = static_cast<uint32_t>((T.c0 >> 3) + blk * 4) + (static_cast<uint32_t>(j) ^ order);
    if (kDrop) {
      uint4 num[4];
      philox8x4(key, kRngDropout, grow0 + lr, group, num);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int g8 = blk * 4 + static_cast<int>(j ^ order);
        const uint32_t uu[4] = {num[j].x, num[j].y, num[j].z, num[j].w};
        // a number in an upper half word is compared where it is
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const bool lo = (uu[t] << 16) >= threshold_hi, hi = uu[t] >= threshold_hi;
          if (C::kHalf) {
            if (!lo) w[j * kPer + t] &= 0xFFFF0000u;
            if (!hi) w[j * kPer + t] &= 0xFFFFu;
          } else {
            if (!lo) w[j * kPer + (2 * t) % kPer] = 0u;
            if (!hi) w[j * kPer + (2 * t + 1) % kPer] = 0u;
          }
        }
        if (p.qt) {   // the column pass reads the masked values
#pragma unroll
          for (int h = 0; h < kPer / 4; ++h)
            *reinterpret_cast<uint4*>(row + 16 * swizzled_group(lr, C::kHalf ? g8 : 2 * g8 + h)) =
                make_uint4(w[j * kPer + 4 * h], w[j * kPer + 4 * h + 1], w[j * kPer + 4 * h + 2],
                           w[j * kPer + 4 * h + 3]);
        }
      }
      if (!p.q) continue;
    }
    float amax;
    if constexpr (C::kHalf) {
      uint32_t m = max_abs_bf16x2(w[0], w[1]);
#pragma unroll
      for (int t = 2; t < 16; ++t) m = max_abs_bf16x2(m, w[t]);
      amax = max_nan(fabsf(bf16_lo_f(m)), fabsf(bf16_hi_f(m)));
    } else {
      amax = amax32(w);
    }
    float inv;
    const uint32_t byte = block_scale(amax * mul, inv);
    srow[(lr & 31) * 16 + (lr >> 5) * 4 + blk] = static_cast<uint8_t>(byte);
    const uint32_t inv2 = bf16_bits(kDrop ? 1.0f : inv) * 0x10001u;
    uint32_t c[4];
    uint4 num[4];
    if (kStoch) philox8x4(key, kRngRows, grow0 + lr, group, num);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y[8];
      if constexpr (C::kHalf) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float2 f = mul_bf16x2_f32(w[j * kPer + t], inv2);
          y[2 * t] = f.x;
          y[2 * t + 1] = f.y;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) y[t] = __uint_as_float(w[j * kPer + t]) * (kDrop ? mul : inv);
      }
      if (kDrop) {   // the dropout factor and the scale one after the other: only the first product is rounded
#pragma unroll
        for (int t = 0; t < 8; ++t) y[t] = (C::kHalf ? y[t] * mul : y[t]) * inv;
      }
      c[j] = kStoch ? pack8_stochastic(y, num[j]) : pack8_e2m1(y);
      if (byte == 255u) c[j] = 0u;
    }
    const bool s0 = order & 1u, s1 = order & 2u;
    const uint32_t a0 = s0 ? c[1] : c[0], a1 = s0 ? c[0] : c[1], a2 = s0 ? c[3] : c[2], a3 = s0 ? c[2] : c[3];
    if (lr < rows)
      *reinterpret_cast<uint4*>(p.q + (static_cast<long long>(grow0 + lr) * p.blocks_c + block) * 16) =
          make_uint4(s1 ? a2 : a0, s1 ? a3 : a1, s1 ? a0 : a2, s1 ? a1 : a3);
  }
}

// Columns: a thread codes one 32-row block of two neighbouring columns (bf16)
// or of one (fp32).
template <int kSrc, bool kDrop, bool kStoch>
__device__ __forceinline__ void code_cols(const QuantParams& p, const uint8_t* tile, uint8_t* scol,
                                          const QuantTile& T, const RngKey& key) {
  using C = QuantConfig<kSrc>;
  constexpr int kCols = C::kHalf ? 2 : 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rb = lane >> 3;
  const int lc = (warp * 8 + (lane & 7)) * kCols;
  const float mul = kDrop ? p.scale : 1.0f;
  const uint8_t* at = tile + rb * 32 * C::kRowBytes + tile_offset<C::kHalf>(rb * 32, lc);
  uint32_t raw[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) raw[i] = *reinterpret_cast<const uint32_t*>(at + i * C::kRowBytes);
  float amax[kCols], inv[kCols];
  if constexpr (C::kHalf) {
    uint32_t m[2] = {raw[0], raw[1]};
#pragma unroll
    for (int i = 2; i < 32; ++i) m[i & 1] = max_abs_bf16x2(m[i & 1], raw[i]);
    m[0] = max_abs_bf16x2(m[0], m[1]);
    amax[0] = fabsf(bf16_lo_f(m[0]));
    amax[1] = fabsf(bf16_hi_f(m[0]));
  } else {
    amax[0] = amax32(raw);
  }
  uint32_t byte[kCols];
#pragma unroll
  for (int h = 0; h < kCols; ++h) {
    byte[h] = block_scale(amax[h] * mul, inv[h]);
    scol[((lc + h) & 31) * 16 + ((lc + h) >> 5) * 4 + rb] = static_cast<uint8_t>(byte[h]);
  }
  const uint32_t inv2 = kDrop ? 0x3F803F80u : bf16_bits(inv[0]) | bf16_bits(inv[kCols - 1]) << 16;
  const uint32_t gcol = static_cast<uint32_t>(T.mat) * static_cast<uint32_t>(p.cols) + static_cast<uint32_t>(T.c0 + lc);
  const uint32_t group0 = static_cast<uint32_t>((T.r0 >> 3) + rb * 4);
  const uint32_t group[4] = {group0, group0 + 1, group0 + 2, group0 + 3};
  uint32_t w[kCols][4];
#pragma unroll
  for (int h = 0; h < kCols; ++h) {
    uint4 num[4];
    if (kStoch) philox8x4(key, kRngCols, gcol + h, group, num);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (C::kHalf) {
          const float2 f = mul_bf16x2_f32(raw[g * 8 + j], inv2);
          y[j] = h ? f.y : f.x;
          if (kDrop) y[j] = y[j] * mul * inv[h];
        } else {
          y[j] = kDrop ? __uint_as_float(raw[g * 8 + j]) * mul * inv[0] : __uint_as_float(raw[g * 8 + j]) * inv[0];
        }
      }
      w[h][g] = kStoch ? pack8_stochastic(y, num[g]) : pack8_e2m1(y);
      if (byte[h] == 255u) w[h][g] = 0u;
    }
  }
  const int block = (T.r0 >> 5) + rb;
#pragma unroll
  for (int h = 0; h < kCols; ++h)
    if (T.c0 + lc + h < p.cols && block < p.blocks_r)
      *reinterpret_cast<uint4*>(p.qt + (static_cast<long long>(gcol + h) * p.blocks_r + block) * 16) =
          make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
}

// Persistent over the tiles. While a tile is coded, the next ones are on their
// way to shared memory; its two scale tiles are written one turn later, after
// the barrier that also hands the tile's buffer back.
template <int kSrc, bool kDrop, bool kStoch>
__global__ void __launch_bounds__(QuantConfig<kSrc>::kThreads, QuantConfig<kSrc>::blocks(kStoch))
    quantize_kernel(const __grid_constant__ QuantParams p) {
  using C = QuantConfig<kSrc>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* scales = smem + C::kStages * C::kTileBytes;   // [turn & 1][rows, columns]
  const int tid = threadIdx.x;
  RngKey key{};
  if (kDrop || kStoch) key = rng_key(p.rng, p.site);
  const int ntiles = p.count * p.tiles_r * p.tiles_c;
  const int step = static_cast<int>(gridDim.x);

  auto flush_scales = [&](const QuantTile& T, int turn) {
    const uint4* s = reinterpret_cast<const uint4*>(scales + (turn & 1) * 2 * kMxTileBytes);
    if (tid < 32) {
      if (p.q) reinterpret_cast<uint4*>(p.s + T.at * kMxTileBytes)[tid] = s[tid];
    } else if (tid < 64) {
      if (p.qt) reinterpret_cast<uint4*>(p.st + T.at_t * kMxTileBytes)[tid - 32] = s[tid];
    }
  };

  int ahead = static_cast<int>(blockIdx.x);   // next tile to fetch
  if (C::kStages > 1) {
    for (int s = 0; s < C::kStages - 1; ++s, ahead += step) {
      if (ahead < ntiles) fill_tile<kSrc>(p, smem + s * C::kTileBytes, quant_tile(p, ahead));
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  QuantTile last{};
  int turn = 0;
  for (int t = static_cast<int>(blockIdx.x); t < ntiles; t += step, ++turn) {
    const QuantTile T = quant_tile(p, t);
    uint8_t* tile = smem + (turn % C::kStages) * C::kTileBytes;
    if (C::kStages == 1) {
      if (turn > 0) __syncthreads();   // the previous tile has been coded
      fill_tile<kSrc>(p, tile, T);
    } else {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages > 1 ? C::kStages - 2 : 0) : "memory");
    }
    __syncthreads();
    if (C::kStages > 1) {
      if (ahead < ntiles)
        fill_tile<kSrc>(p, smem + ((turn + C::kStages - 1) % C::kStages) * C::kTileBytes, quant_tile(p, ahead));
      ahead += step;
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    if (turn > 0) flush_scales(last, turn - 1);
    uint8_t* srow = scales + (turn & 1) * 2 * kMxTileBytes;
    if (p.q || kDrop) code_rows<kSrc, kDrop, kStoch>(p, tile, srow, T, key);
    if (p.qt) {
      if (kDrop) __syncthreads();
      code_cols<kSrc, kDrop, kStoch>(p, tile, srow + kMxTileBytes, T, key);
    }
    last = T;
  }
  __syncthreads();
  if (turn > 0) flush_scales(last, turn - 1);
}

// The kernel of a variant, for its launch and for its preparation.
template <int kSrc, bool kDrop, bool kStoch>
static cudaError_t launch_one(const QuantParams* p, int sms, cudaStream_t s) {
  using C = QuantConfig<kSrc>;
  if (!p)
    return cudaFuncSetAttribute(quantize_kernel<kSrc, kDrop, kStoch>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::kSmem);
  const int tiles = p->count * p->tiles_r * p->tiles_c, most = C::blocks(kStoch) * sms;
  quantize_kernel<kSrc, kDrop, kStoch><<<tiles < most ? tiles : most, C::kThreads, C::kSmem, s>>>(*p);
  return cudaGetLastError();
}

template <int kSrc>
static cudaError_t launch_src(const QuantParams& p, int sms, cudaStream_t s) {
  if constexpr (QuantConfig<kSrc>::kBlend) {
    return launch_one<kSrc, false, false>(&p, sms, s);
  } else {
    if (p.threshold)
      return p.stochastic ? launch_one<kSrc, true, true>(&p, sms, s) : launch_one<kSrc, true, false>(&p, sms, s);
    return p.stochastic ? launch_one<kSrc, false, true>(&p, sms, s) : launch_one<kSrc, false, false>(&p, sms, s);
  }
}

cudaError_t launch_quantize(const QuantParams& p, bool bf16, int sms, cudaStream_t s) {
  if (p.ema) return bf16 ? launch_src<kSrcBlendBf16>(p, sms, s) : launch_src<kSrcBlendF32>(p, sms, s);
  return bf16 ? launch_src<kSrcBf16>(p, sms, s) : launch_src<kSrcF32>(p, sms, s);
}

template <int kSrc>
static cudaError_t prepare_src() {
  cudaError_t e = launch_one<kSrc, false, false>(nullptr, 0, nullptr);
  if constexpr (!QuantConfig<kSrc>::kBlend) {
    if (e == cudaSuccess) e = launch_one<kSrc, false, true>(nullptr, 0, nullptr);
    if (e == cudaSuccess) e = launch_one<kSrc, true, false>(nullptr, 0, nullptr);
    if (e == cudaSuccess) e = launch_one<kSrc, true, true>(nullptr, 0, nullptr);
  }
  return e;
}

cudaError_t quantize_prepare() {
  cudaError_t e = prepare_src<kSrcBf16>();
  if (e == cudaSuccess) e = prepare_src<kSrcF32>();
  if (e == cudaSuccess) e = prepare_src<kSrcBlendBf16>();
  if (e == cudaSuccess) e = prepare_src<kSrcBlendF32>();
  return e;
}

// ------------------------------------------------------------------ read-back
// 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : (byte == 255u ? 0x7FC00000u : byte << 23));
}

// Eight codes; the first n of them have scale byte b0, the others b1.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t b0, uint32_t b1, int n, float (&v)[8]) {
  const float scale0 = scale_value(b0), scale1 = scale_value(b1);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h2;
    asm("{\n\t.reg .b8 b;\n\tmov.b16 {b, _}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(h2)
        : "h"(static_cast<uint16_t>((w >> (8 * j)) & 0xFFu)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    v[2 * j] = f.x * (2 * j < n ? scale0 : scale1);
    v[2 * j + 1] = f.y * (2 * j + 1 < n ? scale0 : scale1);
  }
}

__device__ __forceinline__ void decode8(uint32_t w, uint32_t byte, float (&v)[8]) { decode8(w, byte, byte, 8, v); }

__device__ __forceinline__ uint32_t scale_at(const DequantParams& p, int mat, int row, int block) {
  const long long t = (static_cast<long long>(mat) * p.tiles_r + (row >> 7)) * p.tiles_c + (block >> 2);
  return p.s[t * kMxTileBytes + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (block & 3)];
}

// Rows whose length is a multiple of 8: one block per 128 x 128 tile, eight
// groups of 8 elements per thread, all in one column of groups: rows 16 apart.
// The scales of rows r, r + 32, .. of a tile share 16 bytes, so two loads
// bring all eight.
template <bool kBf16>
__global__ void __launch_bounds__(256) dequantize_kernel(const __grid_constant__ DequantParams p) {
  const int per_mat = p.tiles_r * p.tiles_c;
  const int mat = static_cast<int>(blockIdx.x) / per_mat, t = static_cast<int>(blockIdx.x) - mat * per_mat;
  const int tr = t / p.tiles_c, tc = t - tr * p.tiles_c;
  const int cg = threadIdx.x & 15, r = threadIdx.x >> 4, col = tc * kMxTile + cg * 8;
  const int rows = col < p.cols ? p.rows - tr * kMxTile : 0;
  const uint4* st = reinterpret_cast<const uint4*>(p.s + static_cast<long long>(blockIdx.x) * kMxTileBytes);
  const uint4 sa = st[r], sb = st[r + 16];
  const uint32_t scale[8] = {sa.x, sb.x, sa.y, sb.y, sa.z, sb.z, sa.w, sb.w};   // row r + 16 i
  const long long row0 = static_cast<long long>(mat) * p.rows + tr * kMxTile + r;
  const int pitch = p.blocks * 16, shift = (cg >> 2) * 8;
  const uint8_t* in = p.q + row0 * pitch + (col >> 1);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r + 16 * i < rows) w[i] = *reinterpret_cast<const uint32_t*>(in + i * 16 * pitch);
  const long long out = row0 * p.cols + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r + 16 * i < rows) {
      float v[8];
      decode8(w[i], (scale[i] >> shift) & 255u, v);
      store8t<kBf16>(p.out, out + static_cast<long long>(16 * i) * p.cols, v);
    }
  }
}

// Other row lengths, from 8 on: out is contiguous, so a thread still stores
// eight elements of the flat array at once. Their codes are a window of two
// words of a row; where a row ends among the eight, the rest begins the next.
template <bool kBf16>
__global__ void __launch_bounds__(256) dequantize_flat_kernel(const __grid_constant__ DequantParams p, uint32_t n) {
  constexpr int kEach = 2;   // groups per thread, all loads first
  struct Window {            // eight codes of a row from some column on, and their scales
    uint32_t lo, hi, s0, s1;
    int col;
  };
  auto fetch = [&](int gr, int c) {
    const int mat = fdiv(gr, p.fd_rows), row = gr - mat * p.rows;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p.q + static_cast<long long>(gr) * p.blocks * 16) + (c >> 3);
    Window x;
    x.lo = w[0];
    x.hi = (c >> 3) + 1 < p.blocks * 4 ? w[1] : 0u;
    x.s0 = scale_at(p, mat, row, c >> 5);
    x.s1 = scale_at(p, mat, row, min((c >> 5) + 1, p.blocks - 1));
    x.col = c;
    return x;
  };
  auto decode = [&](const Window& x, float (&v)[8]) {
    decode8(__funnelshift_r(x.lo, x.hi, 4 * (x.col & 7)), x.s0, x.s1, 32 - (x.col & 31), v);
  };
  const uint32_t at0 = blockIdx.x * (2048u * kEach) + threadIdx.x * 8u;
  Window own[kEach];
  int row[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const uint32_t at = at0 + 2048u * e;
    if (at < n) {
      row[e] = fdiv(static_cast<int>(at), p.fd_cols);
      own[e] = fetch(row[e], static_cast<int>(at) - row[e] * p.cols);
    }
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const uint32_t at = at0 + 2048u * e;
    if (at >= n) continue;
    float v[8];
    decode(own[e], v);
    const int left = p.cols - own[e].col;
    if (left < 8 && at + left < n) {
      float t[8];
      decode(fetch(row[e] + 1, 0), t);
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        // v[j] = t[j - left] for j >= left, without indexing registers
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (j - left == i) v[j] = t[i];
      }
    }
    if (at + 8 <= n) {
      store8t<kBf16>(p.out, at, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < n) store1t<kBf16>(p.out, at + j, v[j]);
    }
  }
}

// Any row length and size, element by element: a warp decodes 32 groups and passes them through shared
// memory, so that neighbouring lanes store neighbouring elements.
template <bool kBf16>
__global__ void __launch_bounds__(256) dequantize_ragged_kernel(const __grid_constant__ DequantParams p) {
  __shared__ float values[8][32 * 9];   // nine words per group: conflict-free both ways
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t step = gridDim.x * 256u;
  for (uint32_t base = blockIdx.x * 256u + warp * 32u; base < p.total; base += step) {
    const uint32_t i = base + lane;
    long long at = 0;
    int len = 0;
    if (i < p.total) {
      const int grow = fdiv(static_cast<int>(i), p.fd_groups);
      const int g = static_cast<int>(i) - grow * p.groups;
      const int mat = fdiv(grow, p.fd_rows), row = grow - mat * p.rows;
      at = static_cast<long long>(grow) * p.cols + g * 8;
      len = min(8, p.cols - g * 8);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p.q + static_cast<long long>(grow) * p.blocks * 16 + g * 4);
      float v[8];
      decode8(w, scale_at(p, mat, row, g >> 2), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) values[warp][lane * 9 + j] = v[j];
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int owner = t * 4 + (lane >> 3), j = lane & 7;
      const long long e = __shfl_sync(0xffffffffu, at, owner) + j;
      if (j < __shfl_sync(0xffffffffu, len, owner)) store1t<kBf16>(p.out, e, values[warp][owner * 9 + j]);
    }
    __syncwarp();
  }
}

cudaError_t launch_dequantize(const DequantParams& p, bool bf16, int sms, cudaStream_t s) {
  const uint32_t want = (p.total + 255) / 256, most = 32u * static_cast<uint32_t>(sms);
  const uint32_t grid = want < most ? want : most;
  if (p.cols % 8 == 0) {
    const uint32_t blocks = static_cast<uint32_t>(p.count) * p.tiles_r * p.tiles_c;
    if (bf16) dequantize_kernel<true><<<blocks, 256, 0, s>>>(p);
    else dequantize_kernel<false><<<blocks, 256, 0, s>>>(p);
  } else if (const long long n = static_cast<long long>(p.count) * p.rows * p.cols;
             p.cols >= 8 && n < (1LL << 31) - 4096) {   // 32-bit flat indices
    const uint32_t blocks = static_cast<uint32_t>((n + 4095) / 4096);
    if (bf16) dequantize_flat_kernel<true><<<blocks, 256, 0, s>>>(p, static_cast<uint32_t>(n));
    else dequantize_flat_kernel<false><<<blocks, 256, 0, s>>>(p, static_cast<uint32_t>(n));
  } else {
    if (bf16) dequantize_ragged_kernel<true><<<grid, 256, 0, s>>>(p);
    else dequantize_ragged_kernel<false><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace muon
