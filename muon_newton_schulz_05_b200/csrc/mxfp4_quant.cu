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
// from shared memory, each with its whole 512-byte scale tile. Rows are coded
// by four lanes per block of 32 columns, columns by one thread per 32-row
// block. Dropout is applied in the row pass, which writes the masked values
// back for the column pass; the blend of the parameters with their average is
// formed while the tile is filled.
#include "dtype_io.cuh"
#include "lowbit.cuh"
#include "philox.cuh"

namespace muon {

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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

// Codes of two values already in e2m1's range: lo in bits 0..3, hi in 4..7.
__device__ __forceinline__ uint32_t pack_e2m1(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b16 %0, {t, 0};\n\t}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// Stochastic code of y (|y| <= 6): between the neighbours of |y|, up when the
// 16-bit number plus one half is below the fraction times 2^16 (all exact).
__device__ __forceinline__ uint32_t stochastic_e2m1(float y, uint32_t u16) {
  const float a = fabsf(y);
  const float steps = a < 2.0f ? 2.0f * a : (a < 4.0f ? a : 0.5f * a);
  const uint32_t base = a < 2.0f ? 0u : (a < 4.0f ? 2u : 4u);
  const float low = floorf(steps);
  const bool up = static_cast<float>(u16) + 0.5f < (steps - low) * 65536.0f;
  return (static_cast<uint32_t>(low) + base + (up ? 1u : 0u)) | (__float_as_uint(y) >> 31 << 3);
}

// The eight codes of eight values of one block, in a 32-bit word. (mul, the
// dropout factor, and inv are applied one after the other: the first product
// is rounded, the second one is exact.)
template <bool kMul>
__device__ __forceinline__ uint32_t code8(const float (&v)[8], float mul, float inv) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    b[j] = kMul ? pack_e2m1(v[2 * j] * mul * inv, v[2 * j + 1] * mul * inv)
                : pack_e2m1(v[2 * j] * inv, v[2 * j + 1] * inv);
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t code8_stochastic(const float (&v)[8], float mul, float inv, const uint4& u) {
  const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w |= stochastic_e2m1(v[2 * j] * mul * inv, uu[j] & 0xFFFFu) << (8 * j);
    w |= stochastic_e2m1(v[2 * j + 1] * mul * inv, uu[j] >> 16) << (8 * j + 4);
  }
  return w;
}

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
  x.mat = t / per_mat;
  const int u = t - x.mat * per_mat;
  const int tr = u / p.tiles_c, tc = u - tr * p.tiles_c;
  x.r0 = tr * kMxTile;
  x.c0 = tc * kMxTile;
  x.at = t;
  x.at_t = static_cast<long long>(x.mat) * per_mat + static_cast<long long>(tc) * p.tiles_r + tr;
  return x;
}

// Copies a tile to shared memory, 16 bytes at a time: asynchronously where
// rows start on 16-byte boundaries, else through registers; what lies outside
// the matrix becomes zero. The blend is formed here, with the roundings of
// readout_blend.
template <int kSrc>
__device__ __forceinline__ void fill_tile(const QuantParams& p, uint8_t* tile, const QuantTile& T) {
  using C = QuantConfig<kSrc>;
  constexpr int kPer = C::kHalf ? 8 : 4;                        // elements per 16-byte group
  constexpr int kGroups = kMxTile / kPer;                       // groups per row
  constexpr int kEach = kMxTile * kGroups / C::kThreads;
  constexpr int kElt = C::kBf16 ? 2 : 4;
  const bool vec = p.cols % 8 == 0;
  const int g = threadIdx.x % kGroups;
  const int col = T.c0 + g * kPer;
  const int n = p.cols - col;
  if (!C::kBlend && vec) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int lr = i * (C::kThreads / kGroups) + static_cast<int>(threadIdx.x) / kGroups;
      const int row = T.r0 + lr;
      const bool exists = row < p.rows && n > 0;
      const long long e = exists ? (static_cast<long long>(T.mat) * p.rows + row) * p.cols + col : 0;
      copy16_async(tile + lr * C::kRowBytes + 16 * swizzled_group(lr, g),
                   static_cast<const uint8_t*>(p.x) + e * kElt, exists);
    }
    return;
  }
#pragma unroll 4
  for (int i = 0; i < kEach; ++i) {
    const int lr = i * (C::kThreads / kGroups) + static_cast<int>(threadIdx.x) / kGroups;
    const int row = T.r0 + lr;
    const long long e = (static_cast<long long>(T.mat) * p.rows + row) * p.cols + col;
    float v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = 0.0f;
    if (row < p.rows && n > 0) {
      if (vec) {   // only the blend comes here: four fp32 averages and four parameters
        const float4 a = *reinterpret_cast<const float4*>(p.ema + e);
        const float em[4] = {a.x, a.y, a.z, a.w};
        float th[4];
        if (C::kBf16) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.x) + e);
          th[0] = bf16_lo_f(w.x); th[1] = bf16_hi_f(w.x); th[2] = bf16_lo_f(w.y); th[3] = bf16_hi_f(w.y);
        } else {
          const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + e);
          th[0] = f.x; th[1] = f.y; th[2] = f.z; th[3] = f.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(p.w_final, th[j], __fmul_rn(p.w_ema, em[j]));
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (j < n) {
            v[j] = load1t<C::kBf16>(p.x, e + j);
            if (C::kBlend) v[j] = fmaf(p.w_final, v[j], __fmul_rn(p.w_ema, p.ema[e + j]));
          }
        }
      }
    }
    uint8_t* at = tile + lr * C::kRowBytes + 16 * swizzled_group(lr, g);
    if (C::kHalf)
      *reinterpret_cast<uint4*>(at) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4 % kPer], v[5 % kPer]),
                     pack_bf16x2(v[6 % kPer], v[7 % kPer]));
    else
      *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// Eight values of group cg (8 columns) of a tile row.
template <bool kHalf>
__device__ __forceinline__ void tile8(const uint8_t* row, int lr, int cg, float (&v)[8]) {
  if (kHalf) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + 16 * swizzled_group(lr, cg));
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v[2 * h] = bf16_lo_f(ww[h]);
      v[2 * h + 1] = bf16_hi_f(ww[h]);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(row + 16 * swizzled_group(lr, 2 * cg));
    const float4 b = *reinterpret_cast<const float4*>(row + 16 * swizzled_group(lr, 2 * cg + 1));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// Rows: 16 lanes per row, four lanes per block of 32 columns.
template <int kSrc, bool kDrop, bool kStoch>
__device__ __forceinline__ void code_rows(const QuantParams& p, uint8_t* tile, uint8_t* srow, const QuantTile& T,
                                          const RngKey& key) {
  using C = QuantConfig<kSrc>;
  const int tid = threadIdx.x, cg = tid & 15, col = T.c0 + cg * 8;
  const float mul = kDrop ? p.scale : 1.0f;
#pragma unroll 2
  for (int i = 0; i < kMxTile * 16 / C::kThreads; ++i) {
    const int lr = i * (C::kThreads / 16) + (tid >> 4), row = T.r0 + lr;
    uint8_t* at = tile + lr * C::kRowBytes;
    float v[8];
    tile8<C::kHalf>(at, lr, cg, v);
    const uint32_t grow = static_cast<uint32_t>(T.mat) * static_cast<uint32_t>(p.rows) + static_cast<uint32_t>(row);
    if (kDrop) {
      const uint4 u = philox8(key, kRngDropout, grow, static_cast<uint32_t>(col >> 3));
      const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (((j & 1) ? uu[j >> 1] >> 16 : uu[j >> 1] & 0xFFFFu) < p.threshold) v[j] = 0.0f;
      if (p.qt) {  // the column pass reads the masked values
        if (C::kHalf) {
          *reinterpret_cast<uint4*>(at + 16 * swizzled_group(lr, cg)) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
        } else {
          *reinterpret_cast<float4*>(at + 16 * swizzled_group(lr, 2 * cg)) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(at + 16 * swizzled_group(lr, 2 * cg + 1)) = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
      if (!p.q) continue;
    }
    float amax = fabsf(v[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) amax = max_nan(amax, fabsf(v[j]));
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    float inv;
    const uint32_t byte = block_scale(amax * mul, inv);
    uint32_t w = kStoch ? code8_stochastic(v, mul, inv, philox8(key, kRngRows, grow, static_cast<uint32_t>(col >> 3)))
                        : code8<kDrop>(v, mul, inv);
    if (byte == 255u) w = 0u;
    if ((tid & 3) == 0) srow[(lr & 31) * 16 + (lr >> 5) * 4 + (cg >> 2)] = static_cast<uint8_t>(byte);
    if (row < p.rows && (col >> 5) < p.blocks_c) {
      const long long qrow = static_cast<long long>(T.mat) * p.rows + row;
      *reinterpret_cast<uint32_t*>(p.q + qrow * (p.blocks_c * 16) + (col >> 1)) = w;
    }
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
  const uint8_t* base = tile + rb * 32 * C::kRowBytes;
  uint32_t raw[32];
  if (C::kHalf) {
    const uint8_t* at = base + 16 * swizzled_group(rb * 32, lc >> 3) + (lc & 7) * 2;
#pragma unroll
    for (int i = 0; i < 32; ++i) raw[i] = *reinterpret_cast<const uint32_t*>(at + i * C::kRowBytes);
  } else {
    const uint8_t* at = base + 16 * swizzled_group(rb * 32, lc >> 2) + (lc & 3) * 4;
#pragma unroll
    for (int i = 0; i < 32; ++i) raw[i] = *reinterpret_cast<const uint32_t*>(at + i * C::kRowBytes);
  }
#pragma unroll
  for (int h = 0; h < kCols; ++h) {
    const int c = T.c0 + lc + h;
    auto value = [&](int i) {
      return C::kHalf ? (h ? bf16_hi_f(raw[i]) : bf16_lo_f(raw[i])) : __uint_as_float(raw[i]);
    };
    float amax = fabsf(value(0));
#pragma unroll
    for (int i = 1; i < 32; ++i) amax = max_nan(amax, fabsf(value(i)));
    float inv;
    const uint32_t byte = block_scale(amax * mul, inv);
    scol[((lc + h) & 31) * 16 + ((lc + h) >> 5) * 4 + rb] = static_cast<uint8_t>(byte);
    const uint32_t gcol = static_cast<uint32_t>(T.mat) * static_cast<uint32_t>(p.cols) + static_cast<uint32_t>(c);
    uint32_t w[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = value(g * 8 + j);
      w[g] = kStoch ? code8_stochastic(v, mul, inv, philox8(key, kRngCols, gcol,
                                                            static_cast<uint32_t>((T.r0 >> 3) + rb * 4 + g)))
                    : code8<kDrop>(v, mul, inv);
      if (byte == 255u) w[g] = 0u;
    }
    const int block = (T.r0 >> 5) + rb;
    if (c < p.cols && block < p.blocks_r) {
      const long long qrow = static_cast<long long>(T.mat) * p.cols + c;
      *reinterpret_cast<uint4*>(p.qt + (qrow * p.blocks_r + block) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
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

template <int kSrc, bool kDrop, bool kStoch>
static cudaError_t launch_one(const QuantParams& p, int sms, cudaStream_t s) {
  using C = QuantConfig<kSrc>;
  const cudaError_t e = cudaFuncSetAttribute(quantize_kernel<kSrc, kDrop, kStoch>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = p.count * p.tiles_r * p.tiles_c, most = C::blocks(kStoch) * sms;
  quantize_kernel<kSrc, kDrop, kStoch><<<tiles < most ? tiles : most, C::kThreads, C::kSmem, s>>>(p);
  return cudaGetLastError();
}

template <int kSrc>
static cudaError_t launch_src(const QuantParams& p, int sms, cudaStream_t s) {
  if constexpr (QuantConfig<kSrc>::kBlend) {
    return launch_one<kSrc, false, false>(p, sms, s);
  } else {
    if (p.threshold)
      return p.stochastic ? launch_one<kSrc, true, true>(p, sms, s) : launch_one<kSrc, true, false>(p, sms, s);
    return p.stochastic ? launch_one<kSrc, false, true>(p, sms, s) : launch_one<kSrc, false, false>(p, sms, s);
  }
}

cudaError_t launch_quantize(const QuantParams& p, bool bf16, int sms, cudaStream_t s) {
  if (p.ema) return bf16 ? launch_src<kSrcBlendBf16>(p, sms, s) : launch_src<kSrcBlendF32>(p, sms, s);
  return bf16 ? launch_src<kSrcBf16>(p, sms, s) : launch_src<kSrcF32>(p, sms, s);
}

// ------------------------------------------------------------------ read-back
__device__ __forceinline__ void decode8(uint32_t w, uint32_t byte, float (&v)[8]) {
  // 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 is NaN
  const float scale = __uint_as_float(byte == 0u ? 0x00400000u : (byte == 255u ? 0x7FC00000u : byte << 23));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h2;
    asm("{\n\t.reg .b8 b;\n\tmov.b16 {b, _}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(h2)
        : "h"(static_cast<uint16_t>((w >> (8 * j)) & 0xFFu)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    v[2 * j] = f.x * scale;
    v[2 * j + 1] = f.y * scale;
  }
}

__device__ __forceinline__ uint32_t scale_at(const DequantParams& p, int mat, int row, int block) {
  const long long t = (static_cast<long long>(mat) * p.tiles_r + (row >> 7)) * p.tiles_c + (block >> 2);
  return p.s[t * kMxTileBytes + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (block & 3)];
}

// Rows whose length is a multiple of 8: four groups of eight elements per
// thread, all loads first.
template <bool kBf16>
__global__ void __launch_bounds__(256) dequantize_kernel(const __grid_constant__ DequantParams p) {
  constexpr int kEach = 4;
  const uint32_t i0 = blockIdx.x * (256u * kEach) + threadIdx.x;
  uint32_t w[kEach], byte[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const uint32_t i = i0 + u * 256u;
    if (i < p.total) {
      const int grow = fdiv(static_cast<int>(i), p.fd_groups);
      const int g = static_cast<int>(i) - grow * p.groups;
      const int mat = fdiv(grow, p.fd_rows), row = grow - mat * p.rows;
      w[u] = *reinterpret_cast<const uint32_t*>(p.q + static_cast<long long>(grow) * p.blocks * 16 + g * 4);
      byte[u] = scale_at(p, mat, row, g >> 2);
    }
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const uint32_t i = i0 + u * 256u;
    if (i < p.total) {
      float v[8];
      decode8(w[u], byte[u], v);
      store8t<kBf16>(p.out, static_cast<long long>(i) * 8, v);
    }
  }
}

// Any row length: a warp decodes 32 groups and passes them through shared
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
    const uint32_t blocks = (p.total + 1023) / 1024;
    if (bf16) dequantize_kernel<true><<<blocks, 256, 0, s>>>(p);
    else dequantize_kernel<false><<<blocks, 256, 0, s>>>(p);
  } else {
    if (bf16) dequantize_ragged_kernel<true><<<grid, 256, 0, s>>>(p);
    else dequantize_ragged_kernel<false><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace muon
