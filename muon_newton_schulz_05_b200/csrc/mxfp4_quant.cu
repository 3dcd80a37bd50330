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
// quantize: one block per 128 x 128 tile reads it once and writes both
// orientations from it, each with its whole 512-byte scale tile. Rows are
// coded from registers (four lanes hold a block of 32 columns); the values
// also go to shared memory, from where each thread codes two neighbouring
// columns of one 32-row block. The tile is stored with its 16-byte groups
// XOR-ed by the row block, so that the column reads (8 column pairs x 4 row
// blocks per warp) touch every bank once.
// Dropout, and the blend of the parameters with their average, are applied to
// the values as they are read.
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

// The eight codes of eight values of one block, in a 32-bit word.
__device__ __forceinline__ uint32_t code8(const float (&v)[8], float mul, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w |= pack_e2m1(v[2 * j] * mul * inv, v[2 * j + 1] * mul * inv) << (8 * j);
  return w;
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

// Eight source values from element `at` on (n of them exist; the rest are 0).
template <int kSrc>
__device__ __forceinline__ void source8(const QuantParams& p, long long at, int n, bool vec, float (&v)[8]) {
  constexpr bool bf16 = kSrc == kSrcBf16 || kSrc == kSrcBlendBf16;
  constexpr bool blend = kSrc >= kSrcBlendBf16;
  if (vec && n >= 8) {
    load8t<bf16>(p.x, at, v);
    if (blend) {
      float e[8];
      load8t<false>(p.ema, at, e);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(p.w_final, v[j], __fmul_rn(p.w_ema, e[j]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (j < n) {
        v[j] = load1t<bf16>(p.x, at + j);
        if (blend) v[j] = fmaf(p.w_final, v[j], __fmul_rn(p.w_ema, p.ema[at + j]));
      }
    }
  }
}

// Shared-memory position (in 16-byte groups) of 16-byte group g of a row.
template <bool kHalf>
__device__ __forceinline__ int swizzled_group(int row, int g) {
  return g ^ ((row >> 5) * (kHalf ? 2 : 4));
}

template <int kSrc>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ QuantParams p) {
  constexpr bool kHalf = kSrc == kSrcBf16;              // the tile is kept as bf16, else as fp32
  constexpr int kRowBytes = kMxTile * (kHalf ? 2 : 4);
  extern __shared__ __align__(16) uint8_t tile[];       // 128 rows, then the two scale tiles
  uint8_t* srow = tile + kMxTile * kRowBytes;
  uint8_t* scol = srow + kMxTileBytes;

  const int per_mat = p.tiles_r * p.tiles_c;
  const int mat = static_cast<int>(blockIdx.x) / per_mat;
  const int t = static_cast<int>(blockIdx.x) - mat * per_mat;
  const int tr = t / p.tiles_c, tc = t - (t / p.tiles_c) * p.tiles_c;
  const int r0 = tr * kMxTile, c0 = tc * kMxTile;
  const int tid = threadIdx.x, lane = tid & 31;
  const bool vec = (p.cols & 7) == 0;
  const bool drop = p.threshold != 0;
  const float mul = drop ? p.scale : 1.0f;
  RngKey key{};
  if (drop || p.stochastic) key = rng_key(p.rng, p.site);

  // ---- rows: 16 lanes per row, four lanes per block of 32 columns
  const int cg = tid & 15;
  const int col = c0 + cg * 8;
  constexpr int kBatch = 4;
#pragma unroll 1
  for (int b = 0; b < 8; b += kBatch) {
    float v[kBatch][8];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = r0 + (b + i) * 16 + (tid >> 4);
      const int n = row < p.rows ? min(8, p.cols - col) : 0;
      source8<kSrc>(p, (static_cast<long long>(mat) * p.rows + row) * p.cols + col, n, vec, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int lr = (b + i) * 16 + (tid >> 4), row = r0 + lr;
      const uint32_t grow = static_cast<uint32_t>(mat) * static_cast<uint32_t>(p.rows) + static_cast<uint32_t>(row);
      if (drop) {
        const uint4 u = philox8(key, kRngDropout, grow, static_cast<uint32_t>(col >> 3));
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (((j & 1) ? uu[j >> 1] >> 16 : uu[j >> 1] & 0xFFFFu) < p.threshold) v[i][j] = 0.0f;
      }
      if (p.qt) {
        uint8_t* at = tile + lr * kRowBytes;
        if (kHalf) {
          *reinterpret_cast<uint4*>(at + 16 * swizzled_group<true>(lr, cg)) =
              make_uint4(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]),
                         pack_bf16x2(v[i][4], v[i][5]), pack_bf16x2(v[i][6], v[i][7]));
        } else {
          *reinterpret_cast<float4*>(at + 16 * swizzled_group<false>(lr, 2 * cg)) =
              make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
          *reinterpret_cast<float4*>(at + 16 * swizzled_group<false>(lr, 2 * cg + 1)) =
              make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
        }
      }
      if (p.q) {
        float amax = fabsf(v[i][0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) amax = max_nan(amax, fabsf(v[i][j]));
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float inv;
        const uint32_t byte = block_scale(amax * mul, inv);
        uint32_t w;
        if (p.stochastic)
          w = code8_stochastic(v[i], mul, inv, philox8(key, kRngRows, grow, static_cast<uint32_t>(col >> 3)));
        else
          w = code8(v[i], mul, inv);
        if (byte == 255u) w = 0u;
        if ((lane & 3) == 0) srow[(lr & 31) * 16 + (lr >> 5) * 4 + (cg >> 2)] = static_cast<uint8_t>(byte);
        if (row < p.rows && (col >> 5) < p.blocks_c) {
          const long long qrow = static_cast<long long>(mat) * p.rows + row;
          *reinterpret_cast<uint32_t*>(p.q + qrow * (p.blocks_c * 16) + (col >> 1)) = w;
        }
      }
    }
  }
  __syncthreads();

  // ---- columns: a thread takes two neighbouring columns of one 32-row block
  if (p.qt) {
    const int rb = (lane >> 3);
    const int lc = ((tid >> 5) * 8 + (lane & 7)) * 2;   // first of the two columns
    float amax[2] = {0.0f, 0.0f};
    uint32_t pk[kHalf ? 32 : 1];
    float2 pf[kHalf ? 1 : 32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int lr = rb * 32 + i;
      const uint8_t* at = tile + lr * kRowBytes;
      float a, b;
      if (kHalf) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(
            at + 16 * swizzled_group<true>(lr, lc >> 3) + (lc & 7) * 2);
        pk[kHalf ? i : 0] = w;
        a = bf16_lo_f(w);
        b = bf16_hi_f(w);
      } else {
        const float2 f = *reinterpret_cast<const float2*>(
            at + 16 * swizzled_group<false>(lr, lc >> 2) + (lc & 3) * 4);
        pf[kHalf ? 0 : i] = f;
        a = f.x;
        b = f.y;
      }
      amax[0] = max_nan(amax[0], fabsf(a));
      amax[1] = max_nan(amax[1], fabsf(b));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + lc + h;
      float inv;
      const uint32_t byte = block_scale(amax[h] * mul, inv);
      scol[((lc + h) & 31) * 16 + ((lc + h) >> 5) * 4 + rb] = static_cast<uint8_t>(byte);
      const uint32_t gcol = static_cast<uint32_t>(mat) * static_cast<uint32_t>(p.cols) + static_cast<uint32_t>(c);
      uint32_t w[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (kHalf) {
            const uint32_t x = pk[kHalf ? g * 8 + j : 0];
            v[j] = h ? bf16_hi_f(x) : bf16_lo_f(x);
          } else {
            const float2 x = pf[kHalf ? 0 : g * 8 + j];
            v[j] = h ? x.y : x.x;
          }
        }
        if (p.stochastic)
          w[g] = code8_stochastic(v, mul, inv,
                                  philox8(key, kRngCols, gcol, static_cast<uint32_t>((r0 >> 3) + rb * 4 + g)));
        else
          w[g] = code8(v, mul, inv);
        if (byte == 255u) w[g] = 0u;
      }
      const int block = (r0 >> 5) + rb;
      if (c < p.cols && block < p.blocks_r) {
        const long long qrow = static_cast<long long>(mat) * p.cols + c;
        *reinterpret_cast<uint4*>(p.qt + (qrow * p.blocks_r + block) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncthreads();
  }

  // ---- the two scale tiles, 512 bytes each
  if (tid < 32 && p.q) {
    const long long at = (static_cast<long long>(mat) * p.tiles_r + tr) * p.tiles_c + tc;
    reinterpret_cast<uint4*>(p.s + at * kMxTileBytes)[tid] = reinterpret_cast<const uint4*>(srow)[tid];
  } else if (tid >= 32 && tid < 64 && p.qt) {
    const long long at = (static_cast<long long>(mat) * p.tiles_c + tc) * p.tiles_r + tr;
    reinterpret_cast<uint4*>(p.st + at * kMxTileBytes)[tid - 32] = reinterpret_cast<const uint4*>(scol)[tid - 32];
  }
}

template <int kSrc>
static cudaError_t launch_src(const QuantParams& p, cudaStream_t s) {
  constexpr int smem = kMxTile * kMxTile * (kSrc == kSrcBf16 ? 2 : 4) + 2 * kMxTileBytes;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(quantize_kernel<kSrc>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = static_cast<unsigned>(p.count) * p.tiles_r * p.tiles_c;
  quantize_kernel<kSrc><<<grid, 256, smem, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_quantize(const QuantParams& p, bool bf16, cudaStream_t s) {
  if (p.ema) return bf16 ? launch_src<kSrcBlendBf16>(p, s) : launch_src<kSrcBlendF32>(p, s);
  return bf16 ? launch_src<kSrcBf16>(p, s) : launch_src<kSrcF32>(p, s);
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

// Rows whose length is a multiple of 8: eight elements per thread.
template <bool kBf16>
__global__ void __launch_bounds__(256) dequantize_kernel(const __grid_constant__ DequantParams p) {
  const uint32_t step = gridDim.x * 256u;
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < p.total; i += step) {
    const int grow = fdiv(static_cast<int>(i), p.fd_groups);
    const int g = static_cast<int>(i) - grow * p.groups;
    const int mat = fdiv(grow, p.fd_rows), row = grow - mat * p.rows;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p.q + static_cast<long long>(grow) * p.blocks * 16 + g * 4);
    float v[8];
    decode8(w, scale_at(p, mat, row, g >> 2), v);
    store8t<kBf16>(p.out, static_cast<long long>(i) * 8, v);
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
    if (bf16) dequantize_kernel<true><<<grid, 256, 0, s>>>(p);
    else dequantize_kernel<false><<<grid, 256, 0, s>>>(p);
  } else {
    if (bf16) dequantize_ragged_kernel<true><<<grid, 256, 0, s>>>(p);
    else dequantize_ragged_kernel<false><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace muon
