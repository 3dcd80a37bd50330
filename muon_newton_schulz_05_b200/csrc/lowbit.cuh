// Plan structures of the dropout and 4-bit (MXFP4) passes, shared by the host
// API and the kernels.
//
// An MXFP4 matrix [rows][cols] is stored as
//   data   : e2m1 codes, two per byte (first element in the low half), rows
//            padded to 32 elements: [rows][blocks * 16] bytes
//   scales : one e8m0 byte per block of 32 elements (2^(byte - 127), 255 = NaN)
//            in tiles of 128 rows x 4 blocks, 512 bytes each, tile (i, j) at
//            (i * ceil(blocks / 4) + j) * 512; inside it row r, block b at
//            (r % 32) * 16 + (r / 32) * 4 + b. This is the order in which the
//            tensor cores' scale memory takes them, so a tile is copied there
//            as it is. The padding is zero.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "muon_b200.h"
#include "plan.cuh"

namespace muon {

constexpr int kMxBlock = 32;    // elements that share a scale
constexpr int kMxTile = 128;    // rows (and columns) of a scale tile
constexpr int kMxTileBytes = 512;

struct DropoutParams {
  const void* x;
  const void* residual;         // NULL: none
  void* out;
  const long long* rng;         // {seed, offset}
  unsigned long long site;
  long long rows;
  int cols;
  int groups;                   // ceil(cols / 8)
  FastDiv fd_groups, fd_cols;
  uint32_t total;               // rows * groups (< 2^31)
  uint32_t threshold;           // dropped when the 16-bit number is below it
  float scale;                  // 2^16 / (2^16 - threshold)
};

struct QuantParams {
  const void* x;                // source, or theta of the blend
  const float* ema;             // blend only
  float w_final, w_ema;         // blend weights
  uint8_t *q, *s;               // blocks along the columns (NULL: not wanted)
  uint8_t *qt, *st;             // transposed, blocks along the rows (NULL: not wanted)
  const long long* rng;
  unsigned long long site;
  int count, rows, cols;
  int tiles_r, tiles_c;         // 128 x 128 tiles
  FastDiv fd_tiles, fd_tiles_c; // by tiles_r * tiles_c, by tiles_c
  int blocks_r, blocks_c;       // 32-element blocks along the rows / columns
  uint32_t threshold;           // dropout; 0: none
  float scale;
  int stochastic;
};

struct DequantParams {
  const uint8_t *q, *s;
  void* out;
  int count, rows, cols;
  int blocks, tiles_r, tiles_c;
  int groups;                   // ceil(cols / 8)
  FastDiv fd_groups, fd_rows, fd_cols;
  uint32_t total;               // count * rows * groups (< 2^31)
};

cudaError_t launch_dropout(const DropoutParams& p, bool bf16, int sms, cudaStream_t s);
cudaError_t quantize_prepare();   // kernel attributes; once per device
cudaError_t launch_quantize(const QuantParams& p, bool bf16, int sms, cudaStream_t s);
cudaError_t launch_dequantize(const DequantParams& p, bool bf16, int sms, cudaStream_t s);

// From api.cu: the current device's SM count, the tensor-map encoder (after
// library_device has succeeded once), the limit of device-side waits and the
// fault mode (muon_set_debug).
muon_status library_device(int* sms);
double wait_limit_seconds();
int fault_mode();
muon_status encode_tiled(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* ptr,
                         const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                         CUtensorMapSwizzle swz);

}  // namespace muon
