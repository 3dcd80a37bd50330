// Launch parameters of the MXFP4 product kernels, and the rule that picks one.
#pragma once
#include "lowbit.cuh"

namespace muon {

// out[c][m][n] = [add +] sum_k A[c][m][k] B[c][n][k]
struct MxGemmParams {
  CUtensorMap rows_l, rows_r;      // codes: uint8 [count][rows][blocks * 16], 128-byte swizzle
  CUtensorMap scales_l, scales_r;  // pair kernel, scale tiles: uint32 [count * tiles][ceil(blocks / 4) * 128]
  CUtensorMap result;              // pair kernel: out [count][m][n], boxes of 32 rows x 128 bytes (if tma_out)
  CUtensorMap addend;              // add, the same way
  int tma_out;
  const uint8_t *sf_l, *sf_r;      // the scale tiles themselves (few-row kernel)
  int sf_groups;                   // tiles per tile row
  const void* add;
  void* out;
  float* part;                     // split products: fp32 partial tiles in the workspace
  int m, n;                        // rows of the left and right operand
  int count;
  int share_l, share_r;            // 1: one matrix serves every product of the call
  int tiles_l, tiles_r;            // 128-row scale tiles per matrix of each operand
  int k64;                         // 64-element steps of K
  int kstages;                     // 256-element pipeline stages of K
  int split, kc;                   // K splits, stages per split
  int ring;                        // few-row kernel: pipeline stages in shared memory
  int tm, tn;                      // output tiles
  int group;                       // row tiles per column sweep (a band)
  FastDiv fd_split, fd_mat, fd_band, fd_group, fd_rest;  // by split, tm * tn, group * tn, group, the last band's rows
  long long stride_l, stride_r, stride_c;  // of out, per left row, right row and matrix
  int* status;
  unsigned long long wait_limit_ns;
  int fault;                       // test hook (muon_set_debug)
};

struct MxGemmShape {
  int64_t count, m, n, k;
};

// How a product is run. few: the few-row kernel (swap: its left operand, the
// one with many rows, is B); otherwise the pair kernel.
struct MxGemmPlan {
  bool few, swap;
  int nt;          // few-row kernel: columns of the tile
  int split, kc;   // K splits (few-row kernel: the CTAs of a cluster)
  int ring;
  int tm, tn;
  size_t part_bytes;
};

MxGemmPlan plan_mx_gemm(const MxGemmShape& s, int pairs, int sms);
cudaError_t mx_gemm_prepare(int* max_pairs);
cudaError_t launch_mx_gemm(const MxGemmParams& p, const MxGemmPlan& plan, bool bf16, int max_pairs,
                           cudaStream_t s);

}  // namespace muon
