// Dropout from a counter-based generator: out = [residual +] x k / (1 - t / 2^16),
// k = 1 where the element's 16-bit number is at least t. The mask is never
// stored; the backward pass is the same call on the output's gradient.
// p is taken to the nearest multiple t of 2^-16 and the scale belongs to that
// t, so the expectation is exact.
#include "dtype_io.cuh"
#include "lowbit.cuh"
#include "philox.cuh"

namespace muon {

__device__ __forceinline__ float dropped(float x, uint32_t u16, uint32_t threshold, float scale) {
  return u16 >= threshold ? x * scale : 0.0f;
}

__device__ __forceinline__ uint32_t half_of(const uint4& w, int j) {
  const uint32_t v = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
  return (j & 1) ? v >> 16 : v & 0xFFFFu;
}

// Rows whose length is a multiple of 8: groups of 8 columns, one Philox call
// each, kEach of them per thread at a time.
template <bool kBf16, bool kResidual, int kEach>
__global__ void __launch_bounds__(256) dropout_kernel(const __grid_constant__ DropoutParams p) {
  const RngKey key = rng_key(p.rng, p.site);
  const uint32_t step = gridDim.x * (256u * kEach);
  for (uint32_t i0 = blockIdx.x * (256u * kEach) + threadIdx.x; i0 < p.total; i0 += step) {
    float x[kEach][8], r[kEach][8];
    uint32_t row[kEach], g[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint32_t i = i0 + 256u * e;
      const long long at = static_cast<long long>(i) * 8;
      if (i < p.total) {
        load8t<kBf16>(p.x, at, x[e]);
        if (kResidual) load8t<kBf16>(p.residual, at, r[e]);
      }
      row[e] = static_cast<uint32_t>(fdiv(static_cast<int>(i), p.fd_groups));
      g[e] = i - row[e] * static_cast<uint32_t>(p.groups);
    }
    uint4 u[kEach];
    philox8n<kEach>(key, kRngDropout, row, g, u);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint32_t i = i0 + 256u * e;
      if (i >= p.total) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[e][j] = dropped(x[e][j], half_of(u[e], j), p.threshold, p.scale);
        if (kResidual) x[e][j] += r[e][j];
      }
      store8t<kBf16>(p.out, static_cast<long long>(i) * 8, x[e]);
    }
  }
}

// Other row lengths, from 16 on: the buffers are contiguous, so a thread still
// takes eight elements of the flat array with 16-byte accesses. They begin
// anywhere in a row: their numbers are those of the group they begin in, which
// this thread forms, and of the next one, which the next thread forms. Where a
// row ends among the eight, the next thread's group is the next row's first.
// Twice the instructions of the aligned form: 32768 x 2559 bf16 98 us at 72 % of
// the issue slots, 2560 columns 60-63.
template <bool kBf16, bool kResidual>
__global__ void __launch_bounds__(256) dropout_flat_kernel(const __grid_constant__ DropoutParams p, uint32_t n) {
  __shared__ uint4 numbers[257];
  const RngKey key = rng_key(p.rng, p.site);
  const uint16_t* u = reinterpret_cast<const uint16_t*>(numbers);
  const uint32_t step = gridDim.x * 2048u;
  for (uint32_t base = blockIdx.x * 2048u; base < n; base += step) {
    const uint32_t at = base + threadIdx.x * 8u;
    const int row = fdiv(static_cast<int>(at), p.fd_cols);
    const int col = static_cast<int>(at) - row * p.cols;
    float x[8], r[8];
    const bool whole = at + 8 <= n;
    if (whole) {
      load8t<kBf16>(p.x, at, x);
      if (kResidual) load8t<kBf16>(p.residual, at, r);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = at + j < n ? load1t<kBf16>(p.x, at + j) : 0.0f;
        if (kResidual) r[j] = at + j < n ? load1t<kBf16>(p.residual, at + j) : 0.0f;
      }
    }
    numbers[threadIdx.x] = philox8(key, kRngDropout, static_cast<uint32_t>(row), static_cast<uint32_t>(col >> 3));
    if (threadIdx.x == 255) {   // the group of the first element behind this block's
      const bool wraps = col + 8 >= p.cols;
      numbers[256] = philox8(key, kRngDropout, static_cast<uint32_t>(wraps ? row + 1 : row),
                             static_cast<uint32_t>((wraps ? col + 8 - p.cols : col + 8) >> 3));
    }
    __syncthreads();
    const int left = p.cols - col;            // elements up to the row's end
    const int first = col & 7;                // of the own group
    uint4 tail = make_uint4(0u, 0u, 0u, 0u);  // the row's last group, where it is neither of the two
    const bool extra = left <= 8 && first + left > 8;
    if (extra)
      tail = philox8(key, kRngDropout, static_cast<uint32_t>(row), static_cast<uint32_t>((col >> 3) + 1));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t k;
      if (j >= left)
        k = u[(threadIdx.x + 1) * 8 + j - left];
      else if (extra && first + j >= 8)
        k = half_of(tail, first + j - 8);
      else
        k = u[threadIdx.x * 8 + first + j];
      x[j] = dropped(x[j], k, p.threshold, p.scale);
      if (kResidual) x[j] += r[j];
    }
    if (whole) {
      store8t<kBf16>(p.out, at, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < n) store1t<kBf16>(p.out, at + j, x[j]);
    }
    __syncthreads();
  }
}

// Any row length and size, element by element: a warp takes 32 groups, forms
// their numbers, and passes them through shared memory so that neighbouring
// lanes handle neighbouring elements.
template <bool kBf16, bool kResidual>
__global__ void __launch_bounds__(256) dropout_ragged_kernel(const __grid_constant__ DropoutParams p) {
  __shared__ uint4 numbers[8][32];
  const RngKey key = rng_key(p.rng, p.site);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t step = gridDim.x * 256u;
  for (uint32_t base = blockIdx.x * 256u + warp * 32u; base < p.total; base += step) {
    const uint32_t i = base + lane;
    long long at = 0;   // this lane's group: first element, and how many there are
    int len = 0;
    if (i < p.total) {
      const int row = fdiv(static_cast<int>(i), p.fd_groups);
      const int g = static_cast<int>(i) - row * p.groups;
      at = static_cast<long long>(row) * p.cols + g * 8;
      len = min(8, p.cols - g * 8);
      numbers[warp][lane] = philox8(key, kRngDropout, static_cast<uint32_t>(row), static_cast<uint32_t>(g));
    }
    __syncwarp();
    const uint16_t* u = reinterpret_cast<const uint16_t*>(numbers[warp]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int owner = t * 4 + (lane >> 3), j = lane & 7;
      const long long e = __shfl_sync(0xffffffffu, at, owner) + j;
      if (j < __shfl_sync(0xffffffffu, len, owner)) {
        float x = dropped(load1t<kBf16>(p.x, e), u[owner * 8 + j], p.threshold, p.scale);
        if (kResidual) x += load1t<kBf16>(p.residual, e);
        store1t<kBf16>(p.out, e, x);
      }
    }
    __syncwarp();
  }
}

template <bool kBf16, bool kResidual>
static cudaError_t launch_typed(const DropoutParams& p, int sms, cudaStream_t s) {
  const uint32_t want = (p.total + 255) / 256, most = 32u * static_cast<uint32_t>(sms);
  const uint32_t grid = want < most ? want : most;
  const long long n = p.rows * p.cols;
  if (p.cols % 8 == 0) {
    // Large bf16 tensors without a residual move so few bytes per number that
    // the Philox chains' latency shows: two groups per thread (32768 x 2560:
    // 57 against 60-66 us). With a residual one group is faster (77 against
    // 87 us), in fp32 and for small tensors two change little or nothing.
    constexpr int kEach = kBf16 && !kResidual ? 2 : 1;
    if (kEach == 2 && want >= 32u * static_cast<uint32_t>(sms)) {
      const uint32_t half = (p.total + 511) / 512;
      dropout_kernel<kBf16, kResidual, kEach><<<half < most ? half : most, 256, 0, s>>>(p);
    } else {
      dropout_kernel<kBf16, kResidual, 1><<<grid, 256, 0, s>>>(p);
    }
  } else if (p.cols >= 16 && n < (1LL << 31) - 4096) {   // 32-bit flat indices
    const uint32_t blocks = static_cast<uint32_t>((n + 2047) / 2048);
    dropout_flat_kernel<kBf16, kResidual><<<blocks < most ? blocks : most, 256, 0, s>>>(p, static_cast<uint32_t>(n));
  } else {
    dropout_ragged_kernel<kBf16, kResidual><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_dropout(const DropoutParams& p, bool bf16, int sms, cudaStream_t s) {
  if (bf16) return p.residual ? launch_typed<true, true>(p, sms, s) : launch_typed<true, false>(p, sms, s);
  return p.residual ? launch_typed<false, true>(p, sms, s) : launch_typed<false, false>(p, sms, s);
}

}  // namespace muon
