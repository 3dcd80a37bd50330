// Product of two MXFP4 matrices on sm_100a tensor cores (tcgen05 kind::mxf4,
// block-scaled): out[m][n] = [add +] sum_k A[m][k] B[n][k], fp32 accumulation
// in TMEM and one rounding at the end.
//
// Both kernels stage 256 elements of K at a time: 128-byte rows of codes
// (TMA, 128-byte swizzle) and 512-byte scale tiles, which the MMA issuer
// copies to TMEM (tcgen05.cp) right before the stage's four K = 64 MMAs.
//
// pair kernel: clusters of 2 CTAs compute 256 x 256 tiles with the 2-SM MMA,
// persistent over the tiles. Two 256-column accumulators and the scales do
// not fit the 512 TMEM columns side by side, so the accumulators overlap by
// 48 columns (0..255 and 208..463; scales above): the epilogue drains the
// shared columns of a tile first, and the next tile's MMAs start as soon as
// it has. Products with few tiles and a long K are split along K into fp32
// partial tiles, which a second kernel adds in split order (deterministic).
//
// few-row kernel: for products with at most 128 rows on one side. The other
// operand, usually the weights, takes the MMA's 128-row side and is streamed
// once; the K range of a tile is split over the CTAs of a cluster, which add
// their partial tiles through distributed shared memory in rank order.
//
// Every wait is bounded (muon::mbar_wait*); a wait that ran out sets the
// workspace's status word, and what was not computed is not written.
#include "dtype_io.cuh"
#include "mxfp4_gemm.cuh"
#include "ptx_mxf4.cuh"

namespace muon {

namespace {

constexpr int kKBytes = 128;                       // bytes of a row per stage (256 elements)
constexpr int kRows = 128;                         // operand rows per CTA and stage
constexpr int kCodeBytes = kRows * kKBytes;        // 16 KB
constexpr int kSfGroupBytes = 2 * kMxTileBytes;    // scales of 128 rows and 256 K
constexpr int kMxEpiWarps = 8;
constexpr int kMxThreads = 64 + 32 * kMxEpiWarps;

// pair kernel
constexpr int kPTile = 256;
constexpr int kPStages = 6;
constexpr int kPStageBytes = 2 * kCodeBytes + 3 * kSfGroupBytes;  // A, B half; A's 128 rows, B's 256
constexpr int kPSmemBytes = kPStages * kPStageBytes + 1024 + 256;
constexpr uint32_t kAccOffset = 208;               // first column of the second accumulator
constexpr uint32_t kSfColumn = 464;                // two buffers of 24 columns
constexpr uint32_t kSfBuf = 24;

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint32_t addr = smem_u32(bar);
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(addr, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return;
  }
}

struct MxTile {
  int c, im, in, split, kb0, nkb;
};

// Tiles run down `group` row tiles before the next column tile, so that the
// CTAs at work at one time share operand rows in L2.
__device__ __forceinline__ MxTile mx_tile(const MxGemmParams& p, int t) {
  MxTile x;
  const int per_mat = p.tm * p.tn;
  x.split = t % p.split;
  t /= p.split;
  x.c = t / per_mat;
  t -= x.c * per_mat;
  const int band = t / (p.group * p.tn);
  const int first = band * p.group;
  const int height = min(p.group, p.tm - first);
  t -= first * p.tn;
  x.in = t / height;
  x.im = first + t - x.in * height;
  x.kb0 = x.split * p.kc;
  x.nkb = min(p.kc, p.kstages - x.kb0);
  return x;
}

// n consecutive outputs of one row, from column `col` on (cols exist up to p.n).
template <bool kBf16>
__device__ __forceinline__ void store_row32(const MxGemmParams& p, long long base, int col, bool vec,
                                            const uint32_t (&r)[32]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int c = col + 8 * g;
    if (vec && c + 8 <= p.n) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[8 * g + j]);
      if (p.add) {
        float a[8];
        load8t<kBf16>(p.add, base + c, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += a[j];
      }
      store8t<kBf16>(p.out, base + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (c + j < p.n) {
          float v = __uint_as_float(r[8 * g + j]);
          if (p.add) v += load1t<kBf16>(p.add, base + c + j);
          store1t<kBf16>(p.out, base + c + j, v);
        }
      }
    }
  }
}

}  // namespace

// ------------------------------------------------------------------ pair kernel
template <bool kBf16, bool kSplit>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMxThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ MxGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPStages * kPStageBytes);
  uint64_t* empty = full + kPStages;
  uint64_t* tfull = empty + kPStages;     // one per accumulator
  uint64_t* tnext = tfull + 2;            // the next tile's accumulator is free
  uint64_t* done = tnext + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.wait_limit_ns;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);
  const int ntiles = p.count * p.tm * p.tn * p.split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&tfull[0], 1);
    mbar_init(&tfull[1], 1);
    mbar_init(tnext, 2 * kMxEpiWarps);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&p.rows_l);
    tma_prefetch_map(&p.rows_r);
    tma_prefetch_map(&p.scales_l);
    tma_prefetch_map(&p.scales_r);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      int stage = 0;
      uint32_t phase = 0;
      int issued[kPStages];
      for (int s = 0; s < kPStages; ++s) issued[s] = -1;
      bool ok = true;
      for (int t = pair; ok && t < ntiles; t += npairs) {
        const MxTile T = mx_tile(p, t);
        const int cl = p.share_l ? 0 : T.c, cr = p.share_r ? 0 : T.c;
        const int lrow = T.im * kPTile + kRows * static_cast<int>(rank);
        const int rrow = T.in * kPTile + kRows * static_cast<int>(rank);
        const int ltile = cl * p.tiles_l + 2 * T.im + static_cast<int>(rank);
        const int rtile = cr * p.tiles_r + 2 * T.in;
        for (int kb = 0; kb < T.nkb; ++kb) {
          if (!mbar_wait_cluster(&empty[stage], phase ^ 1u, abort_flag, p.status, limit)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + stage * kPStageBytes;
          const uint32_t bar = full_leader + 8u * static_cast<uint32_t>(stage);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kPStageBytes);
          const int k = T.kb0 + kb;
          tma_load_3d_pair(st, &p.rows_l, bar, k * kKBytes, lrow, cl);
          tma_load_3d_pair(st + kCodeBytes, &p.rows_r, bar, k * kKBytes, rrow, cr);
          tma_load_2d_pair(st + 2 * kCodeBytes, &p.scales_l, bar, k * 256, ltile);
          tma_load_2d_pair(st + 2 * kCodeBytes + kSfGroupBytes, &p.scales_r, bar, k * 256, rtile);
          issued[stage] = static_cast<int>(phase);
          if (++stage == kPStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (rank == 0)
        for (int s = 0; s < kPStages; ++s)
          if (issued[s] >= 0) drain(&full[s], static_cast<uint32_t>(issued[s]), limit);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      if (rank == 0) {
        // -------------------------------------------------- MMA issuer (leader)
        int stage = 0, old_stage = kPStages - 2;   // old_stage: the one used two stages ago
        uint32_t phase = 0, old_phase = 1, uses = 0;
        uint32_t acc = 0, tfree = 0;
        bool ok = true, first = true;
        for (int t = pair; ok && t < ntiles; t += npairs) {
          const MxTile T = mx_tile(p, t);
          if (!first) {
            if (!mbar_wait_cluster(tnext, tfree, abort_flag, p.status, limit)) {
              ok = false;
              break;
            }
            tfree ^= 1u;
          }
          first = false;
          tc_fence_after();
          const uint32_t d = tmem_base + acc * kAccOffset;
          for (int kb = 0; kb < T.nkb; ++kb) {
            // the scale buffer is free once the MMAs of two stages ago are done
            if ((uses >= 2 && !mbar_wait_cluster(&empty[old_stage], old_phase, abort_flag, p.status, limit)) ||
                !mbar_wait_cluster(&full[stage], phase, abort_flag, p.status, limit)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a = smem_u32(smem + stage * kPStageBytes);
            const uint32_t b = a + kCodeBytes, sa = b + kCodeBytes, sb = sa + kSfGroupBytes;
            const uint32_t sfa = tmem_base + kSfColumn + (uses & 1u) * kSfBuf, sfb = sfa + 8;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              tmem_copy_scales_pair(sfa + 4 * g, smem_desc_scales(sa + g * kMxTileBytes));
              tmem_copy_scales_pair(sfb + 8 * g, smem_desc_scales(sb + g * kMxTileBytes));
              tmem_copy_scales_pair(sfb + 8 * g + 4, smem_desc_scales(sb + kSfGroupBytes + g * kMxTileBytes));
            }
            const int steps = min(4, p.k64 - 4 * (T.kb0 + kb));
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              if (ks < steps)
                umma_mxf4_pair(d, smem_desc_sw128(a + ks * 32, 16, 1024), smem_desc_sw128(b + ks * 32, 16, 1024),
                               idesc_mxf4(kPTile, kPTile, 2 * (ks & 1)), sfa + 4 * (ks >> 1), sfb + 8 * (ks >> 1),
                               (kb > 0 || ks > 0) ? 1u : 0u);
            }
            umma_commit_pair(&empty[stage]);
            ++uses;
            if (++stage == kPStages) { stage = 0; phase ^= 1u; }
            if (++old_stage == kPStages) { old_stage = 0; old_phase ^= 1u; }
          }
          if (!ok) break;
          umma_commit_pair(&tfull[acc]);
          acc ^= 1u;
        }
        umma_commit_pair(done);
      }
      drain(done, 0, limit);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // warp w reads TMEM lanes 32 (w % 4) ..; warps 2..5 the accumulator's
    // columns 0..127, warps 6..9 columns 128..255, 32 at a time, the columns
    // that the next tile's accumulator overlaps first.
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tnext_leader = mapa_shared(smem_u32(tnext), 0);
    const bool vec = (p.n % 8) == 0;
    uint32_t acc = 0, phase = 0;
    bool ok = true;
    for (int t = pair; ok && t < ntiles; t += npairs) {
      const MxTile T = mx_tile(p, t);
      const bool overlapped = (acc == 0) == (half == 1);
      if (!overlapped) {  // this warp holds nothing the next tile's MMAs would overwrite
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_cta(tnext_leader);
      }
      const bool got = mbar_wait_cluster(&tfull[acc], phase, abort_flag, p.status, limit);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * kAccOffset + half * 128;
      const int row = T.im * kPTile + kRows * static_cast<int>(rank) + 32 * q + lane;
      const int col = T.in * kPTile + half * 128;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int j = acc == 0 ? 3 - i : i;
        uint32_t r[32];
        tmem_ld32(tb + j * 32, r);
        tmem_ld_wait();
        if (overlapped && i == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_cta(tnext_leader);
        }
        if (kSplit) {
          // partial tile: the 32 x 32 chunk as 8 rows of 32 float4, one per lane
          float4* dst = reinterpret_cast<float4*>(
              p.part + static_cast<long long>(t) * (kPTile * kPTile) +
              ((((rank * 4 + q) * 2 + half) * 4 + j) * 1024));
#pragma unroll
          for (int g = 0; g < 8; ++g)
            dst[g * 32 + lane] = make_float4(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1]),
                                             __uint_as_float(r[4 * g + 2]), __uint_as_float(r[4 * g + 3]));
        } else if (row < p.m) {
          const long long base = T.c * p.stride_c + static_cast<long long>(row) * p.n;
          store_row32<kBf16>(p, base, col + j * 32, vec, r);
        }
      }
      acc ^= 1u;
      if (acc == 0) phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// Adds the partial tiles of a split product in split order. One warp per
// 32 x 32 chunk, turned through shared memory so that rows are stored whole.
template <bool kBf16>
__global__ void __launch_bounds__(256) mx_reduce_kernel(const __grid_constant__ MxGemmParams p) {
  __shared__ float turn[8][32][33];
  if (*reinterpret_cast<const volatile int*>(p.status) != 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunk = static_cast<int>(blockIdx.x & 7u) * 8 + warp;  // 64 chunks per tile, eight blocks
  const int tile = static_cast<int>(blockIdx.x >> 3);
  const MxTile T = mx_tile(p, tile * p.split);
  const int j = chunk & 3, half = (chunk >> 2) & 1, q = (chunk >> 3) & 3, rank = chunk >> 5;
  const int row0 = T.im * kPTile + kRows * rank + 32 * q, col = T.in * kPTile + half * 128 + j * 32 + lane;
  float4 acc[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < p.split; ++s) {
    const float4* src = reinterpret_cast<const float4*>(
        p.part + (static_cast<long long>(tile) * p.split + s) * (kPTile * kPTile) + chunk * 1024);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const float4 v = src[g * 32 + lane];
      acc[g].x += v.x; acc[g].y += v.y; acc[g].z += v.z; acc[g].w += v.w;
    }
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    turn[warp][lane][4 * g] = acc[g].x;
    turn[warp][lane][4 * g + 1] = acc[g].y;
    turn[warp][lane][4 * g + 2] = acc[g].z;
    turn[warp][lane][4 * g + 3] = acc[g].w;
  }
  __syncwarp();
  if (col >= p.n) return;
  for (int i = 0; i < 32 && row0 + i < p.m; ++i) {
    const long long at = T.c * p.stride_c + static_cast<long long>(row0 + i) * p.n + col;
    float v = turn[warp][i][lane];
    if (p.add) v += load1t<kBf16>(p.add, at);
    store1t<kBf16>(p.out, at, v);
  }
}

// -------------------------------------------------------------- few-row kernel
// One tile of 128 left rows x NT right rows per cluster; CTA r of the cluster
// takes K stages r * kc .. and the cluster adds the parts. 192 threads: warp 0
// loads, warp 1 issues the MMAs, warps 2..5 are the epilogue.
constexpr int kFewThreads = 192;

template <int NT>
__host__ __device__ constexpr int few_stage_bytes() { return kCodeBytes + NT * kKBytes + 2 * kSfGroupBytes; }

template <int NT>
__host__ __device__ constexpr uint32_t few_tmem_columns() { return NT + 16 <= 32 ? 32 : NT + 16 <= 64 ? 64 : NT + 16 <= 128 ? 128 : 256; }

template <int NT, bool kBf16>
__global__ void __launch_bounds__(kFewThreads) mx_gemm_few_kernel(const __grid_constant__ MxGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[16], empty[16], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  constexpr int kStage = few_stage_bytes<NT>();
  constexpr uint32_t kCols = few_tmem_columns<NT>();
  constexpr uint32_t kSf = NT;               // 8 columns for the left scales, 8 for the right
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.wait_limit_ns;
  volatile int* abort_flag = &abort_word;
  const int split = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int c = tile / p.tm, im = tile - c * p.tm;
  const int kb0 = split * p.kc, nkb = min(p.kc, p.kstages - kb0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const int cl = p.share_l ? 0 : c, cr = p.share_r ? 0 : c;
      int stage = 0;
      uint32_t phase = 0;
      int sent = 0;
      for (int kb = 0; kb < nkb; ++kb, ++sent) {
        if (kb >= p.ring && !mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, limit)) break;
        uint8_t* st = smem + stage * kStage;
        const int k = kb0 + kb;
        mbar_arrive_expect_tx(&full[stage], kStage);
        tma_load_3d(st, &p.rows_l, &full[stage], k * kKBytes, im * kRows, cl);
        tma_load_3d(st + kCodeBytes, &p.rows_r, &full[stage], k * kKBytes, 0, cr);
        tma_load_2d(st + kCodeBytes + NT * kKBytes, &p.scales_l, &full[stage], k * 256, cl * p.tiles_l + im);
        tma_load_2d(st + kCodeBytes + NT * kKBytes + kSfGroupBytes, &p.scales_r, &full[stage], k * 256,
                    cr * p.tiles_r);
        if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      }
      // every load has landed before shared memory is reused or released
      for (int kb = sent > p.ring ? sent - p.ring : 0; kb < sent; ++kb)
        drain(&full[kb % p.ring], static_cast<uint32_t>(kb / p.ring) & 1u, limit);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait(&full[stage], phase, abort_flag, p.status, limit)) break;
        if (kb > 0) {  // one scale buffer: the MMAs of the stage before are done
          const int before = kb - 1;
          if (!mbar_wait(&empty[before % p.ring], static_cast<uint32_t>(before / p.ring) & 1u, abort_flag,
                         p.status, limit))
            break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + stage * kStage);
        const uint32_t b = a + kCodeBytes, sa = b + NT * kKBytes, sb = sa + kSfGroupBytes;
        const uint32_t sfa = tmem_base + kSf, sfb = sfa + 8;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          tmem_copy_scales(sfa + 4 * g, smem_desc_scales(sa + g * kMxTileBytes));
          tmem_copy_scales(sfb + 4 * g, smem_desc_scales(sb + g * kMxTileBytes));
        }
        const int steps = min(4, p.k64 - 4 * (kb0 + kb));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          if (ks < steps)
            umma_mxf4(tmem_base, smem_desc_sw128(a + ks * 32, 16, 1024), smem_desc_sw128(b + ks * 32, 16, 1024),
                      idesc_mxf4(kRows, NT, 2 * (ks & 1)), sfa + 4 * (ks >> 1), sfb + 4 * (ks >> 1),
                      (kb > 0 || ks > 0) ? 1u : 0u);
        }
        umma_commit(&empty[stage]);
        if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      }
      umma_commit(&done);
    }
    __syncwarp();
  }
  // every warp waits: the parts are exchanged through the loads' shared memory
  ok = mbar_wait(&done, 0, abort_flag, p.status, limit);
  if (!ok) drain(&done, 0, limit);
  ok = __syncthreads_and(ok && *abort_flag == 0);
  tc_fence_after();

  // element (left row i, right row x) of this CTA's part, as [x][i]
  float* mine = reinterpret_cast<float*>(smem);
  const int q = warp & 3;
  if (p.split == 1) {
    if (ok && warp >= 2) {
      const int l = im * kRows + 32 * q + lane;
#pragma unroll 1
      for (int x0 = 0; x0 < NT; x0 += 8) {
        if (x0 >= p.n) break;
        uint32_t r[8];
        tmem_ld8(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + x0, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (l < p.m && x0 + j < p.n) {
            const long long at = c * p.stride_c + l * p.stride_l + (x0 + j) * p.stride_r;
            float v = __uint_as_float(r[j]);
            if (p.add) v += load1t<kBf16>(p.add, at);
            store1t<kBf16>(p.out, at, v);
          }
        }
      }
    }
  } else {
    if (warp >= 2) {
#pragma unroll 1
      for (int x0 = 0; x0 < NT; x0 += 8) {
        uint32_t r[8];
        tmem_ld8(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + x0, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) mine[(x0 + j) * kRows + 32 * q + lane] = __uint_as_float(r[j]);
      }
    }
    // a part that failed poisons the status word; nothing of the tile is stored then
    __shared__ int cluster_ok;
    if (threadIdx.x == 0) cluster_ok = ok ? 1 : 0;
    __syncthreads();
    cluster_sync();
    bool all_ok = true;
    for (int s = 0; s < p.split; ++s)
      all_ok = all_ok && __float_as_int(ld_shared_cluster(mapa_shared(smem_u32(&cluster_ok), s))) != 0;
    if (all_ok) {
      const int per = (NT * kRows + p.split - 1) / p.split;
      const int e1 = min((split + 1) * per, NT * kRows);
      for (int e = split * per + static_cast<int>(threadIdx.x); e < e1; e += kFewThreads) {
        const int x = e >> 7, l = im * kRows + (e & 127);
        if (x >= p.n) break;
        if (l >= p.m) continue;
        float v = 0.0f;
        for (int s = 0; s < p.split; ++s) v += ld_shared_cluster(mapa_shared(smem_u32(mine + e), s));
        const long long at = c * p.stride_c + l * p.stride_l + x * p.stride_r;
        if (p.add) v += load1t<kBf16>(p.add, at);
        store1t<kBf16>(p.out, at, v);
      }
    }
    cluster_sync();   // the others have read this CTA's part
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kCols);
  }
}

// ------------------------------------------------------------------- launches
MxGemmPlan plan_mx_gemm(const MxGemmShape& s, int pairs, int sms) {
  MxGemmPlan pl{};
  const int kstages = static_cast<int>((s.k + 255) / 256);
  const int64_t small = s.m < s.n ? s.m : s.n, large = s.m < s.n ? s.n : s.m;
  if (small <= kRows) {
    pl.few = true;
    pl.swap = s.m <= s.n;  // the left operand of the kernel is the one with many rows
    pl.nt = small <= 16 ? 16 : small <= 32 ? 32 : small <= 64 ? 64 : 128;
    pl.tm = static_cast<int>((large + kRows - 1) / kRows);
    pl.tn = 1;
    // split K over the CTAs of a cluster (a power of two, up to 8) while that
    // still adds CTAs the device has room for
    pl.split = 1;
    while (pl.split < 8 && pl.split * 2 <= kstages && s.count * pl.tm * pl.split * 2 <= 2 * sms) pl.split *= 2;
    pl.kc = (kstages + pl.split - 1) / pl.split;
    while (pl.split > 1 && pl.kc * (pl.split - 1) >= kstages) {  // no empty part
      pl.split /= 2;
      pl.kc = (kstages + pl.split - 1) / pl.split;
    }
    const int cap = pl.nt <= 32 ? 5 : 4;
    pl.ring = pl.kc < cap ? pl.kc : cap;
    return pl;
  }
  pl.tm = static_cast<int>((s.m + kPTile - 1) / kPTile);
  pl.tn = static_cast<int>((s.n + kPTile - 1) / kPTile);
  const int64_t tiles = s.count * pl.tm * pl.tn;
  pl.split = 1;
  if (tiles * 2 <= pairs) {
    int64_t sp = pairs / tiles;
    if (sp > kstages / 4) sp = kstages / 4;  // at least four stages each
    if (sp > 16) sp = 16;
    if (sp > 1) pl.split = static_cast<int>(sp);
  }
  pl.kc = (kstages + pl.split - 1) / pl.split;
  pl.split = (kstages + pl.kc - 1) / pl.kc;
  if (pl.split > 1) pl.part_bytes = static_cast<size_t>(tiles) * pl.split * kPTile * kPTile * 4;
  return pl;
}

static const void* pair_kernel(bool bf16, bool split) {
  if (split) return reinterpret_cast<const void*>(&mx_gemm_pair_kernel<false, true>);
  return bf16 ? reinterpret_cast<const void*>(&mx_gemm_pair_kernel<true, false>)
              : reinterpret_cast<const void*>(&mx_gemm_pair_kernel<false, false>);
}

template <int NT>
static const void* few_kernel_nt(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&mx_gemm_few_kernel<NT, true>)
              : reinterpret_cast<const void*>(&mx_gemm_few_kernel<NT, false>);
}

static const void* few_kernel(int nt, bool bf16) {
  return nt == 16 ? few_kernel_nt<16>(bf16)
                  : nt == 32 ? few_kernel_nt<32>(bf16) : nt == 64 ? few_kernel_nt<64>(bf16) : few_kernel_nt<128>(bf16);
}

// Shared memory of the few-row kernel: the ring, which later holds the part.
static int few_smem(const MxGemmPlan& pl) {
  const int stage = kCodeBytes + pl.nt * kKBytes + 2 * kSfGroupBytes;
  int bytes = pl.ring * stage;
  const int part = pl.split > 1 ? pl.nt * kRows * 4 : 0;
  if (part > bytes) bytes = part;
  return bytes + 1024;
}

cudaError_t mx_gemm_prepare(int* max_pairs) {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 3 && e == cudaSuccess; ++i)
    e = cudaFuncSetAttribute(pair_kernel(i & 1, i & 2), cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmemBytes);
  for (int nt = 16; nt <= 128; nt *= 2)
    for (int b = 0; b < 2 && e == cudaSuccess; ++b)
      e = cudaFuncSetAttribute(few_kernel(nt, b), cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  *max_pairs = sms / 2;
  return cudaSuccess;
}

cudaError_t launch_mx_gemm(const MxGemmParams& p, const MxGemmPlan& plan, bool bf16, int max_pairs,
                           int sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {const_cast<MxGemmParams*>(&p)};
  if (plan.few) {
    attr[0].val.clusterDim.x = plan.split;
    cfg.gridDim = dim3(static_cast<unsigned>(p.count) * plan.tm * plan.split, 1, 1);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = few_smem(plan);
    return cudaLaunchKernelExC(&cfg, few_kernel(plan.nt, bf16), args);
  }
  const int64_t tiles = static_cast<int64_t>(p.count) * plan.tm * plan.tn;
  int pairs = max_pairs;
  if (tiles * plan.split < pairs) pairs = static_cast<int>(tiles * plan.split);
  cfg.numAttrs = 0;   // the cluster shape is the kernel's own
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(kMxThreads, 1, 1);
  cfg.dynamicSmemBytes = kPSmemBytes;
  cudaError_t e = cudaLaunchKernelExC(&cfg, pair_kernel(bf16, plan.split > 1), args);
  if (e != cudaSuccess || plan.split == 1) return e;
  const unsigned blocks = static_cast<unsigned>(tiles) * 8u;
  if (bf16)
    mx_reduce_kernel<true><<<blocks, 256, 0, s>>>(p);
  else
    mx_reduce_kernel<false><<<blocks, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace muon
