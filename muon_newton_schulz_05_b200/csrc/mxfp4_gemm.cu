// Product of two MXFP4 matrices on sm_100a tensor cores (tcgen05 kind::mxf4,
// block-scaled): out[m][n] = [add +] sum_k A[m][k] B[n][k], fp32 accumulation
// in TMEM and one rounding at the end.
//
// Both kernels stage 256 elements of K at a time: 128-byte rows of codes
// (TMA, 128-byte swizzle) and 512-byte scale tiles, which go on to TMEM.
//
// pair kernel: clusters of 2 CTAs compute 256 x 256 tiles with the 2-SM MMA,
// persistent over the tiles. Four warps per CTA move the scales from shared
// memory to TMEM (tcgen05.st), up to four stages ahead of the MMAs. (Copies
// issued by the MMA thread, tcgen05.cp, take their turn in the tensor pipe:
// the six of a stage cost it about 170 ns of 610, whether issued right before
// the stage's MMAs or a stage ahead.)
// Two 256-column accumulators and four scale buffers do not fit the 512 TMEM
// columns side by side, so the accumulators overlap by 96 columns (0..255 and
// 160..415; scales above): the epilogue drains the shared columns of a tile
// first, and the next tile's MMAs start as soon as it has. 16384 x 10240 x 2560
// takes 164-171 us in bursts of up to 50 ms (5.2 PFLOP/s) and 194-197 under
// lasting load, when the board's power cap holds the clock at 1.2 GHz; K 8192
// 448-468 (6.1) and 536-550. The tensor pipe is busy for 58 % of the cycles at
// K 2560 and 79 % at K 8192; a tile costs 2600-2900 cycles without MMAs.
// Products with few tiles and a long K are split along K into fp32 partial
// tiles, which a second kernel adds in split order (deterministic).
//
// few-row kernel: for products with at most 64 rows on one side. The other
// operand, usually the weights, takes the MMA's 128-row side and is streamed
// once; the K range of a tile is split over the CTAs of a cluster, which add
// their partial tiles through distributed shared memory in rank order.
//
// Every wait for a barrier in shared memory is bounded (muon::mbar_wait*); a
// wait that ran out sets the workspace's status word, and what was not computed
// is not written. Two waits have no limit of their own: the cluster barrier,
// which every CTA comes to after bounded waits only, and the TMEM allocation,
// which waits while other CTAs of the SM hold the columns. A CTA that holds
// columns may therefore wait for nothing that another CTA's allocation has to
// come before: the few-row kernel, several of whose CTAs share an SM (more than
// the 512 columns serve, where K is short), frees its columns before it waits
// for its cluster. A pair kernel's CTA has its SM to itself (shared memory).
#include <type_traits>

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
constexpr int kMxScaleWarps = 4;
constexpr int kMxThreads = 96 + 32 * (kMxEpiWarps + kMxScaleWarps);

// pair kernel
constexpr int kPTile = 256;
constexpr int kPStages = 5;                        // 4 where the epilogue loads addends by TMA and takes the rest
constexpr int kPStageBytes = 2 * kCodeBytes;
constexpr int kSfSlots = 8;                        // the scales' own ring
constexpr int kPScaleBytes = 3 * kSfGroupBytes;    // A's 128 rows, B's 256
constexpr int kPChunkBytes = 32 * 128;             // an epilogue warp's buffer: 32 rows of 128 bytes
constexpr int kPSmemBytes =
    kPStages * kPStageBytes + kSfSlots * kPScaleBytes + kMxEpiWarps * kPChunkBytes + 1024 + 512;
static_assert(kMxEpiWarps * kPChunkBytes <= kPStageBytes, "a second buffer per epilogue warp in place of a stage");
constexpr uint32_t kAccOffset = 160;               // first column of the second accumulator
constexpr int kSfBufs = 4;
constexpr uint32_t kSfBuf = 24;                    // A: 8 columns, B: 16
constexpr uint32_t kSfColumn = 512 - kSfBufs * kSfBuf;
constexpr int kOverlapChunks = 3;                  // 32-column chunks that the accumulators share
static_assert(kAccOffset + kPTile <= kSfColumn, "the second accumulator ends below the scales");
static_assert(kPTile - kAccOffset <= kOverlapChunks * 32, "the shared columns are drained first");

// Waits for what is in flight (copies, MMAs) and certain to come, before the
// memory it goes to is given up. A bound of its own: the limit of the other
// waits is the user's and may be what has just run out.
constexpr uint64_t kDrainNs = 10000000000ull;

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
  if (mbar_try_wait(addr, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(addr, parity)) {
    if (global_timer_ns() - t0 > kDrainNs) return;
  }
}

// What the roles of a CTA pair did before one of them gave up: stages whose
// loads the CTA's producer issued, and for which each scale warp arrived.
struct GaveUp {
  int issued;
  int scaled[kMxScaleWarps];
  int peer;   // the other CTA gave up
};

struct MxTile {
  int c, im, in, split, kb0, nkb;
};

// Tiles run down `group` row tiles before the next column tile, so that the
// CTAs at work at one time share operand rows in L2.
__device__ __forceinline__ MxTile mx_tile(const MxGemmParams& p, int t) {
  MxTile x;
  const int u = fdiv(t, p.fd_split);
  x.split = t - u * p.split;
  x.c = fdiv(u, p.fd_mat);
  t = u - x.c * (p.tm * p.tn);
  const int band = fdiv(t, p.fd_band);
  const int first = band * p.group;
  t -= first * p.tn;
  const bool whole = first + p.group <= p.tm;
  x.in = fdiv(t, whole ? p.fd_group : p.fd_rest);
  x.im = first + t - x.in * (whole ? p.group : p.tm - first);
  x.kb0 = x.split * p.kc;
  x.nkb = min(p.kc, p.kstages - x.kb0);
  return x;
}

// A warp's 32 x 64 bf16 results, two 32 x 32 chunks with one row per lane, into
// its buffer: rows of 128 bytes, 16-byte group g of row r at g ^ (r & 7) (TMA's
// 128-byte swizzle; conflict-free by rows and by columns). chunk a is half ha.
__device__ __forceinline__ void stage_bf16(uint8_t* buf, int lane, const uint32_t* a, int ha, const uint32_t* b) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t* r = c ? b : a;
    const int h = c ? 1 - ha : ha;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16x2(__uint_as_float(r[8 * g + 2 * i]), __uint_as_float(r[8 * g + 2 * i + 1]));
      *reinterpret_cast<uint4*>(buf + lane * 128 + (((4 * h + g) ^ (lane & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// The same results added to the addends that are in the buffer, each lane its
// own row in place (bf16: two chunks; fp32: one, whose rows are 128 bytes).
template <bool kBf16>
__device__ __forceinline__ void add_staged(uint8_t* buf, int lane, const uint32_t* a, int ha, const uint32_t* b) {
#pragma unroll
  for (int c = 0; c < (kBf16 ? 2 : 1); ++c) {
    const uint32_t* r = c ? b : a;
    const int h = kBf16 ? (c ? 1 - ha : ha) : 0;
#pragma unroll
    for (int g = 0; g < (kBf16 ? 4 : 8); ++g) {
      uint4* at = reinterpret_cast<uint4*>(buf + lane * 128 + (((4 * h + g) ^ (lane & 7)) << 4));
      const uint4 x = *at;
      const uint32_t xx[4] = {x.x, x.y, x.z, x.w};
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = kBf16 ? pack_bf16x2(__uint_as_float(r[8 * g + 2 * i]) + bf16_lo_f(xx[i]),
                                   __uint_as_float(r[8 * g + 2 * i + 1]) + bf16_hi_f(xx[i]))
                     : __float_as_uint(__uint_as_float(r[4 * g + i]) + __uint_as_float(xx[i]));
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// The pair of chunks by TMA: one store in bf16, two in fp32 (a chunk's rows are
// 128 bytes there).
template <bool kBf16>
__device__ __forceinline__ void store_pair_tma(const MxGemmParams& p, uint8_t* buf, int lane, const uint32_t* a,
                                               int ha, const uint32_t* b, int c, int row, int col) {
  const bool rows = row < p.m;
#pragma unroll
  for (int t = 0; t < (kBf16 ? 1 : 2); ++t) {
    const uint32_t* r = t ? b : a;
    const int at = kBf16 ? col : col + 32 * (t ? 1 - ha : ha);
    if (lane == 0) bulk_wait_read<0>();   // the store before has read the buffer
    __syncwarp();
    if (kBf16) {
      stage_bf16(buf, lane, a, ha, b);
    } else {
#pragma unroll
      for (int g = 0; g < 8; ++g)
        *reinterpret_cast<uint4*>(buf + lane * 128 + ((g ^ (lane & 7)) << 4)) =
            make_uint4(r[4 * g], r[4 * g + 1], r[4 * g + 2], r[4 * g + 3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && rows && at < p.n) {
      tma_store_3d(&p.result, buf, at, row, c);
      bulk_commit();
    }
  }
}

// A chunk for outputs that TMA cannot address, perhaps with an addend: turned in
// shared memory (16-byte group g of row r at g ^ (r & 7)) so that neighbouring
// lanes load and store neighbouring columns, four at a time where rows of bf16
// have a multiple of 4 elements (in fp32 those go by TMA). The addends of 16
// rows are on their way at once. (Rows that start anywhere: 4 x 1000 x 1537 x
// 771 takes 12.2-12.8 us, 1536 columns by TMA 9.1.)
template <bool kBf16, bool kAdd>
__device__ __forceinline__ void store_chunk(const MxGemmParams& p, uint8_t* buf, int lane, const uint32_t* r,
                                            long long base, int row, int col, bool vec) {
  __syncwarp();   // the previous chunk has been read
#pragma unroll
  for (int g = 0; g < 8; ++g)
    *reinterpret_cast<uint4*>(buf + lane * 128 + ((g ^ (lane & 7)) << 4)) =
        make_uint4(r[4 * g], r[4 * g + 1], r[4 * g + 2], r[4 * g + 3]);
  __syncwarp();
  const int rows = min(32, p.m - row);
  if (rows <= 0) return;
  if (kBf16 && vec) {   // 8 lanes per row, 4 columns each
    const int c = col + 4 * (lane & 7);
    if (c >= p.n) return;
    const long long at = base + static_cast<long long>(row) * p.n + c;
    uint2 add[8];
    if (kAdd) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        add[i] = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.add) + at +
                                                 static_cast<long long>(min(4 * i + (lane >> 3), rows - 1)) * p.n);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rr = 4 * i + (lane >> 3);
      float4 v = *reinterpret_cast<const float4*>(buf + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
      if (kAdd) {
        v.x += bf16_lo_f(add[i].x); v.y += bf16_hi_f(add[i].x); v.z += bf16_lo_f(add[i].y); v.w += bf16_hi_f(add[i].y);
      }
      if (rr < rows)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at + static_cast<long long>(rr) * p.n) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
  } else if (col + lane < p.n) {   // one column per lane
    using E = std::conditional_t<kBf16, __nv_bfloat16, float>;
    const long long at = base + static_cast<long long>(row) * p.n + col + lane;
    E* out = static_cast<E*>(p.out) + at;
    const E* add = static_cast<const E*>(p.add) + at;
    const uint8_t* src = buf + (lane & 3) * 4;
    const int g = lane >> 2;
    if (rows == 32) {   // no test per row; 16 at a time, 32 addends do not fit the registers
#pragma unroll 1
      for (int r0 = 0; r0 < 32; r0 += 16, src += 16 * 128) {
        float v[16];
        if (kAdd) {
#pragma unroll
          for (int i = 0; i < 16; ++i, add += p.n) v[i] = load1t<kBf16>(add, 0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i, out += p.n) {
          const float y = *reinterpret_cast<const float*>(src + i * 128 + ((g ^ (i & 7)) << 4));
          store1t<kBf16>(out, 0, kAdd ? v[i] + y : y);
        }
      }
    } else {
#pragma unroll 1
      for (int rr = 0; rr < rows; ++rr, out += p.n, add += p.n) {
        const float y = *reinterpret_cast<const float*>(src + rr * 128 + ((g ^ (rr & 7)) << 4));
        store1t<kBf16>(out, 0, kAdd ? load1t<kBf16>(add, 0) + y : y);
      }
    }
  }
}

// Brings the addends of a warp's 32 x 128 part of a tile (row per lane) to L2.
// Loaded from DRAM when the accumulator is there, chunk after chunk, they cost
// more than the rest of the tile.
template <bool kBf16>
__device__ __forceinline__ void prefetch_addends(const MxGemmParams& p, long long base, int row, int col) {
  constexpr int kLine = kBf16 ? 64 : 32;   // elements in 128 bytes
  const int end = min(col + 128, p.n);
  if (row >= p.m || col >= end) return;
  const long long at = base + static_cast<long long>(row) * p.n;
  for (int c = col; c < end; c += kLine) prefetch_l2(static_cast<const uint8_t*>(p.add) + (at + c) * (kBf16 ? 2 : 4));
  prefetch_l2(static_cast<const uint8_t*>(p.add) + (at + end - 1) * (kBf16 ? 2 : 4));
}

// Test hook: in fault modes 1 and 2 one loading thread of each of the first four
// pairs (codes or scales, of either CTA) stops before its first or its eighth
// stage, so that waits for what it would have loaded run out.
__device__ __forceinline__ bool withheld(const MxGemmParams& p, bool scales, int issued) {
  return p.fault != 0 && blockIdx.x < 8 && issued == (p.fault == 1 ? 0 : 7) &&
         (blockIdx.x & 1u) == ((blockIdx.x >> 1) & 1u) && scales == (blockIdx.x >= 4);
}

// After a wait of the pair ran out: lets the last use of each stage whose loads
// either CTA issued complete, and waits for it. The leader's barrier of a stage
// counts its producer's arrival, the bytes of both CTAs' loads and the scale
// warps of both; what will not come is put in its place. (An earlier use of the
// stage has completed: the loads of a use wait for the MMAs of the one before.)
// Called by one thread of the leader; no other role of the pair is at work.
template <int kStages>
__device__ __noinline__ void finish_stages(uint64_t* full, volatile GaveUp* record) {
  const uint32_t peer = mapa_shared(smem_u32(const_cast<GaveUp*>(record)), 1);
  const int issued0 = record->issued, issued1 = ld_cluster(peer);
  for (int s = 0; s < kStages; ++s) {
    // the last use of stage s among `issued` ones; -1 (or less): none
    const int u0 = issued0 > s ? issued0 - 1 - (issued0 - 1 - s) % kStages : -1;
    const int u1 = issued1 > s ? issued1 - 1 - (issued1 - 1 - s) % kStages : -1;
    const int u = max(u0, u1);
    if (u < 0) continue;
    const uint32_t parity = static_cast<uint32_t>(u / kStages) & 1u;
    if (mbar_test(smem_u32(&full[s]), parity)) continue;
    if (u0 < u) mbar_arrive_expect_tx(&full[s], 2 * kCodeBytes);   // the other CTA's loads alone
    if (u1 < u) mbar_complete_tx(&full[s], 2 * kCodeBytes);        // expected, never issued
    for (int w = 0; w < 2 * kMxScaleWarps; ++w) {
      const int scaled = w < kMxScaleWarps ? record->scaled[w] : ld_cluster(peer + 4u * (1 + w - kMxScaleWarps));
      if (scaled <= u) mbar_arrive(&full[s]);
    }
    drain(&full[s], parity);
  }
}

}  // namespace

// ------------------------------------------------------------------ pair kernel
// How results leave: partial tiles of a split product, TMA stores (and addends by
// TMA loads), or loads and stores of the epilogue warps where out's rows do not
// start on 16-byte boundaries. One kernel each: together they spill registers
// (apart, the one for partial tiles 36 bytes and the fp32 one by TMA 8).
enum PairStore : int { kStoreParts = 0, kStoreTma = 1, kStoreTmaAdd = 2, kStorePlain = 3, kStoreAdd = 4 };

template <bool kBf16, int kStore>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMxThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ MxGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);   // 1024-byte aligned, and known to be shared memory
  constexpr bool kTmaAdd = kStore == kStoreTmaAdd;
  constexpr int kStages = kTmaAdd ? kPStages - 1 : kPStages;
  constexpr int kChunkBytes = kTmaAdd ? 2 * kPChunkBytes : kPChunkBytes;   // per epilogue warp
  static_assert(kStages >= kSfBufs, "a scale buffer's last use is among the stages in flight");
  uint8_t* slots = smem + kStages * kPStageBytes;
  uint8_t* chunks = slots + kSfSlots * kPScaleBytes;
  // both CTAs' codes in shared memory and scales in TMEM
  uint64_t* full = reinterpret_cast<uint64_t*>(chunks + kMxEpiWarps * kChunkBytes);
  uint64_t* empty = full + kStages;
  uint64_t* sfull = empty + kStages;     // scales in shared memory, this CTA's
  uint64_t* sempty = sfull + kSfSlots;
  uint64_t* tfull = sempty + kSfSlots;    // one per accumulator
  // the accumulator of the tile after this one is free; one per accumulator,
  // because a warp may arrive for a tile while a slower one has yet to arrive
  // for the tile before (but not for the one before that: the MMAs between
  // waited for it)
  uint64_t* tnext = tfull + 2;
  uint64_t* done = tnext + 2;
  uint64_t* addfull = done + 1;           // addends in an epilogue warp's two buffers
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(addfull + 2 * kMxEpiWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile GaveUp* record = reinterpret_cast<volatile GaveUp*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.wait_limit_ns;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);
  const int ntiles = p.count * p.tm * p.tn * p.split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1 + 2 * kMxScaleWarps);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], kMxScaleWarps);
    }
    mbar_init(&tfull[0], 1);
    mbar_init(&tfull[1], 1);
    mbar_init(&tnext[0], 2 * kMxEpiWarps);
    mbar_init(&tnext[1], 2 * kMxEpiWarps);
    mbar_init(done, 1);
    for (int s = 0; s < 2 * kMxEpiWarps; ++s) mbar_init(&addfull[s], 1);
    *abort_flag = 0;
    record->peer = 0;
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
  // the other CTA's barriers are initialised before any remote signal (thread
  // 0 has fenced its own, so the arrival need not order anything)
  cluster_arrive_relaxed();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < ntiles; t += npairs) {
        const MxTile T = mx_tile(p, t);
        const int cl = p.share_l ? 0 : T.c, cr = p.share_r ? 0 : T.c;
        const int lrow = T.im * kPTile + kRows * static_cast<int>(rank);
        const int rrow = T.in * kPTile + kRows * static_cast<int>(rank);
        for (int kb = 0; kb < T.nkb; ++kb) {
          if (withheld(p, false, issued) || !mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, limit)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + stage * kPStageBytes;
          const uint32_t bar = full_leader + 8u * static_cast<uint32_t>(stage);
          const int k = T.kb0 + kb;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 4 * kCodeBytes);
          tma_load_3d_pair(st, &p.rows_l, bar, k * kKBytes, lrow, cl);
          tma_load_3d_pair(st + kCodeBytes, &p.rows_r, bar, k * kKBytes, rrow, cr);
          ++issued;
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      record->issued = issued;
      // the MMAs' signals for the last stages come from the leader: this CTA
      // may not leave before they have arrived
      for (int u = max(0, issued - kStages); ok && u < issued; ++u)
        ok = mbar_wait(&empty[u % kStages], static_cast<uint32_t>(u / kStages) & 1u, abort_flag, p.status, limit);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // -------------------------------------------------- MMA issuer (leader)
      // Four MMAs take the tensor pipe 512 cycles, and this warp's work per
      // stage must take less: one barrier per stage (codes and scales arrive on
      // the same one), asked for the next stage before this one's MMAs and
      // looked at after them; the whole warp runs the loop, so that addresses
      // and descriptors are uniform values, and they change by additions only
      // (K step: 32 bytes, stage: kPStageBytes). Lane 0 issues.
      const uint64_t desc0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      constexpr uint32_t kStageStep = kPStageBytes >> 4, kOperandB = kCodeBytes >> 4;
      constexpr uint32_t id0 = idesc_mxf4(kPTile, kPTile, 0), id2 = idesc_mxf4(kPTile, kPTile, 2);
      const bool issuer = lane == 0;
      const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0), sf0 = tmem + kSfColumn;
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      uint32_t stage = 0, phase = 0, sf = 0;   // sf: scale column of the stage
      uint64_t a = desc0;
      uint32_t tile = 0;   // tiles of this pair so far; their parity is the accumulator
      bool ok = true, ready = false;
      for (int t = pair; ok && t < ntiles; t += npairs) {
        const int kb0 = p.split == 1 ? 0 : t % p.split * p.kc;
        const int nkb = min(p.kc, p.kstages - kb0), tail = p.k64 - 4 * (kb0 + nkb - 1);   // K steps of the last stage
        if (tile > 0 && !__all_sync(0xffffffffu, mbar_wait(&tnext[(tile - 1) & 1u], ((tile - 1) >> 1) & 1u,
                                                           abort_flag, p.status, limit))) {
          ok = false;
          break;
        }
        const uint32_t d = tmem + (tile & 1u) * kAccOffset;
        uint32_t accumulate = 0;
#pragma unroll 1
        for (int kb = 0; kb < nkb; ++kb) {
          if (!ready && !__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, p.status, limit))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a0 = a;
          const uint32_t sfa = sf0 + sf, sfb = sfa + 8, used = empty0 + 8u * stage;
          const bool whole = kb + 1 < nkb || tail >= 4;
          a += kStageStep;
          sf = sf == (kSfBufs - 1) * kSfBuf ? 0u : sf + kSfBuf;
          if (++stage == kStages) { stage = 0; phase ^= 1u; a = desc0; }
          const bool next = mbar_test(full0 + 8u * stage, phase);
          if (whole) {
            if (issuer) {
              umma_mxf4_pair(d, a0, a0 + kOperandB, id0, sfa, sfb, accumulate);
              umma_mxf4_pair(d, a0 + 2, a0 + kOperandB + 2, id2, sfa, sfb, 1u);
              umma_mxf4_pair(d, a0 + 4, a0 + kOperandB + 4, id0, sfa + 4, sfb + 8, 1u);
              umma_mxf4_pair(d, a0 + 6, a0 + kOperandB + 6, id2, sfa + 4, sfb + 8, 1u);
              umma_commit_pair(used);
            }
          } else if (issuer) {   // the end of K
            umma_mxf4_pair(d, a0, a0 + kOperandB, id0, sfa, sfb, accumulate);
            if (tail > 1) umma_mxf4_pair(d, a0 + 2, a0 + kOperandB + 2, id2, sfa, sfb, 1u);
            if (tail > 2) umma_mxf4_pair(d, a0 + 4, a0 + kOperandB + 4, id0, sfa + 4, sfb + 8, 1u);
            umma_commit_pair(used);
          }
          accumulate = 1;
          ready = __all_sync(0xffffffffu, next);
        }
        if (!ok) break;
        if (issuer) umma_commit_pair(&tfull[tile & 1u]);
        ++tile;
      }
      if (issuer) umma_commit_pair(done);
      // the last tile's hand-over signals have arrived too: half of them come
      // from the other CTA, and nothing else waits for them
      if (ok) mbar_wait(&tnext[(tile - 1) & 1u], ((tile - 1) >> 1) & 1u, abort_flag, p.status, limit);
    }
    __syncwarp();
  } else if (warp == 2 + kMxEpiWarps + kMxScaleWarps) {
    if (lane == 0) {
      // ---------------------------------------------------- scale producer
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < ntiles; t += npairs) {
        const MxTile T = mx_tile(p, t);
        const int ltile = (p.share_l ? 0 : T.c) * p.tiles_l + 2 * T.im + static_cast<int>(rank);
        const int rtile = (p.share_r ? 0 : T.c) * p.tiles_r + 2 * T.in;
        for (int kb = 0; kb < T.nkb; ++kb) {
          if (withheld(p, true, issued) || !mbar_wait(&sempty[slot], phase ^ 1u, abort_flag, p.status, limit)) {
            ok = false;
            break;
          }
          uint8_t* at = slots + slot * kPScaleBytes;
          mbar_arrive_expect_tx(&sfull[slot], kPScaleBytes);
          tma_load_2d(at, &p.scales_l, &sfull[slot], (T.kb0 + kb) * 256, ltile);
          tma_load_2d(at + kSfGroupBytes, &p.scales_r, &sfull[slot], (T.kb0 + kb) * 256, rtile);
          ++issued;
          if (++slot == kSfSlots) { slot = 0; phase ^= 1u; }
        }
      }
      // every load has landed before shared memory is released
      for (int u = max(0, issued - kSfSlots); u < issued; ++u)
        drain(&sfull[u % kSfSlots], static_cast<uint32_t>(u / kSfSlots) & 1u);
    }
  } else if (warp >= 2 + kMxEpiWarps) {
    // ------------------------------------------------------ scales to TMEM
    // Word j of lane l of a scale tile belongs to row 32 j + l: that is TMEM
    // column j, the same in all four lane quadrants (one per warp).
    const uint32_t quad = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
    // stage: the one these scales go with; old_stage: the one used kSfBufs stages before
    int stage = 0, old_stage = kStages - kSfBufs, slot = 0;
    uint32_t phase = 0, old_phase = 1, uses = 0;
    bool ok = true;
    for (int t = pair; ok && t < ntiles; t += npairs) {
      const MxTile T = mx_tile(p, t);
      for (int kb = 0; kb < T.nkb; ++kb) {
        // the scales have landed
        if (!__all_sync(0xffffffffu, mbar_wait(&sfull[slot], phase, abort_flag, p.status, limit))) {
          ok = false;
          break;
        }
        const uint4* sf = reinterpret_cast<const uint4*>(slots + slot * kPScaleBytes) + lane;
        // a 512-byte tile is 32 uint4; A: K halves 0, 1; B: row tile 0 halves 0, 1, row tile 1 halves 0, 1
        const uint4 a0 = sf[0], a1 = sf[32], b00 = sf[64], b01 = sf[96], b10 = sf[128], b11 = sf[160];
        // a buffer is free once the MMAs that used it are done
        if (uses >= kSfBufs &&
            !__all_sync(0xffffffffu,
                        mbar_wait(&empty[old_stage], old_phase, abort_flag, p.status, limit))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t buf = uses % kSfBufs;
        const uint32_t at = tmem_base + quad + kSfColumn + buf * kSfBuf;
        tmem_st8(at, a0, a1);
        tmem_st16(at + 8, b00, b10, b01, b11);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // the slot goes back only now that its values have been used: an
          // arrival right behind the loads lets the refill overtake them
          mbar_arrive(&sempty[slot]);
          mbar_arrive_cluster_cta(full_leader + 8u * static_cast<uint32_t>(stage));
        }
        ++uses;
        if (++stage == kStages) stage = 0;
        if (++slot == kSfSlots) { slot = 0; phase ^= 1u; }
        if (++old_stage == kStages) { old_stage = 0; old_phase ^= 1u; }
      }
    }
    if (lane == 0) record->scaled[warp & 3] = static_cast<int>(uses);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // warp w reads TMEM lanes 32 (w % 4) ..; warps 2..5 the accumulator's
    // columns 0..127, warps 6..9 columns 128..255, 32 at a time, the columns
    // that the next tile's accumulator overlaps first.
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tnext_leader = mapa_shared(smem_u32(tnext), 0);
    const bool vec = (p.n % 4) == 0;
    uint8_t* buf = chunks + (warp - 2) * kChunkBytes;
    uint32_t acc = 0, phase = 0;
    bool ok = true;
    auto prefetch = [&](int t) {
      const MxTile T = mx_tile(p, t);
      prefetch_addends<kBf16>(p, T.c * p.stride_c, T.im * kPTile + kRows * static_cast<int>(rank) + 32 * q + lane,
                              T.in * kPTile + half * 128);
    };
    if ((kStore == kStoreAdd || kTmaAdd) && pair < ntiles) prefetch(pair);
    // Addends by TMA: a tile's boxes of 32 rows x 128 bytes in the order in
    // which the results come out of TMEM, one load ahead of the one at work
    // (into the next tile too), the two buffers taken in turn.
    constexpr int kBoxes = kBf16 ? 2 : 4;
    uint64_t* bar = addfull + 2 * (warp - 2);
    uint32_t loads = 0, used = 0;
    auto load_addends = [&](const MxTile& T, uint32_t acc, int i) {   // lane 0; the buffer's last store has read it
      const bool back = half == 1 && acc == 0;
      const int x = kBf16 ? (back ? 1 - i : i) * 64 : (back ? (i < 2 ? 2 + i : 3 - i) : i) * 32;
      mbar_arrive_expect_tx(&bar[loads & 1u], kPChunkBytes);
      tma_load_3d(buf + (loads & 1u) * kPChunkBytes, &p.addend, &bar[loads & 1u], T.in * kPTile + half * 128 + x,
                  T.im * kPTile + kRows * static_cast<int>(rank) + 32 * q, T.c);
      ++loads;
    };
    if (kTmaAdd && lane == 0 && pair < ntiles) load_addends(mx_tile(p, pair), 0, 0);
    for (int t = pair; ok && t < ntiles; t += npairs) {
      const MxTile T = mx_tile(p, t);
      if ((kStore == kStoreAdd || kTmaAdd) && t + npairs < ntiles) prefetch(t + npairs);
      int box = 0;
      const bool overlapped = (acc == 0) == (half == 1);
      if (!overlapped) {  // this warp holds nothing the next tile's MMAs would overwrite
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_cta(tnext_leader + 8u * acc);
      }
      const bool got = mbar_wait(&tfull[acc], phase, abort_flag, p.status, limit);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * kAccOffset + half * 128;
      const int row = T.im * kPTile + kRows * static_cast<int>(rank) + 32 * q;
      const int col = T.in * kPTile + half * 128;
      auto store_pair = [&](const uint32_t* a, int ha, const uint32_t* b, int j) {   // chunks j + ha, j + 1 - ha
        if constexpr (kStore == kStoreParts) {
          // partial tile: a 32 x 32 chunk as 8 rows of 32 float4, one per lane
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t* r = c ? b : a;
            float4* dst = reinterpret_cast<float4*>(
                p.part + static_cast<long long>(t) * (kPTile * kPTile) +
                ((((rank * 4 + q) * 2 + half) * 4 + j + (c ? 1 - ha : ha)) * 1024));
#pragma unroll
            for (int g = 0; g < 8; ++g)
              dst[g * 32 + lane] = make_float4(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1]),
                                               __uint_as_float(r[4 * g + 2]), __uint_as_float(r[4 * g + 3]));
          }
        } else if constexpr (kTmaAdd) {
#pragma unroll
          for (int i = 0; i < (kBf16 ? 1 : 2); ++i) {
            const int x = kBf16 ? col + j * 32 : col + (j + (i ? 1 - ha : ha)) * 32;
            uint8_t* at = buf + (used & 1u) * kPChunkBytes;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&bar[used & 1u], (used >> 1) & 1u, abort_flag, p.status, limit));
            if (!ok) return;
            add_staged<kBf16>(at, lane, i ? b : a, ha, b);
            fence_proxy_async_smem();
            __syncwarp();
            ++used;
            ++box;
            if (lane == 0) {
              if (row < p.m && x < p.n) tma_store_3d(&p.result, at, x, row, T.c);
              bulk_commit();
              bulk_wait_read<1>();   // the store before this one has read the other buffer
              if (box < kBoxes) load_addends(T, acc, box);
              else if (t + npairs < ntiles) load_addends(mx_tile(p, t + npairs), acc ^ 1u, 0);
            }
          }
        } else if constexpr (kStore == kStoreTma) {
          store_pair_tma<kBf16>(p, buf, lane, a, ha, b, T.c, row, col + j * 32);
        } else {
          constexpr bool kAdd = kStore == kStoreAdd;
          store_chunk<kBf16, kAdd>(p, buf, lane, a, T.c * p.stride_c, row, col + (j + ha) * 32, vec);
          store_chunk<kBf16, kAdd>(p, buf, lane, b, T.c * p.stride_c, row, col + (j + 1 - ha) * 32, vec);
        }
      };
      // Three of the warp's four chunks are taken to registers first: with them
      // the columns that the two accumulators share (the last ones of acc 0,
      // the first ones of acc 1). They are a whole pair and a chunk of the
      // other one, whose partner follows.
      static_assert(kOverlapChunks == 3, "chunks in registers");
      uint32_t r0[32], r1[32], r2[32];
      const bool back = overlapped && acc == 0;
      const int pair0 = back ? 2 : 0, lone = back ? 1 : 2, rest = back ? 0 : 3;
      tmem_ld32(tb + pair0 * 32, r0);
      tmem_ld32(tb + pair0 * 32 + 32, r1);
      tmem_ld32(tb + lone * 32, r2);
      tmem_ld_wait();
      if (overlapped) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_cta(tnext_leader + 8u * acc);
      }
      store_pair(r0, 0, r1, pair0);
      tmem_ld32(tb + rest * 32, r0);
      tmem_ld_wait();
      store_pair(r2, lone & 1 ? 1 : 0, r0, back ? 0 : 2);
      acc ^= 1u;
      if (acc == 0) phase ^= 1u;
    }
    if (lane == 0) {
      // after a wait that ran out: a load under way lands before shared memory is released
      if (loads > used) drain(&bar[used & 1u], (used >> 1) & 1u);
      bulk_wait_all();   // every bulk store of this warp has completed
    }
    __syncwarp();
  }

  // let the kernel that adds the parts be launched (it waits for this grid)
  if (kStore == kStoreParts) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  // Where every wait of the pair has succeeded, every load has been used, no
  // MMA is in flight, and the CTAs may part. Where one ran out, both hear of it
  // here, and stay until the loads of either have landed.
  const bool gave_up = *abort_flag != 0;
  if (!gave_up && threadIdx.x == 0) drain(done, 0);
  __syncwarp();
  if (gave_up) {
    if (threadIdx.x == 0) st_cluster(mapa_shared(smem_u32(const_cast<int*>(&record->peer)), rank ^ 1u), 1);
    __syncwarp();
    cluster_arrive();
  } else {
    cluster_arrive_relaxed();
  }
  cluster_wait();
  if (gave_up || record->peer != 0) {
    cluster_sync();   // both CTAs' records are complete and visible, and `done` is committed
    if (threadIdx.x == 0) {
      if (rank == 0) finish_stages<kStages>(full, record);
      drain(done, 0);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// Adds the partial tiles of a split product in split order. One block per
// 32 x 32 chunk (a partial tile has 64): thread (g, lane) adds columns 4 g .. of
// row `lane`, all parts on their way at once, and the chunk is turned in shared
// memory so that rows are stored whole.
template <bool kBf16>
__global__ void __launch_bounds__(256) mx_reduce_kernel(const __grid_constant__ MxGemmParams p) {
  __shared__ float turn[32][33];
  const int chunk = static_cast<int>(blockIdx.x & 63u), tile = static_cast<int>(blockIdx.x >> 6);
  const MxTile T = mx_tile(p, tile * p.split);
  const int j = chunk & 3, half = (chunk >> 2) & 1, q = (chunk >> 3) & 3, rank = chunk >> 5;
  const int row0 = T.im * kPTile + kRows * rank + 32 * q, col0 = T.in * kPTile + half * 128 + j * 32;
  if (row0 >= p.m || col0 >= p.n) return;
  // this thread's output: four columns of row tid / 8
  const int row = row0 + static_cast<int>(threadIdx.x >> 3), col = col0 + 4 * static_cast<int>(threadIdx.x & 7u);
  const bool exists = row < p.m && col < p.n, vec = (p.n & 3) == 0;
  const long long at = T.c * p.stride_c + static_cast<long long>(row) * p.n + col;
  float add[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.add && exists) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < p.n) add[i] = load1t<kBf16>(p.add, at + i);
  }
  // launched while the pair kernel still runs: its partial tiles are complete
  // once this returns (the addends are not its work)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (*reinterpret_cast<const volatile int*>(p.status) != 0) return;
  const float4* src = reinterpret_cast<const float4*>(
      p.part + static_cast<long long>(tile) * p.split * (kPTile * kPTile) + chunk * 1024) + threadIdx.x;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < p.split; s0 += 8) {
    float4 v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < p.split) v[s] = src[static_cast<long long>(s0 + s) * (kPTile * kPTile / 4)];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (s0 + s < p.split) {
        acc.x += v[s].x; acc.y += v[s].y; acc.z += v[s].z; acc.w += v[s].w;
      }
    }
  }
  const int g = threadIdx.x >> 5, lane = threadIdx.x & 31;
  turn[lane][4 * g] = acc.x;
  turn[lane][4 * g + 1] = acc.y;
  turn[lane][4 * g + 2] = acc.z;
  turn[lane][4 * g + 3] = acc.w;
  __syncthreads();
  if (!exists) return;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = turn[threadIdx.x >> 3][4 * (threadIdx.x & 7u) + i] + add[i];
  if (vec) {
    if (kBf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
          make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < p.n) store1t<kBf16>(p.out, at + i, y[i]);
  }
}

// -------------------------------------------------------------- few-row kernel
// One tile of 128 left rows x NT right rows per cluster; CTA r of the cluster
// takes K stages r * kc .. and sends its part to the CTAs that add it up, each
// some of the right rows, by bulk copies between the CTAs' shared memories,
// counted on the receiver's barrier. (Reading the parts out of the other CTAs'
// memory took another cluster barrier; sending them value by value with
// st.async took 0.13 us per right row.) 192 threads: warp 0 loads,
// warp 1 issues the MMAs, warps 2..5 are the epilogue.
constexpr int kFewThreads = 192;
constexpr int kFewSplit = 8;       // most CTAs per cluster

// Four neighbouring outputs of one row (whose length is a multiple of 4).
template <bool kBf16>
__device__ __forceinline__ void store_quad(const MxGemmParams& p, long long at, float (&y)[4]) {
  if (kBf16) {
    if (p.add) {
      const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.add) + at);
      y[0] += bf16_lo_f(a.x); y[1] += bf16_hi_f(a.x); y[2] += bf16_lo_f(a.y); y[3] += bf16_hi_f(a.y);
    }
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  } else {
    if (p.add) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p.add) + at);
      y[0] += a.x; y[1] += a.y; y[2] += a.z; y[3] += a.w;
    }
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
  }
}

template <int NT>
__host__ __device__ constexpr int few_stage_bytes() { return kCodeBytes + NT * kKBytes + 2 * kSfGroupBytes; }

// Stages in shared memory at most; each has scale columns of its own in TMEM
// (8 for the left operand, 8 for the right), so that the MMAs of one stage do
// not wait for those of the stage before. With the accumulator: 128 columns.
template <int NT>
__host__ __device__ constexpr int few_ring() { return NT == 16 ? 5 : 4; }

constexpr uint32_t kFewColumns = 128;

template <int NT, bool kBf16>
__global__ void __launch_bounds__(kFewThreads) mx_gemm_few_kernel(const __grid_constant__ MxGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);   // 1024-byte aligned, and known to be shared memory
  __shared__ uint64_t full[few_ring<NT>()], empty[few_ring<NT>()], sready[few_ring<NT>()], done, parts;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ int sent;                // this CTA's part is on its way to the others
  __shared__ volatile int gave_up;    // a CTA of the cluster did
  constexpr int kStage = few_stage_bytes<NT>();
  static_assert(NT + 16 * few_ring<NT>() <= kFewColumns, "accumulator and scales");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.wait_limit_ns;
  volatile int* abort_flag = &abort_word;
  const int split = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int c = tile / p.tm, im = tile - c * p.tm;
  const int kb0 = split * p.kc, nkb = min(p.kc, p.kstages - kb0);
  // test hook: stages that one CTA (the first or the last of the first cluster) loads
  const int last = p.fault != 0 && static_cast<int>(blockIdx.x) == (p.fault == 1 ? 0 : p.split - 1) ? nkb - 1 : nkb;
  // split tiles: this CTA adds up the right rows x0 .. x0 + xn - 1
  const int xs = (NT + p.split - 1) / p.split, x0 = split * xs, xn = max(0, min(xs, p.n - x0));
  uint8_t* received = smem + max(p.ring * kStage, NT * kRows * 4);

  auto load = [&](int kb, int stage) {
    const int cl = p.share_l ? 0 : c, cr = p.share_r ? 0 : c;
    uint8_t* st = smem + stage * kStage;
    const int k = kb0 + kb;
    const uint32_t sf = static_cast<uint32_t>(min(2, p.sf_groups - 2 * k)) * kMxTileBytes;
    uint8_t* sl = st + kCodeBytes + NT * kKBytes;
    mbar_arrive_expect_tx(&full[stage], kCodeBytes + NT * kKBytes + 2 * sf);
    tma_load_3d(st, &p.rows_l, &full[stage], k * kKBytes, im * kRows, cl);
    tma_load_3d(st + kCodeBytes, &p.rows_r, &full[stage], k * kKBytes, 0, cr);
    // contiguous, so they need no tensor map (fetching one costs a cold call
    // about half a microsecond)
    bulk_load(sl, p.sf_l + (static_cast<long long>(cl * p.tiles_l + im) * p.sf_groups + 2 * k) * kMxTileBytes, sf,
              &full[stage]);
    bulk_load(sl + kSfGroupBytes, p.sf_r + (static_cast<long long>(cr) * p.tiles_r * p.sf_groups + 2 * k) * kMxTileBytes,
              sf, &full[stage]);
  };

  if (threadIdx.x == 64) tma_prefetch_map(&p.rows_l);
  if (threadIdx.x == 96) tma_prefetch_map(&p.rows_r);
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sready[s], 4);
    }
    mbar_init(&done, 1);
    mbar_init(&parts, 1);
    abort_word = sent = gave_up = 0;
    fence_mbar_init();
    if (p.split > 1) mbar_arrive_expect_tx(&parts, static_cast<uint32_t>(p.split * xn * kRows * 4));
    // the first loads leave before the TMEM allocation and the barrier
#pragma unroll 1
    for (int kb = 0; kb < min(p.ring, last); ++kb) load(kb, kb);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kFewColumns);
    tmem_relinquish();
  }
  if (p.add && warp >= 2) {   // the addends to L2: 32 left rows at a time where those are neighbours in out
    const int per = p.stride_l == 1 ? 4 : kRows, total = p.stride_l == 1 ? 4 * p.n : kRows;
    for (int i = static_cast<int>(threadIdx.x) - 64; i < total; i += 128) {
      const int l = im * kRows + i % per * (kRows / per);
      if (l < p.m)
        prefetch_l2(static_cast<const uint8_t*>(p.add) +
                    (c * p.stride_c + l * p.stride_l + i / per * p.stride_r) * (kBf16 ? 2 : 4));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_arrive_relaxed();   // this CTA's barriers are initialised (and fenced)
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = min(p.ring, last);
      uint32_t phase = 0;
      for (int kb = issued; kb < last; ++kb, ++issued) {
        if (!mbar_wait(&empty[stage], phase, abort_flag, p.status, limit)) break;
        load(kb, stage);
        if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      }
      // every load has landed before shared memory is released
      for (int kb = max(0, issued - p.ring); kb < issued; ++kb)
        drain(&full[kb % p.ring], static_cast<uint32_t>(kb / p.ring) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      const uint64_t desc0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      // kept short (no unrolling): a call's few stages run from a cold
      // instruction cache
#pragma unroll 1
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait(&full[stage], phase, abort_flag, p.status, limit) ||
            !mbar_wait(&sready[stage], phase, abort_flag, p.status, limit))
          break;
        tc_fence_after();
        const uint32_t sfa = tmem_base + NT + static_cast<uint32_t>(stage) * 16u, sfb = sfa + 8;
        const uint64_t a = desc0 + static_cast<uint32_t>(stage * (kStage >> 4)), b = a + (kCodeBytes >> 4);
        const int steps = min(4, p.k64 - 4 * (kb0 + kb));
#pragma unroll 1
        for (int ks = 0; ks < steps; ++ks)
          umma_mxf4(tmem_base, a + 2 * ks, b + 2 * ks, idesc_mxf4(kRows, NT, 2 * (ks & 1)), sfa + 4 * (ks >> 1),
                    sfb + 4 * (ks >> 1), (kb > 0 || ks > 0) ? 1u : 0u);
        umma_commit(&empty[stage]);
        if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      }
      umma_commit(&done);
    }
    __syncwarp();
  } else {
    // scales to TMEM, as in the pair kernel (one lane quadrant per warp)
    int stage = 0;
    uint32_t phase = 0;
#pragma unroll 1
    for (int kb = 0; kb < nkb; ++kb) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, p.status, limit))) break;
      const uint4* sf = reinterpret_cast<const uint4*>(smem + stage * kStage + kCodeBytes + NT * kKBytes) + lane;
      tc_fence_after();
      tmem_st16(tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + NT + static_cast<uint32_t>(stage) * 16u,
                sf[0], sf[32], sf[64], sf[96]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sready[stage]);
      if (++stage == p.ring) { stage = 0; phase ^= 1u; }
    }
    __syncwarp();
  }
  bool ok = mbar_wait(&done, 0, abort_flag, p.status, limit);
  if (!ok) drain(&done, 0);
  ok = __syncthreads_and(ok && *abort_flag == 0);
  tc_fence_after();

  const int q = warp & 3;
  const uint32_t tlane = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
  auto free_columns = [&] {   // once every warp has read the accumulator
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc(tmem_base, kFewColumns);
    }
  };
  if (p.split == 1) {
    if (ok && warp >= 2) {
      const int l = im * kRows + 32 * q + lane;
#pragma unroll 1
      for (int x = 0; x < p.n; x += 8) {
        uint32_t r[8];
        tmem_ld8(tlane + x, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (l < p.m && x + j < p.n) {
            const long long at = c * p.stride_c + l * p.stride_l + (x + j) * p.stride_r;
            float v = __uint_as_float(r[j]);
            if (p.add) v += load1t<kBf16>(p.add, at);
            store1t<kBf16>(p.out, at, v);
          }
        }
      }
    }
    free_columns();
  } else {
    // the part as [right row][128], in the ring's memory (its loads have been
    // consumed)
    float* mine = reinterpret_cast<float*>(smem);
    if (ok && warp >= 2) {
#pragma unroll 1
      for (int x = 0; x < p.n; x += 8) {
        uint32_t r[8];
        tmem_ld8(tlane + x, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) mine[(x + j) * kRows + 32 * q + lane] = __uint_as_float(r[j]);
      }
      fence_proxy_async_smem();
    }
    // before the cluster barrier: a CTA of this cluster may still wait for
    // columns that another cluster's CTA holds, and that one for this CTA's
    free_columns();
    __syncwarp();
    cluster_wait();   // every CTA's `parts` is initialised
    if (ok && threadIdx.x == 0) sent = 1;
    if (ok && threadIdx.x < static_cast<unsigned>(p.split)) {
      // thread r sends CTA r the right rows it adds up
      const int owner = static_cast<int>(threadIdx.x), n = max(0, min(xs, p.n - owner * xs));
      if (n > 0)
        bulk_copy_cluster(mapa_shared(smem_u32(received) + static_cast<uint32_t>(split * xs * kRows * 4), owner),
                          mine + owner * xs * kRows, static_cast<uint32_t>(n * kRows * 4),
                          mapa_shared(smem_u32(&parts), owner));
    }
    // four left rows of a right row per thread; the parts are added in rank
    // order. A part that never came leaves the tile unwritten.
    if (xn > 0) ok = mbar_wait_cluster(&parts, 0, abort_flag, p.status, limit) && ok;
    ok = __syncthreads_and(ok);
    if (ok) {
      cluster_arrive_relaxed();   // what this CTA was sent has arrived
    } else {
      // a part is missing, here or for the others: every CTA has to know
      if (threadIdx.x < static_cast<unsigned>(p.split))
        st_cluster(mapa_shared(smem_u32(const_cast<int*>(&gave_up)), threadIdx.x), 1);
      __syncwarp();
      cluster_arrive();
    }
    if (xn > 0) {
      const float4* part = reinterpret_cast<const float4*>(received);
      if (ok) {
#pragma unroll 1
        for (int e = static_cast<int>(threadIdx.x); e < xn * (kRows / 4); e += kFewThreads) {
          float4 v[kFewSplit];
#pragma unroll
          for (int s = 0; s < kFewSplit; ++s)
            if (s < p.split) v[s] = part[s * xs * (kRows / 4) + e];
          float y[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
          for (int s = 1; s < kFewSplit; ++s) {
            if (s < p.split) {
              y[0] += v[s].x; y[1] += v[s].y; y[2] += v[s].z; y[3] += v[s].w;
            }
          }
          const int l = im * kRows + (e & 31) * 4;
          const long long at = c * p.stride_c + l * p.stride_l + (x0 + (e >> 5)) * p.stride_r;
          if (p.stride_l == 1 && (p.stride_r & 3) == 0) {   // four neighbours of one row of out
            if (l < p.m) store_quad<kBf16>(p, at, y);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (l + j < p.m) {
                if (p.add) y[j] += load1t<kBf16>(p.add, at + j * p.stride_l);
                store1t<kBf16>(p.out, at + j * p.stride_l, y[j]);
              }
            }
          }
        }
      }
    }
    __syncwarp();
    cluster_wait();   // and so has what it sent: its memory may go
    if (gave_up != 0) {
      // unless a CTA gave up: then parts may be on their way to it still. It
      // counts those that were never sent itself, and waits for the others.
      cluster_sync();   // every CTA's `sent` is final and visible
      if (threadIdx.x == 0 && xn > 0) {
        int missing = 0;
        for (int r = 0; r < p.split; ++r) missing += ld_cluster(mapa_shared(smem_u32(&sent), r)) == 0 ? 1 : 0;
        if (missing > 0) mbar_complete_tx(&parts, static_cast<uint32_t>(missing * xn * kRows * 4));
        drain(&parts, 0);
      }
      __syncwarp();
      cluster_sync();
    }
  }
}

// ------------------------------------------------------------------- launches
MxGemmPlan plan_mx_gemm(const MxGemmShape& s, int pairs, int sms) {
  MxGemmPlan pl{};
  const int kstages = static_cast<int>((s.k + 255) / 256);
  const int64_t small = s.m < s.n ? s.m : s.n, large = s.m < s.n ? s.n : s.m;
  // Few rows on one side. Few-row against pair kernel, in us: up to 32 rows 32 x
  // 2560 x 2560 6.0 / 7.7, 16 x 50304 x 768 9.2 / 10.2, 32 x 10240 x 2560 8.9 /
  // 9.1, 48 of 16 x 768 x 768 8.3 / 8.3, but 32 x 50304 x 768 10.6 / 10.3. Up to 64
  // rows where the other side has few tiles too, so that K can be split over
  // many CTAs: 64 x 2560 x 2560 7.4 / 8.4, 64 x 768 x 3200 6.7 / 8.7 (64 x 10240 x
  // 2560 would be 12.9 / 9.3). At that limit and with a short K the pair kernel
  // is a little faster: 64 x 4736 x 2560 9.0 / 8.6, 64 x 768 x 768 6.0 / 5.7.
  const int64_t tall = (large + kRows - 1) / kRows;
  if (small <= 32 || (small <= 64 && s.count * tall <= sms / 4)) {
    pl.few = true;
    pl.swap = s.m <= s.n;  // the left operand of the kernel is the one with many rows
    pl.nt = small <= 16 ? 16 : small <= 32 ? 32 : 64;
    pl.tm = static_cast<int>(tall);
    pl.tn = 1;
    // as many K parts as one wave of CTAs holds; two fit an SM, with 64
    // columns one
    const int64_t slots = pl.nt == 64 ? sms : 2 * sms;
    int64_t split = slots / (s.count * tall);
    if (split > kFewSplit) split = kFewSplit;
    if (split > kstages) split = kstages;
    if (split < 1) split = 1;
    pl.kc = static_cast<int>((kstages + split - 1) / split);
    pl.split = (kstages + pl.kc - 1) / pl.kc;   // no empty part
    const int cap = pl.nt == 16 ? few_ring<16>() : few_ring<32>();
    pl.ring = pl.kc < cap ? pl.kc : cap;
    return pl;
  }
  pl.tm = static_cast<int>((s.m + kPTile - 1) / kPTile);
  pl.tn = static_cast<int>((s.n + kPTile - 1) / kPTile);
  const int64_t tiles = s.count * pl.tm * pl.tn;
  // Few tiles and a long K: split it. A stage takes a pair about 0.29 us; the
  // partial tiles and the kernel that adds them cost 3 us with one tile (4 MB
  // of them) and 8 with 36 (19 MB), so 12 stages have to be saved, and one more
  // for every two tiles. In us, unsplit against split: 200 x 200 (1 tile), K 3584
  // 9.1 / 9.1, K 4096 9.7 / 9.3, K 8192 14.7 / 9.8; 768 x 768 (9), K 4096
  // 11.5 / 11.6, K 5120 12.7 / 11.6, K 8192 16.2 / 12.8; 1000 x 1000 (16), K 6144
  // 13.3 / 13.3, K 8192 15.6 / 14.1; 1500 x 1500 (36), K 8192 16.6 / 19.8,
  // K 12288 21.2 / 22.7, K 16384 25.9 / 25.5.
  pl.split = 1;
  if (tiles * 2 <= pairs) {
    const int64_t sp = pairs / tiles < 16 ? pairs / tiles : 16;
    if (2 * (kstages - (kstages + sp - 1) / sp) >= 24 + tiles) pl.split = static_cast<int>(sp);
  }
  pl.kc = (kstages + pl.split - 1) / pl.split;
  pl.split = (kstages + pl.kc - 1) / pl.kc;
  if (pl.split > 1) pl.part_bytes = static_cast<size_t>(tiles) * pl.split * kPTile * kPTile * 4;
  return pl;
}

template <int kStore>
static const void* pair_kernel_store(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&mx_gemm_pair_kernel<true, kStore>)
              : reinterpret_cast<const void*>(&mx_gemm_pair_kernel<false, kStore>);
}

static const void* pair_kernel(bool bf16, int store) {
  switch (store) {
    case kStoreParts: return reinterpret_cast<const void*>(&mx_gemm_pair_kernel<false, kStoreParts>);
    case kStoreTma: return pair_kernel_store<kStoreTma>(bf16);
    case kStoreTmaAdd: return pair_kernel_store<kStoreTmaAdd>(bf16);
    case kStorePlain: return pair_kernel_store<kStorePlain>(bf16);
    default: return pair_kernel_store<kStoreAdd>(bf16);
  }
}

template <int NT>
static const void* few_kernel_nt(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&mx_gemm_few_kernel<NT, true>)
              : reinterpret_cast<const void*>(&mx_gemm_few_kernel<NT, false>);
}

static const void* few_kernel(int nt, bool bf16) {
  return nt == 16 ? few_kernel_nt<16>(bf16) : nt == 32 ? few_kernel_nt<32>(bf16) : few_kernel_nt<64>(bf16);
}

// Shared memory of the few-row kernel: the ring, which later holds the CTA's
// part, and the parts received.
static int few_smem(const MxGemmPlan& pl) {
  const int ring = pl.ring * (kCodeBytes + pl.nt * kKBytes + 2 * kSfGroupBytes), part = pl.nt * kRows * 4;
  const int received = (pl.nt + pl.split - 1) / pl.split * pl.split * kRows * 4;
  return (pl.split > 1 ? (ring > part ? ring : part) + received : ring) + 1024;
}

cudaError_t mx_gemm_prepare(int* max_pairs) {
  cudaError_t e = cudaSuccess;
  for (int store = kStoreParts; store <= kStoreAdd; ++store)
    for (int b = 0; b < 2 && e == cudaSuccess; ++b)
      e = cudaFuncSetAttribute(pair_kernel(b, store), cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmemBytes);
  for (int nt = 16; nt <= 64; nt *= 2)
    for (int b = 0; b < 2 && e == cudaSuccess; ++b)
      e = cudaFuncSetAttribute(few_kernel(nt, b), cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  *max_pairs = sms / 2;
  return cudaSuccess;
}

cudaError_t launch_mx_gemm(const MxGemmParams& p, const MxGemmPlan& plan, bool bf16, int max_pairs,
                           cudaStream_t s) {
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
  const int store = plan.split > 1 ? kStoreParts : p.tma_out ? (p.add ? kStoreTmaAdd : kStoreTma) : p.add ? kStoreAdd : kStorePlain;
  cudaError_t e = cudaLaunchKernelExC(&cfg, pair_kernel(bf16, store), args);
  if (e != cudaSuccess || plan.split == 1) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * 64u, 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg,
                             bf16 ? reinterpret_cast<const void*>(&mx_reduce_kernel<true>)
                                  : reinterpret_cast<const void*>(&mx_reduce_kernel<false>),
                             args);
}

}  // namespace muon
