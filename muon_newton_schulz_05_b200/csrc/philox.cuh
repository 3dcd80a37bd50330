// Counter-based random numbers: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011). Nothing is stored:
// an element's 16-bit number is a function of (seed, offset + site, domain,
// row, column), so a backward pass or a replay forms the same numbers again.
//   key     = seed (64 bits)
//   counter = (column >> 3, row, lo32(n), hi30(n) | domain << 30), n = offset + site
// One call gives eight columns: column c takes half (c & 1) of word (c & 7) >> 1.
#pragma once
#include <stdint.h>

namespace muon {

enum RngDomain : uint32_t { kRngDropout = 0, kRngRows = 1, kRngCols = 2 };

struct RngKey {
  uint32_t k0, k1, n_lo, n_hi;
};

// rng: {seed, offset} in device memory, so that a captured graph draws new
// numbers when the caller advances the offset between replays.
__device__ __forceinline__ RngKey rng_key(const long long* rng, unsigned long long site) {
  const unsigned long long seed = static_cast<unsigned long long>(__ldg(rng));
  const unsigned long long n = static_cast<unsigned long long>(__ldg(rng + 1)) + site;
  return RngKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32),
                static_cast<uint32_t>(n), static_cast<uint32_t>(n >> 32) & 0x3FFFFFFFu};
}

// Ten rounds; the 16 bytes are the numbers of columns 8 g .. 8 g + 7 of `row`.
__device__ __forceinline__ uint4 philox8(const RngKey& key, uint32_t domain, uint32_t row, uint32_t g) {
  uint32_t c0 = g, c1 = row, c2 = key.n_lo, c3 = key.n_hi | (domain << 30);
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t q = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(q >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(q);
    c2 = static_cast<uint32_t>(p >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// N calls at once: the round keys are formed once, and the chains fill each
// other's latencies.
template <int N>
__device__ __forceinline__ void philox8n(const RngKey& key, uint32_t domain, const uint32_t (&row)[N],
                                         const uint32_t (&g)[N], uint4 (&out)[N]) {
  uint32_t c0[N], c1[N], c2[N], c3[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    c0[j] = g[j];
    c1[j] = row[j];
    c2[j] = key.n_lo;
    c3[j] = key.n_hi | (domain << 30);
  }
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * c0[j];
      const uint64_t q = static_cast<uint64_t>(0xCD9E8D57u) * c2[j];
      c0[j] = static_cast<uint32_t>(q >> 32) ^ c1[j] ^ k0;
      c1[j] = static_cast<uint32_t>(q);
      c2[j] = static_cast<uint32_t>(p >> 32) ^ c3[j] ^ k1;
      c3[j] = static_cast<uint32_t>(p);
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) out[j] = make_uint4(c0[j], c1[j], c2[j], c3[j]);
}

// Four calls for groups g[0..3] of one row.
__device__ __forceinline__ void philox8x4(const RngKey& key, uint32_t domain, uint32_t row,
                                          const uint32_t (&g)[4], uint4 (&out)[4]) {
  const uint32_t rows[4] = {row, row, row, row};
  philox8n<4>(key, domain, rows, g, out);
}

}  // namespace muon
