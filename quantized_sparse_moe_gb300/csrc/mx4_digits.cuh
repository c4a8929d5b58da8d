// Activations as base-8 digit planes in e2m1 (the mathematics is in
// mx4_stream.cu), and what the kernels that use them share on the host.
#pragma once

#include <mutex>

#include "mx4_common.cuh"

namespace qsm {
namespace mx4 {

constexpr int kDigits = 6;
constexpr uint32_t kDigitBias = 149796u;  // sum of 4 * 8^i, i < 6

// Rows of the MMA's digit operand for n rows of x.
__host__ __device__ constexpr int digit_rows(int n) { return (kDigits * n + 7) / 8 * 8; }

// The digit planes of eight values as e2m1 codes (one word each), and the
// scale byte of plane 0 (plane i: + 3 i; 255: not a number).  Lanes 4 j ..
// 4 j + 3 hold the four quarters of a block.
__device__ __forceinline__ uint32_t digits_of(const float (&v)[8], uint32_t (&plane)[kDigits]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  // E, at least -111 so that 2^(15 - E) is finite; 127 and up (2^127,
  // infinities, NaN) have no scale for their top digit
  const int e = max((int)(m >> 23) - 127, -111);
  const bool bad = e >= 127;
  const float f = __uint_as_float((uint32_t)(15 - (bad ? 0 : e) + 127) << 23);
  uint32_t y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = (uint32_t)__float2int_rn(bad ? 0.f : v[j] * f) + kDigitBias;
#pragma unroll
  for (int i = 0; i < kDigits; ++i) {
    uint32_t w = 0;  // eight unsigned digits 0..7, one per nibble
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int sh = 3 * i - 4 * j;
      w |= (sh >= 0 ? y[j] >> (sh & 31) : y[j] << (-sh & 31)) & (7u << (4 * j));
    }
    // digit - 4 as a code: 4..7 -> 0..3, 0..3 -> sign and magnitude 4 - digit
    const uint32_t low = w & 0x33333333u, neg = ~w & 0x44444444u;
    const uint32_t mask = (neg << 2) - (neg >> 2);
    plane[i] = (mask & (0xCCCCCCCCu - low)) | (~mask & low);
  }
  return bad ? 255u : (uint32_t)(e - 14 + 127);
}

// The planes of row i, columns 8 c8 .. of a segment of 256, into the segment's
// digit rows at `dig` (row 6 i + plane, 128 bytes each, 128-byte swizzle) and,
// by lanes 0..2 of the block's four, their scales into its two column tiles
// of `groups` row tiles each at `sf`.
__device__ __forceinline__ void store_digits(const uint32_t (&plane)[kDigits], uint32_t sb, int i, int c8,
                                             unsigned char* dig, unsigned char* sf, int groups) {
#pragma unroll
  for (int pl = 0; pl < kDigits; ++pl) {
    const int r = kDigits * i + pl;
    *reinterpret_cast<uint32_t*>(dig + r * 128 + (((c8 >> 2) ^ (r & 7)) << 4) + (c8 & 3) * 4) = plane[pl];
  }
  const int q = c8 & 3;
  if (q < kDigits / 2) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int pl = 2 * q + z, r = kDigits * i + pl;
      sf[((c8 >> 4) * groups + (r >> 7)) * kTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4 + ((c8 >> 2) & 3)] =
          (unsigned char)(sb == 255u ? 255u : sb + 3 * pl);
    }
  }
}

// Clusters of cs CTAs of `kernel` that the current device holds at once; 0 when
// the query fails.  Allows the kernel smem_max bytes of dynamic shared memory.
// The last kKept answers (device, kernel, sizes) are kept: the query takes
// longer than a small product.
inline int resident_clusters(void* kernel, int cs, int threads, int smem, int smem_max) {
  constexpr int kKept = 64;
  static std::mutex mu;
  static struct {
    int dev;
    void* k;
    int cs, smem, n;
  } kept[kKept];
  static int next = 0;  // a kernel of null: not yet written
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  for (const auto& c : kept)
    if (c.dev == dev && c.k == kernel && c.cs == cs && c.smem == smem) return c.n;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_max) != cudaSuccess)
    return 0;
  int n = sm_count();
  if (cs > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n / cs * cs);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
  }
  kept[next] = {dev, kernel, cs, smem, n};
  next = (next + 1) % kKept;
  return n;
}

}  // namespace mx4
}  // namespace qsm
