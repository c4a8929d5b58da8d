// Activations as base-8 digit planes in e2m1 (the mathematics is in
// mx4_stream.cu), and what the kernels that use them share on the host.
#pragma once

#include <mutex>

#include "kept_answers.cuh"
#include "mx4_common.cuh"

namespace qsm {
namespace mx4 {

constexpr int kDigits = 6;
constexpr uint32_t kDigitBias = 149796u;  // sum of 4 * 8^i, i < 6

// Rows of the MMA's digit operand for n rows of x.
__host__ __device__ constexpr int digit_rows(int n) { return (kDigits * n + 7) / 8 * 8; }

__device__ __forceinline__ uint32_t select_bytes(uint32_t lo, uint32_t hi, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(lo), "r"(hi), "r"(sel));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The digits are bound by integer instructions, of which the packing of two
// columns a word, the table and the fused rounding save a third (16 x 19456 x
// 2048: 15.5 -> 13.3 us; two groups of eight at a time gave nothing).
//
// The digit planes of eight values as e2m1 codes (one word each), and the
// scale byte of plane 0 (plane i: + 3 i; 255: not a number).  Lanes 4 j ..
// 4 j + 3 hold the four quarters of a block.
__device__ __forceinline__ uint32_t digits_of(const float (&v)[8], uint32_t (&plane)[kDigits]) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(v[j]));
  uint32_t m = __float_as_uint(top);  // a NaN: above every number
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  // E, at least -111 so that 2^(15 - E) is finite; 127 and up (2^127,
  // infinities, NaN) have no scale for their top digit
  const int e = max((int)(m >> 23) - 127, -111);
  const bool bad = e >= 127;
  const float f = __uint_as_float((uint32_t)(15 - (bad ? 0 : e) + 127) << 23);
  // X + kDigitBias in the low 18 bits: the sum lies between 2^23 and 2^24, where
  // fp32 holds integers, so the fused operation rounds v f to the nearest one
  // (ties to even: the constant is even).  Where bad, the digits do not matter.
  uint32_t y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = __float_as_uint(fmaf(v[j], f, 12582912.f + (float)kDigitBias));
  // bits 0..15 (digits 0 to 4) of two neighbours in a word, and bits 8..23
  uint32_t low[4], high[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    low[k] = select_bytes(y[2 * k], y[2 * k + 1], 0x5410u);
    high[k] = select_bytes(y[2 * k], y[2 * k + 1], 0x6521u);
  }
#pragma unroll
  for (int i = 0; i < kDigits; ++i) {
    // the unsigned digits 0..7 of the even columns, one per nibble, and of the
    // odd ones in the upper half: selectors from a table of the codes of digit - 4
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t from = i < 5 ? low[k] : high[k];
      const int sh = (i < 5 ? 3 * i : 7) - 4 * k;
      w |= (sh >= 0 ? from >> (sh & 31) : from << (-sh & 31)) & (0x00070007u << (4 * k));
    }
    plane[i] = select_bytes(0x090A0B0Cu, 0x03020100u, w) | select_bytes(0x90A0B0C0u, 0x30201000u, w >> 16);
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
// Answers are kept: a program with several projections and a varying number of
// rows asks for hundreds of geometries in turn.
inline int resident_clusters(void* kernel, int cs, int threads, int smem, int smem_max) {
  static std::mutex mu;
  static KeptAnswers kept;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (kept.find(dev, kernel, cs, smem, &n)) return n;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_max) != cudaSuccess)
    return 0;
  n = sm_count();
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
  kept.put(dev, kernel, cs, smem, n);
  return n;
}

}  // namespace mx4
}  // namespace qsm
