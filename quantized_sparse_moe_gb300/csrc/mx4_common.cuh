// MXFP4: 4-bit floating-point codes (e2m1: sign, two exponent bits, one
// mantissa bit; 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one power-of-two scale
// (e8m0: 2^(s - 127), 255 = not a number) per block of 32 columns, and the
// tensor-core building blocks that multiply them without expanding them.
//
// Layout of a matrix [rows, cols] (cols a multiple of 32):
//   codes   [rows, cols / 2] bytes, column 2c in the low nibble of byte c
//   scales  tiles of 128 rows x 4 blocks (128 columns), 512 bytes each, in
//           order [row tile][column tile]; byte 16 (r % 32) + 4 (r / 32) + b
//           of a tile is the scale of row r, block b.  This is the order in
//           which the tensor cores take scales (32 lanes x 16 bytes), so a
//           tile goes from global to shared to tensor memory as it is.  Rows
//           and blocks past the matrix are padded with the byte 0: their
//           codes read as 0, and 0 x 2^-127 adds nothing (255 would make
//           the sum not a number).
#pragma once

#include "tc_common.cuh"

namespace qsm {
namespace mx4 {

constexpr int kBlock = 32;        // columns per scale
constexpr int kTileRows = 128;    // rows of a scale tile
constexpr int kTileCols = 128;    // columns of a scale tile
constexpr int kTileBytes = 512;
constexpr int kStageK = 256;      // columns per pipeline stage: 128 bytes of codes a row

// (any size up to 2^31 - 1)
__host__ __device__ inline int col_tiles(int cols) { return cols / kTileCols + (cols % kTileCols != 0); }
__host__ __device__ inline int k_stages(int cols) { return cols / kStageK + (cols % kStageK != 0); }
__host__ __device__ inline int row_tiles(int rows) { return rows / kTileRows + (rows % kTileRows != 0); }

// Byte offset, within a matrix's scale tiles, of the four scales of row r
// in column tile ct.
__host__ __device__ inline size_t scale_word(int r, int ct, int cts) {
  return ((size_t)(r >> 7) * cts + ct) * kTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Division of n < 2^31 by a divisor fixed at launch, by one multiplication
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct FastDiv {
  uint32_t d, m, l;
  __host__ FastDiv(uint32_t div = 1) : d(div), m(0), l(0) {
    while ((1ull << l) < d) ++l;
    m = (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> l; }
};

// A shared-memory box (swizzled as `map` says) to global memory; parts
// outside the tensor are left out.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's stores have read their shared memory / have been written.
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// --------------------------------------------------------------- e2m1 codes

// Eight values (already divided by the block's scale) to eight codes, the
// first in the lowest nibble: round to nearest, ties to the even code,
// magnitudes over 6 become 6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The scale byte of a block whose largest magnitude has these fp32 bits:
// two binades below it (e2m1's largest value is 1.5 x 2^2), at least 2^-127;
// 255 when the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return e >= 255 ? 255u : (uint32_t)max(e - 2, 0);
}
// 1 / 2^(s - 127): exact, for every s that scale_of gives but 255.
__device__ __forceinline__ float inv_scale(uint32_t s) {
  return __uint_as_float((254u - s) << 23);
}
// 2^(s - 127), NaN for s = 255 (2^-127 is subnormal).
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// ------------------------------------------------- block-scaled tensor cores

// Shared-memory descriptor of a scale tile for the copy into tensor memory:
// no swizzle, four groups of 8 rows x 16 bytes, 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(128u >> 4) << 16;
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  return d;
}

// One scale tile (512 bytes) into four tensor-memory columns, repeated in
// each of the four 32-lane quarters: column c, lane l holds the four scales
// of row 32 c + l.  Ordered before the MMAs this thread issues later.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"(scale_desc(saddr))
               : "memory");
}

// Instruction descriptor, kind::mxf4: e2m1 A and B (K-major), e8m0 scales
// per 32, fp32 D, M = 128, N = n (a multiple of 8, at most 256).  `half`
// picks which two of a column tile's four blocks the 64-wide step uses.
__device__ __forceinline__ uint32_t idesc_mxf4(int n, int half) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(128 >> 4) << 24) | ((uint32_t)(2 * half) << 29) |
         ((uint32_t)(2 * half) << 4);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 consecutive 32-bit columns of this warp's 32 lanes, without the wait.
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
// The loads into r[0..31] have arrived: the registers pass through the wait,
// so that nothing reads them before it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// ------------------------------------------------- one thread of a warp

using tc::elect_one;
// A value that all lanes hold, as a uniform one.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// ----------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrive on the mbarrier at cluster address `addr`; this thread's (and,
// through a preceding __syncwarp, its warp's) stores before it are visible
// to whoever waits for the phase.
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// ------------------------------------------------------------ bounded waits

// Bounded mbarrier wait shared by all roles of a CTA: gives up when the
// abort flag is set or the limit runs out (then sets the flag and the
// device status).
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                              int32_t* status) {
  for (uint32_t i = 0; i < kWaitIters; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  set_status(status, QSM_DEV_TIMEOUT);
  return false;
}

// The same by all lanes of a warp, as one decision.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int32_t* status) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, status));
}
__device__ __forceinline__ bool warp_aborted(volatile int* abort_flag) {
  return __any_sync(0xffffffffu, *abort_flag != 0);
}

// The waits again, for barriers that other CTAs of the cluster arrive on.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             int32_t* status) {
  for (uint32_t i = 0; i < kWaitIters; ++i) {
    if (try_wait_cluster(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  set_status(status, QSM_DEV_TIMEOUT);
  return false;
}

// ---------------------------------------------------------------------- host

inline int sm_count() {
  static int n[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (n[dev] == 0) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    n[dev] = v > 0 ? v : 152;
  }
  return n[dev];
}

// The codes [rows, cols / 2] as a tensor map of 128-byte x box_rows boxes
// with the 128-byte swizzle; columns and rows outside read as 0.
inline bool make_codes_map(CUtensorMap* m, const void* codes, uint64_t rows, int cols,
                           uint32_t box_rows) {
  return tc::make_map_2d(m, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, (uint64_t)cols / 2,
                         128, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows of `bytes` bytes in memory, `ld` bytes apart; one row, or ld 0: a vector.
struct Rows {
  const void* p;
  size_t n, ld, bytes;
};

// Whether rows of a and b may have a byte in common.  Exact for rows of the same
// stride and for a vector beside rows; true for others whose extents meet.
inline bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const size_t lda = a.n > 1 ? a.ld : 0, ldb = b.n > 1 ? b.ld : 0;
  if (pa + (a.n - 1) * lda + a.bytes <= pb || pb + (b.n - 1) * ldb + b.bytes <= pa) return false;
  const size_t ld = lda ? lda : ldb;
  if (!ld || (lda && ldb && lda != ldb)) return true;
  // b's place in a row of a, up to whole rows; in a column of their own they do not meet
  const size_t d = pb >= pa ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;
  return !(d >= a.bytes && d + b.bytes <= ld);
}

}  // namespace mx4
}  // namespace qsm
