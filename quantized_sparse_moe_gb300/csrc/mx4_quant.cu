// Quantization to MXFP4 and back (layout in mx4_common.cuh).
//
//   s[r, b]    = 2^(floor(log2 max|x[r, 32b .. 32b+31]|) - 2), at least 2^-127
//   code[r, c] = the e2m1 value nearest to x[r, c] / s[r, c / 32], ties to
//                the even code, magnitudes over 6 become 6
//   y[r, c]    = code[r, c] * s[r, c / 32]
//
// Both are bound by memory: x once in, 4.25 bits a value out, and the
// reverse.  The scale is a power of two, so the division is exact and the one
// rounding is the one to the code.
//
// Eight lanes take the 128 columns of one column of scale tiles, of the four
// rows r, r + 32, r + 64 and r + 96 whose scales lie together in a tile: a lane
// has two chunks of eight columns of each, all its loads are under way at
// once, a block's maximum is two shuffles (16-bit ones two blocks at a time),
// and the sixteen scales are one load or store.
//
// Quantizing 4096 x 2048 bf16 takes 6.3 us of GPU time (3.4 TB/s, half of it
// launch and latency), 65536 x 2048 63 us (5.4 TB/s), 2050 x 1056 fp32 4.1, one
// row of 2048 1.6; dequantizing the same 5.6, 50.5 (6.7 TB/s), 4.1 and 1.4.
// One after the other, the bf16 sizes take 9.0 and (one row) 3.0, 2050 x 1056
// fp32 4.4.  Before, each group of lanes worked on
// one row with its own scale word, four such in turn: twice the address
// arithmetic and shuffles a value (4096 x 2048, both: 11.3; dequantizing 65536
// x 2048: 72).  CTAs of 128 threads: 14.3 for that, of 512 10.5, where 256 took
// 10.2.
#include "mx4_common.cuh"

namespace qsm {
namespace mx4 {
namespace {

constexpr int kThreads = 256;
constexpr size_t kMaxGroups = 1u << 28;  // of a call, eight lanes and 512 values each

// Eight columns of a row as raw words.
template <int DT>
struct Raw {
  uint4 v[DT == QSM_FP32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw<DT> load8(const char* p) {
  Raw<DT> r;
  r.v[0] = __ldg(reinterpret_cast<const uint4*>(p));
  if (DT == QSM_FP32) r.v[DT == QSM_FP32] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  return r;
}
template <int DT>
__device__ __forceinline__ void widen(const Raw<DT>& r, float (&v)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.v);
  if (DT == QSM_FP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else if (DT == QSM_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
// The fp32 bits of the largest magnitudes of a's and b's blocks, whose 32
// columns four lanes hold: magnitudes compare as integers, 16-bit ones two at
// a time.
template <int DT>
__device__ __forceinline__ uint2 block_max(const Raw<DT>& a, const Raw<DT>& b) {
  const uint32_t* wa = reinterpret_cast<const uint32_t*>(a.v);
  const uint32_t* wb = reinterpret_cast<const uint32_t*>(b.v);
  uint32_t ma = 0, mb = 0;
  if constexpr (DT == QSM_FP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ma = max(ma, wa[i] & 0x7fffffffu);
      mb = max(mb, wb[i] & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ma = max(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    }
    return make_uint2(ma, mb);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ma = __vmaxu2(ma, wa[i] & 0x7fff7fffu);
      mb = __vmaxu2(mb, wb[i] & 0x7fff7fffu);
    }
    uint32_t m = __vmaxu2(__byte_perm(ma, mb, 0x5410), __byte_perm(ma, mb, 0x7632));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (DT == QSM_BF16) return make_uint2(m << 16, m & 0xffff0000u);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return make_uint2(__float_as_uint(f.x), __float_as_uint(f.y));
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
mx4_quantize_kernel(const char* __restrict__ x, size_t row_bytes, uint32_t rows, uint32_t cols,
                    FastDiv cts, uint32_t groups, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales, int32_t* status) {
  constexpr int kSize = DT == QSM_FP32 ? 4 : 2;
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t g = (blockIdx.x * kThreads + threadIdx.x) >> 3, l = threadIdx.x & 7;
  if (g >= groups) return;  // whole warps: groups is a multiple of 32
  const uint32_t q = cts.div(g), ct = g - q * cts.d;
  const uint32_t r0 = (q >> 5) * kTileRows + (q & 31), c = ct * kTileCols + 8 * l;
  const char* src = x + (size_t)r0 * row_bytes + (size_t)c * kSize;
  const bool live[2] = {c < cols, c + 64 < cols};
  Raw<DT> raw[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      raw[k][h] = {};
      if (live[h] && r0 + 32 * k < rows) raw[k][h] = load8<DT>(src + (size_t)(32 * k) * row_bytes + 64 * kSize * h);
    }
  uint8_t* dst = codes + ((size_t)r0 * cols + c) / 2;
  uint32_t sw[4];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint2 m = block_max<DT>(raw[k][0], raw[k][1]);
    const uint32_t s[2] = {scale_of(m.x), scale_of(m.y)};
    bad |= s[0] == 255u || s[1] == 255u;
    sw[k] = (s[0] | s[1] << 16) << (8 * (l >> 2));
    sw[k] |= __shfl_xor_sync(0xffffffffu, sw[k], 4);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float inv = s[h] == 255u ? 0.f : inv_scale(s[h]);
      float v[8];
      widen<DT>(raw[k][h], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= inv;
      if (live[h] && r0 + 32 * k < rows)
        *reinterpret_cast<uint32_t*>(dst + (size_t)(16 * k) * cols + 32 * h) = f32x8_to_e2m1x8(v);
    }
  }
  if (l == 0) *reinterpret_cast<uint4*>(scales + scale_word(r0, ct, cts.d)) = make_uint4(sw[0], sw[1], sw[2], sw[3]);
  if (bad) set_status(status, QSM_DEV_NONFINITE);
}

// Two e2m1 codes (a byte, the first in the low nibble) as fp32 values.
__device__ __forceinline__ float2 code_values(uint32_t byte) {
  uint32_t h;
  asm("{\n .reg .b8 t, u, v, w;\n mov.b32 {t, u, v, w}, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
mx4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      uint32_t rows, FastDiv rts, uint32_t cols, FastDiv cts, uint32_t groups,
                      char* __restrict__ y) {
  constexpr int kSize = DT == QSM_FP32 ? 4 : 2;
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t g = (blockIdx.x * kThreads + threadIdx.x) >> 3, l = threadIdx.x & 7;
  if (g >= groups) return;
  const uint32_t q = cts.div(g), ct = g - q * cts.d, rt = q >> 5;  // rt: row tile of all experts
  const uint32_t e = rts.div(rt), r0 = (rt - e * rts.d) * kTileRows + (q & 31), c = ct * kTileCols + 8 * l;
  const uint4 sv = __ldg(reinterpret_cast<const uint4*>(scales + ((size_t)rt * cts.d + ct) * kTileBytes + (q & 31) * 16));
  const size_t at = ((size_t)e * rows + r0) * cols + c;  // the first value
  const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
  const bool live[2] = {c < cols, c + 64 < cols};
  uint32_t w[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[k][h] = 0;
      if (live[h] && r0 + 32 * k < rows)
        w[k][h] = __ldg(reinterpret_cast<const uint32_t*>(codes + at / 2 + (size_t)(16 * k) * cols + 32 * h));
    }
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float s = scale_value((sw[k] >> (16 * h + 8 * (l >> 2))) & 255u);
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f = code_values(w[k][h] >> (8 * i));
        f.x *= s;
        f.y *= s;
        if (DT == QSM_FP32) {
          v[2 * i] = __float_as_uint(f.x);
          v[2 * i + 1] = __float_as_uint(f.y);
        } else if (DT == QSM_BF16) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
          v[i] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
          const __half2 b = __floats2half2_rn(f.x, f.y);
          v[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      if (!live[h] || r0 + 32 * k >= rows) continue;
      uint4* dst = reinterpret_cast<uint4*>(y + (at + (size_t)(32 * k) * cols + 64 * h) * kSize);
      dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
      if (DT == QSM_FP32) dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

unsigned grid_for(size_t groups) { return (unsigned)((groups + kThreads / 8 - 1) / (kThreads / 8)); }

bool valid_dtype(int dt) { return dt == QSM_BF16 || dt == QSM_FP16 || dt == QSM_FP32; }

}  // namespace

// Whether w describes a matrix that the kernels can read: `experts` and the
// sizes positive, cols a multiple of 32, both arrays 16-byte aligned.
bool mx4_valid(const qsm_mx4* w) {
  return w && w->experts >= 1 && w->rows >= 1 && w->cols >= kBlock && w->cols % kBlock == 0 &&
         w->codes && w->scales && aligned16(w->codes) && aligned16(w->scales);
}

}  // namespace mx4
}  // namespace qsm

extern "C" size_t mx4_scale_bytes(int32_t rows, int32_t cols) {
  if (rows < 0 || cols < 0) return 0;
  return (size_t)qsm::mx4::row_tiles(rows) * qsm::mx4::col_tiles(cols) * qsm::mx4::kTileBytes;
}

extern "C" qsm_status mx4_quantize(const void* x, int32_t dtype, int64_t row_stride, int32_t rows,
                                   int32_t cols, uint8_t* codes, uint8_t* scales,
                                   int32_t* dev_status, cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::mx4;
  if (!valid_dtype(dtype) || rows < 0 || cols < kBlock || cols % kBlock || row_stride < cols ||
      row_stride % 8)
    return QSM_ERR_INVALID_ARGUMENT;
  if (rows == 0) return QSM_OK;
  if (!x || !codes || !scales || !dev_status || !aligned16(x) || !aligned16(codes) ||
      !aligned16(scales) || !aligned4(dev_status))
    return QSM_ERR_INVALID_ARGUMENT;
  const int cts = col_tiles(cols);
  const size_t groups = (size_t)row_tiles(rows) * 32 * cts;
  if (groups > kMaxGroups) return QSM_ERR_UNSUPPORTED;
  const dim3 grid(grid_for(groups));
  auto* kernel = dtype == QSM_BF16   ? mx4_quantize_kernel<QSM_BF16>
                 : dtype == QSM_FP16 ? mx4_quantize_kernel<QSM_FP16>
                                     : mx4_quantize_kernel<QSM_FP32>;
  QSM_CUDA_TRY(launch_pdl(kernel, grid, dim3(kThreads), 0, stream, static_cast<const char*>(x),
                          (size_t)row_stride * (dtype == QSM_FP32 ? 4 : 2), (uint32_t)rows,
                          (uint32_t)cols, FastDiv(cts), (uint32_t)groups, codes,
                          scales, dev_status));
  return QSM_OK;
}

extern "C" qsm_status mx4_dequantize(const qsm_mx4* a, int32_t dtype, void* y,
                                     cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::mx4;
  if (!a || !valid_dtype(dtype)) return QSM_ERR_INVALID_ARGUMENT;
  if (a->rows == 0 && a->experts >= 1) return QSM_OK;
  if (!mx4_valid(a) || !y || !aligned16(y)) return QSM_ERR_INVALID_ARGUMENT;
  const int cts = col_tiles(a->cols);
  const int rts = row_tiles(a->rows);
  const size_t groups = (size_t)a->experts * rts * 32 * cts;
  if (groups > kMaxGroups) return QSM_ERR_UNSUPPORTED;
  const dim3 grid(grid_for(groups));
  auto* kernel = dtype == QSM_BF16   ? mx4_dequantize_kernel<QSM_BF16>
                 : dtype == QSM_FP16 ? mx4_dequantize_kernel<QSM_FP16>
                                     : mx4_dequantize_kernel<QSM_FP32>;
  QSM_CUDA_TRY(launch_pdl(kernel, grid, dim3(kThreads), 0, stream, a->codes, a->scales,
                          (uint32_t)a->rows, FastDiv(rts), (uint32_t)a->cols, FastDiv(cts),
                          (uint32_t)groups, static_cast<char*>(y)));
  return QSM_OK;
}
