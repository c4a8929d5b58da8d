// The residual stream around a block, in one pass over the rows:
//
//   d  = gate * post(y)            y: the block's output
//   x' = x + scale * d             rounded once, when it is stored
//   h  = pre(x')                   of the unrounded x'; stored in 16 or 32 bits or as MXFP4
//
//   RMS:    n(v) = w v / sqrt(mean(v^2) + eps)  (+ b)
//   layer:  n(v) = w (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps)  (+ b)
//
// Everything between the loads and the stores is fp32 in registers: a row is
// held by the threads of one CTA (or by one warp), V chunks of eight columns
// each, so mean and variance take a pass each over registers, not over
// memory, and the variance is that of the centred values.
//
// Bound by memory for many rows, by latency and the launch for few.  Measured (GPU time
// of a replayed call, inputs rotating over more than L2 where they are large):
//   1 x 2048 bf16 2.1 us; 300 x 2048 with a gate to MXFP4 (and dequantized again) 5.6
//   4096 x 2048 bf16, both norms 15.0 us = 4.5 TB/s, 16384 x 2048 45.0 = 6.0 TB/s: 4 us of a
//     launch are its first rows' latency, ten rows an SM at once, and the last ones
//   2050 x 1056 fp32 x, bf16 y and gate, layer norm with a bias 9.0 us = 3.4 TB/s; the same
//   4096 x 2048 bf16 to MXFP4 13.8 us, with a norm on either side 16.6, 16384 rows 39.9
#include "mx4_common.cuh"

namespace qsm {
namespace rnorm {
namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxT = 1 << 30;
constexpr int kWarpRows = 4;       // rows of a CTA when a warp holds a row
constexpr size_t kBuffers = 216 * 1024;        // shared memory of the many-row kernel
constexpr long long kManyValues = 3 << 19;

struct Side {  // a norm
  int kind;
  float eps;
  const float* w;
  const float* b;
};

struct Params {
  const char* x;
  const char* y;
  const char* gate;
  char* xo;
  char* h;
  uint8_t* hs;
  size_t ldx, ldy, ldg, ldo, ldh;  // bytes from row to row
  int T, rows, H, tpr;             // rows: T, or up to a whole scale tile
  int gt, ht, gate_kind, sigmoid;
  float scale;
  Side post, pre;
  int32_t* status;
};

// Eight columns as they lie in memory.
template <int DT>
struct Raw {
  uint4 v[DT == QSM_FP32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Raw<DT> load8(const char* row, int c) {
  Raw<DT> r;
  const uint4* p = reinterpret_cast<const uint4*>(row) + (DT == QSM_FP32 ? 2 : 1) * c;
  r.v[0] = *p;
  if (DT == QSM_FP32) r.v[DT == QSM_FP32] = p[1];
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

template <int DT>
__device__ __forceinline__ void store8(char* row, int c, const float (&v)[8]) {
  if constexpr (DT == QSM_FP32) {
    float4* p = reinterpret_cast<float4*>(row) + 2 * c;
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == QSM_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    reinterpret_cast<uint4*>(row)[c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Sum over the threads that hold the row.  Calls alternate between two
// buffers, so that one barrier a call is enough.
struct RowSum {
  float (*red)[32];
  int tpr, turn, bar;  // the hardware barrier of these threads, 0: the CTA's
  __device__ __forceinline__ void sync() const {
    if (tpr == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
  }
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    float* r = red[turn];
    turn ^= 1;
    const int lane = threadIdx.x & 31, warps = tpr >> 5;
    if (lane == 0) r[(threadIdx.x >> 5) % warps] = v;
    sync();
    return warp_sum(lane < warps ? r[lane] : 0.f);
  }
};

// Eight fp32 of a vector (in global memory, or in the CTA's shared memory).
__device__ __forceinline__ void eight(const float* p, int c, float (&u)[8]) {
  const float4* at = reinterpret_cast<const float4*>(p) + 2 * c;
  const float4 a = at[0], b = at[1];
  u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w, u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
}

// v <- n(v); chunks past the row hold zeros and stay so.
template <int V>
__device__ __forceinline__ void normalize(float (&v)[V][8], const Side& n, int H, int c0, int step, RowSum& sum) {
  if (n.kind == QSM_NORM_NONE) return;
  if (n.kind == QSM_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[i][j];
    const float mean = sum(s) / (float)H;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((c0 + i * step) * 8 < H)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) q = fmaf(v[i][j], v[i][j], q);
  const float f = __frsqrt_rn(sum(q) / (float)H + n.eps);
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= f;
  if (n.w) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((c0 + i * step) * 8 < H) {
        float u[8];
        eight(n.w, c0 + i * step, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= u[j];
      }
  }
  if (n.b) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((c0 + i * step) * 8 < H) {
        float u[8];
        eight(n.b, c0 + i * step, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += u[j];
      }
  }
}

// The row's eight columns of chunk c as MXFP4 (mx4_common.cuh): four lanes
// hold a block, sixteen the four blocks of a scale word.  All lanes of a warp
// come here; those past the row stand for blocks of zeros (what they hold is NaN
// when the row is).
__device__ __forceinline__ void store_mx4(const Params& p, int row, int c, const float (&v)[8], bool& bad) {
  const int lane = threadIdx.x & 31;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  if (c * 8 >= p.H) m = 0;
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t s = mx4::scale_of(m);
  bad |= s == 255u;
  uint32_t sw = s << (8 * ((lane >> 2) & 3));
  sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
  sw |= __shfl_xor_sync(0xffffffffu, sw, 8);
  if (c * 8 >= p.H) return;
  const float inv = s == 255u ? 0.f : mx4::inv_scale(s);
  float u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = v[j] * inv;
  reinterpret_cast<uint32_t*>(p.h + (size_t)row * p.ldh)[c] = mx4::f32x8_to_e2m1x8(u);
  if ((lane & 15) == 0)
    *reinterpret_cast<uint32_t*>(p.hs + mx4::scale_word(row, c >> 4, mx4::col_tiles(p.H))) = sw;
}

// v *= gate (of whatever type); gr: the row's values, or value.
template <int V, int DT>
__device__ __forceinline__ void apply_gate(const Params& p, const char* gr, int c0, float (&v)[V][8]) {
  const auto value = [&](float g) { return p.sigmoid ? 1.0f / (1.0f + expf(-g)) : g; };
  if (p.gate_kind == QSM_GATE_TOKENS) {
    float one;
    if (DT == QSM_FP32) one = *reinterpret_cast<const float*>(gr);
    else if (DT == QSM_BF16) one = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(gr));
    else one = __half2float(*reinterpret_cast<const __half*>(gr));
    one = value(one);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= one;
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * p.tpr;
    if (c * 8 >= p.H) continue;
    float g[8];
    widen<DT>(load8<DT>(gr, c), g);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= value(g[j]);
  }
}

template <int V, int DT>
__device__ __forceinline__ void store_row(char* row, int H, int c0, int step, const float (&v)[V][8]) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    if ((c0 + i * step) * 8 < H) store8<DT>(row, c0 + i * step, v[i]);
}

// Between the loads and the stores of one row: v holds y (or, without y, x)
// on entry; x(i, u) gives the row's x of chunk i.
template <int V, int XT, typename GetX, typename Read>
__device__ __forceinline__ void one_row(const Params& p, const Side& post, const Side& pre, const char* gate, int row, int c0, float (&v)[V][8], RowSum& sum, bool& bad,
                                        GetX x, Read read) {
  const int H = p.H;
  if (p.y) {
    normalize<V>(v, post, H, c0, p.tpr, sum);
    if (p.gate_kind != QSM_GATE_NONE) {
      if (p.gt == QSM_BF16) apply_gate<V, QSM_BF16>(p, gate, c0, v);
      else if (p.gt == QSM_FP32) apply_gate<V, QSM_FP32>(p, gate, c0, v);
      else apply_gate<V, QSM_FP16>(p, gate, c0, v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float u[8];
      x(i, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf(p.scale, v[i][j], u[j]);
    }
  }
  read();  // the row's inputs are in registers
  if (p.xo) store_row<V, XT>(p.xo + (size_t)row * p.ldo, H, c0, p.tpr, v);
  if (!p.h) return;
  normalize<V>(v, pre, H, c0, p.tpr, sum);
  char* hr = p.h + (size_t)row * p.ldh;
  if (p.ht == QSM_MXFP4) {
#pragma unroll
    for (int i = 0; i < V; ++i) store_mx4(p, row, c0 + i * p.tpr, v[i], bad);
  } else if (p.ht == QSM_BF16) {
    store_row<V, QSM_BF16>(hr, H, c0, p.tpr, v);
  } else if (p.ht == QSM_FP32) {
    store_row<V, QSM_FP32>(hr, H, c0, p.tpr, v);
  } else {
    store_row<V, QSM_FP16>(hr, H, c0, p.tpr, v);
  }
}

// Whether the gate has a row for each token.
__host__ __device__ inline bool gate_rows(const Params& p) { return p.gate_kind == QSM_GATE_ROWS && p.ldg != 0; }

// Zero scales of a row past the last one of a scale tile.
__device__ __forceinline__ void pad_row(const Params& p, int row, int c0) {
  for (int ct = c0; ct < mx4::col_tiles(p.H); ct += p.tpr)
    *reinterpret_cast<uint32_t*>(p.hs + mx4::scale_word(row, ct, mx4::col_tiles(p.H))) = 0u;
}

// Few rows: a CTA (for short rows, a warp) has one, a thread eight columns of it.
template <int XT, int YT>
__global__ void __launch_bounds__(1024)
row_kernel(const __grid_constant__ Params p) {
  __shared__ float red[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int per = blockDim.x / p.tpr;  // rows of this CTA
  const int sub = per > 1 ? threadIdx.x >> 5 : 0, row = blockIdx.x * per + sub, c0 = threadIdx.x - sub * p.tpr;
  if (row >= p.rows) return;  // whole rows, and no barrier where a CTA has several
  if (row >= p.T) return pad_row(p, row, c0);
  RowSum sum{red, p.tpr, 0, 0};
  Raw<XT> xraw = {};
  Raw<YT> yraw = {};
  if (c0 * 8 < p.H) {
    xraw = load8<XT>(p.x + (size_t)row * p.ldx, c0);
    if (p.y) yraw = load8<YT>(p.y + (size_t)row * p.ldy, c0);
  }
  float v[1][8];
  bool bad = false;
  if (p.y) widen<YT>(yraw, v[0]);
  else widen<XT>(xraw, v[0]);
  one_row<1, XT>(p, p.post, p.pre, p.gate + (size_t)row * p.ldg, row, c0, v, sum, bad, [&](int, float (&u)[8]) { widen<XT>(xraw, u); }, [] {});
  if (bad) set_status(p.status, QSM_DEV_NONFINITE);
}

// Many rows: a CTA per SM, groups of tpr threads that take row after row.  Each
// group has a buffer in shared memory, which bulk copies fill with the next
// row (x, y and the gate) as soon as the present one is in registers; the
// norms' vectors lie beside them.  Four chunks a thread and up to twenty groups
// (4096 x 2048 15.0 us; eight chunks, whose rows of 2048 are a warp's without a barrier, and twelve
// groups 16.3, 4096 x 5120 32 against 44).
constexpr int kRowsThreads = 640, kMaxGroups = kRowsThreads / 32, kChunks = 4;

template <int XT, int YT>
__global__ void __launch_bounds__(kRowsThreads, 1)
rows_kernel(const __grid_constant__ Params p, int groups, int vectors) {
  constexpr int V = kChunks;
  extern __shared__ __align__(128) unsigned char buffers[];
  __shared__ float red[kMaxGroups][2][32];
  __shared__ __align__(8) uint64_t full[kMaxGroups], vec_bar;
  __shared__ int abort_flag;
  constexpr int kX = XT == QSM_FP32 ? 4 : 2, kY = YT == QSM_FP32 ? 4 : 2;
  const int g = threadIdx.x / p.tpr, c0 = threadIdx.x - g * p.tpr, H = p.H;
  const uint32_t xb = (uint32_t)H * kX, yb = p.y ? (uint32_t)H * kY : 0u;
  const uint32_t gb = gate_rows(p) ? (uint32_t)H * (p.gt == QSM_FP32 ? 4 : 2) : 0u, bytes = xb + yb + gb;
  if (threadIdx.x == 0) {
    for (int i = 0; i < groups; ++i) mbar_init(&full[i], 1);
    mbar_init(&vec_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  // the norms' vectors, once per CTA, before the rows (which would hold them up)
  Side post = p.post, pre = p.pre;
  if (vectors) {
    unsigned char* at = buffers + (size_t)groups * bytes;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&vec_bar, (uint32_t)vectors * H * 4);
    const auto keep = [&](const float*& src) {
      if (!src) return;
      if (threadIdx.x == 0) bulk_g2s(at, src, (uint32_t)H * 4, &vec_bar);
      src = reinterpret_cast<const float*>(at);
      at += (size_t)H * 4;
    };
    keep(post.w);
    keep(post.b);
    keep(pre.w);
    keep(pre.b);
    __syncthreads();
  }
  unsigned char* mine = buffers + (size_t)g * bytes;
  const int stride = gridDim.x * groups;
  uint32_t issued = 0;  // copies that this thread has asked for
  const auto fetch = [&](int row) {
    ++issued;
    mbar_arrive_expect_tx(&full[g], bytes);
    bulk_g2s(mine, p.x + (size_t)row * p.ldx, xb, &full[g]);
    if (yb) bulk_g2s(mine + xb, p.y + (size_t)row * p.ldy, yb, &full[g]);
    if (gb) bulk_g2s(mine + xb + yb, p.gate + (size_t)row * p.ldg, gb, &full[g]);
  };
  int row = blockIdx.x * groups + g;
  if (c0 == 0 && row < p.T) fetch(row);
  // a copy that never comes: the rows go on with what is there, no more are
  // asked for, and the call is reported
  volatile int* abort_p = &abort_flag;
  if (vectors) mx4::wait_or_abort(&vec_bar, 0, abort_p, p.status);
  RowSum sum{red[g], p.tpr, 0, g + 1};
  bool bad = false;
  const char* xs = reinterpret_cast<const char*>(mine);
  const char* ys = xs + xb;
  for (uint32_t parity = 0; row < p.T; row += stride, parity ^= 1) {
    mx4::wait_or_abort(&full[g], parity, abort_p, p.status);
    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + i * p.tpr;
      if (p.y) {
        Raw<YT> y = {};
        if (c * 8 < H) y = load8<YT>(ys, c);
        widen<YT>(y, v[i]);
      } else {
        Raw<XT> x = {};
        if (c * 8 < H) x = load8<XT>(xs, c);
        widen<XT>(x, v[i]);
      }
    }
    one_row<V, XT>(p, post, pre, gb ? ys + yb : p.gate + (size_t)row * p.ldg, row, c0, v, sum, bad,
                   [&](int i, float (&u)[8]) {
                     Raw<XT> x = {};
                     if ((c0 + i * p.tpr) * 8 < H) x = load8<XT>(xs, c0 + i * p.tpr);
                     widen<XT>(x, u);
                   },
                   [&] {
                     sum.sync();
                     if (c0 == 0 && row + (long long)stride < p.T && !*abort_p) fetch(row + stride);
                   });
  }
  for (; row < p.rows; row += stride) pad_row(p, row, c0);
  if (*abort_p) {  // the copies in flight land before the CTA leaves
    if (issued) mbar_wait_bounded(&full[g], (issued - 1) & 1, kWaitIters);
    if (vectors) mbar_wait_bounded(&vec_bar, 0, kWaitIters);
  }
  if (bad) set_status(p.status, QSM_DEV_NONFINITE);
}

bool dtype_ok(int t) { return t == QSM_BF16 || t == QSM_FP16 || t == QSM_FP32; }
size_t size_of(int t) { return t == QSM_FP32 ? 4 : 2; }

bool norm_ok(const qsm_norm& n) {
  if (n.kind == QSM_NORM_NONE) return !n.weight && !n.bias;
  return (n.kind == QSM_NORM_RMS || n.kind == QSM_NORM_LAYER) && n.eps >= 0.f && n.eps < INFINITY &&
         (!n.weight || aligned16(n.weight)) && (!n.bias || aligned16(n.bias));
}

using mx4::Rows;
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.ld == b.ld && a.bytes == b.bytes; }

// Which kernel.  The few-row one has many warps on an SM and starts at once, but
// each of them goes through a row's latencies alone.  From 1.5 M values on the
// other is faster (bf16, both norms, us, few rows' kernel and the other: 1 M values as 512 x 2048 4.6 4.7,
// 1.5 M 6.0 5.2, 2 M 7.0 5.5, 3 M 9.0 8.3, 6 M 17.3 13.5; 192 x 8192 7.8 6.2; with a gate for each value
// and fp32 h 768 x 2048 7.3 7.3, 1024 8.6 7.6), unless five eighths of its lanes' chunks lie past the row
// (4096 x 384 6.5 6.5; 6144 x 256 4.7 8.5).
template <int XT, int YT>
qsm_status launch(Params& p, cudaStream_t stream) {
  const int chunks = p.H / 8, sms = mx4::sm_count();
  const auto threads = [&](int v) { return ((chunks + v - 1) / v + 31) / 32 * 32; };
  const bool many = (long long)p.T * p.H >= kManyValues && 8 * chunks >= 3 * kChunks * threads(kChunks);
  if (!many && chunks <= 1024) {
    p.tpr = threads(1);
    const int per = p.tpr == 32 ? kWarpRows : 1;
    QSM_CUDA_TRY(launch_pdl(row_kernel<XT, YT>, dim3((p.rows + per - 1) / per), dim3(p.tpr * per), 0, stream, p));
    return QSM_OK;
  }
  p.tpr = threads(kChunks);
  const size_t row = (size_t)p.H * ((XT == QSM_FP32 ? 4 : 2) + (p.y ? YT == QSM_FP32 ? 4 : 2 : 0) +
                                    (gate_rows(p) ? p.gt == QSM_FP32 ? 4 : 2 : 0));
  int groups = kRowsThreads / p.tpr;
  while (groups > 1 && groups * row > kBuffers) --groups;
  // as few groups as take no more rounds (4096 x 2048, three rounds: nine 15.0 us, ten 15.4, eleven 16.4)
  const int rounds = (p.T + groups * sms - 1) / (groups * sms);
  groups = (p.T + rounds * sms - 1) / (rounds * sms);
  int ctas = (p.rows + groups - 1) / groups;
  if (ctas > sms) ctas = sms;
  int vectors = (p.post.w != nullptr) + (p.post.b != nullptr) + (p.pre.w != nullptr) + (p.pre.b != nullptr);
  if (groups * row + (size_t)vectors * p.H * 4 > kBuffers) vectors = 0;  // they stay in global memory
  const size_t smem = groups * row + (size_t)vectors * p.H * 4;
  auto* kernel = rows_kernel<XT, YT>;
  QSM_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBuffers));
  QSM_CUDA_TRY(launch_pdl(kernel, dim3(ctas), dim3(p.tpr * groups), smem, stream, p, groups, vectors));
  return QSM_OK;
}

}  // namespace
}  // namespace rnorm
}  // namespace qsm

extern "C" qsm_status residual_norm(const qsm_residual_norm* n, int32_t T, const void* x, int64_t ldx,
                                    const void* y, int64_t ldy, const void* gate, int64_t ldg,
                                    void* x_out, int64_t ldo, void* h, int64_t ldh, uint8_t* h_scales,
                                    int32_t* dev_status, cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::rnorm;
  if (!n || T < 0 || n->H < 8 || n->H % 8) return QSM_ERR_INVALID_ARGUMENT;
  const int H = n->H;
  const bool mx = n->h_dtype == QSM_MXFP4;
  if (!dtype_ok(n->x_dtype) || (y && !dtype_ok(n->y_dtype)) || !norm_ok(n->post) || !norm_ok(n->pre) ||
      !(n->scale > -INFINITY && n->scale < INFINITY))
    return QSM_ERR_INVALID_ARGUMENT;
  if (n->gate < QSM_GATE_NONE || n->gate > QSM_GATE_TOKENS || (n->gate_sigmoid & ~1) ||
      (n->gate == QSM_GATE_NONE) != (gate == nullptr) || (gate && (!y || !dtype_ok(n->gate_dtype))))
    return QSM_ERR_INVALID_ARGUMENT;
  if (h && (n->pre.kind == QSM_NORM_NONE || (!mx && !dtype_ok(n->h_dtype)) || (mx && H % mx4::kBlock)))
    return QSM_ERR_INVALID_ARGUMENT;
  if (H > kMaxH || T > kMaxT) return QSM_ERR_UNSUPPORTED;
  if (T == 0) return QSM_OK;
  if (!x || (!h && !x_out) || (h && mx && (!h_scales || !dev_status))) return QSM_ERR_INVALID_ARGUMENT;
  const auto rows_ok = [&](const void* p, int64_t ld, int64_t unit) {
    return !p || (aligned16(p) && (T == 1 || (ld >= H && ld % unit == 0)));
  };
  const auto unit = [](int t) { return t == QSM_FP32 ? 4 : 8; };
  if (!rows_ok(x, ldx, unit(n->x_dtype)) || !rows_ok(y, ldy, unit(n->y_dtype)) ||
      !rows_ok(x_out, ldo, unit(n->x_dtype)) || (h && !mx && !rows_ok(h, ldh, unit(n->h_dtype))) ||
      (mx && h && (!aligned16(h) || !aligned16(h_scales))) || (dev_status && !aligned4(dev_status)))
    return QSM_ERR_INVALID_ARGUMENT;
  if (gate) {
    const size_t g = size_of(n->gate_dtype);
    if (n->gate == QSM_GATE_ROWS ? !(aligned16(gate) && (T == 1 || ldg == 0 || (ldg >= H && ldg % unit(n->gate_dtype) == 0)))
                                 : (reinterpret_cast<uintptr_t>(gate) % g || ldg < 0))
      return QSM_ERR_INVALID_ARGUMENT;
  }
  // x_out and h may be x or y (a thread reads its columns of both before it
  // writes them); nothing that is written may be read or written otherwise
  const auto rows = [&](const void* p, int64_t ld, int type) {
    return Rows{p, (size_t)T, (T == 1 ? 0 : (size_t)ld) * size_of(type), (size_t)H * size_of(type)};
  };
  const Rows rx = rows(x, ldx, n->x_dtype), ry = rows(y, ldy, n->y_dtype), ro = rows(x_out, ldo, n->x_dtype);
  const Rows rh = mx ? Rows{h, (size_t)T, (size_t)H / 2, (size_t)H / 2} : rows(h, ldh, n->h_dtype);
  const Rows rg = n->gate == QSM_GATE_TOKENS
                      ? Rows{gate, (size_t)T, (size_t)ldg * size_of(n->gate_dtype), size_of(n->gate_dtype)}
                      : rows(gate, ldg, n->gate_dtype);
  const auto vec = [](const void* p, size_t bytes) { return Rows{p, 1, 0, bytes}; };
  const size_t H4 = (size_t)H * 4;
  const Rows weights[4] = {vec(n->post.weight, H4), vec(n->post.bias, H4), vec(n->pre.weight, H4), vec(n->pre.bias, H4)};
  const Rows written[3] = {ro, rh, vec(mx && h ? h_scales : nullptr, mx4_scale_bytes(T, H))};
  using mx4::overlap;
  for (int i = 0; i < 3; ++i) {
    const Rows& w = written[i];
    if ((overlap(w, rx) && !same(w, rx)) || (overlap(w, ry) && !same(w, ry)) || overlap(w, rg))
      return QSM_ERR_INVALID_ARGUMENT;
    for (const Rows& r : weights)
      if (overlap(w, r)) return QSM_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(w, written[j])) return QSM_ERR_INVALID_ARGUMENT;
  }
  Params p = {};
  p.x = static_cast<const char*>(x);
  p.y = static_cast<const char*>(y);
  p.gate = static_cast<const char*>(gate);
  p.xo = static_cast<char*>(x_out);
  p.h = static_cast<char*>(h);
  p.hs = h_scales;
  p.ldx = rx.ld;
  p.ldy = ry.ld;
  p.ldg = rg.ld;
  p.ldo = ro.ld;
  p.ldh = rh.ld;
  p.T = T;
  p.rows = mx && h ? mx4::row_tiles(T) * mx4::kTileRows : T;
  p.H = H;
  p.gt = n->gate_dtype;
  p.ht = n->h_dtype;
  p.gate_kind = n->gate;
  p.sigmoid = n->gate_sigmoid;
  p.scale = n->scale;
  p.post = {n->post.kind, n->post.eps, n->post.weight, n->post.bias};
  p.pre = {n->pre.kind, n->pre.eps, n->pre.weight, n->pre.bias};
  p.status = dev_status;
  switch (3 * n->x_dtype + (y ? n->y_dtype : n->x_dtype)) {
    case 0: return launch<QSM_BF16, QSM_BF16>(p, stream);
    case 1: return launch<QSM_BF16, QSM_FP16>(p, stream);
    case 2: return launch<QSM_BF16, QSM_FP32>(p, stream);
    case 3: return launch<QSM_FP16, QSM_BF16>(p, stream);
    case 4: return launch<QSM_FP16, QSM_FP16>(p, stream);
    case 5: return launch<QSM_FP16, QSM_FP32>(p, stream);
    case 6: return launch<QSM_FP32, QSM_BF16>(p, stream);
    case 7: return launch<QSM_FP32, QSM_FP16>(p, stream);
    default: return launch<QSM_FP32, QSM_FP32>(p, stream);
  }
}
