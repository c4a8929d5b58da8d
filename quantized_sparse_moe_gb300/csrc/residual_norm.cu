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
#include "mx4_common.cuh"

namespace qsm {
namespace rnorm {
namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxT = 1 << 30;
constexpr int kWarpRows = 4;       // rows of a CTA when a warp holds a row

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
  int xt, yt, gt, ht, gate_kind, sigmoid;
  float scale;
  Side post, pre;
  int32_t* status;
};

struct Raw {
  uint4 v[2];
};

__device__ __forceinline__ Raw load8(const char* row, int c, int type) {
  Raw r;
  if (type == QSM_FP32) {
    const uint4* p = reinterpret_cast<const uint4*>(row) + 2 * c;
    r.v[0] = p[0];
    r.v[1] = p[1];
  } else {
    r.v[0] = reinterpret_cast<const uint4*>(row)[c];
    r.v[1] = make_uint4(0, 0, 0, 0);
  }
  return r;
}

__device__ __forceinline__ void widen(const Raw& r, int type, float (&v)[8]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
  if (type == QSM_FP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else if (type == QSM_BF16) {
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

__device__ __forceinline__ void store8(char* row, int c, int type, const float (&v)[8]) {
  if (type == QSM_FP32) {
    float4* p = reinterpret_cast<float4*>(row) + 2 * c;
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint32_t w[4];
  if (type == QSM_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  reinterpret_cast<uint4*>(row)[c] = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the threads that hold the row.  Calls alternate between two
// buffers, so that one barrier a call is enough.
struct RowSum {
  float (*red)[32];
  int tpr, turn;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    float* r = red[turn];
    turn ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < (tpr >> 5) ? r[lane] : 0.f);
  }
};

// v <- n(v); live[i]: whether the thread has a chunk i (the others hold zeros).
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
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * step;
    if (c * 8 >= H) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= f;
    if (n.w) {
      const float4* w = reinterpret_cast<const float4*>(n.w) + 2 * c;
      const float4 a = __ldg(w), b = __ldg(w + 1);
      v[i][0] *= a.x, v[i][1] *= a.y, v[i][2] *= a.z, v[i][3] *= a.w;
      v[i][4] *= b.x, v[i][5] *= b.y, v[i][6] *= b.z, v[i][7] *= b.w;
    }
    if (n.b) {
      const float4* w = reinterpret_cast<const float4*>(n.b) + 2 * c;
      const float4 a = __ldg(w), b = __ldg(w + 1);
      v[i][0] += a.x, v[i][1] += a.y, v[i][2] += a.z, v[i][3] += a.w;
      v[i][4] += b.x, v[i][5] += b.y, v[i][6] += b.z, v[i][7] += b.w;
    }
  }
}

// The row's eight columns of chunk c as MXFP4 (mx4_common.cuh): four lanes
// hold a block, sixteen the four blocks of a scale word.  All lanes of a warp
// come here, those past the row with zeros.
__device__ __forceinline__ void store_mx4(const Params& p, int row, int c, const float (&v)[8], bool& bad) {
  const int lane = threadIdx.x & 31;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
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

// Threads of a row at most: 128 registers hold four chunks.
constexpr int max_threads(int v) { return v == 1 ? 1024 : 512; }

template <int V>
__global__ void __launch_bounds__(max_threads(V))
residual_norm_kernel(const __grid_constant__ Params p) {
  __shared__ float red[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int per = blockDim.x / p.tpr;  // rows of this CTA
  const int sub = per > 1 ? threadIdx.x >> 5 : 0;
  const int row = blockIdx.x * per + sub, c0 = threadIdx.x - sub * p.tpr, H = p.H;
  if (row >= p.rows) return;  // whole rows, and no barrier where a CTA has several
  if (row >= p.T) {           // past the last row of a scale tile: zero scales
    for (int ct = c0; ct < mx4::col_tiles(H); ct += p.tpr)
      *reinterpret_cast<uint32_t*>(p.hs + mx4::scale_word(row, ct, mx4::col_tiles(H))) = 0u;
    return;
  }
  RowSum sum{red, p.tpr, 0};
  const char* xr = p.x + (size_t)row * p.ldx;
  Raw xraw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    xraw[i] = {};
    if ((c0 + i * p.tpr) * 8 < H) xraw[i] = load8(xr, c0 + i * p.tpr, p.xt);
  }
  float v[V][8];
  if (p.y) {
    const char* yr = p.y + (size_t)row * p.ldy;
    Raw raw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      raw[i] = {};
      if ((c0 + i * p.tpr) * 8 < H) raw[i] = load8(yr, c0 + i * p.tpr, p.yt);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) widen(raw[i], p.yt, v[i]);
    normalize<V>(v, p.post, H, c0, p.tpr, sum);
    if (p.gate_kind != QSM_GATE_NONE) {
      const char* gr = p.gate + (size_t)row * p.ldg;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + i * p.tpr;
        if (c * 8 >= H) continue;
        float g[8];
        if (p.gate_kind == QSM_GATE_TOKENS) {
          float one;
          if (p.gt == QSM_FP32) one = *reinterpret_cast<const float*>(gr);
          else if (p.gt == QSM_BF16) one = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(gr));
          else one = __half2float(*reinterpret_cast<const __half*>(gr));
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = one;
        } else {
          widen(load8(gr, c, p.gt), p.gt, g);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= p.sigmoid ? 1.0f / (1.0f + expf(-g[j])) : g[j];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float x[8];
      widen(xraw[i], p.xt, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf(p.scale, v[i][j], x[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) widen(xraw[i], p.xt, v[i]);
  }
  if (p.xo) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((c0 + i * p.tpr) * 8 < H) store8(p.xo + (size_t)row * p.ldo, c0 + i * p.tpr, p.xt, v[i]);
  }
  if (!p.h) return;
  normalize<V>(v, p.pre, H, c0, p.tpr, sum);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * p.tpr;
    if (p.ht == QSM_MXFP4) store_mx4(p, row, c, v[i], bad);
    else if (c * 8 < H) store8(p.h + (size_t)row * p.ldh, c, p.ht, v[i]);
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

// T rows of `bytes` bytes, `ld` bytes apart.
struct Rows {
  const void* p;
  size_t ld, bytes;
};

// Whether rows of a and b have a byte in common.
bool overlap(const Rows& a, const Rows& b, int T) {
  if (!a.p || !b.p) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const size_t sa = (size_t)(T - 1) * a.ld + a.bytes, sb = (size_t)(T - 1) * b.ld + b.bytes;
  if (pa + sa <= pb || pb + sb <= pa) return false;
  if (a.ld != b.ld || a.ld == 0) return true;
  // columns side by side in one matrix
  const size_t d = pb >= pa ? (pb - pa) % a.ld : (a.ld - (pa - pb) % a.ld) % a.ld;
  return !(d >= a.bytes && d + b.bytes <= a.ld);
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.ld == b.ld && a.bytes == b.bytes; }

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
    return Rows{p, (T == 1 ? 0 : (size_t)ld) * size_of(type), (size_t)H * size_of(type)};
  };
  const Rows rx = rows(x, ldx, n->x_dtype), ry = rows(y, ldy, n->y_dtype), ro = rows(x_out, ldo, n->x_dtype);
  const Rows rh = mx ? Rows{h, (size_t)H / 2, (size_t)H / 2} : rows(h, ldh, n->h_dtype);
  const Rows rg = n->gate == QSM_GATE_TOKENS
                      ? Rows{gate, (size_t)ldg * size_of(n->gate_dtype), size_of(n->gate_dtype)}
                      : rows(gate, ldg, n->gate_dtype);
  const Rows all_scales = {mx && h ? h_scales : nullptr, 0, mx4_scale_bytes(T, H)};
  const auto H4 = [&](const float* p) { return Rows{p, 0, (size_t)H * 4}; };
  const Rows weights[4] = {H4(n->post.weight), H4(n->post.bias), H4(n->pre.weight), H4(n->pre.bias)};
  const Rows written[3] = {ro, rh, all_scales};
  for (int i = 0; i < 3; ++i) {
    const Rows& w = written[i];
    if ((overlap(w, rx, T) && !same(w, rx)) || (overlap(w, ry, T) && !same(w, ry)) || overlap(w, rg, T))
      return QSM_ERR_INVALID_ARGUMENT;
    for (const Rows& r : weights)
      if (overlap(w, r, T)) return QSM_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(w, written[j], T)) return QSM_ERR_INVALID_ARGUMENT;
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
  p.xt = n->x_dtype;
  p.yt = n->y_dtype;
  p.gt = n->gate_dtype;
  p.ht = n->h_dtype;
  p.gate_kind = n->gate;
  p.sigmoid = n->gate_sigmoid;
  p.scale = n->scale;
  p.post = {n->post.kind, n->post.eps, n->post.weight, n->post.bias};
  p.pre = {n->pre.kind, n->pre.eps, n->pre.weight, n->pre.bias};
  p.status = dev_status;
  // Few rows: one chunk a thread, the shortest way through a row; many rows:
  // as many chunks as registers hold, fewer barriers and more loads in flight.
  const int chunks = H / 8;
  int v = T <= mx4::sm_count() ? 1 : 4;
  while ((chunks + v - 1) / v > max_threads(v)) v *= 2;
  while (v > 1 && (chunks + v - 1) / v <= 16) v /= 2;
  p.tpr = ((chunks + v - 1) / v + 31) / 32 * 32;
  const int per = p.tpr == 32 ? kWarpRows : 1;
  const dim3 grid((p.rows + per - 1) / per), block(p.tpr * per);
  auto* kernel = v == 1 ? residual_norm_kernel<1> : v == 2 ? residual_norm_kernel<2> : residual_norm_kernel<4>;
  QSM_CUDA_TRY(launch_pdl(kernel, grid, block, 0, stream, p));
  return QSM_OK;
}
