// The MoE layer with MXFP4 weights: routing as in the other paths, the expert
// products in one of two ways, and the combine
//   y[t] = g[t] o_shared(t) + sum_j w[t, j] o(t, j)      (j ascending).
//
// QSM_ACTS_BF16 (few tokens): one launch for one or two (mx4_decode.cu); else
// gate_up + SwiGLU and down by the streaming kernel (mx4_stream.cu) over slots
// of up to 4 or 8 tokens of an expert, with activations of 16 bits and more; h and
// o are fp32.  Bound by the touched weights.
//
// QSM_ACTS_MX4 (many tokens): the token rows are quantized once and written
// to their places in the grouped order, each expert's rows padded to blocks
// of 128 (so that every block starts a scale tile); one grouped product
// forms h, quantized in its epilogue, and a second one o, in fp16 with a power of
// two per row and 128 columns (11 bits against the 8 of the bf16 result, at every
// magnitude; with a fixed 1/16 outputs lost bits below 2^-10 and were 0 below
// 2^-21).
//
// Every assignment's output is written once and the combine adds them in a
// fixed order, instead of reductions into y: the result does not depend on
// timing, and nothing has to be zeroed.  (The one launch has no combine: its
// order of sums is fixed too, but another one, see mx4_decode.cu.)
#include "mx4_decode.cuh"
#include "mx4_gemm.cuh"
#include "mx4_stream.cuh"

namespace qsm {
namespace dlayer {
extern int g_barrier_skew;  // qsm_debug_barrier_skew
}

namespace mx4 {
namespace {

constexpr int kPrepThreads = 256;
constexpr int kCombThreads = 128;
constexpr int kGatedThreads = 512;  // at most, with a shared gate
constexpr int kCombCols = 8;
constexpr int kCombCtas = 8;  // per SM: 64 registers; ten spilled and were slower
constexpr int kMaxK = 32;

// base[e] (shared memory): what takes a sorted position of expert e to its row
// when every expert's rows are padded to blocks of 128, the first at row
// 128 * first: 128 (first + blocks of the experts before) - offsets[e].
__device__ __forceinline__ void block_bases(const int32_t* counts, const int32_t* offsets, int E, int first,
                                            int* base) {
  __shared__ int warp_tot[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  int done = first;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + tid;
    const int v = e < E ? (__ldcg(counts + e) + 127) >> 7 : 0;
    const int off = e < E ? __ldcg(offsets + e) : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int before = done, all = done;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += warp_tot[w];
      all += warp_tot[w];
    }
    if (e < E) base[e] = 128 * (before + incl - v) - off;
    done = all;
    __syncthreads();
  }
}

// The tokens' rows in MXFP4, at every place where the grouped products read
// them: row t (shared expert), and for assignment (t, j) row
//   128 (shared_tiles + blocks of the experts before) + its rank in the expert,
// kept in pos[t k + j] for the combine (-1: no valid expert).  One warp takes
// 32 blocks (1024 columns) of a token, a block to a lane: x is read once, the
// maximum needs no other lane, and each of the k + 1 copies of a block's
// codes is one 16-byte store.  The lanes whose block starts a scale tile's
// row store the row's four scales.  Bound by the copies, 9 of 1.1 KB a token:
// 4096 tokens of 2048 with 8 experts each 15 us (57 MB, 3.7 TB/s).  CTAs that
// stay, with the next token's loads under way, made the layer 191.2 -> 187.8 us
// against one pass of as many CTAs as it takes.
__global__ void __launch_bounds__(kPrepThreads)
mx4_scatter_kernel(const uint16_t* __restrict__ x, int T, int k, int H, int E,
                   const int32_t* __restrict__ topk_idx, const int32_t* __restrict__ inv_perm,
                   const int32_t* __restrict__ counts, const int32_t* __restrict__ offsets,
                   int shared_tiles, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                   int32_t* __restrict__ pos, int32_t* status) {
  extern __shared__ int base[];  // [E]
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int cts = col_tiles(H), cgs = (H + 1023) / 1024;
  const int units = T * cgs, stride = gridDim.x * (kPrepThreads / 32);
  bool bad = false;
  // the next unit's loads are under way while one is worked on
  uint4 next[4];
  int next_e = 0, next_at = -1;
  auto fetch = [&](int u) {
    const int t = u / cgs, b = (u - t * cgs) * 32 + lane;
    const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)t * H + (b * kBlock < H ? b : 0) * kBlock);
#pragma unroll
    for (int i = 0; i < 4; ++i) next[i] = __ldg(src + i);
    if (lane < k) {
      next_e = __ldcg(topk_idx + (size_t)t * k + lane);
      next_at = __ldcg(inv_perm + (size_t)t * k + lane);
    }
  };
  int u = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
  if (u < units) fetch(u);
  block_bases(counts, offsets, E, shared_tiles, base);
  for (; u < units; u += stride) {
    const int t = u / cgs, cg = u - t * cgs, b = cg * 32 + lane;  // token, block
    const bool live = b * kBlock < H;
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = next[i];
    int dst = -1;  // lane j: the row of assignment (t, j)
    if (lane < k) {
      if (next_at >= 0 && next_e >= 0 && next_e < E) dst = base[next_e] + next_at;
      if (cg == 0) pos[(size_t)t * k + lane] = dst;
    }
    if (u + stride < units) fetch(u + stride);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      m = max(m, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
    const uint32_t s = scale_of(m);
    if (live && s == 255u) bad = true;
    const float inv = s == 255u ? 0.f : inv_scale(s);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(w[4 * i + j]) * inv;
        v[2 * j + 1] = bf16_hi(w[4 * i + j]) * inv;
      }
      c[i] = f32x8_to_e2m1x8(v);
    }
    const uint4 code = make_uint4(c[0], c[1], c[2], c[3]);
    uint32_t sw = s << (8 * (lane & 3));
    sw |= __shfl_xor_sync(0xffffffffu, sw, 1);
    sw |= __shfl_xor_sync(0xffffffffu, sw, 2);
    for (int j = -1; j < k; ++j) {
      const int r = j < 0 ? t : __shfl_sync(0xffffffffu, dst, j);
      if (r < 0 || !live) continue;
      reinterpret_cast<uint4*>(codes)[(size_t)r * (H / kBlock) + b] = code;
      if ((lane & 3) == 0) *reinterpret_cast<uint32_t*>(scales + scale_word(r, b >> 2, cts)) = sw;
    }
  }
  if (bad) set_status(status, QSM_DEV_NONFINITE);
}

// y[t] from the shared expert's output row and those of the token's
// assignments.  HALF: o holds fp16 to be multiplied with oscale [row, H / kOutCols],
// rows at[t k + j] and t; else fp32,
// rows t k + j (where at, the chosen expert, is valid) and T k + t.  A thread
// takes 8 columns of one token, with the loads of eight assignments in flight.
// Bound by reading o: 4096 tokens of 2048 with 8 experts each 35.5 us (168 MB in,
// 17 out, 5.2 TB/s), and 4 more for the powers of two.  A warp to 256 columns of a
// token took the layer from 197 to 212 us, column passes that keep o in L2 from
// 197.6 to 199.5, the powers by way of shared memory from 191.5 to 198.7 (spills).
//
// GATED: one CTA has a whole token, because y may be x: it has read all of x[t]
// for the gate when it writes y[t], and no other CTA reads x[t].  (The 128
// threads that add up x . shared_gate are those of an ungated CTA.)
template <bool HALF, bool GATED>
__global__ void __launch_bounds__(GATED ? kGatedThreads : kCombThreads,
                                  GATED ? (HALF ? 2 : 1) : (HALF ? kCombCtas : 4))
mx4_combine_kernel(const void* __restrict__ o, const float* __restrict__ oscale, const int32_t* __restrict__ at,
                   const float* __restrict__ topk_w, const uint16_t* x,
                   const float* __restrict__ sgate, int T, int k, int H, int E,
                   uint16_t* y, float* y32) {
  __shared__ int rows[kMaxK];
  __shared__ float wts[kMaxK], red[kCombThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int per = GATED ? 1 : (H / kCombCols + kCombThreads - 1) / kCombThreads;  // CTAs per token
  const int t = blockIdx.x / per, tid = threadIdx.x;
  if (tid < k) {
    const int r = __ldcg(at + (size_t)t * k + tid);
    rows[tid] = HALF ? r : (unsigned)r < (unsigned)E ? t * k + tid : -1;
    wts[tid] = __ldcg(topk_w + (size_t)t * k + tid);
  }
  float g = 1.f;
  if (GATED && tid < kCombThreads) {
    float z = 0.f;
    for (int c = tid; c < H; c += kCombThreads)
      z = fmaf(__uint_as_float((uint32_t)x[(size_t)t * H + c] << 16), __ldg(sgate + c), z);
    z = warp_sum(z);
    if ((tid & 31) == 0) red[tid >> 5] = z;
  }
  __syncthreads();
  if (GATED) {
    float z = 0.f;
#pragma unroll
    for (int w = 0; w < kCombThreads / 32; ++w) z += red[w];
    g = 1.0f / (1.0f + __expf(-z));
  }
  constexpr int NV = HALF ? 1 : 2;  // 16-byte loads per row
  struct Row {
    uint4 v[NV];
    float s;
  };
  auto columns = [&](const int c) {  // columns c .. c + 7 of y[t]
    auto load = [&](size_t row) {
      Row r;
      r.s = HALF ? __ldcg(oscale + row * (H / kOutCols) + c / kOutCols) : 1.f;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(o) + (row * H + c) * (HALF ? 2 : 4));
#pragma unroll
      for (int i = 0; i < NV; ++i) r.v[i] = __ldcg(src + i);
      return r;
    };
    auto add = [&](float (&s)[kCombCols], const Row& r, float w) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(r.v);
      if (HALF) w *= r.s;  // exact
#pragma unroll
      for (int i = 0; i < kCombCols; ++i) {
        float v;
        if (HALF) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(q + i / 2));
          v = i & 1 ? f.y : f.x;
        } else {
          v = __uint_as_float(q[i]);
        }
        s[i] = fmaf(w, v, s[i]);
      }
    };
    float s[kCombCols] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const Row first = load(HALF ? (size_t)t : (size_t)T * k + t);
    for (int j0 = 0; j0 < k; j0 += 8) {  // eight rows' loads in flight
      Row v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < k && rows[j0 + j] >= 0) v[j] = load((size_t)rows[j0 + j]);
      if (j0 == 0) add(s, first, g);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < k && rows[j0 + j] >= 0) add(s, v[j], wts[j0 + j]);
    }
    const size_t off = (size_t)t * H + c;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(s[2 * i], s[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(y + off) = make_uint4(w[0], w[1], w[2], w[3]);
    if (y32) {
      *reinterpret_cast<float4*>(y32 + off) = make_float4(s[0], s[1], s[2], s[3]);
      *reinterpret_cast<float4*>(y32 + off + 4) = make_float4(s[4], s[5], s[6], s[7]);
    }
  };
  if (GATED) {
    for (int c = tid * kCombCols; c < H; c += blockDim.x * kCombCols) columns(c);
  } else {
    const int c = (blockIdx.x % per * kCombThreads + tid) * kCombCols;
    if (c < H) columns(c);
  }
}

// ---------------------------------------------------------------------- host

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Everything a call keeps in its workspace.
struct Plan {
  int acts, tile_rows, shared_tiles, max_tiles;
  StreamParams gu, dn;      // QSM_ACTS_BF16: geometry
  bool one;                 // QSM_ACTS_BF16, few tokens: one launch
  DecodeParams dec;
  int dec_smem, dec_ctas;
  size_t rows;              // rows of h and o (BF16: T k + T; MX4: padded)
  size_t route, route_end, counts, offsets, perm, inv_perm, tile_map, n_tiles;
  size_t xc, xs, hc, hs, h, o, oscale, pos, total;
};

bool shape_ok(const qsm_mx4_layer* L) {
  return L && L->H >= 128 && L->H % 128 == 0 && L->H <= 16384 && L->I >= 128 && L->I % 128 == 0 &&
         L->I <= 16384 && L->E >= 1 && L->E <= 1024 && L->k >= 1 && L->k <= L->E && L->k <= kMaxK;
}

// Splits the acts argument: false when it is none of the values.
bool acts_of(int arg, int* acts, bool* one_launch) {
  *one_launch = (arg & QSM_ACTS_SEPARATE_LAUNCHES) == 0;
  *acts = arg & ~QSM_ACTS_SEPARATE_LAUNCHES;
  return *acts == QSM_ACTS_BF16 || (*acts == QSM_ACTS_MX4 && *one_launch);
}

bool plan_of(const qsm_mx4_layer* L, int T, int acts_arg, Plan* out) {
  int acts;
  bool one_launch;
  if (!shape_ok(L) || T < 1 || !acts_of(acts_arg, &acts, &one_launch)) return false;
  if ((long long)T * L->k > (1 << 24)) return false;
  const int H = L->H, I = L->I, E = L->E, k = L->k;
  Plan p = {};
  p.acts = acts;
  if (acts == QSM_ACTS_BF16 && one_launch && plan_decode(L, T, &p.dec, &p.dec_smem, &p.dec_ctas)) {
    p.one = true;
    p.total = decode_workspace_bytes(p.dec);
    *out = p;
    return true;
  }
  if (acts == QSM_ACTS_BF16) {
    if (T > QSM_MX4_MOE_MAX_ROWS) return false;
    const int touched = (long long)T * k < E ? T * k : E;
    bool fit = false;
    // Rows of a slot: a power of two, no more than the tokens need.  Four leave
    // more shared memory to the ring of weights, eight read the weights of an
    // expert with many tokens less often.  H 2048, I 512, four against eight (us):
    // 256 experts, 8 of them: T = 8 38.7 40.8, 16 50.7 51.9, 37 72.5 72.6, the
    // same with uneven routing: 24 41.0 40.2, 37 48.0 44.6, 64 65.3 58.4; 64
    // experts, 8: 16 38.2 40.3, 64 57.3 48.7; 8 experts, 2: 12 21.3 22.8.
    int tok = T <= 16 ? 4 : 8;
    while (tok > 1 && tok / 2 >= T) tok /= 2;
    for (; tok >= 1 && !fit; tok /= 2) {
      const int slots = touched + (T + tok - 1) / tok;
      p.gu.K = H;
      p.gu.N = 2 * I;
      p.dn.K = I;
      p.dn.N = H;
      fit = plan_rows(&p.gu, kRowsGateUp, slots * (I / 128), tok, sm_count()) &&
            plan_rows(&p.dn, kRowsDown, slots * (H / 128), tok, sm_count());
      p.tile_rows = tok;
    }
    if (!fit) return false;
  } else {
    p.tile_rows = 128;
  }
  p.shared_tiles = (T + p.tile_rows - 1) / p.tile_rows;
  p.max_tiles = moe_group_max_tiles(T, k, E, p.tile_rows);
  p.rows = acts == QSM_ACTS_BF16 ? (size_t)T * k + T : (size_t)(p.shared_tiles + p.max_tiles) * 128;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += up256(bytes);
    return at;
  };
  const size_t A = (size_t)T * k;
  p.route = take(moe_route_workspace_bytes(T, H, E));
  p.route_end = off;
  if (acts == QSM_ACTS_MX4) {
    p.counts = take((size_t)E * 4);
    p.offsets = take((size_t)(E + 1) * 4);
    p.perm = take(A * 4);
    p.inv_perm = take(A * 4);
    p.tile_map = take((size_t)p.max_tiles * 8);
    p.n_tiles = take(4);
  }
  if (acts == QSM_ACTS_BF16) {
    p.h = take(p.rows * I * 4);
    p.o = take(p.rows * H * 4);
  } else {
    p.xc = take(p.rows * H / 2);
    p.xs = take(mx4_scale_bytes((int)p.rows, H));
    p.hc = take(p.rows * I / 2);
    p.hs = take(mx4_scale_bytes((int)p.rows, I));
    p.o = take(p.rows * H * 2);
    p.oscale = take(p.rows * (H / kOutCols) * 4);
    p.pos = take(A * 4);
  }
  p.total = off;
  *out = p;
  return true;
}

bool weights_ok(const qsm_mx4& w, int experts, int rows, int cols) {
  return mx4_valid(&w) && w.experts == experts && w.rows == rows && w.cols == cols;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p < q + nb && q < p + na;
}

qsm_status few_tokens(const qsm_mx4_layer* L, const Plan& pl, const uint16_t* x, int T,
                      const int32_t* topk_idx, char* ws, int32_t* status, cudaStream_t stream) {
  const int H = L->H, I = L->I, E = L->E;
  StreamParams p = pl.gu;
  if (!make_codes_map(&p.w, L->gate_up.codes, (uint64_t)E * 2 * I, H, 128) ||
      !make_codes_map(&p.w_sh, L->shared_gate_up.codes, (uint64_t)2 * I, H, 128))
    return QSM_ERR_CUDA;
  p.w_scales = L->gate_up.scales;
  p.w_scales_sh = L->shared_gate_up.scales;
  p.ntiles = FastDiv(I / 128);
  p.T = T;
  p.k = L->k;
  p.I = I;
  p.H = H;
  p.topk_idx = topk_idx;
  p.E = E;
  p.k_div = FastDiv(L->k);
  p.tok_log = pl.tile_rows == 8 ? 3 : pl.tile_rows / 2;
  p.shared_tiles = pl.shared_tiles;
  p.x = x;
  p.ldx = H;
  p.h = reinterpret_cast<float*>(ws + pl.h);
  p.o = reinterpret_cast<float*>(ws + pl.o);
  p.status = status;
  StreamParams d = pl.dn;
  if (!make_codes_map(&d.w, L->down.codes, (uint64_t)E * H, I, 128) ||
      !make_codes_map(&d.w_sh, L->shared_down.codes, (uint64_t)H, I, 128))
    return QSM_ERR_CUDA;
  d.w_scales = L->down.scales;
  d.w_scales_sh = L->shared_down.scales;
  d.ntiles = FastDiv(H / 128);
  d.T = T;
  d.k = L->k;
  d.I = I;
  d.H = H;
  d.topk_idx = topk_idx;
  d.E = E;
  d.k_div = FastDiv(L->k);
  d.tok_log = pl.tile_rows == 8 ? 3 : pl.tile_rows / 2;
  d.shared_tiles = pl.shared_tiles;
  d.h = p.h;
  d.o = p.o;
  d.status = status;
  const int slots = pl.shared_tiles + pl.max_tiles;
  const qsm_status st = launch_rows(p, kRowsGateUp, slots * (I / 128), stream);
  return st != QSM_OK ? st : launch_rows(d, kRowsDown, slots * (H / 128), stream);
}

qsm_status one_launch(const qsm_mx4_layer* L, const Plan& pl, const uint16_t* x, const float* w_router,
                      const float* logit_bias, int flags, int32_t* topk_idx, float* topk_w, uint16_t* y,
                      float* y32, char* ws, int32_t* status, cudaStream_t stream) {
  const int H = L->H, I = L->I, E = L->E;
  DecodeParams p = pl.dec;
  if (!make_codes_map(&p.gu, L->gate_up.codes, (uint64_t)E * 2 * I, H, 128) ||
      !make_codes_map(&p.gu_sh, L->shared_gate_up.codes, (uint64_t)2 * I, H, 128) ||
      !make_codes_map(&p.dn, L->down.codes, (uint64_t)E * H, I, 128) ||
      !make_codes_map(&p.dn_sh, L->shared_down.codes, (uint64_t)H, I, 128))
    return QSM_ERR_CUDA;
  p.gu_sc = L->gate_up.scales;
  p.gu_sc_sh = L->shared_gate_up.scales;
  p.dn_sc = L->down.scales;
  p.dn_sc_sh = L->shared_down.scales;
  p.x = x;
  p.w_router = w_router;
  p.bias = logit_bias;
  p.sgate = L->shared_gate;
  p.flags = flags;
  p.skew = dlayer::g_barrier_skew;
  p.topk_idx = topk_idx;
  p.topk_w = topk_w;
  p.y = y;
  p.y32 = y32;
  p.ticket = reinterpret_cast<unsigned long long*>(ws);
  p.logits = reinterpret_cast<unsigned long long*>(ws + 256);
  p.h = reinterpret_cast<unsigned long long*>(ws + 256 + up256((size_t)p.T * E * 8));
  p.status = status;
  return launch_decode(p, pl.dec_smem, pl.dec_ctas, stream);
}

qsm_status many_tokens(const qsm_mx4_layer* L, const Plan& pl, const uint16_t* x, int T,
                       const int32_t* topk_idx, const qsm_grouping& g, char* ws, int32_t* status,
                       cudaStream_t stream) {
  const int H = L->H, I = L->I, E = L->E;
  uint8_t* xc = reinterpret_cast<uint8_t*>(ws + pl.xc);
  uint8_t* xs = reinterpret_cast<uint8_t*>(ws + pl.xs);
  const long long units = (long long)T * ((H + 1023) / 1024);
  const long long ctas = (units + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
  const int grid = (int)(ctas < 4ll * sm_count() ? ctas : 4ll * sm_count());
  QSM_CUDA_TRY(launch_pdl(mx4_scatter_kernel, dim3(grid), dim3(kPrepThreads), (size_t)E * 4, stream, x,
                          T, (int)L->k, H, E, topk_idx, (const int32_t*)g.inv_perm,
                          (const int32_t*)g.counts, (const int32_t*)g.offsets, pl.shared_tiles, xc, xs,
                          reinterpret_cast<int32_t*>(ws + pl.pos), status));
  GemmParams p = {};
  bool ok = make_a_maps(&p, xc, pl.rows, H) &&
            make_codes_map(&p.w, L->gate_up.codes, (uint64_t)E * 2 * I, H, 128) &&
            make_codes_map(&p.w_sh, L->shared_gate_up.codes, (uint64_t)2 * I, H, 128);
  p.a_scales = xs;
  p.w_scales = L->gate_up.scales;
  p.w_scales_sh = L->shared_gate_up.scales;
  p.N = 2 * I;
  p.K = H;
  p.nsub = I / 128;
  p.T = T;
  p.I = I;
  p.shared_tiles = pl.shared_tiles;
  p.offsets = g.offsets;
  p.tile_map = g.tile_map;
  p.n_tiles = g.n_tiles;
  p.h_codes = reinterpret_cast<uint8_t*>(ws + pl.hc);
  p.h_scales = reinterpret_cast<uint8_t*>(ws + pl.hs);
  p.status = status;
  GemmParams d = p;
  ok &= make_a_maps(&d, p.h_codes, pl.rows, I) &&
        make_codes_map(&d.w, L->down.codes, (uint64_t)E * H, I, kDownRows) &&
        make_codes_map(&d.w_sh, L->shared_down.codes, (uint64_t)H, I, kDownRows);
  if (!ok) return QSM_ERR_CUDA;
  d.a_scales = p.h_scales;
  d.w_scales = L->down.scales;
  d.w_scales_sh = L->shared_down.scales;
  d.N = H;
  d.K = I;
  d.nsub = (H + kDownRows - 1) / kDownRows;
  d.y = ws + pl.o;
  d.y_scale = reinterpret_cast<float*>(ws + pl.oscale);
  const qsm_status st = launch_grouped(p, kGateUp, pl.rows, stream);
  return st != QSM_OK ? st : launch_grouped(d, kDown, pl.rows, stream);
}

}  // namespace
}  // namespace mx4
}  // namespace qsm

extern "C" size_t moe_mx4_workspace_bytes(const qsm_mx4_layer* L, int32_t T, int32_t acts) {
  qsm::mx4::Plan p;
  return qsm::mx4::plan_of(L, T, acts, &p) ? p.total : 0;
}

extern "C" qsm_status moe_mx4_forward(const qsm_mx4_layer* L, const uint16_t* x, int32_t T,
                                      int32_t acts, const float* w_router, const float* logit_bias,
                                      int32_t flags, int32_t* topk_idx, float* topk_w, uint16_t* y,
                                      float* y_f32, void* workspace, size_t workspace_bytes,
                                      int32_t* dev_status, cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::mx4;
  int kind;
  bool one;
  if (!L || T < 0 || !acts_of(acts, &kind, &one) ||
      (flags & ~(QSM_ROUTE_RENORMALIZE | QSM_ROUTE_BIAS_SELECT_ONLY)))
    return QSM_ERR_INVALID_ARGUMENT;
  if (!shape_ok(L)) return QSM_ERR_UNSUPPORTED;
  if (T == 0) return QSM_OK;
  if (!x || !w_router || !topk_idx || !topk_w || !y || !workspace || !dev_status || !aligned16(x) ||
      !aligned16(w_router) || !aligned16(workspace) || !aligned16(topk_idx) || !aligned16(topk_w) ||
      !aligned16(y) || (y_f32 && !aligned16(y_f32)) || !aligned4(dev_status) ||
      (logit_bias && !aligned4(logit_bias)) || (L->shared_gate && !aligned16(L->shared_gate)))
    return QSM_ERR_INVALID_ARGUMENT;
  if (!weights_ok(L->gate_up, L->E, 2 * L->I, L->H) || !weights_ok(L->down, L->E, L->H, L->I) ||
      !weights_ok(L->shared_gate_up, 1, 2 * L->I, L->H) || !weights_ok(L->shared_down, 1, L->H, L->I))
    return QSM_ERR_INVALID_ARGUMENT;
  // y may be x, but x is read until y is written
  const size_t n = (size_t)T * L->H;
  if (L->shared_gate && ((y != x && overlap(y, n * 2, x, n * 2)) || (y_f32 && overlap(y_f32, n * 4, x, n * 2))))
    return QSM_ERR_INVALID_ARGUMENT;
  Plan p;
  if (!plan_of(L, T, acts, &p)) return QSM_ERR_UNSUPPORTED;
  if (workspace_bytes < p.total) return QSM_ERR_WORKSPACE_TOO_SMALL;
  char* ws = static_cast<char*>(workspace);
  if (p.one)
    return one_launch(L, p, x, w_router, logit_bias, flags, topk_idx, topk_w, y, y_f32, ws, dev_status, stream);
  auto i32 = [&](size_t off) { return reinterpret_cast<int32_t*>(ws + off); };
  const qsm_grouping g = {i32(p.counts),   i32(p.offsets), i32(p.perm), i32(p.inv_perm),
                          i32(p.tile_map), i32(p.n_tiles), p.tile_rows, p.max_tiles};
  const size_t route_bytes = p.route_end - p.route;
  const bool half = kind == QSM_ACTS_MX4;
  qsm_status st = moe_route(x, w_router, logit_bias, T, L->H, L->E, L->k, flags, topk_idx, topk_w,
                            ws + p.route, route_bytes, dev_status, stream);
  if (st == QSM_OK && half) st = moe_group_tokens(topk_idx, T, L->k, L->E, &g, dev_status, stream);
  if (st != QSM_OK) return st;
  st = half ? many_tokens(L, p, x, T, topk_idx, g, ws, dev_status, stream)
            : few_tokens(L, p, x, T, topk_idx, ws, dev_status, stream);
  if (st != QSM_OK) return st;
  const bool gated = L->shared_gate != nullptr;
  int threads = kCombThreads;
  if (gated) {
    const int all = (L->H / kCombCols + 31) / 32 * 32;
    threads = all < kCombThreads ? kCombThreads : all < kGatedThreads ? all : kGatedThreads;
  }
  const dim3 grid((unsigned)T * (gated ? 1 : (L->H / kCombCols + kCombThreads - 1) / kCombThreads));
  auto* comb = half ? (gated ? mx4_combine_kernel<true, true> : mx4_combine_kernel<true, false>)
                    : (gated ? mx4_combine_kernel<false, true> : mx4_combine_kernel<false, false>);
  QSM_CUDA_TRY(launch_pdl(comb, grid, dim3(threads), 0, stream, (const void*)(ws + p.o),
                          (const float*)(ws + p.oscale), half ? (const int32_t*)i32(p.pos) : (const int32_t*)topk_idx,
                          (const float*)topk_w, x, L->shared_gate, T, (int)L->k, (int)L->H, (int)L->E, y, y_f32));
  return QSM_OK;
}
