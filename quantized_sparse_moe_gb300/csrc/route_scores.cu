// Routing by scores.  With l = x W^T (fp32 accuracy), for each token
//
//   s[e] = exp(l[e]) / sum_e' exp(l[e'])   or   1 / (1 + exp(-l[e])),
//   c[e] = s[e] + bias[e],
//
// the experts lie in G equal groups, a group is worth the sum of its best one
// or two c; the best groups stay (ties to the lower index), of their experts
// the k with the largest c (ties to the lower index) are taken in descending
// c, and weighted with s, divided by the sum over the taken ones if asked
// for, times a factor.
//
// The logits are a tensor-core product over an exact three-way bf16 split of
// the fp32 weights (hi, mid, lo: 3 x 8 bits of the 24; bf16 x makes every
// product exact), accumulated in fp32.  The experts are the MMA's 128 rows
// and the tokens its N, so that a tile takes 16 to 256 tokens: few tokens
// share a tile and the weights are split over many SMs, many tokens make
// large tiles that read the weights less often.  hi and mid + lo have an
// accumulator each: the small parts are not cut off at the size of the sum,
// and the sum collects a third of the roundings.
//
// A cluster of KS x MB CTAs has one tile of tokens: CTA (q, m) computes the
// logits of experts 128 m .. 128 m + 127 over slice q of H.  The partial
// logits go to shared memory, and after a cluster barrier each CTA takes its
// share of the tile's tokens: a warp reads a token's slices through
// distributed shared memory, adds them in slice order, and selects.  The
// call needs no workspace and leaves nothing behind.
#include "mx4_common.cuh"

namespace qsm {
qsm_status route_split_launch(const float* w, size_t n, void* out, cudaStream_t stream);

namespace rscores {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int BM = 128;                  // experts of a CTA
constexpr int BK = 64;
constexpr int kPartBytes = BM * BK * 2;  // one part of the weights
constexpr int kMaxE = 512, kMaxK = 32, kMaxGroups = 32;
constexpr int kMaxStages = 4;
constexpr int kRowFloats = BM + 4;       // of a token's partial logits
constexpr int kEpiWarp = 4;              // first of eight (or four) warps that read the accumulators

struct Params {
  CUtensorMap x;  // [T, H] bf16, box {64, nt}
  CUtensorMap w;  // [3 E, H] bf16, box {64, 128}
  const float* bias;
  int T, H, E, k, nt, ks, stages;
  int sigmoid, groups, kept, best, gsize, renorm;
  float scale;
  int32_t* idx;
  float* wts;
  int32_t* status;
};

// bf16 A and B (K-major), fp32 D, M = 128.
__device__ __forceinline__ uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// The larger and the second largest of two pairs, each in order.
__device__ __forceinline__ void best_two(float& a, float& b, float c, float d) {
  b = fmaxf(fminf(a, c), fmaxf(b, d));
  a = fmaxf(a, c);
}

// Sorts N = 4 or 8 descending (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_desc(unsigned long long* c) {
  cas_desc(c[0], c[1]); cas_desc(c[2], c[3]);
  cas_desc(c[0], c[2]); cas_desc(c[1], c[3]);
  cas_desc(c[1], c[2]);
  if constexpr (N == 8) {
    cas_desc(c[4], c[5]); cas_desc(c[6], c[7]);
    cas_desc(c[4], c[6]); cas_desc(c[5], c[7]);
    cas_desc(c[5], c[6]);
    cas_desc(c[0], c[4]); cas_desc(c[1], c[5]); cas_desc(c[2], c[6]); cas_desc(c[3], c[7]);
    cas_desc(c[2], c[4]); cas_desc(c[3], c[5]);
    cas_desc(c[1], c[2]); cas_desc(c[3], c[4]); cas_desc(c[5], c[6]);
  }
}

// One token by one warp.  l: its logits, expert 128 m + 4 lane + j at
// l[4 m + j]; sc: the warp's scratch [E]; grp: the groups of the lane's
// experts.
template <int MB>
__device__ __forceinline__ void select_token(const Params& p, float (&l)[4 * MB], const int (&grp)[4 * MB],
                                             float* sc, int lane, size_t t) {
  constexpr int N = 4 * MB;
  constexpr uint32_t kAll = 0xffffffffu;
  const auto expert = [&](int i) { return 128 * (i >> 2) + 4 * lane + (i & 3); };
  bool bad = false;
  uint32_t fine = 0;  // finite logits of experts that exist
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = expert(i) < p.E, ok = isfinite(l[i]);
    if (in && ok) fine |= 1u << i;
    bad |= in && !ok;
  }
  float s[N];
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = (fine >> i) & 1u ? 1.0f / (1.0f + expf(-l[i])) : 0.f;
  } else {
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((fine >> i) & 1u) top = fmaxf(top, l[i]);
    top = warp_max(top);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = (fine >> i) & 1u ? expf(l[i] - top) : 0.f;
      sum += s[i];
    }
    sum = warp_sum(sum);
    if (sum > 0.f) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] /= sum;
    }
  }
  float c[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = expert(i);
    c[i] = -INFINITY;
    if ((fine >> i) & 1u) {
      c[i] = p.bias ? s[i] + __ldg(p.bias + e) : s[i];
      if (!(c[i] < INFINITY)) {  // a bias that is +infinity or NaN
        bad = true;
        c[i] = -INFINITY;
      }
    }
  }
  if (__any_sync(kAll, bad) && lane == 0) set_status(p.status, QSM_DEV_NONFINITE);

  uint32_t keep = kAll;  // bit g: group g stays
  if (p.kept < p.groups) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (expert(i) < p.E) sc[expert(i)] = c[i];
    __syncwarp();
    // `per` lanes a group (a power of two) look through its experts, from
    // different places so that their reads fall into different banks
    int per = 32;
    while (per * p.groups > 32) per >>= 1;
    const int g = lane / per, q = lane - g * per;
    float a = -INFINITY, b = -INFINITY;
    if (g < p.groups)
      for (int j = q, at = (q + g) % p.gsize; j < p.gsize; j += per) {
        best_two(a, b, sc[g * p.gsize + at], -INFINITY);
        at += per;
        if (at >= p.gsize) at %= p.gsize;
      }
    for (int o = 1; o < per; o <<= 1) {
      const float c2 = __shfl_xor_sync(kAll, a, o), d2 = __shfl_xor_sync(kAll, b, o);
      best_two(a, b, c2, d2);
    }
    const float value = p.best == 2 ? a + b : a;
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const float v = __shfl_sync(kAll, value, o * per);
      rank += v > value || (v == value && o < g);
    }
    const uint32_t in = __ballot_sync(kAll, g < p.groups && q == 0 && rank < p.kept);
    keep = 0;
    for (int o = 0; o < p.groups; ++o) keep |= ((in >> (o * per)) & 1u) << o;
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (expert(i) < p.E) sc[expert(i)] = s[i];

  unsigned long long key[N];  // (order of c, ~expert): a strict order; 0 where there is none
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = expert(i) < p.E && ((keep >> grp[i]) & 1u);
    key[i] = in ? ((unsigned long long)order_key(c[i]) << 32) | (uint32_t)~expert(i) : 0ull;
  }
  constexpr int kList = N < 8 ? N : 8;
#pragma unroll
  for (int n = 0; n < N; n += kList) sort_desc<kList>(key + n);
  int my_e = 0;
  float my_c = -INFINITY;
  for (int j = 0; j < p.k; ++j) {
    unsigned long long head = key[0];
    if constexpr (N > 8) head = key[0] > key[8] ? key[0] : key[8];
    const uint32_t hk = (uint32_t)(head >> 32), hi = (uint32_t)head;
    const uint32_t mk = __reduce_max_sync(kAll, hk);
    const uint32_t mi = __reduce_max_sync(kAll, hk == mk ? hi : 0u);
    if (hk == mk && hi == mi) {  // this lane's: drop it
      if (N <= 8 || key[0] == head) {
#pragma unroll
        for (int i = 0; i < kList - 1; ++i) key[i] = key[i + 1];
        key[kList - 1] = 0ull;
      } else {
#pragma unroll
        for (int i = N - kList; i < N - 1; ++i) key[i] = key[i + 1];
        key[N - 1] = 0ull;
      }
    }
    if (lane == j) {
      my_c = key_value(mk);
      my_e = (int)~mi;
    }
  }
  __syncwarp();
  float w = 0.f;
  if (lane < p.k && my_c > -INFINITY) w = sc[my_e];  // a closed expert has weight 0
  if (p.renorm) {
    const float sum = warp_sum(w);
    w = sum > 0.f ? w / sum : 0.f;
  }
  if (lane < p.k) {
    p.idx[t * p.k + lane] = my_e;
    p.wts[t * p.k + lane] = w * p.scale;
  }
  __syncwarp();
}

template <int MB>
__global__ void __launch_bounds__(kThreads, 1)
route_scores_kernel(const __grid_constant__ Params p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int warp = mx4::uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int cta = (int)mx4::cluster_rank(), q = cta / MB, m = cta - q * MB;
  const int nt = p.nt, csize = p.ks * MB, tile = blockIdx.x / csize;
  const int stage_bytes = 3 * kPartBytes + nt * BK * 2;
  const int cols = nt < 16 ? 32 : 2 * nt;  // of tensor memory
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&done_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    tc::prefetch_map(&p.x);
    tc::prefetch_map(&p.w);
  }
  if (warp == 1) tc::tmem_alloc(&tmem_base, cols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = mx4::uniform(tmem_base);
  pdl_wait();
  pdl_launch_dependents();
  volatile int* abort_p = &abort_flag;
  const int all = p.H / BK, first = (int)((long long)all * q / p.ks);
  const int steps = (int)((long long)all * (q + 1) / p.ks) - first;

  if (warp == 0) {
    int st = 0;
    for (int s = 0, round = 0; st < steps; ++st) {
      if (round > 0 && !mx4::warp_wait(&empty_bar[s], (round - 1) & 1, abort_p, p.status)) break;
      if (mx4::warp_aborted(abort_p)) break;
      if (tc::elect_one()) {
        unsigned char* sb = smem + s * stage_bytes;
        mbar_arrive_expect_tx(&full_bar[s], stage_bytes);
#pragma unroll
        for (int part = 0; part < 3; ++part)
          tc::tma_load_2d(sb + part * kPartBytes, &p.w, (first + st) * BK, part * p.E + m * BM, &full_bar[s]);
        tc::tma_load_2d(sb + 3 * kPartBytes, &p.x, (first + st) * BK, tile * nt, &full_bar[s]);
      }
      __syncwarp();
      if (++s == p.stages) {
        s = 0;
        ++round;
      }
    }
    if (mx4::warp_aborted(abort_p))  // the copies in flight land before the CTA leaves
      for (int i = st > p.stages ? st - p.stages : 0; i < st; ++i)
        mbar_wait_bounded(&full_bar[i % p.stages], (i / p.stages) & 1, kWaitIters);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16(nt);
    int st = 0;
    for (int s = 0, round = 0; st < steps; ++st) {
      if (!mx4::warp_wait(&full_bar[s], round & 1, abort_p, p.status)) break;
      tc::tc_fence_after();
      if (tc::elect_one()) {
        const uint32_t a0 = smem_u32(smem + s * stage_bytes), b0 = a0 + 3 * kPartBytes;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint64_t b = tc::sw128_desc(b0 + kk * 32);
          const uint32_t more = st > 0 || kk > 0;
          tc::mma_f16(tmem + nt, tc::sw128_desc(a0 + 2 * kPartBytes + kk * 32), b, idesc, more);
          tc::mma_f16(tmem + nt, tc::sw128_desc(a0 + kPartBytes + kk * 32), b, idesc, 1u);
          tc::mma_f16(tmem, tc::sw128_desc(a0 + kk * 32), b, idesc, more);
        }
        tc::mma_commit(&empty_bar[s]);
        if (st == steps - 1) tc::mma_commit(&done_bar);
      }
      __syncwarp();
      if (++s == p.stages) {
        s = 0;
        ++round;
      }
    }
    if (st < steps) {  // gave up: the MMAs in flight end before tensor memory is freed
      if (tc::elect_one()) tc::mma_commit(&done_bar);
      __syncwarp();
      mbar_wait_bounded(&done_bar, 0, kWaitIters);
    }
  } else if (warp >= kEpiWarp && warp < kEpiWarp + 8) {
    // lane = expert, column = token: to [token][expert], over the stages
    // (every MMA has completed)
    const int quarter = warp & 3, half = (warp - kEpiWarp) >> 2;
    const bool ok = mx4::warp_wait(&done_bar, 0, abort_p, p.status);
    tc::tc_fence_after();
    float* out = reinterpret_cast<float*>(smem) + 32 * quarter + lane;
    const uint32_t taddr = tmem + ((uint32_t)(32 * quarter) << 16);
    if (ok) {
      for (int c = 16 * half; c < nt; c += 32) {
        uint32_t hi[16], lo[16];
        tc::tmem_ld16_nowait(taddr + c, hi);
        tc::tmem_ld16_nowait(taddr + nt + c, lo);
        tc::tmem_wait_ld(hi, lo);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          out[(c + i) * kRowFloats] = __uint_as_float(hi[i]) + __uint_as_float(lo[i]);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, cols);
  }
  cluster_sync_all();  // every slice of the tile is in its CTA's shared memory

  // a CTA that gave up leaves no logits: its flag is read with them
  const int per = nt / csize, rows = min(nt, p.T - tile * nt);
  int aborted = 0;
  for (int r = 0; r < csize; ++r) {
    int f;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(f) : "r"(dsmem_addr(&abort_flag, r)) : "memory");
    aborted |= f;
  }
  if (!aborted) {
    int grp[4 * MB];
#pragma unroll
    for (int i = 0; i < 4 * MB; ++i) grp[i] = min((128 * (i >> 2) + 4 * lane + (i & 3)) / p.gsize, 31);
    float* sc = reinterpret_cast<float*>(smem + (size_t)nt * kRowFloats * 4) + warp * p.E;
    for (int i = warp; i < per; i += kWarps) {
      const int row = cta * per + i;
      if (row >= rows) break;
      float l[4 * MB];
      const uint32_t at = smem_u32(smem) + (row * kRowFloats + 4 * lane) * 4;
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        float4 a = dsmem_ld_f4(dsmem_addr_u32(at, b));
        for (int s = 1; s < p.ks; ++s) {
          const float4 v = dsmem_ld_f4(dsmem_addr_u32(at, s * MB + b));
          a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
        l[4 * b] = a.x, l[4 * b + 1] = a.y, l[4 * b + 2] = a.z, l[4 * b + 3] = a.w;
      }
      select_token<MB>(p, l, grp, sc, lane, (size_t)tile * nt + row);
    }
  }
  cluster_sync_all();  // no CTA leaves while another still reads its slices
}

// ---------------------------------------------------------------------- host

struct Config {
  int nt, ks, stages;
  size_t smem;
};

constexpr size_t kSmem = 220 * 1024;  // dynamic, of the 227 KB; the rest is static

// Stages and shared memory of a tile of nt tokens.
bool fit(int nt, int E, Config* c) {
  const size_t stage = 3 * kPartBytes + (size_t)nt * BK * 2;
  const size_t rows = (size_t)nt * kRowFloats * 4 + (size_t)kWarps * E * 4;  // over the stages, later
  if (rows + 1024 > kSmem) return false;
  int stages = (int)((kSmem - 1024) / stage);
  c->nt = nt;
  c->stages = stages < kMaxStages ? stages : kMaxStages;
  const size_t ring = (size_t)c->stages * stage;
  c->smem = (ring > rows ? ring : rows) + 1024;
  return c->stages >= 2;
}

int row_blocks(int E) { return E <= BM ? 1 : E <= 2 * BM ? 2 : 4; }

bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows) {
  tc::EncodeTiledFn fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
  const cuuint32_t box[2] = {BK, box_rows}, one[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool router_ok(const qsm_router* r) {
  return r && r->H >= BK && r->H % BK == 0 && r->E >= 1 && r->k >= 1 && r->k <= r->E &&
         (r->score == QSM_SCORE_SOFTMAX || r->score == QSM_SCORE_SIGMOID) && (r->renormalize & ~1) == 0 &&
         r->groups >= 1 && r->E % r->groups == 0 && r->groups_kept >= 1 && r->groups_kept <= r->groups &&
         r->group_best >= 1 && r->group_best <= 2 && r->group_best <= r->E / r->groups &&
         (long long)r->groups_kept * (r->E / r->groups) >= r->k && r->scale > -INFINITY && r->scale < INFINITY;
}

long long tiles_of(int T, int nt) { return ((long long)T + nt - 1) / nt; }

void choose(const qsm_router* r, int T, Config* out) {
  const int mb = row_blocks(r->E), steps = r->H / BK;
  const int most = 8 / mb;  // slices of a portable cluster
  int nt = 16;
  while (nt < 256 && tiles_of(T, nt) * 8 > mx4::sm_count()) nt *= 2;
  while (!fit(nt, r->E, out)) nt /= 2;
  out->ks = 1;
  while (out->ks * 2 <= most && out->ks * 2 <= steps) out->ks *= 2;
}

}  // namespace
}  // namespace rscores
}  // namespace qsm

extern "C" size_t moe_router_split_bytes(int32_t E, int32_t H) {
  return E < 1 || H < 1 ? 0 : (size_t)3 * E * H * 2;
}

extern "C" qsm_status moe_router_split(const float* w_router, int32_t E, int32_t H, uint16_t* w_split,
                                       cudaStream_t stream) {
  using namespace qsm;
  if (E < 1 || H < rscores::BK || H % rscores::BK || !w_router || !w_split || !aligned16(w_router) ||
      !aligned16(w_split))
    return QSM_ERR_INVALID_ARGUMENT;
  return route_split_launch(w_router, (size_t)E * H, w_split, stream);
}

extern "C" qsm_status moe_route_scores(const qsm_router* r, const uint16_t* x, int64_t ldx, int32_t T,
                                       int32_t* topk_idx, float* topk_w, int32_t* dev_status,
                                       cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::rscores;
  if (!router_ok(r) || T < 0) return QSM_ERR_INVALID_ARGUMENT;
  if (r->E > kMaxE || r->k > kMaxK || r->groups > kMaxGroups) return QSM_ERR_UNSUPPORTED;
  if (T == 0) return QSM_OK;
  if (T == 1) ldx = r->H;
  if (!x || !topk_idx || !topk_w || !dev_status || !r->w_split || !aligned16(x) || !aligned16(r->w_split) ||
      !aligned4(topk_idx) || !aligned4(topk_w) || !aligned4(dev_status) || (r->bias && !aligned4(r->bias)) ||
      ldx < r->H || ldx % 8)
    return QSM_ERR_INVALID_ARGUMENT;
  const int mb = row_blocks(r->E);
  Config c;
  choose(r, T, &c);
  const long long ctas = tiles_of(T, c.nt) * c.ks * mb;
  if (ctas > 0x7fffffffll || ldx > (1ll << 38)) return QSM_ERR_UNSUPPORTED;
  Params p = {};
  if (!make_map(&p.x, x, T, r->H, ldx, c.nt) || !make_map(&p.w, r->w_split, 3ull * r->E, r->H, r->H, BM))
    return QSM_ERR_CUDA;
  p.bias = r->bias;
  p.T = T;
  p.H = r->H;
  p.E = r->E;
  p.k = r->k;
  p.nt = c.nt;
  p.ks = c.ks;
  p.stages = c.stages;
  p.sigmoid = r->score == QSM_SCORE_SIGMOID;
  p.groups = r->groups;
  p.kept = r->groups_kept;
  p.best = r->group_best;
  p.gsize = r->E / r->groups;
  p.renorm = r->renormalize;
  p.scale = r->scale;
  p.idx = topk_idx;
  p.wts = topk_w;
  p.status = dev_status;
  auto* kernel = mb == 1 ? route_scores_kernel<1> : mb == 2 ? route_scores_kernel<2> : route_scores_kernel<4>;
  QSM_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem));
  QSM_CUDA_TRY(launch_pdl_cluster(kernel, dim3((unsigned)ctas), dim3(kThreads), c.ks * mb, c.smem, stream, p));
  return QSM_OK;
}
