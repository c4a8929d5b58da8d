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
//
// Measured (GPU time of a replayed call; H 2048, 256 experts unless said):
//   1 token 8.5 us: latency.  The copies of the 3.1 MB of split weights take 3.3, the exchanges take 2.5 and the selection 2
//   37 tokens 8.3 us, 300 tokens of H 1024 and 64 experts 7.2: the same chain
//   4096 tokens in 8 groups 20.8 us: 22 clusters of six CTAs (three slices); each tile of tokens reads all
//     the weights, 69 MB of the 81 that L2 moves.  In two slices, 36 tiles and 110 MB, it took 21.5,
//     of which the copies took 9 and the selection 6; the MMAs alone would take 6.7.  (With clusters that
//     come in two waves it took 50.)
//   384 and 512 experts (both read as 512; that kernel spills 620 bytes a thread): 1 token 16.1 and 16.5 us,
//     300 17.6 and 18.0, 4096 44 and 46
//
// The split weights lie in the order in which a CTA takes them: for each 64
// columns and each 128 experts the three parts, 128 x 64 each, in the image
// that the MMA reads (rows of 128 bytes, 16-byte unit u of row r at u ^ (r & 7)), so
// that a step's 48 KB are one plain bulk copy.  Missing experts are zeros.
#include "mx4_digits.cuh"

namespace qsm {
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
  const unsigned char* w;  // the split weights
  const float* bias;
  int T, H, E, k, nt, ks, stages, scratch;  // scratch: offset of the warps' own
  int sigmoid, groups, kept, best, gsize, renorm;
  mx4::FastDiv gdiv;  // by gsize
  float scale;
  int32_t* idx;
  float* wts;
  int32_t* status;
};

int row_blocks(int E) { return E <= BM ? 1 : E <= 2 * BM ? 2 : 4; }

// The split of w_router [E, H]: a thread has eight columns of a row.
__global__ void __launch_bounds__(256)
split_kernel(const float* __restrict__ w, int E, int H, int mb, unsigned char* __restrict__ out, long long units) {
  pdl_wait();
  pdl_launch_dependents();
  const long long u = blockIdx.x * 256ll + threadIdx.x;
  if (u >= units) return;
  const int c8 = (int)(u % (H / 8)), e = (int)(u / (H / 8));  // eight columns, row (of all blocks)
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (e < E) {
    const float4* src = reinterpret_cast<const float4*>(w + (size_t)e * H) + 2 * c8;
    const float4 a = __ldg(src), b = __ldg(src + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  const int r = e % BM, step = c8 / (BK / 8), unit = c8 % (BK / 8);
  unsigned char* dst = out + ((size_t)step * mb + e / BM) * 3 * kPartBytes + r * 128 + ((unit ^ (r & 7)) << 4);
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat16 h = __float2bfloat16_rn(v[i]);
      v[i] -= __bfloat162float(h);  // exact
      o[i / 2] |= (uint32_t)__bfloat16_as_ushort(h) << (16 * (i & 1));
    }
    *reinterpret_cast<uint4*>(dst + (size_t)part * kPartBytes) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

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

// The expert at position i of lane `lane`: a lane has four that follow one
// another of every 128.
__device__ __forceinline__ int expert_at(int i, int lane) { return 128 * (i >> 2) + 4 * lane + (i & 3); }

// A warp's scratch, in floats: one for each of the 128 MB experts, the ids and the
// order keys of the taken ones, and (up to 256 experts) the lanes' sorted lists.
template <int MB>
__host__ __device__ constexpr int scratch_floats() {
  return 128 * MB + 2 * kMaxK + (MB <= 2 ? 2 * 128 * MB : 0);
}

// What a lane knows of its experts, once for all tokens.
template <int MB>
struct Experts {
  float bias[4 * MB];   // -infinity for those that are closed
  uint32_t group[MB];   // four groups, a byte each
  uint32_t in;          // bit i: there is such an expert
  int per, plog, start; // group values: lanes per group, its logarithm, and where this lane starts
};

template <int MB>
__device__ __forceinline__ Experts<MB> load_experts(const Params& p, int lane) {
  Experts<MB> x;
  x.in = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4 * MB; ++i) {
    const int e = expert_at(i, lane);
    x.bias[i] = 0.f;
    if (e < p.E) {
      x.in |= 1u << i;
      if (p.bias) x.bias[i] = __ldg(p.bias + e);
      if (!(x.bias[i] < INFINITY)) {  // +infinity or NaN
        bad = true;
        x.bias[i] = -INFINITY;
      }
    }
    if ((i & 3) == 0) x.group[i >> 2] = 0;
    x.group[i >> 2] |= (uint32_t)min((int)p.gdiv.div(e), 31) << (8 * (i & 3));
  }
  if (bad) set_status(p.status, QSM_DEV_NONFINITE);
  x.plog = 5;
  while ((p.groups << x.plog) > 32 || (1 << x.plog) > p.gsize) --x.plog;
  x.per = 1 << x.plog;
  const int at = (lane & (x.per - 1)) + (lane >> x.plog);
  x.start = at - (int)p.gdiv.div(at) * p.gsize;
  return x;
}

// One token by one warp.  l: its logits, in the order of expert_at; sc: the
// warp's scratch.  dry: goes through the motions and writes nothing.
template <int MB>
__device__ __forceinline__ void select_token(const Params& p, const Experts<MB>& x, float (&l)[4 * MB], float* sc,
                                             int lane, size_t t, bool dry) {
  constexpr int N = 4 * MB;
  constexpr uint32_t kAll = 0xffffffffu;
  unsigned long long* taken = reinterpret_cast<unsigned long long*>(sc + 128 * MB);
  uint32_t fine = x.in;
  float zero[MB];  // NaN when a logit is not finite
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!((x.in >> i) & 1u)) l[i] = 0.f;
    zero[i >> 2] = (i & 3) ? fmaf(l[i], 0.f, zero[i >> 2]) : l[i] * 0.f;
  }
#pragma unroll
  for (int b = 1; b < MB; ++b) zero[0] += zero[b];
  if (__any_sync(kAll, zero[0] != 0.f)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!isfinite(l[i])) {
        fine &= ~(1u << i);
        l[i] = 0.f;
      }
    if (lane == 0 && !dry) set_status(p.status, QSM_DEV_NONFINITE);
  }
  // The scores by the fast exponential and quotient: 2 units in the last place and |l| 2^-24, as much as a
  // rounding of l itself changes e^l, and 2 units.  Largest relative errors of the weights against 64 bits
  // (plain fp32 form, with expf and a division, so): 4096 tokens, sigmoid 9.4e-7 3.7e-7 4.1e-7; 300, softmax
  // 4.7e-6 1.5e-6 1.8e-6; one token 1.5e-7 1.2e-7 1.3e-7.  expf and divisions: 0.5 to 0.9 us more a call, 1.9
  // with more than 256 experts.
  float s[N];
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __fdividef(1.0f, 1.0f + __expf(-l[i]));
  } else {
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((fine >> i) & 1u) top = fmaxf(top, l[i]);
    top = key_value(__reduce_max_sync(kAll, order_key(top)));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = (fine >> i) & 1u ? __expf(l[i] - top) : 0.f;
      sum += s[i];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.f ? __fdividef(1.0f, sum) : 0.f;  // 1 .. E
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] *= inv;
  }
  float c[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool ok = (fine >> i) & 1u;
    if (!ok) s[i] = 0.f;
    c[i] = ok ? s[i] + x.bias[i] : -INFINITY;
  }

  uint32_t allowed = x.in;  // bit i: expert i of this lane may be taken
  if (p.kept < p.groups) {
    // `per` lanes a group (a power of two) look through its experts
    const int g = lane >> x.plog;
    float a = -INFINITY, b = -INFINITY;
    if ((p.gsize & 3) == 0) {  // a lane's four neighbours are of one group: their best two stand for them
      float2* two = reinterpret_cast<float2*>(sc);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const float hi = fmaxf(c[4 * i], c[4 * i + 1]), lo = fminf(c[4 * i], c[4 * i + 1]);
        float2 v = make_float2(hi, lo);
        best_two(v.x, v.y, fmaxf(c[4 * i + 2], c[4 * i + 3]), fminf(c[4 * i + 2], c[4 * i + 3]));
        two[32 * i + lane] = v;
      }
      __syncwarp();
      if (g < p.groups) {
        const int quads = p.gsize >> 2;
#pragma unroll 2
        for (int j = lane & (x.per - 1); j < quads; j += x.per) {
          const float2 v = two[g * quads + j];
          best_two(a, b, v.x, v.y);
        }
      }
    } else {  // from different places, so that the lanes' reads fall into different banks
#pragma unroll
      for (int i = 0; i < MB; ++i)
        reinterpret_cast<float4*>(sc)[32 * i + lane] = make_float4(c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]);
      __syncwarp();
      if (g < p.groups) {
        const float* gc = sc + g * p.gsize;
        int at = x.start;
#pragma unroll 1
        for (int j = lane & (x.per - 1); j < p.gsize; j += x.per) {
          best_two(a, b, gc[at], -INFINITY);
          at += x.per;
          if (at >= p.gsize) at -= p.gsize;
        }
      }
    }
    __syncwarp();
    for (int o = 1; o < x.per; o <<= 1) {
      const float c2 = __shfl_xor_sync(kAll, a, o), d2 = __shfl_xor_sync(kAll, b, o);
      best_two(a, b, c2, d2);
    }
    const float value = p.best == 2 ? a + b : a;
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < p.groups; ++o) {
      const float v = __shfl_sync(kAll, value, o << x.plog);
      rank += v > value || (v == value && o < g);
    }
    // lane o finds out about group o
    const uint32_t in = __ballot_sync(kAll, g < p.groups && rank < p.kept);
    const uint32_t keep = __ballot_sync(kAll, lane < p.groups && ((in >> ((lane << x.plog) & 31)) & 1u));
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!((keep >> ((x.group[i >> 2] >> (8 * (i & 3))) & 31)) & 1u)) allowed &= ~(1u << i);
  }
#pragma unroll
  for (int b = 0; b < MB; ++b)
    reinterpret_cast<float4*>(sc)[32 * b + lane] = make_float4(s[4 * b], s[4 * b + 1], s[4 * b + 2], s[4 * b + 3]);

  // The k rounds take the best head of the lanes' sorted lists.  Two lanes with
  // the same key are rare: the first time through, a round only notes that it
  // saw them (the vote is not waited for), and then all is done again with care.
  constexpr int kList = N < 8 ? N : 8;
#pragma unroll 1
  for (int careful = 0; careful < 2; ++careful) {
    unsigned long long key[N];  // (order of c, ~expert): a strict order; 0 where there is none
#pragma unroll
    for (int i = 0; i < N; ++i)
      key[i] = (allowed >> i) & 1u ? ((unsigned long long)order_key(c[i]) << 32) | (uint32_t)~expert_at(i, lane) : 0ull;
#pragma unroll
    for (int n = 0; n < N; n += kList) sort_desc<kList>(key + n);
    uint32_t twice = 0;
    // Whether this lane's head is the best one.  (Ties dropped by several lanes can
    // empty all lists before round k: a head of 0 is none, and never the best.)
    const auto best = [&](unsigned long long head) {
      const uint32_t hk = (uint32_t)(head >> 32);
      const bool mine = hk == __reduce_max_sync(kAll, hk) && hk != 0;
      const uint32_t who = __ballot_sync(kAll, mine);
      twice |= who & (who - 1);
      return mine;
    };
    const auto one_of = [&](bool mine, unsigned long long head) {
      return (uint32_t)head == __reduce_max_sync(kAll, mine ? (uint32_t)head : 0u) && mine;
    };
    if constexpr (N <= 8) {  // the lists lie in shared memory: a round reads one key, in place of moving eight
      unsigned long long* next = reinterpret_cast<unsigned long long*>(sc + 128 * MB + 2 * kMaxK) + lane;
#pragma unroll
      for (int i = 1; i < N; ++i) next[32 * (i - 1)] = key[i];
      next[32 * (N - 1)] = 0ull;
      unsigned long long head = key[0];
      if (!careful) {
#pragma unroll 4
        for (int j = 0; j < p.k; ++j)
          if (best(head)) {
            taken[j] = head;
            head = *next;
            next += 32;
          }
      } else {
#pragma unroll 1
        for (int j = 0; j < p.k; ++j)
          if (one_of(best(head), head)) {
            taken[j] = head;
            head = *next;
            next += 32;
          }
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < p.k; ++j) {
        const bool second = key[8] > key[0];  // the head is the second list's
        const unsigned long long head = second ? key[8] : key[0];
        bool mine = best(head);
        if (careful) mine = one_of(mine, head);
        if (mine) taken[j] = head;
#pragma unroll
        for (int n = 0; n < N; n += kList) {
          const bool pop = mine && second == (n > 0);
#pragma unroll
          for (int i = n; i < n + kList; ++i) key[i] = !pop ? key[i] : i + 1 < n + kList ? key[i + 1] : 0ull;
        }
      }
    }
    if (twice == 0) break;
  }
  __syncwarp();
  float w = 0.f;
  int my_e = 0;
  if (lane < p.k) {
    const unsigned long long mine = taken[lane];
    my_e = min((int)~(uint32_t)mine & 0x7fffffff, 128 * MB - 1);  // (always less than E)
    if (key_value((uint32_t)(mine >> 32)) > -INFINITY) w = sc[my_e];  // a closed expert has weight 0
  }
  if (p.renorm) {
    float sum = w;
    for (int o = 1; o < p.k; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);  // the lanes from k on hold zeros
    w = sum > 1e-30f ? __fdividef(w, sum) : sum > 0.f ? w / sum : 0.f;
  }
  if (lane < p.k && !dry) {
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
  int cols = 32;  // of tensor memory
  while (cols < 2 * nt) cols *= 2;
  float* sc = reinterpret_cast<float*>(smem + p.scratch) + warp * scratch_floats<MB>();
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&done_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    tc::prefetch_map(&p.x);
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
  Experts<MB> experts;
  if (warp != 0) experts = load_experts<MB>(p, lane);  // the copies' warp has no time for it yet

  const auto product = [&] {
    if (warp == 0) {
      int st = 0;
      for (int s = 0, round = 0; st < steps; ++st) {
        if (round > 0 && !mx4::warp_wait(&empty_bar[s], (round - 1) & 1, abort_p, p.status)) break;
        if (mx4::warp_aborted(abort_p)) break;
        if (tc::elect_one()) {
          unsigned char* sb = smem + s * stage_bytes;
          mbar_arrive_expect_tx(&full_bar[s], stage_bytes);
          bulk_g2s(sb, p.w + ((size_t)(first + st) * MB + m) * 3 * kPartBytes, 3 * kPartBytes, &full_bar[s]);
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
  };

  // The selection stands here once and is gone through twice: first by the warps
  // that have no part in the product, which fetch its code meanwhile, then
  // by all.
  int tokens = 0, row0 = 0, aborted = 0;  // this warp's, every kWarps-th row from row0 on
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const bool dry = pass == 0;
    if (dry) {
      if (warp >= kEpiWarp + 8) tokens = 1;
      else product();
      if (warp == 0) experts = load_experts<MB>(p, lane);
    } else {
      tc::tc_fence_before();
      __syncthreads();
      if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, cols);
      }
      cluster_sync_all();  // every slice of the tile is in its CTA's shared memory
      // a CTA that gave up leaves no logits: its flag is read with them
      if (lane < csize)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(aborted) : "r"(dsmem_addr(&abort_flag, lane)) : "memory");
      const int per = (nt + csize - 1) / csize;
      const int rows = min(min(nt, p.T - tile * nt), (cta + 1) * per);
      row0 = cta * per + warp;
      tokens = row0 >= rows ? 0 : (rows - row0 + kWarps - 1) / kWarps;
    }
#pragma unroll 1
    for (int i = 0; i < tokens; ++i) {
      const int row = row0 + i * kWarps;
      float l[4 * MB];
#pragma unroll
      for (int j = 0; j < 4 * MB; ++j) l[j] = 0.f;
      if (!dry) {
        const uint32_t at = smem_u32(smem) + (row * kRowFloats + 4 * lane) * 4;
        for (int s0 = 0; s0 < p.ks; s0 += 4) {  // four slices' reads under way at once
          float4 v[4][MB];
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int b = 0; b < MB; ++b)
              if (s0 + s < p.ks) v[s][b] = dsmem_ld_f4(dsmem_addr_u32(at, (s0 + s) * MB + b));
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int b = 0; b < MB; ++b)
              if (s0 + s < p.ks) {
                l[4 * b] += v[s][b].x, l[4 * b + 1] += v[s][b].y;
                l[4 * b + 2] += v[s][b].z, l[4 * b + 3] += v[s][b].w;
              }
        }
      }
      if (__any_sync(0xffffffffu, aborted)) break;
      select_token<MB>(p, experts, l, sc, lane, (size_t)tile * nt + row, dry);
    }
  }
  cluster_sync_all();  // no CTA leaves while another still reads its slices
}

// ---------------------------------------------------------------------- host

constexpr size_t kSmem = 220 * 1024;  // dynamic, of the 227 KB; the rest is static

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

void* kernel_of(int mb) {
  return mb == 1   ? reinterpret_cast<void*>(route_scores_kernel<1>)
         : mb == 2 ? reinterpret_cast<void*>(route_scores_kernel<2>)
                   : reinterpret_cast<void*>(route_scores_kernel<4>);
}

// Clusters of 16 CTAs have to be allowed, once per device and kernel.
bool allow_large_clusters(int mb) {
  static std::atomic<uint64_t> done[5];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && (done[mb].load() >> dev & 1u)) return true;
  if (cudaFuncSetAttribute(kernel_of(mb), cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (dev < 64) done[mb].fetch_or(1ull << dev);
  return true;
}

// How a call is cut up: nt tokens a tile, the sum over H in ks slices.
struct Config {
  int nt, ks, stages, scratch;
  long long tiles;
  size_t smem;
};

// A cluster of ks x mb CTAs has a tile; the device holds so many at once (a
// GB300: 76 of 2, 36 of 4, 15 of 8, 7 of 16), and with tiles for all of them a launch takes one
// wave.  Least time, by the terms of a fit to 20 sizes from 1 to 16384 tokens and 8 to 384 experts: a
// CTA's copies, its accumulators, the tokens of a warp, and the exchange, which grows with the cluster.
// The choice is within 5% of the best one for each of them; us for 1, 2, 3, 4, 6, 8, 16 slices:
//   H 2048, 256 experts: 1 token 19.5 12.4 10.3 8.8 8.4 8.3 -, 1000 20.4 13.9 12.5 12.4 13.1 13.3 -,
//     4096 25.8 20.3 20.0 38.6 38.4 51.8 -
//   H 2048, 64 experts: 1 token 18.5 11.7 9.6 8.3 7.6 6.5 7.0, 4096 21.5 15.6 14.3 13.7 15.1 28.7 44.9
Config choose(const qsm_router* r, int T) {
  struct Kept {
    int dev, T, H, E;
    Config c;
  };
  static thread_local Kept kept[4];  // the last answers of this thread: asking takes longer than a small call
  static thread_local unsigned turn = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return Config{};
  for (const Kept& k : kept)
    if (k.T == T && k.H == r->H && k.E == r->E && k.dev == dev) return k.c;
  const int mb = row_blocks(r->E), steps = r->H / BK;
  Config best = {};
  double least = 0;
  static const int kSlices[] = {1, 2, 3, 4, 6, 8, 16};
  const int most_ctas = allow_large_clusters(mb) ? 16 : 8;
  for (int ks : kSlices) {
    if (ks * mb > most_ctas || ks > steps) break;
    const int resident = mx4::resident_clusters(kernel_of(mb), ks * mb, kThreads, (int)kSmem, (int)kSmem);
    if (resident < 1) continue;
    Config c = {};
    const long long each = ((long long)T + resident - 1) / resident;
    c.nt = each > 256 ? 256 : (int)(each + 15) / 16 * 16;
    c.ks = ks;
    c.tiles = ((long long)T + c.nt - 1) / c.nt;
    const long long waves = (c.tiles + resident - 1) / resident;
    const int cut = ks * mb, rounds = ((c.nt + cut - 1) / cut + kWarps - 1) / kWarps;
    const double us = (double)waves * (3.0 + (steps + ks - 1) / ks * (3 * kPartBytes + c.nt * BK * 2) / 131e3 +
                                       c.nt * 0.01 + rounds * 0.8 + cut * 0.15);
    if (best.nt == 0 || us < least) {
      best = c;
      least = us;
    }
  }
  if (best.nt == 0) return best;
  const int stage = 3 * kPartBytes + best.nt * BK * 2, rows = best.nt * kRowFloats * 4, sc = kWarps * 4 * (mb == 1 ? scratch_floats<1>() : mb == 2 ? scratch_floats<2>() : scratch_floats<4>());
  int most = (int)((kSmem - 1024 - sc) / stage);
  if (most > kMaxStages) most = kMaxStages;
  best.stages = most;
  best.scratch = most * stage > rows ? most * stage : rows;
  best.smem = (size_t)best.scratch + sc + 1024;
  kept[turn++ % 4] = {dev, T, r->H, r->E, best};
  return best;
}

}  // namespace
}  // namespace rscores
}  // namespace qsm

extern "C" size_t moe_router_split_bytes(int32_t E, int32_t H) {
  using namespace qsm::rscores;
  if (E < 1 || E > kMaxE || H < BK || H % BK) return 0;
  return (size_t)(H / BK) * row_blocks(E) * 3 * kPartBytes;
}

extern "C" qsm_status moe_router_split(const float* w_router, int32_t E, int32_t H, uint16_t* w_split,
                                       cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::rscores;
  if (E < 1 || H < BK || H % BK || !w_router || !w_split || !aligned16(w_router) || !aligned16(w_split))
    return QSM_ERR_INVALID_ARGUMENT;
  if (E > kMaxE) return QSM_ERR_UNSUPPORTED;
  const int mb = row_blocks(E);
  if (mx4::overlap(mx4::Rows{w_router, 1, 0, (size_t)E * H * 4}, mx4::Rows{w_split, 1, 0, moe_router_split_bytes(E, H)}))
    return QSM_ERR_INVALID_ARGUMENT;
  const long long units = (long long)mb * BM * (H / 8);
  QSM_CUDA_TRY(launch_pdl(split_kernel, dim3((unsigned)((units + 255) / 256)), dim3(256), 0, stream, w_router, (int)E,
                          (int)H, mb, reinterpret_cast<unsigned char*>(w_split), units));
  return QSM_OK;
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
  // the tokens are selected at different times: what is written may hold nothing that is read
  const auto vec = [](const void* p, size_t bytes) { return mx4::Rows{p, 1, 0, bytes}; };
  const size_t out = (size_t)T * r->k * 4;
  const mx4::Rows rx = {x, (size_t)T, (size_t)ldx * 2, (size_t)r->H * 2};
  const mx4::Rows ids = vec(topk_idx, out), wts = vec(topk_w, out), split = vec(r->w_split, moe_router_split_bytes(r->E, r->H));
  const mx4::Rows bias = vec(r->bias, (size_t)r->E * 4);
  if (mx4::overlap(ids, wts)) return QSM_ERR_INVALID_ARGUMENT;
  for (const mx4::Rows& w : {ids, wts})
    if (mx4::overlap(w, rx) || mx4::overlap(w, split) || mx4::overlap(w, bias)) return QSM_ERR_INVALID_ARGUMENT;
  const int mb = row_blocks(r->E);
  const Config c = choose(r, T);
  if (c.nt == 0) return QSM_ERR_CUDA;
  const long long ctas = c.tiles * c.ks * mb;
  if (ctas > 0x7fffffffll || ldx > (1ll << 38)) return QSM_ERR_UNSUPPORTED;
  Params p = {};
  if (!make_map(&p.x, x, T, r->H, ldx, c.nt)) return QSM_ERR_CUDA;
  p.w = reinterpret_cast<const unsigned char*>(r->w_split);
  p.bias = r->bias;
  p.T = T;
  p.H = r->H;
  p.E = r->E;
  p.k = r->k;
  p.nt = c.nt;
  p.ks = c.ks;
  p.stages = c.stages;
  p.scratch = c.scratch;
  p.sigmoid = r->score == QSM_SCORE_SIGMOID;
  p.groups = r->groups;
  p.kept = r->groups_kept;
  p.best = r->group_best;
  p.gsize = r->E / r->groups;
  p.gdiv = mx4::FastDiv(p.gsize);
  p.renorm = r->renormalize;
  p.scale = r->scale;
  p.idx = topk_idx;
  p.wts = topk_w;
  p.status = dev_status;
  auto* kernel = mb == 1 ? route_scores_kernel<1> : mb == 2 ? route_scores_kernel<2> : route_scores_kernel<4>;
  // (choose has allowed the kernel its shared memory and clusters)
  QSM_CUDA_TRY(launch_pdl_cluster(kernel, dim3((unsigned)ctas), dim3(kThreads), c.ks * mb, c.smem, stream, p));
  return QSM_OK;
}
