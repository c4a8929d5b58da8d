// The MoE layer with MXFP4 weights and 16-bit activations for one or two
// tokens, in one launch: router, selection, gate_up + SwiGLU, down and
// combine.
//
// The products are those of mx4_stream.cu (activations as base-8 digit
// planes, weights as the MMA's rows); what is different is what surrounds
// them.  At one token the layer's 17 MB take 2.5 us of HBM time and the four
// launches of the other form 20 us, nearly all of it latency: each launch
// waits for the last CTA of the one before, looks its work up and waits for
// its first copies.  Here every CTA is resident from the start (clusters of
// four, one CTA per SM) and the phases hand over by words that carry the
// call's tag, which a reader polls: the data and its readiness in one trip
// through L2 (as in decode_layer.cu).
//
//   A  CTA c computes the logits of its experts (arithmetic of moe_route) and
//      publishes them as (tag, logit) words.  Meanwhile two warps make the
//      digits of x for the CTA's quarter of H: every expert's product uses
//      the same ones, so they are off the path.
//   B  Every CTA collects the logits, selects (code of moe_route: same ids and
//      weights) and forms the sorted set U of the chosen experts.  Slot 0 is the
//      shared expert, slot s the s-th of U; a slot is computed for all T
//      tokens (an MMA of 16 digit rows costs what one of 8 does).  Cluster q
//      takes the items (slot, 128 intermediates) q, q + clusters, ..; its CTAs
//      split H and exchange partial sums through distributed shared memory, as
//      in mx4_stream.cu; h goes out as (tag, h) words in fp32.
//   C  Cluster q < H / 128 owns rows 128 q .. of y.  Its CTA r takes the slots r,
//      r + 4, ..: the digits of (routing weight x h), accumulated over its slots in
//      one tensor-memory accumulator, so that the combine is part of the
//      product; the four CTAs' sums are exchanged like the others and y is
//      written once.  The down weights are requested as soon as U is known, ahead
//      of h.
//
// One token takes 15.6 us (17 MB in L2; H 2048, I 512, 256 experts, 8 of them; 16.8 with
// the weights from HBM), against 20.6 in separate launches: what is left is the latency of the chain from the
// router's rows to y.
//
// With more tokens phase C, which has 64 SMs for the down weights, and the
// computing of all pairs cost more than the launches save (T = 2: 21.2 us against
// 24.4, T = 3: 28.5 against 25.2 (now 23.8), T = 8: 83.8 against 42.3 (38.7)): they take the other
// form.
//
// Sums run in a fixed order (by slot within a CTA, then the four CTAs): y depends
// on nothing but the inputs.  With two tokens U holds the experts of both, so
// which slots share an accumulator, and with it the last fp32 bits of one
// token's y, depends on the other token's choices.  Every wait
// is bounded (QSM_DEV_TIMEOUT; the results are then invalid and the workspace
// must be zeroed).  The tag is 1 + the calls so far, from a ticket that every
// CTA adds 1 to; every word that a call reads it has written before.
#include "mx4_decode.cuh"

#include "route_select.cuh"

namespace qsm {
namespace mx4 {
namespace {

constexpr int kThreads = 512;
constexpr int kCs = 4;                // CTAs per cluster
constexpr int kConvWarps = 10;        // of the down phase
constexpr int kXWarps = 2;            // of the digits of x
constexpr int kRouteThreads = 384;    // warps 4..15
constexpr int kTPE = 128;             // threads per expert
constexpr int kMaxT = 2;
constexpr int kMaxE = 256;
constexpr int kMaxK = 32;
constexpr int kMaxStages = 6;
constexpr int kSmemMax = 222 * 1024;
constexpr int kStage = 2 * (128 * 128 + 2 * kTileBytes);
constexpr uint32_t kPolls = 1u << 20;      // of a tagged word: about a second
constexpr uint32_t kShortWait = 1u << 10;  // after a timeout

__device__ __forceinline__ unsigned long long ld_word(const unsigned long long* p) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_word(unsigned long long* p, uint32_t tag, float v) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p),
               "l"(((unsigned long long)tag << 32) | __float_as_uint(v))
               : "memory");
}
__device__ __forceinline__ void route_bar() {
  asm volatile("barrier.sync 2, %0;" ::"n"(kRouteThreads) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1) mx4_layer_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], xdig, rows_bar, rdy, hdig_full[2],
      hdig_empty[2], acc_full[2], acc_empty[2], dacc_full, part_full[2], part_empty[2], done;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ float rsum[3][kTPE / 32][kMaxT];
  __shared__ int sel_e[kMaxT][kMaxK];
  __shared__ float sel_w[kMaxT][kMaxK];
  __shared__ unsigned bitmap[kMaxE / 32];
  __shared__ float sgate_v[kMaxT];
  __shared__ int ulist[kMaxT * kMaxK];   // at most T k distinct experts
  __shared__ int s_nu;
  __shared__ uint32_t s_tag;
  volatile int* abort_p = &abort_flag;

  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), clus = blockIdx.x / kCs, nclus = gridDim.x / kCs;
  const int T = p.T, H = p.H, I = p.I, E = p.E, k = p.k;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&xdig, kXWarps);
    mbar_init(&rows_bar, 1);
    mbar_init(&rdy, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&hdig_full[b], kConvWarps);
      mbar_init(&hdig_empty[b], 1);
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
      mbar_init(&part_full[b], kCs);
      mbar_init(&part_empty[b], 4 * kCs);
    }
    mbar_init(&dacc_full, 1);
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < kMaxE / 32) bitmap[threadIdx.x] = 0u;
  if (warp == 0 && lane == 0) {
    tc::prefetch_map(&p.gu);
    tc::prefetch_map(&p.gu_sh);
    tc::prefetch_map(&p.dn);
    tc::prefetch_map(&p.dn_sh);
  }
  if (warp == 2) tc::tmem_alloc(&tmem_base, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  cluster_sync_all();
  const uint32_t tmem = uniform(tmem_base);
  pdl_wait();
  pdl_launch_dependents();

  const int nst = (H + kStageK - 1) / kStageK, cts = col_tiles(H);  // gate_up: this CTA's stages
  const int s0 = nst * rank / kCs, s1 = nst * (rank + 1) / kCs;
  const int dst_n = (I + kStageK - 1) / kStageK, dcts = col_tiles(I);  // down: stages per slot
  const int ntI = I / 128, ytiles = H / 128;
  const bool owns = clus < ytiles;
  const int drows = digit_rows(T);
  // tensor memory: two pairs of gate_up accumulators, down's, two stages' scales
  const uint32_t dacc = tmem + 4 * p.acc_cols, sf0 = dacc + p.acc_cols;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return wait_or_abort(bar, parity, abort_p, p.status);
  };

  if (warp == 0) {
    // -------------------------------------------------------------- loads
    int st = 0;
    uint32_t round = 0;
    auto next_stage = [&]() {  // the stage's turn: false after an abort
      return round == 0 || __all_sync(0xffffffffu, wait(&empty[st], (round - 1) & 1));
    };
    auto load_gu = [&](int item) {
      const int slot = item / ntI, tile = item - slot * ntI;
      const int e = slot == 0 ? 0 : uniform(ulist[slot - 1]);
      const CUtensorMap* map = slot == 0 ? &p.gu_sh : &p.gu;
      const int row0 = e * 2 * I + tile * 128;
      const uint8_t* sc = (slot == 0 ? p.gu_sc_sh : p.gu_sc) + (size_t)(row0 >> 7) * cts * kTileBytes;
      for (int ks = s0; ks < s1; ++ks) {
        if (!next_stage()) return false;
        if (elect_one()) {
          unsigned char* base = smem + st * kStage;
          const uint32_t sfb = (uint32_t)min(2, cts - 2 * ks) * kTileBytes;
          mbar_arrive_expect_tx(&full[st], 2 * (128 * 128 + sfb));
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            tc::tma_load_2d(base + m * 128 * 128, map, ks * 128, row0 + m * I, &full[st]);
            bulk_g2s(base + 2 * 128 * 128 + m * 2 * kTileBytes,
                     sc + ((size_t)m * (I >> 7) * cts + 2 * ks) * kTileBytes, sfb, &full[st]);
          }
        }
        __syncwarp();
        if (++st == p.stages) st = 0, ++round;
      }
      return true;
    };
    // this CTA's router rows, then (before the selection) a tile of the shared
    // expert where the cluster starts with one
    const int ea = blockIdx.x * p.epc, ne = min(E, ea + p.epc) - ea;
    if (elect_one()) {
      mbar_arrive_expect_tx(&rows_bar, ne > 0 ? (uint32_t)ne * H * 4 : 0u);
      if (ne > 0) bulk_g2s(smem + p.rows_off, p.w_router + (size_t)ea * H, ne * H * 4, &rows_bar);
    }
    __syncwarp();
    int item = clus;
    bool ok = true;
    if (item < ntI) {
      ok = load_gu(item);
      item += nclus;
    }
    ok = ok && __all_sync(0xffffffffu, wait(&rdy, 0));
    const int nu = ok ? uniform(s_nu) : 0;
    for (; ok && item < (nu + 1) * ntI; item += nclus) ok = load_gu(item);
    for (int slot = rank; ok && owns && slot <= nu; slot += kCs) {
      const int e = slot == 0 ? 0 : uniform(ulist[slot - 1]);
      const CUtensorMap* map = slot == 0 ? &p.dn_sh : &p.dn;
      const int row0 = e * H + clus * 128;
      const uint8_t* sc = (slot == 0 ? p.dn_sc_sh : p.dn_sc) + (size_t)(row0 >> 7) * dcts * kTileBytes;
      for (int ks = 0; ks < dst_n; ++ks) {
        if (!(ok = next_stage())) break;
        if (elect_one()) {
          unsigned char* base = smem + st * kStage;
          const uint32_t sfb = (uint32_t)min(2, dcts - 2 * ks) * kTileBytes;
          mbar_arrive_expect_tx(&full[st], 128 * 128 + sfb);
          tc::tma_load_2d(base, map, ks * 128, row0, &full[st]);
          bulk_g2s(base + 2 * 128 * 128, sc + (size_t)2 * ks * kTileBytes, sfb, &full[st]);
        }
        __syncwarp();
        if (++st == p.stages) st = 0, ++round;
      }
    }
    // after an abort, let the copies in flight land before the CTA exits
    for (int i = 0; i < p.stages; ++i) {
      const uint32_t r = i < st ? round : round - 1;
      if (i < st || round > 0) mbar_wait_bounded(&full[i], r & 1, 1u << 16);
    }
    mbar_wait_bounded(&rows_bar, 0, 1u << 16);
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMAs
    int st = 0, ab = 0;
    uint32_t round = 0, fs = 0, acc_round = 0;
    const uint32_t base = smem_u32(smem);
    const uint64_t desc0 = tc::sw128_desc(base);
    // one stage: `nm` tiles of 128 weight rows times a segment of digits
    auto stage_mma = [&](int nm, uint32_t acc, int dig_off, int sf_off, int kv, bool fresh) {
      const uint32_t wsf = base + st * kStage + 2 * 128 * 128;
      const uint64_t wd = desc0 + (uint64_t)(st * (kStage >> 4)), xd = desc0 + (uint64_t)(dig_off >> 4);
      const uint32_t sfw = sf0 + (fs & 1) * 24, sfx = sfw + 16;
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        if (ct * kTileCols >= kv) break;
        copy_scales(sfw + 4 * ct, wsf + ct * kTileBytes);
        if (nm == 2) copy_scales(sfw + 8 + 4 * ct, wsf + (2 + ct) * kTileBytes);
        copy_scales(sfx + 4 * ct, base + sf_off + ct * kTileBytes);
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk * 64 >= kv) break;
        const uint32_t more = fresh && kk == 0 ? 0u : 1u, id = idesc_mxf4(drows, kk & 1);
        mma_mxf4(acc, wd + 2 * kk, xd + 2 * kk, id, sfw + 4 * (kk >> 1), sfx + 4 * (kk >> 1), more);
        if (nm == 2)
          mma_mxf4(acc + p.acc_cols, wd + (128 * 128 >> 4) + 2 * kk, xd + 2 * kk, id, sfw + 8 + 4 * (kk >> 1),
                   sfx + 4 * (kk >> 1), more);
      }
      tc::mma_commit(&empty[st]);
    };
    auto advance = [&]() {
      ++fs;
      if (++st == p.stages) st = 0, ++round;
    };
    int nu = 0;
    bool ok = __all_sync(0xffffffffu, wait(&xdig, 0)), know = false;
    for (int item = clus; ok; item += nclus) {
      if (!know && item >= ntI) {  // past the shared expert's: the selection
        if (!(ok = __all_sync(0xffffffffu, wait(&rdy, 0)))) break;
        nu = uniform(s_nu);
        know = true;
      }
      if (know && item >= (nu + 1) * ntI) break;
      if (acc_round > 0 && !(ok = __all_sync(0xffffffffu, wait(&acc_empty[ab], (acc_round - 1) & 1)))) break;
      for (int ks = s0; ks < s1; ++ks) {
        if (!(ok = __all_sync(0xffffffffu, wait(&full[st], round & 1)))) break;
        tc::tc_fence_after();
        if (elect_one()) {
          stage_mma(2, tmem + ab * 2 * p.acc_cols, p.x_off + (ks - s0) * p.seg_bytes,
                    p.xsf_off + (ks - s0) * 2 * kTileBytes, min(kStageK, H - ks * kStageK), ks == s0);
          if (ks == s1 - 1) tc::mma_commit(&acc_full[ab]);
        }
        __syncwarp();
        advance();
      }
      if (ok && ++ab == 2) ab = 0, ++acc_round;
    }
    int n = 0;  // slots done
    for (int slot = rank; ok && owns && slot <= nu; slot += kCs, ++n) {
      const int b = n & 1;
      if (!(ok = __all_sync(0xffffffffu, wait(&hdig_full[b], (n >> 1) & 1)))) break;
      for (int ks = 0; ks < dst_n; ++ks) {
        if (!(ok = __all_sync(0xffffffffu, wait(&full[st], round & 1)))) break;
        tc::tc_fence_after();
        if (elect_one()) {
          stage_mma(1, dacc, p.h_off + (b * dst_n + ks) * p.seg_bytes,
                    p.hsf_off + (b * dst_n + ks) * 2 * kTileBytes, min(kStageK, I - ks * kStageK),
                    n == 0 && ks == 0);
          if (ks == dst_n - 1) {
            tc::mma_commit(&hdig_empty[b]);
            if (slot + kCs > nu) tc::mma_commit(&dacc_full);
          }
        }
        __syncwarp();
        advance();
      }
    }
    // every MMA issued has completed before tensor memory is freed
    if (elect_one()) tc::mma_commit(&done);
    __syncwarp();
    mbar_wait_bounded(&done, 0, kWaitIters);
  } else {
    bool bad = false;
    // eight values of row i from column c of segment seg become digits at
    // `dig` (segments of seg_bytes) and scales at `sf`
    auto put_digits = [&](const float (&v)[8], int i, int seg, int c8, unsigned char* dig, unsigned char* sf) {
      uint32_t plane[kDigits];
      const uint32_t sb = digits_of(v, plane);
      if (sb == 255u) bad = true;
      store_digits(plane, sb, i, c8, dig + seg * p.seg_bytes, sf + seg * 2 * kTileBytes, 1);
    };
    if (warp < 4) {
      // ------------------------------------------- digits of x, a quarter of H
      const int total = (s1 - s0) * T * 32;
      for (int u = (warp - 2) * 32 + lane; u - lane < total; u += 32 * kXWarps) {
        const int q = u >> 5, seg = q / T, i = q - seg * T, c = (s0 + seg) * kStageK + 8 * lane;
        float v[8];
        uint4 a = make_uint4(0u, 0u, 0u, 0u);
        if (c < H) a = __ldcg(reinterpret_cast<const uint4*>(p.x + (size_t)i * H + c));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = bf16_lo(w[j]);
          v[2 * j + 1] = bf16_hi(w[j]);
        }
        put_digits(v, i, seg, lane, smem + p.x_off, smem + p.xsf_off);
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&xdig);
    } else {
      // ---------------------------------------------------------- A: logits
      const int rt = threadIdx.x - 128, sub = rt / kTPE, tt = rt % kTPE;
      const int ea = blockIdx.x * p.epc, eb = min(E, ea + p.epc);
      if (rt == 0) {
        // every earlier call on this workspace has completed: the ticket holds
        // its CTAs' arrivals and some of this call's
        const unsigned long long t = ld_word(p.ticket);
        asm volatile("red.relaxed.gpu.global.add.u64 [%0], 1;" ::"l"(p.ticket) : "memory");
        s_tag = (uint32_t)(t / gridDim.x) + 1u;
      }
      uint16_t* xs = reinterpret_cast<uint16_t*>(smem + p.xs_off);
      const float* wr = reinterpret_cast<const float*>(smem + p.rows_off);
      for (int i = rt; i < T * H / 8; i += kRouteThreads)
        reinterpret_cast<uint4*>(xs)[i] = __ldcg(reinterpret_cast<const uint4*>(p.x) + i);
      wait(&rows_bar, 0);  // (after a timeout, later waits are short)
      route_bar();
      const uint32_t tag = s_tag;
      const int H4 = H / 4;
      for (int e0 = ea; e0 < eb; e0 += 3) {
        const int e = e0 + sub;
        const bool mine = e < eb;
        const float4* wrow = reinterpret_cast<const float4*>(wr + (size_t)(mine ? e - ea : 0) * H);
#pragma unroll 1
        for (int t = 0; t < T; ++t) {  // products and sums in the order of moe_route
          const uint2* xr = reinterpret_cast<const uint2*>(xs + (size_t)t * H);
          float a = 0.f;
          for (int h4 = tt; h4 < H4; h4 += kTPE) {
            const float4 wv = wrow[h4];
            const uint2 xv = xr[h4];
            a = fmaf(wv.x, bf16_lo(xv.x), a);
            a = fmaf(wv.y, bf16_hi(xv.x), a);
            a = fmaf(wv.z, bf16_lo(xv.y), a);
            a = fmaf(wv.w, bf16_hi(xv.y), a);
          }
          const float s = warp_sum(a);
          if (lane == 0) rsum[sub][tt / 32][t] = s;
        }
        route_bar();
        if (rt < 3 * kMaxT) {
          const int s = rt / kMaxT, t = rt % kMaxT;
          if (e0 + s < eb && t < T) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kTPE / 32; ++w) v += rsum[s][w][t];
            st_word(p.logits + (size_t)t * E + e0 + s, tag, v);
          }
        }
        route_bar();
      }
      if (p.sgate) {  // sigmoid(x . shared_gate), a warp per token
        for (int t = warp - 4; t < T; t += kRouteThreads / 32) {
          float z = 0.f;
          for (int h = lane; h < H; h += 32)
            z = fmaf(__uint_as_float((uint32_t)xs[(size_t)t * H + h] << 16), __ldg(p.sgate + h), z);
          z = warp_sum(z);
          if (lane == 0) sgate_v[t] = 1.0f / (1.0f + __expf(-z));
        }
      }
      // ------------------------------------------------------- B: selection
      // a warp per token; the logits go where the router rows were (every
      // read of those is behind the last barrier)
      float* lg = reinterpret_cast<float*>(smem + p.rows_off);
      const int t = warp - 4;
      if (t < T) {
        float* row = lg + t * E;
        const unsigned long long* src = p.logits + (size_t)t * E;
        const uint32_t iters = *abort_p ? kShortWait : kPolls;
        uint32_t want = 0;  // bit i: expert lane + 32 i is still to come
        for (int i = 0; lane + 32 * i < E; ++i) want |= 1u << i;
        for (uint32_t n = 0; __any_sync(0xffffffffu, want != 0); ++n) {
          if (n >= iters) {
            *abort_p = 1;
            set_status(p.status, QSM_DEV_TIMEOUT);
            break;
          }
          unsigned long long v[kMaxE / 32];
#pragma unroll
          for (int i = 0; i < kMaxE / 32; ++i)
            if (want & (1u << i)) v[i] = ld_word(src + lane + 32 * i);
#pragma unroll
          for (int i = 0; i < kMaxE / 32; ++i)
            if ((want & (1u << i)) && (uint32_t)(v[i] >> 32) == tag + (uint32_t)p.skew) {
              row[lane + 32 * i] = __uint_as_float((uint32_t)v[i]);
              want &= ~(1u << i);
            }
          if (n > 8) __nanosleep(32);
        }
        __syncwarp();
        int my_e;
        float my_l, my_w;
        // the common shape with its sizes known to the compiler
        if (E == kMaxE && k == 8)
          route_select_warp<kMaxE / 32, true>(row, p.bias, kMaxE, 8, p.flags, p.status, my_e, my_l, my_w);
        else
          route_select_warp<kMaxE / 32, true>(row, p.bias, E, k, p.flags, p.status, my_e, my_l, my_w);
        if (lane < k) {
          sel_e[t][lane] = my_e;
          sel_w[t][lane] = my_w;
          if (blockIdx.x == 0) {
            p.topk_idx[(size_t)t * k + lane] = my_e;
            p.topk_w[(size_t)t * k + lane] = my_w;
          }
          atomicOr(&bitmap[my_e >> 5], 1u << (my_e & 31));
        }
      }
      route_bar();
      if (warp == 4) {  // the sorted distinct ids: prefix popcounts of the bitmap
        const unsigned word = lane < kMaxE / 32 ? bitmap[lane] : 0u;
        const int cnt = __popc(word);
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        int at = incl - cnt;
        for (unsigned w = word; w; w &= w - 1) ulist[at++] = 32 * lane + (__ffs(w) - 1);
        if (lane == 31) s_nu = incl;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&rdy);
      }
    }
    const bool sel_ok = __all_sync(0xffffffffu, wait(&rdy, 0));
    const int nu = sel_ok ? uniform(s_nu) : -1;
    const uint32_t tag = uniform(s_tag);

    if (warp >= 4 && warp < 8) {
      // ------------------------------------- sums of gate_up and of down
      const int q4 = warp & 3;
      const uint32_t lanes = (uint32_t)(32 * q4) << 16;
      float* part = reinterpret_cast<float*>(smem + p.part_off);  // [2][kCs][2 T][32]
      int j = 0;  // exchanges
      // this CTA's partial sums v[i] (i < n) of its row go to the CTA that owns
      // the row.  There, row `lane`'s sums over the CTAs of the w values of token
      // q4 come out in out[]
      auto exchange = [&](const float* v, int n, int w, float* out) {
        const int b = j & 1;
        if (j >= 2 && !__all_sync(0xffffffffu, wait_cluster(&part_empty[b], (j / 2 - 1) & 1, abort_p, p.status)))
          return false;
        const uint32_t dst = dsmem_addr(part + (size_t)(b * kCs + rank) * 2 * kMaxT * 32 + lane, q4);
#pragma unroll
        for (int i = 0; i < 2 * kMaxT; ++i)
          if (i < n) dsmem_st_f32(dst + i * 32 * 4, v[i]);
        __syncwarp();
        if (lane == 0) arrive_cluster(dsmem_addr(&part_full[b], q4));
        if (!__all_sync(0xffffffffu, wait_cluster(&part_full[b], (j / 2) & 1, abort_p, p.status))) return false;
        const float* mine = part + (size_t)b * kCs * 2 * kMaxT * 32 + lane;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int i = w * q4 + z;
          float s = 0.f;
          if (z < w && i < n)
#pragma unroll
            for (int c = 0; c < kCs; ++c) s += mine[(c * 2 * kMaxT + i) * 32];
          out[z] = s;
        }
        __syncwarp();
        if (lane < kCs) arrive_cluster(dsmem_addr(&part_empty[b], lane));
        ++j;
        return true;
      };
      // the digits' sums of rows 0 .. T - 1 of x in accumulator `acc`, the
      // smallest digits first
      auto digit_sums = [&](uint32_t acc, float* v) {
#pragma unroll
        for (int i0 = 0; i0 < kMaxT; i0 += 2) {
          if (i0 >= T) break;
          float d[16];
          tc::tmem_ld16(acc + lanes + kDigits * i0, d);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float a = 0.f;
#pragma unroll
            for (int z = 0; z < kDigits; ++z) a += d[kDigits * u + z];
            v[i0 + u] = a;
          }
        }
      };
      int ab = 0;
      uint32_t acc_round = 0;
      bool ok = sel_ok;
      for (int item = clus; ok && item < (nu + 1) * ntI; item += nclus) {
        if (!(ok = __all_sync(0xffffffffu, wait(&acc_full[ab], acc_round & 1)))) break;
        tc::tc_fence_after();
        // value 2 t: gate, 2 t + 1: up of token t
        float g[kMaxT], u[kMaxT], v[2 * kMaxT], out[2];
        digit_sums(tmem + ab * 2 * p.acc_cols, g);
        digit_sums(tmem + (ab * 2 + 1) * p.acc_cols, u);
#pragma unroll
        for (int t = 0; t < kMaxT; ++t) v[2 * t] = g[t], v[2 * t + 1] = u[t];
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&acc_empty[ab]);
        if (++ab == 2) ab = 0, ++acc_round;
        if (!(ok = exchange(v, 2 * T, 2, out))) break;
        const int slot = item / ntI, c = (item - slot * ntI) * 128 + 32 * rank + lane;
        if (q4 < T) st_word(p.h + ((size_t)slot * T + q4) * I + c, tag, silu(out[0]) * out[1]);
      }
      if (ok && owns) {
        float v[2 * kMaxT], out[2];
#pragma unroll
        for (int i = 0; i < 2 * kMaxT; ++i) v[i] = 0.f;
        if (rank <= nu) {  // this CTA had a slot
          ok = __all_sync(0xffffffffu, wait(&dacc_full, 0));
          tc::tc_fence_after();
          if (ok) digit_sums(dacc, v);
        }
        if (ok && exchange(v, T, 1, out)) {
          const int r = clus * 128 + 32 * rank + lane;
          if (q4 < T) {
            p.y[(size_t)q4 * H + r] = __bfloat16_as_ushort(__float2bfloat16_rn(out[0]));
            if (p.y32) p.y32[(size_t)q4 * H + r] = out[0];
          }
        }
      }
    } else if (owns && sel_ok) {
      // --------------------------------- digits of (weight x h) of this CTA's slots
      const int ct = (warp < 4 ? warp - 2 : warp - 6) * 32 + lane;
      int n = 0;
      for (int slot = rank; slot <= nu; slot += kCs, ++n) {
        const int b = n & 1;
        if (n >= 2 && !__all_sync(0xffffffffu, wait(&hdig_empty[b], (n / 2 - 1) & 1))) break;
        const int total = dst_n * T * 32;
        const int e = slot == 0 ? -1 : ulist[slot - 1];
        bool ok = true;
        for (int u = ct; u - lane < total; u += 32 * kConvWarps) {
          const int q = u >> 5, seg = q / T, i = q - seg * T, c = seg * kStageK + 8 * lane;
          float wt = 0.f;
          bool chosen = e < 0;
          if (e < 0) wt = p.sgate ? sgate_v[i] : 1.f;
          for (int z = 0; e >= 0 && z < k; ++z)
            if (sel_e[i][z] == e) wt = sel_w[i][z], chosen = true;
          float v[8];
#pragma unroll
          for (int z = 0; z < 8; ++z) v[z] = 0.f;
          if (c < I) {  // wait until the eight words carry the tag
            const unsigned long long* src = p.h + ((size_t)slot * T + i) * I + c;
            const uint32_t iters = *abort_p ? kShortWait : kPolls;
            uint32_t want = 0xffu;
            for (uint32_t tries = 0; want; ++tries) {
              if (tries >= iters) {
                ok = false;
                break;
              }
              unsigned long long w[8];
#pragma unroll
              for (int z = 0; z < 8; ++z)
                if (want & (1u << z)) w[z] = ld_word(src + z);
#pragma unroll
              for (int z = 0; z < 8; ++z)
                if ((want & (1u << z)) && (uint32_t)(w[z] >> 32) == tag) {
                  // a token that did not choose the expert adds nothing; a weight of 0
                  // (an underflow) times an h that is not finite is not a number
                  v[z] = chosen ? wt * __uint_as_float((uint32_t)w[z]) : 0.f;
                  want &= ~(1u << z);
                }
              if (tries > 8) __nanosleep(32);
            }
          }
          __syncwarp();
          put_digits(v, i, seg, lane, smem + p.h_off + b * dst_n * p.seg_bytes,
                     smem + p.hsf_off + b * dst_n * 2 * kTileBytes);
        }
        if (!__all_sync(0xffffffffu, ok)) {
          *abort_p = 1;
          if (lane == 0) set_status(p.status, QSM_DEV_TIMEOUT);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&hdig_full[b]);
      }
    }
    if (bad) set_status(p.status, QSM_DEV_NONFINITE);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 2) tc::tmem_dealloc(tmem, 512);
  cluster_sync_all();  // no CTA leaves while another writes to it
}

// ---------------------------------------------------------------------- host

inline size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Shared memory; false when it does not fit.  The router's region (rows, then
// logits, and x) is used again by the digits of h and the exchanges.
bool layout(DecodeParams* p, int* smem) {
  const int segs = ((p->H + kStageK - 1) / kStageK + kCs - 1) / kCs;
  const int dsegs = (p->I + kStageK - 1) / kStageK;
  p->seg_bytes = digit_rows(p->T) * 128;
  const size_t route = up((size_t)p->epc * p->H * 4 > (size_t)p->T * p->E * 4 ? (size_t)p->epc * p->H * 4
                                                                             : (size_t)p->T * p->E * 4, 1024) +
                       (size_t)p->T * p->H * 2;
  const size_t hdig = up((size_t)2 * dsegs * p->seg_bytes, 1024) + (size_t)2 * dsegs * 2 * kTileBytes;
  const size_t xdig = up((size_t)segs * p->seg_bytes, 1024) + (size_t)segs * 2 * kTileBytes;
  const size_t part = (size_t)2 * kCs * 2 * kMaxT * 32 * 4;
  const size_t rest = xdig + up(route > hdig ? route : hdig, 1024) + part;
  if (rest + 3 * kStage + 1024 > kSmemMax) return false;
  const int room = (int)((kSmemMax - 1024 - rest) / kStage);
  p->stages = room < kMaxStages ? room : kMaxStages;
  size_t off = (size_t)p->stages * kStage;
  p->x_off = (int)off;
  p->xsf_off = (int)(off + up((size_t)segs * p->seg_bytes, 1024));
  off += xdig;
  off = up(off, 1024);
  p->rows_off = p->h_off = (int)off;
  p->xs_off = (int)(off + route - (size_t)p->T * p->H * 2);
  p->hsf_off = (int)(off + up((size_t)2 * dsegs * p->seg_bytes, 1024));
  off += up(route > hdig ? route : hdig, 1024);
  p->part_off = (int)off;
  off += part;
  *smem = (int)off + 1024;
  return *smem <= kSmemMax;
}

}  // namespace

size_t decode_workspace_bytes(const DecodeParams& p) {
  const int slots = (p.T * p.k < p.E ? p.T * p.k : p.E) + 1;
  return 256 + up((size_t)p.T * p.E * 8, 256) + (size_t)slots * p.T * p.I * 8;
}

bool plan_decode(const qsm_mx4_layer* L, int T, DecodeParams* p, int* smem, int* ctas) {
  p->T = T;
  p->H = L->H;
  p->I = L->I;
  p->E = L->E;
  p->k = L->k;
  if (T < 1 || T > kMaxT || L->E > kMaxE || L->k > kMaxK || L->H <= 3 * kStageK || L->I > 4096) return false;
  p->acc_cols = (digit_rows(T) + 31) / 32 * 32;
  // as many clusters as are resident at once (all must be), at the largest
  // shared memory; one per y tile at least
  p->epc = 0;
  const int n = resident_clusters(reinterpret_cast<void*>(mx4_layer_kernel), kCs, kThreads, kSmemMax, kSmemMax);
  if (n < 1 || n < L->H / 128) return false;
  p->epc = (L->E + n * kCs - 1) / (n * kCs);
  *ctas = n * kCs;
  return layout(p, smem);
}

qsm_status launch_decode(const DecodeParams& p, int smem, int ctas, cudaStream_t stream) {
  QSM_CUDA_TRY(launch_pdl_cluster(mx4_layer_kernel, dim3(ctas), dim3(kThreads), kCs, smem, stream, p));
  return QSM_OK;
}

}  // namespace mx4
}  // namespace qsm
