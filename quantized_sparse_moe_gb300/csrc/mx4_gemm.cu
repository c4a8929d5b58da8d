// The product of two MXFP4 matrices on the block-scaled tensor cores, and
// the grouped products of an MoE layer whose activations are MXFP4 as well.
//
//   y[m, n] = sum_b 2^(sa[m,b] + sw[n,b] - 254) sum_{c in b} a[m, c] w[n, c]
//
// The tensor cores take the 4-bit codes and the scales as they lie in
// memory, so nothing is expanded: a stage of the pipeline is 256 columns of
// 128 rows of a and of BN rows of w (128 bytes a row, TMA with the 128-byte
// swizzle) and their scale tiles (bulk copies), which go on to tensor
// memory with tcgen05.cp; four 64-wide MMAs then work off a stage.  Every
// product of two codes is exact, and the sums are fp32.
//
// Roles in a persistent CTA (one per SM): warp 0 loads, warp 1 issues the
// scale copies and the MMAs, warps 4-11 are the epilogue.  One accumulator
// of BN columns: the epilogue's threads take their half rows into registers
// at once (BN / 2 columns each), hand the accumulator back and convert and
// store while the next tile's MMAs run.  The outputs leave through swizzled
// boxes of 32 rows x 128 bytes per warp and TMA stores (or, where rows of y
// are not 16-byte aligned, through padded boxes and plain stores).  Of a
// short tile only the 32-row groups that exist are loaded and stored.
#include "mx4_gemm.cuh"

namespace qsm {
namespace mx4 {

namespace {

// Rows of y (pitch ldy elements) as boxes of 32 rows.
bool make_out_map(CUtensorMap* m, void* y, CUtensorMapDataType dt, int el, uint64_t rows, int cols,
                  size_t ldy, int box_cols, CUtensorMapSwizzle swz) {
  tc::EncodeTiledFn fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, rows};
  const cuuint64_t strides[1] = {ldy * el};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, 32};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, dt, 2, y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kStagePitch = 144;  // bytes of a row in a padded box (128 + 16)

template <int MODE, int BN, bool F32>
struct Cfg {
  static constexpr int kGroups = BN >= 128 ? BN / 128 : 1;  // scale tiles per column tile of w
  static constexpr int kABytes = 128 * 128;
  static constexpr int kWBytes = BN * 128;
  static constexpr int kSfaBytes = 2 * kTileBytes;
  static constexpr int kSfwBytes = 2 * kTileBytes * kGroups;
  static constexpr int kStage = kABytes + kWBytes + kSfaBytes + kSfwBytes;
  static constexpr int kStages = MODE == kGateUp ? 4 : BN == 256 ? 3 : BN == 128 ? 4 : 6;
  // the epilogue: a thread's columns, the bytes of them that make a box's
  // row, and the boxes of a warp (at most two at a time)
  static constexpr int NC = BN / 2;
  static constexpr int kEl = F32 ? 4 : 2;
  static constexpr int kInner = NC * kEl < 128 ? NC * kEl : 128;
  static constexpr int kBoxCols = kInner / kEl;
  static constexpr int kBoxes = NC / kBoxCols < 2 ? 1 : 2;
  static constexpr int kBoxBytes = kBoxes * 32 * kInner;
  static constexpr int kWarpBytes = MODE == kGateUp ? 0
                                    : kBoxBytes > 32 * kStagePitch ? kBoxBytes : (32 * kStagePitch + 1023) / 1024 * 1024;
  static constexpr int kSmem = kStages * kStage + kEpiWarps * kWarpBytes + 1024;
  static constexpr int kSfCols = 8 + 8 * kGroups;  // scale columns of one stage
  static constexpr int kTmem = BN == 256 ? 512 : BN == 128 ? 256 : 128;
  static_assert(kStage % 1024 == 0 && BN + 2 * kSfCols <= kTmem && kSmem <= 226 * 1024, "tile");
};

// Where a tile's operands and results lie.
struct Tile {
  int a_row, a_tile;   // first row of a, and its row tile of scales
  int cnt;             // rows of a that exist
  int e;               // expert, -1 = shared (grouped modes)
  int n0;              // first column of y (dense, down) or intermediate (gate_up)
  int w_row[2];        // first row of each box of w
  int w_tile[2];       // row tile of the scales of each 128 rows of w, -1: none
};

template <int MODE, int BN>
__device__ __forceinline__ Tile tile_of(const GemmParams& p, int item) {
  Tile t;
  const int tau = item / p.nsub, sub = item - tau * p.nsub;
  t.a_tile = tau;
  t.a_row = tau * 128;
  t.e = -1;
  int ebase = 0;  // the expert's first row of w
  if (MODE == kDense) {
    t.cnt = min(128, p.M - t.a_row);
  } else if (tau < p.shared_tiles) {
    t.cnt = min(128, p.T - t.a_row);
  } else {
    const int2 te = __ldcg(reinterpret_cast<const int2*>(p.tile_map) + (tau - p.shared_tiles));
    t.e = te.x;
    t.cnt = min(128, __ldcg(p.offsets + te.x + 1) - te.y);
    ebase = te.x * p.N;
  }
  if (MODE == kGateUp) {
    t.n0 = sub * 128;
    t.w_row[0] = ebase + t.n0;
    t.w_row[1] = ebase + p.N / 2 + t.n0;
    t.w_tile[0] = t.w_row[0] >> 7;
    t.w_tile[1] = t.w_row[1] >> 7;
  } else {
    t.n0 = sub * BN;
    t.w_row[0] = t.w_row[1] = ebase + t.n0;
    t.w_tile[0] = (ebase >> 7) + (t.n0 >> 7);
    t.w_tile[1] = t.n0 + 128 < p.N ? t.w_tile[0] + 1 : -1;
  }
  return t;
}

__device__ __forceinline__ Tile uniform_tile(Tile t) {
  t.e = uniform(t.e);
  t.cnt = uniform(t.cnt);
  t.a_row = uniform(t.a_row);
  t.a_tile = uniform(t.a_tile);
  t.w_row[0] = uniform(t.w_row[0]);
  t.w_row[1] = uniform(t.w_row[1]);
  t.w_tile[0] = uniform(t.w_tile[0]);
  t.w_tile[1] = uniform(t.w_tile[1]);
  return t;
}

// Eight (bf16) or four (fp32) consecutive outputs of a row, one by one, at
// column n of N.
template <bool F32>
__device__ __forceinline__ void store_chunk(void* y, size_t off, int n, int N, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 8); ++i) {
    if (n + i >= N) break;
    if (F32) static_cast<uint32_t*>(y)[off + i] = w[i];
    else static_cast<uint16_t*>(y)[off + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// This thread's NC columns of its row into registers: halves of the tile's
// columns for the dense and down modes; in gate_up, 64 gate columns and the
// 64 up columns of the same intermediates.
template <int MODE, int BN>
__device__ __forceinline__ void take_acc(uint32_t taddr, int half, uint32_t (&r)[BN / 2]) {
  constexpr int NC = BN / 2;
#pragma unroll
  for (int c = 0; c < NC; c += 32) {
    const int col = MODE == kGateUp ? (c < NC / 2 ? half * (NC / 2) + c : NC + half * (NC / 2) + c - NC / 2)
                                    : half * NC + c;
    tmem_ld32_nowait(taddr + col, r + c);
  }
#pragma unroll
  for (int c = 0; c < NC; c += 32) tmem_wait_ld32(r + c);
}

template <int MODE, int BN, bool F32>
__global__ void __launch_bounds__(kThreads, 1) mx4_gemm_kernel(const __grid_constant__ GemmParams p) {
  using C = Cfg<MODE, BN, F32>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], acc_full, acc_empty, done;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  volatile int* abort_p = &abort_flag;

  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&acc_empty, kEpiWarps);
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_map(&p.a);
    tc::prefetch_map(&p.w);
  }
  if (warp == 2) tc::tmem_alloc(&tmem_base, C::kTmem);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = uniform(tmem_base);

  // Grouped: the routing and the weights are older than the previous launch
  // (which let this one start after its own wait), so the first stages' weights
  // are requested before the wait; a (and what the epilogue overwrites) is
  // the previous launch's.
  if (MODE == kDense) {
    pdl_wait();
    pdl_launch_dependents();
  }
  const int tiles = MODE == kDense ? p.tiles : p.shared_tiles + uniform(__ldcg(p.n_tiles));
  const int total = tiles * p.nsub;
  const int nst = (p.K + kStageK - 1) / kStageK;
  const int cts = col_tiles(p.K);
  if (MODE != kDense && warp != 0) {
    pdl_wait();
    pdl_launch_dependents();
  }

  if (warp == 0) {
    int st = 0;          // ring position, and how often it came round
    uint32_t round = 0;
    bool waited = MODE == kDense;
    for (int item = blockIdx.x; item < total && !warp_aborted(abort_p); item += gridDim.x) {
      const Tile t = uniform_tile(tile_of<MODE, BN>(p, item));
      const bool sh = MODE != kDense && t.e < 0;
      const CUtensorMap* wm = sh ? &p.w_sh : &p.w;
      const uint8_t* wsc = sh ? p.w_scales_sh : p.w_scales;
      const int groups = C::kGroups == 1 || t.w_tile[1] < 0 ? 1 : 2;
      const uint8_t* asf = p.a_scales + (size_t)t.a_tile * cts * kTileBytes;
      const uint8_t* wsf0 = wsc + (size_t)t.w_tile[0] * cts * kTileBytes;
      const uint8_t* wsf1 = wsc + (size_t)(groups == 2 ? t.w_tile[1] : 0) * cts * kTileBytes;
      const int a32 = (t.cnt + 31) >> 5;  // groups of 32 rows of a that exist
      const uint32_t abytes = a32 * 32 * 128;
      auto load_w = [&](int ks, int s) {
        unsigned char* wb = smem + s * C::kStage + C::kABytes;
        const uint32_t sfb = (uint32_t)min(2, cts - 2 * ks) * kTileBytes;  // scale bytes of a row tile
        mbar_arrive_expect_tx(&full[s], abytes + C::kWBytes + sfb * (1 + groups));
        tc::tma_load_2d(wb, wm, ks * 128, t.w_row[0], &full[s]);
        if (MODE == kGateUp) tc::tma_load_2d(wb + 128 * 128, wm, ks * 128, t.w_row[1], &full[s]);
        unsigned char* sf = wb + C::kWBytes + C::kSfaBytes;
        bulk_g2s(sf, wsf0 + ks * 2 * kTileBytes, sfb, &full[s]);
        if (groups == 2) bulk_g2s(sf + 2 * kTileBytes, wsf1 + ks * 2 * kTileBytes, sfb, &full[s]);
      };
      auto load_a = [&](int ks, int s) {
        unsigned char* base = smem + s * C::kStage;
        const uint32_t sfb = (uint32_t)min(2, cts - 2 * ks) * kTileBytes;
        if (a32 == 4) {
          tc::tma_load_2d(base, &p.a, ks * 128, t.a_row, &full[s]);
        } else {
          for (int i = 0; i < a32; ++i)
            tc::tma_load_2d(base + i * 32 * 128, &p.a32, ks * 128, t.a_row + 32 * i, &full[s]);
        }
        bulk_g2s(base + C::kABytes + C::kWBytes, asf + ks * 2 * kTileBytes, sfb, &full[s]);
      };
      int k0 = 0;
      if (!waited) {  // the ring is empty
        k0 = min(nst, C::kStages);
        if (elect_one())
          for (int ks = 0; ks < k0; ++ks) load_w(ks, ks);
        __syncwarp();
        pdl_wait();
        pdl_launch_dependents();
        waited = true;
        if (elect_one())
          for (int ks = 0; ks < k0; ++ks) load_a(ks, ks);
        __syncwarp();
        st = k0 % C::kStages;
        round = k0 / C::kStages;
      }
      bool ok = true;
      for (int ks = k0; ks < nst; ++ks) {
        if (round > 0 && !warp_wait(&empty[st], (round - 1) & 1, abort_p, p.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          load_w(ks, st);
          load_a(ks, st);
        }
        __syncwarp();
        if (++st == C::kStages) st = 0, ++round;
      }
      if (!ok) break;
    }
    if (!waited) {  // no item
      pdl_wait();
      pdl_launch_dependents();
    }
    // after an abort, let the copies in flight land before the CTA exits
    for (int i = 0; i < C::kStages; ++i) {
      const uint32_t r = i < st ? round : round - 1;  // the last round of this position
      if (i < st || round > 0) mbar_wait_bounded(&full[i], r & 1, 1u << 16);
    }
    __syncwarp();
  } else if (warp == 1) {
    int st = 0, j = 0;
    uint32_t round = 0;
    const uint64_t desc0 = tc::sw128_desc(smem_u32(smem));
    for (int item = blockIdx.x; item < total && !warp_aborted(abort_p); item += gridDim.x, ++j) {
      // in tiles of 64 rows of w, every other one starts in the middle of a
      // scale tile: two columns on
      const int sf_off = BN == 64 ? ((item % p.nsub) & 1) * 2 : 0;
      if (j >= 1 && !warp_wait(&acc_empty, (j - 1) & 1, abort_p, p.status)) break;
      bool ok = true;
      for (int ks = 0; ks < nst; ++ks) {
        if (!warp_wait(&full[st], round & 1, abort_p, p.status)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = desc0 + (uint64_t)(st * (C::kStage >> 4)), wd = ad + (C::kABytes >> 4);
          const uint32_t sfa_s = smem_u32(smem) + st * C::kStage + C::kABytes + C::kWBytes;
          const uint32_t sfw_s = sfa_s + C::kSfaBytes;
          const uint32_t sfa = tmem + BN + (ks & 1) * C::kSfCols, sfw = sfa + 8;
          const int kv = min(kStageK, p.K - ks * kStageK);
#pragma unroll
          for (int ct = 0; ct < 2; ++ct) {
            if (ct * kTileCols >= kv) break;
            copy_scales(sfa + 4 * ct, sfa_s + ct * kTileBytes);
#pragma unroll
            for (int g = 0; g < C::kGroups; ++g)
              copy_scales(sfw + 4 * (ct * C::kGroups + g), sfw_s + (2 * g + ct) * kTileBytes);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk * 64 >= kv) break;
            mma_mxf4(tmem, ad + 2 * kk, wd + 2 * kk, idesc_mxf4(BN, kk & 1), sfa + 4 * (kk >> 1),
                     sfw + 4 * C::kGroups * (kk >> 1) + sf_off, (ks > 0 || kk > 0) ? 1u : 0u);
          }
          tc::mma_commit(&empty[st]);
          if (ks == nst - 1) tc::mma_commit(&acc_full);
        }
        __syncwarp();
        if (++st == C::kStages) st = 0, ++round;
      }
      if (!ok) break;
    }
    // every MMA issued has completed before tensor memory is freed
    if (elect_one()) tc::mma_commit(&done);
    __syncwarp();
    mbar_wait_bounded(&done, 0, kWaitIters);
  } else if (warp >= 4) {
    const int q4 = warp & 3, half = (warp - 4) >> 2;
    const int row = 32 * q4 + lane;
    unsigned char* stage = smem + C::kStages * C::kStage + (warp - 4) * C::kWarpBytes;
    const bool by_tma = p.vec != 0;
    const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16);
    bool bad = false;
    int j = 0;
    for (int item = blockIdx.x; item < total; item += gridDim.x, ++j) {
      if (warp_aborted(abort_p)) break;
      const Tile t = tile_of<MODE, BN>(p, item);
      if (!warp_wait(&acc_full, j & 1, abort_p, p.status)) break;
      tc::tc_fence_after();
      constexpr int NC = C::NC;
      if (32 * q4 >= t.cnt) {  // none of the warp's rows exist
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&acc_empty);
        continue;
      }
      uint32_t r[NC];
      take_acc<MODE, BN>(taddr, half, r);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&acc_empty);
      if (MODE == kGateUp) {
        // h of this row's 64 intermediates, quantized where it is formed
        if (row < t.cnt) {
          const size_t pos = (size_t)t.a_row + row;
          uint32_t sbytes = 0;
#pragma unroll
          for (int b = 0; b < NC / 64; ++b) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float h = silu(__uint_as_float(r[32 * b + i])) * __uint_as_float(r[NC / 2 + 32 * b + i]);
              r[32 * b + i] = __float_as_uint(h);
              m = max(m, r[32 * b + i] & 0x7fffffffu);
            }
            const uint32_t s = scale_of(m);
            if (s == 255u) bad = true;
            const float inv = s == 255u ? 0.f : inv_scale(s);
            uint32_t c[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[32 * b + 8 * w + i]) * inv;
              c[w] = f32x8_to_e2m1x8(v);
            }
            *reinterpret_cast<uint4*>(p.h_codes + (pos * p.I + t.n0 + half * (NC / 2) + 32 * b) / 2) =
                make_uint4(c[0], c[1], c[2], c[3]);
            sbytes |= s << (8 * b);
          }
          uint8_t* sw = p.h_scales + scale_word((int)pos, t.n0 >> 7, p.I >> 7);
          *reinterpret_cast<uint16_t*>(sw + 2 * half) = (uint16_t)sbytes;
        }
      } else {
        // 16-byte pieces of a row's outputs, from column c on
        __half2 top = __half2half2(__ushort_as_half(0));
        auto piece = [&](int c) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
              w[i] = r[c + i];
              continue;
            }
            const float a = __uint_as_float(r[c + 2 * i]), b = __uint_as_float(r[c + 2 * i + 1]);
            if (MODE == kDown) {  // fp16 of 1/16 the value
              const __half2 h = __floats2half2_rn(a * kOutScale, b * kOutScale);
              top = __hmax2(top, __habs2(h));
              w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
              w[i] = pack_bf16(a, b);
            }
          }
          return make_uint4(w[0], w[1], w[2], w[3]);
        };
        constexpr int kStep = C::kBoxes * C::kBoxCols;    // columns staged at a time
        constexpr int kPer = 16 / C::kEl;                 // columns in a piece
        const int col = t.n0 + half * NC;
#pragma unroll
        for (int c0 = 0; c0 < NC; c0 += kStep) {
          if (by_tma) {
            if (lane == 0) store_wait_read();  // the boxes may be written again
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kStep; c += kPer) {
              const int box = c / C::kBoxCols, ch = c % C::kBoxCols / kPer;
              const int sw = C::kInner == 128 ? lane & 7 : (lane >> 1) & 3;
              *reinterpret_cast<uint4*>(stage + box * 32 * C::kInner + lane * C::kInner + ((ch ^ sw) << 4)) =
                  piece(c0 + c);
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
              for (int box = 0; box < C::kBoxes; ++box)
                if (col + c0 + box * C::kBoxCols < p.N)
                  tma_store_2d(&p.y_map, stage + box * 32 * C::kInner, col + c0 + box * C::kBoxCols,
                               t.a_row + 32 * q4);
              store_commit();
            }
          } else {
#pragma unroll
            for (int box = 0; box < C::kBoxes; ++box) {
              __syncwarp();
#pragma unroll
              for (int ch = 0; ch < C::kInner / 16; ++ch)
                *reinterpret_cast<uint4*>(stage + lane * kStagePitch + ch * 16) =
                    piece(c0 + box * C::kBoxCols + ch * kPer);
              __syncwarp();
              constexpr int kChunks = C::kInner / 16;
              for (int i = lane; i < 32 * kChunks; i += 32) {
                const int rr = i / kChunks, ch = i % kChunks;
                const int n = col + c0 + box * C::kBoxCols + ch * kPer;
                if (32 * q4 + rr < t.cnt && n < p.N)
                  store_chunk<F32>(p.y, ((size_t)t.a_row + 32 * q4 + rr) * p.ldy + n, n, p.N,
                                   *reinterpret_cast<const uint4*>(stage + rr * kStagePitch + ch * 16));
              }
            }
          }
        }
        if (MODE == kDown && row < t.cnt && (__hisinf(__low2half(top)) || __hisinf(__high2half(top)))) bad = true;
      }
    }
    if (MODE != kGateUp && lane == 0) store_wait();
    if (bad) set_status(p.status, MODE == kGateUp ? QSM_DEV_NONFINITE : QSM_DEV_FP16_RANGE);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 2) tc::tmem_dealloc(tmem, C::kTmem);
}

template <int MODE, int BN, bool F32>
qsm_status launch_tile(GemmParams& p, int most, uint64_t rows, cudaStream_t stream) {
  using C = Cfg<MODE, BN, F32>;
  auto* k = mx4_gemm_kernel<MODE, BN, F32>;
  static thread_local int ready_dev = -1;  // the attribute is per device
  int dev = 0;
  QSM_CUDA_TRY(cudaGetDevice(&dev));
  if (ready_dev != dev) {
    QSM_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
    ready_dev = dev;
  }
  if (MODE != kGateUp && p.vec &&
      !make_out_map(&p.y_map, p.y, MODE == kDown ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                   : F32         ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    C::kEl, rows, p.N, p.ldy, C::kBoxCols,
                    C::kInner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return QSM_ERR_CUDA;
  const int grid = most < sm_count() ? most : sm_count();
  QSM_CUDA_TRY(launch_pdl(k, dim3(grid), dim3(kThreads), C::kSmem, stream, p));
  return QSM_OK;
}

template <int BN>
qsm_status launch_dense(GemmParams& p, const qsm_mx4* w, bool f32, cudaStream_t stream) {
  if (!make_codes_map(&p.w, w->codes, w->rows, w->cols, BN)) return QSM_ERR_CUDA;
  p.nsub = (p.N + BN - 1) / BN;
  if ((long long)p.tiles * p.nsub > (1ll << 30)) return QSM_ERR_UNSUPPORTED;
  const int most = p.tiles * p.nsub;
  return f32 ? launch_tile<kDense, BN, true>(p, most, p.M, stream)
             : launch_tile<kDense, BN, false>(p, most, p.M, stream);
}

}  // namespace

bool make_a_maps(GemmParams* p, const void* codes, uint64_t rows, int K) {
  return make_codes_map(&p->a, codes, rows, K, 128) && make_codes_map(&p->a32, codes, rows, K, 32);
}

qsm_status launch_grouped(GemmParams& p, int mode, uint64_t rows, cudaStream_t stream) {
  const int most = 1 << 30;  // how many tiles there are is known on the device only
  return mode == kGateUp ? launch_tile<kGateUp, 256, false>(p, most, rows, stream)
                         : launch_tile<kDown, 256, false>(p, most, rows, stream);
}

}  // namespace mx4
}  // namespace qsm

extern "C" qsm_status mx4_gemm(const qsm_mx4* a, const qsm_mx4* w, int32_t dtype, void* y,
                               int64_t ldy, int32_t* dev_status, cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::mx4;
  if (!a || !w || (dtype != QSM_BF16 && dtype != QSM_FP32)) return QSM_ERR_INVALID_ARGUMENT;
  if (a->experts != 1 || w->experts != 1 || a->cols != w->cols || a->rows < 0 || w->rows < 0 ||
      ldy < w->rows)
    return QSM_ERR_INVALID_ARGUMENT;
  if (a->rows == 0 || w->rows == 0) return QSM_OK;
  const size_t el = dtype == QSM_FP32 ? 4 : 2;
  if (!mx4_valid(a) || !mx4_valid(w) || !y || !dev_status || !aligned4(dev_status) ||
      reinterpret_cast<uintptr_t>(y) % el)
    return QSM_ERR_INVALID_ARGUMENT;
  GemmParams p = {};
  p.M = a->rows;
  p.N = w->rows;
  p.K = a->cols;
  p.tiles = row_tiles(p.M);
  p.y = y;
  p.ldy = (size_t)ldy;
  p.vec = aligned16(y) && (size_t)ldy * el % 16 == 0;
  p.a_scales = a->scales;
  p.w_scales = w->scales;
  p.status = dev_status;
  if (!make_a_maps(&p, a->codes, a->rows, a->cols)) return QSM_ERR_CUDA;
  // the widest tile that still gives every SM one
  const int nsm = sm_count();
  const long long t256 = (long long)p.tiles * ((p.N + 255) / 256);
  const long long t128 = (long long)p.tiles * ((p.N + 127) / 128);
  const bool f32 = dtype == QSM_FP32;
  if (t256 >= nsm) return launch_dense<256>(p, w, f32, stream);
  if (t128 >= nsm) return launch_dense<128>(p, w, f32, stream);
  return launch_dense<64>(p, w, f32, stream);
}
