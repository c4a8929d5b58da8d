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
// scale copies and the MMAs, warps 4-11 are the epilogue.  Two accumulators
// of BN columns, or one of 256 (two leave no tensor memory for the scales).
// The epilogue's threads take their half rows into registers at once (BN / 2
// columns each), hand the accumulator back and convert and store while the
// next tile's MMAs run.  Of a short tile only the rows that exist are loaded
// (in groups of 8) and stored.
//
// Measured (graph replay): 300 x 2048 x 2048 4.5 us, 4096 x 8192 x 2048 31 us (4.4
// PFLOP/s), x 8192 78 us (7.0; a pair of SMs per tile, see there).  In the MoE layer of H 2048,
// I 512 and 256 experts, gate_up takes 50 us at 300 tokens (286 MB of weights, 5.7
// TB/s: HBM) and 55 at 4096 (802 MB through L2, 14 TB/s: that), down 26 and 51.
#include <mutex>

#include "mx4_gemm.cuh"

namespace qsm {
namespace mx4 {

namespace {

// fp16 outputs [rows, cols] as swizzled boxes of 64 columns and box_rows rows.
bool make_out_map(CUtensorMap* m, void* y, uint64_t rows, int cols, int box_rows) {
  return tc::make_map_2d(m, y, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, rows, cols, 64, box_rows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kDownBox = 32 * 128;  // bytes of a swizzled box of down: 32 rows of 64 outputs
constexpr int kBoxBytes = 64;   // of a row in a warp's box, for outputs that are not aligned
constexpr int kBoxPitch = 80;   // 16 more: the rows fall in different banks

template <int MODE, int BN, bool F32>
struct Cfg {
  static constexpr int kGroups = (BN + 127) / 128;  // scale tiles per column tile of w
  static constexpr int kABytes = 128 * 128;
  static constexpr int kWBytes = BN * 128;
  static constexpr int kSfaBytes = 2 * kTileBytes;
  static constexpr int kSfwBytes = 2 * kTileBytes * kGroups;
  static constexpr int kStage = kABytes + kWBytes + kSfaBytes + kSfwBytes;
  static constexpr int kStages = MODE == kDown ? 3 : BN == 256 ? 4 : 6;
  static constexpr int NC = BN / 2;  // columns of an epilogue thread
  static constexpr int kWarpBytes = MODE == kGateUp ? 0 : MODE == kDown ? NC / 64 * kDownBox : 32 * kBoxPitch;
  static constexpr int kSmem = kStages * kStage + kEpiWarps * kWarpBytes + 1024;
  static constexpr int kSfCols = 8 + 8 * kGroups;  // scale columns of one stage
  static constexpr int kAcc = BN == 256 ? 1 : 2;   // accumulators
  static constexpr int kTmem = BN == 64 ? 256 : 512;
  static_assert(kStage % 1024 == 0 && kAcc * BN + 2 * kSfCols <= kTmem && kSmem <= 226 * 1024, "tile");
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

// Which expert (-1: shared) row tile tau of a grouped product belongs to, and
// how many of its rows exist: two dependent loads, 1.3 us.
__device__ __forceinline__ int2 group_of(const GemmParams& p, int tau) {
  if (tau < p.shared_tiles) return make_int2(-1, min(128, p.T - tau * 128));
  const int2 te = __ldcg(reinterpret_cast<const int2*>(p.tile_map) + (tau - p.shared_tiles));
  return make_int2(te.x, min(128, __ldcg(p.offsets + te.x + 1) - te.y));
}

// So a CTA looks its items' tiles up together, once; the first kTab of them.
constexpr int kTab = 64;

// The n-th item of the CTA.
template <int MODE, int BN>
__device__ __forceinline__ Tile tile_of(const GemmParams& p, const int2* tab, int item, int n) {
  Tile t;
  const int tau = item / p.nsub, sub = item - tau * p.nsub;
  t.a_tile = tau;
  t.a_row = tau * 128;
  t.e = -1;
  int ebase = 0;  // the expert's first row of w
  if (MODE == kDense) {
    t.cnt = min(128, p.M - t.a_row);
  } else {
    const int2 g = n < kTab ? tab[n] : group_of(p, tau);
    t.e = g.x;
    t.cnt = g.y;
    ebase = max(g.x, 0) * p.N;
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
    t.w_tile[0] = t.w_row[0] >> 7;
    t.w_tile[1] = (t.n0 & ~127) + 128 < p.N ? t.w_tile[0] + 1 : -1;
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

__device__ __forceinline__ void store_sector(void* dst, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
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

// The NC outputs that each lane of a warp holds of its row (row 32 q4 + lane of
// the cnt that exist from row0 on), columns col .. of y.  Where rows of y are
// aligned they go out from the registers, a sector of 32 bytes per lane and
// instruction: shared memory has enough to do with the operands (4096 x 8192 x
// 2048: 31.3 us; by swizzled boxes and TMA 34.7).  Else by way of the warp's box
// at `stage`, so that lanes write neighbouring bytes.
template <int BN, bool F32>
__device__ __forceinline__ void store_dense(const GemmParams& p, const uint32_t (&r)[BN / 2], int row0,
                                            int cnt, int col, int q4, int lane, unsigned char* stage) {
  using C = Cfg<kDense, BN, F32>;
  constexpr int kEl = F32 ? 4 : 2, kPer = 16 / kEl;  // kPer: columns in a 16-byte piece
  auto piece = [&](int c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = F32 ? r[c + i] : pack_bf16(__uint_as_float(r[c + 2 * i]), __uint_as_float(r[c + 2 * i + 1]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  if (p.align >= 16) {
    if (32 * q4 + lane >= cnt) return;
    const size_t at = ((size_t)row0 + 32 * q4 + lane) * p.ldy + col;
#pragma unroll
    for (int c = 0; c < C::NC; c += 2 * kPer) {
      const uint4 v0 = piece(c), v1 = piece(c + kPer);
      if (col + c + 2 * kPer <= p.N) {
        char* dst = static_cast<char*>(p.y) + (at + c) * kEl;
        if (p.align == 32) {
          store_sector(dst, v0, v1);
        } else {
          reinterpret_cast<uint4*>(dst)[0] = v0;
          reinterpret_cast<uint4*>(dst)[1] = v1;
        }
      } else {
        store_chunk<F32>(p.y, at + c, col + c, p.N, v0);
        store_chunk<F32>(p.y, at + c + kPer, col + c + kPer, p.N, v1);
      }
    }
  } else {
    constexpr int kChunks = kBoxBytes / 16;
#pragma unroll
    for (int c0 = 0; c0 < C::NC; c0 += kChunks * kPer) {
      __syncwarp();
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch)
        *reinterpret_cast<uint4*>(stage + lane * kBoxPitch + ch * 16) = piece(c0 + ch * kPer);
      __syncwarp();
      for (int i = lane; i < 32 * kChunks; i += 32) {
        const int rr = i / kChunks, ch = i % kChunks;
        const int n = col + c0 + ch * kPer;
        if (32 * q4 + rr < cnt && n < p.N)
          store_chunk<F32>(p.y, ((size_t)row0 + 32 * q4 + rr) * p.ldy + n, n, p.N,
                           *reinterpret_cast<const uint4*>(stage + rr * kBoxPitch + ch * 16));
      }
    }
  }
}

// The same of down, in fp16 with a power of two of the row's 128 columns taken
// out, which goes to y_scale: the largest magnitude lies in 2^14 .. 2^15 then,
// and what is down to 2^-29 of it keeps 11 bits (the bf16 result has 8), whatever
// the magnitude; under 2^-86 the power stays 2^-100.  It is at most 2^4, so
// that an output that does not fit (2^20 and more) is reported (bad).  By way of
// swizzled boxes of 32 rows x 128 bytes at `stage` and TMA: with two stages
// of K per tile the outputs are what counts, and whole lines cost L2 less than
// sectors (4096 tokens, H = 2048: 185.1 us a layer, with sectors 188.6, both
// before the powers of two).
template <int BN>
__device__ __forceinline__ void store_down(const GemmParams& p, const uint32_t (&r)[BN / 2], int row0, int cnt,
                                           int col, int q4, int lane, unsigned char* stage, bool& bad) {
  constexpr int NC = BN / 2;
  static_assert(NC == kOutCols, "a thread has a power of two's columns");
  if (col >= p.N) return;  // N is a multiple of NC: all of them
  float top = 0.f;  // (a NaN does not count, and stays one)
#pragma unroll
  for (int c = 0; c < NC; ++c) top = fmaxf(top, fabsf(__uint_as_float(r[c])));
  const int sh = min(max(14 + 127 - (int)(__float_as_uint(top) >> 23), -4), 100);
  const float f = __uint_as_float((uint32_t)(127 + sh) << 23);
  if (lane == 0) store_wait_read();  // the boxes may be written again
  __syncwarp();
#pragma unroll
  for (int c = 0; c < NC; c += 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(__uint_as_float(r[c + 2 * i]) * f,
                                          __uint_as_float(r[c + 2 * i + 1]) * f);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(stage + c / 64 * kDownBox + lane * 128 + ((c % 64 / 8 ^ (lane & 7)) << 4)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  tc::fence_async_smem();
  __syncwarp();
  const int rows = cnt - 32 * q4;  // that exist of the warp's 32
  if (lane == 0) {
#pragma unroll
    for (int box = 0; box < NC / 64; ++box) {
      const unsigned char* src = stage + box * kDownBox;
      if (rows > 24) {
        tma_store_2d(&p.y_map, src, col + 64 * box, row0 + 32 * q4);
      } else {
        for (int i = 0; i < rows; i += 8)
          tma_store_2d(&p.y8_map, src + i * 128, col + 64 * box, row0 + 32 * q4 + i);
      }
    }
    store_commit();
  }
  if (lane < rows) {
    p.y_scale[((size_t)row0 + 32 * q4 + lane) * (p.N / NC) + col / NC] = __uint_as_float((uint32_t)(127 - sh) << 23);
    if (top >= 65520.f * 16.f) bad = true;  // rounds past the largest fp16 (or is infinite)
  }
}

template <int MODE, int BN, bool F32>
__global__ void __launch_bounds__(kThreads, 1) mx4_gemm_kernel(const __grid_constant__ GemmParams p) {
  using C = Cfg<MODE, BN, F32>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], acc_full[C::kAcc],
      acc_empty[C::kAcc], done;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ int2 tab[MODE == kDense ? 1 : kTab];
  volatile int* abort_p = &abort_flag;

  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kAcc; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
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
  const int nst = k_stages(p.K);
  const int cts = col_tiles(p.K);
  if (MODE != kDense) {
    const int item = blockIdx.x + threadIdx.x * gridDim.x;
    if (threadIdx.x < kTab && item < total) tab[threadIdx.x] = group_of(p, item / p.nsub);
    __syncthreads();
  }
  if (MODE != kDense && warp != 0) {
    pdl_wait();
    pdl_launch_dependents();
  }

  if (warp == 0) {
    int st = 0;          // ring position, and how often it came round
    uint32_t round = 0;
    bool waited = MODE == kDense;
    int n = 0;
    for (int item = blockIdx.x; item < total && !warp_aborted(abort_p); item += gridDim.x, ++n) {
      const Tile t = uniform_tile(tile_of<MODE, BN>(p, tab, item, n));
      const bool sh = MODE != kDense && t.e < 0;
      const CUtensorMap* wm = sh ? &p.w_sh : &p.w;
      const uint8_t* wsc = sh ? p.w_scales_sh : p.w_scales;
      const int groups = C::kGroups == 1 || t.w_tile[1] < 0 ? 1 : 2;
      const uint8_t* asf = p.a_scales + (size_t)t.a_tile * cts * kTileBytes;
      const uint8_t* wsf0 = wsc + (size_t)t.w_tile[0] * cts * kTileBytes;
      const uint8_t* wsf1 = wsc + (size_t)(groups == 2 ? t.w_tile[1] : 0) * cts * kTileBytes;
      // rows of a that exist, in groups of 8 (up to 32) or of 32
      const int a8 = (t.cnt + 7) >> 3, a32 = (t.cnt + 31) >> 5;
      const uint32_t abytes = (a8 <= 4 ? a8 * 8 : a32 * 32) * 128;
      auto load_w = [&](int ks, int s) {
        unsigned char* wb = smem + s * C::kStage + C::kABytes;
        const uint32_t sfb = (uint32_t)min(2, cts - 2 * ks) * kTileBytes;  // scale bytes of a row tile
        mbar_arrive_expect_tx(&full[s], abytes + C::kWBytes + sfb * (1 + groups));
        tc::tma_load_2d(wb, wm, ks * 128, t.w_row[0], &full[s]);
        if (MODE == kGateUp) tc::tma_load_2d(wb + 128 * 128, wm, ks * 128, t.w_row[1], &full[s]);
        unsigned char* sf = wb + C::kWBytes + C::kSfaBytes;
        bulk_g2s(sf, wsf0 + (size_t)ks * 2 * kTileBytes, sfb, &full[s]);
        if (groups == 2) bulk_g2s(sf + 2 * kTileBytes, wsf1 + (size_t)ks * 2 * kTileBytes, sfb, &full[s]);
      };
      auto load_a = [&](int ks, int s) {
        unsigned char* base = smem + s * C::kStage;
        const uint32_t sfb = (uint32_t)min(2, cts - 2 * ks) * kTileBytes;
        if (a32 == 4) {
          tc::tma_load_2d(base, &p.a, ks * 128, t.a_row, &full[s]);
        } else if (a8 > 4) {
          for (int i = 0; i < a32; ++i)
            tc::tma_load_2d(base + i * 32 * 128, &p.a32, ks * 128, t.a_row + 32 * i, &full[s]);
        } else {
          for (int i = 0; i < a8; ++i)
            tc::tma_load_2d(base + i * 8 * 128, &p.a8, ks * 128, t.a_row + 8 * i, &full[s]);
        }
        bulk_g2s(base + C::kABytes + C::kWBytes, asf + (size_t)ks * 2 * kTileBytes, sfb, &full[s]);
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
    uint32_t round = 0, fs = 0;
    const uint64_t desc0 = tc::sw128_desc(smem_u32(smem));
    for (int item = blockIdx.x; item < total && !warp_aborted(abort_p); item += gridDim.x, ++j) {
      // tiles of 64 rows of w: every other one starts in the middle
      // of a scale tile, two columns on
      const int sf_off = BN % 128 ? ((item % p.nsub) & 1) * 2 : 0;
      const int ab = j % C::kAcc;
      const uint32_t acc = tmem + ab * BN;
      if (j >= C::kAcc && !warp_wait(&acc_empty[ab], (j / C::kAcc - 1) & 1, abort_p, p.status)) break;
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
          const uint32_t sfa = tmem + C::kAcc * BN + (fs & 1) * C::kSfCols, sfw = sfa + 8;
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
            mma_mxf4(acc, ad + 2 * kk, wd + 2 * kk, idesc_mxf4(BN, kk & 1), sfa + 4 * (kk >> 1),
                     sfw + 4 * C::kGroups * (kk >> 1) + sf_off, (ks > 0 || kk > 0) ? 1u : 0u);
          }
          tc::mma_commit(&empty[st]);
          if (ks == nst - 1) tc::mma_commit(&acc_full[ab]);
        }
        __syncwarp();
        ++fs;
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
    const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16);
    bool bad = false;
    int j = 0;
    for (int item = blockIdx.x; item < total; item += gridDim.x, ++j) {
      if (warp_aborted(abort_p)) break;
      const Tile t = tile_of<MODE, BN>(p, tab, item, j);
      const int ab = j % C::kAcc;
      if (!warp_wait(&acc_full[ab], (j / C::kAcc) & 1, abort_p, p.status)) break;
      tc::tc_fence_after();
      constexpr int NC = C::NC;
      if (32 * q4 >= t.cnt) {  // none of the warp's rows exist
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&acc_empty[ab]);
        continue;
      }
      uint32_t r[NC];
      take_acc<MODE, BN>(taddr + ab * BN, half, r);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&acc_empty[ab]);
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
      } else if constexpr (MODE == kDown) {
        store_down<BN>(p, r, t.a_row, t.cnt, t.n0 + half * NC, q4, lane, stage, bad);
      } else {
        store_dense<BN, F32>(p, r, t.a_row, t.cnt, t.n0 + half * NC, q4, lane, stage);
      }
    }
    if (MODE == kDown && lane == 0) store_wait();
    if (bad) set_status(p.status, MODE == kGateUp ? QSM_DEV_NONFINITE : QSM_DEV_FP16_RANGE);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 2) tc::tmem_dealloc(tmem, C::kTmem);
}

// The dense product on pairs of SMs: one MMA of 256 rows of a x 256 rows of w
// runs on the tensor cores of both CTAs of a cluster.  Each CTA loads its own
// 128 rows of a and half of the rows of w, and the hardware reads the other
// half from its neighbour: 256 rows a stage and CTA instead of 384, which is
// what counts, because a 128 x 256 tile on one SM is bound by what an SM can
// take from L2 (55 bytes a cycle, 26 us for 4096 x 8192 x 2048, where the MMAs
// need 15; with the pair the copies alone take 16 us, with the MMAs 25, with the
// 67 MB of outputs 31; with four stages of K instead of five 33).  Every copy
// of either CTA reports to the leader's (rank 0) barrier; the leader issues the
// scale copies, which move each CTA's tiles into its own tensor memory, and the
// MMAs, and its commits arrive in both.  The scales of w are needed whole in
// both.
template <bool F32>
struct Pair {
  using C = Cfg<kDense, 256, F32>;
  static constexpr int kHalf = 128 * 128;  // codes of 128 rows
  static constexpr int kStage = 2 * kHalf + 6 * kTileBytes;
  static constexpr int kStages = 5;
  static constexpr int kSmem = kStages * kStage + kEpiWarps * C::kWarpBytes + 1024;
  static_assert(kStage % 1024 == 0 && kSmem <= 226 * 1024, "stages");
};

// TMA load of a CTA pair: the box to this CTA, its bytes to the barrier at
// cluster address `bar`, in either CTA.
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, int c0, int c1,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_copy_scales(uint32_t taddr, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(scale_desc(saddr))
               : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs once every MMA issued so far has completed.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 1) mx4_gemm_pair_kernel(const __grid_constant__ GemmParams p) {
  using C = Cfg<kDense, 256, F32>;
  using P = Pair<F32>;
  extern __shared__ unsigned char smem_raw[];
  // the same offset in both CTAs: descriptors and barriers are shared
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[P::kStages], empty[P::kStages], acc_full, acc_empty, done;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  volatile int* abort_p = &abort_flag;

  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < P::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&acc_empty, 2 * kEpiWarps);
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc::tc_fence_after();
  const uint32_t tmem = uniform(tmem_base);

  pdl_wait();
  pdl_launch_dependents();
  const int total = p.tiles * p.nsub, pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  const int nst = k_stages(p.K), cts = col_tiles(p.K);

  if (warp == 0) {
    int st = 0;
    uint32_t round = 0;
    for (int item = pair; item < total && !warp_aborted(abort_p); item += pairs) {
      const int mt = item / p.nsub, nt = item - mt * p.nsub;
      const int a_tile = 2 * mt + rank, w_row = nt * 256 + rank * 128;
      bool ok = true;
      for (int ks = 0; ks < nst; ++ks) {
        if (round > 0 && !warp_wait(&empty[st], (round - 1) & 1, abort_p, p.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          unsigned char* base = smem + st * P::kStage;
          const uint32_t bar = dsmem_addr(&full[st], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * P::kStage);
          pair_load_2d(base, &p.a, ks * 128, a_tile * 128, bar);
          pair_load_2d(base + P::kHalf, &p.w, ks * 128, w_row, bar);
          unsigned char* sf = base + 2 * P::kHalf;  // two column tiles of each row tile
          pair_load_2d(sf, &p.a_sf, 0, a_tile * cts + 2 * ks, bar);
          pair_load_2d(sf + 2 * kTileBytes, &p.w_sf, 0, 2 * nt * cts + 2 * ks, bar);
          pair_load_2d(sf + 4 * kTileBytes, &p.w_sf, 0, (2 * nt + 1) * cts + 2 * ks, bar);
        }
        __syncwarp();
        if (++st == P::kStages) st = 0, ++round;
      }
      if (!ok) break;
    }
    // after an abort, let the copies in flight land before the CTAs exit (neither
    // does before the cluster barrier at the end): the leader waits for both
    // CTAs' on its barriers, which the other cannot wait on; as the two may have
    // stopped at different stages, each stays for a millisecond besides, hundreds
    // of times what a copy takes
    if (rank == 0)
      for (int i = 0; i < P::kStages; ++i) {
        const uint32_t r = i < st ? round : round - 1;  // the last round of this position
        if (i < st || round > 0) mbar_wait_bounded(&full[i], r & 1, 1u << 16);
      }
    if (warp_aborted(abort_p))
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      int st = 0, j = 0;
      uint32_t round = 0;
      const uint64_t desc0 = tc::sw128_desc(smem_u32(smem));
      for (int item = pair; item < total && !warp_aborted(abort_p); item += pairs, ++j) {
        if (j >= 1 && !__all_sync(0xffffffffu, wait_cluster(&acc_empty, (j - 1) & 1, abort_p, p.status)))
          break;
        bool ok = true;
        for (int ks = 0; ks < nst; ++ks) {
          if (!warp_wait(&full[st], round & 1, abort_p, p.status)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = desc0 + (uint64_t)(st * (P::kStage >> 4)), wd = ad + (P::kHalf >> 4);
            const uint32_t sf = smem_u32(smem) + st * P::kStage + 2 * P::kHalf;
            const uint32_t sfa = tmem + 256 + (ks & 1) * 24, sfw = sfa + 8;
            const int kv = min(kStageK, p.K - ks * kStageK);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
              if (ct * kTileCols >= kv) break;
              pair_copy_scales(sfa + 4 * ct, sf + ct * kTileBytes);
              pair_copy_scales(sfw + 8 * ct, sf + (2 + ct) * kTileBytes);
              pair_copy_scales(sfw + 8 * ct + 4, sf + (4 + ct) * kTileBytes);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk * 64 >= kv) break;
              // M = 256: twice the rows of the one-CTA descriptor
              pair_mma(tmem, ad + 2 * kk, wd + 2 * kk, idesc_mxf4(256, kk & 1) + (8u << 24),
                       sfa + 4 * (kk >> 1), sfw + 8 * (kk >> 1), (ks > 0 || kk > 0) ? 1u : 0u);
            }
            pair_commit(&empty[st]);
            if (ks == nst - 1) pair_commit(&acc_full);
          }
          __syncwarp();
          if (++st == P::kStages) st = 0, ++round;
        }
        if (!ok) break;
      }
      // every MMA issued has completed before tensor memory is freed
      if (elect_one()) pair_commit(&done);
      __syncwarp();
    }
    mbar_wait_bounded(&done, 0, kWaitIters);
  } else if (warp >= 4) {
    const int q4 = warp & 3, half = (warp - 4) >> 2;
    unsigned char* stage = smem + P::kStages * P::kStage + (warp - 4) * C::kWarpBytes;
    const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16);
    const uint32_t acc_bar = dsmem_addr(&acc_empty, 0);
    int j = 0;
    for (int item = pair; item < total; item += pairs, ++j) {
      if (warp_aborted(abort_p)) break;
      const int mt = item / p.nsub, nt = item - mt * p.nsub;
      const int row0 = (2 * mt + rank) * 128, cnt = min(128, p.M - row0);
      if (!warp_wait(&acc_full, j & 1, abort_p, p.status)) break;
      tc::tc_fence_after();
      uint32_t r[C::NC];
      if (32 * q4 < cnt) take_acc<kDense, 256>(taddr, half, r);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(acc_bar);
      if (32 * q4 < cnt) store_dense<256, F32>(p, r, row0, cnt, nt * 256 + half * C::NC, q4, lane, stage);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while the other's copies and MMAs use it
  tc::tc_fence_after();
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int MODE, int BN, bool F32>
qsm_status launch_tile(GemmParams& p, int most, cudaStream_t stream) {
  using C = Cfg<MODE, BN, F32>;
  auto* k = mx4_gemm_kernel<MODE, BN, F32>;
  static thread_local int ready_dev = -1;  // the attribute is per device
  int dev = 0;
  QSM_CUDA_TRY(cudaGetDevice(&dev));
  if (ready_dev != dev) {
    QSM_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
    ready_dev = dev;
  }
  const int grid = most < sm_count() ? most : sm_count();
  QSM_CUDA_TRY(launch_pdl(k, dim3(grid), dim3(kThreads), C::kSmem, stream, p));
  return QSM_OK;
}

// Clusters of two that the device holds at once (asked once per device).
int resident_pairs(void* kernel, int smem) {
  static std::mutex mu;
  static int known[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sm_count() / 2 * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
    known[dev] = n;
  }
  return known[dev];
}

// Scale tiles of [rows, cols] as rows of 512 bytes, two at a time.
bool make_scales_map(CUtensorMap* m, const uint8_t* scales, int rows, int cols) {
  return tc::make_map_2d(m, scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4,
                         (uint64_t)row_tiles(rows) * col_tiles(cols), kTileBytes / 4, kTileBytes / 4, 2,
                         CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <bool F32>
qsm_status launch_pair(GemmParams& p, const qsm_mx4* a, const qsm_mx4* w, cudaStream_t stream) {
  using P = Pair<F32>;
  auto* k = mx4_gemm_pair_kernel<F32>;
  static thread_local int ready_dev = -1;
  int dev = 0;
  QSM_CUDA_TRY(cudaGetDevice(&dev));
  if (ready_dev != dev) {
    QSM_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem));
    ready_dev = dev;
  }
  p.tiles = (p.M + 255) / 256;
  p.nsub = (p.N + 255) / 256;
  if ((long long)p.tiles * p.nsub > (1ll << 30)) return QSM_ERR_UNSUPPORTED;
  if (!make_codes_map(&p.w, w->codes, w->rows, w->cols, 128) ||
      !make_scales_map(&p.a_sf, a->scales, a->rows, a->cols) ||
      !make_scales_map(&p.w_sf, w->scales, w->rows, w->cols))
    return QSM_ERR_CUDA;
  const int most = resident_pairs(reinterpret_cast<void*>(k), P::kSmem), items = p.tiles * p.nsub;
  if (most < 1) return QSM_ERR_CUDA;
  QSM_CUDA_TRY(launch_pdl_cluster(k, dim3(2 * (items < most ? items : most)), dim3(kThreads), 2, P::kSmem,
                                  stream, p));
  return QSM_OK;
}

template <int BN>
qsm_status launch_dense(GemmParams& p, const qsm_mx4* w, bool f32, cudaStream_t stream) {
  if (!make_codes_map(&p.w, w->codes, w->rows, w->cols, BN)) return QSM_ERR_CUDA;
  p.nsub = (p.N + BN - 1) / BN;
  if ((long long)p.tiles * p.nsub > (1ll << 30)) return QSM_ERR_UNSUPPORTED;
  const int most = p.tiles * p.nsub;
  return f32 ? launch_tile<kDense, BN, true>(p, most, stream)
             : launch_tile<kDense, BN, false>(p, most, stream);
}

}  // namespace

bool make_a_maps(GemmParams* p, const void* codes, uint64_t rows, int K) {
  return make_codes_map(&p->a, codes, rows, K, 128) && make_codes_map(&p->a32, codes, rows, K, 32) &&
         make_codes_map(&p->a8, codes, rows, K, 8);
}

qsm_status launch_grouped(GemmParams& p, int mode, uint64_t rows, cudaStream_t stream) {
  const int most = 1 << 30;  // how many tiles there are is known on the device only
  if (mode == kDown && (!make_out_map(&p.y_map, p.y, rows, p.N, 32) || !make_out_map(&p.y8_map, p.y, rows, p.N, 8)))
    return QSM_ERR_CUDA;
  return mode == kGateUp ? launch_tile<kGateUp, 256, false>(p, most, stream)
                         : launch_tile<kDown, kDownRows, false>(p, most, stream);
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
  const uintptr_t bits = reinterpret_cast<uintptr_t>(y) | (uintptr_t)ldy * el;
  p.align = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 0;
  p.a_scales = a->scales;
  p.w_scales = w->scales;
  p.status = dev_status;
  if (!make_a_maps(&p, a->codes, a->rows, a->cols)) return QSM_ERR_CUDA;
  // The width with the least waves of tiles x cost of a wave, which is about
  // 6 : 7 : 12 for tiles of 64, 128 and 256 columns, and 12 for 256 x 256 on
  // a pair of SMs.  Measured, in that order (us): 300 x 2048 x 2048 4.5 5.1 6.6
  // 7.0, 512 x 4096 x 2048 6.7 5.3 6.8 7.2, 640 x 8192 x 2048 13.7 9.8 10.1 10.8,
  // 1024 x 4096 x 2048 11.5 7.7 6.9 7.8, 2048 x 4096 x 2048 18.5 12.5 10.7 11.6.
  // Among equals the wider tile, and the pair where its smaller operand traffic
  // pays (128, 256, pair): 4096 x 8192 x 1024 23.8 22.1 24.4, x 2048 36.9 31.5
  // 31.2, x 4096 67.0 51.0 47.3, x 8192 126 89.2 78.6; 1024 x 8192 x 2048 13.0
  // 11.2 11.9, x 4096 21.2 16.4 16.0, x 8192 38.7 28.9 26.6.
  const int nsm = sm_count();
  const bool f32 = dtype == QSM_FP32;
  auto waves = [](long long tiles, int at_once) { return (tiles + at_once - 1) / at_once; };
  auto tiles = [&](int bn) { return (long long)p.tiles * ((p.N + bn - 1) / bn); };
  const long long c64 = 6 * waves(tiles(64), nsm), c128 = 7 * waves(tiles(128), nsm),
                  c256 = 12 * waves(tiles(256), nsm),
                  pair = waves((p.tiles + 1) / 2 * (long long)((p.N + 255) / 256), nsm / 2);
  const long long least = c64 < c128 ? (c64 < c256 ? c64 : c256) : (c128 < c256 ? c128 : c256);
  if (12 * pair <= least && p.K >= 2048 && pair * p.K >= 8192)
    return f32 ? launch_pair<true>(p, a, w, stream) : launch_pair<false>(p, a, w, stream);
  if (c256 == least) return launch_dense<256>(p, w, f32, stream);
  if (c128 == least) return launch_dense<128>(p, w, f32, stream);
  return launch_dense<64>(p, w, f32, stream);
}
