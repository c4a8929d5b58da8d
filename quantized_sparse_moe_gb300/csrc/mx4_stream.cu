// A few rows of 16-bit (or 32-bit) activations times MXFP4 weights, on the
// block-scaled tensor cores, with the weights streamed once and never
// expanded.
//
//   y[t, n] = sum_c x[t, c] w[n, c]
//
// The tensor cores multiply e2m1 by e2m1 only, so the activations are
// written as sums of e2m1 matrices.  A block of 32 values of a row becomes
// integers X = round(x 2^(15 - E)), E the exponent of its largest magnitude
// (|X| <= 2^16), and X six digits of base 8 in -4..3:
//   X = sum_i d_i 8^i,   x = sum_i (d_i / 2) 2^(E - 14 + 3 i)
// d_i / 2 is one of 0, +-0.5, +-1, +-1.5, -2: an e2m1 value, and the power of
// two is its block's scale.  A row of x is thus six rows of an MXFP4 matrix,
// the six results are added in fp32, and every product is exact.  The one
// rounding is that to X, at most 2^-16 of the block's largest magnitude: a
// bf16 within 2^-8 of that magnitude is kept whole, and the fp32 h of the MoE
// layer to twice the bits of its bf16 result.  Taken as unsigned after adding
// the bias sum_i 4 8^i, the digits are bit fields.
//
// The weights are the MMA's 128 rows and the digit rows its N, 6 per row of
// x: an MMA of 128 x 8 x 64 takes 39 cycles and one of 128 x 64 x 64 48 (what
// reading the weights from shared memory costs), so the sixfold width is
// almost free up to ten rows, and up to 32 rows the kernel stays bound by HBM
// (24 bytes per SM and cycle).  A dequantising kernel needs at least one
// integer instruction per weight, which is what bounds the affine-4 kernels
// of decode_stream.cu.
//
// Work items are (slot, tile of 128 rows of w); a slot is up to `tok` rows
// of x (of one expert's).  A cluster of `cs` CTAs works on an item together,
// each on its part of K, and exchanges partial sums through distributed
// shared memory: CTA q adds up and writes rows 128 q / cs .. of the tile, in
// CTA order.  Roles in a CTA: warp 0 loads (stages of 256 columns: codes by
// TMA with the 128-byte swizzle, scale tiles by bulk copy), warp 1 issues the
// scale copies and MMAs, warps 4-7 are the epilogue, the other ten make the
// digits of the next slot while the current one is multiplied.
//
// Measured (graph replay): 1 x 512 x 2048 4.4 us, 5 x 2048 x 8192 7.9, 1 x 128256
// x 2048 25.3 (139.7 MB, 5.5 TB/s), 16 rows of the same 35.8: a row of 2048 costs
// a CTA about half a microsecond of integer instructions for its digits.  37
// tokens of the layer below take 37 us in gate_up (204 MB, 5.5 TB/s) and 22 in
// down (103 MB, 4.6 TB/s).
//
// In the MoE layer the slots are formed here, by every CTA for itself, from
// the router's choices (a bit per token and expert: counts and ranks; a prefix
// sum; then the lists of the CTA's own slots), instead of by a launch of its
// own (H 2048, I 512, 256 experts, 8 of them: T = 6: 38.6 -> 36.1 us a layer,
// T = 37: 76.6 -> 74.6, T = 64: 99.0 -> 95.3; T = 4: 28.5 -> 28.9; since then
// T = 3: 24.3, 8: 37.8, 37: 72.5, 64: 93.3).  h and o
// are indexed by the assignment t k + j.
#include <type_traits>

#include "mx4_stream.cuh"

namespace qsm {
namespace mx4 {
namespace {

constexpr int kThreads = 512;
constexpr int kConvWarps = 10;  // of the digits: 24 x 128256 x 2048 44.5 us, 8 47.5
constexpr int kMaxStages = 7;  // of the ring: 1 x 128256 x 2048 25.4 us, 4 25.8, 9 25.8, 12 27.1
// dynamic shared memory; barriers and the table of slots take some of the rest
constexpr int smem_max(int mode) { return (mode == kRows ? 224 : 218) * 1024; }
constexpr int kMaxSplit = 8;          // CTAs per cluster
constexpr int kMaxSegs = 32;          // stages of K per CTA
template <int MODE>
constexpr int mats() { return MODE == kRowsGateUp ? 2 : 1; }  // row tiles of w per item

struct Slot {
  int e;     // expert, -1: shared expert or dense
  int row0;  // first row of x (dense, shared), or the slot's row of `list`
  int cnt;
};

constexpr int kSlotTab = 128;   // slots of a CTA's run of items
constexpr int kMaxTok = 8;      // rows of a routed slot
constexpr int kMaxE = 1024;
constexpr int kMaxChunks = 4;   // of kThreads assignments: 64 tokens, 32 experts each

// What a CTA knows about its run of slots.  In 16 bits, 7 KB: with twice that
// the gate_up product of H = 2048 and 8 rows would not keep three stages of
// its whole K (T = 37: 82 us a layer).
struct SlotTable {
  struct { int16_t e, row0, cnt; } slot[kSlotTab];
  uint16_t list[kSlotTab][kMaxTok];  // a routed slot's assignments
  uint16_t count[kMaxE], start[kMaxE];
  int warp_sum[kThreads / 32];
};

// The chosen experts of this thread's assignments.
__device__ __forceinline__ void load_choices(const StreamParams& p, int (&id)[kMaxChunks]) {
  const int A = p.T * p.k;
#pragma unroll
  for (int c = 0; c < kMaxChunks; ++c) {
    const int a = c * kThreads + threadIdx.x;
    id[c] = a < A ? __ldcg(p.topk_idx + a) : -1;
  }
}
// Of those the valid ones (others become -1), their ranks among the expert's,
// and the experts' counts.  A token has an expert at most once, and there are
// at most 64: a bit per token in the expert's mask (at `mask`, 8 bytes an
// expert, zeros) gives both, the same in every CTA.
__device__ __forceinline__ void assign_ranks(const StreamParams& p, SlotTable& t, uint2* mask,
                                             int (&id)[kMaxChunks], int (&rank)[kMaxChunks]) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int c = 0; c < kMaxChunks; ++c) {
    if (id[c] < 0 || id[c] >= p.E) id[c] = -1;
    rank[c] = (int)p.k_div.div(c * kThreads + tid);  // the token
  }
#pragma unroll
  for (int c = 0; c < kMaxChunks; ++c)
    if (id[c] >= 0)
      atomicOr(rank[c] < 32 ? &mask[id[c]].x : &mask[id[c]].y, 1u << (rank[c] & 31));
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kMaxChunks; ++c) {
    if (id[c] < 0) continue;
    const uint2 m = mask[id[c]];
    const uint32_t below = (1u << (rank[c] & 31)) - 1u;
    rank[c] = rank[c] < 32 ? __popc(m.x & below) : __popc(m.x) + __popc(m.y & below);
  }
  for (int e = tid; e < p.E; e += kThreads) t.count[e] = (uint16_t)(__popc(mask[e].x) + __popc(mask[e].y));
  tc::fence_async_smem();  // the ring's copies come next
}

// The first slot of every expert, and how many slots there are.
__device__ __forceinline__ int slot_starts(const StreamParams& p, SlotTable& t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int done = p.shared_tiles;
  for (int e0 = 0; e0 < p.E; e0 += kThreads) {
    const int e = e0 + tid;
    const int v = e < p.E ? (t.count[e] + p.tok - 1) >> p.tok_log : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) t.warp_sum[warp] = incl;
    __syncthreads();
    int before = done;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int n = t.warp_sum[w];
      if (w < warp) before += n;
      done += n;
    }
    if (e < p.E) t.start[e] = (uint16_t)(before + incl - v);
    __syncthreads();
  }
  return done;
}

// The slots tab0 .. tab0 + n - 1.
__device__ __forceinline__ void fill_slots(const StreamParams& p, SlotTable& t, const int (&id)[kMaxChunks],
                                           const int (&rank)[kMaxChunks], int tab0, int n) {
  const int tid = threadIdx.x;
  if (tid < n && tab0 + tid < p.shared_tiles) {
    const int row0 = (tab0 + tid) * p.tok;
    t.slot[tid] = {-1, (int16_t)row0, (int16_t)min(p.tok, p.T - row0)};
  }
  for (int e = tid; e < p.E; e += kThreads) {
    const int cnt = t.count[e], s0 = t.start[e] - tab0;
    for (int m = 0; m * p.tok < cnt; ++m)
      if (s0 + m >= 0 && s0 + m < n)
        t.slot[s0 + m] = {(int16_t)e, (int16_t)(s0 + m), (int16_t)min(p.tok, cnt - m * p.tok)};
  }
#pragma unroll
  for (int c = 0; c < kMaxChunks; ++c) {
    if (id[c] < 0) continue;
    const int s = t.start[id[c]] + (rank[c] >> p.tok_log) - tab0;
    if (s >= 0 && s < n) t.list[s][rank[c] & (p.tok - 1)] = (uint16_t)(c * kThreads + tid);
  }
}

// Slot s, by all lanes of a warp.
template <int MODE>
__device__ __forceinline__ Slot slot_of(const StreamParams& p, const SlotTable* t, int tab0, int s) {
  Slot r;
  if (MODE == kRows) {
    r = {-1, s * p.tok, min(p.tok, p.T - s * p.tok)};
  } else {
    const auto& w = t->slot[s - tab0];
    r = {w.e, w.row0, w.cnt};
  }
  r.e = uniform(r.e);
  r.row0 = uniform(r.row0);
  r.cnt = uniform(r.cnt);
  return r;
}
// The row of h and o of the slot's row i.
__device__ __forceinline__ int assignment(const StreamParams& p, const SlotTable* t, const Slot& s, int i) {
  return s.e < 0 ? p.T * p.k + s.row0 + i : t->list[s.row0][i];
}

// Eight consecutive values of row i of the slot, from column c (zeros past K).
template <int MODE>
__device__ __forceinline__ void load_acts(const StreamParams& p, const SlotTable* t, const Slot& s, int i, int c,
                                          float (&v)[8]) {
  if (c >= p.K) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    return;
  }
  if (MODE == kRowsDown) {
    const float4* src = reinterpret_cast<const float4*>(p.h + (size_t)assignment(p, t, s, i) * p.I + c);
    const float4 a = __ldcg(src), b = __ldcg(src + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const int row = MODE == kRowsGateUp && s.e >= 0 ? (int)p.k_div.div(t->list[s.row0][i]) : s.row0 + i;
    const uint4 a = __ldcg(reinterpret_cast<const uint4*>(p.x + (size_t)row * p.ldx + c));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(w[j]);
      v[2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) mx4_rows_kernel(const __grid_constant__ StreamParams p) {
  constexpr int NM = mats<MODE>();
  // the dense product starts on a segment's digits as soon as they are there
  // (5 x 2048 x 8192: 9.3 -> 8.4 us); the layer's slots are short, and the
  // code for it costs them more (T = 1: 20.3 -> 20.8 us)
  constexpr bool kBySeg = MODE == kRows;
  constexpr int kStage = NM * (128 * 128 + 2 * kTileBytes);
  extern __shared__ unsigned char smem_raw[];
  // the same offset in every CTA of a cluster, so that a shared-memory
  // address of this CTA maps to the same place of the others
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], dig_full[2][kBySeg ? kMaxSegs : 1],
      dig_empty[2],
      acc_full[2], acc_empty[2], part_full[2], part_empty[2], done;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ typename std::conditional<MODE == kRows, char, SlotTable>::type tab_space;
  SlotTable* tab = MODE == kRows ? nullptr : reinterpret_cast<SlotTable*>(&tab_space);
  volatile int* abort_p = &abort_flag;

  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int cs = p.cs, stages = p.stages;
  // Down: the routing and the weights are older than the previous launch
  // (which let this one start after its own wait), so the slots are formed and
  // the loading warp goes on without waiting; h is the previous launch's.
  int id[kMaxChunks], rank_of[kMaxChunks];
  if (MODE == kRowsDown) load_choices(p, id);
  if (MODE != kRows)
    for (int e = threadIdx.x; e < p.E; e += kThreads) reinterpret_cast<uint2*>(smem)[e] = make_uint2(0u, 0u);
  const int rank = cs > 1 ? (int)cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&dig_empty[b], 1);
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
      mbar_init(&part_full[b], cs < 4 ? 4 : cs);
      mbar_init(&part_empty[b], 4 * cs);
    }
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 3 && lane < (kBySeg ? p.segs : 1)) {
    for (int b = 0; b < 2; ++b) mbar_init(&dig_full[b][lane], kConvWarps);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) tc::prefetch_map(&p.w);
  if (warp == 2) tc::tmem_alloc(&tmem_base, p.tmem_cols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (cs > 1) cluster_sync_all();
  const uint32_t tmem = uniform(tmem_base);

  // this CTA's stages of K
  const int nst = (p.K + kStageK - 1) / kStageK, cts = col_tiles(p.K);
  const int s0 = nst * rank >> p.cs_log, s1 = nst * (rank + 1) >> p.cs_log;
  if (MODE != kRowsDown) {
    pdl_wait();
    pdl_launch_dependents();
  }
  // This cluster's contiguous run of items (slot, tile).
  uint32_t slots = p.slots;
  if (MODE != kRows) {
    if (MODE == kRowsGateUp) load_choices(p, id);
    assign_ranks(p, *tab, reinterpret_cast<uint2*>(smem), id, rank_of);
    slots = slot_starts(p, *tab);
  }
  const uint32_t nclus = gridDim.x >> p.cs_log, clus = blockIdx.x >> p.cs_log;
  const uint32_t items = slots * p.ntiles.d, each = items / nclus, more = items - each * nclus;
  const int first = uniform((int)(clus * each + min(clus, more)));
  const int last = uniform(first + (int)(each + (clus < more ? 1 : 0)));
  const int tab0 = p.ntiles.div(first);
  if (MODE != kRows) {
    if (first < last) fill_slots(p, *tab, id, rank_of, tab0, (int)p.ntiles.div(last - 1) - tab0 + 1);
    __syncthreads();
  }
  if (MODE == kRowsDown && warp != 0) {
    pdl_wait();
    pdl_launch_dependents();
  }

  if (warp == 0) {
    int st = 0, slot = -1;  // ring position
    uint32_t round = 0;     // how often it came round
    Slot sl = {};
    for (int item = first; item < last && !warp_aborted(abort_p); ++item) {
      const int s = p.ntiles.div(item), tile = item - s * p.ntiles.d;
      if (s != slot) sl = slot_of<MODE>(p, tab, tab0, slot = s);
      const bool sh = MODE != kRows && sl.e < 0;
      const CUtensorMap* wm = sh ? &p.w_sh : &p.w;
      const int row0 = (sl.e < 0 ? 0 : sl.e * p.N) + tile * 128;
      const uint8_t* wsf = (sh ? p.w_scales_sh : p.w_scales) + (size_t)(row0 >> 7) * cts * kTileBytes;
      bool ok = true;
      for (int ks = s0; ks < s1; ++ks) {
        if (round > 0 && !warp_wait(&empty[st], (round - 1) & 1, abort_p, p.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          unsigned char* base = smem + st * kStage;
          const uint32_t sfb = (uint32_t)min(2, cts - 2 * ks) * kTileBytes;
          mbar_arrive_expect_tx(&full[st], NM * (128 * 128 + sfb));
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            tc::tma_load_2d(base + m * 128 * 128, wm, ks * 128, row0 + m * (p.N / 2), &full[st]);
            bulk_g2s(base + NM * 128 * 128 + m * 2 * kTileBytes,
                     wsf + ((size_t)m * (p.N >> 8) * cts + 2 * ks) * kTileBytes, sfb, &full[st]);
          }
        }
        __syncwarp();
        if (++st == stages) st = 0, ++round;
      }
      if (!ok) break;
    }
    // after an abort, let the copies in flight land before the CTA exits
    for (int i = 0; i < stages; ++i) {
      const uint32_t r = i < st ? round : round - 1;  // the last round of this position
      if (i < st || round > 0) mbar_wait_bounded(&full[i], r & 1, 1u << 16);
    }
    __syncwarp();
  } else if (warp == 1) {
    int st = 0, slot = -1, db = 0, rows = 0, ndig = 0, ab = 0;
    uint32_t round = 0, acc_round = 0, fs = 0, dig_phase = 0;
    const int sfc = 8 * NM + 8 * p.groups;  // scale columns of one stage
    const uint32_t sf0 = tmem + p.nacc * NM * p.acc_cols;
    const uint32_t base = smem_u32(smem);
    const uint64_t desc0 = tc::sw128_desc(base);
    for (int item = first; item < last && !warp_aborted(abort_p); ++item) {
      const int s = p.ntiles.div(item);
      const bool fresh = s != slot;
      bool ok = true;
      if (fresh) {  // the next slot's digits; the previous one's are free
        if (slot >= 0 && elect_one()) tc::mma_commit(&dig_empty[db]);
        __syncwarp();
        slot = s;
        rows = digit_rows(slot_of<MODE>(p, tab, tab0, s).cnt);
        db = p.nb == 2 ? ndig & 1 : 0;
        dig_phase = (p.nb == 2 ? ndig >> 1 : ndig) & 1;
        ++ndig;
      }
      if (acc_round > 0 && !warp_wait(&acc_empty[ab], (acc_round - 1) & 1, abort_p, p.status)) break;
      const uint32_t acc = tmem + ab * NM * p.acc_cols;
      for (int ks = s0; ks < s1; ++ks) {
        const int seg = ks - s0;
        if ((fresh && (kBySeg || seg == 0) &&
             !warp_wait(&dig_full[db][kBySeg ? seg : 0], dig_phase, abort_p, p.status)) ||
            !warp_wait(&full[st], round & 1, abort_p, p.status)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        if (elect_one()) {
          const uint32_t wsf = base + st * kStage + NM * 128 * 128;
          const uint32_t xsf = base + p.sf_off + (db * p.segs + seg) * 2 * p.groups * kTileBytes;
          const uint64_t wd = desc0 + (uint64_t)(st * (kStage >> 4));
          const uint64_t xd = desc0 + (uint64_t)((p.dig_off + (db * p.segs + seg) * p.seg_bytes) >> 4);
          const uint32_t sfw = sf0 + (fs & 1) * sfc, sfx = sfw + 8 * NM;
          const int kv = min(kStageK, p.K - ks * kStageK);
#pragma unroll
          for (int ct = 0; ct < 2; ++ct) {
            if (ct * kTileCols >= kv) break;
#pragma unroll
            for (int m = 0; m < NM; ++m) copy_scales(sfw + 8 * m + 4 * ct, wsf + (2 * m + ct) * kTileBytes);
            copy_scales(sfx + 4 * ct * p.groups, xsf + ct * p.groups * kTileBytes);
            if (p.groups == 2) copy_scales(sfx + 4 * (2 * ct + 1), xsf + (2 * ct + 1) * kTileBytes);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk * 64 >= kv) break;
#pragma unroll
            for (int m = 0; m < NM; ++m)
              mma_mxf4(acc + m * p.acc_cols, wd + m * (128 * 128 >> 4) + 2 * kk, xd + 2 * kk,
                       idesc_mxf4(rows, kk & 1), sfw + 8 * m + 4 * (kk >> 1),
                       sfx + 4 * p.groups * (kk >> 1), (seg > 0 || kk > 0) ? 1u : 0u);
          }
          tc::mma_commit(&empty[st]);
          if (ks == s1 - 1) tc::mma_commit(&acc_full[ab]);
        }
        __syncwarp();
        ++fs;
        if (++st == stages) st = 0, ++round;
      }
      if (!ok) break;
      if (++ab == p.nacc) ab = 0, ++acc_round;
    }
    // every MMA issued has completed before tensor memory is freed
    if (elect_one()) tc::mma_commit(&done);
    __syncwarp();
    mbar_wait_bounded(&done, 0, kWaitIters);
  } else if (warp < 4 || warp >= 8) {
    // digits: rows 6 i .. 6 i + 5 of the buffer are the planes of row i, in
    // segments of 256 columns with the 128-byte swizzle
    const int ct = (warp < 4 ? warp - 2 : warp - 6) * 32 + lane;
    int ndig = 0, slot = -1;
    bool bad = false;
    for (int item = first; item < last; ++item) {
      const int s = p.ntiles.div(item);
      if (s == slot) continue;
      slot = s;
      const int db = p.nb == 2 ? ndig & 1 : 0;
      if (ndig >= p.nb &&
          !warp_wait(&dig_empty[db], ((p.nb == 2 ? ndig >> 1 : ndig) - 1) & 1, abort_p, p.status))
        break;
      ++ndig;
      const Slot sl = slot_of<MODE>(p, tab, tab0, s);
      // groups of 8 columns, 32 to a row and segment, segment by segment (one
      // is done when every warp has passed it); u / 32 / cnt by a multiplication
      // (exact below 2^11)
      const int total = (s1 - s0) * sl.cnt * 32;
      const uint32_t magic = (65535u + (uint32_t)sl.cnt) / (uint32_t)sl.cnt;
      unsigned char* dig = smem + p.dig_off + db * p.segs * p.seg_bytes;
      unsigned char* sf = smem + p.sf_off + db * p.segs * 2 * p.groups * kTileBytes;
      int told = 0;  // segments that this warp has reported
      auto report = [&](int upto) {
        tc::fence_async_smem();
        __syncwarp();
        if (!kBySeg && lane == 0) tc::mbar_arrive(&dig_full[db][0]);
        for (; kBySeg && told < upto; ++told)
          if (lane == 0) tc::mbar_arrive(&dig_full[db][told]);
      };
      float next[8];
      auto fetch = [&](int u) {
        const int seg = (int)(((uint32_t)u >> 5) * magic >> 16), i = (u >> 5) - seg * sl.cnt;
        load_acts<MODE>(p, tab, sl, i, (s0 + seg) * kStageK + 8 * (u & 31), next);
      };
      if (ct - lane < total) fetch(ct);
      for (int u = ct; u - lane < total; u += 32 * kConvWarps) {  // total is a multiple of 32
        const int seg = (int)(((uint32_t)u >> 5) * magic >> 16), i = (u >> 5) - seg * sl.cnt, c8 = u & 31;
        if (kBySeg && seg > told) report(seg);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = next[j];
        if (u - lane + 32 * kConvWarps < total) fetch(u + 32 * kConvWarps);
        uint32_t plane[kDigits];
        const uint32_t sb = digits_of(v, plane);
        if (sb == 255u) bad = true;
        store_digits(plane, sb, i, c8, dig + seg * p.seg_bytes, sf + seg * 2 * p.groups * kTileBytes, p.groups);
      }
      report(s1 - s0);
    }
    if (bad) set_status(p.status, QSM_DEV_NONFINITE);
  } else {
    const int q4 = warp & 3, row = 32 * q4 + lane, et = threadIdx.x - 128;
    const int R = 128 >> p.cs_log;  // rows of a tile that a CTA of the cluster writes
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    float* part = reinterpret_cast<float*>(smem + p.part_off);
    int slot = -1, j = 0, ab = 0;
    uint32_t acc_round = 0;
    Slot sl = {};
    for (int item = first; item < last; ++item, ++j) {
      const int pb = j & 1;
      const int s = p.ntiles.div(item), tile = item - s * p.ntiles.d;
      if (s != slot) sl = slot_of<MODE>(p, tab, tab0, slot = s);
      if (!warp_wait(&acc_full[ab], acc_round & 1, abort_p, p.status)) break;
      tc::tc_fence_after();
      if (cs > 1 && j >= 2 &&
          !__all_sync(0xffffffffu, wait_cluster(&part_empty[pb], (j / 2 - 1) & 1, abort_p, p.status)))
        break;
      // the value of (row `rr` of the tile, row i of the slot) goes out
      auto put = [&](int i, int rr, float a, float b) {
        const size_t hrow = MODE == kRows ? 0 : (size_t)assignment(p, tab, sl, i);
        const int c = tile * 128 + rr;
        if (MODE == kRowsGateUp) p.h[hrow * p.I + c] = silu(a) * b;
        else if (MODE == kRowsDown) p.o[hrow * p.H + c] = a;
        else if (c < p.N)
          p.y[(size_t)(sl.row0 + i) * p.N + c] = __bfloat16_as_ushort(__float2bfloat16_rn(a));
      };
      const uint32_t acc = tmem + lanes + ab * NM * p.acc_cols;
      const int owner = row >> (7 - p.cs_log);
      const uint32_t dst = cs > 1 ? dsmem_addr(part + ((size_t)(pb * cs + rank) * NM * p.tok) * R + (row & (R - 1)),
                                               owner)
                                  : 0u;
      for (int i0 = 0; i0 < sl.cnt; i0 += 2) {
        float v[NM][16];
#pragma unroll
        for (int m = 0; m < NM; ++m) tc::tmem_ld16(acc + m * p.acc_cols + kDigits * i0, v[m]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (i0 + u >= sl.cnt) break;
          float sum[2];
#pragma unroll
          for (int m = 0; m < NM; ++m) {  // the smallest digits first
            float a = 0.f;
#pragma unroll
            for (int d = 0; d < kDigits; ++d) a += v[m][kDigits * u + d];
            sum[m] = a;
          }
          if (cs == 1) {
            put(i0 + u, row, sum[0], sum[NM - 1]);
          } else {
#pragma unroll
            for (int m = 0; m < NM; ++m)
              dsmem_st_f32(dst + (uint32_t)((i0 + u) * NM + m) * R * 4, sum[m]);
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&acc_empty[ab]);
      if (++ab == p.nacc) ab = 0, ++acc_round;
      if (cs > 1) {
        // tell the CTAs that this warp wrote to; then add up this CTA's rows
        if (lane < (cs == 8 ? 2 : 1))
          arrive_cluster(dsmem_addr(&part_full[pb], cs == 8 ? 2 * q4 + lane : owner));
        if (!__all_sync(0xffffffffu, wait_cluster(&part_full[pb], (j / 2) & 1, abort_p, p.status))) break;
        const float* mine = part + (size_t)pb * cs * NM * p.tok * R;
        for (int u = et; u < sl.cnt * R; u += 128) {
          const int i = u >> (7 - p.cs_log), rr = u & (R - 1);
          float a = 0.f, b = 0.f;
          for (int c = 0; c < cs; ++c) {
            const float* src = mine + ((size_t)c * p.tok + i) * NM * R + rr;
            a += src[0];
            if (NM == 2) b += src[R];
          }
          put(i, rank * R + rr, a, b);
        }
        __syncwarp();
        if (lane < cs) arrive_cluster(dsmem_addr(&part_empty[pb], lane));
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 2) tc::tmem_dealloc(tmem, p.tmem_cols);
  if (cs > 1) cluster_sync_all();  // no CTA leaves while another writes to it
}

template <int MODE>
constexpr int stage_bytes() { return mats<MODE>() * (128 * 128 + 2 * kTileBytes); }

// Shared memory of a geometry with `stages` ring stages; fills the offsets.
int layout(StreamParams* p, int stage, int nm) {
  p->dig_off = p->stages * stage;
  p->seg_bytes = digit_rows(p->tok) * 128;
  p->sf_off = p->dig_off + p->nb * p->segs * p->seg_bytes;
  p->part_off = p->sf_off + p->nb * p->segs * 2 * p->groups * kTileBytes;
  return p->part_off + (p->cs > 1 ? 2 * nm * p->tok * 128 * 4 : 0) + 1024;
}

void* kernel_of(int mode) {
  return mode == kRows         ? reinterpret_cast<void*>(mx4_rows_kernel<kRows>)
         : mode == kRowsGateUp ? reinterpret_cast<void*>(mx4_rows_kernel<kRowsGateUp>)
                               : reinterpret_cast<void*>(mx4_rows_kernel<kRowsDown>);
}

template <int MODE>
qsm_status launch_mode(StreamParams& p, int items, cudaStream_t stream) {
  auto* k = mx4_rows_kernel<MODE>;
  constexpr int NM = mats<MODE>();
  int smem = layout(&p, stage_bytes<MODE>(), NM);
  const int nc = resident_clusters(reinterpret_cast<void*>(k), p.cs, kThreads, smem, smem_max(MODE));
  if (nc < 1) return QSM_ERR_CUDA;
  // With few items a CTA takes only the shared and tensor memory that its
  // own need: the next launch's CTAs then start beside it.
  const int per = (items + nc - 1) / nc;
  if (per == 1) p.nb = p.nacc = 1;
  if (MODE != kRows && per / (int)p.ntiles.d + 2 > kSlotTab) return QSM_ERR_UNSUPPORTED;
  if (per * p.segs < p.stages) p.stages = per * p.segs;
  p.cs_log = p.cs == 8 ? 3 : p.cs / 2;
  smem = layout(&p, stage_bytes<MODE>(), NM);
  const int cols = p.nacc * NM * p.acc_cols + 2 * (8 * NM + 8 * p.groups);
  p.tmem_cols = 32;
  while (p.tmem_cols < cols) p.tmem_cols *= 2;
  const dim3 grid((items < nc ? items : nc) * p.cs);
  if (p.cs > 1)
    QSM_CUDA_TRY(launch_pdl_cluster(k, grid, dim3(kThreads), p.cs, smem, stream, p));
  else
    QSM_CUDA_TRY(launch_pdl(k, grid, dim3(kThreads), smem, stream, p));
  return QSM_OK;
}

}  // namespace

bool plan_rows(StreamParams* p, int mode, int tiles, int tok, int nsm) {
  const int nm = mode == kRowsGateUp ? 2 : 1;
  const int stage = mode == kRowsGateUp ? stage_bytes<kRowsGateUp>() : stage_bytes<kRows>();
  const int nst = (p->K + kStageK - 1) / kStageK;
  p->tok = tok;
  p->nb = mode == kRows ? 1 : 2;
  p->groups = (kDigits * tok + 127) / 128;
  p->acc_cols = (digit_rows(tok) + 31) / 32 * 32;
  p->nacc = 2 * nm * p->acc_cols + 2 * (8 * nm + 8 * p->groups) <= 512 ? 2 : 1;
  auto fit = [&](int cs) {  // the digits, and at least three stages
    p->cs = cs;
    p->segs = (nst + cs - 1) / cs;
    p->stages = 0;
    const int room = (smem_max(mode) - layout(p, stage, nm)) / stage;
    p->stages = room < kMaxStages ? room : kMaxStages;
    return room >= 3 && p->segs <= kMaxSegs;
  };
  // K is split as long as all items still run at once (clusters of 8 do not
  // fill every SM): 1 x 512 x 2048 4.5 us against 5.6 unsplit, 5 x 2048 x 8192
  // 8.4 against 18.2, 32 x 2048 x 2048 11.5 against 18.3 (before the digits
  // became faster); and further until the
  // digits fit
  int cs = 1;
  while (2 * cs <= kMaxSplit && 2 * cs <= nst && tiles * 2 * cs <= nsm && fit(2 * cs) &&
         tiles <= resident_clusters(kernel_of(mode), 2 * cs, kThreads, layout(p, stage, nm), smem_max(mode)))
    cs *= 2;
  for (; cs <= kMaxSplit && cs <= nst; cs *= 2)
    if (fit(cs)) return true;
  return false;
}

qsm_status launch_rows(StreamParams& p, int mode, int items, cudaStream_t stream) {
  switch (mode) {
    case kRows: return launch_mode<kRows>(p, items, stream);
    case kRowsGateUp: return launch_mode<kRowsGateUp>(p, items, stream);
    default: return launch_mode<kRowsDown>(p, items, stream);
  }
}

}  // namespace mx4
}  // namespace qsm

extern "C" qsm_status mx4_gemv(const uint16_t* x, int64_t row_stride, int32_t T, const qsm_mx4* w,
                               uint16_t* y, int32_t* dev_status, cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::mx4;
  if (!w || T < 0 || w->experts != 1 || w->rows < 0) return QSM_ERR_INVALID_ARGUMENT;
  if (T > QSM_MX4_GEMV_MAX_ROWS || w->cols > 65536) return QSM_ERR_UNSUPPORTED;
  if (T == 0 || w->rows == 0) return QSM_OK;
  if (!mx4_valid(w) || !x || !y || !dev_status || !aligned16(x) || !aligned4(dev_status) ||
      reinterpret_cast<uintptr_t>(y) % 2 || row_stride < w->cols || row_stride % 8)
    return QSM_ERR_INVALID_ARGUMENT;
  StreamParams p = {};
  p.N = w->rows;
  p.K = w->cols;
  p.T = T;
  p.k = 1;
  p.x = x;
  p.ldx = (size_t)row_stride;
  p.y = y;
  p.w_scales = w->scales;
  p.status = dev_status;
  const int ntiles = row_tiles(p.N);
  p.ntiles = FastDiv(ntiles);
  int tok = T;  // all rows at once, or as many as fit
  while (tok > 0 && !plan_rows(&p, kRows, ntiles, tok, sm_count())) --tok;
  if (tok == 0) return QSM_ERR_UNSUPPORTED;
  // Where K is split only because the digits of all rows do not fit (every SM
  // has a tile without), halves of the rows that need no split are faster up to
  // K of 4096, below 24 rows of 3584, although the weights are read twice, the second
  // time in part from L2.  N of 19456, 32768, 65536, halves against the split (us):
  //   K 2048, 26 rows 14.0 18.9, 22.9 27.9, 35.5 41.8; 32 rows 15.7 21.7, 25.9 32.0, 39.2 48.8
  //   K 3328, 18 rows 16.7 19.0, 26.9 27.9, 45.0 43.6; 22 rows 18.4 21.8, 30.6 30.9, 49.1 48.1
  //   K 3584, 18 rows 17.5 19.2, 30.2 27.8, 48.7 44.5; 22 rows 19.3 22.0, 34.4 31.2, 53.2 48.8
  //   K 3584, 26 rows 21.4 27.4, 37.7 38.7, 58.4 66.5; K 3840 22.8 27.8, 41.1 39.2, 61.9 68.5
  // and beyond: 16 x 65536 x 4096 52.0 45.9, 8 x 32768 x 8192 46.3 36.3.
  if (p.cs > 1 && ntiles >= sm_count() && p.K < (T < 24 ? 3584 : 4096)) {
    StreamParams half = p;
    if (plan_rows(&half, kRows, ntiles, (T + 1) / 2, sm_count()) && half.cs == 1) p = half;
  }
  p.slots = (T + p.tok - 1) / p.tok;
  if (!make_codes_map(&p.w, w->codes, w->rows, w->cols, 128)) return QSM_ERR_CUDA;
  if ((long long)p.slots * ntiles > (1ll << 30)) return QSM_ERR_UNSUPPORTED;
  return launch_rows(p, kRows, p.slots * ntiles, stream);
}
