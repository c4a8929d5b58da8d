// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = y[t] + c[a] B[a] (A[a] x[t]),     a = ids[t] (none: out[t] = y[t])
//
// in one launch.  A cluster of CTAs has tokens of one adapter after another:
//
//   up to 64 tokens: the distinct adapters of the call are its slots, and a cluster
//     takes the slots s, s + S, ...;
//   more: the tokens of each adapter, wherever they are, make items of up to 64 tokens
//     each, an item a cluster.  Every CTA counts the ids for itself (3 us for 4096), so
//     there is neither a second launch nor a workspace;
//
// and one of NS parts of the columns.  For a slot or an item:
//
//   1. v = A[a] x[t]: every warp of the cluster has a piece of K for all ranks and
//      tokens (16 ranks x 8 tokens x 16 per MMA); the warps' partial sums are added
//      in a fixed order, first in the CTA, then over the cluster through distributed
//      shared memory;
//   2. out = y + (c v) B[a]^T: a warp takes 32 or 64 columns of all the tokens (16 tokens
//      x 8 columns x 16 per MMA) and adds y in fp32.
//
// With NS > 1 each part forms v again for itself (A comes from L2 then), which
// is cheaper than a launch or a grid-wide exchange between the two products.
// Measured (bf16; GPU time of a replayed call, inputs from HBM or L2 as they come):
//   1 token, 2048 x 2048, rank 16: 5.3 us; latency (ids, A, exchange, B and y in turn)
//   37 tokens, 2048 x 8192, up to 64 ranks: 10 us; the same, with 12 MB of A and B
//   64 tokens with adapters of their own, 8192 x 2048, rank 64: 24.4 us = 3.5 TB/s of A and
//     B; the SMs have one or two CTAs each, and plain loads give at most 5.4 TB/s
//   4096 tokens, 2048 x 8192, rank 32: 41 us = 3.7 TB/s: 5 the items and their rows, 10 the first
//     product and its exchange, 23 y and out at the rate of a plain copy; 16384: 128 us = 4.7 TB/s
//   the same with 64 ranks 65 us, 128 109; with fp32 y and out 59 (32 ranks), 92 (64), 154 (128)
// At 128 registers a thread the kernels for up to 32 ranks spill 32 to 68 bytes, those for 65 to 128 ranks 32
// to 276 (the latter's fp32 form); those between do not.
// The products themselves are small: mma.sync with operands in registers does
// not limit any of them (tensor pipe 19% busy in the last case).
//
// Operands go from global memory straight into MMA fragments: the order of the
// products of a sum is free, so a lane takes 8 or 16 consecutive values (16 or 32 bytes) of
// a row where the fragment's own order would have it take four times two.  In
// the same way the columns of the second product's MMAs are dealt so that a lane ends up
// with 8 or 16 consecutive columns of a token.  (A staged in shared memory by copies of
// 512 bytes was slower, 2 TB/s; so were y's lines asked for in L2 ahead, 57 us for 54.)
//
// v is rounded for the second product: c v is split into bf16 parts, two of them
// (2^-17 relative) for 16-bit outputs, which are rounded to 2^-8 anyway, three
// (exact but for fp32's own rounding) for 32-bit ones.
#include "lora_cut.cuh"
#include "mx4_digits.cuh"

namespace qsm {
namespace lora {
namespace {

constexpr int kMaxRank = 128;
constexpr int kMaxSide = 1 << 28;  // of K and N
constexpr int kMostSmem = 200 * 1024;  // dynamic

struct Params {
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  const int32_t* ranks;
  const int32_t* ids;
  const char* y;   // null: zeros
  char* out;
  int64_t ldx, ldy, ldo;  // elements
  int T, K, N, R, n;      // R: ranks that an adapter has room for
  int cs, lanes, parts;   // CTAs of a cluster, slots' lanes S (or clusters for items), column parts NS
  int room;               // items that run at once
  int tile, rows;         // tokens of a tile, and that rounded up to 8: what the buffers hold
  int wide_in, wide_out;  // whether 32 bytes of a and x, and of out, can be one access
  int how;                // kRagged, kUnitsOfY or kDirect
  int copy;               // whether tokens without an adapter have to be copied
  int32_t* status;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The first `n` of eight bf16.
__device__ __forceinline__ uint4 first_of(uint4 v, int n) {
  if (n >= 8) return v;
  const auto keep = [n](uint32_t w, int i) { return n >= i + 2 ? w : n > i ? w & 0xffffu : 0u; };
  return make_uint4(keep(v.x, 0), keep(v.y, 2), keep(v.z, 4), keep(v.w, 6));
}

// Sizes that follow from RK, the blocks of 32 ranks an adapter has room for.
template <int RK>
struct Shape {
  static constexpr int kRanks = 32 * RK;
  static constexpr int kTokTiles = 8 / RK;            // of 8 tokens, at once: 64 accumulators a lane
  static constexpr int kPartRow = kRanks + 4;         // floats: banks 8 apart for a lane's tokens
  static constexpr int kVRow = kRanks + (RK == 1 ? 0 : 32);  // bf16: rows 16 banks apart
};

// A warp's rows of expand_ragged.
constexpr int kStageBytes = 16 * 128;
// A warp's units of y (16 rows of 128 bytes), three of them, and 64 rows of B.
constexpr int kUnitBytes = 16 * 128, kUnits = 3, kWarpBytes = kUnits * kUnitBytes + 64 * 64;

// Bytes of shared memory for tiles of `rows` tokens.
template <int RK>
__host__ __device__ constexpr size_t parts_bytes(int rows) {
  const int at_once = rows < 8 * Shape<RK>::kTokTiles ? rows : 8 * Shape<RK>::kTokTiles;
  return (size_t)kWarps * at_once * Shape<RK>::kPartRow * 4;
}
__host__ __device__ constexpr int v_rows(int rows) { return rows + 16; }  // an MMA may read 15 behind the last
template <int RK, int SPLIT>
__host__ __device__ constexpr size_t v_bytes(int rows) {
  return (size_t)SPLIT * v_rows(rows) * Shape<RK>::kVRow * 2;
}
// How y and out are read and written: rows that are not whole 16-byte units; units of y
// through shared memory (where RK = 1); straight from and to global memory.
enum { kRagged = 0, kUnitsOfY = 1, kDirect = 2 };
// Where v and the CTA's sums lie: v over the partial sums, which have been read by
// then; where there are units of y, those come over the partial sums, and v behind.
template <int RK, int SPLIT>
__host__ __device__ constexpr size_t v_at(int rows, int how) {
  const size_t a = parts_bytes<RK>(rows), b = (size_t)kWarps * kWarpBytes;
  return RK == 1 && how == kUnitsOfY ? (a > b ? a : b) : 0;
}
template <int RK, int SPLIT>
__host__ __device__ constexpr size_t stage_at(int rows, int how) {
  return v_at<RK, SPLIT>(rows, how) + v_bytes<RK, SPLIT>(rows);
}
template <int RK, int SPLIT>
__host__ __device__ constexpr size_t sums_at(int rows, int how) {
  const size_t a = parts_bytes<RK>(rows), b = stage_at<RK, SPLIT>(rows, how) + (how == kRagged ? kWarps * kStageBytes : 0);
  return a > b ? a : b;
}
template <int RK, int SPLIT>
__host__ __device__ constexpr size_t smem_bytes(int rows, int how) {
  return sums_at<RK, SPLIT>(rows, how) + (size_t)rows * Shape<RK>::kRanks * 4;
}

// Eight columns of y or out in one row, as they lie in memory.
template <bool F32>
struct Raw {
  uint4 v[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(const void* src) {
  Raw<F32> r;
  r.v[0] = *reinterpret_cast<const uint4*>(src);
  if (F32) r.v[F32] = reinterpret_cast<const uint4*>(src)[1];
  return r;
}

template <bool F32>
struct Element {
  using type = uint16_t;
};
template <>
struct Element<true> {
  using type = uint32_t;
};

// The accumulators of 16 tokens (8, with H = 1) and 32 columns begin: bf16 with y;
// fp32 with -0, which leaves y as it is where there is no adapter: y comes last, for its full
// accuracy.  y: of tokens g and g + 8.
template <bool F32, int H>
__device__ __forceinline__ void begin_sums(const Raw<F32> (&y)[H], float (&d)[4][4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t pair = h < H && !F32 ? reinterpret_cast<const uint32_t*>(y[h < H ? h : 0].v)[j] : F32 ? 0x80008000u : 0u;
      d[j][2 * h] = bf16_lo(pair);
      d[j][2 * h + 1] = bf16_hi(pair);
    }
}

// Eight columns of out: the MMAs of tiles 0 .. 3 hold two of them each, at d[j][at]
// and d[j][at + 1].
template <bool F32>
__device__ __forceinline__ void store_out(void* dst, const Raw<F32>& y, const float (&d)[4][4], int at) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(y.v);
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (F32) {
      o[2 * j] = __float_as_uint(__uint_as_float(w[2 * j * F32]) + d[j][at]);
      o[2 * j + 1] = __float_as_uint(__uint_as_float(w[(2 * j + 1) * F32]) + d[j][at + 1]);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(d[j][at], d[j][at + 1]);
      o[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
  if (F32) reinterpret_cast<uint4*>(dst)[F32] = make_uint4(o[4], o[5], o[6], o[7]);
}

// 32 columns of B: tile j's column g is row n + 2 j of it (n: the lane's), and the lane
// has 8 ranks of each block of 32.  Rows past the last column repeat it (their sums are not used);
// ranks that do not count are zeros (they may hold anything, and 0 x NaN is not 0).
template <int RK>
__device__ __forceinline__ void load_b(const Params& p, const uint16_t* B, int rank, int n, uint4 (&w)[4][RK]) {
  const int tq = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint16_t* row = B + (size_t)min(n + 2 * j, p.N - 1) * p.R + 8 * tq;
#pragma unroll
    for (int b = 0; b < RK; ++b)
      w[j][b] = 32 * b + 8 * tq < rank ? __ldg(reinterpret_cast<const uint4*>(row + 32 * b)) : make_uint4(0, 0, 0, 0);
  }
  if (rank & 7) {
#pragma unroll
    for (int b = 0; b < RK; ++b)
      if (rank - (32 * b + 8 * tq) < 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j][b] = first_of(w[j][b], max(rank - (32 * b + 8 * tq), 0));
  }
}

// Sixteen bf16 in one access (32-byte aligned).
struct Wide {
  uint4 v[2];
};
__device__ __forceinline__ Wide load_wide(const uint16_t* p) {
  Wide w;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w.v[0].x), "=r"(w.v[0].y), "=r"(w.v[0].z), "=r"(w.v[0].w), "=r"(w.v[1].x), "=r"(w.v[1].y),
                 "=r"(w.v[1].z), "=r"(w.v[1].w)
               : "l"(p));
  return w;
}

// N blocks of 64 columns from k on, 16 of them a lane: whole 128-byte lines of the
// rows.
template <int RK, int N>
__device__ __forceinline__ void shrink_wide(const uint16_t* const (&ap)[2 * RK][2], const uint16_t* xp, int k, int tiles,
                                            float (&acc)[2 * RK][1][4]) {
  Wide xv[N], av[N][2 * RK][2];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    xv[u] = load_wide(xp + k + 64 * u);
#pragma unroll
    for (int i = 0; i < 2 * RK; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (i < tiles) av[u][i][h] = load_wide(ap[i][h] + 8 * (threadIdx.x & 3) + k + 64 * u);
        else av[u][i][h] = {};
  }
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int i = 0; i < 2 * RK; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint4 &lo = av[u][i][0].v[q], &hi = av[u][i][1].v[q], &x = xv[u].v[q];
        mma_bf16(acc[i][0], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        mma_bf16(acc[i][0], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
      }
}

// N blocks of 32 columns from k on; in: whether this lane's columns exist.
template <int RK, int NT, int N>
__device__ __forceinline__ void shrink_blocks(const uint16_t* const (&ap)[2 * RK][2], const uint16_t* const (&xp)[NT], int k,
                                              bool in, int tiles, float (&acc)[2 * RK][NT][4]) {
  uint4 xv[N][NT], av[N][2 * RK][2];
#pragma unroll
  for (int u = 0; u < N; ++u) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      xv[u][j] = in ? __ldg(reinterpret_cast<const uint4*>(xp[j] + k + 32 * u)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * RK; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        av[u][i][h] = in && i < tiles ? __ldg(reinterpret_cast<const uint4*>(ap[i][h] + k + 32 * u)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int i = 0; i < 2 * RK; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 &lo = av[u][i][0], &hi = av[u][i][1];
        mma_bf16(acc[i][j], lo.x, hi.x, lo.y, hi.y, xv[u][j].x, xv[u][j].y);
        mma_bf16(acc[i][j], lo.z, hi.z, lo.w, hi.w, xv[u][j].z, xv[u][j].w);
      }
}

template <int RK, int NT>
__device__ __forceinline__ void put_sums(const float (&acc)[2 * RK][NT][4], int tiles, int m, float* mine) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int i = 0; i < 2 * RK; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (i >= tiles || 8 * j >= m) break;
      float* at = mine + (8 * j + 2 * tq) * Shape<RK>::kPartRow + 16 * i + g;
      at[0] = acc[i][j][0];
      at[Shape<RK>::kPartRow] = acc[i][j][1];
      at[8] = acc[i][j][2];
      at[Shape<RK>::kPartRow + 8] = acc[i][j][3];
    }
}

// v of at most 8 tokens over the CTA's blocks kfirst .. klast - 1 of 32 columns, into
// the warps' partial sums [token][rank].  Sixteen rows of A are under way at once, of
// as many blocks as that makes; the warps take them in turn, so that they read up to a KB
// of each row together.  Rows past the last rank and tokens past the last one
// repeat that one: their sums are not used.
template <int RK>
__device__ __forceinline__ void shrink_few(const Params& p, const uint16_t* A, int rank, const int* mem, int64_t t0, int m,
                                           int kfirst, int klast, float* mine) {
  constexpr int U = 4 / RK;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3, tiles = (rank + 15) / 16;
  float acc[2 * RK][1][4] = {};
  const uint16_t *ap[2 * RK][2], *xp[1];
#pragma unroll
  for (int i = 0; i < 2 * RK; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) ap[i][h] = A + (size_t)min(16 * i + 8 * h + g, rank - 1) * p.K + 8 * tq;
  xp[0] = p.x + (t0 + mem[min(g, m - 1)]) * p.ldx + 8 * tq;
  const int warp = threadIdx.x >> 5, whole = min(klast, p.K / 32);  // the blocks before it have no column past K
  int kb = kfirst;
  if (RK <= 2 && p.wide_in) {
#pragma unroll 1
    for (; kb + U * kWarps <= whole; kb += U * kWarps)  // (8 tq more: 16 columns a lane)
      shrink_wide<RK, U >= 2 ? U / 2 : 1>(ap, xp[0] + 8 * tq, (kb + U * warp) * 32, tiles, acc);
  }
#pragma unroll 1
  for (; kb + U * kWarps <= whole; kb += U * kWarps)
    shrink_blocks<RK, 1, U>(ap, xp, (kb + U * warp) * 32, true, tiles, acc);
#pragma unroll 1
  for (kb += warp; kb < klast; kb += kWarps) shrink_blocks<RK, 1, 1>(ap, xp, kb * 32, kb * 32 + 8 * tq < p.K, tiles, acc);
  put_sums<RK, 1>(acc, tiles, m, mine);
}

// The same for up to 8 NT tokens, N blocks under way at once: with one, as below, each waits for
// memory by itself (1000 tokens 4096 x 4096, rank 32: 18.1 us against 20.0).  Only up to 32 ranks: with
// 64 the registers do not hold it (4096 x 8192 69 us against 65).
template <int RK, int NT, int N>
__device__ __forceinline__ void shrink_some(const Params& p, const uint16_t* A, int rank, const int* mem, int64_t t0, int m,
                                            int kfirst, int klast, float* mine) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3, tiles = (rank + 15) / 16;
  float acc[2 * RK][NT][4] = {};
  const uint16_t *ap[2 * RK][2], *xp[NT];
#pragma unroll
  for (int i = 0; i < 2 * RK; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) ap[i][h] = A + (size_t)min(16 * i + 8 * h + g, rank - 1) * p.K + 8 * tq;
#pragma unroll
  for (int j = 0; j < NT; ++j) xp[j] = p.x + (t0 + mem[min(8 * j + g, m - 1)]) * p.ldx + 8 * tq;
  const int warp = threadIdx.x >> 5, whole = min(klast, p.K / 32);  // the blocks before it have no column past K
  int kb = kfirst;
#pragma unroll 1
  for (; kb + N * kWarps <= whole; kb += N * kWarps) shrink_blocks<RK, NT, N>(ap, xp, (kb + N * warp) * 32, true, tiles, acc);
#pragma unroll 1
  for (kb += warp; kb < klast; kb += kWarps) shrink_blocks<RK, NT, 1>(ap, xp, kb * 32, kb * 32 + 8 * tq < p.K, tiles, acc);
  put_sums<RK, NT>(acc, tiles, m, mine);
}

// The same for up to 8 kTokTiles tokens, block by block.
template <int RK>
__device__ __forceinline__ void shrink_many(const Params& p, const uint16_t* A, int rank, const int* mem, int64_t t0,
                                            int m, int kfirst, int klast, float* mine) {
  constexpr int NT = Shape<RK>::kTokTiles;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3, tiles = (rank + 15) / 16;
  float acc[2 * RK][NT][4] = {};
  int row[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) row[j] = mem[min(8 * j + g, m - 1)];
#pragma unroll 1
  for (int kb = kfirst + (int)(threadIdx.x >> 5); kb < klast; kb += kWarps) {
    const int k = kb * 32 + 8 * tq;
    const bool in = k < p.K;
    uint4 xv[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
      xv[j] = in ? __ldg(reinterpret_cast<const uint4*>(p.x + (t0 + row[j]) * p.ldx + k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * RK; ++i) {
      if (i >= tiles) break;
      uint4 a[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        a[h] = in ? __ldg(reinterpret_cast<const uint4*>(A + (size_t)min(16 * i + 8 * h + g, rank - 1) * p.K + k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_bf16(acc[i][j], a[0].x, a[1].x, a[0].y, a[1].y, xv[j].x, xv[j].y);
        mma_bf16(acc[i][j], a[0].z, a[1].z, a[0].w, a[1].w, xv[j].z, xv[j].w);
      }
    }
  }
  put_sums<RK, NT>(acc, tiles, m, mine);
}

// d (+)= v B^T for 16 tokens (8 with H = 1) and the 32 columns whose rows of B are in w.
template <int RK, int SPLIT, int H>
__device__ __forceinline__ void product(const __nv_bfloat16* v, int part, int rank, const uint4 (&w)[4][RK],
                                        float (&d)[4][4]) {
#pragma unroll
  for (int b = 0; b < RK; ++b) {
    if (32 * b >= rank) break;
#pragma unroll
    for (int s = SPLIT - 1; s >= 0; --s) {  // the small parts first
      const uint4 lo = *reinterpret_cast<const uint4*>(v + s * part + 32 * b);
      uint4 hi = make_uint4(0, 0, 0, 0);
      if (H == 2) hi = *reinterpret_cast<const uint4*>(v + s * part + 32 * b + 8 * Shape<RK>::kVRow);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_bf16(d[j], lo.x, hi.x, lo.y, hi.y, w[j][b].x, w[j][b].y);
        mma_bf16(d[j], lo.z, hi.z, lo.w, hi.w, w[j][b].z, w[j][b].w);
      }
    }
  }
}

// This warp's columns of the slot's tokens, 16 at a time (8, with H = 1, where there are no
// more).  Lanes g, tq: columns 8 tq .. 8 tq + 7 of a chunk of 32, of tokens g and g + 8; U
// times 16 tokens' y are under way at once.  y and out have those columns as whole 16-byte units.
template <int RK, bool F32, int H, int U>
__device__ __forceinline__ void expand(const Params& p, const uint16_t* B, int rank, const int64_t* yrow,
                                       const int64_t* orow, int m, const __nv_bfloat16* vbuf, int vrows, int chunk0,
                                       int chunks, int stride) {
  using S = Shape<RK>;
  constexpr int kEl = F32 ? 4 : 2;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const __nv_bfloat16* v = vbuf + (size_t)g * S::kVRow + 8 * tq;
  const int part = vrows * S::kVRow;
#pragma unroll 1
  for (int ch = chunk0; ch < chunks; ch += stride) {
    const int n = ch * 32 + 8 * tq;
    uint4 w[4][RK];
    load_b<RK>(p, B, rank, ch * 32 + 8 * (g >> 1) + (g & 1), w);
#pragma unroll 1
    for (int m0 = 0; m0 < m; m0 += 16 * U) {
      Raw<F32> y[U][H];
      bool in[U][H];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int row = m0 + 16 * u + 8 * h + g;
          in[u][h] = row < m && n < p.N;
          y[u][h] = {};
          if (p.y && in[u][h]) y[u][h] = load_raw<F32>(p.y + (yrow[row] + n) * kEl);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (m0 + 16 * u >= m) break;
        float d[4][4];
        begin_sums<F32, H>(y[u], d);
        product<RK, F32 ? 3 : 2, H>(v + (m0 + 16 * u) * S::kVRow, part, rank, w, d);
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (in[u][h]) store_out<F32>(p.out + (orow[m0 + 16 * u + 8 * h + g] + n) * kEl, y[u][h], d, 2 * h);
      }
    }
  }
}

// The same for rows that begin anywhere, or end inside a unit of 16 bytes: the warp reads
// and writes its columns of a row side by side, an element a lane, and turns them into
// fragments in 16 rows of its own shared memory; the next rows are on their way meanwhile.
// (4096 x 8191 bf16, rank 32: 86 us; with an element at a
// time straight into the fragments' lanes 179.  Two elements a lane: 95, for want of registers.)
template <int RK, bool F32, int H>
__device__ __forceinline__ void expand_ragged(const Params& p, const uint16_t* B, int rank, const int64_t* yrow,
                                              const int64_t* orow, int m, const __nv_bfloat16* vbuf, int vrows, int chunk0,
                                              int chunks, int stride, unsigned char* stage) {
  using S = Shape<RK>;
  using El = typename Element<F32>::type;
  constexpr int kRow = 32 * sizeof(El);
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const __nv_bfloat16* v = vbuf + (size_t)g * S::kVRow + 8 * tq;
  const int part = vrows * S::kVRow;
  const El* y = reinterpret_cast<const El*>(p.y) + lane;
  El* out = reinterpret_cast<El*>(p.out) + lane;
  El* mine = reinterpret_cast<El*>(stage) + lane;
  unsigned char* frag = stage + g * kRow + 8 * tq * sizeof(El);
  El next[8 * H];
  const auto load = [&](int ch, int m0) {
    const bool in = p.y && ch * 32 + lane < p.N;
#pragma unroll
    for (int r = 0; r < 8 * H; ++r) next[r] = in && m0 + r < m ? y[yrow[m0 + r] + ch * 32] : El(0);
  };
  if (chunk0 < chunks) load(chunk0, 0);
#pragma unroll 1
  for (int ch = chunk0; ch < chunks; ch += stride) {
    const bool in = ch * 32 + lane < p.N;
    uint4 w[4][RK];
    load_b<RK>(p, B, rank, ch * 32 + 8 * (g >> 1) + (g & 1), w);
#pragma unroll 1
    for (int m0 = 0; m0 < m; m0 += 8 * H) {
#pragma unroll
      for (int r = 0; r < 8 * H; ++r) mine[32 * r] = next[r];
      __syncwarp();
      if (m0 + 8 * H < m) load(ch, m0 + 8 * H);
      else if (ch + stride < chunks) load(ch + stride, 0);
      Raw<F32> u[H];
#pragma unroll
      for (int h = 0; h < H; ++h) u[h] = load_raw<F32>(frag + 8 * h * kRow);
      float d[4][4];
      begin_sums<F32, H>(u, d);
      product<RK, F32 ? 3 : 2, H>(v + m0 * S::kVRow, part, rank, w, d);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < H; ++h) store_out<F32>(frag + 8 * h * kRow, u[h], d, 2 * h);
      __syncwarp();
#pragma unroll
      for (int r = 0; r < 8 * H; ++r)
        if (in && m0 + r < m) out[orow[m0 + r] + ch * 32] = mine[32 * r];
      __syncwarp();
    }
  }
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last n groups of this thread's copies have landed.
template <int n>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// The same for adapters of at most 32 ranks and more than 8 tokens.  A warp works on
// units of 16 tokens and 128 bytes of their rows (64 columns, 32 of fp32), whole
// lines; two units' y and the next columns' rows of B are on their way into the warp's own
// shared memory while one is worked on.  (With y straight into registers the loads waited for
// the MMAs and stores before them: 4096 x 8192 bf16 33 us without an adapter, a plain copy 21.)
template <bool F32>
__device__ __forceinline__ void expand_units(const Params& p, const uint16_t* B, int rank, const int64_t* yrow,
                                             const int64_t* orow, int m, const __nv_bfloat16* vbuf, int vrows, int chunk0,
                                             int stride, unsigned char* mine) {
  using S = Shape<1>;
  constexpr int kEl = F32 ? 4 : 2, kCols = 128 / kEl, Q = kCols / 32, SPLIT = F32 ? 3 : 2;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int first = chunk0 * kCols, step = stride * kCols;
  unsigned char* bbuf = mine + kUnits * kUnitBytes;
  // 16 bytes c of row r of a unit lie at unit c ^ (r & 7) of the row: eight lanes' reads are in different banks
  int ahead_m = 0, ahead_n = first, ahead_at = 0;  // the unit that is fetched next, and where to
  const auto fetch = [&] {
    if (ahead_n < p.N && p.y) {
      const int n = ahead_n + (lane & 7) * (16 / kEl);
      unsigned char* to = mine + ahead_at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 3) + 4 * i;
        if (ahead_m + r < m && n < p.N) copy16(to + r * 128 + (((lane & 7) ^ (r & 7)) << 4), p.y + (yrow[ahead_m + r] + n) * kEl);
      }
    }
    copies_commit();
    ahead_m += 16;
    if (ahead_m >= m) ahead_m = 0, ahead_n += step;
    ahead_at = ahead_at == (kUnits - 1) * kUnitBytes ? 0 : ahead_at + kUnitBytes;
  };
  const auto fetch_b = [&](int n0) {  // rows of B as they are, R ranks each
    if (rank > 0 && n0 < p.N)
      for (int i = lane; i < min(kCols, p.N - n0) * p.R / 8; i += 32) copy16(bbuf + i * 16, B + (size_t)n0 * p.R + i * 8);
  };
  fetch_b(first);
  fetch();
  fetch();
  uint4 w[Q][4];
  int at = 0;
#pragma unroll 1
  for (int n0 = first, mt = 0; n0 < p.N;) {
    if (m <= 16) copies_wait<0>();  // (the rows of B came with the last unit)
    else copies_wait<1>();
    __syncwarp();
    if (mt == 0) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // the lane's columns of a unit are 8 Q tq .. 8 Q tq + 8 Q - 1; past the last column it repeats
          const int n = min(8 * Q * (g >> 1) + 8 * q + 2 * j + (g & 1), p.N - 1 - n0);
          w[q][j] = make_uint4(0, 0, 0, 0);
          if (8 * tq < rank) w[q][j] = first_of(*reinterpret_cast<const uint4*>(bbuf + (n * p.R + 8 * tq) * 2), rank - 8 * tq);
        }
      __syncwarp();
      fetch_b(n0 + step);
    }
    const unsigned char* from = mine + at;
    at = at == (kUnits - 1) * kUnitBytes ? 0 : at + kUnitBytes;
    Raw<true> y[2];  // 32 bytes
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        y[h].v[i] = p.y ? *reinterpret_cast<const uint4*>(from + (8 * h + g) * 128 + (((2 * tq + i) ^ g) << 4)) : make_uint4(0, 0, 0, 0);
    __syncwarp();
    fetch();  // over the unit before this one
    const __nv_bfloat16* vr = vbuf + (size_t)(mt + g) * S::kVRow + 8 * tq;
    uint4 v[SPLIT][2];
#pragma unroll
    for (int s = 0; s < SPLIT; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) v[s][h] = *reinterpret_cast<const uint4*>(vr + (size_t)(s * vrows + 8 * h) * S::kVRow);
    Raw<true> o[2];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float d[4][4];
      // bf16: the sum begins with y; fp32: y comes last (see expand)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t pair = F32 ? 0x80008000u : reinterpret_cast<const uint32_t*>(y[h].v)[4 * q + j];
          d[j][2 * h] = bf16_lo(pair);
          d[j][2 * h + 1] = bf16_hi(pair);
        }
      if (rank > 0) {
#pragma unroll
        for (int s = SPLIT - 1; s >= 0; --s)  // the small parts first
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_bf16(d[j], v[s][0].x, v[s][1].x, v[s][0].y, v[s][1].y, w[q][j].x, w[q][j].y);
            mma_bf16(d[j], v[s][0].z, v[s][1].z, v[s][0].w, v[s][1].w, w[q][j].z, w[q][j].w);
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t* out = reinterpret_cast<uint32_t*>(o[h].v);
          if (F32) {
            const uint32_t* in = reinterpret_cast<const uint32_t*>(y[h].v);
            out[2 * j] = __float_as_uint(__uint_as_float(in[2 * j]) + d[j][2 * h]);
            out[2 * j + 1] = __float_as_uint(__uint_as_float(in[2 * j + 1]) + d[j][2 * h + 1]);
          } else {
            const __nv_bfloat162 two = __floats2bfloat162_rn(d[j][2 * h], d[j][2 * h + 1]);
            out[4 * q + j] = *reinterpret_cast<const uint32_t*>(&two);
          }
        }
    }
    const int n = n0 + 8 * Q * tq;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = mt + 8 * h + g;
      if (row >= m) continue;
      char* to = p.out + (orow[row] + n) * kEl;
      if (p.wide_out && n + 8 * Q <= p.N) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(o[h].v[0].x), "r"(o[h].v[0].y),
                     "r"(o[h].v[0].z), "r"(o[h].v[0].w), "r"(o[h].v[1].x), "r"(o[h].v[1].y), "r"(o[h].v[1].z), "r"(o[h].v[1].w)
                     : "memory");
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (n + i * (16 / kEl) < p.N) reinterpret_cast<uint4*>(to)[i] = o[h].v[i];
      }
    }
    mt += 16;
    if (mt >= m) mt = 0, n0 += step;
  }
  copies_wait<0>();
  __syncwarp();
}

// Item `item` of many tokens, the same cut in every CTA: the tokens of an adapter, wherever
// they are (those without one come last), are shared out evenly over as few items as the tile
// allows, in their order; the tile is the smallest that makes no more items than
// run at once.  Its tokens go to mem, m of them (0: there is no such item).  Returns the adapter,
// -1: none.  cnt: n + 1 counters; all: room for the ids.  (The code is gone through once, so that its
// size counts, too: with 16 ids of a lane in registers it took 6.5 us for 4096 tokens, so 5.)
__device__ __forceinline__ int find_item(const Params& p, int item, int* cnt, int* all, int* mem, int* sums, int& m) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll 1
  for (int t = tid; t < p.T; t += kThreads)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(all + t)), "l"(p.ids + t) : "memory");
  copies_commit();
#pragma unroll 1
  for (int i = tid; i <= p.n; i += kThreads) cnt[i] = 0;
  copies_wait<0>();
  __syncthreads();
  const int per = (p.T + 32 * kWarps - 1) / (32 * kWarps) * 32, t0 = warp * per, t1 = min(t0 + per, p.T);  // this warp's
  bool bad = false;
#pragma unroll 4
  for (int t = t0 + lane; t < t1; t += 32) {
    const int id = all[t], of = (int)min((uint32_t)id, (uint32_t)p.n);
    bad |= id >= p.n;
    all[t] = of;
    atomicAdd(cnt + of, 1);
  }
  if (bad && blockIdx.x == 0) set_status(p.status, QSM_DEV_BAD_ADAPTER_ID);
  __syncthreads();
  const int ids = p.n + p.copy;  // whose tokens have to be looked at
  int tile = min(max(((p.T + p.room - 1) / p.room + 7) / 8 * 8, 16), kTile);  // less makes too many
#pragma unroll 1
  for (; tile < kTile; tile += 8) {
    int count = 0, used = 0;
#pragma unroll 1
    for (int i = lane; i < ids; i += 32) {
      count += (cnt[i] + tile - 1) / tile;
      used += cnt[i] > 0;
    }
    if (__reduce_add_sync(0xffffffffu, count) <= p.room) break;
    if (__reduce_add_sync(0xffffffffu, used) > p.room) {  // no tile does
      tile = kTile;
      break;
    }
  }
  int id = 0, from = 0, before = 0;
  m = 0;
  for (int i0 = 0; i0 < ids; i0 += 32) {  // the adapter whose items have it among them
    const int c = i0 + lane < ids ? cnt[i0 + lane] : 0, parts = (c + tile - 1) / tile;
    int upto = parts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    upto += before;
    const uint32_t in = __ballot_sync(0xffffffffu, upto > item);
    if (in) {
      const int at = __ffs(in) - 1, nth = item - (upto - parts);
      id = i0 + at;
      from = __shfl_sync(0xffffffffu, parts ? c * nth / parts : 0, at);
      m = __shfl_sync(0xffffffffu, parts ? c * (nth + 1) / parts : 0, at) - from;
      break;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  if (m == 0) return -1;
  int mine = 0;
#pragma unroll 4
  for (int t = t0 + lane; t < t1; t += 32) mine += all[t] == id;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  int rank = -from;
  for (int w = 0; w < warp; ++w) rank += sums[w];
  if (mine && rank < m && rank + mine > 0)
#pragma unroll 1
    for (int t = t0; t < t1 && rank < m; t += 32) {
      const bool is = t + lane < t1 && all[t + lane] == id;
      const uint32_t who = __ballot_sync(0xffffffffu, is);
      const int at = rank + __popc(who & ((1u << lane) - 1));
      if (is && at >= 0 && at < m) mem[at] = t + lane;
      rank += __popc(who);
    }
  __syncthreads();
  return id < p.n ? id : -1;
}

// GROUPED: a cluster has one item; otherwise it has slots of a tile.
template <int RK, bool F32, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 2)
lora_kernel(const __grid_constant__ Params p) {
  using S = Shape<RK>;
  constexpr int SPLIT = F32 ? 3 : 2;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) int ids[kTile];
  __shared__ unsigned long long slot_tokens[kTile];
  __shared__ int slot_id[kTile], mem[kTile], ranks[kTile], leaders[2], sums[kWarps];
  __shared__ float factor[kTile];
  __shared__ int64_t yrow[kTile], orow[kTile];  // where the slot's tokens have their rows, in elements
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank_cta = p.cs > 1 ? (int)mx4::cluster_rank() : 0;
  int cl = blockIdx.x / p.cs;  // cluster: (tile, slot lane or item, column part), the part fastest
  const int part = cl % p.parts;
  cl /= p.parts;
  const int slot0 = GROUPED ? 0 : cl % p.lanes, lanes = GROUPED ? 1 : p.lanes;
  const int64_t t0 = GROUPED ? 0 : (int64_t)(cl / p.lanes) * p.tile;
  pdl_wait();
  pdl_launch_dependents();

  int slots = 1, total = 0;
  if constexpr (GROUPED) {
    int* cnt = reinterpret_cast<int*>(smem + smem_bytes<RK, SPLIT>(p.rows, p.how));
    const int id = find_item(p, cl, cnt, reinterpret_cast<int*>(smem), mem, sums, total);
    if (total == 0) return;  // the whole cluster
    if (tid < total) {
      yrow[tid] = mem[tid] * p.ldy;
      orow[tid] = mem[tid] * p.ldo;
      ranks[tid] = id < 0 ? 0 : p.ranks ? min(max(__ldg(p.ranks + id), 0), p.R) : p.R;
      factor[tid] = id >= 0 && p.scale ? __ldg(p.scale + id) : 1.f;
    }
    if (tid == 0) slot_id[0] = id;
  } else {
    const int count = (int)min((int64_t)p.tile, p.T - t0);
    // ids of the tile; -1: none
    if (tid < kTile) {
      int id = tid < count ? __ldg(p.ids + t0 + tid) : -2;
      if (tid < count && id < 0) id = -1;
      if (id >= p.n) {
        id = -1;
        if (rank_cta == 0 && slot0 == 0 && part == 0) set_status(p.status, QSM_DEV_BAD_ADAPTER_ID);
      }
      ids[tid] = id;
    }
    __syncthreads();
    // slots in the order of their first tokens
    if (tid < kTile) {
      const int id = ids[tid];
      unsigned long long same = 0;
#pragma unroll
      for (int j = 0; j < kTile; j += 4) {
        const int4 o = *reinterpret_cast<const int4*>(ids + j);
        same |= (unsigned long long)((o.x == id) | (o.y == id) << 1 | (o.z == id) << 2 | (o.w == id) << 3) << j;
      }
      const bool leader = id != -2 && (same & ((1ull << tid) - 1)) == 0 && (id != -1 || p.copy);
      const uint32_t all = __ballot_sync(0xffffffffu, leader);
      if (lane == 0) leaders[warp] = (int)all;
      asm volatile("bar.sync 1, 64;" ::: "memory");
      if (leader) {
        const int at = __popc(all & ((1u << lane) - 1)) + (warp ? __popc((uint32_t)leaders[0]) : 0);
        slot_id[at] = id;
        slot_tokens[at] = same;
      }
    }
    __syncthreads();
    slots = __popc((uint32_t)leaders[0]) + __popc((uint32_t)leaders[1]);
    if (slot0 >= slots) return;  // the whole cluster

    // The tokens of this cluster's slots, slot by slot.
    for (int slot = slot0; slot < slots; slot += lanes) {
      const unsigned long long tokens = slot_tokens[slot];
      if (tid < kTile && ((tokens >> tid) & 1ull)) {
        const int at = total + __popcll(tokens & ((1ull << tid) - 1)), id = ids[tid];
        mem[at] = tid;
        yrow[at] = (t0 + tid) * p.ldy;
        orow[at] = (t0 + tid) * p.ldo;
        ranks[at] = id < 0 ? 0 : p.ranks ? min(max(__ldg(p.ranks + id), 0), p.R) : p.R;
        factor[at] = id >= 0 && p.scale ? __ldg(p.scale + id) : 1.f;
      }
      total += __popcll(tokens);
    }
  }
  __syncthreads();

  float* parts = reinterpret_cast<float*>(smem);
  __nv_bfloat16* vbuf = reinterpret_cast<__nv_bfloat16*>(smem + v_at<RK, SPLIT>(p.rows, p.how));
  float* psum = reinterpret_cast<float*>(smem + sums_at<RK, SPLIT>(p.rows, p.how));  // [token][rank], read by the cluster
  const int at_once = min(p.rows, 8 * S::kTokTiles), vrows = v_rows(p.rows);
  float* mine = parts + (size_t)warp * at_once * S::kPartRow;

  const int kblocks = (p.K + 31) / 32;  // this CTA's blocks of K
  const int kfirst = (int)((long long)kblocks * rank_cta / p.cs), klast = (int)((long long)kblocks * (rank_cta + 1) / p.cs);
  const int stride = p.parts * p.cs * kWarps, chunk0 = (part * p.cs + rank_cta) * kWarps + warp;  // of columns

  // v of all of them
  for (int slot = slot0, at = 0; slot < slots; slot += lanes) {
    const int id = slot_id[slot], m = GROUPED ? total : __popcll(slot_tokens[slot]), rank = ranks[at];
    if (rank > 0) {
      const uint16_t* A = p.a + (size_t)id * p.R * p.K;
      const uint16_t* B = p.b + (size_t)id * p.N * p.R;
      // what the second product will read is on its way to L2 meanwhile
      if (m <= 8)
        for (int n = chunk0 * 32; n < p.N && n < (chunk0 + 4 * stride) * 32; n += stride * 32) {
          if (lane == 0) bulk_prefetch_l2(B + (size_t)n * p.R, (uint32_t)min(32, p.N - n) * p.R * 2);
          if (p.y && lane < m) prefetch_l2(p.y + (yrow[at + lane] + n) * (F32 ? 4 : 2));
        }
      const int used = (rank + 15) / 16 * 16;
      for (int c0 = 0; c0 < m; c0 += 8 * S::kTokTiles) {  // tokens at once
        const int mt = min(m - c0, 8 * S::kTokTiles);
        if (mt <= 8) shrink_few<RK>(p, A, rank, mem + at + c0, t0, mt, kfirst, klast, mine);
        else if (RK == 1 && mt <= 16) shrink_some<RK, 2, 4>(p, A, rank, mem + at + c0, t0, mt, kfirst, klast, mine);
        else if (RK == 1 && mt <= 32) shrink_some<RK, 4, 2>(p, A, rank, mem + at + c0, t0, mt, kfirst, klast, mine);
        else shrink_many<RK>(p, A, rank, mem + at + c0, t0, mt, kfirst, klast, mine);
        __syncthreads();
        for (int e = tid; e < mt * (used / 4); e += kThreads) {  // four ranks of a token
          const int tok = e / (used / 4), r = (e - tok * (used / 4)) * 4;
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(parts + ((size_t)w * at_once + tok) * S::kPartRow + r);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
          }
          *reinterpret_cast<float4*>(psum + (at + c0 + tok) * S::kRanks + r) = s;
        }
        __syncthreads();
      }
    }
    at += m;
  }
  if (p.cs > 1) cluster_sync_all();  // every CTA's sums are there
  // c v in bf16 parts, zeros behind the ranks
  for (int e = tid; e < total * (S::kRanks / 4); e += kThreads) {
    const int tok = e / (S::kRanks / 4), r = (e - tok * (S::kRanks / 4)) * 4, rank = ranks[tok];
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < rank) {
      const uint32_t at = smem_u32(psum + tok * S::kRanks + r);
      if (p.cs > 1) {
        float4 u[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < p.cs) u[q] = dsmem_ld_f4(dsmem_addr_u32(at, q));
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < p.cs) v[0] += u[q].x, v[1] += u[q].y, v[2] += u[q].z, v[3] += u[q].w;
      } else {
        const float4 u = *reinterpret_cast<const float4*>(psum + tok * S::kRanks + r);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
      }
    }
    uint32_t w[SPLIT][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float rest = r + i < rank ? v[i] * factor[tok] : 0.f;
#pragma unroll
      for (int s = 0; s < SPLIT; ++s) {
        const __nv_bfloat16 h = __float2bfloat16_rn(rest);
        const uint32_t bits = __bfloat16_as_ushort(h);
        if (i & 1) w[s][i / 2] |= bits << 16;
        else w[s][i / 2] = bits;
        // an infinity stays one: its rest would be infinity - infinity
        rest = isfinite(__bfloat162float(h)) ? rest - __bfloat162float(h) : 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < SPLIT; ++s)
      *reinterpret_cast<uint2*>(vbuf + ((size_t)s * vrows + tok) * S::kVRow + r) = make_uint2(w[s][0], w[s][1]);
  }
  __syncthreads();
  if (p.cs > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // has read the others' sums

  // out of all of them (an MMA reads the rows of up to 15 tokens behind a slot's last one: their sums are not used)
  for (int slot = slot0, at = 0; slot < slots; slot += lanes) {
    const int id = slot_id[slot], m = GROUPED ? total : __popcll(slot_tokens[slot]), rank = ranks[at];
    const uint16_t* B = p.b + (size_t)(id < 0 ? 0 : id) * p.N * p.R;
    const __nv_bfloat16* v = vbuf + (size_t)at * S::kVRow;
    const int64_t *yr = yrow + at, *og = orow + at;
    const int chunks = (p.N + 31) / 32;
    if (p.how == kRagged) {
      unsigned char* stage = smem + stage_at<RK, SPLIT>(p.rows, kRagged) + warp * kStageBytes;
      if (m <= 8) expand_ragged<RK, F32, 1>(p, B, rank, yr, og, m, v, vrows, chunk0, chunks, stride, stage);
      else expand_ragged<RK, F32, 2>(p, B, rank, yr, og, m, v, vrows, chunk0, chunks, stride, stage);
    } else if (m <= 8) {
      expand<RK, F32, 1, 1>(p, B, rank, yr, og, m, v, vrows, chunk0, chunks, stride);
    } else {
      if constexpr (RK == 1) expand_units<F32>(p, B, rank, yr, og, m, v, vrows, chunk0, stride, smem + warp * kWarpBytes);
      else expand<RK, F32, 2, F32 || RK == 4 ? 2 : 4>(p, B, rank, yr, og, m, v, vrows, chunk0, chunks, stride);
    }
    at += m;
  }
  // no CTA leaves while another may still read its sums
  if (p.cs > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int RK, bool GROUPED>
qsm_status launch(Params& p, bool f32, cudaStream_t stream) {
  static_assert(parts_bytes<RK>(kTile) >= kMostGrouped * 4, "find_item has the ids there");
  auto* kernel = f32 ? lora_kernel<RK, true, GROUPED> : lora_kernel<RK, false, GROUPED>;
  if (p.how != kRagged) p.how = RK == 1 && p.T > 8 ? kUnitsOfY : kDirect;
  p.tile = p.T < kTile ? p.T : kTile;
  p.rows = (p.tile + 7) / 8 * 8;
  const int smem = (int)(f32 ? smem_bytes<RK, 3>(p.rows, p.how) : smem_bytes<RK, 2>(p.rows, p.how)) + (GROUPED ? (p.n + 1) * 4 : 0);
  void* asked = reinterpret_cast<void*>(kernel);
  // Registers allow two CTAs an SM, shared memory only one to fp32 with more than 64 ranks where rows are not whole
  // 16-byte units, or beside 820 adapters' counters (4096 tokens, 2048 x 2050, rank 128, 100 adapters: 265 us, cut for two 299).
  int each = mx4::resident_ctas(asked, kThreads, smem, kMostSmem);
  if (each > 2) each = 2;
  const Cut c = cut(GROUPED, p.T, p.n, p.N, (long long)each * mx4::sm_count(),
                    [&](int cs) { return mx4::resident_clusters(asked, cs, kThreads, smem, kMostSmem); });
  if (c.ctas < 1) return QSM_ERR_CUDA;
  p.cs = c.cs;
  p.lanes = c.lanes;
  p.parts = c.parts;
  p.room = c.room;
  if (c.ctas > 0x7fffffffll) return QSM_ERR_UNSUPPORTED;
  QSM_CUDA_TRY(launch_pdl_cluster(kernel, dim3((unsigned)c.ctas), dim3(kThreads), p.cs, (size_t)smem, stream, p));
  return QSM_OK;
}

}  // namespace
}  // namespace lora
}  // namespace qsm

extern "C" qsm_status lora_add(const qsm_lora* L, const uint16_t* x, int64_t ldx, int32_t T,
                               const int32_t* ids, int32_t dtype, const void* y, int64_t ldy, void* out,
                               int64_t ldo, int32_t* dev_status, cudaStream_t stream) {
  using namespace qsm;
  using namespace qsm::lora;
  if (!L || T < 0 || L->n < 1 || L->K < 8 || L->K % 8 || L->N < 1 || L->rank < 8 || L->rank % 8 ||
      (dtype != QSM_BF16 && dtype != QSM_FP32))
    return QSM_ERR_INVALID_ARGUMENT;
  if (L->rank > kMaxRank || L->K > kMaxSide || L->N > kMaxSide) return QSM_ERR_UNSUPPORTED;
  if (T == 0) return QSM_OK;
  if (T == 1) {
    ldx = L->K;
    ldy = ldo = (L->N + 7ll) / 8 * 8;
  }
  const size_t el = dtype == QSM_FP32 ? 4 : 2;
  const auto on = [](const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
  if (!x || !ids || !out || !dev_status || !L->a || !L->b || !aligned16(x) || !aligned16(L->a) || !aligned16(L->b) ||
      !aligned4(ids) || !aligned4(dev_status) || (L->scale && !aligned4(L->scale)) ||
      (L->ranks && !aligned4(L->ranks)) || !on(out, el) || (y && !on(y, el)) || ldx < L->K || ldx % 8 ||
      (y && ldy < L->N) || ldo < L->N)
    return QSM_ERR_INVALID_ARGUMENT;
  using mx4::Rows;
  const size_t t = T, N = L->N;
  const Rows rx = {x, t, (size_t)ldx * 2, (size_t)L->K * 2}, ry = {y, t, (size_t)ldy * el, N * el};
  const Rows ro = {out, t, (size_t)ldo * el, N * el};
  const auto meets = [&](const void* p, size_t bytes) { return mx4::overlap(ro, Rows{p, 1, 0, bytes}); };
  const bool same = y == out && ldy == ldo;
  if (mx4::overlap(ro, rx) || (!same && mx4::overlap(ro, ry)) || meets(ids, t * 4) ||
      meets(L->a, (size_t)L->n * L->rank * L->K * 2) || meets(L->b, (size_t)L->n * L->rank * N * 2) ||
      meets(L->scale, (size_t)L->n * 4) || meets(L->ranks, (size_t)L->n * 4))
    return QSM_ERR_INVALID_ARGUMENT;
  Params p = {};
  p.x = x;
  p.a = L->a;
  p.b = L->b;
  p.scale = L->scale;
  p.ranks = L->ranks;
  p.ids = ids;
  p.y = static_cast<const char*>(y);
  p.out = static_cast<char*>(out);
  p.ldx = ldx;
  p.ldy = ldy;
  p.ldo = ldo;
  p.T = T;
  p.K = L->K;
  p.N = L->N;
  p.R = L->rank;
  p.n = L->n;
  const int64_t wide = 16 / (int64_t)el < 8 ? 4 : 8;
  p.how = N % 8 == 0 && on(out, 16) && ldo % wide == 0 && (!y || (on(y, 16) && ldy % wide == 0)) ? kDirect : kRagged;
  const auto on32 = [&](const void* q) { return on(q, 32); };
  p.wide_in = on32(x) && on32(L->a) && L->K % 16 == 0 && ldx % 16 == 0;
  p.wide_out = on32(out) && ldo * el % 32 == 0;
  p.copy = !same;
  p.status = dev_status;
  const bool f32 = dtype == QSM_FP32;
  if (grouped(T, L->n))
    return L->rank <= 32 ? launch<1, true>(p, f32, stream) : L->rank <= 64 ? launch<2, true>(p, f32, stream) : launch<4, true>(p, f32, stream);
  return L->rank <= 32 ? launch<1, false>(p, f32, stream) : L->rank <= 64 ? launch<2, false>(p, f32, stream) : launch<4, false>(p, f32, stream);
}
