// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = y[t] + c[a] B[a] (A[a] x[t]),     a = ids[t] (none: out[t] = y[t])
//
// in one launch.  The tokens are cut into tiles of 64 that follow one another;
// the distinct adapters of a tile are its slots, and a cluster of CTAs takes
// the slots s, s + S, ... of a tile and one of NS parts of the columns:
//
//   1. v = A[a] x[t] for the slot's tokens: every warp of the cluster has a
//      piece of K for all ranks and tokens (16 ranks x 8 tokens x 16 per MMA);
//      the warps' partial sums are added in a fixed order, first in the CTA,
//      then over the cluster through distributed shared memory;
//   2. out = y + (c v) B[a]^T: a warp takes 32 columns of all the slot's tokens
//      (16 tokens x 8 columns x 16 per MMA) and adds y in fp32.
//
// With NS > 1 each part forms v again for itself (A comes from L2 then), which
// is cheaper than a launch or a grid-wide exchange between the two products.
// A few tokens: bound by the latency of two dependent rounds of loads; many
// adapters: by reading them; prompts: by x, y and out.
//
// Operands go from global memory straight into MMA fragments: the order of the
// products of a sum is free, so a lane takes 8 consecutive values (16 bytes) of
// a row where the fragment's own order would have it take four times two.  In
// the same way the columns of four MMAs are dealt so that a lane ends up with 8
// consecutive columns of a token.
//
// v is rounded for the second product: c v is split into bf16 parts, two of them
// (2^-17 relative) for 16-bit outputs, which are rounded to 2^-9 anyway, three
// (exact but for fp32's own rounding) for 32-bit ones.
#include "mx4_common.cuh"

namespace qsm {
namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;    // tokens
constexpr int kMaxRank = 128;

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
  int cs, lanes, parts;   // CTAs of a cluster, slots' lanes S, column parts NS
  int rows;               // tokens of a tile, rounded up to 8: what the buffers hold
  int vec;                // whether eight columns of y and out can be one access
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
  static constexpr int kRowTiles = 2 * RK;            // of 16 ranks
  static constexpr int kTokTiles = 8 / RK;            // of 8 tokens, at once: 64 accumulators a lane
  static constexpr int kPartRow = kRanks + 4;         // floats: banks 8 apart for a lane's tokens
  static constexpr int kVRow = kRanks + (RK == 1 ? 0 : 32);  // bf16: rows 16 banks apart
};

// Bytes of shared memory for tiles of `rows` tokens.
template <int RK>
__host__ __device__ constexpr size_t parts_bytes(int rows) {
  const int at_once = rows < 8 * Shape<RK>::kTokTiles ? rows : 8 * Shape<RK>::kTokTiles;
  return (size_t)kWarps * at_once * Shape<RK>::kPartRow * 4;
}
template <int RK, int SPLIT>
__host__ __device__ constexpr size_t v_bytes(int rows) {
  return (size_t)SPLIT * ((rows + 15) / 16 * 16) * Shape<RK>::kVRow * 2;
}
template <int RK, int SPLIT>
__host__ __device__ constexpr size_t smem_bytes(int rows) {
  const size_t a = parts_bytes<RK>(rows), b = v_bytes<RK, SPLIT>(rows);
  return (a > b ? a : b) + (size_t)rows * Shape<RK>::kRanks * 4;
}

template <int RK, bool F32>
__global__ void __launch_bounds__(kThreads, 2)
lora_kernel(const __grid_constant__ Params p) {
  using S = Shape<RK>;
  constexpr int SPLIT = F32 ? 3 : 2;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) int ids[kTile];
  __shared__ unsigned long long slot_tokens[kTile];
  __shared__ int slot_id[kTile], mem[kTile], leaders[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int rank_cta = p.cs > 1 ? (int)mx4::cluster_rank() : 0;
  int cl = blockIdx.x / p.cs;  // cluster: (tile, slot lane, column part), the part fastest
  const int part = cl % p.parts;
  cl /= p.parts;
  const int slot0 = cl % p.lanes, t0 = cl / p.lanes * kTile;
  const int count = min(kTile, p.T - t0);
  pdl_wait();
  pdl_launch_dependents();

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
  const int slots = __popc((uint32_t)leaders[0]) + __popc((uint32_t)leaders[1]);

  float* parts = reinterpret_cast<float*>(smem);
  __nv_bfloat16* vbuf = reinterpret_cast<__nv_bfloat16*>(smem);  // after the partial sums
  const size_t psum_at = max(parts_bytes<RK>(p.rows), v_bytes<RK, SPLIT>(p.rows));
  float* psum = reinterpret_cast<float*>(smem + psum_at);        // [token][rank], read by the cluster
  const int at_once = min(p.rows, 8 * S::kTokTiles);

  const int kblocks = (p.K + 31) / 32, kw = p.cs * kWarps;
  const int kfirst = (int)((long long)kblocks * (rank_cta * kWarps + warp) / kw);
  const int klast = (int)((long long)kblocks * (rank_cta * kWarps + warp + 1) / kw);
  const int chunks = (p.N + 31) / 32, stride = p.parts * kw;  // of 32 columns
  const int chunk0 = (part * p.cs + rank_cta) * kWarps + warp;

  for (int slot = slot0; slot < slots; slot += p.lanes) {
    const int id = slot_id[slot];
    const unsigned long long tokens = slot_tokens[slot];
    const int m = __popcll(tokens);
    if (tid < kTile && ((tokens >> tid) & 1ull)) mem[__popcll(tokens & ((1ull << tid) - 1))] = tid;
    int rank = 0;
    if (id >= 0) rank = p.ranks ? min(max(__ldg(p.ranks + id), 0), p.R) : p.R;
    __syncthreads();
    const uint16_t* A = p.a + (size_t)(id < 0 ? 0 : id) * p.R * p.K;
    const uint16_t* B = p.b + (size_t)(id < 0 ? 0 : id) * p.N * p.R;

    if (rank > 0) {
      if (chunk0 < chunks) {  // the first columns' rows of B are on their way to L2 meanwhile
        const int nrow = chunk0 * 32 + lane;
        if (nrow < p.N) prefetch_l2(B + (size_t)nrow * p.R);
      }
      for (int c0 = 0; c0 < m; c0 += 8 * S::kTokTiles) {  // tokens at once
        const int mt = min(m - c0, 8 * S::kTokTiles);
        float acc[S::kRowTiles][S::kTokTiles][4];
#pragma unroll
        for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
          for (int j = 0; j < S::kTokTiles; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
        const uint16_t* xr[S::kTokTiles];
#pragma unroll
        for (int j = 0; j < S::kTokTiles; ++j)
          xr[j] = 8 * j + g < mt ? p.x + (size_t)(t0 + mem[c0 + 8 * j + g]) * p.ldx : nullptr;
        for (int kb = kfirst; kb < klast; ++kb) {
          const int k = kb * 32 + 8 * tq;
          const bool in = k < p.K;
          uint4 xv[S::kTokTiles];
#pragma unroll
          for (int j = 0; j < S::kTokTiles; ++j) {
            xv[j] = make_uint4(0, 0, 0, 0);
            if (in && xr[j]) xv[j] = __ldg(reinterpret_cast<const uint4*>(xr[j] + k));
          }
#pragma unroll
          for (int i = 0; i < S::kRowTiles; ++i) {
            if (16 * i >= rank) break;
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            if (in && 16 * i + g < rank) lo = __ldg(reinterpret_cast<const uint4*>(A + (size_t)(16 * i + g) * p.K + k));
            if (in && 16 * i + 8 + g < rank) hi = __ldg(reinterpret_cast<const uint4*>(A + (size_t)(16 * i + 8 + g) * p.K + k));
#pragma unroll
            for (int j = 0; j < S::kTokTiles; ++j) {
              if (8 * j >= mt) break;
              mma_bf16(acc[i][j], lo.x, hi.x, lo.y, hi.y, xv[j].x, xv[j].y);
              mma_bf16(acc[i][j], lo.z, hi.z, lo.w, hi.w, xv[j].z, xv[j].w);
            }
          }
        }
        float* mine = parts + (size_t)warp * at_once * S::kPartRow;
#pragma unroll
        for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
          for (int j = 0; j < S::kTokTiles; ++j) {
            if (16 * i >= rank || 8 * j >= mt) break;
            float* at = mine + (8 * j + 2 * tq) * S::kPartRow + 16 * i + g;
            at[0] = acc[i][j][0];
            at[S::kPartRow] = acc[i][j][1];
            at[8] = acc[i][j][2];
            at[S::kPartRow + 8] = acc[i][j][3];
          }
        __syncthreads();
        const int used = (rank + 15) / 16 * 16;
        for (int e = tid; e < mt * (used / 4); e += kThreads) {  // four ranks of a token
          const int tok = e / (used / 4), r = (e - tok * (used / 4)) * 4;
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(parts + ((size_t)w * at_once + tok) * S::kPartRow + r);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
          }
          *reinterpret_cast<float4*>(psum + (c0 + tok) * S::kRanks + r) = s;
        }
        __syncthreads();
      }
      if (p.cs > 1) cluster_sync_all();  // every CTA's sums are there
      // c v in bf16 parts, zeros up to whole MMAs
      const float c = p.scale ? __ldg(p.scale + id) : 1.f;
      const int blocks = (rank + 31) / 32, vrows = (m + 15) / 16 * 16;
      for (int e = tid; e < vrows * blocks * 8; e += kThreads) {
        const int tok = e / (blocks * 8), r = (e - tok * (blocks * 8)) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (tok < m && r < (rank + 15) / 16 * 16) {
          const uint32_t at = smem_u32(psum + tok * S::kRanks + r);
          for (int q = 0; q < p.cs; ++q) {
            const float4 u = p.cs > 1 ? dsmem_ld_f4(dsmem_addr_u32(at, q)) : *reinterpret_cast<const float4*>(psum + tok * S::kRanks + r);
            v[0] += u.x, v[1] += u.y, v[2] += u.z, v[3] += u.w;
          }
        }
        uint32_t w[SPLIT][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float rest = r + i < rank ? v[i] * c : 0.f;
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
          *reinterpret_cast<uint2*>(vbuf + ((size_t)s * ((p.rows + 15) / 16 * 16) + tok) * S::kVRow + r) =
              make_uint2(w[s][0], w[s][1]);
      }
      __syncthreads();
    }

    // columns
    const int blocks = (rank + 31) / 32;
    for (int ch = chunk0; ch < chunks; ch += stride) {
      uint4 bw[4][RK];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = ch * 32 + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
        for (int b = 0; b < RK; ++b) {
          const int r = 32 * b + 8 * tq;
          bw[j][b] = make_uint4(0, 0, 0, 0);
          if (n < p.N && r < rank)
            bw[j][b] = first_of(__ldg(reinterpret_cast<const uint4*>(B + (size_t)n * p.R + r)), rank - r);
        }
      }
      const int n = ch * 32 + 8 * tq;  // this lane's eight columns of tokens g and g + 8
      for (int mt = 0; mt < m; mt += 16) {
        float d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) d[j][e] = 0.f;
        float base[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = mt + 8 * h + g;
#pragma unroll
          for (int e = 0; e < 8; ++e) base[h][e] = 0.f;
          if (!p.y || row >= m || n >= p.N) continue;
          const char* src = p.y + ((size_t)(t0 + mem[row]) * p.ldy + n) * (F32 ? 4 : 2);
          if (p.vec) {
            if (F32) {
              const float4 u = *reinterpret_cast<const float4*>(src), v = *reinterpret_cast<const float4*>(src + 16);
              base[h][0] = u.x, base[h][1] = u.y, base[h][2] = u.z, base[h][3] = u.w;
              base[h][4] = v.x, base[h][5] = v.y, base[h][6] = v.z, base[h][7] = v.w;
            } else {
              const uint4 u = *reinterpret_cast<const uint4*>(src);
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                base[h][2 * e] = bf16_lo(w[e]);
                base[h][2 * e + 1] = bf16_hi(w[e]);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (n + e < p.N)
                base[h][e] = F32 ? reinterpret_cast<const float*>(src)[e]
                                 : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(src)[e] << 16);
          }
        }
#pragma unroll
        for (int b = 0; b < RK; ++b) {
          if (b >= blocks) break;
#pragma unroll
          for (int s = SPLIT - 1; s >= 0; --s) {  // the small parts first
            const __nv_bfloat16* vr = vbuf + ((size_t)s * ((p.rows + 15) / 16 * 16) + mt + g) * S::kVRow + 32 * b + 8 * tq;
            const uint4 lo = *reinterpret_cast<const uint4*>(vr), hi = *reinterpret_cast<const uint4*>(vr + 8 * S::kVRow);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma_bf16(d[j], lo.x, hi.x, lo.y, hi.y, bw[j][b].x, bw[j][b].y);
              mma_bf16(d[j], lo.z, hi.z, lo.w, hi.w, bw[j][b].z, bw[j][b].w);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = mt + 8 * h + g;
          if (row >= m || n >= p.N) continue;
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = base[h][e] + d[e >> 1][2 * h + (e & 1)];
          char* dst = p.out + ((size_t)(t0 + mem[row]) * p.ldo + n) * (F32 ? 4 : 2);
          if (F32) {
            if (p.vec) {
              reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
              reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (n + e < p.N) reinterpret_cast<float*>(dst)[e] = v[e];
            }
          } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
              w[e] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            if (p.vec) {
              *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (n + e < p.N) reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            }
          }
        }
      }
    }
    // the sums have been read everywhere, mem and v here, before they are written again (or the CTA leaves)
    if (p.cs > 1 && rank > 0) cluster_sync_all();
    else __syncthreads();
  }
}

template <int RK>
qsm_status launch(const Params& p, bool f32, long long ctas, cudaStream_t stream) {
  auto* kernel = f32 ? lora_kernel<RK, true> : lora_kernel<RK, false>;
  const size_t smem = f32 ? smem_bytes<RK, 3>(p.rows) : smem_bytes<RK, 2>(p.rows);
  const size_t most = f32 ? smem_bytes<RK, 3>(kTile) : smem_bytes<RK, 2>(kTile);
  QSM_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
  QSM_CUDA_TRY(launch_pdl_cluster(kernel, dim3((unsigned)ctas), dim3(kThreads), p.cs, smem, stream, p));
  return QSM_OK;
}

// A matrix of T rows of `bytes` bytes, `ld` bytes apart: whether two of them may
// have a byte in common (rows side by side in one matrix do not).
struct Rows {
  const void* p;
  size_t ld, bytes;
};
bool overlap(const Rows& a, size_t ta, const Rows& b, size_t tb) {
  if (!a.p || !b.p || !ta || !tb) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const size_t sa = (ta - 1) * a.ld + a.bytes, sb = (tb - 1) * b.ld + b.bytes;
  if (pa + sa <= pb || pb + sb <= pa) return false;
  if (a.ld != b.ld || a.ld == 0) return true;
  const size_t d = pb >= pa ? (pb - pa) % a.ld : (a.ld - (pa - pb) % a.ld) % a.ld;
  return !(d >= a.bytes && d + b.bytes <= a.ld);
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
  if (L->rank > kMaxRank) return QSM_ERR_UNSUPPORTED;
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
  const size_t t = T, N = L->N;
  const Rows rx = {x, (size_t)ldx * 2, (size_t)L->K * 2}, ry = {y, (size_t)ldy * el, N * el};
  const Rows ro = {out, (size_t)ldo * el, N * el};
  const auto flat = [](const void* p, size_t bytes) { return Rows{p, 0, bytes}; };
  const bool same = y == out && ldy == ldo;
  if (overlap(ro, t, rx, t) || (!same && overlap(ro, t, ry, t)) || overlap(ro, t, flat(ids, t * 4), 1) ||
      overlap(ro, t, flat(L->a, (size_t)L->n * L->rank * L->K * 2), 1) ||
      overlap(ro, t, flat(L->b, (size_t)L->n * L->rank * N * 2), 1) ||
      overlap(ro, t, flat(L->scale, (size_t)L->n * 4), 1) || overlap(ro, t, flat(L->ranks, (size_t)L->n * 4), 1))
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
  p.rows = T < kTile ? (T + 7) / 8 * 8 : kTile;
  const int64_t wide = 16 / (int64_t)el < 8 ? 4 : 8;
  p.vec = N % 8 == 0 && on(out, 16) && ldo % wide == 0 && (!y || (on(y, 16) && ldy % wide == 0));
  p.copy = !same;
  p.status = dev_status;
  // Clusters of 8 CTAs; as many slots' lanes as a tile can have slots while there are few tiles,
  // and columns in parts while that leaves SMs idle.
  p.cs = 8;
  const long long tiles = ((long long)T + kTile - 1) / kTile;
  const int slots = L->n + 1ll < (T < kTile ? T : kTile) ? L->n + 1 : (T < kTile ? T : kTile);
  const long long want = 4ll * mx4::sm_count() / p.cs;
  p.lanes = (int)(tiles * slots <= want ? slots : want / tiles < 1 ? 1 : want / tiles);
  p.parts = 1;
  const int chunks = (int)((N + 31) / 32);
  while (tiles * p.lanes * p.parts * 2 * p.cs <= mx4::sm_count() && p.parts * 2 * p.cs * kWarps <= chunks) p.parts *= 2;
  const long long ctas = tiles * p.lanes * p.parts * p.cs;
  if (ctas > 0x7fffffffll) return QSM_ERR_UNSUPPORTED;
  return L->rank <= 32 ? launch<1>(p, dtype == QSM_FP32, ctas, stream)
         : L->rank <= 64 ? launch<2>(p, dtype == QSM_FP32, ctas, stream)
                         : launch<4>(p, dtype == QSM_FP32, ctas, stream);
}
