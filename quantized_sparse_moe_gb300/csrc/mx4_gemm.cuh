// Parameters of the MXFP4 product kernel (mx4_gemm.cu), shared with the MoE
// layer that issues its grouped modes (mx4_moe.cu).
#pragma once

#include "mx4_common.cuh"

namespace qsm {
namespace mx4 {

// kDense: y = a w^T.  kGateUp: rows of a grouped by expert, 128 gate and the
// 128 up rows of the same intermediates, h = silu(gate) * up quantized to
// MXFP4.  kDown: the grouped h times the expert's down rows, one row per row
// of a, in fp16 with a power of two per row and kOutCols columns.
enum { kDense = 0, kGateUp = 1, kDown = 2 };

constexpr int kOutCols = 128;  // columns of the grouped outputs that share a power of two
// Rows of w per tile of kDown (H = 2048, I = 512: 183.9 us a layer at 4096
// tokens and 109.7 at 300; 192, which leave room for two accumulators: 186.7
// and 110.0; 128: 190.6 and 113.3; all before the outputs' powers of two).
constexpr int kDownRows = 256;

struct GemmParams {
  CUtensorMap a, a32, a8;  // codes of a, boxes of 128, 32 and 8 rows
  CUtensorMap w, w_sh;   // codes of w (routed, shared), boxes of BN rows (gate_up: 128)
  CUtensorMap y_map, y8_map;  // down: the outputs, boxes of 32 and 8 rows
  CUtensorMap a_sf, w_sf;  // scale tiles, boxes of two (pairs of CTAs)
  const uint8_t* a_scales;
  const uint8_t* w_scales;
  const uint8_t* w_scales_sh;
  int M, N, K;           // N: rows of w (per expert)
  int tiles;             // row tiles of a (dense)
  int nsub;              // column tiles
  void* y;               // dense and down
  float* y_scale;        // down: [rows, N / kOutCols], what the fp16 in y are to be multiplied with
  size_t ldy;            // dense
  int align;             // dense, of the rows of y: 32 or 16 bytes, 0: less
  // grouped: tile tau < shared_tiles holds tokens 128 tau .. of the shared
  // expert, the others the blocks of tile_map (expert, first sorted row);
  // tile tau's rows of a (and of h and of y) start at 128 tau
  int T, I, shared_tiles;
  const int32_t* offsets;
  const int32_t* tile_map;
  const int32_t* n_tiles;
  uint8_t* h_codes;      // [tiles * 128, I / 2]
  uint8_t* h_scales;
  int32_t* status;
};

bool mx4_valid(const qsm_mx4* w);
// The maps of a (rows x K codes).
bool make_a_maps(GemmParams* p, const void* codes, uint64_t rows, int K);
// gate_up, or down with p.y of `rows` rows of p.N fp16 and p.y_scale.
qsm_status launch_grouped(GemmParams& p, int mode, uint64_t rows, cudaStream_t stream);

}  // namespace mx4
}  // namespace qsm
