// Parameters of the few-row MXFP4 product kernel (mx4_stream.cu): the dense
// product of a few rows, and the two expert products of the MoE layer with
// 16-bit activations (mx4_moe.cu).
#pragma once

#include "mx4_digits.cuh"

namespace qsm {
namespace mx4 {

// kRows: y = x w^T.  kRowsGateUp: tiles of 128 gate and the 128 up rows of
// one expert, h = silu(gate) * up in fp32.  kRowsDown: the expert's down rows
// times h, the fp32 output of every assignment.
enum { kRows = 0, kRowsGateUp = 1, kRowsDown = 2 };

struct StreamParams {
  CUtensorMap w, w_sh;  // codes of w (routed, shared), boxes of 128 rows
  const uint8_t* w_scales;
  const uint8_t* w_scales_sh;
  int N, K;             // rows of w (per expert), columns
  FastDiv ntiles;       // items per slot: row tiles of w (gate_up: pairs of them)
  int slots;            // kRows: groups of `tok` rows of x
  int T, k, I, H;
  // MoE: the router's choices [T, k], and the slots of the shared expert,
  // which come first
  const int32_t* topk_idx;
  int E, shared_tiles, tok_log;
  FastDiv k_div;
  const uint16_t* x;    // [T, ldx] bf16 (kRows, kRowsGateUp)
  size_t ldx;
  float* h;             // [T k + T, I] fp32, by assignment, then the shared expert's: written by gate_up,
                        // read by down
  float* o;             // [T k + T, H] fp32 (kRowsDown)
  uint16_t* y;          // [T, N] bf16 (kRows)
  int32_t* status;
  // geometry (host): CTAs per cluster (the split of K), rows of x per slot,
  // digit buffers, ring stages, accumulators, and shared-memory offsets
  int cs, tok, nb, segs, stages, nacc, acc_cols, groups, tmem_cols;
  int cs_log;           // log2 cs
  int seg_bytes;        // digits of one stage's columns
  int dig_off, sf_off, part_off;
};

// Fills the geometry of p for slots of `tok` rows, with about `tiles` items
// for nsm SMs; false when the digits do not fit.
bool plan_rows(StreamParams* p, int mode, int tiles, int tok, int nsm);
// One launch over at most `items` items.
qsm_status launch_rows(StreamParams& p, int mode, int items, cudaStream_t stream);
bool mx4_valid(const qsm_mx4* w);

}  // namespace mx4
}  // namespace qsm
