// Parameters of the one-launch MXFP4 MoE layer (mx4_decode.cu).
#pragma once

#include "mx4_digits.cuh"

namespace qsm {
namespace mx4 {

struct DecodeParams {
  CUtensorMap gu, gu_sh, dn, dn_sh;  // codes, boxes of 128 rows
  const uint8_t* gu_sc;              // scale tiles
  const uint8_t* gu_sc_sh;
  const uint8_t* dn_sc;
  const uint8_t* dn_sc_sh;
  const uint16_t* x;        // [T, H] bf16
  const float* w_router;    // [E, H]
  const float* bias;        // [E] or null
  const float* sgate;       // [H] or null
  int T, H, I, E, k, flags;
  int epc;                  // experts per CTA in the router
  int32_t* topk_idx;
  float* topk_w;
  uint16_t* y;
  float* y32;
  unsigned long long* ticket;  // arrivals of all calls
  unsigned long long* logits;  // [T, E] (tag, logit)
  unsigned long long* h;       // [slots, T, I] (tag, h)
  int32_t* status;
  // geometry: ring stages, accumulator columns, shared-memory offsets
  int stages, acc_cols, seg_bytes;
  int x_off, xsf_off, rows_off, xs_off, h_off, hsf_off, part_off;
  int skew;                 // test hook: added to the awaited tag of the logits (0)
};

// Whether the layer and T can run in one launch here (geometry into p), and
// what the launch takes.
bool plan_decode(const qsm_mx4_layer* L, int T, DecodeParams* p, int* smem, int* ctas);
size_t decode_workspace_bytes(const DecodeParams& p);
qsm_status launch_decode(const DecodeParams& p, int smem, int ctas, cudaStream_t stream);

}  // namespace mx4
}  // namespace qsm
