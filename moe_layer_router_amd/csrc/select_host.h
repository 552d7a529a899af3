// What the host code of the selection (select.hip) shares with the layer's
// backward pass, whose router gradient may go through it.
#pragma once
#include "host.h"

namespace moe {

constexpr int kSelMaxK = 16, kSelMaxE = 1024, kSelMaxGroups = 64, kSelWaves = 4;

struct SelArgs {
  const float* logits;       // [T][E]
  const float* bias;         // [E] or NULL
  int32_t* ids;              // [T][k]
  float* w;                  // [T][k]
  long T;
  int E, k, sigmoid, groups, keep, top, renorm;
  int lanes_log2;            // lanes that share a group, as a power of two
  int direct;                // E <= 256, and a group is the same 2 (E <= 128) or 4 experts of each of those lanes
  int per;                   // experts of a group
  float per_inv;
  float tol;                 // what fp32 scores are compared up to, relative
  float scale;
  // backward
  const int32_t* ids_in;
  const float* dw;           // [T][k]
  float* dl;                 // [T][E], or (for the layer's backward pass) with what `aux` adds as two BF16 parts:
  const float* aux;          // [T][E] or NULL
  uint16_t* hi;
  uint16_t* lo;
};

// The gradient's launch (select.hip), for the layer's backward pass too.
moe_status launch_select_bwd(const SelArgs& a, int cus, hipStream_t st);
// What it takes of a selection, its inputs checked.
moe_status select_bwd_args(const moe_selection* s, const float* logits, const int32_t* topk_ids, SelArgs* out);

}  // namespace moe
