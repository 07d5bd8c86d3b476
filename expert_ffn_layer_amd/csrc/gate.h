// Launchers of the gate: experts chosen by scores with a bias, groups and weights as a rule says, and its gradient.
#pragma once
#include "common.h"

namespace moe {

constexpr int GATE_GROUPS_MAX = 64;

struct GateArgs {
  const float* logits;    // [nparts][T][ldl]: parts that are added, with ldl >= E
  const float* bias;      // [E] or NULL
  float* sums;            // [T][E] or NULL: the added logits
  int32_t* idx;           // [T][k]
  float* w;               // [T][k]
  const int32_t* chosen;  // gradient: idx as input
  const float* dw;        // [T][k]
  float* dlogits;         // [T][E]
  double scale;
  int ldl, nparts, T, E, k;
  int sigmoid, renormalize, groups, top_groups, group_top;
  int whole;              // rows are read 16 bytes at a time (set by the launch)
};

GateArgs gate_args(const moe_shape& s, const moe_gate_rule& r);  // of T, E, k and the rule, for logits [T][E]
hipError_t launch_gate(const GateArgs& a, hipStream_t st);
hipError_t launch_gate_backward(const GateArgs& a, hipStream_t st);

}  // namespace moe
