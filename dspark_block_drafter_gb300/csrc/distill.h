// Distillation of the head from a teacher's listed tokens: the call's plan and the host
// launchers.  The products, the statistics and the sums over rows are the head loss's (loss.h),
// with the most probable listed token of a row as its label; what the other listed tokens add is done
// by the kernels here.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "loss.h"

namespace dspark {

constexpr int kMaxTargets = 256;      // listed tokens of a row, at most

struct DistillPlan {
  LossPlan p;                // its labels are `label` below
  int k;
  float scale;               // of the teacher's logits
  const int32_t* ids;        // [T][k]
  const float *logits, *t_lse;        // [T][k], [T] or NULL
  // workspace
  int32_t* label;            // [T] most probable listed token of the row, -1: none, V: refused
  int32_t* row;              // [T][k] head rows of the listed tokens, -1: absent; of the compact
                             // rows' tokens, compact head rows once their logits are known
  float* log_q;              // [T][k]
  float* mass;               // [T] sum of q
  float* z;                  // [Tp][k] logits of the listed tokens of the compact rows; with
                             // several pieces -log p of them once it is known
  float* w;                  // [Tp] w_t of the compact rows (LossPlan::wrow has w_t times mass)
};

constexpr int kDistillDone = 6;       // control word: row CTAs whose loss is written

cudaError_t launch_distill_targets(const DistillPlan& d);             // label, row, log_q, mass
cudaError_t launch_distill_logits(const DistillPlan& d);              // z, w, after the loss's plan
// losses and total; with `entries` (one piece) q's entries of the listed tokens too
cudaError_t launch_distill_loss(const DistillPlan& d, bool entries);
// q's entries of the listed tokens among columns [v0, v1), after the losses without them
cudaError_t launch_distill_entries(const DistillPlan& d, int v0, int v1);

}  // namespace dspark
