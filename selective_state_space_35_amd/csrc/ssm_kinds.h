// Kinds of kernels behind those of ssm_profile.h, for ssm_profile_read().  They stand in a header of their own: ssm_profile.h
// is a source of every scan, and the scans' committed counters hold for the sources that they were taken on.
#pragma once

#include "ssm_profile.h"

namespace ssm {

enum : int {
  kKindDeltaTri = kNumKinds,                // 26, gated delta rule: triangular inverses of the chunks
  kKindDeltaSweep = kNumKinds + 1,          // gated delta rule: a sweep over the sequence (outputs, states, or their gradients)
  kKindDeltaGrad = kNumKinds + 2,           // gated delta rule backward: the chunks' gradients
  kKindDeltaReduce = kNumKinds + 3,         // gated delta rule backward: sums over the heads of a group
  kKindDeltaUpdate = kNumKinds + 4,         // gated delta rule: single-token state update
  kKindBlockNormFwd = kNumKinds + 5,        // norms around a block
  kKindBlockNormBwd = kNumKinds + 6,        // norms around a block, backward: gradients, partial parameter gradients
  kKindBlockNormReduce = kNumKinds + 7,     // norms around a block, backward: sums of the partial parameter gradients
  kKindDeltaChain = kNumKinds + 8,          // gated delta rule: states leaving the parts of a cut sequence
  kAllKinds = kNumKinds + 9
};

}  // namespace ssm
