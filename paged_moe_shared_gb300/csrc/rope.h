// The rotation that a rope handle holds, for kernels that turn heads themselves.
#pragma once

#include <cstdint>

#include "../../include/rimuru.h"

namespace rimuru {

constexpr int kMaxPairs = 128;

struct RopeTurns {
  uint64_t turn[kMaxPairs];  // 2^-64 turns per position
  float mscale;
  int pairs, layout;
};
void rope_turns(rimuru_rope_t rope, RopeTurns* out);

}  // namespace rimuru
