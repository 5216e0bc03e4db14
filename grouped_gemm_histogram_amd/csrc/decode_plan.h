// decode_plan.h -- what the first kernel of the layer for few tokens leaves for the second.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kDecodeTokens = 16;               // tokens of a call
constexpr int kDecodeRows = kDecodeTokens * 16; // routed rows

struct alignas(16) DecodePlan {
  int active;                           // experts that have rows
  int unused[3];
  float weight[kDecodeRows];            // of each routed row
  uint16_t expert[kDecodeRows];         // the active experts
  uint8_t count[kDecodeRows];           // rows of each
  uint8_t rows[kDecodeRows][kDecodeTokens];   // their routed rows, ascending
};

}  // namespace moe
