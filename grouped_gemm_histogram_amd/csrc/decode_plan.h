// decode_plan.h -- what the first kernel of the layer for few tokens leaves for the second.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kDecodeTokens = 16;               // tokens of a call
constexpr int kDecodeRows = kDecodeTokens * 16; // routed rows

// The list of experts that have rows, an expert once for each eight of them.
struct alignas(16) DecodePlan {
  int entries;
  int most;                         // rows of the largest of them
  int unused[2];
  float weight[kDecodeRows];        // of each routed row
  uint16_t id[kDecodeRows];         // its expert
  uint16_t expert[kDecodeRows];     // of each entry
  uint8_t count[kDecodeRows];       // its rows, 1 to 8
  uint8_t rows[kDecodeRows][8];     // the routed rows, ascending
  uint8_t tokens[kDecodeRows][8];   // and their tokens
};

}  // namespace moe
