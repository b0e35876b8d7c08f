// How many tokens a launch takes, so that its grid stays below 2^32 threads. Plain C++: a test
// on the host includes it.
#pragma once

namespace moeq {

constexpr long GRID_MAX_BLOCKS = 0x7FFFFF;  // of 512 threads

// The tiled INT8 products, whose smallest tile is 32 channels x 64 tokens: 2^16 tokens, fewer
// for more than 2^18 channels (1984 for 2^23).
constexpr long int8_tokens(int rows) {
  const long t = GRID_MAX_BLOCKS / (((long)rows + 31) / 32) * 64;
  return t < (1 << 16) ? t : 1 << 16;
}

// The router: 2^22 tokens are 2^20 tiles of 64 tokens x 64 of up to 1024 experts (whose hidden
// size is not split at that number), and 2^20 work-groups of four tokens.
constexpr long ROUTER_TOKENS = 1 << 22;

// Packing and dequantisation of INT4 tensors: work-groups of 256 threads to a launch, with four tiles
// of 2048 weights or 256 times eight weights each.
constexpr long INT4_BLOCKS = 1 << 23;

}  // namespace moeq
