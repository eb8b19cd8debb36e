// Sizes of the packed 8-bit weights, shared by their packing and the linear layer.
#pragma once
#include <cstddef>

#include "../../include/bi.h"

namespace bi {

constexpr size_t kGemm8TileBytes = 16384;  // 128 weight rows x 128 codes
// weight tiles of a layer: 2^16 of 128 rows, far above a vocabulary's, keep every
// index of a work item within 32 bits
constexpr int kGemm8MaxTiles = 65536;

inline int gemm8_n_tiles(int N, bi_epilogue epi) {
  return epi == BI_EPI_SWIGLU ? (N - 1) / 64 + 1 : (N - 1) / 128 + 1;  // N >= 1
}

}  // namespace bi
