// Scales of 8-bit blocks: byte e stands for 2^(e - 127), 255 for NaN (include/psd.h).
#pragma once

#include "device.cuh"

namespace psd {

// Blocks of a pool: the byte of token slot `slot` and KV head h is at[(slot / block) * Hkv + h].
struct BlockScales {
  const uint8_t *k = nullptr, *v = nullptr;
  int shift = 0;  // log2 of the block
};

__device__ __forceinline__ float scale_value(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fffffffu : e << 23);
}

}  // namespace psd
