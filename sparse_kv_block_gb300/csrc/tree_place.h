// tree_place.h -- where in a request's tiles a CTA's range begins (plain C++
// too, so that it can be checked at sizes that would run for long).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define OASIS_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define OASIS_HOST_DEVICE inline
#endif

namespace oasis {

struct TreePlace {
  int pair, tile;  // pair: KV head * blocks of rows + block; tile of its tiles
};
// Tile `in` of a request whose pairs have `tiles` each.  16384 tiles x 4 blocks
// x 65535 heads are more than 2^31 and 2^32, so `in` has 64 bits; pairs fit in 32.
// (A division of 64 bits only where it is one.)
OASIS_HOST_DEVICE TreePlace tree_place(int64_t in, int tiles) {
  const int pair = static_cast<int>(in >> 32 ? in / tiles : static_cast<uint32_t>(in) / static_cast<uint32_t>(tiles));
  return {pair, static_cast<int>(in - static_cast<int64_t>(pair) * tiles)};
}

}  // namespace oasis
