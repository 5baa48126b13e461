// Where the shares of a line of tiles may begin (attn_plan.cuh): plain integers,
// for the device and for a host compiler.
#pragma once

namespace qknr {

// A share is to begin `o` of `u` units into a tile, `over` of which are its
// beginning and end: the unit where it does begin, `u` for the next tile's first.
// No cut where it saves little, less than two blocks from an end of the tile's
// blocks: such a place moves to the nearer end of the tile, and where that is
// its beginning and the tile may be cut before here, to the last such cut.  A
// larger `o` never moves before a smaller one's place: shares that began in
// another order than their CTAs' would leave parts of a tile to nobody.
__host__ __device__ __forceinline__ int share_cut(int o, int u, int over) {
  const int last = u - over - 2;                  // the last unit for a cut
  if (o < 2) return 0;
  if (o <= last) return o;
  return 2 * o >= u ? u : last >= 2 ? last : 0;
}

}  // namespace qknr
