// evo_seq_index.h — index arithmetic of the causal-sequence kernels that no run on a GPU checks well: it has
// to hold up to the longest sequences (2^31 keys) and the widest groups (128 heads), and a wait must be for
// the phase that it means.  Plain C++, compiled for the host too.
#pragma once

#if defined(__CUDACC__)
#define EVO_HD __host__ __device__ __forceinline__
#else
#define EVO_HD inline
#endif

namespace evo {

// The first row (token by token, `group` heads each) of a tile of TQ tokens that sees a key
// `ahead` tokens behind the tile's first one (negative: in front of it, and every row sees it).
// A key in front of the tile may be 2^31 tokens away: the product is taken of no more than a tile.
EVO_HD int first_row(int ahead, int TQ, int group) { return (ahead > -TQ ? ahead : -TQ) * group; }

// Rows of a tile of TQ tokens that hold a token, where the sequence ends `left` tokens behind the
// tile's first one (up to 2^31: counted within the tile before the product).
EVO_HD int tile_rows(int left, int TQ, int group) { return (left < TQ ? left : TQ) * group; }

// The newest of the phases, counted from 0, that slot i of a ring has gone through after `uses` > i uses
// (the slots take turns, a phase each).
EVO_HD unsigned newest_phase(unsigned uses, unsigned slots, unsigned i) { return (uses - 1 - i) / slots; }

}  // namespace evo
