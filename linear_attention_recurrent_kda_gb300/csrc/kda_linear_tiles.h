// The schedule of the product's form for many tiles (kda_linear.cu): which tiles a pair of
// CTAs takes, which part of them a warp of its epilogue, and when that warp asks for a
// part's residual.  Plain C++ that the host compiles too: tests/test_linear_schedule.py
// walks it on the CPU.
#pragma once

#ifdef __CUDACC__
#define KDA_BOTH __host__ __device__ __forceinline__
#else
#define KDA_BOTH inline
#endif

namespace kda {
namespace linear {

constexpr int kTileRows = 256, kTileCols = 256;  // tokens and features of a pair's tile
constexpr int kChunkRows = 32, kChunkCols = 64;  // of a warp's part of it
constexpr int kGroupRows = 8;                    // tiles along the tokens that run side by side

struct Tile {
  int row, col;
};
// Tiles in groups of kGroupRows along the tokens, so that those that run at a time
// share their operands in L2.
KDA_BOTH Tile tile_of(int n, int tiles_m, int tiles_n) {
  const int group = n / (kGroupRows * tiles_n), first = group * kGroupRows;
  const int left = tiles_m - first, high = kGroupRows < left ? kGroupRows : left;
  const int at = n - first * tiles_n;
  return Tile{(first + at % high) * kTileRows, at / high * kTileCols};
}

// A warp's chunks: one of each tile of its pair, in their order.  A tile at the output's end
// may have none for it (`there`).
struct Chunks {
  int rows, outer;                               // of the output
  int pair, pairs, row, col;                     // the pair's number; where in a tile

  KDA_BOTH int tiles_m() const { return (rows + kTileRows - 1) / kTileRows; }
  KDA_BOTH int tiles_n() const { return (outer + kTileCols - 1) / kTileCols; }
  // The chunk of the pair's q-th tile; whether there is such a tile.
  KDA_BOTH bool of(int q, Tile *at) const {
    const int n = pair + q * pairs;
    if (n >= tiles_m() * tiles_n()) return false;
    *at = tile_of(n, tiles_m(), tiles_n());
    at->row += row;
    at->col += col;
    return true;
  }
  KDA_BOTH bool there(const Tile &at) const { return at.row < rows && at.col < outer; }
};

// Calls work(q, chunk, there) for each tile, until one returns false, and before it, for
// each chunk that is there, fetch(chunk) once: for the first tile ahead of all, for the
// others when the tile before has been worked on, whether its own chunk was there or not.
template <class Fetch, class Work>
KDA_BOTH void walk_chunks(const Chunks &chunks, Fetch fetch, Work work) {
  Tile at = {0, 0};
  bool more = chunks.of(0, &at), there = more && chunks.there(at);
  for (int q = 0; more; ++q) {
    if (there) fetch(at);
    if (!work(q, at, there)) return;
    more = chunks.of(q + 1, &at);
    there = more && chunks.there(at);
  }
}

}  // namespace linear
}  // namespace kda
