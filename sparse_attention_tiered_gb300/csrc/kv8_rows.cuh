// Attention where every token has its own list of pages (spin_kv8_attend_rows): the tiles of tokens that its kernels share.
#pragma once

#include "kv8_dev.cuh"

namespace spin {
namespace kv8 {

// A tile: as many neighbouring tokens of a request as have at most 32 rows of one head between them. Neighbours list much
// the same pages, so a tile's items are the pages that any of its rows lists, each with a bit per row; and a page
// costs a tile of 32 rows little more than it costs one of 8.
constexpr int kRowsOfTile = 32;
__host__ __device__ __forceinline__ int tile_tokens(int G) { return kRowsOfTile / G; }

struct alignas(16) Tile {
  int32_t b, h;
  int32_t token0, tokens;  // rows of q and out: tokens [token0, token0 + tokens)
  int32_t see0;            // what the first of them sees: tokens 0 .. see0 - 1; the next one more, and so on
  int32_t full, tail;      // the request's complete pages, and tokens behind them
  int32_t listed;          // pages
  int32_t items;           // those, and one more for the tail if a row sees it
  int32_t reserved[3];
};
static_assert(sizeof(Tile) == 48, "");

struct alignas(16) Item {
  int32_t page;   // of the pool
  int32_t pos;    // of its first token
  uint32_t rows;  // row r of the tile attends it: bit r
  int32_t reserved;
};

struct RowsSpace {
  int32_t* tiles_there;  // number of tiles
  Tile* tiles;
  Item* items;           // of a tile: from place_of() on, in the order of the pages
};

// A tile has room for what its tokens list one by one, and the page that each is in.
__device__ __forceinline__ int64_t place_of(const Tile& t, int Hkv, int topk) {
  return ((int64_t)t.token0 * Hkv + (int64_t)t.h * t.tokens) * (topk + 1);
}

}  // namespace kv8
}  // namespace spin
