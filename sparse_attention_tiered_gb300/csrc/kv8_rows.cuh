// Attention where every token has its own list of pages (spin_kv8_attend_rows): blocks of rows, and the pages that their
// tokens list.
#pragma once

#include "kv8_dev.cuh"

namespace spin {
namespace kv8 {

// Rows of a block: two tiles, or as many rows as 64 tokens have, so that a page's tokens are two words of bits. (256 rows
// of one head are 32 tokens of a group of 8.)
__host__ __device__ __forceinline__ int list_rows(int G) { return G < 4 ? 64 * G : 2 * kTileRows; }
// Tokens that have rows in a block, at most.
__host__ __device__ __forceinline__ int list_tokens(int G) { return list_rows(G) % G ? (list_rows(G) - 1) / G + 2 : list_rows(G) / G; }

// A block's items are pairs, a step each: item 2 n + t is for tile t. Where one of the tiles has fewer, its places are empty.
struct alignas(16) RowBlock {
  int32_t b, h, first_row;
  int32_t row0, n_new;  // of the request, n_new as if the block were its last
  int32_t past, full, tail;
  int32_t shared;       // at most 128 rows: both tiles have them, and take their pages in turn
  int32_t steps;
  int32_t weight;       // steps, and what beginning and ending the block costs; 0: there are none
  int32_t reserved;
  int64_t place;        // of its items
  int64_t reserved2;
};
static_assert(sizeof(RowBlock) == 64, "");

constexpr int kNoItem = -1, kTailItem = -2;
struct alignas(16) RowItem {
  int32_t page;        // of the pool, or kNoItem, kTailItem
  int32_t number;      // of the request
  uint32_t tokens[2];  // of the block, that list it: bit per token
};

struct RowLists {
  int32_t* n_blocks;
  RowBlock* blocks;
  RowItem* items;
};

}  // namespace kv8

// Attention of blocks over their lists (k_kv8_lists.cu).
cudaError_t launch_kv8_lists(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const kv8::RowLists& lists,
                             void* workspace, int sm_count, cudaStream_t st);

}  // namespace spin
