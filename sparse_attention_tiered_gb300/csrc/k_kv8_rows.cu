// spin_kv8_attend_rows: attention where every token has its own list of pages.
//
// One token a request: its list goes to the few-row kernel as it is, but in order and without pages twice. More than one:
// blocks of rows attend the pages that any of their tokens lists (k_kv8_lists.cu). The lists are made here, by a launch
// before. (A token at a time, the few-row kernel takes 720 clocks a page and token.)
#include "kv8_rows.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 2048;  // pages that are marked at a time
// Steps that beginning and ending a block costs. (Six ragged prompts: 68.1 us with 1, 58.4 with 4, 57.8 with 8, 60.8 with 20; one long
// chunk, whose blocks are alike, 513 to 521.)
constexpr int kUnitSteps = 8;
// Of the blocks that are laid out at a time, and their items. A block's are sized for lists that have nothing in common, so tokens
// by the ten thousand take turns: three launches each, which is little beside the attention of that many.
constexpr int64_t kTurnBytes = 4ll << 30;

// A CTA a block and head, of the rows of tokens t0 .. t1 - 1. The tokens' pages are marked in a window of shared memory, a bit a token, and read out in order;
// what lies beyond the window waits for the next, which begins at the lowest page that is left. One chain of loads (lengths,
// lists, table) and no more than a GPU's worth of CTAs for 512 tokens of 8 heads: 10 us alone, cold, whatever the lists.
__global__ void __launch_bounds__(kThreads)
kv8_rows_blocks(const Kv8Args a, const Rows out, const int32_t* sel, int topk, int64_t cap, int t0, int t1, RowLists s) {
  __shared__ __align__(16) uint32_t marks[2][kWindow];
  __shared__ int64_t scratch[36];
  __shared__ uint32_t bits[kMaxRequests / 32];
  __shared__ int found[kWarps][2], next[kWarps], most[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = list_rows(a.G);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = blockIdx.x % a.Hkv, number = blockIdx.x / a.Hkv;
  int row0, n_new, past;
  bool strange;
  // Requests that count share no row, so that their blocks are no more than were launched and have a place (most_blocks).
  const Place pl = locate_rows(
      a, scratch, bits, blockIdx.x == 0, strange,
      [&](int row, int n, int) { return ((int64_t)max(0, min(row + n, t1) - max(row, t0)) * a.G + R - 1) / R; },
      [&](int64_t) { return (int64_t)number; });
  if (blockIdx.x == 0 && tid == 0) *s.n_blocks = (int)pl.total * a.Hkv;
  if (pl.b >= a.B || !kv8_request(a, pl.b, false, row0, n_new, past)) return;
  RowBlock t;
  t.b = pl.b;
  t.h = h;
  t.first_row = max(0, t0 - row0) * a.G + (int)(number - pl.before) * R;
  t.row0 = row0;
  t.n_new = (int)(min((int64_t)min(n_new, t1 - row0) * a.G, (int64_t)t.first_row + R) + a.G - 1) / a.G;
  t.past = past;
  t.full = (past + n_new) >> 6;
  t.tail = (past + n_new) & (kPart - 1);
  t.reserved = 0;
  t.reserved2 = 0;
  t.place = (int64_t)blockIdx.x * cap;
  const int i0 = t.first_row / a.G, tokens = t.n_new - i0;
  // Tokens that have rows in the first tile of 128, [0, in0), and in the second, from from1 on.
  const int skip = t.first_row - i0 * a.G, rows = min(R, t.n_new * a.G - t.first_row);
  t.shared = rows <= kTileRows;
  const int in0 = min(tokens, (kTileRows - 1 + skip) / a.G + 1), from1 = (kTileRows + skip) / a.G;
  const int64_t unit = (int64_t)t.b * a.Hkv + h;
  const int32_t* table = a.table + unit * a.max_pages;
  const int32_t* lists = sel + ((int64_t)(row0 + i0) * a.Hkv + h) * topk;
  const int64_t step = (int64_t)a.Hkv * topk;
  RowItem* items = s.items + t.place;
  int count[2] = {0, 0};  // pages of each tile; shared: of the block, the first alone
  for (int base = 0; base != 0x7fffffff;) {
    for (int x = tid * 4; x < 2 * kWindow; x += 4 * kThreads) *reinterpret_cast<uint4*>(marks[0] + x) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int beyond = 0x7fffffff, last = -1;
    auto mark = [&](int p, int token) {
      if (p < base) return;
      if (p - base < kWindow) {
        atomicOr(&marks[token >> 5][p - base], 1u << (token & 31));
        last = max(last, p - base);
      } else {
        beyond = min(beyond, p);
      }
    };
    for (int x = tid; x < tokens * topk; x += kThreads) {
      const int i = x / topk, p = lists[i * step + x - i * topk];
      if (p >= 0 && p < (past + i0 + i + 1) >> 6) mark(p, i);  // pages that it sees whole
    }
    if (tid < tokens) {  // the page that it is in
      const int see = past + i0 + tid + 1;
      if (see >> 6 < t.full && (see & (kPart - 1))) mark(see >> 6, tid);
    }
    beyond = __reduce_min_sync(0xffffffffu, beyond);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) next[warp] = beyond, most[warp] = last;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) beyond = min(beyond, next[w]), last = max(last, most[w]);
    for (int x = 0; x <= last; x += kThreads) {
      RowItem it = RowItem{0, base + x + tid, {marks[0][x + tid], marks[1][x + tid]}};
      bool there = (it.tokens[0] | it.tokens[1]) != 0;
      if (there) {
        it.page = table[it.number];
        if (it.page < 0 || (int64_t)it.page >= a.n_pages) {
          atomicOr(a.err, (uint32_t)kErrIndex);
          there = false;
        }
      }
      // For the tiles that have such tokens.
      const uint64_t who = (uint64_t)it.tokens[1] << 32 | it.tokens[0];
      const bool in[2] = {there && (t.shared || (who & (in0 < 64 ? (1ull << in0) - 1 : ~0ull)) != 0), there && !t.shared && from1 < 64 && who >> from1 != 0};
      uint32_t vote[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        vote[k] = __ballot_sync(0xffffffffu, in[k]);
        if (lane == 0) found[warp][k] = __popc(vote[k]);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int at = count[k] + __popc(vote[k] & ((1u << lane) - 1u));
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) at += found[w][k];
          count[k] += found[w][k];
        }
        at = t.shared ? at : 2 * at + k;
        if (in[k] && at < cap) *reinterpret_cast<uint4*>(items + at) = make_uint4(it.page, it.number, it.tokens[0], it.tokens[1]);
      }
      __syncthreads();
    }
    base = beyond;
    __syncthreads();
  }
  // The tail is the last page of every tile that sees some of it; then what is missing to whole steps.
  const int first_sees = past + i0 + in0;  // what the first tile's last token sees
  if (tid < 2 && !(t.shared && tid)) {
    const bool sees = t.tail && (t.shared || tid ? past + t.n_new : first_sees) > t.full * kPart;
    const int at = t.shared ? count[0] : 2 * count[tid] + tid;
    if (sees && at < cap) *reinterpret_cast<uint4*>(items + at) = make_uint4((uint32_t)kTailItem, t.full, 0xffffffffu, 0xffffffffu);
  }
  if (t.tail && past + t.n_new > t.full * kPart) ++count[t.shared ? 0 : 1];
  if (!t.shared && t.tail && first_sees > t.full * kPart) ++count[0];
  t.steps = t.shared ? (count[0] + 1) / 2 : max(count[0], count[1]);
  t.weight = t.steps ? t.steps + kUnitSteps : 0;
  for (int x = (t.shared ? count[0] : 2 * min(count[0], count[1])) + tid; x < 2 * t.steps; x += kThreads)
    if ((t.shared || x >> 1 >= count[x & 1]) && x < cap)
      *reinterpret_cast<uint4*>(items + x) = make_uint4((uint32_t)kNoItem, 0, 0, 0);
  if (tid == 0) s.blocks[blockIdx.x] = t;
  if (t.steps == 0) {  // its rows see nothing
    for (int x = tid; x < rows * 16; x += kThreads) {
      const int row = t.first_row + (x >> 4), i = row / a.G;
      reinterpret_cast<uint4*>(out.p + (int64_t)(row0 + i) * out.ts + (int64_t)(h * a.G + row - i * a.G) * out.hs)[x & 15] =
          make_uint4(0, 0, 0, 0);
    }
  }
}

// One token a request: a warp a request and head. The same with a bit a page, so that a long cache is one window.
constexpr int kBits = 65536;

__global__ void __launch_bounds__(32)
kv8_rows_single(const Kv8Args a, const int32_t* sel, int topk, int32_t* lists) {
  __shared__ uint32_t marks[kBits / 32];
  const int lane = threadIdx.x, b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int row0, n_new, past;
  if (!kv8_request(a, b, false, row0, n_new, past) || n_new == 0) return;  // (the attention passes it over)
  const int full = (past + n_new) >> 6;
  const int32_t* list = sel + ((int64_t)row0 * a.Hkv + h) * topk;
  int32_t* out = lists + (int64_t)blockIdx.x * topk;
  int count = 0;
  for (int base = 0; base != 0x7fffffff;) {
    const int words = min(kBits / 32, (full - base + 31) >> 5);
    for (int x = lane; x < words; x += 32) marks[x] = 0;
    __syncwarp();
    int beyond = 0x7fffffff;
    for (int x = lane; x < topk; x += 32) {
      const int p = list[x];
      if (p < base || p >= full) continue;
      if (p - base < kBits) atomicOr(&marks[(p - base) >> 5], 1u << ((p - base) & 31));
      else beyond = min(beyond, p);
    }
    __syncwarp();
    for (int x = 0; x < words; x += 32) {
      uint32_t bits = x + lane < words ? marks[x + lane] : 0;
      if (!__any_sync(0xffffffffu, bits)) continue;
      const int n = __popc(bits);
      int sum = n;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      for (int at = count + sum - n; bits; bits &= bits - 1) out[at++] = base + (x + lane) * 32 + __ffs(bits) - 1;
      count += __shfl_sync(0xffffffffu, sum, 31);
    }
    base = __reduce_min_sync(0xffffffffu, beyond);
    __syncwarp();
  }
  for (int x = count + lane; x < topk; x += 32) out[x] = -1;
}

int64_t most_blocks(const Kv8Args& a, int64_t tokens) {  // of each head
  return tokens * a.G / list_rows(a.G) + (a.B < tokens ? a.B : tokens);
}

int64_t most_items(const Kv8Args& a, int topk) {  // of a block
  const int64_t n = (int64_t)list_tokens(a.G) * (topk + 1);
  return 2 * ((n < a.max_pages ? n : a.max_pages) + 1);  // of each tile, and the tail
}

int64_t block_bytes(const Kv8Args& a, int topk) {  // of all heads'
  return a.Hkv * ((int64_t)sizeof(RowBlock) + most_items(a, topk) * (int64_t)sizeof(RowItem));
}

// Tokens of a turn: as many as have no more blocks than kTurnBytes hold, by either bound on the requests among them.
int64_t turn_tokens(const Kv8Args& a, int topk) {
  const int64_t blocks = kTurnBytes / block_bytes(a, topk), R = list_rows(a.G);
  const int64_t few = (blocks - a.B) * R / a.G, many = blocks * R / (R + a.G);
  const int64_t n = few > many ? few : many > 1 ? many : 1;
  return n < a.total_new ? n : a.total_new;
}

}  // namespace

int64_t kv8_rows_workspace(const Kv8Args& a, int topk) {
  const int64_t lists = (int64_t)a.B * a.Hkv * topk * 4;
  const int64_t many = 16 + most_blocks(a, turn_tokens(a, topk)) * block_bytes(a, topk);
  return kv8_attend_workspace(a) + (many > lists ? many : lists);
}

cudaError_t launch_kv8_rows(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel, int topk,
                            void* workspace, int sm_count, cudaStream_t st) {
  uint8_t* rest = static_cast<uint8_t*>(workspace) + kv8_attend_workspace(a);
  if (a.max_new == 1) {
    int32_t* lists = reinterpret_cast<int32_t*>(rest);
    const cudaError_t e = launch_early(kv8_rows_single, dim3((unsigned)(a.B * a.Hkv)), 32, 0, st, a, sel, topk, lists);
    return e != cudaSuccess ? e : launch_kv8_attend(a, q, out, scale, lists, topk, workspace, sm_count, st);
  }
  const int64_t turn = turn_tokens(a, topk), most = most_blocks(a, turn) * a.Hkv;
  RowLists s;
  s.n_blocks = reinterpret_cast<int32_t*>(rest);
  s.blocks = reinterpret_cast<RowBlock*>(rest + 16);
  s.items = reinterpret_cast<RowItem*>(s.blocks + most);
  for (int64_t t = 0; t < a.total_new; t += turn) {
    const int64_t tokens = t + turn < a.total_new ? turn : a.total_new - t, blocks = most_blocks(a, tokens) * a.Hkv;
    cudaError_t e = launch_early(kv8_rows_blocks, dim3((unsigned)blocks), kThreads, 0, st, a, out, sel, topk, most_items(a, topk), (int)t,
                                 (int)(t + tokens), s);
    if (e == cudaSuccess) e = launch_kv8_lists(a, q, out, scale, s, workspace, sm_count, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace spin
