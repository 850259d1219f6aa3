// The page pool of an 8-bit cache: spin_kv8_reserve, spin_kv8_fork, spin_kv8_compact.
//
// The pool's state is one count per page, of the table entries that name it. Pages are handed out in ascending order, so
// that what a call does follows from the counts alone: a bit per free page and a number per 1024 of them are made first
// (4 bytes a page, read once), and the j-th free page is then found by a search in the sums of those numbers, which
// every CTA makes for itself, and in 32 words of bits. No list of free pages has to be kept in order.
//
// All but the moving of many pages is a chain of dependent loads and two launches, the second of which begins under the first.
// Reserving one token of 256 requests from a pool of 858,000 pages, 3.4 MB of counts, takes 16 us through the Python call; the
// chunks of 24 requests, from a small pool, take 13 (both with a copy of some 3 us that puts the state back).
#include "kv8_dev.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 1024;  // pages of a chunk: a word of bits a lane

struct PoolSpace {  // the workspace of a call
  uint32_t* free_bits;  // [chunks][32]
  int32_t* free_in;     // [chunks]
  int32_t* wanted;      // [B] pages that a request needs
};

__host__ __device__ __forceinline__ int64_t chunks_of(int64_t n_pages) { return (n_pages + kChunk - 1) / kChunk; }

PoolSpace space_of(const Kv8Args& a, void* workspace) {
  const int64_t chunks = chunks_of(a.n_pages);
  PoolSpace s;
  s.free_bits = static_cast<uint32_t*>(workspace);
  s.free_in = reinterpret_cast<int32_t*>(s.free_bits + 32 * chunks);
  s.wanted = s.free_in + chunks;
  return s;
}

// The pages that a request's step completes: entries [first, first + pages) of each of its heads.
__device__ __forceinline__ int completes(const Kv8Args& a, int b, bool report, int& first) {
  int row0, n_new, past;
  if (!kv8_request(a, b, report, row0, n_new, past)) n_new = 0;
  first = past >> 6;
  return n_new ? ((past + n_new) >> 6) - first : 0;
}

// A warp a chunk of counts; and (requests > 0) a warp a request, for the entries that want a page.
__global__ void __launch_bounds__(kThreads)
kv8_pool_count(const Kv8Args a, const int32_t* refs, PoolSpace s, int requests) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t chunks = chunks_of(a.n_pages);
  int64_t i = (int64_t)blockIdx.x * kWarps + warp;
  if (i < chunks) {
    const int64_t first = i * kChunk;
    uint32_t mine = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const int64_t page = first + w * 32 + lane;
      const uint32_t bits = __ballot_sync(0xffffffffu, page < a.n_pages && refs[page] == 0);
      if (lane == w) mine = bits;
    }
    s.free_bits[i * 32 + lane] = mine;
    const int n = __reduce_add_sync(0xffffffffu, __popc(mine));
    if (lane == 0) s.free_in[i] = n;
    return;
  }
  i -= chunks;
  if (i >= requests) return;
  const int b = (int)i;
  int first;
  const int pages = completes(a, b, lane == 0, first), all = pages * a.Hkv;
  int n = 0;
  for (int x = lane; x < all; x += 32) {
    const int h = x / pages, p = first + x - h * pages;
    n += a.table[((int64_t)b * a.Hkv + h) * a.max_pages + p] < 0;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) s.wanted[b] = n;
}

// The sums of n numbers before each of them, to `out`, and their sum. Every thread of the CTA comes here.
__device__ int prefix_sums(const int32_t* in, int n, int32_t* out, int32_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int before = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int x = base + tid < n ? in[base + tid] : 0;
    int sum = x;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    int mine = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) mine += scratch[w];
      before += scratch[w];
    }
    if (out && base + tid < n) out[base + tid] = mine + sum - x;
    __syncthreads();
  }
  return before;
}

// The j-th free page, or the j-th that is not free, j below their number.
template <bool FREE>
__device__ __forceinline__ int nth_page(const PoolSpace& s, const int32_t* sums, int chunks, int j) {
  auto before = [&](int c) { return FREE ? sums[c] : c * kChunk - sums[c]; };
  int lo = 0, hi = chunks;  // the last chunk with no more than j before it
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before(mid) <= j) lo = mid;
    else hi = mid;
  }
  int rest = j - before(lo);
  const uint4* words = reinterpret_cast<const uint4*>(s.free_bits + (int64_t)lo * 32);
  int at = 0;
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint4 v = words[k];
    const uint32_t w[4] = {FREE ? v.x : ~v.x, FREE ? v.y : ~v.y, FREE ? v.z : ~v.z, FREE ? v.w : ~v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = __popc(w[e]);
      if (rest >= 0 && rest < n) bits = w[e], at = k * 4 + e;
      if (rest >= 0) rest = rest < n ? rest - 0x10000 : rest - n;  // found: negative from here on
    }
  }
  rest += 0x10000;
  for (; rest > 0; --rest) bits &= bits - 1;
  return lo * kChunk + at * 32 + (__ffs(bits) - 1);
}

// Free pages below this one (which is in the pool).
__device__ __forceinline__ int free_before(const PoolSpace& s, const int32_t* sums, int page) {
  const int c = page / kChunk, last = page >> 5 & 31;
  int n = sums[c];
  const uint4* words = reinterpret_cast<const uint4*>(s.free_bits + (int64_t)c * 32);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint4 v = words[k];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = k * 4 + e;
      n += x < last ? __popc(w[e]) : x == last ? __popc(w[e] & ((1u << (page & 31)) - 1u)) : 0;
    }
  }
  return n;
}

// A CTA a request: its first page is the one after those of the requests before it, and all or none are taken, so every CTA
// adds up what all requests want (65 KB at most, from L2).
__global__ void __launch_bounds__(kThreads)
kv8_pool_reserve(const Kv8Args a, int32_t* refs, PoolSpace s, int32_t* free_pages) {
  extern __shared__ int32_t sums[];  // [chunks]
  __shared__ int32_t scratch[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int mine = s.wanted[b];
  if (mine == 0 && b != 0) return;
  const int chunks = (int)chunks_of(a.n_pages);
  const int free = prefix_sums(s.free_in, chunks, sums, scratch);
  int64_t before = 0, all = 0;
  for (int x = tid; x < a.B; x += kThreads) {
    const int n = s.wanted[x];
    all += n;
    if (x < b) before += n;
  }
  __shared__ int64_t part[2][kWarps];
  for (int o = 16; o; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) part[0][warp] = all, part[1][warp] = before;
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all += part[0][w], before += part[1][w];
  const bool enough = all <= free;
  if (b == 0 && tid == 0) {
    if (!enough) atomicOr(a.err, (uint32_t)kErrCapacity);
    if (free_pages) *free_pages = enough ? free - (int)all : free;
  }
  if (!enough || mine == 0) return;
  int first;
  const int pages = completes(a, b, false, first), entries = pages * a.Hkv;
  int rank = (int)before;
  for (int base = 0; base < entries; base += kThreads) {
    const int x = base + tid;
    int32_t* entry = nullptr;
    bool want = false;
    if (x < entries) {
      const int h = x / pages;
      entry = const_cast<int32_t*>(a.table) + ((int64_t)b * a.Hkv + h) * a.max_pages + first + x - h * pages;
      want = *entry < 0;
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, want);
    if (lane == 0) scratch[warp] = __popc(vote);
    __syncthreads();
    int j = rank + __popc(vote & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) j += scratch[w];
      rank += scratch[w];
    }
    __syncthreads();
    if (want && j < free) {
      const int page = nth_page<true>(s, sums, chunks, j);
      *entry = page;
      refs[page] = 1;
    }
  }
}

// Of the U pages in use those with ids of U and more go to the free ones below U, in order: the j-th of them is the j-th page
// in use behind those below U, and its place is the j-th free one, so every CTA finds both ends of what it copies for itself,
// all of them at once. A CTA a page at a time, 16 bytes a thread and load, four on their way. The table's entries follow by the same rule.
// Bound by HBM: 16,000 pages, 527 MB to and from, 95 us alone, 5.6 TB/s or 0.82 of the copy's rate.
__global__ void __launch_bounds__(kThreads)
kv8_pool_move(const Kv8Args a, int32_t* refs, PoolSpace s, int32_t* free_pages) {
  extern __shared__ int32_t sums[];  // [chunks]
  __shared__ int32_t scratch[kWarps];
  __shared__ int2 ends[kThreads];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int chunks = (int)chunks_of(a.n_pages);
  const int free = prefix_sums(s.free_in, chunks, sums, scratch);
  const int used = (int)a.n_pages - free;
  if (blockIdx.x == 0 && tid == 0 && free_pages) *free_pages = free;
  const int holes = used < a.n_pages ? free_before(s, sums, used) : 0;  // as many as pages that go
  constexpr int kVec = kKv8PageBytes / 16 / kThreads;
  for (int64_t first = blockIdx.x; first < holes; first += (int64_t)kThreads * gridDim.x) {  // a thread a page, for its ends
    const int64_t j = first + (int64_t)tid * gridDim.x;
    __syncthreads();
    if (j < holes) ends[tid] = make_int2(nth_page<false>(s, sums, chunks, used - holes + (int)j), nth_page<true>(s, sums, chunks, (int)j));
    __syncthreads();
    const int n = (int)min((int64_t)kThreads, (holes - first + gridDim.x - 1) / gridDim.x);
    for (int i = 0; i < n; ++i) {
      const int from = ends[i].x, to = ends[i].y;
      const uint4* src = reinterpret_cast<const uint4*>(a.pages + (int64_t)from * kKv8PageBytes);
      uint4* dst = reinterpret_cast<uint4*>(a.pages + (int64_t)to * kKv8PageBytes);
      uint4 v[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] = __ldcs(src + k * kThreads + tid);
#pragma unroll
      for (int k = 0; k < kVec; ++k) dst[k * kThreads + tid] = v[k];
      if (tid == 0) *reinterpret_cast<float2*>(a.scales + 2 * (int64_t)to) = *reinterpret_cast<const float2*>(a.scales + 2 * (int64_t)from);
      if (tid == 32) refs[to] = refs[from], refs[from] = 0;
    }
  }
  const int64_t entries = (int64_t)a.B * a.Hkv * a.max_pages;
  int32_t* table = const_cast<int32_t*>(a.table);
  for (int64_t x = (int64_t)blockIdx.x * kThreads + tid; x < entries; x += (int64_t)gridDim.x * kThreads) {
    const int e = table[x];
    if (e < 0) continue;
    if (e >= a.n_pages || (s.free_bits[e >> 5] >> (e & 31) & 1)) atomicOr(a.err, (uint32_t)kErrIndex);  // a page that is not in use
    else if (e >= used) table[x] = nth_page<true>(s, sums, chunks, e - free_before(s, sums, e) - (used - holes));
  }
}

// ---------------------------------------------------------------------------
// Forking. Requests' rows change places among themselves, in place: a CTA takes a range of columns of all moved
// requests, reads every source into registers, and only then writes. No copy of the rows has to be kept anywhere, and
// any map of requests to requests will do. Summaries go along whichever page an entry named before.
// One prompt of 469 pages into 7 others, 29 MB: 14 to 17 us a call; 64 of 128 requests of 20 to 98 pages, 35 MB: 20.5 us (both with a
// copy of some 3 us that puts the state back). The lengths' launch takes 3: they may change only when every CTA has read them.
// ---------------------------------------------------------------------------
constexpr int kForkThreads = 512;
constexpr int kHeld = 32;         // 32-bit registers a thread, of the columns that pass through it
constexpr int kMostRows = kHeld / 4 * kForkThreads;  // that a CTA can hold 16 bytes each of

struct Move {
  int32_t to, from, len;  // `from` -1: emptied
};

// Elements (m, c), c < width, of all moves: get(m, c) for all of them, then put(m, c, element).
template <typename E, typename Get, typename Put>
__device__ __forceinline__ void pass(int moves, int log_width, Get get, Put put) {
  constexpr int N = kHeld * 4 / sizeof(E);
  const int n = moves << log_width;
  E v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = threadIdx.x + k * kForkThreads;
    v[k] = i < n ? get(i >> log_width, i & ((1 << log_width) - 1)) : E{};
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = threadIdx.x + k * kForkThreads;
    if (i < n) put(i >> log_width, i & ((1 << log_width) - 1), v[k]);
  }
}

template <typename E>
__device__ __forceinline__ int log_width(int moves, int most) {  // lanes a row: up to `most`, some four elements a thread
  int w = 0;
  const int cap = moves > 4 * kForkThreads ? kHeld * 4 / (int)sizeof(E) * kForkThreads : 4 * kForkThreads;
  while (1 << (w + 1) <= most && (int64_t)moves << (w + 1) <= cap) ++w;
  return w;
}

template <typename E>
__device__ void copy_summaries(const Kv8Args& a, const Move* moves, int n_moves, int h, int page0, int bytes) {
  // head h's rows from page0 on, `bytes` of them, of all moves' requests, as far as the source has pages that are whole
  const int64_t stride = (int64_t)a.Hkv * a.max_pages * kD * 4, off = ((int64_t)h * a.max_pages + page0) * kD * 4;
  const int lw = log_width<E>(n_moves, bytes / (int)sizeof(E));
  for (int x = 0; x < bytes; x += (int)sizeof(E) << lw) {
    __syncthreads();
    auto there = [&](int m, int c) {
      return moves[m].from >= 0 && page0 + (x + c * (int)sizeof(E)) / (kD * 4) < moves[m].len / kPart;
    };
    auto at = [&](int b, int c) {
      return reinterpret_cast<E*>(reinterpret_cast<uint8_t*>(a.summaries) + b * stride + off + x + c * (int64_t)sizeof(E));
    };
    pass<E>(
        n_moves, lw, [&](int m, int c) { return there(m, c) ? *at(moves[m].from, c) : E{}; },
        [&](int m, int c, const E& v) { if (there(m, c)) *at(moves[m].to, c) = v; });
  }
}

template <typename E>
__device__ void copy_tails(const Kv8Args& a, const Move* moves, int n_moves, int64_t off, int bytes) {
  const int lw = log_width<E>(n_moves, bytes / (int)sizeof(E));
  const int64_t stride = (int64_t)a.Hkv * kPageElems * 2;
  for (int x = 0; x < bytes; x += (int)sizeof(E) << lw) {
    __syncthreads();
    auto there = [&](int m, int c) {
      const int row = (int)((off + x + c * (int)sizeof(E)) & (kPart * kD * 2 - 1)) / (kD * 2);
      return moves[m].from >= 0 && row < (moves[m].len & (kPart - 1));
    };
    auto at = [&](int b, int c) {
      return reinterpret_cast<E*>(reinterpret_cast<uint8_t*>(a.tails) + b * stride + off + x + c * (int64_t)sizeof(E));
    };
    pass<E>(
        n_moves, lw, [&](int m, int c) { return there(m, c) ? *at(moves[m].from, c) : E{}; },
        [&](int m, int c, const E& v) { if (there(m, c)) *at(moves[m].to, c) = v; });
  }
}

constexpr int kTailBytes = 2048;  // of an item

// MANY: batches of more requests than a CTA can hold 16 bytes each of.
template <bool MANY>
__global__ void __launch_bounds__(kForkThreads, MANY ? 1 : 2)
kv8_pool_fork(const Kv8Args a, int32_t* refs, const int32_t* len, const int32_t* src, int log_columns) {
  extern __shared__ Move moves[];  // [B]
  __shared__ int n_moves, most_pages;
  const int tid = threadIdx.x;
  if (tid == 0) n_moves = most_pages = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  for (int b = tid; b < a.B; b += kForkThreads) {  // (their order does not matter)
    const int from = src[b];
    if (from == b) continue;
    uint32_t bad = from < -1 || from >= a.B ? (uint32_t)kErrIndex : 0u;
    int n = 0;
    if (!bad && from >= 0) {
      n = len[from];
      if (n < 0) bad = kErrIndex;
      else if ((int64_t)n > (int64_t)a.max_pages * kPart + kPart - 1) bad = kErrCapacity;
    }
    if (bad) {
      if (blockIdx.x == 0) atomicOr(a.err, bad);
      continue;
    }
    moves[atomicAdd(&n_moves, 1)] = Move{b, from, n};
    atomicMax(&most_pages, n / kPart);
  }
  __syncthreads();
  const int n = n_moves;
  if (n == 0) return;
  constexpr int kEntries = MANY ? kHeld : kHeld / 4;  // table entries that a thread holds
  const bool narrow = MANY && n > kMostRows;
  const int columns = 1 << log_columns, groups = (a.max_pages + columns - 1) / columns, tail_items = kPageElems * 2 / kTailBytes;
  const int64_t items = (int64_t)a.Hkv * (groups + tail_items);
  int32_t* table = const_cast<int32_t*>(a.table);
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    __syncthreads();
    const int h = (int)(item % a.Hkv), g = (int)(item / a.Hkv);
    if (g < tail_items) {
      const int64_t off = (int64_t)h * kPageElems * 2 + (int64_t)g * kTailBytes;
      if constexpr (MANY) {
        if (narrow) copy_tails<uint32_t>(a, moves, n, off, kTailBytes);
      }
      if (!narrow) copy_tails<uint4>(a, moves, n, off, kTailBytes);
      continue;
    }
    const int p0 = (g - tail_items) * columns, pages = min(columns, a.max_pages - p0);
    auto entry = [&](int b, int p) { return table + ((int64_t)b * a.Hkv + h) * a.max_pages + p; };
    // Entries: all of an item's of a request at a time, fewer where there are too many requests. Sources are read before any entry is written.
    int lw = log_columns;
    while (lw > 0 && (int64_t)n << lw > kEntries * kForkThreads) --lw;
    for (int x = 0; x < pages; x += 1 << lw) {
      __syncthreads();
      int32_t v[kEntries];
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        if (k * kForkThreads >= n << lw) break;
        const int i = tid + k * kForkThreads, m = i >> lw, c = i & ((1 << lw) - 1), p = p0 + x + c;
        v[k] = -1;
        if (m < n && p < a.max_pages && moves[m].from >= 0 && p < moves[m].len / kPart) v[k] = *entry(moves[m].from, p);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        if (k * kForkThreads >= n << lw) break;
        const int i = tid + k * kForkThreads, m = i >> lw, p = p0 + x + (i & ((1 << lw) - 1));
        if (m >= n || p >= a.max_pages) continue;
        int32_t* e = entry(moves[m].to, p);
        const int old = *e;
        if (old == v[k]) continue;
        *e = v[k];
        if (old >= 0) {
          if (old < a.n_pages) atomicSub(refs + old, 1);
          else atomicOr(a.err, (uint32_t)kErrIndex);
        }
        if (v[k] >= 0) {
          if (v[k] < a.n_pages) atomicAdd(refs + v[k], 1);
          else atomicOr(a.err, (uint32_t)kErrIndex);
        }
      }
    }
    if (a.summaries && p0 < most_pages) {
      if constexpr (MANY) {
        if (narrow) copy_summaries<uint32_t>(a, moves, n, h, p0, pages * kD * 4);
      }
      if (!narrow) copy_summaries<uint4>(a, moves, n, h, p0, pages * kD * 4);
    }
  }
}

// The lengths follow: one CTA, all read before any is written.
__global__ void __launch_bounds__(1024)
kv8_pool_lengths(const Kv8Args a, int32_t* len, const int32_t* src) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int v[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int b = k * 1024 + threadIdx.x;
    v[k] = -1;
    if (b >= a.B) continue;
    const int from = src[b];
    if (from == b || from < -1 || from >= a.B) continue;
    const int n = from < 0 ? 0 : len[from];
    if (n >= 0 && (int64_t)n <= (int64_t)a.max_pages * kPart + kPart - 1) v[k] = n;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (v[k] >= 0) len[k * 1024 + threadIdx.x] = v[k];
}

unsigned at_most(int64_t n, int64_t limit) { return (unsigned)(n < 1 ? 1 : n < limit ? n : limit); }

// A launch may have 48 KB of shared memory unasked, the kernel's own included: 2.1 KB at most here.
cudaError_t shared_bytes(const void* kernel, size_t bytes) {
  return bytes <= 40 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

cudaError_t count(const Kv8Args& a, const int32_t* refs, const PoolSpace& s, int requests, cudaStream_t st) {
  const int64_t warps = chunks_of(a.n_pages) + requests;
  return launch_early(kv8_pool_count, dim3((unsigned)((warps + kWarps - 1) / kWarps)), kThreads, 0, st, a, refs, s, requests);
}

}  // namespace

int64_t kv8_pool_workspace(const Kv8Args& a) { return 4 * (33 * chunks_of(a.n_pages) + a.B); }

cudaError_t launch_kv8_reserve(const Kv8Args& a, int32_t* refs, int32_t* free_pages, void* workspace, cudaStream_t st) {
  const PoolSpace s = space_of(a, workspace);
  const size_t bytes = chunks_of(a.n_pages) * 4;
  cudaError_t e = shared_bytes(reinterpret_cast<const void*>(kv8_pool_reserve), bytes);
  if (e == cudaSuccess) e = count(a, refs, s, a.B, st);
  if (e != cudaSuccess) return e;
  return launch_early(kv8_pool_reserve, dim3((unsigned)a.B), kThreads, bytes, st, a, refs, s, free_pages);
}

cudaError_t launch_kv8_compact(const Kv8Args& a, int32_t* refs, int32_t* free_pages, void* workspace, int sm_count, cudaStream_t st) {
  const PoolSpace s = space_of(a, workspace);
  const size_t bytes = chunks_of(a.n_pages) * 4;
  cudaError_t e = shared_bytes(reinterpret_cast<const void*>(kv8_pool_move), bytes);
  if (e == cudaSuccess) e = count(a, refs, s, 0, st);
  if (e != cudaSuccess) return e;
  return launch_early(kv8_pool_move, dim3((unsigned)sm_count * 8), kThreads, bytes, st, a, refs, s, free_pages);
}

cudaError_t launch_kv8_fork(const Kv8Args& a, int32_t* refs, int32_t* len, const int32_t* src, int sm_count, cudaStream_t st) {
  const size_t bytes = (size_t)a.B * sizeof(Move);
  const bool many = a.B > kMostRows;
  cudaError_t e = many ? shared_bytes(reinterpret_cast<const void*>(kv8_pool_fork<true>), bytes)
                       : shared_bytes(reinterpret_cast<const void*>(kv8_pool_fork<false>), bytes);
  if (e != cudaSuccess) return e;
  // Pages of an item: 8, or 4 or 2 where the GPU could not be filled by items of 8. (64 of 128 requests of 20 to 98 pages:
  // 18.5 us with 2 or 4, 20.6 with 8; of 7 to 15 pages 13.0, 13.3 and 18.6; 7 of 8 requests of 469 pages: 23.9 with 2, 18.4 with 4,
  // 14.8 with 8.)
  int log_columns = 3;
  auto groups = [&] { return (int64_t)a.Hkv * ((a.max_pages + (1 << log_columns) - 1) >> log_columns); };
  while (log_columns > 1 && groups() < (int64_t)sm_count * 2) --log_columns;
  const int64_t items = groups() + (int64_t)a.Hkv * (kPageElems * 2 / kTailBytes);
  const int32_t* lengths = len;
  e = many ? launch_early(kv8_pool_fork<true>, dim3(at_most(items, sm_count)), kForkThreads, bytes, st, a, refs, lengths, src, log_columns)
           : launch_early(kv8_pool_fork<false>, dim3(at_most(items, (int64_t)sm_count * 2)), kForkThreads, bytes, st, a, refs, lengths, src, log_columns);
  if (e != cudaSuccess) return e;
  return launch_early(kv8_pool_lengths, dim3(1), 1024, 0, st, a, len, src);
}

}  // namespace spin
