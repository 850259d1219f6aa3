// Device code shared by the attention kernels of the 8-bit paged cache: barriers and copies,
// conversions, and the split of a call's work over its CTAs.
#pragma once

#include <cuda_fp16.h>

#include "kv8.cuh"

namespace spin {
namespace kv8 {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t tx) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(tx) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// A try that may suspend the thread for up to a microsecond.
__device__ __forceinline__ bool mbar_try_1us(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000)
      : "memory");
  return ok != 0;
}

// Waits until the phase with this parity has completed. Bounded: after 2^21 tries (of about a
// microsecond at most), or once another wait of the CTA has run out, it returns false with *abort
// (shared memory) set.
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 21); ++it) {
    if (mbar_try_1us(bar, parity)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  atomicOr(err, (uint32_t)kErrTimeout);
  return false;
}

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  if (mbar_try(bar, parity)) return true;
  return mbar_wait_slow(bar, parity, abort, err);
}

// After a wait has run out: copies and products in flight are given a quarter of a second to end before
// the memory that they use goes.
__device__ __forceinline__ void settle_down() {
  for (int i = 0; i < 250000; ++i) __nanosleep(1000);
}

// The same by a whole warp; `ok` is one for all lanes, and no wait succeeds once it is false.
__device__ __forceinline__ void warp_wait(bool& ok, uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  const bool there = mbar_try(bar, parity);
  if (!__all_sync(0xffffffffu, there && ok)) ok = __all_sync(0xffffffffu, ok && mbar_wait_slow(bar, parity, abort, err));
}

// A whole page [2][64] rows of 128 bytes, 16-byte chunk c of row r at chunk c ^ (r & 7).
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(page), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Two e4m3 codes to two halves, exactly.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t w, bool high) {
  uint32_t r;
  const uint16_t c = (uint16_t)(high ? w >> 16 : w);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 2^n for a whole n in the normal range.
__device__ __forceinline__ float pow2(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }

// The exponent e, clamped to [-60, 128], that puts bf16 values of up to `amax` (its bits, finite) below 2^e:
// times 2^(15 - e) they use fp16's whole range, so that every bf16 down to 2^-29 of the largest is exact.
__device__ __forceinline__ int half_exponent(uint32_t amax) { return max((int)(amax >> 7) - 126, -60); }

// log2 of a page's scale: exact for powers of two.
__device__ __forceinline__ float scale_log2(float s) {
  const uint32_t u = __float_as_uint(s);
  if (s != s) return s;
  return (float)((int)(u >> 23 & 255u) - 127) + __log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
}

// ---------------------------------------------------------------------------
// The split of a call's work. A unit is one (request, KV head); a tile is a block of its rows (row r:
// token r / G, head r % G). Per tile, a unit's items are the pages that the tile's last token may see
// (or its list of pages), and the tail; the few-row kernel takes the tail first, the other one last. The items
// of all units lie in one row, each unit's behind unit_cost places that stand for the work of beginning
// and ending it, and CTA c of P takes the places from c W / P on. The cost is in pages: 8 for the few-row
// kernel (48 requests of 0 to 16384 tokens take 26.1 us; with 4, 6 and 11 places 30.2, 29.3 and 25.4; lists of 32
// pages 33.9, and 34.3, 34.1 and 33.7); 6 where the many-row kernel's two tiles have rows of their own, and 11
// where they share a block and pass a page in half of the time (prompts of 300 to 6000 tokens take 575 us with 6
// places, 587 with 8, 592 with 11; drafts of 5 tokens 139, 137 and 136). Measured at those sizes, not derived: a unit's
// beginning and end in page times, which a longer tail or a shorter list moves little.
// ---------------------------------------------------------------------------
constexpr int kTileRows = 128;  // of the many-row kernel
__device__ __forceinline__ int unit_cost(int block_rows, int rows_there) {
  return block_rows < kTileRows ? 8 : rows_there > kTileRows ? 6 : 11;
}

struct Unit {  // of one request: the same for all of its heads
  int row0, n_new, past;
  int full;     // complete pages
  int tail;     // tokens of the tail
  int pages;    // entries of the page list
  int items;    // pages, and one for the tail if the tile sees it
  int weight;   // items + unit_cost, or 0
};

// A request's numbers; n_new and the rest 0 where they are out of range.
__device__ __forceinline__ Unit request_of(const Kv8Args& a, int b, bool report) {
  Unit u;
  const bool ok = kv8_request(a, b, report, u.row0, u.n_new, u.past);
  const int len = u.past + u.n_new;
  u.full = ok ? len >> 6 : 0;
  u.tail = ok ? len & (kPart - 1) : 0;
  u.pages = u.items = u.weight = 0;
  return u;
}

// The items that a block of rows of the request has.
__device__ __forceinline__ void set_rows(const Kv8Args& a, Unit& u, int first_row, int rows, int topk) {
  u.pages = u.items = u.weight = 0;
  if ((int64_t)u.n_new * a.G <= first_row) return;  // the block has no row of this request
  const int last = min(u.n_new, (first_row + rows - 1) / a.G + 1);  // tokens up to the block's last row
  const int seen = u.past + last;
  u.pages = topk ? topk : min(u.full, (seen + kPart - 1) >> 6);
  u.items = u.pages + (u.tail && seen > u.full * kPart ? 1 : 0);
  u.weight = u.items ? u.items + unit_cost(rows, u.n_new * a.G - first_row) : 0;
}

__device__ __forceinline__ Unit unit_of(const Kv8Args& a, int b, int first_row, int rows, int topk, bool report) {
  Unit u = request_of(a, b, report);
  set_rows(a, u, first_row, rows, topk);
  return u;
}

struct Place {
  int64_t total;   // places of all units
  int b;           // request of the place looked for
  int64_t before;  // places of the requests before it
};

// The request of place `at(total)` for every thread of the CTA, where request b has weight(b) places
// (scratch: 34 words). Each thread adds up a run of requests; the one whose run holds the place walks it.
template <typename Weight, typename At>
__device__ __forceinline__ Place locate(int requests, int64_t* scratch, Weight weight, At at) {
  const int tid = threadIdx.x, n = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = n >> 5;
  if (requests <= 128) {  // every warp for itself, up to four requests a lane
    const int run = (requests + 31) >> 5;
    int64_t m[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = lane * run + i;
      m[i] = i < run && x < requests ? weight(x, true) : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) mine += m[i];
    int64_t sum = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const int64_t total = __shfl_sync(0xffffffffu, sum, 31), want = at(total);
    int64_t before = sum - mine;
    int b = lane * run;
    const uint32_t holds = __ballot_sync(0xffffffffu, want >= before && want < sum);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (want >= before + m[i]) before += m[i], ++b;
      else break;
    const int from = holds ? __ffs(holds) - 1 : 0;
    b = __shfl_sync(0xffffffffu, b, from);
    before = __shfl_sync(0xffffffffu, before, from);
    __syncthreads();  // as below: the caller counts on one
    return holds ? Place{total, b, before} : Place{total, requests, total};
  }
  const int run = (requests + n - 1) / n, b0 = min(requests, tid * run), b1 = min(requests, b0 + run);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += weight(b, true);
  int64_t sum = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) scratch[warp] = sum;
  __syncthreads();
  int64_t base = 0, total = 0;
  for (int w = 0; w < warps; ++w) {
    const int64_t x = scratch[w];
    if (w < warp) base += x;
    total += x;
  }
  const int64_t lo = base + sum - mine, want = at(total);
  if (tid == 0) {
    scratch[32] = requests;
    scratch[33] = total;
  }
  __syncthreads();
  if (want >= lo && want < lo + mine) {
    int64_t before = lo;
    for (int b = b0; b < b1; ++b) {
      const int64_t m = weight(b, false);
      if (want < before + m) {
        scratch[32] = b;
        scratch[33] = before;
        break;
      }
      before += m;
    }
  }
  __syncthreads();
  return Place{total, (int)scratch[32], scratch[33]};
}

// ---------------------------------------------------------------------------
// Requests that count where a call has room for no more than its total_new rows (blocks, tiles, a place a row). While cu_new
// ascends no two requests have a row in common, and those in range have total_new between them at most. Where it descends
// they may name rows twice, each of them in range by itself. So a request counts if it is in range and begins behind
// the end of every one before it that is and has rows: those that count never share a row. (Where cu_new descends there is a request
// that ends before it begins, so the error word tells.)
// ---------------------------------------------------------------------------
// f(b, counts, row0, n_new) for all requests, a lane each, by a warp.
template <typename F>
__device__ __forceinline__ void each_request(const Kv8Args& a, F f) {
  const int lane = threadIdx.x & 31;
  int end = 0;  // of the requests so far
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    int row0 = 0, n_new = 0, past;
    const bool ok = b0 + lane < a.B && kv8_request(a, b0 + lane, false, row0, n_new, past);
    int most = ok && n_new ? row0 + n_new : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, most, o);
      if (lane >= o) most = max(most, y);
    }
    const int before = __shfl_up_sync(0xffffffffu, most, 1);
    f(b0 + lane, ok && row0 >= max(end, lane ? before : 0), row0, n_new);
    end = max(end, __shfl_sync(0xffffffffu, most, 31));
  }
}

// As locate, where a request that counts has weight(row0, n_new, past) places and the others none. `strange`: some
// request is out of range; only then there are any that might not count (bits: kMaxRequests / 32 words of shared memory).
template <typename Weight, typename At>
__device__ __forceinline__ Place locate_rows(const Kv8Args& a, int64_t* scratch, uint32_t* bits, bool report, bool& strange, Weight weight, At at) {
  bool mine = false;
  strange = false;
  for (;;) {
    const Place p = locate(
        a.B, scratch,
        [&](int b, bool first) {
          int row0, n_new, past;
          const bool ok = kv8_request(a, b, first && report, row0, n_new, past);
          mine |= !ok;
          return ok && (!strange || (bits[b >> 5] >> (b & 31) & 1)) ? weight(row0, n_new, past) : (int64_t)0;
        },
        at);
    // (locate has every warp look at up to 128 requests)
    if (strange || !(a.B <= 128 ? __any_sync(0xffffffffu, mine) : __syncthreads_or(mine))) return p;
    strange = true;
    if (threadIdx.x < 32)
      each_request(a, [&](int b, bool counts, int, int) {
        const uint32_t word = __ballot_sync(0xffffffffu, counts);
        if ((b & 31) == 0) bits[b >> 5] = word;
      });
    __syncthreads();
  }
}

// a / b of numbers that are not negative: a division in 32 bits takes a third of the one in 64, which is on the way
// to a CTA's first load.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The first place of CTA c's share of n, and the CTA whose share has place x.
__device__ __forceinline__ int64_t share_start(int64_t total, int c, int n) { return quotient(total * c, n); }
__device__ __forceinline__ int share_of(int64_t total, int64_t x, int n) { return (int)quotient((x + 1) * n - 1, total); }

// What a CTA does of the unit that holds the place `at` of its request (or row block), with `left` of its share to go.
struct Part {
  int h, from, to;  // items [from, to) of head h; none where from >= to
  int64_t took;
};

__device__ __forceinline__ Part part_of(const Unit& u, int64_t at, int64_t left) {
  Part x;
  x.h = (int)quotient(at, u.weight);
  const int f = (int)(at - (int64_t)x.h * u.weight), t = (int)min((int64_t)u.weight, f + left);
  x.took = t - f;
  x.from = max(0, f - (u.weight - u.items));
  x.to = max(0, t - (u.weight - u.items));
  return x;
}

// What a CTA leaves of a unit that it begins and does not end (parts 0: there is none), in the
// workspace's first bytes; the partials follow, two blocks of rows for each share: number 2 x for the
// unit that share x found begun, 2 x + 1 for the one that it began.
struct JoinRecord {
  int64_t total;  // places of all units
  int32_t parts, row0, n_new, h, first_row, reserved;
};
constexpr int kMaxCtas = 160;  // CTAs that a call's work is split over, at most
constexpr size_t kRecordBytes = kMaxCtas * sizeof(JoinRecord);
constexpr float kLog2e = 1.4426950408889634f;

// `end`: the place behind the unit's last.
__device__ __forceinline__ JoinRecord record_of(const Unit& u, int h, int first_row, int64_t total, int64_t end, int cta, int ctas) {
  return JoinRecord{total, share_of(total, end - 1, ctas) - cta + 1, u.row0, u.n_new, h, first_row, 0};
}

}  // namespace kv8
}  // namespace spin
