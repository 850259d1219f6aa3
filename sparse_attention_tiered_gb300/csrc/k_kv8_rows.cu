// spin_kv8_attend_rows: attention where every token has its own list of pages.
//
// A first launch makes the lists of tiles of tokens out of those of tokens (kv8_rows.cuh), a second attends them, the third
// of spin_kv8_attend joins what CTAs shared.
//
// Products. A tile has up to 32 rows, an item is a page of 64 tokens: the tokens are the products' wide side, and the codes of
// the pages are their operands as they lie in memory, e4m3 by a copy into shared memory, so that no key or value is
// ever converted. What is not e4m3 is split: a number is a sum of e4m3 numbers of falling size, exactly for a
// bf16 query (8 bits: two pieces, the second times 16) and an fp16 weight (11 bits: three pieces, times 1, 16 and
// 256). Pieces are columns of their own on the narrow side, where columns are nearly free, and are added
// up in fp32. A step takes two pages:
//   S[128 tokens x 64] = K (shared memory) Q^T, 32 rows in two pieces, 4 products of depth 32,
//   O[128 dimensions x 96] += V^T P^T (shared memory, both with the tokens as rows), 32 rows in three pieces, 4 products.
// (The tensor cores' sums were measured against exact ones: off by 2^-20.7 of the sum of the terms' sizes at most.)
//
// A weight's pieces cost no conversion either: an fp16 number below 2 has its exponent's top bit clear, and the seven bits
// below are the e4m3 code of 256 times it, cut to 4 bits, subnormal numbers included. What was cut is subtracted, exactly,
// and so on. Weights are kept up to 1, so that what was cut is below 1 again when it is taken 16 times: 2^-5 at the
// reference, which is raised when one passes 1. Below 2^-14 they lose bits; what is below 2^-25 of 1 is lost.
//
// Arithmetic as in the few-row kernel of spin_kv8_attend: with s = score * k * log2(e) per page, weights are
// 2^((s - M) + (log2(v) - V)), the softmax sum takes weight / v; M, V per row.
//
// Roles, by warp:
//   0-3, 4-7  softmax, every second step each, a token a thread, with a reference, sums and an output of their own;
//   8         copies pages, one step's keys and values a stage, five stages;
//   9         issues the products;
//   10        walks the CTA's share of the items and splits the queries;
//   11, 12    the tail: bf16 rows to two e4m3 pieces, 64 tokens as 128 rows; scores of both pieces are added, and the
//             weights of the second are 1/16 of the first's.
#include "kv8_rows.cuh"
#include "kv8_tc.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kWindow = 2048;  // pages that are marked at a time

// A warp a tile. The tokens' pages are marked in a window of shared memory, a bit a token, and read out in order; what lies
// beyond the window waits for the next, which begins at the lowest page that is left.
__global__ void __launch_bounds__(32)
kv8_rows_lists(const Kv8Args a, const Rows rows, const int32_t* sel, int topk, RowsSpace s) {
  __shared__ __align__(16) uint32_t marks[kWindow];
  __shared__ int64_t scratch[36];
  const int lane = threadIdx.x, T = tile_tokens(a.G);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = blockIdx.x % a.Hkv, number = blockIdx.x / a.Hkv;
  int row0, n_new, past;
  const Place pl = locate(
      a.B, scratch,
      [&](int b, bool report) {
        return kv8_request(a, b, report && blockIdx.x == 0, row0, n_new, past) ? (int64_t)(n_new + T - 1) / T : 0ll;
      },
      [&](int64_t) { return (int64_t)number; });
  if (blockIdx.x == 0 && lane == 0) *s.tiles_there = (int)pl.total * a.Hkv;
  if (pl.b >= a.B || !kv8_request(a, pl.b, false, row0, n_new, past)) return;
  const int i0 = (int)(number - pl.before) * T;
  Tile t;
  t.b = pl.b;
  t.h = h;
  t.token0 = row0 + i0;
  t.tokens = min(T, n_new - i0);
  t.see0 = past + i0 + 1;
  t.full = (past + n_new) >> 6;
  t.tail = (past + n_new) & (kPart - 1);
  const int64_t unit = (int64_t)t.b * a.Hkv + h;
  const int32_t* table = a.table + unit * a.max_pages;
  Item* out = s.items + place_of(t, a.Hkv, topk);
  int count = 0;
  for (int base = 0; base != 0x7fffffff;) {
    for (int x = lane * 4; x < kWindow; x += 128) *reinterpret_cast<uint4*>(marks + x) = make_uint4(0, 0, 0, 0);
    __syncwarp();
    int next = 0x7fffffff, most = -1;
    auto mark = [&](int p, int token) {
      if (p < base) return;
      if (p - base < kWindow) {
        atomicOr(marks + (p - base), 1u << token);
        most = max(most, p - base);
      } else {
        next = min(next, p);
      }
    };
    for (int i = 0; i < t.tokens; ++i) {
      const int32_t* mine = sel + ((int64_t)(t.token0 + i) * a.Hkv + h) * topk;
      const int whole = (t.see0 + i) >> 6;  // pages that it sees whole
      for (int x = lane; x < topk; x += 32) {
        const int p = mine[x];
        if (p >= 0 && p < whole) mark(p, i);
      }
      if (lane == 0 && whole < t.full && ((t.see0 + i) & (kPart - 1))) mark(whole, i);  // the page that it is in
    }
    __syncwarp();
    next = __reduce_min_sync(0xffffffffu, next);
    most = __reduce_max_sync(0xffffffffu, most);
    for (int x = 0; x <= most; x += 32) {
      uint32_t bits = marks[x + lane];
      int page = 0;
      if (bits) {
        page = table[base + x + lane];
        if (page < 0 || (int64_t)page >= a.n_pages) {
          atomicOr(a.err, (uint32_t)kErrIndex);
          bits = 0;
        }
      }
      const uint32_t there = __ballot_sync(0xffffffffu, bits != 0);
      if (bits) {
        Item it;
        it.pos = (base + x + lane) * kPart;
        it.page = page;
        it.rows = 0;
        it.reserved = 0;
        for (; bits; bits &= bits - 1) it.rows |= ((1u << a.G) - 1u) << ((__ffs(bits) - 1) * a.G);
        out[count + __popc(there & ((1u << lane) - 1u))] = it;
      }
      count += __popc(there);
    }
    base = next;
    __syncwarp();
  }
  t.listed = count;
  t.items = count + (t.tail && t.see0 + t.tokens - 1 > t.full * kPart ? 1 : 0);
  if (lane == 0) s.tiles[blockIdx.x] = t;
  if (t.items == 0)  // its rows see nothing
    for (int i = 0; i < t.tokens; ++i)
      for (int x = lane; x < a.G * 16; x += 32)
        reinterpret_cast<uint4*>(rows.p + (int64_t)(t.token0 + i) * rows.ts + (int64_t)(h * a.G + (x >> 4)) * rows.hs)[x & 15] =
            make_uint4(0, 0, 0, 0);
}

constexpr int kThreads = 512;  // three warps idle: registers are given to four warps at a time
constexpr int kProducer = 8, kMmaWarp = 9, kPlanner = 10, kTailKeys = 11;  // and the values' after it
constexpr int kStages = 5, kTasks = 4, kReaders = 8 + 1 + 1 + 2;  // of a task: softmax, producer, products, tails
constexpr int kStageBytes = 2 * kKv8PageBytes;                    // two pages' keys, then their values
constexpr int kQueryBytes = 2 * kRowsOfTile * kD;                 // [piece][row][128]
constexpr int kWeightBytes = 2 * kPart * 128;                     // [token][piece][row], 128 bytes a token
constexpr uint32_t kColS = 0, kColO = 256;                        // tensor memory: S, two of 64 columns each; O, 128 each
constexpr float kShift = -5.f;                                    // log2 of a weight at the reference
constexpr float kFar = 2048.f;                                    // a sum of two exponents is right to 2^-13 below it
constexpr int kUnitCost = 6;                                      // pages that beginning and ending a tile cost

struct Task {
  Tile t;
  int from, to;  // items; none: the share is done
};

// Steps of a task: its pages two by two, and the tail.
__device__ __forceinline__ int task_pages(const Task& x) { return max(0, min(x.to, x.t.listed) - x.from); }
__device__ __forceinline__ int task_steps(const Task& x) { return ((task_pages(x) + 1) >> 1) + (x.to > x.t.listed ? 1 : 0); }

struct alignas(16) PageMeta {  // of a page of a step
  float kfac, vlog, vinv;
  int pos;
  uint32_t rows, bad;  // bad: a row that sees a token of it is NaN (the other numbers are finite all the same)
  uint32_t reserved[2];
};
struct WarpRows {  // of a softmax warp, a row each: minus the reference's score (without the query's factor), its other part
  float neg_m[kRowsOfTile], w[kRowsOfTile], f[kRowsOfTile];  // with the page's, and what a raised reference leaves of sums
};

struct Smem {
  uint64_t full[kStages], empty[kStages], tail_go[kStages];
  uint64_t task_full[kTasks], task_empty[kTasks], q_full[kTasks], q_empty[2];
  uint64_t s_full[2][2], p_full[2], pv_done[2];
  Task tasks[kTasks];
  PageMeta meta[kStages][2];
  float tail_kfac[kStages][kPart], tail_vlog[kStages][kPart], tail_vinv[kStages][kPart];
  uint8_t tail_bad[kStages][2][kPart];
  alignas(16) float qs[kTasks][kRowsOfTile];
  alignas(16) WarpRows rows[8];
  uint32_t wrong[kTasks];          // rows whose query is not finite
  float m[2][kRowsOfTile], w[2][kRowsOfTile], sum[2][kRowsOfTile];
  uint32_t poison[2][4];
  int top[2][kRowsOfTile];
  int64_t scratch[36];
  uint32_t tmem;
  int abort;
  float minus_zero;
};
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + 2 * kQueryBytes + 2 * kWeightBytes + sizeof(Smem);
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

// e4m3 x e4m3 -> fp32, M = 128; rows_depth: both operands are stored with their depth as rows.
constexpr uint32_t shape(int n, bool rows_depth) {
  return 1u << 4 | (rows_depth ? 3u << 15 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

__device__ __forceinline__ void mma_f8(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(leader)
      : "memory");
}

// Four numbers below 2^8 as two e4m3 pieces each: x = high + low / 16, exactly for 8 bits.
__device__ __forceinline__ void two_pieces(const float (&x)[4], uint32_t& high, uint32_t& low) {
  uint16_t h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    const uint32_t back = e4m3x2_half2(h[i], false);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l[i]) : "f"((x[2 * i + 1] - f.y) * 16.f), "f"((x[2 * i] - f.x) * 16.f));
  }
  high = h[0] | (uint32_t)h[1] << 16;
  low = l[0] | (uint32_t)l[1] << 16;
}

// Largest absolute value of a warp's bf16 pairs, its bits.
__device__ __forceinline__ uint32_t largest_of(uint2 w) {
  const uint32_t top = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
  return __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
}

// Numbers whose order as signed integers is that of the floats.
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x);
  return b ^ (b >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float float_of(int k) { return __int_as_float(k ^ (k >> 31 & 0x7fffffff)); }

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(addr));
  return x;
}

__global__ void __launch_bounds__(kThreads, 1)
kv8_rows_attend(const Kv8Args a, const __grid_constant__ CUtensorMap map, const Rows q, const Rows out, float scale, int topk,
                RowsSpace s, JoinRecord* records, float* partials) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (through an integer it would be a pointer to anywhere)
  const uint32_t ring = smem_u32(base), sq = ring + kStages * kStageBytes, sp = sq + 2 * kQueryBytes;
  Smem& sm = *reinterpret_cast<Smem*>(base + kStages * kStageBytes + 2 * kQueryBytes + 2 * kWeightBytes);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile int* abort = &sm.abort;
  const int ctas = gridDim.x, cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 2);
      mbar_init(smem_u32(&sm.empty[i]), 1);
      mbar_init(smem_u32(&sm.tail_go[i]), 1);
    }
    for (int i = 0; i < kTasks; ++i) {
      mbar_init(smem_u32(&sm.task_full[i]), 1);
      mbar_init(smem_u32(&sm.task_empty[i]), kReaders);
      mbar_init(smem_u32(&sm.q_full[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.q_empty[i]), 1);
      mbar_init(smem_u32(&sm.s_full[i][0]), 1);
      mbar_init(smem_u32(&sm.s_full[i][1]), 1);
      mbar_init(smem_u32(&sm.p_full[i]), 4);
      mbar_init(smem_u32(&sm.pv_done[i]), 1);
    }
    sm.abort = 0;
    *(volatile float*)&sm.minus_zero = -0.f;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // The launch may begin before what is before it on the stream has ended; nothing in memory is touched until then.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tmem_before();
  const int n_tiles = *s.tiles_there;
  auto weight = [&](int x) {
    const int n = s.tiles[x].items;
    return n ? n + kUnitCost : 0;
  };
  const Place pl = locate(
      n_tiles, sm.scratch, [&](int x, bool) { return (int64_t)weight(x); },
      [&](int64_t total) { return share_start(total, cta, ctas); });
  __syncthreads();
  tmem_after();
  const uint32_t tmem = sm.tmem;
  bool ok = true;
  uint32_t task = 0;   // tasks so far
  uint32_t step = 0;   // steps so far, of all tasks: stage step % kStages
  auto stage_of = [&](uint32_t n) { return n % kStages; };
  auto turn_of = [&](uint32_t n) { return n / kStages & 1; };
  auto next = [&]() {  // the next task is there and is not the end
    warp_wait(ok, smem_u32(&sm.task_full[task % kTasks]), task / kTasks & 1, abort, a.err);
    return ok && sm.tasks[task % kTasks].from < sm.tasks[task % kTasks].to;
  };
  auto done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.task_empty[task % kTasks]));
    ++task;
  };

  // Registers: 512 threads x 128 at launch = 256 x 168 + 256 x 80, and some.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  }
  if (warp < 8) {
    // ------------------------------ softmax, a token a thread ------------------------------
    const int grp = warp >> 2, quad = warp & 3, token = quad * 32 + lane, half = quad >> 1;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t S0 = lanes + kColS + grp * 128, O = lanes + kColO + grp * 128;
    const uint32_t weights = sp + grp * kWeightBytes;
    WarpRows& my = sm.rows[warp];
    uint32_t phase = 0;  // this group's steps so far
    const uint64_t zero2 = twice(*(volatile float*)&sm.minus_zero);
    auto group_any = [&](bool x) {
      int any;
      asm volatile(
          "{\n\t.reg .pred p, r;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.or.pred r, %2, 128, p;\n\tselp.s32 %0, 1, 0, r;\n\t}"
          : "=r"(any)
          : "r"((int)x), "r"(2 + grp)
          : "memory");
      return any != 0;
    };
    auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(2 + grp) : "memory"); };
    auto both_sync = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    auto both_well = [&](bool well) {  // no warp is left alone at a barrier
      int all;
      asm volatile(
          "{\n\t.reg .pred p, r;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.and.pred r, 1, 256, p;\n\tselp.s32 %0, 1, 0, r;\n\t}"
          : "=r"(all)
          : "r"((int)well)
          : "memory");
      return all != 0;
    };
    for (;;) {
      const bool more = next();
      if (ok) warp_wait(ok, smem_u32(&sm.q_full[task % kTasks]), task / kTasks & 1, abort, a.err);
      ok = both_well(ok);
      if (!ok || !more) break;
      const Task& x = sm.tasks[task % kTasks];
      const float* qs = sm.qs[task % kTasks];
      const int steps = task_steps(x), rows_there = x.t.tokens * a.G;
      const bool has_tail = x.to > x.t.listed;
      const float my_qs = qs[lane];
      uint64_t l[16];  // softmax sums of the thread's own tokens, rows two by two
#pragma unroll
      for (int i = 0; i < 16; ++i) l[i] = 0;
      // Lane r of every warp has row r's reference: a score, without the query's factor, and kShift - log2 of its values' scale.
      float M = 0.f, w = 0.f;
      uint32_t seen = 0;    // rows that have one. Before that exponents are scores, with the values' scale
      uint32_t poison = 0;  // rows that see, here, what makes them NaN
      my.neg_m[lane] = 0.f;
      int mine = 0;  // steps of this group in the task
      for (int n = grp; n < steps; n += 2, ++mine, ++phase) {
        const uint32_t at = step + n, stage = stage_of(at), S = S0 + (phase & 1) * 64;
        {  // (both tries are on their way at once)
          const uint32_t bars[2] = {smem_u32(&sm.s_full[grp][phase & 1]), smem_u32(&sm.full[stage])};
          const bool there = mbar_try(bars[0], phase >> 1 & 1) & mbar_try(bars[1], turn_of(at));
          if (!__all_sync(0xffffffffu, there && ok)) {
            warp_wait(ok, bars[0], phase >> 1 & 1, abort, a.err);
            warp_wait(ok, bars[1], turn_of(at), abort, a.err);
          }
        }
        // The group's last products: done, its weights' place is free and its output at rest.
        auto settled = [&]() {
          if (mine) warp_wait(ok, smem_u32(&sm.pv_done[grp]), (phase - 1) & 1, abort, a.err);
          tmem_after();
        };
        tmem_after();
        const bool tail = has_tail && n == steps - 1;
        const int j = token & (kPart - 1);
        PageMeta me = sm.meta[stage][half];
        if (tail) {
          me.kfac = sm.tail_kfac[stage][j];
          me.vlog = sm.tail_vlog[stage][j];
          me.vinv = token < kPart ? sm.tail_vinv[stage][j] : 0.f;  // a token counts once
          me.pos = x.t.full * kPart;
          me.rows = rows_there < 32 ? (1u << rows_there) - 1u : 0xffffffffu;
          me.bad = sm.tail_bad[stage][0][j] | sm.tail_bad[stage][1][j];
        }
        const float kfac = me.kfac, vlog = me.vlog;
        const uint32_t rows = me.rows;
        const int pos = me.pos + j;
        const int late = pos - x.t.see0 + 1;  // tokens of the tile that do not see it
        uint32_t allowed = late <= 0 ? rows : late < x.t.tokens ? rows & 0xffffffffu << late * a.G : 0u;
        if (!ok) allowed = 0;
        if (me.bad) poison |= allowed;
        const bool own = __any_sync(0xffffffffu, tail || late > 0);  // tokens have factors or masks of their own
        if (tail) {  // both pieces' scores are added, through the weights' place, and put back
          auto place = [&](int r, int tok) { return weights + (r * 128 + tok) * 4; };
          settled();
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {
            uint32_t hi[16], lo[16];
            tmem_load16(S + g * 16, hi);
            tmem_load16(S + 32 + g * 16, lo);
            tmem_loaded();
            settle16(hi);
            settle16(lo);
#pragma unroll
            for (int i = 0; i < 16; ++i) sts32(place(g * 16 + i, token), __float_as_uint(fmaf(__uint_as_float(lo[i]), 0.0625f, __uint_as_float(hi[i]))));
          }
          group_sync();
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              hi[i] = __float_as_uint(fmaf(__uint_as_float(lds32(place(g * 16 + i, j + kPart))), 0.0625f, __uint_as_float(lds32(place(g * 16 + i, j)))));
              lo[i] = 0;
            }
            tmem_store16(S + g * 16, hi);
            tmem_store16(S + 32 + g * 16, lo);
          }
          tmem_stored();
          group_sync();  // before the weights come
        }
        // Scores are multiplied by the page's factor and rounded before a reference is taken off: a product and a sum that
        // follows would be one operation, and the largest score less itself not 0. (zero2 holds them apart.)
        float e[32];  // exponents: (t - M) * qs + (w + vlog)
        for (bool again = false;; again = true) {
          my.w[lane] = rows >> lane & 1 ? w + (tail ? 0.f : vlog) : -INFINITY;
          __syncwarp();
          float top = -INFINITY;
          if (rows == 0) {  // no page: what lies in its place is not looked at
#pragma unroll
            for (int r = 0; r < 32; ++r) e[r] = -INFINITY;
          } else {
            const uint64_t sixteenth = twice(0.0625f), k2 = twice(kfac);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t hi[16], lo[16];
              tmem_load16(S + g * 16, hi);
              tmem_load16(S + 32 + g * 16, lo);
              tmem_loaded();
              settle16(hi);
              settle16(lo);
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                const ulonglong2 m2 = *reinterpret_cast<const ulonglong2*>(my.neg_m + g * 16 + 2 * i);
                const ulonglong2 w2 = *reinterpret_cast<const ulonglong2*>(my.w + g * 16 + 2 * i);
                const ulonglong2 q2 = *reinterpret_cast<const ulonglong2*>(qs + g * 16 + 2 * i);
                auto exponents = [&](int c, uint64_t m, uint64_t q, uint64_t ww, float* y) {
                  const uint64_t t = fma2(fma2(pack2(lo[c], lo[c + 1]), sixteenth, pack2(hi[c], hi[c + 1])), k2, zero2);
                  unpack2(fma2(add2(t, m), q, ww), y[0], y[1]);
                };
                exponents(2 * i, m2.x, q2.x, w2.x, e + g * 16 + 2 * i);
                exponents(2 * i + 2, m2.y, q2.y, w2.y, e + g * 16 + 2 * i + 2);
              }
            }
            if (own) {
#pragma unroll
              for (int r = 0; r < 32; ++r) e[r] = allowed >> r & 1 ? tail ? e[r] + vlog : e[r] : -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < 32; ++r) top = fmaxf(top, e[r]);
          }
          if (again) break;
          const bool news = top > 0.f || (rows & ~seen);
          if (!group_any(news || !ok)) break;
          // A weight has passed 1, or a row has no reference: the rows, and the largest exponent of each. As a rule few threads
          // have one to tell.
          int* most = sm.top[grp];
          if (quad == 0) most[lane] = order_of(-INFINITY);
          settled();
          if (group_any(!ok)) {
            ok = false;
            break;
          }
          if (__any_sync(0xffffffffu, rows & ~seen)) {
#pragma unroll
            for (int r = 0; r < 32; ++r) {
              const int y = __reduce_max_sync(0xffffffffu, order_of(e[r]));
              if (lane == r) atomicMax(most + r, y);
            }
          } else if (top > 0.f) {
#pragma unroll
            for (int r = 0; r < 32; ++r)
              if (e[r] > 0.f) atomicMax(most + r, __float_as_int(e[r]));
          }
          group_sync();
          float passed = float_of(most[lane]), factor = 1.f;
          if (seen >> lane & 1 && !(passed > 0.f)) passed = -INFINITY;
          uint32_t over = __ballot_sync(0xffffffffu, passed != -INFINITY);
          const bool fresh = !(seen >> lane & 1), there = passed != -INFINITY;
          if (__all_sync(0xffffffffu, !there || (fresh ? fabsf(passed) < kFar : passed < 64.f))) {
            if (there && fresh) {
              M = passed / my_qs;  // a power of two
              w = kShift;
              factor = 0.f;
              my.neg_m[lane] = -M;
            } else if (there) {  // by little: the row takes a power of two off
              const float d = ceilf(passed) - kShift;
              factor = pow2(-(int)d);
              w -= d;
            }
            seen |= over;
          } else {
            // A score far from 0, or far above all others: the reference goes to the step's largest score and then, with
            // differences of scores, to the largest values' scale: their sum would lose it.
            auto of_group = [&](auto of) {  // of row `lane`; rows that are not known before are read again
              group_sync();
              if (quad == 0) most[lane] = order_of(-INFINITY);
              group_sync();
#pragma unroll 1
              for (int r = 0; r < 32; ++r) {
                uint32_t hi, lo;
                tmem_load1(S + r, hi);
                tmem_load1(S + 32 + r, lo);
                tmem_loaded();
                asm volatile("" : "+r"(hi), "+r"(lo));
                const float y = of(__fmul_rn(fmaf(__uint_as_float(lo), 0.0625f, __uint_as_float(hi)), kfac), r);
                const int top = __reduce_max_sync(0xffffffffu, order_of(allowed >> r & 1 ? y : -INFINITY));
                if (lane == 0) atomicMax(most + r, top);
              }
              group_sync();
              return float_of(most[lane]);
            };
            const float score = of_group([&](float t, int) { return t; });
            my.neg_m[lane] = -score;
            __syncwarp();
            const float values = of_group([&](float t, int r) { return fmaf(t + my.neg_m[r], qs[r], vlog); });
            const bool raise = score != -INFINITY && (fresh || !(fmaf(score - M, my_qs, values + w) <= 0.f));
            if (raise) {
              factor = fresh ? 0.f : ex2(fmaf(M - score, my_qs, kShift - values - w));
              M = score;
              w = kShift - values;
            }
            my.neg_m[lane] = -M;
            over = __ballot_sync(0xffffffffu, raise);
            seen |= over;
          }
          my.f[lane] = factor;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const ulonglong2 f2 = *reinterpret_cast<const ulonglong2*>(my.f + 2 * i);
            l[i] = mul2(l[i], f2.x);
            l[i + 1] = mul2(l[i + 1], f2.y);
          }
          if (mine) {
#pragma unroll 1
            for (uint32_t left = over; left; left &= left - 1) {
              const int r = __ffs(left) - 1;
              const float f = my.f[r];
              uint32_t y[3];
#pragma unroll
              for (int k = 0; k < 3; ++k) tmem_load1(O + k * 32 + r, y[k]);
              tmem_loaded();
#pragma unroll
              for (int k = 0; k < 3; ++k) {
                asm volatile("" : "+r"(y[k]));
                tmem_store1(O + k * 32 + r, __float_as_uint(__uint_as_float(y[k]) * f));
              }
            }
            tmem_stored();
          }
        }
        if (!ok) continue;
        const uint64_t u2 = twice(me.vinv);
        const __half2 sixteen = __float2half2_rn(16.f), part = __float2half2_rn(tail && token >= kPart ? 0.0625f : 1.f);
        const uint32_t row = weights + token * 128;
        uint32_t piece[2][3][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // four rows
            uint32_t h[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float y0 = ex2(e[g * 16 + 4 * i + 2 * c]), y1 = ex2(e[g * 16 + 4 * i + 2 * c + 1]);
              uint64_t& sum = l[g * 8 + 2 * i + c];
              sum = fma2(pack2(__float_as_uint(y0), __float_as_uint(y1)), u2, sum);
              h[c] = pack_half2(y0, y1);
              if (tail) {
                const __half2 z = __hmul2(*reinterpret_cast<__half2*>(&h[c]), part);
                h[c] = *reinterpret_cast<const uint32_t*>(&z);
              }
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              piece[g][k][i] = __byte_perm(h[0] << 1, h[1] << 1, 0x7531);
              if (k == 2) break;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t cut = h[c] & 0xff80ff80u;
                const __half2 z = __hmul2(__hsub2(*reinterpret_cast<__half2*>(&h[c]), *reinterpret_cast<const __half2*>(&cut)), sixteen);
                h[c] = *reinterpret_cast<const uint32_t*>(&z);
              }
            }
          }
        }
        settled();
        if (!ok) continue;
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int k = 0; k < 3; ++k)
            sts128(row + (((2 * k + g) ^ (token & 7)) << 4), piece[g][k][0], piece[g][k][1], piece[g][k][2], piece[g][k][3]);
        proxy_fence();
        tmem_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[grp]));
      }
      step += steps;

      // ---- the task's end: sums over tokens, then the groups' outputs ----
      if (mine) warp_wait(ok, smem_u32(&sm.pv_done[grp]), (phase - 1) & 1, abort, a.err);
      tmem_after();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float l0, l1;
        unpack2(l[i], l0, l1);
        sts32(weights + (2 * i * 128 + token) * 4, __float_as_uint(l0));
        sts32(weights + ((2 * i + 1) * 128 + token) * 4, __float_as_uint(l1));
      }
      group_sync();
      {
        const int r = token >> 2, part = token & 3;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) sum += __uint_as_float(lds32(weights + (r * 128 + part * 32 + ((k + lane) & 31)) * 4));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (part == 0) sm.sum[grp][r] = sum;
      }
      poison = __reduce_or_sync(0xffffffffu, poison);
      if (lane == 0) sm.poison[grp][quad] = poison;
      if (quad == 0) {
        sm.m[grp][lane] = seen >> lane & 1 ? M * my_qs : -INFINITY;
        sm.w[grp][lane] = w;
      }
      group_sync();  // the sums have been read
#pragma unroll 1
      for (int g = 0; g < 2; ++g) {
        uint32_t p0[16], p1[16], p2[16];
        if (mine && ok) {
          tmem_load16(O + g * 16, p0);
          tmem_load16(O + 32 + g * 16, p1);
          tmem_load16(O + 64 + g * 16, p2);
          tmem_loaded();
          settle16(p0);
          settle16(p1);
          settle16(p2);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float y = fmaf(fmaf(__uint_as_float(p2[i]), 0.0625f, __uint_as_float(p1[i])), 0.0625f, __uint_as_float(p0[i]));
          sts32(weights + ((g * 16 + i) * 128 + token) * 4, mine && ok ? __float_as_uint(y) : 0u);
        }
      }
      both_sync();
      if (grp == 0) {
        const bool whole = x.from == 0 && x.to == x.t.items;
        // Lane r has row r's factors and place. 2^(M - w) is the unit of a group's numbers: differences of scores first.
        const float m0 = sm.m[0][lane], m1 = sm.m[1][lane], top = fmaxf(m0, m1), at = top == -INFINITY ? 0.f : top;
        const float e0 = m0 == -INFINITY ? m0 : (m0 - at) - sm.w[0][lane], e1 = m1 == -INFINITY ? m1 : (m1 - at) - sm.w[1][lane];
        const float most = top == -INFINITY ? 0.f : fmaxf(e0, e1);
        float f0 = ex2(e0 - most), f1 = ex2(e1 - most);
        float L = sm.sum[0][lane] * f0 + sm.sum[1][lane] * f1;
        uint32_t bad = L != 0.f ? sm.wrong[task % kTasks] : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) bad |= sm.poison[0][k] | sm.poison[1][k];
        if (bad >> lane & 1) L = __uint_as_float(0x7fc00000u);
        const float unit = whole ? L == 0.f ? 0.f : 0x1p-8f / L : 0x1p-8f;  // (codes are 256 times their fp16 number)
        f0 *= unit;
        f1 *= unit;
        uint64_t to;
        if (whole) {
          const int i = lane / a.G;
          to = reinterpret_cast<uint64_t>(out.p + (int64_t)(x.t.token0 + i) * out.ts + (int64_t)(x.t.h * a.G + lane - i * a.G) * out.hs);
        } else {
          float* p = partials + ((int64_t)(2 * cta + (x.from == 0 ? 1 : 0)) * kRowsOfTile + lane) * kPartialStride;
          if (quad == 0 && lane < rows_there) *reinterpret_cast<float4*>(p) = make_float4(top, L, most, 0.f);
          to = reinterpret_cast<uint64_t>(p + 4);
        }
#pragma unroll 4
        for (int r = 0; r < rows_there; ++r) {
          const uint32_t at = weights + (r * 128 + token) * 4;
          const float y = __uint_as_float(lds32(at)) * __shfl_sync(0xffffffffu, f0, r) +
                          __uint_as_float(lds32(at + kWeightBytes)) * __shfl_sync(0xffffffffu, f1, r);
          const uint64_t place = __shfl_sync(0xffffffffu, to, r);
          if (!ok) continue;
          if (whole) {
            const __nv_bfloat16 v = __float2bfloat16_rn(y);
            reinterpret_cast<uint16_t*>(place)[token] = *reinterpret_cast<const uint16_t*>(&v);
          } else {
            reinterpret_cast<float*>(place)[token] = y;
          }
        }
      }
      both_sync();  // the other group's output has been read
      done();
    }
  } else if (warp == kProducer) {
    // ------------------------------ pages ------------------------------
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map)) : "memory");
    while (next()) {
      const Task x = sm.tasks[task % kTasks];
      done();
      const Item* items = s.items + place_of(x.t, a.Hkv, topk) + x.from;
      const int pages = task_pages(x);
      Item it;
      float2 sc;
      auto look = [&](int i) {
        it.page = -1;
        if (i < pages) {
          const uint4 v = *reinterpret_cast<const uint4*>(items + i);
          it.page = (int)v.x;
          it.pos = (int)v.y;
          it.rows = v.z;
          sc = *reinterpret_cast<const float2*>(a.scales + 2 * (int64_t)it.page);
        }
      };
      look(lane);
      for (int p0 = 0; p0 < pages; p0 += 32) {
        const Item my = it;
        const float2 my_sc = sc;
        look(p0 + 32 + lane);
        const int n = min(32, pages - p0);
        for (int i = 0; i < n; i += 2, ++step) {
          const uint32_t stage = stage_of(step), full = smem_u32(&sm.full[stage]);
          warp_wait(ok, smem_u32(&sm.empty[stage]), turn_of(step) ^ 1, abort, a.err);
          if (!ok) break;
          const int c = lane - i;
          if (c == 0 || c == 1) {
            PageMeta& me = sm.meta[stage][c];
            const bool there = lane < n, bad = there && (my_sc.x != my_sc.x || my_sc.y != my_sc.y);
            me.kfac = !there || bad ? 0.f : my_sc.x * scale * kLog2e;
            me.bad = bad;
            me.vlog = !there || bad ? 0.f : scale_log2(my_sc.y);
            me.vinv = !there || bad ? 1.f : 1.f / my_sc.y;
            me.pos = there ? my.pos : 0;
            me.rows = there ? my.rows : 0u;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_expect_tx(full, i + 1 < n ? 2 * kKv8PageBytes : kKv8PageBytes);
            mbar_arrive(full);
          }
          __syncwarp();
          if ((c == 0 || c == 1) && lane < n) {
            const uint32_t to = ring + stage * kStageBytes + c * kKv8HalfBytes;
            tma_half(to, &map, my.page, 0, full);
            tma_half(to + kKv8PageBytes, &map, my.page, 1, full);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (!ok) break;
      if (x.to > x.t.listed) {  // the tail warps, which pass over all other stages, must not take an earlier turn of one for theirs
        const uint32_t stage = stage_of(step);
        warp_wait(ok, smem_u32(&sm.empty[stage]), turn_of(step) ^ 1, abort, a.err);
        if (!ok) break;
        if (lane == 0) mbar_arrive(smem_u32(&sm.tail_go[stage]));
        ++step;
      }
    }
    // What was copied last has landed before the CTA's shared memory goes: the products wait for it, unless a wait ran out.
  } else if (warp == kMmaWarp) {
    // ------------------------------ products ------------------------------
    const uint32_t leader = elect();
    const uint64_t dring = operand(ring, 16, 1024), dq = operand(sq, 16, 1024), dp = operand(sp, 16, 1024);
    uint32_t outs[2] = {0, 0}, ins[2] = {0, 0};  // steps of each group so far, by their outputs and by their scores
    while (next()) {
      const Task x = sm.tasks[task % kTasks];
      const int pages = task_pages(x), steps = task_steps(x);
      warp_wait(ok, smem_u32(&sm.q_full[task % kTasks]), task / kTasks & 1, abort, a.err);
      // Scores are made three steps ahead: a group's next ones are there when it comes to them.
      for (int n = -3; n < steps; ++n) {
        if (n >= 0) {  // the weights of step n are there, and the place of its scores is free
          const uint32_t g = n & 1, stage = stage_of(step + n);
          warp_wait(ok, smem_u32(&sm.p_full[g]), outs[g]++ & 1, abort, a.err);
          tmem_after();
          if (!ok) break;
          const uint64_t v = dring + ((stage * kStageBytes + kKv8PageBytes) >> 4), p = dp + (g * kWeightBytes >> 4);
          const uint32_t d = tmem + kColO + g * 128;
          const bool one = 2 * n + 1 == pages;  // a page alone
          mma_f8(leader, d, v, p, shape(96, true), n >= 2);
          mma_f8(leader, d, v + (4096 >> 4), p + (4096 >> 4), shape(96, true), 1);
          if (!one) {
            mma_f8(leader, d, v + (8192 >> 4), p + (8192 >> 4), shape(96, true), 1);
            mma_f8(leader, d, v + (12288 >> 4), p + (12288 >> 4), shape(96, true), 1);
          }
          mma_commit(leader, smem_u32(&sm.empty[stage]));
          mma_commit(leader, smem_u32(&sm.pv_done[g]));
        }
        if (n + 3 < steps) {
          const uint32_t at = step + n + 3, stage = stage_of(at), g = (n + 3) & 1, buffer = ins[g]++ & 1;
          warp_wait(ok, smem_u32(&sm.full[stage]), turn_of(at), abort, a.err);
          tmem_after();
          if (!ok) break;
          const uint64_t k = dring + (stage * kStageBytes >> 4), b = dq + ((task & 1) * kQueryBytes >> 4);
          const uint32_t d = tmem + kColS + g * 128 + buffer * 64;
#pragma unroll
          for (int c = 0; c < 4; ++c) mma_f8(leader, d, k + 2 * c, b + 2 * c, shape(64, false), c > 0);
          mma_commit(leader, smem_u32(&sm.s_full[g][buffer]));
          if (n + 4 == steps) mma_commit(leader, smem_u32(&sm.q_empty[task & 1]));
        }
      }
      step += steps;
      done();
    }
    // The last arrivals have landed before the CTA's shared memory goes.
#pragma unroll
    for (int g = 0; g < 2; ++g)
      if (outs[g]) warp_wait(ok, smem_u32(&sm.pv_done[g]), (outs[g] - 1) & 1, abort, a.err);
  } else if (warp == kPlanner) {
    // ------------------------------ plan, and query operands ------------------------------
    JoinRecord open = JoinRecord{};
    int64_t at = share_start(pl.total, cta, ctas), before = pl.before;
    const int64_t stop = share_start(pl.total, cta + 1, ctas);
    int tile = pl.b;
    for (bool more = true; more && ok; ++task) {
      Task x;
      x.from = x.to = 0;
      while (at < stop && tile < n_tiles) {
        const int wgt = weight(tile);
        if (wgt == 0 || at >= before + wgt) {
          before += wgt;
          ++tile;
          continue;
        }
        x.t = s.tiles[tile];
        const int f = (int)(at - before), t = (int)min((int64_t)wgt, f + (stop - at));
        at += t - f;
        x.from = max(0, f - kUnitCost);
        x.to = max(0, t - kUnitCost);
        if (x.from < x.to) break;
      }
      more = x.from < x.to;
      const uint32_t slot = task % kTasks;
      warp_wait(ok, smem_u32(&sm.task_empty[slot]), (task / kTasks & 1) ^ 1, abort, a.err);
      if (!ok) break;
      if (lane == 0) {
        sm.tasks[slot] = x;
        mbar_arrive(smem_u32(&sm.task_full[slot]));
      }
      if (more) warp_wait(ok, smem_u32(&sm.q_empty[task & 1]), (task >> 1 & 1) ^ 1, abort, a.err);
      if (!ok) break;
      const int rows = more ? x.t.tokens * a.G : 0;
      const uint32_t to = sq + (task & 1) * kQueryBytes;
      uint32_t wrong = 0;
#pragma unroll 1
      for (int r0 = 0; more && r0 < kRowsOfTile; r0 += 4) {
        uint2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + i, y = r / a.G;
          v[i] = make_uint2(0, 0);
          if (r < rows)
            v[i] = *reinterpret_cast<const uint2*>(q.p + (int64_t)(x.t.token0 + y) * q.ts + (int64_t)(x.t.h * a.G + r - y * a.G) * q.hs + lane * 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + i;
          uint32_t top = largest_of(v[i]);
          if (top >= 0x7f80u) {  // not finite: the row is NaN if it sees anything
            wrong |= 1u << r;
            v[i] = make_uint2(0, 0);
            top = 0x3f80u;
          }
          const int e = half_exponent(top);
          const float f = pow2(8 - e);
          const float y[4] = {lo_f(v[i].x) * f, hi_f(v[i].x) * f, lo_f(v[i].y) * f, hi_f(v[i].y) * f};
          uint32_t high, low;
          two_pieces(y, high, low);
          const uint32_t place = to + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
          sts32(place, high);
          sts32(place + kRowsOfTile * 128, low);
          if (lane == 0) sm.qs[slot][r] = pow2(e - 8);
        }
      }
      if (lane == 0) sm.wrong[slot] = wrong;
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[slot]));
      if (more && x.from == 0 && x.to < x.t.items) {  // (once at most: the last of the share)
        open.total = pl.total;
        open.parts = share_of(pl.total, before + weight(tile) - 1, ctas) - cta + 1;
        open.row0 = x.t.token0;
        open.n_new = x.t.tokens;
        open.h = x.t.h;
        open.first_row = 0;
      }
    }
    if (lane == 0) records[cta] = open;
  } else if (warp < kTailKeys + 2) {
    // ------------------------------ tails ------------------------------
    const int half = warp - kTailKeys;
    uint32_t gone = 0;  // a bit per stage: the parity of its tails so far
    while (next()) {
      const Task x = sm.tasks[task % kTasks];
      done();
      const int steps = task_steps(x);
      step += steps;
      if (x.to <= x.t.listed) continue;
      const uint32_t at = step - 1, stage = stage_of(at);
      warp_wait(ok, smem_u32(&sm.tail_go[stage]), gone >> stage & 1, abort, a.err);
      if (!ok) break;
      gone ^= 1u << stage;
      const uint32_t to = ring + stage * kStageBytes + half * kKv8PageBytes;
      const uint16_t* src = a.tails + ((int64_t)x.t.b * a.Hkv + x.t.h) * kPageElems + half * kPart * kD + lane * 4;
#pragma unroll 1
      for (int r0 = 0; r0 < kPart; r0 += 4) {
        uint2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = r0 + i < x.t.tail ? *reinterpret_cast<const uint2*>(src + (r0 + i) * kD) : make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + i;
          bool wrong = false;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t& y = k ? v[i].y : v[i].x;
            const bool lo = (y & 0x7f80u) == 0x7f80u, hi = (y & 0x7f800000u) == 0x7f800000u;
            wrong |= lo | hi;
            if (lo) y &= 0xffff0000u;
            if (hi) y &= 0x0000ffffu;
          }
          wrong = __any_sync(0xffffffffu, wrong);
          const int e = half_exponent(largest_of(v[i]));
          const float f = pow2(8 - e);
          const float y[4] = {lo_f(v[i].x) * f, hi_f(v[i].x) * f, lo_f(v[i].y) * f, hi_f(v[i].y) * f};
          uint32_t high, low;
          two_pieces(y, high, low);
          const uint32_t place = to + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
          sts32(place, high);
          sts32(place + kKv8HalfBytes, low);
          if (lane == 0) {
            sm.tail_bad[stage][half][r] = wrong;
            if (half == 0) {
              sm.tail_kfac[stage][r] = scale * kLog2e * pow2(e - 8);
            } else {
              sm.tail_vlog[stage][r] = (float)(e - 8);
              sm.tail_vinv[stage][r] = f;
            }
          }
        }
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.full[stage]));
    }
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  if (warp == kMmaWarp) {
    if (*abort) settle_down();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

int64_t most_tiles(const Kv8Args& a) {
  const int64_t n = a.total_new;
  return (n / tile_tokens(a.G) + (a.B < n ? a.B : n)) * a.Hkv;
}

constexpr int64_t kPartialBytes = (int64_t)2 * kMaxCtas * kRowsOfTile * kPartialStride * 4;

RowsSpace space_of(const Kv8Args& a, void* workspace) {
  RowsSpace s;
  s.tiles_there = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + kRecordBytes + kPartialBytes);
  s.tiles = reinterpret_cast<Tile*>(s.tiles_there + 4);
  s.items = reinterpret_cast<Item*>(s.tiles + most_tiles(a));
  return s;
}

}  // namespace

int64_t kv8_rows_workspace(const Kv8Args& a, int topk) {
  return (int64_t)kRecordBytes + kPartialBytes + 16 + most_tiles(a) * (int64_t)sizeof(Tile) +
         (int64_t)a.total_new * a.Hkv * (topk + 1) * (int64_t)sizeof(Item);
}

cudaError_t launch_kv8_rows(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel, int topk,
                            void* workspace, int sm_count, cudaStream_t st) {
  const RowsSpace s = space_of(a, workspace);
  CUtensorMap map;
  cudaError_t e = kv8_page_map(a, kPart, &map);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kv8_rows_attend, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e == cudaSuccess) e = launch_early(kv8_rows_lists, dim3((unsigned)most_tiles(a)), 32, 0, st, a, out, sel, topk, s);
  if (e != cudaSuccess) return e;
  const int ctas = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  e = launch_early(kv8_rows_attend, dim3((unsigned)ctas), kThreads, kSmemBytes, st, a, map, q, out, scale, topk, s,
                   static_cast<JoinRecord*>(workspace), reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kRecordBytes));
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_kv8_join(a, out, ctas, kRowsOfTile, workspace, kRowsOfTile, st);
}

}  // namespace spin
