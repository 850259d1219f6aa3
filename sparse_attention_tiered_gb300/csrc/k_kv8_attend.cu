// spin_kv8_attend: exact attention over the 8-bit paged cache.
//
// Few rows a unit (single tokens, a few drafted ones) read the whole cache once: 256 bytes a
// token and KV head against 4 * 128 * G flops, far below the tensor cores' rate, so the kernel is
// built to keep the memory busy. One persistent CTA per SM takes an equal share of all pages of
// all units in order (a unit may begin and end inside CTAs' shares). A plan warp walks the share, and
// works out each unit's query operands ahead of their use; a producer warp streams pages into rings
// of 16 KB slots with one TMA copy each; groups of consumer warps take them, four to a page with 16 tokens
// each, every warp with a softmax state and output of its own. Those are joined through shared
// memory at the end of a unit, and over CTAs by a second launch. A unit's tail, whose bf16 rows take
// longest, comes first, under its pages.
//
// Arithmetic. m16n8k16 products on fp16 operands with fp32 sums: tokens x dimensions x rows for the
// scores, dimensions x tokens x rows for the output. Rows are the narrow side, so eight of them, the usual
// group, waste nothing. Codes go to fp16 exactly; queries and tail rows are scaled by a power of two into
// fp16's range. Each 64-token page has scales k and v: with s = score * k * log2(e) and P = 2^((s - M) + (log2(v) - V) + 14),
// the output's weight is P and the softmax sum's is P / v. So blocks whose values differ by any factor share one
// fp16 range, whose 28 binary orders below the largest weight are normal numbers. The reference is a pair, a token's
// s and its log2(v), so that scores may be of any size: s - M is exact near the reference, where s - (M - 14) would be
// rounded to a step of M. It moves only where a weight passes it by more than a factor of 2 (P may reach 2^15), so
// that a page costs one vote in place of a maximum over lanes.
//
// Operand layout. The k index of a product and its two outer ones may be permuted as long as the operands
// agree, which is chosen so that no byte has to move between lanes: a lane's 16-byte chunk of a key row is
// its own k indices of four products, and 16 bytes of a value row its dimensions of 8 products. With the
// copy's 128-byte swizzle and tokens in the order 0 5 2 7 4 1 6 3, all of these 16-byte loads touch every
// bank once. Values need two tokens of one dimension side by side: one byte permutation for two such
// pairs. Weights come out of the first product with a token a lane group and go into the second with a
// row a lane group: an 8 x 8 transposition each.
//
// Measured: 32 requests of 32768 tokens, 8 KV heads in groups of 5: 2.15 GB in 316 us, 6.80 TB/s, what a plain
// copy reaches on this GPU. HBM bounds it; the schedulers issue in 37% of the cycles, the tensor pipe works in
// 17%. With rows as the products' wide side (16 rows' registers and products for 8) it took 352 us. Small calls are
// bound by the chain to the first page (lengths, table, scale, copy): one request of 4096 tokens takes 8.5 us a
// call, 10.3 without the launch that begins while the last one ends.
#include "kv8_dev.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kMostRows = 16;       // of a unit: a token's group, or a few tokens of a small one
constexpr int kUnits = 4;           // announced ahead
constexpr float kShift = 14.f;      // weights reach 2^14, and 2^15 before the reference moves
constexpr float kFar = 2048.f;      // a sum of two exponents is right to 2^-13 below it
constexpr float kNone = -3e38f;     // below all scores, and finite: a hidden token's -inf less this is -inf

// A group is four consumer warps: as many groups as the registers have room for. A ring of 16 KB slots each (a
// tail takes two). For 8 requests of 32768 tokens on 8 heads, 3 groups of 3 slots take 93 us; 4 of 2
// (104 registers a thread) 99, 2 of 5 96, 2 of 4 97.
constexpr int kGroups = 3, kPer = 3, kSlots = kGroups * kPer;
constexpr int kConsWarps = 4 * kGroups, kProducer = kConsWarps, kPlanner = kConsWarps + 1;
constexpr int kThreads = (kConsWarps + 4) * 32;
constexpr size_t kRingBytes = (size_t)kSlots * kKv8PageBytes;
constexpr size_t kJoinBytes = (size_t)kConsWarps * 8 * kD * 4;

struct SlotMeta {
  float kfac;  // score factor: page scale * softmax scale * log2(e); NaN where one of the page's scales is
  float vlog;  // log2 of the values' scale
  float vinv;  // 1 / the values' scale
  int pos0;    // position of its first token; -1: nothing to do
};

// What this CTA does of a unit.
struct Task {
  Unit u;
  int b, h, from, to;  // items [from, to); none: the share is done
};

struct Smem {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t task_full[kUnits], q_full[kUnits], task_empty[kUnits];
  SlotMeta meta[kSlots];
  Task tasks[kUnits];
  float qs[kUnits][kMostRows];   // a row's score factor
  int see[kUnits][kMostRows];    // tokens that a row sees
  int64_t scratch[36];
  float m[kConsWarps][8], v[kConsWarps][8], both[kConsWarps][8], l[kConsWarps][8];
  int abort;
};
constexpr size_t kQueryBytes = (size_t)kUnits * 2 * 8 * 32 * 8;
constexpr size_t kSmemBytes = 1024 + kRingBytes + kJoinBytes + kQueryBytes + sizeof(Smem);
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsWarps * 32) : "memory"); }

// The same, and whether all of them are well.
__device__ __forceinline__ bool consumers_agree(bool ok) {
  int all;
  asm volatile(
      "{\n.reg .pred p, r;\nsetp.ne.s32 p, %1, 0;\nbarrier.cta.red.and.pred r, 1, %2, p;\nselp.s32 %0, 1, 0, r;\n}"
      : "=r"(all)
      : "r"((int)ok), "n"(kConsWarps * 32)
      : "memory");
  return all != 0;
}

// A warp's softmax state. Lane (g, t) has rows 8 r + 2 t and 8 r + 2 t + 1 (index e), and of them dimensions
// 16 g .. 16 g + 15 of the output: 2 j and 2 j + 1 of those are o[r][j][e] and o[r][j][2 + e].
template <int R>
struct State {
  float o[R][8][4];
  float m[R][2], w[R][2];  // the reference: a score (kNone: nothing seen yet), and kShift - log2 of its values' scale
  float l[R][2];           // of the lane's own tokens
};

// The transposed 8 x 8 matrix of 16-bit elements.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Takes the lane's scores z (of its rows: tokens g, g, g + 8, g + 8 in the permuted order, e alternating) into
// the state; fp16 weights come out, p[r] for the tokens' halves. vlog, vinv: of the values' scale.
template <int R>
__device__ __forceinline__ void softmax_step(State<R>& st, const float (&z)[R][4], float vlog, float vinv, uint32_t (&p)[R][2]) {
  float x[R][4];  // exponents
  for (float most = kShift + 1.f;; most = INFINITY) {  // twice at most: nothing is above the second limit
    float top = -INFINITY;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[r][e] = (z[r][e] - st.m[r][e & 1]) + (vlog + st.w[r][e & 1]);
        top = fmaxf(top, x[r][e]);
      }
    if (!__any_sync(0xffffffffu, top > most)) break;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float score = fmaxf(z[r][e], z[r][2 + e]);
        score = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, 4));
        score = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, 8));
        score = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, 16));
        const float above = (score - st.m[r][e]) + (vlog + st.w[r][e]);
        float f = 1.f;
        if (above > kShift) {
          f = ex2(kShift - above);
          st.m[r][e] = score;
          st.w[r][e] = kShift - vlog;
        }
        st.l[r][e] *= f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          st.o[r][j][e] *= f;
          st.o[r][j][2 + e] *= f;
        }
      }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = ex2(x[r][e]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float s = y[e] + y[2 + e];
      st.l[r][e] += s == 0.f ? 0.f : s * vinv;  // a row that sees nothing here takes nothing of a NaN page
    }
    p[r][0] = transposed(pack_half2(y[0], y[1]));
    p[r][1] = transposed(pack_half2(y[2], y[3]));
  }
}

// z = score * factor for the tokens a row may see, else -inf. `tok`: position of the lane's first token.
template <int R>
__device__ __forceinline__ void finish_scores(float (&z)[R][4], const float2 (&qs)[R], float kfac, bool masked, int tok,
                                              const int* see) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float& x = z[r][e];
      x = __fmul_rn(x, kfac * (e & 1 ? qs[r].y : qs[r].x));  // rounded before the reference is taken off
    }
  if (masked) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int2 s = *reinterpret_cast<const int2*>(see + 8 * r);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (tok + (e >> 1) * 8 >= (e & 1 ? s.y : s.x)) z[r][e] = -INFINITY;
    }
  }
}

// Clears what is not finite of eight bf16; whether there was any; the largest of the others, folded into `top`.
__device__ __forceinline__ bool clean(uint4& w, uint32_t& top) {
  uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
  bool wrong = false;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const bool lo = (ww[y] & 0x7f80u) == 0x7f80u, hi = (ww[y] & 0x7f800000u) == 0x7f800000u;
    wrong |= lo | hi;
    if (lo) ww[y] &= 0xffff0000u;
    if (hi) ww[y] &= 0x0000ffffu;
    top = __vmaxu2(top, ww[y] & 0x7fff7fffu);
  }
  return wrong;
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1)
kv8_decode_kernel(const Kv8Args a, const __grid_constant__ CUtensorMap map, const Rows q, const Rows out, float scale,
                  const int32_t* sel, int topk, JoinRecord* records, float* partials) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* join = reinterpret_cast<float*>(ring + kRingBytes);                 // [warps][8 rows][128]
  uint2* queries = reinterpret_cast<uint2*>(ring + kRingBytes + kJoinBytes);  // [kUnits][R][8][32]
  Smem& sm = *reinterpret_cast<Smem*>(ring + kRingBytes + kJoinBytes + kQueryBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kRows = 8 * R;
  volatile int* abort = &sm.abort;

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 4);
    }
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(smem_u32(&sm.task_full[s]), 1);
      mbar_init(smem_u32(&sm.q_full[s]), 1);
      mbar_init(smem_u32(&sm.task_empty[s]), kConsWarps + 1);
    }
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // The launch may begin before what is before it on the stream has ended; nothing in memory is touched until then.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ctas = gridDim.x, cta = blockIdx.x;
  const Place pl = locate(
      a.B, sm.scratch, [&](int x, bool first) { return (int64_t)unit_of(a, x, 0, kRows, topk, cta == 0 && first).weight * a.Hkv; },
      [&](int64_t total) { return share_start(total, cta, ctas); });
  bool ok = true;
  uint32_t task = 0;  // units of the share so far

  // Registers: 512 threads x 128 at launch = 128 x 56 + 384 x 152.
  if (warp >= kConsWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kPlanner) {
      // ------------------------------ plan, and query operands ------------------------------
      const int g = lane >> 2, t = lane & 3;
      JoinRecord open = JoinRecord{};
      Task x = Task{};
      x.b = pl.b;
      int64_t at = share_start(pl.total, cta, ctas), before = pl.before;
      const int64_t stop = share_start(pl.total, cta + 1, ctas);
      for (bool more = true; more && ok; ++task) {
        x.from = x.to = 0;
        while (at < stop && x.b < a.B) {
          x.u = unit_of(a, x.b, 0, kRows, topk, false);
          if (x.u.weight == 0 || at >= before + (int64_t)x.u.weight * a.Hkv) {
            before += (int64_t)x.u.weight * a.Hkv;
            ++x.b;
            continue;
          }
          const Part p = part_of(x.u, at - before, stop - at);
          at += p.took;
          if (p.from >= p.to) continue;
          x.h = p.h;
          x.from = p.from;
          x.to = p.to;
          break;
        }
        more = x.from < x.to;
        const uint32_t slot = task % kUnits;
        warp_wait(ok, smem_u32(&sm.task_empty[slot]), (task / kUnits & 1) ^ 1, abort, a.err);
        if (!ok) break;
        if (lane == 0) {
          sm.tasks[slot] = x;
          mbar_arrive(smem_u32(&sm.task_full[slot]));
        }
        // Queries as the products want them: lane (g, t) holds dimensions 16 t .. and 64 + 16 t .. of its rows, four
        // to a product, scaled by a power of two into fp16's range.
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int row = r * 8 + g, i = row / a.G, head = x.h * a.G + row - i * a.G;
          const bool there = more && row < x.u.n_new * a.G;
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = 0;
          if (there) {
            const uint4* src = reinterpret_cast<const uint4*>(q.p + (int64_t)(x.u.row0 + i) * q.ts + (int64_t)head * q.hs);
#pragma unroll
            for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(w + 4 * k) = src[(k >> 1) * 8 + 2 * t + (k & 1)];
          }
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < 16; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
          top = max(top & 0xffffu, top >> 16);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = half_exponent(top);
          const float f = pow2(15 - e);
          if (t == 0) {
            sm.qs[slot][row] = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2(e - 15);
            sm.see[slot][row] = there ? x.u.past + i + 1 : 0;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            queries[((slot * R + r) * 8 + k) * 32 + lane] = make_uint2(pack_half2(lo_f(w[2 * k]) * f, hi_f(w[2 * k]) * f),
                                                                       pack_half2(lo_f(w[2 * k + 1]) * f, hi_f(w[2 * k + 1]) * f));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[slot]));
        if (more && x.from == 0 && x.to < x.u.items)  // (once at most: the last of the share)
          open = record_of(x.u, x.h, 0, pl.total, before + (int64_t)(x.h + 1) * x.u.weight, cta, ctas);
      }
      if (lane == 0) records[cta] = open;
      return;
    }
    if (warp != kProducer) return;

    // ------------------------------ producer ------------------------------
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map)) : "memory");
    // Items go to the groups in turn, each with a ring of its own: next[0] is the next slot of the group
    // whose turn it is, with the ring's parity above bit 8. (In one ring for all, a group could reach a
    // slot whose last copy, another group's, had not landed yet, and take that phase for its own.)
    uint32_t next[kGroups];
#pragma unroll
    for (int x = 0; x < kGroups; ++x) next[x] = x * kPer;
    auto step = [&]() {
      const uint32_t s = next[0] & 255u, p = next[0] >> 8;
      next[0] = s % kPer == kPer - 1 ? (s - (kPer - 1)) | (p ^ 1) << 8 : s + 1 | p << 8;
    };
    auto pass = [&]() {
      const uint32_t first = next[0];
#pragma unroll
      for (int x = 0; x + 1 < kGroups; ++x) next[x] = next[x + 1];
      next[kGroups - 1] = first;
    };
    for (;; ++task) {
      warp_wait(ok, smem_u32(&sm.task_full[task % kUnits]), task / kUnits & 1, abort, a.err);
      if (!ok) break;
      const Task x = sm.tasks[task % kUnits];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.task_empty[task % kUnits]));
      if (x.from >= x.to) break;
      const int64_t unit = (int64_t)x.b * a.Hkv + x.h;
      const int tail_items = x.u.items - x.u.pages;  // the tail is item 0
      int p0 = max(0, x.from - tail_items);
      const int p1 = x.to - tail_items;
      // 32 page ids and scales at a time, a batch ahead of the copies
      int id = -1, pos = -1;
      float2 sc = make_float2(1.f, 1.f);
      auto look = [&](int i) {
        id = pos = -1;
        if (i < p1) {
          const int p = topk ? sel[unit * topk + i] : i;
          if (p >= 0 && p < x.u.full) {
            id = a.table[unit * a.max_pages + p];
            if (id < 0 || (int64_t)id >= a.n_pages) {
              atomicOr(a.err, (uint32_t)kErrIndex);
              id = -1;
            } else {
              pos = p * kPart;
              sc = *reinterpret_cast<const float2*>(a.scales + 2 * (int64_t)id);
            }
          }
        }
      };
      look(p0 + lane);
      if (x.from < tail_items) {  // the tail: keys in one slot, values in the next
        for (int i = 0; i < 2; ++i) {
          const uint32_t slot = next[0] & 255u, parity = next[0] >> 8;
          if (lane == 0) {
            const uint32_t full = smem_u32(&sm.full[slot]);
            const uint32_t bytes = x.u.tail * kD * 2;
            ok = ok && mbar_wait(smem_u32(&sm.empty[slot]), parity ^ 1, abort, a.err);
            if (ok) {
              bulk_copy(smem_u32(ring) + slot * kKv8PageBytes, a.tails + unit * kPageElems + i * kPart * kD, bytes, full);
              sm.meta[slot] = SlotMeta{scale * kLog2e, 0.f, 1.f, x.u.full * kPart};
              mbar_arrive_expect_tx(full, bytes);
            }
          }
          __syncwarp();
          step();
        }
        pass();
        ok = __all_sync(0xffffffffu, ok);
      }
      for (; p0 < p1; p0 += 32) {
        const int my_id = id, my_pos = pos;
        const float2 my_sc = sc;
        look(p0 + 32 + lane);
        const int n = min(32, p1 - p0);
        for (int i = 0; i < n; ++i) {
          const uint32_t slot = next[0] & 255u, parity = next[0] >> 8;
          if (lane == i) {
            const uint32_t full = smem_u32(&sm.full[slot]);
            ok = ok && mbar_wait(smem_u32(&sm.empty[slot]), parity ^ 1, abort, a.err);
            if (ok) {
              if (my_id >= 0) tma_page(smem_u32(ring) + slot * kKv8PageBytes, &map, my_id, full);
              const bool bad = my_sc.x != my_sc.x || my_sc.y != my_sc.y;  // (a hidden token's -inf stays: it is set later)
              sm.meta[slot] = SlotMeta{bad ? __uint_as_float(0x7fc00000u) : my_sc.x * scale * kLog2e, bad ? 0.f : scale_log2(my_sc.y),
                                       bad ? 1.f : 1.f / my_sc.y, my_pos};
              mbar_arrive_expect_tx(full, my_id >= 0 ? kKv8PageBytes : 0);
            }
          }
          __syncwarp();  // slots are filled in order: a lane that ran ahead would take a phase for a later one
          step();
          pass();
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    // No copy may be in flight when the CTA's shared memory goes. The consumers wait for every slot
    // that was filled, unless a wait ran out.
    if (lane == 0 && !ok) settle_down();
    return;
  }

  // ------------------------------ consumers ------------------------------
  asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
  const int g = lane >> 2, t = lane & 3;
  const int group = warp >> 2, quarter = warp & 3;
  const int pg = (g & 1) ? g ^ 4 : g;        // token order 0 5 2 7 4 1 6 3
  State<R> st;
  uint32_t slot = group * kPer, parity = 0;  // of the group's own ring
  auto step = [&]() {
    if (++slot == (group + 1) * kPer) slot = group * kPer, parity ^= 1;
  };
  int turn = 0;
  for (;; ++task) {
    const uint32_t ts = task % kUnits;
    warp_wait(ok, smem_u32(&sm.q_full[ts]), task / kUnits & 1, abort, a.err);
    ok = consumers_agree(ok);  // no warp is left alone at the barriers below; and the join area is free again
    if (!ok) break;
    const Task& x = sm.tasks[ts];
    const int from = x.from, to = x.to;
    if (from >= to) break;
    const int tail_items = x.u.items - x.u.pages, past = x.u.past;
    float2 qs[R];
    const int* see = &sm.see[ts][2 * t];  // rows 8 r, and the next
#pragma unroll
    for (int r = 0; r < R; ++r) {
      qs[r] = *reinterpret_cast<const float2*>(&sm.qs[ts][8 * r + 2 * t]);
    }
    auto query = [&](int r, int k) -> uint2 { return queries[((ts * R + r) * 8 + k) * 32 + lane]; };
#pragma unroll
    for (int r = 0; r < R; ++r) {
      st.m[r][0] = st.m[r][1] = kNone;
      st.w[r][0] = st.w[r][1] = kShift;
      st.l[r][0] = st.l[r][1] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) st.o[r][j][0] = st.o[r][j][1] = st.o[r][j][2] = st.o[r][j][3] = 0.f;
    }

    for (int it = from; it < to; ++it, turn = turn + 1 == kGroups ? 0 : turn + 1) {
      if (turn != group) continue;
      if (it >= tail_items) {
        warp_wait(ok, smem_u32(&sm.full[slot]), parity, abort, a.err);
        const SlotMeta me = sm.meta[slot];
        if (ok && me.pos0 >= 0) {
          const uint32_t keys = smem_u32(ring) + slot * kKv8PageBytes + quarter * 16 * kD;
          const uint32_t vals = keys + kKv8HalfBytes;
          uint4 kr[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = keys + (i * 8 + pg) * kD;
            kr[i][0] = lds128(at + ((t ^ pg) << 4));
            kr[i][1] = lds128(at + (((t + 4) ^ pg) << 4));
          }
          float z[R][4], z1[R][4];  // even and odd products apart: shorter chains
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[r][e] = z1[r][e] = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t w0 = reinterpret_cast<const uint32_t*>(&kr[0][k >> 2])[k & 3];
            const uint32_t w1 = reinterpret_cast<const uint32_t*>(&kr[1][k >> 2])[k & 3];
            const uint4 keys4 = make_uint4(e4m3x2_half2(w0, false), e4m3x2_half2(w1, false), e4m3x2_half2(w0, true), e4m3x2_half2(w1, true));
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const uint2 b = query(r, k);
              mma_f16(k & 1 ? z1[r] : z[r], keys4, b.x, b.y);
            }
          }
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[r][e] += z1[r][e];
          uint4 vr[4];  // value rows 2 t, (2 t) ^ 5, and those 8 further
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = (x & 1) ? (2 * t) ^ 5 : 2 * t;
            vr[x] = lds128(vals + ((x >> 1) * 8 + row) * kD + ((g ^ row) << 4));
          }
          finish_scores<R>(z, qs, me.kfac, me.pos0 + kPart > past + 1, me.pos0 + quarter * 16 + pg, see);
          uint32_t p[R][2];
          softmax_step<R>(st, z, me.vlog, me.vinv, p);
          const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vr[0]);
          const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vr[1]);
          const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vr[2]);
          const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vr[3]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {  // dimensions 4 x + 2 y, 4 x + 2 y + 1 of the lane's 16
              const uint32_t lo = __byte_perm(v0[x], v1[x], y ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(v2[x], v3[x], y ? 0x7362 : 0x5140);
              const uint4 vals4 = make_uint4(e4m3x2_half2(lo, false), e4m3x2_half2(lo, true), e4m3x2_half2(hi, false), e4m3x2_half2(hi, true));
#pragma unroll
              for (int r = 0; r < R; ++r) mma_f16(st.o[r][2 * x + y], vals4, p[r][0], p[r][1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
        step();
        continue;
      }
      // The tail. Rows are bf16; each warp scales its 16 tokens' keys, and values, by a power of two.
      const uint32_t s0 = slot;
      warp_wait(ok, smem_u32(&sm.full[slot]), parity, abort, a.err);
      step();
      warp_wait(ok, smem_u32(&sm.full[slot]), parity, abort, a.err);
      const SlotMeta me = sm.meta[s0];
      const int have = x.u.tail - quarter * 16;  // of this warp's tokens
      if (ok && have > 0) {
        const uint32_t keys = smem_u32(ring) + s0 * kKv8PageBytes + quarter * 16 * kD * 2;
        const uint32_t vals = smem_u32(ring) + slot * kKv8PageBytes + quarter * 16 * kD * 2;
        bool bad[2];  // the lane's tokens that hold something not finite
        // keys: per token tile, 16 + 16 dimensions of the lane's token
        uint4 kr[2][4];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          bool wrong = false;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            kr[i][x] = make_uint4(0, 0, 0, 0);
            if (i * 8 + pg < have) kr[i][x] = lds128(keys + (i * 8 + pg) * kD * 2 + ((x >> 1) * 8 + 2 * t + (x & 1)) * 16);
            wrong |= clean(kr[i][x], top);
          }
          bad[i] = (__ballot_sync(0xffffffffu, wrong) >> (4 * g) & 0xfu) != 0;
        }
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const int ke = half_exponent(top);
        const float kf = pow2(15 - ke);
        float z[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) z[r][0] = z[r][1] = z[r][2] = z[r][3] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t w[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t x = reinterpret_cast<const uint32_t*>(&kr[i][k >> 1])[(k & 1) * 2 + y];
              w[i][y] = pack_half2(lo_f(x) * kf, hi_f(x) * kf);
            }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint2 b = query(r, k);
            mma_f16(z[r], make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]), b.x, b.y);
          }
        }
        // values: four tokens' 16 dimensions
        uint4 vr[4][2];
        top = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = (x >> 1) * 8 + ((x & 1) ? (2 * t) ^ 5 : 2 * t);
          bool wrong = false;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            vr[x][y] = make_uint4(0, 0, 0, 0);
            if (row < have) vr[x][y] = lds128(vals + row * kD * 2 + (2 * g + y) * 16);
            wrong |= clean(vr[x][y], top);
          }
          const uint32_t who = __ballot_sync(0xffffffffu, wrong);
          if ((x & 1) == (g & 1)) bad[x >> 1] |= (who & 0x11111111u << (g >> 1)) != 0;
        }
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const int ve = half_exponent(top);
        const float vf = pow2(15 - ve);
        finish_scores<R>(z, qs, me.kfac * pow2(ke - 15), true, me.pos0 + quarter * 16 + pg, see);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (bad[e >> 1] && z[r][e] != -INFINITY) z[r][e] = __uint_as_float(0x7fc00000u);
        uint32_t p[R][2];
        softmax_step<R>(st, z, (float)(ve - 15), vf, p);
#pragma unroll
        for (int y = 0; y < 8; ++y) {  // words of two dimensions
          const uint32_t w0 = reinterpret_cast<const uint32_t*>(&vr[0][y >> 2])[y & 3];
          const uint32_t w1 = reinterpret_cast<const uint32_t*>(&vr[1][y >> 2])[y & 3];
          const uint32_t w2 = reinterpret_cast<const uint32_t*>(&vr[2][y >> 2])[y & 3];
          const uint32_t w3 = reinterpret_cast<const uint32_t*>(&vr[3][y >> 2])[y & 3];
          const uint4 vals4 = make_uint4(pack_half2(lo_f(w0) * vf, lo_f(w1) * vf), pack_half2(hi_f(w0) * vf, hi_f(w1) * vf),
                                         pack_half2(lo_f(w2) * vf, lo_f(w3) * vf), pack_half2(hi_f(w2) * vf, hi_f(w3) * vf));
#pragma unroll
          for (int r = 0; r < R; ++r) mma_f16(st.o[r][y], vals4, p[r][0], p[r][1]);
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&sm.empty[s0]));
        mbar_arrive(smem_u32(&sm.empty[slot]));
      }
      step();
    }

    // ---- the unit's part of this CTA is done: join the warps' states, 8 rows at a time ----
    const bool whole = from == 0 && to == x.u.items;
    const int row0 = x.u.row0, h = x.h, rows = x.u.n_new * a.G;
    const int pslot = 2 * cta + (from == 0 ? 1 : 0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r * 8 >= rows) break;
      if (r) consumers_sync();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.l[r][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) {
          const float v = kShift - st.w[r][e];
          sm.m[warp][2 * t + e] = st.m[r][e];
          sm.v[warp][2 * t + e] = v;
          sm.both[warp][2 * t + e] = st.m[r][e] + v;
          sm.l[warp][2 * t + e] = l;
        }
        // chunk c of four dimensions of row x lies at c ^ (x >> 1)
        float* dst = join + (warp * 8 + 2 * t + e) * kD;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(dst + ((4 * g + i) ^ t) * 4) =
              make_float4(st.o[r][2 * i][e], st.o[r][2 * i][2 + e], st.o[r][2 * i + 1][e], st.o[r][2 * i + 1][2 + e]);
      }
      consumers_sync();
      const int d0 = lane * 4, row = r * 8 + warp;  // a warp a row, four dimensions a lane
      if (warp < 8 && row < rows) {
        float rel[kConsWarps], M = -INFINITY, V = 0.f;
#pragma unroll
        for (int w = 0; w < kConsWarps; ++w) {
          rel[w] = sm.both[w][warp];
          M = fmaxf(M, rel[w]);
        }
        float base = M;
        if (fabsf(M) >= kFar) {  // differences of scores first
          M = V = -INFINITY;
#pragma unroll
          for (int w = 0; w < kConsWarps; ++w) M = fmaxf(M, sm.m[w][warp]);
#pragma unroll
          for (int w = 0; w < kConsWarps; ++w) {
            rel[w] = (sm.m[w][warp] - M) + sm.v[w][warp];
            V = fmaxf(V, rel[w]);
          }
          base = V;
        }
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kConsWarps; ++w) {
          const float f = ex2(rel[w] - base);
          L += sm.l[w][warp] * f;
          const float4 y = *reinterpret_cast<const float4*>(join + (w * 8 + warp) * kD + (lane ^ (warp >> 1)) * 4);
          o = make_float4(o.x + y.x * f, o.y + y.y * f, o.z + y.z * f, o.w + y.w * f);
        }
        if (whole) {
          const int i = row / a.G, head = h * a.G + row - i * a.G;
          const float inv = L == 0.f ? 0.f : 1.f / L;
          const __nv_bfloat162 v0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), v1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
          *reinterpret_cast<uint2*>(out.p + (int64_t)(row0 + i) * out.ts + (int64_t)head * out.hs + d0) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
        } else {
          float* part = partials + ((int64_t)pslot * kMostRows + row) * kPartialStride;
          if (lane == 0) *reinterpret_cast<float4*>(part) = make_float4(M, L, V, 0.f);
          *reinterpret_cast<float4*>(part + 4 + d0) = o;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.task_empty[ts]));
  }
  // The producer may have left before the wait ran out, with its last copies still in flight.
  if (!ok) settle_down();
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// The pool as [n_pages][128 rows][128 bytes], a box of one page.
cudaError_t page_map(const Kv8Args& a, CUtensorMap* m) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorSymbolNotFound;
  const cuuint64_t dims[3] = {kD, 2 * kPart, (cuuint64_t)a.n_pages};
  const cuuint64_t strides[2] = {kD, kKv8PageBytes};
  const cuuint32_t box[3] = {kD, 2 * kPart, 1}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.pages, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int R>
cudaError_t launch_decode(const Kv8Args& a, const CUtensorMap& map, const Rows& q, const Rows& out, float scale,
                          const int32_t* sel, int topk, void* workspace, int sm_count, cudaStream_t st) {
  const int ctas = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  cudaError_t e = cudaFuncSetAttribute(kv8_decode_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_early(kv8_decode_kernel<R>, dim3((unsigned)ctas), kThreads, kSmemBytes, st, a, map, q, out, scale, sel, topk,
                   static_cast<JoinRecord*>(workspace), reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kRecordBytes));
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_kv8_join(a, out, ctas, a.max_new * a.G, workspace, kMostRows, st);
}

}  // namespace

int64_t kv8_attend_workspace(const Kv8Args&) {
  const int64_t few = (int64_t)2 * kMaxCtas * kMostRows * kPartialStride * 4, many = kv8_prefill_workspace();
  return (int64_t)kRecordBytes + (few > many ? few : many);
}

cudaError_t launch_kv8_attend(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel,
                              int topk, void* workspace, int sm_count, cudaStream_t st) {
  const int64_t rows = (int64_t)a.max_new * a.G;  // of a unit, at most
  if (rows > kMostRows) return launch_kv8_prefill(a, q, out, scale, sel, topk, workspace, sm_count, st);
  CUtensorMap map;
  const cudaError_t e = page_map(a, &map);
  if (e != cudaSuccess) return e;
  return rows <= 8 ? launch_decode<1>(a, map, q, out, scale, sel, topk, workspace, sm_count, st)
                   : launch_decode<2>(a, map, q, out, scale, sel, topk, workspace, sm_count, st);
}

}  // namespace spin
