// Attention of blocks of rows over their lists of pages, for spin_kv8_attend_rows.
//
// A block has up to 256 rows of one head, two tiles of 128, and each tile a list of its own: the pages that any of its
// tokens lists, with a bit per token. (Neighbouring tokens list much the same pages: 16 tokens with 32 pages each list 72 to
// 135 between them where a token keeps 0.98 or 0.9 of the last one's likes, and 320 of 480 where it keeps nothing; 32
// tokens 99, 209 and 427.) A step takes one page for each tile. A block of at most 128 rows is held by both tiles,
// which take its pages in turn; tile 1's result is joined to tile 0's through shared memory at the end.
//
// As in the many-row kernel, whose arithmetic this is, products are tcgen05.mma on fp16 operands with fp32 accumulators in
// tensor memory, with Q and the pages' K and V in shared memory as fp16:
//   S_t[128 x 64] = Q_t K_t^T, 8 products of depth 16, and O_t[128 x 128] += P_t V_t, 4 products, P_t in S_t's place.
// A chain of 8 products on one accumulator takes 760 clocks however few columns it has, so a tile has two places for scores, and
// those of the step after next are made under a step's softmax. (A tile may so be done with two steps before the products'
// warp has looked for the first: what is done has a barrier for each place.)
// Roles, by warp: 0-3, 4-7 softmax of tile 0 and 1, a row a thread; 8-11 keys to fp16 in shared memory; 12-15 values; 16 the
// products; 17 walks the CTA's share of the work. A loader warp copies its 2 KB of a step's pages to shared memory in bulk, takes
// them into registers as soon as they are there, and has the next step's under way while it waits, converts and stores.
//
// A step of two pages takes some 2,350 clocks where nothing else is in the way (96 more pages a tile on 512 blocks of 152 CTAs:
// 400 us). The products alone take 1,430; what bounds it is the shared memory, 256 KB a step at 128 bytes a clock: Q for the
// scores 64 KB, K and V for the products 64, their stores 64, the codes in and out 64. (Conversions made several times
// cheaper change nothing. With loads straight into registers the chunk of 2048 tokens onto 30000 takes the same 514 us, and five
// drafts of 16 requests, whose pages come from HBM, 79 us instead of 70.)
#include <type_traits>

#include "kv8_rows.cuh"
#include "kv8_tc.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kTile = kTileRows;
constexpr int kBlockRows = 2 * kTile;
constexpr int kThreads = 640;
constexpr int kKeyWarp = 8, kValueWarp = 12, kMmaWarp = 16, kPlanWarp = 17;
constexpr int kSegReaders = 17;      // warps that read a segment: softmax, loaders, products
constexpr float kUp = 6.f;           // a weight at the reference is 2^kUp
constexpr float kMostSum = 32768.f;  // of 64 weights: none of them is above it
constexpr float kFar = 2048.f;       // a reference from which on differences are taken before anything is added
constexpr int kPlane = 32768;        // K or V: [2 planes of 64 dimensions][2 steps][2 pages][64 tokens][128 bytes]
constexpr uint32_t kColO = 0, kColS = 256;

// One block, and the part of its steps that this CTA does.
struct Segment {
  RowBlock r;
  int from, to;  // steps; none: the share is done
};
constexpr int kSegments = 4;  // announced ahead

// What the softmax warps have to know of a step's tokens, by groups of 16; of page t for tile t.
struct alignas(16) StepMeta {
  float kfac[8];  // score factor, without the row's
  float vlog[8], vinv[8];
  // Bit per token: a row that sees it is NaN (the other numbers are finite all the same). From the value
  // loaders only where the page is the tail.
  uint16_t bad_keys[8], bad_vals[8];
  int pos[2], count[2];    // position of each page's first token, tokens it holds (0: no page)
  uint32_t tokens[2][2];   // of the block, that list it
  int tail[2];             // the page is the tail
};

struct Smem {
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2][2], p_full[2][2], pv_done[2][2];
  uint64_t codes[2][4][2];  // of keys and values, by loader warp: its rows of each tile's page are there
  StepMeta meta[4];  // by step mod 4: the loaders are at most that far ahead of a softmax warp
  Segment segs[kSegments];
  int64_t scratch[36];
  uint32_t tmem;
  int abort;
};

constexpr size_t kQBytes = (size_t)kBlockRows * kD * 2;  // 64 KB: [tile][2 planes][128 rows][128 bytes]
constexpr size_t kKvBytes = (size_t)2 * kPlane;          // 64 KB each
constexpr int kRun = 16 * kD;                             // bytes of codes: a loader warp's rows of a page
constexpr size_t kCodeBytes = 2 * 4 * 2 * kRun;            // 32 KB: [keys, values][warp][page]
constexpr size_t kSmemBytes = 1024 + kQBytes + 2 * kKvBytes + kCodeBytes + sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "a CTA has 227 KB");

// fp16 x fp16 -> fp32, M = 128; b_rows_depth: B is stored with its depth as rows.
constexpr uint32_t shape(int n, bool b_rows_depth) {
  return 1u << 4 | (b_rows_depth ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(kTile >> 4) << 24;
}

// One product of depth 16, issued by the lane that has `leader` set. The whole warp runs the code around it
// together, with operands' descriptors that are sums of a base and constants: they stay in uniform
// registers, where an issue from divergent code would move them there for every product.
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "n"(ADD ? 1 : 0), "r"(leader)
      : "memory");
}

template <bool ADD>
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "n"(ADD ? 1 : 0), "r"(leader)
      : "memory");
}

// 16 bytes to shared memory without a register on the way; zeros where `there` is not (`from` is not read then).
__device__ __forceinline__ void copy16(uint32_t to, uint64_t from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copied() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__global__ void __launch_bounds__(kThreads, 1)
kv8_lists_attend(const Kv8Args a, const Rows q, const Rows out, float scale, const RowLists lists, JoinRecord* records,
                 float* partials) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const uint32_t sq = smem_u32(base), sk = sq + (uint32_t)kQBytes, sv = sk + (uint32_t)kKvBytes;
  Smem& sm = *reinterpret_cast<Smem*>(base + kQBytes + 2 * kKvBytes + kCodeBytes);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile int* abort = &sm.abort;
  const int ctas = gridDim.x, cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(smem_u32(&sm.seg_full[i]), 1);
      mbar_init(smem_u32(&sm.seg_empty[i]), kSegReaders);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.q_full[i]), 4);
      mbar_init(smem_u32(&sm.k_full[i]), 4);
      mbar_init(smem_u32(&sm.v_full[i]), 4);
      mbar_init(smem_u32(&sm.p_full[i][0]), 4);
      mbar_init(smem_u32(&sm.p_full[i][1]), 4);
      mbar_init(smem_u32(&sm.k_empty[i]), 1);
      mbar_init(smem_u32(&sm.v_empty[i]), 1);
      mbar_init(smem_u32(&sm.s_full[i][0]), 1);
      mbar_init(smem_u32(&sm.s_full[i][1]), 1);
      mbar_init(smem_u32(&sm.pv_done[i][0]), 1);
      mbar_init(smem_u32(&sm.pv_done[i][1]), 1);
      for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&sm.codes[i][w][0]), 1), mbar_init(smem_u32(&sm.codes[i][w][1]), 1);
    }
    sm.abort = 0;
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
  const int n_blocks = *lists.n_blocks;
  const Place pl = locate(
      n_blocks, sm.scratch, [&](int x, bool) { return (int64_t)lists.blocks[x].weight; },
      [&](int64_t total) { return share_start(total, cta, ctas); });
  __syncthreads();
  tmem_after();
  const uint32_t tmem = sm.tmem;
  bool ok = true;
  uint32_t seg = 0;  // segments read so far
  auto next = [&]() {  // the next segment is there and is not the end
    warp_wait(ok, smem_u32(&sm.seg_full[seg % kSegments]), seg / kSegments & 1, abort, a.err);
    return ok && sm.segs[seg % kSegments].from < sm.segs[seg % kSegments].to;
  };
  // 640 threads x 96 registers at launch = 256 x 120 + 256 x 88 + 128 x 64.

  if (warp < kKeyWarp) {
    // ------------------------------ softmax, a row a thread ------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    const int tile = warp >> 2, quad = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t S0 = lanes + kColS + tile * kTile, O = lanes + kColO + tile * kTile;
    uint32_t count = 0;  // steps of the CTA so far
    // The two tiles' warps of the same 32 rows meet at barriers in a shared block, so they go into a segment together
    // or not at all: one of them alone may have lost `ok` to a wait that ran out.
    auto both = [&](bool well) {
      int all;
      asm volatile(
          "{\n\t.reg .pred p, r;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.and.pred r, %2, 64, p;\n\tselp.s32 %0, 1, 0, r;\n\t}"
          : "=r"(all)
          : "r"((int)well), "r"(1 + quad)
          : "memory");
      return all != 0;
    };
    while (both(next())) {
      const Segment& s = sm.segs[seg % kSegments];
      const RowBlock& u = s.r;
      const bool shared = u.shared;  // both tiles have tile 0's rows, and every second page
      const int row = u.first_row + (shared ? 0 : tile * kTile) + quad * 32 + lane;
      const bool mine = row < u.n_new * a.G;
      const int i = row / a.G, head = u.h * a.G + row - i * a.G, at_token = mine ? i - u.first_row / a.G : 0;
      const int see = u.past + i + 1, steps = s.to - s.from;
      float qs = 1.f;
      bool wrong = false;   // the row's query is not finite: NaN, if it sees a token
      bool poison = false;  // the row's result is NaN
      {
        // The warp's 32 rows go to their places as they are, 16 lanes a row, all on their way at once. Then each lane
        // turns its row into fp16, scaled by the power of two that the largest element asks for (and back out: qs).
        // scale's sign goes here too.
        const uint32_t rows = sq + tile * (kTile * kD * 2) + quad * 32 * 128;
        const uint64_t mine_at = reinterpret_cast<uint64_t>(q.p + (int64_t)(u.row0 + i) * q.ts + (int64_t)head * q.hs);
        const int c16 = lane & 15;
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const int r = 2 * y + (lane >> 4);
          const uint64_t at = __shfl_sync(0xffffffffu, mine_at, r);
          const bool there = __shfl_sync(0xffffffffu, (int)mine, r);
          copy16(rows + (c16 >> 3) * (kTile * 128) + r * 128 + (((c16 & 7) ^ (r & 7)) << 4),
                 there ? at + c16 * 16 : reinterpret_cast<uint64_t>(q.p), there);
        }
        copied();
        __syncwarp();
        auto place = [&](int c) { return rows + (c >> 3) * (kTile * 128) + lane * 128 + (((c & 7) ^ (lane & 7)) << 4); };
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint4 w = lds128(place(c));
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
        }
        top = max(top & 0xffffu, top >> 16);
        const int e = half_exponent(top);
        const float f = scale < 0.f ? -pow2(15 - e) : pow2(15 - e);
        wrong = top >= 0x7f80u;
        qs = wrong ? 1.f : pow2(e - 15);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          uint4 w = lds128(place(c));
          if (wrong) w = make_uint4(0, 0, 0, 0);  // a page that it does not list must not make it NaN
          sts128(place(c), pack_half2(lo_f(w.x) * f, hi_f(w.x) * f), pack_half2(lo_f(w.y) * f, hi_f(w.y) * f),
                 pack_half2(lo_f(w.z) * f, hi_f(w.z) * f), pack_half2(lo_f(w.w) * f, hi_f(w.w) * f));
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[tile]));
      }

      float M = -INFINITY, V = 0.f, L = 0.f;  // the row's reference, and the sum relative to it
      // What the exponents take, and a page's sum from which on its weights are worked out again. Both follow the reference.
      float up = kUp, limit = wrong ? INFINITY : kMostSum;
      auto aim = [&]() {
        up = kUp - V - (M == -INFINITY ? 0.f : M);
        limit = wrong ? INFINITY : M != -INFINITY && !(fabsf(M) < kFar) ? -1.f : kMostSum;
      };
      for (int turn = 0; turn < steps; ++turn) {
        const uint32_t c = count + turn, S = S0 + (c & 1) * kPart;
        warp_wait(ok, smem_u32(&sm.s_full[tile][c & 1]), c >> 1 & 1, abort, a.err);
        if (!ok) continue;
        const StepMeta& me = sm.meta[c & 3];
        if (me.tail[tile]) {  // its values have a scale of their own, known once loaded
          warp_wait(ok, smem_u32(&sm.v_full[c & 1]), c >> 1 & 1, abort, a.err);
          if (!ok) continue;
        }
        tmem_after();
        const bool on = mine && (me.tokens[tile][at_token >> 5] >> (at_token & 31) & 1);
        const int vis = on ? min(see - me.pos[tile], me.count[tile]) : 0;  // tokens that the row sees
        // A page's 64 scores at a time. A group of 16 tokens has one scale; what the groups need is read as
        // vectors, once: a warp alone on its scheduler waits for every dependent instruction.
        uint32_t x[kPart];
        float4 fac, vlog;
        auto fetch = [&]() {
          tmem_load32(S, x);
          tmem_load32(S + 32, x + 32);
          fac = *reinterpret_cast<const float4*>(&me.kfac[4 * tile]);
          vlog = *reinterpret_cast<const float4*>(&me.vlog[4 * tile]);
          // not 0, which would make NaN of a hidden token's -inf
          fac = make_float4(fmaxf(fac.x * qs, 1e-37f), fmaxf(fac.y * qs, 1e-37f), fmaxf(fac.z * qs, 1e-37f), fmaxf(fac.w * qs, 1e-37f));
          const bool some = __any_sync(0xffffffffu, on && vis < kPart);
          tmem_loaded();
          settle32(x);
          settle32(x + 32);
          if (some) {
#pragma unroll
            for (int c = 0; c < kPart; ++c) x[c] = !on || c < vis ? x[c] : 0xff800000u;
          }
        };
        // Puts (tm, tv) at the page's largest weight, if that is above it.
        auto largest = [&](float& tm, float& tv) {
#pragma unroll
          for (int grp = 0; grp < 4; ++grp) {
            float s = __uint_as_float(x[grp * 16]);
#pragma unroll
            for (int c = 1; c < 16; ++c) s = fmaxf(s, __uint_as_float(x[grp * 16 + c]));
            s = __fmul_rn(s, grp == 0 ? fac.x : grp == 1 ? fac.y : grp == 2 ? fac.z : fac.w);
            const float l = grp == 0 ? vlog.x : grp == 1 ? vlog.y : grp == 2 ? vlog.z : vlog.w;
            if ((s - tm) + (l - tv) > 0.f) tm = s, tv = l;
          }
        };
        // What was added up so far, times f: L, and the output once its products are done. (f is 1 for some rows, a power of
        // two for the others.)
        auto rescale = [&](float f) {
          L *= f;
          if (turn == 0) return;
          warp_wait(ok, smem_u32(&sm.pv_done[tile][(c - 1) & 1]), (c - 1) >> 1 & 1, abort, a.err);
          if (!ok) return;
          tmem_after();
          uint32_t y[8];
#pragma unroll 1
          for (int k = 0; k < kD; k += 8) {
            tmem_load8(O + k, y);
            tmem_loaded();
            settle8(y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
            tmem_store8(O + k, y);
          }
        };
        uint32_t p[32];
        if (!__any_sync(0xffffffffu, on)) {  // nobody's page
#pragma unroll
          for (int k = 0; k < 16; ++k) p[k] = 0;
          tmem_store16(S, p);
          tmem_store16(S + 16, p);
        } else {
          fetch();
          if (__any_sync(0xffffffffu, M == -INFINITY && on)) {  // no reference yet: the page's maximum
            float tm = M, tv = V;
            if (on) largest(tm, tv);
            if (M == -INFINITY) M = tm, V = tv;
            aim();
          }
          float sum[4];
          float shift = on ? up : -INFINITY, most = limit;
          for (;;) {  // twice at most: no sum is above the second time's limit
#pragma unroll
            for (int grp = 0; grp < 4; ++grp) {
              const uint64_t k2 = twice(grp == 0 ? fac.x : grp == 1 ? fac.y : grp == 2 ? fac.z : fac.w);
              const uint64_t c2 = twice((grp == 0 ? vlog.x : grp == 1 ? vlog.y : grp == 2 ? vlog.z : vlog.w) + shift);
              uint64_t sum2[2] = {0, 0};
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                float y0, y1;
                unpack2(fma2(pack2(x[grp * 16 + c], x[grp * 16 + c + 1]), k2, c2), y0, y1);
                y0 = ex2(y0);
                y1 = ex2(y1);
                sum2[c >> 1 & 1] = add2(sum2[c >> 1 & 1], pack2(__float_as_uint(y0), __float_as_uint(y1)));
                p[grp * 8 + c / 2] = pack_half2(y0, y1);
              }
              float s0, s1;
              unpack2(add2(sum2[0], sum2[1]), s0, s1);
              sum[grp] = s0 + s1;
            }
            if (!__any_sync(0xffffffffu, (sum[0] + sum[1]) + (sum[2] + sum[3]) > most)) break;
            most = INFINITY;
            // Rare. The reference goes to the page's largest weight, for the rows where that is far above it: by a whole
            // power of two, which fp16 weights take exactly, unless nothing is left of them. Then every exponent is at
            // most kUp + 3, with the score's difference taken first.
            fetch();
            float tm = M, tv = V, d = 0.f;
            if (on) largest(tm, tv);
            const float above = (tm - M) + (tv - V);
            if (above > 3.f && !wrong) {
              d = above < 64.f ? ceilf(above) : above;
              V = above < 64.f ? V + (d - (tm - M)) : tv;
              M = tm;
            }
            if (__any_sync(0xffffffffu, d > 0.f)) rescale(ex2(-d));
            aim();
            const float at = M == -INFINITY ? 0.f : M;
            auto apart = [&](int grp, float f) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                x[grp * 16 + c] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(x[grp * 16 + c]), f), at));
            };
            apart(0, fac.x), apart(1, fac.y), apart(2, fac.z), apart(3, fac.w);
            fac = make_float4(1.f, 1.f, 1.f, 1.f);
            shift = on ? kUp - V : -INFINITY;
          }
          const float4 vinv = *reinterpret_cast<const float4*>(&me.vinv[4 * tile]);
          L += fmaf(sum[0], vinv.x, sum[1] * vinv.y) + fmaf(sum[2], vinv.z, sum[3] * vinv.w);
          tmem_store16(S, p);  // half of the columns that the scores had
          tmem_store16(S + 16, p + 16);
          if (!ok) continue;
          // tokens that make NaN of the rows that see them
          uint2 bad = *reinterpret_cast<const uint2*>(&me.bad_keys[4 * tile]);
          if (me.tail[tile]) {
            const uint2 more = *reinterpret_cast<const uint2*>(&me.bad_vals[4 * tile]);
            bad = make_uint2(bad.x | more.x, bad.y | more.y);
          }
          poison |= wrong && vis > 0;
          if (bad.x | bad.y)
            poison |= ((vis < 32 ? bad.x & ((1u << max(vis, 0)) - 1u) : bad.x) |
                       (vis < 64 ? bad.y & ((1u << max(vis - 32, 0)) - 1u) : bad.y)) != 0;
        }
        tmem_stored();
        tmem_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[tile][c & 1]));
      }
      count += steps;

      // ---- the row's end ----
      if (poison) L = __uint_as_float(0x7fc00000u);
      // (The second last product may be done or not: with a barrier for both, neither phase could be waited for.)
      warp_wait(ok, smem_u32(&sm.pv_done[tile][(count - 1) & 1]), (count - 1) >> 1 & 1, abort, a.err);
      tmem_after();
      // Rows go through the warp's own rows of Q, which no product reads any more, so that they are stored in
      // runs of whole rows: 16-byte chunk c of row r at c ^ (r & 7), as everywhere.
      const uint32_t stage = sq + tile * (kTile * kD * 2) + quad * 32 * 128;
      // Tile 1's half of a shared block crosses over there too, 32 columns at a time, between the two warps of
      // a row: M, L and V in the second plane, the output in the first.
      const uint32_t other = sq + kTile * kD * 2 + quad * 32 * 128;
      auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory"); };
      float f0 = 1.f, f1 = 0.f;  // the tiles' weights
      if (shared && tile == 1) {
        sts128(other + kTile * 128 + lane * 16, __float_as_uint(M), __float_as_uint(L), __float_as_uint(V), 0u);
        pair_sync();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t y[32];
          tmem_load32(O + c * 32, y);
          tmem_loaded();
          settle32(y);
          if (c) pair_sync();
#pragma unroll
          for (int k = 0; k < 8; ++k) sts128(other + lane * 128 + ((k ^ (lane & 7)) << 4), y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
          pair_sync();
        }
        pair_sync();  // the next block's rows come here only once these have been read
      } else if (shared) {
        pair_sync();
        const uint4 w = lds128(other + kTile * 128 + lane * 16);
        const float m1 = __uint_as_float(w.x), l1 = __uint_as_float(w.y), v1 = __uint_as_float(w.z);
        const float top = fmaxf(M, m1), at = top == -INFINITY ? 0.f : top;
        const float a0 = (M - at) + V, a1 = (m1 - at) + v1;
        V = top == -INFINITY ? 0.f : fmaxf(a0, a1);
        f0 = ex2(a0 - V);
        f1 = ex2(a1 - V);
        L = L * f0 + l1 * f1;
        M = top;
      }
      // 32 columns of the row's output
      auto columns = [&](int c, uint32_t* y) {
        tmem_load32(O + c * 32, y);
        tmem_loaded();
        settle32(y);
        if (!shared) return;
        pair_sync();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4 v = lds128(other + lane * 128 + ((k ^ (lane & 7)) << 4));
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // (a tile that has seen nothing has nothing in its columns)
            const float y0 = f0 == 0.f ? 0.f : __uint_as_float(y[4 * k + e]) * f0, y1 = f1 == 0.f ? 0.f : __uint_as_float(w[e]) * f1;
            y[4 * k + e] = __float_as_uint(y0 + y1);
          }
        }
        pair_sync();
      };
      if (!shared || tile == 0) {
        const bool whole = s.from == 0 && s.to == u.steps;
        float* part = partials + ((int64_t)(2 * cta + (s.from == 0 ? 1 : 0)) * kBlockRows + tile * kTile + quad * 32) * kPartialStride;
        if (!whole && mine) *reinterpret_cast<float4*>(part + lane * kPartialStride) = make_float4(M, L, V, 0.f);
        __syncwarp();
        if (whole) {
          const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t y[32];
            columns(c, y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(y[k * 8 + 2 * e]) * inv, __uint_as_float(y[k * 8 + 2 * e + 1]) * inv);
                w[e] = *reinterpret_cast<const uint32_t*>(&v);
              }
              sts128(stage + (c >> 1) * (kTile * 128) + lane * 128 + ((((c & 1) * 4 + k) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
          const uint64_t mine_at = reinterpret_cast<uint64_t>(out.p + (int64_t)(u.row0 + i) * out.ts + (int64_t)head * out.hs);
          const int r2 = lane >> 4, c16 = lane & 15;
#pragma unroll 4
          for (int x = 0; x < 16; ++x) {
            const int r = 2 * x + r2;
            const uint64_t at = __shfl_sync(0xffffffffu, mine_at, r);
            const bool there = __shfl_sync(0xffffffffu, (int)mine, r);
            const uint4 v = lds128(stage + (c16 >> 3) * (kTile * 128) + r * 128 + (((c16 & 7) ^ (r & 7)) << 4));
            if (there && ok) reinterpret_cast<uint4*>(at)[c16] = v;
          }
        } else {
          const int rows = min(32, u.n_new * a.G - (u.first_row + tile * kTile + quad * 32));  // the warp's
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t y[32];
            columns(c, y);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) sts128(stage + lane * 128 + ((k ^ (lane & 7)) << 4), y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const int r = 4 * x + (lane >> 3), k = lane & 7;
              const uint4 v = lds128(stage + r * 128 + ((k ^ (r & 7)) << 4));
              if (r < rows) *reinterpret_cast<uint4*>(part + r * kPartialStride + 4 + c * 32 + k * 4) = v;
            }
          }
        }
        __syncwarp();
      }
      tmem_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[seg % kSegments]));
      ++seg;
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------ loaders: four warps of keys, four of values ------------------------------
    // Warp w has rows 16 w .. 16 w + 15 of every page. In load x, eight lanes have 64 bytes of two neighbouring
    // rows each, the odd row's from its other half, so that both the loads and the 16-byte stores fall on
    // eight different columns.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int half = warp >= kValueWarp ? 1 : 0;
    const int w4 = warp & 3, c4 = lane & 3, odd = lane >> 2 & 1, row0 = (lane >> 3) * 2 + odd;
    const uint32_t run = sv + (uint32_t)kKvBytes + (half * 4 + w4) * 2 * kRun;
    uint64_t* codes = sm.codes[half][w4];
    uint32_t turn = 0;  // bit per page: the parity of its next codes
    const uint32_t operand0 = half ? sv : sk;
    uint64_t* full = half ? sm.v_full : sm.k_full;
    uint64_t* empty = half ? sm.v_empty : sm.k_empty;
    uint32_t count = 0;
    while (next()) {
      const Segment& s = sm.segs[seg % kSegments];
      const RowBlock& u = s.r;
      const int64_t unit = (int64_t)u.b * a.Hkv + u.h;
      const RowItem* items = lists.items + u.place;
      const int end = 2 * s.to;
      int id = -1, pos = -1, id_base = 2 * s.from;
      // Page ids of 32 items, a lane each (the last two are looked up again with the next), and for the keys' warps
      // what the softmax has to know of the pages.
      float kfac = 0.f, vlog = 0.f, vinv = 1.f;
      bool bad = false;
      uint32_t who[2] = {0, 0};  // tokens that list the page
      auto look = [&](int first) {
        id_base = first;
        const int it = first + lane;
        id = -1;
        pos = 0;
        kfac = vlog = 0.f;
        vinv = 1.f;
        bad = false;
        who[0] = who[1] = 0;
        if (it < end) {
          const uint4 v = *reinterpret_cast<const uint4*>(items + it);
          id = (int)v.x;
          pos = (int)v.y * kPart;
          who[0] = v.z;
          who[1] = v.w;
          if (id >= 0 && !half) {
            const float2 sc = *reinterpret_cast<const float2*>(a.scales + 2 * (int64_t)id);
            bad = !(sc.x == sc.x && sc.y == sc.y);
            kfac = bad ? 0.f : sc.x * fabsf(scale) * kLog2e;
            vlog = bad ? 0.f : scale_log2(sc.y);
            vinv = bad ? 1.f : 1.f / sc.y;
          }
        }
      };
      // The codes of a page come in one copy, which is under way again as soon as they are in registers.
      uint4 raw[8];
      auto load = [&](int pg, int page) {
        if (page < 0 || lane) return;
        mbar_arrive_expect_tx(smem_u32(&codes[pg]), kRun);
        bulk_copy(run + pg * kRun, a.pages + (int64_t)page * kKv8PageBytes + half * kKv8HalfBytes + w4 * kRun, kRun, smem_u32(&codes[pg]));
      };
      auto take = [&](int pg, int page) {
        if (page >= 0) {
          warp_wait(ok, smem_u32(&codes[pg]), turn >> pg & 1, abort, a.err);
          turn ^= 1u << pg;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          raw[pg * 4 + x] = page >= 0 ? lds128(run + pg * kRun + (row0 + (x >> 1) * 8) * kD + ((x & 1) ^ odd) * 64 + c4 * 16) : make_uint4(0, 0, 0, 0);
      };
      auto put_page = [&](uint32_t at, int pg) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = w4 * 16 + row0 + (x >> 1) * 8;
          const uint4 v = raw[pg * 4 + x];
          const uint32_t dst = at + ((x & 1) ^ odd) * kPlane + (pg * kPart + row) * 128;
          sts128(dst + (((c4 * 2 + 0) ^ (row & 7)) << 4), e4m3x2_half2(v.x, false), e4m3x2_half2(v.x, true),
                 e4m3x2_half2(v.y, false), e4m3x2_half2(v.y, true));
          sts128(dst + (((c4 * 2 + 1) ^ (row & 7)) << 4), e4m3x2_half2(v.z, false), e4m3x2_half2(v.z, true),
                 e4m3x2_half2(v.w, false), e4m3x2_half2(v.w, true));
        }
      };
      // The tail as page pg: the warp's 16 rows scaled by a power of two. Twice over the rows (they are in
      // L1 by then), to hold no more than one of them.
      auto put_tail = [&](uint32_t at, int pg, StepMeta& me) {
        const uint16_t* src = a.tails + unit * kPageElems + half * kPart * kD;
        const int r4 = lane >> 3, c8 = lane & 7;
        uint32_t wrong = 0, top = 0;
        auto row_of = [&](int x) {
          const int row = w4 * 16 + (x >> 1) * 4 + r4;
          uint4 t = make_uint4(0, 0, 0, 0);
          if (row < u.tail) t = *(reinterpret_cast<const uint4*>(src + row * kD + c8 * 16) + (x & 1));
          uint32_t* tt = reinterpret_cast<uint32_t*>(&t);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool lo = (tt[e] & 0x7f80u) == 0x7f80u, hi = (tt[e] & 0x7f800000u) == 0x7f800000u;
            if (lo) tt[e] &= 0xffff0000u;
            if (hi) tt[e] &= 0x0000ffffu;
            if (lo || hi) wrong |= 1u << ((x >> 1) * 4 + r4);
          }
          return t;
        };
#pragma unroll 1
        for (int x = 0; x < 8; ++x) {
          const uint4 t = row_of(x);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(t.x & 0x7fff7fffu, t.y & 0x7fff7fffu), __vmaxu2(t.z & 0x7fff7fffu, t.w & 0x7fff7fffu)));
        }
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const int e = half_exponent(top);
        const float f = pow2(15 - e);
#pragma unroll 1
        for (int x = 0; x < 8; ++x) {
          const uint4 t = row_of(x);
          const int row = w4 * 16 + (x >> 1) * 4 + r4;
          sts128(at + (c8 >> 2) * kPlane + (pg * kPart + row) * 128 + ((((c8 & 3) * 2 + (x & 1)) ^ (row & 7)) << 4),
                 pack_half2(lo_f(t.x) * f, hi_f(t.x) * f), pack_half2(lo_f(t.y) * f, hi_f(t.y) * f),
                 pack_half2(lo_f(t.z) * f, hi_f(t.z) * f), pack_half2(lo_f(t.w) * f, hi_f(t.w) * f));
        }
        wrong = __reduce_or_sync(0xffffffffu, wrong);
        if (lane == 0) {
          if (half) {
            me.vlog[pg * 4 + w4] = (float)(e - 15);
            me.vinv[pg * 4 + w4] = f;
            me.bad_vals[pg * 4 + w4] = (uint16_t)wrong;
          } else {
            me.kfac[pg * 4 + w4] = fabsf(scale) * kLog2e * pow2(e - 15);
            me.bad_keys[pg * 4 + w4] = (uint16_t)wrong;
          }
        }
      };
      look(2 * s.from);
      auto id_of = [&](int it) { return __shfl_sync(0xffffffffu, id, it - id_base); };
      int id0 = id_of(2 * s.from), id1 = id_of(2 * s.from + 1);
      load(0, id0);
      load(1, id1);
      for (int it = 2 * s.from; it < end && ok; it += 2, ++count) {
        const uint32_t slot = count & 1, at = operand0 + slot * 16384;
        StepMeta& me = sm.meta[count & 3];
        const int now0 = id0, now1 = id1;
        id0 = id1 = kNoItem;
        if (it + 2 < end) {
          if (it + 2 >= id_base + 32) look(it);
          id0 = id_of(it + 2);
          id1 = id_of(it + 3);
        }
        take(0, now0);
        take(1, now1);
        proxy_fence();  // what was read is read before the next copy writes
        __syncwarp();
        if (!ok) break;
        load(0, id0);
        load(1, id1);
        warp_wait(ok, smem_u32(&empty[slot]), (count >> 1 & 1) ^ 1, abort, a.err);
        if (!ok) break;
        const int x = lane - (it - id_base);
        if (!half && (x & ~1) == 0) {  // what the softmax has to know of the pages
          if (id != kTailItem) {
            me.kfac[x * 4 + w4] = kfac;
            me.vlog[x * 4 + w4] = vlog;
            me.vinv[x * 4 + w4] = vinv;
            me.bad_keys[x * 4 + w4] = bad ? 0xffffu : 0u;
          }
          if (w4 == 0) {
            me.tail[x] = id == kTailItem;
            me.count[x] = id == kTailItem ? u.tail : id >= 0 ? kPart : 0;
            me.pos[x] = pos;
            me.tokens[x][0] = who[0];
            me.tokens[x][1] = who[1];
          }
        }
        if (now0 == kTailItem) put_tail(at, 0, me);
        else put_page(at, 0);
        if (now1 == kTailItem) put_tail(at, 1, me);
        else put_page(at, 1);
        proxy_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&full[slot]));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[seg % kSegments]));
      ++seg;
    }
  } else {
    // ------------------------------ products ------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == kMmaWarp) {
      const uint32_t leader = elect();
      auto wait = [&](const uint64_t& bar, uint32_t parity) {
        warp_wait(ok, smem_u32(&bar), parity, abort, a.err);
      };
      uint32_t count = 0;
      const uint64_t dq = operand(sq, 16, 1024), dk = operand(sk, 16, 1024), dv = operand(sv, kPlane, 1024);
      // Tile t's page is the step's t-th: 64 rows of 128 bytes further.
      auto scores = [&](auto tile, uint32_t c) {
        constexpr int t = decltype(tile)::value;
        const uint32_t d = tmem + kColS + t * kTile + (c & 1) * kPart;
        const uint64_t q0 = dq + t * (kTile * kD * 2 >> 4), k0 = dk + (c & 1) * (16384 >> 4) + t * (8192 >> 4);
        mma_ss<false>(leader, d, q0, k0, shape(kPart, false));
#pragma unroll
        for (int k = 1; k < 8; ++k)
          mma_ss<true>(leader, d, q0 + ((k >> 2) * (kTile * 128 >> 4) + (k & 3) * 2), k0 + ((k >> 2) * (kPlane >> 4) + (k & 3) * 2),
                       shape(kPart, false));
        mma_commit(leader, smem_u32(&sm.s_full[t][c & 1]));
      };
      auto values = [&](auto tile, uint32_t c, bool add) {
        constexpr int t = decltype(tile)::value;
        const uint32_t d = tmem + kColO + t * kTile, p = tmem + kColS + t * kTile + (c & 1) * kPart;
        const uint64_t v0 = dv + (c & 1) * (16384 >> 4) + t * (8192 >> 4);
        if (add) mma_ts<true>(leader, d, p, v0, shape(kD, true));
        else mma_ts<false>(leader, d, p, v0, shape(kD, true));
#pragma unroll
        for (int k = 1; k < 4; ++k) mma_ts<true>(leader, d, p + k * 8, v0 + k * (2048 >> 4), shape(kD, true));
        mma_commit(leader, smem_u32(&sm.pv_done[t][c & 1]));
      };
      constexpr std::integral_constant<int, 0> kTile0;
      constexpr std::integral_constant<int, 1> kTile1;
      auto both_scores = [&](uint32_t c) {
        wait(sm.k_full[c & 1], c >> 1 & 1);
        tmem_after();
        if (!ok) return;
        scores(kTile0, c);
        scores(kTile1, c);
        mma_commit(leader, smem_u32(&sm.k_empty[c & 1]));
      };
      while (next()) {
        const Segment& s = sm.segs[seg % kSegments];
        const int steps = s.to - s.from;
        wait(sm.q_full[0], seg & 1);
        wait(sm.q_full[1], seg & 1);
        both_scores(count);
        if (steps > 1) both_scores(count + 1);
#pragma unroll 1
        for (int step = 0; step < steps; ++step, ++count) {
          wait(sm.v_full[count & 1], count >> 1 & 1);
          wait(sm.p_full[0][count & 1], count >> 1 & 1);
          tmem_after();
          if (ok) values(kTile0, count, step > 0);
          wait(sm.p_full[1][count & 1], count >> 1 & 1);
          tmem_after();
          if (ok) values(kTile1, count, step > 0);
          if (ok) mma_commit(leader, smem_u32(&sm.v_empty[count & 1]));
          if (step + 2 < steps) both_scores(count + 2);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[seg % kSegments]));
        ++seg;
      }
      // The last arrivals have landed before the CTA's shared memory goes.
      if (count > 0) {
        wait(sm.k_empty[(count - 1) & 1], (count - 1) >> 1 & 1);
        wait(sm.v_empty[(count - 1) & 1], (count - 1) >> 1 & 1);
      }
    }
    if (warp == kPlanWarp && lane == 0) {
      int x = pl.b;
      int64_t at = share_start(pl.total, cta, ctas), before = pl.before;
      const int64_t stop = share_start(pl.total, cta + 1, ctas);
      JoinRecord open = JoinRecord{};
      Segment s;
      for (bool more = true; more && ok; ++seg) {
        s.from = s.to = 0;
        while (at < stop && x < n_blocks) {
          s.r = lists.blocks[x];
          const int weight = s.r.weight;
          if (weight == 0 || at >= before + weight) {
            before += weight;
            ++x;
            continue;
          }
          const int f = (int)(at - before), t = (int)min((int64_t)weight, f + (stop - at));
          at += t - f;
          s.from = max(0, f - (weight - s.r.steps));
          s.to = max(0, t - (weight - s.r.steps));
          if (s.from >= s.to) continue;
          if (s.from == 0 && s.to < s.r.steps)
            open = JoinRecord{pl.total, share_of(pl.total, before + weight - 1, ctas) - cta + 1, s.r.row0, s.r.n_new, s.r.h, s.r.first_row, 0};
          break;
        }
        more = s.from < s.to;
        ok = ok && mbar_wait(smem_u32(&sm.seg_empty[seg % kSegments]), (seg / kSegments & 1) ^ 1, abort, a.err);
        if (!ok) break;
        sm.segs[seg % kSegments] = s;
        mbar_arrive(smem_u32(&sm.seg_full[seg % kSegments]));
      }
      records[cta] = open;
    }
    __syncwarp();
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  if (warp == kMmaWarp) {
    if (*abort) settle_down();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace

cudaError_t launch_kv8_lists(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const RowLists& lists,
                             void* workspace, int sm_count, cudaStream_t st) {
  const int ctas = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  cudaError_t e = cudaFuncSetAttribute(kv8_lists_attend, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_early(kv8_lists_attend, dim3((unsigned)ctas), kThreads, kSmemBytes, st, a, q, out, scale, lists,
                   static_cast<JoinRecord*>(workspace), reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kRecordBytes));
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_kv8_join(a, out, ctas, 16, workspace, kBlockRows, st);
}

}  // namespace spin
