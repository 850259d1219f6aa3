// spin_kv8_attend for many rows a unit: prompt chunks, and drafted tokens of a large group.
//
// With M = 128 rows of queries per tile a page costs 4 * 128 * 128 * 64 flops and 16 KB, so the tensor
// cores are what can be busy: one persistent CTA per SM holds 256 rows (two tiles) of one unit and
// takes two pages (128 tokens) a step. All products are tcgen05.mma on fp16 operands with fp32
// accumulators in tensor memory:
//   S_t[128 x 128] = Q_t (shared memory) K^T (shared memory), 8 products of depth 16,
//   O_t[128 x 128] += P_t (tensor memory, in the place of S_t) V (shared memory, tokens as depth).
// Roles, by warp:
//   0-3, 4-7  softmax of tile 0 and 1, one row a thread: scores out of tensor memory, fp16 weights back into
//             it, relative to a reference that is the maximum of the row's first step. A later step looks
//             for no maximum: its sums say whether a weight may have left fp16's range, and then,
//             which is rare, the reference is raised, once, and what was added up so far scaled. Rows are
//             stored at the end;
//   8-11      keys from HBM to fp16 in shared memory, 128-byte swizzled. A step's loads are in registers
//             one step ahead of their use, so no shared memory holds codes;
//   12-15     values, likewise;
//   17        walks the CTA's share of the work and announces its segments;
//   16        issues the products: P_0 V, S_0, P_1 V, S_1 of each step, so that one tile's softmax
//             runs under the other's products.
// A block of at most 128 rows (drafted tokens, the end of a prompt) is held by both tiles, which take the
// steps in turn, so that the one's softmax still runs under the other's products; tile 1's result is
// joined to tile 0's through shared memory at the end.
// Tensor memory: O_0, O_1, S_0, S_1 of 128 columns each. Shared memory: Q_0, Q_1 and two steps of
// K and of V, 32 KB each.
//
// The arithmetic is that of the few-row kernel: with s = score * k * log2(e) per page, weights are
// 2^((s - M) + (log2(v) - V) + 6), the softmax sum takes weight / v. The reference is a pair, a score M and the
// log2 of a values' scale V: scores may be of any size, where one sum of the two would lose V (and the shift) to
// the sum's rounding. Weights up to 2^15 are let pass. Up to |M| = 2^11 an exponent is one fused operation,
// s + (log2(v) - V + 6 - M), off by at most 2^-12; a page of a row beyond it, or one that raises the reference, is
// taken again with s - M first, which is exact near the reference. (The chunk below takes 3340 us where all rows are beyond.)
//
// Measured: 2048 tokens onto 30000, 8 KV heads in groups of 8: 2.08 TFLOP in 2000 us, 1.04 PFLOP/s. A step of two
// tiles takes 4930 clocks. Its 32 products need 2048 at the tensor cores' rate; their operands share the shared
// memory with the loaders' stores, and they take 3300. The rest is a softmax that the other tile's products do not
// cover. A block costs another 5 us for its queries, its first step and its output: prompts of 300 to 6000
// tokens run at 0.7 PFLOP/s. Queries that go to shared memory through registers, four rows a time, cost 5 us
// a block more. Drafts of 5 tokens in groups of 8 (40 of a tile's 128 rows) read 0.33 GB in 135 us: 66 steps a CTA
// that are a chain of load, conversion, product, softmax and product with one step's codes in flight. Nothing is
// saturated there (DRAM 31%, the tensor pipe 27%, issue slots 36%).
#include "kv8_dev.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kTile = kTileRows;
constexpr int kBlockRows = 2 * kTile;
constexpr int kStep = 2 * kPart;  // tokens of a step
constexpr int kThreads = 640;
constexpr int kKeyWarp = 8, kValueWarp = 12, kMmaWarp = 16, kPlanWarp = 17;
constexpr int kSegReaders = 17;  // warps that read a segment: softmax, loaders, products
constexpr float kUp = 6.f;          // a weight at the reference is 2^kUp
constexpr float kMostSum = 32768.f;  // of 64 weights: none of them is above it
constexpr float kFar = 2048.f;      // a reference from which on differences are taken before anything is added
constexpr int kPlane = 32768;  // K or V: [2 planes of 64 dimensions][2 steps][128 tokens][128 bytes]
constexpr uint32_t kColO = 0, kColS = 256;

// One row block of one head, and the part of its items that this CTA does.
struct Segment {
  Unit u;
  int b, h, first_row, from, to;
  int steps;           // of two items each; 0: the share is done
  int limit0, limit1;  // items that a tile's last row may see; limit1 0: it has none, and the tiles share tile 0's
  __device__ __forceinline__ int limit(int tile) const { return tile ? limit1 : limit0; }
  __device__ __forceinline__ bool shared() const { return limit1 == 0; }
  __device__ __forceinline__ bool active(int tile, int step) const { return from + 2 * step < min(to, limit(tile)); }
};
constexpr int kSegments = 4;  // announced ahead

// What the softmax warps have to know of a step's tokens, by groups of 16.
struct alignas(16) StepMeta {
  float kfac[8];       // score factor, without the row's
  float vlog[8], vinv[8];
  // Bit per token: a row that sees it is NaN (the other numbers are finite all the same). From the value
  // loaders only where the page is the tail.
  uint16_t bad_keys[8], bad_vals[8];
  int pos[2], count[2];  // position of each page's first token, tokens it holds (0: no page)
};

struct Smem {
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done[2];
  StepMeta meta[4];  // by step mod 4: a softmax warp may be two steps behind the loaders, which run one ahead
  Segment segs[kSegments];
  int64_t scratch[36];
  uint32_t tmem;
  int abort;
};

constexpr size_t kQBytes = (size_t)kBlockRows * kD * 2;       // 64 KB: [tile][2 planes][128 rows][128 bytes]
constexpr size_t kKvBytes = (size_t)2 * kPlane;               // 64 KB each
constexpr size_t kSmemBytes = 1024 + kQBytes + 2 * kKvBytes + sizeof(Smem);
// 196 KB with the 1 KB that the system takes: the next size of the SM's shared memory would leave the L1
// too small to have the loaders' loads in flight (11% slower, with few rows 25%).
static_assert(kSmemBytes + 1024 <= 196 * 1024, "shared memory of a CTA");
constexpr int kWeights = 4096;  // requests' weights, in Q's place before there is a Q
static_assert(kWeights * 8 <= kQBytes, "");

// Shared memory descriptor of a 128-byte swizzled operand: 8-row groups `sbo` bytes apart, and for an
// operand whose rows are the depth, 64-element blocks `lbo` bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

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

// The barrier is arrived at once all products issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(leader)
      : "memory");
}

__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r;
}

__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define SPIN_R8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), "+r"(a[i + 5]), "+r"(a[i + 6]), "+r"(a[i + 7])
#define SPIN_W8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define SPIN_I8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of the warp's 32 lanes, one lane a thread. The values are there after tmem_loaded().
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SPIN_W8(r, 0), SPIN_W8(r, 8), SPIN_W8(r, 16), SPIN_W8(r, 24)
      : "r"(addr)
      : "memory");
}

// After tmem_loaded(): uses of the loaded registers stay behind it.
__device__ __forceinline__ void settle32(uint32_t* r) {
  asm volatile("" : SPIN_R8(r, 0), SPIN_R8(r, 8), SPIN_R8(r, 16), SPIN_R8(r, 24));
}

__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::SPIN_I8(r, 0),
      SPIN_I8(r, 8), "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : SPIN_W8(r, 0)
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::SPIN_I8(r, 0), "r"(addr)
               : "memory");
}

__device__ __forceinline__ void settle8(uint32_t* r) { asm volatile("" : SPIN_R8(r, 0)); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t twice(float x) { return pack2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

__device__ __forceinline__ int64_t blocks_weight(const Kv8Args& a, int b, int topk, bool report) {
  const Unit u = request_of(a, b, report);
  const int64_t rows = (int64_t)u.n_new * a.G;
  // set_rows() block after block, the division by G carried along
  int token = (kBlockRows - 1) / a.G, rest = (kBlockRows - 1) - token * a.G;
  const int token_step = kBlockRows / a.G, rest_step = kBlockRows - token_step * a.G;
  int64_t sum = 0;
  for (int64_t row = 0; row < rows; row += kBlockRows) {
    const int seen = u.past + min(u.n_new, token + 1);
    const int pages = topk ? topk : min(u.full, (seen + kPart - 1) >> 6);
    const int items = pages + (u.tail && seen > u.full * kPart ? 1 : 0);
    sum += items ? items + unit_cost(kBlockRows, (int)min(rows - row, (int64_t)kBlockRows)) : 0;
    token += token_step;
    rest += rest_step;
    if (rest >= a.G) {
      rest -= a.G;
      ++token;
    }
  }
  return sum * a.Hkv;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__global__ void __launch_bounds__(kThreads, 1)
kv8_prefill_kernel(const Kv8Args a, const Rows q, const Rows out, float scale, const int32_t* sel, int topk,
                   JoinRecord* records, float* partials) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sq = smem_u32(base), sk = sq + (uint32_t)kQBytes, sv = sk + (uint32_t)kKvBytes;
  Smem& sm = *reinterpret_cast<Smem*>(base + kQBytes + 2 * kKvBytes);
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
      mbar_init(smem_u32(&sm.p_full[i]), 4);
      mbar_init(smem_u32(&sm.k_empty[i]), 1);
      mbar_init(smem_u32(&sm.v_empty[i]), 1);
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.pv_done[i]), 1);
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
  // Requests' weights, a warp each; beyond kWeights requests, a thread each, twice over.
  const bool few = a.B <= kWeights;
  int64_t* weights = reinterpret_cast<int64_t*>(base);
  if (few) {
    for (int b = warp; b < a.B; b += kThreads / 32) {
      Unit u = request_of(a, b, cta == 0 && lane == 0);
      const int blocks = (int)(((int64_t)u.n_new * a.G + kBlockRows - 1) / kBlockRows);
      int64_t sum = 0;
      for (int k = lane; k < blocks; k += 32) {
        set_rows(a, u, k * kBlockRows, kBlockRows, topk);
        sum += u.weight;
      }
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) weights[b] = sum * a.Hkv;
    }
    __syncthreads();
  }
  const Place pl = locate(
      a.B, sm.scratch, [&](int x, bool first) { return few ? weights[x] : blocks_weight(a, x, topk, first && cta == 0); },
      [&](int64_t total) { return share_start(total, cta, ctas); });
  tmem_after();
  const uint32_t tmem = sm.tmem;
  bool ok = true;
  uint32_t seg = 0;  // segments read so far
  auto next = [&]() {  // the next segment is there and is not the end
    warp_wait(ok, smem_u32(&sm.seg_full[seg % kSegments]), seg / kSegments & 1, abort, a.err);
    return ok && sm.segs[seg % kSegments].steps > 0;
  };
  // 640 threads x 96 registers at launch = 256 x 128 + 256 x 80 + 128 x 64.

  if (warp < kKeyWarp) {
    // ------------------------------ softmax, a row a thread ------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    const int tile = warp >> 2, quad = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t S = lanes + kColS + tile * kTile, O = lanes + kColO + tile * kTile;
    uint32_t done = 0;    // steps of this tile so far
    uint32_t count = 0;   // steps of the CTA so far
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
      const bool shared = s.shared();  // both tiles have tile 0's rows, and every second step
      const int row = s.first_row + (shared ? 0 : tile * kTile) + quad * 32 + lane;
      const bool mine = row < s.u.n_new * a.G;
      const int i = row / a.G, head = s.h * a.G + row - i * a.G;
      const int see = mine ? s.u.past + i + 1 : 0x7fffffff;  // rows that are not there see all: no masks for them
      float qs = 1.f;
      bool wrong = false;   // the row's query is not finite: NaN, if it sees a token
      bool poison = false;  // the row's result is NaN
      const int all_steps = max(0, (min(s.to, shared ? s.limit0 : s.limit(tile)) - s.from + 1) / 2);
      const int my_steps = shared ? (all_steps - tile + 1) / 2 : all_steps;
      if (my_steps) {
        // The warp's 32 rows go to their places as they are, 16 lanes a row, all on their way at once. Then each lane
        // turns its row into fp16, scaled by the power of two that the largest element asks for (and back out: qs).
        // scale's sign goes here too.
        const uint32_t rows = sq + tile * (kTile * kD * 2) + quad * 32 * 128;
        const uint64_t mine_at = reinterpret_cast<uint64_t>(q.p + (int64_t)(s.u.row0 + i) * q.ts + (int64_t)head * q.hs);
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
          const uint4 w = lds128(place(c));
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
      for (int turn = 0; turn < my_steps; ++turn, ++done) {
        const int step = shared ? 2 * turn + tile : turn;
        warp_wait(ok, smem_u32(&sm.s_full[tile]), done & 1, abort, a.err);
        if (!ok) continue;
        const StepMeta& me = sm.meta[(count + step) & 3];
        const int halves = s.from + 2 * step + 1 < s.to ? 2 : 1;
        if (s.from + 2 * step + halves > s.u.pages) {  // the tail's values have a scale of their own, known once loaded
          const uint32_t c = count + step;
          warp_wait(ok, smem_u32(&sm.v_full[c & 1]), c >> 1 & 1, abort, a.err);
          if (!ok) continue;
        }
        tmem_after();
        // A page's 64 scores at a time. A group of 16 tokens has one scale; what the groups need is read as
        // vectors, once: a warp alone on its scheduler waits for every dependent instruction.
        uint32_t x[kPart];
        float4 fac, vlog;
        auto tokens = [&](int hf) { return min(see - me.pos[hf], me.count[hf]); };  // that the row sees
        auto fetch = [&](int hf) {
          tmem_load32(S + hf * kPart, x);
          tmem_load32(S + hf * kPart + 32, x + 32);
          fac = *reinterpret_cast<const float4*>(&me.kfac[4 * hf]);
          vlog = *reinterpret_cast<const float4*>(&me.vlog[4 * hf]);
          // not 0, which would make NaN of a hidden token's -inf
          fac = make_float4(fmaxf(fac.x * qs, 1e-37f), fmaxf(fac.y * qs, 1e-37f), fmaxf(fac.z * qs, 1e-37f), fmaxf(fac.w * qs, 1e-37f));
          const int vis = tokens(hf);
          const bool some = __any_sync(0xffffffffu, vis < kPart);
          tmem_loaded();
          settle32(x);
          settle32(x + 32);
          if (some) {
#pragma unroll
            for (int c = 0; c < kPart; ++c) x[c] = c < vis ? x[c] : 0xff800000u;
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
        // What was added up so far, times f: L, the output once its products are done, the weights of the step's
        // first page if that is done. (f is 1 for some rows, a power of two for the others.)
        auto rescale = [&](float f, bool page) {
          L *= f;
          uint32_t y[8];
          if (turn > 0) {
            warp_wait(ok, smem_u32(&sm.pv_done[tile]), (done - 1) & 1, abort, a.err);
            if (!ok) return;
            tmem_after();
#pragma unroll 1
            for (int c = 0; c < kD; c += 8) {
              tmem_load8(O + c, y);
              tmem_loaded();
              settle8(y);
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
              tmem_store8(O + c, y);
            }
          }
          tmem_stored();
          const __half2 f2 = __float2half2_rn(f);
#pragma unroll 1
          for (int c = 0; c < (page ? 32 : 0); c += 8) {
            tmem_load8(S + c, y);
            tmem_loaded();
            settle8(y);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __half2 z = __hmul2(*reinterpret_cast<__half2*>(&y[k]), f2);
              y[k] = *reinterpret_cast<const uint32_t*>(&z);
            }
            tmem_store8(S + c, y);
          }
        };
        if (__any_sync(0xffffffffu, M == -INFINITY)) {  // no reference yet: the step's maximum
          float tm = M, tv = V;
#pragma unroll 1
          for (int hf = 0; hf < halves; ++hf) {
            fetch(hf);
            largest(tm, tv);
          }
          if (M == -INFINITY) M = tm, V = tv;
          aim();
        }
#pragma unroll 1
        for (int hf = 0; hf < halves; ++hf) {
          fetch(hf);
          uint32_t p[32];
          float sum[4];
          float shift = up, most = limit;
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
            fetch(hf);
            float tm = M, tv = V, d = 0.f;
            largest(tm, tv);
            const float above = (tm - M) + (tv - V);
            if (above > 3.f && !wrong) {
              d = above < 64.f ? ceilf(above) : above;
              V = above < 64.f ? V + (d - (tm - M)) : tv;
              M = tm;
            }
            if (__any_sync(0xffffffffu, d > 0.f)) rescale(ex2(-d), hf == 1);
            aim();
            const float at = M == -INFINITY ? 0.f : M;
            auto apart = [&](int grp, float f) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                x[grp * 16 + c] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(x[grp * 16 + c]), f), at));
            };
            apart(0, fac.x), apart(1, fac.y), apart(2, fac.z), apart(3, fac.w);
            fac = make_float4(1.f, 1.f, 1.f, 1.f);
            shift = kUp - V;
          }
          const float4 vinv = *reinterpret_cast<const float4*>(&me.vinv[4 * hf]);
          L += fmaf(sum[0], vinv.x, sum[1] * vinv.y) + fmaf(sum[2], vinv.z, sum[3] * vinv.w);
          tmem_store16(S + hf * kPart, p);  // half of the columns that the scores had
          tmem_store16(S + hf * kPart + 16, p + 16);
        }
        if (!ok) continue;
        // tokens that make NaN of the rows that see them
        for (int hf = 0; hf < halves; ++hf) {
          uint2 bad = *reinterpret_cast<const uint2*>(&me.bad_keys[4 * hf]);
          if (s.from + 2 * step + hf == s.u.pages) {
            const uint2 more = *reinterpret_cast<const uint2*>(&me.bad_vals[4 * hf]);
            bad = make_uint2(bad.x | more.x, bad.y | more.y);
          }
          const int vis = tokens(hf);
          poison |= wrong && vis > 0;
          if (bad.x | bad.y)
            poison |= ((vis < 32 ? bad.x & ((1u << max(vis, 0)) - 1u) : bad.x) |
                       (vis < 64 ? bad.y & ((1u << max(vis - 32, 0)) - 1u) : bad.y)) != 0;
        }
        tmem_stored();
        tmem_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[tile]));
      }
      count += s.steps;

      // ---- the row's end ----
      if (poison) L = __uint_as_float(0x7fc00000u);
      if (my_steps) {
        warp_wait(ok, smem_u32(&sm.pv_done[tile]), (done - 1) & 1, abort, a.err);
        tmem_after();
      }
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
      if (shared ? tile == 0 : s.limit(tile) > 0) {
        const bool whole = s.from == 0 && s.to == s.u.items;
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
          const uint64_t mine_at = reinterpret_cast<uint64_t>(out.p + (int64_t)(s.u.row0 + i) * out.ts + (int64_t)head * out.hs);
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
          const int rows = min(32, s.u.n_new * a.G - (s.first_row + tile * kTile + quad * 32));  // the warp's
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
              if (r < rows && my_steps) *reinterpret_cast<uint4*>(part + r * kPartialStride + 4 + c * 32 + k * 4) = v;
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
    // rows each: their 16-byte stores then fall on eight different columns of the swizzle.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    const int half = warp >= kValueWarp ? 1 : 0;
    const int w4 = warp & 3, c4 = lane & 3, row0 = w4 * 16 + (lane >> 3) * 2 + (lane >> 2 & 1);
    const uint32_t operand0 = half ? sv : sk;
    uint64_t* full = half ? sm.v_full : sm.k_full;
    uint64_t* empty = half ? sm.v_empty : sm.k_empty;
    uint32_t count = 0;
    while (next()) {
      const Segment& s = sm.segs[seg % kSegments];
      const int64_t unit = (int64_t)s.b * a.Hkv + s.h;
      const int pages = min(s.to, s.u.pages);
      int id = -1, pos = -1, id_base = s.from;
      // Page ids of 32 items, a lane each, and for the keys' warps what the softmax has to know of the pages.
      float kfac = 0.f, vlog = 0.f, vinv = 1.f;
      bool bad = false;
      auto look = [&](int first) {
        id_base = first;
        const int it = first + lane;
        id = pos = -1;
        kfac = vlog = 0.f;
        vinv = 1.f;
        bad = false;
        if (it < pages) {
          const int p = topk ? sel[unit * topk + it] : it;
          if (p >= 0 && p < s.u.full) {
            id = a.table[unit * a.max_pages + p];
            if (id < 0 || (int64_t)id >= a.n_pages) {
              if (w4 == 0) atomicOr(a.err, (uint32_t)kErrIndex);
              id = -1;
            } else {
              pos = p * kPart;
              if (!half) {
                const float2 sc = *reinterpret_cast<const float2*>(a.scales + 2 * (int64_t)id);
                bad = !(sc.x == sc.x && sc.y == sc.y);
                kfac = bad ? 0.f : sc.x * fabsf(scale) * kLog2e;
                vlog = bad ? 0.f : scale_log2(sc.y);
                vinv = bad ? 1.f : 1.f / sc.y;
              }
            }
          }
        }
      };
      uint4 raw[8];  // of two pages, four loads each
      auto load = [&](int it, int pg) {
        const int page = it < pages ? __shfl_sync(0xffffffffu, id, it - id_base) : -1;
        const uint8_t* src = a.pages + (int64_t)page * kKv8PageBytes + half * kKv8HalfBytes + row0 * kD + c4 * 16;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          raw[pg * 4 + x] = page >= 0 ? __ldcg(reinterpret_cast<const uint4*>(src + (x >> 1) * 8 * kD + (x & 1) * 64))
                                      : make_uint4(0, 0, 0, 0);
      };
      auto put_page = [&](uint32_t at, int pg) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = row0 + (x >> 1) * 8;
          const uint4 v = raw[pg * 4 + x];
          const uint32_t dst = at + (x & 1) * kPlane + (pg * kPart + row) * 128;
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
          if (row < s.u.tail) t = *(reinterpret_cast<const uint4*>(src + row * kD + c8 * 16) + (x & 1));
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
      look(s.from);
      load(s.from, 0);
      load(s.from + 1, 1);
      for (int step = 0; step < s.steps; ++step, ++count) {
        const uint32_t slot = count & 1, at = operand0 + slot * 16384;
        const int it = s.from + 2 * step, tail = s.u.pages - it;  // the tail's place, if it is in this step
        StepMeta& me = sm.meta[count & 3];
        warp_wait(ok, smem_u32(&empty[slot]), (count >> 1 & 1) ^ 1, abort, a.err);
        if (ok) {
          if (!half) {  // what the softmax has to know of the pages
            const int x = lane - (it - id_base);
            if ((x & ~1) == 0 && it + x < pages) {
              me.kfac[x * 4 + w4] = kfac;
              me.vlog[x * 4 + w4] = vlog;
              me.vinv[x * 4 + w4] = vinv;
              me.bad_keys[x * 4 + w4] = bad ? 0xffffu : 0u;
              if (w4 == 0) me.count[x] = pos >= 0 ? kPart : 0, me.pos[x] = max(pos, 0);
            }
            if (w4 == 0 && lane < 2 && it + lane >= pages) {
              me.count[lane] = it + lane < s.to ? s.u.tail : 0;
              me.pos[lane] = s.u.full * kPart;
            }
          }
          // The next step's loads, each as soon as its registers are free.
          const bool more = it + 2 < pages;
          if (more && it + 2 >= id_base + 32) look(it + 2);  // (32 items are a whole number of steps)
          if (tail > 0) put_page(at, 0);
          if (more) load(it + 2, 0);
          if (tail > 1 && it + 1 < s.to) put_page(at, 1);
          if (more) load(it + 3, 1);
          if (tail <= 1 && it + tail < s.to) put_tail(at, tail, me);
          proxy_fence();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&full[slot]));
        }
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
      uint32_t count = 0, q_phase = 0, p_phase = 0;  // phases: a bit per tile
      const uint64_t dq = operand(sq, 16, 1024), dk = operand(sk, 16, 1024), dv = operand(sv, kPlane, 1024);
      auto scores = [&](int tile, uint32_t c, int pages) {
        const uint32_t d = tmem + kColS + tile * kTile;
        const uint64_t q0 = dq + tile * (kTile * kD * 2 >> 4), k0 = dk + (c & 1) * (16384 >> 4);
        const uint32_t idesc = pages == 2 ? shape(kStep, false) : shape(kPart, false);
        mma_ss<false>(leader, d, q0, k0, idesc);
#pragma unroll
        for (int k = 1; k < 8; ++k)
          mma_ss<true>(leader, d, q0 + ((k >> 2) * (kTile * 128 >> 4) + (k & 3) * 2), k0 + ((k >> 2) * (kPlane >> 4) + (k & 3) * 2), idesc);
        mma_commit(leader, smem_u32(&sm.s_full[tile]));
      };
      auto values = [&](int tile, uint32_t c, int pages, bool add) {
        const uint32_t d = tmem + kColO + tile * kTile, p = tmem + kColS + tile * kTile;
        const uint64_t v0 = dv + (c & 1) * (16384 >> 4);
        if (add) mma_ts<true>(leader, d, p, v0, shape(kD, true));
        else mma_ts<false>(leader, d, p, v0, shape(kD, true));
#pragma unroll
        for (int k = 1; k < 8; ++k) if (k < 4 * pages)
          mma_ts<true>(leader, d, p + (k >> 2) * kPart + (k & 3) * 8, v0 + k * (2048 >> 4), shape(kD, true));
        mma_commit(leader, smem_u32(&sm.pv_done[tile]));
      };
      while (next()) {
        const Segment& s = sm.segs[seg % kSegments];
        auto pages_of = [&](int step) { return min(2, s.to - s.from - 2 * step); };
        if (s.shared()) {  // the tiles take the steps in turn
          const int steps = s.steps;
#pragma unroll 1
          for (int step = -2; step < steps; ++step) {
            const int t = step & 1;
            if (step >= 0) {
              const uint32_t c = count + step;
              wait(sm.v_full[c & 1], c >> 1 & 1);
              wait(sm.p_full[t], p_phase >> t & 1);
              p_phase ^= 1u << t;
              tmem_after();
              if (ok) values(t, c, pages_of(step), step >= 2);
              if (ok) mma_commit(leader, smem_u32(&sm.v_empty[c & 1]));
            }
            if (step + 2 < steps) {
              const uint32_t c = count + step + 2;
              wait(sm.k_full[c & 1], c >> 1 & 1);
              if (step < 0) {
                wait(sm.q_full[t], q_phase >> t & 1);
                q_phase ^= 1u << t;
                tmem_after();
              }
              if (ok) scores(t, c, pages_of(step + 2));
              if (ok) mma_commit(leader, smem_u32(&sm.k_empty[c & 1]));
            }
          }
          count += steps;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[seg % kSegments]));
          ++seg;
          continue;
        }
        wait(sm.k_full[count & 1], count >> 1 & 1);
#pragma unroll 1
        for (int t = 0; t < 2; ++t)
          if (s.active(t, 0)) {
            wait(sm.q_full[t], q_phase >> t & 1);
            q_phase ^= 1u << t;
            tmem_after();
            if (ok) scores(t, count, pages_of(0));
          }
        if (ok) mma_commit(leader, smem_u32(&sm.k_empty[count & 1]));
        for (int step = 0; step < s.steps; ++step, ++count) {
          const int pages = pages_of(step);
          const bool more = step + 1 < s.steps;
          wait(sm.v_full[count & 1], count >> 1 & 1);
          if (more) wait(sm.k_full[(count + 1) & 1], (count + 1) >> 1 & 1);
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            if (s.active(t, step)) {
              wait(sm.p_full[t], p_phase >> t & 1);
              p_phase ^= 1u << t;
              tmem_after();
              if (ok) values(t, count, pages, step > 0);
            }
            if (t == 1 && ok) mma_commit(leader, smem_u32(&sm.v_empty[count & 1]));
            if (more && s.active(t, step + 1) && ok) scores(t, count + 1, pages_of(step + 1));
          }
          if (more && ok) mma_commit(leader, smem_u32(&sm.k_empty[(count + 1) & 1]));
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
    int block = 0;
    int64_t before = pl.before;
    if (warp == kPlanWarp && pl.b < a.B) {  // the share's first block, 32 at a time
      const int64_t at = share_start(pl.total, cta, ctas);
      Unit u = request_of(a, pl.b, false);
      for (;; block += 32) {
        set_rows(a, u, min((int64_t)(block + lane) * kBlockRows, (int64_t)0x7fffff00), kBlockRows, topk);
        const int64_t mine = (int64_t)u.weight * a.Hkv;
        int64_t sum = mine;
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, mine == 0 || at < before + sum);
        if (past) {
          const int l = __ffs(past) - 1;
          before += __shfl_sync(0xffffffffu, sum - mine, l);
          block += l;
          break;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    if (warp == kPlanWarp && lane == 0) {
      int b = pl.b;
      int64_t at = share_start(pl.total, cta, ctas);
      const int64_t stop = share_start(pl.total, cta + 1, ctas);
      JoinRecord open = JoinRecord{};
      Segment s;
      s.u = request_of(a, min(b, a.B - 1), false);
      for (bool more = true; more && ok; ++seg) {
        s.steps = 0;
        while (at < stop && b < a.B) {
          set_rows(a, s.u, block * kBlockRows, kBlockRows, topk);
          if (s.u.weight == 0) {  // the request has no more rows
            if (++b < a.B) s.u = request_of(a, b, false);
            block = 0;
            continue;
          }
          if (at >= before + (int64_t)s.u.weight * a.Hkv) {
            before += (int64_t)s.u.weight * a.Hkv;
            ++block;
            continue;
          }
          const Part x = part_of(s.u, at - before, stop - at);
          at += x.took;
          if (x.from >= x.to) continue;
          if (x.from == 0 && x.to < s.u.items)
            open = record_of(s.u, x.h, block * kBlockRows, pl.total, before + (int64_t)(x.h + 1) * s.u.weight, cta, ctas);
          s.b = b;
          s.h = x.h;
          s.first_row = block * kBlockRows;
          s.from = x.from;
          s.to = x.to;
          s.steps = (x.to - x.from + 1) / 2;
          Unit t = s.u;
          set_rows(a, t, s.first_row, kTile, topk);
          s.limit0 = t.items;
          set_rows(a, t, s.first_row + kTile, kTile, topk);
          s.limit1 = t.items;
          break;
        }
        more = s.steps > 0;
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

int64_t kv8_prefill_workspace() { return (int64_t)2 * kMaxCtas * kBlockRows * kPartialStride * 4; }

cudaError_t launch_kv8_prefill(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel,
                               int topk, void* workspace, int sm_count, cudaStream_t st) {
  const int ctas = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  cudaError_t e = cudaFuncSetAttribute(kv8_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_early(kv8_prefill_kernel, dim3((unsigned)ctas), kThreads, kSmemBytes, st, a, q, out, scale, sel, topk,
                   static_cast<JoinRecord*>(workspace), reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kRecordBytes));
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_kv8_join(a, out, ctas, 16, workspace, kBlockRows, st);
}

}  // namespace spin
