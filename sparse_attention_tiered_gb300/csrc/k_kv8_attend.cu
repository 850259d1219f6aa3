// spin_kv8_attend: exact attention over the 8-bit paged cache.
//
// Few rows a unit (single tokens, a few drafted ones) read the whole cache once: 256 bytes a
// token and KV head against 4 * 128 * G flops, far below the tensor cores' rate, so the kernel is
// built to keep the memory busy. One persistent CTA per SM takes an equal share of all pages of
// all units in order (a unit may begin and end inside CTAs' shares). A producer warp streams pages
// into a ring of 16 KB slots with one TMA copy each; eight consumer warps take them, four to a
// page with 16 tokens each, every warp with a softmax state and output of its own. Those are
// joined through shared memory at the end of a unit, and over CTAs by a second launch.
//
// Arithmetic. m16n8k16 products on fp16 operands with fp32 sums: rows x dimensions x tokens for
// the scores, rows x tokens x dimensions for the output. Codes go to fp16 exactly; queries and
// tail rows are scaled by a power of two into fp16's range. Each 64-token page has scales k and v:
// with z = score * k * log2(e) + log2(v), the running maximum M of z (not of the score) and
// P = 2^(z - M + 14), the output's weight is P and the softmax sum's is P / v. So blocks whose
// values differ by any factor share one fp16 range, whose 28 binary orders below the largest weight
// are normal numbers.
//
// Operand layout. The k index of a product and the n index may be permuted as long as both
// operands agree, which is chosen so that no byte has to move between lanes: a lane's 16-byte chunk
// of a key row is its own k indices of four products, and 16 bytes of a value row its n index of 16
// products. With the copy's 128-byte swizzle and tokens in the order 0 5 2 7 4 1 6 3, all of these
// 16-byte loads touch every bank once. Values need two tokens of one dimension side by side: one
// byte permutation for two such pairs.
#include "kv8_dev.cuh"

#ifndef FEW_ROWS
#define FEW_ROWS 16
#endif

namespace spin {

namespace {

using namespace kv8;

constexpr int kAccPad = 144;        // floats of a row in the join: 4 x (32 + 4)
constexpr int kMaxTileRows = 32;
constexpr int kMaxConsWarps = 12;
constexpr int kMaxSlots = 10;
constexpr float kShift = 14.f;                          // weights reach 2^14

struct SlotMeta {
  float kfac;  // score factor: page scale * softmax scale * log2(e)
  float vlog;  // log2 of the values' scale
  float vinv;  // 1 / the values' scale
  int pos0;    // position of its first token; -1: nothing to do
};

// The kernel's forms: MT tiles of 16 rows, of which the last has its upper half in use (R = 2) or
// not (R = 1: at most 8 rows, the usual group). Consumer warps come in groups of four; registers
// allow three groups with one tile's output and two with two tiles'. The fourth warpgroup (or third)
// is the producer's, of which one warp works. Registers: 512 threads x 128 at launch = 128 x 56 +
// 384 x 152, or 384 x 168 = 128 x 56 + 256 x 224.
template <int MT>
struct Dec {
  static constexpr int kGroups = MT == 1 ? 3 : 2;
  static constexpr int kPer = MT == 1 ? 3 : 5;  // slots of a group's ring, 16 KB each
  static constexpr int kSlots = kGroups * kPer;
  static constexpr int kWarps = 4 * kGroups;
  static constexpr int kThreads = (kWarps + 4) * 32;
  static constexpr size_t kRingBytes = (size_t)kSlots * kKv8PageBytes;
  static constexpr size_t kJoinBytes = (size_t)kWarps * 8 * kAccPad * 4;
  static constexpr size_t kQBytes = (size_t)8 * MT * 512;
};

struct DecSmem {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  SlotMeta meta[kMaxSlots];
  int64_t scratch[36];
  float m[kMaxConsWarps][8], l[kMaxConsWarps][8];
  int abort;
};

template <int MT>
constexpr size_t dec_smem_bytes() {
  return 1024 + Dec<MT>::kRingBytes + Dec<MT>::kJoinBytes + Dec<MT>::kQBytes + sizeof(DecSmem);
}
static_assert(dec_smem_bytes<1>() <= 232448 && dec_smem_bytes<2>() <= 232448, "shared memory of a CTA");

template <int MT>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(Dec<MT>::kWarps * 32) : "memory");
}

// A warp's softmax state of MT x 16 rows: lane (g, t) has rows g and g + 8 of each, and of them
// dimensions 32 t .. 32 t + 31 of the output: element e of o[j] is row g + 8 (e / 2), dimension
// 32 t + 16 (e % 2) + j.
template <int MT>
struct State {
  float o[MT][16][4];
  float m[MT][2], l[MT][2];
};

// Takes the lane's scores z (four tokens of each of its rows) into the state; fp16 weights come out.
template <int MT, int R>
__device__ __forceinline__ void softmax_step(State<MT>& st, float (&z)[MT][2][4], float vinv, uint4 (&p)[MT]) {
  float top[MT][R];
  bool grew = false;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x = fmaxf(fmaxf(z[mt][0][2 * r], z[mt][0][2 * r + 1]), fmaxf(z[mt][1][2 * r], z[mt][1][2 * r + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      top[mt][r] = fmaxf(st.m[mt][r], x);
      grew |= top[mt][r] > st.m[mt][r];
    }
  if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = top[mt][r] == -INFINITY ? 1.f : ex2(st.m[mt][r] - top[mt][r]);
        st.m[mt][r] = top[mt][r];
        st.l[mt][r] *= f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          st.o[mt][j][2 * r] *= f;
          st.o[mt][j][2 * r + 1] *= f;
        }
      }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    uint32_t w[2][2] = {};  // [row half][token tile]
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float base = st.m[mt][r] == -INFINITY ? -kShift : st.m[mt][r] - kShift;
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = ex2(z[mt][e >> 1][2 * r + (e & 1)] - base);  // a hidden token's z is -inf
      const float s = (y[0] + y[1]) + (y[2] + y[3]);
      st.l[mt][r] += s == 0.f ? 0.f : s * vinv;  // a row that sees nothing here takes nothing of a NaN page
      w[r][0] = pack_half2(y[0], y[1]);
      w[r][1] = pack_half2(y[2], y[3]);
    }
    p[mt] = make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]);
  }
}

// z = score * factor + vlog for the tokens a row may see, else -inf. `tok`: position of the warp's first token.
template <int MT, int R>
__device__ __forceinline__ void finish_scores(float (&z)[MT][2][4], const float (&qs)[MT][2], float kfac, float vlog,
                                              bool masked, int tok, const int (&see)[MT][2], int t) {
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float f = kfac * qs[mt][r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float& x = z[mt][e >> 1][2 * r + (e & 1)];
        x = fmaf(x, f, vlog);
        if (masked && tok + (e >> 1) * 8 + ((e & 1) ? (2 * t) ^ 5 : 2 * t) >= see[mt][r]) x = -INFINITY;
      }
    }
}

template <int MT, int R>
__global__ void __launch_bounds__(Dec<MT>::kThreads, 1)
kv8_decode_kernel(const Kv8Args a, const __grid_constant__ CUtensorMap map, const Rows q, const Rows out, float scale,
                  const int32_t* __restrict__ sel, int topk, JoinRecord* __restrict__ records, float* __restrict__ partials) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* join = reinterpret_cast<float*>(ring + Dec<MT>::kRingBytes);  // [warps][8 rows][kAccPad]
  uint4* qfrag = reinterpret_cast<uint4*>(ring + Dec<MT>::kRingBytes + Dec<MT>::kJoinBytes);  // [8][MT][32]
  DecSmem& sm = *reinterpret_cast<DecSmem*>(ring + Dec<MT>::kRingBytes + Dec<MT>::kJoinBytes + Dec<MT>::kQBytes);
  constexpr int kGroups = Dec<MT>::kGroups, kPer = Dec<MT>::kPer;
  constexpr int kConsWarps = Dec<MT>::kWarps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kRows = R == 1 ? 8 : 16 * MT;
  const int first_row = (int)blockIdx.y * kRows;
  volatile int* abort = &sm.abort;

  if (tid == 0) {
    for (int s = 0; s < Dec<MT>::kSlots; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 4);
    }
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ctas = gridDim.x, cta = blockIdx.x;
  const bool report = cta == 0 && blockIdx.y == 0;
  const Place pl = locate(
      a.B, sm.scratch,
      [&](int x, bool first) { return (int64_t)unit_of(a, x, first_row, kRows, topk, report && first).weight * a.Hkv; },
      [&](int64_t total) { return share_start(total, cta, ctas); });
  const int64_t start = share_start(pl.total, cta, ctas), stop = share_start(pl.total, cta + 1, ctas);
  JoinRecord* record = records + (ctas > 1 ? (int)blockIdx.y * ctas + cta : 0);  // one CTA a tile: never read
  if (start >= stop) {
    if (tid == 0) *record = JoinRecord{};
    return;
  }

  if (warp >= kConsWarps) {
    // ------------------------------ producer ------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp != kConsWarps) return;
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
    JoinRecord open = JoinRecord{};
    bool ok = true;
    int b = pl.b;
    int64_t at = start, before = pl.before;
    while (at < stop) {
      const Unit u = unit_of(a, b, first_row, kRows, topk, false);
      if (u.weight == 0 || at >= before + (int64_t)u.weight * a.Hkv) {
        before += (int64_t)u.weight * a.Hkv;
        ++b;
        continue;
      }
      const Part x = part_of(u, at - before, stop - at);
      at += x.took;
      const int from = x.from, to = x.to;
      if (from >= to) continue;
      if (from == 0 && to < u.items)
        open = record_of(u, x.h, first_row, pl.total, before + (int64_t)(x.h + 1) * u.weight, cta, ctas);
      const int64_t unit = (int64_t)b * a.Hkv + x.h;
      // 32 page ids and scales at a time, a batch ahead of the copies
      int id = -1, pos = -1;
      float2 sc = make_float2(1.f, 1.f);
      auto look = [&](int i) {
        id = pos = -1;
        if (i < min(to, u.pages)) {
          const int p = topk ? sel[unit * topk + i] : i;
          if (p >= 0 && p < u.full) {
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
      look(from + lane);
      for (int base = from; base < min(to, u.pages); base += 32) {
        const int my_id = id, my_pos = pos;
        const float2 my_sc = sc;
        look(base + 32 + lane);
        const int n = min(32, min(to, u.pages) - base);
        for (int i = 0; i < n; ++i) {
          const uint32_t slot = next[0] & 255u, parity = next[0] >> 8;
          if (lane == i) {
            const uint32_t full = smem_u32(&sm.full[slot]);
            ok = ok && mbar_wait(smem_u32(&sm.empty[slot]), parity ^ 1, abort, a.err);
            if (ok) {
              if (my_id >= 0) tma_page(smem_u32(ring) + slot * kKv8PageBytes, &map, my_id, full);
              sm.meta[slot] = SlotMeta{my_sc.x * scale * kLog2e, scale_log2(my_sc.y), 1.f / my_sc.y, my_pos};
              mbar_arrive_expect_tx(full, my_id >= 0 ? kKv8PageBytes : 0);
            }
          }
          __syncwarp();  // slots are filled in order: a lane that ran ahead would take a phase for a later one
          step();
          pass();
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (to > u.pages) {  // the tail: keys in one slot, values in the next
        for (int i = 0; i < 2; ++i) {
          const uint32_t slot = next[0] & 255u, parity = next[0] >> 8;
          if (lane == 0) {
            const uint32_t full = smem_u32(&sm.full[slot]);
            const uint32_t bytes = u.tail * kD * 2;
            ok = ok && mbar_wait(smem_u32(&sm.empty[slot]), parity ^ 1, abort, a.err);
            if (ok) {
              bulk_copy(smem_u32(ring) + slot * kKv8PageBytes, a.tails + unit * kPageElems + i * kPart * kD, bytes, full);
              sm.meta[slot] = SlotMeta{scale * kLog2e, 0.f, 1.f, u.full * kPart};
              mbar_arrive_expect_tx(full, bytes);
            }
          }
          __syncwarp();
          step();
        }
        pass();
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    if (lane == 0) *record = open;
    // No copy may be in flight when the CTA's shared memory goes. The consumers wait for every slot
    // that was filled, unless a wait ran out.
    if (lane == 0 && !ok) settle_down();
    return;
  }

  // ------------------------------ consumers ------------------------------
  if (MT == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
  const int g = lane >> 2, t = lane & 3;
  const int group = warp >> 2, quarter = warp & 3;
  const int pg = (g & 1) ? g ^ 4 : g;                // token order 0 5 2 7 4 1 6 3
  State<MT> st;
  uint32_t slot = group * kPer, parity = 0;  // of the group's own ring
  auto step = [&]() {
    if (++slot == (group + 1) * kPer) slot = group * kPer, parity ^= 1;
  };
  bool ok = true;
  int b = pl.b, turn = 0;
  int64_t at = start, before = pl.before;
  while (at < stop) {
    const Unit u = unit_of(a, b, first_row, kRows, topk, false);
    if (u.weight == 0 || at >= before + (int64_t)u.weight * a.Hkv) {
      before += (int64_t)u.weight * a.Hkv;
      ++b;
      continue;
    }
    const Part x = part_of(u, at - before, stop - at);
    at += x.took;
    const int from = x.from, to = x.to, h = x.h;
    if (from >= to) continue;
    const int rows = min(kRows, u.n_new * a.G - first_row);

    // Queries, as the products want them: lane (g, t) holds dimensions 16 t .. and 64 + 16 t .. of its
    // rows, four to a product. Every warp works out the rows' factors, warp 0 leaves the operands in
    // shared memory. (All warps are past the last unit's products: they have joined its state.)
    float qs[MT][2];
    int see[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        qs[mt][r] = 1.f;
        see[mt][r] = 0;
        const int row = mt * 16 + r * 8 + g;
        const int i = (first_row + row) / a.G, head = h * a.G + (first_row + row) - i * a.G;
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = 0;
        if (row < rows) {
          see[mt][r] = u.past + i + 1;
          const uint4* src = reinterpret_cast<const uint4*>(q.p + (int64_t)(u.row0 + i) * q.ts + (int64_t)head * q.hs);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(w + 4 * x) = src[(x >> 1) * 8 + 2 * t + (x & 1)];
        }
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < 16; ++x) top = __vmaxu2(top, w[x] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = half_exponent(top);
        const float f = pow2(15 - e);
        qs[mt][r] = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2(e - 15);
        if (warp == 0)
#pragma unroll
          for (int x = 0; x < 16; ++x)
            reinterpret_cast<uint32_t*>(&qfrag[((x >> 1) * MT + mt) * 32 + lane])[(x & 1) * 2 + r] =
                pack_half2(lo_f(w[x]) * f, hi_f(w[x]) * f);
      }
    consumers_sync<MT>();
    auto query = [&](int mt, int k) -> uint4 { return qfrag[(k * MT + mt) * 32 + lane]; };

#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        st.m[mt][r] = -INFINITY;
        st.l[mt][r] = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) st.o[mt][j][2 * r] = st.o[mt][j][2 * r + 1] = 0.f;
      }

    for (int it = from; it < to; ++it, turn = turn + 1 == kGroups ? 0 : turn + 1) {
      if (turn != group) continue;
      if (it < u.pages) {
        {
          ok = mbar_wait(smem_u32(&sm.full[slot]), parity, abort, a.err) && ok;
          ok = __all_sync(0xffffffffu, ok);
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
            float z[MT][2][4], z1[MT][2][4];  // even and odd products apart: shorter chains
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[mt][i][e] = z1[mt][i][e] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const uint4 qk = query(mt, k);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t w = reinterpret_cast<const uint32_t*>(&kr[i][k >> 2])[k & 3];
                  mma_f16(k & 1 ? z1[mt][i] : z[mt][i], qk, e4m3x2_half2(w, false), e4m3x2_half2(w, true));
                }
              }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2 * R; ++e) z[mt][i][e] += z1[mt][i][e];
            uint4 vr[4];  // value rows 2 t, (2 t) ^ 5, and those 8 further
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int row = (x & 1) ? (2 * t) ^ 5 : 2 * t;
              vr[x] = lds128(vals + ((x >> 1) * 8 + row) * kD + ((g ^ row) << 4));
            }
            const int pos = me.pos0 + quarter * 16;
            finish_scores<MT, R>(z, qs, me.kfac, me.vlog, me.pos0 + kPart > u.past + 1, pos, see, t);
            uint4 p[MT];
            softmax_step<MT, R>(st, z, me.vinv, p);
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
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t b0 = e4m3x2_half2(lo, e), b1 = e4m3x2_half2(hi, e);
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) mma_f16(st.o[mt][4 * x + 2 * y + e], p[mt], b0, b1);
                }
              }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
        }
        step();
        continue;
      }
      // The tail. Rows are bf16; each warp scales its 16 tokens' keys, and values, by a power of two.
      const uint32_t s0 = slot, p0 = parity;
      step();
      const uint32_t s1 = slot;
      {
        ok = mbar_wait(smem_u32(&sm.full[s0]), p0, abort, a.err) && ok;
        ok = mbar_wait(smem_u32(&sm.full[s1]), parity, abort, a.err) && ok;
        ok = __all_sync(0xffffffffu, ok);
        const SlotMeta me = sm.meta[s0];
        const int have = u.tail - quarter * 16;  // of this warp's tokens
        if (ok && have > 0) {
          const uint32_t keys = smem_u32(ring) + s0 * kKv8PageBytes + quarter * 16 * kD * 2;
          const uint32_t vals = smem_u32(ring) + s1 * kKv8PageBytes + quarter * 16 * kD * 2;
          uint32_t bad[2][2];  // tokens of the lane's columns that hold something not finite
          // keys: per token tile, 16 + 16 dimensions of the lane's token
          uint4 kr[2][4];
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t wrong = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint4 w = make_uint4(0, 0, 0, 0);
              if (i * 8 + pg < have) w = lds128(keys + (i * 8 + pg) * kD * 2 + ((x >> 1) * 8 + 2 * t + (x & 1)) * 16);
              uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t inf_lo = (ww[y] & 0x7f80u) == 0x7f80u, inf_hi = (ww[y] & 0x7f800000u) == 0x7f800000u;
                wrong |= inf_lo | inf_hi;
                if (inf_lo) ww[y] &= 0xffff0000u;
                if (inf_hi) ww[y] &= 0x0000ffffu;
                top = __vmaxu2(top, ww[y] & 0x7fff7fffu);
              }
              kr[i][x] = w;
            }
            const uint32_t who = __ballot_sync(0xffffffffu, wrong != 0);
            bad[i][0] = who >> (8 * t) & 0xfu;
            bad[i][1] = who >> (8 * t + 4) & 0xfu;
          }
          top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
          const int ke = half_exponent(top);
          const float kf = pow2(15 - ke);
          float z[MT][2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) z[mt][i][0] = z[mt][i][1] = z[mt][i][2] = z[mt][i][3] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t* ww = reinterpret_cast<const uint32_t*>(&kr[i][k >> 1]);
              const uint32_t w0 = ww[(k & 1) * 2], w1 = ww[(k & 1) * 2 + 1];
              const uint32_t b0 = pack_half2(lo_f(w0) * kf, hi_f(w0) * kf), b1 = pack_half2(lo_f(w1) * kf, hi_f(w1) * kf);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma_f16(z[mt][i], query(mt, k), b0, b1);
            }
          }
          // values: four tokens' 16 dimensions
          uint4 vr[4][2];
          top = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = (x >> 1) * 8 + ((x & 1) ? (2 * t) ^ 5 : 2 * t);
            uint32_t wrong = 0;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint4 w = make_uint4(0, 0, 0, 0);
              if (row < have) w = lds128(vals + row * kD * 2 + (2 * g + y) * 16);
              uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t inf_lo = (ww[c] & 0x7f80u) == 0x7f80u, inf_hi = (ww[c] & 0x7f800000u) == 0x7f800000u;
                wrong |= inf_lo | inf_hi;
                if (inf_lo) ww[c] &= 0xffff0000u;
                if (inf_hi) ww[c] &= 0x0000ffffu;
                top = __vmaxu2(top, ww[c] & 0x7fff7fffu);
              }
              vr[x][y] = w;
            }
            const uint32_t who = __ballot_sync(0xffffffffu, wrong != 0);
            bad[x >> 1][x & 1] |= who & (0x11111111u << t);
          }
          top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
          const int ve = half_exponent(top);
          const float vf = pow2(15 - ve);
          finish_scores<MT, R>(z, qs, me.kfac * pow2(ke - 15), (float)(ve - 15), true, me.pos0 + quarter * 16, see, t);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (bad[i][e & 1] && z[mt][i][e] != -INFINITY) z[mt][i][e] = __uint_as_float(0x7fc00000u);
          uint4 p[MT];
          softmax_step<MT, R>(st, z, vf, p);
#pragma unroll
          for (int y = 0; y < 8; ++y) {  // words of two dimensions
            const uint32_t w0 = reinterpret_cast<const uint32_t*>(&vr[0][y >> 2])[y & 3];
            const uint32_t w1 = reinterpret_cast<const uint32_t*>(&vr[1][y >> 2])[y & 3];
            const uint32_t w2 = reinterpret_cast<const uint32_t*>(&vr[2][y >> 2])[y & 3];
            const uint32_t w3 = reinterpret_cast<const uint32_t*>(&vr[3][y >> 2])[y & 3];
            const uint32_t b0 = pack_half2(lo_f(w0) * vf, lo_f(w1) * vf), b1 = pack_half2(lo_f(w2) * vf, lo_f(w3) * vf);
            const uint32_t d0 = pack_half2(hi_f(w0) * vf, hi_f(w1) * vf), d1 = pack_half2(hi_f(w2) * vf, hi_f(w3) * vf);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_f16(st.o[mt][2 * y], p[mt], b0, b1);
              mma_f16(st.o[mt][2 * y + 1], p[mt], d0, d1);
            }
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm.empty[s0]));
          mbar_arrive(smem_u32(&sm.empty[s1]));
        }
      }
      step();
    }

    // ---- the unit's part of this CTA is done: join the warps' states, 8 rows at a time ----
    const bool whole = from == 0 && to == u.items;
    const int pslot = 2 * ((int)blockIdx.y * ctas + cta) + (from == 0 ? 1 : 0);
#pragma unroll
    for (int part = 0; part < 2 * MT; ++part) {
      const int mt = part >> 1, r = part & 1;
      if (part * 8 >= rows) break;
      consumers_sync<MT>();  // the join area is free again
      float l = st.l[mt][r];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (t == 0) {
        sm.m[warp][g] = st.m[mt][r];
        sm.l[warp][g] = l;
      }
      float* dst = join + (warp * 8 + g) * kAccPad + t * 36;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(dst + 16 * e + j) =
              make_float4(st.o[mt][j][2 * r + e], st.o[mt][j + 1][2 * r + e], st.o[mt][j + 2][2 * r + e], st.o[mt][j + 3][2 * r + e]);
      consumers_sync<MT>();
      const int mine = tid >> 5, d0 = lane * 4, row = part * 8 + mine;  // a warp a row, four dimensions a lane
      if (mine < 8 && row < rows) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kConsWarps; ++w) M = fmaxf(M, sm.m[w][mine]);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kConsWarps; ++w) {
          const float f = ex2(sm.m[w][mine] - base);
          L += sm.l[w][mine] * f;
          const float4 x = *reinterpret_cast<const float4*>(join + (w * 8 + mine) * kAccPad + (d0 >> 5) * 36 + (d0 & 31));
          o = make_float4(o.x + x.x * f, o.y + x.y * f, o.z + x.z * f, o.w + x.w * f);
        }
        if (whole) {
          const int i = (first_row + row) / a.G, head = h * a.G + (first_row + row) - i * a.G;
          const float inv = L == 0.f ? 0.f : 1.f / L;
          const __nv_bfloat162 v0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), v1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
          *reinterpret_cast<uint2*>(out.p + (int64_t)(u.row0 + i) * out.ts + (int64_t)head * out.hs + d0) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
        } else {
          float* to_part = partials + ((int64_t)pslot * kMaxTileRows + row) * kPartialStride;
          if (lane == 0) *reinterpret_cast<float2*>(to_part) = make_float2(M, L);
          *reinterpret_cast<float4*>(to_part + 4 + d0) = o;
        }
      }
    }
  }
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

template <int MT, int R>
cudaError_t launch_decode(const Kv8Args& a, const CUtensorMap& map, const Rows& q, const Rows& out, float scale,
                          const int32_t* sel, int topk, void* workspace, int sm_count, cudaStream_t st) {
  const int rows = R == 1 ? 8 : 16 * MT;
  const int64_t tiles = ((int64_t)a.max_new * a.G + rows - 1) / rows;
  if (tiles > 65535) return cudaErrorInvalidConfiguration;
  const int sms = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  const int ctas = tiles >= sms ? 1 : (int)(sms / tiles);  // a tile; ctas > 1 only if all of them fit the workspace
  cudaError_t e = cudaFuncSetAttribute(kv8_decode_kernel<MT, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dec_smem_bytes<MT>());
  if (e != cudaSuccess) return e;
  kv8_decode_kernel<MT, R><<<dim3((unsigned)ctas, (unsigned)tiles), Dec<MT>::kThreads, dec_smem_bytes<MT>(), st>>>(
      a, map, q, out, scale, sel, topk, static_cast<JoinRecord*>(workspace),
      reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kRecordBytes));
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_kv8_join(a, out, ctas, (int)tiles, rows, workspace, kMaxTileRows, st);
}

}  // namespace

int64_t kv8_attend_workspace(const Kv8Args&) {
  const int64_t few = (int64_t)2 * kMaxCtas * kMaxTileRows * kPartialStride * 4, many = kv8_prefill_workspace();
  return (int64_t)kRecordBytes + (few > many ? few : many);
}

cudaError_t launch_kv8_attend(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel,
                              int topk, void* workspace, int sm_count, cudaStream_t st) {
  if ((int64_t)a.max_new * a.G > FEW_ROWS) return launch_kv8_prefill(a, q, out, scale, sel, topk, workspace, sm_count, st);
  CUtensorMap map;
  const cudaError_t e = page_map(a, &map);
  if (e != cudaSuccess) return e;
  if ((int64_t)a.max_new * a.G <= 8) return launch_decode<1, 1>(a, map, q, out, scale, sel, topk, workspace, sm_count, st);
  if ((int64_t)a.max_new * a.G <= 16) return launch_decode<1, 2>(a, map, q, out, scale, sel, topk, workspace, sm_count, st);
  return launch_decode<2, 2>(a, map, q, out, scale, sel, topk, workspace, sm_count, st);
}

}  // namespace spin
