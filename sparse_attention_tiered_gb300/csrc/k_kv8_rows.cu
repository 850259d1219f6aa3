// spin_kv8_attend_rows: attention where every token has its own list of pages.
//
// A first launch makes the lists of tiles of tokens out of those of tokens (kv8_rows.cuh), a second attends them.
#include "kv8_rows.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kWindow = 2048;  // pages that are marked at a time

// A warp a tile. The tokens' pages are marked in a window of shared memory, a bit a token, and read out in order; what lies
// beyond the window waits for the next, which begins at the lowest page that is left.
__global__ void __launch_bounds__(32)
kv8_rows_lists(const Kv8Args a, const int32_t* sel, int topk, RowsSpace s) {
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
      const uint32_t there = __ballot_sync(0xffffffffu, bits != 0);
      if (bits) {
        const int p = base + x + lane, page = table[p];
        Item it;
        it.pos = p * kPart;
        it.page = page;
        it.rows = 0;
        it.reserved = 0;
        const uint32_t group = a.G < 32 ? (1u << a.G) - 1u : 0xffffffffu;
        for (; bits; bits &= bits - 1) it.rows |= group << ((__ffs(bits) - 1) * a.G);
        if (page < 0 || (int64_t)page >= a.n_pages) {
          atomicOr(a.err, (uint32_t)kErrIndex);
          it.page = -1;
        }
        out[count + __popc(there & ((1u << lane) - 1u))] = it;
      }
      count += __popc(there);
    }
    base = next;
    __syncwarp();
  }
  t.items = count + (t.tail && t.see0 + t.tokens - 1 > t.full * kPart ? 1 : 0);
  if (lane == 0) s.tiles[blockIdx.x] = t;
}

// A CTA a tile, a warp a row at a time, a token at a time.
constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
kv8_rows_attend(const Kv8Args a, const Rows q, const Rows out, float scale, int topk, RowsSpace s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x >= *s.tiles_there) return;
  const Tile t = s.tiles[blockIdx.x];
  const int64_t unit = (int64_t)t.b * a.Hkv + t.h;
  const Item* items = s.items + place_of(t, a.Hkv, topk);
  const int listed = t.items - (t.tail && t.see0 + t.tokens - 1 > t.full * kPart ? 1 : 0);
  for (int r = warp; r < t.tokens * a.G; r += kThreads / 32) {
    const int i = r / a.G, head = t.h * a.G + r - i * a.G, see = t.see0 + i;
    const uint2 w = *reinterpret_cast<const uint2*>(q.p + (int64_t)(t.token0 + i) * q.ts + (int64_t)head * q.hs + lane * 4);
    const float qv[4] = {lo_f(w.x), hi_f(w.x), lo_f(w.y), hi_f(w.y)};
    bool poison = false;
    const bool wrong = __any_sync(0xffffffffu, !(fabsf(qv[0]) < INFINITY && fabsf(qv[1]) < INFINITY && fabsf(qv[2]) < INFINITY && fabsf(qv[3]) < INFINITY));
    float M = -INFINITY, L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    auto token = [&](const float* k, const float* v, float kf, float vf) {
      float x = qv[0] * k[0] + qv[1] * k[1] + qv[2] * k[2] + qv[3] * k[3];
      for (int y = 16; y; y >>= 1) x += __shfl_xor_sync(0xffffffffu, x, y);
      x *= kf * scale;
      const float top = fmaxf(M, x), f = M == top ? 1.f : exp2f((M - top) * kLog2e), p = exp2f((x - top) * kLog2e);
      M = top;
      L = L * f + p;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = o[e] * f + p * (v[e] * vf);
    };
    for (int it = 0; it < t.items; ++it) {
      if (it < listed) {
        const Item x = items[it];
        if (!(x.rows >> r & 1) || x.page < 0) continue;
        const float2 sc = *reinterpret_cast<const float2*>(a.scales + 2 * (int64_t)x.page);
        poison |= !(sc.x == sc.x && sc.y == sc.y);
        for (int j = 0; j < kPart && x.pos + j < see; ++j) {
          const uint32_t* at = reinterpret_cast<const uint32_t*>(a.pages + (int64_t)x.page * kKv8PageBytes + j * kD) + lane;
          float kv[2][4];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t c = at[half * (kKv8HalfBytes / 4)];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t f2 = e4m3x2_half2(c, y);
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f2));
              kv[half][2 * y] = f.x;
              kv[half][2 * y + 1] = f.y;
            }
          }
          token(kv[0], kv[1], sc.x, sc.y);
        }
      } else {
        const uint16_t* at = a.tails + unit * kPageElems + lane * 4;
        for (int j = 0; t.full * kPart + j < see; ++j) {
          float kv[2][4];
          bool bad = false;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint2 c = *reinterpret_cast<const uint2*>(at + (half * kPart + j) * kD);
            kv[half][0] = lo_f(c.x), kv[half][1] = hi_f(c.x), kv[half][2] = lo_f(c.y), kv[half][3] = hi_f(c.y);
#pragma unroll
            for (int e = 0; e < 4; ++e) bad |= !(fabsf(kv[half][e]) < INFINITY);
          }
          poison |= __any_sync(0xffffffffu, bad);
          token(kv[0], kv[1], 1.f, 1.f);
        }
      }
    }
    poison |= wrong && (L != 0.f);
    const float inv = poison ? __uint_as_float(0x7fc00000u) : L == 0.f ? 0.f : 1.f / L;
    const __nv_bfloat162 v0 = __floats2bfloat162_rn(o[0] * inv, o[1] * inv), v1 = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(out.p + (int64_t)(t.token0 + i) * out.ts + (int64_t)head * out.hs + lane * 4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
  }
}

int64_t most_tiles(const Kv8Args& a) {
  const int64_t n = a.total_new;
  return (n / tile_tokens(a.G) + (a.B < n ? a.B : n)) * a.Hkv;
}

RowsSpace space_of(const Kv8Args& a, void* workspace) {
  RowsSpace s;
  s.tiles_there = static_cast<int32_t*>(workspace);
  s.tiles = reinterpret_cast<Tile*>(s.tiles_there + 4);
  s.items = reinterpret_cast<Item*>(s.tiles + most_tiles(a));
  return s;
}

}  // namespace

int64_t kv8_rows_workspace(const Kv8Args& a, int topk) {
  return 16 + most_tiles(a) * (int64_t)sizeof(Tile) + (int64_t)a.total_new * a.Hkv * (topk + 1) * (int64_t)sizeof(Item);
}

cudaError_t launch_kv8_rows(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel, int topk,
                            void* workspace, int sm_count, cudaStream_t st) {
  const RowsSpace s = space_of(a, workspace);
  const unsigned tiles = (unsigned)most_tiles(a);
  cudaError_t e = launch_early(kv8_rows_lists, dim3(tiles), 32, 0, st, a, sel, topk, s);
  if (e != cudaSuccess) return e;
  return launch_early(kv8_rows_attend, dim3(tiles), kThreads, 0, st, a, q, out, scale, topk, s);
}

}  // namespace spin
