// spin_kv8_append: position rotation of a step's queries and keys, and the append of its keys
// and values to the 8-bit paged cache, in one launch.
//
// A pair (x0, x1) at position n turns by n * f_j: y0 = x0 cos - x1 sin, y1 = x0 sin + x1 cos.
// The angle is n * step mod 2^64 in 2^-64 turns. Its top 6 bits pick one of 64 tabulated angles a, the
// rest is |d| <= 2 pi / 128, and cos(a + d) = cos a + (cos a (cos d - 1) - sin a sin d) with short
// Taylor sums of cos d - 1 and sin d: as a pair (16 tabulated bits, a float), cos and sin are right to
// 2^-28. Keys use the pair (16 bits x 8 bits of a bf16 are exact in fp32), so that a key's bf16, and
// through it the page's codes, is the exact product's rounding in all but about 2^-16 of the
// elements; queries use the plain fp32 sum. (A table of 256 entries has 2 bits more, and its gathers touch
// four times the L1 lines.)
//
// The work is memory bound: a prompt token reads (Hq + 2 Hkv) rows of 256 bytes and writes Hq
// rows and 2 Hkv rows of 128. Two kinds of CTAs share the launch:
//   rows (one warp per token and some of its heads): queries, and the keys and values that stay in
//     bf16. Eight lanes a row, so a lane's angles serve all heads of its token; two passes' loads at
//     a time;
//   page items (one CTA per completed page and KV head): 64 rows of keys and values in registers,
//     8 lanes a row with 16 elements each, one maximum over them, codes out. The page's maximum
//     is what its elements wait for, so nothing is read twice.
// Measured: a prompt of 8191 tokens, 40 query and 8 KV heads: 218 MB in 51 us, 4.3 TB/s, 0.63 of the copy's rate (53 us
// without the launch that begins while the last one ends).
// Nothing is saturated (DRAM 45%, issue slots 49%, by sines, rotations and rounding): a warp of the rows has two
// passes' loads in flight, and none while it computes. More CTAs an SM (48 registers a thread) spill and take 12%
// longer, page items between the rows 5%, before them the same. 256 requests of one token: 9.5 us,
// one chain of dependent loads.
// A request that completes a page leaves its remaining rows to the page item of its first
// completed page, which has read the old tail by then: no other CTA touches that tail.
#include "kv8.cuh"

namespace spin {

namespace {

constexpr int kThreads = 256;

constexpr int kTurnBits = 6;
constexpr int kTurns = 1 << kTurnBits;

// cos and sin of 2 pi i / kTurns: hi a multiple of 2^-15, lo the rest.
struct Turn {
  float ch, cl, sh, sl;
};
struct alignas(16) TurnTable {
  Turn t[kTurns];
};

constexpr double taylor(double x, bool sine) {
  double term = sine ? x : 1.0, sum = 0.0;
  for (int n = sine ? 1 : 0; n < 40; n += 2) {
    sum += term;
    term *= -x * x / ((n + 1) * (n + 2));
  }
  return sum;
}

constexpr double hi_part(double x) { return (double)(long long)(x * 32768.0) / 32768.0; }

constexpr TurnTable make_turns() {
  TurnTable r{};
  for (int i = 0; i < kTurns; ++i) {
    // the first octant's values, mirrored: exact zeros and ones on the axes
    const int quarter = kTurns / 4, q = i / quarter, m = i % quarter;
    const double step = 6.283185307179586476925 / kTurns;
    const double a = 2 * m <= quarter ? taylor(m * step, false) : taylor((quarter - m) * step, true);
    const double b = 2 * m <= quarter ? taylor(m * step, true) : taylor((quarter - m) * step, false);
    const double c = q == 0 ? a : q == 1 ? -b : q == 2 ? -a : b;
    const double s = q == 0 ? b : q == 1 ? a : q == 2 ? -b : -a;
    r.t[i].ch = (float)hi_part(c);
    r.t[i].cl = (float)(c - hi_part(c));
    r.t[i].sh = (float)hi_part(s);
    r.t[i].sl = (float)(s - hi_part(s));
  }
  return r;
}

__device__ const TurnTable g_turns = make_turns();

__device__ __forceinline__ Turn turn_of(uint64_t phase) {
  const uint32_t i = (uint32_t)((phase + (1ull << (63 - kTurnBits))) >> (64 - kTurnBits));  // nearest, mod kTurns
  const int64_t d = (int64_t)(phase - ((uint64_t)i << (64 - kTurnBits)));                   // within half a step
  const float4 t = __ldg(reinterpret_cast<const float4*>(&g_turns.t[i & (kTurns - 1)]));
  const float x = (float)(int32_t)(d >> 26) * (6.2831853071795865f / 274877906944.f);  // radians; 2^38
  const float x2 = x * x;
  const float sd = fmaf(x * x2, fmaf(x2, 1.f / 120.f, -1.f / 6.f), x);
  const float cd = x2 * fmaf(x2, 1.f / 24.f, -0.5f);  // cos d - 1
  const float C = t.x + t.y, S = t.z + t.w;
  Turn r;
  r.ch = t.x;
  r.cl = t.y + fmaf(C, cd, -(S * sd));
  r.sh = t.z;
  r.sl = t.w + fmaf(S, cd, C * sd);
  return r;
}

// p + r + lo for exact products p and r: their rounding error is kept, the sum is rounded once.
__device__ __forceinline__ float sum_exact(float p, float r, float lo) {
  const float s = __fadd_rn(p, r);
  const float bb = __fsub_rn(s, p);
  const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(s, bb)), __fsub_rn(r, bb));
  return __fadd_rn(s, __fadd_rn(e, lo));
}

template <bool EXACT>
__device__ __forceinline__ void rotate_pair(float x0, float x1, const Turn& t, float& y0, float& y1) {
  if (EXACT) {
    y0 = sum_exact(__fmul_rn(x0, t.ch), __fmul_rn(-x1, t.sh), fmaf(x0, t.cl, -(x1 * t.sl)));
    y1 = sum_exact(__fmul_rn(x0, t.sh), __fmul_rn(x1, t.ch), fmaf(x0, t.sl, x1 * t.cl));
  } else {
    const float c = t.ch + t.cl, s = t.sh + t.sl;
    y0 = fmaf(x0, c, -(x1 * s));
    y1 = fmaf(x0, s, x1 * c);
  }
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Lane i of the 8 lanes of a row holds two 16-byte chunks of it (8 elements each): with split
// pairs, chunk i and its partner half a rotation further; past the rotated part, and with
// interleaved pairs, two neighbours. Either way its pairs are 8 i .. 8 i + 7.
__device__ __forceinline__ void lane_chunks(const RopeArgs& r, int i, int& c0, int& c1) {
  const int n = r.half / 8;  // rotating lanes
  if (i < n && !r.interleaved) {
    c0 = i;
    c1 = i + n;
  } else {
    c0 = 2 * i;
    c1 = 2 * i + 1;
  }
}

// The lane's pairs of a row, turned: pair j of turn(j).
template <bool EXACT, typename T>
__device__ __forceinline__ void lane_rotate(const RopeArgs& r, int i, T turn, uint4& a, uint4& b) {
  if (8 * i >= r.half) return;
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
  if (r.interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y0, y1;
      rotate_pair<EXACT>(lo_f(wa[j]), hi_f(wa[j]), turn(j), y0, y1);
      wa[j] = pack(y0, y1);
      rotate_pair<EXACT>(lo_f(wb[j]), hi_f(wb[j]), turn(4 + j), y0, y1);
      wb[j] = pack(y0, y1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y0, y1, z0, z1;
      rotate_pair<EXACT>(lo_f(wa[j]), lo_f(wb[j]), turn(2 * j), y0, y1);
      rotate_pair<EXACT>(hi_f(wa[j]), hi_f(wb[j]), turn(2 * j + 1), z0, z1);
      wa[j] = pack(y0, z0);
      wb[j] = pack(y1, z1);
    }
  }
}

// A key's row: the angles are worked out one by one, which holds few registers. One copy of it: a short call is
// over before the code of four would have been fetched.
struct TwoChunks {
  uint4 a, b;
};
__device__ __noinline__ TwoChunks rotate_key(const RopeArgs& r, int i, int64_t pos, TwoChunks x) {
  lane_rotate<true>(r, i, [&](int j) { return turn_of((uint64_t)pos * r.step[8 * i + j]); }, x.a, x.b);
  return x;
}
__device__ __forceinline__ void lane_rotate_key(const RopeArgs& r, int i, int64_t pos, uint4& a, uint4& b) {
  const TwoChunks y = rotate_key(r, i, pos, TwoChunks{a, b});
  a = y.a;
  b = y.b;
}

// The largest b in [0, B) with f(b) <= x, for ascending f with f(0) <= x; any b in range otherwise.
// The warp probes 32 places at a time.
template <typename F>
__device__ __forceinline__ int warp_find(int B, int x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, lane == 0 || (at < n && f(lo + at) <= x));
    // the leading run of lanes that are <= x: for ascending f that is all of them
    const int k = (le == 0xffffffffu ? 32 : __ffs(~le) - 1) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

__device__ __forceinline__ uint4 abs_max(uint4 m, uint4 x) {
  m.x = __vmaxu2(m.x, x.x & 0x7fff7fffu);
  m.y = __vmaxu2(m.y, x.y & 0x7fff7fffu);
  m.z = __vmaxu2(m.z, x.z & 0x7fff7fffu);
  m.w = __vmaxu2(m.w, x.w & 0x7fff7fffu);
  return m;
}

__device__ __forceinline__ uint32_t fold(uint4 m) {
  const uint32_t w = __vmaxu2(__vmaxu2(m.x, m.y), __vmaxu2(m.z, m.w));
  return max(w & 0xffffu, w >> 16);
}

// The scale of a half whose largest |x| has these bf16 bits, and its inverse (both powers of
// two): 448 = 0.875 * 2^9, so x = m 2^e with m in [0.5, 1) wants 2^(e-9), or 2^(e-8) above 0.875.
__device__ __forceinline__ void scale_of(uint32_t amax, float& scale, float& inv) {
  if (amax >= 0x7f80u) {  // an infinity or a NaN: the half is NaN, its codes are 0
    scale = __uint_as_float(0x7fc00000u);
    inv = 0.f;
    return;
  }
  int e = (int)(amax >> 7) - 126;   // amax = m 2^e (subnormals: below any used scale)
  const uint32_t m = amax & 0x7fu;  // 0.5 (1 + m / 128) > 0.875 when m > 96
  e = max(e - 9 + (m > 96u ? 1 : 0), kKv8MinScaleExp);
  scale = __uint_as_float((uint32_t)(e + 127) << 23);
  inv = __uint_as_float((uint32_t)(127 - e) << 23);
}

__device__ __forceinline__ uint32_t code2(uint32_t w, float inv, bool zero) {
  if (zero) return 0u;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi_f(w) * inv), "f"(lo_f(w) * inv));
  return r;
}

__device__ __forceinline__ uint2 codes8(uint4 x, float inv, bool zero) {
  return make_uint2(code2(x.x, inv, zero) | code2(x.y, inv, zero) << 16,
                    code2(x.z, inv, zero) | code2(x.w, inv, zero) << 16);
}

__device__ __forceinline__ const uint4* chunk(const Rows& r, int64_t t, int64_t h, int c) {
  return reinterpret_cast<const uint4*>(r.p + t * r.ts + h * r.hs) + c;
}

__device__ __forceinline__ int64_t position(const RopeArgs& r, int row, int64_t fallback) {
  return r.positions ? (int64_t)r.positions[row] : fallback;
}

__global__ void __launch_bounds__(kThreads, 4)
kv8_append_kernel(const Kv8Args a, const __grid_constant__ RopeArgs r, const Rows q, const Rows q_out, const Rows k,
                  const Rows v, int row_ctas, int iters) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i8 = lane & 7;
  int c0, c1;
  lane_chunks(r, i8, c0, c1);
  // The launch may begin before what is before it on the stream has ended; nothing in memory is touched until then.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if ((int)blockIdx.x >= row_ctas) {
    // ---- a completed page of one head ----
    // Request b owns the items cu[b] / 64 + b .. : its completed pages are at most
    // (63 + new) / 64, which is no more than the items before request b + 1. With one new token a
    // request at most, request b has item b.
    __shared__ uint32_t s_max[2][kThreads / 32];
    __shared__ __align__(16) uint16_t s_keys[kPart * kD];
    const int place = (int)blockIdx.x - row_ctas, item = place / a.Hkv, h = place - item * a.Hkv;
    const bool single = a.max_new == 1;
    const int b = single ? item : warp_find(a.B, item, [&](int x) { return (a.cu[x] >> 6) + x; });
    int row0, n_new, past;
    if (!kv8_request(a, b, false, row0, n_new, past)) return;
    const int j = single ? 0 : item - ((row0 >> 6) + b);
    const int old = past & (kPart - 1);             // rows in the tail
    const int p0 = past >> 6;
    const int n_done = (old + n_new) >> 6;          // pages completed by this step
    if (j < 0 || j >= n_done) return;
    const int64_t unit = (int64_t)b * a.Hkv + h;
    uint16_t* tail = a.tails + unit * kPageElems;
    const int page = a.table[unit * a.max_pages + p0 + j];
    const bool ok = page >= 0 && (int64_t)page < a.n_pages;
    if (!ok && tid == 0) atomicOr(a.err, kErrIndex);

    uint4 kk[2][2], vv[2][2];
    uint4 mk = make_uint4(0, 0, 0, 0), mv = mk;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = u * 32 + (tid >> 3);
      const int t = j * kPart + row - old;  // the new token of this row; below 0: a row of the tail
      if (t < 0) {
        const uint4* src = reinterpret_cast<const uint4*>(tail + row * kD);
        kk[u][0] = src[c0];
        kk[u][1] = src[c1];
        vv[u][0] = src[c0 + kPart * kD / 8];
        vv[u][1] = src[c1 + kPart * kD / 8];
      } else {
        kk[u][0] = *chunk(k, row0 + t, h, c0);
        kk[u][1] = *chunk(k, row0 + t, h, c1);
        vv[u][0] = *chunk(v, row0 + t, h, c0);
        vv[u][1] = *chunk(v, row0 + t, h, c1);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = u * 32 + (tid >> 3);
      const int t = j * kPart + row - old;
      if (t >= 0) {
        lane_rotate_key(r, i8, position(r, row0 + t, (int64_t)past + t), kk[u][0], kk[u][1]);
      }
      mk = abs_max(abs_max(mk, kk[u][0]), kk[u][1]);
      mv = abs_max(abs_max(mv, vv[u][0]), vv[u][1]);
      if (a.summaries) {
        *reinterpret_cast<uint4*>(s_keys + row * kD + 8 * c0) = kk[u][0];
        *reinterpret_cast<uint4*>(s_keys + row * kD + 8 * c1) = kk[u][1];
      }
    }
    const uint32_t wk = __reduce_max_sync(0xffffffffu, fold(mk)), wv = __reduce_max_sync(0xffffffffu, fold(mv));
    if (lane == 0) {
      s_max[0][warp] = wk;
      s_max[1][warp] = wv;
    }
    __syncthreads();  // also: every old row of the tail has been read
    uint32_t ak = 0, av = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      ak = max(ak, s_max[0][w]);
      av = max(av, s_max[1][w]);
    }
    float sk, ik, sv, iv;
    scale_of(ak, sk, ik);
    scale_of(av, sv, iv);
    if (ok) {
      uint8_t* dst = a.pages + (int64_t)page * kKv8PageBytes;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = u * 32 + (tid >> 3);
        uint2* dk = reinterpret_cast<uint2*>(dst + row * kD);
        uint2* dv = reinterpret_cast<uint2*>(dst + kKv8HalfBytes + row * kD);
        dk[c0] = codes8(kk[u][0], ik, ik == 0.f);
        dk[c1] = codes8(kk[u][1], ik, ik == 0.f);
        dv[c0] = codes8(vv[u][0], iv, iv == 0.f);
        dv[c1] = codes8(vv[u][1], iv, iv == 0.f);
      }
      if (tid == 0) *reinterpret_cast<float2*>(a.scales + 2 * (int64_t)page) = make_float2(sk, sv);
      if (a.summaries && tid < kD) {
        // row order, as Index + Offload sums a partition
        float s = 0.f;
        for (int row = 0; row < kPart; ++row) s += __uint_as_float((uint32_t)s_keys[row * kD + tid] << 16);
        a.summaries[(unit * a.max_pages + p0 + j) * kD + tid] = s / (float)kPart;
      }
    }
    if (j == 0) {  // the rows behind the request's last completed page
      const int rest = (old + n_new) & (kPart - 1);
      for (int row = tid >> 3; row < rest; row += kThreads / 8) {
        const int t = n_done * kPart + row - old;
        uint4 x0 = *chunk(k, row0 + t, h, c0), x1 = *chunk(k, row0 + t, h, c1);
        lane_rotate_key(r, i8, position(r, row0 + t, (int64_t)past + t), x0, x1);
        uint4* dst = reinterpret_cast<uint4*>(tail + row * kD);
        dst[c0] = x0;
        dst[c1] = x1;
        dst[c0 + kPart * kD / 8] = *chunk(v, row0 + t, h, c0);
        dst[c1 + kPart * kD / 8] = *chunk(v, row0 + t, h, c1);
      }
    }
    return;
  }

  // ---- rows: queries, and keys and values of requests that complete no page ----
  const int n_q = q.p ? a.Hq : 0, q_groups = (n_q + 3) / 4;  // of 4 rows: one warp pass
  const int groups = q_groups + (2 * a.Hkv + 3) / 4;
  const int per_token = (groups + iters - 1) / iters;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  const int t = (int)(w / per_token);
  if (t >= a.total_new) return;
  const int part = (int)(w - (int64_t)t * per_token);
  // With one new token a request, which is most calls, row t is request t.
  int b = min(t, a.B - 1);
  if (!(a.cu[b] <= t && t < a.cu[b + 1])) b = warp_find(a.B, t, [&](int x) { return a.cu[x]; });
  int row0, n_new, past;
  const bool good = kv8_request(a, b, part == 0 && lane == 0, row0, n_new, past);
  if (!good || t < row0 || t >= row0 + n_new) return;  // padding, or a request that is left out
  const int64_t pos = position(r, t, (int64_t)past + (t - row0));
  const int first = part * iters, last = min(groups, first + iters), sub = lane >> 3;
  if (first < q_groups) {
    float2 turns[8];
    if (8 * i8 < r.half) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Turn x = turn_of((uint64_t)pos * r.step[8 * i8 + j]);
        turns[j] = make_float2(x.ch + x.cl, x.sh + x.sl);
      }
    }
    auto turn = [&](int j) { return Turn{turns[j].x, 0.f, turns[j].y, 0.f}; };
    for (int g = first; g < min(last, q_groups); g += 2) {
      uint4 x[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (g + k) * 4 + sub;
        if (g + k < last && row < n_q) {
          x[k][0] = *chunk(q, t, row, c0);
          x[k][1] = *chunk(q, t, row, c1);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (g + k) * 4 + sub;
        if (g + k < last && row < n_q) {
          lane_rotate<false>(r, i8, turn, x[k][0], x[k][1]);
          uint4* dst = reinterpret_cast<uint4*>(q_out.p + (int64_t)t * q_out.ts + (int64_t)row * q_out.hs);
          dst[c0] = x[k][0];
          dst[c1] = x[k][1];
        }
      }
    }
  }
  if ((past & (kPart - 1)) + n_new >= kPart) return;  // the page items take the keys and values
  for (int g = max(first, q_groups); g < last; ++g) {
    const int row = (g - q_groups) * 4 + sub;
    if (row >= 2 * a.Hkv) continue;
    const int h = row < a.Hkv ? row : row - a.Hkv;
    uint16_t* tail = a.tails + ((int64_t)b * a.Hkv + h) * kPageElems + ((past & (kPart - 1)) + (t - row0)) * kD;
    uint4 x0, x1;
    if (row < a.Hkv) {
      x0 = *chunk(k, t, h, c0);
      x1 = *chunk(k, t, h, c1);
      lane_rotate_key(r, i8, pos, x0, x1);
    } else {
      x0 = *chunk(v, t, h, c0);
      x1 = *chunk(v, t, h, c1);
      tail += kPart * kD;
    }
    reinterpret_cast<uint4*>(tail)[c0] = x0;
    reinterpret_cast<uint4*>(tail)[c1] = x1;
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Args& a, const RopeArgs& r, const Rows& q, const Rows& q_out, const Rows& k,
                              const Rows& v, int sm_count, cudaStream_t st) {
  const int64_t page_items = (a.max_new == 1 ? (int64_t)a.B : (int64_t)a.total_new / kPart + a.B) * a.Hkv;
  const int groups = ((q.p ? a.Hq : 0) + 3) / 4 + (2 * a.Hkv + 3) / 4;
  // Few tokens: spread a token's rows over warps, one pass each. Many: a warp keeps its token's angles
  // for more of its rows, as long as there are some waves of warps.
  const int64_t warps_wanted = (int64_t)sm_count * 128;
  int64_t iters = (int64_t)a.total_new * groups / warps_wanted;
  iters = iters < 1 ? 1 : iters > groups ? groups : iters;
  const int64_t per_token = (groups + iters - 1) / iters;
  const int64_t row_ctas = ((int64_t)a.total_new * per_token + kThreads / 32 - 1) / (kThreads / 32);
  if (page_items + row_ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_early(kv8_append_kernel, dim3((unsigned)(page_items + row_ctas)), kThreads, 0, st, a, r, q, q_out, k, v, (int)row_ctas,
                      (int)iters);
}

}  // namespace spin
