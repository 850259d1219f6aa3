// spin_kv8_select: the pages of the 8-bit cache that each new token attends, the k best of those that it sees whole by
// (sum of its group's queries) . (mean key of the page).
//
// What is asked for is the order of exact scores, and that is what comes out: the same pages however the tokens were split
// into calls and whatever else is in the batch. Scores are made twice. First for all pages, as bf16 products with fp32 sums:
// both factors are split into two bf16 numbers, x = h + l + r with |r| <= 2^-18 |x|, and h h' + h l' + l h' is off by at most
// E = 2^-15 (|q| + |a| / 32) |s|: three terms of 2^-18 each for what is left out and 24 sums of 16 products, each rounded to
// 2^-22 of the norms' product at worst, make 0.6 of the first part; the group's queries are added in fp32, off by
// 2^-20 of the sum a of their absolute values at most. If x is the k-th largest of these scores, pages above x + 2 E
// are among the k best and pages below x - 2 E are not. Those in between, two or three where scores are spread like
// a normal distribution, are scored again in 64 bits, where ties go to the lower page. (With tf32 products, a third
// of the work, the doubtful range would be 16 times as wide.)
//
// Two launches. The first is a product of [pages] x [128] x [tokens]: summaries are read once by a few tokens, where it is
// bound by HBM, and for a chunk's tokens from L2. A lane's 16-byte piece of a summary row is its k indices of one product:
// the k index may be permuted as long as the queries agree, so nothing moves between lanes. The second finds the k-th largest
// of a row's scores by bisection on their bits: a warp a row, the scores in registers, a count a step, and done once a
// step leaves k of them above it, some 8 steps. Alone, with cold caches: 32 requests of 512 pages, 67 MB, 19 us and 18; a chunk of
// 2048 tokens over 500 pages, 8 heads, 53 us (tensor pipe 22%, issue slots 32%: 520 CTAs are 1.7 turns) and 39 (issue slots 65%).
#include "kv8_dev.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStrip = 16;               // pages of a warp's product
constexpr int kPitch = kD + 16;          // bf16 elements of a query row in shared memory: no two rows of 8 on one bank
constexpr int kWide = 512;               // threads of a row of many pages
constexpr int kRows = 2;                 // a CTA, of few pages each
constexpr int64_t kSlabBytes = 1ll << 30;

struct SelectSpace {
  float* scores;    // [rows][pitch]
  uint64_t* exact;  // [rows][pitch]: keys of exact scores, where there are many to be settled
  float* norms;     // [units][pitch / 16] largest norm of a strip's summaries
  float* qnorms;    // [rows]
  int32_t* strange; // whether some request is out of range
  int64_t pitch;    // pages of a row
  int t0, t1;       // tokens of this slab: row (t - t0) * Hkv + h
};

__host__ __device__ __forceinline__ int64_t pitch_of(int max_pages) { return ((int64_t)max_pages + 31) / 32 * 32; }

int64_t slab_tokens(const Kv8Args& a) {
  const int64_t per = a.Hkv * (pitch_of(a.max_pages) * 12 + 4);
  const int64_t n = kSlabBytes / per;
  return n < 1 ? 1 : n < a.total_new ? n : a.total_new < 1 ? 1 : a.total_new;
}

// x as two bf16 numbers, two x at a time.
__device__ __forceinline__ void split(float x, float y, uint32_t& high, uint32_t& low) {
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(high) : "f"(y), "f"(x));
  const float rx = x - lo_f(high), ry = y - hi_f(high);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(low) : "f"(ry), "f"(rx));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A norm that is not too small: squares below 2^-149 are lost.
__device__ __forceinline__ float norm_of(float sum_of_squares) { return sqrtf(sum_of_squares) * 1.0001f + 1e-21f; }

// A request's tokens in [t0, t1): the first, and how many.
__device__ __forceinline__ int tokens_of(const SelectSpace& s, int row0, int n_new, int& first) {
  first = max(row0, s.t0);
  return max(0, min(row0 + n_new, s.t1) - first);
}

// The request that a token belongs to, of those that count, or -1: by a warp. The slow way, where cu_new may not ascend.
__device__ __noinline__ int owner_of(const Kv8Args a, int token) {
  int owner = -1;
  each_request(a, [&](int b, bool counts, int row0, int n_new) {
    const uint32_t its = __ballot_sync(0xffffffffu, counts && token >= row0 && token < row0 + n_new);
    if (its) owner = b - (int)(threadIdx.x & 31) + __ffs(its) - 1;
  });
  return owner;
}

// CTA (tile, head, x): 8 NT tokens of a request, and every X-th run of eight strips of the pages that the last of them sees.
template <int NT>
__global__ void __launch_bounds__(kThreads, 2)
kv8_select_scores(const Kv8Args a, const Rows q, SelectSpace s, int X) {
  constexpr int kTokens = 8 * NT;
  __shared__ __align__(16) uint16_t sq[2][kTokens][kPitch];
  __shared__ int64_t scratch[36];
  __shared__ uint32_t bits[kMaxRequests / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = blockIdx.x % X, th = blockIdx.x / X, h = th % a.Hkv, tile = th / a.Hkv;
  int first, row0, n_new, past;
  bool strange;
  // Requests that count share no row: as many tiles as were launched are enough, and no two write one row's scores.
  const Place pl = locate_rows(
      a, scratch, bits, blockIdx.x == 0, strange,
      [&](int row, int n, int) { return (int64_t)(tokens_of(s, row, n, first) + kTokens - 1) / kTokens; },
      [&](int64_t) { return (int64_t)tile; });
  if (blockIdx.x == 0 && tid == 0) *s.strange = strange;
  if (pl.b >= a.B || !kv8_request(a, pl.b, false, row0, n_new, past)) return;
  int tokens = tokens_of(s, row0, n_new, first);
  const int skip = (int)(tile - pl.before) * kTokens;
  first += skip;
  tokens = min(tokens - skip, kTokens);
  const int pages = (past + (first - row0) + tokens) >> 6;
  // Whole strips are read, so that a strip has one norm whoever writes it.
  const int full = (past + n_new) >> 6;
  const int64_t unit = (int64_t)pl.b * a.Hkv + h;
  const float* summaries = a.summaries + unit * a.max_pages * kD;
  // Lane (g, t) has dimensions 16 j + 4 t .. + 3 of pages g and g + 8 of a strip. The first strip is on its way while the queries
  // are added up.
  float4 v[2][8];
  auto load = [&](int p0) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int p = p0 + r * 8 + g;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[r][j] = p < full ? *reinterpret_cast<const float4*>(summaries + (int64_t)p * kD + j * 16 + t * 4)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  int p0 = (x * kWarps + warp) * kStrip;
  load(p0 < pages ? p0 : full);
  // The tokens' queries, summed over the group: 16 lanes a token, eight dimensions each.
  for (int i = tid >> 4; i < kTokens; i += kThreads / 16) {
    float v[8], abs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = abs[e] = 0.f;
    if (i < tokens) {
      const uint16_t* src = q.p + (int64_t)(first + i) * q.ts + (int64_t)h * a.G * q.hs + (tid & 15) * 8;
#pragma unroll 1
      for (int k = 0; k < a.G; k += 4) {  // (four loads on their way)
        uint4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[c] = k + c < a.G ? *reinterpret_cast<const uint4*>(src + (k + c) * q.hs) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t ww[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] += lo_f(ww[e]);
            v[2 * e + 1] += hi_f(ww[e]);
            abs[2 * e] += fabsf(lo_f(ww[e]));
            abs[2 * e + 1] += fabsf(hi_f(ww[e]));
          }
        }
      }
    }
    uint32_t hi[4], lo[4];
    float sum = 0.f, sum_abs = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      split(v[2 * e], v[2 * e + 1], hi[e], lo[e]);
      sum = fmaf(v[2 * e], v[2 * e], fmaf(v[2 * e + 1], v[2 * e + 1], sum));
      sum_abs = fmaf(abs[2 * e], abs[2 * e], fmaf(abs[2 * e + 1], abs[2 * e + 1], sum_abs));
    }
    *reinterpret_cast<uint4*>(&sq[0][i][(tid & 15) * 8]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(&sq[1][i][(tid & 15) * 8]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    for (int o = 1; o < 16; o <<= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sum_abs += __shfl_xor_sync(0xffffffffu, sum_abs, o);
    }
    if ((tid & 15) == 0 && i < tokens && x == 0)
      s.qnorms[(int64_t)(first + i - s.t0) * a.Hkv + h] = norm_of(sum) + norm_of(sum_abs) * 0.03125f;
  }
  __syncthreads();
  float* rows = s.scores + ((int64_t)(first - s.t0) * a.Hkv + h) * s.pitch;
  const int64_t row_step = a.Hkv * s.pitch;
  for (bool more = false; p0 < pages; p0 += X * kWarps * kStrip, more = true) {
    if (more) load(p0);
    float c[NT][4], d[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[n][e] = d[n][e] = 0.f;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4 w = v[r][j];
        split(w.x, w.y, hi[r], lo[r]);
        split(w.z, w.w, hi[2 + r], lo[2 + r]);
        sum[r] = fmaf(w.x, w.x, fmaf(w.y, w.y, fmaf(w.z, w.z, fmaf(w.w, w.w, sum[r]))));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint2 bh = *reinterpret_cast<const uint2*>(&sq[0][n * 8 + g][j * 16 + t * 4]);
        const uint2 bl = *reinterpret_cast<const uint2*>(&sq[1][n * 8 + g][j * 16 + t * 4]);
        mma_bf16(c[n], hi, bh.x, bh.y);
        mma_bf16(d[n], hi, bl.x, bl.y);
        mma_bf16(d[n], lo, bh.x, bh.y);
      }
    }
    bool wrong = !(sum[0] + sum[1] < INFINITY);  // (a maximum would lose a NaN)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
    }
    float top = fmaxf(sum[0], sum[1]);
    for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    wrong = __any_sync(0xffffffffu, wrong);
    if (lane == 0) s.norms[unit * (s.pitch / kStrip) + p0 / kStrip] = wrong ? INFINITY : norm_of(top);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = n * 8 + 2 * t + (e & 1), p = p0 + (e >> 1) * 8 + g;
        if (i < tokens && p < pages) rows[i * row_step + p] = c[n][e] + d[n][e];
      }
  }
}

// Numbers whose order as unsigned integers is that of the scores; what is no number is as low as -infinity.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x != x ? -INFINITY : x == 0.f ? 0.f : x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// The same of first scores, none of which is missing unless all are doubtful: any key but 0 will do for it.
__device__ __forceinline__ uint32_t quick_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return max(u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u), 1u);
}
__device__ __forceinline__ float score_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x != x ? -INFINITY : x == 0.0 ? 0.0 : x);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// The threads that share a row: a warp, or kWide threads. Thread r of them has pages r, r + T, ..
template <int T>
struct Team {
  int32_t* s;      // shared memory of a wide team: [2][warps] counts, a turn each
  uint64_t* keys;  // [32] keys
  int32_t* pages;  // [32] and their pages
  int32_t* listed;  // how many there are, 0 at the start
  uint16_t* found;  // a count for each warp and turn
  uint32_t* near;   // [T] keys that may be the k-th, and
  int32_t* n_near;  // how many there are, 0 at the start
  int turn = 0;
  __device__ __forceinline__ int rank() const { return T == 32 ? threadIdx.x & 31 : threadIdx.x; }
  // What the warps' values are; `none` for lanes that stand for no warp.
  __device__ __forceinline__ uint32_t told(uint32_t x, uint32_t none) {
    int32_t* at = s + (turn ^= 1) * (T / 32);
    const int lane = threadIdx.x & 31;
    if (lane == 0) at[threadIdx.x >> 5] = (int32_t)x;
    __syncthreads();
    return lane < T / 32 ? (uint32_t)at[lane] : none;
  }
  __device__ __forceinline__ int sum(int x) {
    uint32_t y = __reduce_add_sync(0xffffffffu, (uint32_t)x);
    if constexpr (T > 32) y = __reduce_add_sync(0xffffffffu, told(y, 0));
    return (int)y;
  }
  __device__ __forceinline__ uint32_t smallest(uint32_t x) {
    x = __reduce_min_sync(0xffffffffu, x);
    if constexpr (T > 32) x = __reduce_min_sync(0xffffffffu, told(x, 0xffffffffu));
    return x;
  }
  __device__ __forceinline__ uint32_t largest(uint32_t x) {
    x = __reduce_max_sync(0xffffffffu, x);
    if constexpr (T > 32) x = __reduce_max_sync(0xffffffffu, told(x, 0));
    return x;
  }
  // How many of the threads before this one have `flag`, and how many of all.
  __device__ __forceinline__ int before(bool flag, int& total) {
    const uint32_t vote = __ballot_sync(0xffffffffu, flag);
    int n = __popc(vote & ((1u << (threadIdx.x & 31)) - 1u));
    if constexpr (T == 32) {
      total = __popc(vote);
    } else {
      int32_t* at = s + (turn ^= 1) * (T / 32);
      if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = __popc(vote);
      __syncthreads();
      total = 0;
      for (int w = 0; w < T / 32; ++w) {
        if (w < (int)(threadIdx.x >> 5)) n += at[w];
        total += at[w];
      }
    }
    return n;
  }
};

struct RowIn {
  int pages, k;
  const float* scores;
  uint64_t* exact;
  const float* summaries;  // of the unit
  const float* norms;
  float qnorm;
  const uint16_t* q;       // the token's first query head of the group
  int64_t hs;
  int G;
  int32_t* out;
};

// N: pages a thread, held in registers; 0: read again where they are needed.
template <int T, int N>
__device__ __forceinline__ void pick(Team<T>& team, const RowIn& in) {
  const int me = team.rank(), lane = threadIdx.x & 31;
  const int turns = (in.pages + T - 1) / T, strips = (in.pages + kStrip - 1) / kStrip;
  float top = me < strips ? in.norms[me] : 0.f;  // (on its way with the scores)
  uint32_t held[N ? N : 1];
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = me + i * T;
      held[i] = p < in.pages ? quick_key(in.scores[p]) : 0;  // 0: no score's key
    }
  }
  auto key = [&](int i) -> uint32_t {  // from memory, where that is rare or there are too many
    const int p = me + i * T;
    return p < in.pages ? quick_key(in.scores[p]) : 0;
  };
  auto each = [&](auto f) {
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) f(i, held[i]);
    } else {
#pragma unroll 4
      for (int i = 0; i < turns; ++i) f(i, key(i));
    }
  };
  uint32_t lo = 0xffffffffu, hi = 0;
  each([&](int, uint32_t x) {
    hi = max(hi, x);
    lo = min(lo, x ? x : 0xffffffffu);
  });
  if (in.k <= T && in.pages >= T) lo = hi;  // the least of the threads' largest ones: T of them reach it
  const uint32_t best = hi;
  lo = team.smallest(lo);
  hi = team.largest(hi);
  for (int i = me + T; i < strips; i += T) top = fmaxf(top, in.norms[i]);
  top = __uint_as_float(team.largest(__float_as_uint(top)));
  const float size = in.qnorm * top;
  const bool sure = size < 1e30f;  // else nothing is known of the scores
  const float margin = sure ? fmaf(size, 0x1p-14f, 2e-35f) : INFINITY;  // 2 E
  // The k-th largest key: k or more are >= lo, fewer are > hi.
  bool clean = false;
  // A wide row's threads have 32 keys each, so a step costs a turn over them. The k-th largest of the threads' best is a bound that
  // few keys reach; those are dealt out, one a thread, and the steps look at them alone. (A chunk of 2048 tokens onto 150000: 754 us
  // without, 641 with; 1M tokens of one request 38.9 and 38.4.)
  bool dealt = false;
  uint32_t mine = 0;
  if constexpr (T > 32 && N > 0) {
    if (sure && in.k <= T && in.pages >= T) {
      uint32_t most = hi;
      while (lo < most) {
        const uint32_t mid = lo + ((most - lo) >> 1) + 1;
        const int n = __syncthreads_count(best >= mid);
        if (n < in.k) most = mid - 1;
        else lo = mid;
        if (n >= in.k && n <= in.k + in.k / 4) break;
      }
      int n = 0;
      each([&](int, uint32_t x) { n += x >= lo; });
      const int all = team.sum(n);
      if (all <= T) {
        int at = n ? atomicAdd(team.n_near, n) : 0;
        each([&](int, uint32_t x) {
          if (x >= lo) team.near[at++] = x;
        });
        __syncthreads();
        mine = me < all ? team.near[me] : 0;
        dealt = true;
      }
    }
  }
  while (lo < hi && sure) {
    const uint32_t mid = lo + ((hi - lo) >> 1) + 1;
    int n = 0;
    if (T > 32 && dealt) {
      n = __syncthreads_count(mine >= mid);
    } else {
      each([&](int, uint32_t x) { n += x >= mid; });
      n = team.sum(n);
    }
    if (n > in.k) lo = mid;
    else if (n < in.k) hi = mid - 1;
    else {
      uint32_t least = 0xffffffffu, next = 0;
      each([&](int, uint32_t x) {
        if (x >= mid) least = min(least, x);
        else next = max(next, x);
      });
      lo = hi = team.smallest(least);
      clean = score_of(lo) - score_of(team.largest(next)) > margin;
      break;
    }
  }
  // [low, high]: the doubtful ones, of which `want` are taken.
  uint32_t low = lo, high = 0;
  int want = 0;
  bool few = false;     // up to 32 of them: a lane each,
  int page = -1;        // of the lane, and
  uint32_t taken = 0;   // a bit a lane. Else:
  uint64_t border = 0;  // those above it are taken, and the first `equal` of those that equal it
  int equal = 0;
  if (!clean) {
    const float x = score_of(lo);
    low = sure ? key_of(x - margin) : 1;
    high = sure ? key_of(x + margin) : 0xffffffffu;
    int above = 0, within = 0;
    each([&](int, uint32_t y) {
      above += y > high;
      within += y >= low && y <= high;
    });
    above = team.sum(above);
    within = team.sum(within);
    want = in.k - above;
    if (want == within) high = 0;  // all of them: as good as clean
    else {
      // The group's queries in 64 bits: four dimensions a lane.
      double qd[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
      for (int g = 0; g < in.G; ++g) {
        const uint2 w = *reinterpret_cast<const uint2*>(in.q + g * in.hs + lane * 4);
        qd[0] += (double)lo_f(w.x), qd[1] += (double)hi_f(w.x), qd[2] += (double)lo_f(w.y), qd[3] += (double)hi_f(w.y);
      }
      auto row = [&](int p) { return *reinterpret_cast<const float4*>(in.summaries + (int64_t)p * kD + lane * 4); };
      auto exact = [&](float4 v) {  // by a warp
        double x = qd[0] * (double)v.x + qd[1] * (double)v.y + qd[2] * (double)v.z + qd[3] * (double)v.w;
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return key_of(x);
      };
      few = within <= 32;
      if (few) {  // a lane each, in any order
        int n = 0;
        each([&](int i, uint32_t y) {
          const bool doubt = y >= low && y <= high;
          if constexpr (T == 32) {
            for (uint32_t left = __ballot_sync(0xffffffffu, doubt); left; left &= left - 1, ++n)
              if (lane == n) page = __ffs(left) - 1 + i * T;
          } else if (doubt) {
            team.pages[atomicAdd(team.listed, 1)] = me + i * T;
          }
        });
        uint64_t mine = 0;
        if constexpr (T == 32) {
          for (int j = 0; j < within; j += 2) {  // two rows on their way
            const int p0 = __shfl_sync(0xffffffffu, page, j), p1 = __shfl_sync(0xffffffffu, page, min(j + 1, within - 1));
            const float4 v0 = row(p0), v1 = row(p1);
            const uint64_t x0 = exact(v0), x1 = exact(v1);
            if (lane == j) mine = x0;
            if (lane == j + 1) mine = x1;
          }
        } else {
          __syncthreads();
          for (int j = threadIdx.x >> 5; j < within; j += T / 32) {
            const uint64_t x = exact(row(team.pages[j]));
            if (lane == 0) team.keys[j] = x;
          }
          __syncthreads();
          page = lane < within ? team.pages[lane] : 0;
          mine = lane < within ? team.keys[lane] : 0;
        }
        int better = 0;
        for (int j = 0; j < within; ++j) {
          const uint64_t x = __shfl_sync(0xffffffffu, mine, j);
          const int p = __shfl_sync(0xffffffffu, page, j);
          better += x > mine || (x == mine && p < page);
        }
        taken = __ballot_sync(0xffffffffu, lane < within && better < want);
      } else {
#pragma unroll 1
        for (int i = 0; i < turns; ++i) {
          const uint32_t y = key(i);
          uint64_t own = 0;
          for (uint32_t left = __ballot_sync(0xffffffffu, y >= low && y <= high); left; left &= left - 1) {  // one after the other
            const int l = __ffs(left) - 1;
            const uint64_t x = exact(row(__shfl_sync(0xffffffffu, me, l) + i * T));
            if (lane == l) own = x;
          }
          const int p = me + i * T;
          if (p < in.pages) in.exact[p] = own;  // 0: not doubtful. Read by this thread alone
        }
        auto each_exact = [&](auto f) {
#pragma unroll 4
          for (int i = 0; i < turns; ++i) {
            const int p = me + i * T;
            if (p < in.pages) f(in.exact[p]);
          }
        };
        // Bisection again, from the top bit down: `border` is the largest number that `want` keys or more reach.
        for (int bit = 63; bit >= 0; --bit) {
          const uint64_t mid = border | 1ull << bit;
          int n = 0;
          each_exact([&](uint64_t x) { n += x >= mid; });
          n = team.sum(n);
          if (n >= want) border = mid;
          if (n == want) break;
        }
        int over = 0;
        each_exact([&](uint64_t x) { over += x > border; });
        equal = want - team.sum(over);
      }
    }
  }
  // In the order of the pages.
  int at = 0, ties = 0, total;
  auto put = [&](int i, bool take) {
    const int rank = at + team.before(take, total);
    at += total;
    if (take && rank < in.k) in.out[rank] = me + i * T;
  };
  const bool settle = high >= low && !clean;
  auto takes = [&](int i, uint32_t y) {  // but where there are many doubtful ones
    if (!settle) return y >= low && y != 0;
    uint32_t doubt = __ballot_sync(0xffffffffu, y >= low && y <= high);
    bool take = y > high;
    for (; doubt; doubt &= doubt - 1) {
      const int l = __ffs(doubt) - 1, p = __shfl_sync(0xffffffffu, me, l) + i * T;
      const bool its = __ballot_sync(0xffffffffu, page == p && (taken >> lane & 1)) != 0;
      if (lane == l) take = its;
    }
    return take;
  };
  if (settle && !few) {
#pragma unroll 1
    for (int i = 0; i < turns; ++i) {
      const uint32_t y = key(i);
      const bool doubt = y >= low && y <= high;
      const uint64_t x = doubt ? in.exact[me + i * T] : 0;
      const int rank = ties + team.before(doubt && x == border, total);
      ties += total;
      put(i, y > high || (doubt && (x > border || (x == border && rank < equal))));
    }
  } else if constexpr (N > 0) {
    // A bit a page, 32 turns a word.
    constexpr int kWords = (N + 31) / 32;
    uint32_t take[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) take[w] = 0;
    each([&](int i, uint32_t y) {
      if (settle ? y > high : y >= low && y != 0) take[i >> 5] |= 1u << (i & 31);
    });
    for (uint32_t left = settle ? taken : 0; left; left &= left - 1) {
      const int p = __shfl_sync(0xffffffffu, page, __ffs(left) - 1);
      if (p % T == me) {
#pragma unroll
        for (int w = 0; w < kWords; ++w)
          if (p / T / 32 == w) take[w] |= 1u << (p / T & 31);
      }
    }
    if constexpr (T == 32) {
#pragma unroll
      for (int i = 0; i < N; ++i) put(i, take[i >> 5] >> (i & 31) & 1);
    } else {
      // Lane i has the votes on turn i, and the number of pages that are taken before them: the CTA meets three times, not once a turn.
      static_assert(N <= 32 && N * (T / 32) <= T, "a lane a turn, a thread a count");
      const int warp = threadIdx.x >> 5, warps = T / 32;
      uint32_t votes = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t vote = __ballot_sync(0xffffffffu, take[0] >> i & 1);
        if (lane == i) votes = vote;
      }
      if (lane < N) team.found[lane * warps + warp] = (uint16_t)__popc(votes);
      __syncthreads();
      const int mine = me < N * warps ? team.found[me] : 0;
      int before = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      const int last = (int)team.told(__shfl_sync(0xffffffffu, before, 31), 0);
      before += (int)__reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)last : 0u) - mine;
      if (me < N * warps) team.found[me] = (uint16_t)before;
      __syncthreads();
      const int first = lane < N ? team.found[lane * warps + warp] : 0;
      for (uint32_t any = __reduce_or_sync(0xffffffffu, take[0]); any; any &= any - 1) {
        const int i = __ffs(any) - 1;
        const uint32_t vote = __shfl_sync(0xffffffffu, votes, i);
        const int rank = __shfl_sync(0xffffffffu, first, i) + __popc(vote & ((1u << lane) - 1u));
        if ((take[0] >> i & 1) && rank < in.k) in.out[rank] = me + i * T;
      }
    }
  } else {
    each([&](int i, uint32_t y) { put(i, takes(i, y)); });
  }
}

// A row: a token and a KV head. T = 32: a warp a row, kRows of them a CTA (with 8 the time is the same); else a CTA a row. N: pages a thread that it holds in registers, if
// that is enough; 64 or 96 registers, for 32 or 20 warps an SM.
template <int T, int N>
__global__ void __launch_bounds__(T == 32 ? kRows * 32 : T, T == 32 ? (N == 16 ? 16 : 10) : 2)
kv8_select_pick(const Kv8Args a, const Rows q, SelectSpace s, int k, int32_t* sel) {
  __shared__ int32_t counts[T == 32 ? 1 : 2 * (T / 32)];
  __shared__ uint64_t keys[T == 32 ? 1 : 32];
  __shared__ int32_t pages[T == 32 ? 1 : 32], listed;
  __shared__ uint16_t found[T == 32 ? 1 : N * (T / 32)];
  __shared__ uint32_t near[T == 32 ? 1 : T];
  __shared__ int32_t n_near;
  if (threadIdx.x == 0) listed = n_near = 0;
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = T == 32 ? (int64_t)blockIdx.x * kRows + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= (int64_t)(s.t1 - s.t0) * a.Hkv) return;
  const int token = s.t0 + (int)(row / a.Hkv), h = (int)(row % a.Hkv);
  const int32_t strange = *s.strange;  // (on its way with the others)
  if (token >= a.cu[a.B] && !strange) return;  // padding
  // The last request that begins at the token or before it: 32 places a look.
  int lo = 0, n = a.B;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lo + lane * step;
    const bool there = lane * step < n && a.cu[at] <= token;
    const int w = max(0, __popc(__ballot_sync(0xffffffffu, there)) - 1);
    lo += w * step;
    n = min(step, n - w * step);
  }
  int row0, n_new, past;
  bool its = kv8_request(a, lo, false, row0, n_new, past) && token >= row0 && token < row0 + n_new;
  if (strange) {  // the search may have gone astray
    lo = owner_of(a, token);
    its = lo >= 0 && kv8_request(a, lo, false, row0, n_new, past);
  }
  if (!its) return;
  const int64_t unit = (int64_t)lo * a.Hkv + h;
  RowIn in;
  in.pages = (past + token - row0 + 1) >> 6;
  in.k = k;
  in.out = sel + ((int64_t)token * a.Hkv + h) * k;
  if (in.pages <= k) {
    for (int i = T == 32 ? lane : threadIdx.x; i < k; i += T) in.out[i] = i < in.pages ? i : -1;
    return;
  }
  in.scores = s.scores + row * s.pitch;
  in.exact = s.exact + row * s.pitch;
  in.summaries = a.summaries + unit * a.max_pages * kD;
  in.norms = s.norms + unit * (s.pitch / kStrip);
  in.qnorm = s.qnorms[row];
  in.q = q.p + (int64_t)token * q.ts + (int64_t)h * a.G * q.hs;
  in.hs = q.hs;
  in.G = a.G;
  Team<T> team{counts, keys, pages, &listed, found, near, &n_near};
  if (in.pages <= N / 2 * T) pick<T, N / 2>(team, in);
  else if (T == 32 || in.pages <= N * T) pick<T, N>(team, in);
  else if constexpr (T > 32) pick<T, 0>(team, in);
}

template <int NT>
cudaError_t launch_scores(const Kv8Args& a, const Rows& q, const SelectSpace& s, int sm_count, cudaStream_t st) {
  const int64_t tokens = s.t1 - s.t0;
  const int64_t tiles = tokens / (8 * NT) + (a.B < tokens ? a.B : tokens);  // at most: each request's last one may be short
  // As many CTAs as two of an SM, where there are not more without: all of them start at once.
  const int64_t runs = ((int64_t)a.max_pages + kWarps * kStrip - 1) / (kWarps * kStrip);
  int64_t X = 2 * (int64_t)sm_count / (tiles * a.Hkv);
  X = X < runs ? X : runs;
  X = X > 1 ? X : 1;
  return launch_early(kv8_select_scores<NT>, dim3((unsigned)(tiles * a.Hkv * X)), kThreads, 0, st, a, q, s, (int)X);
}

}  // namespace

int64_t kv8_select_workspace(const Kv8Args& a) {
  const int64_t pitch = pitch_of(a.max_pages), rows = slab_tokens(a) * a.Hkv;
  return rows * (pitch * 12 + 4) + (int64_t)a.B * a.Hkv * (pitch / kStrip) * 4 + 4;
}

cudaError_t launch_kv8_select(const Kv8Args& a, const Rows& q, int topk, int32_t* sel, void* workspace, int sm_count,
                              cudaStream_t st) {
  SelectSpace s;
  s.pitch = pitch_of(a.max_pages);
  const int64_t slab = slab_tokens(a), rows = slab * a.Hkv;
  s.exact = static_cast<uint64_t*>(workspace);
  s.scores = reinterpret_cast<float*>(s.exact + rows * s.pitch);
  s.norms = s.scores + rows * s.pitch;
  s.qnorms = s.norms + (int64_t)a.B * a.Hkv * (s.pitch / kStrip);
  s.strange = reinterpret_cast<int32_t*>(s.qnorms + rows);
  for (int64_t t = 0; t < a.total_new; t += slab) {
    s.t0 = (int)t;
    s.t1 = (int)(t + slab < a.total_new ? t + slab : a.total_new);
    // 8 tokens a CTA or 32 (here and below: calls back to back, 8 KV heads, inputs larger than L2): 32 requests of 512 pages with 1 token
    // each 28.1 and 34.7 us, with 8 32.4 and 39.7, with 12 41.3 and 40.6, with 64 112 and 83.
    cudaError_t e = a.max_new <= 8 ? launch_scores<1>(a, q, s, sm_count, st) : launch_scores<4>(a, q, s, sm_count, st);
    if (e != cudaSuccess) return e;
    const int64_t n = (int64_t)(s.t1 - s.t0) * a.Hkv;
    // A warp a row, holding 16 or 64 scores a lane, or a CTA a row. Up to 512 pages: 32 requests 28.2, 30.9 and 35.6 us, a
    // chunk of 2048 tokens 82, 108 and 641. 1000 pages: 4 requests 18.2 with a warp a row and 20.9 with a CTA, 32 requests 43.4 and
    // 47.5, a chunk 143 and 535. 2048 pages: 1 request 25.6 and 18.4, 75 requests 134 and 129, 120 requests 206 and 209, a chunk 304
    // and 620: a CTA passes a row in a third of a warp's time, which pays for three turns of two an SM. A warp cannot hold more.
    // What is known here is the table's width, not the rows': short rows of a table of more than 2048 pages take a CTA each, too.
    const bool warps = a.max_pages <= 1024 || (a.max_pages <= 2048 && n > 6 * (int64_t)sm_count);
    const dim3 narrow((unsigned)((n + kRows - 1) / kRows));
    e = a.max_pages <= 512    ? launch_early(kv8_select_pick<32, 16>, narrow, kRows * 32, 0, st, a, q, s, topk, sel)
        : warps               ? launch_early(kv8_select_pick<32, 64>, narrow, kRows * 32, 0, st, a, q, s, topk, sel)
                              : launch_early(kv8_select_pick<kWide, 32>, dim3((unsigned)n), kWide, 0, st, a, q, s, topk, sel);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace spin
