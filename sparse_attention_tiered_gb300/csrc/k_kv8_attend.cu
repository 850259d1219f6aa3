// spin_kv8_attend: exact attention over the 8-bit paged cache.
//
// One CTA per (new token, KV head): four warps take pages in turn, a lane scores two tokens of
// a page against the group's queries, then every lane gathers four dimensions of the values.
// Running maximum and sum per query head and warp, joined at the end.
#include "kv8.cuh"

namespace spin {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float bf(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

__device__ __forceinline__ float e4m3(uint8_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
  const uint16_t h = (uint16_t)r;
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
  return f;
}

__global__ void __launch_bounds__(kWarps * 32)
kv8_attend_simple_kernel(const Kv8Args a, const Rows q, const Rows out, float scale, const int32_t* sel, int topk) {
  __shared__ float s_q[kMaxGroup][kD];
  __shared__ float s_p[kWarps][kMaxGroup][kPart];
  __shared__ float s_acc[kWarps][kMaxGroup][kD];
  __shared__ float s_m[kWarps][kMaxGroup], s_l[kWarps][kMaxGroup];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int b = 0;
  for (int lo = 0, n = a.B; n > 0;) {  // the last b with cu[b] <= t
    const int half = n / 2;
    if (a.cu[lo + half] <= t) {
      b = lo + half;
      lo += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  int row0, n_new, past;
  if (!kv8_request(a, b, tid == 0, row0, n_new, past) || t < row0 || t >= row0 + n_new) return;
  const int64_t unit = (int64_t)b * a.Hkv + h;
  const int len = past + n_new, full = len >> 6, seen = past + (t - row0) + 1;
  for (int i = tid; i < a.G * kD; i += kWarps * 32)
    s_q[i / kD][i % kD] = bf(q.p[(int64_t)t * q.ts + (int64_t)(h * a.G + i / kD) * q.hs + i % kD]);
  __syncthreads();
  float m[kMaxGroup], l[kMaxGroup], acc[kMaxGroup][4];
  for (int g = 0; g < a.G; ++g) {
    m[g] = -INFINITY;
    l[g] = acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
  }
  const int items = sel ? topk + 1 : full + 1;  // the last one: the tail
  for (int it = warp; it < items; it += kWarps) {
    const bool is_tail = it == items - 1;
    const int p = is_tail ? full : sel ? sel[unit * topk + it] : it;
    if (!is_tail && (p < 0 || p >= full)) continue;
    const int rows = min(is_tail ? len & (kPart - 1) : kPart, seen - p * kPart);  // seen by this token
    if (rows <= 0) continue;
    const uint8_t* page = nullptr;
    const uint16_t* tail = a.tails + unit * kPageElems;
    float ks = 1.f, vs = 1.f;
    if (!is_tail) {
      const int id = a.table[unit * a.max_pages + p];
      if (id < 0 || (int64_t)id >= a.n_pages) {
        if (lane == 0) atomicOr(a.err, kErrIndex);
        continue;
      }
      page = a.pages + (int64_t)id * kKv8PageBytes;
      ks = a.scales[2 * (int64_t)id];
      vs = a.scales[2 * (int64_t)id + 1];
    }
    for (int g = 0; g < a.G; ++g) {
      float s[2];
      for (int u = 0; u < 2; ++u) {
        const int row = u * 32 + lane;
        float x = 0.f;
        if (is_tail && row < rows)  // a value that is not finite makes NaN of every row that sees its token
          for (int d = 0; d < kD; ++d)
            x += bf(tail[row * kD + d]) * 0.f + bf(tail[kPart * kD + row * kD + d]) * 0.f;
        if (row < rows)
          for (int d = 0; d < kD; ++d) x += s_q[g][d] * (is_tail ? bf(tail[row * kD + d]) : e4m3(page[row * kD + d]));
        s[u] = row < rows ? x * ks * scale : -INFINITY;
      }
      float top = fmaxf(s[0], s[1]);
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m2 = fmaxf(m[g], top);
      const float base = m2 == -INFINITY ? 0.f : m2;  // every score NaN
      const float keep = expf(m[g] - base);
      float sum = 0.f;
      for (int u = 0; u < 2; ++u) {
        const float pr = u * 32 + lane < rows ? expf(s[u] - base) : 0.f;
        s_p[warp][g][u * 32 + lane] = pr;
        sum += pr;
      }
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[g] = l[g] * keep + sum;
      m[g] = m2;
      for (int d = 0; d < 4; ++d) acc[g][d] *= keep;
    }
    __syncwarp();
    for (int row = 0; row < rows; ++row) {
      float x[4];
      for (int d = 0; d < 4; ++d) {
        const int at = kPart * kD + row * kD + lane * 4 + d;
        x[d] = vs * (is_tail ? bf(tail[at]) : e4m3(page[at]));
      }
      for (int g = 0; g < a.G; ++g)
        for (int d = 0; d < 4; ++d) acc[g][d] += s_p[warp][g][row] * x[d];
    }
    __syncwarp();
  }
  for (int g = 0; g < a.G; ++g) {
    for (int d = 0; d < 4; ++d) s_acc[warp][g][lane * 4 + d] = acc[g][d];
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
  }
  __syncthreads();
  for (int i = tid; i < a.G * kD; i += kWarps * 32) {
    const int g = i / kD, d = i % kD;
    float top = -INFINITY;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][g]);
    const float base = top == -INFINITY ? 0.f : top;
    float L = 0.f, o = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = expf(s_m[w][g] - base);
      L += s_l[w][g] * f;
      o += s_acc[w][g][d] * f;
    }
    const __nv_bfloat16 y = __float2bfloat16_rn(L == 0.f ? 0.f : o / L);
    out.p[(int64_t)t * out.ts + (int64_t)(h * a.G + g) * out.hs + d] = *reinterpret_cast<const uint16_t*>(&y);
  }
}

}  // namespace

int64_t kv8_attend_workspace(const Kv8Args&) { return 16; }

cudaError_t launch_kv8_attend(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel,
                              int topk, void*, int, cudaStream_t st) {
  kv8_attend_simple_kernel<<<dim3((unsigned)a.total_new, (unsigned)a.Hkv), kWarps * 32, 0, st>>>(a, q, out, scale, sel, topk);
  return cudaGetLastError();
}

}  // namespace spin
