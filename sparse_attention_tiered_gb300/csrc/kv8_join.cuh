// The join of partial attention results, shared by the attention kernels of the 8-bit paged cache.
#pragma once

#include "kv8_dev.cuh"

namespace spin {
namespace kv8 {

constexpr int kMaxCtas = 160;  // CTAs that a call's work is split over, at most
constexpr int kJoinThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

// The unit that holds the last place of share c, at `before` of its request's or row block's places: if
// its first item is in share c and its last is not, its rows are joined. A partial is (M, L, -, -, o[128]) per
// row: weights relative to 2^M, their sum, the weighted values. Share x's is number 2 x, or 2 c + 1 in
// share c itself, with `stride` rows each.
__device__ __forceinline__ void join_parts(const Kv8Args& a, const Rows& out, const Unit& u, const Place& pl,
                                           int64_t before, int first_row, int tile_rows, int c, int ctas,
                                           const float* __restrict__ partials, int stride) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float s_w[kMaxCtas], s_m[kWarps], s_l[kWarps], s_o[kWarps][kD];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t start = share_start(pl.total, c, ctas), stop = share_start(pl.total, c + 1, ctas);
  const int h = (int)((stop - 1 - before) / u.weight);
  const int64_t begin = before + (int64_t)h * u.weight + kUnitCost, end = begin + u.items;
  if (begin < start || begin >= stop || end <= stop) return;
  const int n = share_of(pl.total, end - 1, ctas) - c + 1;  // at most kMaxCtas
  const int rows = min(tile_rows, u.n_new * a.G - first_row);
  const int64_t part_floats = (int64_t)stride * kPartialStride;
  auto empty = [&](int x) {  // with fewer places than CTAs some shares are
    return share_start(pl.total, c + x, ctas) >= share_start(pl.total, c + x + 1, ctas);
  };
  if (n <= 4) {  // a row a warp
    for (int row = blockIdx.y * kWarps + warp; row < rows; row += gridDim.y * kWarps) {
      float M = -INFINITY, L = 0.f;
      float2 ml[4];
      float4 y[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        ml[x] = make_float2(-INFINITY, 0.f);
        y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < n && !empty(x)) {
          const float* part = partials + (int64_t)(2 * (c + x) + (x == 0 ? 1 : 0)) * part_floats + (int64_t)row * kPartialStride;
          ml[x] = *reinterpret_cast<const float2*>(part);
          y[x] = *reinterpret_cast<const float4*>(part + 4 + 4 * lane);  // (not written where nothing was seen)
        }
        M = fmaxf(M, ml[x].x);
      }
      const float base = M == -INFINITY ? 0.f : M;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float f = ex2(ml[x].x - base);
        L += ml[x].y * f;
        if (f != 0.f) o = make_float4(o.x + y[x].x * f, o.y + y[x].y * f, o.z + y[x].z * f, o.w + y[x].w * f);
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const int i = (first_row + row) / a.G, head = h * a.G + (first_row + row) - i * a.G;
      const __nv_bfloat162 v0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), v1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(out.p + (int64_t)(u.row0 + i) * out.ts + (int64_t)head * out.hs + 4 * lane) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
    }
    return;
  }
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const float* mine = partials + (int64_t)row * kPartialStride;
    auto part = [&](int x) { return mine + (int64_t)(2 * (c + x) + (x == 0 ? 1 : 0)) * part_floats; };
    constexpr int kMost = (kMaxCtas + kJoinThreads - 1) / kJoinThreads;
    float2 ml[kMost];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int x = i * kJoinThreads + tid;
      ml[i] = make_float2(-INFINITY, 0.f);
      if (x < n && !empty(x)) ml[i] = *reinterpret_cast<const float2*>(part(x));
      M = fmaxf(M, ml[i].x);
    }
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    __syncthreads();  // the last row's sums have been read
    if (lane == 0) s_m[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int x = i * kJoinThreads + tid;
      const float f = ex2(ml[i].x - base);
      L += ml[i].y * f;
      if (x < n) s_w[x] = f;
    }
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = warp; x < n; x += kWarps) {
      const float f = s_w[x];
      if (f == 0.f) continue;  // nothing seen there, or an empty share, which wrote nothing
      const float4 y = *reinterpret_cast<const float4*>(part(x) + 4 + 4 * lane);
      o = make_float4(o.x + y.x * f, o.y + y.y * f, o.z + y.z * f, o.w + y.w * f);
    }
    *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = o;
    __syncthreads();
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += s_l[w];
      x += s_o[w][tid];
    }
    const int i = (first_row + row) / a.G, head = h * a.G + (first_row + row) - i * a.G;
    const __nv_bfloat16 y = __float2bfloat16_rn(sum == 0.f ? 0.f : x / sum);
    out.p[(int64_t)(u.row0 + i) * out.ts + (int64_t)head * out.hs + tid] = *reinterpret_cast<const uint16_t*>(&y);
  }
}

}  // namespace kv8
}  // namespace spin
