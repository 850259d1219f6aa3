// The join of partial attention results over the 8-bit paged cache, for the units that several CTAs of
// an attention launch shared. A CTA that begins such a unit leaves a record of it; every sharer
// leaves a partial (M, L, V, -, o[128]) per row: weights relative to 2^(M + V), their sum, the weighted
// values. M is a score and may be of any size, V is small: M's differences are taken first. Parts are added in a fixed order. The launch waits for the attention launch by a programmatic
// dependency, so it is resident when that ends. It takes 4 us, a launch and three loads that wait for one
// another; with weights before the parts' loads it took 7.
#include "kv8_dev.cuh"

namespace spin {

namespace {

using namespace kv8;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
static_assert(kThreads >= kMaxCtas, "a thread a part");
constexpr float kFar = 2048.f;  // a sum of two exponents is right to 2^-13 below it

__device__ __forceinline__ void add(float4& o, const float4& y, float f) {
  if (f != 0.f) o = make_float4(o.x + y.x * f, o.y + y.y * f, o.z + y.z * f, o.w + y.w * f);
}

__device__ __forceinline__ float3 load_mlv(const float* part) {
  const float4 x = *reinterpret_cast<const float4*>(part);
  return make_float3(x.x, x.y, x.z);
}

// CTA (c, y): rows y, y + gridDim.y, .. (or as many warps' rows) of the unit that share c begins. What it
// takes is the chain of loads (the record, then a row's parts, all at once), so no load hangs on a value
// that another one brings: a part that nobody wrote is loaded too, and left out.
__global__ void __launch_bounds__(kThreads)
kv8_join_kernel(int G, const Rows out, int ctas, const JoinRecord* records, const float* partials,
                int part_rows) {
  __shared__ float s_w[kMaxCtas], s_m[kWarps], s_v[kWarps], s_l[kWarps], s_o[kWarps][kD];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // by every CTA: this launch must not end before the first
  const JoinRecord r = records[c];
  const int n = r.parts;
  if (n == 0) return;
  const int rows = min(part_rows, r.n_new * G - r.first_row);
  const int64_t part_floats = (int64_t)part_rows * kPartialStride;
  auto empty = [&](int x) {    // with fewer places than CTAs some shares are, and wrote nothing
    return r.total < ctas && share_start(r.total, c + x, ctas) >= share_start(r.total, c + x + 1, ctas);
  };
  auto part = [&](int x, int row) {
    return partials + (int64_t)(2 * (c + x) + (x == 0 ? 1 : 0)) * part_floats + (int64_t)row * kPartialStride;
  };
  auto dst = [&](int row) {
    const int i = (r.first_row + row) / G, head = r.h * G + (r.first_row + row) - i * G;
    return out.p + (int64_t)(r.row0 + i) * out.ts + (int64_t)head * out.hs;
  };
  if (n <= 4) {  // a row a warp
    for (int row = blockIdx.y * kWarps + warp; row < rows; row += gridDim.y * kWarps) {
      float M = -INFINITY, V = -INFINITY, L = 0.f;
      float3 mlv[4];
      float4 y[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        mlv[x] = make_float3(-INFINITY, 0.f, 0.f);
        y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < n) {
          mlv[x] = load_mlv(part(x, row));
          y[x] = *reinterpret_cast<const float4*>(part(x, row) + 4 + 4 * lane);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (x < n && empty(x)) mlv[x] = make_float3(-INFINITY, 0.f, 0.f);
        M = fmaxf(M, mlv[x].x);
      }
      const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        mlv[x].x = (mlv[x].x - base) + mlv[x].z;
        V = fmaxf(V, mlv[x].x);
      }
      if (V == -INFINITY) V = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float f = ex2(mlv[x].x - V);
        L += mlv[x].y * f;
        add(o, y[x], f);
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const __nv_bfloat162 v0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), v1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(dst(row) + 4 * lane) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
    }
    return;
  }
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {  // a row a CTA
    constexpr int kFirst = 5;  // parts of a warp that are on their way before the weights are known
    float3 mlv = make_float3(-INFINITY, 0.f, 0.f);
    if (tid < n) mlv = load_mlv(part(tid, row));
    float4 y[kFirst];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
      const int x = warp + i * kWarps;
      if (x < n) y[i] = *reinterpret_cast<const float4*>(part(x, row) + 4 + 4 * lane);
    }
    if (tid < n && empty(tid)) mlv = make_float3(-INFINITY, 0.f, 0.f);
    // Where scores are small, one maximum does; the barrier also says that the last row's sums have been read.
    const bool far = __syncthreads_or(mlv.x != -INFINITY && !(fabsf(mlv.x) < kFar));
    auto largest = [&](float x, float* s) {  // of the CTA; 0 where there is none
      for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      if (lane == 0) s[warp] = x;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x = fmaxf(x, s[w]);
      return x == -INFINITY ? 0.f : x;
    };
    const float a = (far ? mlv.x - largest(mlv.x, s_m) : mlv.x) + mlv.z;
    const float f = ex2(a - largest(a, s_v));
    if (tid < n) s_w[tid] = f;
    float L = mlv.y * f;
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
      if (warp + i * kWarps < n) add(o, y[i], s_w[warp + i * kWarps]);
    for (int x = warp + kFirst * kWarps; x < n; x += kFirst * kWarps) {
#pragma unroll
      for (int i = 0; i < kFirst; ++i)
        if (x + i * kWarps < n) y[i] = *reinterpret_cast<const float4*>(part(x + i * kWarps, row) + 4 + 4 * lane);
#pragma unroll
      for (int i = 0; i < kFirst; ++i)
        if (x + i * kWarps < n) add(o, y[i], s_w[x + i * kWarps]);
    }
    *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = o;
    __syncthreads();
    if (tid < kD) {
      float sum = 0.f, x = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        sum += s_l[w];
        x += s_o[w][tid];
      }
      const __nv_bfloat16 v = __float2bfloat16_rn(sum == 0.f ? 0.f : x / sum);
      dst(row)[tid] = *reinterpret_cast<const uint16_t*>(&v);
    }
  }
}

}  // namespace

cudaError_t launch_kv8_join(const Kv8Args& a, const Rows& out, int ctas, int rows, void* workspace,
                            int part_rows, cudaStream_t st) {
  return launch_early(kv8_join_kernel, dim3((unsigned)ctas, (unsigned)rows), kThreads, 0, st, a.G, out, ctas,
                      static_cast<const JoinRecord*>(workspace),
                      reinterpret_cast<const float*>(static_cast<uint8_t*>(workspace) + kRecordBytes), part_rows);
}

}  // namespace spin
