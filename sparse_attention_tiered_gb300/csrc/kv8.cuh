// Shared by the kernels of the 8-bit paged cache (spin_kv8 in include/spin.h) and their host
// entry points. Not part of the public ABI.
#pragma once

#include "spin_internal.cuh"

namespace spin {

constexpr int kKv8HalfBytes = kPart * kD;         // the keys (or values) of a page, e4m3
constexpr int kKv8PageBytes = 2 * kKv8HalfBytes;  // 16384
constexpr int kKv8MinScaleExp = -64;              // the append's smallest scale is 2^-64

struct Rows {  // spin_rows with a bf16 pointer
  uint16_t* p;
  int64_t ts, hs;
};

struct Kv8Args {
  int32_t B, Hq, Hkv, G, max_pages, total_new, max_new;
  int64_t n_pages;
  uint8_t* pages;
  float* scales;
  uint16_t* tails;
  float* summaries;
  const int32_t* table;
  uint32_t* err;
  const int32_t* past;
  const int32_t* cu;
};

// Position rotation: angles are kept in 2^-64 turns, so position * step wraps exactly.
struct RopeArgs {
  uint64_t step[kD / 2];
  int32_t half;         // pairs = rot_dim / 2
  int32_t interleaved;
  const int32_t* positions;
};

// One request's step, checked: false (with the error word set by the thread that reports)
// where its numbers are out of range, and then nobody touches its rows.
__device__ __forceinline__ bool kv8_request(const Kv8Args& a, int b, bool report, int& row0, int& n_new, int& past) {
  row0 = a.cu[b];
  const int row1 = a.cu[b + 1];
  past = a.past[b];
  const bool rows_ok = row0 >= 0 && row1 >= row0 && row1 <= a.total_new;
  n_new = rows_ok ? row1 - row0 : 0;
  uint32_t bad = 0;
  if (!rows_ok || n_new > a.max_new || past < 0) bad = kErrIndex;
  else if ((int64_t)past + n_new > (int64_t)a.max_pages * kPart + kPart - 1) bad = kErrCapacity;
  if (bad) {
    if (report) atomicOr(a.err, bad);
    n_new = 0;
  }
  return bad == 0;
}

cudaError_t launch_kv8_append(const Kv8Args& a, const RopeArgs& r, const Rows& q, const Rows& q_out, const Rows& k,
                              const Rows& v, int sm_count, cudaStream_t st);
cudaError_t launch_kv8_attend(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel,
                              int topk, void* workspace, int sm_count, cudaStream_t st);
cudaError_t launch_kv8_prefill(const Kv8Args& a, const Rows& q, const Rows& out, float scale, const int32_t* sel,
                               int topk, void* workspace, int sm_count, cudaStream_t st);
// Launches a kernel that may begin while the launch before it on the stream ends: each of its CTAs waits for
// that one's end (griddepcontrol.wait) before it touches memory. No pointer of such a kernel is __restrict__: what a
// pointer to const with it points to counts as unchanged while the kernel runs, so its loads could be moved to
// before the wait, or go through a cache that is not coherent.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t shared, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Joins what the shares of `ctas` CTAs left in the workspace, with `rows` CTAs for each.
cudaError_t launch_kv8_join(const Kv8Args& a, const Rows& out, int ctas, int rows, void* workspace,
                            int part_rows, cudaStream_t st);
int64_t kv8_attend_workspace(const Kv8Args& a);
int64_t kv8_prefill_workspace();

}  // namespace spin
