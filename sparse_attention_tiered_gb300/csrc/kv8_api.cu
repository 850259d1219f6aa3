// Host entry points of the 8-bit paged cache (spin_kv8_* in include/spin.h): argument
// checks, then one launch sequence on the caller's stream. Nothing is allocated or kept.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>

#include "../../include/spin.h"
#include "kv8.cuh"

namespace spin {

void set_global_error(const char* msg);

namespace {

int refuse(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_global_error(buf);
  return code;
}

struct OnDevice {  // the cache's device for the call, the caller's afterwards
  int prev = -1;
  bool ok = false;
  explicit OnDevice(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      cudaGetLastError();
      prev = -1;
    }
    ok = prev == dev || cudaSetDevice(dev) == cudaSuccess;
    if (!ok) cudaGetLastError();
    if (prev == dev) prev = -1;
  }
  ~OnDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

bool off(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

int check_cache(const char* who, const spin_kv8* c) {
  if (!c) return refuse(SPIN_ERR_INVALID, "%s: cache is NULL", who);
  if (c->batch < 1 || c->batch > kMaxRequests) return refuse(SPIN_ERR_INVALID, "%s: batch must be 1 .. %d", who, kMaxRequests);
  if (c->kv_heads < 1 || c->kv_heads > 4096 || c->q_heads < 1 || c->q_heads % c->kv_heads != 0 ||
      c->q_heads / c->kv_heads > kMaxGroup)
    return refuse(SPIN_ERR_INVALID, "%s: q_heads must be a multiple of kv_heads (1 .. 4096) with a group of at most %d", who,
                  kMaxGroup);
  if (c->max_pages < 1 || c->max_pages > (1 << 24) || c->n_pages < 1 || c->n_pages > (1 << 24))
    return refuse(SPIN_ERR_INVALID, "%s: max_pages and n_pages must be 1 .. 2^24", who);
  if (!c->pages || !c->scales || !c->tails || !c->table || !c->error)
    return refuse(SPIN_ERR_INVALID, "%s: pages, scales, tails, table and error must not be NULL", who);
  if (off(c->pages, 128) || off(c->scales, 8) || off(c->tails, 16) || off(c->summaries, 16) || off(c->table, 4) ||
      off(c->error, 4))
    return refuse(SPIN_ERR_INVALID, "%s: pages must be 128-byte, tails and summaries 16-byte, scales 8-byte, table and error "
                  "4-byte aligned", who);
  if (c->device < 0 || c->reserved != 0) return refuse(SPIN_ERR_INVALID, "%s: device must be >= 0 and reserved 0", who);
  return SPIN_OK;
}

int check_step(const char* who, const spin_kv8_step* s) {
  if (!s || !s->past || !s->cu_new) return refuse(SPIN_ERR_INVALID, "%s: step, past and cu_new must not be NULL", who);
  if (off(s->past, 4) || off(s->cu_new, 4)) return refuse(SPIN_ERR_INVALID, "%s: past and cu_new must be 4-byte aligned", who);
  if (s->total_new < 0) return refuse(SPIN_ERR_INVALID, "%s: total_new must be >= 0", who);
  if (s->max_new < 1 || s->max_new > (1 << 20)) return refuse(SPIN_ERR_INVALID, "%s: max_new must be 1 .. 2^20", who);
  return SPIN_OK;
}

// `rows` may be an empty tensor's: with no rows its address is not used.
int check_rows(const char* who, const char* name, const spin_rows* r, int32_t total) {
  if (!r || (!r->ptr && total > 0)) return refuse(SPIN_ERR_INVALID, "%s: %s must not be NULL", who, name);
  if (off(r->ptr, 16) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0)
    return refuse(SPIN_ERR_INVALID, "%s: %s must be 16-byte aligned, with strides that are multiples of 8 elements", who, name);
  return SPIN_OK;
}

// A written array's rows must not overlap: either the heads of a token lie together inside
// its row, or the tokens of a head inside its plane.
int check_apart(const char* who, const char* name, const spin_rows* r, int32_t total, int32_t heads) {
  const int64_t t = std::llabs((long long)r->token_stride), h = std::llabs((long long)r->head_stride);
  const bool one_t = total <= 1, one_h = heads <= 1;
  const bool ok = (one_t && one_h) || (one_t && h >= kD) || (one_h && t >= kD) ||
                  (h >= kD && t >= h * (heads - 1) + kD) || (t >= kD && h >= t * ((int64_t)total - 1) + kD);
  return ok ? SPIN_OK : refuse(SPIN_ERR_INVALID, "%s: the rows of %s overlap", who, name);
}

int check_pool(const char* who, const int32_t* refs, const int32_t* free_pages) {
  if (!refs || off(refs, 4) || off(free_pages, 4))
    return refuse(SPIN_ERR_INVALID, "%s: refs must not be NULL; refs and free_pages must be 4-byte aligned", who);
  return SPIN_OK;
}

Kv8Args make_args(const spin_kv8* c, const spin_kv8_step* s) {
  Kv8Args a;
  a.B = c->batch;
  a.Hq = c->q_heads;
  a.Hkv = c->kv_heads;
  a.G = c->q_heads / c->kv_heads;
  a.max_pages = c->max_pages;
  a.total_new = s ? s->total_new : 0;
  a.max_new = s ? s->max_new : 1;
  a.n_pages = c->n_pages;
  a.pages = c->pages;
  a.scales = c->scales;
  a.tails = c->tails;
  a.summaries = c->summaries;
  a.table = c->table;
  a.err = c->error;
  a.past = s ? s->past : nullptr;
  a.cu = s ? s->cu_new : nullptr;
  return a;
}

Rows make_rows(const spin_rows* r) {
  if (!r) return Rows{nullptr, 0, 0};
  return Rows{static_cast<uint16_t*>(r->ptr), r->token_stride, r->head_stride};
}

// An error left by earlier, unrelated work would be reported as this call's; report it as
// what it is and launch nothing.
int ready(const char* who, const OnDevice& d, int device, int* sms) {
  if (!d.ok) return refuse(SPIN_ERR_CUDA, "%s: cannot select device %d", who, device);
  if (cudaGetLastError() != cudaSuccess)
    return refuse(SPIN_ERR_CUDA, "%s: a CUDA error from earlier work was pending; nothing was launched", who);
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || *sms < 1) {
    cudaGetLastError();
    return refuse(SPIN_ERR_CUDA, "%s: no usable CUDA device", who);
  }
  return SPIN_OK;
}

int launched(const char* who, cudaError_t e) {
  if (e == cudaSuccess) return SPIN_OK;
  cudaGetLastError();
  return refuse(SPIN_ERR_CUDA, "%s: launching failed: %s", who, cudaGetErrorString(e));
}

}  // namespace
}  // namespace spin

extern "C" {

int spin_kv8_append(const spin_kv8* cache, const spin_kv8_step* step, const spin_rows* q, const spin_rows* q_out,
                    const spin_rows* k, const spin_rows* v, const int32_t* positions, spin_stream_t stream) {
  using namespace spin;
  const char* who = "spin_kv8_append";
  int rc = check_cache(who, cache);
  if (!rc) rc = check_step(who, step);
  if (rc) return rc;
  if (cache->rot_dim < 0 || cache->rot_dim > kD || cache->rot_dim % 16 != 0)
    return refuse(SPIN_ERR_INVALID, "%s: rot_dim must be a multiple of 16 between 0 and 128", who);
  if (cache->rot_dim > 0 && !cache->inv_freq) return refuse(SPIN_ERR_INVALID, "%s: inv_freq must not be NULL", who);
  if (cache->interleaved != 0 && cache->interleaved != 1)
    return refuse(SPIN_ERR_INVALID, "%s: interleaved must be 0 or 1", who);
  if ((q == nullptr) != (q_out == nullptr))
    return refuse(SPIN_ERR_INVALID, "%s: q and q_out must both be given, or neither", who);
  if (q && ((rc = check_rows(who, "q", q, step->total_new)) || (rc = check_rows(who, "q_out", q_out, step->total_new)) ||
            (rc = check_apart(who, "q_out", q_out, step->total_new, cache->q_heads))))
    return rc;
  if ((rc = check_rows(who, "k", k, step->total_new)) || (rc = check_rows(who, "v", v, step->total_new))) return rc;
  if (q && q->ptr == q_out->ptr && (q->token_stride != q_out->token_stride || q->head_stride != q_out->head_stride))
    return refuse(SPIN_ERR_INVALID, "%s: q_out in place of q must have its strides", who);
  if (off(positions, 4)) return refuse(SPIN_ERR_INVALID, "%s: positions must be 4-byte aligned", who);
  RopeArgs r;
  r.half = cache->rot_dim / 2;
  r.interleaved = cache->interleaved;
  r.positions = positions;
  for (int j = 0; j < kD / 2; ++j) {
    r.step[j] = 0;
    if (j >= r.half) continue;
    const double f = cache->inv_freq[j];
    if (!std::isfinite(f)) return refuse(SPIN_ERR_INVALID, "%s: inv_freq[%d] is not finite", who, j);
    double turn = f * 0.15915494309189533577;  // 1 / (2 pi)
    turn -= std::floor(turn);
    const double scaled = turn * 18446744073709551616.0;  // 2^64
    r.step[j] = scaled < 18446744073709551616.0 ? (uint64_t)scaled : 0;
  }
  OnDevice dev(cache->device);
  int sms = 0;
  if ((rc = ready(who, dev, cache->device, &sms))) return rc;
  if (step->total_new == 0) return SPIN_OK;
  return launched(who, launch_kv8_append(make_args(cache, step), r, make_rows(q), make_rows(q_out), make_rows(k),
                                         make_rows(v), sms, static_cast<cudaStream_t>(stream)));
}

int spin_kv8_workspace(const spin_kv8* cache, int64_t* bytes) {
  using namespace spin;
  const int rc = check_cache("spin_kv8_workspace", cache);
  if (rc) return rc;
  if (!bytes) return refuse(SPIN_ERR_INVALID, "spin_kv8_workspace: bytes is NULL");
  *bytes = kv8_attend_workspace(make_args(cache, nullptr));
  return SPIN_OK;
}

int spin_kv8_attend(const spin_kv8* cache, const spin_kv8_step* step, const spin_rows* q, const spin_rows* out,
                    float scale, const int32_t* sel, int32_t topk, void* workspace, int64_t workspace_bytes,
                    spin_stream_t stream) {
  using namespace spin;
  const char* who = "spin_kv8_attend";
  int rc = check_cache(who, cache);
  if (!rc) rc = check_step(who, step);
  if (!rc) rc = check_rows(who, "q", q, step->total_new);
  if (!rc) rc = check_rows(who, "out", out, step->total_new);
  if (!rc) rc = check_apart(who, "out", out, step->total_new, cache->q_heads);
  if (rc) return rc;
  if (q->ptr == out->ptr && (q->token_stride != out->token_stride || q->head_stride != out->head_stride))
    return refuse(SPIN_ERR_INVALID, "%s: out in place of q must have its strides", who);
  if (!std::isfinite(scale)) return refuse(SPIN_ERR_INVALID, "%s: scale must be finite", who);
  if ((sel != nullptr) != (topk != 0) || topk < 0 || topk > (1 << 24))
    return refuse(SPIN_ERR_INVALID, "%s: sel needs topk between 1 and 2^24, no sel needs topk 0", who);
  if (off(sel, 4)) return refuse(SPIN_ERR_INVALID, "%s: sel must be 4-byte aligned", who);
  const Kv8Args a = make_args(cache, step);
  if (!workspace || off(workspace, 16) || workspace_bytes < kv8_attend_workspace(a))
    return refuse(SPIN_ERR_INVALID, "%s: workspace must be 16-byte aligned and of spin_kv8_workspace bytes", who);
  OnDevice dev(cache->device);
  int sms = 0;
  if ((rc = ready(who, dev, cache->device, &sms))) return rc;
  if (step->total_new == 0) return SPIN_OK;
  return launched(who, launch_kv8_attend(a, make_rows(q), make_rows(out), scale, sel, topk, workspace, sms,
                                         static_cast<cudaStream_t>(stream)));
}

int spin_kv8_select_workspace(const spin_kv8* cache, int32_t total_new, int64_t* bytes) {
  using namespace spin;
  const char* who = "spin_kv8_select_workspace";
  const int rc = check_cache(who, cache);
  if (rc) return rc;
  if (!bytes || total_new < 0) return refuse(SPIN_ERR_INVALID, "%s: bytes must not be NULL, total_new must be >= 0", who);
  Kv8Args a = make_args(cache, nullptr);
  a.total_new = total_new;
  *bytes = kv8_select_workspace(a);
  return SPIN_OK;
}

int spin_kv8_select(const spin_kv8* cache, const spin_kv8_step* step, const spin_rows* q, int32_t topk, int32_t* sel,
                    void* workspace, int64_t workspace_bytes, spin_stream_t stream) {
  using namespace spin;
  const char* who = "spin_kv8_select";
  int rc = check_cache(who, cache);
  if (!rc) rc = check_step(who, step);
  if (!rc) rc = check_rows(who, "q", q, step->total_new);
  if (rc) return rc;
  if (!cache->summaries) return refuse(SPIN_ERR_INVALID, "%s: the cache has no summaries", who);
  if (topk < 1 || topk > kMaxTopk) return refuse(SPIN_ERR_INVALID, "%s: topk must be 1 .. %d", who, kMaxTopk);
  if ((!sel && step->total_new > 0) || off(sel, 4)) return refuse(SPIN_ERR_INVALID, "%s: sel must not be NULL, and 4-byte aligned", who);
  const Kv8Args a = make_args(cache, step);
  if (!workspace || off(workspace, 16) || workspace_bytes < kv8_select_workspace(a))
    return refuse(SPIN_ERR_INVALID, "%s: workspace must be 16-byte aligned and of spin_kv8_select_workspace bytes", who);
  OnDevice dev(cache->device);
  int sms = 0;
  if ((rc = ready(who, dev, cache->device, &sms))) return rc;
  if (step->total_new == 0) return SPIN_OK;
  return launched(who, launch_kv8_select(a, make_rows(q), topk, sel, workspace, sms, static_cast<cudaStream_t>(stream)));
}

int spin_kv8_attend_rows_workspace(const spin_kv8* cache, int32_t total_new, int32_t topk, int64_t* bytes) {
  using namespace spin;
  const char* who = "spin_kv8_attend_rows_workspace";
  const int rc = check_cache(who, cache);
  if (rc) return rc;
  if (!bytes || total_new < 0 || topk < 1 || topk > kMaxTopk)
    return refuse(SPIN_ERR_INVALID, "%s: bytes must not be NULL, total_new must be >= 0 and topk 1 .. %d", who, kMaxTopk);
  Kv8Args a = make_args(cache, nullptr);
  a.total_new = total_new;
  *bytes = kv8_rows_workspace(a, topk);
  return SPIN_OK;
}

int spin_kv8_attend_rows(const spin_kv8* cache, const spin_kv8_step* step, const spin_rows* q, const spin_rows* out, float scale,
                         const int32_t* sel, int32_t topk, void* workspace, int64_t workspace_bytes, spin_stream_t stream) {
  using namespace spin;
  const char* who = "spin_kv8_attend_rows";
  int rc = check_cache(who, cache);
  if (!rc) rc = check_step(who, step);
  if (!rc) rc = check_rows(who, "q", q, step->total_new);
  if (!rc) rc = check_rows(who, "out", out, step->total_new);
  if (!rc) rc = check_apart(who, "out", out, step->total_new, cache->q_heads);
  if (rc) return rc;
  if (q->ptr == out->ptr && (q->token_stride != out->token_stride || q->head_stride != out->head_stride))
    return refuse(SPIN_ERR_INVALID, "%s: out in place of q must have its strides", who);
  if (!std::isfinite(scale)) return refuse(SPIN_ERR_INVALID, "%s: scale must be finite", who);
  if (topk < 1 || topk > kMaxTopk) return refuse(SPIN_ERR_INVALID, "%s: topk must be 1 .. %d", who, kMaxTopk);
  if ((!sel && step->total_new > 0) || off(sel, 4)) return refuse(SPIN_ERR_INVALID, "%s: sel must not be NULL, and 4-byte aligned", who);
  const Kv8Args a = make_args(cache, step);
  if (!workspace || off(workspace, 16) || workspace_bytes < kv8_rows_workspace(a, topk))
    return refuse(SPIN_ERR_INVALID, "%s: workspace must be 16-byte aligned and of spin_kv8_attend_rows_workspace bytes", who);
  OnDevice dev(cache->device);
  int sms = 0;
  if ((rc = ready(who, dev, cache->device, &sms))) return rc;
  if (step->total_new == 0) return SPIN_OK;
  return launched(who, launch_kv8_rows(a, make_rows(q), make_rows(out), scale, sel, topk, workspace, sms,
                                       static_cast<cudaStream_t>(stream)));
}

int spin_kv8_pool_workspace(const spin_kv8* cache, int64_t* bytes) {
  using namespace spin;
  const int rc = check_cache("spin_kv8_pool_workspace", cache);
  if (rc) return rc;
  if (!bytes) return refuse(SPIN_ERR_INVALID, "spin_kv8_pool_workspace: bytes is NULL");
  *bytes = kv8_pool_workspace(make_args(cache, nullptr));
  return SPIN_OK;
}

int spin_kv8_reserve(const spin_kv8* cache, const spin_kv8_step* step, int32_t* refs, int32_t* free_pages, void* workspace,
                     int64_t workspace_bytes, spin_stream_t stream) {
  using namespace spin;
  const char* who = "spin_kv8_reserve";
  int rc = check_cache(who, cache);
  if (!rc) rc = check_step(who, step);
  if (!rc) rc = check_pool(who, refs, free_pages);
  if (rc) return rc;
  const Kv8Args a = make_args(cache, step);
  if (!workspace || off(workspace, 16) || workspace_bytes < kv8_pool_workspace(a))
    return refuse(SPIN_ERR_INVALID, "%s: workspace must be 16-byte aligned and of spin_kv8_pool_workspace bytes", who);
  OnDevice dev(cache->device);
  int sms = 0;
  if ((rc = ready(who, dev, cache->device, &sms))) return rc;
  return launched(who, launch_kv8_reserve(a, refs, free_pages, workspace, static_cast<cudaStream_t>(stream)));
}

int spin_kv8_fork(const spin_kv8* cache, int32_t* refs, int32_t* len, const int32_t* src, spin_stream_t stream) {
  using namespace spin;
  const char* who = "spin_kv8_fork";
  int rc = check_cache(who, cache);
  if (!rc) rc = check_pool(who, refs, nullptr);
  if (rc) return rc;
  if (!len || !src || off(len, 4) || off(src, 4) || len == src)
    return refuse(SPIN_ERR_INVALID, "%s: len and src must be two arrays, not NULL and 4-byte aligned", who);
  OnDevice dev(cache->device);
  int sms = 0;
  if ((rc = ready(who, dev, cache->device, &sms))) return rc;
  return launched(who, launch_kv8_fork(make_args(cache, nullptr), refs, len, src, sms, static_cast<cudaStream_t>(stream)));
}

int spin_kv8_compact(const spin_kv8* cache, int32_t* refs, int32_t* free_pages, void* workspace, int64_t workspace_bytes,
                     spin_stream_t stream) {
  using namespace spin;
  const char* who = "spin_kv8_compact";
  int rc = check_cache(who, cache);
  if (!rc) rc = check_pool(who, refs, free_pages);
  if (rc) return rc;
  const Kv8Args a = make_args(cache, nullptr);
  if (!workspace || off(workspace, 16) || workspace_bytes < kv8_pool_workspace(a))
    return refuse(SPIN_ERR_INVALID, "%s: workspace must be 16-byte aligned and of spin_kv8_pool_workspace bytes", who);
  OnDevice dev(cache->device);
  int sms = 0;
  if ((rc = ready(who, dev, cache->device, &sms))) return rc;
  return launched(who, launch_kv8_compact(a, refs, free_pages, workspace, sms, static_cast<cudaStream_t>(stream)));
}

int spin_kv8_status(const spin_kv8* cache, spin_stream_t stream) {
  using namespace spin;
  const char* who = "spin_kv8_status";
  int rc = check_cache(who, cache);
  if (rc) return rc;
  OnDevice dev(cache->device);
  if (!dev.ok) return refuse(SPIN_ERR_CUDA, "%s: cannot select device %d", who, cache->device);
  uint32_t w = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&w, cache->error, sizeof(w), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return refuse(SPIN_ERR_CUDA, "%s: reading the error word failed: %s", who, cudaGetErrorString(e));
  }
  if (w & kErrTimeout) return refuse(SPIN_ERR_TIMEOUT, "%s: a bounded device wait ran out (device error 0x%x)", who, w);
  if (w & kErrCapacity) return refuse(SPIN_ERR_CAPACITY, "%s: a request outgrew its table row, or the pool has too few free pages (device error 0x%x)", who, w);
  if (w) return refuse(SPIN_ERR_INVALID, "%s: lengths or page ids out of range (device error 0x%x)", who, w);
  return SPIN_OK;
}

}  // extern "C"
