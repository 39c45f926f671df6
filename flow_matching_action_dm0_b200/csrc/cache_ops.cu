// Entry points of the operators over key/value caches: argument checks, the
// calls' descriptions, and launches.  Nothing is allocated after
// rtv_ops_create and nothing is kept between calls but the status word.
#include "cache_ops.h"

#include <algorithm>
#include <cmath>
#include <new>
#include <string>

#include "runtime.h"

using namespace rtv;

struct rtv_ops {
  int device = 0;
  AttnDevice attn{};
  unsigned* status = nullptr;
  std::string last_error;
};

namespace {

constexpr long long kTimeoutNs = 2000000000LL;   // limit of a kernel's wait for its own copies and products

rtv_status ofail(rtv_ops* h, rtv_status s, const std::string& msg) {
  h->last_error = msg;
  return s;
}

// No exception crosses the C boundary.
template <typename F>
rtv_status guarded(rtv_ops* h, F&& body) {
  if (!h) return RTV_ERR_ARG;
  try {
    return body();
  } catch (...) {
    return RTV_ERR_OOM;
  }
}

long long elt_bytes(int dtype) { return dtype == RTV_F32 ? 4 : dtype == RTV_BF16 ? 2 : 1; }

// Device memory of the handle's GPU, aligned.
rtv_status check_ptr(rtv_ops* h, const void* p, const char* what, uintptr_t align) {
  if (!p) return ofail(h, RTV_ERR_ARG, std::string(what) + ": null pointer");
  if ((uintptr_t)p % align) return ofail(h, RTV_ERR_ARG, std::string(what) + ": not " + std::to_string(align) + "-byte aligned");
  cudaPointerAttributes at{};
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return ofail(h, RTV_ERR_ARG, std::string(what) + ": not a device pointer");
  }
  if ((at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) || (at.type == cudaMemoryTypeDevice && at.device != h->device))
    return ofail(h, RTV_ERR_ARG, std::string(what) + ": not memory of the handle's GPU");
  return RTV_OK;
}

#define OTRY(expr)                       \
  do {                                   \
    const rtv_status _s = (expr);        \
    if (_s != RTV_OK) return _s;         \
  } while (0)

// Whether the rows of `inner` elements of an array that is written may share
// elements: each stride, from the smallest, has to step over all that the
// smaller ones reach.
bool overlaps(long long inner, const int (&n)[3], const long long (&s)[3]) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return s[a] < s[b]; });
  long long reach = inner;
  for (const int i : order) {
    if (n[i] <= 1) continue;
    if (s[i] < reach) return true;
    if (s[i] > (1LL << 62) / n[i]) return false;   // (nothing allocated is that long; the rest steps further)
    reach = std::max(reach, s[i] * (n[i] - 1) + reach);
  }
  return false;
}

// Strides of an array with a dense head_dim: multiples of 16 bytes, not
// negative, and of rows that do not overlap when they are written.
rtv_status check_strides(rtv_ops* h, const char* what, long long eb, bool written, int dim, int n0, long long s0, int n1,
                         long long s1, int n2, long long s2) {
  const int n[3] = {n0, n1, n2};
  const long long s[3] = {s0, s1, s2};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] < 0 || (s[i] * eb) % 16 || s[i] > (1LL << 39) / eb))
      return ofail(h, RTV_ERR_ARG, std::string(what) + ": strides must be multiples of 16 bytes, from 0 to 2^39");
  if (written && overlaps(dim, n, s)) return ofail(h, RTV_ERR_ARG, std::string(what) + ": rows that are written overlap");
  return RTV_OK;
}

rtv_status check_dim(rtv_ops* h, int d) {
  if (d != 64 && d != 128 && d != 256) return ofail(h, RTV_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  return RTV_OK;
}

rtv_status check_kv_shape(rtv_ops* h, const rtv_kv* a, const char* what) {
  if (!a) return ofail(h, RTV_ERR_ARG, std::string(what) + ": null pointer");
  if (a->dtype != RTV_F32 && a->dtype != RTV_BF16 && a->dtype != RTV_FP8_E4M3)
    return ofail(h, RTV_ERR_ARG, std::string(what) + ": bad dtype");
  if (a->batch < 0 || a->n_tokens < 0 || a->n_heads <= 0)
    return ofail(h, RTV_ERR_SHAPE, std::string(what) + ": bad sizes");
  if (a->batch > 65535 || a->n_heads > 65535) return ofail(h, RTV_ERR_SHAPE, std::string(what) + ": more than 65535 elements or heads");
  if ((long long)a->n_tokens * a->n_heads >= 1LL << 30) return ofail(h, RTV_ERR_SHAPE, std::string(what) + ": 2^30 rows of an element or more");
  return check_dim(h, a->head_dim);
}

// Pointers, strides and scales of keys and values that will be touched.
rtv_status check_kv_memory(rtv_ops* h, const rtv_kv* a, const std::string& what, bool written) {
  OTRY(check_ptr(h, a->k, (what + " k").c_str(), 16));
  OTRY(check_ptr(h, a->v, (what + " v").c_str(), 16));
  OTRY(check_strides(h, what.c_str(), elt_bytes(a->dtype), written, a->head_dim, a->batch, a->batch_stride, a->n_tokens,
                     a->token_stride, a->n_heads, a->head_stride));
  // rows of one call's source may be shared between elements and heads, not between tokens
  if (a->n_tokens > 1 && a->token_stride == 0) return ofail(h, RTV_ERR_ARG, what + ": token stride 0");
  if (written && (a->k == a->v || (a->dtype == RTV_FP8_E4M3 && a->k_scale == a->v_scale)))
    return ofail(h, RTV_ERR_ARG, what + ": keys and values are written to the same place");
  if (a->dtype != RTV_FP8_E4M3) return RTV_OK;
  OTRY(check_ptr(h, a->k_scale, (what + " k_scale").c_str(), 4));
  OTRY(check_ptr(h, a->v_scale, (what + " v_scale").c_str(), 4));
  const int n[3] = {a->batch, a->n_tokens, a->n_heads};
  const long long s[3] = {a->scale_batch_stride, a->scale_token_stride, a->scale_head_stride};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] < 0 || s[i] > (1LL << 39))) return ofail(h, RTV_ERR_ARG, what + ": bad scale stride");
  if (written && overlaps(1, n, s)) return ofail(h, RTV_ERR_ARG, what + ": scales that are written overlap");
  return RTV_OK;
}

rtv_status launched(rtv_ops* h, cudaError_t e, const char* what) {
  if (e == cudaSuccess) return RTV_OK;
  cudaGetLastError();
  return ofail(h, RTV_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

CacheCall cache_call(const rtv_ops* h, const rtv_kv* rows, const rtv_kv* cache) {
  CacheCall c{};
  c.rows.base = (char*)rows->k;
  c.rows.outer_bytes = (char*)rows->v - (char*)rows->k;
  c.rows.sb = rows->batch_stride;
  c.rows.st = rows->token_stride;
  c.rows.sh = rows->head_stride;
  c.cache.codes = (uint8_t*)cache->k;
  c.cache.codes_outer = (uint8_t*)cache->v - (uint8_t*)cache->k;
  c.cache.scales = cache->k_scale;
  c.cache.scales_outer = (char*)cache->v_scale - (char*)cache->k_scale;
  c.cache.sb = cache->batch_stride;
  c.cache.st = cache->token_stride;
  c.cache.sh = cache->head_stride;
  c.cache.fb = cache->scale_batch_stride;
  c.cache.ft = cache->scale_token_stride;
  c.cache.fh = cache->scale_head_stride;
  c.outer = 2;
  c.batch = rows->batch;
  c.tokens = rows->n_tokens;
  c.heads = rows->n_heads;
  c.dim = rows->head_dim;
  c.capacity = cache->n_tokens;
  c.bf16 = rows->dtype == RTV_BF16;
  c.status = h->status;
  return c;
}

rtv_status check_cache_pair(rtv_ops* h, const rtv_kv* rows, const char* what, const rtv_kv* cache) {
  OTRY(check_kv_shape(h, rows, what));
  OTRY(check_kv_shape(h, cache, "cache"));
  if (rows->dtype == RTV_FP8_E4M3) return ofail(h, RTV_ERR_ARG, std::string(what) + ": fp32 or bf16 rows expected");
  if (cache->dtype != RTV_FP8_E4M3) return ofail(h, RTV_ERR_ARG, "cache: E4M3 codes expected");
  if (rows->batch != cache->batch || rows->n_heads != cache->n_heads || rows->head_dim != cache->head_dim)
    return ofail(h, RTV_ERR_SHAPE, std::string(what) + " and cache differ in batch, heads or head_dim");
  return RTV_OK;
}

// Checks of the shapes of an attention call, and its description without pointers.
rtv_status attention_shape(rtv_ops* h, const rtv_queries* q, const rtv_kv* pre, const rtv_kv* own, AttnCall* c) {
  if (!q) return ofail(h, RTV_ERR_ARG, "queries: null pointer");
  if (q->dtype != RTV_F32 && q->dtype != RTV_BF16) return ofail(h, RTV_ERR_ARG, "queries: fp32 or bf16 expected");
  if (q->batch < 0 || q->n_tokens < 0 || q->n_heads <= 0) return ofail(h, RTV_ERR_SHAPE, "queries: bad sizes");
  OTRY(check_dim(h, q->head_dim));
  if (!std::isfinite(q->scale) || !std::isnormal(q->scale * 1.4426950408889634f))
    return ofail(h, RTV_ERR_ARG, "queries: scale must be a normal number");
  const rtv_kv* any = own ? own : pre;
  for (const rtv_kv* a : {pre, own}) {
    if (!a) continue;
    const char* what = a == pre ? "prefix" : "keys";
    OTRY(check_kv_shape(h, a, what));
    if (a->head_dim != q->head_dim || a->n_heads != any->n_heads || q->n_heads % a->n_heads)
      return ofail(h, RTV_ERR_SHAPE, std::string(what) + ": heads or head_dim do not fit the queries");
    if (a->dtype != q->dtype && a->dtype != RTV_FP8_E4M3)
      return ofail(h, RTV_ERR_ARG, std::string(what) + ": neither the queries' dtype nor E4M3");
    if (a->batch != (a == pre ? 1 : q->batch)) return ofail(h, RTV_ERR_SHAPE, std::string(what) + ": wrong batch");
  }
  const long long rows = (long long)q->batch * q->n_tokens;
  if (rows * q->n_heads > 0x7FFFFFFFLL) return ofail(h, RTV_ERR_SHAPE, "queries: more than 2^31 - 1 rows");
  *c = AttnCall{};
  c->bf16 = q->dtype == RTV_BF16;
  c->B = q->batch;
  c->Tq = q->n_tokens;
  c->Hq = q->n_heads;
  c->Hkv = any->n_heads;
  c->group = c->Hq / c->Hkv;
  c->D = q->head_dim;
  auto source = [](const rtv_kv* a, KvSource* s, int* f8) {
    if (!a) return;
    *f8 = a->dtype == RTV_FP8_E4M3;
    s->len = a->n_tokens;
  };
  source(pre, &c->pre, &c->pre_f8);
  source(own, &c->own, &c->own_f8);
  if (rows > 0) c->plan = plan_attention(*c, h->attn);
  return RTV_OK;
}

rtv_status attention(rtv_ops* h, const rtv_queries* q, const rtv_kv* pre, const unsigned char* pre_mask,
                     const rtv_kv* own, const int* lens, const unsigned char* mask, long long mask_stride,
                     void* workspace, size_t workspace_bytes, rtv_stream stream) {
  AttnCall c;
  OTRY(attention_shape(h, q, pre, own, &c));
  if (c.B == 0 || c.Tq == 0) return RTV_OK;
  OTRY(check_ptr(h, q->q, "q", 16));
  OTRY(check_ptr(h, q->out, "out", 16));
  const long long eb = elt_bytes(q->dtype);
  OTRY(check_strides(h, "q", eb, false, c.D, c.B, q->q_batch_stride, c.Tq, q->q_token_stride, c.Hq, q->q_head_stride));
  OTRY(check_strides(h, "out", eb, true, c.D, c.B, q->out_batch_stride, c.Tq, q->out_token_stride, c.Hq, q->out_head_stride));
  if (q->lse) OTRY(check_ptr(h, q->lse, "lse", 4));
  auto source = [&](const rtv_kv* a, const char* what, const int* l, const unsigned char* m, long long ms, KvSource* s) -> rtv_status {
    if (!a || a->n_tokens == 0) return RTV_OK;
    OTRY(check_kv_memory(h, a, what, false));
    if (l) OTRY(check_ptr(h, l, "lengths", 4));
    if (m) OTRY(check_ptr(h, m, "mask", 1));
    if (m && ms < 0) return ofail(h, RTV_ERR_ARG, "mask: negative stride");
    s->k = a->k;
    s->v = a->v;
    s->ks = a->k_scale;
    s->vs = a->v_scale;
    s->sb = a->batch_stride;
    s->st = a->token_stride;
    s->sh = a->head_stride;
    s->fb = a->scale_batch_stride;
    s->ft = a->scale_token_stride;
    s->fh = a->scale_head_stride;
    s->lens = l;
    s->mask = m;
    s->mask_sb = ms;
    return RTV_OK;
  };
  OTRY(source(pre, "prefix", nullptr, pre_mask, 0, &c.pre));
  OTRY(source(own, "keys", lens, mask, mask_stride, &c.own));
  const size_t need = attention_workspace(c);
  if (need) {
    if (workspace_bytes < need) return ofail(h, RTV_ERR_SHAPE, "workspace: " + std::to_string(need) + " bytes needed");
    OTRY(check_ptr(h, workspace, "workspace", 256));
  }
  c.q = q->q;
  c.out = q->out;
  c.lse = q->lse;
  c.qb = q->q_batch_stride;
  c.qt = q->q_token_stride;
  c.qh = q->q_head_stride;
  c.ob = q->out_batch_stride;
  c.ot = q->out_token_stride;
  c.oh = q->out_head_stride;
  c.scale_log2 = (float)((double)q->scale * 1.4426950408889634);
  c.status = h->status;
  c.timeout_ns = kTimeoutNs;
  DeviceGuard dg(h->device);
  return launched(h, launch_attention(c, workspace, (cudaStream_t)stream), "attention");
}

}  // namespace

extern "C" {

rtv_status rtv_ops_create(int cuda_device, rtv_ops** out) {
  if (!out) return RTV_ERR_ARG;
  *out = nullptr;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || cuda_device < 0 || cuda_device >= ndev) {
    cudaGetLastError();
    return RTV_ERR_CUDA;
  }
  rtv_ops* h = new (std::nothrow) rtv_ops();
  if (!h) return RTV_ERR_OOM;
  h->device = cuda_device;
  DeviceGuard dg(cuda_device);
  cudaError_t e = configure_attention(&h->attn);
  if (e == cudaSuccess) e = cudaMalloc(&h->status, sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, sizeof(unsigned));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaGetLastError();
    rtv_ops_destroy(h);
    return e == cudaErrorMemoryAllocation ? RTV_ERR_OOM : RTV_ERR_CUDA;
  }
  *out = h;
  return RTV_OK;
}

rtv_status rtv_kv_write(rtv_ops* ops, const rtv_kv* src, const rtv_kv* cache, const int* start, int first,
                        const int* count, rtv_stream stream) {
  return guarded(ops, [&]() -> rtv_status {
    OTRY(check_cache_pair(ops, src, "source", cache));
    if (src->batch == 0 || src->n_tokens == 0) return RTV_OK;
    if (cache->n_tokens == 0) return ofail(ops, RTV_ERR_SHAPE, "cache: no tokens");
    if (!start && (first < 0 || (!count && (long long)first + src->n_tokens > cache->n_tokens)))
      return ofail(ops, RTV_ERR_SHAPE, "tokens fall outside the cache");
    OTRY(check_kv_memory(ops, src, "source", false));
    OTRY(check_kv_memory(ops, cache, "cache", true));
    if (start) OTRY(check_ptr(ops, start, "start", 4));
    if (count) OTRY(check_ptr(ops, count, "count", 4));
    CacheCall c = cache_call(ops, src, cache);
    c.first = first;
    c.start = start;
    c.lens = count;
    DeviceGuard dg(ops->device);
    return launched(ops, launch_kv_write(c, (cudaStream_t)stream), "cache write");
  });
}

rtv_status rtv_kv_read(rtv_ops* ops, const rtv_kv* cache, int first, const int* lens, const rtv_kv* dst,
                       rtv_stream stream) {
  return guarded(ops, [&]() -> rtv_status {
    OTRY(check_cache_pair(ops, dst, "destination", cache));
    if (dst->batch == 0 || dst->n_tokens == 0) return RTV_OK;
    if (first < 0 || (long long)first + dst->n_tokens > cache->n_tokens)
      return ofail(ops, RTV_ERR_SHAPE, "tokens fall outside the cache");
    OTRY(check_kv_memory(ops, cache, "cache", false));
    OTRY(check_kv_memory(ops, dst, "destination", true));
    if (lens) OTRY(check_ptr(ops, lens, "lengths", 4));
    CacheCall c = cache_call(ops, dst, cache);
    c.first = first;
    c.lens = lens;
    DeviceGuard dg(ops->device);
    return launched(ops, launch_kv_read(c, (cudaStream_t)stream), "cache read");
  });
}

rtv_status rtv_cross_attention(rtv_ops* ops, const rtv_queries* q, const rtv_kv* kv, const int* lens,
                               const unsigned char* mask, long long mask_stride, void* workspace,
                               size_t workspace_bytes, rtv_stream stream) {
  return guarded(ops, [&]() -> rtv_status {
    if (!kv) return ofail(ops, RTV_ERR_ARG, "keys: null pointer");
    return attention(ops, q, nullptr, nullptr, kv, lens, mask, mask_stride, workspace, workspace_bytes, stream);
  });
}

rtv_status rtv_cross_attention_workspace(rtv_ops* ops, const rtv_queries* q, const rtv_kv* kv, size_t* bytes) {
  return guarded(ops, [&]() -> rtv_status {
    if (!kv || !bytes) return ofail(ops, RTV_ERR_ARG, "null pointer");
    AttnCall c;
    OTRY(attention_shape(ops, q, nullptr, kv, &c));
    *bytes = attention_workspace(c);
    return RTV_OK;
  });
}

rtv_status rtv_shared_attention(rtv_ops* ops, const rtv_queries* q, const rtv_kv* prefix,
                                const unsigned char* prefix_mask, const rtv_kv* own, const int* own_lens,
                                void* workspace, size_t workspace_bytes, rtv_stream stream) {
  return guarded(ops, [&]() -> rtv_status {
    if (!prefix) return ofail(ops, RTV_ERR_ARG, "prefix: null pointer");
    if (own && own->dtype == RTV_FP8_E4M3) return ofail(ops, RTV_ERR_UNSUPPORTED, "own keys in E4M3");
    return attention(ops, q, prefix, prefix_mask, own, own_lens, nullptr, 0, workspace, workspace_bytes, stream);
  });
}

rtv_status rtv_shared_attention_workspace(rtv_ops* ops, const rtv_queries* q, const rtv_kv* prefix, const rtv_kv* own,
                                          size_t* bytes) {
  return guarded(ops, [&]() -> rtv_status {
    if (!prefix || !bytes) return ofail(ops, RTV_ERR_ARG, "null pointer");
    AttnCall c;
    OTRY(attention_shape(ops, q, prefix, own, &c));
    *bytes = attention_workspace(c);
    return RTV_OK;
  });
}

rtv_status rtv_ops_device_status(rtv_ops* ops, unsigned* bits) {
  return guarded(ops, [&]() -> rtv_status {
    if (!bits) return ofail(ops, RTV_ERR_ARG, "null pointer");
    DeviceGuard dg(ops->device);
    unsigned v = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&v, ops->status, sizeof v, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && v) e = cudaMemset(ops->status, 0, sizeof v);
    OTRY(launched(ops, e, "device status"));
    *bits = v;
    if (v & RTV_DEV_TIMEOUT) return ofail(ops, RTV_ERR_TIMEOUT, "a device-side wait gave up");
    return RTV_OK;
  });
}

const char* rtv_ops_last_error(rtv_ops* ops) { return ops ? ops->last_error.c_str() : "null operator handle"; }

void rtv_ops_destroy(rtv_ops* ops) {
  if (!ops) return;
  DeviceGuard dg(ops->device);
  cudaDeviceSynchronize();
  if (ops->status) cudaFree(ops->status);
  cudaGetLastError();
  delete ops;
}

}  // extern "C"
