// The expert's prefix cache parked in E4M3 and installed again: the cache
// operators' write and read over the library's own cache, every layer's keys
// and values in one launch.
#include <string>

#include "cache_ops.h"
#include "fastpath.h"
#include "runtime.h"

namespace {

rtv_status sfail(rtv_ctx* ctx, rtv_status s, const std::string& msg) {
  ctx->last_error = msg;
  return s;
}

rtv_status check_memory(rtv_ctx* ctx, const void* p, const char* what) {
  cudaPointerAttributes at{};
  if (!p || (uintptr_t)p % 16) return sfail(ctx, RTV_ERR_ARG, std::string(what) + ": null or not 16-byte aligned");
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess || at.type != cudaMemoryTypeDevice || at.device != ctx->device) {
    cudaGetLastError();
    return sfail(ctx, RTV_ERR_ARG, std::string(what) + ": not device memory of the context's GPU");
  }
  return RTV_OK;
}

// The library's cache [L][2][Bmax][Hkv][Pmax][D] beside codes [L][2][batch][Hkv][P][D] and their scales.
rtv::CacheCall describe(rtv_ctx* ctx, void* codes, float* scales, int P, int batch) {
  const rtv_expert_config& k = ctx->cfg;
  rtv::CacheCall c{};
  c.rows.base = (char*)ctx->prefix_kv;
  c.rows.st = k.head_dim;
  c.rows.sh = (long long)k.max_prefix_len * k.head_dim;
  c.rows.sb = c.rows.sh * k.n_kv_heads;
  c.rows.outer_bytes = c.rows.sb * k.max_batch * ctx->elt;
  c.cache.codes = (uint8_t*)codes;
  c.cache.scales = scales;
  c.cache.st = k.head_dim;
  c.cache.sh = (long long)P * k.head_dim;
  c.cache.sb = c.cache.sh * k.n_kv_heads;
  c.cache.codes_outer = c.cache.sb * batch;
  c.cache.ft = 1;
  c.cache.fh = P;
  c.cache.fb = (long long)P * k.n_kv_heads;
  c.cache.scales_outer = c.cache.fb * batch * (long long)sizeof(float);
  c.outer = 2 * k.n_layers;
  c.batch = batch;
  c.tokens = c.capacity = P;
  c.heads = k.n_kv_heads;
  c.dim = k.head_dim;
  c.bf16 = k.dtype == RTV_BF16;
  c.status = ctx->status;
  return c;
}

rtv_status check_dim(rtv_ctx* ctx) {
  const int d = ctx->cfg.head_dim;
  return d == 64 || d == 128 || d == 256 ? RTV_OK : sfail(ctx, RTV_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
}

}  // namespace

extern "C" {

rtv_status rtv_get_prefix_kv_quantized(rtv_ctx* ctx, void* codes, float* scales, int prefix_len, int batch,
                                       rtv_stream stream) {
  if (!ctx) return RTV_ERR_ARG;
  if (!ctx->have_prefix) return sfail(ctx, RTV_ERR_STATE, "no prefix is installed");
  if (prefix_len != ctx->prefix_len || batch != ctx->prefix_batch)
    return sfail(ctx, RTV_ERR_SHAPE, "the installed prefix has another length or batch");
  rtv_status s = check_dim(ctx);
  if (s == RTV_OK) s = check_memory(ctx, codes, "codes");
  if (s == RTV_OK) s = check_memory(ctx, scales, "scales");
  if (s != RTV_OK) return s;
  rtv::DeviceGuard dg(ctx->device);
  const cudaError_t e = rtv::launch_kv_write(describe(ctx, codes, scales, ctx->prefix_len, ctx->prefix_batch), (cudaStream_t)stream);
  return e == cudaSuccess ? RTV_OK : sfail(ctx, RTV_ERR_CUDA, std::string("prefix quantisation: ") + cudaGetErrorString(e));
}

rtv_status rtv_set_prefix_kv_quantized(rtv_ctx* ctx, const void* codes, const float* scales, int prefix_len, int batch,
                                       rtv_stream stream) {
  if (!ctx) return RTV_ERR_ARG;
  const rtv_expert_config& k = ctx->cfg;
  if (prefix_len <= 0 || prefix_len > k.max_prefix_len || batch <= 0 || batch > k.max_batch)
    return sfail(ctx, RTV_ERR_SHAPE, "prefix_len or batch out of range");
  if (ctx->use_fast && !rtv::fast_supports_prefix(ctx, prefix_len))
    return sfail(ctx, RTV_ERR_UNSUPPORTED, "prefix length not supported by the tensor-core path");
  rtv_status s = check_dim(ctx);
  if (s == RTV_OK) s = check_memory(ctx, codes, "codes");
  if (s == RTV_OK) s = check_memory(ctx, scales, "scales");
  if (s != RTV_OK) return s;
  rtv::DeviceGuard dg(ctx->device);
  const cudaError_t e = rtv::launch_kv_read(describe(ctx, const_cast<void*>(codes), const_cast<float*>(scales), prefix_len, batch),
                                            (cudaStream_t)stream);
  if (e != cudaSuccess) return sfail(ctx, RTV_ERR_CUDA, std::string("prefix read: ") + cudaGetErrorString(e));
  // The rows are the new prefix's from here on: until the tiles are too, no call may read either.
  ctx->have_prefix = false;
  if (ctx->use_fast) s = rtv::fast_prefix_update(ctx, batch, prefix_len, (cudaStream_t)stream);
  if (s != RTV_OK) return s;
  ctx->prefix_len = prefix_len;
  ctx->prefix_batch = batch;
  ctx->have_prefix = true;
  return RTV_OK;
}

}  // extern "C"
