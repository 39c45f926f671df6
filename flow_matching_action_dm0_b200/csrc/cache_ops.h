// Operators over key/value caches: what the entry points (cache_ops.cu), the
// fp32 kernels and the tensor-core attention (cache_attn_tc.cu) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rtv.h"

namespace rtv {

// Keys and values one attention call reads: one prefix for every batch
// element, or each element's own tokens.
struct KvSource {
  const void *k, *v;
  const float *ks, *vs;        // E4M3 only
  long long sb, st, sh;        // element strides: batch, token, head
  long long fb, ft, fh;        // scale strides
  int len;                     // tokens (0: the source is absent)
  const int* lens;             // [B] valid tokens, or nullptr
  const uint8_t* mask;         // key mask (row b at b * mask_sb), or nullptr
  long long mask_sb;
};

// How an attention call is split over CTAs.  A "row" is one (query token,
// query head) of a KV head's group: row r of element b is token r / group,
// head kvh * group + r % group.  Stacked units take bm_s consecutive rows of
// the whole batch over a range of the prefix; element units take bm_e rows of
// one element over a range of [prefix ; own keys] (prefix_in_elem) or of its
// own keys.  Each row has n_slots partial results (slot = range), joined by
// combine_kernel when there is more than one; ranges of a unit that form a
// cluster join in it and count as one.
struct AttnPlan {
  int bm_s, bm_e;              // rows of a stacked and of an element unit
  int kt_s, kt_e;              // keys of their tiles
  int rows_b;                  // rows of one element: query tokens * group
  int tiles_s, ns;             // stacked units: row tiles, key ranges (0: none)
  int tiles_e, ne;             // element units: row tiles per element, key ranges (0: none)
  int prefix_in_elem;          // element units read the prefix too
  int decode;                  // element units are the few-row kernel's
  int cluster;                 // a unit's ranges, whose CTAs join by distributed shared memory (1: not so)
  int unpack_pre, unpack_own;  // E4M3 sources that are read back to bf16 in the workspace first
  int n_slots;                 // partial results of a row
};

struct AttnCall {
  const void* q;
  void* out;
  float* lse;
  long long qb, qt, qh;        // element strides of q: batch, token, head
  long long ob, ot, oh;
  int out_tiled_rows;          // > 0: out is the tiled GEMM input of that many block rows (bf16)
  int bf16;                    // queries and output: 1 bf16, 0 fp32
  int B, Tq, Hq, Hkv, group, D;
  float scale_log2;            // scale * log2(e)
  KvSource pre, own;
  int pre_f8, own_f8;
  AttnPlan plan;
  unsigned unit0;              // first unit of a launch
  float* part_o;               // [Hkv][n_slots][B * rows_b][D] unnormalised rows (n_slots > 1)
  float* part_ml;              // [Hkv][n_slots][B * rows_b][2] their maximum (base 2) and sum
  unsigned* status;
  long long timeout_ns;
};

constexpr int kMaxCluster = 8;
// What a plan needs to know of a GPU.  Each handle holds its own, filled when
// it is made, so that a call's split (and workspace, and the order of its
// sums) depends on its shape and its GPU alone.
struct AttnDevice {
  int num_sms;
  int at_once[3][kMaxCluster + 1];   // [head_dim 64, 128, 256][ranks]: CTAs of the tensor-core kernel that run at once in clusters
};
// Sets the kernels' attributes on the current device (outside any capture) and describes it.
cudaError_t configure_attention(AttnDevice* dev);
// Chooses the split for a call whose shape fields are set.
AttnPlan plan_attention(const AttnCall& c, const AttnDevice& dev);
// Bytes of the partial results of a planned call.
size_t attention_workspace(const AttnCall& c);
// Enqueues a planned call; workspace as above.
cudaError_t launch_attention(AttnCall& c, void* workspace, cudaStream_t st);
// Plans and enqueues a call whose workspace is given; makes fewer ranges of the keys where it is too small.
cudaError_t run_attention(AttnCall& c, const AttnDevice& dev, void* workspace, size_t workspace_bytes, cudaStream_t st);
// The tensor-core kernel (bf16 queries).
cudaError_t configure_attention_tc(AttnDevice* dev);
cudaError_t launch_attention_tc(const AttnCall& c, cudaStream_t st);
int attention_tc_rows(int D);   // rows of a CTA
constexpr int attention_tc_keys(int D) { return D == 256 ? 64 : 128; }   // keys of a tile
// The few-row kernel (bf16 queries, 16 rows of an element or less).
cudaError_t configure_attention_decode();
cudaError_t launch_attention_decode(const AttnCall& c, cudaStream_t st);
constexpr int kDecodeRows = 16;
constexpr int decode_groups(int D) { return D == 256 ? 6 : 4; }                          // of 16 keys each, in a tile
constexpr int attention_decode_ctas(int D) { return D == 256 ? 1 : D == 128 ? 3 : 4; }   // CTAs of an SM

// One tensor of rows [outer][batch][token][head][D] for the cache kernels;
// strides in elements, the outer index (keys, values, or layers of both)
// in bytes, so that it can step between two allocations.
struct RowsView {
  char* base;
  long long outer_bytes;
  long long sb, st, sh;
};
struct CacheView {
  uint8_t* codes;
  float* scales;
  long long codes_outer, scales_outer;   // bytes
  long long sb, st, sh, fb, ft, fh;
};
struct CacheCall {
  RowsView rows;               // fp32 or bf16 rows: source of a write, destination of a read
  CacheView cache;
  int outer, batch, tokens, heads, dim, capacity, bf16;
  int first;
  const int* start;            // write: [batch] or nullptr
  const int* lens;             // write: count; read: valid tokens ([batch] or nullptr)
  int skip;                    // read: tokens behind the valid ones are left as they are, not zeroed
  unsigned* status;
};
cudaError_t launch_kv_write(const CacheCall& c, cudaStream_t st);
cudaError_t launch_kv_read(const CacheCall& c, cudaStream_t st);

// What one CTA of an attention kernel computes.
struct AttnUnit {
  int kvh, b;                  // b: the element of an element unit (0 for a stacked one)
  long long row0;              // first row in [0, B * rows_b)
  int nrows, slot;
  int t0, t1;                  // its tiles of the list [prefix tiles ; own tiles]
  int n0;                      // prefix tiles in the list
  int len0, len1;              // keys of the two sources it may read
};

__device__ __forceinline__ int valid_len(const KvSource& s, int b, unsigned* status) {
  if (!s.lens) return s.len;
  const int n = s.lens[b];
  if ((n < 0 || n > s.len) && threadIdx.x == 0) atomicOr(status, RTV_DEV_BOUNDS);
  return min(max(n, 0), s.len);
}

__device__ __forceinline__ AttnUnit attn_unit(const AttnCall& c) {
  const AttnPlan& p = c.plan;
  AttnUnit u;
  u.kvh = blockIdx.y;
  unsigned x = blockIdx.x + c.unit0;
  const unsigned stacked = (unsigned)p.tiles_s * p.ns;
  int split, nsplit, kt;
  if (x < stacked) {
    kt = p.kt_s;
    const bool by_range = p.cluster > 1;   // a cluster's CTAs are neighbours; otherwise those of a range are
    const unsigned inner = by_range ? p.ns : p.tiles_s, y = x / inner, z = x - y * inner;
    split = (int)(by_range ? z : y);
    const int tile = (int)(by_range ? y : z);
    nsplit = p.ns;
    u.slot = split;
    u.b = 0;
    u.row0 = (long long)tile * p.bm_s;
    u.nrows = (int)min((long long)p.bm_s, (long long)c.B * p.rows_b - u.row0);
    u.len0 = valid_len(c.pre, 0, c.status);
    u.len1 = 0;
  } else {
    x -= stacked;
    kt = p.kt_e;
    const bool by_range = p.cluster > 1;
    const unsigned inner = by_range ? p.ne : p.tiles_e, outer = by_range ? p.tiles_e : p.ne;
    const unsigned y = x / inner, z = x - y * inner;
    u.b = (int)(y / outer);
    const unsigned w = y - (unsigned)u.b * outer;
    split = (int)(by_range ? z : w);
    const int tile = (int)(by_range ? w : z);
    nsplit = p.ne;
    u.slot = p.n_slots > 1 ? p.ns + split : 0;
    u.row0 = (long long)u.b * p.rows_b + (long long)tile * p.bm_e;
    u.nrows = min(p.bm_e, p.rows_b - tile * p.bm_e);
    u.len0 = p.prefix_in_elem ? valid_len(c.pre, 0, c.status) : 0;
    u.len1 = valid_len(c.own, u.b, c.status);
  }
  u.n0 = (u.len0 + kt - 1) / kt;
  const unsigned n = u.n0 + (u.len1 + kt - 1) / kt;
  if (nsplit == 1) {
    u.t0 = 0;
    u.t1 = (int)n;
  } else {
    const unsigned each = n / (unsigned)nsplit, rest = n - each * nsplit;   // the first `rest` ranges take one tile more
    u.t0 = (int)(each * split + min((unsigned)split, rest));
    u.t1 = u.t0 + (int)each + ((unsigned)split < rest ? 1 : 0);
  }
  return u;
}

// Where elements d.. of a query's output go (bf16; d and the run within 8 elements).
__device__ __forceinline__ __nv_bfloat16* out_bf16(const AttnCall& c, unsigned b, unsigned t, unsigned h, int d) {
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(c.out);
  if (c.out_tiled_rows == 0) return o + b * c.ob + t * c.ot + h * c.oh + d;
  // the projections' tiled input: [column / 64][row][64], 16-byte chunks permuted by the row
  const unsigned row = b * c.Tq + t, col = h * c.D + d;
  return o + ((size_t)(col >> 6) * c.out_tiled_rows + row) * 64 + ((((col >> 3) & 7) ^ (row & 7)) << 3) + (col & 7);
}

// Where a row's partial result goes.
__device__ __forceinline__ long long part_row(const AttnCall& c, const AttnUnit& u, long long row) {
  return ((long long)u.kvh * c.plan.n_slots + u.slot) * ((long long)c.B * c.plan.rows_b) + row;
}

}  // namespace rtv
