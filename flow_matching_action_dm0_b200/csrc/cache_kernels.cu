// Kernels of the operators over key/value caches that run outside the tensor
// cores: the E4M3 cache's write and read, fp32 attention, and the join of
// partial attention results.
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "cache_ops.h"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace rtv {

namespace {

__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t two) {
  uint32_t h2;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "r"(two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}
// Two fp32 values to E4M3 codes, nearest even (lo in the low byte).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t t;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(t) : "f"(hi), "f"(lo));
  return t;
}

// ---------------------------------------------------------------------------
// Cache write: scale = 2^e, e = max(-126, least e with max|x| <= 448 * 2^e);
// codes = E4M3(x * 2^-e) (exact product, one rounding).  A row is D/8 lanes
// of 8 elements; the maximum over the row's magnitudes is taken on their bit
// patterns, which order like the values with infinities and NaN on top.
// Four rows' loads are in flight a thread (one: 92 us), past L1 as nothing is
// read twice.  Measured on B200: 64 x 816 tokens x 8 heads x 128, bf16, 57 us
// for 245 MB (some sequences short) and 72 us for the whole 324 MB, 4.3-4.5
// TB/s where a copy reaches 6.6.  What holds it is the instructions, not the
// memory: issue slots are 82% in use, DRAM 46%.  fp32 rows bring twice the
// bytes to the same work and reach 6.7 TB/s (538 MB in 80 us).
// ---------------------------------------------------------------------------
constexpr int kRowsAhead = 4;                   // rows whose loads a thread has in flight

template <typename T, int D>
__global__ void __launch_bounds__(256) kv_write_kernel(const __grid_constant__ CacheCall c) {
  constexpr int LPR = D / 8;                    // lanes of a row
  constexpr int RPB = 256 / LPR;                // rows of a block's step
  constexpr int U = kRowsAhead;
  const int b = blockIdx.y, o = blockIdx.z;
  const int lane = threadIdx.x % LPR;
  int n = c.tokens;
  if (c.lens) {
    const int want = c.lens[b];
    n = min(max(want, 0), c.tokens);
    if (n != want && threadIdx.x == 0 && blockIdx.x == 0) atomicOr(c.status, RTV_DEV_BOUNDS);
  }
  const long long at0 = (long long)c.first + (c.start ? c.start[b] : 0);
  const unsigned rows = (unsigned)n * c.heads, step = gridDim.x * RPB * U;   // (tokens * heads < 2^30)
  const char* src0 = c.rows.base + o * c.rows.outer_bytes + (b * c.rows.sb + lane * 8) * (long long)sizeof(T);
  uint8_t* dst0 = c.cache.codes + o * c.cache.codes_outer + b * c.cache.sb + lane * 8;
  float* f0 = reinterpret_cast<float*>(reinterpret_cast<char*>(c.cache.scales) + o * c.cache.scales_outer) + b * c.cache.fb;
  for (unsigned r0 = blockIdx.x * RPB * U; r0 < rows; r0 += step) {
    uint4 v[U][sizeof(T) / 2];
    unsigned t[U], h[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const unsigned r = r0 + k * RPB + threadIdx.x / LPR;
      t[k] = r / (unsigned)c.heads;
      h[k] = r - t[k] * c.heads;
      const uint4* src = reinterpret_cast<const uint4*>(src0 + ((long long)t[k] * c.rows.st + h[k] * c.rows.sh) * (long long)sizeof(T));
#pragma unroll
      for (int w = 0; w < (int)sizeof(T) / 2; ++w) v[k][w] = r < rows ? __ldcs(src + w) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float x[8];
      if (sizeof(T) == 2) {
        const uint32_t w[4] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16);
          x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      } else {
        constexpr int q = sizeof(T) / 2 - 1;
        x[0] = __uint_as_float(v[k][0].x), x[1] = __uint_as_float(v[k][0].y), x[2] = __uint_as_float(v[k][0].z);
        x[3] = __uint_as_float(v[k][0].w), x[4] = __uint_as_float(v[k][q].x), x[5] = __uint_as_float(v[k][q].y);
        x[6] = __uint_as_float(v[k][q].z), x[7] = __uint_as_float(v[k][q].w);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
      for (int i = LPR / 2; i > 0; i >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, i));
      if (r0 + k * RPB + threadIdx.x / LPR >= rows) continue;
      const long long at = at0 + t[k];
      if (at < 0 || at >= c.capacity) {
        if (lane == 0) atomicOr(c.status, RTV_DEV_BOUNDS);
        continue;
      }
      // 448 = 1.75 * 2^8
      const int e = max(-126, (int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0));
      const bool finite = top < 0x7F800000u;
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      uint2 codes = make_uint2(0u, 0u);
      if (finite) {
        codes.x = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) | f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16;
        codes.y = f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) | f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16;
      }
      *reinterpret_cast<uint2*>(dst0 + at * c.cache.st + h[k] * c.cache.sh) = codes;
      if (lane == 0)
        f0[at * c.cache.ft + h[k] * c.cache.fh] = finite ? __uint_as_float((uint32_t)(127 + e) << 23) : __uint_as_float(0x7FC00000u);
    }
  }
}

// Cache read: code * scale in fp32, rounded to T.  A row is D/16 lanes of 16
// codes, 32 bytes of bf16 a lane.  72 x 816 tokens x 4 heads of 256 dims, 333
// MB in 65 us, 5.1 TB/s: warps wait for their loads (issue slots 48% in use).
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ CacheCall c) {
  constexpr int LPR = D / 16;
  constexpr int RPB = 256 / LPR;
  constexpr int U = kRowsAhead;
  const int b = blockIdx.y, o = blockIdx.z;
  const int lane = threadIdx.x % LPR;
  int n = c.capacity;   // valid cache tokens
  if (c.lens) {
    const int want = c.lens[b];
    n = min(max(want, 0), c.capacity);
    if (n != want && threadIdx.x == 0 && blockIdx.x == 0) atomicOr(c.status, RTV_DEV_BOUNDS);
  }
  const unsigned rows = (unsigned)c.tokens * c.heads, step = gridDim.x * RPB * U;   // (tokens * heads < 2^30)
  const uint8_t* src0 = c.cache.codes + o * c.cache.codes_outer + b * c.cache.sb + lane * 16;
  const float* f0 = reinterpret_cast<const float*>(reinterpret_cast<const char*>(c.cache.scales) + o * c.cache.scales_outer) + b * c.cache.fb;
  char* dst0 = c.rows.base + o * c.rows.outer_bytes + (b * c.rows.sb + lane * 16) * (long long)sizeof(T);
  for (unsigned r0 = blockIdx.x * RPB * U; r0 < rows; r0 += step) {
    uint4 v[U];
    float s[U];
    unsigned t[U], h[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const unsigned r = r0 + k * RPB + threadIdx.x / LPR;
      t[k] = r / (unsigned)c.heads;
      h[k] = r - t[k] * c.heads;
      const long long at = (long long)c.first + t[k];
      const bool real = r < rows && at < n;
      v[k] = real ? __ldcs(reinterpret_cast<const uint4*>(src0 + at * c.cache.st + h[k] * c.cache.sh)) : make_uint4(0u, 0u, 0u, 0u);
      s[k] = real ? f0[at * c.cache.ft + h[k] * c.cache.fh] : 1.f;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (r0 + k * RPB + threadIdx.x / LPR >= rows || (c.skip && (long long)c.first + t[k] >= n)) continue;
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      float x[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 p = e4m3x2_to_f32x2((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
        x[2 * i] = p.x * s[k];
        x[2 * i + 1] = p.y * s[k];
      }
      uint4* dst = reinterpret_cast<uint4*>(dst0 + ((long long)t[k] * c.rows.st + h[k] * c.rows.sh) * (long long)sizeof(T));
      if (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          __stcs(dst + i, make_uint4(ptx::pack_bf16x2(x[8 * i], x[8 * i + 1]), ptx::pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                     ptx::pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), ptx::pack_bf16x2(x[8 * i + 6], x[8 * i + 7])));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __stcs(dst + i, make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                                     __float_as_uint(x[4 * i + 3])));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// fp32 attention: BM rows against tiles of 64 keys, 256 threads as 16 x 16;
// thread (ty, tx) holds rows ty + 16 i, keys tx + 16 j of the scores and
// columns 4 tx + 64 c of the output.  One pass over the keys with the running
// maximum (base 2) and sum of each row.  The next keys are copied while the
// values are used and the next values while the keys are.  Hidden keys score
// -inf and are copied as zeros, whatever they hold.  The work is fp32 (no
// tensor core keeps 24 bits), so the bound is the FMA pipe and, before it, the
// shared memory that feeds it: 64 rows reuse a key or value four times from
// registers, 16 rows (taken where a unit has no more) once.  Measured on
// B200: 8 suffixes of 51 tokens x 4 heads of 64 dims over up to 561 keys, 21
// us, 6 of them the join's; 3 suffixes of nine tokens over 73, 14 us, 11 of
// them the kernel's.
// ---------------------------------------------------------------------------
constexpr int kKeys = 64;

__host__ __device__ constexpr int attn_f32_smem(int bm, int d) {
  return 4 * (bm * (d + 4) + kKeys * (d + 4) + kKeys * d + bm * (kKeys + 4) + 2 * kKeys);
}

// Four E4M3 codes of a key or value row times the row's scale.
__device__ __forceinline__ float4 load_codes4(const void* base, const float* scales, long long off, long long foff) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(base) + off);
  const float s = scales[foff];
  const float2 a = e4m3x2_to_f32x2(w & 0xFFFFu), b = e4m3x2_to_f32x2(w >> 16);
  return make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
}

template <int D, int BM>
__global__ void __launch_bounds__(256) attn_f32_kernel(const __grid_constant__ AttnCall c) {
  constexpr int TM = BM / 16, LD = D + 4, LP = kKeys + 4, C4 = D / 4;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + BM * LD;
  float* Vs = Ks + kKeys * LD;
  float* Ps = Vs + kKeys * D;
  float* Ok = Ps + BM * LP;       // [2][kKeys] 1: the tile's key is seen
  const AttnUnit u = attn_unit(c);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  ptx::pdl_launch_dependents();   // (combine_kernel waits for this grid's end before it reads)

  for (int i = tid; i < BM * C4; i += 256) {
    const int r = i / C4, d = (i - r * C4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < u.nrows) {
      const long long row = u.row0 + r;
      const long long b = row / c.plan.rows_b;
      const int rr = (int)(row - b * c.plan.rows_b), t = rr / c.group, g = rr - t * c.group;
      v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(c.q) + b * c.qb + t * c.qt +
                                           (long long)(u.kvh * c.group + g) * c.qh + d);
    }
    *reinterpret_cast<float4*>(Qs + r * LD + d) = v;
  }

  float m[TM], l[TM];
  float4 acc[TM][D / 64];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 64; ++k) acc[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  auto look = [&](int tile) {     // which keys of a tile are seen
    if (tile >= u.t1 || tid >= kKeys) return;
    const bool pre = tile < u.n0;
    const int k = (pre ? tile : tile - u.n0) * kKeys + tid;
    const uint8_t* mask = pre ? c.pre.mask : c.own.mask ? c.own.mask + u.b * c.own.mask_sb : nullptr;
    Ok[(tile & 1) * kKeys + tid] = k < (pre ? u.len0 : u.len1) && (!mask || mask[k]) ? 1.f : 0.f;
  };
  auto copy = [&](int tile, bool val) {   // its keys or values (after look and a barrier); one commit group
    if (tile < u.t1) {
      const bool pre = tile < u.n0, f8 = pre ? c.pre_f8 : c.own_f8;
      const int k0 = (pre ? tile : tile - u.n0) * kKeys;
      const long long st = pre ? c.pre.st : c.own.st, ft = pre ? c.pre.ft : c.own.ft;
      const long long base = (pre ? 0 : u.b * c.own.sb) + k0 * st + u.kvh * (pre ? c.pre.sh : c.own.sh);
      const long long fbase = (pre ? 0 : u.b * c.own.fb) + k0 * ft + u.kvh * (pre ? c.pre.fh : c.own.fh);
      const void* src = pre ? (val ? c.pre.v : c.pre.k) : (val ? c.own.v : c.own.k);
      const float* scales = pre ? (val ? c.pre.vs : c.pre.ks) : (val ? c.own.vs : c.own.ks);
      float* dst = val ? Vs : Ks;
      const int ld = val ? D : LD;
#pragma unroll 4
      for (int i = tid; i < kKeys * C4; i += 256) {
        const int r = i / C4, d = (i - r * C4) * 4;
        const bool on = Ok[(tile & 1) * kKeys + r] != 0.f;
        if (f8) {
          *reinterpret_cast<float4*>(dst + r * ld + d) =
              on ? load_codes4(src, scales, base + r * st + d, fbase + r * ft) : make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
          const float* from = reinterpret_cast<const float*>(src) + (on ? base + r * st + d : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst + r * ld + d)), "l"(from), "r"(on ? 16 : 0)
                       : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  look(u.t0);
  __syncthreads();
  copy(u.t0, false);
  copy(u.t0, true);
  for (int tile = u.t0; tile < u.t1; ++tile) {
    const float* ok = Ok + (tile & 1) * kKeys;
    look(tile + 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");   // the keys
    __syncthreads();
    float sc[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll (TM == 1 ? 8 : 4)
    for (int d = 0; d < D; d += 4) {
      float4 qv[TM], kv[4];
#pragma unroll
      for (int i = 0; i < TM; ++i) qv[i] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * LD + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * LD + d);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sc[i][j] = fmaf(qv[i].x, kv[j].x,
                          fmaf(qv[i].y, kv[j].y, fmaf(qv[i].z, kv[j].z, fmaf(qv[i].w, kv[j].w, sc[i][j]))));
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sc[i][j] = ok[tx + 16 * j] != 0.f ? sc[i][j] * c.scale_log2 : -INFINITY;
        top = fmaxf(top, sc[i][j]);
      }
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float mn = fmaxf(m[i], top);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m[i] - base);   // 0 before the row's first key
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(sc[i][j] - base);
        Ps[(ty + 16 * i) * LP + tx + 16 * j] = p;
        sum += p;
      }
      l[i] = l[i] * corr + sum;   // this lane's share of the row's sum
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        acc[i][k].x *= corr;
        acc[i][k].y *= corr;
        acc[i][k].z *= corr;
        acc[i][k].w *= corr;
      }
    }
    __syncthreads();              // (a row's weights are written and read by the same half-warp) the keys are done with
    copy(tile + 1, false);
    asm volatile("cp.async.wait_group 1;" ::: "memory");   // the values
    __syncthreads();
#pragma unroll (TM == 1 ? 4 : 2)
    for (int k4 = 0; k4 < kKeys; k4 += 4) {
      float4 p[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) p[i] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * LP + k4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc) {
          const float4 v = *reinterpret_cast<const float4*>(Vs + (k4 + kk) * D + 64 * cc + 4 * tx);
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
            acc[i][cc].x = fmaf(w, v.x, acc[i][cc].x);
            acc[i][cc].y = fmaf(w, v.y, acc[i][cc].y);
            acc[i][cc].z = fmaf(w, v.z, acc[i][cc].z);
            acc[i][cc].w = fmaf(w, v.w, acc[i][cc].w);
          }
        }
      }
    }
    __syncthreads();              // the values are done with
    copy(tile + 1, true);
  }

#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], k);
    const int r = ty + 16 * i;
    if (r >= u.nrows) continue;
    const long long row = u.row0 + r;
    if (c.plan.n_slots > 1) {
      const long long pr = part_row(c, u, row);
      // a NaN sum counts with every weight, a sum of 0 (nothing seen) with none
      const float mo = l[i] != l[i] ? INFINITY : l[i] == 0.f ? -INFINITY : m[i];
      if (tx == 0) *reinterpret_cast<float2*>(c.part_ml + pr * 2) = make_float2(mo, l[i]);
      if (mo == -INFINITY) continue;   // the join does not read an empty part
#pragma unroll
      for (int k = 0; k < D / 64; ++k) *reinterpret_cast<float4*>(c.part_o + pr * D + 64 * k + 4 * tx) = acc[i][k];
      continue;
    }
    const long long b = row / c.plan.rows_b;
    const int rr = (int)(row - b * c.plan.rows_b), t = rr / c.group, h = u.kvh * c.group + rr - t * c.group;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    float* dst = reinterpret_cast<float*>(c.out) + b * c.ob + t * c.ot + h * c.oh + 4 * tx;
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      *reinterpret_cast<float4*>(dst + 64 * k) =
          make_float4(acc[i][k].x * inv, acc[i][k].y * inv, acc[i][k].z * inv, acc[i][k].w * inv);
    if (c.lse && tx == 0)
      c.lse[(b * c.Tq + t) * c.Hq + h] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
  }
}

// Join of a row's partial results: out = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k.
// `per` warps share a row, each taking every per-th slot with its loads in
// flight together; their sums are added in warp order.  Empty parts (m = -inf)
// do not count.  Bound by the latency of its two dependent loads; it starts
// while the attention ends and waits for it.
template <typename QT, int D>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnCall c, int per) {
  constexpr int V = D >= 128 ? 4 : 2, NC = D / (32 * V);   // elements of a lane's load, loads of a lane
  __shared__ float sums[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % per;
  const long long rows = (long long)c.B * c.plan.rows_b;
  const long long row = (long long)blockIdx.x * (8 / per) + warp / per;
  const int kvh = blockIdx.y, n = c.plan.n_slots;
  const bool real = row < rows;
  const long long base = (long long)kvh * n * rows + row;
  ptx::pdl_wait();
  float top = -INFINITY, sum = 0.f;
  float acc[NC][V] = {};
  if (real) {
    const float2* ml = reinterpret_cast<const float2*>(c.part_ml) + base;
    for (int k = lane; k < n; k += 32) top = fmaxf(top, ml[k * rows].x);
    top = warp_max(top);
    for (int k = lane; k < n; k += 32) {
      const float2 x = ml[k * rows];
      if (x.x != -INFINITY) sum += exp2f(x.x - top) * x.y;
    }
    sum = warp_sum(sum);
#pragma unroll 4
    for (int k = sub; k < n; k += per) {
      const float mk = ml[k * rows].x;            // (an empty part is loaded, whatever it holds, and not used)
      const float w = mk == -INFINITY ? 0.f : exp2f(mk - top);
      const float* src = c.part_o + (base + k * rows) * D + lane * V;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float v[V];
        if (V == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src + 32 * V * i);
        else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src + 32 * V * i);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[i][e] = mk == -INFINITY ? acc[i][e] : fmaf(w, v[e], acc[i][e]);
      }
    }
  }
  if (per > 1) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) sums[warp][32 * V * i + lane * V + e] = acc[i][e];
    __syncthreads();
    if (sub == 0)
      for (int k = 1; k < per; ++k)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) acc[i][e] += sums[warp + k][32 * V * i + lane * V + e];
  }
  if (!real || sub) return;
  const unsigned b = (unsigned)row / (unsigned)c.plan.rows_b, rr = (unsigned)row - b * (unsigned)c.plan.rows_b;
  const unsigned t = rr / (unsigned)c.group, h = kvh * c.group + rr - t * (unsigned)c.group;
  const float inv = top == -INFINITY ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = 32 * V * i + lane * V;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      if (sizeof(QT) == 4)
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(c.out) + b * c.ob + t * c.ot + h * c.oh + d + e) =
            make_float2(acc[i][e] * inv, acc[i][e + 1] * inv);
      else
        *reinterpret_cast<uint32_t*>(out_bf16(c, b, t, h, d + e)) = ptx::pack_bf16x2(acc[i][e] * inv, acc[i][e + 1] * inv);
    }
  }
  if (c.lse && lane == 0)
    c.lse[((long long)b * c.Tq + t) * c.Hq + h] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int D, int BM>
cudaError_t launch_f32_units(AttnCall& c, unsigned first, long long units, cudaStream_t st) {
  if (units == 0) return cudaSuccess;
  c.unit0 = first;
  attn_f32_kernel<D, BM><<<dim3((unsigned)units, c.Hkv), 256, attn_f32_smem(BM, D), st>>>(c);
  return cudaGetLastError();
}
// Stacked and element units may have different rows: a launch each.
template <int D>
cudaError_t launch_f32(AttnCall& c, cudaStream_t st) {
  const AttnPlan& p = c.plan;
  const long long ns = (long long)p.tiles_s * p.ns, ne = (long long)c.B * p.tiles_e * p.ne;
  cudaError_t e = p.bm_s == 16 ? launch_f32_units<D, 16>(c, 0, ns, st) : launch_f32_units<D, 64>(c, 0, ns, st);
  if (e == cudaSuccess)
    e = p.bm_e == 16 ? launch_f32_units<D, 16>(c, (unsigned)ns, ne, st) : launch_f32_units<D, 64>(c, (unsigned)ns, ne, st);
  c.unit0 = 0;
  return e;
}

template <typename QT, int D>
cudaError_t launch_combine(const AttnCall& c, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const int per = c.plan.n_slots >= 16 ? 8 : c.plan.n_slots >= 4 ? 2 : 1;   // warps of a row
  cfg.gridDim = dim3((unsigned)(((long long)c.B * c.plan.rows_b * per + 7) / 8), c.Hkv);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<QT, D>, c, per);
}

template <int D>
cudaError_t launch_all(AttnCall& c, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (!c.bf16) e = launch_f32<D>(c, st);
  if (c.bf16 && (c.plan.ns || !c.plan.decode)) e = launch_attention_tc(c, st);
  if (e == cudaSuccess && c.plan.decode && c.plan.ne) {
    c.unit0 = (unsigned)c.plan.tiles_s * c.plan.ns;
    e = launch_attention_decode(c, st);
  }
  if (e != cudaSuccess || c.plan.n_slots == 1) return e;
  return c.bf16 ? launch_combine<__nv_bfloat16, D>(c, st) : launch_combine<float, D>(c, st);
}

template <int D, int BM>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(attn_f32_kernel<D, BM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              attn_f32_smem(BM, D));
}

template <typename T, int D>
cudaError_t write_d(const CacheCall& c, const dim3& grid, cudaStream_t st) {
  kv_write_kernel<T, D><<<grid, 256, 0, st>>>(c);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t read_d(const CacheCall& c, const dim3& grid, cudaStream_t st) {
  kv_read_kernel<T, D><<<grid, 256, 0, st>>>(c);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write(const CacheCall& c, cudaStream_t st) {
  const long long rpb = 2048 / c.dim * kRowsAhead, rows = (long long)c.tokens * c.heads;
  const dim3 grid((unsigned)std::min((rows + rpb - 1) / rpb, 65535LL), c.batch, c.outer);
  if (c.bf16) return c.dim == 64    ? write_d<__nv_bfloat16, 64>(c, grid, st)
                     : c.dim == 128 ? write_d<__nv_bfloat16, 128>(c, grid, st)
                                    : write_d<__nv_bfloat16, 256>(c, grid, st);
  return c.dim == 64 ? write_d<float, 64>(c, grid, st)
         : c.dim == 128 ? write_d<float, 128>(c, grid, st) : write_d<float, 256>(c, grid, st);
}

cudaError_t launch_kv_read(const CacheCall& c, cudaStream_t st) {
  const long long rpb = 4096 / c.dim * kRowsAhead, rows = (long long)c.tokens * c.heads;
  const dim3 grid((unsigned)std::min((rows + rpb - 1) / rpb, 65535LL), c.batch, c.outer);
  if (c.bf16) return c.dim == 64    ? read_d<__nv_bfloat16, 64>(c, grid, st)
                     : c.dim == 128 ? read_d<__nv_bfloat16, 128>(c, grid, st)
                                    : read_d<__nv_bfloat16, 256>(c, grid, st);
  return c.dim == 64 ? read_d<float, 64>(c, grid, st)
         : c.dim == 128 ? read_d<float, 128>(c, grid, st) : read_d<float, 256>(c, grid, st);
}

// How many key ranges a unit's tiles are split over, and about how long the
// launch then takes (us).  `fixed` is a CTA's start and end, `tile` a key tile
// at an SM's full rate and `alone` with one CTA on it; a second range brings
// the join: its launch, and every row's parts written and read, or, for up to
// eight ranges where `at_once` knows how many CTAs run in clusters of that
// size, the cluster's own.  (Measured on B200, head_dim 256: 64 units of 128
// rows x 816 keys take 22.4 us in one range, 20.5 in two that join in a
// cluster and 26.5 in two with the join's launch; 32 units of 5070 keys 90 us
// in one, 43 in a cluster of four, 49 in four with the join's launch.)
constexpr float kClusterJoin = 2.f;   // us
struct Split {
  int n;
  bool cluster;
  float us;
};
template <typename AtOnce>
static Split best_split(long long units, int tiles, int slots, int per_sm, float fixed, float tile, float alone, float join,
                        float join_each, AtOnce at_once) {
  Split best{1, false, 1e30f};
  for (int n = 1; n <= std::min(std::max(tiles, 1), 64); ++n) {
    const long long ctas = units * n;
    const float shared = (float)std::min<long long>(per_sm, (ctas + slots - 1) / slots) * tile;   // CTAs of an SM share its rate
    const float range = fixed + (float)((tiles + n - 1) / n) * std::max(alone, shared);
    auto waves = [&](long long together) { return (float)((ctas + together - 1) / together); };
    const float us = waves((long long)slots * per_sm) * range + (n > 1 ? join : 0.f) + join_each * n;
    if (us < best.us) best = {n, false, us};
    const int together = n > 1 && n <= kMaxCluster ? at_once(n) : 0;
    const float us_c = together ? waves(together) * (range + kClusterJoin) : 1e30f;
    if (us_c < best.us) best = {n, true, us_c};
  }
  return best;
}

AttnPlan plan_attention(const AttnCall& c, const AttnDevice& dev) {
  AttnPlan p{};
  p.rows_b = c.Tq * c.group;
  p.cluster = 1;
  p.decode = c.bf16 && p.rows_b <= kDecodeRows;
  // Rows of several elements share a tile (and its pass over the prefix) when
  // one element's rows would leave half of it empty.
  const bool stack = c.pre.len > 0 && c.B > 1 && p.rows_b <= (c.bf16 ? 64 : 16);
  p.prefix_in_elem = c.pre.len > 0 && !stack;
  // E4M3: the few-row kernel reads one source of codes itself; the others are
  // read back to bf16 first, once for all of the rows that go over them, by a
  // launch that moves five times the codes' bytes.  (Measured on B200, 32
  // caches of 16384 tokens x 2 heads x 128: 16 rows from the codes 80 us, 20
  // rows read back first 250, where bf16 caches take 113 and 104.  One prefix
  // of 8192 tokens for 64 single tokens with own keys: 33 us, in bf16 28.)
  const bool codes = p.decode && !stack && (!c.pre.len || !c.own.len);
  p.unpack_pre = c.bf16 && c.pre.len > 0 && c.pre_f8 && !codes;
  p.unpack_own = c.bf16 && c.own.len > 0 && c.own_f8 && !codes;
  const long long rows = (long long)c.B * p.rows_b;
  const float join = 3.f, join_each = (float)(rows * c.Hkv * c.D) * 8.f / 4e6f;   // us: launch; a part of all rows at 4 TB/s
  auto tiles_of = [](long long keys, int kt) { return (int)((keys + kt - 1) / kt); };
  // Rows of a unit and its ranges, for `elems` elements of `rows_e` rows over `keys` keys.
  auto shape = [&](long long elems, long long rows_e, long long keys, int kt, bool alone_kind, int* bm, int* tiles, int* n) {
    float best = 1e30f;
    const int choices[2] = {c.bf16 ? 128 : 16, c.bf16 ? attention_tc_rows(c.D) : 64};
    for (const int rows_u : choices) {
      const long long tu = (rows_e + rows_u - 1) / rows_u;
      float fixed, tile, alone;
      int per_sm = 1;
      if (c.bf16) {
        // two row tiles share a CTA's loads
        fixed = 6.f;
        tile = alone = c.D == 256 ? 0.85f : c.D == 128 ? (rows_u == 256 ? 1.95f : 1.1f) : (rows_u == 256 ? 1.5f : 0.9f);
      } else {
        fixed = 4.f;
        tile = (rows_u == 64 ? 2.6f : 1.f) * (float)c.D / 64.f;
        alone = (rows_u == 64 ? 4.5f : 3.f) * (float)c.D / 64.f;
        per_sm = std::max(1, 227 * 1024 / (attn_f32_smem(rows_u, c.D) + 1024));
      }
      // clusters: all of the call's units are of one kind and the tensor cores'
      const Split s = best_split(elems * tu * c.Hkv, tiles_of(keys, kt), dev.num_sms, per_sm, fixed, tile, alone, join, join_each,
                                 [&](int ranks) { return c.bf16 && alone_kind ? dev.at_once[c.D / 128][ranks] : 0; });
      if (s.us < best) {
        best = s.us;
        *bm = rows_u;
        *tiles = (int)tu;
        *n = s.n;
        p.cluster = s.cluster ? s.n : 1;
      }
    }
  };
  p.kt_s = c.bf16 ? attention_tc_keys(c.D) : kKeys;
  p.kt_e = p.decode ? 16 * decode_groups(c.D) : p.kt_s;
  p.bm_s = c.bf16 ? 128 : 64;
  if (stack) shape(1, rows, c.pre.len, p.kt_s, c.own.len == 0, &p.bm_s, &p.tiles_s, &p.ns);
  if (!stack || c.own.len > 0) {
    const long long keys = (long long)c.own.len + (p.prefix_in_elem ? c.pre.len : 0);
    if (p.decode) {
      p.bm_e = kDecodeRows;
      p.tiles_e = 1;
      const long long units = (long long)c.B * c.Hkv, slots = (long long)attention_decode_ctas(c.D) * dev.num_sms;
      p.ne = (int)std::max(1LL, std::min<long long>({slots / units, tiles_of(keys, p.kt_e), 64}));
      // Up to eight ranges join in a cluster, without a second launch.
      if (!stack && p.ne > 1) {
        if (p.ne <= 16) p.ne = std::min(p.ne, 8);
        if (p.ne <= 8) p.cluster = p.ne;
      }
    } else {
      shape(c.B, p.rows_b, keys, p.kt_e, !stack, &p.bm_e, &p.tiles_e, &p.ne);
    }
  }
  p.n_slots = p.cluster > 1 ? 1 : p.ns + p.ne;
  return p;
}

namespace {
size_t round_256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t part_bytes(const AttnCall& c) {
  if (c.plan.n_slots <= 1) return 0;
  return round_256((size_t)c.Hkv * c.plan.n_slots * ((size_t)c.B * c.plan.rows_b) * (size_t)(c.D + 2) * 4);
}
// K (and as much V) of a source in bf16.
size_t unpacked_bytes(const AttnCall& c, const KvSource& s, int batch) {
  return round_256((size_t)batch * c.Hkv * s.len * c.D * 2);
}
// Reads a source back to bf16 at `to`, dense [batch][head][token][D], and points the call at it.
cudaError_t unpack(const AttnCall& c, KvSource& s, int batch, char* to, cudaStream_t st) {
  const size_t bytes = unpacked_bytes(c, s, batch);
  CacheCall r{};
  r.rows.base = to;
  r.rows.outer_bytes = (long long)bytes;
  r.rows.sh = (long long)s.len * c.D;
  r.rows.sb = r.rows.sh * c.Hkv;
  r.rows.st = c.D;
  r.cache.codes = (uint8_t*)s.k;
  r.cache.codes_outer = (const char*)s.v - (const char*)s.k;
  r.cache.scales = (float*)s.ks;
  r.cache.scales_outer = (const char*)s.vs - (const char*)s.ks;
  r.cache.sb = s.sb, r.cache.st = s.st, r.cache.sh = s.sh;
  r.cache.fb = s.fb, r.cache.ft = s.ft, r.cache.fh = s.fh;
  r.outer = 2;
  r.batch = batch;
  r.tokens = r.capacity = s.len;
  r.heads = c.Hkv;
  r.dim = c.D;
  r.bf16 = 1;
  r.lens = s.lens;
  r.skip = 1;
  r.status = c.status;
  s.k = to;
  s.v = to + bytes;
  s.ks = s.vs = nullptr;
  s.sb = r.rows.sb, s.st = r.rows.st, s.sh = r.rows.sh;
  return launch_kv_read(r, st);
}
}  // namespace

size_t attention_workspace(const AttnCall& c) {
  return part_bytes(c) + (c.plan.unpack_pre ? 2 * unpacked_bytes(c, c.pre, 1) : 0) +
         (c.plan.unpack_own ? 2 * unpacked_bytes(c, c.own, c.B) : 0);
}

cudaError_t configure_attention(AttnDevice* dev) {
  *dev = AttnDevice{};
  int id = 0;
  cudaError_t e = cudaGetDevice(&id);
  auto chain = [&](cudaError_t x) { e = e == cudaSuccess ? x : e; };
  chain(cudaDeviceGetAttribute(&dev->num_sms, cudaDevAttrMultiProcessorCount, id));
  chain(set_smem<64, 16>());
  chain(set_smem<64, 64>());
  chain(set_smem<128, 16>());
  chain(set_smem<128, 64>());
  chain(set_smem<256, 16>());
  chain(set_smem<256, 64>());
  chain(configure_attention_tc(dev));
  chain(configure_attention_decode());
  return e;
}

cudaError_t launch_attention(AttnCall& c, void* workspace, cudaStream_t st) {
  char* at = (char*)workspace;
  c.part_o = (float*)at;
  c.part_ml = c.part_o + (size_t)c.Hkv * c.plan.n_slots * ((size_t)c.B * c.plan.rows_b) * c.D;
  at += part_bytes(c);
  cudaError_t e = cudaSuccess;
  if (c.plan.unpack_pre) {
    const size_t bytes = 2 * unpacked_bytes(c, c.pre, 1);
    e = unpack(c, c.pre, 1, at, st);
    at += bytes;
    c.pre_f8 = 0;
  }
  if (e == cudaSuccess && c.plan.unpack_own) {
    e = unpack(c, c.own, c.B, at, st);
    c.own_f8 = 0;
  }
  if (e != cudaSuccess) return e;
  return c.D == 64 ? launch_all<64>(c, st) : c.D == 128 ? launch_all<128>(c, st) : launch_all<256>(c, st);
}

cudaError_t run_attention(AttnCall& c, const AttnDevice& dev, void* workspace, size_t workspace_bytes, cudaStream_t st) {
  c.plan = plan_attention(c, dev);
  // fewer ranges where the caller's workspace holds no more parts
  while (attention_workspace(c) > workspace_bytes && (c.plan.ns > 1 || c.plan.ne > 1)) {
    int& n = c.plan.ns > c.plan.ne ? c.plan.ns : c.plan.ne;
    --n;
    c.plan.n_slots = c.plan.ns + c.plan.ne;
  }
  if (attention_workspace(c) > workspace_bytes) return cudaErrorInvalidValue;
  return launch_attention(c, workspace, st);
}

}  // namespace rtv
