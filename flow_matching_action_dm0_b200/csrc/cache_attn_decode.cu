// bf16 attention over key/value caches for few rows (single tokens: 16 rows
// or less of an element's KV head group), bf16 or E4M3 caches.
//
// Bound by the bytes of the cache, which are read once, straight into
// registers in the layout of the warp-level matrix instruction (m16n8k16, fp32
// accumulate), with no pass through shared memory:
//   S = Q K^T    the order of the dims in a dot product is free, so lane
//                (n, c) reads 16 neighbouring dims of key n in each 64 and
//                they are four k-steps of its B fragment;
//   O = P V      lane (n, c) reads 8 neighbouring dims of its four keys, and
//                the eight of them are eight column tiles of its B fragment
//                (an output column stands for another dim, undone on writing).
// Each warp takes 16 of the 64 keys of a tile with a running maximum of its
// own (raised, and O rescaled, when it has grown by more than 8 in base 2);
// the warps, and the CTAs of a cluster that share a row's keys, join at the
// end, in order.  Keys that are hidden are not read at all.
#include <type_traits>

#include "cache_ops.h"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace rtv {

namespace {

constexpr int kRows = 16, kWarps = 4, kTile = 16 * kWarps;
constexpr float kLazy = 8.f;

__host__ __device__ constexpr int q_row_bytes(int d) { return d * 2 + 16; }   // fragment reads of 8 lanes hit all banks
__host__ __device__ constexpr int o_row_floats(int d) { return d + 4; }
__host__ __device__ constexpr int decode_smem(int d) {
  return kRows * q_row_bytes(d) + kWarps * kRows * (o_row_floats(d) + 2) * 4 + kRows * 8;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two E4M3 codes (low byte first) to two bf16 values, exactly (both fit in f16 and bf16).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  uint32_t h2;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "r"(two));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  return ptx::pack_bf16x2(f.x, f.y);
}

template <int D, bool F8>
__global__ void __launch_bounds__(32 * kWarps, attention_decode_ctas(D))
    attn_decode_kernel(const __grid_constant__ AttnCall c, int cluster) {
  constexpr int NI = D / 64, LO = o_row_floats(D);
  extern __shared__ __align__(16) uint8_t sm[];
  uint8_t* Qs = sm;
  float* Os = reinterpret_cast<float*>(sm + kRows * q_row_bytes(D));   // [kWarps][kRows][LO]
  float2* ML = reinterpret_cast<float2*>(Os + kWarps * kRows * LO);    // [kWarps][kRows] maximum and sum
  float2* Joined = ML + kWarps * kRows;                                // [kRows] of the CTA
  const AttnUnit u = attn_unit(c);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, cc = lane & 3;
  ptx::pdl_launch_dependents();   // (combine_kernel waits for this grid's end before it reads)

  for (int i = tid; i < kRows * (D / 8); i += 32 * kWarps) {
    const int r = i / (D / 8), ch = i - r * (D / 8);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < u.nrows) {
      const int t = r / c.group, g = r - t * c.group;
      v = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(c.q) + u.b * c.qb + t * c.qt +
                                          (long long)(u.kvh * c.group + g) * c.qh + ch * 8);
    }
    *reinterpret_cast<uint4*>(Qs + r * q_row_bytes(D) + ch * 16) = v;
  }
  __syncthreads();

  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // rows n and n + 8
  const float scale = c.scale_log2;
  // One source's type holds for the whole unit; a tile is described by where
  // its 16 keys of this warp begin.
  struct Tile {
    const char *k, *v;
    long long base, st;
    uint32_t bits[2];                               // key k of the first and second eight is seen: bit 4k
    float ks[2], vs[2];                             // E4M3: scales of keys n and n + 8
  };
  constexpr int EB = F8 ? 1 : 2, KW = F8 ? 1 : 2;
  uint4 kr[2][NI][KW];                              // K of the next tile to be scored
  Tile cur{}, nxt{};
  // Looks a tile up and asks for its keys: 16 dims of each 64 for the lane's two keys.
  auto begin = [&](int tile, Tile& t) {
    t.bits[0] = t.bits[1] = 0u;
    if (tile >= u.t1) return;
    const bool pre = tile < u.n0;
    const int k0 = (pre ? tile : tile - u.n0) * kTile + 16 * warp, len = pre ? u.len0 : u.len1;
    if (k0 >= len) return;
    t.st = pre ? c.pre.st : c.own.st;
    t.base = (pre ? 0 : u.b * c.own.sb) + (long long)k0 * t.st + u.kvh * (pre ? c.pre.sh : c.own.sh);
    t.k = reinterpret_cast<const char*>(pre ? c.pre.k : c.own.k);
    t.v = reinterpret_cast<const char*>(pre ? c.pre.v : c.own.v);
    const uint8_t* mask = pre ? c.pre.mask : c.own.mask ? c.own.mask + u.b * c.own.mask_sb : nullptr;
    const long long fb = (pre ? 0 : u.b * c.own.fb) + u.kvh * (pre ? c.pre.fh : c.own.fh), ft = pre ? c.pre.ft : c.own.ft;
    const float *kf = pre ? c.pre.ks : c.own.ks, *vf = pre ? c.pre.vs : c.own.vs;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + n + 8 * h;
      const bool see = k < len && (!mask || mask[k]);
      t.bits[h] = __ballot_sync(0xffffffffu, see);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          kr[h][i][w] = make_uint4(0u, 0u, 0u, 0u);
          if (see)
            kr[h][i][w] =
                __ldcs(reinterpret_cast<const uint4*>(t.k + EB * (t.base + (long long)(n + 8 * h) * t.st + 64 * i + 16 * cc)) + w);
        }
      t.ks[h] = t.vs[h] = 1.f;
      if (F8 && see) {
        t.ks[h] = kf[fb + (long long)k * ft];
        t.vs[h] = vf[fb + (long long)k * ft];
      }
    }
  };
  begin(u.t0, nxt);
  for (int tile = u.t0; tile < u.t1; ++tile) {
    cur = nxt;
    if ((cur.bits[0] | cur.bits[1]) == 0u) {        // (the same in every lane)
      begin(tile + 1, nxt);
      continue;
    }
    // V: 8 dims of each 64 for the lane's four keys, 2c, 2c + 1, then + 8
    using VT = typename std::conditional<F8, uint2, uint4>::type;
    VT vr[NI][4];
    auto load_v = [&](int i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = 2 * cc + (q & 1);
        vr[i][q] = VT{};
        if ((cur.bits[q >> 1] >> (4 * k)) & 1u)
          vr[i][q] = __ldcs(reinterpret_cast<const VT*>(cur.v + EB * (cur.base + (long long)(k + 8 * (q >> 1)) * cur.st + 64 * i + 8 * n)));
      }
    };
    constexpr int NV = D == 256 && !F8 ? 1 : NI;    // V chunks asked for ahead of the scores
#pragma unroll
    for (int i = 0; i < NV; ++i) load_v(i);
    const uint32_t bits[2] = {cur.bits[0], cur.bits[1]};

    float s[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      // Q rows n and n + 8, dims 64 i + 16 c ..: four k-steps of the A fragment
      const uint8_t* qa = Qs + n * q_row_bytes(D) + (64 * i + 16 * cc) * 2;
      const uint4 q0 = *reinterpret_cast<const uint4*>(qa), q1 = *reinterpret_cast<const uint4*>(qa + 16);
      const uint4 q2 = *reinterpret_cast<const uint4*>(qa + 8 * q_row_bytes(D)),
                  q3 = *reinterpret_cast<const uint4*>(qa + 8 * q_row_bytes(D) + 16);
      const uint32_t a[4][4] = {{q0.x, q2.x, q0.y, q2.y}, {q0.z, q2.z, q0.w, q2.w}, {q1.x, q3.x, q1.y, q3.y}, {q1.z, q3.z, q1.w, q3.w}};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t b[8];
        if (F8) {
          const uint32_t w[4] = {kr[h][i][0].x, kr[h][i][0].y, kr[h][i][0].z, kr[h][i][0].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) b[e] = e4m3x2_to_bf16x2((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
        } else {
          b[0] = kr[h][i][0].x, b[1] = kr[h][i][0].y, b[2] = kr[h][i][0].z, b[3] = kr[h][i][0].w;
          b[4] = kr[h][i][KW - 1].x, b[5] = kr[h][i][KW - 1].y, b[6] = kr[h][i][KW - 1].z, b[7] = kr[h][i][KW - 1].w;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) ptx::mma_bf16_16816(s[h], a[t], b[2 * t], b[2 * t + 1]);
      }
    }
    begin(tile + 1, nxt);                           // its keys arrive while this tile's values are used
    // scores of rows n, n + 8 with keys 2c, 2c + 1 (+ 8 h)
    float top[2] = {-INFINITY, -INFINITY}, vw[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = 2 * cc + e;
        const bool on = (bits[h] >> (4 * k)) & 1u;
        const float f = F8 ? __shfl_sync(0xffffffffu, cur.ks[h], 4 * k) * scale : scale;
        vw[h][e] = F8 ? __shfl_sync(0xffffffffu, cur.vs[h], 4 * k) : 1.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          s[h][2 * r + e] = on ? s[h][2 * r + e] * f : -INFINITY;
          top[r] = fmaxf(top[r], s[h][2 * r + e]);
        }
      }
    bool grow = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(m[r], fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2)));
      grow = grow || top[r] - m[r] > kLazy;         // (from -inf too)
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = m[r] == top[r] ? 1.f : ex2(m[r] - top[r]);
        m[r] = top[r];
        l[r] *= f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][2 * r] *= f;
          o[j][2 * r + 1] *= f;
        }
      }
    }
    uint32_t p[4];
    {
      float w[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float b = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = ex2(s[h][2 * r + e] - b);
            l[r] += x;
            // (a hidden key's value is not read, so its scale must not count either)
            w[h][2 * r + e] = F8 ? ((bits[h] >> (4 * (2 * cc + e))) & 1u ? x * vw[h][e] : 0.f) : x;
          }
      }
      p[0] = ptx::pack_bf16x2(w[0][0], w[0][1]);
      p[1] = ptx::pack_bf16x2(w[0][2], w[0][3]);
      p[2] = ptx::pack_bf16x2(w[1][0], w[1][1]);
      p[3] = ptx::pack_bf16x2(w[1][2], w[1][3]);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (i + 1 >= NV && i + 1 < NI) load_v(i + 1);
      uint32_t v[4][4];                             // [key][dims 2w, 2w + 1]
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&vr[i][q]);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[q][e] = F8 ? e4m3x2_to_bf16x2((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) : w[F8 ? 0 : e];
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        ptx::mma_bf16_16816(o[8 * i + 2 * w], p, __byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x5410));
        ptx::mma_bf16_16816(o[8 * i + 2 * w + 1], p, __byte_perm(v[0][w], v[1][w], 0x7632), __byte_perm(v[2][w], v[3][w], 0x7632));
      }
    }
  }

  // ---- join of the warps -------------------------------------------------------
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int row = n + 8 * r;
    // a NaN sum counts with every weight, a sum of 0 (nothing seen) with none
    if (cc == 0) ML[warp * kRows + row] = make_float2(l[r] != l[r] ? INFINITY : l[r] == 0.f ? -INFINITY : m[r], l[r]);
    if (row < u.nrows) {
      float* dst = Os + (warp * kRows + row) * LO + 16 * cc;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 8; e += 4) {            // columns 2c and 2c + 1 are dims 16c + e and 16c + 8 + e
          *reinterpret_cast<float4*>(dst + 64 * i + e) =
              make_float4(o[8 * i + e][2 * r], o[8 * i + e + 1][2 * r], o[8 * i + e + 2][2 * r], o[8 * i + e + 3][2 * r]);
          *reinterpret_cast<float4*>(dst + 64 * i + 8 + e) =
              make_float4(o[8 * i + e][2 * r + 1], o[8 * i + e + 1][2 * r + 1], o[8 * i + e + 2][2 * r + 1], o[8 * i + e + 3][2 * r + 1]);
        }
    }
  }
  __syncthreads();
  const int ranks = cluster > 1 ? cluster : 1;
  const bool split = cluster <= 1 && c.plan.n_slots > 1;
  // Rows r, 64 dims a warp: the four warps' parts, in order, into the first one's place.
  for (int p = warp; p < u.nrows * NI; p += kWarps) {
    const int r = p / NI, d = 64 * (p - r * NI) + 2 * lane;
    float2 ml[kWarps], x[kWarps];
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      ml[k] = ML[k * kRows + r];
      x[k] = *reinterpret_cast<const float2*>(Os + (k * kRows + r) * LO + d);
      top = fmaxf(top, ml[k].x);
    }
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (ml[k].x == -INFINITY) continue;
      const float w = exp2f(ml[k].x - top);
      sum += w * ml[k].y;
      acc.x = fmaf(w, x[k].x, acc.x);
      acc.y = fmaf(w, x[k].y, acc.y);
    }
    const float2 mine = make_float2(sum != sum ? INFINITY : sum == 0.f ? -INFINITY : top, sum);
    if (ranks > 1) {
      *reinterpret_cast<float2*>(Os + r * LO + d) = acc;
      if (d == 0) Joined[r] = mine;
      continue;
    }
    const long long row = u.row0 + r;
    if (split) {
      const long long pr = part_row(c, u, row);
      if (d == 0) *reinterpret_cast<float2*>(c.part_ml + pr * 2) = mine;
      if (sum != 0.f) *reinterpret_cast<float2*>(c.part_o + pr * D + d) = acc;
    } else {
      const int t = r / c.group, h = u.kvh * c.group + r - t * c.group;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(c.out) + u.b * c.ob + t * c.ot + h * c.oh + d) =
          ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
      if (d == 0 && c.lse)
        c.lse[((long long)u.b * c.Tq + t) * c.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
  }
  if (ranks == 1) return;
  // The CTAs of the cluster, in order, by distributed shared memory.
  ptx::cluster_sync();
  const int rank = (int)ptx::cluster_ctarank();
  const uint32_t os_a = ptx::smem_u32(Os), j_a = ptx::smem_u32(Joined);
  for (int p = rank * kWarps + warp; p < u.nrows * NI; p += ranks * kWarps) {
    const int r = p / NI, d = 64 * (p - r * NI) + 2 * lane;
    float2 ml[8], x[8];
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      x[k] = make_float2(0.f, 0.f);
      if (k < ranks) {
        ml[k] = ptx::ld_dsmem_f32x2(ptx::mapa(j_a + r * 8, k));
        x[k] = ptx::ld_dsmem_f32x2(ptx::mapa(os_a + (r * LO + d) * 4, k));
      }
      top = fmaxf(top, ml[k].x);
    }
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (ml[k].x == -INFINITY) continue;
      const float w = exp2f(ml[k].x - top);
      sum += w * ml[k].y;
      acc.x = fmaf(w, x[k].x, acc.x);
      acc.y = fmaf(w, x[k].y, acc.y);
    }
    const int t = r / c.group, h = u.kvh * c.group + r - t * c.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(c.out) + u.b * c.ob + t * c.ot + h * c.oh + d) =
        ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
    if (d == 0 && c.lse)
      c.lse[((long long)u.b * c.Tq + t) * c.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  }
  ptx::cluster_sync();                              // the others have read this CTA's shared memory
}

template <int D, bool F8>
cudaError_t launch(const AttnCall& c, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)c.B * c.plan.tiles_e * c.plan.ne), c.Hkv);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = decode_smem(D);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = c.plan.cluster;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, F8>, c, c.plan.cluster);
}

template <int D, bool F8>
cudaError_t configure() {
  return cudaFuncSetAttribute(attn_decode_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, decode_smem(D));
}

}  // namespace

cudaError_t configure_attention_decode() {
  cudaError_t e = cudaSuccess;
  auto chain = [&](cudaError_t x) { e = e == cudaSuccess ? x : e; };
  chain(configure<64, false>());
  chain(configure<128, false>());
  chain(configure<256, false>());
  chain(configure<64, true>());
  chain(configure<128, true>());
  chain(configure<256, true>());
  return e;
}

cudaError_t launch_attention_decode(const AttnCall& c, cudaStream_t st) {
  const bool f8 = c.own.len ? c.own_f8 : c.pre_f8;   // (the plan takes one type)
  if (f8) return c.D == 64 ? launch<64, true>(c, st) : c.D == 128 ? launch<128, true>(c, st) : launch<256, true>(c, st);
  return c.D == 64 ? launch<64, false>(c, st) : c.D == 128 ? launch<128, false>(c, st) : launch<256, false>(c, st);
}

}  // namespace rtv
