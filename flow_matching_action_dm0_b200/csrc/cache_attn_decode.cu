// bf16 attention over key/value caches for few rows (single tokens: 16 rows
// or less of an element's KV head group), bf16 or E4M3 caches.
//
// Bound by the bytes of the cache, which are read once, by a ring of
// asynchronous copies of each warp's own (16 keys a stage, hidden keys filled
// with zeros and not read), and multiplied by the warp-level matrix
// instruction (m16n8k16, fp32 accumulate):
//   S = Q K^T    the order of the dims in a dot product is free, so lane
//                (n, c) takes 16 neighbouring dims of key n in each 64 and
//                they are four k-steps of its B fragment;
//   O = P V      lane (n, c) takes 8 neighbouring dims of its four keys, and
//                the eight of them are eight column tiles of its B fragment
//                (an output column stands for another dim, undone on writing).
// E4M3 codes become f16 (exactly, one conversion for two) and so do the
// queries, each row times a power of two that brings its largest magnitude to
// 2^14 (what is lost is below 2^-38 of it).  Their products with P are in
// units of 2^(mv - 7), mv the running maximum of score + log2(value scale):
// f16 weights (2^15 at most) hold what matters whatever the scales, 2^-11 of
// each down to 2^-21 of the largest and 2^-32 of the largest below it.  The
// row's sum keeps the maximum m of the scores alone, and O is brought to it at
// the end.
// A group takes 16 keys of a tile with a running maximum of its own (raised,
// and O rescaled, when it has grown by more than 8 in base 2); at head_dim
// 256 it is two warps, each with half of the dims, that add their scores.
// The groups, and the CTAs of a cluster that share a row's keys, join at the
// end, in order.
//
// Measured on B200 (cold L2): 32 single tokens, 8 heads on 2, over E4M3
// caches of up to 16,384 tokens of 128 dims (210 MB), 64 us, 3.3 TB/s; with
// all of them that long (268 MB) 78 us.  The conversions of the codes hold it,
// and with lengths that differ the longest sequences, whose keys are split
// over as many CTAs as the shortest's.  One token, 8 heads on one, over 816 tokens of 256 dims: 12 us, not
// much more than the host takes for the call.

#include "cache_ops.h"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace rtv {

namespace {

constexpr int kRows = 16;
constexpr float kLazy = 8.f;
constexpr float kUp = 7.f;                        // E4M3: weights count in units of 2^(mv - kUp); kUp + kLazy < 16 (f16's range)

template <int D, bool F8>
struct Cfg {
  static constexpr int HV = D == 256 ? 2 : 1;             // warps of a group: each has DW dims
  static constexpr int DW = D / HV, NI = DW / 64;
  static constexpr int G = decode_groups(D);              // groups of a CTA
  static constexpr int kThreads = 32 * G * HV;
  static constexpr int EB = F8 ? 1 : 2;
  static constexpr int CPR = DW * EB / 16;                // 16-byte chunks of a key's row
  static constexpr int kRow = DW * EB, kTileBytes = 16 * kRow;
  static constexpr int kStage = 2 * kTileBytes + 160;     // K, V, 16 + 16 scales, visible keys
  static constexpr int NST = F8 ? 4 : D == 64 ? 3 : 2;       // a warp's stages
  static constexpr int kQRow = D * 2 + 16;                // fragment reads of 8 lanes hit all banks
  static constexpr int LO = D + 4;                        // floats of a staged output row
  static constexpr int kRing = G * HV * NST * kStage;
  static constexpr int kJoin = G * kRows * (LO + 2) * 4 + kRows * 8;
  static constexpr int kMain = kRing > kJoin ? kRing : kJoin;   // the join is staged over the ring
  static constexpr int kExchange = HV == 2 ? G * 2 * 32 * 32 : 0;   // scores of each half
  static constexpr int kSmem = kRows * kQRow + kMain + kExchange + kRows * 4;   // and the queries' factors
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four E4M3 codes (low byte first) to two pairs of f16, exactly.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// C[16x8] += A[16x16] * B[16x8], f16 in, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F8>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F8) mma_f16_16816(c, a, b0, b1);
  else ptx::mma_bf16_16816(c, a, b0, b1);
}
// `bytes` of 16 (16-byte chunks) or 4 from global to shared memory; nothing is read, and zeros written, unless `on`.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::kThreads, attention_decode_ctas(D))
    attn_decode_kernel(const __grid_constant__ AttnCall c, int cluster) {
  using C = Cfg<D, F8>;
  constexpr int NI = C::NI, LO = C::LO, G = C::G, HV = C::HV, CPR = C::CPR, NST = C::NST;
  extern __shared__ __align__(16) uint8_t sm[];
  uint8_t* Qs = sm;
  uint8_t* main_sm = sm + kRows * C::kQRow;
  float* Os = reinterpret_cast<float*>(main_sm);                       // [G][kRows][LO], after the loop
  float2* ML = reinterpret_cast<float2*>(Os + G * kRows * LO);         // [G][kRows] maximum and sum
  float2* Joined = ML + G * kRows;                                     // [kRows] of the CTA
  const AttnUnit u = attn_unit(c);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, cc = lane & 3;
  const int grp = warp % G, half = warp / G, d0 = half * C::DW;        // the warp's keys and dims
  ptx::pdl_launch_dependents();   // (combine_kernel waits for this grid's end before it reads)
  uint8_t* ring = main_sm + warp * NST * C::kStage;
  const uint32_t ring_a = ptx::smem_u32(ring);

  // Where chunk ch of key k lies in a stage's tile: permuted so that the
  // fragment reads of K (two keys a phase) and of V (four) hit all banks.
  auto place = [&](int k, int ch) { return k * C::kRow + ((ch ^ (((((k >> 1) & 3) * 2) ^ ((k & 1) * (F8 ? 4 : 1))) & (CPR - 1))) << 4); };
  // Asks for the warp's 16 keys of a tile; one commit group a tile.
  auto request = [&](int tile, int slot) {
    if (tile < u.t1) {
      const bool pre = tile < u.n0;
      const int k0 = (pre ? tile : tile - u.n0) * (16 * G) + 16 * grp, len = pre ? u.len0 : u.len1;
      const long long st = pre ? c.pre.st : c.own.st;
      const long long base = (pre ? 0 : u.b * c.own.sb) + (long long)k0 * st + u.kvh * (pre ? c.pre.sh : c.own.sh) + d0;
      const uint8_t* mask = pre ? c.pre.mask : c.own.mask ? c.own.mask + u.b * c.own.mask_sb : nullptr;
      const char* kp = reinterpret_cast<const char*>(pre ? c.pre.k : c.own.k);
      const char* vp = reinterpret_cast<const char*>(pre ? c.pre.v : c.own.v);
      const int key = lane & 15;
      const bool see = k0 + key < len && (!mask || mask[k0 + key]);
      const uint32_t bits = __ballot_sync(0xffffffffu, see) & 0xFFFFu;
      const uint32_t dst = ring_a + slot * C::kStage;
#pragma unroll
      for (int i = 0; i < CPR / 2; ++i) {
        const int k = i * (32 / CPR) + lane / CPR, ch = lane % CPR;
        const bool on = (bits >> k) & 1u;
        const long long off = on ? C::EB * (base + (long long)k * st) + ch * 16 : 0;
        copy16(dst + place(k, ch), kp + off, on);
        copy16(dst + C::kTileBytes + place(k, ch), vp + off, on);
      }
      if (F8) {
        const long long off = (pre ? 0 : u.b * c.own.fb) + u.kvh * (pre ? c.pre.fh : c.own.fh) + (long long)(k0 + key) * (pre ? c.pre.ft : c.own.ft);
        copy4(dst + 2 * C::kTileBytes + lane * 4, (lane < 16 ? (pre ? c.pre.ks : c.own.ks) : (pre ? c.pre.vs : c.own.vs)) + (see ? off : 0), see);
      }
      if (lane == 0) *reinterpret_cast<uint32_t*>(ring + slot * C::kStage + 2 * C::kTileBytes + 128) = bits;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) request(u.t0 + i, i);

  for (int i = tid; i < kRows * (D / 8); i += C::kThreads) {
    const int r = i / (D / 8), ch = i - r * (D / 8);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < u.nrows) {
      const int t = r / c.group, g = r - t * c.group;
      v = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(c.q) + u.b * c.qb + t * c.qt +
                                          (long long)(u.kvh * c.group + g) * c.qh + ch * 8);
    }
    *reinterpret_cast<uint4*>(Qs + r * C::kQRow + ch * 16) = v;
  }
  __syncthreads();
  float qf[2] = {1.f, 1.f};                         // factors of rows n and n + 8
  if (F8) {
    float* factor = reinterpret_cast<float*>(sm + C::kSmem) - kRows;
    for (int r = warp; r < kRows; r += G * HV) {
      uint32_t* row = reinterpret_cast<uint32_t*>(Qs + r * C::kQRow);
      uint32_t x[D / 64], top = 0u;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        x[i] = row[i * 32 + lane];
        top = max(top, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      // 2^(14 - exponent of the largest), and its inverse for the scores; 1 for a row of zeros or one that is not finite
      const int e = top == 0u || top >= 0x7F80u ? 0 : min(max((int)(top >> 7) - 127 - 14, -126), 126);
      const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        row[i * 32 + lane] = pack_f16x2(__uint_as_float(x[i] << 16) * f, __uint_as_float(x[i] & 0xFFFF0000u) * f);
      if (lane == 0) factor[r] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
    __syncthreads();
    qf[0] = factor[n];
    qf[1] = factor[n + 8];
  }

  float o[NI * 8][4];
#pragma unroll
  for (int j = 0; j < NI * 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // rows n and n + 8
  float mv[2] = {-INFINITY, -INFINITY};             // E4M3: O counts in units of 2^(mv - kUp) (bf16: of 2^m)
  const float scale = c.scale_log2;
  int slot = 0;
  for (int tile = u.t0; tile < u.t1; ++tile) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
    __syncwarp();
    const uint8_t* stage = ring + slot * C::kStage;
    const uint32_t bits = *reinterpret_cast<const uint32_t*>(stage + 2 * C::kTileBytes + 128);
    // the slot that was used last is free: every lane is past it
    request(tile + NST - 1, slot == 0 ? NST - 1 : slot - 1);
    slot = slot + 1 == NST ? 0 : slot + 1;
    if (bits == 0u) continue;                       // (the same in the warps of a group)

    float s[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      // Q rows n and n + 8, dims 64 i + 16 c ..: four k-steps of the A fragment
      const uint8_t* qa = Qs + n * C::kQRow + (d0 + 64 * i + 16 * cc) * 2;
      const uint4 q0 = *reinterpret_cast<const uint4*>(qa), q1 = *reinterpret_cast<const uint4*>(qa + 16);
      const uint4 q2 = *reinterpret_cast<const uint4*>(qa + 8 * C::kQRow), q3 = *reinterpret_cast<const uint4*>(qa + 8 * C::kQRow + 16);
      const uint32_t a[4][4] = {{q0.x, q2.x, q0.y, q2.y}, {q0.z, q2.z, q0.w, q2.w}, {q1.x, q3.x, q1.y, q3.y}, {q1.z, q3.z, q1.w, q3.w}};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t b[8];
        const int k = n + 8 * h;
        if (F8) {
          const uint4 x = *reinterpret_cast<const uint4*>(stage + place(k, 4 * i + cc));
          e4m3x4_to_f16x4(x.x, b[0], b[1]);
          e4m3x4_to_f16x4(x.y, b[2], b[3]);
          e4m3x4_to_f16x4(x.z, b[4], b[5]);
          e4m3x4_to_f16x4(x.w, b[6], b[7]);
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(stage + place(k, 8 * i + 2 * cc));
          const uint4 y = *reinterpret_cast<const uint4*>(stage + place(k, 8 * i + 2 * cc + 1));
          b[0] = x.x, b[1] = x.y, b[2] = x.z, b[3] = x.w, b[4] = y.x, b[5] = y.y, b[6] = y.z, b[7] = y.w;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) mma<F8>(s[h], a[t], b[2 * t], b[2 * t + 1]);
      }
    }
    if (HV == 2) {   // the halves' scores, added in the same order by both
      float4* ex = reinterpret_cast<float4*>(main_sm + C::kMain) + (size_t)grp * 2 * 64;
      ex[half * 64 + lane] = make_float4(s[0][0], s[0][1], s[0][2], s[0][3]);
      ex[half * 64 + 32 + lane] = make_float4(s[1][0], s[1][1], s[1][2], s[1][3]);
      named_sync(1 + grp, 64);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 x = ex[32 * h + lane], y = ex[64 + 32 * h + lane];
        s[h][0] = x.x + y.x, s[h][1] = x.y + y.y, s[h][2] = x.z + y.z, s[h][3] = x.w + y.w;
      }
      named_sync(1 + grp, 64);
    }
    // scores of rows n, n + 8 with keys 2c, 2c + 1 (+ 8 h)
    float top[2] = {-INFINITY, -INFINITY}, topv[2] = {-INFINITY, -INFINITY};
    const float* sc = reinterpret_cast<const float*>(stage + 2 * C::kTileBytes);
    float vw[4] = {1.f, 1.f, 1.f, 1.f}, lv[4] = {0.f, 0.f, 0.f, 0.f};   // value scales of keys 2c, 2c + 1, then + 8; their logarithms
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 kw = make_float2(1.f, 1.f);
      if (F8) {
        kw = *reinterpret_cast<const float2*>(sc + 8 * h + 2 * cc);
        const float2 x = *reinterpret_cast<const float2*>(sc + 16 + 8 * h + 2 * cc);
        vw[2 * h] = x.x, vw[2 * h + 1] = x.y;
        lv[2 * h] = lg2(fabsf(x.x)), lv[2 * h + 1] = lg2(fabsf(x.y));   // (a hidden key's scale was filled with 0: -inf)
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool on = (bits >> (8 * h + 2 * cc + e)) & 1u;
        const float f = F8 ? (e ? kw.y : kw.x) * scale : scale;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          s[h][2 * r + e] = on ? s[h][2 * r + e] * (F8 ? f * qf[r] : f) : -INFINITY;
          top[r] = fmaxf(top[r], s[h][2 * r + e]);
          if (F8) topv[r] = fmaxf(topv[r], s[h][2 * r + e] + lv[2 * h + e]);
        }
      }
    }
    bool grow = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(m[r], fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2)));
      if (F8) {
        topv[r] = fmaxf(topv[r], __shfl_xor_sync(0xffffffffu, topv[r], 1));
        topv[r] = fmaxf(mv[r], fmaxf(topv[r], __shfl_xor_sync(0xffffffffu, topv[r], 2)));
        l[r] *= m[r] == top[r] ? 1.f : ex2(m[r] - top[r]);
        m[r] = top[r];
        grow = grow || topv[r] - mv[r] > kLazy;
      } else {
        grow = grow || top[r] - m[r] > kLazy;       // (from -inf too)
      }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float f;
        if (F8) {
          f = mv[r] == topv[r] ? 1.f : ex2(mv[r] - topv[r]);
          mv[r] = topv[r];
        } else {
          f = m[r] == top[r] ? 1.f : ex2(m[r] - top[r]);
          m[r] = top[r];
          l[r] *= f;
        }
#pragma unroll
        for (int j = 0; j < NI * 8; ++j) {
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
        const float b = m[r] == -INFINITY ? 0.f : m[r], bv = mv[r] == -INFINITY ? 0.f : mv[r] - kUp;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = ex2(s[h][2 * r + e] - b);
            l[r] += x;
            w[h][2 * r + e] = F8 ? copysignf(ex2(s[h][2 * r + e] + lv[2 * h + e] - bv), vw[2 * h + e]) : x;
          }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = w[k >> 1][2 * (k & 1)], b = w[k >> 1][2 * (k & 1) + 1];
        p[k] = F8 ? pack_f16x2(a, b) : ptx::pack_bf16x2(a, b);
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      // keys k, k + 1 and k + 8, k + 9 (k = 2c); dims 2w, 2w + 1 of 8
      const uint8_t* vt = stage + C::kTileBytes;
      const int k = 2 * cc;
      if (F8) {
        uint2 x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          x[q] = *reinterpret_cast<const uint2*>(vt + place(k + (q & 1) + 8 * (q >> 1), 4 * i + (n >> 1)) + (n & 1) * 8);
#pragma unroll
        for (int w = 0; w < 4; ++w) {               // the codes of two keys side by side, then to f16
          const uint32_t a0 = w < 2 ? x[0].x : x[0].y, a1 = w < 2 ? x[1].x : x[1].y;
          const uint32_t a2 = w < 2 ? x[2].x : x[2].y, a3 = w < 2 ? x[3].x : x[3].y;
          uint32_t b0, b1, b2, b3;
          e4m3x4_to_f16x4(__byte_perm(a0, a1, (w & 1) ? 0x7362 : 0x5140), b0, b1);
          e4m3x4_to_f16x4(__byte_perm(a2, a3, (w & 1) ? 0x7362 : 0x5140), b2, b3);
          mma<F8>(o[8 * i + 2 * w], p, b0, b2);
          mma<F8>(o[8 * i + 2 * w + 1], p, b1, b3);
        }
      } else {
        uint32_t v[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 x = *reinterpret_cast<const uint4*>(vt + place(k + (q & 1) + 8 * (q >> 1), 8 * i + n));
          v[q][0] = x.x, v[q][1] = x.y, v[q][2] = x.z, v[q][3] = x.w;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          mma<F8>(o[8 * i + 2 * w], p, __byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x5410));
          mma<F8>(o[8 * i + 2 * w + 1], p, __byte_perm(v[0][w], v[1][w], 0x7632), __byte_perm(v[2][w], v[3][w], 0x7632));
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();                                  // (the join is staged over the rings)

  // ---- join of the groups -------------------------------------------------------
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int row = n + 8 * r;
    if (F8) {
      // (in two steps: with value scales below 2^-119 the whole factor is less than the least normal number, and ex2 gives 0)
      const float f = m[r] == -INFINITY ? 1.f : ex2(0.5f * (mv[r] - kUp - m[r]));
#pragma unroll
      for (int j = 0; j < NI * 8; ++j) {
        o[j][2 * r] = o[j][2 * r] * f * f;
        o[j][2 * r + 1] = o[j][2 * r + 1] * f * f;
      }
    }
    // a NaN sum counts with every weight, a sum of 0 (nothing seen) with none
    if (cc == 0 && half == 0) ML[grp * kRows + row] = make_float2(l[r] != l[r] ? INFINITY : l[r] == 0.f ? -INFINITY : m[r], l[r]);
    if (row < u.nrows) {
      float* dst = Os + (grp * kRows + row) * LO + d0 + 16 * cc;
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
  // Rows r, 64 dims a warp: the groups' parts, in order, into the first one's place.
  constexpr int ND = D / 64, NW = G * HV;
  for (int p = warp; p < u.nrows * ND; p += NW) {
    const int r = p / ND, d = 64 * (p - r * ND) + 2 * lane;
    float2 ml[G], x[G];
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) {
      ml[k] = ML[k * kRows + r];
      x[k] = *reinterpret_cast<const float2*>(Os + (k * kRows + r) * LO + d);
      top = fmaxf(top, ml[k].x);
    }
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < G; ++k) {
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
      *reinterpret_cast<uint32_t*>(out_bf16(c, u.b, t, h, d)) =
          ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
      if (d == 0 && c.lse)
        c.lse[((long long)u.b * c.Tq + t) * c.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
  }
  if (c.plan.ns) ptx::pdl_wait();                   // the prefix's grid: combine_kernel waits for this one alone
  if (ranks == 1) return;
  // The CTAs of the cluster, in order, by distributed shared memory.
  ptx::cluster_sync();
  const int rank = (int)ptx::cluster_ctarank();
  const uint32_t os_a = ptx::smem_u32(Os), j_a = ptx::smem_u32(Joined);
  for (int p = rank * NW + warp; p < u.nrows * ND; p += ranks * NW) {
    const int r = p / ND, d = 64 * (p - r * ND) + 2 * lane;
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
    *reinterpret_cast<uint32_t*>(out_bf16(c, u.b, t, h, d)) =
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
  cfg.blockDim = dim3(Cfg<D, F8>::kThreads);
  cfg.dynamicSmemBytes = Cfg<D, F8>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c.plan.cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  // Beside the prefix's grid, which it does not need: that one's CTAs are all
  // running, and all that came before it has ended, when this one may start.
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = c.plan.ns ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, F8>, c, c.plan.cluster);
}

template <int D, bool F8>
cudaError_t configure() {
  return cudaFuncSetAttribute(attn_decode_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, F8>::kSmem);
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
