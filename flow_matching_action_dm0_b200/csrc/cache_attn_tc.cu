// bf16 attention over key/value caches on the tensor cores: one kernel for
// cross attention, for a prefix shared by a batch and for each element's own
// keys, bf16 or E4M3.
//
// A CTA takes 128 rows (query token x head of a KV head's group) against a
// range of 128-key tiles, in one pass:
//   S = Q K^T    tcgen05, 128 x 128, K chunks of 64 dims from a ring of 16 KB
//                stages filled by TMA                             -> TMEM
//   P = 2^(S - m) a thread per row, straight from TMEM; the row's sum is kept
//                in fp32, P rounded to bf16 (the MMA's input type) and
//                written over S in TMEM
//   O += P V     tcgen05 with P as the TMEM operand and V row-major (keys x
//                dims) as an MN-major operand, so V is never transposed
// m is the running maximum, raised (and O rescaled) only when a row's maximum
// has grown by more than 8 in base 2: weights stay below 2^8, and the result
// is the same quotient.  Roles: warp 0 issues the loads, warp 1 the MMAs,
// warps 4-7 the softmax (and the output); with an E4M3 source warps 8-11 widen
// codes to bf16 stages (exactly), and the scales multiply S and P in fp32.
#include <cuda.h>

#include <algorithm>

#include "cache_ops.h"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace rtv {

namespace {

constexpr int kStage = 16384;                    // a bf16 stage: 128 rows of 128 bytes
constexpr int kRaw = 8192;                       // the E4M3 codes of a stage: 128 rows of 64 bytes
constexpr int kTile = 128;                       // rows of a unit, keys of a tile
constexpr float kLazy = 8.f;                     // growth of a maximum (base 2) that rescales O
constexpr long long kDrainNs = 200000000LL;      // limit of the waits for what is in flight after a timeout

// Tensor maps of the two sources' keys and values, and whether a source's
// batch and head index move at all (0: one row set serves every index).
struct __align__(64) AttnMaps {
  CUtensorMap pre_k, pre_v, own_k, own_v;
  int pre_h, own_b, own_h;
};

template <int D, bool F8>
struct Cfg {
  static constexpr int NC = D / 64;                       // stages of a K or V tile
  static constexpr int VK = 8192 / D;                     // keys of a V stage
  static constexpr bool kTwo = D <= 128 && !F8;           // two CTAs share an SM
  static constexpr int TCOLS = kTwo ? 256 : 512;          // tensor memory columns of the CTA
  static constexpr int NSB = kTwo ? 1 : 2;                // S buffers
  static constexpr int QB = kTile * D * 2;
  static constexpr int NST = kTwo ? (D == 64 ? 5 : 4) : F8 ? 6 : 10;
  static constexpr int NRAW = F8 ? 6 : 0;
  static constexpr int kThreads = F8 ? 384 : 256;
  static constexpr bool kHold = !F8 && !kTwo;             // a thread has the registers for a row of S
  static constexpr int kOff = QB + NST * kStage + NRAW * kRaw;   // barriers behind the tiles
  static constexpr int kSmem = 1024 + kOff + 512 + (F8 ? 2 * 2 * kTile * 4 : 0);
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int t, int h, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(map), "r"(x), "r"(t), "r"(h), "r"(b), "r"(ptx::smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], bf16 inputs, fp32 accumulator.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}

// Descriptor of an MN-major operand with the 128-byte swizzle: rows (K index)
// of 64 elements, 8-row atoms of 1024 bytes; the next 64 elements of the MN
// index are `mn_bytes` further.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t mn_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(mn_bytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kBTransposed = 1u << 16;      // instruction descriptor: B is MN-major

#define R8(o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define W8(o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])
#define I8(o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
// 32 lanes x 32 columns; the registers hold the data after tmem_wait_ld on them.
__device__ __forceinline__ void tmem_ld_32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : R8(0), R8(8), R8(16), R8(24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : W8(0), W8(8), W8(16), W8(24)::"memory");
}
__device__ __forceinline__ void tmem_st_32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      I8(0), I8(8), I8(16), I8(24)
      : "memory");
}
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      I8(0), I8(8)
      : "memory");
}
#undef R8
#undef W8
#undef I8
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Two E4M3 codes (low byte first) to two bf16 values, exactly (both fit in f16 and bf16).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  uint32_t h2;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "r"(two));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  return ptx::pack_bf16x2(f.x, f.y);
}

// What every role derives from the unit: the order of the tiles' loads, which
// is that of the MMAs: with two S buffers K(0), K(1), V(0), K(2), V(1), ...,
// with one K(0), V(0), K(1), V(1), ...
template <int NSB>
struct Order {
  int n;                                          // tiles
  __device__ int count() const { return 2 * n; }
  // i-th load: tile * 2 + (1: values)
  __device__ int at(int i) const {
    if (NSB == 1) return i;
    if (i == 0) return 0;
    if (i == 2 * n - 1) return 2 * (n - 1) + 1;
    return (i & 1) ? 2 * ((i + 1) >> 1) : 2 * ((i >> 1) - 1) + 1;
  }
  // loads before V(j)
  __device__ int before_v(int j) const { return NSB == 1 ? 2 * j + 1 : min(j + 2, n) + j; }
};

struct TileAt {
  bool pre;
  int k0, nk;                                     // first key, keys of the tile
};
__device__ __forceinline__ TileAt tile_at(const AttnUnit& u, int t) {
  TileAt a;
  a.pre = t < u.n0;
  a.k0 = (a.pre ? t : t - u.n0) * kTile;
  a.nk = min(kTile, (a.pre ? u.len0 : u.len1) - a.k0);
  return a;
}

// The tile may hold hidden keys: its end, or a mask.
__device__ __forceinline__ bool has_hidden(const AttnCall& c, const TileAt& t) {
  return t.nk < kTile || (t.pre ? c.pre.mask : c.own.mask) != nullptr;
}

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::kThreads, Cfg<D, F8>::kTwo ? 2 : 1)
    attn_cache_kernel(const __grid_constant__ AttnCall c, const __grid_constant__ AttnMaps maps) {
  using C = Cfg<D, F8>;
  constexpr int NC = C::NC, NSB = C::NSB, NST = C::NST, VK = C::VK;
  constexpr int NRAW = F8 ? C::NRAW : 1;
  extern __shared__ uint8_t sm_raw[];
  __shared__ int s_abort;
  uint8_t* Qs = (uint8_t*)(((uintptr_t)sm_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = Qs + C::QB;
  uint8_t* raw = ring + NST * kStage;
  uint64_t* bars = (uint64_t*)(Qs + C::kOff);
  uint64_t* ready = bars;                         // [NST] stage holds its operand
  uint64_t* empty = ready + NST;                  // [NST] its MMAs have completed
  uint64_t* s_full = empty + NST;                 // [2] S of a buffer is complete
  uint64_t* p_ready = s_full + 2;                 // [2] P of a buffer is written (and hidden values are zeroed)
  uint64_t* pv_done = p_ready + 2;                // O += P V has completed
  uint64_t* q_ready = pv_done + 1;
  uint64_t* o_done = q_ready + 1;                 // every MMA of the CTA has completed
  uint64_t* v_landed = o_done + 1;                // values of a tile with hidden keys are in their stages
  uint64_t* raw_full = v_landed + 1;              // [NRAW]
  uint64_t* raw_empty = raw_full + NRAW;          // [NRAW]
  uint32_t* tslot = (uint32_t*)(raw_empty + NRAW);
  uint32_t* seen = tslot + 2;                     // [2][4] visible keys of a tile, 32 to a word
  float* scales = (float*)(bars + 64);            // [2][K, V][128] of a tile (E4M3)
  static_assert((2 * NST + 8 + 2 * NRAW) * 8 + 8 + 32 <= 512, "barriers fit their space");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttnUnit u = attn_unit(c);
  const int n = u.t1 - u.t0;
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < NST; ++i) {
      ptx::mbar_init(&ready[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s_full[i], 1);
      ptx::mbar_init(&p_ready[i], 128);
    }
    ptx::mbar_init(pv_done, 1);
    ptx::mbar_init(q_ready, C::kThreads - 64);
    ptx::mbar_init(o_done, 1);
    ptx::mbar_init(v_landed, 1);
    if (F8)
      for (int i = 0; i < NRAW; ++i) {
        ptx::mbar_init(&raw_full[i], 1);
        ptx::mbar_init(&raw_empty[i], 1);
      }
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tslot, C::TCOLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t o_tmem = tmem + NSB * kTile;     // S buffers first, then O
  const long long limit = c.timeout_ns;
  const Order<NSB> order{n};
  // After a wait has run out every other one gives up at once, so that all
  // warps reach the end (and the barriers among them) without their data.
  auto wait = [&](uint64_t* bar, int parity) {
    if (*(volatile int*)&s_abort) return false;
    if (ptx::mbar_wait(bar, (uint32_t)parity & 1u, limit)) return true;
    atomicOr(c.status, RTV_DEV_TIMEOUT);
    atomicOr(&s_abort, 1);
    return false;
  };

  if (warp == 0) {
    // ---- loads -------------------------------------------------------------
    if (lane == 0) {
      int st = 0, rw = 0;                         // stages and raw stages filled so far
      bool ok = true;
      for (int i = 0; i < order.count() && ok; ++i) {
        const int o = order.at(i);
        const bool val = o & 1;
        const TileAt t = tile_at(u, u.t0 + (o >> 1));
        const CUtensorMap* map = t.pre ? (val ? &maps.pre_v : &maps.pre_k) : (val ? &maps.own_v : &maps.own_k);
        const int h = t.pre ? u.kvh * maps.pre_h : u.kvh * maps.own_h, b = t.pre ? 0 : u.b * maps.own_b;
        const bool codes = F8 && (t.pre ? c.pre_f8 : c.own_f8);
        for (int cc = 0; cc < NC && ok; ++cc, ++st) {
          uint8_t* dst;
          uint64_t* bar;
          int row;                                // bytes of a row
          if (codes) {
            const int r = rw % NRAW;
            if (!(ok = wait(&raw_empty[r], rw / NRAW + 1))) break;
            dst = raw + r * kRaw;
            bar = &raw_full[r];
            row = 64;
            ++rw;
          } else {
            // (behind codes: the converters wait for these stages in their own
            // time, and a parity tells a phase only from its neighbours)
            if (F8 && rw > 0 && !(ok = wait(&raw_empty[(rw - 1) % NRAW], (rw - 1) / NRAW))) break;
            const int s = st % NST;
            if (!(ok = wait(&empty[s], st / NST + 1))) break;
            dst = ring + s * kStage;
            bar = &ready[s];
            row = 128;
          }
          ptx::mbar_expect_tx(bar, 128u * row);
          if (!val) tma_load_4d(dst, map, 64 * cc, t.k0, h, b, bar);
          else
#pragma unroll
            for (int dc = 0; dc < NC; ++dc) tma_load_4d(dst + dc * VK * row, map, 64 * dc, t.k0 + cc * VK, h, b, bar);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMAs --------------------------------------------------------------
    if (lane == 0 && n > 0) {
      const uint32_t id_s = ptx::idesc_bf16_f32(128, kTile), id_o = ptx::idesc_bf16_f32(128, D) | kBTransposed;
      const uint32_t qa = ptx::smem_u32(Qs), ra = ptx::smem_u32(ring);
      int st = 0;
      bool ok = wait(q_ready, 0);
      for (int i = 0; i < order.count() && ok; ++i) {
        const int o = order.at(i), j = o >> 1, buf = NSB == 1 ? 0 : j & 1;
        const uint32_t s_tmem = tmem + buf * kTile;
        if (!(o & 1)) {
          // S(j) overwrites P(j - NSB)
          if (j >= NSB && !(ok = wait(pv_done, j - NSB))) break;
          for (int cc = 0; cc < NC && ok; ++cc, ++st) {
            const int s = st % NST;
            if (!(ok = wait(&ready[s], st / NST))) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              ptx::umma_bf16(s_tmem, ptx::sw128_kmajor_desc(qa + cc * 16384 + kk * 32),
                             ptx::sw128_kmajor_desc(ra + s * kStage + kk * 32), id_s, (cc | kk) != 0);
            ptx::umma_commit(&empty[s]);
          }
          if (ok) ptx::umma_commit(&s_full[buf]);
        } else {
          if (has_hidden(c, tile_at(u, u.t0 + j))) {
            for (int cc = 0; cc < NC && ok; ++cc) ok = wait(&ready[(st + cc) % NST], (st + cc) / NST);
            if (!ok) break;
            ptx::mbar_arrive(v_landed);
          }
          if (!(ok = wait(&p_ready[buf], j / NSB))) break;
          for (int cc = 0; cc < NC && ok; ++cc, ++st) {
            const int s = st % NST;
            if (!(ok = wait(&ready[s], st / NST))) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < VK / 16; ++kk)
              umma_bf16_ts(o_tmem, s_tmem + (cc * VK + kk * 16) / 2,
                           sw128_mnmajor_desc(ra + s * kStage + kk * 2048, VK * 128), id_o, (j | cc | kk) != 0);
            ptx::umma_commit(&empty[s]);
          }
          if (ok) ptx::umma_commit(pv_done);
        }
      }
      // every MMA completes before the tensor memory is read for the last time and freed
      ptx::umma_commit(o_done);
      if (!ptx::mbar_wait(o_done, 0, kDrainNs)) atomicOr(c.status, RTV_DEV_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ---- Q rows, 16 bytes a lane, in the K-major swizzled layout ------------
    {
      constexpr int CPR = D / 8;                  // 16-byte chunks of a row
      const uint32_t flip = c.scale_log2 < 0.f ? 0x80008000u : 0u;   // a negative scale becomes -q and its magnitude
      for (int i = tid - 64; i < kTile * CPR; i += C::kThreads - 64) {
        const int r = i / CPR, ch = i - r * CPR;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < u.nrows) {
          const long long row = u.row0 + r;
          const int b = (int)(row / c.plan.rows_b), rr = (int)(row - (long long)b * c.plan.rows_b);
          const int t = rr / c.group, g = rr - t * c.group;
          v = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(c.q) + b * c.qb + t * c.qt +
                                              (long long)(u.kvh * c.group + g) * c.qh + ch * 8);
          v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
        }
        *reinterpret_cast<uint4*>(Qs + (ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(q_ready);
    }
    if (warp >= 8) {
      // ---- E4M3 codes to bf16 stages ---------------------------------------
      if (F8) {
        const int ct = tid - 256;
        int st = 0, rw = 0;
        for (int i = 0; i < order.count(); ++i) {
          const TileAt t = tile_at(u, u.t0 + (order.at(i) >> 1));
          if (!(t.pre ? c.pre_f8 : c.own_f8)) {
            st += NC;
            continue;
          }
          for (int cc = 0; cc < NC; ++cc, ++st, ++rw) {
            const int s = st % NST, r = rw % NRAW;
            wait(&raw_full[r], rw / NRAW);
            wait(&empty[s], st / NST + 1);
            const uint8_t* src = raw + r * kRaw;
            uint8_t* dst = ring + s * kStage;
            uint4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4*>(src + (q * 128 + ct) * 16);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int id = q * 128 + ct, row = id >> 2, c16 = id & 3;
              const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint4 o;
                o.x = e4m3x2_to_bf16x2(w[2 * h] & 0xFFFFu);
                o.y = e4m3x2_to_bf16x2(w[2 * h] >> 16);
                o.z = e4m3x2_to_bf16x2(w[2 * h + 1] & 0xFFFFu);
                o.w = e4m3x2_to_bf16x2(w[2 * h + 1] >> 16);
                *reinterpret_cast<uint4*>(dst + row * 128 + (((2 * c16 + h) ^ (row & 7)) << 4)) = o;
              }
            }
            ptx::fence_proxy_async_smem();
            named_sync(2, 128);
            if (ct == 0) {
              ptx::mbar_arrive(&ready[s]);
              ptx::mbar_arrive(&raw_empty[r]);
            }
          }
        }
      }
    } else if (warp >= 4) {
      // ---- softmax: a row a thread --------------------------------------------
      const int r = tid - 128;                    // row, and key whose visibility this thread looks up
      const uint32_t lanes = (uint32_t)(32 * (warp - 4)) << 16;
      const float scale = fabsf(c.scale_log2);
      const bool live = 32 * (warp - 4) < u.nrows;   // the warp has rows
      float m = -INFINITY, l = 0.f;
      int partial = 0;                            // tiles with hidden keys so far
      // the scales of the next tile's key r are fetched a tile ahead
      float ks = 0.f, vs = 0.f;
      auto fetch = [&](int t) {
        if (!F8 || t >= u.t1) return;
        const TileAt a = tile_at(u, t);
        ks = vs = 1.f;
        if (!(a.pre ? c.pre_f8 : c.own_f8) || r >= a.nk) return;
        const KvSource& s = a.pre ? c.pre : c.own;
        const long long off = (a.pre ? 0 : u.b) * s.fb + (long long)(a.k0 + r) * s.ft + u.kvh * s.fh;
        ks = s.ks[off];
        vs = s.vs[off];
      };
      fetch(u.t0);
      for (int j = 0; j < n; ++j) {
        const int buf = NSB == 1 ? 0 : j & 1;
        const TileAt t = tile_at(u, u.t0 + j);
        const KvSource& src = t.pre ? c.pre : c.own;
        const bool whole = !has_hidden(c, t);
        if (!whole || F8) {
          bool mine = true;
          if (!whole) {
            mine = r < t.nk && (!src.mask || src.mask[(t.pre ? 0 : u.b) * src.mask_sb + t.k0 + r]);
            const uint32_t word = __ballot_sync(0xffffffffu, mine);
            if (lane == 0) seen[(j & 1) * 4 + warp - 4] = word;
          }
          if (F8) {
            scales[(j & 1) * 256 + r] = mine ? ks : 1.f;
            scales[(j & 1) * 256 + 128 + r] = mine ? vs : 0.f;
            fetch(u.t0 + j + 1);
          }
          named_sync(1, 128);
        }
        wait(&s_full[buf], j / NSB);
        ptx::tc_fence_after();
        const uint32_t s_tmem = tmem + buf * kTile + lanes;
        const float* sc = scales + (j & 1) * 256;
        if (!whole && live) {
          // scores of hidden keys become -inf, so that nothing below looks at the mask
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            const uint32_t vis = seen[(j & 1) * 4 + cc];
            uint32_t y[32];
            tmem_ld_32_async(s_tmem + 32 * cc, y);
            tmem_wait_ld(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = (vis >> e) & 1u ? y[e] : 0xFF800000u;
            tmem_st_32(s_tmem + 32 * cc, y);
          }
          tmem_wait_st();
        }
        if (live) {
          // With registers to spare the whole row is held; otherwise it is read
          // twice from tensor memory, 32 columns at a time.
          float top = -INFINITY;
          uint32_t x[C::kHold ? 4 : 1][32];
          auto load = [&](int cc) {
            tmem_ld_32_async(s_tmem + 32 * cc, x[C::kHold ? cc : 0]);
            if (!C::kHold) tmem_wait_ld(x[0]);
          };
          if (C::kHold) {
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) load(cc);
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) tmem_wait_ld(x[C::kHold ? cc : 0]);
          }
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            if (!C::kHold) load(cc);
            uint32_t(&xc)[32] = x[C::kHold ? cc : 0];
            float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float y = __uint_as_float(xc[e]);
              if (F8) y *= sc[32 * cc + e];
              t4[e & 3] = fmaxf(t4[e & 3], y);
            }
            top = fmaxf(top, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])));
          }
          const float mn = fmaxf(m, top == -INFINITY ? -INFINITY : top * scale);
          if (j == 0) {
            m = mn;
          } else if (__any_sync(0xffffffffu, mn - m > kLazy)) {
            wait(pv_done, j - 1);
            ptx::tc_fence_after();
            const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
            m = mn;
            l *= f;
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t y[32];
              tmem_ld_32_async(o_tmem + lanes + 32 * cc, y);
              tmem_wait_ld(y);
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
              tmem_st_32(o_tmem + lanes + 32 * cc, y);
            }
            tmem_wait_st();
          }
          const float base = m == -INFINITY ? 0.f : m;
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            if (!C::kHold) load(cc);
            uint32_t(&xc)[32] = x[C::kHold ? cc : 0];
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float p[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float y = __uint_as_float(xc[e + k]);
                if (F8) y *= sc[32 * cc + e + k];
                p[k] = ex2(fmaf(y, scale, -base));
                l4[(e + k) & 3] += p[k];
                if (F8) p[k] *= sc[128 + 32 * cc + e + k];
              }
              w[e / 2] = ptx::pack_bf16x2(p[0], p[1]);
            }
            tmem_st_16(s_tmem + 16 * cc, w);   // over S columns that have been read
          }
          l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
        }
        if (!whole) {
          // hidden values become zeros: their weight is 0, and 0 times anything stored there must be 0
          wait(v_landed, partial++);
          if (!((seen[(j & 1) * 4 + warp - 4] >> lane) & 1u)) {
            uint8_t* dst = ring + ((order.before_v(j) * NC + r / VK) % NST) * kStage + (r % VK) * 128;
#pragma unroll 1
            for (int q = 0; q < NC * 8; ++q)
              *reinterpret_cast<uint4*>(dst + (q >> 3) * VK * 128 + (q & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            ptx::fence_proxy_async_smem();
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&p_ready[buf]);
      }
      // ---- output --------------------------------------------------------------
      if (n > 0) wait(o_done, 0);
      ptx::tc_fence_after();
      const bool split = c.plan.n_slots > 1;
      const bool mine = r < u.nrows;
      const long long row = u.row0 + (mine ? r : 0);
      const int b = (int)(row / c.plan.rows_b), rr = (int)(row - (long long)b * c.plan.rows_b);
      const int t = rr / c.group, h = u.kvh * c.group + rr - t * c.group;
      const long long pr = part_row(c, u, row);
      if (mine && split) {
        // a NaN sum counts with every weight, a sum of 0 (nothing seen) with none
        const float mo = l != l ? INFINITY : l == 0.f ? -INFINITY : m;
        *reinterpret_cast<float2*>(c.part_ml + pr * 2) = make_float2(mo, l);
      }
      if (mine && !split && c.lse)
        c.lse[((long long)b * c.Tq + t) * c.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      const float inv = split ? 1.f : l == 0.f ? 0.f : 1.f / l;
      if (live) {
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(c.out) + b * c.ob + t * c.ot + h * c.oh;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t x[32];
          if (n > 0) {
            tmem_ld_32_async(o_tmem + lanes + 32 * cc, x);
            tmem_wait_ld(x);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = 0u;
          }
          if (!mine) continue;
          if (split) {
            if (l == 0.f) continue;               // the join does not read an empty part
            float4* dst = reinterpret_cast<float4*>(c.part_o + pr * D + 32 * cc);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]), __uint_as_float(x[4 * e + 2]),
                                   __uint_as_float(x[4 * e + 3]));
          } else {
            uint4* dst = reinterpret_cast<uint4*>(out + 32 * cc);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = ptx::pack_bf16x2(__uint_as_float(x[8 * e + 2 * k]) * inv, __uint_as_float(x[8 * e + 2 * k + 1]) * inv);
              dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (s_abort) {   // after a timeout loads may be in flight: give them time to land before the CTA's memory is reused
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 2000000ull) {
    }
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TCOLS);
  }
}

// ---- host --------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return (EncodeFn) nullptr;
    }
    return (EncodeFn)p;
  }();
  return fn;
}

// Map of one tensor [batch][token][head][D] with boxes of 64 dims x `keys` tokens.
bool encode(CUtensorMap* m, const void* base, bool f8, int D, int keys, int len, int heads, long long st, long long sh,
            int batch, long long sb) {
  const long long eb = f8 ? 1 : 2, dense = (long long)D * eb;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)len, (cuuint64_t)heads, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {(cuuint64_t)(len > 1 ? st * eb : dense), (cuuint64_t)(heads > 1 ? sh * eb : dense),
                                 (cuuint64_t)(batch > 1 ? sb * eb : dense)};
  const cuuint32_t box[4] = {64, (cuuint32_t)keys, 1, 1}, one[4] = {1, 1, 1, 1};
  return encode_fn()(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
                     dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F8>
cudaError_t launch_tc(const AttnCall& c, cudaStream_t st) {
  using C = Cfg<D, F8>;
  AttnMaps m{};
  bool ok = true;
  auto source = [&](const KvSource& s, int f8, int batch, CUtensorMap* k, CUtensorMap* v, int* hm, int* bm) {
    if (s.len == 0) return;
    *hm = c.Hkv > 1 && s.sh == 0 ? 0 : 1;
    *bm = batch > 1 && s.sb == 0 ? 0 : 1;
    const int heads = *hm ? c.Hkv : 1, nb = *bm ? batch : 1;
    ok = ok && encode(k, s.k, f8, D, kTile, s.len, heads, s.st, s.sh, nb, s.sb) &&
         encode(v, s.v, f8, D, C::VK, s.len, heads, s.st, s.sh, nb, s.sb);
  };
  int pre_b = 0;
  source(c.pre, c.pre_f8, 1, &m.pre_k, &m.pre_v, &m.pre_h, &pre_b);
  source(c.own, c.own_f8, c.B, &m.own_k, &m.own_v, &m.own_h, &m.own_b);
  if (!ok) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((long long)c.plan.tiles_s * c.plan.ns + (long long)c.B * c.plan.tiles_e * c.plan.ne), c.Hkv);
  attn_cache_kernel<D, F8><<<grid, C::kThreads, C::kSmem, st>>>(c, m);
  return cudaGetLastError();
}

template <int D, bool F8>
cudaError_t configure() {
  return cudaFuncSetAttribute(attn_cache_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, F8>::kSmem);
}

}  // namespace

cudaError_t configure_attention_tc() {
  if (!encode_fn()) return cudaErrorNotSupported;
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

int attention_tc_ctas_per_sm(int D, bool f8) { return D <= 128 && !f8 ? 2 : 1; }

cudaError_t launch_attention_tc(const AttnCall& c, cudaStream_t st) {
  const bool f8 = (c.pre.len && c.pre_f8) || (c.own.len && c.own_f8);
  if (f8)
    return c.D == 64 ? launch_tc<64, true>(c, st) : c.D == 128 ? launch_tc<128, true>(c, st) : launch_tc<256, true>(c, st);
  return c.D == 64 ? launch_tc<64, false>(c, st) : c.D == 128 ? launch_tc<128, false>(c, st) : launch_tc<256, false>(c, st);
}

}  // namespace rtv
