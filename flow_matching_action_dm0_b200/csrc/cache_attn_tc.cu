// bf16 attention over key/value caches on the tensor cores: one kernel for
// cross attention, for a prefix shared by a batch and for each element's own
// keys.
//
// A CTA takes up to 256 rows (query token x head of a KV head's group; 128 at
// head_dim 256) against a range of key tiles, in one pass over them:
//   S = Q K^T    tcgen05, 128 rows x 128 keys (64 at head_dim 256), K from a
//                ring of 16 KB stages filled by TMA                 -> TMEM
//   P = 2^(S - m) a thread per row, straight from TMEM; the row's sum is kept
//                in fp32, P rounded to bf16 (the MMA's input type: at most
//                2^-8 of each weight, as much as the output's own rounding;
//                relative L2 against fp64 0.0023, where fp32 weights have
//                0.0017) and written over S in TMEM
//   O += P V     tcgen05 with P as the TMEM operand and V row-major (keys x
//                dims) as an MN-major operand, so V is never transposed
// m is the running maximum, raised (and O rescaled) only when a row's maximum
// has grown by more than 8 in base 2: weights stay below 2^8, and the result
// is the same quotient.
//
// Work goes in steps q that alternate between two S buffers and two softmax
// groups of four warps: with more than 128 rows, step q is row tile q & 1
// against key tile q >> 1 (both row tiles read a key tile's stages once);
// with fewer, key tile q for the one row tile, the groups handing its maximum
// on.  The MMA warp issues S(q + 1) before PV(q), so that the tensor cores
// have work while a group exponentiates.  Warp 0 issues the loads, warp 1 the
// MMAs, warps 4-11 are the groups.
//
// At head_dim 256 O takes half of the tensor memory.  Key tiles of 64 leave
// room there for Q too, so that the ring has 14 stages instead of 10: three
// and a half tiles of keys and values.  (A 64-key step takes 1.6-1.7 thousand
// cycles, 1.1 thousand of them the tensor cores'; with 128-key tiles and Q in
// shared memory two such steps' worth took 4.3 thousand.)
//
// Few units are split over key ranges.  Up to eight ranges of a unit form a
// cluster, stage their rows in shared memory and join them there, each CTA a
// share of the rows; more are joined by combine_kernel.
//
// What it reaches, and what bounds it (B200, cold L2): 2050 queries x 4001
// keys x 4 elements at head_dim 128, 305-312 us, 870 TFLOP/s of the 1657 a
// matrix product reaches: a step's chain S -> softmax -> P V, of which the
// exponentials and their conversion are the longest part, fills the time of
// two steps' products, and 528 CTAs on 148 SMs leave the last of four waves
// 43% empty.  16 suffixes of 51 tokens x 8 heads at head_dim 256 over 816 keys: 20.5
// us, launch 2.5, Q and the first tiles 3, tiles 6, join 5.
#include <cuda.h>

#include <algorithm>

#include "cache_ops.h"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace rtv {

namespace {

constexpr int kStage = 16384;                    // a bf16 stage: 128 rows of 128 bytes
constexpr int kTile = 128;                       // rows of a row tile
constexpr float kLazy = 8.f;                     // growth of a maximum (base 2) that rescales O
constexpr int kFirst = 2;                        // loads of the ring that go before Q has been read
constexpr long long kDrainNs = 200000000LL;      // limit of the waits for what is in flight after a timeout

// Tensor maps of the two sources' keys and values, and whether a source's
// batch and head index move at all (0: one row set serves every index).
struct __align__(64) AttnMaps {
  CUtensorMap pre_k, pre_v, own_k, own_v;
  int pre_h, own_b, own_h;
};

template <int D>
struct Cfg {
  static constexpr int DC = D / 64;                       // chunks of 64 dims
  static constexpr int KT = attention_tc_keys(D);         // keys of a tile
  static constexpr int CK = kStage / (KT * 128);          // chunks of a K stage
  static constexpr int VK = 8192 / D;                     // keys of a V stage
  static constexpr int NC = DC / CK;                      // stages of a K or V tile
  static_assert(NC * VK == KT, "as many V stages");
  static constexpr int MT = D == 256 ? 1 : 2;             // row tiles that fit the tensor memory
  static constexpr bool kQInTmem = D == 256;              // Q's place: tensor memory, or shared memory
  static constexpr int QB = kQInTmem ? 0 : kTile * D * 2; // bytes of a Q tile in shared memory
  static constexpr int NST = kQInTmem ? 14 : 10;
  static constexpr int kO = 2 * KT, kQ = kO + D;          // tensor memory: two S buffers, O (128 columns a row tile of two), Q
  static_assert(!kQInTmem || kQ + D / 2 <= 512, "tensor memory");
  static constexpr int kThreads = 384;
  static constexpr int kSoft = 4;                         // first softmax warp
  // Registers of a softmax thread (it holds a row of S) and of the others:
  // together what the CTA was launched with.
  static constexpr int kLaunchRegs = 168, kSoftRegs = 208, kOtherRegs = 88;
  static_assert(256 * kSoftRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs, "register shares");
  static constexpr int kOff = MT * QB + NST * kStage;     // barriers behind the tiles
  static constexpr int kSmall = 512 + 512 + 64;           // barriers, maxima, visible keys
  static constexpr int kSmem = 1024 + kOff + kSmall;
  static constexpr int kRowBytes = D * 4 + 16;            // a staged output row
  static constexpr int kStaged = MT * kTile * kRowBytes;  // and behind them, for a cluster's join, maxima and sums
  static_assert(kStaged + MT * kTile * 8 <= kOff, "output rows are staged where the tiles were");
  static_assert(3 * NC <= NST, "V(j), the next K and the one behind it are held at once");
  static_assert(kSmem <= 232448 - 64, "shared memory of a CTA");
};

// A box of [64 dims, tokens from t, 64-dim chunks from ch] of head h, element b.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int t, int ch, int h, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(map), "r"(0), "r"(t), "r"(ch), "r"(h), "r"(b), "r"(ptx::smem_u32(bar))
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
__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
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
__device__ __forceinline__ void tmem_ld_16_raw(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : R8(0), R8(8)
      : "r"(taddr)
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
// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The order of a unit's loads is that of their first use: with two row tiles
// K(0), V(0), K(1), V(1), ...; with one, S runs a key tile ahead:
// K(0), K(1), V(0), K(2), V(1), ...
struct Order {
  int n;                                          // key tiles
  bool two;                                       // row tiles: two, or one
  // i-th load: key tile * 2 + (1: values)
  __device__ int at(int i) const {
    if (two) return i;
    if (i == 0) return 0;
    if (i == 2 * n - 1) return 2 * (n - 1) + 1;
    return (i & 1) ? 2 * ((i + 1) >> 1) : 2 * ((i >> 1) - 1) + 1;
  }
  __device__ int of_k(int j) const { return two ? 2 * j : j == 0 ? 0 : 2 * j - 1; }
  __device__ int of_v(int j) const { return two ? 2 * j + 1 : min(2 * j + 2, 2 * n - 1); }
};

struct TileAt {
  bool pre;
  int k0, nk;                                     // first key, keys of the tile
};
template <int KT>
__device__ __forceinline__ TileAt tile_at(const AttnUnit& u, int t) {
  TileAt a;
  a.pre = t < u.n0;
  a.k0 = (a.pre ? t : t - u.n0) * KT;
  a.nk = min(KT, (a.pre ? u.len0 : u.len1) - a.k0);
  return a;
}

// The tile may hold hidden keys: its end, or a mask.
template <int KT>
__device__ __forceinline__ bool has_hidden(const AttnCall& c, const TileAt& t) {
  return t.nk < KT || (t.pre ? c.pre.mask : c.own.mask) != nullptr;
}

// Named barriers: 1 all softmax warps, 2 and 3 a softmax group, 4.. a pair of warps of the groups.
__device__ __forceinline__ void named_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// `bytes` (a multiple of 16, both addresses 16-byte aligned) from shared to global memory.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(ptx::smem_u32(src)), "r"(bytes)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    attn_cache_kernel(const __grid_constant__ AttnCall c, const __grid_constant__ AttnMaps maps) {
  using C = Cfg<D>;
  constexpr int NC = C::NC, NST = C::NST, VK = C::VK, KT = C::KT;
  extern __shared__ uint8_t sm_raw[];
  __shared__ int s_abort, s_loads;                // a wait has run out; loads issued
  uint8_t* Qs = (uint8_t*)(((uintptr_t)sm_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = Qs + C::MT * C::QB;
  uint64_t* ready = (uint64_t*)(Qs + C::kOff);    // [NST] the stage holds its operand
  uint64_t* empty = ready + NST;                  // [NST] the stage's MMAs have completed
  uint64_t* s_full = empty + NST;                 // [2] S of a buffer is complete
  uint64_t* p_ready = s_full + 2;                 // [2] P of a buffer is written (and hidden values are zeroed)
  uint64_t* q_ready = p_ready + 2;                // [2] Q rows of a group
  uint64_t* pv_done = q_ready + 2;                // one row tile: O += P V of a step has completed
  uint64_t* o_done = pv_done + 1;                 // every MMA of the CTA has completed
  uint32_t* tslot = (uint32_t*)(o_done + 1);
  static_assert((2 * NST + 8) * 8 + 8 <= 512, "barriers fit their space");
  float* m_row = (float*)(Qs + C::kOff + 512);    // [128] the maximum that the groups hand on (one row tile)
  uint32_t* seen = (uint32_t*)(m_row + 128);      // [2 groups][4] visible keys of the group's tile

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (uniform)
  if (tid == 0) {
    s_abort = s_loads = 0;
    for (int i = 0; i < NST; ++i) {
      ptx::mbar_init(&ready[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s_full[i], 1);
      ptx::mbar_init(&p_ready[i], 4);
      ptx::mbar_init(&q_ready[i], 4);
    }
    ptx::mbar_init(pv_done, 1);
    ptx::mbar_init(o_done, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tslot, 512);
    ptx::tmem_relinquish();
  }
  const AttnUnit u = attn_unit(c);
  const int n = u.t1 - u.t0;
  const bool two = C::MT == 2 && u.nrows > kTile;
  const int steps = two ? 2 * n : n;
  const Order order{n, two};
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);
  ptx::pdl_launch_dependents();                   // (tensor memory is allocated; combine_kernel waits for this grid's end)
  const uint32_t o_tmem = tmem + C::kO;
  // After a wait has run out every other one gives up at once, so that all
  // warps reach the end (and the barriers among them) without their data.
  auto wait = [&](uint64_t* bar, int parity) {
    const uint32_t par = (uint32_t)parity & 1u;
    if (ptx::mbar_try_wait(bar, par)) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (!*(volatile int*)&s_abort) {
      if (ptx::mbar_try_wait(bar, par)) return true;
      if ((long long)(ptx::globaltimer() - t0) > c.timeout_ns) {
        atomicOr(c.status, RTV_DEV_TIMEOUT);
        atomicOr(&s_abort, 1);
      }
    }
    return false;
  };
  if (warp == 0) {
    // ---- loads ---------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (lane == 0) {
      const int pre_h = u.kvh * maps.pre_h, own_h = u.kvh * maps.own_h, own_b = u.b * maps.own_b;
      bool ok = true;
      int s = 0, ph = 1, loads = 0;
      for (int i = 0; i < 2 * n && ok; ++i) {
        if (C::kQInTmem && i == kFirst) {   // (Q passes through the ring's other stages)
          ok = wait(&q_ready[0], 0);
          ok = wait(&q_ready[1], 0) && ok;
          if (!ok) break;
        }
        const int o = order.at(i);
        const TileAt t = tile_at<KT>(u, u.t0 + (o >> 1));
        const CUtensorMap* map = (o & 1) ? (t.pre ? &maps.pre_v : &maps.own_v) : (t.pre ? &maps.pre_k : &maps.own_k);
        const int h = t.pre ? pre_h : own_h, b = t.pre ? 0 : own_b;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
          ok = ok && wait(&empty[s], ph);
          if (!ok) break;
          ptx::mbar_expect_tx(&ready[s], (uint32_t)kStage);
          // a K stage is CK chunks of 64 dims of the tile's keys, a V stage all dims of VK keys
          if (o & 1) tma_load(ring + s * kStage, map, t.k0 + cc * VK, 0, h, b, &ready[s]);
          else tma_load(ring + s * kStage, map, t.k0, cc * C::CK, h, b, &ready[s]);
          ++loads;
          if (++s == NST) s = 0, ph ^= 1;
        }
      }
      s_loads = loads;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMAs: the whole warp walks the steps, one lane issues -----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (n > 0) {
      const uint32_t id_s = ptx::idesc_bf16_f32(128, KT), id_o = ptx::idesc_bf16_f32(128, D) | kBTransposed;
      const uint64_t qd = ptx::sw128_kmajor_desc(ptx::smem_u32(Qs)), kd = ptx::sw128_kmajor_desc(ptx::smem_u32(ring));
      const uint64_t vd = sw128_mnmajor_desc(ptx::smem_u32(ring), VK * 128);
      const bool leader = elect_one();
      const uint32_t s_hi = (uint32_t)(kd >> 32), v_hi = (uint32_t)(vd >> 32), q_lo = (uint32_t)qd, k_lo = (uint32_t)kd,
                     v_lo = (uint32_t)vd;
      bool ok = true;
      // the NC stages of a load of the order, from its position
      auto landed = [&](int pos) {
        int s = (pos * NC) % NST, ph = (pos * NC) / NST;
        for (int cc = 0; cc < NC; ++cc) {
          ok = ok && wait(&ready[s], ph);
          if (++s == NST) s = 0, ++ph;
        }
      };
      auto scores = [&](int q) {                  // S(q), over P(q - 2), whose MMA comes before it in this thread's order
        const int buf = q & 1, rt = two ? buf : 0, pos = order.of_k(two ? q >> 1 : q) * NC;
        int s = pos % NST;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
          if (leader && ok) {
            const uint32_t qa = q_lo + rt * (C::QB >> 4) + cc * (16384 >> 4), ka = k_lo + s * (kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 4 * C::CK; ++kk) {
              const uint64_t kdesc = desc64(ka + (kk >> 2) * (KT * 128 >> 4) + 2 * (kk & 3), s_hi);
              if (C::kQInTmem) umma_bf16_ts(tmem + buf * KT, tmem + C::kQ + cc * 32 * C::CK + 8 * kk, kdesc, id_s, (cc | kk) != 0);
              else ptx::umma_bf16(tmem + buf * KT, desc64(qa + 2 * kk, s_hi), kdesc, id_s, (cc | kk) != 0);
            }
            if (!two || rt == 1) ptx::umma_commit(&empty[s]);   // the key tile's last use
          }
          if (++s == NST) s = 0;
        }
        if (leader && ok) {
          ptx::umma_commit(&s_full[buf]);
        }
      };
      ok = wait(&q_ready[0], 0);
      if (!two) ok = wait(&q_ready[1], 0) && ok;
      landed(order.of_k(0));
      ptx::tc_fence_after();
      scores(0);
      if (steps > 1) {
        if (two) ok = wait(&q_ready[1], 0) && ok;
        else landed(order.of_k(1));
        ptx::tc_fence_after();
        scores(1);
      }
      for (int q = 0; q < steps && ok; ++q) {
        const int buf = q & 1, rt = two ? buf : 0, j = two ? q >> 1 : q;
        const bool next = q + 2 < steps;
        if (rt == 0) {
          landed(order.of_v(j));
          if (next) landed(order.of_k(two ? j + 1 : q + 2));
        }
        ok = ok && wait(&p_ready[buf], q >> 1);
        ptx::tc_fence_after();
        const int pos = order.of_v(j) * NC;
        int s = pos % NST;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
          if (leader && ok) {
            const uint32_t va = v_lo + s * (kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < VK / 16; ++kk)
              umma_bf16_ts(o_tmem + rt * kTile, tmem + buf * KT + (cc * VK + kk * 16) / 2, desc64(va + kk * (2048 >> 4), v_hi),
                           id_o, (j | cc | kk) != 0);
            if (!two || rt == 1) ptx::umma_commit(&empty[s]);
          }
          if (++s == NST) s = 0;
        }
        if (leader && ok) {
          if (!two) ptx::umma_commit(pv_done);
        }
        if (next) scores(q + 2);
      }
      // every MMA completes before the tensor memory is read for the last time and freed
      if (leader) {
        ptx::umma_commit(o_done);
        if (!ptx::mbar_wait(o_done, 0, kDrainNs)) atomicOr(c.status, RTV_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp < C::kSoft) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
  } else {
    // ---- softmax: a row a thread ----------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    const int grp = (warp - C::kSoft) >> 2, quarter = warp & 3;
    const int r = 32 * quarter + lane;            // row of the row tile, and key whose visibility this thread looks up
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int tile_row = two ? grp * kTile : 0;
    const bool live = tile_row + 32 * quarter < u.nrows;   // the warp has rows
    const bool mine = tile_row + r < u.nrows;
    const long long row = u.row0 + (mine ? tile_row + r : 0);
    const unsigned b = (unsigned)row / (unsigned)c.plan.rows_b, rr = (unsigned)row - b * (unsigned)c.plan.rows_b;
    const unsigned t_row = rr / (unsigned)c.group, h_row = u.kvh * c.group + rr - t_row * (unsigned)c.group;
    // Q rows, negated for a negative scale
    const long long off = b * c.qb + (long long)t_row * c.qt + (long long)h_row * c.qh;
    const uint32_t flip = c.scale_log2 < 0.f ? 0x80008000u : 0u;
    if (C::kQInTmem) {   // a row a thread, half of its dims a group; whole rows are read, and turned where the ring is not yet in use
      constexpr int CPR = D / 16, RPI = 32 / CPR, LD = D + 16;   // 16-byte chunks of half a row, rows of a warp's step, bytes of one
      static_assert(kFirst * NC * kStage + 8 * 32 * LD <= NST * kStage, "the ring's rest holds Q");
      uint8_t* at = ring + kFirst * NC * kStage + (warp - C::kSoft) * 32 * LD;
      const int ch = lane % CPR;
      uint4 v[CPR];
#pragma unroll
      for (int k = 0; k < CPR; ++k) {
        const int rl = k * RPI + lane / CPR;
        const long long o = __shfl_sync(0xffffffffu, off, rl);
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (32 * quarter + rl < u.nrows)
          v[k] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(c.q) + o + grp * (D / 2) + ch * 8);
      }
#pragma unroll
      for (int k = 0; k < CPR; ++k) *reinterpret_cast<uint4*>(at + (k * RPI + lane / CPR) * LD + ch * 16) = v[k];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < CPR; ++k) v[k] = *reinterpret_cast<const uint4*>(at + lane * LD + k * 16);
#pragma unroll
      for (int k = 0; k < D / 16; k += 4) {
        const uint32_t w[16] = {v[k].x ^ flip,     v[k].y ^ flip,     v[k].z ^ flip,     v[k].w ^ flip,
                                v[k + 1].x ^ flip, v[k + 1].y ^ flip, v[k + 1].z ^ flip, v[k + 1].w ^ flip,
                                v[k + 2].x ^ flip, v[k + 2].y ^ flip, v[k + 2].z ^ flip, v[k + 2].w ^ flip,
                                v[k + 3].x ^ flip, v[k + 3].y ^ flip, v[k + 3].z ^ flip, v[k + 3].w ^ flip};
        tmem_st_16(tmem + C::kQ + grp * (D / 4) + 4 * k + lanes, w);
      }
      tmem_wait_st();
      ptx::tc_fence_before();
      ptx::fence_proxy_async_smem();
    } else {             // the warp's own 32 (with one row tile the groups take 16 each), 16 bytes a lane
      constexpr int CPR = D / 8, RPI = 32 / CPR;  // 16-byte chunks of a row, rows of a warp's step
      uint8_t* qt = Qs + (two ? grp * C::QB : 0);
      const int r0 = two ? 0 : 16 * grp, nr = two ? 32 : 16, ch = lane % CPR;
      uint4 v[32 / RPI < 16 ? 32 / RPI : 16];     // all of a group's rows at once (32 at head_dim 256 are never asked of one)
      constexpr int NB = sizeof(v) / 16;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int rl = r0 + k * RPI + lane / CPR;               // row of the warp's 32
        const long long o = __shfl_sync(0xffffffffu, off, rl & 31);
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (k * RPI < nr && tile_row + 32 * quarter + rl < u.nrows)
          v[k] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(c.q) + o + ch * 8);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int rq = 32 * quarter + r0 + k * RPI + lane / CPR;
        if (k * RPI >= nr) continue;
        v[k].x ^= flip, v[k].y ^= flip, v[k].z ^= flip, v[k].w ^= flip;
        *reinterpret_cast<uint4*>(qt + (ch >> 3) * 16384 + rq * 128 + (((ch & 7) ^ (rq & 7)) << 4)) = v[k];
      }
      ptx::fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&q_ready[grp]);
    const float scale = fabsf(c.scale_log2);
    float m = -INFINITY, l = 0.f;                 // l counts in units of 2^m
    // Whether key r of the tile of step q is seen; looked up a step ahead.
    auto sees = [&](int q) {
      if (q >= steps) return false;
      const TileAt t = tile_at<KT>(u, u.t0 + (two ? q >> 1 : q));
      const uint8_t* mask = t.pre ? c.pre.mask : c.own.mask;
      return r < t.nk && (!mask || mask[(t.pre ? 0 : u.b * c.own.mask_sb) + t.k0 + r]);
    };
    bool next_vis = sees(grp);
    for (int q = grp; q < steps; q += 2) {
      const int j = two ? q >> 1 : q;
      const TileAt t = tile_at<KT>(u, u.t0 + j);
      const bool whole = !has_hidden<KT>(c, t);
      if (!whole) {
        const uint32_t word = __ballot_sync(0xffffffffu, next_vis);
        // (the group's last look at the words of its previous step was before its P was complete)
        named_sync(2 + grp, 128);
        if (lane == 0) seen[grp * 4 + quarter] = word;
        named_sync(2 + grp, 128);
      }
      next_vis = sees(q + 2);
      wait(&s_full[grp], q >> 1);
      ptx::tc_fence_after();
      const uint32_t s_tmem = tmem + grp * KT + lanes;
      if (live) {
        uint32_t x[KT / 32][32];                  // the row of S
#pragma unroll
        for (int cc = 0; cc < KT / 32; ++cc) tmem_ld_32_async(s_tmem + 32 * cc, x[cc]);
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int cc = 0; cc < KT / 32; ++cc) {
          tmem_wait_ld(x[cc]);
          if (!whole) {
            const uint32_t vis = seen[grp * 4 + cc];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[cc][e] = (vis >> e) & 1u ? x[cc][e] : 0xFF800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) t4[e & 3] = fmaxf(t4[e & 3], __uint_as_float(x[cc][e]));
        }
        const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        float before = m;
        if (!two) {   // the other group's step comes first
          if (q > 0) named_sync(4 + 2 * quarter + grp, 64);
          before = q > 0 ? m_row[r] : -INFINITY;
        }
        const float mn = fmaxf(before, top * scale);
        float now = before;
        if (j == 0) {
          now = mn;
        } else if (__any_sync(0xffffffffu, mn - before > kLazy)) {
          now = mn;
          // O's last MMA: PV(q - 2) of two row tiles came before S(q)
          if (!two) {
            wait(pv_done, q - 1);
            ptx::tc_fence_after();
          }
          const float f = before == now ? 1.f : ex2(before - now);
          const uint32_t o_addr = o_tmem + (two ? grp * kTile : 0) + lanes;
#pragma unroll 1
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t y[16];
            tmem_ld_16_raw(o_addr + 16 * cc, y);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
            tmem_st_16(o_addr + 16 * cc, y);
          }
          tmem_wait_st();
        }
        if (!two && q + 1 < steps) {
          m_row[r] = now;
          named_arrive(4 + 2 * quarter + (grp ^ 1), 64);
        }
        if (m != now) {                            // (the groups hand maxima on, or a rescale just above)
          l *= ex2(m - now);
          m = now;
        }
        const float base = m == -INFINITY ? 0.f : m;
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 scale2 = make_float2(scale, scale), base2 = make_float2(-base, -base);
#pragma unroll
        for (int cc = 0; cc < KT / 32; ++cc) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float2 p[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              p[k] = fma2(make_float2(__uint_as_float(x[cc][e + 2 * k]), __uint_as_float(x[cc][e + 2 * k + 1])), scale2, base2);
              p[k].x = ex2(p[k].x);
              p[k].y = ex2(p[k].y);
              l2[k] = add2(l2[k], p[k]);
            }
            w[e / 2] = ptx::pack_bf16x2(p[0].x, p[0].y);
            w[e / 2 + 1] = ptx::pack_bf16x2(p[1].x, p[1].y);
          }
          tmem_st_16(s_tmem + 16 * cc, w);        // over S columns that have been read
        }
        l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        tmem_wait_st();
      }
      if (!whole && !(two && grp)) {
        // hidden values become zeros: their weight is 0, and 0 times anything stored there must be 0
        // (a stage's earlier uses had landed before S of this step, so its parity means this one)
        const int cnt = order.of_v(j) * NC;
        for (int cc = 0; cc < NC; ++cc) wait(&ready[(cnt + cc) % NST], (cnt + cc) / NST);
        const uint32_t hidden = 32 * quarter < KT ? ~seen[grp * 4 + quarter] : 0u;
        if (hidden) {                             // (the same in the warp's lanes: 8 of them write a key's 128 bytes)
#pragma unroll 1
          for (int k = lane >> 3; k < 32; k += 4) {
            if (!((hidden >> k) & 1u)) continue;
            const int key = 32 * quarter + k;
            uint8_t* dst = ring + ((cnt + key / VK) % NST) * kStage + (key % VK) * 128 + (lane & 7) * 16;
#pragma unroll
            for (int dc = 0; dc < C::DC; ++dc) *reinterpret_cast<uint4*>(dst + dc * VK * 128) = make_uint4(0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&p_ready[grp]);
    }
    // ---- output: rows staged where the tiles were, a bulk copy each -------------
    if (n > 0) wait(o_done, 0);
    ptx::tc_fence_after();
    if (!two) {   // both groups' sums, in units of the last maximum; each writes half of the columns
      float2* ml = reinterpret_cast<float2*>(Qs);
      named_sync(1, 256);
      ml[grp * 128 + r] = make_float2(m, l);
      named_sync(1, 256);
      const float2 other = ml[(grp ^ 1) * 128 + r];
      named_sync(1, 256);                         // (the rows below are staged over this)
      const float top = fmaxf(m, other.x);
      l = l * (m == top ? 1.f : ex2(m - top)) + other.y * (other.x == top ? 1.f : ex2(other.x - top));
      m = top;
    }
    const bool join = c.plan.cluster > 1, split = c.plan.n_slots > 1 || join, first = two || grp == 0;
    const long long pr = part_row(c, u, row);
    float2* ml_sm = reinterpret_cast<float2*>(Qs + C::kStaged);
    if (mine && first && split) {
      // a NaN sum counts with every weight, a sum of 0 (nothing seen) with none
      const float mo = l != l ? INFINITY : l == 0.f ? -INFINITY : m;
      *(join ? ml_sm + tile_row + r : reinterpret_cast<float2*>(c.part_ml + pr * 2)) = make_float2(mo, l);
    }
    if (mine && first && !split && c.lse)
      c.lse[((long long)b * c.Tq + t_row) * c.Hq + h_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (live) {
      const int cols = two ? D : D / 2, c0 = two ? 0 : grp * (D / 2);
      uint8_t* stage = Qs + (tile_row + r) * C::kRowBytes + c0 * (split ? 4 : 2);
#pragma unroll 1
      for (int cc = 0; cc < cols; cc += 32) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld_32_async(o_tmem + (two ? grp * kTile : 0) + lanes + c0 + cc, x);
          tmem_wait_ld(x);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0u;
        }
        if (split) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(stage + cc * 4 + e * 16) = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = ptx::pack_bf16x2(__uint_as_float(x[8 * e + 2 * k]) * inv, __uint_as_float(x[8 * e + 2 * k + 1]) * inv);
            *reinterpret_cast<uint4*>(stage + cc * 2 + e * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      ptx::fence_proxy_async_smem();
      if (mine && !join) {
        if (split) {
          if (l != 0.f) bulk_store(c.part_o + pr * D + c0, stage, cols * 4);   // (the join does not read an empty part)
        } else if (c.out_tiled_rows == 0) {
          bulk_store(out_bf16(c, b, t_row, h_row, c0), stage, cols * 2);
        } else {
          for (int d = 0; d < cols; d += 8)
            *reinterpret_cast<uint4*>(out_bf16(c, b, t_row, h_row, c0 + d)) = *reinterpret_cast<const uint4*>(stage + d * 2);
        }
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (join) {   // the ranges' parts of a row, in order: a warp takes four rows at a time, from every CTA of the cluster
      __syncwarp();
      ptx::cluster_sync();
      constexpr int V = D >= 128 ? 4 : 2, NV = D / (32 * V), R = 4;   // elements of a lane's load, loads of a lane, rows
      const int ranks = c.plan.cluster, rank = (int)ptx::cluster_ctarank();
      const uint32_t ml_a = ptx::smem_u32(ml_sm), o_a = ptx::smem_u32(Qs) + lane * V * 4;
      for (int p = (rank * 8 + warp - C::kSoft) * R; p < u.nrows; p += ranks * 8 * R) {
        // lane 8 i + k: row p + i of CTA k
        float2 part = make_float2(-INFINITY, 0.f);
        if ((lane & 7) < ranks && p + (lane >> 3) < u.nrows)
          part = ptx::ld_dsmem_f32x2(ptx::mapa(ml_a + (p + (lane >> 3)) * 8, lane & 7));
        const unsigned jr = (unsigned)(u.row0 + p) + (lane >> 3), jb = jr / (unsigned)c.plan.rows_b, jx = jr - jb * (unsigned)c.plan.rows_b;
        const unsigned jt = jx / (unsigned)c.group, jh = u.kvh * c.group + jx - jt * (unsigned)c.group;
        float top = part.x;
#pragma unroll
        for (int k = 4; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float w = part.x == -INFINITY ? 0.f : exp2f(part.x - top);
        float sum = part.x == -INFINITY ? 0.f : w * part.y;
#pragma unroll
        for (int k = 4; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        float acc[R][NV][V] = {};
#pragma unroll 2
        for (int k = 0; k < ranks; ++k) {
          const uint32_t from = ptx::mapa(o_a + p * C::kRowBytes, k);   // (rows past the last lie behind it in the stage)
          float v[R][NV][V];
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              const uint32_t at = from + i * C::kRowBytes + j * 128 * V;
              if (k == rank) {   // (its own memory is not read by way of the cluster, at a quarter of the rate)
                const uint8_t* own = Qs + (p + i) * C::kRowBytes + j * 128 * V + lane * V * 4;
                if (V == 4) *reinterpret_cast<float4*>(v[i][j]) = *reinterpret_cast<const float4*>(own);
                else *reinterpret_cast<float2*>(v[i][j]) = *reinterpret_cast<const float2*>(own);
              } else if (V == 4) *reinterpret_cast<float4*>(v[i][j]) = ptx::ld_dsmem_f32x4(at);
              else *reinterpret_cast<float2*>(v[i][j]) = ptx::ld_dsmem_f32x2(at);
            }
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float wk = __shfl_sync(0xffffffffu, w, 8 * i + k);
            const bool any = __shfl_sync(0xffffffffu, part.x, 8 * i + k) != -INFINITY;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
              for (int e = 0; e < V; ++e) acc[i][j][e] = any ? fmaf(wk, v[i][j][e], acc[i][j][e]) : acc[i][j][e];
          }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float rtop = __shfl_sync(0xffffffffu, top, 8 * i), rsum = __shfl_sync(0xffffffffu, sum, 8 * i);
          const unsigned rb = __shfl_sync(0xffffffffu, jb, 8 * i), rt = __shfl_sync(0xffffffffu, jt, 8 * i), rh = __shfl_sync(0xffffffffu, jh, 8 * i);
          if (p + i >= u.nrows) break;
          const float inv = rtop == -INFINITY ? 0.f : 1.f / rsum;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            uint32_t* to = reinterpret_cast<uint32_t*>(out_bf16(c, rb, rt, rh, j * 32 * V + lane * V));
            if (V == 4) *reinterpret_cast<uint2*>(to) = make_uint2(ptx::pack_bf16x2(acc[i][j][0] * inv, acc[i][j][1] * inv),
                                                                   ptx::pack_bf16x2(acc[i][j][V - 2] * inv, acc[i][j][V - 1] * inv));
            else *to = ptx::pack_bf16x2(acc[i][j][0] * inv, acc[i][j][1] * inv);
          }
          if (c.lse && lane == 0)
            c.lse[((long long)rb * c.Tq + rt) * c.Hq + rh] = rtop == -INFINITY ? -INFINITY : (rtop + log2f(rsum)) * 0.6931471805599453f;
        }
      }
    }
  }
  if (c.plan.cluster > 1) {
    __syncwarp();
    if (warp < C::kSoft) ptx::cluster_sync();     // (the softmax warps' before their join)
    ptx::cluster_sync();                          // the others have read this CTA's rows
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (s_abort) {   // after a timeout loads may be in flight: they land before the CTA's memory is another's
    if (tid == 0)
      for (int i = max(s_loads - NST, 0); i < s_loads; ++i)
        if (!ptx::mbar_wait(&ready[i % NST], (uint32_t)(i / NST) & 1u, kDrainNs)) atomicOr(c.status, RTV_DEV_TIMEOUT);
    __syncthreads();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
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

// Map of one tensor [batch][token][head][D] as [batch][head][64-dim chunk][token][64], with boxes of `keys` tokens of
// `chunks` chunks: a box lies in shared memory chunk by chunk, rows of 128 bytes.
bool encode(CUtensorMap* m, const void* base, int D, int chunks, int keys, int len, int heads, long long st, long long sh,
            int batch, long long sb) {
  const long long dense = 2LL * D;
  const cuuint64_t dims[5] = {64, (cuuint64_t)len, (cuuint64_t)(D / 64), (cuuint64_t)heads, (cuuint64_t)batch};
  const cuuint64_t strides[4] = {(cuuint64_t)(len > 1 ? 2 * st : dense), 128, (cuuint64_t)(heads > 1 ? 2 * sh : dense),
                                 (cuuint64_t)(batch > 1 ? 2 * sb : dense)};
  const cuuint32_t box[5] = {64, (cuuint32_t)keys, (cuuint32_t)chunks, 1, 1}, one[5] = {1, 1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchAttribute cluster_of(int ranks) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ranks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  return at;
}

template <int D>
cudaError_t launch_tc(const AttnCall& c, cudaStream_t st) {
  using C = Cfg<D>;
  AttnMaps m{};
  bool ok = true;
  auto source = [&](const KvSource& s, int batch, CUtensorMap* k, CUtensorMap* v, int* hm, int* bm) {
    if (s.len == 0) return;
    *hm = c.Hkv > 1 && s.sh == 0 ? 0 : 1;
    *bm = batch > 1 && s.sb == 0 ? 0 : 1;
    const int heads = *hm ? c.Hkv : 1, nb = *bm ? batch : 1;
    ok = ok && encode(k, s.k, D, C::CK, C::KT, s.len, heads, s.st, s.sh, nb, s.sb) &&
         encode(v, s.v, D, C::DC, C::VK, s.len, heads, s.st, s.sh, nb, s.sb);
  };
  int pre_b = 0;
  source(c.pre, 1, &m.pre_k, &m.pre_v, &m.pre_h, &pre_b);
  if (!c.plan.decode) source(c.own, c.B, &m.own_k, &m.own_v, &m.own_h, &m.own_b);
  if (!ok) return cudaErrorInvalidValue;
  const long long elems = c.plan.decode ? 0 : (long long)c.B * c.plan.tiles_e * c.plan.ne;
  const dim3 grid((unsigned)((long long)c.plan.tiles_s * c.plan.ns + elems), c.Hkv);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at = cluster_of(c.plan.cluster);
  cfg.attrs = &at;
  cfg.numAttrs = c.plan.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_cache_kernel<D>, c, m);
}

template <int D>
cudaError_t configure(AttnDevice* dev) {
  cudaError_t e = cudaFuncSetAttribute(attn_cache_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  for (int n = 2; n <= kMaxCluster && e == cudaSuccess; ++n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n * 256);
    cfg.blockDim = dim3(Cfg<D>::kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmem;
    cudaLaunchAttribute at = cluster_of(n);
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, attn_cache_kernel<D>, &cfg);
    dev->at_once[D / 128][n] = clusters * n;
  }
  return e;
}

}  // namespace

cudaError_t configure_attention_tc(AttnDevice* dev) {
  if (!encode_fn()) return cudaErrorNotSupported;
  cudaError_t e = configure<64>(dev);
  if (e == cudaSuccess) e = configure<128>(dev);
  if (e == cudaSuccess) e = configure<256>(dev);
  return e;
}

int attention_tc_rows(int D) { return D == 256 ? 128 : 256; }

cudaError_t launch_attention_tc(const AttnCall& c, cudaStream_t st) {
  return c.D == 64 ? launch_tc<64>(c, st) : c.D == 128 ? launch_tc<128>(c, st) : launch_tc<256>(c, st);
}

}  // namespace rtv
