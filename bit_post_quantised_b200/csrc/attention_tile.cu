// attention_tile.cu -- attention of many query rows on the tensor cores
// (tcgen05): tiles of 256 queries against tiles of 128 keys.
//
//   o[r] = sum_j p_j v[j] / sum_j p_j,   p_j = 2^(scale log2(e) (q[r].k[j] - m)),
//
// one pass over the keys with a running reference m and sum.  A unit is two
// 128-row query tiles of one head, both resident in shared memory; their K and
// V tiles stream through one ring (TMA, 128-byte swizzle).  CTAs are
// persistent, one per SM, and every role runs ahead into its next unit: with
// few keys the loads and the output of one unit hide behind the products of
// another (4096 x 512 x 24 heads: 30 us, 45 us as one CTA per unit).  Per key
// tile and query tile: S = Q K^T into 128 TMEM columns; four softmax warps
// read S (a thread owns a row), write P as bf16 over the first half of S;
// O += P V with P from TMEM and V as stored (rows of keys: the MN-major form of
// the B operand), O staying in TMEM over all keys.  While one query tile's
// softmax runs, the other's products do.
//
//   warps 0-3, 4-7  softmax of query tile 0 / 1
//   warp 8          issues the MMAs        warp 9   TMA
//   warp 10         validity of the keys (masked launches)
//   warps 12-15     output of both query tiles, while the softmax warps are
//                   in the next unit already (written by those themselves:
//                   4096 x 512 +5%, 4096 x 77 +10%)
//
// Where units leave SMs idle (few query rows, many keys), a cluster of 2 to 8
// CTAs shares the keys of one: each runs its own key tiles, leaves O and (m,
// sum) in its ring once that is done with, and joins a part of the rows through
// distributed shared memory (2 x 300 x 4000 x 6 heads of 64: 50 -> 21 us, 512 x
// 16,384 x 8 of 128: 205 -> 65).  No workspace, and the same order every time.
//
// The reference m only follows the running maximum when that has grown by
// more than 8 in log2 units: until then probabilities are at most 2^8, which
// costs nothing in fp32 sums or in bf16's relative precision, and O needs no
// rescaling.  When it moves, the softmax warps rescale O themselves after
// the previous product has finished.  P is rounded to bf16 (relative 2^-8 at
// most) because the tensor core takes both operands in one 16-bit type; the
// sum is of the unrounded values.
//
// What bounds it: for two query tiles and one key tile of 128 channels the
// tensor core needs 2048 cycles and their 32,768 exponentials, at 16 a cycle,
// as many.  Measured, a query tile's chain is its softmax (scores 100, maximum
// 300, exponentials 1450 of at least 1024, barriers) and then the product and
// the next scores (1024 and their latencies): a period of some 3300 cycles,
// with the two query tiles half a period apart; 4608 x 4608 x 24 heads take
// 200 us, 0.77 of the measured cuBLAS rate.  Tried and slower: part of the
// exponentials as polynomials on the FMA pipe (the softmax is bound by its
// dependent issue, not by the exponentials' pipe alone: +3 to +9%), 64-key
// steps with two score buffers a query tile (scores of 64 keys read Q from
// shared memory at 48 cycles per 32-cycle MMA: +4 to +18%), an issuing warp per
// query tile (the softmaxes fall into step: +29%; taking turns: -1.5% there,
// +3% elsewhere), two threads a row (+4%), the search for the maximum between
// exponentials that start from the old one (+4%), the last quarter's
// exponentials in the output warps (+6%).
//
// Masked keys: S is replaced by -inf there (whatever it holds) and their V
// rows are overwritten with zeros in shared memory, since 0 * NaN would reach
// O.  Key tiles past kv_len are not loaded.  A row without a valid key gives
// zeros; one with valid keys whose highest score is not finite, NaN.
#include <cfloat>

#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"

namespace tern {

namespace {

constexpr int kBM = 128;        // query rows per tile, two tiles a CTA
constexpr int kBN = 128;        // keys per K or V tile in shared memory
constexpr int kFirst = 96;      // keys of a tile whose P is handed over first
constexpr int kPanel = 16384;   // 128 rows x 64 channels of bf16
constexpr int kThreads = 512;
constexpr int kSoftmaxRegs = 192, kOtherRegs = 72, kOutRegs = 56;
// What the register split asks for has to be there at launch (__launch_bounds__ gives 128 a thread).
constexpr int kLaunchRegs = 128;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs + 128 * kOutRegs <= kThreads * kLaunchRegs, "register split");

template <int DP>
struct TileShape {
  static constexpr int kPanels = DP / 64;
  static constexpr int kTile = kPanels * kPanel;         // bytes of a Q, K or V tile
  static constexpr int kStages = DP == 128 ? 5 : 8;      // K and V tiles in the ring
  static constexpr int kSmem = (2 + kStages) * kTile + 1024;
  static constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kBN >> 3) << 17) |
                                      (uint32_t(kBM >> 4) << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (uint32_t(DP >> 3) << 17) |
                                      (uint32_t(kBM >> 4) << 24);  // bit 16: B is MN-major
  static_assert(kSmem <= 227 * 1024 - 1024, "shared memory");
};

// Shared-memory descriptor of an MN-major bf16 tile written by TMA with
// 128-byte swizzle: 64 consecutive N (channels) per 128-byte row of one k
// (key); 8-key groups 1024 bytes apart, 64-channel panels kPanel apart.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= uint64_t((saddr & 0x3FFFFu) >> 4);
  d |= uint64_t(kPanel >> 4) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

// Four k16 MMAs of one 64-channel panel, D (+)= A B^T with A and B in shared
// memory (K-major): issued by the elected lane of the converged warp.
__device__ __forceinline__ void mma_ss_panel(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|p, 0xffffffff;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Four k16 MMAs D (+)= P V: A from TMEM (8 columns per step), B MN-major in
// shared memory (16 keys, 2048 bytes, per step).
__device__ __forceinline__ void mma_ts_4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync _|p, 0xffffffff;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// The same for two k16 steps.
__device__ __forceinline__ void mma_ts_2(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\t"
      "elect.sync _|p, 0xffffffff;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.s64 b1, %2, 128;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Waits like mbar_wait, in little code: the issuers' and the softmax warps'
// loops are long enough to be bound by instruction fetches where every wait
// carries its polling loop.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, unsigned int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64(), limit = (long long)(limit_ns * 2ull);
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > limit) {
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

// u / d for the u < 2^31 that the reciprocal was made for (see div_by in internal.h).
__device__ __forceinline__ int div_of(int u, const DivBy& d) { return d.mul ? int(__umulhi(unsigned(u), d.mul) >> d.shift) : u; }

// One work unit: two query tiles of a head.
struct Unit {
  int b, h, hk, q0;
  int nq;   // query tiles with a row
  int len;  // keys before kv_len
  int j0;   // first key tile
  int n;    // key tiles
};
template <bool MASK, bool SPLIT>
__device__ __forceinline__ Unit unit_of(const AttnTileArgs& t, int u) {
  const AttnArgs& a = t.a;
  Unit x;
  const int bh = div_of(u, t.by_pairs);
  x.b = div_of(bh, t.by_heads);
  x.h = bh - x.b * a.H;
  x.hk = div_of(x.h, t.by_group);
  x.q0 = (u - bh * t.pairs) * 2 * kBM;
  x.nq = x.q0 + kBM < a.Lq ? 2 : 1;
  x.len = MASK && a.kv_len ? max(0, min(a.Lk, a.kv_len[x.b])) : a.Lk;
  x.j0 = 0;
  x.n = (x.len + kBN - 1) / kBN;
  if constexpr (SPLIT) {  // this CTA's share
    const int share = (x.n + t.splits - 1) / t.splits;
    x.j0 = min(x.n, int(cluster_ctarank()) * share);
    x.n = min(share, x.n - x.j0);
  }
  return x;
}

// Joins the shares that a cluster's NS CTAs left in their shared memory (each
// row's O, kRow floats apart, and its (m, sum)): this CTA's part of the rows,
// by the threads of the softmax warps.  A thread takes eight channels of a
// row at a time; all that it needs from the other CTAs for up to 8 / NS of
// them is asked for before the first is used, since that is latency.
template <int DP, int NS>
__device__ __forceinline__ void join(uint32_t ring, int stats, int row_floats, int rows, float sl, uint16_t* o, const AttnArgs& a) {
  constexpr int kGroups = DP / 8, kItems = 8 / NS, kMine = 2 * kBM / NS;  // rows of this CTA
  constexpr int kTurns = kMine * kGroups / (256 * kItems);
  static_assert(kTurns * 256 * kItems == kMine * kGroups, "whole turns");
  const int first = int(cluster_ctarank()) * kMine;
#pragma unroll 1
  for (int turn = 0; turn < kTurns; ++turn) {
    float2 ms[kItems][NS];
    float4 v[kItems][NS][2];
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int k = (turn * kItems + n) * 256 + int(threadIdx.x), row = first + k / kGroups, ch = k % kGroups * 8;
#pragma unroll
      for (int p = 0; p < NS; ++p) {
        ms[n][p] = ld_cluster_f2(mapa_shared(ring + uint32_t(stats + 8 * row), p));
        const uint32_t at = mapa_shared(ring + uint32_t((row * row_floats + ch) * 4), p);
        v[n][p][0] = ld_cluster_f4(at);
        v[n][p][1] = ld_cluster_f4(at + 16);
      }
    }
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int k = (turn * kItems + n) * 256 + int(threadIdx.x), row = first + k / kGroups, ch = k % kGroups * 8;
      float top = -INFINITY, total = 0.f, acc[8];
#pragma unroll
      for (int p = 0; p < NS; ++p) top = fmaxf(top, ms[n][p].x);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
      for (int p = 0; p < NS; ++p) {
        // Without a key there O was not written.
        const bool none = ms[n][p].x == -INFINITY;
        const float f = none ? 1.f : exp2_fast((ms[n][p].x - top) * sl);
        total = fmaf(ms[n][p].y, f, total);
        const float w[8] = {v[n][p][0].x, v[n][p][0].y, v[n][p][0].z, v[n][p][0].w,
                            v[n][p][1].x, v[n][p][1].y, v[n][p][1].z, v[n][p][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = none ? acc[e] : fmaf(w[e], f, acc[e]);
      }
      const float inv = top == -INFINITY ? 0.f : isinf(top * sl) ? NAN : 1.f / total;
      if (row < rows && ch < a.D)
        *reinterpret_cast<uint4*>(o + (long long)row * a.o_l + ch) =
            make_uint4(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv), pack2(acc[4] * inv, acc[5] * inv),
                       pack2(acc[6] * inv, acc[7] * inv));
    }
  }
}

// SPLIT: the CTAs of a cluster share the keys of one unit, each its own run of
// key tiles, and join their (m, sum, O) through distributed shared memory.
template <int DP, bool MASK, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) attention_tile_kernel(const __grid_constant__ AttnTileArgs t) {
  using C = TileShape<DP>;
  constexpr int S = C::kStages;
  constexpr int kMaskSlots = 4;
  __shared__ __align__(8) uint64_t q_full[2];      // a query tile has landed
  __shared__ __align__(8) uint64_t q_empty[2];     // the unit's last scores are done
  __shared__ __align__(8) uint64_t kv_full[S];     // ring slot landed
  __shared__ __align__(8) uint64_t kv_empty[S];    // every product reading the slot is done
  __shared__ __align__(8) uint64_t s_full[2];      // S of the next key tile is in TMEM
  __shared__ __align__(8) uint64_t p_full[2][2];   // P of the first keys is there (and O rescaled); of the rest
  __shared__ __align__(8) uint64_t o_done[2];      // the unit's O is complete
  __shared__ __align__(8) uint64_t o_free[2];      // the unit's O has been read
  __shared__ __align__(8) uint64_t sum_full[2];    // 1 / sum of the unit's rows
  __shared__ float inv_sum[2][kBM];
  __shared__ __align__(8) uint64_t drain_bar;      // every MMA issued is done
  __shared__ __align__(8) uint64_t v_ready[MASK ? kMaskSlots : 1];   // masked rows of a tile's V are zero
  __shared__ __align__(8) uint64_t m_full[MASK ? kMaskSlots : 1];    // validity of a key tile written
  __shared__ __align__(8) uint64_t m_empty[MASK ? kMaskSlots : 1];   // ... and read by every softmax warp
  __shared__ __align__(16) uint32_t m_words[MASK ? kMaskSlots : 1][4];
  __shared__ uint32_t tmem_base_sh;
  extern __shared__ uint8_t dyn_smem[];

  const AttnArgs& a = t.a;
  const uint64_t lim = t.wait_limit_ns;
  unsigned int* const st = t.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  const uint32_t ring = smem_base + 2 * C::kTile;
  const int units = t.units, u0 = SPLIT ? int(blockIdx.x) / t.splits : int(blockIdx.x), ustep = SPLIT ? units : int(gridDim.x);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&q_full[i]), 1);
      mbar_init(smem_u32(&q_empty[i]), 1);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i][0]), 4);
      mbar_init(smem_u32(&p_full[i][1]), 4);
      mbar_init(smem_u32(&o_done[i]), 1);
      mbar_init(smem_u32(&o_free[i]), 4);
      mbar_init(smem_u32(&sum_full[i]), 4);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&kv_full[s]), 1);
      mbar_init(smem_u32(&kv_empty[s]), 1);
    }
    if (MASK)
      for (int s = 0; s < kMaskSlots; ++s) {
        mbar_init(smem_u32(&m_full[s]), 1);
        mbar_init(smem_u32(&v_ready[s]), 1);
        mbar_init(smem_u32(&m_empty[s]), 8);
      }
    mbar_init(smem_u32(&drain_bar), 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&tmem_base_sh), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp < 8) {
    // ------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2;  // query tile
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + i * kBN, to = tmem + lane_off + 256 + i * DP;
    const float sl = a.scale_log2;
    const float2 sl2 = make_float2(sl, sl);
    uint32_t sp = 0, fp = 1;  // phases of s_full and o_free
    int mt = 0;  // key tiles so far (the slot and phase of the validity words)
    float m = -INFINITY, sum = 0.f;
    bool ok = true, seen = false;  // a valid key in the unit
    for (int u = u0; u < units && ok; u += ustep) {
      const Unit x = unit_of<MASK, SPLIT>(t, u);
      if (i >= x.nq) {
        if constexpr (MASK) {  // not this warp's keys, but its turn in the slots
          for (int j = 0; j < x.n && ok; ++j, ++mt) {
            const int ms = mt % kMaskSlots;
            ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&m_full[ms]), (mt / kMaskSlots) & 1, lim, st));
            if (lane == 0) mbar_arrive(smem_u32(&m_empty[ms]));
          }
        }
        continue;
      }
      m = -INFINITY, sum = 0.f;
      seen = !MASK && x.n > 0;
      for (int j = 0; j < x.n; ++j) {
        ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&s_full[i]), sp, lim, st));
        if (!ok) break;
        sp ^= 1;
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, v[c]);
        tmem_wait_ld();
        if (MASK || x.len - (x.j0 + j) * kBN < kBN) {
          uint32_t w[4];  // validity of the tile's keys
          if constexpr (MASK) {
            const int ms = mt % kMaskSlots;
            ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&m_full[ms]), (mt / kMaskSlots) & 1, lim, st));
            if (!ok) break;
            const uint4 mw = *reinterpret_cast<const uint4*>(m_words[ms]);
            w[0] = mw.x, w[1] = mw.y, w[2] = mw.z, w[3] = mw.w;
            seen |= (mw.x | mw.y | mw.z | mw.w) != 0u;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&m_empty[ms]));
            ++mt;
          } else {
            const int rem = x.len - (x.j0 + j) * kBN;
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = rem >= 32 * c + 32 ? ~0u : rem <= 32 * c ? 0u : (1u << (rem - 32 * c)) - 1u;
          }
          if (!MASK || (w[0] & w[1] & w[2] & w[3]) != ~0u) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((w[c] >> e) & 1u)) v[c][e] = 0xFF800000u;  // -inf
          }
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          top[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
          for (int e = 2; e < 32; e += 2) top[c] = max3(top[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
        }
        const float to_max = fmaxf(max3(m, top[0], top[1]), fmaxf(top[2], top[3]));
        const bool move = (to_max - m) * sl > 8.f;  // false for NaN: both still -inf, or a NaN score
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? exp2_fast((m - to_max) * sl) : 1.f;
          if (move) m = to_max;
          sum *= f;
          if (j > 0) {
            // These scores were issued behind the last product: that one is done.
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
              uint32_t y[32];
              tmem_ld32(to + c, y);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
              tmem_st32(to + c, y);
            }
          }
        }
        float base = m == -INFINITY ? 0.f : -m * sl;
        // The multiply-add below rounds m * sl but not v * sl: a factor of up to
        // 2^(2^-24 |m * sl|) common to the row's probabilities, which would
        // overflow where scores are that far from zero.  There the reference is
        // taken off first.  (The test costs 4608 x 4608 x 24 heads 1 %.)
        if (fabsf(base) > 1048576.f) {
          base = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) v[c][e] = __float_as_uint(__uint_as_float(v[c][e]) - m);
        }
        const float2 base2 = make_float2(base, base);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 y = fma2(make_float2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])), sl2, base2);
            y.x = exp2_fast(y.x);
            y.y = exp2_fast(y.y);
            acc[e & 1] = add2(acc[e & 1], y);
            p[e] = pack2(y.x, y.y);
          }
          tmem_st16(ts + 16 * c, p);  // P over the first 64 columns of S
          if (32 * c + 32 == kFirst || c == 3) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[i][c == 3]));
          }
        }
        acc[0] = add2(acc[0], acc[1]);
        sum += acc[0].x + acc[0].y;
      }
      if (!ok) break;
      if constexpr (SPLIT) {
        // Only NaN and -inf among valid keys: told from no key by a maximum that is finite.
        if (seen && m == -INFINITY) m = -FLT_MAX;
      }
      if (SPLIT || x.n == 0) continue;
      // The rows' sums to the output warps, once they are through with the unit before.
      ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&o_free[i]), fp, lim, st));
      if (!ok) break;
      fp ^= 1;
      inv_sum[i][(warp & 3) * 32 + lane] = !seen ? 0.f : isinf(m * sl) ? NAN : 1.f / sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sum_full[i]));
    }
    if constexpr (SPLIT) {
      const Unit x = unit_of<MASK, SPLIT>(t, u0);
      // Every product of this CTA is done, so its ring is free: O and (m, sum)
      // of its rows go there.
      for (int k = 0; k < x.nq && x.n > 0 && ok; ++k)
        ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&o_done[k]), 0, lim, st));
      constexpr int kRow = DP + 4;  // floats: a warp's rows start in different banks
      constexpr int kStats = 2 * kBM * kRow * 4;
      static_assert(kStats + 2 * kBM * 8 <= S * C::kTile, "the join fits the ring");
      const int r = i * kBM + (warp & 3) * 32 + lane;
      if (ok) {
        tc_fence_after();
        const uint32_t row = ring + uint32_t(r * kRow * 4);
        if (i < x.nq && x.n > 0)
#pragma unroll 1
          for (int c = 0; c < DP; c += 32) {
            uint32_t y[32];
            tmem_ld32(to + c, y);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + uint32_t(4 * (c + e))), "r"(y[e]),
                           "r"(y[e + 1]), "r"(y[e + 2]), "r"(y[e + 3])
                           : "memory");
          }
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ring + uint32_t(kStats + 8 * r)), "f"(m), "f"(sum) : "memory");
      }
      cluster_sync();
      const int rows = min(2 * kBM, a.Lq - x.q0);
      uint16_t* const o = a.o + x.b * a.o_b + (long long)x.q0 * a.o_l + x.h * a.o_h;
      if (t.splits == 2) join<DP, 2>(ring, kStats, kRow, rows, sl, o, a);
      else if (t.splits == 4) join<DP, 4>(ring, kStats, kRow, rows, sl, o, a);
      else join<DP, 8>(ring, kStats, kRow, rows, sl, o, a);
      cluster_sync_relaxed();  // no CTA leaves while another may still read its shared memory
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------ output
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    uint32_t ph = 0;  // bit i: phase of o_done and sum_full
    bool ok = true;
    for (int u = u0; !SPLIT && u < units && ok; u += ustep) {
      const Unit x = unit_of<MASK, SPLIT>(t, u);
#pragma unroll 1
      for (int i = 0; i < x.nq; ++i) {
        const uint32_t to = tmem + lane_off + 256 + i * DP;
        float inv = 0.f;
        if (x.n > 0) {
          ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&sum_full[i]), (ph >> i) & 1, lim, st) &&
                                           bar_wait(smem_u32(&o_done[i]), (ph >> i) & 1, lim, st));
          if (!ok) break;
          ph ^= 1u << i;
          tc_fence_after();
          inv = inv_sum[i][r];
        }
        const int row = x.q0 + i * kBM + r;
        uint16_t* o_row = a.o + x.b * a.o_b + (long long)row * a.o_l + x.h * a.o_h;
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
          uint32_t y[32];
          if (x.n > 0) {
            tmem_ld32(to + c, y);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = 0u;
          }
          if (x.n > 0 && c + 32 == DP) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&o_free[i]));
          }
          if (row < a.Lq) {
            uint32_t z[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) z[e] = pack2(__uint_as_float(y[2 * e]) * inv, __uint_as_float(y[2 * e + 1]) * inv);
            // A thread's row is contiguous, its neighbours' rows are far: whole
            // 32-byte sectors where o's alignment allows (a.D % 16 == 0 then).
            if (t.o_sectors) {
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                if (c + 2 * e < a.D)
                  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o_row + c + 2 * e), "r"(z[e]),
                               "r"(z[e + 1]), "r"(z[e + 2]), "r"(z[e + 3]), "r"(z[e + 4]), "r"(z[e + 5]), "r"(z[e + 6]),
                               "r"(z[e + 7])
                               : "memory");
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                if (c + 2 * e < a.D)
                  *reinterpret_cast<uint4*>(o_row + c + 2 * e) = make_uint4(z[e], z[e + 1], z[e + 2], z[e + 3]);
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---------------------------------------------------- MMA issuer
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      bool ok = true;
      // Every lane with `need` waits for a barrier of its own: one poll, of
      // some 150 cycles, for all that a step needs.
      auto wait_all = [&](uint32_t bar, uint32_t parity, bool need) {
        bool done = !need || mbar_try_wait(bar, parity);
        if (__all_sync(0xffffffffu, done)) return true;
        const long long t0 = clock64(), limit = (long long)(lim * 2ull);
#pragma unroll 1
        while (true) {
          if (!done) done = mbar_try_wait(bar, parity);
          if (__all_sync(0xffffffffu, done)) return true;
          if (__any_sync(0xffffffffu, clock64() - t0 > limit)) {
            if (lane == 0) atomicOr(st, kStatusTimeout);
            return false;
          }
        }
      };
      // Key tiles in order, over all units; for each query tile in turn its
      // product and right behind it the scores of the next key tile (of the
      // next unit, too) into the same S: MMAs of one thread run in order.
      // Taking the query tiles in turn also keeps their softmaxes half a
      // period apart, one with the other's products.  This warp's own time
      // between its MMAs is what the tensor core idles, so it polls
      // together for what a step needs: lane 0 for V, 1 for K, 2 for P, 3 for the query tile, 4 for
      // O to be free, 5 for V's masked rows.
      const uint64_t qd0 = sw128_kmajor_desc(smem_base);
      const uint64_t kd0 = sw128_kmajor_desc(ring), vd0 = sw128_mnmajor_desc(ring);
      constexpr uint32_t kSlot = C::kTile >> 4;  // in descriptor units
      const uint32_t full0 = smem_u32(&kv_full[0]), empty0 = smem_u32(&kv_empty[0]);
      const uint32_t own_bar = lane == 2 ? smem_u32(&p_full[0][0]) : lane == 3 ? smem_u32(&q_full[0]) : smem_u32(&o_free[0]);
      auto next_unit = [&](int u, Unit& x) {  // the first unit from u on with keys
        for (; u < units; u += ustep) {
          x = unit_of<MASK, SPLIT>(t, u);
          if (x.n > 0) break;
        }
        return u;
      };
      Unit y{};  // the unit of the tile whose scores are next
      int un = next_unit(u0, y), yj = 0;
      bool last = false;                       // the tile whose product is next is its unit's last
      int nq = 0, nq_next = un < units ? y.nq : 0;  // query tiles of that tile (0: none), and of the next
      int j = 0, tile = 0;                     // its place in the unit and among all
      int ks = 0, vs = 1 % S;
      uint32_t kp = 0, vp = 0;                 // phases of the ring
      uint32_t pp = 0, qp = 0, op = 3;         // bit i: of p_full, q_full, o_free
      while (nq | nq_next) {
        const bool last_next = yj == y.n - 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool mul = i < nq, score = i < nq_next;
          {
            uint32_t bar = own_bar + (lane == 2 ? 16 : 8) * i, parity = ((lane == 2 ? pp : lane == 3 ? qp : op) >> i) & 1;
            bool need = lane == 2 ? mul : lane == 3 ? score && yj == 0 : lane == 4 ? mul && j == 0 : false;
            if (i == 0 && lane < 2) {
              bar = full0 + 8 * (lane == 0 ? vs : ks);
              parity = lane == 0 ? vp : kp;
              need = lane == 0 ? mul : score;
            }
            if (MASK && i == 0 && lane == 5) {
              bar = smem_u32(&v_ready[tile % kMaskSlots]);
              parity = (tile / kMaskSlots) & 1;
              need = mul;
            }
            ok = wait_all(bar, parity, need);
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t ts = tm + i * kBN, to = tm + 256 + i * DP;
          if (mul) {
            const uint64_t vd = vd0 + uint32_t(vs) * kSlot;
            mma_ts_4(to, ts, vd, C::kIdescO, j > 0);
            mma_ts_2(to, ts + 32, vd + 512, C::kIdescO, 1);
            ok = wait_all(smem_u32(&p_full[i][1]), (pp >> i) & 1, true);
            if (!ok) break;
            tc_fence_after();
            mma_ts_2(to, ts + 48, vd + 768, C::kIdescO, 1);
            if (last) mma_commit_elected(smem_u32(&o_done[i]));
            if (i == nq - 1) mma_commit_elected(empty0 + 8 * vs);
            pp ^= 1u << i;
            if (j == 0) op ^= 1u << i;
          }
          if (score) {
            const uint64_t qd = qd0 + uint32_t(i) * kSlot, kd = kd0 + uint32_t(ks) * kSlot;
            mma_ss_panel(ts, qd, kd, C::kIdescS, 0);
            if constexpr (C::kPanels == 2) mma_ss_panel(ts, qd + (kPanel >> 4), kd + (kPanel >> 4), C::kIdescS, 1);
            mma_commit_elected(smem_u32(&s_full[i]));
            if (last_next) mma_commit_elected(smem_u32(&q_empty[i]));
            if (i == nq_next - 1) mma_commit_elected(empty0 + 8 * ks);
            if (yj == 0) qp ^= 1u << i;
          }
        }
        if (!ok) break;
        if (nq > 0) {
          vs += 2, vp ^= uint32_t(vs >= S), vs -= vs >= S ? S : 0;
          ++tile;
        }
        nq = nq_next, j = yj, last = last_next;
        if (nq_next > 0) {
          ks += 2, kp ^= uint32_t(ks >= S), ks -= ks >= S ? S : 0;
          if (++yj == y.n) {
            yj = 0;
            un = next_unit(un + ustep, y);
            nq_next = un < units ? y.nq : 0;
          }
        }
      }
      mma_commit_elected(smem_u32(&drain_bar));
      __syncwarp();
      mbar_wait(smem_u32(&drain_bar), 0, lim, st);
    } else if (warp == 9) {
      // ---------------------------------------------------- TMA
      if (lane == 0) {
        prefetch_tensormap(&t.tq);
        prefetch_tensormap(&t.tk);
        prefetch_tensormap(&t.tv);
        auto load = [&](uint32_t dst, const CUtensorMap* map, int r, int hh, int bb, uint64_t* bar) {
          mbar_arrive_expect_tx(smem_u32(bar), C::kTile);
#pragma unroll
          for (int p = 0; p < C::kPanels; ++p) tma_load_4d(dst + p * kPanel, map, 64 * p, r, hh, bb, smem_u32(bar));
        };
        int it = 0, qc[2] = {0, 0};
        bool ok = true;
        for (int u = u0; u < units && ok; u += ustep) {
          const Unit x = unit_of<MASK, SPLIT>(t, u);
          for (int k = 0; k < 2 * x.n && ok; ++k) {
            const int s = it % S;
            ok = mbar_wait(smem_u32(&kv_empty[s]), ((it / S) & 1) ^ 1, lim, st);
            if (!ok) break;
            if (k & 1)
              load(ring + s * C::kTile, &t.tv, (x.j0 + (k >> 1)) * kBN, x.hk * t.v_h, x.b * t.v_b, &kv_full[s]);
            else
              load(ring + s * C::kTile, &t.tk, (x.j0 + (k >> 1)) * kBN, x.hk * t.k_h, x.b * t.k_b, &kv_full[s]);
            ++it;
            if (k == 0) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (i >= x.nq || !ok) break;
                ok = mbar_wait(smem_u32(&q_empty[i]), (qc[i] & 1) ^ 1, lim, st);
                if (!ok) break;
                load(smem_base + i * C::kTile, &t.tq, x.q0 + i * kBM, x.h * t.q_h, x.b * t.q_b, &q_full[i]);
                ++qc[i];
              }
            }
          }
        }
        // No copy may still be landing when the CTA exits.
        for (int i = 0; i < 2; ++i)
          if (qc[i] > 0) mbar_wait(smem_u32(&q_full[i]), (qc[i] - 1) & 1, lim, st);
        for (int k = it > S ? it - S : 0; k < it; ++k) mbar_wait(smem_u32(&kv_full[k % S]), (k / S) & 1, lim, st);
      }
      __syncwarp();
    } else if (MASK && warp == 10) {
      // ---------------------------------------------------- key validity
      int mt = 0;
      bool ok = true;
      for (int u = u0; u < units && ok; u += ustep) {
        const Unit x = unit_of<MASK, SPLIT>(t, u);
        const uint8_t* mask = a.key_mask ? a.key_mask + x.b * a.mask_ld : nullptr;
        for (int j = 0; j < x.n && ok; ++j, ++mt) {
          const int ms = mt % kMaskSlots, it = 2 * mt + 1, vs = it % S;
          uint32_t w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = (x.j0 + j) * kBN + 32 * c + lane;
            w[c] = __ballot_sync(0xffffffffu, key < x.len && (!mask || mask[key]));
          }
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m_empty[ms]), ((mt / kMaskSlots) & 1) ^ 1, lim, st));
          if (!ok) break;
          if (lane == 0) {
            *reinterpret_cast<uint4*>(m_words[ms]) = make_uint4(w[0], w[1], w[2], w[3]);
            mbar_arrive(smem_u32(&m_full[ms]));
          }
          // The slot's V has landed before its masked rows are cleared; the
          // clearing is made visible to the tensor core before the arrival.
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&kv_full[vs]), (it / S) & 1, lim, st));
          if (!ok) break;
          if ((w[0] & w[1] & w[2] & w[3]) != ~0u) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (!((w[c] >> lane) & 1u)) {
                uint8_t* r = dyn_smem + (ring - smem_u32(dyn_smem)) + vs * C::kTile + (32 * c + lane) * 128;
#pragma unroll
                for (int p = 0; p < C::kPanels; ++p)
#pragma unroll
                  for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(r + p * kPanel + 16 * k) = make_uint4(0u, 0u, 0u, 0u);
              }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&v_ready[ms]));
        }
      }
    }
  }
  if constexpr (SPLIT) {
    if (warp >= 8) {  // the softmax warps' two
      __syncwarp();
      cluster_sync();
      cluster_sync_relaxed();
    }
  }
  // Every role is done with TMEM and the barriers.
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP, bool MASK, bool SPLIT>
cudaError_t launch_one(const AttnTileArgs& t, cudaStream_t stream) {
  using C = TileShape<DP>;
  // Per device: the kernel's shared memory, and that it was compiled to the
  // registers which the split between its warps counts on (waiting for ones
  // that are not there would never end).
  static thread_local int ready_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready_dev != dev) {
    cudaFuncAttributes f;
    if ((e = cudaFuncGetAttributes(&f, attention_tile_kernel<DP, MASK, SPLIT>)) != cudaSuccess) return e;
    if (f.numRegs * kThreads < 256 * kSoftmaxRegs + 128 * kOtherRegs + 128 * kOutRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(attention_tile_kernel<DP, MASK, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready_dev = dev;
  }
  const int grid = SPLIT ? t.units * t.splits : t.units < t.ctas ? t.units : t.ctas;
  return launch_pdl(attention_tile_kernel<DP, MASK, SPLIT>, dim3(unsigned(grid)), dim3(kThreads), C::kSmem, stream,
                    SPLIT ? unsigned(t.splits) : 1u, t);
}

}  // namespace

template <bool SPLIT>
static cudaError_t launch_tile(const AttnTileArgs& t, cudaStream_t stream) {
  const bool mask = t.a.kv_len || t.a.key_mask;
  if (t.a.D <= 64) return mask ? launch_one<64, true, SPLIT>(t, stream) : launch_one<64, false, SPLIT>(t, stream);
  return mask ? launch_one<128, true, SPLIT>(t, stream) : launch_one<128, false, SPLIT>(t, stream);
}

cudaError_t launch_attention_tile(const AttnTileArgs& t, cudaStream_t stream) {
  return t.splits > 1 ? launch_tile<true>(t, stream) : launch_tile<false>(t, stream);
}

}  // namespace tern
