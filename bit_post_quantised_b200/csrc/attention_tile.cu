// attention_tile.cu -- attention of many query rows on the tensor cores
// (tcgen05): tiles of 256 queries against tiles of 128 keys.
//
//   o[r] = sum_j p_j v[j] / sum_j p_j,   p_j = 2^(scale log2(e) (q[r].k[j] - m)),
//
// one pass over the keys with a running reference m and sum.  A CTA owns two
// 128-row query tiles of one head, both resident in shared memory, and
// streams K and V tiles (TMA, 128-byte swizzle) through one ring.  Per key
// tile and query tile: S = Q K^T into 128 TMEM columns; four softmax warps
// read S (a thread owns a row), write P as bf16 over the first half of S;
// O += P V with P from TMEM and V as stored (rows of keys: the MN-major form of
// the B operand), O staying in TMEM over all keys.  While one query tile's
// softmax runs, the other's products do.
//
//   warps 0-3, 4-7  softmax and output of query tile 0 / 1
//   warp 8          issues the MMAs        warp 9   TMA
//   warp 10         validity of the keys (masked launches)
//
// The reference m only follows the running maximum when that has grown by
// more than 8 in log2 units: until then probabilities are at most 2^8, which
// costs nothing in fp32 sums or in bf16's relative precision, and O needs no
// rescaling.  When it moves, the softmax warps rescale O themselves after
// the previous product has finished.  P is rounded to bf16 (relative 2^-8 at
// most) because the tensor core takes both operands in one 16-bit type; the
// sum is of the unrounded values.
//
// Masked keys: S is replaced by -inf there (whatever it holds) and their V
// rows are overwritten with zeros in shared memory, since 0 * NaN would reach
// O.  Key tiles past kv_len are not loaded.  A row without a valid key gives
// zeros.
#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"

namespace tern {

namespace {

constexpr int kBM = 128;        // query rows per tile, two tiles a CTA
constexpr int kBN = 128;        // keys per tile
constexpr int kPanel = 16384;   // 128 rows x 64 channels of bf16
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
// What the register split asks for has to be there at launch (__launch_bounds__ gives 168 a thread).
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register split");

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

template <int DP, bool MASK>
__global__ void __launch_bounds__(kThreads, 1) attention_tile_kernel(const __grid_constant__ AttnTileArgs t) {
  using C = TileShape<DP>;
  constexpr int S = C::kStages;
  constexpr int kMaskSlots = 4;
  __shared__ __align__(8) uint64_t q_full[2];      // a query tile has landed
  __shared__ __align__(8) uint64_t kv_full[S];     // ring slot landed
  __shared__ __align__(8) uint64_t kv_empty[S];    // every product reading the slot is done
  __shared__ __align__(8) uint64_t s_full[2];      // S of the next key tile is in TMEM
  __shared__ __align__(8) uint64_t p_full[2];      // P is in TMEM (and O rescaled)
  __shared__ __align__(8) uint64_t o_done[2];      // O += P V is done
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

  const int pair = int(blockIdx.x % unsigned(t.pairs));
  const int bh = int(blockIdx.x / unsigned(t.pairs));
  const int h = bh % a.H, b = bh / a.H;
  const int hk = h / (a.H / a.Hkv);
  const int q0 = pair * 2 * kBM;
  const int nq = q0 + kBM < a.Lq ? 2 : 1;  // query tiles with a row

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&q_full[i]), 1);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), 4);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&kv_full[s]), 1);
      mbar_init(smem_u32(&kv_empty[s]), 1);
    }
    if (MASK)
      for (int s = 0; s < kMaskSlots; ++s) {
        mbar_init(smem_u32(&m_full[s]), 1);
        mbar_init(smem_u32(&v_ready[s]), 1);
        mbar_init(smem_u32(&m_empty[s]), 4 * nq);
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
  const int len = MASK && a.kv_len ? max(0, min(a.Lk, a.kv_len[b])) : a.Lk;
  const int n = (len + kBN - 1) / kBN;  // key tiles

  if (warp < 8) {
    // ------------------------------------------------------ softmax, output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2;  // query tile
    const int row = q0 + i * kBM + (warp & 3) * 32 + lane;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + i * kBN, to = tmem + lane_off + 256 + i * DP;
    const float sl = a.scale_log2;
    float m = -INFINITY, sum = 0.f;
    bool ok = true;
    if (i < nq) {
      for (int j = 0; j < n; ++j) {
        uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};  // validity of the tile's keys
        if constexpr (MASK) {
          const int ms = j % kMaskSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m_full[ms]), (j / kMaskSlots) & 1, lim, st));
          if (!ok) break;
          const uint4 mw = *reinterpret_cast<const uint4*>(m_words[ms]);
          w[0] = mw.x, w[1] = mw.y, w[2] = mw.z, w[3] = mw.w;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&m_empty[ms]));
        } else if (len - j * kBN < kBN) {
          const int rem = len - j * kBN;
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = rem >= 32 * c + 32 ? ~0u : rem <= 32 * c ? 0u : (1u << (rem - 32 * c)) - 1u;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s_full[i]), j & 1, lim, st));
        if (!ok) break;
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, v[c]);
        tmem_wait_ld();
        if ((w[0] & w[1] & w[2] & w[3]) != ~0u) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((w[c] >> e) & 1u)) v[c][e] = 0xFF800000u;  // -inf
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          top[c] = __uint_as_float(v[c][0]);
#pragma unroll
          for (int e = 1; e < 32; ++e) top[c] = fmaxf(top[c], __uint_as_float(v[c][e]));
        }
        const float to_max = fmaxf(fmaxf(m, fmaxf(top[0], top[1])), fmaxf(top[2], top[3]));
        const bool move = (to_max - m) * sl > 8.f;  // false for NaN: both still -inf
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? exp2_fast((m - to_max) * sl) : 1.f;
          if (move) m = to_max;
          sum *= f;
          if (j > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&o_done[i]), (j - 1) & 1, lim, st));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
              uint32_t x[32];
              tmem_ld32(to + c, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
              tmem_st32(to + c, x);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : -m * sl;
        const float2 sl2 = make_float2(sl, sl), base2 = make_float2(base, base);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 x = fma2(make_float2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])), sl2, base2);
            x.x = exp2_fast(x.x);
            x.y = exp2_fast(x.y);
            acc[e & 1] = add2(acc[e & 1], x);
            p[e] = pack2(x.x, x.y);
          }
          tmem_st16(ts + 16 * c, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[i]));
        acc[0] = add2(acc[0], acc[1]);
        sum += acc[0].x + acc[0].y;
      }
      if (ok && n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&o_done[i]), (n - 1) & 1, lim, st));
        tc_fence_after();
      }
      if (ok) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t* op = a.o + b * a.o_b + (long long)row * a.o_l + h * a.o_h;
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
          uint32_t x[32];
          if (n > 0) {
            tmem_ld32(to + c, x);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = 0u;
          }
          if (row < a.Lq) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              if (c + e < a.D) {
                uint32_t y[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  y[u] = pack2(__uint_as_float(x[e + 2 * u]) * inv, __uint_as_float(x[e + 2 * u + 1]) * inv);
                *reinterpret_cast<uint4*>(op + c + e) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          }
        }
        tc_fence_before();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---------------------------------------------------- MMA issuer
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      bool ok = n > 0;
      auto wait = [&](uint64_t* bar, int parity) {
        return __shfl_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, lim, st), 0);
      };
      auto scores = [&](int i, int slot) {
        const uint64_t qd = sw128_kmajor_desc(smem_base + i * C::kTile), kd = sw128_kmajor_desc(ring + slot * C::kTile);
        mma_ss_panel(tm + i * kBN, qd, kd, C::kIdescS, 0);
        if constexpr (C::kPanels == 2)
          mma_ss_panel(tm + i * kBN, qd + (kPanel >> 4), kd + (kPanel >> 4), C::kIdescS, 1);
        mma_commit_elected(smem_u32(&s_full[i]));
      };
      for (int i = 0; i < nq && ok; ++i) {
        ok = wait(&q_full[i], 0) && (i > 0 || wait(&kv_full[0], 0));
        if (!ok) break;
        tc_fence_after();
        scores(i, 0);
      }
      if (ok) mma_commit_elected(smem_u32(&kv_empty[0]));
      for (int j = 0; j < n && ok; ++j) {
        const int it = 2 * j + 1, vs = it % S;                // V of tile j
        const int kt = it + 1, ks = kt % S;                   // K of tile j + 1
        ok = wait(&kv_full[vs], (it / S) & 1) && (!MASK || wait(&v_ready[j % kMaskSlots], (j / kMaskSlots) & 1));
        for (int i = 0; i < nq && ok; ++i) {
          ok = wait(&p_full[i], j & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = sw128_mnmajor_desc(ring + vs * C::kTile);
          mma_ts_4(tm + 256 + i * DP, tm + i * kBN, vd, C::kIdescO, j > 0);
          mma_ts_4(tm + 256 + i * DP, tm + i * kBN + 32, vd + 512, C::kIdescO, 1);
          mma_commit_elected(smem_u32(&o_done[i]));
          if (i == nq - 1) mma_commit_elected(smem_u32(&kv_empty[vs]));
          if (j + 1 < n) {
            // S of the next tile overwrites this P: MMAs of one thread run in order.
            if (i == 0) ok = wait(&kv_full[ks], (kt / S) & 1);
            if (!ok) break;
            tc_fence_after();
            scores(i, ks);
            if (i == nq - 1) mma_commit_elected(smem_u32(&kv_empty[ks]));
          }
        }
      }
      if (n > 0) {
        mma_commit_elected(smem_u32(&drain_bar));
        __syncwarp();
        mbar_wait(smem_u32(&drain_bar), 0, lim, st);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------- TMA
      if (lane == 0 && n > 0) {
        prefetch_tensormap(&t.tq);
        prefetch_tensormap(&t.tk);
        prefetch_tensormap(&t.tv);
        auto load = [&](uint32_t dst, const CUtensorMap* map, int r, int hh, int bb, uint64_t* bar) {
          mbar_arrive_expect_tx(smem_u32(bar), C::kTile);
#pragma unroll
          for (int p = 0; p < C::kPanels; ++p) tma_load_4d(dst + p * kPanel, map, 64 * p, r, hh, bb, smem_u32(bar));
        };
        load(smem_base, &t.tq, q0, h * t.q_h, b * t.q_b, &q_full[0]);
        int it = 0;
        bool ok = true;
        for (; it < 2 * n; ++it) {
          const int s = it % S;
          ok = mbar_wait(smem_u32(&kv_empty[s]), ((it / S) & 1) ^ 1, lim, st);
          if (!ok) break;
          if (it & 1)
            load(ring + s * C::kTile, &t.tv, (it >> 1) * kBN, hk * t.v_h, b * t.v_b, &kv_full[s]);
          else
            load(ring + s * C::kTile, &t.tk, (it >> 1) * kBN, hk * t.k_h, b * t.k_b, &kv_full[s]);
          if (it == 0 && nq > 1) load(smem_base + C::kTile, &t.tq, q0 + kBM, h * t.q_h, b * t.q_b, &q_full[1]);
        }
        // No copy may still be landing when the CTA exits.
        for (int i = 0; i < nq && (i == 0 || it > 0); ++i) mbar_wait(smem_u32(&q_full[i]), 0, lim, st);
        for (int x = it > S ? it - S : 0; x < it; ++x) mbar_wait(smem_u32(&kv_full[x % S]), (x / S) & 1, lim, st);
      }
      __syncwarp();
    } else if (MASK && warp == 10) {
      // ---------------------------------------------------- key validity
      const uint8_t* mask = a.key_mask ? a.key_mask + b * a.mask_ld : nullptr;
      for (int j = 0; j < n; ++j) {
        const int ms = j % kMaskSlots, it = 2 * j + 1, vs = it % S;
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int key = j * kBN + 32 * c + lane;
          w[c] = __ballot_sync(0xffffffffu, key < len && (!mask || mask[key]));
        }
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&m_empty[ms]), ((j / kMaskSlots) & 1) ^ 1, lim, st))) break;
        if (lane == 0) {
          *reinterpret_cast<uint4*>(m_words[ms]) = make_uint4(w[0], w[1], w[2], w[3]);
          mbar_arrive(smem_u32(&m_full[ms]));
        }
        // The slot's V has landed before its masked rows are cleared; the
        // clearing is made visible to the tensor core before the arrival.
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&kv_full[vs]), (it / S) & 1, lim, st))) break;
        if ((w[0] & w[1] & w[2] & w[3]) != ~0u) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (!((w[c] >> lane) & 1u)) {
              uint8_t* r = dyn_smem + (ring - smem_u32(dyn_smem)) + vs * C::kTile + (32 * c + lane) * 128;
#pragma unroll
              for (int p = 0; p < C::kPanels; ++p)
#pragma unroll
                for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(r + p * kPanel + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
            }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&v_ready[ms]));
      }
    }
  }
  // Every role is done with TMEM and the barriers.
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int DP, bool MASK>
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
    if ((e = cudaFuncGetAttributes(&f, attention_tile_kernel<DP, MASK>)) != cudaSuccess) return e;
    if (f.numRegs * kThreads < 256 * kSoftmaxRegs + 128 * kOtherRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(attention_tile_kernel<DP, MASK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready_dev = dev;
  }
  return launch_pdl(attention_tile_kernel<DP, MASK>, dim3(unsigned(t.pairs) * unsigned(t.a.B * t.a.H)), dim3(kThreads),
                    C::kSmem, stream, 1, t);
}

}  // namespace

cudaError_t launch_attention_tile(const AttnTileArgs& t, cudaStream_t stream) {
  const bool mask = t.a.kv_len || t.a.key_mask;
  if (t.a.D <= 64) return mask ? launch_one<64, true>(t, stream) : launch_one<64, false>(t, stream);
  return mask ? launch_one<128, true>(t, stream) : launch_one<128, false>(t, stream);
}

}  // namespace tern
