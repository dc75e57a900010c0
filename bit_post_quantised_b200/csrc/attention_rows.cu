// attention_rows.cu -- attention of few query rows to an encoder's states:
// one read of the keys and values, split over the keys and joined inside a
// cluster.
//
//   o[r] = sum_j softmax_j(scale q[r].k[j]) v[j]   over the valid keys j.
//
// The G = H / Hkv query heads that share a key-value head are rows of one
// 16-row tile (row r: query r / G, head r % G of the group), so K and V are
// read once for all of them; with few rows the bound is that read.  A unit is
// (batch entry, key-value head, 16 rows); a cluster of up to 16 CTAs splits its
// keys in blocks of 16 dealt round-robin to all its warps.  A warp keeps its
// running row maxima, sums and 16 x D output in registers, all fp32, and has
// a ring of its own in shared memory for its next blocks (cp.async, no barrier
// with other warps; loaded straight into registers, one block ahead, two
// thirds of the warps' time was the wait for V: 1.5 TB/s on 16,384 keys).
//   - the order of the products' channels is free as long as q and k agree,
//     so thread t of a quad takes channels 32 i + 8 t .. + 7 of a key, 16
//     bytes, as two k16 steps' fragments;
//   - the output channels' places in the n8 tiles are free too: row g of the
//     quad owns channels 64 c + 8 g .. + 7 of a value row, and keys 2t, 2t + 1
//     of each eight, the ones whose scores it holds.
// 16-byte groups are swizzled by the key so that both reads meet every bank.
// The probabilities go to the tensor cores as the sum of two bf16 (value and
// remainder): the extra product is free under the memory bound and leaves
// only the final rounding.  Masked keys have their score replaced (not added
// to) and their value row zeroed, so whatever they hold is not seen; a row
// without a valid key gives zeros.  Where the valid keys' scores are all -inf or
// NaN the maximum becomes -FLT_MAX, to tell the row from one without a key: it
// has nothing to divide by, or a sum that is NaN, and gives NaN.
//
// The ring is sized for two CTAs an SM, which also lets eight clusters of 16
// be resident.  Many heads are bound by memory (64 x 1 query, 4096 keys, 8 heads:
// 153 us, 7.0 TB/s); few of them by a block's chain in its warp and the loads'
// latency alike (16,384 keys x 8 heads: 21.1 us, 3.2 TB/s; 17 with the copies
// alone, 17.4 without them; blocks of 32 keys, one CTA an SM, leave room for
// seven clusters only: 46 us), short calls by their latency (512 keys x 24 heads,
// one query: 6.8 us, of which the copies and the join are 5.6).
//
// Join: the four warps of a CTA combine their (max, sum, output) through
// shared memory, then the CTAs of the cluster through distributed shared
// memory, each CTA writing a slice of the rows: one launch, no workspace.
#include <cfloat>

#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"

namespace tern {

namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;
constexpr int kKeys = 16;  // of a block

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint16_t* src, bool ok) {
  // 16 bytes, or zeros where !ok (nothing is read then)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint4 load16(const uint16_t* p, bool ok) {
  return ok ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// hi = bf16 pair of (x, y), lo = bf16 pair of what that rounding left.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  const float rx = x - __uint_as_float(hi << 16), ry = y - __uint_as_float(hi & 0xFFFF0000u);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(ry), "f"(rx));
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// Shared memory of a CTA: the warps' rings, then (over them) the join.
template <int DP>
struct RowsSmem {
  static constexpr int kBlock = kKeys * DP * 2;               // bytes of a block's keys or values
  static constexpr int kStages = DP == 128 ? 3 : 6;           // of a warp's ring, K and V each
  static constexpr int kRing = kWarps * kStages * 2 * kBlock;  // 96 KB
  static constexpr int kJoin = kWarps * kRows * (DP + 2) * 4 + kRows * (DP + 2) * 4;
  static constexpr int kBytes = kRing > kJoin ? kRing : kJoin;
};

// NI: 32-channel groups of the head (D <= 32 NI).
template <int NI>
__global__ void __launch_bounds__(kWarps * 32, 2) attention_rows_kernel(const __grid_constant__ AttnArgs a, int splits) {
  constexpr int NC = (NI + 1) / 2;  // 64-channel groups
  constexpr int DP = 64 * NC;
  constexpr int kChunks = DP / 8;   // 16-byte groups of a row
  using M = RowsSmem<DP>;
  constexpr int ST = M::kStages;
  extern __shared__ __align__(128) uint8_t dyn[];
  auto sm_o = reinterpret_cast<float(*)[kRows][DP]>(dyn);                                     // output of each warp
  auto sm_ml = reinterpret_cast<float(*)[kRows][2]>(dyn + kWarps * kRows * DP * 4);           // its maximum (log2 units), sum
  auto cta_o = reinterpret_cast<float(*)[DP]>(dyn + kWarps * kRows * (DP + 2) * 4);           // the CTA's own, read by
  auto cta_ml = reinterpret_cast<float(*)[2]>(dyn + kWarps * kRows * (DP + 2) * 4 + kRows * DP * 4);  // the cluster

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int split = int(blockIdx.x) % splits;
  const long long unit = blockIdx.x / splits;
  const int G = a.H / a.Hkv;
  const long long R = (long long)a.Lq * G;
  const int row_blocks = int((R + kRows - 1) / kRows);
  const int rb = int(unit % row_blocks);
  const int hk = int(unit / row_blocks % a.Hkv);
  const int b = int(unit / row_blocks / a.Hkv);
  pdl_wait();
  pdl_trigger();
  const int len = a.kv_len ? max(0, min(a.Lk, a.kv_len[b])) : a.Lk;
  const uint8_t* mask = a.key_mask ? a.key_mask + b * a.mask_ld : nullptr;
  const uint16_t* kp = a.k + b * a.k_b + hk * a.k_h;
  const uint16_t* vp = a.v + b * a.v_b + hk * a.v_h;

  // The query rows' fragments.
  uint32_t q[2 * NI][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const long long r = (long long)rb * kRows + g + 8 * half;
    const uint16_t* qp = a.q + b * a.q_b + (r / G) * a.q_l + (hk * G + r % G) * a.q_h;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int d = 32 * i + 8 * t;
      const uint4 v = load16(qp + d, r < R && d < a.D);
      q[2 * i][half] = v.x, q[2 * i][2 + half] = v.y;
      q[2 * i + 1][half] = v.z, q[2 * i + 1][2 + half] = v.w;
    }
  }
  float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
  bool seen = false;  // a valid key
  float o[8 * NC][4];
#pragma unroll
  for (int j = 0; j < 8 * NC; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

  const int blocks = (len + kKeys - 1) / kKeys;
  const int stride = splits * kWarps;
  const uint32_t ring = smem_u32(dyn) + uint32_t(warp * ST * 2 * M::kBlock);
  // The keys and values of block `blk` into ring stage `stage`.  A lane copies
  // group `lane % kChunks` of every kStep-th key; the swizzle of K is the
  // lane's own then, that of V one of four.
  constexpr int kStep = 32 / kChunks;
  const int r0 = lane / kChunks, c0 = lane % kChunks;
  const bool in_head = 8 * c0 < a.D;
  const uint32_t k_at = uint32_t(r0 * DP * 2) + 16 * (c0 ^ ((r0 & 1) << 2));
  uint32_t v_at[8 / kStep];
#pragma unroll
  for (int n = 0; n < 8 / kStep; ++n) {
    const int r = r0 + n * kStep;
    v_at[n] = uint32_t(M::kBlock + r * DP * 2) + 16 * (c0 ^ (r & 6));
  }
  auto fetch = [&](int blk, int stage) {
    const uint32_t base = ring + uint32_t(stage * 2 * M::kBlock);
    const int key0 = blk * kKeys + r0;
    const uint16_t* kr = kp + (long long)key0 * a.k_l + 8 * c0;
    const uint16_t* vr = vp + (long long)key0 * a.v_l + 8 * c0;
    const long long k_step = kStep * a.k_l, v_step = kStep * a.v_l;
#pragma unroll
    for (int n = 0; n < kKeys / kStep; ++n) {
      static_assert(8 % kStep == 0 && kStep % 2 == 0, "the swizzles repeat every eight keys");
      const bool ok = in_head && key0 + n * kStep < len;
      copy16(base + k_at + n * (kStep * DP * 2), ok ? kr : kp, ok);
      copy16(base + v_at[n % (8 / kStep)] + n / (8 / kStep) * (8 * DP * 2), ok ? vr : vp, ok);
      kr += k_step;
      vr += v_step;
    }
  };
  const int first = split * kWarps + warp;
#pragma unroll
  for (int n = 0; n < ST - 1; ++n) {
    if (first + n * stride < blocks) fetch(first + n * stride, n);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  int stage = 0;
  for (int blk = first; blk < blocks; blk += stride) {
    // Keys of this thread: its score columns and its value rows are the same.
    const bool whole = !mask && (blk + 1) * kKeys <= len;
    bool ok[2][2] = {{true, true}, {true, true}};
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = blk * kKeys + nt * 8 + 2 * t + e;
          ok[nt][e] = key < len && (!mask || mask[key]);
          seen |= ok[nt][e];
        }
    } else {
      seen = true;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
    __syncwarp();  // every lane's copies are in, and its reads of the stage refilled next are done
    if (blk + (ST - 1) * stride < blocks) fetch(blk + (ST - 1) * stride, stage == 0 ? ST - 1 : stage - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const uint32_t kb = ring + uint32_t(stage * 2 * M::kBlock), vb = kb + M::kBlock;
    stage = stage == ST - 1 ? 0 : stage + 1;
    // Two sums a tile, so that four products are in flight.
    float s[2][4], s2[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      uint4 k4[2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        k4[nt] = lds16(kb + uint32_t((nt * 8 + g) * DP * 2) + 16 * ((4 * i + t) ^ ((g & 1) << 2)));
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        mma_16816(s[nt], q[2 * i][0], q[2 * i][1], q[2 * i][2], q[2 * i][3], k4[nt].x, k4[nt].y);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        mma_16816(s2[nt], q[2 * i + 1][0], q[2 * i + 1][1], q[2 * i + 1][2], q[2 * i + 1][3], k4[nt].z, k4[nt].w);
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = (s[nt][e] + s2[nt][e]) * a.scale_log2;
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!ok[nt][e & 1]) s[nt][e] = -INFINITY;
    }
    float top[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) top[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
#pragma unroll
    for (int x = 1; x <= 2; x *= 2)
#pragma unroll
      for (int h = 0; h < 2; ++h) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], x));
    // The reference follows the maximum when that has grown by more than 8 (log2
    // units): probabilities of up to 2^8 cost the fp32 sums nothing.
    if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float to = fmaxf(m[h], top[h]);
        const float f = to == -INFINITY ? 1.f : exp2_fast(m[h] - to);
        m[h] = to;
        sum[h] *= f;
#pragma unroll
        for (int j = 0; j < 8 * NC; ++j) o[j][2 * h] *= f, o[j][2 * h + 1] *= f;
      }
    }
    uint32_t hi[4], lo[4];  // A fragment of P: (row g | g + 8) x (keys 2t, 2t + 1 | + 8)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float base = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float p0 = exp2_fast(s[nt][2 * h] - base), p1 = exp2_fast(s[nt][2 * h + 1] - base);
        sum[h] += p0 + p1;
        split2(p0, p1, hi[2 * nt + h], lo[2 * nt + h]);
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      uint4 vv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 2 * t + (e & 1) + (e >> 1) * 8;
        vv[e] = lds16(vb + uint32_t(r * DP * 2) + 16 * ((8 * c + g) ^ (r & 6)));
      }
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!ok[e >> 1][e & 1]) vv[e] = make_uint4(0u, 0u, 0u, 0u);
      }
      const uint32_t* w0 = &vv[0].x;
      const uint32_t* w1 = &vv[1].x;
      const uint32_t* w2 = &vv[2].x;
      const uint32_t* w3 = &vv[3].x;
      uint32_t b0[8], b1[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
        b0[i] = __byte_perm(w0[i / 2], w1[i / 2], sel), b1[i] = __byte_perm(w2[i / 2], w3[i / 2], sel);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) mma_16816(o[8 * c + i], hi[0], hi[1], hi[2], hi[3], b0[i], b1[i]);
#pragma unroll
      for (int i = 0; i < 8; ++i) mma_16816(o[8 * c + i], lo[0], lo[1], lo[2], lo[3], b0[i], b1[i]);
    }
  }
  // ---- join, over the rings once every warp is through with its own
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  seen = __any_sync(0xffffffffu, seen);  // the keys are the same for every row
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (seen && m[h] == -INFINITY) m[h] = -FLT_MAX;
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
    if (t == 0) {
      sm_ml[warp][g + 8 * h][0] = m[h];
      sm_ml[warp][g + 8 * h][1] = sum[h];
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // channels 64 c + 8 (2t + e) + 0..7
        float4* dst = reinterpret_cast<float4*>(&sm_o[warp][g + 8 * h][64 * c + 16 * t + 8 * e]);
        dst[0] = make_float4(o[8 * c + 0][2 * h + e], o[8 * c + 1][2 * h + e], o[8 * c + 2][2 * h + e], o[8 * c + 3][2 * h + e]);
        dst[1] = make_float4(o[8 * c + 4][2 * h + e], o[8 * c + 5][2 * h + e], o[8 * c + 6][2 * h + e], o[8 * c + 7][2 * h + e]);
      }
  }
  __syncthreads();
  // The CTA's own (max, sum, output): thread = (row, part of the channels).
  {
    const int r = threadIdx.x >> 3, part = threadIdx.x & 7;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_ml[w][r][0]);
    float f[kWarps], total = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = sm_ml[w][r][0];
      f[w] = mw == -INFINITY ? 0.f : exp2_fast(mw - top);
      total = fmaf(sm_ml[w][r][1], f[w], total);
    }
    if (part == 0) cta_ml[r][0] = top, cta_ml[r][1] = total;
    for (int d = part * 2; d < DP; d += 16) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(&sm_o[w][r][d]);
        x = fmaf(v.x, f[w], x);
        y = fmaf(v.y, f[w], y);
      }
      *reinterpret_cast<float2*>(&cta_o[r][d]) = make_float2(x, y);
    }
  }
  if (splits > 1) cluster_sync();
  else __syncthreads();
  const uint32_t ml0 = smem_u32(&cta_ml[0][0]), o0 = smem_u32(&cta_o[0][0]);
  for (int i = split * (kWarps * 32) + int(threadIdx.x); i < kRows * DP / 2; i += splits * (kWarps * 32)) {
    const int r = i / (DP / 2), d = 2 * (i % (DP / 2));
    const long long row = (long long)rb * kRows + r;
    if (row >= R || d >= a.D) continue;
    float x = 0.f, y = 0.f, total = 0.f, top = -INFINITY;
    if (splits == 1) {
      top = cta_ml[r][0], total = cta_ml[r][1];
      x = cta_o[r][d], y = cta_o[r][d + 1];
    } else {
      for (int s = 0; s < splits; ++s) top = fmaxf(top, ld_cluster_f2(mapa_shared(ml0 + r * 8, s)).x);
      for (int s = 0; s < splits; ++s) {
        const float2 ml = ld_cluster_f2(mapa_shared(ml0 + r * 8, s));
        const float2 v = ld_cluster_f2(mapa_shared(o0 + (r * DP + d) * 4, s));
        const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top);
        total = fmaf(ml.y, f, total);
        x = fmaf(v.x, f, x);
        y = fmaf(v.y, f, y);
      }
    }
    const float inv = top == -INFINITY ? 0.f : 1.f / total;
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y * inv), "f"(x * inv));
    *reinterpret_cast<uint32_t*>(a.o + b * a.o_b + (row / G) * a.o_l + (hk * G + row % G) * a.o_h + d) = w;
  }
  // No CTA leaves while another may still read its shared memory.
  if (splits > 1) cluster_sync_relaxed();
}

template <int NI>
cudaError_t launch_ni(const AttnArgs& a, int splits, cudaStream_t stream) {
  constexpr int kBytes = RowsSmem<64 * ((NI + 1) / 2)>::kBytes;
  static thread_local int ready_dev = -1;  // once per device: shared memory above 48 KB, clusters above 8
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready_dev != dev) {
    if ((e = cudaFuncSetAttribute(attention_rows_kernel<NI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(attention_rows_kernel<NI>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
      return e;
    ready_dev = dev;
  }
  const long long rows = (long long)a.Lq * (a.H / a.Hkv);
  const long long units = (rows + kRows - 1) / kRows * a.Hkv * a.B;
  return launch_pdl(attention_rows_kernel<NI>, dim3(unsigned(units * splits)), dim3(kWarps * 32), kBytes, stream,
                    unsigned(splits), a, splits);
}

}  // namespace

int attention_rows_splits(long long units, long long Lk, int sms) {
  // While the CTAs fit the GPU at once (two an SM) and each warp keeps a block.
  int splits = 1;
  while (splits < 16 && units * splits * 2 <= 2 * sms && splits * 2 * kWarps <= (Lk + kKeys - 1) / kKeys) splits *= 2;
  return splits;
}

cudaError_t launch_attention_rows(const AttnArgs& a, int sms, cudaStream_t stream) {
  const long long rows = (long long)a.Lq * (a.H / a.Hkv);
  const long long units = (rows + kRows - 1) / kRows * a.Hkv * a.B;
  const int splits = attention_rows_splits(units, a.Lk, sms);
  switch ((a.D + 31) / 32) {
    case 1: return launch_ni<1>(a, splits, stream);
    case 2: return launch_ni<2>(a, splits, stream);
    case 3: return launch_ni<3>(a, splits, stream);
    case 4: return launch_ni<4>(a, splits, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace tern
