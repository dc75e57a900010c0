// rope.cu -- rotary position embedding with several axes (time, height,
// width): the (cos, sin) table of token positions, and the rotation of query
// and key heads by it.
//
// Table: pair j of axis a (d_a channels, d_a / 2 pairs, i = the pair's place
// on its axis) of token m turns by ids[m, a] * theta^(-2 i / d_a).  Far
// positions turn by thousands of radians, where one fp32 ulp of the angle is
// already visible in its cosine, so the angle is counted in quarter turns and
// reduced to [-1/2, 1/2] in 64 bits.  There the sine and cosine are their
// Taylor polynomials (degrees 11 and 12: truncation below 7e-12), rounded
// once to fp32.  A lane owns a token and its warp walks over pairs, so the
// frequency is one constant operand for the warp (a frequency per lane, read
// from the parameters, serialised 32 constant reads: 21 us for 57,677 tokens
// of 64 pairs); the block's 32 rows are turned around in shared memory so
// that stores are consecutive.
//
// Rotation: bound by HBM (each element read once, written once).  A thread
// owns 16 bytes of channels of a token (for half-split pairs 8 bytes of each
// half: the same four pairs) and walks over heads, so the table, shared by
// all heads, stays in registers.  fp32 products, one rounding to bf16.
#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"

namespace tern {

namespace {

// ------------------------------------------------------------------- table
constexpr int kTableThreads = 256;
constexpr int kTableRows = 32;  // token rows per block, one per lane

// sin(pi/2 f) / f and cos(pi/2 f): Taylor coefficients (pi/2)^k / k! with
// alternating signs.  In constant memory they are operands of the 64-bit
// multiply-adds; as literals each took two moves into registers per use.
constexpr double kH = 1.57079632679489661923, kH2 = kH * kH, kH4 = kH2 * kH2, kH6 = kH4 * kH2, kH8 = kH4 * kH4,
                 kH10 = kH6 * kH4, kH12 = kH6 * kH6;
__constant__ double kSin[6] = {kH, -kH * kH2 / 6, kH * kH4 / 120, -kH * kH6 / 5040, kH * kH8 / 362880,
                               -kH * kH10 / 39916800};
__constant__ double kCos[7] = {1.0, -kH2 / 2, kH4 / 24, -kH6 / 720, kH8 / 40320, -kH10 / 3628800, kH12 / 479001600};

// cos and sin of x * w quarter turns, each rounded once to fp32 (|x w| < 2^50).
__device__ __forceinline__ float2 cos_sin(double x, double w) {
  // Adding 1.5 * 2^52 leaves the nearest integer n (its low bits count the
  // quarter turns); the remainder x w - n, in [-1/2, 1/2], is rounded once.
  const double magic = 6755399441055744.0;
  const double u = fma(x, w, magic);
  const int q = __double2loint(u);
  const double f = fma(x, w, magic - u);
  const double z = f * f;
  const double s = f * fma(z, fma(z, fma(z, fma(z, fma(z, kSin[5], kSin[4]), kSin[3]), kSin[2]), kSin[1]), kSin[0]);
  const double c = fma(z, fma(z, fma(z, fma(z, fma(z, fma(z, kCos[6], kCos[5]), kCos[4]), kCos[3]), kCos[2]), kCos[1]), 1.0);
  const float fs = float(s), fc = float(c);
  const float cc = (q & 1) ? fs : fc, ss = (q & 1) ? fc : fs;
  // cos changes its sign for quarter turns 1 and 2, sin for 2 and 3.
  return make_float2(__uint_as_float(__float_as_uint(cc) ^ (uint32_t(q + 1) << 30 & 0x80000000u)),
                     __uint_as_float(__float_as_uint(ss) ^ (uint32_t(q) << 30 & 0x80000000u)));
}

__global__ void __launch_bounds__(kTableThreads)
    rope_table_kernel(const float* __restrict__ ids, int L, const __grid_constant__ RopeFreqs f, float2* cs) {
  extern __shared__ float2 tile[];  // [kTableRows][pairs | 1]: a column of lanes meets every bank
  pdl_wait();
  pdl_trigger();
  const int P = f.pairs, pitch = P | 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = int(blockIdx.x) * kTableRows, rows = min(kTableRows, L - m0);
  float2* const row = tile + lane * pitch;
  int end = 0;
#pragma unroll 1
  for (int a = 0; a < f.n_axes; ++a) {
    const int begin = end;
    end += f.axis_pairs[a];
    const double x = lane < rows ? double(ids[(long long)(m0 + lane) * f.n_axes + a]) : 0.0;
    for (int j = begin + warp; j < end; j += kTableThreads / 32) row[j] = cos_sin(x, f.turns[j]);
  }
  __syncthreads();
  float2* out = cs + (long long)m0 * P;
  for (int r = warp; r < rows; r += kTableThreads / 32)
    for (int j = lane; j < P; j += 32) out[r * P + j] = tile[r * pitch + j];
}

// ---------------------------------------------------------------- rotation
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// The adjacent pair (a, b) of one word turned by (c, s).
__device__ __forceinline__ uint32_t turn(uint32_t w, float c, float s) {
  const float a = lo_f(w), b = hi_f(w);
  return pack2(a * c - b * s, a * s + b * c);
}

constexpr int kBatch = 4;  // heads a thread has in flight

// threadIdx.x is the group of channels, .y the first head, .z the token row of
// the block; blockIdx.y the tensor.  The table's entries stay in registers
// while the thread walks over heads; its loads of kBatch heads are issued
// before the first store (x may be y, so the compiler cannot move them).
template <bool HALVES>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int unit = threadIdx.x;
  const unsigned m = blockIdx.x * blockDim.z + threadIdx.z;
  if (m >= unsigned(a.rows)) return;
  const unsigned b = a.L == a.rows ? 0u : m / unsigned(a.L), l = m - b * unsigned(a.L);
  const bool turned = unit < a.rot / 8;
  // First channel of this thread's 16 bytes; half-split: of 8 bytes in each half.
  const int c0 = HALVES && turned ? 4 * unit : 8 * unit;
  const int c1 = HALVES && turned ? a.rot / 2 + 4 * unit : 8 * unit + 4;
  float4 cs[2];  // (cos, sin) of four pairs
  if (turned) {
    const float4* t = reinterpret_cast<const float4*>(a.cs + ((long long)(a.cs_per_batch ? m : l) * (a.rot / 2) + 4 * unit) * 2);
    cs[0] = __ldg(t);
    cs[1] = __ldg(t + 1);
  }
  const RopeTensor& T = a.t[blockIdx.y];
  const uint16_t* const x = T.x + b * T.x_b + l * T.x_l;
  uint16_t* const y = T.y + b * T.y_b + l * T.y_l;
  for (int h0 = threadIdx.y; h0 < T.heads; h0 += kBatch * blockDim.y) {
    uint2 v[kBatch], w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * blockDim.y;
      if (h < T.heads) {
        const uint16_t* p = x + h * T.x_h;
        if constexpr (HALVES) {
          v[i] = *reinterpret_cast<const uint2*>(p + c0);
          w[i] = *reinterpret_cast<const uint2*>(p + c1);
        } else {
          const uint4 q = *reinterpret_cast<const uint4*>(p + c0);
          v[i] = make_uint2(q.x, q.y), w[i] = make_uint2(q.z, q.w);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * blockDim.y;
      if (h < T.heads) {
        uint16_t* p = y + h * T.y_h;
        uint2 r0 = v[i], r1 = w[i];
        if (turned) {
          if constexpr (HALVES) {
            const float a0 = lo_f(r0.x), a1 = hi_f(r0.x), a2 = lo_f(r0.y), a3 = hi_f(r0.y);
            const float b0 = lo_f(r1.x), b1 = hi_f(r1.x), b2 = lo_f(r1.y), b3 = hi_f(r1.y);
            r0.x = pack2(a0 * cs[0].x - b0 * cs[0].y, a1 * cs[0].z - b1 * cs[0].w);
            r0.y = pack2(a2 * cs[1].x - b2 * cs[1].y, a3 * cs[1].z - b3 * cs[1].w);
            r1.x = pack2(a0 * cs[0].y + b0 * cs[0].x, a1 * cs[0].w + b1 * cs[0].z);
            r1.y = pack2(a2 * cs[1].y + b2 * cs[1].x, a3 * cs[1].w + b3 * cs[1].z);
          } else {
            r0.x = turn(r0.x, cs[0].x, cs[0].y);
            r0.y = turn(r0.y, cs[0].z, cs[0].w);
            r1.x = turn(r1.x, cs[1].x, cs[1].y);
            r1.y = turn(r1.y, cs[1].z, cs[1].w);
          }
        }
        if constexpr (HALVES) {
          *reinterpret_cast<uint2*>(p + c0) = r0;
          *reinterpret_cast<uint2*>(p + c1) = r1;
        } else {
          *reinterpret_cast<uint4*>(p + c0) = make_uint4(r0.x, r0.y, r1.x, r1.y);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_table(const float* ids, int L, const RopeFreqs& f, float* cs, cudaStream_t stream) {
  const unsigned grid = (unsigned(L) + kTableRows - 1) / kTableRows;
  return launch_pdl(rope_table_kernel, dim3(grid), dim3(kTableThreads), kTableRows * (f.pairs | 1) * sizeof(float2), stream,
                    1, ids, L, f, reinterpret_cast<float2*>(cs));
}

cudaError_t launch_rope(const RopeArgs& a, bool halves, cudaStream_t stream) {
  int count = 0, heads = 1;
  for (int i = 0; i < kRopeTensors; ++i)
    if (a.t[i].heads > 0) count = i + 1, heads = max(heads, a.t[i].heads);
  // About 256 threads: a batch of heads for each, then further token rows.
  const int units = a.head_dim / 8, slots = 256 / units;
  const int ny = min(slots, (heads + kBatch - 1) / kBatch), nz = min(slots / ny, 64);
  // unsigned: rows may be next to 2^31
  const dim3 grid((unsigned(a.rows) + unsigned(nz) - 1) / unsigned(nz), unsigned(count)), block(units, ny, nz);
  return halves ? launch_pdl(rope_kernel<true>, grid, block, 0, stream, 1, a)
                : launch_pdl(rope_kernel<false>, grid, block, 0, stream, 1, a);
}

}  // namespace tern
