// internal.h -- structures shared by the host API (tern_api.cu) and the
// kernels.  Not part of the public ABI.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace tern {

// One ternary linear problem as the grouped tcgen05 kernel sees it.
struct alignas(64) Problem {
  CUtensorMap tmap_x;       // x [M, K] bf16, box {64 k, TOK rows}, 128-byte swizzle
  const uint8_t* packed;    // tile-interleaved codes
  const float* scales;      // [N]
  const __nv_bfloat16* bias;  // [N] or null
  __nv_bfloat16* y;         // [M, N]
  union {
    float* ws;              // ternary_mma: split-K partials [splits][tiles][TOK][128] (splits > 1);
                            // ternary_fp8: the E4M3 row scales a [M]
    const float* rope;      // ternary_mma2: (cos, sin) per token row and channel pair [M][64][2], or null
  };
  int* counters;            // one arrival counter per output tile (splits > 1), zero at rest
  int M, N, K;
  int n_tiles, m_tiles, splits;
  int chunks_per_split;     // 64-wide k chunks per split
  int unit_begin;            // first work unit (CTA, or 2-SM tile) of this problem
  int act;                   // epilogue activation (kActNone / kActGeluTanh)
  int act_col0;              // first output column the activation applies to
  const __nv_bfloat16* residual;  // [M, N] or null: y = residual + gate * act(v)
  const __nv_bfloat16* gate;      // [N] or null (gate 1)
  int norm_col0, norm_col1;       // RMS-normalised columns (128-column groups), empty if equal
  float norm_eps;
  int ldy;                        // elements between rows of y (and of the residual), >= N
  const __nv_bfloat16* norm_weight;  // [N] or null (weight 1)
};
static_assert(sizeof(Problem) == 256, "Problem layout");

// Launches `kernel` with programmatic dependent launch allowed (see
// pdl_wait in ptx.cuh: the kernel may be scheduled while the previous one of
// the stream drains, and waits for it before touching global memory) and,
// for cluster_x > 1, a cluster of cluster_x CTAs along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              unsigned cluster_x, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

constexpr int kMaxProblems = 15;  // keeps the kernel parameter block under 4 KiB

struct Batch {
  Problem p[kMaxProblems];
  int count;
  int total_units;
  unsigned long long wait_limit_ns;
  unsigned int* status;     // per-device status word (bounded waits report here)
};
static_assert(sizeof(Batch) <= 4096, "kernel parameter block");

// Token-tile sizes (UMMA N) with a compiled kernel.
constexpr int kTokTiles[] = {32, 64, 128};

// Per-tile geometry, shared by host (launch) and device (kernel).
template <int TOK>
struct TileCfg {
  static constexpr int kCh = 128;                 // output channels per CTA (UMMA M)
  static constexpr int kBK = 64;                  // k per pipeline stage
  static constexpr int kXBytes = TOK * 128;       // TOK rows x 64 bf16, 128-byte swizzled
  static constexpr int kCBytes = kCh * 16;        // 128 rows x 16 bytes of codes
  static constexpr int kStageBytes = kXBytes + kCBytes;
  // Stage counts also size shared memory so that at most two CTAs fit on an
  // SM: two CTAs use all 512 TMEM columns.
  static constexpr int kStages = TOK <= 16 ? 20 : TOK <= 32 ? 14 : TOK <= 64 ? 8 : 5;
  static constexpr int kASlots = 4;               // decoded-weight slots in TMEM
  static constexpr int kACols = kBK / 2;          // 32-bit TMEM columns per slot (bf16x2)
  static constexpr int kDCols = TOK < 32 ? 32 : TOK;
  static constexpr int kTmemCols = (kDCols + kASlots * kACols) <= 256 ? 256 : 512;
  static constexpr int kDecWarps = TOK <= 64 ? 8 : 4;
  static constexpr int kThreads = (2 + kDecWarps) * 32;
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024;
  // Instruction descriptor, kind::f16: D fp32, A bf16, B bf16, both K-major,
  // N = TOK, M = 128.
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                     (uint32_t(TOK >> 3) << 17) | (uint32_t(128 >> 4) << 24);
  static_assert(TOK % 16 == 0 && TOK >= 16 && TOK <= 256, "UMMA N for M=128");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static_assert(3 * (kSmemBytes + 1024) > 228 * 1024, "a third CTA per SM would exceed TMEM");
};

cudaError_t launch_ternary_mma(int tok, const Batch& batch, cudaStream_t stream);
cudaError_t launch_quantize_pack(const __nv_bfloat16* W, int N, int K, float eps, uint8_t* packed,
                                 float* scales, cudaStream_t stream);
cudaError_t launch_dequantize(const uint8_t* packed, const float* scales, int N, int K,
                              __nv_bfloat16* out, cudaStream_t stream);
cudaError_t launch_wait_selftest(unsigned long long limit_ns, unsigned int* status,
                                 cudaStream_t stream);
// adaLN modulation of layer-normalised token rows (one warp per row, the row
// in registers): K % 8 == 0, K <= kAdaMaxK, 16-byte aligned rows, scale and
// shift rows mod_ld elements apart.
constexpr int kAdaMaxK = 4096;
cudaError_t launch_adaln_modulate(const __nv_bfloat16* x, int M, int K, const __nv_bfloat16* scale,
                                  const __nv_bfloat16* shift, int mod_ld, int tokens_per_row, float eps,
                                  __nv_bfloat16* out, cudaStream_t stream);
int smem_bytes_for_tok(int tok);
// Persistent tcgen05 tile kernel: tok-token tiles of 256 channels on CTA pairs
// (pair, cta_group::2; tok 256 for M > 64) or of 128 channels on single CTAs
// (!pair; tok 64 for 16 < M <= 64).  Problems use n_tiles = N / (256 or 128),
// m_tiles = ceil(M / tok), splits = 1 and a 3-D x tensor map {64 k, M,
// K / 64} whose box is {64, tok / 2 or tok rows, x_chunks_2sm(tok) chunks}
// (the 64-k chunks of one pipeline stage); ctas_or_pairs work units run at
// once.
cudaError_t launch_ternary_mma2(int tok, bool pair, const Batch& batch, int ctas_or_pairs, cudaStream_t stream);
int max_active_clusters_2sm();
int x_chunks_2sm(int tok);
// Small-M kernel (M <= 8 nt tokens, nt in {1, 2}), persistent over work
// units (problem, 128-channel slab): grid (splits, ctas) with clusters of
// `splits` CTAs along k (splits > 1 needs ctas == total_units); problems use
// n_tiles = N / 128 slabs, unit_begin = first slab in the launch,
// chunks_per_split 64-k chunks per CTA and a 3-D x tensor map {64 k, M,
// K / 64} whose box is {64, min(M, 8 nt), 16 (nt = 1) or 8 chunks}.
cudaError_t launch_ternary_gemv(int nt, const Batch& batch, int splits, int ctas, cudaStream_t stream);
// FP8 (E4M3) activations: per-token absmax quantisation of x (one warp per
// row, k interleaved inside 16-element groups), and the CTA-pair tile kernel
// with kind::f8f6f4 MMAs (one problem: N % 256 == 0, tmap_x = the 2-D E4M3 map
// {K, M} with box {128, 128}, ws = the per-token scales).
cudaError_t launch_quantize_act_e4m3(const __nv_bfloat16* x, int M, int K, uint8_t* xq, float* a,
                                     cudaStream_t stream);
cudaError_t launch_ternary_fp8(const Batch& batch, int pairs, cudaStream_t stream);

// Rotary table: the frequency of every channel pair and the pairs of every axis.
constexpr int kRopeMaxPairs = 128;
struct RopeFreqs {
  double turns[kRopeMaxPairs];  // theta^(-2 i / d_a), in quarter turns
  int axis_pairs[4];
  int pairs, n_axes;
};
// cs [L][pairs][2] from ids [L][n_axes].
cudaError_t launch_rope_table(const float* ids, int L, const RopeFreqs& f, float* cs, cudaStream_t stream);

// Rotation of up to kRopeTensors head tensors of the same tokens.
constexpr int kRopeTensors = 4;
struct RopeTensor {
  const uint16_t* x;
  uint16_t* y;
  long long x_b, x_l, x_h, y_b, y_l, y_h;  // elements between batch entries, tokens, heads
  int heads;
};
struct RopeArgs {
  RopeTensor t[kRopeTensors];  // unused ones have no heads
  const float* cs;
  int rows, L;        // rows = batch * L
  int head_dim, rot;
  int cs_per_batch;   // the table has a row per (batch entry, token), not per token
};
cudaError_t launch_rope(const RopeArgs& a, bool halves, cudaStream_t stream);

// Gated residual update with the norms around it; rows of K elements, K % 8 == 0.
constexpr int kNormNone = 0, kNormRms = 1, kNormLayer = 2;
constexpr int kResNormMaxK = 16384;
struct ResNormArgs {
  const uint16_t *x, *o;
  uint16_t *x_out, *h;  // h may be null
  const uint16_t *gate, *scale, *shift, *post_weight, *pre_weight;  // each may be null (scale and shift together)
  long long M, ld_x, ld_o, ld_xo, ld_h, mod_ld, tokens_per_row;
  int K, post, pre, gate_tanh;
  float post_eps, pre_eps, residual_scale;
};
cudaError_t launch_gated_residual_norm(const ResNormArgs& a, int sms, cudaStream_t stream);

// Attention of q [B, Lq, H, D] to k, v [B, Lk, Hkv, D] (strides in elements).
constexpr int kAttnMaxD = 128;
struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  long long q_b, q_l, q_h, k_b, k_l, k_h, v_b, v_l, v_h, o_b, o_l, o_h;
  const int* kv_len;        // [B] or null
  const uint8_t* key_mask;  // [B] rows mask_ld apart, or null
  long long mask_ld;
  int B, Lq, Lk, H, Hkv, D;
  float scale_log2;         // softmax scale * log2(e)
};
// Division of u < 2^31 by d: u * ceil(2^(31 + l) / d) >> (31 + l), l =
// ceil(log2 d), is exact since the multiplier is off by less than 2^l / d units;
// mul = 0 stands for d = 1.
struct DivBy {
  unsigned mul, shift;
};
inline DivBy div_by(unsigned d) {
  unsigned l = 0;
  while (l < 31 && (1u << l) < d) ++l;
  if (l == 0) return {0u, 0u};
  const unsigned long long s = 1ull << (31 + l);
  return {unsigned((s + d - 1) / d), l - 1};
}
// The same with the tensor maps {D, L, H, B} (box {64, 128, 1, 1}, 128-byte
// swizzle) that the tile kernel loads through; q_h ... are 0 for a dimension
// that the map has once (a broadcast), else 1.
struct alignas(64) AttnTileArgs {
  CUtensorMap tq, tk, tv;
  AttnArgs a;
  int q_b, q_h, k_b, k_h, v_b, v_h;
  int pairs;  // of 128-row query tiles, per head
  int units;  // pairs * B * H
  int ctas;   // resident at once
  int splits;  // CTAs (a cluster) that share the keys of a unit: 1, or 2 to 8 where all units are resident at once
  int o_sectors;  // o's rows are made of whole 32-byte sectors
  DivBy by_pairs, by_heads, by_group;  // pairs, H, H / Hkv
  unsigned long long wait_limit_ns;
  unsigned int* status;
};
cudaError_t launch_attention_tile(const AttnTileArgs& t, cudaStream_t stream);
// CTAs that share the keys of one unit (16 query rows of a key-value head) in the row kernel.
int attention_rows_splits(long long units, long long Lk, int sms);
// One read of k and v for up to 16 packed query rows; see attention_rows.cu.
cudaError_t launch_attention_rows(const AttnArgs& a, int sms, cudaStream_t stream);

}  // namespace tern
