// fp8.cuh -- what the FP8 block-128 kernels and their entry points share.
#pragma once

#include "chord_internal.cuh"

namespace chord {

constexpr int kFp8Block = 128;  // elements under one scale
constexpr float kFp8Max = 448.f;

__host__ __device__ inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// Workspace of the products: the zero-once header, then the unit lists of the grouped
// layouts (units of 16 to 256 rows, written by the routing pass).
struct Fp8Workspace {
  int64_t max_positions, ntp_offset, expert_ids_offset, block_row0_offset, sorted_ids_offset, total;
};
Fp8Workspace fp8_workspace(int64_t rows, int E);

enum Fp8Layout { kFp8Dense = 0, kFp8Contiguous = 1, kFp8Masked = 2 };

struct Fp8Args {
  const uint8_t* xq;  // e4m3 [rows, K]
  const float* xs;    // [fp8_blocks(K), rows]
  const uint8_t* w;   // e4m3 [E, N, K]
  const float* ws;    // [E, fp8_blocks(N), fp8_blocks(K)]
  void* out;          // [rows, N] bf16, or FP32 if out_f32
  int64_t rows;
  int K, N, E, layout;
  int out_f32;
  // grouped layouts: units of bm rows (the routing pass's lists); dense: null
  const int32_t* sorted_ids;  // row of each position, -1 where it belongs to no expert
  const int32_t* expert_ids;  // expert of each unit
  const int32_t* block_row0;  // row of each unit's first position
  const int32_t* ntp;         // units * bm
  int bm;
  uint32_t* status;
  int num_sms;
  float* out_scales;  // gate_up: scales of the codes in `out`
};

struct Fp8QuantArgs {
  const void* x;
  int dtype;  // CHORD_DTYPE_F32 or CHORD_DTYPE_BF16
  int64_t ld, rows;
  int K;      // columns of the codes
  int silu;   // x holds [gate | up], 2K columns
  const int32_t* masked_m;  // or null
  int64_t max_m;
  uint8_t* q;
  float* scales;
};

// ---- quantisation of a block (used where rows are quantised and where a product ends in it)

// Two FP32 to two E4M3 codes, nearest even, saturating; NaN stays NaN. lo is the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// The scale of a block (or its inverse) from the bits of its largest |x| (as integers a NaN is
// above infinity, infinity above the rest; both give a NaN scale).
__device__ __forceinline__ float block_quotient(uint32_t amax_bits, bool inverse) {
  const float amax = fmaxf(__uint_as_float(amax_bits), 0x1p-100f);
  const float q = __fdiv_rn(inverse ? kFp8Max : amax, inverse ? amax : kFp8Max);
  return amax_bits < 0x7f800000u ? q : __uint_as_float(0x7fffffffu);
}
__device__ __forceinline__ void block_scale(uint32_t amax_bits, float* scale, float* inverse) {
  *scale = block_quotient(amax_bits, false);
  *inverse = block_quotient(amax_bits, true);
}
// silu(g) * u. The reciprocal of d = 1 + exp(-g) is the hardware's approximation and one step
// of Newton's iteration, half the instructions of a division; below -80, where exp(-g) nears
// the end of the range, 1/d is exp(g) to FP32.
__device__ __forceinline__ float silu_times(float g, float u) {
  if (g < -80.f) return g * expf(g) * u;
  const float d = 1.f + expf(-g);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  r = fmaf(r, fmaf(-d, r, 1.f), r);
  return g * r * u;
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, cudaStream_t stream);
// a.bm in {16, 32, 64}; `split` CTAs (a power of two up to 8, at most the k blocks) share an item.
constexpr int kFp8StreamCtas = 2;  // resident per SM
cudaError_t launch_fp8_stream(const Fp8Args& a, int split, cudaStream_t stream);
// Dense gate_up as launch_fp8_tile_gate_up; clusters of 2 x split CTAs, split <= 4.
cudaError_t launch_fp8_stream_gate_up(const Fp8Args& a, int split, cudaStream_t stream);
// a.bm = 128: single CTAs with tiles of 128 x 128; 256: CTA pairs, 256 x 256.
cudaError_t launch_fp8_tile(const Fp8Args& a, cudaStream_t stream);
// Dense, w = [gate; up] with a.N = 2 I: SiLU(gate) * up quantised to q [rows, I], scales [I/128, rows].
cudaError_t launch_fp8_tile_gate_up(const Fp8Args& a, cudaStream_t stream);

}  // namespace chord
