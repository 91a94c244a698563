// fp8_quant.cu -- activations to E4M3 with one FP32 scale per 128 columns of a row.
//
//   amax = max(max |x|, 2^-100);  s = amax / 448;  q = e4m3(x * (448 / amax))
//
// each operation rounded to FP32 (the floor keeps 448 / amax finite; both quotients are
// IEEE divisions, one of each per block, so the codes are a function of the inputs alone).
// With SILU, x = silu(gate) * up from [gate | up] rows, in FP32.
//
// Bound: bytes. A bf16 element is 2 (SILU: 4) read and 1 written; the scale adds 4 / 128.
// 16 lanes hold a block (8 elements each: one 16-byte load of bf16, one 8-byte store of
// codes), so a warp's load covers 512 contiguous bytes, and a warp takes kSteps of them at
// once to keep loads in flight. A CTA's eight warps take the same columns of eight
// neighbouring rows, so the scales of a block (block-major) fill whole 32-byte sectors.
#include "fp8.cuh"

namespace chord {
namespace {

constexpr int kQuantWarps = 8;
constexpr int kSteps = 4;                        // warp loads in flight
constexpr int kChunk = 256 * kSteps;             // columns of a row per warp item

__device__ __forceinline__ void load8(const void* base, int dtype, int64_t at, float v[8]) {
  if (dtype == CHORD_DTYPE_BF16) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

template <int DTYPE, bool SILU>
__global__ void __launch_bounds__(32 * kQuantWarps) fp8_quantize_kernel(const Fp8QuantArgs a) {
  grid_dep_wait();
  grid_dep_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int64_t groups = (a.rows + kQuantWarps - 1) / kQuantWarps;
  for (int64_t item = blockIdx.x; item < groups * chunks; item += gridDim.x) {
    const int64_t grp = item / chunks;
    const int c0 = int(item - grp * chunks) * kChunk;
    const int64_t row = grp * kQuantWarps + warp;
    if (row >= a.rows) continue;
    if (a.masked_m) {
      const int64_t e = row / a.max_m;
      if (row - e * a.max_m >= __ldg(a.masked_m + e)) continue;
    }
    float v[kSteps][8], up[SILU ? kSteps : 1][8];
    (void)up;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = c0 + 256 * s + 8 * lane;
      if (c < a.K) {
        load8(a.x, DTYPE, row * a.ld + c, v[s]);
        if (SILU) load8(a.x, DTYPE, row * a.ld + a.K + c, up[SILU ? s : 0]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[s][i] = 0.f;
        if (SILU)
#pragma unroll
          for (int i = 0; i < 8; ++i) up[SILU ? s : 0][i] = 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = c0 + 256 * s + 8 * lane;
      if (c0 + 256 * s >= a.K) break;
      // the largest |x| by its bits: a NaN's are above infinity's, infinity's above the rest
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (SILU) v[s][i] = silu_times(v[s][i], up[SILU ? s : 0][i]);
        m = max(m, abs_bits(v[s][i]));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      float scale, r;
      block_scale(m, &scale, &r);
      if (c < a.K) {
        uint2 code;
        code.x = e4m3x4(v[s][0] * r, v[s][1] * r, v[s][2] * r, v[s][3] * r);
        code.y = e4m3x4(v[s][4] * r, v[s][5] * r, v[s][6] * r, v[s][7] * r);
        *reinterpret_cast<uint2*>(a.q + row * a.K + c) = code;
        if ((lane & 15) == 0) a.scales[int64_t(c / kFp8Block) * a.rows + row] = scale;
      }
    }
  }
}

template <int DTYPE, bool SILU>
cudaError_t launch(const Fp8QuantArgs& a, cudaStream_t stream) {
  const int64_t items = (a.rows + kQuantWarps - 1) / kQuantWarps * ((a.K + kChunk - 1) / kChunk);
  const int64_t most = int64_t(a.num_sms) * 8;
  const cudaError_t err = launch_pdl(true, fp8_quantize_kernel<DTYPE, SILU>, dim3(unsigned(items < most ? items : most)),
                                     dim3(32 * kQuantWarps), 0, stream, a);
  count_launches(1);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, cudaStream_t stream) {
  if (a.dtype == CHORD_DTYPE_BF16)
    return a.silu ? launch<CHORD_DTYPE_BF16, true>(a, stream) : launch<CHORD_DTYPE_BF16, false>(a, stream);
  return a.silu ? launch<CHORD_DTYPE_F32, true>(a, stream) : launch<CHORD_DTYPE_F32, false>(a, stream);
}

}  // namespace chord
