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
// codes), so a warp's load covers 512 contiguous bytes, and a warp requests kSteps of them
// before it uses any. A CTA's eight warps take the same columns of eight neighbouring rows,
// so the scales of a block (block-major) fill whole 32-byte sectors. One item a CTA: the
// CTAs of dead rows end at once and the others spread evenly.
//
// Measured: 8191 x 7168 28.0 us from bf16 rows (with the two divisions of a block in every lane 4 us
// more) and 43.0 from FP32 ones: 6.3 and 6.8 TB/s of the 2 + 1 and 4 + 1 bytes an element, part of
// which never reaches HBM, as output stays in L2 for its reader. SILU fills neither HBM nor the
// SM (25 % and 57 % in a capture, 42 % of the warps): a block's loads, its arithmetic, two special
// functions and about 20 instructions an element, and its stores follow one another. 6144 live
// of 12288 rows x 2048 take 20.7 us from HBM, 19.3 from L2, 13.7 without the arithmetic.
#include "fp8.cuh"

namespace chord {
namespace {

constexpr int kQuantWarps = 8;
constexpr int kSteps = 4;                        // warp loads in flight
constexpr int kChunk = 256 * kSteps;             // columns of a row per warp item

// Eight elements as they are in memory, and as FP32.
template <int DTYPE>
struct Raw {
  uint4 v[DTYPE == CHORD_DTYPE_BF16 ? 1 : 2];
};
__device__ __forceinline__ uint4 ldg_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
template <int DTYPE>
__device__ __forceinline__ void load8(Raw<DTYPE>& r, const void* base, int64_t at) {
  if (DTYPE == CHORD_DTYPE_BF16) {
    r.v[0] = ldg_once(static_cast<const uint16_t*>(base) + at);
  } else {
    r.v[0] = ldg_once(static_cast<const float*>(base) + at);
    r.v[DTYPE == CHORD_DTYPE_BF16 ? 0 : 1] = ldg_once(static_cast<const float*>(base) + at + 4);
  }
}
template <int DTYPE>
__device__ __forceinline__ void unpack8(const Raw<DTYPE>& r, float v[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
  if (DTYPE == CHORD_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const uint4 h = r.v[DTYPE == CHORD_DTYPE_BF16 ? 0 : 1];
    const uint32_t x[8] = {w[0], w[1], w[2], w[3], h.x, h.y, h.z, h.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x[i]);
  }
}
// The largest |x| of eight, as the bits of an FP32.
template <int DTYPE>
__device__ __forceinline__ uint32_t raw_max(const Raw<DTYPE>& r) {
  if (DTYPE == CHORD_DTYPE_BF16) {  // bf16 magnitudes compare as 16-bit integers, two at a time
    const uint32_t m = __vmaxu2(__vmaxu2(r.v[0].x & 0x7fff7fffu, r.v[0].y & 0x7fff7fffu),
                                __vmaxu2(r.v[0].z & 0x7fff7fffu, r.v[0].w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
  float v[8];
  unpack8(r, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

// Plain bf16 rows: 40 registers for 48 warps an SM (42 allow 40 warps and cost 5%); the other
// forms would spill.
template <int DTYPE, bool SILU>
__global__ void __launch_bounds__(32 * kQuantWarps, DTYPE == CHORD_DTYPE_BF16 && !SILU ? 6 : 1) fp8_quantize_kernel(const Fp8QuantArgs a) {
  grid_dep_wait();
  grid_dep_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int64_t grp = blockIdx.x / unsigned(chunks);
  const int c0 = int(blockIdx.x - grp * chunks) * kChunk;
  const int64_t row = grp * kQuantWarps + warp;
  if (row >= a.rows) return;
  if (a.masked_m) {
    const int64_t e = row / a.max_m;
    if (row - e * a.max_m >= __ldcg(a.masked_m + e)) return;
  }
  Raw<DTYPE> raw[kSteps], raw_up[SILU ? kSteps : 1];
  (void)raw_up;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int c = c0 + 256 * s + 8 * lane;
    raw[s] = Raw<DTYPE>{};
    if (SILU) raw_up[SILU ? s : 0] = Raw<DTYPE>{};
    if (c < a.K) {
      load8(raw[s], a.x, row * a.ld + c);
      if (SILU) load8(raw_up[SILU ? s : 0], a.x, row * a.ld + a.K + c);
    }
  }
  // the largest |x| of each step's block, in every lane of its half warp
  uint32_t m[kSteps];
  float act[SILU ? kSteps : 1][8];
  (void)act;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (SILU) {
      float g[8], u[8];
      unpack8(raw[s], g);
      unpack8(raw_up[SILU ? s : 0], u);
      m[s] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        act[SILU ? s : 0][i] = silu_times(g[i], u[i]);
        m[s] = max(m[s], abs_bits(act[SILU ? s : 0][i]));
      }
    } else {
      m[s] = raw_max(raw[s]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m[s] = max(m[s], __shfl_xor_sync(0xffffffffu, m[s], o));
  }
  // one division a lane: lane s of a half warp forms the scale of step s, lane 4 + s its inverse
  static_assert(kSteps == 4, "eight lanes share the divisions");
  const uint32_t mine = (lane & 2) ? ((lane & 1) ? m[3] : m[2]) : ((lane & 1) ? m[1] : m[0]);
  const float quotient = block_quotient(mine, lane & 4);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int c = c0 + 256 * s + 8 * lane;
    const float sc = __shfl_sync(0xffffffffu, quotient, (lane & 16) | s);
    const float r = __shfl_sync(0xffffffffu, quotient, (lane & 16) | 4 | s);
    if (c >= a.K) continue;
    float v[8];
    if (SILU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act[SILU ? s : 0][i];
    } else {
      unpack8(raw[s], v);
    }
    uint2 code;
    code.x = e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
    code.y = e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r);
    *reinterpret_cast<uint2*>(a.q + row * a.K + c) = code;
    if ((lane & 15) == 0) a.scales[int64_t(c / kFp8Block) * a.rows + row] = sc;
  }
}

template <int DTYPE, bool SILU>
cudaError_t launch(const Fp8QuantArgs& a, cudaStream_t stream) {
  const int64_t items = (a.rows + kQuantWarps - 1) / kQuantWarps * ((a.K + kChunk - 1) / kChunk);
  if (items >= int64_t(1) << 31) return cudaErrorInvalidValue;
  const cudaError_t err = launch_pdl(true, fp8_quantize_kernel<DTYPE, SILU>, dim3(unsigned(items)),
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
