// fp8_stream.cu -- FP8 block-128 products for few rows: the weights stream through once.
//
// out[m, n] = sum_kb xs[kb, m] * ws[n/128, kb] * (xq[m, kb] . w[n, kb])
//
// With a handful of rows the product reads N*K weight bytes for 2*N*K*rows operations, so
// HBM bounds it. A CTA owns 16 weight rows of one unit (up to 8, 16 or 32 activation rows);
// its eight warps share out the 128-wide k blocks, so a CTA streams 8 x 2 KiB at a time.
// Weights go straight from global memory to mma.m16n8k32 fragments (weight rows in the M
// slot, activation rows in N): a dot product does not care in which order its k are
// numbered, so lane (g, t) takes the 16 contiguous bytes at 16t of each 64-byte half of its
// rows, for weights and activations alike, and every load is a full 16 bytes.
// The four products of a block start from zero, and their sum joins the FP32 accumulator
// through one fused multiply-add with xs * ws. The warps' accumulators meet in shared
// memory and are added in warp order.
#include "fp8.cuh"

namespace chord {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;  // weight rows of a CTA item

__device__ __forceinline__ void mma_e4m3_16832(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int NT>
struct Frag {
  uint4 a[2][2];   // [row g, g + 8][64-byte half]
  uint4 b[NT][2];  // [activation rows 8 nt + g][half]
  float s[NT][2];  // scales of activation rows 8 nt + 2t, + 1, times the weight scale
};

template <int NT>
__global__ void __launch_bounds__(32 * kWarps) fp8_stream_kernel(const Fp8Args p) {
  constexpr int TC = 8 * NT;
  __shared__ float red[kWarps][TC][kRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int KB = fp8_blocks(p.K), NB = fp8_blocks(p.N);
  const int tiles = (p.N + kRows - 1) / kRows;
  const int64_t units = p.layout == kFp8Dense ? (p.rows + TC - 1) / TC : p.ntp[0] / TC;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  for (int64_t item = blockIdx.x; item < units * tiles; item += gridDim.x) {
    const int64_t u = item / tiles;
    const int n0 = int(item - u * tiles) * kRows;
    const int e = p.layout == kFp8Dense ? 0 : __ldg(p.expert_ids + u);
    auto row_of = [&](int j) -> int64_t {  // activation row of the unit's position j, or -1
      if (p.layout == kFp8Dense) return u * TC + j < p.rows ? u * TC + j : -1;
      return __ldg(p.sorted_ids + u * TC + j);
    };
    int64_t rb[NT], rs[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      rb[i] = row_of(8 * i + g);
      rs[i][0] = row_of(8 * i + 2 * t);
      rs[i][1] = row_of(8 * i + 2 * t + 1);
    }
    // rows past N repeat the last one; they are not stored
    const uint8_t* w0 = p.w + (int64_t(e) * p.N + min(n0 + g, p.N - 1)) * p.K;
    const uint8_t* w1 = p.w + (int64_t(e) * p.N + min(n0 + g + 8, p.N - 1)) * p.K;
    const float* ws = p.ws + (int64_t(e) * NB + n0 / kFp8Block) * KB;

    auto load = [&](int kb, Frag<NT>& f) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kb * kFp8Block + 64 * h + 16 * t;  // K % 16 == 0: a vector is all in or all out
        const bool in = k < p.K;
        f.a[0][h] = in ? ldg_stream(w0 + k) : zero;
        f.a[1][h] = in ? ldg_stream(w1 + k) : zero;
#pragma unroll
        for (int i = 0; i < NT; ++i)
          f.b[i][h] = in && rb[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.xq + rb[i] * p.K + k)) : zero;
      }
      const float sw = __ldg(ws + kb);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) f.s[i][j] = rs[i][j] >= 0 ? __ldg(p.xs + kb * p.rows + rs[i][j]) * sw : 0.f;
    };

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    Frag<NT> cur, nxt;
    if (warp < KB) load(warp, cur);
    for (int kb = warp; kb < KB; kb += kWarps) {
      if (kb + kWarps < KB) load(kb + kWarps, nxt);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_e4m3_16832(c, cur.a[0][h].x, cur.a[1][h].x, cur.a[0][h].y, cur.a[1][h].y, cur.b[i][h].x, cur.b[i][h].y);
          mma_e4m3_16832(c, cur.a[0][h].z, cur.a[1][h].z, cur.a[0][h].w, cur.a[1][h].w, cur.b[i][h].z, cur.b[i][h].w);
        }
        acc[i][0] = fmaf(c[0], cur.s[i][0], acc[i][0]);
        acc[i][1] = fmaf(c[1], cur.s[i][1], acc[i][1]);
        acc[i][2] = fmaf(c[2], cur.s[i][0], acc[i][2]);
        acc[i][3] = fmaf(c[3], cur.s[i][1], acc[i][3]);
      }
      cur = nxt;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[warp][8 * i + 2 * t + (j & 1)][g + 8 * (j >> 1)] = acc[i][j];
    __syncthreads();
    for (int i = threadIdx.x; i < TC * kRows; i += 32 * kWarps) {
      const int j = i / kRows, r = i % kRows, n = n0 + r;
      const int64_t row = row_of(j);
      if (row < 0 || n >= p.N) continue;
      float s = red[0][j][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) s += red[w][j][r];
      if (p.out_f32) static_cast<float*>(p.out)[row * p.N + n] = s;
      else static_cast<uint16_t*>(p.out)[row * p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    }
    __syncthreads();  // red is rewritten by the next item
  }
}

template <int NT>
cudaError_t launch(const Fp8Args& a, int64_t items, cudaStream_t stream) {
  const int64_t most = int64_t(a.num_sms) * 4;
  fp8_stream_kernel<NT><<<unsigned(items < most ? items : most), 32 * kWarps, 0, stream>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_stream(const Fp8Args& a, cudaStream_t stream) {
  // upper bound of the items (the grouped unit count is on the device)
  const int64_t units = (a.rows + a.bm - 1) / a.bm + (a.layout == kFp8Dense ? 0 : a.E);
  const int64_t items = units * ((a.N + kRows - 1) / kRows);
  if (a.bm == 8) return launch<1>(a, items, stream);
  if (a.bm == 16) return launch<2>(a, items, stream);
  return launch<4>(a, items, stream);
}

}  // namespace chord
