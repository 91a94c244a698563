// fp8_stream.cu -- FP8 block-128 products for few rows of an expert: the weights stream
// through once.
//
//   out[m, n] = sum_kb s[m, kb] * P_kb[n, m],   P_kb = w[n, kb] . xq[m, kb],
//   s = xs[kb, m] * ws[n/128, kb]
//
// With few rows the product reads N*K weight bytes for 2*N*K*rows operations, so HBM bounds
// it. The operands are swapped against fp8_tile.cu: a tile of 128 weight rows (one block of
// the weight scales) is the M side of the MMA and TN = 16, 32 or 64 activation rows the N side,
// so a weight byte is fetched once for all of them and the MMA's size follows the rows.
//
//   warp 0      TMA producer: per k block 128 weight rows and TN activation rows, 128 bytes
//               wide (128-byte swizzle), into a ring of stages.
//   warp 1      MMA issuer: four tcgen05.mma (M = 128, N = TN, K = 32) into one of several
//               tensor-memory buffers.
//   warp 2      scales: s of eight k blocks at a time into a ring in shared memory.
//   warps 4..7  promotion: one weight row per thread, TN columns; FP32 accumulation in
//               registers, s read as broadcast vectors.
//
// An item is (unit of TN rows, weight tile). With many items a CTA runs them one after
// another. With few (one token against a 4096 x 7168 matrix has 32) a cluster of S CTAs
// shares an item, each taking 1/S of the k blocks; their FP32 sums meet through distributed
// shared memory, are added in rank order, and each CTA writes its share of the rows. For
// gate_up a cluster holds the gate and the up tile of the same columns and its last step is
// SiLU(gate) * up and the FP8 quantisation.
//
// Measured: 384 rows over 46 of 48 experts of 4096 x 7168 (1.35 GB of weights) 207 to 212 us, 6.4
// TB/s; one row against 4096 x 7168 7.4 us from L2, of which about 4 are start and reduction, and
// 9.6 from HBM.
//
// All waits are bounded; on a timeout the CTA raises CHORD_DEV_TIMEOUT, writes nothing more (nor
// do the others of its cluster), waits (bounded) for what it has in flight and returns.
#include "fp8_tc.cuh"

namespace chord {
namespace {

constexpr int kWRows = 128;                     // weight rows of a tile
constexpr int kWBytes = kWRows * kFp8Block;
constexpr int kThreads = 256;
constexpr int kFirstPromote = 4, kPromote = 4;  // warps
constexpr int kMaxSplit = 8;                    // CTAs of a cluster (16, an opt-in, took 8 us longer)
constexpr int kGroupKb = 8;                     // k blocks of a scale group

template <int TN>
struct StreamCfg {
  // two CTAs share an SM (half the shared memory and tensor memory, 128 registers a thread),
  // so one's start and end overlap the other's streaming
  static constexpr int kCtas = kFp8StreamCtas;
  static constexpr int kStageBytes = kWBytes + TN * kFp8Block;
  static constexpr int kGroups = 3;                               // scale groups in the ring
  static constexpr int kScaleBytes = kGroups * kGroupKb * TN * 4;
  static constexpr int kFixed = 1024 + kScaleBytes;
  static constexpr int kBudget = 113 * 1024 - 1024;  // less alignment slack
  static constexpr int kStages = (kBudget - kFixed) / kStageBytes;
  static constexpr int kSmem = 1024 + (kFixed + 1023) / 1024 * 1024 + kStages * kStageBytes;
  static constexpr int kBufs = 4;
  static constexpr int kCols = kBufs * TN;                        // 64, 128 or 256
  static constexpr int kChunk = 16;
};

struct StreamMaps {
  CUtensorMap x, w;
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// kRowsOut: rows of the output. kGateUpOut: w = [gate; up] (N = 2 I); a cluster of 2 x split CTAs
// holds a gate tile (the first half of its ranks) and the up tile of the same columns, and
// ends in SiLU(gate) * up quantised to FP8: a row's block of 128 columns is one warp's work.
enum StreamOut { kRowsOut = 0, kGateUpOut = 1 };

template <int TN, int OUT>
__global__ void __launch_bounds__(kThreads, StreamCfg<TN>::kCtas)
    fp8_stream_kernel(const __grid_constant__ StreamMaps maps, const Fp8Args p, int split) {
  using Cfg = StreamCfg<TN>;
  constexpr int S = Cfg::kStages, B = Cfg::kBufs, W = Cfg::kChunk;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);  // [S]
  uint64_t* done = full + S;                           // [S] stage multiplied: it may be refilled, its
                                                       // product read
  uint64_t* acc_empty = done + S;                      // [B]
  uint64_t* sc_full = acc_empty + B;                   // [kGroups]
  uint64_t* sc_empty = sc_full + Cfg::kGroups;         // [kGroups]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_empty + Cfg::kGroups);
  float* scales = reinterpret_cast<float*>(smem + 1024);  // [kGroups][kGroupKb][TN]
  uint8_t* ring = smem + (Cfg::kFixed + 1023) / 1024 * 1024;
  float* partial = reinterpret_cast<float*>(ring);        // [TN][128], once the ring is spent
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&done[s], 1);
    }
    for (int b = 0; b < B; ++b) mbar_init(&acc_empty[b], kPromote);
    for (int g = 0; g < Cfg::kGroups; ++g) {
      mbar_init(&sc_full[g], 32);
      mbar_init(&sc_empty[g], kPromote);
    }
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc<1>(tmem_slot, Cfg::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  volatile int* abort_v = &abort_flag;
  grid_dep_wait();
  grid_dep_trigger();

  const int ctas = OUT == kGateUpOut ? 2 * split : split;  // of a cluster
  const int rank = ctas > 1 ? int(cluster_rank()) : 0;
  const int half = rank / split;                           // kGateUpOut: 1 for the up tile
  const int KB = fp8_blocks(p.K), NB = fp8_blocks(p.N);    // NB: tiles, and row blocks of the weight scales
  const int NT = OUT == kGateUpOut ? NB / 2 : NB;          // items of a unit
  const int kb_begin = (rank - half * split) * KB / split, kb_end = (rank - half * split + 1) * KB / split;
  const int units = p.layout == kFp8Dense ? int((p.rows + TN - 1) / TN) : p.ntp[0] / TN;
  const int items = units * NT;
  const int first = ctas > 1 ? int(cluster_id_x()) : int(blockIdx.x);
  const int step = ctas > 1 ? int(num_clusters_x()) : int(gridDim.x);  // a grid of clusters covers all items
  auto unit_row0 = [&](int u) { return p.layout == kFp8Dense ? u * TN : __ldcg(p.block_row0 + u); };
  auto unit_expert = [&](int u) { return p.layout == kFp8Dense ? 0 : __ldcg(p.expert_ids + u); };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t fill = 0;
      bool ok = true;
      for (int i = first; i < items && ok; i += step) {
        const int u = i / NT, row = unit_row0(u), wrow = unit_expert(u) * p.N + (half * NT + i - u * NT) * kWRows;
        for (int kb = kb_begin; kb < kb_end; ++kb, ++fill) {
          const uint32_t s = fill % S;
          if (fill >= S && !mbar_wait(&done[s], ((fill / S) - 1) & 1, abort_v, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
          const uint32_t st = smem_u32(ring + s * Cfg::kStageBytes);
          tma_2d<1>(st, &maps.w, kb * kFp8Block, wrow, smem_u32(&full[s]));
          tma_2d<1>(st + kWBytes, &maps.x, kb * kFp8Block, row, smem_u32(&full[s]));
        }
      }
      int dummy = 0;  // the last copies have landed before the CTA ends
      for (uint32_t f = fill > S ? fill - S : 0; f < fill; ++f) mbar_wait(&full[f % S], (f / S) & 1, &dummy, p.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(kWRows, TN);
      uint32_t it = 0;
      bool ok = true;
      for (int i = first; i < items && ok; i += step) {
        for (int kb = kb_begin; kb < kb_end; ++kb, ++it) {
          const uint32_t s = it % S, b = it % B;
          if ((it >= B && !mbar_wait(&acc_empty[b], ((it / B) - 1) & 1, abort_v, p.status)) ||
              !mbar_wait(&full[s], (it / S) & 1, abort_v, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(ring + s * Cfg::kStageBytes);
          const uint64_t ad = sw128_kmajor_desc(st), bd = sw128_kmajor_desc(st + kWBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_e4m3<1>(tmem + b * TN, ad + 2 * k, bd + 2 * k, idesc, k > 0);
          commit<1>(&done[s]);
        }
      }
      if (it > 0) {  // no MMA writes tensor memory once it is freed
        int dummy = 0;
        mbar_wait(&done[(it - 1) % S], ((it - 1) / S) & 1, &dummy, p.status);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    uint32_t grp = 0;
    bool ok = true;
    for (int i = first; i < items && ok; i += step) {
      const int u = i / NT, nb = half * NT + i - u * NT;
      const int64_t row0 = unit_row0(u);
      const float* ws = p.ws + (int64_t(unit_expert(u)) * NB + nb) * KB;
      for (int kb0 = kb_begin; kb0 < kb_end; kb0 += kGroupKb, ++grp) {
        const uint32_t g = grp % Cfg::kGroups;
        constexpr int PER = kGroupKb * TN / 32;
        float v[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int at = 32 * j + lane, kb = kb0 + at / TN;
          const int64_t row = row0 + at % TN;
          // rows and blocks that do not exist are never used
          v[j] = kb < kb_end && row < p.rows ? __ldcg(p.xs + kb * p.rows + row) * __ldcg(ws + kb) : 0.f;
        }
        if (grp >= Cfg::kGroups && !mbar_wait_warp(&sc_empty[g], ((grp / Cfg::kGroups) - 1) & 1, abort_v, p.status)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) scales[g * kGroupKb * TN + 32 * j + lane] = v[j];
        mbar_arrive(&sc_full[g]);
      }
    }
  } else if (warp >= kFirstPromote) {
    const int q = warp & 3;  // the tensor-memory lanes this warp may read
    const int r = q * 32 + lane;
    const uint32_t src = tmem + (uint32_t(q * 32) << 16);
    uint32_t it = 0, grp = 0;
    bool ok = true;
    for (int i = first; i < items && ok; i += step) {
      const int u = i / NT, n = (i - u * NT) * kWRows + r;
      uint64_t sum[TN / 2];  // columns 2j, 2j + 1
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) sum[j] = 0;
      for (int kb = kb_begin; kb < kb_end; ++kb, ++it) {
        const uint32_t g = grp % Cfg::kGroups;
        const int in_group = (kb - kb_begin) % kGroupKb;
        if (in_group == 0) ok = mbar_wait_warp(&sc_full[g], (grp / Cfg::kGroups) & 1, abort_v, p.status);
        const uint32_t b = it % B;
        ok = ok && mbar_wait_warp(&done[it % S], (it / S) & 1, abort_v, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sc = smem_u32(scales + (g * kGroupKb + in_group) * TN);
        uint32_t v[2][W];
        tmem_ld_async(src + b * TN, v[0]);
#pragma unroll
        for (int c = 0; c < TN / W; ++c) {
          tmem_wait_ld(v[c & 1]);
          if (c + 1 < TN / W) {
            tmem_ld_async(src + b * TN + W * (c + 1), v[(c + 1) & 1]);
          } else {  // the buffer is read: hand it back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
          }
#pragma unroll
          for (int j = 0; j < W; j += 4) {
            const uint4 s4 = lds128(sc + (W * c + j) * 4);
            fma2(sum[(W * c + j) / 2], v[c & 1][j], v[c & 1][j + 1], (uint64_t(s4.y) << 32) | s4.x);
            fma2(sum[(W * c + j) / 2 + 1], v[c & 1][j + 2], v[c & 1][j + 3], (uint64_t(s4.w) << 32) | s4.z);
          }
        }
        if (in_group == kGroupKb - 1 || kb == kb_end - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_empty[g]);
          ++grp;
        }
      }
      if (!ok) break;
      if (ctas > 1) {
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) {
          float lo, hi;
          unpack2(sum[j], lo, hi);
          partial[(2 * j) * kWRows + r] = lo;
          partial[(2 * j + 1) * kWRows + r] = hi;
        }
        continue;
      }
      // a row of the output at a time: 32 neighbouring columns a warp
      const int row0 = unit_row0(u);
#pragma unroll
      for (int j0 = 0; j0 < TN; j0 += 32) {
        const int j = j0 + lane;
        const bool mine = j < TN && (p.layout == kFp8Dense ? row0 + j < p.rows : __ldcg(p.sorted_ids + u * TN + j) >= 0);
        const uint32_t live = __ballot_sync(0xffffffffu, mine);
        if (n >= p.N) continue;
#pragma unroll
        for (int k = 0; k < 32 && j0 + k < TN; ++k) {
          if (!((live >> k) & 1u)) continue;
          float lo, hi;
          unpack2(sum[(j0 + k) / 2], lo, hi);
          const float x = (k & 1) ? hi : lo;
          const int64_t at = int64_t(row0 + j0 + k) * p.N + n;
          if (p.out_f32) static_cast<float*>(p.out)[at] = x;
          else static_cast<uint16_t*>(p.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (ctas > 1) {
    // without one CTA's sums there is no result: where one gave up, none of its cluster writes
    if (abort_flag && int(threadIdx.x) < ctas) st_cluster_u32(cluster_addr(&abort_flag, threadIdx.x), 1u);
    cluster_sync_all();  // every CTA's sums are in its shared memory, every flag is known
    const int j_begin = rank * TN / ctas, j_end = (rank + 1) * TN / ctas;
    if (OUT == kGateUpOut && first < items && !abort_flag) {
      // a row's 128 columns a warp, four a lane; every CTA's share requested before any is added
      const int u = first / NT, nt = first - u * NT, row0 = unit_row0(u), I = p.N / 2;
      for (int j = j_begin + warp; j < j_end; j += kThreads / 32) {
        const int64_t row = row0 + j;
        if (row >= p.rows) break;
        const float* mine = partial + j * kWRows + 4 * lane;
        float4 part[kMaxSplit];
#pragma unroll
        for (int c = 0; c < kMaxSplit; ++c)
          if (c < ctas) part[c] = ld_cluster4(cluster_addr(mine, c));
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f), x = g;
#pragma unroll
        for (int c = 0; c < kMaxSplit; ++c) {
          if (c < split) g.x += part[c].x, g.y += part[c].y, g.z += part[c].z, g.w += part[c].w;
          else if (c < ctas) x.x += part[c].x, x.y += part[c].y, x.z += part[c].z, x.w += part[c].w;
        }
        x = make_float4(silu_times(g.x, x.x), silu_times(g.y, x.y), silu_times(g.z, x.z), silu_times(g.w, x.w));
        const uint32_t m = __reduce_max_sync(0xffffffffu, max(max(abs_bits(x.x), abs_bits(x.y)),
                                                              max(abs_bits(x.z), abs_bits(x.w))));
        float scale, inv;
        block_scale(m, &scale, &inv);
        reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * I + nt * kWRows)[lane] =
            e4m3x4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        if (lane == 0) p.out_scales[nt * p.rows + row] = scale;
      }
    }
    if (OUT == kRowsOut && first < items && !abort_flag) {
      const int u = first / NT, n0 = (first - u * NT) * kWRows, row0 = unit_row0(u);
      // four neighbouring columns a thread, every CTA's share requested before any is added
      for (int i = threadIdx.x; i < (j_end - j_begin) * (kWRows / 4); i += kThreads) {
        const int j = j_begin + i / (kWRows / 4), c0 = i % (kWRows / 4) * 4, n = n0 + c0;
        const bool live = p.layout == kFp8Dense ? row0 + j < p.rows : __ldcg(p.sorted_ids + u * TN + j) >= 0;
        if (!live || n >= p.N) continue;  // N % 8 == 0: four columns are all in or all out
        const float* mine = partial + j * kWRows + c0;
        float4 part[kMaxSplit];
#pragma unroll
        for (int c = 0; c < kMaxSplit; ++c)
          if (c < split) part[c] = ld_cluster4(cluster_addr(mine, c));
        float4 x = part[0];
#pragma unroll
        for (int c = 1; c < kMaxSplit; ++c)
          if (c < split) x.x += part[c].x, x.y += part[c].y, x.z += part[c].z, x.w += part[c].w;
        const int64_t at = int64_t(row0 + j) * p.N + n;
        if (p.out_f32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = x;
        } else {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
          uint2 v;
          v.x = *reinterpret_cast<const uint32_t*>(&lo);
          v.y = *reinterpret_cast<const uint32_t*>(&hi);
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = v;
        }
      }
    }
    __syncthreads();
    cluster_sync_all();  // the sums have been read before their CTA ends
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, Cfg::kCols);
  }
}

template <int TN, int OUT>
cudaError_t launch(const Fp8Args& a, int split, cudaStream_t stream) {
  using Cfg = StreamCfg<TN>;
  static_assert(Cfg::kStages >= Cfg::kBufs, "a stage's barrier must not complete twice before its product is read");
  static_assert(Cfg::kStages * Cfg::kStageBytes >= TN * kWRows * 4, "the sums fit where the ring was");
  auto kern = fp8_stream_kernel<TN, OUT>;
  static std::atomic<bool> allowed[kMaxSettingDevices];
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), Cfg::kSmem, allowed);
  if (err != cudaSuccess) return err;
  StreamMaps maps;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if ((err = matrix_map(&maps.x, u8, 1, a.xq, a.rows, a.K, TN)) != cudaSuccess) return err;
  if ((err = matrix_map(&maps.w, u8, 1, a.w, int64_t(a.E) * a.N, a.K, kWRows)) != cudaSuccess) return err;
  const int ctas = OUT == kGateUpOut ? 2 * split : split;
  const int64_t tiles = (a.N + kWRows - 1) / kWRows / (OUT == kGateUpOut ? 2 : 1);
  // upper bound of the items (the grouped unit count is on the device)
  const int64_t items = ((a.rows + TN - 1) / TN + (a.layout == kFp8Dense ? 0 : a.E)) * tiles;
  if (items >= int64_t(1) << 28) return cudaErrorInvalidValue;
  const int64_t slots = int64_t(a.num_sms) * Cfg::kCtas;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(ctas > 1 ? items * ctas : (items < slots ? items : slots)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kern, maps, a, split);
  count_launches(1);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_stream(const Fp8Args& a, int split, cudaStream_t stream) {
  switch (a.bm) {
    case 16: return launch<16, kRowsOut>(a, split, stream);
    case 32: return launch<32, kRowsOut>(a, split, stream);
    default: return launch<64, kRowsOut>(a, split, stream);
  }
}

cudaError_t launch_fp8_stream_gate_up(const Fp8Args& a, int split, cudaStream_t stream) {
  switch (a.bm) {
    case 16: return launch<16, kGateUpOut>(a, split, stream);
    case 32: return launch<32, kGateUpOut>(a, split, stream);
    default: return launch<64, kGateUpOut>(a, split, stream);
  }
}

}  // namespace chord
