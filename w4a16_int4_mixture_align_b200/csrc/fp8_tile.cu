// fp8_tile.cu -- FP8 block-128 products on the tensor cores (tcgen05) for many rows.
//
//   out[m, n] = sum_kb s[m, n/128, kb] * P_kb[m, n],   P_kb = xq[m, kb] . w[n, kb],
//   s = xs[kb, m] * ws[n/128, kb]
//
// The FP32 scales are arbitrary, so the tensor core cannot apply them: it forms P_kb, the
// product of one 128-wide k block, in tensor memory, and CUDA cores add s * P_kb to FP32
// registers while it forms the next one in another of two buffers (four of 128 columns).
// Activation rows are the M side, so a thread owns one row and a block costs it one scale and
// one fused multiply-add per column.
//
//   warp 0      TMA producer: per k block 128 activation rows and this CTA's weight rows, 128
//               bytes wide (128-byte swizzle), into a ring of stages.
//   warp 2      the same k blocks' scales into a ring in shared memory, by 4-byte asynchronous
//               copies; a stage counts as full with them.
//   warps 1, 3  MMA issuers (one thread each, for even and odd k blocks): four tcgen05.mma
//               (K = 32) per k block, the first overwriting the buffer; a commit frees the
//               stage and publishes the buffer.
//   warps 4..11 promotion: tcgen05.ld of the buffer (two warps per quadrant of 32 lanes, each
//               half of the columns), FP32 accumulation in registers, output.
//
// The promotion warps load nothing from global memory while they add: a wait for a tensor-memory
// load lasts until the warp's other loads in flight are back as well, 1000 cycles and more
// under the kernel's own traffic. With scales loaded to registers (two k blocks ahead) 4096 x
// 4096 x 7168 (M x N x K) takes 124 us, with the ring 114.
//
// CG = 2 runs a CTA pair (cta_group::2): M = 256, each CTA holding 128 activation rows and
// half of the weight rows: 32 KiB per 256 x 256 x 128 step and CTA. Single CTAs with 128 x 128
// tiles serve products of few tiles (512 x 4096 x 7168: 19 us against 29) and experts of one
// block (48 of 7168 x 2048: 145 us against 203; 128 x 256 tiles 149).
//
// Bound: the round trip of a tensor-memory buffer. A block's four MMAs take 512 cycles (a K of
// 32 takes 128 at N = 256, 64 at N = 128), their end is seen about 200 later, reading the buffer
// and adding half of it takes 250 (the additions alone keep the FP32 pipe busy for 256 a block),
// handing it back 250; two buffers of 256 columns fill tensor memory, so a block takes about
// 780, 2.3 PFLOP/s at 8192 x 4096 x 7168 (212 us). Neither MMAs of one column half each with
// four buffers (same time) nor sixteen promotion warps (260 us) nor the whole reading by halves
// of 32-column loads (spills, 249 us) shorten it. The TMA feed runs 6000 cycles ahead.
//
// All waits are bounded. On a timeout a CTA raises CHORD_DEV_TIMEOUT, waits (bounded) for
// its copies and MMAs in flight, frees its tensor memory and returns.
#include <mutex>

#include "fp8_tc.cuh"

namespace chord {
namespace {

constexpr int kPromoteWarps = 8;
constexpr int kFirstPromoteWarp = 4;           // the producers and MMA issuers fill a warpgroup
constexpr int kTileThreads = 32 * (kFirstPromoteWarp + kPromoteWarps);
constexpr int kBM = 128;                       // activation rows of a CTA
constexpr int kABytes = kBM * kFp8Block;
constexpr int kFixedBytes = 1024;              // barriers and the TMEM slot
constexpr int kStagingBytes = 4096;            // output staging of a promotion warp
constexpr int kOutBytes = kPromoteWarps * kStagingBytes;
constexpr int kScaleBytes = 4 * (kBM + 4);     // scales of a k block: 128 rows', two column blocks'
constexpr int kScaleLag = 2;                   // k blocks of scales on their way (1 and 2 take the same)
constexpr int kSmemBudget = 232448 - 1024 - kFixedBytes - kOutBytes;  // 227 KiB less alignment slack

template <int CG, int BN>
struct TileCfg {
  static constexpr int kBRows = BN / CG;
  static constexpr int kStageBytes = kABytes + kBRows * kFp8Block;
  static constexpr int kBufs = 512 / BN;       // tensor-memory buffers
  static constexpr int kStages = (kSmemBudget - (8 + kBufs) * kScaleBytes) / kStageBytes;
  static constexpr int kScaleSlots = kStages + kBufs;
  static constexpr int kSmemBytes = 1024 + kFixedBytes + kStages * kStageBytes + kOutBytes + kScaleSlots * kScaleBytes;
  static constexpr int kCols = BN / 2;         // columns of a promotion warp
  static constexpr int kChunk = BN == 128 ? 32 : 16;       // columns of a tensor-memory load: two of
                                                           // 32 would spill behind 128 sums
};

// Registers per thread: 384 threads launch with 168 each (64512 together); the 256 promotion
// threads take 232 and leave 40 to the other 128 (59392 + 5120 = 64512).
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct TileMaps {
  CUtensorMap x, w, out;
};

// Four bytes to shared memory without a register in between.
__device__ __forceinline__ void copy_async4(uint32_t dst, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but this thread's last N groups have landed.
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One thread: the staged box to the matrix at column `col`, row `row`.
__device__ __forceinline__ void store_box(const CUtensorMap& map, int col, int row, uint32_t buf) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(&map)),
               "r"(col), "r"(row), "r"(buf)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// A warp's 32 rows (one per lane) x COLS columns to the output, in boxes of 32 rows x 128
// bytes staged in `buf` (1024-byte aligned, 128-byte swizzle so that the eight lanes
// of a store phase hit different banks).
template <int COLS, bool F32>
__device__ __forceinline__ void store_rows(const CUtensorMap& map, const float (&acc)[COLS], uint32_t buf, int n0,
                                           int row0, int N) {
  constexpr int W = F32 ? 32 : 64;  // columns of a box
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < COLS; c += W) {
    if (n0 + c >= N) break;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // `buf` is free again
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = F32 ? __float_as_uint(acc[c + 4 * j + (F32 ? i : 0)])
                   : bf16_pair(acc[c + (F32 ? 0 : 8 * j + 2 * i)], acc[c + (F32 ? 0 : 8 * j + 2 * i + 1)]);
      sts128(buf + lane * 128 + ((j ^ (lane & 7)) << 4), v);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) store_box(map, n0 + c, row0, buf);
  }
}

// What becomes of a tile: rows of the output, or (kGateUp) SiLU(gate) * up quantised to FP8. A
// kGateUp tile holds 128 gate columns and the 128 up columns of the same intermediate ones
// (rank 0 of the pair loads the former's weight rows, rank 1 the latter's); a promotion
// thread takes 64 of each, so the product needs no exchange, and the block's maximum one of
// a word per row between two warps.
enum Epilogue { kRows = 0, kGateUp = 1 };

template <int CG, int BN, int EPI>
__global__ void __launch_bounds__(kTileThreads, 1)
    fp8_tile_kernel(const __grid_constant__ TileMaps maps, const Fp8Args p) {
  using Cfg = TileCfg<CG, BN>;
  constexpr int S = Cfg::kStages, COLS = Cfg::kCols, B = Cfg::kBufs, D = Cfg::kScaleSlots;
  static_assert(EPI == kRows || (CG == 2 && BN == 256), "the gate_up tile");
  static_assert(S <= 8 && S > kScaleLag, "ring");
  static_assert(S >= B, "a stage's barriers must not be a phase behind: done for the adding warps, full for the issuers");
  static_assert(B % 2 == 0, "a buffer belongs to one issuer");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);  // [S] stage loaded (rank 0's is used)
  uint64_t* done = full + S;                           // [S] stage multiplied: it may be refilled, its
                                                       // product read
  uint64_t* acc_empty = done + S;                      // [B] buffer read by every warp (rank 0's is used)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + B);
  __shared__ int abort_flag;
  // kGateUp: maxima of the rows by column half, in the half of a staging box it does not use
  uint32_t(*row_max)[kBM] =
      reinterpret_cast<uint32_t(*)[kBM]>(smem + kFixedBytes + S * Cfg::kStageBytes + kStagingBytes / 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const uint32_t scales = sbase + kFixedBytes + S * Cfg::kStageBytes + kOutBytes;  // [D] slots
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1 + CG);  // the copies and each CTA's scales
      mbar_init(&done[s], 1);
    }
    for (int b = 0; b < B; ++b) mbar_init(&acc_empty[b], kPromoteWarps * CG);
    fence_barrier_init();
  }
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // the peer's barriers exist before anything arrives on them
  if (warp == 1) tmem_alloc<CG>(tmem_slot, B * BN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  volatile int* abort_v = &abort_flag;
  grid_dep_wait();
  grid_dep_trigger();

  const int KB = fp8_blocks(p.K), NT = (p.N + BN - 1) / BN, NB = fp8_blocks(p.N);
  const int I = p.N / 2;  // kGateUp
  // 32 bits: the host checks that the tiles' number fits
  const int units = p.layout == kFp8Dense ? int((p.rows + kBM * CG - 1) / (kBM * CG)) : p.ntp[0] / (kBM * CG);
  const int tiles = units * NT;
  const int cid = CG == 2 ? cluster_id_x() : blockIdx.x, ncl = CG == 2 ? num_clusters_x() : gridDim.x;

  if (warp < kFirstPromoteWarp) {
    give_registers<40>();
    const uint32_t full0 = CG == 2 ? cluster_addr(full, 0) : smem_u32(full);
    if (warp == 0) {
      if (lane == 0) {
        uint32_t fill = 0;
        bool ok = true;
        for (int t = cid; t < tiles && ok; t += ncl) {
          const int u = t / NT, nt = t - u * NT;
          const int xrow = (p.layout == kFp8Dense ? u * kBM * CG : __ldcg(p.block_row0 + u)) + int(rank) * kBM;
          int wrow;
          if (EPI == kGateUp) wrow = int(rank) * I + nt * kFp8Block;
          else wrow = (p.layout == kFp8Dense ? 0 : __ldcg(p.expert_ids + u)) * p.N + nt * BN + int(rank) * Cfg::kBRows;
          for (int kb = 0; kb < KB; ++kb, ++fill) {
            const uint32_t s = fill % S;
            if (fill >= S && !mbar_wait(&done[s], ((fill / S) - 1) & 1, abort_v, p.status)) {
              ok = false;
              break;
            }
            const uint32_t st = sbase + kFixedBytes + s * Cfg::kStageBytes, bar = full0 + s * 8;
            if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * Cfg::kStageBytes);
            tma_2d<CG>(st, &maps.x, kb * kFp8Block, xrow, bar);
            tma_2d<CG>(st + kABytes, &maps.w, kb * kFp8Block, wrow, bar);
          }
        }
        // the last copies have landed before the CTA ends (rank 0's barriers count both CTAs')
        if (rank == 0) {
          int dummy = 0;
          for (uint32_t f = fill > S ? fill - S : 0; f < fill; ++f)
            mbar_wait(&full[f % S], (f / S) & 1, &dummy, p.status);
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // scales of the k blocks into a ring of D = S + B slots: a stage is filled again once its
      // product is formed, which took the buffer of B blocks before it, whose scales had been read
      uint32_t fill = 0, told = 0;
      bool ok = true;
      auto tell = [&] {  // the oldest block's scales are there
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) mbar_arrive_cluster(full0 + told % S * 8);
          else mbar_arrive(&full[told % S]);
        }
        ++told;
      };
      for (int t = cid; t < tiles && ok; t += ncl) {
        const int u = t / NT, nt = t - u * NT;
        const int row0 = (p.layout == kFp8Dense ? u * kBM * CG : __ldcg(p.block_row0 + u)) + int(rank) * kBM;
        const int e = p.layout == kFp8Dense ? 0 : __ldcg(p.expert_ids + u);
        const float* xs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = row0 + 32 * i + lane;
          xs[i] = p.xs + (row < p.rows ? row : 0);  // rows that are not stored read row 0's
        }
        // lanes 0 and 1: of the two halves of the columns (kGateUp: gate, up)
        const int nb = EPI == kGateUp ? nt + (lane & 1) * (I / kFp8Block) : min((nt * BN + (lane & 1) * COLS) / kFp8Block, NB - 1);
        const float* ws = p.ws + (int64_t(e) * NB + nb) * KB;
        for (int kb = 0; kb < KB; ++kb, ++fill) {
          if (fill >= S && !mbar_wait_warp(&done[fill % S], ((fill / S) - 1) & 1, abort_v, p.status)) {
            ok = false;
            break;
          }
          const uint32_t dst = scales + fill % D * kScaleBytes + 4 * lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            copy_async4(dst + 128 * i, xs[i]);
            xs[i] += p.rows;
          }
          if (lane < 2) copy_async4(dst + 4 * kBM, ws + kb);
          copy_async_commit();
          if (fill - told >= kScaleLag) {
            copy_async_wait<kScaleLag>();
            tell();
          }
        }
      }
      copy_async_wait<0>();
      while (told < fill) tell();
    } else if (lane == 0 && rank == 0) {
      // warp 1 multiplies the even k blocks, warp 3 the odd ones: issuing a block's MMAs holds
      // its thread for about their time, so a single issuer's waits and commits between two
      // blocks were time that the tensor core stood still
      constexpr uint32_t idesc = idesc_e4m3(kBM * CG, BN);
      const uint32_t blocks = uint32_t(cid < tiles ? (tiles - cid + ncl - 1) / ncl : 0) * uint32_t(KB);
      uint32_t it = warp == 1 ? 0 : 1;
      for (; it < blocks; it += 2) {
        const uint32_t s = it % S, b = it % B;
        // The buffer first, then the stage. A wait sees the parity of a phase only, and where S is
        // odd a stage changes hands between the issuers, so this one may never have waited for the
        // phase of block it - S: while that copy was still under way, a wait for the phase of block
        // `it` would pass at once. That block it - B has been added says that it - S <= it - B landed.
        if ((it >= B && !mbar_wait(&acc_empty[b], ((it / B) - 1) & 1, abort_v, p.status)) ||
            !mbar_wait(&full[s], (it / S) & 1, abort_v, p.status))
          break;
        tc_fence_after();
        const uint32_t st = sbase + kFixedBytes + s * Cfg::kStageBytes;
        const uint64_t ad = sw128_kmajor_desc(st), bd = sw128_kmajor_desc(st + kABytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_e4m3<CG>(tmem + b * BN, ad + 2 * k, bd + 2 * k, idesc, k > 0);
        commit<CG>(&done[s]);
      }
      if (it >= 2) {  // no MMA writes tensor memory once it is freed
        int dummy = 0;
        mbar_wait(&done[(it - 2) % S], ((it - 2) / S) & 1, &dummy, p.status);
      }
    }
    __syncwarp();
  } else {
    take_registers<232>();
    const int q = warp & 3;            // the tensor-memory lanes this warp may read
    const int h = (warp - kFirstPromoteWarp) >> 2;     // its half of the columns
    const int r = q * 32 + lane;
    const uint32_t empty0 = CG == 2 ? cluster_addr(acc_empty, 0) : smem_u32(acc_empty);
    const uint32_t src = tmem + (uint32_t(q * 32) << 16) + (EPI == kGateUp ? h * 64 : h * COLS);
    // column (from src) of chunk c: a kGateUp warp's second half are the up columns
    auto chunk = [](int c) { return EPI == kGateUp && c >= 64 / Cfg::kChunk ? 128 + Cfg::kChunk * c - 64 : Cfg::kChunk * c; };
    const uint32_t staging = sbase + kFixedBytes + S * Cfg::kStageBytes + (warp - kFirstPromoteWarp) * kStagingBytes;
    uint32_t it = 0;
    bool ok = true;
    // a kGateUp warp that gave up still meets its partner's barriers (its waits return at once)
    for (int t = cid; t < tiles && (ok || EPI == kGateUp); t += ncl) {
      const int u = t / NT;
      const int n0 = EPI == kGateUp ? (t - u * NT) * kFp8Block + h * 64 : (t - u * NT) * BN + h * COLS;
      const int pos = u * kBM * CG + int(rank) * kBM + r;
      const int64_t row = p.layout == kFp8Dense ? pos : __ldcg(p.block_row0 + u) + int(rank) * kBM + r;
      const bool live = p.layout == kFp8Dense ? row < p.rows : __ldcg(p.sorted_ids + pos) >= 0;
      uint64_t sum[COLS / 2];  // columns 2i, 2i + 1
#pragma unroll
      for (int c = 0; c < COLS / 2; ++c) sum[c] = 0;
      // half of the columns at a time: the second half is in registers, and the buffer handed
      // back, before it is added
      constexpr int W = Cfg::kChunk, CH = COLS / W / 2;
      uint32_t v[CH][W];
#pragma unroll 1
      for (int kb = 0; kb < KB; ++kb) {
        ok = mbar_wait_warp(&done[it % S], (it / S) & 1, abort_v, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t b = it % B, slot = scales + it % D * kScaleBytes;
        ++it;
#pragma unroll
        for (int c = 0; c < CH; ++c) tmem_ld_async(src + b * BN + chunk(c), v[c]);
        const float x = lds_f32(slot + 4 * r), w0 = lds_f32(slot + 4 * kBM + (EPI == kGateUp ? 0 : 4 * h));
        const uint64_t s = pack2(x * w0, x * w0);
        uint64_t s_up = s;
        if (EPI == kGateUp) {
          const float w1 = lds_f32(slot + 4 * kBM + 4);
          s_up = pack2(x * w1, x * w1);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          tmem_wait_ld(v[c]);
#pragma unroll
          for (int j = 0; j < W; j += 2) fma2(sum[(W * c + j) / 2], v[c][j], v[c][j + 1], s);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) tmem_ld_async(src + b * BN + chunk(CH + c), v[c]);
#pragma unroll
        for (int c = 0; c < CH; ++c) tmem_wait_ld(v[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) mbar_arrive_cluster(empty0 + b * 8);
          else mbar_arrive(&acc_empty[b]);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < W; j += 2) fma2(sum[(W * (CH + c) + j) / 2], v[c][j], v[c][j + 1], s_up);
      }
      if (!ok && EPI != kGateUp) continue;
      float acc[COLS];
#pragma unroll
      for (int c = 0; c < COLS / 2; ++c) unpack2(sum[c], acc[2 * c], acc[2 * c + 1]);
      if (EPI == kGateUp) {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          acc[c] = silu_times(acc[c], acc[c + 64]);
          m = max(m, abs_bits(acc[c]));
        }
        row_max[h][r] = m;
        named_bar_sync(1 + q, 64);  // the two warps of these rows
        m = max(m, row_max[h ^ 1][r]);
        named_bar_sync(1 + q, 64);  // both have read before the next tile's maxima
        float scale, inv;
        block_scale(m, &scale, &inv);
        if (ok && row < p.rows && h == 0) p.out_scales[int64_t(n0 / kFp8Block) * p.rows + row] = scale;
        const int row0 = int(row) - lane;
        if (!ok || row0 >= p.rows) continue;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // 64-byte rows, 64-byte swizzle
          uint32_t code[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 16 * j + 4 * i;
            code[i] = e4m3x4(acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv);
          }
          sts128(staging + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), code);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) store_box(maps.out, n0, row0, staging);
        continue;
      }
      // 32 whole rows leave through shared memory by TMA, 128 bytes wide, while the next tile
      // runs (stores of a row per lane held the promotion for about 4 us a tile); rows past a
      // dense matrix are cut off by the copy. Where some rows are not to be written, each lane
      // stores its own.
      const bool whole = p.layout == kFp8Dense || __all_sync(0xffffffffu, live);
      if (whole) {
        const int row0 = int(row) - lane;
        if (row0 >= p.rows) continue;
        if (p.out_f32) store_rows<COLS, true>(maps.out, acc, staging, n0, row0, p.N);
        else store_rows<COLS, false>(maps.out, acc, staging, n0, row0, p.N);
      } else if (live && p.out_f32) {
        float* o = static_cast<float*>(p.out) + row * p.N + n0;
#pragma unroll
        for (int c = 0; c < COLS; c += 4)
          if (n0 + c < p.N) *reinterpret_cast<float4*>(o + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
      } else if (live) {
        uint16_t* o = static_cast<uint16_t*>(p.out) + row * p.N + n0;
#pragma unroll
        for (int c = 0; c < COLS; c += 8)
          if (n0 + c < p.N)
            *reinterpret_cast<uint4*>(o + c) = make_uint4(bf16_pair(acc[c], acc[c + 1]), bf16_pair(acc[c + 2], acc[c + 3]),
                                                          bf16_pair(acc[c + 4], acc[c + 5]), bf16_pair(acc[c + 6], acc[c + 7]));
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // nothing of either CTA is in flight towards the other
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem, B * BN);
  }
}

// ------------------------------------------------------------------------------------ host

template <int CG, int BN, int EPI>
cudaError_t launch(const Fp8Args& a, cudaStream_t stream) {
  using Cfg = TileCfg<CG, BN>;
  auto kern = fp8_tile_kernel<CG, BN, EPI>;
  static std::atomic<bool> allowed[kMaxSettingDevices];
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), Cfg::kSmemBytes, allowed);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // clusters that fit at once, per device (they must fit inside a GPC)
  static std::mutex mu;
  static int fits[64];
  int dev = 0;
  if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int most;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (fits[dev] == 0) {
      cfg.gridDim = dim3(unsigned(a.num_sms / CG * CG));
      if ((err = cudaOccupancyMaxActiveClusters(&fits[dev], kern, &cfg)) != cudaSuccess) return err;
    }
    most = fits[dev];
  }
  if (most < 1) return cudaErrorLaunchOutOfResources;
  if (most > a.num_sms / CG) most = a.num_sms / CG;
  TileMaps maps;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if ((err = matrix_map(&maps.x, u8, 1, a.xq, a.rows, a.K, kBM)) != cudaSuccess) return err;
  if ((err = matrix_map(&maps.w, u8, 1, a.w, int64_t(a.E) * a.N, a.K, Cfg::kBRows)) != cudaSuccess) return err;
  if (EPI == kGateUp) err = matrix_map(&maps.out, u8, 1, a.out, a.rows, a.N / 2, 32, 64);
  else err = matrix_map(&maps.out, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   a.out_f32 ? 4 : 2, a.out, a.rows, a.N, 32);
  if (err != cudaSuccess) return err;
  // upper bound of the tiles (the grouped unit count is on the device)
  const int64_t units = (a.rows + kBM * CG - 1) / (kBM * CG) + (a.layout == kFp8Dense ? 0 : a.E);
  const int64_t tiles = units * ((a.N + BN - 1) / BN);
  if (tiles >= int64_t(1) << 30) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(unsigned((tiles < most ? tiles : most) * CG));
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kern, maps, a);
  count_launches(1);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_tile(const Fp8Args& a, cudaStream_t stream) {
  if (a.bm == 256) return launch<2, 256, kRows>(a, stream);
  return launch<1, 128, kRows>(a, stream);
}

cudaError_t launch_fp8_tile_gate_up(const Fp8Args& a, cudaStream_t stream) {
  return launch<2, 256, kGateUp>(a, stream);
}

}  // namespace chord
