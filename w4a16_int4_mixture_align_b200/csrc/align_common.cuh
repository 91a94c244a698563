// align_common.cuh -- pieces of the block-padded routing sort: what align.cu and router.cu
// share, and the sort by one CTA or one cluster with which the scored router ends. The
// tensors and the method are described in align.cu.
#pragma once

#include "chord_internal.cuh"
#include "tc_common.cuh"

namespace chord {
namespace {

__device__ __forceinline__ int ld_cluster_i32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ bool is_local(int e, int E) { return unsigned(e) < unsigned(E); }

// Lanes of the warp holding the same key as this lane (key < 2^nbits), from one ballot
// per key bit: cheaper than __match_any_sync when a step holds many distinct keys.
__device__ __forceinline__ unsigned peers_of(unsigned key, int nbits) {
  unsigned eq = 0xffffffffu;
  for (int b = 0; b < nbits; ++b) {
    const unsigned bit = (key >> b) & 1u;
    const unsigned m = __ballot_sync(0xffffffffu, bit);
    eq &= bit ? m : ~m;
  }
  return eq;
}

__host__ __device__ inline int key_bits(int E) {
  int b = 1;
  while ((1 << b) <= E) ++b;  // keys 0..E fit in b bits
  return b;
}

// Exclusive prefix sum over vals[0..count) in shared memory (count <= blockDim.x <= 1024),
// returns the total. All threads of the block must call it.
__device__ int block_exclusive_scan(int* vals, int count, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nwarps = (blockDim.x + 31) >> 5;
  int v = tid < count ? vals[tid] : 0;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = lane < nwarps ? warp_sums[lane] : 0;
    int wi = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      int o = __shfl_up_sync(0xffffffffu, wi, d);
      if (lane >= d) wi += o;
    }
    if (lane < nwarps) warp_sums[lane] = wi - w;  // exclusive warp offsets
    if (lane == 31) warp_sums[32] = wi;           // total
  }
  __syncthreads();
  if (tid < count) vals[tid] = incl - v + warp_sums[warp];
  const int total = warp_sums[32];
  __syncthreads();
  return total;
}

// Exclusive prefix of vals[0, count) in place for any count (each thread sums a run of
// consecutive values, the runs' sums are scanned across the block); returns the total.
// tmp holds blockDim.x ints, warp_sums 33.
__device__ int block_exclusive_scan_runs(int* vals, int count, int* tmp, int* warp_sums) {
  const int tid = threadIdx.x;
  const int per = (count + int(blockDim.x) - 1) / int(blockDim.x);
  const int b = tid * per;
  int sum = 0;
  for (int i = 0; i < per; ++i)
    if (b + i < count) sum += vals[b + i];
  tmp[tid] = sum;
  __syncthreads();
  const int total = block_exclusive_scan(tmp, int(blockDim.x), warp_sums);
  int run = tmp[tid];
  for (int i = 0; i < per; ++i)
    if (b + i < count) {
      const int x = vals[b + i];
      vals[b + i] = run;
      run += x;
    }
  __syncthreads();
  return total;
}

// ---- the whole sort by one CTA or one cluster ----------------------------------------
//
// C CTAs (rank: this one's number) of NW warps each. A CTA sorts the flat slots [begin, end);
// the CTAs' ranges follow one another and cover [0, n). Warp w of a CTA owns `steps`
// consecutive 32-slot steps (steps <= MAXS) and counts them by expert in its row of `hist`;
// a prefix over the warps (one warp per expert, a lane per row), over the CTAs' totals
// (distributed shared memory) and over the experts' padded totals then gives every warp the
// position of its first slot of each expert. `smem`: align_smem_bytes().
template <int NW>
__host__ __device__ inline size_t align_smem_bytes(int E) {
  return (size_t(NW) * (E | 1) + 3 * E + E + 1 + 32 * NW + 33) * sizeof(int);
}

template <int C, int NW, int MAXS>
__device__ __forceinline__ void align_body(const int32_t* ids, int64_t n, int64_t begin, int64_t end, int rank, int E,
                                           int block_m, int64_t cap, int64_t nblocks, int32_t* sorted_ids,
                                           int32_t* expert_ids, int32_t* ntp_out, int32_t* offsets_out, int* smem) {
  static_assert(NW <= 32, "a lane per warp's row");
  // rows of an odd length, so that the lanes of a column's prefix hit different banks
  const int ldh = E | 1;
  int* hist = smem;              // [NW][ldh]
  int* own = hist + NW * ldh;    // [E] this CTA's slots of each expert
  int* cnt = own + E;            // [E] all of them
  int* base = cnt + E;           // [E] position of this CTA's first slot
  int* off = base + E;           // [E + 1] position of the expert's first slot
  int* tmp = off + E + 1;        // [32 * NW]
  int* wsum = tmp + 32 * NW;     // [33]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned lower = (1u << lane) - 1u;
  for (int i = tid; i < NW * ldh; i += 32 * NW) hist[i] = 0;
  __syncthreads();

  const int nbits = key_bits(E);
  const int steps = int((end - begin + 32 * NW - 1) / (32 * NW));
  const int64_t c0 = begin + int64_t(warp) * steps * 32;
  int* row = hist + warp * ldh;
  int v[MAXS];
#pragma unroll
  for (int s = 0; s < MAXS; ++s) {  // all loads at once
    const int64_t f = c0 + 32 * s + lane;
    v[s] = s < steps && f < end ? ids[f] : -1;
  }
#pragma unroll
  for (int s = 0; s < MAXS; ++s) {
    if (s >= steps) break;
    if (is_local(v[s], E)) atomicAdd(row + v[s], 1);  // integers: any order gives the same counts
  }
  __syncthreads();

#pragma unroll 2
  for (int e = warp; e < E; e += NW) {
    const int c = lane < NW ? hist[lane * ldh + e] : 0;
    int incl = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane < NW) hist[lane * ldh + e] = incl - c;
    if (lane == 31) own[e] = incl;
  }
  if (C > 1) cluster_sync_all();
  else __syncthreads();
  for (int e = tid; e < E; e += 32 * NW) {
    int before = 0, total = 0, c[C];
#pragma unroll
    for (int r = 0; r < C; ++r) c[r] = C > 1 ? ld_cluster_i32(cluster_addr(own + e, r)) : own[e];
#pragma unroll
    for (int r = 0; r < C; ++r) {
      total += c[r];
      before += r < rank ? c[r] : 0;
    }
    cnt[e] = total;
    off[e] = (total + block_m - 1) / block_m * block_m;
    base[e] = before;
  }
  __syncthreads();
  const int total = block_exclusive_scan_runs(off, E, tmp, wsum);
  if (tid == 0) off[E] = total;
  for (int e = tid; e < E; e += 32 * NW) base[e] += off[e];
  __syncthreads();

#pragma unroll
  for (int s = 0; s < MAXS; ++s) {
    if (s >= steps) break;
    const int e = v[s];
    const bool loc = is_local(e, E);
    const unsigned peers = peers_of(loc ? unsigned(e) : unsigned(E), nbits);
    if (loc) sorted_ids[base[e] + row[e] + __popc(peers & lower)] = int32_t(c0 + 32 * s + lane);
    __syncwarp();
    if (loc && lane == __ffs(peers) - 1) row[e] += __popc(peers);
    __syncwarp();
  }
  // sentinels: a warp per expert's padding, then the tail; expert_ids: a thread per block
  const int threads = C * 32 * NW, worker = rank * 32 * NW + tid;
  for (int e = rank * NW + warp; e < E; e += C * NW)
    for (int i = off[e] + cnt[e] + lane; i < off[e + 1]; i += 32) sorted_ids[i] = int32_t(n);
  for (int64_t i = total + worker; i < cap; i += threads) sorted_ids[i] = int32_t(n);
  for (int64_t b = worker; b < nblocks; b += threads) {
    int val = -1;
    if (b * block_m < total) {
      // largest e with off[e] <= b*block_m (experts with empty regions are skipped)
      int lo = 0, hi = E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= int(b * block_m)) lo = mid;
        else hi = mid - 1;
      }
      val = lo;
    }
    expert_ids[b] = val;
  }
  if (worker == 0) {
    ntp_out[0] = total;
    ntp_out[1] = routing_tag(block_m);
  }
  if (offsets_out)
    for (int e = worker; e <= E; e += threads) offsets_out[e] = off[e];
  if (C > 1) cluster_sync_all();  // `own` has been read before its CTA ends
}

}  // namespace
}  // namespace chord
