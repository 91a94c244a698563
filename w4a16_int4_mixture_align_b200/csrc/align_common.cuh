// align_common.cuh -- the block-padded routing sort by one CTA, shared by the sort kernels
// and the routers that sort in the same launch. The method is described in align.cu.
#pragma once

#include "chord_internal.cuh"

namespace chord {
namespace {

constexpr int kChunk = 1024;       // flat slots per warp chunk (largest)
constexpr int kSteps = kChunk / 32;

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

// Loads the ids of `steps` (<= kSteps) 32-slot steps starting at c0, all up front so the
// loads overlap; slots past n read as -1 (not local).
__device__ __forceinline__ void load_steps(const int32_t* ids, int64_t n, int64_t c0, int steps,
                                           int v[kSteps]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t f = c0 + int64_t(s) * 32 + lane;
    v[s] = (s < steps && f < n) ? __ldg(ids + f) : -1;
  }
}

// hist_row[e] += number of local slots of expert e among the loaded steps (warp-cooperative).
// Non-local slots carry key E.
__device__ __forceinline__ void chunk_count(const int v[kSteps], int steps, int E, int nbits,
                                            int* hist_row) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (s >= steps) break;
    const int e = v[s];
    const bool loc = is_local(e, E);
    const unsigned peers = peers_of(loc ? unsigned(e) : unsigned(E), nbits);
    if (loc && lane == __ffs(peers) - 1) hist_row[e] += __popc(peers);
    __syncwarp();
  }
}

// Places every local slot of the loaded steps at run_row[e] + (rank inside the expert),
// advancing run_row[e]. Ranks follow increasing flat index.
__device__ __forceinline__ void chunk_scatter(const int v[kSteps], int steps, int64_t c0, int E,
                                              int nbits, int* run_row, int32_t* sorted_ids) {
  const int lane = threadIdx.x & 31;
  const unsigned lower = (1u << lane) - 1u;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (s >= steps) break;
    const int e = v[s];
    const bool loc = is_local(e, E);
    const unsigned peers = peers_of(loc ? unsigned(e) : unsigned(E), nbits);
    if (loc) sorted_ids[run_row[e] + __popc(peers & lower)] = int32_t(c0 + int64_t(s) * 32 + lane);
    __syncwarp();
    if (loc && lane == __ffs(peers) - 1) run_row[e] += __popc(peers);
    __syncwarp();
  }
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

// Sentinel fill and expert_ids, shared by both paths.
// cnt[e] = local slots, off[0..E] = padded offsets. Work items are distributed over
// `worker` in [0, nworkers) threads.
__device__ void fill_tail(const int* cnt, const int* off, int E, int block_m, int64_t n, int64_t cap,
                          int64_t nblocks, int32_t* sorted_ids, int32_t* expert_ids,
                          int64_t worker, int64_t nworkers) {
  const int ntp = off[E];
  // padding slots inside each expert's region
  for (int e = int(worker); e < E; e += int(nworkers)) {
    for (int i = off[e] + cnt[e]; i < off[e + 1]; ++i) sorted_ids[i] = int32_t(n);
  }
  for (int64_t i = ntp + worker; i < cap; i += nworkers) sorted_ids[i] = int32_t(n);
  const int64_t used_blocks = ntp / block_m;
  for (int64_t b = worker; b < nblocks; b += nworkers) {
    int val = -1;
    if (b < used_blocks) {
      // largest e with off[e] <= b*block_m (experts with empty regions are skipped)
      const int row = int(b * block_m);
      int lo = 0, hi = E - 1;
      while (lo < hi) {
        int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= row) lo = mid; else hi = mid - 1;
      }
      val = lo;
    }
    expert_ids[b] = val;
  }
}

// ---- single CTA (n <= kSingleMaxChunks chunks) ---------------------------------------
// The whole sort by one CTA of 1024 threads; `smem` holds (32 + 2) * E + 34 ints.
__device__ __forceinline__ void align_single_body(
    const int32_t* __restrict__ ids, int64_t n, int E, int block_m, int64_t cap, int64_t nblocks,
    int32_t* __restrict__ sorted_ids, int32_t* __restrict__ expert_ids, int32_t* __restrict__ ntp_out,
    int32_t* __restrict__ offsets_out, int* smem) {
  int* hist = smem;                 // [32][E]
  int* cnt = hist + 32 * E;         // [E]
  int* off = cnt + E;               // [E+1]
  int* wsum = off + E + 1;          // [33]
  const int tid = threadIdx.x, warp = tid >> 5;
  for (int i = tid; i < 32 * E; i += blockDim.x) hist[i] = 0;
  __syncthreads();

  // warp w owns `steps` consecutive 32-slot steps, so every warp works even for small n
  const int nbits = key_bits(E);
  const int steps = int((n + 32 * 32 - 1) / (32 * 32));
  const int64_t c0 = int64_t(warp) * steps * 32;
  int v[kSteps];
  load_steps(ids, n, c0, steps, v);
  if (c0 < n) chunk_count(v, steps, E, nbits, hist + warp * E);
  __syncthreads();

  for (int e = tid; e < E; e += blockDim.x) {
    int run = 0;
    for (int w = 0; w < 32; ++w) {
      int c = hist[w * E + e];
      hist[w * E + e] = run;
      run += c;
    }
    cnt[e] = run;
    off[e] = (run + block_m - 1) / block_m * block_m;
  }
  __syncthreads();
  const int total = block_exclusive_scan(off, E, wsum);
  if (tid == 0) off[E] = total;
  for (int i = tid; i < 32 * E; i += blockDim.x) hist[i] += off[i % E];
  __syncthreads();

  if (c0 < n) chunk_scatter(v, steps, c0, E, nbits, hist + warp * E, sorted_ids);
  fill_tail(cnt, off, E, block_m, n, cap, nblocks, sorted_ids, expert_ids, tid, blockDim.x);
  if (tid == 0) {
    ntp_out[0] = off[E];
    ntp_out[1] = routing_tag(block_m);
  }
  if (offsets_out)
    for (int e = tid; e <= E; e += blockDim.x) offsets_out[e] = off[e];
}

// Dynamic shared memory of align_single_body.
__host__ __device__ inline size_t align_single_smem_bytes(int E) {
  return (size_t(32) * E + E + E + 1 + 33) * sizeof(int);
}

}  // namespace
}  // namespace chord
