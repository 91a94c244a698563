// router.cu -- scored routing to experts: softmax or sigmoid scores, a balance bias on the
// choice, expert groups, top-k, renormalised and scaled weights.
//
// Per token, with logits l_e, bias b_e (optional) and G experts in n_group equal runs:
//   s_e = sigmoid(l_e), or softmax over the token's unmasked logits;
//   c_e = s_e + b_e               what experts are chosen by (a masked expert never is);
//   group score = sum of the group_top (1 or 2) largest c of the group; the topk_group
//   best groups stay; then the topk largest c among them, in descending order;
//   w = s_e of the chosen (without the bias), over their sum if renormalised, x scale.
// A logit that is NaN, -inf or the lowest value of its type masks its expert.
//
// The choice is that of exact arithmetic, ties going to the lower id, although almost all
// of the work is in FP32: two experts whose c differ by less than FP32 resolves would
// otherwise be ordered by rounding. One warp owns a token:
//   1. c in FP32 for every expert (lane l: experts l, l + 32, ...). Without a bias both
//      scores grow with the logit, so the logit itself is the key and nothing rounds.
//   2. the k-th largest of the 32 lane maxima is at most the k-th largest c, so every
//      expert of the answer is among those with c >= that threshold minus twice the FP32
//      error bound. Typically 8 to 12 of 384 experts are; they are compacted to one per lane.
//   3. one c in FP64 per lane, the rank of each by counting larger ones, and the weights.
// Groups are scored in FP32 as well; a border between a kept and a dropped group closer
// than the error bound, more than 32 candidates, or k > 32 take the slow way: every c in
// FP64 in shared memory, then k rounds of a warp-wide maximum.
//
// Bound: 8192 tokens of 384 FP32 logits take 15 us where reading them (12.6 MB) would take 2: a
// token is about 1100 instructions, many of them dependent, and 32 warps fit an SM, so the
// batch is two rounds of 5 us. One token is 4 us of that chain and 3 more of instruction
// fetches; the sort behind it adds 3.
#include <math.h>

#include "align_common.cuh"

namespace chord {
namespace {

constexpr int kRouterWarps = 8;
constexpr unsigned kFull = 0xffffffffu;
// How far a c in FP32 may be off, with u = 2^-24. Softmax: the denominator 46 u (each exponential
// 4 u and, where it weighs most, 5 u for its rounded argument, up to 31 + 5 additions, one
// division), common to all experts of a token; the expert's own exponential 4 u (2 ulp; the
// 1.173 |x| more of a large |x| come with an e^x that falls faster), its argument u, the product u:
// 52 u = 3.1e-6 in all, times s <= 1. Sigmoid 8 u. Adding the bias rounds by u |c|. The sum of a
// group's two best is off by 46 u (s1 + s2) + 12 u <= 58 u = 3.5e-6, as s1 + s2 <= 1. So a slack of
// 4e-6 + 1e-6 |c| bounds each of these, and two of them a comparison of two.
constexpr float kSlackAbs = 4e-6f, kSlackRel = 1e-6f;

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float warp_max(float v) { return order_value(__reduce_max_sync(kFull, order_key(v))); }
__device__ __forceinline__ float warp_min(float v) { return order_value(__reduce_min_sync(kFull, order_key(v))); }
template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

constexpr float kLowestF32 = -3.402823466e38f, kLowestBf16 = -3.38953139e38f, kLowestF16 = -65504.f;
// The logit, -inf where it masks its expert, +inf as the largest finite value.
__device__ __forceinline__ float masked_logit(float v, float lowest) { return v > lowest ? fminf(v, -lowest) : -INFINITY; }
__device__ __forceinline__ float load_logit(const RouterArgs& p, int64_t row, int e) {
  if (p.dtype == CHORD_DTYPE_F32) return masked_logit(__ldcg(static_cast<const float*>(p.logits) + row + e), kLowestF32);
  const uint16_t bits = __ldcg(static_cast<const uint16_t*>(p.logits) + row + e);
  if (p.dtype == CHORD_DTYPE_BF16) return masked_logit(__uint_as_float(uint32_t(bits) << 16), kLowestBf16);
  return masked_logit(__half2float(__ushort_as_half(bits)), kLowestF16);
}

// 1 / d for 2^-100 <= d <= 2^100, within a few 2^-52: Newton's iteration r <- r (2 - d r) doubles the 23 bits of an
// FP32 reciprocal twice.
__device__ __forceinline__ double reciprocal64(double d) {
  double r = double(1.0f / float(d));
  r = fma(r, fma(-d, r, 1.0), r);
  return fma(r, fma(-d, r, 1.0), r);
}
// s in FP64; `lmax` and `rz` (one over the softmax denominator) are unused for sigmoid. Not
// inlined: the code is long, it is used in several places, and a small call runs it cold.
__device__ __noinline__ double score64_of(int score, float l, float lmax, double rz) {
  if (score == CHORD_SCORE_SOFTMAX) return exp(double(l) - double(lmax)) * rz;
  return 1.0 / (1.0 + exp(-double(l)));
}
__device__ __forceinline__ double score64(const RouterArgs& p, float l, float lmax, double rz) {
  return score64_of(p.score, l, lmax, rz);
}
// s in FP32, within the bound above.
__device__ __forceinline__ float score32(const RouterArgs& p, float l, float lmax, float rz) {
  if (p.score == CHORD_SCORE_SOFTMAX) return __expf(l - lmax) * rz;
  return __fdividef(1.f, 1.f + __expf(-fminf(fmaxf(l, -80.f), 80.f)));
}

// One over the softmax denominator of token t in FP64 (1 if every logit is masked).
__device__ __noinline__ double softmax_sum64(const RouterArgs& p, int64_t t, float lmax) {
  double z = 0.0;
  for (int e = threadIdx.x & 31; e < p.G; e += 32) {
    const float l = load_logit(p, t * p.ld, e);
    if (l > -INFINITY) z += exp(double(l) - double(lmax));
  }
  z = warp_sum(z);
  return z > 0.0 ? 1.0 / z : 1.0;
}

// The kept groups of the token as a bit mask, from the keys v[0..G) in shared memory
// (-inf: masked); V = float: approximate scores, `near` reports a border that their error
// could move; V = double: exact. A team of 32 / (n_group rounded up to a power of two) lanes
// scans each group.
template <typename V>
__device__ __forceinline__ uint32_t kept_groups(const RouterArgs& p, const V* v, float lmax, bool* near) {
  const int lane = threadIdx.x & 31;
  int teams = 1;
  while (teams < p.n_group) teams <<= 1;
  const int width = 32 / teams;
  const int g = lane / width, sub = lane % width;
  V a1 = V(-INFINITY), a2 = V(-INFINITY);
  if (g < p.n_group) {
    const V* of = v + g * p.group_size;
#pragma unroll 4
    for (int j = sub; j < p.group_size; j += width) {
      const V x = of[j];
      const V lo = x < a1 ? x : a1;
      a1 = x < a1 ? a1 : x;
      a2 = a2 < lo ? lo : a2;
    }
  }
#pragma unroll 1
  for (int o = 1; o < width; o <<= 1) {
    const V b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
    const V lo = a1 < b1 ? a1 : b1;
    a1 = a1 < b1 ? b1 : a1;
    a2 = a2 < b2 ? b2 : a2;
    a2 = a2 < lo ? lo : a2;
  }
  const bool any = a1 > V(-INFINITY), two = p.group_top == 2 && a2 > V(-INFINITY);
  V score = a1;
  float off = 0.f;  // how far `score` may be off
  if (any && (p.group_top == 2 || p.bias)) {
    // without a bias the keys are logits: their scores add up, not they themselves (the
    // softmax denominator is common to all groups and left out)
    if (!p.bias && p.group_top == 2) {
      if constexpr (sizeof(V) == 8)
        score = score64(p, float(a1), lmax, 1.0) + (two ? score64(p, float(a2), lmax, 1.0) : 0.0);
      else
        score = score32(p, a1, lmax, 1.f) + (two ? score32(p, a2, lmax, 1.f) : 0.f);
    } else if (two) {
      score += a2;
    }
    off = kSlackAbs + kSlackRel * (fabsf(float(a1)) + (two ? fabsf(float(a2)) : 0.f));
  }
  // lane i < n_group takes group i's score; rank by counting
  V mine = __shfl_sync(kFull, score, (lane * width) & 31);
  const float mine_off = __shfl_sync(kFull, off, (lane * width) & 31);
  if (lane >= p.n_group) mine = V(-INFINITY);
  int rank = 0;
#pragma unroll 4
  for (int i = 0; i < p.n_group; ++i) {
    const V o = __shfl_sync(kFull, mine, i);
    rank += (o > mine || (o == mine && i < lane)) ? 1 : 0;
  }
  const bool real = mine > V(-INFINITY);
  const uint32_t kept = __ballot_sync(kFull, real && rank < p.topk_group);
  *near = false;
  if constexpr (sizeof(V) == 4) {
    // in doubt where the least a kept group may have is no more than a dropped one may have
    const bool in = (kept >> lane) & 1u;
    const float low = warp_min(in ? mine - mine_off : INFINITY);
    const float high = warp_max(real && !in ? mine + mine_off : -INFINITY);
    *near = high >= low && (p.bias || p.group_top == 2);
  }
  return kept;
}

// Doubles as unsigned integers of the same order.
__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t b = uint64_t(__double_as_longlong(v));
  return b ^ ((b >> 63) ? ~uint64_t(0) : uint64_t(1) << 63);
}
// Rank of this lane's candidate (lane < n) by c descending, ties to the lower lane. `keys`: 32
// shared 64-bit words of this warp.
__device__ __forceinline__ int rank_of(double c, int n, uint64_t* keys) {
  const int lane = threadIdx.x & 31;
  const uint64_t mine = order_key64(c + 0.0);  // -0 is the same number as 0
  __syncwarp();
  keys[lane] = mine;  // lanes from n on hold -inf, below every candidate
  __syncwarp();
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; j += 2) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(keys + j);
    rank += (o.x > mine || (o.x == mine && j < lane)) ? 1 : 0;
    rank += (o.y > mine || (o.y == mine && j + 1 < lane)) ? 1 : 0;
  }
  return rank;
}
// Whether two of the n candidates are closer than `d`.
__device__ __forceinline__ bool any_closer(double c, int n, double d) {
  const int lane = threadIdx.x & 31;
  bool close = false;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(kFull, c, j);
    close = close || (j != lane && lane < n && fabs(o - c) <= d);
  }
  return __any_sync(kFull, close);
}

// Every c in FP64 (shared memory), k rounds of a warp-wide maximum.
__device__ __noinline__ void route_exact(const RouterArgs& p, int64_t t, float lmax, double* c64) {
  const int lane = threadIdx.x & 31;
  const int per = (p.G + 31) / 32;
  const double rz = p.score == CHORD_SCORE_SOFTMAX ? softmax_sum64(p, t, lmax) : 1.0;
  __syncwarp();
  for (int e = lane; e < p.G; e += 32) {
    const float l = load_logit(p, t * p.ld, e);
    double c = -INFINITY;
    if (l > -INFINITY) c = p.bias ? score64(p, l, lmax, rz) + double(p.bias[e]) : double(l);
    c64[e] = c;
  }
  __syncwarp();
  uint32_t kept = kFull;
  if (p.n_group > 1) {
    bool near;
    kept = kept_groups<double>(p, c64, lmax, &near);
  }
  uint32_t open = 0;  // this lane's experts that may still be chosen
  for (int i = 0; i < per; ++i) {
    const int e = lane + 32 * i;
    if (e < p.G && c64[e] > -INFINITY && (p.n_group == 1 || ((kept >> (e / p.group_size)) & 1u))) open |= 1u << i;
  }
  double sum = 0.0;
  int n = 0;
  for (; n < p.k; ++n) {
    double best = -INFINITY;
    int be = 0x7fffffff;
    for (int i = 0; i < per; ++i)
      if ((open >> i) & 1u) {
        const double c = c64[lane + 32 * i];
        if (c > best) {
          best = c;
          be = lane + 32 * i;
        }
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double oc = __shfl_xor_sync(kFull, best, o);
      const int oe = __shfl_xor_sync(kFull, be, o);
      if (oc > best || (oc == best && oe < be)) {
        best = oc;
        be = oe;
      }
    }
    if (be == 0x7fffffff) break;
    if ((be & 31) == lane) open &= ~(1u << (be >> 5));
    const double s = score64(p, load_logit(p, t * p.ld, be), lmax, rz);
    sum += s;
    if (lane == 0) {
      p.topk_ids[t * p.k + n] = be;
      p.topk_weights[t * p.k + n] = float(s * double(p.scale));
    }
  }
  __syncwarp();
  for (int r = lane; r < p.k; r += 32) {
    if (r >= n) {
      p.topk_ids[t * p.k + r] = -1;
      p.topk_weights[t * p.k + r] = 0.f;
    } else if (p.renormalize) {
      const int e = p.topk_ids[t * p.k + r];
      const double s = score64(p, load_logit(p, t * p.ld, e), lmax, rz);
      p.topk_weights[t * p.k + r] = sum > 0.0 ? float(s / sum * double(p.scale)) : 0.f;
    }
  }
  __syncwarp();
}

// One token by one warp, with router_scratch_bytes() of shared memory of its own.
template <int PER>
__device__ __forceinline__ void route_token(const RouterArgs& p, int64_t t, uint8_t* scratch) {
  const int lane = threadIdx.x & 31;
  double* c64 = reinterpret_cast<double*>(scratch);
  float* c32 = reinterpret_cast<float*>(scratch);
  uint64_t* keys = reinterpret_cast<uint64_t*>(scratch + (size_t(p.G) * 8 + 15) / 16 * 16);
  int* cand_e = reinterpret_cast<int*>(keys + 32);
  float* cand_l = reinterpret_cast<float*>(cand_e + 32);

  float l[PER], c[PER];
  if (p.dtype == CHORD_DTYPE_F32) {
    const float* row = static_cast<const float*>(p.logits) + t * p.ld;
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = lane + 32 * i < p.G ? masked_logit(__ldcg(row + lane + 32 * i), kLowestF32) : -INFINITY;
  } else {
    const uint16_t* row = static_cast<const uint16_t*>(p.logits) + t * p.ld;
    const bool half = p.dtype == CHORD_DTYPE_F16;
    const float lowest = half ? kLowestF16 : kLowestBf16;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t bits = lane + 32 * i < p.G ? __ldcg(row + lane + 32 * i) : 0u;
      const float v = half ? __half2float(__ushort_as_half(uint16_t(bits))) : __uint_as_float(bits << 16);
      l[i] = lane + 32 * i < p.G ? masked_logit(v, lowest) : -INFINITY;
    }
  }
  float b[PER];
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < PER; ++i) b[i] = lane + 32 * i < p.G ? p.bias[lane + 32 * i] : 0.f;
  }
  float lmax = 0.f, rz32 = 1.f;
  if (p.score == CHORD_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    lmax = m > -INFINITY ? m : 0.f;
    if (p.bias || !p.renormalize) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) z += expf(l[i] - lmax);  // exp(-inf) = 0 for masked experts
      z = warp_sum(z);
      rz32 = z > 0.f ? __fdiv_rn(1.f, z) : 1.f;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    c[i] = !p.bias ? l[i] : l[i] > -INFINITY ? score32(p, l[i], lmax, rz32) + b[i] : -INFINITY;

  if (p.n_group > 1) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      if (e < p.G) c32[e] = c[i];
    }
    __syncwarp();
    bool near;
    const uint32_t kept = kept_groups<float>(p, c32, lmax, &near);
    if (near) {
      route_exact(p, t, lmax, c64);
      return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t g = uint32_t((uint64_t(lane + 32 * i) * p.group_magic) >> 32);
      if (!((kept >> (g & 31)) & 1u)) c[i] = -INFINITY;
    }
  }

  // threshold: the k-th largest lane maximum, the least of those with fewer than k above
  float thr = -INFINITY;
  bool fits = p.k <= 32;
  if (fits) {
    float best = c[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = fmaxf(best, c[i]);
    cand_l[lane] = best;
    __syncwarp();
    int above = 0;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(cand_l + j);
      above += (o.x > best) + (o.y > best) + (o.z > best) + (o.w > best);
    }
    thr = warp_min(above < p.k ? best : INFINITY);
    if (p.bias && thr > -INFINITY) thr -= 2.f * kSlackAbs + 2.f * kSlackRel * fabsf(thr);
    __syncwarp();
  }
  int n = 0;
  if (fits) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = c[i] >= thr && c[i] > -INFINITY;
      const uint32_t who = __ballot_sync(kFull, in);
      const int at = n + __popc(who & ((1u << lane) - 1u));
      if (in && at < 32) {
        cand_e[at] = lane + 32 * i;
        cand_l[at] = l[i];
      }
      n += __popc(who);
    }
    fits = n <= 32;
  }
  if (!fits) {
    route_exact(p, t, lmax, c64);
    return;
  }
  __syncwarp();
  // candidates stand in increasing id, so a tie goes to the lower lane
  const bool mine = lane < n;
  const int e = mine ? cand_e[lane] : 0;
  const float lc = mine ? cand_l[lane] : 0.f;
  __syncwarp();
  double s = 0.0, rz = double(rz32);
  if (mine) s = score64(p, lc, lmax, rz);
  double key = mine ? (p.bias ? s + double(p.bias[e]) : double(lc)) : -INFINITY;
  int rank = rank_of(key, n, keys);
  if (p.bias && p.score == CHORD_SCORE_SOFTMAX && any_closer(key, n, 2.0 * kSlackAbs)) {
    // the denominator's FP32 error could swap two experts: once more with it in FP64
    rz = softmax_sum64(p, t, lmax);
    if (mine) s = score64(p, lc, lmax, rz);
    if (mine) key = s + double(p.bias[e]);
    rank = rank_of(key, n, keys);
  }
  const bool chosen = mine && rank < p.k;
  if (p.renormalize) {
    const double sum = warp_sum(chosen ? s : 0.0);
    s = sum > 0x1p-100 ? s * reciprocal64(sum) : sum > 0.0 ? s / sum : 0.0;
  }
  if (chosen) {
    p.topk_ids[t * p.k + rank] = e;
    p.topk_weights[t * p.k + rank] = float(s * double(p.scale));
  }
  for (int r = n + lane; r < p.k; r += 32) {
    p.topk_ids[t * p.k + r] = -1;
    p.topk_weights[t * p.k + r] = 0.f;
  }
}

// Of a warp: G doubles, 32 64-bit keys, 32 candidates' ids and logits.
__host__ __device__ inline size_t router_scratch_bytes(int G) { return (size_t(G) * 8 + 15) / 16 * 16 + 32 * 16; }

template <int PER>
__global__ void __launch_bounds__(32 * kRouterWarps, PER <= 12 ? 4 : PER <= 16 ? 3 : 2) router_scored_kernel(const __grid_constant__ RouterArgs p) {
  extern __shared__ __align__(16) uint8_t router_smem[];
  grid_dep_wait();
  grid_dep_trigger();
  const int warp = threadIdx.x >> 5;
  uint8_t* scratch = router_smem + warp * router_scratch_bytes(p.G);
  for (int64_t t = int64_t(blockIdx.x) * kRouterWarps + warp; t < p.T; t += int64_t(gridDim.x) * kRouterWarps)
    route_token<PER>(p, t, scratch);
}

// Decode batches in one launch: C CTAs (a cluster) route T / C tokens each, a warp per token,
// then sort the ids together.
constexpr int kFusedWarps = 16;
constexpr int kFusedCtas = 8;
constexpr int kFusedMaxTokens = 2 * kFusedCtas * kFusedWarps;  // two rounds of tokens a warp
constexpr int kFusedMaxSteps = 4;  // 32 tokens x 64 slots a CTA, over 16 x 32 lanes

template <int PER, int C>
__global__ void __launch_bounds__(32 * kFusedWarps) router_scored_align_kernel(
    const __grid_constant__ RouterArgs p, int E, int block_m, int64_t cap, int64_t nblocks, int32_t* sorted_ids,
    int32_t* expert_ids, int32_t* ntp, int32_t* offsets) {
  extern __shared__ __align__(16) uint8_t router_smem[];
  grid_dep_wait();
  grid_dep_trigger();
  const int warp = threadIdx.x >> 5;
  const int rank = C > 1 ? int(cluster_rank()) : 0;
  const int64_t t0 = p.T * rank / C, t1 = p.T * (rank + 1) / C;
#pragma unroll 1
  for (int64_t t = t0 + warp; t < t1; t += kFusedWarps)
    route_token<PER>(p, t, router_smem + warp * router_scratch_bytes(p.G));
  __syncthreads();
  align_body<C, kFusedWarps, kFusedMaxSteps>(p.topk_ids, p.T * p.k, t0 * p.k, t1 * p.k, rank, E, block_m, cap, nblocks,
                                             sorted_ids, expert_ids, ntp, offsets,
                                             reinterpret_cast<int*>(router_smem));
}

// Larger batches sort by one cluster of kSortCtas CTAs of 32 warps, up to MAXS steps a warp;
// still larger ones by the kernels of align.cu. 65536 slots of 48 experts take 9 us after the
// router, against 21 of the three kernels.
constexpr int kSortCtas = 8;
template <int MAXS>
constexpr int64_t kClusterSlots = int64_t(kSortCtas) * 32 * 32 * MAXS;

template <int MAXS>
__global__ void __launch_bounds__(1024) sort_cluster_kernel(const int32_t* ids, int64_t n, int E, int block_m,
                                                            int64_t cap, int64_t nblocks, int32_t* sorted_ids,
                                                            int32_t* expert_ids, int32_t* ntp, int32_t* offsets) {
  extern __shared__ __align__(16) uint8_t router_smem[];
  grid_dep_wait();
  grid_dep_trigger();
  const int rank = int(cluster_rank());
  align_body<kSortCtas, 32, MAXS>(ids, n, n * rank / kSortCtas, n * (rank + 1) / kSortCtas, rank, E, block_m, cap,
                                  nblocks, sorted_ids, expert_ids, ntp, offsets, reinterpret_cast<int*>(router_smem));
}

// The most that 1024 experts need in any of these kernels is 152 KiB.
constexpr int kMaxSmem = 160 * 1024;

// Launches `kern` as clusters of `ctas` CTAs, one cluster in all, early.
template <typename... Params, typename... Args>
cudaError_t launch_one_cluster(void (*kern)(Params...), std::atomic<bool> (&allowed)[kMaxSettingDevices], int ctas,
                               int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), kMaxSmem, allowed);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kern, args...);
  count_launches(1);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <int PER, int C>
cudaError_t launch_fused(const RouterArgs& p, int E, int block_m, int64_t cap, int64_t nblocks, int32_t* sorted_ids,
                         int32_t* expert_ids, int32_t* ntp, int32_t* offsets, cudaStream_t stream) {
  const size_t route = router_scratch_bytes(p.G) * kFusedWarps, sort = align_smem_bytes<kFusedWarps>(E);
  static std::atomic<bool> allowed[kMaxSettingDevices];
  return launch_one_cluster(router_scored_align_kernel<PER, C>, allowed, C, 32 * kFusedWarps, route > sort ? route : sort, stream,
                            p, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets);
}

template <int MAXS>
cudaError_t launch_sort(const int32_t* ids, int64_t n, int E, int block_m, int64_t cap, int64_t nblocks,
                        int32_t* sorted_ids, int32_t* expert_ids, int32_t* ntp, int32_t* offsets, cudaStream_t stream) {
  static std::atomic<bool> allowed[kMaxSettingDevices];
  return launch_one_cluster(sort_cluster_kernel<MAXS>, allowed, kSortCtas, 1024, align_smem_bytes<32>(E), stream, ids, n, E,
                            block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets);
}

template <int PER>
cudaError_t launch_per(const RouterArgs& p, int E, int block_m, int64_t cap, int64_t nblocks, int32_t* sorted_ids,
                       int32_t* expert_ids, int32_t* ntp, int32_t* offsets, void* workspace, int num_sms,
                       cudaStream_t stream) {
  if (p.T <= kFusedWarps)
    return launch_fused<PER, 1>(p, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, stream);
  if (p.T <= kFusedMaxTokens)
    return launch_fused<PER, kFusedCtas>(p, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, stream);
  const size_t route = router_scratch_bytes(p.G) * kRouterWarps;
  static std::atomic<bool> allowed[kMaxSettingDevices];
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(router_scored_kernel<PER>), kMaxSmem, allowed);
  if (err != cudaSuccess) return err;
  const int64_t want = (p.T + kRouterWarps - 1) / kRouterWarps, most = int64_t(num_sms) * 8;
  err = launch_pdl(true, router_scored_kernel<PER>, dim3(unsigned(want < most ? want : most)), dim3(32 * kRouterWarps),
                   route, stream, p);
  count_launches(1);
  if (err == cudaSuccess) err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const int64_t n = p.T * p.k;
  if (n <= kClusterSlots<8>)
    return launch_sort<8>(p.topk_ids, n, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, stream);
  if (n <= kClusterSlots<32>)
    return launch_sort<32>(p.topk_ids, n, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, stream);
  return launch_align(p.topk_ids, n, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, workspace, stream);
}

}  // namespace

cudaError_t launch_router_scored(const RouterArgs& p, int E, int block_m, int64_t cap, int64_t nblocks,
                                 int32_t* sorted_ids, int32_t* expert_ids, int32_t* ntp, int32_t* offsets,
                                 void* workspace, int num_sms, cudaStream_t stream) {
  const int per = (p.G + 31) / 32;  // the smallest instantiated count that covers G
  if (per <= 4)
    return launch_per<4>(p, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, workspace, num_sms, stream);
  if (per <= 8)
    return launch_per<8>(p, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, workspace, num_sms, stream);
  if (per <= 12)
    return launch_per<12>(p, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, workspace, num_sms, stream);
  if (per <= 16)
    return launch_per<16>(p, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, workspace, num_sms, stream);
  return launch_per<32>(p, E, block_m, cap, nblocks, sorted_ids, expert_ids, ntp, offsets, workspace, num_sms, stream);
}

}  // namespace chord
