// fp8_api.cu -- entry points of the FP8 block-128 operators: argument checks, the choice of
// the schedule and the launch sequence.
#include <math.h>

#include "fp8.cuh"

namespace chord {

Fp8Workspace fp8_workspace(int64_t rows, int E) {
  const GroupedWorkspace g = grouped_workspace(rows, E);
  Fp8Workspace w;
  w.max_positions = g.max_positions;
  w.ntp_offset = g.ntp_offset;
  w.expert_ids_offset = g.expert_ids_offset;
  w.block_row0_offset = g.block_row0_offset;
  w.sorted_ids_offset = g.sorted_ids_offset;
  w.total = g.partial_offset;  // the unit lists end where the W4A16 GEMM's partial sums begin
  return w;
}

namespace {

bool misaligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1); }

chord_status_t check_rows(int64_t rows) {
  if (rows < 0) return fail(CHORD_ERR_INVALID_ARG, "rows=%lld", (long long)rows);
  // the unit lists number up to two positions a row in 32 bits
  if (rows >= int64_t(1) << 30) return fail(CHORD_ERR_UNSUPPORTED, "rows=%lld >= 2^30", (long long)rows);
  return CHORD_OK;
}

// Shapes, flags and alignment that all products share.
chord_status_t check_product(const uint8_t* xq, const float* xs, int64_t rows, int K, const uint8_t* w,
                             const float* ws, int E, int N, const void* out, const void* workspace, size_t have,
                             size_t need, int flags) {
  if (E < 1 || E > 1024) return fail(CHORD_ERR_UNSUPPORTED, "E=%d outside [1, 1024]", E);
  if (K < 16 || K % 16 || N < 8 || N % 8)
    return fail(CHORD_ERR_UNSUPPORTED, "K=%d must be a positive multiple of 16 and N=%d of 8", K, N);
  if (int64_t(E) * N >= (int64_t(1) << 31)) return fail(CHORD_ERR_UNSUPPORTED, "E=%d times N=%d >= 2^31", E, N);
  const chord_status_t st = check_rows(rows);
  if (st != CHORD_OK) return st;
  if (flags & ~(CHORD_FLAG_FORCE_STREAM | CHORD_FLAG_FORCE_TENSOR | CHORD_FLAG_OUTPUT_FP32))
    return fail(CHORD_ERR_INVALID_ARG, "flags=0x%x", unsigned(flags));
  if ((flags & CHORD_FLAG_FORCE_STREAM) && (flags & CHORD_FLAG_FORCE_TENSOR))
    return fail(CHORD_ERR_INVALID_ARG, "FORCE_STREAM and FORCE_TENSOR are exclusive");
  if (!w || !ws || !workspace) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  if (rows > 0 && (!xq || !xs || !out)) return fail(CHORD_ERR_INVALID_ARG, "null activation or output pointer");
  if (misaligned(workspace, 256)) return fail(CHORD_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  if (misaligned(xq, 16) || misaligned(w, 16) || misaligned(out, 16))
    return fail(CHORD_ERR_INVALID_ARG, "xq, w and out must be 16-byte aligned");
  if (misaligned(xs, 4) || misaligned(ws, 4)) return fail(CHORD_ERR_INVALID_ARG, "scales must be 4-byte aligned");
  if (have < need)
    return fail(CHORD_ERR_WORKSPACE_TOO_SMALL, "FP8 workspace needs %zu bytes, got %zu", need, have);
  return CHORD_OK;
}

Fp8Args product_args(const uint8_t* xq, const float* xs, int64_t rows, int K, const uint8_t* w, const float* ws,
                     int E, int N, void* out, void* workspace, int flags, int layout, int num_sms) {
  Fp8Args a{};
  a.xq = xq;
  a.xs = xs;
  a.w = w;
  a.ws = ws;
  a.out = out;
  a.rows = rows;
  a.K = K;
  a.N = N;
  a.E = E;
  a.layout = layout;
  a.out_f32 = (flags & CHORD_FLAG_OUTPUT_FP32) != 0;
  a.status = static_cast<uint32_t*>(workspace);
  a.num_sms = num_sms;
  return a;
}

// CTAs that share an item of the streaming kernel: as many as keep the likely items within
// one wave, each with two k blocks at least.
int stream_split(int64_t items, int KB, int64_t slots) {
  int split = 1;
  while (split < 8 && items * split * 2 <= slots && KB >= 4 * split) split *= 2;
  return split;
}

// Estimates of the streaming kernel with units of 16, 32 and 64 rows, in us: to start, and per k
// block of an item.
constexpr double kStreamStart[3] = {4.6, 5.0, 6.4}, kStreamPerKb[3] = {0.37, 0.39, 0.52};

struct Plan {
  bool tensor;  // the tile kernel (fp8_tile.cu) or the streaming one (fp8_stream.cu)
  int bm;       // rows of a unit
  int split;    // streaming: CTAs that share an item
  double us;    // estimate
};

// The schedule with the least estimated time. An estimate is a start-up time plus, for each
// wave of the CTAs, the k blocks of an item times a time per block (and a time per tile),
// fitted to measurements on a B200 over M = 8 .. 4096 of 4096 x 7168, 7168 x 2048, 512 x 7168,
// 576 x 1520 and 7168 x 256 (N x K); it lies within a quarter of them. On both sides of some
// borders, in us, for 64-row streaming, 128 x 128 and 256 x 256 tiles: 4096 x 7168 M=128 14.3,
// 17.5, 29.1; M=512 35.3, 19.0, 29.5; M=1024 -, 33.8, 31.0; M=4096 -, 121, 115; 512 x 7168 M=512
// 12.1, 17.4, 28.6; 7168 x 2048 M=512 26, 12.9, 13.0. 48 experts (contiguous) of 7168 x 2048 with
// one block each 216, 145, 203, two 482, 240, 211. `expected`: rows per expert; masked experts
// are taken to hold up to 1.25 times as many.
Plan choose_plan(const Fp8Args& a, int64_t expected, int flags) {
  const int KB = fp8_blocks(a.K);
  // contiguous: every 128-row block is a unit, or several; pairs of an expert's blocks are units
  // of 256 rows where experts have more than one
  const int64_t blocks = (a.rows + 127) / 128;
  auto units_of = [&](int bm) -> int64_t {
    if (a.layout == kFp8Dense) return (a.rows + bm - 1) / bm;
    if (a.layout == kFp8Masked) return a.E * int64_t(ceil(1.25 * expected / bm));
    if (bm <= 128) return blocks * (128 / bm);
    return 2 * blocks >= 3 * int64_t(a.E) ? (blocks + 1) / 2 : blocks;
  };
  auto waves = [](int64_t items, int64_t slots) { return double((items + slots - 1) / slots); };
  Plan best{};
  best.us = 1e30;
  auto offer = [&](bool tensor, int bm, int split, double us) {
    if (us < best.us) best = Plan{tensor, bm, split, us};
  };
  if (!(flags & CHORD_FLAG_FORCE_TENSOR)) {
    const int64_t slots = int64_t(a.num_sms) * kFp8StreamCtas, tiles = (a.N + 127) / 128;
    for (int i = 0; i < 3; ++i) {
      const int bm = 16 << i;
      const int64_t items = units_of(bm) * tiles;
      int split = stream_split(items, KB, slots);
      // a split grid covers every unit there may be, so it has to stay small
      const int64_t most = ((a.rows + bm - 1) / bm + (a.layout == kFp8Dense ? 0 : a.E)) * tiles;
      if (most * split > 8 * slots) split = 1;
      offer(false, bm, split, kStreamStart[i] + waves(items * split, slots) * ((KB + split - 1) / split) * kStreamPerKb[i]);
    }
  }
  if (!(flags & CHORD_FLAG_FORCE_STREAM)) {
    const double small = waves(units_of(128) * ((a.N + 127) / 128), a.num_sms);
    offer(true, 128, 1, 2.6 + small * (KB * (small > 3 ? 0.275 : 0.265) + 1.4));
    offer(true, 256, 1, 3.0 + waves(units_of(256) * ((a.N + 255) / 256), a.num_sms / 2) * (KB * 0.485 + 0.9));
  }
  return best;
}

// The product by the schedule chosen for `expected` rows per expert.
chord_status_t run_product(Fp8Args a, int64_t expected, const int32_t* m_indices, const int32_t* masked_m,
                           int64_t max_m, void* workspace, int flags, cudaStream_t stream) {
  if (expected > a.rows) expected = a.rows;
  const Plan plan = choose_plan(a, expected, flags);
  const bool tensor = plan.tensor;
  a.bm = plan.bm;
  cudaError_t err;
  if (a.layout != kFp8Dense) {
    const Fp8Workspace ws = fp8_workspace(a.rows, a.E);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    int32_t* ntp = reinterpret_cast<int32_t*>(base + ws.ntp_offset);
    int32_t* expert_ids = reinterpret_cast<int32_t*>(base + ws.expert_ids_offset);
    int32_t* block_row0 = reinterpret_cast<int32_t*>(base + ws.block_row0_offset);
    int32_t* sorted_ids = reinterpret_cast<int32_t*>(base + ws.sorted_ids_offset);
    err = launch_grouped_route(m_indices, a.rows, masked_m, a.E, max_m, a.bm, expert_ids, block_row0, sorted_ids, ntp,
                               a.status, stream);
    if (err != cudaSuccess) return cuda_fail(err, "FP8 grouped routing launch");
    a.ntp = ntp;
    a.expert_ids = expert_ids;
    a.block_row0 = block_row0;
    a.sorted_ids = sorted_ids;
  }
  err = tensor ? launch_fp8_tile(a, stream) : launch_fp8_stream(a, plan.split, stream);
  return err == cudaSuccess ? CHORD_OK : cuda_fail(err, tensor ? "FP8 tensor-core GEMM launch" : "FP8 streaming GEMM launch");
}

// The same for gate_up (a.N = 2 I): streaming by clusters of 2 x split CTAs or 256-row x 128-column
// tiles, both ending in the quantised SiLU(gate) * up; or, for up to kTwoStepRows rows (split = 0),
// the product in FP32 and a quantisation. In us for 4096 x 7168: M=16 9.6, 31.9, 11.7; M=128
// 15.3, 32.1, 19.2; M=512 -, 33.2, 26.7; M=1024 -, 34.8, 39.4.
constexpr int64_t kTwoStepRows = 1024;
Plan choose_gate_up(const Fp8Args& a, int flags) {
  const int KB = fp8_blocks(a.K);
  Plan best{};
  best.us = 1e30;
  if (!(flags & CHORD_FLAG_FORCE_TENSOR)) {
    const int64_t slots = int64_t(a.num_sms) * kFp8StreamCtas;
    for (int i = 0; i < 3; ++i) {
      const int bm = 16 << i;
      const int64_t items = (a.rows + bm - 1) / bm * (a.N / 256);
      const int most = stream_split(2 * items, KB, slots), split = most < 4 ? most : 4;
      const double us = kStreamStart[i] + 1.0 +
                        double((2 * items * split + slots - 1) / slots) * ((KB + split - 1) / split) * kStreamPerKb[i];
      if (us < best.us) best = Plan{false, bm, split, us};
    }
  }
  if (!(flags & CHORD_FLAG_FORCE_STREAM)) {
    const int64_t tiles = (a.rows + 255) / 256 * (a.N / 256), pairs = a.num_sms / 2;
    const double us = 3.0 + double((tiles + pairs - 1) / pairs) * (KB * 0.485 + 2.0);
    if (us < best.us) best = Plan{true, 256, 1, us};
  }
  if (!(flags & (CHORD_FLAG_FORCE_TENSOR | CHORD_FLAG_FORCE_STREAM)) && a.rows <= kTwoStepRows) {
    const double us = choose_plan(a, a.rows, flags).us + 4.5 + double(a.rows) * a.N * 8 / 5e6;
    if (us < best.us) best = Plan{false, 0, 0, us};
  }
  return best;
}

chord_status_t quantize(const void* x, int dtype, int64_t ld, int64_t rows, int K, int silu, const int32_t* masked_m,
                        int E, uint8_t* q, float* scales, cudaStream_t stream) {
  if (K < 16 || K % 16 || K >= (1 << 30))
    return fail(CHORD_ERR_UNSUPPORTED, "%d columns: a positive multiple of 16 is needed", K);
  chord_status_t st = check_rows(rows);
  if (st != CHORD_OK) return st;
  if (dtype != CHORD_DTYPE_F32 && dtype != CHORD_DTYPE_BF16)
    return fail(CHORD_ERR_UNSUPPORTED, "dtype=%d: FP32 or BF16 is needed", dtype);
  const int64_t width = silu ? 2 * int64_t(K) : K;
  const int size = dtype == CHORD_DTYPE_F32 ? 4 : 2;
  if (ld < width || ld % (16 / size))
    return fail(CHORD_ERR_INVALID_ARG, "row distance %lld must be >= %lld and a multiple of 16 bytes", (long long)ld,
                (long long)width);
  if (masked_m && (E < 1 || E > 1024 || rows % E))
    return fail(CHORD_ERR_INVALID_ARG, "rows=%lld are not E=%d times max_m", (long long)rows, E);
  if (!masked_m && E != 0) return fail(CHORD_ERR_INVALID_ARG, "E=%d without masked_m", E);
  if (rows == 0) return CHORD_OK;
  if (!x || !q || !scales) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  if (misaligned(x, 16) || misaligned(q, 16) || misaligned(scales, 4))
    return fail(CHORD_ERR_INVALID_ARG, "x and q must be 16-byte and scales 4-byte aligned");
  if ((st = current_device(nullptr)) != CHORD_OK) return st;
  Fp8QuantArgs a{};
  a.x = x;
  a.dtype = dtype;
  a.ld = ld;
  a.rows = rows;
  a.K = K;
  a.silu = silu;
  a.masked_m = masked_m;
  a.max_m = masked_m ? rows / E : rows;
  a.q = q;
  a.scales = scales;
  const cudaError_t err = launch_fp8_quantize(a, stream);
  return err == cudaSuccess ? CHORD_OK : cuda_fail(err, "FP8 quantise launch");
}

}  // namespace
}  // namespace chord

using namespace chord;

extern "C" {

size_t chord_fp8_workspace_bytes(int64_t rows, int E) {
  if (rows < 0 || E < 1) return 0;
  return size_t(fp8_workspace(rows, E).total);
}

chord_status_t chord_fp8_quantize(const void* x, int x_dtype, int64_t ldx, int64_t rows, int K,
                                  const int32_t* masked_m, int E, uint8_t* q, float* scales, chord_stream_t stream) {
  clear_detail();
  return quantize(x, x_dtype, ldx, rows, K, 0, masked_m, E, q, scales, reinterpret_cast<cudaStream_t>(stream));
}

chord_status_t chord_fp8_silu_quantize(const void* h, int h_dtype, int64_t ldh, int64_t rows, int I,
                                       const int32_t* masked_m, int E, uint8_t* q, float* scales,
                                       chord_stream_t stream) {
  clear_detail();
  return quantize(h, h_dtype, ldh, rows, I, 1, masked_m, E, q, scales, reinterpret_cast<cudaStream_t>(stream));
}

chord_status_t chord_fp8_gemm(const uint8_t* xq, const float* xs, int64_t M, int K, const uint8_t* w, const float* ws,
                              int N, void* out, void* workspace, size_t workspace_bytes, int flags,
                              chord_stream_t stream) {
  clear_detail();
  chord_status_t st = check_product(xq, xs, M, K, w, ws, 1, N, out, workspace, workspace_bytes,
                                    M < 0 ? 0 : chord_fp8_workspace_bytes(M, 1), flags);
  if (st != CHORD_OK) return st;
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != CHORD_OK) return st;
  if (M == 0) return CHORD_OK;
  return run_product(product_args(xq, xs, M, K, w, ws, 1, N, out, workspace, flags, kFp8Dense, num_sms), M, nullptr,
                     nullptr, 0, workspace, flags, reinterpret_cast<cudaStream_t>(stream));
}

chord_status_t chord_fp8_grouped_contiguous(const uint8_t* xq, const float* xs, int64_t M, int K,
                                            const int32_t* m_indices, const uint8_t* w, const float* ws, int E, int N,
                                            void* out, void* workspace, size_t workspace_bytes, int flags,
                                            chord_stream_t stream) {
  clear_detail();
  chord_status_t st = check_product(xq, xs, M, K, w, ws, E, N, out, workspace, workspace_bytes,
                                    M < 0 ? 0 : chord_fp8_workspace_bytes(M, E), flags);
  if (st != CHORD_OK) return st;
  if (M > 0 && !m_indices) return fail(CHORD_ERR_INVALID_ARG, "null m_indices");
  if (misaligned(m_indices, 16)) return fail(CHORD_ERR_INVALID_ARG, "m_indices must be 16-byte aligned");
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != CHORD_OK) return st;
  if (M == 0) return CHORD_OK;
  return run_product(product_args(xq, xs, M, K, w, ws, E, N, out, workspace, flags, kFp8Contiguous, num_sms),
                     (M + E - 1) / E, m_indices, nullptr, 0, workspace, flags, reinterpret_cast<cudaStream_t>(stream));
}

chord_status_t chord_fp8_grouped_masked(const uint8_t* xq, const float* xs, int E, int64_t max_m, int K,
                                        const int32_t* masked_m, int64_t expected_m, const uint8_t* w,
                                        const float* ws, int N, void* out, void* workspace, size_t workspace_bytes,
                                        int flags, chord_stream_t stream) {
  clear_detail();
  if (max_m < 1 || expected_m < 1)
    return fail(CHORD_ERR_INVALID_ARG, "max_m=%lld expected_m=%lld", (long long)max_m, (long long)expected_m);
  if (max_m >= (int64_t(1) << 31)) return fail(CHORD_ERR_UNSUPPORTED, "max_m=%lld", (long long)max_m);
  if (E < 1 || E > 1024) return fail(CHORD_ERR_UNSUPPORTED, "E=%d outside [1, 1024]", E);
  const int64_t rows = int64_t(E) * max_m;
  chord_status_t st = check_product(xq, xs, rows, K, w, ws, E, N, out, workspace, workspace_bytes,
                                    chord_fp8_workspace_bytes(rows, E), flags);
  if (st != CHORD_OK) return st;
  if (!masked_m) return fail(CHORD_ERR_INVALID_ARG, "null masked_m");
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != CHORD_OK) return st;
  return run_product(product_args(xq, xs, rows, K, w, ws, E, N, out, workspace, flags, kFp8Masked, num_sms),
                     expected_m, nullptr, masked_m, max_m, workspace, flags, reinterpret_cast<cudaStream_t>(stream));
}

size_t chord_fp8_gate_up_workspace_bytes(int64_t M, int I) {
  if (M < 0 || I < 1) return 0;
  const int64_t sums = M < kTwoStepRows ? M : kTwoStepRows;  // FP32, rows of the two-step form
  return chord_fp8_workspace_bytes(M, 1) + size_t(align256(uint64_t(sums) * 2 * I * 4));
}

chord_status_t chord_fp8_gate_up(const uint8_t* xq, const float* xs, int64_t M, int H, const uint8_t* w13,
                                 const float* ws13, int I, uint8_t* q, float* scales, void* workspace,
                                 size_t workspace_bytes, int flags, chord_stream_t stream) {
  clear_detail();
  if (I < kFp8Block || I % kFp8Block || I >= (1 << 29))
    return fail(CHORD_ERR_UNSUPPORTED, "I=%d must be a positive multiple of 128", I);
  if (flags & CHORD_FLAG_OUTPUT_FP32) return fail(CHORD_ERR_INVALID_ARG, "the output of gate_up is FP8");
  chord_status_t st = check_product(xq, xs, M, H, w13, ws13, 1, 2 * I, q, workspace, workspace_bytes,
                                    M < 0 ? 0 : chord_fp8_gate_up_workspace_bytes(M, I), flags);
  if (st != CHORD_OK) return st;
  if (M > 0 && !scales) return fail(CHORD_ERR_INVALID_ARG, "null scales");
  if (misaligned(scales, 4)) return fail(CHORD_ERR_INVALID_ARG, "scales must be 4-byte aligned");
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != CHORD_OK) return st;
  if (M == 0) return CHORD_OK;
  Fp8Args a = product_args(xq, xs, M, H, w13, ws13, 1, 2 * I, q, workspace, flags, kFp8Dense, num_sms);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const Plan plan = choose_gate_up(a, flags);
  if (plan.split == 0) {
    a.out = static_cast<uint8_t*>(workspace) + chord_fp8_workspace_bytes(M, 1);
    a.out_f32 = 1;
    st = run_product(a, M, nullptr, nullptr, 0, workspace, flags, cs);
    if (st != CHORD_OK) return st;
    return quantize(a.out, CHORD_DTYPE_F32, 2 * int64_t(I), M, I, 1, nullptr, 0, q, scales, cs);
  }
  a.out_scales = scales;
  a.bm = plan.bm;
  const cudaError_t err = plan.tensor ? launch_fp8_tile_gate_up(a, cs) : launch_fp8_stream_gate_up(a, plan.split, cs);
  return err == cudaSuccess ? CHORD_OK : cuda_fail(err, "FP8 gate_up launch");
}

}  // extern "C"
