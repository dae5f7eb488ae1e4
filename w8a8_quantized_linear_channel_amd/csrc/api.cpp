// C ABI of libq8: argument validation, workspace carving and kernel dispatch.
// Every check that needs no device runs first, so argument errors are
// reported before any HIP call (and can be exercised on a machine without a
// GPU); then the device of the stream is checked once per device and cached.
#include "q8.h"
#include "q8_bench.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include "q8_bench_kernels.hpp"
#include "q8_group.hpp"
#include "q8_kernels.hpp"
#include "q8_kv.hpp"
#include "q8_linear_impl.hpp"

namespace {

constexpr int64_t kMaxK = 65536;          // keeps acc - Z*rowsum inside int32 (|.| <= 32512 K)
constexpr int64_t kMaxRows = (1LL << 31) - 1;
constexpr size_t kAlign = 256;
constexpr int64_t kMaxTokens = 1LL << 30;       // of one batch over the cache, and of a window
constexpr int64_t kMaxMaskWords = 1 << 15;      // of a drafted token's mask (64 tokens each)
constexpr int kMaxLayers = 512;                 // of one call over the caches of all layers
constexpr int64_t kMaxGroups = 1024;            // experts of one grouped call (the kernels' bound)

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(int d) { return d == Q8_F32 || d == Q8_F16 || d == Q8_BF16; }

// M rows of K; min_m = 0 admits an empty batch of activations
q8_status check_mk(int64_t M, int64_t K, int64_t min_m = 1) {
  if (M < min_m || K < 1 || M > kMaxRows) return Q8_ERR_BAD_SHAPE;
  if (K % 16 != 0 || K > kMaxK) return Q8_ERR_BAD_SHAPE;
  return Q8_OK;
}

// M activation rows (0: an empty batch), N weight rows, K features
q8_status check_mnk(int64_t M, int64_t N, int64_t K) {
  q8_status s = check_mk(M, K, 0);
  if (s != Q8_OK) return s;
  if (N < 1 || N > kMaxRows) return Q8_ERR_BAD_SHAPE;
  // the GEMM indexes its operands and output with 32-bit offsets
  if (M * K > kMaxRows || N * K > kMaxRows || M * N > kMaxRows) return Q8_ERR_BAD_SHAPE;
  return Q8_OK;
}

// Bump allocator over the caller's workspace; every piece 256-byte aligned.
struct Carve {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off = (off + bytes + kAlign - 1) / kAlign * kAlign;
    return o;
  }
};

// The int8 product and epilogue on quantized activations: the streaming GEMV
// for decode-sized M, the MFMA GEMM tiles above.
hipError_t int8_on_codes(const int8_t* xq, const float* xs, const int32_t* rs, int64_t M, int64_t K,
                         const int8_t* wq, const float* w_scale, const float* w_zp, int64_t N, const float* bias,
                         void* y, int y_dtype, int32_t* acc_out, hipStream_t st, double y_inv = 0.0) {
  if (M <= q8::kGemvMaxM)
    return q8::launch_gemv_q8(xq, xs, rs, M, K, wq, w_scale, w_zp, N, bias, y, y_dtype, acc_out, st, y_inv);
  q8::GemmArgs g{};
  g.a = reinterpret_cast<const uint8_t*>(xq);
  g.b = reinterpret_cast<const uint8_t*>(wq);
  g.a_scale = xs;
  g.a_rowsum = rs;
  g.b_scale = w_scale;
  g.b_zp = w_zp;
  g.bias = bias;
  g.y = y;
  g.acc_out = acc_out;
  g.M = M;
  g.N = N;
  g.K = K;
  g.y_inv = y_inv;
  return q8::launch_gemm(q8::GEMM_INT8, g, y_dtype, st);
}

struct LinearWs { size_t xq, xs, rs, total; };

// Static path: the codes, the per-row copy of the static scale and the code
// sums always pass through the workspace.
LinearWs static_ws(int64_t M, int64_t K) {
  Carve c;
  LinearWs w;
  w.xq = c.take((size_t)M * K);
  w.xs = c.take((size_t)M * 4);
  w.rs = c.take((size_t)M * 4);
  w.total = c.off;
  return w;
}
LinearWs linear_ws(int64_t M, int64_t K) {
  LinearWs w{0, 0, 0, 0};
  if (M <= q8::kGemvFusedMaxM) return w;   // fused decode path: the codes stay in LDS, no scratch
  Carve c;
  w.xq = c.take((size_t)M * K);
  w.xs = c.take((size_t)M * 4);
  w.rs = c.take((size_t)M * 4);
  w.total = c.off;
  return w;
}

// Per-group path: codes, scales and the group code sums [K / group, M], sized
// for the smallest group (64); none for the fused decode path.
struct GroupedWs { size_t xq, xs, gs, total; };
GroupedWs grouped_ws(int64_t M, int64_t K) {
  GroupedWs w{0, 0, 0, 0};
  if (M <= q8::kGemvFusedMaxM) return w;
  Carve c;
  w.xq = c.take((size_t)M * K);
  w.xs = c.take((size_t)M * 4);
  w.gs = c.take((size_t)M * (K / 64) * 4);
  w.total = c.off;
  return w;
}
bool valid_group(int64_t group, int64_t K) { return (group == 64 || group == 128) && K % group == 0; }

// LLM.int8: codes, scales, row sums, column flags, outlier list and count,
// and the fp16 panels of the first kPanelCols outlier columns of X and W.
struct DecompWs { size_t xq, xs, rs, flags, idx, cnt, xp, wp, total; };
DecompWs decomp_ws(int64_t M, int64_t N, int64_t K) {
  if (M == 0) return DecompWs{};   // an empty batch needs no scratch
  Carve c;
  DecompWs w;
  w.xq = c.take((size_t)M * K);
  w.xs = c.take((size_t)M * 4);
  w.rs = c.take((size_t)M * 4);
  w.flags = c.take((size_t)K);
  w.idx = c.take((size_t)K * 4);
  w.cnt = c.take(4);
  w.xp = c.take((size_t)M * q8::kPanelCols * 2);
  w.wp = c.take((size_t)N * q8::kPanelCols * 2);
  w.total = c.off;
  return w;
}

struct Fp8Ws { size_t xq, xs, total; };
Fp8Ws fp8_ws(int64_t M, int64_t K) {
  Carve c;
  Fp8Ws w;
  w.xq = c.take((size_t)M * K);
  w.xs = c.take((size_t)M * 4);
  w.total = c.off;
  return w;
}

// Block-scaled FP8: codes and the scales [ceil(K / 128), M].
Fp8Ws fp8_block_ws(int64_t M, int64_t K) {
  Fp8Ws w{0, 0, 0};
  if (q8::fp8_block_is_fused(M)) return w;      // the codes stay in LDS
  Carve c;
  w.xq = c.take((size_t)M * K);
  w.xs = c.take((size_t)M * ((K + q8::kScaleBlock - 1) / q8::kScaleBlock) * 4);
  w.total = c.off;
  return w;
}

// Sizes shared by the calls on the paged cache.
q8_status check_kv(int64_t T, int64_t Hkv, int64_t D, int64_t S, int64_t max_pages, int64_t max_q, int64_t num_pages,
                   int64_t page) {
  if (T < 0 || T > kMaxTokens || S < 1 || S > 32768 || Hkv < 1 || Hkv > 1024 || max_q < 0 || max_q > kMaxRows)
    return Q8_ERR_BAD_SHAPE;
  if (D != 64 && D != 128 && D != 256) return Q8_ERR_BAD_SHAPE;
  if (page != 32 && page != 64 && page != 128) return Q8_ERR_BAD_SHAPE;
  if (num_pages < 1 || num_pages * Hkv > kMaxRows || num_pages > kMaxRows || max_pages < 1 || max_pages > kMaxRows / page - 256)
    return Q8_ERR_BAD_SHAPE;
  return Q8_OK;
}
// (a sequence's rows, tokens x heads that share a kv head, are counted in 32 bits, a block past the end)
bool valid_heads(int64_t T, int64_t Hq, int64_t Hkv) {
  return Hq >= 1 && Hq <= 65536 && Hq % Hkv == 0 && T <= (kMaxRows - 1024) / (Hq / Hkv);
}

q8::KvView kv_view(const uint8_t* k, const uint8_t* ke, const uint8_t* v, const uint8_t* ve, const int32_t* q_start,
                   const int32_t* kv_len, const int32_t* table, int64_t T, int64_t Hkv, int64_t S, int64_t max_pages,
                   int64_t num_pages, int64_t page) {
  q8::KvView kv{};
  kv.k = const_cast<uint8_t*>(k);
  kv.ke = const_cast<uint8_t*>(ke);
  kv.v = const_cast<uint8_t*>(v);
  kv.ve = const_cast<uint8_t*>(ve);
  kv.q_start = q_start;
  kv.kv_len = kv_len;
  kv.table = table;
  kv.num_pages = (int)num_pages;
  kv.kv_heads = (int)Hkv;
  kv.seqs = (int)S;
  kv.max_pages = (int)max_pages;
  kv.page = (int)page;
  kv.tokens = (int)T;
  return kv;
}

// Splits' partial sums: float [splits, T, Hq, D] and their (maximum, sum) pairs.
struct AttnWs { size_t part, ml, total; };
AttnWs attn_ws(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t S, int64_t max_q, int64_t max_kv, int64_t window,
               bool tree = false) {
  AttnWs w{0, 0, 0};
  if (T == 0) return w;
  const int64_t splits = (tree ? q8::tree_splits : q8::attn_splits)((int)Hq, (int)Hkv, (int)D, (int)S, max_q, max_kv, (int)window);
  if (splits <= 1) return w;
  Carve c;
  w.part = c.take((size_t)splits * T * Hq * D * 4);
  w.ml = c.take((size_t)splits * T * Hq * (tree ? 12 : 8));
  w.total = c.off;
  return w;
}
// max_q and max_kv as the kernels use them: at least 1, at most what can occur
int64_t bound_of(int64_t given, int64_t most) { return given < 1 ? 1 : (given > most ? (most < 1 ? 1 : most) : given); }

// ---- device check: gfx950 only, cached per device
constexpr int kMaxDevices = 64;
std::atomic<int> g_dev_state[kMaxDevices];   // 0 unknown, 1 gfx950, 2 other

q8_status device_of(hipStream_t st, int* dev) {
  if (st != nullptr) {
    if (hipStreamGetDevice(st, dev) != hipSuccess) return Q8_ERR_DEVICE;
  } else if (hipGetDevice(dev) != hipSuccess) {
    return Q8_ERR_DEVICE;
  }
  return (*dev >= 0 && *dev < kMaxDevices) ? Q8_OK : Q8_ERR_DEVICE;
}

q8_status check_device(hipStream_t st) {
  int dev = -1;
  q8_status s = device_of(st, &dev);
  if (s != Q8_OK) {
    (void)hipGetLastError();   // do not leave a sticky error for the caller
    return s;
  }
  int state = g_dev_state[dev].load(std::memory_order_relaxed);
  if (state == 0) {
    hipDeviceProp_t p;
    if (hipGetDeviceProperties(&p, dev) != hipSuccess) {
      (void)hipGetLastError();
      return Q8_ERR_DEVICE;
    }
    state = (std::strncmp(p.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_dev_state[dev].store(state, std::memory_order_relaxed);
  }
  return state == 1 ? Q8_OK : Q8_ERR_DEVICE;
}

// Optional (Q8_DEBUG_VALIDATE=1): every pointer must be device memory of the
// stream's device.
bool debug_validate() {
  static const bool on = [] {
    const char* e = std::getenv("Q8_DEBUG_VALIDATE");
    return e != nullptr && e[0] == '1';
  }();
  return on;
}

q8_status check_ptrs(hipStream_t st, std::initializer_list<const void*> ptrs) {
  if (!debug_validate()) return Q8_OK;
  int dev = -1;
  if (device_of(st, &dev) != Q8_OK) return Q8_ERR_DEVICE;
  for (const void* p : ptrs) {
    if (p == nullptr) continue;
    hipPointerAttribute_t a;
    if (hipPointerGetAttributes(&a, p) != hipSuccess) {
      (void)hipGetLastError();
      return Q8_ERR_BAD_ARG;
    }
    if (a.type != hipMemoryTypeDevice || a.device != dev) return Q8_ERR_BAD_ARG;
  }
  return Q8_OK;
}

q8_status launched(hipError_t e) { return e == hipSuccess ? Q8_OK : Q8_ERR_LAUNCH; }

#define Q8_TRY(expr)                 \
  do {                               \
    const q8_status s_ = (expr);     \
    if (s_ != Q8_OK) return s_;      \
  } while (0)

}  // namespace

namespace q8 {

q8_status linear_check_args(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, const int8_t* wq,
                            const float* w_scale, const float* w_zp, int64_t N, const float* bias, const void* y,
                            q8_dtype y_dtype, const int32_t* acc_out, size_t* workspace_needed) {
  if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mnk(M, N, K));
  if (!wq || !w_scale || !w_zp || (M > 0 && (!x || !y))) return Q8_ERR_NULL_PTR;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(w_zp) || !aligned16(y) ||
      (bias && !aligned16(bias)) || (acc_out && !aligned16(acc_out)))
    return Q8_ERR_ALIGN;
  *workspace_needed = linear_ws(M, K).total;
  return Q8_OK;
}

q8_status linear_run(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, const int8_t* wq, const float* w_scale,
                     const float* w_zp, int64_t N, const float* bias, void* y, q8_dtype y_dtype, void* workspace,
                     int32_t* acc_out, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, wq, w_scale, w_zp, bias, y, workspace, acc_out}));
  if (M == 0) return Q8_OK;

  if (M <= q8::kGemvFusedMaxM)
    return launched(q8::launch_gemv_i8(x, x_dtype, M, K, wq, w_scale, w_zp, N, bias, y, y_dtype,
                                       acc_out, st));

  const LinearWs ws = linear_ws(M, K);
  char* base = static_cast<char*>(workspace);
  int8_t* xq = reinterpret_cast<int8_t*>(base + ws.xq);
  float* xs = reinterpret_cast<float*>(base + ws.xs);
  int32_t* rs = reinterpret_cast<int32_t*>(base + ws.rs);
  Q8_TRY(launched(q8::launch_quant_act_i8(x, x_dtype, M, K, xq, xs, rs, st)));
  return launched(int8_on_codes(xq, xs, rs, M, K, wq, w_scale, w_zp, N, bias, y, y_dtype, acc_out, st));
}

q8_status stream_device(void* stream, int* dev) { return device_of(static_cast<hipStream_t>(stream), dev); }

}  // namespace q8

extern "C" {

const char* q8_status_str(q8_status s) {
  switch (s) {
    case Q8_OK: return "Q8_OK";
    case Q8_ERR_NULL_PTR: return "Q8_ERR_NULL_PTR";
    case Q8_ERR_BAD_SHAPE: return "Q8_ERR_BAD_SHAPE";
    case Q8_ERR_BAD_DTYPE: return "Q8_ERR_BAD_DTYPE";
    case Q8_ERR_BAD_FORMAT: return "Q8_ERR_BAD_FORMAT";
    case Q8_ERR_BAD_ARG: return "Q8_ERR_BAD_ARG";
    case Q8_ERR_ALIGN: return "Q8_ERR_ALIGN";
    case Q8_ERR_WORKSPACE: return "Q8_ERR_WORKSPACE";
    case Q8_ERR_DEVICE: return "Q8_ERR_DEVICE";
    case Q8_ERR_LAUNCH: return "Q8_ERR_LAUNCH";
  }
  return "Q8_ERR_UNKNOWN";
}

size_t q8_workspace_bytes(q8_op op, int64_t M, int64_t N, int64_t K) {
  if (check_mnk(M, N, K) != Q8_OK) return 0;
  switch (op) {
    case Q8_OP_LINEAR: return linear_ws(M, K).total;
    case Q8_OP_DECOMP: return decomp_ws(M, N, K).total;
    case Q8_OP_FP8: return fp8_ws(M, K).total;
    case Q8_OP_STATIC: return static_ws(M, K).total;
    case Q8_OP_GROUPED: return grouped_ws(M, K).total;
    case Q8_OP_FP8_BLOCK: return fp8_block_ws(M, K).total;
  }
  return 0;
}

q8_status q8_quantize_weight(q8_format fmt, const void* w, q8_dtype w_dtype, int64_t N, int64_t K,
                             void* wq, float* w_scale, float* w_zp, void* stream) {
  if (fmt != Q8_INT8_ASYM && fmt != Q8_FP8_E4M3) return Q8_ERR_BAD_FORMAT;
  if (!valid_dtype(w_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mk(N, K));
  if (!w || !wq || !w_scale) return Q8_ERR_NULL_PTR;
  if (fmt == Q8_INT8_ASYM && !w_zp) return Q8_ERR_NULL_PTR;
  if (fmt == Q8_FP8_E4M3 && w_zp) return Q8_ERR_BAD_ARG;
  if (!aligned16(w) || !aligned16(wq) || !aligned16(w_scale) || (w_zp && !aligned16(w_zp)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {w, wq, w_scale, w_zp}));
  if (fmt == Q8_INT8_ASYM)
    return launched(q8::launch_quant_weight_i8(w, w_dtype, N, K, static_cast<int8_t*>(wq), w_scale,
                                               w_zp, st));
  return launched(q8::launch_quant_rows_fp8(w, w_dtype, N, K, INFINITY, static_cast<uint8_t*>(wq),
                                            w_scale, st));
}

q8_status q8_quantize_act(q8_format fmt, const void* x, q8_dtype x_dtype, int64_t M, int64_t K,
                          float scale_ub, void* xq, float* x_scale, int32_t* x_rowsum, void* stream) {
  if (fmt != Q8_INT8_SYM && fmt != Q8_FP8_E4M3) return Q8_ERR_BAD_FORMAT;
  if (!valid_dtype(x_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mk(M, K, 0));
  if (M > 0 && (!x || !xq || !x_scale)) return Q8_ERR_NULL_PTR;
  if (fmt == Q8_FP8_E4M3) {
    if (x_rowsum) return Q8_ERR_BAD_ARG;
    if (std::isnan(scale_ub) || scale_ub <= 0.0f) return Q8_ERR_BAD_ARG;
  }
  if (!aligned16(x) || !aligned16(xq) || !aligned16(x_scale) || (x_rowsum && !aligned16(x_rowsum)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, xq, x_scale, x_rowsum}));
  if (M == 0) return Q8_OK;
  if (fmt == Q8_INT8_SYM)
    return launched(q8::launch_quant_act_i8(x, x_dtype, M, K, static_cast<int8_t*>(xq),
                                            x_scale, x_rowsum, st));
  return launched(q8::launch_quant_rows_fp8(x, x_dtype, M, K, scale_ub, static_cast<uint8_t*>(xq),
                                            x_scale, st));
}

q8_status q8_linear(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, const int8_t* wq,
                    const float* w_scale, const float* w_zp, int64_t N, const float* bias, void* y,
                    q8_dtype y_dtype, void* workspace, size_t workspace_bytes, int32_t* acc_out,
                    void* stream) {
  size_t need = 0;
  Q8_TRY(q8::linear_check_args(x, x_dtype, M, K, wq, w_scale, w_zp, N, bias, y, y_dtype, acc_out, &need));
  if (need > 0 && (!workspace || workspace_bytes < need)) return Q8_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return Q8_ERR_ALIGN;
  return q8::linear_run(x, x_dtype, M, K, wq, w_scale, w_zp, N, bias, y, y_dtype, workspace, acc_out, stream);
}

q8_status q8_linear_int8_decomp(const void* x, int64_t M, int64_t K, const int8_t* wq,
                                const float* w_scale, const float* w_zp, int64_t N, float threshold,
                                const float* bias, void* y, void* workspace, size_t workspace_bytes,
                                int32_t* outlier_idx, int32_t* n_outliers, int32_t* acc_out,
                                void* stream) {
  Q8_TRY(check_mnk(M, N, K));
  if (!wq || !w_scale || !w_zp || (M > 0 && (!x || !y))) return Q8_ERR_NULL_PTR;
  if (std::isnan(threshold)) return Q8_ERR_BAD_ARG;
  const DecompWs ws = decomp_ws(M, N, K);
  if (ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return Q8_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(w_zp) || !aligned16(y) ||
      !aligned16(workspace) || (bias && !aligned16(bias)) || (acc_out && !aligned16(acc_out)) ||
      (outlier_idx && !aligned16(outlier_idx)) || (n_outliers && !aligned16(n_outliers)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, wq, w_scale, w_zp, bias, y, workspace, outlier_idx, n_outliers, acc_out}));
  if (M == 0) {
    // the outlier set of an empty batch is empty: only the count is written,
    // by the quantizer's compaction workgroup alone (no flags, no rows)
    if (n_outliers)
      return launched(q8::launch_quant_act_f16_outliers(nullptr, 0, K, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                        n_outliers, nullptr, nullptr, q8::OutlierPanels{}, st));
    return Q8_OK;
  }

  char* base = static_cast<char*>(workspace);
  int8_t* xq = reinterpret_cast<int8_t*>(base + ws.xq);
  float* xs = reinterpret_cast<float*>(base + ws.xs);
  int32_t* rs = reinterpret_cast<int32_t*>(base + ws.rs);
  uint8_t* flags = reinterpret_cast<uint8_t*>(base + ws.flags);
  int32_t* idx = reinterpret_cast<int32_t*>(base + ws.idx);
  int32_t* cnt = reinterpret_cast<int32_t*>(base + ws.cnt);
  uint16_t* xp = reinterpret_cast<uint16_t*>(base + ws.xp);
  uint16_t* wp = reinterpret_cast<uint16_t*>(base + ws.wp);
  const uint16_t* xh = static_cast<const uint16_t*>(x);

  // threshold <= 0: no outlier columns (the decomposition is off)
  const bool on = threshold > 0.0f;
  if (on) Q8_TRY(launched(q8::launch_outlier_flags(xh, M, K, threshold, flags, st)));
  // the panels are needed only when there can be outlier columns
  const q8::OutlierPanels pan{wq, w_scale, w_zp, N, on ? xp : nullptr, wp};
  Q8_TRY(launched(q8::launch_quant_act_f16_outliers(xh, M, K, on ? flags : nullptr, xq, xs, rs, idx, cnt,
                                                    outlier_idx, n_outliers, pan, st)));
  q8::GemmArgs g{};
  g.a = reinterpret_cast<const uint8_t*>(xq);
  g.b = reinterpret_cast<const uint8_t*>(wq);
  g.a_scale = xs;
  g.a_rowsum = rs;
  g.b_scale = w_scale;
  g.b_zp = w_zp;
  g.bias = bias;
  g.y = y;
  g.acc_out = acc_out;
  g.M = M;
  g.N = N;
  g.K = K;
  g.x_f16 = xh;
  g.out_idx = idx;
  g.out_cnt = cnt;
  g.x_panel = xp;
  g.w_panel = wp;
  return launched(q8::launch_gemm(q8::GEMM_INT8_DECOMP, g, Q8_F16, st));
}

q8_status q8_linear_fp8(const void* x, int64_t M, int64_t K, const uint8_t* wq, const float* w_scale,
                        int64_t N, float scale_ub, const float* bias, void* y, void* workspace,
                        size_t workspace_bytes, void* stream) {
  Q8_TRY(check_mnk(M, N, K));
  if (!wq || !w_scale || (M > 0 && (!x || !y))) return Q8_ERR_NULL_PTR;
  if (std::isnan(scale_ub) || scale_ub <= 0.0f) return Q8_ERR_BAD_ARG;
  const Fp8Ws ws = fp8_ws(M, K);
  if (ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return Q8_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(y) || !aligned16(workspace) ||
      (bias && !aligned16(bias)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, wq, w_scale, bias, y, workspace}));
  if (M == 0) return Q8_OK;

  char* base = static_cast<char*>(workspace);
  uint8_t* xq = reinterpret_cast<uint8_t*>(base + ws.xq);
  float* xs = reinterpret_cast<float*>(base + ws.xs);
  Q8_TRY(launched(q8::launch_quant_rows_fp8(x, Q8_BF16, M, K, scale_ub, xq, xs, st)));
  q8::GemmArgs g{};
  g.a = xq;
  g.b = wq;
  g.a_scale = xs;
  g.b_scale = w_scale;
  g.bias = bias;
  g.y = y;
  g.M = M;
  g.N = N;
  g.K = K;
  return launched(q8::launch_gemm(q8::GEMM_FP8, g, Q8_BF16, st));
}

q8_status q8_linear_fp8_grouped(const void* x, int64_t T, int64_t K, const int32_t* expert_offsets, int64_t E,
                                const uint8_t* wq, const float* w_scale, int64_t N, float scale_ub, void* y,
                                void* workspace, size_t workspace_bytes, void* stream) {
  Q8_TRY(check_mnk(T, N, K));
  if (E < 1 || E > kMaxGroups || E * N > kMaxRows) return Q8_ERR_BAD_SHAPE;
  if (!expert_offsets || !wq || !w_scale || (T > 0 && (!x || !y))) return Q8_ERR_NULL_PTR;
  if (std::isnan(scale_ub) || scale_ub <= 0.0f) return Q8_ERR_BAD_ARG;
  const Fp8Ws ws = fp8_ws(T, K);
  if (ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return Q8_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(y) || !aligned16(workspace) ||
      !aligned4(expert_offsets))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, expert_offsets, wq, w_scale, y, workspace}));
  if (T == 0) return Q8_OK;

  char* base = static_cast<char*>(workspace);
  uint8_t* xq = reinterpret_cast<uint8_t*>(base + ws.xq);
  float* xs = reinterpret_cast<float*>(base + ws.xs);
  // per-token scales do not depend on the expert: one pass over all routed rows
  Q8_TRY(launched(q8::launch_quant_rows_fp8(x, Q8_BF16, T, K, scale_ub, xq, xs, st)));
  q8::GemmArgs g{};
  g.a = xq;
  g.b = wq;
  g.a_scale = xs;
  g.b_scale = w_scale;
  g.y = y;
  g.M = T;
  g.N = N;
  g.K = K;
  g.groups = (int)E;
  g.group_offsets = expert_offsets;
  return launched(q8::launch_gemm_fp8_grouped(g, st));
}

q8_status q8_gemm_int8(const int8_t* xq, const float* x_scale, const int32_t* x_rowsum, int64_t M,
                       int64_t K, const int8_t* wq, const float* w_scale, const float* w_zp, int64_t N,
                       const float* bias, void* y, q8_dtype y_dtype, int32_t* acc_out, void* stream) {
  if (!valid_dtype(y_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mnk(M, N, K));
  if (!wq || !w_scale || !w_zp || (M > 0 && (!xq || !x_scale || !x_rowsum || !y))) return Q8_ERR_NULL_PTR;
  if (!aligned16(xq) || !aligned16(x_scale) || !aligned16(x_rowsum) || !aligned16(wq) ||
      !aligned16(w_scale) || !aligned16(w_zp) || !aligned16(y) || (bias && !aligned16(bias)) ||
      (acc_out && !aligned16(acc_out)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {xq, x_scale, x_rowsum, wq, w_scale, w_zp, bias, y, acc_out}));
  if (M == 0) return Q8_OK;
  return launched(int8_on_codes(xq, x_scale, x_rowsum, M, K, wq, w_scale, w_zp, N, bias, y, y_dtype, acc_out, st));
}

q8_status q8_quantize_act_static(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, float x_scale,
                                 int8_t* xq, int32_t* x_rowsum, void* stream) {
  if (!valid_dtype(x_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mk(M, K, 0));
  if (M > 0 && (!x || !xq)) return Q8_ERR_NULL_PTR;
  if (!std::isfinite(x_scale) || x_scale <= 0.0f) return Q8_ERR_BAD_ARG;
  if (!aligned16(x) || !aligned16(xq) || (x_rowsum && !aligned16(x_rowsum))) return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, xq, x_rowsum}));
  if (M == 0) return Q8_OK;
  return launched(q8::launch_quant_act_i8_static(x, x_dtype, M, K, x_scale, xq, nullptr, x_rowsum, st));
}

q8_status q8_linear_static(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, float x_scale,
                           const int8_t* wq, const float* w_scale, const float* w_zp, int64_t N,
                           const float* bias, float y_scale, int8_t* yq, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!valid_dtype(x_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mnk(M, N, K));
  if (!wq || !w_scale || !w_zp || (M > 0 && (!x || !yq))) return Q8_ERR_NULL_PTR;
  if (!std::isfinite(x_scale) || x_scale <= 0.0f || !std::isfinite(y_scale) || y_scale <= 0.0f)
    return Q8_ERR_BAD_ARG;
  const LinearWs ws = static_ws(M, K);
  if (ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return Q8_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(w_zp) || !aligned16(yq) ||
      (bias && !aligned16(bias)) || !aligned16(workspace))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, wq, w_scale, w_zp, bias, yq, workspace}));
  if (M == 0) return Q8_OK;
  char* base = static_cast<char*>(workspace);
  int8_t* xq = reinterpret_cast<int8_t*>(base + ws.xq);
  float* xs = reinterpret_cast<float*>(base + ws.xs);
  int32_t* rs = reinterpret_cast<int32_t*>(base + ws.rs);
  Q8_TRY(launched(q8::launch_quant_act_i8_static(x, x_dtype, M, K, x_scale, xq, xs, rs, st)));
  const double y_inv = 1.0 / (double)y_scale;
  return launched(int8_on_codes(xq, xs, rs, M, K, wq, w_scale, w_zp, N, bias, yq, q8::kOutInt8, nullptr, st, y_inv));
}

q8_status q8_linear_w8a16(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, const int8_t* wq,
                          const float* w_scale, const float* w_zp, int64_t N, const float* bias, void* y,
                          q8_dtype y_dtype, void* stream) {
  if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype) || x_dtype == Q8_F32) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mnk(M, N, K));
  if (M > q8::kW8A16MaxM) return Q8_ERR_BAD_SHAPE;
  if (!wq || !w_scale || !w_zp || (M > 0 && (!x || !y))) return Q8_ERR_NULL_PTR;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(w_zp) || !aligned16(y) ||
      (bias && !aligned16(bias)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, wq, w_scale, w_zp, bias, y}));
  if (M == 0) return Q8_OK;
  return launched(q8::launch_gemv_w8a16(x, x_dtype, M, K, wq, w_scale, w_zp, N, bias, y, y_dtype, st));
}

q8_status q8_quantize_weight_grouped(const void* w, q8_dtype w_dtype, int64_t N, int64_t K, int64_t group,
                                     int8_t* wq, float* w_scale, float* w_zp, void* stream) {
  if (!valid_dtype(w_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mk(N, K));
  if (!valid_group(group, K)) return Q8_ERR_BAD_SHAPE;
  if (!w || !wq || !w_scale || !w_zp) return Q8_ERR_NULL_PTR;
  if (!aligned16(w) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(w_zp)) return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {w, wq, w_scale, w_zp}));
  return launched(q8::launch_quant_weight_grouped(w, w_dtype, N, K, group, wq, w_scale, w_zp, st));
}

q8_status q8_linear_grouped(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, const int8_t* wq,
                            const float* w_scale, const float* w_zp, int64_t group, int64_t N, const float* bias,
                            void* y, q8_dtype y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mnk(M, N, K));
  if (!valid_group(group, K)) return Q8_ERR_BAD_SHAPE;
  if (!wq || !w_scale || !w_zp || (M > 0 && (!x || !y))) return Q8_ERR_NULL_PTR;
  const GroupedWs ws = grouped_ws(M, K);
  if (ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return Q8_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(w_zp) || !aligned16(y) ||
      (bias && !aligned16(bias)) || (ws.total > 0 && !aligned16(workspace)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, wq, w_scale, w_zp, bias, y, workspace}));
  if (M == 0) return Q8_OK;
  if (M <= q8::kGemvFusedMaxM)
    return launched(q8::launch_gemv_i8_grouped(x, x_dtype, M, K, wq, w_scale, w_zp, group, N, bias, y, y_dtype, st));
  char* base = static_cast<char*>(workspace);
  int8_t* xq = reinterpret_cast<int8_t*>(base + ws.xq);
  float* xs = reinterpret_cast<float*>(base + ws.xs);
  int32_t* gs = reinterpret_cast<int32_t*>(base + ws.gs);
  Q8_TRY(launched(q8::launch_quant_act_i8_groups(x, x_dtype, M, K, group, xq, xs, gs, st)));
  if (M <= q8::kGroupGemvMaxM)
    return launched(q8::launch_gemv_group(xq, xs, gs, M, K, wq, w_scale, w_zp, group, N, bias, y, y_dtype, st));
  return launched(q8::launch_gemm_group(xq, xs, gs, M, K, wq, w_scale, w_zp, group, N, bias, y, y_dtype, st));
}

namespace {

// The arguments that q8_kv_append and q8_kv_append_norm share, checked, and what the kernels take.
struct Norms {
  const void *q_weight, *k_weight;
  q8_dtype w_dtype;
  float eps;
  const int32_t* positions;      // of the tokens, or null
};
q8_status append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 q8_dtype dtype, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, const Norms* norms, const float* cos,
                 const float* sin, int64_t positions, int64_t rot_dim, int interleaved, const int32_t* q_start,
                 const int32_t* kv_len, const int32_t* block_table, int64_t S, int64_t max_pages, int64_t max_q,
                 uint8_t* k_cache, uint8_t* k_exp, uint8_t* v_cache, uint8_t* v_exp, int64_t num_pages, int64_t page,
                 void* q_out, void* stream) {
  if (!valid_dtype(dtype)) return Q8_ERR_BAD_DTYPE;
  if (norms && (norms->q_weight || norms->k_weight) && !valid_dtype(norms->w_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_kv(T, Hkv, D, S, max_pages, max_q, num_pages, page));
  if (!q_start || !kv_len || !block_table || !k_cache || !k_exp || !v_cache || !v_exp || (T > 0 && (!k || !v)))
    return Q8_ERR_NULL_PTR;
  const bool rotate = cos != nullptr || sin != nullptr;
  if (rotate && (!cos || !sin)) return Q8_ERR_NULL_PTR;
  const bool has_q = q != nullptr || q_out != nullptr;
  if (T > 0 && has_q && (!q || !q_out)) return Q8_ERR_NULL_PTR;
  if (has_q && (Hq < 1 || Hq > 65536)) return Q8_ERR_BAD_SHAPE;
  if (rotate && (positions < 1 || positions > kMaxRows || rot_dim < 16 || rot_dim > D || rot_dim % 16 != 0))
    return Q8_ERR_BAD_SHAPE;
  const int64_t unit = dtype == Q8_F32 ? 4 : 8;      // elements in 16 bytes
  auto bad_stride = [&](int64_t st, int64_t H) { return st < H * D || st % unit != 0; };
  if (T > 1 && (bad_stride(k_stride, Hkv) || bad_stride(v_stride, Hkv) || (has_q && bad_stride(q_stride, Hq))))
    return Q8_ERR_BAD_SHAPE;
  if (norms && (norms->q_weight || norms->k_weight) && !(norms->eps > 0.0f && std::isfinite(norms->eps))) return Q8_ERR_BAD_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cos) || !aligned16(sin) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(q_out) || !aligned4(q_start) || !aligned4(kv_len) || !aligned4(block_table) ||
      (norms && (!aligned16(norms->q_weight) || !aligned16(norms->k_weight) || !aligned4(norms->positions))))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {q, k, v, cos, sin, q_start, kv_len, block_table, k_cache, k_exp, v_cache, v_exp, q_out,
                         norms ? norms->q_weight : nullptr, norms ? norms->k_weight : nullptr,
                         norms ? norms->positions : nullptr}));
  if (T == 0) return Q8_OK;
  q8::AppendArgs a{};
  a.kv = kv_view(k_cache, k_exp, v_cache, v_exp, q_start, kv_len, block_table, T, Hkv, S, max_pages, num_pages, page);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.heads = has_q ? (int)Hq : 1;
  a.cos = cos;
  a.sin = sin;
  a.positions = rotate ? (int)positions : 1;
  a.rot = rotate ? (int)rot_dim : 0;
  a.interleaved = interleaved != 0;
  const int64_t mq = bound_of(max_q, T);
  a.max_q = (int)mq;
  if (!norms) return launched(q8::launch_kv_append(a, dtype, (int)D, st));
  a.qw = norms->q_weight;
  a.kw = norms->k_weight;
  a.w_dt = norms->w_dtype;
  a.eps = norms->eps;
  a.pos = norms->positions;
  return launched(q8::launch_kv_append_norm(a, dtype, (int)D, st));
}

}  // namespace

q8_status q8_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, q8_dtype dtype, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                       const float* cos, const float* sin, int64_t positions, int64_t rot_dim, int interleaved,
                       const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table, int64_t S,
                       int64_t max_pages, int64_t max_q, uint8_t* k_cache, uint8_t* k_exp, uint8_t* v_cache,
                       uint8_t* v_exp, int64_t num_pages, int64_t page, void* q_out, void* stream) {
  return append(q, q_stride, k, k_stride, v, v_stride, dtype, T, Hq, Hkv, D, nullptr, cos, sin, positions, rot_dim,
                interleaved, q_start, kv_len, block_table, S, max_pages, max_q, k_cache, k_exp, v_cache, v_exp, num_pages,
                page, q_out, stream);
}

q8_status q8_kv_append_norm(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, q8_dtype dtype, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                            const void* q_weight, const void* k_weight, q8_dtype w_dtype, float eps, const float* cos,
                            const float* sin, int64_t positions, int64_t rot_dim, int interleaved,
                            const int32_t* token_positions, const int32_t* q_start, const int32_t* kv_len,
                            const int32_t* block_table, int64_t S, int64_t max_pages, int64_t max_q, uint8_t* k_cache,
                            uint8_t* k_exp, uint8_t* v_cache, uint8_t* v_exp, int64_t num_pages, int64_t page,
                            void* q_out, void* stream) {
  const Norms norms{q_weight, k_weight, w_dtype, eps, token_positions};
  return append(q, q_stride, k, k_stride, v, v_stride, dtype, T, Hq, Hkv, D, &norms, cos, sin, positions, rot_dim,
                interleaved, q_start, kv_len, block_table, S, max_pages, max_q, k_cache, k_exp, v_cache, v_exp, num_pages,
                page, q_out, stream);
}

namespace {

size_t attention_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t S, int64_t max_q, int64_t max_kv,
                       int64_t window, bool tree) {
  if (check_kv(T, Hkv, D, S, 1, max_q, 1, 32) != Q8_OK || !valid_heads(T, Hq, Hkv) || max_kv < 0 ||
      max_kv > kMaxRows || window < 0)
    return 0;
  window = window > kMaxTokens ? 0 : window;
  return attn_ws(T, Hq, Hkv, D, S, bound_of(max_q, T), bound_of(max_kv, kMaxRows), window, tree).total;
}

}  // namespace

size_t q8_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t S, int64_t max_q,
                                    int64_t max_kv, int64_t window) {
  return attention_bytes(T, Hq, Hkv, D, S, max_q, max_kv, window, false);
}
size_t q8_attention_tree_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t S, int64_t max_q,
                                         int64_t max_kv, int64_t window) {
  return attention_bytes(T, Hq, Hkv, D, S, max_q, max_kv, window, true);
}

namespace {

// The tree of drafted tokens that the new ones are; null: a sequence.
struct Tree {
  const uint64_t* mask;
  int64_t words;
  const int32_t* positions;
};
q8_status attention(const void* q, int64_t q_stride, q8_dtype dtype, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                    const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table, int64_t S,
                    int64_t max_pages, int64_t max_q, int64_t max_kv, const uint8_t* k_cache, const uint8_t* k_exp,
                    const uint8_t* v_cache, const uint8_t* v_exp, int64_t num_pages, int64_t page, const Tree* tree,
                    float scale, int causal, int64_t window, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (dtype != Q8_F16 && dtype != Q8_BF16) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_kv(T, Hkv, D, S, max_pages, max_q, num_pages, page));
  if (!valid_heads(T, Hq, Hkv) || max_kv < 0 || max_kv > kMaxRows) return Q8_ERR_BAD_SHAPE;
  if (tree && (tree->words < 1 || tree->words > kMaxMaskWords)) return Q8_ERR_BAD_SHAPE;
  if (T > 1 && (q_stride < Hq * D || q_stride % 8 != 0)) return Q8_ERR_BAD_SHAPE;
  if (!q_start || !kv_len || !block_table || !k_cache || !k_exp || !v_cache || !v_exp || (T > 0 && (!q || !out)))
    return Q8_ERR_NULL_PTR;
  if (tree && T > 0 && !tree->mask) return Q8_ERR_NULL_PTR;
  if (!std::isfinite(scale) || window < 0) return Q8_ERR_BAD_ARG;
  window = window > kMaxTokens ? 0 : window;           // wider than any sequence: no window
  const int64_t mq = bound_of(max_q, T), mkv = bound_of(max_kv, kMaxRows);
  const AttnWs ws = attn_ws(T, Hq, Hkv, D, S, mq, mkv, window, tree != nullptr);
  if (ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return Q8_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || (lse && !aligned4(lse)) ||
      (ws.total > 0 && !aligned16(workspace)) || !aligned4(q_start) || !aligned4(kv_len) || !aligned4(block_table) ||
      (tree && ((reinterpret_cast<uintptr_t>(tree->mask) & 7) != 0 || !aligned4(tree->positions))))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {q, q_start, kv_len, block_table, k_cache, k_exp, v_cache, v_exp, out, lse,
                         ws.total > 0 ? workspace : nullptr, tree ? tree->mask : nullptr,
                         tree ? tree->positions : nullptr}));
  if (T == 0) return Q8_OK;
  q8::AttnArgs a{};
  a.kv = kv_view(k_cache, k_exp, v_cache, v_exp, q_start, kv_len, block_table, T, Hkv, S, max_pages, num_pages, page);
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.heads = (int)Hq;
  a.causal = causal != 0;
  a.window = (int)window;
  a.max_q = (int)mq;
  a.max_kv = mkv;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (ws.total > 0) {
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.part);
    a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.ml);
  }
  if (!tree) return launched(q8::launch_attention(a, dtype, (int)D, st));
  a.mask = tree->mask;
  a.words = (int)tree->words;
  a.pos = tree->positions;
  return launched(q8::launch_attention_tree(a, dtype, (int)D, st));
}

}  // namespace

q8_status q8_attention_kv8(const void* q, int64_t q_stride, q8_dtype dtype, int64_t T, int64_t Hq, int64_t Hkv,
                           int64_t D, const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                           int64_t S, int64_t max_pages, int64_t max_q, int64_t max_kv, const uint8_t* k_cache,
                           const uint8_t* k_exp, const uint8_t* v_cache, const uint8_t* v_exp, int64_t num_pages,
                           int64_t page, float scale, int causal, int64_t window, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return attention(q, q_stride, dtype, T, Hq, Hkv, D, q_start, kv_len, block_table, S, max_pages, max_q, max_kv, k_cache,
                   k_exp, v_cache, v_exp, num_pages, page, nullptr, scale, causal, window, out, lse, workspace,
                   workspace_bytes, stream);
}

q8_status q8_attention_kv8_tree(const void* q, int64_t q_stride, q8_dtype dtype, int64_t T, int64_t Hq, int64_t Hkv,
                                int64_t D, const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                                int64_t S, int64_t max_pages, int64_t max_q, int64_t max_kv, const uint8_t* k_cache,
                                const uint8_t* k_exp, const uint8_t* v_cache, const uint8_t* v_exp, int64_t num_pages,
                                int64_t page, const uint64_t* mask, int64_t mask_words, const int32_t* token_positions,
                                float scale, int64_t window, void* out, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  const Tree tree{mask, mask_words, token_positions};
  return attention(q, q_stride, dtype, T, Hq, Hkv, D, q_start, kv_len, block_table, S, max_pages, max_q, max_kv, k_cache,
                   k_exp, v_cache, v_exp, num_pages, page, &tree, scale, 0, window, out, lse, workspace, workspace_bytes,
                   stream);
}

namespace {

// The caches of all layers: every pointer given and aligned.
q8_status check_layers(uint8_t* const* k, uint8_t* const* ke, uint8_t* const* v, uint8_t* const* ve, int64_t layers) {
  if (layers < 1 || layers > kMaxLayers) return Q8_ERR_BAD_SHAPE;
  if (!k || !ke || !v || !ve) return Q8_ERR_NULL_PTR;
  for (int64_t i = 0; i < layers; ++i) {
    if (!k[i] || !ke[i] || !v[i] || !ve[i]) return Q8_ERR_NULL_PTR;
    if (!aligned16(k[i]) || !aligned16(v[i])) return Q8_ERR_ALIGN;
  }
  return Q8_OK;
}
// The memory of a call over the caches: no array that is written may share any with another.
struct Ranges {
  struct Range {
    uintptr_t from, to;
    bool written;
  } r[4 * kMaxLayers + 16];
  int n = 0;
  void add(const void* p, int64_t bytes, bool written) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (bytes > 0) r[n++] = Range{at, at + (uint64_t)bytes, written};
  }
  void ints(const void* p, int64_t count, bool written) { add(p, 4 * count, written); }
  void caches(uint8_t* const* k, uint8_t* const* ke, uint8_t* const* v, uint8_t* const* ve, int64_t layers, int64_t pages,
              int64_t Hkv, int64_t page, int64_t D) {
    for (int64_t i = 0; i < layers; ++i) {
      add(k[i], pages * Hkv * page * D, true);
      add(v[i], pages * Hkv * page * D, true);
      add(ke[i], pages * Hkv, true);
      add(ve[i], pages * Hkv, true);
    }
  }
  bool apart() {
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.from < b.from; });
    uintptr_t read = 0, written = 0;               // the ends of what lies before
    for (int i = 0; i < n; ++i) {
      if (r[i].from < written || (r[i].written && r[i].from < read)) return false;
      uintptr_t& end = r[i].written ? written : read;
      end = end > r[i].to ? end : r[i].to;
    }
    return true;
  }
};
q8_status check_layer_ptrs(hipStream_t st, uint8_t* const* k, uint8_t* const* ke, uint8_t* const* v, uint8_t* const* ve,
                           int64_t layers) {
  for (int64_t i = 0; i < layers; ++i) Q8_TRY(check_ptrs(st, {k[i], ke[i], v[i], ve[i]}));
  return Q8_OK;
}
void take_layers(q8::CacheLayer* to, uint8_t* const* k, uint8_t* const* ke, uint8_t* const* v, uint8_t* const* ve,
                 int64_t from, int n) {
  for (int i = 0; i < n; ++i) to[i] = q8::CacheLayer{k[from + i], v[from + i], ke[from + i], ve[from + i]};
}
struct ForkWs { size_t first, fresh, taken, copies, total; };
ForkWs fork_ws(int64_t S, int64_t S_out, int64_t num_pages) {
  Carve c;
  ForkWs w;
  w.first = c.take((size_t)S * 4);
  w.fresh = c.take((size_t)S_out * 4);
  w.taken = c.take((size_t)num_pages * 4);
  w.copies = c.take((size_t)S_out * 8);
  w.total = c.off;
  return w;
}

}  // namespace

q8_status q8_kv_compact(uint8_t* const* k_cache, uint8_t* const* k_exp, uint8_t* const* v_cache, uint8_t* const* v_exp,
                        int64_t layers, int64_t Hkv, int64_t D, const int32_t* q_start, const int32_t* kv_len,
                        const int32_t* block_table, int64_t S, int64_t max_pages, int64_t num_pages, int64_t page,
                        const int32_t* keep, int64_t max_keep, const int32_t* n_keep, int32_t* len_out, void* stream) {
  Q8_TRY(check_kv(0, Hkv, D, S, max_pages, 0, num_pages, page));
  if (max_keep < 0 || max_keep > kMaxTokens) return Q8_ERR_BAD_SHAPE;
  if (!q_start || !kv_len || !block_table || (max_keep > 0 && !keep) || !n_keep || !len_out) return Q8_ERR_NULL_PTR;
  Q8_TRY(check_layers(k_cache, k_exp, v_cache, v_exp, layers));
  if (!aligned4(q_start) || !aligned4(kv_len) || !aligned4(block_table) || !aligned4(keep) || !aligned4(n_keep) ||
      !aligned4(len_out))
    return Q8_ERR_ALIGN;
  Ranges mem;
  mem.caches(k_cache, k_exp, v_cache, v_exp, layers, num_pages, Hkv, page, D);
  mem.ints(len_out, S, true);                      // (every workgroup reads the others while one writes it)
  mem.ints(kv_len, S, false);
  mem.ints(q_start, S + 1, false);
  mem.ints(n_keep, S, false);
  mem.ints(block_table, S * max_pages, false);
  mem.ints(keep, S * max_keep, false);
  if (!mem.apart()) return Q8_ERR_BAD_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {q_start, kv_len, block_table, keep, n_keep, len_out}));
  if (debug_validate()) Q8_TRY(check_layer_ptrs(st, k_cache, k_exp, v_cache, v_exp, layers));
  q8::CompactArgs a{};
  a.kv = kv_view(nullptr, nullptr, nullptr, nullptr, q_start, kv_len, block_table, 0, Hkv, S, max_pages, num_pages, page);
  a.keep = keep;
  a.n_keep = n_keep;
  a.len_out = len_out;
  a.width = (int)max_keep;
  for (int64_t i = 0; i < layers; i += q8::kLayers) {
    const int n = (int)(layers - i < q8::kLayers ? layers - i : q8::kLayers);
    take_layers(a.layer, k_cache, k_exp, v_cache, v_exp, i, n);
    Q8_TRY(launched(q8::launch_kv_compact(a, (int)D, n, st)));
    a.len_out = nullptr;
  }
  return Q8_OK;
}

size_t q8_kv_fork_workspace_bytes(int64_t S, int64_t S_out, int64_t num_pages) {
  if (S < 1 || S > 32768 || S_out < 1 || S_out > 32768 || num_pages < 1 || num_pages > kMaxRows) return 0;
  return fork_ws(S, S_out, num_pages).total;
}

q8_status q8_kv_fork(uint8_t* const* k_cache, uint8_t* const* k_exp, uint8_t* const* v_cache, uint8_t* const* v_exp,
                     int64_t layers, int64_t Hkv, int64_t D, int64_t num_pages, int64_t page,
                     const int32_t* block_table, const int32_t* kv_len, const int32_t* refs, int64_t S,
                     int64_t max_pages, const int32_t* parent, int64_t S_out, int64_t room, int32_t* table_out,
                     int32_t* len_out, int32_t* refs_out, int32_t* missing, void* workspace, size_t workspace_bytes,
                     void* stream) {
  Q8_TRY(check_kv(0, Hkv, D, S, max_pages, 0, num_pages, page));
  if (S_out < 1 || S_out > 32768 || room < 0 || room > kMaxTokens || S_out * max_pages > kMaxRows) return Q8_ERR_BAD_SHAPE;
  if (!block_table || !kv_len || !refs || !parent || !table_out || !len_out || !refs_out || !missing) return Q8_ERR_NULL_PTR;
  Q8_TRY(check_layers(k_cache, k_exp, v_cache, v_exp, layers));
  const ForkWs ws = fork_ws(S, S_out, num_pages);
  if (!workspace || workspace_bytes < ws.total) return Q8_ERR_WORKSPACE;
  if (!aligned4(block_table) || !aligned4(kv_len) || !aligned4(refs) || !aligned4(parent) || !aligned4(table_out) ||
      !aligned4(len_out) || !aligned4(refs_out) || !aligned4(missing) || !aligned16(workspace))
    return Q8_ERR_ALIGN;
  Ranges mem;
  mem.caches(k_cache, k_exp, v_cache, v_exp, layers, num_pages, Hkv, page, D);
  mem.ints(table_out, S_out * max_pages, true);
  mem.ints(len_out, S_out, true);
  mem.ints(refs_out, num_pages, true);
  mem.ints(missing, 1, true);
  mem.add(workspace, (int64_t)ws.total, true);
  mem.ints(block_table, S * max_pages, false);
  mem.ints(kv_len, S, false);
  mem.ints(refs, num_pages, false);
  mem.ints(parent, S_out, false);
  if (!mem.apart()) return Q8_ERR_BAD_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {block_table, kv_len, refs, parent, table_out, len_out, refs_out, missing, workspace}));
  if (debug_validate()) Q8_TRY(check_layer_ptrs(st, k_cache, k_exp, v_cache, v_exp, layers));
  char* const base = static_cast<char*>(workspace);
  q8::ForkArgs a{};
  a.table = block_table;
  a.kv_len = kv_len;
  a.refs = refs;
  a.parent = parent;
  a.table_out = table_out;
  a.len_out = len_out;
  a.refs_out = refs_out;
  a.missing = missing;
  a.first = reinterpret_cast<int32_t*>(base + ws.first);
  a.fresh = reinterpret_cast<int32_t*>(base + ws.fresh);
  a.taken = reinterpret_cast<int32_t*>(base + ws.taken);
  a.copies = reinterpret_cast<int32_t*>(base + ws.copies);
  a.room = room;
  a.page_bytes = Hkv * page * D;
  a.seqs = (int)S;
  a.outs = (int)S_out;
  a.max_pages = (int)max_pages;
  a.num_pages = (int)num_pages;
  a.page = (int)page;
  a.kv_heads = (int)Hkv;
  Q8_TRY(launched(q8::launch_kv_fork(a, st)));
  for (int64_t i = 0; i < layers; i += q8::kLayers) {
    const int n = (int)(layers - i < q8::kLayers ? layers - i : q8::kLayers);
    take_layers(a.layer, k_cache, k_exp, v_cache, v_exp, i, n);
    Q8_TRY(launched(q8::launch_copy_pages(a, n, st)));
  }
  return Q8_OK;
}

q8_status q8_quantize_weight_block(const void* w, q8_dtype w_dtype, int64_t N, int64_t K, uint8_t* wq, float* w_scale,
                                   void* stream) {
  if (!valid_dtype(w_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mk(N, K));
  if (N * K > kMaxRows) return Q8_ERR_BAD_SHAPE;
  if (!w || !wq || !w_scale) return Q8_ERR_NULL_PTR;
  if (!aligned16(w) || !aligned16(wq) || !aligned16(w_scale)) return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {w, wq, w_scale}));
  return launched(q8::launch_quant_weight_block(w, w_dtype, N, K, wq, w_scale, st));
}

q8_status q8_quantize_act_block(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, uint8_t* xq, float* x_scale,
                                void* stream) {
  if (!valid_dtype(x_dtype)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mk(M, K, 0));
  if (M * K > kMaxRows) return Q8_ERR_BAD_SHAPE;
  if (M > 0 && (!x || !xq || !x_scale)) return Q8_ERR_NULL_PTR;
  if (!aligned16(x) || !aligned16(xq) || !aligned16(x_scale)) return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, xq, x_scale}));
  if (M == 0) return Q8_OK;
  return launched(q8::launch_quant_act_block(x, x_dtype, M, K, xq, x_scale, st));
}

q8_status q8_gemm_fp8_block(const uint8_t* xq, const float* x_scale, int64_t M, int64_t K, const uint8_t* wq,
                            const float* w_scale, int64_t N, const float* bias, void* y, q8_dtype y_dtype,
                            void* stream) {
  if (y_dtype != Q8_F16 && y_dtype != Q8_BF16) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mnk(M, N, K));
  if (!wq || !w_scale || (M > 0 && (!xq || !x_scale || !y))) return Q8_ERR_NULL_PTR;
  if (!aligned16(xq) || !aligned16(x_scale) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(y) ||
      (bias && !aligned16(bias)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {xq, x_scale, wq, w_scale, bias, y}));
  if (M == 0) return Q8_OK;
  return launched(q8::launch_gemm_fp8_block(xq, x_scale, M, K, wq, w_scale, N, bias, y, y_dtype, st));
}

q8_status q8_linear_fp8_block(const void* x, q8_dtype x_dtype, int64_t M, int64_t K, const uint8_t* wq,
                              const float* w_scale, int64_t N, const float* bias, void* y, q8_dtype y_dtype,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(x_dtype) || (y_dtype != Q8_F16 && y_dtype != Q8_BF16)) return Q8_ERR_BAD_DTYPE;
  Q8_TRY(check_mnk(M, N, K));
  if (!wq || !w_scale || (M > 0 && (!x || !y))) return Q8_ERR_NULL_PTR;
  const Fp8Ws ws = fp8_block_ws(M, K);
  if (ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return Q8_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(y) || (bias && !aligned16(bias)) ||
      (ws.total > 0 && !aligned16(workspace)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {x, wq, w_scale, bias, y, ws.total > 0 ? workspace : nullptr}));
  if (M == 0) return Q8_OK;
  if (q8::fp8_block_is_fused(M))
    return launched(q8::launch_gemv_fp8_block(x, x_dtype, M, K, wq, w_scale, N, bias, y, y_dtype, st));
  char* base = static_cast<char*>(workspace);
  uint8_t* xq = reinterpret_cast<uint8_t*>(base + ws.xq);
  float* xs = reinterpret_cast<float*>(base + ws.xs);
  Q8_TRY(launched(q8::launch_quant_act_block(x, x_dtype, M, K, xq, xs, st)));
  return launched(q8::launch_gemm_fp8_block(xq, xs, M, K, wq, w_scale, N, bias, y, y_dtype, st));
}

q8_status q8_bench_mfma_loop(q8_format fmt, int64_t iters, int64_t workgroups, int32_t* sink, void* stream) {
  if (fmt != Q8_INT8_SYM && fmt != Q8_FP8_E4M3) return Q8_ERR_BAD_FORMAT;
  if (iters < 1 || iters > kMaxRows || workgroups < 1 || workgroups > 65536) return Q8_ERR_BAD_ARG;
  if (!sink) return Q8_ERR_NULL_PTR;
  if (!aligned16(sink)) return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {sink}));
  return launched(q8::launch_mfma_loop(fmt == Q8_INT8_SYM ? 0 : 2, iters, workgroups, sink, st));
}

q8_status q8_bench_stream_read(const void* src, int64_t bytes, int64_t workgroups, int32_t* sink, void* stream) {
  if (bytes < 16 || bytes % 16 != 0 || bytes >= (int64_t(1) << 31) || workgroups < 1 || workgroups > 65536)
    return Q8_ERR_BAD_ARG;
  if (!src || !sink) return Q8_ERR_NULL_PTR;
  if (!aligned16(src) || !aligned16(sink)) return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {src, sink}));
  return launched(q8::launch_stream_read(src, bytes, workgroups, sink, st));
}

q8_status q8_probe_fp8_mfma(const uint8_t* a, const uint8_t* b, const float* c, float* d, int64_t count,
                            void* stream) {
  if (count < 1 || count > 65536) return Q8_ERR_BAD_ARG;
  if (!a || !b || !c || !d) return Q8_ERR_NULL_PTR;
  if (!aligned16(a) || !aligned16(b) || !aligned16(c) || !aligned16(d)) return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {a, b, c, d}));
  return launched(q8::launch_probe_fp8_mfma(a, b, c, d, count, st));
}

q8_status q8_gemm_tile(q8_op op, int64_t M, int64_t N, int64_t K, int32_t* bm, int32_t* bn) {
  if (op != Q8_OP_LINEAR && op != Q8_OP_STATIC && op != Q8_OP_DECOMP && op != Q8_OP_FP8) return Q8_ERR_BAD_ARG;
  Q8_TRY(check_mnk(M, N, K));
  if (!bm || !bn) return Q8_ERR_NULL_PTR;
  *bm = *bn = 0;
  if (M == 0 || ((op == Q8_OP_LINEAR || op == Q8_OP_STATIC) && M <= q8::kGemvMaxM)) return Q8_OK;
  const q8::GemmKind kind = op == Q8_OP_DECOMP ? q8::GEMM_INT8_DECOMP : op == Q8_OP_FP8 ? q8::GEMM_FP8 : q8::GEMM_INT8;
  int tm = 0, tn = 0;
  q8::gemm_tile(kind, M, N, &tm, &tn);
  *bm = tm;
  *bn = tn;
  return Q8_OK;
}

q8_status q8_gemm_fp8(const uint8_t* xq, const float* x_scale, int64_t M, int64_t K, const uint8_t* wq,
                      const float* w_scale, int64_t N, const float* bias, void* y, void* stream) {
  Q8_TRY(check_mnk(M, N, K));
  if (!wq || !w_scale || (M > 0 && (!xq || !x_scale || !y))) return Q8_ERR_NULL_PTR;
  if (!aligned16(xq) || !aligned16(x_scale) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(y) ||
      (bias && !aligned16(bias)))
    return Q8_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Q8_TRY(check_device(st));
  Q8_TRY(check_ptrs(st, {xq, x_scale, wq, w_scale, bias, y}));
  if (M == 0) return Q8_OK;
  q8::GemmArgs g{};
  g.a = xq;
  g.b = wq;
  g.a_scale = x_scale;
  g.b_scale = w_scale;
  g.bias = bias;
  g.y = y;
  g.M = M;
  g.N = N;
  g.K = K;
  return launched(q8::launch_gemm(q8::GEMM_FP8, g, Q8_BF16, st));
}

}  // extern "C"
