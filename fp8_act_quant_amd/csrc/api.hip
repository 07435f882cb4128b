// api.hip -- the C ABI declared in include/fp8q.h: host-side validation, then one launch
// on the caller's stream. Nothing here allocates, synchronises or keeps state beyond a
// per-device "is this a gfx950" cache.
#include <fp8q.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "launch.h"

namespace {

constexpr int64_t kBlock = 128;
constexpr int kMaxDevices = 64;
// launch-geometry limits of the kernels (grid dimensions are 32-bit)
constexpr int64_t kMaxElems = (int64_t)1 << 46;
constexpr int64_t kMaxWeightBlockRows = 65535;
// The GEMM addresses a workgroup's rows of A and W (at most 256 rows of K bytes) through
// buffer resources whose byte count is 32-bit and which read zero past it: 256 * K must stay
// below 2^32, so K < 2^24 (a count of exactly 2^32 cannot be stated, and its last bytes would
// read as zero).
constexpr int64_t kMaxGemmK = ((int64_t)1 << 24) - 128;
// grid dimensions of the two-dimensional launches
constexpr int64_t kMaxGridX = 0x7FFFFFFF, kMaxGridY = 65535;
// a grid dimension counts at most 2^32 - 1 work-items: workgroups of 256 threads along it
constexpr int64_t kMaxBlocks256 = 0xFFFFFFFFll / 256;
// The bf16 GEMM advances K in steps of 64 elements and addresses a workgroup's rows (at most
// 256 of 2K bytes) through 32-bit buffer resources: K < 2^23.
constexpr int64_t kBf16Step = 64;
constexpr int64_t kMaxBf16K = ((int64_t)1 << 23) - kBf16Step;
// K-block-major activation scales are addressed with 32-bit byte offsets: M * K/128 < 2^29
constexpr int64_t kMaxKmajorScales = (int64_t)1 << 29;
// The GEMMs count tile rows and columns in 32-bit ints (64-row tiles at the smallest), and a
// grid holds at most 2^32 / 256 workgroups; with M, N <= 2^36 the counts stay far inside
// both. (No device holds such an operand: 2^36 rows of K >= 64 elements.)
constexpr int64_t kMaxGemmRows = (int64_t)1 << 36;

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// 0 = unknown, 1 = gfx950, 2 = other / unusable
std::atomic<int> g_dev_kind[kMaxDevices];

int check_device() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return FP8Q_ERR_UNSUPPORTED;
    if (dev < 0 || dev >= kMaxDevices) return FP8Q_ERR_UNSUPPORTED;
    int kind = g_dev_kind[dev].load(std::memory_order_relaxed);
    if (kind == 0) {
        hipDeviceProp_t prop;
        kind = 2;
        if (hipGetDeviceProperties(&prop, dev) == hipSuccess && std::strncmp(prop.gcnArchName, "gfx950", 6) == 0)
            kind = 1;
        g_dev_kind[dev].store(kind, std::memory_order_relaxed);
    }
    return kind == 1 ? FP8Q_OK : FP8Q_ERR_UNSUPPORTED;
}

int shape_ok(int64_t rows, int64_t K) {
    if (rows < 0 || K < 0 || (K % kBlock) != 0) return FP8Q_ERR_SHAPE;
    if (K > 0 && rows > kMaxElems / K) return FP8Q_ERR_SHAPE;
    return FP8Q_OK;
}

// Routed-expert layer: a row (of logits, of assignments) is a wave's or a workgroup's, so its
// count is bounded by the grid (256 threads each); assignments and rows are 32-bit.
constexpr int64_t kMaxTokens = kMaxBlocks256;
constexpr int64_t kMaxTopK = 32, kMaxGroups = 64;
// 8-bit products: the sum of K products of at most 2^14 fits 32 bits while K < 2^17
constexpr int64_t kInt8Step = 16, kMaxInt8K = ((int64_t)1 << 17) - kInt8Step;
constexpr int64_t kMaxGatherBytes = 0xFFFFFFF0ll;   // gathered rows have 32-bit byte offsets

bool is_type(int dtype) { return dtype == FP8Q_OUT_F32 || dtype == FP8Q_OUT_BF16; }

// T rows of top_k of `experts` experts
bool routing_ok(int64_t T, int64_t experts, int64_t top_k) {
    return T >= 0 && T <= kMaxTokens && experts >= 1 && experts <= fp8q::kMaxGroupedExperts && top_k >= 1 &&
           top_k <= kMaxTopK && T <= (INT32_MAX - 1) / top_k;
}

int combine_ok(int dtype, int64_t T, int64_t rows, int64_t H, int64_t top_k) {
    if (!is_type(dtype)) return FP8Q_ERR_DTYPE;
    if (T < 0 || rows < 0 || H < 0 || top_k < 1 || top_k > kMaxTopK || rows > INT32_MAX) return FP8Q_ERR_SHAPE;
    // one workgroup of 256 threads per token (and, forward, of 128 per 512 elements at the least)
    if (T > kMaxTokens || T > INT32_MAX / top_k || (H + 511) / 512 > kMaxGridY) return FP8Q_ERR_SHAPE;
    return FP8Q_OK;
}

int int8_ok(int dtype, int64_t M, int64_t N, int64_t K) {
    if (!is_type(dtype)) return FP8Q_ERR_DTYPE;
    if (M < 0 || N < 0 || K < 0 || K % kInt8Step || K > kMaxInt8K) return FP8Q_ERR_SHAPE;
    if (M > kMaxGemmRows || N > kMaxGemmRows || (M > 0 && N > kMaxElems / M)) return FP8Q_ERR_SHAPE;
    return FP8Q_OK;
}

int norm_ok(int dtype, int flags, int64_t T, int64_t H) {
    if (!is_type(dtype) || (flags & ~FP8Q_NORM_GATES)) return FP8Q_ERR_DTYPE;
    if (T < 0 || H < fp8q::kMinNormH || H > fp8q::kMaxNormH || T > kMaxElems / H) return FP8Q_ERR_SHAPE;
    return FP8Q_OK;
}

// The dense block's products: rows of operands are 16-byte pieces, addressed within a tile by 32-bit byte
// offsets (256 rows of 2 K bytes), 32 of a tile's rows at the least are a workgroup of 256 threads or more
constexpr int64_t kDenseStep = 8, kMaxDenseK = ((int64_t)1 << 23) - kDenseStep, kMaxDenseRows = (int64_t)1 << 26;
constexpr int64_t kMaxDenseN = (int64_t)1 << 28;

bool gated_ok(int64_t M, int64_t F, int64_t K) {
    return M >= 0 && F >= 0 && K >= 0 && F % kDenseStep == 0 && K % kDenseStep == 0 && K <= kMaxDenseK &&
           2 * F <= kMaxDenseK && M <= kMaxDenseRows;
}

size_t gated_gradient_bytes(int64_t M, int64_t F, int64_t K, bool wide) {
    if (!gated_ok(M, F, K)) return 0;
    const fp8q::GatedGradPlans plans = fp8q::gated_gradient_plans(M, F, K, wide);
    return plans.fits ? fp8q::gated_linear_backward_workspace_bytes(plans, M, F, K) : 0;
}

bool adapter_ok(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank) {
    return M >= 0 && N >= 0 && K >= 0 && K % kDenseStep == 0 && K <= kMaxDenseK && M <= kMaxDenseRows &&
           N <= kMaxDenseN && adapters >= 0 && adapters <= INT32_MAX && rank >= kDenseStep && rank % kDenseStep == 0 &&
           rank <= fp8q::kMaxRank;   // (an adapter's A is below 2^32 - 2^12 bytes)
}

int finish(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_LAUNCH; }

}  // namespace

extern "C" {

int fp8_act_quant(const uint16_t *x, uint8_t *q, float *s, int64_t M, int64_t K, void *stream) {
    if (int e = shape_ok(M, K)) return e;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !q || !s) return FP8Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(q, 16) || misaligned(s, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_act_quant(x, q, s, M, K, false, static_cast<hipStream_t>(stream)));
}

int fp8_act_quant_kmajor(const uint16_t *x, uint8_t *q, float *s, int64_t M, int64_t K, void *stream) {
    if (int e = shape_ok(M, K)) return e;
    if (K > 0 && M >= kMaxKmajorScales / (K / kBlock)) return FP8Q_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !q || !s) return FP8Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(q, 16) || misaligned(s, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_act_quant(x, q, s, M, K, true, static_cast<hipStream_t>(stream)));
}

int fp8_weight_quant(const uint16_t *w, uint8_t *q, float *s, int64_t N, int64_t K, void *stream) {
    if (int e = shape_ok(N, K)) return e;
    if ((N + kBlock - 1) / kBlock > kMaxWeightBlockRows) return FP8Q_ERR_SHAPE;
    if (K / kBlock > kMaxBlocks256) return FP8Q_ERR_SHAPE;   // one workgroup per 128-column block
    if (N == 0 || K == 0) return FP8Q_OK;
    if (!w || !q || !s) return FP8Q_ERR_NULL;
    if (misaligned(w, 16) || misaligned(q, 16) || misaligned(s, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_weight_quant(w, q, s, N, K, static_cast<hipStream_t>(stream)));
}

int fp8_weight_dequant(const uint8_t *q, const float *s, uint16_t *w, int64_t N, int64_t K, void *stream) {
    if (int e = shape_ok(N, K)) return e;
    if (N == 0 || K == 0) return FP8Q_OK;
    if (!w || !q || !s) return FP8Q_ERR_NULL;
    if (misaligned(w, 16) || misaligned(q, 16) || misaligned(s, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_weight_dequant(q, s, w, N, K, static_cast<hipStream_t>(stream)));
}

int fp8_block_gemm(const uint8_t *aq, const float *sa, const uint8_t *wq, const float *sw, void *y,
                   int y_dtype, int64_t M, int64_t N, int64_t K, void *workspace, size_t workspace_bytes,
                   void *stream) {
    return fp8_block_gemm_bias(aq, sa, wq, sw, nullptr, y, y_dtype, M, N, K, workspace, workspace_bytes, stream);
}

int fp8_block_gemm_bias(const uint8_t *aq, const float *sa, const uint8_t *wq, const float *sw, const float *bias,
                        void *y, int y_dtype, int64_t M, int64_t N, int64_t K, void *workspace,
                        size_t workspace_bytes, void *stream) {
    const int dtype = y_dtype & 0xFF;
    const bool sa_kmajor = (y_dtype & FP8Q_SA_KMAJOR) != 0;
    const int mode = y_dtype & ~0xFF & ~FP8Q_SA_KMAJOR;
    if (dtype != FP8Q_OUT_F32 && dtype != FP8Q_OUT_BF16) return FP8Q_ERR_DTYPE;
    if (mode != 0 && mode != FP8Q_GEMM_FP8_PRODUCTS && mode != FP8Q_GEMM_EXACT_SLICES) return FP8Q_ERR_DTYPE;
    if (int e = shape_ok(M, K)) return e;
    if (int e = shape_ok(N, K)) return e;
    if (M > 0 && N > kMaxElems / M) return FP8Q_ERR_SHAPE;
    if (K > kMaxGemmK || M > kMaxGemmRows || N > kMaxGemmRows) return FP8Q_ERR_SHAPE;
    if (sa_kmajor && K > 0 && M >= kMaxKmajorScales / (K / kBlock)) return FP8Q_ERR_SHAPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!y) return FP8Q_ERR_NULL;
    if (K > 0 && (!aq || !sa || !wq || !sw)) return FP8Q_ERR_NULL;
    if (misaligned(aq, 16) || misaligned(wq, 16) || misaligned(y, 16) || misaligned(sa, 4) ||
        misaligned(sw, 4) || misaligned(bias, 4))
        return FP8Q_ERR_ALIGN;
    if (workspace == nullptr) workspace_bytes = 0;
    if (workspace_bytes && misaligned(workspace, 16)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    // default contraction: exact slices for fp32 output, the FP8 matrix unit for bf16 output
    const bool exact = mode == FP8Q_GEMM_EXACT_SLICES || (mode == 0 && dtype == FP8Q_OUT_F32);
    return finish(fp8q::launch_block_gemm(aq, sa, wq, sw, bias, y, dtype == FP8Q_OUT_BF16, exact, sa_kmajor, M, N,
                                          K, workspace, workspace_bytes, static_cast<hipStream_t>(stream)));
}

int fp8_bf16_gemm(const uint16_t *x, const uint16_t *w, const float *bias, void *y, int y_dtype, int64_t M,
                  int64_t N, int64_t K, void *stream) {
    if (y_dtype != FP8Q_OUT_F32 && y_dtype != FP8Q_OUT_BF16) return FP8Q_ERR_DTYPE;
    if (M < 0 || N < 0 || K < 0 || (K % kBf16Step) != 0 || K > kMaxBf16K) return FP8Q_ERR_SHAPE;
    if ((K > 0 && (M > kMaxElems / K || N > kMaxElems / K)) || (M > 0 && N > kMaxElems / M)) return FP8Q_ERR_SHAPE;
    if (M > kMaxGemmRows || N > kMaxGemmRows) return FP8Q_ERR_SHAPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!y || (K > 0 && (!x || !w))) return FP8Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(w, 16) || misaligned(y, 4) || misaligned(bias, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_bf16_gemm(x, w, bias, y, y_dtype == FP8Q_OUT_BF16, M, N, K,
                                         static_cast<hipStream_t>(stream)));
}

int fp8_block_gemm_noalloc(const uint8_t *aq, const float *sa, const uint8_t *wq, const float *sw, void *y,
                           int y_dtype, int64_t M, int64_t N, int64_t K, void *stream) {
    static_assert(FP8Q_NOALLOC_SCRATCH_BYTES == fp8q::kNoallocScratchBytes, "scratch size in the header");
    const int dtype = y_dtype & 0xFF;
    const bool sa_kmajor = (y_dtype & FP8Q_SA_KMAJOR) != 0;
    const int mode = y_dtype & ~0xFF & ~FP8Q_SA_KMAJOR;
    if (dtype != FP8Q_OUT_F32 && dtype != FP8Q_OUT_BF16) return FP8Q_ERR_DTYPE;
    if (mode != 0 && mode != FP8Q_GEMM_FP8_PRODUCTS && mode != FP8Q_GEMM_EXACT_SLICES) return FP8Q_ERR_DTYPE;
    if (int e = shape_ok(M, K)) return e;
    if (int e = shape_ok(N, K)) return e;
    if (M > 0 && N > kMaxElems / M) return FP8Q_ERR_SHAPE;
    if (K > kMaxGemmK || M > kMaxGemmRows || N > kMaxGemmRows) return FP8Q_ERR_SHAPE;
    if (sa_kmajor && K > 0 && M >= kMaxKmajorScales / (K / kBlock)) return FP8Q_ERR_SHAPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    const bool exact = mode == FP8Q_GEMM_EXACT_SLICES || (mode == 0 && dtype == FP8Q_OUT_F32);
    // the split-K plan fp8_block_gemm would use with its full workspace must fit the static scratch
    if (K > 0 && fp8q::gemm_workspace_bytes(M, N, K, dtype == FP8Q_OUT_BF16, exact) > FP8Q_NOALLOC_SCRATCH_BYTES)
        return FP8Q_ERR_WORKSPACE;
    if (!y) return FP8Q_ERR_NULL;
    if (K > 0 && (!aq || !sa || !wq || !sw)) return FP8Q_ERR_NULL;
    if (misaligned(aq, 16) || misaligned(wq, 16) || misaligned(y, 16) || misaligned(sa, 4) || misaligned(sw, 4))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_block_gemm_noalloc(aq, sa, wq, sw, y, dtype == FP8Q_OUT_BF16, exact, sa_kmajor, M, N,
                                                  K, static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm(const uint8_t *aq, const float *sa, const uint8_t *wq, const float *sw, const int64_t *offsets,
                     void *y, int y_dtype, int64_t experts, int64_t rows, int64_t N, int64_t K, void *stream) {
    const int dtype = y_dtype & 0xFF;
    const int mode = y_dtype & ~0xFF;
    if (dtype != FP8Q_OUT_F32 && dtype != FP8Q_OUT_BF16) return FP8Q_ERR_DTYPE;
    if (mode != 0 && mode != FP8Q_GEMM_FP8_PRODUCTS && mode != FP8Q_GEMM_EXACT_SLICES) return FP8Q_ERR_DTYPE;
    if (experts < 1 || experts > fp8q::kMaxGroupedExperts) return FP8Q_ERR_SHAPE;
    if (int e = shape_ok(rows, K)) return e;
    if (int e = shape_ok(N, K)) return e;
    if (N > 0 && experts > kMaxElems / N) return FP8Q_ERR_SHAPE;
    if (int e = shape_ok(experts * N, K)) return e;
    if (rows > 0 && N > kMaxElems / rows) return FP8Q_ERR_SHAPE;
    if (K > kMaxGemmK || rows > INT32_MAX / 2 || N > kMaxGemmRows) return FP8Q_ERR_SHAPE;
    if (rows == 0 || N == 0) return FP8Q_OK;
    if (!y || !offsets) return FP8Q_ERR_NULL;
    if (K > 0 && (!aq || !sa || !wq || !sw)) return FP8Q_ERR_NULL;
    if (misaligned(aq, 16) || misaligned(wq, 16) || misaligned(y, 16) || misaligned(sa, 4) || misaligned(sw, 4) ||
        misaligned(offsets, 8))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    const bool exact = mode == FP8Q_GEMM_EXACT_SLICES || (mode == 0 && dtype == FP8Q_OUT_F32);
    return finish(fp8q::launch_grouped_gemm(aq, sa, wq, sw, offsets, y, dtype == FP8Q_OUT_BF16, exact, experts, rows,
                                            N, K, static_cast<hipStream_t>(stream)));
}

int fp8_act_quant_t(const uint16_t *x, uint8_t *qt, float *st, int64_t M, int64_t C, void *stream) {
    if (M < 0 || C < 0 || (C % 8) != 0) return FP8Q_ERR_SHAPE;
    const int64_t ldq = (M + kBlock - 1) / kBlock * kBlock;
    if ((C > 0 && ldq > kMaxElems / C) || (C + 127) / 128 > kMaxGridY || ldq / kBlock > kMaxBlocks256) return FP8Q_ERR_SHAPE;
    if (M == 0 || C == 0) return FP8Q_OK;
    if (!x || !qt || !st) return FP8Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(qt, 16) || misaligned(st, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_act_quant_t(x, qt, st, M, C, static_cast<hipStream_t>(stream)));
}

int fp8_weight_transpose(const uint8_t *wq, const float *sw, uint8_t *wqt, float *swt, int64_t N, int64_t K,
                         void *stream) {
    if (int e = shape_ok(N, K)) return e;
    if ((N + 63) / 64 > kMaxGridY || K / 64 > kMaxBlocks256) return FP8Q_ERR_SHAPE;   // 64x64-byte tiles
    if (N == 0 || K == 0) return FP8Q_OK;
    if (!wq || !sw || !wqt || !swt) return FP8Q_ERR_NULL;
    if (misaligned(wq, 16) || misaligned(wqt, 16) || misaligned(sw, 4) || misaligned(swt, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_weight_transpose(wq, sw, wqt, swt, N, K, static_cast<hipStream_t>(stream)));
}

int fp8_rowwise_gemm(const uint8_t *aq, const float *sa, const uint8_t *bq, const float *sb, void *y, int y_dtype,
                     int64_t M, int64_t N, int64_t K, void *workspace, size_t workspace_bytes, void *stream) {
    const int dtype = y_dtype & 0xFF;
    const int mode = y_dtype & ~0xFF;
    if (dtype != FP8Q_OUT_F32 && dtype != FP8Q_OUT_BF16) return FP8Q_ERR_DTYPE;
    if (mode != 0 && mode != FP8Q_GEMM_FP8_PRODUCTS && mode != FP8Q_GEMM_EXACT_SLICES) return FP8Q_ERR_DTYPE;
    if (int e = shape_ok(M, K)) return e;
    if (int e = shape_ok(N, K)) return e;
    if (M > 0 && N > kMaxElems / M) return FP8Q_ERR_SHAPE;
    if (K > kMaxGemmK || M > kMaxGemmRows || N > kMaxGemmRows) return FP8Q_ERR_SHAPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!y) return FP8Q_ERR_NULL;
    if (K > 0 && (!aq || !sa || !bq || !sb)) return FP8Q_ERR_NULL;
    if (misaligned(aq, 16) || misaligned(bq, 16) || misaligned(y, 16) || misaligned(sa, 4) || misaligned(sb, 4))
        return FP8Q_ERR_ALIGN;
    if (workspace == nullptr) workspace_bytes = 0;
    if (workspace_bytes && misaligned(workspace, 16)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    const bool exact = mode == FP8Q_GEMM_EXACT_SLICES || (mode == 0 && dtype == FP8Q_OUT_F32);
    return finish(fp8q::launch_rowwise_gemm(aq, sa, bq, sb, y, dtype == FP8Q_OUT_BF16, exact, M, N, K, workspace,
                                            workspace_bytes, static_cast<hipStream_t>(stream)));
}

size_t fp8_rowwise_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int y_dtype) {
    if (M <= 0 || N <= 0 || K <= 0 || (K % kBlock) != 0 || K > kMaxGemmK) return 0;
    if (N > kMaxElems / M || shape_ok(M, K) || shape_ok(N, K) || M > kMaxGemmRows || N > kMaxGemmRows) return 0;
    const int dtype = y_dtype & 0xFF;
    const int mode = y_dtype & ~0xFF;
    if (dtype != FP8Q_OUT_F32 && dtype != FP8Q_OUT_BF16) return 0;
    if (mode != 0 && mode != FP8Q_GEMM_FP8_PRODUCTS && mode != FP8Q_GEMM_EXACT_SLICES) return 0;
    const bool exact = mode == FP8Q_GEMM_EXACT_SLICES || (mode == 0 && dtype == FP8Q_OUT_F32);
    return fp8q::gemm_workspace_bytes(M, N, K, dtype == FP8Q_OUT_BF16, exact, true);
}

size_t fp8_block_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int y_dtype) {
    if (M <= 0 || N <= 0 || K <= 0 || (K % kBlock) != 0 || K > kMaxGemmK) return 0;
    if (N > kMaxElems / M || shape_ok(M, K) || shape_ok(N, K) || M > kMaxGemmRows || N > kMaxGemmRows) return 0;
    const int dtype = y_dtype & 0xFF;
    const int mode = y_dtype & ~0xFF & ~FP8Q_SA_KMAJOR;   // (the scale layout does not change the plan)
    if (dtype != FP8Q_OUT_F32 && dtype != FP8Q_OUT_BF16) return 0;
    if (mode != 0 && mode != FP8Q_GEMM_FP8_PRODUCTS && mode != FP8Q_GEMM_EXACT_SLICES) return 0;
    const bool exact = mode == FP8Q_GEMM_EXACT_SLICES || (mode == 0 && dtype == FP8Q_OUT_F32);
    return fp8q::gemm_workspace_bytes(M, N, K, dtype == FP8Q_OUT_BF16, exact);
}

int moe_route(const void *logits, int dtype, const float *bias, float *weights, int32_t *experts, int64_t T, int64_t E,
              int64_t top_k, int64_t groups, int64_t topk_groups, float scale, int flags, void *stream) {
    if (!is_type(dtype) || (flags & ~(FP8Q_MOE_SOFTMAX | FP8Q_MOE_GROUP_MAX | FP8Q_MOE_KEEP_SCORES)))
        return FP8Q_ERR_DTYPE;
    if (!routing_ok(T, E, top_k) || groups < 1 || groups > kMaxGroups || E % groups || topk_groups < 1 ||
        topk_groups > groups || top_k > topk_groups * (E / groups))
        return FP8Q_ERR_SHAPE;
    if (T == 0) return FP8Q_OK;
    if (!logits || !weights || !experts) return FP8Q_ERR_NULL;
    if (misaligned(logits, dtype == FP8Q_OUT_BF16 ? 2 : 4) || misaligned(bias, 4) || misaligned(weights, 4) ||
        misaligned(experts, 4))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_moe_route(logits, dtype == FP8Q_OUT_BF16, bias, weights, experts, T, (int)E, (int)top_k,
                                         (int)groups, (int)topk_groups, flags & FP8Q_MOE_SOFTMAX,
                                         !(flags & FP8Q_MOE_GROUP_MAX), !(flags & FP8Q_MOE_KEEP_SCORES), scale,
                                         static_cast<hipStream_t>(stream)));
}

int moe_route_backward(const float *dweights, const void *logits, int dtype, const int32_t *experts, void *dlogits,
                       int64_t T, int64_t E, int64_t top_k, float scale, int flags, void *stream) {
    if (!is_type(dtype) || (flags & ~(FP8Q_MOE_SOFTMAX | FP8Q_MOE_KEEP_SCORES))) return FP8Q_ERR_DTYPE;
    if (!routing_ok(T, E, top_k)) return FP8Q_ERR_SHAPE;
    if (T == 0) return FP8Q_OK;
    if (!dweights || !logits || !experts || !dlogits) return FP8Q_ERR_NULL;
    const uintptr_t size = dtype == FP8Q_OUT_BF16 ? 2 : 4;
    if (misaligned(logits, size) || misaligned(dlogits, size) || misaligned(dweights, 4) || misaligned(experts, 4))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_moe_route_backward(dweights, logits, dtype == FP8Q_OUT_BF16, experts, dlogits, T, (int)E,
                                                  (int)top_k, flags & FP8Q_MOE_SOFTMAX,
                                                  !(flags & FP8Q_MOE_KEEP_SCORES), scale,
                                                  static_cast<hipStream_t>(stream)));
}

size_t moe_place_workspace_bytes(int64_t T, int64_t top_k, int64_t experts) {
    if (!routing_ok(T, experts, top_k) || T == 0) return 0;
    return fp8q::moe_place_workspace_bytes(T * top_k, experts);
}

int moe_place(const int32_t *assigned, int64_t *offsets, int32_t *rows, int32_t *slots, int64_t T, int64_t top_k,
              int64_t experts, int64_t first, void *workspace, size_t workspace_bytes, void *stream) {
    if (!routing_ok(T, experts, top_k) || first < 0 || first > INT32_MAX - experts) return FP8Q_ERR_SHAPE;
    if (!offsets || (T > 0 && (!assigned || !rows || !slots))) return FP8Q_ERR_NULL;
    if (misaligned(assigned, 4) || misaligned(offsets, 8) || misaligned(rows, 4) || misaligned(slots, 4) ||
        misaligned(workspace, 4))
        return FP8Q_ERR_ALIGN;
    if (fp8q::moe_place_workspace_bytes(T * top_k, experts) > (workspace ? workspace_bytes : 0))
        return FP8Q_ERR_WORKSPACE;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_moe_place(assigned, offsets, rows, slots, T, (int)top_k, (int)experts, (int)first,
                                         workspace, static_cast<hipStream_t>(stream)));
}

int moe_combine(const void *h, int dtype, const int32_t *slots, const float *weights, void *y, int64_t T,
                int64_t top_k, int64_t rows, int64_t H, void *stream) {
    if (int e = combine_ok(dtype, T, rows, H, top_k)) return e;
    if (T == 0 || H == 0) return FP8Q_OK;
    if (!slots || !y || (rows > 0 && !h)) return FP8Q_ERR_NULL;
    const uintptr_t size = dtype == FP8Q_OUT_BF16 ? 2 : 4;
    if (misaligned(h, size) || misaligned(y, size) || misaligned(slots, 4) || misaligned(weights, 4))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_moe_combine(h, dtype == FP8Q_OUT_BF16, slots, weights, y, T, rows, H, (int)top_k,
                                           static_cast<hipStream_t>(stream)));
}

int moe_combine_backward(const void *dy, const void *h, int dtype, const int32_t *slots, const float *weights, void *dh,
                         float *dweights, int64_t T, int64_t top_k, int64_t rows, int64_t H, void *stream) {
    if (int e = combine_ok(dtype, T, rows, H, top_k)) return e;
    if (T == 0) return FP8Q_OK;
    if (!slots || !weights || !dweights || (H > 0 && (!dy || (rows > 0 && (!h || !dh))))) return FP8Q_ERR_NULL;
    const uintptr_t size = dtype == FP8Q_OUT_BF16 ? 2 : 4;
    if (misaligned(dy, size) || misaligned(h, size) || misaligned(dh, size) || misaligned(slots, 4) ||
        misaligned(weights, 4) || misaligned(dweights, 4))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_moe_combine_backward(dy, h, dtype == FP8Q_OUT_BF16, slots, weights, dh, dweights, T,
                                                    rows, H, (int)top_k, static_cast<hipStream_t>(stream)));
}

int int8_quant(const uint16_t *x, int8_t *q, float *s, int64_t M, int64_t K, void *stream) {
    if (M < 0 || K < 0 || K % kInt8Step || (K > 0 && M > kMaxElems / K) || M > kMaxTokens) return FP8Q_ERR_SHAPE;
    if (M == 0 || K == 0) return FP8Q_OK;
    if (!x || !q || !s) return FP8Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(q, 16) || misaligned(s, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_int8_quant(x, q, s, M, K, static_cast<hipStream_t>(stream)));
}

int int8_gemm(const int8_t *a, const float *sa, const int8_t *w, const float *sw, const float *bias, void *y,
              int y_dtype, int64_t M, int64_t N, int64_t K, void *stream) {
    if (int e = int8_ok(y_dtype, M, N, K)) return e;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!y || (K > 0 && (!a || !sa || !w || !sw))) return FP8Q_ERR_NULL;
    if (misaligned(a, 16) || misaligned(w, 16) || misaligned(y, 4) || misaligned(sa, 4) || misaligned(sw, 4) ||
        misaligned(bias, 4))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_int8_gemm(a, sa, w, sw, bias, y, y_dtype == FP8Q_OUT_BF16, M, N, K,
                                         static_cast<hipStream_t>(stream)));
}

size_t int8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (int8_ok(FP8Q_OUT_F32, M, N, K) || M == 0 || N == 0 || M > kMaxTokens) return 0;
    return fp8q::int8_linear_workspace_bytes(M, N, K);
}

int int8_linear(const uint16_t *x, const int8_t *w, const float *sw, const float *bias, void *y, int y_dtype, int64_t M,
                int64_t N, int64_t K, void *workspace, size_t workspace_bytes, void *stream) {
    if (int e = int8_ok(y_dtype, M, N, K)) return e;
    if (M > kMaxTokens) return FP8Q_ERR_SHAPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!y || (K > 0 && (!x || !w || !sw))) return FP8Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(w, 16) || misaligned(y, 4) || misaligned(sw, 4) || misaligned(bias, 4) ||
        misaligned(workspace, 16))
        return FP8Q_ERR_ALIGN;
    if (fp8q::int8_linear_workspace_bytes(M, N, K) > (workspace ? workspace_bytes : 0)) return FP8Q_ERR_WORKSPACE;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_int8_linear(x, w, sw, bias, y, y_dtype == FP8Q_OUT_BF16, M, N, K, workspace,
                                           static_cast<hipStream_t>(stream)));
}

int int8_grouped_gemm(const int8_t *a, const float *sa, const int8_t *w, const float *sw, const int64_t *offsets,
                      const int32_t *rows, void *y, int y_dtype, int64_t experts, int64_t M, int64_t tokens, int64_t N,
                      int64_t K, void *stream) {
    if (int e = int8_ok(y_dtype, M, N, K)) return e;
    if (experts < 1 || experts > fp8q::kMaxGroupedExperts || M > INT32_MAX / 2) return FP8Q_ERR_SHAPE;
    if (N > 0 && K > 0 && experts > kMaxElems / N / K) return FP8Q_ERR_SHAPE;
    if (tokens < 0 || tokens > INT32_MAX || (!rows && M > 0 && tokens != M)) return FP8Q_ERR_SHAPE;
    if (rows && K > 0 && tokens > kMaxGatherBytes / K) return FP8Q_ERR_SHAPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!y || !offsets || (K > 0 && (!w || !sw || (tokens > 0 && (!a || !sa))))) return FP8Q_ERR_NULL;
    if (misaligned(a, 16) || misaligned(w, 16) || misaligned(y, 4) || misaligned(sa, 4) || misaligned(sw, 4) ||
        misaligned(offsets, 8) || misaligned(rows, 4))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_int8_grouped_gemm(a, sa, w, sw, offsets, rows, y, y_dtype == FP8Q_OUT_BF16, experts, M,
                                                 tokens, N, K, static_cast<hipStream_t>(stream)));
}

int residual_norm(const void *x, const void *y, int dtype, const float *weight, const float *post, const void *gate,
                  int flags, float scale, float eps, void *t, void *z, int64_t T, int64_t H, void *stream) {
    if (int e = norm_ok(dtype, flags, T, H)) return e;
    if (T == 0) return FP8Q_OK;
    if (!x || (weight ? !z : !t)) return FP8Q_ERR_NULL;
    const bool gates = gate && (flags & FP8Q_NORM_GATES);
    const uintptr_t size = dtype == FP8Q_OUT_BF16 ? 2 : 4;
    if (misaligned(x, size) || misaligned(y, size) || misaligned(t, size) || misaligned(z, size) ||
        misaligned(gate, gates ? size : 4) || misaligned(weight, 4) || misaligned(post, 4))
        return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_residual_norm(x, y, dtype == FP8Q_OUT_BF16, weight, y ? post : nullptr,
                                             y && !gates ? static_cast<const float *>(gate) : nullptr,
                                             y && gates ? gate : nullptr, scale, eps, t, weight ? z : nullptr, T, H,
                                             static_cast<hipStream_t>(stream)));
}

size_t residual_norm_backward_workspace_bytes(int64_t T, int64_t H) {
    return norm_ok(FP8Q_OUT_F32, 0, T, H) ? 0 : fp8q::residual_norm_grad_workspace_bytes(T, H);
}

int residual_norm_backward(const void *dt, const void *dz, const void *t, const void *y, int dtype, const float *weight,
                           const float *post, const void *gate, int flags, float scale, float eps, void *dx, void *dy,
                           float *dweight, float *dpost, void *dgate, int64_t T, int64_t H, void *workspace,
                           size_t workspace_bytes, void *stream) {
    if (int e = norm_ok(dtype, flags, T, H)) return e;
    if (!y && T > 0) post = nullptr, gate = nullptr;   // (no rows: the sums are wanted whatever y points to)
    const bool gates = gate && (flags & FP8Q_NORM_GATES);
    if ((weight && !dweight) || (post && !dpost) || (gate && !dgate && (!gates || T > 0))) return FP8Q_ERR_NULL;
    if (T > 0 && (!dx || (y && !dy) || (weight && (!dz || !t)) || (!weight && !dt))) return FP8Q_ERR_NULL;
    const uintptr_t size = dtype == FP8Q_OUT_BF16 ? 2 : 4;
    if (misaligned(dt, size) || misaligned(dz, size) || misaligned(t, size) || misaligned(y, size) ||
        misaligned(dx, size) || misaligned(dy, size) || misaligned(gate, gates ? size : 4) ||
        misaligned(dgate, gates ? size : 4) || misaligned(weight, 4) || misaligned(post, 4) || misaligned(dweight, 4) ||
        misaligned(dpost, 4) || misaligned(workspace, 16))
        return FP8Q_ERR_ALIGN;
    if (fp8q::residual_norm_grad_workspace_bytes(T, H) > (workspace ? workspace_bytes : 0)) return FP8Q_ERR_WORKSPACE;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_residual_norm_backward(
        dt, dz, t, y, dtype == FP8Q_OUT_BF16, weight, post, gate && !gates ? static_cast<const float *>(gate) : nullptr,
        gates ? gate : nullptr, scale, eps, dx, dy, weight ? dweight : nullptr, post ? dpost : nullptr,
        gate && !gates ? static_cast<float *>(dgate) : nullptr, gates ? dgate : nullptr, T, H, workspace,
        static_cast<hipStream_t>(stream)));
}

int gated_linear(const uint16_t *x, const uint16_t *w, void *h, int h_dtype, uint16_t *gu, int act, int64_t M,
                 int64_t F, int64_t K, void *stream) {
    if (!is_type(h_dtype) || (act != FP8Q_ACT_SILU && act != FP8Q_ACT_GELU)) return FP8Q_ERR_DTYPE;
    if (!gated_ok(M, F, K)) return FP8Q_ERR_SHAPE;
    if (M == 0 || F == 0) return FP8Q_OK;
    if (!h || (K > 0 && (!x || !w))) return FP8Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(w, 16) || misaligned(h, 4) || misaligned(gu, 4)) return FP8Q_ERR_ALIGN;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_gated_linear(x, w, h, h_dtype == FP8Q_OUT_BF16, gu, act == FP8Q_ACT_GELU, M, F, K,
                                            static_cast<hipStream_t>(stream)));
}

size_t gated_linear_backward_workspace_bytes(int64_t M, int64_t F, int64_t K) {
    return gated_gradient_bytes(M, F, K, false);
}

size_t gated_linear_backward_wide_workspace_bytes(int64_t M, int64_t F, int64_t K) {
    return gated_gradient_bytes(M, F, K, true);
}

int gated_linear_backward(const uint16_t *dh, const uint16_t *x, const uint16_t *w, const uint16_t *gu, int act, void *dx,
                          int dx_dtype, void *dw, int dw_dtype, int64_t M, int64_t F, int64_t K, void *workspace,
                          size_t workspace_bytes, void *stream) {
    const bool wide = act >= 0 && (act & FP8Q_GATED_WIDE);
    if (wide) act -= FP8Q_GATED_WIDE;
    if (!is_type(dx_dtype) || !is_type(dw_dtype) || (act != FP8Q_ACT_SILU && act != FP8Q_ACT_GELU)) return FP8Q_ERR_DTYPE;
    if (!gated_ok(M, F, K)) return FP8Q_ERR_SHAPE;
    if (K == 0 || (!dx && !dw)) return FP8Q_OK;
    if (M > 0 && F > 0 && (!dh || !w || !x)) return FP8Q_ERR_NULL;
    if (misaligned(dh, 16) || misaligned(x, 16) || misaligned(w, 16) || misaligned(gu, 16) || misaligned(dx, 4) ||
        misaligned(dw, 4) || misaligned(workspace, 16))
        return FP8Q_ERR_ALIGN;
    const fp8q::GatedGradPlans plans = fp8q::gated_gradient_plans(M, F, K, wide);
    if (!plans.fits) return FP8Q_ERR_SHAPE;
    if (fp8q::gated_linear_backward_workspace_bytes(plans, M, F, K) > (workspace ? workspace_bytes : 0)) return FP8Q_ERR_WORKSPACE;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_gated_linear_backward(dh, x, w, gu, act == FP8Q_ACT_GELU, dx, dx_dtype == FP8Q_OUT_BF16, dw,
                                                     dw_dtype == FP8Q_OUT_BF16, M, F, K, plans, workspace,
                                                     static_cast<hipStream_t>(stream)));
}

size_t adapter_linear_workspace_bytes(int64_t M, int64_t K, int64_t rank) {
    return adapter_ok(M, 0, K, 0, rank) ? fp8q::adapter_linear_workspace_bytes(M, K, rank) : 0;
}

int adapter_linear(const uint16_t *x, const uint16_t *w, const float *bias, const uint16_t *a, const uint16_t *b,
                   const float *scales, const int32_t *ids, const void *base, void *y, int y_dtype, int64_t M,
                   int64_t N, int64_t K, int64_t adapters, int64_t rank, void *workspace, size_t workspace_bytes,
                   void *stream) {
    if (!is_type(y_dtype)) return FP8Q_ERR_DTYPE;
    if (!adapter_ok(M, N, K, adapters, rank)) return FP8Q_ERR_SHAPE;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (!y || !ids || (K > 0 && !x) || (K > 0 && !w && !base) || (adapters > 0 && (!b || (K > 0 && !a)))) return FP8Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(w, 16) || misaligned(a, 16) || misaligned(b, 16) || misaligned(bias, 4) ||
        misaligned(scales, 4) || misaligned(ids, 4) || misaligned(base, 4) || misaligned(y, 4) || misaligned(workspace, 16))
        return FP8Q_ERR_ALIGN;
    if (adapters > 0 && fp8q::adapter_linear_workspace_bytes(M, K, rank) > (workspace ? workspace_bytes : 0))
        return FP8Q_ERR_WORKSPACE;
    if (int e = check_device()) return e;
    return finish(fp8q::launch_adapter_linear(x, w, bias, a, b, scales, ids, base, y, y_dtype == FP8Q_OUT_BF16, M, N, K,
                                              adapters, rank, workspace, static_cast<hipStream_t>(stream)));
}

int fp8q_gemm_force_config(int config, int splits) {
    return fp8q::gemm_force_config(config, splits) ? FP8Q_OK : FP8Q_ERR_SHAPE;
}

const char *fp8q_gemm_config_name(int config) { return fp8q::gemm_config_name(config); }

int fp8q_gemm_plan(int64_t M, int64_t N, int64_t K, int y_dtype, int *config, int *splits) {
    if (!config || !splits) return FP8Q_ERR_NULL;
    const int dtype = y_dtype & 0xFF;
    const int mode = y_dtype & ~0xFF & ~FP8Q_SA_KMAJOR;   // (the scale layout does not change the plan)
    if (dtype != FP8Q_OUT_F32 && dtype != FP8Q_OUT_BF16) return FP8Q_ERR_DTYPE;
    if (mode != 0 && mode != FP8Q_GEMM_FP8_PRODUCTS && mode != FP8Q_GEMM_EXACT_SLICES) return FP8Q_ERR_DTYPE;
    if (M <= 0 || N <= 0 || K <= 0 || (K % kBlock) != 0 || K > kMaxGemmK) return FP8Q_ERR_SHAPE;
    if (N > kMaxElems / M || shape_ok(M, K) || shape_ok(N, K) || M > kMaxGemmRows || N > kMaxGemmRows)
        return FP8Q_ERR_SHAPE;
    const bool exact = mode == FP8Q_GEMM_EXACT_SLICES || (mode == 0 && dtype == FP8Q_OUT_F32);
    fp8q::gemm_plan(M, N, K, dtype == FP8Q_OUT_BF16, exact, config, splits);
    return FP8Q_OK;
}

int fp8q_dense_plan(int call, int64_t M, int64_t N, int64_t K, int64_t rank, int64_t *plan) {
    if (call < FP8Q_PLAN_GATED || call > FP8Q_PLAN_GATED_BACKWARD_WIDE) return FP8Q_ERR_DTYPE;
    const bool adapters = call == FP8Q_PLAN_ADAPTER || call == FP8Q_PLAN_ADAPTER_ADD;
    if (M <= 0 || N <= 0 || (adapters ? !adapter_ok(M, N, K, 1, rank) : !gated_ok(M, N, K))) return FP8Q_ERR_SHAPE;
    if (!plan) return FP8Q_ERR_NULL;
    fp8q::LaunchReport r[2] = {};
    if (call == FP8Q_PLAN_GATED) fp8q::gated_report(M, N, K, r);
    else if (adapters) fp8q::adapter_report(M, N, K, rank, call == FP8Q_PLAN_ADAPTER_ADD, r);
    else fp8q::gated_gradient_report(M, N, K, call == FP8Q_PLAN_GATED_BACKWARD_WIDE, r);
    for (int i = 0; i < 2; ++i) {
        const int64_t row[6] = {r[i].rows, r[i].columns, r[i].parts, r[i].shared, r[i].workgroups, r[i].threads};
        for (int j = 0; j < 6; ++j) plan[6 * i + j] = row[j];
    }
    return FP8Q_OK;
}

const char *fp8q_strerror(int status) {
    switch (status) {
    case FP8Q_OK: return "ok";
    case FP8Q_ERR_NULL: return "a required pointer is NULL";
    case FP8Q_ERR_SHAPE: return "invalid shape (negative size, K not a multiple of 128 (8-bit integers: 16; the dense block: sizes of 8), or too large)";
    case FP8Q_ERR_ALIGN: return "pointer alignment below what the entry point requires";
    case FP8Q_ERR_DTYPE: return "unknown element type or flag";
    case FP8Q_ERR_UNSUPPORTED: return "no gfx950 device is current";
    case FP8Q_ERR_LAUNCH: return "kernel launch failed";
    case FP8Q_ERR_WORKSPACE:
        return "the shape's split-K schedule needs more scratch than the static scratch holds "
               "(FP8Q_NOALLOC_SCRATCH_BYTES); call fp8_block_gemm with a workspace instead (moe_place, int8_linear: "
               "the workspace is smaller than their _workspace_bytes)";
    default: return "unknown status";
    }
}

int fp8q_version(void) { return (1 << 16) | 8; }

}  // extern "C"
