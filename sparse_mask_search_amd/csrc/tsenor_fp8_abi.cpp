// tsenor_fp8_abi.cpp -- the extern "C" boundary declared in include/tsenor_fp8.h:
// argument checks on the host, before any HIP call, and the launches.  Nothing
// here allocates or is kept between calls.
#include <hip/hip_runtime.h>

#include "tsenor_fp8.h"
#include "tsenor_internal.h"

namespace {

// Operands of at most this many entries keep every offset and every count of workgroups
// inside int64; whether the workgroups fit one launch is for the launch functions (grid_fits).
constexpr int64_t kMaxEntries = int64_t(1) << 40;

bool misaligned(const void* p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}
int64_t blocks128(int64_t v) { return (v + 127) / 128; }
// rows x cols entries, each padded by up to `pad`, without overflow
bool too_big(int64_t rows, int64_t cols, int64_t pad = 0) {
    return rows > kMaxEntries || cols > kMaxEntries || (cols > 0 && rows + pad > kMaxEntries / (cols + pad));
}
bool float_type(int t) { return t == TSENOR_F32 || t == TSENOR_BF16; }
uintptr_t element_size(int t) { return t == TSENOR_F32 ? 4 : 2; }

int status(int e, const char* where) {
    if (e == tsenor::kGridTooLarge) return TSENOR_ERR_SHAPE;
    return e == hipSuccess ? TSENOR_OK : tsenor::hip_error(e, where);
}

}  // namespace

extern "C" {

int tsenor_quant_fp8(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                     uint8_t* values, uint8_t* scales, uint8_t* values_t, uint8_t* scales_t,
                     void* stream) {
    if ((values == nullptr) != (scales == nullptr) || (values_t == nullptr) != (scales_t == nullptr) ||
        (values == nullptr && values_t == nullptr) || (X == nullptr && rows != 0))
        return TSENOR_ERR_NULL;
    if (!float_type(dtype)) return TSENOR_ERR_DTYPE;
    if (rows < 0 || cols <= 0 || ldx < cols || too_big(rows, ldx, 128)) return TSENOR_ERR_SHAPE;
    if (misaligned(values, 16) || misaligned(values_t, 16) || misaligned(X, element_size(dtype)))
        return TSENOR_ERR_SHAPE;
    if (rows == 0) return TSENOR_OK;
    return status(tsenor::launch_quant_fp8(X, dtype == TSENOR_BF16, rows, cols, ldx, values, scales,
                                           values_t, scales_t, stream),
                  "quant_fp8 kernel launch");
}

int tsenor_compress24_fp8(const void* W, int dtype, int64_t batch, int64_t stride, int64_t rows,
                          int64_t cols, int64_t ld, const uint32_t* mask, uint8_t* values,
                          uint32_t* meta, uint8_t* scales, uint8_t* values_t, uint32_t* meta_t,
                          uint8_t* scales_t, int* bad, int* bad_t, void* stream) {
    const int given = (values != nullptr) + (meta != nullptr) + (scales != nullptr);
    const int given_t = (values_t != nullptr) + (meta_t != nullptr) + (scales_t != nullptr);
    if (W == nullptr || mask == nullptr || given % 3 != 0 || given_t % 3 != 0 || given + given_t == 0)
        return TSENOR_ERR_NULL;
    if (!float_type(dtype)) return TSENOR_ERR_DTYPE;
    if (batch < 0 || rows <= 0 || cols <= 0 || rows % 4 != 0 || cols % 4 != 0 || ld < cols ||
        too_big(rows, ld) || (batch > 1 && stride < rows * ld) || too_big(batch, stride) ||
        too_big(batch, (rows + 128) * (cols + 128)))
        return TSENOR_ERR_SHAPE;
    if (misaligned(W, element_size(dtype)) || misaligned(mask, 4) || misaligned(values, 16) ||
        misaligned(meta, 16) || misaligned(values_t, 16) || misaligned(meta_t, 16) ||
        misaligned(bad, 4) || misaligned(bad_t, 4))
        return TSENOR_ERR_SHAPE;
    if (batch == 0) return TSENOR_OK;
    return status(tsenor::launch_compress24_fp8(W, dtype == TSENOR_BF16, batch, stride, rows, cols, ld,
                                                mask, values, meta, scales, values_t, meta_t, scales_t,
                                                bad, bad_t, stream),
                  "compress24_fp8 kernel launch");
}

int tsenor_spmm24_fp8(const void* X, int xtype, const uint8_t* xscales, int64_t n, int64_t ldx,
                      const uint8_t* values, const uint32_t* meta, const uint8_t* scales,
                      int64_t m, int64_t k, void* Y, int ytype, int64_t ldy, void* stream) {
    if (values == nullptr || meta == nullptr || scales == nullptr ||
        (n != 0 && (X == nullptr || Y == nullptr || (xtype == TSENOR_E4M3 && xscales == nullptr))))
        return TSENOR_ERR_NULL;
    if ((xtype != TSENOR_E4M3 && xtype != TSENOR_BF16) || !float_type(ytype)) return TSENOR_ERR_DTYPE;
    if (n < 0 || m <= 0 || k <= 0 || ldy < m || too_big(m, k, 128) || too_big(n, ldx) || too_big(n, ldy))
        return TSENOR_ERR_SHAPE;
    if (xtype == TSENOR_E4M3 ? (ldx < 128 * blocks128(k) || ldx % 16 != 0 || misaligned(X, 16))
                             : (n > 16 || ldx < k || misaligned(X, 2)))
        return TSENOR_ERR_SHAPE;
    if (misaligned(values, 16) || misaligned(meta, 16) || misaligned(Y, element_size(ytype)))
        return TSENOR_ERR_SHAPE;
    if (n == 0) return TSENOR_OK;
    return status(tsenor::launch_spmm24_fp8(X, xtype == TSENOR_BF16, xscales, n, ldx, values, meta, scales,
                                            m, k, Y, ytype == TSENOR_BF16, ldy, stream),
                  "spmm24_fp8 kernel launch");
}

int tsenor_gemm_fp8(const uint8_t* A, const uint8_t* a_scales, int64_t p, const uint8_t* B,
                    const uint8_t* b_scales, int64_t q, int64_t k, const uint32_t* mask, void* C,
                    int ctype, int64_t ldc, void* stream) {
    if (C == nullptr || (k != 0 && (A == nullptr || a_scales == nullptr || B == nullptr || b_scales == nullptr)))
        return TSENOR_ERR_NULL;
    if (!float_type(ctype)) return TSENOR_ERR_DTYPE;
    if (p <= 0 || q <= 0 || k < 0 || ldc < q || too_big(p, k, 128) || too_big(q, k, 128) || too_big(p, ldc))
        return TSENOR_ERR_SHAPE;
    if (misaligned(A, 16) || misaligned(B, 16) || misaligned(mask, 4) || misaligned(C, element_size(ctype)))
        return TSENOR_ERR_SHAPE;
    return status(tsenor::launch_gemm_fp8(A, a_scales, p, B, b_scales, q, k, mask, C, ctype == TSENOR_BF16,
                                          ldc, stream),
                  "gemm_fp8 kernel launch");
}

// The workspace's parts, each on a multiple of 256 bytes.
struct MoeLayout {
    size_t logits, xpad, hidden, weights, counts, chosen, lists, gains, total;
};
static MoeLayout moe_layout(int64_t n, int64_t d, int64_t f, int64_t experts, int topk) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    MoeLayout w;
    w.logits = 0;
    w.xpad = up((size_t)(n * experts) * sizeof(double));
    w.hidden = w.xpad + up((size_t)(n * blocks128(d) * 128) * 2);
    w.weights = w.hidden + up((size_t)(n * topk * blocks128(f) * 128) * 4);
    w.counts = w.weights + up((size_t)(n * topk) * sizeof(float));
    w.chosen = w.counts + up((size_t)experts * sizeof(int));
    w.lists = w.chosen + up((size_t)experts * sizeof(int));
    w.gains = w.lists + up((size_t)experts * 64 * sizeof(int));
    w.total = w.gains + up((size_t)(n * topk * ((d + 3) / 4 * 4)) * sizeof(float));
    return w;
}
static int moe_check(int64_t n, int64_t d, int64_t f, int64_t experts, int topk) {
    if (topk < 1 || topk > 16 || experts > 512 || topk > experts) return TSENOR_ERR_PARAM;
    if (n < 0 || n > 64 || d <= 0 || f <= 0 || d > (1 << 20) || f > (1 << 20) || too_big(experts * 128, d + 128) ||
        too_big(experts * 128, f + 128) || too_big(experts * (d + 128), f + 128))
        return TSENOR_ERR_SHAPE;
    return TSENOR_OK;
}

size_t tsenor_moe24_fp8_workspace(int64_t n, int64_t d, int64_t f, int64_t experts, int topk) {
    if (moe_check(n, d, f, experts, topk) != TSENOR_OK) return 0;
    return moe_layout(n, d, f, experts, topk).total;
}

int tsenor_moe24_fp8(const uint16_t* X, int64_t n, int64_t ldx, int64_t d, const uint16_t* router,
                     int64_t ldr, int64_t experts, int topk, const uint8_t* gate_values,
                     const uint32_t* gate_meta, const uint8_t* gate_scales,
                     const uint8_t* up_values, const uint32_t* up_meta, const uint8_t* up_scales,
                     const uint8_t* down_values, const uint32_t* down_meta,
                     const uint8_t* down_scales, int64_t f, void* workspace,
                     size_t workspace_bytes, uint16_t* Y, int64_t ldy, int* ids, float* weights,
                     void* stream) {
    if (router == nullptr || gate_values == nullptr || gate_meta == nullptr || gate_scales == nullptr ||
        up_values == nullptr || up_meta == nullptr || up_scales == nullptr || down_values == nullptr ||
        down_meta == nullptr || down_scales == nullptr ||
        (n != 0 && (X == nullptr || Y == nullptr || workspace == nullptr)))
        return TSENOR_ERR_NULL;
    const int code = moe_check(n, d, f, experts, topk);
    if (code != TSENOR_OK) return code;
    if (ldx < d || ldr < d || ldy < d || too_big(experts, ldr) || too_big(64, ldx) || too_big(64, ldy))
        return TSENOR_ERR_SHAPE;
    const MoeLayout w = moe_layout(n, d, f, experts, topk);
    if (misaligned(X, 2) || misaligned(router, 2) || misaligned(gate_values, 16) ||
        misaligned(gate_meta, 16) || misaligned(up_values, 16) || misaligned(up_meta, 16) ||
        misaligned(down_values, 16) || misaligned(down_meta, 16) || misaligned(workspace, 16) ||
        misaligned(Y, 2) || misaligned(ids, 4) || misaligned(weights, 4) || workspace_bytes < w.total)
        return TSENOR_ERR_SHAPE;
    if (n == 0) return TSENOR_OK;
    char* ws = static_cast<char*>(workspace);
    tsenor::MoeJob job;
    job.x = X;
    job.router = router;
    job.gate = {gate_values, gate_meta, gate_scales};
    job.up = {up_values, up_meta, up_scales};
    job.down = {down_values, down_meta, down_scales};
    job.n = n;
    job.d = d;
    job.f = f;
    job.experts = experts;
    job.ldx = ldx;
    job.ldr = ldr;
    job.ldy = ldy;
    job.topk = topk;
    job.logits = reinterpret_cast<double*>(ws + w.logits);
    job.xpad = reinterpret_cast<uint16_t*>(ws + w.xpad);
    job.hidden = reinterpret_cast<uint16_t*>(ws + w.hidden);
    job.weights = reinterpret_cast<float*>(ws + w.weights);
    job.counts = reinterpret_cast<int*>(ws + w.counts);
    job.chosen = reinterpret_cast<int*>(ws + w.chosen);
    job.lists = reinterpret_cast<int*>(ws + w.lists);
    job.gains = reinterpret_cast<float*>(ws + w.gains);
    job.xvec = !misaligned(X, 16) && ldx % 8 == 0;
    job.rvec = !misaligned(router, 16) && ldr % 8 == 0;
    job.y = Y;
    job.ids_out = ids;
    job.weights_out = weights;
    return status(tsenor::launch_moe24_fp8(job, stream), "moe24_fp8 kernel launch");
}

}  // extern "C"
