// tsenor_ops_abi.cpp -- the extern "C" boundary declared in include/tsenor_ops.h:
// argument checks on the host, before any HIP call, and the launches.  Nothing
// here allocates or is kept between calls.
#include <hip/hip_runtime.h>

#include "tsenor_checks.h"
#include "tsenor_internal.h"
#include "tsenor_ops.h"
#include "tsenor_ops_internal.h"

namespace {

using namespace tsenor;

constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxReduce = int64_t(1) << 17;
constexpr int64_t kMaxExperts = 1024;

// rows of four neighbouring entries may be written at once
bool four(const void* p, int type, int64_t ld) { return !misaligned(p, 4 * element_size(type)) && ld % 4 == 0; }
// rows of eight bf16 entries
bool eight(const void* p, int64_t ld) { return !misaligned(p, 16) && ld % 8 == 0; }

// Whether a gradient is one that the kernels can take.
int grad_check(const tsenor_grad& g, bool write) {
    if (g.rows < 0 || g.cols < 0 || g.ld < g.cols || too_big(g.rows, g.ld)) return TSENOR_ERR_SHAPE;
    if (!float_type(g.dtype)) return TSENOR_ERR_DTYPE;
    if (g.rows == 0 || g.cols == 0) return TSENOR_OK;
    if (g.grad == nullptr || (write && g.out == nullptr)) return TSENOR_ERR_NULL;
    if (write && (g.ldo < g.cols || too_big(g.rows, g.ldo) || (g.out == g.grad && g.ldo != g.ld)))
        return TSENOR_ERR_SHAPE;
    if (misaligned(g.grad, element_size(g.dtype)) || misaligned(g.mask, 4) ||
        (write && misaligned(g.out, element_size(g.dtype))))
        return TSENOR_ERR_SHAPE;
    return TSENOR_OK;
}

GradJob grad_job(const tsenor_grad& g, bool write) {
    GradJob j;
    j.grad = g.grad;
    j.out = write ? g.out : nullptr;
    j.mask = g.mask;
    j.rows = g.rows;
    j.cols = g.cols;
    j.ld = g.rows == 1 ? g.cols : g.ld;
    j.ldo = write ? (g.rows == 1 ? g.cols : g.ldo) : j.ld;
    j.bf16 = g.dtype == TSENOR_BF16;
    const bool aligned = !misaligned(g.grad, 16) && (!write || !misaligned(g.out, 16));
    const int64_t per16 = 16 / element_size(g.dtype);
    const bool flat = aligned && j.ld == j.cols && j.ldo == j.cols;
    if (flat && g.mask == nullptr)
        j.layout = kFlat;
    else if (aligned && j.cols % 8 == 0 && j.ld % per16 == 0 && j.ldo % per16 == 0)
        j.layout = kRows;
    else
        j.layout = flat && (j.cols >= 8 || j.rows == 1) ? kFlat : kLoose;
    return j;
}

// Calls fn(list, blocks, blocks of the launches before) for the tensors of each launch; the
// number of all blocks in *total.
template <class F>
int each_launch(const tsenor_grad* grads, int count, bool write, int* total, F fn) {
    int before = 0;
    GradList list;
    list.count = 0;
    int64_t chunks = 0;
    const auto flush = [&]() {
        if (list.count == 0) return (int)hipSuccess;
        list.chunks = (int32_t)chunks;
        const int blocks = chunks < kGradBlocks ? (int)chunks : kGradBlocks;
        const int e = fn(list, blocks, before);
        before += blocks;
        list.count = 0;
        chunks = 0;
        return e;
    };
    for (int i = 0; i < count; ++i) {
        if (grads[i].rows == 0 || grads[i].cols == 0) continue;
        const int64_t n = (grads[i].rows * grads[i].cols + grad_chunk() - 1) / grad_chunk();
        if (list.count == kGradsPerLaunch) {  // their chunks, at most 2^25 each, fit 31 bits
            const int e = flush();
            if (e != hipSuccess) return e;
        }
        GradJob& j = list.job[list.count++];
        j = grad_job(grads[i], write);
        j.first = (int32_t)chunks;
        chunks += n;
    }
    const int e = flush();
    *total = before;
    return e;
}

int grads_check(const tsenor_grad* grads, int count, bool write, const void* workspace, size_t bytes,
                const float* norm) {
    if (count < 0) return TSENOR_ERR_PARAM;
    if (workspace == nullptr || norm == nullptr || (count > 0 && grads == nullptr)) return TSENOR_ERR_NULL;
    for (int i = 0; i < count; ++i) {
        const int code = grad_check(grads[i], write);
        if (code != TSENOR_OK) return code;
    }
    if (misaligned(workspace, 8) || misaligned(norm, 4) || bytes < tsenor_grads_workspace(count))
        return TSENOR_ERR_SHAPE;
    return TSENOR_OK;
}

}  // namespace

extern "C" {

int tsenor_grouped_mm(const uint16_t* X, int64_t rows, int64_t ldx, const uint16_t* W, int transpose,
                      int64_t experts, int64_t stride, int64_t ldw, int64_t m, int64_t k, const int* ends,
                      void* Y, int ytype, int64_t ldy, void* stream) {
    if (W == nullptr || ends == nullptr || (rows != 0 && (X == nullptr || Y == nullptr))) return TSENOR_ERR_NULL;
    if (!float_type(ytype)) return TSENOR_ERR_DTYPE;
    if ((transpose != 0 && transpose != 1) || experts < 1 || experts > kMaxExperts) return TSENOR_ERR_PARAM;
    const int64_t wrows = transpose ? k : m, wcols = transpose ? m : k;
    if (rows < 0 || rows >= kMaxRows || m <= 0 || k <= 0 || k >= kMaxRows || ldx < k || ldy < m || ldw < wcols)
        return TSENOR_ERR_SHAPE;
    if (too_big(rows, ldx) || too_big(rows, ldy) || too_big(wrows, ldw) || (experts > 1 && stride < wrows * ldw) ||
        too_big(experts, stride))
        return TSENOR_ERR_SHAPE;
    if (misaligned(X, 2) || misaligned(W, 2) || misaligned(ends, 4) || misaligned(Y, element_size(ytype)))
        return TSENOR_ERR_SHAPE;
    if (rows == 0) return TSENOR_OK;
    GroupedJob j = {};
    j.a = W;
    j.b = X;
    j.lda = 2 * ldw;
    j.ldb = 2 * ldx;
    j.astride = 2 * stride;
    j.inner = m;
    j.kbytes = 2 * k;
    j.rows = (int32_t)rows;
    j.experts = (int32_t)experts;
    j.ends = ends;
    j.out = Y;
    j.ldo = ldy;
    j.ovec = four(Y, ytype, ldy);
    j.ovec8 = eight(Y, ldy);
    return status(launch_grouped_mm(j, transpose == 1, ytype == TSENOR_BF16, stream), "grouped_mm kernel launch");
}

int tsenor_grouped_wgrad(const uint16_t* dY, int64_t lddy, const uint16_t* X, int64_t ldx, int64_t rows,
                         int64_t experts, int64_t m, int64_t k, const int* ends, const uint32_t* mask, void* C,
                         int ctype, int64_t stride, int64_t ldc, void* stream) {
    if (C == nullptr || ends == nullptr || (rows != 0 && (X == nullptr || dY == nullptr))) return TSENOR_ERR_NULL;
    if (!float_type(ctype)) return TSENOR_ERR_DTYPE;
    if (experts < 1 || experts > kMaxExperts) return TSENOR_ERR_PARAM;
    if (rows < 0 || rows >= kMaxRows || m <= 0 || k <= 0 || lddy < m || ldx < k || ldc < k || too_big(rows, lddy) ||
        too_big(rows, ldx) || too_big(m, ldc) || (experts > 1 && stride < m * ldc) || too_big(experts, stride) ||
        too_big(experts, m * ldc))
        return TSENOR_ERR_SHAPE;
    if (misaligned(X, 2) || misaligned(dY, 2) || misaligned(ends, 4) || misaligned(mask, 4) ||
        misaligned(C, element_size(ctype)))
        return TSENOR_ERR_SHAPE;
    GroupedJob j = {};
    j.a = X;
    j.b = dY;
    j.lda = 2 * ldx;
    j.ldb = 2 * lddy;
    j.inner = k;
    j.outer = m;
    j.rows = (int32_t)rows;
    j.experts = (int32_t)experts;
    j.ends = ends;
    j.mask = mask;
    j.out = C;
    j.ldo = ldc;
    j.ostride = stride;
    j.ovec = four(C, ctype, ldc) && (experts == 1 || stride % 4 == 0);
    j.ovec8 = eight(C, ldc) && (experts == 1 || stride % 8 == 0);
    return status(launch_grouped_wgrad(j, ctype == TSENOR_BF16, stream), "grouped_wgrad kernel launch");
}

int tsenor_quant_int8(const void* X, int dtype, int64_t batch, int64_t stride, int64_t rows, int64_t cols,
                      int64_t ldx, int8_t* values, float* scales, void* stream) {
    if (batch < 0 || rows < 0 || cols <= 0) return TSENOR_ERR_SHAPE;
    const bool none = batch == 0 || rows == 0;
    if (!none && (X == nullptr || values == nullptr || scales == nullptr)) return TSENOR_ERR_NULL;
    if (!float_type(dtype)) return TSENOR_ERR_DTYPE;
    if (cols > kMaxReduce || ldx < cols || too_big(rows, ldx) || (batch > 1 && stride < rows * ldx) ||
        too_big(batch, stride) || too_big(batch, rows) || too_big(batch * rows, cols + 127))
        return TSENOR_ERR_SHAPE;
    if (misaligned(X, element_size(dtype)) || misaligned(values, 16) || misaligned(scales, 4)) return TSENOR_ERR_SHAPE;
    if (none) return TSENOR_OK;
    return status(launch_quant_int8(X, dtype == TSENOR_BF16, batch, stride, rows, cols, ldx, values, scales, stream),
                  "quant_int8 kernel launch");
}

int tsenor_gemm_int8(const void* X, int xtype, const float* xscales, int64_t rows, int64_t ldx, const int8_t* A,
                     const float* ascales, int64_t experts, int64_t m, int64_t k, const int* ends, void* Y, int ytype,
                     int64_t ldy, void* stream) {
    const bool ready = xtype == TSENOR_INT8;
    if (A == nullptr || ascales == nullptr ||
        (rows != 0 && (X == nullptr || Y == nullptr || (ready && xscales == nullptr))))
        return TSENOR_ERR_NULL;
    if ((!ready && xtype != TSENOR_BF16) || !float_type(ytype)) return TSENOR_ERR_DTYPE;
    if (experts < 1 || experts > kMaxExperts || (ends == nullptr && experts != 1)) return TSENOR_ERR_PARAM;
    if (rows < 0 || rows >= kMaxRows || m <= 0 || m >= kMaxRows || k <= 0 || k > kMaxReduce || ldy < m)
        return TSENOR_ERR_SHAPE;
    const int64_t kpad = (k + 127) / 128 * 128;
    if (ready ? ldx != kpad : ldx < k || rows > 16 || rows * kpad > kMaxTokenEntries || ends != nullptr)
        return TSENOR_ERR_SHAPE;
    if (too_big(rows, ldx) || too_big(rows, ldy) || too_big(m, kpad) || too_big(experts, m * kpad))
        return TSENOR_ERR_SHAPE;
    if (misaligned(X, ready ? 16 : 2) || misaligned(xscales, 4) || misaligned(A, 16) || misaligned(ascales, 4) ||
        misaligned(ends, 4) || misaligned(Y, element_size(ytype)))
        return TSENOR_ERR_SHAPE;
    if (rows == 0) return TSENOR_OK;
    GroupedJob j = {};
    j.a = A;
    j.b = X;
    j.lda = kpad;
    j.ldb = ready ? kpad : 2 * ldx;
    j.astride = m * kpad;
    j.inner = m;
    j.kbytes = kpad;
    j.rows = (int32_t)rows;
    j.experts = (int32_t)experts;
    j.ends = ends;
    j.as = ascales;
    j.bs = xscales;
    j.out = Y;
    j.ldo = ldy;
    j.bcols = k;
    j.bvec = !misaligned(X, 16) && ldx % 8 == 0;
    j.ovec = four(Y, ytype, ldy);
    j.ovec8 = eight(Y, ldy);
    return status(launch_gemm_int8(j, !ready, ytype == TSENOR_BF16, stream), "gemm_int8 kernel launch");
}

size_t tsenor_grads_workspace(int count) {
    const int64_t launches = count <= 0 ? 1 : ((int64_t)count + kGradsPerLaunch - 1) / kGradsPerLaunch;
    return (size_t)(launches * kGradBlocks) * sizeof(double);  // a partial sum for each workgroup
}

int tsenor_grad_norm(const tsenor_grad* grads, int count, void* workspace, size_t workspace_bytes, float* norm,
                     void* stream) {
    const int code = grads_check(grads, count, false, workspace, workspace_bytes, norm);
    if (code != TSENOR_OK) return code;
    double* sums = static_cast<double*>(workspace);
    int n = 0;
    int e = each_launch(grads, count, false, &n, [&](const GradList& list, int blocks, int before) {
        return launch_grad_squares(list, blocks, sums + before, stream);
    });
    if (e == hipSuccess) e = launch_grad_finish(sums, n, norm, stream);
    return status(e, "grad_norm kernel launch");
}

int tsenor_clip_grads(const tsenor_grad* grads, int count, float max_norm, void* workspace, size_t workspace_bytes,
                      float* norm, void* stream) {
    if (!(max_norm >= 0.f)) return TSENOR_ERR_PARAM;
    const int code = grads_check(grads, count, true, workspace, workspace_bytes, norm);
    if (code != TSENOR_OK) return code;
    double* sums = static_cast<double*>(workspace);
    int n = 0, launches = 0;
    int e = each_launch(grads, count, true, &n, [&](const GradList& list, int blocks, int before) {
        ++launches;
        return launch_grad_squares(list, blocks, sums + before, stream);
    });
    if (e != hipSuccess || launches == 0) {
        if (e == hipSuccess) e = launch_grad_finish(sums, 0, norm, stream);
        return status(e, "clip_grads kernel launch");
    }
    int again = 0;
    e = each_launch(grads, count, true, &again, [&](const GradList& list, int blocks, int before) {
        return launch_grad_scale(list, blocks, sums, n, max_norm, before == 0 ? norm : nullptr, stream);
    });
    return status(e, "clip_grads kernel launch");
}

}  // extern "C"
