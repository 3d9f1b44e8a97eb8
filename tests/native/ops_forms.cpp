// The C entry points of include/tsenor_ops.h over launches that run nothing and note which form the
// library's own rule (tsenor_grouped_forms.h) gives the product: for tests without a GPU.
#include "tsenor.h"
#include "tsenor_grouped_forms.h"
#include "tsenor_internal.h"

namespace {
const char* const kNames[] = {"few64", "few32", "few16", "few32x32", "any", "staged256x128", "256x256", "256x128",
                              "128x128", "64x64"};
const char* form = "";
}  // namespace

namespace tsenor {
int launch_grouped_mm(const GroupedJob& job, bool transposed, bool, void*) {
    form = kNames[transposed ? pick_form<kProduct, true, false>(job, 2) : pick_form<kProduct, false, false>(job, 2)];
    return 0;
}
int launch_grouped_wgrad(const GroupedJob& job, bool, void*) {
    form = kNames[pick_form<kGradient, true, true>(job, 2)];
    return 0;
}
int launch_gemm_int8(const GroupedJob& job, bool bf16x, bool, void*) {
    form = bf16x ? "tokens" : kNames[pick_form<kProduct, false, false>(job, 1)];
    return 0;
}
int launch_quant_int8(const void*, int, int64_t, int64_t, int64_t, int64_t, int64_t, int8_t*, float*, void*) { return 0; }
int launch_grad_squares(const GradList&, int, double*, void*) { return 0; }
int launch_grad_finish(const double*, int, float*, void*) { return 0; }
int launch_grad_scale(const GradList&, int, const double*, int, float, float*, void*) { return 0; }
int grad_chunk() { return 32768; }
int hip_error(int, const char*) { return TSENOR_ERR_HIP; }
}  // namespace tsenor

extern "C" const char* last_form() { return form; }
extern "C" int64_t lds_of_tile(int gradient, int columns, int rows, int ring) {
    return tsenor::tile_lds(gradient ? tsenor::kGradient : tsenor::kProduct, columns, rows, ring);
}
extern "C" int64_t workgroups_of_cu(int gradient, int columns, int rows, int ring) {
    return tsenor::at_once(gradient ? tsenor::kGradient : tsenor::kProduct, columns, rows, ring);
}
