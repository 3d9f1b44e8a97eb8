// tsenor_ops_internal.h -- shared between the ABI layer and the kernels of
// include/tsenor_ops.h.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace tsenor {

// A product grouped by expert, as its kernels see it.  "Inner" is the output's contiguous
// dimension (features of a product, input features of a weight gradient).
struct GroupedJob {
    const void* a;      // weights, expert e at + e * astride; weight gradient: X
    const void* b;      // tokens; weight gradient: dY
    int64_t lda, ldb;   // bytes from row to row
    int64_t astride;    // bytes from expert to expert
    int64_t inner;      // columns of the output
    int64_t outer;      // weight gradient: rows of one expert's output
    int64_t kbytes;     // bytes of a row along the reduction (not for a weight gradient)
    int32_t rows, experts;
    const int* ends;    // or nullptr: one expert owns all rows
    const float *as, *bs;  // scales of 8-bit integers
    const uint32_t* mask;  // weight gradient, or nullptr
    void* out;
    int64_t ldo, ostride;  // elements
    int64_t bcols;      // entries of a token's row that is quantised on the way
    bool bvec;          // it may be read 16 bytes at a time
    bool ovec, ovec8;   // four (eight bf16) neighbouring outputs may be written at once
};

// transposed: weights [k][m].  They return a hipError_t
// value or kGridTooLarge.
int launch_grouped_mm(const GroupedJob& job, bool transposed, bool bf16out, void* stream);
int launch_grouped_wgrad(const GroupedJob& job, bool bf16out, void* stream);

int launch_quant_int8(const void* X, int bf16, int64_t batch, int64_t stride, int64_t rows, int64_t cols,
                      int64_t ldx, int8_t* values, float* scales, void* stream);
constexpr int kMaxTokenEntries = 32768;  // bf16 tokens that are quantised on the way, padded
// bf16x: job.b holds bf16 tokens (at most 16), quantised on the way
int launch_gemm_int8(const GroupedJob& job, bool bf16x, bool bf16out, void* stream);

// One gradient of a list, as the kernels see it.
enum GradLayout { kLoose, kFlat, kRows };
struct GradJob {
    const void* grad;
    void* out;
    const uint32_t* mask;
    int64_t rows, cols, ld, ldo;
    int32_t first;                // chunks of the tensors before it
    int16_t bf16, layout;
};
constexpr int kGradsPerLaunch = 48;   // as kernel arguments
constexpr int kGradBlocks = 512;      // most workgroups of a launch, one partial sum each
struct GradList {
    GradJob job[kGradsPerLaunch];
    int32_t count, chunks;
};
// Sums of squares to sums[0 .. blocks); then factor and result from all partial sums.
int launch_grad_squares(const GradList& list, int blocks, double* sums, void* stream);
int launch_grad_finish(const double* sums, int n, float* norm, void* stream);
int launch_grad_scale(const GradList& list, int blocks, const double* sums, int n, float max_norm, float* norm,
                      void* stream);
int grad_chunk();  // entries of a chunk

}  // namespace tsenor
