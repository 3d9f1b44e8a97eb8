// tsenor_int8.hip -- rows to 8-bit integers with a scale each
// (include/tsenor_ops.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor_internal.h"
#include "tsenor_ops_device.h"

namespace tsenor {
namespace {

using namespace ops;

// G threads hold a row of up to 8 V G entries in registers (V vectors of 8 each), so that it is read once; a
// wave's shuffles, or four waves' LDS words, give its largest magnitude.  Memory bounds it: bf16 11008 x 4096 in
// 26 to 29 us (4.7 to 5.2 TB/s).
template <class T, int G, int V>
__global__ __launch_bounds__(256) void quant_int8_kernel(const T* __restrict__ X, int64_t stride, int64_t rows,
                                                         int64_t all, int64_t cols, int64_t ldx, bool vec,
                                                         int8_t* __restrict__ values, float* __restrict__ scales) {
    constexpr bool kWide = sizeof(T) == 4;
    __shared__ uint32_t part[256 / 64];
    const int tid = threadIdx.x, l = tid % G;
    const int64_t row = (int64_t)blockIdx.x * (256 / G) + tid / G;
    if (G == 64 && row >= all) return;
    const int64_t kpad = (cols + 127) / 128 * 128;
    const T* x = X + row / rows * stride + row % rows * ldx;
    Eight<T> v[V];
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i].load(x, 8 * (int64_t)(l + G * i), cols, vec);
        most = max(most, v[i].magnitude());
    }
    // rows longer than the registers: read a second time below
    for (int64_t c = 8 * (int64_t)(l + G * V); c < cols; c += 8 * G) {
        Eight<T> w;
        w.load(x, c, cols, vec);
        most = max(most, w.magnitude());
    }
    most = max64(most);
    if constexpr (G > 64) {
        if ((tid & 63) == 0) part[tid >> 6] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 256 / 64; ++i) most = max(most, part[i]);
    }
    const TokenScale s = token_scale(most);
    const double factor = s.factor == 0.f ? 0.0 : 127.0 / (double)bits_float(most);
    const auto quantised = [&](const Eight<T>& w) {
        if constexpr (kWide) return integers(w, factor);
        else return integers(w, s.factor, s.exponent);
    };
    int8_t* to = values + row * kpad;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t c = 8 * (int64_t)(l + G * i);
        if (c < kpad) *reinterpret_cast<u32x2*>(to + c) = quantised(v[i]);
    }
    for (int64_t c = 8 * (int64_t)(l + G * V); c < kpad; c += 8 * G) {
        Eight<T> w;
        w.load(x, c, cols, vec);
        *reinterpret_cast<u32x2*>(to + c) = quantised(w);
    }
    if (l == 0) scales[row] = s.scale;
}

template <class T>
int quant(const void* X, int64_t batch, int64_t stride, int64_t rows, int64_t cols, int64_t ldx, int8_t* values,
          float* scales, hipStream_t stream) {
    const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && (ldx * sizeof(T)) % 16 == 0 &&
                     (batch == 1 || (stride * sizeof(T)) % 16 == 0);
    const int64_t all = batch * rows;
    const auto go = [&](auto kernel, int lanes) {
        const int64_t blocks = (all + 256 / lanes - 1) / (256 / lanes);
        if (!grid_fits(blocks, 256)) return (int)kGridTooLarge;
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, stream, static_cast<const T*>(X), stride,
                           rows, all, cols, ldx, vec, values, scales);
        return (int)hipGetLastError();
    };
    if (cols <= 2048) return go(quant_int8_kernel<T, 64, 4>, 64);
    if (cols <= 4096) return go(quant_int8_kernel<T, 256, 2>, 256);
    return go(quant_int8_kernel<T, 256, 8>, 256);
}

}  // namespace

int launch_quant_int8(const void* X, int bf16, int64_t batch, int64_t stride, int64_t rows, int64_t cols,
                      int64_t ldx, int8_t* values, float* scales, void* stream) {
    return bf16 ? quant<uint16_t>(X, batch, stride, rows, cols, ldx, values, scales, (hipStream_t)stream)
                : quant<float>(X, batch, stride, rows, cols, ldx, values, scales, (hipStream_t)stream);
}

}  // namespace tsenor
