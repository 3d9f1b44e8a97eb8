// tsenor_fp8_operands.hip -- building the 8-bit operands: activations and
// gradients quantised along rows and columns, weights compressed to 2:4 under
// their mask along both.  Formats: include/tsenor_fp8.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor_fp8_device.h"
#include "tsenor_internal.h"

namespace tsenor {
namespace {

using namespace fp8;

// Along the rows only: 16 lanes hold one block of 128 (8 entries each).
template <class T>
__global__ __launch_bounds__(256) void quant_rows_kernel(const T* __restrict__ X, int64_t rows,
                                                         int64_t cols, int64_t ldx, bool vec,
                                                         uint8_t* __restrict__ values,
                                                         uint8_t* __restrict__ scales) {
    const int64_t blocks = (cols + 127) / 128;
    const int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);  // (row, block)
    if (g >= rows * blocks) return;
    const int64_t r = g / blocks, b = g - r * blocks;
    const int l = threadIdx.x & 15;
    T raw[8];
    load8(X + r * ldx, b * 128 + 8 * l, cols, vec, raw);
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_magnitude(widen(raw[i])));
    const int s = scale_exponent(max16(m));
    const float inv = inverse_scale(s);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = scaled(widen(raw[i]), inv);
    const u32x2 q = {pack4(y[0], y[1], y[2], y[3]), pack4(y[4], y[5], y[6], y[7])};
    *reinterpret_cast<u32x2*>(values + r * (blocks * 128) + b * 128 + 8 * l) = q;
    if (l == 0) scales[b * rows + r] = (uint8_t)(s + 127);
}

// Along the columns, and along the rows too when `values` is given: one
// workgroup per 128 x 128 tile, read once and kept in LDS.
template <class T>
__global__ __launch_bounds__(256) void quant_tile_kernel(const T* __restrict__ X, int64_t rows,
                                                         int64_t cols, int64_t ldx, bool vec,
                                                         uint8_t* __restrict__ values,
                                                         uint8_t* __restrict__ scales,
                                                         uint8_t* __restrict__ values_t,
                                                         uint8_t* __restrict__ scales_t) {
    constexpr int kLd = 128 + 16 / sizeof(T);
    __shared__ T tile[128 * kLd];
    __shared__ uint32_t colmax[2][128];
    const int64_t cblocks = (cols + 127) / 128, rblocks = (rows + 127) / 128;
    const int64_t rb = blockIdx.x / cblocks, cb = blockIdx.x - rb * cblocks;
    const int tid = threadIdx.x, l = tid & 15;
    for (int p = 0; p < 8; ++p) {
        const int lr = 16 * p + (tid >> 4);
        const int64_t r = rb * 128 + lr;
        T raw[8];
        if (r < rows) {
            load8(X + r * ldx, cb * 128 + 8 * l, cols, vec, raw);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) raw[i] = (T)0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) tile[lr * kLd + 8 * l + i] = raw[i];
        if (values != nullptr) {  // uniform
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, finite_magnitude(widen(raw[i])));
            const int s = scale_exponent(max16(m));
            const float inv = inverse_scale(s);
            if (r < rows) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = scaled(widen(raw[i]), inv);
                const u32x2 q = {pack4(y[0], y[1], y[2], y[3]), pack4(y[4], y[5], y[6], y[7])};
                *reinterpret_cast<u32x2*>(values + r * (cblocks * 128) + cb * 128 + 8 * l) = q;
                if (l == 0) scales[cb * rows + r] = (uint8_t)(s + 127);
            }
        }
    }
    __syncthreads();
    // a thread holds half a column (64 rows)
    const int c = tid & 127, half = tid >> 7;
    uint32_t m = 0u;
    for (int i = 0; i < 64; ++i) m = max(m, finite_magnitude(widen(tile[(64 * half + i) * kLd + c])));
    colmax[half][c] = m;
    __syncthreads();
    const int64_t col = cb * 128 + c;
    if (col >= cols) return;
    const int s = scale_exponent(max(colmax[0][c], colmax[1][c]));
    const float inv = inverse_scale(s);
    uint8_t* out = values_t + col * (rblocks * 128) + rb * 128 + 64 * half;
    for (int v = 0; v < 4; ++v) {
        u32x4 q;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = scaled(widen(tile[(64 * half + 16 * v + 4 * w + i) * kLd + c]), inv);
            q[w] = pack4(y[0], y[1], y[2], y[3]);
        }
        *reinterpret_cast<u32x4*>(out + 16 * v) = q;
    }
    if (half == 0) scales_t[rb * cols + col] = (uint8_t)(s + 127);
}

// First two set bits of a group's four mask bits, as the four bits of its
// metadata (unused slots point at a free position), and its two values.
__device__ __forceinline__ uint32_t take24(uint32_t bits, uint32_t q, uint32_t* v0, uint32_t* v1,
                                           int* over) {
    const uint32_t rest = bits & (bits - 1u);
    uint32_t p0 = bits ? (uint32_t)__builtin_ctz(bits) : 0u;
    uint32_t p1 = rest ? (uint32_t)__builtin_ctz(rest) : (bits ? (p0 == 3u ? 2u : 3u) : 1u);
    *v0 = bits ? (q >> (8 * p0)) & 0xFFu : 0u;
    *v1 = rest ? (q >> (8 * p1)) & 0xFFu : 0u;
    *over += (rest & (rest - 1u)) != 0u;
    return p0 | (p1 << 2);
}

// One workgroup per 128 x 128 tile of one matrix.  The tile's kept entries
// give the one scale that both orientations share; the 8-bit numbers go to LDS
// once, and are compressed from there along the rows and along the columns.
template <class T>
__global__ __launch_bounds__(256) void compress24_fp8_kernel(
    const T* __restrict__ W, int64_t stride, int64_t rows, int64_t cols, int64_t ld, bool vec,
    const uint32_t* __restrict__ mask, uint8_t* __restrict__ values, uint32_t* __restrict__ meta,
    uint8_t* __restrict__ scales, uint8_t* __restrict__ values_t, uint32_t* __restrict__ meta_t,
    uint8_t* __restrict__ scales_t, int* __restrict__ bad, int* __restrict__ bad_t) {
    constexpr int kLd = 144;  // bytes of a tile row
    __shared__ __attribute__((aligned(16))) uint8_t q8[128 * kLd];
    __shared__ uint32_t bits[128][5];  // mask words of the tile's rows (padded against bank conflicts)
    __shared__ uint32_t wmax[4];
    const int64_t cblocks = (cols + 127) / 128, rblocks = (rows + 127) / 128;
    const int64_t per = rblocks * cblocks;
    const int64_t mat = blockIdx.x / per, t = blockIdx.x - mat * per;
    const int64_t rb = t / cblocks, cb = t - rb * cblocks;
    const int64_t wpr = (cols + 31) / 32;
    const int tid = threadIdx.x, l = tid & 15;
    W += mat * stride;
    mask += mat * rows * wpr;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int lr = (tid + 256 * i) >> 2, w = tid & 3;
        const int64_t r = rb * 128 + lr, word = cb * 4 + w;
        uint32_t m = 0u;
        if (r < rows && word < wpr) {
            m = mask[r * wpr + word];
            const int64_t left = cols - word * 32;  // bits behind the last column are ignored
            if (left < 32) m &= (1u << left) - 1u;
        }
        bits[lr][w] = m;
    }
    __syncthreads();
    T raw[8][8];
    uint32_t m = 0u;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int lr = 16 * p + (tid >> 4);
        const int64_t r = rb * 128 + lr;
        if (r < rows) {
            load8(W + r * ld, cb * 128 + 8 * l, cols, vec, raw[p]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) raw[p][i] = (T)0;
        }
        const uint32_t keep = bits[lr][l >> 2] >> (8 * (l & 3));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!((keep >> i) & 1u)) raw[p][i] = (T)0;
            m = max(m, finite_magnitude(widen(raw[p][i])));
        }
    }
    m = max16(m);
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor(m, d, 64));
    if ((tid & 63) == 0) wmax[tid >> 6] = m;
    __syncthreads();
    const int s = scale_exponent(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
    const float inv = inverse_scale(s);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int lr = 16 * p + (tid >> 4);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = scaled(widen(raw[p][i]), inv);
        const u32x2 q = {pack4(y[0], y[1], y[2], y[3]), pack4(y[4], y[5], y[6], y[7])};
        *reinterpret_cast<u32x2*>(&q8[lr * kLd + 8 * l]) = q;
    }
    if (tid == 0) {
        if (scales != nullptr) scales[mat * per + rb * cblocks + cb] = (uint8_t)(s + 127);
        if (scales_t != nullptr) scales_t[mat * per + cb * rblocks + rb] = (uint8_t)(s + 127);
    }
    __syncthreads();
    const int a = tid & 127, half = tid >> 7;  // a row (or column) and 64 entries along it
    if (values != nullptr && rb * 128 + a < rows) {
        const int64_t r = mat * rows + rb * 128 + a;
        int over = 0;
        uint32_t out[8], mw[2] = {0u, 0u};
#pragma unroll
        for (int g = 0; g < 16; g += 2) {
            const int c = 64 * half + 4 * g;
            const uint32_t word = bits[a][c >> 5];
            uint32_t v[4];
            const uint32_t n0 = take24((word >> (c & 31)) & 15u,
                                       *reinterpret_cast<const uint32_t*>(&q8[a * kLd + c]), v, v + 1, &over);
            const uint32_t n1 = take24((word >> ((c & 31) + 4)) & 15u,
                                       *reinterpret_cast<const uint32_t*>(&q8[a * kLd + c + 4]), v + 2,
                                       v + 3, &over);
            out[g / 2] = v[0] | (v[1] << 8) | (v[2] << 16) | (v[3] << 24);
            mw[g >> 3] |= (n0 << (4 * (g & 7))) | (n1 << (4 * ((g + 1) & 7)));
        }
        u32x4* ov = reinterpret_cast<u32x4*>(values + r * (cblocks * 64) + cb * 64 + 32 * half);
        ov[0] = u32x4{out[0], out[1], out[2], out[3]};
        ov[1] = u32x4{out[4], out[5], out[6], out[7]};
        *reinterpret_cast<u32x2*>(meta + r * (cblocks * 4) + cb * 4 + 2 * half) = u32x2{mw[0], mw[1]};
        if (over && bad != nullptr) atomicAdd(bad, over);
    }
    if (values_t != nullptr && cb * 128 + a < cols) {
        const int64_t c = mat * cols + cb * 128 + a;
        int over = 0;
        uint32_t out[8], mw[2] = {0u, 0u};
#pragma unroll
        for (int g = 0; g < 16; g += 2) {
            uint32_t b[2] = {0u, 0u}, q[2] = {0u, 0u}, v[4], n[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 64 * half + 4 * g + i;
                b[i >> 2] |= ((bits[r][a >> 5] >> (a & 31)) & 1u) << (i & 3);
                q[i >> 2] |= (uint32_t)q8[r * kLd + a] << (8 * (i & 3));
            }
            n[0] = take24(b[0], q[0], v, v + 1, &over);
            n[1] = take24(b[1], q[1], v + 2, v + 3, &over);
            out[g / 2] = v[0] | (v[1] << 8) | (v[2] << 16) | (v[3] << 24);
            mw[g >> 3] |= (n[0] << (4 * (g & 7))) | (n[1] << (4 * ((g + 1) & 7)));
        }
        u32x4* ov = reinterpret_cast<u32x4*>(values_t + c * (rblocks * 64) + rb * 64 + 32 * half);
        ov[0] = u32x4{out[0], out[1], out[2], out[3]};
        ov[1] = u32x4{out[4], out[5], out[6], out[7]};
        *reinterpret_cast<u32x2*>(meta_t + c * (rblocks * 4) + rb * 4 + 2 * half) = u32x2{mw[0], mw[1]};
        if (over && bad_t != nullptr) atomicAdd(bad_t, over);
    }
}

template <class T>
bool rows16(const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
}

template <class T>
int quant(const void* Xv, int64_t rows, int64_t cols, int64_t ldx, uint8_t* values, uint8_t* scales,
          uint8_t* values_t, uint8_t* scales_t, hipStream_t stream) {
    const T* X = static_cast<const T*>(Xv);
    const bool vec = rows16<T>(X, ldx);
    const int64_t cb = (cols + 127) / 128, rb = (rows + 127) / 128;
    if (values_t == nullptr)
        hipLaunchKernelGGL((quant_rows_kernel<T>), dim3((unsigned)((rows * cb + 15) / 16)), dim3(256),
                           0, stream, X, rows, cols, ldx, vec, values, scales);
    else
        hipLaunchKernelGGL((quant_tile_kernel<T>), dim3((unsigned)(rb * cb)), dim3(256), 0, stream, X,
                           rows, cols, ldx, vec, values, scales, values_t, scales_t);
    return (int)hipGetLastError();
}

}  // namespace

int launch_quant_fp8(const void* X, int bf16, int64_t rows, int64_t cols, int64_t ldx,
                     uint8_t* values, uint8_t* scales, uint8_t* values_t, uint8_t* scales_t,
                     void* stream) {
    return bf16 ? quant<uint16_t>(X, rows, cols, ldx, values, scales, values_t, scales_t,
                                  (hipStream_t)stream)
                : quant<float>(X, rows, cols, ldx, values, scales, values_t, scales_t,
                               (hipStream_t)stream);
}

int launch_compress24_fp8(const void* W, int bf16, int64_t batch, int64_t stride, int64_t rows,
                          int64_t cols, int64_t ld, const uint32_t* mask, uint8_t* values,
                          uint32_t* meta, uint8_t* scales, uint8_t* values_t, uint32_t* meta_t,
                          uint8_t* scales_t, int* bad, int* bad_t, void* stream) {
    const int64_t es = bf16 ? 2 : 4;
    const bool vec = (reinterpret_cast<uintptr_t>(W) & 15u) == 0 && (ld * es) % 16 == 0 &&
                     (batch == 1 || (stride * es) % 16 == 0);
    const int64_t blocks = batch * ((rows + 127) / 128) * ((cols + 127) / 128);
    if (bf16)
        hipLaunchKernelGGL((compress24_fp8_kernel<uint16_t>), dim3((unsigned)blocks), dim3(256), 0,
                           (hipStream_t)stream, static_cast<const uint16_t*>(W), stride, rows, cols, ld,
                           vec, mask, values, meta, scales, values_t, meta_t, scales_t, bad, bad_t);
    else
        hipLaunchKernelGGL((compress24_fp8_kernel<float>), dim3((unsigned)blocks), dim3(256), 0,
                           (hipStream_t)stream, static_cast<const float*>(W), stride, rows, cols, ld,
                           vec, mask, values, meta, scales, values_t, meta_t, scales_t, bad, bad_t);
    return (int)hipGetLastError();
}

}  // namespace tsenor
