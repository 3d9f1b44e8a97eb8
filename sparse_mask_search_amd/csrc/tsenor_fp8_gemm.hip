// tsenor_fp8_gemm.hip -- products of block-scaled 8-bit operands
// (include/tsenor_fp8.h): Y = X A^T with a 2:4 operand A on the sparse matrix
// cores (v_smfmac_f32_16x16x128_fp8_fp8), and C = A B^T of two dense operands
// on the scaled matrix cores (v_mfma_scale_f32_16x16x128_f8f6f4).
//
// Operand layout of smfmac 16x16x128 (measured on gfx950 with an in-bounds
// probe), for lane l, q = l / 16: A row l % 16; with the operand's 16 values
// and its metadata word taken as entries 32q .. 32q+31 of the block of 128, B
// (column l % 16) holds entries 16q .. 16q+15 and 64+16q .. 64+16q+15.  D: column
// l % 16, rows 4q .. 4q+3.  One instruction spans one block of 128, so its
// result is scaled and added in fp32; A is put on the rows (m), so that a lane
// holds four neighbouring entries of a row of Y.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor_fp8_device.h"
#include "tsenor_internal.h"

namespace tsenor {
namespace {

using namespace fp8;

// Four neighbouring entries of an output row, columns c .. c+3 (< cols written).
__device__ __forceinline__ void store4(float* y, int64_t c, int64_t cols, bool vec, f32x4 v) {
    if (vec && c + 4 <= cols) {
        *reinterpret_cast<f32x4*>(y + c) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < cols) y[c + i] = v[i];
    }
}
__device__ __forceinline__ void store4(uint16_t* y, int64_t c, int64_t cols, bool vec, f32x4 v) {
    if (vec && c + 4 <= cols) {
        *reinterpret_cast<u32x2*>(y + c) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < cols) y[c + i] = to_bf16(v[i]);
    }
}

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
    return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Eight bf16 entries as e4m3 after scaling.
__device__ __forceinline__ u32x2 quant8(const uint16_t v[8], float inv) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = scaled(widen(v[i]), inv);
    return u32x2{pack4(y[0], y[1], y[2], y[3]), pack4(y[4], y[5], y[6], y[7])};
}

// This lane's part of one block of a bf16 row (entries 16q .. and 64+16q .. of
// the 128 at k0), quantised; the four lanes that hold the block share its scale.
__device__ __forceinline__ i32x8 quant_fragment(const uint16_t* row, int64_t k0, int64_t k, bool vec,
                                                int q, int* s) {
    uint16_t v[4][8];
    uint32_t m = 0u;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        load8(row, k0 + 16 * q + 64 * (p >> 1) + 8 * (p & 1), k, vec, v[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, finite_magnitude(widen(v[p][i])));
    }
    m = max(m, (uint32_t)__shfl_xor(m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor(m, 32, 64));
    *s = scale_exponent(m);
    const float inv = inverse_scale(*s);
    const u32x2 a = quant8(v[0], inv), b = quant8(v[1], inv), c = quant8(v[2], inv), d = quant8(v[3], inv);
    return i32x8{(int)a.x, (int)a.y, (int)b.x, (int)b.y, (int)c.x, (int)c.y, (int)d.x, (int)d.y};
}

// Any shape: a wave owns 16 rows of A and 16 NT rows of X, operands straight
// from memory.  QX: X is bf16 and quantised on the way.
template <int NT, bool QX, class TY>
__global__ __launch_bounds__(256) void spmm24_fp8_kernel(const void* __restrict__ X,
                                                         const uint8_t* __restrict__ xs, int64_t n,
                                                         int64_t ldx, bool xvec,
                                                         const uint8_t* __restrict__ values,
                                                         const uint32_t* __restrict__ meta,
                                                         const uint8_t* __restrict__ scales, int64_t m,
                                                         int64_t k, TY* __restrict__ Y, int64_t ldy,
                                                         bool yvec) {
    const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
    const int64_t mt = (m + 63) / 64;
    const int64_t m0 = (blockIdx.x % mt) * 64 + 16 * (threadIdx.x >> 6);
    const int64_t n0 = (blockIdx.x / mt) * (16 * NT);
    if (m0 >= m) return;
    const int64_t kb = (k + 127) / 128;
    const int64_t row = min(m0 + l16, m - 1);
    const uint8_t* arow = values + row * (kb * 64) + 16 * q;
    const uint32_t* mrow = meta + row * (kb * 4) + q;
    const uint8_t* srow = scales + (m0 >> 7) * kb;
    int64_t col[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) col[j] = min(n0 + 16 * j + l16, n - 1);
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t t = 0; t < kb; ++t) {
        const i32x4 a = *reinterpret_cast<const i32x4*>(arow + 64 * t);
        const int idx = (int)mrow[4 * t];
        const int sa = srow[t];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            i32x8 b;
            int sx;
            if constexpr (QX) {
                b = quant_fragment(static_cast<const uint16_t*>(X) + col[j] * ldx, 128 * t, k, xvec, q, &sx);
                sx += 127;
            } else {
                const uint8_t* x = static_cast<const uint8_t*>(X) + col[j] * ldx + 128 * t + 16 * q;
                b = join(*reinterpret_cast<const u32x4*>(x), *reinterpret_cast<const u32x4*>(x + 64));
                sx = xs[t * n + col[j]];
            }
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
            d = __builtin_amdgcn_smfmac_f32_16x16x128_fp8_fp8(a, b, d, idx, 0, 0);
            const float f = scale_product(sa, sx);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_fmaf(d[i], f, acc[j][i]);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
        if (n0 + 16 * j + l16 < n) store4(Y + col[j] * ldy, m0 + 4 * q, m, yvec, acc[j]);
}

// C = A B^T, any shape: a wave owns 16 columns of C (rows of B) and 64 rows.
template <class TC>
__global__ __launch_bounds__(256) void gemm_fp8_kernel(const uint8_t* __restrict__ A,
                                                       const uint8_t* __restrict__ as, int64_t p,
                                                       const uint8_t* __restrict__ B,
                                                       const uint8_t* __restrict__ bs, int64_t qn,
                                                       int64_t kb, const uint32_t* __restrict__ mask,
                                                       TC* __restrict__ C, int64_t ldc, bool cvec) {
    constexpr int NT = 4;
    const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
    const int64_t mt = (qn + 63) / 64;
    const int64_t m0 = (blockIdx.x % mt) * 64 + 16 * (threadIdx.x >> 6);
    const int64_t n0 = (blockIdx.x / mt) * (16 * NT);
    if (m0 >= qn) return;
    const int64_t row = min(m0 + l16, qn - 1);
    int64_t col[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) col[j] = min(n0 + 16 * j + l16, p - 1);
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t t = 0; t < kb; ++t) {
        const uint8_t* b = B + row * (kb * 128) + 128 * t + 16 * q;
        const i32x8 bv = join(*reinterpret_cast<const u32x4*>(b), *reinterpret_cast<const u32x4*>(b + 64));
        const int sb = bs[t * qn + row];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint8_t* a = A + col[j] * (kb * 128) + 128 * t + 16 * q;
            const i32x8 av = join(*reinterpret_cast<const u32x4*>(a), *reinterpret_cast<const u32x4*>(a + 64));
            acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc[j], 0, 0, 0, sb, 0,
                                                                      as[t * p + col[j]]);
        }
    }
    const int64_t wpr = (qn + 31) / 32, c0 = m0 + 4 * q;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (n0 + 16 * j + l16 >= p || c0 >= qn) continue;
        if (mask != nullptr) {
            const uint32_t bits = mask[col[j] * wpr + (c0 >> 5)] >> (c0 & 31);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!((bits >> i) & 1u)) acc[j][i] = 0.f;
        }
        store4(C + col[j] * ldc, c0, qn, cvec, acc[j]);
    }
}

template <class TY>
bool row4(const void* y, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(y) % (4 * sizeof(TY))) == 0 && ld % 4 == 0;
}

template <class TY>
int spmm(const void* X, int bf16x, const uint8_t* xs, int64_t n, int64_t ldx, const uint8_t* values,
         const uint32_t* meta, const uint8_t* scales, int64_t m, int64_t k, void* Yv, int64_t ldy,
         hipStream_t stream) {
    TY* Y = static_cast<TY*>(Yv);
    const bool yvec = row4<TY>(Yv, ldy);
    const int64_t mt = (m + 63) / 64;
    if (bf16x) {
        const bool xvec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && ldx % 8 == 0;
        hipLaunchKernelGGL((spmm24_fp8_kernel<1, true, TY>), dim3((unsigned)mt), dim3(256), 0, stream, X,
                           nullptr, n, ldx, xvec, values, meta, scales, m, k, Y, ldy, yvec);
    } else {
        hipLaunchKernelGGL((spmm24_fp8_kernel<4, false, TY>), dim3((unsigned)(mt * ((n + 63) / 64))),
                           dim3(256), 0, stream, X, xs, n, ldx, true, values, meta, scales, m, k, Y, ldy,
                           yvec);
    }
    return (int)hipGetLastError();
}

template <class TC>
int gemm(const uint8_t* A, const uint8_t* as, int64_t p, const uint8_t* B, const uint8_t* bs,
         int64_t q, int64_t k, const uint32_t* mask, void* C, int64_t ldc, hipStream_t stream) {
    const int64_t blocks = ((q + 63) / 64) * ((p + 63) / 64);
    hipLaunchKernelGGL((gemm_fp8_kernel<TC>), dim3((unsigned)blocks), dim3(256), 0, stream, A, as, p, B,
                       bs, q, (k + 127) / 128, mask, static_cast<TC*>(C), ldc, row4<TC>(C, ldc));
    return (int)hipGetLastError();
}

}  // namespace

int launch_spmm24_fp8(const void* X, int bf16x, const uint8_t* xs, int64_t n, int64_t ldx,
                      const uint8_t* values, const uint32_t* meta, const uint8_t* scales, int64_t m,
                      int64_t k, void* Y, int bf16y, int64_t ldy, void* stream) {
    return bf16y ? spmm<uint16_t>(X, bf16x, xs, n, ldx, values, meta, scales, m, k, Y, ldy,
                                  (hipStream_t)stream)
                 : spmm<float>(X, bf16x, xs, n, ldx, values, meta, scales, m, k, Y, ldy,
                               (hipStream_t)stream);
}

int launch_gemm_fp8(const uint8_t* A, const uint8_t* as, int64_t p, const uint8_t* B,
                    const uint8_t* bs, int64_t q, int64_t k, const uint32_t* mask, void* C,
                    int bf16c, int64_t ldc, void* stream) {
    return bf16c ? gemm<uint16_t>(A, as, p, B, bs, q, k, mask, C, ldc, (hipStream_t)stream)
                 : gemm<float>(A, as, p, B, bs, q, k, mask, C, ldc, (hipStream_t)stream);
}

}  // namespace tsenor
