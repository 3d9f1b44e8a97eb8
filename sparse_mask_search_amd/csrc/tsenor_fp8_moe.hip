// tsenor_fp8_moe.hip -- a mixture-of-experts layer for a few tokens
// (include/tsenor_fp8.h: tsenor_moe24_fp8).  Three launches:
//   logits  x R^T in fp64, and x copied to rows padded with zeros;
//   hidden  per expert and 16 rows of gate and up: the tokens that chose the
//           expert (each workgroup ranks its expert among the logits), both
//           products, silu, product, bf16;
//   output  per 16 rows of down: every token's experts, weighted and summed.
// The weights' 8-bit numbers become bf16 exactly, their scale folded into the
// conversion (v_cvt_scalef32_pk_bf16_fp8), and multiply the bf16 activations on
// the sparse matrix cores (v_smfmac_f32_16x16x64_bf16).  Operand layout of that
// instruction (measured with an in-bounds probe), lane l, q = l / 16: A row
// l % 16, eight values that cover 16 entries; when these are entries
// 32q + 16j .. 32q + 16j + 15 of a block of 128 (j = 0, 1: the two instructions
// of the block), B column l % 16 holds entries 32(q/2) + 16j + 8(q%2) .. +7 and
// the eight 64 further on.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor_fp8_device.h"
#include "tsenor_internal.h"

namespace tsenor {
namespace {

using namespace fp8;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x16 __attribute__((ext_vector_type(16)));

constexpr int kMaxTokens = 64, kMaxTop = 16;

// logits[t][e] in fp64: products of bf16 numbers are exact in fp32.  A wave
// per (expert, token).  Workgroups behind those copy x.
__global__ __launch_bounds__(256) void moe_logits_kernel(MoeJob a) {
    const int lane = threadIdx.x & 63;
    const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (u < a.n * a.experts) {
        const int64_t t = u / a.experts, e = u - t * a.experts;
        const uint16_t *x = a.x + t * a.ldx, *r = a.router + e * a.ldr;
        double sum = 0.0;
        for (int64_t i = lane; i < a.d; i += 64) sum += (double)(widen(x[i]) * widen(r[i]));
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
        if (lane == 0) a.logits[t * a.experts + e] = sum;
    } else if (u < a.n * a.experts + a.n) {
        const int64_t t = u - a.n * a.experts, dp = pad128(a.d);
        for (int64_t i = lane; i < dp; i += 64)
            a.xpad[t * dp + i] = i < a.d ? a.x[t * a.ldx + i] : (uint16_t)0;
    }
}

// How many experts come before e in token t's order: larger logit first, ties
// to the lower index, NaN last.
__device__ __forceinline__ int rank_of(const double* l, int e, int experts) {
    const double le = l[e];
    const bool ne = le != le;
    int r = 0;
    for (int j = 0; j < experts; ++j) {
        const double lj = l[j];
        const bool nj = lj != lj;
        const bool before = ne ? (!nj || j < e) : (lj > le || (lj == le && j < e));
        r += before ? 1 : 0;
    }
    return r;
}

// One block of 128 of a 2:4 row as the two A operands of the block: the lane's
// 16 e4m3 values in bf16, scaled.
__device__ __forceinline__ void widen_block(u32x4 v, float scale, bf16x8 a[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * j + w], scale, false);
            const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * j + w], scale, true);
            a[j][4 * w] = lo[0];
            a[j][4 * w + 1] = lo[1];
            a[j][4 * w + 2] = hi[0];
            a[j][4 * w + 3] = hi[1];
        }
}
// The lane's B operands of the block at x (a row of activations).
__device__ __forceinline__ void load_block(const uint16_t* x, int q, bf16x16 b[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint16_t* p = x + 32 * (q >> 1) + 16 * j + 8 * (q & 1);
        const u32x4 lo = *reinterpret_cast<const u32x4*>(p);
        const u32x4 hi = *reinterpret_cast<const u32x4*>(p + 64);
        typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
        const u32x8 w = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        b[j] = __builtin_bit_cast(bf16x16, w);
    }
}
// The conversion takes the exponent field of its scale operand: the byte itself.
__device__ __forceinline__ float scale_value(int byte) { return bits_float((uint32_t)byte << 23); }

// hidden: one wave per (expert, 16 rows of gate and up); writes
// h[t * topk + rank][fpad] and ids[t * topk + rank].
__global__ __launch_bounds__(64) void moe_hidden_kernel(MoeJob a) {
    __shared__ int slots[kMaxTokens];
    const int lane = threadIdx.x, q = lane >> 4, l16 = lane & 15;
    const int64_t ft = (a.f + 15) / 16;
    const int e = (int)(blockIdx.x / ft);
    const int64_t f0 = (blockIdx.x - e * ft) * 16;
    int rank = kMaxTop;
    if (lane < a.n) rank = rank_of(a.logits + lane * a.experts, e, (int)a.experts);
    const bool mine = lane < a.n && rank < a.topk;
    const uint64_t who = __ballot(mine);
    if (who == 0) return;
    const int count = __popcll(who);
    if (mine) slots[__popcll(who & ((1ull << lane) - 1ull))] = lane * a.topk + rank;
    if (mine && f0 == 0) a.ids[lane * a.topk + rank] = e;
    __syncthreads();
    const int64_t kb = (a.d + 127) / 128, dp = kb * 128, fp = pad128(a.f);
    const int64_t row = e * a.f + min(f0 + l16, a.f - 1);
    const int64_t sb = (e * ((a.f + 127) / 128) + (f0 >> 7)) * kb;
    for (int c0 = 0; c0 < count; c0 += 16) {
        const int slot = slots[min(c0 + l16, count - 1)];
        const uint16_t* x = a.xpad + (slot / a.topk) * dp;
        f32x4 g = {0.f, 0.f, 0.f, 0.f}, u = {0.f, 0.f, 0.f, 0.f};
        for (int64_t t = 0; t < kb; ++t) {
            bf16x16 b[2];
            load_block(x + 128 * t, q, b);
            bf16x8 av[2];
            widen_block(*reinterpret_cast<const u32x4*>(a.gate.values + row * (kb * 64) + 64 * t + 16 * q),
                        scale_value(a.gate.scales[sb + t]), av);
            uint32_t idx = a.gate.meta[row * (kb * 4) + 4 * t + q];
            g = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[0], b[0], g, (int)idx, 0, 0);
            g = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[1], b[1], g, (int)(idx >> 16), 0, 0);
            widen_block(*reinterpret_cast<const u32x4*>(a.up.values + row * (kb * 64) + 64 * t + 16 * q),
                        scale_value(a.up.scales[sb + t]), av);
            idx = a.up.meta[row * (kb * 4) + 4 * t + q];
            u = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[0], b[0], u, (int)idx, 0, 0);
            u = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[1], b[1], u, (int)(idx >> 16), 0, 0);
        }
        if (c0 + l16 < count) {
            uint16_t* h = a.hidden + slot * fp;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = f0 + 4 * q + i;
                const float v = g[i] / (1.f + __expf(-g[i])) * u[i];
                h[r] = r < a.f ? to_bf16(v) : (uint16_t)0;  // rows behind f are padding
            }
            if (f0 + 16 >= a.f)  // the last tile clears the rest of the padding
                for (int64_t r = f0 + 16 + q; r < fp; r += 4) h[r] = 0;
        }
    }
}

// Softmax weight of slot (t, r) over token t's chosen logits; they are in
// descending order, so the first is the largest.
__device__ __forceinline__ float weight_of(const MoeJob& a, int64_t t, int r) {
    const double* l = a.logits + t * a.experts;
    const double top = l[a.ids[t * a.topk]];
    float sum = 0.f, mine = 0.f;
    for (int j = 0; j < a.topk; ++j) {
        const float v = expf((float)(l[a.ids[t * a.topk + j]] - top));
        sum += v;
        mine = j == r ? v : mine;
    }
    return mine / sum;
}

// output: one workgroup per 16 rows of down.  A wave takes the experts e = wave,
// wave + 4, ...; a token's partial sums per wave are joined in the wave order.
__global__ __launch_bounds__(256) void moe_output_kernel(MoeJob a) {
    __shared__ float part[4][kMaxTokens][17];
    __shared__ float wts[kMaxTokens * kMaxTop];
    __shared__ int slots[4][kMaxTokens];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
    const int64_t d0 = (int64_t)blockIdx.x * 16;
    const int64_t kb = (a.f + 127) / 128, fp = kb * 128;
    for (int i = tid; i < 4 * kMaxTokens * 17; i += 256) (&part[0][0][0])[i] = 0.f;
    for (int i = tid; i < a.n * a.topk; i += 256) {
        const float w = weight_of(a, i / a.topk, i % a.topk);
        wts[i] = w;
        if (blockIdx.x == 0) {
            if (a.ids_out != nullptr) a.ids_out[i] = a.ids[i];
            if (a.weights_out != nullptr) a.weights_out[i] = w;
        }
    }
    __syncthreads();
    for (int e = wave; e < a.experts; e += 4) {
        int slot = -1;
        if (lane < a.n)
            for (int j = 0; j < a.topk; ++j)
                if (a.ids[lane * a.topk + j] == e) slot = lane * a.topk + j;
        const uint64_t who = __ballot(slot >= 0);
        const int count = __popcll(who);
        if (count == 0) continue;
        if (slot >= 0) slots[wave][__popcll(who & ((1ull << lane) - 1ull))] = slot;
        __builtin_amdgcn_wave_barrier();
        const int64_t row = e * a.d + min(d0 + l16, a.d - 1);
        const int64_t sb = (e * ((a.d + 127) / 128) + (d0 >> 7)) * kb;
        for (int c0 = 0; c0 < count; c0 += 16) {
            const int s = slots[wave][min(c0 + l16, count - 1)];
            const uint16_t* h = a.hidden + s * fp;
            f32x4 y = {0.f, 0.f, 0.f, 0.f};
            for (int64_t t = 0; t < kb; ++t) {
                bf16x16 b[2];
                load_block(h + 128 * t, q, b);
                bf16x8 av[2];
                widen_block(*reinterpret_cast<const u32x4*>(a.down.values + row * (kb * 64) + 64 * t + 16 * q),
                            scale_value(a.down.scales[sb + t]), av);
                const uint32_t idx = a.down.meta[row * (kb * 4) + 4 * t + q];
                y = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[0], b[0], y, (int)idx, 0, 0);
                y = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[1], b[1], y, (int)(idx >> 16), 0, 0);
            }
            if (c0 + l16 < count)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[wave][s / a.topk][4 * q + i] += wts[s] * y[i];
        }
    }
    __syncthreads();
    for (int i = tid; i < a.n * 16; i += 256) {
        const int t = i >> 4, r = i & 15;
        const float y = (part[0][t][r] + part[1][t][r]) + (part[2][t][r] + part[3][t][r]);
        if (d0 + r < a.d) a.y[t * a.ldy + d0 + r] = to_bf16(y);
    }
}

}  // namespace

int launch_moe24_fp8(const MoeJob& a, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    const int64_t waves = a.n * a.experts + a.n;
    hipLaunchKernelGGL(moe_logits_kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL(moe_hidden_kernel, dim3((unsigned)(a.experts * ((a.f + 15) / 16))), dim3(64), 0, s,
                       a);
    e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL(moe_output_kernel, dim3((unsigned)((a.d + 15) / 16)), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace tsenor
