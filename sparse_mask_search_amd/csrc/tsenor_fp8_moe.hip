// tsenor_fp8_moe.hip -- a mixture-of-experts layer for a few tokens
// (include/tsenor_fp8.h: tsenor_moe24_fp8).  Three launches:
//   logits  x R^T in fp64, and x copied to rows padded with zeros;
//   hidden  per expert and 16 rows of gate and up: the tokens that chose the
//           expert (each workgroup ranks it among the logits), both products,
//           silu, product;
//   output  per 16 rows of down: every token's experts, weighted and summed.
// Reading the chosen experts' weights bounds the layer, so a workgroup's eight
// waves share the reduction out in stretches and keep several blocks' loads in
// flight; the waves' sums meet in LDS in wave order, without atomics.
// The hidden entries are kept as the sum of two bf16 numbers (16 fraction bits;
// one alone would lose as much as the rounding of y itself), which costs two more
// matrix instructions per block where the memory is waited for.
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
constexpr int kHiddenWaves = 8, kOutputWaves = 16;

// logits[e][t] in fp64 (products of bf16 numbers are exact in fp32).  A workgroup
// per expert and four tokens, its four waves a quarter of d each; the workgroups
// behind those copy x.
constexpr int kLogitTokens = 4;
__global__ __launch_bounds__(256) void moe_logits_kernel(MoeJob a) {
    __shared__ double part[4][kLogitTokens];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t groups = (a.n + kLogitTokens - 1) / kLogitTokens;
    if (blockIdx.x >= groups * a.experts) {
        const int64_t t = blockIdx.x - groups * a.experts, dp = pad128(a.d);
        for (int64_t i = tid; i < dp; i += 256)
            a.xpad[t * dp + i] = i < a.d ? a.x[t * a.ldx + i] : (uint16_t)0;
        return;
    }
    const int64_t e = blockIdx.x / groups, t0 = (blockIdx.x - e * groups) * kLogitTokens;
    const uint16_t* r = a.router + e * a.ldr;
    const uint16_t* x[kLogitTokens];
#pragma unroll
    for (int j = 0; j < kLogitTokens; ++j) x[j] = a.x + min(t0 + j, a.n - 1) * a.ldx;
    double sum[kLogitTokens] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t i = 8 * tid; i < a.d; i += 8 * 256) {
        uint16_t rv[8], xv[kLogitTokens][8];
        load8(r, i, a.d, a.rvec, rv);
#pragma unroll
        for (int j = 0; j < kLogitTokens; ++j) load8(x[j], i, a.d, a.xvec, xv[j]);
#pragma unroll
        for (int j = 0; j < kLogitTokens; ++j)
#pragma unroll
            for (int c = 0; c < 8; ++c) sum[j] += (double)(widen(xv[j][c]) * widen(rv[c]));
    }
#pragma unroll
    for (int j = 0; j < kLogitTokens; ++j) {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum[j] += __shfl_xor(sum[j], d, 64);
        if (lane == 0) part[wave][j] = sum[j];
    }
    __syncthreads();
    if (tid < kLogitTokens && t0 + tid < a.n)
        a.logits[e * a.n + t0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
}

// Whether expert j comes before expert e in a token's order: larger logit first,
// ties to the lower index, NaN last.
__device__ __forceinline__ bool before(double lj, int j, double le, int e) {
    if (le != le) return lj == lj || j < e;
    return lj > le || (lj == le && j < e);
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

// With few tokens only some experts are chosen: a grid over the at most n * topk
// chosen ones is far smaller than one over all.  Each workgroup then ranks all
// experts itself (n * experts logits in LDS) and takes the blockIdx-th chosen one.
constexpr int kCompactLogits = 2048;
__host__ __device__ __forceinline__ bool compact(const MoeJob& a) {
    return a.n * a.topk < a.experts && a.n * a.experts <= kCompactLogits;
}

// hidden: one workgroup per (expert, 16 MT rows of gate and up).  Expert number j of the
// grid (j-th chosen, or j itself) leaves its tokens' slots t * topk + rank in
// lists[j], for the output.
template <int MT>
__global__ __launch_bounds__(64 * kHiddenWaves) void moe_hidden_kernel(MoeJob a) {
    constexpr int kThreads = 64 * kHiddenWaves;
    __shared__ union {
        f32x4 sums[kHiddenWaves][2 * MT][64];
        struct {
            double logits[kCompactLogits];
            uint16_t rank[kCompactLogits];
        } all;
    } lds;
    __shared__ uint32_t chosen[16];
    __shared__ int ranks[kHiddenWaves][kMaxTokens];
    __shared__ int slots[kMaxTokens];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t ft = (a.f + 16 * MT - 1) / (16 * MT);
    const int j = (int)(blockIdx.x / ft), n = (int)a.n, experts = (int)a.experts;
    const int64_t f0 = (blockIdx.x - j * ft) * (16 * MT);
    int e = j, r = 0;
    if (compact(a)) {
        if (tid < 16) chosen[tid] = 0u;
        for (int i = tid; i < n * experts; i += kThreads) lds.all.logits[i] = a.logits[i];
        __syncthreads();
        for (int i = tid; i < n * experts; i += kThreads) {
            const int c = i / n, t = i - c * n;
            const double mine = lds.all.logits[i];
            int rank = 0;
#pragma unroll 8
            for (int o = 0; o < experts; ++o) rank += before(lds.all.logits[o * n + t], o, mine, c) ? 1 : 0;
            lds.all.rank[i] = (uint16_t)rank;
            if (rank < a.topk) atomicOr(&chosen[c >> 5], 1u << (c & 31));
        }
        __syncthreads();
        int left = j;
        e = -1;
        for (int w = 0; w < 16 && e < 0; ++w) {  // uniform
            uint32_t bits = chosen[w];
            const int c = __popc(bits);
            if (left >= c) {
                left -= c;
                continue;
            }
            for (; left > 0; --left) bits &= bits - 1u;
            e = 32 * w + __builtin_ctz(bits);
        }
        if (e < 0) {  // fewer experts chosen than the grid allows
            if (f0 == 0 && tid == 0) a.counts[j] = 0;
            return;
        }
        e = __builtin_amdgcn_readfirstlane(e);
        if (lane < n) r = lds.all.rank[e * n + lane];
    } else {
        // rank of e for token `lane`; each wave compares with every eighth expert
        if (lane < n) {
            const double le = a.logits[e * n + lane];
#pragma unroll 8
            for (int o = wave; o < experts; o += kHiddenWaves)
                r += before(a.logits[o * n + lane], o, le, e) ? 1 : 0;
        }
        ranks[wave][lane] = r;
        __syncthreads();
        r = 0;
#pragma unroll
        for (int w = 0; w < kHiddenWaves; ++w) r += ranks[w][lane];
    }
    const bool mine = lane < n && r < a.topk;
    const uint64_t who = __ballot(mine);  // the same in every wave
    const int count = __popcll(who);
    if (wave == 0) {
        const int at = __popcll(who & ((1ull << lane) - 1ull)), slot = lane * a.topk + r;
        if (mine) slots[at] = slot;
        if (f0 == 0) {
            if (lane == 0) {
                a.counts[j] = count;
                a.chosen[j] = e;
            }
            if (mine) {
                a.lists[j * kMaxTokens + at] = slot;
                a.ids[slot] = e;
            }
        }
    }
    if (count == 0) return;
    __syncthreads();
    constexpr int kAhead = 2;
    const int kb = (int)((a.d + 127) / 128);
    const int64_t dp = kb * 128, fp = pad128(a.f);
    int64_t row[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) row[m] = (e * a.f + min(f0 + 16 * m + l16, a.f - 1)) * kb;
    const int64_t sb = (e * ((a.f + 127) / 128) + (f0 >> 7)) * kb;  // 16 MT rows lie in one block of 128
    const int tbegin = kb * wave / kHiddenWaves, tend = kb * (wave + 1) / kHiddenWaves;
    for (int c0 = 0; c0 < count; c0 += 16) {
        const uint16_t* x = a.xpad + (slots[min(c0 + l16, count - 1)] / a.topk) * dp;
        f32x4 acc[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int t0 = tbegin; t0 < tend; t0 += kAhead) {
            u32x4 v[kAhead][MT][2];
            uint32_t idx[kAhead][MT][2];
            int sc[kAhead][2];
            bf16x16 b[kAhead][2];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int t = min(t0 + u, tend - 1);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    v[u][m][0] = *reinterpret_cast<const u32x4*>(a.gate.values + (row[m] + t) * 64 + 16 * q);
                    v[u][m][1] = *reinterpret_cast<const u32x4*>(a.up.values + (row[m] + t) * 64 + 16 * q);
                    idx[u][m][0] = a.gate.meta[(row[m] + t) * 4 + q];
                    idx[u][m][1] = a.up.meta[(row[m] + t) * 4 + q];
                }
                sc[u][0] = a.gate.scales[sb + t];
                sc[u][1] = a.up.scales[sb + t];
                load_block(x + 128 * t, q, b[u]);
            }
            __builtin_amdgcn_sched_barrier(0);  // all loads first
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (t0 + u >= tend) break;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        bf16x8 av[2];
                        widen_block(v[u][m][i], scale_value(sc[u][i]), av);
                        acc[m][i] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[0], b[u][0], acc[m][i],
                                                                              (int)idx[u][m][i], 0, 0);
                        acc[m][i] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[1], b[u][1], acc[m][i],
                                                                              (int)(idx[u][m][i] >> 16), 0, 0);
                    }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            lds.sums[wave][2 * m][lane] = acc[m][0];
            lds.sums[wave][2 * m + 1][lane] = acc[m][1];
        }
        __syncthreads();
        if (wave < MT && c0 + l16 < count) {
            f32x4 g = lds.sums[0][2 * wave][lane], u = lds.sums[0][2 * wave + 1][lane];
#pragma unroll
            for (int w = 1; w < kHiddenWaves; ++w) {
                g += lds.sums[w][2 * wave][lane];
                u += lds.sums[w][2 * wave + 1][lane];
            }
            const int64_t f1 = f0 + 16 * wave;
            uint16_t *hi = a.hidden + slots[c0 + l16] * fp, *lo = hi + a.n * a.topk * fp;
            u32x2 ph = {0u, 0u}, pl = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float h = f1 + 4 * q + i < a.f ? g[i] / (1.f + expf(-g[i])) * u[i] : 0.f;
                const uint16_t top = to_bf16(h);
                // what the first number leaves; nothing behind an infinity
                const float rest = (top & 0x7F80u) == 0x7F80u ? 0.f : h - widen(top);
                ph[i >> 1] |= (uint32_t)top << (16 * (i & 1));
                pl[i >> 1] |= (uint32_t)to_bf16(rest) << (16 * (i & 1));
            }
            if (f1 < fp) {
                *reinterpret_cast<u32x2*>(hi + f1 + 4 * q) = ph;
                *reinterpret_cast<u32x2*>(lo + f1 + 4 * q) = pl;
            }
            if (wave == MT - 1 && f1 + 16 >= a.f)  // the last tile clears the padding behind it
                for (int64_t i = f1 + 16 + q; i < fp; i += 4) hi[i] = lo[i] = 0;
        }
        __syncthreads();
    }
}

// Softmax weight of slot (t, r) over token t's chosen logits; they are in
// descending order, so the first is the largest.
__device__ __forceinline__ float weight_of(const MoeJob& a, int64_t t, int r) {
    const double top = a.logits[a.ids[t * a.topk] * a.n + t];
    float sum = 0.f, mine = 0.f;
    for (int j = 0; j < a.topk; ++j) {
        const float v = expf((float)(a.logits[a.ids[t * a.topk + j] * a.n + t] - top));
        sum += v;
        mine = j == r ? v : mine;
    }
    return mine / sum;
}

// output: one workgroup per 16 rows of down.  The work is a sequence of blocks of 128
// (expert after expert, 16 of its tokens after 16); each wave takes an equal stretch of
// it and adds what an expert's tokens gain to its own partial sums.
__global__ __launch_bounds__(64 * kOutputWaves) void moe_output_kernel(MoeJob a, int groups) {
    constexpr int kMaxUnits = 512 + 64;  // (expert, 16 tokens) pairs: at most experts + n topk / 16
    __shared__ float part[kOutputWaves][kMaxTokens][17];
    __shared__ float wts[kMaxTokens * kMaxTop];
    __shared__ uint16_t unit_group[kMaxUnits], unit_expert[kMaxUnits], unit_slot[kMaxUnits][16];
    __shared__ uint8_t unit_first[kMaxUnits], unit_count[kMaxUnits];
    __shared__ int total_units;
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t d0 = (int64_t)blockIdx.x * 16;
    const int kb = (int)((a.f + 127) / 128);
    const int64_t fp = kb * 128;
    if (wave == 0) {  // the sequence: prefix sums of the experts' numbers of 16 tokens
        int base = 0;
        for (int g0 = 0; g0 < groups; g0 += 64) {
            const int g = g0 + lane, count = g < groups ? a.counts[g] : 0, units = (count + 15) >> 4;
            const int e = count > 0 ? a.chosen[g] : 0;
            int before = units;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(before, d, 64);
                if (lane >= d) before += o;
            }
            for (int i = 0; i < units; ++i) {
                unit_group[base + before - units + i] = (uint16_t)g;
                unit_expert[base + before - units + i] = (uint16_t)e;
                unit_first[base + before - units + i] = (uint8_t)(16 * i);
                unit_count[base + before - units + i] = (uint8_t)min(16, count - 16 * i);
            }
            base += __shfl(before, 63, 64);
        }
        if (lane == 0) total_units = base;
    }
    for (int i = tid; i < kOutputWaves * kMaxTokens * 17; i += 64 * kOutputWaves) (&part[0][0][0])[i] = 0.f;
    for (int i = tid; i < a.n * a.topk; i += 64 * kOutputWaves) {
        const float w = weight_of(a, i / a.topk, i % a.topk);
        wts[i] = w;
        if (blockIdx.x == 0) {
            if (a.ids_out != nullptr) a.ids_out[i] = a.ids[i];
            if (a.weights_out != nullptr) a.weights_out[i] = w;
        }
    }
    __syncthreads();
    const int total = __builtin_amdgcn_readfirstlane(total_units);
    for (int i = tid; i < total * 16; i += 64 * kOutputWaves) {
        const int u = i >> 4;
        unit_slot[u][i & 15] =
            (uint16_t)a.lists[unit_group[u] * kMaxTokens + unit_first[u] + min(i & 15, unit_count[u] - 1)];
    }
    __syncthreads();
    constexpr int kAhead = 4;
    const int steps = total * kb;
    const int begin = (int)((int64_t)steps * wave / kOutputWaves), end = (int)((int64_t)steps * (wave + 1) / kOutputWaves);
    const int64_t dr = min(d0 + l16, a.d - 1);
    const int64_t drows = (a.d + 127) / 128;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    // weighted sums of unit u's tokens so far into this wave's partial sums
    const auto flush = [&](int u) {
        if (l16 < unit_count[u]) {
            const int slot = unit_slot[u][l16];
#pragma unroll
            for (int i = 0; i < 4; ++i) part[wave][slot / a.topk][4 * q + i] += wts[slot] * y[i];
        }
        y = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    for (int s0 = begin; s0 < end; s0 += kAhead) {
        u32x4 v[kAhead];
        uint32_t idx[kAhead];
        int sc[kAhead];
        const uint16_t* h[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int s = min(s0 + u, end - 1), unit = s / kb, t = s - unit * kb;
            const int e = unit_expert[unit], slot = unit_slot[unit][l16];
            const int64_t row = e * a.d + dr;
            v[u] = *reinterpret_cast<const u32x4*>(a.down.values + (row * kb + t) * 64 + 16 * q);
            idx[u] = a.down.meta[(row * kb + t) * 4 + q];
            sc[u] = a.down.scales[(e * drows + (d0 >> 7)) * kb + t];
            h[u] = a.hidden + slot * fp + 128 * t;
        }
        // the weights come from far, the hidden entries from L2: those follow in pairs
#pragma unroll
        for (int p = 0; p < kAhead; p += 2) {
            bf16x16 hi[2][2], lo[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                load_block(h[p + u], q, hi[u]);
                load_block(h[p + u] + a.n * a.topk * fp, q, lo[u]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int s = s0 + p + u;
                if (s >= end) break;
                bf16x8 av[2];
                widen_block(v[p + u], scale_value(sc[p + u]), av);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int x = (int)(idx[p + u] >> (16 * i));
                    y = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[i], hi[u][i], y, x, 0, 0);
                    y = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[i], lo[u][i], y, x, 0, 0);
                }
                if (s + 1 == end || (s + 1) % kb == 0) flush(s / kb);
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.n * 16; i += 64 * kOutputWaves) {
        const int t = i >> 4, r = i & 15;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kOutputWaves; ++w) sum += part[w][t][r];
        if (d0 + r < a.d) a.y[t * a.ldy + d0 + r] = to_bf16(sum);
    }
}

}  // namespace

int launch_moe24_fp8(const MoeJob& a, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    const int64_t logit_blocks = a.experts * ((a.n + kLogitTokens - 1) / kLogitTokens) + a.n;
    hipLaunchKernelGGL(moe_logits_kernel, dim3((unsigned)logit_blocks), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    // 64 rows per workgroup where that leaves two workgroups per CU, else 32 or 16
    const int64_t groups = compact(a) ? a.n * a.topk : a.experts;
    const auto tiles = [&](int rows) { return groups * ((a.f + rows - 1) / rows); };
    const dim3 threads(64 * kHiddenWaves);
    if (tiles(64) >= 512) hipLaunchKernelGGL(moe_hidden_kernel<4>, dim3((unsigned)tiles(64)), threads, 0, s, a);
    else if (tiles(32) >= 512) hipLaunchKernelGGL(moe_hidden_kernel<2>, dim3((unsigned)tiles(32)), threads, 0, s, a);
    else hipLaunchKernelGGL(moe_hidden_kernel<1>, dim3((unsigned)tiles(16)), threads, 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL(moe_output_kernel, dim3((unsigned)((a.d + 15) / 16)), dim3(64 * kOutputWaves), 0, s, a,
                       (int)groups);
    return (int)hipGetLastError();
}

}  // namespace tsenor
