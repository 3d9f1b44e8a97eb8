// tsenor_fp8_moe.hip -- a mixture-of-experts layer for a few tokens
// (include/tsenor_fp8.h: tsenor_moe24_fp8).  Five launches:
//   logits  x R^T in fp64, and x copied to rows padded with zeros;
//   route   each token's experts and weights, each chosen expert's tokens;
//   hidden  per chosen expert and some rows of gate and up: both products, silu, product;
//   down    per chosen expert and some rows of down: what each of its tokens gains;
//   sum     a token's gains, weighted, in the order of its choices.
// Reading the chosen experts' weights bounds the layer, so a workgroup's four
// waves share the reduction out in stretches and keep several blocks' loads in
// flight; the waves' sums meet in LDS in wave order, without atomics.  33 tokens, 4 of 16
// experts, 4096 x 2048, over weights in turn: hidden 43 us for 168 MB (3.9 TB/s), down 27 us for
// 84 MB (3.1 TB/s), logits, route and sum 16 us together (38, 25 and 16 with the same weights
// again, in part from the last-level cache); one token, 6 of 64, 2048 x 1408: 10.8 + 5.8 + 10.4
// us, where the five launches and their dependent loads count more than the 32 MB.
// The hidden entries are kept as the sum of two bf16 numbers (16 fraction bits;
// one alone would lose as much as the rounding of y itself), which costs two more
// matrix instructions per block where the memory is waited for.
// The weights' 8-bit numbers become bf16, their scale folded into the conversion
// (v_cvt_scalef32_pk_bf16_fp8): exactly, subnormal ones too, but for bits below 2^-133
// (blocks with a scale below 2^-124).  They multiply the bf16 activations on the sparse
// matrix cores (v_smfmac_f32_16x16x64_bf16).  Operand layout of that
// instruction (measured with an in-bounds probe), lane l, q = l / 16: A row
// l % 16, eight values that cover 16 entries; when these are entries
// 32q + 16j .. 32q + 16j + 15 of a block of 128 (j = 0, 1: the two instructions
// of the block), B column l % 16 holds entries 32(q/2) + 16j + 8(q%2) .. +7 and
// the eight 64 further on.  Both activations are kept in the order of those loads
// (place_of), so that the four lanes of a row read 64 bytes at a time: in their own order
// they would read pieces of 32 bytes, at half the rate of the address unit.
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
constexpr int kWaves = 4;  // of the hidden and down workgroups

// Where entry k of a row of activations is kept: eight entries stay together; within
// their block of 128, load i = 2j + (half) of lane group q finds them at 8 (4i + q).
__device__ __forceinline__ int place_of(int k) {
    const int half = (k >> 6) & 1, q = ((k >> 4) & 2) | ((k >> 3) & 1), j = (k >> 4) & 1;
    return (k & ~127) | (8 * (4 * (2 * j + half) + q)) | (k & 7);
}

// logits[e][t] in fp64, products too (those of bf16 numbers reach from 2^-266 to 2^256: fp32
// loses the ends).  A workgroup per expert and kLogitTokens tokens, its four waves a quarter of
// d each; the workgroups behind those copy x.
template <int kLogitTokens>
__global__ __launch_bounds__(256) void moe_logits_kernel(MoeJob a) {
    __shared__ double part[4][kLogitTokens];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t groups = (a.n + kLogitTokens - 1) / kLogitTokens;
    if (blockIdx.x >= groups * a.experts) {
        const int64_t t = blockIdx.x - groups * a.experts, dp = pad128(a.d);
        for (int64_t i = tid; i < dp; i += 256)
            a.xpad[t * dp + place_of((int)i)] = i < a.d ? a.x[t * a.ldx + i] : (uint16_t)0;
        return;
    }
    const int64_t e = blockIdx.x / groups, t0 = (blockIdx.x - e * groups) * kLogitTokens;
    const uint16_t* r = a.router + e * a.ldr;
    const uint16_t* x[kLogitTokens];
#pragma unroll
    for (int j = 0; j < kLogitTokens; ++j) x[j] = a.x + min(t0 + j, a.n - 1) * a.ldx;
    double sum[kLogitTokens] = {};
    for (int64_t i = 8 * tid; i < a.d; i += 8 * 256) {
        uint16_t rv[8], xv[kLogitTokens][8];
        load8(r, i, a.d, a.rvec, rv);
#pragma unroll
        for (int j = 0; j < kLogitTokens; ++j) load8(x[j], i, a.d, a.xvec, xv[j]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const double w = (double)widen(rv[c]);
#pragma unroll
            for (int j = 0; j < kLogitTokens; ++j) sum[j] = __builtin_fma((double)widen(xv[j][c]), w, sum[j]);
        }
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

// A token's logit as the key of its order: larger first, NaN last.  Ties go to the lower
// expert, which the comparison of the keys' holders adds.
__device__ __forceinline__ uint64_t logit_key(double l) {
    if (l != l) return 0u;
    const uint64_t b = __builtin_bit_cast(uint64_t, l == 0.0 ? 0.0 : l);  // both zeros alike
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// Largest value of the wave, in every lane (the partial maxima move by DPP: lane 63 ends up
// with all of them).
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t max_from(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_from<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8: within rows of 16 lanes
    v = max_from<0x112, 0xF>(v);
    v = max_from<0x114, 0xF>(v);
    v = max_from<0x118, 0xF>(v);
    v = max_from<0x142, 0xA>(v);  // row_bcast 15 and 31: on to the rows above
    v = max_from<0x143, 0xC>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// One workgroup.  A wave takes a token: its lanes hold the experts' keys (e = lane + 64 i),
// and each round takes the largest.  Then the chosen experts are numbered in ascending
// order: number j is expert chosen[j] with counts[j] entries in lists[j], in the tokens'
// order: the slot t * topk + rank, and t in the upper 16 bits.  The last entry is repeated
// up to a multiple of 16.
constexpr int kRouteWaves = 16, kMaxExperts = 512;
template <int kHeld>  // experts of a lane: 64 kHeld in all
__global__ __launch_bounds__(64 * kRouteWaves) void moe_route_kernel(MoeJob a, int groups) {
    __shared__ uint16_t taken[kMaxTokens * kMaxTop];
    __shared__ unsigned long long tokens[kMaxExperts];  // bit t: token t chose the expert
    __shared__ int number[kMaxExperts];
    __shared__ int wave_chosen[8];
    const int tid = threadIdx.x, lane = tid & 63, n = (int)a.n, experts = (int)a.experts, topk = a.topk;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (tid < kMaxExperts) tokens[tid] = 0ull;
    __syncthreads();
    for (int t = wave; t < n; t += kRouteWaves) {
        double l[kHeld];
        uint64_t key[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) l[i] = lane + 64 * i < experts ? a.logits[(lane + 64 * i) * n + t] : 0.0;
        uint32_t left = 0u;  // this lane's experts that are not taken yet
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            key[i] = logit_key(l[i]);
            left |= lane + 64 * i < experts ? 1u << i : 0u;
        }
        double mine = 0.0;
        int mine_e = 0;
        for (int r = 0; r < topk; ++r) {
            uint64_t best = 0u;
            int at = -1;
#pragma unroll
            for (int i = kHeld - 1; i >= 0; --i)  // downwards: of equal keys the lowest expert stays
                if ((left >> i) & 1u && key[i] >= best) {
                    best = key[i];
                    at = i;
                }
            // the largest key (its halves in turn), then the lowest expert among its holders
            const uint32_t hi = wave_max(at < 0 ? 0u : (uint32_t)(best >> 32));
            const bool in = at >= 0 && (uint32_t)(best >> 32) == hi;
            const uint32_t lo = wave_max(in ? (uint32_t)best : 0u);
            const int e = kMaxExperts - (int)wave_max(in && (uint32_t)best == lo ? kMaxExperts - (lane + 64 * at) : 0u);
            double v = 0.0;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) v = (e >> 6) == i ? l[i] : v;
            v = __shfl(v, e & 63, 64);
            if ((e & 63) == lane) left &= ~(1u << (e >> 6));
            if (lane == r) {
                mine = v;
                mine_e = e;
            }
        }
        // softmax over the chosen logits; the first is the largest
        const double top = __shfl(mine, 0, 64);
        const float p = lane < topk ? expf((float)(mine - top)) : 0.f;
        float sum = p;
#pragma unroll
        for (int d = 1; d < kMaxTop; d <<= 1) sum += __shfl_xor(sum, d, 64);
        if (lane < topk) {
            const int slot = t * topk + lane;
            taken[slot] = (uint16_t)mine_e;
            atomicOr(&tokens[mine_e], 1ull << t);
            a.weights[slot] = p / sum;
            if (a.ids_out != nullptr) a.ids_out[slot] = mine_e;
            if (a.weights_out != nullptr) a.weights_out[slot] = p / sum;
        }
    }
    __syncthreads();
    const int count = tid < experts ? __popcll(tokens[tid]) : 0;  // a thread per expert
    const uint64_t who = __ballot(count > 0);
    if (wave < 8 && lane == 0) wave_chosen[wave] = __popcll(who);
    __syncthreads();
    int j = __popcll(who & ((1ull << lane) - 1ull)), total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        j += w < wave ? wave_chosen[w] : 0;
        total += wave_chosen[w];
    }
    if (count > 0) {
        a.counts[j] = count;
        a.chosen[j] = tid;
        number[tid] = j;
    }
    if (total + tid < groups) a.counts[total + tid] = 0;  // fewer chosen than the grid allows
    __syncthreads();
    if (tid < n * topk) {  // a thread per slot
        const int t = tid / topk, e = taken[tid], entry = tid | (t << 16);
        const uint64_t others = tokens[e];
        const int at = __popcll(others & ((1ull << t) - 1ull)), c = __popcll(others);
        int* list = a.lists + number[e] * kMaxTokens;
        list[at] = entry;
        if (at == c - 1)
            for (int i = c; i < ((c + 15) & ~15); ++i) list[i] = entry;
    }
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
// The lane's B operands of the block at x (a row of activations in that order).
__device__ __forceinline__ void load_block(const uint16_t* x, int q, bf16x16 b[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const u32x4 lo = *reinterpret_cast<const u32x4*>(x + 64 * j + 8 * q);
        const u32x4 hi = *reinterpret_cast<const u32x4*>(x + 64 * j + 32 + 8 * q);
        typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
        const u32x8 w = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        b[j] = __builtin_bit_cast(bf16x16, w);
    }
}
// The conversion takes the exponent field of its scale operand: the byte itself (0 is 2^-127).
__device__ __forceinline__ float scale_value(int byte) { return bits_float((uint32_t)byte << 23); }

// hidden: one workgroup per (chosen expert, 16 MT rows of gate and up).
template <int MT>
__global__ __launch_bounds__(64 * kWaves) void moe_hidden_kernel(MoeJob a) {
    __shared__ f32x4 sums[kWaves][2 * MT][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t ft = (a.f + 16 * MT - 1) / (16 * MT);
    const int j = (int)(blockIdx.x / ft);
    const int64_t f0 = (blockIdx.x - j * ft) * (16 * MT);
    const int count = a.counts[j], e = a.chosen[j], first = a.lists[j * kMaxTokens + l16];
    if (count == 0) return;
    const int kb = (int)((a.d + 127) / 128);
    const int64_t dp = kb * 128, fp = pad128(a.f);
    int64_t row[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) row[m] = (e * a.f + min(f0 + 16 * m + l16, a.f - 1)) * kb;
    const int64_t sb = (e * ((a.f + 127) / 128) + (f0 >> 7)) * kb;  // 16 MT rows lie in one block of 128
    const int tbegin = kb * wave / kWaves, tend = kb * (wave + 1) / kWaves;
    for (int c0 = 0; c0 < count; c0 += 16) {
        const int entry = c0 == 0 ? first : a.lists[j * kMaxTokens + c0 + l16], slot = entry & 0xFFFF;
        const uint16_t* x = a.xpad + (entry >> 16) * dp;
        f32x4 acc[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int t0 = tbegin; t0 < tend; t0 += 4) {
            uint32_t idx[MT][2][4];
            u32x4 own[MT][2];
            const int tq = min(t0 + q, tend - 1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                own[m][0] = *reinterpret_cast<const u32x4*>(a.gate.meta + (row[m] + tq) * 4);
                own[m][1] = *reinterpret_cast<const u32x4*>(a.up.meta + (row[m] + tq) * 4);
            }
#pragma unroll
            for (int p = 0; p < 4; p += 2) {
                if (p > 0 && t0 + p >= tend) break;
                u32x4 v[2][MT][2];
                int sc[2][2];
                bf16x16 b[2][2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = min(t0 + p + u, tend - 1);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        v[u][m][0] = *reinterpret_cast<const u32x4*>(a.gate.values + (row[m] + t) * 64 + 16 * q);
                        v[u][m][1] = *reinterpret_cast<const u32x4*>(a.up.values + (row[m] + t) * 64 + 16 * q);
                    }
                    sc[u][0] = a.gate.scales[sb + t];
                    sc[u][1] = a.up.scales[sb + t];
                    load_block(x + 128 * t, q, b[u]);
                }
                __builtin_amdgcn_sched_barrier(0);  // all loads first
                if (p == 0)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i) words_of_blocks(own[m][i], idx[m][i]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (t0 + p + u >= tend) break;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            bf16x8 av[2];
                            widen_block(v[u][m][i], scale_value(sc[u][i]), av);
                            const uint32_t x = idx[m][i][p + u];
                            acc[m][i] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[0], b[u][0], acc[m][i], (int)x, 0, 0);
                            acc[m][i] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[1], b[u][1], acc[m][i],
                                                                                  (int)(x >> 16), 0, 0);
                        }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            sums[wave][2 * m][lane] = acc[m][0];
            sums[wave][2 * m + 1][lane] = acc[m][1];
        }
        __syncthreads();
        if (wave < MT && c0 + l16 < count) {
            f32x4 g = sums[0][2 * wave][lane], u = sums[0][2 * wave + 1][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                g += sums[w][2 * wave][lane];
                u += sums[w][2 * wave + 1][lane];
            }
            const int64_t f1 = f0 + 16 * wave;
            uint16_t *hi = a.hidden + slot * fp, *lo = hi + a.n * a.topk * fp;
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
                *reinterpret_cast<u32x2*>(hi + place_of((int)f1 + 4 * q)) = ph;
                *reinterpret_cast<u32x2*>(lo + place_of((int)f1 + 4 * q)) = pl;
            }
            if (wave == MT - 1 && f1 + 16 >= a.f)  // the last tile clears the padding behind it
                for (int i = (int)f1 + 16 + q; i < fp; i += 4) hi[place_of(i)] = lo[place_of(i)] = 0;
        }
        __syncthreads();
    }
}

// down: one workgroup per (chosen expert, 16 MT rows of down): what each of the expert's tokens
// gains, unweighted, into gains[slot].
template <int MT>
__global__ __launch_bounds__(64 * kWaves) void moe_down_kernel(MoeJob a) {
    __shared__ f32x4 sums[kWaves][MT][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t dt = (a.d + 16 * MT - 1) / (16 * MT);
    const int j = (int)(blockIdx.x / dt);
    const int64_t d0 = (blockIdx.x - j * dt) * (16 * MT);
    const int count = a.counts[j], e = a.chosen[j], first = a.lists[j * kMaxTokens + l16];
    if (count == 0) return;
    const int kb = (int)((a.f + 127) / 128);
    const int64_t fp = kb * 128, lo_at = a.n * a.topk * fp, dp = (a.d + 3) & ~(int64_t)3;
    int64_t row[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) row[m] = (e * a.d + min(d0 + 16 * m + l16, a.d - 1)) * kb;
    const int64_t sb = (e * ((a.d + 127) / 128) + (d0 >> 7)) * kb;  // 16 MT rows lie in one block of 128
    const int tbegin = kb * wave / kWaves, tend = kb * (wave + 1) / kWaves;
    for (int c0 = 0; c0 < count; c0 += 16) {
        const int slot = (c0 == 0 ? first : a.lists[j * kMaxTokens + c0 + l16]) & 0xFFFF;
        const uint16_t* h = a.hidden + slot * fp;
        f32x4 acc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int t0 = tbegin; t0 < tend; t0 += 4) {
            uint32_t idx[MT][4];
            u32x4 own[MT];
            const int tq = min(t0 + q, tend - 1);
#pragma unroll
            for (int m = 0; m < MT; ++m) own[m] = *reinterpret_cast<const u32x4*>(a.down.meta + (row[m] + tq) * 4);
#pragma unroll
            for (int p = 0; p < 4; p += 2) {
                if (p > 0 && t0 + p >= tend) break;
                u32x4 v[2][MT];
                int sc[2];
                bf16x16 hi[2][2], lo[2][2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = min(t0 + p + u, tend - 1);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        v[u][m] = *reinterpret_cast<const u32x4*>(a.down.values + (row[m] + t) * 64 + 16 * q);
                    sc[u] = a.down.scales[sb + t];
                    load_block(h + 128 * t, q, hi[u]);
                    load_block(h + lo_at + 128 * t, q, lo[u]);
                }
                __builtin_amdgcn_sched_barrier(0);  // all loads first
                if (p == 0)
#pragma unroll
                    for (int m = 0; m < MT; ++m) words_of_blocks(own[m], idx[m]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (t0 + p + u >= tend) break;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        bf16x8 av[2];
                        widen_block(v[u][m], scale_value(sc[u]), av);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int x = (int)(idx[m][p + u] >> (16 * i));
                            acc[m] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[i], hi[u][i], acc[m], x, 0, 0);
                            acc[m] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[i], lo[u][i], acc[m], x, 0, 0);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) sums[wave][m][lane] = acc[m];
        __syncthreads();
        if (wave < MT && c0 + l16 < count) {
            f32x4 y = sums[0][wave][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) y += sums[w][wave][lane];
            const int64_t r = d0 + 16 * wave + 4 * q;
            if (r < dp) *reinterpret_cast<f32x4*>(a.gains + slot * dp + r) = y;
        }
        __syncthreads();
    }
}

// y: a token's gains, weighted and summed in the order of its choices.  One workgroup per
// token and 1024 entries.
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeJob a) {
    const int64_t parts = (a.d + 1023) / 1024, t = blockIdx.x / parts, c0 = (blockIdx.x - t * parts) * 1024;
    const int64_t c = c0 + 4 * threadIdx.x, dp = (a.d + 3) & ~(int64_t)3;
    if (c >= dp) return;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int j = 0; j < a.topk; ++j) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(a.gains + (t * a.topk + j) * dp + c);
        const float w = a.weights[t * a.topk + j];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(w, v[i], y[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < a.d) a.y[t * a.ldy + c + i] = to_bf16(y[i]);
}

}  // namespace

int launch_moe24_fp8(const MoeJob& a, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    const int64_t groups = a.n * a.topk < a.experts ? a.n * a.topk : a.experts;  // chosen experts at most
    const auto tiles = [&](int64_t length, int rows) { return groups * ((length + rows - 1) / rows); };
    const int rows_hidden = tiles(a.f, 32) >= 512 ? 32 : 16, rows_down = tiles(a.d, 64) >= 128 ? 64 : 16;
    if (!grid_fits(tiles(a.f, rows_hidden), 64 * kWaves) || !grid_fits(tiles(a.d, rows_down), 64 * kWaves))
        return kGridTooLarge;
    if (a.n < 4) hipLaunchKernelGGL(moe_logits_kernel<1>, dim3((unsigned)(a.experts * a.n + a.n)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(moe_logits_kernel<4>, dim3((unsigned)(a.experts * ((a.n + 3) / 4) + a.n)), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    const auto route = a.experts <= 64 ? moe_route_kernel<1> : a.experts <= 128 ? moe_route_kernel<2> : moe_route_kernel<8>;
    hipLaunchKernelGGL(route, dim3(1), dim3(64 * kRouteWaves), 0, s, a, (int)groups);
    e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    // Rows of a workgroup: several tiles of 16, so that a token's activations are read once for
    // all of them, unless too few workgroups would be left.  Measured (us, four waves; eight are
    // slower by 0 to 20%, as their stretches end inside the four blocks whose metadata one load
    // brings) with 16 / 32 / 64 rows: hidden, one token, 6 experts, 2048 x 1408: 9.9 / 11.6 / 12.7;
    // 33 tokens, 16 experts, 4096 x 2048: 44 / 39 / 41; down: 6.8 / 6.0 / 5.8 and 49 / 32 / 25.
    const dim3 threads(64 * kWaves);
    if (rows_hidden == 32)
        hipLaunchKernelGGL(moe_hidden_kernel<2>, dim3((unsigned)tiles(a.f, 32)), threads, 0, s, a);
    else
        hipLaunchKernelGGL(moe_hidden_kernel<1>, dim3((unsigned)tiles(a.f, 16)), threads, 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    if (rows_down == 64)
        hipLaunchKernelGGL(moe_down_kernel<4>, dim3((unsigned)tiles(a.d, 64)), threads, 0, s, a);
    else
        hipLaunchKernelGGL(moe_down_kernel<1>, dim3((unsigned)tiles(a.d, 16)), threads, 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL(moe_sum_kernel, dim3((unsigned)(a.n * ((a.d + 1023) / 1024))), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace tsenor
