// tsenor_grouped.hip -- products grouped by expert (include/tsenor_ops.h): bf16
// products, weight gradients, 8-bit integer products.
//
// A product is tiles of (inner columns) x (rows); the operand along the inner dimension
// is on the rows of the matrix instruction, so that a lane holds four neighbouring
// entries of an output row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor_internal.h"
#include "tsenor_ops_device.h"

namespace tsenor {
namespace {

using namespace ops;

enum Kind { kProduct, kGradient };

// Sixteen bytes of a row of which `valid` are there, at any alignment of the entries; zeros
// behind them.
template <class T>
__device__ __forceinline__ u32x4 load16(const uint8_t* p, int64_t valid) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (valid >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else if (valid > 0) {
#pragma unroll
        for (int i = 0; i < 16 / T::kSize; ++i)
            if (i * T::kSize < valid) {
                const uint32_t x = T::kSize == 2 ? reinterpret_cast<const uint16_t*>(p)[i] : p[i];
                v[i * T::kSize / 4] |= x << (8 * (i * T::kSize % 4));
            }
    }
    return v;
}

// Any alignment and any size: tiles of 64 x 64, four waves of 32 x 32, operands through
// registers into two LDS buffers.  AT, BT: the operand is contiguous along its columns.
template <class T, bool AT, bool BT, Kind K, class TO>
__global__ __launch_bounds__(256) void product_any_kernel(const GroupedJob job) {
    __shared__ u32x4 ta[2][256], tb[2][256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t across = (job.inner + 63) / 64, bid = blockIdx.x;
    const int64_t inner0 = bid % across * 64;
    int64_t outer0, outer_end;  // rows of the output
    int64_t count;              // weight gradient: rows of the reduction
    const uint8_t *a = static_cast<const uint8_t*>(job.a), *b = static_cast<const uint8_t*>(job.b);
    TO* out = static_cast<TO*>(job.out);
    int expert;
    if constexpr (K == kProduct) {
        RowTile t;
        if (!row_tile(job.ends, job.experts, job.rows, 64, (int)(bid / across), &t)) return;
        expert = t.expert;
        outer0 = t.first;
        outer_end = t.end;
        count = 0;
        if (expert < 0) {
            for (int i = tid; i < 64 * 64; i += 256)
                if (outer0 + (i >> 6) < outer_end && inner0 + (i & 63) < job.inner)
                    out[(outer0 + (i >> 6)) * job.ldo + inner0 + (i & 63)] = TO(0);
            return;
        }
        a += expert * job.astride + (AT ? inner0 * T::kSize : inner0 * job.lda);
        b += outer0 * job.ldb;
    } else {
        const int64_t down = (job.outer + 63) / 64, t = bid / across;
        expert = (int)(t / down);
        outer0 = t % down * 64;
        outer_end = job.outer;
        const int first = expert == 0 ? 0 : end_of(job.ends, expert - 1, job.rows);
        count = max(end_of(job.ends, expert, job.rows) - first, 0);
        a += first * job.lda + inner0 * T::kSize;
        b += first * job.ldb + outer0 * T::kSize;
        out += expert * job.ostride;
    }
    const int64_t ahave = job.inner - inner0, bhave = outer_end - outer0;  // columns of the tile that exist
    const int64_t reduce = K == kGradient ? count * T::kSize : job.kbytes;
    const int steps = (int)((reduce + 63) / 64);

    auto fetch = [&](const uint8_t* base, int64_t ld, int64_t have, bool turned, int s) {
        if (!turned) {
            const int r = tid >> 2, c = 64 * s + 16 * (tid & 3);
            return load16<T>(base + min((int64_t)r, have - 1) * ld + c, reduce - c);
        }
        const int r = 32 * s + (tid >> 3), c = 8 * (tid & 7);
        return load16<T>(base + r * ld + c * T::kSize, r * T::kSize < reduce ? (have - c) * T::kSize : 0);
    };
    const int slot_row = row_slot(tid >> 2, tid & 3), slot_turned = turned_slot<64>(tid >> 3, tid & 7);
    typename T::Sum acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0;
    u32x4 va, vb;
    if (steps > 0) {
        va = fetch(a, job.lda, ahave, AT, 0);
        vb = fetch(b, job.ldb, bhave, BT, 0);
    }
    const int ia = 32 * (wave & 1), ib = 32 * (wave >> 1);
    for (int s = 0; s < steps; ++s) {
        ta[s & 1][AT ? slot_turned : slot_row] = va;
        tb[s & 1][BT ? slot_turned : slot_row] = vb;
        __syncthreads();
        if (s + 1 < steps) {
            va = fetch(a, job.lda, ahave, AT, s + 1);
            vb = fetch(b, job.ldb, bhave, BT, s + 1);
        }
#pragma unroll
        for (int kc = 0; kc < 2; ++kc) {
            const u32x4 fa = AT ? turned_fragment<64>(ta[s & 1], ia, kc, lane) : row_fragment(ta[s & 1], ia, kc, lane);
            const u32x4 fb = BT ? turned_fragment<64>(tb[s & 1], ib, kc, lane) : row_fragment(tb[s & 1], ib, kc, lane);
            acc = T::mma(fa, fb, acc);
        }
    }
    const int64_t row = outer0 + ib + (lane & 31), c0 = inner0 + ia;
    if (row >= outer_end || c0 >= job.inner) return;
    uint32_t keep = 0xFFFFFFFFu;
    if constexpr (K == kGradient) {
        if (job.mask != nullptr) {
            const int64_t wpr = (job.inner + 31) / 32;
            keep = job.mask[(expert * job.outer + row) * wpr + (c0 >> 5)];
        }
    }
    float scale = 1.f;
    if constexpr (T::kSize == 1) scale = job.bs[row];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t c = c0 + 8 * i + 4 * (lane >> 5);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = (float)acc[4 * i + e];
            if constexpr (T::kSize == 1) v[e] = v[e] * scale * job.as[expert * job.inner + min(c + e, job.inner - 1)];
            if constexpr (K == kGradient)
                if (!((keep >> (8 * i + 4 * (lane >> 5) + e)) & 1u)) v[e] = 0.f;
        }
        put4(out + row * job.ldo, c, job.inner, job.ovec, v);
    }
}

// Few rows (at most 16 NT for an expert): reading the weights bounds the product, so a
// workgroup owns 16 MT columns of the output (rows of the weights) and each of its eight waves
// a stretch of the reduction, with the loads of kAhead units of 128 bytes in flight; the waves'
// sums meet in LDS, in wave order.  A lane q = lane / 16 takes bytes 32 q .. 32 q + 31 of a unit of
// both operands: the two instructions may take the reduction in any order that is the same for both.
// QX: bf16 tokens become 8-bit integers on the way.  Each workgroup takes the largest
// magnitudes of all tokens first, while its first weights are loaded.
constexpr int kFewWaves = 8;

template <class T, bool QX, int NT, int MT, class TO>
__global__ __launch_bounds__(64 * kFewWaves) void product_few_kernel(const GroupedJob job) {
    constexpr int kAhead = NT * MT >= 4 ? 1 : NT * MT >= 2 ? 2 : 4;
    typedef typename T::Sum4 Sum4;
    __shared__ Sum4 sums[kFewWaves][MT * NT][64];
    __shared__ TokenScale scale[QX ? 16 : 1];
    __shared__ uint32_t part[QX ? 16 : 1][kFewWaves];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t across = (job.inner + 16 * MT - 1) / (16 * MT);
    const int64_t inner0 = blockIdx.x % across * (16 * MT);
    TO* out = static_cast<TO*>(job.out);
    RowTile t;
    if (!row_tile(job.ends, job.experts, job.rows, 16 * NT, (int)(blockIdx.x / across), &t)) return;
    const int rows = min(t.end - t.first, 16 * NT);
    if (t.expert < 0) {
        for (int i = tid; i < rows * 16 * MT; i += 64 * kFewWaves)
            if (inner0 + i % (16 * MT) < job.inner)
                out[(t.first + (int64_t)(i / (16 * MT))) * job.ldo + inner0 + i % (16 * MT)] = TO(0);
        return;
    }
    const uint8_t *arow[MT], *brow[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        arow[m] = static_cast<const uint8_t*>(job.a) + t.expert * job.astride +
                  min(inner0 + 16 * m + l16, job.inner - 1) * job.lda + 32 * q;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        brow[n] = static_cast<const uint8_t*>(job.b) + (t.first + (int64_t)min(16 * n + l16, rows - 1)) * job.ldb +
                  (QX ? 0 : 32 * q);
    Sum4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = Sum4{0, 0, 0, 0};
    const int units = (int)((job.kbytes + 127) / 128);
    const int u0 = (int)((int64_t)units * wave / kFewWaves), u1 = (int)((int64_t)units * (wave + 1) / kFewWaves);
    const int whole = (int)(job.kbytes / 128);  // units without an end of the rows

    u32x4 av[kAhead][MT][2];
    auto load_a = [&](int u) {  // units u .. u + kAhead - 1; behind the stretch: its last one again, not used
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int v = min(u + i, u1 - 1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint8_t* p = arow[m] + 128 * (int64_t)v;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (v < whole) __builtin_memcpy(&av[i][m][c], p + 16 * c, 16);
                    else av[i][m][c] = load16<T>(p + 16 * c, job.kbytes - 128 * (int64_t)v - 32 * q - 16 * c);
                }
            }
        }
    };
    if (u0 < u1) load_a(u0);
    float to_int = 0.f;  // this lane's token
    int exponent = 0;
    if constexpr (QX) {
        const int64_t k = job.kbytes;  // entries: one byte of the weights each
        for (int r = 0; r < rows; ++r) {
            const uint16_t* x = static_cast<const uint16_t*>(job.b) + (t.first + (int64_t)r) * (job.ldb / 2);
            uint32_t most = 0u;
            for (int64_t c = 8 * tid; c < k; c += 8 * 64 * kFewWaves) {
                Eight<uint16_t> v;
                v.load(x, c, job.bcols, job.bvec);
                most = max(most, v.magnitude());
            }
            most = max64(most);
            if (lane == 0) part[r][wave] = most;
        }
        __syncthreads();
        if (tid < rows) {
            uint32_t most = 0u;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) most = max(most, part[tid][w]);
            scale[tid] = token_scale(most);
        }
        __syncthreads();
        const TokenScale mine = scale[min(l16, rows - 1)];
        to_int = mine.factor;
        exponent = mine.exponent;
    }
    for (int u = u0; u < u1; u += kAhead) {
        if (u > u0) load_a(u);
        u32x4 bv[kAhead][NT][2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int v = min(u + i, u1 - 1);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if constexpr (QX) {
                        const int64_t at = 128 * (int64_t)v + 32 * q + 16 * c;  // entry
                        const uint16_t* x = reinterpret_cast<const uint16_t*>(brow[n]);
                        Eight<uint16_t> lo, hi;
                        lo.load(x, at, job.bcols, job.bvec);
                        hi.load(x, at + 8, job.bcols, job.bvec);
                        const u32x2 a = integers(lo, to_int, exponent), b = integers(hi, to_int, exponent);
                        bv[i][n][c] = u32x4{a.x, a.y, b.x, b.y};
                    } else {
                        const uint8_t* p = brow[n] + 128 * (int64_t)v + 16 * c;
                        if (v < whole) __builtin_memcpy(&bv[i][n][c], p, 16);
                        else bv[i][n][c] = load16<T>(p, job.kbytes - 128 * (int64_t)v - 32 * q - 16 * c);
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (u + i >= u1) break;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[m][n] = T::mma(av[i][m][c], bv[i][n][c], acc[m][n]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) sums[wave][m * NT + n][lane] = acc[m][n];
    __syncthreads();
    for (int i = tid; i < MT * NT * 64; i += 64 * kFewWaves) {
        Sum4 v = sums[0][i >> 6][i & 63];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += sums[w][i >> 6][i & 63];
        const int l = i & 63, n = (i >> 6) % NT, m = (i >> 6) / NT, r = 16 * n + (l & 15);
        if (r >= rows) continue;
        const int64_t row = t.first + (int64_t)r, c0 = inner0 + 16 * m + 4 * (l >> 4);
        f32x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = (float)v[e];
            if constexpr (T::kSize == 1)
                y[e] = y[e] * (QX ? scale[QX ? r : 0].scale : job.bs[row]) *
                       job.as[t.expert * job.inner + min(c0 + e, job.inner - 1)];
        }
        put4(out + row * job.ldo, c0, job.inner, job.ovec, y);
    }
}

template <class T, bool AT, bool BT, Kind K, class TO>
int any(const GroupedJob& job, void* stream) {
    const int64_t across = (job.inner + 63) / 64;
    const int64_t down = K == kGradient ? (job.outer + 63) / 64 * job.experts
                                        : most_row_tiles(job.rows, job.experts, 64, job.ends != nullptr);
    if (across > (int64_t)0xFFFFFFFF / 256 / down) return kGridTooLarge;
    hipLaunchKernelGGL((product_any_kernel<T, AT, BT, K, TO>), dim3((unsigned)(across * down)), dim3(256), 0,
                       (hipStream_t)stream, job);
    return (int)hipGetLastError();
}

template <class T, bool QX, int NT, int MT, class TO>
int few(const GroupedJob& job, void* stream) {
    const int64_t across = (job.inner + 16 * MT - 1) / (16 * MT);
    const int64_t down = most_row_tiles(job.rows, job.experts, 16 * NT, job.ends != nullptr);
    if (across > (int64_t)0xFFFFFFFF / (64 * kFewWaves) / down) return kGridTooLarge;
    hipLaunchKernelGGL((product_few_kernel<T, QX, NT, MT, TO>), dim3((unsigned)(across * down)),
                       dim3(64 * kFewWaves), 0, (hipStream_t)stream, job);
    return (int)hipGetLastError();
}

}  // namespace

int launch_grouped_mm(const GroupedJob& job, bool transposed, bool bf16out, void* stream) {
    if (transposed)
        return bf16out ? any<Bf16, true, false, kProduct, uint16_t>(job, stream)
                       : any<Bf16, true, false, kProduct, float>(job, stream);
    return bf16out ? any<Bf16, false, false, kProduct, uint16_t>(job, stream)
                   : any<Bf16, false, false, kProduct, float>(job, stream);
}

int launch_grouped_wgrad(const GroupedJob& job, bool bf16out, void* stream) {
    return bf16out ? any<Bf16, true, true, kGradient, uint16_t>(job, stream)
                   : any<Bf16, true, true, kGradient, float>(job, stream);
}

int launch_gemm_int8(const GroupedJob& job, bool bf16x, bool bf16out, void* stream) {
    if (bf16x)
        return bf16out ? few<Int8, true, 1, 1, uint16_t>(job, stream) : few<Int8, true, 1, 1, float>(job, stream);
    return bf16out ? any<Int8, false, false, kProduct, uint16_t>(job, stream)
                   : any<Int8, false, false, kProduct, float>(job, stream);
}

}  // namespace tsenor
