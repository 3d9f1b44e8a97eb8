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

// This lane's part of one block of a bf16 row (entries 16q .. and 64+16q .. of
// the 128 at k0), quantised; the four lanes that hold the block share its scale.
__device__ __forceinline__ i32x8 quant_fragment(const uint16_t* row, int64_t k0, int64_t k, bool vec,
                                                int q, int* s) {
    Eight<uint16_t> v[4];
    uint32_t m = 0u;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        v[p].load(row, k0 + 16 * q + 64 * (p >> 1) + 8 * (p & 1), k, vec);
        m = max(m, v[p].magnitude());
    }
    if (__any(m >= kSpecial)) {
        m = 0u;
#pragma unroll
        for (int p = 0; p < 4; ++p) m = max(m, v[p].finite_only());
    }
    m = max(m, (uint32_t)__shfl_xor(m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor(m, 32, 64));
    *s = scale_exponent(m);
    const float inv = inverse_scale(*s);
    const u32x2 a = v[0].quantised(inv), b = v[1].quantised(inv), c = v[2].quantised(inv), d = v[3].quantised(inv);
    return i32x8{(int)a.x, (int)a.y, (int)b.x, (int)b.y, (int)c.x, (int)c.y, (int)d.x, (int)d.y};
}

// Few tokens (n <= 16 NT): reading A bounds the product, so a workgroup owns 16 MT rows of A
// and each of its eight waves a stretch of k, with the loads of kAhead blocks in flight
// (stretches, not blocks in turn: the workgroup then reads whole rows at a time, over all
// memory channels); the waves' sums meet in LDS, in wave order.  QX: X is bf16 and quantised
// on the way, by each workgroup for itself between its loads of A.  One quantised token,
// 28672 x 8192: 147 MB in 35 us, 4.2 TB/s (29 us with A in the last-level cache), from bf16
// 50; 4096 x 4096: 5 us, of which some 2 are the launch, from bf16 7.5.
constexpr int kFewWaves = 8;

template <int NT, int MT, bool QX, class TY>
__global__ __launch_bounds__(64 * kFewWaves) void spmm24_fp8_few_kernel(
    const void* __restrict__ X, const uint8_t* __restrict__ xs, int64_t n, int64_t ldx, bool xvec,
    const uint8_t* __restrict__ values, const uint32_t* __restrict__ meta,
    const uint8_t* __restrict__ scales, int64_t m, int64_t k, TY* __restrict__ Y, int64_t ldy,
    bool yvec) {
    constexpr int kAhead = QX ? 2 : NT * MT >= 4 ? 2 : 4;  // divides 4
    __shared__ f32x4 sums[kFewWaves][MT * NT][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t mt = (m + 16 * MT - 1) / (16 * MT);
    const int64_t m0 = blockIdx.x % mt * (16 * MT), n0 = blockIdx.x / mt * (16 * NT);
    const int kb = (int)((k + 127) / 128);
    int64_t row[MT], col[NT];
#pragma unroll
    for (int a = 0; a < MT; ++a) row[a] = min(m0 + 16 * a + l16, m - 1);
#pragma unroll
    for (int j = 0; j < NT; ++j) col[j] = min(n0 + 16 * j + l16, n - 1);
    const uint8_t* srow = scales + (m0 >> 7) * kb;  // 16 MT rows lie in one block of 128
    f32x4 acc[MT][NT];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[a][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int tend = (int)((int64_t)kb * (wave + 1) / kFewWaves);
    for (int t0 = (int)((int64_t)kb * wave / kFewWaves); t0 < tend; t0 += 4) {
        u32x4 own[MT];
        uint32_t idx[MT][4];
#pragma unroll
        for (int a = 0; a < MT; ++a)
            own[a] = *reinterpret_cast<const u32x4*>(meta + (row[a] * kb + min(t0 + q, tend - 1)) * 4);
#pragma unroll
        for (int p = 0; p < 4; p += kAhead) {
            if (p > 0 && t0 + p >= tend) break;
            i32x4 av[kAhead][MT];
            int sa[kAhead], sx[kAhead][NT];
            i32x8 bv[kAhead][NT];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int t = min(t0 + p + u, tend - 1);  // behind the end: loaded, not used
                sa[u] = srow[t];
#pragma unroll
                for (int a = 0; a < MT; ++a)
                    av[u][a] = *reinterpret_cast<const i32x4*>(values + (row[a] * kb + t) * 64 + 16 * q);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if constexpr (QX) {
                        bv[u][j] = quant_fragment(static_cast<const uint16_t*>(X) + col[j] * ldx, 128 * (int64_t)t,
                                                  k, xvec, q, &sx[u][j]);
                        sx[u][j] += 127;
                    } else {
                        const uint8_t* x = static_cast<const uint8_t*>(X) + col[j] * ldx + 128 * (int64_t)t + 16 * q;
                        bv[u][j] = join(*reinterpret_cast<const u32x4*>(x), *reinterpret_cast<const u32x4*>(x + 64));
                        sx[u][j] = xs[t * n + col[j]];
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);  // all loads first
            if (p == 0)
#pragma unroll
                for (int a = 0; a < MT; ++a) words_of_blocks(own[a], idx[a]);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (t0 + p + u >= tend) break;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float f = scale_product(sa[u], sx[u][j]);
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        f32x4 d = {0.f, 0.f, 0.f, 0.f};
                        d = __builtin_amdgcn_smfmac_f32_16x16x128_fp8_fp8(av[u][a], bv[u][j], d, (int)idx[a][p + u], 0, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[a][j][i] = __builtin_fmaf(d[i], f, acc[a][j][i]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[wave][a * NT + j][lane] = acc[a][j];
    __syncthreads();
    for (int u = tid; u < MT * NT * 64; u += 64 * kFewWaves) {
        f32x4 v = sums[0][u >> 6][u & 63];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += sums[w][u >> 6][u & 63];
        const int l = u & 63, j = (u >> 6) % NT, a = (u >> 6) / NT;
        const int64_t c = n0 + 16 * j + (l & 15);
        if (c < n) store4(Y + c * ldy, m0 + 16 * a + 4 * (l >> 4), m, yvec, v);
    }
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

// ---- tiled products -----------------------------------------------------------
//
// A workgroup of WM x WN waves owns TM x TN of the output, a wave (TM / WM) x
// (TN / WN) in tiles of 32 x 32, and walks k in blocks of 128.  Operands reach LDS by
// direct loads (no register staging) into a ring of R buffers filled R - 1 steps ahead.
// Rows keep their 16-byte chunks swizzled so that the 16 rows of one pass of a 16-byte
// LDS read hit 16 different bank groups: rows of 128 bytes keep chunk c at
// c ^ ((r >> 1) & 7), rows of 64 bytes at c ^ ((r >> 2) & 3).  Rows behind an operand's
// end repeat its last row; nothing of them is stored.

constexpr int64_t kMaxRow = int64_t(1) << 23;  // bytes of a row: offsets inside a tile fit 32 bits

// Operand layout of the 32 x 32 x 64 instructions, lane l, h = l / 32 (probed like
// the 16 x 16 x 128 one): A row l % 32 with entries 32h .. 32h+31 of a 2:4 operand's
// 64; B column l % 32 with entries 16h .. 16h+15 and 32+16h .. 32+16h+15; D column l % 32,
// rows 8 i0 + 4h + i1 in register 4 i0 + i1.  The dense instruction takes any order of
// the entries that is the same for both operands.

// 2^e for e <= 127; 0 below 2^-126.
__device__ __forceinline__ float power(int e) { return bits_float(e < -126 ? 0u : (uint32_t)(127 + e) << 23); }

// Y = X A^T (A on the rows of the instruction).  8192 x 28672 x 8192 in 1.39 to 1.48 ms, by
// the card's clock: 2.6 to 2.8 PFLOP/s dense-equivalent, of 8.3 that the instruction reaches
// in registers.  Neither the matrix cores (1024 of some 3300 cycles a step) nor the VALU (160
// instructions a wave) nor L2 bound it alone: the eight waves of the one workgroup that fits a CU go through the same phases (wait,
// LDS reads, multiply) together, and the clock is at 2 GHz under the load.
template <int TM, int TN, int WM, int WN, int R, class TY>
__global__ __launch_bounds__(64 * WM * WN) void spmm24_fp8_tile_kernel(
    const uint8_t* __restrict__ X, const uint8_t* __restrict__ xs, int64_t n, int64_t ldx,
    const uint8_t* __restrict__ values, const uint32_t* __restrict__ meta,
    const uint8_t* __restrict__ scales, int64_t m, int64_t k, TY* __restrict__ Y, int64_t ldy,
    bool yvec) {
    constexpr int W = WM * WN, TA = TM / WM / 32, TB = TN / WN / 32;
    // direct loads of a wave per step: X, values and as many of metadata, one of scales
    constexpr int QX = TN / 8 / W, QA = TM / 16 / W;
    static_assert(QX * 8 * W == TN && QA * 16 * W == TM && TN / 64 < W, "tile");
    struct Buffer {
        u32x4 x[TN * 8];
        u32x4 a[TM * 4];
        uint32_t meta[TM * 4];
        uint32_t scale[TN + 64];  // of the X rows; of the blocks of A rows (the first two)
    };
    __shared__ Buffer ring[R];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, h = lane >> 5, l32 = lane & 31;
    int64_t tm, tn;
    tile_of(blockIdx.x, (m + TM - 1) / TM, (n + TN - 1) / TN, tm, tn);
    const int64_t m0 = tm * TM, n0 = tn * TN, kb = (k + 127) / 128;
    const int steps = (int)kb;

    // rows behind the operands' ends, from the tile's first row
    const int xlast = (int)min(n - 1 - n0, (int64_t)TN), alast = (int)min(m - 1 - m0, (int64_t)TM);
    const uint8_t *xbase = X + n0 * ldx, *abase = values + m0 * (kb * 64);
    const uint8_t* mbase = reinterpret_cast<const uint8_t*>(meta + m0 * (kb * 4));
    // the first waves bring 64 X rows' scales each, the others all the same 64 (of A's blocks)
    const bool xw = wave < TN / 64;
    const uint8_t* sbase = xw ? xs + n0 : scales + (m0 >> 7) * kb;
    const int64_t sstep = xw ? n : 1;
    const int sdst = 64 * min(wave, TN / 64);

    f32x16 acc[TA][TB];
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

    // Each column's sums are held in units of 2^unit[b]: the scale product of the last block
    // that went in.
    int unit[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) unit[b] = 0;

    // load number j of step t into `buf` (behind the last step: the last step again, into a
    // buffer that nobody reads any more)
    constexpr int kLoads = QX + 2 * QA + 1;
    auto load = [&](int j, int t, Buffer& buf) {
        const int64_t s = t < steps ? t : steps - 1;
        const int l = lane;
        if (j < QX) {
            const int r = 8 * (wave * QX + j) + (l >> 3), c = l & 7;
            dma16(xbase + 128 * s, __umul24(min(r, xlast), (uint32_t)ldx) + 16 * (c ^ ((r >> 1) & 7)),
                  lds_offset(buf.x + 64 * (wave * QX + j)));
        } else if (j < QX + 2 * QA) {
            const int i = (j - QX) >> 1, r = 16 * (wave * QA + i) + (l >> 2), c = l & 3;
            const uint32_t row = __umul24(min(r, alast), (uint32_t)kb);
            if (((j - QX) & 1) == 0)
                dma16(abase + 64 * s, 64 * row + 16 * (c ^ ((r >> 2) & 3)), lds_offset(buf.a + 64 * (wave * QA + i)));
            else
                dma4(mbase + 16 * s, 16 * row + 4 * c, lds_offset(buf.meta + 64 * (wave * QA + i)));
        } else {
            const uint32_t so = xw ? min(64 * wave + l, xlast)
                                   : min(l & (TM / 128 > 1 ? 1 : 0), (int)(((m - 1) >> 7) - (m0 >> 7))) * (uint32_t)kb;
            dma_byte(sbase + s * sstep, so, lds_offset(buf.scale + sdst));
        }
    };
    // part a of TA of the loads of step t: spread over a step, they do not stall all waves on
    // the address unit at once (8192 x 28672 x 8192: 1610 -> 1555 us); with two buffers they are
    // needed in the next step and go out first (2048 x 4096 x 4096: 43 us against 49)
    auto load_part = [&](int a, int t, Buffer& buf) {
        constexpr int kParts = R > 2 ? TA : 1;
        if (a >= kParts) return;
#pragma unroll
        for (int j = a * kLoads / kParts; j < (a + 1) * kLoads / kParts; ++j) load(j, t, buf);
    };
    i32x8 bv[2][TB];
    i32x4 av[2][2];
    int idx[2][2];
    int u[TB];  // the block's scale product, as the sum of both bytes
    auto read_a = [&](int a, const Buffer& buf) {  // 32 rows of A into the set a & 1
        const int l = lane, lh = l >> 5, lr = l & 31;
        const int r = (TM / WM) * wm + 32 * a + lr, sw = (lr >> 2) & 3;
#pragma unroll
        for (int kc = 0; kc < 2; ++kc) {
            av[a & 1][kc] = __builtin_bit_cast(i32x4, buf.a[4 * r + ((2 * kc + lh) ^ sw)]);
            idx[a & 1][kc] = (int)buf.meta[4 * r + 2 * kc + lh];
        }
    };
    // Step t up to its first operands.
    auto begin = [&](const Buffer& buf) {
        // this step's loads have landed when at most the next R - 2 steps' are outstanding,
        // and this wave's LDS reads of the step before are done; after the barrier that holds
        // for all waves, so the buffer that step t + R - 1 fills (during this one) is free
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((R - 2) * kLoads) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const int l = lane, lh = l >> 5, lr = l & 31;
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int r = (TN / WN) * wn + 32 * b + lr, sw = (lr >> 1) & 7;
            u[b] = (int)buf.scale[r] + (int)buf.scale[TN + (TM > 128 ? wm : 0)];
#pragma unroll
            for (int kc = 0; kc < 2; ++kc)
                bv[kc][b] = join(buf.x[8 * r + ((4 * kc + lh) ^ sw)], buf.x[8 * r + ((4 * kc + 2 + lh) ^ sw)]);
        }
        read_a(0, buf);
    };
    // The sums change to this block's unit and the block is added in place: 16
    // multiplications a tile, where a fresh partial tile takes 16 clears and 16 multiply-adds.
    // No sum passes 2^60 times what its largest block can hold.
    auto add_near = [&](int t, const Buffer& buf, Buffer& free) {
        float f[TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            f[b] = power(unit[b] - u[b]);
            unit[b] = u[b];
        }
#pragma unroll
        for (int a = 0; a < TA; ++a) {
            if (R == 2) load_part(a, t + R - 1, free);
            if (a + 1 < TA) read_a(a + 1, buf);
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[a][b][e] *= f[b];
#pragma unroll
            for (int kc = 0; kc < 2; ++kc)
#pragma unroll
                for (int b = 0; b < TB; ++b)
                    acc[a][b] = __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(av[a & 1][kc], bv[kc][b], acc[a][b],
                                                                            idx[a & 1][kc], 0, 0);
            if (R > 2) load_part(a, t + R - 1, free);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Any block: the sums keep the larger unit, and the block is summed apart and scaled down.
    auto add_far = [&](int t, const Buffer& buf, Buffer& free) {
        float f[TB], g[TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int to = max(unit[b], u[b]);
            f[b] = power(unit[b] - to);
            g[b] = power(u[b] - to);
            unit[b] = to;
        }
#pragma unroll
        for (int a = 0; a < TA; ++a) {
            if (a + 1 < TA) read_a(a + 1, buf);
            load_part(a, t + R - 1, free);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                f32x16 d;
#pragma unroll
                for (int e = 0; e < 16; ++e) d[e] = 0.f;
#pragma unroll
                for (int kc = 0; kc < 2; ++kc)
                    d = __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(av[a & 1][kc], bv[kc][b], d, idx[a & 1][kc], 0, 0);
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[a][b][e] = __builtin_fmaf(d[e], g[b], acc[a][b][e] * f[b]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
#pragma unroll
    for (int t = 0; t < R - 1; ++t)
#pragma unroll
        for (int j = 0; j < kLoads; ++j) load(j, t, ring[t]);
    // Whether all blocks of each of the wave's columns are within 2^60 of each other.  (The
    // waves stay in step: one barrier a step in either loop.)
    bool near = true;
    {
        const uint8_t* as = scales + ((m0 + (TM / WM) * wm) >> 7 < (m + 127) >> 7 ? (m0 + (TM / WM) * wm) >> 7 : m0 >> 7) * kb;
        const uint8_t* x = xs + min(n0 + (TN / WN) * wn + (lane & (TN / WN - 1)), n - 1);
        int lo = 1 << 16, hi = 0;
#pragma unroll 16
        for (int t = 0; t < steps; ++t) {
            const int v = (int)x[t * n] + (int)as[t];
            lo = min(lo, v);
            hi = max(hi, v);
        }
        near = __all(hi - lo <= 60);
    }
    int cur = 0;
    const auto next_of = [](int v) { return v == R - 1 ? 0 : v + 1; };
    if (near) {
        for (int t = 0; t < steps; ++t, cur = next_of(cur)) {
            begin(ring[cur]);
            add_near(t, ring[cur], ring[cur == 0 ? R - 1 : cur - 1]);
        }
    } else {
        for (int t = 0; t < steps; ++t, cur = next_of(cur)) {
            begin(ring[cur]);
            add_far(t, ring[cur], ring[cur == 0 ? R - 1 : cur - 1]);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int b = 0; b < TB; ++b) {
        const int64_t col = n0 + (TN / WN) * wn + 32 * b + l32;
        if (col >= n) continue;
        TY* y = Y + col * ldy;
#pragma unroll
        for (int a = 0; a < TA; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __builtin_ldexpf(acc[a][b][4 * i + e], unit[b] - 254);
                store4(y, m0 + (TM / WM) * wm + 32 * a + 8 * i + 4 * h, m, yvec, v);
            }
    }
}

// C = A B^T (B on the rows of the instruction); the scaled instruction applies both
// operands' scales and adds in place.
template <int TM, int TN, int WM, int WN, int R, class TC>
__global__ __launch_bounds__(64 * WM * WN) void gemm_fp8_tile_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ as, int64_t p,
    const uint8_t* __restrict__ B, const uint8_t* __restrict__ bs, int64_t qn, int64_t kb,
    const uint32_t* __restrict__ mask, TC* __restrict__ C, int64_t ldc, bool cvec) {
    constexpr int W = WM * WN, TA = TM / WM / 32, TB = TN / WN / 32;
    constexpr int QB = TM / 8 / W, QA = TN / 8 / W;
    static_assert(QB * 8 * W == TM && QA * 8 * W == TN && (TM + TN) / 64 <= W, "tile");
    struct Buffer {
        u32x4 b[TM * 8];  // rows of B (columns of C)
        u32x4 a[TN * 8];
        uint32_t scale[TM + TN];
    };
    __shared__ Buffer ring[R];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, h = lane >> 5, l32 = lane & 31;
    int64_t tm, tn;
    tile_of(blockIdx.x, (qn + TM - 1) / TM, (p + TN - 1) / TN, tm, tn);
    const int64_t m0 = tm * TM, n0 = tn * TN;
    const int steps = (int)kb;
    const int blast = (int)min(qn - 1 - m0, (int64_t)TM), alast = (int)min(p - 1 - n0, (int64_t)TN);
    const uint8_t *bbase = B + m0 * (kb * 128), *abase = A + n0 * (kb * 128);
    // each wave brings 64 rows' scales, of B first (waves left over: of the last 64 again)
    const int sgroup = min(wave, (TM + TN) / 64 - 1);
    const bool bw = sgroup < TM / 64;
    const uint8_t* sbase = bw ? bs + m0 : as + n0;
    const int64_t sstep = bw ? qn : p;
    const int srow = 64 * (bw ? sgroup : sgroup - TM / 64);

    f32x16 acc[TA][TB];
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

    auto issue = [&](int t, Buffer& buf) {
        const int64_t s = t < steps ? t : steps - 1;
        const int l = lane;
        const uint32_t ld = (uint32_t)(kb * 128);
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int r = 8 * (wave * QB + j) + (l >> 3), c = 16 * ((l & 7) ^ ((r >> 1) & 7));
            dma16(bbase + 128 * s, __umul24(min(r, blast), ld) + c, lds_offset(buf.b + 64 * (wave * QB + j)));
        }
#pragma unroll
        for (int j = 0; j < QA; ++j) {
            const int r = 8 * (wave * QA + j) + (l >> 3), c = 16 * ((l & 7) ^ ((r >> 1) & 7));
            dma16(abase + 128 * s, __umul24(min(r, alast), ld) + c, lds_offset(buf.a + 64 * (wave * QA + j)));
        }
        dma_byte(sbase + s * sstep, min(srow + l, bw ? blast : alast), lds_offset(buf.scale + 64 * sgroup));
    };
    auto step = [&](int t, Buffer& buf, Buffer& next) {  // as in the product above
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((R - 2) * (QB + QA + 1)) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        issue(t + R - 1, next);
        int sn[TB];
        i32x8 nv[2][TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int r = (TN / WN) * wn + 32 * b + l32, sw = (l32 >> 1) & 7;
            sn[b] = (int)buf.scale[TM + r];
#pragma unroll
            for (int kc = 0; kc < 2; ++kc)
                nv[kc][b] = join(buf.a[8 * r + ((4 * kc + h) ^ sw)], buf.a[8 * r + ((4 * kc + 2 + h) ^ sw)]);
        }
        i32x8 mv[2][2];
        int sm[2];
        auto read_b = [&](int a) {
            const int r = (TM / WM) * wm + 32 * a + l32, sw = (l32 >> 1) & 7;
            sm[a & 1] = (int)buf.scale[r];
#pragma unroll
            for (int kc = 0; kc < 2; ++kc)
                mv[a & 1][kc] = join(buf.b[8 * r + ((4 * kc + h) ^ sw)], buf.b[8 * r + ((4 * kc + 2 + h) ^ sw)]);
        };
        read_b(0);
#pragma unroll
        for (int a = 0; a < TA; ++a) {
            if (a + 1 < TA) read_b(a + 1);
#pragma unroll
            for (int kc = 0; kc < 2; ++kc)
#pragma unroll
                for (int b = 0; b < TB; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        mv[a & 1][kc], nv[kc][b], acc[a][b], 0, 0, 0, sm[a & 1], 0, sn[b]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (steps > 0)
#pragma unroll
        for (int t = 0; t < R - 1; ++t) issue(t, ring[t]);
    int cur = 0;
    for (int t = 0; t < steps; ++t) {
        step(t, ring[cur], ring[cur == 0 ? R - 1 : cur - 1]);
        cur = cur == R - 1 ? 0 : cur + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int64_t wpr = (qn + 31) / 32;
#pragma unroll
    for (int b = 0; b < TB; ++b) {
        const int64_t col = n0 + (TN / WN) * wn + 32 * b + l32;
        if (col >= p) continue;
        TC* c = C + col * ldc;
#pragma unroll
        for (int a = 0; a < TA; ++a) {
            const int64_t c0 = m0 + (TM / WM) * wm + 32 * a;  // a multiple of 32: one mask word
            if (c0 >= qn) continue;
            const uint32_t keep = mask != nullptr ? mask[col * wpr + (c0 >> 5)] : 0xFFFFFFFFu;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = (keep >> (8 * i + 4 * h + e)) & 1u ? acc[a][b][4 * i + e] : 0.f;
                store4(c, c0 + 8 * i + 4 * h, qn, cvec, v);
            }
        }
    }
}

// The same product for many 256 x 256 tiles.  A step is half a block (64 entries): rows of
// 64 bytes, four chunks kept at c ^ ((r >> 2) & 3), which leaves room for four buffers.
// The operands of the next step's first instructions are read while this step's last ones
// run, so the barrier that publishes the next buffer stands in the middle of a step, where
// no wave waits for LDS.  The matrix cores are busy 64% of the time (51% with whole blocks
// per step and the barrier at its start); the clock falls from 1.94 to 1.76 GHz with it, so
// that the power limit takes back most of the gain: 8192^3 504 -> 475 us on one card, 2.3
// PFLOP/s (445 to 450 on others, where a dense library product takes 360).  Four
// waves of 128 x 128 measured 490 us; smaller tiles are slower in this form (128 x 128 at
// 8192 x 4096 x 8192: 352 us against 290).
template <int TM, int TN, int WM, int WN, int R, class TC>
__global__ __launch_bounds__(64 * WM * WN) void gemm_fp8_wide_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ as, int64_t p,
    const uint8_t* __restrict__ B, const uint8_t* __restrict__ bs, int64_t qn, int64_t kb,
    const uint32_t* __restrict__ mask, TC* __restrict__ C, int64_t ldc, bool cvec) {
    constexpr int W = WM * WN, TA = TM / WM / 32, TB = TN / WN / 32;
    // direct loads of a wave per step: of B, of A, and of 64 rows' scales
    constexpr int QB = TM / 16 / W, QA = TN / 16 / W, G = (TM + TN) / 64, QS = (G + W - 1) / W;
    static_assert(QB * 16 * W == TM && QA * 16 * W == TN && R >= 3, "tile");
    struct Buffer {
        u32x4 b[TM * 4];  // rows of B (columns of C)
        u32x4 a[TN * 4];
        uint32_t scale[TM + TN];
    };
    __shared__ Buffer ring[R];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, h = lane >> 5, l32 = lane & 31;
    int64_t tm, tn;
    tile_of(blockIdx.x, (qn + TM - 1) / TM, (p + TN - 1) / TN, tm, tn);
    const int64_t m0 = tm * TM, n0 = tn * TN;
    const int steps = 2 * (int)kb;
    const int blast = (int)min(qn - 1 - m0, (int64_t)TM), alast = (int)min(p - 1 - n0, (int64_t)TN);
    const uint8_t *bbase = B + m0 * (kb * 128), *abase = A + n0 * (kb * 128);
    f32x16 acc[TA][TB];
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

    // load number j of step t into its buffer (behind the last step: the last step again,
    // into a buffer that nobody reads any more)
    constexpr int kLoads = QB + QA + QS, kLate = TA > 1 ? kLoads / 2 : 0;
    auto load = [&](int j, int t, Buffer& buf) {
        const int64_t s = t < steps ? t : steps - 1;
        const int l = lane;
        const uint32_t ld = (uint32_t)(kb * 128);
        if (j < QB) {
            const int r = 16 * (wave * QB + j) + (l >> 2), c = 16 * ((l & 3) ^ ((r >> 2) & 3));
            dma16(bbase + 64 * s, __umul24(min(r, blast), ld) + c, lds_offset(buf.b + 64 * (wave * QB + j)));
        } else if (j < QB + QA) {
            const int i = wave * QA + j - QB, r = 16 * i + (l >> 2), c = 16 * ((l & 3) ^ ((r >> 2) & 3));
            dma16(abase + 64 * s, __umul24(min(r, alast), ld) + c, lds_offset(buf.a + 64 * i));
        } else {
            // 64 rows' scales, of B first (waves left over: of the last 64 again)
            const int g = min(wave + (j - QB - QA) * W, G - 1);
            const bool ofb = g < TM / 64;
            const int64_t rows = ofb ? qn : p;
            dma_byte((ofb ? bs + m0 : as + n0) + (s >> 1) * rows,
                     min(64 * (ofb ? g : g - TM / 64) + l, ofb ? blast : alast), lds_offset(buf.scale + 64 * g));
        }
    };
    i32x8 nv[2][TB], mv[2];
    int sn[2][TB], sm[2];
    auto read_b = [&](int a, const Buffer& buf) {  // 32 rows of B into the set a & 1
        const int l = lane, r = (TM / WM) * wm + 32 * a + (l & 31), c = (l >> 5) ^ ((l >> 2) & 3);
        sm[a & 1] = (int)buf.scale[r];
        mv[a & 1] = join(buf.b[4 * r + c], buf.b[4 * r + (c ^ 2)]);
    };
    auto read_a = [&](int set, const Buffer& buf) {
        const int l = lane, c = (l >> 5) ^ ((l >> 2) & 3);
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int r = (TN / WN) * wn + 32 * b + (l & 31);
            sn[set][b] = (int)buf.scale[TM + r];
            nv[set][b] = join(buf.a[4 * r + c], buf.a[4 * r + (c ^ 2)]);
        }
    };
    // Step t, whose first operands are in registers (set t & 1).  The loads of step
    // t + R - 1 go out one by one between the matrix instructions (all at once they would
    // stall every wave on the address unit): the first ones after the barrier, the last
    // kLate in the first half of the next step.
    auto step = [&](int t, int set, const Buffer& buf, const Buffer& next, Buffer& early, Buffer& late) {
#pragma unroll
        for (int a = 0; a < TA; ++a) {
            if (a == TA / 2) {
                // the next step's loads have landed, and every wave is past the step before
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"((R - 3) * kLoads) : "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
            }
            if (a + 1 < TA) {
                read_b(a + 1, buf);
            } else {
                read_a(set ^ 1, next);
                if (TA > 1) read_b(0, next);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    mv[a & 1], nv[set][b], acc[a][b], 0, 0, 0, sm[a & 1], 0, sn[set][b]);
                __builtin_amdgcn_sched_barrier(0);
                constexpr int kSlots = TA > 1 ? TA / 2 * TB : TB;  // of a half step
                const int slot = (a >= TA / 2 ? a - TA / 2 : a) * TB + b;
                if (a >= TA / 2) {
#pragma unroll
                    for (int j = slot; j < kLoads - kLate; j += kSlots) load(j, t + R - 1, early);
                } else {
#pragma unroll
                    for (int j = slot; j < kLate; j += kSlots) load(kLoads - kLate + j, t + R - 2, late);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (TA == 1) read_b(0, next);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (steps > 0) {
#pragma unroll
        for (int t = 0; t < R - 1; ++t)
#pragma unroll
            for (int j = 0; j < (t == R - 2 ? kLoads - kLate : kLoads); ++j) load(j, t, ring[t]);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((R - 2) * kLoads - kLate) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        read_a(0, ring[0]);
        read_b(0, ring[0]);
        const auto inc = [](int v) { return v == R - 1 ? 0 : v + 1; };
        const auto dec = [](int v) { return v == 0 ? R - 1 : v - 1; };
        int cur = 0;
        for (int t = 0; t < steps; t += 2) {
            const int one = inc(cur), two = inc(one), last = dec(cur);
            step(t, 0, ring[cur], ring[one], ring[last], ring[dec(last)]);
            step(t + 1, 1, ring[one], ring[two], ring[cur], ring[last]);
            cur = two;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    const int64_t wpr = (qn + 31) / 32;
#pragma unroll
    for (int b = 0; b < TB; ++b) {
        const int64_t col = n0 + (TN / WN) * wn + 32 * b + l32;
        if (col >= p) continue;
        TC* c = C + col * ldc;
#pragma unroll
        for (int a = 0; a < TA; ++a) {
            const int64_t c0 = m0 + (TM / WM) * wm + 32 * a;  // a multiple of 32: one mask word
            if (c0 >= qn) continue;
            const uint32_t keep = mask != nullptr ? mask[col * wpr + (c0 >> 5)] : 0xFFFFFFFFu;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = (keep >> (8 * i + 4 * h + e)) & 1u ? acc[a][b][4 * i + e] : 0.f;
                store4(c, c0 + 8 * i + 4 * h, qn, cvec, v);
            }
        }
    }
}

int64_t tiles(int64_t a, int64_t b, int64_t ta, int64_t tb) { return ((a + ta - 1) / ta) * ((b + tb - 1) / tb); }

// The largest tile that leaves every CU a workgroup (256 x 256), or two of them (smaller
// tiles leave room for several on a CU): 0: 256 x 256, 1: 128 x 128, 2: 128 x 64, 3: 64 x 64.
// Measured (us, the product alone) for 0 / 1 / 2 / 3: 4096 x 11008 x 4096: 199 / 258 / 329 / 378;
// 2048 x 4096 x 4096: 51 / 46 / 62 / 71; 1000 x 4096 x 4096: 46 / 38 / 33 / 40; 300 x 4096 x 4096:
// 43 / 28 / 20 / 18; dense 4096 x 11008 over 4096: 208 / 227 / 290 / 327, 2048 x 2048 over 512: 18.4 /
// 10.6 / 9.9 / 11.0, 1024 x 1024 over 1001: 20.7 / 11.0 / 8.3 / 6.7.
int pick_tile(int64_t a, int64_t b) {
    if (tiles(a, b, 256, 256) >= 256) return 0;
    if (tiles(a, b, 128, 128) >= 512) return 1;
    return tiles(a, b, 128, 64) >= 512 ? 2 : 3;
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
    bool fits = true;
    const bool tiled = !bf16x && n > 64 && m >= 64 && ldx < kMaxRow && k < kMaxRow;
    if (tiled) {
        const auto go = [&](auto kernel, int tm, int tn, int waves) {
            fits = grid_fits(tiles(m, n, tm, tn), 64 * waves);
            if (!fits) return;
            hipLaunchKernelGGL(kernel, dim3((unsigned)tiles(m, n, tm, tn)), dim3(64 * waves), 0, stream,
                               static_cast<const uint8_t*>(X), xs, n, ldx, values, meta, scales, m, k, Y, ldy, yvec);
        };
        switch (pick_tile(m, n)) {
            case 0: go(spmm24_fp8_tile_kernel<256, 256, 2, 4, 3, TY>, 256, 256, 8); break;
            case 1: go(spmm24_fp8_tile_kernel<128, 128, 2, 2, 2, TY>, 128, 128, 4); break;
            case 2: go(spmm24_fp8_tile_kernel<128, 64, 2, 2, 3, TY>, 128, 64, 4); break;
            default: go(spmm24_fp8_tile_kernel<64, 64, 2, 2, 3, TY>, 64, 64, 4); break;
        }
        return fits ? (int)hipGetLastError() : kGridTooLarge;
    }
    const bool xvec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && ldx % 8 == 0;
    const auto few = [&](auto kernel, int nt, int mt) {
        const int64_t ny = (n + 16 * nt - 1) / (16 * nt), nx = (m + 16 * mt - 1) / (16 * mt);
        fits = grid_fits(nx * ny, 64 * kFewWaves);
        if (!fits) return;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(nx * ny)), dim3(64 * kFewWaves), 0, stream, X, xs, n,
                           ldx, xvec, values, meta, scales, m, k, Y, ldy, yvec);
    };
    // A fragment of X touches 16 rows for each fragment of A that it meets, so with more tokens
    // a workgroup takes more rows of A, as long as about 160 workgroups remain.  Measured (us)
    // with 16 / 32 / 64 rows: 64 tokens, 11008 x 4096: 28.1 / 22.2 / 15.9; 16 tokens: 11.6 / 11.0 /
    // 9.5; 1 token: 7.5 / 8.8 / 8.6; 64 tokens, 4096 x 11008: 25.3 / 28.3 / 34.1.
    const int rows = m >= 64 * 160 ? 4 : m >= 32 * 160 ? 2 : 1;
    if (bf16x) few(spmm24_fp8_few_kernel<1, 1, true, TY>, 1, 1);
    else if (n <= 4) few(spmm24_fp8_few_kernel<1, 1, false, TY>, 1, 1);
    else {
        const auto pick = [&](auto one, auto two, auto four, int nt) {
            if (rows == 4) few(four, nt, 4);
            else if (rows == 2) few(two, nt, 2);
            else few(one, nt, 1);
        };
#define FEW(NT) pick(spmm24_fp8_few_kernel<NT, 1, false, TY>, spmm24_fp8_few_kernel<NT, 2, false, TY>, \
                     spmm24_fp8_few_kernel<NT, 4, false, TY>, NT)
        if (n <= 16) FEW(1);
        else if (n <= 32) FEW(2);
        else if (n <= 48) FEW(3);
        else FEW(4);
#undef FEW
    }
    return fits ? (int)hipGetLastError() : kGridTooLarge;
}

template <class TC>
int gemm(const uint8_t* A, const uint8_t* as, int64_t p, const uint8_t* B, const uint8_t* bs,
         int64_t q, int64_t k, const uint32_t* mask, void* C, int64_t ldc, hipStream_t stream) {
    bool fits = true;
    if (p >= 64 && q >= 64 && k < kMaxRow) {
        const auto go = [&](auto kernel, int tm, int tn, int waves) {
            fits = grid_fits(tiles(q, p, tm, tn), 64 * waves);
            if (!fits) return;
            hipLaunchKernelGGL(kernel, dim3((unsigned)tiles(q, p, tm, tn)), dim3(64 * waves), 0, stream, A, as, p, B,
                               bs, q, (k + 127) / 128, mask, static_cast<TC*>(C), ldc, row4<TC>(C, ldc));
        };
        switch (pick_tile(q, p)) {
            case 0: go(gemm_fp8_wide_kernel<256, 256, 2, 4, 4, TC>, 256, 256, 8); break;
            case 1: go(gemm_fp8_tile_kernel<128, 128, 2, 2, 2, TC>, 128, 128, 4); break;
            case 2: go(gemm_fp8_tile_kernel<128, 64, 2, 2, 3, TC>, 128, 64, 4); break;
            default: go(gemm_fp8_tile_kernel<64, 64, 2, 2, 3, TC>, 64, 64, 4); break;
        }
        return fits ? (int)hipGetLastError() : kGridTooLarge;
    }
    const int64_t blocks = ((q + 63) / 64) * ((p + 63) / 64);
    if (!grid_fits(blocks, 256)) return kGridTooLarge;
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
