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

// Along the rows only: 16 lanes hold one block of 128 (8 entries each).  Bound by memory:
// 4096 x 11008 bf16 in 28 us (4.8 TB/s read and written; 25 us where the last-level cache still
// holds the input).  f32: 37 us.
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
    Eight<T> v;
    v.load(X + r * ldx, b * 128 + 8 * l, cols, vec);
    uint32_t m = v.magnitude();
    if (__any(m >= kSpecial)) m = v.finite_only();
    const int s = scale_exponent(max16(m));
    const u32x2 q = v.quantised(inverse_scale(s));
    *reinterpret_cast<u32x2*>(values + r * (blocks * 128) + b * 128 + 8 * l) = q;
    if (l == 0) scales[b * rows + r] = (uint8_t)(s + 127);
}

// Along the columns, and along the rows too when `values` is given: one
// workgroup per 128 x 128 tile, read once and kept in LDS.  A thread holds a part of one
// column (f32: 64 rows) or of two (bf16: 32 rows of a pair, one LDS word a row) in registers;
// the 8-bit columns leave through LDS, so that eight lanes write the 128 bytes of a column
// side by side (written by the threads that hold them, each store would touch 64 lines).
// Both ways, 4096 x 11008 bf16: 40 us, 4.6 TB/s (34 us with the input in the last-level cache);
// along the columns only 32.  f32, whose tile takes twice the LDS: 68 us, 4.0 TB/s; columns only 57.
template <class T>
__global__ __launch_bounds__(256) void quant_tile_kernel(const T* __restrict__ X, int64_t rows,
                                                         int64_t cols, int64_t ldx, bool vec,
                                                         uint8_t* __restrict__ values,
                                                         uint8_t* __restrict__ scales,
                                                         uint8_t* __restrict__ values_t,
                                                         uint8_t* __restrict__ scales_t) {
    constexpr bool kPairs = sizeof(T) == 2;
    constexpr int kLd = 128 + 16 / sizeof(T), kOut = 144;  // a tile row's elements, an output column's bytes
    constexpr int kParts = kPairs ? 4 : 2, kLen = 128 / kParts;
    __shared__ __attribute__((aligned(16))) T tile[128 * kLd];
    __shared__ uint32_t colmax[kParts][128];
    uint8_t* out = reinterpret_cast<uint8_t*>(tile);  // after the tile has been read
    static_assert(128 * kOut <= (int)sizeof(tile), "output columns fit the tile's place");
    const int64_t cblocks = (cols + 127) / 128, rblocks = (rows + 127) / 128;
    const int64_t rb = blockIdx.x / cblocks, cb = blockIdx.x - rb * cblocks;
    const int tid = threadIdx.x, l = tid & 15;
#pragma unroll 4
    for (int p = 0; p < 8; ++p) {
        const int lr = 16 * p + (tid >> 4);
        const int64_t r = rb * 128 + lr;
        Eight<T> v;
        if (r < rows) v.load(X + r * ldx, cb * 128 + 8 * l, cols, vec);
        else v.clear();
        v.store(&tile[lr * kLd + 8 * l]);
        if (values != nullptr) {  // uniform
            uint32_t m = v.magnitude();
            if (__any(m >= kSpecial)) m = v.finite_only();
            const int s = scale_exponent(max16(m));
            if (r < rows) {
                *reinterpret_cast<u32x2*>(values + r * (cblocks * 128) + cb * 128 + 8 * l) =
                    v.quantised(inverse_scale(s));
                if (l == 0) scales[cb * rows + r] = (uint8_t)(s + 127);
            }
        }
    }
    __syncthreads();
    const int c = kPairs ? 2 * (tid & 63) : tid & 127, part = kPairs ? tid >> 6 : tid >> 7;
    uint32_t w[kLen], m0 = 0u, m1 = 0u;
    u16x2 pairs = {0, 0};
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
        w[i] = *reinterpret_cast<const uint32_t*>(&tile[(kLen * part + i) * kLd + c]);
        if constexpr (kPairs) pairs = pair_max(pairs, w[i]);
        else m0 = max(m0, w[i] & 0x7FFFFFFFu);
    }
    if constexpr (kPairs) {
        m0 = (uint32_t)pairs[0] << 16;
        m1 = (uint32_t)pairs[1] << 16;
    }
    if (__any(max(m0, m1) >= kSpecial)) {
        m0 = m1 = 0u;
#pragma unroll
        for (int i = 0; i < kLen; ++i) {
            if constexpr (kPairs) {
                (void)finite_pair(&w[i]);  // NaN where it was not finite
                const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
                m0 = max(m0, lo < 0x7F80u ? lo << 16 : 0u);
                m1 = max(m1, hi < 0x7F80u ? hi << 16 : 0u);
            } else {
                m0 = max(m0, finite_one(&w[i]));
            }
        }
    }
    colmax[part][c] = m0;
    if constexpr (kPairs) colmax[part][c + 1] = m1;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < (kPairs ? 2 : 1); ++k) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < kParts; ++i) m = max(m, colmax[i][c + k]);
        const int s = scale_exponent(m);
        const float inv = inverse_scale(s);
        const auto entry = [&](int i) { return !kPairs ? w[i] : k ? w[i] & 0xFFFF0000u : w[i] << 16; };
#pragma unroll
        for (int v = 0; v < kLen; v += 16) {
            u32x4 q;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[e] = pack_words(entry(v + 4 * e), entry(v + 4 * e + 1), entry(v + 4 * e + 2), entry(v + 4 * e + 3), inv);
            *reinterpret_cast<u32x4*>(out + (c + k) * kOut + kLen * part + v) = q;
        }
        if (part == 0 && cb * 128 + c + k < cols) scales_t[rb * cols + cb * 128 + c + k] = (uint8_t)(s + 127);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = tid + 256 * i, col = u >> 3, chunk = 16 * (u & 7);
        if (cb * 128 + col < cols)
            *reinterpret_cast<u32x4*>(values_t + (cb * 128 + col) * (rblocks * 128) + rb * 128 + chunk) =
                *reinterpret_cast<const u32x4*>(out + col * kOut + chunk);
    }
}

// What a group's four mask bits ask for: in the low half the byte permutation that takes
// its first two kept values (0x0C: a zero byte for an unused slot), in bits 16..19 its
// metadata (unused slots point at a free position), in bit 31 whether more than two are kept.
__device__ __forceinline__ uint32_t group_entry(uint32_t bits) {
    const uint32_t rest = bits & (bits - 1u);
    const uint32_t p0 = bits ? (uint32_t)__builtin_ctz(bits) : 0u;
    const uint32_t p1 = rest ? (uint32_t)__builtin_ctz(rest) : (bits ? (p0 == 3u ? 2u : 3u) : 1u);
    return (bits ? p0 : 0x0Cu) | ((rest ? p1 : 0x0Cu) << 8) | ((p0 | (p1 << 2)) << 16) |
           ((rest & (rest - 1u)) ? 0x80000000u : 0u);
}
// Two groups' values (entries a and b of the table) as one word.
__device__ __forceinline__ uint32_t take_two(uint32_t a, uint32_t qa, uint32_t b, uint32_t qb) {
    // the selectors' upper bytes are the table's other fields: those bytes are not used
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(0u, qb, b & 0xFFFFu), __builtin_amdgcn_perm(0u, qa, a & 0xFFFFu),
                                 0x05040100u);
}

// One workgroup per 128 x 128 tile of one matrix.  The tile's kept entries
// give the one scale that both orientations share.  The rows are compressed from the
// registers that hold them (16 lanes a row, two groups each); for the columns the 8-bit
// numbers go to LDS, a thread turns 4 x 4 cells of them around with byte permutations, and
// the compressed columns leave through LDS as whole lines.  11008 x 4096 bf16 both ways: 48 us
// for 152 MB (42 with the input in the last-level cache; one way 33 to 37); some 1000 VALU
// instructions a thread keep it from the memory's rate.  8192 x 8192 f32: 80 us for 361 MB.  The
// compressed columns take the tile's place in LDS (19.5 KB in all against 29), which is worth 4 to 8%.
template <class T>
__global__ __launch_bounds__(256) void compress24_fp8_kernel(
    const T* __restrict__ W, int64_t stride, int64_t rows, int64_t cols, int64_t ld, bool vec,
    const uint32_t* __restrict__ mask, uint8_t* __restrict__ values, uint32_t* __restrict__ meta,
    uint8_t* __restrict__ scales, uint8_t* __restrict__ values_t, uint32_t* __restrict__ meta_t,
    uint8_t* __restrict__ scales_t, int* __restrict__ bad, int* __restrict__ bad_t) {
    constexpr int kLd = 132, kOut = 80;  // bytes of a tile row, of a compressed column
    __shared__ __attribute__((aligned(16))) uint8_t q8[128 * kLd];
    uint8_t* out = q8;  // the compressed columns and their metadata, once all have been taken
    uint16_t* out_meta = reinterpret_cast<uint16_t*>(q8 + 128 * kOut);
    static_assert(128 * (kOut + 16) <= (int)sizeof(q8), "columns fit the tile's place");
    __shared__ uint32_t bits[128][5];  // mask words of the tile's rows (padded against bank conflicts)
    __shared__ uint32_t wmax[4], table[16];
    const int64_t cblocks = (cols + 127) / 128, rblocks = (rows + 127) / 128;
    const int64_t per = rblocks * cblocks;
    const int64_t mat = blockIdx.x / per, t = blockIdx.x - mat * per;
    const int64_t rb = t / cblocks, cb = t - rb * cblocks;
    const int64_t wpr = (cols + 31) / 32;
    const int tid = threadIdx.x, l = tid & 15;
    W += mat * stride;
    mask += mat * rows * wpr;
    if (tid < 16) table[tid] = group_entry((uint32_t)tid);
    Eight<T> raw[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = rb * 128 + 16 * p + (tid >> 4);
        if (r < rows) raw[p].load(W + r * ld, cb * 128 + 8 * l, cols, vec);
        else raw[p].clear();
    }
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
    uint32_t m = 0u;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        raw[p].keep(bits[16 * p + (tid >> 4)][l >> 2] >> (8 * (l & 3)));
        m = max(m, raw[p].magnitude());
    }
    if (__any(m >= kSpecial)) {
        m = 0u;
#pragma unroll
        for (int p = 0; p < 8; ++p) m = max(m, raw[p].finite_only());
    }
    m = max16(m);
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor(m, d, 64));
    if ((tid & 63) == 0) wmax[tid >> 6] = m;
    __syncthreads();
    const int s = scale_exponent(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
    const float inv = inverse_scale(s);
    int over = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int lr = 16 * p + (tid >> 4);
        const int64_t r = rb * 128 + lr;
        const u32x2 q = raw[p].quantised(inv);
        if (values != nullptr) {  // uniform
            const uint32_t keep = bits[lr][l >> 2] >> (8 * (l & 3));
            const uint32_t g0 = table[keep & 15u], g1 = table[(keep >> 4) & 15u];
            over += (int)(g0 >> 31) + (int)(g1 >> 31);
            const uint32_t n0 = (g0 >> 16) & 15u, n1 = (g1 >> 16) & 15u;
            uint32_t word = (n0 | (n1 << 4)) << (8 * (l & 3));  // four lanes share a word
            word |= (uint32_t)__shfl_xor(word, 1, 64);
            word |= (uint32_t)__shfl_xor(word, 2, 64);
            if (r < rows) {
                const int64_t at = (mat * rows + r) * cblocks + cb;
                *reinterpret_cast<uint32_t*>(values + at * 64 + 4 * l) = take_two(g0, q.x, g1, q.y);
                if ((l & 3) == 0) meta[at * 4 + (l >> 2)] = word;
            }
        }
        if (values_t != nullptr) {
            *reinterpret_cast<uint32_t*>(&q8[lr * kLd + 8 * l]) = q.x;
            *reinterpret_cast<uint32_t*>(&q8[lr * kLd + 8 * l + 4]) = q.y;
        }
    }
    if (over && bad != nullptr) atomicAdd(bad, over);
    if (tid == 0) {
        if (scales != nullptr) scales[mat * per + rb * cblocks + cb] = (uint8_t)(s + 127);
        if (scales_t != nullptr) scales_t[mat * per + cb * rblocks + rb] = (uint8_t)(s + 127);
    }
    if (values_t == nullptr) return;
    __syncthreads();
    over = 0;
    const int cq = tid & 31, part = tid >> 5;  // four columns, 16 rows
    uint32_t v[4][2], mw[4] = {};
#pragma unroll
    for (int g2 = 0; g2 < 4; g2 += 2) {
        uint32_t col[2][4], entry[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t q[4], kept = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * part + 4 * (g2 + g) + i;
                q[i] = *reinterpret_cast<const uint32_t*>(&q8[r * kLd + 4 * cq]);
                kept |= ((bits[r][cq >> 3] >> (4 * (cq & 7))) & 15u) << (4 * i);
            }
            // bytes of four rows to bytes of four columns
            const uint32_t a = __builtin_amdgcn_perm(q[1], q[0], 0x05010400u);
            const uint32_t b = __builtin_amdgcn_perm(q[3], q[2], 0x05010400u);
            const uint32_t c = __builtin_amdgcn_perm(q[1], q[0], 0x07030602u);
            const uint32_t d = __builtin_amdgcn_perm(q[3], q[2], 0x07030602u);
            col[g][0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
            col[g][1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
            col[g][2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
            col[g][3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = (kept >> j) & 0x1111u;  // this column's bits, one in each nibble
                entry[g][j] = table[(x | (x >> 3) | (x >> 6) | (x >> 9)) & 15u];
                over += (int)(entry[g][j] >> 31);
                mw[j] |= ((entry[g][j] >> 16) & 15u) << (4 * (g2 + g));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j][g2 >> 1] = take_two(entry[0][j], col[0][j], entry[1][j], col[1][j]);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<u32x2*>(&out[(4 * cq + j) * kOut + 8 * part]) = u32x2{v[j][0], v[j][1]};
        out_meta[(4 * cq + j) * 8 + part] = (uint16_t)mw[j];
    }
    if (over && bad_t != nullptr) atomicAdd(bad_t, over);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int u = tid + 256 * i, c = u >> 2, chunk = 16 * (u & 3);
        if (cb * 128 + c < cols)
            *reinterpret_cast<u32x4*>(values_t + ((mat * cols + cb * 128 + c) * rblocks + rb) * 64 + chunk) =
                *reinterpret_cast<const u32x4*>(&out[c * kOut + chunk]);
    }
    if (tid < 128 && cb * 128 + tid < cols)
        *reinterpret_cast<u32x4*>(meta_t + ((mat * cols + cb * 128 + tid) * rblocks + rb) * 4) =
            *reinterpret_cast<const u32x4*>(&out_meta[tid * 8]);
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
    if (!grid_fits(values_t == nullptr ? (rows * cb + 15) / 16 : rb * cb, 256)) return kGridTooLarge;
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
    if (!grid_fits(blocks, 256)) return kGridTooLarge;
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
