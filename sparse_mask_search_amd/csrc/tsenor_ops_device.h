// tsenor_ops_device.h -- device helpers of the grouped and 8-bit integer
// products: matrix instructions, LDS tiles and their fragments, rows of experts.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor_fp8_device.h"
#include "tsenor_ops_internal.h"

namespace tsenor {
namespace ops {

using namespace fp8;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// One matrix instruction takes 64 bytes of the reduction (32 bf16 or 64 integers), 16 from each
// lane quarter q = lane / 16: A row lane % 16, B column lane % 16; result column lane % 16, rows
// 4 q .. 4 q + 3.  The 32 x 32 instructions, at the same rate, read and write twice as many bytes
// of sums for a product; under the card's power limit that costs clock.
struct Bf16 {
    static constexpr int kSize = 2;
    typedef f32x4 Sum;
    __device__ static __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
};
struct Int8 {
    static constexpr int kSize = 1;
    typedef i32x4 Sum;
    __device__ static __forceinline__ i32x4 mma(u32x4 a, u32x4 b, i32x4 c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c,
                                                     0, 0, 0);
    }
};

// LDS tiles of one step, 64 bytes of the reduction for `W` rows or columns, in chunks of 16
// bytes.  An operand that is contiguous along the reduction is kept by rows of 64 bytes, chunk c of
// row r at c ^ (-(r / 4) & 3).  A 16-byte read serves lanes 0-3, 12-15, 20-23 and 24-27 at once, then
// 4-11, 16-19 and 28-31, and so on (measured: c ^ (r / 4 & 3) conflicts); with lane % 16 the row and
// lane / 16 the chunk, these lie in different banks.  One that is contiguous along its columns
// (bf16) is kept as it lies, 32 rows of the reduction of W entries, and turned by the transposing
// read below; pairs of chunks are moved so that the eight rows of half such a read hit different banks.
__device__ __forceinline__ int row_slot(int r, int c) { return 4 * r + (c ^ (-(r >> 2) & 3)); }
template <int W>
__device__ __forceinline__ int turned_slot(int r, int c) {  // chunk c of reduction row r
    constexpr int kChunks = W / 8;
    const int f = W >= 128 ? (r & 3) | ((r >> 1) & 4) : ((r >> 1) & 1) | ((r >> 2) & 2);
    return kChunks * r + (c ^ (2 * f));
}

// Rows row0 .. row0 + 15: chunk q of row lane % 16.
__device__ __forceinline__ u32x4 row_fragment(const u32x4* tile, int row0, int lane) {
    return tile[row_slot(row0 + (lane & 15), lane >> 4)];
}
// The same of a column-contiguous tile.  ds_read_b64_tr_b16, for each 16 lanes: lane i gives the
// address of 4 entries, of row i / 4 and columns 4 (i % 4) ..; it receives column i of the four
// rows (probed).  Two such reads give a lane the eight reduction entries of its column.
template <int W>
__device__ __forceinline__ u32x4 turned_fragment(const u32x4* tile, int col0, int lane) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int i = lane & 15, row = 8 * (lane >> 4) + (i >> 2), chunk = (col0 >> 3) + ((i & 3) >> 1);
    const uint8_t* base = reinterpret_cast<const uint8_t*>(tile) + 8 * (i & 1);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + 16 * turned_slot<W>(row, chunk)));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + 16 * turned_slot<W>(row + 4, chunk)));
    const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
    return u32x4{a.x, a.y, b.x, b.y};
}

// A value that all lanes have, as the compiler has to know it for scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
    const u32x2 v = __builtin_bit_cast(u32x2, p);
    return __builtin_bit_cast(const uint8_t*, u32x2{(uint32_t)uniform((int)v.x), (uint32_t)uniform((int)v.y)});
}

constexpr int kMaxExperts = 1024;

// Where the rows of one tile lie.
struct RowTile {
    int expert;      // -1: rows of no expert
    int first, end;  // rows first .. min(first + tile, end) - 1
};

// Sum and maximum over the lanes up to each one, and each lane's value from the lane before (0 for the first): DPP
// moves along rows of 16 lanes, then each row's last value into the rows behind.
template <int CTRL, int ROWS>
__device__ __forceinline__ int from_lane(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, true);
}
__device__ __forceinline__ int sum_up_to(int v) {
    v += from_lane<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v += from_lane<0x112, 0xF>(v);
    v += from_lane<0x114, 0xF>(v);
    v += from_lane<0x118, 0xF>(v);
    v += from_lane<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3
    v += from_lane<0x143, 0xC>(v);  // row_bcast 31 into rows 2 and 3
    return v;
}
__device__ __forceinline__ int max_up_to(int v) {  // of values that are not negative
    v = max(v, from_lane<0x111, 0xF>(v));
    v = max(v, from_lane<0x112, 0xF>(v));
    v = max(v, from_lane<0x114, 0xF>(v));
    v = max(v, from_lane<0x118, 0xF>(v));
    v = max(v, from_lane<0x142, 0xA>(v));
    return max(v, from_lane<0x143, 0xC>(v));
}
__device__ __forceinline__ int lane_before(int v) { return from_lane<0x138, 0xF>(v); }  // wave_shr 1

// Where the rows of experts e0 .. e0 + 63 end, one expert a lane: the largest entry up to its own, within
// 0 .. rows (so that whatever `ends` holds, experts never share a row).  `before`: that of the expert
// before e0, or 0; behind the last expert it stays.
__device__ __forceinline__ int end_of_lane(const int* ends, int experts, int rows, int e0, int before) {
    const int e = e0 + (threadIdx.x & 63);
    return max(max_up_to(e < experts ? min(max(ends[e], 0), rows) : 0), before);
}
// Rows first .. end - 1 of one expert, the same in all lanes.
__device__ __forceinline__ void rows_of(const int* ends, int rows, int expert, int* first, int* end) {
    int last = 0;
    for (int e0 = 0;; e0 += 64) {
        const int hi = end_of_lane(ends, expert + 1, rows, e0, last);
        if (expert < e0 + 64) {
            *first = expert == e0 ? last : __builtin_amdgcn_readlane(hi, expert - e0 - 1);
            *end = __builtin_amdgcn_readlane(hi, expert - e0);
            return;
        }
        last = __builtin_amdgcn_readlane(hi, 63);
    }
}

// Tiles of `size` rows, expert after expert, then those of no expert: tile t, if there is one (64 experts at a
// time, one a lane).  Every lane gets the same answer.
__device__ __forceinline__ bool row_tile(const int* ends, int experts, int rows, int size, int t, RowTile* to) {
    const int lane = threadIdx.x & 63;
    int before = 0, last = 0;
    if (ends == nullptr) {
        before = (rows + size - 1) / size;
        last = rows;
        if (t < before) {
            *to = {0, t * size, rows};
            return true;
        }
    } else {
        for (int e0 = 0; e0 < experts; e0 += 64) {
            const int e = e0 + lane;
            const int hi = end_of_lane(ends, experts, rows, e0, last);
            int lo = lane_before(hi);
            if (lane == 0) lo = last;
            const int n = e < experts ? (hi - lo + size - 1) / size : 0;
            const int sum = sum_up_to(n);
            const uint64_t behind = __ballot(before + sum > t);
            if (behind != 0) {
                const int l = __builtin_ctzll(behind);
                const int start = before + __builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(n, l);
                const int first = __builtin_amdgcn_readlane(lo, l);
                *to = {e0 + l, first + (t - start) * size, __builtin_amdgcn_readlane(hi, l)};
                return true;
            }
            before += __builtin_amdgcn_readlane(sum, 63);
            last = __builtin_amdgcn_readlane(hi, 63);
        }
    }
    *to = {-1, last + (t - before) * size, rows};
    return to->first < rows;
}

// One T of the workgroup in LDS.
template <class T>
__device__ __forceinline__ T& lds() {
    __shared__ T one;
    return one;
}

// The rows of all experts, and up to 64 experts by falling numbers of rows (ties in order).
struct ExpertRows {
    int end[kMaxExperts], order[64];
};
__device__ __forceinline__ void expert_rows(const int* ends, int experts, int rows, ExpertRows& table) {
    const int lane = threadIdx.x & 63;
    int last = 0, n = 0;  // rows of the first 64 experts, one a lane
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int hi = end_of_lane(ends, experts, rows, e0, last);
        if (e0 + lane < experts && threadIdx.x < 64) table.end[e0 + lane] = hi;
        if (e0 == 0) n = lane < experts ? hi - lane_before(hi) : 0;
        last = __builtin_amdgcn_readlane(hi, 63);
    }
    if (experts > 64) return;
    int rank = 0;
    for (int e = 0; e < experts; ++e) {
        const int o = __builtin_amdgcn_readlane(n, e);
        rank += o > n || (o == n && e < lane) ? 1 : 0;
    }
    if (threadIdx.x < experts) table.order[rank] = lane;
}

// The rows of all experts in LDS, which the workgroup fills once: for each expert its first row and how many
// tiles the experts before it have, of more than `half` rows and of at most that many (an expert's last one);
// in the last entries the first row of no expert and all tiles.
struct RowTable {
    int row[kMaxExperts + 1], tile[kMaxExperts + 1], tail[kMaxExperts + 1];
};
__device__ __forceinline__ void row_table(const int* ends, int experts, int rows, int size, int half, RowTable& table) {
    const int lane = threadIdx.x & 63;
    int tiles = 0, tails = 0, last = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        const int hi = ends == nullptr ? rows : end_of_lane(ends, experts, rows, e0, last);
        int lo = ends == nullptr ? 0 : lane_before(hi);
        if (lane == 0) lo = last;
        const int n = e < experts ? hi - lo : 0, rest = n % size;
        const int full = n / size + (rest > half ? 1 : 0), tail = rest != 0 && rest <= half ? 1 : 0;
        const int sum = sum_up_to(full), tail_sum = sum_up_to(tail);
        if (e < experts && threadIdx.x < 64) {
            table.row[e] = lo;
            table.tile[e] = tiles + sum - full;
            table.tail[e] = tails + tail_sum - tail;
        }
        tiles += __builtin_amdgcn_readlane(sum, 63);
        tails += __builtin_amdgcn_readlane(tail_sum, 63);
        last = __builtin_amdgcn_readlane(hi, 63);
    }
    if (threadIdx.x == 0) {
        table.row[experts] = last;
        table.tile[experts] = tiles;
        table.tail[experts] = tails;
    }
}
// Tile t of `before` (table.tile or table.tail): the last expert before which there are no more than t.
__device__ __forceinline__ int expert_of(const int* before, int experts, int t) {
    const int lane = threadIdx.x & 63;
    int e = -1;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const uint64_t begun = __ballot(e0 + lane < experts && before[min(e0 + lane, experts)] <= t);
        e += __builtin_popcountll(begun);
        if (begun != ~uint64_t(0)) break;
    }
    return e;
}

// The most tiles that row_tile can give.
inline int64_t most_row_tiles(int64_t rows, int64_t experts, int64_t size, bool grouped) {
    return grouped ? rows / size + (experts + 1 < rows ? experts + 1 : rows) : (rows + size - 1) / size;
}

// ---- 8-bit integers --------------------------------------------------------
//
// q = nearest-even(x * 127 / amax), as if taken exactly.  With x = X 2^a, amax = M 2^b, X and
// M integers below 2^p (p = 8 for bf16, 24 for fp32), x * 127 / amax is a half h / 2 exactly or
// off it by |254 X - h M 2^(b-a)| / (254 X) >= 1 / (254 X) > 2^-(p+8) of its value (the numerator is
// a multiple of 2^min(0, b-a), and where b < a, M 2^(b-a) < 2^p takes X's place likewise).  The
// quotient computed as x * (127 / amax) is off by less than 2 half steps: 2^-23 in fp32, 2^-52 in
// fp64.  So a computed value within 2^-20 (bf16 in fp32; 2^-16 apart) or 2^-40 (fp32 in fp64; 2^-32
// apart) of a half is that half, and goes to the even side; any other rounds the right way.

struct TokenScale {
    float factor;  // bf16: 127 / (amax * 2^-exponent), so that no quotient leaves fp32's range
    int exponent;
    float scale;   // amax / 127
};
// amax as fp32 bits; kSpecial or more: a row with an infinity or a NaN.
__device__ __forceinline__ TokenScale token_scale(uint32_t amax) {
    const float m = bits_float(amax);
    if (amax >= kSpecial) return {0.f, 0, bits_float(0x7FC00000u)};
    if (amax == 0u) return {0.f, 0, 0.f};
    const int e = __builtin_amdgcn_frexp_expf(m);
    return {127.f / __builtin_ldexpf(m, -e), e, m / 127.f};
}
// One entry as an integer (any where the row's factor is 0: see integers below).
__device__ __forceinline__ int integer(float x, float factor, int exponent) {
    const float t = __builtin_ldexpf(x, -exponent) * factor;
    const float n = __builtin_rintf(t);
    const bool half = __builtin_fabsf(__builtin_fabsf(t - n) - 0.5f) <= __builtin_fabsf(t) * 0x1p-20f;
    return (int)(half ? 2.f * __builtin_rintf(0.5f * t) : n);
}
__device__ __forceinline__ int integer(float x, double factor) {
    const double t = (double)x * factor, n = __builtin_rint(t);
    const bool half = __builtin_fabs(__builtin_fabs(t - n) - 0.5) <= __builtin_fabs(t) * 0x1p-40;
    return (int)(half ? 2.0 * __builtin_rint(0.5 * t) : n);
}
__device__ __forceinline__ uint32_t pack_integers(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}
// Eight bf16 entries; all 0 where the row's factor is 0.
__device__ __forceinline__ u32x2 integers(const Eight<uint16_t>& v, float factor, int exponent) {
    int n[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        n[2 * i] = integer(bits_float(v.w[i] << 16), factor, exponent);
        n[2 * i + 1] = integer(bits_float(v.w[i] & 0xFFFF0000u), factor, exponent);
    }
    const u32x2 packed = {pack_integers(n[0], n[1], n[2], n[3]), pack_integers(n[4], n[5], n[6], n[7])};
    return factor == 0.f ? u32x2{0u, 0u} : packed;
}
__device__ __forceinline__ u32x2 integers(const Eight<float>& v, double factor) {
    int n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = integer(bits_float(v.w[i]), factor);
    const u32x2 packed = {pack_integers(n[0], n[1], n[2], n[3]), pack_integers(n[4], n[5], n[6], n[7])};
    return factor == 0.0 ? u32x2{0u, 0u} : packed;
}
// Largest value over the wave.
__device__ __forceinline__ uint32_t max64(uint32_t v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor(v, d, 64));
    return v;
}

// Four neighbouring entries of an output row, columns c .. c+3 (< cols written).
__device__ __forceinline__ void put4(float* y, int64_t c, int64_t cols, bool vec, f32x4 v) {
    if (vec && c + 4 <= cols) {
        *reinterpret_cast<f32x4*>(y + c) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < cols) y[c + i] = v[i];
    }
}
__device__ __forceinline__ void put4(uint16_t* y, int64_t c, int64_t cols, bool vec, f32x4 v) {
    if (vec && c + 4 <= cols) {
        *reinterpret_cast<u32x2*>(y + c) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < cols) y[c + i] = to_bf16(v[i]);
    }
}

}  // namespace ops
}  // namespace tsenor
