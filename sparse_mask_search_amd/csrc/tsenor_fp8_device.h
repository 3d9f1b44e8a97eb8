// tsenor_fp8_device.h -- device helpers shared by the 8-bit kernels: block
// scales, conversion to e4m3, element loads.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsenor {
namespace fp8 {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__host__ __device__ __forceinline__ int64_t pad128(int64_t k) { return (k + 127) / 128 * 128; }

__device__ __forceinline__ float bits_float(uint32_t b) { return __builtin_bit_cast(float, b); }

__device__ __forceinline__ float widen(uint16_t b) { return bits_float((uint32_t)b << 16); }

// The scale exponent s of a block: least s >= -127 with amax <= 448 * 2^s.
// With amax = 1.f * 2^(E-127) and 448 = 1.75 * 2^8, s = E-135 if 1.f <= 1.75
// and E-134 otherwise; subnormal amax (E = 0) clamps.
__device__ __forceinline__ int scale_exponent(uint32_t amax) {
    const int E = (int)(amax >> 23);
    const int s = E - ((amax & 0x7FFFFFu) <= 0x600000u ? 135 : 134);
    return amax == 0u ? 0 : (s < -127 ? -127 : s);
}

// 2^-s for the exponents scale_exponent gives (-127 .. 120): always normal.
__device__ __forceinline__ float inverse_scale(int s) { return bits_float((uint32_t)(127 - s) << 23); }

// 2^e for two scale bytes a and b (e = a + b - 254), clamped to [0, 2^127]:
// the factor of a block's sum.  Subnormal powers down to 2^-149 are exact.
__device__ __forceinline__ float scale_product(int a, int b) {
    const int e = a + b - 127;  // exponent field of the product
    const uint32_t normal = (uint32_t)min(e, 254) << 23;
    const uint32_t subnormal = 0x400000u >> min(max(-e, 0), 31);
    return bits_float(e >= 1 ? normal : subnormal);
}

// Four e4m3 numbers, nearest even.  |arguments| <= 448 or NaN.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// fp32 to bf16, nearest even (one instruction on gfx950).
__device__ __forceinline__ uint16_t to_bf16(float x) {
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return (uint32_t)to_bf16(lo) | ((uint32_t)to_bf16(hi) << 16);
}

// Entries c .. c+7 of a row of `cols` entries (zeros behind it).  vec: the row
// may be read 16 bytes at a time.
__device__ __forceinline__ void load8(const uint16_t* row, int64_t c, int64_t cols, bool vec,
                                      uint16_t v[8]) {
    if (vec && c + 8 <= cols) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = (uint16_t)w[i];
            v[2 * i + 1] = (uint16_t)(w[i] >> 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? row[c + i] : (uint16_t)0;
    }
}

// Eight neighbouring entries in registers, bf16 as four pairs.  Magnitudes order like the
// bits below the sign, so a maximum needs no conversion; one of kSpecial or more tells of an
// infinity or a NaN, and only then are entries looked at one by one (finite_only).
constexpr uint32_t kSpecial = 0x7F800000u;
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 pair_max(u16x2 m, uint32_t w) {
    return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu));
}
// The magnitude of a pair's larger entry, as fp32 bits.
__device__ __forceinline__ uint32_t pair_magnitude(u16x2 m) {
    return (uint32_t)max(m[0], m[1]) << 16;
}
// Infinities of a pair become NaN; the larger finite magnitude.
__device__ __forceinline__ uint32_t finite_pair(uint32_t* w) {
    const uint32_t lo = *w & 0x7FFFu, hi = (*w >> 16) & 0x7FFFu;
    if (lo >= 0x7F80u) *w |= 0x7FFFu;
    if (hi >= 0x7F80u) *w |= 0x7FFF0000u;
    return max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u) << 16;
}
__device__ __forceinline__ uint32_t finite_one(uint32_t* w) {
    const uint32_t a = *w & 0x7FFFFFFFu;
    if (a >= kSpecial) *w |= 0x7FFFFFFFu;
    return a < kSpecial ? a : 0u;
}
// Entries of two pairs (of four fp32 words) as e4m3.
__device__ __forceinline__ uint32_t pack_pairs(uint32_t a, uint32_t b, float inv) {
    return pack4(bits_float(a << 16) * inv, bits_float(a & 0xFFFF0000u) * inv, bits_float(b << 16) * inv,
                 bits_float(b & 0xFFFF0000u) * inv);
}
__device__ __forceinline__ uint32_t pack_words(uint32_t a, uint32_t b, uint32_t c, uint32_t d, float inv) {
    return pack4(bits_float(a) * inv, bits_float(b) * inv, bits_float(c) * inv, bits_float(d) * inv);
}

template <class T>
struct Eight;
template <>
struct Eight<uint16_t> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint16_t* row, int64_t c, int64_t cols, bool vec) {
        if (vec && c + 8 <= cols) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = c + 2 * i < cols ? row[c + 2 * i] : 0u;
                const uint32_t hi = c + 2 * i + 1 < cols ? row[c + 2 * i + 1] : 0u;
                w[i] = lo | (hi << 16);
            }
        }
    }
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void keep(uint32_t bits) {  // bit i: entry i stays
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = (uint32_t)__builtin_amdgcn_sbfe((int)bits, 2 * i, 1);
            const uint32_t hi = (uint32_t)__builtin_amdgcn_sbfe((int)bits, 2 * i + 1, 1);
            w[i] &= (lo & 0xFFFFu) | (hi & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ uint32_t magnitude() const {
        u16x2 m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = pair_max(m, w[i]);
        return pair_magnitude(m);
    }
    __device__ __forceinline__ uint32_t finite_only() {
        return max(max(finite_pair(w), finite_pair(w + 1)), max(finite_pair(w + 2), finite_pair(w + 3)));
    }
    __device__ __forceinline__ u32x2 quantised(float inv) const {
        return u32x2{pack_pairs(w[0], w[1], inv), pack_pairs(w[2], w[3], inv)};
    }
    __device__ __forceinline__ void store(uint16_t* to) const {
        *reinterpret_cast<u32x4*>(to) = u32x4{w[0], w[1], w[2], w[3]};
    }
};
template <>
struct Eight<float> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const float* row, int64_t c, int64_t cols, bool vec) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(row) + c;
        if (vec && c + 8 <= cols) {
            const u32x4 a = *reinterpret_cast<const u32x4*>(from);
            const u32x4 b = *reinterpret_cast<const u32x4*>(from + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = a[i];
                w[4 + i] = b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = c + i < cols ? from[i] : 0u;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void keep(uint32_t bits) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] &= (uint32_t)__builtin_amdgcn_sbfe((int)bits, i, 1);
    }
    __device__ __forceinline__ uint32_t magnitude() const {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ uint32_t finite_only() {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, finite_one(w + i));
        return m;
    }
    __device__ __forceinline__ u32x2 quantised(float inv) const {
        return u32x2{pack_words(w[0], w[1], w[2], w[3], inv), pack_words(w[4], w[5], w[6], w[7], inv)};
    }
    __device__ __forceinline__ void store(float* to) const {
        *reinterpret_cast<u32x4*>(to) = u32x4{w[0], w[1], w[2], w[3]};
        *reinterpret_cast<u32x4*>(to + 4) = u32x4{w[4], w[5], w[6], w[7]};
    }
};

// Direct loads from global memory to LDS, from a uniform base plus the lane's
// offset: lane l's 16 bytes (or 4, or its byte widened to 32 bits) land at the LDS
// base + 16 l (4 l).  Written in asm because the
// compiler cannot tell the buffers of a ring apart and would wait for every
// outstanding direct load before each LDS read; the kernels wait for them
// themselves (vmcnt) before the barrier that publishes a buffer.  No register
// receives data.  M0 carries the LDS base; the clobber tells the compiler.
typedef __attribute__((address_space(3))) void lds_void_t;
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(const lds_void_t*)p;
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // M0 is a reserved register; see above
__device__ __forceinline__ void dma16(const void* base, uint32_t offset, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %2"
                 :: "v"(offset), "s"(lds_base), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t offset, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, %2"
                 :: "v"(offset), "s"(lds_base), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void dma_byte(const void* base, uint32_t offset, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %2"
                 :: "v"(offset), "s"(lds_base), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop

// Tile (tm, tn) of workgroup `bid` in a tiles_m x tiles_n grid.  Workgroups go
// to the chip's 8 XCDs round robin and each XCD has its own L2, so XCD x gets a
// contiguous range of an order that walks groups of up to 8 m-tiles column by
// column: the tiles that it runs at one time form a compact block of the grid
// and share their operands' rows.  A bijection for any grid.
__device__ __forceinline__ void tile_of(int64_t bid, int64_t tiles_m, int64_t tiles_n, int64_t& tm,
                                        int64_t& tn) {
    constexpr int64_t kXcd = 8, kGroup = 8;
    const int64_t nb = tiles_m * tiles_n, x = bid % kXcd, rest = nb % kXcd;
    const int64_t t = x * (nb / kXcd) + (x < rest ? x : rest) + bid / kXcd;
    const int64_t grp = t / (kGroup * tiles_n), first = grp * kGroup;
    const int64_t gm = tiles_m - first < kGroup ? tiles_m - first : kGroup;
    const int64_t r = t - grp * kGroup * tiles_n;
    tm = first + r % gm;
    tn = r / gm;
}

// Metadata of four blocks of a row at once.  A block's four words are for the four lane
// groups q = lane / 16; read one by one, a load brings 16 bytes of each of 16 rows and costs
// the address unit as much as one that brings 64.  So lane group g reads all four words of
// block g, and a 4 x 4 transposition across the lane groups hands each its own: word[u] is
// then this lane group's word of block u.
__device__ __forceinline__ void words_of_blocks(const u32x4 mine, uint32_t word[4]) {
    const u32x2 a = __builtin_amdgcn_permlane32_swap(mine[0], mine[2], false, false);
    const u32x2 b = __builtin_amdgcn_permlane32_swap(mine[1], mine[3], false, false);
    const u32x2 c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const u32x2 d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    word[0] = c[0];
    word[1] = c[1];
    word[2] = d[0];
    word[3] = d[1];
}

// Maximum over the 16 lanes of a row of lanes.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
        const uint32_t o = __shfl_xor(v, d, 64);
        v = o > v ? o : v;
    }
    return v;
}

}  // namespace fp8
}  // namespace tsenor
