// tsenor_grouped.hip -- products grouped by expert (include/tsenor_ops.h): bf16
// products, weight gradients, 8-bit integer products.
//
// A product is tiles of (inner columns) x (rows); the operand along the inner dimension
// is on the rows of the matrix instruction, so that a lane holds four neighbouring
// entries of an output row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor_grouped_forms.h"
#include "tsenor_internal.h"
#include "tsenor_ops_device.h"

namespace tsenor {
namespace {

using namespace ops;

// Sixteen bytes at any alignment of the entries.  (Global loads by name: a pointer that the compiler
// cannot place makes it a flat load, which waits for LDS too.)
typedef u32x4 __attribute__((aligned(1), may_alias)) any16;
typedef __attribute__((address_space(1))) const uint8_t global_byte;
__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
    return *(__attribute__((address_space(1))) const any16*)(global_byte*)p;
}
// The same of bf16 entries of which `valid` bytes are there; zeros behind them.  (Rows of 8-bit integers are whole
// units.)
__device__ __forceinline__ u32x4 load16(const uint8_t* p, int64_t valid) {
    if (valid >= 16) return load16(p);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (valid > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (2 * i < valid) {
                const uint32_t x = ((__attribute__((address_space(1))) const uint16_t*)(global_byte*)p)[i];
                v[i / 2] |= x << (16 * (i % 2));
            }
    }
    return v;
}

// Four neighbouring results of a lane, at columns c .. c + 3 of a row, scaled or masked, to `y`.
template <class T, Kind K, class TO>
__device__ __forceinline__ void finish(const GroupedJob& job, int expert, int64_t row, int64_t c, typename T::Sum sum,
                                       TO* y) {
    if (c >= job.inner) return;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)sum[e];
    if constexpr (T::kSize == 1) {
        const float scale = job.bs[row], *as = job.as + expert * job.inner;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = v[e] * scale * as[min(c + e, job.inner - 1)];
    }
    if constexpr (K == kGradient) {
        if (job.mask != nullptr) {  // c is a multiple of four: one word
            const uint32_t keep = job.mask[(expert * job.outer + row) * ((job.inner + 31) / 32) + (c >> 5)] >> (c & 31);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!((keep >> e) & 1u)) v[e] = 0.f;
        }
    }
    put4(y, c, job.inner, job.ovec, v);
}

// Any alignment and any size: tiles of 64 x 64, four waves of 32 x 32, operands through
// registers into two LDS buffers.  AT, BT: the operand is contiguous along its columns.  Loads that straddle
// lines bound it: 8192 rows of 16 experts 4095 x 2047, data gradients 806 us (170 TFLOP/s; 16-byte aligned rows,
// by the tiles below, 164).
template <class T, bool AT, bool BT, Kind K, class TO>
__global__ __launch_bounds__(256) void product_any_kernel(const GroupedJob job) {
    static_assert(T::kSize == 2, "rows of 8-bit integers are aligned");
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
        int first, end;
        rows_of(job.ends, job.rows, expert, &first, &end);
        count = end - first;
        a += first * job.lda + inner0 * T::kSize;
        b += first * job.ldb + outer0 * T::kSize;
        out += expert * job.ostride;
    }
    const int64_t ahave = job.inner - inner0, bhave = outer_end - outer0;  // columns of the tile that exist
    const int64_t reduce = K == kGradient ? count * T::kSize : job.kbytes;
    const int steps = (int)((reduce + 63) / 64);

    auto fetch = [&](const uint8_t* base, int64_t ld, int64_t have, bool turned, int s) {
        if (!turned) {
            const int r = tid >> 2;
            const int64_t c = 64 * (int64_t)s + 16 * (tid & 3);
            return load16(base + min((int64_t)r, have - 1) * ld + c, reduce - c);
        }
        const int r = 32 * s + (tid >> 3), c = 8 * (tid & 7);
        return load16(base + r * ld + c * T::kSize, r * T::kSize < reduce ? (have - c) * T::kSize : 0);
    };
    const int slot_row = row_slot(tid >> 2, tid & 3), slot_turned = turned_slot<64>(tid >> 3, tid & 7);
    typename T::Sum acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = typename T::Sum{0, 0, 0, 0};
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
        u32x4 fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ra = ia + 16 * i, rb = ib + 16 * i;
            fa[i] = AT ? turned_fragment<64>(ta[s & 1], ra, lane) : row_fragment(ta[s & 1], ra, lane);
            fb[i] = BT ? turned_fragment<64>(tb[s & 1], rb, lane) : row_fragment(tb[s & 1], rb, lane);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = T::mma(fa[i >> 1], fb[i & 1], acc[i >> 1][i & 1]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t row = outer0 + ib + 16 * j + (lane & 15);
        if (row >= outer_end) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            finish<T, K>(job, expert, row, inner0 + ia + 16 * i + 4 * (lane >> 4), acc[i][j], out + row * job.ldo);
    }
}

// Few rows (16 NT of one expert to a workgroup): reading the weights bounds the product (16 rows 11008 x 4096 25 us,
// 3.6 TB/s of them; 6 rows of 64 experts 1408 x 2048 12 us, of which 4 are the launch and `ends`: k = 128), so a
// workgroup owns 16 MT columns of the output (rows of the weights) and each of its eight waves
// a stretch of the reduction, with the loads of kAhead units of 128 bytes in flight; the waves'
// sums meet in LDS, in wave order.  A lane q = lane / 16 takes bytes 32 q .. 32 q + 31 of a unit of
// both operands: the two instructions may take the reduction in any order that is the same for both.
// QX: bf16 tokens become 8-bit integers in LDS first, in each workgroup, while its first weights are
// loaded (as fragments, each lane for itself, 16 lanes would do the same work: 12 us for one token
// 4096 x 4096, against 7.7; 7.5 from ready integers).
constexpr int kFewWaves = 8;
constexpr int kFewEntries = kMaxTokenEntries;  // of tokens in LDS, padded rows

template <class T, bool QX, int NT, int MT, class TO>
__global__ __launch_bounds__(64 * kFewWaves) void product_few_kernel(const GroupedJob job) {
    constexpr bool kWhole = T::kSize == 1;  // units only
    constexpr int kAhead = NT * MT >= 4 ? 1 : NT * MT >= 2 ? 2 : 4;  // more registers would leave a CU one workgroup
    typedef typename T::Sum Sum4;
    __shared__ Sum4 sums[kFewWaves][MT * NT][64];
    __shared__ TokenScale scale[QX ? 16 : 1];
    __shared__ uint32_t part[QX ? 16 : 1][kFewWaves];
    __shared__ u32x4 token[QX ? kFewEntries / 16 + 16 : 1];  // rows of kpad + 16 bytes: no two on the same banks
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
        brow[n] = static_cast<const uint8_t*>(job.b) + (t.first + (int64_t)min(16 * n + l16, rows - 1)) * job.ldb + 32 * q;
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
                    if (kWhole || v < whole) av[i][m][c] = load16(p + 16 * c);
                    else av[i][m][c] = load16(p + 16 * c, job.kbytes - 128 * (int64_t)v - 32 * q - 16 * c);
                }
            }
        }
    };
    if (u0 < u1) load_a(u0);
    const int pitch = (int)(job.kbytes / 16) + 1;  // of a token in LDS
    if constexpr (QX) {
        const int vectors = (int)(job.kbytes / 8);  // of a padded row
        Eight<uint16_t> first;  // of row 0: all there is of one short token
        for (int r = 0; r < rows; ++r) {
            const uint16_t* x = static_cast<const uint16_t*>(job.b) + (t.first + (int64_t)r) * (job.ldb / 2);
            uint32_t most = 0u;
            for (int c = tid; c < vectors; c += 64 * kFewWaves) {
                Eight<uint16_t> v;
                v.load(x, 8 * c, job.bcols, job.bvec);
                if (r == 0 && c == tid) first = v;
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
        for (int r = 0; r < rows; ++r) {
            const uint16_t* x = static_cast<const uint16_t*>(job.b) + (t.first + (int64_t)r) * (job.ldb / 2);
            const TokenScale s = scale[r];
            for (int c = tid; c < vectors; c += 64 * kFewWaves) {
                Eight<uint16_t> v = first;
                if (r > 0 || c != tid) v.load(x, 8 * c, job.bcols, job.bvec);
                reinterpret_cast<u32x2*>(token + r * pitch)[c] = integers(v, s.factor, s.exponent);
            }
        }
        __syncthreads();
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
                        bv[i][n][c] = token[min(16 * n + l16, rows - 1) * pitch + 8 * v + 2 * q + c];
                    } else {
                        const uint8_t* p = brow[n] + 128 * (int64_t)v + 16 * c;
                        if (kWhole || v < whole) bv[i][n][c] = load16(p);
                        else bv[i][n][c] = load16(p, job.kbytes - 128 * (int64_t)v - 32 * q - 16 * c);
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

// ---- tiles fed by direct loads -------------------------------------------------
//
// A workgroup of WM x WN waves owns TM inner columns x TN rows of the output, a wave (TM / WM) x
// (TN / WN) in tiles of 32 x 32, and walks the reduction in steps of 64 bytes.  Operands reach LDS by
// direct loads (no registers between) into a ring of R buffers filled R - 1 steps ahead.
// The operands of the next step's first instructions are read while this step's last ones run,
// so the barrier that publishes the next buffer stands in the middle of a step, where no wave
// waits for LDS; loads go out one by one between the matrix instructions, since all at once they
// would stall every wave on the address unit.  Rows and columns behind an operand's end
// repeat its last one (nothing of them is stored); behind the reduction's end zeros are loaded.
// As many workgroups as the LDS holds walk over the tiles, so that the ring never runs empty between two.
// Measured: 8192 x 8192 x 8192 806 us, 1.36 PFLOP/s, the matrix cores 74% busy at 1.50 GHz, which the card's power
// sets (the plain library product 689 us on the same inputs).  16384 rows of 8 experts 11008 x 4096 1.27 ms (1.16 PFLOP/s),
// 8192 of 8-bit integers 360 us (2.05 POP/s): the last round of tiles too.  8192 rows of 16 experts 2048 x 4096: data
// gradients 164 us (44% busy at 2.1 GHz; 127 with as many rows for each), weight gradients under masks 178 us, of which 47
// are the results' way out: a step's wait is for the stores before it too.  (The last from seven inputs in turn, 700 MB;
// 162 from one, which the last-level cache holds.  The cut of the rows counts for less: 175 to 184 over four.)

__device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};

// Direct load from a lane's own address (the steps with an end of the reduction).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16_at(const void* p, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds_base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// One operand of a tile, `S` rows (or columns) wide, as its direct loads see it.
template <class T, bool TURNED, int S, int WAVES>
struct Loads {
    static constexpr int kCount = S / 16 / WAVES;  // of a wave per step, 1024 bytes each
    static_assert(kCount * 16 * WAVES == S, "tile");
    const uint8_t* base;      // the tile's first entry
    int64_t step;             // bytes from step to step
    uint32_t offset[kCount];  // of this lane
    // have: rows (columns) of the tile that exist
    __device__ __forceinline__ void init(const uint8_t* first, int64_t ld, int have, int wave, int lane) {
        base = uniform(first);
        step = TURNED ? 32 * ld : 64;
#pragma unroll
        for (int j = 0; j < kCount; ++j) {
            const int slot = 64 * (wave * kCount + j) + lane;
            if constexpr (TURNED) {
                const int r = slot / (S / 8), c = turned_slot<S>(r, slot % (S / 8)) - r * (S / 8);
                offset[j] = __umul24(r, (uint32_t)ld) + 16 * min(c, (have - 1) / 8);
            } else {
                const int r = slot / 4, c = row_slot(r, slot % 4) - 4 * r;
                offset[j] = __umul24(min(r, have - 1), (uint32_t)ld) + 16 * c;
            }
        }
    }
    // Step s; not inside: with zeros behind the reduction's `reduce` bytes (turned: of one column).
    __device__ static __forceinline__ void load(const Loads& of, bool inside, int j, int64_t s, int64_t reduce,
                                                const u32x4* tile, int wave, int lane) {
        const uint32_t to = lds_offset(tile + 64 * (wave * kCount + j));
        if (inside) {
            dma16(of.base + s * of.step, of.offset[j], to);
            return;
        }
        const int slot = 64 * (wave * kCount + j) + lane;
        int64_t at;
        if constexpr (TURNED) {
            at = (32 * s + slot / (S / 8)) * T::kSize;
        } else {
            const int r = slot / 4;
            at = 64 * s + 16 * (row_slot(r, slot % 4) - 4 * r);
        }
        const uint8_t* p = at < reduce ? of.base + s * of.step + of.offset[j] : reinterpret_cast<const uint8_t*>(&kZeros);
        dma16_at(p, to);
    }
    // The same through a register, at any alignment (not turned); store() puts it where load() would.
    __device__ static __forceinline__ u32x4 fetch(const Loads& of, bool inside, int j, int64_t s, int64_t reduce, int wave,
                                                  int lane) {
        const uint8_t* p = of.base + s * of.step + of.offset[j];
        if (inside) return load16(p);
        const int slot = 64 * (wave * kCount + j) + lane, r = slot / 4;
        return load16(p, reduce - 64 * s - 16 * (row_slot(r, slot % 4) - 4 * r));
    }
    __device__ static __forceinline__ void store(u32x4* tile, int j, u32x4 v, int wave, int lane) {
        tile[64 * (wave * kCount + j) + lane] = v;
    }
    __device__ static __forceinline__ u32x4 fragment(const u32x4* tile, int at, int lane) {
        if constexpr (TURNED) return turned_fragment<S>(tile, at, lane);
        else return row_fragment(tile, at, lane);
    }
};

// Weight gradients, the largest part of what such a call moves, leave past the caches: 8192 rows of 16
// experts 2048 x 4096 under masks 183 -> 178 us, 1022 rows of 16 1792 x 7680 in fp32 192 -> 180 (under masks 239 -> 244).
// A product's results do not (8192 x 4096 over 1024: 69 -> 72 us).
template <Kind K, class V>
__device__ __forceinline__ void put_last(V* to, V v) {
    if constexpr (K == kGradient) __builtin_nontemporal_store(v, to);
    else *to = v;
}

// The results of a wave's FA x FB tiles of 16 x 16, rows row0 + STEP j, columns c0 + 16 i + 4 q (c0 a
// multiple of 32).  Where all rows and columns exist, what scales them is loaded first (a load among the
// stores would wait for all of those before it), mask words come from LDS (`words`, kWords a row) if they are
// there, and a store writes 16 bytes a lane.
template <class T, Kind K, int FA, int FB, int STEP, int kWords, class TO>
__device__ __forceinline__ void store_tile(const GroupedJob& job, int expert, int row0, bool complete, int rows, int c0,
                                           int q, const typename T::Sum* sums, const uint32_t* words, TO* out) {
    constexpr bool kScaled = T::kSize == 1, kMasked = K == kGradient, kHalf = sizeof(TO) == 2;
    const bool elsewhere = kMasked && job.mask != nullptr && words == nullptr;
    if (!complete || elsewhere || c0 + 16 * FA > (int)job.inner || !(kHalf ? job.ovec8 : job.ovec)) {
#pragma unroll
        for (int j = 0; j < FB; ++j) {
            const int row = row0 + STEP * j;
            if (row >= rows) continue;
#pragma unroll
            for (int i = 0; i < FA; ++i) {
                __builtin_amdgcn_sched_barrier(0);  // or results of several stores are made at once, and spilled
                finish<T, K>(job, expert, row, c0 + 16 * i + 4 * q, sums[i * FB + j], out + row * job.ldo);
            }
        }
        return;
    }
    f32x4 across[kScaled ? FA : 1];
    float down[kScaled ? FB : 1];
    if constexpr (kScaled) {
        const float* as = job.as + expert * job.inner + c0 + 4 * q;
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) across[i][e] = as[16 * i + e];
#pragma unroll
        for (int j = 0; j < FB; ++j) down[j] = job.bs[row0 + STEP * j];
    }
    // Sixteen bytes of a lane's row, from one (fp32) or two neighbouring tiles (bf16: they change
    // places between the lane quarters): 64 bytes of each of 16 rows.
    const auto piece = [&](int i, int j) __attribute__((always_inline)) {
        uint32_t keep = 0xFFFFFFFFu;
        if constexpr (kMasked)
            if (words != nullptr) keep = words[STEP * j * kWords + i / 2];
        f32x4 v[kHalf ? 2 : 1];
#pragma unroll
        for (int p = 0; p < (kHalf ? 2 : 1); ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = (float)sums[(i + p) * FB + j][e];
                if constexpr (kScaled) x = x * down[j] * across[i + p][e];
                if constexpr (kMasked) x = (keep >> (16 * ((i + p) & 1) + 4 * q + e)) & 1u ? x : 0.f;
                v[p][e] = x;
            }
        if constexpr (kHalf) {
            const u32x2 lo = __builtin_amdgcn_permlane16_swap(pack_bf16(v[0][0], v[0][1]), pack_bf16(v[1][0], v[1][1]),
                                                              false, false);
            const u32x2 hi = __builtin_amdgcn_permlane16_swap(pack_bf16(v[0][2], v[0][3]), pack_bf16(v[1][2], v[1][3]),
                                                              false, false);
            return u32x4{lo.x, hi.x, lo.y, hi.y};
        } else {
            return __builtin_bit_cast(u32x4, v[0]);
        }
    };
    constexpr int kPiece = kHalf ? 2 : 1;         // tiles of one
    // Two pieces to each store, whole lines of 8 rows, for weight gradients: 1022 rows of 16 experts 1792 x
    // 7680 in fp32 297 -> 180 us (5.1 TB/s), 8192 rows of 16 2048 x 4096 under masks 272 -> 230, in bf16 192 -> 178.
    // Products, whose results are a smaller part, gain nothing.
    constexpr bool kLines = K == kGradient && FA % (2 * kPiece) == 0;
    const int l16 = threadIdx.x & 15, col = kHalf ? 16 * (q & 1) + 8 * (q >> 1) : 4 * q;
    TO* y = out + (kLines ? row0 - (l16 & 8) : row0) * job.ldo + c0 + col + (kLines ? (l16 >> 3) * 16 * kPiece : 0);
#pragma unroll
    for (int j = 0; j < FB; ++j) {
#pragma unroll
        for (int i = 0; i < FA; i += (kLines ? 2 : 1) * kPiece) {
            __builtin_amdgcn_sched_barrier(0);
            const u32x4 a = piece(i, j);
            if constexpr (kLines) {
                // lanes 8 .. 15 of 16 take the second piece of the first eight rows, and give their first piece
                const u32x4 b = piece(i + kPiece, j);
                u32x4 upper, lower;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    upper[e] = (uint32_t)__builtin_amdgcn_update_dpp((int)a[e], (int)b[e], 0x128, 0xF, 0xC, false);
                    lower[e] = (uint32_t)__builtin_amdgcn_update_dpp((int)b[e], (int)a[e], 0x128, 0xF, 0x3, false);
                }
                put_last<K>(reinterpret_cast<u32x4*>(y + 16 * i), upper);
                put_last<K>(reinterpret_cast<u32x4*>(y + 8 * job.ldo + 16 * i), lower);
            } else {
                put_last<K>(reinterpret_cast<u32x4*>(y + 16 * i), a);
            }
        }
        y += STEP * job.ldo;
    }
}

// Work t of `count` for workgroup `bid`: workgroups go to the chip's 8 XCDs round robin and each
// XCD has its own L2, so XCD x gets a contiguous range.
__device__ __forceinline__ int in_order(int bid, int count) {
    const int x = bid % 8, rest = count % 8;
    return x * (count / 8) + min(x, rest) + bid / 8;
}
// Tile t of a grid, in groups of up to 8 tm column by column: a range forms a compact block.
__device__ __forceinline__ void grid_tile(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int grp = t / (8 * tiles_n), first = grp * 8, gm = min(tiles_m - first, 8);
    const int r = t - grp * 8 * tiles_n;
    tm = uniform(first + r % gm);
    tn = uniform(r / gm);
}

// Whether a step's loads may meet the reduction's end.
struct Inside {
    static constexpr bool value = false;
};
struct AtEnd {
    static constexpr bool value = true;
};
template <int N>
struct MaskWords {
    uint32_t word[N];
};
template <int N>
struct Count {
    static constexpr int value = N;
};

template <class T, bool AT, bool BT, Kind K, int TM, int TN, int WM, int WN, int R, bool LONG, bool DIRECT, class TO>
__global__ __launch_bounds__(64 * WM * WN) void product_tile_kernel(const GroupedJob job) {
    constexpr int W = WM * WN, TA = TM / WM / 32, TB = TN / WN / 32;
    typedef Loads<T, AT, TM, W> LoadsA;
    typedef Loads<T, BT, TN, W> LoadsB;
    constexpr bool kMasked = K == kGradient && LONG;
    constexpr int kHalf = TB > 1 ? TN / 2 : 0;  // an expert's last rows, if they are no more, take half a tile's products
    static_assert(DIRECT ? R >= 4 : R == 3 && !AT && !BT && T::kSize == 2, "ring");
    struct Buffer {
        u32x4 a[TM * 4];
        u32x4 b[TN * 4];
    };
    __shared__ Buffer ring[R];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int across = (int)((job.inner + TM - 1) / TM);
    const int down = K == kGradient ? (int)((job.outer + TN - 1) / TN) : 0;  // of one expert

    // The mask words of a weight gradient's tile come by direct loads too, before its first step: they have
    // landed when its results are written.  Two sets in turn, since other waves may still be at
    // the tile before.
    constexpr int kWords = TM / 32, kMaskLoads = kMasked ? TN * kWords / 64 / W : 0;
    static_assert(kMaskLoads * 64 * W == (kMasked ? TN * kWords : 0), "mask words");
    uint32_t* words = nullptr;
    if constexpr (kMasked) words = lds<MaskWords<2 * TN * kWords>>().word;

    struct Tile {  // the same in all lanes, but for the loads' offsets
        int expert, inner0, outer0, outer_end, full, steps;
        int64_t reduce;
        LoadsA la;
        LoadsB lb;
    };
    int total, work = blockIdx.x;  // work of the launch (it fits a grid); this workgroup's next piece
    if constexpr (K == kProduct) {
        static_assert(LONG, "products");
        const RowTable& table = lds<RowTable>();
        // Half tiles go behind all others where workgroups have few tiles, so that none begins a whole one last: 8192
        // rows of 16 experts 2048 x 4096 210 -> 197 us, 4096 x 2048 transposed 169 -> 164, but 4096 rows of 8 11008 x 4096
        // 412 -> 432.  With more they are farther from those that read the same weights, for nothing: 16384 rows of 8
        // experts 11008 x 4096 1269 -> 1276 us.
        const bool last = across * (int64_t)(job.rows / TN) < 4 * (int64_t)gridDim.x;
        row_table(job.ends, job.experts, job.rows, TN, last ? kHalf : 0, lds<RowTable>());
        __syncthreads();
        const int none = job.rows - uniform(table.row[job.experts]);
        total = across * (uniform(table.tile[job.experts] + table.tail[job.experts]) + (none + TN - 1) / TN);
    } else {
        total = across * down * job.experts;
        if constexpr (LONG) {
            expert_rows(job.ends, job.experts, job.rows, lds<ExpertRows>());
            __syncthreads();
        }
    }
    // The next tile that has something to add up; the others' results are zeros, written here.
    const auto find = [&](Tile& to) __attribute__((always_inline)) {
        for (; work < total; work += LONG ? (int)gridDim.x : total) {
            const uint8_t *a = static_cast<const uint8_t*>(job.a), *b = static_cast<const uint8_t*>(job.b);
            int tm = 0, tn = 0;
            if constexpr (K == kProduct) {
                // tiles, half tiles, rows of no expert
                const RowTable& table = lds<RowTable>();
                const int tiles = uniform(table.tile[job.experts]), w = work - across * tiles;
                if (w < 0) {
                    grid_tile(in_order(work, across * tiles), across, tiles, tm, tn);
                    to.expert = uniform(expert_of(table.tile, job.experts, tn));
                    to.outer0 = uniform(table.row[to.expert]) + (tn - uniform(table.tile[to.expert])) * TN;
                    to.outer_end = uniform(table.row[to.expert + 1]);
                } else if (const int tails = uniform(table.tail[job.experts]); w < across * tails) {
                    grid_tile(in_order(w, across * tails), across, tails, tm, tn);
                    to.expert = uniform(expert_of(table.tail, job.experts, tn));
                    to.outer_end = uniform(table.row[to.expert + 1]);
                    to.outer0 = to.outer_end - (to.outer_end - uniform(table.row[to.expert])) % TN;
                } else {
                    tn = (w - across * tails) / across;
                    tm = w - across * (tails + tn);
                    to.expert = -1;
                    to.outer0 = uniform(table.row[job.experts]) + tn * TN;
                    to.outer_end = job.rows;
                }
                to.inner0 = tm * TM;
                to.reduce = to.expert < 0 ? 0 : job.kbytes;
                a += to.expert * job.astride + (AT ? (int64_t)to.inner0 * T::kSize : to.inner0 * job.lda);
                b += to.outer0 * job.ldb;
            } else {
                // Expert after expert, each spread over all XCDs.  Workgroups that take many tiles go
                // through the experts by falling numbers of rows, every other round the other way, so
                // that all add up about as many rows.
                const int per = across * down, g = gridDim.x, round = work / g;
                int w = work;
                if (LONG && round % 2 == 1 && (round + 1) * g <= total) w = (2 * round + 1) * g - 1 - work;
                to.expert = uniform(w / per);
                if constexpr (LONG) {
                    if (job.experts <= 64) to.expert = uniform(lds<ExpertRows>().order[to.expert]);
                }
                grid_tile(in_order(w % per, per), across, down, tm, tn);
                to.inner0 = tm * TM;
                to.outer0 = tn * TN;
                to.outer_end = (int)job.outer;
                int first, end;
                if constexpr (LONG) {
                    const ExpertRows& table = lds<ExpertRows>();
                    first = to.expert == 0 ? 0 : table.end[to.expert - 1];
                    end = table.end[to.expert];
                } else {
                    rows_of(job.ends, job.rows, to.expert, &first, &end);
                }
                first = uniform(first);
                to.reduce = (int64_t)uniform(end - first) * T::kSize;
                a += first * job.lda + (int64_t)to.inner0 * T::kSize;
                b += first * job.ldb + (int64_t)to.outer0 * T::kSize;
            }
            if (to.reduce == 0) {
                TO* out = static_cast<TO*>(job.out) + (K == kGradient ? to.expert * job.ostride : 0);
                for (int i = tid; i < TM * TN; i += 64 * W)
                    if (to.outer0 + i / TM < to.outer_end && to.inner0 + i % TM < job.inner)
                        out[(to.outer0 + (int64_t)(i / TM)) * job.ldo + to.inner0 + i % TM] = TO(0);
                continue;
            }
            to.full = (int)(to.reduce / 64);
            to.steps = max(2 * (int)((to.reduce + 127) / 128), R < 4 ? 4 : (R + 1) / 2 * 2);  // loads reach into one tile behind
            to.la.init(a, job.lda, (int)min(job.inner - to.inner0, (int64_t)TM), wave, lane);
            to.lb.init(b, job.ldb, min(to.outer_end - to.outer0, TN), wave, lane);
            work += LONG ? (int)gridDim.x : total;
            return true;
        }
        return false;
    };
    Tile cur, nxt;
    if (!find(cur)) return;
    nxt = cur;
    nxt.full = 0;
    nxt.reduce = 0;  // nothing: zeros are loaded

    // Load number j of the tile's step t into its buffer; steps behind the last are the next tile's first
    // ones, so that they are on their way while this tile's results are written.
    constexpr int kLoads = LoadsA::kCount + LoadsB::kCount, kLate = TA > 1 ? kLoads / 2 : 0;
    const auto load = [&](auto end, int j, int t, Buffer& buf) __attribute__((always_inline)) {
        const bool ahead = end.value && t >= cur.steps;
        const int s = ahead ? t - cur.steps : t;
        const bool inside = !end.value || s < (ahead ? nxt.full : cur.full);
        if (j < LoadsA::kCount)
            LoadsA::load(ahead ? nxt.la : cur.la, inside, j, s, ahead ? nxt.reduce : cur.reduce, buf.a, wave, lane);
        else
            LoadsB::load(ahead ? nxt.lb : cur.lb, inside, j - LoadsA::kCount, s, ahead ? nxt.reduce : cur.reduce, buf.b,
                         wave, lane);
    };
    // Not DIRECT: what step t + 1 needs is written to LDS in the first half of step t, and what step t + 3
    // needs is fetched into the same registers in the second.
    u32x4 held[DIRECT ? 1 : 2][DIRECT ? 1 : kLoads];
    const auto fetch = [&](auto end, int j, int t, int set) __attribute__((always_inline)) {
        const bool ahead = end.value && t >= cur.steps;
        const int s = ahead ? t - cur.steps : t;
        const bool inside = !end.value || s < (ahead ? nxt.full : cur.full);
        if (j < LoadsA::kCount)
            held[set][j] = LoadsA::fetch(ahead ? nxt.la : cur.la, inside, j, s, ahead ? nxt.reduce : cur.reduce, wave, lane);
        else
            held[set][j] = LoadsB::fetch(ahead ? nxt.lb : cur.lb, inside, j - LoadsA::kCount, s,
                                         ahead ? nxt.reduce : cur.reduce, wave, lane);
    };
    const auto store = [&](int j, int set, Buffer& buf) __attribute__((always_inline)) {
        if (j < LoadsA::kCount) LoadsA::store(buf.a, j, held[set][j], wave, lane);
        else LoadsB::store(buf.b, j - LoadsA::kCount, held[set][j], wave, lane);
    };
    int set = 0;  // of mask words
    const auto load_words = [&]() __attribute__((always_inline)) {
        const int64_t wpr = (job.inner + 31) / 32;
        const uint8_t* first = uniform(reinterpret_cast<const uint8_t*>(
            job.mask + (cur.expert * job.outer + cur.outer0) * wpr + cur.inner0 / 32));
        const int rows = min(cur.outer_end - cur.outer0, TN), have = min((int)wpr - cur.inner0 / 32, kWords);
#pragma unroll
        for (int j = 0; j < kMaskLoads; ++j) {
            const int slot = 64 * (wave * kMaskLoads + j) + lane;
            dma4(first, 4 * (__umul24(min(slot / kWords, rows - 1), (uint32_t)wpr) + min(slot % kWords, have - 1)),
                 lds_offset(words + TN * kWords * set + 64 * (wave * kMaskLoads + j)));
        }
    };
    typename T::Sum acc[TA][2][TB][2];  // pairs of 16: tiles of 32 x 32
    u32x4 fa[2][2], fb[2][TB][2];
    const auto read_a = [&](int i, const Buffer& buf) __attribute__((always_inline)) {  // into the set i & 1
#pragma unroll
        for (int p = 0; p < 2; ++p) fa[i & 1][p] = LoadsA::fragment(buf.a, (TM / WM) * wm + 32 * i + 16 * p, lane);
    };
    // (a wave's rows lie WN fragments apart, so that all waves share what a short tile has)
    const auto read_b = [&](auto pairs, int set, const Buffer& buf) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < pairs.value; ++j)
#pragma unroll
            for (int p = 0; p < 2; ++p)
                fb[set][j][p] = LoadsB::fragment(buf.b, 16 * (WN * (2 * j + p) + wn), lane);
    };
    // Step t, whose first operands are in registers (set t & 1).  The loads of step t + R - 1 go
    // out after the barrier, the last kLate of them in the first half of the next step.
    const auto step = [&](auto end, auto pairs, int t, int set, const Buffer& buf, Buffer& next, Buffer& early,
                          Buffer& late) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TA; ++i) {
            if (i == TA / 2) {
                // the next step's loads have landed, and every wave is past the step before
                if constexpr (DIRECT) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((R - 3) * kLoads) : "memory");
                else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
            }
            if (i + 1 < TA) {
                read_a(i + 1, buf);
            } else {
                if constexpr (end.value) read_b(Count<TB>(), set ^ 1, next);
                else read_b(pairs, set ^ 1, next);
                if (TA > 1) read_a(0, next);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < pairs.value; ++j) {
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    acc[i][p >> 1][j][p & 1] = T::mma(fa[i & 1][p >> 1], fb[set][j][p & 1], acc[i][p >> 1][j][p & 1]);
                __builtin_amdgcn_sched_barrier(0);
                constexpr int kSlots = TA > 1 ? TA / 2 * pairs.value : pairs.value;  // of a half step
                const int slot = (i >= TA / 2 ? i - TA / 2 : i) * pairs.value + j;
                if constexpr (!DIRECT) {
                    if (i >= TA / 2) {
#pragma unroll
                        for (int l = slot; l < kLoads; l += kSlots) fetch(end, l, t + 3, set ^ 1);
                    } else {
#pragma unroll
                        for (int l = slot; l < kLoads; l += kSlots) store(l, set ^ 1, next);
                    }
                } else if (i >= TA / 2) {
#pragma unroll
                    for (int l = slot; l < kLoads - kLate; l += kSlots) load(end, l, t + R - 1, early);
                } else {
#pragma unroll
                    for (int l = slot; l < kLate; l += kSlots) load(end, kLoads - kLate + l, t + R - 2, late);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (TA == 1) read_a(0, next);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    bool more = false;
    if constexpr (DIRECT) {
#pragma unroll
        for (int t = 0; t < R - 1; ++t)
#pragma unroll
            for (int j = 0; j < (t == R - 2 ? kLoads - kLate : kLoads); ++j) load(AtEnd(), j, t, ring[t]);
        if constexpr (LONG) more = find(nxt);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((R - 2) * kLoads - kLate) : "memory");
    } else {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            fetch(AtEnd(), j, 0, 0);
            fetch(AtEnd(), j, 1, 1);
        }
        if constexpr (LONG) more = find(nxt);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            store(j, 0, ring[0]);
            fetch(AtEnd(), j, 2, 0);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read_b(Count<TB>(), 0, ring[0]);
    read_a(0, ring[0]);
    const auto inc = [](int v) { return v == R - 1 ? 0 : v + 1; };
    const auto dec = [](int v) { return v == 0 ? R - 1 : v - 1; };
    int at = 0;  // the buffer of the current step
    for (;;) {
#pragma unroll
        for (int i = 0; i < 2 * TA; ++i)
#pragma unroll
            for (int j = 0; j < 2 * TB; ++j) acc[i >> 1][i & 1][j >> 1][j & 1] = typename T::Sum{0, 0, 0, 0};
        if constexpr (kMasked) {
            set ^= 1;
            if (job.mask != nullptr) load_words();
        }
        int t = 0;
        const auto two_steps = [&](auto end, auto pairs) __attribute__((always_inline)) {
            const int one = inc(at), two = inc(one), last = dec(at);
            step(end, pairs, t, 0, ring[at], ring[one], ring[last], ring[dec(last)]);
            step(end, pairs, t + 1, 1, ring[one], ring[two], ring[at], ring[last]);
            at = two;
        };
        const auto all_steps = [&](auto pairs) __attribute__((always_inline)) {
            // two steps reach as far as t + R (DIRECT) or t + 4
            for (; t + (DIRECT ? R : 4) < cur.full; t += 2) two_steps(Inside(), pairs);
            for (; t < cur.steps; t += 2) two_steps(AtEnd(), pairs);
        };
        if (K == kProduct && cur.outer_end - cur.outer0 <= kHalf) all_steps(Count<TB / 2 + (TB == 1)>());
        else all_steps(Count<TB>());
        const int row0 = cur.outer0 + 16 * wn + (lane & 15), c0 = cur.inner0 + (TM / WM) * wm;
        const uint32_t* kept =
            kMasked && job.mask != nullptr ? words + TN * kWords * set + (16 * wn + (lane & 15)) * kWords + TM / WM / 32 * wm
                                           : nullptr;
        store_tile<T, K, 2 * TA, 2 * TB, 16 * WN, kWords>(
            job, cur.expert, row0, cur.outer_end - cur.outer0 >= TN, cur.outer_end, c0, lane >> 4, &acc[0][0][0][0], kept,
            static_cast<TO*>(job.out) + (K == kGradient ? cur.expert * job.ostride : 0));
        if (!more) break;
        cur = nxt;
        more = find(nxt);
        if (!more) {
            nxt.full = 0;
            nxt.reduce = 0;
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
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

template <class T, bool AT, bool BT, Kind K, int TM, int TN, int WM, int WN, int R, bool LONG, bool DIRECT, class TO>
int tile(const GroupedJob& job, void* stream) {
    const int64_t across = (job.inner + TM - 1) / TM;
    const int64_t down = K == kGradient ? (job.outer + TN - 1) / TN * job.experts
                                        : most_row_tiles(job.rows, job.experts, TN, job.ends != nullptr);
    if (across > (int64_t)0xFFFFFFFF / (64 * WM * WN) / down) return kGridTooLarge;
    static_assert(sizeof(RowTable) == kRowTableBytes && sizeof(ExpertRows) == kExpertRowsBytes, "LDS");
    const int64_t most = kCus * at_once(K, TM, TN, R);
    const int64_t groups = LONG && across * down > most ? most : across * down;
    hipLaunchKernelGGL((product_tile_kernel<T, AT, BT, K, TM, TN, WM, WN, R, LONG, DIRECT, TO>), dim3((unsigned)groups),
                       dim3(64 * WM * WN), 0, (hipStream_t)stream, job);
    return (int)hipGetLastError();
}

template <class T, bool AT, bool BT, Kind K, class TO>
int product(const GroupedJob& job, void* stream) {
    const Form form = pick_form<K, AT, BT>(job, T::kSize);
    if constexpr (K == kProduct && !AT) {
        if (form == kFew64) return few<T, false, 1, 4, TO>(job, stream);
        if (form == kFew32) return few<T, false, 1, 2, TO>(job, stream);
        if (form == kFew16) return few<T, false, 1, 1, TO>(job, stream);
        if (form == kFew32x32) return few<T, false, 2, 2, TO>(job, stream);
    }
    if constexpr (T::kSize == 2) {
        if constexpr (!AT && !BT)
            if (form == kStaged256x128) return tile<T, AT, BT, K, 256, 128, 2, 4, 3, true, false, TO>(job, stream);
        if (form == kAny) return any<T, AT, BT, K, TO>(job, stream);
    }
    if (form == k256x256) return tile<T, AT, BT, K, 256, 256, 2, 4, 4, true, true, TO>(job, stream);
    if (form == k128x128) return tile<T, AT, BT, K, 128, 128, 2, 4, 8, true, true, TO>(job, stream);
    if constexpr (K == kProduct) {
        if (form == k256x128) return tile<T, AT, BT, K, 256, 128, 2, 4, 6, true, true, TO>(job, stream);
        return tile<T, AT, BT, K, 64, 64, 2, 2, 8, true, true, TO>(job, stream);
    } else {
        return tile<T, AT, BT, K, 64, 64, 2, 2, 4, false, true, TO>(job, stream);
    }
}

}  // namespace

int launch_grouped_mm(const GroupedJob& job, bool transposed, bool bf16out, void* stream) {
    if (transposed)
        return bf16out ? product<Bf16, true, false, kProduct, uint16_t>(job, stream)
                       : product<Bf16, true, false, kProduct, float>(job, stream);
    return bf16out ? product<Bf16, false, false, kProduct, uint16_t>(job, stream)
                   : product<Bf16, false, false, kProduct, float>(job, stream);
}

int launch_grouped_wgrad(const GroupedJob& job, bool bf16out, void* stream) {
    return bf16out ? product<Bf16, true, true, kGradient, uint16_t>(job, stream)
                   : product<Bf16, true, true, kGradient, float>(job, stream);
}

int launch_gemm_int8(const GroupedJob& job, bool bf16x, bool bf16out, void* stream) {
    if (bf16x)
        return bf16out ? few<Int8, true, 1, 1, uint16_t>(job, stream) : few<Int8, true, 1, 1, float>(job, stream);
    return bf16out ? product<Int8, false, false, kProduct, uint16_t>(job, stream)
                   : product<Int8, false, false, kProduct, float>(job, stream);
}

}  // namespace tsenor
