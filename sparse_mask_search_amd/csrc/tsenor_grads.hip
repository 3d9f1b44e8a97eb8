// tsenor_grads.hip -- the norm of a list of gradients and their clipping
// (include/tsenor_ops.h).
//
// A launch takes up to kGradsPerLaunch tensors as arguments and walks their chunks of
// kChunk entries with a fixed grid; a workgroup keeps one partial sum, in 64 bits (a
// square of any fp32 number fits, and sums of 2^40 of them lose nothing that fp32 would
// show).  The scaling launches add all partial sums in one order, in every workgroup:
// no atomics, no launch between, the same result on every run.
// Memory bounds both: four layers of a model of width 4096 (810M bf16 entries under masks) 331 us for the sums
// (5.2 TB/s) and 731 for the scaling (4.6 TB/s, reading and writing).  One layer of width 64 takes 6.5 us each,
// which is latency: arguments, entries, the workgroup's sum.
// Adding all partial sums in every workgroup of every scaling launch is quadratic in the list.  It shows where thousands
// of tensors have many chunks each: scaling tensors of 1408 x 2048 in bf16 to others runs at 5.4 TB/s for 480 of them, 5.1 for
// 1920, 4.6 for 4800 and 3.8 for 9600 (the sums at 5.0 to 5.1); a stack of them is one tensor.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor_internal.h"
#include "tsenor_ops_device.h"

namespace tsenor {
namespace {

using namespace ops;

constexpr int kThreads = 1024, kUnroll = 4;
constexpr int kChunk = kThreads * 8 * kUnroll;  // entries
constexpr int kWaves = kThreads / 64;

// Bits of the entries c .. c+7 of a mask row of `words` words; bits behind the row are 0.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* row, int64_t words, int64_t c) {
    const int64_t w = c >> 5;
    const int s = (int)(c & 31);
    uint32_t bits = row[w] >> s;
    if (s > 24 && w + 1 < words) bits |= row[w + 1] << (32 - s);
    return bits & 0xFFu;
}

// Entry `at` of a job (row by row): its row and column.  at = base + near with base uniform:
// one 64-bit division a chunk, a 32-bit one a vector.
struct Place {
    int64_t row, col;
};
__device__ __forceinline__ Place place_of(int64_t base_row, int64_t base_col, int64_t near, int64_t cols) {
    const int64_t c = base_col + near;
    if (c < cols) return {base_row, c};
    if (cols <= 0x7FFFFFFF && c <= 0x7FFFFFFF) {
        const uint32_t r = (uint32_t)c / (uint32_t)cols;
        return {base_row + r, (int64_t)((uint32_t)c - r * (uint32_t)cols)};
    }
    const int64_t r = c / cols;
    return {base_row + r, c - r * cols};
}

template <class T>
__device__ __forceinline__ double squares(const Eight<T>& v) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x;
        if constexpr (sizeof(T) == 2) x = bits_float(i & 1 ? v.w[i >> 1] & 0xFFFF0000u : v.w[i >> 1] << 16);
        else x = bits_float(v.w[i]);
        s = __builtin_fma((double)x, (double)x, s);
    }
    return s;
}
template <class T>
__device__ __forceinline__ void scale(Eight<T>& v, float f) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v.w[i] = pack_bf16(bits_float(v.w[i] << 16) * f, bits_float(v.w[i] & 0xFFFF0000u) * f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.w[i] = __builtin_bit_cast(uint32_t, bits_float(v.w[i]) * f);
    }
}
template <class T>
__device__ __forceinline__ T scaled_one(const T* p, bool keep, float f) {
    if constexpr (sizeof(T) == 2) return keep ? to_bf16(widen(*p) * f) : (uint16_t)0;
    else return keep ? *p * f : 0.f;
}

// Results leave past the caches, which keep gradients for the scaling instead: 810M bf16 entries to other
// tensors 881 -> 839 us, under masks 1095 -> 1060; in place 908 and 1109 either way.  fp32 results do not (405M entries under
// masks 944 -> 957, without 919 -> 966).
template <class T>
__device__ __forceinline__ void store_last(const Eight<T>& v, T* to) {
    if constexpr (sizeof(T) == 2)
        __builtin_nontemporal_store(u32x4{v.w[0], v.w[1], v.w[2], v.w[3]}, reinterpret_cast<u32x4*>(to));
    else
        v.store(to);
}

// Where vector n of a chunk lies (kRows): `row` rows behind the chunk's first, vector `at` of that row.
struct Vector {
    int row, at;
};
// The chunk begins at vector v0 of a row of `per` vectors; q = v0 + n < 2^24, so that it is exact in
// fp32 and the quotient by per is off by one at most.
__device__ __forceinline__ Vector vector_of(int q, int per, float inv) {
    int r = (int)((float)q * inv), c = q - r * per;
    if (c < 0) {
        --r;
        c += per;
    } else if (c >= per) {
        ++r;
        c -= per;
    }
    return {r, c};
}

// One chunk of one gradient.  kFlat: contiguous and 16-byte aligned, a vector of a masked one may reach
// into the next row (of at least 8 entries); kRows: rows of whole vectors, aligned; kLoose: any
// other, entry by entry.
template <class T, bool SCALE>
__device__ __forceinline__ void chunk(const GradJob& g, int64_t begin, float f, double* sum) {
    const T* x = static_cast<const T*>(g.grad);
    T* y = static_cast<T*>(g.out);
    const int64_t size = g.rows * g.cols, words = (g.cols + 31) / 32;
    const bool placed = g.layout != kFlat || g.mask != nullptr;
    const int64_t row0 = g.rows == 1 || !placed ? 0 : begin / g.cols, col0 = begin - row0 * g.cols;
    const int tid = threadIdx.x;
    if (g.layout == kRows && g.cols < (int64_t)1 << 26) {  // vectors of a row and of a chunk: less than 2^24
        const int per = (int)(g.cols >> 3), v0 = (int)(col0 >> 3), left = (int)min((size - begin) >> 3, (int64_t)kChunk / 8);
        const float inv = 1.f / (float)per;
        const T* from = x + row0 * g.ld;
        T* to = y + row0 * g.ldo;
        const uint8_t* keep =  // a byte a vector
            g.mask == nullptr ? nullptr : reinterpret_cast<const uint8_t*>(g.mask + row0 * words);
        Eight<T> v[kUnroll];
        Vector p[kUnroll];
        uint32_t bits[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int n = u * kThreads + tid;
            v[u].clear();
            bits[u] = 0xFFu;
            p[u] = vector_of(v0 + n, per, inv);
            if (n >= left) continue;
            v[u].load(from, p[u].row * g.ld + 8 * p[u].at, (int64_t)1 << 60, true);
            if (g.mask != nullptr) bits[u] = keep[p[u].row * (4 * words) + p[u].at];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (SCALE) scale(v[u], f);
            if (g.mask != nullptr) v[u].keep(bits[u]);
            if constexpr (!SCALE) {
                *sum += squares(v[u]);
            } else if (u * kThreads + tid < left) {
                store_last(v[u], to + p[u].row * g.ldo + 8 * p[u].at);
            }
        }
        return;
    }
    if (g.layout == kFlat) {
        Eight<T> v[kUnroll];
        uint32_t bits[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t at = begin + 8 * (u * kThreads + tid);
            v[u].clear();
            bits[u] = 0xFFu;
            if (at >= size) continue;
            if (g.mask != nullptr) {
                const Place p = place_of(row0, col0, at - begin, g.cols);
                const uint32_t* row = g.mask + p.row * words;
                bits[u] = mask_bits(row, words, p.col);
                const int here = (int)min(g.cols - p.col, (int64_t)8);  // the others lie in the next row
                if (here < 8) {
                    bits[u] &= (1u << here) - 1u;
                    if (p.row + 1 < g.rows) bits[u] |= mask_bits(row + words, words, 0) << here;
                }
            }
            v[u].load(x, at, size, true);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t at = begin + 8 * (u * kThreads + tid);
            if (SCALE) scale(v[u], f);
            if (g.mask != nullptr) v[u].keep(bits[u]);
            if constexpr (!SCALE) {
                *sum += squares(v[u]);
            } else if (at + 8 <= size) {
                store_last(v[u], y + at);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (at + i >= size) continue;
                    if constexpr (sizeof(T) == 2) y[at + i] = (uint16_t)(v[u].w[i >> 1] >> (16 * (i & 1)));
                    else y[at + i] = bits_float(v[u].w[i]);
                }
            }
        }
        return;
    }
    const int64_t end = min(size - begin, (int64_t)kChunk);
    for (int64_t near = tid; near < end; near += kThreads) {
        const Place p = place_of(row0, col0, near, g.cols);
        const bool keep = g.mask == nullptr || ((g.mask[p.row * words + (p.col >> 5)] >> (p.col & 31)) & 1u) != 0u;
        const T* from = x + p.row * g.ld + p.col;
        if constexpr (SCALE) {
            y[p.row * g.ldo + p.col] = scaled_one(from, keep, f);
        } else if (keep) {
            double v;
            if constexpr (sizeof(T) == 2) v = widen(*from);
            else v = *from;
            *sum = __builtin_fma(v, v, *sum);
        }
    }
}

// Sum over the workgroup, in one order; every thread gets it.
__device__ __forceinline__ double sum_all(double v, double* lds) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += lds[w];
    return s;
}
__device__ __forceinline__ double sum_of(const double* sums, int n, double* lds) {
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) v += sums[i];
    return sum_all(v, lds);
}

template <bool SCALE>
__device__ __forceinline__ void walk(const GradList& list, float f, double* sum) {
    // The last chunks read by the sums are the first to be scaled: the last-level cache still has them.
    int i = SCALE ? list.count - 1 : 0;
    for (int n = blockIdx.x; n < list.chunks; n += gridDim.x) {
        const int c = SCALE ? list.chunks - 1 - n : n;
        while (!SCALE && i + 1 < list.count && list.job[i + 1].first <= c) ++i;
        while (SCALE && list.job[i].first > c) --i;
        const GradJob& g = list.job[i];
        const int64_t begin = (int64_t)(c - g.first) * kChunk;
        if (SCALE && f == 1.f && g.mask == nullptr && g.grad == g.out) continue;  // nothing changes
        if (g.bf16) chunk<uint16_t, SCALE>(g, begin, f, sum);
        else chunk<float, SCALE>(g, begin, f, sum);
    }
}

__global__ __launch_bounds__(kThreads) void grad_squares_kernel(const GradList list, double* sums) {
    __shared__ double lds[kWaves];
    double sum = 0.0;
    walk<false>(list, 1.f, &sum);
    sum = sum_all(sum, lds);
    if (threadIdx.x == 0) sums[blockIdx.x] = sum;
}

__global__ __launch_bounds__(kThreads) void grad_finish_kernel(const double* sums, int n, float* norm) {
    __shared__ double lds[kWaves];
    const double s = sum_of(sums, n, lds);
    if (threadIdx.x == 0) *norm = (float)__builtin_sqrt(s);
}

__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const GradList list, const double* sums, int n,
                                                              float max_norm, float* norm) {
    __shared__ double lds[kWaves];
    const double s = __builtin_sqrt(sum_of(sums, n, lds));
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)s;
    // not "s > max_norm": a NaN norm gives NaN
    const float f = s <= (double)max_norm ? 1.f : (float)((double)max_norm / s);
    double none = 0.0;
    walk<true>(list, f, &none);
}

}  // namespace

int grad_chunk() { return kChunk; }

int launch_grad_squares(const GradList& list, int blocks, double* sums, void* stream) {
    hipLaunchKernelGGL(grad_squares_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, (hipStream_t)stream, list, sums);
    return (int)hipGetLastError();
}
int launch_grad_finish(const double* sums, int n, float* norm, void* stream) {
    hipLaunchKernelGGL(grad_finish_kernel, dim3(1), dim3(kThreads), 0, (hipStream_t)stream, sums, n, norm);
    return (int)hipGetLastError();
}
int launch_grad_scale(const GradList& list, int blocks, const double* sums, int n, float max_norm, float* norm,
                      void* stream) {
    hipLaunchKernelGGL(grad_scale_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, (hipStream_t)stream, list, sums, n,
                       max_norm, norm);
    return (int)hipGetLastError();
}

}  // namespace tsenor
