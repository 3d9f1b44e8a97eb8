// tsenor_grouped_forms.h -- which kernel of tsenor_grouped.hip takes a product, by what the host knows of
// it: sizes, strides and alignment.  Apart from the kernels, so that it can be looked at without a GPU.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "tsenor_ops_internal.h"

namespace tsenor {

// Times here are of graphs that take three to twelve inputs in turn, more than the last-level cache holds.

enum Kind { kProduct, kGradient };

// kFew64, kFew32, kFew16: 16 rows and that many columns a workgroup; kFew32x32: 32 of both; kStaged256x128:
// rows that are not 16-byte aligned, through registers; kAny: any alignment and size; the others: tiles fed
// by direct loads (columns x rows).
enum Form { kFew64, kFew32, kFew16, kFew32x32, kAny, kStaged256x128, k256x256, k256x128, k128x128, k64x64 };

constexpr int64_t kCus = 256;
constexpr int64_t kMaxRow = int64_t(1) << 23;  // bytes of a row: offsets inside a tile fit 32 bits

// LDS of a tile's kernel whose workgroups walk over tiles: the ring (64 bytes of each row and column), the
// experts' rows, and for a weight gradient two sets of its tile's mask words.
constexpr int64_t kLdsOfCu = 160 * 1024;
constexpr int64_t kMostExperts = 1024, kRowTableBytes = 3 * (kMostExperts + 1) * 4, kExpertRowsBytes = (kMostExperts + 64) * 4;
constexpr int64_t tile_lds(Kind kind, int columns, int rows, int ring) {
    return 64 * (int64_t)(columns + rows) * ring +
           (kind == kProduct ? kRowTableBytes : kExpertRowsBytes + 2 * rows * (columns / 32) * 4);
}
// Workgroups of a CU at one time: 2 of 64 x 64, 1 of the others.  (Two of the staged 256 x 128 tile, whose ring
// alone would let them in, run one after the other, each with half of the tiles: 16384 rows of 8 experts 11009 x
// 4095 3210 us, one 2960; 8192 rows of 16 4095 x 2047 398, 385; 2000 rows 11009 x 4095 340, 345.)
constexpr int64_t at_once(Kind kind, int columns, int rows, int ring) {
    return kLdsOfCu / tile_lds(kind, columns, rows, ring);
}

// Direct loads take 16 bytes of an aligned row at a time.
inline bool direct(const void* p, int64_t ld, int64_t stride, int64_t width) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0 && stride % 16 == 0 && width % 16 == 0;
}

// Tiles of a launch, as far as the host can know: a little more than half a tile counted for each expert.
template <Kind K>
int64_t tiles_of(const GroupedJob& job, int64_t m, int64_t n) {
    const int64_t across = (job.inner + m - 1) / m;
    return across * (K == kGradient ? (job.outer + n - 1) / n * job.experts
                                    : (job.rows + n - 1) / n + (job.ends != nullptr ? job.experts * 9 / 16 : 0));
}

// The tile whose rounds of workgroups take the least time.  Measured, hundredths of a microsecond for a step
// (64 bytes of the reduction) of one round: 256 x 256: 60; 256 x 128: 43; 128 x 128: 31; 64 x 64: 19 with one
// workgroup on a CU, 28 with two (weight gradients: 27 and, with four, 50).  (One or two inputs in turn, which the
// last-level cache holds: what a step costs.)  Examples (us), in that order: 1542 rows 2048 x 5952 122 / 100 / 69 / 111;
// 600 rows 8192 x 4096 87 / 78 / 95 / 110; 600 rows of 16 experts 2048 x 4096 95 / 90 / 71 / 80; 1003 rows 103 / 92 / 92 / 85,
// where the rule takes the second; 2048 rows 112 / 96 / 108 / 127; 4096 rows 115 / 155 / 147 / 210; data gradients, 200
// rows of 8 experts 2048 x 4096 68 / 60 / 44 / 38; 16384 rows of 8 experts 11008 x 4096 1268 / 1681 / 2053 / 4168.
// A weight gradient's reduction is short, so that beginning and ending a tile counts too: 7, 6 and 4 us a round, and
// 4 and 2.5 us once with a ring of more than 64 KB; where each workgroup has one tile, the largest expert's
// rows count (taken as 1.6 times the mean), else a third of what they exceed it by.  Examples, 256 x 256 / 128 x
// 128 / 64 x 64: 8192 rows 2048 x 2048 166 / 88 / 154; experts 1024 x 1024, 1024 rows of 4: 19 / 13 / 9, 4096 rows of
// 8: 30 / 24 / 22, 8000 rows: 49 / 37 / 44, 8192 rows of 16: 42 / 44 / 50; 2048 rows of 16 experts 2048 x 2048 47 / 97 / 83.
template <Kind K>
Form pick_tile(const GroupedJob& job) {
    const auto rounds = [&](int64_t m, int64_t n, int64_t at_once) {
        return (tiles_of<K>(job, m, n) + at_once - 1) / at_once;
    };
    const double steps = K == kGradient ? job.rows / (32. * job.experts) : 1.;
    const auto cost = [&](int64_t count, double step, double begin, double once) {
        if (K == kProduct) return count * step;
        return count * (step * steps * (job.experts == 1 ? 1. : count == 1 ? 1.6 : 1.2) + begin) + once;
    };
    Form best = k256x256;
    double least = cost(rounds(256, 256, kCus), 60, 700, 400);
    const auto take = [&](Form tile, double cost) {
        if (cost < least) {
            best = tile;
            least = cost;
        }
    };
    if (K == kProduct) take(k256x128, cost(rounds(256, 128, kCus), 43, 0, 0));
    take(k128x128, cost(rounds(128, 128, kCus), 31, 600, 250));
    const int64_t small = tiles_of<K>(job, 64, 64);
    if (K == kProduct) take(k64x64, small <= kCus ? 19. : std::max(28., 28. * small / (2 * kCus)));  // not in rounds
    else if (small <= kCus) take(k64x64, 27 * steps + 400);
    else take(k64x64, rounds(64, 64, 4 * kCus) * (50 * steps + 400));  // a CU's four have different experts' rows
    return best;
}

template <Kind K, bool AT, bool BT>
Form pick_form(const GroupedJob& job, int size) {  // size: bytes of an operand's entry
    if (K == kProduct && !AT) {
        // Few rows: on average up to eight an expert, or up to 64 where tiles would leave CUs without work.
        // Measured (us), 16 columns a wave / 64 x 64 tiles: 6 rows of 64 experts 1408 x 2048: 12 / 17; 64 rows:
        // 49 / 52; 512 rows: 72 / 82; 64 rows of 16 experts 2048 x 4096: 52 / 58; 16 rows 11008 x 4096: 25 / 26; 64 rows
        // 4096 x 4096 19 / 29, 11008 x 4096 50 / 32.  The host knows the average only: where all 512 rows are one of
        // the 64 experts', its weights are read again for each 16 rows, and tiles would be faster: 31 / 17.  As many
        // columns as leave 160 workgroups: one row 4096 x 4096 in 10 / 14 / 21 for 16 / 32 / 64; 16 rows 11008 x 4096 in
        // 29 / 30 / 25.
        const int64_t parts = job.ends != nullptr ? std::min<int64_t>(job.rows, job.experts) : 1;
        if (job.rows <= 16 || job.rows <= 8 * (int64_t)job.experts) {
            if ((job.inner + 63) / 64 * parts >= 160) return kFew64;
            if ((job.inner + 31) / 32 * parts >= 160) return kFew32;
            return kFew16;
        }
        if (job.rows <= 64 && tiles_of<K>(job, 64, 64) < 128) return kFew32x32;
    }
    if (size == 2) {  // 8-bit integers are aligned, and their rows short
        // tiles count rows, columns and the bytes between rows in 32 bits
        if (job.inner > (K == kGradient ? 1 << 26 : 0x7FFFFF00) || job.outer > 0x7FFFFF00 || job.lda >= kMaxRow ||
            job.ldb >= kMaxRow)
            return kAny;
        const int64_t as = (K == kGradient || job.experts == 1) ? 0 : job.astride;
        if (!direct(job.a, job.lda, as, AT ? job.inner * size : job.kbytes) ||
            !direct(job.b, job.ldb, 0, BT ? job.outer * size : job.kbytes)) {
            // Tiles of 64 x 64 / 256 x 128 (us): 16384 rows of 8 experts 11009 x 4095: 5860 / 2990; 1003 rows of 16
            // experts 2047 x 4095: 137 / 158; column-contiguous operands, 8192 rows of 16 experts 4095 x 2047, one input:
            // 764 / 829, weight gradients 739 / 800 (with many inputs 806 and 696 by 64 x 64).
            return !AT && !BT && tiles_of<K>(job, 256, 128) >= 160 ? kStaged256x128 : kAny;
        }
    }
    return pick_tile<K>(job);
}

}  // namespace tsenor
