// Which kernel of mxfp4.hip a product runs in, and the workspace that follows
// from it.  Host code without HIP types, so that it can be compiled alone.
//
// The kernels are shaped like those of the int8 product, a byte of codes for a
// byte, and so are the forms (Int8Choice); the estimates are their own.
#pragma once

#include "int8_choice.h"

namespace kbit {

// Tiles of kPairedRows rows and channels take their scales in the order of pairs
// of steps.
constexpr int kPairedRows = 256;

// The least of estimated times, in microseconds, fitted to 200 shapes spread over
// M = 1 .. 8192 and N, K = 64 .. 16384 in every form, operands from memory; what
// the rule picks was 1.8% slower than the fastest form on average, 27% at most
// (4170 x 810 x 298: 9.8 us in tiles of 128, 7.7 in 64).  Both sides: 77 x 11008 x 4096
// 14.1 us in 80 x 48 pieces of few rows, 16.5 in tiles of 32; 512 x 4096 x 4096 9.9 in
// tiles of 64, 12.2 in 128; 2048 x 4096 x 4096 23.5 in 128, 30.1 in 64; 666 x 3328 x 11520 39
// in 3 parts of the depth, 48 in one.
struct MxTile {
    int bm, bn;
    // us: a launch; 10 MB of operands; where every workgroup has a compute unit of
    // its own a step, and with all of them at work more, and a workgroup's rest;
    // where they share one a step and the rest, a round; the weight of whole
    // rounds against parts of one
    double base, operands, step, step_all, rest_all, step_round, rest_round, whole;
};
constexpr MxTile kMxTiles[] = {{32, 128, 3.59, 1.83, 0.321, -0.225, 3.25, 0.332, 0.95, 0.75},
                               {64, 128, 5.12, 0.39, 0.303, 0.202, 1.01, 0.467, 1.33, 0.37},
                               {128, 128, 6.20, 1.86, 0.410, 0.179, 1.29, 0.464, 1.80, 0.31},
                               {256, 256, 5.00, 3.63, 1.041, 0.0, 8.27, 1.041, 8.27, 0.99}};
// Parts of the depth: the second launch, and 10 MB of the parts' sums.
constexpr double kMxPartsLaunch = 3.3, kMxPartsSums = 2.6;

inline double mx_tile_us(const MxTile& t, int64_t tiles, int64_t cus, double steps, double operands) {
    const double all = static_cast<double>(tiles) / cus;
    if (t.bm < kPairedRows && tiles <= cus)
        return t.base + t.operands * operands + (t.step + t.step_all * all) * steps + t.rest_all * all;
    const double r = rounds_of(tiles, cus, t.whole);
    return t.base + t.operands * operands + t.step_round * r * steps + t.rest_round * r;
}

// K: bytes of a row of codes.
inline Int8Choice mx_choose(int64_t M, int N, int K, int64_t cus) {
    Int8Choice best{};
    double least = 1e30;
    const double operands = 1e-7 * (static_cast<double>(M) + N) * K;
    for (const Int8Few& f : kFew) {
        if (f.mt > 5) continue;  // not built here: tiles were faster wherever they fit
        const double us = 1.93 + 1.31 * operands +
                          rounds_of(tiles_of(M, N, 16 * f.mt, 16 * f.tn), cus, 1.0) *
                              (2.69 + 0.173 * f.mt * f.tn + 1.88e-5 * 16.0 * (f.mt + f.tn) * K);
        if (us < least) {
            least = us;
            best = Int8Choice{f, 0, 1};
        }
    }
    const double steps = (K + kDepth - 1) / kDepth;
    for (const MxTile& t : kMxTiles) {
        if (M < t.bm || N < t.bn) continue;
        const int64_t tiles = tiles_of(M, N, t.bm, t.bn);
        const double us = mx_tile_us(t, tiles, cus, steps, operands);
        if (us < least) {
            least = us;
            best = Int8Choice{{}, t.bm, 1};
        }
        if (t.bm != kSplitTile) continue;
        for (const int n : kParts) {
            const int depth = split_depth(K, n), parts = (K + depth - 1) / depth;
            if (parts < 2 || tiles * parts > 2 * cus) continue;
            const double split = mx_tile_us(t, tiles * parts, cus, depth / kDepth, operands) + kMxPartsLaunch +
                                 kMxPartsSums * 4e-7 * static_cast<double>(parts) * M * N;
            if (split < 0.97 * least) {  // it takes memory
                least = split;
                best = Int8Choice{{}, t.bm, parts};
            }
        }
    }
    return best;
}

// Whether the product takes the scales of both operands in the order of pairs
// of steps, so that a caller that quantizes them may write them so.
inline bool mx_paired(int64_t M, int64_t N, int K) {
    return M >= 1 && M <= kRowBlock && N <= kMaxChannels &&
           mx_choose(M, static_cast<int>(N), K, device_cu_count()).bm == kPairedRows;
}

// Bytes of scales in that order.
inline int64_t mx_paired_bytes(int64_t rows, int K) { return rows * ((K + 2 * kDepth - 1) / (2 * kDepth)) * 16; }

// Bytes of workspace of a product on the current device: the sums of parts of
// the depth, or scales that are not paired yet.
inline int64_t mx_product_workspace(int64_t M, int N, int K, bool x_paired = false, bool w_paired = false) {
    const int64_t cus = device_cu_count();
    int64_t most = 0;
    // the blocks' sizes: whole ones and what is left
    for (const int64_t m : {M < kRowBlock ? M : kRowBlock, M % kRowBlock})
        for (const int64_t n : {N < kMaxChannels ? N : kMaxChannels, N % kMaxChannels}) {
            if (m == 0 || n == 0) continue;
            const Int8Choice c = mx_choose(m, static_cast<int>(n), K, cus);
            int64_t need = c.parts > 1 ? c.parts * m * sums_ld(static_cast<int>(n)) * 4 : 0;
            if (c.bm == kPairedRows)
                need = (x_paired ? 0 : mx_paired_bytes(m, K)) + (w_paired ? 0 : mx_paired_bytes(n, K));
            if (need > most) most = need;
        }
    return most;
}

// No less than that for any number of rows up to M, and never less for more
// rows (the sums of parts are bounded as for int8: at most two workgroups a
// compute unit).
inline int64_t mx_product_workspace_up_to(int64_t M, int N, int K) {
    const int64_t sums = int8_product_workspace_up_to(M, N, K);
    if (M < kPairedRows || N < kPairedRows) return sums;
    const int64_t scales = mx_paired_bytes((M < kRowBlock ? M : kRowBlock) + (N < kMaxChannels ? N : kMaxChannels), K);
    return scales > sums ? scales : sums;
}

}  // namespace kbit
