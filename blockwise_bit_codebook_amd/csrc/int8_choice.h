// Which kernel of int8.hip a product of int8 codes runs in, and what follows
// from it for the caller: the limits of the one-kernel form for tokens and the
// workspace.  Host code without HIP types, so that it can be compiled alone.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "kbit_internal.h"

namespace kbit {

// Codes of a row a step of the product.
constexpr int kDepth = 128;

// Blocks of rows and channels, a launch each, keep the grids (below 2^32
// threads) and the kernels' 32-bit offsets in range.
constexpr int64_t kRowBlock = int64_t(1) << 15;
constexpr int64_t kFarRows = int64_t(1) << 22;  // bytes between rows
constexpr int64_t kMaxChannels = int64_t(1) << 20;

// Tokens quantized inside the product's kernel: a wave takes 512 values of a
// row at a time, at most kItems times, and the codes stay in LDS.
constexpr int kItems = 4;
constexpr int kTokenBytes = 28 * 1024;  // of codes, rows kTokenPad apart from whole steps
constexpr int kTokenPad = 16;
constexpr int kMaxTokens = 8;

// Whether M tokens fit.
inline bool int8_tokens_fit(int64_t M, int N, int K, int64_t ldw) {
    if (M > kMaxTokens || N > kMaxChannels || (N > 1 && ldw >= kFarRows)) return false;
    const int64_t per_row = (K + 511) / 512, steps = (K + kDepth - 1) / kDepth;
    return M * (steps * kDepth + kTokenPad) <= kTokenBytes && M * per_row <= 8 * kItems;
}

constexpr int kSplitTile = 128;  // rows and channels of the tiles whose depth may be in parts

// Sums of one part: rows of whole 16-byte pieces.
inline int64_t sums_ld(int N) { return (static_cast<int64_t>(N) + 3) / 4 * 4; }

// Depth of a part: whole pairs of steps.
inline int split_depth(int K, int parts) {
    const int pairs = (K + 2 * kDepth - 1) / (2 * kDepth);
    return (pairs + parts - 1) / parts * 2 * kDepth;
}

// Which kernel and tile: the least of estimated times, in microseconds.  The
// estimates were fitted to 2100 measurements, every variant at 130 shapes
// spread over M = 1 .. 8192 and N, K = 64 .. 16384 with operands from memory
// and from cache: what the rule picked was 0.7% slower than the fastest variant
// on average, 11% at most.  (Since then few rows join 1 us faster, the ends of
// 256 x 256 rounds and partial steps 1 to 3 us; measured again over 140 shapes
// the rule is within 4% on average, 23% at most.)  Both sides of it, as fitted
// (operands from memory): 77 x 11008 x 4096 18.3 us in 80 x 48 and 19.7 us in 80 x 64 pieces of
// few rows, 26.7 in tiles of 32 x 128; 112 x 11008 x 4096 20.6 in 112 x 48 pieces,
// 25.5 in 80 x 48 and 29.4 in tiles; 500 x 4099 x 3840 27.1 in tiles of 64 x
// 128, 27.3 in 32 x 128, 30.1 in 80 x 64 pieces, 31.7 in 128 x 128; 4096 x 4096 x
// 4096 58.8 in 256 x 256, 71.5 in 128 x 128.
struct Int8Few {
    int mt, tn;
};
struct Int8Tile {
    int bm, bn;
    // us: a launch, a step alone, a step a round, a round, a partial step, 10
    // MB of operands; the weight of whole rounds against parts of one
    double base, least, step, round, tail, operands, whole;
};
constexpr Int8Few kFew[] = {{1, 1}, {1, 2}, {1, 3}, {1, 4}, {2, 2}, {2, 4}, {3, 2}, {3, 4}, {4, 4},
                             {5, 3}, {5, 4}, {7, 3}, {8, 3}};
constexpr Int8Tile kTiles[] = {{32, 128, 0.84, 0.497, 0.253, 1.08, 2.32, 1.29, 0.255},
                               {64, 128, 0.0, 0.572, 0.382, 1.85, 3.01, 1.07, 0.454},
                               {128, 128, 0.0, 0.799, 0.544, 2.70, 3.31, 0.11, 0.742},
                               {256, 256, 0.0, 1.189, 1.386, 7.47, 2.93, 0.83, 1.0}};

// Parts of the depth, in 128 x 128: where the tiles alone leave compute units
// idle or half a round empty and the depth is long.  us: the second launch, and
// 10 MB of the parts' sums.  Measured on 70 shapes with 32, 64, 128 and 256
// rows: 128 alone gives what all of them give within 1%.  Without and with parts
// (operands from memory): 512 x 4096 x 11008 54.2 and 45.1 us in 4, 1024 x 2048 x
// 8192 51.5 and 34.1 in 4, 562 x 2432 x 11776 51.5 and 35.2 in 4, but 256 x 4096 x
// 4096 15.3 and 20.0, 1024 x 1024 x 4096 13.3 and 18.1.  At most as many workgroups
// as are resident at once, two a compute unit: 4778 x 857 x 13738 would take 126 us
// without and 146 in 2 parts (532 workgroups).
constexpr int kParts[] = {2, 3, 4, 8};
constexpr int64_t kMostParts = 8;
constexpr double kPartsLaunch = 4.5, kPartsSums = 1.5;

struct Int8Choice {
    Int8Few few;  // or
    int bm;       // tiles of bm rows, where not 0
    int parts;    // of the depth; 1: no split
};

// Workgroups a compute unit: a part of a round is cheaper than a whole one
// where several workgroups fit a compute unit (whole < 1).
inline int64_t tiles_of(int64_t M, int64_t N, int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }
inline double rounds_of(int64_t tiles, int64_t cus, double whole) {
    const double r = whole * static_cast<double>((tiles + cus - 1) / cus) + (1.0 - whole) * tiles / cus;
    return r < 1.0 ? 1.0 : r;
}

inline Int8Choice choose_form(int64_t M, int N, int K, int64_t cus) {
    Int8Choice best{};
    double least = 1e30;
    const double operands = 1e-7 * (static_cast<double>(M) + N) * K;
    for (const Int8Few& f : kFew) {
        if (f.mt > 5 && M > 16 * f.mt) continue;  // made to read the weights once
        const double us = 1.34 + 0.68 * operands +
                          rounds_of(tiles_of(M, N, 16 * f.mt, 16 * f.tn), cus, 1.0) *
                              (1.783 + 0.204 * f.mt * f.tn + 1.297e-5 * 16.0 * (f.mt + f.tn) * K +
                               (K % kDepth ? 0.286 * (f.mt + f.tn) : 0.0));
        if (us < least) {
            least = us;
            best = Int8Choice{f, 0, 1};
        }
    }
    const int rest = K % (2 * kDepth);
    const double steps = K / (2 * kDepth) * 2 + (rest > 0 ? 1 : 0) + (rest > kDepth ? 1 : 0);
    for (const Int8Tile& t : kTiles) {
        if (M < t.bm || N < t.bn) continue;
        const int64_t tiles = tiles_of(M, N, t.bm, t.bn);
        const double r = rounds_of(tiles, cus, t.whole);
        const double us = t.base + (t.step * r > t.least ? t.step * r : t.least) * steps + t.round * r +
                          (K % kDepth ? t.tail : 0.0) + t.operands * operands;
        if (us < least) {
            least = us;
            best = Int8Choice{{}, t.bm, 1};
        }
        if (t.bm != kSplitTile) continue;
        for (const int n : kParts) {
            const int depth = split_depth(K, n), parts = (K + depth - 1) / depth;
            if (parts < 2 || tiles * parts > 2 * cus) continue;
            const double rp = rounds_of(tiles * parts, cus, t.whole);
            const double split = t.base + (t.step * rp > t.least ? t.step * rp : t.least) * (depth / kDepth) +
                                 t.round * rp + t.operands * operands + kPartsLaunch +
                                 kPartsSums * 4e-7 * static_cast<double>(parts) * M * N;
            if (split < 0.95 * least) {  // it takes memory
                least = split;
                best = Int8Choice{{}, t.bm, parts};
            }
        }
    }
    return best;
}

// Bytes that the parts' sums of a product take on the current device.
inline int64_t int8_product_workspace(int64_t M, int N, int K) {
    const int64_t cus = device_cu_count();
    int64_t most = 0;
    // the blocks' sizes: whole ones and what is left
    for (const int64_t m : {M < kRowBlock ? M : kRowBlock, M % kRowBlock})
        for (const int64_t n : {N < kMaxChannels ? N : kMaxChannels, N % kMaxChannels}) {
            if (m == 0 || n == 0) continue;
            const Int8Choice c = choose_form(m, static_cast<int>(n), K, cus);
            const int64_t need = c.parts > 1 ? c.parts * m * sums_ld(static_cast<int>(n)) * 4 : 0;
            if (need > most) most = need;
        }
    return most;
}

// No less than that for any number of rows up to M, and never less for more
// rows, so that one buffer serves all batches: at most two workgroups a compute
// unit, each with the sums of one tile (64 KB).
inline int64_t int8_product_workspace_up_to(int64_t M, int N, int K) {
    const int64_t cus = device_cu_count(), pairs = (static_cast<int64_t>(K) + 2 * kDepth - 1) / (2 * kDepth);
    if (M < kSplitTile || pairs < 2) return 0;
    const int64_t rows = M < kRowBlock ? M : kRowBlock, parts = pairs < kMostParts ? pairs : kMostParts;
    int64_t most = 0;
    for (const int64_t n : {N < kMaxChannels ? N : kMaxChannels, N % kMaxChannels}) {
        if (n < kSplitTile || (n + kSplitTile - 1) / kSplitTile > cus) continue;  // too many for two parts of one row of tiles
        const int64_t all = parts * rows * sums_ld(static_cast<int>(n)), tiles = 2 * cus * kSplitTile * kSplitTile;
        const int64_t need = 4 * (all < tiles ? all : tiles);
        if (need > most) most = need;
    }
    return most;
}

// Workspace of the dynamic form: the codes, their scales, the product's own.
// Its rows of codes are whole cache lines, so that no step of 128 codes lies
// across two.
inline int64_t dynamic_ld(int32_t K) { return (static_cast<int64_t>(K) + kDepth - 1) / kDepth * kDepth; }
struct DynamicParts {
    int64_t scale, product;  // where they start
};
inline DynamicParts dynamic_parts(int64_t M, int32_t K) {
    DynamicParts w;
    w.scale = M * dynamic_ld(K);
    w.product = w.scale + (4 * M + 15) / 16 * 16;
    return w;
}

}  // namespace kbit
