// Microscaled 4-bit floating point (MXFP4) for gfx950: rows and columns to
// codes, codes to values, and the product of two coded matrices.
//
//   block    32 values along a row; e = max(floor(log2(max |x|)) - 2, -127), held
//            as the byte e + 127; code = x / 2^e rounded to the nearest of 0,
//            1/2, 1, 3/2, 2, 3, 4, 6 (ties to the even code, at most 6) and a
//            sign.  A block with a NaN or an infinity has the byte 255, which is
//            NaN, and codes 0.  Values past a row's end are codes 0.
//   codes    two a byte, the first in the low half, 16 bytes a block.
//   product  acc[m][n] = sum over blocks b of 2^(xs + ws) sum over k in b of
//            x[m][k] w[n][k], in fp32 on the matrix cores, out = RN_T(acc + bias).
#include "kbit_internal.h"
#include "launch.h"
#include "matrix.h"
#include "mx_internal.h"

#include <type_traits>

namespace kbit {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// values to codes
// ---------------------------------------------------------------------------
// The scale byte of a block from the bits of its largest magnitude (ordered
// like the magnitudes, with NaN above infinity above the rest).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : max(e, 2u) - 2u;
}

// The converters take the scale's exponent from a float's bits and round half
// to even, at most 6; PLACE is the byte of the word that two codes go to.
template <class E, int PLACE>
__device__ __forceinline__ uint32_t pack2(uint32_t word, uint32_t two, float scale) {
    if constexpr (std::is_same<E, QB16>::value)
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(bf16x2, two), scale, PLACE);
    else
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, __builtin_bit_cast(f16x2, two), scale, PLACE);
}
template <int PLACE>
__device__ __forceinline__ uint32_t pack2(uint32_t word, float a, float b, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, a, b, scale, PLACE);
}

// Largest magnitudes of both halves of two words of 16-bit values, whose bits
// are ordered like the magnitudes, with NaN above infinity above the rest.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
constexpr uint32_t kAbs16x2 = 0x7FFF7FFFu, kAbs32 = 0x7FFFFFFFu;

// The bits of a 16-bit magnitude as fp32.
template <class E>
__device__ __forceinline__ uint32_t wide_bits(uint32_t half) {
    return __float_as_uint(E::one(static_cast<uint16_t>(half)));
}

// The scale byte of a lane's 8 neighbouring values, four lanes a block, and
// their codes (0 where the block is not finite).
template <class E>
__device__ __forceinline__ uint32_t row_byte(const u32x4 (&r)[E::kVec]) {
    uint32_t m;
    if constexpr (sizeof(typename E::T) == 4) {
        m = r[0][0] & kAbs32;
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, r[i / 4][i % 4] & kAbs32);
    } else {
        m = max16x2(max16x2(r[0][0] & kAbs16x2, r[0][1] & kAbs16x2), max16x2(r[0][2] & kAbs16x2, r[0][3] & kAbs16x2));
        m = wide_bits<E>(max(m & 0xFFFFu, m >> 16));
    }
    m = max(m, dpp_u32<kDppXor1>(m));
    m = max(m, dpp_u32<kDppXor2>(m));
    return scale_byte(m);
}
template <class E>
__device__ __forceinline__ uint32_t row_codes(const u32x4 (&r)[E::kVec], uint32_t byte) {
    const float s = __uint_as_float(byte << 23);
    uint32_t q = 0;
    if constexpr (sizeof(typename E::T) == 4) {
        q = pack2<0>(q, __uint_as_float(r[0][0]), __uint_as_float(r[0][1]), s);
        q = pack2<1>(q, __uint_as_float(r[0][2]), __uint_as_float(r[0][3]), s);
        q = pack2<2>(q, __uint_as_float(r[1][0]), __uint_as_float(r[1][1]), s);
        q = pack2<3>(q, __uint_as_float(r[1][2]), __uint_as_float(r[1][3]), s);
    } else {
        q = pack2<E, 0>(q, r[0][0], s);
        q = pack2<E, 1>(q, r[0][1], s);
        q = pack2<E, 2>(q, r[0][2], s);
        q = pack2<E, 3>(q, r[0][3], s);
    }
    return byte == 255u ? 0u : q;
}

// Where the scale of a block of a row stands.
__device__ __forceinline__ int pair_place(int block) {  // of its 16 bytes, see pair_order
    return 2 * (block & 6) + (block & 8) / 4 + (block & 1);
}
__device__ __forceinline__ uint8_t* scale_place(const MxCoded& c, int64_t row, int64_t block) {
    return c.paired ? c.scales + (block >> 4) * c.lds + row * 16 + pair_place(static_cast<int>(block & 15))
                    : c.scales + row * c.lds + block;
}

// Rows: 8 values a lane, four lanes a block, kRowItems pieces of 512 values a
// wave on their way together.  Piece i of all rows: row i / per_row.  Memory
// bounds it: 8192 x 11008 bf16 43.3 us (5.3 TB/s), 8192 x 4096 18.4; two pieces 43.1.
// Codes stored past the caches take 2 us less here and 2 more in the product that
// reads them.
constexpr int kRowItems = 4;
template <class E>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const typename E::T* __restrict__ X, uint32_t items,
                                                               uint32_t per_row, int d, int64_t ldx,
                                                               const MxCoded out) {
    const int lane = __lane_id();
    const uint32_t first = (blockIdx.x * kWavesPerGroup + threadIdx.x / kWave) * kRowItems;
    const int end = (d + kMxBlock - 1) / kMxBlock * kMxBlock;
    u32x4 v[kRowItems][E::kVec];
    uint32_t rows[kRowItems];
    int cols[kRowItems];
    uint32_t row = first / per_row, at = first - row * per_row;
#pragma unroll
    for (int i = 0; i < kRowItems; ++i) {
        rows[i] = row;
        cols[i] = first + i < items ? static_cast<int>(at) * 512 + lane * 8 : end;
        if (cols[i] < end) load8_raw<E>(X + row * ldx, cols[i], d, v[i]);
        if (++at == per_row) {
            at = 0;
            ++row;
        }
    }
#pragma unroll
    for (int i = 0; i < kRowItems; ++i) {
        if (cols[i] < end) {  // end is a whole number of blocks: quads stay together
            const uint32_t byte = row_byte<E>(v[i]);
            *reinterpret_cast<uint32_t*>(out.codes + rows[i] * out.ldc + cols[i] / 2) = row_codes<E>(v[i], byte);
            if ((lane & 3) == 0) *scale_place(out, rows[i], cols[i] / kMxBlock) = static_cast<uint8_t>(byte);
        }
    }
}

// Columns, and rows in the same pass: a workgroup takes 8 blocks of 32 rows, a
// wave each, and 64 kCols columns.  A lane has kCols columns of its block, 8
// bytes of a row, so that a column's maximum needs no other lane and a row's a
// few neighbours; the columns' codes cross LDS so that they leave as whole
// cache lines.  sums: the columns' sums over the workgroup's rows.  8192 x 4096
// bf16 18.8 us (4.5 TB/s), fp32 27.5 (5.5); with the rows in the same reading 25 against
// 37 in two.
constexpr int kColBlocks = 8;
template <class E>
constexpr int kCols = 8 / sizeof(typename E::T);

// The matrices of a launch, their workgroups one after the other: those of job
// i are the ones below end[i] that job i - 1 leaves, `across` of them abreast.
struct ColumnJobs {
    MxColumns job[kMxColumnJobs];
    uint32_t end[kMxColumnJobs], across[kMxColumnJobs];
};

template <class E, bool ROWS>
__global__ __launch_bounds__(kColBlocks* kWave) void mx_quantize_columns_kernel(const ColumnJobs jobs, uint32_t first) {
    using T = typename E::T;
    constexpr int C = kCols<E>, kTile = kWave * C;
    const uint32_t group = first + blockIdx.x;
    const int which = group < jobs.end[0] ? 0 : group < jobs.end[1] ? 1 : 2;
    const uint32_t in_job = group - (which == 0 ? 0u : jobs.end[which - 1]), across = jobs.across[which];
    const uint32_t down = in_job / across, over = in_job - down * across;
    const MxColumns& job = jobs.job[which];
    const T* __restrict__ X = static_cast<const T*>(job.X);
    const int64_t rows = job.rows, ldx = job.ldx;
    const int cols = job.cols;
    const MxCoded columns = job.columns;
    float* __restrict__ sums = job.sums;
    constexpr bool kWide = sizeof(T) == 4;
    __shared__ __align__(16) uint8_t tile[kTile * kColBlocks * kMxBlockBytes];
    __shared__ __align__(8) uint8_t bytes[kTile * kColBlocks];
    __shared__ float partial[kColBlocks][kTile];
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t block0 = static_cast<int64_t>(down) * kColBlocks, row_blocks = (rows + kMxBlock - 1) / kMxBlock;
    const int col0 = over * kTile, col = col0 + C * lane;
    const int64_t r0 = (block0 + wave) * kMxBlock;
    if (r0 < rows) {
        const int n = static_cast<int>(min<int64_t>(rows - r0, kMxBlock));
        uint32_t v[kMxBlock][2];
        const T* x = X + r0 * ldx;
        if (cols >= C) {
            // The last columns' lanes read the matrix's last 8 bytes of a row and move
            // what is theirs down; rows past the last repeat it, and count as zeros.
            const int from = min(col, cols - C), past = min(col - from, C) * 8 * static_cast<int>(sizeof(T));
#pragma unroll
            for (int r = 0; r < kMxBlock; ++r) {
                const u32x2_any f = *reinterpret_cast<const u32x2_any*>(x + min(r, n - 1) * ldx + from);
                v[r][0] = f[0];
                v[r][1] = f[1];
            }
            if (col0 + kTile > cols || n < kMxBlock) {
#pragma unroll
                for (int r = 0; r < kMxBlock; ++r) {
                    uint64_t f = v[r][0] | static_cast<uint64_t>(v[r][1]) << 32;
                    f = past < 64 && r < n ? f >> past : 0u;
                    v[r][0] = static_cast<uint32_t>(f);
                    v[r][1] = static_cast<uint32_t>(f >> 32);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < kMxBlock; ++r) {
                v[r][0] = v[r][1] = 0u;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const T f = x[min(r, n - 1) * ldx + min(col + c, cols - 1)];
                    if (r >= n || col + c >= cols) continue;
                    if constexpr (kWide) v[r][c] = __float_as_uint(f);
                    else v[r][c / 2] |= static_cast<uint32_t>(f) << (16 * (c & 1));
                }
            }
        }
        if (columns.codes) {
            uint32_t m[2] = {0u, 0u};
#pragma unroll
            for (int r = 0; r < kMxBlock; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    m[i] = kWide ? max(m[i], v[r][i] & kAbs32) : max16x2(m[i], v[r][i] & kAbs16x2);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint32_t byte = scale_byte(kWide ? m[c % 2] : wide_bits<E>(m[c / 2] >> (16 * (c & 1)) & 0xFFFFu));
                const float s = __uint_as_float(byte << 23);
                u32x4 q;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t word = 0;
                    if constexpr (kWide) {
                        word = pack2<0>(word, __uint_as_float(v[8 * w][c]), __uint_as_float(v[8 * w + 1][c]), s);
                        word = pack2<1>(word, __uint_as_float(v[8 * w + 2][c]), __uint_as_float(v[8 * w + 3][c]), s);
                        word = pack2<2>(word, __uint_as_float(v[8 * w + 4][c]), __uint_as_float(v[8 * w + 5][c]), s);
                        word = pack2<3>(word, __uint_as_float(v[8 * w + 6][c]), __uint_as_float(v[8 * w + 7][c]), s);
                    } else {  // the column's values of two rows
                        constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;
                        auto two = [&](int r) {
                            return __builtin_amdgcn_perm(v[r + 1][c / 2], v[r][c / 2], (c & 1) ? kHigh : kLow);
                        };
                        word = pack2<E, 0>(word, two(8 * w), s);
                        word = pack2<E, 1>(word, two(8 * w + 2), s);
                        word = pack2<E, 2>(word, two(8 * w + 4), s);
                        word = pack2<E, 3>(word, two(8 * w + 6), s);
                    }
                    q[w] = byte == 255u ? 0u : word;
                }
                // a column's blocks are xor-ed with its lane, so that neighbours write different banks
                *reinterpret_cast<u32x4*>(tile + ((C * lane + c) * kColBlocks + (wave ^ (lane & 7))) * kMxBlockBytes) = q;
                bytes[(C * lane + c) * kColBlocks + wave] = static_cast<uint8_t>(byte);
            }
        }
        if (sums) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float total = 0.0f;
#pragma unroll
                for (int r = 0; r < kMxBlock; ++r)
                    total += kWide ? __uint_as_float(v[r][c % 2]) : E::one(static_cast<T>(v[r][c / 2] >> (16 * (c & 1)) & 0xFFFFu));
                partial[wave][C * lane + c] = total;
            }
        }
        if (ROWS && which == 0) {  // blocks of 32 columns: 32 / C lanes
            const MxCoded by_rows = jobs.job[0].by_rows;
#pragma unroll
            for (int r = 0; r < kMxBlock; ++r) {
                uint32_t m = kWide ? max(v[r][0] & kAbs32, v[r][1] & kAbs32)
                                   : max16x2(v[r][0] & kAbs16x2, v[r][1] & kAbs16x2);
                if constexpr (!kWide) m = max(m & 0xFFFFu, m >> 16);
                m = max(m, dpp_u32<kDppXor1>(m));
                m = max(m, dpp_u32<kDppXor2>(m));
                m = max(m, dpp_u32<kDppHalfMirror>(m));
                if (kWide) m = max(m, dpp_u32<kDppMirror>(m));
                const uint32_t byte = scale_byte(kWide ? m : wide_bits<E>(m));
                const float s = __uint_as_float(byte << 23);
                uint32_t q = 0;
                if constexpr (kWide) {
                    q = pack2<0>(q, __uint_as_float(v[r][0]), __uint_as_float(v[r][1]), s);
                } else {
                    q = pack2<E, 0>(q, v[r][0], s);
                    q = pack2<E, 1>(q, v[r][1], s);
                }
                if (byte == 255u) q = 0u;
                const int end = (cols + kMxBlock - 1) / kMxBlock * kMxBlock;
                if (r < n && col < end) {
                    uint8_t* to = by_rows.codes + (r0 + r) * by_rows.ldc + col / 2;
                    if constexpr (kWide) *to = static_cast<uint8_t>(q);
                    else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(q);
                    if (col % kMxBlock == 0)
                        *scale_place(by_rows, r0 + r, col / kMxBlock) = static_cast<uint8_t>(byte);
                }
            }
        }
    } else if (sums) {
#pragma unroll
        for (int c = 0; c < C; ++c) partial[wave][C * lane + c] = 0.0f;
    }
    __syncthreads();
    if (sums && static_cast<int>(threadIdx.x) < kTile && col0 + static_cast<int>(threadIdx.x) < cols) {
        float total = partial[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kColBlocks; ++w) total += partial[w][threadIdx.x];
        sums[down * static_cast<int64_t>(cols) + col0 + threadIdx.x] = total;
    }
    if (!columns.codes) return;
    const int live = static_cast<int>(min<int64_t>(row_blocks - block0, kColBlocks));
#pragma unroll
    for (int t = threadIdx.x; t < kTile * kColBlocks; t += kColBlocks * kWave) {
        const int c = t / kColBlocks, b = t % kColBlocks;
        if (b < live && col0 + c < cols)
            *reinterpret_cast<u32x4*>(columns.codes + (col0 + c) * columns.ldc + (block0 + b) * kMxBlockBytes) =
                *reinterpret_cast<const u32x4*>(tile + (c * kColBlocks + (b ^ (c / C & 7))) * kMxBlockBytes);
    }
    const int c = threadIdx.x;
    if (c < kTile && col0 + c < cols) {
        if (live == kColBlocks && !columns.paired) {
            *reinterpret_cast<u32x2_any*>(columns.scales + (col0 + c) * columns.lds + block0) =
                *reinterpret_cast<const u32x2_any*>(bytes + c * kColBlocks);
        } else {
            for (int b = 0; b < live; ++b) *scale_place(columns, col0 + c, block0 + b) = bytes[c * kColBlocks + b];
        }
    }
}

// A column a thread, all groups in order.
__global__ __launch_bounds__(kWave) void mx_add_sums_kernel(const float* __restrict__ sums, int64_t groups, int cols,
                                                            float* __restrict__ out) {
    const int c = blockIdx.x * kWave + threadIdx.x;
    if (c >= cols) return;
    float s = 0.0f;
#pragma unroll 32
    for (int64_t g = 0; g < groups; ++g) s += sums[g * cols + c];  // many on their way
    out[c] = s;
}

__global__ __launch_bounds__(kThreads) void mx_zero_kernel(float* __restrict__ out, int64_t rows, int cols, int64_t ldo) {
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
        for (int c = blockIdx.x * kThreads + threadIdx.x; c < cols; c += gridDim.x * kThreads) out[r * ldo + c] = 0.0f;
}

// ---------------------------------------------------------------------------
// codes to values
// ---------------------------------------------------------------------------
// 8 values a lane.  The scale 255 is NaN, which the converter does not know.
// 8192 x 11008 bf16 45 us (5.05 TB/s), 35 with the codes still in cache.
template <class E>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint8_t* __restrict__ codes, int64_t ldc,
                                                                 const uint8_t* __restrict__ scales, int64_t lds,
                                                                 uint32_t items, uint32_t per_row, int d,
                                                                 typename E::T* __restrict__ out, int64_t ldo) {
    const int lane = __lane_id();
    const uint32_t first = (blockIdx.x * kWavesPerGroup + threadIdx.x / kWave) * kRowItems;
    uint32_t row = first / per_row, at = first - row * per_row;
    const uint32_t row_first = row, at_first = at;
    uint32_t q[kRowItems], s[kRowItems];
#pragma unroll
    for (int i = 0; i < kRowItems; ++i) {
        const int64_t c = static_cast<int64_t>(at) * 512 + lane * 8;
        if (first + i < items && c < d) {
            q[i] = *reinterpret_cast<const uint32_t*>(codes + row * ldc + c / 2);
            s[i] = scales[row * lds + c / kMxBlock];
        }
        if (++at == per_row) {
            at = 0;
            ++row;
        }
    }
    row = row_first;
    at = at_first;
#pragma unroll
    for (int i = 0; i < kRowItems; ++i) {
        const int64_t c = static_cast<int64_t>(at) * 512 + lane * 8;
        if (first + i < items && c < d) {
            const float scale = __uint_as_float(s[i] << 23);
            float v[8];
            const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 0);
            const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 1);
            const auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 2);
            const auto f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 3);
            v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = e[0], v[5] = e[1], v[6] = f[0], v[7] = f[1];
            if (s[i] == 255u) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(0x7FC00000u);
            }
            store8<E>(out + row * ldo, static_cast<int>(c), d, v);
        }
        if (++at == per_row) {
            at = 0;
            ++row;
        }
    }
}

// ---------------------------------------------------------------------------
// What the product kernels share
// ---------------------------------------------------------------------------
// A step is kDepth = 128 bytes of a row: 256 codes, 8 scales.  The matrix
// instruction takes 128 codes of a row, 32 of them (one block, one scale) in
// each of the four lanes l / 16: half h of a step takes block 2 (l / 16) + h,
// so that a lane's two scales of a step are neighbours in memory and reach the
// instruction as bytes of one register.  Which blocks meet in an instruction
// only changes the order of the sum.
//
// LDS serves the 16-byte reads of 8 rows and two neighbouring lane groups at a
// time, and the rows' parity picks the half of its banks: with pieces 2 (l / 16) +
// h the lowest bit of a row's key has to stand in bit 1, or the two groups meet
// (keys as for int8, bit 0: half of the LDS cycles were conflicts, 8192 x 11008 x 4096
// in 205 us).
__device__ __forceinline__ int mx_key(int k) { return (k & 4) | (k >> 1 & 1) | (k & 1) << 1; }
__device__ __forceinline__ int mx_key_x(int row) { return mx_key(key_x(row)); }
template <int TN>
__device__ __forceinline__ int mx_key_w(int row) {
    return mx_key(key_w<TN>(row));
}

template <int SEL>
__device__ __forceinline__ f32x4 mfma(const i32x4& w, const i32x4& x, const f32x4& acc, uint32_t ws, uint32_t xs) {
    const i32x8 a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, SEL, static_cast<int>(ws), SEL,
                                                            static_cast<int>(xs));
}

// Between LDS accesses of one wave whose lanes read what other lanes wrote, or
// write over what other lanes read, without a barrier: the hardware executes a
// wave's LDS accesses in order, and this holds the compiler to it as well.  No
// instruction comes of it.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 16 scales of a row in the order of a pair of steps: word q has those of lane
// group q, halves 0 and 1 of the even step, then of the odd one.
__device__ __forceinline__ u32x4 pair_order(const u32x4& s) {
    return u32x4{__builtin_amdgcn_perm(s[2], s[0], 0x05040100u), __builtin_amdgcn_perm(s[2], s[0], 0x07060302u),
                 __builtin_amdgcn_perm(s[3], s[1], 0x05040100u), __builtin_amdgcn_perm(s[3], s[1], 0x07060302u)};
}

// Up to 8 scales of a row from block k on, as two words; past the row's end 0,
// which no code meets (a 255 there would).
__device__ __forceinline__ uint2 tail_scales(const uint8_t* row, int k, int blocks) {
    uint32_t r[2] = {0u, 0u};
    uint8_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = row[min(k + i, blocks - 1)];  // on their way together
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i >> 2] |= k + i < blocks ? static_cast<uint32_t>(v[i]) << (8 * (i & 3)) : 0u;
    return make_uint2(r[0], r[1]);
}

// Four neighbouring outputs of a row.
template <class E>
__device__ __forceinline__ void store_out4(const MxProduct& p, int64_t m, int n, const f32x4& acc, bool packed) {
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        v[r] = acc[r];
        if (p.bias) v[r] = v[r] + E::one(static_cast<const typename E::T*>(p.bias)[min(n + r, p.N - 1)]);
    }
    typename E::T* out = static_cast<typename E::T*>(p.out) + m * p.ldo + n;
    if (packed && n + 4 <= p.N) {
        if constexpr (sizeof(typename E::T) == 4)
            store16<false>(out, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                      __float_as_uint(v[3])});
        else
            *reinterpret_cast<uint2*>(out) = make_uint2(E::pack(v[0], v[1]), E::pack(v[2], v[3]));
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < p.N) out[r] = E::narrow(v[r]);
    }
}

// Whether every row of the output starts at a multiple of `bytes`.
bool out_aligned(const MxProduct& p, int64_t esize, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(p.out) % bytes == 0 && (p.M == 1 || p.ldo * esize % bytes == 0);
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
// A workgroup takes 16 MT rows and 16 TN channels.  Its waves split the depth
// and work alone, each with two steps of both operands in LDS of its own and no
// barrier; a lane's scales of a step go straight to registers.  At the end each
// wave leaves its sums where its operands were, and after the one barrier every
// thread adds four channels of all waves, in their order.  16 x 4096 x 4096 takes
// 5.9 us, of which reading the 9 MB of weights would be 1.7: the launch and the
// latency of the few steps that a wave has.
template <class E, int MT, int TN, int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void mx_few_rows_kernel(const MxProduct p, int m_tiles, bool packed) {
    constexpr int BM = MT * 16, BN = TN * 16, kStep = (BM + BN) * kDepth;
    __shared__ __align__(1024) uint8_t even[WAVES * kStep], odd[WAVES * kStep];
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, q = lane >> 4;
    // Workgroups id, id + 8, ... run on one XCD: it takes a run of tiles with
    // the m tiles of a block of channels after each other, so that they share
    // its weights in that L2.
    const int per = gridDim.x >> 3, t = static_cast<int>(blockIdx.x & 7) * per + static_cast<int>(blockIdx.x >> 3);
    const int n0 = t / m_tiles * BN;
    const int64_t m0 = static_cast<int64_t>(t % m_tiles) * BM;
    if (n0 >= p.N) return;
    const int rows = static_cast<int>(min<int64_t>(p.M - m0, BM)), cols = min(p.N - n0, BN);
    const uint8_t* xb = p.x + m0 * p.ldx;
    const uint8_t* wb = p.w + static_cast<int64_t>(n0) * p.ldw;
    const uint8_t* xsb = p.xs + m0 * p.ldxs;
    const uint8_t* wsb = p.ws + static_cast<int64_t>(n0) * p.ldws;
    const int ldx = static_cast<int>(p.ldx), ldw = static_cast<int>(p.ldw);

    // Load i covers rows 8 i .. 8 i + 7 of a tile; rows past the matrix read
    // its last row, their outputs are not stored.
    const int row0 = lane >> 3, piece0 = lane & 7;
    int xo[2 * MT], wo[2 * TN], xso[MT], wso[TN];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
        xo[i] = min(8 * i + row0, rows - 1) * ldx + 16 * (piece0 ^ mx_key_x(8 * i + row0));
#pragma unroll
    for (int i = 0; i < 2 * TN; ++i)
        wo[i] = min(8 * i + row0, cols - 1) * ldw + 16 * (piece0 ^ mx_key_w<TN>(8 * i + row0));
#pragma unroll
    for (int i = 0; i < MT; ++i) xso[i] = min(16 * i + l16, rows - 1) * static_cast<int>(p.ldxs) + 2 * q;
#pragma unroll
    for (int j = 0; j < TN; ++j)
        wso[j] = min(operand_channel<TN>(j, l16), cols - 1) * static_cast<int>(p.ldws) + 2 * q;
    struct Scales {
        uint32_t x[MT], w[TN];
    };
    auto fetch = [&](int s, uint8_t* to, Scales& sc, bool live) {
        const int range = live ? 0x7FFFFFFF : 0;  // not live: issued, but reads nothing
        const auto xsr = buf_rsrc(xsb, range), wsr = buf_rsrc(wsb, range);
#pragma unroll
        for (int j = 0; j < TN; ++j) sc.w[j] = __builtin_amdgcn_raw_buffer_load_b16(wsr, wso[j], 8 * s, 0);
#pragma unroll
        for (int i = 0; i < MT; ++i) sc.x[i] = __builtin_amdgcn_raw_buffer_load_b16(xsr, xso[i], 8 * s, 0);
        const auto xr = buf_rsrc(xb, range), wr = buf_rsrc(wb, range);
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i) load16_to_lds(wr, to + (BM + 8 * i) * kDepth, wo[i], s * kDepth);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) load16_to_lds(xr, to + 8 * i * kDepth, xo[i], s * kDepth);
    };
    f32x4 acc[MT][TN] = {};
    i32x4 x[2][MT], w[2][TN];
    auto read = [&](const uint8_t* from) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = operand_channel<TN>(j, l16);
                w[h][j] = *reinterpret_cast<const i32x4*>(from + (BM + row) * kDepth + 16 * ((2 * q + h) ^ mx_key_w<TN>(row)));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
                x[h][i] = *reinterpret_cast<const i32x4*>(from + (16 * i + l16) * kDepth + 16 * ((2 * q + h) ^ mx_key_x(l16)));
        }
    };
    auto multiply = [&](const Scales& sc) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma<0>(w[0][j], x[0][i], acc[i][j], sc.w[j], sc.x[i]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma<1>(w[1][j], x[1][i], acc[i][j], sc.w[j], sc.x[i]);
    };
    const int steps = p.K / kDepth;
    uint8_t *const e = even + wave * kStep, *const o = odd + wave * kStep;
    Scales se, so;
    // A step's operands have arrived in LDS (of the loads on their way only
    // the next step's are newer), and have left it (lgkmcnt(0)) before the
    // loads of the step after the next go over them.  Past the last step everything but
    // the products is done all the same: branches around loads to LDS make
    // the compiler wait for all of them.
    auto turn_step = [&](int s, uint8_t* at, Scales& sc) {
        landed<3 * (MT + TN)>();
        read(at);
        const Scales now = sc;
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        fetch(s + 2 * WAVES, at, sc, s + 2 * WAVES < steps);
        if (s < steps) multiply(now);
    };
    fetch(wave, e, se, wave < steps);
    fetch(wave + WAVES, o, so, wave + WAVES < steps);
    for (int s = wave; s < steps; s += 2 * WAVES) {
        turn_step(s, e, se);
        turn_step(s + WAVES, o, so);
    }
    __builtin_amdgcn_s_waitcnt(0);
    if (steps * kDepth < p.K && steps % WAVES == wave) {  // the depth's partial step, zeros past K
        const int k = steps * kDepth, blocks = p.K / kMxBlockBytes;
        const u32x4 none = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int row = 8 * i + row0, at = k + 16 * (piece0 ^ mx_key_x(row));
            *reinterpret_cast<u32x4*>(e + 8 * i * kDepth + lane * 16) =
                at < p.K ? load16<false>(xb + static_cast<int64_t>(min(row, rows - 1)) * ldx + at) : none;
        }
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i) {
            const int row = 8 * i + row0, at = k + 16 * (piece0 ^ mx_key_w<TN>(row));
            *reinterpret_cast<u32x4*>(e + (BM + 8 * i) * kDepth + lane * 16) =
                at < p.K ? load16<false>(wb + static_cast<int64_t>(min(row, cols - 1)) * ldw + at) : none;
        }
        auto two = [&](const uint8_t* from) {  // the lane's scales: blocks 8 steps + 2 q and the one after it
            const int b = 8 * steps + 2 * q;
            uint32_t r = b < blocks ? from[8 * steps] : 0u;
            if (b + 1 < blocks) r |= static_cast<uint32_t>(from[8 * steps + 1]) << 8;
            return r;
        };
#pragma unroll
        for (int i = 0; i < MT; ++i) se.x[i] = two(xsb + xso[i]);
#pragma unroll
        for (int j = 0; j < TN; ++j) se.w[j] = two(wsb + wso[j]);
        wave_order();
        read(e);
        multiply(se);
    }
    wave_order();
    // Block (i, j) of sums: 1 KB of the wave's own operands, whose last reads
    // are done.
    constexpr int kFirst = kStep / 1024 < MT * TN ? kStep / 1024 : MT * TN;
    static_assert(MT * TN - kFirst <= kStep / 1024, "the sums fit over the operands");
    auto block = [&](int n, int w) {
        return n < kFirst ? even + w * kStep + n * 1024 : odd + w * kStep + (n - kFirst) * 1024;
    };
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            *reinterpret_cast<f32x4*>(block(i * TN + j, wave) + sum_place(l16, q, TN * q + j)) = acc[i][j];
    __syncthreads();
    for (int t = threadIdx.x; t < BM * BN / 4; t += WAVES * kWave) {
        const int r = t / (BN / 4), c = t % (BN / 4);
        if (r >= rows || 4 * c >= cols) continue;
        const int n = (r >> 4) * TN + c % TN, at = sum_place(r & 15, c / TN, c);
        f32x4 sum = *reinterpret_cast<const f32x4*>(block(n, 0) + at);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += *reinterpret_cast<const f32x4*>(block(n, w) + at);
        store_out4<E>(p, m0 + r, n0 + 4 * c, sum, packed);
    }
}

// ---------------------------------------------------------------------------
// A few tokens, quantized on the way
// ---------------------------------------------------------------------------
// The few-rows kernel for a few tokens whose codes every workgroup makes for
// itself, in LDS, while its first weights are on their way: one launch
// instead of two, for a reading of the tokens from cache by each workgroup.
// 1 x 4096 x 4096 4.2 us with weights from cache, 5.0 from memory.
template <class E, int TN, int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void mx_tokens_kernel(const MxProduct p, int d,
                                                                 const typename E::T* __restrict__ X, int64_t ldX,
                                                                 bool packed) {
    constexpr int BN = TN * 16, kStep = BN * kDepth;
    __shared__ __align__(1024) uint8_t even[WAVES * kStep], odd[WAVES * kStep];
    __shared__ __align__(16) uint8_t codes[kMxTokenBytes];
    __shared__ __align__(8) uint8_t bytes[kMxTokenBytes / kMxBlockBytes];
    static_assert(TN * 1024 <= kStep, "the sums fit over the operands");
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, q = lane >> 4;
    const int rows = static_cast<int>(p.M), n0 = blockIdx.x * BN, cols = min(p.N - n0, BN);
    const uint8_t* wb = p.w + static_cast<int64_t>(n0) * p.ldw;
    const uint8_t* wsb = p.ws + static_cast<int64_t>(n0) * p.ldws;
    const int ldw = static_cast<int>(p.ldw);
    const int row0 = lane >> 3, piece0 = lane & 7;
    int wo[2 * TN], wso[TN];
#pragma unroll
    for (int i = 0; i < 2 * TN; ++i)
        wo[i] = min(8 * i + row0, cols - 1) * ldw + 16 * (piece0 ^ mx_key_w<TN>(8 * i + row0));
#pragma unroll
    for (int j = 0; j < TN; ++j)
        wso[j] = min(operand_channel<TN>(j, l16), cols - 1) * static_cast<int>(p.ldws) + 2 * q;
    struct Scales {
        uint32_t w[TN];
    };
    auto fetch = [&](int s, uint8_t* to, Scales& sc, bool live) {
        const int range = live ? 0x7FFFFFFF : 0;
        const auto wr = buf_rsrc(wb, range), wsr = buf_rsrc(wsb, range);
#pragma unroll
        for (int j = 0; j < TN; ++j) sc.w[j] = __builtin_amdgcn_raw_buffer_load_b16(wsr, wso[j], 8 * s, 0);
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i) load16_to_lds(wr, to + 8 * i * kDepth, wo[i], s * kDepth);
    };
    const int steps = p.K / kDepth, all_steps = (p.K + kDepth - 1) / kDepth;
    uint8_t *const e = even + wave * kStep, *const o = odd + wave * kStep;
    Scales se, so;
    fetch(wave, e, se, wave < steps);
    fetch(wave + WAVES, o, so, wave + WAVES < steps);

    // The tokens' codes and scales, zeros from K to a whole step.
    const int per_row = (all_steps * 256 + 511) / 512, items = rows * per_row;
    const int pitch = all_steps * kDepth + kMxTokenPad, pitch_s = all_steps * 8;
    u32x4 keep[kMxTokenItems][E::kVec];
#pragma unroll
    for (int t = 0; t < kMxTokenItems; ++t) {
        const int item = wave + t * WAVES;
        if (item < items) {
            const int r = item / per_row;
            load8_raw<E>(X + r * ldX, (item - r * per_row) * 512 + lane * 8, d, keep[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < kMxTokenItems; ++t) {
        const int item = wave + t * WAVES;
        if (item < items) {
            const int r = item / per_row, c = (item - r * per_row) * 512 + lane * 8;
            const uint32_t byte = row_byte<E>(keep[t]);
            if (c < all_steps * 256) {
                *reinterpret_cast<uint32_t*>(codes + r * pitch + c / 2) = row_codes<E>(keep[t], byte);
                if ((lane & 3) == 0) bytes[r * pitch_s + c / kMxBlock] = static_cast<uint8_t>(byte);
            }
        }
    }
    __syncthreads();

    f32x4 acc[TN] = {};
    i32x4 x[2], w[2][TN];
    uint32_t xs;
    const uint8_t* mine = codes + min(l16, rows - 1) * pitch + 32 * q;  // rows past the last repeat it
    const uint8_t* mine_s = bytes + min(l16, rows - 1) * pitch_s + 2 * q;
    auto read = [&](const uint8_t* from, int s) {
        const int at = min(s, all_steps - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = operand_channel<TN>(j, l16);
                w[h][j] = *reinterpret_cast<const i32x4*>(from + row * kDepth + 16 * ((2 * q + h) ^ mx_key_w<TN>(row)));
            }
            x[h] = *reinterpret_cast<const i32x4*>(mine + at * kDepth + 16 * h);
        }
        xs = *reinterpret_cast<const uint16_t*>(mine_s + 8 * at);
    };
    auto multiply = [&](const Scales& sc) {
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[j] = mfma<0>(w[0][j], x[0], acc[j], sc.w[j], xs);
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[j] = mfma<1>(w[1][j], x[1], acc[j], sc.w[j], xs);
    };
    auto turn_step = [&](int s, uint8_t* at, Scales& sc) {  // as in the few-rows kernel
        landed<3 * TN>();
        read(at, s);
        const Scales now = sc;
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        fetch(s + 2 * WAVES, at, sc, s + 2 * WAVES < steps);
        if (s < steps) multiply(now);
    };
    for (int s = wave; s < steps; s += 2 * WAVES) {
        turn_step(s, e, se);
        turn_step(s + WAVES, o, so);
    }
    __builtin_amdgcn_s_waitcnt(0);
    if (steps * kDepth < p.K && steps % WAVES == wave) {
        const int k = steps * kDepth, blocks = p.K / kMxBlockBytes;
        const u32x4 none = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i) {
            const int row = 8 * i + row0, at = k + 16 * (piece0 ^ mx_key_w<TN>(row));
            *reinterpret_cast<u32x4*>(e + 8 * i * kDepth + lane * 16) =
                at < p.K ? load16<false>(wb + static_cast<int64_t>(min(row, cols - 1)) * ldw + at) : none;
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int b = 8 * steps + 2 * q;
            const uint8_t* from = wsb + wso[j] + 8 * steps;
            se.w[j] = b < blocks ? from[0] : 0u;
            if (b + 1 < blocks) se.w[j] |= static_cast<uint32_t>(from[1]) << 8;
        }
        wave_order();
        read(e, steps);
        multiply(se);
    }
    wave_order();
#pragma unroll
    for (int j = 0; j < TN; ++j)
        *reinterpret_cast<f32x4*>(e + j * 1024 + sum_place(l16, q, TN * q + j)) = acc[j];
    __syncthreads();
    for (int t = threadIdx.x; t < rows * BN / 4; t += WAVES * kWave) {
        const int r = t / (BN / 4), c = t % (BN / 4);
        if (4 * c >= cols) continue;
        const uint8_t* at = even + c % TN * 1024 + sum_place(r, c / TN, c);
        f32x4 sum = *reinterpret_cast<const f32x4*>(at);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += *reinterpret_cast<const f32x4*>(at + w * kStep);
        store_out4<E>(p, r, n0 + 4 * c, sum, packed);
    }
}

// ---------------------------------------------------------------------------
// Many rows: tiles through LDS.
// ---------------------------------------------------------------------------
// A workgroup of WM x WN waves takes a tile of 16 TM WM rows and 64 WN channels:
// 256 x 256 with two steps of both operands in LDS (mx_large_kernel), the smaller
// ones with a ring of two or four (mx_ring_kernel).
template <class E>
constexpr bool kSums = std::is_same<typename E::T, void>::value;  // the sums themselves, no bias

struct MSums {
    using T = void;
};

// A wave's 16 TM x 64 outputs, through a region of LDS that is the wave's own,
// so that a row leaves as one run of 64 channels.  The 16-byte pieces of a row
// are xor-ed with the row like the operands'.  NT: stores that do not stay in
// L2.  m, n: the wave's first row and channel.
template <class E, class T, int TM, int kRegion, bool NT>
__device__ __forceinline__ void store_tile(const MxProduct& p, T* out, uint8_t* region, int lane, int64_t m, int n,
                                           const f32x4 (&acc)[TM][4], const float (&bias)[16], bool packed) {
    constexpr int kSize = sizeof(T), kRow = 64 * kSize;
    constexpr int kFit = kRegion / (16 * kRow) < TM ? kRegion / (16 * kRow) : TM;
    constexpr int kPass = TM % kFit == 0 ? kFit : 1;  // blocks of 16 rows a pass
    static_assert(kFit >= 1, "a block fits");
    const int l16 = lane & 15, q = lane >> 4;
    out += m * p.ldo + n;
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += kPass) {
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
            const int row = 16 * i + l16;
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                v[e] = acc[i0 + i][e >> 2][e & 3];
                if (!kSums<E> && p.bias) v[e] = v[e] + bias[e];
            }
#pragma unroll
            for (int c = 0; c < kSize; ++c) {  // the lane's 16 kSize bytes
                u32x4 d;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (kSize == 4) d[r] = __float_as_uint(v[4 * c + r]);
                    else d[r] = E::pack(v[8 * c + 2 * r], v[8 * c + 2 * r + 1]);
                }
                *reinterpret_cast<u32x4*>(region + row * kRow + 16 * ((q * kSize + c) ^ (row & 7))) = d;
            }
        }
        wave_order();
        constexpr int kPieces = kRow / 16, kRows = kWave / kPieces;  // rows a store instruction
#pragma unroll
        for (int r0 = 0; r0 < kPass * 16; r0 += kRows) {
            const int row = r0 + lane / kPieces, piece = lane % kPieces;
            const u32x4 d = *reinterpret_cast<const u32x4*>(region + row * kRow + 16 * (piece ^ (row & 7)));
            T* to = out + (16 * i0 + row) * p.ldo + piece * (16 / kSize);
            if (packed) store16<NT>(to, d);
            else store16_any(to, d);
        }
        if (i0 + kPass < TM) wave_order();  // the next pass goes over the region
    }
}

// Tiles of 256 x 256, 2 x 4 waves of 128 rows and 64 channels, two steps of both
// operands in LDS: while the matrix cores work on one, the loads of the next go
// into the other.
//
// The scales come in the order of pairs of steps (MxCoded) and go to LDS like the
// operands: in rows, 16 bytes of a cache line would be fetched again for every
// pair, as much as half the operands.  What the depth does not fill is fetched
// from past the operand's range, which leaves zeros.
//
// The matrix pipes are busy 48 to 57% of the cycles.  Matrix instructions alone, on
// registers, reach 6.6 to 7.0 PFLOP/s with random codes (9.6 with zeros: the power
// bounds them).  8192^3 takes 237 to 265 us over cards and runs (4.15 to 4.6
// PFLOP/s), 8192 x 11008 x 4096 176 to 206; between them are the tiles' ends, rounds
// that are not full (1376 tiles are 5.4 of 256) and the reads from LDS, 15% of whose
// cycles are bank conflicts.
constexpr int kNowhere = INT32_MIN;  // an offset past every range

template <class E>
__global__ __launch_bounds__(8 * kWave) void mx_large_kernel(const MxProduct p, int m_tiles, int n_tiles, bool packed) {
    using T = typename E::T;
    constexpr int WM = 2, TM = 8, TN = 4, kT = 8 * kWave, BM = kPairedRows, BN = 256;
    constexpr int kXLoads = BM * 8 / kT, kLoads = kXLoads + BN * 8 / kT;  // a thread a step
    constexpr int kRound = kT / 8;                                        // rows a load
    static_assert(kRound % (8 * TN) == 0, "the keys repeat from load to load");
    // Arrays by name, and code that names the one it means: the compiler then
    // sees that the operands it reads are not those on their way, and puts no
    // wait for the loads before the reads.
    __shared__ __align__(1024) uint8_t x_even[BM * kDepth], x_odd[BM * kDepth], w_even[BN * kDepth], w_odd[BN * kDepth];
    // The scales of a pair of steps, 16 bytes a row, see pair_order.  Its alignment
    // puts it before the other arrays: the reads' constant offsets, at most 64 KB,
    // reach it from one register.
    __shared__ __align__(4096) uint8_t scales[2][(BM + BN) * 16];
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, q = lane >> 4;
    const int wm = (wave % WM) * TM * 16, wn = (wave / WM) * TN * 16;

    // Each XCD works through a contiguous range of tiles, in groups of 8 rows
    // of tiles, so that its L2 holds the operands its workgroups share.
    const int tiles = m_tiles * n_tiles, per = (tiles + 7) / 8;
    const int t = static_cast<int>(blockIdx.x & 7) * per + static_cast<int>(blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= per || t >= tiles) return;
    constexpr int kGroupM = 8;
    const int group = t / (kGroupM * n_tiles), in = t - group * kGroupM * n_tiles;
    const int gm = min(kGroupM, m_tiles - group * kGroupM);
    // The last tiles of a row or column are moved inside the matrix (M >= BM, N >=
    // BN): outputs computed twice get the same values twice.
    const int64_t m0 = min<int64_t>(static_cast<int64_t>(group * kGroupM + in % gm) * BM, p.M - BM);
    const int n0 = min(in / gm * BN, p.N - BN), K = p.K;
    const uint8_t* xb = p.x + m0 * p.ldx;
    const uint8_t* wb = p.w + static_cast<int64_t>(n0) * p.ldw;
    const int row0 = threadIdx.x >> 3, piece0 = lane & 7;
    const int ldx = static_cast<int>(p.ldx), ldw = static_cast<int>(p.ldw);
    const int xpiece = 16 * (piece0 ^ mx_key_x(row0)), wpiece = 16 * (piece0 ^ mx_key_w<TN>(row0));
    struct Fetch {  // of a step
        int k, xo, wo;
    };
    auto fetch_of = [&](int s) {
        const int k = s * kDepth;
        return Fetch{k, k + xpiece < K ? row0 * ldx + xpiece : kNowhere, k + wpiece < K ? row0 * ldw + wpiece : kNowhere};
    };
    auto fetch_one = [&](int n, const Fetch& f, uint8_t* xd, uint8_t* wd) {
        if (n < kXLoads)
            load16_to_lds(buf_rsrc(xb, 0x7FFFFFFF), xd + (n * kT + wave * kWave) * 16, f.xo, f.k + n * kRound * ldx);
        else
            load16_to_lds(buf_rsrc(wb, 0x7FFFFFFF), wd + ((n - kXLoads) * kT + wave * kWave) * 16, f.wo,
                          f.k + (n - kXLoads) * kRound * ldw);
    };
    auto fetch = [&](int s, uint8_t* xd, uint8_t* wd) {
        const Fetch f = fetch_of(s);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) fetch_one(n, f, xd, wd);
    };
    // 64 rows' scales a wave.
    const bool of_x = wave < BM / kWave;
    const uint8_t* sb = of_x ? p.xs + (m0 + wave * kWave) * 16 : p.ws + (n0 + wave * kWave - BM) * 16;
    const int64_t plane = of_x ? p.ldxs : p.ldws;
    const int steps = (K + kDepth - 1) / kDepth;
    auto fetch_scales = [&](int pair, uint8_t* to) {
        load16_to_lds(buf_rsrc(sb + pair * plane, 2 * pair < steps ? 0x7FFFFFFF : 0), to + wave * kWave * 16, 16 * lane, 0);
    };

    // Half a step's operands (4 blocks) in LDS; the keys do not change with i
    // and j, 16 and 4 rows on.
    const int w_row = operand_channel<TN>(0, l16);
    const int xp[2] = {(wm + l16) * kDepth + 16 * ((2 * q) ^ mx_key_x(l16)),
                       (wm + l16) * kDepth + 16 * ((2 * q + 1) ^ mx_key_x(l16))};
    const int wp[2] = {(wn + w_row) * kDepth + 16 * ((2 * q) ^ mx_key_w<TN>(w_row)),
                       (wn + w_row) * kDepth + 16 * ((2 * q + 1) ^ mx_key_w<TN>(w_row))};
    const int xsp = (wm + l16) * 16 + 4 * q, wsp = (BM + wn + w_row) * 16 + 4 * q;
    f32x4 acc[TM][TN] = {};
    i32x4 x[TM], w0[TN], w1[TN];
    uint32_t sx[TM], sw[TN], sw_next[TN];
    auto read_x = [&](const uint8_t* xd, int h, int i) {
        x[i] = *reinterpret_cast<const i32x4*>(xd + xp[h] + 16 * i * kDepth);
    };
    auto read_w = [&](const uint8_t* wd, int h, int j) {
        return *reinterpret_cast<const i32x4*>(wd + wp[h] + 4 * j * kDepth);
    };
    auto read_sx = [&](const uint8_t* from, int i) { return *reinterpret_cast<const uint32_t*>(from + xsp + 16 * i * 16); };
    auto read_sw = [&](const uint8_t* from, int j) { return *reinterpret_cast<const uint32_t*>(from + wsp + 4 * j * 16); };
    // The products of half a step.  Each operand of x is replaced by half h of (xn,
    // wn) as soon as its last product is issued, and the next weights are read on
    // the way; in the last half of a pair (SEL 3) the next pair's scales as well.
    // Beside them a part of the loads to LDS is issued, load(n).  The order is held
    // group by group: left to itself the compiler puts reads right before their
    // use (8192^3 272 -> 258 us, 8192 x 11008 x 4096 234 -> 213).
    auto multiply = [&](auto sel, const i32x4 (&w)[TN], const uint8_t* xn, const uint8_t* wn, int h, i32x4 (&w_next)[TN],
                        const uint8_t* scales_next, const auto& load) {
        constexpr int SEL = decltype(sel)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma<SEL>(w[j], x[i], acc[i][j], sw[j], sx[i]);
            read_x(xn, h, i);
            if (i < TN) {
                w_next[i] = read_w(wn, h, i);
                if (SEL == 3) sw_next[i] = read_sw(scales_next, i);
            }
            if (SEL == 3) sx[i] = read_sx(scales_next, i);
            load(i);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (SEL == 3) {
#pragma unroll
            for (int j = 0; j < TN; ++j) sw[j] = sw_next[j];
        }
    };
    static_assert(kLoads == TM, "a load a group");

    // Software pipeline: while half a step is multiplied the next half is read
    // from LDS, and the step after it is on its way from memory.  The one
    // barrier of a step stands between its halves: past it every wave's loads
    // of step s + 1 have arrived and nobody reads step s any more, so that
    // step s + 2 may be fetched over it.
    auto arrive = [&] {
        __builtin_amdgcn_s_waitcnt(0);  // loads to LDS are counted with the vector loads: a barrier does not wait for them
        __syncthreads();
    };
    const auto nothing = [](int) {};
    fetch(0, x_even, w_even);
    fetch(1, x_odd, w_odd);
    fetch_scales(0, scales[0]);
    arrive();
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        w0[j] = read_w(w_even, 0, j);
        sw[j] = read_sw(scales[0], j);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        read_x(x_even, 0, i);
        sx[i] = read_sx(scales[0], i);
    }
    for (int s = 0; s < steps; s += 2) {  // what lies past the last step is zeros
        uint8_t* const next = scales[(s >> 1) + 1 & 1];
        multiply(std::integral_constant<int, 0>{}, w0, x_even, w_even, 1, w1, next, nothing);
        arrive();
        fetch_scales((s >> 1) + 1, next);
        const Fetch even = fetch_of(s + 2);
        multiply(std::integral_constant<int, 1>{}, w1, x_odd, w_odd, 0, w0, next,
                 [&](int n) { fetch_one(n, even, x_even, w_even); });
        multiply(std::integral_constant<int, 2>{}, w0, x_odd, w_odd, 1, w1, next, nothing);
        arrive();
        const Fetch odd = fetch_of(s + 3);
        multiply(std::integral_constant<int, 3>{}, w1, x_even, w_even, 0, w0, next,
                 [&](int n) { fetch_one(n, odd, x_odd, w_odd); });
    }
    float bias[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) bias[e] = 0.0f;
    if (p.bias) {
#pragma unroll
        for (int e = 0; e < 16; ++e) bias[e] = E::one(static_cast<const T*>(p.bias)[n0 + wn + 16 * q + e]);
    }
    arrive();  // the operands are read, and the last loads are done
    // A region for each wave, in the array that has room for it.
    constexpr int kPart = 16384, kIn = BM * kDepth / kPart;
    static_assert(BM == BN && 4 * kIn >= 8, "a region for every wave");
    uint8_t* region = (wave < 4 ? (wave < kIn ? x_even : x_odd) : (wave - 4 < kIn ? w_even : w_odd)) + wave % kIn * kPart;
    store_tile<E, T, TM, kPart, true>(p, static_cast<T*>(p.out), region, lane, m0 + wm, n0 + wn, acc, bias,
                                      packed && (n0 * sizeof(T)) % 16 == 0);
}

// The smaller tiles, of 32 TM rows and 128 channels, four waves, with a ring of S
// steps in LDS: a step's loads are issued S - 1 steps ahead, so that their latency
// is not what a step takes.  What the depth does not fill is fetched from past
// the operand's range, which leaves zeros.
//
// With E = MSums the depth is split as well: workgroups (x, y) take the bytes
// from y part_depth on, at most part_depth (whole pairs of steps), and store
// their sums as they are, one matrix after the other.
constexpr int kRingChannels = 128;

template <class E, int TM, int S>
__global__ __launch_bounds__(kThreads) void mx_ring_kernel(const MxProduct p, int m_tiles, int n_tiles, int part_depth,
                                                           bool packed) {
    constexpr bool kSplit = kSums<E>;
    using T = std::conditional_t<kSplit, float, typename E::T>;
    constexpr int WM = 2, TN = 4, BM = WM * TM * 16, BN = kRingChannels, kStage = (BM + BN) * kDepth;
    constexpr int kXLoads = TM, kWLoads = 4, kLoads = kXLoads + kWLoads;  // a thread a step
    constexpr int kRound = kThreads / 8;                                   // rows a load
    static_assert(S == 2 || S == 4, "whole pairs of steps, stages with names");
    // The rows whose scales a thread carries: whole waves for x, then those of w.
    constexpr int kXWaves = (BM + kWave - 1) / kWave, kWRows = kXWaves * kWave;
    static_assert(kWRows + BN <= kThreads, "a thread for the scales of every row");
    // Arrays by name: the compiler then sees that the operands it reads are not
    // those on their way, and puts no wait for the loads before the reads.
    __shared__ __align__(1024) uint8_t stage0[kStage], stage1[kStage], stage2[S > 2 ? kStage : 16],
        stage3[S > 3 ? kStage : 16];
    __shared__ __align__(4096) uint8_t scales[2][kThreads * 16];  // of a pair of steps, see pair_order
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, q = lane >> 4;
    const int wm = (wave % WM) * TM * 16, wn = (wave / WM) * TN * 16;
    const int tiles = m_tiles * n_tiles, per = (tiles + 7) / 8;
    const int t = static_cast<int>(blockIdx.x & 7) * per + static_cast<int>(blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= per || t >= tiles) return;
    const int first = kSplit ? static_cast<int>(blockIdx.y) * part_depth : 0;
    const int K = kSplit ? min(p.K - first, part_depth) : p.K;
    // XCDs and the tiles' order: see mx_large_kernel.
    constexpr int kGroupM = 8;
    const int group = t / (kGroupM * n_tiles), in = t - group * kGroupM * n_tiles;
    const int gm = min(kGroupM, m_tiles - group * kGroupM);
    const int64_t m0 = min<int64_t>(static_cast<int64_t>(group * kGroupM + in % gm) * BM, p.M - BM);
    const int n0 = min(in / gm * BN, p.N - BN);
    const uint8_t* xb = p.x + m0 * p.ldx + first;
    const uint8_t* wb = p.w + static_cast<int64_t>(n0) * p.ldw + first;
    const uint8_t* sb = (wave < kXWaves ? p.xs + m0 * p.ldxs : p.ws + n0 * p.ldws) + first / kMxBlockBytes;
    const int so = wave < kXWaves ? min(static_cast<int>(threadIdx.x), BM - 1) * static_cast<int>(p.ldxs)
                                  : min(static_cast<int>(threadIdx.x) - kWRows, BN - 1) * static_cast<int>(p.ldws);

    const int row0 = threadIdx.x >> 3, piece0 = lane & 7;
    const int ldx = static_cast<int>(p.ldx), ldw = static_cast<int>(p.ldw);
    static_assert(kRound % (8 * TN) == 0, "the keys repeat from load to load");
    const int xpiece = 16 * (piece0 ^ mx_key_x(row0)), wpiece = 16 * (piece0 ^ mx_key_w<TN>(row0));
    struct Fetch {  // of a step
        int k, xo, wo;
    };
    auto fetch_of = [&](int s) {
        const int k = s * kDepth;
        return Fetch{k, k + xpiece < K ? row0 * ldx + xpiece : kNowhere, k + wpiece < K ? row0 * ldw + wpiece : kNowhere};
    };
    auto fetch_one = [&](int n, const Fetch& f, uint8_t* to) {
        if (n < kXLoads)
            load16_to_lds(buf_rsrc(xb, 0x7FFFFFFF), to + (n * kThreads + wave * kWave) * 16, f.xo, f.k + n * kRound * ldx);
        else
            load16_to_lds(buf_rsrc(wb, 0x7FFFFFFF), to + (n * kThreads + wave * kWave) * 16, f.wo,
                          f.k + (n - kXLoads) * kRound * ldw);
    };
    auto fetch = [&](int s, uint8_t* to) {
        const Fetch f = fetch_of(s);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) fetch_one(n, f, to);
    };
    // Scales of a pair: those of whole pairs from memory, the last, partial one's
    // fetched byte by byte beforehand, zeros past it.
    const int blocks = K / kMxBlockBytes, whole = blocks / 16;
    auto fetch_scales = [&](int pair) -> u32x4 {
        return __builtin_amdgcn_raw_buffer_load_b128(buf_rsrc(sb, whole > 0 ? 0x7FFFFFFF : 0), so, 16 * min(pair, max(whole - 1, 0)), 0);
    };
    u32x4 last = {0u, 0u, 0u, 0u};
    if (whole * 16 < blocks) {
        const uint2 a = tail_scales(sb + so, whole * 16, blocks), b = tail_scales(sb + so, whole * 16 + 8, blocks);
        last = u32x4{a.x, a.y, b.x, b.y};
    }
    auto put_scales = [&](int pair, const u32x4& v) {
        u32x4 s;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = pair < whole ? v[i] : pair == whole ? last[i] : 0u;
        *reinterpret_cast<u32x4*>(scales[pair & 1] + threadIdx.x * 16) = pair_order(s);
    };

    const int w_row = operand_channel<TN>(0, l16);
    const int xp = (wm + l16) * kDepth, wp = (BM + wn + w_row) * kDepth;
    const int xkey = mx_key_x(l16), wkey = mx_key_w<TN>(w_row);
    const int xsp = (wm + l16) * 16 + 4 * q, wsp = (kWRows + wn + w_row) * 16 + 4 * q;
    f32x4 acc[TM][TN] = {};
    i32x4 x[TM], w0[TN], w1[TN];
    uint32_t sx[TM], sw[TN], sw_next[TN];
    auto read_x = [&](const uint8_t* from, int h, int i) {
        x[i] = *reinterpret_cast<const i32x4*>(from + xp + 16 * ((2 * q + h) ^ xkey) + 16 * i * kDepth);
    };
    auto read_w = [&](const uint8_t* from, int h, int j) {
        return *reinterpret_cast<const i32x4*>(from + wp + 16 * ((2 * q + h) ^ wkey) + 4 * j * kDepth);
    };
    auto read_sx = [&](const uint8_t* from, int i) { return *reinterpret_cast<const uint32_t*>(from + xsp + 16 * i * 16); };
    auto read_sw = [&](const uint8_t* from, int j) { return *reinterpret_cast<const uint32_t*>(from + wsp + 4 * j * 16); };
    // As in mx_large_kernel: half h of `next` is read while half a step is
    // multiplied, in SEL 3 the next pair's scales with it.
    constexpr int kPer = TN / TM, kPerLoads = (kLoads + TM - 1) / TM;
    auto multiply = [&](auto sel, const i32x4 (&w)[TN], const uint8_t* next, int h, i32x4 (&w_next)[TN], const uint8_t* scales_next,
                        const auto& load) {
        constexpr int SEL = decltype(sel)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma<SEL>(w[j], x[i], acc[i][j], sw[j], sx[i]);
            read_x(next, h, i);
#pragma unroll
            for (int j = i * kPer; j < (i + 1) * kPer; ++j) {
                w_next[j] = read_w(next, h, j);
                if (SEL == 3) sw_next[j] = read_sw(scales_next, j);
            }
            if (SEL == 3) sx[i] = read_sx(scales_next, i);
#pragma unroll
            for (int n = i * kPerLoads; n < (i + 1) * kPerLoads && n < kLoads; ++n) load(n);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (SEL == 3) {
#pragma unroll
            for (int j = 0; j < TN; ++j) sw[j] = sw_next[j];
        }
    };
    // A step: its first half's operands are in registers.  Past the barrier the
    // next step's operands have arrived (of the loads on their way only those of
    // the steps after it are newer), and nobody reads this step's stage any more,
    // over which the step S further goes.
    auto step = [&](auto odd, int s, uint8_t* now, const uint8_t* next, u32x4& carried) {
        constexpr int SEL = 2 * decltype(odd)::value;
        uint8_t* const scales_next = scales[(s >> 1) + 1 & 1];
        multiply(std::integral_constant<int, SEL>{}, w0, now, 1, w1, scales_next, [](int) {});
        landed<(S - 2) * kLoads>();
        barrier_in_flight();
        if constexpr (SEL == 0) {
            put_scales((s >> 1) + 1, carried);
            carried = fetch_scales((s >> 1) + 1 + S / 2);
            __builtin_amdgcn_sched_barrier(0);  // older than the step's loads: to wait for it is not to wait for them
        }
        const Fetch f = fetch_of(s + S);
        multiply(std::integral_constant<int, SEL + 1>{}, w1, next, 0, w0, scales_next, [&](int n) { fetch_one(n, f, now); });
    };
    const int steps = (K + kDepth - 1) / kDepth;
    const u32x4 scales0 = fetch_scales(0);
    u32x4 carried[S / 2];
#pragma unroll
    for (int i = 0; i < S / 2; ++i) carried[i] = fetch_scales(i + 1);
    __builtin_amdgcn_sched_barrier(0);
    uint8_t* const stage[4] = {stage0, stage1, stage2, stage3};
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, stage[i]);
    put_scales(0, scales0);
    landed<(S - 1) * kLoads>();
    barrier_in_flight();
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        w0[j] = read_w(stage0, 0, j);
        sw[j] = read_sw(scales[0], j);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        read_x(stage0, 0, i);
        sx[i] = read_sx(scales[0], i);
    }
    for (int s = 0; s < steps; s += S) {  // what lies past the last step is zeros
#pragma unroll
        for (int i = 0; i < S; i += 2) {
            step(std::integral_constant<int, 0>{}, s + i, stage[i % S], stage[(i + 1) % S], carried[i / 2]);
            step(std::integral_constant<int, 1>{}, s + i + 1, stage[(i + 1) % S], stage[(i + 2) % S], carried[i / 2]);
        }
    }
    T* out = static_cast<T*>(p.out);
    if constexpr (kSplit) out += blockIdx.y * p.M * p.ldo;
    float bias[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) bias[e] = 0.0f;
    if constexpr (!kSplit) {
        if (p.bias) {
#pragma unroll
            for (int e = 0; e < 16; ++e) bias[e] = E::one(static_cast<const T*>(p.bias)[n0 + wn + 16 * q + e]);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();  // the operands are read, and the last loads are done
    constexpr int kPart = BM >= 128 ? 8192 : 4096;  // a region for each wave
    static_assert(4 * kPart <= kStage, "they fit into a stage");
    store_tile<E, T, TM, kPart, (BM >= 128 && !kSplit)>(p, out, stage0 + wave * kPart, lane, m0 + wm, n0 + wn, acc, bias,
                                                        packed && (n0 * sizeof(T)) % 16 == 0);
}

// Scales of rows to the order of pairs of steps: a wave takes 8 pairs of 8 rows,
// whole cache lines on either side.  11008 x 4096: 4.9 us.  With scales read in
// rows 8192^3 took 249 us, with these 237.
__global__ __launch_bounds__(kThreads) void mx_pair_scales_kernel(const uint8_t* __restrict__ from, int64_t lds, int64_t rows,
                                                                  int blocks, uint8_t* __restrict__ to, int64_t plane) {
    const int lane = __lane_id();
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * kWavesPerGroup + threadIdx.x / kWave) * 8 + lane / 8;
    if (row >= rows) return;
    for (int pair = blockIdx.y * 8 + lane % 8; pair * 16 < blocks; pair += gridDim.y * 8) {
        const uint8_t* at = from + row * lds + pair * 16;
        u32x4 s = {0u, 0u, 0u, 0u};
        if (pair * 16 + 16 <= blocks) {
            s = load16_any(at);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (pair * 16 + i < blocks) s[i / 4] |= static_cast<uint32_t>(at[i]) << (8 * (i % 4));
        }
        *reinterpret_cast<u32x4*>(to + pair * plane + row * 16) = pair_order(s);
    }
}

// Adds the parts' sums and the bias: four channels a thread.
template <class E>
__global__ __launch_bounds__(kThreads) void mx_add_parts_kernel(const MxProduct p, const float* __restrict__ sums,
                                                                int64_t ld, int parts, bool packed) {
    const uint32_t pieces = static_cast<uint32_t>(p.N + 3) / 4, at = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t m = at / pieces;
    if (m >= p.M) return;
    const int n = static_cast<int>(at - m * pieces) * 4;
    const float* s = sums + m * ld + n;
    f32x4 acc = *reinterpret_cast<const f32x4*>(s);
    for (int i = 1; i < parts; ++i) acc += *reinterpret_cast<const f32x4*>(s + i * (p.M * ld));
    store_out4<E>(p, m, n, acc, packed);
}

template <class E, int MT, int TN, int WAVES>
int launch_few(const MxProduct& p, void* stream) {
    const int m_tiles = static_cast<int>((p.M + MT * 16 - 1) / (MT * 16)), n_tiles = (p.N + TN * 16 - 1) / (TN * 16);
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(m_tiles) * n_tiles + 7) / 8 * 8);
    hipLaunchKernelGGL((mx_few_rows_kernel<E, MT, TN, WAVES>), dim3(grid), dim3(WAVES * kWave), 0,
                       static_cast<hipStream_t>(stream), p, m_tiles, out_aligned(p, sizeof(typename E::T), 4 * sizeof(typename E::T)));
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_large(const MxProduct& p, void* stream) {
    const int m_tiles = static_cast<int>((p.M + 255) / 256), n_tiles = (p.N + 255) / 256;
    hipLaunchKernelGGL((mx_large_kernel<E>), dim3(static_cast<unsigned>((static_cast<int64_t>(m_tiles) * n_tiles + 7) / 8 * 8)),
                       dim3(8 * kWave), 0, static_cast<hipStream_t>(stream), p, m_tiles, n_tiles,
                       out_aligned(p, sizeof(typename E::T), 16));
    return static_cast<int>(hipGetLastError());
}

// Four steps of the ring where every workgroup has a compute unit of its own, two
// where several share one and hide each other's latency.  64 x 128, 512 x 4096 x
// 4096 (256 workgroups): 12.9 us with two, 9.9 with four, but 1024 x 4096 x 4096 16.8
// and 18.3, 4096 x 4096 x 512 17.0 and 33.0; 128 x 128, 1024 x 4096 x 4096 16.3 and 14.6,
// 2048 x 4096 x 4096 23.5 and 27.4.
template <class E, int TM>
int launch_ring(const MxProduct& p, void* stream) {
    constexpr int BM = 32 * TM;
    const int m_tiles = static_cast<int>((p.M + BM - 1) / BM), n_tiles = (p.N + kRingChannels - 1) / kRingChannels;
    const int64_t tiles = static_cast<int64_t>(m_tiles) * n_tiles;
    const dim3 grid(static_cast<unsigned>((tiles + 7) / 8 * 8));
    const bool packed = out_aligned(p, sizeof(typename E::T), 16);
    if (tiles <= device_cu_count())
        hipLaunchKernelGGL((mx_ring_kernel<E, TM, 4>), grid, dim3(kThreads), 0, static_cast<hipStream_t>(stream), p, m_tiles,
                           n_tiles, 0, packed);
    else
        hipLaunchKernelGGL((mx_ring_kernel<E, TM, 2>), grid, dim3(kThreads), 0, static_cast<hipStream_t>(stream), p, m_tiles,
                           n_tiles, 0, packed);
    return static_cast<int>(hipGetLastError());
}

// Tiles of 128 x 128 with the depth in parts (as many as split_depth leaves).
template <class E>
int launch_split(const MxProduct& p, int parts, void* workspace, void* stream) {
    const int m_tiles = static_cast<int>((p.M + kSplitTile - 1) / kSplitTile);
    const int n_tiles = (p.N + kSplitTile - 1) / kSplitTile;
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(m_tiles) * n_tiles + 7) / 8 * 8);
    const int part_depth = split_depth(p.K, parts);
    MxProduct s = p;
    s.out = workspace;
    s.ldo = sums_ld(p.N);
    if (static_cast<int64_t>(m_tiles) * n_tiles * parts <= device_cu_count())
        hipLaunchKernelGGL((mx_ring_kernel<MSums, 4, 4>), dim3(grid, parts), dim3(kThreads), 0,
                           static_cast<hipStream_t>(stream), s, m_tiles, n_tiles, part_depth, true);
    else
        hipLaunchKernelGGL((mx_ring_kernel<MSums, 4, 2>), dim3(grid, parts), dim3(kThreads), 0,
                           static_cast<hipStream_t>(stream), s, m_tiles, n_tiles, part_depth, true);
    const int e = static_cast<int>(hipGetLastError());
    if (e != 0) return e;
    const uint32_t pieces = static_cast<uint32_t>(p.M) * (static_cast<uint32_t>(p.N + 3) / 4);
    hipLaunchKernelGGL((mx_add_parts_kernel<E>), dim3((pieces + kThreads - 1) / kThreads), dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), p, static_cast<const float*>(workspace), s.ldo, parts,
                       out_aligned(p, sizeof(typename E::T), 4 * sizeof(typename E::T)));
    return static_cast<int>(hipGetLastError());
}

// The waves that split the depth: up to eight whose operands do not fill the LDS
// (another one that does took 8 x 16256 x 3968 from 12.8 to 13.9 us, 48 x 6272 x 3200
// from 9.2 to 10.3, 7007 x 103 x 2304 from 8.4 to 8.9; two fewer 13.0, 9.7, 8.8), but
// for the smallest pieces, several of which share a compute unit.  16 x 16, in 4 / 8 /
// 16 waves with operands from memory: 6 x 1216 x 768 3.1 / 3.4 / 4.0 us, 16 x 4096 x 4096
// 5.5 / 5.9 / 7.2, 16 x 1024 x 8192 6.8 / 6.9 / 8.1, 1 x 4096 x 8192 7.1 / 6.9 / 7.7, 16 x
// 2048 x 16384 10.2 / 10.5 / 11.9, 8 x 1024 x 32768 15.0 / 14.3 / 16.1: 4 up to a depth of
// 8192, beyond which the two are within 5% of each other.
template <class E>
int launch_few_tile(const MxProduct& p, Int8Few f, void* stream) {
    switch (10 * f.mt + f.tn) {
        case 11: return p.K <= 4096 ? launch_few<E, 1, 1, 4>(p, stream) : launch_few<E, 1, 1, 8>(p, stream);
        case 12: return launch_few<E, 1, 2, 8>(p, stream);
        case 13: return launch_few<E, 1, 3, 8>(p, stream);
        case 14: return launch_few<E, 1, 4, 7>(p, stream);
        case 22: return launch_few<E, 2, 2, 8>(p, stream);
        case 24: return launch_few<E, 2, 4, 6>(p, stream);
        case 32: return launch_few<E, 3, 2, 6>(p, stream);
        case 34: return launch_few<E, 3, 4, 5>(p, stream);
        case 44: return launch_few<E, 4, 4, 4>(p, stream);
        case 53: return launch_few<E, 5, 3, 4>(p, stream);
        default: return launch_few<E, 5, 4, 4>(p, stream);
    }
}

template <class E>
int launch_form(const MxProduct& p, const Int8Choice& c, void* workspace, void* stream) {
    if (c.parts > 1) return launch_split<E>(p, c.parts, workspace, stream);
    switch (c.bm) {
        case 0: return launch_few_tile<E>(p, c.few, stream);
        case 32: return launch_ring<E, 1>(p, stream);
        case 64: return launch_ring<E, 2>(p, stream);
        case 128: return launch_ring<E, 4>(p, stream);
        default: return launch_large<E>(p, stream);
    }
}

// Scales that are not in the order of pairs of steps yet, to the workspace.
int pair_scales(MxProduct& p, uint8_t* workspace, void* stream) {
    auto pair = [&](const uint8_t*& scales, int64_t& ld, int64_t rows, bool& paired) {
        if (paired) return 0;
        const int64_t plane = rows * 16;
        const int eights = (p.K + 16 * kDepth - 1) / (16 * kDepth);
        constexpr int kRows = 8 * kWavesPerGroup;
        hipLaunchKernelGGL(mx_pair_scales_kernel,
                           dim3(static_cast<unsigned>((rows + kRows - 1) / kRows), eights < 4096 ? eights : 4096),
                           dim3(kThreads), 0, static_cast<hipStream_t>(stream), scales, ld, rows, p.K / kMxBlockBytes, workspace,
                           plane);
        scales = workspace;
        ld = plane;
        paired = true;
        workspace += mx_paired_bytes(rows, p.K);
        return static_cast<int>(hipGetLastError());
    };
    const int e = pair(p.xs, p.ldxs, p.M, p.x_paired);
    return e != 0 ? e : pair(p.ws, p.ldws, p.N, p.w_paired);
}

template <class E>
int launch_product_e(const MxProduct& whole, void* workspace, void* stream) {
    using T = typename E::T;
    const int64_t cus = device_cu_count();
    for (int64_t n = 0; n < whole.N; n += kMaxChannels) {
        for (int64_t m = 0; m < whole.M; m += kRowBlock) {
            MxProduct p = whole;
            p.M = whole.M - m < kRowBlock ? whole.M - m : kRowBlock;
            p.N = static_cast<int>(whole.N - n < kMaxChannels ? whole.N - n : kMaxChannels);
            p.x += m * p.ldx;
            p.xs += m * p.ldxs;  // m = 0 and n = 0 where the scales are paired
            p.w += n * p.ldw;
            p.ws += n * p.ldws;
            if (p.bias) p.bias = static_cast<const T*>(p.bias) + n;
            p.out = static_cast<T*>(p.out) + m * p.ldo + n;
            const Int8Choice c = mx_choose(p.M, p.N, p.K, cus);
            int e = c.bm == kPairedRows ? pair_scales(p, static_cast<uint8_t*>(workspace), stream) : 0;
            if (e != 0) return e;
            e = launch_form<E>(p, c, workspace, stream);
            if (e != 0) return e;
        }
    }
    return 0;
}

template <class E, int TN, int WAVES>
int launch_tokens_t(const MxProduct& p, int d, const void* X, int64_t ldX, void* stream) {
    hipLaunchKernelGGL((mx_tokens_kernel<E, TN, WAVES>), dim3((p.N + TN * 16 - 1) / (TN * 16)), dim3(WAVES * kWave), 0,
                       static_cast<hipStream_t>(stream), p, d, static_cast<const typename E::T*>(X), ldX,
                       out_aligned(p, sizeof(typename E::T), 4 * sizeof(typename E::T)));
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_tokens_e(const MxProduct& p, int d, const void* X, int64_t ldX, void* stream) {
    // Channels a workgroup by the rounds they take, a wider one's counted two and three
    // times.  With 16, 48 and 64: 1 x 4096 x 4096 5.0, 6.7 and 7.9 us, 1 x 11008 x 4096
    // 11.9, 7.8 and 8.8, 1 x 14336 x 4096 15.3, 13.1 and 9.3, 4 x 16384 x 4096 18.6, 14.8 and
    // 10.2 (weights from memory).
    const int cus = device_cu_count();
    auto rounds = [&](int channels) { return (p.N + channels * cus - 1) / (channels * cus); };
    const int c16 = rounds(16), c48 = 2 * rounds(48), c64 = 3 * rounds(64);
    if (c64 <= c48 && c64 <= c16) return launch_tokens_t<E, 4, 8>(p, d, X, ldX, stream);
    if (c48 <= c16) return launch_tokens_t<E, 3, 8>(p, d, X, ldX, stream);
    return launch_tokens_t<E, 1, 16>(p, d, X, ldX, stream);
}

// Rows of a launch: the threads of their pieces of 512 values, 16 a piece,
// count in 32 bits.
int64_t rows_a_launch(int64_t per_row) { return (int64_t(1) << 27) / per_row; }

template <class E>
int launch_quantize_e(const void* X, int64_t rows, int d, int64_t ldx, const MxCoded& out, void* stream) {
    const uint32_t per_row = static_cast<uint32_t>((d + 511) / 512);
    const int64_t most = rows_a_launch(per_row);
    for (int64_t r = 0; r < rows; r += most) {
        const uint32_t items = static_cast<uint32_t>((rows - r < most ? rows - r : most) * per_row);
        const dim3 grid((items + kWavesPerGroup * kRowItems - 1) / (kWavesPerGroup * kRowItems));
        MxCoded c = out;
        c.codes += r * c.ldc;
        c.scales += r * (c.paired ? 16 : c.lds);
        hipLaunchKernelGGL((mx_quantize_kernel<E>), grid, dim3(kThreads), 0, static_cast<hipStream_t>(stream),
                           static_cast<const typename E::T*>(X) + r * ldx, items, per_row, d, ldx, c);
        const int e = static_cast<int>(hipGetLastError());
        if (e != 0) return e;
    }
    return 0;
}

template <class E>
int launch_columns_e(const MxColumns* jobs, int count, void* stream) {
    static_assert(kMxSumRows == int64_t(kMxBlock) * kColBlocks, "a row of sums a row of workgroups");
    constexpr int kTile = kWave * kCols<E>;
    constexpr uint32_t kMost = 1u << 22;  // workgroups of a launch: its threads count in 32 bits
    ColumnJobs c{};
    uint32_t all = 0;
    for (int i = 0; i < kMxColumnJobs; ++i) {
        if (i < count) {
            c.job[i] = jobs[i];
            c.across[i] = static_cast<uint32_t>((jobs[i].cols + kTile - 1) / kTile);
            all += c.across[i] * static_cast<uint32_t>(mx_sum_groups(jobs[i].rows));
        }
        c.end[i] = all;
    }
    for (uint32_t first = 0; first < all; first += kMost) {
        const dim3 grid(all - first < kMost ? all - first : kMost);
        if (c.job[0].by_rows.codes)
            hipLaunchKernelGGL((mx_quantize_columns_kernel<E, true>), grid, dim3(kColBlocks * kWave), 0,
                               static_cast<hipStream_t>(stream), c, first);
        else
            hipLaunchKernelGGL((mx_quantize_columns_kernel<E, false>), grid, dim3(kColBlocks * kWave), 0,
                               static_cast<hipStream_t>(stream), c, first);
        const int e = static_cast<int>(hipGetLastError());
        if (e != 0) return e;
    }
    return 0;
}

template <class E>
int launch_dequantize_e(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t rows, int d,
                        void* out, int64_t ldo, void* stream) {
    const uint32_t per_row = static_cast<uint32_t>((d + 511) / 512);
    const int64_t most = rows_a_launch(per_row);
    for (int64_t r = 0; r < rows; r += most) {
        const uint32_t items = static_cast<uint32_t>((rows - r < most ? rows - r : most) * per_row);
        const dim3 grid((items + kWavesPerGroup * kRowItems - 1) / (kWavesPerGroup * kRowItems));
        hipLaunchKernelGGL((mx_dequantize_kernel<E>), grid, dim3(kThreads), 0, static_cast<hipStream_t>(stream),
                           codes + r * ldc, ldc, scales + r * lds, lds, items, per_row, d,
                           static_cast<typename E::T*>(out) + r * ldo, ldo);
        const int e = static_cast<int>(hipGetLastError());
        if (e != 0) return e;
    }
    return 0;
}

}  // namespace

#define KBIT_BY_DTYPE(F, ...)                       \
    switch (t) {                                    \
        case Dtype::fp32: return F<QF32>(__VA_ARGS__); \
        case Dtype::fp16: return F<QF16>(__VA_ARGS__); \
        default: return F<QB16>(__VA_ARGS__);       \
    }

// The last pair of scales where it is not whole: what no block fills stays zero
// (a 255 there would make the zeros that stand for its codes NaN).
int clear_last_pair(const MxCoded& c, int64_t rows, int64_t blocks, void* stream) {
    if (!c.paired || blocks % 16 == 0) return 0;
    return launch_mx_zero(reinterpret_cast<float*>(c.scales + blocks / 16 * c.lds), rows, 4, 4, stream);
}

int launch_mx_quantize(Dtype t, const void* X, int64_t rows, int d, int64_t ldx, const MxCoded& c, void* stream) {
    const int e = clear_last_pair(c, rows, mx_blocks(d), stream);
    if (e != 0) return e;
    KBIT_BY_DTYPE(launch_quantize_e, X, rows, d, ldx, c, stream)
}

int launch_mx_quantize_columns(Dtype t, const MxColumns* jobs, int count, void* stream) {
    for (int i = 0; i < count; ++i) {
        const MxColumns& j = jobs[i];
        int e = j.columns.codes ? clear_last_pair(j.columns, j.cols, mx_blocks(j.rows), stream) : 0;
        if (e == 0 && j.by_rows.codes) e = clear_last_pair(j.by_rows, j.rows, mx_blocks(j.cols), stream);
        if (e != 0) return e;
    }
    KBIT_BY_DTYPE(launch_columns_e, jobs, count, stream)
}

int launch_mx_add_sums(const float* sums, int64_t groups, int cols, float* out, void* stream) {
    hipLaunchKernelGGL(mx_add_sums_kernel, dim3((cols + kWave - 1) / kWave), dim3(kWave), 0,
                       static_cast<hipStream_t>(stream), sums, groups, cols, out);
    return static_cast<int>(hipGetLastError());
}

int launch_mx_zero(float* out, int64_t rows, int cols, int64_t ldo, void* stream) {
    const dim3 grid(cols < 16 * kThreads ? (cols + kThreads - 1) / kThreads : 16, static_cast<unsigned>(rows < 4096 ? rows : 4096));
    hipLaunchKernelGGL(mx_zero_kernel, grid, dim3(kThreads), 0, static_cast<hipStream_t>(stream), out, rows, cols, ldo);
    return static_cast<int>(hipGetLastError());
}

int launch_mx_dequantize(Dtype t, const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t rows,
                         int d, void* out, int64_t ldo, void* stream) {
    KBIT_BY_DTYPE(launch_dequantize_e, codes, ldc, scales, lds, rows, d, out, ldo, stream)
}

int launch_mx_product(Dtype t, const MxProduct& p, void* workspace, void* stream) {
    KBIT_BY_DTYPE(launch_product_e, p, workspace, stream)
}

int launch_mx_tokens(Dtype t, const MxProduct& p, int d, const void* X, int64_t ldX, void* stream) {
    KBIT_BY_DTYPE(launch_tokens_e, p, d, X, ldX, stream)
}

}  // namespace kbit
