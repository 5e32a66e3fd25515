// Layer norm of rows and its gradient, for gfx950.
//
//   y  = (x - mean) r w + b,  r = 1 / sqrt(var + eps), var = mean((x - mean)^2)
//   dx = r (h - mean(h) - xh mean(h xh)),  h = dy w, xh = (x - mean) r
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// fp32 inside, one rounding to T.  A row stays in registers between its
// sums.  The mean is a pair m0 + m1: m0 the rounded mean of x, m1 that of
// x - m0, so that rows far from zero keep their digits (x - m0 is exact where
// it matters), and the variance is mean((x - m0)^2) - m1^2, which takes
// nothing more than the sums that m1 needs.
#include "kbit_internal.h"
#include "launch.h"
#include "matrix.h"
#include "mx_internal.h"

namespace kbit {
namespace {

// Sum over a wave; every lane ends with it.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_f32<kDppXor1>(v);
    v += dpp_f32<kDppXor2>(v);
    v += dpp_f32<kDppHalfMirror>(v);
    v += dpp_f32<kDppMirror>(v);
    v += shfl_xor_f32(v, 16);
    v += shfl_xor_f32(v, 32);
    return v;
}

// N sums over the WAVES waves of a row.  `red`: WAVES x N floats of LDS that
// no other sum before the next barrier uses.
template <int WAVES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (WAVES > 1) {
        if (__lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[wave * N + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = red[i];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) s += red[w * N + i];
            v[i] = s;
        }
    }
}

// Where a thread's elements stand: 8 neighbours in each of P pieces where
// rows start at 16 bytes, else single elements a thread apart.
template <bool VEC, int LANES>
__device__ __forceinline__ int column(int piece, int t, int e) {
    return VEC ? (piece * LANES + t) * 8 + e : (piece * 8 + e) * LANES + t;
}

template <class E, bool VEC, int LANES>
__device__ __forceinline__ void load_piece(const typename E::T* row, int piece, int t, int d, float (&x)[8]) {
    if constexpr (VEC) {
        load8<E, true>(row, (piece * LANES + t) * 8, d, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<VEC, LANES>(piece, t, e);
            x[e] = c < d ? E::one(row[c]) : 0.0f;
        }
    }
}

template <class E, bool VEC, int LANES>
__device__ __forceinline__ void load_weight(const void* w, bool fp32, int piece, int t, int d, float (&x)[8]) {
    if (fp32) load_piece<QF32, VEC, LANES>(static_cast<const float*>(w), piece, t, d, x);
    else load_piece<E, VEC, LANES>(static_cast<const typename E::T*>(w), piece, t, d, x);
}

template <class E, bool VEC, int LANES>
__device__ __forceinline__ void store_piece(typename E::T* row, int piece, int t, int d, const float (&v)[8]) {
    const int c0 = column<VEC, LANES>(piece, t, 0);
    if (VEC && c0 + 8 <= d) {
        if constexpr (sizeof(typename E::T) == 4) {
            store16<false>(row + c0, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
            store16<false>(row + c0 + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
        } else {
            store16<false>(row + c0, u32x4{E::pack(v[0], v[1]), E::pack(v[2], v[3]), E::pack(v[4], v[5]), E::pack(v[6], v[7])});
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<VEC, LANES>(piece, t, e);
            if (c < d) row[c] = E::narrow(v[e]);
        }
    }
}

// What a row's sums give.
struct Stats {
    float m0, m1, r;
};
__device__ __forceinline__ Stats stats_of(float m0, float sum1, float sum2, float inv_d, float eps) {
    const float m1 = sum1 * inv_d;
    const float var = fmaxf(sum2 * inv_d - m1 * m1, 0.0f);
    // fmaxf drops a NaN: a row that has one keeps it
    return Stats{m0, m1, 1.0f / sqrtf((sum2 != sum2 ? sum2 : var) + eps)};
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// WAVES waves a row, 4 / WAVES rows a workgroup of at least four waves; P
// pieces a thread.
template <class E, int WAVES, int P, bool VEC>
__global__ __launch_bounds__((WAVES < 4 ? 4 : WAVES) * kWave) void layer_norm_kernel(const LayerNormArgs p) {
    using T = typename E::T;
    constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1, LANES = WAVES * kWave;
    __shared__ float red[2][kRows * WAVES * 2];
    const int wave = threadIdx.x / kWave, t = threadIdx.x % LANES, sub = threadIdx.x / LANES, part = wave % WAVES;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub;
    if (WAVES == 1 && row >= p.rows) return;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const float inv_d = 1.0f / static_cast<float>(p.d);
    float v[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (i * LANES * 8 < p.d) {
            load_piece<E, VEC, LANES>(x, i, t, p.d, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[i][e];
    row_sums<WAVES, 1>(s, red[0] + sub * WAVES, part);
    const float m0 = s[0] * inv_d;
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[i][e] = column<VEC, LANES>(i, t, e) < p.d ? v[i][e] - m0 : 0.0f;
            s2[0] += v[i][e];
            s2[1] += v[i][e] * v[i][e];
        }
    row_sums<WAVES, 2>(s2, red[1] + sub * WAVES * 2, part);
    const Stats st = stats_of(m0, s2[0], s2[1], inv_d, p.eps);
    T* out = static_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (i * LANES * 8 >= p.d) break;
        float w[8], b[8];
        load_weight<E, VEC, LANES>(p.weight, p.weight_fp32, i, t, p.d, w);
        if (p.bias) load_weight<E, VEC, LANES>(p.bias, p.weight_fp32, i, t, p.d, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[i][e] = (v[i][e] - st.m1) * st.r * w[e];
            if (p.bias) v[i][e] = v[i][e] + b[e];
        }
        store_piece<E, VEC, LANES>(out, i, t, p.d, v[i]);
    }
}

// Rows that no workgroup holds: read once for each of the three steps, a row a
// workgroup of 16 waves.
constexpr int kLongWaves = 16, kLongLanes = kLongWaves * kWave;

template <class E, bool VEC>
__device__ __forceinline__ Stats long_stats(const typename E::T* x, int d, float eps, float (*red)[kLongWaves * 2]) {
    const int wave = threadIdx.x / kWave, t = threadIdx.x, pieces = (d + kLongLanes * 8 - 1) / (kLongLanes * 8);
    const float inv_d = 1.0f / static_cast<float>(d);
    float s[1] = {0.0f};
    for (int i = 0; i < pieces; ++i) {
        float v[8];
        load_piece<E, VEC, kLongLanes>(x, i, t, d, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[e];
    }
    row_sums<kLongWaves, 1>(s, red[0], wave);
    const float m0 = s[0] * inv_d;
    float s2[2] = {0.0f, 0.0f};
    for (int i = 0; i < pieces; ++i) {
        float v[8];
        load_piece<E, VEC, kLongLanes>(x, i, t, d, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = column<VEC, kLongLanes>(i, t, e) < d ? v[e] - m0 : 0.0f;
            s2[0] += c;
            s2[1] += c * c;
        }
    }
    row_sums<kLongWaves, 2>(s2, red[1], wave);
    return stats_of(m0, s2[0], s2[1], inv_d, eps);
}

template <class E, bool VEC>
__global__ __launch_bounds__(kLongLanes) void layer_norm_long_kernel(const LayerNormArgs p) {
    using T = typename E::T;
    __shared__ float red[2][kLongWaves * 2];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const Stats st = long_stats<E, VEC>(x, p.d, p.eps, red);
    T* out = static_cast<T*>(p.out) + row * p.ldo;
    const int t = threadIdx.x, pieces = (p.d + kLongLanes * 8 - 1) / (kLongLanes * 8);
    for (int i = 0; i < pieces; ++i) {
        float v[8], w[8], b[8];
        load_piece<E, VEC, kLongLanes>(x, i, t, p.d, v);
        load_weight<E, VEC, kLongLanes>(p.weight, p.weight_fp32, i, t, p.d, w);
        if (p.bias) load_weight<E, VEC, kLongLanes>(p.bias, p.weight_fp32, i, t, p.d, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = (v[e] - st.m0 - st.m1) * st.r * w[e];
            if (p.bias) v[e] = v[e] + b[e];
        }
        store_piece<E, VEC, kLongLanes>(out, i, t, p.d, v);
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// A workgroup takes rows groups apart and keeps the sums of the weights'
// gradients in registers; at the end they are one row of the workspace.
template <class E, int WAVES, int P, bool VEC>
__global__ __launch_bounds__((WAVES < 4 ? 4 : WAVES) * kWave) void layer_norm_back_kernel(const LayerNormBackArgs p,
                                                                                         float* __restrict__ partial) {
    using T = typename E::T;
    constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1, LANES = WAVES * kWave;
    __shared__ float red[3][kRows * WAVES * 2];  // one each for a row's three sums: a row's barriers part them from the next row's
    const int wave = threadIdx.x / kWave, t = threadIdx.x % LANES, sub = threadIdx.x / LANES, part = wave % WAVES;
    const float inv_d = 1.0f / static_cast<float>(p.d);
    constexpr bool kKeepWeight = P <= 2;  // in registers, else read from cache for every row
    float w[kKeepWeight ? P : 1][8], dw[P][8], db[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (kKeepWeight) load_weight<E, VEC, LANES>(p.weight, p.weight_fp32, i, t, p.d, w[kKeepWeight ? i : 0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.0f;
    }
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub; row < p.rows;
         row += static_cast<int64_t>(gridDim.x) * kRows) {
        const T* x = static_cast<const T*>(p.x) + row * p.ldx;
        const T* g = static_cast<const T*>(p.g) + row * p.ldg;
        float v[P][8], h[P][8];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            load_piece<E, VEC, LANES>(x, i, t, p.d, v[i]);
            load_piece<E, VEC, LANES>(g, i, t, p.d, h[i]);
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += v[i][e];
        row_sums<WAVES, 1>(s, red[0] + sub * WAVES, part);
        const float m0 = s[0] * inv_d;
        float s2[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = column<VEC, LANES>(i, t, e) < p.d ? v[i][e] - m0 : 0.0f;
                s2[0] += v[i][e];
                s2[1] += v[i][e] * v[i][e];
            }
        row_sums<WAVES, 2>(s2, red[1] + sub * WAVES * 2, part);
        const Stats st = stats_of(m0, s2[0], s2[1], inv_d, p.eps);
        const void* weight = p.weight;
        asm volatile("" : "+s"(weight));  // the loads stay in the loop
        float s3[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = kKeepWeight ? i : 0;
            if (!kKeepWeight) load_weight<E, VEC, LANES>(weight, p.weight_fp32, i, t, p.d, w[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (v[i][e] - st.m1) * st.r;
                v[i][e] = xh;
                dw[i][e] += h[i][e] * xh;
                db[i][e] += h[i][e];
                h[i][e] = h[i][e] * w[k][e];
                s3[0] += h[i][e];
                s3[1] += h[i][e] * xh;
            }
        }
        row_sums<WAVES, 2>(s3, red[2] + sub * WAVES * 2, part);
        const float mh = s3[0] * inv_d, mhx = s3[1] * inv_d;
        T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = st.r * (h[i][e] - mh - v[i][e] * mhx);
            store_piece<E, VEC, LANES>(dx, i, t, p.d, v[i]);
        }
    }
    if constexpr (kRows > 1) {  // the workgroup's rows, in their order
        __shared__ float sums[kRows - 1][2][P * 8 * LANES];
        if (sub > 0) {
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sums[sub - 1][0][(i * 8 + e) * LANES + t] = dw[i][e];
                    sums[sub - 1][1][(i * 8 + e) * LANES + t] = db[i][e];
                }
        }
        __syncthreads();
        if (sub > 0) return;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int r = 0; r < kRows - 1; ++r) {
                    dw[i][e] += sums[r][0][(i * 8 + e) * LANES + t];
                    db[i][e] += sums[r][1][(i * 8 + e) * LANES + t];
                }
    }
    float* to = partial + static_cast<int64_t>(blockIdx.x) * 2 * p.d;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<VEC, LANES>(i, t, e);
            if (c < p.d) {
                to[c] = dw[i][e];
                to[p.d + c] = db[i][e];
            }
        }
}

// Long rows: dx and the rows' statistics, then the sums over rows.
template <class E, bool VEC>
__global__ __launch_bounds__(kLongLanes) void layer_norm_back_long_kernel(const LayerNormBackArgs p,
                                                                          float* __restrict__ stats) {
    using T = typename E::T;
    __shared__ float red[3][kLongWaves * 2];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* g = static_cast<const T*>(p.g) + row * p.ldg;
    const Stats st = long_stats<E, VEC>(x, p.d, p.eps, red);
    const int t = threadIdx.x, wave = threadIdx.x / kWave, pieces = (p.d + kLongLanes * 8 - 1) / (kLongLanes * 8);
    const float inv_d = 1.0f / static_cast<float>(p.d);
    float s[2] = {0.0f, 0.0f};
    for (int i = 0; i < pieces; ++i) {
        float v[8], h[8], w[8];
        load_piece<E, VEC, kLongLanes>(x, i, t, p.d, v);
        load_piece<E, VEC, kLongLanes>(g, i, t, p.d, h);
        load_weight<E, VEC, kLongLanes>(p.weight, p.weight_fp32, i, t, p.d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // past the row h is 0
            s[0] += h[e] * w[e];
            s[1] += h[e] * w[e] * ((v[e] - st.m0 - st.m1) * st.r);
        }
    }
    row_sums<kLongWaves, 2>(s, red[2], wave);
    const float mh = s[0] * inv_d, mhx = s[1] * inv_d;
    if (t == 0) {
        stats[row * 4] = st.m0;
        stats[row * 4 + 1] = st.m1;
        stats[row * 4 + 2] = st.r;
    }
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    for (int i = 0; i < pieces; ++i) {
        float v[8], h[8], w[8];
        load_piece<E, VEC, kLongLanes>(x, i, t, p.d, v);
        load_piece<E, VEC, kLongLanes>(g, i, t, p.d, h);
        load_weight<E, VEC, kLongLanes>(p.weight, p.weight_fp32, i, t, p.d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = st.r * (h[e] * w[e] - mh - (v[e] - st.m0 - st.m1) * st.r * mhx);
        store_piece<E, VEC, kLongLanes>(dx, i, t, p.d, v);
    }
}

// A column a thread, rows groups apart.
template <class E>
__global__ __launch_bounds__(kThreads) void layer_norm_column_sums_kernel(const LayerNormBackArgs p,
                                                                          const float* __restrict__ stats,
                                                                          float* __restrict__ partial) {
    using T = typename E::T;
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= p.d) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float x = E::one(static_cast<const T*>(p.x)[row * p.ldx + c]);
        const float g = E::one(static_cast<const T*>(p.g)[row * p.ldg + c]);
        dw += g * ((x - stats[row * 4] - stats[row * 4 + 1]) * stats[row * 4 + 2]);
        db += g;
    }
    float* to = partial + static_cast<int64_t>(blockIdx.y) * 2 * p.d;
    to[c] = dw;
    to[p.d + c] = db;
}

// Adds the partial rows: 64 columns a workgroup, each wave a quarter of the
// rows, in a fixed order.
__global__ __launch_bounds__(kThreads) void layer_norm_add_kernel(const float* __restrict__ partial, int groups, int d,
                                                                  float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float sums[kWavesPerGroup][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + lane, width = 2 * static_cast<int64_t>(d);
    const int per = (groups + kWavesPerGroup - 1) / kWavesPerGroup;
    float s = 0.0f;
    if (c < width) {
        const int end = min(groups, (wave + 1) * per);
#pragma unroll 8
        for (int g = wave * per; g < end; ++g) s += partial[g * width + c];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < width) {
        s = ((sums[0][lane] + sums[1][lane]) + sums[2][lane]) + sums[3][lane];
        if (c < d) dweight[c] = s;
        else dbias[c - d] = s;
    }
}

template <class E, int WAVES, int P>
int launch_forward(const LayerNormArgs& p, bool vec, void* stream) {
    constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
    const dim3 grid(static_cast<unsigned>((p.rows + kRows - 1) / kRows)), block((WAVES < 4 ? 4 : WAVES) * kWave);
    if (vec)
        hipLaunchKernelGGL((layer_norm_kernel<E, WAVES, P, true>), grid, block, 0, static_cast<hipStream_t>(stream), p);
    else
        hipLaunchKernelGGL((layer_norm_kernel<E, WAVES, P, false>), grid, block, 0, static_cast<hipStream_t>(stream), p);
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_forward_e(const LayerNormArgs& whole, bool vec, void* stream) {
    using T = typename E::T;
    constexpr int64_t kMost = int64_t(1) << 22;  // rows a launch: its threads count in 32 bits
    for (int64_t r = 0; r < whole.rows; r += kMost) {
        LayerNormArgs p = whole;
        p.x = static_cast<const T*>(p.x) + r * p.ldx;
        p.out = static_cast<T*>(p.out) + r * p.ldo;
        p.rows = whole.rows - r < kMost ? whole.rows - r : kMost;
        int e;
        if (p.d <= 512) e = launch_forward<E, 1, 1>(p, vec, stream);
        else if (p.d <= 2048 && p.rows >= 4 * device_cu_count()) e = launch_forward<E, 1, 4>(p, vec, stream);
        else if (p.d <= 2048) e = launch_forward<E, 4, 1>(p, vec, stream);
        else if (p.d <= 4096) e = launch_forward<E, 4, 2>(p, vec, stream);
        else if (p.d <= 16384) e = launch_forward<E, 4, 8>(p, vec, stream);
        else if (p.d <= 32768) e = launch_forward<E, 16, 4>(p, vec, stream);
        else {
            if (vec)
                hipLaunchKernelGGL((layer_norm_long_kernel<E, true>), dim3(static_cast<unsigned>(p.rows)), dim3(kLongLanes), 0,
                                   static_cast<hipStream_t>(stream), p);
            else
                hipLaunchKernelGGL((layer_norm_long_kernel<E, false>), dim3(static_cast<unsigned>(p.rows)), dim3(kLongLanes), 0,
                                   static_cast<hipStream_t>(stream), p);
            e = static_cast<int>(hipGetLastError());
        }
        if (e != 0) return e;
    }
    return 0;
}

template <class E, int WAVES, int P, bool ANY = true>
int launch_back(const LayerNormBackArgs& p, int* groups, bool vec, void* stream) {
    constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
    const int64_t g = (p.rows + kRows - 1) / kRows;
    *groups = static_cast<int>(g < kLayerNormPartials ? g : kLayerNormPartials);
    const dim3 grid(static_cast<unsigned>(*groups)), block((WAVES < 4 ? 4 : WAVES) * kWave);
    if (vec)
        hipLaunchKernelGGL((layer_norm_back_kernel<E, WAVES, P, true>), grid, block, 0, static_cast<hipStream_t>(stream), p,
                           p.workspace);
    else if constexpr (ANY)
        hipLaunchKernelGGL((layer_norm_back_kernel<E, WAVES, P, false>), grid, block, 0, static_cast<hipStream_t>(stream),
                           p, p.workspace);
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_back_e(const LayerNormBackArgs& p, bool vec, void* stream) {
    int groups = 0, e = 0;
    if (p.rows == 0) {
        // the sum of no rows: groups = 0 below
    } else if (p.d <= 512) {
        e = launch_back<E, 1, 1>(p, &groups, vec, stream);
    } else if (p.d <= 2048) {
        e = launch_back<E, 4, 1>(p, &groups, vec, stream);
    } else if (p.d <= 4096) {
        e = launch_back<E, 4, 2>(p, &groups, vec, stream);
    } else if (p.d <= kLayerNormKeptAny) {
        e = launch_back<E, 8, 2>(p, &groups, vec, stream);
    } else if (p.d <= kLayerNormKept && vec) {  // 16 elements more a thread do not fit beside single elements' addresses
        e = launch_back<E, 8, 4, false>(p, &groups, vec, stream);
    } else {
        groups = static_cast<int>(p.rows < kLayerNormPartials ? p.rows : kLayerNormPartials);
        float* stats = p.workspace + static_cast<int64_t>(groups) * 2 * p.d;
        constexpr int64_t kMost = int64_t(1) << 21;
        for (int64_t r = 0; r < p.rows && e == 0; r += kMost) {
            using T = typename E::T;
            LayerNormBackArgs q = p;
            q.x = static_cast<const T*>(p.x) + r * p.ldx;
            q.g = static_cast<const T*>(p.g) + r * p.ldg;
            q.dx = static_cast<T*>(p.dx) + r * p.lddx;
            const dim3 grid(static_cast<unsigned>(p.rows - r < kMost ? p.rows - r : kMost));
            if (vec)
                hipLaunchKernelGGL((layer_norm_back_long_kernel<E, true>), grid, dim3(kLongLanes), 0,
                                   static_cast<hipStream_t>(stream), q, stats + r * 4);
            else
                hipLaunchKernelGGL((layer_norm_back_long_kernel<E, false>), grid, dim3(kLongLanes), 0,
                                   static_cast<hipStream_t>(stream), q, stats + r * 4);
            e = static_cast<int>(hipGetLastError());
        }
        if (e != 0) return e;
        hipLaunchKernelGGL((layer_norm_column_sums_kernel<E>), dim3((p.d + kThreads - 1) / kThreads, groups), dim3(kThreads),
                           0, static_cast<hipStream_t>(stream), p, stats, p.workspace);
        e = static_cast<int>(hipGetLastError());
    }
    if (e != 0) return e;
    hipLaunchKernelGGL(layer_norm_add_kernel, dim3(static_cast<unsigned>((2 * static_cast<int64_t>(p.d) + kWave - 1) / kWave)),
                       dim3(kThreads), 0, static_cast<hipStream_t>(stream), p.workspace, groups, p.d, p.dweight, p.dbias);
    return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_layer_norm(Dtype t, const LayerNormArgs& p, bool vec, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_forward_e<QF32>(p, vec, stream);
        case Dtype::fp16: return launch_forward_e<QF16>(p, vec, stream);
        default: return launch_forward_e<QB16>(p, vec, stream);
    }
}

int launch_layer_norm_back(Dtype t, const LayerNormBackArgs& p, bool vec, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_back_e<QF32>(p, vec, stream);
        case Dtype::fp16: return launch_back_e<QF16>(p, vec, stream);
        default: return launch_back_e<QB16>(p, vec, stream);
    }
}

}  // namespace kbit
