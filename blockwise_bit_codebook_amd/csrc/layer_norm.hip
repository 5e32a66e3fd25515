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

// N sums over the WAVES waves of a row (a power of two, at most 16), through
// `red`: WAVES x N floats of LDS that no other sum before the next barrier uses.
// Every lane fetches one wave's and adds them up with its neighbours.
template <int WAVES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (WAVES > 1) {
        if (__lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[wave * N + i] = v[i];
        }
        barrier_in_flight();  // the next row's loads and the last one's stores go on
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = red[__lane_id() % WAVES * N + i];
            s += dpp_f32<kDppXor1>(s);
            if (WAVES >= 4) s += dpp_f32<kDppXor2>(s);
            if (WAVES >= 8) s += dpp_f32<kDppHalfMirror>(s);
            if (WAVES >= 16) s += dpp_f32<kDppMirror>(s);
            v[i] = s;
        }
    }
}

// A thread's elements: 8 neighbours in each of P pieces, LANES x 8 elements
// apart.
template <int LANES>
__device__ __forceinline__ int column(int piece, int t) {
    return (piece * LANES + t) * 8;
}

// The same for rows that registers hold: loads and stores without a branch, so
// that the next row's may be on their way through a loop (a load under a
// condition is copied where the paths meet, which waits for it: 8192 x 4096 bf16
// gradient 55 us).  A piece that passes the row's end is moved back to end with
// it; the elements that it then shares with its neighbour count once, `counts`,
// but are computed and written by both, the same bits.  TINY: rows shorter than 8,
// element by element.
template <class E, int LANES, int P, bool TINY>
struct Pieces {
    using T = typename E::T;
    int at[P], skip[P], d;
    __device__ __forceinline__ Pieces(int t, int d_) : d(d_) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = column<LANES>(i, t);
            at[i] = TINY ? c : min(c, d - 8);
            skip[i] = c - at[i];
        }
    }
    __device__ __forceinline__ bool counts(int i, int e) const { return TINY ? at[i] + e < d : e >= skip[i]; }
    // The sum of a piece's values, of their products: only the last lanes of a row
    // have any that do not count.
    __device__ __forceinline__ float sum(int i, const float (&v)[8]) const {
        float s = v[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) s += v[e];
        if (TINY || skip[i] > 0) {
            s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += counts(i, e) ? v[e] : 0.0f;
        }
        return s;
    }
    __device__ __forceinline__ float sum(int i, const float (&a)[8], const float (&b)[8]) const {
        float s = a[0] * b[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) s = fmaf(a[e], b[e], s);
        if (TINY || skip[i] > 0) {
            s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = counts(i, e) ? fmaf(a[e], b[e], s) : s;
        }
        return s;
    }
    template <class F>
    __device__ __forceinline__ void load_raw(const typename F::T* row, int i, u32x4 (&r)[F::kVec]) const {
        if constexpr (TINY) {
            load8_raw<F>(row, at[i], d, r);
        } else {
#pragma unroll
            for (int k = 0; k < F::kVec; ++k) r[k] = load16_any(row + at[i] + 4 * k);
        }
    }
    __device__ __forceinline__ void load(const T* row, int i, float (&x)[8]) const {
        u32x4 r[E::kVec];
        load_raw<E>(row, i, r);
        E::widen(r, x);
    }
    __device__ __forceinline__ void weight(const void* w, bool fp32, int i, float (&x)[8]) const {
        if (fp32) {
            u32x4 r[QF32::kVec];
            load_raw<QF32>(static_cast<const float*>(w), i, r);
            QF32::widen(r, x);
        } else {
            load(static_cast<const T*>(w), i, x);
        }
    }
    // streamed: not to stay in L2
    __device__ __forceinline__ void store(T* row, int i, const float (&v)[8], bool streamed) const {
        if (TINY) {
            store8<E>(row, at[i], d, v);
        } else if (skip[i] < 8) {
            u32x4 r[E::kVec];
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int k = 0; k < 8; ++k) r[k / 4][k % 4] = __float_as_uint(v[k]);
            } else {
                r[0] = u32x4{E::pack(v[0], v[1]), E::pack(v[2], v[3]), E::pack(v[4], v[5]), E::pack(v[6], v[7])};
            }
#pragma unroll
            for (int k = 0; k < E::kVec; ++k) {
                auto* to = reinterpret_cast<u32x4_any*>(row + at[i] + 4 * k);
                if (streamed) __builtin_nontemporal_store(r[k], to);
                else *to = r[k];
            }
        }
    }
};

template <class E>
__device__ __forceinline__ void load8_any(const typename E::T* row, int c, int d, float (&x)[8]) {
    u32x4 r[E::kVec];
    load8_raw<E>(row, c, d, r);
    E::widen(r, x);
}

template <class E>
__device__ __forceinline__ void load_weight(const void* w, bool fp32, int c, int d, float (&x)[8]) {
    if (fp32) load8_any<QF32>(static_cast<const float*>(w), c, d, x);
    else load8_any<E>(static_cast<const typename E::T*>(w), c, d, x);
}

// What a row's sums give: (x - m0) r + shift is its normed value.
struct Stats {
    float r, shift, m1;
};
// 1 / sqrt(v), within 1 ulp: the instruction's own for all but the smallest v,
// which it would take for 0.
__device__ __forceinline__ float reciprocal_root(float v) {
    const bool small = v < 0x1p-100f;
    const float r = __builtin_amdgcn_rsqf(small ? v * 0x1p100f : v);
    return small ? r * 0x1p50f : r;
}
__device__ __forceinline__ Stats stats_of(float sum1, float sum2, float inv_d, float eps) {
    const float m1 = sum1 * inv_d;
    const float var = fmaxf(sum2 * inv_d - m1 * m1, 0.0f);
    // fmaxf drops a NaN: a row that has one keeps it
    const float r = reciprocal_root((sum2 != sum2 ? sum2 : var) + eps);
    return Stats{r, -m1 * r, m1};
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// WAVES waves a row, 4 / WAVES rows a workgroup of at least four waves; P
// pieces a thread.  Memory bounds it: 8192 x 4096 bf16 30 us (4.5 TB/s; a copy
// of that size runs at 5.2), 8192 x 1024 8.9, 2048 x 16384 31; 16 x 4096 4.4 us is the
// launch and two sums over a row.
template <class E, int WAVES, int P, bool TINY>
__global__ __launch_bounds__((WAVES < 4 ? 4 : WAVES) * kWave) void layer_norm_kernel(const LayerNormArgs p, bool streamed) {
    using T = typename E::T;
    constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1, LANES = WAVES * kWave;
    __shared__ float red[2][kRows * WAVES * 2];
    const int wave = threadIdx.x / kWave, t = threadIdx.x % LANES, sub = threadIdx.x / LANES, part = wave % WAVES;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub;
    if (WAVES == 1 && row >= p.rows) return;
    const Pieces<E, LANES, P, TINY> at(t, p.d);
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const float inv_d = 1.0f / static_cast<float>(p.d);
    float v[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) at.load(x, i, v[i]);
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < P; ++i) s[0] += at.sum(i, v[i]);
    row_sums<WAVES, 1>(s, red[0] + sub * WAVES, part);
    const float m0 = s[0] * inv_d;
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] - m0;
        s2[0] += at.sum(i, v[i]);
        s2[1] += at.sum(i, v[i], v[i]);
    }
    row_sums<WAVES, 2>(s2, red[1] + sub * WAVES * 2, part);
    const Stats st = stats_of(s2[0], s2[1], inv_d, p.eps);
    T* out = static_cast<T*>(p.out) + row * p.ldo;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (i * LANES * 8 >= p.d) break;
        float w[8], b[8];
        at.weight(p.weight, p.weight_fp32, i, w);
        if (p.bias) at.weight(p.bias, p.weight_fp32, i, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float xh = fmaf(v[i][e], st.r, st.shift);
            v[i][e] = p.bias ? fmaf(xh, w[e], b[e]) : xh * w[e];
        }
        at.store(out, i, v[i], streamed);
    }
}

// Rows that no workgroup holds: read once for each of the three steps, a row a
// workgroup of 16 waves.  512 x 70000 bf16 55 us, of which one reading and the
// outputs would be 28.
constexpr int kLongWaves = 16, kLongLanes = kLongWaves * kWave;

template <class E>
__device__ __forceinline__ Stats long_stats(const typename E::T* x, int d, float eps, float (*red)[kLongWaves * 2], float& m0) {
    const int wave = threadIdx.x / kWave, t = threadIdx.x, pieces = (d + kLongLanes * 8 - 1) / (kLongLanes * 8);
    const float inv_d = 1.0f / static_cast<float>(d);
    float s[1] = {0.0f};
    for (int i = 0; i < pieces; ++i) {
        float v[8];
        load8_any<E>(x, column<kLongLanes>(i, t), d, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[e];
    }
    row_sums<kLongWaves, 1>(s, red[0], wave);
    m0 = s[0] * inv_d;
    float s2[2] = {0.0f, 0.0f};
    for (int i = 0; i < pieces; ++i) {
        float v[8];
        load8_any<E>(x, column<kLongLanes>(i, t), d, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = column<kLongLanes>(i, t) + e < d ? v[e] - m0 : 0.0f;
            s2[0] += c;
            s2[1] += c * c;
        }
    }
    row_sums<kLongWaves, 2>(s2, red[1], wave);
    return stats_of(s2[0], s2[1], inv_d, eps);
}

template <class E>
__global__ __launch_bounds__(kLongLanes) void layer_norm_long_kernel(const LayerNormArgs p) {
    using T = typename E::T;
    __shared__ float red[2][kLongWaves * 2];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    float m0;
    const Stats st = long_stats<E>(x, p.d, p.eps, red, m0);
    T* out = static_cast<T*>(p.out) + row * p.ldo;
    const int t = threadIdx.x, pieces = (p.d + kLongLanes * 8 - 1) / (kLongLanes * 8);
    for (int i = 0; i < pieces; ++i) {
        float v[8], w[8], b[8];
        load8_any<E>(x, column<kLongLanes>(i, t), p.d, v);
        load_weight<E>(p.weight, p.weight_fp32, column<kLongLanes>(i, t), p.d, w);
        if (p.bias) load_weight<E>(p.bias, p.weight_fp32, column<kLongLanes>(i, t), p.d, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float xh = fmaf(v[e] - m0, st.r, st.shift);
            v[e] = p.bias ? fmaf(xh, w[e], b[e]) : xh * w[e];
        }
        store8<E>(out, column<kLongLanes>(i, t), p.d, v);
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// A workgroup takes ROWS rows at a time, WAVES waves each, and keeps the sums of
// the weights' gradients in registers; at the end they are one row of the
// workspace.  Two sums a row: its mean, then with c = x - m0 those of c, c^2, h
// and h c, from which mean(h xh) = r (sum(h c) - m1 sum(h)) / d.  The next row
// is on its way while one is summed.  8192 x 4096 bf16 41 us and 4 for the sums
// of 512 workgroups (4.4 TB/s together); shorter rows wait for the two sums of each
// row in turn: 8192 x 1024 22.6 us (2.2 TB/s).  256, 768 and 1024 workgroups were slower.
template <class E, int WAVES, int ROWS, int P, bool TINY>
__global__ __launch_bounds__(WAVES* ROWS* kWave) void layer_norm_back_kernel(const LayerNormBackArgs p,
                                                                             float* __restrict__ partial, bool streamed) {
    using T = typename E::T;
    constexpr int LANES = WAVES * kWave;
    __shared__ float red[2][ROWS * WAVES * 4];  // one for each of a row's two sums: its barriers part them from the next row's
    const int wave = threadIdx.x / kWave, t = threadIdx.x % LANES, sub = threadIdx.x / LANES, part = wave % WAVES;
    const float inv_d = 1.0f / static_cast<float>(p.d);
    const Pieces<E, LANES, P, TINY> at(t, p.d);
    // Four pieces a thread leave no registers for the weight, which is read from
    // cache for every row then, nor for the next row.
    constexpr bool kKeepWeight = P <= 2, kAhead = P <= 2;
    float w[kKeepWeight ? P : 1][8], dw[P][8], db[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (kKeepWeight) at.weight(p.weight, p.weight_fp32, i, w[kKeepWeight ? i : 0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.0f;
    }
    struct Row {  // as it stands in memory
        u32x4 x[P][E::kVec], g[P][E::kVec];
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    auto fetch = [&](int64_t row, Row& to) {  // past the last row it is fetched again
        row = min(row, p.rows - 1);
        const T* x = static_cast<const T*>(p.x) + row * p.ldx;
        const T* g = static_cast<const T*>(p.g) + row * p.ldg;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            at.template load_raw<E>(x, i, to.x[i]);
            at.template load_raw<E>(g, i, to.g[i]);
        }
    };
    int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + sub;
    auto turn = [&](Row& now, Row& next) {
        float v[P][8], h[P][8];
        if (!kAhead) fetch(row, now);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            E::widen(now.x[i], v[i]);
            E::widen(now.g[i], h[i]);
        }
        if (kAhead) fetch(row + step, next);
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < P; ++i) s[0] += at.sum(i, v[i]);
        row_sums<WAVES, 1>(s, red[0] + sub * WAVES, part);
        const float m0 = s[0] * inv_d;
        const void* weight = p.weight;
        asm volatile("" : "+s"(weight));  // the loads stay in the loop
        float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = kKeepWeight ? i : 0;
            if (!kKeepWeight) at.weight(weight, p.weight_fp32, i, w[k]);
            float hw[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = v[i][e] - m0;
                hw[e] = h[i][e] * w[k][e];
            }
            s4[0] += at.sum(i, v[i]);
            s4[1] += at.sum(i, v[i], v[i]);
            s4[2] += at.sum(i, hw);
            s4[3] += at.sum(i, hw, v[i]);
        }
        row_sums<WAVES, 4>(s4, red[1] + sub * WAVES * 4, part);
        const Stats st = stats_of(s4[0], s4[1], inv_d, p.eps);
        const float mh = s4[2] * inv_d, mhx = st.r * (s4[3] - st.m1 * s4[2]) * inv_d;
        if (ROWS == 1 || row < p.rows) {
            T* dx = static_cast<T*>(p.dx) + row * p.lddx;
            const float down = -st.r * mh, along = -st.r * mhx;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int k = kKeepWeight ? i : 0;
                if (!kKeepWeight) at.weight(weight, p.weight_fp32, i, w[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = fmaf(v[i][e], st.r, st.shift);
                    dw[i][e] = fmaf(h[i][e], xh, dw[i][e]);
                    db[i][e] += h[i][e];
                    v[i][e] = fmaf(xh, along, fmaf(h[i][e] * w[k][e], st.r, down));
                }
                at.store(dx, i, v[i], streamed);
            }
        }
        row += step;
    };
    // Two rows by name, as a copy of one that is on its way would wait for it.
    // Every row of a workgroup takes part in its barriers.
    Row even, odd;
    if (kAhead) fetch(row, even);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS; first < p.rows;) {
        turn(even, odd);
        first += step;
        if (first >= p.rows) break;
        turn(odd, even);
        first += step;
    }
    if constexpr (ROWS > 1) {  // the workgroup's rows, in their order
        __shared__ float sums[ROWS - 1][2][P * 8 * LANES];
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
                for (int r = 0; r < ROWS - 1; ++r) {
                    dw[i][e] += sums[r][0][(i * 8 + e) * LANES + t];
                    db[i][e] += sums[r][1][(i * 8 + e) * LANES + t];
                }
    }
    float* to = partial + static_cast<int64_t>(blockIdx.x) * 2 * p.d;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (TINY) {
            store8<QF32>(to, at.at[i], p.d, dw[i]);
            store8<QF32>(to + p.d, at.at[i], p.d, db[i]);
        } else if (at.skip[i] < 8) {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                store16_any(to + at.at[i] + e, u32x4{__float_as_uint(dw[i][e]), __float_as_uint(dw[i][e + 1]),
                                                     __float_as_uint(dw[i][e + 2]), __float_as_uint(dw[i][e + 3])});
                store16_any(to + p.d + at.at[i] + e, u32x4{__float_as_uint(db[i][e]), __float_as_uint(db[i][e + 1]),
                                                           __float_as_uint(db[i][e + 2]), __float_as_uint(db[i][e + 3])});
            }
        }
    }
}

// Long rows: their statistics, then the sums over rows, and dx last, which may
// overwrite dout.  Three readings: 512 x 70000 bf16 126 us, 2048 x 20000 138.
template <class E>
__global__ __launch_bounds__(kLongLanes) void layer_norm_back_long_stats_kernel(const LayerNormBackArgs p,
                                                                                float* __restrict__ stats) {
    using T = typename E::T;
    __shared__ float red[3][kLongWaves * 2];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* g = static_cast<const T*>(p.g) + row * p.ldg;
    float m0;
    const Stats st = long_stats<E>(x, p.d, p.eps, red, m0);
    const int t = threadIdx.x, wave = threadIdx.x / kWave, pieces = (p.d + kLongLanes * 8 - 1) / (kLongLanes * 8);
    const float inv_d = 1.0f / static_cast<float>(p.d);
    float s[2] = {0.0f, 0.0f};
    for (int i = 0; i < pieces; ++i) {
        float v[8], h[8], w[8];
        load8_any<E>(x, column<kLongLanes>(i, t), p.d, v);
        load8_any<E>(g, column<kLongLanes>(i, t), p.d, h);
        load_weight<E>(p.weight, p.weight_fp32, column<kLongLanes>(i, t), p.d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // past the row h is 0
            s[0] += h[e] * w[e];
            s[1] = fmaf(h[e] * w[e], fmaf(v[e] - m0, st.r, st.shift), s[1]);
        }
    }
    row_sums<kLongWaves, 2>(s, red[2], wave);
    if (t == 0) {
        float* to = stats + row * kLayerNormStats;
        to[0] = m0;
        to[1] = st.r;
        to[2] = st.shift;
        to[3] = s[0] * inv_d;
        to[4] = s[1] * inv_d;
    }
}

template <class E>
__global__ __launch_bounds__(kLongLanes) void layer_norm_back_long_kernel(const LayerNormBackArgs p,
                                                                          const float* __restrict__ stats) {
    using T = typename E::T;
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* g = static_cast<const T*>(p.g) + row * p.ldg;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    const float* of = stats + row * kLayerNormStats;
    const float m0 = of[0], r = of[1], shift = of[2], mh = of[3], mhx = of[4];
    const int t = threadIdx.x, pieces = (p.d + kLongLanes * 8 - 1) / (kLongLanes * 8);
    for (int i = 0; i < pieces; ++i) {
        float v[8], h[8], w[8];
        load8_any<E>(x, column<kLongLanes>(i, t), p.d, v);
        load8_any<E>(g, column<kLongLanes>(i, t), p.d, h);
        load_weight<E>(p.weight, p.weight_fp32, column<kLongLanes>(i, t), p.d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = r * (h[e] * w[e] - mh - fmaf(v[e] - m0, r, shift) * mhx);
        store8<E>(dx, column<kLongLanes>(i, t), p.d, v);
    }
}

// 8 columns a thread, rows groups apart.
template <class E>
__global__ __launch_bounds__(kThreads) void layer_norm_column_sums_kernel(const LayerNormBackArgs p,
                                                                          const float* __restrict__ stats,
                                                                          float* __restrict__ partial) {
    using T = typename E::T;
    static_assert(kLayerNormColumns == 8 * kThreads, "the groups count workgroups of so many columns");
    const int c = (blockIdx.x * kThreads + threadIdx.x) * 8;
    if (c >= p.d) return;
    float dw[8] = {}, db[8] = {};
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        float x[8], g[8];
        load8_any<E>(static_cast<const T*>(p.x) + row * p.ldx, c, p.d, x);
        load8_any<E>(static_cast<const T*>(p.g) + row * p.ldg, c, p.d, g);
        const float* of = stats + row * kLayerNormStats;
        const float m0 = of[0], r = of[1], shift = of[2];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[e] = fmaf(g[e], fmaf(x[e] - m0, r, shift), dw[e]);
            db[e] += g[e];
        }
    }
    float* to = partial + static_cast<int64_t>(blockIdx.y) * 2 * p.d;
    store8<QF32>(to, c, p.d, dw);
    store8<QF32>(to + p.d, c, p.d, db);
}

// Adds the partial rows: 32 columns a workgroup, each half wave a run of the
// rows, in a fixed order.
constexpr int kAddWaves = 16, kAddColumns = 32, kAddParts = 2 * kAddWaves;
__global__ __launch_bounds__(kAddWaves* kWave) void layer_norm_add_kernel(const float* __restrict__ partial, int groups, int d,
                                                                          float* __restrict__ dweight,
                                                                          float* __restrict__ dbias) {
    __shared__ float sums[kAddParts][kAddColumns];
    const int lane = threadIdx.x % kAddColumns, part = threadIdx.x / kAddColumns;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kAddColumns + lane, width = 2 * static_cast<int64_t>(d);
    const int per = (groups + kAddParts - 1) / kAddParts;
    float s = 0.0f;
    if (c < width) {
        const int end = min(groups, (part + 1) * per);
#pragma unroll 8
        for (int g = part * per; g < end; ++g) s += partial[g * width + c];
    }
    sums[part][lane] = s;
    __syncthreads();
    if (part == 0 && c < width) {
#pragma unroll
        for (int i = 1; i < kAddParts; ++i) s += sums[i][lane];
        if (c < d) dweight[c] = s;
        else dbias[c - d] = s;
    }
}

// Outputs of many rows do not stay in L2: 8192 x 4096 bf16 32.2 us, 31.1 so, 8192 x
// 1024 10.0 and 8.8.
bool streamed(int64_t rows) { return rows >= 4 * device_cu_count(); }

template <class E, int WAVES, int P, bool TINY = false>
int launch_forward(const LayerNormArgs& p, void* stream) {
    constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;
    hipLaunchKernelGGL((layer_norm_kernel<E, WAVES, P, TINY>), dim3(static_cast<unsigned>((p.rows + kRows - 1) / kRows)),
                       dim3((WAVES < 4 ? 4 : WAVES) * kWave), 0, static_cast<hipStream_t>(stream), p, streamed(p.rows));
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_forward_e(const LayerNormArgs& whole, void* stream) {
    using T = typename E::T;
    constexpr int64_t kMost = int64_t(1) << 21;  // rows a launch: its threads count in 32 bits
    for (int64_t r = 0; r < whole.rows; r += kMost) {
        LayerNormArgs p = whole;
        p.x = static_cast<const T*>(p.x) + r * p.ldx;
        p.out = static_cast<T*>(p.out) + r * p.ldo;
        p.rows = whole.rows - r < kMost ? whole.rows - r : kMost;
        int e;
        // As few waves a row as hold it in a few pieces a thread: 3001 x 777 fp16 4.9 us in
        // one wave of two pieces, 5.7 in one of four; 8192 x 1024 8.9 in one, 12.1 in four
        // waves; 8192 x 2048 16.6 in four, 17.5 in one; 8192 x 4096 30.0 in four, 30.5 in
        // eight; 2048 x 8192 19.4 in four, 19.9 in sixteen.  A width between the forms
        // pays for the pieces of the next one: 8192 x 4097 72 us, 8192 x 5120 56, 2048 x 8193
        // 25, 2048 x 12288 29; rows under 512 for a whole wave: 16384 x 64 6.4.
        if (p.d < 8) {
            e = launch_forward<E, 1, 1, true>(p, stream);
        } else if (p.d <= 512) {
            e = launch_forward<E, 1, 1>(p, stream);
        } else if (p.d <= 1024) {
            e = launch_forward<E, 1, 2>(p, stream);
        } else if (p.d <= 2048) {
            e = launch_forward<E, 4, 1>(p, stream);
        } else if (p.d <= 4096) {
            e = launch_forward<E, 4, 2>(p, stream);
        } else if (p.d <= 16384) {
            e = launch_forward<E, 4, 8>(p, stream);
        } else if (p.d <= 32768) {
            e = launch_forward<E, 16, 4>(p, stream);
        } else {
            hipLaunchKernelGGL((layer_norm_long_kernel<E>), dim3(static_cast<unsigned>(p.rows)), dim3(kLongLanes), 0,
                               static_cast<hipStream_t>(stream), p);
            e = static_cast<int>(hipGetLastError());
        }
        if (e != 0) return e;
    }
    return 0;
}

template <class E, int WAVES, int ROWS, int P, bool TINY = false>
int launch_back(const LayerNormBackArgs& p, int* groups, void* stream) {
    const int64_t g = (p.rows + ROWS - 1) / ROWS;
    *groups = static_cast<int>(g < kLayerNormPartials ? g : kLayerNormPartials);
    hipLaunchKernelGGL((layer_norm_back_kernel<E, WAVES, ROWS, P, TINY>), dim3(static_cast<unsigned>(*groups)),
                       dim3(WAVES * ROWS * kWave), 0, static_cast<hipStream_t>(stream), p, p.workspace, streamed(p.rows));
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_back_e(const LayerNormBackArgs& p, void* stream) {
    int groups = 0, e = 0;
    if (p.rows == 0) {
        // the sum of no rows: groups = 0 below
    // One piece a thread up to 8192: 8192 x 1024 bf16 22.7 us with two rows of four
    // waves, 34.5 with one row of eight; 8192 x 4096 45.7 with a row of eight waves, 48.4
    // with two of four and two pieces; 2048 x 8192 36.6 and 36.7.  Above, four pieces in
    // eight waves: two in sixteen do not fit the registers (2048 x 8193 63, 2048 x 12288 62,
    // 2048 x 16384 75).  Between the forms 8192 x 5120 takes 80.
    } else if (p.d < 8) {
        e = launch_back<E, 1, 4, 1, true>(p, &groups, stream);
    } else if (p.d <= 512) {
        e = launch_back<E, 1, 4, 1>(p, &groups, stream);
    } else if (p.d <= 2048) {
        e = launch_back<E, 4, 2, 1>(p, &groups, stream);
    } else if (p.d <= 4096) {
        e = launch_back<E, 8, 1, 1>(p, &groups, stream);
    } else if (p.d <= 8192) {
        e = launch_back<E, 16, 1, 1>(p, &groups, stream);
    } else if (p.d <= kLayerNormKept) {
        e = launch_back<E, 8, 1, 4>(p, &groups, stream);
    } else {
        groups = static_cast<int>(layer_norm_groups(p.rows, p.d));
        float* stats = p.workspace + static_cast<int64_t>(groups) * 2 * p.d;
        // all rows, kMost a launch, in one kernel or the other
        const auto rows = [&](auto kernel) {
            using T = typename E::T;
            constexpr int64_t kMost = int64_t(1) << 21;
            for (int64_t r = 0; r < p.rows && e == 0; r += kMost) {
                LayerNormBackArgs q = p;
                q.x = static_cast<const T*>(p.x) + r * p.ldx;
                q.g = static_cast<const T*>(p.g) + r * p.ldg;
                q.dx = static_cast<T*>(p.dx) + r * p.lddx;
                hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(p.rows - r < kMost ? p.rows - r : kMost)), dim3(kLongLanes),
                                   0, static_cast<hipStream_t>(stream), q, stats + r * kLayerNormStats);
                e = static_cast<int>(hipGetLastError());
            }
        };
        rows(layer_norm_back_long_stats_kernel<E>);
        if (e != 0) return e;
        hipLaunchKernelGGL((layer_norm_column_sums_kernel<E>), dim3((p.d + kLayerNormColumns - 1) / kLayerNormColumns, groups), dim3(kThreads),
                           0, static_cast<hipStream_t>(stream), p, stats, p.workspace);
        e = static_cast<int>(hipGetLastError());
        rows(layer_norm_back_long_kernel<E>);
    }
    if (e != 0) return e;
    hipLaunchKernelGGL(layer_norm_add_kernel,
                       dim3(static_cast<unsigned>((2 * static_cast<int64_t>(p.d) + kAddColumns - 1) / kAddColumns)),
                       dim3(kAddWaves * kWave), 0, static_cast<hipStream_t>(stream), p.workspace, groups, p.d, p.dweight,
                       p.dbias);
    return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_layer_norm(Dtype t, const LayerNormArgs& p, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_forward_e<QF32>(p, stream);
        case Dtype::fp16: return launch_forward_e<QF16>(p, stream);
        default: return launch_forward_e<QB16>(p, stream);
    }
}

int launch_layer_norm_back(Dtype t, const LayerNormBackArgs& p, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_back_e<QF32>(p, stream);
        case Dtype::fp16: return launch_back_e<QF16>(p, stream);
        default: return launch_back_e<QB16>(p, stream);
    }
}

}  // namespace kbit
