// Passes over the heads of queries, keys and values: rotary positions, the
// RMS norm of every head with the rotation in the same pass, its gradient,
// and the append to a paged cache with the rotation on the way.
//
// Mathematics, per row (one head of one token, D elements, the first `rot`
// of them rotated):
//   norm      x <- x / sqrt(mean(x^2) + eps) * w
//   rotation  (a, b) -> (a c - b s, b c + a s) for every pair; c and s are
//             the token's row of the table (amplitude times cosine and sine
//             of position times frequency, fp64 rounded once to fp32).  The
//             pairs are (i, i + rot / 2) in the half layout and (2i, 2i + 1)
//             in the interleaved one; elements from `rot` on pass through.
//   gradient  of the norm with rotation: u = R^T g (the rotation with s
//             negated), xhat = x / sqrt(mean(x^2) + eps) =: x r,
//             dw = sum over tokens and heads of u xhat,
//             dx = r (u w - xhat mean(u w xhat)).
// All of it in fp32 without contraction, rounded once to the element type.
//
// Layout: a group of GP lanes (a power of two) holds one row, each lane two
// 16-byte (32-byte for fp32) pieces chosen so that both elements of every
// pair are in the same lane: pieces j and j + rot/16 in the half layout, j
// and j + half of the pieces in the interleaved one.  So a row is read once, the sum of
// squares needs log2(GP) exchanges, and writing in place is safe.  A lane
// group takes R heads of one token, so that the token's cosines and sines
// are fetched once for R rows and all R rows' loads are in flight together.
// Rows whose sizes or addresses do not allow 16-byte pieces go element by
// element, one wave a row, with the same arithmetic.
//
// All passes read and write each element once and are bound by memory from
// some thousand tokens on (a large copy on this card runs at 5.8 TB/s), by the
// launch below that.  Heads of 128 in 16 bits: rotation of 8193 x 32 24.1 us
// (5.6 TB/s), norm of 8191 x 40 32.4 (5.3), append of 8179 x 8 14.0 (5.1),
// gradient of 8192 x 40 52.1 with the addition of the weights' partial sums
// (4.9).
#include "device.h"
#include "kbit_internal.h"
#include "launch.h"
#include "layer_internal.h"

namespace kbit {
namespace {

// Workgroups of a pass over heads at most; beyond it a group takes several units.
constexpr unsigned kMaxHeadsGrid = 1u << 22;

constexpr int kHalf = 0, kInterleaved = 1;

// Element types: 8 consecutive elements as raw vectors, widened exactly.
struct HF32 {
    using T = float;
    static constexpr int kVec = 2;
    static __device__ float one(T v) { return v; }
    static __device__ T narrow(float v) { return v; }
    static __device__ void widen(const u32x4* r, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(r[0][i]);
            x[4 + i] = __uint_as_float(r[1][i]);
        }
    }
    static __device__ void store8(T* p, const float (&v)[8]) {
        store16<true>(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                __float_as_uint(v[3])});
        store16<true>(p + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                    __float_as_uint(v[7])});
    }
};

struct HF16 {
    using T = uint16_t;
    static constexpr int kVec = 1;
    static __device__ float one(T v) { return Fp16::h2f(v); }
    static __device__ T narrow(float v) { return static_cast<T>(pack_f16x2(v, 0.0f) & 0xFFFFu); }
    static __device__ void widen(const u32x4* r, float (&x)[8]) { Fp16::unpack(r, x); }
    static __device__ void store8(T* p, const float (&v)[8]) {
        store16<true>(p, u32x4{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                                pack_f16x2(v[6], v[7])});
    }
};

struct HB16 {
    using T = uint16_t;
    static constexpr int kVec = 1;
    static __device__ float one(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
    static __device__ T narrow(float v) { return static_cast<T>(pack_bf16x2(v, 0.0f) & 0xFFFFu); }
    static __device__ void widen(const u32x4* r, float (&x)[8]) { Bf16::unpack(r, x); }
    static __device__ void store8(T* p, const float (&v)[8]) {
        store16<true>(p, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                pack_bf16x2(v[6], v[7])});
    }
};

// Which 16 elements of its row a lane holds.  Vector form: piece A is the 8
// elements from `a`, piece B the 8 from `b` (negative: none).  Element form
// (one wave a row): pair i of the lane is pair slot lane + 64 i.
struct Slots {
    int a, b;    // vector form: first elements, or -1
    int pa, pb;  // vector form: table columns of the lane's first and second 4 pairs
    bool ra, rb; // vector form: piece A (and in the half layout B with it) / piece B rotated
};

template <int LAYOUT>
__device__ __forceinline__ Slots vector_slots(int j, int D, int rot) {
    // Neighbouring lanes hold neighbouring pieces, so that a load or store of
    // a wave covers whole lines.
    Slots s;
    if constexpr (LAYOUT == kHalf) {
        const int half = rot >> 1;
        s.ra = s.rb = 8 * j < half;
        s.pa = 8 * j;
        s.pb = 8 * j + 4;
        if (s.ra) {
            s.a = 8 * j;
            s.b = half + 8 * j;
        } else {  // the elements that pass through, in two runs of pieces
            const int u = j - (half >> 3), pieces = (D - rot) >> 3, run = (pieces + 1) >> 1;
            s.a = u < run ? rot + 8 * u : -1;
            s.b = u < run && u + run < pieces ? rot + 8 * (u + run) : -1;
        }
    } else {
        const int pieces = D >> 3, run = (pieces + 1) >> 1;
        s.a = j < run ? 8 * j : -1;
        s.b = j < run && j + run < pieces ? 8 * (j + run) : -1;
        s.ra = s.a >= 0 && s.a < rot;
        s.rb = s.b >= 0 && s.b < rot;
        s.pa = s.a >> 1;
        s.pb = s.b >> 1;
    }
    return s;
}

// Element form: elements (ea, eb) of pair slot p (negative: none) and
// whether they are rotated.
template <int LAYOUT>
__device__ __forceinline__ void element_pair(int p, int D, int rot, int& ea, int& eb, bool& turned) {
    if constexpr (LAYOUT == kHalf) {
        const int half = rot >> 1;
        turned = p < half;
        ea = turned ? p : rot + 2 * (p - half);
        eb = turned ? p + half : ea + 1;
    } else {
        ea = 2 * p;
        eb = ea + 1;
        turned = ea < rot;
    }
    if (ea >= D) ea = -1;
    if (eb >= D) eb = -1;
}

// How a lane holds its elements: the vector form (kVector), 8 + 8 in two
// pieces, or the element form with 1 or 8 pairs a lane, as the row needs.
constexpr int kVector = 0;
constexpr int count_of(int form) { return form == kVector ? 8 : form; }

// A lane's raw elements before widening.
template <class E, int FORM>
struct Raw {
    u32x4 v[FORM == kVector ? 2 * E::kVec : 1];
    typename E::T s[FORM == kVector ? 1 : 2 * FORM];
};

template <class E, int LAYOUT, int FORM>
__device__ __forceinline__ void load_row(const typename E::T* p, int lane, int D, int rot, const Slots& sl,
                                         Raw<E, FORM>& r) {
    if constexpr (FORM == kVector) {
        constexpr int V = E::kVec;
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) r.v[i] = u32x4{0u, 0u, 0u, 0u};
        if (sl.a >= 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) r.v[i] = load16<false>(p + sl.a + 4 * i);
        }
        if (sl.b >= 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) r.v[V + i] = load16<false>(p + sl.b + 4 * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < FORM; ++i) {
            int ea, eb;
            bool turned;
            element_pair<LAYOUT>(lane + kWave * i, D, rot, ea, eb, turned);
            r.s[i] = ea >= 0 ? p[ea] : typename E::T(0);
            r.s[FORM + i] = eb >= 0 ? p[eb] : typename E::T(0);
        }
    }
}

template <class E, int FORM>
__device__ __forceinline__ void widen_row(const Raw<E, FORM>& r, float (&a)[count_of(FORM)],
                                          float (&b)[count_of(FORM)]) {
    if constexpr (FORM == kVector) {
        E::widen(r.v, a);
        E::widen(r.v + E::kVec, b);
    } else {
#pragma unroll
        for (int i = 0; i < FORM; ++i) {
            a[i] = E::one(r.s[i]);
            b[i] = E::one(r.s[FORM + i]);
        }
    }
}

template <class E, int LAYOUT, int FORM>
__device__ __forceinline__ void store_row(typename E::T* p, int lane, int D, int rot, const Slots& sl,
                                          const float (&a)[count_of(FORM)], const float (&b)[count_of(FORM)]) {
    if constexpr (FORM == kVector) {
        if (sl.a >= 0) E::store8(p + sl.a, a);
        if (sl.b >= 0) E::store8(p + sl.b, b);
    } else {
#pragma unroll
        for (int i = 0; i < FORM; ++i) {
            int ea, eb;
            bool turned;
            element_pair<LAYOUT>(lane + kWave * i, D, rot, ea, eb, turned);
            if (ea >= 0) p[ea] = E::narrow(a[i]);
            if (eb >= 0) p[eb] = E::narrow(b[i]);
        }
    }
}

// The lane's 8 cosines and sines (1 and 0 where nothing is rotated, so that
// the rotation leaves those elements as they are: x * 1 - y * 0 is x for
// finite y only, hence turn() skips them instead).
template <int FORM>
struct Angles {
    float c[count_of(FORM)], s[count_of(FORM)];
};

template <int LAYOUT, int FORM>
__device__ __forceinline__ void load_angles(const float* table, int64_t pos, int64_t max_pos, int lane, int D, int rot,
                                            const Slots& sl, float sign, Angles<FORM>& g) {
    // A position outside the table poisons the rotated elements.
    const bool ok = pos >= 0 && pos < max_pos;
    const float* row = table + (ok ? pos : 0) * rot;
    const float bad = __uint_as_float(0x7FC00000u);
    if constexpr (FORM == kVector) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool live = LAYOUT == kHalf ? sl.ra : (h == 0 ? sl.ra : sl.rb);
            u32x4 c = u32x4{0u, 0u, 0u, 0u}, s = c;
            if (live) {
                const int at = h == 0 ? sl.pa : sl.pb;
                c = load16<false>(row + at);
                s = load16<false>(row + (rot >> 1) + at);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g.c[4 * h + i] = ok ? __uint_as_float(c[i]) : bad;
                g.s[4 * h + i] = ok ? sign * __uint_as_float(s[i]) : bad;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < FORM; ++i) {
            const int p = lane + kWave * i;
            const bool live = p < (rot >> 1);
            g.c[i] = ok ? (live ? row[p] : 1.0f) : bad;
            g.s[i] = ok ? (live ? sign * row[(rot >> 1) + p] : 0.0f) : bad;
        }
    }
}

__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s, bool on) {
    const float nx = x * c - y * s, ny = y * c + x * s;
    x = on ? nx : x;
    y = on ? ny : y;
}

template <int LAYOUT, int FORM>
__device__ __forceinline__ void turn(float (&a)[count_of(FORM)], float (&b)[count_of(FORM)], const Angles<FORM>& g, int lane, int D, int rot,
                                     const Slots& sl) {
    if constexpr (FORM != kVector) {
#pragma unroll
        for (int i = 0; i < FORM; ++i) turn_pair(a[i], b[i], g.c[i], g.s[i], lane + kWave * i < (rot >> 1));
    } else if constexpr (LAYOUT == kHalf) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], g.c[i], g.s[i], sl.ra);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn_pair(a[2 * i], a[2 * i + 1], g.c[i], g.s[i], sl.ra);
            turn_pair(b[2 * i], b[2 * i + 1], g.c[4 + i], g.s[4 + i], sl.rb);
        }
    }
}

// Sum over the lane group (lanes = 1 .. 64, uniform over the grid).
__device__ __forceinline__ float group_sum(float v, int lanes) {
    if (lanes >= 2) v += dpp_f32<kDppXor1>(v);
    if (lanes >= 4) v += dpp_f32<kDppXor2>(v);
    if (lanes >= 8) v += dpp_f32<kDppHalfMirror>(v);
    if (lanes >= 16) v += dpp_f32<kDppMirror>(v);
    if (lanes >= 32) v += shfl_xor_f32(v, 16);
    if (lanes >= 64) v += shfl_xor_f32(v, 32);
    return v;
}

__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, bool wide) {
    return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

template <class E, int LAYOUT, int FORM>
__device__ __forceinline__ void load_weight(const void* w, bool w_fp32, int lane, int D, int rot, const Slots& sl,
                                            float (&a)[count_of(FORM)], float (&b)[count_of(FORM)]) {
    if (w_fp32) {
        Raw<HF32, FORM> r;
        load_row<HF32, LAYOUT, FORM>(static_cast<const float*>(w), lane, D, rot, sl, r);
        widen_row<HF32, FORM>(r, a, b);
    } else {
        Raw<E, FORM> r;
        load_row<E, LAYOUT, FORM>(static_cast<const typename E::T*>(w), lane, D, rot, sl, r);
        widen_row<E, FORM>(r, a, b);
    }
}

// One pass over up to two sets of heads (queries and keys, or keys and
// values).  NORM: norm before the rotation.  PAGED: the output row is found
// through the token's slot; set 1 is copied.
template <class E, int LAYOUT, bool NORM, bool PAGED, int FORM, int R>
__global__ __launch_bounds__(kThreads) void heads_kernel(const HeadsArgs p) {
    using T = typename E::T;
    const int lg = FORM == kVector ? p.log2_lanes : 6;
    const int lane = threadIdx.x & ((1 << lg) - 1);
    const uint32_t step = gridDim.x * (kThreads >> lg);
    const uint32_t per_token = p.set[0].units + p.set[1].units;
    const int64_t b = blockIdx.y;
    for (uint32_t unit = blockIdx.x * (kThreads >> lg) + (threadIdx.x >> lg); unit < p.units; unit += step) {
        // Neighbouring lane groups take neighbouring rows in memory: heads of
        // a token, or tokens of a head where those are closer.
        const uint32_t tokens = static_cast<uint32_t>(p.tokens);
        const uint32_t major = unit / (p.tokens_first ? tokens : per_token);
        const uint32_t minor = unit - major * (p.tokens_first ? tokens : per_token);
        const uint32_t t = p.tokens_first ? minor : major;
        uint32_t u = p.tokens_first ? major : minor;
        const bool second = u >= static_cast<uint32_t>(p.set[0].units);
        const HeadSet& set = p.set[second ? 1 : 0];
        if (second) u -= p.set[0].units;
        // Heads u, u + units, ...: a load of the wave covers neighbouring rows.
        const int h0 = static_cast<int>(u), dh = set.units;
        const int D = set.dim, rot = set.rot;
        const Slots sl = vector_slots<LAYOUT>(lane, D, rot);

        int64_t at = 0;
        if constexpr (PAGED) {
            const int64_t slot = load_index(p.slots, t, p.slots_wide);
            if (slot < 0 || slot >= p.n_slots) continue;  // padding, or outside the cache: nothing is written
            const uint32_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size);
            const uint32_t off = static_cast<uint32_t>(slot) - page * p.page_size;
            at = page * set.out_b + off * set.out_s;
        } else {
            at = b * set.out_b + t * set.out_s;
        }
        T* out = static_cast<T*>(set.out) + at;
        const T* in = static_cast<const T*>(set.in) + b * set.in_b + t * set.in_s;
        Raw<E, FORM> raw[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (h0 + r * dh < set.heads)
                load_row<E, LAYOUT, FORM>(in + (h0 + r * dh) * set.in_h, lane, D, rot, sl, raw[r]);
        Angles<FORM> g;
        if (rot > 0) {
            const int64_t pos = load_index(p.positions, b * p.tokens + t, p.positions_wide);
            load_angles<LAYOUT, FORM>(p.table, pos, p.max_pos, lane, D, rot, sl, p.sign, g);
        }
        float wa[count_of(FORM)], wb[count_of(FORM)];
        if constexpr (NORM) load_weight<E, LAYOUT, FORM>(set.weight, p.weight_fp32, lane, D, rot, sl, wa, wb);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (h0 + r * dh >= set.heads) break;
            float xa[count_of(FORM)], xb[count_of(FORM)];
            widen_row<E, FORM>(raw[r], xa, xb);
            if constexpr (NORM) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < count_of(FORM); ++i) ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
                ss = group_sum(ss, 1 << lg);
                const float rs = rsqrtf(ss * p.inv_dim + p.eps);
#pragma unroll
                for (int i = 0; i < count_of(FORM); ++i) {
                    xa[i] = xa[i] * rs * wa[i];
                    xb[i] = xb[i] * rs * wb[i];
                }
            }
            if (rot > 0) turn<LAYOUT, FORM>(xa, xb, g, lane, D, rot, sl);
            store_row<E, LAYOUT, FORM>(out + (h0 + r * dh) * set.out_h, lane, D, rot, sl, xa, xb);
        }
    }
}

// Gradient of the norm with rotation.  Workgroups below `first_groups` work
// through the rows of set 0, the others through set 1's; each keeps its sum
// of u * xhat in registers, adds its lane groups in LDS in a fixed order and
// stores one partial row of D sums, which norm_weight_grad_kernel adds in a
// fixed order: the result does not depend on scheduling.
template <class E, int LAYOUT, int FORM, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_back_kernel(const NormBackArgs p) {
    using T = typename E::T;
    __shared__ __align__(16) float red[THREADS * 16];
    const int lg = FORM == kVector ? p.log2_lanes : 6;
    const int groups = THREADS >> lg;
    const int lane = threadIdx.x & ((1 << lg) - 1);
    const int group = threadIdx.x >> lg;
    const bool second = blockIdx.x >= static_cast<unsigned>(p.first_groups);
    const BackSet& set = p.set[second ? 1 : 0];
    const int block = blockIdx.x - (second ? p.first_groups : 0);
    const int blocks = second ? gridDim.x - p.first_groups : p.first_groups;
    const int D = p.dim, rot = p.rot;
    const Slots sl = vector_slots<LAYOUT>(lane, D, rot);
    float wa[count_of(FORM)], wb[count_of(FORM)], da[count_of(FORM)], db[count_of(FORM)];
    load_weight<E, LAYOUT, FORM>(set.weight, p.weight_fp32, lane, D, rot, sl, wa, wb);
#pragma unroll
    for (int i = 0; i < count_of(FORM); ++i) da[i] = db[i] = 0.0f;

    const uint32_t rows = set.rows;
    for (uint32_t row = block * groups + group; row < rows; row += blocks * groups) {
        const uint32_t bt = row / static_cast<uint32_t>(set.heads);
        const uint32_t h = row - bt * set.heads;
        const uint32_t b = bt / static_cast<uint32_t>(p.tokens);
        const uint32_t t = bt - b * p.tokens;
        const T* x = static_cast<const T*>(set.x) + b * set.x_b + t * set.x_s + h * set.x_h;
        const T* gr = static_cast<const T*>(set.g) + b * set.g_b + t * set.g_s + h * set.g_h;
        T* dx = static_cast<T*>(set.dx) + b * set.dx_b + t * set.dx_s + h * set.dx_h;
        Raw<E, FORM> rx, rg;
        load_row<E, LAYOUT, FORM>(x, lane, D, rot, sl, rx);
        load_row<E, LAYOUT, FORM>(gr, lane, D, rot, sl, rg);
        Angles<FORM> g;
        const int64_t pos = load_index(p.positions, bt, p.positions_wide);
        load_angles<LAYOUT, FORM>(p.table, pos, p.max_pos, lane, D, rot, sl, -1.0f, g);
        float xa[count_of(FORM)], xb[count_of(FORM)], ga[count_of(FORM)], gb[count_of(FORM)];
        widen_row<E, FORM>(rx, xa, xb);
        widen_row<E, FORM>(rg, ga, gb);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < count_of(FORM); ++i) ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
        ss = group_sum(ss, 1 << lg);
        const float rs = rsqrtf(ss * p.inv_dim + p.eps);
        turn<LAYOUT, FORM>(ga, gb, g, lane, D, rot, sl);
        float inner = 0.0f;
#pragma unroll
        for (int i = 0; i < count_of(FORM); ++i) {
            xa[i] *= rs;
            xb[i] *= rs;
            da[i] = fmaf(ga[i], xa[i], da[i]);
            db[i] = fmaf(gb[i], xb[i], db[i]);
            ga[i] *= wa[i];
            gb[i] *= wb[i];
            inner = fmaf(ga[i], xa[i], fmaf(gb[i], xb[i], inner));
        }
        inner = group_sum(inner, 1 << lg) * p.inv_dim;
#pragma unroll
        for (int i = 0; i < count_of(FORM); ++i) {
            xa[i] = rs * (ga[i] - xa[i] * inner);
            xb[i] = rs * (gb[i] - xb[i] * inner);
        }
        store_row<E, LAYOUT, FORM>(dx, lane, D, rot, sl, xa, xb);
    }
    float* mine = red + group * D;  // groups * D <= THREADS * 16
    if constexpr (FORM == kVector) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {  // D is a multiple of 8: 16-byte pieces
            if (sl.a >= 0) *reinterpret_cast<float4*>(mine + sl.a + i) = make_float4(da[i], da[i + 1], da[i + 2], da[i + 3]);
            if (sl.b >= 0) *reinterpret_cast<float4*>(mine + sl.b + i) = make_float4(db[i], db[i + 1], db[i + 2], db[i + 3]);
        }
    } else {
        store_row<HF32, LAYOUT, FORM>(mine, lane, D, rot, sl, da, db);
    }
    __syncthreads();
    if constexpr (THREADS == kThreads) {
        for (int e = threadIdx.x; e < D; e += THREADS) {
            float sum = red[e];
            for (int q = 1; q < groups; ++q) sum += red[q * D + e];
            p.partial[static_cast<int64_t>(blockIdx.x) * D + e] = sum;
        }
    } else {  // up to 1024 lane groups, and nobody else at work: halves added to halves
        for (int s = groups >> 1; s >= 1; s >>= 1) {
            for (int i = threadIdx.x; i < s * D; i += THREADS) red[i] += red[i + s * D];
            __syncthreads();
        }
        for (int e = threadIdx.x; e < D; e += THREADS) p.direct[second ? 1 : 0][e] = red[e];
    }
}

// Adds the partial rows: 16 columns a workgroup, 64 row strides, then a tree.
constexpr int kGradCols = 16, kGradSplits = 64;
__global__ __launch_bounds__(kGradCols* kGradSplits) void norm_weight_grad_kernel(const float* __restrict__ partial,
                                                                                 int D, int first, int total,
                                                                                 float* __restrict__ d0,
                                                                                 float* __restrict__ d1) {
    __shared__ float red[kGradSplits][kGradCols + 1];
    const int c = threadIdx.x % kGradCols, r = threadIdx.x / kGradCols;
    const int e = blockIdx.x * kGradCols + c;
    const int lo = blockIdx.y == 0 ? 0 : first, hi = blockIdx.y == 0 ? first : total;
    float sum = 0.0f;
    if (e < D)
        for (int i = lo + r; i < hi; i += 8 * kGradSplits) {  // eight loads on their way at a time
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = i + j * kGradSplits;
                v[j] = row < hi ? partial[static_cast<int64_t>(row) * D + e] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[j];
        }
    red[r][c] = sum;
    __syncthreads();
    for (int s = kGradSplits / 2; s > 0; s >>= 1) {
        if (r < s) red[r][c] += red[r + s][c];
        __syncthreads();
    }
    if (r == 0 && e < D) (blockIdx.y == 0 ? d0 : d1)[e] = red[0][c];
}

// table[p][i] = RN32(amplitude cos(p f_i)), table[p][rot/2 + i] the sine.
__global__ __launch_bounds__(kThreads) void rope_table_kernel(const double* __restrict__ freq, int half,
                                                              int64_t max_pos, double amplitude,
                                                              float* __restrict__ table) {
    const int64_t n = max_pos * half;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; k < n;
         k += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t pos = k / half;
        const int i = static_cast<int>(k - pos * half);
        double s, c;
        sincos(static_cast<double>(pos) * freq[i], &s, &c);
        table[pos * 2 * half + i] = static_cast<float>(amplitude * c);
        table[pos * 2 * half + half + i] = static_cast<float>(amplitude * s);
    }
}

template <class E, int LAYOUT, bool NORM, bool PAGED, int FORM, int R>
int launch_heads_r(HeadsArgs& p, int64_t batch, void* stream) {
    for (auto& s : p.set) s.units = (s.heads + R - 1) / R;
    p.tokens_first = p.set[0].in_s < p.set[0].in_h;
    const int lg = FORM == kVector ? p.log2_lanes : 6;
    p.units = static_cast<uint32_t>(p.tokens * (p.set[0].units + p.set[1].units));
    unsigned grid = (p.units + (kThreads >> lg) - 1) / (kThreads >> lg);
    if (grid > kMaxHeadsGrid) grid = kMaxHeadsGrid;  // a launch holds fewer than 2^32 threads
    hipLaunchKernelGGL((heads_kernel<E, LAYOUT, NORM, PAGED, FORM, R>), dim3(grid, static_cast<unsigned>(batch)),
                       dim3(kThreads), 0, static_cast<hipStream_t>(stream), p);
    return static_cast<int>(hipGetLastError());
}

// Several heads a lane group once the groups fill the device all the same
// (4 workgroups a compute unit), else one.  8192 tokens, heads of 128 in 16
// bits, R = 1 / 2 / 4 / 8: rotation of 32 heads 26.6 / 24.7 / 25.8 / 29.7 us,
// norm of 40 heads 47.8 / 38.0 / 34.9 / 36.2, append of 8 heads 14.1 / 14.3 /
// 12.9 / 12.7.
template <class E, int LAYOUT, bool NORM, bool PAGED, int FORM>
int launch_heads_f(HeadsArgs& p, int64_t batch, void* stream) {
    constexpr int R = NORM || PAGED || FORM == 1 ? 4 : 2;
    const int lg = FORM == kVector ? p.log2_lanes : 6;
    const int64_t units = p.tokens * ((p.set[0].heads + R - 1) / R + (p.set[1].heads + R - 1) / R) * batch;
    if ((units << lg) >= static_cast<int64_t>(device_cu_count()) * 4 * kThreads)
        return launch_heads_r<E, LAYOUT, NORM, PAGED, FORM, R>(p, batch, stream);
    return launch_heads_r<E, LAYOUT, NORM, PAGED, FORM, 1>(p, batch, stream);
}

// Pairs a lane in the element form: one a lane covers heads of 128.  Rotation
// of 40 of 72 elements, 8192 tokens x 32 heads: 176 us with room for 8 pairs a
// lane, 40 with one.
bool one_pair_a_lane(int dim0, int dim1) { return dim0 <= 2 * kWave && dim1 <= 2 * kWave; }

template <class E, int LAYOUT, bool NORM, bool PAGED>
int launch_heads_l(HeadsArgs& p, int64_t batch, bool vec, void* stream) {
    if (vec) return launch_heads_f<E, LAYOUT, NORM, PAGED, kVector>(p, batch, stream);
    if (one_pair_a_lane(p.set[0].dim, p.set[1].dim)) return launch_heads_f<E, LAYOUT, NORM, PAGED, 1>(p, batch, stream);
    return launch_heads_r<E, LAYOUT, NORM, PAGED, 8, 1>(p, batch, stream);
}

template <class E>
int launch_heads_e(HeadsArgs& p, int64_t batch, HeadsKind kind, int layout, bool vec, void* stream) {
    if (layout == kHalf) {
        switch (kind) {
            case HeadsKind::rope: return launch_heads_l<E, kHalf, false, false>(p, batch, vec, stream);
            case HeadsKind::norm: return launch_heads_l<E, kHalf, true, false>(p, batch, vec, stream);
            default: return launch_heads_l<E, kHalf, false, true>(p, batch, vec, stream);
        }
    }
    switch (kind) {
        case HeadsKind::rope: return launch_heads_l<E, kInterleaved, false, false>(p, batch, vec, stream);
        case HeadsKind::norm: return launch_heads_l<E, kInterleaved, true, false>(p, batch, vec, stream);
        default: return launch_heads_l<E, kInterleaved, false, true>(p, batch, vec, stream);
    }
}

// Threads of a workgroup that makes a whole weight gradient: as many as its
// registers allow.
constexpr int direct_threads(int form) { return form <= 1 ? 1024 : 512; }

template <class E, int LAYOUT, int FORM>
int launch_back_f(const NormBackArgs& p, int grid, void* stream) {
    if (p.direct[0] != nullptr)
        hipLaunchKernelGGL((norm_back_kernel<E, LAYOUT, FORM, direct_threads(FORM)>), dim3(grid),
                           dim3(direct_threads(FORM)), 0, static_cast<hipStream_t>(stream), p);
    else
        hipLaunchKernelGGL((norm_back_kernel<E, LAYOUT, FORM, kThreads>), dim3(grid), dim3(kThreads), 0,
                           static_cast<hipStream_t>(stream), p);
    return static_cast<int>(hipGetLastError());
}

template <class E, int LAYOUT>
int launch_back_l(const NormBackArgs& p, bool vec, int grid, void* stream) {
    if (vec) return launch_back_f<E, LAYOUT, kVector>(p, grid, stream);
    if (one_pair_a_lane(p.dim, p.dim)) return launch_back_f<E, LAYOUT, 1>(p, grid, stream);
    return launch_back_f<E, LAYOUT, 8>(p, grid, stream);
}

template <class E>
int launch_back_e(const NormBackArgs& p, int layout, bool vec, int grid, void* stream) {
    return layout == kHalf ? launch_back_l<E, kHalf>(p, vec, grid, stream)
                           : launch_back_l<E, kInterleaved>(p, vec, grid, stream);
}

}  // namespace

int launch_heads(Dtype t, HeadsArgs& p, int64_t batch, HeadsKind kind, int layout, bool vec, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_heads_e<HF32>(p, batch, kind, layout, vec, stream);
        case Dtype::fp16: return launch_heads_e<HF16>(p, batch, kind, layout, vec, stream);
        default: return launch_heads_e<HB16>(p, batch, kind, layout, vec, stream);
    }
}

int launch_norm_back(Dtype t, NormBackArgs& p, int layout, bool vec, float* d0, float* d1, void* stream) {
    const int groups = kThreads >> (vec ? p.log2_lanes : 6);
    // Workgroups in the proportion of the two sets' rows, at least one each
    // (a set without rows has its weight gradient written as zeros).
    int64_t n[2];
    for (int i = 0; i < 2; ++i) n[i] = (static_cast<int64_t>(p.set[i].rows) + groups - 1) / groups;
    int64_t g0 = n[0], g1 = n[1];
    if (n[0] + n[1] > kNormBackGroups) {
        g0 = n[0] * kNormBackGroups / (n[0] + n[1]);
        g1 = kNormBackGroups - g0;
    }
    if (g0 < 1) g0 = 1;
    if (g1 < 1) g1 = 1;
    // Up to a row a lane group in one large workgroup a set: its sums are the
    // result, and there is no second launch.  Heads of 128 in 16 bits, in a
    // graph (and called from Python): 16 tokens x 8 heads, a row a lane group,
    // 6.3 us (6.7) against 6.3 (7.9) in two launches; 32 tokens, two rows, 8.7
    // (9.0) against 6.4 (7.9); 1 token 5.3 (5.8) against 6.3 (8.0).
    const int direct_groups =
        direct_threads(vec ? kVector : one_pair_a_lane(p.dim, p.dim) ? 1 : 8) >> (vec ? p.log2_lanes : 6);
    const bool direct = p.set[0].rows <= static_cast<uint32_t>(direct_groups) &&
                        p.set[1].rows <= static_cast<uint32_t>(direct_groups);
    if (direct) {
        g0 = g1 = 1;
        p.direct[0] = d0;
        p.direct[1] = d1;
    }
    p.first_groups = static_cast<int>(g0);
    const int grid = static_cast<int>(g0 + g1);
    int e;
    switch (t) {
        case Dtype::fp32: e = launch_back_e<HF32>(p, layout, vec, grid, stream); break;
        case Dtype::fp16: e = launch_back_e<HF16>(p, layout, vec, grid, stream); break;
        default: e = launch_back_e<HB16>(p, layout, vec, grid, stream); break;
    }
    if (e != 0 || direct) return e;
    hipLaunchKernelGGL(norm_weight_grad_kernel, dim3((p.dim + kGradCols - 1) / kGradCols, 2),
                       dim3(kGradCols * kGradSplits), 0, static_cast<hipStream_t>(stream), p.partial, p.dim,
                       p.first_groups, grid, d0, d1);
    return static_cast<int>(hipGetLastError());
}

int launch_rope_table(const double* freq, int rot, int64_t max_pos, double amplitude, float* table, void* stream) {
    const int64_t n = max_pos * (rot / 2);
    int64_t grid = (n + kThreads - 1) / kThreads;
    if (grid > 65536) grid = 65536;
    hipLaunchKernelGGL(rope_table_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), freq, rot / 2, max_pos, amplitude, table);
    return static_cast<int>(hipGetLastError());
}

}  // namespace kbit
