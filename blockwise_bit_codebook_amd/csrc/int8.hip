// 8-bit integer linear layer for gfx950: rows to int8 codes with one scale
// each, and the product of two coded matrices with the scales in its
// epilogue.
//
//   codes    amax = max |x| over the row, scale = RN(amax / 127),
//            q = rint(RN(x * RN(127 * RN(1 / amax)))), half to even; |q| <= 127
//            (two roundings of the step, as in a division through the
//            reciprocal; RN(127 / amax) differs for 24% of the bf16 amax).
//            A row below 2^-100 throughout (1 / amax could leave the fp32
//            range) gets scale 0 and codes 0; a row with a NaN or an
//            infinity gets scale NaN and codes 0, so that its outputs are NaN.
//   product  acc[m][n] = sum over k of x[m][k] * w[n][k], exact in int32,
//            out = RN_T(RN(RN(RN(acc) * xs[m]) * ws[n]) + bias[n]).
#include "device.h"
#include "int8_choice.h"
#include "kbit_internal.h"
#include "launch.h"
#include "layer_internal.h"

#include <type_traits>

namespace kbit {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------
struct QF32 {
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
};
struct QF16 {
    using T = uint16_t;
    static constexpr int kVec = 1;
    static __device__ float one(T v) { return Fp16::h2f(v); }
    static __device__ T narrow(float v) { return static_cast<T>(pack_f16x2(v, 0.0f) & 0xFFFFu); }
    static __device__ uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
    static __device__ void widen(const u32x4* r, float (&x)[8]) { Fp16::unpack(r, x); }
};
struct QB16 {
    using T = uint16_t;
    static constexpr int kVec = 1;
    static __device__ float one(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
    static __device__ T narrow(float v) { return static_cast<T>(pack_bf16x2(v, 0.0f) & 0xFFFFu); }
    static __device__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
    static __device__ void widen(const u32x4* r, float (&x)[8]) { Bf16::unpack(r, x); }
};

// ---------------------------------------------------------------------------
// rows to codes
// ---------------------------------------------------------------------------
// 8 elements of a row from column c, 0 beyond d.
template <class E, bool VEC>
__device__ __forceinline__ void load8(const typename E::T* row, int c, int d, float (&x)[8]) {
    if (VEC && c + 8 <= d) {
        u32x4 r[E::kVec];
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) r[i] = load16<false>(row + c + 4 * i);
        E::widen(r, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = c + i < d ? E::one(row[c + i]) : 0.0f;
    }
}

__device__ __forceinline__ uint32_t pack_codes(const float* x, float inv) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= (static_cast<uint32_t>(static_cast<int>(rintf(x[i] * inv))) & 0xFFu) << (8 * i);
    return r;
}

// The row's scale and 127 (1 / amax) from the bits of its largest magnitude
// (ordered like the magnitudes, with NaN above infinity above the rest).
__device__ __forceinline__ void row_scale(uint32_t amax_bits, float& scale, float& inv) {
    const float amax = __uint_as_float(amax_bits);
    scale = amax / 127.0f;
    inv = 127.0f * (1.0f / amax);
    if (amax_bits < 0x0D800000u) scale = inv = 0.0f;  // below 2^-100
    if (amax_bits >= 0x7F800000u) {
        scale = __uint_as_float(0x7FC00000u);
        inv = 0.0f;
    }
}

// One row a wave, four a workgroup, no barrier: rows of up to 4096 values stay
// in registers between the two steps.
constexpr int kWavePieces = 8;
template <class E, bool VEC>
__global__ __launch_bounds__(kThreads) void quantize_rows_wave_kernel(const typename E::T* __restrict__ X, int64_t rows,
                                                                      int d, int64_t ldx, int8_t* __restrict__ codes,
                                                                      int64_t ldc, float* __restrict__ scale) {
    const int lane = __lane_id();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWavesPerGroup + threadIdx.x / kWave;
    if (row >= rows) return;
    const typename E::T* x = X + row * ldx;
    const int end = (d + 15) / 16 * 16;
    float v[kWavePieces][8];
#pragma unroll
    for (int i = 0; i < kWavePieces; ++i) {
        const int c = (i * kWave + lane) * 8;
        if (i * kWave * 8 < d && c < d) {
            load8<E, VEC>(x, c, d, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kWavePieces; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) m = max(m, shfl_xor_u32(m, s));
    float sc, inv;
    row_scale(m, sc, inv);
    int8_t* out = codes + row * ldc;
#pragma unroll
    for (int i = 0; i < kWavePieces; ++i) {
        const int c = (i * kWave + lane) * 8;
        uint2 q = make_uint2(pack_codes(v[i], inv), pack_codes(v[i] + 4, inv));
        if (m >= 0x7F800000u) q = make_uint2(0u, 0u);
        if (c < end) *reinterpret_cast<uint2*>(out + c) = q;
    }
    if (lane == 0) scale[row] = sc;
}

// One row a workgroup, where rows are few or long; the first kKeep pieces of
// each thread stay in registers between the two steps, longer rows are read a
// second time (from cache).  In a row that is not finite inv is 0 and inf * 0 must not become
// a code, so such rows store zeros outright.
constexpr int kKeep = 4;
template <class E, bool VEC>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const typename E::T* __restrict__ X, int64_t rows,
                                                                 int d, int64_t ldx, int8_t* __restrict__ codes,
                                                                 int64_t ldc, float* __restrict__ scale) {
    __shared__ uint32_t red[kWavesPerGroup];
    const int pieces = ((d + 15) / 16) * 2;  // the row's codes end at a multiple of 16
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const typename E::T* x = X + row * ldx;
        float keep[kKeep][8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int c = (threadIdx.x + i * kThreads);
            if (c < pieces) load8<E, VEC>(x, c * 8, d, keep[i]);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) keep[i][e] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(keep[i][e]) & 0x7FFFFFFFu);
        for (int c = threadIdx.x + kKeep * kThreads; c < pieces; c += kThreads) {
            float v[8];
            load8<E, VEC>(x, c * 8, d, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int s = 1; s < kWave; s <<= 1) m = max(m, shfl_xor_u32(m, s));
        __syncthreads();  // the last row's reads of red are done
        if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = m;
        __syncthreads();
        m = max(max(red[0], red[1]), max(red[2], red[3]));
        float sc, inv;
        row_scale(m, sc, inv);
        const bool finite = m < 0x7F800000u;
        int8_t* out = codes + row * ldc;
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int c = threadIdx.x + i * kThreads;
            uint2 q = make_uint2(pack_codes(keep[i], inv), pack_codes(keep[i] + 4, inv));
            if (!finite) q = make_uint2(0u, 0u);
            if (c < pieces) *reinterpret_cast<uint2*>(out + c * 8) = q;
        }
        for (int c = threadIdx.x + kKeep * kThreads; c < pieces; c += kThreads) {
            float v[8];
            load8<E, VEC>(x, c * 8, d, v);
            uint2 q = make_uint2(pack_codes(v, inv), pack_codes(v + 4, inv));
            if (!finite) q = make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(out + c * 8) = q;
        }
        if (threadIdx.x == 0) scale[row] = sc;
    }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
// 16 codes of a row from column k, zeros beyond K; nothing beyond K is read.
// ALIGNED: row + k is a multiple of 16, so that the last, partial piece is at
// most one load each of 8, 4, 2 and 1 codes.
template <bool ALIGNED>
__device__ __forceinline__ u32x4 load_codes(const int8_t* row, int k, int K) {
    u32x4 r = u32x4{0u, 0u, 0u, 0u};
    if (k >= K) return r;
    const int8_t* p = row + k;
    if constexpr (ALIGNED) {
        if (k + 16 <= K) return load16<false>(p);
        const int n = K - k;
        if (n & 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            r[0] = v.x;
            r[1] = v.y;
        }
        uint32_t last = 0;
        if (n & 2) last = *reinterpret_cast<const uint16_t*>(p + (n & 12));
        if (n & 1) last |= static_cast<uint32_t>(static_cast<uint8_t>(p[n - 1])) << (8 * (n & 2));
        const uint32_t word = (n & 4) ? *reinterpret_cast<const uint32_t*>(p + (n & 8)) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if ((n & 4) && i == (n & 8) >> 2) r[i] = word;
            if ((n & 3) && i == n >> 2) r[i] = last;
        }
    } else {
        typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
        if (k + 16 <= K) return *reinterpret_cast<const u32x4_any*>(p);
        for (int i = 0; i < K - k; ++i) {
            const uint32_t v = static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * (i & 3));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i >> 2 == j) r[j] |= v;
        }
    }
    return r;
}

template <class E>
__device__ __forceinline__ void store_out(const Int8Product& p, int64_t m, int n, int acc) {
    float v = static_cast<float>(acc) * p.xs[m];
    v = v * p.ws[n];
    if (p.bias) v = v + E::one(static_cast<const typename E::T*>(p.bias)[n]);
    static_cast<typename E::T*>(p.out)[m * p.ldo + n] = E::narrow(v);
}

// Any shape and alignment: a tile of 32 B x 32 B a workgroup, four waves of
// half its side, 128 codes deep a step through LDS (rows 144 bytes apart, so
// that the 16 rows of a fragment start in different banks).  The loads need no
// alignment and go through registers: those of the next step are on their way
// while a step is multiplied.  For rows that do not all start at 16 bytes, which
// the kernels below need: 8192 x 11008 x 4096 697 us with one operand 8 bytes
// off and 735 to 862 with both, against their 328, 77 x 11008 x 4096 32 against
// 13.3, 500 x 4099 x 3840 40 against 20.
constexpr int kGenStep = 128, kGenPitch = 144;
template <class E, int B>
__global__ __launch_bounds__(kThreads) void int8_generic_kernel(const Int8Product p) {
    constexpr int kTile = 32 * B, kLoads = kTile * 8 / kThreads;
    __shared__ __align__(16) uint8_t lds[2][kTile * kGenPitch];
    const int lane = __lane_id(), wave = threadIdx.x / kWave;
    const int l16 = lane & 15, q = lane >> 4;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile;
    const int n0 = blockIdx.x * kTile;
    const int wm = (wave & 1) * 16 * B, wn = (wave >> 1) * 16 * B;
    const int row0 = threadIdx.x >> 3, piece = (threadIdx.x & 7) * 16;
    u32x4 xv[kLoads], wv[kLoads];
    auto load = [&](int k) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {  // rows past the matrix repeat its last one: they are not stored
            const int row = row0 + 32 * i;
            xv[i] = load_codes<false>(p.x + min<int64_t>(m0 + row, p.M - 1) * p.ldx, k + piece, p.K);
            wv[i] = load_codes<false>(p.w + static_cast<int64_t>(min(n0 + row, p.N - 1)) * p.ldw, k + piece, p.K);
        }
    };
    i32x4 acc[B][B] = {};
    load(0);
    for (int k = 0; k < p.K; k += kGenStep) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            *reinterpret_cast<u32x4*>(&lds[0][(row0 + 32 * i) * kGenPitch + piece]) = xv[i];
            *reinterpret_cast<u32x4*>(&lds[1][(row0 + 32 * i) * kGenPitch + piece]) = wv[i];
        }
        __syncthreads();
        if (k + kGenStep < p.K) load(k + kGenStep);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4 a[B], b[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                a[i] = *reinterpret_cast<const i32x4*>(&lds[0][(wm + 16 * i + l16) * kGenPitch + 64 * h + 16 * q]);
                b[i] = *reinterpret_cast<const i32x4*>(&lds[1][(wn + 16 * i + l16) * kGenPitch + 64 * h + 16 * q]);
            }
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int j = 0; j < B; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    }
    // lane l holds rows 4q + r, column l % 16 of each 16 x 16 block
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t m = m0 + wm + 16 * i + 4 * q + r;
                const int n = n0 + wn + 16 * j + l16;
                if (m < p.M && n < p.N) store_out<E>(p, m, n, acc[i][j][r]);
            }
}

// ---------------------------------------------------------------------------
// What the two product kernels share
// ---------------------------------------------------------------------------
// Operands reach the matrix cores through LDS, kDepth = 128 codes of a row a step: one
// cache line, and all banks of the LDS.  A lane needs 16 codes of row
// lane % 16, so reading them from memory directly would touch 16 rows with
// every 16 lanes (measured: 38 GB/s a CU against 115 for whole lines).  The
// loads write LDS themselves, linearly; the 16-byte pieces of a row stand at
// positions xor-ed with a key of the row, so that the 8 rows which a read
// touches at a time lie in different banks (no conflicts counted), and each
// lane fetches the piece that belongs at its position.
//
// The weight is the first matrix operand, so that lane l holds channels
// 4 (l / 16) .. + 3 of row l % 16; channel 4 TN (i / 4) + 4 j + i % 4 sits in
// row i of operand j, which makes a lane's 4 TN channels neighbours.
template <int TN>
__device__ __forceinline__ int operand_channel(int j, int i) {
    return 4 * TN * (i >> 2) + 4 * j + (i & 3);
}

typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes a lane from memory to LDS: lane l's go to lds + 16 l.  Counted with
// the vector loads, in order: landed<N>() waits until at most the last N are
// still on their way.
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, void* lds, int lane_offset, int offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, lane_offset, offset, 0, 0);
}

template <int N>
__device__ __forceinline__ void landed() {
    static_assert(N < 64, "the counter has six bits");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// Between LDS accesses of one wave whose lanes read what other lanes wrote, or
// write over what other lanes read, without a barrier: the hardware executes a
// wave's LDS accesses in order, and this holds the compiler to it as well.  No
// instruction comes of it.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ int key_x(int row) { return row & 7; }
template <int TN>
__device__ __forceinline__ int key_w(int row) {  // see operand_channel
    return (row & 3) | (row / (4 * TN) & 1) << 2;
}

// Where a lane's four sums stand in a 1 KB block of 16 rows (l16) and 4 x 4
// channels (q): the rows of neighbouring pieces c of 4 channels are xor-ed
// apart, so that neither the lanes that write a block nor the threads that
// read a row of several blocks meet in a bank.  (Integer atomics into one
// cleared array met four to a bank: 77 x 11008 x 4096 17.7 us, 16.6 so.)
__device__ __forceinline__ int sum_place(int l16, int q, int c) { return 16 * (16 * q + (l16 ^ c)); }

// Four neighbouring outputs of a row.
template <class E>
__device__ __forceinline__ void store_out4(const Int8Product& p, int64_t m, int n, const i32x4& acc, float xs,
                                           bool packed) {
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int c = min(n + r, p.N - 1);
        v[r] = static_cast<float>(acc[r]) * xs;
        v[r] = v[r] * p.ws[c];
        if (p.bias) v[r] = v[r] + E::one(static_cast<const typename E::T*>(p.bias)[c]);
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
bool out_aligned(const Int8Product& p, int64_t esize, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(p.out) % bytes == 0 && (p.M == 1 || p.ldo * esize % bytes == 0);
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
// A workgroup takes 16 MT rows and 16 TN channels.  Its waves split the depth
// and work alone, each with two steps of both operands in LDS of its own and
// no barrier: while one step is multiplied the next is on its way.  At the
// end each leaves its int32 sums where its operands were, and after the one
// barrier every thread adds four channels of all waves.  The weights are read from memory once; the rows of x come
// from cache.  Bound by the weights' bytes (77 x 11008 x 4096 in 13.3 us, 3.4
// TB/s) and, for the smallest, by the latency of a few loads and the launch.
template <class E, int MT, int TN, int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void int8_few_rows_kernel(const Int8Product p, int m_tiles, bool packed) {
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
    const int8_t* xb = p.x + m0 * p.ldx;
    const int8_t* wb = p.w + static_cast<int64_t>(n0) * p.ldw;
    const int ldx = static_cast<int>(p.ldx), ldw = static_cast<int>(p.ldw);

    // Load i covers rows 8 i .. 8 i + 7 of a tile; rows past the matrix read
    // its last row, their outputs are not stored.
    const int row0 = lane >> 3, piece0 = lane & 7;
    int xo[2 * MT], wo[2 * TN];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
        xo[i] = min(8 * i + row0, rows - 1) * ldx + 16 * (piece0 ^ key_x(8 * i + row0));
#pragma unroll
    for (int i = 0; i < 2 * TN; ++i)
        wo[i] = min(8 * i + row0, cols - 1) * ldw + 16 * (piece0 ^ key_w<TN>(8 * i + row0));
    auto fetch = [&](int s, uint8_t* to, bool live) {
        const int range = live ? 0x7FFFFFFF : 0;  // not live: issued, but reads nothing
        const auto xr = buf_rsrc(xb, range), wr = buf_rsrc(wb, range);
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i) load16_to_lds(wr, to + (BM + 8 * i) * kDepth, wo[i], s * kDepth);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            load16_to_lds(xr, to + 8 * i * kDepth, xo[i], s * kDepth);
    };
    i32x4 acc[MT][TN] = {}, x[2][MT], w[2][TN];
    auto read = [&](const uint8_t* from) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = operand_channel<TN>(j, l16);
                w[h][j] = *reinterpret_cast<const i32x4*>(from + (BM + row) * kDepth + 16 * ((4 * h + q) ^ key_w<TN>(row)));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
                x[h][i] = *reinterpret_cast<const i32x4*>(from + (16 * i + l16) * kDepth + 16 * ((4 * h + q) ^ key_x(l16)));
        }
    };
    auto multiply = [&] {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][j], x[h][i], acc[i][j], 0, 0, 0);
    };
    const int steps = p.K / kDepth;
    uint8_t *const e = even + wave * kStep, *const o = odd + wave * kStep;
    // A step's operands have arrived in LDS (of the loads on their way only
    // the next step's are newer), and have left it (lgkmcnt(0)) before the
    // loads of the step after the next go over them.  Past the last step everything but
    // the products is done all the same: branches around loads to LDS make
    // the compiler wait for all of them.
    auto turn_step = [&](int s, uint8_t* at) {
        landed<2 * (MT + TN)>();
        read(at);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        fetch(s + 2 * WAVES, at, s + 2 * WAVES < steps);
        if (s < steps) multiply();
    };
    fetch(wave, e, wave < steps);
    fetch(wave + WAVES, o, wave + WAVES < steps);
    for (int s = wave; s < steps; s += 2 * WAVES) {
        turn_step(s, e);
        turn_step(s + WAVES, o);
    }
    __builtin_amdgcn_s_waitcnt(0);
    if (steps * kDepth < p.K && steps % WAVES == wave) {  // the depth's partial step, zeros past K
        const int k = steps * kDepth;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int row = 8 * i + row0;
            *reinterpret_cast<u32x4*>(e + 8 * i * kDepth + lane * 16) = load_codes<true>(
                xb + static_cast<int64_t>(min(row, rows - 1)) * ldx, k + 16 * (piece0 ^ key_x(row)), p.K);
        }
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i) {
            const int row = 8 * i + row0;
            *reinterpret_cast<u32x4*>(e + (BM + 8 * i) * kDepth + lane * 16) = load_codes<true>(
                wb + static_cast<int64_t>(min(row, cols - 1)) * ldw, k + 16 * (piece0 ^ key_w<TN>(row)), p.K);
        }
        wave_order();
        read(e);
        multiply();
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
            *reinterpret_cast<i32x4*>(block(i * TN + j, wave) + sum_place(l16, q, TN * q + j)) = acc[i][j];
    __syncthreads();
    for (int t = threadIdx.x; t < BM * BN / 4; t += WAVES * kWave) {
        const int r = t / (BN / 4), c = t % (BN / 4);
        if (r >= rows || 4 * c >= cols) continue;
        const int n = (r >> 4) * TN + c % TN, at = sum_place(r & 15, c / TN, c);
        i32x4 sum = *reinterpret_cast<const i32x4*>(block(n, 0) + at);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += *reinterpret_cast<const i32x4*>(block(n, w) + at);
        store_out4<E>(p, m0 + r, n0 + 4 * c, sum, p.xs[m0 + r], packed);
    }
}

// ---------------------------------------------------------------------------
// A few tokens, quantized on the way
// ---------------------------------------------------------------------------
// The few-rows kernel for a few tokens whose codes every workgroup makes for
// itself, in LDS, while its first weights are on their way: one launch
// instead of two, for a reading of the tokens from cache by each workgroup.
// bf16, weights from memory, two launches and one: 1 x 4096 x 4096 9.6 and 6.5
// us (2.6 TB/s; its 16.8 MB alone would take 3.2 us), 1 x 32000 x 4096 35.1 and
// 32.4 (4.0 TB/s), 8 x 4096 x 2048 8.4 and 7.4, but 4 x 11008 x 4096 15.9 and
// 16.3.
template <class E, int TN, int WAVES, bool VEC>
__global__ __launch_bounds__(WAVES* kWave) void int8_tokens_kernel(const Int8Product p,
                                                                   const typename E::T* __restrict__ X, int64_t ldX,
                                                                   bool packed) {
    constexpr int BN = TN * 16, kStep = BN * kDepth;
    __shared__ __align__(1024) uint8_t even[WAVES * kStep], odd[WAVES * kStep];
    __shared__ __align__(16) int8_t codes[kTokenBytes];
    __shared__ uint32_t amax[WAVES * kItems];
    __shared__ float scale[kMaxTokens];
    static_assert(TN * 1024 <= kStep, "the sums fit over the operands");
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, q = lane >> 4;
    const int rows = static_cast<int>(p.M), n0 = blockIdx.x * BN, cols = min(p.N - n0, BN);
    const int8_t* wb = p.w + static_cast<int64_t>(n0) * p.ldw;
    const int ldw = static_cast<int>(p.ldw);
    const int row0 = lane >> 3, piece0 = lane & 7;
    int wo[2 * TN];
#pragma unroll
    for (int i = 0; i < 2 * TN; ++i)
        wo[i] = min(8 * i + row0, cols - 1) * ldw + 16 * (piece0 ^ key_w<TN>(8 * i + row0));
    auto fetch = [&](int s, uint8_t* to, bool live) {
        const auto wr = buf_rsrc(wb, live ? 0x7FFFFFFF : 0);
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i) load16_to_lds(wr, to + 8 * i * kDepth, wo[i], s * kDepth);
    };
    const int steps = p.K / kDepth;
    uint8_t *const e = even + wave * kStep, *const o = odd + wave * kStep;
    fetch(wave, e, wave < steps);
    fetch(wave + WAVES, o, wave + WAVES < steps);

    // The tokens' codes.
    const int per_row = (p.K + 511) / 512, items = rows * per_row;
    const int pitch = (p.K + kDepth - 1) / kDepth * kDepth + kTokenPad;
    float keep[kItems][8];
#pragma unroll
    for (int t = 0; t < kItems; ++t) {
        const int item = wave + t * WAVES;
        if (item < items) {
            const int r = item / per_row;
            load8<E, VEC>(X + r * ldX, (item - r * per_row) * 512 + lane * 8, p.K, keep[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < kItems; ++t) {
        const int item = wave + t * WAVES;
        if (item < items) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(keep[t][i]) & 0x7FFFFFFFu);
#pragma unroll
            for (int d = 1; d < kWave; d <<= 1) m = max(m, shfl_xor_u32(m, d));
            if (lane == 0) amax[item] = m;
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kItems; ++t) {
        const int item = wave + t * WAVES;
        if (item < items) {
            const int r = item / per_row, c = (item - r * per_row) * 512 + lane * 8;
            uint32_t m = 0;
            for (int i = 0; i < per_row; ++i) m = max(m, amax[r * per_row + i]);
            float sc, inv;
            row_scale(m, sc, inv);
            uint2 v = make_uint2(pack_codes(keep[t], inv), pack_codes(keep[t] + 4, inv));
            if (m >= 0x7F800000u) v = make_uint2(0u, 0u);
            if (c < pitch - kTokenPad) *reinterpret_cast<uint2*>(codes + r * pitch + c) = v;
            if (c == 0) scale[r] = sc;
        }
    }
    __syncthreads();

    i32x4 acc[TN] = {}, x[2], w[2][TN];
    const int8_t* mine = codes + min(l16, rows - 1) * pitch + 16 * q;  // rows past the last repeat it
    auto read = [&](const uint8_t* from, int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = operand_channel<TN>(j, l16);
                w[h][j] = *reinterpret_cast<const i32x4*>(from + row * kDepth + 16 * ((4 * h + q) ^ key_w<TN>(row)));
            }
            x[h] = *reinterpret_cast<const i32x4*>(mine + min(s, (p.K - 1) / kDepth) * kDepth + 64 * h);
        }
    };
    auto multiply = [&] {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][j], x[h], acc[j], 0, 0, 0);
    };
    auto turn_step = [&](int s, uint8_t* at) {  // as in the few-rows kernel
        landed<2 * TN>();
        read(at, s);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        fetch(s + 2 * WAVES, at, s + 2 * WAVES < steps);
        if (s < steps) multiply();
    };
    for (int s = wave; s < steps; s += 2 * WAVES) {
        turn_step(s, e);
        turn_step(s + WAVES, o);
    }
    __builtin_amdgcn_s_waitcnt(0);
    if (steps * kDepth < p.K && steps % WAVES == wave) {
        const int k = steps * kDepth;
#pragma unroll
        for (int i = 0; i < 2 * TN; ++i) {
            const int row = 8 * i + row0;
            *reinterpret_cast<u32x4*>(e + 8 * i * kDepth + lane * 16) = load_codes<true>(
                wb + static_cast<int64_t>(min(row, cols - 1)) * ldw, k + 16 * (piece0 ^ key_w<TN>(row)), p.K);
        }
        wave_order();
        read(e, steps);
        multiply();
    }
    wave_order();
#pragma unroll
    for (int j = 0; j < TN; ++j)
        *reinterpret_cast<i32x4*>(e + j * 1024 + sum_place(l16, q, TN * q + j)) = acc[j];
    __syncthreads();
    for (int t = threadIdx.x; t < rows * BN / 4; t += WAVES * kWave) {
        const int r = t / (BN / 4), c = t % (BN / 4);
        if (4 * c >= cols) continue;
        const uint8_t* at = even + c % TN * 1024 + sum_place(r, c / TN, c);
        i32x4 sum = *reinterpret_cast<const i32x4*>(at);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += *reinterpret_cast<const i32x4*>(at + w * kStep);
        store_out4<E>(p, r, n0 + 4 * c, sum, scale[r], packed);
    }
}

// ---------------------------------------------------------------------------
// Many rows: tiles through LDS.
// ---------------------------------------------------------------------------
// A workgroup of WM x WN waves takes a tile of 16 TM WM rows and 64 WN
// channels, two steps of both operands in LDS: while the matrix cores work on
// one, the loads of the next go into the other.  Tiles of 256 x 256 on 8 waves
// need 1/256 byte of operands an operation, half of what 128 x 128 needs, and
// run 8192 x 11008 x 4096 in 328 us with its scales (2.25 POP/s; the library's
// product into int32, without scales, takes 334 to 341); the smaller ones are for what
// would not fill the device (choose_form).  The matrix pipes are busy for 53%
// of the kernel's cycles, without one bank conflict: what is lost goes to the
// step's barrier, to the rounds' ends (one workgroup fits a compute unit: 7.5
// us each, 5 where a workgroup stays, see below) and to the last, partly filled
// round.  Not kept, 4096^3 in 61 us:
// fetching the next operands into L2 first 68, steps of 64 codes in a ring of
// four 67.5, a second launch for the last round no gain.
//
// A wave's 16 TM x 64 outputs, through a region of LDS that is the wave's own,
// so that a row leaves as one run of 64 channels: a lane's 16 channels alone
// are 32 bytes of a line, and writing those cost 36 us a tile of 256 x 256.
// The 16-byte pieces of a row are xor-ed with the row like the operands'.
// NT, stores that do not stay in L2: 8192 x 11008 x 4096 380 -> 368 us in tiles
// of 256 rows, 435 -> 408 us in 128, but 75.0 -> 80.3 us (1000 x 11008) in 64.
// m, n: the wave's first row and channel.
template <class E>
constexpr bool kSums = std::is_same<typename E::T, int>::value;  // the sums themselves, no scales

template <int TM>
struct Scales {  // of a lane's 16 channels and TM rows
    float w[16], bias[16], x[TM];
};
template <class E, int TM>
__device__ __forceinline__ void load_scales(const Int8Product& p, int lane, int64_t m, int n, Scales<TM>& s) {
    const int l16 = lane & 15, q = lane >> 4;
    if constexpr (!kSums<E>) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            s.w[e] = p.ws[n + 16 * q + e];
            s.bias[e] = 0.0f;
        }
        if (p.bias) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s.bias[e] = E::one(static_cast<const typename E::T*>(p.bias)[n + 16 * q + e]);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) s.x[i] = p.xs[m + 16 * i + l16];
    }
}

template <class E, int TM, int kRegion, bool NT>
__device__ __forceinline__ void store_tile(const Int8Product& p, typename E::T* out, uint8_t* region, int lane,
                                           int64_t m, int n, const i32x4 (&acc)[TM][4], const Scales<TM>& s,
                                           bool packed) {
    using T = typename E::T;
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
            for (int e = 0; e < 16 && !kSums<E>; ++e) {
                v[e] = static_cast<float>(acc[i0 + i][e >> 2][e & 3]) * s.x[i0 + i] * s.w[e];
                if (p.bias) v[e] = v[e] + s.bias[e];
            }
#pragma unroll
            for (int c = 0; c < kSize; ++c) {  // the lane's 16 kSize bytes
                u32x4 d;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (kSums<E>) d[r] = acc[i0 + i][c][r];
                    else if constexpr (kSize == 4) d[r] = __float_as_uint(v[4 * c + r]);
                    else d[r] = E::pack(v[8 * c + 2 * r], v[8 * c + 2 * r + 1]);
                }
                *reinterpret_cast<u32x4*>(region + row * kRow + 16 * ((q * kSize + c) ^ (row & 7))) = d;
            }
        }
        wave_order();
        if (packed) {
            constexpr int kPieces = kRow / 16, kRows = kWave / kPieces;  // rows a store instruction
#pragma unroll
            for (int r0 = 0; r0 < kPass * 16; r0 += kRows) {
                const int row = r0 + lane / kPieces, piece = lane % kPieces;
                const u32x4 d = *reinterpret_cast<const u32x4*>(region + row * kRow + 16 * (piece ^ (row & 7)));
                store16<NT>(out + (16 * i0 + row) * p.ldo + piece * (16 / kSize), d);
            }
        } else {
            for (int row = 0; row < kPass * 16; ++row) {
                const int piece = lane / (16 / kSize), at = lane % (16 / kSize);
                out[(16 * i0 + row) * p.ldo + lane] = reinterpret_cast<const T*>(
                    region + row * kRow + 16 * (piece ^ (row & 7)))[at];
            }
        }
        if (i0 + kPass < TM) wave_order();  // the next pass goes over the region
    }
}

// The partial step of an operand to LDS: rows row0, row0 + ROUND, ... from
// column 0 of `from`, `left` codes each, zeros past them (nothing else is
// read).  The loads of all rows are on their way together.
template <int LOADS, int ROUND, class Key>
__device__ __forceinline__ void store_partial(const int8_t* from, int64_t ld, int left, uint8_t* to, int row0, int piece0,
                                              const Key& key) {
    const int full = left >> 4, n = left & 15;  // whole pieces, codes of the one after them
    const int8_t* row[LOADS];
    int piece[LOADS];
    u32x4 d[LOADS];
    uint2 b8[LOADS];
    uint32_t b4[LOADS], b2[LOADS], b1[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        row[i] = from + (row0 + i * ROUND) * ld;
        piece[i] = piece0 ^ key(row0 + i * ROUND);
        d[i] = u32x4{0u, 0u, 0u, 0u};
        b8[i] = make_uint2(0u, 0u);
        b4[i] = b2[i] = b1[i] = 0u;
        if (piece[i] < full) d[i] = load16<false>(row[i] + 16 * piece[i]);
        row[i] += 16 * full;
    }
    if (n & 8) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (piece[i] == full) b8[i] = *reinterpret_cast<const uint2*>(row[i]);
    }
    if (n & 4) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (piece[i] == full) b4[i] = *reinterpret_cast<const uint32_t*>(row[i] + (n & 8));
    }
    if (n & 2) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (piece[i] == full) b2[i] = *reinterpret_cast<const uint16_t*>(row[i] + (n & 12));
    }
    if (n & 1) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (piece[i] == full) b1[i] = static_cast<uint8_t>(row[i][n & 14]);
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        if (piece[i] == full) {
            const uint32_t last = b2[i] | b1[i] << (8 * (n & 2));
            d[i] = u32x4{b8[i].x, b8[i].y, 0u, 0u};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if ((n & 4) && w == (n & 8) >> 2) d[i][w] = b4[i];
                if ((n & 3) && w == n >> 2) d[i][w] = last;
            }
        }
        *reinterpret_cast<u32x4*>(to + (row0 + i * ROUND) * kDepth + 16 * piece0) = d[i];
    }
}

// With E = QSums the depth is split as well: workgroups (x, y) take the codes
// from y part_depth on, at most part_depth (whole pairs of steps), and store
// their sums as they are, one matrix after the other.
struct QSums {
    using T = int;
    static __device__ T narrow(float);  // unused
    static __device__ float one(T);
};

// With STAY a workgroup takes one tile after the other: the first two steps of
// the next are on their way while the outputs of one leave, through LDS of
// their own, and the next one's products do not wait for those stores.  For
// whole pairs of steps and outputs of whole 16-byte pieces.  8192 x 11008 x 1024
// 126.9 us without, 112.7 with; 6000 x 6000 x 2048 106 and 101, 4096^3 59.8 and
// 58.2, no difference from 8192 x 8192 x 8192 on.
template <class E, int WM, int WN, int TM, bool STAY>
__global__ __launch_bounds__(WM* WN* kWave) void int8_tile_kernel(const Int8Product p, int m_tiles, int n_tiles,
                                                                  int part_depth, bool packed) {
    using T = typename E::T;
    constexpr bool kSplit = kSums<E>;
    constexpr int TN = 4, kT = WM * WN * kWave;
    constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
    constexpr int kXLoads = BM * 8 / kT, kWLoads = BN * 8 / kT;
    static_assert(BM * 8 % kT == 0 && BN * 8 % kT == 0, "whole rounds of loads");
    // Four arrays by name, and code that names the one it means: the compiler
    // then sees that the operands it reads are not those on their way, and
    // puts no wait for the loads before the reads.
    __shared__ __align__(1024) uint8_t x_even[BM * kDepth], x_odd[BM * kDepth], w_even[BN * kDepth], w_odd[BN * kDepth];
    constexpr int kPassing = 1024 * sizeof(T);  // 16 rows of outputs a wave
    __shared__ __align__(1024) uint8_t passing[STAY ? WM * WN * kPassing : 16];
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, q = lane >> 4;
    const int wm = (wave % WM) * TM * 16, wn = (wave / WM) * TN * 16;

    // Each XCD works through a contiguous range of tiles, in groups of 8 rows
    // of tiles, so that its L2 holds the operands its workgroups share.
    const int tiles = m_tiles * n_tiles;
    const int per = (tiles + 7) / 8;
    const int end = min(static_cast<int>(blockIdx.x & 7) * per + per, tiles);
    int t = static_cast<int>(blockIdx.x & 7) * per + static_cast<int>(blockIdx.x >> 3);
    if (t >= end) return;
    const int first = kSplit ? static_cast<int>(blockIdx.y) * part_depth : 0;
    const int K = kSplit ? min(p.K - first, part_depth) : p.K;
    int64_t m0;
    int n0;
    const int8_t *xb, *wb;
    auto to_tile = [&] {
        constexpr int kGroupM = 8;
        const int group = t / (kGroupM * n_tiles), in = t - group * kGroupM * n_tiles;
        const int gm = min(kGroupM, m_tiles - group * kGroupM);
        // The last tiles of a row or column are moved inside the matrix (M >=
        // BM, N >= BN): outputs computed twice get the same values twice.
        m0 = min<int64_t>(static_cast<int64_t>(group * kGroupM + in % gm) * BM, p.M - BM);
        n0 = min(in / gm * BN, p.N - BN);
        xb = p.x + m0 * p.ldx + first;
        wb = p.w + static_cast<int64_t>(n0) * p.ldw + first;
    };
    to_tile();
    // A round of loads covers kRound rows; the keys repeat from round to
    // round, but for the weights' where a round is shorter than their period.
    constexpr int kRound = kT / 8;
    constexpr bool kTwoKeys = kRound % (8 * TN) != 0;
    const int row0 = (wave * kWave + lane) >> 3, piece0 = lane & 7;
    const int ldx = static_cast<int>(p.ldx), ldw = static_cast<int>(p.ldw);
    const int xo = row0 * ldx + 16 * (piece0 ^ key_x(row0));
    const int wo0 = row0 * ldw + 16 * (piece0 ^ key_w<TN>(row0));
    const int wo1 = kTwoKeys ? row0 * ldw + 16 * (piece0 ^ key_w<TN>(row0 + kRound)) : wo0;
    // Loads that are not `live` are issued all the same, to an empty range, and
    // read no memory: a branch around them would make the compiler wait.
    auto fetch = [&](int k, uint8_t* xd, uint8_t* wd, bool live) {
        const int range = live ? 0x7FFFFFFF : 0;
        const auto xr = buf_rsrc(xb, range), wr = buf_rsrc(wb, range);
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
            load16_to_lds(xr, xd + (i * kT + wave * kWave) * 16, xo, k + i * kRound * ldx);
#pragma unroll
        for (int i = 0; i < kWLoads; ++i)
            load16_to_lds(wr, wd + (i * kT + wave * kWave) * 16, (i & 1) ? wo1 : wo0, k + i * kRound * ldw);
    };

    // Half a step's operands (64 codes deep) in LDS; the keys do not change
    // with i and j, 16 and 4 rows on.
    const int w_row = operand_channel<TN>(0, l16);
    const int xp[2] = {(wm + l16) * kDepth + 16 * (q ^ key_x(l16)), (wm + l16) * kDepth + 16 * ((4 + q) ^ key_x(l16))};
    const int wp[2] = {(wn + w_row) * kDepth + 16 * (q ^ key_w<TN>(w_row)),
                       (wn + w_row) * kDepth + 16 * ((4 + q) ^ key_w<TN>(w_row))};
    i32x4 acc[TM][TN];
    i32x4 x[TM], w0[TN], w1[TN];
    auto read_x = [&](const uint8_t* xd, int h, int i) {
        x[i] = *reinterpret_cast<const i32x4*>(xd + xp[h] + 16 * i * kDepth);
    };
    auto read_w = [&](const uint8_t* wd, int h, int j) {
        return *reinterpret_cast<const i32x4*>(wd + wp[h] + 4 * j * kDepth);
    };
    auto read = [&](const uint8_t* xd, const uint8_t* wd, int h, i32x4 (&w)[TN]) {
#pragma unroll
        for (int j = 0; j < TN; ++j) w[j] = read_w(wd, h, j);
#pragma unroll
        for (int i = 0; i < TM; ++i) read_x(xd, h, i);
    };
    // The products of half a step; each operand of x is replaced by half h of
    // (xn, wn) as soon as its last product is issued, and the next weights are
    // read on the way.
    constexpr int kPer = TM < TN ? TN / TM : 1;
    auto multiply = [&](const i32x4 (&w)[TN], const uint8_t* xn, const uint8_t* wn, int h, i32x4 (&w_next)[TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], x[i], acc[i][j], 0, 0, 0);
            read_x(xn, h, i);
#pragma unroll
            for (int j = i * kPer; j < (i + 1) * kPer && j < TN; ++j) w_next[j] = read_w(wn, h, j);
            __builtin_amdgcn_sched_group_barrier(0x008, TN, 0);
            if (i * kPer < TN) __builtin_amdgcn_sched_group_barrier(0x100, 1 + kPer, 0);
            else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
    };
    auto multiply_all = [&](const i32x4 (&w)[TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], x[i], acc[i][j], 0, 0, 0);
    };

    // Software pipeline: while half a step is multiplied the next half is read
    // from LDS, and the step after it is on its way from memory.  The one
    // barrier of a step stands between its halves: past it every wave's loads
    // of step s + 1 have arrived and nobody reads step s any more, so that
    // step s + 2 may be fetched over it.
    auto arrive = [&] {
        __builtin_amdgcn_s_waitcnt(0);  // loads to LDS are counted with the vector loads: a barrier does not wait for them
        __syncthreads();
    };
    const int steps = K / (2 * kDepth) * 2;
    // One step from (xd, wd), the next one's first half from (xn, wn).
    auto step = [&](int s, uint8_t* xd, uint8_t* wd, const uint8_t* xn, const uint8_t* wn) {
        multiply(w0, xd, wd, 1, w1);
        arrive();
        fetch((s + 2) * kDepth, xd, wd, s + 2 < steps);
        multiply(w1, xn, wn, 0, w0);
    };
    constexpr int kStores = TM * sizeof(T);  // a wave's stores of a tile
    bool fetched = false;
    for (;;) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
        // The pipeline takes pairs of steps.  What the depth has beyond them
        // comes first (the sums are exact in any order): a whole step like the
        // others, a partial one piece by piece through registers, zeros past K.
        if constexpr (!STAY) {
            auto alone = [&] {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    read(x_even, w_even, h, w0);
                    multiply_all(w0);
                }
                __syncthreads();
            };
            int k = steps * kDepth;
            if (k + kDepth <= K) {
                fetch(k, x_even, w_even, true);
                arrive();
                alone();
                k += kDepth;
            }
            if (k < K) {
                store_partial<kXLoads, kRound>(xb + k, ldx, K - k, x_even, row0, piece0, [](int row) { return key_x(row); });
                store_partial<kWLoads, kRound>(wb + k, ldw, K - k, w_even, row0, piece0,
                                               [](int row) { return key_w<TN>(row); });
                __syncthreads();
                alone();
            }
        }
        if (STAY && fetched) {
            landed<kStores>();  // the operands are older than the last tile's stores
            __syncthreads();
        } else {
            fetch(0, x_even, w_even, steps > 0);
            fetch(kDepth, x_odd, w_odd, steps > 0);
            arrive();
        }
        read(x_even, w_even, 0, w0);
        for (int s = 0; s < steps; s += 2) {  // past the last step it reads operands that nobody multiplies
            step(s, x_even, w_even, x_odd, w_odd);
            step(s + 1, x_odd, w_odd, x_even, w_even);
        }
        // What follows runs once a tile: its addresses are made anew from the
        // thread's number, so that the loop above keeps no registers for them.
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        T* out = static_cast<T*>(p.out);
        if constexpr (kSplit) out += blockIdx.y * p.M * p.ldo;
        const int64_t m = m0 + wm;
        const int n = n0 + wn;
        Scales<TM> scales;
        load_scales<E, TM>(p, tid & 63, m, n, scales);
        arrive();  // the operands are read, and the empty loads of the last steps are done
        if constexpr (STAY) {
            t += static_cast<int>(gridDim.x >> 3);
            fetched = t < end;
            if (fetched) {
                to_tile();
                fetch(0, x_even, w_even, true);
                fetch(kDepth, x_odd, w_odd, true);
            }
            store_tile<E, TM, kPassing, true>(p, out, passing + wave * kPassing, tid & 63, m, n, acc, scales, true);
            if (!fetched) return;
        } else {
            // A region for each wave, in the array that has room for it.
            constexpr int kPart = (BM < BN ? BM : BN) >= 256 ? 16384 : (BM < BN ? BM : BN) >= 64 ? 8192 : 4096;
            static_assert(kPart <= BM * kDepth && kPart <= BN * kDepth, "a region fits into either array");
            constexpr int kInX = BM * kDepth / kPart, kInW = BN * kDepth / kPart;
            static_assert(2 * kInX + 2 * kInW >= WM * WN, "a region for every wave");
            uint8_t* region = wave < kInX ? x_even + wave * kPart
                              : wave < 2 * kInX ? x_odd + (wave - kInX) * kPart
                              : wave < 2 * kInX + kInW ? w_even + (wave - 2 * kInX) * kPart
                                                       : w_odd + (wave - 2 * kInX - kInW) * kPart;
            store_tile<E, TM, kPart, (BM >= 128 && !kSplit)>(p, out, region, tid & 63, m, n, acc, scales,
                                                             packed && (n0 * sizeof(T)) % 16 == 0);
            return;
        }
    }
}

// Adds the parts' sums and applies the scales: four channels a thread.
template <class E>
__global__ __launch_bounds__(kThreads) void int8_add_parts_kernel(const Int8Product p, const int* __restrict__ sums,
                                                                  int64_t ld, int parts, bool packed) {
    const uint32_t pieces = static_cast<uint32_t>(p.N + 3) / 4, at = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t m = at / pieces;
    if (m >= p.M) return;
    const int n = static_cast<int>(at - m * pieces) * 4;
    const int* s = sums + m * ld + n;
    i32x4 acc = *reinterpret_cast<const i32x4*>(s);
    for (int i = 1; i < parts; ++i) acc += *reinterpret_cast<const i32x4*>(s + i * (p.M * ld));
    store_out4<E>(p, m, n, acc, p.xs[m], packed);
}

template <class E, int MT, int TN, int WAVES>
int launch_few(const Int8Product& p, void* stream) {
    const int m_tiles = static_cast<int>((p.M + MT * 16 - 1) / (MT * 16)), n_tiles = (p.N + TN * 16 - 1) / (TN * 16);
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(m_tiles) * n_tiles + 7) / 8 * 8);
    hipLaunchKernelGGL((int8_few_rows_kernel<E, MT, TN, WAVES>), dim3(grid), dim3(WAVES * kWave), 0,
                       static_cast<hipStream_t>(stream), p, m_tiles, out_aligned(p, sizeof(typename E::T), 4 * sizeof(typename E::T)));
    return static_cast<int>(hipGetLastError());
}

template <class E, int WM, int WN, int TM, bool STAY>
int launch_tile(const Int8Product& p, void* stream) {
    constexpr int BM = WM * TM * 16, BN = WN * 64;
    const int m_tiles = static_cast<int>((p.M + BM - 1) / BM), n_tiles = (p.N + BN - 1) / BN;
    unsigned grid = static_cast<unsigned>((static_cast<int64_t>(m_tiles) * n_tiles + 7) / 8 * 8);
    if (STAY) {  // one workgroup a compute unit, the same number on each XCD
        const unsigned resident = device_cu_count() < 8 ? 8u : static_cast<unsigned>(device_cu_count()) / 8 * 8;
        if (grid > resident) grid = resident;
    }
    hipLaunchKernelGGL((int8_tile_kernel<E, WM, WN, TM, STAY>), dim3(grid), dim3(WM * WN * kWave), 0,
                       static_cast<hipStream_t>(stream), p, m_tiles, n_tiles, 0, out_aligned(p, sizeof(typename E::T), 16));
    return static_cast<int>(hipGetLastError());
}

// Tiles of 128 x 128 with the depth in parts (as many as split_depth leaves).
template <class E>
int launch_split(const Int8Product& p, int parts, void* workspace, void* stream) {
    const int m_tiles = static_cast<int>((p.M + kSplitTile - 1) / kSplitTile);
    const int n_tiles = (p.N + kSplitTile - 1) / kSplitTile;
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(m_tiles) * n_tiles + 7) / 8 * 8);
    const int part_depth = split_depth(p.K, parts);
    Int8Product s = p;
    s.out = workspace;
    s.ldo = sums_ld(p.N);
    hipLaunchKernelGGL((int8_tile_kernel<QSums, 2, 2, 4, false>), dim3(grid, parts), dim3(4 * kWave), 0,
                       static_cast<hipStream_t>(stream), s, m_tiles, n_tiles, part_depth, true);
    const int e = static_cast<int>(hipGetLastError());
    if (e != 0) return e;
    const uint32_t pieces = static_cast<uint32_t>(p.M) * (static_cast<uint32_t>(p.N + 3) / 4);
    hipLaunchKernelGGL((int8_add_parts_kernel<E>), dim3((pieces + kThreads - 1) / kThreads), dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), p, static_cast<const int*>(workspace), s.ldo, parts,
                       out_aligned(p, sizeof(typename E::T), 4 * sizeof(typename E::T)));
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_generic(const Int8Product& p, void* stream) {
    const auto grid = [&](int tile) {
        return dim3((p.N + tile - 1) / tile, static_cast<unsigned>((p.M + tile - 1) / tile));
    };
    const dim3 large = grid(128);  // half the operands' traffic, once its tiles fill the device
    if (static_cast<int64_t>(large.x) * large.y >= device_cu_count())
        hipLaunchKernelGGL((int8_generic_kernel<E, 4>), large, dim3(kThreads), 0, static_cast<hipStream_t>(stream), p);
    else
        hipLaunchKernelGGL((int8_generic_kernel<E, 2>), grid(64), dim3(kThreads), 0, static_cast<hipStream_t>(stream), p);
    return static_cast<int>(hipGetLastError());
}

// The waves that split the depth: as many as their operands fit into LDS, but
// for the smallest pieces, several of which share a compute unit.  16 x 16, in 4 /
// 8 / 16 waves with operands from memory: 6 x 1216 x 768 3.1 / 3.6 / 4.1 us, 16 x
// 4096 x 2048 4.6 / 4.7 / 5.6, 16 x 4096 x 4096 6.4 / 6.6 / 6.9, 16 x 1024 x 8192
// 7.6 / 7.4 / 7.7.
template <class E>
int launch_few_tile(const Int8Product& p, Int8Few f, void* stream) {
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
        case 54: return launch_few<E, 5, 4, 4>(p, stream);
        case 73: return launch_few<E, 7, 3, 4>(p, stream);
        default: return launch_few<E, 8, 3, 3>(p, stream);
    }
}

template <class E>
int launch_form(const Int8Product& p, const Int8Choice& c, void* workspace, void* stream) {
    if (c.parts > 1) return launch_split<E>(p, c.parts, workspace, stream);
    switch (c.bm) {
        case 0: return launch_few_tile<E>(p, c.few, stream);
        case 32: return launch_tile<E, 2, 2, 1, false>(p, stream);
        case 64: return launch_tile<E, 2, 2, 2, false>(p, stream);
        case 128: return launch_tile<E, 2, 2, 4, false>(p, stream);
        default: break;
    }
    constexpr int kSize = sizeof(typename E::T);
    return p.K % (2 * kDepth) == 0 && p.N * kSize % 16 == 0 && out_aligned(p, kSize, 16)
               ? launch_tile<E, 2, 4, 8, true>(p, stream)
               : launch_tile<E, 2, 4, 8, false>(p, stream);
}

template <class E>
int launch_product_e(const Int8Product& whole, bool aligned, void* workspace, void* stream) {
    using T = typename E::T;
    const int64_t cus = device_cu_count();
    // The other kernels' offsets inside a tile are 32 bits wide.
    const bool far = (whole.M > 1 && whole.ldx >= kFarRows) || (whole.N > 1 && whole.ldw >= kFarRows);
    for (int64_t n = 0; n < whole.N; n += kMaxChannels) {
        for (int64_t m = 0; m < whole.M; m += kRowBlock) {
            Int8Product p = whole;
            p.M = whole.M - m < kRowBlock ? whole.M - m : kRowBlock;
            p.N = static_cast<int>(whole.N - n < kMaxChannels ? whole.N - n : kMaxChannels);
            p.x += m * p.ldx;
            p.xs += m;
            p.w += n * p.ldw;
            p.ws += n;
            if (p.bias) p.bias = static_cast<const T*>(p.bias) + n;
            p.out = static_cast<T*>(p.out) + m * p.ldo + n;
            const int e = !aligned || far
                              ? launch_generic<E>(p, stream)
                              : launch_form<E>(p, choose_form(p.M, p.N, p.K, cus), workspace, stream);
            if (e != 0) return e;
        }
    }
    return 0;
}

template <class E, int TN, int WAVES>
int launch_tokens_t(const Int8Product& p, const void* X, int64_t ldX, bool vec, void* stream) {
    const dim3 grid((p.N + TN * 16 - 1) / (TN * 16)), block(WAVES * kWave);
    const auto* x = static_cast<const typename E::T*>(X);
    const bool packed = out_aligned(p, sizeof(typename E::T), 4 * sizeof(typename E::T));
    if (vec)
        hipLaunchKernelGGL((int8_tokens_kernel<E, TN, WAVES, true>), grid, block, 0, static_cast<hipStream_t>(stream), p,
                           x, ldX, packed);
    else
        hipLaunchKernelGGL((int8_tokens_kernel<E, TN, WAVES, false>), grid, block, 0, static_cast<hipStream_t>(stream),
                           p, x, ldX, packed);
    return static_cast<int>(hipGetLastError());
}

// Channels a workgroup (one fits a compute unit): 16, 48 or 64, whose rounds
// over the device take about 1 : 2 : 3, the largest of equals.  One token x
// 4096 in 16 / 48 / 64: 4096 channels 6.5 / 9.4 / 10.8 us, 6000 10.8 / 10.3 / 11.3,
// 11008 15.9 / 13.6 / 13.8, 14336 20.3 / 20.7 / 15.9, 32000 39.0 / 33.5 / 32.4; two
// tokens, 20000 x 2048, 22.3 / 14.7 / 16.4.  Pieces of 16 in 16 waves, not 8: 1 x
// 4096 x 4096 6.5 against 8.5 us, 1 x 4096 x 1024 4.4 against 4.2.
template <class E>
int launch_tokens_e(const Int8Product& p, const void* X, int64_t ldX, bool vec, void* stream) {
    const int cus = device_cu_count();
    auto rounds = [&](int channels) { return (p.N + channels * cus - 1) / (channels * cus); };
    const int c16 = rounds(16), c48 = 2 * rounds(48), c64 = 3 * rounds(64);
    if (c64 <= c48 && c64 <= c16) return launch_tokens_t<E, 4, 8>(p, X, ldX, vec, stream);
    if (c48 <= c16) return launch_tokens_t<E, 3, 8>(p, X, ldX, vec, stream);
    return launch_tokens_t<E, 1, 16>(p, X, ldX, vec, stream);
}

template <class E, bool VEC>
int launch_rows_v(const typename E::T* x, int64_t rows, int d, int64_t ldx, int8_t* codes, int64_t ldc, float* scale,
                  void* stream) {
    // A wave a row once that gives every compute unit a workgroup: 8192 rows
    // of 4096 in bf16 28.2 us with a workgroup a row, 22.7 with a wave (4.4 TB/s).
    const int64_t groups = (rows + kWavesPerGroup - 1) / kWavesPerGroup;
    if (groups >= device_cu_count() && groups < (1 << 24) && d <= kWavePieces * kWave * 8) {
        hipLaunchKernelGGL((quantize_rows_wave_kernel<E, VEC>), dim3(static_cast<unsigned>(groups)), dim3(kThreads), 0,
                           static_cast<hipStream_t>(stream), x, rows, d, ldx, codes, ldc, scale);
    } else {
        const unsigned grid = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
        hipLaunchKernelGGL((quantize_rows_kernel<E, VEC>), dim3(grid), dim3(kThreads), 0,
                           static_cast<hipStream_t>(stream), x, rows, d, ldx, codes, ldc, scale);
    }
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_rows_e(const void* X, int64_t rows, int d, int64_t ldx, int8_t* codes, int64_t ldc, float* scale, bool vec,
                  void* stream) {
    const auto* x = static_cast<const typename E::T*>(X);
    return vec ? launch_rows_v<E, true>(x, rows, d, ldx, codes, ldc, scale, stream)
               : launch_rows_v<E, false>(x, rows, d, ldx, codes, ldc, scale, stream);
}

}  // namespace

int launch_quantize_rows(Dtype t, const void* X, int64_t rows, int d, int64_t ldx, int8_t* codes, int64_t ldc,
                         float* scale, bool vec, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_rows_e<QF32>(X, rows, d, ldx, codes, ldc, scale, vec, stream);
        case Dtype::fp16: return launch_rows_e<QF16>(X, rows, d, ldx, codes, ldc, scale, vec, stream);
        default: return launch_rows_e<QB16>(X, rows, d, ldx, codes, ldc, scale, vec, stream);
    }
}

int launch_int8_tokens(Dtype t, const Int8Product& p, const void* X, int64_t ldX, bool vec, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_tokens_e<QF32>(p, X, ldX, vec, stream);
        case Dtype::fp16: return launch_tokens_e<QF16>(p, X, ldX, vec, stream);
        default: return launch_tokens_e<QB16>(p, X, ldX, vec, stream);
    }
}

int launch_int8_product(Dtype t, const Int8Product& p, bool aligned, void* workspace, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_product_e<QF32>(p, aligned, workspace, stream);
        case Dtype::fp16: return launch_product_e<QF16>(p, aligned, workspace, stream);
        default: return launch_product_e<QB16>(p, aligned, workspace, stream);
    }
}

}  // namespace kbit
