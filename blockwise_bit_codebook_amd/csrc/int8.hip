// 8-bit integer linear layer for gfx950: rows to int8 codes with one scale
// each, and the product of two coded matrices with the scales in its
// epilogue.
//
//   codes    amax = max |x| over the row, scale = RN(amax / 127),
//            q = rint(RN(x * RN(127 / amax))), half to even; |q| <= 127.
//            A row below 2^-100 throughout (127 / amax would leave the fp32
//            range) gets scale 0 and codes 0; a row with a NaN or an
//            infinity gets scale NaN and codes 0, so that its outputs are NaN.
//   product  acc[m][n] = sum over k of x[m][k] * w[n][k], exact in int32,
//            out = RN_T(RN(RN(RN(acc) * xs[m]) * ws[n]) + bias[n]).
#include "device.h"
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
    static __device__ void widen(const u32x4* r, float (&x)[8]) { Fp16::unpack(r, x); }
};
struct QB16 {
    using T = uint16_t;
    static constexpr int kVec = 1;
    static __device__ float one(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
    static __device__ T narrow(float v) { return static_cast<T>(pack_bf16x2(v, 0.0f) & 0xFFFFu); }
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

// The row's scale and 127 / amax from the bits of its largest magnitude
// (ordered like the magnitudes, with NaN above infinity above the rest).
__device__ __forceinline__ void row_scale(uint32_t amax_bits, float& scale, float& inv) {
    const float amax = __uint_as_float(amax_bits);
    scale = amax / 127.0f;
    inv = 127.0f / amax;
    if (amax_bits < 0x0D800000u) scale = inv = 0.0f;  // below 2^-100
    if (amax_bits >= 0x7F800000u) {
        scale = __uint_as_float(0x7FC00000u);
        inv = 0.0f;
    }
}

// One row a workgroup; the first kKeep pieces of each thread stay in
// registers between the two steps, longer rows are read a second time (from
// cache).  In a row that is not finite inv is 0 and inf * 0 must not become
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
// 16 codes of a row from column k (zeros beyond K and outside the matrix).
template <bool ALIGNED>
__device__ __forceinline__ u32x4 load_codes(const int8_t* row, bool live, int k, int K) {
    u32x4 r = u32x4{0u, 0u, 0u, 0u};
    if (!live || k >= K) return r;
    if (ALIGNED && k + 16 <= K) return load16<false>(row + k);
    const int n = min(16, K - k);
    for (int i = 0; i < n; ++i) r[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + i])) << (8 * (i & 3));
    return r;
}

template <class E>
__device__ __forceinline__ void store_out(const Int8Product& p, int64_t m, int n, int acc) {
    float v = static_cast<float>(acc) * p.xs[m];
    v = v * p.ws[n];
    if (p.bias) v = v + E::one(static_cast<const typename E::T*>(p.bias)[n]);
    static_cast<typename E::T*>(p.out)[m * p.ldo + n] = E::narrow(v);
}

// Any shape and alignment: a 64 x 64 tile a workgroup, four waves of 32 x 32,
// 64 codes deep a step through LDS (rows 80 bytes apart, so that the 16 rows
// of a fragment start in different banks).
constexpr int kGenTile = 64, kGenStep = 64, kGenPitch = 80;
template <class E, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void int8_generic_kernel(const Int8Product p) {
    __shared__ __align__(16) uint8_t lds[2][kGenTile * kGenPitch];
    const int lane = __lane_id(), wave = threadIdx.x / kWave;
    const int l16 = lane & 15, q = lane >> 4;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kGenTile;
    const int n0 = blockIdx.x * kGenTile;
    const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
    const int row = threadIdx.x >> 2, piece = (threadIdx.x & 3) * 16;
    const bool x_ok = m0 + row < p.M, w_ok = n0 + row < p.N;
    const int8_t* xr = p.x + (m0 + row) * p.ldx;
    const int8_t* wr = p.w + static_cast<int64_t>(n0 + row) * p.ldw;
    i32x4 acc[2][2] = {};
    for (int k = 0; k < p.K; k += kGenStep) {
        const u32x4 xv = load_codes<ALIGNED>(xr, x_ok, k + piece, p.K);
        const u32x4 wv = load_codes<ALIGNED>(wr, w_ok, k + piece, p.K);
        __syncthreads();
        *reinterpret_cast<u32x4*>(&lds[0][row * kGenPitch + piece]) = xv;
        *reinterpret_cast<u32x4*>(&lds[1][row * kGenPitch + piece]) = wv;
        __syncthreads();
        i32x4 a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = *reinterpret_cast<const i32x4*>(&lds[0][(wm + 16 * i + l16) * kGenPitch + 16 * q]);
            b[i] = *reinterpret_cast<const i32x4*>(&lds[1][(wn + 16 * i + l16) * kGenPitch + 16 * q]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    // lane l holds rows 4q + r, column l % 16 of each 16 x 16 block
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t m = m0 + wm + 16 * i + 4 * q + r;
                const int n = n0 + wn + 16 * j + l16;
                if (m < p.M && n < p.N) store_out<E>(p, m, n, acc[i][j][r]);
            }
}

template <class E>
int launch_product_e(const Int8Product& p, bool aligned, void* stream) {
    const dim3 grid((p.N + kGenTile - 1) / kGenTile, static_cast<unsigned>((p.M + kGenTile - 1) / kGenTile));
    if (aligned)
        hipLaunchKernelGGL((int8_generic_kernel<E, true>), grid, dim3(kThreads), 0, static_cast<hipStream_t>(stream),
                           p);
    else
        hipLaunchKernelGGL((int8_generic_kernel<E, false>), grid, dim3(kThreads), 0, static_cast<hipStream_t>(stream),
                           p);
    return static_cast<int>(hipGetLastError());
}

template <class E>
int launch_rows_e(const void* X, int64_t rows, int d, int64_t ldx, int8_t* codes, int64_t ldc, float* scale, bool vec,
                  void* stream) {
    const unsigned grid = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
    const auto* x = static_cast<const typename E::T*>(X);
    if (vec)
        hipLaunchKernelGGL((quantize_rows_kernel<E, true>), dim3(grid), dim3(kThreads), 0,
                           static_cast<hipStream_t>(stream), x, rows, d, ldx, codes, ldc, scale);
    else
        hipLaunchKernelGGL((quantize_rows_kernel<E, false>), dim3(grid), dim3(kThreads), 0,
                           static_cast<hipStream_t>(stream), x, rows, d, ldx, codes, ldc, scale);
    return static_cast<int>(hipGetLastError());
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

int64_t int8_product_workspace(int64_t, int, int) { return 0; }

int launch_int8_product(Dtype t, const Int8Product& p, bool aligned, void*, void* stream) {
    switch (t) {
        case Dtype::fp32: return launch_product_e<QF32>(p, aligned, stream);
        case Dtype::fp16: return launch_product_e<QF16>(p, aligned, stream);
        default: return launch_product_e<QB16>(p, aligned, stream);
    }
}

}  // namespace kbit
