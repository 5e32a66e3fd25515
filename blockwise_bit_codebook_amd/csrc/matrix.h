// What the kernels over rows and the matrix products share: element types,
// pieces of rows, operands on their way to LDS.
#pragma once

#include "device.h"

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

// 16 and 8 bytes at any address of an element: the memory unit takes them.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
__device__ __forceinline__ u32x4 load16_any(const void* p) { return *reinterpret_cast<const u32x4_any*>(p); }
__device__ __forceinline__ void store16_any(void* p, const u32x4& v) { *reinterpret_cast<u32x4_any*>(p) = v; }

// 8 elements of a row from column c at any alignment, as they stand, 0 beyond d.
template <class E>
__device__ __forceinline__ void load8_raw(const typename E::T* row, int c, int d, u32x4 (&r)[E::kVec]) {
    if (c + 8 <= d) {
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) r[i] = load16_any(row + c + 4 * i);
    } else {
        // the last element stands in for those past it: eight loads without a
        // branch between them, on their way together
        typename E::T v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = row[min(c + e, d - 1)];
        uint32_t w[4 * E::kVec];
#pragma unroll
        for (int i = 0; i < 4 * E::kVec; ++i) {
            if constexpr (sizeof(typename E::T) == 4) {
                w[i] = c + i < d ? __float_as_uint(v[i]) : 0u;
            } else {
                w[i] = c + 2 * i < d ? v[2 * i] : 0u;
                if (c + 2 * i + 1 < d) w[i] |= static_cast<uint32_t>(v[2 * i + 1]) << 16;
            }
        }
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) r[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    }
}

// 8 values to a row from column c at any alignment, none beyond d.
template <class E>
__device__ __forceinline__ void store8(typename E::T* row, int c, int d, const float (&v)[8]) {
    if (c + 8 <= d) {
        if constexpr (sizeof(typename E::T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; i += 4)
                store16_any(row + c + i, u32x4{__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                                               __float_as_uint(v[i + 3])});
        } else {
            store16_any(row + c, u32x4{E::pack(v[0], v[1]), E::pack(v[2], v[3]), E::pack(v[4], v[5]), E::pack(v[6], v[7])});
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < d) row[c + e] = E::narrow(v[e]);
    }
}

// A barrier that waits for the wave's LDS accesses but not for its loads, as
// __syncthreads would.  The fences emit nothing and hold the compiler to the order:
// the wait counts as touching no memory, so that without the one before it an
// access might come to stand between wait and barrier.
__device__ __forceinline__ void barrier_in_flight() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// ---------------------------------------------------------------------------
// operands in LDS
// ---------------------------------------------------------------------------
// A step of an operand's row is 128 bytes in LDS, the 16-byte pieces of which
// stand at positions xor-ed with a key of the row (key_x, key_w), so that the 8
// rows which a read touches at a time lie in different banks.  The weight is
// the first matrix operand, so that lane l holds channels 4 (l / 16) .. + 3 of
// row l % 16; channel 4 TN (i / 4) + 4 j + i % 4 sits in row i of operand j,
// which makes a lane's 4 TN channels neighbours.
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

}  // namespace
}  // namespace kbit
