// Internal launcher interface of the operators around a quantized layer
// (include/kbit_layer.h), between layer_api.cpp and the HIP translation
// units.  No HIP types cross this boundary; arguments are already validated.
#pragma once

#include <stdint.h>

#include "kbit_internal.h"

namespace kbit {

// Largest head the passes over heads take: 64 lanes of 16 elements.
constexpr int kMaxHeadDim = 1024;

// Largest depth of the int8 product: |sum of K products| <= 2^14 K < 2^31.
constexpr int kMaxInt8Depth = 131071;

enum class HeadsKind : int { rope, norm, append };

// One set of heads of a pass.  Strides in elements; for the append out_b,
// out_s and out_h are the cache's page, in-page and head strides.
struct HeadSet {
    const void* in;
    void* out;
    const void* weight;
    int64_t in_b, in_s, in_h, out_b, out_s, out_h;
    int heads, dim, rot;
    int units;  // lane groups per token, set by the launcher
};

struct HeadsArgs {
    HeadSet set[2];  // the second may have no heads
    const void* positions;
    const float* table;
    const void* slots;
    int64_t tokens, max_pos, n_slots;
    int page_size;
    int log2_lanes;  // lanes a row in the vector form
    float sign, eps, inv_dim;
    bool positions_wide, slots_wide, weight_fp32;
    uint32_t units;      // set by the launcher
    bool tokens_first;   // set by the launcher
};

int launch_heads(Dtype t, HeadsArgs& p, int64_t batch, HeadsKind kind, int layout, bool vec, void* stream);

struct BackSet {
    const void *x, *g, *weight;
    void* dx;
    int64_t x_b, x_s, x_h, g_b, g_s, g_h, dx_b, dx_s, dx_h;
    int heads;
    uint32_t rows;  // batch * tokens * heads
};

// Workgroups of the gradient pass, each with one partial row of D sums: four a
// compute unit of 256, as many as its registers let run at once (8192 tokens,
// 40 heads of 128: 512 / 1024 / 1280 / 2048 workgroups 59 / 51 / 59 / 58 us).
constexpr int kNormBackGroups = 1024;

struct NormBackArgs {
    BackSet set[2];
    const void* positions;
    const float* table;
    float* partial;    // [(kNormBackGroups + 2) * dim]
    float* direct[2];  // set by the launcher: where a lone workgroup's sums are the result
    int64_t max_pos;
    int64_t tokens;
    int dim, rot, log2_lanes;
    int first_groups;  // set by the launcher
    float eps, inv_dim;
    bool positions_wide, weight_fp32;
};

int launch_norm_back(Dtype t, NormBackArgs& p, int layout, bool vec, float* d0, float* d1, void* stream);

int launch_rope_table(const double* freq, int rot, int64_t max_pos, double amplitude, float* table, void* stream);

// Rows to int8 codes with one scale each; vec: 16-byte loads are possible.
int launch_quantize_rows(Dtype t, const void* X, int64_t rows, int d, int64_t ldx, int8_t* codes, int64_t ldc,
                         float* scale, bool vec, void* stream);

struct Int8Product {
    const int8_t* x;
    const float* xs;
    const int8_t* w;
    const float* ws;
    const void* bias;
    void* out;
    int64_t M, ldx, ldw, ldo;
    int N, K;
};

// aligned: both operands' rows start at multiples of 16 bytes.  workspace: of
// int8_product_workspace bytes on the current device, 16-byte aligned.
int launch_int8_product(Dtype t, const Int8Product& p, bool aligned, void* workspace, void* stream);

// A few tokens quantized inside the product's kernel, where int8_tokens_fit
// (the weights' rows start at multiples of 16 bytes; p.x and p.xs are not
// looked at).
int launch_int8_tokens(Dtype t, const Int8Product& p, const void* X, int64_t ldX, bool vec, void* stream);

}  // namespace kbit
