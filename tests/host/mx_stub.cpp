// Stands in for the HIP launchers behind csrc/mx_api.cpp: each counts its calls
// and products record what they were given, so that a test sees on the host what
// an entry point would launch.  Nothing is dereferenced.
#include "mx_internal.h"

namespace kbit {
namespace {
int launches = 0, products = 0, tokens = 0, row_passes = 0, column_passes = 0;
MxProduct product;
}  // namespace

int device_cu_count() { return 256; }
bool device_usable() { return true; }

int launch_mx_quantize(Dtype, const void*, int64_t, int, int64_t, const MxCoded&, void*) {
    ++row_passes;
    return ++launches, 0;
}
int launch_mx_quantize_columns(Dtype, const MxColumns*, int count, void*) {
    column_passes += count;
    return launches += count > 0, 0;
}
int launch_mx_add_sums(const float*, int64_t, int, float*, void*) { return ++launches, 0; }
int launch_mx_zero(float*, int64_t, int, int64_t, void*) { return ++launches, 0; }
int launch_mx_dequantize(Dtype, const uint8_t*, int64_t, const uint8_t*, int64_t, int64_t, int, void*, int64_t, void*) {
    return ++launches, 0;
}
int launch_mx_product(Dtype, const MxProduct& p, void*, void*) {
    product = p;
    ++products;
    return ++launches, 0;
}
int launch_mx_tokens(Dtype, const MxProduct&, int, const void*, int64_t, void*) {
    ++tokens;
    return ++launches, 0;
}
int launch_layer_norm(Dtype, const LayerNormArgs&, void*) { return ++launches, 0; }
int launch_layer_norm_back(Dtype, const LayerNormBackArgs&, void*) { return ++launches, 0; }
}  // namespace kbit

extern "C" {
// Launches so far: all, products, of tokens, over rows; matrices over columns.
void stub_counts(int* to) {
    to[0] = kbit::launches;
    to[1] = kbit::products;
    to[2] = kbit::tokens;
    to[3] = kbit::row_passes;
    to[4] = kbit::column_passes;
}
int stub_paired() { return kbit::product.x_paired + 2 * kbit::product.w_paired; }

// What one product of depth K needs, in bytes.
int64_t stub_mx_workspace(int64_t M, int N, int K) { return kbit::mx_product_workspace(M, N, kbit::mx_depth(K)); }

// Its form on `cus` compute units: rows of the tile, or 0 and the pieces of few
// rows in 16 x 16; parts of the depth.
void stub_mx_form(int64_t M, int N, int K, int64_t cus, int* to) {
    const kbit::Int8Choice c = kbit::mx_choose(M, N, kbit::mx_depth(K), cus);
    to[0] = c.bm;
    to[1] = c.few.mt;
    to[2] = c.few.tn;
    to[3] = c.parts;
}
}
