// Stands in for the HIP launchers behind csrc/layer_api.cpp: each records what
// it was given, so that a test sees on the host which way an entry point sends
// a call.  Nothing is dereferenced.
#include "int8_choice.h"
#include "layer_internal.h"

namespace kbit {
namespace {
Int8Product product;
int product_launches = 0, product_on_fast_path = -1;
}  // namespace

int device_cu_count() { return 256; }
bool device_usable() { return true; }

int launch_heads(Dtype, HeadsArgs&, int64_t, HeadsKind, int, bool, void*) { return 0; }
int launch_norm_back(Dtype, NormBackArgs&, int, bool, float*, float*, void*) { return 0; }
int launch_rope_table(const double*, int, int64_t, double, float*, void*) { return 0; }
int launch_quantize_rows(Dtype, const void*, int64_t, int, int64_t, int8_t*, int64_t, float*, bool, void*) { return 0; }
int launch_int8_product(Dtype, const Int8Product& p, bool aligned, void*, void*) {
    product = p;
    product_on_fast_path = aligned;
    ++product_launches;
    return 0;
}
int launch_int8_tokens(Dtype, const Int8Product&, const void*, int64_t, bool, void*) { return 0; }
}  // namespace kbit

extern "C" {
int stub_product_launches() { return kbit::product_launches; }
int stub_product_on_fast_path() { return kbit::product_on_fast_path; }

// What one product needs, in bytes.
int64_t stub_product_workspace(int64_t M, int N, int K) { return kbit::int8_product_workspace(M, N, K); }

// The form of a product on `cus` compute units: rows of the tile, or 0 and the
// pieces of few rows in 16 x 16; parts of the depth.
void stub_form(int64_t M, int N, int K, int64_t cus, int* bm, int* mt, int* tn, int* parts) {
    const kbit::Int8Choice c = kbit::choose_form(M, N, K, cus);
    *bm = c.bm;
    *mt = c.few.mt;
    *tn = c.few.tn;
    *parts = c.parts;
}
}
