// Stands in for the HIP launchers behind csrc/mx_api.cpp: each records which
// bytes of the workspace it would write, so that a test sees on the host that
// the parts of a call lie inside it and apart.  Nothing is dereferenced.
#include <vector>

#include "mx_internal.h"

namespace kbit {
namespace {
struct Range {
    int64_t at, bytes;
};
std::vector<Range> written;

int64_t address(const void* p) { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)); }
void codes(const MxCoded& c, int64_t rows, int64_t d) {
    if (!c.codes) return;
    written.push_back({address(c.codes), rows * c.ldc});
    written.push_back({address(c.scales), c.paired ? (mx_blocks(d) + 15) / 16 * c.lds : rows * c.lds});
}
}  // namespace

int device_cu_count() { return 256; }
bool device_usable() { return true; }

int launch_mx_quantize(Dtype, const void*, int64_t rows, int d, int64_t, const MxCoded& c, void*) {
    return codes(c, rows, d), 0;
}
int launch_mx_quantize_columns(Dtype, const MxColumns* jobs, int count, void*) {
    for (int i = 0; i < count; ++i) {
        codes(jobs[i].columns, jobs[i].cols, jobs[i].rows);
        codes(jobs[i].by_rows, jobs[i].rows, jobs[i].cols);
        if (jobs[i].sums) written.push_back({address(jobs[i].sums), 4 * mx_sum_groups(jobs[i].rows) * jobs[i].cols});
    }
    return 0;
}
int launch_mx_add_sums(const float*, int64_t, int, float*, void*) { return 0; }
int launch_mx_zero(float*, int64_t, int, int64_t, void*) { return 0; }
int launch_mx_dequantize(Dtype, const uint8_t*, int64_t, const uint8_t*, int64_t, int64_t, int, void*, int64_t, void*) { return 0; }
int launch_mx_product(Dtype, const MxProduct& p, void* workspace, void*) {
    const int64_t need = mx_product_workspace(p.M, p.N, p.K, p.x_paired, p.w_paired);
    if (need > 0) written.push_back({address(workspace), need});
    return 0;
}
int launch_mx_tokens(Dtype, const MxProduct&, int, const void*, int64_t, void*) { return 0; }
int launch_layer_norm(Dtype, const LayerNormArgs&, void*) { return 0; }
int launch_layer_norm_back(Dtype, const LayerNormBackArgs&, void*) { return 0; }
}  // namespace kbit

extern "C" {
// The ranges written since the last call: address, bytes; at most `most` of them.
int space_written(int64_t* to, int most) {
    int n = 0;
    for (const kbit::Range& r : kbit::written)
        if (n < most) to[2 * n] = r.at, to[2 * n + 1] = r.bytes, ++n;
    kbit::written.clear();
    return n;
}
// What one call's backward pass needs for the gradients that are set.
int64_t space_back(int64_t M, int N, int K, int dX, int dW, int db) {
    return kbit::mx_back_workspace(M, N, K, dX != 0, dW != 0, db != 0);
}
}
