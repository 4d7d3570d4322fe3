// The stand-in for the device of quant_host.cpp, with the launches of the window decodes and of the
// table builder, which keep their parameters.
#include "quant_host.cpp"

namespace {
oxd::WindowParams window_params;
oxd::TablesParams tables_params;
}  // namespace

extern "C" {
const void* fake_window(void) { return &window_params; }
int fake_window_scale_sign(void) { return window_params.scale_log2 > 0 ? 1 : -1; }
int fake_window_shape(int i) {
    const int v[] = {window_params.batch, window_params.num_qo_heads, window_params.num_kv_heads,
                     window_params.group, window_params.page_shift, window_params.layout,
                     window_params.num_indices, window_params.window, window_params.sinks};
    return v[i];
}
int fake_tables_shape(int i) {
    const int v[] = {tables_params.batch, tables_params.page_shift, tables_params.row_pages,
                     tables_params.num_indices, tables_params.num_tokens, tables_params.num_free,
                     tables_params.window, tables_params.sinks,
                     tables_params.token_request != nullptr, tables_params.slots != nullptr};
    return v[i];
}
}

namespace oxd {
cudaError_t launch_window_decode(WindowParams p, int, cudaStream_t, bool) {
    window_params = p;
    ++launches;
    return cudaSuccess;
}
cudaError_t launch_window_quant(WindowParams p, int, cudaStream_t, bool) {
    window_params = p;
    ++launches;
    return cudaSuccess;
}
cudaError_t launch_build_tables(const TablesParams& p, cudaStream_t) {
    tables_params = p;
    ++launches;
    return cudaSuccess;
}
}  // namespace oxd
