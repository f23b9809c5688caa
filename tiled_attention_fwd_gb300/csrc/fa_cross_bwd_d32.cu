// Gradients of cross attention, head dimension 32.
#include "fa_cross_bwd_short.cuh"

namespace fa {
int launch_cross_bwd_d32(const CrossArgs& a, const LaunchCtx& ctx) { return launch_cross_bwd<32>(a, ctx); }
size_t cross_bwd_ws_bytes_d32(int B, int rows, int heads, int group) { return cross_bwd_ws<32>(nullptr, B, rows, heads, group, nullptr); }
}
