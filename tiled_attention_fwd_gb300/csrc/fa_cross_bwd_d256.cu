// Gradients of cross attention, head dimension 256.
#include "fa_cross_bwd_short.cuh"

namespace fa {
int launch_cross_bwd_d256(const CrossArgs& a, const LaunchCtx& ctx) { return launch_cross_bwd<256>(a, ctx); }
size_t cross_bwd_ws_bytes_d256(int B, int rows, int heads, int group) { return cross_bwd_ws<256>(nullptr, B, rows, heads, group, nullptr); }
}
