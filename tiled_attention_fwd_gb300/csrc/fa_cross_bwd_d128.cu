// Gradients of cross attention, head dimension 128.
#include "fa_cross_bwd_short.cuh"

namespace fa {
int launch_cross_bwd_d128(const CrossArgs& a, const LaunchCtx& ctx) { return launch_cross_bwd<128>(a, ctx); }
size_t cross_bwd_ws_bytes_d128(int B, int rows, int heads, int group) { return cross_bwd_ws<128>(nullptr, B, rows, heads, group, nullptr); }
}
