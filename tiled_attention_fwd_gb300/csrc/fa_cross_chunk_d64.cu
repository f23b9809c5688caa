// Cross attention of longer sequences (and the joining of parts), head dimension 64.
#include "fa_paged_chunk.cuh"

namespace fa {
template int launch_paged_chunk<64, true>(const PagedFwdArgs& a, const LaunchCtx& ctx);
template int launch_paged_join<64, true>(const PagedFwdArgs& a, bool chunks, const LaunchCtx& ctx);
}
