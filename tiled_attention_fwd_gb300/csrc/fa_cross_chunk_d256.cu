// Cross attention of longer sequences (and the joining of parts), head dimension 256.
#include "fa_paged_chunk.cuh"

namespace fa {
template int launch_paged_chunk<256, true>(const PagedFwdArgs& a, const LaunchCtx& ctx);
template int launch_paged_join<256, true>(const PagedFwdArgs& a, bool chunks, const LaunchCtx& ctx);
}
