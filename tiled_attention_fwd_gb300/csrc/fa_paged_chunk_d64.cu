// Paged attention of chunks and prompts, head dimension 64.
#include "fa_paged_chunk.cuh"

namespace fa {
template int launch_paged_chunk<64>(const PagedFwdArgs& a, const LaunchCtx& ctx);
}
