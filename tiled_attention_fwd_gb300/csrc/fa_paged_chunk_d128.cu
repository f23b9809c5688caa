// Paged attention of chunks and prompts, head dimension 128.
#include "fa_paged_chunk.cuh"

namespace fa {
template int launch_paged_chunk<128>(const PagedFwdArgs& a, const LaunchCtx& ctx);
}
