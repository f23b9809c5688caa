// Paged attention of few rows, head dimension 32.
#include "fa_paged_few.cuh"

namespace fa {
template int launch_paged_few<32>(const PagedFwdArgs& a, bool behind_chunks, const LaunchCtx& ctx);
}
