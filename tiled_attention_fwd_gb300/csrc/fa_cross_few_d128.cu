// Cross attention of few rows, head dimension 128.
#include "fa_paged_few.cuh"

namespace fa {
template int launch_paged_few<128, true>(const PagedFwdArgs& a, bool behind_chunks, const LaunchCtx& ctx);
}
