// Tables of the paged cache, built on the device: fa_paged_extend and
// fa_paged_release (declared in include/fa_gb300.h).
//
// Both are sums over the sequences in order (pages needed, rows, pages given
// back) with a little work for each page and row, and cost what a launch and
// a few dependent memory round trips cost.  So each is one launch of one thread-block cluster:
// every CTA makes the sums for itself (they are short), the cluster's barrier
// stands between reading the old lengths and writing the new ones, and the
// CTAs share out pages and rows.  No atomics on results: the order is fixed.
#include <atomic>
#include <cstdint>

#include "../../include/fa_gb300.h"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kTableThreads = 1024;
constexpr int kTableWarps = kTableThreads / 32;
constexpr int kTableCtas = 16;  // of the cluster where the device takes one of that many, else half of them

__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Store a word to another CTA's shared memory (a shared::cluster address).
__device__ __forceinline__ void st_cluster(uint32_t addr, int x) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

// Inclusive sums over the CTA's threads, N values at a time, and the sums of all.
template <int N>
__device__ __forceinline__ void block_scan(long long (&x)[N], long long (&sum)[N], long long (*s)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto warp_scan = [&](long long v) {
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, k);
      if (lane >= k) v += y;
    }
    return v;
  };
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = warp_scan(x[i]);
    if (lane == 31) s[i][warp] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long y = warp_scan(s[i][lane]);
    const long long before = __shfl_sync(0xffffffffu, y, warp > 0 ? warp - 1 : 0);
    sum[i] = __shfl_sync(0xffffffffu, y, 31);
    if (warp > 0) x[i] += before;
  }
  __syncthreads();
}

struct TableArgs {
  int* free_pages;
  int* free_count;
  int num_pages;
  int ps_log2;
  int* table;
  long long stride;
  int max_pages;
  int* lens;
  int B;
  int* status;
  // fa_paged_extend
  const int* new_rows;
  int* cu_rows;
  long long* slots;
  int* positions;
  int rows;
  // fa_paged_release
  const uint8_t* done;
  int parts_log2;  // a sequence's entries are shared out to 2^parts_log2 warps
};

__device__ __forceinline__ int pages_of(long long tokens, int ps_log2) {
  return static_cast<int>((tokens + (1 << ps_log2) - 1) >> ps_log2);
}

// Pages on the stack, cut to what it can hold.
__device__ __forceinline__ int free_count(const TableArgs& a, bool& bad) {
  const int n = *a.free_count;
  bad = bad || n < 0 || n > a.num_pages;
  return min(max(n, 0), a.num_pages);
}

__global__ void __launch_bounds__(kTableThreads, 1) fa_paged_extend_kernel(const TableArgs a) {
  __shared__ long long s_scan[2][32];
  // Of the 1024 sequences at hand: first new row, length before, and where on the stack its new pages begin (from the top).
  __shared__ int s_row[kTableThreads + 1];
  __shared__ int s_old[kTableThreads];
  __shared__ int s_top[kTableThreads];
  __shared__ int s_taken;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_ctas());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad = false, none_left = false;
  const int free = free_count(a, bad);
  if (threadIdx.x == 0) s_taken = 0;
  auto page_at = [&](int from_top) -> int {
    const int page = a.free_pages[free - 1 - from_top];
    return page >= 0 && page < a.num_pages ? page : -1;
  };
  long long need0 = 0, rows0 = 0, cu0 = 0;  // of the sequences before these 1024
  for (int b0 = 0; b0 < a.B; b0 += kTableThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const bool in = b < a.B;
    const int old = in ? a.lens[b] : 0, n = in ? a.new_rows[b] : 0;
    const long long want = static_cast<long long>(old) + n;
    const bool fits = in && old >= 0 && n >= 0 && want <= static_cast<long long>(a.max_pages) << a.ps_log2;
    const int need = fits ? pages_of(want, a.ps_log2) - pages_of(old, a.ps_log2) : 0;
    long long x[2] = {need, fits ? n : 0}, sum[2];
    block_scan(x, sum, s_scan);
    const bool room = rows0 + x[1] <= a.rows, pages = need == 0 || need0 + x[0] <= free;
    const bool served = fits && room && pages;
    bad = bad || (in && !fits) || (fits && n > 0 && !room);
    none_left = none_left || (fits && room && !pages);
    // Those served that need pages are the first of those that fit: the sums over these are where their pages begin.
    if (served && need > 0) atomicMax(&s_taken, static_cast<int>(need0 + x[0]));
    long long r[1] = {served ? n : 0}, rsum[1];
    block_scan(r, rsum, s_scan);
    const int row = static_cast<int>(cu0 + r[0] - (served ? n : 0));
    s_row[threadIdx.x] = row;
    s_old[threadIdx.x] = old;
    s_top[threadIdx.x] = static_cast<int>(min(need0 + x[0] - need, static_cast<long long>(a.num_pages)));  // (those not served: behind all)
    if (threadIdx.x == kTableThreads - 1) s_row[kTableThreads] = static_cast<int>(cu0 + rsum[0]);
    const long long need_first = need0;
    need0 += sum[0];
    rows0 += sum[1];
    cu0 += rsum[0];
    cluster_sync_all();  // every CTA has read these lengths
    if (rank == 0 && in) {
      a.cu_rows[b] = row;
      if (served && n > 0) a.lens[b] = static_cast<int>(want);
    }
    // New pages into the table, one a thread: the served sequences' needs lie one behind another from the top of the stack on.
    const long long pages_end = min(need0, static_cast<long long>(s_taken));
    for (long long t = need_first + rank * kTableThreads + threadIdx.x; t < pages_end; t += ctas * kTableThreads) {
      int i = 0;  // the sequence that takes it: the last one whose pages begin there or before
#pragma unroll
      for (int step = kTableThreads / 2; step > 0; step >>= 1)
        if (s_top[i + step] <= t) i += step;
      const int page = page_at(static_cast<int>(t));
      bad = bad || page < 0;
      a.table[static_cast<long long>(b0 + i) * a.stride + pages_of(s_old[i], a.ps_log2) + (static_cast<int>(t) - s_top[i])] = page;
    }
    // Slots and positions, four rows a thread (both arrays are 16-byte aligned, so a group of four is stored whole).
    const int first = s_row[0], last = s_row[kTableThreads];
    const long long at0 = (first & ~3) + 4ll * (rank * kTableThreads + static_cast<int>(threadIdx.x));
    for (long long at = at0; at < last; at += 4ll * ctas * kTableThreads) {
      const int t0 = static_cast<int>(at), from = max(t0, first);
      // The sequence that holds row `from`: the last one that begins there or before.
      int i = 0;
#pragma unroll
      for (int step = kTableThreads / 2; step > 0; step >>= 1)
        if (s_row[i + step] <= from) i += step;
      long long slot[4];
      int pos[4];
      const int mask = (1 << a.ps_log2) - 1;
      // The page of position x of sequence i, -1 where it is none of the cache's.
      auto page_of = [&](int x) -> int {
        const int k = x >> a.ps_log2, held = pages_of(s_old[i], a.ps_log2);
        int page = k < held ? a.table[static_cast<long long>(b0 + i) * a.stride + k] : page_at(s_top[i] + k - held);
        page = page < a.num_pages ? page : -1;
        bad = bad || page < 0;
        return page;
      };
      int k_last = -1, i_last = -1, page = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + e;
        slot[e] = -1;
        pos[e] = 0;
        if (t < first || t >= last) continue;
        while (t >= s_row[i + 1]) ++i;
        pos[e] = s_old[i] + (t - s_row[i]);
        const int k = pos[e] >> a.ps_log2;
        if (k != k_last || i != i_last) {
          page = page_of(pos[e]);
          k_last = k;
          i_last = i;
        }
        if (page >= 0)
          slot[e] = (static_cast<long long>(page) << a.ps_log2) + (pos[e] & mask);
      }
      if (t0 >= first && t0 + 4 <= last) {
        if (a.slots) {
          reinterpret_cast<longlong2*>(a.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
          reinterpret_cast<longlong2*>(a.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
        }
        if (a.positions) *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t0 + e >= first && t0 + e < last) {
            if (a.slots) a.slots[t0 + e] = slot[e];
            if (a.positions) a.positions[t0 + e] = pos[e];
          }
      }
    }
  }
  // (s_taken is complete: barriers of the scans lie behind the last atomicMax.)
  if (rank == 0 && threadIdx.x == 0) {
    a.cu_rows[a.B] = static_cast<int>(cu0);
    *a.free_count = free - s_taken;
  }
  if (bad) atomicOr(a.status, kBadBatchBit);
  if (none_left) atomicOr(a.status, kNoPagesBit);
}

__global__ void __launch_bounds__(kTableThreads, 1) fa_paged_release_kernel(const TableArgs a) {
  __shared__ long long s_scan[1][32];
  // Of the 1024 parts of sequences at hand: pages to give back, and where on the stack they go.
  __shared__ int s_count[kTableThreads];
  __shared__ int s_at[kTableThreads];
  // Of this CTA's own parts: their entries.
  __shared__ int2 s_part[kTableThreads];
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_ctas());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad = false;
  // A CTA's shared memory may be written by another one when it has started: all arrive here and wait before their first such store.
  cluster_arrive();
  bool all_started = false;
  const int free = free_count(a, bad);
  const long long units = static_cast<long long>(a.B) << a.parts_log2;
  auto valid = [&](int page) { return page >= 0 && page < a.num_pages; };
  long long base = free;
  for (long long u0 = 0; u0 < units; u0 += kTableThreads) {
    // (A warp's parts together, so that their loads are on their way together.)
    constexpr int PARTS = kTableThreads / (kTableCtas * kTableWarps);
    for (int i0 = rank * kTableWarps + warp; i0 < kTableThreads; i0 += PARTS * ctas * kTableWarps) {
      bool on[PARTS];
      int2 part[PARTS];
      int count[PARTS];
      long long len[PARTS];
#pragma unroll
      for (int e = 0; e < PARTS; ++e) {
        const long long u = u0 + i0 + e * ctas * kTableWarps;
        on[e] = u < units && a.done[u >> a.parts_log2];
        len[e] = u < units ? a.lens[u >> a.parts_log2] : 0;
      }
#pragma unroll
      for (int e = 0; e < PARTS; ++e) {
        const long long u = u0 + i0 + e * ctas * kTableWarps;
        const int p = static_cast<int>(u) & ((1 << a.parts_log2) - 1);
        const long long most = static_cast<long long>(a.max_pages) << a.ps_log2;
        bad = bad || (on[e] && (len[e] < 0 || len[e] > most));
        const int held = on[e] ? pages_of(min(max(len[e], 0ll), most), a.ps_log2) : 0;
        const int each = (held + (1 << a.parts_log2) - 1) >> a.parts_log2;
        part[e] = make_int2(min(p * each, held), min((p + 1) * each, held));
        const int* from = a.table + (u >> a.parts_log2) * a.stride;
        int mine = 0;
#pragma unroll 8
        for (int k = part[e].x + lane; k < part[e].y; k += 32) mine += valid(from[k]) ? 1 : 0;
        count[e] = __reduce_add_sync(0xffffffffu, mine);
        bad = bad || count[e] != part[e].y - part[e].x;
      }
      if (!all_started) cluster_wait();
      all_started = true;
#pragma unroll
      for (int e = 0; e < PARTS; ++e) {
        const int i = i0 + e * ctas * kTableWarps;
        if (lane == 0) s_part[i] = part[e];
        if (lane < ctas) st_cluster(mapa_shared(smem_u32(&s_count[i]), lane), count[e]);
      }
    }
    cluster_sync_all();
    long long x[1] = {s_count[threadIdx.x]}, sum[1];
    const long long mine = x[0];
    block_scan(x, sum, s_scan);
    s_at[threadIdx.x] = static_cast<int>(min(base + x[0] - mine, static_cast<long long>(a.num_pages)));
    base += sum[0];
    __syncthreads();
    for (int i = rank * kTableWarps + warp; i < kTableThreads && u0 + i < units; i += ctas * kTableWarps) {
      const int b = static_cast<int>((u0 + i) >> a.parts_log2);
      if (!a.done[b]) continue;
      int* from = a.table + b * a.stride;
      int at = s_at[i];
      const int2 part = s_part[i];
#pragma unroll 4
      for (int k0 = part.x; k0 < part.y; k0 += 32) {
        const int k = k0 + lane;
        const int page = k < part.y ? from[k] : -1;
        const uint32_t have = __ballot_sync(0xffffffffu, valid(page));
        const int to = at + __popc(have & ((1u << lane) - 1));
        if (valid(page)) {
          if (to < a.num_pages)
            a.free_pages[to] = page;
          else
            bad = true;
        }
        if (k < part.y) from[k] = -1;
        at = min(at + __popc(have), a.num_pages);
      }
      if (lane == 0 && (i & ((1 << a.parts_log2) - 1)) == 0) a.lens[b] = 0;
    }
    if (u0 + kTableThreads < units) cluster_sync_all();  // every CTA has read its counts
  }
  if (rank == 0 && threadIdx.x == 0) *a.free_count = static_cast<int>(min(base, static_cast<long long>(a.num_pages)));
  if (bad) atomicOr(a.status, kBadBatchBit);
}

// One cluster of kTableCtas CTAs: 16 is more than every device has to take, so it is asked once (`fit`: 0 not asked, else the
// CTAs).  In a graph with 16 (8, 1) CTAs 200 thousand slots take 12.5 (17, 85) us, the pages of 128 long sequences 11.2 (17, 89), a step's 256
// rows 6.6 with any: a launch, a barrier and the dependent reads of lengths, stack and table.
int launch_cluster(void (*kernel)(const TableArgs), const TableArgs& a, std::atomic<int> (&fit)[64], cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kTableThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto ctas = [&](int n) {
    cfg.gridDim = dim3(n);
    attr[0].val.clusterDim.x = n;
  };
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  std::atomic<int>& known = fit[dev & 63];
  int n = known.load(std::memory_order_relaxed);
  if (n == 0) {
    ctas(kTableCtas);
    int clusters = 0;
    const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0;
    if (!ok) cudaGetLastError();  // (an answer, not an error)
    n = ok ? kTableCtas : kTableCtas / 2;
    known.store(n, std::memory_order_relaxed);
  }
  ctas(n);
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Checks that both calls share; fills the shared arguments.
int take(const fa_page_pool* pool, int* table, long long stride, int max_pages, int* lens, int B, TableArgs* a) {
  if (!pool || !pool->free_pages || !pool->free_count || !table || !lens) return FA_ERR_NULL_POINTER;
  int log2 = 4;
  while (log2 < 10 && (1 << log2) != pool->page_size) ++log2;
  if ((1 << log2) != pool->page_size || pool->num_pages < 1) return FA_ERR_BAD_SHAPE;
  // (The kernels take 1024 sequences at a time, counted in 32 bits.)
  if (B < 1 || B > 0x7ffff000 || max_pages < 1 || stride < max_pages) return FA_ERR_BAD_SHAPE;
  // As fa_paged_batch: positions are 32-bit, those at the end of a tile, too.
  if ((static_cast<long long>(max_pages) << log2) > 0x7ffff000LL) return FA_ERR_BAD_SHAPE;
  if (misaligned(pool->free_pages, 4) || misaligned(pool->free_count, 4) || misaligned(table, 4) || misaligned(lens, 4))
    return FA_ERR_MISALIGNED;
  *a = {};
  a->free_pages = pool->free_pages;
  a->free_count = pool->free_count;
  a->num_pages = pool->num_pages;
  a->ps_log2 = log2;
  a->table = table;
  a->stride = stride;
  a->max_pages = max_pages;
  a->lens = lens;
  a->B = B;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_paged_extend(const fa_page_pool* pool, int* page_table, long long table_stride, int max_pages, int* kv_lens,
                    const int* new_rows, int* cu_rows, long long* slots, int* positions, int B, int rows, void* stream) {
  if (!new_rows || !cu_rows) return FA_ERR_NULL_POINTER;
  fa::TableArgs a;
  int rc = fa::take(pool, page_table, table_stride, max_pages, kv_lens, B, &a);
  if (rc != FA_OK) return rc;
  if (rows < 0 || rows > 0x7ffff000) return FA_ERR_BAD_SHAPE;
  if (fa::misaligned(new_rows, 4) || fa::misaligned(cu_rows, 4) || fa::misaligned(slots, 16) || fa::misaligned(positions, 16))
    return FA_ERR_MISALIGNED;
  fa::LaunchCtx ctx;
  rc = fa::current_ctx(&ctx, stream);
  if (rc != FA_OK) return rc;
  a.new_rows = new_rows;
  a.cu_rows = cu_rows;
  a.slots = slots;
  a.positions = positions;
  a.rows = rows;
  a.status = ctx.status;
  static std::atomic<int> fit[64];
  return fa::launch_cluster(fa::fa_paged_extend_kernel, a, fit, ctx.stream);
}

int fa_paged_release(const fa_page_pool* pool, int* page_table, long long table_stride, int max_pages, int* kv_lens,
                     const unsigned char* done, int B, void* stream) {
  if (!done) return FA_ERR_NULL_POINTER;
  fa::TableArgs a;
  int rc = fa::take(pool, page_table, table_stride, max_pages, kv_lens, B, &a);
  if (rc != FA_OK) return rc;
  fa::LaunchCtx ctx;
  rc = fa::current_ctx(&ctx, stream);
  if (rc != FA_OK) return rc;
  a.done = done;
  a.status = ctx.status;
  // Long rows of few sequences are shared out until every warp of the cluster has two parts (the pages of 17 of 256 sequences of up to
  // 512: 6.5 us; with one part a warp 7.2).
  while (a.parts_log2 < 10 && (static_cast<long long>(B) << a.parts_log2) < 32 * fa::kTableWarps && (max_pages >> a.parts_log2) > 64)
    ++a.parts_log2;
  static std::atomic<int> fit[64];
  return fa::launch_cluster(fa::fa_paged_release_kernel, a, fit, ctx.stream);
}

}  // extern "C"
