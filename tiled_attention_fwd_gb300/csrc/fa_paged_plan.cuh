// How the paged attention's work is dealt out.  The lengths live on the device,
// so the kernels plan for themselves: the key tiles of all (sequence, head[,
// query block]) units form one line, sequence by sequence, and CTA c of n takes
// the tiles [W c / n, W (c + 1) / n).  Every CTA has the same number of tiles,
// whatever the lengths are; a unit that a CTA does not hold whole leaves a
// partial result in the workspace, and the joining kernel adds those up in the
// order of their CTAs (so results do not depend on timing).
#pragma once

#include <atomic>

#include "fa_paged.cuh"

namespace fa {

constexpr int kPlanCtas = 160;  // CTAs of an attention kernel at most (GB300: 152 SMs, one CTA each)

// What a CTA found out about its share.
struct PlanShare {
  long long total;   // W: tiles of all sequences
  long long start;   // first tile of this CTA
  long long end;     // behind its last
  int ctas;          // n: CTAs that have tiles
  int b;             // sequence of tile `start`
  long long offset;  // `start` within that sequence's tiles
};

struct PlanScratch {
  long long warp_sum[16];
  long long base;
  int b;
};

// CTA that holds tile x of W dealt to n CTAs.
__host__ __device__ __forceinline__ int plan_cta_of(long long x, long long total, int n) {
  return static_cast<int>(((x + 1) * n - 1) / total);
}

// All THREADS threads of the CTA take part.  tiles(b): the length of sequence b's
// tiles on the line (the same value whenever it is asked); a CTA has `least` of it at least.
template <int THREADS, class F>
__device__ __forceinline__ PlanShare plan_share(int B, int ctas, int cta, const F& tiles, int least, PlanScratch& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Sum of one chunk of THREADS sequences up to and including this thread's, and of the whole chunk.
  auto scan = [&](long long w, long long& sum) -> long long {
    long long x = w;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, k);
      if (lane >= k) x += y;
    }
    if (lane == 31) s.warp_sum[warp] = x;
    __syncthreads();
    sum = 0;
    long long before = 0;
    for (int k = 0; k < THREADS / 32; ++k) {
      const long long y = s.warp_sum[k];
      if (k < warp) before += y;
      sum += y;
    }
    __syncthreads();
    return x + before;
  };
  long long total = 0, w = 0, upto = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    w = b < B ? tiles(b) : 0;
    long long sum;
    upto = scan(w, sum);
    total += sum;
  }
  PlanShare p;
  p.total = total;
  p.ctas = total / least < ctas ? static_cast<int>(total / least) : ctas;
  p.start = p.end = 0;
  p.b = 0;
  p.offset = 0;
  if (cta >= p.ctas) return p;
  p.start = total * cta / p.ctas;
  p.end = total * (cta + 1) / p.ctas;
  long long base = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    long long sum = total;
    if (B > THREADS) {
      w = b < B ? tiles(b) : 0;
      upto = scan(w, sum);
    }
    const long long first = base + upto - w;
    if (w > 0 && first <= p.start && p.start < first + w) {
      s.b = b;
      s.base = first;
    }
    base += sum;
  }
  __syncthreads();
  p.b = s.b;
  p.offset = p.start - s.base;
  return p;
}

// A unit that several CTAs hold: written by the CTA that holds its first tile
// (its part 1); the parts of the next `more` CTAs (their part 0) follow.
struct alignas(16) PlanRecord {
  int b;     // -1: no such unit
  int head;  // key/value head
  int qb;    // query block
  int more;
};

// Workspace of fa_paged_fwd.  A part holds a row's log2-sum-exp2 L (log2 units of the scaled logits) and its
// normalised O in fp32; parts join as O = sum 2^(L_i - L) O_i, L = log2 sum 2^L_i.
struct PagedWs {
  PlanRecord* few_rec[2];  // of the one or two launches of the few-row kernel: [kPlanCtas]
  PlanRecord* chunk_rec;   // [kPlanCtas]
  int* odd;                // [kPlanCtas][4]: a correction warp of the chunk kernel met an infinity or a NaN in O
  float* few_part[2];      // [kPlanCtas][2][part_floats(kFewMost, d)]
  float* chunk_part;       // [kPlanCtas][2][part_floats(chunk_rows(d), d)]
};
constexpr int kFewMost = 32;  // rows of a unit of the few-row kernel at most
constexpr __host__ __device__ int chunk_rows(int d) { return d <= 128 ? 256 : 128; }  // of a query block
constexpr __host__ __device__ size_t part_floats(int rows, int d) { return static_cast<size_t>(rows) * (d + 1); }
inline size_t paged_ws_layout(char* p, int d, PagedWs* w) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* x = p + at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return x;
  };
  PagedWs x;
  for (int i = 0; i < 2; ++i) x.few_rec[i] = reinterpret_cast<PlanRecord*>(take(kPlanCtas * sizeof(PlanRecord)));
  x.chunk_rec = reinterpret_cast<PlanRecord*>(take(kPlanCtas * sizeof(PlanRecord)));
  x.odd = reinterpret_cast<int*>(take(kPlanCtas * 4 * sizeof(int)));
  for (int i = 0; i < 2; ++i)
    x.few_part[i] = reinterpret_cast<float*>(take(kPlanCtas * 2 * part_floats(kFewMost, d) * sizeof(float)));
  x.chunk_part = reinterpret_cast<float*>(take(kPlanCtas * 2 * part_floats(chunk_rows(d), d) * sizeof(float)));
  if (w) *w = x;
  return at;
}
inline size_t paged_ws_bytes(int d) { return paged_ws_layout(nullptr, d, nullptr); }
inline PagedWs paged_ws(char* p, int d) {
  PagedWs w;
  paged_ws_layout(p, d, &w);
  return w;
}

// Programmatic dependent launch: let the next kernel of the stream be scheduled / wait for the previous one's writes.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Entry points of the attention kernels' translation units; each returns a cudaError_t-like code.
template <int D, bool PACKED = false>
int launch_paged_few(const PagedFwdArgs& a, bool behind_chunks, const LaunchCtx& ctx);
template <int D, bool PACKED = false>
int launch_paged_chunk(const PagedFwdArgs& a, const LaunchCtx& ctx);
template <int D, bool PACKED = false>
int launch_paged_join(const PagedFwdArgs& a, bool chunks, const LaunchCtx& ctx);

// Launch behind the stream's previous kernel, which may still run: the kernel waits for it itself (pdl_wait).
template <class... P, class... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Allow a kernel its dynamic shared memory, once per device (the attribute is per function and device).
template <class K>
int allow_smem(K* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return static_cast<int>(e);
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return 0;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return static_cast<int>(e);
}

}  // namespace fa
