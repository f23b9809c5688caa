// Shared parts of the paged-cache kernels: the cache and the batch as the
// kernels see them, and the checked look-ups of sequences and pages.
//
// Nothing that the device arrays name is trusted: a row range, a length or a
// page that is not there is cut to what is, and reported in the status word.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

static_assert(kStatusBadBatch == kBadBatchBit, "status bit of FA_ERR_BAD_BATCH");

constexpr int kMaxGroup = 128;  // query heads per key/value head (one token's rows fit a 128-row tile)

// fa_paged_cache and fa_paged_batch by value (element strides; ps_log2: log2(page_size)).
struct PagedKv {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  long long ks[3];
  long long vs[3];
  int num_pages;
  int ps_log2;
  int heads;
};
struct PagedBatch {
  const int* page_table;
  const int* cu_rows;
  const int* kv_lens;
  long long table_stride;
  int max_pages;
  int B;
  int rows;
};

struct PagedSeq {
  int row0;  // first row
  int n;     // rows
  int len;   // tokens, cut to what the page table can hold
};

// Sequence b, cut to what is there; `bad` is set if anything had to be.
__host__ __device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& pb, int ps_log2, int b, bool& bad) {
  PagedSeq s;
  const int lo = pb.cu_rows[b], hi = pb.cu_rows[b + 1];
  int len = pb.kv_lens[b];
  const long long most = static_cast<long long>(pb.max_pages) << ps_log2;
  bad = false;
  s.row0 = lo;
  s.n = hi - lo;
  if (lo < 0 || hi < lo || hi > pb.rows) {
    s.row0 = 0;
    s.n = 0;
    bad = true;
  }
  if (len < 0 || len > most) {
    len = len < 0 ? 0 : static_cast<int>(most);
    bad = true;
  }
  s.len = len;
  return s;
}

// Reports the batch if any sequence had to be cut; run by all threads of one block.
__device__ __forceinline__ void paged_report(const PagedBatch& pb, int ps_log2, int* status) {
  bool any = false;
  for (int b = threadIdx.x; b < pb.B; b += blockDim.x) {
    bool bad;
    paged_seq(pb, ps_log2, b, bad);
    any = any || bad;
  }
  if (any) atomicOr(status, kStatusBadBatch);
}

// Page of position pos of sequence b, or -1 if the table names none that exists.
__host__ __device__ __forceinline__ int paged_page(const PagedBatch& pb, const PagedKv& kv, int b, int pos) {
  const int page = pb.page_table[b * pb.table_stride + (pos >> kv.ps_log2)];
  return (page >= 0 && page < kv.num_pages) ? page : -1;
}

// 2^(byte - 127); byte 255 is NaN, byte 0 is 2^-127 (a denormal).
__device__ __forceinline__ float scale_of_byte(uint32_t byte) {
  const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23;
  return __uint_as_float(bits);
}

// Two e4m3 bytes (low byte first) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}

// Arguments of the attention kernels.
struct PagedFwdArgs {
  PagedKv kv;
  PagedBatch pb;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;  // [q_heads][rows]
  long long qs[2];
  long long os[2];
  int q_heads;
  int group;     // query heads per key/value head
  int max_rows;
  int few_rows;  // rows (tokens x group) of a sequence that the few-row kernel takes at most
  int few_sets;  // its launches (1 or 2)
  float scale;
  bool causal;
  bool e4m3;
  int d;
  char* workspace;
};

}  // namespace fa
