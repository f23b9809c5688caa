// Shared parts of the cross-attention kernels: the batch as the kernels see it
// and the checked look-up of its sequences.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

constexpr int kCrossGroup = 32;  // query heads per key/value head at most

// fa_cross_batch by value.
struct CrossBatch {
  const int* cu_rows;
  const int* cu_keys;
  const int* key_lens;  // or null
  int B;
  int rows;
  int keys;
};

struct CrossSeq {
  int row0;    // first row
  int n;       // rows
  int key0;    // first place
  int places;
  int len;     // keys: the first `len` places
};

// Sequence b, cut to what is there; `bad` is set if anything had to be.
__host__ __device__ __forceinline__ CrossSeq cross_seq(const CrossBatch& cb, int b, bool& bad) {
  CrossSeq s;
  const int lo = cb.cu_rows[b], hi = cb.cu_rows[b + 1];
  const int klo = cb.cu_keys[b], khi = cb.cu_keys[b + 1];
  bad = lo < 0 || hi < lo || hi > cb.rows;
  s.row0 = bad ? 0 : lo;
  s.n = bad ? 0 : hi - lo;
  const bool no_keys = klo < 0 || khi < klo || khi > cb.keys;
  s.key0 = no_keys ? 0 : klo;
  s.places = no_keys ? 0 : khi - klo;
  const int len = cb.key_lens ? cb.key_lens[b] : s.places;
  s.len = len < 0 ? 0 : len > s.places ? s.places : len;
  bad = bad || no_keys || len != s.len;
  return s;
}

// Arguments of the kernels ({row, head} element strides).
struct CrossArgs {
  CrossBatch cb;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* o;
  const float* lse;  // [q_heads][rows]
  const __nv_bfloat16* dout;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  long long st[8][2];  // of q, k, v, o, dout, dq, dk, dv
  int q_heads;
  int heads;
  int group;
  int max_rows;
  float scale;
  int* status;
  char* workspace;
};

// The backward pass for one head dimension (fa_cross_bwd_d<D>.cu); a cudaError_t-like code.  And the bytes of its workspace.
int launch_cross_bwd_d32(const CrossArgs& a, const LaunchCtx& ctx);
int launch_cross_bwd_d64(const CrossArgs& a, const LaunchCtx& ctx);
int launch_cross_bwd_d128(const CrossArgs& a, const LaunchCtx& ctx);
int launch_cross_bwd_d256(const CrossArgs& a, const LaunchCtx& ctx);
size_t cross_bwd_ws_bytes_d32(int B, int rows, int heads, int group);
size_t cross_bwd_ws_bytes_d64(int B, int rows, int heads, int group);
size_t cross_bwd_ws_bytes_d128(int B, int rows, int heads, int group);
size_t cross_bwd_ws_bytes_d256(int B, int rows, int heads, int group);

}  // namespace fa
