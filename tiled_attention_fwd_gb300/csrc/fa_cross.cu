// Cross attention of ragged batches: fa_cross_fwd and fa_cross_bwd (declared in
// include/fa_gb300.h) - argument checks and dispatch.
#include <cmath>

#include "../../include/fa_gb300.h"
#include "fa_cross.cuh"
#include "fa_paged_plan.cuh"

namespace fa {
namespace {

// The forward pass is the paged attention's kernels on keys that lie packed (PACKED: a key tile is one TMA box of a sequence's rows, boxes
// may reach into the next sequence's, whose keys are masked and whose values are cleared): longer sequences (unless max_rows says that
// there are none), then those of few rows, then what CTAs left in parts.  64 sequences of 1 to 5 rows over 512 to 4096 keys, 32 over 8 heads,
// d = 128: 110 us, 0.83 of the memory's rate (5.6 TB/s); 4 of 1 to 4 K rows over 2 to 8 K keys, d = 128: 355 us, 1.42 PFLOP/s, 0.74.
//
// d <= 64: the chunk kernel takes the heads in pairs (PAIRED), and all sequences, for its stages hold tiles of two heads then and single tiles read
// keys as fast as they come: 32 sequences of 17 to 200 rows over 100 to 1024 keys, d = 64, 16 heads: 39 us instead of 57.  Against the
// others in us, 16 heads, d = 64 (d = 32, 8 heads): 32 sequences of 40 rows over 600 keys 29 against 38 (26, 34: 16 heads), of 256 46 and 52 (27 and 29), 4
// of 2048 over 4096 147 and 154 (75 and 77); 63 of one row and one of 100 over 2000 98 and 153.  Up to 16 rows the few-row kernel alone is
// the faster one: 32 of 16 over 1000 34 and 39, of 5 28 and 39 (of 17 to 32 it is not: 41 and 29).
template <int D>
int launch_fwd_d(PagedFwdArgs& a, const LaunchCtx& ctx) {
  const long long most = static_cast<long long>(a.max_rows) * a.group;
  a.paired = D <= 64 && a.kv.heads > 1 && most > 16;
  if (a.paired) {
    const int e = launch_paged_chunk<D, true>(a, ctx);
    return e != 0 ? e : launch_paged_join<D, true>(a, true, ctx);
  }
  // 8 or 16 rows where that is all there can be, else 32 (d = 256: 16), as fa_paged_fwd.
  a.few_rows = most <= 8 ? 8 : most <= 16 || D == 256 ? 16 : kFewMost;
  a.few_sets = 1;
  const bool chunks = most > a.few_rows;
  int e = chunks ? launch_paged_chunk<D, true>(a, ctx) : 0;
  if (e == 0) e = launch_paged_few<D, true>(a, chunks, ctx);
  if (e == 0) e = launch_paged_join<D, true>(a, chunks, ctx);
  return e;
}

// ------------------------------------------------------------------ checks
bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// {row, head} element strides: each >= 1 and < 2^38, multiples of 16 bytes.
int check_strides(const long long* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] < 1 || s[i] >= (1LL << 38)) return FA_ERR_BAD_SHAPE;
  for (int i = 0; i < n; ++i)
    if (s[i] % 8 != 0) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// Checks that both passes share; fills the batch and the shape.
int take(const fa_cross_batch* b, int q_heads, int heads, int d, float scale, CrossArgs* a) {
  if (!b || !b->cu_rows || !b->cu_keys) return FA_ERR_NULL_POINTER;
  // Positions at the end of a tile are 32-bit, too, and so are the tiles of all sequences.
  if (b->B < 1 || b->rows < 0 || b->keys < 0 || b->rows > 0x7ffff000 - b->B || b->keys > 0x7ffff000) return FA_ERR_BAD_SHAPE;
  if (heads < 1 || heads > 65535 || q_heads < 1 || q_heads % heads != 0 || q_heads / heads > kCrossGroup) return FA_ERR_BAD_SHAPE;
  if (d != 32 && d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED_D;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_BAD_SCALE;
  if (misaligned(b->cu_rows, 4) || misaligned(b->cu_keys, 4) || misaligned(b->key_lens, 4)) return FA_ERR_MISALIGNED;
  a->cb = CrossBatch{b->cu_rows, b->cu_keys, b->key_lens, b->B, b->rows, b->keys};
  a->q_heads = q_heads;
  a->heads = heads;
  a->group = q_heads / heads;
  a->scale = scale;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_cross_fwd_workspace_bytes(int d) { return d == 32 || d == 64 || d == 128 || d == 256 ? fa::paged_ws_bytes(d) : 0; }

int fa_cross_fwd(const void* q, const long long* q_stride, const void* k, const long long* k_stride, const void* v,
                 const long long* v_stride, const fa_cross_batch* batch, void* o, const long long* o_stride, float* lse,
                 int q_heads, int heads, int d, int max_rows, float scale, void* workspace, size_t workspace_bytes,
                 void* stream) {
  fa::CrossArgs a = {};
  int rc = fa::take(batch, q_heads, heads, d, scale, &a);
  if (rc != FA_OK) return rc;
  if (!q || !o || !lse || !workspace || !q_stride || !k_stride || !v_stride || !o_stride || (batch->keys > 0 && (!k || !v)))
    return FA_ERR_NULL_POINTER;
  if (max_rows < 0) return FA_ERR_BAD_SHAPE;
  const long long* st[4] = {q_stride, k_stride, v_stride, o_stride};
  for (int i = 0; i < 4; ++i) {
    rc = fa::check_strides(st[i], 2);
    if (rc != FA_OK) return rc;
  }
  if (fa::misaligned(q, 16) || fa::misaligned(k, 16) || fa::misaligned(v, 16) || fa::misaligned(o, 16) ||
      fa::misaligned(lse, 4) || fa::misaligned(workspace, 256))
    return FA_ERR_MISALIGNED;
  if (workspace_bytes < fa_cross_fwd_workspace_bytes(d)) return FA_ERR_WORKSPACE;
  fa::LaunchCtx ctx;
  rc = fa::current_ctx(&ctx, stream);
  if (rc != FA_OK || batch->rows == 0) return rc;
  fa::PagedFwdArgs p = {};
  // Without keys the tensor maps are made of something that is there (65535 dense heads, at most 34 MB, are less than the workspace's
  // parts at every d; the caller's head stride may lead out of it).  Nothing is read through them: no kernel loads a tile without keys.
  const bool none = batch->keys == 0;
  p.kv.k = const_cast<void*>(none ? workspace : k);
  p.kv.v = const_cast<void*>(none ? workspace : v);
  for (int i = 0; i < 2; ++i) {
    p.qs[i] = q_stride[i];
    p.kv.ks[i] = none ? d : k_stride[i];
    p.kv.vs[i] = none ? d : v_stride[i];
    p.os[i] = o_stride[i];
  }
  p.kv.heads = heads;
  p.pb.B = batch->B;
  p.pb.rows = batch->rows;
  p.cb = a.cb;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.q_heads = q_heads;
  p.group = a.group;
  p.max_rows = max_rows;
  p.scale = scale;
  p.d = d;
  p.workspace = static_cast<char*>(workspace);
  int e;
  switch (d) {
    case 32: e = fa::launch_fwd_d<32>(p, ctx); break;
    case 64: e = fa::launch_fwd_d<64>(p, ctx); break;
    case 128: e = fa::launch_fwd_d<128>(p, ctx); break;
    default: e = fa::launch_fwd_d<256>(p, ctx); break;
  }
  return e == 0 ? FA_OK : FA_ERR_CUDA;
}

size_t fa_cross_bwd_workspace_bytes(int B, int rows, int q_heads, int heads, int d) {
  if (B < 1 || rows < 0 || rows > 0x7ffff000 - B || heads < 1 || heads > 65535 || q_heads < 1 || q_heads % heads != 0 ||
      q_heads / heads > fa::kCrossGroup || (d != 32 && d != 64 && d != 128 && d != 256))
    return 0;
  switch (d) {
    case 32: return fa::cross_bwd_ws_bytes_d32(B, rows, heads, q_heads / heads);
    case 64: return fa::cross_bwd_ws_bytes_d64(B, rows, heads, q_heads / heads);
    case 128: return fa::cross_bwd_ws_bytes_d128(B, rows, heads, q_heads / heads);
    default: return fa::cross_bwd_ws_bytes_d256(B, rows, heads, q_heads / heads);
  }
}

int fa_cross_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                 void* dq, void* dk, void* dv, const long long* strides, const fa_cross_batch* batch, int q_heads,
                 int heads, int d, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  fa::CrossArgs a = {};
  int rc = fa::take(batch, q_heads, heads, d, scale, &a);
  if (rc != FA_OK) return rc;
  if (!strides || !workspace || (batch->rows > 0 && (!q || !o || !lse || !dout || !dq)) ||
      (batch->keys > 0 && (!k || !v || !dk || !dv)))
    return FA_ERR_NULL_POINTER;
  rc = fa::check_strides(strides, 16);
  if (rc != FA_OK) return rc;
  for (int i = 0; i < 16; ++i) a.st[i >> 1][i & 1] = strides[i];
  const void* all[] = {q, k, v, o, dout, dq, dk, dv};
  for (const void* p : all)
    if (fa::misaligned(p, 16)) return FA_ERR_MISALIGNED;
  if (fa::misaligned(lse, 4) || fa::misaligned(workspace, 256)) return FA_ERR_MISALIGNED;
  if (workspace_bytes < fa_cross_bwd_workspace_bytes(batch->B, batch->rows, q_heads, heads, d)) return FA_ERR_WORKSPACE;
  fa::LaunchCtx ctx;
  rc = fa::current_ctx(&ctx, stream);
  if (rc != FA_OK || (batch->rows == 0 && batch->keys == 0)) return rc;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.o = static_cast<const __nv_bfloat16*>(o);
  a.lse = lse;
  a.dout = static_cast<const __nv_bfloat16*>(dout);
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.status = ctx.status;
  a.workspace = static_cast<char*>(workspace);
  int e;
  switch (d) {
    case 32: e = fa::launch_cross_bwd_d32(a, ctx); break;
    case 64: e = fa::launch_cross_bwd_d64(a, ctx); break;
    case 128: e = fa::launch_cross_bwd_d128(a, ctx); break;
    default: e = fa::launch_cross_bwd_d256(a, ctx); break;
  }
  return e == 0 ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
