// Cross attention of ragged batches: fa_cross_fwd and fa_cross_bwd (declared in
// include/fa_gb300.h) - argument checks and dispatch.
#include <cmath>

#include "../../include/fa_gb300.h"
#include "fa_cross.cuh"
#include "fa_paged_plan.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

template <int D>
__device__ __forceinline__ float dot_row(const float* x, const __nv_bfloat16* y) {
  float sum = 0.f;
  for (int c = 0; c < D; c += 2) {
    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(y + c));
    sum = fmaf(x[c], v.x, fmaf(x[c + 1], v.y, sum));
  }
  return sum;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
  return x;
}

// Simple kernels: one warp to a row of outputs, a block to a sequence (grid.y) at a time.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) fa_cross_dq_plain(const CrossArgs a) {
  __shared__ float s_q[kWarps][D], s_do[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = blockIdx.y; b < a.cb.B; b += gridDim.y) {
    bool bad;
    const CrossSeq s = cross_seq(a.cb, b, bad);
    if (bad) atomicOr(a.status, kBadBatchBit);
    for (long long unit = blockIdx.x * kWarps + warp; unit < static_cast<long long>(s.n) * a.q_heads; unit += gridDim.x * kWarps) {
      const long long t = s.row0 + unit / a.q_heads;
      const int h = static_cast<int>(unit % a.q_heads), hk = h / a.group;
      __syncwarp();
      float dsum = 0.f;
      for (int c = lane; c < D; c += 32) {
        s_q[warp][c] = __bfloat162float(a.q[t * a.st[0][0] + h * a.st[0][1] + c]);
        s_do[warp][c] = __bfloat162float(a.dout[t * a.st[4][0] + h * a.st[4][1] + c]);
        dsum = fmaf(s_do[warp][c], __bfloat162float(a.o[t * a.st[3][0] + h * a.st[3][1] + c]), dsum);
      }
      dsum = warp_sum(dsum);
      __syncwarp();
      const float L = a.lse[static_cast<long long>(h) * a.cb.rows + t];
      float acc[D / 32] = {};
      for (int j0 = 0; j0 < s.len; j0 += 32) {
        const int j = j0 + lane;
        float ds = 0.f;
        if (j < s.len) {
          const long long at = static_cast<long long>(s.key0) + j;
          const float p = expf(dot_row<D>(s_q[warp], a.k + at * a.st[1][0] + hk * a.st[1][1]) * a.scale - L);
          ds = p * (dot_row<D>(s_do[warp], a.v + at * a.st[2][0] + hk * a.st[2][1]) - dsum);
        }
        for (int i = 0; i < min(32, s.len - j0); ++i) {
          const float di = __shfl_sync(0xffffffffu, ds, i);
          const __nv_bfloat16* k = a.k + (static_cast<long long>(s.key0) + j0 + i) * a.st[1][0] + hk * a.st[1][1];
          for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(di, __bfloat162float(k[c * 32 + lane]), acc[c]);
        }
      }
      for (int c = 0; c < D / 32; ++c)
        a.dq[t * a.st[5][0] + h * a.st[5][1] + c * 32 + lane] = __float2bfloat16_rn(acc[c] * a.scale);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) fa_cross_dkv_plain(const CrossArgs a) {
  __shared__ float s_k[kWarps][D], s_v[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = blockIdx.y; b < a.cb.B; b += gridDim.y) {
    bool bad;
    const CrossSeq s = cross_seq(a.cb, b, bad);
    for (long long unit = blockIdx.x * kWarps + warp; unit < static_cast<long long>(s.places) * a.heads; unit += gridDim.x * kWarps) {
      const int j = static_cast<int>(unit / a.heads), hk = static_cast<int>(unit % a.heads);
      const long long at = static_cast<long long>(s.key0) + j;
      __syncwarp();
      for (int c = lane; c < D; c += 32) {
        s_k[warp][c] = __bfloat162float(a.k[at * a.st[1][0] + hk * a.st[1][1] + c]);
        s_v[warp][c] = __bfloat162float(a.v[at * a.st[2][0] + hk * a.st[2][1] + c]);
      }
      __syncwarp();
      float dk[D / 32] = {}, dv[D / 32] = {};
      const long long rows = j < s.len ? static_cast<long long>(s.n) * a.group : 0;
      for (long long r0 = 0; r0 < rows; r0 += 32) {
        const long long r = r0 + lane;
        float p = 0.f, ds = 0.f;
        if (r < rows) {
          const long long t = s.row0 + r / a.group;
          const int h = hk * a.group + static_cast<int>(r % a.group);
          const __nv_bfloat16* dout = a.dout + t * a.st[4][0] + h * a.st[4][1];
          const __nv_bfloat16* o = a.o + t * a.st[3][0] + h * a.st[3][1];
          float dsum = 0.f;
          for (int c = 0; c < D; ++c) dsum = fmaf(__bfloat162float(dout[c]), __bfloat162float(o[c]), dsum);
          p = expf(dot_row<D>(s_k[warp], a.q + t * a.st[0][0] + h * a.st[0][1]) * a.scale - a.lse[static_cast<long long>(h) * a.cb.rows + t]);
          ds = p * (dot_row<D>(s_v[warp], dout) - dsum);
        }
        for (int i = 0; i < static_cast<int>(min(32ll, rows - r0)); ++i) {
          const float pi = __shfl_sync(0xffffffffu, p, i), di = __shfl_sync(0xffffffffu, ds, i);
          const long long t = s.row0 + (r0 + i) / a.group;
          const int h = hk * a.group + static_cast<int>((r0 + i) % a.group);
          for (int c = 0; c < D / 32; ++c) {
            dk[c] = fmaf(di, __bfloat162float(a.q[t * a.st[0][0] + h * a.st[0][1] + c * 32 + lane]), dk[c]);
            dv[c] = fmaf(pi, __bfloat162float(a.dout[t * a.st[4][0] + h * a.st[4][1] + c * 32 + lane]), dv[c]);
          }
        }
      }
      for (int c = 0; c < D / 32; ++c) {
        a.dk[at * a.st[6][0] + hk * a.st[6][1] + c * 32 + lane] = __float2bfloat16_rn(dk[c] * a.scale);
        a.dv[at * a.st[7][0] + hk * a.st[7][1] + c * 32 + lane] = __float2bfloat16_rn(dv[c]);
      }
    }
  }
}

// The forward pass is the paged attention's kernels on keys that lie packed: longer sequences (unless max_rows says that there are
// none), then those of few rows, then what CTAs left in parts.
template <int D>
int launch_fwd_d(PagedFwdArgs& a, const LaunchCtx& ctx) {
  const long long most = static_cast<long long>(a.max_rows) * a.group;
  // 8 or 16 rows where that is all there can be, else 32 (d = 256: 16), as fa_paged_fwd.
  a.few_rows = most <= 8 ? 8 : most <= 16 || D == 256 ? 16 : kFewMost;
  a.few_sets = 1;
  const bool chunks = most > a.few_rows;
  int e = chunks ? launch_paged_chunk<D, true>(a, ctx) : 0;
  if (e == 0) e = launch_paged_few<D, true>(a, chunks, ctx);
  if (e == 0) e = launch_paged_join<D, true>(a, chunks, ctx);
  return e;
}

template <int D>
int launch_bwd_plain(const CrossArgs& a, const LaunchCtx& ctx) {
  const dim3 grid(16, a.cb.B < 1024 ? a.cb.B : 1024);
  fa_cross_dq_plain<D><<<grid, kWarps * 32, 0, ctx.stream>>>(a);
  fa_cross_dkv_plain<D><<<grid, kWarps * 32, 0, ctx.stream>>>(a);
  return static_cast<int>(cudaGetLastError());
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
  if (b->B < 1 || b->rows < 0 || b->keys < 0 || b->rows > 0x7ffff000 || b->keys > 0x7ffff000) return FA_ERR_BAD_SHAPE;
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
  // (Without keys the tensor maps are made of something that is there; nothing is read through them.)
  p.kv.k = const_cast<void*>(batch->keys > 0 ? k : workspace);
  p.kv.v = const_cast<void*>(batch->keys > 0 ? v : workspace);
  for (int i = 0; i < 2; ++i) {
    p.qs[i] = q_stride[i];
    p.kv.ks[i] = k_stride[i];
    p.kv.vs[i] = v_stride[i];
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
  if (B < 1 || rows < 0 || rows > 0x7ffff000 || heads < 1 || heads > 65535 || q_heads < 1 || q_heads % heads != 0 ||
      q_heads / heads > fa::kCrossGroup || (d != 32 && d != 64 && d != 128 && d != 256))
    return 0;
  return 256 + static_cast<size_t>(rows) * q_heads * 8;
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
    case 32: e = fa::launch_bwd_plain<32>(a, ctx); break;
    case 64: e = fa::launch_bwd_plain<64>(a, ctx); break;
    case 128: e = fa::launch_bwd_plain<128>(a, ctx); break;
    default: e = fa::launch_bwd_plain<256>(a, ctx); break;
  }
  return e == 0 ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
