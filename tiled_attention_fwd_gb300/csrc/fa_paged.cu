// The paged key/value cache: fa_paged_write, fa_paged_read, fa_paged_fwd
// (declared in include/fa_gb300.h) - argument checks, the kernels that move
// rows between token-major tensors and pages, and the dispatch of the attention.
#include <cmath>

#include "../../include/fa_gb300.h"
#include "fa_paged_plan.cuh"

namespace fa {
namespace {

// ------------------------------------------------------------------ moving rows
// One block moves a few tokens: first a warp per token finds its sequence, page
// and slot, then every thread takes 8 elements (e4m3: 16) of a row (one token, one head,
// K or V) at a time, several rows in flight, so a warp's accesses are whole
// 128-byte lines on both sides.
//
// Bound by memory: a row is read once and written once (2d bytes on the
// token side, 2d or d + 1 on the cache's).  Measured: prefixes of
// 350 MB read at 6.1 TB/s (bf16, 8 heads, d = 128) and 6.0 TB/s (e4m3, 16 heads, d = 64),
// 0.9 of a copy's rate; prompts of 41 K tokens (8 heads, d = 128) written in 56 us, to bf16 pages (338 MB
// moved) at 6.0 TB/s and to e4m3 pages (254 MB) at 4.5 TB/s (0.67): not the stores bound those (without any the kernel
// took as long) but how soon the rows are asked for - behind the look-ups, two items a thread.
struct MoveArgs {
  PagedKv kv;
  PagedBatch pb;
  const __nv_bfloat16* k_in;
  const __nv_bfloat16* v_in;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  long long ks[2];  // {row, head} strides of the token-major K, V
  long long vs[2];
  int tokens_per_block;
  int* status;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 32;  // tokens of a block at most
constexpr __host__ __device__ int move_batch(bool e4m3) { return e4m3 ? 2 : 4; }  // items of a thread at a time

// The sequence whose rows hold row t: the number of b with cu_rows[b + 1] <= t,
// found by the whole warp in steps of 32 sub-ranges.
__device__ __forceinline__ int find_seq(const int* cu_rows, int B, int t, int lane) {
  int lo = 0, count = B;  // the answer lies in [lo, lo + count]
  while (count > 0) {
    const int step = (count + 31) / 32;
    const int at = lo + (lane + 1) * step;  // cu_rows[at] is the end of sequence at - 1
    const bool below = at <= lo + count && cu_rows[at] <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    lo += k * step;
    count = min(step - 1, B - lo);
    if (step == 1) break;
  }
  return lo;
}

// Two threads hold 64 bytes in a row, the even one the first 32: afterwards the even one has the 16-byte units 0 and 2,
// the odd one 1 and 3 (and the other way round), so that a warp's accesses are whole 32-byte sectors.
__device__ __forceinline__ void swap_in_pair(uint4& a, uint4& b, int lane) {
  const bool odd = lane & 1;
  uint4 x = odd ? a : b;
  x.x = __shfl_xor_sync(0xffffffffu, x.x, 1);
  x.y = __shfl_xor_sync(0xffffffffu, x.y, 1);
  x.z = __shfl_xor_sync(0xffffffffu, x.z, 1);
  x.w = __shfl_xor_sync(0xffffffffu, x.w, 1);
  (odd ? a : b) = x;
}

template <int D, bool E4M3, bool WRITE>
__global__ void __launch_bounds__(kMoveThreads) fa_paged_move_kernel(const MoveArgs a) {
  __shared__ int s_page[kMoveTokens];  // -1: nothing to move
  __shared__ int s_slot[kMoveTokens];
  constexpr int EPT = E4M3 ? 16 : 8;  // elements of a thread's item
  constexpr int LPR = D / EPT;        // threads a row
  constexpr int U = move_batch(E4M3);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * a.tokens_per_block;
  const int nt = min(a.tokens_per_block, a.pb.rows - t0);
  if (blockIdx.x == 0) paged_report(a.pb, a.kv.ps_log2, a.status);
  for (int i = warp; i < nt; i += kMoveThreads / 32) {
    const int t = t0 + i;
    const int b = find_seq(a.pb.cu_rows, a.pb.B, t, lane);
    int page = -1, slot = 0;
    if (b < a.pb.B) {
      bool bad;
      const PagedSeq s = paged_seq(a.pb, a.kv.ps_log2, b, bad);
      if (t >= s.row0 && t < s.row0 + s.n) {
        // A cut length moves the positions: nothing of such a sequence is moved.
        const int pos = s.len - s.n + (t - s.row0);
        if (!bad && pos >= 0) {
          page = paged_page(a.pb, a.kv, b, pos);
          slot = pos & ((1 << a.kv.ps_log2) - 1);
          bad = page < 0;
        }
      } else if (t >= a.pb.cu_rows[0]) {
        bad = true;
      }
      if (bad && lane == 0) atomicOr(a.status, kStatusBadBatch);
    }
    if (lane == 0) {
      s_page[i] = page;
      s_slot[i] = slot;
    }
  }
  __syncthreads();
  // Thread x takes items x, x + 256, ... of the block's; item = (token, K or V, head, part of the row).  U items at a
  // time, their loads before any store.
  const int per_token = 2 * a.kv.heads * LPR;
  const int items = nt * per_token;
  const int step_i = kMoveThreads / per_token, step_r = kMoveThreads % per_token;
  int i = static_cast<int>(threadIdx.x) / per_token, r = static_cast<int>(threadIdx.x) % per_token;
  for (int i0 = 0; i0 < items; i0 += U * kMoveThreads) {
    bool active[U];
    uint4 x[U][E4M3 ? 2 : 1];
    char* c_at[U];          // in the cache
    __nv_bfloat16* t_at[U];  // in the token-major tensor (e4m3: the first of this thread's two places)
    uint8_t* s_at[U];       // e4m3: the row's scale
    uint8_t byte[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (The threads of a row stay together: LPR divides 32 and `items`.)
      const int page = i < nt ? s_page[i] : -1, slot = i < nt ? s_slot[i] : 0;
      active[u] = page >= 0;
      const int part = r % LPR;
      const bool is_v = r / LPR >= a.kv.heads;
      const int h = r / LPR - (is_v ? a.kv.heads : 0);
      const long long* cs = is_v ? a.kv.vs : a.kv.ks;
      const long long* ts = is_v ? a.vs : a.ks;
      c_at[u] = static_cast<char*>(is_v ? a.kv.v : a.kv.k) +
                (page * cs[0] + h * cs[1] + slot * cs[2] + part * EPT) * (E4M3 ? 1 : 2);
      const __nv_bfloat16* t = WRITE ? (is_v ? a.v_in : a.k_in) : (is_v ? a.v_out : a.k_out);
      t_at[u] = const_cast<__nv_bfloat16*>(t) + (t0 + i) * ts[0] + h * ts[1] +
                (E4M3 ? (part & ~1) * EPT + (part & 1) * 8 : part * EPT);
      if constexpr (E4M3)
        s_at[u] = (is_v ? a.kv.v_scale : a.kv.k_scale) +
                  ((static_cast<long long>(page) * a.kv.heads + h) << a.kv.ps_log2) + slot;
      i += step_i;
      r += step_r;
      if (r >= per_token) {
        r -= per_token;
        ++i;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u][0] = make_uint4(0, 0, 0, 0);
      if constexpr (E4M3 && WRITE) x[u][1] = make_uint4(0, 0, 0, 0);
      if (!active[u]) continue;
      if constexpr (!E4M3) {
        x[u][0] = *reinterpret_cast<const uint4*>(WRITE ? reinterpret_cast<const char*>(t_at[u]) : c_at[u]);
      } else if constexpr (WRITE) {
        x[u][0] = *reinterpret_cast<const uint4*>(t_at[u]);
        x[u][1] = *reinterpret_cast<const uint4*>(t_at[u] + 16);
      } else {
        x[u][0] = *reinterpret_cast<const uint4*>(c_at[u]);
        byte[u] = *s_at[u];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (!E4M3) {
        if (active[u]) *reinterpret_cast<uint4*>(WRITE ? c_at[u] : reinterpret_cast<char*>(t_at[u])) = x[u][0];
      } else if constexpr (WRITE) {
        swap_in_pair(x[u][0], x[u][1], lane);
        // The row's largest magnitude as bits: bf16 magnitudes order as integers (infinities and NaN on top).
        const uint32_t* w = reinterpret_cast<const uint32_t*>(x[u]);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
#pragma unroll
        for (int m = LPR / 2; m > 0; m >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, m));
        top = max(top & 0xffffu, top >> 16) << 16;  // as fp32 bits
        const bool fine = top < 0x7f800000u;
        // amax = (1 + f) 2^x: the least e with amax 2^-e <= 448 = 1.75 * 2^8 is x - 8, or x - 7 where 1 + f > 1.75.
        int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = e < 0 ? 0 : e;  // (top < 2^128, so e <= 247)
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        // At the largest scale 256 would dequantise to 2^128: codes stop at 240 there.
        const float most = e == 247 ? 240.f : 448.f;
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float y[4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            y[2 * n] = __uint_as_float(w[2 * k + n] << 16) * inv;
            y[2 * n + 1] = __uint_as_float(w[2 * k + n] & 0xffff0000u) * inv;
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) y[n] = fminf(fmaxf(y[n], -most), most);
          c[k] = fine ? pack_e4m3x4(y[0], y[1], y[2], y[3]) : 0u;
        }
        if (active[u]) {
          *reinterpret_cast<uint4*>(c_at[u]) = make_uint4(c[0], c[1], c[2], c[3]);
          if (lane % LPR == 0) *s_at[u] = static_cast<uint8_t>(fine ? e : 255);
        }
      } else {
        const float f = active[u] ? scale_of_byte(byte[u]) : 0.f;
        const uint32_t w[4] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w};
        uint32_t out[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t h2 = e4m3x2_to_f16x2(static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1))));
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          out[k] = pack_bf16x2(y.x * f, y.y * f);
        }
        uint4 y0 = make_uint4(out[0], out[1], out[2], out[3]), y1 = make_uint4(out[4], out[5], out[6], out[7]);
        swap_in_pair(y0, y1, lane);
        if (active[u]) {
          *reinterpret_cast<uint4*>(t_at[u]) = y0;
          *reinterpret_cast<uint4*>(t_at[u] + 16) = y1;
        }
      }
    }
  }
}

template <int D, bool WRITE>
int launch_move_d(const MoveArgs& a, bool e4m3, const LaunchCtx& ctx) {
  const int grid = (a.pb.rows + a.tokens_per_block - 1) / a.tokens_per_block;
  if (e4m3)
    fa_paged_move_kernel<D, true, WRITE><<<grid, kMoveThreads, 0, ctx.stream>>>(a);
  else
    fa_paged_move_kernel<D, false, WRITE><<<grid, kMoveThreads, 0, ctx.stream>>>(a);
  return static_cast<int>(cudaGetLastError());
}

template <bool WRITE>
int launch_move(MoveArgs& a, int d, bool e4m3, const LaunchCtx& ctx) {
  // Tokens a block: an item for every thread; more once the blocks outnumber what the SMs hold at once (8 each), up to
  // two batches of items a thread, so that there are enough blocks to hide how long each takes to find its places
  // (41 K tokens of 8 heads, d = 128, quantised: 57 us; with 32 tokens a block instead of these 8: 61, with 4: 61).
  const int per_token = 2 * a.kv.heads * (d / (e4m3 ? 16 : 8));
  int tb = (kMoveThreads + per_token - 1) / per_token;
  const int even = a.pb.rows / (ctx.num_sms * 8), most = 2 * move_batch(e4m3) * kMoveThreads / per_token;
  const int more = even < most ? even : most;
  tb = tb < more ? more : tb;
  a.tokens_per_block = tb > kMoveTokens ? kMoveTokens : tb;
  a.status = ctx.status;
  int e;
  switch (d) {
    case 32: e = launch_move_d<32, WRITE>(a, e4m3, ctx); break;
    case 64: e = launch_move_d<64, WRITE>(a, e4m3, ctx); break;
    case 128: e = launch_move_d<128, WRITE>(a, e4m3, ctx); break;
    default: e = launch_move_d<256, WRITE>(a, e4m3, ctx); break;
  }
  return e == 0 ? FA_OK : FA_ERR_CUDA;
}

// ------------------------------------------------------------------ attention, mending
// The chunk kernel multiplies whole tiles: P = 0 where a row does not see a key,
// and 0 times an infinity or a NaN in that key's V is NaN.  It notes whether any
// O came out infinite or NaN; if so, this kernel looks at the O of every row of a chunk
// and computes those NaN rows again, plainly, that have such a V behind them (a key that
// some rows of its sequence see and others do not is a new token).  One warp per (row, query head): 32 keys at
// a time, a key per lane for the logits (q from shared memory), then the lanes
// share out the d columns of V.  It is launched behind every causal chunk call and
// leaves at once where there is nothing to mend.
constexpr int kMendWarps = 4;

struct MendParams {
  PagedFwdArgs a;
  const int* odd;
  int n_odd;
};

// (A scale byte of 248 and more, which paged_write never stores, may take a code beyond bf16's range: an infinity in the tile.)
template <int D, bool E4M3>
__device__ __forceinline__ bool row_is_odd(const PagedKv& kv, int page, int head, int slot) {
  const uint8_t* v = static_cast<const uint8_t*>(kv.v) +
                     (page * kv.vs[0] + head * kv.vs[1] + slot * kv.vs[2]) * (E4M3 ? 1 : 2);
  bool odd = E4M3 && kv.v_scale[((static_cast<long long>(page) * kv.heads + head) << kv.ps_log2) + slot] >= 248;
#pragma unroll
  for (int i = 0; i < D * (E4M3 ? 1 : 2) / 16; ++i) {
    const uint4 x = reinterpret_cast<const uint4*>(v)[i];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      odd = odd || (E4M3 ? __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) : __vcmpgeu2(w[k] & 0x7fff7fffu, 0x7f807f80u)) != 0;
  }
  return odd;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kMendWarps * 32) fa_paged_mend_kernel(const __grid_constant__ MendParams p) {
  __shared__ float s_q[kMendWarps][D];
  pdl_wait();
  const PagedFwdArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool any = false;
#pragma unroll
  for (int i = 0; i < kPlanCtas * 4; i += 128) {  // all loads at once: the flags are all that most calls look at
    const int4 x = i + 4 * lane < p.n_odd ? reinterpret_cast<const int4*>(p.odd)[i / 4 + lane] : make_int4(0, 0, 0, 0);
    any = any || (x.x | x.y | x.z | x.w) != 0;
  }
  if (!__any_sync(0xffffffffu, any)) return;
  const long long units = static_cast<long long>(a.pb.rows) * a.q_heads;
  for (long long unit = static_cast<long long>(blockIdx.x) * kMendWarps + warp; unit < units;
       unit += static_cast<long long>(gridDim.x) * kMendWarps) {
    const int t = static_cast<int>(unit / a.q_heads), hq = static_cast<int>(unit % a.q_heads);
    const int hk = hq / a.group;
    const int b = find_seq(a.pb.cu_rows, a.pb.B, t, lane);
    if (b >= a.pb.B) continue;
    bool bad;
    const PagedSeq s = paged_seq(a.pb, a.kv.ps_log2, b, bad);
    if (t < s.row0 || t >= s.row0 + s.n || s.n > a.max_rows || (s.n <= kFewMost && s.n * a.group <= a.few_rows)) continue;
    // Such a V has made the row's O a NaN (0 times it); all other rows are done with here.
    bool spoiled = false;
#pragma unroll
    for (int c = 0; c < D; c += 32) spoiled = spoiled || __hisnan(a.o[t * a.os[0] + hq * a.os[1] + c + lane]);
    if (!__any_sync(0xffffffffu, spoiled)) continue;
    const int see = s.len - s.n + (t - s.row0) + 1;  // keys 0 .. see - 1
    bool odd = false;
    for (int j = max(see, 0) + lane; j < s.len; j += 32) {
      const int page = paged_page(a.pb, a.kv, b, j);
      odd = odd || (page >= 0 && row_is_odd<D, E4M3>(a.kv, page, hk, j & ((1 << a.kv.ps_log2) - 1)));
    }
    if (!__any_sync(0xffffffffu, odd)) continue;
    __syncwarp();
    for (int c = lane; c < D; c += 32) s_q[warp][c] = __bfloat162float(a.q[t * a.qs[0] + hq * a.qs[1] + c]);
    __syncwarp();
    const float sl2 = a.scale * 1.4426950408889634f;
    constexpr int CPL = D / 32;  // columns a lane
    float acc[CPL] = {};
    float m = -INFINITY, l = 0.f;
    for (int j0 = 0; j0 < see; j0 += 32) {
      const int j = j0 + lane;
      float x = -INFINITY;
      int page = -1;
      if (j < see) {
        page = paged_page(a.pb, a.kv, b, j);
        const int slot = j & ((1 << a.kv.ps_log2) - 1);
        float dot = 0.f;
        if (page < 0) {
          // (reported by the kernels before)
        } else if constexpr (E4M3) {
          const uint8_t* k = static_cast<const uint8_t*>(a.kv.k) + page * a.kv.ks[0] + hk * a.kv.ks[1] + slot * a.kv.ks[2];
          for (int c = 0; c < D; c += 2) {
            const uint32_t h2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(k + c));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            dot = fmaf(s_q[warp][c], y.x, fmaf(s_q[warp][c + 1], y.y, dot));
          }
          dot *= scale_of_byte(a.kv.k_scale[((static_cast<long long>(page) * a.kv.heads + hk) << a.kv.ps_log2) + slot]);
        } else {
          const __nv_bfloat16* k =
              static_cast<const __nv_bfloat16*>(a.kv.k) + page * a.kv.ks[0] + hk * a.kv.ks[1] + slot * a.kv.ks[2];
          for (int c = 0; c < D; c += 2) {
            const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(k + c));
            dot = fmaf(s_q[warp][c], y.x, fmaf(s_q[warp][c + 1], y.y, dot));
          }
        }
        x = dot * sl2;
      }
      float top = x;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float m_new = fmaxf(m, top);
      const float alpha = m_new == m ? 1.f : ex2(m - m_new);
      const float p = j < see ? ex2(x - (m_new == -INFINITY ? 0.f : m_new)) : 0.f;
      float sum = p;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      l = l * alpha + sum;
      m = m_new;
#pragma unroll
      for (int c = 0; c < CPL; ++c) acc[c] *= alpha;
      const int nk = min(32, see - j0);
      for (int i = 0; i < nk; ++i) {
        const float pi = __shfl_sync(0xffffffffu, p, i);
        const int pg = __shfl_sync(0xffffffffu, page, i);
        if (pg < 0) continue;
        const int slot = (j0 + i) & ((1 << a.kv.ps_log2) - 1);
        const long long off = pg * a.kv.vs[0] + hk * a.kv.vs[1] + slot * a.kv.vs[2];
        if constexpr (E4M3) {
          const float f =
              scale_of_byte(a.kv.v_scale[((static_cast<long long>(pg) * a.kv.heads + hk) << a.kv.ps_log2) + slot]);
          const uint8_t* v = static_cast<const uint8_t*>(a.kv.v) + off;
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            const uint32_t h2 = e4m3x2_to_f16x2(v[c * 32 + lane]);
            acc[c] = fmaf(pi, __low2float(*reinterpret_cast<const __half2*>(&h2)) * f, acc[c]);
          }
        } else {
          const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.kv.v) + off;
#pragma unroll
          for (int c = 0; c < CPL; ++c) acc[c] = fmaf(pi, __bfloat162float(v[c * 32 + lane]), acc[c]);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int c = 0; c < CPL; ++c)
      a.o[t * a.os[0] + hq * a.os[1] + c * 32 + lane] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[c] * inv);
    if (lane == 0)
      a.lse[static_cast<long long>(hq) * a.pb.rows + t] = (m + log2f(l)) * 0.69314718055994531f;
  }
}

template <int D>
int launch_mend(const PagedFwdArgs& a, const LaunchCtx& ctx) {
  const int ctas = ctx.num_sms < kPlanCtas ? ctx.num_sms : kPlanCtas;
  const MendParams p{a, paged_ws(a.workspace, D).odd, ctas * 4};
  return a.e4m3 ? launch_dependent(fa_paged_mend_kernel<D, true>, dim3(ctas * 4), kMendWarps * 32, 0, ctx.stream, p)
                : launch_dependent(fa_paged_mend_kernel<D, false>, dim3(ctas * 4), kMendWarps * 32, 0, ctx.stream, p);
}

// The chunks (unless max_rows says that there are none), then the sequences of few rows, whose blocks begin on SMs
// that have done their share of the chunks, then what CTAs left in parts.
template <int D>
int launch_fwd_d(PagedFwdArgs& a, const LaunchCtx& ctx) {
  const long long most = static_cast<long long>(a.max_rows) * a.group;
  // 8 or 16 rows where that is all there can be, else 32 (d = 256: 16, a thread's registers hold no more outputs).
  a.few_rows = most <= 8 ? 8 : most <= 16 || D == 256 ? 16 : kFewMost;
  const bool chunks = most > a.few_rows;
  a.few_sets = a.e4m3 && a.few_rows > 16 && static_cast<long long>(a.pb.B) * a.kv.heads >= 2 * ctx.num_sms ? 2 : 1;
  int e = chunks ? launch_paged_chunk<D>(a, ctx) : 0;
  if (e == 0) e = launch_paged_few<D>(a, chunks, ctx);
  if (e == 0) e = launch_paged_join<D>(a, chunks, ctx);
  if (e == 0 && chunks && a.causal) e = launch_mend<D>(a, ctx);
  return e;
}

// ------------------------------------------------------------------ checks
bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// n element strides: each >= 1 and < 2^38, multiples of 16 bytes.
int check_strides(const long long* s, int n, int elem_bytes) {
  for (int i = 0; i < n; ++i)
    if (s[i] < 1 || s[i] >= (1LL << 38)) return FA_ERR_BAD_SHAPE;
  for (int i = 0; i < n; ++i)
    if (s[i] * elem_bytes % 16 != 0) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// The cache and the batch, checked and copied.
int take(const fa_paged_cache* c, const fa_paged_batch* b, PagedKv* kv, PagedBatch* pb, bool* e4m3) {
  if (!c || !b || !c->k || !c->v || !b->page_table || !b->cu_rows || !b->kv_lens) return FA_ERR_NULL_POINTER;
  if (!c->k_scale != !c->v_scale) return FA_ERR_NULL_POINTER;
  *e4m3 = c->k_scale != nullptr;
  if (c->num_pages < 1 || c->heads < 1 || c->heads > 65535) return FA_ERR_BAD_SHAPE;
  int log2 = 4;
  while (log2 < 10 && (1 << log2) != c->page_size) ++log2;
  if ((1 << log2) != c->page_size) return FA_ERR_BAD_SHAPE;
  if (b->B < 1 || b->rows < 0 || b->max_pages < 1 || b->table_stride < b->max_pages) return FA_ERR_BAD_SHAPE;
  if (c->d != 32 && c->d != 64 && c->d != 128 && c->d != 256) return FA_ERR_UNSUPPORTED_D;
  // Positions are 32-bit, those at the end of a tile (512 keys at most) and of the batch of tiles behind it, too.
  if ((static_cast<long long>(b->max_pages) << log2) > 0x7ffff000LL) return FA_ERR_BAD_SHAPE;
  const int eb = *e4m3 ? 1 : 2;
  int rc = check_strides(c->k_stride, 3, eb);
  if (rc == FA_OK) rc = check_strides(c->v_stride, 3, eb);
  if (rc != FA_OK) return rc;
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 16) || misaligned(c->v_scale, 16) ||
      misaligned(b->page_table, 4) || misaligned(b->cu_rows, 4) || misaligned(b->kv_lens, 4))
    return FA_ERR_MISALIGNED;
  kv->k = c->k;
  kv->v = c->v;
  kv->k_scale = c->k_scale;
  kv->v_scale = c->v_scale;
  for (int i = 0; i < 3; ++i) {
    kv->ks[i] = c->k_stride[i];
    kv->vs[i] = c->v_stride[i];
  }
  kv->num_pages = c->num_pages;
  kv->ps_log2 = log2;
  kv->heads = c->heads;
  pb->page_table = b->page_table;
  pb->cu_rows = b->cu_rows;
  pb->kv_lens = b->kv_lens;
  pb->table_stride = b->table_stride;
  pb->max_pages = b->max_pages;
  pb->B = b->B;
  pb->rows = b->rows;
  return FA_OK;
}

template <bool WRITE>
int move(const fa_paged_cache* cache, const fa_paged_batch* batch, const void* k, const long long* k_stride,
         const void* v, const long long* v_stride, void* stream) {
  if (!k || !v || !k_stride || !v_stride) return FA_ERR_NULL_POINTER;
  MoveArgs a = {};
  bool e4m3;
  int rc = take(cache, batch, &a.kv, &a.pb, &e4m3);
  if (rc != FA_OK) return rc;
  rc = check_strides(k_stride, 2, 2);
  if (rc == FA_OK) rc = check_strides(v_stride, 2, 2);
  if (rc != FA_OK) return rc;
  if (misaligned(k, 16) || misaligned(v, 16)) return FA_ERR_MISALIGNED;
  LaunchCtx ctx;
  rc = current_ctx(&ctx, stream);
  if (rc != FA_OK || batch->rows == 0) return rc;
  if (WRITE) {
    a.k_in = static_cast<const __nv_bfloat16*>(k);
    a.v_in = static_cast<const __nv_bfloat16*>(v);
  } else {
    a.k_out = static_cast<__nv_bfloat16*>(const_cast<void*>(k));
    a.v_out = static_cast<__nv_bfloat16*>(const_cast<void*>(v));
  }
  for (int i = 0; i < 2; ++i) {
    a.ks[i] = k_stride[i];
    a.vs[i] = v_stride[i];
  }
  return launch_move<WRITE>(a, cache->d, e4m3, ctx);
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_paged_write(const fa_paged_cache* cache, const fa_paged_batch* batch, const void* k, const long long* k_stride,
                   const void* v, const long long* v_stride, void* stream) {
  return fa::move<true>(cache, batch, k, k_stride, v, v_stride, stream);
}

int fa_paged_read(const fa_paged_cache* cache, const fa_paged_batch* batch, void* k, const long long* k_stride,
                  void* v, const long long* v_stride, void* stream) {
  return fa::move<false>(cache, batch, k, k_stride, v, v_stride, stream);
}

size_t fa_paged_fwd_workspace_bytes(int B, int heads, int d) {
  if (B < 1 || heads < 1 || heads > 65535 || (d != 32 && d != 64 && d != 128 && d != 256)) return 0;
  return fa::paged_ws_bytes(d);
}

int fa_paged_fwd(const void* q, const long long* q_stride, const fa_paged_cache* cache, const fa_paged_batch* batch,
                 void* o, const long long* o_stride, float* lse, int q_heads, int max_rows, float scale, int causal,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !q_stride || !o || !o_stride || !lse || !workspace) return FA_ERR_NULL_POINTER;
  fa::PagedFwdArgs a = {};
  int rc = fa::take(cache, batch, &a.kv, &a.pb, &a.e4m3);
  if (rc != FA_OK) return rc;
  if (q_heads < 1 || q_heads % cache->heads != 0 || q_heads / cache->heads > fa::kMaxGroup || max_rows < 0)
    return FA_ERR_BAD_SHAPE;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_BAD_SCALE;
  rc = fa::check_strides(q_stride, 2, 2);
  if (rc == FA_OK) rc = fa::check_strides(o_stride, 2, 2);
  if (rc != FA_OK) return rc;
  if (fa::misaligned(q, 16) || fa::misaligned(o, 16) || fa::misaligned(lse, 4) || fa::misaligned(workspace, 256))
    return FA_ERR_MISALIGNED;
  if (workspace_bytes < fa_paged_fwd_workspace_bytes(batch->B, cache->heads, cache->d)) return FA_ERR_WORKSPACE;
  fa::LaunchCtx ctx;
  rc = fa::current_ctx(&ctx, stream);
  if (rc != FA_OK || batch->rows == 0) return rc;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  for (int i = 0; i < 2; ++i) {
    a.qs[i] = q_stride[i];
    a.os[i] = o_stride[i];
  }
  a.q_heads = q_heads;
  a.group = q_heads / cache->heads;
  a.max_rows = max_rows;
  a.scale = scale;
  a.causal = causal != 0;
  a.d = cache->d;
  a.workspace = static_cast<char*>(workspace);
  int e;
  switch (a.d) {
    case 32: e = fa::launch_fwd_d<32>(a, ctx); break;
    case 64: e = fa::launch_fwd_d<64>(a, ctx); break;
    case 128: e = fa::launch_fwd_d<128>(a, ctx); break;
    default: e = fa::launch_fwd_d<256>(a, ctx); break;
  }
  return e == 0 ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
