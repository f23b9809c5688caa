// Attention of few rows over a paged cache: sequences whose rows (n_b tokens x
// the query heads of one key/value head) fit 16, decoding above all.
//
//   s_ij = scale q_i . k_j,  m, l: running maximum and sum,  o_i = sum_j p_ij v_j / l_i
//
// Bound by reading K and V once, so everything serves to keep reads in flight:
//  * one CTA per SM; each warp is a pipeline of its own: it takes every NW-th
//    group of 16 keys, loads K and V of a group with TMA boxes of 16 tokens
//    (a page holds whole groups) into its own ring of stages, and issues the
//    load S groups ahead, across the borders of units; no barrier between
//    warps but where a unit ends;
//  * the 16 rows are the M of mma.sync m16n8k16 (a tcgen05 tile of 128 rows
//    would multiply 7/8 padding, and its softmax would cost 128 rows);
//  * softmax state m, l and the output stay in registers; at a unit's end the
//    warps' results are joined in shared memory, in a fixed order.
// e4m3 pages: codes are exact in fp16, so S = Q K^T runs in fp16 with the codes
// as they are and every q row multiplied by a power of two that brings its
// largest element to [2^13, 2^14) (exact down to 2^-37 of that element); the
// rows' and the keys' powers of two multiply the fp32 result.  V's scales go
// into P: P' = p 2^(e_j - E) 2^14 in fp16, E the largest exponent so far (kept
// like the maximum: a larger one rescales the output, exactly).  P' is rounded
// to 11 bits down to p 2^(e_j - E) = 2^-28, finer than bf16's 8.
#pragma once

#include "fa_paged_plan.cuh"

namespace fa {

template <int D, bool E4M3>
struct FewCfg {
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int ROWB = D * EB;                     // bytes of a K or V row
  static constexpr int NW = D == 256 ? 4 : 8;             // warps; d = 256 keeps 128 output registers a thread
  static constexpr int THREADS = 32 * NW;
  static constexpr int KT = 16 * NW;                      // keys of a tile (one group per warp)
  static constexpr int SWB = ROWB < 128 ? ROWB : 128;     // swizzle span
  static constexpr int REGIONS = ROWB / SWB;
  static constexpr int REGION = 16 * SWB;
  static constexpr int KV = 16 * ROWB;                    // bytes of 16 rows
  static constexpr int FIT = (E4M3 ? 184 : 192) * 1024 / (NW * 2 * KV);
  static constexpr int S = FIT > 8 ? 8 : FIT;             // stages of a warp's ring
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_JOIN = NW * S * 2 * KV;        // joining: O of half the warps, fp32 [NW / 2][16][D]
  static constexpr int OFF_ML = OFF_JOIN + NW / 2 * 16 * D * 4;  // their m and l [NW / 2][2][16]
  static constexpr int OFF_SCALE = OFF_ML + NW / 2 * 32 * 4;     // e4m3: K and V scale bytes [NW][S][32]
  static constexpr int OFF_BAR = OFF_SCALE + (E4M3 ? NW * S * 32 : 0);
  static constexpr int OFF_PLAN = OFF_BAR + NW * S * 8;
  static constexpr int OFF_ABORT = OFF_PLAN + static_cast<int>(sizeof(PlanScratch));
  static constexpr int SMEM = OFF_ABORT + 16 + 1024;      // + slack for 1024-byte alignment
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(S >= 2 && OFF_SCALE % 16 == 0 && OFF_BAR % 8 == 0 && OFF_PLAN % 8 == 0, "layout");
  static constexpr uint32_t TX = 2 * KV + (E4M3 ? 32 : 0);
  static constexpr int KS = D / 16;                       // K steps of Q K^T = pairs of 8-column output tiles
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a b, m16n8k16, fp32 accumulators; bf16 or fp16 operands.
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct FewParams {
  PagedFwdArgs a;
  bool scan;  // look for infinities and NaN in the chunks' new V (see fa_paged_mend_kernel)
  PagedWs ws;
  int* status;
  unsigned long long limit_ns;
};

// Tiles of KT keys of one head of sequence b in this kernel (0: not one of its sequences).
template <int KT>
__device__ __forceinline__ int few_tiles(const PagedFwdArgs& a, const PagedSeq& s) {
  if (s.n < 1 || s.n > a.max_rows || s.n > kFewRows || s.n * a.group > kFewRows) return 0;
  return s.len <= KT ? 1 : (s.len + KT - 1) / KT;  // without keys too: the rows get their zeros
}

// Walks the tiles of a CTA's share.
template <int KT>
struct FewCursor {
  int b, head, j, nt;
  PagedSeq s;
  long long left;
  __device__ __forceinline__ void load(const PagedFwdArgs& a) {
    bool bad;
    s = paged_seq(a.pb, a.kv.ps_log2, b, bad);
    nt = few_tiles<KT>(a, s);
  }
  __device__ __forceinline__ void start(const PagedFwdArgs& a, const PlanShare& p) {
    left = p.end - p.start;
    b = p.b;
    if (left == 0) return;
    load(a);
    head = static_cast<int>(p.offset / nt);
    j = static_cast<int>(p.offset - static_cast<long long>(head) * nt);
  }
  // Move on by k tiles of the present unit.
  __device__ __forceinline__ void advance(const PagedFwdArgs& a, int k) {
    left -= k;
    j += k;
    if (left == 0 || j < nt) return;
    j = 0;
    if (++head < a.kv.heads) return;
    head = 0;
    do {
      ++b;
      load(a);
    } while (nt == 0);
  }
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(FewCfg<D, E4M3>::THREADS, 1)
    fa_paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ FewParams p) {
  using C = FewCfg<D, E4M3>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const PagedFwdArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, jq = lane & 3;  // row (and row + 8) and column pair of mma fragments
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_ABORT);
  const WaitGuard guard{abort_flag, p.status, p.limit_ns};
  const uint32_t bars = base + C::OFF_BAR + warp * C::S * 8;
  const uint32_t ring = base + C::OFF_KV + warp * C::S * 2 * C::KV;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NW * C::S; ++i) mbar_init(base + C::OFF_BAR + 8 * i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (blockIdx.x == 0) {
    // Sequences that are not there, or that have more rows than the caller said.
    bool any = false;
    for (int b = threadIdx.x; b < a.pb.B; b += C::THREADS) {
      bool bad;
      const PagedSeq s = paged_seq(a.pb, a.kv.ps_log2, b, bad);
      any = any || bad || s.n > a.max_rows;
    }
    if (any) atomicOr(p.status, kStatusBadBatch);
  }
  __syncthreads();
  const PlanShare share = plan_share<C::THREADS>(
      a.pb.B, gridDim.x, blockIdx.x,
      [&](int b) -> long long {
        bool bad;
        return static_cast<long long>(a.kv.heads) * few_tiles<C::KT>(a, paged_seq(a.pb, a.kv.ps_log2, b, bad));
      },
      *reinterpret_cast<PlanScratch*>(gbase + C::OFF_PLAN));

  // ---- the warp's loads
  FewCursor<C::KT> ahead;  // next group to load
  ahead.start(a, share);
  uint32_t issued = 0, done = 0;
  const uint64_t policy = policy_evict_first();  // a unit's K and V are read once
  auto issue = [&]() {
    while (ahead.left > 0 && ahead.j * C::KT + warp * 16 >= ahead.s.len) ahead.advance(a, 1);
    if (ahead.left == 0) return;
    const int key0 = ahead.j * C::KT + warp * 16;
    if (lane == 0) {
      const int page = paged_page(a.pb, a.kv, ahead.b, key0);
      const int slot = key0 & ((1 << a.kv.ps_log2) - 1);
      if (page < 0) atomicOr(p.status, kStatusBadBatch);
      // A page that is not there reads as zeros (a coordinate outside the tensor).
      const int pg = page < 0 ? a.kv.num_pages : page;
      const uint32_t st = issued % C::S;
      const uint32_t bar = bars + 8 * st;
      const uint32_t dst = ring + st * 2 * C::KV;
      mbar_arrive_expect_tx(bar, E4M3 && page < 0 ? 2 * C::KV : C::TX);
#pragma unroll
      for (int r = 0; r < C::REGIONS; ++r) {
        tma_load_4d(dst + r * C::REGION, &tm_k, bar, r * (C::SWB / C::EB), slot, ahead.head, pg, policy);
        tma_load_4d(dst + C::KV + r * C::REGION, &tm_v, bar, r * (C::SWB / C::EB), slot, ahead.head, pg, policy);
      }
      if (E4M3 && page >= 0) {
        const uint32_t sc = base + C::OFF_SCALE + (warp * C::S + st) * 32;
        const long long off = ((static_cast<long long>(page) * a.kv.heads + ahead.head) << a.kv.ps_log2) + slot;
        bulk_load(sc, a.kv.k_scale + off, 16, bar);
        bulk_load(sc + 16, a.kv.v_scale + off, 16, bar);
      }
    }
    ++issued;
    ahead.advance(a, 1);
  };
#pragma unroll 1
  for (int i = 0; i < C::S; ++i) issue();

  // ---- units
  FewCursor<C::KT> at;
  at.start(a, share);
  bool ok = true;
  bool recorded = false;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  // Swizzled place of 16-byte unit `unit` of row `row` in a K or V tile of a stage.
  auto place = [](uint32_t row, uint32_t unit) -> uint32_t {
    constexpr uint32_t U = C::SWB / 16;
    const uint32_t x = C::SWB == 128 ? row & 7 : C::SWB == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
    return (unit / U) * C::REGION + row * C::SWB + (((unit % U) ^ x) << 4);
  };

#pragma unroll 1
  while (at.left > 0) {
    const PagedSeq s = at.s;
    const int rows = s.n * a.group;
    const int j0 = at.j;
    const int j1 = at.left < at.nt - j0 ? j0 + static_cast<int>(at.left) : at.nt;
    // This thread's rows g and g + 8: query token and head, last visible key.
    int lim[2];
    const __nv_bfloat16* qp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      const int tok = r / a.group;
      lim[i] = r >= rows ? -1 : a.causal ? s.len - s.n + tok : s.len - 1;
      qp[i] = r >= rows ? nullptr : a.q + static_cast<long long>(s.row0 + tok) * a.qs[0] +
                                        static_cast<long long>(at.head * a.group + r % a.group) * a.qs[1];
    }
    // Rows that exist see the keys up to here (row 0 sees the fewest).
    const int lim_all = a.causal ? s.len - s.n : s.len - 1;
    uint32_t qf[C::KS][4];
    float rowf[2] = {scale_log2, scale_log2};
    if constexpr (!E4M3) {
#pragma unroll
      for (int k = 0; k < C::KS; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const __nv_bfloat16* q = qp[x & 1];
          qf[k][x] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 * (x >> 1) + 2 * jq) : 0u;
        }
    } else {
      // fp16 elements 16k + 4 jq .. + 3 (the order in which an e4m3 fragment of K holds its elements).
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint2 w[C::KS];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
          w[k] = qp[i] ? *reinterpret_cast<const uint2*>(qp[i] + 16 * k + 4 * jq) : make_uint2(0u, 0u);
          top = __vmaxu2(top, __vmaxu2(w[k].x & 0x7fff7fffu, w[k].y & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = static_cast<int>(top >> 7);  // biased exponent of the row's largest element
        e = e == 255 ? 140 : e < 27 ? 27 : e;
        const float f = __uint_as_float(static_cast<uint32_t>(267 - e) << 23);  // 2^(13 - (e - 127))
        rowf[i] = scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 13) << 23);
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
          qf[k][i] = pack_f16x2(__uint_as_float(w[k].x << 16) * f, __uint_as_float(w[k].x & 0xffff0000u) * f);
          qf[k][2 + i] = pack_f16x2(__uint_as_float(w[k].y << 16) * f, __uint_as_float(w[k].y & 0xffff0000u) * f);
        }
      }
    }
    float o[2 * C::KS][4];
#pragma unroll
    for (int c = 0; c < 2 * C::KS; ++c)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[c][x] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int vexp = 0;  // e4m3: the largest V scale byte so far; o is in units of 2^(vexp - 127 - 14)

#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      const int key0 = j * C::KT + warp * 16;
      if (key0 >= s.len) break;
      const uint32_t st = done % C::S;
      if (ok) ok = warp_wait_bar(bars + 8 * st, (done / C::S) & 1, guard, kStatusTimeoutLoad);
      if (!ok) break;
      const uint32_t kt = ring + st * 2 * C::KV, vt = kt + C::KV;
      uint8_t* vt_g = gbase + (vt - base);
      const uint8_t* sc = gbase + C::OFF_SCALE + (warp * C::S + st) * 32;
      float x[2][4];  // logits: keys 8t + 2jq, + 1 of rows g (x[t][0..1]) and g + 8 (x[t][2..3])
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][i] = 0.f;
      if constexpr (!E4M3) {
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
          uint32_t b[4];
          ldsm_x4(kt + place((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b);
          mma_16816<false>(x[0], qf[k], b[0], b[1]);
          mma_16816<false>(x[1], qf[k], b[2], b[3]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < C::KS; k += 2) {
          uint32_t b[4];
          ldsm_x4(kt + place((lane & 7) + ((lane >> 4) << 3), k + ((lane >> 3) & 1)), b);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_16816<true>(x[i >> 1], qf[k + (i & 1)], e4m3x2_to_f16x2(static_cast<uint16_t>(b[i])),
                            e4m3x2_to_f16x2(static_cast<uint16_t>(b[i] >> 16)));
        }
      }
      float pf[4] = {1.f, 1.f, 1.f, 1.f};  // e4m3: 2^14 times V's scales of this thread's four keys, in units of 2^(vexp - 127)
      float vdown = 1.f;
      if constexpr (E4M3) {
        uint32_t kb[4], vb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at_key = 8 * (i >> 1) + 2 * jq + (i & 1);
          kb[i] = sc[at_key];
          vb[i] = key0 + at_key < s.len ? sc[16 + at_key] : 0u;
        }
        int top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, vb[i] == 255u ? 0 : static_cast<int>(vb[i]));
        top = max(vexp, __reduce_max_sync(0xffffffffu, top));
        const int fall = top - vexp;  // 0 .. 254
        vdown = fall > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - fall) << 23);
        vexp = top;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 127 + 14 + static_cast<int>(vb[i]) - top;
          pf[i] = vb[i] == 255u ? __uint_as_float(0x7fc00000u) : e < 1 ? 0.f : __uint_as_float(static_cast<uint32_t>(e) << 23);
          const float kf = scale_of_byte(kb[i]);
          x[i >> 1][i & 1] *= rowf[0] * kf;
          x[i >> 1][2 + (i & 1)] *= rowf[1] * kf;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[t][i] *= scale_log2;
      }
      const bool edge = key0 + 15 > lim_all;  // some row does not see some key
      if (edge || rows < kFewRows) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 8 * t + 2 * jq + (i & 1) > lim[i >> 1]) x[t][i] = -INFINITY;
      }
      float alpha[2], pr[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float m_new = fmaxf(m[i], top);
        alpha[i] = m_new == m[i] ? 1.f : ex2(m[i] - m_new);
        m[i] = m_new;
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            pr[t][2 * i + k] = ex2(x[t][2 * i + k] - ref);
            sum += pr[t][2 * i + k];
          }
        l[i] = l[i] * alpha[i] + sum;  // this thread's keys only; joined over the quad at the unit's end
        alpha[i] *= vdown;
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int c = 0; c < 2 * C::KS; ++c) {
          o[c][0] *= alpha[0];
          o[c][1] *= alpha[0];
          o[c][2] *= alpha[1];
          o[c][3] *= alpha[1];
        }
      }
      bool plain = true;  // the products below may meet every value of V
      if (edge) {
        // Slots behind the last token hold anything: their V rows become zeros.
        if (key0 + 16 > s.len) {
          for (int i = lane; i < 16 * (C::ROWB / 16); i += 32) {
            const int row = i / (C::ROWB / 16);
            if (key0 + row >= s.len) st_shared_v4(vt + place(row, i % (C::ROWB / 16)), 0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // before the next load into this stage
        }
        __syncwarp();
        // A token that some rows do not see may hold an infinity or a NaN, and 0 times that is NaN.
        bool odd = false;
        for (int i = lane; i < 16 * (C::ROWB / 16); i += 32) {
          const uint4 v = *reinterpret_cast<const uint4*>(vt_g + place(i / (C::ROWB / 16), i % (C::ROWB / 16)));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (E4M3)
              odd = odd || __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
            else
              odd = odd || __vcmpgeu2(w[k] & 0x7fff7fffu, 0x7f807f80u) != 0;
          }
        }
        plain = !__any_sync(0xffffffffu, odd);
      }
      uint32_t pa[4];
      if constexpr (E4M3) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              y[k] = pr[t][2 * i + k] * pf[2 * t + k];
              // A scale of NaN reaches only the rows that see its token.
              if (edge && key0 + 8 * t + 2 * jq + k > lim[i]) y[k] = 0.f;
              pr[t][2 * i + k] = y[k];
            }
            pa[2 * t + i] = pack_f16x2(y[0], y[1]);
          }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) pa[2 * t + i] = pack_bf16x2(pr[t][2 * i], pr[t][2 * i + 1]);
      }
      if (plain) {
        if constexpr (!E4M3) {
#pragma unroll
          for (int c = 0; c < C::KS; ++c) {
            uint32_t b[4];
            ldsm_x4_t(vt + place(lane & 15, 2 * c + (lane >> 4)), b);
            mma_16816<false>(o[2 * c], pa, b[0], b[1]);
            mma_16816<false>(o[2 * c + 1], pa, b[2], b[3]);
          }
        } else {
          // A transposed fragment holds two columns of two keys; columns 16c + 2u go to tile 2c, 16c + 2u + 1 to 2c + 1.
#pragma unroll
          for (int c = 0; c < C::KS; c += 2) {
            uint32_t b[4];
            ldsm_x4_t(vt + place(lane & 15, c + (lane >> 4)), b);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = __byte_perm(b[2 * h], 0, 0x3120), hi = __byte_perm(b[2 * h + 1], 0, 0x3120);
              mma_16816<true>(o[2 * (c + h)], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(lo)),
                              e4m3x2_to_f16x2(static_cast<uint16_t>(hi)));
              mma_16816<true>(o[2 * (c + h) + 1], pa, e4m3x2_to_f16x2(static_cast<uint16_t>(lo >> 16)),
                              e4m3x2_to_f16x2(static_cast<uint16_t>(hi >> 16)));
            }
          }
        }
      } else {
        // Key by key, and only for the rows that see the key.
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          float pv[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float lo = (i & 1) ? pr[0][2 * r + 1] : pr[0][2 * r];
            const float hi = (i & 1) ? pr[1][2 * r + 1] : pr[1][2 * r];
            pv[r] = __shfl_sync(0xffffffffu, i >= 8 ? hi : lo, (lane & 28) | ((i & 7) >> 1));
          }
          const bool see[2] = {key0 + i <= lim[0], key0 + i <= lim[1]};
#pragma unroll
          for (int c = 0; c < C::KS; ++c) {
            float v[4];  // the columns of o[2c][0], o[2c][1], o[2c + 1][0], o[2c + 1][1]
            if constexpr (!E4M3) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(vt_g + place(i, 2 * c + h) + 4 * jq);
                v[2 * h] = __uint_as_float(w << 16);
                v[2 * h + 1] = __uint_as_float(w & 0xffff0000u);
              }
            } else {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(vt_g + place(i, c) + 4 * jq);
              const uint32_t a0 = e4m3x2_to_f16x2(static_cast<uint16_t>(w)), a1 = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
              const float2 y0 = __half22float2(*reinterpret_cast<const __half2*>(&a0));
              const float2 y1 = __half22float2(*reinterpret_cast<const __half2*>(&a1));
              v[0] = y0.x;
              v[1] = y1.x;
              v[2] = y0.y;
              v[3] = y1.y;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int h = 0; h < 4; ++h)
                if (see[r]) o[2 * c + (h >> 1)][2 * r + (h & 1)] = fmaf(pv[r], v[h], o[2 * c + (h >> 1)][2 * r + (h & 1)]);
          }
        }
      }
      __syncwarp();  // the stage has been read
      ++done;
      issue();
    }
    if constexpr (E4M3) {
      const float f = scale_of_byte(static_cast<uint32_t>(vexp));
#pragma unroll
      for (int c = 0; c < 2 * C::KS; ++c)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[c][x] = o[c][x] * 0x1p-14f * f;
    }
    // The sums' shares of the quad's threads.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    // ---- join the warps: the upper half hands its results to the lower, again and again.
    float* join_o = reinterpret_cast<float*>(gbase + C::OFF_JOIN);
    float* join_ml = reinterpret_cast<float*>(gbase + C::OFF_ML);
#pragma unroll 1
    for (int half = C::NW / 2; half > 0; half >>= 1) {
      if (warp >= half && warp < 2 * half) {
        float* jo = join_o + (warp - half) * 16 * D;
#pragma unroll
        for (int c = 0; c < 2 * C::KS; ++c)
          *reinterpret_cast<float4*>(jo + (c * 32 + lane) * 4) = make_float4(o[c][0], o[c][1], o[c][2], o[c][3]);
        if (jq == 0) {
          float* ml = join_ml + (warp - half) * 32;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ml[g + 8 * i] = m[i];
            ml[16 + g + 8 * i] = l[i];
          }
        }
      }
      __syncthreads();
      if (warp < half) {
        const float* jo = join_o + warp * 16 * D;
        const float* ml = join_ml + warp * 32;
        float mine[2], other[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m2 = ml[g + 8 * i], l2 = ml[16 + g + 8 * i];
          const float top = fmaxf(m[i], m2);
          mine[i] = m[i] == top ? 1.f : ex2(m[i] - top);
          other[i] = m2 == top ? 1.f : ex2(m2 - top);
          m[i] = top;
          l[i] = l[i] * mine[i] + l2 * other[i];
        }
#pragma unroll
        for (int c = 0; c < 2 * C::KS; ++c) {
          const float4 y = *reinterpret_cast<const float4*>(jo + (c * 32 + lane) * 4);
          o[c][0] = o[c][0] * mine[0] + y.x * other[0];
          o[c][1] = o[c][1] * mine[0] + y.y * other[0];
          o[c][2] = o[c][2] * mine[1] + y.z * other[1];
          o[c][3] = o[c][3] * mine[1] + y.w * other[1];
        }
      }
      __syncthreads();
    }
    // ---- the unit's rows, or this CTA's part of them
    const bool whole = j0 == 0 && j1 == at.nt;
    if (warp == 0 && *abort_flag == 0) {
      if (whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = g + 8 * i;
          if (r >= rows) continue;
          const int row = s.row0 + r / a.group, hq = at.head * a.group + r % a.group;
          const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
          __nv_bfloat16* dst = a.o + static_cast<long long>(row) * a.os[0] + static_cast<long long>(hq) * a.os[1];
#pragma unroll
          for (int c = 0; c < C::KS; ++c) {
            const float y0 = o[2 * c][2 * i] * inv, y1 = o[2 * c][2 * i + 1] * inv;
            const float y2 = o[2 * c + 1][2 * i] * inv, y3 = o[2 * c + 1][2 * i + 1] * inv;
            if constexpr (!E4M3) {
              *reinterpret_cast<uint32_t*>(dst + 16 * c + 2 * jq) = pack_bf16x2(y0, y1);
              *reinterpret_cast<uint32_t*>(dst + 16 * c + 8 + 2 * jq) = pack_bf16x2(y2, y3);
            } else {
              *reinterpret_cast<uint2*>(dst + 16 * c + 4 * jq) = make_uint2(pack_bf16x2(y0, y2), pack_bf16x2(y1, y3));
            }
          }
          if (jq == 0) a.lse[static_cast<long long>(hq) * a.pb.rows + row] = (m[i] + log2f(l[i])) * 0.69314718055994531f;
        }
      } else {
        float* part = p.ws.few_part + (blockIdx.x * 2 + (j0 == 0 ? 1 : 0)) * few_floats(D);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = g + 8 * i;
          float* dst = part + 32 + r * D;
#pragma unroll
          for (int c = 0; c < C::KS; ++c) {
            if constexpr (!E4M3) {
              *reinterpret_cast<float2*>(dst + 16 * c + 2 * jq) = make_float2(o[2 * c][2 * i], o[2 * c][2 * i + 1]);
              *reinterpret_cast<float2*>(dst + 16 * c + 8 + 2 * jq) = make_float2(o[2 * c + 1][2 * i], o[2 * c + 1][2 * i + 1]);
            } else {
              *reinterpret_cast<float4*>(dst + 16 * c + 4 * jq) =
                  make_float4(o[2 * c][2 * i], o[2 * c + 1][2 * i], o[2 * c][2 * i + 1], o[2 * c + 1][2 * i + 1]);
            }
          }
          if (jq == 0) {
            part[r] = m[i];
            part[16 + r] = l[i];
          }
        }
        if (j0 == 0) {
          const long long last = share.end - at.left + at.nt - 1;  // the unit's last tile
          if (lane == 0)
            p.ws.few_rec[blockIdx.x] =
                PlanRecord{at.b, at.head, 0, plan_cta_of(last, share.total, share.ctas) - static_cast<int>(blockIdx.x)};
          recorded = true;
        }
      }
    }
    at.advance(a, j1 - j0);
  }
  if (threadIdx.x == 0 && !recorded) p.ws.few_rec[blockIdx.x].b = -1;
  if (p.scan) {
    // Rows of the chunk kernel's sequences, dealt out evenly; a thread takes 16 bytes of a row at a time.
    __syncthreads();
    const PlanShare part = plan_share<C::THREADS>(
        a.pb.B, gridDim.x, blockIdx.x,
        [&](int b) -> long long {
          bool bad;
          const PagedSeq s = paged_seq(a.pb, a.kv.ps_log2, b, bad);
          return s.n > 1 && s.n <= a.max_rows && few_tiles<C::KT>(a, s) == 0 ? s.n : 0;
        },
        *reinterpret_cast<PlanScratch*>(gbase + C::OFF_PLAN));
    long long rest = part.end - part.start;
    int b = part.b, row = static_cast<int>(part.offset);
    bool odd = false;
    while (rest > 0) {
      bool bad;
      const PagedSeq s = paged_seq(a.pb, a.kv.ps_log2, b, bad);
      const bool chunk = s.n > 1 && s.n <= a.max_rows && few_tiles<C::KT>(a, s) == 0;
      const int take = !chunk ? 0 : rest < s.n - row ? static_cast<int>(rest) : s.n - row;
      constexpr int UPR = C::ROWB / 16;
      const long long items = static_cast<long long>(take) * a.kv.heads * UPR;
#pragma unroll 4
      for (long long it = threadIdx.x; it < items; it += C::THREADS) {
        const int unit = static_cast<int>(it % UPR);
        const int head = static_cast<int>(it / UPR % a.kv.heads);
        const int pos = s.len - s.n + row + static_cast<int>(it / UPR / a.kv.heads);
        const int page = pos < 0 ? -1 : paged_page(a.pb, a.kv, b, pos);
        if (page < 0) continue;
        const int slot = pos & ((1 << a.kv.ps_log2) - 1);
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.kv.v) +
                                                        (page * a.kv.vs[0] + head * a.kv.vs[1] + slot * a.kv.vs[2]) * C::EB +
                                                        unit * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          odd = odd || (E4M3 ? __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) : __vcmpgeu2(w[k] & 0x7fff7fffu, 0x7f807f80u)) != 0;
        if (E4M3 && unit == 0)
          odd = odd || a.kv.v_scale[((static_cast<long long>(page) * a.kv.heads + head) << a.kv.ps_log2) + slot] == 255;
      }
      rest -= take;
      row = 0;
      ++b;
    }
    const int any = __syncthreads_or(odd);
    if (threadIdx.x == 0) p.ws.odd[blockIdx.x] = any;
  }
  // After a wait that gave up, what was loaded must land before the CTA leaves.
  for (; done < issued; ++done) {
    const uint32_t bar = bars + 8 * (done % C::S);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, (done / C::S) & 1))
      if (globaltimer_ns() - t0 > p.limit_ns) {
        atomicOr(p.status, kStatusTimeoutDrain);
        break;
      }
  }
}

// Joins the parts of units that several CTAs held; block c looks after the unit that CTA c began.
template <int D>
__global__ void __launch_bounds__(128) fa_paged_few_join_kernel(const __grid_constant__ FewParams p) {
  pdl_wait();
  const PagedFwdArgs& a = p.a;
  const PlanRecord rec = p.ws.few_rec[blockIdx.x];
  if (rec.b < 0) return;
  bool bad;
  const PagedSeq s = paged_seq(a.pb, a.kv.ps_log2, rec.b, bad);
  const int rows = s.n * a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto part = [&](int i) -> const float* {
    return p.ws.few_part + ((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * few_floats(D);
  };
  for (int r = warp; r < rows; r += 4) {
    float m = -INFINITY;
    for (int i = 0; i <= rec.more; ++i) m = fmaxf(m, part(i)[r]);
    float l = 0.f, o[D / 32] = {};
    for (int i = 0; i <= rec.more; ++i) {
      const float* x = part(i);
      const float f = x[r] == m ? 1.f : ex2(x[r] - m);
      l += x[16 + r] * f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[c] += x[32 + r * D + c * 32 + lane] * f;
    }
    const int row = s.row0 + r / a.group, hq = rec.head * a.group + r % a.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16* dst = a.o + static_cast<long long>(row) * a.os[0] + static_cast<long long>(hq) * a.os[1];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) dst[c * 32 + lane] = __float2bfloat16_rn(o[c] * inv);
    if (lane == 0) a.lse[static_cast<long long>(hq) * a.pb.rows + row] = (m + log2f(l)) * 0.69314718055994531f;
  }
}

template <int D, bool E4M3>
int launch_paged_few_impl(const PagedFwdArgs& a, const LaunchCtx& ctx) {
  using C = FewCfg<D, E4M3>;
  auto kernel = fa_paged_few_kernel<D, E4M3>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return static_cast<int>(e);
  CUtensorMap mk, mv;
  const long long dims[4] = {D, 1LL << a.kv.ps_log2, a.kv.heads, a.kv.num_pages};
  const long long ks[3] = {a.kv.ks[2], a.kv.ks[1], a.kv.ks[0]}, vs[3] = {a.kv.vs[2], a.kv.vs[1], a.kv.vs[0]};
  if (encode_paged_map(&mk, a.kv.k, C::EB, dims, ks, C::SWB / C::EB, 16, 1, C::SWB, true) != 0) return -1;
  if (encode_paged_map(&mv, a.kv.v, C::EB, dims, vs, C::SWB / C::EB, 16, 1, C::SWB, true) != 0) return -1;
  FewParams p;
  p.a = a;
  p.scan = a.causal && static_cast<long long>(a.max_rows) * a.group > kFewRows;
  p.ws = paged_ws(a.workspace, D);
  p.status = ctx.status;
  p.limit_ns = ctx.limit_ns;
  const int grid = ctx.num_sms < kPlanCtas ? ctx.num_sms : kPlanCtas;
  kernel<<<grid, C::THREADS, C::SMEM, ctx.stream>>>(mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(128);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, fa_paged_few_join_kernel<D>, p));
}

template <int D>
int launch_paged_few(const PagedFwdArgs& a, const LaunchCtx& ctx) {
  return a.e4m3 ? launch_paged_few_impl<D, true>(a, ctx) : launch_paged_few_impl<D, false>(a, ctx);
}

}  // namespace fa
