// Attention of few rows over a paged cache: sequences whose rows (n_b tokens x
// the query heads of one key/value head) fit 16 (or 32), decoding above all.
//
//   s_ij = scale q_i . k_j,  m, l: running maximum and sum,  o_i = sum_j p_ij v_j / l_i
//
// Bound by reading K and V once, so everything serves to keep reads in flight:
//  * one CTA per SM; each warp is a pipeline of its own: it takes every NW-th
//    group of KG keys, loads K and V of a group with TMA boxes of 16 or 32 tokens
//    (a page holds whole boxes) into its own ring of stages, and issues the
//    load S groups ahead, across the borders of units; no barrier between
//    warps but where a unit ends;
//  * the rows are the M of mma.sync m16n8k16, one or two tiles of 16 (a tcgen05
//    tile of 128 rows would multiply mostly padding, and its softmax would cost
//    128 rows); two tiles share every K and V fragment;
//  * softmax state m, l and the output stay in registers; at a unit's end the
//    warps' results are joined in shared memory, in a fixed order.
// e4m3 pages: codes are exact in fp16, so S = Q K^T runs in fp16 with the codes
// as they are and every q row multiplied by a power of two that brings its
// largest element to [2^13, 2^14) (exact down to 2^-37 of that element); the
// rows' and the keys' powers of two multiply the fp32 result.  V's scales go
// into P: P' = p 2^(e_j - E) 2^14 in fp16, E the largest exponent so far (kept
// like the maximum: a larger one rescales the output, exactly).  P' is rounded
// to 11 bits down to p 2^(e_j - E) = 2^-28, finer than bf16's 8.  A group is 32
// keys there (16 in bf16): half the bytes a key, so what a group costs besides
// its products has to serve twice the keys.
#pragma once

#include "fa_paged_plan.cuh"

namespace fa {

template <int D, bool E4M3, int MT>
struct FewCfg {
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int ROWB = D * EB;                     // bytes of a K or V row
  static constexpr int NW = D == 256 ? 4 : 8;             // warps; d = 256 keeps 128 output registers a thread
  static constexpr int THREADS = 32 * NW;
  static constexpr int KG = E4M3 ? 32 : 16;               // keys of a group
  static constexpr int NG = KG / 16;
  static constexpr int KT = KG * NW;                      // keys of a tile (one group per warp)
  static constexpr int SWB = ROWB < 128 ? ROWB : 128;     // swizzle span
  static constexpr int REGIONS = ROWB / SWB;
  static constexpr int REGION = KG * SWB;
  static constexpr int KV = KG * ROWB;                    // bytes of a group of K or V
  static constexpr int JOIN = NW / 2 * 16 * D * 4;        // joining: O of half the warps, fp32 [NW / 2][16][D]
  static constexpr int QS = MT > 1 ? MT * 16 * D * 2 : 0; // two tiles: q in shared memory (registers hold 128 outputs)
  static constexpr int MISC = 6 * 1024;
  static constexpr int FIT = (226 * 1024 - JOIN - QS - MISC) / (NW * 2 * KV);
  static constexpr int S = FIT > 8 ? 8 : FIT;             // stages of a warp's ring
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_Q = NW * S * 2 * KV;
  static constexpr int OFF_JOIN = OFF_Q + QS;
  static constexpr int OFF_ML = OFF_JOIN + JOIN;          // their m and l [NW / 2][2][16]
  static constexpr int OFF_ROWF = OFF_ML + NW / 2 * 32 * 4;      // e4m3, two tiles: the rows' factors [MT * 16]
  static constexpr int OFF_SCALE = OFF_ROWF + 128;               // e4m3: K and V scale bytes [NW][S][2][KG]
  static constexpr int OFF_BAR = OFF_SCALE + (E4M3 ? NW * S * 2 * KG : 0);
  static constexpr int OFF_PLAN = OFF_BAR + NW * S * 8;
  static constexpr int OFF_ABORT = OFF_PLAN + static_cast<int>(sizeof(PlanScratch));
  static constexpr int SMEM = OFF_ABORT + 16 + 1024;      // + slack for 1024-byte alignment
  static_assert(OFF_ABORT + 16 - OFF_ML <= MISC && SMEM <= 227 * 1024, "shared memory budget");
  static_assert(S >= 2 && OFF_SCALE % 16 == 0 && OFF_BAR % 8 == 0 && OFF_PLAN % 8 == 0, "layout");
  static_assert(MT == 1 || (MT == 2 && D <= 128), "row tiles");
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
  PagedWs ws;
  int* status;
  unsigned long long limit_ns;
  int box;  // tokens of a K/V box: 16, or 32 where groups and pages hold as many
};

// Tiles of KT keys of one head of sequence b in this kernel (0: not one of its sequences).
template <int KT>
__device__ __forceinline__ int few_tiles(const PagedFwdArgs& a, const PagedSeq& s) {
  if (s.n < 1 || s.n > a.max_rows || s.n > kFewMost || s.n * a.group > a.few_rows) return 0;
  return s.len <= KT ? 1 : (s.len + KT - 1) / KT;  // without keys too: the rows get their zeros
}

// Walks the tiles of a CTA's share.
template <int KT>
struct FewCursor {
  int b, head, j, nt, left;
  PagedSeq s;
  __device__ __forceinline__ void load(const PagedFwdArgs& a) {
    bool bad;
    s = paged_seq(a.pb, a.kv.ps_log2, b, bad);
    nt = few_tiles<KT>(a, s);
  }
  __device__ __forceinline__ void start(const PagedFwdArgs& a, const PlanShare& p) {
    left = static_cast<int>(p.end - p.start);  // (W / 152 tiles: W < 2^38)
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

template <int D, bool E4M3, int MT>
__global__ void __launch_bounds__(FewCfg<D, E4M3, MT>::THREADS, 1)
    fa_paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ FewParams p) {
  using C = FewCfg<D, E4M3, MT>;
  constexpr int NG = C::NG;
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
  const int box_log2 = p.box == 32 ? 5 : 4;
  const int slot_mask = (1 << a.kv.ps_log2) - 1;
  auto issue = [&]() {
    while (ahead.left > 0 && ahead.j * C::KT + warp * C::KG >= ahead.s.len) ahead.advance(a, 1);
    if (ahead.left == 0) return;
    const int key0 = ahead.j * C::KT + warp * C::KG;
    const uint32_t st = issued % C::S;
    const uint32_t bar = bars + 8 * st;
    // Boxes that hold keys of the sequence; lanes 2i and 2i + 1 load K and V of box i.
    const int nbox = NG == 1 ? 1 : (min(C::KG, ahead.s.len - key0) + p.box - 1) >> box_log2;
    if (lane == 0) mbar_arrive_expect_tx(bar, 2 * (nbox << box_log2) * (C::ROWB + (E4M3 ? 1 : 0)));
    __syncwarp();
    if (lane < 2 * nbox) {
      const int is_v = lane & 1, row = (lane >> 1) << box_log2;
      const int page = paged_page(a.pb, a.kv, ahead.b, key0 + row);
      const int slot = (key0 + row) & slot_mask;
      if (page < 0) atomicOr(p.status, kStatusBadBatch);
      // A page that is not there reads as zeros (a coordinate outside the tensor).
      const int pg = page < 0 ? a.kv.num_pages : page;
      const uint32_t dst = ring + st * 2 * C::KV + is_v * C::KV + row * C::SWB;
#pragma unroll
      for (int r = 0; r < C::REGIONS; ++r)
        tma_load_4d(dst + r * C::REGION, is_v ? &tm_v : &tm_k, bar, r * (C::SWB / C::EB), slot, ahead.head, pg, policy);
      if constexpr (E4M3) {
        const uint32_t sc = base + C::OFF_SCALE + ((warp * C::S + st) * 2 + is_v) * C::KG + row;
        // (For a page that is not there any scales do.)
        const long long off = ((static_cast<long long>(max(page, 0)) * a.kv.heads + ahead.head) << a.kv.ps_log2) + slot;
        bulk_load(sc, (is_v ? a.kv.v_scale : a.kv.k_scale) + off, p.box, bar);
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
  // The same for q in shared memory (rows of 2 D bytes).
  auto q_place = [](uint32_t row, uint32_t unit) -> uint32_t {
    return row * (D * 2) + ((unit ^ (D >= 64 ? row & 7 : (row >> 1) & 3)) << 4);
  };
  // Scale and fp16 conversion of a row whose largest magnitude has the bf16 bits `top` (see above).
  auto row_scale = [&](uint32_t top, float& rowf) -> float {
    int e = static_cast<int>(top >> 7);  // biased exponent
    e = e == 255 ? 140 : e < 27 ? 27 : e;
    rowf = fmaxf(scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 13) << 23), 0x1p-126f);  // never 0 (times -inf)
    return __uint_as_float(static_cast<uint32_t>(267 - e) << 23);  // 2^(13 - (e - 127))
  };

#pragma unroll 1
  while (at.left > 0) {
    const PagedSeq s = at.s;
    const int rows = s.n * a.group;
    const int j0 = at.j;
    const int j1 = at.left < at.nt - j0 ? j0 + at.left : at.nt;
    // Tile mt's rows of this thread, 16 mt + g and + 8: their last visible key (rows behind the last: any).
    int lim[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * mt + g + 8 * i;
        lim[mt][i] = a.causal && r < rows ? s.len - s.n + r / a.group : s.len - 1;
      }
    auto q_row = [&](int r) -> const __nv_bfloat16* {
      return r >= rows ? nullptr : a.q + static_cast<long long>(s.row0 + r / a.group) * a.qs[0] +
                                       static_cast<long long>(at.head * a.group + r % a.group) * a.qs[1];
    };
    // Rows that exist see the keys up to here (row 0 sees the fewest).
    const int lim_all = a.causal ? s.len - s.n : s.len - 1;
    uint32_t qf[MT == 1 ? C::KS : 1][4];
    float rowf[MT][2];
    if constexpr (MT == 1) {
      if constexpr (!E4M3) {
        const __nv_bfloat16* qp[2] = {q_row(g), q_row(g + 8)};
#pragma unroll
        for (int k = 0; k < C::KS; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const __nv_bfloat16* q = qp[x & 1];
            qf[k][x] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 * (x >> 1) + 2 * jq) : 0u;
          }
        rowf[0][0] = rowf[0][1] = scale_log2;
      } else {
        // fp16 elements 16k + 4 jq .. + 3 (the order in which an e4m3 fragment of K holds its elements).
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const __nv_bfloat16* q = q_row(g + 8 * i);
          uint2 w[C::KS];
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < C::KS; ++k) {
            w[k] = q ? *reinterpret_cast<const uint2*>(q + 16 * k + 4 * jq) : make_uint2(0u, 0u);
            top = __vmaxu2(top, __vmaxu2(w[k].x & 0x7fff7fffu, w[k].y & 0x7fff7fffu));
          }
          top = max(top & 0xffffu, top >> 16);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float f = row_scale(top, rowf[0][i]);
#pragma unroll
          for (int k = 0; k < C::KS; ++k) {
            qf[k][i] = pack_f16x2(__uint_as_float(w[k].x << 16) * f, __uint_as_float(w[k].x & 0xffff0000u) * f);
            qf[k][2 + i] = pack_f16x2(__uint_as_float(w[k].y << 16) * f, __uint_as_float(w[k].y & 0xffff0000u) * f);
          }
        }
      }
    } else {
      // q into shared memory: a warp per row, four elements a lane.
      float* rf = reinterpret_cast<float*>(gbase + C::OFF_ROWF);
      for (int r = warp; r < 16 * MT; r += C::NW) {
        const __nv_bfloat16* q = q_row(r);
        const bool mine = lane < D / 4;
        const uint2 w = q && mine ? *reinterpret_cast<const uint2*>(q + 4 * lane) : make_uint2(0u, 0u);
        uint8_t* dst = gbase + C::OFF_Q;
        if constexpr (!E4M3) {
          if (mine) *reinterpret_cast<uint2*>(dst + q_place(r, lane >> 1) + (lane & 1) * 8) = w;
        } else {
          uint32_t top = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
          top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
          float factor;
          const float f = row_scale(top, factor);
          // Elements 4x, 4x + 1 of a 16-element block stand where a fragment has k = 2x, 2x + 1, the others at 8 + 2x.
          if (mine) {
            const int blk = lane >> 2, x = lane & 3;
            *reinterpret_cast<uint32_t*>(dst + q_place(r, 2 * blk) + 4 * x) =
                pack_f16x2(__uint_as_float(w.x << 16) * f, __uint_as_float(w.x & 0xffff0000u) * f);
            *reinterpret_cast<uint32_t*>(dst + q_place(r, 2 * blk + 1) + 4 * x) =
                pack_f16x2(__uint_as_float(w.y << 16) * f, __uint_as_float(w.y & 0xffff0000u) * f);
          }
          if (lane == 0) rf[r] = factor;
        }
      }
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) rowf[mt][i] = E4M3 ? rf[16 * mt + g + 8 * i] : scale_log2;
    }
    float o[MT][2 * C::KS][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int c = 0; c < 2 * C::KS; ++c)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[mt][c][x] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[mt][i] = -INFINITY;
        l[mt][i] = 0.f;
      }
    }
    int vexp = 0;  // e4m3: the largest V scale byte so far; o is in units of 2^(vexp - 127 - 14)

#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      const int key0 = j * C::KT + warp * C::KG;
      if (key0 >= s.len) break;
      const uint32_t st = done % C::S;
      if (ok) ok = warp_wait_bar(bars + 8 * st, (done / C::S) & 1, guard, kStatusTimeoutLoad);
      if (!ok) break;
      const uint32_t kt = ring + st * 2 * C::KV, vt = kt + C::KV;
      uint8_t* vt_g = gbase + (vt - base);
      // Logits / scale: keys 8t + 2jq, + 1 of rows g (x[.][t][0..1]) and g + 8 (x[.][t][2..3]).
      float x[MT][2 * NG][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int t = 0; t < 2 * NG; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[mt][t][i] = 0.f;
#pragma unroll
      for (int k = 0; k < C::KS; k += E4M3 ? 2 : 1) {
        uint32_t qa[E4M3 ? 2 : 1][MT][4];
#pragma unroll
        for (int h = 0; h < (E4M3 ? 2 : 1); ++h)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if constexpr (MT == 1) {
#pragma unroll
              for (int i = 0; i < 4; ++i) qa[h][mt][i] = qf[k + h][i];
            } else {
              ldsm_x4(base + C::OFF_Q + q_place(16 * mt + (lane & 15), 2 * (k + h) + (lane >> 4)), qa[h][mt]);
            }
          }
#pragma unroll
        for (int sg = 0; sg < NG; ++sg) {
          uint32_t b[4];
          if constexpr (!E4M3) {
            ldsm_x4(kt + place(16 * sg + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_16816<false>(x[mt][2 * sg], qa[0][mt], b[0], b[1]);
              mma_16816<false>(x[mt][2 * sg + 1], qa[0][mt], b[2], b[3]);
            }
          } else {
            ldsm_x4(kt + place(16 * sg + (lane & 7) + ((lane >> 4) << 3), k + ((lane >> 3) & 1)), b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b0 = e4m3x2_to_f16x2(static_cast<uint16_t>(b[i]));
              const uint32_t b1 = e4m3x2_to_f16x2(static_cast<uint16_t>(b[i] >> 16));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma_16816<true>(x[mt][2 * sg + (i >> 1)], qa[i & 1][mt], b0, b1);
            }
          }
        }
      }
      const bool edge = key0 + C::KG - 1 > lim_all;  // some row does not see some key
      float pf[2 * NG][2];  // e4m3: 2^14 times V's scales of this thread's keys, in units of 2^(vexp - 127)
      float vdown = 1.f;
      if constexpr (E4M3) {
        const uint8_t* sc = gbase + C::OFF_SCALE + (warp * C::S + st) * 2 * C::KG;
        int vb[2 * NG][2], top = 0;
#pragma unroll
        for (int t = 0; t < 2 * NG; ++t) {
          const uint32_t k2 = *reinterpret_cast<const uint16_t*>(sc + 8 * t + 2 * jq);
          const uint32_t v2 = *reinterpret_cast<const uint16_t*>(sc + C::KG + 8 * t + 2 * jq);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float kf = scale_of_byte((k2 >> (8 * i)) & 255u);
            vb[t][i] = (v2 >> (8 * i)) & 255u;
            if (edge && key0 + 8 * t + 2 * jq + i >= s.len) vb[t][i] = 0;
            top = max(top, vb[t][i] == 255 ? 0 : vb[t][i]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              x[mt][t][i] *= kf;
              x[mt][t][2 + i] *= kf;
            }
          }
        }
        top = max(vexp, __reduce_max_sync(0xffffffffu, top));
        const int fall = top - vexp;  // 0 .. 254
        vdown = fall > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - fall) << 23);
        vexp = top;
#pragma unroll
        for (int t = 0; t < 2 * NG; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            pf[t][i] = vb[t][i] == 255 ? __uint_as_float(0x7fc00000u)
                                       : __uint_as_float(static_cast<uint32_t>(max(127 + 14 + vb[t][i] - top, 0)) << 23);
      }
      uint32_t pa[MT][NG][4];
      float pr[MT][2 * NG][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (edge) {
#pragma unroll
          for (int t = 0; t < 2 * NG; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + 8 * t + 2 * jq + (i & 1) > lim[mt][i >> 1]) x[mt][t][i] = -INFINITY;
        }
        float alpha[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = fmaxf(x[mt][0][2 * i], x[mt][0][2 * i + 1]);
#pragma unroll
          for (int t = 1; t < 2 * NG; ++t) top = fmax3(top, x[mt][t][2 * i], x[mt][t][2 * i + 1]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float m_new = fmaxf(m[mt][i], top * rowf[mt][i]);
          alpha[i] = m_new == m[mt][i] ? 1.f : ex2(m[mt][i] - m_new);
          m[mt][i] = m_new;
          const float ref = m_new == -INFINITY ? 0.f : -m_new;
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 2 * NG; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float y = ex2(fmaf(x[mt][t][2 * i + k], rowf[mt][i], ref));
              sum += y;
              pr[mt][t][2 * i + k] = y;
            }
          l[mt][i] = l[mt][i] * alpha[i] + sum;  // this thread's keys only; joined over the quad at the unit's end
          alpha[i] *= vdown;
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int c = 0; c < 2 * C::KS; ++c) {
            o[mt][c][0] *= alpha[0];
            o[mt][c][1] *= alpha[0];
            o[mt][c][2] *= alpha[1];
            o[mt][c][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int t = 0; t < 2 * NG; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (E4M3) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                pr[mt][t][2 * i + k] *= pf[t][k];
                // A scale of NaN reaches only the rows that see its token.
                if (edge && key0 + 8 * t + 2 * jq + k > lim[mt][i]) pr[mt][t][2 * i + k] = 0.f;
              }
              pa[mt][t >> 1][2 * (t & 1) + i] = pack_f16x2(pr[mt][t][2 * i], pr[mt][t][2 * i + 1]);
            } else {
              pa[mt][t >> 1][2 * (t & 1) + i] = pack_bf16x2(pr[mt][t][2 * i], pr[mt][t][2 * i + 1]);
            }
          }
      }
      bool plain = true;  // the products below may meet every value of V
      if (edge) {
        // Slots behind the last token hold anything: their V rows become zeros.
        if (key0 + C::KG > s.len) {
          for (int i = lane; i < C::KG * (C::ROWB / 16); i += 32) {
            const int row = i / (C::ROWB / 16);
            if (key0 + row >= s.len) st_shared_v4(vt + place(row, i % (C::ROWB / 16)), 0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // before the next load into this stage
        }
        __syncwarp();
        // A token that some rows do not see may hold an infinity or a NaN, and 0 times that is NaN.
        bool odd = false;
        for (int i = lane; i < C::KG * (C::ROWB / 16); i += 32) {
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
      if (plain) {
#pragma unroll
        for (int sg = 0; sg < NG; ++sg) {
#pragma unroll
          for (int c = 0; c < C::KS; c += E4M3 ? 2 : 1) {
            uint32_t b[4];
            if constexpr (!E4M3) {
              ldsm_x4_t(vt + place(16 * sg + (lane & 15), 2 * c + (lane >> 4)), b);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_16816<false>(o[mt][2 * c], pa[mt][sg], b[0], b[1]);
                mma_16816<false>(o[mt][2 * c + 1], pa[mt][sg], b[2], b[3]);
              }
            } else {
              // A transposed fragment holds two columns of two keys; columns 16c + 2u go to tile 2c, 16c + 2u + 1 to 2c + 1.
              ldsm_x4_t(vt + place(16 * sg + (lane & 15), c + (lane >> 4)), b);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t lo = __byte_perm(b[2 * h], 0, 0x3120), hi = __byte_perm(b[2 * h + 1], 0, 0x3120);
                const uint32_t b0 = e4m3x2_to_f16x2(static_cast<uint16_t>(lo));
                const uint32_t b1 = e4m3x2_to_f16x2(static_cast<uint16_t>(hi));
                const uint32_t b2 = e4m3x2_to_f16x2(static_cast<uint16_t>(lo >> 16));
                const uint32_t b3 = e4m3x2_to_f16x2(static_cast<uint16_t>(hi >> 16));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  mma_16816<true>(o[mt][2 * (c + h)], pa[mt][sg], b0, b1);
                  mma_16816<true>(o[mt][2 * (c + h) + 1], pa[mt][sg], b2, b3);
                }
              }
            }
          }
        }
      } else {
        // Key by key, and only for the rows that see the key.
#pragma unroll
        for (int sg = 0; sg < NG; ++sg)
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          const int key = 16 * sg + i;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float pv[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float lo = (i & 1) ? pr[mt][2 * sg][2 * r + 1] : pr[mt][2 * sg][2 * r];
              const float hi = (i & 1) ? pr[mt][2 * sg + 1][2 * r + 1] : pr[mt][2 * sg + 1][2 * r];
              pv[r] = __shfl_sync(0xffffffffu, i >= 8 ? hi : lo, (lane & 28) | ((i & 7) >> 1));
            }
            const bool see[2] = {key0 + key <= lim[mt][0], key0 + key <= lim[mt][1]};
#pragma unroll
            for (int c = 0; c < C::KS; ++c) {
              float v[4];  // the columns of o[2c][0], o[2c][1], o[2c + 1][0], o[2c + 1][1]
              if constexpr (!E4M3) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t w = *reinterpret_cast<const uint32_t*>(vt_g + place(key, 2 * c + h) + 4 * jq);
                  v[2 * h] = __uint_as_float(w << 16);
                  v[2 * h + 1] = __uint_as_float(w & 0xffff0000u);
                }
              } else {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(vt_g + place(key, c) + 4 * jq);
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
                  if (see[r])
                    o[mt][2 * c + (h >> 1)][2 * r + (h & 1)] = fmaf(pv[r], v[h], o[mt][2 * c + (h >> 1)][2 * r + (h & 1)]);
            }
          }
        }
      }
      __syncwarp();  // the stage has been read
      ++done;
      issue();
    }
    const bool whole = j0 == 0 && j1 == at.nt;
    const float vf = E4M3 ? scale_of_byte(static_cast<uint32_t>(vexp)) : 1.f;
    float* join_o = reinterpret_cast<float*>(gbase + C::OFF_JOIN);
    float* join_ml = reinterpret_cast<float*>(gbase + C::OFF_ML);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if constexpr (E4M3) {
#pragma unroll
        for (int c = 0; c < 2 * C::KS; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[mt][c][k] = o[mt][c][k] * 0x1p-14f * vf;
      }
      // The sums' shares of the quad's threads.
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 1);
        l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 2);
      }
      // ---- join the warps: the upper half hands its results to the lower, again and again.
#pragma unroll 1
      for (int half = C::NW / 2; half > 0; half >>= 1) {
        if (warp >= half && warp < 2 * half) {
          float* jo = join_o + (warp - half) * 16 * D;
#pragma unroll
          for (int c = 0; c < 2 * C::KS; ++c)
            *reinterpret_cast<float4*>(jo + (c * 32 + lane) * 4) =
                make_float4(o[mt][c][0], o[mt][c][1], o[mt][c][2], o[mt][c][3]);
          if (jq == 0) {
            float* ml = join_ml + (warp - half) * 32;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              ml[g + 8 * i] = m[mt][i];
              ml[16 + g + 8 * i] = l[mt][i];
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
            const float top = fmaxf(m[mt][i], m2);
            mine[i] = m[mt][i] == top ? 1.f : ex2(m[mt][i] - top);
            other[i] = m2 == top ? 1.f : ex2(m2 - top);
            m[mt][i] = top;
            l[mt][i] = l[mt][i] * mine[i] + l2 * other[i];
          }
#pragma unroll
          for (int c = 0; c < 2 * C::KS; ++c) {
            const float4 y = *reinterpret_cast<const float4*>(jo + (c * 32 + lane) * 4);
            o[mt][c][0] = o[mt][c][0] * mine[0] + y.x * other[0];
            o[mt][c][1] = o[mt][c][1] * mine[0] + y.y * other[0];
            o[mt][c][2] = o[mt][c][2] * mine[1] + y.z * other[1];
            o[mt][c][3] = o[mt][c][3] * mine[1] + y.w * other[1];
          }
        }
        __syncthreads();
      }
      // ---- the unit's rows, or this CTA's part of them
      if (warp == 0 && *abort_flag == 0) {
        float* part = p.ws.few_part + (blockIdx.x * 2 + (j0 == 0 ? 1 : 0)) * part_floats(kFewMost, D);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 16 * mt + g + 8 * i;
          if (r >= rows) continue;
          const int row = s.row0 + r / a.group, hq = at.head * a.group + r % a.group;
          const float inv = l[mt][i] == 0.f ? 0.f : 1.f / l[mt][i];
          const float lsum = m[mt][i] + log2f(l[mt][i]);
          __nv_bfloat16* dst = a.o + static_cast<long long>(row) * a.os[0] + static_cast<long long>(hq) * a.os[1];
          float* pdst = part + kFewMost + r * D;
#pragma unroll
          for (int c = 0; c < C::KS; ++c) {
            const float y0 = o[mt][2 * c][2 * i] * inv, y1 = o[mt][2 * c][2 * i + 1] * inv;
            const float y2 = o[mt][2 * c + 1][2 * i] * inv, y3 = o[mt][2 * c + 1][2 * i + 1] * inv;
            if (whole) {
              if constexpr (!E4M3) {
                *reinterpret_cast<uint32_t*>(dst + 16 * c + 2 * jq) = pack_bf16x2(y0, y1);
                *reinterpret_cast<uint32_t*>(dst + 16 * c + 8 + 2 * jq) = pack_bf16x2(y2, y3);
              } else {
                *reinterpret_cast<uint2*>(dst + 16 * c + 4 * jq) = make_uint2(pack_bf16x2(y0, y2), pack_bf16x2(y1, y3));
              }
            } else {
              if constexpr (!E4M3) {
                *reinterpret_cast<float2*>(pdst + 16 * c + 2 * jq) = make_float2(y0, y1);
                *reinterpret_cast<float2*>(pdst + 16 * c + 8 + 2 * jq) = make_float2(y2, y3);
              } else {
                *reinterpret_cast<float4*>(pdst + 16 * c + 4 * jq) = make_float4(y0, y2, y1, y3);
              }
            }
          }
          if (jq == 0) {
            if (whole)
              a.lse[static_cast<long long>(hq) * a.pb.rows + row] = lsum * 0.69314718055994531f;
            else
              part[r] = lsum;
          }
        }
      }
    }
    if (!whole && j0 == 0) {
      if (threadIdx.x == 0) {
        const long long last = share.end - at.left + at.nt - 1;  // the unit's last tile
        p.ws.few_rec[blockIdx.x] =
            PlanRecord{at.b, at.head, 0, plan_cta_of(last, share.total, share.ctas) - static_cast<int>(blockIdx.x)};
      }
      recorded = true;
    }
    at.advance(a, j1 - j0);
  }
  if (threadIdx.x == 0 && !recorded) p.ws.few_rec[blockIdx.x].b = -1;
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

template <int D, bool E4M3, int MT>
int launch_paged_few_impl(const PagedFwdArgs& a, const LaunchCtx& ctx) {
  using C = FewCfg<D, E4M3, MT>;
  auto kernel = fa_paged_few_kernel<D, E4M3, MT>;
  static std::atomic<unsigned long long> allowed{0};
  const int e = allow_smem(kernel, C::SMEM, allowed);
  if (e != 0) return e;
  FewParams p;
  p.a = a;
  p.ws = paged_ws(a.workspace, D);
  p.status = ctx.status;
  p.limit_ns = ctx.limit_ns;
  p.box = C::KG == 32 && a.kv.ps_log2 >= 5 ? 32 : 16;
  CUtensorMap mk, mv;
  const long long dims[4] = {D, 1LL << a.kv.ps_log2, a.kv.heads, a.kv.num_pages};
  const long long ks[3] = {a.kv.ks[2], a.kv.ks[1], a.kv.ks[0]}, vs[3] = {a.kv.vs[2], a.kv.vs[1], a.kv.vs[0]};
  if (encode_paged_map(&mk, a.kv.k, C::EB, dims, ks, C::SWB / C::EB, p.box, 1, C::SWB, true) != 0) return -1;
  if (encode_paged_map(&mv, a.kv.v, C::EB, dims, vs, C::SWB / C::EB, p.box, 1, C::SWB, true) != 0) return -1;
  const int grid = ctx.num_sms < kPlanCtas ? ctx.num_sms : kPlanCtas;
  kernel<<<grid, C::THREADS, C::SMEM, ctx.stream>>>(mk, mv, p);
  return static_cast<int>(cudaGetLastError());
}

template <int D>
int launch_paged_few(const PagedFwdArgs& a, const LaunchCtx& ctx) {
  if constexpr (D <= 128)
    if (a.few_rows > 16) return a.e4m3 ? launch_paged_few_impl<D, true, 2>(a, ctx) : launch_paged_few_impl<D, false, 2>(a, ctx);
  return a.e4m3 ? launch_paged_few_impl<D, true, 1>(a, ctx) : launch_paged_few_impl<D, false, 1>(a, ctx);
}

}  // namespace fa
