// Attention of few rows over a paged cache: sequences whose rows (n_b tokens x
// the query heads of one key/value head) are 32 at most, decoding above all.
//
//   s_ij = scale q_i . k_j,  m, l: running maximum and sum,  o_i = sum_j p_ij v_j / l_i
//
// Bound by reading K and V once, so everything serves to keep reads in flight:
//  * one CTA per SM; each warp is a pipeline of its own: it takes every NW-th
//    group of KG keys, loads K and V of a group with TMA boxes of 16 or 32 tokens
//    (a page holds whole boxes) into its own ring of stages, and issues the
//    load S groups ahead, across the borders of units; no barrier between
//    warps but where a unit ends;
//  * products by mma.sync m16n8k16 with the rows as N, 8 to a tile: S^T = K Q^T and
//    O^T = V^T P^T, so that 8 rows cost half of what 16 do (mma.sync measured 2
//    cycles a 16x8x16 product and SM on this GPU; with two warps a scheduler what
//    bounds e4m3 pages is the instructions of a warp and their latencies, and a
//    padded M of 16 has twice the logits; a tcgen05 tile of 128 rows would multiply mostly
//    padding, and its softmax would cost 128 rows); the row tiles share every K and
//    V fragment, and every row tile is computed whether it holds rows or not (with a
//    branch each the compiler cannot interleave them: e4m3, 4 tiles, 3.2 us a tile of
//    256 keys instead of 2.7);
//  * softmax state m, l and the output stay in registers; at a unit's end the
//    warps' results are joined in shared memory, in the warps' order.
// e4m3 pages: codes are exact in fp16, so S = Q K^T runs in fp16 with the codes
// as they are and every q row multiplied by a power of two that brings its
// largest element to [2^13, 2^14) (exact down to 2^-37 of that element); the
// rows' and the keys' powers of two multiply the fp32 result.  V's scales go
// into P: P' = p 2^(e_j - E) 2^6 in fp16, e_j the scale's exponent and E a warp's
// fixed one (of tokens that all rows see).  So that no token of small weight, and
// none that a row does not see, takes bits from that row, what counts for the
// reference m is the row's largest product p_j 2^(e_j - E), not its largest p_j:
//   m = max_j (x_j + e_j - E),  p_j = 2^(x_j - m),  x_j the logit in log2 units.
// P' is then rounded to 11 bits down to 2^-20 of the row's largest product, finer
// than bf16's 8, and to 2^-31 of it below; l and o stand for 2^m whatever m is.
// m moves only when x_j + e_j - E exceeds it by more than 8, so P' <= 2^14 and most
// groups need neither the rows' maxima nor a rescale: one vote of the warp says so
// (with the group's largest e_j for every key's).  (With E the largest exponent so far and m the largest logit, as plain as
// can be, a hidden token 2^24 times larger than the others cost the earlier rows their bits; it was as fast with
// single tokens and 3 % faster with drafts.)
//
// Measured: single tokens of 64 sequences, 1.24 GB of bf16 pages, d = 128: 188 us, 6.6 TB/s (0.97 of a copy's rate);
// 1.12 GB of e4m3 pages 171 us, 6.5 TB/s; 2 to 8 drafted tokens of 4 heads over 376 MB of e4m3 pages 124 us, 3.0 TB/s
// (issue slots 36 % used with two warps a scheduler, tensor pipe 30 %: latencies), over 743 MB of bf16 pages 135 us, 5.5 TB/s.
#pragma once

#include <type_traits>

#include "fa_paged_plan.cuh"

namespace fa {

// NT: tiles of 8 rows (1, 2 or 4).
template <int D, bool E4M3, int NT>
struct FewCfg {
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int ROWB = D * EB;                     // bytes of a K or V row
  static constexpr int NW = D == 256 ? 4 : 8;             // warps (d = 256: a group of 16 KB, three in flight)
  static constexpr int THREADS = 32 * NW;
  // Keys of a group: 4 KB of K, so that what a group costs besides its products is spread over as many keys as
  // registers hold logits of.
  static constexpr int KG = E4M3 ? (D >= 128 || NT == 4 ? 32 : 64) : (D >= 128 ? 16 : D == 64 ? 32 : 64);
  static constexpr int NG = KG / 16;
  static constexpr int KT = KG * NW;                      // keys of a tile (one group per warp)
  static constexpr int SWB = ROWB < 128 ? ROWB : 128;     // swizzle span
  static constexpr int REGIONS = ROWB / SWB;
  static constexpr int REGION = KG * SWB;
  static constexpr int KV = KG * ROWB;                    // bytes of a group of K or V
  // Joining the warps: O of 8 rows of every warp, fp32, a row padded by 4 so that a warp's stores meet every bank once.
  static constexpr int JROW = D + 4;
  static constexpr int JOIN = NW * 8 * JROW * 4;
  static constexpr int QS = NT * D > 256 ? NT * 8 * D * 2 : 0;  // q in shared memory where registers are full of outputs
  static constexpr int MISC = 8 * 1024;
  static constexpr int FIT = (226 * 1024 - JOIN - QS - MISC) / (NW * 2 * KV);
  static constexpr int S = FIT > 8 ? 8 : FIT;             // stages of a warp's ring
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_Q = NW * S * 2 * KV;
  static constexpr int OFF_JOIN = OFF_Q + QS;
  static constexpr int OFF_ML = OFF_JOIN + JOIN;          // the warps' m and l (e4m3: and m + E) [NW][ML / 8][8]
  static constexpr int ML = E4M3 ? 24 : 16;
  static constexpr int OFF_ROWF = OFF_ML + NW * ML * 4;   // e4m3, q in shared memory: the rows' factors [NT * 8]
  static constexpr int OFF_SCALE = OFF_ROWF + 128;        // e4m3: K and V scale bytes [NW][S][2][KG]
  static constexpr int OFF_BAR = OFF_SCALE + (E4M3 ? NW * S * 2 * KG : 0);
  static constexpr int OFF_PLAN = OFF_BAR + NW * S * 8;
  static constexpr int OFF_ABORT = OFF_PLAN + static_cast<int>(sizeof(PlanScratch));
  static constexpr int SMEM = OFF_ABORT + 16 + 1024;      // + slack for 1024-byte alignment
  static_assert(OFF_ABORT + 16 - OFF_ML <= MISC && SMEM <= 227 * 1024, "shared memory budget");
  static_assert(S >= 2 && OFF_SCALE % 16 == 0 && OFF_BAR % 8 == 0 && OFF_PLAN % 8 == 0, "layout");
  static_assert(NT == 1 || NT == 2 || (NT == 4 && D <= 128), "row tiles");
  // Pages looked up a group ahead: where a warp's instructions are the bound, not memory (e4m3, single tokens of 128
  // sequences, d = 128: 178 us instead of 183, d = 64: 122 and 138; bf16 and d = 256 the same; four row tiles have no
  // registers left).
  static constexpr bool EARLY = E4M3 && NT <= 2 && D <= 128;
  static constexpr int KS = D / 16;                       // K steps of S^T = 16-column tiles of O^T
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
// 8 x 8 matrix of 16-bit elements, a row to four threads: transposed across the warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Tiles that a unit costs besides its own (beginning it, joining the warps): measured 1.4 to 3.6 us a unit with one row
// tile and 6 to 8 with four, against 1.4 to 2.9 us a tile (drafts of ragged lengths 177 us without it, 157 with it).
constexpr int kFewUnitCost = 2;
constexpr float kFewSlack = 8.f;  // log2 units by which a logit may exceed the reference maximum
// e4m3: how far e_j may count above and below E in m.  Where one lies farther above, E grows; one farther below (its P' is what
// it is) counts as E - kFewBelow, and a scale byte of 0 (zeros, or values below 2^-118) as E - kFewZero.  So a row's largest
// p_j lies within 2^-kFewAbove .. 2^(kFewBelow + 8): l holds every weight that counts, and stays finite whatever E grows
// by, where the scales of V in a sequence (zeros aside) lie within 2^190 of each other.
constexpr int kFewAbove = 96, kFewBelow = 96, kFewZero = 64;
constexpr int kNoBase = -256;  // E before the first group

struct FewParams {
  PagedFwdArgs a;
  PlanRecord* rec;  // of this launch's units
  float* part;
  int* status;
  unsigned long long limit_ns;
  int from, most;  // the launch takes sequences of more than `from` rows and of `most` at most
  int box_log2;  // log2 of the tokens of a K/V box: a page or a group, whichever is smaller
};

// Tiles of KT keys of one head of sequence b in this kernel (0: not one of its sequences).
template <int KT>
__device__ __forceinline__ int few_tiles(const FewParams& p, const PagedSeq& s) {
  if (s.n < 1 || s.n > p.a.max_rows || s.n > kFewMost || s.n * p.a.group > p.most || s.n * p.a.group <= p.from) return 0;
  return s.len <= KT ? 1 : (s.len + KT - 1) / KT;  // without keys too: the rows get their zeros
}

// Length of sequence b's units on the line of work.
template <int KT>
__device__ __forceinline__ long long few_length(const FewParams& p, const PagedSeq& s) {
  const int nt = few_tiles<KT>(p, s);
  return nt == 0 ? 0 : static_cast<long long>(p.a.kv.heads) * (nt + kFewUnitCost);
}

// Walks the tiles of a CTA's share; `left`: what is left of it on the line (0: no more tiles).
template <int KT>
struct FewCursor {
  int b, head, j, nt, left;
  PagedSeq s;
  __device__ __forceinline__ void load(const FewParams& p) {
    bool bad;
    s = paged_seq(p.a.pb, p.a.kv.ps_log2, b, bad);
    nt = few_tiles<KT>(p, s);
  }
  __device__ __forceinline__ void start(const FewParams& p, const PlanShare& w) {
    left = static_cast<int>(w.end - w.start);  // (W / 152 tiles: W < 2^38)
    b = w.b;
    if (left == 0) return;
    load(p);
    head = static_cast<int>(w.offset / (nt + kFewUnitCost));
    j = static_cast<int>(w.offset - static_cast<long long>(head) * (nt + kFewUnitCost));
    if (j >= nt) {  // behind a unit's tiles (a share is longer than that)
      left += j - nt;
      j = nt;
      advance(p, 0);
    }
  }
  // Move on by k tiles of the present unit.
  __device__ __forceinline__ void advance(const FewParams& p, int k) {
    left -= k;
    j += k;
    if (j < nt) return;
    left = max(left - kFewUnitCost, 0);
    if (left == 0) return;
    j = 0;
    if (++head < p.a.kv.heads) return;
    head = 0;
    do {
      ++b;
      load(p);
    } while (nt == 0);
  }
};

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(FewCfg<D, E4M3, NT>::THREADS, 1)
    fa_paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ FewParams p) {
  using C = FewCfg<D, E4M3, NT>;
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
        return few_length<C::KT>(p, paged_seq(a.pb, a.kv.ps_log2, b, bad));
      },
      1 + kFewUnitCost,
      *reinterpret_cast<PlanScratch*>(gbase + C::OFF_PLAN));

  // ---- the warp's loads
  FewCursor<C::KT> ahead;  // next group to load
  ahead.start(p, share);
  uint32_t issued = 0, done = 0;
  const int box_log2 = p.box_log2;
  const int slot_mask = (1 << a.kv.ps_log2) - 1;
  // The next group with keys; where EARLY, its page's number is on its way until the group is issued.
  int next_page = -1;
  auto find = [&]() {
    while (ahead.left > 0 && ahead.j * C::KT + warp * C::KG >= ahead.s.len) ahead.advance(p, 1);
    if constexpr (C::EARLY) {
      const int key = ahead.j * C::KT + warp * C::KG + ((lane >> 1) << box_log2);  // lanes 2i and 2i + 1: box i
      if (ahead.left > 0 && lane < 2 * NG && key < ahead.s.len)
        next_page = a.pb.page_table[ahead.b * a.pb.table_stride + (key >> a.kv.ps_log2)];
    }
  };
  auto issue = [&]() {
    if constexpr (!C::EARLY) find();
    if (ahead.left == 0) return;
    const uint64_t policy = policy_evict_first();  // a unit's K and V are read once (made here: registers are full)
    const int key0 = ahead.j * C::KT + warp * C::KG;
    const uint32_t st = issued % C::S;
    const uint32_t bar = bars + 8 * st;
    // Boxes that hold keys of the sequence; lanes 2i and 2i + 1 load K and V of box i.
    const int nbox = NG == 1 ? 1 : (min(C::KG, ahead.s.len - key0) + (1 << box_log2) - 1) >> box_log2;
    if (lane == 0) mbar_arrive_expect_tx(bar, 2 * (nbox << box_log2) * (C::ROWB + (E4M3 ? 1 : 0)));
    __syncwarp();
    if (lane < 2 * nbox) {
      const int is_v = lane & 1, row = (lane >> 1) << box_log2;
      int page = next_page >= 0 && next_page < a.kv.num_pages ? next_page : -1;
      if constexpr (!C::EARLY) page = paged_page(a.pb, a.kv, ahead.b, key0 + row);
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
        bulk_load(sc, (is_v ? a.kv.v_scale : a.kv.k_scale) + off, 1 << box_log2, bar);
      }
    }
    ++issued;
    ahead.advance(p, 1);
    if constexpr (C::EARLY) find();
  };
  if constexpr (C::EARLY) find();
#pragma unroll 1
  for (int i = 0; i < C::S; ++i) issue();

  // ---- units
  FewCursor<C::KT> at;
  at.start(p, share);
  bool ok = true;
  bool recorded = false;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  const uint32_t group_magic = 65536u / a.group + 1;
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
    // Times 2^24: a key's factor is 2^-24 of its scale, for |x| < 2^31 (d 2^14 448) times a scale (2^120 at most, from
    // paged_write) may pass fp32's range where a tiny q keeps the logit in it.  Never 0 (times -inf) nor infinite (times 0).
    rowf = scale_log2 * 0x1p24f * __uint_as_float(static_cast<uint32_t>(e - 13) << 23);
    rowf = fminf(fmaxf(rowf, 0x1p-126f), 0x1.fffffep127f);
    return __uint_as_float(static_cast<uint32_t>(267 - e) << 23);  // 2^(13 - (e - 127))
  };

#pragma unroll 1
  while (at.left > 0) {
    const PagedSeq s = at.s;
    const int rows = s.n * a.group;
    const int j0 = at.j;
    const int j1 = at.left < at.nt - j0 ? j0 + at.left : at.nt;
    const int na = (rows + 7) >> 3;  // row tiles that hold rows
    // r / group of a row (exact: r (magic - 65536 / group) < 32 and a group is 32 at most).
    auto token_of = [&](int r) -> int { return static_cast<int>(static_cast<uint32_t>(r) * group_magic >> 16); };
    // The last key that row r sees (rows behind the last: any).
    auto sees = [&](int r) -> int { return a.causal && r < rows ? s.len - s.n + token_of(r) : s.len - 1; };
    auto q_row = [&](int r) -> const __nv_bfloat16* {
      const int tok = token_of(r);
      return r >= rows ? nullptr : a.q + static_cast<long long>(s.row0 + tok) * a.qs[0] +
                                       static_cast<long long>(at.head * a.group + r - tok * a.group) * a.qs[1];
    };
    // Rows that exist see the keys up to here (row 0 sees the fewest).
    const int lim_all = a.causal ? s.len - s.n : s.len - 1;
    // q as the B operand: row 8t + g, elements 16k + 2jq, + 1 and 16k + 8 + 2jq, + 1.
    uint32_t qf[C::QS ? 1 : NT][C::QS ? 1 : C::KS][2];
    float rowf[NT][2];  // factors of rows 8t + 2jq, + 1 (q in shared memory: read again for every group)
    const float2* rf = reinterpret_cast<const float2*>(gbase + C::OFF_ROWF);
    if constexpr (C::QS == 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const __nv_bfloat16* q = q_row(8 * t + g);
        if constexpr (!E4M3) {
#pragma unroll
          for (int k = 0; k < C::KS; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              qf[t][k][x] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 * x + 2 * jq) : 0u;
          rowf[t][0] = rowf[t][1] = scale_log2;
        } else {
          // fp16 elements 16k + 4 jq .. + 3 (the order in which an e4m3 fragment of K holds its elements).
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
          float factor;
          const float f = row_scale(top, factor);
#pragma unroll
          for (int k = 0; k < C::KS; ++k) {
            qf[t][k][0] = pack_f16x2(__uint_as_float(w[k].x << 16) * f, __uint_as_float(w[k].x & 0xffff0000u) * f);
            qf[t][k][1] = pack_f16x2(__uint_as_float(w[k].y << 16) * f, __uint_as_float(w[k].y & 0xffff0000u) * f);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) rowf[t][i] = __shfl_sync(0xffffffffu, factor, (2 * jq + i) * 4);
        }
      }
    } else {
      // q into shared memory: a warp per row, four elements a lane.
      constexpr int CH = (D / 4 + 31) / 32, RW = 8 * NT / C::NW;
      uint2 w[RW][CH];
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const __nv_bfloat16* q = q_row(warp + i * C::NW);
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          const int at4 = ch * 32 + lane;  // elements 4 at4 ..
          w[i][ch] = q && at4 < D / 4 ? *reinterpret_cast<const uint2*>(q + 4 * at4) : make_uint2(0u, 0u);
        }
      }
      uint8_t* dst = gbase + C::OFF_Q;
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const int r = warp + i * C::NW;
        if constexpr (!E4M3) {
#pragma unroll
          for (int ch = 0; ch < CH; ++ch) {
            const int at4 = ch * 32 + lane;
            if (at4 < D / 4) *reinterpret_cast<uint2*>(dst + q_place(r, at4 >> 1) + (at4 & 1) * 8) = w[i][ch];
          }
        } else {
          uint32_t top = 0;
#pragma unroll
          for (int ch = 0; ch < CH; ++ch) top = __vmaxu2(top, __vmaxu2(w[i][ch].x & 0x7fff7fffu, w[i][ch].y & 0x7fff7fffu));
          top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
          float factor;
          const float f = row_scale(top, factor);
          // Elements 4x, 4x + 1 of a 16-element block stand where a fragment has k = 2x, 2x + 1, the others at 8 + 2x.
#pragma unroll
          for (int ch = 0; ch < CH; ++ch) {
            const int at4 = ch * 32 + lane, blk = at4 >> 2, x = at4 & 3;
            if (at4 >= D / 4) continue;
            *reinterpret_cast<uint32_t*>(dst + q_place(r, 2 * blk) + 4 * x) =
                pack_f16x2(__uint_as_float(w[i][ch].x << 16) * f, __uint_as_float(w[i][ch].x & 0xffff0000u) * f);
            *reinterpret_cast<uint32_t*>(dst + q_place(r, 2 * blk + 1) + 4 * x) =
                pack_f16x2(__uint_as_float(w[i][ch].y << 16) * f, __uint_as_float(w[i][ch].y & 0xffff0000u) * f);
          }
          if (lane == 0) reinterpret_cast<float*>(gbase + C::OFF_ROWF)[r] = factor;
        }
      }
      __syncthreads();
    }
    // O^T: columns 16c + g and 16c + g + 8 (e4m3: 16c + 2g and 16c + 2g + 1) of rows 8t + 2jq, + 1.
    float o[NT][C::KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < C::KS; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][c][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[t][i] = -INFINITY;
        l[t][i] = 0.f;
      }
    }
    int vbase = kNoBase;  // e4m3: E as a scale byte; o is in units of 2^(vbase - 127 - 6)

#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      const int key0 = j * C::KT + warp * C::KG;
      if (key0 >= s.len) break;
      const uint32_t st = done % C::S;
      if (ok) ok = warp_wait_bar(bars + 8 * st, (done / C::S) & 1, guard, kStatusTimeoutLoad);
      if (!ok) break;
      const uint32_t kt = ring + st * 2 * C::KV, vt = kt + C::KV;
      uint8_t* vt_g = gbase + (vt - base);
      // Logits / scale: keys 16 sg + g (x[.][sg][0..1]) and + 8 (x[.][sg][2..3]) of rows 8t + 2jq, + 1.
      float x[NT][NG][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int sg = 0; sg < NG; ++sg)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[t][sg][i] = 0.f;
#pragma unroll
      for (int k = 0; k < C::KS; k += 2) {
        uint32_t qb[NT][2][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (C::QS == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 2; ++i) qb[t][h][i] = qf[t][k + h][i];
          } else {
            uint32_t r[4];
            ldsm_x4(base + C::OFF_Q + q_place(8 * t + (lane & 7), 2 * k + (lane >> 3)), r);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 2; ++i) qb[t][h][i] = r[2 * h + i];
          }
        }
#pragma unroll
        for (int sg = 0; sg < NG; ++sg) {
          uint32_t ka[2][4];
          if constexpr (!E4M3) {
            ldsm_x4(kt + place(16 * sg + (lane & 15), 2 * k + (lane >> 4)), ka[0]);
            ldsm_x4(kt + place(16 * sg + (lane & 15), 2 * k + 2 + (lane >> 4)), ka[1]);
          } else {
            uint32_t b[4];  // keys 0..7 and 8..15 of 16 elements, then of the next 16
            ldsm_x4(kt + place(16 * sg + (lane & 15), k + (lane >> 4)), b);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ka[h][0] = e4m3x2_to_f16x2(static_cast<uint16_t>(b[2 * h]));
              ka[h][1] = e4m3x2_to_f16x2(static_cast<uint16_t>(b[2 * h + 1]));
              ka[h][2] = e4m3x2_to_f16x2(static_cast<uint16_t>(b[2 * h] >> 16));
              ka[h][3] = e4m3x2_to_f16x2(static_cast<uint16_t>(b[2 * h + 1] >> 16));
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma_16816<E4M3>(x[t][sg], ka[h], qb[t][h][0], qb[t][h][1]);
        }
      }
      const bool edge = key0 + C::KG - 1 > lim_all;  // some row does not see some key
      float pf[NG][2];  // e4m3: 2^6 times V's scales of keys 16 sg + g, + 8, in units of 2^(vbase - 127)
      float slack = kFewSlack;  // e4m3: less by the log2 of the largest of these scales (without the 2^6)
      if constexpr (E4M3) {
        // A lane turns the scales of keys 32 r + lane into factors; a fragment's come by shuffle.
        constexpr int KPL = C::KG / 32;
        const uint8_t* sc = gbase + C::OFF_SCALE + (warp * C::S + st) * 2 * C::KG + lane;
        uint32_t vb[KPL];
        float mine[KPL];
        uint32_t top = 0;
#pragma unroll
        for (int r = 0; r < KPL; ++r) {
          const uint32_t kb = sc[32 * r];
          mine[r] = __uint_as_float(kb == 255 ? 0x7fc00000u : kb << 23) * 0x1p-24f;  // (0 and 1: 0)
          vb[r] = sc[C::KG + 32 * r];
          if (edge && key0 + 32 * r + lane >= s.len) vb[r] = 0;
          top = max(top, vb[r] == 255 ? 0 : vb[r]);
        }
        float kf[NG][2];
#pragma unroll
        for (int sg = 0; sg < NG; ++sg)
#pragma unroll
          for (int i = 0; i < 2; ++i) kf[sg][i] = __shfl_sync(0xffffffffu, mine[sg >> 1], (16 * sg + 8 * i + g) & 31);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int sg = 0; sg < NG; ++sg)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[t][sg][i] *= kf[sg][i >> 1];
        }
        const int most = static_cast<int>(__reduce_max_sync(0xffffffffu, top));
        if (most - vbase > kFewAbove) {
          if (vbase == kNoBase) {
            // The largest scale of keys that every row sees, or the first key's: the rows that see anything here see that.
            uint32_t all = 0;
#pragma unroll
            for (int r = 0; r < KPL; ++r)
              if (vb[r] != 255 && key0 + 32 * r + lane <= max(lim_all, key0)) all = max(all, vb[r]);
            all = __reduce_max_sync(0xffffffffu, all);
            vbase = all == 0 ? 127 : max(static_cast<int>(all), 80);
          }
          // (o is in units of 2^(E + m): both change, it does not.)
          const int up = max(most - kFewAbove - vbase, 0);  // <= 78
          vbase += up;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              m[t][i] -= static_cast<float>(up);
              l[t][i] *= __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            }
        }
        slack = kFewSlack - static_cast<float>(max(most - vbase, -kFewZero));
#pragma unroll
        for (int r = 0; r < KPL; ++r)
          mine[r] = vb[r] == 255 ? __uint_as_float(0x7fc00000u)
                                 : __uint_as_float(static_cast<uint32_t>(max(127 + 6 + static_cast<int>(vb[r]) - vbase, 0)) << 23);
#pragma unroll
        for (int sg = 0; sg < NG; ++sg)
#pragma unroll
          for (int i = 0; i < 2; ++i) pf[sg][i] = __shfl_sync(0xffffffffu, mine[sg >> 1], (16 * sg + 8 * i + g) & 31);
      }
      if constexpr (C::QS != 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float2 f = E4M3 ? rf[4 * t + jq] : make_float2(scale_log2, scale_log2);
          rowf[t][0] = f.x;
          rowf[t][1] = f.y;
        }
      }
      uint32_t pb[NT][NG][2];  // P^T as the B operand
      // This thread's largest logit of row 8t + 2jq + i, scaled.
      auto largest = [&](int t, int i) -> float {
        float y = fmaxf(x[t][0][i], x[t][0][2 + i]);
#pragma unroll
        for (int sg = 1; sg < NG; ++sg) y = fmax3(y, x[t][sg][i], x[t][sg][2 + i]);
        return y * rowf[t][i];
      };
      bool moves = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (edge) {
          const int lim[2] = {sees(8 * t + 2 * jq), sees(8 * t + 2 * jq + 1)};
#pragma unroll
          for (int sg = 0; sg < NG; ++sg)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + 16 * sg + 8 * (i >> 1) + g > lim[i & 1]) x[t][sg][i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) moves = moves || largest(t, i) > m[t][i] + slack;
      }
      if (__any_sync(0xffffffffu, moves)) {
        float ve[NG][2];  // e4m3: e_j - E of this thread's keys (a scale of NaN: 0)
        if constexpr (E4M3) {
#pragma unroll
          for (int sg = 0; sg < NG; ++sg)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = static_cast<int>(__float_as_uint(pf[sg][h]) >> 23) - (127 + 6);
              const int low = e <= -min(vbase, 127 + 6) ? -kFewZero : max(e, -kFewBelow);
              ve[sg][h] = e > kFewAbove ? 0.f : static_cast<float>(low);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float alpha[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y = -INFINITY;
            if constexpr (E4M3) {
#pragma unroll
              for (int sg = 0; sg < NG; ++sg)
                y = fmax3(y, fmaf(x[t][sg][i], rowf[t][i], ve[sg][0]), fmaf(x[t][sg][2 + i], rowf[t][i], ve[sg][1]));
            } else {
              y = largest(t, i);
            }
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
            const float m_new = fmaxf(m[t][i], y);
            alpha[i] = m_new == m[t][i] ? 1.f : ex2(m[t][i] - m_new);
            m[t][i] = m_new;
            l[t][i] *= alpha[i];
          }
#pragma unroll
          for (int c = 0; c < C::KS; ++c) {
            o[t][c][0] *= alpha[0];
            o[t][c][1] *= alpha[1];
            o[t][c][2] *= alpha[0];
            o[t][c][3] *= alpha[1];
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float ref = m[t][i] == -INFINITY ? 0.f : -m[t][i];
          float sum = 0.f;
#pragma unroll
          for (int sg = 0; sg < NG; ++sg)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& y = x[t][sg][2 * h + i];
              y = ex2(fmaf(y, rowf[t][i], ref));
              sum += y;
            }
          l[t][i] += sum;  // this thread's keys only; summed up at the unit's end
        }
#pragma unroll
        for (int sg = 0; sg < NG; ++sg)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float* y = &x[t][sg][2 * h];
            if constexpr (E4M3) {
              y[0] *= pf[sg][h];
              y[1] *= pf[sg][h];
              if (edge) {  // a scale of NaN reaches only the rows that see its token
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (key0 + 16 * sg + 8 * h + g > sees(8 * t + 2 * jq + i)) y[i] = 0.f;
              }
              pb[t][sg][h] = transpose_8x8(pack_f16x2(y[0], y[1]));
            } else {
              pb[t][sg][h] = transpose_8x8(pack_bf16x2(y[0], y[1]));
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
              ldsm_x4_t(vt + place(16 * sg + (lane & 7) + ((lane >> 4) << 3), 2 * c + ((lane >> 3) & 1)), b);
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma_16816<false>(o[t][c], b, pb[t][sg][0], pb[t][sg][1]);
            } else {
              // A transposed fragment holds two columns of two keys: 16c + 2g becomes row g of the operand, 16c + 2g + 1 row g + 8.
              ldsm_x4_t(vt + place(16 * sg + (lane & 15), c + (lane >> 4)), b);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t lo = __byte_perm(b[2 * h], 0, 0x3120), hi = __byte_perm(b[2 * h + 1], 0, 0x3120);
                const uint32_t va[4] = {
                    e4m3x2_to_f16x2(static_cast<uint16_t>(lo)), e4m3x2_to_f16x2(static_cast<uint16_t>(lo >> 16)),
                    e4m3x2_to_f16x2(static_cast<uint16_t>(hi)), e4m3x2_to_f16x2(static_cast<uint16_t>(hi >> 16))};
#pragma unroll
                for (int t = 0; t < NT; ++t)
                  mma_16816<true>(o[t][c + h], va, pb[t][sg][0], pb[t][sg][1]);
              }
            }
          }
        }
      } else {
        // Key by key, and only for the rows that see the key.
#pragma unroll 1
        for (int key = 0; key < C::KG; ++key) {
          // (One copy of this code for all of a group's keys: unrolled it would crowd out what runs often.)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t >= na) continue;
            uint32_t mine = 0;  // of row 8t + g: keys 2jq, + 1 of the key's eight
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i) mine = key >> 3 == i ? pb[t][i >> 1][i & 1] : mine;
            float pv[2];
            bool see[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t pair = __shfl_sync(0xffffffffu, mine, (2 * jq + r) * 4 + ((key & 7) >> 1));
              const uint32_t one = key & 1 ? pair >> 16 : pair & 0xffffu;
              pv[r] = E4M3 ? __half2float(__ushort_as_half(static_cast<uint16_t>(one))) : __uint_as_float(one << 16);
              see[r] = key0 + key <= sees(8 * t + 2 * jq + r);
            }
#pragma unroll
            for (int c = 0; c < C::KS; ++c) {
              float v[2];  // the columns of o[t][c][0..1] and o[t][c][2..3]
              if constexpr (!E4M3) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  v[h] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(vt_g + place(key, 2 * c + h) + 2 * g));
              } else {
                const uint32_t h2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vt_g + place(key, c) + 2 * g));
                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                v[0] = y.x;
                v[1] = y.y;
              }
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                  if (see[r]) o[t][c][2 * h + r] = fmaf(pv[r], v[h], o[t][c][2 * h + r]);
            }
          }
        }
      }
      __syncwarp();  // the stage has been read
      ++done;
      issue();
    }
    // ---- join the warps, 8 rows at a time: each writes its O, m and l, then a warp takes a row.
    const bool whole = j0 == 0 && j1 == at.nt;
    float* join_o = reinterpret_cast<float*>(gbase + C::OFF_JOIN);
    float* join_ml = reinterpret_cast<float*>(gbase + C::OFF_ML);
#pragma unroll 1
    for (int t8 = 0; t8 < na; ++t8) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t != t8) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 4);
          l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 8);
          l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 16);
          float* dst = join_o + (warp * 8 + 2 * jq + i) * C::JROW;
#pragma unroll
          for (int c = 0; c < C::KS; ++c) {
            if constexpr (E4M3) {
              *reinterpret_cast<float2*>(dst + 16 * c + 2 * g) = make_float2(o[t][c][i], o[t][c][2 + i]);
            } else {
              dst[16 * c + g] = o[t][c][i];
              dst[16 * c + 8 + g] = o[t][c][2 + i];
            }
          }
          if (g == 0) {
            join_ml[warp * C::ML + 2 * jq + i] = m[t][i];
            join_ml[warp * C::ML + 8 + 2 * jq + i] = l[t][i];
            if constexpr (E4M3) join_ml[warp * C::ML + 16 + 2 * jq + i] = m[t][i] + static_cast<float>(vbase);
          }
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int r8 = warp; r8 < 8; r8 += C::NW) {
        const int r = 8 * t8 + r8;
        if (r >= rows || *abort_flag != 0) break;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::NW; ++w) top = fmaxf(top, join_ml[w * C::ML + r8]);
        float lsum = 0.f, acc[D / 32] = {};
        float otop = -INFINITY;  // e4m3: the largest E + m, O's reference
        if constexpr (E4M3) {
#pragma unroll
          for (int w = 0; w < C::NW; ++w) otop = fmaxf(otop, join_ml[w * C::ML + 16 + r8]);
        }
#pragma unroll
        for (int w = 0; w < C::NW; ++w) {
          const float mw = join_ml[w * C::ML + r8];
          float f = mw == top ? 1.f : ex2((E4M3 ? 0.5f : 1.f) * (mw - top));
          if constexpr (!E4M3) {
            lsum = fmaf(join_ml[w * C::ML + 8 + r8], f, lsum);
          } else {
            // (The m of warps may lie 2^200 apart, where one has a large l and the other a small one: by halves.)
            lsum = fmaf(join_ml[w * C::ML + 8 + r8] * f, f, lsum);
            const float ow = join_ml[w * C::ML + 16 + r8];
            f = ow == otop ? 1.f : ex2(ow - otop);
          }
          const float* src = join_o + (w * 8 + r8) * C::JROW + lane;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(src[32 * c], f, acc[c]);
        }
        const int tok = token_of(r), row = s.row0 + tok, hq = at.head * a.group + r - tok * a.group;
        float inv = lsum == 0.f ? 0.f : 1.f / lsum;
        if constexpr (E4M3) {
          // From 2^otop to 2^top in V's units, by halves, too (no keys seen: m = -inf, O = 0).
          const float f = top == -INFINITY ? 0.f : ex2(0.5f * (otop - top - (127.f + 6.f)));
          inv *= f;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) acc[c] *= f;
        }
        const float lg = top + log2f(lsum);
        if (whole) {
          __nv_bfloat16* dst = a.o + static_cast<long long>(row) * a.os[0] + static_cast<long long>(hq) * a.os[1] + lane;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) dst[32 * c] = __float2bfloat16_rn(acc[c] * inv);
          if (lane == 0) a.lse[static_cast<long long>(hq) * a.pb.rows + row] = lg * 0.69314718055994531f;
        } else {
          float* part = p.part + (blockIdx.x * 2 + (j0 == 0 ? 1 : 0)) * part_floats(kFewMost, D);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) part[kFewMost + r * D + 32 * c + lane] = acc[c] * inv;
          if (lane == 0) part[r] = lg;
        }
      }
      __syncthreads();
    }
    if (!whole && j0 == 0) {
      if (threadIdx.x == 0) {
        const long long last = share.end - at.left + at.nt - 1;  // the unit's last tile
        p.rec[blockIdx.x] =
            PlanRecord{at.b, at.head, 0, plan_cta_of(last, share.total, share.ctas) - static_cast<int>(blockIdx.x)};
      }
      recorded = true;
    }
    at.advance(p, j1 - j0);
  }
  if (threadIdx.x == 0 && !recorded) p.rec[blockIdx.x].b = -1;
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
  pdl_wait();  // what waits for this kernel waits for the chunks' kernel before it, too
}

template <int D, bool E4M3, int NT>
int launch_paged_few_impl(const PagedFwdArgs& a, int set, int from, int most, bool behind, const LaunchCtx& ctx) {
  using C = FewCfg<D, E4M3, NT>;
  auto kernel = fa_paged_few_kernel<D, E4M3, NT>;
  static std::atomic<unsigned long long> allowed{0};
  const int e = allow_smem(kernel, C::SMEM, allowed);
  if (e != 0) return e;
  FewParams p;
  p.a = a;
  const PagedWs ws = paged_ws(a.workspace, D);
  p.rec = ws.few_rec[set];
  p.part = ws.few_part[set];
  p.from = from;
  p.most = most;
  p.status = ctx.status;
  p.limit_ns = ctx.limit_ns;
  const int box = (1 << a.kv.ps_log2) < C::KG ? 1 << a.kv.ps_log2 : C::KG;
  for (p.box_log2 = 4; (1 << p.box_log2) < box; ++p.box_log2) {
  }
  CUtensorMap mk, mv;
  const long long dims[4] = {D, 1LL << a.kv.ps_log2, a.kv.heads, a.kv.num_pages};
  const long long ks[3] = {a.kv.ks[2], a.kv.ks[1], a.kv.ks[0]}, vs[3] = {a.kv.vs[2], a.kv.vs[1], a.kv.vs[0]};
  if (encode_paged_map(&mk, a.kv.k, C::EB, dims, ks, C::SWB / C::EB, box, 1, C::SWB, true) != 0) return -1;
  if (encode_paged_map(&mv, a.kv.v, C::EB, dims, vs, C::SWB / C::EB, box, 1, C::SWB, true) != 0) return -1;
  const int grid = ctx.num_sms < kPlanCtas ? ctx.num_sms : kPlanCtas;
  if (behind) return launch_dependent(kernel, dim3(grid), C::THREADS, C::SMEM, ctx.stream, mk, mv, p);
  kernel<<<grid, C::THREADS, C::SMEM, ctx.stream>>>(mk, mv, p);
  return static_cast<int>(cudaGetLastError());
}

// Row tiles cost nothing while reading K and V bounds the kernel (bf16: 1.4 us a tile of 128 keys with 1, 2 or 4), but
// with e4m3 pages they do (256 keys, d = 128: 1.4, 1.65 and 2.7 us), so sequences of more than 16 rows are a launch of
// their own there, if there is work enough for two.  Which sequences have how many rows only the device knows; B times the
// heads decides.  4 query heads to a key/value head, 0.8 to 8 K tokens, us in one launch / two:
//   B heads                        32       64       128      192      320       640       1280
//   2 to 8 new tokens a sequence   33 / 43  46 / 61  72 / 75  89 / 92  149 / 139 259 / 233 500 / 456
//   1, rarely 8                    29 / 34  44 / 43  70 / 60  86 / 79  149 / 119 260 / 183 492 / 330
//   5 to 8 (all in the first)      34 / 38  47 / 51  75 / 79  92 / 96  150 / 155 263 / 264 502 / 508
template <int D>
int launch_paged_few(const PagedFwdArgs& a, bool behind_chunks, const LaunchCtx& ctx) {
  auto launch = [&](auto nt, int set, int from, int most, bool behind) -> int {
    constexpr int NT = decltype(nt)::value;
    return a.e4m3 ? launch_paged_few_impl<D, true, NT>(a, set, from, most, behind, ctx)
                  : launch_paged_few_impl<D, false, NT>(a, set, from, most, behind, ctx);
  };
  using std::integral_constant;
  if (a.few_rows <= 8) return launch(integral_constant<int, 1>{}, 0, 0, 8, behind_chunks);
  if constexpr (D <= 128) {
    if (a.few_rows > 16) {
      const int e = launch(integral_constant<int, 4>{}, 0, a.few_sets == 2 ? 16 : 0, kFewMost, behind_chunks);
      if (e != 0 || a.few_sets == 1) return e;
      return launch(integral_constant<int, 2>{}, 1, 0, 16, true);
    }
  }
  return launch(integral_constant<int, 2>{}, 0, 0, 16, behind_chunks);
}

}  // namespace fa
