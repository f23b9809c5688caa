// Gradients of cross attention over ragged batches: the backward pass's two
// kernels (fa_bwd_tc.cuh: a key-parallel one for dK and dV, a query-parallel
// one for dQ, no atomics on results) on work that is found on the device, and
// the kernels before and behind them.
//
//   P = 2^(scale log2e q k^T - L log2e),  D = sum_c dO O,  dS = P (dO v^T - D),
//   dV = P^T dO,  dK = scale dS^T Q (both summed over the heads of a group),  dQ = scale dS K.
//
//  * Rows.  The G query heads of a key/value head share tiles, token by token
//    (a 3-D TMA box {columns, G heads, tokens}), so a group's heads add up in one
//    accumulator, short sequences fill tiles, and K and V are read once for all of them.
//      MODE 0 (dK, dV): a unit is 128 keys of one head; tiles of BS / G tokens of Q and dO stream past.
//      MODE 1 (dQ): a unit is 128 / G tokens of one key/value head; tiles of BS keys of K and V stream past.
//    d = 256: two accumulators of 128 x 256 leave no tensor memory for S and dP, so dV (MODE 3: S, dV) and dK (MODE 4: S, dP, dK)
//    are passes of their own: five products a tile, and six where two units with half of the columns each make both.
//    Rows of a streamed tile that are no token's or key's (anything, NaN too) meet zeros of P and dS in the accumulations, and 0
//    times NaN is NaN: the warpgroup that forms these sets such rows to zero first, behind S and dP of the tile.
//  * Sequences of few rows have a kernel of their own (fa_cross_bwd_short.cuh, MODE 2 here) that makes all three gradients
//    in one pass; these two take the others.
//  * Work.  The streamed tiles of all (sequence, head, unit) form one line that
//    is cut into equal shares (fa_paged_plan.cuh), with room for UNIT_COST more behind
//    each unit.  The load warp walks this CTA's share and hands segments (a run of one unit's
//    streamed tiles) to the other warps through a ring in shared memory.
//  * Output.  A unit held whole is written as it is finished; parts of others go to
//    the workspace in fp32 and the joining kernel adds them up in the order of their CTAs.
//  * Roundings.  P and dS are rounded to bf16 for the products (half a step, 2^-8, of each term), as in the contiguous
//    pass; S, dP, D, L and all sums are fp32, gradients are rounded once.  (The tensor core takes both operands in one 16-bit type, and Q, K and dO
//    are bf16; the rest of P and dS would be a second product each.  As it is the gradients are 2.4e-3 from the definition in the 2-norm, 1.7e-3 of it
//    their own rounding.)
//
// Bound: at d <= 128 by a tile's way through products and elementwise step (4 of 1 to 4 K rows over 2 to 8 K keys, d = 128: dK and
// dV 714 us, dQ 479 of 1.28 ms, 0.51 of the tensor cores for the five products that there must be and 0.71 for the seven that
// this split makes); at d = 256 by the latency of the streamed tiles, of which two fit (6 of 100 to 700 rows: some 36 + 46 + 49 under a profiler, of 150.5 us),
// then by parts (120 MB through L2, 20 us).  All modes in one launch, CTAs dealt by work, took longer: 1.37 ms and 210 us (then 173).
#pragma once

#include "fa_bwd_tc.cuh"
#include "fa_cross.cuh"
#include "fa_paged_plan.cuh"

namespace fa {

constexpr int kBwdSegRing = 4;

// d = 256 (MODE 1, 3, 4).  The streamed tensors have a ring each: A holds what S is made of (Q, or K), B the other.  The
// accumulations read A, too (dV's: B); the one that only a first product reads needs fewer slots, and 64 rows a tile
// fit where pairs of tiles left room for 32 (half as many products; 6 sequences of 100 to 700 rows: 172 to 160 us, and 157 with regions).
template <int MODE>
struct BwdWideCfg {
  static constexpr bool DP = MODE != 3;
  static constexpr int BM = 128;
  static constexpr int BS = 64;
  static constexpr int OUTW = 256, NOUT = 1;
  static constexpr int SWB = 128;
  static constexpr uint32_t SWZ = 2u;
  static constexpr int RC = 64, NR = 4;
  static constexpr int FIX_REGION = BM * SWB, S_REGION = BS * SWB;
  static constexpr int FIX_TILE = BM * 512, S_TILE = BS * 512;
  static constexpr int VEC_BYTES = BS * 4;
  static constexpr int NA = 2;            // slots
  // dQ, dK: one slot for what dP alone reads, loaded and freed region by region (64 columns, four products), so that most of a tile is on
  // its way again while the rest is multiplied; dV: whole tiles.
  static constexpr int NB = DP ? NR : 3;
  static constexpr int B_BYTES = DP ? S_REGION : S_TILE;
  static constexpr int OFF_FIX = 0;
  static constexpr int OFF_A = (DP ? 2 : 1) * FIX_TILE;  // dV: K alone
  static constexpr int OFF_B = OFF_A + NA * S_TILE;
  static constexpr int OFF_MISC = OFF_B + NB * B_BYTES;
  // The ring that the accumulations read; the vectors come with its tiles.
  static constexpr int NST = DP ? NA : NB;
  static constexpr int STAGE = S_TILE;
  static constexpr int OFF_ST = DP ? OFF_A : OFF_B;
  static constexpr int VECS = MODE == 1 ? 0 : DP ? 2 : 1;  // -L log2e, -D
  static constexpr int MISC = 1024 + NST * VECS * VEC_BYTES;
  static constexpr int OFF_TMEM_SLOT = OFF_MISC + 512;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int SMEM_ALLOC = OFF_MISC + MISC + 1024;  // + slack for 1024-byte alignment
  static constexpr int TM_S = 0, TM_DP = 2 * BS, TM_OUT = 4 * BS, TM_COLS = 512;
  static constexpr int MMA_WARP = 8, LOAD_WARP = 9;
  static_assert(TM_OUT + OUTW <= TM_COLS && SMEM_ALLOC <= 227 * 1024, "TMEM and shared memory budgets");
};
template <int D, int MODE>
struct BwdBaseOf {
  using type = BwdCfg<D, MODE>;
};
template <int MODE>
struct BwdBaseOf<256, MODE> {
  using type = BwdWideCfg<MODE>;
};
template <int D, int MODE>
using BwdBase = typename BwdBaseOf<D, MODE>::type;

// Rows of a streamed tile where K and V stay, and of a tile of the vectors.
template <int D>
constexpr __host__ __device__ int bwd_rows0() { return BwdBase<D, D == 256 ? 3 : 0>::BS; }

// Whether a unit is 128 keys (else 128 rows), and which of the workspace's three records and parts are a mode's.
constexpr __host__ __device__ bool bwd_by_key(int mode) { return mode == 0 || mode >= 3; }
constexpr __host__ __device__ int bwd_place(int mode) { return mode == 3 ? 0 : mode == 4 ? 2 : mode; }

// Tokens of a streamed tile of MODE 0 and of a fixed tile of MODE 1.
template <int D>
constexpr __host__ __device__ int bwd_tokens0(int group) { return bwd_rows0<D>() / group; }
constexpr __host__ __device__ int bwd_tokens1(int group) { return 128 / group; }

// -L log2e and -D of the rows, as MODE 0 streams them: BS values a tile of tokens, [heads][tiles][BS]; the tiles of sequences with
// rows and keys lie one behind another, in the sequences' order (CrossBwdWs::tile0).  As many as there can be: ranges that share no
// rows have rows / t0 whole tiles together at most, and B others.
template <int D>
__host__ __device__ __forceinline__ long long bwd_tiles(int rows, int B, int group) {
  return rows / bwd_tokens0<D>(group) + static_cast<long long>(B);
}

// 128-row tiles of a sequence's rows (all heads of a group) that MODE 2 takes at most (d = 256: none): as many as tensor memory holds dQ
// of.  There it is the faster one up to this bound (32 sequences over 1000 keys, 8 heads, at the bound and at half of it, us, against the
// kernels of longer sequences: d = 32 119 and 73 against 183 and 115, d = 64 90 and 62 against 145 and 111, d = 128 114 and 94 against 138 and 121).
constexpr __host__ __device__ int bwd_short_tiles(int d) { return d == 32 ? 4 : d == 64 ? 2 : d == 128 ? 1 : 0; }
template <int D>
__host__ __device__ __forceinline__ bool bwd_short(const CrossSeq& s, int group) {
  return s.n <= bwd_short_tiles(D) * bwd_tokens1(group);
}

// Units, fixed and streamed tiles of a kernel.
template <int D, int MODE>
struct BwdWork {
  static constexpr int STR = BwdBase<D, MODE>::BS;
  static constexpr size_t PART = static_cast<size_t>(128) * BwdBase<D, MODE>::NOUT * BwdBase<D, MODE>::OUTW;  // floats of a part
  // Streamed tiles that a unit costs besides its own (loading the fixed tiles, the output).
  // (6 sequences of 100 to 700 rows, d = 256, with 1/2/4/6/8/12: 162/157/155/156/156/159 us; of 1 to 4 K rows, d = 128, 1290
  // with 1 or 2, 1260 to 1280 with more.)
  static constexpr int UNIT_COST = 4;  // (of places on the line, as a streamed tile is one)
};
template <int D>
struct BwdWork<D, 2> {
  static constexpr int STR = 128;
  static constexpr size_t PART = static_cast<size_t>(128) * bwd_short_tiles(D) * D;
  static constexpr int QT = D <= 64 ? 64 : 32;  // rows of an item (fa_cross_bwd_short.cuh), which is a place on the line
  // Items that a streamed tile costs besides its own (its loads, its dK and dV), and a unit (32 sequences of 17 to 200 rows, d = 64,
  // with 1/2/4 of the one: 101.4/102.7/106.8 us, with 1/3/6 of the other 108.5/102.7/102.0).
  static constexpr int TILE_COST = 1;
  static constexpr int UNIT_COST = 3;
};

// Workspace of fa_cross_bwd.
struct CrossBwdWs {
  PlanRecord* rec[3];  // of the kernels (bwd_place): [kPlanCtas]
  int* part0;          // [kPlanCtas]: MODE 2's CTA has written its part 0
  uint32_t* tile0;     // [B]: first tile of a sequence's vectors (written where it has rows and keys)
  float* l2;           // [heads][tiles][BS]
  float* dsum;
  float* part[3];      // [kPlanCtas][2][part floats]
};
template <int D>
size_t cross_bwd_ws(char* p, int B, int rows, int heads, int group, CrossBwdWs* w) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* x = p + at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return x;
  };
  CrossBwdWs x;
  // (One head more than there are: see CrossBwdWalk::load.)
  const size_t vec = (static_cast<size_t>(heads) + 1) * bwd_tiles<D>(rows, B, group) * bwd_rows0<D>() * sizeof(float);
  for (int i = 0; i < 3; ++i) x.rec[i] = reinterpret_cast<PlanRecord*>(take(kPlanCtas * sizeof(PlanRecord)));
  x.part0 = reinterpret_cast<int*>(take(kPlanCtas * sizeof(int)));
  x.tile0 = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(B) * sizeof(uint32_t)));
  x.l2 = reinterpret_cast<float*>(take(vec));
  x.dsum = reinterpret_cast<float*>(take(vec));
  x.part[0] = reinterpret_cast<float*>(take(kPlanCtas * 2 * BwdWork<D, D == 256 ? 3 : 0>::PART * sizeof(float)));
  x.part[1] = reinterpret_cast<float*>(take(kPlanCtas * 2 * BwdWork<D, 1>::PART * sizeof(float)));
  x.part[2] = reinterpret_cast<float*>(take(kPlanCtas * 2 * BwdWork<D, D == 256 ? 4 : 2>::PART * sizeof(float)));
  if (w) *w = x;
  return at;
}

struct CrossBwdParams {
  CrossArgs a;
  CrossBwdWs ws;
  unsigned long long limit_ns;
  float scale_log2;
  long long tiles;  // of the vectors, a head
};

// A run of streamed tiles of one unit.
struct alignas(16) BwdSeg {
  int valid;
  int head;   // key/value head
  int fix0;   // first row of the fixed tile in its tensor
  int fix_n;  // its keys (bwd_by_key) or tokens
  int tok0;   // MODE 1: its first token within the sequence
  int str0;   // the sequence's first row in the streamed tensor
  int str_n;  // its tokens (bwd_by_key) or keys
  int vec0;   // its first tile of the vectors
  int s0;     // first streamed tile
  int n;      // streamed tiles
  int pad;
  int out;    // 0: the unit is whole; 1, 2: part 0, part 1 of this CTA
};
static_assert(sizeof(BwdSeg) == 48, "segment size");

template <int D, int MODE>
struct CrossBwdCfg : BwdBase<D, MODE> {
  using C = BwdBase<D, MODE>;
  static constexpr int OFF_SEG = C::OFF_MISC + 576;
  static constexpr int OFF_PLAN = OFF_SEG + kBwdSegRing * static_cast<int>(sizeof(BwdSeg));
  static constexpr bool BY_KEY = bwd_by_key(MODE);      // K and V stay, Q and dO stream past, with the vectors
  static constexpr bool DV = MODE == 0 || MODE == 3;
  static constexpr bool DP = MODE != 3;                 // dP is formed, and dK or dQ
  // Warps: 0-7 elementwise, 8 MMA, 9 load; d = 256: 10 MMA of the accumulators, 11 of dP.  One warp takes some 65 cycles for each
  // product, which of few streamed rows is more than the tensor core takes (6 sequences of 100 to 700 rows, d = 256, 32 rows a tile: 242 us
  // with one, 203 with two); else the warps' signals to each other cost more (d = 128, 1 to 4 K rows: 1.27 ms with one, 1.41 with two).
  static constexpr bool ACC_APART = D == 256;
  static constexpr int ACC_WARP = C::LOAD_WARP + 1;
  static constexpr bool DP_APART = ACC_APART && DP;
  static constexpr int THREADS = DP_APART ? 384 : ACC_APART ? 352 : 320;
  static constexpr int READERS = THREADS / 32 - 1;
  // A stage's vectors.
  static __device__ __forceinline__ int off_vec(int st) {
    return MODE == 0 ? C::OFF_ST + st * C::STAGE + 2 * C::S_TILE : C::OFF_MISC + 1024 + st * (DP ? 2 : 1) * C::VEC_BYTES;
  }
  static_assert(C::OFF_ABORT + 4 <= OFF_SEG && OFF_PLAN + sizeof(PlanScratch) <= C::OFF_MISC + 1024, "misc area");
};

template <int D, int MODE>
struct CrossBwdBars : BwdBars<D, MODE> {
  using Base = BwdBars<D, MODE>;
  __device__ __forceinline__ uint32_t seg_full(int i) const { return this->b0 + 256 + 8u * i; }
  __device__ __forceinline__ uint32_t seg_empty(int i) const { return this->b0 + 288 + 8u * i; }
  static_assert(Base::COUNT * 8 <= 256, "barrier area");
};
template <int MODE>
struct CrossBwdBars<256, MODE> {
  using C = BwdWideCfg<MODE>;
  uint32_t b0;
  __device__ __forceinline__ uint32_t fix_full() const { return b0; }
  __device__ __forceinline__ uint32_t fix_empty() const { return b0 + 8; }
  __device__ __forceinline__ uint32_t a_full(int i) const { return b0 + 16 + 8u * i; }
  __device__ __forceinline__ uint32_t a_empty(int i) const { return b0 + 32 + 8u * i; }
  __device__ __forceinline__ uint32_t b_full(int i) const { return b0 + 48 + 8u * i; }
  __device__ __forceinline__ uint32_t b_empty(int i) const { return b0 + 184 + 8u * i; }
  __device__ __forceinline__ uint32_t st_full(int i) const { return C::DP ? a_full(i) : b_full(i); }
  __device__ __forceinline__ uint32_t st_empty(int i) const { return C::DP ? a_empty(i) : b_empty(i); }
  __device__ __forceinline__ uint32_t s_full(int b) const { return b0 + 96 + 8u * b; }
  __device__ __forceinline__ uint32_t p_ready(int b) const { return b0 + 112 + 8u * b; }
  // The accumulations that read P or dS in buffer b are complete.
  __device__ __forceinline__ uint32_t buf_free(int b) const { return b0 + 128 + 8u * b; }
  __device__ __forceinline__ uint32_t out_done() const { return b0 + 144; }
  __device__ __forceinline__ uint32_t out_free() const { return b0 + 152; }
  __device__ __forceinline__ uint32_t drain() const { return b0 + 160; }
  __device__ __forceinline__ uint32_t drain_acc() const { return b0 + 168; }
  __device__ __forceinline__ uint32_t drain_dp() const { return b0 + 176; }
  __device__ __forceinline__ uint32_t seg_full(int i) const { return b0 + 256 + 8u * i; }
  __device__ __forceinline__ uint32_t seg_empty(int i) const { return b0 + 288 + 8u * i; }
  static_assert(C::NA <= 2 && C::NB <= 4, "barrier area");
};

// Products of d = 256.
template <int MODE>
struct BwdWideMma {
  using C = BwdWideCfg<MODE>;
  static constexpr uint32_t IDESC_S = make_idesc_bf16(128, C::BS, 0);
  static constexpr uint32_t IDESC_O = make_idesc_bf16(128, C::OUTW, 1);
  static constexpr uint32_t HI = sdesc_hi(8 * C::SWB, C::SWZ);
  template <int REGION>
  static constexpr __host__ __device__ uint32_t k_step(int kk) {
    return ((kk * 16 / C::RC) * REGION + (kk * 16 % C::RC) * 2) >> 4;
  }
  template <int OFF>
  struct Steps {  // runs that start at K step OFF
    static constexpr __host__ __device__ uint32_t da(int k) { return k_step<C::FIX_REGION>(OFF + k) - k_step<C::FIX_REGION>(OFF + k - 1); }
    static constexpr __host__ __device__ uint32_t db(int k) { return k_step<C::S_REGION>(OFF + k) - k_step<C::S_REGION>(OFF + k - 1); }
  };
  struct AccSteps {
    static constexpr __host__ __device__ uint32_t ta(int) { return 8; }
    static constexpr __host__ __device__ uint32_t db(int) { return 16 * C::SWB >> 4; }
  };
  uint32_t tmem, base;
  // S = A1 A^T with the tile in `slot` of ring A, into buffer b.
  __device__ __forceinline__ void s(uint32_t slot, int b) const {
    const uint32_t d = tmem + C::TM_S + b * C::BS, x = sdesc_lo(base + C::OFF_FIX, 16);
    const uint32_t y = sdesc_lo(base + C::OFF_A, 16) + slot * (C::S_TILE >> 4);
    mma_ss_run<8, Steps<0>>(d, x, HI, y, HI, IDESC_S, 0u);
    mma_ss_run<8, Steps<8>>(d, x + k_step<C::FIX_REGION>(8), HI, y + k_step<C::S_REGION>(8), HI, IDESC_S, 1u);
  }
  // Region r of dP = A2 B^T, into buffer b.
  __device__ __forceinline__ void dp(uint32_t r, int b) const {
    mma_ss_run<4, Steps<0>>(tmem + C::TM_DP + b * C::BS, sdesc_lo(base + C::OFF_FIX + C::FIX_TILE, 16) + r * (C::FIX_REGION >> 4), HI,
                            sdesc_lo(base + C::OFF_B, 16) + r * (C::S_REGION >> 4), HI, IDESC_S, r > 0 ? 1u : 0u);
  }
  // dQ (+)= dS K, dV (+)= P^T dO, dK (+)= dS^T Q.
  __device__ __forceinline__ void add(uint32_t slot, int b, bool acc) const {
    mma_ts_run<C::BS / 16, AccSteps>(tmem + C::TM_OUT, tmem + (C::DP ? C::TM_DP : C::TM_S) + b * C::BS,
                                     sdesc_lo(base + C::OFF_ST, C::S_REGION) + slot * (C::S_TILE >> 4), HI, IDESC_O, acc ? 1u : 0u);
  }
};

// The units of a sequence.
struct BwdUnits {
  int fix;    // fixed tiles a head
  int str;    // streamed tiles
  int units;  // fixed tiles x heads
  int w;      // places of a streamed tile on the line
  // Places of a unit.
  template <int COST>
  __host__ __device__ __forceinline__ int length() const { return str * w + COST; }
};
template <int D, int MODE>
__host__ __device__ __forceinline__ BwdUnits bwd_units(const CrossArgs& a, const CrossSeq& s) {
  using C = BwdWork<D, MODE>;
  BwdUnits u = {0, 0, 0, 1};
  if (s.n == 0 || s.len == 0) return u;  // the gradients are zeros: the preparing kernel writes them
  if (bwd_short<D>(s, a.group) != (MODE == 2)) return u;
  if (MODE == 2) {
    u.fix = 1;
    u.str = (s.len + C::STR - 1) / C::STR;
    if constexpr (MODE == 2) {
      const int t = bwd_tokens1(a.group), full = s.n / t, rest = s.n % t;  // whole row tiles, and tokens of the last one
      u.w = full * ((t * a.group + C::QT - 1) / C::QT) + (rest * a.group + C::QT - 1) / C::QT + C::TILE_COST;
    }
  } else if (bwd_by_key(MODE)) {
    const int t = bwd_tokens0<D>(a.group);
    u.fix = (s.len + 127) / 128;
    u.str = (s.n + t - 1) / t;
  } else {
    const int t = bwd_tokens1(a.group);
    u.fix = (s.n + t - 1) / t;
    u.str = (s.len + C::STR - 1) / C::STR;
  }
  u.units = u.fix * a.heads;
  return u;
}

// ------------------------------------------------------------------ segments
template <int D, int MODE>
struct CrossBwdWalk {
  using C = BwdWork<D, MODE>;
  int b, u, j;
  int vec0;  // the sequence's first tile of the vectors
  CrossSeq s;
  BwdUnits c;
  long long pos, end;   // on the line
  long long last_tile;  // of the latest segment's unit
  int record_u;         // the latest segment's unit
  int record_b;
  __device__ __forceinline__ void load(const CrossBwdParams& p) {
    bool bad;
    s = cross_seq(p.a.cb, b, bad);
    c = bwd_units<D, MODE>(p.a, s);
    // (Written by a kernel that is not the one before: past L1.  Not written where there is nothing to multiply, nor for what ranges that share
    // rows have too much: there it is anything, cut so that a sequence's tiles from there on are the workspace's.)
    vec0 = static_cast<int>(min(__ldcg(p.ws.tile0 + b), static_cast<uint32_t>(p.tiles)));
  }
  __device__ __forceinline__ void start(const CrossBwdParams& p, const PlanShare& w) {
    pos = w.start;
    end = w.end;
    b = w.b;
    if (pos >= end) return;
    load(p);
    const int unit = c.template length<C::UNIT_COST>();
    u = static_cast<int>(w.offset / unit);
    const int in = static_cast<int>(w.offset - static_cast<long long>(u) * unit);
    // The first tile that begins at the share's first place or behind it.
    j = (in + c.w - 1) / c.w;
    if (j >= c.str) {
      pos += unit - in;
      enter(p);
    } else {
      pos += j * c.w - in;
    }
  }
  // On to the next unit, if the share reaches it.
  __device__ __forceinline__ void enter(const CrossBwdParams& p) {
    j = 0;
    if (pos >= end) return;
    if (++u < c.units) return;
    u = 0;
    do {
      ++b;
      load(p);
    } while (c.units == 0);
  }
  __device__ __forceinline__ BwdSeg next(const CrossBwdParams& p) {
    BwdSeg g = {};
    if (pos >= end) return g;
    const long long begin = (end - pos + c.w - 1) / c.w;  // tiles that begin before the share's end
    const int n = begin < c.str - j ? static_cast<int>(begin) : c.str - j;
    g.valid = 1;
    const int tile = u % c.fix;
    g.head = u / c.fix;
    if (bwd_by_key(MODE)) {
      g.fix0 = s.key0 + tile * 128;
      g.fix_n = min(128, s.len - tile * 128);
      g.str0 = s.row0;
      g.str_n = s.n;
    } else {
      g.tok0 = tile * bwd_tokens1(p.a.group);
      g.fix0 = s.row0 + g.tok0;
      g.fix_n = MODE == 2 ? s.n : min(bwd_tokens1(p.a.group), s.n - g.tok0);
      g.str0 = s.key0;
      g.str_n = s.len;
    }
    g.vec0 = vec0;
    g.s0 = j;
    g.n = n;
    g.out = n == c.str ? 0 : j == 0 ? 2 : 1;
    last_tile = pos + static_cast<long long>(c.str - 1 - j) * c.w;
    record_u = u;
    record_b = b;
    pos += static_cast<long long>(n) * c.w;
    j += n;
    if (j == c.str) {
      pos += C::UNIT_COST;
      enter(p);
    }
    return g;
  }
};

// warp_wait_bar; d = 256: all but the first try out of line (with five or six roles and less code 150.5 us instead of 155 at 6 sequences of 100
// to 700 rows; in the kernels of d <= 128 it costs 1 to 5 %).
static __device__ __noinline__ bool bwd_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit_ns, int code) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, WaitGuard{abort, status, limit_ns}, code));
}
template <int D>
__device__ __forceinline__ bool bwd_wait(uint32_t bar, uint32_t parity, const WaitGuard& g, int code) {
  if constexpr (D == 256)
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || bwd_wait_slow(bar, parity, g.abort, g.status, g.limit_ns, code);
  else
    return warp_wait_bar(bar, parity, g, code);
}

// Segment k of the ring at `ring`, read by a whole warp of a role other than the load warp.
template <class Bars>
__device__ __forceinline__ bool bwd_seg_read(BwdSeg& g, int k, const uint8_t* ring, const Bars& bar, const WaitGuard& guard) {
  if (!warp_wait_bar(bar.seg_full(k % kBwdSegRing), (k / kBwdSegRing) & 1, guard, kStatusTimeoutLoad)) return false;
  const int4* src = reinterpret_cast<const int4*>(reinterpret_cast<const BwdSeg*>(ring) + (k % kBwdSegRing));
  int4* dst = reinterpret_cast<int4*>(&g);
#pragma unroll
  for (int i = 0; i < 3; ++i) dst[i] = src[i];
  warp_arrive(bar.seg_empty(k % kBwdSegRing));
  return true;
}

// ------------------------------------------------------------------ load warp
template <int D, int MODE>
__device__ __forceinline__ void cross_bwd_load(const CUtensorMap* tm_a1, const CUtensorMap* tm_a2, const CUtensorMap* tm_b1,
                                               const CUtensorMap* tm_b2, const CrossBwdParams& p,
                                               const CrossBwdBars<D, MODE>& bar, uint32_t base, uint8_t* gbase,
                                               const PlanShare& share, const WaitGuard& g) {
  using C = CrossBwdCfg<D, MODE>;
  const int lane = threadIdx.x & 31;
  const uint64_t pol_fix = policy_evict_first();  // read by one unit
  const uint64_t pol_str = policy_evict_last();   // read by every unit of the head
  const int group = p.a.group;
  const int t0 = bwd_tokens0<D>(group), t1 = bwd_tokens1(group);
  uint32_t pos = 0;       // stages issued so far
  uint32_t issued = 0;    // bit i: stage i has been loaded at least once
  uint32_t last_par = 0;  // bit i: parity of stage i's latest load
  int last_fix = -1;      // latest segment whose fixed tiles were loaded
  bool recorded = false, ok = true;
  CrossBwdWalk<D, MODE> walk;
  walk.start(p, share);
  for (int k = 0;; ++k) {
    const int i = k % kBwdSegRing;
    if (!(ok = bwd_wait<D>(bar.seg_empty(i), ((k / kBwdSegRing) & 1) ^ 1, g, kStatusTimeoutLoad))) break;
    const BwdSeg w = walk.next(p);
    if (lane == 0) {
      reinterpret_cast<BwdSeg*>(gbase + C::OFF_SEG)[i] = w;
      if (w.out == 2)  // this unit's first part: who holds the rest
        p.ws.rec[bwd_place(MODE)][blockIdx.x] =
            PlanRecord{walk.record_b, w.head, walk.record_u,
                       plan_cta_of(walk.last_tile, share.total, share.ctas) - static_cast<int>(blockIdx.x)};
    }
    recorded = recorded || w.out == 2;
    warp_arrive(bar.seg_full(i));
    if (!w.valid) break;
    // The fixed tiles: K, V (128 keys of a head), or Q, dO (a group's heads of 128 / G tokens).
    if (!(ok = bwd_wait<D>(bar.fix_empty(), (k & 1) ^ 1, g, kStatusTimeoutLoad))) break;
    if (lane == 0) {
      const int rows = C::BY_KEY ? 128 : t1 * group;
      mbar_arrive_expect_tx(bar.fix_full(), (C::DP ? 2 : 1) * C::NR * rows * C::SWB);
      for (int r = 0; r < C::NR; ++r) {
        const uint32_t dst = base + C::OFF_FIX + r * C::FIX_REGION;
        const int h = C::BY_KEY ? w.head : w.head * group;
        tma_load_3d(dst, tm_a1, bar.fix_full(), r * C::RC, h, w.fix0, pol_fix);
        if (C::DP) tma_load_3d(dst + C::FIX_TILE, tm_a2, bar.fix_full(), r * C::RC, h, w.fix0, pol_fix);
      }
    }
    last_fix = k;
    for (int t = 0; t < w.n; ++t) {
      if constexpr (D == 256) {
        const int rows = C::BY_KEY ? t0 * group : C::BS;
        const int s = w.s0 + t, h = C::BY_KEY ? w.head * group : w.head;
        const int row = w.str0 + s * (C::BY_KEY ? t0 : C::BS);
        // Into slot `slot` of a ring (A: x = 0): the regions [r0, r1), and the vectors.
        auto load = [&](int x, int slot, uint32_t par, int r0, int r1, bool vecs) -> bool {
          if (!bwd_wait<D>(x ? bar.b_empty(slot) : bar.a_empty(slot), par ^ 1, g, kStatusTimeoutLoad)) return false;
          if (lane == 0) {
            const uint32_t full = x ? bar.b_full(slot) : bar.a_full(slot);
            const uint32_t dst = base + (x ? C::OFF_B + slot * C::B_BYTES : C::OFF_A + slot * C::S_TILE);
            mbar_arrive_expect_tx(full, (r1 - r0) * rows * C::SWB + (vecs ? (C::DP ? 2 : 1) * C::VEC_BYTES : 0));
            for (int r = r0; r < r1; ++r)
              tma_load_3d(dst + (r - r0) * C::S_REGION, x ? tm_b2 : tm_b1, full, r * C::RC, h, row, pol_str);
            if (vecs) {
              const long long off = (w.head * p.tiles + w.vec0 + s) * C::BS;
              bulk_load(base + C::off_vec(slot), p.ws.l2 + off, C::VEC_BYTES, full);
              if (C::DP) bulk_load(base + C::off_vec(slot) + C::VEC_BYTES, p.ws.dsum + off, C::VEC_BYTES, full);
            }
          }
          const int bit = x * 4 + slot;
          issued |= 1u << bit;
          last_par = (last_par & ~(1u << bit)) | (par << bit);
          return true;
        };
        // (What dP alone reads is free first.)
        if constexpr (C::DP)
          for (int r = 0; ok && r < C::NR; ++r) ok = load(1, r, pos & 1, r, r + 1, false);
        ok = ok && load(0, pos % C::NA, (pos / C::NA) & 1, 0, C::NR, C::BY_KEY && C::DP);
        if constexpr (!C::DP) ok = ok && load(1, pos % C::NB, (pos / C::NB) & 1, 0, C::NR, true);
        if (!ok) break;
        ++pos;
      } else {
        const int st = pos % C::NST;
        const uint32_t par = (pos / C::NST) & 1;
        if (!(ok = bwd_wait<D>(bar.st_empty(st), par ^ 1, g, kStatusTimeoutLoad))) break;
        if (lane == 0) {
          const uint32_t s0 = base + C::OFF_ST + st * C::STAGE;
          const uint32_t full = bar.st_full(st);
          const int rows = C::BY_KEY ? t0 * group : C::BS;
          mbar_arrive_expect_tx(full, 2 * C::NR * rows * C::SWB + (C::BY_KEY ? (C::DP ? 2 : 1) * C::VEC_BYTES : 0));
          const int s = w.s0 + t, h = C::BY_KEY ? w.head * group : w.head;
          const int row = w.str0 + s * (C::BY_KEY ? t0 : C::BS);
          for (int r = 0; r < C::NR; ++r) {
            tma_load_3d(s0 + r * C::S_REGION, tm_b1, full, r * C::RC, h, row, pol_str);
            tma_load_3d(s0 + C::S_TILE + r * C::S_REGION, tm_b2, full, r * C::RC, h, row, pol_str);
          }
          if constexpr (C::BY_KEY) {
            // (BS * 4 is a multiple of 16.)
            const long long off = (w.head * p.tiles + w.vec0 + s) * C::BS;
            const uint32_t vec = base + C::off_vec(st);
            bulk_load(vec, p.ws.l2 + off, C::VEC_BYTES, full);
            if (C::DP) bulk_load(vec + C::VEC_BYTES, p.ws.dsum + off, C::VEC_BYTES, full);
          }
        }
        issued |= 1u << st;
        last_par = (last_par & ~(1u << st)) | (par << st);
        ++pos;
      }
    }
    if (!ok) break;
  }
  if (lane == 0 && !recorded) p.ws.rec[bwd_place(MODE)][blockIdx.x].b = -1;
  // Every issued copy must land before the CTA may exit.
  if constexpr (D == 256) {
    for (int i = 0; i < 8; ++i)
      if (issued & (1u << i)) bwd_wait_drain(i < 4 ? bar.a_full(i) : bar.b_full(i - 4), (last_par >> i) & 1, g);
  } else {
    for (int i = 0; i < C::NST; ++i)
      if (issued & (1u << i)) bwd_wait_drain(bar.st_full(i), (last_par >> i) & 1, g);
  }
  if (last_fix >= 0) bwd_wait_drain(bar.fix_full(), last_fix & 1, g);
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issuer
template <int D>
struct CrossIssuer {
  const WaitGuard& g;
  __device__ __forceinline__ bool wait(uint32_t b, uint32_t par) const {
    if constexpr (D == 256) return bwd_wait<D>(b, par, g, kStatusTimeoutMma);
    const bool r = mbar_test_wait(b, par) || wait_bar(b, par, g, kStatusTimeoutMma);
    return __all_sync(0xffffffffu, r);
  }
  // All products issued must complete before TMEM is released.
  __device__ __forceinline__ void finish(uint32_t drain) const {
    mma_commit_elect(drain);
    bwd_wait_drain(drain, 0, g);
    __syncwarp();
  }
};

// bwd_mma's order of products, segment by segment.
template <int D, int MODE>
__device__ __forceinline__ void cross_bwd_mma(const CrossBwdBars<D, MODE>& bar, uint32_t base,
                                              uint8_t* gbase, uint32_t tmem, const WaitGuard& g) {
  using C = CrossBwdCfg<D, MODE>;
  const BwdMma<D, MODE> M(tmem, base);
  const CrossIssuer<D> is{g};
  uint32_t pos = 0;            // streamed stages consumed before the current segment
  uint32_t pr0 = 0, pr1 = 0;   // p_ready phases consumed, per buffer
  bool ok = true;
  for (int k = 0; ok; ++k) {
    BwdSeg w;
    if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
    const int n = w.n;
    if (!(ok = is.wait(bar.fix_full(), k & 1))) break;
    tc_fence_after();
    auto stage_of = [&](int t) -> uint32_t { return (pos + t) % C::NST; };
    auto acquire = [&](int t) -> bool {
      const uint32_t q = pos + t;
      if (!is.wait(bar.st_full(q % C::NST), (q / C::NST) & 1)) return false;
      tc_fence_after();
      return true;
    };
    for (int t = 0; ok && t < n && t < 2; ++t) {
      if (!(ok = acquire(t))) break;
      M.sdp(stage_of(t), t & 1);
      mma_commit_elect(bar.s_full(t & 1));
      if (t == n - 1) mma_commit_elect(bar.fix_empty());
    }
    for (int t = 0; ok && t < n; ++t) {
      const int b = t & 1;
      uint32_t& pr = b ? pr1 : pr0;
      if (!(ok = is.wait(bar.p_ready(b), pr & 1))) break;
      ++pr;
      tc_fence_after();
      if (t == 0 && k > 0) {
        if (!(ok = is.wait(bar.out_free(), (k - 1) & 1))) break;
        tc_fence_after();
      }
      M.accumulate(stage_of(t), b, t > 0, 0);
      mma_commit_elect(bar.st_empty(stage_of(t)));
      if (t + 2 < n) {
        if (!(ok = acquire(t + 2))) break;
        M.sdp(stage_of(t + 2), b);
        mma_commit_elect(bar.s_full(b));
        if (t + 2 == n - 1) mma_commit_elect(bar.fix_empty());
      }
    }
    if (!ok) break;
    pos += n;
    mma_commit_elect(bar.out_done());
  }
  is.finish(bar.drain());
}

// d = 256: S (X = 0) or dP, segment by segment, up to two tiles ahead of the accumulations.
template <int MODE, int X>
__device__ __forceinline__ void cross_bwd_first(const CrossBwdBars<256, MODE>& bar, uint32_t base, uint8_t* gbase, uint32_t tmem,
                                                const WaitGuard& g) {
  using C = CrossBwdCfg<256, MODE>;
  const BwdWideMma<MODE> M{tmem, base};
  const CrossIssuer<256> is{g};
  uint32_t pos = 0;                // streamed tiles issued
  uint32_t used[2] = {0, 0};       // into the buffers
  bool ok = true;
  for (int k = 0; ok; ++k) {
    BwdSeg w;
    if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
    if (!(ok = is.wait(bar.fix_full(), k & 1))) break;
    for (int t = 0; ok && t < w.n; ++t, ++pos) {
      const int b = t & 1;
      uint32_t& u = b ? used[1] : used[0];
      if (u > 0 && !(ok = is.wait(bar.buf_free(b), (u - 1) & 1))) break;
      ++u;
      if constexpr (X == 0) {
        const uint32_t slot = pos % C::NA;
        if (!(ok = is.wait(bar.a_full(slot), (pos / C::NA) & 1))) break;
        tc_fence_after();
        M.s(slot, b);
        mma_commit_elect(bar.s_full(b));
        if (!C::DP) mma_commit_elect(bar.a_empty(slot));  // (no other product reads the tile)
      } else {
#pragma unroll 1
        for (int r = 0; r < C::NR; ++r) {
          if (!(ok = is.wait(bar.b_full(r), pos & 1))) break;
          tc_fence_after();
          M.dp(r, b);
          mma_commit_elect(bar.b_empty(r));
        }
        if (!ok) break;
        mma_commit_elect(bar.s_full(b));
      }
      if (t == w.n - 1) mma_commit_elect(bar.fix_empty());
    }
  }
  is.finish(X ? bar.drain_dp() : bar.drain());
}

// d = 256: the accumulations.
template <int MODE>
__device__ __forceinline__ void cross_bwd_acc(const CrossBwdBars<256, MODE>& bar, uint32_t base, uint8_t* gbase, uint32_t tmem,
                                              const WaitGuard& g) {
  using C = CrossBwdCfg<256, MODE>;
  const BwdWideMma<MODE> M{tmem, base};
  const CrossIssuer<256> is{g};
  uint32_t pos = 0;            // streamed tiles consumed
  uint32_t pr0 = 0, pr1 = 0;   // p_ready phases consumed, per buffer
  bool ok = true;
  for (int k = 0; ok; ++k) {
    BwdSeg w;
    if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
    for (int t = 0; t < w.n; ++t, ++pos) {
      const int b = t & 1;
      const uint32_t slot = pos % C::NST;
      uint32_t& pr = b ? pr1 : pr0;
      if (!(ok = is.wait(bar.st_full(slot), (pos / C::NST) & 1))) break;
      if (!(ok = is.wait(bar.p_ready(b), pr & 1))) break;
      ++pr;
      if (t == 0 && k > 0 && !(ok = is.wait(bar.out_free(), (k - 1) & 1))) break;
      tc_fence_after();
      M.add(slot, b, t > 0);
      mma_commit_elect(bar.buf_free(b));
      mma_commit_elect(bar.st_empty(slot));
    }
    if (!ok) break;
    mma_commit_elect(bar.out_done());
  }
  is.finish(bar.drain_acc());
}

// ------------------------------------------------------------------ elementwise warpgroups
// bwd_elementwise without a causal mask; outputs as bf16, or a part's in fp32.
template <int D, int MODE>
__device__ __forceinline__ void cross_bwd_elementwise(const CrossBwdParams& p, const CrossBwdBars<D, MODE>& bar,
                                                      uint8_t* gbase, uint32_t tmem, int b, int quarter, int lane,
                                                      const WaitGuard& g) {
  using C = CrossBwdCfg<D, MODE>;
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const float sl2 = p.scale_log2;
  const uint64_t sl2x2 = f2_pack(sl2, sl2);
  // MODE 1: this thread's token within the fixed tile, and its head of the group.
  const int per = C::BY_KEY ? bwd_tokens0<D>(p.a.group) : C::BS;  // tokens or keys of a streamed tile
  const int tok_r = C::BY_KEY ? 0 : r / p.a.group, head_r = C::BY_KEY ? 0 : r - tok_r * p.a.group;
  uint32_t sf = 0;    // s_full(b) phases consumed
  uint32_t pos = 0;   // streamed stages before the current segment
  bool ok = true;
  for (int k = 0; ok; ++k) {
    BwdSeg w;
    if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
    const int n = w.n;
    const bool mine = C::BY_KEY ? r < w.fix_n : tok_r < w.fix_n;  // (tokens: fix_n <= 128 / G)
    uint64_t l2_row = 0, d_row = 0;  // MODE 1: this row's -L * log2(e) and -D, twice
    if constexpr (MODE == 1) {
      float l2 = -INFINITY, dsum = 0.f;
      if (mine) {
        const int t0 = bwd_tokens0<D>(p.a.group), tok = w.tok0 + tok_r;
        const long long at = (w.head * p.tiles + w.vec0 + tok / t0) * bwd_rows0<D>() + tok % t0 * p.a.group + head_r;
        // (Written by a kernel that is not the one before: past L1.)
        l2 = __ldcg(p.ws.l2 + at);
        dsum = __ldcg(p.ws.dsum + at);
      }
      l2_row = f2_pack(l2, l2);
      d_row = f2_pack(dsum, dsum);
    }
    for (int t = b; ok && t < n; t += 2) {
      ok = bwd_wait<D>(bar.s_full(b), sf & 1, g, kStatusTimeoutSoftmax);
      if (!ok) break;
      ++sf;
      const uint32_t q = pos + t;
      const int st = q % C::NST;
      if constexpr (C::BY_KEY) {
        // The stage's vectors were written by TMA; observe that completion here too.
        ok = bwd_wait<D>(bar.st_full(st), (q / C::NST) & 1, g, kStatusTimeoutSoftmax);
        if (!ok) break;
      }
      tc_fence_after();
      // Rows of the tile that are a token's or a key's; the others are not looked at in S and dP, but meet zeros of P and dS in
      // the accumulations.
      const int there = C::BY_KEY ? min(w.str_n - (w.s0 + t) * per, per) * p.a.group : w.str_n - (w.s0 + t) * per;
      const bool need_mask = there < C::BS;
      if (need_mask) {
        // (Of the tiles that the accumulations read: MODE 0 both.)
        const uint32_t tile = smem_u32(gbase + C::OFF_ST + st * C::STAGE);
        for (int x = r; x < (MODE == 0 ? 2 : 1) * C::BS; x += 128) {
          const int row = x % C::BS;
          if (row < there) continue;
#pragma unroll
          for (int u = 0; u < D / 8; ++u)
            st_shared_v4(tile + x / C::BS * C::S_TILE + u / (C::SWB / 16) * C::S_REGION + row * C::SWB + u % (C::SWB / 16) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      const float4* vl2 = reinterpret_cast<const float4*>(gbase + (C::BY_KEY ? C::off_vec(st) : 0));
      const float4* vd = vl2 + C::BS / 4;
#pragma unroll 1
      for (int h = 0; h < C::BS / 32; ++h) {
        uint32_t rs[32], rd[32];
        tmem_ld32(tmem + lane_off + C::TM_S + b * C::BS + h * 32, rs);
        if constexpr (C::DP) tmem_ld32(tmem + lane_off + C::TM_DP + b * C::BS + h * 32, rd);
        tmem_wait_ld(rs);
        if constexpr (C::DP) tmem_wait_ld(rd);
        uint32_t pk[16], dk[16];
#pragma unroll
        for (int c4 = 0; c4 < 8; ++c4) {
          // -L * log2(e) and -D of the four streamed rows (MODE 0) or of this row (MODE 1).
          uint64_t nl[2], nd[2];
          if constexpr (C::BY_KEY) {
            const float4 a = vl2[h * 8 + c4];
            nl[0] = f2_pack(a.x, a.y);
            nl[1] = f2_pack(a.z, a.w);
            if constexpr (C::DP) {
              const float4 d4 = vd[h * 8 + c4];
              nd[0] = f2_pack(d4.x, d4.y);
              nd[1] = f2_pack(d4.z, d4.w);
            }
          } else {
            nl[0] = nl[1] = l2_row;
            nd[0] = nd[1] = d_row;
          }
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            const int c = c4 * 4 + e2 * 2;
            const float2 x = f2_unpack(f2_fma(f2_pack(__uint_as_float(rs[c]), __uint_as_float(rs[c + 1])), sl2x2, nl[e2]));
            float p0 = ex2(x.x), p1 = ex2(x.y);
            float2 ds = {0.f, 0.f};
            if constexpr (C::DP)
              ds = f2_unpack(f2_mul(f2_pack(p0, p1), f2_add(f2_pack(__uint_as_float(rd[c]), __uint_as_float(rd[c + 1])), nd[e2])));
            if (need_mask) {
              if (h * 32 + c >= there) p0 = ds.x = 0.f;
              if (h * 32 + c + 1 >= there) p1 = ds.y = 0.f;
            }
            pk[c4 * 2 + e2] = pack_bf16x2(p0, p1);
            dk[c4 * 2 + e2] = pack_bf16x2(ds.x, ds.y);
          }
        }
        // As in bwd_elementwise: chunk h's bf16 pairs land behind what has been read.
        if constexpr (C::DV) tmem_st16(tmem + lane_off + C::TM_S + b * C::BS + h * 16, pk);
        if constexpr (C::DP) tmem_st16(tmem + lane_off + C::TM_DP + b * C::BS + h * 16, dk);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bar.p_ready(b));
    }
    if (!ok) break;
    pos += n;
    // Read the unit's accumulators out.
    ok = bwd_wait<D>(bar.out_done(), k & 1, g, kStatusTimeoutSoftmax);
    if (!ok) break;
    tc_fence_after();
    const bool second = MODE == 0 && b == 1;
    const bool dv = second || MODE == 3;
    const uint32_t acc = tmem + lane_off + C::TM_OUT + (second ? C::OUTW : 0);
    const float f = dv ? 1.f : p.a.scale;  // dK and dQ carry the softmax scale
    const uint64_t f2 = f2_pack(f, f);
    __nv_bfloat16* out = MODE == 1 ? p.a.dq : dv ? p.a.dv : p.a.dk;
    const long long* os = p.a.st[MODE == 1 ? 5 : dv ? 7 : 6];
    const int head = C::BY_KEY ? w.head : w.head * p.a.group + head_r;
    const long long row = w.fix0 + (C::BY_KEY ? r : tok_r);
    __nv_bfloat16* orow = out + row * os[0] + head * os[1];
    float4* part = reinterpret_cast<float4*>(p.ws.part[bwd_place(MODE)] + (blockIdx.x * 2 + (w.out - 1)) * BwdWork<D, MODE>::PART +
                                             (second ? 128 * C::OUTW : 0)) + r;
#pragma unroll 1
    for (int c = 0; c < C::OUTW / 32; ++c) {
      if (MODE != 0 && (c & 1) != b) continue;
      uint32_t v[32];
      tmem_ld32(acc + c * 32, v);
      tmem_wait_ld(v);
      if (w.out == 0) {
        uint32_t packed[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 y = f2_unpack(f2_mul(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2));
          packed[i] = pack_bf16x2(y.x, y.y);
        }
        if (mine) {
          uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(packed[4 * i], packed[4 * i + 1], packed[4 * i + 2], packed[4 * i + 3]);
        }
      } else {
        // 16-byte block i of all 128 rows together.
#pragma unroll
        for (int i = 0; i < 8; ++i)
          part[(c * 8 + i) * 128] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
      }
    }
    tc_fence_before();
    warp_arrive(bar.out_free());
  }
}

// ------------------------------------------------------------------ kernel
template <int D, int MODE>
__global__ void __launch_bounds__(CrossBwdCfg<D, MODE>::THREADS, 1)
    fa_cross_bwd_kernel(const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_a2,
                        const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ CUtensorMap tm_b2,
                        const __grid_constant__ CrossBwdParams p) {
  using C = CrossBwdCfg<D, MODE>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  CrossBwdBars<D, MODE> bar;
  bar.b0 = base + C::OFF_MISC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_TMEM_SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_ABORT);

  // The kernel that comes first waits for the preparing one; those behind it begin when all of its CTAs have done so.
  constexpr bool FIRST = MODE == 3;
  const PlanShare share = plan_share<C::THREADS>(
      p.a.cb.B, gridDim.x, blockIdx.x,
      [&](int b) -> long long {
        bool bad;
        const BwdUnits u = bwd_units<D, MODE>(p.a, cross_seq(p.a.cb, b, bad));
        return u.units == 0 ? 0ll : static_cast<long long>(u.units) * u.template length<BwdWork<D, MODE>::UNIT_COST>();
      },
      1 + BwdWork<D, MODE>::UNIT_COST, *reinterpret_cast<PlanScratch*>(gbase + C::OFF_PLAN));
  if (D < 256 && share.start >= share.end) {  // (where all sequences are short: out of the way at once)
    pdl_launch_dependents();
    if (threadIdx.x == 0) p.ws.rec[bwd_place(MODE)][blockIdx.x].b = -1;
    pdl_wait();
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(bar.fix_full(), 1);
    mbar_init(bar.fix_empty(), C::DP_APART ? 2 : 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar.s_full(b), C::DP_APART ? 2 : 1);
      mbar_init(bar.p_ready(b), 4);
    }
    if constexpr (C::ACC_APART) {
      for (int i = 0; i < C::NA; ++i) {
        mbar_init(bar.a_full(i), 1);
        mbar_init(bar.a_empty(i), 1);
      }
      for (int i = 0; i < C::NB; ++i) {
        mbar_init(bar.b_full(i), 1);
        mbar_init(bar.b_empty(i), 1);
      }
      for (int b = 0; b < 2; ++b) mbar_init(bar.buf_free(b), 1);
      mbar_init(bar.drain_acc(), 1);
      mbar_init(bar.drain_dp(), 1);
    } else {
      for (int i = 0; i < C::NST; ++i) {
        mbar_init(bar.st_full(i), 1);
        mbar_init(bar.st_empty(i), 1);
      }
    }
    mbar_init(bar.out_done(), 1);
    mbar_init(bar.out_free(), 8);
    mbar_init(bar.drain(), 1);
    for (int i = 0; i < kBwdSegRing; ++i) {
      mbar_init(bar.seg_full(i), 1);
      mbar_init(bar.seg_empty(i), C::READERS);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::LOAD_WARP && lane == 0) {
    prefetch_tmap(&tm_a1);
    prefetch_tmap(&tm_a2);
    prefetch_tmap(&tm_b1);
    prefetch_tmap(&tm_b2);
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TM_COLS);
    tmem_relinquish();
  }
  if (FIRST) pdl_wait();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitGuard g{abort_flag, p.a.status, p.limit_ns};

  if (warp < 8) {
    cross_bwd_elementwise<D, MODE>(p, bar, gbase, tmem, warp >> 2, warp & 3, lane, g);
  } else if (warp == C::MMA_WARP) {
    if constexpr (C::ACC_APART)
      cross_bwd_first<MODE, 0>(bar, base, gbase, tmem, g);
    else
      cross_bwd_mma<D, MODE>(bar, base, gbase, tmem, g);
  } else if (warp == C::LOAD_WARP) {
    cross_bwd_load<D, MODE>(&tm_a1, &tm_a2, &tm_b1, &tm_b2, p, bar, base, gbase, share, g);
  } else if (C::ACC_APART && warp == C::ACC_WARP) {
    if constexpr (C::ACC_APART) cross_bwd_acc<MODE>(bar, base, gbase, tmem, g);
  } else {
    if constexpr (C::DP_APART) cross_bwd_first<MODE, 1>(bar, base, gbase, tmem, g);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  if (!FIRST) pdl_wait();  // what waits for this kernel waits for those before it, too
}

// ------------------------------------------------------------------ preparing
// -L log2e and -D of every row into the vectors (-inf and 0 behind a sequence's last), and zeros.
constexpr int kPrepThreads = 256;

// Zeros where no product is made: dK and dV of places behind a sequence's keys and of sequences without rows, dQ of rows without
// keys.  Several blocks to a sequence, a warp to a row.
template <int D>
struct BwdZeros {
  static constexpr int CPR = D / 8;
  int per, x, grid, warp, warps;  // blocks of a sequence; this block's next (sequence, share); ..
  int at = 0, to = 0, q_to = 0;   // the sequence's next row of this warp's; behind its places; behind its rows without keys
  CrossSeq s;
  // `shares`: of different sequences, that a block has where there are fewer sequences than blocks.
  __device__ __forceinline__ BwdZeros(const CrossArgs& a, int block, int grid_, int warp_, int warps_, int shares)
      : per(max(grid_ * shares / a.cb.B, 1)), x(block), grid(grid_), warp(warp_), warps(warps_) {}
  // One row of dK and dV, or of dQ; false behind the last.
  __device__ __forceinline__ bool row(const CrossBwdParams& p) {
    const CrossArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    if (at >= max(to, q_to)) {
      if (x / per >= a.cb.B) return false;
      bool bad;
      s = cross_seq(a.cb, x / per, bad);
      at = x % per * warps + warp + (s.n > 0 ? s.len : 0);
      to = s.places;
      q_to = s.len == 0 ? s.n : 0;
      x += grid;
      return true;
    }
    auto clear = [&](__nv_bfloat16* out, const long long* st, int row0, int heads) {
      for (int c = lane; c < heads * CPR; c += 32)
        *reinterpret_cast<uint4*>(out + (static_cast<long long>(row0) + at) * st[0] + c / CPR * st[1] + c % CPR * 8) = make_uint4(0, 0, 0, 0);
    };
    if (at < to) {
      clear(a.dk, a.st[6], s.key0, a.heads);
      clear(a.dv, a.st[7], s.key0, a.heads);
    }
    if (at < q_to) clear(a.dq, a.st[5], s.row0, a.q_heads);
    at += per * warps;
    return true;
  }
};

// (`zeros`: the kernel for short sequences, which writes them else, is not launched behind this one.)
template <int D>
__global__ void __launch_bounds__(kPrepThreads) fa_cross_prep_kernel(const __grid_constant__ CrossBwdParams p, bool zeros) {
  constexpr int BS = bwd_rows0<D>();
  constexpr int CPR = D / 8;     // 16-byte chunks per row
  constexpr int RPW = 32 / CPR;  // rows per warp step
  constexpr int WARPS = kPrepThreads / 32;
  __shared__ uint32_t s_warp[kPrepThreads / 32], s_first, s_group;
  const CrossArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (blockIdx.x == 0) {
    bool any = false;
    for (int b = threadIdx.x; b < a.cb.B; b += kPrepThreads) {
      bool bad;
      cross_seq(a.cb, b, bad);
      any = any || bad;
    }
    if (any) atomicOr(a.status, kBadBatchBit);
  }
  const int t0 = bwd_tokens0<D>(a.group);
  const int sub = lane / CPR, chunk = lane % CPR;
  // The tiles of all sequences lie on a line, one behind another and heads fastest, that is cut into equal shares.  (A search for a tile's
  // sequence among the offsets would lead astray where one of them names what is not there.)  All is counted in 32 bits and divided
  // so where it fits, with two barriers, for this is the way to a small batch's first product (one sequence of 20 rows, in a graph: 15.4
  // us, with the plan of the products' kernels 17.8).
  auto tiles_of = [&](const CrossSeq& s) -> int { return s.len == 0 ? 0 : (s.n + t0 - 1) / t0; };
  auto tiles_at = [&](int b) -> int {
    bool bad;
    return tiles_of(cross_seq(a.cb, b, bad));
  };
  // Sums end at `most`: ranges that share rows may have more tiles than there are places (those behind are left out then).
  const uint32_t most = static_cast<uint32_t>(p.tiles);
  auto add = [&](uint32_t x, uint32_t y) -> uint32_t { return min(x + y, most); };
  auto scan = [&](uint32_t x) -> uint32_t {
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, k);
      if (lane >= k) x = add(x, y);
    }
    return x;
  };
  // A thread adds up `per` sequences (2000 sequences of 3 rows, whole calls: 292 us; scanned 256 at a time 314).
  const int per = (a.cb.B + kPrepThreads - 1) / kPrepThreads;
  uint32_t mine = 0;
  for (int b = static_cast<int>(threadIdx.x) * per; b < min((static_cast<int>(threadIdx.x) + 1) * per, a.cb.B); ++b) mine = add(mine, tiles_at(b));
  mine = scan(mine);
  auto behind_last = [&](uint32_t x) -> uint32_t {  // of the lane before
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, 1);
    return lane > 0 ? y : 0;
  };
  uint32_t first_of = behind_last(mine);
  if (lane == 31) s_warp[warp] = mine;
  if (threadIdx.x == 0) s_group = s_first = 0;
  __syncthreads();
  uint32_t sum = 0, below = 0;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) {
    if (k == warp) below = sum;
    sum = add(sum, s_warp[k]);
  }
  const uint64_t places = static_cast<uint64_t>(sum) * a.heads;
  auto over = [](uint64_t x, uint32_t y) -> uint64_t { return x >> 32 ? x / y : static_cast<uint32_t>(x) / y; };
  const uint64_t share = places <= gridDim.x ? 1 : over(places + gridDim.x - 1, gridDim.x);
  const uint64_t start = share * blockIdx.x, end = min(start + share, places);
  const uint32_t tile_at = static_cast<uint32_t>(over(start, a.heads));  // of all sequences'
  first_of = add(first_of, below);
  if (first_of <= tile_at && tile_at < add(mine, below)) {
    s_group = threadIdx.x;
    s_first = first_of;
  }
  __syncthreads();
  int b = static_cast<int>(s_group) * per;
  uint32_t before = s_first;  // tiles of the sequences before b
  for (bool found = per == 1 || start >= end; !found && b < a.cb.B;) {  // the sequence of these that holds the share's first tile
    const uint32_t y = scan(b + lane < a.cb.B ? tiles_at(b + lane) : 0u), y0 = behind_last(y);
    const uint32_t behind = __ballot_sync(0xffffffffu, add(before, y) > tile_at);
    found = behind != 0;
    const int at = found ? __ffs(behind) - 1 : 31;
    before = add(before, __shfl_sync(0xffffffffu, found ? y0 : y, at));
    b += found ? at : 32;
  }
  int tile = static_cast<int>(tile_at - before), head = static_cast<int>(start - static_cast<uint64_t>(tile_at) * a.heads);
  int tiles = 0;
  uint32_t tile0 = 0;
  CrossSeq s = {};
  auto load = [&]() {
    bool bad;
    s = cross_seq(a.cb, b, bad);
    tiles = tiles_of(s);
    tile0 = min(before, most - tiles);
  };
  uint32_t left = start < end ? static_cast<uint32_t>(end - start) : 0u;
  if (left > 0) load();
  for (; left > 0; --left) {
    if (tile == 0 && head == 0 && threadIdx.x == 0) p.ws.tile0[b] = tile0;
    const int first = tile * t0;  // token of the tile's first row
#pragma unroll 1
    for (int r = warp * RPW + sub; r < BS; r += WARPS * RPW) {
      const int tok = r / a.group, hq = head * a.group + r % a.group;
      const bool valid = tok < t0 && first + tok < s.n;
      float acc = 0.f, lse = 0.f;
      if (valid) {
        const long long row = static_cast<long long>(s.row0) + first + tok;
        if (chunk == 0) lse = a.lse[static_cast<long long>(hq) * a.cb.rows + row];
        const uint4 u4 = *reinterpret_cast<const uint4*>(a.o + row * a.st[3][0] + hq * a.st[3][1] + chunk * 8);
        const uint4 v4 = *reinterpret_cast<const uint4*>(a.dout + row * a.st[4][0] + hq * a.st[4][1] + chunk * 8);
        const uint32_t uv[4] = {u4.x, u4.y, u4.z, u4.w}, vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&uv[e]));
          const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&vv[e]));
          acc = fmaf(u.x, v.x, acc);
          acc = fmaf(u.y, v.y, acc);
        }
      }
#pragma unroll
      for (int m = CPR / 2; m >= 1; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
      if (chunk == 0) {
        const long long at = (head * p.tiles + static_cast<int>(tile0) + tile) * BS + r;
        p.ws.dsum[at] = valid ? -acc : 0.f;
        p.ws.l2[at] = valid ? -lse * 1.4426950408889634f : -INFINITY;
      }
    }
    if (++head < a.heads) continue;
    head = 0;
    if (++tile < tiles) continue;
    tile = 0;
    before = add(before, tiles);
    if (left == 1) break;
    do {
      ++b;
      load();
    } while (tiles == 0);
  }
  if (zeros) {
    BwdZeros<D> z(a, blockIdx.x, gridDim.x, warp, WARPS, 1);
    while (z.row(p)) {
    }
  }
}

// ------------------------------------------------------------------ joining
// Joins the parts of the units that several CTAs held; blocks (c, .) those of the unit that CTA c began.  A warp takes 16
// columns of 32 rows, a row a lane (a part holds blocks of 4 columns of 128 rows: MODE 0: dK, then dV; MODE 2: tile by tile).
template <int D, int MODE>
__device__ __forceinline__ void cross_bwd_join(const CrossBwdParams& p) {
  using C = BwdWork<D, MODE>;
  const CrossArgs& a = p.a;
  const PlanRecord rec = p.ws.rec[bwd_place(MODE)][blockIdx.x];
  if (rec.b < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad;
  const CrossSeq s = cross_seq(a.cb, rec.b, bad);
  const BwdUnits u = bwd_units<D, MODE>(a, s);
  const int tile0 = rec.qb % u.fix;
  constexpr size_t stride = 2 * C::PART;  // from one CTA's parts to the next's
  const float* first = p.ws.part[bwd_place(MODE)] + blockIdx.x * stride + stride / 2;
  const float* rest = first + stride / 2 - stride;  // part 0 of CTA + i at rest + i * stride
  const int n = rec.more + 1;
  constexpr bool BY_KEY = bwd_by_key(MODE);
  constexpr int BLOCKS = static_cast<int>(C::PART / (128 * D));  // dK and dV, one of them, dQ, or dQ's tiles
  constexpr int COLS = BLOCKS * D / 16;
  for (int job = blockIdx.y * 4 + warp; job < 4 * COLS; job += gridDim.y * 4) {
    const int r = job % 4 * 32 + lane, c16 = job / 4;
    const int block = c16 * 16 / D, c = c16 * 16 % D;
    const int tile = MODE == 2 ? block : tile0;
    const int tok = BY_KEY ? r : r / a.group;
    const int left = BY_KEY ? s.len - tile * 128 : s.n - tile * bwd_tokens1(a.group);
    if (tok >= left || (!BY_KEY && tok >= bwd_tokens1(a.group))) continue;
    float4 acc[4] = {};
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      if (MODE == 2 && i > 0 && p.ws.part0[blockIdx.x + i] == 0) continue;  // no tile began in that CTA's share
      const float4* x = reinterpret_cast<const float4*>(i == 0 ? first : rest + i * stride) + r;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 y = x[(c16 * 4 + k) * 128];
        acc[k].x += y.x;
        acc[k].y += y.y;
        acc[k].z += y.z;
        acc[k].w += y.w;
      }
    }
    const bool is_dv = MODE == 3 || (MODE == 0 && block == 1);
    const float f = is_dv ? 1.f : a.scale;
    const int head = BY_KEY ? rec.head : rec.head * a.group + r % a.group;
    const long long row = BY_KEY ? static_cast<long long>(s.key0) + tile * 128 + r
                                    : static_cast<long long>(s.row0) + tile * bwd_tokens1(a.group) + tok;
    const long long* os = a.st[!BY_KEY ? 5 : is_dv ? 7 : 6];
    uint4* dst = reinterpret_cast<uint4*>((!BY_KEY ? a.dq : is_dv ? a.dv : a.dk) + row * os[0] + head * os[1] + c);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      dst[k] = make_uint4(pack_bf16x2(acc[2 * k].x * f, acc[2 * k].y * f), pack_bf16x2(acc[2 * k].z * f, acc[2 * k].w * f),
                          pack_bf16x2(acc[2 * k + 1].x * f, acc[2 * k + 1].y * f),
                          pack_bf16x2(acc[2 * k + 1].z * f, acc[2 * k + 1].w * f));
  }
}

// The parts of the kernels, one to blockIdx.z (the first may be the only one).
template <int D>
__global__ void __launch_bounds__(128) fa_cross_bwd_join_kernel(const __grid_constant__ CrossBwdParams p) {
  pdl_wait();
  if (blockIdx.z == 0)
    cross_bwd_join<D, D == 256 ? 3 : 2>(p);
  else if (blockIdx.z == 1)
    cross_bwd_join<D, D == 256 ? 4 : 0>(p);
  else
    cross_bwd_join<D, 1>(p);
}

// ------------------------------------------------------------------ launch
template <int D, int MODE>
int launch_cross_bwd_mode(const CrossBwdParams& p, int grid, const LaunchCtx& ctx) {
  using C = CrossBwdCfg<D, MODE>;
  auto kernel = fa_cross_bwd_kernel<D, MODE>;
  static std::atomic<unsigned long long> allowed{0};
  const int e = allow_smem(kernel, C::SMEM_ALLOC, allowed);
  if (e != 0) return e;
  const CrossArgs& a = p.a;
  CUtensorMap mq, mo, mk, mv;
  // Boxes of a group's heads of some tokens, and of one head of some keys.
  const int tokens = C::BY_KEY ? bwd_tokens0<D>(a.group) : bwd_tokens1(a.group), keys = C::BY_KEY ? 128 : C::BS;
  const long long qd[3] = {D, a.q_heads, a.cb.rows}, kd[3] = {D, a.heads, a.cb.keys};
  auto encode = [&](CUtensorMap* m, const void* t, int i, const long long* dims, int box1, int box2) {
    const long long st[2] = {a.st[i][1], a.st[i][0]};
    return encode_paged_map(m, t, 2, dims, st, C::RC, box1, box2, C::SWB, false);
  };
  if (encode(&mq, a.q, 0, qd, a.group, tokens) != 0 || encode(&mo, a.dout, 4, qd, a.group, tokens) != 0 ||
      encode(&mk, a.k, 1, kd, 1, keys) != 0 || encode(&mv, a.v, 2, kd, 1, keys) != 0)
    return -1;
  return C::BY_KEY ? launch_dependent(kernel, dim3(grid), C::THREADS, C::SMEM_ALLOC, ctx.stream, mk, mv, mq, mo, p)
                   : launch_dependent(kernel, dim3(grid), C::THREADS, C::SMEM_ALLOC, ctx.stream, mq, mo, mk, mv, p);
}

}  // namespace fa
