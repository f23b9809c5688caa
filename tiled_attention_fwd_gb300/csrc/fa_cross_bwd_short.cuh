// Gradients of cross attention for sequences of few rows (all heads of a group
// within 512, 256 or 128 rows at d = 32, 64, 128): dQ, dK and dV in one pass
// over the keys, and the launch of the whole backward pass.
//
// A unit is one key/value head of a sequence: its Q and dO stay in shared memory,
// tiles of 128 keys of K and V stream past, and each tile's dK and dV are finished
// with it, for all rows that add to them are there.  Five products a tile, where
// the two kernels for longer sequences (fa_cross_bwd.cuh) need seven, and every
// tensor is read or written once.  An item is QT rows against 128 keys:
//   S^T = K Q^T, dP^T = V dO^T          128 lanes = keys, QT columns = rows, double-buffered in tensor memory
//   P^T, dS^T in bf16 over them         two warpgroups take turns
//   dV += P^T dO, dK += dS^T Q          A from tensor memory; read out and stored by a third warpgroup, key tile by key tile
//   dQ += dS K                          A = dS^T, which the warpgroups also write to shared memory (M-major), over all key tiles;
//                                       issued by a warp of its own (d <= 64)
// Items run on across key tiles and units, two of them in flight; Q and dO come in 128-row
// tiles through a ring of their own, so that the next unit's are there when this one ends.
//
// Bound by an item's chain of products, elementwise step and products (some 4000 cycles, two in flight), not by memory or the tensor
// cores: 32 sequences of 17 to 200 rows over 100 to 1024 keys, 16 heads, d = 64: 100 us with the other kernels (180 MB: 0.26 of the
// memory's rate).  Other shapes of it that were measured there, whole calls: 128 rows an item, single-buffered, 16 elementwise warps 116; S and dV
// issued by one warp, dP and dK by another 132; both warpgroups on every item 116.
#pragma once

#include "fa_cross_bwd.cuh"

namespace fa {

template <int D>
struct ShortCfg {
  static constexpr int QT = BwdWork<D, 2>::QT;          // rows of an item
  static constexpr int EW_WARPS = 4;                    // of an item
  static constexpr int SUBS = 128 / QT;                 // items of a full row tile
  static constexpr int TILES = bwd_short_tiles(D);      // 128-row tiles of a unit at most
  static constexpr int SLOTS = D == 32 ? 6 : D == 64 ? 2 : 1;  // of the ring of Q and dO tiles
  static constexpr int SWB = (D * 2 >= 128) ? 128 : D * 2;  // swizzle span in bytes
  static constexpr uint32_t SWZ = (SWB == 128) ? 2u : 4u;   // descriptor swizzle code
  static constexpr int RC = SWB / 2;                    // bf16 columns per swizzle region
  static constexpr int NR = D / RC;
  static constexpr int REGION = 128 * SWB;
  static constexpr int TILE = 128 * D * 2;              // bytes of 128 rows or keys
  static constexpr int STAGE = 2 * TILE;                // K, V
  // Shared memory: [Q, dO tiles][K/V stages][dS^T: 2 regions of 64 rows, 128 keys][misc].
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_ST = SLOTS * 2 * TILE;
  static constexpr int DS_REGION = 128 * 128;
  static constexpr int DS = 2 * DS_REGION;
  static constexpr int VEC = 2 * 128 * 4;               // bytes of -L log2e and -D of a tile's rows
  // Output goes through shared memory, 32 rows of up to 64 columns a warp, so that a store is of whole rows (direct stores of a
  // thread's own row touch 32 lines each: 3700 cycles a key tile at d = 64); d = 128 has no room left.
  static constexpr bool STAGED = D <= 64;
  static constexpr int OUT_BUF = 32 * D * 2;
  static constexpr int OUT = STAGED ? 4 * OUT_BUF : 0;
  static constexpr int MISC = 1024 + SLOTS * VEC;
  static constexpr int SMEM_LIMIT = 227 * 1024;
  static constexpr int NST_FIT = (SMEM_LIMIT - 1024 - MISC - DS - OUT - OFF_ST) / STAGE;
  static constexpr int NST = NST_FIT > 4 ? 4 : NST_FIT;
  static constexpr int OFF_DS = OFF_ST + NST * STAGE;
  static constexpr int OFF_OUT = OFF_DS + DS;
  static constexpr int OFF_MISC = OFF_OUT + OUT;
  static constexpr int OFF_TMEM_SLOT = OFF_MISC + 384;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int OFF_SEG = OFF_MISC + 400;
  static constexpr int OFF_PLAN = OFF_SEG + kBwdSegRing * static_cast<int>(sizeof(BwdSeg));
  static constexpr int OFF_VEC = OFF_MISC + 1024;
  static constexpr int SMEM_USED = OFF_MISC + MISC + 1024;  // + slack for 1024-byte alignment
  static constexpr int SMEM_ALLOC = SMEM_USED < 120 * 1024 ? 120 * 1024 : SMEM_USED;
  // TMEM columns: S^T buffers, dP^T buffers, dK, dV, dQ's tiles.
  static constexpr int TM_S = 0;
  static constexpr int TM_DP = 2 * QT;
  static constexpr int TM_DK = 4 * QT;
  static constexpr int TM_DV = 4 * QT + D;
  static constexpr int TM_DQ = 4 * QT + 2 * D;
  static constexpr int TM_COLS = 512;
  // Warps: 0-7 elementwise, 8-11 output, 12 MMA of S and dP, 13 load, 14 MMA of dK and dV, 15 MMA of dQ.
  static constexpr int OUT_WARP0 = 8;
  static constexpr int S_WARP = 12;
  static constexpr int LOAD_WARP = 13;
  static constexpr int KV_WARP = 14;
  // (Only where a row tile has two items: the warp waits for each buffer once a row tile, and with four it could miss a phase.)
  static constexpr bool DQ_APART = SUBS == 2;
  static constexpr int DQ_WARP = 15;
  static constexpr int THREADS = DQ_APART ? 512 : 480;
  static constexpr int READERS = DQ_APART ? 15 : 14;
  static_assert(TM_DQ + TILES * D <= TM_COLS, "TMEM budget");
  static_assert(SLOTS >= TILES && NST >= 2 && SMEM_USED <= SMEM_LIMIT, "shared memory budget");
  static_assert(OFF_PLAN % 8 == 0 && OFF_PLAN + sizeof(PlanScratch) <= OFF_VEC, "misc area");
};

template <int D>
struct ShortBars {
  using C = ShortCfg<D>;
  uint32_t b0;
  __device__ __forceinline__ uint32_t s_full(int b) const { return b0 + 8u * b; }         // S^T and dP^T of buffer b
  __device__ __forceinline__ uint32_t p_ready(int b) const { return b0 + 16 + 8u * b; }   // P^T and dS^T (EW_WARPS)
  __device__ __forceinline__ uint32_t buf_free(int b) const { return b0 + 32 + 8u * b; }  // multiplied into dV and dK
  // dS^T in shared memory (its m-th row tile) has been read.  Two barriers take turns: where a row tile is one item, a warpgroup
  // may come to tile m + 2 before tile m has been read, and a barrier two phases behind looks as if it had.
  __device__ __forceinline__ uint32_t ds_empty(uint32_t m) const { return b0 + 48 + 8u * (m & 1); }
  __device__ __forceinline__ uint32_t kv_done() const { return b0 + 64; }   // dK and dV of a key tile
  __device__ __forceinline__ uint32_t kv_free() const { return b0 + 72; }   // read out (4 warps)
  __device__ __forceinline__ uint32_t dq_done() const { return b0 + 80; }
  __device__ __forceinline__ uint32_t dq_free() const { return b0 + 88; }
  __device__ __forceinline__ uint32_t drain(int i) const { return b0 + 96 + 8u * i; }  // of the issuing warps
  __device__ __forceinline__ uint32_t seg_full(int i) const { return b0 + 120 + 8u * i; }
  __device__ __forceinline__ uint32_t seg_empty(int i) const { return b0 + 152 + 8u * i; }
  __device__ __forceinline__ uint32_t st_full(int i) const { return b0 + 184 + 8u * i; }
  __device__ __forceinline__ uint32_t st_empty(int i) const { return b0 + 184 + 8u * (C::NST + i); }
  // A tile of Q and dO and its vectors (the copies, and the load warp's own stores) / used for the last time.
  __device__ __forceinline__ uint32_t q_full(int i) const { return b0 + 184 + 16u * C::NST + 8u * i; }
  __device__ __forceinline__ uint32_t q_empty(int i) const { return b0 + 184 + 16u * C::NST + 8u * (C::SLOTS + i); }
  static_assert(184 + 16 * (C::NST + C::SLOTS) <= 384 && kBwdSegRing == 4, "barrier area");
};

// Rows of tile i of a unit of n tokens.
__device__ __forceinline__ int short_rows(int n, int i, int t1, int group) { return min(n - i * t1, t1) * group; }

// A place in a ring of N: its index and the parity of its phase.
template <int N>
struct RingPos {
  uint32_t at = 0, par = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      par ^= 1;
    }
  }
};

// Walks the items of this CTA's segments: key tiles, within them the unit's items, SUBS to a row tile.
template <int D>
struct ShortItem {
  using C = ShortCfg<D>;
  int n;             // key tiles of the segment
  int items;         // items of a key tile
  int j, m;          // key tile, item of it
  RingPos<C::NST> st;        // the key tile's stage
  uint32_t slot0 = 0;        // row tiles of the segments before this one's, modulo SLOTS, and the parity of their phase
  uint32_t slot0_par = 0;
  // A segment has been read.
  __device__ __forceinline__ void enter(const BwdSeg& w, int t1, int group) {
    const int nt = (w.fix_n + t1 - 1) / t1;
    n = w.n;
    items = (nt - 1) * C::SUBS + (short_rows(w.fix_n, nt - 1, t1, group) + C::QT - 1) / C::QT;
    j = m = 0;
  }
  __device__ __forceinline__ int tile() const { return m / C::SUBS; }  // row tile of the unit
  __device__ __forceinline__ int sub() const { return m % C::SUBS; }
  __device__ __forceinline__ bool last_sub() const { return sub() == C::SUBS - 1 || m == items - 1; }
  __device__ __forceinline__ bool last() const { return m == items - 1; }
  __device__ __forceinline__ void slot(uint32_t& at, uint32_t& par) const {
    at = slot0 + tile();
    par = slot0_par;
    if (at >= C::SLOTS) {  // (a unit has SLOTS row tiles at most)
      at -= C::SLOTS;
      par ^= 1;
    }
  }
  // On to the next item; false where that is the next segment's first.
  __device__ __forceinline__ bool next() {
    if (++m < items) return true;
    m = 0;
    st.next();
    if (++j < n) return true;
    slot0 += (items + C::SUBS - 1) / C::SUBS;
    if (slot0 >= C::SLOTS) {
      slot0 -= C::SLOTS;
      slot0_par ^= 1;
    }
    return false;
  }
};

// ------------------------------------------------------------------ load warp
template <int D>
__device__ __forceinline__ void short_load(const CUtensorMap* tm_q, const CUtensorMap* tm_do, const CUtensorMap* tm_k,
                                           const CUtensorMap* tm_v, const CrossBwdParams& p, const ShortBars<D>& bar,
                                           uint32_t base, uint8_t* gbase, const PlanShare& share, const WaitGuard& g) {
  using C = ShortCfg<D>;
  const int lane = threadIdx.x & 31;
  const uint64_t policy = policy_evict_first();  // everything is read once
  const int group = p.a.group, t1 = bwd_tokens1(group), t0 = bwd_tokens0<D>(group);
  uint32_t pos = 0;       // stages issued so far
  uint32_t issued = 0;    // bit i: stage i has been loaded at least once
  uint32_t last_par = 0;  // bit i: parity of stage i's latest load
  uint32_t slots = 0;     // row tiles issued so far; and as for the stages:
  uint32_t q_issued = 0, q_par = 0;
  bool recorded = false, part0 = false, ok = true;
  CrossBwdWalk<D, 2> walk;
  walk.start(p, share);
  for (int k = 0;; ++k) {
    const int i = k % kBwdSegRing;
    if (!(ok = warp_wait_bar(bar.seg_empty(i), ((k / kBwdSegRing) & 1) ^ 1, g, kStatusTimeoutLoad))) break;
    const BwdSeg w = walk.next(p);
    if (lane == 0) {
      reinterpret_cast<BwdSeg*>(gbase + C::OFF_SEG)[i] = w;
      if (w.out == 2)  // this unit's first part: who holds the rest
        p.ws.rec[2][blockIdx.x] =
            PlanRecord{walk.record_b, w.head, walk.record_u,
                       plan_cta_of(walk.last_tile, share.total, share.ctas) - static_cast<int>(blockIdx.x)};
    }
    recorded = recorded || w.out == 2;
    part0 = part0 || w.out == 1;
    warp_arrive(bar.seg_full(i));
    if (!w.valid) break;
    auto load_kv = [&](int t) -> bool {
      const int st = pos % C::NST;
      const uint32_t par = (pos / C::NST) & 1;
      if (!warp_wait_bar(bar.st_empty(st), par ^ 1, g, kStatusTimeoutLoad)) return false;
      if (lane == 0) {
        const uint32_t s0 = base + C::OFF_ST + st * C::STAGE;
        const int row = w.str0 + (w.s0 + t) * 128;
        mbar_arrive_expect_tx(bar.st_full(st), C::STAGE);
        for (int r = 0; r < C::NR; ++r) {
          tma_load_3d(s0 + r * C::REGION, tm_k, bar.st_full(st), r * C::RC, w.head, row, policy);
          tma_load_3d(s0 + C::TILE + r * C::REGION, tm_v, bar.st_full(st), r * C::RC, w.head, row, policy);
        }
      }
      issued |= 1u << st;
      last_par = (last_par & ~(1u << st)) | (par << st);
      ++pos;
      return true;
    };
    auto load_q = [&](int x) -> bool {
      const int slot = slots % C::SLOTS;
      const uint32_t par = (slots / C::SLOTS) & 1;
      // The vectors are on their way while the slot may still be read.
      float l2[4], dsum[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = e * 32 + lane, tok = x * t1 + r / group, h = r % group;
        l2[e] = -INFINITY;
        dsum[e] = 0.f;
        if (r < t1 * group && tok < w.fix_n) {
          const long long at = (w.head * p.tiles + w.vec0 + tok / t0) * bwd_rows0<D>() + tok % t0 * group + h;
          l2[e] = __ldcg(p.ws.l2 + at);
          dsum[e] = __ldcg(p.ws.dsum + at);
        }
      }
      if (!warp_wait_bar(bar.q_empty(slot), par ^ 1, g, kStatusTimeoutLoad)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar.q_full(slot), 2 * C::NR * t1 * group * C::SWB);
        for (int r = 0; r < C::NR; ++r) {
          const uint32_t dst = base + C::OFF_Q + slot * 2 * C::TILE + r * C::REGION;
          tma_load_3d(dst, tm_q, bar.q_full(slot), r * C::RC, w.head * group, w.fix0 + x * t1, policy);
          tma_load_3d(dst + C::TILE, tm_do, bar.q_full(slot), r * C::RC, w.head * group, w.fix0 + x * t1, policy);
        }
      }
      float* vec = reinterpret_cast<float*>(gbase + C::OFF_VEC + slot * C::VEC);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        vec[e * 32 + lane] = l2[e];
        vec[128 + e * 32 + lane] = dsum[e];
      }
      warp_arrive(bar.q_full(slot));
      q_issued |= 1u << slot;
      q_par = (q_par & ~(1u << slot)) | (par << slot);
      ++slots;
      return true;
    };
    // The first K and V come before Q and dO, whose place is free later.
    const int nt = (w.fix_n + t1 - 1) / t1;
    ok = load_kv(0);
    for (int x = 0; ok && x < nt; ++x) ok = load_q(x);
    for (int t = 1; ok && t < w.n; ++t) ok = load_kv(t);
    if (!ok) break;
  }
  if (lane == 0 && !recorded) p.ws.rec[2][blockIdx.x].b = -1;
  if (lane == 0) p.ws.part0[blockIdx.x] = part0 ? 1 : 0;
  // Every issued copy must land before the CTA may exit.
  for (int i = 0; i < C::NST; ++i)
    if (issued & (1u << i)) bwd_wait_drain(bar.st_full(i), (last_par >> i) & 1, g);
  for (int i = 0; i < C::SLOTS; ++i)
    if (q_issued & (1u << i)) bwd_wait_drain(bar.q_full(i), (q_par >> i) & 1, g);
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issuer
template <int D>
struct ShortMma {
  using C = ShortCfg<D>;
  static constexpr uint32_t IDESC_S = make_idesc_bf16(128, C::QT, 0);  // S^T, dP^T: B K-major
  static constexpr uint32_t IDESC_O = make_idesc_bf16(128, D, 1);      // dV, dK: A in TMEM, B MN-major
  static constexpr uint32_t IDESC_Q = IDESC_O | (1u << 15);            // dQ: A M-major
  static constexpr uint32_t HI = sdesc_hi(8 * C::SWB, C::SWZ);
  static constexpr uint32_t HI_DS = sdesc_hi(8 * 128, 2);
  static constexpr __host__ __device__ uint32_t k_step(int kk) {
    return ((kk * 16 / C::RC) * C::REGION + (kk * 16 % C::RC) * 2) >> 4;
  }
  struct SSteps {
    static constexpr __host__ __device__ uint32_t da(int k) { return k_step(k) - k_step(k - 1); }
    static constexpr __host__ __device__ uint32_t db(int k) { return k_step(k) - k_step(k - 1); }
  };
  struct AccSteps {
    static constexpr __host__ __device__ uint32_t ta(int) { return 8; }  // 16 bf16 = 8 TMEM columns
    static constexpr __host__ __device__ uint32_t db(int) { return 16 * C::SWB >> 4; }
  };
  struct QSteps {
    static constexpr __host__ __device__ uint32_t da(int) { return 16 * 128 >> 4; }  // 16 keys of dS^T
    static constexpr __host__ __device__ uint32_t db(int) { return 16 * C::SWB >> 4; }
  };
  uint32_t tmem;
  uint32_t q_lo, q_mn;    // Q of slot 0 (dO lies a tile behind), K-major and MN-major
  uint32_t kv_lo, k_mn;   // K of stage 0 (V lies a tile behind)
  uint32_t ds_lo;
  __device__ __forceinline__ ShortMma(uint32_t tmem_, uint32_t base) : tmem(tmem_) {
    q_lo = sdesc_lo(base + C::OFF_Q, 16);
    q_mn = sdesc_lo(base + C::OFF_Q, C::REGION);
    kv_lo = sdesc_lo(base + C::OFF_ST, 16);
    k_mn = sdesc_lo(base + C::OFF_ST, C::REGION);
    ds_lo = sdesc_lo(base + C::OFF_DS, C::DS_REGION);
  }
  static constexpr uint32_t V = C::TILE >> 4;
  static __device__ __forceinline__ uint32_t q_off(uint32_t slot, int s) {
    return slot * (2 * C::TILE >> 4) + static_cast<uint32_t>(s) * (C::QT * C::SWB >> 4);
  }
  // S^T and dP^T of rows s QT .. of the tile in `slot` and the keys at stage st, into buffer b.
  __device__ __forceinline__ void sdp(uint32_t st, uint32_t slot, int s, uint32_t b) const {
    const uint32_t k = kv_lo + st * (C::STAGE >> 4), q = q_lo + q_off(slot, s);
    mma_ss_run<D / 16, SSteps>(tmem + C::TM_S + b * C::QT, k, HI, q, HI, IDESC_S, 0u);
    mma_ss_run<D / 16, SSteps>(tmem + C::TM_DP + b * C::QT, k + V, HI, q + V, HI, IDESC_S, 0u);
  }
  // dV (+)= P^T dO, dK (+)= dS^T Q.
  __device__ __forceinline__ void dkv(uint32_t slot, int s, uint32_t b, bool acc) const {
    const uint32_t q = q_mn + q_off(slot, s);
    const uint32_t f = acc ? 1u : 0u;
    constexpr int N = C::QT / 16;
    mma_ts_run<N, AccSteps>(tmem + C::TM_DV, tmem + C::TM_S + b * C::QT, q + V, HI, IDESC_O, f);
    mma_ts_run<N, AccSteps>(tmem + C::TM_DK, tmem + C::TM_DP + b * C::QT, q, HI, IDESC_O, f);
  }
  // dQ of row tile i (+)= dS K.
  __device__ __forceinline__ void dq(uint32_t st, int i, bool acc) const {
    mma_ss_run<8, QSteps>(tmem + C::TM_DQ + i * D, ds_lo, HI_DS, k_mn + st * (C::STAGE >> 4), HI, IDESC_Q, acc ? 1u : 0u);
  }
};

// Three warps issue the products (their instructions, about 10 for each small product, bound a single one: 32 sequences of 17 to 200 rows
// 138 us with one, 116 with dQ apart): S^T and dP^T; dV and dK (DQ_APART false: and dQ); dQ.  What one warp's products read and
// another's overwrite is handed over by a barrier (buf_free), for only those of one warp complete in order.
template <int D>
__device__ __forceinline__ void short_mma_s(const CrossBwdParams& p, const ShortBars<D>& bar, uint32_t base, uint8_t* gbase,
                                            uint32_t tmem, const WaitGuard& g) {
  using C = ShortCfg<D>;
  const ShortMma<D> M(tmem, base);
  const CrossIssuer<D> is{g};
  const int group = p.a.group, t1 = bwd_tokens1(group);
  ShortItem<D> it;
  int k = 0;
  bool begun = false, ok = true;
  for (uint32_t n = 0; ok; ++n) {
    if (!begun) {
      BwdSeg w;
      if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
      it.enter(w, t1, group);
    }
    uint32_t slot, par;
    it.slot(slot, par);
    if (it.m == 0 && !(ok = is.wait(bar.st_full(it.st.at), it.st.par))) break;
    if (it.j == 0 && it.sub() == 0 && !(ok = is.wait(bar.q_full(slot), par))) break;
    if (n >= 2 && !(ok = is.wait(bar.buf_free(n & 1), ((n >> 1) - 1) & 1))) break;
    tc_fence_after();
    M.sdp(it.st.at, slot, it.sub(), n & 1);
    mma_commit_elect(bar.s_full(n & 1));
    if (!(begun = it.next())) ++k;
  }
  is.finish(bar.drain(0));
}

template <int D>
__device__ __forceinline__ void short_mma_kv(const CrossBwdParams& p, const ShortBars<D>& bar, uint32_t base, uint8_t* gbase,
                                             uint32_t tmem, const WaitGuard& g) {
  using C = ShortCfg<D>;
  const ShortMma<D> M(tmem, base);
  const CrossIssuer<D> is{g};
  const int group = p.a.group, t1 = bwd_tokens1(group);
  ShortItem<D> it;
  int k = 0;
  uint32_t tiles = 0;  // key tiles whose dK and dV were begun
  uint32_t dqs = 0;    // row tiles of dS^T multiplied here
  bool begun = false, ok = true;
  for (uint32_t n = 0; ok; ++n) {
    if (!begun) {
      BwdSeg w;
      if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
      it.enter(w, t1, group);
    }
    uint32_t slot, par;
    it.slot(slot, par);
    const uint32_t b = n & 1;
    if (!(ok = is.wait(bar.p_ready(b), (n >> 1) & 1))) break;
    if (it.m == 0) {
      if (tiles > 0 && !(ok = is.wait(bar.kv_free(), (tiles - 1) & 1))) break;
      ++tiles;
    }
    tc_fence_after();
    M.dkv(slot, it.sub(), b, it.m > 0);
    mma_commit_elect(bar.buf_free(b));
    if (it.last()) mma_commit_elect(bar.kv_done());
    const bool end = it.last_sub() && it.j == it.n - 1;
    if (end) mma_commit_elect(bar.q_empty(slot));  // Q and dO of this row tile have been used for the last time
    if (!C::DQ_APART && it.last_sub()) {
      if (it.j == 0 && it.tile() == 0 && k > 0) {
        if (!(ok = is.wait(bar.dq_free(), (k - 1) & 1))) break;
        tc_fence_after();
      }
      M.dq(it.st.at, it.tile(), it.j > 0);
      mma_commit_elect(bar.ds_empty(dqs++));
      if (it.last()) {
        mma_commit_elect(bar.st_empty(it.st.at));
        if (end) mma_commit_elect(bar.dq_done());
      }
    }
    if (!(begun = it.next())) ++k;
  }
  is.finish(bar.drain(1));
}

// dQ, row tile by row tile.
template <int D>
__device__ __forceinline__ void short_mma_dq(const CrossBwdParams& p, const ShortBars<D>& bar, uint32_t base, uint8_t* gbase,
                                             uint32_t tmem, const WaitGuard& g) {
  using C = ShortCfg<D>;
  const ShortMma<D> M(tmem, base);
  const CrossIssuer<D> is{g};
  const int group = p.a.group, t1 = bwd_tokens1(group);
  ShortItem<D> it;
  int k = 0;
  uint32_t n = 0, dqs = 0;
  bool begun = false, ok = true;
  while (ok) {
    if (!begun) {
      BwdSeg w;
      if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
      it.enter(w, t1, group);
    }
    if (it.last_sub()) {
      // The row tile's last items are ready, one in each buffer (and so are those before them; none behind them is before this
      // tile has been multiplied, so the phases are these).
      if (it.sub() > 0 && !(ok = is.wait(bar.p_ready((n - 1) & 1), ((n - 1) >> 1) & 1))) break;
      if (!(ok = is.wait(bar.p_ready(n & 1), (n >> 1) & 1))) break;
      if (it.j == 0 && it.tile() == 0 && k > 0 && !(ok = is.wait(bar.dq_free(), (k - 1) & 1))) break;
      tc_fence_after();
      M.dq(it.st.at, it.tile(), it.j > 0);
      mma_commit_elect(bar.ds_empty(dqs++));
      if (it.last()) {
        mma_commit_elect(bar.st_empty(it.st.at));
        if (it.j == it.n - 1) mma_commit_elect(bar.dq_done());
      }
    }
    ++n;
    if (!(begun = it.next())) ++k;
  }
  is.finish(bar.drain(2));
}

// ------------------------------------------------------------------ elementwise warpgroups
// Thread = key.  What would meet a zero of P^T or dS^T in a product (Q and dO behind a tile's
// last row, K behind the last key: anything, and 0 times NaN is NaN) is set to zero in the first item that reads
// it, behind that item's S^T and dP^T, whose rows and columns there are not looked at.
template <int D>
__device__ __forceinline__ void short_elementwise(const CrossBwdParams& p, const ShortBars<D>& bar, uint32_t base, uint8_t* gbase,
                                                  uint32_t tmem, int wg, int quarter, int lane, const WaitGuard& g) {
  using C = ShortCfg<D>;
  constexpr int UNITS = D / 8;  // 16-byte units of a row
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint64_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
  const int group = p.a.group, t1 = bwd_tokens1(group);
  uint32_t dqs = 0;  // row tiles of dS^T before this item's
  auto zero_row = [&](uint32_t tile, int row) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) st_shared_v4(tile + u / (C::SWB / 16) * C::REGION + row * C::SWB + u % (C::SWB / 16) * 16, 0, 0, 0, 0);
  };
  ShortItem<D> it;
  BwdSeg w;
  int k = 0;
  bool begun = false, ok = true;
  for (uint32_t n = 0; ok; ++n) {
    if (!begun) {
      if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
      it.enter(w, t1, group);
    }
    const uint32_t b = n & 1;
    if (b == static_cast<uint32_t>(wg)) {
      uint32_t slot, par;
      it.slot(slot, par);
      const int rows = short_rows(w.fix_n, it.tile(), t1, group) - it.sub() * C::QT;  // of this item's QT on
      const int left = w.str_n - (w.s0 + it.j) * 128;
      const bool key = r < left;  // this thread's key is one
      if (!(ok = warp_wait_bar(bar.s_full(b), (n >> 1) & 1, g, kStatusTimeoutSoftmax))) break;
      // (Complete, for the MMA warp has waited for it: this makes the vectors visible here.)
      if (!(ok = warp_wait_bar(bar.q_full(slot), par, g, kStatusTimeoutSoftmax))) break;
      tc_fence_after();
      const bool need_mask = left < 128 || rows < C::QT;
      if (need_mask) {
        if (it.j == 0 && rows < C::QT) {  // first Q's, then dO's
          const uint32_t tile = base + C::OFF_Q + slot * 2 * C::TILE;
          for (int x = r; x < 2 * C::QT; x += 128) {
            const int row = x % C::QT;
            if (row >= rows) zero_row(tile + x / C::QT * C::TILE, it.sub() * C::QT + row);
          }
        }
        if (it.m == 0 && !key) zero_row(base + C::OFF_ST + it.st.at * C::STAGE, r);
        __syncwarp();
      }
      const float4* vl2 = reinterpret_cast<const float4*>(gbase + C::OFF_VEC + slot * C::VEC) + it.sub() * C::QT / 4;
      const float4* vd = vl2 + 32;
#pragma unroll 1
      for (int h = 0; h < C::QT / 32; ++h) {
        uint32_t rs[32], rd[32];
        tmem_ld32(tmem + lane_off + C::TM_S + b * C::QT + 32 * h, rs);
        tmem_ld32(tmem + lane_off + C::TM_DP + b * C::QT + 32 * h, rd);
        tmem_wait_ld(rs);
        tmem_wait_ld(rd);
        uint32_t pk[16], dk[16];
#pragma unroll
        for (int c4 = 0; c4 < 8; ++c4) {
          const float4 a = vl2[h * 8 + c4], d4 = vd[h * 8 + c4];
          const uint64_t nl[2] = {f2_pack(a.x, a.y), f2_pack(a.z, a.w)}, nd[2] = {f2_pack(d4.x, d4.y), f2_pack(d4.z, d4.w)};
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            const int c = c4 * 4 + e2 * 2;
            const float2 x = f2_unpack(f2_fma(f2_pack(__uint_as_float(rs[c]), __uint_as_float(rs[c + 1])), sl2x2, nl[e2]));
            const float p0 = ex2(x.x), p1 = ex2(x.y);
            const float2 ds = f2_unpack(
                f2_mul(f2_pack(p0, p1), f2_add(f2_pack(__uint_as_float(rd[c]), __uint_as_float(rd[c + 1])), nd[e2])));
            pk[c4 * 2 + e2] = pack_bf16x2(p0, p1);
            dk[c4 * 2 + e2] = pack_bf16x2(ds.x, ds.y);
          }
        }
        if (need_mask) {
          // (Bits, so that a NaN goes, too; outside the loop above, whose instructions are what an item costs.)
          const int v = rows - 32 * h;  // columns of this thread's that are rows
          const uint32_t keep = key ? 0xffffffffu : 0u;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint32_t m = v >= 2 * c + 2 ? keep : v == 2 * c + 1 ? keep & 0xffffu : 0u;
            pk[c] &= m;
            dk[c] &= m;
          }
        }
        // The bf16 pairs land over what this warpgroup has read.
        tmem_st16(tmem + lane_off + C::TM_S + b * C::QT + 16 * h, pk);
        tmem_st16(tmem + lane_off + C::TM_DP + b * C::QT + 16 * h, dk);
        // The row tile's dS^T before this one has been read.
        if (h == 0 && dqs > 0 && !(ok = warp_wait_bar(bar.ds_empty(dqs - 1), ((dqs - 1) >> 1) & 1, g, kStatusTimeoutSoftmax))) break;
        // dS^T into shared memory: key r's row of 64 rows of Q a region, 128-byte swizzled.
        const int q0 = it.sub() * C::QT + 32 * h;
        const uint32_t row = base + C::OFF_DS + (q0 >> 6) * C::DS_REGION + r * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          st_shared_v4(row + (((((q0 & 63) >> 3) + u) ^ (r & 7)) << 4), dk[4 * u], dk[4 * u + 1], dk[4 * u + 2], dk[4 * u + 3]);
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      fence_proxy_async_smem();
      warp_arrive(bar.p_ready(b));
    }
    if (it.last_sub()) ++dqs;
    if (!(begun = it.next())) ++k;
  }
}

// ------------------------------------------------------------------ output
template <int D>
__device__ __forceinline__ void short_output(const CrossBwdParams& p, const ShortBars<D>& bar, uint8_t* gbase, uint32_t tmem,
                                             int quarter, int lane, const WaitGuard& g) {
  using C = ShortCfg<D>;
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const int group = p.a.group, t1 = bwd_tokens1(group);
  const int tok_r = r / group, head_r = r - tok_r * group;
  uint32_t tiles = 0;  // key tiles read out
  bool ok = true;
  // The zeros of dK and dV, a few rows behind each key tile (32 padded sequences of 100 to 1024 places, with 2/4/8/12/16 of them or all
  // behind the first: 109/105/100/100/101/103 us; written by the kernel before, one share of a sequence a block: 106 and 101).
  BwdZeros<D> zeros(p.a, blockIdx.x, gridDim.x, quarter, 4, 8);
  bool more = true;
  // 32 columns of TMEM.
  auto chunk = [&](uint32_t at, uint32_t (&v)[32]) {
    tmem_ld32(tmem + lane_off + at, v);
    tmem_wait_ld(v);
  };
  // D columns of TMEM from `at` on, times f, as bf16.
  auto take = [&](uint32_t at, float f, uint32_t (&y)[D / 2]) {
    const uint64_t f2 = f2_pack(f, f);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t v[32];
      chunk(at + c * 32, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 x = f2_unpack(f2_mul(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2));
        y[c * 16 + i] = pack_bf16x2(x.x, x.y);
      }
    }
  };
  // The warp's 32 rows of D columns to where `to` says (each thread's own row's place; null: nowhere).
  const uint32_t buf = smem_u32(gbase + C::OFF_OUT) + static_cast<uint32_t>(quarter) * C::OUT_BUF;
  constexpr int UR = D / 8;                   // 16-byte units of a row
  constexpr int RPL = UR < 8 ? 8 / UR : 1;    // rows of a 128-byte line
  auto place = [&](int row, int u) -> uint32_t { return buf + row * (D * 2) + ((u ^ ((row / RPL) & (UR - 1))) << 4); };
  auto put = [&](const uint32_t (&y)[D / 2], __nv_bfloat16* to) {
    if constexpr (C::STAGED) {
      __syncwarp();  // the rows before these have been read
#pragma unroll
      for (int u = 0; u < UR; ++u) st_shared_v4(place(lane, u), y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
      __syncwarp();
      const unsigned long long mine = reinterpret_cast<unsigned long long>(to);
#pragma unroll 2
      for (int i = 0; i < UR; ++i) {  // 32 / UR rows at a time
        const int row = i * (32 / UR) + lane / UR, u = lane % UR;
        const unsigned long long there = __shfl_sync(0xffffffffu, mine, row);
        uint32_t x0, x1, x2, x3;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                     : "r"(place(row, u)));
        if (there) reinterpret_cast<uint4*>(there)[u] = make_uint4(x0, x1, x2, x3);
      }
    } else {
      if (to) {
#pragma unroll
        for (int u = 0; u < UR; ++u) reinterpret_cast<uint4*>(to)[u] = make_uint4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
      }
    }
  };
  for (int k = 0; ok; ++k) {
    BwdSeg w;
    if (!(ok = bwd_seg_read(w, k, gbase + C::OFF_SEG, bar, g)) || !w.valid) break;
    for (int j = 0; j < w.n; ++j) {
      if (!(ok = warp_wait_bar(bar.kv_done(), tiles & 1, g, kStatusTimeoutSoftmax))) break;
      ++tiles;
      tc_fence_after();
      const int at = (w.s0 + j) * 128 + r;
      const bool mine = at < w.str_n;
      const long long row = static_cast<long long>(w.str0) + at;
      __nv_bfloat16* dk = p.a.dk + row * p.a.st[6][0] + w.head * p.a.st[6][1];
      __nv_bfloat16* dv = p.a.dv + row * p.a.st[7][0] + w.head * p.a.st[7][1];
      // (d = 32: both are read out before they are stored, for the next tile's products wait for that.)
      constexpr bool BOTH = D <= 32;
      uint32_t yk[D / 2], yv[D / 2];
      take(C::TM_DK, p.a.scale, yk);
      if constexpr (!BOTH) put(yk, mine ? dk : nullptr);
      take(C::TM_DV, 1.f, yv);
      tc_fence_before();
      warp_arrive(bar.kv_free());
      if constexpr (BOTH) put(yk, mine ? dk : nullptr);
      put(yv, mine ? dv : nullptr);
      for (int i = 0; i < 8 && more; ++i) more = zeros.row(p);
    }
    if (!ok || !(ok = warp_wait_bar(bar.dq_done(), k & 1, g, kStatusTimeoutSoftmax))) break;
    tc_fence_after();
    const int nt = (w.fix_n + t1 - 1) / t1;
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      const int tok = i * t1 + tok_r;
      if (w.out == 0) {
        const bool mine = tok_r < t1 && tok < w.fix_n;
        __nv_bfloat16* dq = p.a.dq + (static_cast<long long>(w.fix0) + tok) * p.a.st[5][0] +
                            static_cast<long long>(w.head * group + head_r) * p.a.st[5][1];
        uint32_t y[D / 2];
        take(C::TM_DQ + i * D, p.a.scale, y);
        put(y, mine ? dq : nullptr);
        continue;
      }
      // 16-byte block b of all 128 rows of the tile together.
      float4* part = reinterpret_cast<float4*>(p.ws.part[2] + (blockIdx.x * 2 + (w.out - 1)) * BwdWork<D, 2>::PART) + r;
#pragma unroll 1
      for (int c = i * (D / 32); c < (i + 1) * (D / 32); ++c) {
        uint32_t v[32];
        chunk(C::TM_DQ + c * 32, v);
#pragma unroll
        for (int b = 0; b < 8; ++b)
          part[(c * 8 + b) * 128] = make_float4(__uint_as_float(v[4 * b]), __uint_as_float(v[4 * b + 1]),
                                                __uint_as_float(v[4 * b + 2]), __uint_as_float(v[4 * b + 3]));
      }
    }
    tc_fence_before();
    warp_arrive(bar.dq_free());
  }
  while (more) more = zeros.row(p);
}

// ------------------------------------------------------------------ kernel
template <int D>
__global__ void __launch_bounds__(ShortCfg<D>::THREADS, 1)
    fa_cross_bwd_short_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                              const __grid_constant__ CrossBwdParams p) {
  using C = ShortCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const ShortBars<D> bar{base + C::OFF_MISC};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_TMEM_SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_ABORT);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.s_full(i), 1);
      mbar_init(bar.p_ready(i), C::EW_WARPS);
      mbar_init(bar.buf_free(i), 1);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(bar.q_full(i), 2);
      mbar_init(bar.q_empty(i), 1);
    }
    mbar_init(bar.ds_empty(0), 1);
    mbar_init(bar.ds_empty(1), 1);
    mbar_init(bar.kv_done(), 1);
    mbar_init(bar.kv_free(), 4);
    mbar_init(bar.dq_done(), 1);
    mbar_init(bar.dq_free(), 4);
    for (int i = 0; i < 3; ++i) mbar_init(bar.drain(i), 1);
    for (int i = 0; i < kBwdSegRing; ++i) {
      mbar_init(bar.seg_full(i), 1);
      mbar_init(bar.seg_empty(i), C::READERS);
    }
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(bar.st_full(i), 1);
      mbar_init(bar.st_empty(i), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::LOAD_WARP && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_do);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == C::S_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TM_COLS);
    tmem_relinquish();
  }
  const PlanShare share = plan_share<C::THREADS>(
      p.a.cb.B, gridDim.x, blockIdx.x,
      [&](int b) -> long long {
        bool bad;
        const BwdUnits u = bwd_units<D, 2>(p.a, cross_seq(p.a.cb, b, bad));
        return u.units == 0 ? 0ll : static_cast<long long>(u.units) * u.template length<BwdWork<D, 2>::UNIT_COST>();
      },
      1 + BwdWork<D, 2>::UNIT_COST, *reinterpret_cast<PlanScratch*>(gbase + C::OFF_PLAN));
  pdl_wait();  // for the preparing kernel; and so have all CTAs when the next kernel's begin
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitGuard g{abort_flag, p.a.status, p.limit_ns};

  if (warp < C::OUT_WARP0) {
    short_elementwise<D>(p, bar, base, gbase, tmem, warp >> 2, warp & 3, lane, g);
  } else if (warp < C::S_WARP) {
    short_output<D>(p, bar, gbase, tmem, warp & 3, lane, g);
  } else if (warp == C::S_WARP) {
    short_mma_s<D>(p, bar, base, gbase, tmem, g);
  } else if (warp == C::KV_WARP) {
    short_mma_kv<D>(p, bar, base, gbase, tmem, g);
  } else if (warp == C::DQ_WARP) {
    if constexpr (C::DQ_APART) short_mma_dq<D>(p, bar, base, gbase, tmem, g);
  } else {
    short_load<D>(&tm_q, &tm_do, &tm_k, &tm_v, p, bar, base, gbase, share, g);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::S_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// ------------------------------------------------------------------ launch
template <int D>
int launch_cross_bwd_short(const CrossBwdParams& p, int grid, const LaunchCtx& ctx) {
  using C = ShortCfg<D>;
  auto kernel = fa_cross_bwd_short_kernel<D>;
  static std::atomic<unsigned long long> allowed{0};
  const int e = allow_smem(kernel, C::SMEM_ALLOC, allowed);
  if (e != 0) return e;
  const CrossArgs& a = p.a;
  CUtensorMap mq, mo, mk, mv;
  const long long qd[3] = {D, a.q_heads, a.cb.rows}, kd[3] = {D, a.heads, a.cb.keys};
  auto encode = [&](CUtensorMap* m, const void* t, int i, const long long* dims, int box1, int box2) {
    const long long st[2] = {a.st[i][1], a.st[i][0]};
    return encode_paged_map(m, t, 2, dims, st, C::RC, box1, box2, C::SWB, false);
  };
  if (encode(&mq, a.q, 0, qd, a.group, bwd_tokens1(a.group)) != 0 || encode(&mo, a.dout, 4, qd, a.group, bwd_tokens1(a.group)) != 0 ||
      encode(&mk, a.k, 1, kd, 1, 128) != 0 || encode(&mv, a.v, 2, kd, 1, 128) != 0)
    return -1;
  return launch_dependent(kernel, dim3(grid), C::THREADS, C::SMEM_ALLOC, ctx.stream, mq, mo, mk, mv, p);
}

// The preparing kernel, the kernel for few rows, the two for more (where there may be such sequences), and the joining of parts.
template <int D>
int launch_cross_bwd(const CrossArgs& a, const LaunchCtx& ctx) {
  CrossBwdParams p;
  p.a = a;
  cross_bwd_ws<D>(a.workspace, a.cb.B, a.cb.rows, a.heads, a.group, &p.ws);
  p.limit_ns = ctx.limit_ns;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.tiles = bwd_tiles<D>(a.cb.rows, a.cb.B, a.group);
  const bool products = a.cb.rows > 0 && a.cb.keys > 0, zeros = D == 256 || !products;
  // Where nothing is to be cleared, a block for each tile that there may be: all blocks plan first, and more than are needed delay each
  // other (5 sequences of 5 to 64 rows, 8 heads, d = 64, in a graph: 18.6 us, with eight blocks an SM 21.4; d = 256 has eight: with
  // fewer 5 of 40 rows took 32.4 us instead of 32.9, but 6 of 100 to 700 rows 158 instead of 151).
  const int full = ctx.num_sms * 8;
  const int prep = !zeros && p.tiles * a.heads < full ? static_cast<int>(p.tiles * a.heads) : full;
  fa_cross_prep_kernel<D><<<prep, kPrepThreads, 0, ctx.stream>>>(p, zeros);
  int e = static_cast<int>(cudaGetLastError());
  if (e != 0 || !products) return e;  // (zeros are all there is)
  const int grid = ctx.num_sms < kPlanCtas ? ctx.num_sms : kPlanCtas;
  const bool longer = D == 256 || a.cb.rows > bwd_short_tiles(D) * bwd_tokens1(a.group);
  if constexpr (D == 256) {
    e = launch_cross_bwd_mode<D, 3>(p, grid, ctx);
    if (e == 0) e = launch_cross_bwd_mode<D, 4>(p, grid, ctx);
  } else {
    e = launch_cross_bwd_short<D>(p, grid, ctx);
    if (e == 0 && longer) e = launch_cross_bwd_mode<D, 0>(p, grid, ctx);
  }
  if (e == 0 && longer) e = launch_cross_bwd_mode<D, 1>(p, grid, ctx);
  if (e == 0) e = launch_dependent(fa_cross_bwd_join_kernel<D>, dim3(grid, 8, longer ? 3 : 1), 128, 0, ctx.stream, p);
  return e;
}

}  // namespace fa
