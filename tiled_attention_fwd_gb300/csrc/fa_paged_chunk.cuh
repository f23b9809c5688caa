// Attention of chunks and prompts over a paged cache: sequences with more rows
// than the few-row kernel takes.  The forward kernel's pipeline (fa_fwd_tc.cuh:
// TMA, tcgen05.mma, S / P and O in tensor memory, softmax and correction
// warpgroups, lazy row maximum) on work that is found on the device:
//
//  * Rows.  A 128-row tile holds 128 / G tokens (rounded down) of the G query
//    heads that share a key/value head, token by token, so a chunk of few
//    tokens fills tiles and K and V are read once for all G heads; Q comes in by one
//    3-D TMA box {columns, G heads, tokens}.  A query block is two tiles
//    (d = 256: one).
//  * Work.  The key tiles of all (sequence, query block, head) units form one
//    line, with room for UNIT_COST more behind each unit (what its beginning and end
//    cost), that is cut into equal shares (fa_paged_plan.cuh).  The load warp walks
//    this CTA's share and hands segments (a run of key tiles of one unit) to
//    the other warps through a ring in shared memory.
//  * Pages.  A key tile is loaded page by page (boxes of min(page, tile) rows);
//    only boxes that hold keys of the sequence are.  V rows behind the last token
//    are set to zero before the tensor core reads them: such slots hold anything,
//    and 0 times NaN is NaN.
//  * e4m3 pages.  The load warp brings codes and scales, the correction warps and
//    two more turn them (d >= 128: in place) into the bf16 tiles that the tensor
//    core reads (exact: a code has 4 significant bits and a scale is a power of
//    two), so the rest of the pipeline is the same.
//  * Output.  A unit held whole is written as it is finished; of others O and
//    the log-sum (base 2) go to the workspace in fp32 and the joining kernel
//    adds them up: O = sum 2^(L_i - L) O_i, L = log2 sum 2^L_i.
//
// Bound by the tensor cores and the softmax as the contiguous forward is (1.55 us a step of 256 rows and 128 keys at
// d = 128), at short lengths by the units' borders (about 2.5 us each), with e4m3 pages by a stage's way through loading,
// converting and multiplying (2.7 us a step, 5 us or more a border).  Measured at d = 128: chunks of 541 to 2048 tokens
// over 7 to 16 K, bf16, 474 GFLOP: 349 us, 1.36 PFLOP/s (340 to 360 with the card's power); 65 to 1024 tokens over 1.7 to 8 K, e4m3, 210 GFLOP: 297 us;
// prompts of 1.7 to 4 K tokens, 161 GFLOP: 180 us.  Of a call's time about 12 us are the joining kernel (40 MB of parts
// through L2) and 2 us the mending kernel's look at its flags.
#pragma once

#include <type_traits>

#include "fa_fwd_tc.cuh"
#include "fa_paged_plan.cuh"

namespace fa {

constexpr int kSegRing = 4;

// warp_wait_bar in less code: the kernel has to stay within the SM's instruction cache (about 128 KB; at 150 KB a
// unit's epilogue, fetched anew each time, took 7000 cycles).
__device__ __forceinline__ bool chunk_wait(uint32_t bar, uint32_t parity, const WaitGuard& g, int code) {
  uint64_t t0 = 0;
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *g.abort)) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (__any_sync(0xffffffffu, now - t0 > g.limit_ns)) {
      *g.abort = 1;
      if ((threadIdx.x & 31) == 0) atomicOr(g.status, code);
      return false;
    }
  }
}

// mbar_try_wait that comes back after about `ns` at the latest.
__device__ __forceinline__ uint32_t mbar_try_wait_ns(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2, %3;\n\t"
      "selp.b32 %0, 1, 0, P1;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(ns)
      : "memory");
  return ok;
}

// A run of key tiles of one unit.
struct alignas(16) ChunkSeg {
  int valid;
  int b;
  int head;   // key/value head
  int row0;   // row of the block's first token
  int ntok;   // tokens of the block
  int pos0;   // position of its first token
  int len;    // tokens of the sequence
  int j0;     // first key tile
  int n0;     // key tiles of query tile 0 in this segment (they start at j0)
  int n1;     // of query tile 1
  int nmax;   // the larger
  int out;    // 0: the unit is whole; 1, 2: part 0, part 1 of this CTA
};
static_assert(sizeof(ChunkSeg) == 48, "segment size");

template <int D, bool E4M3>
struct ChunkCfg : TcCfg<D> {
  using T = TcCfg<D>;
  // Staged output: buffers of 32 rows x 32 columns per correction warp; e4m3 has one less, and scale bytes there.
  static constexpr int OUT_BUFS = E4M3 ? T::OSTB - 1 : T::OSTB;
  static constexpr int OFF_OUT = T::OFF_OST;
  static constexpr int OFF_SCALE = T::OFF_OST + 4 * OUT_BUFS * T::OST_BUF;  // [2][2][BK]
  // e4m3: where the codes of a stage's tiles are loaded to.  d >= 128: into the tile itself, its upper half: the codes
  // of a row (d bytes, in columns of 128) lie where the row's last bf16 columns go, so a warp that has read a row may
  // write it.  d <= 64: into two buffers of their own.
  static constexpr bool IN_PLACE = D >= 128;
  static constexpr int CODE_COLS = D < 128 ? D : 128;
  static constexpr int CODES = T::BK * D;  // bytes of a tile's codes
  static constexpr int OFF_CODES = T::OFF_OST + T::OST;  // [2][2][CODES]
  static constexpr int SMEM_E4M3 = OFF_CODES + (IN_PLACE ? 0 : 4 * CODES) + 1024;
  static constexpr int SMEM_CHUNK = E4M3 && SMEM_E4M3 > T::SMEM_ALLOC ? SMEM_E4M3 : T::SMEM_ALLOC;
  static_assert(SMEM_CHUNK <= T::SMEM_LIMIT && 4 * T::BK <= 4 * T::OST_BUF, "shared memory budget");
  static_assert(!IN_PLACE || T::NST == 2, "a stage and its codes have the same index");
  // Two tiles: the softmax warps rescale O themselves where a row's maximum moved far (rare, see LAZY_MAX), so the
  // correction warps are free for the output and, with e4m3 pages, for most of the conversion.
  static constexpr bool SELF_RESCALE = T::NQT == 2;
  static constexpr int OFF_SEG = T::OFF_MISC + 6672;
  static constexpr int OFF_PLAN = T::OFF_ALPHA;  // before the roles start
  static constexpr int CONV_WARPS = !E4M3 ? 0 : SELF_RESCALE ? 6 : 2;  // warps that convert e4m3 tiles
  static constexpr int CONV_WARP0 = T::LOAD_WARP + 1;                  // the last two; the others are the correction warps
  // d = 256, bf16: a second load warp issues the boxes of the tiles at position 1.  A warp needs about 130 cycles a box,
  // and tiles of 16-token pages have 32 of them (prompts on pages of 16: 368 us, with one load warp 496; of 64: 346 and
  // 351).  d = 128 has half as many boxes and loses more at the borders of units (180 and 180 us; pages of 64: 182 and 172).
  static constexpr int LOADERS = !E4M3 && D == 256 ? 2 : 1;
  static constexpr int SEG_READERS = T::SOFTMAX_WARPS + 4 + 1 + (E4M3 ? 2 : LOADERS - 1);
  static constexpr int ROWS = T::NQT * 128;
  // Key tiles that a unit costs besides its own (its beginning, its end, its output).  Measured on ragged batches, us with
  // 0/1/2/3: prompts, bf16, d = 128: 202/186/190/195; d = 256: 438/387/353/349; chunks, e4m3, with 2/4/5/7: d = 128:
  // 313/305/303/309, d = 64: 277/261/263/259, d = 256: 567/572/575/581.
  static constexpr int UNIT_COST = E4M3 ? (D == 256 ? 2 : 5) : (D == 256 ? 2 : 1);
  static_assert(T::OFF_ABORT + 4 <= OFF_SEG && OFF_SEG % 16 == 0, "misc area");
  static_assert(OFF_SEG + kSegRing * static_cast<int>(sizeof(ChunkSeg)) <= T::OFF_MISC + T::MISC, "misc area");
  static_assert(sizeof(PlanScratch) <= 2048, "plan scratch");
};

template <int D, bool E4M3>
struct ChunkBars : TcBars<D, TcCfg<D>::NQT, kVarBf16> {
  using Base = TcBars<D, TcCfg<D>::NQT, kVarBf16>;
  __device__ __forceinline__ uint32_t seg_full(int i) const { return this->b0 + 256 + 8u * i; }
  __device__ __forceinline__ uint32_t seg_empty(int i) const { return this->b0 + 288 + 8u * i; }
  // e4m3: the codes of a stage have landed / (d <= 64) have been read.
  __device__ __forceinline__ uint32_t code_full(int i) const { return this->b0 + 320 + 8u * i; }
  __device__ __forceinline__ uint32_t code_empty(int i) const { return this->b0 + 336 + 8u * i; }
  // m and l of this accumulator's k-th unit: the softmax may finish the next unit (one key tile) while the
  // correction warpgroup has not come to this one yet, so two barriers take turns.
  __device__ __forceinline__ uint32_t ml_full(int t, int k) const { return this->b0 + 448 + 8u * (2 * t + (k & 1)); }
  // Two tiles: O of tile t has been read out (there are no alphas to publish, so the barrier is free).
  __device__ __forceinline__ uint32_t o_free(int t) const { return this->a_full(t, 0); }
  static_assert(Base::COUNT * 8 <= 256, "barrier area");
};

struct ChunkParams {
  PagedFwdArgs a;
  PagedWs ws;
  int* status;
  unsigned long long limit_ns;
  float scale_log2;
  int tpt;      // tokens of a 128-row tile: 128 / group
  int box;      // rows of a K/V box, a power of two
  int box_log2;
  bool tma_o;   // a warp's 32 rows are a box of O (the group is a power of two)
};

// sum over i in [0, n) of floor((a i + b) / m), a, b >= 0, a n + b < 2^32: the lattice points under a line, counted by Euclid's
// algorithm (Graham, Knuth and Patashnik, Concrete Mathematics, 3.5, reduce such sums this way): whole parts of a / m and
// b / m are summed directly, then the axes change places.
__host__ __device__ inline long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long sum = 0;
  while (n > 0) {
    sum += static_cast<long long>(n) * (n - 1) / 2 * (a / m) + static_cast<long long>(n) * (b / m);
    a %= m;
    b %= m;
    const uint32_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// The query blocks of a sequence (TQ tokens each) and the key tiles they visit.
struct ChunkBlocks {
  int n, len, tq, bk;
  int unit;  // key tiles that a unit costs besides its own
  bool causal;
  __host__ __device__ __forceinline__ int count() const { return (n + tq - 1) / tq; }
  // Key tiles of the first `ntok` tokens of block q: those up to the last token's position (one at least).
  __host__ __device__ __forceinline__ int tiles(int q, int ntok) const {
    int end = len;
    if (causal) {
      const int pos = len - n + q * tq + ntok;
      end = pos < len ? pos : len;
    }
    return end <= bk ? 1 : (end + bk - 1) / bk;
  }
  __host__ __device__ __forceinline__ int tokens(int q) const { return n - q * tq < tq ? n - q * tq : tq; }
  // Length on the line of blocks 0 .. k - 1 of one head.
  __host__ __device__ __forceinline__ long long before(int k) const { return tiles_before(k) + static_cast<long long>(unit) * k; }
  // Their key tiles.
  __host__ __device__ __forceinline__ long long tiles_before(int k) const {
    if (k == 0) return 0;
    const long long last = tiles(k - 1, tokens(k - 1));
    if (!causal) return k * last;
    // Block i < k - 1 ends behind position x_i = len - n + (i + 1) tq < len; the first `one` of them have x_i <= 0.
    const int past = len - n;
    int one = past < 0 ? -past / tq : 0;
    one = one < k - 1 ? one : k - 1;
    // (Positions are below 2^31, so the sums of a block's end and bk are below 2^32.)
    return one + floor_sum(k - 1 - one, bk, tq, static_cast<uint32_t>(past + (one + 1) * tq + bk - 1)) + last;
  }
};

template <int D, bool E4M3>
__host__ __device__ __forceinline__ ChunkBlocks chunk_blocks(const ChunkParams& p, const PagedSeq& s) {
  ChunkBlocks c;
  const bool mine = s.n >= 1 && s.n <= p.a.max_rows && (s.n > kFewMost || s.n * p.a.group > p.a.few_rows);
  c.n = mine ? s.n : 0;
  c.len = s.len;
  c.tq = p.tpt * TcCfg<D>::NQT;
  c.bk = TcCfg<D>::BK;
  c.unit = ChunkCfg<D, E4M3>::UNIT_COST;
  c.causal = p.a.causal;
  return c;
}

// ------------------------------------------------------------------ segments
// The load warp's walk over its CTA's share.
template <int D, bool E4M3>
struct ChunkWalk {
  using C = ChunkCfg<D, E4M3>;
  int b, q, head, j, nt;
  PagedSeq s;
  ChunkBlocks c;
  long long pos, end;   // on the line
  long long last_tile;  // of the latest segment's unit
  int record_q;         // its query block
  __host__ __device__ __forceinline__ void load(const ChunkParams& p) {
    bool bad;
    s = paged_seq(p.a.pb, p.a.kv.ps_log2, b, bad);
    c = chunk_blocks<D, E4M3>(p, s);
  }
  // On to the next unit, if the share reaches it.
  __host__ __device__ __forceinline__ void advance(const ChunkParams& p) {
    pos += nt - j + C::UNIT_COST;
    j = 0;
    if (pos >= end) return;
    if (++head == p.a.kv.heads) {
      head = 0;
      ++q;
      while (q == c.count()) {
        ++b;
        q = 0;
        load(p);
      }
      nt = c.tiles(q, c.tokens(q));
    }
  }
  __host__ __device__ __forceinline__ ChunkSeg next(const ChunkParams& p) {
    ChunkSeg g = {};
    if (pos >= end) return g;
    const int ntok = c.tokens(q);
    const int n = end - pos < nt - j ? static_cast<int>(end - pos) : nt - j;
    g.valid = 1;
    g.b = b;
    g.head = head;
    g.row0 = s.row0 + q * c.tq;
    g.ntok = ntok;
    g.pos0 = s.len - s.n + q * c.tq;
    g.len = s.len;
    g.j0 = j;
    g.nmax = n;
    g.n0 = n;
    if (ntok > p.tpt) {
      // Tile 0's tokens come first: they may be done with their keys before tile 1's.
      const int first = c.tiles(q, p.tpt) - j;
      g.n0 = first < 0 ? 0 : first < n ? first : n;
      g.n1 = n;
    }
    g.out = n == nt ? 0 : j == 0 ? 2 : 1;
    last_tile = pos + (nt - 1 - j);
    record_q = q;
    pos += n;
    j += n;
    if (j == nt) advance(p);
    return g;
  }
};

template <int D, bool E4M3>
__device__ __forceinline__ ChunkSeg* seg_slot(uint8_t* gbase, int k) {
  return reinterpret_cast<ChunkSeg*>(gbase + ChunkCfg<D, E4M3>::OFF_SEG) + (k % kSegRing);
}

// Segment k, read by a whole warp of a role other than the load warp.
// (INLINE: the softmax warps' registers are full, and a call would spill them.)
template <int D, bool E4M3, bool INLINE = false>
__device__ __forceinline__ bool seg_read(ChunkSeg& g, int k, uint8_t* gbase, const ChunkBars<D, E4M3>& bar,
                                         const WaitGuard& guard) {
  const uint32_t full = bar.seg_full(k % kSegRing), par = (k / kSegRing) & 1;
  if (!(INLINE ? warp_wait_bar(full, par, guard, kStatusTimeoutLoad) : chunk_wait(full, par, guard, kStatusTimeoutLoad)))
    return false;
  const int4* src = reinterpret_cast<const int4*>(seg_slot<D, E4M3>(gbase, k));
  int4* dst = reinterpret_cast<int4*>(&g);
#pragma unroll
  for (int i = 0; i < 3; ++i) dst[i] = src[i];
  warp_arrive(bar.seg_empty(k % kSegRing));
  return true;
}

// A K or V tile of the stream.
struct ChunkTile {
  int kind;  // 0: none, 1: K, 2: V
  int b, head, key0, len;
};
template <int D>
__device__ __forceinline__ ChunkTile chunk_tile(int kind, const ChunkSeg& g, int j) {
  return ChunkTile{kind, g.b, g.head, (g.j0 + j) * TcCfg<D>::BK, g.len};
}

// The order in which stages are filled and read (see tc_producer): get(k, seg)
// fetches segment k, unit(seg, k) is called where segment k's Q may be loaded,
// stage(t0, t1) for every stage with the tiles at its positions 0 and 1.
template <int D, class Get, class Unit, class Stage>
__device__ __forceinline__ bool chunk_stream(const Get& get, const Unit& unit, const Stage& stage) {
  using C = TcCfg<D>;
  const ChunkTile none{0, 0, 0, 0, 0};
  ChunkSeg w;
  if (!get(0, w)) return false;
#pragma unroll 1
  for (int k = 0; w.valid; ++k) {
    ChunkSeg wn;
    if (C::NQT == 2 && !get(k + 1, wn)) return false;
    if (!unit(w, k)) return false;
    // Two tiles: the first stage of all holds K_0 alone; one tile: every unit begins with K_0 and K_1.
#pragma unroll 1
    for (int j = C::NQT == 1 || k == 0 ? -1 : 0; j < w.nmax; ++j) {
      ChunkTile t1 = none;
      if constexpr (C::NQT == 2) {
        if (j >= 0 && j + 1 < w.nmax)
          t1 = chunk_tile<D>(1, w, j + 1);
        else if (j >= 0 && wn.valid)
          t1 = chunk_tile<D>(1, wn, 0);
      } else {
        const int next = j < 0 ? 1 : j + C::LA;
        if (next < w.nmax) t1 = chunk_tile<D>(1, w, next);
      }
      if (!stage(j < 0 ? chunk_tile<D>(1, w, 0) : chunk_tile<D>(2, w, j), t1)) return false;
    }
    if (C::NQT == 1 && !get(k + 1, wn)) return false;
    w = wn;
  }
  return true;
}

// Offset of the codes of the tile at position i of stage st (buffer cb).
template <int D>
__device__ __forceinline__ uint32_t chunk_codes(int st, int cb, int i) {
  using C = ChunkCfg<D, true>;
  return C::IN_PLACE ? C::OFF_KV + st * C::STAGE + i * C::KV_TILE + C::KV_TILE / 2 : C::OFF_CODES + (cb * 2 + i) * C::CODES;
}

// ------------------------------------------------------------------ load warp
// What a load warp has issued.
struct ChunkLoaded {
  uint32_t issued;    // bit i: stage (e4m3: codes) i has been loaded
  uint32_t last_par;  // bit i: parity of its latest load
};

// Every issued copy must land before the CTA may exit.
template <int D, bool E4M3>
__device__ __forceinline__ void chunk_drain(const ChunkBars<D, E4M3>& bar, const ChunkLoaded& done, const WaitGuard& g) {
  for (int i = 0; i < (E4M3 ? 2 : TcCfg<D>::NST); ++i)
    if (done.issued & (1u << i)) wait_bar_drain(E4M3 ? bar.code_full(i) : bar.kv_full(i), (done.last_par >> i) & 1, g);
}

// Loads the tiles of the pos-th stage: t0 where bit 0 of `which` is set, t1 where bit 1 is.
template <int D, bool E4M3>
__device__ __forceinline__ bool chunk_load_stage(const CUtensorMap* tm_k, const CUtensorMap* tm_v, const ChunkParams& p,
                                                 const ChunkBars<D, E4M3>& bar, uint32_t base, uint32_t pos, int which,
                                                 const ChunkTile& t0, const ChunkTile& t1, ChunkLoaded& done,
                                                 const WaitGuard& g) {
  using C = ChunkCfg<D, E4M3>;
  const int lane = threadIdx.x & 31;
  const uint64_t pol_kv = policy_evict_last();
  // Boxes of up to `rows` keys from key0 on, one lane each: those that begin before the sequence's end.
  auto boxes = [&](const ChunkTile& t, int key0, int rows) -> int {
    const int n = min(rows, t.len - key0);
    return n <= 0 ? 0 : (n + p.box - 1) >> p.box_log2;
  };
  auto page_of = [&](const ChunkTile& t, int key) -> int {
    const int page = paged_page(p.a.pb, p.a.kv, t.b, key);
    if (page < 0) atomicOr(p.status, kStatusBadBatch);
    return page < 0 ? p.a.kv.num_pages : page;  // a coordinate outside the tensor reads as zeros
  };
  const int slot_mask = (1 << p.a.kv.ps_log2) - 1;
  const int st = pos % C::NST, cb = pos & 1;
  const bool own = E4M3 && !C::IN_PLACE;  // codes have buffers of their own
  const uint32_t full = E4M3 ? bar.code_full(cb) : bar.kv_full(st);
  const int n0 = which & 1 ? boxes(t0, t0.key0, C::BK) : 0, n1 = (which & 2) && t1.kind ? boxes(t1, t1.key0, C::BK) : 0;
  // The pages are looked up while the stage is still being read.
  const int row = lane << p.box_log2;
  const int page0 = lane < n0 ? page_of(t0, t0.key0 + row) : 0;
  const int page1 = lane < n1 ? page_of(t1, t1.key0 + row) : 0;
  const uint32_t par = own ? (pos >> 1) & 1 : (pos / C::NST) & 1;
  if (!chunk_wait(own ? bar.code_empty(cb) : bar.kv_empty(st), par ^ 1, g, kStatusTimeoutLoad)) return false;
  if (lane == 0) mbar_arrive_expect_tx(full, ((n0 + n1) << p.box_log2) * (E4M3 ? D + 1 : D * 2));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const ChunkTile& t = i == 0 ? t0 : t1;
    if (lane < (i == 0 ? n0 : n1)) {
      const int key = t.key0 + row, page = i == 0 ? page0 : page1;
      const CUtensorMap* tm = t.kind == 1 ? tm_k : tm_v;
      if constexpr (!E4M3) {
        const uint32_t dst = base + C::OFF_KV + st * C::STAGE + i * C::KV_TILE + row * C::SWB;
        for (int r = 0; r < C::NR; ++r)
          tma_load_4d(dst + r * C::K_REGION, tm, full, r * C::RC, key & slot_mask, t.head, page, pol_kv);
      } else {
        const uint32_t dst = base + chunk_codes<D>(st, cb, i) + row * C::CODE_COLS;
        for (int r = 0; r < D / C::CODE_COLS; ++r)
          tma_load_4d(dst + r * C::BK * C::CODE_COLS, tm, full, r * C::CODE_COLS, key & slot_mask, t.head, page, pol_kv);
        // (For a page that is not there any scales do.)
        const long long pg = page == p.a.kv.num_pages ? 0 : page;
        bulk_load(base + C::OFF_SCALE + (cb * 2 + i) * C::BK + row,
                  (t.kind == 1 ? p.a.kv.k_scale : p.a.kv.v_scale) +
                      (((pg * p.a.kv.heads + t.head) << p.a.kv.ps_log2) + (key & slot_mask)),
                  p.box, full);
      }
    }
  }
  const int slot = E4M3 ? cb : st;
  const uint32_t load_par = E4M3 ? (pos >> 1) & 1 : par;
  done.issued |= 1u << slot;
  done.last_par = (done.last_par & ~(1u << slot)) | (load_par << slot);
  return true;
}

// The load warp, or the second one (bf16), which reads the segments that the first finds and loads the tiles at
// position 1.
template <int D, bool E4M3>
__device__ __forceinline__ void chunk_load(const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                           const ChunkParams& p, const ChunkBars<D, E4M3>& bar, uint32_t base,
                                           uint8_t* gbase, const PlanShare& share, bool second, const WaitGuard& g) {
  using C = ChunkCfg<D, E4M3>;
  const int lane = threadIdx.x & 31;
  const uint64_t pol_q = policy_evict_first();
  uint32_t pos = 0;          // stages filled so far
  ChunkLoaded done{0, 0};
  int last_q = -1;           // latest segment whose Q tiles were loaded
  bool recorded = false;

  ChunkWalk<D, E4M3> walk;
  walk.pos = share.start;
  walk.end = share.end;
  if (walk.pos < walk.end && !second) {
    walk.b = share.b;
    walk.load(p);
    // The block that holds the share's first place: 32 candidates at a time.
    for (int q0 = 0;; q0 += 32) {
      const int q = q0 + lane;
      bool here = false;
      long long first = 0;
      int nt = 0;
      if (q < walk.c.count()) {
        nt = walk.c.tiles(q, walk.c.tokens(q));
        first = p.a.kv.heads * walk.c.before(q);
        here = first <= share.offset && share.offset < first + static_cast<long long>(p.a.kv.heads) * (nt + C::UNIT_COST);
      }
      const uint32_t who = __ballot_sync(0xffffffffu, here);
      if (who != 0) {
        const int from = __ffs(who) - 1;
        walk.q = q0 + from;
        walk.nt = __shfl_sync(0xffffffffu, nt, from);
        const long long in = share.offset - __shfl_sync(0xffffffffu, first, from);
        walk.head = static_cast<int>(in / (walk.nt + C::UNIT_COST));
        walk.j = static_cast<int>(in - static_cast<long long>(walk.head) * (walk.nt + C::UNIT_COST));
        if (walk.j >= walk.nt) walk.advance(p);  // behind a unit's tiles: its first tile is the next unit's
        break;
      }
      if (q0 + 32 >= walk.c.count()) {  // cannot be: the share lies within the sequence's places
        walk.pos = walk.end;
        break;
      }
    }
  }

  auto get = [&](int k, ChunkSeg& w) -> bool {
    const int i = k % kSegRing;
    if (C::LOADERS == 2 && second) return seg_read<D, E4M3>(w, k, gbase, bar, g);
    if (!chunk_wait(bar.seg_empty(i), ((k / kSegRing) & 1) ^ 1, g, kStatusTimeoutLoad)) return false;
    w = walk.next(p);
    if (lane == 0) {
      *seg_slot<D, E4M3>(gbase, k) = w;
      if (w.out == 2) {  // this unit's first part: who holds the rest
        p.ws.chunk_rec[blockIdx.x] = PlanRecord{w.b, w.head, walk.record_q,
                                                plan_cta_of(walk.last_tile, share.total, share.ctas) - static_cast<int>(blockIdx.x)};
      }
    }
    recorded = recorded || w.out == 2;
    warp_arrive(bar.seg_full(i));
    return true;
  };
  auto unit = [&](const ChunkSeg& w, int k) -> bool {
    if (C::LOADERS == 2 && second) return true;
    for (int t = 0; t < C::NQT; ++t) {
      if (!chunk_wait(bar.q_empty(t), (k & 1) ^ 1, g, kStatusTimeoutLoad)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar.q_full(t), p.tpt * p.a.group * D * 2);
        for (int r = 0; r < C::NR; ++r)
          tma_load_3d(base + C::OFF_Q + t * C::Q_TILE + r * C::Q_REGION, tm_q, bar.q_full(t), r * C::RC,
                      w.head * p.a.group, w.row0 + t * p.tpt, pol_q);
      }
    }
    last_q = k;
    return true;
  };
  auto stage = [&](const ChunkTile& t0, const ChunkTile& t1) -> bool {
    if (!chunk_load_stage<D, E4M3>(tm_k, tm_v, p, bar, base, pos, C::LOADERS == 1 ? 3 : second ? 2 : 1, t0, t1, done, g)) return false;
    ++pos;
    return true;
  };
  chunk_stream<D>(get, unit, stage);
  if (lane == 0 && !recorded && !second) p.ws.chunk_rec[blockIdx.x].b = -1;
  chunk_drain<D, E4M3>(bar, done, g);
  for (int t = 0; t < C::NQT; ++t)
    if (last_q >= 0) wait_bar_drain(bar.q_full(t), last_q & 1, g);
  __syncwarp();
}

// ------------------------------------------------------------------ e4m3 -> bf16
// Eight codes (two words) to eight bf16, times the scale: the bits of a code are
// put where bf16 has them (sign; 4 exponent bits below bf16's 8; 3 mantissa
// bits), which is the value times 2^-120, also for denormals; one multiplication
// by 2^(120 + e) makes it right (two where that power is beyond bf16).  Only the
// NaN codes 0x7f and 0xff come out as +-480 and are set apart.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_bf16x4(uint32_t x, uint32_t f, uint32_t& lo, uint32_t& hi) {
  const uint32_t h = (x & 0x80808080u) | ((x >> 4) & 0x07070707u);  // high bytes: sign, upper 3 exponent bits
  const uint32_t l = (x << 4) & 0xf0f0f0f0u;                        // low bytes: lowest exponent bit, mantissa
  lo = mul_bf16x2(__byte_perm(l, h, 0x5140), f);
  hi = mul_bf16x2(__byte_perm(l, h, 0x7362), f);
}

// A top bit is set where a byte of x holds a NaN code: one more carries out of its seven ones (2 operations a word; they
// and the vote cost chunks of e4m3 pages 287 to 297 us, for conversion is short of integer operations).
__device__ __forceinline__ uint32_t e4m3x4_any_nan(uint32_t x) { return (x + 0x01010101u) ^ x; }
// The top bit of each byte that holds a NaN code (the others: anything).
__device__ __forceinline__ uint32_t e4m3x4_nan(uint32_t x) { return (x & 0x7f7f7f7fu) + 0x01010101u; }
// Bits of a bf16 NaN where bytes 0 and 1 (HIGH: 2 and 3) of `nan` have their top bit set.
template <bool HIGH>
__device__ __forceinline__ uint32_t nan_bf16x2(uint32_t nan) {
  uint32_t r;  // (a selector's bit 3: the byte's sign, eight times)
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(nan), "n"(HIGH ? 0xbbaa : 0x9988));
  return r & 0x7fff7fffu;
}

// Stage after stage, groups of 16 rows dealt out to WARPS warps, this one the cw-th.  wait(bar, parity) waits, get
// fetches segments.
template <int D, bool E4M3, class Get, class Wait>
__device__ __forceinline__ bool chunk_convert(const ChunkParams& p, const ChunkBars<D, E4M3>& bar, uint32_t base,
                                              uint8_t* gbase, int cw, const Get& get, const Wait& wait) {
  using C = ChunkCfg<D, E4M3>;
  constexpr int WARPS = C::CONV_WARPS;
  constexpr int UPR = D / 8;              // 16-byte units of a bf16 row
  constexpr int RPP = 32 / UPR;           // rows of a pass of the warp
  constexpr int PASSES = 16 / RPP;
  constexpr int BATCH = RPP * 4 >= 8 ? (PASSES < 4 ? PASSES : 4) : 8 / RPP;
  constexpr int UR = C::SWB / 16;
  static_assert(PASSES % BATCH == 0 && BATCH * RPP % 8 == 0, "a batch of passes is a whole number of swizzle periods");
  const int lane = threadIdx.x & 31;
  const int row0 = lane / UPR, unit16 = lane % UPR;
  // This thread's places within 8 / RPP passes of rows.
  uint32_t to[BATCH];
#pragma unroll
  for (int k = 0; k < BATCH; ++k) {
    const int r = k * RPP + row0;
    const uint32_t sw = C::SWB == 128 ? r & 7 : (r >> 1) & 3;
    to[k] = (unit16 / UR) * C::K_REGION + r * C::SWB + (((unit16 % UR) ^ sw) << 4);
  }
  const uint32_t from = unit16 / (C::CODE_COLS / 8) * (C::BK * C::CODE_COLS) + row0 * C::CODE_COLS +
                        unit16 % (C::CODE_COLS / 8) * 8;
  uint32_t pos = 0;
  auto unit = [&](const ChunkSeg&, int) -> bool { return true; };
  auto stage = [&](const ChunkTile& t0, const ChunkTile& t1) -> bool {
    const int st = pos % C::NST, cb = pos & 1;
    if (!C::IN_PLACE && !wait(bar.kv_empty(st), ((pos / C::NST) & 1) ^ 1)) return false;
    if (!wait(bar.code_full(cb), (pos >> 1) & 1)) return false;
    ++pos;
    const int groups = t1.kind ? C::BK / 8 : C::BK / 16;
#pragma unroll 1
    for (int gr = cw; gr < groups; gr += WARPS) {
      const int i = gr / (C::BK / 16), r16 = gr % (C::BK / 16) * 16;
      const int end = (i == 0 ? t0.len - t0.key0 : t1.len - t1.key0) - r16;  // rows of these 16 that are keys
      const uint8_t* codes = gbase + chunk_codes<D>(st, cb, i) + r16 * C::CODE_COLS + from;
      const uint8_t* scales = gbase + C::OFF_SCALE + (cb * 2 + i) * C::BK + r16;
      const uint32_t dst = base + C::OFF_KV + st * C::STAGE + i * C::KV_TILE + r16 * C::SWB;
      const uint32_t big = lane < 4 ? __vcmpgtu4(reinterpret_cast<const uint32_t*>(scales)[lane], 0x86868686u) : 0u;  // a byte > 134
      // From `pass` on; where not `checked`, up to the first batch that holds a NaN code.
      auto convert = [&](auto checked, int pass) -> int {
#pragma unroll 1
        for (; pass < PASSES; pass += BATCH) {
          uint2 x[BATCH];
          uint32_t byte[BATCH], w[BATCH][4];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            x[k] = *reinterpret_cast<const uint2*>(codes + (pass + k) * RPP * C::CODE_COLS);
            byte[k] = scales[(pass + k) * RPP + row0];
          }
          if constexpr (!decltype(checked)::value) {
            uint32_t nan = 0;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) nan |= e4m3x4_any_nan(x[k].x) | e4m3x4_any_nan(x[k].y);
            if (__any_sync(0xffffffffu, (nan & 0x80808080u) != 0)) return pass;
          }
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            uint32_t f = byte[k] * 0x00800080u + 120u * 0x00800080u;  // 2^(120 + e), twice
            if constexpr (decltype(checked)::value)
              f = byte[k] == 255u ? 0x7fc07fc0u : byte[k] > 134u ? 0x7f007f00u : f;  // NaN, or 2^127 at most
            e4m3x4_to_bf16x4(x[k].x, f, w[k][0], w[k][1]);
            e4m3x4_to_bf16x4(x[k].y, f, w[k][2], w[k][3]);
            if constexpr (decltype(checked)::value) {
              const uint32_t f2 = byte[k] > 134u && byte[k] != 255u ? (byte[k] - 7u) * 0x00800080u : 0x3f803f80u;  // 2^(e - 7)
              const bool past = (pass + k) * RPP + row0 >= end;
#pragma unroll
              for (int i2 = 0; i2 < 4; ++i2) {
                const uint32_t nan = e4m3x4_nan(i2 < 2 ? x[k].x : x[k].y);
                w[k][i2] = past ? 0u : mul_bf16x2(w[k][i2], f2) | (i2 & 1 ? nan_bf16x2<true>(nan) : nan_bf16x2<false>(nan));
              }
            }
          }
          if constexpr (C::IN_PLACE) __syncwarp();  // the rows have been read by all of the warp
#pragma unroll
          for (int k = 0; k < BATCH; ++k) st_shared_v4(dst + to[k] + pass * RPP * C::SWB, w[k][0], w[k][1], w[k][2], w[k][3]);
        }
        return PASSES;
      };
      const int done = end >= 16 && !__any_sync(0xffffffffu, big != 0) ? convert(std::false_type{}, 0) : 0;
      if (done < PASSES) convert(std::true_type{}, done);
    }
    fence_proxy_async_smem();  // before the tensor core reads them
    if constexpr (!C::IN_PLACE) warp_arrive(bar.code_empty(cb));
    warp_arrive(bar.kv_full(st));
    return true;
  };
  return chunk_stream<D>(get, unit, stage);
}

// ------------------------------------------------------------------ MMA issuer
// tc_mma's order of products, segment by segment.
template <int D, bool E4M3>
__device__ __forceinline__ void chunk_mma(const ChunkParams& p, const ChunkBars<D, E4M3>& bar, uint32_t base,
                                          uint8_t* gbase, uint32_t tmem, const WaitGuard& g) {
  using C = ChunkCfg<D, E4M3>;
  const TcMma<D, C::NQT, kVarBf16> M(tmem, base);
  const int lane = threadIdx.x & 31;
  auto wait = [&](uint32_t b, uint32_t par) -> bool {
    return __all_sync(0xffffffffu, mbar_test_wait(b, par)) || chunk_wait(b, par, g, kStatusTimeoutMma);
  };
  uint32_t pos = 0;
  uint32_t go0 = 0;
  bool ok = true;
  auto stage_acquire = [&](uint32_t& st) -> bool {
    st = pos % C::NST;
    const bool r = wait(bar.kv_full(st), (pos / C::NST) & 1);
    ++pos;
    if (r) tc_fence_after();
    return r;
  };
  // V rows behind the sequence's end in the tile at stage st (key tile j of w): zeros.
  auto clear_tail = [&](const ChunkSeg& w, int j, uint32_t st) {
    if constexpr (!E4M3) {
      const int end = w.len - (w.j0 + j) * C::BK;
      if (end >= C::BK) return;
      const int from = end < 0 ? 0 : end;
      constexpr int UR = C::SWB / 16;
      const uint32_t vt = base + C::OFF_KV + 2 * st * C::KV_TILE;
      for (int r = 0; r < C::NR; ++r)
        for (int i = from * UR + lane; i < C::BK * UR; i += 32) st_shared_v4(vt + r * C::V_REGION + i * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
    }
  };
  auto get = [&](int k, ChunkSeg& w) -> bool { return seg_read<D, E4M3>(w, k, gbase, bar, g); };

  ChunkSeg w;
  ok = get(0, w);
  if constexpr (C::NQT == 2) {
    auto tiles_of = [](const ChunkSeg& x, int t) -> int { return t == 0 ? x.n0 : x.n1; };
    // S of key tile 0 of segment k for both tiles, K_0 at position kpos.
    auto first_qk = [&](const ChunkSeg& x, int k, uint32_t kpos) -> bool {
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        if (!wait(bar.q_full(t), k & 1)) return false;
        tc_fence_after();
        if (tiles_of(x, t) > 0) M.qk(t, t, kpos, bar.s_full(t));
        if (tiles_of(x, t) <= 1) M.commit(bar.q_empty(t));
      }
      return true;
    };
    uint32_t go = 0;    // bit t: parity of tile t's P V products
    uint32_t free_par = 0;  // bit t: parity of its units' first ones
    bool begun = false;
#pragma unroll 1
    for (int k = 0; ok && w.valid; ++k) {
      ChunkSeg wn;
      if (!(ok = get(k + 1, wn))) break;
#pragma unroll 1
      for (int j = begun ? 0 : -1; ok && j < w.nmax; ++j) {
        uint32_t st;
        if (!(ok = stage_acquire(st))) break;
        if (j >= 0) {
          clear_tail(w, j, st);
          // P V_t j, then S_t of key tile j + 1, tile by tile (unrolled: this warp's pace is the tensor core's).
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int n = tiles_of(w, t);
            if (j >= n || !ok) continue;
            const uint32_t par = (go >> t) & 1;
            if (j == 0) {  // O has been read out (or is free from the start)
              if (!(ok = wait(bar.o_free(t), (free_par >> t) & 1))) break;
              free_par ^= 1u << t;
            }
            if (!(ok = wait(bar.pv_go(t, 0), par))) break;
            tc_fence_after();
            if constexpr (C::PV_SPLIT) {
              M.pv_half(t, t, 2 * st, 0, j > 0);
              if (!(ok = wait(bar.pv_go(t, 1), par))) break;
              tc_fence_after();
              M.pv_half(t, t, 2 * st, 1, true);
            } else {
              M.pv(t, t, 2 * st, j > 0);
            }
            go ^= 1u << t;
            if (j == n - 1) {
              M.commit(bar.o_done(t));
            } else {
              M.qk(t, t, 2 * st + 1, bar.s_full(t));
              if (j + 1 == n - 1) M.commit(bar.q_empty(t));
            }
          }
        }
        // The next segment's first products (in the stage of this one's last V; the very first K_0 stands alone).
        if (ok && (j < 0 || (j == w.nmax - 1 && wn.valid)))
          ok = first_qk(j < 0 ? w : wn, j < 0 ? k : k + 1, j < 0 ? 2 * st : 2 * st + 1);
        if (ok) M.commit(bar.kv_empty(st));
      }
      begun = true;
      w = wn;
    }
  } else {
    uint32_t qk_total = 0;
    for (int k = 0; ok && w.valid; ++k) {
      if (!(ok = wait(bar.q_full(0), k & 1))) break;
      tc_fence_after();
      uint32_t st;
      if (!(ok = stage_acquire(st))) break;
      const int n = w.n0;
      const uint32_t qk_base = qk_total;
      for (int t = 0; t < C::LA && t < n; ++t) {
        M.qk(0, qk_total & 1, 2 * st + t, bar.s_full(qk_total & 1));
        ++qk_total;
      }
      M.commit(bar.kv_empty(st));
      if (n <= C::LA) M.commit(bar.q_empty(0));
      for (int j = 0; j < n; ++j) {
        if (!(ok = stage_acquire(st))) break;
        clear_tail(w, j, st);
        if (!(ok = wait(bar.pv_go(0, go0 & 1), (go0 >> 1) & 1))) break;
        ++go0;
        tc_fence_after();
        M.pv(0, (qk_base + j) & 1, 2 * st, j > 0);
        M.commit(bar.o_done(0));
        if (j + C::LA < n) {
          M.qk(0, qk_total & 1, 2 * st + 1, bar.s_full(qk_total & 1));
          ++qk_total;
          if (j + C::LA == n - 1) M.commit(bar.q_empty(0));
        }
        M.commit(bar.kv_empty(st));
      }
      if (ok) ok = get(k + 1, w);
    }
  }
  (void)go0;
  M.commit(bar.drain());
  wait_bar_drain(bar.drain(), 0, g);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
// tc_softmax with the rows' limits taken from the segment.
template <int D, bool E4M3>
__device__ __forceinline__ void chunk_softmax(const ChunkParams& p, const ChunkBars<D, E4M3>& bar, uint8_t* gbase,
                                              uint32_t tmem, int wg, int quarter, int lane, const WaitGuard& g) {
  using C = ChunkCfg<D, E4M3>;
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const int ot = (C::NQT == 2) ? wg : 0;
  float* alpha_s = reinterpret_cast<float*>(gbase + C::OFF_ALPHA) + ot * 256;
  uint32_t a_pub = 0;
  float* stat_m = reinterpret_cast<float*>(gbase + C::OFF_STAT_M) + ot * 128;
  float* stat_l = reinterpret_cast<float*>(gbase + C::OFF_STAT_L) + ot * 128;
  const float sl2 = p.scale_log2;
  const uint64_t sl2x2 = f2_pack(sl2, sl2);
  uint32_t s_waits = 0;
  int fin = 0;  // units finished by this warpgroup
  bool ok = true;
  const int tok_r = min(wg * p.tpt + r / p.a.group, (wg + 1) * p.tpt - 1);  // this row's token within the block

  for (int uk = 0; ok; ++uk) {
    int n, j0, lim0, min_lim, len;
    {
      ChunkSeg w;
      ok = seg_read<D, E4M3, true>(w, uk, gbase, bar, g);
      if (!ok || !w.valid) break;
      n = wg == 0 ? w.n0 : w.n1;
      j0 = w.j0;
      len = w.len;
      // Rows behind the block's last token take that one's limit (they are not written).
      lim0 = p.a.causal ? w.pos0 + min(tok_r, w.ntok - 1) : w.len - 1;
      min_lim = p.a.causal ? w.pos0 + wg * p.tpt : w.len - 1;
    }
    if (n == 0) continue;
    lim0 = min(lim0, len - 1);
    float m = -INFINITY;
    float l = 0.f;
    float lres = 0.f;
    for (int j = 0; j < n; ++j) {
      const int buf = (C::NQT == 2) ? wg : static_cast<int>(s_waits & 1);
      const uint32_t par = (C::NQT == 2) ? (s_waits & 1) : ((s_waits >> 1) & 1);
      ok = warp_wait_bar(bar.s_full(buf), par, g, kStatusTimeoutSoftmax);
      if (!ok) break;
      ++s_waits;
      tc_fence_after();
      const uint32_t ts = tmem + lane_off + C::TM_S + buf * C::TM_SB;
      const int key0 = (j0 + j) * C::BK;
      float s[C::BK];
      float rmax;
      auto fetch = [&]() {
        float cmax[C::BK / 32];
        {
          uint32_t raw_s[C::BK / 32][32];
#pragma unroll
          for (int c = 0; c < C::BK / 32; ++c) tmem_ld32_max(ts + c * 32, raw_s[c], cmax[c]);
#pragma unroll
          for (int c = 0; c < C::BK / 32; ++c) tmem_wait_ld(raw_s[c], cmax[c]);
#pragma unroll
          for (int c = 0; c < C::BK / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(raw_s[c][i]);
        }
        if (key0 + C::BK - 1 > min_lim) {
          const int lim = lim0 - key0;
          const int lo = __reduce_min_sync(0xffffffffu, lim);
#pragma unroll
          for (int cb = 0; cb < C::BK / 32; ++cb) {
            if (32 * cb + 31 > lo) {
              // Bit i: column 32 cb + i is behind the limit.
              const int v = lim - 32 * cb;
              const uint32_t hide = v < 0 ? 0xffffffffu : v >= 31 ? 0u : 0xfffffffeu << v;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((hide >> i) & 1) s[32 * cb + i] = -INFINITY;
            }
          }
          constexpr int KC = C::BK / 8;
          float mx[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v = fmax3(s[i], s[i + 8], s[i + 16]);
#pragma unroll
            for (int k = 3; k + 1 < KC; k += 2) v = fmax3(v, s[i + 8 * k], s[i + 8 * (k + 1)]);
            if ((KC - 3) % 2 == 1) v = fmaxf(v, s[i + 8 * (KC - 1)]);
            mx[i] = v;
          }
          rmax = fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7]));
        } else {
          rmax = cmax[0];
#pragma unroll
          for (int c = 1; c < C::BK / 32; ++c) rmax = fmaxf(rmax, cmax[c]);
        }
      };
      fetch();
      if constexpr (C::SELF_RESCALE) {
        // The reference maximum moves (rarely) where the row's exceeds it by more than MAX_SLACK.
        const float rm = rmax * sl2;
        const bool moves = rm > m + C::MAX_SLACK;
        if (__any_sync(0xffffffffu, moves)) {
          const float alpha = moves ? ex2(m - rm) : 1.f;
          m = moves ? rm : m;
          l *= alpha;
          lres *= alpha;
          if (j > 0) {
            // Rescale O (P V j - 1 is done: S j was issued behind it), then fetch S again: the registers hold one of them.
            // (A second copy of the fetch: as a loop the common path took 5 % longer.)
            const uint32_t to = tmem + lane_off + C::TM_O + ot * D;
            const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(to + c * 32, v);
              tmem_wait_ld(v);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 y = f2_unpack(f2_mul(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), a2));
                v[i] = __float_as_uint(y.x);
                v[i + 1] = __float_as_uint(y.y);
              }
              tmem_st32(to + c * 32, v);
            }
            tmem_wait_st();
            fetch();
          }
        }
      }
      uint32_t after = 0;  // (0; the exponentials below are scheduled behind the arrival, as in tc_softmax)
      if constexpr (!C::SELF_RESCALE) {
        const float m_new = fmaxf(m, rmax * sl2);
        const float alpha = (m_new == m) ? 1.f : ex2(m - m_new);
        l *= alpha;
        m = m_new;
        if (j > 0) {
          alpha_s[(a_pub & 1) * 128 + r] = alpha;
          after = warp_arrive_token(bar.a_full(ot, a_pub & 1));
          ++a_pub;
        }
      }
      float nb = (m == -INFINITY) ? 0.f : -m;
      if constexpr (!C::SELF_RESCALE) nb = fmaf(0.f, __uint_as_float(after), nb);
      const uint64_t nb2 = f2_pack(nb, nb);
      if constexpr (C::LAZY_MAX) {
        const float pmax = ex2(fmaf(rmax, sl2, nb));
        const float pr = __uint_as_float(pack_bf16x2(pmax, 0.f) << 16);
        lres += pr - pmax;
      }
      uint64_t acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = 0ull;
#pragma unroll
      for (int h = 0; h < C::BK / 64; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 64 * h; c < 64 * h + 64; c += 2) {
          const float2 x = f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), sl2x2, nb2));
          const float p0 = ex2(x.x);
          const float p1 = ex2(x.y);
          pk[(c >> 1) & 31] = pack_bf16x2(p0, p1);
          acc[(c >> 1) & 3] = f2_add(acc[(c >> 1) & 3], f2_pack(p0, p1));
        }
        tmem_st32(ts + h * C::P_COLS_64, pk);
        if constexpr (C::PV_SPLIT) {
          if (h == 0) {
            tmem_wait_st();
            tc_fence_before();
            warp_arrive_elect(bar.pv_go(ot, 0));
          }
        }
      }
      const float2 a01 = f2_unpack(f2_add(acc[0], acc[1]));
      const float2 a23 = f2_unpack(f2_add(acc[2], acc[3]));
      l += (a01.x + a01.y) + (a23.x + a23.y);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(C::NQT == 2 ? bar.pv_go(ot, C::PV_SPLIT ? 1 : 0) : bar.pv_go(0, (s_waits - 1) & 1));
    }
    if (!ok) break;
    // The row's log2-sum-exp2 and O's normaliser.
    stat_m[(fin & 1) * 256 + r] = m + log2f(l);
    stat_l[(fin & 1) * 256 + r] = l + lres;
    warp_arrive(bar.ml_full(ot, fin));
    ++fin;
  }
}

// ------------------------------------------------------------------ correction + output
template <int D, bool E4M3>
__device__ __forceinline__ void chunk_correction(const ChunkParams& p, const CUtensorMap* tm_o,
                                                 const ChunkBars<D, E4M3>& bar, uint32_t base, uint8_t* gbase,
                                                 uint32_t tmem, int quarter, int lane, const WaitGuard& g) {
  using C = ChunkCfg<D, E4M3>;
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const float* alpha_base = reinterpret_cast<const float*>(gbase + C::OFF_ALPHA);
  const float* stat_m = reinterpret_cast<const float*>(gbase + C::OFF_STAT_M);
  const float* stat_l = reinterpret_cast<const float*>(gbase + C::OFF_STAT_L);
  constexpr bool PER_PV_DONE = (C::NQT == 1);
  const int tok_r = r / p.a.group, head_r = r - tok_r * p.a.group;
  const uint32_t out = smem_u32(gbase + C::OFF_OUT) + static_cast<uint32_t>(quarter * C::OUT_BUFS * C::OST_BUF);
  uint32_t out_n = 0;  // chunks staged by this warp
  uint32_t a_cnt = 0, od = 0, lf = 0;  // counts modulo 4 of tile t in bits 2t, 2t + 1
  uint32_t go_arr = 0;
  bool ok = true;
  uint64_t odd2 = 0;  // sums of 0 times every O of this thread: NaN if one was infinite or NaN
  auto release_o = [&](int t) {
    if (C::SELF_RESCALE) {
      warp_arrive(bar.o_free(t));
    } else {
      warp_arrive(bar.pv_go(0, go_arr & 1));
      ++go_arr;
    }
  };
  auto count = [](uint32_t c, int t) -> uint32_t { return (c >> (2 * t)) & 3; };
  auto up = [](uint32_t& c, int t) { c = (c & ~(3u << (2 * t))) | ((((c >> (2 * t)) + 1) & 3u) << (2 * t)); };
  auto rescale = [&](int t) -> bool {
    const uint32_t ac = count(a_cnt, t);
    bool k = chunk_wait(bar.a_full(t, ac & 1), ac >> 1, g, kStatusTimeoutSoftmax);
    if (!k) return false;
    const float alpha = alpha_base[t * 256 + (ac & 1) * 128 + r];
    up(a_cnt, t);
    if (PER_PV_DONE) {
      k = chunk_wait(bar.o_done(t), count(od, t) & 1, g, kStatusTimeoutSoftmax);
      if (!k) return false;
      up(od, t);
    }
    if (__any_sync(0xffffffffu, alpha != 1.f)) {
      tc_fence_after();
      const uint32_t to = tmem + lane_off + C::TM_O + t * D;
      const uint64_t a2 = f2_pack(alpha, alpha);
      constexpr int RG = (C::NQT == 1) ? (D / 32 < 4 ? D / 32 : 4) : 1;
#pragma unroll 1
      for (int c = 0; c < D / 32; c += RG) {
        uint32_t v[RG][32];
#pragma unroll
        for (int k2 = 0; k2 < RG; ++k2) tmem_ld32(to + (c + k2) * 32, v[k2]);
#pragma unroll
        for (int k2 = 0; k2 < RG; ++k2) tmem_wait_ld(v[k2]);
#pragma unroll
        for (int k2 = 0; k2 < RG; ++k2) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 y = f2_unpack(f2_mul(f2_pack(__uint_as_float(v[k2][i]), __uint_as_float(v[k2][i + 1])), a2));
            v[k2][i] = __float_as_uint(y.x);
            v[k2][i + 1] = __float_as_uint(y.y);
          }
        }
#pragma unroll
        for (int k2 = 0; k2 < RG; ++k2) tmem_st32(to + (c + k2) * 32, v[k2]);
      }
      tmem_wait_st();
    }
    tc_fence_before();
    release_o(t);
    return true;
  };
  // O of tile t: the rows of a whole unit, or this CTA's part of them.
  auto epilogue = [&](const ChunkSeg& w, int t) -> bool {
    const int su = count(lf, t) & 1;
    bool k = chunk_wait(bar.o_done(t), count(od, t) & 1, g, kStatusTimeoutSoftmax);
    k = k && chunk_wait(bar.ml_full(t, su), count(lf, t) >> 1, g, kStatusTimeoutSoftmax);
    if (!k) return false;
    up(od, t);
    up(lf, t);
    tc_fence_after();
    const float lsum = stat_m[su * 256 + t * 128 + r];
    const float lrow = stat_l[su * 256 + t * 128 + r];
    const float inv_l = lrow == 0.f ? 0.f : 1.f / lrow;
    const uint64_t il2 = f2_pack(inv_l, inv_l);
    const int tok = t * p.tpt + tok_r;
    const bool mine = tok_r < p.tpt && tok < w.ntok;
    const uint32_t to = tmem + lane_off + C::TM_O + t * D;
    const int hq = w.head * p.a.group + head_r;
    // Where this row of O is (-1: it is no row).
    const long long row_off =
        mine ? static_cast<long long>(w.row0 + tok) * p.a.os[0] + static_cast<long long>(hq) * p.a.os[1] : -1ll;
    float* part = p.ws.chunk_part + (static_cast<size_t>(blockIdx.x) * 2 + (w.out - 1)) * part_floats(C::ROWS, D);
    float4* pblk = reinterpret_cast<float4*>(part + C::ROWS + static_cast<size_t>(t) * 128 * D) + r;
    // All 32 rows of this warp are rows of O: a box of min(G, 32) heads.
    const int in = quarter * 32 / p.a.group;
    const bool boxed = p.tma_o && t * p.tpt + (quarter * 32 + 31) / p.a.group < w.ntok;
    const int box_head = w.head * p.a.group + (quarter * 32 - in * p.a.group), box_row = w.row0 + t * p.tpt + in;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t v[32];
      tmem_ld32(to + c * 32, v);
      tmem_wait_ld(v);
      if (c == D / 32 - 1) {
        tc_fence_before();
        release_o(t);
      }
      if (mine) {
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          odd2 = f2_fma(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), 0ull, odd2);
      }
      if (w.out == 0) {
        uint32_t y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = f2_unpack(f2_mul(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), il2));
          y[i] = pack_bf16x2(x.x, x.y);
        }
        if (boxed) {
          // As in tc_correction: staged in shared memory, stored by TMA.
          const uint32_t buf = out + (out_n % C::OUT_BUFS) * C::OST_BUF;
          ++out_n;
          if (lane == 0) bulk_wait_group_read<C::OUT_BUFS - 1>();
          __syncwarp();
          const uint32_t rb = buf + static_cast<uint32_t>(lane) * 64;
          const uint32_t sw = static_cast<uint32_t>((lane >> 1) & 3);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            st_shared_v4(rb + ((static_cast<uint32_t>(u) ^ sw) << 4), y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(tm_o, buf, c * 32, box_head, box_row);
            bulk_commit_group();
          }
        } else if (mine) {
          uint4* dst = reinterpret_cast<uint4*>(p.a.o + row_off + c * 32);
#pragma unroll
          for (int u = 0; u < 4; ++u) dst[u] = make_uint4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
        }
      } else {
        // 16-byte block i of all 128 rows of the tile together.
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 x = f2_unpack(f2_mul(f2_pack(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), il2));
          const float2 y = f2_unpack(f2_mul(f2_pack(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), il2));
          pblk[(c * 8 + i) * 128] = make_float4(x.x, x.y, y.x, y.y);
        }
      }
      __syncwarp();
    }
    if (mine) {
      if (w.out == 0)
        p.a.lse[static_cast<long long>(hq) * p.a.pb.rows + w.row0 + tok] = lsum * 0.69314718055994531f;
      else
        part[t * 128 + r] = lsum;
    }
    return true;
  };

  release_o(0);
  if (C::NO == 2) release_o(1);
  // A tile whose keys all lie before this part has nothing to add.
  auto nothing = [&](const ChunkSeg& w) {
    if (C::NQT == 2 && w.n0 == 0)
      p.ws.chunk_part[(static_cast<size_t>(blockIdx.x) * 2 + (w.out - 1)) * part_floats(C::ROWS, D) + r] = -INFINITY;
  };
  if constexpr (!(E4M3 && C::SELF_RESCALE)) {
    for (int uk = 0; ok; ++uk) {
      ChunkSeg w;
      ok = seg_read<D, E4M3>(w, uk, gbase, bar, g);
      if (!ok || !w.valid) break;
      nothing(w);
      if constexpr (!C::SELF_RESCALE) {
#pragma unroll 1
        for (int j = 1; ok && j < w.nmax; ++j) ok = rescale(0);
      }
#pragma unroll 1
      for (int t = 0; ok && t < C::NO; ++t)
        if ((t == 0 ? w.n0 : w.n1) > 0) ok = epilogue(w, t);
    }
  } else {
    // Converting, and in between the outputs as they are finished.  A segment is held in the ring until its output is
    // out, so the waits below have to go on with the outputs (the load warp may wait for the ring, the MMA warp for O).
    int seen = 0, out_k = 0, out_t = 0;  // segments fetched; the next output
    auto output = [&](bool block) -> bool {
      if (out_k >= seen) return true;
      const ChunkSeg& w = *seg_slot<D, E4M3>(gbase, out_k);
      if (out_t < 2) {
        if ((out_t == 0 ? w.n0 : w.n1) == 0) {
          if (out_t == 0) nothing(w);
          ++out_t;
        } else if (block || __all_sync(0xffffffffu, mbar_test_wait(bar.o_done(out_t), count(od, out_t) & 1))) {
          const ChunkSeg copy = w;
          if (!epilogue(copy, out_t)) return false;
          ++out_t;
        }
      }
      if (out_t == 2) {
        warp_arrive(bar.seg_empty(out_k % kSegRing));
        ++out_k;
        out_t = 0;
      }
      return true;
    };
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
      uint64_t t0 = 0;
      while (true) {
        if (__all_sync(0xffffffffu, mbar_test_wait(b, parity))) return true;
        const int before = out_k * 2 + out_t;
        if (!output(false)) return false;
        // The other tile's output, if that is ready, goes first, too: its accumulator waits for it (in place, chunks of
        // 64 tokens over 512: 306 to 275 us; with buffers of their own the codes are there earlier, and it costs 2 %).
        if (C::IN_PLACE && out_k * 2 + out_t != before) continue;
        if (__all_sync(0xffffffffu, mbar_try_wait_ns(b, parity, 300))) return true;
        if (__any_sync(0xffffffffu, *g.abort)) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, now - t0 > g.limit_ns)) {
          *g.abort = 1;
          if (lane == 0) atomicOr(g.status, kStatusTimeoutLoad);
          return false;
        }
      }
    };
    auto get = [&](int k, ChunkSeg& w) -> bool {
      if (!wait(bar.seg_full(k % kSegRing), (k / kSegRing) & 1)) return false;
      w = *seg_slot<D, E4M3>(gbase, k);
      if (w.valid) seen = k + 1;
      return true;
    };
    ok = chunk_convert<D, E4M3>(p, bar, base, gbase, quarter, get, wait);
    while (ok && out_k < seen) ok = output(true);
  }
  if (lane == 0) bulk_wait_group_all();  // staged chunks are written before the CTA leaves
  __syncwarp();
  const float2 odd = f2_unpack(odd2);
  const int any = __any_sync(0xffffffffu, odd.x != 0.f || odd.y != 0.f);
  if (lane == 0) p.ws.odd[blockIdx.x * 4 + quarter] = any;
}

// ------------------------------------------------------------------ kernel
template <int D, bool E4M3>
__global__ void __launch_bounds__(TcCfg<D>::THREADS, 1)
    fa_paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                          const __grid_constant__ ChunkParams p) {
  using C = ChunkCfg<D, E4M3>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  ChunkBars<D, E4M3> bar;
  bar.b0 = base + C::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_TMEM_SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_ABORT);

  pdl_launch_dependents();  // the few-row kernel's blocks take the SMs as this kernel's leave them
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar.q_full(t), 1);
      mbar_init(bar.q_empty(t), 1);
    }
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(bar.kv_full(i), E4M3 ? C::CONV_WARPS : C::LOADERS);
      mbar_init(bar.kv_empty(i), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar.s_full(b), 1);
      mbar_init(bar.pv_go(b, 0), C::SELF_RESCALE ? 4 : 8);  // 4 softmax warps (+ 4 correction warps)
      mbar_init(bar.pv_go(b, 1), C::SELF_RESCALE ? 4 : 8);
      mbar_init(bar.a_full(b, 0), 4);
      mbar_init(bar.a_full(b, 1), 4);
      mbar_init(bar.o_done(b), 1);
      mbar_init(bar.ml_full(b, 0), 4);
      mbar_init(bar.ml_full(b, 1), 4);
    }
    mbar_init(bar.drain(), 1);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(bar.seg_full(i), 1);
      mbar_init(bar.seg_empty(i), C::SEG_READERS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.code_full(i), 1);
      mbar_init(bar.code_empty(i), E4M3 ? C::CONV_WARPS : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::LOAD_WARP && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_o);
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TM_COLS);
    tmem_relinquish();
  }
  const PlanShare share = plan_share<C::THREADS>(
      p.a.pb.B, gridDim.x, blockIdx.x,
      [&](int b) -> long long {
        bool bad;
        const ChunkBlocks c = chunk_blocks<D, E4M3>(p, paged_seq(p.a.pb, p.a.kv.ps_log2, b, bad));
        return c.n == 0 ? 0 : p.a.kv.heads * c.before(c.count());
      },
      1 + C::UNIT_COST,
      *reinterpret_cast<PlanScratch*>(gbase + C::OFF_PLAN));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitGuard g{abort_flag, p.status, p.limit_ns};

  if (warp < C::SOFTMAX_WARPS) {
    if constexpr (C::SPLIT_REGS) regs_increase<C::REG_SOFTMAX>();
    chunk_softmax<D, E4M3>(p, bar, gbase, tmem, warp >> 2, warp & 3, lane, g);
  } else if (warp < C::SOFTMAX_WARPS + 4) {
    if constexpr (C::SPLIT_REGS) regs_decrease<C::reg_corr(false)>();
    chunk_correction<D, E4M3>(p, &tm_o, bar, base, gbase, tmem, warp & 3, lane, g);
  } else {
    if constexpr (C::SPLIT_REGS) regs_decrease<C::REG_CORR_OTHER - C::reg_corr(false)>();
    if (warp >= C::LOAD_WARP && warp < C::LOAD_WARP + C::LOADERS)
      chunk_load<D, E4M3>(&tm_q, &tm_k, &tm_v, p, bar, base, gbase, share, warp > C::LOAD_WARP, g);
    if (warp == C::MMA_WARP) chunk_mma<D, E4M3>(p, bar, base, gbase, tmem, g);
    if constexpr (E4M3)
      if (warp >= C::CONV_WARP0)
        chunk_convert<D, E4M3>(
            p, bar, base, gbase, warp - C::CONV_WARP0 + C::CONV_WARPS - 2,
            [&](int k, ChunkSeg& w) -> bool { return seg_read<D, E4M3>(w, k, gbase, bar, g); },
            [&](uint32_t b, uint32_t parity) -> bool { return chunk_wait(b, parity, g, kStatusTimeoutLoad); });
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// ------------------------------------------------------------------ joining
struct JoinParams {
  PagedFwdArgs a;
  PagedWs ws;
  bool chunks;   // the chunk kernel has run
  int few_sets;  // launches of the few-row kernel
  int tpt;
};

// Joins the parts of the units that several CTAs held; blocks (c, .) those of the unit that CTA c began.
template <int D>
__global__ void __launch_bounds__(128) fa_paged_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float s_o[3][D];
  pdl_wait();
  const PagedFwdArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.chunks) {
    const PlanRecord rec = p.ws.chunk_rec[blockIdx.x];
    if (rec.b >= 0) {
      // A warp takes 16 columns of 32 rows, a row a lane (parts hold blocks of 4 columns of all rows of a tile).
      constexpr int ROWS = chunk_rows(D);
      bool bad;
      const PagedSeq s = paged_seq(a.pb, a.kv.ps_log2, rec.b, bad);
      constexpr size_t stride = 2 * part_floats(ROWS, D);  // from one CTA's parts to the next's
      const float* first = p.ws.chunk_part + blockIdx.x * stride + stride / 2;
      const float* rest = first + stride / 2 - stride;  // part 0 of CTA + i at rest + i * stride
      const int n = rec.more + 1;
      for (int job = blockIdx.y * 4 + warp; job < ROWS / 32 * (D / 16); job += gridDim.y * 4) {
        const int r = job % (ROWS / 32) * 32 + lane, c16 = job / (ROWS / 32);
        const int tr = (r & 127) / a.group, head = (r & 127) % a.group;
        const int tok = (rec.qb * (ROWS / 128) + (r >> 7)) * p.tpt + tr;
        if (tr >= p.tpt || tok >= s.n) continue;
        float m = -INFINITY;
#pragma unroll 4
        for (int i = 0; i < n; ++i) m = fmaxf(m, (i == 0 ? first : rest + i * stride)[r]);
        float l = 0.f;
        float4 o[4] = {};
        const size_t at = ROWS + static_cast<size_t>(r >> 7) * 128 * D + (static_cast<size_t>(c16) * 4 * 128 + (r & 127)) * 4;
#pragma unroll 2
        for (int i = 0; i < n; ++i) {
          const float* x = i == 0 ? first : rest + i * stride;
          const float lg = x[r];
          if (lg == -INFINITY) continue;  // (a part that saw none of the row's keys holds no O)
          const float f = ex2(lg - m);
          l += f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 y = *reinterpret_cast<const float4*>(x + at + k * 512);
            o[k].x = fmaf(y.x, f, o[k].x);
            o[k].y = fmaf(y.y, f, o[k].y);
            o[k].z = fmaf(y.z, f, o[k].z);
            o[k].w = fmaf(y.w, f, o[k].w);
          }
        }
        const int row = s.row0 + tok, hq = rec.head * a.group + head;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint4* dst = reinterpret_cast<uint4*>(a.o + static_cast<long long>(row) * a.os[0] +
                                              static_cast<long long>(hq) * a.os[1] + c16 * 16);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          dst[k] = make_uint4(pack_bf16x2(o[2 * k].x * inv, o[2 * k].y * inv), pack_bf16x2(o[2 * k].z * inv, o[2 * k].w * inv),
                              pack_bf16x2(o[2 * k + 1].x * inv, o[2 * k + 1].y * inv),
                              pack_bf16x2(o[2 * k + 1].z * inv, o[2 * k + 1].w * inv));
        if (c16 == 0) a.lse[static_cast<long long>(hq) * a.pb.rows + row] = (m + log2f(l)) * 0.69314718055994531f;
      }
    }
  }
#pragma unroll 1
  for (int set = 0; set < p.few_sets; ++set) {
    const PlanRecord rec = p.ws.few_rec[set][blockIdx.x];
    if (rec.b < 0) continue;
    bool bad;
    const PagedSeq s = paged_seq(a.pb, a.kv.ps_log2, rec.b, bad);
    constexpr size_t stride = 2 * part_floats(kFewMost, D);
    const float* first = p.ws.few_part[set] + blockIdx.x * stride + stride / 2;
    const float* rest = first + stride / 2 - stride;
    const int n = rec.more + 1;
    // Few parts: a warp to a row.  Many: the four warps share out a row's parts.
    const bool split = n > 4;
    const int step = split ? gridDim.y : gridDim.y * 4;
    for (int r = split ? blockIdx.y : blockIdx.y * 4 + warp; r < s.n * a.group; r += step) {
      // m: the largest L; l: sum of 2^(L - m).
      float m = -INFINITY;
      for (int i = lane; i < n; i += 32) m = fmaxf(m, (i == 0 ? first : rest + i * stride)[r]);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      float l = 0.f, o[D / 32] = {};
      for (int i0 = 0; i0 < n; i0 += 32) {
        float w = -1.f;  // (no part, or one that saw none of the row's keys)
        if (i0 + lane < n) {
          const float x = (i0 + lane == 0 ? first : rest + (i0 + lane) * stride)[r];
          if (x != -INFINITY) w = ex2(x - m);
        }
        float sum = w < 0.f ? 0.f : w;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        l += sum;
        const int to = min(32, n - i0);
#pragma unroll 4
        for (int i = split ? warp : 0; i < to; i += split ? 4 : 1) {
          const float f = __shfl_sync(0xffffffffu, w, i);
          const float* x = (i0 + i == 0 ? first : rest + (i0 + i) * stride) + kFewMost + static_cast<size_t>(r) * D;
          if (f >= 0.f) {  // (where f = 0, too: a NaN that the row sees counts at any weight; f = NaN is in l already)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] = fmaf(x[c * 32 + lane], f, o[c]);
          }
        }
      }
      if (split) {
        if (warp > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) s_o[warp - 1][c * 32 + lane] = o[c];
        }
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
            o[c] = (o[c] + s_o[0][c * 32 + lane]) + (s_o[1][c * 32 + lane] + s_o[2][c * 32 + lane]);
        }
        __syncthreads();
        if (warp > 0) continue;
      }
      const int row = s.row0 + r / a.group, hq = rec.head * a.group + r % a.group;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      __nv_bfloat16* dst = a.o + static_cast<long long>(row) * a.os[0] + static_cast<long long>(hq) * a.os[1];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) dst[c * 32 + lane] = __float2bfloat16_rn(o[c] * inv);
      if (lane == 0) a.lse[static_cast<long long>(hq) * a.pb.rows + row] = (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

template <int D>
int launch_paged_join(const PagedFwdArgs& a, bool chunks, const LaunchCtx& ctx) {
  const int ctas = ctx.num_sms < kPlanCtas ? ctx.num_sms : kPlanCtas;
  const JoinParams p{a, paged_ws(a.workspace, D), chunks, a.few_sets, 128 / a.group};
  return launch_dependent(fa_paged_join_kernel<D>, dim3(ctas, 16), 128, 0, ctx.stream, p);
}

// ------------------------------------------------------------------ launch
template <int D, bool E4M3>
int launch_paged_chunk_impl(const PagedFwdArgs& a, const LaunchCtx& ctx) {
  using C = ChunkCfg<D, E4M3>;
  auto kernel = fa_paged_chunk_kernel<D, E4M3>;
  if constexpr (C::SPLIT_REGS) {
    // The register split is sized for exactly LAUNCH_REGS a thread (see launch_tc_impl).
    static std::atomic<int> checked_regs{-1};
    int regs = checked_regs.load(std::memory_order_relaxed);
    if (regs < 0) {
      cudaFuncAttributes attr;
      cudaError_t ea = cudaFuncGetAttributes(&attr, kernel);
      if (ea != cudaSuccess) return static_cast<int>(ea);
      regs = attr.numRegs;
      checked_regs.store(regs, std::memory_order_relaxed);
    }
    if (regs != C::LAUNCH_REGS) return -2;
  }
  static std::atomic<unsigned long long> allowed{0};
  const int e = allow_smem(kernel, C::SMEM_CHUNK, allowed);
  if (e != 0) return e;
  ChunkParams p;
  p.a = a;
  p.ws = paged_ws(a.workspace, D);
  p.status = ctx.status;
  p.limit_ns = ctx.limit_ns;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.tpt = 128 / a.group;
  p.box = (1 << a.kv.ps_log2) < C::BK ? 1 << a.kv.ps_log2 : C::BK;
  for (p.box_log2 = 4; (1 << p.box_log2) < p.box; ++p.box_log2) {
  }
  CUtensorMap mq, mk, mv, mo;
  const long long qdims[3] = {D, a.q_heads, a.pb.rows};
  const long long qst[2] = {a.qs[1], a.qs[0]};
  if (encode_paged_map(&mq, a.q, 2, qdims, qst, C::RC, a.group, p.tpt, C::SWB, false) != 0) return -1;
  p.tma_o = (a.group & (a.group - 1)) == 0;
  const int oh = a.group < 32 ? a.group : 32;
  const long long ost[2] = {a.os[1], a.os[0]};
  mo = mq;
  if (p.tma_o && encode_paged_map(&mo, a.o, 2, qdims, ost, 32, oh, 32 / oh, 64, false) != 0) return -1;
  const long long dims[4] = {D, 1LL << a.kv.ps_log2, a.kv.heads, a.kv.num_pages};
  const long long ks[3] = {a.kv.ks[2], a.kv.ks[1], a.kv.ks[0]}, vs[3] = {a.kv.vs[2], a.kv.vs[1], a.kv.vs[0]};
  // bf16: 64-column regions in the operand layout; e4m3: rows of codes, 128 columns at a time, unswizzled.
  const int cols = E4M3 ? C::CODE_COLS : C::RC, swizzle = E4M3 ? 0 : C::SWB;
  if (encode_paged_map(&mk, a.kv.k, E4M3 ? 1 : 2, dims, ks, cols, p.box, 1, swizzle, true) != 0) return -1;
  if (encode_paged_map(&mv, a.kv.v, E4M3 ? 1 : 2, dims, vs, cols, p.box, 1, swizzle, true) != 0) return -1;
  const int grid = ctx.num_sms < kPlanCtas ? ctx.num_sms : kPlanCtas;
  kernel<<<grid, C::THREADS, C::SMEM_CHUNK, ctx.stream>>>(mq, mk, mv, mo, p);
  return static_cast<int>(cudaGetLastError());
}

template <int D>
int launch_paged_chunk(const PagedFwdArgs& a, const LaunchCtx& ctx) {
  return a.e4m3 ? launch_paged_chunk_impl<D, true>(a, ctx) : launch_paged_chunk_impl<D, false>(a, ctx);
}

}  // namespace fa
