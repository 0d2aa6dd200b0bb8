// Attention of a batch's new tokens over a paged latent cache, on the
// 5th-generation tensor cores.
//
//   s[j] = scale * (q_lat . c_kv[j] + q_pe . k_pe[j]),  j visible to the token
//   o_lat = sum_j softmax_j(s) c_kv[j]
//
// Rows are (token, head) pairs; a block is 128 consecutive rows of one
// sequence, and its keys are walked in tiles of 64.  A CTA pair (a 2-CTA
// cluster) works on one block at a time:
//   * The 512-wide fp32 output of 128 rows fills a CTA's tensor memory, so the
//     pair splits the latent dimension: CTA r holds latent columns [256 r, +256)
//     and RoPE dimensions [32 r, +32) of queries and keys, and its 256 columns
//     of the output.  Each CTA's score product is thus a partial sum over half
//     the contraction, for all 128 rows.
//   * The partial scores are reduced between the CTAs by rows: CTA r owns rows
//     with (row / 16) % 2 == r.  Four sender warps pass the other CTA's 64 rows
//     on to it in fp32, 4 KB a warp and tile as one bulk copy (stored to its shared
//     memory 16 bytes a thread, they kept the SM's way out busy for 1000 of a
//     tile's 2200 cycles: chunks over 16-row pages took 268 us, then 255); softmax warps
//     add what arrives to their own half, so scores are full fp32 sums and each
//     row's softmax is computed once in the pair.  P (fp16) of the owned rows is
//     stored to both CTAs, with the factor by which the row's earlier output has
//     to shrink if its running maximum grew.  (Exchanging all partial scores in
//     fp16 and computing every softmax twice takes the same bytes on the wire,
//     twice the exponentials, and rounds the scores.)
//   * What bounds it: the shared memory, through which a tile moves 216 KB (its
//     load 36, operands of the products 92, partial scores 64, P 24), 1700 cycles
//     at 128 bytes a cycle of the 2050 that a tile takes; the tensor pipe is busy
//     for 1080, the way to the other CTA for 1330.  A tile stays in its stage from
//     its load to its P V, ~8500 cycles, so the four stages allow no less than 2100
//     either.  Eight warps share a tile's softmax (16 keys of a row per thread);
//     two sets of four that take the tiles in turn were 1-2% slower, and so were
//     16 warps.  512 queries of 128 heads at 33K rows: 3.61 ms, 1305 TFLOP/s, 68%
//     of the measured rate; 32 tokens at 4K to 32K rows: 156 us, 4.4 TB/s (one set of
//     pages again and again; new ones each time 3.67 ms and 166 us).
//   * O += P V on tcgen05, V read in place from the cache tile (N-major view).
//   * A piece's queries come through the ring of cache tiles too, as two stages
//     before its first tile, so that they are there when the piece before has
//     issued its last score product.  (Loaded by the sender warps themselves they
//     took 9-11k cycles a piece.)
//   * fp16 pages come in by TMA as they are, and so do the RoPE parts of e4m3
//     pages; their codes come into the second half of the tile's stage, where
//     producer warps turn them into the fp16 tile (code x scale, exact).  (With a
//     ring of their own for the codes there is room for three stages: 3% slower.)
//     A sequence whose chunk has several blocks would have its codes converted once
//     per block: its visible rows are converted once, before, into the workspace,
//     and the kernel for fp16 pages takes it, the e4m3 kernel the other sequences.
// Work split: a block costs its tiles plus `kPieceCost`; the costs of all
// blocks form one run, which the clusters share evenly.  A cluster's piece that
// is a whole block writes o_lat; a block cut by a cluster boundary leaves fp32
// partials (at most two per cluster) that paged_combine_kernel merges.
// Every wait on an mbarrier is bounded; a warp that gave one up still comes to the
// named barriers, and its CTA leaves when what it had under way has ended.
#include <string.h>

#include <atomic>

#include "kernels.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kRows = 128;                   // query rows of a block (MMA M)
constexpr int kBK = 64;                      // keys per tile
constexpr int kOwn = kRows / 2;              // rows whose softmax a CTA computes
// A tile of latents lies in groups of eight keys, a group in chunks of 64 dims:
// 128-byte rows, evenly spaced groups, and the part of a tile that lies in one page
// (16 rows at least) is one block, so that one load brings it whatever the page's size.
constexpr int kChunk = 8 * 128;              // 1 KB: 8 keys x 64 fp16
constexpr int kGroup = 4 * kChunk;           // 4 KB: 8 keys x this CTA's 256 latent dims
constexpr int kLatStage = kBK / 8 * kGroup;  // 32 KB
constexpr int kLatStages = 4;                // tile stages
// e4m3: a tile's codes (64 keys x 256, this CTA's half) arrive in the second half of
// its stage, their rows' 16 scale bytes beside it.
constexpr int kRawOff = kLatStage / 2, kRawScale = kBK * 16, kRawBytes = kBK * 256 + kRawScale;
constexpr int kRopeStages = 2;               // a RoPE tile is done with after its score product
constexpr int kRopeHalf = 32;
constexpr int kRopeChunk = kBK * kRopeHalf * 2;     // 4 KB
constexpr int kQRopeBytes = kRows * kRopeHalf * 2;  // 8 KB
constexpr int kPBytes = kRows * 128;         // 16 KB: two halves of 128 rows x 32 keys fp16
constexpr int kXBytes = kOwn * kBK * 4;      // 16 KB: 64 rows x 64 keys fp32
constexpr int kPTx = kOwn * kBK * 2 + kOwn * 4;     // bytes a CTA gets per tile: the other's P rows and factors
constexpr int kOffLat = kQRopeBytes;
constexpr int kOffScale = kOffLat + kLatStages * kLatStage;  // (e4m3)
constexpr int kOffRope = kOffScale + kLatStages * kRawScale;
constexpr int kOffP = kOffRope + kRopeStages * kRopeChunk;
constexpr int kOffX = kOffP + 2 * kPBytes;
constexpr int kOffXs = kOffX + kXBytes;              // what goes to the other CTA
constexpr int kOffStg = kOffXs + kXBytes;            // epilogue staging, 2 KB per warp
constexpr int kOffAlpha = kOffStg + 4 * 2048;        // [2][128] output factors
constexpr int kOffL = kOffAlpha + 2 * kRows * 4;     // [4][128] row sums
constexpr int kOffM = kOffL + 4 * kRows * 4;         // [2][2][64] row maxima of the key halves, by tile parity
constexpr int kOffBar = kOffM + 2 * 2 * kOwn * 4;
constexpr int kBarBytes = 512;
constexpr int kSmem = 1024 + kOffBar + kBarBytes;
static_assert(kSmem <= 232448, "shared memory");

// Warp roles: softmax 0-3 (keys 0-31 of a tile) and 4-7 (keys 32-63), senders
// (and Q loads) 8-11, output 12-15, score MMAs 16, P V MMAs 17, TMA loads 18, and
// for e4m3 pages the producers 19-22.
constexpr int kSendWarp = 8, kOutWarp = 12, kQkWarp = 16, kPvWarp = 17, kLoadWarp = 18, kProdWarp = 19;
constexpr int kBarMax = 1;                   // + q, named: the row maxima (sums) of warps q and q + 4 are in sM
constexpr int kBarProd = 5;                  // the producers
constexpr int kProducerWarps = 4;
__host__ __device__ constexpr int threads(bool e4m3) { return 32 * (kProdWarp + (e4m3 ? kProducerWarps : 0)); }
// 19 warps: 5 per sub-partition, 96 registers a thread; 23 warps: 6, 80.
__host__ __device__ constexpr int max_regs(bool e4m3) { return e4m3 ? 80 : 96; }

constexpr uint32_t kTmQ = 0, kTmS = 128, kTmO = 256;   // TMEM columns: Q 128, two score buffers of 64, O 256
// P in fp16 is exp2(score - m + kPShift), m the running maximum, which lags behind the
// largest score by at most kRescaleThreshold: P stays <= 2^15.  The factor is in the row
// sums and the partials' weights too, and cancels.  A probability keeps fp16's 11 bits
// down to 2^-21 of the largest and counts down to 2^-32 of it (without the shift 2^-14
// and 2^-25: of 98304 rows, all 16 below one key in score, 6% were lost).
constexpr float kRescaleThreshold = 8.0f;    // log2 units
constexpr float kPShift = 7.0f;

// What the P V warp asks of the output warps, besides a rescale of O (tile >= 0).  A
// piece may be millions of tiles long and never need one, so the limit of their wait
// grows by kTileUs with every tile of the cluster (one takes ~1.1 us).  (A request for
// nothing every 4096 tiles instead made the P V warp's loop 0.5% slower.)
constexpr int kCmdOutput = -1, kCmdStop = -2;
// A request kCmdMove - u moves what O holds before tile u's P V to the piece's partial in
// the workspace; O starts anew.  The tensor cores' fp32 sums are not rounded but cut
// off: with every 16 keys O loses 2^-24 of itself on average, and over a million rows
// 0.65% were missing.  Every kMoveTiles tiles (65536 rows, 2.4e-4) O is therefore added
// to the partial, rounded to nearest: 152 tokens at a million rows 33.4 -> 34.1 ms.  Its
// code makes shorter calls 1% slower (32 tokens 156.6 -> 158.2 us), so it is an
// instantiation of its own (kLong), for calls in which a block can have as many tiles.
constexpr int kCmdMove = -3, kMoveTiles = 1024;
constexpr int64_t kTileUs = 16;
constexpr uint64_t kGaveUpNs = 200000;       // from a wait that ran out to the CTA's end

constexpr int kPieceCost = 3;                // start-up of a piece (5-6k cycles) in tiles
constexpr float kCutCost = 4.f;              // of a share (see there)

// Ring stages that a piece's queries take before its first tile.  Tile u (counted
// over all pieces) of piece k has ring position u + (k + 1) kQSlots.
constexpr int kQSlots = 2;

struct __align__(16) Rec {     // the block that starts in cluster c and ends in a later one
  int64_t end;        // where it ends in the run of costs
  int64_t total;      // the run's length
  int64_t qrow0;      // its first (token, head) row
  int32_t nvalid;     // its rows (0: no such block)
  int32_t share;      // of every cluster; 0: all have total / G
  // Clusters whose range starts before `end`.  No more than there are: with a cu that
  // decreases, the cluster's walk and the total may disagree on the blocks, and `end`
  // lie behind the total.
  MLA_DEVINL int clusters(int G) const {
    int64_t n;
    if (share > 0) n = (static_cast<uint32_t>(end) + share - 1) / share;
    else if (total < (1 << 24))
      n = (static_cast<uint32_t>(end) * G + static_cast<uint32_t>(total) - 1) / static_cast<uint32_t>(total);
    else n = (end * G + total - 1) / total;
    return static_cast<int>(min(n, static_cast<int64_t>(G)));
  }
};

// Staging of e4m3 latents as fp16 (rows of 512): up to kStageRows rows of the
// sequences with at least kStageBlocks blocks, in batches of at most kStageSeqs.
// Measured with and without, one sequence of 128 heads (a query is a block) at 33K
// rows: 8 queries 93 and 86 us, 12 121 and 121, 16 150 and 156, 152 1071 and 1333;
// the staging and a second launch cost ~10 us, so at 2000 rows 16 queries take 37 and
// 28 us, 64 66 and 60, 256 153 and 164.
constexpr int kStageRows = 131072, kStageSeqs = 1024, kStageBlocks = 16;

// Which sequences a launch takes.
enum Take : int32_t { kTakeAll, kTakeStaged, kTakeUnstaged };

struct TcArgs {
  PagedAttnArgs p;
  Take take;
  float* ws_o;        // fp32 [2 G][128][512] partials, normalised by their own sums
  float* ws_ml;       // fp32 [2 G][128][2] running maximum (log2 units, less kPShift) and sum
  Rec* rec;           // [G]
  int32_t* stage_base;   // [B] a sequence's first staged row, -1: not staged (unless take is kTakeAll)
  uint16_t* stage;       // fp16 [kStageRows][512]
  int32_t n_slots;
  int32_t n_rows;     // rows of the page pool
};

// ---------------------------------------------------------------------------
// Blocks.  Sequence b's blocks get slots cu[b] H / 128 + b, ...: these ranges
// do not overlap (the sum of ceil(n H / 128) over earlier sequences is at most
// floor(cu[b] H / 128) + b), so a slot's sequence is found by a search in cu
// alone, with no prefix sums over the batch.  Slots without a block cost 0.
// ---------------------------------------------------------------------------
MLA_DEVINL int64_t slot_of_seq(const PagedAttnArgs& a, int b) {
  const int32_t c = max(0, min(a.T, __ldg(a.cu + b)));
  return static_cast<int64_t>(c) * a.H / kRows + b;
}

struct Item {
  int32_t b;                  // sequence
  int32_t kend, wlo;          // keys some row of the block sees: [0, n_sink) and [wlo, kend)
  int32_t first, sink_tiles;  // tile t of the block is t < sink_tiles ? t : first + t - sink_tiles
  int32_t t_lo, n_tiles;      // this piece: tiles [t_lo, t_lo + n_tiles)
  int32_t nvalid;             // rows
  int32_t pos0;               // position of the sequence's first new token
  uint32_t row0;              // first row within the sequence's new rows
  int64_t qrow0;              // first row in the token array
  bool open;                  // the block goes on past this piece
  bool once;                  // the sequence has one or two blocks
  MLA_DEVINL bool whole() const { return t_lo == 0 && !open; }
  // The piece in [lo, hi) of the run of costs, in which the block's n tiles start at r0.
  MLA_DEVINL bool cut(int64_t lo, int64_t hi, int64_t r0, int n) {
    const int64_t p_lo = max(lo, r0), p_hi = min(hi, r0 + n);
    if (p_lo >= p_hi) return false;
    t_lo = static_cast<int32_t>(p_lo - r0);
    n_tiles = static_cast<int32_t>(p_hi - p_lo);
    open = p_hi < r0 + n;
    return true;
  }
  MLA_DEVINL int key_tile(int t) const {
    const int x = t_lo + t;
    return x < sink_tiles ? x : first + x - sink_tiles;
  }
};

// Walks the slots in order.
struct Walker {
  int b;                // sequence of the last slot asked for
  int64_t s0, s1;       // its first slot, and the next sequence's
  PagedSeq seq;
  uint32_t rows;        // seq.n * H

  MLA_DEVINL void load(const TcArgs& t) {
    const PagedAttnArgs& a = t.p;
    s0 = slot_of_seq(a, b);
    s1 = b + 1 < a.B ? slot_of_seq(a, b + 1) : INT64_MAX;
    bool bad;
    seq = paged_seq(a.cu, a.seq_len, b, a.T, a.c.max_rows(), bad);
    rows = static_cast<uint32_t>(seq.n) * static_cast<uint32_t>(a.H);
    if (t.take != kTakeAll && (__ldg(t.stage_base + b) >= 0) != (t.take == kTakeStaged)) rows = 0;
  }
  MLA_DEVINL void init(const TcArgs& t, int64_t g) {
    const PagedAttnArgs& a = t.p;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (slot_of_seq(a, m) <= g) lo = m; else hi = m;
    }
    b = lo;
    load(t);
  }
  // Tiles of slot g's block (0: no block); g must not decrease between calls.
  MLA_DEVINL int block(const TcArgs& t, int64_t g, Item& it) {
    const PagedAttnArgs& a = t.p;
    while (g >= s1) {
      ++b;
      load(t);
    }
    const int64_t i = g - s0;
    if (i < 0 || i * kRows >= rows) return 0;
    const uint32_t H = static_cast<uint32_t>(a.H), r0 = static_cast<uint32_t>(i) * kRows;
    const uint32_t r1 = min(r0 + kRows, rows);
    it.b = b;
    it.nvalid = static_cast<int32_t>(r1 - r0);
    it.once = rows <= 2 * kRows;
    it.row0 = r0;
    it.qrow0 = static_cast<int64_t>(seq.q0) * a.H + r0;
    it.pos0 = seq.len - seq.n;
    it.kend = it.pos0 + static_cast<int32_t>((r1 - 1) / H) + 1;
    it.wlo = a.window > 0 ? max(0, it.pos0 + static_cast<int32_t>(r0 / H) - a.window + 1) : 0;
    it.first = it.wlo / kBK;
    it.sink_tiles = min((min(a.n_sink, it.wlo) + kBK - 1) / kBK, it.first);
    return it.sink_tiles + (it.kend + kBK - 1) / kBK - it.first;
  }
};

struct Start {
  int64_t lo, hi;     // the cluster's range in the run of costs
  int64_t S;          // where slot g's cost starts in it (ends, if it has the first piece)
  int32_t g;          // first slot that ends after lo (n_slots: none)
  int32_t b;          // and its sequence
  int32_t share;      // of every cluster (the last one's may be less); 0: all have total / G
  int64_t total;
  Item it;            // the cluster's first piece, in slot g (n_tiles 0: none there)
};

// This cluster's pieces in order; every role walks the same sequence.
struct Iter {
  Walker w;
  const Start* st;
  int64_t lo, hi, S;
  int32_t g;
  bool first;                  // the next piece is st->it
  MLA_DEVINL void init(const Start& start) {
    st = &start;
    lo = start.lo;
    hi = start.hi;
    S = start.S;
    g = start.g;
    w.b = start.b - 1;         // loaded by the first block asked for
    w.s1 = -1;
    first = start.it.n_tiles > 0;
    if (first) ++g;
  }
  MLA_DEVINL bool next(const TcArgs& a, Item& it) {
    if (first) {
      first = false;
      it = st->it;
      return true;
    }
    while (g < a.n_slots && S < hi) {
      const int n = w.block(a, g++, it);
      if (n == 0) continue;
      const int64_t r0 = S + kPieceCost;
      S = r0 + n;
      if (it.cut(lo, hi, r0, n)) return true;
    }
    return false;
  }
};

// Keys [k, k + n) hold one that some row of the block sees.
MLA_DEVINL bool any_visible(const TcArgs& a, const Item& it, int k, int n) {
  return k < it.kend && (k + n > it.wlo || k < a.p.n_sink);
}
MLA_DEVINL bool key_visible(const TcArgs& a, const Item& it, int k) {
  return k < it.kend && (k >= it.wlo || k < a.p.n_sink);
}

// Staging takes whole tiles of the keys that some new token of the sequence
// sees (the first token's window starts lowest).  Staged row of key tile kt,
// given the sequence's first staged row.
MLA_DEVINL int32_t seq_first_tile(const PagedAttnArgs& a, int32_t pos0, int32_t& sink_tiles) {
  const int32_t wlo = a.window > 0 ? max(0, pos0 - a.window + 1) : 0;
  const int32_t first = wlo / kBK;
  sink_tiles = min((min(a.n_sink, wlo) + kBK - 1) / kBK, first);
  return first;
}
MLA_DEVINL int32_t staged_row(const TcArgs& a, const Item& it, int32_t base, int kt) {
  int32_t sink;
  const int32_t first = seq_first_tile(a.p, it.pos0, sink);
  return base + kBK * (kt < sink ? kt : kt - first + sink);
}

// Barriers (u counts this cluster's tiles, k its pieces).
struct Bars {
  uint64_t lat_full[4];             // tile in its stage
  uint64_t lat_empty[4];            // P V has read it (or the senders, queries; e4m3: and the producers saw them)
  uint64_t raw_full[4];             // e4m3: its codes and scales (or queries)
  uint64_t rope_full[kRopeStages];
  uint64_t rope_empty[kRopeStages];
  uint64_t s_full[2];               // partial scores in TMEM
  uint64_t s_free[2];               // both the softmax and the sender warps have read them
  uint64_t x_full[4];               // the other CTA's partials of warp q's 16 owned rows have arrived
  uint64_t x_empty[4];              // the other CTA has read what this one's sender warp q sent
  uint64_t p_full[2];               // P and factors of all 128 rows
  uint64_t pv_done[2];              // P V done in both CTAs: P buffer, factors and O of that tile
  uint64_t q_ready;                 // piece k's queries in TMEM and shared memory
  uint64_t o_ready;                 // piece k's last P V done
  uint64_t l_full[4];               // piece k's row sums (slot k % 4)
  uint64_t cmd_full, cmd_done;      // the P V warp's requests to the output warps
  uint32_t tmem;
  int32_t cmd;                      // kCmd.. (kCmdMove - u), or a tile u: rescale O by its factors
  Start st;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

MLA_DEVINL bool wait_all(uint64_t* bar, uint32_t parity, const TcArgs& a) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.p.wait_us, a.p.err));
}
MLA_DEVINL bool wait_cl(uint64_t* bar, uint32_t parity, const TcArgs& a) {
  return __all_sync(0xffffffffu, tc::mbar_wait_cluster_bounded(bar, parity, a.p.wait_us, a.p.err));
}

// 16-byte unit u (8 halves) of a row in a 128-byte-swizzled K-major tile, and
// in a 64-byte-swizzled one (rows of 32 halves).
MLA_DEVINL uint32_t unit128(int row, int u) { return static_cast<uint32_t>(row * 128 + ((u ^ (row & 7)) << 4)); }
MLA_DEVINL uint32_t unit64(int row, int u) { return static_cast<uint32_t>(row * 64 + ((u ^ ((row >> 1) & 3)) << 4)); }

// Sum of 0 <= x < 2^52 over the warp: two reductions of 26 bits.
MLA_DEVINL long long warp_sum_wide(long long x) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x) & 0x3FFFFFFu);
  const uint32_t hi = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 26));
  return (static_cast<long long>(hi) << 26) + lo;
}

MLA_DEVINL void st_async_b32(uint32_t remote_addr, uint32_t v, uint32_t remote_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(remote_addr), "r"(v),
               "r"(remote_bar)
               : "memory");
}

MLA_DEVINL void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// `bytes` of this CTA's shared memory to the peer's, counted on its barrier.
MLA_DEVINL void bulk_to_peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// 16 TMEM lanes, 16 columns per thread: threads 0-15 at columns [c, c + 16),
// threads 16-31 the same lanes at [c + 16, c + 32).
MLA_DEVINL void tmem_ld16x2_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 16;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Arrive on `bar` of both CTAs of the pair when every MMA issued so far has
// completed.  Whole warp; one lane issues.
MLA_DEVINL void mma_commit_pair_warp(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Two fp32 in one register pair: packed adds and multiply-adds are one
// instruction, and three-input maxima save a third (the softmax is bound by its
// instruction stream).
MLA_DEVINL uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
MLA_DEVINL float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
MLA_DEVINL uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
MLA_DEVINL uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// a and b plus the halves of w (fp16), added in fp32.
MLA_DEVINL void add_f16x2(float& a, float& b, uint32_t w) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %1, h, %1;\n\t}"
      : "+f"(a), "+f"(b) : "r"(w));
}
MLA_DEVINL float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 64 bytes of each of a warp's 32 rows (lane = row) to dst_row0 + row * stride,
// through the warp's 2 KB staging slice, so that each store instruction writes
// 8 rows x 64 contiguous bytes.  Rows >= nrows are not stored.
MLA_DEVINL void store_rows(uint8_t* stg, int lane, const uint4 (&w)[4], uint8_t* dst_row0, int64_t stride, int nrows) {
#pragma unroll
  for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4*>(stg + unit64(lane, v)) = w[v];
  __syncwarp();
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int rr = (lane >> 2) + 8 * m, part = lane & 3;
    const uint4 x = *reinterpret_cast<const uint4*>(stg + unit64(rr, part));
    if (rr < nrows) *reinterpret_cast<uint4*>(dst_row0 + rr * stride + part * 16) = x;
  }
  __syncwarp();
}

// 32 rows (lane = row) x 256 columns of O, plus g times what `part` holds of them (`add`),
// times f: as fp32 to `part`, or as fp16 to `out`.
__device__ __noinline__ void move_o(uint32_t taddr, uint8_t* stg, uint8_t* part, int nrows, bool add, float g, float f,
                                    uint8_t* out) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int cc = 0; cc < 16; ++cc) {
    uint32_t r[16];
    tc::tmem_ld16(taddr + 16 * cc, r);
    tc::tmem_ld_wait();
    float o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(r[e]);
    if (add && lane < nrows) {
      const float4* p = reinterpret_cast<const float4*>(part + lane * (kLatent * 4) + cc * 64);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float4 x = p[v];
        o[4 * v] = fmaf(x.x, g, o[4 * v]);
        o[4 * v + 1] = fmaf(x.y, g, o[4 * v + 1]);
        o[4 * v + 2] = fmaf(x.z, g, o[4 * v + 2]);
        o[4 * v + 3] = fmaf(x.w, g, o[4 * v + 3]);
      }
    }
    __syncwarp();
    if (out != nullptr) {
      if (lane < nrows) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = pack_f16x2(o[2 * e] * f, o[2 * e + 1] * f);
        uint4* q = reinterpret_cast<uint4*>(out + lane * (kLatent * 2) + cc * 32);
        q[0] = make_uint4(h[0], h[1], h[2], h[3]);
        q[1] = make_uint4(h[4], h[5], h[6], h[7]);
      }
    } else {
      uint4 w[4];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        w[v] = make_uint4(__float_as_uint(o[4 * v] * f), __float_as_uint(o[4 * v + 1] * f),
                          __float_as_uint(o[4 * v + 2] * f), __float_as_uint(o[4 * v + 3] * f));
      store_rows(stg, lane, w, part + cc * 64, kLatent * 4, nrows);
    }
  }
}

MLA_DEVINL uint4 bf16x8_to_f16x8(uint4 v) {
  uint4 o;
  float2 f;
  f = bf16x2_to_f32(v.x); o.x = pack_f16x2(f.x, f.y);
  f = bf16x2_to_f32(v.y); o.y = pack_f16x2(f.x, f.y);
  f = bf16x2_to_f32(v.z); o.z = pack_f16x2(f.x, f.y);
  f = bf16x2_to_f32(v.w); o.w = pack_f16x2(f.x, f.y);
  return o;
}

// ---------------------------------------------------------------------------
// e4m3 producer: this CTA's 256 codes of a tile's 64 rows into fp16, in place: the
// codes lie in the second half of the tile's stage.  Step j of thread pt (of 128)
// takes 16 codes each at 16 c0 + 128 h, h < 2, of key k0 + 16 j; all offsets are
// constants of the thread.  Steps 2 and 3 overwrite codes: those of steps 0 and 1,
// and of 2 and 3.  Eight consecutive lanes take half of the units of two adjacent
// keys, the one's lower and the other's upper half: their loads and stores then lie
// in eight different 16-byte columns of the banks (one key's eight units, whose
// stores meet in four, took 3% longer).  Four warps, a step at a time: eight warps, or
// codes loaded a step ahead, make the hot code larger and the kernel 2-6% slower.
// 8 tokens at 98304 rows: 225 us.
// ---------------------------------------------------------------------------
constexpr int kProdKeys = 4 * kProducerWarps;
static_assert(kBK / kProdKeys == 4, "steps");

MLA_DEVINL int prod_key(int pt) { return 2 * (pt >> 4) + ((pt >> 2) & 1); }
MLA_DEVINL int prod_unit(int pt) { return (pt & 3) | (((pt >> 2) ^ (pt >> 3)) & 1) << 2; }

struct Codes {
  uint4 v[2];
  uint2 d;                                     // the key's scale bytes of this CTA
};
MLA_DEVINL void load_codes(Codes& c, const uint8_t* lat, const uint8_t* scale, int rank, int pt, int j) {
  const int key = prod_key(pt) + kProdKeys * j;
  const uint8_t* src = lat + kRawOff + key * 256 + 16 * prod_unit(pt);
  c.v[0] = *reinterpret_cast<const uint4*>(src);
  c.v[1] = *reinterpret_cast<const uint4*>(src + 128);
  c.d = *reinterpret_cast<const uint2*>(scale + key * 16 + 8 * rank);
}
MLA_DEVINL void store_f16(const Codes& c, uint8_t* lat, int pt, int j) {
  const int k0 = prod_key(pt), c0 = prod_unit(pt);
  const uint32_t dst = (k0 >> 3) * kGroup + (c0 >> 2) * kChunk + unit128(k0 & 7, 2 * (c0 & 3));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t s = e4m3_scale_f16x2(__byte_perm(h ? c.d.y : c.d.x, 0u, 0x4440 + (c0 >> 1)));
    uint4 lo, hi;
    e4m3x4_to_f16x4(c.v[h].x, s, lo.x, lo.y);
    e4m3x4_to_f16x4(c.v[h].y, s, lo.z, lo.w);
    e4m3x4_to_f16x4(c.v[h].z, s, hi.x, hi.y);
    e4m3x4_to_f16x4(c.v[h].w, s, hi.z, hi.w);
    uint8_t* q = lat + 2 * kChunk * h + kProdKeys / 8 * kGroup * j;
    *reinterpret_cast<uint4*>(q + dst) = lo;
    *reinterpret_cast<uint4*>(q + (dst ^ 16u)) = hi;
  }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
// kFewRows: blocks of fewer rows than 128, as single tokens of few heads are: warps
// whose rows all lie behind a block's do no softmax, and their scores stay where they
// are (32 tokens at 4K-32K rows, 16 heads: 138 us, without it 147; 64 heads 143 and
// 149, 96 heads 149 and 152).  Its own instantiation, because the tests make full
// blocks 2% slower; for e4m3 pages it gains nothing.
template <bool kE4m3, bool kFewRows, bool kLong>
__global__ void __cluster_dims__(2, 1, 1) __maxnreg__(max_regs(kE4m3))
    paged_attn_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope,
                      const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_scale,
                      const __grid_constant__ TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQr = sm;
  uint8_t* sLat = sm + kOffLat;
  uint8_t* sScale = sm + kOffScale;
  uint8_t* sRope = sm + kOffRope;
  uint8_t* sP = sm + kOffP;
  uint8_t* sX = sm + kOffX;
  uint8_t* sXs = sm + kOffXs;
  uint8_t* sStg = sm + kOffStg;
  float* sAlpha = reinterpret_cast<float*>(sm + kOffAlpha);
  float* sL = reinterpret_cast<float*>(sm + kOffL);
  float* sM = reinterpret_cast<float*>(sm + kOffM);
  Bars& B = *reinterpret_cast<Bars*>(sm + kOffBar);

  const uint32_t rank = tc::cluster_ctarank(), peer = rank ^ 1u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = static_cast<int>(blockIdx.x >> 1), G = static_cast<int>(gridDim.x >> 1);
  constexpr int NT = threads(kE4m3);

  // ---- setup ---------------------------------------------------------------
  if (warp == kPvWarp) {
    // a lane per barrier: how many arrivals complete a phase
    auto init = [&](int l, uint64_t* bars, int n, uint32_t count) {
      if (lane >= l && lane < l + n) mbar_init(bars + lane - l, count);
    };
    static_assert(kLatStages == 4 && kRopeStages == 2, "lanes below");
    init(0, B.raw_full, 4, 1);
    init(0, B.lat_full, 4, kE4m3 ? kProducerWarps : 1);
    init(4, B.lat_empty, 4, 1);
    init(8, B.rope_full, 2, 1);
    init(10, B.rope_empty, 2, 1);
    init(12, B.s_full, 2, 1);
    init(14, B.s_free, 2, 12);
    init(16, B.x_full, 4, 1);
    init(16, B.x_empty, 4, 1);
    init(20, B.p_full, 2, 9);
    init(22, B.pv_done, 2, 2);
    init(24, &B.q_ready, 1, 4);
    init(25, &B.o_ready, 1, 1);
    init(26, B.l_full, 4, 5);
    init(30, &B.cmd_full, 1, 1);
    init(31, &B.cmd_done, 1, 4);
    tc::fence_mbar_init();
    // what the peer sends for the first use of each buffer
    if (lane >= 16 && lane < 20) mbar_arrive_expect_tx(&B.x_full[lane - 16], kXBytes / 4);
    if (lane >= 20 && lane < 22) mbar_arrive_expect_tx(&B.p_full[lane - 20], kPTx);
    if (lane >= 26 && lane < 30) mbar_arrive_expect_tx(&B.l_full[lane - 26], kOwn * 4);
  }
  if (threadIdx.x == 0) {
    B.st.g = a.n_slots;
    B.st.lo = B.st.hi = B.st.S = 0;
    B.st.b = 0;
    B.st.it.n_tiles = 0;
  }
  if (warp == kQkWarp) {
    tc::tmem_alloc(&B.tmem, 512);
    tc::tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    tc::prefetch_tmap(&tm_lat);
    tc::prefetch_tmap(&tm_rope);
    tc::prefetch_tmap(&tm_q);
    if (kE4m3) tc::prefetch_tmap(&tm_scale);
  }
  // The peer's barriers are ready once its threads have come here: waited for below.
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  // All above may run while the kernel before finishes (programmatic launch).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.p.cu, a.p.seq_len, a.p.B, a.p.T, a.p.c.max_rows(), a.p.err);
  {
    // The run of all blocks' costs: each thread sums a share of the slots (one
    // slot, as a rule), a scan over the block gives its start, and the thread
    // whose share holds this cluster's first unit finds the slot.
    long long* red = reinterpret_cast<long long*>(sStg);
    const int per = (a.n_slots + NT - 1) / NT;
    const int g0 = min(a.n_slots, static_cast<int>(threadIdx.x) * per), g1 = min(a.n_slots, g0 + per);
    Walker w;
    Item it;
    long long sum = 0;
    if (g0 < g1) {
      w.init(a, g0);
      int g = g0;
      do {
        const int n = w.block(a, g, it);
        sum += n > 0 ? n + kPieceCost : 0;
      } while (++g < g1);
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    const long long part = lane < NT / 32 ? red[lane] : 0;
    const long long total = warp_sum_wide(part), before = warp_sum_wide(lane < warp ? part : 0);
    const long long S0 = before + incl - sum;
    // Cluster x of G takes [total x / G, total (x + 1) / G).  Short work takes fewer
    // clusters, with an equal share each: a shorter piece saves its tiles' time, another
    // piece of the block costs the merge.  The sum is least near share = sqrt(cost of a
    // block / kCutCost); blocks of up to two tiles are not cut.  (One token at 257 rows,
    // 16 heads, shares of 1, 2, 3, 8: 12.5, 12.8, 13.2, 14.3 us; 128 heads at 4000 rows
    // 26.6, 20.4, 19.1, 22.2, the rule 19.8; at 16000 shares of 3.3 and 8 31.5 and 26.5.)
    long long lo, hi;
    uint32_t share = 0;
    if (total < (1 << 24)) {
      const uint32_t units = static_cast<uint32_t>(total);
      const float blocks =                                        // about
          fmaxf(static_cast<float>(a.p.B), static_cast<float>(a.p.T) * a.p.H * (1.f / kRows));
      share = kPieceCost + 2;
      if (units > blocks * share) {
        const float x = __fdividef(static_cast<float>(units), blocks * kCutCost);
        share = max(1u, static_cast<uint32_t>(x * rsqrtf(x) + 0.5f));
      }
      if (units <= static_cast<uint32_t>(G) * share) {
        lo = min(units, static_cast<uint32_t>(c) * share);
        hi = min(units, static_cast<uint32_t>(c + 1) * share);
      } else {                           // (32-bit divisions: the 64-bit ones are slow code, run once)
        share = 0;
        lo = units * static_cast<uint32_t>(c) / static_cast<uint32_t>(G);
        hi = units * static_cast<uint32_t>(c + 1) / static_cast<uint32_t>(G);
      }
    } else {
      lo = total * c / G;
      hi = total * (c + 1) / G;
    }
    if (lo < hi && sum > 0 && S0 <= lo && lo < S0 + sum) {
      long long S = S0;
      int g = g0, n = static_cast<int>(sum) - kPieceCost;
      if (per > 1) {                     // else `it` and n are the slot's
        w.init(a, g0);
        for (; g < g1; ++g) {
          n = w.block(a, g, it);
          const long long e = S + (n > 0 ? n + kPieceCost : 0);
          if (lo < e) break;
          S = e;
        }
      }
      const bool piece = it.cut(lo, hi, S + kPieceCost, n);
      B.st.share = static_cast<int32_t>(share);
      B.st.total = total;
      B.st.lo = lo;
      B.st.hi = hi;
      B.st.S = piece ? S + kPieceCost + n : S;
      B.st.g = g;
      B.st.b = w.b;
      if (piece) B.st.it = it;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  tc::fence_after_sync();
  const uint32_t tmem = B.tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Iter items;
  items.init(B.st);
  Item it;
  bool ok = true;

  if (warp < kSendWarp) {
    // ================================ softmax ==================================
    // Four threads per owned row: warps q and q + 4, lanes l and l + 16, 16 keys
    // of every tile each.  A warp whose 16 rows all lie behind the block's (kFewRows)
    // leaves their P as it is: no output takes it.  A wait that gave up makes the warp `dead`: it goes on
    // through the tiles with nothing but the named barriers, on which its partner
    // waits without a limit.
    const int half = warp >> 2, q4 = warp & 3, hh = lane >> 4;
    const int lrow = 16 * q4 + (lane & 15);                                      // among the owned rows
    const int i = 32 * q4 + 16 * static_cast<int>(rank) + (lane & 15);           // row = TMEM lane
    const int col = 32 * half + 16 * hh;                                         // first key of this thread
    const uint32_t lanes = static_cast<uint32_t>(32 * q4 + 16 * rank) << 16;
    const float c2 = a.p.scale_log2;
    const uint32_t peer_p = tc::mapa(smem_u32(sP), peer), peer_pfull = tc::mapa(smem_u32(&B.p_full[0]), peer);
    const uint32_t peer_alpha = tc::mapa(smem_u32(sAlpha), peer), peer_l = tc::mapa(smem_u32(sL), peer);
    const uint32_t peer_lfull = tc::mapa(smem_u32(&B.l_full[0]), peer);
    const uint32_t peer_xempty = tc::mapa(smem_u32(&B.x_empty[q4]), peer);
    bool dead = false;
    int u = 0, k = 0, xu = 0;          // tiles, pieces, tiles of pieces in which some row is this warp's
#pragma unroll 1
    while (items.next(a, it)) {
      const bool rvalid = i < it.nvalid;
      const bool mine = !kFewRows || 32 * q4 + 16 * static_cast<int>(rank) < it.nvalid;
      // keys [wl, lim] and the sinks are visible to this row
      const int lim = rvalid ? it.pos0 + static_cast<int>((it.row0 + i) / static_cast<uint32_t>(a.p.H)) : it.kend - 1;
      const int wl = a.p.window > 0 ? max(0, lim - a.p.window + 1) : 0;
      float m_run = -INFINITY, l_h = 0.f;      // the running maximum, less kPShift; the sum
#pragma unroll 1
      for (int t = 0; t < it.n_tiles; ++t, ++u) {
        const int sb = u & 1;
        const uint32_t ph = (u >> 1) & 1, xph = (kFewRows ? xu : u) & 1;
        const int base = it.key_tile(t) * kBK, k0 = base + col;
        uint64_t s[8];                           // the scores, in pairs
        float mrow = -INFINITY;
        // Barriers are tested ahead of their use, so that their latencies
        // overlap; one that is not complete yet is waited for there.
        const bool s_test = mbar_test(&B.s_full[sb], ph), x_test = tc::mbar_test_cluster(&B.x_full[q4], xph);
        if (!dead && !__all_sync(0xffffffffu, s_test)) dead = !wait_all(&B.s_full[sb], ph, a);
        if (!dead && !mine && lane == 0) mbar_arrive(&B.s_free[sb]);
        if (!dead && mine) {
          tc::fence_after_sync();
          uint32_t r[16];
          tmem_ld16x2_16(tmem + lanes + kTmS + sb * 64 + 32 * half, r);
          tc::tmem_ld_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.s_free[sb]);
          if (!__all_sync(0xffffffffu, x_test)) dead = !wait_cl(&B.x_full[q4], xph, a);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = pack2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
        }
        if (!dead && mine) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const ulonglong2 x =
                *reinterpret_cast<const ulonglong2*>(sX + q4 * (kXBytes / 4) + (col / 4 + g) * 256 + (lane & 15) * 16);
            s[2 * g] = add2(s[2 * g], x.x);
            s[2 * g + 1] = add2(s[2 * g + 1], x.y);
          }
          if (k0 + 15 > lim || (k0 < wl && k0 + 15 >= a.p.n_sink)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float2 v = unpack2(s[e]);
              const int k = k0 + 2 * e;
              if (k > lim || (k < wl && k >= a.p.n_sink)) v.x = -INFINITY;
              if (k + 1 > lim || (k + 1 < wl && k + 1 >= a.p.n_sink)) v.y = -INFINITY;
              s[e] = pack2(v.x, v.y);
            }
          }
          float mx = -INFINITY, my = -INFINITY;
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 v = unpack2(s[e]), w = unpack2(s[e + 1]);
            mx = max3(mx, v.x, v.y);
            my = max3(my, w.x, w.y);
          }
          const float mown = fmaxf(mx, my) * c2;
          mrow = fmaxf(mown, __shfl_xor_sync(0xffffffffu, mown, 16));
          if (hh == 0) sM[(2 * sb + half) * kOwn + lrow] = mrow;
        }
        const bool p_test = u < 2 || tc::mbar_test_cluster(&B.pv_done[sb], ((u >> 1) - 1) & 1);
        tc::named_bar_sync(kBarMax + q4, 64);
        float alpha = 1.f;
        uint32_t pk[8];
        if (!dead && mine) {
          ++xu;
          // Every value that the two warps read from the exchange buffer went into
          // their maxima, so the peer may refill it (and a relaxed arrival suffices).
          if (half == 0 && lane == 0) {
            mbar_arrive_expect_tx(&B.x_full[q4], kXBytes / 4);
            tc::mbar_arrive_remote_relaxed(peer_xempty);
          }
          mrow = fmaxf(mrow, sM[(2 * sb + (half ^ 1)) * kOwn + lrow]);
          // Lazy rescale: only when the row maximum grew by more than the
          // threshold.  A row may see none of the tile's keys (or none so far):
          // its maximum stays -inf, its P zero.
          if (mrow > m_run + (kRescaleThreshold + kPShift)) {
            alpha = tc::exp2_approx(m_run - (mrow - kPShift));
            m_run = mrow - kPShift;
            l_h *= alpha;
          }
          const float mb = m_run == -INFINITY ? 0.f : m_run;
          const uint64_t cc = pack2(c2, c2), mm = pack2(-mb, -mb);
          // The row sum adds the probabilities as P V takes them, rounded: the weights
          // of the values then sum to one, and a leading key's rounding cancels.  (With
          // scores six times as large the error falls from 2.4e-4 to 2.1e-4 of the
          // norm, the largest from 6.6e-4 to 3.9e-4.  Converted back and added in pairs
          // they took 0.3% longer for 32 tokens and 1.8% over e4m3 pages.)
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 x = unpack2(fma2(s[e], cc, mm));
            const float p0 = tc::exp2_approx(x.x), p1 = tc::exp2_approx(x.y);
            pk[e] = pack_f16x2(p0, p1);
            add_f16x2(ls[2 * (e & 1)], ls[2 * (e & 1) + 1], pk[e]);
          }
          l_h += (ls[0] + ls[2]) + (ls[1] + ls[3]);
        }
        if (!dead) {
          // The P buffer and the factors of tile u - 2 have been used in both CTAs.
          if (!__all_sync(0xffffffffu, p_test)) dead = !wait_cl(&B.pv_done[sb], ((u >> 1) - 1) & 1, a);
          if (!dead) {
            uint8_t* pt = sP + sb * kPBytes + half * (kPBytes / 2);
            if (mine) {
#pragma unroll
              for (int g = 0; g < 2; ++g)
                *reinterpret_cast<uint4*>(pt + unit64(i, 2 * hh + g)) =
                    make_uint4(pk[4 * g], pk[4 * g + 1], pk[4 * g + 2], pk[4 * g + 3]);
            }
            if (half == 0 && hh == 0) {
              const float f = t == 0 ? 1.f : alpha;      // the piece's first P V overwrites O
              st_async_b32(peer_alpha + (sb * kRows + i) * 4, __float_as_uint(f), peer_pfull + sb * 8);
              sAlpha[sb * kRows + i] = f;
            }
            // A tile with keys that no row of the block sees: their values must
            // not enter P V (0 x NaN).  The score product has read the tile.
            if (base + kBK > it.kend || (base < it.wlo && base + kBK > a.p.n_sink)) {
              uint8_t* stage = sLat + ((u + kQSlots * (k + 1)) % kLatStages) * kLatStage;
              for (int q = threadIdx.x; q < kBK * 32; q += 256)
                if (!key_visible(a, it, base + (q >> 5)))
                  *reinterpret_cast<uint4*>(stage + (q >> 8) * kGroup + ((q >> 3) & 3) * kChunk + ((q >> 5) & 7) * 128 +
                                            (q & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {                       // the warp's 16 rows x 64 bytes, to the peer too
              const uint32_t off = sb * kPBytes + half * (kPBytes / 2) + (32 * q4 + 16 * rank) * 64;
              bulk_to_peer(peer_p + off, smem_u32(sP) + off, 16 * 64, peer_pfull + sb * 8);
              mbar_arrive(&B.p_full[sb]);
            }
          }
        }
      }
      // Row sums to both CTAs' output warps.  Slot k % 4 is free: the last P V
      // waited for followed the output of piece k - 3.
      float l_row = l_h + __shfl_xor_sync(0xffffffffu, l_h, 16);
      if (half == 1 && hh == 0) sM[(2 * (u & 1) + 1) * kOwn + lrow] = l_row;     // free: tile u - 2's maxima
      tc::named_bar_sync(kBarMax + q4, 64);
      if (half == 0 && !dead) {
        if (hh == 0) {
          l_row += sM[(2 * (u & 1) + 1) * kOwn + lrow];
          sL[(k & 3) * kRows + i] = l_row;
          st_async_b32(peer_l + ((k & 3) * kRows + i) * 4, __float_as_uint(l_row), peer_lfull + (k & 3) * 8);
          if (!it.whole() && rvalid) {
            float* ml = a.ws_ml + 2 * ((2 * static_cast<int64_t>(c) + (it.t_lo > 0 ? 0 : 1)) * kRows + i);
            ml[0] = m_run;
            ml[1] = l_row;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.l_full[k & 3]);
      }
      // (The sums read above are overwritten by tile u's maxima at the earliest.)
      tc::named_bar_sync(kBarMax + q4, 64);
      ++k;
    }
    ok = !dead;
  } else if (warp < kOutWarp) {
    // ===================== queries, and the peer's partial scores ==============
    const int q4 = warp - kSendWarp, hh = lane >> 4;
    const uint32_t lanes = static_cast<uint32_t>(32 * q4 + 16 * peer) << 16;     // the peer's rows
    uint8_t* xs = sXs + q4 * (kXBytes / 4);      // [keys / 4][16 rows][4 keys]
    const uint32_t peer_x = tc::mapa(smem_u32(sX), peer) + q4 * (kXBytes / 4);
    const uint32_t peer_xfull = tc::mapa(smem_u32(&B.x_full[q4]), peer);
    uint32_t qrun = 0;
    int u = 0, k = 0, xu = 0;          // tiles, pieces, tiles with something to send
#pragma unroll 1
    while (ok && items.next(a, it)) {
      // Q of the piece.  The last score product of the previous piece is
      // complete: this warp has read its result.
      {
        uint8_t* slice = sQr + q4 * 2048;
        const int rr = lane >> 2, part = lane & 3, nrows = it.nvalid - 32 * q4;
        const uint32_t tq = tmem + (static_cast<uint32_t>(32 * q4) << 16) + kTmQ;
        const uint4* qp = reinterpret_cast<const uint4*>(a.p.q_pe + (it.qrow0 + 32 * q4 + rr) * kRope) + 4 * rank + part;
        uint4 pe[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
          pe[m] = rr + 8 * m < nrows ? __ldg(qp + m * 8 * (kRope / 8)) : make_uint4(0, 0, 0, 0);
        // From the two ring stages (128 rows x 64 dims twice each), a row per
        // lane.  Rows past the block's are zero.
#pragma unroll 1
        for (int q = 0; q < kQSlots && ok; ++q) {
          const int r0 = u + kQSlots * k + q, ls = r0 % kLatStages;
          ok = wait_all(kE4m3 ? &B.raw_full[ls] : &B.lat_full[ls], (r0 / kLatStages) & 1, a);
          if (!ok) break;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const uint8_t* src = sLat + ls * kLatStage + h * (kLatStage / 2);
            uint32_t r[32];
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              const uint4 x = lane < nrows ? *reinterpret_cast<const uint4*>(src + unit128(32 * q4 + lane, w))
                                           : make_uint4(0, 0, 0, 0);
              r[4 * w] = x.x; r[4 * w + 1] = x.y; r[4 * w + 2] = x.z; r[4 * w + 3] = x.w;
            }
            tc::tmem_st32(tq + 64 * q + 32 * h, r);
          }
        }
        if (!ok) break;
        tc::tmem_st_wait();
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          qrun = bf16x2_absmax(bf16x2_absmax(qrun, pe[m].x), pe[m].y);
          qrun = bf16x2_absmax(bf16x2_absmax(qrun, pe[m].z), pe[m].w);
          *reinterpret_cast<uint4*>(slice + unit64(rr + 8 * m, part)) = bf16x8_to_f16x8(pe[m]);
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.q_ready);
      }
      const bool theirs = !kFewRows || 32 * q4 + 16 * static_cast<int>(peer) < it.nvalid;
#pragma unroll 1
      for (int t = 0; t < it.n_tiles; ++t, ++u) {
        const int sb = u & 1;
        const int xc = kFewRows ? xu : u;
        const bool x_test = xc < 1 || tc::mbar_test_cluster(&B.x_empty[q4], (xc - 1) & 1);
        ok = wait_all(&B.s_full[sb], (u >> 1) & 1, a);
        if (!ok) break;
        tc::fence_after_sync();        // also before the next piece's queries, where nothing is read here
        if (!theirs) {
          if (lane == 0) mbar_arrive(&B.s_free[sb]);
          continue;
        }
        uint32_t r[32];
        tc::tmem_ld16x2<32>(tmem + lanes + kTmS + sb * 64, r);
        tc::tmem_ld_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.s_free[sb]);
        // (read there means that the copy below has left its source, too)
        if (!__all_sync(0xffffffffu, x_test)) ok = wait_cl(&B.x_empty[q4], (xc - 1) & 1, a);
        if (!ok) break;
#pragma unroll
        for (int g = 0; g < 8; ++g)
          *reinterpret_cast<uint4*>(xs + (8 * hh + g) * 256 + (lane & 15) * 16) =
              make_uint4(r[4 * g], r[4 * g + 1], r[4 * g + 2], r[4 * g + 3]);
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) bulk_to_peer(peer_x, smem_u32(xs), kXBytes / 4, peer_xfull);
        ++xu;
      }
      ++k;
    }
    if (bf16x2_absmax_overflows(qrun)) record_error(a.p.err, MLA_ERR_RANGE);
  } else if (warp < kQkWarp) {
    // ================================= output ==================================
    // Requests of the P V warp, in order: rescale O before a P V, move it, or write
    // a finished piece's output.
    const int q4 = warp - kOutWarp, i = 32 * q4 + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
    uint8_t* stg = sStg + q4 * 2048;
    const uint32_t limit_us = static_cast<uint32_t>(
        min(a.p.wait_us + kTileUs * (B.st.hi - B.st.lo), static_cast<int64_t>(UINT32_MAX)));
    int k = 0;
    bool moved = false;                // some of the piece under way is in its partial,
    float g = 1.f;                     // which this row's factor since then has yet to shrink
    auto partial = [&](const Item& x) {  // this warp's rows in it
      const int64_t slot = 2 * static_cast<int64_t>(c) + (x.t_lo > 0 ? 0 : 1);
      return reinterpret_cast<uint8_t*>(a.ws_o + (slot * kRows + 32 * q4) * kLatent + 256 * rank);
    };
#pragma unroll 1
    for (int n = 0; ok; ++n) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&B.cmd_full, n & 1, limit_us, a.p.err));
      if (!ok) break;
      const int u = *reinterpret_cast<volatile int32_t*>(&B.cmd);
      if (u == kCmdStop) break;
      if (kLong && u <= kCmdMove) {
        const int m = kCmdMove - u;
        ok = wait_cl(&B.pv_done[(m - 1) & 1], ((m - 1) >> 1) & 1, a);
        if (!ok) break;
        tc::fence_after_sync();
        Iter ahead = items;            // (the output looks the piece up again)
        if (!ahead.next(a, it)) break;
        move_o(tmem + lanes + kTmO, stg, partial(it), it.nvalid - 32 * q4, moved, g, 1.f, nullptr);
        moved = true;
        g = sAlpha[(m & 1) * kRows + i];
      } else if (u >= 0) {
        const float f = sAlpha[(u & 1) * kRows + i];
        ok = wait_cl(&B.pv_done[(u - 1) & 1], ((u - 1) >> 1) & 1, a);
        if (!ok) break;
        tc::fence_after_sync();
        if (kLong) g *= f;
        if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            uint32_t o[32];
            tc::tmem_ld32(tmem + lanes + kTmO + 32 * cc, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tc::tmem_st32(tmem + lanes + kTmO + 32 * cc, o);
          }
          tc::tmem_st_wait();
        }
      } else {
        if (!items.next(a, it)) break;
        ok = wait_all(&B.o_ready, k & 1, a) && wait_cl(&B.l_full[k & 3], (k >> 2) & 1, a);
        if (!ok) break;
        if (warp == kOutWarp && lane == 0) mbar_arrive_expect_tx(&B.l_full[k & 3], kOwn * 4);   // piece k + 4
        tc::fence_after_sync();
        const float l = sL[(k & 3) * kRows + i];
        const float inv = l > 0.f ? 1.f / l : 0.f;     // a row that sees no key of this piece
        const int nrows = it.nvalid - 32 * q4;
        if (kLong && moved) {
          uint16_t* out = a.p.o_lat + (it.qrow0 + 32 * q4) * kLatent + 256 * rank;
          move_o(tmem + lanes + kTmO, stg, partial(it), nrows, true, g, inv,
                 it.whole() ? reinterpret_cast<uint8_t*>(out) : nullptr);
          moved = false;
        } else if (kFewRows && nrows <= 0) {
          // none of the block's rows
        } else if (it.whole()) {
          uint8_t* dst = reinterpret_cast<uint8_t*>(a.p.o_lat + (it.qrow0 + 32 * q4) * kLatent + 256 * rank);
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            uint32_t o[32];
            tc::tmem_ld32(tmem + lanes + kTmO + 32 * cc, o);
            tc::tmem_ld_wait();
            uint4 w[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              w[v].x = pack_f16x2(__uint_as_float(o[8 * v]) * inv, __uint_as_float(o[8 * v + 1]) * inv);
              w[v].y = pack_f16x2(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv);
              w[v].z = pack_f16x2(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv);
              w[v].w = pack_f16x2(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv);
            }
            store_rows(stg, lane, w, dst + cc * 64, kLatent * 2, nrows);
          }
        } else {
          uint8_t* dst = partial(it);
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            uint32_t o[32];
            tc::tmem_ld32(tmem + lanes + kTmO + 32 * cc, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              uint4 w[4];
#pragma unroll
              for (int v = 0; v < 4; ++v)
                w[v] = make_uint4(__float_as_uint(__uint_as_float(o[16 * h2 + 4 * v]) * inv),
                                  __float_as_uint(__uint_as_float(o[16 * h2 + 4 * v + 1]) * inv),
                                  __float_as_uint(__uint_as_float(o[16 * h2 + 4 * v + 2]) * inv),
                                  __float_as_uint(__uint_as_float(o[16 * h2 + 4 * v + 3]) * inv));
              store_rows(stg, lane, w, dst + (32 * cc + 16 * h2) * 4, kLatent * 4, nrows);
            }
          }
        }
        ++k;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.cmd_done);
    }
  } else if (warp == kQkWarp) {
    // ============================== score MMAs =================================
    constexpr uint32_t idesc = tc::idesc_f16(128, kBK, false, false, false);
    Rec rec = {0, 0, 0, 0, 0};
    int u = 0, k = 0;
#pragma unroll 1
    while (ok && items.next(a, it)) {
      if (it.t_lo == 0 && it.open) rec = {items.S, items.st->total, it.qrow0, it.nvalid, items.st->share};
      ok = wait_all(&B.q_ready, k & 1, a);
      // e4m3: the producers, too, must have seen the queries' loads.  One that looked only
      // after the next load into the stage had landed would wait for a parity that has
      // come and gone.
      if constexpr (kE4m3) {
        for (int r = u + kQSlots * k; ok && r < u + kQSlots * (k + 1); ++r)
          ok = wait_all(&B.lat_full[r % kLatStages], (r / kLatStages) & 1, a);
      }
      tc::fence_after_sync();
      // the queries have left the ring
      if (ok && lane < kQSlots) mbar_arrive(&B.lat_empty[(u + kQSlots * k + lane) % kLatStages]);
      ++k;
#pragma unroll 1
      for (int t = 0; ok && t < it.n_tiles; ++t, ++u) {
        const int r = u + kQSlots * k, ls = r % kLatStages, rs = u % kRopeStages, sb = u & 1;
        // The last to complete is the tile, as a rule: the others are tested
        // while it is awaited.
        const bool r_test = mbar_test(&B.rope_full[rs], (u / kRopeStages) & 1);
        const bool s_test = u < 2 || mbar_test(&B.s_free[sb], ((u >> 1) - 1) & 1);
        ok = wait_all(&B.lat_full[ls], (r / kLatStages) & 1, a);
        if (!__all_sync(0xffffffffu, r_test)) ok = ok && wait_all(&B.rope_full[rs], (u / kRopeStages) & 1, a);
        if (!__all_sync(0xffffffffu, s_test)) ok = ok && wait_all(&B.s_free[sb], ((u >> 1) - 1) & 1, a);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t k0 = smem_u32(sLat + ls * kLatStage), d = tmem + kTmS + sb * 64;
#pragma unroll 8
        for (int ks = 0; ks < 16; ++ks)        // latent half: A = Q from TMEM
          tc::mma_ts_warp(d, tmem + kTmQ + ks * 8, tc::sdesc_sw128(k0 + (ks >> 2) * kChunk + (ks & 3) * 32, 16, kGroup),
                          idesc, ks > 0 ? 1u : 0u);
        const uint32_t q0 = smem_u32(sQr), r0 = smem_u32(sRope + rs * kRopeChunk);
#pragma unroll
        for (int ks = 0; ks < kRopeHalf / 16; ++ks)
          tc::mma_ss_warp(d, tc::sdesc_sw64(q0 + ks * 32), tc::sdesc_sw64(r0 + ks * 32), idesc, 1u);
        tc::mma_commit_warp(&B.rope_empty[rs]);
        tc::mma_commit_warp(&B.s_full[sb]);
      }
    }
    if (!ok) rec.nvalid = 0;
    if (rank == 0 && lane == 0) a.rec[c] = rec;
  } else if (warp == kPvWarp) {
    // =============================== P V MMAs ==================================
    constexpr uint32_t idesc = tc::idesc_f16(128, 256, false, false, true);
    int u = 0, k = 0, n = 0;           // tiles, pieces, requests posted to the output warps
    auto post = [&](int cmd) {
      if (n > 0) ok = ok && wait_all(&B.cmd_done, (n - 1) & 1, a);
      if (!ok) return;
      if (lane == 0) {
        *reinterpret_cast<volatile int32_t*>(&B.cmd) = cmd;
        mbar_arrive(&B.cmd_full);
      }
      ++n;
    };
#pragma unroll 1
    while (ok && items.next(a, it)) {
#pragma unroll 1
      for (int t = 0; t < it.n_tiles; ++t, ++u) {
        const int ls = (u + kQSlots * (k + 1)) % kLatStages, sb = u & 1;
        const bool move = kLong && t > 0 && t % kMoveTiles == 0;
        ok = wait_cl(&B.p_full[sb], (u >> 1) & 1, a);
        if (!ok) break;
        if (t == 0) {
          if (n > 0) ok = wait_all(&B.cmd_done, (n - 1) & 1, a);          // the previous output has left O
        } else {
          const float4 f = *reinterpret_cast<const float4*>(sAlpha + sb * kRows + 4 * lane);
          if (move || __any_sync(0xffffffffu, f.x != 1.f || f.y != 1.f || f.z != 1.f || f.w != 1.f)) {
            post(move ? kCmdMove - u : u);
            if (ok) ok = wait_all(&B.cmd_done, (n - 1) & 1, a);
          }
        }
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t v0 = smem_u32(sLat + ls * kLatStage), p0 = smem_u32(sP + sb * kPBytes);
#pragma unroll
        for (int ks = 0; ks < kBK / 16; ++ks)
          tc::mma_ss_warp(tmem + kTmO, tc::sdesc_sw64(p0 + (ks >> 1) * (kPBytes / 2) + (ks & 1) * 32),
                          tc::sdesc_sw128(v0 + ks * 2 * kGroup, kChunk, kGroup), idesc,
                          ((t > 0 && !move) || ks > 0) ? 1u : 0u);
        tc::mma_commit_warp(&B.lat_empty[ls]);
        mma_commit_pair_warp(&B.pv_done[sb]);
        if (lane == 0) mbar_arrive_expect_tx(&B.p_full[sb], kPTx);     // tile u + 2's P
      }
      if (!ok) break;
      tc::mma_commit_warp(&B.o_ready);
      post(kCmdOutput);
      ++k;
    }
    if (ok) post(kCmdStop);
  } else if (warp == kLoadWarp) {
    // ============================== TMA loader =================================
    // Lane 3 j + c: box j, the part of the tile that lies in one page, looked up a
    // tile ahead: its RoPE half (c = 0), its latents or e4m3 codes (1), their scales
    // (2).  A box without a visible row is loaded from behind the last row, which
    // reads as zero.
    const int shift = min(6, a.p.c.page_shift), box = 1 << shift, nb = kBK >> shift;
    const int j = lane / 3, ch = lane % 3;
    const bool mine = j < nb, staged = !kE4m3 && a.p.c.e4m3;
    const int rope_x = (a.p.c.e4m3 ? 0 : kLatent) + kRopeHalf * static_cast<int>(rank);
    // A box's table entry, and its row given the entry.
    auto entry = [&](int t) -> int32_t {
      const int key = it.key_tile(t) * kBK + j * box;
      return mine && any_visible(a, it, key, box)
                 ? __ldg(a.p.c.table + it.b * a.p.c.table_stride + (key >> a.p.c.page_shift)) : 0;
    };
    auto row_at = [&](int t, int32_t id) -> int {
      const int key = it.key_tile(t) * kBK + j * box;
      if (!mine || !any_visible(a, it, key, box)) return a.n_rows;
      if (id >= 0 && id < a.p.c.n_pages) return (id << a.p.c.page_shift) + (key & ((1 << a.p.c.page_shift) - 1));
      record_error(a.p.err, MLA_ERR_INVALID_ARG);
      return a.n_rows;
    };
    int u = 0, k = 0;
#pragma unroll 1
    while (ok && items.next(a, it)) {
      const int32_t id0 = entry(0);            // (on its way while the queries are asked for)
#pragma unroll 1
      for (int q = 0; q < kQSlots; ++q) {           // the queries: 128 rows x 64 dims twice a stage
        const int r = u + kQSlots * k + q, ls = r % kLatStages;
        if (r >= kLatStages) ok = wait_all(&B.lat_empty[ls], ((r / kLatStages) - 1) & 1, a);
        if (!ok) break;
        uint64_t* full = kE4m3 ? &B.raw_full[ls] : &B.lat_full[ls];
        if (lane == 0) mbar_arrive_expect_tx(full, kLatStage);
        __syncwarp();
        if (lane == 0)
          tc::tma_load_3d(sLat + ls * kLatStage, &tm_q, full, 0, static_cast<int>(it.qrow0),
                          4 * static_cast<int>(rank) + 2 * q);
      }
      if (!ok) break;
      ++k;
      const int32_t base = staged ? __ldg(a.stage_base + it.b) : 0;
      int row_n = row_at(0, id0);
#pragma unroll 1
      for (int t = 0; t < it.n_tiles; ++t, ++u) {
        const int rs = u % kRopeStages, row = row_n;
        if (t + 1 < it.n_tiles) row_n = row_at(t + 1, entry(t + 1));
        // Rows that few blocks read come from HBM: each CTA has half of the next
        // tile's rows on their way into L2 (32 tokens at 4K-32K rows: 175 -> 157
        // us; for chunks, whose rows L2 holds, it costs 3-4%, and for e4m3 pages,
        // which the ring loads further ahead, it changes nothing).
        constexpr int kRowBytes = kE4m3 ? kRowE4m3 : kRowF16;
        if (it.once && !staged && ch == 0 && row_n < a.n_rows)
          tc::prefetch_l2(a.p.c.pages + (static_cast<int64_t>(row_n) + (rank ? box / 2 : 0)) * kRowBytes,
                          static_cast<uint32_t>(box / 2 * kRowBytes));
        auto load_rope = [&] {
          if (u >= kRopeStages) ok = wait_all(&B.rope_empty[rs], ((u / kRopeStages) - 1) & 1, a);
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(&B.rope_full[rs], kRopeChunk);
          __syncwarp();
          if (mine && ch == 0)
            tc::tma_load_3d(sRope + rs * kRopeChunk + j * box * 64, &tm_rope, &B.rope_full[rs], rope_x, row, 0);
        };
        // Codes go first: they are still to be converted, and the RoPE part's stage
        // waits for a score product that comes late (8 tokens at 98304 rows 225 us,
        // after it 246).
        if (!kE4m3) load_rope();
        if (!ok) break;
        const int r = u + kQSlots * k, ls = r % kLatStages;
        if (r >= kLatStages) ok = wait_all(&B.lat_empty[ls], ((r / kLatStages) - 1) & 1, a);
        if (!ok) break;
        uint64_t* full = kE4m3 ? &B.raw_full[ls] : &B.lat_full[ls];
        if (lane == 0) mbar_arrive_expect_tx(full, kE4m3 ? kRawBytes : kLatStage);
        __syncwarp();
        uint8_t* dst = sLat + ls * kLatStage;
        const int c0 = 4 * static_cast<int>(rank);
        if (kE4m3) {
          if (mine && ch == 1)
            tc::tma_load_3d(dst + kRawOff + j * box * 256, &tm_lat, full, 128 * static_cast<int>(rank), row, 0);
          else if (mine && ch == 2)
            tc::tma_load_3d(sScale + ls * kRawScale + j * box * 16, &tm_scale, full, kE4m3ScaleOff / 2, row, 0);
        } else if (staged) {
          if (lane == 0)
            tma_load_4d(dst, &tm_lat, full, 0, 0, c0, staged_row(a, it, base, it.key_tile(t)) / 8);
        } else if (mine && ch == 1) {
          tma_load_4d(dst + j * box / 8 * kGroup, &tm_lat, full, 0, 0, c0, row / 8);
        }
        if (kE4m3) load_rope();
        if (!ok) break;
      }
    }
  } else if constexpr (kE4m3) {
    // ============================ e4m3 producers ===============================
    // (a warp whose wait gave up goes on with nothing but the named barriers)
    const int pt = static_cast<int>(threadIdx.x) - kProdWarp * 32;
    bool dead = false;
    int r = 0;                         // ring position
#pragma unroll 1
    while (items.next(a, it)) {
#pragma unroll 1
      for (int q = 0; q < kQSlots; ++q, ++r) {      // the queries: a phase like the tiles'
        if (!dead) dead = !wait_all(&B.raw_full[r % kLatStages], (r / kLatStages) & 1, a);
        if (!dead && lane == 0) mbar_arrive(&B.lat_full[r % kLatStages]);
      }
#pragma unroll 1
      for (int t = 0; t < it.n_tiles; ++t, ++r) {
        const int ls = r % kLatStages;
        uint8_t* lat = sLat + ls * kLatStage;
        if (!dead) dead = !wait_all(&B.raw_full[ls], (r / kLatStages) & 1, a);
#pragma unroll 1
        for (int j = 0; j < kBK / kProdKeys; ++j) {
          Codes c;
          if (!dead) load_codes(c, lat, sScale + ls * kRawScale, static_cast<int>(rank), pt, j);
          if (j >= 2) tc::named_bar_sync(kBarProd, 32 * kProducerWarps);
          if (!dead) store_f16(c, lat, pt, j);
        }
        if (dead) continue;
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.lat_full[ls]);
      }
    }
    ok = !dead;
  }

  tc::fence_before_sync();
  if (__syncthreads_or(!ok)) {
    // A wait ran out.  Loads, copies to the other CTA and products may be under way that
    // nobody waits for any more: they take a few microseconds.
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < kGaveUpNs) __nanosleep(1000);
  }
  tc::cluster_sync();                 // nothing may be sent to a CTA that has left
  if (warp == kQkWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Merge the partials of every block that a cluster boundary cut: four warps a row,
// 4 columns a lane.  (One warp a row, 16 columns a lane, took 20 us longer for a row
// cut into 76 pieces.)  Grid: x = the cluster in which the block starts, y = group of
// 4 rows; with few blocks (kFew) x = which of the cut blocks, so that one token does
// not start 2432 blocks for a few that have work, and eight partials are under way
// with the statistics, in twice the registers.  (With and without: 128 heads, one
// token at 100 rows 11.9 and 14.0 us, 4 tokens at 2000 rows 18.9 and 19.5, 8 tokens at
// 1000 rows 18.9 and 19.1, but 16 heads at 257 rows 12.6 and 12.2; past the rule's
// bound it loses: 32 tokens took 31.7 and 29.4.)
// Launched as a programmatic dependent of the attention.
// ---------------------------------------------------------------------------
constexpr int kCombRows = 4, kMaxClusters = 128;

template <bool kFew>
__global__ void __launch_bounds__(128 * kCombRows, kFew ? 2 : 4) paged_combine_kernel(const TcArgs a, int G) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kCombRows + (warp >> 2), col = 128 * (warp & 3) + 4 * lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int c = static_cast<int>(blockIdx.x);
  if constexpr (kFew) {
    int cut[kMaxClusters / 32], before = 0;
#pragma unroll
    for (int q = 0; q < kMaxClusters / 32; ++q) cut[q] = 32 * q + lane < G ? a.rec[32 * q + lane].nvalid : 0;
    c = -1;
#pragma unroll
    for (int q = 0; q < kMaxClusters / 32; ++q) {
      const uint32_t some = __ballot_sync(0xffffffffu, cut[q] > 0);
      const int rank = before + __popc(some & ((1u << lane) - 1));
      const uint32_t mine = __ballot_sync(0xffffffffu, cut[q] > 0 && rank == static_cast<int>(blockIdx.x));
      if (mine) c = 32 * q + __ffs(mine) - 1;
      before += __popc(some);
    }
    if (c < 0) return;
  }
  const Rec r = a.rec[c];
  if (row >= r.nvalid) return;
  const int n = r.clusters(G) - c;               // pieces: one in each of these clusters
  auto slot = [&](int s) { return (2 * static_cast<int64_t>(c + s) + (s == 0 ? 1 : 0)) * kRows + row; };
  auto stat = [&](int s) {
    return s < n ? *reinterpret_cast<const float2*>(a.ws_ml + 2 * slot(s)) : make_float2(-INFINITY, 0.f);
  };
  float4 v[8];
  auto fetch = [&](int s0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = s0 + j < n ? *reinterpret_cast<const float4*>(a.ws_o + slot(s0 + j) * kLatent + col)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  if (kFew) fetch(0);
  float2 ml = stat(lane);
  float M = ml.x;
  for (int s = lane + 32; s < n; s += 32) M = fmaxf(M, a.ws_ml[2 * slot(s)]);
  M = warp_max(M);
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += 32) {
    if (s0 > 0) ml = stat(s0 + lane);
    const float w = s0 + lane < n ? exp2f(ml.x - M) * ml.y : 0.f;      // lane: partial s0 + lane's weight
    L += w;
    for (int j0 = 0; j0 < min(32, n - s0); j0 += 8) {
      if (!kFew || s0 + j0 > 0) fetch(s0 + j0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j0 + j);
        acc.x = fmaf(wj, v[j].x, acc.x);
        acc.y = fmaf(wj, v[j].y, acc.y);
        acc.z = fmaf(wj, v[j].z, acc.z);
        acc.w = fmaf(wj, v[j].w, acc.w);
      }
    }
  }
  const float inv = 1.f / warp_sum(L);
  *reinterpret_cast<uint2*>(a.p.o_lat + (r.qrow0 + row) * kLatent + col) =
      make_uint2(pack_f16x2(acc.x * inv, acc.y * inv), pack_f16x2(acc.z * inv, acc.w * inv));
}

// ---------------------------------------------------------------------------
// Staging: the latents of chosen sequences' visible rows as fp16.  Each block
// scans the batch for the sequences' first staged rows (those that still fit
// are staged), then the warps take four rows at a time; rows that no new token
// sees become zero.  HBM-bound: 656 bytes in (512 + 16 used), 1024 out a row.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256, 4) paged_stage_kernel(const TcArgs a) {
  __shared__ int32_t s_end[kStageSeqs];        // staged rows up to and with sequence b
  __shared__ long long s_warp[8];
  __shared__ int32_t s_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  long long sum = 0;
  int32_t rows[kStageSeqs / 256];
#pragma unroll
  for (int q = 0; q < kStageSeqs / 256; ++q) {
    const int b = tid * (kStageSeqs / 256) + q;
    rows[q] = 0;
    if (b < a.p.B) {
      bool bad;
      const PagedSeq s = paged_seq(a.p.cu, a.p.seq_len, b, a.p.T, a.p.c.max_rows(), bad);
      if (static_cast<int64_t>(s.n) * a.p.H > (kStageBlocks - 1) * kRows) {
        int32_t sink;
        const int32_t first = seq_first_tile(a.p, s.len - s.n, sink);
        const int64_t r = static_cast<int64_t>(sink + (s.len + kBK - 1) / kBK - first) * kBK;
        rows[q] = static_cast<int32_t>(min(r, static_cast<int64_t>(kStageRows + 1)));
      }
    }
    sum += rows[q];
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (tid == 0) s_total = 0;
  __syncthreads();
  long long end = incl - sum;
  for (int w = 0; w < warp; ++w) end += s_warp[w];
  // The sequences before the first that does not fit are staged.
#pragma unroll
  for (int q = 0; q < kStageSeqs / 256; ++q) {
    const int b = tid * (kStageSeqs / 256) + q;
    const long long base = end;
    end += rows[q];
    s_end[b] = static_cast<int32_t>(min(end, static_cast<long long>(INT32_MAX)));
    if (end <= kStageRows) atomicMax(&s_total, static_cast<int32_t>(end));
    if (blockIdx.x == 0 && b < a.p.B)
      a.stage_base[b] = rows[q] > 0 && end <= kStageRows ? static_cast<int32_t>(base) : -1;
  }
  __syncthreads();
  const int32_t total = s_total;
  // Staged row r: the sequence, the position, the pool row (-1: zero).
  auto lookup = [&](int32_t r) -> int32_t {
    if (r >= total) return -1;
    int lo = 0, hi = kStageSeqs - 1;           // the first sequence with s_end > r
    while (lo < hi) {
      const int m = (lo + hi) >> 1;
      if (s_end[m] > r) hi = m; else lo = m + 1;
    }
    bool bad;
    const PagedSeq s = paged_seq(a.p.cu, a.p.seq_len, lo, a.p.T, a.p.c.max_rows(), bad);
    const int32_t pos0 = s.len - s.n, x = r - (lo > 0 ? s_end[lo - 1] : 0);
    int32_t sink;
    const int32_t first = seq_first_tile(a.p, pos0, sink);
    const int32_t t = x / kBK, p = (t < sink ? t : t - sink + first) * kBK + x % kBK;
    const int32_t wlo = a.p.window > 0 ? max(0, pos0 - a.p.window + 1) : 0;
    if (p >= s.len || (p < wlo && p >= a.p.n_sink)) return -1;
    return static_cast<int32_t>(a.p.c.row_of(lo, p));      // a bad page: recorded by the attention
  };
  const int32_t step = 4 * static_cast<int32_t>(gridDim.x) * 8;
  int32_t r0 = 4 * (static_cast<int32_t>(blockIdx.x) * 8 + warp);
  int32_t row_n = lane < 4 ? lookup(r0 + lane) : -1;
  for (; r0 < total; r0 += step) {
    const int32_t row_l = row_n;
    uint2 v[8];
    uint32_t sc = 0x70707070u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int32_t row = __shfl_sync(0xffffffffu, row_l, k >> 1);
      v[k] = row >= 0 ? __ldg(reinterpret_cast<const uint2*>(a.p.c.pages + static_cast<int64_t>(row) * kRowE4m3) + lane +
                              32 * (k & 1))
                      : make_uint2(0, 0);
    }
    const int32_t row_s = __shfl_sync(0xffffffffu, row_l, (lane >> 2) & 3);
    if (lane < 16 && row_s >= 0)
      sc = __ldg(reinterpret_cast<const uint32_t*>(a.p.c.pages + static_cast<int64_t>(row_s) * kRowE4m3 + kE4m3ScaleOff) +
                 (lane & 3));
    if (lane < 4) row_n = lookup(r0 + step + lane);
    uint4* dst = reinterpret_cast<uint4*>(a.stage + static_cast<int64_t>(r0) * kLatent) + lane;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // unit lane + 32 (k & 1): scale byte lane / 4 + 8 (k & 1) of the row
      const uint32_t w = __shfl_sync(0xffffffffu, sc, 4 * (k >> 1) + 2 * (k & 1) + (lane >> 4));
      const uint32_t d = e4m3_scale_f16x2((w >> (8 * ((lane >> 2) & 3))) & 0xFFu);
      uint4 o;
      e4m3x4_to_f16x4(v[k].x, d, o.x, o.y);
      e4m3x4_to_f16x4(v[k].y, d, o.z, o.w);
      dst[32 * k] = o;
    }
  }
}

int clusters() { return max(1, min(kMaxClusters, device_sm_count() / 2)); }

// Workspace: partials, their sums, the clusters' records (all multiples of 16
// bytes), then the staging.
size_t partial_bytes() {
  const size_t rows = static_cast<size_t>(2 * clusters()) * kRows;
  return rows * kLatent * sizeof(float) + rows * 2 * sizeof(float) + clusters() * sizeof(Rec);
}

template <bool kE4m3, bool kFewRows, bool kLong>
cudaError_t launch_pair(const CUtensorMap& tm, const CUtensorMap& tr, const CUtensorMap& tq, const CUtensorMap& ts,
                        const TcArgs& a, cudaStream_t stream) {
  auto kern = paged_attn_kernel<kE4m3, kFewRows, kLong>;
  static std::atomic<uint64_t> set{0};         // devices on which the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || (set.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  const int G = clusters();
  e = launch_dependent(kern, dim3(2 * G), dim3(threads(kE4m3)), kSmem, stream, tm, tr, tq, ts, a);
  if (e != cudaSuccess) return e;
  // at most n_slots blocks, of at most T x H rows
  const int64_t rows = min(static_cast<int64_t>(kRows), static_cast<int64_t>(a.p.T) * a.p.H);
  const int groups = static_cast<int>((rows + kCombRows - 1) / kCombRows);
  const bool few = a.n_slots < G && a.n_slots * groups <= 10 * G;
  return launch_dependent(few ? paged_combine_kernel<true> : paged_combine_kernel<false>,
                          dim3(static_cast<unsigned>(few ? a.n_slots : G), static_cast<unsigned>(groups)),
                          dim3(128 * kCombRows), 0, stream, a, G);
}

// kLong: a block of the call can have more than kMoveTiles tiles.  Its keys are at most a
// table row's, or those of a window over its tokens (128 / 16 and two, at most) and the
// sinks, with the tiles that these cut at both ends.
bool any_long(const PagedAttnArgs& p) {
  int64_t rows = min(static_cast<int64_t>(p.c.max_pages) << p.c.page_shift, static_cast<int64_t>(INT32_MAX));
  if (p.window > 0) rows = min(rows, static_cast<int64_t>(p.window) + p.n_sink + kRows / 16 + 2 + 4 * kBK);
  return rows > kMoveTiles * kBK;
}

template <bool kE4m3, bool kFewRows>
cudaError_t launch_for(const CUtensorMap& tm, const CUtensorMap& tr, const CUtensorMap& tq, const CUtensorMap& ts,
                       const TcArgs& a, cudaStream_t stream) {
  return any_long(a.p) ? launch_pair<kE4m3, kFewRows, true>(tm, tr, tq, ts, a, stream)
                       : launch_pair<kE4m3, kFewRows, false>(tm, tr, tq, ts, a, stream);
}

}  // namespace

size_t paged_attn_workspace_bytes() {
  return partial_bytes() + kStageSeqs * sizeof(int32_t) + static_cast<size_t>(kStageRows) * kLatent * 2;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& p, cudaStream_t stream) {
  const int G = clusters();
  const size_t rows = static_cast<size_t>(2 * G) * kRows;
  TcArgs a = {};
  a.p = p;
  a.ws_o = static_cast<float*>(p.workspace);
  a.ws_ml = a.ws_o + rows * kLatent;
  a.rec = reinterpret_cast<Rec*>(a.ws_ml + rows * 2);
  int32_t* stage_base = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(p.workspace) + partial_bytes());
  a.stage = reinterpret_cast<uint16_t*>(stage_base + kStageSeqs);
  a.n_slots = static_cast<int32_t>(static_cast<int64_t>(p.T) * p.H / kRows + p.B);
  a.n_rows = p.c.n_pages << p.c.page_shift;
  // The latents of fp16 pages or of staged rows, in groups of eight rows; the
  // queries, as 64-dim chunks (dims, rows, chunks).  The RoPE parts are fp16 in
  // either row type.
  CUtensorMap tm, tr, tq;
  const uint32_t box = static_cast<uint32_t>(min(kBK, 1 << p.c.page_shift));
  const uint64_t n = static_cast<uint64_t>(a.n_rows);
  cudaError_t e;
  const uint64_t qrows = static_cast<uint64_t>(p.T) * static_cast<uint64_t>(p.H);
  e = make_tmap_3d(&tq, p.q_lat, false, 64, qrows, kLatent / 64, kLatent * 2, 128, 64, kRows, 2);
  if (e != cudaSuccess) return e;
  if (!p.c.e4m3) {
    e = make_tmap_row_groups(&tm, p.c.pages, n / 8, kRow / 64, kRowF16, box / 8, 4);
    if (e != cudaSuccess) return e;
    e = make_tmap_3d(&tr, p.c.pages, false, kRow, n, 1, kRowF16, n * kRowF16, kRopeHalf, box, 1, 64);
    if (e != cudaSuccess) return e;
    // a block of single tokens has H rows
    return p.T <= p.B && p.H <= kRows - 16 ? launch_for<false, true>(tm, tr, tq, tq, a, stream)
                                           : launch_for<false, false>(tm, tr, tq, tq, a, stream);
  }
  // In elements of two bytes, as the rows are: a CTA's 256 codes, and the 16 scales.
  CUtensorMap tcodes, tscales;
  e = make_tmap_3d(&tcodes, p.c.pages, false, kRowE4m3 / 2, n, 1, kRowE4m3, n * kRowE4m3, 128, box, 1, 0);
  if (e != cudaSuccess) return e;
  e = make_tmap_3d(&tscales, p.c.pages, false, kRowE4m3 / 2, n, 1, kRowE4m3, n * kRowE4m3, 8, box, 1, 0);
  if (e != cudaSuccess) return e;
  e = make_tmap_3d(&tr, p.c.pages + kE4m3RopeOff, false, kRope, n, 1, kRowE4m3, n * kRowE4m3, kRopeHalf, box, 1, 64);
  if (e != cudaSuccess) return e;
  // A batch of single tokens (T <= B) has no sequence of several blocks, bar one
  // with empty sequences beside it.
  if (p.T > p.B && p.B <= kStageSeqs && static_cast<int64_t>(p.T) * p.H > (kStageBlocks - 1) * kRows) {
    a.stage_base = stage_base;
    e = make_tmap_row_groups(&tm, a.stage, kStageRows / 8, kLatent / 64, kLatent * 2, kBK / 8, 4);
    if (e != cudaSuccess) return e;
    e = launch_dependent(paged_stage_kernel, dim3(device_sm_count() * 4), dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
    a.take = kTakeStaged;
    e = launch_for<false, false>(tm, tr, tq, tq, a, stream);
    if (e != cudaSuccess) return e;
    a.take = kTakeUnstaged;
  }
  return launch_for<true, false>(tcodes, tr, tq, tscales, a, stream);
}

}  // namespace mla
