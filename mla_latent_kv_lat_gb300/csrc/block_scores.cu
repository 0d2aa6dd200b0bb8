// The cheap score by which block-sparse attention chooses: for a token at position p
// and each block j < p / 64 of 64 positions before its own
//
//   score[t][j] = scale * max_h (q_lat[t][h] . kbar[j][0..511] + q_pe[t][h] . kbar[j][512..575])
//
// with kbar[j] the block's mean row; -inf for the others.
//
// On the 5th-generation tensor cores with the blocks as rows (M = 128) and the
// queries of `gt` tokens, H each, as columns (N = gt H <= 128): the largest head of a
// block then is a maximum over one thread's registers, with no exchange.
//   * A run is 128 blocks of one sequence and consecutive new tokens of it.  The mean
//     rows' latent part stays in tensor memory (256 columns), the RoPE part in shared
//     memory; queries stream through a ring of 16 KB stages by TMA.  (With the rows in
//     shared memory, both operands of each product would come from there: 128 bytes a
//     cycle, all it has.)
//   * Mean rows lie with their pages: four warps gather them with 16-byte asynchronous
//     copies, 64 dims at a time, and move them into tensor memory.  The same warps turn
//     q_pe (bf16) into fp16, the type of the mean rows.
//   * Single tokens have nothing to keep: their mean rows' products are taken from shared
//     memory, where all nine chunks come at once (through tensor memory 1 us more a run).
//   * Two accumulators of 128 columns: four warps reduce one while the next is filled.
// A chunk is bound by the queries' way into the SMs: a group of 128 columns and a tile take
// 147 KB and 2300 cycles of the tensor cores, and 3300 in fact, 44 bytes a cycle and SM
// (pairs of CTAs that load half each and multicast it were no faster).  512 tokens of 128
// heads, 520 blocks: 38 us on the GPU (queries of 75 MB in L2: 34), 1020 TFLOP/s, 53% of the measured
// rate; 48% of the tensor cores' cycles.  A single token is bound by the chain: lengths and
// shares 2.5k cycles, table 1.2k, rows 1.5k, products 3k, maxima and end 1.5k.  32 tokens,
// 4K to 98K rows: 12.8 us; one of 16 heads at 20001 rows: 5.6 us.
#include <atomic>
#include <type_traits>

#include "kernels.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kTile = 128;                   // blocks of a tile (MMA M)
constexpr int kMaxN = 128;                   // (token, head) columns
constexpr int kChunk = 128 * 128;            // 128 rows x 64 fp16
constexpr int kStage = 2 * kChunk;
constexpr int kChunks = kLatent / 64, kGroupStages = kChunks / 2;
constexpr int kBarBytes = 1024;
// kKeep: a run has many groups, and its mean rows stay in tensor memory; they come
// through three chunks, of which two hold q_pe afterwards.  Else they stay in shared memory.
template <bool kKeep>
struct Cfg {
  static constexpr int kStages = kKeep ? 5 : 2;                // of queries, two chunks each
  static constexpr int kFeed = kKeep ? 3 : 1;                  // q_pe (and mean rows on their way)
  static constexpr int kQr = kKeep ? 2 : 1;                    // q_pe
  static constexpr int kRowChunks = kKeep ? 1 : kChunks + 1;   // mean rows: the RoPE part, or all
  static constexpr int kOffFeed = kRowChunks * kChunk;
  static constexpr int kOffRing = kOffFeed + kFeed * kChunk;
  static constexpr int kOffBar = kOffRing + kStages * kStage;
  static constexpr int kSmem = 1024 + kOffBar + kBarBytes;
};
static_assert(Cfg<true>::kSmem <= 232448 && Cfg<false>::kSmem <= 232448, "shared memory");
constexpr int kFeedWarp = 4, kLoadWarp = 8, kMmaWarp = 9, kThreads = 320;
constexpr int kBarFeed = 1;
constexpr uint32_t kTmS = 0, kTmK = 256;
constexpr uint64_t kGaveUpNs = 200000;       // from a wait that ran out to the CTA's end

struct Args {
  BlockScoresArgs p;
  int32_t gt_shift;    // log2 of the tokens of a group
  int32_t tiles;       // of a row of scores
};

// Where a CTA's share of the work begins.  Work: for each sequence and each tile that
// some new token has a block in, the groups with such a token (the last ones, since
// positions grow), plus kRunCost for the run's start: one run of costs over all
// sequences, which the CTAs share evenly.  (Its length is at most (1 + kRunCost) T
// tiles, and a row of scores has 128 values a tile: it passes 2^32 with more than 512 GB
// of scores.)
constexpr int kRunCost = 3;            // mean rows' load, in groups
struct Start {
  uint32_t lo, hi;     // this CTA's range in the run of costs
  uint32_t S;          // where sequence b's cost starts in it
  int32_t b;           // the sequence that holds lo (B: nothing to do)
};

struct Bars {
  uint64_t full[5], empty[5];
  uint64_t k_full[kChunks + 1];        // the run's mean rows are there, by chunk (kKeep: [0] all of them; [1 + i]
                                       // the first run's have left stage i)
  uint64_t k_free;                     // its last product is done
  uint64_t qr_full[2], qr_empty[2];
  uint64_t s_full[2], s_empty[2];
  uint32_t tmem;
  Start st;
  uint32_t red[kThreads / 32];
  int32_t row[kTile];                  // the run's mean rows in the pool, -1: none
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers");

struct Group {
  int32_t t0, nt;                      // tokens [t0, t0 + nt)
  int32_t pos;                         // of the first
  bool fresh;                          // the first of its run: mean rows are loaded
};

// A sequence's tiles and groups.
struct Seq {
  PagedSeq s;
  MLA_DEVINL void load(const Args& a, int b) {
    bool bad;
    s = paged_seq(a.p.cu, a.p.seq_len, b, a.p.T, a.p.c.max_rows(), bad);
  }
  MLA_DEVINL int tiles(const Args& a) const {
    return s.n > 0 ? min(a.tiles, (((s.len - 1) >> kBlockShift) + kTile - 1) / kTile) : 0;
  }
  MLA_DEVINL int groups(const Args& a) const { return (s.n + (1 << a.gt_shift) - 1) >> a.gt_shift; }
  // The first group whose last token has a block in `tile` (< tiles()).
  MLA_DEVINL int first(const Args& a, int tile) const {
    const int need = (tile * kTile + 1) * kBlockRows - (s.len - s.n);       // tokens before one that has
    return max(0, need) >> a.gt_shift;
  }
  MLA_DEVINL uint32_t cost(const Args& a) const {
    uint32_t c = 0;
    for (int tile = tiles(a) - 1; tile >= 0; --tile) c += kRunCost + groups(a) - first(a, tile);
    return c;
  }
};

// This CTA's groups in order; every role walks the same ones.
struct Walk {
  uint32_t lo, hi, S;
  int32_t b, tile, tiles, i, i1;
  Seq q;
  MLA_DEVINL void init(const Args& a, const Start& st) {
    lo = st.lo;
    hi = st.hi;
    S = st.S;
    b = st.b;
    tile = -1;
    i = i1 = 0;
    tiles = 0;
    if (b < a.p.B) {
      q.load(a, b);
      tiles = q.tiles(a);
    }
  }
  MLA_DEVINL bool next(const Args& a, Group& r) {
    r.fresh = false;
    while (i >= i1) {                  // the next run
      ++tile;
      while (tile >= tiles) {
        if (++b >= a.p.B || S >= hi) return false;
        q.load(a, b);
        tiles = q.tiles(a);
        tile = 0;
      }
      if (S >= hi) return false;
      const int first = q.first(a, tile), n = q.groups(a) - first;
      const uint32_t r0 = S + kRunCost;
      S = r0 + n;
      const uint32_t p_lo = max(lo, r0), p_hi = min(hi, S);
      if (p_lo >= p_hi) continue;
      i = first + static_cast<int32_t>(p_lo - r0);
      i1 = first + static_cast<int32_t>(p_hi - r0);
      r.fresh = true;
    }
    const int t = i << a.gt_shift;
    r.t0 = q.s.q0 + t;
    r.nt = min(1 << a.gt_shift, q.s.n - t);
    r.pos = q.s.len - q.s.n + t;
    ++i;
    return true;
  }
};

MLA_DEVINL bool wait_all(uint64_t* bar, uint32_t parity, const Args& a) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.p.wait_us, a.p.err));
}

MLA_DEVINL void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
MLA_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MLA_DEVINL void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
MLA_DEVINL float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <bool kKeep>
__global__ void __launch_bounds__(kThreads, 1)
    block_scores_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  using C = Cfg<kKeep>;
  constexpr int kStages = C::kStages, kFeed = C::kFeed, kQr = C::kQr;
  uint8_t* sK = sm;
  uint8_t* sFeed = sm + C::kOffFeed;
  uint8_t* sRing = sm + C::kOffRing;
  Bars& B = *reinterpret_cast<Bars*>(sm + C::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == kLoadWarp && lane == 0) {
    tc::prefetch_tmap(&tm_q);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&B.full[i], 1);
      mbar_init(&B.empty[i], 1);
    }
    for (int i = 0; i <= kChunks; ++i) mbar_init(&B.k_full[i], 4);
    mbar_init(&B.k_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.qr_full[i], 4);
      mbar_init(&B.qr_empty[i], 1);
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.s_empty[i], 4);
    }
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&B.tmem, kKeep ? 512 : 256);
    tc::tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.p.cu, a.p.seq_len, a.p.B, a.p.T, a.p.c.max_rows(), a.p.err);

  {
    // The run of all sequences' costs: each thread sums a share of the sequences, a scan
    // gives its start, and the thread whose share holds the CTA's first unit finds the sequence.
    const int per = (a.p.B + kThreads - 1) / kThreads;
    const int b0 = min(a.p.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.p.B, b0 + per);
    Seq q;
    uint32_t sum = 0;
    for (int b = b0; b < b1; ++b) {
      q.load(a, b);
      sum += q.cost(a);
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) B.red[warp] = incl;
    if (threadIdx.x == 0) B.st = {0, 0, 0, a.p.B};
    tc::fence_before_sync();
    __syncthreads();                   // (the barriers and tensor memory are ready, too)
    tc::fence_after_sync();
    uint32_t total = 0, S = incl - sum;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      total += B.red[w];
      if (w < warp) S += B.red[w];
    }
    const uint32_t share = total / gridDim.x, more = total % gridDim.x;    // the first `more` CTAs take one more
    const uint32_t lo = share * blockIdx.x + min(blockIdx.x, more), hi = lo + share + (blockIdx.x < more ? 1 : 0);
    if (lo < hi && S <= lo && lo < S + sum) {
      int b = b0;
      if (per > 1) {
        for (; b < b1; ++b) {
          q.load(a, b);
          const uint32_t c = q.cost(a);
          if (lo < S + c) break;
          S += c;
        }
      }
      B.st = {lo, hi, S, b};
    }
    __syncthreads();
  }
  const uint32_t tmem = B.tmem;
  const int H = a.p.H, N = H << a.gt_shift;
  Walk walk;
  walk.init(a, B.st);
  Group r;
  bool ok = true;

  if (warp < kFeedWarp) {
    // ============================== maxima, output ==============================
    // First what needs no product: of each token, the scores behind its last tile.
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kFeedWarp + warp; t < a.p.T; t += static_cast<int64_t>(gridDim.x) * kFeedWarp) {
      Seq q;
      q.load(a, find_seq_warp(a.p.cu, a.p.B, static_cast<int32_t>(t)));
      if (t < q.s.q0 || t >= q.s.q0 + q.s.n) continue;
      // (the tiles of its group are computed whole)
      const int last = min(q.s.n, ((static_cast<int>(t - q.s.q0) >> a.gt_shift) + 1) << a.gt_shift) - 1;
      const int own = (q.s.len - q.s.n + last) >> kBlockShift;
      if (own > a.p.W && lane == 0) record_error(a.p.err, MLA_ERR_INVALID_ARG);
      for (int j = min((own + kTile - 1) / kTile, a.tiles) * kTile + lane; j < a.p.W; j += 32)
        a.p.scores[t * a.p.stride + j] = -INFINITY;
    }
    const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
    int u = 0;
    while (ok && walk.next(a, r)) {
      const int j = walk.tile * kTile + 32 * warp + lane;
      float* out = a.p.scores + static_cast<int64_t>(r.t0) * a.p.stride + j;
      const int sb = u & 1;
      ok = wait_all(&B.s_full[sb], (u >> 1) & 1, a);
      if (!ok) break;
      tc::fence_after_sync();
      float m = -INFINITY;
      int t = 0, c = 0;                  // token of the group, columns of it seen
#pragma unroll 1
      for (int c0 = 0; c0 < r.nt * H; c0 += 32) {
        uint32_t x[32];
        tc::tmem_ld32(tmem + lanes + kTmS + sb * kMaxN + c0, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (t >= r.nt) break;          // (half of the last 32 may lie behind the group)
#pragma unroll
          for (int e = 0; e < 16; e += 2) m = max3(m, __uint_as_float(x[16 * h + e]), __uint_as_float(x[16 * h + e + 1]));
          c += 16;
          if (c == H) {
            if (j < a.p.W) *out = j < (r.pos + t) >> kBlockShift ? m * a.p.scale : -INFINITY;
            out += a.p.stride;
            m = -INFINITY;
            c = 0;
            ++t;
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.s_empty[sb]);
      ++u;
    }
  } else if (warp < kLoadWarp) {
    // ======================== mean rows, RoPE parts of queries ==================
    // (a warp whose wait gave up goes on with nothing but the named barriers)
    const int ft = threadIdx.x - 32 * kFeedWarp, q4 = warp - kFeedWarp, un = ft & 7;
    const int per_shift = a.p.c.page_shift - kBlockShift;
    const int64_t qrows = static_cast<int64_t>(a.p.T) * H;
    uint32_t qrun = 0;
    bool dead = false;
    int u = 0, k = 0;
    while (walk.next(a, r)) {
      // q_pe of the group: N rows x 64, eight 16-byte units a thread
      const int64_t row0 = static_cast<int64_t>(r.t0) * H;
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = (ft >> 3) + 16 * i;
        v[i] = row < r.nt * H && row0 + row < qrows
                   ? __ldg(reinterpret_cast<const uint4*>(a.p.q_pe + (row0 + row) * kRope) + un) : make_uint4(0, 0, 0, 0);
      }
      if (r.fresh) {
        // The sequence's blocks before its last token's own are there; the others are zero.
        const int n_there = (walk.q.s.len - 1) >> kBlockShift;
        const int j = walk.tile * kTile + ft;
        int32_t mine = -1;
        if (j < n_there) {
          const int32_t id = __ldg(a.p.c.table + walk.b * a.p.c.table_stride + (j >> per_shift));
          if (id >= 0 && id < a.p.c.n_pages) mine = (id << per_shift) + (j & ((1 << per_shift) - 1));
          else record_error(a.p.err, MLA_ERR_INVALID_ARG);
        }
        B.row[ft] = mine;
        __syncwarp();
        // A warp brings its own 32 rows: unit lane + 32 i of its part of a chunk, row r0 + 4 i.
        const int r0 = 32 * q4 + (lane >> 3);
        const uint16_t* src[8];
        uint32_t there = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t row = B.row[r0 + 4 * i];
          src[i] = a.p.keys + static_cast<int64_t>(max(row, 0)) * kRow + 8 * un;
          there |= row >= 0 ? 1u << i : 0u;
        }
        // The last products of the run before have read its rows (and q_pe of all groups).
        if (k > 0 && !dead) {
          dead = !wait_all(&B.k_free, (k - 1) & 1, a);
          tc::fence_after_sync();          // (tensor memory that they read is written next)
        }
        auto fetch = [&](uint8_t* to, int c) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = r0 + 4 * i;
            cp_async16(smem_u32(to) + row * 128 + ((un ^ (row & 7)) << 4), src[i] + 64 * c, (there >> i & 1) != 0);
          }
          cp_async_commit();
        };
        if constexpr (kKeep) {
          // 64 dims of this warp's rows from a chunk into tensor memory, a row a lane.
          auto keep = [&](const uint8_t* from, int c) {
            const int row = 32 * q4 + lane;
            uint32_t x[32];
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              const uint4 v = *reinterpret_cast<const uint4*>(from + row * 128 + ((w ^ (row & 7)) << 4));
              x[4 * w] = v.x; x[4 * w + 1] = v.y; x[4 * w + 2] = v.z; x[4 * w + 3] = v.w;
            }
            tc::tmem_st32(tmem + (static_cast<uint32_t>(32 * q4) << 16) + kTmK + 32 * c, x);
            __syncwarp();
          };
          if (k == 0) {
            // The first run's come all at once, through the stages that the queries take afterwards.
            if (!dead) {
              fetch(sK, kChunks);
#pragma unroll 1
              for (int c = 0; c < kChunks; ++c) fetch(sRing + c * kChunk, c);
#pragma unroll 1
              for (int c = 0; c < kChunks; ++c) {
                if (c == 0) cp_async_wait<kChunks / 2>();
                if (c == kChunks / 2) cp_async_wait<0>();
                __syncwarp();
                keep(sRing + c * kChunk, c);
                if (c & 1) {
                  tc::fence_proxy_async();       // (bulk copies of queries go where these copies went)
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&B.k_full[1 + c / 2]);
                }
              }
            }
          } else if (!dead) {
            fetch(sK, kChunks);
            for (int c = 0; c < kFeed; ++c) fetch(sFeed + c * kChunk, c);
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
              cp_async_wait<kFeed - 1>();
              __syncwarp();
              keep(sFeed + (c % kFeed) * kChunk, c);
              if (c + kFeed < kChunks) fetch(sFeed + (c % kFeed) * kChunk, c + kFeed);
              else cp_async_commit();      // (an empty group keeps the count)
            }
          }
          if (!dead) {
            tc::tmem_st_wait();
            tc::fence_proxy_async();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.k_full[0]);
          }
          // (q_pe goes where other warps' rows were)
          tc::named_bar_sync(kBarFeed, 128);
        } else if (!dead) {
          // all at once; a chunk is passed on when it has arrived, from the fifth on behind the next one's request
          auto arrived = [&](int c) {
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.k_full[c]);
          };
#pragma unroll 1
          for (int c = 0; c <= kChunks; ++c) {
            fetch(sK + c * kChunk, c);
            if (c >= 5) {
              cp_async_wait<5>();
              arrived(c - 5);
            }
          }
          cp_async_wait<4>(); arrived(4);
          cp_async_wait<3>(); arrived(5);
          cp_async_wait<2>(); arrived(6);
          cp_async_wait<1>(); arrived(7);
          cp_async_wait<0>(); arrived(8);
        }
        ++k;
      }
      if (dead) continue;
      const int qb = u % kQr;
      if (u >= kQr) dead = !wait_all(&B.qr_empty[qb], (u / kQr - 1) & 1, a);
      if (dead) continue;
      uint8_t* to = sFeed + qb * kChunk;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = (ft >> 3) + 16 * i;
        qrun = bf16x2_absmax(bf16x2_absmax(qrun, v[i].x), v[i].y);
        qrun = bf16x2_absmax(bf16x2_absmax(qrun, v[i].z), v[i].w);
        uint4 o;
        float2 f;
        f = bf16x2_to_f32(v[i].x); o.x = pack_f16x2(f.x, f.y);
        f = bf16x2_to_f32(v[i].y); o.y = pack_f16x2(f.x, f.y);
        f = bf16x2_to_f32(v[i].z); o.z = pack_f16x2(f.x, f.y);
        f = bf16x2_to_f32(v[i].w); o.w = pack_f16x2(f.x, f.y);
        *reinterpret_cast<uint4*>(to + row * 128 + ((un ^ (row & 7)) << 4)) = o;
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.qr_full[qb]);
      ++u;
    }
    if (bf16x2_absmax_overflows(qrun)) record_error(a.p.err, MLA_ERR_RANGE);
    ok = !dead;
  } else if (warp == kLoadWarp) {
    // ============================== queries (TMA) ===============================
    int st = 0, use = 0;                 // the next stage, and how often the ring has been through
    while (ok && walk.next(a, r)) {
#pragma unroll 1
      for (int c = 0; c < kGroupStages; ++c) {
        if (use > 0) ok = ok && wait_all(&B.empty[st], (use - 1) & 1, a);
        else if (kKeep && st < kGroupStages) ok = ok && wait_all(&B.k_full[1 + st], 0, a);      // the first run's mean rows
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&B.full[st], static_cast<uint32_t>(N) * 256);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tc::tma_load_3d(sRing + st * kStage + h * kChunk, &tm_q, &B.full[st], 0, r.t0 * H, 2 * c + h);
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          ++use;
        }
      }
    }
  } else {
    // ================================== MMAs ====================================
    const uint32_t idesc = tc::idesc_f16(128, N, false, false, false);
    // Addresses are constants beside this one, which a reduction makes known to be the
    // same in all lanes: held in lanes' registers, each product's operands would be moved
    // over first, and the issue, not the tensor cores, would be the limit.
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
    const uint64_t ring = tc::sdesc_sw128(smem_u32(sRing), 16, 1024), rows = tc::sdesc_sw128(smem_u32(sK), 16, 1024),
                   qpe = tc::sdesc_sw128(smem_u32(sFeed), 16, 1024);
    auto at = [](uint64_t desc, int bytes) { return desc + static_cast<uint64_t>(bytes >> 4); };
    int u = 0, k = 0, st = 0, use = 0;
    while (ok && walk.next(a, r)) {
      const bool fresh = r.fresh;
      if (fresh) {
        // the run before is done with its mean rows when its products are
        if (k > 0) tc::mma_commit_warp(&B.k_free);
        if (kKeep) ok = wait_all(&B.k_full[0], k & 1, a);
        if (!ok) break;
        ++k;
      }
      auto group = [&](auto buf) {
        constexpr int sb = decltype(buf)::value, qb = sb % kQr;
        const uint32_t d = tm + kTmS + sb * kMaxN;
        if (u >= 2) ok = wait_all(&B.s_empty[sb], ((u >> 1) - 1) & 1, a);
        if (!ok) return;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < kGroupStages; ++c) {
          ok = ok && wait_all(&B.full[st], use & 1, a);
          if (!kKeep && fresh) ok = ok && wait_all(&B.k_full[2 * c], (k - 1) & 1, a) && wait_all(&B.k_full[2 * c + 1], (k - 1) & 1, a);
          if (!ok) return;
          tc::fence_after_sync();
          const uint32_t stage = __reduce_max_sync(0xffffffffu, st * (kStage >> 4));
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const uint64_t qd = at(ring + stage, (h >> 2) * kChunk + 32 * (h & 3));
            if constexpr (kKeep) tc::mma_ts_warp(d, tm + kTmK + 64 * c + 8 * h, qd, idesc, (c | h) != 0);
            else tc::mma_ss_warp(d, at(rows, (2 * c + (h >> 2)) * kChunk + 32 * (h & 3)), qd, idesc, (c | h) != 0);
          }
          tc::mma_commit_warp(&B.empty[st]);
          if (++st == kStages) {
            st = 0;
            ++use;
          }
        }
        ok = wait_all(&B.qr_full[qb], (u / kQr) & 1, a);
        if (!kKeep && fresh) ok = ok && wait_all(&B.k_full[kChunks], (k - 1) & 1, a);
        if (!ok) return;
        tc::fence_after_sync();
#pragma unroll
        for (int h = 0; h < 4; ++h)
          tc::mma_ss_warp(d, at(rows, (C::kRowChunks - 1) * kChunk + 32 * h), at(qpe, qb * kChunk + 32 * h), idesc, 1u);
        tc::mma_commit_warp(&B.qr_empty[qb]);
        tc::mma_commit_warp(&B.s_full[sb]);
      };
      if (u & 1) group(std::integral_constant<int, 1>());
      else group(std::integral_constant<int, 0>());
      ++u;
    }
  }

  tc::fence_before_sync();
  if (__syncthreads_or(!ok)) {
    // A wait ran out: loads and products may be under way that nobody waits for any more.
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < kGaveUpNs) __nanosleep(1000);
  }
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kKeep ? 512 : 256);
  }
}

template <bool kKeep>
cudaError_t launch(const CUtensorMap& tq, const Args& a, cudaStream_t stream) {
  auto kern = block_scores_kernel<kKeep>;
  static std::atomic<uint64_t> set{0};         // devices on which the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || (set.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<kKeep>::kSmem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  const int64_t sms = device_sm_count();
  // a run of single tokens is one group: no more CTAs than there can be runs
  const int64_t grid = a.p.T > a.p.B ? sms : min(sms, static_cast<int64_t>(a.p.T) * a.tiles);
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), Cfg<kKeep>::kSmem, stream, tq, a);
}

}  // namespace

cudaError_t launch_block_scores(const BlockScoresArgs& p, cudaStream_t stream) {
  Args a = {};
  a.p = p;
  // Tokens of a group are of one sequence: with single tokens there is one.
  if (p.T > p.B)
    while ((2 * p.H << a.gt_shift) <= kMaxN) ++a.gt_shift;
  a.tiles = (p.W - 1) / kTile + 1;
  CUtensorMap tq;
  const uint64_t qrows = static_cast<uint64_t>(p.T) * static_cast<uint64_t>(p.H);
  cudaError_t e = make_tmap_3d(&tq, p.q_lat, false, 64, qrows, kChunks, kLatent * 2, 128, 64,
                               static_cast<uint32_t>(p.H << a.gt_shift), 1);
  if (e != cudaSuccess) return e;
  // Mean rows are kept from 2.5 groups an SM on.  (From shared memory and kept, 3 tiles:
  // 64 heads, 8 sequences of 32 tokens 12.7 and 12.7 us, of 64 22.3 and 20.7, 32 of 4 10.5
  // and 10.9, of 32 39.7 and 32.3; one of 64 7.8 and 8.6.)
  const bool keep = p.T > p.B && 2 * static_cast<int64_t>(p.T >> a.gt_shift) * a.tiles > 5 * device_sm_count();
  return keep ? launch<true>(tq, a, stream) : launch<false>(tq, a, stream);
}

}  // namespace mla
