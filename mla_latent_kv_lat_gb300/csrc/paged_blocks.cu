// What block-sparse attention needs beside its scores: the mean row of each block of
// 64 positions, and the choice of a token's blocks from their scores.
#include "kernels.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace mla {
namespace {

// ---------------------------------------------------------------------------
// Mean rows.  A block that the new tokens complete (its last position is one of
// theirs) gets keys[page][block of the page] = mean of its 64 rows, summed in fp32 and
// rounded once.  Slots: sequence b's completed blocks get slots cu[b] / 64 + b, ...
// (n new tokens complete at most ceil(n / 64) blocks, so ranges do not overlap).
// HBM-bound: a block of threads reads a block's 64 rows whole, each thread 16 bytes
// of every kGroups-th row, eight of them under way at once (sixteen leave room for
// half the blocks on an SM: 23.5 us instead of 19.5; a grid that stays, its next block
// looked up beside the rows: 19.8, for e4m3 18.2 instead of 16.8).  98304 fp16 rows: 19.5 us,
// 5.9 TB/s, 88% of the copy rate; e4m3 16.8 us; the one block that 64 single tokens complete:
// 3.3 us, a launch and the lookups.
// ---------------------------------------------------------------------------
template <bool kE4m3>
struct KeyCfg {
  static constexpr int kUnits = kE4m3 ? 40 : 72;        // 16-byte units of a row's values
  static constexpr int kGroups = kE4m3 ? 8 : 4;         // row groups
  static constexpr int kThreads = kUnits * kGroups;     // 320, 288
  static constexpr int kRowsEach = kBlockRows / kGroups;
  static constexpr int kAtOnce = 8;                     // loads of a thread under way
  static_assert(!kE4m3 || kRowsEach == kAtOnce, "one pass");
};

// The two halves of w (fp16) added to x[0], x[1] in fp32.
MLA_DEVINL void add2(float* x, uint32_t w) {
  x[0] = tc::add_f16lo_f32(w, x[0]);
  x[1] = tc::add_f16hi_f32(w, x[1]);
}

MLA_DEVINL int64_t key_slot(const BlockKeysArgs& a, int b) {
  return (max(0, min(a.T, __ldg(a.cu + b))) >> kBlockShift) + b;
}

template <bool kE4m3>
__global__ void __launch_bounds__(KeyCfg<kE4m3>::kThreads, kE4m3 ? 3 : 4) block_keys_kernel(const BlockKeysArgs a) {
  using C = KeyCfg<kE4m3>;
  __shared__ float part[C::kGroups][kRow];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, a.c.max_rows(), a.err);
  const int unit = threadIdx.x % C::kUnits, grp = threadIdx.x / C::kUnits;
  const int64_t slots = (a.T >> kBlockShift) + a.B;
  // First row of slot g's block, -1: none.
  auto find = [&](int64_t g) -> int64_t {
    int lo = 0, n = a.B;                       // the largest b with key_slot(b) <= g, 32 at a time
    const int lane = threadIdx.x & 31;
    while (n > 1) {
      const int step = (n + 31) / 32, m = lo + lane * step;
      const uint32_t le = __ballot_sync(0xffffffffu, lane == 0 || (m < lo + n && key_slot(a, m) <= g));
      const int k = 31 - __clz(le);
      n = min(step, n - k * step);
      lo += k * step;
    }
    bool bad;
    const PagedSeq s = paged_seq(a.cu, a.seq_len, lo, a.T, a.c.max_rows(), bad);
    const int64_t g0 = key_slot(a, lo), j = ((s.len - s.n) >> kBlockShift) + (g - g0);     // the sequence's block
    if (s.n == 0 || g < g0 || j >= (s.len >> kBlockShift)) return -1;
    const int64_t row0 = a.c.row_of(lo, j << kBlockShift);
    if (row0 < 0 && threadIdx.x == 0) record_error(a.err, MLA_ERR_INVALID_ARG);
    return row0;
  };
  for (int64_t g = blockIdx.x; g < slots; g += gridDim.x) {
    const int64_t row0 = find(g);
    if (row0 < 0) continue;
    constexpr int kBytes = kE4m3 ? kRowE4m3 : kRowF16;
    const uint8_t* src = a.c.pages + row0 * kBytes;
    if constexpr (!kE4m3) {
      float x[8] = {};
#pragma unroll 1
      for (int r0 = 0; r0 < C::kRowsEach; r0 += C::kAtOnce) {
        uint4 v[C::kAtOnce];
#pragma unroll
        for (int r = 0; r < C::kAtOnce; ++r)
          v[r] = __ldg(reinterpret_cast<const uint4*>(src + (grp + C::kGroups * (r0 + r)) * kBytes) + unit);
#pragma unroll
        for (int r = 0; r < C::kAtOnce; ++r) {
          const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) add2(x + 2 * q, w[q]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e += 4)
        *reinterpret_cast<float4*>(&part[grp][8 * unit + e]) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    } else {
      // units 0-31: 16 codes each, half of a scale's block; 32-39: eight RoPE values
      uint4 v[C::kAtOnce];
      uint32_t d[C::kAtOnce];
#pragma unroll
      for (int r = 0; r < C::kAtOnce; ++r) {
        const uint8_t* row = src + (grp + C::kGroups * r) * kBytes;
        v[r] = __ldg(reinterpret_cast<const uint4*>(row) + unit);
        d[r] = unit < 32 ? __ldg(row + kE4m3ScaleOff + unit / 2) : 0u;
      }
      float x[16] = {};
#pragma unroll
      for (int r = 0; r < C::kAtOnce; ++r) {
        const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
        if (unit < 32) {
          const uint32_t sc = e4m3_scale_f16x2(d[r]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t lo2, hi2;
            e4m3x4_to_f16x4(w[q], sc, lo2, hi2);
            add2(x + 4 * q, lo2);
            add2(x + 4 * q + 2, hi2);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) add2(x + 2 * q, w[q]);
        }
      }
      float* dst = &part[grp][unit < 32 ? 16 * unit : kLatent + 8 * (unit - 32)];
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        if (unit < 32 || e < 8) *reinterpret_cast<float4*>(dst + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
    __syncthreads();
    uint32_t* out = reinterpret_cast<uint32_t*>(a.keys + (row0 >> kBlockShift) * kRow);
    for (int c = threadIdx.x; c < kRow / 2; c += C::kThreads) {
      float p = 0.f, q = 0.f;
#pragma unroll
      for (int r = 0; r < C::kGroups; ++r) {
        const float2 f = *reinterpret_cast<const float2*>(&part[r][2 * c]);
        p += f.x;
        q += f.y;
      }
      out[c] = pack_f16x2(p * (1.f / kBlockRows), q * (1.f / kBlockRows));
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The choice.  A token at position p takes its own block p / 64, the n_local - 1
// before it, the first n_sink, and of the others those with the largest scores, K in
// all; equal scores go to the lower block.  Written in ascending order, -1 behind.
//
// A score becomes a key that orders as its value (larger is better; -0 as 0; a NaN
// below everything).  The key of the last one taken is found bit by bit, the largest x
// with at least R candidates of keys >= x, or until some x has exactly R.  A block of
// kWarps warps takes a token, with kPer keys in each thread's registers: a warp alone
// counts with no barrier, and with many tokens that is what it is bound by
// (instructions, two a key and bit); more warps are quicker for one token.  4595 tokens
// over 313 to 1024 blocks, 59 of them chosen: 14.4 us, 2000 instructions a token, issued
// in 64% of the cycles (eight warps a token 105 us, a warp without the closer search 20.5);
// 32 tokens of up to 1536 blocks: 5.2 us, eight warps each (a warp each 9.6).
// ---------------------------------------------------------------------------
MLA_DEVINL uint32_t score_key(float s) {
  const uint32_t u = __float_as_uint(s + 0.f);            // (-0 + 0 = 0)
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 1u;         // NaN; -inf is 0x007FFFFF
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// A token's part of the choice.
struct Choice {
  int own;            // its block
  int c0, n;          // candidates [c0, c0 + n); the others up to `own` are taken as they are
  int R;              // candidates to take
};
// False: the token gets nothing (padding, or recorded).
MLA_DEVINL bool choice_of(const SelectBlocksArgs& a, int64_t t, int tid, int nthreads, Choice& c) {
  const int b = find_seq_warp(a.cu, a.B, static_cast<int32_t>(t));
  bool bad;
  const PagedSeq s = paged_seq(a.cu, a.seq_len, b, a.T, INT32_MAX - 4096, bad);
  if (t < s.q0 || t >= s.q0 + s.n) return false;
  c.own = (s.len - s.n + static_cast<int>(t - s.q0)) >> kBlockShift;
  if (c.own >= a.W) {                    // its blocks have no scores
    if (tid == 0) {
      record_error(a.err, MLA_ERR_INVALID_ARG);
      a.counts[t] = 0;
    }
    for (int i = tid; i < a.K; i += nthreads) a.blocks[t * a.K + i] = -1;
    return false;
  }
  const int c1 = max(0, c.own - a.n_local + 1);
  c.c0 = min(a.n_sink, c1);
  c.n = c1 - c.c0;
  c.R = min(c.n, a.K - (c.own + 1 - c.n));
  return true;
}
// What needs no scores: the first blocks, the last, what lies behind them, the count;
// with R == n all.
MLA_DEVINL void write_sure(const SelectBlocksArgs& a, int64_t t, int tid, int nthreads, const Choice& c) {
  int32_t* out = a.blocks + t * a.K;
  const int total = c.own + 1 - c.n + c.R, head = c.R == c.n ? total : c.c0;
  for (int i = tid; i < a.K; i += nthreads) {
    if (i < head) out[i] = i;
    else if (i >= c.c0 + c.R) out[i] = i < total ? c.own - (total - 1 - i) : -1;
  }
  if (tid == 0) a.counts[t] = total;
}

constexpr int kClose = 8;      // keys of a lane in the closer search

// A block of threads takes one token; of those that are a warp's, kSingles.
constexpr int kSingles = 4;

template <int kWarps, int kPer>
__global__ void __launch_bounds__(kWarps == 1 ? 32 * kSingles : 32 * kWarps, kWarps > 1 ? 1 : kPer == 32 ? 8 : 5)
    select_blocks_kernel(const SelectBlocksArgs a) {
  constexpr int kN = 32 * kWarps, kWaves = kPer * kWarps, kEach = (kWaves + 31) / 32, kTok = kWarps == 1 ? kSingles : 1;
  __shared__ int s_cnt[2][kWarps];
  __shared__ uint32_t s_waves[kTok][32 * kEach];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, INT32_MAX - 4096, a.err);
  const int lane = threadIdx.x & 31, warp = kWarps == 1 ? 0 : static_cast<int>(threadIdx.x >> 5);
  const int tok = kWarps == 1 ? static_cast<int>(threadIdx.x >> 5) : 0, tid = kWarps == 1 ? lane : static_cast<int>(threadIdx.x);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTok + tok;
  if (t >= a.T) return;
  uint32_t* s_wave = s_waves[tok];
  Choice c;
  if (!choice_of(a, t, tid, kN, c)) return;
  const float* src = a.scores + t * a.stride + c.c0;
  uint32_t key[kPer];                    // of candidates tid + k kN (0: there is none)
  if (c.R > 0 && c.R < c.n) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) key[k] = tid + k * kN < c.n ? score_key(__ldg(src + tid + k * kN)) : 0u;
  }
  write_sure(a, t, tid, kN, c);
  if (c.R == 0 || c.R == c.n) return;
  int32_t* out = a.blocks + t * a.K + c.c0;
  if constexpr (kWarps == 1) {
    // Of up to 32 (64) to take none lies below the least of the lanes' largest (second
    // largest) keys, for each lane has that one or better.  What is left, a quarter as a
    // rule, is written closely, in order, and the search goes on in an eighth of the keys.
    uint32_t m1 = 0, m2 = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      m2 = max(m2, min(m1, key[k]));
      m1 = max(m1, key[k]);
    }
    const uint32_t least = max(1u, __reduce_min_sync(0xffffffffu, c.R <= 32 ? m1 : m2)), top = __reduce_max_sync(0xffffffffu, m1);
    int left = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) left += key[k] >= least;
    left = __reduce_add_sync(0xffffffffu, left);
    if (c.R <= 64 && left <= 32 * kClose) {
      __shared__ uint32_t s_keys[kTok][32 * kClose];
      __shared__ uint16_t s_ats[kTok][32 * kClose];
      uint32_t* s_key = s_keys[tok];
      uint16_t* s_at = s_ats[tok];
      const uint32_t below = (1u << lane) - 1;
      int at = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const uint32_t m = __ballot_sync(0xffffffffu, key[k] >= least);
        if (key[k] >= least) {
          const int p = at + __popc(m & below);
          s_key[p] = key[k];
          s_at[p] = static_cast<uint16_t>(lane + 32 * k);
        }
        at += __popc(m);
      }
      __syncwarp();
      uint32_t close[kClose];
#pragma unroll
      for (int k = 0; k < kClose; ++k) close[k] = lane + 32 * k < left ? s_key[lane + 32 * k] : 0u;
      auto count = [&](uint32_t y) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < kClose; ++k) n += close[k] >= y;
        return static_cast<int>(__reduce_add_sync(0xffffffffu, n));
      };
      // All keys left share the bits above `bits`.  Where they are just the R to take there
      // is nothing to search, and x is the least of them: those bits may all be 0, which
      // the slots behind `left` hold.
      const int bits = 32 - __clz(top ^ least);
      uint32_t x = left == c.R ? least : bits < 32 ? top >> bits << bits : 0u;
      int n_x = left;                      // keys >= x
      for (int bit = bits - 1; bit >= 0 && n_x != c.R; --bit) {
        const uint32_t y = x | (1u << bit);
        const int n = count(y);
        if (n >= c.R) {
          x = y;
          n_x = n;
        }
      }
      const int ties = n_x == c.R ? c.R : c.R - (x == 0xFFFFFFFFu ? 0 : count(x + 1));
      int larger = 0, equal = 0;           // before this wave
#pragma unroll
      for (int k = 0; k < kClose; ++k) {
        const uint32_t gt = __ballot_sync(0xffffffffu, close[k] > x), eq = __ballot_sync(0xffffffffu, close[k] == x);
        const int eq_r = equal + __popc(eq & below);
        if (close[k] > x || (close[k] == x && eq_r < ties))
          out[larger + __popc(gt & below) + min(eq_r, ties)] = c.c0 + s_at[lane + 32 * k];
        larger += __popc(gt);
        equal += __popc(eq);
      }
      return;
    }
  }
  int buf = 0;
  auto count = [&](uint32_t y) -> int {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) n += key[k] >= y;
    n = __reduce_add_sync(0xffffffffu, n);
    if constexpr (kWarps > 1) {
      if (lane == 0) s_cnt[buf][warp] = n;
      __syncthreads();
      n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) n += s_cnt[buf][w];
      buf ^= 1;
    }
    return n;
  };
  uint32_t x = 0;
  int least = c.n;                       // keys >= x
  for (int bit = 31; bit >= 0 && least != c.R; --bit) {
    const uint32_t y = x | (1u << bit);
    const int n = count(y);
    if (n >= c.R) {
      x = y;
      least = n;
    }
  }
  // Keys > x are taken, and of those equal to it the first `ties`.
  const int ties = least == c.R ? c.R : c.R - (x == 0xFFFFFFFFu ? 0 : count(x + 1));
  // Wave k of warp w, in this order, holds kWaves x 32 candidates in order.
  uint32_t wave[kPer];                   // larger ones in the low half, equal ones in the high
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t gt = __ballot_sync(0xffffffffu, key[k] > x), eq = __ballot_sync(0xffffffffu, key[k] == x);
    wave[k] = __popc(gt) | __popc(eq) << 16;
    if (lane == 0) s_wave[k * kWarps + warp] = wave[k];
  }
  if constexpr (kWarps > 1) __syncthreads();
  else __syncwarp();
  uint32_t mine[kEach], sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int w = lane * kEach + e;
    mine[e] = sum;
    sum += w < kWaves ? s_wave[w] : 0u;
  }
  uint32_t before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  before -= sum;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t gt = __ballot_sync(0xffffffffu, key[k] > x), eq = __ballot_sync(0xffffffffu, key[k] == x);
    const int w = k * kWarps + warp;
    uint32_t p = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint32_t v = __shfl_sync(0xffffffffu, before + mine[e], w / kEach);
      if (w % kEach == e) p = v;
    }
    const uint32_t below = (1u << lane) - 1;
    const int gt_r = static_cast<int>(p & 0xFFFFu) + __popc(gt & below), eq_r = static_cast<int>(p >> 16) + __popc(eq & below);
    if (key[k] > x || (key[k] == x && eq_r < ties)) out[gt_r + min(eq_r, ties)] = c.c0 + tid + k * kN;
  }
}

// Rows of any length: the keys are read again for each bit.
constexpr int kLongWarps = 8, kLongThreads = 32 * kLongWarps;

__global__ void __launch_bounds__(kLongThreads) select_long_kernel(const SelectBlocksArgs a) {
  __shared__ int s_cnt[2][kLongWarps];
  __shared__ int2 s_wave[kLongWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, INT32_MAX - 4096, a.err);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t = blockIdx.x;
  Choice c;
  if (!choice_of(a, t, tid, kLongThreads, c)) return;
  write_sure(a, t, tid, kLongThreads, c);
  if (c.R == 0 || c.R == c.n) return;
  const float* src = a.scores + t * a.stride + c.c0;
  int buf = 0;
  auto count = [&](uint32_t y) -> int {
    int n = 0;
#pragma unroll 4
    for (int i = tid; i < c.n; i += kLongThreads) n += score_key(__ldg(src + i)) >= y;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s_cnt[buf][warp] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kLongWarps; ++w) n += s_cnt[buf][w];
    buf ^= 1;
    return n;
  };
  uint32_t x = 0;
  int least = c.n;
  for (int bit = 31; bit >= 0 && least != c.R; --bit) {
    const uint32_t y = x | (1u << bit);
    const int n = count(y);
    if (n >= c.R) {
      x = y;
      least = n;
    }
  }
  const int ties = least == c.R ? c.R : c.R - (x == 0xFFFFFFFFu ? 0 : count(x + 1));
  int32_t* out = a.blocks + t * a.K + c.c0;
  int larger = 0, equal = 0;                   // before this wave
  for (int i0 = 0; i0 < c.n; i0 += kLongThreads) {
    const uint32_t key = i0 + tid < c.n ? score_key(__ldg(src + i0 + tid)) : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, key > x), eq = __ballot_sync(0xffffffffu, key == x);
    if (lane == 0) s_wave[warp] = make_int2(__popc(gt), __popc(eq));
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
    int gt_r = larger + __popc(gt & below), eq_r = equal + __popc(eq & below);
#pragma unroll
    for (int w = 0; w < kLongWarps; ++w) {
      const int2 v = s_wave[w];
      if (w < warp) { gt_r += v.x; eq_r += v.y; }
      larger += v.x;
      equal += v.y;
    }
    if (key > x || (key == x && eq_r < ties)) out[gt_r + min(eq_r, ties)] = c.c0 + i0 + tid;
    __syncthreads();
  }
}

template <int kWarps, int kPer>
cudaError_t launch_select(const SelectBlocksArgs& a, cudaStream_t stream) {
  return launch_dependent(select_blocks_kernel<kWarps, kPer>, dim3(static_cast<unsigned>(kWarps == 1 ? (a.T - 1) / kSingles + 1 : a.T)),
                          dim3(32 * (kWarps == 1 ? kSingles : kWarps)), 0, stream, a);
}

}  // namespace

cudaError_t launch_block_keys(const BlockKeysArgs& a, cudaStream_t stream) {
  const int64_t slots = (static_cast<int64_t>(a.T) >> kBlockShift) + a.B;
  const int64_t blocks = min(slots, static_cast<int64_t>(device_sm_count()) * 16);
  if (a.c.e4m3)
    return launch_dependent(block_keys_kernel<true>, dim3(static_cast<unsigned>(blocks)), dim3(KeyCfg<true>::kThreads), 0,
                            stream, a);
  return launch_dependent(block_keys_kernel<false>, dim3(static_cast<unsigned>(blocks)), dim3(KeyCfg<false>::kThreads), 0,
                          stream, a);
}

cudaError_t launch_select_blocks(const SelectBlocksArgs& a, cudaStream_t stream) {
  // More tokens than the SMs hold blocks of few warps: as few warps as the row's keys fit.
  const bool many = a.T > 8 * device_sm_count();
  if (a.W <= 1024) return many ? launch_select<1, 32>(a, stream) : launch_select<4, 8>(a, stream);
  if (a.W <= 2048) return many ? launch_select<1, 64>(a, stream) : launch_select<8, 8>(a, stream);
  if (a.W <= 8192) return launch_select<8, 32>(a, stream);
  return launch_dependent(select_long_kernel, dim3(static_cast<unsigned>(a.T)), dim3(kLongThreads), 0, stream, a);
}

}  // namespace mla
