// What block-sparse attention needs beside its scores: the mean row of each block of
// 64 positions, and the choice of a token's blocks from their scores.
#include "kernels.cuh"
#include "paged.cuh"

namespace mla {
namespace {

// ---------------------------------------------------------------------------
// Mean rows.  A block that the new tokens complete (its last position is one of
// theirs) gets keys[page][block of the page] = mean of its 64 rows, summed in fp32 and
// rounded once.  Slots: sequence b's completed blocks get slots cu[b] / 64 + b, ...
// (n new tokens complete at most ceil(n / 64) blocks, so ranges do not overlap).
// HBM-bound: a block of threads reads a block's 64 rows whole, each thread 16 bytes
// of every kGroups-th row, all of them under way at once.
// ---------------------------------------------------------------------------
template <bool kE4m3>
struct KeyCfg {
  static constexpr int kUnits = kE4m3 ? 40 : 72;        // 16-byte units of a row's values
  static constexpr int kGroups = kE4m3 ? 8 : 4;         // row groups
  static constexpr int kThreads = kUnits * kGroups;     // 320, 288
  static constexpr int kRowsEach = kBlockRows / kGroups;
};

MLA_DEVINL int64_t key_slot(const BlockKeysArgs& a, int b) {
  return (max(0, min(a.T, __ldg(a.cu + b))) >> kBlockShift) + b;
}

template <bool kE4m3>
__global__ void __launch_bounds__(KeyCfg<kE4m3>::kThreads) block_keys_kernel(const BlockKeysArgs a) {
  using C = KeyCfg<kE4m3>;
  __shared__ float part[C::kGroups][kRow];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, a.c.max_rows(), a.err);
  const int unit = threadIdx.x % C::kUnits, grp = threadIdx.x / C::kUnits;
  const int64_t slots = (a.T >> kBlockShift) + a.B;
  for (int64_t g = blockIdx.x; g < slots; g += gridDim.x) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (key_slot(a, m) <= g) lo = m; else hi = m;
    }
    bool bad;
    const PagedSeq s = paged_seq(a.cu, a.seq_len, lo, a.T, a.c.max_rows(), bad);
    const int64_t j = ((s.len - s.n) >> kBlockShift) + (g - key_slot(a, lo));     // the sequence's block
    if (s.n == 0 || g < key_slot(a, lo) || j >= (s.len >> kBlockShift)) continue;
    const int64_t row0 = a.c.row_of(lo, j << kBlockShift);
    if (row0 < 0) {
      if (threadIdx.x == 0) record_error(a.err, MLA_ERR_INVALID_ARG);
      continue;
    }
    constexpr int kBytes = kE4m3 ? kRowE4m3 : kRowF16;
    const uint8_t* src = a.c.pages + row0 * kBytes;
    if constexpr (!kE4m3) {
      uint4 v[C::kRowsEach];
#pragma unroll
      for (int r = 0; r < C::kRowsEach; ++r)
        v[r] = __ldg(reinterpret_cast<const uint4*>(src + (grp + C::kGroups * r) * kBytes) + unit);
      float x[8] = {};
#pragma unroll
      for (int r = 0; r < C::kRowsEach; ++r) {
        const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = f16x2_to_f32(w[q]);
          x[2 * q] += f.x;
          x[2 * q + 1] += f.y;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e += 4)
        *reinterpret_cast<float4*>(&part[grp][8 * unit + e]) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    } else {
      // units 0-31: 16 codes each, half of a scale's block; 32-39: eight RoPE values
      uint4 v[C::kRowsEach];
      uint32_t d[C::kRowsEach];
#pragma unroll
      for (int r = 0; r < C::kRowsEach; ++r) {
        const uint8_t* row = src + (grp + C::kGroups * r) * kBytes;
        v[r] = __ldg(reinterpret_cast<const uint4*>(row) + unit);
        d[r] = unit < 32 ? __ldg(row + kE4m3ScaleOff + unit / 2) : 0u;
      }
      float x[16] = {};
#pragma unroll
      for (int r = 0; r < C::kRowsEach; ++r) {
        const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
        if (unit < 32) {
          const uint32_t sc = e4m3_scale_f16x2(d[r]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t lo2, hi2;
            e4m3x4_to_f16x4(w[q], sc, lo2, hi2);
            const float2 f = f16x2_to_f32(lo2), h = f16x2_to_f32(hi2);
            x[4 * q] += f.x;
            x[4 * q + 1] += f.y;
            x[4 * q + 2] += h.x;
            x[4 * q + 3] += h.y;
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 f = f16x2_to_f32(w[q]);
            x[2 * q] += f.x;
            x[2 * q + 1] += f.y;
          }
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
// below everything).  The key of the last one taken is found bit by bit: the largest
// x with at least R candidates of keys >= x.  One block of threads a token; its keys
// stay in registers (up to kHeld a thread; for longer rows they are read again in
// each step).  Latency-bound: 32 counts over the block, ~60 cycles each.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32, kHeld = 16;

MLA_DEVINL uint32_t score_key(float s) {
  const uint32_t u = __float_as_uint(s + 0.f);            // (-0 + 0 = 0)
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 1u;         // NaN; -inf is 0x007FFFFF
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

template <bool kHold>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const SelectBlocksArgs a) {
  __shared__ int s_cnt[2][kSelWarps];
  __shared__ int2 s_wave[kSelWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, INT32_MAX - 4096, a.err);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t = blockIdx.x;
  const int b = find_seq(a.cu, a.B, static_cast<int32_t>(t));
  bool bad;
  const PagedSeq s = paged_seq(a.cu, a.seq_len, b, a.T, INT32_MAX - 4096, bad);
  if (t < s.q0 || t >= s.q0 + s.n) return;
  const int own = (s.len - s.n + static_cast<int>(t - s.q0)) >> kBlockShift;
  int32_t* out = a.blocks + t * a.K;
  if (own >= a.W) {                      // its blocks have no scores
    if (tid == 0) {
      record_error(a.err, MLA_ERR_INVALID_ARG);
      a.counts[t] = 0;
    }
    for (int i = tid; i < a.K; i += kSelThreads) out[i] = -1;
    return;
  }
  // candidates: [c0, c1); the others up to `own` are taken as they are
  const int c1 = max(0, own - a.n_local + 1), c0 = min(a.n_sink, c1), n = c1 - c0;
  const int forced = own + 1 - n, R = min(n, a.K - forced), total = forced + R;
  const float* src = a.scores + t * a.stride + c0;
  uint32_t held[kHold ? kHeld : 1];
  if constexpr (kHold) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const int i = tid + k * kSelThreads;
      held[k] = i < n && R < n ? score_key(__ldg(src + i)) : 0u;
    }
  }
  auto key = [&](int k) -> uint32_t {    // of candidate tid + k kSelThreads (0: there is none)
    if constexpr (kHold) return held[k];
    const int i = tid + k * kSelThreads;
    return i < n ? score_key(__ldg(src + i)) : 0u;
  };
  const int steps = (n + kSelThreads - 1) / kSelThreads;
  // the largest x with at least R keys >= x, and how many keys are larger
  uint32_t x = 0;
  int above = 0;
  if (R > 0 && R < n) {
    int buf = 0;
    auto count = [&](uint32_t y) -> int {
      int c = 0;
      if constexpr (kHold) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) c += held[k] >= y;
      } else {
        for (int k = 0; k < steps; ++k) c += key(k) >= y;
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) s_cnt[buf][warp] = c;
      __syncthreads();
      c = 0;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) c += s_cnt[buf][w];
      buf ^= 1;
      return c;
    };
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t y = x | (1u << bit);
      if (count(y) >= R) x = y;
    }
    above = x == 0xFFFFFFFFu ? 0 : count(x + 1);
  }
  // written in ascending order: a wave of kSelThreads blocks at a time
  const int ties = R < n ? R - above : 0;      // of the keys equal to x, the first ones
  int taken = 0, equal = 0;                    // before this wave
  for (int i0 = 0; i0 <= own; i0 += kSelThreads) {
    const int i = i0 + tid;                    // block
    const int c = i - c0;                      // candidate
    uint32_t kx = 0;
    const bool cand = c >= 0 && c < n;
    if (cand && R < n) kx = score_key(__ldg(src + c));
    const bool sure = i <= own && (!cand || R == n || (R > 0 && kx > x));
    const bool tie = cand && R < n && R > 0 && kx == x;
    const uint32_t tie_w = __ballot_sync(0xffffffffu, tie), sure_w = __ballot_sync(0xffffffffu, sure);
    if (lane == 0) s_wave[warp] = make_int2(__popc(sure_w), __popc(tie_w));
    __syncthreads();
    int sure_b = 0, tie_b = 0, sure_all = 0, tie_all = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      const int2 v = s_wave[w];
      if (w < warp) { sure_b += v.x; tie_b += v.y; }
      sure_all += v.x;
      tie_all += v.y;
    }
    const uint32_t below = (1u << lane) - 1;
    const int sure_r = taken + sure_b + __popc(sure_w & below);          // sure ones before block i
    const int tie_r = equal + tie_b + __popc(tie_w & below);             // ties before block i
    if (sure || (tie && tie_r < ties)) {
      const int at = sure_r + min(tie_r, ties);
      if (at < a.K) out[at] = i;
    }
    taken += sure_all;
    equal += tie_all;
    __syncthreads();
  }
  for (int i = total + tid; i < a.K; i += kSelThreads) out[i] = -1;
  if (tid == 0) a.counts[t] = total;
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
  return launch_dependent(a.W <= kSelThreads * kHeld ? select_blocks_kernel<true> : select_blocks_kernel<false>,
                          dim3(static_cast<unsigned>(a.T)), dim3(kSelThreads), 0, stream, a);
}

}  // namespace mla
