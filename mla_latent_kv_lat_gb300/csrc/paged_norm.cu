// The projections' outputs of new tokens made ready for attention, in one pass:
//
//   queries  q[t][h] (192) -> x = q / sqrt(mean(q^2) + eps) * w   (with a weight), else x = q
//            q_nope = x[0..127], q_pe = RoPE(x[128..191], position)
//   keys     kv[t] = [latent 512 | rope 64] -> the token's row in its page:
//            [latent / sqrt(mean(latent^2) + eps) * w | RoPE(rope, position)]
//
// Sums of squares, the rotation and all products are fp32; each output value is
// rounded once, to bf16 (queries) or to the page's type.
#include "kernels.cuh"
#include "paged.cuh"

namespace mla {
namespace {

constexpr int kHead = kNope + kRope;          // 192

// Sine and cosine of pos * turn[4 l8 + q] turns, q < 4 (as the append has it: the
// fraction of a turn is the low 64 bits of the integer product).
MLA_DEVINL void rope_angles(int32_t pos, const uint64_t* turn, int l8, float (&sn)[4], float (&cs)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint64_t f = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * turn[4 * l8 + q];
    sincospif(static_cast<float>(static_cast<uint32_t>(f >> 32)) * 0x1p-31f, &sn[q], &cs[q]);
  }
}

MLA_DEVINL void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = bf16x2_to_f32(w[q]);
    x[2 * q] = f.x;
    x[2 * q + 1] = f.y;
  }
}

// Position of token j (a warp's), or -1 for padding and invalid sequences; b its sequence.
MLA_DEVINL int32_t token_pos(const NormAppendArgs& a, int32_t j, int& b) {
  b = find_seq_warp(a.cu, a.B, j);
  bool bad;
  const PagedSeq s = paged_seq(a.cu, a.seq_len, b, a.T, a.c.max_rows(), bad);
  return j >= s.q0 && j < s.q0 + s.n ? s.len - s.n + (j - s.q0) : -1;
}

// A warp's task: one token's row, or 4 `iters` heads of one token's queries.  Eight
// lanes share a head, three units each: two of the part that stays, one to rotate,
// so that a head's sum takes three exchanges and every access is 128 bytes wide.
// The angles are computed once a task: a head's own would cost more than its loads.
// HBM-bound: 8192 tokens of 128 heads into e4m3 rows 122 us, 6.7 TB/s; 64 tokens into
// fp16 rows 3.1 us, a launch and the lookups.
template <bool kE4m3>
__global__ void __launch_bounds__(256, 4) norm_append_kernel(const __grid_constant__ NormAppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, a.c.max_rows(), a.err);
  const int lane = threadIdx.x & 31, l8 = lane & 7;
  int64_t task = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int groups = (a.H / 4 + a.iters - 1) / a.iters;       // of a token's heads
  if (task >= a.T) {
    // ------------------------------ queries ----------------------------------
    task -= a.T;
    const int64_t t = task / groups;
    if (t >= a.T) return;
    const int g0 = static_cast<int>(task - t * groups) * a.iters, g1 = min(g0 + a.iters, a.H / 4);
    const uint16_t* src = a.q + t * a.q_token + (lane >> 3) * a.q_head + 8 * l8;
    auto load = [&](int g, uint4 (&v)[3]) {
#pragma unroll
      for (int j = 0; j < 3; ++j) v[j] = __ldg(reinterpret_cast<const uint4*>(src + 4 * g * a.q_head + 64 * j));
    };
    uint4 v[3];
    load(g0, v);
    int b;
    const int32_t pos = token_pos(a, static_cast<int32_t>(t), b);
    if (pos < 0) return;
    float sn[4], cs[4];
    rope_angles(pos, a.turn, l8, sn, cs);
    for (int g = g0; g < g1; ++g) {
      uint4 n[3];
      if (g + 1 < g1) load(g + 1, n);
      float x[3][8];
#pragma unroll
      for (int j = 0; j < 3; ++j) unpack8(v[j], x[j]);
      if (a.q_weight != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 3; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[j][e], x[j][e], ss);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / kHead) + a.eps);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          float w[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(a.q_weight + 8 * l8 + 64 * j)), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[j][e] = x[j][e] * r * w[e];
        }
      }
      const int64_t head = t * a.H + 4 * g + (lane >> 3);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint4*>(a.q_nope + head * kNope + 64 * j + 8 * l8) =
            make_uint4(pack_bf16x2(x[j][0], x[j][1]), pack_bf16x2(x[j][2], x[j][3]), pack_bf16x2(x[j][4], x[j][5]),
                       pack_bf16x2(x[j][6], x[j][7]));
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float u = x[2][2 * q], y = x[2][2 * q + 1];
        w[q] = pack_bf16x2(u * cs[q] - y * sn[q], u * sn[q] + y * cs[q]);
      }
      *reinterpret_cast<uint4*>(a.q_pe + head * kRope + 8 * l8) = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int j = 0; j < 3; ++j) v[j] = n[j];
    }
    return;
  }
  // --------------------------------- keys --------------------------------------
  // 64 units of latents, two a lane; the rope part in lanes 0-7.
  const uint16_t* src = a.kv + task * a.kv_token;
  uint4 v[2], pe = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < 2; ++k) v[k] = __ldg(reinterpret_cast<const uint4*>(src) + lane + 32 * k);
  if (lane < 8) pe = __ldg(reinterpret_cast<const uint4*>(src + kLatent) + lane);
  int b;
  const int32_t pos = token_pos(a, static_cast<int32_t>(task), b);
  if (pos < 0) return;
  const int64_t row = a.c.row_of(b, pos);
  if (row < 0) {
    if (lane == 0) record_error(a.err, MLA_ERR_INVALID_ARG);
    return;
  }
  float x[2][8], ss = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    unpack8(v[k], x[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[k][e], x[k][e], ss);
  }
  const float r = rsqrtf(warp_sum(ss) * (1.f / kLatent) + a.eps);
  uint8_t* dst = a.c.pages + row * (kE4m3 ? kRowE4m3 : kRowF16);
  float amax = 0.f;
  bool big = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int u = lane + 32 * k;
    float w[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(a.kv_weight) + u), w);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[k][e] = x[k][e] * r * w[e];
      m = f32_absmax(m, x[k][e]);
    }
    if constexpr (!kE4m3) {
      amax = f32_absmax(amax, m);
      *reinterpret_cast<uint4*>(dst + 16 * u) = make_uint4(pack_f16x2(x[k][0], x[k][1]), pack_f16x2(x[k][2], x[k][3]),
                                                           pack_f16x2(x[k][4], x[k][5]), pack_f16x2(x[k][6], x[k][7]));
    } else {
      // four lanes hold a block of 32 (as the append quantises it)
      m = f32_absmax(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = f32_absmax(m, __shfl_xor_sync(0xffffffffu, m, 2));
      big = big || !(m <= kE4m3MaxValue);
      const int e = e4m3_scale_exp(m);
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);   // 2^-e: the product is exact
      uint32_t c[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) c[q] = e4m3x2(x[k][2 * q] * inv, x[k][2 * q + 1] * inv);
      *reinterpret_cast<uint2*>(dst + 8 * u) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      uint32_t sc = static_cast<uint32_t>(e + 127);
      sc |= __shfl_down_sync(0xffffffffu, sc, 4) << 8;
      sc |= __shfl_down_sync(0xffffffffu, sc, 8) << 16;
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(dst + kE4m3ScaleOff + 8 * k + (lane >> 2)) = sc;
    }
  }
  if (lane < 8) {
    float sn[4], cs[4], y[8];
    rope_angles(pos, a.turn, lane, sn, cs);
    unpack8(pe, y);
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float p0 = y[2 * q] * cs[q] - y[2 * q + 1] * sn[q], p1 = y[2 * q] * sn[q] + y[2 * q + 1] * cs[q];
      amax = f32_absmax(f32_absmax(amax, p0), p1);
      w[q] = pack_f16x2(p0, p1);
    }
    *reinterpret_cast<uint4*>(dst + (kE4m3 ? kE4m3RopeOff : 2 * kLatent) + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (big || f32_overflows_f16(amax)) record_error(a.err, MLA_ERR_RANGE);
}

}  // namespace

cudaError_t launch_norm_append(const NormAppendArgs& args, cudaStream_t stream) {
  NormAppendArgs a = args;
  // Few tokens: a warp for every four heads.  Many: up to 32 heads a warp, so that a
  // token's angles are computed for more of its heads, while every SM still gets 64 warps.
  const int64_t quads = static_cast<int64_t>(a.T) * (a.H / 4);
  const int64_t warps = static_cast<int64_t>(device_sm_count()) * 64;
  a.iters = static_cast<int32_t>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(8), quads / warps)));
  const int64_t groups = (a.H / 4 + a.iters - 1) / a.iters;
  const int64_t blocks = (a.T + a.T * groups + 7) / 8;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_dependent(a.c.e4m3 ? norm_append_kernel<true> : norm_append_kernel<false>,
                          dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, a);
}

}  // namespace mla
