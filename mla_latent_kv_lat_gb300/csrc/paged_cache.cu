// Writing new tokens' rows into a paged latent cache and reading rows back.
#include "kernels.cuh"
#include "paged.cuh"

namespace mla {
namespace {

// Rotate this lane's 8 RoPE values (pairs 4 l8 .. 4 l8 + 3) by pos * turn[i]
// turns: the fraction of a turn is the low 64 bits of the integer product
// (exact), its top 32 bits the angle for sincospif; fp32, rounded once to the
// pages' fp16.
MLA_DEVINL uint4 rope8_f16(uint4 v, int32_t pos, const uint64_t* turn, int l8, float& amax) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint64_t f = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * turn[4 * l8 + q];
    float sn, cs;
    sincospif(static_cast<float>(static_cast<uint32_t>(f >> 32)) * 0x1p-31f, &sn, &cs);
    const float2 x = bf16x2_to_f32(w[q]);
    const float a = x.x * cs - x.y * sn, b = x.x * sn + x.y * cs;
    amax = f32_absmax(f32_absmax(amax, a), b);
    w[q] = pack_f16x2(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

MLA_DEVINL uint4 bf16x8_to_f16(uint4 v) {
  uint4 o;
  float2 f;
  f = bf16x2_to_f32(v.x); o.x = pack_f16x2(f.x, f.y);
  f = bf16x2_to_f32(v.y); o.y = pack_f16x2(f.x, f.y);
  f = bf16x2_to_f32(v.z); o.z = pack_f16x2(f.x, f.y);
  f = bf16x2_to_f32(v.w); o.w = pack_f16x2(f.x, f.y);
  return o;
}

// Exponent e of the smallest scale 2^e in [2^-15, 2^7] with amax <= 448 * 2^e.
// 448 = 1.75 * 2^8, so with amax = m * 2^k (m in [1, 2)) it is k - 8 for
// m <= 1.75 and k - 7 otherwise.  (A subnormal amax clamps to -15.)
MLA_DEVINL int e4m3_scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(kE4m3MinExp, min(kE4m3MaxExp, e));
}

// Two fp32 values to two e4m3 codes (nearest even, saturating).
MLA_DEVINL uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// A warp per token: the latent values in two passes of 256 (8 per lane), then
// the 64 RoPE values on lanes 0-7.
__global__ void __launch_bounds__(256) paged_append_kernel(PagedAppendArgs a) {
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, a.c.max_rows(), a.err);
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  uint32_t run = 0;
  float amax_pe = 0.f;
  bool bad_page = false, big = false;
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); j < a.T; j += warps) {
    const int b = find_seq(a.cu, a.B, static_cast<int32_t>(j));
    bool bad;
    const PagedSeq s = paged_seq(a.cu, a.seq_len, b, a.T, a.c.max_rows(), bad);
    if (j < s.q0 || j >= s.q0 + s.n) continue;              // padding, or an invalid sequence
    const int32_t pos = s.len - s.n + static_cast<int32_t>(j - s.q0);
    const int64_t row = a.c.row_of(b, pos);
    if (row < 0) {
      bad_page = true;
      continue;
    }
    uint8_t* dst = a.c.pages + row * a.c.row_bytes();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.c_kv + j * kLatent + 256 * h + 8 * lane));
      if (!a.c.e4m3) {
        run = bf16x2_absmax(bf16x2_absmax(run, v.x), v.y);
        run = bf16x2_absmax(bf16x2_absmax(run, v.z), v.w);
        *reinterpret_cast<uint4*>(dst + 2 * (256 * h + 8 * lane)) = bf16x8_to_f16(v);
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float x[8], amax = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = bf16x2_to_f32(w[q]);
          x[2 * q] = f.x;
          x[2 * q + 1] = f.y;
          amax = f32_absmax(f32_absmax(amax, f.x), f.y);
        }
        // a NaN stays in the maximum (max.NaN in f32_absmax) and is reported
        amax = f32_absmax(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = f32_absmax(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        big = big || !(amax <= kE4m3MaxValue);
        const int e = e4m3_scale_exp(amax);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);   // 2^-e: the product is exact
        uint2 c;
        c.x = e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16);
        c.y = e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16);
        *reinterpret_cast<uint2*>(dst + 256 * h + 8 * lane) = c;
        if ((lane & 3) == 0) dst[kE4m3ScaleOff + 8 * h + (lane >> 2)] = static_cast<uint8_t>(e + 127);
      }
    }
    if (lane < 8) {
      const uint4 v = rope8_f16(__ldg(reinterpret_cast<const uint4*>(a.k_pe + j * kRope + 8 * lane)), pos, a.turn,
                                lane, amax_pe);
      *reinterpret_cast<uint4*>(dst + (a.c.e4m3 ? kE4m3RopeOff : 2 * kLatent) + 16 * lane) = v;
    }
  }
  if (bad_page) record_error(a.err, MLA_ERR_INVALID_ARG);
  if (big || bf16x2_absmax_overflows(run) || f32_overflows_f16(amax_pe)) record_error(a.err, MLA_ERR_RANGE);
}

// A warp per row, 8 values per lane and pass.
template <bool kOutF16>
__global__ void __launch_bounds__(256) paged_gather_kernel(PagedGatherArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  bool bad = false;
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); j < a.R; j += warps) {
    const int b = find_seq(a.cu, a.B, static_cast<int32_t>(j));
    const int32_t c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
    if (j < c0 || j >= c1) continue;                          // padding
    const int64_t pos = (a.row0 != nullptr ? __ldg(a.row0 + b) : 0) + (j - c0);
    const int64_t row = c0 >= 0 && pos >= 0 && pos < a.c.max_rows() ? a.c.row_of(b, pos) : -1;
    if (row < 0) {
      bad = true;
      continue;
    }
    const uint8_t* src = a.c.pages + row * a.c.row_bytes();
    uint4* dst = reinterpret_cast<uint4*>(a.out + j * kRow);
#pragma unroll
    for (int u = lane; u < kRow / 8; u += 32) {
      uint32_t w[4];
      if (!a.c.e4m3 || u >= kLatent / 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + (a.c.e4m3 ? kE4m3RopeOff + 16 * (u - kLatent / 8)
                                                                             : 16 * u)));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(src + 8 * u));
        const uint32_t d = e4m3_scale_f16x2(__ldg(src + kE4m3ScaleOff + (u >> 2)));
        e4m3x4_to_f16x4(c.x, d, w[0], w[1]);
        e4m3x4_to_f16x4(c.y, d, w[2], w[3]);
      }
      if (!kOutF16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = f16x2_to_f32(w[q]);
          w[q] = pack_bf16x2(f.x, f.y);
        }
      }
      dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (bad) record_error(a.err, MLA_ERR_INVALID_ARG);
}

unsigned warp_blocks(int64_t n) {
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 8;
  return static_cast<unsigned>(max(static_cast<int64_t>(1), min(cap, (n + 7) / 8)));
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  paged_append_kernel<<<warp_blocks(a.T), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_paged_gather(const PagedGatherArgs& a, bool out_f16, cudaStream_t stream) {
  if (out_f16)
    paged_gather_kernel<true><<<warp_blocks(a.R), 256, 0, stream>>>(a);
  else
    paged_gather_kernel<false><<<warp_blocks(a.R), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
