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

// Both kernels: a warp takes four consecutive rows of the call's array at a time.
// Lane k < 4 looks up row k's place in the pages, one group ahead, so that the
// chain cu -> seq_len -> table -> row is off the path of the data; all loads of a
// group are issued before its first store, and the warp's accesses to the
// contiguous side cover whole lines.
constexpr int kGroup = 4;

// Place of token j (pool row, or -1 for padding, an invalid sequence or a bad
// page; `bad` for the last) and its position.
MLA_DEVINL int32_t token_row(const PagedAppendArgs& a, int64_t j, int32_t& pos, bool& bad) {
  pos = 0;
  if (j >= a.T) return -1;
  const int b = find_seq(a.cu, a.B, static_cast<int32_t>(j));
  bool bad_seq;
  const PagedSeq s = paged_seq(a.cu, a.seq_len, b, a.T, a.c.max_rows(), bad_seq);
  if (j < s.q0 || j >= s.q0 + s.n) return -1;
  pos = s.len - s.n + static_cast<int32_t>(j - s.q0);
  const int64_t row = a.c.row_of(b, pos);
  bad = bad || row < 0;
  return static_cast<int32_t>(row);
}

// HBM-bound: 1152 bytes in and 1152 (fp16) or 656 (e4m3) out per token.
template <bool kE4m3>
__global__ void __launch_bounds__(256, 4) paged_append_kernel(PagedAppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, a.c.max_rows(), a.err);
  const int lane = threadIdx.x & 31;
  const int64_t step = kGroup * static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  constexpr int64_t kBytes = kE4m3 ? kRowE4m3 : kRowF16;
  uint32_t run = 0;
  float amax_pe = 0.f;
  bool bad_page = false, big = false;
  int64_t j0 = kGroup * (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5));
  int32_t pos_n = 0, row_n = lane < kGroup ? token_row(a, j0 + lane, pos_n, bad_page) : -1;
  for (; j0 < a.T; j0 += step) {
    const int32_t row_l = row_n, pos_l = pos_n;
    // The latents: 64 units of 8 values a token, two passes each; then the RoPE
    // parts, 8 lanes a token.
    uint4 v[2 * kGroup], pe = make_uint4(0, 0, 0, 0);
    const uint4* src = reinterpret_cast<const uint4*>(a.c_kv + j0 * kLatent) + lane;
    const int n = static_cast<int>(min(static_cast<int64_t>(kGroup), a.T - j0));
#pragma unroll
    for (int k = 0; k < 2 * kGroup; ++k) v[k] = (k >> 1) < n ? __ldg(src + 32 * k) : make_uint4(0, 0, 0, 0);
    if ((lane >> 3) < n) pe = __ldg(reinterpret_cast<const uint4*>(a.k_pe + j0 * kRope) + lane);
    if (lane < kGroup) row_n = token_row(a, j0 + step + lane, pos_n, bad_page);
#pragma unroll
    for (int k = 0; k < 2 * kGroup; ++k) {
      const int32_t row = __shfl_sync(0xffffffffu, row_l, k >> 1);
      if (row < 0) continue;                                  // the whole warp
      uint8_t* dst = a.c.pages + row * kBytes;
      const int u = lane + 32 * (k & 1);
      if constexpr (!kE4m3) {
        run = bf16x2_absmax(bf16x2_absmax(run, v[k].x), v[k].y);
        run = bf16x2_absmax(bf16x2_absmax(run, v[k].z), v[k].w);
        *reinterpret_cast<uint4*>(dst + 16 * u) = bf16x8_to_f16(v[k]);
      } else {
        // Four lanes hold a block of 32.  The largest |x| as a bf16 pattern (a
        // NaN or infinity is the largest of all), then the scale's exponent.
        uint32_t m = bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(v[k].x & 0x7FFF7FFFu, v[k].y), v[k].z), v[k].w);
        m = max(m & 0xFFFFu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const float amax = __uint_as_float(m << 16);
        big = big || !(amax <= kE4m3MaxValue);
        const int e = e4m3_scale_exp(amax);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);   // 2^-e: the product is exact
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = bf16x2_to_f32(w[q]);
          c[q] = e4m3x2(f.x * inv, f.y * inv);
        }
        *reinterpret_cast<uint2*>(dst + 8 * u) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        // the scale bytes of lanes 4 i, packed: 8 in a pass, 4 to a word
        uint32_t sc = static_cast<uint32_t>(e + 127);
        sc |= __shfl_down_sync(0xffffffffu, sc, 4) << 8;
        sc |= __shfl_down_sync(0xffffffffu, sc, 8) << 16;
        if ((lane & 15) == 0)
          *reinterpret_cast<uint32_t*>(dst + kE4m3ScaleOff + 8 * (k & 1) + (lane >> 2)) = sc;
      }
    }
    const int32_t row = __shfl_sync(0xffffffffu, row_l, lane >> 3), pos = __shfl_sync(0xffffffffu, pos_l, lane >> 3);
    if (row >= 0)
      *reinterpret_cast<uint4*>(a.c.pages + row * kBytes + (kE4m3 ? kE4m3RopeOff : 2 * kLatent) + 16 * (lane & 7)) =
          rope8_f16(pe, pos, a.turn, lane & 7, amax_pe);
  }
  if (bad_page) record_error(a.err, MLA_ERR_INVALID_ARG);
  if (big || bf16x2_absmax_overflows(run) || f32_overflows_f16(amax_pe)) record_error(a.err, MLA_ERR_RANGE);
}

// Pool row of row j of a gather's output, or -1.
MLA_DEVINL int32_t gather_row(const PagedGatherArgs& a, int64_t j, bool& bad) {
  if (j >= a.R) return -1;
  const int b = find_seq(a.cu, a.B, static_cast<int32_t>(j));
  const int32_t c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
  if (j < c0 || j >= c1) return -1;                           // padding
  const int64_t pos = (a.row0 != nullptr ? __ldg(a.row0 + b) : 0) + (j - c0);
  const int64_t row = c0 >= 0 && pos >= 0 && pos < a.c.max_rows() ? a.c.row_of(b, pos) : -1;
  bad = bad || row < 0;
  return static_cast<int32_t>(row);
}

template <bool kOutF16>
MLA_DEVINL uint4 out8(uint4 v) {
  if (kOutF16) return v;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = f16x2_to_f32(w[q]);
    w[q] = pack_bf16x2(f.x, f.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// HBM-bound: 1152 (fp16) or 656 (e4m3) bytes in and 1152 out per row.
template <bool kE4m3, bool kOutF16>
__global__ void __launch_bounds__(256, 4) paged_gather_kernel(PagedGatherArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t step = kGroup * static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  constexpr int kUnits = kRow / 8;                            // 16-byte units of an output row
  bool bad = false;
  int64_t j0 = kGroup * (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5));
  int32_t row_n = lane < kGroup ? gather_row(a, j0 + lane, bad) : -1;
  for (; j0 < a.R; j0 += step) {
    const int32_t row_l = row_n;
    uint4* dst = reinterpret_cast<uint4*>(a.out + j0 * kRow);
    if constexpr (!kE4m3) {
      // the four rows' 288 units, 9 a lane
      uint4 v[kGroup * kUnits / 32];
      bool ok[kGroup * kUnits / 32];
#pragma unroll
      for (int k = 0; k < kGroup * kUnits / 32; ++k) {
        const int x = lane + 32 * k;
        const int32_t row = __shfl_sync(0xffffffffu, row_l, x / kUnits);
        ok[k] = row >= 0;
        v[k] = ok[k] ? __ldg(reinterpret_cast<const uint4*>(a.c.pages + static_cast<int64_t>(row) * kRowF16) + x % kUnits)
                     : make_uint4(0, 0, 0, 0);
      }
      if (lane < kGroup) row_n = gather_row(a, j0 + step + lane, bad);
#pragma unroll
      for (int k = 0; k < kGroup * kUnits / 32; ++k)
        if (ok[k]) dst[lane + 32 * k] = out8<kOutF16>(v[k]);
    } else {
      // 64 units of 8 codes a row in two passes, the scale bytes (lanes 4 r + w:
      // word w of row r's), the RoPE parts (8 lanes a row)
      uint2 v[2 * kGroup];
      uint32_t sc = 0x70707070u;
      uint4 pe = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 2 * kGroup; ++k) {
        const int32_t row = __shfl_sync(0xffffffffu, row_l, k >> 1);
        v[k] = row >= 0 ? __ldg(reinterpret_cast<const uint2*>(a.c.pages + static_cast<int64_t>(row) * kRowE4m3) + lane +
                                32 * (k & 1))
                        : make_uint2(0, 0);
      }
      const int32_t row_s = __shfl_sync(0xffffffffu, row_l, (lane >> 2) & 3);
      if (lane < 16 && row_s >= 0)
        sc = __ldg(reinterpret_cast<const uint32_t*>(a.c.pages + static_cast<int64_t>(row_s) * kRowE4m3 + kE4m3ScaleOff) +
                   (lane & 3));
      const int32_t row_p = __shfl_sync(0xffffffffu, row_l, lane >> 3);
      if (row_p >= 0)
        pe = __ldg(reinterpret_cast<const uint4*>(a.c.pages + static_cast<int64_t>(row_p) * kRowE4m3 + kE4m3RopeOff) +
                   (lane & 7));
      if (lane < kGroup) row_n = gather_row(a, j0 + step + lane, bad);
#pragma unroll
      for (int k = 0; k < 2 * kGroup; ++k) {
        // unit lane + 32 (k & 1): scale byte lane / 4 + 8 (k & 1) of the row
        const uint32_t w = __shfl_sync(0xffffffffu, sc, 4 * (k >> 1) + 2 * (k & 1) + (lane >> 4));
        const uint32_t d = e4m3_scale_f16x2((w >> (8 * ((lane >> 2) & 3))) & 0xFFu);
        uint4 o;
        e4m3x4_to_f16x4(v[k].x, d, o.x, o.y);
        e4m3x4_to_f16x4(v[k].y, d, o.z, o.w);
        if (__shfl_sync(0xffffffffu, row_l, k >> 1) >= 0) dst[(k >> 1) * kUnits + lane + 32 * (k & 1)] = out8<kOutF16>(o);
      }
      if (row_p >= 0) dst[(lane >> 3) * kUnits + kLatent / 8 + (lane & 7)] = out8<kOutF16>(pe);
    }
  }
  if (blockIdx.x == 0) {
    // sequences whose rows leave the output (here, cu is in the cache)
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
      const int32_t c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
      bad = bad || c0 < 0 || c1 < c0 || c1 > a.R;
    }
  }
  if (bad) record_error(a.err, MLA_ERR_INVALID_ARG);
}

// Four blocks of 256 threads fit an SM.
unsigned row_blocks(int64_t n) {
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 4;
  return static_cast<unsigned>(max(static_cast<int64_t>(1), min(cap, (n + 8 * kGroup - 1) / (8 * kGroup))));
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  auto kern = a.c.e4m3 ? paged_append_kernel<true> : paged_append_kernel<false>;
  return launch_dependent(kern, dim3(row_blocks(a.T)), dim3(256), 0, stream, a);
}

cudaError_t launch_paged_gather(const PagedGatherArgs& a, bool out_f16, cudaStream_t stream) {
  auto kern = a.c.e4m3 ? (out_f16 ? paged_gather_kernel<true, true> : paged_gather_kernel<true, false>)
                       : (out_f16 ? paged_gather_kernel<false, true> : paged_gather_kernel<false, false>);
  return launch_dependent(kern, dim3(row_blocks(a.R)), dim3(256), 0, stream, a);
}

}  // namespace mla
