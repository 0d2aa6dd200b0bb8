// Attention of a batch's new tokens over a paged latent cache.
#include "kernels.cuh"
#include "paged.cuh"

namespace mla {
namespace {

constexpr int kQ = 16, kK = 32;                  // query rows (heads of one token) and keys of a tile
constexpr int kSmem = (kQ + kK) * kRow * 4 + kQ * kK * 4;

MLA_DEVINL float e4m3_to_f32(uint32_t c) {
  const uint32_t e = (c >> 3) & 15u, m = c & 7u;
  const float v = e == 0 ? static_cast<float>(m) * 0x1p-9f : __uint_as_float(((e + 120u) << 23) | (m << 20));
  return (c & 128u) ? -v : v;
}

// A block per 16 heads of a token; keys in tiles of 32, all in fp32.
__global__ void __launch_bounds__(256) paged_attn_kernel(PagedAttnArgs a) {
  extern __shared__ float sm[];
  float* q = sm;
  float* k = q + kQ * kRow;
  float* p = k + kK * kRow;
  if (blockIdx.x == 0) record_bad_seqs(a.cu, a.seq_len, a.B, a.T, a.c.max_rows(), a.err);
  const int64_t rho = static_cast<int64_t>(blockIdx.x) * kQ;
  const int32_t tok = static_cast<int32_t>(rho / a.H);
  const int b = find_seq(a.cu, a.B, tok);
  bool bad;
  const PagedSeq s = paged_seq(a.cu, a.seq_len, b, a.T, a.c.max_rows(), bad);
  if (tok < s.q0 || tok >= s.q0 + s.n) return;
  const int32_t pos = s.len - s.n + (tok - s.q0);
  const int32_t wlo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  for (int i = threadIdx.x; i < kQ * kRow; i += 256) {
    const int r = i / kRow, c = i % kRow;
    q[i] = c < kLatent ? f16_to_f32(a.q_lat[(rho + r) * kLatent + c]) : bf16_to_f32(a.q_pe[(rho + r) * kRope + c - kLatent]);
  }
  const int row = threadIdx.x >> 4, part = threadIdx.x & 15;     // 16 threads per query row
  float o[32], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = 0.f;
  for (int32_t j0 = 0; j0 <= pos; j0 += kK) {
    if (j0 + kK <= wlo && j0 >= a.n_sink) continue;
    __syncthreads();
    for (int i = threadIdx.x; i < kK * kRow; i += 256) {
      const int r = i / kRow, c = i % kRow;
      const int32_t j = j0 + r;
      float v = 0.f;
      if (j <= pos && (j >= wlo || j < a.n_sink)) {
        const int64_t cr = a.c.row_of(b, j);
        if (cr < 0) {
          record_error(a.err, MLA_ERR_INVALID_ARG);
        } else {
          const uint8_t* src = a.c.pages + cr * a.c.row_bytes();
          if (!a.c.e4m3)
            v = f16_to_f32(reinterpret_cast<const uint16_t*>(src)[c]);
          else if (c >= kLatent)
            v = f16_to_f32(reinterpret_cast<const uint16_t*>(src + kE4m3RopeOff)[c - kLatent]);
          else
            v = e4m3_to_f32(src[c]) * __uint_as_float(static_cast<uint32_t>(src[kE4m3ScaleOff + (c >> 5)]) << 23);
        }
      }
      k[i] = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kQ * kK; i += 256) {
      const int r = i / kK, c = i % kK;
      float x = 0.f;
      for (int d = 0; d < kRow; ++d) x = fmaf(q[r * kRow + d], k[c * kRow + d], x);
      const int32_t j = j0 + c;
      p[i] = j <= pos && (j >= wlo || j < a.n_sink) ? x * a.scale_log2 : -INFINITY;
    }
    __syncthreads();
    float mx = m;
    for (int c = 0; c < kK; ++c) mx = fmaxf(mx, p[row * kK + c]);
    const float base = mx == -INFINITY ? 0.f : mx, alpha = exp2f(m - base);
    m = mx;
    l *= alpha;
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] *= alpha;
    for (int c = 0; c < kK; ++c) {
      const float w = exp2f(p[row * kK + c] - base);
      l += w;
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = fmaf(w, k[c * kRow + part + 16 * e], o[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 32; ++e) a.o_lat[(rho + row) * kLatent + part + 16 * e] = f32_to_f16(o[e] / l);
}

}  // namespace

size_t paged_attn_workspace_bytes() { return 256; }

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<<<static_cast<unsigned>(static_cast<int64_t>(a.T) * a.H / kQ), 256, kSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
