// The paged latent cache: row formats, the sequence table, page lookup, and
// the launchers of the paged operators (append, gather, attention).
#pragma once

#include "common.cuh"

namespace mla {

// An e4m3 row: 512 one-byte codes, 64 fp16 RoPE values, 16 scale bytes (one
// for 32 codes).  656 = 41 x 16, so every row starts on a 16-byte boundary.
constexpr int kRowE4m3 = 656;
constexpr int kRowF16 = 2 * kRow;             // 1152 bytes
constexpr int kE4m3RopeOff = kLatent;         // byte offset of the RoPE part
constexpr int kE4m3ScaleOff = kLatent + 2 * kRope;
constexpr int kE4m3MinExp = -15, kE4m3MaxExp = 7;   // scales 2^-15 .. 2^7
constexpr float kE4m3MaxValue = 57344.f;      // 448 x 2^7, the largest value an e4m3 row holds

struct PagedCache {
  uint8_t* pages;            // [n_pages][page_size] rows
  const int32_t* table;      // [B][table_stride] page ids
  int64_t table_stride;
  int32_t max_pages;         // entries of a table row that may be read
  int32_t n_pages;
  int32_t page_shift;        // log2(page_size)
  bool e4m3;

  MLA_DEVINL int64_t row_bytes() const { return e4m3 ? kRowE4m3 : kRowF16; }
  // Rows a table row can name; positions stay clear of 2^31 when they are rounded up to tiles.
  MLA_DEVINL int64_t max_rows() const {
    return min(static_cast<int64_t>(max_pages) << page_shift, static_cast<int64_t>(INT32_MAX - 4096));
  }
  // Row of `pages` that holds position p (0 <= p < max_rows()) of sequence b,
  // or -1 if the table names no page of the cache there.
  MLA_DEVINL int64_t row_of(int b, int64_t p) const {
    const int32_t id = __ldg(table + b * table_stride + (p >> page_shift));
    if (id < 0 || id >= n_pages) return -1;
    return (static_cast<int64_t>(id) << page_shift) + (p & ((1 << page_shift) - 1));
  }
};

// Sequence b of a batch: its new tokens are rows [q0, q0 + n) of the call's
// token arrays and the last n of its `len` cache rows.
struct PagedSeq {
  int32_t q0, n, len;
};

// n = 0 for a sequence without new tokens and for an invalid one (new tokens
// outside [0, T), more of them than cache rows, more rows than its table row
// can name); `bad` says which.
MLA_DEVINL PagedSeq paged_seq(const int32_t* cu, const int32_t* seq_len, int b, int32_t T, int64_t max_rows,
                              bool& bad) {
  PagedSeq s;
  s.q0 = __ldg(cu + b);
  const int32_t q1 = __ldg(cu + b + 1);
  s.len = __ldg(seq_len + b);
  bad = s.q0 < 0 || q1 < s.q0 || q1 > T || s.len < 0 || s.len > max_rows || (!(q1 < s.q0) && q1 - s.q0 > s.len);
  s.n = bad ? 0 : q1 - s.q0;
  return s;
}

// The largest b in [0, B) with cu[b] <= j (0 if there is none): the sequence
// that holds token j when cu does not decrease.
MLA_DEVINL int find_seq(const int32_t* cu, int B, int32_t j) {
  int lo = 0, hi = B;                          // cu[lo] <= j < cu[hi], taking cu[B] as infinite
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (__ldg(cu + m) <= j) lo = m; else hi = m;
  }
  return lo;
}

// Record the batch's invalid sequences (one block of a launch calls it).
MLA_DEVINL void record_bad_seqs(const int32_t* cu, const int32_t* seq_len, int B, int32_t T, int64_t max_rows,
                                int* err) {
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    bool bad;
    (void)paged_seq(cu, seq_len, b, T, max_rows, bad);
    if (bad) record_error(err, MLA_ERR_INVALID_ARG);
  }
}

struct PagedAppendArgs {
  PagedCache c;
  const uint16_t* c_kv;      // bf16 [T][512]
  const uint16_t* k_pe;      // bf16 [T][64], not yet rotated
  const int32_t* cu;         // [B + 1]
  const int32_t* seq_len;    // [B]
  int32_t B, T;
  int* err;
  uint64_t turn[kRope / 2];  // turns per position of pair i, as 0.64 fixed point
};

struct PagedGatherArgs {
  PagedCache c;
  const int32_t* row0;       // [B] or null
  const int32_t* cu;         // [B + 1]
  int32_t B, R;
  uint16_t* out;             // bf16 or fp16 [R][576]
  int* err;
};

struct PagedAttnArgs {
  PagedCache c;
  const uint16_t* q_lat;     // fp16 [T][H][512]
  const uint16_t* q_pe;      // bf16 [T][H][64]
  const int32_t* cu;         // [B + 1]
  const int32_t* seq_len;    // [B]
  int32_t B, T, H;
  int32_t window;            // 0: the whole context
  int32_t n_sink;
  float scale_log2;          // softmax scale * log2(e)
  uint16_t* o_lat;           // fp16 [T][H][512]
  void* workspace;           // paged_attn_workspace_bytes()
  int* err;
  uint32_t wait_us;
};

// 2^(s - 127) for a scale byte s in [112, 134] as fp16, in both halves (2^-15, s =
// 112, is the subnormal 0x0200).
MLA_DEVINL uint32_t e4m3_scale_f16x2(uint32_t s) { return max((s - 112u) << 10, 0x0200u) * 0x00010001u; }

// Two e4m3 codes (the low 16 bits of c) to two fp16 values (exact).
MLA_DEVINL uint32_t e4m3x2_to_f16x2(uint32_t c) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(c));
  return r;
}

// Four e4m3 codes times the scale d (in both halves): four fp16 values, exact.
MLA_DEVINL void e4m3x4_to_f16x4(uint32_t c, uint32_t d, uint32_t& lo, uint32_t& hi) {
  const uint32_t x0 = e4m3x2_to_f16x2(c & 0xFFFFu), x1 = e4m3x2_to_f16x2(c >> 16);
  const __half2 s = *reinterpret_cast<const __half2*>(&d);
  const __half2 r0 = __hmul2(*reinterpret_cast<const __half2*>(&x0), s);
  const __half2 r1 = __hmul2(*reinterpret_cast<const __half2*>(&x1), s);
  lo = *reinterpret_cast<const uint32_t*>(&r0);
  hi = *reinterpret_cast<const uint32_t*>(&r1);
}

// A launch that may begin while the kernel before it in the stream finishes (the
// kernel waits with griddepcontrol.wait before its first access to global memory).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Rows of 16-bit elements in groups of eight, in chunks of 64 elements (dims:
// element, row of the group, chunk, group), with 128-byte swizzle.
cudaError_t make_tmap_row_groups(CUtensorMap* map, const void* base, uint64_t groups, uint64_t chunks,
                                 uint64_t row_bytes, uint32_t box_groups, uint32_t box_chunks);

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream);
cudaError_t launch_paged_gather(const PagedGatherArgs& a, bool out_f16, cudaStream_t stream);
size_t paged_attn_workspace_bytes();
cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream);

}  // namespace mla
