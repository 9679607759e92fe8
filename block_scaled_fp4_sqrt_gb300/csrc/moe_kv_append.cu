// The paged cache's writer (moe_kv_append): token l of request b goes to position seq_lens[b] - L + l, in the
// cache's own format.  A copy with a quantiser in it: each thread takes eight columns of one head of one token, of K and
// of V (two 16-byte loads; four neighbouring lanes hold one MX block), looks their page up once and stores 16 bytes of
// bf16, 8 bytes of E4M3 or 4 bytes of E2M1 twice.  The loads of the new values do not wait for the page lookup.
// Memory-bound for prompts, latency-bound (length -> page -> store) for a step's few rows.  All index arithmetic is 32-bit
// with divisions by multiplication: with 64-bit divisions, and K and V in threads of their own, instructions were the
// bound (81 % of the issue slots, 15.2 us for a prompt of 8191 tokens, 8 heads of 128 in bf16).  Measured now: that prompt
// 7.0 us where it stays in the L2 cache, 32,000 tokens 43.7 us (6.0 TB/s), a step of 64 x 8 rows in MXFP8 2.2 us.  Into MXFP4:
// 64 x 8 rows 2.4 us, 8191 tokens from HBM 12.3 (floor 6.3; bf16 12.5, MXFP8 11.4), 32,000 tokens 39 (floor 24.6; MXFP8 36.5).
#include <algorithm>

#include "moe_decode_device.cuh"

namespace moe {

namespace {

struct AppendParams {
  moe_kv_cache_t c;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  int64_t k_stride, v_stride;
  int64_t row0;      // the call's first row (request b0, token l0) in k_new and v_new
  int b0, l0, L;
  uint32_t n_units;  // rows * heads * threads a head, below 2^31
  PageDiv page, heads, len;
};

template <int FMT>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p) {
  pdl_trigger();
  pdl_wait();
  const moe_kv_cache_t& c = p.c;
  const int log_cols = c.head_dim == 128 ? 4 : 3;  // threads a head: 16 or 8
  // unit = (row * heads + head) * cols + column group.  n_units is a multiple of 8 and the stride of the loop of 256,
  // so the four lanes of an MX block leave the loop together; the shuffles below name only those lanes.
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t quad = 0xFu << (lane & ~3u);
  for (uint32_t u = blockIdx.x * 256u + threadIdx.x; u < p.n_units; u += gridDim.x * 256u) {
    const int col = (int)(u & ((1u << log_cols) - 1u)) * 8;
    int head, l;
    const int row = page_of((int)(u >> log_cols), p.heads, c.n_kv_heads, &head);
    const int64_t src_row = p.row0 + row;
    const int src_col = head * c.head_dim + col;
    uint4 raw[2];
    raw[0] = __ldg(reinterpret_cast<const uint4*>(p.k_new + src_row * p.k_stride + src_col));
    raw[1] = __ldg(reinterpret_cast<const uint4*>(p.v_new + src_row * p.v_stride + src_col));
    const int b = p.b0 + page_of(p.l0 + row, p.len, p.L, &l);
    const int pos = seq_len_of(c, b) - p.L + l;
    int page = -1, prow = 0;
    if (pos >= 0) {
      const int j = page_of(pos, p.page, c.page_size, &prow);
      page = __ldg(c.block_table + (int64_t)b * c.max_pages + j);
      if (page < 0 || page >= c.n_pages) {
        set_status(c.status, MOE_KV_BAD_PAGE);
        page = -1;
      }
    }
    const int64_t at = page * c.page_stride + prow * c.row_stride + head * c.head_stride + col;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (FMT == MOE_KV_BF16) {
        if (page >= 0) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(i ? c.v : c.k) + at) = raw[i];
      } else {
        float v[8];
        bf16x8_to_f32(raw[i], v);
        if constexpr (FMT == MOE_KV_MXFP8) {
          float amax = 0.f;
#pragma unroll
          for (int x = 0; x < 8; ++x) amax = fmaxf(amax, fabsf(v[x]));
          amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 2));
          const int e = mxfp8_block_exp(amax);
          if (page >= 0) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(i ? c.v : c.k) + at) = e4m3_8(v, exp2_neg_int(e));
            if ((lane & 3) == 0) (i ? c.v_s : c.k_s)[at >> 5] = (uint8_t)(e + 127);
          }
        } else {
          uint32_t top = abs_max_bits(v);
          top = max(top, __shfl_xor_sync(quad, top, 1));
          top = max(top, __shfl_xor_sync(quad, top, 2));
          uint32_t codes;
          const uint8_t scale = mxfp4_quad(v, top, codes);
          if (page >= 0) {
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(i ? c.v : c.k) + (at >> 1)) = codes;
            if ((lane & 3) == 0) (i ? c.v_s : c.k_s)[at >> 5] = scale;
          }
        }
      }
    }
  }
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_kv_append(const moe_kv_cache_t* cache, const void* k_new, int64_t k_stride,
                                      const void* v_new, int64_t v_stride, int32_t L, moe_stream_t stream) {
  moe_status_t st = check_cache(cache, "moe_kv_append");
  if (st != MOE_OK) return st;
  const moe_kv_cache_t& c = *cache;
  if (L < 0) return decode_fail(MOE_ERR_INVALID_ARG, "moe_kv_append: L = %d is negative", L);
  const int64_t width = (int64_t)c.n_kv_heads * c.head_dim;
  if (!k_stride) k_stride = width;
  if (!v_stride) v_stride = width;
  if (k_stride < width || v_stride < width || k_stride % 8 || v_stride % 8)
    return decode_fail(MOE_ERR_INVALID_ARG,
                       "moe_kv_append: row strides (%lld, %lld) must be multiples of 8, at least n_kv_heads * head_dim",
                       (long long)k_stride, (long long)v_stride);
  if (!aligned_to(k_new, 16) || !aligned_to(v_new, 16))
    return decode_fail(MOE_ERR_INVALID_ARG, "moe_kv_append: k_new and v_new must be 16-byte aligned");
  if (L == 0 || c.n_seqs == 0) return MOE_OK;
  if (!k_new || !v_new) return decode_fail(MOE_ERR_INVALID_ARG, "moe_kv_append: k_new or v_new is NULL");
  if (!c.seq_lens) return decode_fail(MOE_ERR_INVALID_ARG, "moe_kv_append: seq_lens is NULL");
  st = check_device(nullptr);
  if (st != MOE_OK) return st;
  if (L > (1 << 30)) return decode_fail(MOE_ERR_UNSUPPORTED, "moe_kv_append: more than 2^30 new tokens a request");
  AppendParams p{};
  p.c = c;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.L = L;
  p.page = page_div((uint32_t)c.page_size);
  p.heads = page_div((uint32_t)c.n_kv_heads);
  p.len = page_div((uint32_t)L);
  const int64_t rows = (int64_t)c.n_seqs * L, row_units = (int64_t)c.n_kv_heads * (c.head_dim / 8);
  // A launch takes at most 2^26 rows and 2^30 units: its indexes (the grid's last stride included) stay below 2^31.
  const int64_t step = std::max<int64_t>(1, std::min<int64_t>(1 << 26, (1 << 30) / row_units));
  for (int64_t row0 = 0; row0 < rows; row0 += step) {
    p.row0 = row0;
    p.b0 = (int)(row0 / L);
    p.l0 = (int)(row0 % L);
    p.n_units = (uint32_t)(std::min(step, rows - row0) * row_units);
    const dim3 grid((p.n_units + 255) / 256 < 152 * 8 ? (p.n_units + 255) / 256 : 152 * 8);  // what the SMs hold
    auto* kernel = c.format == MOE_KV_MXFP8   ? kv_append_kernel<MOE_KV_MXFP8>
                   : c.format == MOE_KV_MXFP4 ? kv_append_kernel<MOE_KV_MXFP4>
                                              : kv_append_kernel<MOE_KV_BF16>;
    const cudaError_t e = launch_pdl(kernel, grid, dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "moe_kv_append: %s", cudaGetErrorString(e));
  }
  return MOE_OK;
}
