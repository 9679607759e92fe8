// The paged cache's writer (moe_kv_append): token l of request b goes to position seq_lens[b] - L + l, in the
// cache's own format.  A copy with a quantiser in it: each thread takes eight columns of one head of one token
// (a 16-byte load; four neighbouring lanes hold one MX block), looks its page up and stores 16 bytes of bf16 or
// 8 bytes of E4M3.  The load of the new values does not wait for the page lookup.
// Memory-bound for prompts, latency-bound (length -> page -> store) for a step's few rows.
#include <algorithm>

#include "moe_decode_device.cuh"

namespace moe {

namespace {

template <bool MX>
__global__ void __launch_bounds__(256) kv_append_kernel(const moe_kv_cache_t c, const __nv_bfloat16* __restrict__ k_new,
                                                        int64_t k_stride, const __nv_bfloat16* __restrict__ v_new,
                                                        int64_t v_stride, int L, int64_t n_units, PageDiv pd) {
  pdl_trigger();
  pdl_wait();
  const int cols = c.head_dim >> 3;  // 8 or 16 threads a head, a power of two
  // unit = ((row * 2 + (0: k, 1: v)) * heads + head) * cols + column group.  n_units is a multiple of 8 and the
  // stride of the loop of 256, so the four lanes of an MX block leave the loop together; the shuffles below
  // name only those lanes.
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t quad = 0xFu << (lane & ~3u);
  for (int64_t u = blockIdx.x * 256ll + threadIdx.x; u < n_units; u += gridDim.x * 256ll) {
    const int64_t hr = u / cols;
    const int col = (int)(u - hr * cols) * 8;
    const int64_t kvrow = hr / c.n_kv_heads;
    const int head = (int)(hr - kvrow * c.n_kv_heads);
    const bool is_v = kvrow & 1;
    const int64_t row = kvrow >> 1;
    const __nv_bfloat16* src = is_v ? v_new + row * v_stride : k_new + row * k_stride;
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(src + head * c.head_dim + col));
    const int b = (int)(row / L), l = (int)(row - (int64_t)b * L);
    const int pos = seq_len_of(c, b) - L + l;
    int page = -1, prow = 0;
    if (pos >= 0) {
      const int j = page_of(pos, pd, c.page_size, &prow);
      page = __ldg(c.block_table + (int64_t)b * c.max_pages + j);
      if (page < 0 || page >= c.n_pages) {
        set_status(c.status, MOE_KV_BAD_PAGE);
        page = -1;
      }
    }
    const int64_t at = page * c.page_stride + prow * c.row_stride + head * c.head_stride + col;
    if (!MX) {
      if (page >= 0) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? c.v : c.k) + at) = raw;
    } else {
      float v[8];
      bf16x8_to_f32(raw, v);
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
      amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 2));
      const int e = mxfp8_block_exp(amax);
      if (page >= 0) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + at) = e4m3_8(v, exp2_neg_int(e));
        if ((lane & 3) == 0) (is_v ? c.v_s : c.k_s)[at >> 5] = (uint8_t)(e + 127);
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
  if (L == 0 || c.n_seqs == 0 || c.max_pages == 0) return MOE_OK;
  if (!k_new || !v_new) return decode_fail(MOE_ERR_INVALID_ARG, "moe_kv_append: k_new or v_new is NULL");
  st = check_device(nullptr);
  if (st != MOE_OK) return st;
  const int64_t units = (int64_t)c.n_seqs * L * 2 * c.n_kv_heads * (c.head_dim / 8);
  const dim3 grid((unsigned)std::min<int64_t>((units + 255) / 256, 152 * 64));
  const PageDiv pd = page_div((uint32_t)c.page_size);
  const cudaError_t e = launch_pdl(c.format == MOE_KV_MXFP8 ? kv_append_kernel<true> : kv_append_kernel<false>, grid,
                                   dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), c,
                                   static_cast<const __nv_bfloat16*>(k_new), k_stride,
                                   static_cast<const __nv_bfloat16*>(v_new), v_stride, (int)L, units, pd);
  if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "moe_kv_append: %s", cudaGetErrorString(e));
  return MOE_OK;
}
