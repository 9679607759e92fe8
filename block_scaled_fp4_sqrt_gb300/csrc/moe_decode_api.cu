// Host-side checks shared by the decode-step operators.
#include <cstdarg>
#include <cstdio>

#include "moe_decode_internal.h"

namespace moe {

moe_status_t decode_fail(moe_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

moe_status_t check_device(int* num_sms) {
  // 0 = not asked yet, > 0 = the SM count of an sm_103 device
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  int sms = dev >= 0 && dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    int major = 0, minor = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    if (major != 10 || minor != 3)
      return decode_fail(MOE_ERR_UNSUPPORTED, "libmoe is built for sm_103a; device %d is sm_%d%d", dev, major, minor);
    if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  }
  if (num_sms) *num_sms = sms;
  return MOE_OK;
}

moe_status_t check_cache(const moe_kv_cache_t* c, const char* call) {
  if (!c) return decode_fail(MOE_ERR_INVALID_ARG, "%s: cache is NULL", call);
  if (c->format != MOE_KV_BF16 && c->format != MOE_KV_MXFP8)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: unknown cache format %d", call, c->format);
  const bool mx = c->format == MOE_KV_MXFP8;
  if (c->head_dim != 64 && c->head_dim != 128)
    return decode_fail(MOE_ERR_UNSUPPORTED, "%s: head_dim (%d) must be 64 or 128", call, c->head_dim);
  if (c->n_pages < 0 || c->page_size < 1 || c->n_kv_heads < 1 || c->n_seqs < 0 || c->max_pages < 0)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: negative size, or page_size / n_kv_heads below 1", call);
  if (c->n_kv_heads > 65535 || c->n_seqs > (1 << 20) || (int64_t)c->max_pages * c->page_size > 0x7fff0000ll ||
      (int64_t)c->n_seqs * c->n_kv_heads > (1 << 24))
    return decode_fail(MOE_ERR_UNSUPPORTED, "%s: more than 65535 heads, 2^20 requests, 2^24 request heads or 2^31 tokens a request",
                       call);
  const int64_t unit = mx ? 32 : 8;
  if (c->page_stride < 0 || c->row_stride < 0 || c->head_stride < 0 || c->page_stride % unit || c->row_stride % unit ||
      c->head_stride % unit)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: cache strides must be non-negative multiples of %d", call, (int)unit);
  if (c->n_seqs > 0 && c->max_pages > 0) {
    if (!c->block_table || !c->seq_lens)
      return decode_fail(MOE_ERR_INVALID_ARG, "%s: block_table or seq_lens is NULL", call);
    if (c->n_pages > 0 && (!c->k || !c->v || (mx && (!c->k_s || !c->v_s))))
      return decode_fail(MOE_ERR_INVALID_ARG, "%s: a page buffer is NULL", call);
  }
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: k and v must be 16-byte aligned", call);
  if (mx) {
    // a row's scale bytes are read as one word
    const size_t a = c->head_dim / 32;
    if (!aligned_to(c->k_s, a) || !aligned_to(c->v_s, a) || (c->page_stride / 32) % (int64_t)a ||
        (c->row_stride / 32) % (int64_t)a || (c->head_stride / 32) % (int64_t)a)
      return decode_fail(MOE_ERR_INVALID_ARG, "%s: scale rows must be aligned to their %d bytes", call, (int)a);
  }
  if (!aligned_to(c->block_table, 4) || !aligned_to(c->seq_lens, 4) || !aligned_to(c->status, 4))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: block_table, seq_lens and status must be 4-byte aligned", call);
  return MOE_OK;
}

PageDiv page_div(uint32_t page_size) {
  // round-up method for a 31-bit dividend: with 2^(s-1) < P <= 2^s, mul = floor(2^(31+s) / P) + 1 fits 32 bits,
  // and n * mul / 2^(31+s) errs by less than n / 2^(31+s) < 1 / P above n / P
  if (page_size <= 1) return {0u, 0u};
  uint32_t s = 0;
  while ((1ull << s) < page_size) ++s;
  return {(uint32_t)(((1ull << (31 + s)) / page_size) + 1ull), s - 1};
}

}  // namespace moe
