// Norms of query and key heads with the position rotation, into rows or straight into the paged cache (moe_head_norm_rope).
//
//   x' = x w rsqrt(mean x^2 + eps);  y_i = x'_i cos a - x'_j sin a,  y_j = x'_i sin a + x'_j cos a,  a = position * frequency
//
// One pass: a row's heads are read once, each by D / 8 lanes with eight neighbouring columns a lane, and written once.
// The angles are shared by all heads of a token, so a block takes a token and computes its rot_dim / 2 of them first.
// A phase is position * turns modulo 2^64, an integer product: exact for every position, where an fp32 angle at position
// 100,000 would be off by 2^-8 of a radian.
#include <algorithm>
#include <cmath>

#include "moe_decode_device.cuh"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;

struct RopeParams {
  moe_kv_cache_t c;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_out;
  const void *q_w, *k_w;
  const uint64_t* turns;
  const uint8_t* axis;
  const int32_t* pos;
  int64_t qs, ks, vs, qos, kos, ps;
  int L, hq, hkv, rot, adjacent, w_f32, heads;  // heads: of q, k and (with a cache) v together
  float eps;
  PageDiv page;
};

constexpr int kNoCache = -1;

template <int D, int FMT>
__global__ void __launch_bounds__(kMaxThreads) head_norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;  // lanes of a head
  __shared__ float2 s_cs[D / 2];
  __shared__ float s_x[kMaxThreads / kLanes][D];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t group = (kLanes == 16 ? 0xFFFFu : 0xFFu) << (lane & ~(kLanes - 1));  // the head's lanes
  const int col = (tid & (kLanes - 1)) * 8;
  const int64_t row = blockIdx.x;
  int pos = 0, page = -1, prow = 0;
  if (FMT != kNoCache) {
    const int b = (int)(row / p.L), l = (int)(row - (int64_t)b * p.L);
    pos = seq_len_of(p.c, b) - p.L + l;
    if (pos >= 0) {
      const int j = page_of(pos, p.page, p.c.page_size, &prow);
      page = __ldg(p.c.block_table + (int64_t)b * p.c.max_pages + j);
      if (page < 0 || page >= p.c.n_pages) {
        set_status(p.c.status, MOE_KV_BAD_PAGE);
        page = -1;
      }
    }
  }
  for (int i = tid; i < p.rot / 2; i += blockDim.x) {
    const int at = p.pos ? __ldg(p.pos + (p.axis ? p.axis[i] : 0) * p.ps + row) : pos;
    const uint64_t phase = (uint64_t)(int64_t)at * __ldg(p.turns + i);
    // the upper 32 bits as a signed fraction of half a turn
    float2 cs;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &cs.y, &cs.x);
    s_cs[i] = cs;
  }
  __syncthreads();
  float* x_row = s_x[tid / kLanes];
  for (int u = tid / kLanes; u < p.heads; u += blockDim.x / kLanes) {
    const bool is_q = u < p.hq, is_k = !is_q && u < p.hq + p.hkv;
    const int head = is_q ? u : is_k ? u - p.hq : u - p.hq - p.hkv;
    const __nv_bfloat16* src = is_q ? p.q + row * p.qs : is_k ? p.k + row * p.ks : p.v + row * p.vs;
    const uint4 raw = *reinterpret_cast<const uint4*>(src + head * D + col);
    float x[8];
    bf16x8_to_f32(raw, x);
    uint4 out = raw;
    const void* w = is_q ? p.q_w : is_k ? p.k_w : nullptr;
    if (is_q || is_k) {
      if (w) {
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) sq += __shfl_xor_sync(group, sq, off);
        const float inv = rsqrtf(fmaf(sq, 1.f / D, p.eps));
        float wv[8];
        if (p.w_f32) {
          const float4* wp = reinterpret_cast<const float4*>(static_cast<const float*>(w) + col);
          const float4 a = __ldg(wp), b = __ldg(wp + 1);
          wv[0] = a.x, wv[1] = a.y, wv[2] = a.z, wv[3] = a.w, wv[4] = b.x, wv[5] = b.y, wv[6] = b.z, wv[7] = b.w;
        } else {
          bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + col)), wv);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wv[i];
      }
      if (p.adjacent) {
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          if (col + i < p.rot) {
            const float2 cs = s_cs[(col + i) >> 1];
            const float a = x[i], b = x[i + 1];
            x[i] = a * cs.x - b * cs.y;
            x[i + 1] = a * cs.y + b * cs.x;
          }
      } else {
        __syncwarp(group);
#pragma unroll
        for (int i = 0; i < 8; ++i) x_row[col + i] = x[i];
        __syncwarp(group);
        const int half = p.rot >> 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = col + i;
          if (c < half) {
            const float2 cs = s_cs[c];
            x[i] = x[i] * cs.x - x_row[c + half] * cs.y;
          } else if (c < p.rot) {
            const float2 cs = s_cs[c - half];
            x[i] = x_row[c - half] * cs.y + x[i] * cs.x;
          }
        }
      }
      if (w || p.rot) out = f32_to_bf16x8(x);  // what is not computed keeps its bits, those of a NaN too
      if (is_q) *reinterpret_cast<uint4*>(p.q_out + row * p.qos + head * D + col) = out;
      if (is_k && p.k_out) *reinterpret_cast<uint4*>(p.k_out + row * p.kos + head * D + col) = out;
    }
    if (FMT != kNoCache && !is_q) {
      const int64_t at = page * p.c.page_stride + prow * p.c.row_stride + head * p.c.head_stride + col;
      void* codes = is_k ? p.c.k : p.c.v;
      uint8_t* scales = is_k ? p.c.k_s : p.c.v_s;
      if constexpr (FMT == MOE_KV_BF16) {
        if (page >= 0) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(codes) + at) = out;
      } else {
        uint8_t scale;  // four neighbouring lanes hold a block
        if constexpr (FMT == MOE_KV_MXFP8) {
          float amax = 0.f;  // of the numbers: a NaN keeps its own code
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
          amax = fmaxf(amax, __shfl_xor_sync(group, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(group, amax, 2));
          const int e = mxfp8_block_exp(amax);
          scale = (uint8_t)(e + 127);
          if (page >= 0) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(codes) + at) = e4m3_8(x, exp2_neg_int(e));
        } else {
          uint32_t top = abs_max_bits(x);
          top = max(top, __shfl_xor_sync(group, top, 1));
          top = max(top, __shfl_xor_sync(group, top, 2));
          uint32_t word;
          scale = mxfp4_quad(x, top, word);
          if (page >= 0) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(codes) + (at >> 1)) = word;
        }
        if (page >= 0 && (lane & 3) == 0) scales[at >> 5] = scale;
      }
    }
  }
}

template <int D>
cudaError_t launch(const RopeParams& p, int fmt, int64_t rows, cudaStream_t s) {
  const int threads = std::min(kMaxThreads, (p.heads * (D / 8) + 31) / 32 * 32);
  auto* kernel = fmt == MOE_KV_BF16    ? head_norm_rope_kernel<D, MOE_KV_BF16>
                 : fmt == MOE_KV_MXFP8 ? head_norm_rope_kernel<D, MOE_KV_MXFP8>
                 : fmt == MOE_KV_MXFP4 ? head_norm_rope_kernel<D, MOE_KV_MXFP4>
                                       : head_norm_rope_kernel<D, kNoCache>;
  return launch_pdl(kernel, dim3((unsigned)rows), dim3(threads), 0, s, p);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_head_norm_rope(const moe_kv_cache_t* cache, const moe_head_rope_t* a, moe_stream_t stream) {
  const char* call = "moe_head_norm_rope";
  moe_status_t st = cache ? check_cache(cache, call) : MOE_OK;
  if (st != MOE_OK) return st;
  if (!a) return decode_fail(MOE_ERR_INVALID_ARG, "%s: args is NULL", call);
  if (a->head_dim != 64 && a->head_dim != 128)
    return decode_fail(MOE_ERR_UNSUPPORTED, "%s: head_dim (%d) must be 64 or 128", call, a->head_dim);
  if (cache && (cache->head_dim != a->head_dim || cache->n_kv_heads != a->n_kv_heads))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: the cache has %d heads of %d, the call %d of %d", call, cache->n_kv_heads,
                       cache->head_dim, a->n_kv_heads, a->head_dim);
  if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 2)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: rot_dim (%d) must be even, 0 to head_dim", call, a->rot_dim);
  if (a->pairs != MOE_ROPE_HALF && a->pairs != MOE_ROPE_ADJACENT)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: unknown pairs %d", call, a->pairs);
  if (!(a->eps >= 0.f) || std::isinf(a->eps))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: eps must be a finite number >= 0", call);
  if (a->n_axes < 1 || a->n_axes > 256) return decode_fail(MOE_ERR_INVALID_ARG, "%s: n_axes (%d) must be 1 to 256", call, a->n_axes);
  if ((cache ? a->L : a->T) < 0) return decode_fail(MOE_ERR_INVALID_ARG, "%s: a negative number of rows", call);
  if (a->n_q_heads < 0 || a->n_kv_heads < 0 || a->n_q_heads > 65535 || a->n_kv_heads > 65535)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: heads (%d, %d) outside [0, 65535]", call, a->n_q_heads, a->n_kv_heads);
  const int64_t rows = cache ? (int64_t)cache->n_seqs * a->L : a->T;
  if (rows > 0x7FFFFFFFll) return decode_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 rows", call);
  const bool with_q = a->q || a->q_out, with_k = cache || a->k || a->k_out;
  RopeParams p{};
  const struct {
    const char* name;
    const void* ptr;
    int64_t stride;
    int64_t width;
    int64_t* to;
  } all[] = {{"q", a->q, a->q_stride, (int64_t)a->n_q_heads * a->head_dim, &p.qs},
             {"k", a->k, a->k_stride, (int64_t)a->n_kv_heads * a->head_dim, &p.ks},
             {"v", cache ? a->v : nullptr, a->v_stride, (int64_t)a->n_kv_heads * a->head_dim, &p.vs},
             {"q_out", a->q_out, a->q_out_stride, (int64_t)a->n_q_heads * a->head_dim, &p.qos},
             {"k_out", a->k_out, a->k_out_stride, (int64_t)a->n_kv_heads * a->head_dim, &p.kos}};
  for (const auto& r : all) {
    *r.to = r.stride ? r.stride : r.width;
    if (r.ptr && (*r.to < r.width || *r.to % 8))
      return decode_fail(MOE_ERR_INVALID_ARG, "%s: row stride of %s (%lld) must be a multiple of 8, at least its heads * head_dim",
                         call, r.name, (long long)*r.to);
    if (!aligned_to(r.ptr, 16)) return decode_fail(MOE_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", call, r.name);
  }
  if (!aligned_to(a->q_weight, 16) || !aligned_to(a->k_weight, 16) || !aligned_to(a->turns, 8) || !aligned_to(a->positions, 4))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: weights must be 16-byte aligned, turns 8-byte, positions 4-byte", call);
  p.ps = a->position_stride ? a->position_stride : rows;
  if (a->positions && a->n_axes > 1 && p.ps < rows)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: position_stride (%lld) is below the number of rows", call, (long long)p.ps);
  if (rows == 0) return MOE_OK;
  if (!with_q && !with_k) return decode_fail(MOE_ERR_INVALID_ARG, "%s: neither q nor k is given", call);
  if (with_q && (!a->q || !a->q_out)) return decode_fail(MOE_ERR_INVALID_ARG, "%s: q and q_out go together", call);
  if (!cache && with_k && (!a->k || !a->k_out)) return decode_fail(MOE_ERR_INVALID_ARG, "%s: k and k_out go together", call);
  if (cache && (!a->k || !a->v)) return decode_fail(MOE_ERR_INVALID_ARG, "%s: k or v is NULL", call);
  if (cache && !cache->seq_lens) return decode_fail(MOE_ERR_INVALID_ARG, "%s: seq_lens is NULL", call);
  if (a->rot_dim && (!a->turns || (!cache && !a->positions)))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: turns or positions is NULL", call);
  st = check_device(nullptr);
  if (st != MOE_OK) return st;
  if (cache) p.c = *cache;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.v = static_cast<const __nv_bfloat16*>(a->v);
  p.q_out = static_cast<__nv_bfloat16*>(a->q_out);
  p.k_out = static_cast<__nv_bfloat16*>(a->k_out);
  p.q_w = a->q_weight;
  p.k_w = a->k_weight;
  p.turns = a->turns;
  p.axis = a->axis;
  p.pos = a->positions;
  p.L = cache ? a->L : 1;
  p.hq = with_q ? a->n_q_heads : 0;
  p.hkv = with_k ? a->n_kv_heads : 0;
  p.heads = p.hq + p.hkv * (cache ? 2 : 1);
  p.rot = a->rot_dim;
  p.adjacent = a->pairs == MOE_ROPE_ADJACENT;
  p.w_f32 = a->weight_f32;
  p.eps = a->eps;
  p.page = cache ? page_div((uint32_t)cache->page_size) : PageDiv{0, 0};
  if (p.heads == 0) return MOE_OK;
  const int fmt = cache ? cache->format : kNoCache;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = a->head_dim == 128 ? launch<128>(p, fmt, rows, s) : launch<64>(p, fmt, rows, s);
  if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "%s: %s", call, cudaGetErrorString(e));
  return MOE_OK;
}
