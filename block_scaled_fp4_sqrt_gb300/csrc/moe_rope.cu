// Norms of query and key heads with the position rotation, into rows or straight into the paged cache (moe_head_norm_rope).
//
//   x' = x w rsqrt(mean x^2 + eps);  y_i = x'_i cos a - x'_j sin a,  y_j = x'_i sin a + x'_j cos a,  a = position * frequency
//
// One pass: a head of a row is read once, by D / 8 lanes, and written once; memory-bound for prompts, latency-bound for a
// step's few rows.
//  * A lane keeps its columns for all heads of a chunk, so that a token's sines and cosines are computed once and stay in
//    registers: no shared memory and no barrier.  Pairs (i, i + rot / 2) are held by one lane, as two groups of four columns
//    half of rot_dim apart (8-byte loads, whole lines a head); only where rot_dim / 2 is no multiple of four (or, for a
//    quantised cache, of an MX block) is the partner fetched through shared memory.
//  * Few rows: a chunk is one head, and every group of lanes computes its own angles; a prompt: up to 16 heads.  (Angles of a
//    token computed by one warp and handed out through shared memory, behind a barrier: 8191 tokens of 40 heads on three
//    axes 175 us; held by lanes that go over the heads: 36, 70 % of the copy rate.  512 rows into an MXFP8 cache: 15 -> 8 us,
//    4099 tokens into an MXFP4 cache 25 us, 53 % of it; one row 4 us.)
//  * A phase is position * turns modulo 2^64, an integer product: exact for every position, where an fp32 angle at position
//    100,000 would be off by 2^-8 of a radian.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_decode_device.cuh"

namespace moe {

namespace {

constexpr int kBlock = 128;
constexpr int kBatch = 4;     // heads whose loads are under way together
// fp32 bits of the mean squares that have fp32's precision: 2^-90 to the largest number
constexpr uint32_t kLeastSquare = 0x12800000u, kLargestSquare = 0x7F7FFFFFu;
constexpr int kMaxChunk = 16; // heads a group of lanes takes

struct RopeParams {
  moe_kv_cache_t c;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_out;
  const void *q_w, *k_w;
  const uint64_t* turns;
  const uint8_t* axis;
  const int32_t* pos;
  int64_t qs, ks, vs, qos, kos, ps;
  int rows, L, hq, hkv, rot, w_f32, heads, chunk, last_axis;  // heads: of q, k and (with a cache) v together
  float eps;
  PageDiv page, len;
};

constexpr int kNoCache = -1;
// How a lane holds its eight columns: two groups of four half of rot_dim apart (the columns behind rot_dim: eight in a row);
// eight in a row, pairs being neighbours; eight in a row, the partners with other lanes.
enum Layout { kHalves, kNeighbours, kExchange };

__device__ __forceinline__ uint2 ld8(const __nv_bfloat16* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void st8(__nv_bfloat16* p, uint2 v) { *reinterpret_cast<uint2*>(p) = v; }

// Four columns of a weight.
__device__ __forceinline__ void weight4(const void* w, int f32, int col, float* to) {
  if (f32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + col));
    to[0] = a.x, to[1] = a.y, to[2] = a.z, to[3] = a.w;
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + col));
    to[0] = __uint_as_float(u.x << 16), to[1] = __uint_as_float(u.x & 0xFFFF0000u);
    to[2] = __uint_as_float(u.y << 16), to[3] = __uint_as_float(u.y & 0xFFFF0000u);
  }
}

template <int D, int FMT, Layout LAY>
__global__ void __launch_bounds__(kBlock, 6) head_norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;  // lanes of a head
  constexpr int kAngles = LAY == kExchange ? 8 : 4;
  __shared__ float s_x[LAY == kExchange ? kBlock / kLanes : 1][D];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, i = tid & (kLanes - 1);
  const int row = blockIdx.x * (kBlock / kLanes) + tid / kLanes;
  if (row >= p.rows) return;
  const uint32_t group = (kLanes == 16 ? 0xFFFFu : 0xFFu) << (lane & ~(kLanes - 1));  // the head's lanes
  const int half = p.rot >> 1;
  const bool turned = LAY != kHalves || i < p.rot / 8;  // (kHalves) this lane's columns are pairs
  const int col0 = LAY != kHalves ? 8 * i : turned ? 4 * i : p.rot + 8 * (i - p.rot / 8);
  const int col1 = LAY == kHalves && turned ? half + 4 * i : col0 + 4;

  // The last heads first: those of the cache take longer, and what begins late should be short (4099 tokens into an MXFP4
  // cache 28.0 -> 24.2 us; with blocks of 256 threads 25.2).
  const int first = (gridDim.y - 1 - blockIdx.y) * p.chunk, last = min(first + p.chunk, p.heads);
  // The heads of a kind (0 q, 1 k, 2 v) are heads kind_at .. of the call's.
  uint2 raw[kBatch][2];
  auto load = [&](auto kind, int h0, int end, uint2 (&to)[kBatch][2]) {
    constexpr int K = decltype(kind)::value;
    const int kind_at = K == 0 ? 0 : K == 1 ? p.hq : p.hq + p.hkv;
    const __nv_bfloat16* src = K == 0 ? p.q + row * p.qs : K == 1 ? p.k + row * p.ks : p.v + row * p.vs;
    src += (int64_t)(h0 - kind_at) * D;
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      if (h0 + n >= end) break;
      if (LAY == kHalves && K < 2) {
        to[n][0] = ld8(src + n * D + col0);
        to[n][1] = ld8(src + n * D + col1);
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(src + n * D + 8 * i);
        to[n][0] = make_uint2(u.x, u.y), to[n][1] = make_uint2(u.z, u.w);
      }
    }
  };
  const std::integral_constant<int, 0> q_heads;
  const std::integral_constant<int, 1> k_heads;
  const std::integral_constant<int, 2> v_heads;
  // what follows does not wait for the first heads
  if (first < p.hq)
    load(q_heads, first, min(last, p.hq), raw);
  else if (first < p.hq + p.hkv)
    load(k_heads, first, min(last, p.hq + p.hkv), raw);
  else
    load(v_heads, first, last, raw);

  int pos = 0, page = -1, prow = 0;
  if (FMT != kNoCache) {
    int l;
    const int b = page_of(row, p.len, p.L, &l);
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
  // the lane's angles: of the pairs of its first group, of its four neighbouring pairs, or of every column
  float cs[kAngles], sn[kAngles];
#pragma unroll
  for (int e = 0; e < kAngles; ++e) {
    const int pair = LAY != kExchange ? 4 * i + e : 8 * i + e < half ? 8 * i + e : 8 * i + e - half;
    cs[e] = 1.f, sn[e] = 0.f;
    if (LAY == kExchange ? 8 * i + e < p.rot : pair < half) {
      const int at = p.pos ? __ldg(p.pos + (p.axis ? min((int)__ldg(p.axis + pair), p.last_axis) : 0) * p.ps + row) : pos;
      const uint64_t phase = (uint64_t)(int64_t)at * __ldg(p.turns + pair);
      // the upper 32 bits as a signed fraction of half a turn
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn[e], &cs[e]);
    }
  }

  // The heads h0 .. end of a kind, the first batch of which has been asked for where `loaded`: while one batch is worked on,
  // the next is on its way.
  auto heads = [&](auto kind, int h0, int end, bool loaded) {
    constexpr int K = decltype(kind)::value;
    const int kind_at = K == 0 ? 0 : K == 1 ? p.hq : p.hq + p.hkv;
    const void* w = K == 0 ? p.q_w : K == 1 ? p.k_w : nullptr;
    float wv[8];
    if (w) {
      weight4(w, p.w_f32, col0, wv);
      weight4(w, p.w_f32, col1, wv + 4);
    }
    auto one = [&](int head, const uint2 (&r)[2]) {
      float x[8];
      bf16x8_to_f32(make_uint4(r[0].x, r[0].y, r[1].x, r[1].y), x);
      uint4 out = make_uint4(r[0].x, r[0].y, r[1].x, r[1].y);
      if constexpr (K < 2) {
        if (w) {
          auto mean_square = [&](float eps) {
            float sq = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
#pragma unroll
            for (int off = 1; off < kLanes; off <<= 1) sq += __shfl_xor_sync(group, sq, off);
            return fmaf(sq, 1.f / D, eps);
          };
          const float total = mean_square(p.eps);
          float inv = rsqrtf(total);
          // Squares that leave fp32's range are summed again in units of 2^80 or 2^-100, which bring every head into it (bf16's
          // numbers lie in 2^-133 .. 2^128).  The lanes of a head go the same way: their sums are the same.  The branch costs
          // 2 % (8191 tokens 34.9 -> 35.6 us, 4099 into MXFP4 24.0 -> 24.6, 512 rows 7.2 -> 8.2); a second look at a batch of
          // heads with one test for all of them spills (38.0, 25.5).
          if (__float_as_uint(total) - kLeastSquare > kLargestSquare - kLeastSquare) {
            const float unit = total < 1.f ? 0x1p100f : 0x1p-80f;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= unit;
            inv = rsqrtf(mean_square(p.eps * unit * unit));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * wv[e];
        }
        if constexpr (LAY == kHalves) {
          if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = x[e], b = x[4 + e];
              x[e] = a * cs[e] - b * sn[e];
              x[4 + e] = a * sn[e] + b * cs[e];
            }
          }
        } else if constexpr (LAY == kNeighbours) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * i + 2 * e < p.rot) {
              const float a = x[2 * e], b = x[2 * e + 1];
              x[2 * e] = a * cs[e] - b * sn[e];
              x[2 * e + 1] = a * sn[e] + b * cs[e];
            }
        } else {
          float* x_row = s_x[tid / kLanes];
          __syncwarp(group);
#pragma unroll
          for (int e = 0; e < 8; ++e) x_row[8 * i + e] = x[e];
          __syncwarp(group);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = 8 * i + e;
            if (c < half)
              x[e] = x[e] * cs[e] - x_row[c + half] * sn[e];
            else if (c < p.rot)
              x[e] = x_row[c - half] * sn[e] + x[e] * cs[e];
          }
        }
        if (w || p.rot) out = f32_to_bf16x8(x);  // what is not computed keeps its bits, those of a NaN too
        __nv_bfloat16* dst = K == 0 ? p.q_out + row * p.qos : p.k_out ? p.k_out + row * p.kos : nullptr;
        if (dst) {
          dst += (int64_t)head * D;
          if (LAY == kHalves) {
            st8(dst + col0, make_uint2(out.x, out.y));
            st8(dst + col1, make_uint2(out.z, out.w));
          } else {
            *reinterpret_cast<uint4*>(dst + col0) = out;
          }
        }
      }
      if constexpr (FMT == kNoCache || K == 0) return;
      const bool split = LAY == kHalves && K == 1;  // the columns lie in two groups
      const int64_t at = page * p.c.page_stride + prow * p.c.row_stride + head * p.c.head_stride;
      void* codes = K == 1 ? p.c.k : p.c.v;
      [[maybe_unused]] uint8_t* scales = K == 1 ? p.c.k_s : p.c.v_s;
      const int c0 = split ? col0 : 8 * i, c1 = split ? col1 : 8 * i + 4;
      if constexpr (FMT == MOE_KV_BF16) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(codes) + at;
        if (page >= 0) {
          if (split) {
            st8(dst + c0, make_uint2(out.x, out.y));
            st8(dst + c1, make_uint2(out.z, out.w));
          } else {
            *reinterpret_cast<uint4*>(dst + c0) = out;
          }
        }
      } else {
        // the largest magnitudes of the blocks of the two groups: pairs half of rot_dim apart lie in two blocks, each held by
        // eight lanes; eight columns in a row in one, held by four
        const bool two = split && turned;
        uint32_t top[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (FMT == MOE_KV_MXFP8) {  // of the numbers: a NaN keeps its own code
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(x[4 * g + e]));
            top[g] = __float_as_uint(m);
          } else {
            top[g] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) top[g] = max(top[g], __float_as_uint(x[4 * g + e]) & 0x7FFFFFFFu);
          }
        }
        if (!two) top[0] = top[1] = max(top[0], top[1]);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          top[g] = max(top[g], __shfl_xor_sync(group, top[g], 1));
          top[g] = max(top[g], __shfl_xor_sync(group, top[g], 2));
          const uint32_t other = __shfl_xor_sync(group, top[g], 4);
          if (two) top[g] = max(top[g], other);
        }
        const bool writes_scale = (i & (two ? 7 : 3)) == 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int64_t to = at + (g ? c1 : c0);
          uint8_t scale;
          if constexpr (FMT == MOE_KV_MXFP8) {
            const int e = mxfp8_block_exp(__uint_as_float(top[g]));
            const float mul = exp2_neg_int(e);
            scale = (uint8_t)(e + 127);
            const uint32_t w = (uint32_t)e4m3x2(x[4 * g] * mul, x[4 * g + 1] * mul) |
                               ((uint32_t)e4m3x2(x[4 * g + 2] * mul, x[4 * g + 3] * mul) << 16);
            if (page >= 0) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(codes) + to) = w;
          } else {
            uint32_t w;
            scale = mxfp4_quad({x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3], 0.f, 0.f, 0.f, 0.f}, top[g], w);
            if (page >= 0) *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(codes) + (to >> 1)) = (uint16_t)w;
          }
          if (page >= 0 && writes_scale && (two || g == 0)) scales[to >> 5] = scale;
        }
      }
    };
    if (!loaded) load(kind, h0, end, raw);
    for (; h0 < end; h0 += kBatch) {
      uint2 next[kBatch][2];
      load(kind, h0 + kBatch, end, next);
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        if (h0 + n >= end) break;
        one(h0 + n - kind_at, raw[n]);
      }
#pragma unroll
      for (int n = 0; n < kBatch; ++n) raw[n][0] = next[n][0], raw[n][1] = next[n][1];
    }
  };
  if (first < p.hq) heads(q_heads, first, min(last, p.hq), true);
  if (first < p.hq + p.hkv && last > p.hq) heads(k_heads, max(first, p.hq), min(last, p.hq + p.hkv), first >= p.hq);
  if (FMT != kNoCache && last > p.hq + p.hkv) heads(v_heads, max(first, p.hq + p.hkv), last, first >= p.hq + p.hkv);
}

template <int D>
cudaError_t launch(RopeParams p, int fmt, bool adjacent, int sms, cudaStream_t s) {
  constexpr int kLanes = D / 8;
  // Equal chunks of heads, the largest that leave 16 warps an SM: fewer and longer ones compute fewer angles (512 rows of 48
  // heads, before the norms looked at their range: 7.2 us; with one head a chunk 11.3, with 12 warps an SM 8.1, with 20 to 32
  // the same).
  const int64_t warps = (int64_t)p.rows * p.heads * kLanes / 32;
  const int chunk = (int)std::max<int64_t>(1, std::min<int64_t>({warps / ((int64_t)sms * 16), kMaxChunk, p.heads}));
  const int chunks = (p.heads + chunk - 1) / chunk;
  p.chunk = (p.heads + chunks - 1) / chunks;
  const bool quantised = fmt == MOE_KV_MXFP8 || fmt == MOE_KV_MXFP4;
  const Layout lay = adjacent ? kNeighbours : p.rot % (quantised ? 64 : 8) == 0 ? kHalves : kExchange;
  const dim3 grid((p.rows + kBlock / kLanes - 1) / (kBlock / kLanes), (p.heads + p.chunk - 1) / p.chunk);
  auto pick = [&](auto f) {
    constexpr int FMT = decltype(f)::value;
    return lay == kHalves       ? head_norm_rope_kernel<D, FMT, kHalves>
           : lay == kNeighbours ? head_norm_rope_kernel<D, FMT, kNeighbours>
                                : head_norm_rope_kernel<D, FMT, kExchange>;
  };
  auto* kernel = fmt == MOE_KV_BF16    ? pick(std::integral_constant<int, MOE_KV_BF16>{})
                 : fmt == MOE_KV_MXFP8 ? pick(std::integral_constant<int, MOE_KV_MXFP8>{})
                 : fmt == MOE_KV_MXFP4 ? pick(std::integral_constant<int, MOE_KV_MXFP4>{})
                                       : pick(std::integral_constant<int, kNoCache>{});
  return launch_pdl(kernel, grid, dim3(kBlock), 0, s, p);
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
  if (a->n_axes < 1 || a->n_axes > 256)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: n_axes (%d) must be 1 to 256", call, a->n_axes);
  if ((cache ? a->L : a->T) < 0) return decode_fail(MOE_ERR_INVALID_ARG, "%s: a negative number of rows", call);
  if (a->n_q_heads < 0 || a->n_kv_heads < 0 || a->n_q_heads > 65535 || a->n_kv_heads > 65535)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: heads (%d, %d) outside [0, 65535]", call, a->n_q_heads, a->n_kv_heads);
  const int64_t rows = cache ? (int64_t)cache->n_seqs * a->L : a->T;
  if (rows > 0x7FFFFF00ll || (int64_t)a->n_q_heads + 2 * (int64_t)a->n_kv_heads > 65535)
    return decode_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^31 - 256 rows or 65535 heads", call);
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
      return decode_fail(MOE_ERR_INVALID_ARG,
                         "%s: row stride of %s (%lld) must be a multiple of 8, at least its heads * head_dim", call, r.name,
                         (long long)*r.to);
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
  int sms = 0;
  st = check_device(&sms);
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
  p.rows = (int)rows;
  p.L = cache ? a->L : 1;
  p.hq = with_q ? a->n_q_heads : 0;
  p.hkv = with_k ? a->n_kv_heads : 0;
  p.heads = p.hq + p.hkv * (cache ? 2 : 1);
  p.rot = a->rot_dim;
  p.last_axis = a->n_axes - 1;
  p.w_f32 = a->weight_f32;
  p.eps = a->eps;
  p.page = cache ? page_div((uint32_t)cache->page_size) : PageDiv{0, 0};
  p.len = page_div((uint32_t)p.L);
  if (p.heads == 0) return MOE_OK;
  const int fmt = cache ? cache->format : kNoCache;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool adjacent = a->pairs == MOE_ROPE_ADJACENT;
  const cudaError_t e = a->head_dim == 128 ? launch<128>(p, fmt, adjacent, sms, s) : launch<64>(p, fmt, adjacent, sms, s);
  if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "%s: %s", call, cudaGetErrorString(e));
  return MOE_OK;
}
