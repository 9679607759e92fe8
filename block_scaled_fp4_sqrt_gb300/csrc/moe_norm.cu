// Residual addition and root-mean-square norm, with the MXFP8 form of the result (moe_add_rms_norm).
//
//   t = x + r,  sum = bf16(t),  y = bf16(t * rsqrt(mean(t^2) + eps) * w),  (q, s) = MXFP8(y)
//
// One pass over the data: a row's fp32 t stays in the registers of the threads that hold it between the sum of
// squares and the outputs.  Memory-bound: 4 (x, r) + 4 (sum, y) + 33/32 (codes, scales) bytes an element.
// Measured: 8192 rows of 4096 in 40.3 us (6.6 TB/s, 99 % of the copy rate), 512 rows in 4.8 us (2.8 us at that rate: a
// launch and one trip to memory are left), one row in 2.3 us.  Each output is one rounding of the fp32 value.
#include <algorithm>
#include <cmath>

#include "moe_decode_device.cuh"

namespace moe {

namespace {

struct NormParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* r;
  const void* w;
  __nv_bfloat16* sum;
  __nv_bfloat16* y;
  uint8_t* q;
  uint8_t* s;
  int64_t xs, rs, ss, ys;
  int T, d;
  float eps, inv_d;
};

// A group of G threads (a warp, or the whole block) holds one row, a thread NV vectors of 8 columns: vector
// j * G + lane of the row, so that every load and store of a warp is contiguous and the four lanes 4i..4i+3
// hold one MX block of 32 columns.  G = 32: several rows per block, no block barrier.
template <int NV, bool WARP_ROWS>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const NormParams p, int w_f32) {
  pdl_trigger();
  pdl_wait();
  const int group = WARP_ROWS ? 32 : blockDim.x;
  const int tid = WARP_ROWS ? threadIdx.x & 31 : threadIdx.x;
  const int row = WARP_ROWS ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP_ROWS && row >= p.T) return;
  const int nvec = p.d >> 3;
  float t[NV][8];
  float sq = 0.f;
  {
    uint4 xr[NV], rr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * group + tid;
      xr[j] = rr[j] = make_uint4(0u, 0u, 0u, 0u);
      if (v < nvec) {
        xr[j] = *reinterpret_cast<const uint4*>(p.x + row * p.xs + v * 8);
        if (p.r) rr[j] = *reinterpret_cast<const uint4*>(p.r + row * p.rs + v * 8);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float a[8], b[8];
      bf16x8_to_f32(xr[j], a);
      bf16x8_to_f32(rr[j], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[j][i] = a[i] + b[i];
        sq = fmaf(t[j][i], t[j][i], sq);
      }
    }
  }
  // the new residual stream does not wait for the norm
  if (p.sum) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * group + tid;
      if (v < nvec) *reinterpret_cast<uint4*>(p.sum + row * p.ss + v * 8) = f32_to_bf16x8(t[j]);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, off);
  if (!WARP_ROWS) {
    __shared__ float part[32];
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = sq;
    __syncthreads();
    sq = (threadIdx.x & 31) < nw ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, off);
  }
  const float inv = rsqrtf(fmaf(sq, p.inv_d, p.eps));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * group + tid;
    const bool in = v < nvec;
    float w[8];
    if (w_f32) {
      const float4* wp = reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + v * 8);
      const float4 a = in ? __ldg(wp) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 b = in ? __ldg(wp + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.w) + v * 8))
                         : make_uint4(0u, 0u, 0u, 0u);
      bf16x8_to_f32(u, w);
    }
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = t[j][i] * inv * w[i];
    const uint4 y8 = f32_to_bf16x8(o);
    if (in && p.y) *reinterpret_cast<uint4*>(p.y + row * p.ys + v * 8) = y8;
    if (p.q) {  // d is a multiple of 32 here: a block's four lanes are in range together
      bf16x8_to_f32(y8, o);
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(o[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int e = mxfp8_block_exp(amax);
      if (in) {
        const uint2 c = e4m3_8(o, exp2_neg_int(e));
        *reinterpret_cast<uint2*>(p.q + (size_t)row * p.d + v * 8) = c;
        if ((tid & 3) == 0) p.s[(size_t)row * (p.d >> 5) + (v >> 2)] = (uint8_t)(e + 127);
      }
    }
  }
}

}  // namespace

// Rows of up to 512 columns take a warp each, eight rows a block; longer ones a block each, with the threads
// that two vectors a thread need (d = 4096: 256), and four or eight vectors a thread above 16384 / 32768 columns.
static cudaError_t launch_add_rms_norm(const NormParams& p, int w_f32, cudaStream_t s) {
  const int nvec = p.d / 8;
  if (nvec <= 64) return launch_pdl(add_rms_norm_kernel<2, true>, dim3((p.T - 1) / 8 + 1), dim3(256), 0, s, p, w_f32);
  const int nv = nvec <= 2048 ? 2 : nvec <= 4096 ? 4 : 8;
  const dim3 block(((nvec + nv - 1) / nv + 31) / 32 * 32), grid(p.T);
  switch (nv) {
    case 2: return launch_pdl(add_rms_norm_kernel<2, false>, grid, block, 0, s, p, w_f32);
    case 4: return launch_pdl(add_rms_norm_kernel<4, false>, grid, block, 0, s, p, w_f32);
    default: return launch_pdl(add_rms_norm_kernel<8, false>, grid, block, 0, s, p, w_f32);
  }
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_add_rms_norm(const moe_norm_t* a, moe_stream_t stream) {
  if (!a) return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: args is NULL");
  if (a->T < 0) return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: T = %d is negative", a->T);
  if (a->d < 8 || a->d % 8 || a->d > 65536)
    return decode_fail(MOE_ERR_UNSUPPORTED, "moe_add_rms_norm: d (%d) must be a multiple of 8 in [8, 65536]", a->d);
  if (!(a->eps >= 0.f) || std::isinf(a->eps))
    return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: eps must be a finite number >= 0");
  if (!a->y_q != !a->y_s) return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: y_q and y_s go together");
  if (a->y_q && a->d % 32)
    return decode_fail(MOE_ERR_UNSUPPORTED, "moe_add_rms_norm: the MXFP8 output needs d (%d) a multiple of 32", a->d);
  NormParams p{};
  const struct {
    const char* name;
    const void* ptr;
    int64_t stride;
    int64_t* to;
  } rows[] = {{"x", a->x, a->x_stride, &p.xs},
              {"residual", a->residual, a->residual_stride, &p.rs},
              {"sum", a->sum, a->sum_stride, &p.ss},
              {"y", a->y, a->y_stride, &p.ys}};
  for (const auto& r : rows) {
    *r.to = r.stride ? r.stride : a->d;
    if (r.ptr && (*r.to < a->d || *r.to % 8))
      return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: row stride of %s (%lld) must be a multiple of 8, at least d",
                         r.name, (long long)*r.to);
    if (!aligned_to(r.ptr, 16)) return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: %s must be 16-byte aligned", r.name);
  }
  if (a->T == 0) return MOE_OK;
  if (!a->sum && !a->y && !a->y_q) return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: no output is given");
  if (!a->x || !a->weight) return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: x or weight is NULL");
  if (!aligned_to(a->weight, 16) || !aligned_to(a->y_q, 8))
    return decode_fail(MOE_ERR_INVALID_ARG, "moe_add_rms_norm: weight must be 16-byte and y_q 8-byte aligned");
  const moe_status_t st = check_device(nullptr);
  if (st != MOE_OK) return st;
  p.x = static_cast<const __nv_bfloat16*>(a->x);
  p.r = static_cast<const __nv_bfloat16*>(a->residual);
  p.w = a->weight;
  p.sum = static_cast<__nv_bfloat16*>(a->sum);
  p.y = static_cast<__nv_bfloat16*>(a->y);
  p.q = a->y_q;
  p.s = a->y_s;
  p.T = a->T;
  p.d = a->d;
  p.eps = a->eps;
  p.inv_d = 1.0f / (float)a->d;
  const cudaError_t e = launch_add_rms_norm(p, a->weight_f32 ? 1 : 0, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "moe_add_rms_norm: %s", cudaGetErrorString(e));
  return MOE_OK;
}
