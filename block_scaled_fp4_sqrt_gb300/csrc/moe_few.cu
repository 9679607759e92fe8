// The whole MoE layer for a few tokens (T <= 8) in one kernel (moe_forward_few): routing, MXFP8 activations,
// both expert products, SwiGLU and the weighted combine, with the arithmetic of moe_forward.
//
// Bound: the touched experts' MXFP4 weights are read once, 13.4 MB an expert at d = 4096, f = 2048 (94 MB for one
// token, about 0.6 GB for eight), so a step should take their time at HBM rate.  What moe_forward loses against that at
// these sizes are the gaps between its five kernels; here one persistent block per SM keeps a ring of weight
// tiles in flight from the routing to the end.
// Measured (d = 4096, f = 2048, 256 experts, graph replays with other rows at every call; moe_forward beside it): one
// token 33 to 35 us over boxes against 44.5 (14.6 at HBM rate: a cooperative launch takes about 5, the routing 6, the
// weights then arrive at 5.7 TB/s), two 46 against 63, three 67 against 64, four 82 against 81, five 98 against 95, eight
// 134 to 140 against 119 (90.8 at HBM rate).  Below three tokens it leads; at eight moe_forward does: x, the partial
// products and the h slices of eight tokens leave shared memory for four stages, and the instructions (60 % of the issue
// slots) get in each other's way.  What it keeps is that a token's row has the same bits alone and in any company.
//
//  1. Router.  Block b computes the fp32 logits of experts b, b + grid, .. for all tokens (its warps split d);
//     the same pass loads x and quantises it to MXFP8.  A grid-wide count, then every block selects the top-k of
//     every token for itself and lists the touched experts (slots) with their tokens.
//  2. Work items, dealt to the blocks in turn: for every slot f/32 gate-up items (32 gate and 32 up rows of W13, one
//     MX block of h), then for every slot d/64 down items (64 rows of W2); the shared expert is the first slot.  The blocks never meet in between: a
//     down item waits for its own slot's gate-up items (a counter a slot), which came earlier in the list, and
//     its weights are already in the ring by then.
//  3. A down item's rows, times their routing weight, go to fp32 rows [token][choice][d]; the last item of a
//     (64 columns, token) pair sums the token's rows in order (choices, then the shared expert) and rounds once.
//
// A block: 2 producer warps (TMA: stages of 64 weight rows x 512, 16 KB with 64-byte swizzle, and their scale atoms,
// two copies a stage), 16 product warps (two groups that take the stages in turn; in a group the stage's 4 K groups x 2
// pairs of row tiles), 2 epilogue warps, and 4 warps that bring the h slices of down stages into the ring.
//
// Products run on mma.sync m16n8k16 with the weight rows as M and up to 8 tokens as N: E2M1 weights become fp16 by
// one conversion a pair (exact); x and h are fp16 too: their E4M3 codes with the block scales folded in relative to
// the row's largest (exact down to 2^-22 of the row's maximum, far below the fp32 sums' rounding).  The product of
// each block of 32 is scaled by the weights' E8M0 byte in fp32.  tcgen05 would spend its 128-row operand on at most
// 8 tokens, and its issue chain and accumulator hand-over are what bounds moe_forward's items at these sizes;
// mma.sync needs 16 of the 47 cycles that a sub-partition has per 16 x 32 weights at full HBM rate.
#include <float.h>

#include <algorithm>

#include "moe_decode_device.cuh"
#include "moe_few.h"

namespace moe {

namespace {

constexpr int kMaxT = kFewMaxT;
constexpr int kMmaWarps = 16, kEpiWarps = 2, kHWarps = 4, kProducers = 2;
constexpr int kThreads = 32 * (kMmaWarps + kEpiWarps + kHWarps + kProducers);  // 24 warps, six a sub-partition
constexpr int kProducer = kMmaWarps + kEpiWarps + kHWarps;
constexpr int kEpiTok = (kFewMaxT + kEpiWarps - 1) / kEpiWarps;
constexpr int kTileBytes = 64 * 64;              // 64 weight rows x 128 E2M1
constexpr int kStageKg = 4;                      // K groups of 128 in a stage
constexpr int kGroups = 2;                       // product groups
constexpr int kGroupWarps = kMmaWarps / kGroups; // one K group of a stage and half of the rows each
constexpr int kSplits = kGroups * kStageKg;      // K splits of an item's sums
constexpr int kStageSf = kStageKg * kTileBytes;  // a stage: codes, then scale atoms, then h rows
constexpr int kStageH = kStageSf + kStageKg * 2 * kSfAtomBytes;
constexpr int kHPitch = kStageKg * 128 * 2 + 64;  // bytes of a token's h slice: two tokens a phase, no conflicts
constexpr int kMaxK = 16;
constexpr int kMaxSlots = kFewMaxSlots;
constexpr int kRedStride = 9;                    // floats a row of the partial products (8 tokens)
constexpr int kRedFloats = kSplits * 64 * kRedStride;
constexpr int kMaxStages = 8;                    // the ring has 2, 4, 6 or 8 stages
constexpr int kFxItems = 16;                     // items in flight: at most the ring's and the two partial buffers'
static_assert(kMaxStages + 2 < kFxItems, "a row factor must outlive its item");

__host__ __device__ constexpr int stage_bytes(int T) { return kStageH + (T * kHPitch + 1023) / 1024 * 1024; }

struct Shared {  // fixed-size part of the block's shared memory
  uint64_t full[kMaxStages], empty[kMaxStages], red_full[2], red_empty[2];
  float part[kMmaWarps][2 * kMaxT];
  float fx[kMaxT];               // x = fp16 value * fx
  float hfx[kFxItems][kMaxT];    // h = fp16 value * hfx, by item and token of the slot
  float w[kMaxT][kMaxK];
  int ids[kMaxT][kMaxK];
  int e_max[kMaxT];
  uint32_t taken[kMaxT];         // choices j that are rows of their own (a repeated id joins its first choice)
  uint32_t touched[32];
  int before[32];                // experts touched in lower words
  int n_slots;
  int abort;
  int slot_expert[kMaxSlots];    // -1: the shared expert
  uint32_t slot_mask[kMaxSlots]; // its tokens
  int slot_ready[kMaxSlots];
  uint8_t slot_tok[kMaxSlots][kMaxT];
  uint8_t slot_j[kMaxSlots][kMaxT];
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Four bytes of E2M1 pairs as fp16 pairs (exact): element 2 i of a byte in the low half.
__device__ __forceinline__ void e2m1_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_hint(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                                 uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}],"
      " [%6];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Waits end when the phase completes, when the budget runs out or when another warp of the block gave up.
struct Waiter {
  Shared* sh;
  int* status;
  uint64_t budget;
  __device__ bool give_up() const {
    *(volatile int*)&sh->abort = 1;
    set_status(status, DEV_TIMEOUT);
    return false;
  }
  __device__ bool bar(uint64_t* b, uint32_t parity) const {
    if (mbar_test(b, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
      if (mbar_try_wait_suspend(b, parity, 20000u)) return true;
      if (*(volatile int*)&sh->abort) return false;
      if (globaltimer_ns() - t0 > budget) return give_up();
    }
  }
  __device__ bool count(const int* p, int target) const {
    if (ld_acquire(p) >= target) return true;
    const uint64_t t0 = globaltimer_ns();
    for (int i = 0;; ++i) {
      if (ld_acquire(p) >= target) return true;
      if ((i & 63) == 63) {
        if (*(volatile int*)&sh->abort) return false;
        if (globaltimer_ns() - t0 > budget) return give_up();
      }
    }
  }
};

template <int NPL>
__device__ __forceinline__ void select_token(const float* __restrict__ score, const float* __restrict__ bias, int E,
                                             int k, float route_scale, int32_t* ids, float* w) {
  const int lane = threadIdx.x & 31;
  float sc[NPL], sel[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    sc[i] = e < E ? __ldcg(score + e) : 0.f;
    sel[i] = e < E ? __ldg(bias + e) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) sel[i] = lane + 32 * i < E ? sc[i] + sel[i] : -FLT_MAX;
  warp_route_topk<NPL>(sc, sel, E, k, route_scale, ids, w);
}

// The sums over the warp of 16 values a lane: value i's total ends up in lanes 2 i and 2 i + 1 (16 shuffles).
__device__ __forceinline__ float warp_sum16(const float (&v)[16]) {
  const int lane = threadIdx.x & 31;
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float keep = lane & 16 ? v[i + 8] : v[i], give = lane & 16 ? v[i] : v[i + 8];
    a[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 16);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = lane & 8 ? a[i + 4] : a[i], give = lane & 8 ? a[i] : a[i + 4];
    b[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 8);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = lane & 4 ? b[i + 2] : b[i], give = lane & 4 ? b[i] : b[i + 2];
    c[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 4);
  }
  const float keep = lane & 2 ? c[1] : c[0], give = lane & 2 ? c[0] : c[1];
  const float s = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 2);
  return s + __shfl_xor_sync(0xFFFFFFFFu, s, 1);
}

__global__ void __launch_bounds__(kThreads, 1)
    few_tokens_kernel(const __grid_constant__ CUtensorMap tm13, const __grid_constant__ CUtensorMap tm2,
                      const __grid_constant__ CUtensorMap tm13s, const __grid_constant__ CUtensorMap tm2s,
                      const __grid_constant__ CUtensorMap sf13, const __grid_constant__ CUtensorMap sf2,
                      const __grid_constant__ CUtensorMap sf13s, const __grid_constant__ CUtensorMap sf2s,
                      const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  // (pointer arithmetic on the array keeps the accesses below shared-memory ones)
  uint8_t* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int T = a.T, E = a.E, k = a.k, d = a.d, f = a.f;
  const int kStageBytes = stage_bytes(T);
  uint8_t* s_x = ring + a.stages * kStageBytes;  // [T][2 d + 64]: the token's fp16 values
  const int x_pitch = 2 * d + 64;                // 64 bytes off a multiple of 128: two tokens a phase, no conflicts
  float* s_red = reinterpret_cast<float*>(s_x + T * x_pitch);  // [buffer][K split][row][token] partial products
  Shared& sh = *reinterpret_cast<Shared*>(s_red + (a.red_shift + 1) * kRedFloats);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Waiter wait{&sh, a.status, a.budget_ns};

  // ---------------------------------------------------------------- set-up (the warps that compute no logits)
  if (tid == kProducer * 32) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&sh.full[i], 2);
      mbar_init(&sh.empty[i], kGroupWarps + 1);  // a group's warps and an h warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.red_full[i], kMmaWarps);
      mbar_init(&sh.red_empty[i], kEpiWarps);
    }
    mbar_fence_init();
    sh.abort = 0;
  }
  if (warp == kMmaWarps) {
    sh.touched[lane] = 0u;
    if (lane < kMaxT) sh.taken[lane] = 0u;
  }
  if (warp > kMmaWarps)
    for (int i = tid - (kMmaWarps + 1) * 32; i < kMaxSlots; i += kThreads - (kMmaWarps + 1) * 32) {
      sh.slot_ready[i] = 0;
      sh.slot_mask[i] = 0u;
    }

  // ---------------------------------------------------------------- router scores
  // Thread (warp, lane) holds 8 columns at 256 warp + 8 lane of every 4096.  The raw x rows are left where their
  // fp16 form will be.
  if (warp < kMmaWarps) {
    if (tid < kMaxT) sh.e_max[tid] = -200;
    for (int e0 = blockIdx.x, first = 1; first || (a.router_w && e0 < E); e0 += 2 * gridDim.x, first = 0) {
      const bool has0 = a.router_w && e0 < E, has1 = a.router_w && e0 + (int)gridDim.x < E;
      float acc[2 * kMaxT];
#pragma unroll
      for (int t = 0; t < 2 * kMaxT; ++t) acc[t] = 0.f;
      for (int base = 0; base < d; base += kMmaWarps * 256) {
        const int c = base + warp * 256 + lane * 8;
        const bool in = c < d;
        float4 w[2][2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float4* wp = reinterpret_cast<const float4*>(a.router_w + (size_t)(e0 + z * gridDim.x) * d + c);
          const bool ok = in && (z ? has1 : has0);
          w[z][0] = ok ? __ldg(wp) : make_float4(0.f, 0.f, 0.f, 0.f);
          w[z][1] = ok ? __ldg(wp + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        uint4 raw[kMaxT];
#pragma unroll
        for (int t = 0; t < kMaxT; ++t)
          raw[t] = in && t < T ? __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)t * d + c)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int t = 0; t < kMaxT; ++t) {
          if (t >= T) continue;
          if (first && in) *reinterpret_cast<uint4*>(s_x + t * x_pitch + 2 * c) = raw[t];
          float v[8];
          bf16x8_to_f32(raw[t], v);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float& s = acc[z * kMaxT + t];
            s = fmaf(w[z][0].x, v[0], s);
            s = fmaf(w[z][0].y, v[1], s);
            s = fmaf(w[z][0].z, v[2], s);
            s = fmaf(w[z][0].w, v[3], s);
            s = fmaf(w[z][1].x, v[4], s);
            s = fmaf(w[z][1].y, v[5], s);
            s = fmaf(w[z][1].z, v[6], s);
            s = fmaf(w[z][1].w, v[7], s);
          }
        }
      }
      if (a.router_w) {
        const float v = warp_sum16(acc);
        if (!(lane & 1)) sh.part[warp][lane >> 1] = v;
        asm volatile("bar.sync 1, %0;" ::"n"(kMmaWarps * 32) : "memory");
        if (tid < 2 * kMaxT) {
          const int z = tid / kMaxT, t = tid % kMaxT;
          if (t < T && (z ? has1 : has0)) {
            float l = 0.f;
#pragma unroll
            for (int i = 0; i < kMmaWarps; ++i) l += sh.part[i][tid];
            __stcg(a.scores + (size_t)t * E + e0 + z * gridDim.x, sqrtf(softplus_f(l)));
            __threadfence();
          }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kMmaWarps * 32) : "memory");
      }
    }
    if (!a.router_w)
      asm volatile("bar.sync 1, %0;" ::"n"(kMmaWarps * 32) : "memory");  // e_max is set (above: the sums' barriers)
    else if (tid == 0)
      atomicAdd(a.counters + kFewScoresDone, 1);
    // x: the largest block exponent of each token (a warp's 256 columns at a time) ..
    for (int base = 0; base < d; base += kMmaWarps * 256) {
      const int c = base + warp * 256 + lane * 8;
      if (c >= d) break;  // d is a multiple of 256
      for (int t = 0; t < T; ++t) {
        float v[8];
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(s_x + t * x_pitch + 2 * c), v);
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
        const int e = __reduce_max_sync(0xFFFFFFFFu, mxfp8_block_exp(amax));
        if (lane == 0) atomicMax(&sh.e_max[t], e);
      }
    }
  }
  __syncthreads();
  // .. then its MXFP8 form (the codes and block exponents of moe_permute), held as fp16 code * 2^(e - E + 7) with E
  // the token's largest block exponent.  Meanwhile the warps that hold no columns select the experts.
  if (warp < kMmaWarps) {
    for (int base = 0; base < d; base += kMmaWarps * 256) {
      const int c = base + warp * 256 + lane * 8;
      if (c >= d) break;
      for (int t = 0; t < T; ++t) {
        uint8_t* at = s_x + t * x_pitch + 2 * c;
        float v[8];
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(at), v);
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const int e = mxfp8_block_exp(amax);
        const float mul = exp2_neg_int(e);
        const float up = __uint_as_float((uint32_t)(127 + max(e - sh.e_max[t] + 7, -126)) << 23);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint16_t code = e4m3x2(v[2 * i] * mul, v[2 * i + 1] * mul);
          uint32_t h2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(code));
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          const __half2 o = __floats2half2_rn(q.x * up, q.y * up);
          h[i] = *reinterpret_cast<const uint32_t*>(&o);
        }
        *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
    if (tid < T) sh.fx[tid] = ldexpf(1.f, sh.e_max[tid] - 7);
  } else if (warp - kMmaWarps < T) {
    const int t = warp - kMmaWarps;  // eight warps, up to eight tokens
    if (!a.router_w) {               // hash layer: the token's table row, ascending
      if (lane == 0) {
        int v = a.tok[t];
        if (v < 0 || v >= a.V) {
          set_status(a.status, DEV_BAD_TOKEN_ID);
          v = 0;
        }
        for (int j = 0; j < k; ++j) {
          int e = a.table[(size_t)v * k + j];
          if (e < 0 || e >= E) {
            set_status(a.status, DEV_BAD_EXPERT_ID);
            e = 0;
          }
          int b = j - 1;
          while (b >= 0 && sh.ids[t][b] > e) {
            sh.ids[t][b + 1] = sh.ids[t][b];
            --b;
          }
          sh.ids[t][b + 1] = e;
          sh.w[t][j] = a.route_scale / (float)k;
        }
      }
    } else {
      bool ok = true;
      if (lane == 0) ok = wait.count(a.counters + kFewScoresDone, (int)gridDim.x);
      if (__shfl_sync(0xFFFFFFFFu, (int)ok, 0)) {
        const float* s = a.scores + (size_t)t * E;
        if (E <= 256)
          select_token<8>(s, a.bias, E, k, a.route_scale, sh.ids[t], sh.w[t]);
        else
          select_token<16>(s, a.bias, E, k, a.route_scale, sh.ids[t], sh.w[t]);
      } else {
        if (lane < k) sh.ids[t][lane] = 0;  // the call fails; keep what follows in range
      }
    }
    __syncwarp();
    if (lane < k) {
      const int e = sh.ids[t][lane];
      const float w = sh.w[t][lane];
      if (blockIdx.x == 0) {
        a.ws_ids[t * k + lane] = e;
        a.ws_w[t * k + lane] = w;
        if (a.out_ids) a.out_ids[t * k + lane] = e;
        if (a.out_w) a.out_w[t * k + lane] = w;
      }
      atomicOr(&sh.touched[e >> 5], 1u << (e & 31));
    }
  }
  __syncthreads();
  // ---------------------------------------------------------------- slots: the shared expert, then experts ascending
  const int has_shared = a.has_shared;
  if (warp == 0) {
    const uint32_t bits = sh.touched[lane];
    int incl = __popc(bits);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    sh.before[lane] = incl - __popc(bits) + has_shared;
    if (lane == 31) sh.n_slots = incl + has_shared;
  }
  __syncthreads();
  // a thread per (token, choice); a token's repeated ids (only a faulty hash table has any) join their first choice
  const int pt = tid / kMaxK, pj = tid % kMaxK;
  const bool pair = pt < T && pj < k && (pj == 0 || sh.ids[pt][pj] != sh.ids[pt][pj - 1]);
  int ps = 0;
  float pw = 0.f;
  if (pair) {
    const int e = sh.ids[pt][pj];
    ps = sh.before[e >> 5] + __popc(sh.touched[e >> 5] & ((1u << (e & 31)) - 1u));
    sh.slot_expert[ps] = e;
    atomicOr(&sh.slot_mask[ps], 1u << pt);
    atomicOr(&sh.taken[pt], 1u << pj);
    pw = sh.w[pt][pj];
    for (int z = pj + 1; z < k && sh.ids[pt][z] == e; ++z) pw += sh.w[pt][z];
  }
  if (has_shared && tid < T) {
    sh.slot_tok[0][tid] = (uint8_t)tid;
    sh.slot_j[0][tid] = (uint8_t)k;
    if (tid == 0) {
      sh.slot_expert[0] = -1;
      sh.slot_mask[0] = (1u << T) - 1u;
    }
  }
  __syncthreads();
  if (pair) {
    const int n = __popc(sh.slot_mask[ps] & ((1u << pt) - 1u));
    sh.slot_tok[ps][n] = (uint8_t)pt;
    sh.slot_j[ps][n] = (uint8_t)pj;
    sh.w[pt][pj] = pw;
  }
  const int aborted = sh.abort;
  __syncthreads();
  if (!aborted) {
  const int S = sh.n_slots;
  const int n_up = f / 32, n_down = d / 64;  // items a slot
  const int items_up = S * n_up, items = items_up + S * n_down;
  const int kg_up = d / 128, kg_down = f / 128;

  if (warp >= kProducer) {
    // -------------------------------------------------------------- producers
    // Two warps take the stages in turn: beside busy product warps one thread's waits and copies do not keep up.  The
    // ring's 2, 4, 6 or 8 stages are even in number: a slot always belongs to the same producer.
    if (lane == 0 && !a.stall) {
      const uint64_t policy = l2_policy_evict_first();
      const int mine = warp - kProducer;
      int stage = 0, n = 0;  // ring slot and number of the next stage of the block
      uint32_t phase = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
        const bool up = it < items_up;
        const int j = up ? it : it - items_up, per = up ? n_up : n_down;
        const int s = j / per, q = j - s * per;
        const int e = sh.slot_expert[s];
        const int KG = up ? kg_up : kg_down;
        const CUtensorMap* map = up ? (e < 0 ? &tm13s : &tm13) : (e < 0 ? &tm2s : &tm2);
        const CUtensorMap* sf = up ? (e < 0 ? &sf13s : &sf13) : (e < 0 ? &sf2s : &sf2);
        const int c1 = up ? (q & 3) * 32 : (q & 3) * 64, c3 = q >> 2, half = up ? 0 : (q & 3) >> 1;
        int row = max(e, 0) * KG;  // the K group's row of the maps
        // a stage past KG brings the next rows along; nobody reads them
        for (int kg = 0; kg < KG; kg += kStageKg, row += kStageKg, ++n) {
          if ((n & 1) == mine) {
            if (!wait.bar(&sh.empty[stage], phase ^ 1u)) {
              ok = false;
              break;
            }
            uint8_t* dst = ring + stage * kStageBytes;
            uint64_t* bar = &sh.full[stage];
            if (up) {
              mbar_arrive_expect_tx(bar, kStageKg * (kTileBytes + 2 * kSfAtomBytes));
              tma_load_5d(dst, map, 0, c1, 0, c3, row, bar, policy);
              tma_load_4d(dst + kStageSf, sf, 0, 0, c3, row, bar);
              mbar_arrive(bar);  // no h to wait for
            } else {
              mbar_arrive_expect_tx(bar, kStageKg * (kTileBytes + kSfAtomBytes));
              tma_load_4d_hint(dst, map, 0, c1, c3, row, bar, policy);
              tma_load_4d(dst + kStageSf, sf, 0, half, c3, row, bar);
            }
          }
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // copies in flight must land before the block ends: this producer's stages issued last must have completed
      for (int i = max(n - a.stages, 0); i < n; ++i) {
        if ((i & 1) != mine) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait_suspend(&sh.full[i % a.stages], (uint32_t)((i / a.stages) & 1), 20000u))
          if (globaltimer_ns() - t0 > a.budget_ns) {
            wait.give_up();
            break;
          }
      }
    }
  } else if (warp < kMmaWarps) {
    // -------------------------------------------------------------- products
    // Group grp takes every second stage of the block; the ring's stages are even in number, so that a slot always
    // belongs to the same group, which sees each of its phases.  While one group waits and loads, the other computes.
    const int grp = warp / kGroupWarps, ks = warp % kGroupWarps >> 1, mh = warp & 1;  // K group of a stage, row half
    const int li = lane >> 2, lc = lane & 3;
    const int lrow = lane & 15, lblk = lane >> 4;  // ldmatrix address: rows 0..15 of the tile, block pair member
    int stage = grp, next = grp;  // ring slot and number of this group's next stage
    uint32_t phase = 0;
    int first = 0;                // number of the item's first stage
    int n_item = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x, ++n_item) {
      const bool up = it < items_up;
      const int j = up ? it : it - items_up, per = up ? n_up : n_down;
      const int s = j / per, q = j - s * per;
      const int KG = up ? kg_up : kg_down;
      const int cnt = __popc(sh.slot_mask[s]);
      const int n = li < cnt ? li : 0;  // this lane's token (columns past the slot's tokens repeat the first)
      const uint8_t* xrow = s_x + sh.slot_tok[s][n] * x_pitch + lc * 16;
      const int hrow = kStageH + n * kHPitch + ks * 256 + lc * 16;
      // Scale words of rows li, li + 8 of the warp's two row tiles: the row half is the gate (first atom) or the up rows
      // (second), or 32 of a down item's rows.
      const int quarter = up ? (q & 3) : (q & 1) * 2 + mh;
      const uint32_t sf_at = smem_addr(ring) + kStageSf + (up ? (2 * ks + mh) * kSfAtomBytes : ks * kSfAtomBytes) +
                             li * 16 + quarter * 4;
      const uint32_t row_at = smem_addr(ring) + ks * kTileBytes + (mh * 32 + lrow) * 64;
      const uint32_t x_at = smem_addr(xrow) + ks * 256, h_at = smem_addr(ring) + hrow;
      const int n_st = (KG + kStageKg - 1) / kStageKg;
      float acc[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
      bool ok = true;
      for (; next < first + n_st; next += kGroups) {
        if (!wait.bar(&sh.full[stage], phase)) {
          ok = false;
          break;
        }
        const uint32_t off = stage * kStageBytes;
        const int kg = (next - first) * kStageKg + ks;  // this warp's K group; the last stage may not have it
        uint32_t wa[2][2][4], sw[2][2];
        uint4 xb[4];
        if (kg < KG) {
          const uint32_t xp = up ? x_at + (next - first) * (kStageKg * 256) : h_at + off;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int sz = (lrow >> 1) & 3;  // 64-byte swizzle
#pragma unroll
            for (int p = 0; p < 2; ++p)  // blocks 2 p, 2 p + 1: [rows 0..7, 8..15] of each
              ldsm4(row_at + off + m * 16 * 64 + (((2 * p + lblk) ^ sz) * 16), wa[m][p]);
            sw[m][0] = lds32(sf_at + off + m * 16 * 16);
            sw[m][1] = lds32(sf_at + off + m * 16 * 16 + 8 * 16);
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) xb[b] = lds128(xp + b * 64);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);  // everything this warp needs is in registers
        if ((stage += kGroups) == a.stages + grp) {
          stage = grp;
          phase ^= 1u;
        }
        if (kg >= KG) continue;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t lo[4], hi[4];
            e2m1_f16(wa[m][b >> 1][2 * (b & 1)], lo);
            e2m1_f16(wa[m][b >> 1][2 * (b & 1) + 1], hi);
            float dd[4];
            mma_f16_zero(dd, lo[0], hi[0], lo[1], hi[1], xb[b].x, xb[b].y);
            mma_f16(dd, lo[2], hi[2], lo[3], hi[3], xb[b].z, xb[b].w);
            const float w0 = e8m0_float(sw[m][0], b), w1 = e8m0_float(sw[m][1], b);
            acc[m][0] = fmaf(dd[0], w0, acc[m][0]);
            acc[m][1] = fmaf(dd[1], w0, acc[m][1]);
            acc[m][2] = fmaf(dd[2], w1, acc[m][2]);
            acc[m][3] = fmaf(dd[3], w1, acc[m][3]);
          }
      }
      // The split is counted from the item's first stage: a row's sum does not depend on where the item came in the
      // block's sequence.
      const int split = ((grp + first) & (kGroups - 1)) * kStageKg + ks;
      first += n_st;
      if (!ok) break;
      const int buf = n_item & a.red_shift;
      if (!wait.bar(&sh.red_empty[buf], (uint32_t)(((n_item >> a.red_shift) & 1) ^ 1))) break;
      float* red = s_red + buf * kRedFloats + (split * 64 + mh * 32 + li) * kRedStride + 2 * lc;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[(m * 16 + (i >> 1) * 8) * kRedStride + (i & 1)] = acc[m][i];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.red_full[buf]);
    }
  } else if (warp < kMmaWarps + kEpiWarps) {
    // -------------------------------------------------------------- epilogue
    const int ew = warp - kMmaWarps;
    int n_item = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x, ++n_item) {
      const bool up = it < items_up;
      const int j = up ? it : it - items_up, per = up ? n_up : n_down;
      const int s = j / per, q = j - s * per;
      const int cnt = __popc(sh.slot_mask[s]);
      const int buf = n_item & a.red_shift;
      if (!wait.bar(&sh.red_full[buf], (uint32_t)((n_item >> a.red_shift) & 1))) break;
      // token n of this item belongs to warp (n + n_item) % kEpiWarps
      const int first = (ew + kEpiWarps - n_item % kEpiWarps) % kEpiWarps;
      float v0[kEpiTok], v1[kEpiTok];
#pragma unroll
      for (int i = 0; i < kEpiTok; ++i) {
        const int n = first + i * kEpiWarps;
        v0[i] = v1[i] = 0.f;
        if (n < cnt) {
          const float* red = s_red + buf * kRedFloats + lane * kRedStride + n;
#pragma unroll
          for (int z = 0; z < kSplits; ++z) {
            v0[i] += red[z * 64 * kRedStride];
            v1[i] += red[z * 64 * kRedStride + 32 * kRedStride];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.red_empty[buf]);
      // all tokens' rows first: one fence and one round of counting for them together
#pragma unroll
      for (int i = 0; i < kEpiTok; ++i) {
        const int n = first + i * kEpiWarps;
        if (n >= cnt) break;
        const int t = sh.slot_tok[s][n], ch = sh.slot_j[s][n];
        const size_t row = (size_t)t * (k + 1) + ch;
        if (up) {  // lane = column of the MX block
          const float g = fminf(v0[i] * sh.fx[t], a.limit);
          const float u = fminf(fmaxf(v1[i] * sh.fx[t], -a.limit), a.limit);
          const float hv = g / (1.f + expf(-g)) * u;
          float amax = fabsf(hv);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
          const int e = mxfp8_block_exp(amax);
          const uint16_t code = e4m3x2(hv * exp2_neg_int(e), 0.f);
          a.h[row * f + q * 32 + lane] = (uint8_t)code;
          if (lane == 0) a.h_s[row * (f / 32) + q] = (uint8_t)(e + 127);
        } else {
          const float w = ch < k ? sh.w[t][ch] : 1.f, fx = sh.hfx[n_item % kFxItems][n];
          float* dst = a.rows + row * d + q * 64;
          __stcg(dst + lane, v0[i] * fx * w);
          __stcg(dst + 32 + lane, v1[i] * fx * w);
        }
      }
      const int mine = first < cnt ? (cnt - first + kEpiWarps - 1) / kEpiWarps : 0;  // tokens of this warp
      if (mine == 0) continue;
      __threadfence();
      __syncwarp();
      if (up) {
        if (lane == 0) atomicAdd(a.counters + kFewSlotDone + s, mine);
        continue;
      }
      bool last = false;  // lane i, token i: its rows are complete in these columns
      if (lane < mine) {
        const int t = sh.slot_tok[s][first + lane * kEpiWarps];
        last = atomicAdd(a.counters + kFewColsDone + q * kMaxT + t, 1) == __popc(sh.taken[t]) + has_shared - 1;
      }
      uint32_t complete = __ballot_sync(0xFFFFFFFFu, last);
      if (complete) __threadfence();
      for (; complete; complete &= complete - 1) {
        const int t = sh.slot_tok[s][first + (__ffs(complete) - 1) * kEpiWarps];
        const float* src = a.rows + (size_t)t * (k + 1) * d + q * 64 + 2 * lane;
        float2 y = make_float2(0.f, 0.f);
        const uint32_t own = sh.taken[t];
#pragma unroll 8
        for (int z = 0; z <= k; ++z) {
          if (z < k ? !((own >> z) & 1u) : !has_shared) continue;
          const float2 r = __ldcg(reinterpret_cast<const float2*>(src + (size_t)z * d));
          y.x += r.x;
          y.y += r.y;
        }
        *reinterpret_cast<__nv_bfloat162*>(a.out + (size_t)t * d + q * 64 + 2 * lane) = __floats2bfloat162_rn(y.x, y.y);
      }
    }
  } else {
    // -------------------------------------------------------------- h slices of the down stages
    // Warp hw owns the ring slots hw, hw + n_own, .. (n_own divides the ring): into the down stages there it puts the
    // slot's tokens' next 512 columns of h, as fp16 code * 2^(e - E + 7) with E the row's largest block exponent.  It
    // waits for and releases all stages of its slots, up stages too, so that it sees each of their phases.
    const int n_own = a.stages == 6 ? 3 : min(kHWarps, a.stages), hw = warp - kMmaWarps - kEpiWarps;
    if (hw < n_own) {
      // The block's down stages are numbered from n_up_st, per_item to a down item; its first down item is it0.
      const int up_st = (kg_up + kStageKg - 1) / kStageKg, per_item = (kg_down + kStageKg - 1) / kStageKg;
      const int G = gridDim.x, b0 = blockIdx.x;
      const int n_ups = b0 < items_up ? (items_up - 1 - b0) / G + 1 : 0;
      const int it0 = b0 + n_ups * G;
      const int n_downs = it0 < items ? (items - 1 - it0) / G + 1 : 0;
      const int n_up_st = n_ups * up_st, n_st = n_up_st + n_downs * per_item;
      // Codes, block scales and row maxima of one stage for up to four tokens of its slot, fetched while earlier stages
      // run, if the slot is complete by then.
      constexpr int kAhead = 4;
      uint4 code[kAhead];
      uint32_t eb[kAhead], top[kAhead];
      auto fetch = [&](int s, int n, int part, uint4& cd, uint32_t& e, uint32_t& m) {
        const size_t row = (size_t)sh.slot_tok[s][n] * (k + 1) + sh.slot_j[s][n];
        const int c = part * kStageKg * 128 + lane * 16;  // this lane's 16 columns, half an MX block
        const bool in = c < f;
        cd = in ? __ldcg(reinterpret_cast<const uint4*>(a.h + row * f + c)) : make_uint4(0u, 0u, 0u, 0u);
        e = in ? __ldcg(a.h_s + row * (f / 32) + c / 32) : 0u;
        m = 0;
        for (int i = lane * 4; i < f / 32; i += 128)
          m = __vmaxu4(m, __ldcg(reinterpret_cast<const uint32_t*>(a.h_s + row * (f / 32) + i)));
      };
      auto place = [&](uint8_t* dst, float* fx, const uint4& cd, uint32_t e, uint32_t top4) {
        uint32_t m = __vmaxu2(top4 & 0x00FF00FFu, (top4 >> 8) & 0x00FF00FFu);
        m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
        const int x = (int)e - (int)m + 7;  // 2^x in fp16, subnormal below -14, 0 below -24
        const uint32_t p = x >= -14 ? (uint32_t)(x + 15) << 10 : x >= -24 ? 1u << (x + 24) : 0u;
        const uint32_t p2 = p | (p << 16);
        const uint32_t cw[4] = {cd.x, cd.y, cd.z, cd.w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t h2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(cw[i >> 1] >> (16 * (i & 1)))));
          asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(h2), "r"(p2));
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + 16) = make_uint4(o[4], o[5], o[6], o[7]);
        if (fx && lane == 0) *fx = ldexpf(1.f, (int)m - 134);
      };
      // whether slot s has all its h blocks; wait_for: wait until it has
      auto slot_complete = [&](int s, int cnt, bool wait_for) {
        bool yes = true;
        if (lane == 0 && !*(volatile int*)&sh.slot_ready[s]) {
          const int* c = a.counters + kFewSlotDone + s;
          yes = wait_for ? wait.count(c, n_up * cnt) : ld_acquire(c) >= n_up * cnt;
          __threadfence_block();
          if (yes) *(volatile int*)&sh.slot_ready[s] = 1;
        }
        return (bool)__shfl_sync(0xFFFFFFFFu, (int)yes, 0);
      };
      int slot = hw, s = 0, cnt = 0, di = 0, part = 0;
      uint32_t phase = 0;
      bool fetched = false, located = false;
      for (int o = hw; o < n_st; o += n_own) {
        const bool down = o >= n_up_st;
        if (down && !located) {  // stage o: part `part` of the block's down item di, slot s
          di = (o - n_up_st) / per_item;
          part = o - n_up_st - di * per_item;
          s = (it0 + di * G - items_up) / n_down;
          cnt = __popc(sh.slot_mask[s]);
        }
        bool ok = true;
        if (lane == 0) ok = wait.bar(&sh.empty[slot], phase ^ 1u);
        if (!__shfl_sync(0xFFFFFFFFu, (int)ok, 0)) break;
        if (down) {
          if (!fetched && !slot_complete(s, cnt, true)) break;
          uint8_t* dst = ring + slot * kStageBytes + kStageH + lane * 32;
          float* fx = part == 0 ? sh.hfx[(n_ups + di) % kFxItems] : nullptr;
          for (int n0 = 0; n0 < cnt; n0 += kAhead) {
            if (!fetched) {
#pragma unroll
              for (int i = 0; i < kAhead; ++i)
                if (n0 + i < cnt) fetch(s, n0 + i, part, code[i], eb[i], top[i]);
            }
            fetched = false;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
              if (n0 + i < cnt) place(dst + (n0 + i) * kHPitch, fx ? fx + n0 + i : nullptr, code[i], eb[i], top[i]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full[slot]);
        }
        if (lane == 0) mbar_arrive(&sh.empty[slot]);
        if ((slot += n_own) >= a.stages) {
          slot = hw;
          phase ^= 1u;
        }
        located = false;
        const int next = o + n_own;
        if (next >= n_up_st && next < n_st) {  // fetch ahead
          di = (next - n_up_st) / per_item;
          part = next - n_up_st - di * per_item;
          s = (it0 + di * G - items_up) / n_down;
          cnt = __popc(sh.slot_mask[s]);
          located = true;
          if (cnt <= kAhead && slot_complete(s, cnt, false)) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
              if (i < cnt) fetch(s, i, part, code[i], eb[i], top[i]);
            fetched = true;
          }
        }
      }
    }
  }
  }
  // ---------------------------------------------------------------- the last block to end clears the counters
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    sh.n_slots = atomicAdd(a.counters + kFewBlocksDone, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (sh.n_slots) {
    __threadfence();
    const int n = few_counters(d);
    for (int i = tid; i < n; i += kThreads) a.counters[i] = 0;
  }
}

}  // namespace

// Shared memory: [ring][x][partial products][Shared].  Two buffers of partial products, one where the second would
// shorten the ring.
static size_t few_smem(int T, int d, int stages, int red_shift) {
  return 1024 + (size_t)stages * stage_bytes(T) + (size_t)T * (2 * d + 64) + (size_t)(red_shift + 1) * kRedFloats * 4 +
         sizeof(Shared);
}

int few_stages(int T, int d, int* red_shift) {
  for (int n = kMaxStages; n >= 2; n -= 2)
    for (int rs = 1; rs >= 0; --rs)
      if (few_smem(T, d, n, rs) <= 232448) {
        if (red_shift) *red_shift = rs;
        return n;
      }
  return 0;
}

cudaError_t launch_few_tokens(const FewMaps& routed, const FewMaps& shared, FewArgs a, int num_sms, cudaStream_t s) {
  a.stages = few_stages(a.T, a.d, &a.red_shift);
  if (!a.stages) return cudaErrorInvalidValue;
  const size_t smem = few_smem(a.T, a.d, a.stages, a.red_shift);
  static PerDeviceOnce once;
  cudaError_t e = once.run(
      [] { return cudaFuncSetAttribute(few_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the blocks wait on one another: all of them must be resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_tokens_kernel, routed.w13, routed.w2, shared.w13, shared.w2, routed.sf13,
                            routed.sf2, shared.sf13, shared.sf2, a);
}

}  // namespace moe
