// The paged attention over an MXFP4 cache (E2M1 codes, two a byte, one E8M0 byte per 32 columns):
//
//   s_t = scale * sum_blk 2^ks[t,blk] (q . e2m1(k[t]))_blk,  p_t = exp(s_t - m),  out = sum p_t 2^vs[t] e2m1(v[t]) / sum p_t
//
// A token of a head is 136 bytes (D = 128), so unpacking and the products weigh more than memory.  What follows from it:
//  * A tile's 64 tokens belong to the block's four warps, 16 each, from the copy into shared memory to the accumulators:
//    no barrier stands inside a unit.  At its end the four warps' sums are joined through shared memory.
//  * The scores' C fragment is the A fragment of the value product as it stands: p never leaves the registers.
//  * Codes become fp16 by one conversion a pair (two cycles; moving bits to bf16 and scaling takes ten).  Which columns and
//    tokens meet in which place of a product is free, so shared memory is read in whole words: a lane's word of K holds
//    eight columns of one block, its words of V hold the same columns of two tokens, whose nibbles pair up by one shift
//    and one select for four columns.
//  * Scores: q in fp16, its row scaled by a power of two to a maximum in [2^14, 2^15); a block's scale multiplies the fp32
//    product of its 32 columns, so keys have fp32's range.
//  * Values: a code times its scale is exact in fp16 while the scale lies in [2^-28, 2^8] (2^5 times it is at least 2^-23, of
//    which half is fp16's smallest number).  Tiles with another scale, among them 255 (a block that held a NaN or an
//    infinity), are summed token by token in fp32, leaving out for each row the tokens that it does not see.
//  * p is at most 2^14 (the running maximum of a row stands 2^6 lower than its largest score, and moves when a score exceeds
//    it by 2^14): fp16 keeps eleven bits of it down to 2^-20 of the row's largest weight and some down to 2^-30.  Its sum
//    is taken in fp32, before that rounding.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_attention_fp4.h"

namespace moe {

namespace {

constexpr float kTop = 6.f;    // the largest p, in log2 units, right after the running maximum has moved
constexpr float kGrow4 = 14.f; // and the one at which it moves
constexpr int kVUp = 5;        // values are held times 2^kVUp
constexpr uint32_t kVLow = 127 - 28, kVHigh = 127 + 8;  // scale bytes that fp16 holds exactly

template <int D, int MT>
struct Cfg4 {
  static constexpr int kRows = 16 * MT;
  static constexpr int kRowBytes = D / 2;  // one token of one head
  static constexpr int kScale = D / 32;
  static constexpr int kPart = kWarpTok * kRowBytes;  // K (or V) of a warp's 16 tokens
  static constexpr int kWarpStage = (2 * kPart + 2 * kWarpTok * kScale + 127) / 128 * 128;
  static constexpr int kQPitch = 2 * D + 16;
  static constexpr int kQBytes = kRows * kQPitch;
  static constexpr int kOBytes = kWarps * kRows * D * 4;  // the warps' sums at a unit's end
  static constexpr int kStatBytes = (2 * kWarps + 2) * kRows * 4;
  static constexpr int kBlocks = MT == 1 ? 3 : 2;
  static constexpr int kBudget = (kBlocks == 2 ? 113 : 75) * 1024 - kQBytes - kOBytes - kStatBytes - 256;
  static constexpr int kFit = kBudget / (kWarps * kWarpStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kWarps * kStages * kWarpStage + kQBytes + kOBytes + kStatBytes + 256;
  static_assert(kStages >= 3, "a late scale must be stored, and a warp barrier passed, before its tile is read");
};

// Which token of eight stands at place n of a product: eight rows of K in one ldmatrix, and the words of V that a
// quarter warp reads, then fall on distinct banks.
template <int D>
__device__ __forceinline__ constexpr int token_at(int n) {
  return D == 128 ? n ^ ((n >> 1) & 1) : (n >> 1) + 4 * (n & 1);
}
// Byte of 16-byte chunk c of token t's row.
template <int D>
__device__ __forceinline__ constexpr int chunk_at(int t, int c) {
  return t * (D / 2) + (D == 128 ? c ^ ((t >> 1) & 3) : c ^ ((t >> 2) & 1)) * 16;
}

// Byte i of w, two E2M1 codes, as an fp16 pair, exact.
template <int I>
__device__ __forceinline__ uint32_t e2m1_f16(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %1;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b%2;\n}"
      : "=r"(r)
      : "r"(w), "n"(I));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ float e2m1_value(uint32_t nibble) {
  const float mag = nibble & 4u ? (nibble & 2u ? 4.f : 2.f) * (nibble & 1u ? 1.5f : 1.f)
                                : (nibble & 2u ? 1.f : 0.f) + (nibble & 1u ? 0.5f : 0.f);
  return nibble & 8u ? -mag : mag;
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, Cfg4<D, MT>::kBlocks) paged_attention_fp4_kernel(const AttnParams p) {
  using C = Cfg4<D, MT>;
  constexpr int kChunks = C::kRowBytes / 16;  // 16-byte pieces of a token row: 4 or 2
  constexpr int kBlk = D / 32;                // MX blocks of a row
  constexpr int kNT = D / 8;                  // 8-column tiles
  constexpr int kW = D / 64;                  // words of V that a lane reads of a token
  constexpr int kQN = kNT / kWarps;           // 8-column tiles of a warp in the join
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((256u - (smem_addr(smem_raw) & 255u)) & 255u);
  uint8_t* s_q = smem + kWarps * C::kStages * C::kWarpStage;
  float4* s_o = reinterpret_cast<float4*>(s_q + C::kQBytes);                 // [warp][a * kNT + n][lane]
  float* s_mx = reinterpret_cast<float*>(s_q + C::kQBytes + C::kOBytes);     // [warp][row]
  float* s_l = s_mx + kWarps * C::kRows;                                     // [warp][row]
  float* s_f = s_l + kWarps * C::kRows;                                      // [row] score factor
  int* s_lim = reinterpret_cast<int*>(s_f + C::kRows);                       // [row] first position the row does not see
  __shared__ int s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int li = lane >> 2, lc = lane & 3;
  const int mrow = lane & 7, mi = lane >> 3;  // this lane's row address in an ldmatrix of four 8 x 16-byte tiles
  pdl_trigger();
  pdl_wait();

  Run run;
  if (!deal_run(p, tid, run)) return;
  Cursor cur = run.cur;
  const int64_t t0 = run.t0, t1 = run.t1, per = run.per;
  int64_t pos = run.pos;

  // ---- loading: lane t < 16 knows where the warp's token t of the tile that is loaded next lies; kChunks lanes fetch a row
  const uint32_t ring = smem_addr(smem) + warp * C::kStages * C::kWarpStage;
  const int tok_first = warp * kWarpTok;
  constexpr int kPerIter = 32 / kChunks;  // tokens a warp instruction covers
  const uint8_t* const k_src = static_cast<const uint8_t*>(p.c.k) + lane % kChunks * 16;
  const uint8_t* const v_src = static_cast<const uint8_t*>(p.c.v) + lane % kChunks * 16;
  constexpr uint32_t kNoRow = 0xFFFFFFFFu;
  Cursor ld = cur;
  int64_t ld_pos = pos;
  int nxt_page = -1, nxt_row = 0;
  auto lookup = [&]() {
    nxt_page = -1;
    const int t = ld.t * kTile + tok_first + lane;
    if (ld_pos < t1 && lane < kWarpTok && t < ld.len) {
      const int j = page_of(t, p.pd, p.c.page_size, &nxt_row);
      nxt_page = __ldg(p.c.block_table + (int64_t)ld.b * p.c.max_pages + j);
      if ((unsigned)nxt_page >= (unsigned)p.c.n_pages) {
        set_status(p.c.status, MOE_KV_BAD_PAGE);
        nxt_page = -1;
      }
    }
  };
  uint32_t late_dst = 0;
  uint16_t late_val = 0;
  auto load_stage = [&](int stage) {
    if constexpr (D == 64) {
      if (late_dst) asm volatile("st.shared.u16 [%0], %1;" ::"r"(late_dst), "h"(late_val) : "memory");
      late_dst = 0;
    }
    if (ld_pos < t1) {
      // a row's place in 16-byte units of codes, which are 32 columns each: also the index of its first scale byte
      const uint32_t off = nxt_page >= 0 ? (uint32_t)nxt_page * p.page_units + (uint32_t)nxt_row * p.row_units +
                                               (uint32_t)ld.head * p.head_units
                                         : kNoRow;
      const uint32_t dst0 = ring + stage * C::kWarpStage;
#pragma unroll
      for (int i = 0; i < kWarpTok; i += kPerIter) {
        const int t = i + lane / kChunks;
        const uint32_t o = __shfl_sync(0xFFFFFFFFu, off, t);
        const bool ok = o != kNoRow;
        const int64_t byte = ok ? (int64_t)o * 16 : (int64_t)0;
        const uint32_t dst = dst0 + chunk_at<D>(t, lane % kChunks);
        cp_async16(dst, k_src + byte, ok);
        cp_async16(dst + C::kPart, v_src + byte, ok);
      }
      {  // lane t: K scales, lane 16 + t: V scales
        const int t = lane % kWarpTok;
        const uint32_t o = __shfl_sync(0xFFFFFFFFu, off, t);
        const bool ok = o != kNoRow, v = lane >= kWarpTok;
        const uint32_t dst = dst0 + 2 * C::kPart + lane * C::kScale;
        const uint8_t* src = (v ? p.c.v_s : p.c.k_s) + (ok ? o : 0u);
        if constexpr (D == 128) {
          cp_async4(dst, src, ok);
        } else {  // two bytes, less than cp.async copies: through a register, stored one tile later
          late_val = ok ? __ldg(reinterpret_cast<const uint16_t*>(src)) : (uint16_t)0;
          late_dst = dst;
        }
      }
      ld_pos += advance_tile(p, ld);
      lookup();
    }
    cp_async_commit();
  };
  lookup();
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) load_stage(s);

  // ---- per-unit state
  float o[MT][kNT][4];
  float m[MT][2], l[MT][2], f[MT][2];  // running maximum less kTop (log2 units), this thread's sum, score factor
  const uint32_t q_base = smem_addr(s_q);
  auto q_frag = [&](int a, int k, uint32_t (&r)[4]) {
    ldsm4(q_base + (a * 16 + (mi & 1) * 8 + mrow) * C::kQPitch + 32 * k + (mi >> 1) * 16, r);
  };

  auto begin_unit = [&]() {
    const int row0 = cur.rt * C::kRows;
    constexpr int kVec = D / 8;  // threads a row, neighbours in a warp: 16 or 8
    constexpr int kIter = C::kRows * kVec / kThreads;
    uint4 raw[kIter];
    int lim[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {  // all loads first
      const int i = it * kThreads + tid, r = row0 + i / kVec;
      const int ql = r < p.rows ? r / p.group : 0, j = r - ql * p.group;
      raw[it] = make_uint4(0u, 0u, 0u, 0u);
      lim[it] = 0;
      if (r < p.rows) {
        raw[it] = __ldg(reinterpret_cast<const uint4*>(p.q + ((int64_t)cur.b * p.L + ql) * p.q_stride +
                                                       ((int64_t)cur.head * p.group + j) * D + (i % kVec) * 8));
        lim[it] = cur.len - p.L + 1 + ql;
      }
    }
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int i = it * kThreads + tid, rr = i / kVec, c8 = i % kVec;
      uint32_t top = __vmaxu2(__vmaxu2(raw[it].x & 0x7FFF7FFFu, raw[it].y & 0x7FFF7FFFu),
                              __vmaxu2(raw[it].z & 0x7FFF7FFFu, raw[it].w & 0x7FFF7FFFu));
      top = max(top & 0xFFFFu, top >> 16);  // largest magnitude, as bf16 bits
#pragma unroll
      for (int x = 1; x < kVec; x <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
      // 2^up brings the row's maximum to [2^14, 2^15); rows below 2^-112 stay below it (their scores vanish in fp32)
      const int be = (int)(top >> 7);
      const int up = be ? min(141 - be, 126) : 126;
      const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
      const float factor =
          be == 255 ? __uint_as_float(0x7FC00000u) : p.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
      float v[8];
      bf16x8_to_f32(raw[it], v);
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = pack_f16(v[2 * e] * mul, v[2 * e + 1] * mul);
      // Lane lc's word of block b holds the columns 32 b + 8 lc ..: bytes 0, 1 are its places 2 lc, 8 + 2 lc of the
      // contraction's step 2 b, bytes 2, 3 those of step 2 b + 1.
      uint8_t* dst = s_q + rr * C::kQPitch + (c8 >> 2) * 64 + (c8 & 3) * 4;
      *reinterpret_cast<uint32_t*>(dst) = h[0];
      *reinterpret_cast<uint32_t*>(dst + 16) = h[1];
      *reinterpret_cast<uint32_t*>(dst + 32) = h[2];
      *reinterpret_cast<uint32_t*>(dst + 48) = h[3];
      if (c8 == 0) {
        s_f[rr] = factor;
        s_lim[rr] = lim[it];
      }
    }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < MT; ++a) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f[a][h] = s_f[a * 16 + li + 8 * h];
        m[a][h] = -INFINITY;
        l[a][h] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[a][n][e] = 0.f;
    }
  };

  // ---- the scores of this warp's 16 tokens, in log2 units less the reference m (or 0): s[a][j][2 h + e] is row
  // 16 a + 8 h + li, token 8 j + token_at(2 lc + e)
  float s[MT][2][4];
  auto scores = [&](uint32_t kb) {
    uint32_t kf[2][kBlk], kw[2][2];
    const uint32_t sb = kb + 2 * C::kPart;
    if constexpr (D == 128) {
#pragma unroll
      for (int j = 0; j < 2; ++j) ldsm4(kb + chunk_at<D>(8 * j + token_at<D>(mrow), mi), kf[j]);
    } else {
      uint32_t r[4];
      ldsm4(kb + chunk_at<D>(8 * (mi >> 1) + token_at<D>(mrow), mi & 1), r);
      kf[0][0] = r[0], kf[0][1] = r[1], kf[1][0] = r[2], kf[1][1] = r[3];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = sb + (8 * j + token_at<D>(2 * lc + e)) * C::kScale;
        kw[j][e] = D == 128 ? lds32(at) : lds16(at);
      }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[a][j][e] = 0.f;
#pragma unroll
    for (int b = 0; b < kBlk; ++b) {
      uint32_t h[2][4];
      float k0[2], k1[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        h[j][0] = e2m1_f16<0>(kf[j][b]);
        h[j][1] = e2m1_f16<1>(kf[j][b]);
        h[j][2] = e2m1_f16<2>(kf[j][b]);
        h[j][3] = e2m1_f16<3>(kf[j][b]);
        k0[j] = e8m0_float(kw[j][0], b);
        k1[j] = e8m0_float(kw[j][1], b);
      }
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        uint32_t q0[4], q1[4];
        q_frag(a, 2 * b, q0);
        q_frag(a, 2 * b + 1, q1);
        float d[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) mma_f16_zero(d[j], q0, h[j][0], h[j][1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) mma_f16(d[j], q1, h[j][2], h[j][3]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          fma2(s[a][j][0], s[a][j][1], d[j][0], d[j][1], k0[j], k1[j]);
          fma2(s[a][j][2], s[a][j][3], d[j][2], d[j][3], k0[j], k1[j]);
        }
      }
    }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = m[a][h] == -INFINITY ? 0.f : m[a][h];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) s[a][j][2 * h + e] = fmaf(s[a][j][2 * h + e], f[a][h], -ref);
      }
    const int tok0 = cur.t * kTile + tok_first;
    if (tok0 + kWarpTok > cur.len - p.L + 1) {  // some row does not see all of them
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int lim = s_lim[a * 16 + li + 8 * h] - tok0;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (8 * j + token_at<D>(2 * lc + e) >= lim) s[a][j][2 * h + e] = -INFINITY;
        }
    }
  };

  // The running maximum of the rows follows their scores: up to kTop below the largest.
  auto move_maximum = [&]() {
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(fmaxf(s[a][0][2 * h], s[a][0][2 * h + 1]), fmaxf(s[a][1][2 * h], s[a][1][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const float old = m[a][h], ref = old == -INFINITY ? 0.f : old;
        const float nm = fmaxf(mx + ref - kTop, old);
        const float c = old == nm ? 1.f : ex2(old - nm);
        const float less = nm == -INFINITY ? 0.f : nm - ref;
        m[a][h] = nm;
        l[a][h] *= c;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) s[a][j][2 * h + e] -= less;
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          o[a][n][2 * h] *= c;
          o[a][n][2 * h + 1] *= c;
        }
      }
  };

  // ---- o += p v; p in s
  // o[a][n][2 h + e] is column (D / 8) (2 lc + e) + n: a lane holds two runs of neighbouring columns
  auto values = [&](uint32_t vb) {
    const uint32_t sb = vb + C::kPart + kWarpTok * C::kScale;
    const int blk = D == 128 ? li >> 1 : li >> 2;
    uint32_t byte[4];  // scales of the tokens at the places 2 lc, 2 lc + 1, 8 + 2 lc, 9 + 2 lc
    uint32_t wv[4][kW];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 8 * (i >> 1) + token_at<D>(2 * lc + (i & 1));
      byte[i] = lds8(sb + t * C::kScale + blk);
      const uint32_t at = vb + (D == 128 ? chunk_at<D>(t, li >> 1) + (li & 1) * 8 : chunk_at<D>(t, li >> 2) + (li & 3) * 4);
      if constexpr (D == 128)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(wv[i][0]), "=r"(wv[i][1]) : "r"(at) : "memory");
      else
        wv[i][0] = lds32(at);
    }
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t any = wv[i][0];
      if constexpr (kW == 2) any |= wv[i][1];
      // (an all-zero block has byte 0)
      odd |= byte[i] - kVLow > kVHigh - kVLow && (byte[i] != 0 || (any & 0x77777777u) != 0);
    }
    if (__any_sync(0xFFFFFFFFu, odd)) {  // token by token
      int lim[MT][2];
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) lim[a][h] = s_lim[a * 16 + li + 8 * h] - (cur.t * kTile + tok_first);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          for (int z = 0; z < 4; ++z) {
            const int t = 8 * j + token_at<D>(2 * z + e);
            float pr[MT][2];
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
              for (int h = 0; h < 2; ++h) pr[a][h] = __shfl_sync(0xFFFFFFFFu, s[a][j][2 * h + e], (lane & ~3) | z);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int col = (D / 8) * (2 * lc + y);
              const float sc = e8m0_float(lds8(sb + t * C::kScale + col / 32), 0) * (float)(1 << kVUp);
#pragma unroll
              for (int n = 0; n < kNT; ++n) {
                const uint32_t code = lds8(vb + chunk_at<D>(t, (col + n) / 32) + (col + n) % 32 / 2) >> (4 * (n & 1));
                const float v = e2m1_value(code) * sc;
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    if (t < lim[a][h]) o[a][n][2 * h + y] = fmaf(pr[a][h], v, o[a][n][2 * h + y]);
              }
            }
          }
      return;
    }
    uint32_t pa[MT][4], mul[2];
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      pa[a][0] = pack_f16(s[a][0][0], s[a][0][1]);
      pa[a][1] = pack_f16(s[a][0][2], s[a][0][3]);
      pa[a][2] = pack_f16(s[a][1][0], s[a][1][1]);
      pa[a][3] = pack_f16(s[a][1][2], s[a][1][3]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
      mul[j] = pack_f16(__uint_as_float((byte[2 * j] + kVUp) << 23), __uint_as_float((byte[2 * j + 1] + kVUp) << 23));
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      uint32_t x[2][2];  // [place half j][even or odd columns]: a byte holds one column of the two tokens
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t a = wv[2 * j][w], b = wv[2 * j + 1][w];
        x[j][0] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
        x[j][1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
      }
      auto column = [&](auto y, int odd_col) {
        constexpr int Y = decltype(y)::value;
        const uint32_t b0 = mul_f16x2(e2m1_f16<Y>(x[0][odd_col]), mul[0]);
        const uint32_t b1 = mul_f16x2(e2m1_f16<Y>(x[1][odd_col]), mul[1]);
#pragma unroll
        for (int a = 0; a < MT; ++a) mma_f16(o[a][8 * w + 2 * Y + odd_col], pa[a], b0, b1);
      };
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        column(std::integral_constant<int, 0>{}, e);
        column(std::integral_constant<int, 1>{}, e);
        column(std::integral_constant<int, 2>{}, e);
        column(std::integral_constant<int, 3>{}, e);
      }
    }
  };

  // ---- a unit's end: the four warps' sums joined, and the rows, or this block's part of them, written
  constexpr size_t kSlot = (size_t)C::kRows * (D + 2);
  auto end_unit = [&](int64_t unit_first) {  // the first place of the unit, kUnitCost before its first tile
    const int row0 = cur.rt * C::kRows;
    const int nrows = min(C::kRows, p.rows - row0);
    float jm[MT][2], jl[MT][2];
    float4 jo[MT][kQN];  // tiles kQN warp .. of all rows
#pragma unroll
    for (int a = 0; a < MT; ++a) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[a][h] += __shfl_xor_sync(0xFFFFFFFFu, l[a][h], 1);
        l[a][h] += __shfl_xor_sync(0xFFFFFFFFu, l[a][h], 2);
        if (lc == 0) {
          s_mx[warp * C::kRows + a * 16 + li + 8 * h] = m[a][h];
          s_l[warp * C::kRows + a * 16 + li + 8 * h] = l[a][h];
        }
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n)
        s_o[(warp * MT * kNT + a * kNT + n) * 32 + lane] = make_float4(o[a][n][0], o[a][n][1], o[a][n][2], o[a][n][3]);
    }
    __syncthreads();
    float c[kWarps][MT][2];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = a * 16 + li + 8 * h;
        float top = s_mx[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_mx[w * C::kRows + r]);
        jm[a][h] = top;
        jl[a][h] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = s_mx[w * C::kRows + r];
          c[w][a][h] = mw == top ? 1.f : ex2(mw - top);
          jl[a][h] = fmaf(s_l[w * C::kRows + r], c[w][a][h], jl[a][h]);
        }
      }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int n = 0; n < kQN; ++n) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 x = s_o[(w * MT * kNT + a * kNT + warp * kQN + n) * 32 + lane];
          t.x = fmaf(x.x, c[w][a][0], t.x), t.y = fmaf(x.y, c[w][a][0], t.y);
          t.z = fmaf(x.z, c[w][a][1], t.z), t.w = fmaf(x.w, c[w][a][1], t.w);
        }
        jo[a][n] = t;
      }
    const int64_t first_tile = unit_first + kUnitCost, unit_end = first_tile + cur.nt;
    auto write_rows = [&]() {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = a * 16 + li + 8 * h;
          if (r >= nrows) continue;
          const int ql = (row0 + r) / p.group, j = row0 + r - ql * p.group;
          const float z = jl[a][h];
          const float inv = z == 0.f ? 0.f : (1.f / (float)(1 << kVUp)) / z;  // a row that sees nothing is 0
          const int64_t token = (int64_t)cur.b * p.L + ql;
          const int head = cur.head * p.group + j;
          __nv_bfloat16* dst = p.out + token * p.out_stride + (int64_t)head * D + warp * kQN;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t w[kQN / 2];
#pragma unroll
            for (int n = 0; n < kQN; n += 2) {
              const float4 x0 = jo[a][n], x1 = jo[a][n + 1];
              w[n / 2] = pack_bf16((h ? (y ? x0.w : x0.z) : (y ? x0.y : x0.x)) * inv,
                                   (h ? (y ? x1.w : x1.z) : (y ? x1.y : x1.x)) * inv);
            }
            __nv_bfloat16* at = dst + (D / 8) * (2 * lc + y);
            if constexpr (kQN == 4)
              *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
            else
              *reinterpret_cast<uint32_t*>(at) = w[0];
          }
          // (m is -inf where no score was above it: z = 0 then gives -inf, a NaN among the scores NaN)
          if (p.lse && warp == 0 && lc == 0) p.lse[token * p.Hq + head] = (jm[a][h] + log2f(z)) * kLn2;
        }
    };
    if (first_tile >= t0 && unit_end <= t1) {  // the whole unit was this block's
      write_rows();
      return;
    }
    // A part is kept as the lanes hold it: [a * kNT + tile][lane], then m and l of the rows.
    auto put_part = [&](float* slot) {
      float4* dst = reinterpret_cast<float4*>(slot);
#pragma unroll
      for (int a = 0; a < MT; ++a) {
#pragma unroll
        for (int n = 0; n < kQN; ++n) __stcg(dst + (a * kNT + warp * kQN + n) * 32 + lane, jo[a][n]);
        if (warp == 0 && lc == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __stcg(slot + C::kRows * D + a * 16 + li + 8 * h, jm[a][h]);
            __stcg(slot + C::kRows * (D + 1) + a * 16 + li + 8 * h, jl[a][h]);
          }
        }
      }
    };
    // jo, jm, jl = the parts 0 .. n_parts - 1 joined in this order
    auto join = [&](int n_parts, auto slot_of) {
#pragma unroll
      for (int a = 0; a < MT; ++a) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          jm[a][h] = -INFINITY;
          jl[a][h] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < kQN; ++n) jo[a][n] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      // kIn parts are under way at once, the last ones repeated where fewer are left
      constexpr int kIn = 2;
      for (int i0 = 0; i0 < n_parts; i0 += kIn) {
        float pm[kIn][MT][2], pl[kIn][MT][2];
        float4 po[kIn][MT][kQN];
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          const float* src = slot_of(min(i0 + u, n_parts - 1));
#pragma unroll
          for (int a = 0; a < MT; ++a) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              pm[u][a][h] = __ldcg(src + C::kRows * D + a * 16 + li + 8 * h);
              pl[u][a][h] = __ldcg(src + C::kRows * (D + 1) + a * 16 + li + 8 * h);
            }
#pragma unroll
            for (int n = 0; n < kQN; ++n)
              po[u][a][n] = __ldcg(reinterpret_cast<const float4*>(src) + (a * kNT + warp * kQN + n) * 32 + lane);
          }
        }
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          if (i0 + u >= n_parts) break;
#pragma unroll
          for (int a = 0; a < MT; ++a) {
            float c0[2], c1[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float nm = fmaxf(jm[a][h], pm[u][a][h]);
              c0[h] = jm[a][h] == nm ? 1.f : ex2(jm[a][h] - nm);
              c1[h] = pm[u][a][h] == nm ? 1.f : ex2(pm[u][a][h] - nm);
              jm[a][h] = nm;
              jl[a][h] = fmaf(pl[u][a][h], c1[h], jl[a][h] * c0[h]);
            }
#pragma unroll
            for (int n = 0; n < kQN; ++n) {
              const float4 x = po[u][a][n];
              jo[a][n].x = fmaf(x.x, c1[0], jo[a][n].x * c0[0]);
              jo[a][n].y = fmaf(x.y, c1[0], jo[a][n].y * c0[0]);
              jo[a][n].z = fmaf(x.z, c1[1], jo[a][n].z * c0[1]);
              jo[a][n].w = fmaf(x.w, c1[1], jo[a][n].w * c0[1]);
            }
          }
        }
      }
    };
    // counts this block in; true for the last of n
    auto last_of = [&](int* counter, int n) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        s_last = atomicAdd(counter, 1) == n - 1;
        if (s_last) *counter = 0;
      }
      __syncthreads();
      if (!s_last) return false;
      __threadfence();
      return true;
    };
    // slot 0 of a block is the unit its run begins in, slot 1 the one that it ends in
    const int b0 = (int)(first_tile / per), b1 = (int)((unit_end - 1) / per), parts = b1 - b0 + 1;
    auto block_slot = [&](int b) { return p.partial + ((size_t)b * 2 + (unit_first > b * per ? 1 : 0)) * kSlot; };
    put_part(block_slot(blockIdx.x));
    int* counter = p.counters + b0;
    if (parts <= kJoin) {
      if (!last_of(counter, parts)) return;
      join(parts, [&](int i) { return block_slot(b0 + i); });
    } else {
      // many parts: blocks 16 g .. 16 g + 15 are joined first, then these groups.  A group can hold the end of one
      // such unit and the beginning of the next, told apart as slots are.
      auto group_at = [&](int g) { return (size_t)g * 2 + (unit_first > (int64_t)g * kJoin * per ? 1 : 0); };
      const int g0 = b0 / kJoin, g1 = b1 / kJoin, g = blockIdx.x / kJoin;
      const int first = max(b0, g * kJoin), n = min(b1, g * kJoin + kJoin - 1) - first + 1;
      if (!last_of(p.group_counters + group_at(g), n)) return;
      join(n, [&](int i) { return block_slot(first + i); });
      put_part(p.group_partial + group_at(g) * kSlot);
      if (!last_of(counter, g1 - g0 + 1)) return;
      join(g1 - g0 + 1, [&](int i) { return p.group_partial + group_at(g0 + i) * kSlot; });
    }
    write_rows();
  };

  // ---- the run
  int stage = 0;
  bool fresh = true;
  while (pos < t1) {
    if (fresh) {
      begin_unit();
      fresh = false;
    }
    cp_async_wait<C::kStages - 2>();
    __syncwarp();  // the warp's tokens have landed for all its lanes, and all are done with the previous ones
    load_stage(stage == 0 ? C::kStages - 1 : stage - 1);
    const uint32_t kb = ring + stage * C::kWarpStage;
    scores(kb);
    bool grow = false;
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        grow |= fmaxf(fmaxf(s[a][0][2 * h], s[a][0][2 * h + 1]), fmaxf(s[a][1][2 * h], s[a][1][2 * h + 1])) >
                (m[a][h] == -INFINITY ? -INFINITY : kGrow4);
    if (__any_sync(0xFFFFFFFFu, grow)) move_maximum();
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) s[a][j][2 * h + e] = ex2(s[a][j][2 * h + e]);
        l[a][h] += (s[a][0][2 * h] + s[a][0][2 * h + 1]) + (s[a][1][2 * h] + s[a][1][2 * h + 1]);
      }
    values(kb + C::kPart);
    stage = stage == C::kStages - 1 ? 0 : stage + 1;
    if (cur.t + 1 == cur.nt || pos + 1 == t1) {
      end_unit(pos - cur.t - kUnitCost);
      fresh = true;
    }
    pos += advance_tile(p, cur);
  }
  cp_async_wait<0>();
}

template <int D, int MT>
cudaError_t launch_one(const AttnParams& p, int num_sms, cudaStream_t s) {
  using C = Cfg4<D, MT>;
  auto* kernel = paged_attention_fp4_kernel<D, MT>;
  static PerDeviceOnce once;
  cudaError_t e =
      once.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(num_sms * C::kBlocks), dim3(kThreads), C::kSmem, s, p);
}

}  // namespace

int attention_fp4_tile_rows(int64_t rows) { return rows <= 16 ? 16 : 32; }

int attention_fp4_blocks(int head_dim, int tile_rows) {
  return head_dim == 128 ? (tile_rows == 16 ? Cfg4<128, 1>::kBlocks : Cfg4<128, 2>::kBlocks)
                         : (tile_rows == 16 ? Cfg4<64, 1>::kBlocks : Cfg4<64, 2>::kBlocks);
}

cudaError_t launch_attention_fp4(const AttnParams& p, int num_sms, cudaStream_t s) {
  const bool one = attention_fp4_tile_rows(p.rows) == 16;
  if (p.c.head_dim == 128) return one ? launch_one<128, 1>(p, num_sms, s) : launch_one<128, 2>(p, num_sms, s);
  return one ? launch_one<64, 1>(p, num_sms, s) : launch_one<64, 2>(p, num_sms, s);
}

}  // namespace moe
