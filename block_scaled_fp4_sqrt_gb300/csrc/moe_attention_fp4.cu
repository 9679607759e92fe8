// The paged attention over an MXFP4 cache (E2M1 codes, two a byte, one E8M0 byte per 32 columns):
//
//   s_t = scale * sum_blk 2^ks[t,blk] (q . e2m1(k[t]))_blk,  p_t = exp(s_t - m),  out = sum p_t 2^vs[t] e2m1(v[t]) / sum p_t
//
// A token of a head is 136 bytes (D = 128), so instructions and their latencies at eight to twelve warps an SM bound it, not
// memory.  64 requests of 100 to 8000 tokens, 8 x 4 heads of 128: one row 41 us (floor 19; 3.1 TB/s), eight rows 90 us (floor
// 20; the products alone 26 on mma.sync); three requests of up to 131,071 tokens 65 us (floor 36, 3.8 TB/s); one request of
// 333 tokens 9 us; two prompts of 500 tokens over up to 3001, 4 x 4 heads of 64, 60.5 us (136 TFLOP/s).  Of the 90 us about 15
// are units' beginnings and ends (two or three to a block), 6 dealing and the first loads, the rest 2,500 cycles a tile, of
// which the softmax's chain of dependent instructions is 900 and a fifth of the instructions the loader's.  What follows:
//  * The products are transposed, S^T = K q^T and O^T = V^T P^T: the 16-row side of a product holds tokens or columns, the
//    8-column side the rows of q, so that one to eight rows cost half of what they would the other way round.
//  * A tile's tokens belong to the block's four warps, WT each, from the copy into shared memory to the accumulators: no
//    barrier stands inside a unit.  At its end the four warps' sums are joined through shared memory.
//  * p goes from the scores' accumulators to the operand of the value product by one transposition of 8 x 8 registers
//    (movmatrix) for eight tokens of eight rows; it never lies in memory.
//  * Codes become fp16 by one conversion a pair (two cycles of the ALU; moving bits to bf16 and scaling takes ten).  Which
//    columns and tokens meet in which place of a product is free, so shared memory is read in whole words: a lane's word of
//    K holds eight columns of one block, its words of V hold the same columns of two tokens, whose nibbles pair up by one
//    shift and one select for four columns.
//  * Scales are converted once, by the lane that fetches the token, on their way to shared memory.
//  * Scores: q in fp16, its row scaled by a power of two to a maximum in [2^14, 2^15); a block's scale multiplies the fp32
//    product of its 32 columns, so keys have fp32's range.
//  * Values: a code times its scale is exact in fp16 while the scale lies in [2^-28, 2^8] (2^5 times it is at least 2^-23, of
//    which half is fp16's smallest number).  A block of 32 columns with another scale, among them 255 (it held a NaN or an
//    infinity), takes part in the products with the multiplier 0 and is added in fp32, for each row that sees its token.
//  * p is at most 2^14: a row's reference stands 6 below its largest score, in log2 units, and moves when a score exceeds it
//    by 14, for the row's own scores alone, so that neither other rows nor tokens that it does not see change its bits.  fp16
//    keeps eleven bits of p down to 2^-20 of the row's largest weight and some down to 2^-30.  Its sum is taken in fp32,
//    before that rounding.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_attention_fp4.h"

namespace moe {

namespace {

constexpr float kTop = 6.f;     // the largest p, in log2 units, right after a row's reference has moved
constexpr float kGrow4 = 14.f;  // and the one at which it moves
constexpr int kVUp = 5;         // values are held times 2^kVUp
// scale bytes at which fp16 holds every code times its scale exactly: half of 2^-23 is its smallest number, 6 2^13 below its
// largest
constexpr uint32_t kVLow = 127 - 23 - kVUp, kVHigh = 127 + 13 - kVUp;

// RT: rows of a row tile, in eights.
template <int D, int RT>
struct Cfg4 {
  static constexpr int kRows = 8 * RT;
  // Tokens of a tile that a warp fetches, and works on at once.  Us for 64 requests, one and eight rows a head: 32 and 32
  // tokens 44 (16 and 16: 54, with a fourth block 52), 32 and 16 tokens 91 (16 and 16: 104).
  static constexpr int kTok = 32;
  static constexpr int kStep = RT <= 2 ? 32 : 16;
  static constexpr int kTile = kWarps * kTok;
  // what beginning and ending a unit costs when the work is dealt, in tiles
  static constexpr int kCost = RT == 1 || D == 64 ? 2 : 3;
  static constexpr int kRowBytes = D / 2;  // one token of one head
  static constexpr int kBlk = D / 32;      // MX blocks of a row
  static constexpr int kPart = kTok * kRowBytes;  // K (or V) of a warp's tokens
  // a warp's stage: K, V, the scales of K in fp32 [token][block], of V in fp16 times 2^kVUp [block][place], and V's bytes
  static constexpr int kKs = 2 * kPart, kVs = kKs + kTok * kBlk * 4, kVb = kVs + kTok * kBlk * 2;
  static constexpr int kWarpStage = (kVb + kTok * kBlk + 127) / 128 * 128;
  static constexpr int kQPitch = 2 * D + 16;
  static constexpr int kQBytes = kRows * kQPitch;
  // the warps' sums at a unit's end, of kORound pairs of columns a warp of eight rows at a time; two buffers, where there is
  // room, so that one is written while the other is read
  static constexpr int kORound = RT == 2 ? D / 64 : 1;
  static constexpr int kOPart = kORound * kWarps * kWarps * 32 * 16;
  static constexpr int kOBuffers = RT > 1 ? 2 : 1;
  static constexpr int kOBytes = kOBuffers * kOPart;
  static constexpr int kStatBytes = (3 * kWarps + 1) * kRows * 4;
  // an SM.  (D = 64, 16 rows and more, with two blocks: 64 x 8 rows 64 us for 57, two prompts 65 for 61.)
  static constexpr int kBlocks = RT == 1 || (D == 64 && RT <= 4) ? 3 : 2;
  // The accumulators leave no registers for the loader's state and the sums of p: they stay in shared memory between the
  // steps.  (Spilled by the compiler they wait for the L2, as shared memory leaves the L1 28 KB.  64 x 8 rows: 102 -> 93 us.)
  static constexpr bool kFar = RT * D >= 384;
  static constexpr int kFarBytes = kFar ? (48 + 8 * RT) * kThreads : 0;
  static constexpr int kBudget =
      (kBlocks == 2 ? 113 : 75) * 1024 - kFarBytes - 512 - kQBytes - kOBytes - kStatBytes - 256;
  static constexpr int kFit = kBudget / (kWarps * kWarpStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kWarps * kStages * kWarpStage + kQBytes + kOBytes + kStatBytes + 256;
  static constexpr bool kQRegs = RT == 1;  // q fragments stay in registers, or are read for every step
  static_assert(kStages >= 3, "scales are stored one load after their codes, and a warp barrier passed, before they are read");
};

// Which token of eight stands at place n of a product, and the inverse: eight rows of K in one ldmatrix, and the words of V
// that a quarter warp reads, then fall on distinct banks.
template <int D>
__device__ __forceinline__ constexpr int token_at(int n) {
  return D == 128 ? n ^ ((n >> 1) & 1) : (n >> 1) + 4 * (n & 1);
}
template <int D>
__device__ __forceinline__ constexpr int place_of(int t) {
  return D == 128 ? t ^ ((t >> 1) & 1) : 2 * (t & 3) + (t >> 2);
}
// Byte of 16-byte chunk c of token t's row.
template <int D>
__device__ __forceinline__ constexpr int chunk_at(int t, int c) {
  return t * (D / 2) + (D == 128 ? c ^ ((t >> 1) & 3) : c ^ ((t >> 2) & 1)) * 16;
}

// Byte of the first of the columns (D / 8) c .. of token t's row.
template <int D>
__device__ __forceinline__ constexpr int v_at(int t, int c) {
  return D == 128 ? chunk_at<D>(t, c >> 1) + (c & 1) * 8 : chunk_at<D>(t, c >> 2) + (c & 3) * 4;
}

// Byte I of w, two E2M1 codes, as an fp16 pair, exact.
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
// (c0, c1) += (a0, a1)
__device__ __forceinline__ void add2(float& c0, float& c1, float a0, float a1) {
  asm("{\n .reg .b64 a, c;\n mov.b64 a, {%2, %3};\n mov.b64 c, {%0, %1};\n add.rn.f32x2 c, c, a;\n"
      " mov.b64 {%0, %1}, c;\n}"
      : "+f"(c0), "+f"(c1)
      : "f"(a0), "f"(a1));
}
// The 8 x 8 matrix of 16-bit elements that the lanes hold (row lane / 4, columns 2 (lane % 4) ..), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ float2 f16x2_float(uint32_t w) {
  float2 r;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}" : "=f"(r.x), "=f"(r.y) : "r"(w));
  return r;
}
// E8M0 bytes 0, 1 (or 2, 3) of w as a bf16 pair, exact.
__device__ __forceinline__ uint32_t e8m0_bf16x2(uint32_t w, bool high) {
  uint32_t r;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"((uint16_t)(high ? w >> 16 : w)));
  return r;
}

// A warp's loader: the tile whose pages have been asked for last (and the places that are left from it on); this lane's
// page and row of its token there, not yet checked (row -1: no token); the place of its token of the tile before that one,
// which is loaded next, its scales, those of the tile before it, and whether there is such a tile.
union Loader {
  struct {
    struct {
      int b, head, rt, t, len, left;
    } ld;
    int row;
    uint32_t off, k_old, v_old;
    int any;
  };
  uint4 w[3];
};

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, Cfg4<D, RT>::kBlocks) paged_attention_fp4_kernel(const AttnParams p) {
  using C = Cfg4<D, RT>;
  constexpr int kTile = C::kTile, kCost = C::kCost, kTok = C::kTok, kBlk = C::kBlk;
  constexpr int kSteps = C::kStep / 16;       // products' steps of 16 tokens that are under way at once
  constexpr int kChunks = C::kRowBytes / 16;  // 16-byte pieces of a token row: 4 or 2
  constexpr int kPairs = D / 16;              // pairs of columns that a lane accumulates of a row
  constexpr int kW = D / 64;                  // words of V that a lane reads of a token
  constexpr int kJoinPairs = kPairs / kWarps; // of a warp in the join
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((256u - (smem_addr(smem_raw) & 255u)) & 255u);
  uint8_t* s_q = smem + kWarps * C::kStages * C::kWarpStage;
  float4* s_o = reinterpret_cast<float4*>(s_q + C::kQBytes);                 // [buffer][warp][pair][lane]
  // [warp][row]: the row's score factor, and minus the warp's reference for it (running maximum less kTop, log2 units)
  float2* s_fr = reinterpret_cast<float2*>(s_q + C::kQBytes + C::kOBytes);
  float* s_l = reinterpret_cast<float*>(s_fr + kWarps * C::kRows);           // [warp][row]
  int* s_lim = reinterpret_cast<int*>(s_l + kWarps * C::kRows);              // [row] first position the row does not see
  __shared__ int s_last;
  // What a unit keeps in shared memory is ordered by barriers:
  //   s_q, s_lim, s_fr.x, s_row  written between begin_unit's two barriers; read until the next unit's first one (s_row last, by
  //                              write_rows, behind end_unit's barriers)
  //   s_fr.y, s_unit             written behind begin_unit's second barrier; read until the next unit's first one
  //   s_l, s_o                   written and read in end_unit, with a barrier between
  __shared__ int3 s_unit;           // request, head, row tile
  __shared__ int2 s_row[C::kRows];  // a row's token (request, new token) of the call and its query head; token -1: no such row
  __shared__ uint4 s_loader[C::kFar ? 3 * kThreads : 1];
  __shared__ float2 s_sums[C::kFar ? RT * kThreads : 1];
  __shared__ uint32_t s_odd[kWarps][C::kStages];  // tokens whose V has a scale that fp16 does not hold

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int li = lane >> 2, lc = lane & 3;
  const int mrow = lane & 7, mi = lane >> 3;  // this lane's row address in an ldmatrix of four 8 x 16-byte tiles
  // Blocks `lanes` g .. have the same run over the requests, each of another kv head: what lies together in memory (a token's
  // heads, the scale bytes of eight of them in one sector) is read at the same time.
  const int lanes = p.lanes, head_groups = p.c.n_kv_heads / lanes, groups = gridDim.x / lanes;
  const int g = blockIdx.x / lanes, lane_head = blockIdx.x - g * lanes;
  if (g >= groups) return;
  pdl_trigger();
  pdl_wait();

  // the run's ends are read from shared memory where they are needed: the accumulators leave no registers for them
  // (a run is shorter than 2^31 places: its tiles would take hours)
  __shared__ int64_t s_t0, s_t1, s_per;
  Cursor cur;
  int left;  // places from cur to the run's end
  {
    Run run;
    if (!deal_run<kTile, kCost>(p, head_groups, groups, g, tid, run)) return;
    if (tid == 0) s_t0 = run.t0, s_t1 = run.t1, s_per = run.per;
    __syncthreads();
    cur = run.cur;
    left = (int)(run.t1 - run.pos);
  }

  // To the next tile, as advance_tile, without the number of a unit's tiles in a register.
  auto advance = [&](auto& c) {
    if (++c.t < tiles_of<kTile>(c.len)) return 1;
    c.t = 0;
    if (++c.rt < p.row_tiles) return 1 + kCost;
    c.rt = 0;
    if (++c.head < head_groups) return 1 + kCost;
    c.head = 0;
    if (++c.b < p.c.n_seqs) c.len = seq_len_of(p.c, c.b);
    return 1 + kCost;
  };

  // This lane's places in a stage, kept in registers (the compiler would work them out again at every step): no multiple of
  // eight tokens changes a row's swizzle.
  uint32_t at_load = chunk_at<D>(lane / kChunks, lane % kChunks);          // its 16 bytes of a row that it fetches
  uint32_t at_k = D == 128 ? chunk_at<D>(token_at<D>(mrow), mi) : chunk_at<D>(8 * (mi >> 1) + token_at<D>(mrow), mi & 1);
  uint32_t at_ks = C::kKs + token_at<D>(li) * kBlk * 4;                    // the scales of its tokens' keys
  uint32_t at_v0 = C::kPart + v_at<D>(token_at<D>(2 * lc), li), at_v1 = C::kPart + v_at<D>(token_at<D>(2 * lc + 1), li);
  uint32_t at_vs = C::kVs + ((D == 128 ? li >> 1 : li >> 2) * kTok + 2 * lc) * 2;
  uint32_t at_q = smem_addr(s_q) + mrow * C::kQPitch + mi * 16;
  uint32_t at_fr = smem_addr(s_fr) + (warp * C::kRows + 2 * lc) * 8;
  asm volatile("" : "+r"(at_load), "+r"(at_k), "+r"(at_ks), "+r"(at_v0), "+r"(at_v1), "+r"(at_vs), "+r"(at_q), "+r"(at_fr));

  // ---- loading: lane t < kTok looks up where the warp's token t lies; kChunks lanes fetch a row of codes.  The scales take
  // the way through lane t's registers.  Nothing waits for memory here: a tile's pages are looked up two steps before its
  // codes are asked for, its scales are asked for one step before them and stored, converted, one step after them.  (A page
  // checked right after its lookup held every step up for the lookup: 1,200 of 3,700 cycles.)
  const uint32_t ring = smem_addr(smem) + warp * C::kStages * C::kWarpStage;
  const int tok_first = warp * kTok;
  constexpr int kPerIter = 32 / kChunks;  // tokens a warp instruction covers
  constexpr uint32_t kNoRow = 0xFFFFFFFFu;
  Loader keep{};  // stays in registers, or (many accumulators) in shared memory between the steps; what memory has been
  int page = 0;   // asked for stays in registers: nothing may wait for it
  uint32_t k_scale = 0, v_scale = 0;
  keep.ld = {cur.b, cur.head, cur.rt, cur.t, cur.len, left};
  auto lookup = [&](Loader& x) {
    x.row = -1;
    const int t = x.ld.t * kTile + tok_first + lane;
    if (x.ld.left > 0 && lane < kTok && t < x.ld.len) {
      const int j = page_of(t, p.pd, p.c.page_size, &x.row);
      page = __ldg(p.c.block_table + (int64_t)x.ld.b * p.c.max_pages + j);
    }
  };
  // The tile that was looked up becomes the next to be loaded: its scales are asked for, and the pages of the one behind it.
  auto look_ahead = [&](Loader& x) {
    // a row's place in 16-byte units of codes, which are 32 columns each: also the index of its first scale byte
    x.off = kNoRow;
    x.any = x.ld.left > 0;
    if (x.row >= 0) {
      if ((unsigned)page < (unsigned)p.c.n_pages)
        x.off = (uint32_t)page * p.page_units + (uint32_t)x.row * p.row_units +
                (uint32_t)(x.ld.head * lanes + lane_head) * p.head_units;
      else
        set_status(p.c.status, MOE_KV_BAD_PAGE);
    }
    x.k_old = k_scale, x.v_old = v_scale;
    k_scale = v_scale = 0x7F7F7F7Fu;  // (a place without a token: codes 0, any scale that is no NaN)
    if (x.off != kNoRow) {
      if constexpr (D == 128) {
        k_scale = __ldg(reinterpret_cast<const uint32_t*>(p.c.k_s + x.off));
        v_scale = __ldg(reinterpret_cast<const uint32_t*>(p.c.v_s + x.off));
      } else {
        k_scale = __ldg(reinterpret_cast<const uint16_t*>(p.c.k_s + x.off));
        v_scale = __ldg(reinterpret_cast<const uint16_t*>(p.c.v_s + x.off));
      }
    }
    if (x.ld.left > 0) {
      x.ld.left -= advance(x.ld);
      lookup(x);
    }
  };
  auto store_scales = [&](int stage, uint32_t ks_bytes, uint32_t vs_bytes) {
    const uint32_t at = ring + stage * C::kWarpStage;
    bool odd = false;
    if (lane < kTok) {
      const uint32_t v_at = at + C::kVs + ((lane & ~7) + place_of<D>(lane & 7)) * 2;
      const uint32_t k0 = e8m0_bf16x2(ks_bytes, false);
#pragma unroll
      for (int b = 0; b < kBlk; b += 2) {
        const uint32_t vs = e8m0_bf16x2(vs_bytes, b == 2), vb = __byte_perm(vs_bytes, 0, b == 2 ? 0x4342 : 0x4140);
        uint32_t vh = pack_f16(__uint_as_float(vs << 16) * (float)(1 << kVUp),
                               __uint_as_float(vs & 0xFFFF0000u) * (float)(1 << kVUp));
        if (vb != __vminu2(__vmaxu2(vb, kVLow * 0x10001u), kVHigh * 0x10001u)) {
          odd = true;
          vh &= __vcmpleu2(kVLow * 0x10001u, vb) & __vcmpleu2(vb, kVHigh * 0x10001u);
        }
        sts16(v_at + b * kTok * 2, vh);
        sts16(v_at + (b + 1) * kTok * 2, vh >> 16);
      }
      if constexpr (D == 128) {
        const uint32_t k1 = e8m0_bf16x2(ks_bytes, true);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + C::kKs + lane * 16), "r"(k0 << 16),
                     "r"(k0 & 0xFFFF0000u), "r"(k1 << 16), "r"(k1 & 0xFFFF0000u)
                     : "memory");
        sts32(at + C::kVb + lane * 4, vs_bytes);
      } else {
        asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at + C::kKs + lane * 8), "r"(k0 << 16), "r"(k0 & 0xFFFF0000u)
                     : "memory");
        sts16(at + C::kVb + lane * 2, vs_bytes);
      }
    }
    const uint32_t any = __ballot_sync(0xFFFFFFFFu, odd);
    if (lane == 0) s_odd[warp][stage] = any;
  };
  // Fills a stage with the next tile, and puts the scales of the one before it in their place: they have arrived, but for the
  // run's first tiles, whose codes are asked for before the wait.
  auto put_loader = [&](const Loader& x) {
#pragma unroll
    for (int i = 0; i < 3; ++i) s_loader[i * kThreads + tid] = x.w[i];
  };
  auto get_loader = [&](Loader& x) {
#pragma unroll
    for (int i = 0; i < 3; ++i) x.w[i] = s_loader[i * kThreads + tid];
  };
  auto load_stage = [&](int stage, Loader& x, auto at_start) {
    constexpr bool kAtStart = decltype(at_start)::value;
    const int before = stage == 0 ? C::kStages - 1 : stage - 1;
    const uint32_t k_old = x.k_old, v_old = x.v_old;
    if (!kAtStart) store_scales(before, k_old, v_old);
    if (x.any) {
      const uint32_t dst0 = ring + stage * C::kWarpStage;
      auto rows = [&](auto all) {
        constexpr bool ALL = decltype(all)::value;
#pragma unroll
        for (int i = 0; i < kTok; i += kPerIter) {
          const int t = i + lane / kChunks;
          uint32_t o = __shfl_sync(0xFFFFFFFFu, x.off, t);
          const bool ok = ALL || o != kNoRow;
          if (!ok) o = 0;
          const int64_t byte = ((int64_t)o + lane % kChunks) * 16;
          const uint32_t dst = dst0 + at_load + i * C::kRowBytes;
          cp_async16(dst, static_cast<const uint8_t*>(p.c.k) + byte, ok);
          cp_async16(dst + C::kPart, static_cast<const uint8_t*>(p.c.v) + byte, ok);
        }
      };
      if (__all_sync(0xFFFFFFFFu, x.off != kNoRow || lane >= kTok))
        rows(std::true_type{});
      else
        rows(std::false_type{});
    }
    cp_async_commit();
    look_ahead(x);
    if (kAtStart && stage > 0) store_scales(before, k_old, v_old);
  };
  int stage = -1;  // of the tile that is worked on; below 0 before the run's first tiles have been asked for
  auto load_first = [&]() {
    look_ahead(keep);
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) load_stage(s, keep, std::true_type{});
    if constexpr (C::kFar) put_loader(keep);
    stage = 0;
  };
  lookup(keep);
  if constexpr (C::kFar) load_first();  // (at the place below it costs registers)

  // ---- per-unit state.  This lane's rows: 8 a + 2 lc + e; o[a][i][2 c + e] is column (D / 8) li + 2 i + c of such a row.
  uint32_t qb[C::kQRegs ? RT : 1][C::kQRegs ? kBlk : 1][4];
  float o[RT][kPairs][4];
  // This lane's sums of p, in registers or (many accumulators) in shared memory.
  struct Sums {
    float2 in_reg[C::kFar ? 1 : RT];
    float2* far;
    __device__ __forceinline__ float2 get(int a) const { return C::kFar ? far[a * kThreads] : in_reg[a]; }
    __device__ __forceinline__ void set(int a, float2 v) { (C::kFar ? far[a * kThreads] : in_reg[a]) = v; }
  } l;
  l.far = s_sums + tid;
  uint32_t unseen;           // rows (bit 2 a + e) that have not met a score yet: their reference is 0
  bool open;                 // some lane's rows are among those
  int seen_end;              // the first position that no row of the unit sees
  // B fragments of rows 8 a .. for the two steps of block b's contraction
  auto q_frag = [&](int a, int b, uint32_t (&r)[4]) { ldsm4(at_q + a * 8 * C::kQPitch + 64 * b, r); };

  auto begin_unit = [&]() {
    const int row0 = cur.rt * C::kRows;
    constexpr int kVec = D / 8;  // threads a row, neighbours in a warp: 16 or 8
    constexpr int kIter = (C::kRows * kVec + kThreads - 1) / kThreads;
    uint4 raw[kIter];
    int lim[kIter];
    int2 place[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {  // all loads first
      const int i = it * kThreads + tid, r = row0 + i / kVec;
      const bool in = i / kVec < C::kRows && r < p.rows;
      const int ql = in ? r / p.group : 0, j = in ? r - ql * p.group : 0;
      raw[it] = make_uint4(0u, 0u, 0u, 0u);
      place[it] = make_int2(-1, 0);
      if (in) {
        place[it] = make_int2(cur.b * p.L + ql, (cur.head * lanes + lane_head) * p.group + j);
        raw[it] = __ldg(reinterpret_cast<const uint4*>(p.q + place[it].x * p.q_stride + (int64_t)place[it].y * D +
                                                       (i % kVec) * 8));
        lim[it] = cur.len - p.L + 1 + ql;
      } else {
        lim[it] = cur.len;  // rows that the tile does not have: their scores are 0 and their results nobody's
      }
    }
    seen_end = cur.len - p.L + 1 + (min(row0 + C::kRows, p.rows) - 1) / p.group;
    if constexpr (!C::kFar) {
      if (stage < 0) load_first();  // behind the run's first rows of q: one wait serves both
    }
    // The last unit's rows have been written: their places in s_row may go.  (Two buffers of s_row that take turns, without this
    // barrier, cost more: 64 x 8 rows 92.1 us for 90.6.)
    __syncthreads();
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
      if (rr < C::kRows) {
        // Lane lc's word of block b holds the columns 32 b + 8 lc ..: bytes 0, 1 are its places 2 lc, 8 + 2 lc of the
        // contraction's step 2 b, bytes 2, 3 those of step 2 b + 1.
        uint8_t* dst = s_q + rr * C::kQPitch + (c8 >> 2) * 64 + (c8 & 3) * 4;
        *reinterpret_cast<uint32_t*>(dst) = h[0];
        *reinterpret_cast<uint32_t*>(dst + 16) = h[1];
        *reinterpret_cast<uint32_t*>(dst + 32) = h[2];
        *reinterpret_cast<uint32_t*>(dst + 48) = h[3];
        if (c8 == 0) {
          s_row[rr] = place[it];
#pragma unroll
          for (int w = 0; w < kWarps; ++w) s_fr[w * C::kRows + rr].x = factor;
          s_lim[rr] = lim[it];
        }
      }
    }
    __syncthreads();
    if constexpr (C::kQRegs) {
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int b = 0; b < kBlk; ++b) q_frag(a, b, qb[a][b]);
    }
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      l.set(a, make_float2(0.f, 0.f));
#pragma unroll
      for (int n = 0; n < kPairs; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[a][n][e] = 0.f;
    }
    for (int i = lane; i < C::kRows; i += 32) s_fr[warp * C::kRows + i].y = 0.f;
    __syncwarp();
    if (tid == 0) s_unit = make_int3(cur.b, cur.head, cur.rt);  // read again at the unit's end
    unseen = (1u << (2 * RT)) - 1u;
    open = true;
  };

  // ---- the products of q and the keys from `first` of a stage on: s[a][k][2 j + e] is row 8 a + 2 lc + e, token
  // first + 16 k + 8 j + token_at(li)
  float s[RT][kSteps][4];
  auto scores = [&](uint32_t stage_at, int first) {
    const uint32_t kb = stage_at + at_k + first * C::kRowBytes, ksb = stage_at + at_ks + first * kBlk * 4;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t kf[2][kBlk];
      float sc[2][kBlk];
      if constexpr (D == 128) {
#pragma unroll
        for (int j = 0; j < 2; ++j) ldsm4(kb + (16 * k + 8 * j) * C::kRowBytes, kf[j]);
      } else {
        uint32_t r[4];
        ldsm4(kb + 16 * k * C::kRowBytes, r);
        kf[0][0] = r[0], kf[0][1] = r[1], kf[1][0] = r[2], kf[1][1] = r[3];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = ksb + (16 * k + 8 * j) * kBlk * 4;
        if constexpr (D == 128) {
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(sc[j][0]), "=f"(sc[j][1]), "=f"(sc[j][2]), "=f"(sc[j][3])
                       : "r"(at)
                       : "memory");
        } else {
          asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(sc[j][0]), "=f"(sc[j][1]) : "r"(at) : "memory");
        }
      }
#pragma unroll
      for (int b = 0; b < kBlk; ++b) {
        const uint32_t a0[4] = {e2m1_f16<0>(kf[0][b]), e2m1_f16<0>(kf[1][b]), e2m1_f16<1>(kf[0][b]), e2m1_f16<1>(kf[1][b])};
        const uint32_t a1[4] = {e2m1_f16<2>(kf[0][b]), e2m1_f16<2>(kf[1][b]), e2m1_f16<3>(kf[0][b]), e2m1_f16<3>(kf[1][b])};
#pragma unroll
        for (int a = 0; a < RT; ++a) {
          uint32_t q[4];
          if constexpr (C::kQRegs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = qb[a][b][i];
          } else {
            q_frag(a, b, q);
          }
          float d[4];
          mma_f16_zero(d, a0, q[0], q[1]);
          mma_f16(d, a1, q[2], q[3]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (b == 0)
              s[a][k][2 * j] = d[2 * j] * sc[j][b], s[a][k][2 * j + 1] = d[2 * j + 1] * sc[j][b];
            else
              fma2(s[a][k][2 * j], s[a][k][2 * j + 1], d[2 * j], d[2 * j + 1], sc[j][b], sc[j][b]);
          }
        }
      }
    }
  };
  // to log2 units less the reference, and -inf where a row does not see the token
  auto relate = [&](int first) {
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      float2 f, r;
      asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(f.x), "=f"(r.x), "=f"(f.y), "=f"(r.y)
                   : "r"(at_fr + a * 64)
                   : "memory");
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x0 = r.x, x1 = r.y;
          fma2(x0, x1, s[a][k][2 * j], s[a][k][2 * j + 1], f.x, f.y);
          s[a][k][2 * j] = x0, s[a][k][2 * j + 1] = x1;
        }
    }
    const int tok0 = cur.t * kTile + tok_first + first;
    if (tok0 + C::kStep > cur.len - p.L + 1) {  // some row does not see all of them
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int lim = s_lim[a * 8 + 2 * lc + e] - tok0 - token_at<D>(li);
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (16 * k + 8 * j >= lim) s[a][k][2 * j + e] = -INFINITY;
        }
    }
  };
  // The rows' references follow their scores: up to kTop below the largest.
  auto move_references = [&]() {
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      float cs[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(s[a][0][e], s[a][0][2 + e]);
#pragma unroll
        for (int k = 1; k < kSteps; ++k) mx = fmaxf(mx, fmaxf(s[a][k][e], s[a][k][2 + e]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        const bool first = unseen >> (2 * a + e) & 1u;
        // by how much the reference moves: by the row's own scores alone, so that its result does not depend on other rows
        float up = first || mx > kGrow4 ? mx - kTop : 0.f;
        if (up == -INFINITY) up = 0.f;  // nothing seen yet
        else unseen &= ~(1u << (2 * a + e));
        const float c = up == 0.f || first ? 1.f : ex2(-up);  // (a row that has seen nothing has no sums to scale)
        if (li == 0) s_fr[warp * C::kRows + a * 8 + 2 * lc + e].y -= up;
        cs[e] = c;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          s[a][k][e] -= up;
          s[a][k][2 + e] -= up;
        }
#pragma unroll
        for (int n = 0; n < kPairs; ++n) {
          o[a][n][e] *= c;
          o[a][n][2 + e] *= c;
        }
      }
      const float2 t = l.get(a);
      l.set(a, make_float2(t.x * cs[0], t.y * cs[1]));
    }
    __syncwarp();
    open = __any_sync(0xFFFFFFFFu, unseen != 0);
  };

  // What the blocks of V add to o whose scales fp16 does not hold, in fp32, for each row from the tokens that it sees (whatever
  // their weight: a NaN counts).
  auto add_odd_values = [&](uint32_t stage_at, int first, uint32_t odd) {
    for (; odd; odd &= odd - 1u) {
      const int t = __ffs(odd) - 1;
      // Zeros add nothing, whatever their scale: cleared pages and heads that a model does not use hold nothing else (added one
      // by one they took 20 times as long).
      const uint32_t byte = lds8(stage_at + C::kVb + t * kBlk + (D / 8) * li / 32);
      const bool outside = byte - kVLow > kVHigh - kVLow;
      uint32_t codes = lds32(stage_at + C::kPart + v_at<D>(t, li));
      if constexpr (D == 128) codes |= lds32(stage_at + C::kPart + v_at<D>(t, li) + 4);
      if (!__any_sync(0xFFFFFFFFu, outside && (byte == 255u || (codes & 0x77777777u)))) continue;
      float pr[RT][2];
      uint32_t sees = 0;  // of this lane's rows (bit 2 a + e)
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = 0.f;
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (first + 16 * k + 8 * j == (t & ~7)) x = s[a][k][2 * j + e];
          pr[a][e] = __shfl_sync(0xFFFFFFFFu, x, 4 * place_of<D>(t & 7) + lc) * (float)(1 << kVUp);
          if (cur.t * kTile + tok_first + t < s_lim[a * 8 + 2 * lc + e]) sees |= 1u << (2 * a + e);
        }
      if (!outside) continue;
      const float sc = e8m0_float(byte, 0);  // finite but for 255, and multiplied last: a zero stays one
      auto column_pair = [&](uint32_t word, auto y, int n) {
        const float2 v = f16x2_float(e2m1_f16<decltype(y)::value>(word));
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (sees >> (2 * a + e) & 1u) {
              o[a][n][e] = fmaf(pr[a][e] * v.x, sc, o[a][n][e]);
              o[a][n][2 + e] = fmaf(pr[a][e] * v.y, sc, o[a][n][2 + e]);
            }
      };
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const uint32_t word = lds32(stage_at + C::kPart + v_at<D>(t, li) + 4 * w);
        column_pair(word, std::integral_constant<int, 0>{}, 4 * w);
        column_pair(word, std::integral_constant<int, 1>{}, 4 * w + 1);
        column_pair(word, std::integral_constant<int, 2>{}, 4 * w + 2);
        column_pair(word, std::integral_constant<int, 3>{}, 4 * w + 3);
      }
    }
  };

  // ---- o += p v; p in s
  auto values = [&](uint32_t stage_at, int first) {
    const uint32_t vb0 = stage_at + at_v0 + first * C::kRowBytes, vb1 = stage_at + at_v1 + first * C::kRowBytes;
    const uint32_t vsb = stage_at + at_vs + first * 2;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t wv[4][kW], mul[2];  // tokens at the places 2 lc, 2 lc + 1, 8 + 2 lc, 9 + 2 lc
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = (i & 1 ? vb1 : vb0) + (16 * k + 8 * (i >> 1)) * C::kRowBytes;
        if constexpr (D == 128) {
          const uint2 w = lds64(at);
          wv[i][0] = w.x, wv[i][1] = w.y;
        } else {
          wv[i][0] = lds32(at);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) mul[j] = lds32(vsb + (16 * k + 8 * j) * 2);
      uint32_t pb[RT][2];
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int j = 0; j < 2; ++j) pb[a][j] = transpose8(pack_f16(s[a][k][2 * j], s[a][k][2 * j + 1]));
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        uint32_t x[2][2];  // [place half j][even or odd columns]: a byte holds one column of the two tokens
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a = wv[2 * j][w], b = wv[2 * j + 1][w];
          x[j][0] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
          x[j][1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
        }
        auto columns = [&](auto y) {
          constexpr int Y = decltype(y)::value;
          const uint32_t v[4] = {mul_f16x2(e2m1_f16<Y>(x[0][0]), mul[0]), mul_f16x2(e2m1_f16<Y>(x[0][1]), mul[0]),
                                 mul_f16x2(e2m1_f16<Y>(x[1][0]), mul[1]), mul_f16x2(e2m1_f16<Y>(x[1][1]), mul[1])};
#pragma unroll
          for (int a = 0; a < RT; ++a) mma_f16(o[a][4 * w + Y], v, pb[a][0], pb[a][1]);
        };
        columns(std::integral_constant<int, 0>{});
        columns(std::integral_constant<int, 1>{});
        columns(std::integral_constant<int, 2>{});
        columns(std::integral_constant<int, 3>{});
      }
    }
  };

  // ---- a unit's end: the four warps' sums joined, and the rows, or this block's part of them, written
  constexpr size_t kSlot = (size_t)C::kRows * (D + 2);
  auto end_unit = [&](int64_t unit_first) {  // the first place of the unit, kCost before its first tile
    float jm[RT][2], jl[RT][2];
    float4 jo[RT][kJoinPairs];  // pairs kJoinPairs warp .. of all rows
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = e ? l.get(a).y : l.get(a).x;
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
        if (li == 0) {
          if (unseen >> (2 * a + e) & 1u) s_fr[warp * C::kRows + a * 8 + 2 * lc + e].y = INFINITY;
          s_l[warp * C::kRows + a * 8 + 2 * lc + e] = sum;
        }
      }
    // a warp joins the pairs kJoinPairs warp .., kORound of them at a time
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      float c[kWarps][2];
#pragma unroll
      for (int n = 0; n < kJoinPairs; n += C::kORound) {
        float4* buf = s_o + (a * kJoinPairs + n) / C::kORound % C::kOBuffers * (C::kOPart / 16);
        if (C::kOBuffers == 1 && n > 0) __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
#pragma unroll
          for (int i = 0; i < C::kORound; ++i) {
            const float(&x)[4] = o[a][kJoinPairs * w + n + i];
            buf[((warp * kWarps + w) * C::kORound + i) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
          }
        __syncthreads();  // (also: all have read the buffer that is written next)
        if (n == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = a * 8 + 2 * lc + e;
            float top = -s_fr[row].y;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, -s_fr[w * C::kRows + row].y);
            jm[a][e] = top;
            jl[a][e] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float mw = -s_fr[w * C::kRows + row].y;
              c[w][e] = mw == top ? 1.f : ex2(mw - top);
              jl[a][e] = fmaf(s_l[w * C::kRows + row], c[w][e], jl[a][e]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < C::kORound; ++i) {
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 y = buf[((w * kWarps + warp) * C::kORound + i) * 32 + lane];
            t.x = fmaf(y.x, c[w][0], t.x), t.y = fmaf(y.y, c[w][1], t.y);
            t.z = fmaf(y.z, c[w][0], t.z), t.w = fmaf(y.w, c[w][1], t.w);
          }
          jo[a][n + i] = t;
        }
      }
    }
    cur.b = s_unit.x, cur.head = s_unit.y, cur.rt = s_unit.z;
    const int64_t first_tile = unit_first + kCost, unit_end = first_tile + tiles_of<kTile>(cur.len);
    const int64_t t0 = s_t0, t1 = s_t1, per = s_per;
    auto write_rows = [&]() {
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int2 row = s_row[a * 8 + 2 * lc + e];
          if (row.x < 0) continue;
          const float z = jl[a][e];
          const float inv = z == 0.f ? 0.f : __fdividef(1.f / (float)(1 << kVUp), z);  // a row that sees nothing is 0
          __nv_bfloat16* dst = p.out + row.x * p.out_stride + (int64_t)row.y * D + (D / 8) * li + warp * kJoinPairs * 2;
          uint32_t w[kJoinPairs];
#pragma unroll
          for (int n = 0; n < kJoinPairs; ++n)
            w[n] = e ? pack_bf16(jo[a][n].y * inv, jo[a][n].w * inv) : pack_bf16(jo[a][n].x * inv, jo[a][n].z * inv);
          if constexpr (kJoinPairs == 2)
            *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
          else
            *reinterpret_cast<uint32_t*>(dst) = w[0];
          // (m is -inf where no score was above it: z = 0 then gives -inf, a NaN among the scores NaN)
          if (p.lse && warp == 0 && li == 0) p.lse[(int64_t)row.x * p.Hq + row.y] = (jm[a][e] + log2f(z)) * kLn2;
        }
    };
    if (first_tile >= t0 && unit_end <= t1) {  // the whole unit was this block's
      write_rows();
      return;
    }
    // A part is kept as the lanes hold it: [a * kPairs + pair][lane], then m and l of the rows.
    auto put_part = [&](float* slot) {
      float4* dst = reinterpret_cast<float4*>(slot);
#pragma unroll
      for (int a = 0; a < RT; ++a) {
#pragma unroll
        for (int n = 0; n < kJoinPairs; ++n) __stcg(dst + (a * kPairs + warp * kJoinPairs + n) * 32 + lane, jo[a][n]);
        if (warp == 0 && li == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            __stcg(slot + C::kRows * D + a * 8 + 2 * lc + e, jm[a][e]);
            __stcg(slot + C::kRows * (D + 1) + a * 8 + 2 * lc + e, jl[a][e]);
          }
        }
      }
    };
    // jo, jm, jl = the parts 0 .. n_parts - 1 joined in this order
    auto join = [&](int n_parts, auto slot_of) {
#pragma unroll
      for (int a = 0; a < RT; ++a) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          jm[a][e] = -INFINITY;
          jl[a][e] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < kJoinPairs; ++n) jo[a][n] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      // (the accumulators are free by now) kIn parts are under way at once, the last ones repeated where fewer are left
      constexpr int kIn = RT > 4 ? 2 : 4;
      for (int i0 = 0; i0 < n_parts; i0 += kIn) {
        float2 pm[kIn][RT], pl[kIn][RT];
        float4 po[kIn][RT][kJoinPairs];
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          const float* src = slot_of(min(i0 + u, n_parts - 1));
#pragma unroll
          for (int a = 0; a < RT; ++a) {
            pm[u][a] = __ldcg(reinterpret_cast<const float2*>(src + C::kRows * D + a * 8 + 2 * lc));
            pl[u][a] = __ldcg(reinterpret_cast<const float2*>(src + C::kRows * (D + 1) + a * 8 + 2 * lc));
#pragma unroll
            for (int n = 0; n < kJoinPairs; ++n)
              po[u][a][n] = __ldcg(reinterpret_cast<const float4*>(src) + (a * kPairs + warp * kJoinPairs + n) * 32 + lane);
          }
        }
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          if (i0 + u >= n_parts) break;
#pragma unroll
          for (int a = 0; a < RT; ++a) {
            float c0[2], c1[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float om = e ? pm[u][a].y : pm[u][a].x;
              const float nm = fmaxf(jm[a][e], om);
              c0[e] = jm[a][e] == nm ? 1.f : ex2(jm[a][e] - nm);
              c1[e] = om == nm ? 1.f : ex2(om - nm);
              jm[a][e] = nm;
              jl[a][e] = fmaf(e ? pl[u][a].y : pl[u][a].x, c1[e], jl[a][e] * c0[e]);
            }
#pragma unroll
            for (int n = 0; n < kJoinPairs; ++n) {
              const float4 x = po[u][a][n];
              jo[a][n].x = fmaf(x.x, c1[0], jo[a][n].x * c0[0]);
              jo[a][n].y = fmaf(x.y, c1[1], jo[a][n].y * c0[1]);
              jo[a][n].z = fmaf(x.z, c1[0], jo[a][n].z * c0[0]);
              jo[a][n].w = fmaf(x.w, c1[1], jo[a][n].w * c0[1]);
            }
          }
        }
      }
    };
    // counts this block in; true for the last of n
    auto last_of = [&](int* counter, int n) {
      __syncthreads();
      if (tid == 0) {
        __threadfence();  // after the barrier: it covers what the block's other threads have written
        s_last = atomicAdd(counter, 1) == n - 1;
        if (s_last) *counter = 0;
        __threadfence();
      }
      __syncthreads();
      return s_last != 0;
    };
    // slot 0 of a block is the unit its run begins in, slot 1 the one that it ends in
    const int b0 = (int)(first_tile / per), b1 = (int)((unit_end - 1) / per), parts = b1 - b0 + 1;
    auto block_slot = [&](int b) {
      return p.partial + (((size_t)b * lanes + lane_head) * 2 + (unit_first > b * per ? 1 : 0)) * kSlot;
    };
    put_part(block_slot(g));
    int* counter = p.counters + b0 * lanes + lane_head;
    if (parts <= kJoin) {
      if (!last_of(counter, parts)) return;
      join(parts, [&](int i) { return block_slot(b0 + i); });
    } else {
      // many parts: blocks 16 g .. 16 g + 15 are joined first, then these groups.  A group can hold the end of one
      // such unit and the beginning of the next, told apart as slots are.
      auto group_at = [&](int k) {
        return ((size_t)k * lanes + lane_head) * 2 + (unit_first > (int64_t)k * kJoin * per ? 1 : 0);
      };
      const int g0 = b0 / kJoin, g1 = b1 / kJoin, k = g / kJoin;
      const int first = max(b0, k * kJoin), n = min(b1, k * kJoin + kJoin - 1) - first + 1;
      if (!last_of(p.group_counters + group_at(k), n)) return;
      join(n, [&](int i) { return block_slot(first + i); });
      put_part(p.group_partial + group_at(k) * kSlot);
      if (!last_of(counter, g1 - g0 + 1)) return;
      join(g1 - g0 + 1, [&](int i) { return p.group_partial + group_at(g0 + i) * kSlot; });
    }
    write_rows();
  };

  // ---- the run
  while (left > 0) {
    begin_unit();
    for (;;) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();  // the warp's tokens have landed for all its lanes, and all are done with the previous ones
      {
        Loader far;
        if constexpr (C::kFar) get_loader(far);
        load_stage(stage == 0 ? C::kStages - 1 : stage - 1, C::kFar ? far : keep, std::false_type{});
        if constexpr (C::kFar) put_loader(far);
      }
      const uint32_t at = ring + stage * C::kWarpStage;
      const uint32_t odd = s_odd[warp][stage];
#pragma unroll 1
      for (int first = 0; first < kTok; first += C::kStep) {
        if (cur.t * kTile + tok_first + first >= seen_end) break;
        const uint32_t odd_here = odd >> first << first & (uint32_t)((2ull << (first + C::kStep - 1)) - 1ull);
        scores(at, first);
        relate(first);
        float top = s[0][0][0];
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s[a][k][i]);
        if (__any_sync(0xFFFFFFFFu, top > kGrow4) || open) move_references();
#pragma unroll
        for (int a = 0; a < RT; ++a) {
          float2 sum = l.get(a);
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[a][k][i] = ex2(s[a][k][i]);
            add2(sum.x, sum.y, s[a][k][0], s[a][k][1]);
            add2(sum.x, sum.y, s[a][k][2], s[a][k][3]);
          }
          l.set(a, sum);
        }
        values(at, first);
        if (odd_here) add_odd_values(at, first, odd_here);
      }
      stage = stage == C::kStages - 1 ? 0 : stage + 1;
      if (left == 1 || cur.t + 1 >= tiles_of<kTile>(cur.len)) break;
      ++cur.t;
      --left;
    }
    end_unit(s_t1 - left - cur.t - kCost);
    left -= advance(cur);
  }
  cp_async_wait<0>();
}

template <int D, int RT>
cudaError_t launch_one(const AttnParams& p, int num_sms, cudaStream_t s) {
  using C = Cfg4<D, RT>;
  auto* kernel = paged_attention_fp4_kernel<D, RT>;
  static PerDeviceOnce once;
  cudaError_t e =
      once.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(num_sms * C::kBlocks), dim3(kThreads), C::kSmem, s, p);
}

template <int D>
cudaError_t launch_rows(const AttnParams& p, int num_sms, cudaStream_t s) {
  switch (attention_fp4_tile_rows(D, p.rows)) {
    case 8: return launch_one<D, 1>(p, num_sms, s);
    case 16: return launch_one<D, 2>(p, num_sms, s);
    case 24: return launch_one<D, 3>(p, num_sms, s);
    case 32: return launch_one<D, 4>(p, num_sms, s);
  }
  if constexpr (D == 64) return launch_one<D, 6>(p, num_sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace

// Rows of a row tile: the smallest multiple of 8 that holds the rows of a kv head, up to 32, and 32 above that; but 33 to 48
// rows of heads of 64, whose accumulators take half of the registers, are one tile of 48 (64 requests: 84 us, two tiles of 32
// 96).  One tile of 64 at two blocks an SM is slower than two of 32 at three (107 us for 96, two prompts 64 for 61).
int attention_fp4_tile_rows(int head_dim, int64_t rows) {
  if (rows <= 32) return rows > 8 ? (int)((rows + 7) / 8 * 8) : 8;
  return head_dim == 64 && rows <= 48 ? 48 : 32;
}

int attention_fp4_blocks(int head_dim, int tile_rows) {
  auto of = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return tile_rows == 8    ? Cfg4<D, 1>::kBlocks
           : tile_rows == 16 ? Cfg4<D, 2>::kBlocks
           : tile_rows == 24 ? Cfg4<D, 3>::kBlocks
           : tile_rows == 32 ? Cfg4<D, 4>::kBlocks
                             : Cfg4<64, 6>::kBlocks;
  };
  return head_dim == 128 ? of(std::integral_constant<int, 128>{}) : of(std::integral_constant<int, 64>{});
}

// The largest number of heads up to 16 that divides them.
int attention_fp4_lanes(int n_kv_heads) {
  int s = n_kv_heads < 16 ? n_kv_heads : 16;
  while (n_kv_heads % s) --s;
  return s;
}

size_t attention_fp4_groups(int n_kv_heads, int blocks) {
  const int lanes = attention_fp4_lanes(n_kv_heads);
  return (size_t)(blocks / lanes / kJoin + 1) * lanes;
}

cudaError_t launch_attention_fp4(const AttnParams& p, int num_sms, cudaStream_t s) {
  return p.c.head_dim == 128 ? launch_rows<128>(p, num_sms, s) : launch_rows<64>(p, num_sms, s);
}

}  // namespace moe
