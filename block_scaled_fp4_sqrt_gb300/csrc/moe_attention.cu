// Attention of the newest L tokens of every request over its paged cache (moe_paged_attention).
//
//   s_t = scale * q . k_t  for t < limit(row),  m = max s,  p_t = exp(s_t - m),  z = sum p,  out = sum p_t v_t / z
//
// The cache is read once, so a step's few rows a key-value head (heads of the group x L) leave it memory-bound where the
// cache is bf16: three requests of up to 131,071 tokens 148 us (6.2 TB/s, 92 % of the copy rate), 64 requests x 8 rows
// 94 us (5.2 TB/s).  An MXFP8 cache is half the bytes, and then the instructions bound it (unpacking, softmax and their
// latencies at 12 to 16 warps an SM): 64 x 8 rows 98 us, 64 x 1 rows 73 us, where memory alone would take 38.  One request
// of 333 tokens takes 8.7 us, of which the join of its six parts is about half.  A prompt is bound by the products: 8191
// new tokens, 8 x 4 heads of 128, 4.4 ms (every row tile walks all key tiles: 125 TFLOP/s of what lies below the diagonal).
// Layout of the work:
//  * A unit is (request, kv head, row tile): the rows r = l * group + j of the query heads that share the kv head,
//    16 MT of them at a time.  Every unit is cut into tiles of 64 tokens; the tiles of all units, in order and with
//    kUnitCost places in front of each unit's first, are dealt to the grid in equal contiguous runs of places, computed by
//    every block from the lengths alone.  A long request is thus spread over the GPU and short ones share a block,
//    whatever the mix of lengths.
//  * A block is four warps.  For a tile each warp fetches 16 tokens (cp.async, a ring of stages), computes the
//    scores of these 16 tokens for all rows, and leaves p in shared memory; after a barrier each warp accumulates
//    a quarter of the columns over all 64 tokens.  The accumulators then take 16 MT D / 128 / 4 registers a thread
//    instead of four times that, quantised values are unpacked once a block, and a unit's end needs no exchange.
//  * The running maximum of a row moves only when a score exceeds it by more than 2^8 (a vote in the barrier that
//    publishes p): p stays below 256, which costs no precision, and accumulators are rescaled rarely.
//  * A unit that several blocks share is joined, in block order, by the last of them to arrive (a counter, zero between
//    calls); more than 16 parts in two steps, of which the first runs in many blocks at once.  The counters stand at the
//    front of the workspace, one for every block that a shared unit can begin in, whatever the call's shape: no call's
//    parts ever lie where another call counts.
//
// Products run on mma.sync, at a measured 605 TFLOP/s for the 16-bit forms (m16n8k16): 29 % (MXFP8) and 31 % (bf16) of
// its cycles at 32 rows a kv head.  The form for tensor memory was built and measured for MXFP8 caches: both products
// transposed, so that the 128-row side is the cache's (K as it lies, block-scaled, times q in two MXFP8 parts; V unpacked
// to bf16 as an MN-major operand), warps of their own for fetching and unpacking, issuing and softmax.  A 128 x 16 x 32
// product takes 80 cycles there whatever its 16 columns hold, and the roles' code together misses the instruction cache;
// 64 requests x 8 rows took 116 us against 96 us here, 64 x 1 rows 93 against 72 us (one set of inputs, repeated).
//  * bf16 cache: both products in bf16 with fp32 accumulation.  p is rounded to bf16 (8 bits, as the output is);
//    its sum is taken before that rounding.  The error against 64 bits is 0.0019 to 0.0022 of the output's rms, where the
//    output's own rounding makes 0.0017: p in more bits would be a second product.
//  * MXFP8 cache, scores: E4M3 codes become fp16 (exact, one conversion a pair) and meet q in fp16, its row scaled by
//    a power of two to a maximum in [2^14, 2^15): bf16's 8 bits are kept down to 2^-28 of the maximum.  A block's
//    E8M0 scale multiplies the fp32 product of its 32 columns.  (mma.sync on E4M3 operands runs the same fp16
//    instructions here, after conversions of both operands: 690 instead of 200 instructions a tile and warp.)
//  * MXFP8 cache, values: E4M3 codes become bf16 by moving bits (value times 2^-120) and one packed multiplication
//    by the block's scale times 2^120; a product of a code and a power of two is exact in bf16 (down to its smallest 2^-133).
#include <float.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_attention_fp4.h"

namespace moe {

namespace {

constexpr int kTile = 64;                 // tokens of a tile
constexpr int kWarpTok = kTile / kWarps;  // tokens of a tile that a warp fetches and scores
// What beginning and ending a unit costs, in tiles, when the work is dealt.  64 requests of 100 to 8000 tokens, us at a
// cost of 0 / 2 / 4 / 7: 8 rows MXFP8 145 / 107 / 105 / 114, 8 rows bf16 117 / 93 / 93 / 95; 200 requests of up to 1500
// tokens 17.8 / 13.9 / 14.6 / 16.0; long requests do not depend on it.
constexpr int kUnitCost = 3;
constexpr int kPPitch = kTile * 2 + 16;   // bytes of a row of p: eight rows fall on distinct banks
constexpr float kGrow = 8.f;              // log2 units by which a score may exceed the running maximum

// Two E4M3 codes (the low or high half of r) as an fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t r, bool high) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(high ? r >> 16 : r)));
  return h;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bytes 0 and 2 (bytes 1 and 3) of four E4M3 codes as a bf16 pair, times 2^-120: the code's exponent and mantissa
// bits at bf16's lowest exponent bits.  Subnormal codes become subnormal bf16 numbers, which the multiplication
// that follows reads as such.
// top: the largest magnitude bits met, kNanBits for a NaN code (which the moved bits would read as 480).
constexpr uint32_t kNanBits = 0x07F0u;
__device__ __forceinline__ void e4m3_bf16(uint32_t r, uint32_t& even, uint32_t& odd, uint32_t& top) {
  const uint32_t e = (r << 4) & 0x07F007F0u, o = (r >> 4) & 0x07F007F0u;
  even = ((r << 8) & 0x80008000u) | e;
  odd = (r & 0x80008000u) | o;
  top = __vimax3_u16x2(top, e, o);
}

template <int D, bool MX, int MT>
struct Cfg {
  static constexpr int kRows = 16 * MT;                      // rows of a row tile
  static constexpr int kRowBytes = MX ? D : 2 * D;           // one token of one head
  static constexpr int kScale = MX ? D / 32 : 0;             // scale bytes of a token
  static constexpr int kHalf = kTile * kRowBytes;            // K (or V) of a stage
  static constexpr int kStageBytes = 2 * kHalf + 2 * kTile * kScale;
  static constexpr int kQPitch = 2 * D + 16;
  static constexpr int kQBytes = kRows * kQPitch;
  static constexpr int kPBytes = kRows * kPPitch;
// q fragments stay in registers, or are read from shared memory for every tile where that makes room for a block more
  static constexpr bool kQRegs = MX ? MT == 2 && D == 64 : MT <= 2;
  // p may take q's place once the fragments are in registers
  static constexpr int kQPBytes = kQRegs ? (kQBytes > kPBytes ? kQBytes : kPBytes) : kQBytes + kPBytes;
  static constexpr int kStatBytes = (2 * kWarps + 2) * kRows * 4;
  // Blocks an SM holds (registers: 255 for two, 168 for three, 128 for four).  Instruction latencies bound a quantised
  // cache, so it takes as many as its row tile's fragments and accumulators leave.  64 requests, us: 128 columns, MXFP8,
  // 1 row a head 77 (three, q in registers) 73 (four); 8 rows 108 (two, q in registers) 138 (three, spilling) 97 (three, q
  // from shared memory); 64 columns, MXFP8, 8 rows 78 (two) 68 (three) 67 (four, but 200 short requests 14.7 -> 15.8), 16
  // rows 107 (two) 153 (three); bf16 of 128 columns, 8 rows 128 (two) 117 (three, with two stages left); of 64 columns,
  // 16 rows 99 (two) 88 (three).
  static constexpr int kBlocks = MX && MT == 1 ? 4 : MT == 4 && (MX || D == 128) ? 2 : 3;
  static constexpr int kBudget = (kBlocks == 2 ? 113 : kBlocks == 3 ? 75 : 56) * 1024 - kQPBytes - kStatBytes - 256;
  static constexpr int kFit = kBudget / kStageBytes;
  static constexpr int kStages = kFit < 2 ? 2 : kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kStages * kStageBytes + kQPBytes + kStatBytes + 256;
  static_assert(kStageBytes % kRowBytes == 0 && 256 % kRowBytes == 0, "the loader flips address bits inside a row");
};

template <int D, bool MX, int MT>
__global__ void __launch_bounds__(kThreads, Cfg<D, MX, MT>::kBlocks) paged_attention_kernel(const AttnParams p) {
  using C = Cfg<D, MX, MT>;
  constexpr int kChunks = C::kRowBytes / 16;   // 16-byte pieces of a token row: 16, 8 or 4
  constexpr int kQ = D / 16;                   // steps of the scores' contraction
  constexpr int kCols = D / kWarps;            // output columns of a warp: 32 or 16
  constexpr int kNT = kCols / 8;               // 8-column tiles of a warp
  extern __shared__ uint8_t smem_raw[];
  // (pointer arithmetic on the array keeps the accesses below shared-memory ones)
  uint8_t* smem = smem_raw + ((256u - (smem_addr(smem_raw) & 255u)) & 255u);
  uint8_t* s_q = smem + C::kStages * C::kStageBytes;          // q, bf16 or (MXFP8) fp16
  uint8_t* s_p = C::kQRegs ? s_q : s_q + C::kQBytes;          // p of the current tile
  float* s_mx = reinterpret_cast<float*>(s_q + C::kQPBytes);  // [warp][row]
  float* s_l = s_mx + kWarps * C::kRows;                      // [warp][row]
  float* s_f = s_l + kWarps * C::kRows;                       // [row] score factor
  int* s_lim = reinterpret_cast<int*>(s_f + C::kRows);        // [row] first position the row does not see
  __shared__ int s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int li = lane >> 2, lc = lane & 3;
  const int mrow = lane & 7, mi = lane >> 3;  // this lane's row address in an ldmatrix of four 8 x 16-byte tiles
  pdl_trigger();
  pdl_wait();

  Run run;
  if (!deal_run<kTile, kUnitCost>(p, p.c.n_kv_heads, gridDim.x, blockIdx.x, tid, run)) return;
  Cursor cur = run.cur;
  const int64_t t0 = run.t0, t1 = run.t1, per = run.per;
  int64_t pos = run.pos;  // place of the tile cur

  // ---- loading: a warp fetches 16 tokens of a tile
  const uint32_t smem_base = smem_addr(smem);
  const int tok_first = warp * kWarpTok;
  auto swz = [](int row, int chunk) {
    return (kChunks >= 8 ? (chunk ^ (row & 7)) : (chunk ^ ((row >> 1) & 3))) * 16;
  };
  // Lane t < 16 knows where its token t of the tile that will be loaded next lies (looked up one tile ahead, so that the
  // table's latency is not in front of the loads); kChunks lanes then fetch a token's row together, taking the place
  // from that lane as a 32-bit count of 16-byte (MXFP8: 16-column) units.  (Two lanes a token, with no exchange, halve
  // the instructions but spread each over 16 rows: 172 instead of 144 us for three long bf16 requests.)
  constexpr int kPerIter = 32 / kChunks;  // tokens a warp instruction covers
  const uint32_t ld_dst = smem_base + (tok_first + lane / kChunks) * C::kRowBytes + swz(lane / kChunks, lane % kChunks);
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
  static_assert(!(MX && D == 64) || C::kStages >= 3,
                "a late scale must be stored, and a barrier passed, before its tile is read");
  auto load_stage = [&](int stage) {
    if constexpr (MX && D == 64) {
      if (late_dst) asm volatile("st.shared.u16 [%0], %1;" ::"r"(late_dst), "h"(late_val) : "memory");
      late_dst = 0;
    }
    if (ld_pos < t1) {
      constexpr int kUnit = MX ? 16 : 8;  // columns of a unit; every stride is a multiple of it
      const uint32_t off = nxt_page >= 0 ? (uint32_t)nxt_page * p.page_units + (uint32_t)nxt_row * p.row_units +
                                               (uint32_t)ld.head * p.head_units
                                         : kNoRow;
      const uint32_t dst0 = ld_dst + stage * C::kStageBytes;
      static_assert(kUnit * (MX ? 1 : 2) == 16, "a unit is 16 bytes");
#pragma unroll
      for (int i = 0; i < kWarpTok; i += kPerIter) {
        const uint32_t o = __shfl_sync(0xFFFFFFFFu, off, i + lane / kChunks);
        const bool ok = o != kNoRow;
        const int64_t byte = ok ? (int64_t)o * 16 : (int64_t)0;
        // row i + lane / kChunks: the swizzle of row i comes on top of the lane's own
        const uint32_t dst = (dst0 ^ swz(i, 0)) + i * C::kRowBytes;
        cp_async16(dst, k_src + byte, ok);
        cp_async16(dst + C::kHalf, v_src + byte, ok);
      }
      if constexpr (MX) {  // lane t: K scales, lane 16 + t: V scales
        const int tk = lane % kWarpTok;
        const uint32_t o = __shfl_sync(0xFFFFFFFFu, off, tk);
        const bool ok = o != kNoRow, v = lane >= kWarpTok;
        const uint32_t dst = smem_base + stage * C::kStageBytes + 2 * C::kHalf + (v ? kTile * C::kScale : 0) +
                             (tok_first + tk) * C::kScale;
        const uint8_t* src = (v ? p.c.v_s : p.c.k_s) + (ok ? o >> 1 : 0u);  // two units a scale byte
        if constexpr (D == 128) {
          cp_async4(dst, src, ok);
        } else {  // two bytes, less than cp.async copies: through a register, stored one tile later
          late_val = ok ? __ldg(reinterpret_cast<const uint16_t*>(src)) : (uint16_t)0;
          late_dst = dst;
        }
      }
      ld_pos += advance_tile<kTile, kUnitCost>(p, p.c.n_kv_heads, ld);
      lookup();
    }
    cp_async_commit();
  };
  lookup();
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) load_stage(s);

  // ---- per-unit state
  uint32_t qa[C::kQRegs ? MT : 1][C::kQRegs ? kQ : 1][4];
  float o[MT][kNT][4];
  float m[MT][2], l[MT][2], f[MT][2];  // running maximum (log2 units), this thread's sum, score factor

  const uint32_t q_base = smem_addr(s_q), p_base = smem_addr(s_p);
  // A fragment of rows 16 a.., step k of the contraction
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
      const int i = it * kThreads + tid, rr = i / kVec, col = (i % kVec) * 8;
      float factor = p.scale_log2;
      if constexpr (!MX) {
        *reinterpret_cast<uint4*>(s_q + rr * C::kQPitch + col * 2) = raw[it];
      } else {
        uint32_t top = __vmaxu2(__vmaxu2(raw[it].x & 0x7FFF7FFFu, raw[it].y & 0x7FFF7FFFu),
                                __vmaxu2(raw[it].z & 0x7FFF7FFFu, raw[it].w & 0x7FFF7FFFu));
        top = max(top & 0xFFFFu, top >> 16);  // largest magnitude, as bf16 bits
#pragma unroll
        for (int x = 1; x < kVec; x <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
        // 2^up brings the row's maximum to [2^14, 2^15); rows below 2^-112 stay below it (their scores vanish in fp32)
        const int be = (int)(top >> 7);
        const int up = be ? min(141 - be, 126) : 126;
        const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
        factor = be == 255 ? __uint_as_float(0x7FC00000u) : p.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
        float v[8];
        bf16x8_to_f32(raw[it], v);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 h2 = __floats2half2_rn(v[2 * e] * mul, v[2 * e + 1] * mul);
          h[e] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        // A lane of the scores' B fragment holds columns 4 c .. 4 c + 3 of a 16-column chunk of K, one word.  So
        // columns 4 c, 4 c + 1 take the places 2 c, 2 c + 1 of the contraction and 4 c + 2, 4 c + 3 the places 8 later.
        uint8_t* dst = s_q + rr * C::kQPitch + (col & ~15) * 2 + (col & 8);
        *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[2]);
        *reinterpret_cast<uint2*>(dst + 16) = make_uint2(h[1], h[3]);
      }
      if (col == 0) {
        s_f[rr] = factor;
        s_lim[rr] = lim[it];
      }
    }
    __syncthreads();
    if constexpr (C::kQRegs) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int k = 0; k < kQ; ++k) q_frag(a, k, qa[a][k]);
    }
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

  // ---- the scores of this warp's 16 tokens, in log2 units less the running maximum (or 0), and their masks
  float s[MT][2][4];
  auto scores = [&](int stage) {
    const uint32_t kb = smem_base + stage * C::kStageBytes + tok_first * C::kRowBytes;
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[a][n][e] = 0.f;
    const int row = (mi >> 1) * 8 + mrow;
    uint32_t kw[2][2];  // MXFP8: scale words of this thread's score columns
    if constexpr (MX) {
      const uint32_t sb = smem_base + stage * C::kStageBytes + 2 * C::kHalf + tok_first * C::kScale;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t at = sb + (n * 8 + 2 * lc) * C::kScale;
        if constexpr (D == 128) {
          asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(kw[n][0]), "=r"(kw[n][1]) : "r"(at));
        } else {
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(kw[n][0]) : "r"(at));
          kw[n][1] = kw[n][0] >> 16;
        }
      }
    }
    auto q_step = [&](int a, int k, uint32_t (&r)[4]) {
      if constexpr (C::kQRegs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = qa[a][k][i];
      } else {
        q_frag(a, k, r);
      }
    };
    if constexpr (!MX) {
#pragma unroll
      for (int k = 0; k < kQ; ++k) {
        uint32_t kf[4];
        ldsm4(kb + row * C::kRowBytes + swz(row, 2 * k + (mi & 1)), kf);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          uint32_t q[4];
          q_step(a, k, q);
          mma_bf16(s[a][0], q, kf[0], kf[1]);
          mma_bf16(s[a][1], q, kf[2], kf[3]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < kQ; k += 2) {  // one MX block
        uint32_t kf[4];  // tokens 0..7: chunks k, k + 1; tokens 8..15: chunks k, k + 1
        ldsm4(kb + row * C::kRowBytes + swz(row, k + (mi & 1)), kf);
        uint32_t b[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b[i][0] = e4m3_f16(kf[i], false);
          b[i][1] = e4m3_f16(kf[i], true);
        }
        float k0[2], k1[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          k0[n] = e8m0_float(kw[n][0], k / 2);
          k1[n] = e8m0_float(kw[n][1], k / 2);
        }
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          uint32_t q0[4], q1[4];
          q_step(a, k, q0);
          q_step(a, k + 1, q1);
          float d[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) mma_f16_zero(d[n], q0, b[2 * n][0], b[2 * n][1]);
#pragma unroll
          for (int n = 0; n < 2; ++n) mma_f16(d[n], q1, b[2 * n + 1][0], b[2 * n + 1][1]);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            fma2(s[a][n][0], s[a][n][1], d[n][0], d[n][1], k0[n], k1[n]);
            fma2(s[a][n][2], s[a][n][3], d[n][2], d[n][3], k0[n], k1[n]);
          }
        }
      }
    }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = m[a][h] == -INFINITY ? 0.f : m[a][h];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) s[a][n][2 * h + e] = fmaf(s[a][n][2 * h + e], f[a][h], -ref);
      }
    const int tok0 = cur.t * kTile + tok_first;
    if (tok0 + kWarpTok > cur.len - p.L + 1) {  // some row does not see all of them
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int lim = s_lim[a * 16 + li + 8 * h] - tok0 - 2 * lc;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (n * 8 + e >= lim) s[a][n][2 * h + e] = -INFINITY;
        }
    }
  };

  // p of this warp's tokens to shared memory; returns this thread's sums
  auto put_p = [&](float (&sum)[MT][2]) {
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = ex2(s[a][i >> 1][2 * h + (i & 1)]);
        sum[a][h] = (e[0] + e[1]) + (e[2] + e[3]);
        const uint32_t at = p_base + (a * 16 + li + 8 * h) * kPPitch + (tok_first + 2 * lc) * 2;
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(pack_bf16(e[0], e[1])) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 16), "r"(pack_bf16(e[2], e[3])) : "memory");
      }
  };

  // ---- o += p v over the tile's 64 tokens, this warp's columns
  auto p_frag = [&](int a, int ks, uint32_t (&r)[4]) {
    ldsm4(p_base + (a * 16 + (mi & 1) * 8 + mrow) * kPPitch + ks * 32 + (mi >> 1) * 16, r);
  };
  auto values_bf16 = [&](uint32_t vb) {
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks) {
      uint32_t vf[kNT / 2][4];
      const int row = ks * 16 + (mi & 1) * 8 + mrow;
#pragma unroll
      for (int n = 0; n < kNT; n += 2)
        ldsm4_trans(vb + row * C::kRowBytes + swz(row, warp * kNT + n + (mi >> 1)), vf[n / 2]);
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        uint32_t pa[4];
        p_frag(a, ks, pa);
#pragma unroll
        for (int n = 0; n < kNT; n += 2) {
          mma_bf16(o[a][n], pa, vf[n / 2][0], vf[n / 2][1]);
          mma_bf16(o[a][n + 1], pa, vf[n / 2][2], vf[n / 2][3]);
        }
      }
    }
  };
  // column of o[.][n][2 h + y] inside the warp's columns
  auto col_of = [&](int n, int y) { return MX ? (n / 2) * 16 + 4 * lc + (n & 1) + 2 * y : n * 8 + 2 * lc + y; };

  // MXFP8.  A warp's columns lie in one block of 32, so a token has one scale here.  pair[ks][i]: scale bytes of
  // tokens 16 ks + 8 i + 2 lc and the next, in 16-bit halves: what a B fragment register holds.
  // A scale above 2^7 does not fit the one multiplier 2^(byte - 127 + 120): LARGE adds a second one.
  auto values_mx = [&](uint32_t vb, const uint32_t (&pair)[kTile / 16][2], auto large) {
    constexpr bool LARGE = decltype(large)::value;
    constexpr int kZ = kCols / 16;  // 16-byte chunks of a warp's columns
    uint32_t top = 0;
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks) {
      uint32_t vf[4];
      if constexpr (kZ == 2) {
        const int row = ks * 16 + (mi & 1) * 8 + mrow;
        ldsm4_trans(vb + row * C::kRowBytes + swz(row, warp * 2 + (mi >> 1)), vf);
      } else {  // one chunk: the four 8-row tiles are the tokens of two steps; the step picks its half
        const int row = (ks & ~1) * 16 + mi * 8 + mrow;
        uint32_t both[4];
        ldsm4_trans(vb + row * C::kRowBytes + swz(row, warp), both);
        vf[0] = both[2 * (ks & 1)];
        vf[1] = both[2 * (ks & 1) + 1];
      }
      uint32_t mul[2], rest[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t b = pair[ks][i];
        if constexpr (LARGE) {
          const uint32_t cut = __vminu2(b, 0x00860086u);
          rest[i] = 0x3F803F80u + ((b - cut) << 7);
          b = cut;
        }
        mul[i] = b * 128u + 0x3C003C00u;
      }
      uint32_t bf[kZ][2][2];
#pragma unroll
      for (int z = 0; z < kZ; ++z)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          e4m3_bf16(vf[2 * z + i], bf[z][0][i], bf[z][1][i], top);
          bf[z][0][i] = mul_bf16x2(bf[z][0][i], mul[i]);
          bf[z][1][i] = mul_bf16x2(bf[z][1][i], mul[i]);
          if constexpr (LARGE) {
            bf[z][0][i] = mul_bf16x2(bf[z][0][i], rest[i]);
            bf[z][1][i] = mul_bf16x2(bf[z][1][i], rest[i]);
          }
        }
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        uint32_t pa[4];
        p_frag(a, ks, pa);
#pragma unroll
        for (int z = 0; z < kZ; ++z) {
          mma_bf16(o[a][2 * z], pa, bf[z][0][0], bf[z][0][1]);      // columns 16 z + 0, 2, 4 ..
          mma_bf16(o[a][2 * z + 1], pa, bf[z][1][0], bf[z][1][1]);  // .. and 1, 3, 5 ..
        }
      }
    }
    if (__any_sync(0xFFFFFFFFu, (top & 0xFFFFu) == kNanBits || (top >> 16) == kNanBits)) {
      // a NaN among the values, and every row sees the tile's tokens: its column becomes NaN
      for (int tk = 0; tk < kTile; ++tk)
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int col = warp * kCols + col_of(n, y);
            uint32_t code;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(code) : "r"(vb + tk * C::kRowBytes + swz(tk, col / 16) + col % 16));
            if ((code & 0x7Fu) == 0x7Fu) {
#pragma unroll
              for (int a = 0; a < MT; ++a) o[a][n][y] = o[a][n][2 + y] = __uint_as_float(0x7FC00000u);
            }
          }
    }
  };
  // Token by token, leaving out for each row the tokens that it does not see (not those with p = 0: a NaN or an infinity
  // that a row sees counts whatever its weight, as in the products).
  auto values_one_by_one = [&](uint32_t vb, uint32_t sb) {
    int lim[MT][2];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) lim[a][h] = s_lim[a * 16 + li + 8 * h] - cur.t * kTile;
    for (int tk = 0; tk < kTile; ++tk) {
      float v[kNT][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int col = warp * kCols + col_of(n, y);
          const int byte = MX ? col : 2 * col;
          const uint32_t at = vb + tk * C::kRowBytes + swz(tk, byte / 16) + byte % 16;
          if constexpr (MX) {
            uint16_t code;
            uint32_t h2, e;
            asm volatile("ld.shared.u8 %0, [%1];" : "=h"(code) : "r"(at));
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e) : "r"(sb + tk * C::kScale + col / 32));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(code));
            v[n][y] = __low2float(*reinterpret_cast<const __half2*>(&h2)) * e8m0_float(e, 0);
          } else {
            uint16_t bits;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(at));
            v[n][y] = __uint_as_float((uint32_t)bits << 16);
          }
        }
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (tk >= lim[a][h]) continue;
          uint16_t bits;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(p_base + (a * 16 + li + 8 * h) * kPPitch + tk * 2));
          const float pr = __uint_as_float((uint32_t)bits << 16);
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) o[a][n][2 * h + y] = fmaf(pr, v[n][y], o[a][n][2 * h + y]);
        }
    }
  };

  auto values = [&](int stage) {
    const uint32_t vb = smem_base + stage * C::kStageBytes + C::kHalf;
    const uint32_t sb = vb + C::kHalf + kTile * C::kScale;
    // Tokens that some rows see and others do not (the step's own new tokens): p = 0 must keep a NaN or an
    // infinity out, which a matrix product would let through.  Rare, so it is looked for only in such tiles.
    if (p.L > 1 && (cur.t + 1) * kTile > cur.len - p.L + 1) {
      bool odd = false;
      for (int i = lane; i < kTile * kCols * (MX ? 1 : 2) / 16; i += 32) {
        constexpr int kPer = kCols * (MX ? 1 : 2) / 16;
        const int row = i / kPer;
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(vb + row * C::kRowBytes + swz(row, warp * kPer + i % kPer)));
#pragma unroll
        for (int z = 0; z < 4; ++z)
          odd |= MX ? (((w[z] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u
                    : __vcmpeq2(w[z] & 0x7F807F80u, 0x7F807F80u) != 0u;
      }
      if constexpr (MX) {  // a scale at which 448 times it leaves bf16's range
        for (int tk = lane; tk < kTile; tk += 32) {
          uint32_t e;
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e) : "r"(sb + tk * C::kScale + warp * kCols / 32));
          odd |= e > 246u;
        }
      }
      if (__any_sync(0xFFFFFFFFu, odd)) {
        values_one_by_one(vb, sb);
        return;
      }
    }
    if constexpr (!MX) {
      values_bf16(vb);
    } else {
      uint32_t pair[kTile / 16][2], top = 0;
      const int blk = warp * kCols / 32;
#pragma unroll
      for (int ks = 0; ks < kTile / 16; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t at = sb + (ks * 16 + 8 * i + 2 * lc) * C::kScale;
          uint32_t w0, w1;
          if constexpr (D == 128) {
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(at));
            w0 = __byte_perm(w0, w1, 0x0400u + 0x0101u * (uint32_t)blk) & 0x00FF00FFu;
          } else {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w0) : "r"(at));
            w0 = (w0 >> (8 * blk)) & 0x00FF00FFu;
          }
          pair[ks][i] = w0;
          top = __vmaxu2(top, w0);
        }
      if (__any_sync(0xFFFFFFFFu, __vmaxu2(top, 0x00860086u) != 0x00860086u))
        values_mx(vb, pair, std::true_type{});
      else
        values_mx(vb, pair, std::false_type{});
    }
  };

  // ---- a unit's end: write the rows, or this block's part of them
  constexpr size_t kSlot = (size_t)C::kRows * (D + 2);
  auto end_unit = [&](int64_t unit_first) {  // the first place of the unit, kUnitCost before its first tile
    const int row0 = cur.rt * C::kRows;
    const int nrows = min(C::kRows, p.rows - row0);
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[a][h] += __shfl_xor_sync(0xFFFFFFFFu, l[a][h], 1);
        l[a][h] += __shfl_xor_sync(0xFFFFFFFFu, l[a][h], 2);
        if (lc == 0) s_l[warp * C::kRows + a * 16 + li + 8 * h] = l[a][h];
      }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = a * 16 + li + 8 * h;
        l[a][h] = (s_l[r] + s_l[C::kRows + r]) + (s_l[2 * C::kRows + r] + s_l[3 * C::kRows + r]);
      }
    const int64_t first_tile = unit_first + kUnitCost, unit_end = first_tile + cur.nt;
    // this thread's rows of the final result: o / l and the logarithm of the sum
    auto write_rows = [&]() {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = a * 16 + li + 8 * h;
          if (r >= nrows) continue;
          const int ql = (row0 + r) / p.group, j = row0 + r - ql * p.group;
          const float z = l[a][h];
          const float inv = z == 0.f ? 0.f : 1.f / z;  // a row that sees nothing is 0; a NaN sum stays NaN
          const int64_t token = (int64_t)cur.b * p.L + ql;
          const int head = cur.head * p.group + j;
          __nv_bfloat16* dst = p.out + token * p.out_stride + (int64_t)head * D + warp * kCols;
          if constexpr (MX) {
#pragma unroll
            for (int n = 0; n < kNT; n += 2)
              *reinterpret_cast<uint2*>(dst + n * 8 + 4 * lc) =
                  make_uint2(pack_bf16(o[a][n][2 * h] * inv, o[a][n + 1][2 * h] * inv),
                             pack_bf16(o[a][n][2 * h + 1] * inv, o[a][n + 1][2 * h + 1] * inv));
          } else {
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              *reinterpret_cast<uint32_t*>(dst + n * 8 + 2 * lc) =
                  pack_bf16(o[a][n][2 * h] * inv, o[a][n][2 * h + 1] * inv);
          }
          // (m is -inf where no score was above it: z = 0 then gives -inf, a NaN among the scores NaN)
          if (p.lse && warp == 0 && lc == 0) p.lse[token * p.Hq + head] = (m[a][h] + log2f(z)) * kLn2;
        }
    };
    if (first_tile >= t0 && unit_end <= t1) {  // the whole unit was this block's
      write_rows();
      return;
    }
    auto put_part = [&](float* slot) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = a * 16 + li + 8 * h;
          if (r >= nrows) continue;
          float* dst = slot + r * D + warp * kCols;
          if constexpr (MX) {
#pragma unroll
            for (int n = 0; n < kNT; n += 2)
              __stcg(reinterpret_cast<float4*>(dst + n * 8 + 4 * lc),
                     make_float4(o[a][n][2 * h], o[a][n + 1][2 * h], o[a][n][2 * h + 1], o[a][n + 1][2 * h + 1]));
          } else {
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              __stcg(reinterpret_cast<float2*>(dst + n * 8 + 2 * lc), make_float2(o[a][n][2 * h], o[a][n][2 * h + 1]));
          }
          if (warp == 0 && lc == 0) {
            __stcg(slot + C::kRows * D + r, m[a][h]);
            __stcg(slot + C::kRows * (D + 1) + r, l[a][h]);
          }
        }
    };
    // o, m, l = the parts 0 .. n_parts - 1 joined in this order
    auto join = [&](int n_parts, auto slot_of) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m[a][h] = -INFINITY;
          l[a][h] = 0.f;
#pragma unroll
          for (int n = 0; n < kNT; ++n) o[a][n][2 * h] = o[a][n][2 * h + 1] = 0.f;
        }
      // kIn parts are under way at once, the last ones repeated where fewer are left
      constexpr int kIn = 2;
      for (int i0 = 0; i0 < n_parts; i0 += kIn) {
        float pm[kIn][MT][2], pl[kIn][MT][2], po[kIn][MT][2][2 * kNT];
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          const float* src = slot_of(min(i0 + u, n_parts - 1));
#pragma unroll
          for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = min(a * 16 + li + 8 * h, nrows - 1);  // idle rows repeat the last one's loads
              pm[u][a][h] = __ldcg(src + C::kRows * D + r);
              pl[u][a][h] = __ldcg(src + C::kRows * (D + 1) + r);
              const float* row = src + r * D + warp * kCols;
              float(&o1)[2 * kNT] = po[u][a][h];
              if constexpr (MX) {
#pragma unroll
                for (int n = 0; n < kNT; n += 2) {
                  const float4 x = __ldcg(reinterpret_cast<const float4*>(row + n * 8 + 4 * lc));
                  o1[2 * n] = x.x, o1[2 * n + 2] = x.y, o1[2 * n + 1] = x.z, o1[2 * n + 3] = x.w;
                }
              } else {
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                  const float2 x = __ldcg(reinterpret_cast<const float2*>(row + n * 8 + 2 * lc));
                  o1[2 * n] = x.x, o1[2 * n + 1] = x.y;
                }
              }
            }
        }
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
          if (i0 + u >= n_parts) break;
#pragma unroll
          for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float nm = fmaxf(m[a][h], pm[u][a][h]);
              const float c0 = m[a][h] == nm ? 1.f : ex2(m[a][h] - nm);
              const float c1 = pm[u][a][h] == nm ? 1.f : ex2(pm[u][a][h] - nm);
              m[a][h] = nm;
              l[a][h] = fmaf(pl[u][a][h], c1, l[a][h] * c0);
#pragma unroll
              for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  o[a][n][2 * h + y] = fmaf(po[u][a][h][2 * n + y], c1, o[a][n][2 * h + y] * c0);
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
    auto block_slot = [&](int b) {
      return p.partial + ((size_t)b * 2 + (unit_first > b * per ? 1 : 0)) * kSlot;
    };
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
    __syncthreads();  // the tile has landed for all warps, and all are done with the previous one
    load_stage(stage == 0 ? C::kStages - 1 : stage - 1);
    scores(stage);
    bool grow = false;
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        grow |= fmaxf(fmaxf(s[a][0][2 * h], s[a][0][2 * h + 1]), fmaxf(s[a][1][2 * h], s[a][1][2 * h + 1])) >
                (m[a][h] == -INFINITY ? -INFINITY : kGrow);
    float add[MT][2];
    put_p(add);
    if (__syncthreads_or(grow)) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = fmaxf(fmaxf(s[a][0][2 * h], s[a][0][2 * h + 1]), fmaxf(s[a][1][2 * h], s[a][1][2 * h + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
          if (lc == 0) s_mx[warp * C::kRows + a * 16 + li + 8 * h] = mx;
        }
      __syncthreads();
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = a * 16 + li + 8 * h;
          // by how much the maximum grows (from 0 where there was none)
          const float up = fmaxf(fmaxf(s_mx[r], s_mx[C::kRows + r]), fmaxf(s_mx[2 * C::kRows + r], s_mx[3 * C::kRows + r]));
          const float old = m[a][h], ref = old == -INFINITY ? 0.f : old;
          const float nm = fmaxf(up + ref, old);
          const float c = old == nm ? 1.f : ex2(old - nm);
          const float less = nm == -INFINITY ? 0.f : nm - ref;
          m[a][h] = nm;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[a][n][2 * h + e] -= less;
          l[a][h] *= c;
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            o[a][n][2 * h] *= c;
            o[a][n][2 * h + 1] *= c;
          }
        }
      put_p(add);
      __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) l[a][h] += add[a][h];
    values(stage);
    stage = stage == C::kStages - 1 ? 0 : stage + 1;
    if (cur.t + 1 == cur.nt || pos + 1 == t1) {
      __syncthreads();  // p is no longer read: its place may take the next unit's q
      end_unit(pos - cur.t - kUnitCost);
      fresh = true;
    }
    pos += advance_tile<kTile, kUnitCost>(p, p.c.n_kv_heads, cur);
  }
  cp_async_wait<0>();
}

template <int D, bool MX, int MT>
cudaError_t launch_one(const AttnParams& p, int num_sms, cudaStream_t s) {
  using C = Cfg<D, MX, MT>;
  auto* kernel = paged_attention_kernel<D, MX, MT>;
  static PerDeviceOnce once;
  cudaError_t e =
      once.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(num_sms * C::kBlocks), dim3(kThreads), C::kSmem, s, p);
}

// Rows of a row tile: the smallest of 16, 32 and 64 that holds the rows of a kv head, 64 above that.
int tile_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int D, bool MX>
cudaError_t launch_rows(const AttnParams& p, int num_sms, cudaStream_t s) {
  switch (tile_rows(p.rows)) {
    case 16: return launch_one<D, MX, 1>(p, num_sms, s);
    case 32: return launch_one<D, MX, 2>(p, num_sms, s);
    default: return launch_one<D, MX, 4>(p, num_sms, s);
  }
}

// Blocks of the grid for row tiles of tr rows.
int grid_blocks(const moe_kv_cache_t& c, int tr, int num_sms) {
  if (c.format == MOE_KV_MXFP4) return num_sms * attention_fp4_blocks(c.head_dim, tr);
  auto of = [&](auto mx, auto d) {
    constexpr bool MX = decltype(mx)::value;
    constexpr int D = decltype(d)::value;
    return tr == 16 ? Cfg<D, MX, 1>::kBlocks : tr == 32 ? Cfg<D, MX, 2>::kBlocks : Cfg<D, MX, 4>::kBlocks;
  };
  const std::integral_constant<int, 64> d64;
  const std::integral_constant<int, 128> d128;
  const bool mx = c.format == MOE_KV_MXFP8;
  return num_sms * (c.head_dim == 128 ? (mx ? of(std::true_type{}, d128) : of(std::false_type{}, d128))
                                      : (mx ? of(std::true_type{}, d64) : of(std::false_type{}, d64)));
}

struct Sizes {
  int64_t rows;
  int row_tiles;
  size_t blocks, groups, slot, bytes;
};

moe_status_t plan(const moe_kv_cache_t& c, int n_q_heads, int L, int num_sms, const char* call, Sizes* z) {
  if (n_q_heads < 1 || n_q_heads % c.n_kv_heads)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", call,
                       n_q_heads, c.n_kv_heads);
  if (L < 0) return decode_fail(MOE_ERR_INVALID_ARG, "%s: L = %d is negative", call, L);
  z->rows = (int64_t)(n_q_heads / c.n_kv_heads) * L;
  if (z->rows > (1 << 20) || (int64_t)n_q_heads * c.head_dim > (1ll << 31))
    return decode_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^20 rows a kv head", call);
  const int tr = c.format == MOE_KV_MXFP4 ? attention_fp4_tile_rows(c.head_dim, z->rows) : tile_rows(z->rows);
  z->row_tiles = (int)((z->rows + tr - 1) / tr);
  const int64_t units = (int64_t)c.n_seqs * c.n_kv_heads * z->row_tiles;
  if (units > (1ll << 30)) return decode_fail(MOE_ERR_UNSUPPORTED, "%s: too many row tiles", call);
  z->blocks = grid_blocks(c, tr, num_sms);
  z->groups = c.format == MOE_KV_MXFP4 ? attention_fp4_groups(c.n_kv_heads, (int)z->blocks) : z->blocks / kJoin + 1;
  if ((z->blocks + 2 * z->groups) * 4 > MOE_ATTENTION_COUNTER_BYTES)
    return decode_fail(MOE_ERR_UNSUPPORTED, "%s: %d SMs", call, num_sms);
  z->slot = (size_t)tr * (c.head_dim + 2) * 4;
  z->bytes = MOE_ATTENTION_COUNTER_BYTES + 2 * (z->blocks + z->groups) * z->slot;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_paged_attention_workspace(const moe_kv_cache_t* cache, int32_t n_q_heads, int32_t L) {
  int sms = 0;
  Sizes z{};
  if (check_cache(cache, "moe_paged_attention_workspace") != MOE_OK || check_device(&sms) != MOE_OK ||
      plan(*cache, n_q_heads, L, sms, "moe_paged_attention_workspace", &z) != MOE_OK)
    return 0;
  return z.bytes;
}

extern "C" moe_status_t moe_paged_attention(const moe_kv_cache_t* cache, const moe_attention_t* a,
                                            moe_stream_t stream) {
  moe_status_t st = check_cache(cache, "moe_paged_attention");
  if (st != MOE_OK) return st;
  if (!a) return decode_fail(MOE_ERR_INVALID_ARG, "moe_paged_attention: args is NULL");
  const moe_kv_cache_t& c = *cache;
  Sizes z{};
  st = plan(c, a->n_q_heads, a->L, 1, "moe_paged_attention", &z);
  if (st != MOE_OK) return st;
  // rows are addressed by 32-bit counts of 16-byte units
  const __int128 last = (__int128)(c.n_pages > 0 ? c.n_pages - 1 : 0) * c.page_stride +
                        (__int128)(c.page_size - 1) * c.row_stride + (__int128)(c.n_kv_heads - 1) * c.head_stride;
  const int64_t unit = c.format == MOE_KV_BF16 ? 8 : c.format == MOE_KV_MXFP8 ? 16 : 32;
  if (last / unit >= 0xFFFFFFFFll)
    return decode_fail(MOE_ERR_UNSUPPORTED, "moe_paged_attention: k or v spans 64 GB or more");
  if (!std::isfinite(a->scale)) return decode_fail(MOE_ERR_INVALID_ARG, "moe_paged_attention: scale is not finite");
  const int64_t width = (int64_t)a->n_q_heads * c.head_dim;
  const int64_t qs = a->q_stride ? a->q_stride : width, os = a->out_stride ? a->out_stride : width;
  if (qs < width || os < width || qs % 8 || os % 8)
    return decode_fail(MOE_ERR_INVALID_ARG,
                       "moe_paged_attention: row strides (%lld, %lld) must be multiples of 8, at least n_q_heads * head_dim",
                       (long long)qs, (long long)os);
  if (!aligned_to(a->q, 16) || !aligned_to(a->out, 16) || !aligned_to(a->lse, 4))
    return decode_fail(MOE_ERR_INVALID_ARG, "moe_paged_attention: q and out must be 16-byte aligned, lse 4-byte");
  if (c.n_seqs == 0 || a->L == 0) return MOE_OK;
  if (!a->q || !a->out) return decode_fail(MOE_ERR_INVALID_ARG, "moe_paged_attention: q or out is NULL");
  if (!c.seq_lens) return decode_fail(MOE_ERR_INVALID_ARG, "moe_paged_attention: seq_lens is NULL");
  int sms = 0;
  st = check_device(&sms);
  if (st == MOE_OK) st = plan(c, a->n_q_heads, a->L, sms, "moe_paged_attention", &z);
  if (st != MOE_OK) return st;
  if (!a->workspace || a->workspace_bytes < z.bytes)
    return decode_fail(MOE_ERR_WORKSPACE, "moe_paged_attention: workspace of %zu bytes, %zu needed",
                       a->workspace ? a->workspace_bytes : (size_t)0, z.bytes);
  if (!aligned_to(a->workspace, 256))
    return decode_fail(MOE_ERR_INVALID_ARG, "moe_paged_attention: workspace must be 256-byte aligned");
  AttnParams p{};
  p.c = c;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.q_stride = qs;
  p.out_stride = os;
  p.L = a->L;
  p.group = a->n_q_heads / c.n_kv_heads;
  p.rows = (int)z.rows;
  p.row_tiles = z.row_tiles;
  p.Hq = a->n_q_heads;
  p.scale_log2 = a->scale * kLog2e;
  p.pd = page_div((uint32_t)c.page_size);
  p.page_units = (uint32_t)(c.page_stride / unit);
  p.row_units = (uint32_t)(c.row_stride / unit);
  p.head_units = (uint32_t)(c.head_stride / unit);
  p.counters = static_cast<int*>(a->workspace);
  p.group_counters = p.counters + z.blocks;
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + MOE_ATTENTION_COUNTER_BYTES);
  p.group_partial = p.partial + 2 * z.blocks * (z.slot / 4);
  p.lanes = attention_fp4_lanes(c.n_kv_heads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool mx = c.format == MOE_KV_MXFP8;
  cudaError_t e = c.format == MOE_KV_MXFP4 ? launch_attention_fp4(p, sms, s)
                  : c.head_dim == 128      ? (mx ? launch_rows<128, true>(p, sms, s) : launch_rows<128, false>(p, sms, s))
                                    : (mx ? launch_rows<64, true>(p, sms, s) : launch_rows<64, false>(p, sms, s));
  if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "moe_paged_attention: %s", cudaGetErrorString(e));
  return MOE_OK;
}
