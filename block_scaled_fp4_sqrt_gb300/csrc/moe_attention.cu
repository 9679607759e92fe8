// Attention of the newest L tokens of every request over its paged cache (moe_paged_attention).
//
//   s_t = scale * q . k_t  for t < limit(row),  m = max s,  p_t = exp(s_t - m),  z = sum p,  out = sum p_t v_t / z
//
// The cache is read once, so a step's few rows a key-value head (heads of the group x L) leave it memory-bound.
// Layout of the work:
//  * A unit is (request, kv head, row tile): the rows r = l * group + j of the query heads that share the kv head,
//    16 MT WM of them at a time.  Every unit is cut into tiles of 64 tokens; the tiles of all units, in order, are
//    dealt to the grid in equal contiguous runs, computed by every block from the lengths alone.  A long request is
//    thus spread over the GPU and short ones share a block, whatever the mix of lengths.
//  * A block is 4 WM warps: each warp owns 16 of a tile's 64 tokens and (WM = 2) half of the rows.  With WM = 1 a
//    warp loads its own tokens (cp.async, a ring of stages) and no barrier of the block is in the loop.
//  * A warp keeps the running maximum and sum of its rows over its own tokens; the four token groups are joined
//    in shared memory at a unit's end, and a unit that several blocks share is joined, in block order, by the last
//    of them to arrive (a counter per unit, zero between calls).
//
// Products run on mma.sync: with at most 64 rows to a kv head a 128-row tcgen05 tile would be mostly padding, its
// accumulator would have to cross tensor memory for every softmax step, and quantised operands could not be
// unpacked in registers.  Measured rates: bf16 m16n8k16 605 TFLOP/s, E4M3 m16n8k32 2.28 PFLOP/s.
//  * bf16 cache: both products in bf16 with fp32 accumulation.  p is rounded to bf16 (8 bits, as the output is);
//    its sum is taken before that rounding.
//  * MXFP8 cache, scores: the E4M3 codes of K enter the tensor cores as they are.  q (8 significant bits) is split
//    exactly into two E4M3 terms of 4 bits each after scaling its row by a power of two (elements below 2^-9 of
//    the row's maximum lose bits: an error under 2^-17 of that maximum); a block's E8M0 scale multiplies the fp32
//    product of its 32 columns.  Two E4M3 instructions replace the unpacking of K and two bf16 ones.
//  * MXFP8 cache, values: E4M3 codes become bf16 by moving bits (value times 2^-120) and one packed multiplication
//    by the block's scale times 2^120; every product of a code and a power of two is exact in bf16.
#include <float.h>

#include <algorithm>
#include <cmath>

#include "moe_decode_device.cuh"

namespace moe {

namespace {

constexpr int kTile = 64;      // tokens of a tile
constexpr int kWarpTok = 16;   // tokens of a tile that a warp owns
constexpr int kTokWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
  moe_kv_cache_t c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  int64_t q_stride, out_stride;
  int L, group, rows, row_tiles, Hq;  // rows = L * group
  float scale_log2;                   // scale * log2(e)
  PageDiv pd;
  int* counters;    // [n_seqs * kv heads * row_tiles], zero between calls
  float* partial;   // [grid][2][rows of a tile][head_dim + 2]
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bytes 0 and 2 (bytes 1 and 3) of four E4M3 codes as a bf16 pair, times 2^-120: the code's exponent and mantissa
// bits at bf16's lowest exponent bits.  Subnormal codes become subnormal bf16 numbers, which the multiplication
// that follows reads as such.
__device__ __forceinline__ uint32_t e4m3_even_bf16(uint32_t r) {
  return ((r << 8) & 0x80008000u) | ((r << 4) & 0x07F007F0u);
}
__device__ __forceinline__ uint32_t e4m3_odd_bf16(uint32_t r) { return (r & 0x80008000u) | ((r >> 4) & 0x07F007F0u); }

// E8M0 byte j of w as a float; byte 0 (2^-127) reads as 0: what it scales is below 2^-118.
__device__ __forceinline__ float e8m0_float(uint32_t w, int j) {
  return __uint_as_float(j == 3 ? (w >> 1) & 0x7F800000u : (w << (23 - 8 * j)) & 0x7F800000u);
}

// Position in the sequence of all tiles: request b (length len, nt tiles), unit w = head * row_tiles + row tile of
// the request, tile t of the unit.
struct Cursor {
  int b, w, t, nt, len;
};

template <int D, bool MX, int MT, int WM>
struct Cfg {
  static constexpr int kWarps = kTokWarps * WM;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 16 * MT * WM;                 // rows of a row tile
  static constexpr int kRowBytes = MX ? D : 2 * D;           // one token of one head
  static constexpr int kScale = MX ? D / 32 : 0;             // scale bytes of a token
  static constexpr int kHalf = kTile * kRowBytes;            // K (or V) of a stage
  static constexpr int kStageBytes = 2 * kHalf + 2 * kTile * kScale;
  static constexpr int kJoinStride = D + 8;                  // floats; 8 rows of a fragment fall on distinct banks
  static constexpr int kJoinBytes = kRows * kJoinStride * 4; // the join's accumulator
  static constexpr int kStatBytes = 2 * kTokWarps * kRows * 4 + 2 * kRows * 4;
  // Blocks an SM holds: two where 16 or 32 rows leave registers for it, one with eight warps.
  static constexpr int kBlocks = WM == 1 ? 2 : 1;
  static constexpr int kBudget = (kBlocks == 2 ? 113 : 226) * 1024 - kJoinBytes - kStatBytes - 256;
  static constexpr int kFit = kBudget / kStageBytes;
  static constexpr int kStages = kFit < 2 ? 2 : kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kStages * kStageBytes + kJoinBytes + kStatBytes + 128;
};

template <int D, bool MX, int MT, int WM>
__global__ void __launch_bounds__(Cfg<D, MX, MT, WM>::kThreads, Cfg<D, MX, MT, WM>::kBlocks)
    paged_attention_kernel(const AttnParams p) {
  using C = Cfg<D, MX, MT, WM>;
  constexpr int kChunks = C::kRowBytes / 16;  // 16-byte pieces of a token row: 16, 8 or 4
  constexpr int kNT = D / 8;                  // output column tiles
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  float* join = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);  // [kRows][kJoinStride]
  float* s_m = join + C::kRows * C::kJoinStride;           // [token warp][row]
  float* s_l = s_m + kTokWarps * C::kRows;    // [token warp][row]
  float* s_M = s_l + kTokWarps * C::kRows;    // [row]
  float* s_Z = s_M + C::kRows;                // [row]
  __shared__ int s_b, s_last;
  __shared__ int64_t s_part[32];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wt = warp % kTokWarps, wm = warp / kTokWarps;  // token group, row half
  const int li = lane >> 2, lc = lane & 3;
  pdl_trigger();
  pdl_wait();

  // ---- this block's run of tiles
  const int B = p.c.n_seqs, HR = p.c.n_kv_heads * p.row_tiles;
  auto tiles_of = [](int len) { return len > 0 ? (len + kTile - 1) / kTile : 1; };
  int64_t sum = 0;
  for (int b = tid; b < B; b += C::kThreads) sum += tiles_of(seq_len_of(p.c, b));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
  if (lane == 0) s_part[warp] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int i = 0; i < C::kWarps; ++i) total += s_part[i];
  total *= HR;
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
  const int64_t t0 = per * blockIdx.x, t1 = t0 + per < total ? t0 + per : total;
  if (t0 >= t1) return;
  Cursor cur;
  int64_t base;  // first tile of request cur.b
  {
    const int64_t want = t0 / HR;  // in tiles of one unit per request
    int64_t carry = 0;
    for (int b0 = 0; b0 < B; b0 += C::kThreads) {
      const int b = b0 + tid;
      const int n = b < B ? tiles_of(seq_len_of(p.c, b)) : 0;
      int64_t incl = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += o;
      }
      __syncthreads();
      if (lane == 31) s_part[warp] = incl;
      __syncthreads();
      int64_t before = carry;
#pragma unroll
      for (int i = 0; i < C::kWarps; ++i) {
        if (i < warp) before += s_part[i];
        carry += s_part[i];
      }
      if (n > 0 && before + incl - n <= want && want < before + incl) {
        s_b = b;
        s_part[31] = before + incl - n;
      }
      __syncthreads();
      if (want < carry) break;
    }
    cur.b = s_b;
    base = s_part[31] * HR;
    cur.len = seq_len_of(p.c, cur.b);
    cur.nt = tiles_of(cur.len);
    const int64_t off = t0 - base;
    cur.w = (int)(off / cur.nt);
    cur.t = (int)(off - (int64_t)cur.w * cur.nt);
  }
  auto advance = [&](Cursor& c) {
    if (++c.t < c.nt) return;
    c.t = 0;
    if (++c.w < HR) return;
    c.w = 0;
    if (++c.b < B) {
      c.len = seq_len_of(p.c, c.b);
      c.nt = tiles_of(c.len);
    }
  };

  // ---- loading: with WM = 1 a warp fetches the 16 tokens it will read; with WM = 2 all warps share the 64
  constexpr int kLoadWarps = WM == 1 ? 1 : C::kWarps;           // warps that share a set of tokens
  constexpr int kLoadTok = WM == 1 ? kWarpTok : kTile;          // tokens in the set
  constexpr int kTokPerWarp = kLoadTok / kLoadWarps;            // tokens one warp fetches: 16 or 8
  const int tok_first = WM == 1 ? wt * kWarpTok : warp * kTokPerWarp;
  const uint32_t smem_base = smem_addr(smem);
  auto swz = [](int row, int chunk) {
    return (kChunks >= 8 ? (chunk ^ (row & 7)) : (chunk ^ ((row >> 1) & 3))) * 16;
  };
  // page of this lane's token of the tile that will be loaded next (lanes 0..kTokPerWarp-1), or -1; looked up one
  // tile ahead, so that the table's latency is not in front of the loads
  Cursor ld = cur;
  int64_t ld_left = t1 - t0;
  int nxt_page = -1, nxt_row = 0;
  auto lookup = [&]() {
    nxt_page = -1;
    const int t = ld.t * kTile + tok_first + lane;
    if (ld_left > 0 && lane < kTokPerWarp && t < ld.len) {
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
  static_assert(!(MX && D == 64) || C::kStages >= 3, "a late scale must be stored, and a barrier passed, before its tile is read");
  auto load_stage = [&](int stage) {
    if constexpr (MX && D == 64) {
      if (late_dst) asm volatile("st.shared.u16 [%0], %1;" ::"r"(late_dst), "h"(late_val) : "memory");
      late_dst = 0;
    }
    if (ld_left > 0) {
      const int head = ld.w / p.row_tiles;
      const int64_t off = nxt_page >= 0 ? nxt_page * p.c.page_stride + nxt_row * p.c.row_stride + head * p.c.head_stride : -1;
      const uint32_t kbase = smem_base + stage * C::kStageBytes;
      constexpr int kPerIter = 32 / kChunks;  // tokens a warp instruction covers
#pragma unroll
      for (int i = 0; i < kTokPerWarp; i += kPerIter) {
        const int tk = i + lane / kChunks, ch = lane % kChunks;
        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, tk);
        const bool ok = o >= 0;
        const uint32_t dst = kbase + (tok_first + tk) * C::kRowBytes + swz(tok_first + tk, ch);
        const int64_t byte = (ok ? o : 0) * (MX ? 1 : 2) + ch * 16;
        cp_async16(dst, static_cast<const uint8_t*>(p.c.k) + byte, ok);
        cp_async16(dst + C::kHalf, static_cast<const uint8_t*>(p.c.v) + byte, ok);
      }
      if constexpr (MX) {  // lane t: K scales, lane 16 + t: V scales (WM = 2: 8 + t)
        const int tk = lane % kTokPerWarp;
        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, tk);
        if (lane < 2 * kTokPerWarp) {
          const bool v = lane >= kTokPerWarp;
          const uint32_t dst = kbase + 2 * C::kHalf + (v ? kTile * C::kScale : 0) + (tok_first + tk) * C::kScale;
          const uint8_t* src = (v ? p.c.v_s : p.c.k_s) + ((o >= 0 ? o : 0) >> 5);
          if constexpr (D == 128) {
            cp_async4(dst, src, o >= 0);
          } else {  // two bytes, less than cp.async copies: through a register, stored one tile later
            late_val = o >= 0 ? __ldg(reinterpret_cast<const uint16_t*>(src)) : (uint16_t)0;
            late_dst = dst;
          }
        }
      }
      --ld_left;
      advance(ld);
      lookup();
    }
    cp_async_commit();
  };
  lookup();
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) load_stage(s);

  // ---- per-unit state
  constexpr int kQ = MX ? D / 32 : D / 16;  // K steps of the scores
  uint32_t qa[MT][kQ][4];
  uint32_t qb[MX ? MT : 1][MX ? kQ : 1][4];  // the second E4M3 term
  float o[MT][kNT][4];
  float m[MT][2], l[MT][2], f[MT][2];        // running maximum (log2 units), this thread's sum, score factor
  int limit[MT][2];

  auto begin_unit = [&]() {
    const int head = cur.w / p.row_tiles, rt = cur.w - head * p.row_tiles;
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = rt * C::kRows + (wm * MT + a) * 16 + li + 8 * h;
        const bool in = r < p.rows;
        const int ql = in ? r / p.group : 0, j = in ? r - ql * p.group : 0;
        limit[a][h] = in ? cur.len - p.L + 1 + ql : 0;
        m[a][h] = -INFINITY;
        l[a][h] = 0.f;
        const __nv_bfloat16* src =
            p.q + ((int64_t)cur.b * p.L + ql) * p.q_stride + ((int64_t)head * p.group + j) * D;
        if constexpr (!MX) {
          f[a][h] = p.scale_log2;
#pragma unroll
          for (int k = 0; k < kQ; ++k) {
            qa[a][k][h] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * lc)) : 0u;
            qa[a][k][h + 2] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * lc)) : 0u;
          }
        } else {
          uint2 raw[kQ][2];
          uint32_t top = 0;  // largest magnitude of the row, as bf16 bits
#pragma unroll
          for (int k = 0; k < kQ; ++k)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              raw[k][z] = in ? __ldg(reinterpret_cast<const uint2*>(src + 32 * k + 16 * z + 4 * lc)) : make_uint2(0u, 0u);
              top = __vmaxu2(top, __vmaxu2(raw[k][z].x & 0x7FFF7FFFu, raw[k][z].y & 0x7FFF7FFFu));
            }
          top = max(top & 0xFFFFu, top >> 16);
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          // 2^up brings the maximum to [2^7, 2^8); rows below 2^-118 stay below it (their scores are 0 in fp32)
          const int be = (int)(top >> 7);
          const int up = be ? min(134 - be, 126) : 126;
          const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
          f[a][h] = be == 255 ? __uint_as_float(0x7FC00000u)
                              : p.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
          for (int k = 0; k < kQ; ++k)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              float v[4] = {__uint_as_float(raw[k][z].x << 16), __uint_as_float(raw[k][z].x & 0xFFFF0000u),
                            __uint_as_float(raw[k][z].y << 16), __uint_as_float(raw[k][z].y & 0xFFFF0000u)};
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] *= mul;
              const uint32_t c0 = e4m3x2(v[0], v[1]), c1 = e4m3x2(v[2], v[3]);
              uint32_t h0, h1;  // the codes back as fp16 pairs (exact)
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((uint16_t)c0));
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((uint16_t)c1));
              const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
              const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
              qa[a][k][h + 2 * z] = c0 | (c1 << 16);
              qb[a][k][h + 2 * z] = (uint32_t)e4m3x2(v[0] - f0.x, v[1] - f0.y) |
                                    ((uint32_t)e4m3x2(v[2] - f1.x, v[3] - f1.y) << 16);
            }
        }
      }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[a][n][e] = 0.f;
  };

  // o += p v, token by token, leaving out the tokens with p = 0
  auto add_values_one_by_one = [&](const float (&s)[MT][2][4], uint32_t vb, uint32_t sb) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        for (int c = 0; c < 4; ++c) {
          const int tk = n * 8 + 2 * c + e;
          float pr[MT][2];
#pragma unroll
          for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) pr[a][h] = __shfl_sync(0xFFFFFFFFu, s[a][n][2 * h + e], (lane & ~3) + c);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int col = MX ? (nt / 2) * 16 + 4 * lc + (nt & 1) + 2 * y : nt * 8 + 2 * lc + y;
              const uint32_t at = vb + tk * C::kRowBytes + swz(tk, (MX ? col : 2 * col) / 16) + (MX ? col : 2 * col) % 16;
              float v;
              if constexpr (MX) {
                uint16_t code;
                uint32_t h2, byte;
                asm volatile("ld.shared.u8 %0, [%1];" : "=h"(code) : "r"(at));
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(sb + (kTile + tk) * C::kScale + col / 32));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(code));
                v = __low2float(*reinterpret_cast<const __half2*>(&h2)) * __uint_as_float(byte << 23);
              } else {
                uint16_t bits;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(at));
                v = __uint_as_float((uint32_t)bits << 16);
              }
#pragma unroll
              for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (pr[a][h] != 0.f) o[a][nt][2 * h + y] = fmaf(pr[a][h], v, o[a][nt][2 * h + y]);
            }
        }
  };

  // ---- one tile: this warp's 16 tokens
  auto tile = [&](int stage) {
    const uint32_t kb = smem_base + stage * C::kStageBytes + wt * kWarpTok * C::kRowBytes;
    const uint32_t vb = kb + C::kHalf;
    const uint32_t sb = smem_base + stage * C::kStageBytes + 2 * C::kHalf + wt * kWarpTok * C::kScale;
    float s[MT][2][4];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[a][n][e] = 0.f;
    const int mrow = lane & 7, mi = lane >> 3;  // this lane's row address in an ldmatrix of four 8 x 16-byte tiles
    if constexpr (!MX) {
#pragma unroll
      for (int k = 0; k < kQ; ++k) {
        const int row = (mi >> 1) * 8 + mrow;
        uint32_t kf[4];
        ldsm4(kb + row * C::kRowBytes + swz(row, 2 * k + (mi & 1)), kf);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          mma_bf16(s[a][0], qa[a][k], kf[0], kf[1]);
          mma_bf16(s[a][1], qa[a][k], kf[2], kf[3]);
        }
      }
    } else {
      uint32_t kw[2][2];  // scale words of this thread's score columns
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t at = sb + (n * 8 + 2 * lc + e) * C::kScale;
          if constexpr (D == 128) {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(kw[n][e]) : "r"(at));
          } else {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(at));
            kw[n][e] = h;
          }
        }
#pragma unroll
      for (int k = 0; k < kQ; ++k) {
        const int row = (mi >> 1) * 8 + mrow;
        uint32_t kf[4];
        ldsm4(kb + row * C::kRowBytes + swz(row, 2 * k + (mi & 1)), kf);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float k0 = e8m0_float(kw[n][0], k), k1 = e8m0_float(kw[n][1], k);
#pragma unroll
          for (int a = 0; a < MT; ++a) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_e4m3(d, qa[a][k], kf[2 * n], kf[2 * n + 1]);
            mma_e4m3(d, qb[a][k], kf[2 * n], kf[2 * n + 1]);
            s[a][n][0] = fmaf(d[0], k0, s[a][n][0]);
            s[a][n][1] = fmaf(d[1], k1, s[a][n][1]);
            s[a][n][2] = fmaf(d[2], k0, s[a][n][2]);
            s[a][n][3] = fmaf(d[3], k1, s[a][n][3]);
          }
        }
      }
    }
    // scale, mask, running maximum
    const int tok0 = cur.t * kTile + wt * kWarpTok;
    const bool edge = tok0 + kWarpTok > cur.len - p.L + 1;  // some row does not see all 16 tokens
    float mx[MT][2];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = s[a][n][2 * h + e] * f[a][h];
            if (edge && tok0 + n * 8 + 2 * lc + e >= limit[a][h]) v = -INFINITY;
            s[a][n][2 * h + e] = v;
          }
        mx[a][h] = fmaxf(fmaxf(s[a][0][2 * h], s[a][0][2 * h + 1]), fmaxf(s[a][1][2 * h], s[a][1][2 * h + 1]));
      }
    bool grow = false;
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[a][h] = fmaxf(mx[a][h], __shfl_xor_sync(0xFFFFFFFFu, mx[a][h], 1));
        mx[a][h] = fmaxf(mx[a][h], __shfl_xor_sync(0xFFFFFFFFu, mx[a][h], 2));
        // the maximum moves only when it is exceeded by more than 2^8: p stays below 256, which costs no
        // precision, and the accumulators are rescaled rarely
        grow |= mx[a][h] > m[a][h] + 8.f;
      }
    if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float nm = fmaxf(m[a][h], mx[a][h]);
          const float c = m[a][h] == nm ? 1.f : ex2(m[a][h] - nm);
          m[a][h] = nm;
          l[a][h] *= c;
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            o[a][n][2 * h] *= c;
            o[a][n][2 * h + 1] *= c;
          }
        }
    }
    uint32_t pa[MT][4];
#pragma unroll
    for (int a = 0; a < MT; ++a) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = m[a][h] == -INFINITY ? 0.f : m[a][h];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) s[a][n][2 * h + e] = ex2(s[a][n][2 * h + e] - ref);
        l[a][h] += (s[a][0][2 * h] + s[a][0][2 * h + 1]) + (s[a][1][2 * h] + s[a][1][2 * h + 1]);
      }
      pa[a][0] = pack_bf16(s[a][0][0], s[a][0][1]);
      pa[a][1] = pack_bf16(s[a][0][2], s[a][0][3]);
      pa[a][2] = pack_bf16(s[a][1][0], s[a][1][1]);
      pa[a][3] = pack_bf16(s[a][1][2], s[a][1][3]);
    }
    // Tokens that some rows see and others do not (the step's own new tokens): p = 0 must keep a NaN or an
    // infinity out, which a matrix product would let through.  Rare, so it is looked for only in such tiles.
    if (edge && p.L > 1) {
      bool odd = false;
      for (int i = lane; i < kWarpTok * C::kRowBytes / 16; i += 32) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(vb + i * 16));
#pragma unroll
        for (int z = 0; z < 4; ++z)
          odd |= MX ? __vcmpeq4(w[z] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u : __vcmpeq2(w[z] & 0x7F807F80u, 0x7F807F80u) != 0u;
      }
      if (__any_sync(0xFFFFFFFFu, odd)) {
        add_values_one_by_one(s, vb, sb);
        return;
      }
    }
    const int vrow = (mi & 1) * 8 + mrow;
    if constexpr (!MX) {
#pragma unroll
      for (int n = 0; n < kNT; n += 2) {
        uint32_t vf[4];
        ldsm4_trans(vb + vrow * C::kRowBytes + swz(vrow, n + (mi >> 1)), vf);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          mma_bf16(o[a][n], pa[a], vf[0], vf[1]);
          mma_bf16(o[a][n + 1], pa[a], vf[2], vf[3]);
        }
      }
    } else {
      // scale words of tokens 2c, 2c + 1 and 2c + 8, 2c + 9: the pairs that a B fragment register holds
      uint32_t vw[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t at = sb + (kTile + n * 8 + 2 * lc + e) * C::kScale;
          if constexpr (D == 128) {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vw[n][e]) : "r"(at));
          } else {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(at));
            vw[n][e] = h;
          }
        }
      // a scale above 2^7 does not fit the one multiplier 2^(byte - 127 + 120): its rest is a second one
      const bool large = __any_sync(0xFFFFFFFFu, (__vcmpgtu4(vw[0][0], 0x86868686u) | __vcmpgtu4(vw[0][1], 0x86868686u) |
                                                  __vcmpgtu4(vw[1][0], 0x86868686u) | __vcmpgtu4(vw[1][1], 0x86868686u)) != 0u);
#pragma unroll
      for (int cc = 0; cc < D / 16; cc += 2) {  // chunks of 16 columns; a pair of chunks is one MX block
        uint32_t vf[4];
        ldsm4_trans(vb + vrow * C::kRowBytes + swz(vrow, cc + (mi >> 1)), vf);
        uint32_t mul[2], rest[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t pair = ((vw[n][0] >> (4 * cc)) & 0xFFu) | (((vw[n][1] >> (4 * cc)) & 0xFFu) << 16);
          rest[n] = 0x3F803F80u;
          if (large) {
            const uint32_t cut = __vminu2(pair, 0x00860086u);
            rest[n] += (pair - cut) << 7;
            pair = cut;
          }
          mul[n] = pair * 128u + 0x3C003C00u;
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {  // chunk cc + z
          uint32_t e0 = mul_bf16x2(e4m3_even_bf16(vf[2 * z]), mul[0]), e1 = mul_bf16x2(e4m3_even_bf16(vf[2 * z + 1]), mul[1]);
          uint32_t d0 = mul_bf16x2(e4m3_odd_bf16(vf[2 * z]), mul[0]), d1 = mul_bf16x2(e4m3_odd_bf16(vf[2 * z + 1]), mul[1]);
          if (large) {
            e0 = mul_bf16x2(e0, rest[0]), e1 = mul_bf16x2(e1, rest[1]);
            d0 = mul_bf16x2(d0, rest[0]), d1 = mul_bf16x2(d1, rest[1]);
          }
#pragma unroll
          for (int a = 0; a < MT; ++a) {
            mma_bf16(o[a][2 * (cc + z)], pa[a], e0, e1);      // columns 16 (cc + z) + 0, 2, 4 ..
            mma_bf16(o[a][2 * (cc + z) + 1], pa[a], d0, d1);  // .. and 1, 3, 5 ..
          }
        }
      }
    }
  };

  // ---- a unit's end: join the token groups, then write the rows, or this block's part of them
  const int64_t cta0 = t0;  // first tile of this block
  auto end_unit = [&](int64_t unit_first, int first_tile) {
    const int head = cur.w / p.row_tiles, rt = cur.w - head * p.row_tiles;
    const int row0 = rt * C::kRows;
    const int nrows = min(C::kRows, p.rows - row0);
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[a][h] += __shfl_xor_sync(0xFFFFFFFFu, l[a][h], 1);
        l[a][h] += __shfl_xor_sync(0xFFFFFFFFu, l[a][h], 2);
        if (lc == 0) s_m[wt * C::kRows + (wm * MT + a) * 16 + li + 8 * h] = m[a][h];
      }
    __syncthreads();  // also: the previous unit's readers of join are done
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (wm * MT + a) * 16 + li + 8 * h;
        float M = s_m[r];
#pragma unroll
        for (int w = 1; w < kTokWarps; ++w) M = fmaxf(M, s_m[w * C::kRows + r]);
        const float c = m[a][h] == -INFINITY ? 0.f : ex2(m[a][h] - M);
        if (lc == 0) {
          s_l[wt * C::kRows + r] = l[a][h] * c;
          if (wt == 0) s_M[r] = M;
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          o[a][n][2 * h] *= c;
          o[a][n][2 * h + 1] *= c;
        }
      }
    // four rounds: in round i token group w adds columns quarter (w + i) % 4, so that all warps work in every
    // round and each quarter receives the groups in a fixed order
    constexpr int kQuarter = kNT / 4;
#pragma unroll
    for (int i = 0; i < kTokWarps; ++i) {
      const int quarter = (wt + i) % kTokWarps;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        if (n / kQuarter != quarter) continue;
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float* row = join + ((wm * MT + a) * 16 + li + 8 * h) * C::kJoinStride;
            // MXFP8: tile 2 cc holds the even columns of chunk cc, tile 2 cc + 1 the odd ones
            const int c0 = MX ? (n / 2) * 16 + 4 * lc + (n & 1) : n * 8 + 2 * lc;
            const int c1 = MX ? c0 + 2 : c0 + 1;
            if (i == 0) {
              row[c0] = o[a][n][2 * h];
              row[c1] = o[a][n][2 * h + 1];
            } else {
              row[c0] += o[a][n][2 * h];
              row[c1] += o[a][n][2 * h + 1];
            }
          }
      }
      __syncthreads();
    }
    if (tid < C::kRows) {
      float z = 0.f;
#pragma unroll
      for (int w = 0; w < kTokWarps; ++w) z += s_l[w * C::kRows + tid];
      s_Z[tid] = z;
    }
    __syncthreads();
    const int64_t unit_end = unit_first + cur.nt;
    auto write_row8 = [&](int r, int c8, const float (&v)[8], float inv) {
      const int ql = (row0 + r) / p.group, j = row0 + r - ql * p.group;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[i] * inv;
      *reinterpret_cast<uint4*>(p.out + ((int64_t)cur.b * p.L + ql) * p.out_stride +
                                ((int64_t)head * p.group + j) * D + c8) = f32_to_bf16x8(y);
    };
    auto write_lse = [&](int r, float M, float z) {
      const int ql = (row0 + r) / p.group, j = row0 + r - ql * p.group;
      p.lse[((int64_t)cur.b * p.L + ql) * p.Hq + head * p.group + j] = M == -INFINITY ? -INFINITY : (M + log2f(z)) * kLn2;
    };
    // rows that see nothing: z = 0, result 0; a NaN sum stays NaN
    auto inverse = [](float z) { return z == 0.f ? 0.f : 1.f / z; };
    if (first_tile == 0 && unit_end <= t1) {  // the whole unit was this block's
      for (int i = tid; i < nrows * (D / 8); i += C::kThreads) {
        const int r = i / (D / 8), c8 = (i % (D / 8)) * 8;
        float v[8];
        *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(join + r * C::kJoinStride + c8);
        *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(join + r * C::kJoinStride + c8 + 4);
        write_row8(r, c8, v, inverse(s_Z[r]));
      }
      if (p.lse && tid < nrows) write_lse(tid, s_M[tid], s_Z[tid]);
      return;
    }
    // part of a unit: slot 0 of a block is the unit its run begins in, slot 1 the one that it ends in
    constexpr size_t kSlot = (size_t)C::kRows * (D + 2);
    float* mine = p.partial + ((size_t)blockIdx.x * 2 + (unit_first > cta0 ? 1 : 0)) * kSlot;
    for (int i = tid; i < nrows * (D / 4); i += C::kThreads) {
      const int r = i / (D / 4), c4 = (i % (D / 4)) * 4;
      __stcg(reinterpret_cast<float4*>(mine + r * D + c4), *reinterpret_cast<const float4*>(join + r * C::kJoinStride + c4));
    }
    if (tid < nrows) {
      __stcg(mine + C::kRows * D + tid, s_M[tid]);
      __stcg(mine + C::kRows * (D + 1) + tid, s_Z[tid]);
    }
    __threadfence();
    __syncthreads();
    const int64_t b0 = unit_first / per, b1 = (unit_end - 1) / per;
    const int parts = (int)(b1 - b0) + 1;
    if (tid == 0) {
      int* counter = p.counters + (int64_t)cur.b * HR + cur.w;
      const int n = atomicAdd(counter, 1);
      s_last = n == parts - 1;
      if (s_last) *counter = 0;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the last block joins the parts in block order
    auto part = [&](int i) {
      return p.partial + ((size_t)(b0 + i) * 2 + (i == 0 && unit_first > b0 * per ? 1 : 0)) * kSlot;
    };
    for (int r = warp; r < nrows; r += C::kWarps) {
      float M = -INFINITY;
      for (int i = lane; i < parts; i += 32) M = fmaxf(M, __ldcg(part(i) + C::kRows * D + r));
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
      const float ref = M == -INFINITY ? 0.f : M;
      float z = 0.f;
      for (int i = lane; i < parts; i += 32)
        z += __ldcg(part(i) + C::kRows * (D + 1) + r) * ex2(__ldcg(part(i) + C::kRows * D + r) - ref);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
      if (lane == 0) {
        s_M[r] = M;
        s_Z[r] = z;
      }
    }
    __syncthreads();
    for (int i = tid; i < nrows * (D / 8); i += C::kThreads) {
      const int r = i / (D / 8), c8 = (i % (D / 8)) * 8;
      const float ref = s_M[r] == -INFINITY ? 0.f : s_M[r];
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int k = 0; k < parts; ++k) {
        const float* src = part(k);
        const float c = ex2(__ldcg(src + C::kRows * D + r) - ref);
        const float4 x = __ldcg(reinterpret_cast<const float4*>(src + r * D + c8));
        const float4 y = __ldcg(reinterpret_cast<const float4*>(src + r * D + c8 + 4));
        v[0] = fmaf(x.x, c, v[0]), v[1] = fmaf(x.y, c, v[1]), v[2] = fmaf(x.z, c, v[2]), v[3] = fmaf(x.w, c, v[3]);
        v[4] = fmaf(y.x, c, v[4]), v[5] = fmaf(y.y, c, v[5]), v[6] = fmaf(y.z, c, v[6]), v[7] = fmaf(y.w, c, v[7]);
      }
      write_row8(r, c8, v, inverse(s_Z[r]));
    }
    if (p.lse && tid < nrows) write_lse(tid, s_M[tid], s_Z[tid]);
  };

  // ---- the run
  int stage = 0;
  int64_t pos = t0;
  int first_tile = cur.t;
  bool fresh = true;
  while (pos < t1) {
    if (fresh) {
      begin_unit();
      fresh = false;
    }
    cp_async_wait<C::kStages - 2>();
    if constexpr (WM == 1)
      __syncwarp();
    else
      __syncthreads();
    // the slot of the previous tile is free (its readers passed the barrier above)
    load_stage(stage == 0 ? C::kStages - 1 : stage - 1);
    tile(stage);
    stage = stage == C::kStages - 1 ? 0 : stage + 1;
    ++pos;
    if (cur.t + 1 == cur.nt || pos == t1) {
      end_unit(pos - 1 - cur.t, first_tile);
      first_tile = 0;
      fresh = true;
    }
    advance(cur);
  }
  cp_async_wait<0>();
}

template <int D, bool MX, int MT, int WM>
cudaError_t launch_one(const AttnParams& p, int num_sms, cudaStream_t s) {
  using C = Cfg<D, MX, MT, WM>;
  auto* kernel = paged_attention_kernel<D, MX, MT, WM>;
  static PerDeviceOnce once;
  cudaError_t e =
      once.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(num_sms * C::kBlocks), dim3(C::kThreads), C::kSmem, s, p);
}

// Rows of a row tile: the smallest of 16, 32 and 64 that holds the rows of a kv head, 64 above that.
int tile_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int D, bool MX>
cudaError_t launch_rows(const AttnParams& p, int num_sms, cudaStream_t s) {
  switch (tile_rows(p.rows)) {
    case 16: return launch_one<D, MX, 1, 1>(p, num_sms, s);
    case 32: return launch_one<D, MX, 2, 1>(p, num_sms, s);
    default: return launch_one<D, MX, 2, 2>(p, num_sms, s);
  }
}

struct Sizes {
  int64_t rows;
  int row_tiles;
  size_t counters, bytes;
};

moe_status_t plan(const moe_kv_cache_t& c, int n_q_heads, int L, int num_sms, const char* call, Sizes* z) {
  if (n_q_heads < 1 || n_q_heads % c.n_kv_heads)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", call,
                       n_q_heads, c.n_kv_heads);
  if (L < 0) return decode_fail(MOE_ERR_INVALID_ARG, "%s: L = %d is negative", call, L);
  z->rows = (int64_t)(n_q_heads / c.n_kv_heads) * L;
  if (z->rows > (1 << 20) || (int64_t)n_q_heads * c.head_dim > (1ll << 31))
    return decode_fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^20 rows a kv head", call);
  const int tr = tile_rows(z->rows);
  z->row_tiles = (int)((z->rows + tr - 1) / tr);
  const int64_t units = (int64_t)c.n_seqs * c.n_kv_heads * z->row_tiles;
  if (units > (1ll << 30)) return decode_fail(MOE_ERR_UNSUPPORTED, "%s: too many row tiles", call);
  z->counters = ((size_t)units * 4 + 255) / 256 * 256;
  const int blocks = num_sms * (tr == 64 ? 1 : 2);
  z->bytes = z->counters + (size_t)blocks * 2 * tr * (c.head_dim + 2) * 4;
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
  p.counters = static_cast<int*>(a->workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + z.counters);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool mx = c.format == MOE_KV_MXFP8;
  cudaError_t e = c.head_dim == 128 ? (mx ? launch_rows<128, true>(p, sms, s) : launch_rows<128, false>(p, sms, s))
                                    : (mx ? launch_rows<64, true>(p, sms, s) : launch_rows<64, false>(p, sms, s));
  if (e != cudaSuccess) return decode_fail(MOE_ERR_CUDA, "moe_paged_attention: %s", cudaGetErrorString(e));
  return MOE_OK;
}
