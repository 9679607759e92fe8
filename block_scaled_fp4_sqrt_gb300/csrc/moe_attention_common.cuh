// What the forms of the paged attention share: the call's parameters, the dealing of the work to the blocks, copies into
// shared memory and the matrix instructions.
//
// A unit is (request, kv head, row tile).  Every unit is cut into tiles of TILE tokens; the tiles of all units, in order and
// with COST places in front of each unit's first, are dealt to the grid in equal contiguous runs of places, computed by
// every block from the lengths alone.
#pragma once

#include "moe_decode_device.cuh"

namespace moe {

struct AttnParams {
  moe_kv_cache_t c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  int64_t q_stride, out_stride;
  int L, group, rows, row_tiles, Hq;  // rows = L * group
  int lanes;  // MXFP4: kv heads that as many blocks read side by side
  uint32_t page_units, row_units, head_units;  // the cache's strides in 16-byte units
  float scale_log2;                   // scale * log2(e)
  PageDiv pd;
  int* counters;    // [grid] of the shared unit that begins in a block (at most one does), zero between calls
  float* partial;   // [grid][2][rows of a tile][head_dim + 2]
  int* group_counters;   // [grid / kJoin + 1][2], zero between calls
  float* group_partial;  // [grid / kJoin + 1][2][rows of a tile][head_dim + 2]
};

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kJoin = 16;                 // parts that are joined in one step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;


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
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b (no accumulator to clear first)
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// (c0, c1) += (a0, a1) * (b0, b1)
__device__ __forceinline__ void fma2(float& c0, float& c1, float a0, float a1, float b0, float b1) {
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%0, %1};\n"
      " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}"
      : "+f"(c0), "+f"(c1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
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

// Position in the sequence of all tiles: request b (length len, nt tiles a unit), kv head, row tile rt, tile t.
struct Cursor {
  int b, head, rt, t, nt, len;
};


// A block's run of places [t0, t1): cur is its first tile, at place pos.
struct Run {
  Cursor cur;
  int64_t t0, t1, per, pos;
};

template <int TILE>
__device__ __forceinline__ int tiles_of(int len) {
  return len > 0 ? (len + TILE - 1) / TILE : 1;
}

// a / b for a >= 0, b > 0 (a 64-bit division takes some hundred cycles).
__device__ __forceinline__ int64_t places_div(int64_t a, int b) {
  return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The run of block `index` of `blocks` over the tiles of `heads` kv heads of every request; false where it has no tile.
// All threads of the block call it.
template <int TILE, int COST>
__device__ __forceinline__ bool deal_run(const AttnParams& p, int heads, int blocks, int index, int tid, Run& run) {
  __shared__ int s_b, s_len;
  __shared__ int64_t s_part[kWarps], s_first;
  const int warp = tid >> 5, lane = tid & 31;
  const int B = p.c.n_seqs, HR = heads * p.row_tiles;
  const int len0 = tid < B ? seq_len_of(p.c, tid) : 0;  // of the first kThreads requests: read once
  auto places = [&](int b) { return tiles_of<TILE>(b == tid ? len0 : seq_len_of(p.c, b)) + COST; };
  int64_t sum = 0;
  for (int b = tid; b < B; b += kThreads) sum += places(b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
  if (lane == 0) s_part[warp] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) total += s_part[i];
  total *= HR;
  const int64_t per = places_div(total + blocks - 1, blocks);
  const int64_t t0 = per * index, t1 = t0 + per < total ? t0 + per : total;
  if (t0 >= t1) return false;
  Cursor cur;
  {
    const int64_t want = places_div(t0, HR);  // in places of one unit per request
    int64_t carry = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
      const int b = b0 + tid;
      const int n = b < B ? places(b) : 0;
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
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += s_part[i];
        carry += s_part[i];
      }
      if (n > 0 && before + incl - n <= want && want < before + incl) {
        s_b = b;
        s_len = b == tid ? len0 : seq_len_of(p.c, b);
        s_first = before + incl - n;
      }
      __syncthreads();
      if (want < carry) break;
    }
    cur.b = s_b;
    cur.len = s_len;
    cur.nt = tiles_of<TILE>(cur.len);
    const int64_t off = t0 - s_first * HR;
    const int w = (int)places_div(off, cur.nt + COST);
    cur.t = (int)(off - (int64_t)w * (cur.nt + COST)) - COST;
    cur.head = w / p.row_tiles;
    cur.rt = w - cur.head * p.row_tiles;
  }
  int64_t pos = t0;  // place of the tile cur
  if (cur.t < 0) {   // the run begins in front of a unit's first tile
    pos -= cur.t;
    cur.t = 0;
  }
  run = {cur, t0, t1, per, pos};
  return pos < t1;
}

// To the next tile; returns how many places further it lies.
template <int TILE, int COST>
__device__ __forceinline__ int advance_tile(const AttnParams& p, int heads, Cursor& c) {
  if (++c.t < c.nt) return 1;
  c.t = 0;
  if (++c.rt < p.row_tiles) return 1 + COST;
  c.rt = 0;
  if (++c.head < heads) return 1 + COST;
  c.head = 0;
  if (++c.b < p.c.n_seqs) {
    c.len = seq_len_of(p.c, c.b);
    c.nt = tiles_of<TILE>(c.len);
  }
  return 1 + COST;
}

}  // namespace

}  // namespace moe
