// The pages of a paged cache: branches, growth with copy on write, truncation, compaction (moe_pages_*), and the copies of
// page contents that these ask for (moe_copy_pages).
//
// The tables are small (a pool of 200,000 pages: 0.8 MB of counts), so their calls are bound by latency: one kernel each, one
// cluster of eight blocks that meet at cluster barriers, no workspace.  What a call decides follows from prefix sums over
// the requests and over the pages: the i-th wanted page is the i-th free one, whatever the order in which blocks run.
// Measured: a step's growth of 256 requests in 200,000 pages 10 us at 30 % held, 18 at 95 %, 51 at 99 % (the walk for free
// pages ends where enough have been met), a fork of 256 requests 8, of two 4; a compaction's plan in 4000 pages 12, in 200,000
// 66 to 78, and with eight requests, whose rows of the table are a warp's work each, 135 to 290.
// The copies are bound by memory: every byte of a page is read and written once, 16 at a time, by blocks that take a window
// of 256 pairs each and deal its pages evenly.  4096 pages of 128 KB 168 us, 92 % of the copy rate.
#include <algorithm>

#include "moe_decode_device.cuh"

namespace moe {

namespace {

constexpr int kCluster = 8;
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;

// Every block's writes before it are read by all blocks after it (global memory past the L1 cache).
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
// The int at `p` of block `rank` of the cluster.
__device__ __forceinline__ int cluster_read(const int* p, int rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// Sum of v over the block's threads before this one; total receives the whole sum.  All threads call it.
__device__ __forceinline__ int block_scan(int v, int& total) {
  __shared__ int s_w[kPoolWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += o;
  }
  __syncthreads();
  if (lane == 31) s_w[warp] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kPoolWarps; ++i) {
    if (i < warp) before += s_w[i];
    total += s_w[i];
  }
  return before + incl - v;
}

// A cluster's sums of v over its blocks before this one, and over all; s holds v of each block and is used for one scan only
// (no block may still read it when it changes, or leave before the others have: a later cluster_meet sees to that).  All
// threads call it.
__device__ __forceinline__ int2 cluster_scan(int2 v, int2* s, int rank, int2& total) {
  if (threadIdx.x == 0) *s = v;
  cluster_meet();
  int2 before = make_int2(0, 0);
  total = make_int2(0, 0);
#pragma unroll
  for (int i = 0; i < kCluster; ++i) {
    const int2 x = make_int2(cluster_read(&s->x, i), cluster_read(&s->y, i));
    if (i < rank) before.x += x.x, before.y += x.y;
    total.x += x.x, total.y += x.y;
  }
  return before;
}

// f(i, page_refs[i]) for this block's part [lo, hi) of the pages, sixteen loads of a thread under way together.
template <typename F>
__device__ __forceinline__ void each_page(const moe_page_pool_t& p, int lo, int hi, F&& f) {
  constexpr int kAhead = 16;
  for (int i0 = lo + (int)threadIdx.x; i0 < hi; i0 += kAhead * kPoolThreads) {
    int r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) r[u] = i0 + u * kPoolThreads < hi ? __ldcg(p.page_refs + i0 + u * kPoolThreads) : 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i0 + u * kPoolThreads < hi) f(i0 + u * kPoolThreads, r[u]);
  }
}

// f(j, row[j]) for a warp's lanes over the entries j0 .. j1 of a request's row of the table, four loads of a lane together.
template <typename F>
__device__ __forceinline__ void each_entry(const int32_t* row, int j0, int j1, F&& f) {
  constexpr int kAhead = 4;
  for (int j = j0 + (int)(threadIdx.x & 31); j < j1; j += kAhead * 32) {
    int e[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) e[u] = j + 32 * u < j1 ? __ldcg(row + j + 32 * u) : -1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j + 32 * u < j1) f(j + 32 * u, e[u]);
  }
}

__device__ __forceinline__ int pages_of(int len, int page_size) { return len / page_size + (len % page_size != 0); }

// A request's length, clamped to what its block table can hold.
__device__ __forceinline__ int pool_len(const moe_page_pool_t& p, int b) {
  const int n = __ldcg(p.seq_lens + b), cap = p.max_pages * p.page_size;
  if (n >= 0 && n <= cap) return n;
  set_status(p.status, MOE_KV_BAD_LENGTH);
  return n < 0 ? 0 : cap;
}
__device__ __forceinline__ bool page_ok(const moe_page_pool_t& p, int page) {
  if ((unsigned)page < (unsigned)p.n_pages) return true;
  set_status(p.status, MOE_KV_BAD_PAGE);
  return false;
}

// ---------------------------------------------------------------------------------------------- fork
__global__ void __launch_bounds__(kPoolThreads, 1) pages_fork_kernel(const moe_page_pool_t p, const int32_t* src,
                                                                  const int32_t* dst, int n) {
  __shared__ int s_claim[MOE_POOL_MAX_SEQS];  // the first pair that names a request as its branch
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = cluster_rank();
  for (int i = tid; i < p.n_seqs; i += kPoolThreads) s_claim[i] = 0x7FFFFFFF;
  __syncthreads();
  for (int i = tid; i < n; i += kPoolThreads) {
    const int d = __ldg(dst + i);
    if ((unsigned)d < (unsigned)p.n_seqs) atomicMin(&s_claim[d], i);
  }
  __syncthreads();
  // a warp of the cluster takes the pairs of its number; n <= MOE_POOL_MAX_SEQS, 32 a warp: lane k keeps the k-th's length
  constexpr int kWarpsAll = kCluster * kPoolWarps;
  static_assert(MOE_POOL_MAX_SEQS <= 32 * kWarpsAll, "a warp remembers 32 pairs");
  int kept = -1;
  int k = 0;
  for (int i = rank * kPoolWarps + warp; i < n; i += kWarpsAll, ++k) {
    const int a = __ldg(src + i), d = __ldg(dst + i);
    const bool in = (unsigned)a < (unsigned)p.n_seqs && (unsigned)d < (unsigned)p.n_seqs;
    if (!in || s_claim[d] != i || __ldcg(p.seq_lens + d) != 0) {
      if (lane == 0) set_status(p.status, MOE_POOL_BAD_REQUEST);
      continue;
    }
    const int len = pool_len(p, a), np = pages_of(len, p.page_size);
    // (a source with pages is no branch of another pair: its row does not change here)
    int32_t* to = p.block_table + (int64_t)d * p.max_pages;
    each_entry(p.block_table + (int64_t)a * p.max_pages, 0, np, [&](int j, int page) {
      to[j] = page;
      if (page_ok(p, page)) atomicAdd(p.page_refs + page, 1);
    });
    if (k == lane) kept = len;
  }
  cluster_meet();  // every length has been read
  k = 0;
  for (int i = rank * kPoolWarps + warp; i < n; i += kWarpsAll, ++k)
    if (k == lane && kept >= 0) p.seq_lens[__ldg(dst + i)] = kept;
}

// ---------------------------------------------------------------------------------------------- resize
__global__ void __launch_bounds__(kPoolThreads, 1) pages_resize_kernel(const moe_page_pool_t p, const int32_t* new_lens,
                                                                    int2* copies) {
  __shared__ int s_end[MOE_POOL_MAX_SEQS];  // pages wanted by the requests up to and with this one; sign bit: with a copy
  __shared__ int2 s_sum;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = cluster_rank();
  const int P = p.page_size;
  const int64_t cap = (int64_t)p.max_pages * P;
  // the length that request b is to get
  auto target = [&](int b, int old) {
    const int n = __ldg(new_lens + b);
    return n >= 0 && n <= cap ? n : old;
  };

  // What the calls of the first requests look up below, asked for now: nothing before the first meeting changes it.
  int first_old = 0, first_now = 0, first_last = -1;
  if (tid < p.n_seqs) {
    first_old = pool_len(p, tid), first_now = target(tid, first_old);
    if (first_now > first_old && first_old % P) first_last = __ldcg(p.block_table + (int64_t)tid * p.max_pages + first_old / P);
  }
  // pages go back, a warp a request
  for (int b = rank * kPoolWarps + warp; b < p.n_seqs; b += kCluster * kPoolWarps) {
    const int old = pool_len(p, b), now = target(b, old);
    if (lane == 0 && now != __ldg(new_lens + b)) set_status(p.status, MOE_KV_BAD_LENGTH);
    int32_t* row = p.block_table + (int64_t)b * p.max_pages;
    each_entry(row, pages_of(now, P), pages_of(old, P), [&](int j, int page) {
      if (page_ok(p, page)) atomicSub(p.page_refs + page, 1);
      row[j] = -1;
    });
  }
  cluster_meet();

  // what the requests want, in order (every block for itself)
  int carry = 0;
  for (int b0 = 0; b0 < p.n_seqs; b0 += kPoolThreads) {
    const int b = b0 + tid;
    int want = 0;
    bool copy = false;
    if (b < p.n_seqs) {
      const int old = b0 ? pool_len(p, b) : first_old, now = b0 ? target(b, old) : first_now;
      if (now > old) {
        if (old % P) {
          const int last = b0 ? __ldcg(p.block_table + (int64_t)b * p.max_pages + old / P) : first_last;
          copy = page_ok(p, last) && __ldcg(p.page_refs + last) > 1;
        }
        want = pages_of(now, P) - pages_of(old, P) + copy;
      }
    }
    int total;
    const int before = block_scan(want, total);
    if (b < p.n_seqs) s_end[b] = (carry + before + want) | (copy ? (int)0x80000000 : 0);
    carry += total;
  }
  __syncthreads();

  // the free pages of this block's part of the pool
  const int per = (p.n_pages + kCluster - 1) / kCluster;
  const int lo = min(p.n_pages, rank * per), hi = min(p.n_pages, lo + per);
  int mine = 0, in_block;
  each_page(p, lo, hi, [&](int, int refs) { mine += refs == 0; });
  block_scan(mine, in_block);
  int2 all;
  int first = cluster_scan(make_int2(in_block, 0), &s_sum, rank, all).x;
  const int n_free = all.x;
  // requests are served in order while the free pages last, and those that want none
  auto end_of = [&](int b) { return s_end[b] & 0x7FFFFFFF; };
  auto start_of = [&](int b) { return b ? end_of(b - 1) : 0; };
  auto served = [&](int b) { return end_of(b) == start_of(b) || end_of(b) <= n_free; };
  const int last_want = min(carry, n_free);
  for (int i0 = lo; i0 < hi && first < last_want; i0 += kPoolThreads) {
    const int i = i0 + tid;
    const bool free = i < hi && __ldcg(p.page_refs + i) == 0;
    int total;
    const int r = first + block_scan(free, total);  // this page's number among the free ones
    first += total;
    if (free && r < last_want) {
      int b = 0;  // the first request whose pages end behind r
      for (int step = MOE_POOL_MAX_SEQS; step; step >>= 1)
        if (b + step <= p.n_seqs && end_of(b + step - 1) <= r) b += step;
      if (served(b)) {
        const int k = r - start_of(b), old = pool_len(p, b);
        const bool copy = s_end[b] < 0;
        int32_t* at = p.block_table + (int64_t)b * p.max_pages + pages_of(old, P) - copy + k;
        if (copy && k == 0) copies[b] = make_int2(*at, i);
        *at = i;
        p.page_refs[i] = 1;
      }
    }
  }
  cluster_meet();  // all free pages have been found: the counts of copied pages may fall

  for (int b = rank * kPoolThreads + tid; b < p.n_seqs; b += kCluster * kPoolThreads) {
    const bool ok = served(b);
    if (ok && s_end[b] < 0)
      atomicSub(p.page_refs + __ldcg(copies + b).x, 1);
    else
      copies[b] = make_int2(-1, -1);
    const int old = pool_len(p, b);
    if (ok)
      p.seq_lens[b] = target(b, old);
    else
      set_status(p.status, MOE_POOL_EXHAUSTED);
  }
}

// ---------------------------------------------------------------------------------------------- compact
__global__ void __launch_bounds__(kPoolThreads, 1) pages_compact_kernel(const moe_page_pool_t p, int2* copies, int capacity) {
  __shared__ int2 s_live, s_moves;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, rank = cluster_rank();
  const int per = (p.n_pages + kCluster - 1) / kCluster;
  const int lo = min(p.n_pages, rank * per), hi = min(p.n_pages, lo + per);
  int live = 0, total;
  int2 all;
  each_page(p, lo, hi, [&](int, int refs) { live += refs != 0; });
  block_scan(live, total);
  cluster_scan(make_int2(total, 0), &s_live, rank, all);
  const int n_live = all.x;
  // live pages from n_live on move into the free ones below: there are as many of the one as of the other
  auto is_hole = [&](int i, int refs) { return i < n_live && refs == 0; };
  auto is_mover = [&](int i, int refs) { return i >= n_live && refs != 0; };
  int holes = 0, movers = 0, total_movers;
  each_page(p, lo, hi, [&](int i, int refs) { holes += is_hole(i, refs), movers += is_mover(i, refs); });
  block_scan(holes, total);
  block_scan(movers, total_movers);
  const int2 before = cluster_scan(make_int2(total, total_movers), &s_moves, rank, all);
  const int n_moves = all.x;
  int hole = before.x, mover = before.y;
  const int moves = min(n_moves, capacity);
  int32_t* flat = reinterpret_cast<int32_t*>(copies);
  for (int i0 = lo; i0 < hi; i0 += kPoolThreads) {
    const int i = i0 + tid, refs = i < hi ? __ldcg(p.page_refs + i) : 0;
    const bool h = i < hi && is_hole(i, refs), m = i < hi && is_mover(i, refs);
    const int rh = hole + block_scan(h, total);
    hole += total;
    const int rm = n_moves - 1 - (mover + block_scan(m, total));  // the highest mover is the first
    mover += total;
    if (h && rh < moves) flat[2 * (int64_t)rh + 1] = i;
    if (m && rm < moves) flat[2 * (int64_t)rm] = i;
  }
  for (int64_t i = moves + rank * kPoolThreads + tid; i < capacity; i += kCluster * kPoolThreads) copies[i] = make_int2(-1, -1);
  cluster_meet();

  // the counts move, and a moved page's count says where to, until the tables have been rewritten
  for (int i = rank * kPoolThreads + tid; i < moves; i += kCluster * kPoolThreads) {
    const int2 c = __ldcg(copies + i);
    p.page_refs[c.y] = __ldcg(p.page_refs + c.x);
    p.page_refs[c.x] = -1 - c.y;
  }
  cluster_meet();
  for (int b = rank * kPoolWarps + warp; b < p.n_seqs; b += kCluster * kPoolWarps) {
    int32_t* row = p.block_table + (int64_t)b * p.max_pages;
    const int np = pages_of(pool_len(p, b), p.page_size);
    each_entry(row, 0, np, [&](int j, int page) {
      if (!page_ok(p, page)) return;
      const int to = -1 - __ldcg(p.page_refs + page);
      if (to >= 0 && to < n_live && page >= n_live) row[j] = to;
    });
  }
  cluster_meet();
  for (int i = rank * kPoolThreads + tid; i < moves; i += kCluster * kPoolThreads) p.page_refs[__ldcg(copies + i).x] = 0;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kPoolThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------------------------------------- copies
// One tensor of a cache: a page is n1 x n2 runs of `units` words of the kernel's width, at these strides in words.
struct CopyTensor {
  uint8_t* base;
  int64_t page_stride, s1, s2;
  uint32_t n2, units, words;  // words = n1 * n2 * units of a page
};
constexpr int kCopyTensors = 64;
struct CopyParams {
  CopyTensor t[kCopyTensors];
  int32_t* status[kCopyTensors];
  int32_t n_pages[kCopyTensors];
  const int2* copies;
  int32_t n, n_tensors;
};
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyItem = kCopyThreads * kCopyUnroll;  // words of an item

template <typename W>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  __shared__ int2 s_pair[kCopyThreads];
  __shared__ int s_live[kCopyThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  uint32_t most = 0;
  for (int i = 0; i < p.n_tensors; ++i) most = max(most, p.t[i].words);
  const uint32_t items = (most + kCopyItem - 1) / kCopyItem;  // of a tensor's page
  // a window of pairs at a time: its pairs that are to be copied, in order (every block has the same list), then their items
  // dealt to all blocks
  uint64_t turn = blockIdx.x;
  for (int w0 = 0; w0 < p.n; w0 += kCopyThreads) {
    const int2 mine = w0 + tid < p.n ? __ldcg(p.copies + w0 + tid) : make_int2(-1, -1);
    const uint32_t live = __ballot_sync(0xFFFFFFFFu, mine.x >= 0);
    __syncthreads();  // the window before has been read
    if ((tid & 31) == 0) s_live[tid >> 5] = __popc(live);
    __syncthreads();
    int at = __popc(live & ((1u << (tid & 31)) - 1u)), n = 0;
    for (int i = 0; i < kCopyThreads / 32; ++i) {
      if (i < tid >> 5) at += s_live[i];
      n += s_live[i];
    }
    if (mine.x >= 0) s_pair[at] = mine;
    __syncthreads();
    const uint64_t all = (uint64_t)n * p.n_tensors * items;
    const uint32_t per_pair = p.n_tensors * items;  // below 2^31
    for (; turn < all; turn += gridDim.x) {
      const uint32_t pair = turn >> 32 ? (uint32_t)(turn / per_pair) : (uint32_t)turn / per_pair;
      const uint32_t rest = (uint32_t)(turn - (uint64_t)pair * per_pair);
      const uint32_t ti = rest / items;
      const CopyTensor& t = p.t[ti];
      const int2 c = s_pair[pair];
      if (c.x >= p.n_pages[ti] || (unsigned)c.y >= (unsigned)p.n_pages[ti]) {
        if (tid == 0) set_status(p.status[ti], MOE_KV_BAD_PAGE);
        continue;
      }
      const W* src = reinterpret_cast<const W*>(t.base) + c.x * t.page_stride;
      W* dst = reinterpret_cast<W*>(t.base) + c.y * t.page_stride;
      W v[kCopyUnroll];
      int64_t off[kCopyUnroll];
#pragma unroll
      for (int k = 0; k < kCopyUnroll; ++k) {
        const uint32_t w = (rest % items) * kCopyItem + k * kCopyThreads + tid;
        off[k] = -1;
        if (w < t.words) {
          off[k] = w;
          if (t.units != t.words) {  // a page in several runs
            const uint32_t run = w / t.units, i2 = run % t.n2, i1 = run / t.n2;
            off[k] = i1 * t.s1 + i2 * t.s2 + (w - run * t.units);
          }
          v[k] = src[off[k]];
        }
      }
#pragma unroll
      for (int k = 0; k < kCopyUnroll; ++k)
        if (off[k] >= 0) dst[off[k]] = v[k];
    }
    turn -= all;  // where this block goes on in the next window
  }
}

moe_status_t check_pool(const moe_page_pool_t* p, const char* call) {
  if (!p) return decode_fail(MOE_ERR_INVALID_ARG, "%s: pool is NULL", call);
  if (p->n_seqs < 0 || p->max_pages < 0 || p->n_pages < 0 || p->page_size < 1)
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: negative size, or page_size below 1", call);
  if (p->n_seqs > MOE_POOL_MAX_SEQS || (int64_t)p->max_pages * p->page_size > 0x7fff0000ll ||
      (int64_t)p->n_seqs * p->max_pages > 0x40000000ll || p->n_pages > 0x40000000)
    return decode_fail(MOE_ERR_UNSUPPORTED, "%s: more than %d requests, 2^31 tokens a request or 2^30 pages", call,
                       MOE_POOL_MAX_SEQS);
  if (!aligned_to(p->block_table, 4) || !aligned_to(p->seq_lens, 4) || !aligned_to(p->page_refs, 4) ||
      !aligned_to(p->status, 4))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: the tables must be 4-byte aligned", call);
  if (p->n_seqs > 0 && (!p->seq_lens || (p->max_pages > 0 && !p->block_table)))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: block_table or seq_lens is NULL", call);
  if (p->n_pages > 0 && !p->page_refs) return decode_fail(MOE_ERR_INVALID_ARG, "%s: page_refs is NULL", call);
  return MOE_OK;
}

moe_status_t launched(cudaError_t e, const char* call) {
  return e == cudaSuccess ? MOE_OK : decode_fail(MOE_ERR_CUDA, "%s: %s", call, cudaGetErrorString(e));
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_pages_fork(const moe_page_pool_t* pool, const int32_t* src, const int32_t* dst, int32_t n,
                                       moe_stream_t stream) {
  const char* call = "moe_pages_fork";
  moe_status_t st = check_pool(pool, call);
  if (st != MOE_OK) return st;
  if (n < 0 || n > pool->n_seqs) return decode_fail(MOE_ERR_INVALID_ARG, "%s: n = %d outside [0, n_seqs]", call, n);
  if (!aligned_to(src, 4) || !aligned_to(dst, 4))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: src and dst must be 4-byte aligned", call);
  if (n == 0) return MOE_OK;
  if (!src || !dst) return decode_fail(MOE_ERR_INVALID_ARG, "%s: src or dst is NULL", call);
  st = check_device(nullptr);
  if (st != MOE_OK) return st;
  return launched(launch_cluster(pages_fork_kernel, reinterpret_cast<cudaStream_t>(stream), *pool, src, dst, n), call);
}

extern "C" moe_status_t moe_pages_resize(const moe_page_pool_t* pool, const int32_t* new_lens, int32_t* copies,
                                         moe_stream_t stream) {
  const char* call = "moe_pages_resize";
  moe_status_t st = check_pool(pool, call);
  if (st != MOE_OK) return st;
  if (!aligned_to(new_lens, 4) || !aligned_to(copies, 8))
    return decode_fail(MOE_ERR_INVALID_ARG, "%s: new_lens must be 4-byte aligned, copies 8-byte", call);
  if (pool->n_seqs == 0) return MOE_OK;
  if (!new_lens || !copies) return decode_fail(MOE_ERR_INVALID_ARG, "%s: new_lens or copies is NULL", call);
  st = check_device(nullptr);
  if (st != MOE_OK) return st;
  return launched(launch_cluster(pages_resize_kernel, reinterpret_cast<cudaStream_t>(stream), *pool, new_lens,
                                 reinterpret_cast<int2*>(copies)), call);
}

extern "C" moe_status_t moe_pages_compact(const moe_page_pool_t* pool, int32_t* copies, int32_t capacity, moe_stream_t stream) {
  const char* call = "moe_pages_compact";
  moe_status_t st = check_pool(pool, call);
  if (st != MOE_OK) return st;
  if (capacity < 0) return decode_fail(MOE_ERR_INVALID_ARG, "%s: capacity = %d is negative", call, capacity);
  if (!aligned_to(copies, 8)) return decode_fail(MOE_ERR_INVALID_ARG, "%s: copies must be 8-byte aligned", call);
  if (capacity == 0) return MOE_OK;
  if (!copies) return decode_fail(MOE_ERR_INVALID_ARG, "%s: copies is NULL", call);
  st = check_device(nullptr);
  if (st != MOE_OK) return st;
  return launched(launch_cluster(pages_compact_kernel, reinterpret_cast<cudaStream_t>(stream), *pool,
                                 reinterpret_cast<int2*>(copies), capacity), call);
}

extern "C" moe_status_t moe_copy_pages(const moe_kv_cache_t* const* caches, int32_t n_caches, const int32_t* copies, int32_t n,
                                       moe_stream_t stream) {
  const char* call = "moe_copy_pages";
  if (n_caches < 0 || n < 0) return decode_fail(MOE_ERR_INVALID_ARG, "%s: a negative number of caches or copies", call);
  if (n_caches > 0 && !caches) return decode_fail(MOE_ERR_INVALID_ARG, "%s: caches is NULL", call);
  if (!aligned_to(copies, 8)) return decode_fail(MOE_ERR_INVALID_ARG, "%s: copies must be 8-byte aligned", call);
  for (int i = 0; i < n_caches; ++i) {
    const moe_status_t st = check_cache(caches[i], call);
    if (st != MOE_OK) return st;
    if (caches[i]->n_pages > 0 && (!caches[i]->k || !caches[i]->v ||
                                   (caches[i]->format != MOE_KV_BF16 && (!caches[i]->k_s || !caches[i]->v_s))))
      return decode_fail(MOE_ERR_INVALID_ARG, "%s: a page buffer is NULL", call);
  }
  if (n == 0 || n_caches == 0) return MOE_OK;
  if (!copies) return decode_fail(MOE_ERR_INVALID_ARG, "%s: copies is NULL", call);
  int sms = 0;
  moe_status_t st = check_device(&sms);
  if (st != MOE_OK) return st;

  // Tensors by the width of the words that their runs, strides and base allow; a launch takes kCopyTensors of one width.
  static constexpr int kWidths[] = {16, 4, 2};
  CopyParams p[3];
  for (auto& x : p) x.n_tensors = 0, x.copies = reinterpret_cast<const int2*>(copies), x.n = n;
  auto launch = [&](int w) {
    CopyParams& x = p[w];
    if (x.n_tensors == 0) return cudaSuccess;
    uint64_t words = 0;
    for (int i = 0; i < x.n_tensors; ++i) words = std::max<uint64_t>(words, x.t[i].words);
    const uint64_t items = (words + kCopyItem - 1) / kCopyItem * x.n_tensors * n;
    const dim3 grid((unsigned)std::min<uint64_t>(items, (uint64_t)sms * 8));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = w == 0   ? launch_pdl(copy_pages_kernel<uint4>, grid, dim3(kCopyThreads), 0, s, x)
                          : w == 1 ? launch_pdl(copy_pages_kernel<uint32_t>, grid, dim3(kCopyThreads), 0, s, x)
                                   : launch_pdl(copy_pages_kernel<uint16_t>, grid, dim3(kCopyThreads), 0, s, x);
    x.n_tensors = 0;
    return e;
  };
  for (int i = 0; i < n_caches; ++i) {
    const moe_kv_cache_t& c = *caches[i];
    if (c.n_pages == 0) continue;
    for (int j = 0; j < (c.format == MOE_KV_BF16 ? 2 : 4); ++j) {
      // bytes: elements times num / den
      const int num = j < 2 && c.format == MOE_KV_BF16 ? 2 : 1, den = j >= 2 ? 32 : c.format == MOE_KV_MXFP4 ? 2 : 1;
      auto bytes = [&](int64_t elements) { return elements * num / den; };
      uint8_t* base = static_cast<uint8_t*>(j == 0 ? c.k : j == 1 ? c.v : j == 2 ? static_cast<void*>(c.k_s) : c.v_s);
      int64_t run = bytes(c.head_dim), n1 = c.page_size, s1 = bytes(c.row_stride), n2 = c.n_kv_heads, s2 = bytes(c.head_stride);
      if (n1 == 1) s1 = 0;
      if (n2 == 1) s2 = 0;
      if (n1 > 1 && (n2 == 1 || s1 < s2)) std::swap(n1, n2), std::swap(s1, s2);  // the shorter stride inside
      if (n2 > 1 && s2 == run) run *= n2, n2 = 1, s2 = 0;
      if (n2 == 1 && n1 > 1 && s1 == run) run *= n1, n1 = 1, s1 = 0;
      int w = 0;
      auto fits = [&](int64_t width) {
        return !(run % width || s1 % width || s2 % width || bytes(c.page_stride) % width || !aligned_to(base, width));
      };
      while (w < 2 && !fits(kWidths[w])) ++w;
      if (run / kWidths[w] * n1 * n2 > 0x3FFFFFFFll) return decode_fail(MOE_ERR_UNSUPPORTED, "%s: a page of 2^30 words", call);
      CopyParams& x = p[w];
      const int width = kWidths[w], k = x.n_tensors++;
      x.t[k] = {base, bytes(c.page_stride) / width, s1 / width, s2 / width, (uint32_t)n2, (uint32_t)(run / width),
                (uint32_t)(run / width * n1 * n2)};
      x.status[k] = c.status;
      x.n_pages[k] = c.n_pages;
      if (x.n_tensors == kCopyTensors) {
        const cudaError_t e = launch(w);
        if (e != cudaSuccess) return launched(e, call);
      }
    }
  }
  for (int w = 0; w < 3; ++w) {
    const cudaError_t e = launch(w);
    if (e != cudaSuccess) return launched(e, call);
  }
  return MOE_OK;
}
