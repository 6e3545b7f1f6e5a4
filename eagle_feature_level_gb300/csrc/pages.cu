// The pages of a paged cache: fork, reserve with copy on write, release,
// compact.  The reference counts are the only allocator state; a block with
// count 0 is free and the lowest free ids go first, in sequence order, so the
// tables after a call follow from the tables before it alone.
//
// reserve and compact are two launches: a plan by one CTA over the tables and
// counts (a few thousand integers: latency), which writes a list of block
// copies, and the copy of those blocks in every layer's K and V pools by the
// whole GPU (bandwidth: each byte read once, written once).  A plan takes 12 us
// for 16384 blocks; the copy of 1.07 GB of moving blocks 335 us, 6.4 TB/s, 0.94
// of a measured copy.
#include <algorithm>

#include "internal.h"
#include "common.cuh"

namespace eagle {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int CP_THREADS = 256;
constexpr int CP_PER = 4;                    // 16-byte pieces a thread has in flight
constexpr int CP_CHUNK = CP_THREADS * CP_PER * 16;
constexpr int CP_PER_SM = 8;

// The page calls' part of the workspace: counts, then PAGES_LISTS lists of
// one int per sequence.
struct PageLists {
  int* n_copies;
  int* first;        // rank of the sequence's first block among those taken
  int* tail;         // block to copy, -1: none
  int* src;          // the copies: block, to block, rows
  int* dst;
  int* rows;
};

struct PagesParams {
  int32_t* table;
  int32_t* len;
  int32_t* ref;
  int32_t* scratch;
  int n_seqs, per, shift, n_blocks;
  PageLists l;
  int* status;
  uint64_t* stamp;

  __device__ int held(int s) const { return min(blocks(len[s]), per); }
  __device__ int blocks(long long rows) const { return static_cast<int>((rows + (1 << shift) - 1) >> shift); }
  __device__ int32_t* row(int s) const { return table + static_cast<size_t>(s) * per; }
  __device__ bool valid(int blk) const { return blk >= 0 && blk < n_blocks; }
};

// Exclusive prefix sums over the CTA's threads, in thread order; `total` is
// the CTA's sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s_warp, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  const T w = lane < nw ? s_warp[lane] : 0;
  T c = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += y;
  }
  total = __shfl_sync(0xffffffffu, c, 31);
  const T before = __shfl_sync(0xffffffffu, c - w, warp);
  return before + x - v;
}

// The counts of blocks b .. b + 3 (b a multiple of 4), 0 past the last block.
__device__ __forceinline__ int4 counts4(const PagesParams& p, int b) {
  if (b + 4 <= p.n_blocks) return *reinterpret_cast<const int4*>(p.ref + b);
  int4 c = make_int4(0, 0, 0, 0);
  if (b < p.n_blocks) c.x = p.ref[b];
  if (b + 1 < p.n_blocks) c.y = p.ref[b + 1];
  if (b + 2 < p.n_blocks) c.z = p.ref[b + 2];
  return c;
}

// ---- fork -------------------------------------------------------------------

// One CTA per (pair, run of columns).  A pair's standing -- in range, its
// destination no pair's source and no earlier pair's destination -- is decided
// alike by all its CTAs from the lists, which nothing writes.
__global__ void __launch_bounds__(CP_THREADS) fork_kernel(const PagesParams p, int n, const int32_t* src,
                                                          const int32_t* dst) {
  const LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int i = blockIdx.x;
  const int s = src[i], d = dst[i];
  bool bad = s < 0 || s >= p.n_seqs || d < 0 || d >= p.n_seqs;
  for (int j = threadIdx.x; j < n; j += CP_THREADS) bad = bad || src[j] == d || (j < i && dst[j] == d);
  if (__syncthreads_or(bad)) {
    if (blockIdx.y == 0 && threadIdx.x == 0) set_status(p.status, EAGLE_ERR_INVALID_ARG);
    return;
  }
  const int L = p.len[s], held = p.held(s);
  for (int c = blockIdx.y * CP_THREADS + threadIdx.x; c < p.per; c += gridDim.y * CP_THREADS) {
    const int old = p.row(d)[c];
    const int now = c < held ? p.row(s)[c] : -1;
    if (p.valid(now)) atomicAdd(&p.ref[now], 1);
    if (p.valid(old)) atomicSub(&p.ref[old], 1);
    p.row(d)[c] = now;
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) p.len[d] = L;
}

// ---- release ----------------------------------------------------------------

__global__ void __launch_bounds__(CP_THREADS) release_kernel(const PagesParams p, const int32_t* keep) {
  const LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int s = blockIdx.x;
  const int k = keep[s];
  if (k < 0) return;
  for (int c = min(p.blocks(k), p.per) + blockIdx.y * CP_THREADS + threadIdx.x; c < p.per; c += gridDim.y * CP_THREADS) {
    const int old = p.row(s)[c];
    if (old >= 0) p.row(s)[c] = -1;
    if (p.valid(old)) atomicSub(&p.ref[old], 1);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0 && p.len[s] > k) p.len[s] = k;
}

// ---- reserve: the plan --------------------------------------------------------

// The block that sequence s would write into its middle: its partly filled
// last one (-1: none, or no rows to add).
__device__ __forceinline__ int tail_block(const PagesParams& p, int s, int add) {
  const int L = p.len[s];
  if (add <= 0 || L <= 0 || (L & ((1 << p.shift) - 1)) == 0 || (L >> p.shift) >= p.per) return -1;
  const int blk = p.row(s)[L >> p.shift];
  return p.valid(blk) ? blk : -1;
}

// The columns [c0, c1) of sequence s without a block: counted, and (`fill`)
// given the blocks ids[at], ids[at + 1], .. in column order.  Every lane of
// a warp calls it for a sequence of its own; a lane with few columns walks
// them alone, the warp takes longer runs (a prompt's) together.
__device__ __forceinline__ int missing_blocks(const PagesParams& p, int s, int c0, int c1, bool fill, int at,
                                              const int32_t* ids) {
  constexpr int ALONE = 8;
  const int lane = threadIdx.x & 31;
  int n = 0;
  if (c1 - c0 <= ALONE) {
    for (int c = c0; c < c1; ++c)
      if (!p.valid(p.row(s)[c])) {
        if (fill) {
          const int blk = ids[at + n];
          p.row(s)[c] = blk;
          p.ref[blk] = 1;
        }
        ++n;
      }
  }
  for (unsigned todo = __ballot_sync(0xffffffffu, c1 - c0 > ALONE); todo; todo &= todo - 1) {
    const int l = __ffs(todo) - 1;
    const int ss = __shfl_sync(0xffffffffu, s, l), a = __shfl_sync(0xffffffffu, c0, l);
    const int z = __shfl_sync(0xffffffffu, c1, l), from = __shfl_sync(0xffffffffu, at, l);
    int m = 0;
    for (int c = a; c < z; c += 32) {
      const bool none = c + lane < z && !p.valid(p.row(ss)[c + lane]);
      const unsigned who = __ballot_sync(0xffffffffu, none);
      if (fill && none) {
        const int blk = ids[from + m + __popc(who & ((1u << lane) - 1u))];
        p.row(ss)[c + lane] = blk;
        p.ref[blk] = 1;
      }
      m += __popc(who);
    }
    if (lane == l) n = m;
  }
  return n;
}

__global__ void __launch_bounds__(PLAN_THREADS) reserve_kernel(const PagesParams p, const int32_t* n_new) {
  const LaunchStamp ls(p.stamp);
  __shared__ int s_warp[32];
  __shared__ long long s_warp64[32];
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int tid = threadIdx.x;
  int* writers = p.scratch;                  // by block: sequences that would write it, ...
  int* last = p.scratch + p.n_blocks;        // ... and the highest of them
  for (int s = tid; s < p.n_seqs; s += PLAN_THREADS) {
    const int t = tail_block(p, s, n_new[s]);
    if (t >= 0) {
      writers[t] = 0;
      last[t] = -1;
    }
  }
  __syncthreads();
  for (int s = tid; s < p.n_seqs; s += PLAN_THREADS) {
    const int t = tail_block(p, s, n_new[s]);
    if (t >= 0) {
      atomicAdd(&writers[t], 1);
      atomicMax(&last[t], s);
    }
  }
  __syncthreads();
  // what each sequence takes: its new blocks, and one for a copied tail
  long long need = 0;
  int copies = 0;
  bool fits = true;
  for (int s0 = 0; s0 < p.n_seqs; s0 += PLAN_THREADS) {
    const int s = s0 + tid;
    int copy = 0, c0 = 0, c1 = 0;
    if (s < p.n_seqs) {
      const int add = n_new[s], L = p.len[s];
      int t = -1;
      if (add > 0) {
        const long long rows = static_cast<long long>(L) + add;
        const bool ok = L >= 0 && rows <= (static_cast<long long>(p.per) << p.shift);
        fits = fits && ok;
        t = tail_block(p, s, add);
        copy = t >= 0 && p.ref[t] > 1 && !(writers[t] >= p.ref[t] && last[t] == s);
        if (ok) {
          c0 = p.blocks(L);
          c1 = p.blocks(rows);
        }
      }
      p.l.tail[s] = copy ? t : -1;
    }
    // blocks already there (reserved ahead) are kept
    const int take = copy + missing_blocks(p, s, c0, c1, false, 0, nullptr);
    long long total;
    int n;
    const long long first = block_scan(static_cast<long long>(take), s_warp64, total);
    const int at = block_scan(copy, s_warp, n);
    if (s < p.n_seqs) {
      p.l.first[s] = static_cast<int>(min(need + first, static_cast<long long>(p.n_blocks)));
      if (copy) {
        p.l.src[copies + at] = p.l.tail[s];
        p.l.rows[copies + at] = p.len[s] & ((1 << p.shift) - 1);
        p.l.dst[copies + at] = s;            // the sequence, until its block is known
      }
    }
    need += total;
    copies += n;
  }
  fits = __syncthreads_and(fits);
  // the `need` lowest free blocks, in order (the marks above are done with)
  int found = 0;
  for (int b0 = 0; fits && found < need && b0 < p.n_blocks; b0 += 4 * PLAN_THREADS) {
    const int b = b0 + 4 * tid;
    const int4 c = counts4(p, b);
    const int count[4] = {c.x, c.y, c.z, c.w};
    int free[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      free[i] = b + i < p.n_blocks && count[i] == 0;
      n += free[i];
    }
    int total;
    int at = found + block_scan(n, s_warp, total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (free[i]) {
        if (at < need) p.scratch[at] = b + i;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  if (!fits || found < need) {
    if (tid == 0) {
      *p.l.n_copies = 0;
      set_status(p.status, EAGLE_ERR_CAPACITY);
    }
    return;
  }
  for (int s0 = 0; s0 < p.n_seqs; s0 += PLAN_THREADS) {
    const int s = s0 + tid;
    const int add = s < p.n_seqs ? n_new[s] : 0;
    int at = 0, c0 = 0, c1 = 0;
    if (add > 0) {
      const int L = p.len[s], t = p.l.tail[s];
      at = p.l.first[s];
      if (t >= 0) {
        const int blk = p.scratch[at++];
        p.row(s)[L >> p.shift] = blk;
        p.ref[blk] = 1;
        atomicSub(&p.ref[t], 1);
      }
      c0 = p.blocks(L);
      c1 = p.blocks(static_cast<long long>(L) + add);
    }
    missing_blocks(p, s, c0, c1, true, at, p.scratch);
  }
  __syncthreads();
  for (int i = tid; i < copies; i += PLAN_THREADS) {
    const int s = p.l.dst[i];
    p.l.dst[i] = p.row(s)[p.len[s] >> p.shift];
  }
  if (tid == 0) *p.l.n_copies = copies;
}

// ---- compact: the plan --------------------------------------------------------

// scratch: the moving blocks by rank, from n_blocks / 2 on their places, and
// from n_blocks on the rank of each id from the live count on (-1: not live).
__global__ void __launch_bounds__(PLAN_THREADS) compact_kernel(const PagesParams p) {
  const LaunchStamp ls(p.stamp);
  __shared__ int s_warp[32];
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int tid = threadIdx.x;
  int live = 0;
  for (int b = 4 * tid; b < p.n_blocks; b += 4 * PLAN_THREADS) {
    const int4 c = counts4(p, b);
    live += (c.x > 0) + (c.y > 0) + (c.z > 0) + (c.w > 0);
  }
  int used;
  block_scan(live, s_warp, used);
  int* src = p.scratch;
  int* dst = p.scratch + p.n_blocks / 2;
  int* to = p.scratch + p.n_blocks;
  int movers = 0, holes = 0;
  for (int b0 = 0; b0 < p.n_blocks; b0 += 4 * PLAN_THREADS) {
    const int b = b0 + 4 * tid;
    const int4 c = counts4(p, b);
    const int count[4] = {c.x, c.y, c.z, c.w};
    int n = 0;                               // of these four ids: movers, and holes 16 bits up
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i < p.n_blocks) n += count[i] > 0 ? (b + i >= used ? 1 : 0) : (b + i < used ? 1 << 16 : 0);
    int total;
    int at = block_scan(n, s_warp, total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i < p.n_blocks) {
        if (b + i >= used) {
          const int rank = movers + (at & 0xffff);
          to[b + i] = count[i] > 0 ? rank : -1;
          if (count[i] > 0) {
            src[rank] = b + i;
            ++at;
          }
        } else if (count[i] <= 0) {
          dst[holes + (at >> 16)] = b + i;
          at += 1 << 16;
        }
      }
    movers += total & 0xffff;
    holes += total >> 16;
  }
  if (tid == 0) {
    *p.l.n_copies = movers;
    p.l.n_copies[1] = used;
  }
}

// ---- the copies ---------------------------------------------------------------

struct CopyParams {
  PagesParams pg;
  const int* n_copies;     // (and, moving, the live count after it)
  const int32_t* src;
  const int32_t* dst;
  const int32_t* rows;     // rows of each copy, null: whole blocks
  int n_layers;
  long long block_elems;   // of one pool: rows x heads x head_dim
  int row_elems;
  int chunks;              // CP_CHUNK pieces of a block
  int move;                // the tables and counts follow (compact)
  uint16_t* k[EAGLE_MAX_LAYERS];
  uint16_t* v[EAGLE_MAX_LAYERS];
};

__global__ void __launch_bounds__(CP_THREADS) copy_kernel(const __grid_constant__ CopyParams p) {
  const LaunchStamp ls(p.pg.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (p.move) {
    const int used = p.n_copies[1];
    const int32_t* rank = p.pg.scratch + p.pg.n_blocks;
    const long long entries = static_cast<long long>(p.pg.n_seqs) * p.pg.per;
    for (long long i = static_cast<long long>(blockIdx.x) * CP_THREADS + tid; i < entries;
         i += static_cast<long long>(gridDim.x) * CP_THREADS) {
      const int blk = p.pg.table[i];
      if (blk >= used && blk < p.pg.n_blocks && rank[blk] >= 0) p.pg.table[i] = p.dst[rank[blk]];
    }
    for (int i = blockIdx.x * CP_THREADS + tid; i < *p.n_copies; i += gridDim.x * CP_THREADS) {
      p.pg.ref[p.dst[i]] = p.pg.ref[p.src[i]];
      p.pg.ref[p.src[i]] = 0;
    }
  }
  const long long per_copy = static_cast<long long>(p.n_layers) * 2 * p.chunks;
  const long long units = *p.n_copies * per_copy;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = static_cast<int>(u / per_copy);
    const int rest = static_cast<int>(u - i * per_copy);
    const int pool = rest / p.chunks, chunk = rest - pool * p.chunks;
    const long long bytes = (p.rows ? static_cast<long long>(p.rows[i]) * p.row_elems : p.block_elems) * 2;
    const long long lo = static_cast<long long>(chunk) * CP_CHUNK;
    if (lo >= bytes) continue;
    uint16_t* base = (pool & 1) ? p.v[pool >> 1] : p.k[pool >> 1];
    const char* from = reinterpret_cast<const char*>(base + p.src[i] * p.block_elems);
    char* to = reinterpret_cast<char*>(base + p.dst[i] * p.block_elems);
    uint4 w[CP_PER];
#pragma unroll
    for (int j = 0; j < CP_PER; ++j) {
      const long long at = lo + (j * CP_THREADS + tid) * 16;
      if (at < bytes) w[j] = *reinterpret_cast<const uint4*>(from + at);
    }
#pragma unroll
    for (int j = 0; j < CP_PER; ++j) {
      const long long at = lo + (j * CP_THREADS + tid) * 16;
      if (at < bytes) *reinterpret_cast<uint4*>(to + at) = w[j];
    }
  }
}

PagesParams pages_of(eagle_ctx* ctx, const eagle_pages& pg, void* ws) {
  PagesParams p{};
  p.table = pg.block_table;
  p.len = pg.len;
  p.ref = pg.ref;
  p.scratch = pg.scratch;
  p.n_seqs = pg.n_seqs;
  p.per = pg.per_seq;
  while ((1 << p.shift) < pg.block_size) ++p.shift;
  p.n_blocks = pg.n_blocks;
  int* base = ws_ptr<int>(ws, ctx->ws.pages);
  const int n = ctx->lim.max_batch;
  p.l = PageLists{base, base + 64, base + 64 + n, base + 64 + 2 * n, base + 64 + 3 * n, base + 64 + 4 * n};
  p.status = ws_ptr<int>(ws, ctx->ws.status);
  p.stamp = stamp_slot(ctx, EAGLE_K_PAGES);
  return p;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pages(eagle_ctx* ctx, void (*kernel)(KArgs...), dim3 grid, int threads, cudaStream_t st,
                         Args&&... args) {
  trace_before(ctx, EAGLE_K_PAGES, st);
  const cudaError_t e = launch_pdl(kernel, grid, dim3(threads), 0, st, std::forward<Args>(args)...);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_PAGES, st);
  return e;
}

cudaError_t launch_copies(eagle_ctx* ctx, const eagle_pages& pg, const eagle_pools& pools, bool move, void* ws,
                          cudaStream_t st) {
  CopyParams c{};
  c.pg = pages_of(ctx, pg, ws);
  c.n_copies = c.pg.l.n_copies;
  c.src = move ? pg.scratch : c.pg.l.src;
  c.dst = move ? pg.scratch + pg.n_blocks / 2 : c.pg.l.dst;
  c.rows = move ? nullptr : c.pg.l.rows;
  c.n_layers = pools.n_layers;
  c.row_elems = ctx->dims.n_kv_heads * ctx->dims.head_dim;
  c.block_elems = static_cast<long long>(pg.block_size) * c.row_elems;
  c.chunks = static_cast<int>((c.block_elems * 2 + CP_CHUNK - 1) / CP_CHUNK);
  c.move = move;
  for (int l = 0; l < pools.n_layers; ++l) {
    c.k[l] = pools.k[l];
    c.v[l] = pools.v[l];
  }
  return launch_pages(ctx, copy_kernel, dim3(ctx->sm_count * CP_PER_SM), CP_THREADS, st, c);
}

unsigned column_ctas(const eagle_pages& pg) {
  return static_cast<unsigned>(std::min(64, ceil_div(pg.per_seq, CP_THREADS)));
}

}  // namespace

cudaError_t launch_pages_fork(eagle_ctx* ctx, const eagle_pages& pg, int n, const int32_t* src, const int32_t* dst,
                              void* ws, cudaStream_t st) {
  return launch_pages(ctx, fork_kernel, dim3(n, column_ctas(pg)), CP_THREADS, st, pages_of(ctx, pg, ws), n, src, dst);
}

cudaError_t launch_pages_release(eagle_ctx* ctx, const eagle_pages& pg, const int32_t* keep, void* ws,
                                 cudaStream_t st) {
  return launch_pages(ctx, release_kernel, dim3(pg.n_seqs, column_ctas(pg)), CP_THREADS, st, pages_of(ctx, pg, ws),
                      keep);
}

cudaError_t launch_pages_reserve(eagle_ctx* ctx, const eagle_pages& pg, const eagle_pools& pools, const int32_t* n_new,
                                 void* ws, cudaStream_t st) {
  const cudaError_t e = launch_pages(ctx, reserve_kernel, dim3(1), PLAN_THREADS, st, pages_of(ctx, pg, ws), n_new);
  if (e != cudaSuccess || pools.n_layers == 0) return e;
  return launch_copies(ctx, pg, pools, false, ws, st);
}

cudaError_t launch_pages_compact(eagle_ctx* ctx, const eagle_pages& pg, const eagle_pools& pools, void* ws,
                                 cudaStream_t st) {
  const cudaError_t e = launch_pages(ctx, compact_kernel, dim3(1), PLAN_THREADS, st, pages_of(ctx, pg, ws));
  if (e != cudaSuccess) return e;
  return launch_copies(ctx, pg, pools, true, ws, st);
}

}  // namespace eagle
