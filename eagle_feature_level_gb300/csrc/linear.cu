// eagle_mx_linear: y = x w^T (+ bias) of matrices in one microscaled format, on the block-scaled tensor-core
// instructions, which take both operands' scales from tensor memory.
//
// The weights are operand A (128 outputs a tile), the rows x operand B (up to 192 a tile, few for single tokens), so one
// kernel serves decoding and prompts: an accumulator holds [128 outputs][rows] and a lane stores its output's column,
// 32 neighbours a warp.  A stage of the ring holds 128 bytes of every row of both (256 four-bit or 128 eight-bit
// elements, 4 MMAs) and their scales, which lie in memory as the 512-byte groups that one tcgen05.cp spreads over tensor
// memory.  Warp roles: TMA producer, MMA issuer, four warps that read the accumulator out; two accumulators, so that
// a tile is read out under the next one's products.
//
// Few tiles: a cluster of CTAs splits a tile's inner dimension; each writes its partial to its own shared memory and
// sums its share of the rows over all of them, in rank order.
#include <algorithm>

#include "internal.h"
#include "common.cuh"
#include "mx.cuh"
#include "sm100.cuh"

namespace eagle {
namespace {

constexpr int LN_THREADS = 192;
constexpr int LN_M = 128;                     // outputs of a tile
constexpr int LN_KB = 128;                    // bytes of a row in a stage
constexpr int LN_MAX_STAGES = 12;
constexpr int LN_A_BYTES = LN_M * LN_KB;
constexpr size_t LN_SMEM = 226 * 1024;     // dynamic: 227 KB less the barriers

struct LinearParams {
  const uint8_t* w_scale;
  const uint8_t* x_scale;
  const float* gw;
  const float* gx;
  const float* bias;
  void* y;
  long long ld_y;
  int f32;
  int rows, outs;
  int kbytes;              // of a row
  int groups;              // 4-scale groups of a row
  int nt;                  // rows of a tile
  int row_tiles, tiles;
  int row_blocks;          // of 128 rows: scales of x
  int rb;                  // 128-row blocks that a tile's scales take at most
  int steps;               // stages of the inner dimension
  int split;               // CTAs of a cluster
  int stages;
  uint32_t stage_bytes, b_bytes;
  uint32_t acc_cols, sf_at, sf_cols, tmem_cols;
  int once;                // weights are read once
  int* status;
  uint64_t* stamp;
};

struct LinearShared {
  uint64_t full[LN_MAX_STAGES], empty[LN_MAX_STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t part_full, part_free;
  uint64_t drained;
  uint32_t tmem;
  int abort, never;
  int issued;              // stages that the producer has asked for
};

template <int FMT>
constexpr int groups_per_stage() { return FMT == EAGLE_MX_FP8 ? 1 : FMT == EAGLE_MX_FP4 ? 2 : 4; }

// Instruction descriptor of the block-scaled kinds: element types at bits 7 and 10 (e4m3 0, e2m1 1), N / 8 at 17, the
// scales' type at 23 (e4m3 0, power of two 1), M / 16 at 24, and which bytes of a 32-bit column of scales the
// instruction takes, at 4 for B and 29 for A.
template <int FMT>
__device__ __forceinline__ uint32_t idesc_of(int n, int sf) {
  const uint32_t type = FMT == EAGLE_MX_FP8 ? 0u : 1u;
  const uint32_t scale = FMT == EAGLE_NV_FP4 ? 0u : 1u;
  return (static_cast<uint32_t>(sf) << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (scale << 23) | (static_cast<uint32_t>(LN_M >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);
}

template <int FMT>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t acc) {
  if (FMT == EAGLE_MX_FP8)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else if (FMT == EAGLE_MX_FP4)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// 512 bytes of scales to four columns, repeated in each quarter of the lanes.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t saddr) {
  // 32 rows of 16 bytes without swizzle: 8-row groups 128 bytes apart
  const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128u >> 4) << 32) |
                        (static_cast<uint64_t>(1u) << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   sm100::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
// Arrive on the twin of `bar` in CTA `rank` of the cluster; what this thread has written (or read) before comes before.
__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(sm100::dsmem_addr(bar, rank))
               : "memory");
}
// mbar_wait for arrivals from the whole cluster.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint64_t t0 = 0;
  uint32_t spins = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, "
        "p;\n}\n"
        : "=r"(ok)
        : "r"(sm100::smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((++spins & 63u) == 0) {
      if (*abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > WAIT_LIMIT_NS) return false;
    }
  }
}

// A tile's place: its weight rows, its rows of x and their first block of scales.
struct TileAt {
  int out0, row0, rb0, n_rb;
};
__device__ __forceinline__ TileAt tile_at(const LinearParams& p, int tile) {
  TileAt t;
  const int m = tile / p.row_tiles;
  t.out0 = m * LN_M;
  t.row0 = (tile - m * p.row_tiles) * p.nt;
  t.rb0 = t.row0 >> 7;
  const int last = min((t.row0 + p.nt - 1) >> 7, p.row_blocks - 1);
  t.n_rb = last - t.rb0 + 1;
  return t;
}

template <int FMT>
__device__ __forceinline__ void produce(const LinearParams& p, LinearShared& sh, uint8_t* ring, const CUtensorMap* wm,
                                        const CUtensorMap* xm, int first, int step, int k0, int k1,
                                        volatile int* abort) {
  constexpr int GPS = groups_per_stage<FMT>();
  const uint64_t policy = sm100::l2_policy_evict_first();
  int slot = 0;
  uint32_t phase = 1;
  for (int tile = first; tile < p.tiles; tile += step) {
    const TileAt at = tile_at(p, tile);
    const uint8_t* sa = p.w_scale + static_cast<size_t>(at.out0 >> 7) * p.groups * 512;
    const uint8_t* sb = p.x_scale + static_cast<size_t>(at.rb0) * p.groups * 512;
    for (int k = k0; k < k1; ++k) {
      if (!sm100::mbar_wait(&sh.empty[slot], phase, abort)) {
        *abort = 1;
        return;
      }
      ++sh.issued;
      uint8_t* st = ring + static_cast<size_t>(slot) * p.stage_bytes;
      uint64_t* bar = &sh.full[slot];
      const uint32_t sf = static_cast<uint32_t>(min(GPS, p.groups - k * GPS)) * 512u;
      sm100::mbar_arrive_expect_tx(bar, LN_A_BYTES + p.b_bytes + sf * static_cast<uint32_t>(1 + at.n_rb));
      if (p.once) sm100::tma_load_2d_hint(st, wm, k * LN_KB, at.out0, bar, policy);
      else sm100::tma_load_2d(st, wm, k * LN_KB, at.out0, bar);
      sm100::tma_load_2d(st + LN_A_BYTES, xm, k * LN_KB, at.row0, bar);
      uint8_t* s = st + LN_A_BYTES + p.b_bytes;
      bulk_load(s, sa + static_cast<size_t>(k) * GPS * 512, sf, bar);
      for (int b = 0; b < at.n_rb; ++b)
        bulk_load(s + (1 + b) * GPS * 512, sb + (static_cast<size_t>(b) * p.groups + static_cast<size_t>(k) * GPS) * 512,
                  sf, bar);
      if (++slot == p.stages) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
}

template <int FMT>
__device__ __forceinline__ void multiply(const LinearParams& p, LinearShared& sh, uint8_t* ring, uint32_t tmem,
                                         int first, int step, int k0, int k1, volatile int* abort) {
  constexpr int GPS = groups_per_stage<FMT>();
  int slot = 0, n = 0, sf_slot = 0;
  uint32_t phase = 0;
  for (int tile = first; tile < p.tiles; tile += step, ++n) {
    const int buf = n & 1;
    const uint32_t b_off = static_cast<uint32_t>((tile % p.row_tiles) * p.nt & 127) >> 5;
    if (!sm100::mbar_wait(&sh.acc_empty[buf], ((n >> 1) & 1) ^ 1, abort)) {
      *abort = 1;
      return;
    }
    sm100::tc_fence_after();
    const uint32_t d = tmem + static_cast<uint32_t>(buf) * p.acc_cols;
    uint32_t acc = 0;
    for (int k = k0; k < k1; ++k) {
      if (!sm100::mbar_wait(&sh.full[slot], phase, abort)) {
        *abort = 1;
        return;
      }
      sm100::tc_fence_after();
      const uint32_t st = sm100::smem_u32(ring + static_cast<size_t>(slot) * p.stage_bytes);
      const uint32_t s = st + LN_A_BYTES + p.b_bytes;
      const uint32_t sfa = tmem + p.sf_at + static_cast<uint32_t>(sf_slot) * p.sf_cols;
      const uint32_t sfb = sfa + 4 * GPS;
#pragma unroll
      for (int g = 0; g < GPS; ++g) copy_scales(sfa + 4 * g, s + 512 * g);
      for (int b = 0; b < p.rb; ++b)
#pragma unroll
        for (int g = 0; g < GPS; ++g)
          copy_scales(sfb + 4 * (g * p.rb + b), s + 512 * ((1 + b) * GPS + g));
      const uint64_t ad = sm100::smem_desc_sw128(st), bd = sm100::smem_desc_sw128(st + LN_A_BYTES);
      const int left = p.kbytes - k * LN_KB;           // bytes: 32 an MMA
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > 0 && 32 * j >= left) break;
        const int g = FMT == EAGLE_MX_FP8 ? 0 : FMT == EAGLE_MX_FP4 ? j / 2 : j;
        const int sf = FMT == EAGLE_MX_FP8 ? j : FMT == EAGLE_MX_FP4 ? 2 * (j & 1) : 0;
        mma_scaled<FMT>(d, ad + 2 * j, bd + 2 * j, idesc_of<FMT>(p.nt, sf), sfa + 4 * g,
                        sfb + 4 * g * p.rb + b_off, acc);
        acc = 1;
      }
      sm100::mma_commit(&sh.empty[slot]);
      sf_slot ^= 1;
      if (++slot == p.stages) {
        slot = 0;
        phase ^= 1;
      }
    }
    sm100::mma_commit(&sh.acc_full[buf]);
  }
}

__device__ __forceinline__ void put(const LinearParams& p, long long at, float v) {
  if (p.f32) static_cast<float*>(p.y)[at] = v;
  else static_cast<uint16_t*>(p.y)[at] = f32_to_bf16(v);
}

__device__ __forceinline__ void read_out(const LinearParams& p, LinearShared& sh, float* part, uint32_t tmem, int first,
                                         int step, uint32_t rank, volatile int* abort) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
  const float scale = (p.gw ? *p.gw : 1.0f) * (p.gx ? *p.gx : 1.0f);
  const int mine = quarter * 32 + lane;
  int n = 0;
  for (int tile = first; tile < p.tiles; tile += step, ++n) {
    const TileAt at = tile_at(p, tile);
    const int buf = n & 1, out = at.out0 + mine;
    const bool in = out < p.outs;
    const float bias = p.bias && in ? p.bias[out] : 0.0f;
    const int rows = min(p.nt, p.rows - at.row0);
    if (!__all_sync(0xffffffffu, sm100::mbar_wait(&sh.acc_full[buf], (n >> 1) & 1, abort))) {
      *abort = 1;
      return;
    }
    sm100::tc_fence_after();
    const uint32_t d = tmem + static_cast<uint32_t>(buf) * p.acc_cols + (static_cast<uint32_t>(quarter * 32) << 16);
    if (p.split > 1 && n > 0 &&
        !__all_sync(0xffffffffu, wait_cluster(&sh.part_free, (n - 1) & 1, abort))) {
      *abort = 1;
      return;
    }
    for (int c = 0; c < rows; c += 16) {
      float v[16];
      sm100::tmem_ld16(d + c, v);
      sm100::tmem_wait_ld();
      if (p.split == 1) {
        const long long y0 = static_cast<long long>(at.row0 + c) * p.ld_y + out;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (in && c + i < rows) put(p, y0 + i * p.ld_y, fmaf(v[i], scale, bias));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * LN_M + mine] = v[i];
      }
    }
    sm100::tc_fence_before();
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&sh.acc_empty[buf]);
    if (p.split == 1) continue;
    if (lane < p.split) arrive_at(&sh.part_full, lane);
    if (!__all_sync(0xffffffffu, wait_cluster(&sh.part_full, n & 1, abort))) {
      *abort = 1;
      return;
    }
    const int share = (rows + p.split - 1) / p.split;
    const int c1 = min(rows, (static_cast<int>(rank) + 1) * share);
    for (int c = static_cast<int>(rank) * share; c < c1; ++c) {
      float v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < p.split) v[r] = sm100::dsmem_ld_f32(sm100::dsmem_addr(part + c * LN_M + mine, r));
      float sum = 0.0f;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < p.split) sum += v[r];
      if (in) put(p, static_cast<long long>(at.row0 + c) * p.ld_y + out, fmaf(sum, scale, bias));
    }
    __syncwarp();
    if (lane < p.split) arrive_at(&sh.part_free, lane);
  }
}

template <int FMT>
__global__ void __launch_bounds__(LN_THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap wm, const __grid_constant__ CUtensorMap xm,
                  const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ LinearShared sh;
  LaunchStamp ls(p.stamp);
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* part = reinterpret_cast<float*>(ring + static_cast<size_t>(p.stages) * p.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &sh.abort;
  const uint32_t rank = p.split > 1 ? sm100::cluster_rank() : 0;
  const int first = blockIdx.x / p.split, step = gridDim.x / p.split;
  // this CTA's stages of the inner dimension
  const int k0 = static_cast<int>(static_cast<long long>(p.steps) * rank / p.split);
  const int k1 = static_cast<int>(static_cast<long long>(p.steps) * (rank + 1) / p.split);
  if (threadIdx.x == 0) {
    sm100::tma_prefetch_desc(&wm);
    sm100::tma_prefetch_desc(&xm);
    for (int i = 0; i < p.stages; ++i) {
      sm100::mbar_init(&sh.full[i], 1);
      sm100::mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&sh.acc_full[i], 1);
      sm100::mbar_init(&sh.acc_empty[i], 4);
    }
    sm100::mbar_init(&sh.part_full, 4 * p.split);
    sm100::mbar_init(&sh.part_free, 4 * p.split);
    sm100::mbar_init(&sh.drained, 1);
    sm100::fence_barrier_init();
    sh.abort = sh.never = sh.issued = 0;
    // the first ring's weights on their way to L2 (not into shared memory: what precedes may still write them)
    const TileAt at = tile_at(p, min(first, p.tiles - 1));
    for (int k = k0; k < min(k1, k0 + p.stages); ++k) prefetch_2d(&wm, k * LN_KB, at.out0);
  }
  if (warp == 1) {
    sm100::tmem_alloc(&sh.tmem, p.tmem_cols);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  if (p.split > 1) sm100::cluster_sync();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  ls.waited();
  pdl_trigger();
  if (warp == 0) {
    if (lane == 0) {
      produce<FMT>(p, sh, ring, &wm, &xm, first, step, k0, k1, abort);
      if (*abort)                                // copies in flight land first
        for (int i = max(0, sh.issued - p.stages); i < sh.issued; ++i)
          sm100::mbar_wait(&sh.full[i % p.stages], (i / p.stages) & 1, &sh.never);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      multiply<FMT>(p, sh, ring, tmem, first, step, k0, k1, abort);
      if (*abort) {                              // and products in flight end
        sm100::mma_commit(&sh.drained);
        sm100::mbar_wait(&sh.drained, 0, &sh.never);
      }
    }
  } else {
    read_out(p, sh, part, tmem, first, step, rank, abort);
  }
  __syncwarp();
  if (p.split > 1) sm100::cluster_sync();        // partials are read by the others
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  if (sh.abort && threadIdx.x == 0) set_status(p.status, EAGLE_ERR_TIMEOUT);
  if (warp == 1) sm100::tmem_dealloc(tmem, p.tmem_cols);
}

bool encode_rows(eagle_ctx* ctx, CUtensorMap* map, const void* data, int kbytes, int rows, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kbytes), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kbytes)};
  const cuuint32_t box[2] = {LN_KB, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return ctx->encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(data), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*LinearKernel)(CUtensorMap, CUtensorMap, LinearParams);

}  // namespace

cudaError_t launch_linear(eagle_ctx* ctx, const eagle_mx* x, const eagle_mx* w, const float* bias, int dtype, void* y,
                          int ld_y, int* status, cudaStream_t st) {
  const int fmt = w->format;
  const int gps = fmt == EAGLE_MX_FP8 ? 1 : fmt == EAGLE_MX_FP4 ? 2 : 4;
  LinearParams p{};
  const MxView xv = mx_view(x), wv = mx_view(w);
  p.w_scale = wv.scale;
  p.x_scale = xv.scale;
  p.gw = wv.g;
  p.gx = xv.g;
  p.bias = bias;
  p.y = y;
  p.ld_y = ld_y;
  p.f32 = dtype == EAGLE_DTYPE_F32;
  p.rows = x->rows;
  p.outs = w->rows;
  p.kbytes = fmt == EAGLE_MX_FP8 ? w->cols : w->cols / 2;
  p.groups = wv.groups;
  p.row_blocks = ceil_div(x->rows, 128);
  p.steps = ceil_div(p.kbytes, LN_KB);
  p.status = status;
  const int m_tiles = ceil_div(w->rows, LN_M);

  // The tile's rows and the split, by the time that a rough count gives them (cycles of an SM): a stage costs its
  // products or its bytes, whichever is more, a tile a fixed time, and the slowest cluster counts.
  struct Try { int nt, split; double cost; } best{0, 1, 1e30};
  for (int split = 1; split <= 8; split *= 2) {
    if (split > p.steps) break;
    const int clusters = ctx->sm_count / split;
    for (int q = 0; q < 4; ++q) {
      int nt = q == 0 ? ceil_div(x->rows, 16) * 16 : 64 * q;
      if (q == 0 ? nt > 192 : nt >= x->rows) continue;
      if (split > 1 && nt > 64) continue;
      const int tiles = m_tiles * ceil_div(x->rows, nt);
      const double bytes = LN_A_BYTES + nt * LN_KB + 512.0 * gps * 3;
      const double stage = std::max(2.0 * nt, bytes / (ceil_div(x->rows, nt) > 1 ? 48.0 : 24.0));
      const double cost = ceil_div(tiles, clusters) * (ceil_div(p.steps, split) * stage + (split > 1 ? 1500.0 : 300.0)) +
                          8.0 * nt;
      if (cost < best.cost) best = {nt, split, cost};
    }
  }
  p.nt = best.nt;
  p.split = best.split;
  p.row_tiles = ceil_div(x->rows, p.nt);
  p.tiles = m_tiles * p.row_tiles;
  p.rb = p.row_tiles > 1 ? (p.nt > 128 ? 2 : 1) : ceil_div(p.nt, 128);
  p.once = p.row_tiles == 1;
  p.b_bytes = static_cast<uint32_t>(p.nt * LN_KB);
  p.stage_bytes = static_cast<uint32_t>(align_up(LN_A_BYTES + p.b_bytes + 512u * gps * (1 + p.rb), 1024));
  const size_t part = p.split > 1 ? static_cast<size_t>(p.nt) * LN_M * 4 : 0;
  const size_t room = LN_SMEM - 1024 - part;
  p.stages = static_cast<int>(std::min<size_t>(LN_MAX_STAGES, room / p.stage_bytes));
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + part;
  p.acc_cols = static_cast<uint32_t>((p.nt + 31) / 32 * 32);
  p.sf_at = 2 * p.acc_cols;
  p.sf_cols = static_cast<uint32_t>(4 * gps * (1 + p.rb));
  p.tmem_cols = 32;
  while (p.tmem_cols < p.sf_at + 2 * p.sf_cols) p.tmem_cols <<= 1;
  if (p.tmem_cols > 512 || p.stages < 2) return cudaErrorInvalidConfiguration;

  CUtensorMap wm, xm;
  if (!encode_rows(ctx, &wm, w->data, p.kbytes, w->rows, LN_M) || !encode_rows(ctx, &xm, x->data, p.kbytes, x->rows, p.nt))
    return cudaErrorInvalidValue;
  const LinearKernel k = fmt == EAGLE_MX_FP8   ? linear_kernel<EAGLE_MX_FP8>
                         : fmt == EAGLE_MX_FP4 ? linear_kernel<EAGLE_MX_FP4>
                                               : linear_kernel<EAGLE_NV_FP4>;
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(k), static_cast<int>(LN_SMEM));
  if (e != cudaSuccess) return e;
  const int clusters = std::min(p.tiles, ctx->sm_count / p.split);
  p.stamp = stamp_slot(ctx, EAGLE_K_LINEAR);
  trace_before(ctx, EAGLE_K_LINEAR, st);
  e = p.split > 1 ? launch_pdl_cluster(k, dim3(clusters * p.split), dim3(LN_THREADS), smem, st, p.split, wm, xm, p)
                  : launch_pdl(k, dim3(clusters), dim3(LN_THREADS), smem, st, wm, xm, p);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_LINEAR, st);
  return e;
}

}  // namespace eagle
