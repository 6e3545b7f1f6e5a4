// eagle_mx_linear: y = x w^T (+ bias) of matrices in one microscaled format, on the block-scaled tensor-core
// instructions, which take both operands' scales from tensor memory.
//
// Few rows: the weights are operand A (128 outputs a tile) and the rows x operand B (16 to 192 a tile); an accumulator
// holds [128 outputs][rows] and a lane stores its output's column, 32 neighbours a warp.  Many rows: x is operand A and
// the weights B, a lane has a row and stores 16 outputs of it at once (in whole sectors; 4096 x 4096 x 4096
// 42 to 32 us); where it pays, two CTAs work on a tile of 256 rows of A, each loading half of B (tcgen05's pairs), so
// that an SM takes in less for as many products.  A stage of the ring holds 128 bytes of every row of both (256 four-bit or
// 128 eight-bit elements, 4 MMAs) and their scales, which lie in memory as the 512-byte groups that one tcgen05.cp spreads
// over tensor memory.  Warp roles: a producer for A and one for B (with the scales), one warp that issues the products and
// one the scales' copies (an instruction of either takes some 60 cycles to issue, 90 from a branch of one lane: 4096 x 8192
// x 10240 310 us so, 154 by a whole warp, 147 by two), four that read the accumulator out; two accumulators, so that a tile is read out under the next one's
// products.
//
// Bound, many rows: what an SM takes in, 64 bytes a cycle: a stage of 192 rows of B is 46 KB for a CTA alone and 34 KB for
// one of a pair (4096 x 8192 x 10240, NV_FP4: 148 and 120 us, 5.7 PFLOP/s), 720 and 530 cycles for products of 384; in 8 bits the
// same bytes are half the products, 233 us, 2.95 PFLOP/s).  Few rows: the weights' bytes from memory (16 x 8192 x 32000,
// NV_FP4: 26 us, 5.8 TB/s, 8 bits 45, 6.1; 1 x 4096 x 12288: 7.9, 3.6 TB/s, of which some 4 us until the first products and
// behind the last).
//
// Few tiles: a cluster of up to 8 CTAs splits a tile's inner dimension; each writes its partial to its own shared memory
// and sums its share of the rows over all of them, in rank order (8 x 8192 x 8192 in 8 bits: 16.1 us by two, 20.5 by one;
// 96 x 27648 x 5120 in FP4 20.5 by three, 26 by two, 35 by one; 442 x 16640 x 1072 in 8 bits, tiles of 128 rows by four
// 19.5, of 64 by two 25.7).
#include <algorithm>

#include "internal.h"
#include "common.cuh"
#include "mx.cuh"
#include "sm100.cuh"

namespace eagle {
namespace {

constexpr int LN_THREADS = 256;
constexpr int LN_M = 128;                     // A's rows of a tile
constexpr int LN_KB = 128;                    // bytes of a row in a stage
constexpr int LN_MAX_STAGES = 12;
constexpr int LN_A_BYTES = LN_M * LN_KB;
constexpr size_t LN_SMEM = 226 * 1024;     // dynamic: 227 KB less the barriers

struct LinearParams {
  const uint8_t* a_scale;
  const uint8_t* b_scale;
  const float* gw;
  const float* gx;
  const float* bias;
  void* y;
  long long ld_y;
  int f32;
  int by32;                // y's rows start at multiples of 32 bytes
  int a_rows, b_rows;      // x's and w's, or the other way round
  int by_row;              // A is x
  int kbytes;              // of a row
  int groups;              // 4-scale groups of a row
  int nt;                  // B's rows of a tile
  int b_tiles, tiles;
  int a_blocks, b_blocks;  // of 128 rows: scales
  int rb;                  // 128-row blocks that a tile's scales of B take at most
  int steps;               // stages of the inner dimension
  int split;               // CTAs of a cluster that split the inner dimension
  int n_acc;               // accumulators
  int stages;
  uint32_t stage_bytes, b_bytes;
  uint32_t acc_cols, sf_at, sf_cols, tmem_cols;
  int sf_log;              // places for a stage's scales in tensor memory, two or four, as a power of two
  int once;                // A is read once
  int* status;
  uint64_t* stamp;
};

struct LinearShared {
  uint64_t full[LN_MAX_STAGES], empty[LN_MAX_STAGES];
  uint64_t sf_full[4];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t part_full, part_free;
  uint64_t drained[2];
  uint32_t tmem;
  int abort, never;
};

template <int FMT>
constexpr int groups_per_stage() { return FMT == EAGLE_MX_FP8 ? 1 : FMT == EAGLE_MX_FP4 ? 2 : 4; }

// Instruction descriptor of the block-scaled kinds: element types at bits 7 and 10 (e4m3 0, e2m1 1), N / 8 at 17, the
// scales' type at 23 (e4m3 0, power of two 1), M / 16 at 24, and which bytes of a 32-bit column of scales the
// instruction takes, at 4 for B and 29 for A.
template <int FMT, bool PAIR>
__device__ __forceinline__ uint32_t idesc_of(int n, int sf) {
  const uint32_t type = FMT == EAGLE_MX_FP8 ? 0u : 1u;
  const uint32_t scale = FMT == EAGLE_NV_FP4 ? 0u : 1u;
  return (static_cast<uint32_t>(sf) << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (scale << 23) | (static_cast<uint32_t>((PAIR ? 2 * LN_M : LN_M) >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);
}

// One product by the lane with `lead`, the operands given as the low words of their descriptors (the high word is
// sm100::DESC_SW128_HI): a predicate instead of a branch, so that the operands can stay in uniform registers.
#define EAGLE_MMA_SCALED(GROUP, KIND)                                                                                  \
  asm volatile(                                                                                                        \
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %7, 0;\n setp.ne.b32 q, %8, 0;\n mov.b64 a, {%1, %6};\n" \
      " mov.b64 b, {%2, %6};\n @q tcgen05.mma." GROUP "." KIND " [%0], a, b, %3, [%4], [%5], p;\n}\n" ::"r"(d),          \
      "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(sm100::DESC_SW128_HI), "r"(acc), "r"(lead)                     \
      : "memory")
template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t acc, uint32_t lead) {
  if (PAIR) {
    if (FMT == EAGLE_MX_FP8) EAGLE_MMA_SCALED("cta_group::2", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    else if (FMT == EAGLE_MX_FP4) EAGLE_MMA_SCALED("cta_group::2", "kind::mxf4nvf4.block_scale.scale_vec::2X");
    else EAGLE_MMA_SCALED("cta_group::2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  } else {
    if (FMT == EAGLE_MX_FP8) EAGLE_MMA_SCALED("cta_group::1", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    else if (FMT == EAGLE_MX_FP4) EAGLE_MMA_SCALED("cta_group::1", "kind::mxf4nvf4.block_scale.scale_vec::2X");
    else EAGLE_MMA_SCALED("cta_group::1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  }
}
#undef EAGLE_MMA_SCALED

// Arrives once what this lane has issued so far is through: on `bar`, for a pair (ALL) on its twin in the other CTA too.
template <bool PAIR, bool ALL>
__device__ __forceinline__ void commit_if(uint64_t* bar, uint32_t lead) {
  if (PAIR && ALL)
    asm volatile(
        "{\n .reg .pred q;\n .reg .b16 m;\n setp.ne.b32 q, %1, 0;\n mov.b16 m, 3;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(
            sm100::smem_u32(bar)),
        "r"(lead)
        : "memory");
  else if (PAIR)
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(sm100::smem_u32(bar)),
        "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(sm100::smem_u32(bar)),
        "r"(lead)
        : "memory");
}

// 512 bytes of scales to four columns, repeated in each quarter of the lanes (a pair: of both CTAs, each from its own
// memory).  (32 rows of 16 bytes without swizzle, 8-row groups 128 bytes apart.)
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t saddr, uint32_t lead) {
  if (PAIR)
    asm volatile(
        "{\n .reg .pred q;\n .reg .b64 d;\n setp.ne.b32 q, %3, 0;\n mov.b64 d, {%1, %2};\n"
        " @q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n}\n" ::"r"(tmem),
        "r"((saddr >> 4) & 0x3FFFu), "r"((128u >> 4) | (1u << 14)), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred q;\n .reg .b64 d;\n setp.ne.b32 q, %3, 0;\n mov.b64 d, {%1, %2};\n"
        " @q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n}\n" ::"r"(tmem),
        "r"((saddr >> 4) & 0x3FFFu), "r"((128u >> 4) | (1u << 14)), "r"(lead)
        : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tmem_take(uint32_t* dst, uint32_t cols) {
  if (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm100::smem_u32(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    sm100::tmem_alloc(dst, cols);
    sm100::tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_give(uint32_t at, uint32_t cols) {
  if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
  else sm100::tmem_dealloc(at, cols);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(yes));
  return yes != 0;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   sm100::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
               : "memory");
}
// (A pair's) tiled load into this CTA, counted on a barrier of the pair's first.
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(sm100::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
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

// A tile's place: this CTA's rows of A, the tile's rows of B and their first block of scales.
struct TileAt {
  int a0, b0, rb0, n_rb;
};
template <bool PAIR>
__device__ __forceinline__ TileAt tile_at(const LinearParams& p, int tile, uint32_t rank) {
  TileAt t;
  const int m = tile / p.b_tiles;
  t.a0 = (PAIR ? 2 * m + static_cast<int>(rank) : m) * LN_M;
  t.b0 = (tile - m * p.b_tiles) * p.nt;
  t.rb0 = t.b0 >> 7;
  const int last = min((t.b0 + p.nt - 1) >> 7, p.b_blocks - 1);
  t.n_rb = last - t.rb0 + 1;
  return t;
}

// The loops below are gone through by whole warps and issue by predicate: what the instructions take then stays in uniform
// registers (issued by a lane that had branched off, a product took 90 cycles and a copy of scales 67).  An instruction
// of the tensor core still takes its warp some 60 cycles, so that the loads of either operand, the copies of scales and
// the products each have a warp of their own (4096 x 8192 x 10240, NV_FP4: one branched-off lane for each of loads and
// tensor core 310 us, whole warps 164, these 147).

// Whose barriers count a CTA's loads: its own, but for a pair the first one's for both.  The CTA with the barriers asks for
// the bytes, and where a wait ran out it stays until the loads under way have landed: the shared memory of a CTA that has
// left may be another's.  (The CTAs of a split load for themselves, whatever their rank.)
constexpr bool counts_loads(bool pair, uint32_t rank) { return !pair || rank == 0; }
static_assert(counts_loads(false, 0) && counts_loads(false, 1) && counts_loads(false, 7), "every CTA of a split waits");
static_assert(counts_loads(true, 0) && !counts_loads(true, 1), "a pair's first CTA waits for both");

// Loads A (X false) or B (X true), and their scales, of this CTA's stages.  A pair's CTAs load 128 rows of A and half of
// the tile's rows of B each (and all of those rows' scales), counted on the first one's barriers; their
// scales come by a map too, whose box may reach into the next 128 rows' groups (no product takes those).
template <int FMT, bool X, bool PAIR>
__device__ __forceinline__ void produce(const LinearParams& p, LinearShared& sh, uint8_t* ring, const CUtensorMap* map,
                                        const CUtensorMap* scales, int first, int step, int k0, int k1, uint32_t rank,
                                        volatile int* abort) {
  constexpr int GPS = groups_per_stage<FMT>();
  const uint64_t policy = sm100::l2_policy_evict_first();
  int slot = 0, issued = 0;
  uint32_t phase = 1;
  for (int tile = first; tile < p.tiles; tile += step) {
    const TileAt at = tile_at<PAIR>(p, tile, rank);
    const int block = X ? at.rb0 : at.a0 >> 7;
    const uint8_t* from =
        (X ? p.b_scale : p.a_scale) + (static_cast<size_t>(block) * p.groups + static_cast<size_t>(k0) * GPS) * 512;
    const size_t next = static_cast<size_t>(p.groups) * 512;
    int left = p.groups - k0 * GPS;              // groups of scales from here on
    for (int k = k0; k < k1; ++k) {
      if (!__all_sync(0xffffffffu, sm100::mbar_wait(&sh.empty[slot], phase, abort))) {
        *abort = 1;
        break;
      }
      ++issued;
      uint8_t* st = ring + static_cast<size_t>(slot) * p.stage_bytes;
      uint64_t* bar = &sh.full[slot];
      uint8_t* s = st + LN_A_BYTES + p.b_bytes;
      if (PAIR) {
        if (elect_one()) {
          const uint32_t both = sm100::dsmem_addr(bar, 0);
          if (counts_loads(PAIR, rank))
            sm100::mbar_arrive_expect_tx(bar, 2 * (X ? p.b_bytes + GPS * 512u * p.rb : LN_A_BYTES + GPS * 512u));
          if (X) {
            pair_load_2d(st + LN_A_BYTES, map, k * LN_KB, at.b0 + static_cast<int>(rank) * (p.nt / 2), both);
            for (int b = 0; b < p.rb; ++b)
              pair_load_2d(s + (1 + b) * GPS * 512, scales, 0, (block + b) * p.groups + k * GPS, both);
          } else {
            pair_load_2d(st, map, k * LN_KB, at.a0, both);
            pair_load_2d(s, scales, 0, block * p.groups + k * GPS, both);
          }
        }
      } else {
        const uint32_t sf = static_cast<uint32_t>(min(GPS, left)) * 512u;
        if (elect_one()) {
          if (X) {
            sm100::mbar_arrive_expect_tx(bar, p.b_bytes + sf * static_cast<uint32_t>(at.n_rb));
            sm100::tma_load_2d(st + LN_A_BYTES, map, k * LN_KB, at.b0, bar);
            bulk_load(s + GPS * 512, from, sf, bar);
            if (at.n_rb > 1) bulk_load(s + 2 * GPS * 512, from + next, sf, bar);
          } else {
            sm100::mbar_arrive_expect_tx(bar, LN_A_BYTES + sf);
            if (p.once) sm100::tma_load_2d_hint(st, map, k * LN_KB, at.a0, bar, policy);
            else sm100::tma_load_2d(st, map, k * LN_KB, at.a0, bar);
            bulk_load(s, from, sf, bar);
          }
        }
      }
      __syncwarp();
      from += GPS * 512;
      left -= GPS;
      if (++slot == p.stages) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (*abort) break;
  }
  if (*abort && counts_loads(PAIR, rank))        // copies in flight land first (if the others asked for theirs too)
    for (int i = max(0, issued - p.stages); i < issued; ++i)
      sm100::mbar_wait(&sh.full[i % p.stages], (i / p.stages) & 1, &sh.never);
}

// Scales to tensor memory, ahead of the products: places in turn, the products of as many stages before being through with
// the one that is written.  RB: 128-row blocks of x's scales in a tile.
template <int FMT, int RB, bool PAIR>
__device__ __forceinline__ void spread_scales(const LinearParams& p, LinearShared& sh, uint8_t* ring, uint32_t tmem,
                                              int first, int step, int k0, int k1, volatile int* abort) {
  constexpr int GPS = groups_per_stage<FMT>();
  const uint32_t ring0 = sm100::smem_u32(ring) + LN_A_BYTES + p.b_bytes;
  const uint32_t lead = elect_one();
  const int places = 1 << p.sf_log;
  int slot = 0, old = p.stages - places;
  uint32_t phase = 0, old_phase = 1;
  const int total = first < p.tiles ? ((p.tiles - first + step - 1) / step) * (k1 - k0) : 0;
  for (int i = 0; i < total; ++i) {
    bool ok = sm100::mbar_wait(&sh.full[slot], phase, abort);
    ok = ok && (i < places || sm100::mbar_wait(&sh.empty[old], old_phase, abort));
    if (!__all_sync(0xffffffffu, ok)) {
      *abort = 1;
      return;
    }
    sm100::tc_fence_after();
    const uint32_t s = ring0 + static_cast<uint32_t>(slot) * p.stage_bytes;
    const int place = i & (places - 1);
    const uint32_t sfa = tmem + p.sf_at + place * p.sf_cols, sfb = sfa + 4 * GPS;
#pragma unroll
    for (int g = 0; g < GPS; ++g) {
      copy_scales<PAIR>(sfa + 4 * g, s + 512 * g, lead);
#pragma unroll
      for (int b = 0; b < RB; ++b) copy_scales<PAIR>(sfb + 4 * (g * RB + b), s + 512 * ((1 + b) * GPS + g), lead);
    }
    commit_if<PAIR, false>(&sh.sf_full[place], lead);
    sm100::mbar_arrive_if(&sh.sf_full[place], lead);   // (and that the stage itself is there)
    if (++slot == p.stages) {
      slot = 0;
      phase ^= 1;
    }
    if (++old == p.stages) {
      old = 0;
      old_phase ^= 1;
    }
  }
}

template <int FMT, int RB, bool PAIR>
__device__ __forceinline__ void multiply(const LinearParams& p, LinearShared& sh, uint8_t* ring, uint32_t tmem,
                                         int first, int step, int k0, int k1, volatile int* abort) {
  constexpr int GPS = groups_per_stage<FMT>();
  const uint32_t ring0 = sm100::smem_u32(ring);
  const uint32_t lead = elect_one();
  int slot = 0, n = 0, i = 0;
  for (int tile = first; tile < p.tiles; tile += step, ++n) {
    const int buf = p.n_acc == 2 ? n & 1 : 0;
    const uint32_t used = static_cast<uint32_t>(p.n_acc == 2 ? n >> 1 : n) & 1u;
    const uint32_t b_off = static_cast<uint32_t>((tile % p.b_tiles) * p.nt & 127) >> 5;
    if (!__all_sync(0xffffffffu, PAIR ? wait_cluster(&sh.acc_empty[buf], used ^ 1u, abort)
                                      : sm100::mbar_wait(&sh.acc_empty[buf], used ^ 1u, abort))) {
      *abort = 1;
      return;
    }
    const uint32_t d = tmem + static_cast<uint32_t>(buf) * p.acc_cols;
    uint32_t acc = 0;
    for (int k = k0; k < k1; ++k, ++i) {
      const int place = i & ((1 << p.sf_log) - 1);
      if (!__all_sync(0xffffffffu, sm100::mbar_wait(&sh.sf_full[place], (i >> p.sf_log) & 1, abort))) {
        *abort = 1;
        return;
      }
      sm100::tc_fence_after();
      const uint32_t st = ring0 + static_cast<uint32_t>(slot) * p.stage_bytes;
      const uint32_t sfa = tmem + p.sf_at + place * p.sf_cols, sfb = sfa + 4 * GPS + b_off;
      const uint32_t ad = st >> 4, bd = (st + LN_A_BYTES) >> 4;
      const int left = p.kbytes - k * LN_KB;           // bytes: 32 a product
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int g = FMT == EAGLE_MX_FP8 ? 0 : FMT == EAGLE_MX_FP4 ? j / 2 : j;
        const int sf = FMT == EAGLE_MX_FP8 ? j : FMT == EAGLE_MX_FP4 ? 2 * (j & 1) : 0;
        if (j == 0 || 32 * j < left)
          mma_scaled<FMT, PAIR>(d, ad + 2 * j, bd + 2 * j, idesc_of<FMT, PAIR>(p.nt, sf), sfa + 4 * g, sfb + 4 * g * RB,
                          j == 0 ? acc : 1u, lead);
      }
      commit_if<PAIR, true>(&sh.empty[slot], lead);
      if (k + 1 == k1) commit_if<PAIR, true>(&sh.acc_full[buf], lead);
      acc = 1;
      if (++slot == p.stages) slot = 0;
    }
  }
}

__device__ __forceinline__ void put(const LinearParams& p, long long at, float v) {
  if (p.f32) static_cast<float*>(p.y)[at] = v;
  else static_cast<uint16_t*>(p.y)[at] = f32_to_bf16(v);
}

// 32 bytes at a multiple of 32: a whole sector a lane.
__device__ __forceinline__ void store_32_bytes(float* to, const float (&y)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(y[0]), "f"(y[1]), "f"(y[2]),
               "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
               : "memory");
}
// Sixteen outputs of a row as bf16, all there, to a multiple of 32 bytes.
__device__ __forceinline__ void put16(const LinearParams& p, long long at, int out, float scale, const float* v) {
  float y[16];
  if (p.bias) {
    float b[16];
    load8(p.bias + out, reinterpret_cast<float(&)[8]>(b[0]));
    load8(p.bias + out + 8, reinterpret_cast<float(&)[8]>(b[8]));
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = fmaf(v[i], scale, b[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = v[i] * scale;
  }
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    w[i] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h));
  }
  store_32_bytes(reinterpret_cast<float*>(static_cast<uint16_t*>(p.y) + at), w);
}

// Eight outputs of a row, of which `n` are there.
__device__ __forceinline__ void put8(const LinearParams& p, long long at, int out, int n, float scale, const float* v) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * scale;
  if (p.bias) {
    float b[8];
    if (n >= 8) load8(p.bias + out, b);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = i < n ? p.bias[out + i] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(v[i], scale, b[i]);
  }
  if (n >= 8) {
    if (p.f32 && p.by32) store_32_bytes(static_cast<float*>(p.y) + at, y);
    else if (p.f32) store8(static_cast<float*>(p.y) + at, y);
    else store8(static_cast<uint16_t*>(p.y) + at, y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) put(p, at + i, y[i]);
  }
}

template <bool PAIR>
__device__ __forceinline__ void read_out(const LinearParams& p, LinearShared& sh, float* part, uint32_t tmem, int first,
                                         int step, uint32_t rank, volatile int* abort) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
  const float scale = (p.gw ? *p.gw : 1.0f) * (p.gx ? *p.gx : 1.0f);
  const int mine = quarter * 32 + lane;
  int n = 0;
  for (int tile = first; tile < p.tiles; tile += step, ++n) {
    const TileAt at = tile_at<PAIR>(p, tile, rank);
    const int buf = p.n_acc == 2 ? n & 1 : 0, out = at.a0 + mine;    // (by rows: the row)
    const uint32_t used = static_cast<uint32_t>(p.n_acc == 2 ? n >> 1 : n) & 1u;
    const bool in = out < p.a_rows;
    const float bias = p.bias && in && !p.by_row ? p.bias[out] : 0.0f;
    const int rows = min(p.nt, p.b_rows - at.b0);
    if (!__all_sync(0xffffffffu, sm100::mbar_wait(&sh.acc_full[buf], used, abort))) {
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
    if (p.by_row) {
      const long long y0 = static_cast<long long>(out) * p.ld_y + at.b0;
      for (int c = 0; c < rows; c += 32) {       // (a tile's columns are a multiple of 16: the accumulator's of 32)
        float v[32];
        sm100::tmem_ld32(d + c, v);
        sm100::tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          if (!in || c + h >= rows) break;
          if (p.by32 && !p.f32 && c + h + 16 <= rows) {
            put16(p, y0 + c + h, at.b0 + c + h, scale, &v[h]);
            continue;
          }
          put8(p, y0 + c + h, at.b0 + c + h, rows - c - h, scale, &v[h]);
          if (c + h + 8 < rows) put8(p, y0 + c + h + 8, at.b0 + c + h + 8, rows - c - h - 8, scale, &v[h + 8]);
        }
      }
    }
    for (int c = 0; c < rows && !p.by_row; c += 16) {
      float v[16];
      sm100::tmem_ld16(d + c, v);
      sm100::tmem_wait_ld();
      if (p.split == 1) {
        const long long y0 = static_cast<long long>(at.b0 + c) * p.ld_y + out;
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
    if (lane == 0) {
      if (PAIR) arrive_at(&sh.acc_empty[buf], 0);
      else sm100::mbar_arrive(&sh.acc_empty[buf]);
    }
    if (p.split == 1) continue;
    if (lane < p.split) arrive_at(&sh.part_full, lane);
    if (!__all_sync(0xffffffffu, wait_cluster(&sh.part_full, n & 1, abort))) {
      *abort = 1;
      return;
    }
    const int share = (rows + p.split - 1) / p.split;
    const int c1 = min(rows, (static_cast<int>(rank) + 1) * share);
    for (int c = static_cast<int>(rank) * share; c < c1; c += 4) {
      float v[4][8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < p.split) {
          const uint32_t from = sm100::dsmem_addr(part + c * LN_M + mine, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i][r] = sm100::dsmem_ld_f32(from + (c + i < c1 ? i : 0) * LN_M * 4);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < p.split) sum += v[i][r];
        if (in && c + i < c1) put(p, static_cast<long long>(at.b0 + c + i) * p.ld_y + out, fmaf(sum, scale, bias));
      }
    }
    __syncwarp();
    if (lane < p.split) arrive_at(&sh.part_free, lane);
  }
}

template <int FMT, bool PAIR>
__global__ void __launch_bounds__(LN_THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap am, const __grid_constant__ CUtensorMap bm,
                  const __grid_constant__ CUtensorMap asc, const __grid_constant__ CUtensorMap bsc,
                  const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ LinearShared sh;
  LaunchStamp ls(p.stamp);
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* part = reinterpret_cast<float*>(ring + static_cast<size_t>(p.stages) * p.stage_bytes);
  const int warp = threadIdx.x >> 5;
  volatile int* abort = &sh.abort;
  const uint32_t rank = PAIR || p.split > 1 ? sm100::cluster_rank() : 0;
  const int ctas = PAIR ? 2 : p.split;
  const int first = blockIdx.x / ctas, step = gridDim.x / ctas;
  // this CTA's stages of the inner dimension
  const int k0 = PAIR ? 0 : static_cast<int>(static_cast<long long>(p.steps) * rank / p.split);
  const int k1 = PAIR ? p.steps : static_cast<int>(static_cast<long long>(p.steps) * (rank + 1) / p.split);
  if (threadIdx.x == 0) {
    sm100::tma_prefetch_desc(&am);
    sm100::tma_prefetch_desc(&bm);
    for (int i = 0; i < p.stages; ++i) {
      sm100::mbar_init(&sh.full[i], 2);
      sm100::mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) sm100::mbar_init(&sh.sf_full[i], 2);
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&sh.acc_full[i], 1);
      sm100::mbar_init(&sh.acc_empty[i], PAIR ? 8 : 4);
    }
    sm100::mbar_init(&sh.part_full, 4 * p.split);
    sm100::mbar_init(&sh.part_free, 4 * p.split);
    sm100::mbar_init(&sh.drained[0], 1);
    sm100::mbar_init(&sh.drained[1], 1);
    sm100::fence_barrier_init();
    sh.abort = sh.never = 0;
    // the first ring's weights on their way to L2 (not into shared memory: what precedes may still write them)
    const TileAt at = tile_at<PAIR>(p, min(first, p.tiles - 1), rank);
    for (int k = k0; k < min(k1, k0 + p.stages); ++k)
      prefetch_2d(p.by_row ? &bm : &am, k * LN_KB, p.by_row ? at.b0 : at.a0);
  }
  if (PAIR) {                                    // (the allocation takes both CTAs)
    __syncwarp();
    sm100::cluster_sync();
  }
  if (warp == 1) tmem_take<PAIR>(&sh.tmem, p.tmem_cols);
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  if (PAIR || p.split > 1) sm100::cluster_sync();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  ls.waited();
  pdl_trigger();
  if (warp == 0) {
    produce<FMT, false, PAIR>(p, sh, ring, &am, &asc, first, step, k0, k1, rank, abort);
  } else if (warp == 3) {
    produce<FMT, true, PAIR>(p, sh, ring, &bm, &bsc, first, step, k0, k1, rank, abort);
  } else if (PAIR && rank == 1 && warp < 3) {
    // (the first CTA issues for both)
  } else if (warp == 1 || warp == 2) {
    if (warp == 1) {
      if (p.rb == 1) multiply<FMT, 1, PAIR>(p, sh, ring, tmem, first, step, k0, k1, abort);
      else multiply<FMT, 2, PAIR>(p, sh, ring, tmem, first, step, k0, k1, abort);
    } else {
      if (p.rb == 1) spread_scales<FMT, 1, PAIR>(p, sh, ring, tmem, first, step, k0, k1, abort);
      else spread_scales<FMT, 2, PAIR>(p, sh, ring, tmem, first, step, k0, k1, abort);
    }
    __syncwarp();
    if (*abort) {                                // what is in flight on the tensor core ends
      commit_if<PAIR, false>(&sh.drained[warp - 1], elect_one());
      __syncwarp();
      sm100::mbar_wait(&sh.drained[warp - 1], 0, &sh.never);
    }
  } else {
    read_out<PAIR>(p, sh, part, tmem, first, step, rank, abort);
  }
  __syncwarp();
  if (PAIR || p.split > 1) sm100::cluster_sync();        // partials and stages are read by the others
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  if (sh.abort && threadIdx.x == 0) set_status(p.status, EAGLE_ERR_TIMEOUT);
  if (warp == 1) tmem_give<PAIR>(tmem, p.tmem_cols);
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

// The 4-scale groups of all blocks of 128 rows as rows of 512 bytes; a box is a stage's.
bool encode_scales(eagle_ctx* ctx, CUtensorMap* map, const void* scale, int blocks, int groups, int gps) {
  const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(blocks) * groups};
  const cuuint64_t strides[1] = {512};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(gps)};
  const cuuint32_t estr[2] = {1, 1};
  return ctx->encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(scale), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*LinearKernel)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, LinearParams);
template <int FMT>
LinearKernel kernel_of(bool pair) {
  return pair ? linear_kernel<FMT, true> : linear_kernel<FMT, false>;
}
LinearKernel kernel_of(int format, bool pair) {
  return format == EAGLE_MX_FP8   ? kernel_of<EAGLE_MX_FP8>(pair)
         : format == EAGLE_MX_FP4 ? kernel_of<EAGLE_MX_FP4>(pair)
                                  : kernel_of<EAGLE_NV_FP4>(pair);
}

// Clusters that the GPU holds at once.  A cluster lies within a group of SMs, so that sizes that do not divide a group's
// leave SMs over: 152 SMs hold 46 clusters of 3 CTAs, 36 of 4, 28 of 5, 23 of 6, 15 of 7 or 8.  One more begins when the
// others have gone through all their tiles (3 x 15488 x 3633 in 8 bits, 29 tiles: by clusters of 5, of which 28 run,
// 25.2 us, by 29 of 4 15.5).
int clusters_of(eagle_ctx* ctx, int format, bool pair, int ctas) {
  if (ctas == 1) return ctx->sm_count;
  int& known = ctx->clusters[format - 1][pair][ctas];
  if (known == 0) {
    const LinearKernel k = kernel_of(format, pair);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctx->sm_count / ctas * ctas);
    cfg.blockDim = dim3(LN_THREADS);
    cfg.dynamicSmemBytes = LN_SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (smem_limit_once(reinterpret_cast<const void*>(k), static_cast<int>(LN_SMEM)) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&known, k, &cfg) != cudaSuccess || known < 1) {
      cudaGetLastError();
      known = ctx->sm_count / ctas;
    }
  }
  return known;
}

}  // namespace

cudaError_t launch_linear(eagle_ctx* ctx, const eagle_mx* x, const eagle_mx* w, const float* bias, int dtype, void* y,
                          int ld_y, int* status, cudaStream_t st) {
  const int fmt = w->format;
  const int gps = fmt == EAGLE_MX_FP8 ? 1 : fmt == EAGLE_MX_FP4 ? 2 : 4;
  LinearParams p{};
  const MxView xv = mx_view(x), wv = mx_view(w);
  p.gw = wv.g;
  p.gx = xv.g;
  p.bias = bias;
  p.y = y;
  p.ld_y = ld_y;
  p.f32 = dtype == EAGLE_DTYPE_F32;
  p.by32 = (reinterpret_cast<uintptr_t>(y) & 31) == 0 && ld_y % (p.f32 ? 8 : 16) == 0;
  p.kbytes = fmt == EAGLE_MX_FP8 ? w->cols : w->cols / 2;
  p.groups = wv.groups;
  p.steps = ceil_div(p.kbytes, LN_KB);
  p.status = status;
  size_t smem = 0;

  // What a choice of the operands' places, of B's rows in a tile, of pairs (256 rows of A a tile) or of the split needs of
  // shared and tensor memory.
  struct Choice { bool by_row; int nt; bool pair; int split; };
  auto settle = [&](const Choice& c) {
    const eagle_mx* a = c.by_row ? x : w;
    const eagle_mx* b = c.by_row ? w : x;
    p.by_row = c.by_row;
    p.a_scale = a->scale;
    p.b_scale = b->scale;
    p.a_rows = a->rows;
    p.b_rows = b->rows;
    p.a_blocks = ceil_div(a->rows, 128);
    p.b_blocks = ceil_div(b->rows, 128);
    p.nt = c.nt;
    p.split = c.split;
    p.b_tiles = ceil_div(b->rows, c.nt);
    p.tiles = ceil_div(a->rows, c.pair ? 2 * LN_M : LN_M) * p.b_tiles;
    p.rb = ceil_div(c.nt, 128);
    p.once = p.b_tiles == 1 && !c.by_row;
    p.b_bytes = static_cast<uint32_t>((c.pair ? c.nt / 2 : c.nt) * LN_KB);
    p.stage_bytes = static_cast<uint32_t>(align_up(LN_A_BYTES + p.b_bytes + 512u * gps * (1 + p.rb), 1024));
    p.acc_cols = static_cast<uint32_t>((c.nt + 31) / 32 * 32);
    p.sf_cols = static_cast<uint32_t>(4 * gps * (1 + p.rb));
    p.n_acc = 2 * p.acc_cols + 2 * p.sf_cols <= 512 ? 2 : 1;
    p.sf_at = static_cast<uint32_t>(p.n_acc) * p.acc_cols;
    const size_t part = c.split > 1 ? static_cast<size_t>(c.nt) * LN_M * 4 : 0;
    p.stages = static_cast<int>(std::min<size_t>(LN_MAX_STAGES, (LN_SMEM - 1024 - part) / p.stage_bytes));
    p.sf_log = p.stages >= 4 && p.sf_at + 4 * p.sf_cols <= 512 ? 2 : 1;
    p.tmem_cols = 32;
    while (p.tmem_cols < p.sf_at + (p.sf_cols << p.sf_log)) p.tmem_cols <<= 1;
    smem = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + part;
  };
  // The one that a rough count of an SM's cycles gives the least time.  A stage costs its products (2 cycles a row of B),
  // its bytes (64 a cycle, and 40), 550 cycles in any case or, where the weights are read once, those that come from memory
  // (24 bytes a cycle and SM with all SMs at it, 33 at most), whichever is the most; a tile is read out under the next one's
  // products where there are two accumulators; the slowest cluster counts.  (Over 25 shapes from 1 to 1001 rows its choice
  // was within 10 % of the best of all.)
  Choice best{false, 0, false, 1};
  double least = 1e30;
  auto consider = [&](const Choice& c) {
    settle(c);
    const int clusters = clusters_of(ctx, fmt, c.pair, c.pair ? 2 : c.split);
    const double bytes = p.stage_bytes;
    const double active = std::min(p.tiles, clusters) * (c.pair ? 2.0 : c.split) / ctx->sm_count;
    const double weights = p.once ? (LN_A_BYTES + 512.0 * gps) * std::max(active / 24.0, 1.0 / 33.0) : 0.0;
    const double stage = std::max({2.0 * c.nt, bytes / 64.0 + 40.0, weights, 550.0});
    const double work = ceil_div(p.steps, c.split) * stage, read = (c.by_row ? 25.0 : 45.0) * c.nt + 400.0;
    const double tile = c.split > 1 ? work + read + 2500.0 : p.n_acc == 1 ? work + read + 2500.0 : std::max(work, read);
    const double cost = ceil_div(p.tiles, clusters) * tile + read;
    if (cost < least) {
      least = cost;
      best = c;
    }
  };
  const int all = ceil_div(x->rows, 16) * 16, outs = ceil_div(w->rows, 16) * 16;
  for (int split = 1; split <= 8 && split <= p.steps; ++split)
    for (int q = 0; q < 4; ++q) {
      const int nt = q == 0 ? all : 64 * q;
      if (q == 0 ? nt > 192 : nt >= x->rows) continue;
      if (split == 1 || nt <= 128) consider({false, nt, false, split});
    }
  for (int by_row = 0; by_row < 2; ++by_row) {   // (B's tiles: places of scales 64 rows apart)
    const int b = by_row ? outs : all, a = by_row ? x->rows : w->rows;
    for (int q = 0; q <= 4; ++q) {
      const int nt = q == 0 ? b : 64 * q;
      if (q == 0 ? nt > 256 : nt >= (by_row ? w->rows : x->rows)) continue;
      if (by_row && x->rows > 64 && nt <= 192) consider({true, nt, false, 1});
      if (a > LN_M && nt >= 64) consider({by_row == 1, nt, true, 1});
    }
  }
  settle(best);
  if (p.tmem_cols > 512 || p.stages < 2) return cudaErrorInvalidConfiguration;

  const eagle_mx* a = best.by_row ? x : w;
  const eagle_mx* b = best.by_row ? w : x;
  CUtensorMap am, bm, asc, bsc;
  if (!encode_rows(ctx, &am, a->data, p.kbytes, a->rows, LN_M) ||
      !encode_rows(ctx, &bm, b->data, p.kbytes, b->rows, best.pair ? p.nt / 2 : p.nt))
    return cudaErrorInvalidValue;
  asc = bsc = am;                                // (only pairs take them)
  if (best.pair && (!encode_scales(ctx, &asc, a->scale, p.a_blocks, p.groups, gps) ||
                    !encode_scales(ctx, &bsc, b->scale, p.b_blocks, p.groups, gps)))
    return cudaErrorInvalidValue;
  const LinearKernel k = kernel_of(fmt, best.pair);
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(k), static_cast<int>(LN_SMEM));
  if (e != cudaSuccess) return e;
  const int ctas = best.pair ? 2 : p.split;
  const int clusters = std::min(p.tiles, clusters_of(ctx, fmt, best.pair, ctas));
  p.stamp = stamp_slot(ctx, EAGLE_K_LINEAR);
  trace_before(ctx, EAGLE_K_LINEAR, st);
  e = ctas > 1 ? launch_pdl_cluster(k, dim3(clusters * ctas), dim3(LN_THREADS), smem, st, ctas, am, bm, asc, bsc, p)
               : launch_pdl(k, dim3(clusters), dim3(LN_THREADS), smem, st, am, bm, asc, bsc, p);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_LINEAR, st);
  return e;
}

}  // namespace eagle
