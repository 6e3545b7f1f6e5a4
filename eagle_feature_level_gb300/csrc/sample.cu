// eagle_sample: a row's distribution under temperature, top-k, top-p and min-p, and a draw from it.
//
// A cluster of CTAs holds a row's logits in shared memory, so that they are read once; the weights
// floor(2^40 e^((z - max) / t)) are computed from them wherever one is needed.  Weights are whole numbers and their sums
// exact, so the order of sums does not matter and a border is where the definition has it.
//
// Tokens within 17 powers of two of the largest weight (the near ones) are few as a rule: each CTA lists where they are,
// and all that needs more than fp32's precision goes over that list, so that the work on them is dense.  The passes are
// loops, not unrolled over registers: each is gone through once a row, and the straight-line form waited for its own
// instructions (one row of 32000: 48 us).
//
// The cut (the last token in falling order that top-k or top-p keeps) is found among fewer still.  Top-k: of the threads'
// own largest tokens, the k-th largest bounds the row's k-th from below, so a histogram of these alone (1024 bins by the
// distance to the row's largest) gives a bin up to which there are at least k tokens, and seldom many more.  Top-p: one
// pass adds up the weight of all tokens and of those within 4, 8, 12 and 17 powers of two of the largest, and the cut lies
// between two of these.  Where such a part has at most 512 tokens, the cluster's first CTA gathers and sorts it; so
// top-k needs the weights of its own tokens alone, and that CTA finishes the row.  Otherwise a histogram of the part's
// tokens, with their number or weight, is summed over the cluster (a slice of the bins a CTA) and scanned by its first
// CTA; a bin that still has more tokens is split by the bits of the logits, 10 at a time, and tokens of one value by
// their ids.
//
// Bound: instructions (216 rows of 32000: greedy 17 us, top-k of 50 41, top-p of 0.9 83 at t = 0.9), and for one row the
// latency of the exchanges and of code run once (16.8 us).  CTAs that go over longer pieces of a row from L2 instead of
// keeping it: greedy 7 us, top-k of 50 17, but top-p 142, a row's work then being one or two CTAs'.
#include <algorithm>

#include "internal.h"
#include "common.cuh"
#include "sm100.cuh"

namespace eagle {
namespace {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_BINS = 1024;
constexpr int SP_LIST = SP_THREADS;
constexpr int SP_MAX_CLUSTER = 16;
constexpr int SP_RUN = 8 * SP_THREADS;          // tokens a CTA takes with eight a thread
constexpr int SP_MAX_RUNS = 4;

struct SampleParams {
  const void* logits;
  long long ld;
  int vocab;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int rows_each;
  const int32_t* rows_used;
  const uint32_t* u;
  int32_t* token;
  int32_t* argmax;
  float* probs;
  long long ld_probs;
  int cluster;
  int each;                // tokens of a thread
  int* status;
  uint64_t* stamp;
};

__device__ const uint64_t kPow2[64] = {
    0x400000000000ull, 0x3f4f83033d22ull, 0x3ea0ecb6dc8bull, 0x3df437dcc2b4ull, 0x3d495f454922ull, 0x3ca05dcf1680ull,
    0x3bf92e66f737ull, 0x3b53cc07b665ull, 0x3ab031b9f749ull, 0x3a0e5a940f13ull, 0x396e41b9df21ull, 0x38cfe25cafa3ull,
    0x383337bb0aa5ull, 0x37983d209784ull, 0x36feede5f6bdull, 0x366745709e2cull, 0x35d13f32b5a7ull, 0x353cd6aaf3fbull,
    0x34aa07647c4bull, 0x3418ccf6bbcbull, 0x3389230547e1ull, 0x32fb053fbc9dull, 0x326e6f619b8cull, 0x31e35d322aeeull,
    0x3159ca845542ull, 0x30d1b3368926ull, 0x304b1332999cull, 0x2fc5e66d9e9dull, 0x2f4228e7d603ull, 0x2ebfd6ac84d0ull,
    0x2e3eebd1d8bfull, 0x2dbf6478ca34ull, 0x2d413cccfe78ull, 0x2cc47104aa44ull, 0x2c48fd6074abull, 0x2bcede2b5a43ull,
    0x2b560fba90a8ull, 0x2ade8e6d6a50ull, 0x2a6856ad3a9full, 0x29f364ed3a59ull, 0x297fb5aa6c54ull, 0x290d456b827aull,
    0x289c10c0c312ull, 0x282c1443ee5cull, 0x27bd4c982468ull, 0x274fb669cb40ull, 0x26e34e6e7554ull, 0x26781164c82eull,
    0x260dfc14636eull, 0x25a50b4dc806ull, 0x253d3bea3fbeull, 0x24d68acbc4faull, 0x2470f4dceac4ull, 0x240c7710c51aull,
    0x23a90e62d173ull, 0x2346b7d6df97ull, 0x22e57078faa3ull, 0x2285355d525cull, 0x222603a024b7ull, 0x21c7d865a7a3ull,
    0x216ab0d9f312ull, 0x210e8a30eb38ull, 0x20b361a62b0bull, 0x2059347cef01ull,
};

// A power of two as a whole number and as a pair of floats.
struct __align__(16) Pow2 {
  uint64_t whole;
  float hi, lo;
};

// What a CTA tells the others about its part of the row: the largest key and its first id, and whether any logit is NaN
// or +inf.
struct Extent {
  uint32_t top, id, bad, pad;
};
// From this distance on a weight (2^23 or less) needs no more than fp32.
constexpr float SP_FAR = 17.0f;
constexpr uint64_t SP_FAR_WEIGHT = 1ull << 23;   // the largest there

// Number and weight of a CTA's tokens within each of the parts' distances, and the weight of all.
constexpr int SP_PARTS = 4;
struct Parts {
  uint64_t weight[SP_PARTS + 1];
  uint32_t count[SP_PARTS + 1];
};
__device__ __forceinline__ float part_reach(int i) {
  return i == 0 ? 4.0f : i == 1 ? 8.0f : i == 2 ? 12.0f : i == 3 ? SP_FAR : 41.0f;
}

struct SampleShared {
  // bins of this CTA's tokens: how many, and their weight in two words
  alignas(16) uint32_t count[SP_BINS];
  uint32_t lo[SP_BINS], hi[SP_BINS];
  // (first CTA) bins of the whole row; tokens, largest first once sorted: key << 32 | ~id
  uint32_t all_count[SP_BINS];
  uint64_t all_weight[SP_BINS];
  uint64_t list[SP_LIST], kept[SP_LIST];
  Parts parts[SP_MAX_CLUSTER], warp_parts[SP_WARPS];
  Pow2 pow2[64];
  Extent extent[SP_MAX_CLUSTER];
  uint64_t total[SP_MAX_CLUSTER];
  uint64_t warp_total[SP_WARPS];
  uint32_t warp_lo[SP_WARPS], warp_hi[SP_WARPS];
  uint64_t scan[SP_WARPS];
  uint32_t scan_n[SP_WARPS];
  Extent warp_extent[SP_WARPS];
  // a search's state, written by the first CTA to all
  uint32_t near_n;               // near tokens of this CTA
  uint32_t listed;               // tokens in this CTA's list
  uint32_t digit, in_digit;      // where the cut falls, and how many tokens fall there
  uint32_t before_n;             // tokens and weight before it
  uint64_t before_w;
  uint32_t cut_key, cut_id;
  uint64_t need_w;
  uint32_t tie[SP_MAX_CLUSTER];  // tokens of the cut's value in each CTA
};

// The row's constants.
struct Row {
  float top, c_hi, c_lo;
  float from, to, bins;          // the part's distances, and bins of one
};

// (top - z) log2(e) / t to fp32's precision; large for what has no weight at all.
__device__ __forceinline__ float distance(const Row& r, float z) { return fminf((r.top - z) * r.c_hi, 100.0f); }

// The difference to the top and its product with log2(e) / t as pairs of floats: the low part of y, given the high one.
__device__ __forceinline__ float low_part(const Row& r, float z, float dh, float yh) {
  const float bb = dh - r.top;
  const float dl = (r.top - (dh - bb)) - (z + bb);
  return fmaf(dh, r.c_hi, -yh) + fmaf(dh, r.c_lo, dl * r.c_hi);
}

// floor(2^40 2^(-y)) from SP_FAR on, off by two units of 2^23 at most: y to both its parts, exp2 to 2 steps of fp32.
__device__ __forceinline__ uint32_t far_weight(const Row& r, float z) {
  const float dh = r.top - z, yh = dh * r.c_hi;
  const float e = sm100::exp2(40.0f - yh);
  const float x = fmaf(e, -0x1.62e43p-1f * low_part(r, z, dh, yh), e);
  const uint32_t w = __float_as_uint(__fadd_rd(fminf(x, 8388607.0f), 8388608.0f)) & 0x7fffffu;
  return yh < 41.0f ? w : 0u;
}

// floor(2^40 2^(-y)), off by a unit where the fraction is near a border.  The difference to the top and its product with
// log2(e) / t are pairs of floats; y = k / 64 + r, |r| <= 1 / 128, and 2^(-r) - 1 = u + u^2 / 2 + u^3 / 6 + u^4 / 24 with
// u = -r ln 2 (the next term is below 2^-44), the linear term a pair, the rest (2^-16) a float; table entry and product
// then meet in 46-bit fixed point.
__device__ __forceinline__ uint64_t near_weight(const SampleShared& s, const Row& r, float z) {
  constexpr float MAGIC = 12582912.0f;           // 1.5 2^23: the sum's low bits are the rounded integer
  constexpr int MAGIC_BITS = 0x4B400000;
  const float dh = r.top - z;
  const float yh = fminf(dh * r.c_hi, SP_FAR);   // (beyond: not used)
  const float yl = low_part(r, z, dh, yh);
  const float kt = fmaf(yh, 64.0f, MAGIC);
  const int k = __float_as_int(kt) - MAGIC_BITS;
  const float rh = fmaf(kt - MAGIC, -0x1p-6f, yh);
  const float rs = rh + yl, rl = yl - (rs - rh);
  constexpr float LN2_HI = 0x1.62e43p-1f, LN2_LO = -0x1.05c61p-29f;
  const float uh = -rs * LN2_HI;
  const float ul = fmaf(-rs, LN2_HI, -uh) - fmaf(rs, LN2_LO, rl * LN2_HI);
  const float v = fmaf(uh * uh, fmaf(uh, fmaf(uh, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f), ul);
  const Pow2 t = s.pow2[k & 63];
  const float a = t.hi * uh;
  const float b = fmaf(t.hi, uh, -a) + fmaf(t.hi, v, t.lo * uh);
  const float c = a + b, cl = b - (c - a);
  const float c1 = fmaf(c, 0x1p24f, MAGIC);
  const float rem = fmaf(c1 - MAGIC, -0x1p-24f, c) + cl;
  const int64_t w = static_cast<int64_t>(t.whole) +
                    (static_cast<int64_t>(__float_as_int(c1) - MAGIC_BITS) << 22) +
                    (__float_as_int(fmaf(rem, 0x1p46f, MAGIC)) - MAGIC_BITS);
  return static_cast<uint64_t>(w) >> (6 + (k >> 6));
}

__device__ __forceinline__ uint64_t weight(const SampleShared& s, const Row& r, float z) {
  const float y = distance(r, z);
  return y < SP_FAR ? near_weight(s, r, z) : far_weight(r, z);
}

// The weights of four tokens, those not wanted 0 (the whole warp calls it).
__device__ __forceinline__ void weights4(const SampleShared& s, const Row& r, const float (&z)[4], const bool (&wanted)[4],
                                         uint64_t (&w)[4]) {
  float y[4];
  bool near = false;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    y[q] = distance(r, z[q]);
    w[q] = wanted[q] ? far_weight(r, z[q]) : 0;
    near |= wanted[q] && y[q] < SP_FAR;
  }
  if (__any_sync(0xffffffffu, near)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t x = near_weight(s, r, z[q]);
      if (wanted[q] && y[q] < SP_FAR) w[q] = x;
    }
  }
}

__device__ __forceinline__ uint32_t bin_of(const Row& r, float z) {
  return static_cast<uint32_t>(fminf((distance(r, z) - r.from) * r.bins, static_cast<float>(SP_BINS - 1)));
}

// The digit of a search's pass `level`: the bin, then 10, 10, 10 and 2 bits of the logit's order.
__device__ __forceinline__ int key_shift(int level) { return level >= 4 ? 0 : 32 - 10 * level; }
__device__ __forceinline__ uint32_t digit_of(const Row& r, float z, int level) {
  if (level == 0) return bin_of(r, z);
  return (order_key(z) >> key_shift(level)) & (level == 4 ? 3u : SP_BINS - 1u);
}

// Exclusive sums over the block of a pair, in thread order.
__device__ __forceinline__ void block_before(SampleShared& s, uint32_t n, uint64_t w, uint32_t& n0, uint64_t& w0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t in = n;
  uint64_t iw = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, in, o);
    const uint64_t b = __shfl_up_sync(0xffffffffu, iw, o);
    if (lane >= o) in += a, iw += b;
  }
  if (lane == 31) s.scan_n[warp] = in, s.scan[warp] = iw;
  __syncthreads();
  n0 = in - n;
  w0 = iw - w;
#pragma unroll
  for (int i = 0; i < SP_WARPS; ++i)
    if (i < warp) n0 += s.scan_n[i], w0 += s.scan[i];
}

__device__ __forceinline__ void st_all_u32(const SampleParams& p, void* local, uint32_t v) {
  for (int c = 0; c < p.cluster; ++c) sm100::dsmem_st_s32(sm100::dsmem_addr(local, c), static_cast<int>(v));
}
__device__ __forceinline__ void st_all_u64(const SampleParams& p, void* local, uint64_t v) {
  for (int c = 0; c < p.cluster; ++c) sm100::dsmem_st_u64(sm100::dsmem_addr(local, c), v);
}
__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Every thread of the cluster; shared-memory accesses before, local or remote, come before those after.
__device__ __forceinline__ void meet(const SampleParams& p) {
  if (p.cluster > 1) sm100::cluster_sync();
  else __syncthreads();
}

// A CTA's tokens in shared memory.  Token i of thread t is at place i * threads + t and is id base(t) + (i / 8) * 256 +
// i % 8: a warp has a run of consecutive ids.
struct Tokens {
  float* all;
  uint16_t* near;          // places of the near tokens
  int n;                   // tokens of a thread
  int first;               // the CTA's first id
  __device__ __forceinline__ float& z(int i) const { return all[i * SP_THREADS + threadIdx.x]; }
  __device__ __forceinline__ int base(int t) const { return first + (t >> 5) * n * 32 + (t & 31) * 8; }
  __device__ __forceinline__ int id(int i) const { return base(threadIdx.x) + (i >> 3) * 256 + (i & 7); }
  __device__ __forceinline__ int id_at(int place) const {
    const int i = place / SP_THREADS;
    return base(place % SP_THREADS) + (i >> 3) * 256 + (i & 7);
  }
  // Calls f(place, z, there) for every near token (dense) or every token, by whole warps.
  template <typename F>
  __device__ __forceinline__ void each(bool dense, uint32_t near_n, F f) const {
    if (!dense) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) f(i * SP_THREADS + static_cast<int>(threadIdx.x), z(i), true);
      return;
    }
    const uint32_t end = near_n;
#pragma unroll 1
    for (uint32_t at = threadIdx.x; at - (threadIdx.x & 31) < end; at += SP_THREADS) {
      const bool there = at < end;
      const uint32_t place = there ? near[at] : 0;
      f(static_cast<int>(place), all[place], there);
      __syncwarp();
    }
  }
};

// Eight logits from id `at` on, those past the end -inf.
__device__ __forceinline__ void load_logits(const float* row, int at, int vocab, bool wide, float (&z)[8]) {
  if (wide && at + 8 <= vocab) {
    const float4 a = *reinterpret_cast<const float4*>(row + at), b = *reinterpret_cast<const float4*>(row + at + 4);
    z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
    z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = at + i < vocab ? row[at + i] : -INFINITY;
  }
}
__device__ __forceinline__ void load_logits(const uint16_t* row, int at, int vocab, bool wide, float (&z)[8]) {
  if (wide && at + 8 <= vocab) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + at);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = __uint_as_float(u[i] << 16);
      z[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = at + i < vocab ? bf16_to_f32(row[at + i]) : -INFINITY;
  }
}

// Sums the CTAs' bins into the first CTA's all_*.
__device__ __forceinline__ void sum_bins(const SampleParams& p, SampleShared& s, bool weighted, uint32_t rank) {
  meet(p);
  const int slice = SP_BINS / p.cluster;
  for (int b = static_cast<int>(rank) * slice + threadIdx.x; b < (static_cast<int>(rank) + 1) * slice; b += SP_THREADS) {
    uint32_t n = 0;
    uint64_t sum = 0;
#pragma unroll 4
    for (int c = 0; c < p.cluster; ++c) {
      n += dsmem_ld_u32(sm100::dsmem_addr(&s.count[b], c));
      if (weighted)
        sum += (static_cast<uint64_t>(dsmem_ld_u32(sm100::dsmem_addr(&s.hi[b], c))) << 32) +
               dsmem_ld_u32(sm100::dsmem_addr(&s.lo[b], c));
    }
    sm100::dsmem_st_s32(sm100::dsmem_addr(&s.all_count[b], 0), static_cast<int>(n));
    if (weighted) sm100::dsmem_st_u64(sm100::dsmem_addr(&s.all_weight[b], 0), sum);
  }
  meet(p);
}

// Where the count or the weight reaches `need` in the first CTA's bins (rising: in their order, else from the last down):
// digit, in_digit (0: nowhere), before_n and before_w of every CTA, the latter on top of those given.
__device__ __forceinline__ void scan_bins(const SampleParams& p, SampleShared& s, bool by_weight, bool rising, uint64_t need,
                                          uint32_t before_n, uint64_t before_w, uint32_t rank) {
  if (rank == 0) {
    constexpr int OWN = SP_BINS / SP_THREADS;
    uint32_t n = 0, cn[OWN];
    uint64_t sum = 0, cw[OWN];
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
      const int at = threadIdx.x * OWN + q, b = rising ? at : SP_BINS - 1 - at;
      cn[q] = s.all_count[b];
      cw[q] = by_weight ? s.all_weight[b] : 0;
      n += cn[q];
      sum += cw[q];
    }
    uint32_t n0;
    uint64_t w0;
    block_before(s, n, sum, n0, w0);
    n0 += before_n;
    w0 += before_w;
    if (threadIdx.x == SP_THREADS - 1 && (by_weight ? w0 + sum : n0 + n) < need) st_all_u32(p, &s.in_digit, 0);
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
      if (by_weight ? w0 < need && w0 + cw[q] >= need : n0 < need && n0 + cn[q] >= need) {
        const int at = threadIdx.x * OWN + q;
        st_all_u32(p, &s.digit, rising ? at : SP_BINS - 1 - at);
        st_all_u32(p, &s.in_digit, cn[q]);
        st_all_u32(p, &s.before_n, n0);
        st_all_u64(p, &s.before_w, w0);
      }
      n0 += cn[q];
      w0 += cw[q];
    }
  }
  meet(p);
}

// The chosen tokens (near ones alone where dense) of all CTAs into the first one's list; how many there are (to every
// CTA), none gathered where they pass SP_LIST.
template <typename Chosen>
__device__ __forceinline__ uint32_t gather(const SampleParams& p, SampleShared& s, const Tokens& tk, bool dense,
                                           uint32_t rank, Chosen chosen) {
  if (threadIdx.x == 0) s.listed = 0;
  __syncthreads();
  tk.each(dense, s.near_n, [&](int place, float z, bool there) {
    if (there && chosen(z)) {
      const uint32_t at = atomicAdd(&s.listed, 1u);
      if (at < SP_LIST)
        s.list[at] = static_cast<uint64_t>(order_key(z)) << 32 | (0xffffffffu - static_cast<uint32_t>(tk.id_at(place)));
    }
  });
  if (p.cluster == 1) {
    __syncthreads();
    return s.listed;
  }
  meet(p);
  uint32_t at = 0;                               // this CTA's place, and all
  uint32_t n = 0;
  for (int c = 0; c < p.cluster; ++c) {
    const uint32_t x = dsmem_ld_u32(sm100::dsmem_addr(&s.listed, c));
    if (c < static_cast<int>(rank)) at += x;
    n += x;
  }
  if (n <= SP_LIST && rank > 0)
    for (uint32_t i = threadIdx.x; i < s.listed; i += SP_THREADS)
      sm100::dsmem_st_u64(sm100::dsmem_addr(&s.list[at + i], 0), s.list[i]);
  meet(p);
  return n;
}

// Sorts the threads' e, the first n of them other than 0, largest first: a bitonic network, by shuffles where partners
// share a warp, else over s.list, by as many warps as it takes.
__device__ __forceinline__ void sort_threads(SampleShared& s, int n, uint64_t& e) {
  const int t = threadIdx.x;
  int width = 32;
  while (width < n) width <<= 1;
  if (t >= width) return;
#pragma unroll 1
  for (int size = 2; size <= width; size <<= 1) {
#pragma unroll 1
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      uint64_t o;
      if (stride < 32) {
        o = __shfl_xor_sync(0xffffffffu, e, stride);
      } else {
        sm100::named_barrier(1, width);
        s.list[t] = e;
        sm100::named_barrier(1, width);
        o = s.list[t ^ stride];
      }
      const bool larger = ((t & stride) == 0) == ((t & size) == 0);   // of the two, this thread keeps the larger
      e = (e > o) == larger ? e : o;
    }
  }
}

// Sorts the n <= SP_LIST tokens of this CTA's list, largest first: thread t gets the t-th and its weight, and the weight
// before it.
__device__ __forceinline__ void sort_list(SampleShared& s, const Row& r, int n, uint64_t& e, uint64_t& w, uint64_t& before) {
  e = static_cast<int>(threadIdx.x) < n ? s.list[threadIdx.x] : 0;
  sort_threads(s, n, e);
  w = e ? weight(s, r, key_value(static_cast<uint32_t>(e >> 32))) : 0;
  uint32_t none;
  block_before(s, 0, w, none, before);
}

__device__ __forceinline__ void tell_cut(const SampleParams& p, SampleShared& s, uint64_t e) {
  st_all_u32(p, &s.cut_key, static_cast<uint32_t>(e >> 32));
  st_all_u32(p, &s.cut_id, 0xffffffffu - static_cast<uint32_t>(e));
}

// ceil(p S), at least 1 and at most S < 2^60: the 24 bits of p times S, shifted down.
__device__ __forceinline__ uint64_t needed(float top_p, uint64_t all) {
  if (!(top_p > 0.0f)) return 1;
  const uint32_t bits = __float_as_uint(top_p), e = bits >> 23;
  const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int sh = 150 - static_cast<int>(e ? e : 1u);             // top_p = m 2^-sh, sh >= 24
  const uint64_t lo = m * all, hi = __umul64hi(m, all);
  uint64_t need, rest;
  if (sh < 64) {
    need = (hi << (64 - sh)) | (lo >> sh);
    rest = lo & ((1ull << sh) - 1);
  } else {
    need = sh < 128 ? hi >> (sh - 64) : 0;
    rest = lo | hi;                              // (need is 0 or small: one more at most)
    if (sh < 128 && sh > 64) rest = lo | (hi & ((1ull << (sh - 64)) - 1));
    if (sh == 64) rest = lo;
  }
  need += rest ? 1 : 0;
  return need < 1 ? 1 : min(need, all);
}

// The cut in the part of the row at distances r.from to r.to, by counting: where the number (by_weight false) or the
// weight of the tokens, on top of those before the part, reaches `need`.  cut_key and cut_id of every CTA; cut_key 0 where
// it never does.
__device__ __noinline__ void count_cut(const SampleParams& p, SampleShared& s, Row r, const Tokens tk, bool by_weight,
                                       uint64_t need, uint32_t before_n, uint64_t before_w, uint32_t rank) {
  uint32_t bin = 0, prefix = 0, there = 0;
  int level = 0;
  r.bins = static_cast<float>(SP_BINS) / (r.to - r.from);
  const bool dense = r.to <= SP_FAR;
  auto chosen = [&](float z) {
    const float y = distance(r, z);
    if (!(y < r.to) || y < r.from) return false;
    if (level == 0) return true;
    if (bin_of(r, z) != bin) return false;
    return level == 1 || order_key(z) >> key_shift(level - 1) == prefix;
  };
  do {
    for (int b = threadIdx.x; b < SP_BINS; b += SP_THREADS) s.count[b] = s.lo[b] = s.hi[b] = 0;
    __syncthreads();
    tk.each(dense, s.near_n, [&](int, float z, bool there) {
      if (!there || !chosen(z)) return;
      const uint32_t d = digit_of(r, z, level);
      atomicAdd(&s.count[d], 1u);
      if (by_weight) {
        const uint64_t wi = weight(s, r, z);
        const uint32_t l = static_cast<uint32_t>(wi), old = atomicAdd(&s.lo[d], l);
        const uint32_t h = static_cast<uint32_t>(wi >> 32) + (old + l < old ? 1u : 0u);
        if (h) atomicAdd(&s.hi[d], h);
      }
    });
    sum_bins(p, s, by_weight, rank);
    // the digits in falling order of z: bins as they are, bits from the largest down
    scan_bins(p, s, by_weight, level == 0, need, before_n, before_w, rank);
    there = s.in_digit;
    if (there == 0) {
      if (threadIdx.x == 0) s.cut_key = 0;
      meet(p);
      return;
    }
    before_n = s.before_n;
    before_w = s.before_w;
    if (level == 0) bin = s.digit;
    else prefix = level == 4 ? prefix << 2 | s.digit : prefix << 10 | s.digit;
    ++level;
    meet(p);                                     // the state is read before the next pass writes it
  } while (there > SP_LIST && level < 5);
  if (there <= SP_LIST) {
    gather(p, s, tk, dense, rank, chosen);
    if (rank == 0) {
      uint64_t e, w, before;
      sort_list(s, r, static_cast<int>(there), e, w, before);
      before += before_w;
      if (e && (by_weight ? before < need && before + w >= need : before_n + threadIdx.x + 1 == need)) tell_cut(p, s, e);
    }
    meet(p);
    return;
  }
  // Tokens of one value, more than the list takes: the cut is the m-th of them by id.
  const uint64_t one = weight(s, r, key_value(prefix));
  const uint32_t m = by_weight ? static_cast<uint32_t>((need - before_w + one - 1) / one)
                               : static_cast<uint32_t>(need) - before_n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t mine = 0;
#pragma unroll 1
  for (int i = 0; i < tk.n; ++i) mine += chosen(tk.z(i)) ? 1u : 0u;
  const uint32_t in_warp = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) s.scan_n[warp] = in_warp;
  __syncthreads();
  uint32_t before = 0, in_cta = 0;
  for (int i = 0; i < SP_WARPS; ++i) {
    if (i < warp) before += s.scan_n[i];
    in_cta += s.scan_n[i];
  }
  if (threadIdx.x == 0) st_all_u32(p, &s.tie[rank], in_cta);
  meet(p);
  for (uint32_t c = 0; c < rank; ++c) before += s.tie[c];
  if (before < m && before + in_warp >= m) {     // in this warp: its runs of 256 ids, then its lanes, then a lane's eight
#pragma unroll 1
    for (int j = 0; j < tk.n / 8; ++j) {
      uint32_t bits = 0;
#pragma unroll 1
      for (int i = 0; i < 8; ++i)
        if (chosen(tk.z(8 * j + i))) bits |= 1u << i;
      uint32_t c = static_cast<uint32_t>(__popc(bits)), upto = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      uint32_t k = before + upto - c;
#pragma unroll 1
      for (int i = 0; i < 8; ++i)
        if (bits >> i & 1u) {
          if (++k == m)
            tell_cut(p, s, static_cast<uint64_t>(prefix) << 32 | (0xffffffffu - static_cast<uint32_t>(tk.id(8 * j + i))));
        }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  meet(p);
}

// Gathers the tokens that may be among the row's k largest into the first CTA's list, by a thread's largest, `mine`; how
// many there are (0: too many, or too few).  With few tokens to keep each CTA bounds them by its own threads' largest
// (up to k tokens and some more a CTA are gathered), else all do together.
__device__ __forceinline__ uint32_t gather_top(const SampleParams& p, SampleShared& s, Row r, const Tokens& tk, float mine,
                                               uint32_t k, uint32_t rank) {
  r.from = 0.0f;
  r.to = 41.0f;
  r.bins = static_cast<float>(SP_BINS) / 41.0f;
  for (int b = threadIdx.x; b < SP_BINS; b += SP_THREADS) s.count[b] = 0;
  __syncthreads();
  if (distance(r, mine) < r.to) atomicAdd(&s.count[bin_of(r, mine)], 1u);
  if (k * static_cast<uint32_t>(p.cluster) <= SP_LIST / 2) {
    if (threadIdx.x == 0) s.digit = SP_BINS - 1;   // fewer than k: all that have weight
    __syncthreads();
    const uint2 two = *reinterpret_cast<const uint2*>(&s.count[2 * threadIdx.x]);
    static_assert(SP_BINS == 2 * SP_THREADS, "two bins a thread");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t upto = two.x + two.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) s.scan_n[warp] = upto;
    __syncthreads();
    uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? s.scan_n[lane] : 0u);
    before += upto - two.x - two.y;
    if (before < k && before + two.x >= k) s.digit = 2 * threadIdx.x;
    else if (before + two.x < k && before + two.x + two.y >= k) s.digit = 2 * threadIdx.x + 1;
    __syncthreads();
  } else {
    sum_bins(p, s, false, rank);
    scan_bins(p, s, false, true, k, 0, 0, rank);
    if (s.in_digit == 0) {
      meet(p);                                   // (the state is read)
      return 0;
    }
  }
  const float end = static_cast<float>(s.digit + 1);
  const uint32_t n = gather(p, s, tk, false, rank, [&](float z) { return distance(r, z) < 41.0f && distance(r, z) * r.bins < end; });
  return n >= k && n <= SP_LIST ? n : 0;
}

// The cut of top-p: where the weight reaches `need` (0: top_p of the weight of all).
// far: the weight of this thread's other than near tokens (32 of 2^23 at most).
__device__ __forceinline__ void top_p_cut(const SampleParams& p, SampleShared& s, Row r, const Tokens& tk, uint32_t far,
                                          uint64_t need, float top_p, uint32_t rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t n[SP_PARTS] = {0, 0, 0, 0};
  uint64_t w[SP_PARTS] = {0, 0, 0, 0};
  tk.each(true, s.near_n, [&](int, float z, bool there) {
    const float y = there ? distance(r, z) : 100.0f;
    const uint64_t x = near_weight(s, r, z);
#pragma unroll
    for (int c = 0; c < SP_PARTS; ++c)
      if (y < part_reach(c)) w[c] += x, ++n[c];
  });
#pragma unroll
  for (int c = 0; c < SP_PARTS; ++c) {
    n[c] = __reduce_add_sync(0xffffffffu, n[c]);
    w[c] = n[c] ? warp_sum_u64(w[c]) : 0;
  }
  const uint64_t far_all = warp_sum_u64(far);
  if (lane == 0) {
    Parts& x = s.warp_parts[warp];
#pragma unroll
    for (int c = 0; c < SP_PARTS; ++c) x.weight[c] = w[c], x.count[c] = n[c];
    x.weight[SP_PARTS] = w[SP_PARTS - 1] + far_all;
    x.count[SP_PARTS] = 0;
  }
  __syncthreads();
  if (threadIdx.x <= SP_PARTS) {                 // a thread a part, told to every CTA
    const int c = threadIdx.x;
    uint64_t a = 0;
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < SP_WARPS; ++i) a += s.warp_parts[i].weight[c], b += s.warp_parts[i].count[c];
    st_all_u64(p, &s.parts[rank].weight[c], a);
    st_all_u32(p, &s.parts[rank].count[c], b);
  }
  meet(p);
  // the first part whose weight, with those before it, reaches what is needed: a lane a part
  uint64_t a = 0;
  uint32_t b = 0;
  if (lane <= SP_PARTS)
    for (int c = 0; c < p.cluster; ++c) a += s.parts[c].weight[lane], b += s.parts[c].count[lane];
  if (need == 0) need = needed(top_p, __shfl_sync(0xffffffffu, a, SP_PARTS));
  const uint32_t enough = __ballot_sync(0xffffffffu, lane < SP_PARTS && a >= need) | 1u << SP_PARTS;
  const int part = __ffs(enough) - 1, last = max(part - 1, 0);
  const uint64_t before_w = part ? __shfl_sync(0xffffffffu, a, last) : 0;
  const uint32_t before_n = part ? __shfl_sync(0xffffffffu, b, last) : 0;
  const uint32_t upto = __shfl_sync(0xffffffffu, b, part);
  const uint32_t there = part < SP_PARTS ? upto - before_n : 0xffffffffu;
  r.from = part ? part_reach(last) : 0.0f;
  r.to = part_reach(part);
  if (there > SP_LIST) {
    count_cut(p, s, r, tk, true, need, before_n, before_w, rank);
    return;
  }
  gather(p, s, tk, true, rank, [&](float z) {
    const float y = distance(r, z);
    return y < r.to && y >= r.from;
  });
  if (rank == 0) {
    uint64_t e, we, before;
    sort_list(s, r, static_cast<int>(there), e, we, before);
    before += before_w;
    if (e && before < need && before + we >= need) tell_cut(p, s, e);
  }
  meet(p);
}

__device__ __forceinline__ void store_probs(float* row, int id, int vocab, bool wide, const float (&v)[8]) {
  if (wide && id + 8 <= vocab) {
    *reinterpret_cast<float4*>(row + id) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(row + id + 4) = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (id + i < vocab) row[id + i] = v[i];
}

template <typename T>
__global__ void __launch_bounds__(SP_THREADS, 2) sample_kernel(SampleParams p) {
  extern __shared__ __align__(16) uint8_t raw_shared[];
  SampleShared& s = *reinterpret_cast<SampleShared*>(raw_shared);
  LaunchStamp ls(p.stamp);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x / p.cluster;
  const uint32_t rank = p.cluster > 1 ? sm100::cluster_rank() : 0;
  if (threadIdx.x < 64) {
    const uint64_t v = kPow2[threadIdx.x];
    const float h = static_cast<float>(v);
    s.pow2[threadIdx.x] =
        Pow2{v, h * 0x1p-46f, static_cast<float>(static_cast<int64_t>(v) - static_cast<int64_t>(h)) * 0x1p-46f};
  }
  if (threadIdx.x == 0) s.near_n = 0;
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int request = row / p.rows_each;
  if (p.rows_used && row - request * p.rows_each >= p.rows_used[request]) return;
  if (p.cluster > 1) sm100::cluster_arrive_relaxed();   // (the others are there before anything is written to them)
  const float temp = p.temperature ? p.temperature[request] : 1.0f;
  const int k = p.top_k ? p.top_k[request] : 0;
  const float top_p = p.top_p ? p.top_p[request] : 1.0f;
  const float min_p = p.min_p ? fminf(p.min_p[request], 1.0f) : 0.0f;
  const uint32_t u = p.token ? p.u[row] : 0;
  const bool greedy = !(temp > 0.0f);

  const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
  const bool wide = (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  Tokens tk;
  tk.all = reinterpret_cast<float*>(raw_shared + sizeof(SampleShared));
  tk.n = p.each;
  tk.near = reinterpret_cast<uint16_t*>(tk.all + tk.n * SP_THREADS);
  tk.first = static_cast<int>(rank) * tk.n * SP_THREADS;
  const int id0 = tk.base(threadIdx.x);
  // the largest logit, and whether any is NaN or +inf
  float top = -INFINITY;                         // NaN if any is
#pragma unroll 2
  for (int j = 0; j < tk.n / 8; ++j) {
    float z[8];
    load_logits(logits, id0 + j * 256, p.vocab, wide, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      tk.z(8 * j + i) = z[i];
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(z[i]));
    }
  }
  {
    const uint32_t key = order_key(top), warp_top = __reduce_max_sync(0xffffffffu, key);
    uint32_t id = 0xffffffffu;
    if (p.argmax || greedy) {
      if (key == warp_top) {
#pragma unroll 1
        for (int i = tk.n - 1; i >= 0; --i)
          if (tk.z(i) == top) id = static_cast<uint32_t>(tk.id(i));
      }
      id = __reduce_min_sync(0xffffffffu, id);
    }
    const bool any = __any_sync(0xffffffffu, !(top < INFINITY));
    if (lane == 0) s.warp_extent[warp] = Extent{warp_top, id, any ? 1u : 0u, 0u};
  }
  __syncthreads();
  if (warp == 0) {
    Extent e = s.warp_extent[lane % SP_WARPS];
    const uint32_t t = __reduce_max_sync(0xffffffffu, e.top);
    e.id = __reduce_min_sync(0xffffffffu, e.top == t ? e.id : 0xffffffffu);
    e.bad = __reduce_or_sync(0xffffffffu, e.bad);
    if (p.cluster > 1) sm100::cluster_wait();
    if (lane < p.cluster) {
      const uint32_t a = sm100::dsmem_addr(&s.extent[rank], lane);
      sm100::dsmem_st_u64(a, t | (static_cast<uint64_t>(e.id) << 32));
      sm100::dsmem_st_u64(a + 8, e.bad);
    }
    __syncwarp();
  } else if (p.cluster > 1) {
    sm100::cluster_wait();
  }
  meet(p);
  Extent all{0, 0xffffffffu, 0, 0};
  for (int c = 0; c < p.cluster; ++c) {
    const Extent e = s.extent[c];
    if (e.top > all.top) all.top = e.top, all.id = e.id;
    all.bad |= e.bad;
  }
  const float zmax = key_value(all.top);
  const bool none = all.bad || !(zmax > -INFINITY);
  float* probs = p.probs ? p.probs + row * p.ld_probs : nullptr;
  const bool wide_out = (reinterpret_cast<uintptr_t>(probs) & 15) == 0;
  if (threadIdx.x == 0 && rank == 0) {
    if (p.argmax) p.argmax[row] = none ? -1 : static_cast<int32_t>(all.id);
    if (none) set_status(p.status, EAGLE_ERR_NUMERIC);
    if ((none || greedy) && p.token) p.token[row] = none ? -1 : static_cast<int32_t>(all.id);
  }
  auto write_probs = [&]() {
#pragma unroll 1
    for (int j = 0; j < tk.n / 8; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = tk.z(8 * j + i);
      store_probs(probs, id0 + j * 256, p.vocab, wide_out, v);
    }
  };
  if (none || greedy) {
    if (probs) {
#pragma unroll 4
      for (int i = 0; i < tk.n; ++i) tk.z(i) = !none && static_cast<uint32_t>(tk.id(i)) == all.id ? 1.0f : 0.0f;
      write_probs();
    }
    return;
  }
  if (!p.token && !probs) return;

  Row r;
  r.top = zmax;
  {
    // log2(e) / t as a pair of floats: the quotient and, over t, what it leaves
    constexpr float LOG2E_HI = 0x1.715476p+0f, LOG2E_LO = 0x1.4ae0cp-26f;
    const float t = fmaxf(temp, 1e-30f);
    r.c_hi = LOG2E_HI / t;
    r.c_lo = (fmaf(-r.c_hi, t, LOG2E_HI) + LOG2E_LO) / t;
    if (!(t < 1e30f)) r.c_lo = 0.0f;
  }
  r.from = r.to = r.bins = 0.0f;
  const bool by_k = k > 0 && k < p.vocab;
  float cut_z = -INFINITY;
  uint32_t cut_id = 0xffffffffu;
  const uint64_t least = min_p > 0.0f ? static_cast<uint64_t>(ceilf(min_p * 0x1p40f)) : 1;
  // the weights of tokens i to i + 3 where the cut (and `floor`) keeps them
  auto kept4 = [&](int i, uint64_t floor, uint64_t (&w)[4]) {
    float z[4];
    bool in[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      z[q] = tk.z(i + q);
      in[q] = z[q] > cut_z || (z[q] == cut_z && static_cast<uint32_t>(tk.id(i + q)) <= cut_id);
    }
    w[0] = w[1] = w[2] = w[3] = 0;
    if (!__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) return;
    weights4(s, r, z, in, w);
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = w[q] >= floor ? w[q] : 0;
  };
  // the weight of what is kept: before this warp, in it, and in the row
  uint64_t before = 0, in_warp = 0, W = 0;
  auto add_up = [&]() {                          // from s.warp_total
    __syncthreads();
    uint64_t in_cta = 0;
    before = 0;
#pragma unroll
    for (int i = 0; i < SP_WARPS; ++i) {
      const uint64_t t = s.warp_total[i];
      if (i < warp) before += t;
      in_cta += t;
    }
    in_warp = s.warp_total[warp];
    if (threadIdx.x == 0) st_all_u64(p, &s.total[rank], in_cta);
    meet(p);
    W = 0;
    for (int c = 0; c < p.cluster; ++c) {
      if (c < static_cast<int>(rank)) before += s.total[c];
      W += s.total[c];
    }
  };
  auto take_cut = [&]() {
    if (s.cut_key != 0) {
      cut_z = key_value(s.cut_key);
      cut_id = s.cut_id;
    }
  };
  if (by_k) {
    const uint32_t n = gather_top(p, s, r, tk, top, static_cast<uint32_t>(k), rank);
    if (n) {                                     // the first CTA has all that is kept
      if (probs) {
#pragma unroll 1
        for (int j = 0; j < tk.n / 8; ++j) {
          const float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
          store_probs(probs, id0 + j * 256, p.vocab, wide_out, v);
        }
        meet(p);
      }
      if (rank > 0) return;
      const int t = threadIdx.x;
      uint64_t e, w, before_t;
      sort_list(s, r, static_cast<int>(n), e, w, before_t);
      bool in = t < k;
      if (top_p < 1.0f) {
        if (t + 1 == k) s.need_w = needed(top_p, before_t + w);   // of the weight up to the k-th
        __syncthreads();
        in = in && before_t < s.need_w;
      }
      in = in && w >= least;
      // those kept by their ids
      s.kept[t] = in ? w : 0;
      e = in ? (e << 32) | static_cast<uint32_t>(SP_THREADS - 1 - t) : 0;
      __syncthreads();
      sort_threads(s, static_cast<int>(n), e);
      w = e ? s.kept[SP_THREADS - 1 - static_cast<uint32_t>(e)] : 0;
      uint32_t none;
      __syncthreads();
      block_before(s, 0, w, none, before_t);
      if (t == SP_THREADS - 1) s.need_w = before_t + w;
      __syncthreads();
      const uint64_t W = s.need_w, at = scale_uniform(u, W);
      if (w) {
        const int token = static_cast<int>(0xffffffffu - static_cast<uint32_t>(e >> 32));
        if (p.token && before_t <= at && at < before_t + w) p.token[row] = token;
        if (probs) probs[token] = static_cast<float>(w) * (1.0f / static_cast<float>(W));
      }
      return;
    }
  }
  // the near tokens' places; the weight of this thread's others where all may count
  bool by_p = top_p < 1.0f;
  const bool want_far = !by_k && (by_p || least <= 1);
  uint32_t far = 0;
#pragma unroll 4
  for (int i = 0; i < tk.n; ++i) {
    const float z = tk.z(i);
    const bool near = distance(r, z) < SP_FAR;
    const uint32_t who = __ballot_sync(0xffffffffu, near);
    if (want_far) far += near ? 0u : far_weight(r, z);
    if (who) {
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&s.near_n, static_cast<uint32_t>(__popc(who)));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
      if (near) tk.near[at] = static_cast<uint16_t>(i * SP_THREADS + threadIdx.x);
    }
  }
  __syncthreads();
  // whether the cut keeps the token at a place, and its weight; a token too far for `floor` needs no weight
  auto kept_at = [&](int place, float z, uint64_t floor, float reach) -> uint64_t {
    if (distance(r, z) > reach || z < cut_z || (z == cut_z && static_cast<uint32_t>(tk.id_at(place)) > cut_id)) return 0;
    const uint64_t wi = near_weight(s, r, z);
    return wi >= floor ? wi : 0;
  };
  // the weight of what is kept, in s.warp_total by the warps that have the tokens: `others`, this thread's far ones, and
  // the near ones from the list
  auto weigh = [&](uint32_t others, uint64_t floor, float reach) {
    const uint64_t t = warp_sum_u64(others);
    if (lane == 0) s.warp_lo[warp] = static_cast<uint32_t>(t), s.warp_hi[warp] = static_cast<uint32_t>(t >> 32);
    __syncthreads();
    tk.each(true, s.near_n, [&](int place, float z, bool there) {
      const uint64_t wi = there ? kept_at(place, z, floor, reach) : 0;
      if (wi) {
        const int owner = (place % SP_THREADS) >> 5;
        const uint32_t l = static_cast<uint32_t>(wi), old = atomicAdd(&s.warp_lo[owner], l);
        const uint32_t h = static_cast<uint32_t>(wi >> 32) + (old + l < old ? 1u : 0u);
        if (h) atomicAdd(&s.warp_hi[owner], h);
      }
    });
    __syncthreads();
    if (threadIdx.x < SP_WARPS)
      s.warp_total[threadIdx.x] = static_cast<uint64_t>(s.warp_hi[threadIdx.x]) << 32 | s.warp_lo[threadIdx.x];
    add_up();
  };
  // this thread's far tokens that the cut keeps
  auto far_kept = [&](uint64_t floor) {
    uint32_t sum = 0;
    if (distance(r, cut_z) < SP_FAR) return sum;
#pragma unroll 2
    for (int i = 0; i < tk.n; ++i) {
      const float z = tk.z(i);
      const bool in = !(distance(r, z) < SP_FAR) && (z > cut_z || (z == cut_z && static_cast<uint32_t>(tk.id(i)) <= cut_id));
      const uint32_t wi = far_weight(r, z);
      sum += in && wi >= floor ? wi : 0u;
    }
    return sum;
  };
  if (by_k) {
    Row whole = r;
    whole.from = 0.0f;
    whole.to = 41.0f;
    count_cut(p, s, whole, tk, false, static_cast<uint64_t>(k), 0, 0, rank);
    take_cut();
    if (by_p) {                                  // the weight of those k
      weigh(far_kept(1), 1, SP_FAR);
      meet(p);                                   // (s.total and s.cut_* are read)
      top_p_cut(p, s, r, tk, 0, needed(top_p, W), top_p, rank);
      take_cut();
    }
  } else if (by_p) {
    top_p_cut(p, s, r, tk, far, 0, top_p, rank);
    take_cut();
  }
  // min_p's reach, generously
  const float reach = least > 1 ? 40.01f - log2f(static_cast<float>(least)) : SP_FAR;
  const bool far_too = least <= SP_FAR_WEIGHT && !(distance(r, cut_z) < SP_FAR);
  weigh(!far_too ? 0u : want_far && !by_p ? far : far_kept(least), least, reach);
  if (p.token) {
    const uint64_t at = scale_uniform(u, W);
    if (before <= at && at < before + in_warp) {
#pragma unroll 1
      for (int i = 0; i < tk.n; i += 8) {
        uint64_t w[8];
        kept4(i, least, reinterpret_cast<uint64_t(&)[4]>(w[0]));
        kept4(i + 4, least, reinterpret_cast<uint64_t(&)[4]>(w[4]));
        uint64_t mine = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) mine += w[q];
        uint64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        uint64_t sofar = before + upto - mine;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (sofar <= at && at < sofar + w[q]) p.token[row] = tk.id(i + q);
          sofar += w[q];
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  if (probs) {
    const float inv = 1.0f / static_cast<float>(W);
#pragma unroll 1
    for (int j = 0; j < tk.n / 8; ++j) {         // the far tokens' (zeros, where none is kept), then the near ones'
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (far_too) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = tk.z(8 * j + i);
          const uint32_t wi = far_weight(r, z);
          const bool in = z > cut_z || (z == cut_z && static_cast<uint32_t>(tk.id(8 * j + i)) <= cut_id);
          v[i] = in && wi >= least ? static_cast<float>(wi) * inv : 0.0f;
        }
      }
      store_probs(probs, id0 + j * 256, p.vocab, wide_out, v);
    }
    __syncthreads();
    tk.each(true, s.near_n, [&](int place, float z, bool there) {
      const uint64_t wi = there ? kept_at(place, z, least, reach) : 0;
      if (wi) probs[tk.id_at(place)] = static_cast<float>(wi) * inv;
      else if (there && far_too) probs[tk.id_at(place)] = 0.0f;
    });
  }
}

typedef void (*SampleKernel)(SampleParams);
}  // namespace

cudaError_t launch_sample(eagle_ctx* ctx, const SampleLaunch& S, cudaStream_t st) {
  SampleParams p{};
  p.logits = S.logits;
  p.ld = S.ld;
  p.vocab = S.vocab;
  p.temperature = S.filter->temperature;
  p.top_k = S.filter->top_k;
  p.top_p = S.filter->top_p;
  p.min_p = S.filter->min_p;
  p.rows_each = S.filter->rows_each;
  p.rows_used = S.filter->rows_used;
  p.u = S.u;
  p.token = S.token;
  p.argmax = S.argmax;
  p.probs = S.probs;
  p.ld_probs = S.ld_probs;
  p.status = S.status;
  // A CTA takes 4096 or 8192 tokens, two CTAs an SM, or 16384, one: whichever gets through the rows in the least time, a
  // round of CTAs counting its tokens and as much again as 8192 for its exchanges.
  int runs = 0;
  auto clusters = [&](int n) {
    int c = 1;
    while (c * SP_RUN * n < S.vocab) c <<= 1;
    return c;
  };
  long long best = 0;
  for (int n = 1; n <= SP_MAX_RUNS; n <<= 1) {
    if (clusters(n) > SP_MAX_CLUSTER) continue;
    const int slots = (n == SP_MAX_RUNS ? 1 : 2) * ctx->sm_count;
    const long long rounds = (static_cast<long long>(clusters(n)) * S.rows + slots - 1) / slots;
    if (runs == 0 || rounds * (n + 2) < best) {
      runs = n;
      best = rounds * (n + 2);
    }
  }
  p.cluster = clusters(runs);
  p.each = 8 * runs;
  const SampleKernel k = S.dtype == EAGLE_DTYPE_F32 ? sample_kernel<float> : sample_kernel<uint16_t>;
  const size_t smem = sizeof(SampleShared) + static_cast<size_t>(runs) * SP_RUN * 6;
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(k),
                                  static_cast<int>(sizeof(SampleShared) + static_cast<size_t>(SP_MAX_RUNS) * SP_RUN * 6));
  if (e != cudaSuccess) return e;
  if (p.cluster > 8) {
    e = cluster_nonportable_once(reinterpret_cast<const void*>(k));
    if (e != cudaSuccess) return e;
  }
  p.stamp = stamp_slot(ctx, EAGLE_K_SAMPLE);
  trace_before(ctx, EAGLE_K_SAMPLE, st);
  const dim3 grid(static_cast<unsigned>(S.rows) * p.cluster);
  e = p.cluster > 1 ? launch_pdl_cluster(k, grid, dim3(SP_THREADS), smem, st, p.cluster, p)
                    : launch_pdl(k, grid, dim3(SP_THREADS), smem, st, p);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_SAMPLE, st);
  return e;
}

}  // namespace eagle
