// eagle_sample: a row's distribution under temperature, top-k, top-p and min-p, and a draw from it.
//
// A cluster of CTAs holds a row: its logits in registers, its weights floor(2^40 e^((z - max) / t)) in shared memory, so
// that the logits are read once.  Weights are whole numbers and sums of them exact, so the order of sums does not
// matter and a border is where the definition has it.
//
// The cut (the last token in falling order that top-k or top-p keeps) is found by counting: a histogram of 2048 bins of
// equal width over the logits' range, with the number and the weight of the tokens in each, summed over the cluster (a
// slice of the bins a CTA) and scanned by its first CTA; the tokens of the bin in which the cut falls go into a list
// there, whose members count those before them.  A bin with more tokens than the list takes is split by the bits of the
// logits, 11 at a time, and tokens of one value by their ids.
#include <algorithm>

#include "internal.h"
#include "common.cuh"
#include "sm100.cuh"

namespace eagle {
namespace {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_BINS = 2048;
constexpr int SP_LIST = 1024;
constexpr int SP_MAX_CLUSTER = 16;

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
  int* status;
  uint64_t* stamp;
};

// 2^(-j / 64) 2^46
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

struct Listed {
  uint32_t key, id;
  uint64_t w;
};

// What a CTA tells the others about its part of the row.
struct Extent {
  uint32_t top, id, low, bad;
};

struct SampleShared {
  // bins of this CTA's tokens: how many, and their weight in two words
  uint32_t count[SP_BINS], lo[SP_BINS], hi[SP_BINS];
  // (first CTA) bins of the whole row
  uint32_t all_count[SP_BINS];
  uint64_t all_weight[SP_BINS];
  Listed list[SP_LIST];
  uint64_t pow2[64];
  float2 pow2f[64];
  Extent extent[SP_MAX_CLUSTER];
  uint64_t total[SP_MAX_CLUSTER];
  uint64_t warp_total[SP_WARPS];
  uint64_t scan[SP_WARPS];
  uint32_t scan_n[SP_WARPS];
  Extent warp_extent[SP_WARPS];
  float c_hi, c_lo;
  // a search's state, written by the first CTA to all
  uint32_t listed;               // tokens in the list
  uint32_t digit, in_digit;      // where the cut falls, and how many tokens fall there
  uint32_t before_n;             // tokens and weight before it
  uint64_t before_w;
  uint32_t cut_key, cut_id;
  uint64_t cut_sum;              // weight up to the cut
  uint64_t need_w;
  uint32_t tie[SP_MAX_CLUSTER];  // tokens of the cut's value in each CTA
};

// The row's constants.
struct Row {
  float top, c_hi, c_lo, bins;   // bins: of the difference to the top
};

// floor(2^40 2^(-y)), y = (top - z) log2(e) / t, off by a unit where the fraction is near a border.  The difference and
// the product with log2(e) / t are pairs of floats; y = k / 64 + r, |r| <= 1 / 128, and 2^(-r) - 1 = u + u^2 / 2 + u^3 / 6 +
// u^4 / 24 with u = -r ln 2 (the next term is below 2^-44), the linear term a pair, the rest (2^-16) a float; table
// entry and product then meet in 46-bit fixed point.
__device__ __forceinline__ uint64_t weight(const SampleShared& s, const Row& r, float z) {
  constexpr float MAGIC = 12582912.0f;           // 1.5 2^23: the sum's low bits are the rounded integer
  constexpr int MAGIC_BITS = 0x4B400000;
  const float dh = r.top - z;
  const float bb = dh - r.top;
  const float dl = (r.top - (dh - bb)) - (z + bb);
  const float yh = dh * r.c_hi;
  if (!(yh < 41.0f)) return 0;
  const float yl = fmaf(dh, r.c_hi, -yh) + fmaf(dh, r.c_lo, dl * r.c_hi);
  const float kt = fmaf(yh, 64.0f, MAGIC);
  const int k = __float_as_int(kt) - MAGIC_BITS;
  const float rh = fmaf(kt - MAGIC, -0x1p-6f, yh);
  const float rs = rh + yl, rl = yl - (rs - rh);
  constexpr float LN2_HI = 0x1.62e43p-1f, LN2_LO = -0x1.05c61p-29f;
  const float uh = -rs * LN2_HI;
  const float ul = fmaf(-rs, LN2_HI, -uh) - fmaf(rs, LN2_LO, rl * LN2_HI);
  const float v = fmaf(uh * uh, fmaf(uh, fmaf(uh, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f), ul);
  const float2 t = s.pow2f[k & 63];
  const float a = t.x * uh;
  const float b = fmaf(t.x, uh, -a) + fmaf(t.x, v, t.y * uh);
  const float c = a + b, cl = b - (c - a);
  const float c1 = fmaf(c, 0x1p24f, MAGIC);
  const float rem = fmaf(c1 - MAGIC, -0x1p-24f, c) + cl;
  const int64_t w = static_cast<int64_t>(s.pow2[k & 63]) +
                    (static_cast<int64_t>(__float_as_int(c1) - MAGIC_BITS) << 22) +
                    (__float_as_int(fmaf(rem, 0x1p46f, MAGIC)) - MAGIC_BITS);
  return static_cast<uint64_t>(w) >> (6 + (k >> 6));
}

__device__ __forceinline__ uint32_t bin_of(const Row& r, float z) {
  return static_cast<uint32_t>(fminf((r.top - z) * r.bins, static_cast<float>(SP_BINS - 1)));
}

// The digit of a search's pass `level`: the bin, then 11, 11 and 10 bits of the logit's order.
__device__ __forceinline__ uint32_t digit_of(const Row& r, float z, int level) {
  if (level == 0) return bin_of(r, z);
  const uint32_t key = order_key(z);
  return level == 1 ? key >> 21 : level == 2 ? (key >> 10) & 2047u : key & 1023u;
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
  for (int i = 0; i < warp; ++i) n0 += s.scan_n[i], w0 += s.scan[i];
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
__device__ __forceinline__ uint32_t dsmem_add(uint32_t a, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
  return old;
}

// Every thread of the cluster; shared-memory accesses before, local or remote, come before those after.
__device__ __forceinline__ void meet(const SampleParams& p) {
  if (p.cluster > 1) sm100::cluster_sync();
  else __syncthreads();
}

// A thread's tokens: register i is id base + (i / 8) * 256 + i % 8, in its warp's run of consecutive ids.
template <int E>
struct Tokens {
  float z[E];
  int base;
  __device__ __forceinline__ int id(int i) const { return base + (i >> 3) * 256 + (i & 7); }
};

// The row's bins of pass `level`, over the tokens that `chosen` picks, in the first CTA's all_*.
template <int E, typename Chosen>
__device__ __forceinline__ void histogram(const SampleParams& p, SampleShared& s, const uint64_t* w, const Row& r,
                                          const Tokens<E>& tk, int level, uint32_t rank, Chosen chosen) {
  for (int b = threadIdx.x; b < SP_BINS; b += SP_THREADS) s.count[b] = s.lo[b] = s.hi[b] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint64_t wi = w[i * SP_THREADS + threadIdx.x];
    if (wi == 0 || !chosen(tk.z[i])) continue;
    const uint32_t d = digit_of(r, tk.z[i], level);
    atomicAdd(&s.count[d], 1u);
    const uint32_t l = static_cast<uint32_t>(wi), old = atomicAdd(&s.lo[d], l);
    const uint32_t h = static_cast<uint32_t>(wi >> 32) + (old + l < old ? 1u : 0u);
    if (h) atomicAdd(&s.hi[d], h);
  }
  meet(p);
  const int slice = SP_BINS / p.cluster;
  for (int b = static_cast<int>(rank) * slice + threadIdx.x; b < (static_cast<int>(rank) + 1) * slice; b += SP_THREADS) {
    uint32_t n = 0;
    uint64_t sum = 0;
    for (int c = 0; c < p.cluster; ++c) {
      n += dsmem_ld_u32(sm100::dsmem_addr(&s.count[b], c));
      sum += (static_cast<uint64_t>(dsmem_ld_u32(sm100::dsmem_addr(&s.hi[b], c))) << 32) +
             dsmem_ld_u32(sm100::dsmem_addr(&s.lo[b], c));
    }
    sm100::dsmem_st_s32(sm100::dsmem_addr(&s.all_count[b], 0), static_cast<int>(n));
    sm100::dsmem_st_u64(sm100::dsmem_addr(&s.all_weight[b], 0), sum);
  }
  meet(p);
}

// The cut at which the count (by_weight false) or the weight of the tokens in falling order first reaches `need`: cut_key,
// cut_id and cut_sum of every CTA; where it never does, cut_key 0 (all are kept) and the weight of all.
template <int E>
__device__ __noinline__ void find_cut(const SampleParams& p, SampleShared& s, const uint64_t* w, const Row& r,
                                      const Tokens<E>& tk, bool by_weight, uint64_t need, uint32_t rank) {
  uint32_t bin = 0, prefix = 0, before_n = 0;
  uint64_t before_w = 0;
  int level = 0;
  auto chosen = [&](float z) {
    if (level == 0) return true;
    if (bin_of(r, z) != bin) return false;
    const uint32_t key = order_key(z);
    return level == 1 || (level == 2 ? key >> 21 : key >> 10) == prefix;
  };
  while (true) {
    histogram(p, s, w, r, tk, level, rank, chosen);
    if (rank == 0) {
      // the digits in falling order of z: bins as they are, bits from the largest down
      uint32_t n = 0, cn[4];
      uint64_t sum = 0, cw[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = threadIdx.x * 4 + q, b = level == 0 ? at : SP_BINS - 1 - at;
        cn[q] = s.all_count[b];
        cw[q] = s.all_weight[b];
        n += cn[q];
        sum += cw[q];
      }
      uint32_t n0;
      uint64_t w0;
      block_before(s, n, sum, n0, w0);
      n0 += before_n;
      w0 += before_w;
      if (threadIdx.x == SP_THREADS - 1 && (by_weight ? w0 + sum : n0 + n) < need) {   // never reached
        st_all_u32(p, &s.in_digit, 0);
        st_all_u64(p, &s.cut_sum, w0 + sum);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool here = by_weight ? w0 < need && w0 + cw[q] >= need : n0 < need && n0 + cn[q] >= need;
        if (here) {
          const int at = threadIdx.x * 4 + q;
          st_all_u32(p, &s.digit, level == 0 ? at : SP_BINS - 1 - at);
          st_all_u32(p, &s.in_digit, cn[q]);
          st_all_u32(p, &s.before_n, n0);
          st_all_u64(p, &s.before_w, w0);
        }
        n0 += cn[q];
        w0 += cw[q];
      }
      if (threadIdx.x == 0) s.listed = 0;
    }
    meet(p);
    const uint32_t there = s.in_digit;
    before_n = s.before_n;
    before_w = s.before_w;
    if (there == 0) {
      if (threadIdx.x == 0) s.cut_key = 0, s.cut_id = 0;
      meet(p);
      return;
    }
    const uint32_t digit = s.digit;
    if (level == 0) bin = digit;
    else prefix = level == 1 ? digit : level == 2 ? (prefix << 11 | digit) : (prefix << 10 | digit);
    ++level;
    if (there <= SP_LIST || level == 4) break;
    meet(p);                                     // the state is read before the next pass writes it
  }
  // the tokens of the last digit
  auto last = [&](float z) {
    if (bin_of(r, z) != bin) return false;
    const uint32_t key = order_key(z);
    return level == 1 || (level == 2 ? key >> 21 : level == 3 ? key >> 10 : key) == prefix;
  };
  if (s.in_digit <= SP_LIST) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint64_t wi = w[i * SP_THREADS + threadIdx.x];
      if (wi == 0 || !last(tk.z[i])) continue;
      const uint32_t at = dsmem_add(sm100::dsmem_addr(&s.listed, 0), 1u);
      const uint32_t a = sm100::dsmem_addr(&s.list[at], 0);
      sm100::dsmem_st_u64(a, static_cast<uint64_t>(order_key(tk.z[i])) | (static_cast<uint64_t>(tk.id(i)) << 32));
      sm100::dsmem_st_u64(a + 8, wi);
    }
    meet(p);
    if (rank == 0) {
      const int n = static_cast<int>(s.in_digit);
      for (int e = threadIdx.x; e < n; e += SP_THREADS) {
        const Listed me = s.list[e];
        uint64_t w0 = before_w;
        uint32_t n0 = before_n;
        for (int o = 0; o < n; ++o) {
          const Listed x = s.list[o];
          const bool first = x.key > me.key || (x.key == me.key && x.id < me.id);
          if (first) w0 += x.w, ++n0;
        }
        if (by_weight ? w0 < need && w0 + me.w >= need : n0 + 1 == need) {
          st_all_u32(p, &s.cut_key, me.key);
          st_all_u32(p, &s.cut_id, me.id);
          st_all_u64(p, &s.cut_sum, w0 + me.w);
        }
      }
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
#pragma unroll
  for (int i = 0; i < E; ++i) mine += w[i * SP_THREADS + threadIdx.x] != 0 && last(tk.z[i]) ? 1u : 0u;
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
    for (int j = 0; j < E / 8; ++j) {
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i / 8 == j && w[i * SP_THREADS + threadIdx.x] != 0 && last(tk.z[i])) bits |= 1u << (i & 7);
      uint32_t c = static_cast<uint32_t>(__popc(bits)), upto = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      uint32_t k = before + upto - c;
      for (int i = 0; i < 8; ++i)
        if (bits >> i & 1u) {
          if (++k == m) {
            st_all_u32(p, &s.cut_key, prefix);
            st_all_u32(p, &s.cut_id, tk.base + j * 256 + i);
            st_all_u64(p, &s.cut_sum, before_w + one * m);
          }
        }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  meet(p);
}

// Eight logits from id on, those past the end -inf.
__device__ __forceinline__ void load_logits(const uint16_t* row, int id, int vocab, bool wide, float (&z)[8]) {
  if (wide && id + 8 <= vocab) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + id);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = __uint_as_float(u[i] << 16);
      z[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = id + i < vocab ? bf16_to_f32(row[id + i]) : -INFINITY;
}
__device__ __forceinline__ void load_logits(const float* row, int id, int vocab, bool wide, float (&z)[8]) {
  if (wide && id + 8 <= vocab) {
    const float4 a = *reinterpret_cast<const float4*>(row + id), b = *reinterpret_cast<const float4*>(row + id + 4);
    z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
    z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = id + i < vocab ? row[id + i] : -INFINITY;
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

template <typename T, int J>
__global__ void __launch_bounds__(SP_THREADS, J == 1 ? 2 : 1) sample_kernel(SampleParams p) {
  constexpr int E = 8 * J;
  extern __shared__ uint64_t w[];                // [E][threads]
  SampleShared& s = *reinterpret_cast<SampleShared*>(w + E * SP_THREADS);
  LaunchStamp ls(p.stamp);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x / p.cluster;
  const uint32_t rank = p.cluster > 1 ? sm100::cluster_rank() : 0;
  if (threadIdx.x < 64) {
    const uint64_t v = kPow2[threadIdx.x];
    s.pow2[threadIdx.x] = v;
    const float h = static_cast<float>(v);
    s.pow2f[threadIdx.x] =
        make_float2(h * 0x1p-46f, static_cast<float>(static_cast<int64_t>(v) - static_cast<int64_t>(h)) * 0x1p-46f);
  }
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int request = row / p.rows_each;
  if (p.rows_used && row - request * p.rows_each >= p.rows_used[request]) return;
  const float temp = p.temperature ? p.temperature[request] : 1.0f;
  const bool greedy = !(temp > 0.0f);
  if (p.cluster > 1) sm100::cluster_arrive_relaxed();   // (the others are there before anything is written to them)

  const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
  const bool wide = (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  Tokens<E> tk;
  tk.base = static_cast<int>(rank) * E * SP_THREADS + warp * E * 32 + lane * 8;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float z[8];
    load_logits(logits, tk.base + j * 256, p.vocab, wide, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) tk.z[8 * j + i] = z[i];
  }
  // the largest logit and its first id, the lowest finite one, and whether any is NaN or +inf
  uint32_t top = 0, low = 0xffffffffu, bad = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float z = tk.z[i];
    if (!(z < INFINITY)) bad = 1;
    const uint32_t key = order_key(z);
    top = max(top, key);
    if (z > -INFINITY) low = min(low, key);
  }
  const uint32_t warp_top = __reduce_max_sync(0xffffffffu, top);
  uint32_t id = 0xffffffffu;
  if (top == warp_top) {
#pragma unroll
    for (int i = E - 1; i >= 0; --i)
      if (order_key(tk.z[i]) == top) id = static_cast<uint32_t>(tk.id(i));
  }
  id = __reduce_min_sync(0xffffffffu, id);
  low = __reduce_min_sync(0xffffffffu, low);
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) s.warp_extent[warp] = Extent{warp_top, id, low, bad};
  __syncthreads();
  if (warp == 0) {
    Extent e = s.warp_extent[lane % SP_WARPS];
    const uint32_t t = __reduce_max_sync(0xffffffffu, e.top);
    e.id = __reduce_min_sync(0xffffffffu, e.top == t ? e.id : 0xffffffffu);
    e.low = __reduce_min_sync(0xffffffffu, e.low);
    e.bad = __reduce_or_sync(0xffffffffu, e.bad);
    if (p.cluster > 1) sm100::cluster_wait();
    if (lane < p.cluster) {
      const uint32_t a = sm100::dsmem_addr(&s.extent[rank], lane);
      sm100::dsmem_st_u64(a, t | (static_cast<uint64_t>(e.id) << 32));
      sm100::dsmem_st_u64(a + 8, e.low | (static_cast<uint64_t>(e.bad) << 32));
    }
    if (lane == 0 && !greedy) {
      const double c = 1.4426950408889634 / fmax(static_cast<double>(temp), 1e-30);
      s.c_hi = static_cast<float>(c);
      s.c_lo = static_cast<float>(c - static_cast<double>(s.c_hi));
    }
    __syncwarp();
  } else if (p.cluster > 1) {
    sm100::cluster_wait();
  }
  meet(p);
  Extent all{0, 0xffffffffu, 0xffffffffu, 0};
  for (int c = 0; c < p.cluster; ++c) {
    const Extent e = s.extent[c];
    if (e.top > all.top) all.top = e.top, all.id = e.id;
    all.low = min(all.low, e.low);
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
  if (none || greedy) {
    if (probs) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = !none && static_cast<uint32_t>(tk.id(8 * j + i)) == all.id ? 1.0f : 0.0f;
        store_probs(probs, tk.base + j * 256, p.vocab, wide_out, v);
      }
    }
    return;
  }
  if (!p.token && !probs) return;

  Row r;
  r.top = zmax;
  r.c_hi = s.c_hi;
  r.c_lo = s.c_lo;
  // bins over the logits that can have weight
  const float span = fminf(zmax - key_value(all.low), 41.0f / r.c_hi);
  r.bins = span > 0.0f ? fminf(static_cast<float>(SP_BINS) / span, 0x1p100f) : 0.0f;
  const int k = p.top_k ? p.top_k[request] : 0;
  const float top_p = p.top_p ? p.top_p[request] : 1.0f;
  const float min_p = p.min_p ? fminf(p.min_p[request], 1.0f) : 0.0f;
  uint64_t sum = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint64_t wi = weight(s, r, tk.z[i]);
    w[i * SP_THREADS + threadIdx.x] = wi;
    sum += wi;
  }
  uint32_t cut_key = 0, cut_id = 0;
  if (k > 0 && k < p.vocab) {
    find_cut(p, s, w, r, tk, false, static_cast<uint64_t>(k), rank);
    cut_key = s.cut_key;
    cut_id = s.cut_id;
  }
  if (top_p < 1.0f) {
    if (!(k > 0 && k < p.vocab)) {               // the weight of all tokens
      sum = warp_sum_u64(sum);
      if (lane == 0) s.warp_total[warp] = sum;
      __syncthreads();
      if (threadIdx.x == 0) {
        uint64_t t = 0;
        for (int i = 0; i < SP_WARPS; ++i) t += s.warp_total[i];
        st_all_u64(p, &s.total[rank], t);
      }
      meet(p);
      if (threadIdx.x == 0) {
        uint64_t t = 0;
        for (int c = 0; c < p.cluster; ++c) t += s.total[c];
        s.cut_sum = t;
      }
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      const uint64_t need = static_cast<uint64_t>(
          ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(s.cut_sum)));
      s.need_w = need < 1 ? 1 : min(need, s.cut_sum);
    }
    __syncthreads();
    const uint64_t need = s.need_w;
    find_cut(p, s, w, r, tk, true, need, rank);
    cut_key = s.cut_key;
    cut_id = s.cut_id;
  }
  const uint64_t least = min_p > 0.0f ? static_cast<uint64_t>(ceilf(min_p * 0x1p40f)) : 1;
  // what is kept
  sum = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    uint64_t wi = w[i * SP_THREADS + threadIdx.x];
    const uint32_t key = order_key(tk.z[i]);
    if (wi < least || key < cut_key || (key == cut_key && static_cast<uint32_t>(tk.id(i)) > cut_id)) {
      wi = 0;
      w[i * SP_THREADS + threadIdx.x] = 0;
    }
    sum += wi;
  }
  const uint64_t in_warp = warp_sum_u64(sum);
  if (lane == 0) s.warp_total[warp] = in_warp;
  __syncthreads();
  uint64_t before = 0, in_cta = 0;
  for (int i = 0; i < SP_WARPS; ++i) {
    if (i < warp) before += s.warp_total[i];
    in_cta += s.warp_total[i];
  }
  if (threadIdx.x == 0) st_all_u64(p, &s.total[rank], in_cta);
  meet(p);
  uint64_t W = 0;
  for (int c = 0; c < p.cluster; ++c) {
    if (c < static_cast<int>(rank)) before += s.total[c];
    W += s.total[c];
  }
  if (p.token) {
    const uint64_t at = scale_uniform(p.u[row], W);
    if (before <= at && at < before + in_warp) {
      for (int j = 0; j < J; ++j) {
        uint64_t mine = 0;
        for (int i = 0; i < 8; ++i) mine += w[(8 * j + i) * SP_THREADS + threadIdx.x];
        uint64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        uint64_t sofar = before + upto - mine;
        if (sofar <= at && at < sofar + mine) {
          for (int i = 0; i < 8; ++i) {
            const uint64_t wi = w[(8 * j + i) * SP_THREADS + threadIdx.x];
            if (sofar <= at && at < sofar + wi) p.token[row] = tk.base + j * 256 + i;
            sofar += wi;
          }
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  if (probs) {
    const float inv = 1.0f / static_cast<float>(W);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(w[(8 * j + i) * SP_THREADS + threadIdx.x]) * inv;
      store_probs(probs, tk.base + j * 256, p.vocab, wide_out, v);
    }
  }
}

typedef void (*SampleKernel)(SampleParams);
template <typename T>
SampleKernel kernel_of(int j) {
  return j == 1 ? sample_kernel<T, 1> : j == 2 ? sample_kernel<T, 2> : sample_kernel<T, 4>;
}

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
  // A CTA takes 4096, 8192 or 16384 tokens: the fewest that still leave every SM at most one CTA.
  int j = 1;
  auto clusters = [&](int jj) {
    int c = 1;
    while (c * SP_THREADS * 8 * jj < S.vocab) c <<= 1;
    return c;
  };
  while (j < 4 && (clusters(j) > SP_MAX_CLUSTER || static_cast<long long>(clusters(j)) * S.rows > ctx->sm_count)) j <<= 1;
  p.cluster = clusters(j);
  const SampleKernel k = S.dtype == EAGLE_DTYPE_F32 ? kernel_of<float>(j) : kernel_of<uint16_t>(j);
  const size_t smem = static_cast<size_t>(8 * j) * SP_THREADS * 8 + sizeof(SampleShared);
  cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(k), static_cast<int>(smem));
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
