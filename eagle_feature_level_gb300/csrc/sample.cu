// eagle_sample: a row's distribution under temperature, top-k, top-p and min-p, and a draw from it.
//
// Weights are whole numbers, floor(2^40 e^((z - max) / t)), and their sums exact, so the order of sums does not matter and
// a border is where the definition has it.
//
// Rows are gone over in chunks of 4096 tokens, a few to a CTA, whatever the number of rows and their length, so that the
// work is even; what the chunks find out meets in the row's state, where the last CTA to arrive draws the conclusion:
//   1. the largest logit, and with it the scale of the row;
//   2. bins of the tokens by their distance from the largest: their number (top-k, eighths of a power of two) or weight
//      (top-p, sixteenths), and from these the bin with the cut, the last token in falling order that is kept;
//   3. the weight of each chunk before that bin, and a list of the bin's tokens (with top-k and top-p both, of all up to
//      it: top-p's part is of those k);
//   4. a CTA a row sorts the list, which gives the cut and the weight of each chunk, and draws: the chunk, then the token;
//   5. the probabilities, where wanted.
// The logits come from memory once and then from L2.  512 tokens are sorted at a time; where a bin has more, they are told
// apart by 1024 bins of the bin, then by the bits of the logits, 10 at a time, then by their ids (many of one value).  A
// list holds 4096; past that (or where the cut is behind 22 powers of two, where weight has no bins) the CTA goes over the
// row itself.
//
// Weights from 2^23 on (the near tokens') take fixed point and pairs of floats, the others fp32.  Near tokens are a small
// part of a row as a rule: a warp lists its own first, so that the work on them is dense.
//
// Bound: instructions where rows are flat (64 rows of 131072 in bf16: top-p of 0.95 at t = 1.3 89 us, issue slots of the
// busy SMs full), else the latency of each kernel's loads and exchanges (greedy 11 us, 15 among controls, top-k of 50 33, top-p
// of 0.7 at t = 0.5 41, min-p of 0.05 28, no cut 43; a row of 32000: top-k of 400 and top-p 17).  A cluster of CTAs that keeps
// a row in shared memory through all steps saves launches, but leaves the SMs waiting for its exchanges: those 64
// rows 209, 26, 66, 89, 56 and 66 us, the one row 17, and 64 rows of all sorts 113 where this takes 56.
//
// Where a list does not hold a row's tokens, one CTA goes over the row once for each of up to five levels of digits and a few
// times more, and that takes as long as it is long: those 64 rows with top-k of 20000 and top-p of 0.9 520 us (one such row
// 312), of 4000 at t = 2 436, top-p at t = 100 469, rows of one value throughout 1700; top-k of 20000 alone, whose list holds
// its bin, 55.
#include <algorithm>

#include "internal.h"
#include "common.cuh"
#include "sm100.cuh"

namespace eagle {
namespace {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_LIST = 8 * SP_THREADS;         // of a row
constexpr int SP_SORT = SP_THREADS;             // sorted at a time
constexpr int SP_CHUNK = 8 * SP_THREADS;        // eight tokens a thread
constexpr int SP_MAX_CHUNKS = EAGLE_MAX_SAMPLE_VOCAB / SP_CHUNK;
constexpr int SP_MAX_PIECES = 3;                // chunks of a CTA from the second kernel on
static_assert(SP_MAX_CHUNKS <= 64, "two chunks a lane");

// From this distance on a weight (2^23 or less) needs no more than fp32, and from the other it is nothing.
constexpr float SP_FAR = 17.0f, SP_NONE = 41.0f;
// A row's bins: where tokens are counted, up to SP_NONE; where they are weighed, up to SP_WEIGHED (the tokens behind it
// have 2^-22 of the largest's weight at most: a cut among them takes a row as flat as it is long).
constexpr float SP_COUNT_BINS = 8.0f, SP_WEIGHT_BINS = 16.0f, SP_WEIGHED = 22.0f;
constexpr int SP_LANE_BINS = 11;                 // of a lane, where a warp goes over them
constexpr int SP_ROW_BINS = 32 * SP_LANE_BINS;
static_assert(SP_NONE * SP_COUNT_BINS <= SP_ROW_BINS && SP_WEIGHED * SP_WEIGHT_BINS <= SP_ROW_BINS, "all bins");
constexpr int SP_BINS = 2 * SP_THREADS;          // of a bin

// What there is to do for a row: nothing, as it has no distribution or is greedy, or to draw from all its weights, from a
// beginning by number or by weight, or from what min_p keeps.
enum RowKind : int { ROW_NONE, ROW_GREEDY, ROW_WHOLE, ROW_COUNT, ROW_WEIGH, ROW_REACH };

// The largest key of some chunks and its first id, and whether any logit is NaN or +inf.
struct alignas(16) Extent {
  uint32_t top, id, bad, pad;
};

// A row's state between the kernels.
struct alignas(16) SampleRow {
  // by the first kernel's last CTA; `from`, `end` by the second's where the row has bins
  float top, c_hi, c_lo;                        // its Row
  int kind;
  float from, end;                              // tokens nearer than `from` are kept, those from `end` on not
  float reach;                                  // distance up to which min_p may keep a token
  uint32_t id;                                  // the argmax
  uint64_t least;                               // min_p's weight
  float top_p;
  uint64_t need, before;                        // the cut's number or weight, and the number or weight before `from`
  uint64_t far;                                 // weight of the tokens behind the bins, where those are weighed
  uint32_t listed;                              // tokens in `list`, or more than it takes
  uint32_t cut_key, cut_id;                     // by the fourth: the last token kept (0: all), and one over the weight
  float inverse;
  Extent extent[SP_MAX_CHUNKS];                 // of each CTA's chunks
  uint64_t total[SP_MAX_CHUNKS];                // weight of each chunk before `from`
  uint64_t bins[SP_ROW_BINS];                   // number or weight of the tokens in each
  uint64_t list[SP_LIST];                       // tokens from `from` to `end`: key << 32 | ~id
};

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
  SampleRow* state;
  int* arrived;            // [2][SAMPLE_ROWS]: of a row's CTAs in the first two kernels, zero between calls
  int row0;                // the launch's first row, whose state is the first
  int chunks, pieces;      // of a row, and of a CTA of it
  int groups;              // CTAs of a row
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

// The row's constants.
struct Row {
  float top, c_hi, c_lo;
};

// A token has one weight, whichever kernel computes it: a row's sums are of one kernel and its draw of another.  So every
// product here that a sum takes is rounded by itself (__fmul_rn) or fused in so many words (fmaf), and none of it is left to
// the compiler.

// (top - z) log2(e) / t to fp32's precision; large for what has no weight at all.
__device__ __forceinline__ float distance(const Row& r, float z) { return fminf(__fmul_rn(r.top - z, r.c_hi), 100.0f); }

// The difference to the top and its product with log2(e) / t as pairs of floats: the low part of y, given the high one.
__device__ __forceinline__ float low_part(const Row& r, float z, float dh, float yh) {
  const float bb = dh - r.top;
  const float dl = (r.top - (dh - bb)) - (z + bb);
  return fmaf(dh, r.c_hi, -yh) + fmaf(dh, r.c_lo, __fmul_rn(dl, r.c_hi));
}

// floor(2^40 2^(-y)) from SP_FAR on, off by two units of 2^23 at most (by one in half a million tokens): y to both its parts,
// exp2 to 2^-22.7 over all of 40 - y's values, which fp32 has, and a product fused into its sum.
__device__ __forceinline__ uint32_t far_weight(const Row& r, float z) {
  const float dh = r.top - z, yh = __fmul_rn(dh, r.c_hi);
  const float e = sm100::exp2(40.0f - yh);
  const float x = fmaf(e, __fmul_rn(-0x1.62e43p-1f, low_part(r, z, dh, yh)), e);
  const uint32_t w = __float_as_uint(__fadd_rd(fminf(x, 8388607.0f), 8388608.0f)) & 0x7fffffu;
  return yh < 41.0f ? w : 0u;
}

// floor(2^40 2^(-y)), or one off where that is within 2^-5 of a whole number.  The difference to the top and its product with
// log2(e) / t are pairs of floats; y = k / 64 + r, |r| <= 1 / 128, and u = -r ln 2 is a pair again, x + l, |l| <= 2^-22 |y|.
// 2^(-r) - 1 = x + x^2 / 2 + x^3 / 6 + x^4 / 24 + (1 + x + x^2 / 2) l + ...: x and x^2 / 2 (up to 2^-16: as one float it
// would cost half a unit) meet in a pair, what is left (2^-25) is a float; x^5 / 120 is taken with x^3 as its best multiple
// of it up to ln(2) / 128, 0.87 (ln(2) / 128)^2 x^3 / 120, to 2^-47.  Table entry and product then meet in 46-bit fixed
// point.  In units of 2^-40: the table and the fixed point 2^-7 each, the series 2^-7, the sums of 2^-25 three times 2^-10.
__device__ __forceinline__ uint64_t near_weight(const Pow2* pow2, const Row& r, float z) {
  constexpr float MAGIC = 12582912.0f;           // 1.5 2^23: the sum's low bits are the rounded integer
  constexpr int MAGIC_BITS = 0x4B400000;
  const float dh = r.top - z;
  const float yh = fminf(__fmul_rn(dh, r.c_hi), SP_FAR);   // (beyond: not used)
  const float yl = low_part(r, z, dh, yh);
  const float kt = fmaf(yh, 64.0f, MAGIC);
  const int k = __float_as_int(kt) - MAGIC_BITS;
  const float rh = fmaf(kt - MAGIC, -0x1p-6f, yh);
  constexpr float LN2_HI = 0x1.62e43p-1f, LN2_LO = -0x1.05c61p-29f;
  const float x = __fmul_rn(-rh, LN2_HI);
  const float l = fmaf(-rh, LN2_HI, -x) - fmaf(rh, LN2_LO, __fmul_rn(yl, LN2_HI));
  const float h = 0.5f * x, p = __fmul_rn(h, x), eh = x + p;
  const float rest = fmaf(__fmul_rn(p, x), fmaf(x, 1.0f / 12.0f, 1.0f / 3.0f + 4.25e-7f), fmaf(h, x, -(eh - x)));
  const float el = fmaf(eh, l, rest) + l;
  const Pow2 t = pow2[k & 63];
  const float a = __fmul_rn(t.hi, eh);
  const float b = fmaf(t.hi, eh, -a) + fmaf(t.hi, el, __fmul_rn(t.lo, eh));
  const float c1 = fmaf(a + b, 0x1p24f, MAGIC);
  const float rem = fmaf(c1 - MAGIC, -0x1p-24f, a) + b;
  const int64_t w = static_cast<int64_t>(t.whole) +
                    (static_cast<int64_t>(__float_as_int(c1) - MAGIC_BITS) << 22) +
                    (__float_as_int(fmaf(rem, 0x1p46f, MAGIC)) - MAGIC_BITS);
  return static_cast<uint64_t>(w) >> (6 + (k >> 6));
}

__device__ __forceinline__ uint64_t weight(const Pow2* pow2, const Row& r, float z) {
  const float y = distance(r, z);
  return y < SP_FAR ? near_weight(pow2, r, z) : far_weight(r, z);
}

// The same, 0 where not wanted, without paths that no thread of the warp needs (the whole warp calls it).
__device__ __forceinline__ uint64_t weight_of(const Pow2* pow2, const Row& r, float z, bool wanted) {
  const bool near = wanted && distance(r, z) < SP_FAR;
  uint64_t w = wanted && !near ? far_weight(r, z) : 0;
  if (__any_sync(0xffffffffu, near)) {
    const uint64_t x = near_weight(pow2, r, z);
    if (near) w = x;
  }
  return w;
}

// Eight logits from id `at` on, those past the end -inf, as they are loaded: what is converted is waited for, so a chunk's
// are loaded under the one before and converted when it is their turn.
template <typename T>
struct Logits;
template <>
struct Logits<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* row, int at, int vocab, bool wide) {
    if (wide && at + 8 <= vocab) {
      a = *reinterpret_cast<const float4*>(row + at);
      b = *reinterpret_cast<const float4*>(row + at + 4);
    } else {
      auto one = [&](int i) { return at + i < vocab ? row[at + i] : -INFINITY; };
      a = make_float4(one(0), one(1), one(2), one(3));
      b = make_float4(one(4), one(5), one(6), one(7));
    }
  }
  __device__ __forceinline__ void get(float (&z)[8]) const {
    z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
    z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
  }
};
template <>
struct Logits<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* row, int at, int vocab, bool wide) {
    if (wide && at + 8 <= vocab) {
      v = *reinterpret_cast<const uint4*>(row + at);
    } else {
      auto one = [&](int i) { return at + i < vocab ? static_cast<uint32_t>(row[at + i]) : 0xff80u; };
      v = make_uint4(one(0) | one(1) << 16, one(2) | one(3) << 16, one(4) | one(5) << 16, one(6) | one(7) << 16);
    }
  }
  __device__ __forceinline__ void get(float (&z)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = __uint_as_float(u[i] << 16);
      z[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <typename T>
__device__ __forceinline__ void load_logits(const T* row, int at, int vocab, bool wide, float (&z)[8]) {
  Logits<T> x;
  x.load(row, at, vocab, wide);
  x.get(z);
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

// Exclusive sums over the block, in thread order.
struct BlockScan {
  uint64_t of[SP_WARPS];
};
__device__ __forceinline__ uint64_t block_before(BlockScan& s, uint64_t w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t upto = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t b = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += b;
  }
  __syncthreads();                               // (the last scan's sums are read)
  if (lane == 31) s.of[warp] = upto;
  __syncthreads();
  upto -= w;
#pragma unroll
  for (int i = 0; i < SP_WARPS; ++i)
    if (i < warp) upto += s.of[i];
  return upto;
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

__device__ __forceinline__ Row row_of(const SampleRow& st) { return Row{st.top, st.c_hi, st.c_lo}; }

__device__ __forceinline__ void fill_pow2(Pow2* pow2) {
  if (threadIdx.x < 64) {
    const uint64_t v = kPow2[threadIdx.x];
    const float h = static_cast<float>(v);
    pow2[threadIdx.x] =
        Pow2{v, h * 0x1p-46f, static_cast<float>(static_cast<int64_t>(v) - static_cast<int64_t>(h)) * 0x1p-46f};
  }
}

// A row behind those that its request uses.
__device__ __forceinline__ bool unused(const SampleParams& p, int row, int request) {
  return p.rows_used && row - request * p.rows_each >= p.rows_used[request];
}

// Of the first id of a thread's eight in a chunk: a warp's are in a row.
__device__ __forceinline__ int chunk_id(int chunk) { return chunk * SP_CHUNK + static_cast<int>(threadIdx.x) * 8; }

__device__ __forceinline__ Extent warp_extent(Extent e) {
  const uint32_t t = __reduce_max_sync(0xffffffffu, e.top);
  e.id = __reduce_min_sync(0xffffffffu, e.top == t ? e.id : 0xffffffffu);
  e.bad = __reduce_or_sync(0xffffffffu, e.bad);
  e.top = t;
  return e;
}

__device__ __forceinline__ float largest(const float (&z)[8]) {
  return fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
}

// The bin where the sum of a row's bins reaches `need` (-1: nowhere), and the sum before it (or of all); a whole warp.
template <typename F>
__device__ __forceinline__ int find_bin(uint64_t need, F bin_at, uint64_t& before) {
  const int lane = threadIdx.x & 31;
  uint64_t own[SP_LANE_BINS], mine = 0;
#pragma unroll
  for (int q = 0; q < SP_LANE_BINS; ++q) {
    own[q] = bin_at(lane * SP_LANE_BINS + q);
    mine += own[q];
  }
  uint64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  uint64_t sofar = upto - mine;
  int bin = -1;
  if (sofar < need && upto >= need) {            // in one of this lane's
#pragma unroll
    for (int q = 0; q < SP_LANE_BINS; ++q) {
      if (bin < 0 && sofar + own[q] >= need) bin = lane * SP_LANE_BINS + q;
      if (bin < 0) sofar += own[q];
    }
  }
  const uint32_t who = __ballot_sync(0xffffffffu, bin >= 0);
  const int from = who ? __ffs(who) - 1 : 31;
  before = __shfl_sync(0xffffffffu, who ? sofar : upto, from);
  return __shfl_sync(0xffffffffu, bin, from);
}

// Whether this CTA is the last of its row's to arrive: it then sees what all of them stored (every thread calls it).
__device__ __forceinline__ bool last_of_row(int* arrived, int ctas) {
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    last = ctas == 1 || arrive_acq_rel(arrived) == ctas - 1;
    if (last && ctas > 1) *arrived = 0;
  }
  __syncthreads();
  return last;
}

__device__ __forceinline__ void add_u64(uint64_t* to, uint64_t v) {
  atomicAdd(reinterpret_cast<unsigned long long*>(to), static_cast<unsigned long long>(v));
}
__device__ __forceinline__ uint64_t ldcg_u64(const uint64_t* at) {
  return __ldcg(reinterpret_cast<const unsigned long long*>(at));
}

// 1. The largest logit of every chunk; a row's last CTA takes the row's and its controls, and finishes greedy tokens.
template <typename T>
__global__ void __launch_bounds__(SP_THREADS) sample_top_kernel(SampleParams p) {
  __shared__ Extent warps[SP_WARPS];
  LaunchStamp ls(p.stamp);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at = blockIdx.x / p.groups, row = p.row0 + at;
  const int chunk0 = (blockIdx.x - at * p.groups) * p.pieces, chunk1 = min(chunk0 + p.pieces, p.chunks);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int request = row / p.rows_each;
  if (unused(p, row, request)) return;
  SampleRow& st = p.state[at];
  const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
  const bool wide = (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  // (for the last CTA, which would wait for them)
  const float temp = p.temperature ? p.temperature[request] : 1.0f;
  const int k = p.top_k ? p.top_k[request] : 0;
  const float top_p = p.top_p ? p.top_p[request] : 1.0f;
  const float min_p = p.min_p ? fminf(p.min_p[request], 1.0f) : 0.0f;
  float top = -INFINITY;                         // NaN if any is
  uint32_t id = 0xffffffffu;
  Logits<T> next;
  next.load(logits, chunk_id(chunk0), p.vocab, wide);
#pragma unroll 1
  for (int chunk = chunk0; chunk < chunk1; ++chunk) {
    float z[8], most = -INFINITY;
    next.get(z);
    if (chunk + 1 < chunk1) next.load(logits, chunk_id(chunk + 1), p.vocab, wide);
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(z[i]));
    if (chunk == chunk0 || most > top) {         // (the first of equals stays; with a NaN the id is not used)
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (z[i] == most) id = static_cast<uint32_t>(chunk_id(chunk) + i);
    }
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(most));
  }
  Extent e = warp_extent(Extent{order_key(top), id, top < INFINITY ? 0u : 1u, 0u});
  if (lane == 0) warps[warp] = e;
  __syncthreads();
  if (warp == 0) {
    e = warp_extent(warps[lane % SP_WARPS]);
    if (lane == 0) *reinterpret_cast<uint4*>(&st.extent[blockIdx.x - at * p.groups]) = make_uint4(e.top, e.id, e.bad, 0);
  }
  if (!last_of_row(p.arrived + at, p.groups)) return;
  if (threadIdx.x < SP_ROW_BINS) st.bins[threadIdx.x] = 0;
  static_assert(SP_ROW_BINS <= SP_THREADS, "a bin a thread");
  if (warp > 0) return;
  e = Extent{0, 0xffffffffu, 0, 0};
#pragma unroll
  for (int c = 0; c < SP_MAX_CHUNKS; c += 32) {
    if (c + lane < p.groups) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(&st.extent[c + lane]));
      if (v.x > e.top) e.top = v.x, e.id = v.y;   // (the later CTA's ids are larger)
      e.bad |= v.z;
    }
  }
  e = warp_extent(e);
  if (lane > 0) return;
  const bool none = e.bad || !(key_value(e.top) > -INFINITY), greedy = !(temp > 0.0f);
  const bool by_k = k > 0 && k < p.vocab, by_p = top_p < 1.0f;
  // log2(e) / t as a pair of floats: the quotient and, over t, what it leaves
  constexpr float LOG2E_HI = 0x1.715476p+0f, LOG2E_LO = 0x1.4ae0cp-26f;
  const float t = fmaxf(temp, 1e-30f), c_hi = LOG2E_HI / t;
  st.top = key_value(e.top);
  st.c_hi = c_hi;
  st.c_lo = t < 1e30f ? (fmaf(-c_hi, t, LOG2E_HI) + LOG2E_LO) / t : 0.0f;
  st.kind = none ? ROW_NONE : greedy ? ROW_GREEDY : by_k ? ROW_COUNT : by_p ? ROW_WEIGH : min_p > 0.0f ? ROW_REACH
                                                                                                      : ROW_WHOLE;
  st.from = st.end = SP_NONE;
  const uint64_t least = min_p > 0.0f ? static_cast<uint64_t>(ceilf(min_p * 0x1p40f)) : 1;
  st.least = least;
  st.reach = least > 1 ? 40.01f - log2f(static_cast<float>(least)) : SP_NONE;   // (generously)
  st.id = e.id;
  st.need = by_k ? static_cast<uint64_t>(k) : 0;
  st.top_p = top_p;
  st.far = 0;
  st.listed = 0;
  if (p.argmax) p.argmax[row] = none ? -1 : static_cast<int32_t>(e.id);
  if (none) set_status(p.status, EAGLE_ERR_NUMERIC);
  if ((none || greedy) && p.token) p.token[row] = none ? -1 : static_cast<int32_t>(e.id);
}

// Lists those of a warp's tokens that are nearer than `from` (SP_FAR at most); how many.
__device__ __forceinline__ uint32_t list_near(const Row& r, const float (&z)[8], float from, float* list) {
  const uint32_t before = (1u << (threadIdx.x & 31)) - 1;
  uint32_t n = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool near = distance(r, z[i]) < from;
    const uint32_t who = __ballot_sync(0xffffffffu, near);
    if (near) list[n + __popc(who & before)] = z[i];
    n += __popc(who);
  }
  __syncwarp();
  return n;
}

// 2. The bins of every chunk; a row's last CTA finds the bin with the cut.
template <typename T>
__global__ void __launch_bounds__(SP_THREADS, 3) sample_bins_kernel(SampleParams p) {
  __shared__ Pow2 pow2[64];
  __shared__ float near_z[SP_WARPS][256];        // a warp's near tokens
  // bins of every four warps: fewer than 4096 tokens' numbers, or weights in parts of 20 bits and 21, stay below 2^32
  constexpr int COPIES = SP_WARPS / 4;
  static_assert(SP_MAX_PIECES * SP_CHUNK / COPIES < 4096, "no sum passes 32 bits");
  __shared__ uint32_t lo[COPIES][SP_ROW_BINS], hi[COPIES][SP_ROW_BINS];
  __shared__ uint64_t sums[SP_WARPS];
  LaunchStamp ls(p.stamp);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at = blockIdx.x / p.groups, row = p.row0 + at;
  const int chunk0 = (blockIdx.x - at * p.groups) * p.pieces, chunk1 = min(chunk0 + p.pieces, p.chunks);
  fill_pow2(pow2);
  for (int b = threadIdx.x; b < COPIES * SP_ROW_BINS; b += SP_THREADS) (&lo[0][0])[b] = (&hi[0][0])[b] = 0;
  __syncthreads();
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int request = row / p.rows_each;
  if (unused(p, row, request)) return;
  SampleRow& st = p.state[at];
  const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
  const bool wide = (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  Logits<T> next;
  next.load(logits, chunk_id(chunk0), p.vocab, wide);
  const int kind = st.kind;
  if (kind != ROW_COUNT && kind != ROW_WEIGH) return;
  const Row r = row_of(st);
  const uint64_t k = st.need;
  const float top_p = st.top_p;
  uint32_t* my_lo = lo[warp % COPIES];
  uint32_t* my_hi = hi[warp % COPIES];
  uint64_t far_all = 0;
#pragma unroll 1
  for (int chunk = chunk0; chunk < chunk1; ++chunk) {
    float z[8];
    next.get(z);
    if (chunk + 1 < chunk1) next.load(logits, chunk_id(chunk + 1), p.vocab, wide);
    if (kind == ROW_COUNT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = distance(r, z[i]);
        if (y < SP_NONE) atomicAdd(&my_lo[static_cast<int>(y * SP_COUNT_BINS)], 1u);
      }
      continue;
    }
    uint32_t far = 0;                            // (256 of less than 2^18)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = distance(r, z[i]);
      const uint32_t w = far_weight(r, z[i]);
      if (y >= SP_FAR && y < SP_WEIGHED) {
        const int bin = static_cast<int>(y * SP_WEIGHT_BINS);
        atomicAdd(&my_lo[bin], w & 0xfffffu);
        if (w >> 20) atomicAdd(&my_hi[bin], w >> 20);
      }
      far += y < SP_WEIGHED ? 0u : w;
    }
    far_all += __reduce_add_sync(0xffffffffu, far);
    const uint32_t n = list_near(r, z, SP_FAR, near_z[warp]);
#pragma unroll 1
    for (uint32_t b = lane; b < n; b += 32) {
      const float x = near_z[warp][b];
      const uint64_t w = near_weight(pow2, r, x);
      const int bin = static_cast<int>(distance(r, x) * SP_WEIGHT_BINS);
      atomicAdd(&my_lo[bin], static_cast<uint32_t>(w) & 0xfffffu);
      atomicAdd(&my_hi[bin], static_cast<uint32_t>(w >> 20));
    }
    __syncwarp();                                // (the list is read)
  }
  if (lane == 0) sums[warp] = far_all;
  __syncthreads();
  if (threadIdx.x < SP_ROW_BINS) {
    const int b = threadIdx.x;
    uint64_t in = 0;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) in += (static_cast<uint64_t>(hi[i][b]) << 20) + lo[i][b];
    if (in) add_u64(&st.bins[b], in);
  } else if (warp == SP_WARPS - 1 && kind == ROW_WEIGH) {
    const uint64_t all = warp_sum_u64(lane < SP_WARPS ? sums[lane] : 0);
    if (lane == 0 && all) add_u64(&st.far, all);
  }
  static_assert(SP_ROW_BINS + 32 <= SP_THREADS, "the last warp has no bins");
  if (!last_of_row(p.arrived + SAMPLE_ROWS + at, p.groups) || warp > 0) return;
  auto bin_at = [&](int b) { return ldcg_u64(&st.bins[b]); };
  uint64_t need = k, before;
  if (kind == ROW_WEIGH) {
    find_bin(~0ull, bin_at, before);
    need = needed(top_p, before + ldcg_u64(&st.far));
  }
  const bool both = kind == ROW_COUNT && top_p < 1.0f;   // (then all k are listed)
  const int bin = find_bin(need, bin_at, before);
  if (lane > 0) return;
  st.need = need;
  const float bins = kind == ROW_COUNT ? SP_COUNT_BINS : SP_WEIGHT_BINS;
  if (bin >= 0) {
    st.before = both ? 0 : before;
    st.from = both ? 0.0f : static_cast<float>(bin) / bins;
    st.end = static_cast<float>(bin + 1) / bins;
  } else {                                       // all that have weight are kept, or the cut is behind the bins
    st.before = kind == ROW_COUNT ? 0 : before;
    if (kind == ROW_WEIGH) st.from = SP_WEIGHED;
    else if (both) st.from = 0.0f;
  }
}

// 3. The weight of every chunk's tokens before the bin with the cut, and a list of that bin's tokens.
template <typename T>
__global__ void __launch_bounds__(SP_THREADS, 3) sample_list_kernel(SampleParams p) {
  __shared__ Pow2 pow2[64];
  __shared__ float near_z[SP_WARPS][256];
  __shared__ uint64_t sums[SP_MAX_PIECES][SP_WARPS];
  LaunchStamp ls(p.stamp);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at = blockIdx.x / p.groups, row = p.row0 + at;
  const int chunk0 = (blockIdx.x - at * p.groups) * p.pieces, chunk1 = min(chunk0 + p.pieces, p.chunks);
  fill_pow2(pow2);
  __syncthreads();
  pdl_wait();
  ls.waited();
  pdl_trigger();
  if (unused(p, row, row / p.rows_each)) return;
  SampleRow& st = p.state[at];
  const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
  const bool wide = (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  Logits<T> next;
  next.load(logits, chunk_id(chunk0), p.vocab, wide);
  if (st.kind < ROW_WHOLE) return;
  const Row r = row_of(st);
  const float from = st.from, end = st.end, reach = st.reach;
  const uint64_t least = st.least;
#pragma unroll 1
  for (int chunk = chunk0; chunk < chunk1; ++chunk) {
    const int id0 = chunk_id(chunk);
    float z[8];
    next.get(z);
    if (chunk + 1 < chunk1) next.load(logits, chunk_id(chunk + 1), p.vocab, wide);
    if (!__any_sync(0xffffffffu, distance(r, largest(z)) < fmaxf(from, end))) {
      if (lane == 0) sums[chunk - chunk0][warp] = 0;
      continue;
    }
    uint64_t sum = 0;
    if (from > SP_FAR && reach > SP_FAR) {       // far tokens too
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = distance(r, z[i]);
        const uint32_t w = far_weight(r, z[i]);
        sum += y >= SP_FAR && y < from && w >= least ? w : 0u;
      }
    }
    const uint32_t n = list_near(r, z, fminf(fminf(from, reach), SP_FAR), near_z[warp]);
#pragma unroll 1
    for (uint32_t b = lane; b < n; b += 32) {
      const uint64_t w = near_weight(pow2, r, near_z[warp][b]);
      sum += w >= least ? w : 0;
    }
    if (__any_sync(0xffffffffu, sum != 0)) sum = warp_sum_u64(sum);   // (the list is read)
    if (lane == 0) sums[chunk - chunk0][warp] = sum;
    uint32_t in = 0;                             // a bit a token
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = distance(r, z[i]);
      in |= y >= from && y < end ? 1u << i : 0u;
    }
    if (!__any_sync(0xffffffffu, in != 0)) continue;
    uint32_t upto = static_cast<uint32_t>(__popc(in));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    uint32_t to = 0;
    if (lane == 31) to = atomicAdd(&st.listed, upto);
    to = __shfl_sync(0xffffffffu, to, 31) + upto - static_cast<uint32_t>(__popc(in));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (in >> i & 1u) {
        if (to < SP_LIST)
          st.list[to] = static_cast<uint64_t>(order_key(z[i])) << 32 | (0xffffffffu - static_cast<uint32_t>(id0 + i));
        ++to;
      }
    }
  }
  __syncthreads();
  for (int chunk = chunk0 + warp; chunk < chunk1; chunk += SP_WARPS) {
    const uint64_t sum = warp_sum_u64(lane < SP_WARPS ? sums[chunk - chunk0][lane] : 0);
    if (lane == 0) st.total[chunk] = sum;
  }
}

struct SampleShared {
  Pow2 pow2[64];
  // bins of a bin: how many tokens, and their weight in two words
  uint32_t count[SP_BINS], lo[SP_BINS], hi[SP_BINS];
  uint64_t list[SP_SORT];        // key << 32 | ~id
  uint32_t total_lo[SP_MAX_CHUNKS], total_hi[SP_MAX_CHUNKS];   // weight of each chunk, in two words
  BlockScan scan;
  uint64_t sum;
  uint32_t listed;
  uint32_t digit, in_digit;      // where the cut falls, and how many tokens fall there
  uint64_t before;               // number or weight before it
  uint32_t cut_key, cut_id;
};

// Adds to a sum in two words of shared memory (its atomic additions are of 32 bits).
__device__ __forceinline__ void add_words(uint32_t& lo, uint32_t& hi, uint64_t w) {
  const uint32_t l = static_cast<uint32_t>(w), old = atomicAdd(&lo, l);
  const uint32_t h = static_cast<uint32_t>(w >> 32) + (old + l < old ? 1u : 0u);
  if (h) atomicAdd(&hi, h);
}

// Sorts the threads' e, the first n of them other than 0 and unlike one another, largest first: a warp's own by a bitonic
// network of shuffles, then runs by twos, each element's place being its own and the number of the other run's before it.
// (One row of 32000 with 430 tokens listed: 17.1 us, 17.4 with the network all the way.)  It overwrites s.list and s.count.
__device__ __forceinline__ void sort_threads(SampleShared& s, int n, uint64_t& e) {
  const int t = threadIdx.x, lane = t & 31;
  int width = 32;
  while (width < n) width <<= 1;
  if (t >= width) return;
#pragma unroll 1
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll 1
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, e, stride);
      const bool larger = ((lane & stride) == 0) == ((lane & size) == 0);   // of the two, this thread keeps the larger
      e = (e > o) == larger ? e : o;
    }
  }
  if (width == 32) return;
  static_assert(sizeof(s.count) >= sizeof(s.list), "a second list");
  uint64_t* from = s.list;
  uint64_t* to = reinterpret_cast<uint64_t*>(s.count);
  from[t] = e;
  sm100::named_barrier(1, width);
#pragma unroll 1
  for (int run = 32; run < width; run <<= 1) {
    const uint64_t* other = from + ((t & ~(run - 1)) ^ run);
    const bool later = (t & run) != 0;           // this run stands behind the other: equals (zeros) of that come first
    int before = 0;
#pragma unroll 1
    for (int step = run; step > 0; step >>= 1) {
      const int at = before + step - 1;
      if (at < run) {
        const uint64_t o = other[at];
        if (o > e || (later && o == e)) before += step;
      }
    }
    to[(t & ~(2 * run - 1)) + (t & (run - 1)) + before] = e;
    sm100::named_barrier(1, width);
    e = to[t];
    uint64_t* spare = from;
    from = to;
    to = spare;
  }
}

__device__ __forceinline__ float z_of(uint64_t e) { return key_value(static_cast<uint32_t>(e >> 32)); }
__device__ __forceinline__ uint32_t id_of(uint64_t e) { return 0xffffffffu - static_cast<uint32_t>(e); }

// Whether the cut keeps a token.
struct Cut {
  float z;
  uint32_t id;
  __device__ __forceinline__ Cut(uint32_t key, uint32_t i)   // (key 0: it keeps all)
      : z(key ? key_value(key) : -INFINITY), id(key ? i : 0xffffffffu) {}
  __device__ __forceinline__ bool keeps(float x, int i) const {
    return x > z || (x == z && static_cast<uint32_t>(i) <= id);
  }
};

// A row's tokens, or those of its list, where that holds all that are asked for.
template <typename T>
struct Tokens {
  const T* logits;
  int vocab;
  const uint64_t* list;
  uint32_t listed;               // 0: the row's
  // Calls f(id, z) for each.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (listed) {
#pragma unroll 1
      for (uint32_t i = threadIdx.x; i < listed; i += SP_THREADS) f(static_cast<int>(id_of(list[i])), z_of(list[i]));
      return;
    }
    const bool wide = (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
#pragma unroll 1
    for (int chunk = 0; chunk * SP_CHUNK < vocab; ++chunk) {
      float z[8];
      load_logits(logits, chunk_id(chunk), vocab, wide, z);
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const float x = z[0];
        f(chunk_id(chunk) + i, x);
#pragma unroll
        for (int q = 0; q < 7; ++q) z[q] = z[q + 1];
      }
    }
  }
};

// The cut among the tokens at distances from `from` to `to`, by going over them: where their number (by_weight false) or
// weight, on top of that before them, reaches `need`.  s.cut_*; the key is 0 where it never does.
template <typename T>
__device__ __noinline__ void find_cut(SampleShared& s, const Row r, const Tokens<T> tk, float from, float to,
                                      bool by_weight, uint64_t need, uint64_t before) {
  const float bins = static_cast<float>(SP_BINS) / (to - from);
  const int t = threadIdx.x;
  uint32_t bin = 0, prefix = 0, there = 0;
  int level = 0;                                 // the bin, then 10, 10, 10 and 2 bits of the logit's order
  auto bin_of = [&](float z) {
    return static_cast<uint32_t>(fminf((distance(r, z) - from) * bins, static_cast<float>(SP_BINS - 1)));
  };
  auto shift = [](int l) { return l >= 4 ? 0 : 32 - 10 * l; };
  auto chosen = [&](float z) {
    const float y = distance(r, z);
    if (!(y < to) || y < from) return false;
    if (level == 0) return true;
    if (bin_of(z) != bin) return false;
    return level == 1 || order_key(z) >> shift(level - 1) == prefix;
  };
  do {
    for (int b = t; b < SP_BINS; b += SP_THREADS) s.count[b] = s.lo[b] = s.hi[b] = 0;
    if (t == 0) s.in_digit = 0;
    __syncthreads();
    tk.each([&](int, float z) {
      if (!chosen(z)) return;
      const uint32_t d = level == 0 ? bin_of(z) : (order_key(z) >> shift(level)) & (level == 4 ? 3u : SP_BINS - 1u);
      atomicAdd(&s.count[d], 1u);
      if (by_weight) add_words(s.lo[d], s.hi[d], weight(s.pow2, r, z));
    });
    __syncthreads();
    // the digits in falling order of z: bins as they are, bits from the largest down
    uint64_t own[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int b = level == 0 ? 2 * t + q : SP_BINS - 1 - 2 * t - q;
      own[q] = by_weight ? static_cast<uint64_t>(s.hi[b]) << 32 | s.lo[b] : s.count[b];
    }
    uint64_t sofar = before + block_before(s.scan, own[0] + own[1]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (sofar < need && sofar + own[q] >= need) {
        const int b = level == 0 ? 2 * t + q : SP_BINS - 1 - 2 * t - q;
        s.digit = b;
        s.in_digit = s.count[b];
        s.before = sofar;
      }
      sofar += own[q];
    }
    __syncthreads();
    there = s.in_digit;
    if (there == 0) {
      if (t == 0) s.cut_key = 0;
      __syncthreads();
      return;
    }
    before = s.before;
    if (level == 0) bin = s.digit;
    else prefix = level == 4 ? prefix << 2 | s.digit : prefix << 10 | s.digit;
    ++level;
    __syncthreads();                             // the state is read before the next pass writes it
  } while (there > SP_SORT && level < 5);
  if (there <= SP_SORT) {
    if (t == 0) s.listed = 0;
    __syncthreads();
    tk.each([&](int id, float z) {
      if (chosen(z))
        s.list[atomicAdd(&s.listed, 1u)] =
            static_cast<uint64_t>(order_key(z)) << 32 | (0xffffffffu - static_cast<uint32_t>(id));
    });
    __syncthreads();
    uint64_t e = t < static_cast<int>(there) ? s.list[t] : 0;
    sort_threads(s, static_cast<int>(there), e);
    const uint64_t w = !e ? 0 : by_weight ? weight(s.pow2, r, z_of(e)) : 1;
    const uint64_t upto = before + block_before(s.scan, w);
    if (upto < need && upto + w >= need) s.cut_key = static_cast<uint32_t>(e >> 32), s.cut_id = id_of(e);
    __syncthreads();
    return;
  }
  // Tokens of one value, more than the list takes: the cut is the m-th of them by id.
  const uint64_t one = by_weight ? weight(s.pow2, r, key_value(prefix)) : 1, m = (need - before + one - 1) / one;
  uint64_t sofar = 0;
  const bool wide = (reinterpret_cast<uintptr_t>(tk.logits) & 15) == 0;
#pragma unroll 1
  for (int chunk = 0; chunk * SP_CHUNK < tk.vocab && sofar < m; ++chunk) {
    float z[8];
    load_logits(tk.logits, chunk_id(chunk), tk.vocab, wide, z);
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) in |= chosen(z[i]) ? 1u << i : 0u;
    uint64_t k = sofar + block_before(s.scan, __popc(in));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (in >> i & 1u) {
        if (++k == m) s.cut_key = prefix, s.cut_id = static_cast<uint32_t>(chunk_id(chunk) + i);
      }
    if (t == SP_THREADS - 1) s.sum = k;
    __syncthreads();
    sofar = s.sum;
    __syncthreads();
  }
}

// 4. A row's cut, the weight of each chunk up to it, and the draw.
template <typename T>
__global__ void __launch_bounds__(SP_THREADS, 2) sample_draw_kernel(SampleParams p) {
  __shared__ SampleShared s;
  LaunchStamp ls(p.stamp);
  const int t = threadIdx.x, lane = t & 31;
  const int row = p.row0 + blockIdx.x;
  fill_pow2(s.pow2);
  if (t == 0) s.cut_key = s.cut_id = 0;
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int request = row / p.rows_each;
  if (unused(p, row, request)) return;
  SampleRow& st = p.state[blockIdx.x];
  // (everything at once: what is not there is not used)
  uint64_t e, sum = 0;
  asm volatile("ld.global.u64 %0, [%1];" : "=l"(e) : "l"(&st.list[t]) : "memory");
  if (t < p.chunks) asm volatile("ld.global.u64 %0, [%1];" : "=l"(sum) : "l"(&st.total[t]) : "memory");
  const int kind = st.kind;
  const Row r = row_of(st);
  const uint64_t least = st.least, need = st.need, before = st.before;
  const float from = st.from, end = st.end;
  const uint32_t n = st.listed;
  const float top_p = kind == ROW_COUNT ? st.top_p : 1.0f;
  const uint32_t u = p.token ? p.u[row] : 0;
  if (kind < ROW_WHOLE) return;
  const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
  if (t < SP_MAX_CHUNKS) {
    s.total_lo[t] = static_cast<uint32_t>(sum);
    s.total_hi[t] = static_cast<uint32_t>(sum >> 32);
  }
  if (t >= static_cast<int>(min(n, static_cast<uint32_t>(SP_SORT)))) e = 0;
  __syncthreads();
  if (n > SP_SORT) {
    const Tokens<T> tk{logits, p.vocab, st.list, n <= SP_LIST ? n : 0};
    find_cut(s, r, tk, from, end, kind == ROW_WEIGH, need, before);
    if (top_p < 1.0f) {                          // of the weight of those k
      const Cut cut(s.cut_key, s.cut_id);
      uint64_t mine = 0;
      tk.each([&](int id, float z) {
        if (cut.keeps(z, id)) mine += weight(s.pow2, r, z);
      });
      const uint64_t upto = block_before(s.scan, mine) + mine;
      if (t == SP_THREADS - 1) s.sum = upto;
      __syncthreads();
      find_cut(s, r, tk, 0.0f, SP_NONE, true, needed(top_p, s.sum), 0);
    }
    const Cut cut(s.cut_key, s.cut_id);
    tk.each([&](int id, float z) {
      const float y = distance(r, z);
      if (y >= from && y < SP_NONE && cut.keeps(z, id)) {
        const uint64_t w = weight(s.pow2, r, z);
        if (w && w >= least) add_words(s.total_lo[id / SP_CHUNK], s.total_hi[id / SP_CHUNK], w);
      }
    });
  } else if (n > 0) {
    sort_threads(s, static_cast<int>(n), e);
    const uint64_t w = e ? weight(s.pow2, r, z_of(e)) : 0;
    bool in = e != 0;
    if (kind == ROW_COUNT) in = in && before + t < need;
    if (kind == ROW_WEIGH || top_p < 1.0f) {     // the weight before each
      uint64_t sofar = block_before(s.scan, in ? w : 0), enough = need;
      if (kind == ROW_COUNT) {
        if (t == SP_THREADS - 1) s.sum = sofar + (in ? w : 0);
        __syncthreads();
        enough = needed(top_p, s.sum);
      } else {
        sofar += before;
      }
      in = in && sofar < enough;
    }
    // the last of those that are in (they are the first)
    const int kept = __syncthreads_count(in);
    if (t == kept - 1) s.cut_key = static_cast<uint32_t>(e >> 32), s.cut_id = id_of(e);
    if (in && w >= least) add_words(s.total_lo[id_of(e) / SP_CHUNK], s.total_hi[id_of(e) / SP_CHUNK], w);
  }
  __syncthreads();
  const Cut cut(s.cut_key, s.cut_id);
  // the chunk with the draw
  static_assert(SP_MAX_CHUNKS == 64, "two chunks a lane");
  const uint64_t a = static_cast<uint64_t>(s.total_hi[2 * lane]) << 32 | s.total_lo[2 * lane];
  const uint64_t b = static_cast<uint64_t>(s.total_hi[2 * lane + 1]) << 32 | s.total_lo[2 * lane + 1];
  uint64_t upto = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const uint64_t W = __shfl_sync(0xffffffffu, upto, 31);
  if (p.probs && t == 0) {
    st.cut_key = s.cut_key;
    st.cut_id = s.cut_id;
    st.inverse = 1.0f / static_cast<float>(W);
  }
  if (!p.token) return;
  const uint64_t at = scale_uniform(u, W);       // (below W)
  const int l = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
  uint64_t sofar = __shfl_sync(0xffffffffu, upto - a - b, l);
  const uint64_t first = __shfl_sync(0xffffffffu, a, l);
  const int chunk = 2 * l + (sofar + first > at ? 0 : 1);
  if (chunk & 1) sofar += first;
  const int id = chunk_id(chunk);
  float z[8];
  load_logits(logits, id, p.vocab, (reinterpret_cast<uintptr_t>(logits) & 15) == 0, z);
  uint64_t w[8], mine = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = weight_of(s.pow2, r, z[i], cut.keeps(z[i], id + i));
    w[i] = w[i] >= least ? w[i] : 0;
    mine += w[i];
  }
  sofar += block_before(s.scan, mine);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (sofar <= at && at < sofar + w[i]) p.token[row] = id + i;
    sofar += w[i];
  }
}

// 5. The probabilities.
template <typename T>
__global__ void __launch_bounds__(SP_THREADS, 3) sample_probs_kernel(SampleParams p) {
  __shared__ Pow2 pow2[64];
  LaunchStamp ls(p.stamp);
  const int at = blockIdx.x / p.groups, row = p.row0 + at;
  const int chunk0 = (blockIdx.x - at * p.groups) * p.pieces, chunk1 = min(chunk0 + p.pieces, p.chunks);
  fill_pow2(pow2);
  __syncthreads();
  pdl_wait();
  ls.waited();
  pdl_trigger();
  if (unused(p, row, row / p.rows_each)) return;
  const SampleRow& st = p.state[at];
  const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
  float* probs = p.probs + row * p.ld_probs;
  const bool wide = (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  const bool wide_out = (reinterpret_cast<uintptr_t>(probs) & 15) == 0;
  Logits<T> next;
  next.load(logits, chunk_id(chunk0), p.vocab, wide);
  const int kind = st.kind;
  const Row r = row_of(st);
  const Cut cut(st.cut_key, st.cut_id);
  const float inverse = st.inverse;
  const uint64_t least = st.least;
  const uint32_t one = kind == ROW_GREEDY ? st.id : 0xffffffffu;
#pragma unroll 1
  for (int chunk = chunk0; chunk < chunk1; ++chunk) {
    const int id = chunk_id(chunk);
    float v[8];
    if (kind < ROW_WHOLE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = static_cast<uint32_t>(id + i) == one ? 1.0f : 0.0f;
    } else {
      float z[8];
      next.get(z);
      if (chunk + 1 < chunk1) next.load(logits, chunk_id(chunk + 1), p.vocab, wide);
      const bool some = __any_sync(0xffffffffu, largest(z) >= cut.z);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = some && cut.keeps(z[i], id + i);
        v[i] = 0.0f;
        if (!some || !__any_sync(0xffffffffu, in)) continue;
        const uint64_t w = weight_of(pow2, r, z[i], in);
        v[i] = w >= least ? static_cast<float>(w) * inverse : 0.0f;
      }
    }
    store_probs(probs, id, p.vocab, wide_out, v);
  }
}

typedef void (*SampleKernel)(SampleParams);
}  // namespace

size_t sample_row_bytes() { return sizeof(SampleRow); }

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
  p.state = static_cast<SampleRow*>(S.rows_state);
  p.arrived = S.arrived;
  p.status = S.status;
  p.chunks = (S.vocab + SP_CHUNK - 1) / SP_CHUNK;
  const bool f32 = S.dtype == EAGLE_DTYPE_F32;
  const SampleKernel kernels[5] = {f32 ? sample_top_kernel<float> : sample_top_kernel<uint16_t>,
                                   f32 ? sample_bins_kernel<float> : sample_bins_kernel<uint16_t>,
                                   f32 ? sample_list_kernel<float> : sample_list_kernel<uint16_t>,
                                   f32 ? sample_draw_kernel<float> : sample_draw_kernel<uint16_t>,
                                   f32 ? sample_probs_kernel<float> : sample_probs_kernel<uint16_t>};
  // bins serve a cut, lists and draws a token or probabilities
  const bool cuts = S.filter->top_k || S.filter->top_p, rest = S.token || S.probs;
  const bool wanted[5] = {true, rest && cuts, rest, rest, S.probs != nullptr};
  for (p.row0 = 0; p.row0 < S.rows; p.row0 += SAMPLE_ROWS) {   // (the state is that of SAMPLE_ROWS rows)
    const int rows = std::min(S.rows - p.row0, SAMPLE_ROWS);
    for (int i = 0; i < 5; ++i) {
      if (!wanted[i]) continue;
      // As many chunks a CTA as let all CTAs, three an SM, take one round in the first kernel, whose rows are alike, and
      // three in the others, where flat rows have more work (64 rows of 131072 of all sorts: one round throughout 79 us,
      // two 59, these 55; the first in two 1.3 more; six in the second 2.5 more).
      const int slots = (i == 0 ? 1 : 3) * 3 * ctx->sm_count, even = (rows * p.chunks + slots - 1) / slots;
      p.pieces = i == 0 ? even : std::min(even, SP_MAX_PIECES);
      p.groups = (p.chunks + p.pieces - 1) / p.pieces;
      p.stamp = stamp_slot(ctx, EAGLE_K_SAMPLE);
      trace_before(ctx, EAGLE_K_SAMPLE, st);
      const cudaError_t e = launch_pdl(kernels[i], dim3(static_cast<unsigned>(rows) * (i == 3 ? 1 : p.groups)),
                                       dim3(SP_THREADS), 0, st, p);
      if (e != cudaSuccess) return e;
      ctx->launches++;
      trace_after(ctx, EAGLE_K_SAMPLE, st);
    }
  }
  return cudaSuccess;
}

}  // namespace eagle
