// eagle_chunk_attn: causal attention of a batch's new rows over the cache
// that holds them, from one token a request to whole prompts.
//
// Rows and items.  The query heads of a kv head share its keys, so a 128-row
// tensor-core tile holds T = 128 / GB tokens x GB heads (GB = the heads per
// kv head, at most 128).  An item is two such tiles (one when the request has
// few rows) of one request and kv head, against the tiles of 128 keys its
// rows can see: max(0, first row's position - window + 1) up to its last
// row's position.  Two tiles read K and V once for 256 rows.
//
// Schedule.  Items differ by orders of magnitude (a decoding token over 64 key
// tiles, a prompt's first rows over one), and their sizes are known on the
// device only.  So the key tiles of all items, laid end to end, are dealt out
// evenly: CTA c of n takes the units [U c / n, U (c + 1) / n), where an item
// counts two units beside its tiles for its ends (queries in, output out, the
// pipeline empty).  Each CTA finds its start itself (a pass of one warp over
// the batch's lengths), walks on from there, and writes the rows of items it
// holds whole; an item that crosses CTAs leaves (max, sum, unnormalised
// output) partials, which the last CTA to arrive combines in CTA order (the
// same bits whoever is last).  Counting the ends took a prompt of 8192 (64/8
// heads) from 819 to 766 us.
//
// One CTA per SM, 384 threads:
//   warp 0      loader: Q tiles, then K and V tiles by TMA into a ring (boxes
//               of one block's rows, out-of-range blocks read as zeros).
//   warps 1, 3  one thread each issues the MMAs of softmax group w = 0, 1:
//               S_w = Q_w K^T into tensor memory in two steps of 64 keys, O_w +=
//               P_w V with P_w (bf16) written over S_w; the next tile's step
//               of S_w goes out behind the products of this tile's.  So
//               a group always has its next 64 scores ready while it is at the
//               exponentials of these.
//   warp 2      scheduler: the walk over items, a few segments ahead; makes
//               rows of V past the request's length zeros.
//   warps 4-11  two softmax warpgroups, thread = query row = tensor-memory
//               lane.  With two tiles warpgroup w has tile w and every key
//               tile; with one, warpgroup w has the key tiles t = w (mod 2) and
//               an O of its own, joined at the item's end.  They also free the
//               ring's slots: scores that are complete show that the products
//               issued before them are (a commit of the MMA threads for each
//               slot cost 250 cycles of their time: 364 -> 342 us in the case
//               below).
// tcgen05, ldmatrix, mma and named barriers take a whole warp: behind a branch
// that lanes take differently they are preceded by __syncwarp, and single
// arrivals between them are predicated instead of branched to (327 -> 319 us).
//
// Bound.  At heads of 128 the products of 128 rows x 128 keys take 1024 cycles
// (measured), in steps of 64 keys 1260: S reads both operands from shared
// memory, 6 KB for 32 cycles of products, 128 bytes a cycle.  A step of the
// softmax takes some 1300 cycles of a warp beside its neighbour.  2048 rows after
// 6144 (64 query / 8 kv heads): 319 us over two inputs in turn, 1.51 PF/s, 0.77
// of a measured bf16 GEMM (342 us, 0.72, over inputs that change every pass);
// tensor pipe 66% active.  S in steps of 128 keys lost more to waiting than it
// gained (384 to 434 us when this took 364).  At heads of 64 the softmax bounds
// it: two prompts of 4096 (16/4 heads) 104 us, 0.66 PF/s.  Heads of 16 and 32
// are staged, multiplied and read as 64: the same case at 12/4 heads of 16, 32
// and 64 takes 71 us each.
//
// The running reference of a row is raised (O and the sum rescaled) only when
// the 64 exponentials of a step add up to more than 256: P stays below 2^8, O / l
// does not depend on when it was raised, and the steps in between take no
// maximum (334 -> 312 us).  P in bf16 (off by 2^-8 of each probability at most) is this
// operator's one rounding besides its output's: with P as a hi + lo pair the
// P V products double, which the fp32 outputs of the tree attention need and a
// bf16 output does not.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "common.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace eagle {
namespace {

constexpr int CH_THREADS = 384;
constexpr int CH_LOAD_WARP = 0, CH_MMA_WARP = 1, CH_SCHED_WARP = 2, CH_SOFT_WARP0 = 4;   // MMA: 1 and 3
constexpr int CH_SOFT_WARPS = 8;
constexpr int CH_SOFT_THREADS = 32 * CH_SOFT_WARPS;
constexpr int CH_KEYS = 128;                 // keys per tile
constexpr int CH_STEP = 64;                  // keys per softmax step
constexpr int CH_ROWS = 128;                 // query rows per tile
constexpr uint32_t CH_HALF = CH_KEYS * 128;  // bytes of 128 rows x 64 elements
constexpr int CH_SEGS = 4;                   // segments the scheduler runs ahead
constexpr float CH_RAISE = 256.0f;           // a step's sum of exponentials from which its reference is raised
constexpr float TK_RAISE = 8.0f;             // in the token phase: the excess of a score over it, in log2 units
constexpr int CH_HEAD = 2;                   // units of an item before its tiles'
constexpr int CH_SNAP = 1;                   // tiles of its ends that no boundary cuts off
constexpr int CH_FOLD = 16;                  // units of a worker from which the token phase pays
// the token phase: requests of at most TK_ROWS query rows a kv head.  At 9 to 16 rows, tiles / token phase: 16 x 2
// rows after 8192 (64/8 heads) 156 / 90 us, 4 x 12 after 4096 (40 heads) 95 / 68, 1 x 12 after 1024 20 / 22.
constexpr int TK_ROWS = 16;
template <int SLOTS>
constexpr int TK_STAGES = SLOTS == 5 ? 3 : 5;  // ring stages of a warp (for heads of 128, of 64 elements)

constexpr uint32_t CH_TM_S = 0, CH_TM_O = 256, CH_TM_COLS = 512;   // S_w / P_w at 128 w, O_w at 256 + 128 w
constexpr int CH_REGS_FEW = 56, CH_REGS_SOFT = 224;
static_assert(128 * CH_REGS_FEW + 256 * CH_REGS_SOFT <= CH_THREADS * 168, "the split fits the launch's registers");

// D: elements of a head as staged (64, or 128); ring slots of one K or V tile.
template <int D>
struct Shape {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t TILE = HALVES * CH_HALF;       // bytes of a Q, K or V tile
  static constexpr int SLOTS = D == 128 ? 5 : 10;
  static constexpr uint32_t TILES = (2 + SLOTS) * TILE;    // two Q tiles, then the ring
};

struct ChunkParams {
  PackedRows rows;
  int hkv, G, GB, T, nsub;                   // kv heads, heads of each, heads and tokens of a tile, tiles for G heads
  int dh;
  long long ld_q, ld_o;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  int out32;                                 // 32-byte aligned rows of out
  int cap, window;
  const int32_t* len;
  PagedKv paged;
  int box;                                   // rows of a K / V box
  int grouped;                               // a box brings whole rows, 8 by 8
  float c;                                   // scale * log2 e
  int tensor;                                // some request may have more rows than the token phase takes
  float* part;                               // [2 grid] partials of split items
  int* cnt;                                  // [grid] arrivals at a split item, by its first CTA
  float* tk_part;                            // the token phase's partials by run,
  int* tk_cnt;                               // and arrivals at split items by their first run
  int* status;
  uint64_t* stamp;
};

// A run of an item's key tiles that one CTA takes.
struct Segment {
  int row0;        // packed row of the item's first token
  int tokens;      // of the item
  int pos0;        // position of the first token
  int len;         // rows of the request in the cache
  int b, hk;       // request, kv head
  int head0, heads;     // first query head, and how many of them the tile's GB hold
  int kt0, nt;     // key tiles [kt0, kt0 + nt)
  int two;         // two query tiles
  int whole;       // the item's only segment
  int part;        // partial slot
  int first_run, n_parts;
  int last;        // no segment: the CTA is done
};

// What the warps share, behind the tiles.
template <int SLOTS>
struct Shared {
  uint64_t full[SLOTS], empty[SLOTS], seg_full[CH_SEGS], seg_empty[CH_SEGS];
  uint64_t raw[SLOTS];                     // V tiles that end past the length: landed, not yet zeroed there
  uint64_t tm_ready, q_full, q_empty, s_full[2][2], p_full[2][2], o_half[2], o_full[2], join, done;
  Segment seg[CH_SEGS];
  float m[2][CH_ROWS], l[2][CH_ROWS];
  uint64_t tk_full[CH_SOFT_WARPS * TK_STAGES<SLOTS>];
  int tk_prev;
  uint64_t tk_done;
  uint32_t tmem;
  int abort, never, prev;
};
template <int D>
constexpr size_t chunk_smem() {
  return Shape<D>::TILES + sizeof(Shared<Shape<D>::SLOTS>);
}
static_assert(chunk_smem<128>() <= (227u << 10) && chunk_smem<64>() <= (227u << 10), "one CTA's shared memory");

// ---- the walk over items (one warp) -------------------------------------------

struct Request {
  int row0, n, len, per, items;              // tokens per item, items per kv head part
  bool bad, over;
};

// Requests of few rows (a decoding step's) are taken by the token phase, the
// others by the tensor-memory phase; each walks the requests of its own class.
enum : int { TENSOR = 0, TOKEN = 1 };

// a / b of non-negative numbers, in 32 bits where they fit (a 64-bit division
// is a few hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (static_cast<unsigned long long>(a | b) >> 32 == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

template <int CLASS>
__device__ __forceinline__ int parts_of(const ChunkParams& p) { return CLASS == TOKEN ? p.hkv : p.hkv * p.nsub; }

// In units of a tile of 128 keys, what an item costs beside its tiles (its
// queries, its output, the empty pipeline at its ends): the first units of an item.
template <int CLASS>
constexpr int HEAD = CLASS == TOKEN ? 0 : CH_HEAD;
template <int CLASS>
constexpr int SNAP = CLASS == TOKEN ? 0 : CH_SNAP;

template <int CLASS>
__device__ __forceinline__ Request request_of(const ChunkParams& p, int b, bool fold) {
  Request r;
  int lo, hi;
  r.bad = !request_rows(p.rows, b, lo, hi);
  const int L = p.len[b];
  r.over = L > p.cap && hi > lo;
  r.len = max(0, min(L, p.cap));
  r.row0 = lo;
  r.n = hi - lo;
  const bool token = !fold && static_cast<long long>(r.n) * p.G <= TK_ROWS;
  if (token != (CLASS == TOKEN)) r.n = 0;
  r.per = CLASS == TOKEN ? max(r.n, 1) : r.n <= p.T ? p.T : 2 * p.T;
  r.items = (r.n + r.per - 1) / r.per;
  return r;
}
__device__ __forceinline__ void take_from(Request& to, const Request& from, int l) {
  to.row0 = __shfl_sync(0xffffffffu, from.row0, l);
  to.n = __shfl_sync(0xffffffffu, from.n, l);
  to.len = __shfl_sync(0xffffffffu, from.len, l);
  to.per = __shfl_sync(0xffffffffu, from.per, l);
  to.items = __shfl_sync(0xffffffffu, from.items, l);
}

// Key tiles [kt0, kt1) of item q (kt1 <= kt0: none of its rows sees a key).
__device__ __forceinline__ void item_tiles(const ChunkParams& p, const Request& r, int q, int& kt0, int& kt1) {
  const int first = r.len - r.n + q * r.per;                 // the first row's position; no sum here passes 32 bits
  const int end = q + 1 < r.items ? first + r.per : r.len;
  const int lo = p.window > 0 && first >= p.window ? first - p.window + 1 : 0;
  kt0 = lo / CH_KEYS;
  kt1 = end > lo ? (end - 1) / CH_KEYS + 1 : kt0;
}
template <int CLASS>
__device__ __forceinline__ int item_units(const ChunkParams& p, const Request& r, int q) {
  int a, z;
  item_tiles(p, r, q, a, z);
  return max(1, z - a) + HEAD<CLASS>;
}

// Units of one kv head part of the lane's own request (every lane calls it;
// requests of many items are summed by the whole warp).
template <int CLASS>
__device__ __forceinline__ long long request_units(const ChunkParams& p, const Request& r, int lane) {
  constexpr int ALONE = 32;                    // (a sum by the warp takes as long as some 30 items by a lane)
  long long w = 0;
  if (r.items <= ALONE)
    for (int q = 0; q < r.items; ++q) w += item_units<CLASS>(p, r, q);
  for (unsigned todo = __ballot_sync(0xffffffffu, r.items > ALONE); todo; todo &= todo - 1) {
    const int l = __ffs(todo) - 1;
    Request s;
    take_from(s, r, l);
    long long part = 0;
    for (int q = lane; q < s.items; q += 32) part += item_units<CLASS>(p, s, q);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == l) w = part;
  }
  return w;
}
template <typename T>
__device__ __forceinline__ T scan_of(T v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
// Inclusive prefix sums of non-negative numbers, in 32 bits where they fit.
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
  if (__any_sync(0xffffffffu, v >> 26)) return scan_of(v, lane);
  return scan_of(static_cast<int>(v), lane);
}

// Units (and items) of the batch's requests, by one warp, 32 requests at a time.
struct Scan {
  Request r;               // the lane's request of the 32 at hand,
  long long units, end;    // its units per kv head part, and the sum up to its end
};
template <int CLASS>
__device__ __forceinline__ void scan_32(const ChunkParams& p, int lane, bool fold, int b0, long long before, Scan& s) {
  s.r = Request{};
  s.r.per = 1;
  if (b0 + lane < p.rows.B) s.r = request_of<CLASS>(p, b0 + lane, fold);
  s.units = request_units<CLASS>(p, s.r, lane);
  s.end = before + warp_scan(s.units * parts_of<CLASS>(p), lane);
}
template <int CLASS>
__device__ __forceinline__ long long scan_batch(const ChunkParams& p, int lane, bool fold, bool report, Scan& s,
                                                int& items) {
  constexpr int MANY = 1 << 16;                // (more than there are workers)
  long long sum = 0;
  items = 0;
  for (int b0 = 0; b0 < p.rows.B; b0 += 32) {
    scan_32<CLASS>(p, lane, fold, b0, sum, s);
    if (report && s.r.bad) set_status(p.status, EAGLE_ERR_INVALID_ARG);
    if (report && s.r.over) set_status(p.status, EAGLE_ERR_CAPACITY);
    items = static_cast<int>(min(static_cast<long long>(MANY),
                                 items + static_cast<long long>(s.r.items) * parts_of<CLASS>(p)));
    sum = __shfl_sync(0xffffffffu, s.end, 31);
  }
  items = __reduce_add_sync(0xffffffffu, items);
  return sum;
}

// The walk's place: item q of kv head part hs of request b, whose first unit
// is `unit` of all.
struct Walk {
  Request r;
  int b, hs, q;
  long long unit;
};

// The item that holds unit u0; s is what scan_batch left.
template <int CLASS>
__device__ __forceinline__ void walk_to(const ChunkParams& p, int lane, bool fold, long long u0, Scan& s, Walk& w) {
  const int parts = parts_of<CLASS>(p);
  long long sum = 0;
  for (int b0 = 0; b0 < p.rows.B; b0 += 32) {
    if (p.rows.B > 32) scan_32<CLASS>(p, lane, fold, b0, sum, s);
    const unsigned past = __ballot_sync(0xffffffffu, s.end > u0);
    if (past) {
      const int l = __ffs(past) - 1;
      w.b = b0 + l;
      take_from(w.r, s.r, l);
      const long long W = __shfl_sync(0xffffffffu, s.units, l);
      const long long begin = __shfl_sync(0xffffffffu, s.end - s.units * parts, l);
      w.hs = static_cast<int>(quotient(u0 - begin, W));
      long long at = begin + W * w.hs;         // first unit of the part
      w.q = 0;
      w.unit = at;
      for (int q0 = 0; CLASS == TENSOR && q0 < w.r.items; q0 += 32) {   // (TOKEN: one item)
        const int q = q0 + lane;
        const long long v = q < w.r.items ? item_units<CLASS>(p, w.r, q) : 0;
        const long long upto = at + warp_scan(v, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, upto > u0 && q < w.r.items);
        if (hit) {
          const int k = __ffs(hit) - 1;
          w.q = q0 + k;
          w.unit = __shfl_sync(0xffffffffu, upto - v, k);
          break;
        }
        at = __shfl_sync(0xffffffffu, upto, 31);
      }
      return;
    }
    sum = __shfl_sync(0xffffffffu, s.end, 31);
  }
}

// To the next item; false at the batch's end.
template <int CLASS>
__device__ __forceinline__ bool walk_on(const ChunkParams& p, bool fold, Walk& w, int lane) {
  if (++w.q < w.r.items) return true;
  w.q = 0;
  if (++w.hs < parts_of<CLASS>(p)) return true;
  w.hs = 0;
  for (int b0 = w.b + 1; b0 < p.rows.B; b0 += 32) {
    Request r{};
    if (b0 + lane < p.rows.B) r = request_of<CLASS>(p, b0 + lane, fold);
    const unsigned some = __ballot_sync(0xffffffffu, r.n > 0);
    if (some) {
      const int l = __ffs(some) - 1;
      w.b = b0 + l;
      take_from(w.r, r, l);
      return true;
    }
  }
  return false;
}

// The units in n even runs; run c, [U c / n, U (c + 1) / n), segment by
// segment.  A boundary within an item's head or SNAP tiles of its ends moves
// there: no run takes a head without tiles, or a few tiles at the price of a
// partial.
template <int CLASS>
struct Runs {
  Scan s;
  Walk w;
  long long U, n, c, at, end;
  int items;
  bool fold;               // every request counts as TENSOR
  static constexpr int NEAR = HEAD<CLASS> + SNAP<CLASS>;   // boundaries up to here move to the item's start
  __device__ __forceinline__ void scan(const ChunkParams& p, int lane, bool all_tensor, bool report) {
    fold = all_tensor;
    U = scan_batch<CLASS>(p, lane, fold, report, s, items);
  }
  // One run a worker; with fewer items than workers, the same number for every item where that idles at most a fifth of
  // them, so that runs of equal items do not cross them (32 items of 8 units: 152 runs 16.2 us, 128 runs 10.3; but 80
  // items of 34 units: 80 runs 100 us, 152 runs 75).  (Two or four runs a worker, claimed one after another, were
  // slower: more partials.)
  __device__ __forceinline__ void split(int workers) {
    n = workers;
    if (items > 0 && items < workers) {
      const int even = workers - workers % items;
      if (5 * even >= 4 * workers) n = even;
    }
    n = min(n, U);
  }
  __device__ __forceinline__ void begin(const ChunkParams& p, int lane, long long run) {
    c = run;
    at = c < n ? quotient(U * c, n) : 0;
    end = c < n ? quotient(U * (c + 1), n) : 0;
    if (at >= end) return;
    walk_to<CLASS>(p, lane, fold, at, s, w);
    const int units = item_units<CLASS>(p, w.r, w.q);
    if (at - w.unit > NEAR && at - w.unit >= units - SNAP<CLASS>) {
      w.unit += units;
      if (!walk_on<CLASS>(p, fold, w, lane)) {
        at = end;
        return;
      }
      at = w.unit;
    } else if (at - w.unit <= NEAR) {
      at = w.unit;
    }
  }
  __device__ __forceinline__ Segment next(const ChunkParams& p, int lane) {
    constexpr int H = HEAD<CLASS>;
    Segment g{};
    g.last = at >= end;
    if (g.last) return g;
    int kt0, kt1;
    item_tiles(p, w.r, w.q, kt0, kt1);
    const int units = max(1, kt1 - kt0) + H;
    const int x0 = static_cast<int>(at - w.unit);
    int x1 = static_cast<int>(min(static_cast<long long>(units), end - w.unit));
    if (x1 < units) {
      g.last = x1 <= NEAR;
      if (g.last) return g;
      if (x1 >= units - SNAP<CLASS>) x1 = units;
    }
    const int nsub = CLASS == TOKEN ? 1 : p.nsub;
    const int hk = w.hs / nsub, sub = w.hs - hk * nsub;
    const int t0 = w.q * w.r.per;
    g.row0 = w.r.row0 + t0;
    g.tokens = min(w.r.per, w.r.n - t0);
    g.pos0 = w.r.len - w.r.n + t0;
    g.len = w.r.len;
    g.b = w.b;
    g.hk = hk;
    g.head0 = hk * p.G + sub * p.GB;
    g.heads = min(p.GB, p.G - sub * p.GB);
    const int first = max(x0 - H, 0);        // of the item's tiles
    g.kt0 = kt0 + first;
    g.nt = kt1 > kt0 ? x1 - H - first : 0;
    g.two = g.tokens > p.T;
    g.whole = x0 == 0 && x1 == units;
    if (!g.whole) {
      // the largest run that begins at or before unit u: u the last from where a boundary moves to the item's start,
      // and the last from where it does not move to its end (a split item is longer than NEAR + SNAP)
      g.first_run = static_cast<int>(quotient((w.unit + NEAR + 1) * n - 1, U));
      g.n_parts = static_cast<int>(quotient((w.unit + units - SNAP<CLASS>) * n - 1, U)) - g.first_run + 1;
      g.part = 2 * static_cast<int>(c) + (x0 == 0 ? 1 : 0);
    }
    at = w.unit + x1;
    if (x1 == units) {
      w.unit += units;
      if (at < end && !walk_on<CLASS>(p, fold, w, lane)) at = end;
    }
    return g;
  }
};

// What the batch holds: requests of few rows, and whether they go with the
// others, without a token phase: where there are others, and a worker's share
// of their units is small.  A token phase of few units is latency, 10 us or
// so; its streaming pays from long prefixes of many requests on.  512 rows of a
// prompt beside single tokens (40 heads), with the phase / in tiles: 2.1 units
// a worker 58 / 50 us, 8.4: 64 / 53, 16.8: 72 / 72, 34: 99 / 109, 135: 264 / 337;
// 64/8 heads, 13.5: 69 / 68, 27: 88 / 99.
struct Mix {
  bool few, fold;
};
__device__ __forceinline__ Mix mix_of(const ChunkParams& p, int lane) {
  constexpr int MANY = 1 << 24;
  int units = 0;
  bool few = false, others = false;
  if (p.G <= TK_ROWS) {
    for (int b = lane; b < p.rows.B; b += 32) {
      const Request r = request_of<TOKEN>(p, b, false);
      int lo, hi;
      request_rows(p.rows, b, lo, hi);
      few = few || r.n > 0;
      others = others || hi - lo > r.n;
      if (r.n > 0)
        units = static_cast<int>(min(static_cast<long long>(MANY),
                                     units + static_cast<long long>(item_units<TOKEN>(p, r, 0)) * parts_of<TOKEN>(p)));
    }
    few = __any_sync(0xffffffffu, few);
    others = __any_sync(0xffffffffu, others);
    units = __reduce_add_sync(0xffffffffu, units);
  }
  return Mix{few, few && others && units < CH_FOLD * static_cast<int>(gridDim.x)};
}

// ---- softmax of one tile -------------------------------------------------------

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The lowest n bits of a word (none below 1, all from 32 on).
__device__ __forceinline__ uint32_t first_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// This thread's row of one step of S_w (64 columns): P_w into tensor memory
// over it, and the row sum.  Column j is visible when lo <= j <= hi (masked; all
// are otherwise).  The exponentials are against the reference of the steps
// before; a row that has none yet takes the step's maximum first.  Only where
// a row's exponentials add up to more than CH_RAISE is its reference raised to
// the step's maximum, O_w and the sum rescaled, and the step done again.
// `at_rest` waits until every product into O_w so far is complete.
template <int D, typename Wait>
__device__ __forceinline__ bool softmax_step(uint32_t s_addr, uint32_t o_addr, bool masked, int lo, int hi,
                                             bool valid, float c, float& m_ref, float& l_sum, uint64_t* p_full,
                                             Wait at_rest) {
  float sv[2][32];
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < 2; ++k) sm100::tmem_ld32(s_addr + 32u * k, sv[k]);
    sm100::tmem_wait_ld();
    if (masked) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t see = first_bits(hi + 1 - 32 * k) & ~first_bits(lo - 32 * k);
#pragma unroll
        for (int j = 0; j < 32; ++j) sv[k][j] = see & (1u << j) ? sv[k][j] : -INFINITY;
      }
    }
  };
  uint32_t pw[32];
  float2 sum;
  auto exps = [&]() {
    const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
    const float2 c2 = make_float2(c, c), nm2 = make_float2(nm, nm);
    sum = make_float2(0.f, 0.f);
    float2 ps[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ps[i] = make_float2(0.f, 0.f);
    constexpr int NB = 8;
    float2 e[2][NB];
#pragma unroll
    for (int g = 0; g <= 32 / NB; ++g) {
      if (g < 32 / NB) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int j = g * NB + i;
          e[g & 1][i] = __ffma2_rn(make_float2(sv[j >> 4][2 * (j & 15)], sv[j >> 4][2 * (j & 15) + 1]), c2, nm2);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(e[g & 1][i].x));
          asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(e[g & 1][i].y));
        }
      }
      if (g > 0) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int j = (g - 1) * NB + i;
          const float2 y = e[(g & 1) ^ 1][i];
          ps[i % 4] = __fadd2_rn(ps[i % 4], y);
          uint32_t w;
          asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y.y), "f"(y.x));
          pw[j] = w;
        }
      }
    }
    sum = __fadd2_rn(__fadd2_rn(ps[0], ps[1]), __fadd2_rn(ps[2], ps[3]));
  };
  auto most = [&]() {
    float mx[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mx[k] = fmaxf(sv[k >> 1][16 * (k & 1)], sv[k >> 1][16 * (k & 1) + 1]);
#pragma unroll
      for (int j = 2; j < 16; j += 2)
        mx[k] = max3(mx[k], sv[k >> 1][16 * (k & 1) + j], sv[k >> 1][16 * (k & 1) + j + 1]);
    }
    return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
  };
  load();
  if (__any_sync(0xffffffffu, valid && m_ref == -INFINITY)) {
    const float mt = most();
    m_ref = m_ref == -INFINITY ? mt : m_ref;   // nothing summed yet
  }
  exps();
  const bool raise = valid && sum.x + sum.y > CH_RAISE;
  if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
    if (!at_rest()) return false;
    sm100::tc_fence_after();
    load();                                    // the scores once more (their registers went to P)
    const float mt = most();
    const float f = raise ? sm100::exp2(m_ref - mt) : 1.f;
#pragma unroll 1
    for (int q = 0; q < D / 16; ++q) {
      float o[16];
      sm100::tmem_ld16(o_addr + 16u * q, o);
      sm100::tmem_wait_ld();
      uint32_t x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(o[j] * f);
      sm100::tmem_st16(o_addr + 16u * q, x);
    }
    l_sum *= f;
    m_ref = raise ? mt : m_ref;
    exps();
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = pw[16 * k + j];
    sm100::tmem_st16(s_addr + 16u * k, x);
  }
  sm100::tmem_wait_st();
  sm100::tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(p_full);
  l_sum += sum.x + sum.y;
  return true;
}

// 16 bf16 elements of a thread's own row, a line that no other thread of the warp writes.
__device__ __forceinline__ void store16(const ChunkParams& p, uint16_t* dst, const uint32_t* x) {
  if (p.out32) {                             // half as many passes as 16-byte stores
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// A split item's partials joined in run order, by the softmax threads: a
// thread takes CN runs of four columns of its row at a time, from c0 on.
template <int D, int CN>
__device__ __forceinline__ void merge_row(const ChunkParams& p, const Segment& g, int r, int c0, int cols,
                                          uint16_t* dst) {
  constexpr int PART = 2 * CH_ROWS * (D + 2);
  const int n_parts = g.n_parts;
  const float* first = p.part + static_cast<size_t>(2 * g.first_run + 1) * PART;
  // the parts after the first are two slots apart, from the first's neighbour on
  auto slot_of = [&](int k) { return first + (k == 0 ? 0 : static_cast<size_t>(2 * k - 1) * PART); };
  float M = -INFINITY;
#pragma unroll 8
  for (int k = 0; k < n_parts; ++k) M = fmaxf(M, __ldcg(slot_of(k) + 2 * CH_ROWS * D + r));
  for (int c = c0; c < c0 + cols; c += CN) {
    float l = 0.f;
    float4 o[CN];
#pragma unroll
    for (int j = 0; j < CN; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll(CN == 1 ? 8 : 2)
    for (int k = 0; k < n_parts; ++k) {
      const float* sp = slot_of(k);
      const float m = __ldcg(sp + 2 * CH_ROWS * D + r), lk = __ldcg(sp + 2 * CH_ROWS * D + 2 * CH_ROWS + r);
      float4 v[CN];
#pragma unroll
      for (int j = 0; j < CN; ++j) v[j] = __ldcg(reinterpret_cast<const float4*>(sp) + (c + j) * (2 * CH_ROWS) + r);
      const float f = m == -INFINITY ? 0.f : sm100::exp2(m - M);
      l = fmaf(f, lk, l);
#pragma unroll
      for (int j = 0; j < CN; ++j) {
        o[j].x = fmaf(f, v[j].x, o[j].x);
        o[j].y = fmaf(f, v[j].y, o[j].y);
        o[j].z = fmaf(f, v[j].z, o[j].z);
        o[j].w = fmaf(f, v[j].w, o[j].w);
      }
    }
    const float z = l > 0.f ? 1.f / l : 0.f;
    uint32_t x[2 * CN];
#pragma unroll
    for (int j = 0; j < CN; ++j) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(o[j].x * z, o[j].y * z);
      const __nv_bfloat162 b = __floats2bfloat162_rn(o[j].z * z, o[j].w * z);
      x[2 * j] = *reinterpret_cast<const uint32_t*>(&a);
      x[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (CN == 8) {
#pragma unroll
      for (int q = 0; q < CN / 4; ++q)
        if (4 * c + 16 * q < p.dh) store16(p, dst + 4 * c + 16 * q, x + 8 * q);
    } else if (4 * c < p.dh) {
      *reinterpret_cast<uint2*>(dst + 4 * c) = make_uint2(x[0], x[1]);
    }
  }
}
template <int D>
__device__ __forceinline__ void merge_parts(const ChunkParams& p, const Segment& g, int st) {
  // rows side by side in the threads (their partials are), as many threads a row as there are
  const int n_rows = g.two ? 2 * CH_ROWS : min(CH_ROWS, g.tokens * p.GB);
  const int log_rows = 32 - __clz(n_rows - 1);           // of the rows rounded up to a power of two
  const int r = st & ((1 << log_rows) - 1);
  const int rt = r & (CH_ROWS - 1), t = rt / p.GB, h = rt - t * p.GB;
  const int ti = (r >= CH_ROWS ? p.T : 0) + t;
  const int per = CH_SOFT_THREADS >> log_rows, cols = max(1, D / 4 / per), c0 = (st >> log_rows) * cols;
  if (t >= p.T || ti >= g.tokens || h >= g.heads || c0 >= D / 4) return;
  uint16_t* dst = p.out + (static_cast<size_t>(g.row0) + ti) * p.ld_o + (g.head0 + h) * p.dh;
  if (cols >= 8) merge_row<D, 8>(p, g, r, c0, cols, dst);
  else merge_row<D, 1>(p, g, r, c0, cols, dst);
}

// ---- the token phase --------------------------------------------------------------
//
// Requests of at most 16 query rows a kv head (one decoding token and its
// group) read every key for a handful of rows: the cache's bytes are all that
// counts.  An item is one kv head of a request; each of the eight softmax warps
// takes 16 of a tile's 128 keys through a ring of its own, with no barrier
// between warps and an online softmax of its own, and the eight states are
// joined at a segment's end.  One lane requests a step by TMA (per-lane 16-byte
// copies spent 2300 of a step's 3100 cycles on addresses and the block table).
// The products are warp-level bf16 tiles with the keys as rows, S^T = K Q^T and
// O^T += V^T P^T (m16n8k16): eight query rows fill the narrow side, where Q as
// the 16-row side would be half padding.  (Eight kv heads side by side over
// the same keys, whole cache rows for DRAM, streamed no faster, and one long
// request then left 152 partials of every head: 128 us where this takes 21.)

template <int D>
struct TokenShape {
  static constexpr int STAGES = D == 128 ? 3 : 5;
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t HALF = 16 * 128;               // 16 keys x 64 elements
  static constexpr uint32_t STAGE = 2 * HALVES * HALF;     // K then V
  static constexpr uint32_t JOIN = CH_SOFT_WARPS * STAGES * STAGE;   // after the rings: [8 warps][8 rows][D] fp32
  static constexpr int PART = TK_ROWS * (D + 2);           // floats of a head's partial
  static_assert(JOIN + CH_SOFT_WARPS * 8 * D * 4 <= Shape<D>::TILES, "the tiles' memory");
};

// A warp's place among the eight, and the L2 policy of the cache's lines (read
// once: the first to go, so that a cache larger than L2 does not push out code
// and tables).
struct TokenWarp {
  int w, lane;
  uint64_t policy;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The blocks of a warp's next 32 steps, one in each lane (blocks of at least
// 16 rows: a step lies in one).
struct TokenBlocks {
  int base, blk;
  __device__ __forceinline__ int of(const ChunkParams& p, const Segment& g, const TokenWarp& tw, int u) {
    if (u < base || u >= base + 32) {
      base = u;
      const int key0 = (g.kt0 + u + tw.lane) * CH_KEYS + 16 * tw.w;
      blk = p.paged.n_blocks;                // out of range: reads as zeros
      if (u + tw.lane < g.nt && key0 < g.len) {
        const int x = p.paged.table[static_cast<size_t>(g.b) * p.paged.per_req + (key0 >> p.paged.shift)];
        if (x >= 0 && x < p.paged.n_blocks) blk = x;
        else set_status(p.status, EAGLE_ERR_INVALID_ARG);
      }
    }
    return __shfl_sync(0xffffffffu, blk, u - base);
  }
};

// Step u of segment g -- the warp's 16 keys of a key tile, K then V -- into
// `stage`.  Rows
// past the length within their block arrive as they are, those of blocks that
// do not exist as zeros.
template <int D>
__device__ __forceinline__ void token_load(const ChunkParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap,
                                           const Segment& g, uint8_t* stage, uint64_t* bar, TokenBlocks& blocks,
                                           const TokenWarp& tw, int u) {
  using T = TokenShape<D>;
  const int key0 = (g.kt0 + u) * CH_KEYS + 16 * tw.w;
  const bool paged = p.paged.table != nullptr;
  const int mask = (1 << p.paged.shift) - 1;
  auto box = [&](int y, int z, int row) {
#pragma unroll
    for (int h = 0; h < T::HALVES; ++h) {
      sm100::tma_load_4d_hint(stage + h * T::HALF + row * 128, kmap, 64 * h, g.hk, y, z, bar, tw.policy);
      sm100::tma_load_4d_hint(stage + (T::HALVES + h) * T::HALF + row * 128, vmap, 64 * h, g.hk, y, z, bar, tw.policy);
    }
  };
  if (tw.lane == 0) sm100::mbar_arrive_expect_tx(bar, T::STAGE);
  if (!paged || p.paged.shift >= 4) {
    const int z = paged ? blocks.of(p, g, tw, u) : g.b;
    if (tw.lane == 0) box(paged ? key0 & mask : key0, z, 0);
  } else {
    __syncwarp();
    const int rows = 1 << p.paged.shift;
    if (tw.lane * rows < 16) {
      const int key = key0 + tw.lane * rows;
      int z = p.paged.n_blocks;
      if (key < g.len) {
        const int x = p.paged.table[static_cast<size_t>(g.b) * p.paged.per_req + (key >> p.paged.shift)];
        if (x >= 0 && x < p.paged.n_blocks) z = x;
        else set_status(p.status, EAGLE_ERR_INVALID_ARG);
      }
      box(0, z, tw.lane * rows);
    }
  }
  __syncwarp();
}

// One segment's softmaxes and products by a warp (its nt units are on their
// way or, the first STAGES of them, already requested).  NT: tiles of 8 query
// rows.
template <int D, int NT>
__device__ __forceinline__ void token_segment(const ChunkParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap,
                                              const Segment& g, uint8_t* ring, uint64_t* bars, uint32_t& phases,
                                              int& slot, volatile int* abort, bool& ok, TokenBlocks& blocks,
                                              const TokenWarp& tw, float (&o)[NT][D / 16][4], float (&m)[NT][2],
                                              float (&l)[NT][2]) {
  using T = TokenShape<D>;
  const int lane = tw.lane, gq = lane >> 2, tq = lane & 3;
  const int rows = g.tokens * p.G;
  // Q^T as the B operand: column = query row, k = elements
  uint32_t qf[NT][D / 16][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = 8 * n + gq, t = r / p.G, h = r - t * p.G;
    const uint16_t* q = p.q + (static_cast<size_t>(g.row0) + t) * p.ld_q + (g.head0 + h) * p.dh + 2 * tq;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const bool there = r < rows && 16 * k < p.dh;
      qf[n][k][0] = there ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
      qf[n][k][1] = there ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }
  // what the thread's rows (8 n + 2 tq, + 1) see: [lo, pos]
  int pos[NT][2], lo[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * n + 2 * tq + i;
      pos[n][i] = r < rows ? g.pos0 + r / p.G : -1;
      lo[n][i] = p.window > 0 ? max(0, pos[n][i] - p.window + 1) : 0;
    }
  const int pos_least = g.pos0, lo_most = p.window > 0 ? max(0, g.pos0 + g.tokens - p.window) : 0;
  const uint32_t ring_a = sm100::smem_u32(ring);
  // ldmatrix addresses within a stage: lanes 0-7, 8-15, .. give the rows of the four 8 x 8 blocks
  const int r8 = lane & 7, q4 = lane >> 3;
  const int krow = r8 + 8 * (q4 & 1), kch = q4 >> 1;       // K: keys 0-7 / 8-15, elements 0-7 / 8-15
  const int vrow = r8 + 8 * (q4 >> 1), vch = q4 & 1;       // V: elements 0-7 / 8-15, keys 0-7 / 8-15
  for (int u = 0; u < g.nt; ++u) {
    ok = ok && __all_sync(0xffffffffu, sm100::mbar_wait(&bars[slot], (phases >> slot) & 1u, abort));
    if (ok) phases ^= 1u << slot;
    const uint32_t stage = ring_a + slot * T::STAGE;
    const int key0 = (g.kt0 + u) * CH_KEYS + 16 * tw.w;
    if (key0 + 16 > g.len) {
      // rows past the length may hold anything, and 0 x NaN is NaN: V's become zeros
      uint8_t* v = ring + slot * T::STAGE + T::HALVES * T::HALF;
      for (int x = lane; x < 16 * 8 * T::HALVES; x += 32)
        if (key0 + ((x >> 3) & 15) >= g.len) *reinterpret_cast<uint4*>(v + x * 16) = make_uint4(0u, 0u, 0u, 0u);
      sm100::fence_proxy_async_smem();         // (the stage's next writer is TMA)
      __syncwarp();
    }
    float s[NT][4], z[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = z[n][i] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t a[4];
      ldsm4(a, stage + (k >> 2) * T::HALF + krow * 128 + ((((2 * k + kch) & 7) ^ (krow & 7)) << 4));
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_16816(k & 1 ? z[n] : s[n], a, qf[n][k][0], qf[n][k][1]);
    }
    const bool masked = key0 + 15 > pos_least || key0 < lo_most;
    bool ask = false;
    float mt[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[n][i] = (s[n][i] + z[n][i]) * p.c;
        if (masked) {
          const int key = key0 + gq + 8 * (i >> 1);
          s[n][i] = key >= lo[n][i & 1] && key <= pos[n][i & 1] ? s[n][i] : -INFINITY;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mt[n][i] = fmaxf(s[n][i], s[n][i + 2]);
        ask = ask || mt[n][i] > m[n][i] + TK_RAISE || (m[n][i] == -INFINITY && mt[n][i] != -INFINITY);
      }
    }
    if (__any_sync(0xffffffffu, ask)) {
      // the rows' maxima over the 16 keys; every lane of a row takes the same step
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = mt[n][i];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          if (x > m[n][i]) {
            const float f = m[n][i] == -INFINITY ? 0.f : sm100::exp2(m[n][i] - x);
            m[n][i] = x;
            l[n][i] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[n][j][i] *= f;
              o[n][j][i + 2] *= f;
            }
          }
        }
      __syncwarp();
    }
    uint32_t b[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float n0 = m[n][0] == -INFINITY ? 0.f : m[n][0], n1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
      const float e0 = sm100::exp2(s[n][0] - n0), e1 = sm100::exp2(s[n][1] - n1);
      const float e2 = sm100::exp2(s[n][2] - n0), e3 = sm100::exp2(s[n][3] - n1);
      l[n][0] += e0 + e2;
      l[n][1] += e1 + e3;
      const __nv_bfloat162 x = __floats2bfloat162_rn(e0, e1), y = __floats2bfloat162_rn(e2, e3);
      b[n][0] = transpose8(*reinterpret_cast<const uint32_t*>(&x));
      b[n][1] = transpose8(*reinterpret_cast<const uint32_t*>(&y));
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t a[4];
      ldsm4_t(a, stage + (T::HALVES + (j >> 2)) * T::HALF + vrow * 128 + ((((2 * j + vch) & 7) ^ (vrow & 7)) << 4));
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_16816(o[n][j], a, b[n][0], b[n][1]);
    }
    __syncwarp();                            // every lane has read the stage
    if (ok && u + T::STAGES < g.nt)
      token_load<D>(p, kmap, vmap, g, ring + slot * T::STAGE, &bars[slot], blocks, tw, u + T::STAGES);
    slot = slot + 1 == T::STAGES ? 0 : slot + 1;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], d);
}

__device__ __forceinline__ void all_soft() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(CH_SOFT_THREADS) : "memory");
}
__device__ __forceinline__ void store_bf16x4(uint16_t* dst, float4 v, float z) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * z, v.y * z), b = __floats2bfloat162_rn(v.z * z, v.w * z);
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ uint16_t* token_row(const ChunkParams& p, const Segment& g, int r) {
  const int t = r / p.G, h = r - t * p.G;
  return p.out + (static_cast<size_t>(g.row0) + t) * p.ld_o + (g.head0 + h) * p.dh;
}

// A segment's end: the warps' states joined, 8 query rows at a time, and the
// rows written (a whole item) or left as a partial.
template <int D, int NT>
__device__ __forceinline__ void token_join(const ChunkParams& p, const Segment& g, float* buf, float* sm_m, float* sm_l,
                                           const TokenWarp& tw, const float (&o)[NT][D / 16][4],
                                           const float (&m)[NT][2], const float (&l)[NT][2]) {
  const int lane = tw.lane, gq = lane >> 2, tq = lane & 3, tid = tw.w * 32 + lane;
  const int rows = g.tokens * p.G;
  float* part = p.tk_part + static_cast<size_t>(g.part) * TokenShape<D>::PART;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    all_soft();                              // the buffer's last use is over
    // [warp][row][D], element d of row r at d ^ 8 (r / 2 % 4): the warp's stores fall on different banks
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        buf[(tw.w * 8 + 2 * tq + (i & 1)) * D + ((16 * j + gq + 8 * (i >> 1)) ^ (8 * tq))] = o[n][j][i];
    if (gq == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sm_m[tw.w * 8 + 2 * tq + i] = m[n][i];
        sm_l[tw.w * 8 + 2 * tq + i] = l[n][i];
      }
    }
    all_soft();
    for (int x = tid; x < 8 * (D / 4); x += CH_SOFT_THREADS) {
      const int r = x / (D / 4), c4 = x - r * (D / 4), rr = 8 * n + r;
      if (rr >= rows || 4 * c4 >= p.dh) continue;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < CH_SOFT_WARPS; ++w) M = fmaxf(M, sm_m[w * 8 + r]);
      float L = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < CH_SOFT_WARPS; ++w) {
        const float f = sm_m[w * 8 + r] == -INFINITY ? 0.f : sm100::exp2(sm_m[w * 8 + r] - M);
        const float4 y = *reinterpret_cast<const float4*>(buf + (w * 8 + r) * D + ((4 * c4) ^ (8 * ((r >> 1) & 3))));
        L = fmaf(f, sm_l[w * 8 + r], L);
        v.x = fmaf(f, y.x, v.x);
        v.y = fmaf(f, y.y, v.y);
        v.z = fmaf(f, y.z, v.z);
        v.w = fmaf(f, y.w, v.w);
      }
      if (g.whole) {
        store_bf16x4(token_row(p, g, rr) + 4 * c4, v, L > 0.f ? 1.f / L : 0.f);
      } else {
        *reinterpret_cast<float4*>(part + rr * D + 4 * c4) = v;
        if (c4 == 0) {
          part[TK_ROWS * D + rr] = M;
          part[TK_ROWS * (D + 1) + rr] = L;
        }
      }
    }
  }
}

// A split item's partials joined in run order, a row per warp at a time: lane =
// part for the row's maximum and sum, then lane = four columns.
template <int D>
__device__ __forceinline__ void token_merge(const ChunkParams& p, const Segment& g, const TokenWarp& tw) {
  using T = TokenShape<D>;
  const int lane = tw.lane;
  const float* first = p.tk_part + static_cast<size_t>(2 * g.first_run + 1) * T::PART;
  // the parts after the first are two slots apart, from the first's neighbour on
  auto slot_of = [&](int k) { return first + (k == 0 ? 0 : static_cast<size_t>(2 * k - 1) * T::PART); };
  for (int r = tw.w; r < g.tokens * p.G; r += CH_SOFT_WARPS) {
    float M = -INFINITY, L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < g.n_parts; k0 += 32) {
      const bool there = k0 + lane < g.n_parts;
      const float* sp = slot_of(there ? k0 + lane : 0) + TK_ROWS * D + r;
      const float mk = there ? __ldcg(sp) : -INFINITY, lk = there ? __ldcg(sp + TK_ROWS) : 0.f;
      const float now = fmaxf(M, warp_max(mk));
      const float old = M == -INFINITY ? 0.f : sm100::exp2(M - now);   // of the 32 parts before
      const float f = mk == -INFINITY ? 0.f : sm100::exp2(mk - now);
      M = now;
      L = fmaf(L, old, warp_sum(f * lk));
      v.x *= old;
      v.y *= old;
      v.z *= old;
      v.w *= old;
      const int n = min(32, g.n_parts - k0);
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const float w = __shfl_sync(0xffffffffu, f, k);
        const float4 y = 4 * lane < D ? __ldcg(reinterpret_cast<const float4*>(slot_of(k0 + k) + r * D) + lane)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
        v.x = fmaf(w, y.x, v.x);
        v.y = fmaf(w, y.y, v.y);
        v.z = fmaf(w, y.z, v.z);
        v.w = fmaf(w, y.w, v.w);
      }
    }
    if (4 * lane < p.dh) store_bf16x4(token_row(p, g, r) + 4 * lane, v, L > 0.f ? 1.f / L : 0.f);
  }
}

template <int D>
__device__ __forceinline__ bool token_phase(const ChunkParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap,
                                            uint8_t* mem, uint64_t* bars, volatile int* abort, float* sm_m, float* sm_l,
                                            int* sm_prev, int sw, int lane) {
  using T = TokenShape<D>;
  if (p.tensor) {
    const Mix mix = mix_of(p, lane);
    if (!mix.few || mix.fold) return true;
  }
  Runs<TOKEN> runs;
  runs.scan(p, lane, false, false);
  runs.split(gridDim.x);
  runs.begin(p, lane, blockIdx.x);
  const TokenWarp tw{sw, lane, sm100::l2_policy_evict_first()};
  uint8_t* ring = mem + sw * T::STAGES * T::STAGE;
  bars += sw * T::STAGES;
  float* buf = reinterpret_cast<float*>(mem + T::JOIN);
  int slot = 0;
  uint32_t phases = 0;                         // of the stages' barriers, a bit each
  bool ok = true;
  TokenBlocks blocks{0, 0};
  // a segment's first steps into the ring, from `slot` on
  auto request = [&](const Segment& g) {
    blocks.base = -32;
    if (!ok) return;
    for (int u = 0; u < min(T::STAGES, g.nt); ++u) {
      const int s = (slot + u) % T::STAGES;
      token_load<D>(p, kmap, vmap, g, ring + s * T::STAGE, &bars[s], blocks, tw, u);
    }
  };
  Segment g = runs.next(p, lane);
  // the segment after this one, on its way while this one is joined
  auto advance = [&]() {
    const Segment next = runs.next(p, lane);
    if (!next.last) request(next);
    return next;
  };
  if (!g.last) request(g);
  // (After a wait that gave up a warp still goes through its segments, waiting and requesting no more: the joins'
  // barriers count on all of them.)
  // A split item's arrival is one atomic, which takes microseconds on a busy memory: its answer is looked at a segment
  // later.
  Segment waiting{};
  bool waits = false;
  int arrived = 0;
  auto settle = [&]() {
    if (!waits) return;
    if (sw == 0 && lane == 0) {
      *sm_prev = arrived;
      if (arrived == waiting.n_parts - 1) p.tk_cnt[waiting.first_run] = 0;
    }
    all_soft();
    if (*sm_prev == waiting.n_parts - 1) token_merge<D>(p, waiting, tw);   // the last of the item's CTAs
    waits = false;
  };
  while (!g.last) {
    Segment next;
    if (g.tokens * p.G <= 8) {
      float o[1][D / 16][4], m[1][2], l[1][2];
      token_segment<D, 1>(p, kmap, vmap, g, ring, bars, phases, slot, abort, ok, blocks, tw, o, m, l);
      next = advance();
      settle();
      token_join<D, 1>(p, g, buf, sm_m, sm_l, tw, o, m, l);
    } else {
      float o[2][D / 16][4], m[2][2], l[2][2];
      token_segment<D, 2>(p, kmap, vmap, g, ring, bars, phases, slot, abort, ok, blocks, tw, o, m, l);
      next = advance();
      settle();
      token_join<D, 2>(p, g, buf, sm_m, sm_l, tw, o, m, l);
    }
    if (!g.whole) {
      all_soft();                            // the partial comes before its arrival
      if (sw == 0 && lane == 0) arrived = arrive_acq_rel(&p.tk_cnt[g.first_run]);
      waiting = g;
      waits = true;
    }
    g = next;
  }
  settle();
  if (!ok) {
    // no copy may still be landing when the CTA leaves
    volatile int never = 0;
    for (int s = 0; s < T::STAGES; ++s) sm100::mbar_wait(&bars[s], (phases >> s) & 1u, &never);
  }
  return ok;
}

// ---- the kernel ------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(CH_THREADS, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ CUtensorMap tkmap, const __grid_constant__ CUtensorMap tvmap) {
  using S = Shape<D>;
  constexpr int SLOTS = S::SLOTS;
  constexpr int PART = 2 * CH_ROWS * (D + 2);            // floats of a partial
  const LaunchStamp ls(p.stamp);
  // no static shared memory: the tiles start at the CTA's window, 1024-byte aligned (checked)
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* ring = sm + 2 * S::TILE;
  Shared<SLOTS>& sh = *reinterpret_cast<Shared<SLOTS>*>(sm + S::TILES);
  if (sm100::smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, EAGLE_ERR_UNSUPPORTED);
    return;
  }

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sh.abort;
  volatile int* never = &sh.never;
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      sm100::mbar_init(&sh.full[i], 1);
      sm100::mbar_init(&sh.raw[i], 1);
      sm100::mbar_init(&sh.empty[i], 2);          // each group: its softmax warps, or its MMA thread
    }
    for (int i = 0; i < CH_SEGS; ++i) {
      sm100::mbar_init(&sh.seg_full[i], 1);
      sm100::mbar_init(&sh.seg_empty[i], 3 + CH_SOFT_WARPS);   // loader, MMA threads, softmax warps
    }
    sm100::mbar_init(&sh.tm_ready, 1);
    sm100::mbar_init(&sh.q_full, 1);
    sm100::mbar_init(&sh.q_empty, 2);
    for (int i = 0; i < 4; ++i) {
      sm100::mbar_init(&sh.s_full[i >> 1][i & 1], 1);
      sm100::mbar_init(&sh.p_full[i >> 1][i & 1], 4);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&sh.o_half[i], 1);
      sm100::mbar_init(&sh.o_full[i], 1);
    }
    sm100::mbar_init(&sh.join, CH_SOFT_WARPS);
    sm100::mbar_init(&sh.tk_done, CH_SOFT_WARPS);
    for (int i = 0; i < CH_SOFT_WARPS * TK_STAGES<SLOTS>; ++i) sm100::mbar_init(&sh.tk_full[i], 1);
    sm100::mbar_init(&sh.done, 2);
    sh.abort = 0;
    sh.never = 0;
    sm100::fence_barrier_init();
  }
  if (warp == CH_LOAD_WARP && lane < (p.tensor ? 5 : 2))
    sm100::tma_prefetch_desc(lane == 0 ? &tkmap : lane == 1 ? &tvmap : lane == 2 ? &qmap : lane == 3 ? &kmap : &vmap);
  __syncthreads();
  pdl_wait();
  ls.waited();
  if (!p.tensor) {
    pdl_trigger();                             // every request has few rows: the token phase is all
  } else if (warp == CH_MMA_WARP) {
    // tensor memory only after the wait (every kernel this one waits for has finished), and dependents start only once
    // every CTA holds its columns; the token phase runs meanwhile
    sm100::tmem_alloc(&sh.tmem, CH_TM_COLS);
    sm100::tmem_relinquish();
    sm100::tc_fence_before();
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&sh.tm_ready);
    pdl_trigger();
  }
  __syncwarp();
  const uint32_t sbase = sm100::smem_u32(sm);
  const uint32_t rbase = sbase + 2 * S::TILE;
  // K and V tiles: bytes from 8 rows to the next 8, and from elements 0 - 63 to 64 - 127
  const uint32_t kv_rows = p.grouped ? 1024u * S::HALVES : 1024u, kv_half = p.grouped ? 1024u : CH_HALF;

  auto give_up = [&]() {
    set_status(p.status, EAGLE_ERR_TIMEOUT);
    sh.abort = 1;
  };
  // every lane waits; the answer is the warp's
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    return static_cast<bool>(__all_sync(0xffffffffu, sm100::mbar_wait(bar, parity, abort_flag)));
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CH_REGS_FEW));
    if (!p.tensor) {
      if (warp == CH_SCHED_WARP && blockIdx.x == 0) {
        Runs<TENSOR> runs;
        runs.scan(p, lane, false, true);       // reports what is wrong with the batch
      }
      return;
    }
    if (warp == CH_SCHED_WARP) {
      // ---- scheduler ----
      Runs<TENSOR> runs;
      runs.scan(p, lane, mix_of(p, lane).fold, blockIdx.x == 0);
      runs.split(gridDim.x);
      runs.begin(p, lane, blockIdx.x);
      bool ok = true;
      int e = 0;                               // ring elements of the segments that are through `finish`
      uint32_t raw = 0;                        // phases of sh.raw, a bit each
      // A segment's last V tile, where it ends past the length: rows there may hold anything, and 0 x NaN is NaN, so
      // they become zeros.  (By the loader, which then waited for the tile, the next segment's loads came 3 to 5
      // thousand cycles later.)
      auto finish = [&](int slot) {
        const int nt = sh.seg[slot].nt, first = sh.seg[slot].len - (sh.seg[slot].kt0 + nt - 1) * CH_KEYS;
        e += 2 * nt;
        if (nt == 0 || first >= CH_KEYS) return true;
        const int s = (e - 1) % SLOTS;
        if (!warp_wait(&sh.raw[s], (raw >> s) & 1u)) return false;
        raw ^= 1u << s;
        uint8_t* v = ring + s * S::TILE;
        const int per = (CH_KEYS - first) * 8;
        for (int x = lane; x < per * S::HALVES; x += 32) {
          const int h = x >= per ? 1 : 0, y = x - h * per, r = first + (y >> 3);
          *reinterpret_cast<uint4*>(v + h * kv_half + (r >> 3) * kv_rows + (r & 7) * 128 + (y & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        sm100::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sh.full[s]);
        return true;
      };
      int i = 0;
      for (bool more = true; ok && more; ++i) {
        const int slot = i % CH_SEGS;
        if (i >= CH_SEGS) {
          ok = warp_wait(&sh.seg_empty[slot], static_cast<uint32_t>((i / CH_SEGS - 1) & 1)) && finish(slot);
          if (!ok) break;
        }
        const Segment g = runs.next(p, lane);
        if (lane == 0) {
          sh.seg[slot] = g;
          sm100::mbar_arrive(&sh.seg_full[slot]);
        }
        __syncwarp();
        more = !g.last;
      }
      for (int j = max(0, i - CH_SEGS); ok && j < i - 1; ++j) ok = finish(j % CH_SEGS);   // (the last one has no tiles)
      if (!ok && lane == 0) give_up();
    } else if (warp == CH_LOAD_WARP) {
      // ---- loader ----
      const bool paged = p.paged.table != nullptr;
      const int boxes = CH_KEYS / p.box;
      int e = 0;                               // ring elements so far: K and V tiles alternate
      int segs = 0;                            // segments with tiles so far
      bool ok = warp_wait(&sh.tk_done, 0u);    // the token phase has used the tiles' memory
      for (int i = 0; ok; ++i) {
        const int slot = i % CH_SEGS;
        ok = warp_wait(&sh.seg_full[slot], static_cast<uint32_t>((i / CH_SEGS) & 1));
        if (!ok) break;
        const Segment g = sh.seg[slot];
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sh.seg_empty[slot]);
        if (g.last) break;
        if (g.nt == 0) continue;
        const int32_t* table = paged ? p.paged.table + static_cast<size_t>(g.b) * p.paged.per_req : nullptr;
        // the table's entry for box j of key tile t, and the block it stands for: out of range (read as zeros) where
        // nothing is to be read
        auto pos_of = [&](int t, int j) { return (g.kt0 + t) * CH_KEYS + j * p.box; };
        auto entry_at = [&](int t, int j) { return pos_of(t, j) < g.len ? table[pos_of(t, j) >> p.paged.shift] : 0; };
        auto block_of = [&](int t, int j, int x) {
          if (pos_of(t, j) >= g.len) return p.paged.n_blocks;
          if (x >= 0 && x < p.paged.n_blocks) return x;
          set_status(p.status, EAGLE_ERR_INVALID_ARG);
          return p.paged.n_blocks;
        };
        // box `lane` of the tile at hand, and the next tile's entry: looked at a tile later, when it has arrived
        int blk = paged && lane < boxes ? block_of(0, lane, entry_at(0, lane)) : 0, ahead = 0;
        auto load = [&](int t, int m) {
          const int s = e % SLOTS;
          if (e >= SLOTS && !warp_wait(&sh.empty[s], static_cast<uint32_t>((e / SLOTS - 1) & 1))) return false;
          uint8_t* dst = ring + s * S::TILE;
          const int k0 = (g.kt0 + t) * CH_KEYS;
          const CUtensorMap* map = m == 0 ? &kmap : &vmap;
          const bool zero = m == 1 && k0 + CH_KEYS > g.len;   // (the scheduler's)
          uint64_t* bar = zero ? &sh.raw[s] : &sh.full[s];
          if (lane == 0) sm100::mbar_arrive_expect_tx(bar, S::TILE);
          __syncwarp();
          for (int j = lane; j < boxes; j += 32) {
            const int z = !paged ? g.b : j < 32 ? blk : block_of(t, j, entry_at(t, j));
            const int y = !paged ? k0 : (k0 + j * p.box) & ((1 << p.paged.shift) - 1);
            if (p.grouped) {
              sm100::tma_load_4d(dst + j * p.box * 128 * S::HALVES, map, 0, 0, g.hk * S::HALVES,
                                 (z << (p.paged.shift - 3)) + (y >> 3), bar);
              continue;
            }
#pragma unroll
            for (int h = 0; h < S::HALVES; ++h)
              sm100::tma_load_4d(dst + h * CH_HALF + j * p.box * 128, map, 64 * h, g.hk, y, z, bar);
          }
          ++e;
          return true;
        };
        auto load_q = [&]() {
          if (segs > 0 && !warp_wait(&sh.q_empty, static_cast<uint32_t>((segs - 1) & 1))) return false;
          ++segs;
          if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(p.GB * p.T) * 128u * S::HALVES;
            const int tiles = g.two ? 2 : 1;
            sm100::mbar_arrive_expect_tx(&sh.q_full, bytes * tiles);
            for (int w = 0; w < tiles; ++w)
              for (int h = 0; h < S::HALVES; ++h)
                sm100::tma_load_3d(sm + w * S::TILE + h * CH_HALF, &qmap, 64 * h, g.head0, g.row0 + w * p.T,
                                   &sh.q_full);
          }
          __syncwarp();
          return true;
        };
        // the first K and V while the item before still uses its Q; the CTA's first Q at once
        const bool first = segs == 0;
        if (first) ok = load_q();
        for (int t = 0; ok && t < g.nt; ++t) {
          const bool more = paged && t + 1 < g.nt && lane < boxes;
          if (more) ahead = entry_at(t + 1, lane);
          ok = load(t, 0) && load(t, 1) && (t > 0 || first || load_q());
          if (more) blk = block_of(t + 1, lane, ahead);
        }
      }
      if (!ok && lane == 0) give_up();
      // no TMA copy may still be landing when the CTA leaves
      for (int u = max(0, e - SLOTS); u < e; ++u)
        sm100::mbar_wait(&sh.full[u % SLOTS], static_cast<uint32_t>((u / SLOTS) & 1), never);
      if (segs > 0) sm100::mbar_wait(&sh.q_full, static_cast<uint32_t>((segs - 1) & 1), never);
    } else {
      // ---- MMA issuers: warp 1 for group 0, warp 3 for group 1 ----
      const int w = warp >> 1;
      if (lane == 0) {
        constexpr uint32_t HI = sm100::DESC_SW128_HI;
        const uint32_t kv_hi = (HI & ~0x3FFFu) | (kv_rows >> 4);
        const uint32_t id_s = sm100::idesc_bf16_f32(CH_ROWS, CH_STEP);
        const uint32_t id_o = sm100::idesc_bf16_f32(CH_ROWS, D) | (1u << 16);     // B (V) MN-major
        bool ok = sm100::mbar_wait(&sh.tm_ready, 0u, abort_flag);
        sm100::tc_fence_after();
        const uint32_t tmem = sh.tmem, s_tm = tmem + CH_TM_S + 128u * w, o_tm = tmem + CH_TM_O + 128u * w;
        int e0 = 0, segs = 0;
        uint32_t p_phase = 0;
        for (int i = 0; ok; ++i) {
          const int slot = i % CH_SEGS;
          ok = sm100::mbar_wait(&sh.seg_full[slot], static_cast<uint32_t>((i / CH_SEGS) & 1), abort_flag);
          if (!ok) break;
          const int nt = sh.seg[slot].nt, last = sh.seg[slot].last;
          const bool two = sh.seg[slot].two;
          sm100::mbar_arrive(&sh.seg_empty[slot]);
          if (last) break;
          if (nt == 0) continue;
          const int t0 = two ? 0 : w;
          // Every segment's queries are waited for, and given free in a segment without tiles for this group (else by
          // its softmax warps), only then: the barriers' phases stay in step with both groups.
          ok = sm100::mbar_wait(&sh.q_full, static_cast<uint32_t>(segs & 1), abort_flag);
          ++segs;
          if (ok && t0 >= nt) sm100::mbar_arrive(&sh.q_empty);
          const uint32_t qlo = sm100::desc_lo(sbase + (two ? w * S::TILE : 0u), 16);
          auto landed = [&](int x) {
            return sm100::mbar_wait(&sh.full[x % SLOTS], static_cast<uint32_t>((x / SLOTS) & 1), abort_flag);
          };
          // S_w of half h of the key tile in ring element x
          auto issue_s = [&](int x, int h) {
            sm100::tc_fence_after();
            const uint32_t klo = sm100::desc_lo(rbase + (x % SLOTS) * S::TILE + h * (CH_STEP / 8) * kv_rows, 16);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t q_off = ((k >> 2) * CH_HALF + (k & 3) * 32) >> 4;
              const uint32_t k_off = ((k >> 2) * kv_half + (k & 3) * 32) >> 4;
              sm100::mma_ss32(s_tm + 64u * h, qlo + q_off, HI, klo + k_off, kv_hi, id_s, k > 0 ? 1u : 0u);
            }
          };
          // O_w += P_w V of the same half of the tile's V
          auto issue_o = [&](int x, int h, uint32_t more) {
            sm100::tc_fence_after();
            const uint32_t vlo = sm100::desc_lo(rbase + (x % SLOTS) * S::TILE + h * (CH_STEP / 8) * kv_rows, kv_half);
#pragma unroll
            for (int k = 0; k < CH_STEP / 16; ++k)
              sm100::mma_ts32(o_tm, s_tm + 64u * h + 8u * k, vlo + ((k * 2 * kv_rows) >> 4), kv_hi, id_o,
                              k > 0 ? 1u : more);
          };
          // a tile of the other group alone: this one is through with it once it is there.  (So every slot's phases
          // pass both MMA threads in turn, and no wait can take one for the one two before.)
          auto pass = [&](int t) {
            for (int x = e0 + 2 * t; ok && x < e0 + 2 * t + 2; ++x) {
              ok = landed(x);
              if (ok) sm100::mbar_arrive(&sh.empty[x % SLOTS]);
            }
          };
          // Tiles t0, t0 + STEP, .. of the segment.  (The loop of the two-tile case has nothing in it but waits and
          // products: tests for the other case in it took 311 to 345 us.)
          auto run = [&](auto both) {
            constexpr bool BOTH = decltype(both)::value;
            constexpr int STEP = BOTH ? 1 : 2;
            if (!BOTH && t0 == 1) pass(0);
            if (!ok || t0 >= nt || !(ok = landed(e0 + 2 * t0))) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              issue_s(e0 + 2 * t0, h);
              sm100::mma_commit(&sh.s_full[w][h]);
            }
            int t = t0;
            for (; t + STEP < nt; t += STEP) {
              const int kx = e0 + 2 * (t + STEP), vx = e0 + 2 * t + 1;    // the next tile's K, this one's V
              ok = landed(vx);
              if (!BOTH) pass(t + 1);
              ok = ok && landed(kx);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                ok = ok && sm100::mbar_wait(&sh.p_full[w][h], p_phase & 1, abort_flag);
                if (!ok) return;
                issue_o(vx, h, h == 1 || t > t0 ? 1u : 0u);
                issue_s(kx, h);
                sm100::mma_commit(&sh.s_full[w][h]);
              }
              ++p_phase;
            }
            // the last tile: the signs that O_w has taken its halves
            ok = landed(e0 + 2 * t + 1);
            if (!BOTH && t + 1 < nt) pass(t + 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = ok && sm100::mbar_wait(&sh.p_full[w][h], p_phase & 1, abort_flag);
              if (!ok) return;
              issue_o(e0 + 2 * t + 1, h, h == 1 || t > t0 ? 1u : 0u);
              sm100::mma_commit(h == 0 ? &sh.o_half[w] : &sh.o_full[w]);
            }
            ++p_phase;
          };
          if (two) run(std::true_type{});
          else run(std::false_type{});
          e0 += 2 * nt;
        }
        if (!ok) give_up();
        // every MMA issued here has completed before the tensor memory goes
        sm100::mma_commit(&sh.done);
        sm100::mbar_wait(&sh.done, 0u, never);
      }
      __syncwarp();
    }
  } else {
    // ---- softmax ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(CH_REGS_SOFT));
    bool tk_ok;
    {
      tk_ok = token_phase<D>(p, &tkmap, &tvmap, sm, sh.tk_full, abort_flag, sh.m[0], sh.l[0], &sh.tk_prev,
                             warp - CH_SOFT_WARP0, lane);
      if (!p.tensor) {
        if (!tk_ok && lane == 0) set_status(p.status, EAGLE_ERR_TIMEOUT);
        return;
      }
      sm100::fence_proxy_async_smem();         // the ring's next writer is TMA
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&sh.tk_done);
    }
    const int w = (warp - CH_SOFT_WARP0) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int st = tid - 32 * CH_SOFT_WARP0;               // 0 .. 255
    const int tok = row / p.GB, head = row - tok * p.GB;   // of this row in its tile
    uint32_t s_phase = 0, o_phase = 0, j_phase = 0;
    int e0 = 0;                                            // ring element of the segment's first K
    const bool frees = quarter == 0 && lane == 0;          // tells the loader what the group's products have read
    bool ok = warp_wait(&sh.tm_ready, 0u) && warp_wait(&sh.tk_done, 0u) && tk_ok;   // (the token phase used m and l)
    sm100::tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t s_addr = tmem + CH_TM_S + 128u * w + lane_base, o_addr = tmem + CH_TM_O + 128u * w + lane_base;
    // all softmax warps: shared memory and tensor memory of the others' last step may be used after it
    auto join = [&]() {
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&sh.join);
      const bool r = warp_wait(&sh.join, j_phase & 1);
      ++j_phase;
      return r;
    };
    for (int i = 0; ok; ++i) {
      const int slot = i % CH_SEGS;
      ok = warp_wait(&sh.seg_full[slot], static_cast<uint32_t>((i / CH_SEGS) & 1));
      if (!ok) break;
      const Segment g = sh.seg[slot];
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&sh.seg_empty[slot]);
      if (g.last) break;
      const bool two = g.two;
      const int t_item = (two ? w * p.T : 0) + tok;        // the row's token in the item
      const bool valid = tok < p.T && t_item < g.tokens && head < g.heads;
      const int pos = g.pos0 + t_item;
      const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      // bounds of the warp's rows, so that a tile they all see whole is not masked
      const int pos_least = __reduce_min_sync(0xffffffffu, valid ? pos : INT_MAX);
      const int lo_most = __reduce_max_sync(0xffffffffu, valid ? lo : INT_MIN);
      const int pos_most = __reduce_max_sync(0xffffffffu, valid ? pos : INT_MIN);
      const int lo_least = __reduce_min_sync(0xffffffffu, valid ? lo : INT_MAX);
      const bool some = __any_sync(0xffffffffu, valid);
      float m_ref = -INFINITY, l_sum = 0.f;
      const int step = two ? 1 : 2, t0 = two ? 0 : w;
      auto release = [&](int x) { sm100::mbar_arrive_if(&sh.empty[x % SLOTS], frees); };   // ring element x is read
      for (int t = t0; ok && t < g.nt; t += step) {
        for (int h = 0; ok && h < 2; ++h) {
          ok = warp_wait(&sh.s_full[w][h], s_phase & 1);
          if (!ok) break;
          if (h == 1) {                        // the tile's scores are complete, and so is what was issued before them
            if (t > t0) release(e0 + 2 * (t - step) + 1);
            release(e0 + 2 * t);
            if (t + step >= g.nt) sm100::mbar_arrive_if(&sh.q_empty, frees);
          }
          sm100::tc_fence_after();
          if (some) {
            const int k0 = (g.kt0 + t) * CH_KEYS + CH_STEP * h;
            if (k0 > pos_most || k0 + CH_STEP <= lo_least) {
              // none of the warp's rows sees a key of the step
              uint32_t zero[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) zero[j] = 0u;
              sm100::tmem_st16(s_addr + 64u * h, zero);
              sm100::tmem_st16(s_addr + 64u * h + 16u, zero);
              sm100::tmem_wait_st();
              sm100::tc_fence_before();
              __syncwarp();
              sm100::mbar_arrive_if(&sh.p_full[w][h], lane == 0);
              continue;
            }
            const bool masked = k0 + CH_STEP - 1 > pos_least || k0 < lo_most;
            // The products before this step are complete when the other half's next scores are, issued after them (in
            // the last step: the sign in their place); before the first step there are none.
            auto at_rest = [&]() {
              if (h == 1 && t + step >= g.nt) return warp_wait(&sh.o_half[w], o_phase & 1);
              return warp_wait(&sh.s_full[w][h ^ 1], (h ? s_phase + 1 : s_phase) & 1);
            };
            ok = softmax_step<D>(s_addr + 64u * h, o_addr, masked, lo - k0, pos - k0, valid, p.c, m_ref, l_sum,
                                 &sh.p_full[w][h], at_rest);
          } else if (lane == 0) {
            sm100::mbar_arrive(&sh.p_full[w][h]);
          }
        }
        ++s_phase;
      }
      if (ok && t0 < g.nt) {
        ok = warp_wait(&sh.o_full[w], o_phase & 1);        // O_w has taken the last tile
        ++o_phase;
        if (ok) release(e0 + 2 * (t0 + (g.nt - 1 - t0) / step * step) + 1);
      }
      if (!ok) break;
      e0 += 2 * g.nt;
      sm100::tc_fence_after();
      // The item's rows are 0 .. 255 (two tiles) or 0 .. 127; this thread holds D columns of its own row, or (one
      // tile, whose key tiles both groups shared) half the columns of the join of O_0 and O_1.
      const int r_item = two ? w * CH_ROWS + row : row;
      float a[2] = {1.f, 0.f};
      float m_row = m_ref, l_row = l_sum;
      if (!two) {
        sh.m[w][row] = m_ref;
        sh.l[w][row] = l_sum;
        ok = join();
        if (!ok) break;
        sm100::tc_fence_after();               // the other group saw its products complete; its O is read here too
        const float m0 = sh.m[0][row], m1 = sh.m[1][row];
        m_row = fmaxf(m0, m1);
        a[0] = m0 == -INFINITY ? 0.f : sm100::exp2(m0 - m_row);
        a[1] = m1 == -INFINITY ? 0.f : sm100::exp2(m1 - m_row);
        l_row = a[0] * sh.l[0][row] + a[1] * sh.l[1][row];
      }
      const int col0 = two ? 0 : w * (D / 2), cols = two ? D : D / 2;
      const float inv = g.whole ? (l_row > 0.f ? 1.f / l_row : 0.f) : 1.f;
      float* part = p.part + static_cast<size_t>(g.part) * PART;
      if (some) {
        for (int cc = col0; cc < col0 + cols; cc += 32) {
          float o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0.f;
          if (g.nt > 0) {
            if (two) {
              sm100::tmem_ld32(o_addr + cc, o);
              sm100::tmem_wait_ld();
            } else {
              // an O whose weight is 0 in every row may never have been written
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (__any_sync(0xffffffffu, a[k] != 0.f)) {
                  float v[32];
                  sm100::tmem_ld32(tmem + CH_TM_O + 128u * k + lane_base + cc, v);
                  sm100::tmem_wait_ld();
                  if (a[k] != 0.f) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = fmaf(a[k], v[j], o[j]);
                  }
                  __syncwarp();
                }
            }
          }
          if (valid) {
            if (l_row == 0.f) {                // no key seen: whatever the tile's products left
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = 0.f;
            }
            if (g.whole) {
              uint16_t* dst = p.out + (static_cast<size_t>(g.row0) + t_item) * p.ld_o + (g.head0 + head) * p.dh + cc;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                if (cc + 16 * q < p.dh) {
                  uint32_t x[8];
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(o[16 * q + 2 * j] * inv, o[16 * q + 2 * j + 1] * inv);
                    x[j] = *reinterpret_cast<const uint32_t*>(&h);
                  }
                  store16(p, dst + 16 * q, x);
                }
              }
            } else {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                reinterpret_cast<float4*>(part)[(cc / 4 + q) * (2 * CH_ROWS) + r_item] =
                    make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
          }
          __syncwarp();                        // the next columns' load is the whole warp's
        }
      }
      if (!g.whole && valid && (two || w == 0)) {
        part[2 * CH_ROWS * D + r_item] = m_row;
        part[2 * CH_ROWS * D + 2 * CH_ROWS + r_item] = l_row;
      }
      sm100::tc_fence_before();
      if (g.whole) {
        // one tile: O_0 and O_1 were read by both groups, the next item's products may not overwrite them before
        if (!two) ok = join();
        continue;
      }
      ok = join();                             // every thread's partials come first
      if (!ok) break;
      if (st == 0) {
        sh.prev = arrive_acq_rel(&p.cnt[g.first_run]);
        if (sh.prev == g.n_parts - 1) p.cnt[g.first_run] = 0;
      }
      ok = join();
      if (!ok) break;
      if (sh.prev == g.n_parts - 1) {
        merge_parts<D>(p, g, st);              // the last of the item's CTAs
      }
    }
    if (!ok && lane == 0) give_up();
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == CH_MMA_WARP) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(sh.tmem, CH_TM_COLS);
  }
}

bool encode(eagle_ctx* ctx, CUtensorMap* map, const void* ptr, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return ctx->encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(ptr), dims,
                     strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_shape(eagle_ctx* ctx, const ChunkParams& p, const CUtensorMap& qm, const CUtensorMap& km,
                         const CUtensorMap& vm, const CUtensorMap& tkm, const CUtensorMap& tvm, cudaStream_t st) {
  const cudaError_t e =
      smem_limit_once(reinterpret_cast<const void*>(chunk_attn_kernel<D>), static_cast<int>(chunk_smem<D>()));
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_attn_kernel<D>, dim3(ctx->sm_count), dim3(CH_THREADS), chunk_smem<D>(), st, p, qm, km, vm,
                    tkm, tvm);
}

}  // namespace

static size_t part_floats(int sm_count, int head_dim) {
  return static_cast<size_t>(2) * sm_count * 2 * CH_ROWS * ((head_dim > 64 ? 128 : 64) + 2);
}
size_t chunk_part_bytes(int sm_count, int head_dim) {
  return (part_floats(sm_count, head_dim) +
          static_cast<size_t>(2) * sm_count * TK_ROWS * ((head_dim > 64 ? 128 : 64) + 2)) * sizeof(float);
}
int chunk_counters(int sm_count) { return 2 * sm_count; }

cudaError_t launch_chunk_attn(eagle_ctx* ctx, int batch, const eagle_rows* rows, const uint16_t* q, int ld_q,
                              const eagle_kv* kv, int window, float scale, uint16_t* out, int ld_out, void* ws,
                              cudaStream_t st) {
  const eagle_dims& D = ctx->dims;
  ChunkParams p{};
  p.rows = PackedRows{rows->row_start, rows->n_rows, batch};
  p.hkv = D.n_kv_heads;
  p.dh = D.head_dim;
  p.G = D.n_q_heads / D.n_kv_heads;
  p.GB = std::min(p.G, CH_ROWS);
  p.T = CH_ROWS / p.GB;
  p.nsub = ceil_div(p.G, p.GB);
  p.out = out;
  p.ld_o = ld_out;
  p.out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && ld_out % 16 == 0;
  p.cap = kv->cap;
  p.window = window >= kv->cap ? 0 : window;   // a window of the whole cache is none
  p.len = kv->len;
  p.q = q;
  p.ld_q = ld_q;
  p.k = kv->k;
  p.v = kv->v;
  p.paged = paged_of(&kv->paging, kv->cap);
  const bool paged = p.paged.table != nullptr;
  const int bs = paged ? kv->paging.block_size : kv->cap;
  p.box = paged ? std::min(bs, CH_KEYS) : CH_KEYS;
  p.c = scale * 1.4426950408889634f;
  p.part = ws_ptr<float>(ws, ctx->ws.attn_part);
  p.cnt = ws_ptr<int>(ws, ctx->ws.chunk_cnt);
  p.tk_part = p.part + part_floats(ctx->sm_count, D.head_dim);
  p.tk_cnt = p.cnt + ctx->sm_count;
  p.status = ws_ptr<int>(ws, ctx->ws.status);
  // q as {element, head, row}; a K or V pool as {element, kv head, row of a block, block} (contiguous: row, request)
  const cuuint64_t e2 = 2, dh = static_cast<cuuint64_t>(p.dh);
  const cuuint64_t qd[3] = {dh, static_cast<cuuint64_t>(D.n_q_heads), static_cast<cuuint64_t>(rows->n_rows)};
  const cuuint64_t qs[2] = {dh * e2, static_cast<cuuint64_t>(ld_q) * e2};
  const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(p.GB), static_cast<cuuint32_t>(p.T)};
  const cuuint64_t kd[4] = {dh, static_cast<cuuint64_t>(p.hkv), static_cast<cuuint64_t>(bs),
                            static_cast<cuuint64_t>(paged ? kv->paging.n_blocks : batch)};
  const cuuint64_t row = dh * p.hkv * e2;
  const cuuint64_t ks[3] = {dh * e2, row, row * bs};
  const cuuint32_t kb[4] = {64, 1, static_cast<cuuint32_t>(p.box), 1};
  // Heads of 128 in blocks of 8 rows or more: a box brings both halves of its rows, 8 rows at a time, from the pool as
  // {64 elements, 8 rows, half of a kv head, 8-row group}.  One copy a block where two took 95 cycles each to issue,
  // which kept the loader behind (40 heads, 512 rows after 4096, blocks of 16: 68 -> 62 us; of 64: 61 either way).
  p.grouped = paged && bs >= 8 && p.dh == 128;
  const cuuint64_t gd[4] = {64, 8, 2 * static_cast<cuuint64_t>(p.hkv), kd[3] * (bs / 8)};
  const cuuint64_t gs[3] = {row, 128, 8 * row};
  const cuuint32_t gb[4] = {64, 8, 2, static_cast<cuuint32_t>(p.box / 8)};
  const cuuint32_t tb[4] = {64, 1, static_cast<cuuint32_t>(std::min(p.box, 16)), 1};   // the token phase's steps
  CUtensorMap qm, km, vm, tkm, tvm;
  p.tensor = static_cast<long long>(rows->n_rows) * p.G > TK_ROWS;
  std::memset(&qm, 0, sizeof(qm));
  std::memset(&km, 0, sizeof(km));
  std::memset(&vm, 0, sizeof(vm));
  if ((p.tensor && (!encode(ctx, &qm, q, 3, qd, qs, qb) ||
                    !encode(ctx, &km, kv->k, 4, p.grouped ? gd : kd, p.grouped ? gs : ks, p.grouped ? gb : kb) ||
                    !encode(ctx, &vm, kv->v, 4, p.grouped ? gd : kd, p.grouped ? gs : ks, p.grouped ? gb : kb))) ||
      !encode(ctx, &tkm, kv->k, 4, kd, ks, tb) ||
      !encode(ctx, &tvm, kv->v, 4, kd, ks, tb))
    return cudaErrorInvalidValue;
  p.stamp = stamp_slot(ctx, EAGLE_K_CHUNK_ATTN);
  trace_before(ctx, EAGLE_K_CHUNK_ATTN, st);
  const cudaError_t e = p.dh > 64 ? launch_shape<128>(ctx, p, qm, km, vm, tkm, tvm, st)
                                    : launch_shape<64>(ctx, p, qm, km, vm, tkm, tvm, st);
  ctx->launches++;
  note_ordered(ctx, st);
  trace_after(ctx, EAGLE_K_CHUNK_ATTN, st);
  return e;
}

}  // namespace eagle
