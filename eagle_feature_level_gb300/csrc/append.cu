// eagle_kv_append: rotary positions of a batch's new rows and their append to
// a (paged) KV cache.
//
// Pair j of a head turns by position * f_j.  With f_j as a 64-bit fraction of
// a turn the product mod 2^64 is the angle's exact fraction, one integer
// multiplication; its top 32 bits as a signed number of turns in [-1/2, 1/2)
// go to sincospif, whose error (2^-24 or so) is then all of the angle's.
//
// The work is a pass over the rows: each element read once, written once.  A
// CTA takes a few rows: one warp per row finds its request and cache row, the
// threads compute the rows' sines and cosines once into shared memory (every
// head of a row shares them), then a thread keeps one place of 16 elements in
// a head (8 pairs: two 16-byte loads of bf16) and goes over the row's heads,
// the sines and cosines of its place in registers and three heads' loads in
// flight.
//
// Bound: memory.  10.4 thousand rows of 64 query and 8 kv heads: 76 us for 429
// MB, 5.6 TB/s, 0.83 of a measured copy; with the sines and cosines read from
// shared memory for every head 83 us.  More rows a CTA (16, 32) and streaming
// hints changed nothing.  A few rows (8 of 40 heads) are latency: 4.6 us.  Each
// row's warp looks at the table's entries of all its request's new rows, which
// long prompts into very small blocks feel: 16384 rows of 8/2 heads of 64 take
// 46 us in blocks of 16 rows, 75 in blocks of one.
#include <algorithm>

#include "internal.h"
#include "common.cuh"
#include "rows.cuh"

namespace eagle {
namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_WARPS = AP_THREADS / 32;
constexpr int AP_ROWS = AP_WARPS;           // rows of a CTA at most
constexpr int AP_UNITS = 3;                  // units of a thread in flight

struct AppendParams {
  PackedRows rows;
  int tile;                // rows a CTA takes
  int row_ctas;            // CTAs for rows; the rest set len_out, a warp per request
  int hq, hkv, dh;
  int rot, interleaved;
  float mscale;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  long long ld_q, ld_qo, ld_k, ld_v;
  uint16_t* kc;
  uint16_t* vc;
  int cap;
  const int32_t* len;
  PagedKv paged;
  const int32_t* pos;
  int32_t* len_out;
  int* status;
  uint64_t* stamp;
  uint64_t turn[EAGLE_MAX_ROPE_PAIRS];
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = f32_to_bf16(x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// (cos, sin) * mscale of the pair at a position.
__device__ __forceinline__ float2 turn_of(uint64_t turn, int pos, float mscale) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turn;
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * mscale, s * mscale);
}

// Eight elements as they were loaded, turned in fp32 and rounded once when
// stored; what passes through bf16 to bf16 is moved as it is.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    w = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// A unit's eight pairs: (x_i, y_i) in the split layout, neighbours otherwise.
template <typename T>
__device__ __forceinline__ void unit_turn(Raw<T>& rx, Raw<T>& ry, const float2 (&cs)[8], int interleaved) {
  float x[8], y[8];
  rx.get(x);
  ry.get(y);
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x1 = x[i], x2 = y[i];
      x[i] = x1 * cs[i].x - x2 * cs[i].y;
      y[i] = x2 * cs[i].x + x1 * cs[i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x1 = x[2 * i], x2 = x[2 * i + 1], y1 = y[2 * i], y2 = y[2 * i + 1];
      x[2 * i] = x1 * cs[i].x - x2 * cs[i].y;
      x[2 * i + 1] = x2 * cs[i].x + x1 * cs[i].y;
      y[2 * i] = y1 * cs[4 + i].x - y2 * cs[4 + i].y;
      y[2 * i + 1] = y2 * cs[4 + i].x + y1 * cs[4 + i].y;
    }
  }
  rx.set(x);
  ry.set(y);
}

// One pair (u < rot / 2) or two elements that pass through: for a rot_dim
// that is no multiple of 16.
template <typename TI, typename TO>
__device__ __forceinline__ void unit2(const AppendParams& p, const float2* cs, const TI* in, TO* out, int u,
                                      bool turn) {
  const bool split = turn && !p.interleaved;
  const int a = split ? u : 2 * u, b = split ? p.rot / 2 + u : 2 * u + 1;
  float x = load1(in + a), y = load1(in + b);
  if (turn) {
    const float2 t = cs[u];
    const float x1 = x, x2 = y;
    x = x1 * t.x - x2 * t.y;
    y = x2 * t.x + x1 * t.y;
  }
  store1(out + a, x);
  store1(out + b, y);
}

// Rows r0 .. r0 + rows - 1, each at its place.  T: element type of the rows
// (uint16_t: bf16 bits, or float); WIDE: units of 16 elements (rot_dim a
// multiple of 16, so that a unit's 16-byte loads are aligned) or of 2 (4864
// rows of 64/8 heads: 41 us as 16, 117 as 2; fp32 rows of 16/4 heads of 64, 25
// and 24).
template <typename T, bool WIDE>
__device__ __forceinline__ void append_rows(const AppendParams& p, int r0, int rows, int hq,
                                            float2 (*s_cs)[EAGLE_MAX_ROPE_PAIRS], const long long* s_at,
                                            const int* s_pos, const int* s_any) {
  const int tid = threadIdx.x;
  const int pairs = p.rot / 2;
  for (int i = tid; i < rows * pairs; i += AP_THREADS) {
    const int r = i / pairs, j = i - r * pairs;
    s_cs[r][j] = turn_of(p.turn[j], s_pos[r], p.mscale);
  }
  __syncthreads();
  const int heads = hq + 2 * p.hkv;
  if (WIDE) {
    // A thread keeps one unit's place in a head, and a row's sines and cosines for it in registers, over the row's
    // heads (dh / 16 is a power of two), AP_UNITS of them in flight.
    const int upr = p.dh / 16, u = tid & (upr - 1), step = AP_THREADS / upr;
    const bool in_rot = 16 * u < p.rot;
    for (int r = 0; r < rows; ++r) {
      if (!s_any[r]) continue;
      float2 cs[8];
      if (in_rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = s_cs[r][8 * u + i];
      }
      const size_t row = static_cast<size_t>(r0) + r;
      const long long at = s_at[r];
      for (int h0 = tid / upr; h0 < heads; h0 += AP_UNITS * step) {
        Raw<T> x[AP_UNITS], y[AP_UNITS];
#pragma unroll
        for (int j = 0; j < AP_UNITS; ++j) {
          const int h = h0 + j * step;
          if (h >= heads || (h >= hq && at < 0)) continue;
          const bool is_v = h >= hq + p.hkv;
          const T* in = h < hq ? static_cast<const T*>(p.q) + row * p.ld_q + h * p.dh
                               : is_v ? static_cast<const T*>(p.v) + row * p.ld_v + (h - hq - p.hkv) * p.dh
                                      : static_cast<const T*>(p.k) + row * p.ld_k + (h - hq) * p.dh;
          const bool split = !is_v && in_rot && !p.interleaved;
          x[j].load(in + (split ? 8 * u : 16 * u));
          y[j].load(in + (split ? p.rot / 2 + 8 * u : 16 * u + 8));
        }
#pragma unroll
        for (int j = 0; j < AP_UNITS; ++j) {
          const int h = h0 + j * step;
          if (h >= heads || (h >= hq && at < 0)) continue;
          const bool is_v = h >= hq + p.hkv, turn = !is_v && in_rot;
          const bool split = turn && !p.interleaved;
          const int a = split ? 8 * u : 16 * u, b = split ? p.rot / 2 + 8 * u : 16 * u + 8;
          if (turn) unit_turn(x[j], y[j], cs, p.interleaved);
          if (h < hq) {
            T* out = static_cast<T*>(p.q_out) + row * p.ld_qo + h * p.dh;
            x[j].store(out + a);
            y[j].store(out + b);
          } else {
            uint16_t* out = is_v ? p.vc + (static_cast<size_t>(at) * p.hkv + (h - hq - p.hkv)) * p.dh
                                 : p.kc + (static_cast<size_t>(at) * p.hkv + (h - hq)) * p.dh;
            x[j].store(out + a);
            y[j].store(out + b);
          }
        }
      }
    }
    return;
  }
  const int upr = p.dh / 2, units = heads * upr;
  for (int r = 0; r < rows; ++r) {
    if (!s_any[r]) continue;
    const size_t row = static_cast<size_t>(r0) + r;
    const long long at = s_at[r];
    for (int i = tid; i < units; i += AP_THREADS) {
      const int h = i / upr, u = i - h * upr;
      if (h < hq) {
        unit2(p, s_cs[r], static_cast<const T*>(p.q) + row * p.ld_q + h * p.dh,
              static_cast<T*>(p.q_out) + row * p.ld_qo + h * p.dh, u, 2 * u < p.rot);
      } else if (at >= 0) {
        const bool is_v = h >= hq + p.hkv;
        const int hk = h - hq - (is_v ? p.hkv : 0);
        unit2(p, s_cs[r], static_cast<const T*>(is_v ? p.v : p.k) + row * (is_v ? p.ld_v : p.ld_k) + hk * p.dh,
              (is_v ? p.vc : p.kc) + (static_cast<size_t>(at) * p.hkv + hk) * p.dh, u, !is_v && 2 * u < p.rot);
      }
    }
  }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(AP_THREADS, 3) append_kernel(const __grid_constant__ AppendParams p) {
  const LaunchStamp ls(p.stamp);
  __shared__ float2 s_cs[AP_ROWS][EAGLE_MAX_ROPE_PAIRS];
  __shared__ long long s_at[AP_ROWS];        // cache row, -1: not written
  __shared__ int s_pos[AP_ROWS];
  __shared__ int s_any[AP_ROWS];             // the row belongs to a request
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hq = p.q ? p.hq : 0;
  // packed row r as the CTA's row w, of request b (-1: none)
  auto place = [&](int w, int r, int b) {
    long long at = -1;
    int pos = 0;
    if (b >= 0) {
      int lo, hi;
      request_rows(p.rows, b, lo, hi);
      const int L = p.len[b], i = r - lo;
      pos = p.pos ? p.pos[r] : L + i;
      if (cache_takes(p.paged, p.cap, b, L, hi - lo, lane))
        at = p.paged.table ? paged_row(p.paged, b, L + i) : static_cast<long long>(b) * p.cap + L + i;
    }
    if (lane == 0) {
      s_at[w] = at;
      s_pos[w] = pos;
      s_any[w] = b >= 0;
    }
  };
  if (static_cast<int>(blockIdx.x) < p.row_ctas) {
    const int r0 = blockIdx.x * p.tile;
    const int rows = min(p.tile, p.rows.n_rows - r0);
    for (int w = warp; w < rows; w += AP_WARPS) place(w, r0 + w, request_of_row(p.rows, r0 + w, lane));
    __syncthreads();
    append_rows<T, WIDE>(p, r0, rows, hq, s_cs, s_at, s_pos, s_any);
    return;
  }
  // the requests' new lengths
  const int b0 = (static_cast<int>(blockIdx.x) - p.row_ctas) * AP_WARPS, b = b0 + warp;
  bool found = true;                         // the CTAs of rows find the request's rows
  if (b < p.rows.B) {
    int lo, hi;
    const bool ok = request_rows(p.rows, b, lo, hi);
    const int L = p.len[b];
    const bool room = cache_takes(p.paged, p.cap, b, L, hi - lo, lane);
    if (lane == 0) {
      p.len_out[b] = room ? L + (hi - lo) : L;
      if (!ok) set_status(p.status, EAGLE_ERR_INVALID_ARG);
      if (!room) set_status(p.status, EAGLE_ERR_CAPACITY);
    }
    if (hi > lo) found = request_of_row(p.rows, lo, lane) == b;
    if (hi > lo + 1) found = found && request_of_row(p.rows, hi - 1, lane) == b;
  }
  if (__syncthreads_and(found)) return;
  // Other requests' starts mislead the search: the rows it does not give to these requests are appended here, so that
  // a request always has all its rows.  A query is turned once, here where the search gives its row to no request.
  for (int e = b0; e < min(b0 + AP_WARPS, p.rows.B); ++e) {
    int lo, hi;
    request_rows(p.rows, e, lo, hi);
    for (int x = lo; x < hi; x += AP_ROWS)
      for (int q = 0; q < 2; ++q) {
        const int r = x + warp;
        if (r < hi) {
          const int s = request_of_row(p.rows, r, lane);
          const bool turns = s < 0 && first_request_of_row(p.rows, r, lane) == e;
          place(warp, r, s != e && turns == (q == 1) ? e : -1);
        }
        __syncthreads();
        append_rows<T, false>(p, x, min(AP_ROWS, hi - x), q ? hq : 0, s_cs, s_at, s_pos, s_any);
        __syncthreads();
      }
  }
}

}  // namespace

cudaError_t launch_append(eagle_ctx* ctx, const AppendLaunch& A, cudaStream_t st) {
  const eagle_dims& D = ctx->dims;
  AppendParams p{};
  p.rows = PackedRows{A.rows->row_start, A.rows->n_rows, A.batch};
  p.hq = D.n_q_heads;
  p.hkv = D.n_kv_heads;
  p.dh = D.head_dim;
  if (A.rope) {
    p.rot = A.rope->rot_dim;
    p.interleaved = A.rope->interleaved;
    p.mscale = A.rope->mscale;
    for (int j = 0; j < EAGLE_MAX_ROPE_PAIRS; ++j) p.turn[j] = A.rope->turn[j];
  }
  p.q = A.q;
  p.k = A.k;
  p.v = A.v;
  p.q_out = A.q_out;
  p.ld_q = A.ld_q;
  p.ld_qo = A.ld_qo;
  p.ld_k = A.ld_k;
  p.ld_v = A.ld_v;
  p.kc = A.kv->k;
  p.vc = A.kv->v;
  p.cap = A.kv->cap;
  p.len = A.kv->len;
  p.paged = paged_of(&A.kv->paging, A.kv->cap);
  p.pos = A.pos;
  p.len_out = A.len_out;
  p.status = A.status;
  // Few rows spread over the SMs, one or two a CTA; with many a CTA's setup pays from 4 and then 8 on.  64/8 heads (no
  // others were measured),
  // 1 / 2 / 4 / 8 rows a CTA: 304 rows 5.6 / 5.8 / 8.1 / 13.3 us, 608: 8.5 / 7.6 / 8.8 / 13.2, 1216: 14.6 / 14.0 /
  // 13.1 / 17.7, 4864: 50 / 43 / 40 / 45, 9728: 93 / 78 / 75 / 74.
  const int per_sm = ceil_div(A.rows->n_rows, ctx->sm_count);
  p.tile = per_sm <= 2 ? 1 : per_sm <= 4 ? 2 : per_sm <= 48 ? 4 : AP_ROWS;
  p.row_ctas = ceil_div(A.rows->n_rows, p.tile);
  p.stamp = stamp_slot(ctx, EAGLE_K_APPEND);
  const dim3 grid(static_cast<unsigned>(p.row_ctas) + ceil_div(A.batch, AP_WARPS));
  const bool wide = p.rot % 16 == 0;
  trace_before(ctx, EAGLE_K_APPEND, st);
  cudaError_t e;
  if (A.dtype == EAGLE_DTYPE_F32)
    e = wide ? launch_pdl(append_kernel<float, true>, grid, dim3(AP_THREADS), 0, st, p)
             : launch_pdl(append_kernel<float, false>, grid, dim3(AP_THREADS), 0, st, p);
  else
    e = wide ? launch_pdl(append_kernel<uint16_t, true>, grid, dim3(AP_THREADS), 0, st, p)
             : launch_pdl(append_kernel<uint16_t, false>, grid, dim3(AP_THREADS), 0, st, p);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_APPEND, st);
  return e;
}

}  // namespace eagle
