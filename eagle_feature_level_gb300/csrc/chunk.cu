// eagle_chunk_attn: causal attention of a batch's new rows over the cache
// that holds them.  One warp per (row, query head): online softmax over the
// row's keys, the head's elements spread over the lanes.
#include <algorithm>

#include "internal.h"
#include "common.cuh"
#include "rows.cuh"

namespace eagle {
namespace {

struct ChunkParams {
  PackedRows rows;
  int hq, hkv, dh, G;
  const uint16_t* q;
  uint16_t* out;
  long long ld_q, ld_o;
  const uint16_t* k;
  const uint16_t* v;
  int cap, window;
  const int32_t* len;
  PagedKv paged;
  float c;                 // scale * log2 e
  int* status;
  uint64_t* stamp;
};

__global__ void __launch_bounds__(128) chunk_simple_kernel(const ChunkParams p) {
  const LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < p.rows.B; b += blockDim.x) {
      int lo, hi;
      if (!request_rows(p.rows, b, lo, hi)) set_status(p.status, EAGLE_ERR_INVALID_ARG);
    }
  const int row = blockIdx.x, h = blockIdx.y * 4 + warp;
  if (h >= p.hq) return;
  const int b = request_of_row(p.rows, row, lane);
  if (b < 0) return;
  int lo, hi;
  request_rows(p.rows, b, lo, hi);
  int L = p.len[b];
  if (L > p.cap) {
    if (lane == 0) set_status(p.status, EAGLE_ERR_CAPACITY);
    L = p.cap;
  }
  const int pos = L - (hi - lo) + (row - lo);
  const int first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const int hk = h / p.G;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = lane + 32 * i < p.dh ? bf16_to_f32(p.q[row * p.ld_q + h * p.dh + lane + 32 * i]) * p.c : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = first; j <= pos; ++j) {
    const long long at = p.paged.table ? paged_row(p.paged, b, j) : static_cast<long long>(b) * p.cap + j;
    float s = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
    if (at >= 0) {
      const size_t base = (static_cast<size_t>(at) * p.hkv + hk) * p.dh;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.dh) {
          s += q[i] * bf16_to_f32(p.k[base + lane + 32 * i]);
          v[i] = bf16_to_f32(p.v[base + lane + 32 * i]);
        }
    } else if (lane == 0) {
      set_status(p.status, EAGLE_ERR_INVALID_ARG);
    }
    s = warp_sum(s);
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * f + w * v[i];
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < p.dh) p.out[row * p.ld_o + h * p.dh + lane + 32 * i] = f32_to_bf16(o[i] * inv);
}

}  // namespace

cudaError_t launch_chunk_attn(eagle_ctx* ctx, int batch, const eagle_rows* rows, const uint16_t* q, int ld_q,
                              const eagle_kv* kv, int window, float scale, uint16_t* out, int ld_out, void* ws,
                              cudaStream_t st) {
  const eagle_dims& D = ctx->dims;
  ChunkParams p{};
  p.rows = PackedRows{rows->row_start, rows->n_rows, batch};
  p.hq = D.n_q_heads;
  p.hkv = D.n_kv_heads;
  p.dh = D.head_dim;
  p.G = D.n_q_heads / D.n_kv_heads;
  p.q = q;
  p.out = out;
  p.ld_q = ld_q;
  p.ld_o = ld_out;
  p.k = kv->k;
  p.v = kv->v;
  p.cap = kv->cap;
  p.window = window >= kv->cap ? 0 : window;   // a window of the whole cache is none
  p.len = kv->len;
  p.paged = paged_of(&kv->paging, kv->cap);
  p.c = scale * 1.4426950408889634f;
  p.status = ws_ptr<int>(ws, ctx->ws.status);
  p.stamp = stamp_slot(ctx, EAGLE_K_CHUNK_ATTN);
  trace_before(ctx, EAGLE_K_CHUNK_ATTN, st);
  const cudaError_t e = launch_pdl(chunk_simple_kernel, dim3(rows->n_rows, ceil_div(D.n_q_heads, 4)), dim3(128), 0, st, p);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_CHUNK_ATTN, st);
  return e;
}

}  // namespace eagle
