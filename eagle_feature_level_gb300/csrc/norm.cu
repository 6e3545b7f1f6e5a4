// eagle_add_norm: h = x + residual, out = h / sqrt(mean(h^2) + eps) * gain, out in bf16, fp32 or a microscaled format.
//
// One pass: a row's h stays in the registers of its threads (eight consecutive elements a unit, up to four units a
// thread, two as a rule), its squares are summed over the warps, then the same registers are scaled, rounded and stored.
// A block goes on with other rows, the next one's loads under the present one's work and the gains kept.
//
// Bound: memory where rows are many (8192 x 8192 to 8 bits with the residual: 86 us, 470 MB, 5.5 TB/s; with blocks that end
// with their rows 96), else the latency of a launch, of loads and of two sums (8 x 4096: 2.2 us; 777 x 5120 in fp32:
// 12.8 us for 56 MB; past 16384 columns a block is alone on its SM: 777 x 28672 80 us, 313 MB).  Blocks of up to 512
// threads are held to 64 registers, so that an SM has two: one waits for its sums while the other works.  Rows past 256
// columns pay for that with spills: none from bf16 with a bf16 residual to bf16 or fp32, 64 bytes a thread with an fp32
// residual, 32 to 104 from bf16 to a microscaled format, up to 216 where all is fp32; past 16384 columns 148 to 596.
#include "internal.h"
#include "common.cuh"
#include "mx.cuh"

namespace eagle {
namespace {

struct NormParams {
  const void* x;
  const void* res;
  void* res_out;
  void* out;
  MxView m;
  long long ld_x, ld_res, ld_ro, ld_out;
  const float* gain;
  float eps;
  int rows, cols;
  int threads;             // of a row: a power of two from 32 on, or a block of 256 or more
  int* status;
  uint64_t* stamp;
};

// OUT: 0 bf16, -1 fp32, otherwise a microscaled format.
template <typename T, typename R, int OUT, int UNITS, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 512 ? 2 : 1) norm_kernel(NormParams p) {
  // (four units leave no registers for gains and the next row)
  constexpr bool AHEAD = UNITS <= 2;
  __shared__ float s_sum[2][32];
  LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = p.threads < 256 ? threadIdx.x & (p.threads - 1) : threadIdx.x;
  const int per_block = blockDim.x / p.threads, step = gridDim.x * per_block;
  int row = blockIdx.x * per_block + threadIdx.x / p.threads;
  const int rounds = (p.rows + step - 1) / step;           // the same for a block's threads
  const MxFactor f = OUT > 0 ? mx_factor(p.m) : MxFactor{1.0f, 1.0f, 1.0f};
  int col[UNITS];
  bool own[UNITS];
  float gain[AHEAD ? UNITS : 1][8];
  Raw8<T> x[UNITS];
  Raw8<R> res[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    col[u] = (u * p.threads + t) * 8;
    own[u] = col[u] < p.cols;
    if (AHEAD && own[u] && row < p.rows) {
      x[u].load(static_cast<const T*>(p.x) + row * p.ld_x + col[u]);
      if (p.res) res[u].load(static_cast<const R*>(p.res) + row * p.ld_res + col[u]);
    }
  }
  auto gains = [&](int u, float (&g)[8]) {
    if (p.gain && own[u]) load8(p.gain + col[u], g);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 1.0f;
  };
  if (AHEAD)
#pragma unroll
    for (int u = 0; u < UNITS; ++u) gains(u, gain[AHEAD ? u : 0]);
  bool bad = false;
  for (int k = 0; k < rounds; ++k, row += step) {
    const bool there = row < p.rows;
    float h[UNITS][8];
    float sum = 0.0f;
    if (!AHEAD)
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
        if (there && own[u]) {
          x[u].load(static_cast<const T*>(p.x) + row * p.ld_x + col[u]);
          if (p.res) res[u].load(static_cast<const R*>(p.res) + row * p.ld_res + col[u]);
        }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      if (there && own[u]) {
        x[u].get(h[u]);
        if (p.res) {
          float r[8];
          res[u].get(r);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[u][i] += r[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[u][i] = 0.0f;
      }
    }
    // the next row is on its way under this one's work
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      if (AHEAD && own[u] && row + step < p.rows) {
        x[u].load(static_cast<const T*>(p.x) + (row + step) * p.ld_x + col[u]);
        if (p.res) res[u].load(static_cast<const R*>(p.res) + (row + step) * p.ld_res + col[u]);
      }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      if (p.res_out && there && own[u]) store8(static_cast<R*>(p.res_out) + row * p.ld_ro + col[u], h[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(h[u][i], h[u][i], sum);
    }
    sum = warp_sum(sum);
    if (p.threads > 32) {
      float* s = s_sum[k & 1];                   // (in turn: the last row's sums may still be read)
      if (lane == 0) s[warp] = sum;
      __syncthreads();
      const int nw = p.threads >> 5, w0 = p.threads < 256 ? warp & ~(nw - 1) : 0;
      sum = warp_sum(lane < nw ? s[w0 + lane] : 0.0f);
    }
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      float y[8];
      if (!AHEAD) gains(u, gain[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[u][i] * inv * gain[AHEAD ? u : 0][i];
      const bool in = there && own[u];
      if (OUT > 0) {
        if (!in)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        bad |= mx_put<OUT>(p.m, f, row, col[u], in, y, lane);
      } else if (in) {
        if (OUT == 0) store8(static_cast<uint16_t*>(p.out) + row * p.ld_out + col[u], y);
        else store8(static_cast<float*>(p.out) + row * p.ld_out + col[u], y);
      }
    }
  }
  if (bad) set_status(p.status, EAGLE_ERR_NUMERIC);
}

typedef void (*NormKernel)(NormParams);

// Rows of up to 8192 columns: 512 threads at most, and registers for them.
template <typename T, typename R, int OUT>
NormKernel kernel_of(int units, int threads) {
  if (threads <= 512) return units == 1 ? norm_kernel<T, R, OUT, 1, 512> : norm_kernel<T, R, OUT, 2, 512>;
  return units <= 2 ? norm_kernel<T, R, OUT, 2, 1024> : norm_kernel<T, R, OUT, 4, 1024>;
}
template <typename T, typename R>
NormKernel kernel_of(const eagle_norm* n, int units, int threads) {
  if (!n->out_mx)
    return n->out_dtype == EAGLE_DTYPE_F32 ? kernel_of<T, R, -1>(units, threads) : kernel_of<T, R, 0>(units, threads);
  switch (n->out_mx->format) {
    case EAGLE_MX_FP8: return kernel_of<T, R, EAGLE_MX_FP8>(units, threads);
    case EAGLE_MX_FP4: return kernel_of<T, R, EAGLE_MX_FP4>(units, threads);
    default: return kernel_of<T, R, EAGLE_NV_FP4>(units, threads);
  }
}

}  // namespace

cudaError_t launch_norm(eagle_ctx* ctx, const eagle_norm* n, int* status, cudaStream_t st) {
  NormParams p{};
  p.x = n->x;
  p.res = n->residual;
  p.res_out = n->residual_out;
  p.out = n->out;
  if (n->out_mx) p.m = mx_view(n->out_mx);
  p.ld_x = n->ld_x;
  p.ld_res = n->ld_res;
  p.ld_ro = n->ld_res_out;
  p.ld_out = n->ld_out;
  p.gain = n->gain;
  p.eps = n->eps;
  p.rows = n->rows;
  p.cols = n->cols;
  p.status = status;
  const int eights = ceil_div(n->cols, 8);
  // two units a thread (four past 16384 columns): as many whole warps as that takes, where a row has a block to itself (777
  // x 5120: 320 threads, three blocks an SM, 12.7 us; 512, the next power of two, 13.5; 8192 rows to NV_FP4 85 and 104)
  p.threads = 32;
  while (p.threads < 256 && p.threads * 2 < eights) p.threads <<= 1;
  if (p.threads * 2 < eights) p.threads = ceil_div(ceil_div(eights, eights <= 2048 ? 2 : 4), 32) * 32;
  const int need = ceil_div(eights, p.threads);
  const int units = need <= 1 ? 1 : need <= 2 ? 2 : 4;
  const int block = p.threads < 256 ? 256 : p.threads;
  const bool f = n->dtype == EAGLE_DTYPE_F32, rf = n->res_dtype == EAGLE_DTYPE_F32;
  const NormKernel k = f && rf ? kernel_of<float, float>(n, units, p.threads)
                       : f     ? kernel_of<float, uint16_t>(n, units, p.threads)
                       : rf    ? kernel_of<uint16_t, float>(n, units, p.threads)
                               : kernel_of<uint16_t, uint16_t>(n, units, p.threads);
  p.stamp = stamp_slot(ctx, EAGLE_K_NORM);
  // as many blocks as fit the GPU at once, each on with the next rows
  int per_sm = 1;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, block, 0) != cudaSuccess || per_sm < 1) per_sm = 1;
  const int blocks = ceil_div(n->rows, block / p.threads), most = per_sm * ctx->sm_count;
  trace_before(ctx, EAGLE_K_NORM, st);
  const cudaError_t e = launch_pdl(k, dim3(blocks < most ? blocks : most), dim3(block), 0, st, p);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_NORM, st);
  return e;
}

}  // namespace eagle
