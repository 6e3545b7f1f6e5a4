// eagle_add_norm: h = x + residual, out = h / sqrt(mean(h^2) + eps) * gain, out in bf16, fp32 or a microscaled format.
//
// One pass: a row's h stays in the registers of its threads (eight consecutive elements a unit, up to four units a
// thread), its squares are summed over the warps, then the same registers are scaled, rounded and stored.
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
  int threads;             // of a row, a power of two from 32 on
  int* status;
  uint64_t* stamp;
};

constexpr int NM_UNITS = 4;

// OUT: 0 bf16, -1 fp32, otherwise a microscaled format.
template <typename T, typename R, int OUT, int UNITS>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p) {
  __shared__ float s_sum[32];
  LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x & (p.threads - 1);
  const int row = blockIdx.x * (blockDim.x / p.threads) + threadIdx.x / p.threads;
  const bool there = row < p.rows;
  float h[UNITS][8];
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int col = (u * p.threads + t) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[u][i] = 0.0f;
    if (there && col < p.cols) {
      load8(static_cast<const T*>(p.x) + row * p.ld_x + col, h[u]);
      if (p.res) {
        float r[8];
        load8(static_cast<const R*>(p.res) + row * p.ld_res + col, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[u][i] += r[i];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int col = (u * p.threads + t) * 8;
    if (p.res_out && there && col < p.cols) store8(static_cast<R*>(p.res_out) + row * p.ld_ro + col, h[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(h[u][i], h[u][i], sum);
  }
  sum = warp_sum(sum);
  if (p.threads > 32) {
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    const int nw = p.threads >> 5, w0 = warp & ~(nw - 1);
    sum = warp_sum(lane < nw ? s_sum[w0 + lane] : 0.0f);
  }
  const float inv = 1.0f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
  const float g = p.m.g ? *p.m.g : 1.0f;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int col = (u * p.threads + t) * 8;
    const bool in = there && col < p.cols;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = h[u][i] * inv;
    if (p.gain && col < p.cols) {
      float gain[8];
      load8(p.gain + col, gain);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= gain[i];
    }
    if (OUT > 0) {
      if (!in)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.0f;
      bad |= mx_put<OUT>(p.m, g, row, col, in, y, lane);
    } else if (in) {
      if (OUT == 0) store8(static_cast<uint16_t*>(p.out) + row * p.ld_out + col, y);
      else store8(static_cast<float*>(p.out) + row * p.ld_out + col, y);
    }
  }
  if (bad) set_status(p.status, EAGLE_ERR_NUMERIC);
}

typedef void (*NormKernel)(NormParams);

template <typename T, typename R, int OUT>
NormKernel kernel_of(int units) {
  return units == 1 ? norm_kernel<T, R, OUT, 1> : units == 2 ? norm_kernel<T, R, OUT, 2> : norm_kernel<T, R, OUT, 4>;
}
template <typename T, typename R>
NormKernel kernel_of(const eagle_norm* n, int units) {
  if (!n->out_mx) return n->out_dtype == EAGLE_DTYPE_F32 ? kernel_of<T, R, -1>(units) : kernel_of<T, R, 0>(units);
  switch (n->out_mx->format) {
    case EAGLE_MX_FP8: return kernel_of<T, R, EAGLE_MX_FP8>(units);
    case EAGLE_MX_FP4: return kernel_of<T, R, EAGLE_MX_FP4>(units);
    default: return kernel_of<T, R, EAGLE_NV_FP4>(units);
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
  p.threads = 32;
  while (p.threads < 1024 && p.threads * NM_UNITS < eights) p.threads <<= 1;
  const int need = ceil_div(eights, p.threads);
  const int units = need <= 1 ? 1 : need <= 2 ? 2 : 4;
  const int block = p.threads < 256 ? 256 : p.threads;
  const bool f = n->dtype == EAGLE_DTYPE_F32, rf = n->res_dtype == EAGLE_DTYPE_F32;
  const NormKernel k = f ? (rf ? kernel_of<float, float>(n, units) : kernel_of<float, uint16_t>(n, units))
                         : (rf ? kernel_of<uint16_t, float>(n, units) : kernel_of<uint16_t, uint16_t>(n, units));
  p.stamp = stamp_slot(ctx, EAGLE_K_NORM);
  trace_before(ctx, EAGLE_K_NORM, st);
  const cudaError_t e = launch_pdl(k, dim3(ceil_div(n->rows, block / p.threads)), dim3(block), 0, st, p);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_NORM, st);
  return e;
}

}  // namespace eagle
