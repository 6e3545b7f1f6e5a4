// eagle_mx_quantize and eagle_mx_unpack: rows to and from the microscaled formats.
//
// A warp takes 256 columns of a row, a lane eight of them: 16 or 32 bytes in, 4 or 8 out, with a block's maximum and
// the four scales of a group exchanged between its lanes.
#include "internal.h"
#include "common.cuh"
#include "mx.cuh"

namespace eagle {
namespace {

constexpr int QT_THREADS = 256;
constexpr int QT_WARPS = QT_THREADS / 32;

struct QuantParams {
  MxView m;
  const void* x;           // quantise: rows in; unpack: rows out
  long long ld;
  int chunks;              // of 256 columns a row
  long long tasks;         // rows x chunks
  int* status;
  uint64_t* stamp;
};

// SiLU(a) b in fp32.
__device__ __forceinline__ float gated(float a, float b) { return a / (1.0f + expf(-a)) * b; }

template <int FMT, typename T, bool SWIGLU>
__global__ void __launch_bounds__(QT_THREADS) quantize_kernel(QuantParams p) {
  LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const float g = p.m.g ? *p.m.g : 1.0f;
  bool bad = false;
  for (long long t = static_cast<long long>(blockIdx.x) * QT_WARPS + (threadIdx.x >> 5); t < p.tasks;
       t += static_cast<long long>(gridDim.x) * QT_WARPS) {
    const int row = static_cast<int>(t / p.chunks), col = static_cast<int>(t % p.chunks) * 256 + lane * 8;
    const bool in = col < p.m.cols;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in) {
      const T* from = static_cast<const T*>(p.x) + row * p.ld + col;
      load8(from, x);
      if (SWIGLU) {
        float y[8];
        load8(from + p.m.cols, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = gated(x[i], y[i]);
      }
    }
    bad |= mx_put<FMT>(p.m, g, row, col, in, x, lane);
  }
  if (bad) set_status(p.status, EAGLE_ERR_NUMERIC);
}

template <int FMT, typename T>
__global__ void __launch_bounds__(QT_THREADS) unpack_kernel(QuantParams p) {
  LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const float g = p.m.g ? *p.m.g : 1.0f;
  for (long long t = static_cast<long long>(blockIdx.x) * QT_WARPS + (threadIdx.x >> 5); t < p.tasks;
       t += static_cast<long long>(gridDim.x) * QT_WARPS) {
    const int row = static_cast<int>(t / p.chunks), col = static_cast<int>(t % p.chunks) * 256 + lane * 8;
    if (col >= p.m.cols) continue;
    float v[8];
    mx_get<FMT>(p.m, g, row, col, v);
    store8(static_cast<T*>(const_cast<void*>(p.x)) + row * p.ld + col, v);
  }
}

typedef void (*QuantKernel)(QuantParams);

template <int FMT>
QuantKernel quantize_of(int dtype, int act) {
  if (dtype == EAGLE_DTYPE_F32)
    return act == EAGLE_ACT_SWIGLU ? quantize_kernel<FMT, float, true> : quantize_kernel<FMT, float, false>;
  return act == EAGLE_ACT_SWIGLU ? quantize_kernel<FMT, uint16_t, true> : quantize_kernel<FMT, uint16_t, false>;
}
template <int FMT>
QuantKernel unpack_of(int dtype) {
  return dtype == EAGLE_DTYPE_F32 ? unpack_kernel<FMT, float> : unpack_kernel<FMT, uint16_t>;
}

cudaError_t launch(eagle_ctx* ctx, QuantKernel k, const eagle_mx* m, const void* x, int ld, int* status,
                   cudaStream_t st) {
  QuantParams p{};
  p.m = mx_view(m);
  p.x = x;
  p.ld = ld;
  p.chunks = ceil_div(m->cols, 256);
  p.tasks = static_cast<long long>(m->rows) * p.chunks;
  p.status = status;
  p.stamp = stamp_slot(ctx, EAGLE_K_QUANT);
  const long long want = (p.tasks + QT_WARPS - 1) / QT_WARPS;
  const long long most = 8ll * ctx->sm_count;
  trace_before(ctx, EAGLE_K_QUANT, st);
  const cudaError_t e = launch_pdl(k, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(QT_THREADS), 0, st, p);
  ctx->launches++;
  trace_after(ctx, EAGLE_K_QUANT, st);
  return e;
}

}  // namespace

cudaError_t launch_quantize(eagle_ctx* ctx, int dtype, int act, const void* x, int ld, const eagle_mx* out, int* status,
                            cudaStream_t st) {
  const QuantKernel k = out->format == EAGLE_MX_FP8   ? quantize_of<EAGLE_MX_FP8>(dtype, act)
                        : out->format == EAGLE_MX_FP4 ? quantize_of<EAGLE_MX_FP4>(dtype, act)
                                                      : quantize_of<EAGLE_NV_FP4>(dtype, act);
  return launch(ctx, k, out, x, ld, status, st);
}

cudaError_t launch_unpack(eagle_ctx* ctx, const eagle_mx* x, int dtype, void* y, int ld, cudaStream_t st) {
  const QuantKernel k = x->format == EAGLE_MX_FP8   ? unpack_of<EAGLE_MX_FP8>(dtype)
                        : x->format == EAGLE_MX_FP4 ? unpack_of<EAGLE_MX_FP4>(dtype)
                                                    : unpack_of<EAGLE_NV_FP4>(dtype);
  return launch(ctx, k, x, y, ld, nullptr, st);
}

}  // namespace eagle
