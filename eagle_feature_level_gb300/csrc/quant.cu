// eagle_mx_quantize and eagle_mx_unpack: rows to and from the microscaled formats.
//
// A warp takes 256 columns and goes down the rows, two in flight; a lane has eight columns: 16 or 32 bytes in, 4 or 8 out,
// with a block's maximum and the four scales of a group exchanged between its lanes.
//
// Bound: the latency of loads, which are waited for in the turn of the loop that asks for them: 4096 x 8192 to NV_FP4 26 us
// (86 MB, 3.3 TB/s) with the issue slots 57 % full and half of the warps there, 1001 x 11008 gated pairs to FP4 15.6 us (50
// MB, slots 52 % full).  Unpacking, which has nothing to exchange, is bound by memory: 8192 x 8192 in 8 bits 33.8 us (203 MB,
// 6.0 TB/s).
#include "internal.h"
#include "common.cuh"
#include "mx.cuh"

namespace eagle {
namespace {

constexpr int QT_THREADS = 256;
constexpr int QT_WARPS = QT_THREADS / 32;

constexpr int QT_ROWS = 2;              // rows of a warp in flight

struct QuantParams {
  MxView m;
  const void* x;           // quantise: rows in; unpack: rows out
  long long ld;
  int chunks;              // of 256 columns a row
  int step;                // warps of a chunk
  int* status;
  uint64_t* stamp;
};

// e^(-a) to two steps of fp32: 2^y of y = -a log2(e), the low part of that product put right behind it (up to the largest
// number: a half step of y is 2^-18.5 of the power there).
__device__ __forceinline__ float exp_minus(float a) {
  constexpr float L = 0x1.715476p+0f, L_LOW = 0x1.4ae0cp-26f, LN2 = 0x1.62e43p-1f;
  const float y = -a * L;
  const float low = fmaf(-a, L, -y) - a * L_LOW;
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
  return fabsf(y) < 128.0f ? fmaf(e, low * LN2, e) : e;
}
// SiLU(a) b in fp32.
__device__ __forceinline__ float gated(float a, float b) {
  const float d = 1.0f + exp_minus(a);
  return d < 0x1p126f ? mx_quotient(a, d, mx_rcp(d)) * b : a / d * b;
}

template <int FMT, typename T, bool SWIGLU>
__global__ void __launch_bounds__(QT_THREADS) quantize_kernel(QuantParams p) {
  LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = blockIdx.x * QT_WARPS + (threadIdx.x >> 5);
  const MxFactor f = mx_factor(p.m);
  const int col = warp % p.chunks * 256 + lane * 8;
  const bool in = col < p.m.cols;
  bool bad = false;
  for (int r0 = warp / p.chunks; r0 < p.m.rows && warp < p.step * p.chunks; r0 += QT_ROWS * p.step) {
    Raw8<T> a[QT_ROWS], b[QT_ROWS];
#pragma unroll
    for (int i = 0; i < QT_ROWS; ++i) {
      const int row = r0 + i * p.step;
      if (in && row < p.m.rows) {
        const T* from = static_cast<const T*>(p.x) + row * p.ld + col;
        a[i].load(from);
        if (SWIGLU) b[i].load(from + p.m.cols);
      }
    }
#pragma unroll
    for (int i = 0; i < QT_ROWS; ++i) {
      const int row = r0 + i * p.step;
      if (row >= p.m.rows) break;
      float x[8];
      a[i].get(x);
      if (SWIGLU) {
        float y[8];
        b[i].get(y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = gated(x[j], y[j]);
      }
      if (!in)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.0f;
      bad |= mx_put<FMT>(p.m, f, row, col, in, x, lane);
    }
  }
  if (bad) set_status(p.status, EAGLE_ERR_NUMERIC);
}

template <int FMT, typename T>
__global__ void __launch_bounds__(QT_THREADS) unpack_kernel(QuantParams p) {
  LaunchStamp ls(p.stamp);
  pdl_wait();
  ls.waited();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = blockIdx.x * QT_WARPS + (threadIdx.x >> 5);
  const float g = p.m.g ? *p.m.g : 1.0f;
  const int col = warp % p.chunks * 256 + lane * 8;
  if (col >= p.m.cols || warp >= p.step * p.chunks) return;
  for (int r0 = warp / p.chunks; r0 < p.m.rows; r0 += QT_ROWS * p.step) {
    MxRaw<FMT> a[QT_ROWS];
#pragma unroll
    for (int i = 0; i < QT_ROWS; ++i)
      if (r0 + i * p.step < p.m.rows) a[i].load(p.m, r0 + i * p.step, col);
#pragma unroll
    for (int i = 0; i < QT_ROWS; ++i) {
      const int row = r0 + i * p.step;
      if (row >= p.m.rows) break;
      float v[8];
      mx_get<FMT>(a[i], g, v);
      store8(static_cast<T*>(const_cast<void*>(p.x)) + row * p.ld + col, v);
    }
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
  // a warp keeps to its 256 columns and goes down the rows; as many warps as there are rows for, up to 96 an SM (4096 x 8192
  // to NV_FP4: two rows in flight 26.1 us, one 29.5, four 26.5; 48 warps an SM 29.4, 160 26.4)
  const int most = 96 * ctx->sm_count / p.chunks;
  p.step = most < 1 ? 1 : m->rows < most ? m->rows : most;
  p.status = status;
  p.stamp = stamp_slot(ctx, EAGLE_K_QUANT);
  trace_before(ctx, EAGLE_K_QUANT, st);
  const cudaError_t e =
      launch_pdl(k, dim3(ceil_div(p.step * p.chunks, QT_WARPS)), dim3(QT_THREADS), 0, st, p);
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
