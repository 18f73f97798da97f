// int8.cu -- the linear layer on a symmetric 8-bit base: quantization of
// weight and activation rows, and the integer product with a scale for each
// token and channel.
//
//   row quantization  s = fl(max |x| / 127), n = clamp(rint(fl(x / s)), -127, 127)
//   forward           Y[t, o]  = s_x[t] (sum_i n_x[t, i] n_w[o, i]) s_w[o] + s U B^T
//   input gradient    dX[t, i] = s_g[t] (sum_o n_g[t, o] n_w[o, i]) + s V A,
//                     n_g, s_g the rows of fl(dY s_w): the channel scale lies
//                     along the sum there, so it goes into what is quantized
//
// The integer sum is exact in 32 bits for up to 131072 terms (127^2 2^17 <
// 2^31), so nothing depends on its order.  Everything after it is fp32, with
// one rounding to the type of the output.
#include "common.cuh"
#include "int8.h"
#include "internal.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

// Largest of non-negative values by their bits, so that a NaN wins over all.
__device__ __forceinline__ uint32_t block_max_bits(uint32_t x) {
  __shared__ uint32_t buf[32];
  x = __reduce_max_sync(0xffffffffu, x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) buf[warp] = x;
  __syncthreads();
  x = buf[0];
  for (int w = 1; w < (int)(blockDim.x >> 5); ++w) x = max(x, buf[w]);
  return x;
}

__device__ __forceinline__ int8_t code_of(float x, float s) {
  if (s == 0.0f) return 0;
  const float q = rintf(__fdiv_rn(x, s));
  return (int8_t)(int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// One CTA per row of P [R x K] (times the column factors f, where given):
// codes [R x pitch] with zeros in the padding, and the row's scale.  hdr:
// raise the non-finite flag; otherwise a row with a NaN or Inf gets a NaN
// scale (and with it a row of NaN outputs).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const T* __restrict__ P, int64_t K, int64_t pitch, const float* __restrict__ f,
                int8_t* __restrict__ codes, float* __restrict__ scale, uint32_t* __restrict__ hdr) {
  const int64_t row = blockIdx.x;
  const T* x = P + row * K;
  uint32_t top = 0;
  for (int64_t k = threadIdx.x; k < K; k += kThreads) {
    const float v = f ? __fmul_rn(to_f32(x[k]), f[k]) : to_f32(x[k]);
    top = max(top, __float_as_uint(fabsf(v)));
  }
  top = block_max_bits(top);
  const bool bad = top >= 0x7f800000u;
  const float s = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(top), 127.0f);
  if (threadIdx.x == 0) {
    scale[row] = s;
    if (bad && hdr) atomicOr(hdr + 2, 1u);
  }
  int8_t* q = codes + row * pitch;
  for (int64_t k = threadIdx.x; k < pitch; k += kThreads) {
    int8_t c = 0;
    if (k < K && !bad) c = code_of(f ? __fmul_rn(to_f32(x[k]), f[k]) : to_f32(x[k]), s);
    q[k] = c;
  }
}

__global__ void __launch_bounds__(kThreads)
    dequantize_rows_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scale,
                           int64_t O, int64_t I, int64_t pitch, float* __restrict__ out) {
  const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (n >= O * I) return;
  const int64_t o = n / I;
  out[n] = __fmul_rn((float)codes[o * pitch + (n - o * I)], scale[o]);
}

struct Layout {
  size_t scale, codes, total;
};
Layout layout(int64_t R, int64_t K) {
  Layout l;
  l.scale = 0;
  l.codes = align_up((size_t)R * 4, 256);
  l.total = l.codes + align_up((size_t)R * (size_t)int8_pitch(K), 256);
  return l;
}

}  // namespace

cudaError_t launch_int8_quantize(const float* W, int64_t O, int64_t I, int8_t* codes, float* scale,
                                 void* ws, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(ws, 0, kWsHeader, st);
  if (e != cudaSuccess || O == 0) return e;
  rows_kernel<float><<<(unsigned)O, kThreads, 0, st>>>(W, I, int8_pitch(I), nullptr, codes, scale,
                                                       (uint32_t*)ws);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_int8_dequantize(const int8_t* codes, const float* scale, int64_t O, int64_t I,
                                   float* out, cudaStream_t st) {
  const int64_t N = O * I;
  if (N == 0) return cudaSuccess;
  dequantize_rows_kernel<<<(unsigned)((N + kThreads - 1) / kThreads), kThreads, 0, st>>>(
      codes, scale, O, I, int8_pitch(I), out);
  count_launch();
  return cudaGetLastError();
}

size_t int8_ws(bool dx, int64_t R, int64_t O, int64_t I, int32_t r) {
  return layout(R, dx ? O : I).total + int8_tc_ws(dx, R, O, I, r);
}

cudaError_t launch_int8_rows(const Int8Call& c, void* ws, cudaStream_t st) {
  const int64_t K = c.dx ? c.O : c.I;
  const Layout l = layout(c.R, K);
  float* xs = (float*)((char*)ws + l.scale);
  int8_t* xq = (int8_t*)ws + l.codes;
  const size_t zero = int8_tc_zeroed(c.dx, c.R, c.O, c.I);
  if (zero) {
    const cudaError_t e = cudaMemsetAsync((char*)ws + l.total, 0, zero, st);
    if (e != cudaSuccess) return e;
  }
  const float* f = c.dx ? c.wscale : nullptr;
  if (c.bf16)
    rows_kernel<__nv_bfloat16><<<(unsigned)c.R, kThreads, 0, st>>>((const __nv_bfloat16*)c.P, K,
                                                                  int8_pitch(K), f, xq, xs, nullptr);
  else
    rows_kernel<float><<<(unsigned)c.R, kThreads, 0, st>>>((const float*)c.P, K, int8_pitch(K), f, xq,
                                                           xs, nullptr);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_int8_product(const Int8Call& c, void* ws, uint32_t* hdr, cudaStream_t st) {
  const Layout l = layout(c.R, c.dx ? c.O : c.I);
  return launch_int8_tc(c, (const int8_t*)ws + l.codes, (const float*)((char*)ws + l.scale),
                        (char*)ws + l.total, hdr, st);
}

}  // namespace qlora
