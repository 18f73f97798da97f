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
// buf: two rows of 32 words, used in turn (one barrier a call).
__device__ __forceinline__ uint32_t block_max_bits(uint32_t x, uint32_t* buf) {
  x = __reduce_max_sync(0xffffffffu, x);
  const int lane = threadIdx.x & 31, warps = (int)(blockDim.x >> 5);
  if (lane == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < warps ? buf[lane] : 0u);
}

// Scale of a row whose largest magnitude has these bits; NaN where the row
// holds a NaN or Inf.
__device__ __forceinline__ float row_scale(uint32_t top) {
  return top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(top), 127.0f);
}

// Code of x as the low byte of the result: rint(fl(x / s)).  The product with
// the reciprocal is within 2^-15 of the quotient (at most 127 in magnitude,
// two roundings), so it rounds to the same integer unless it lies that close
// to a half; only then (and for scales whose reciprocal is not a normal
// number: inv is NaN) is the division done.  Adding 1.5 2^23 rounds to the
// nearest integer, ties to even, and leaves it in the low bits.
__device__ __forceinline__ uint32_t code_of(float x, float s, float inv) {
  const float y = __fmul_rn(x, inv);
  float t = __fadd_rn(y, 12582912.0f);
  if (!(fabsf(__fsub_rn(y, __fsub_rn(t, 12582912.0f))) < 0.49995f)) {
    const float q = s > 0.0f ? fminf(fmaxf(__fdiv_rn(x, s), -127.0f), 127.0f) : 0.0f;
    t = __fadd_rn(q, 12582912.0f);
  }
  return __float_as_uint(t) & 255u;
}
__device__ __forceinline__ float reciprocal(float s) {
  return s >= 1e-37f ? __fdiv_rn(1.0f, s) : __uint_as_float(0x7fc00000u);
}

// Two runs of 16-byte words to clear for the kernels after, by CTA cta of ctas.
struct Clear {
  uint4* p[2];
  int64_t n[2];
};
__device__ __forceinline__ void clear_part(const Clear& c, int64_t cta, int64_t ctas) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    for (int64_t i = cta * blockDim.x + threadIdx.x; i < c.n[k]; i += ctas * blockDim.x)
      c.p[k][i] = make_uint4(0, 0, 0, 0);
}

struct RowsArgs {
  const void* P;       // [R x K]
  int64_t R, K, pitch;
  const float* f;      // [K] column factors, nullable
  int8_t* codes;       // [R x pitch], zeros in the padding
  float* scale;        // [R]
  uint32_t* hdr;       // non-finite flag, nullable
  Clear clear;
};

// 16 bytes of activations as floats (8 bf16 or 4 fp32).
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void open(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void open(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
};

// Rows that take 16-byte accesses (K a multiple of 16, P aligned): a thread
// keeps its NV vectors of the row in registers between the maximum and the
// codes, so the row is read once; its column factors stay in registers over
// all the rows the CTA takes, and the next row is on its way while this one
// is reduced.
template <typename T, int NV, bool FACTOR>
__global__ void __launch_bounds__(512) rows_kernel(const RowsArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ uint32_t buf[2][32];
  const int64_t nvec = a.K / N;
  float f[FACTOR ? NV * N : 1];
  if (FACTOR) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t v = threadIdx.x + (int64_t)i * blockDim.x;
#pragma unroll
      for (int j = 0; j < N; ++j) f[i * N + j] = v < nvec ? __ldg(a.f + v * N + j) : 0.0f;
    }
  }
  uint4 next[NV];
  auto load = [&](int64_t row) {
    const uint4* x = reinterpret_cast<const uint4*>((const T*)a.P + row * a.K);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t v = threadIdx.x + (int64_t)i * blockDim.x;
      next[i] = v < nvec ? __ldg(x + v) : make_uint4(0, 0, 0, 0);
    }
  };
  int64_t row = blockIdx.x;
  if (row < a.R) load(row);
  clear_part(a.clear, blockIdx.x, gridDim.x);
  for (int k = 0; row < a.R; k ^= 1) {
    uint4 cur[NV];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cur[i] = next[i];
      float x[N];
      Vec<T>::open(cur[i], x);
#pragma unroll
      for (int j = 0; j < N; ++j)
        top = max(top, __float_as_uint(fabsf(FACTOR ? __fmul_rn(x[j], f[i * N + j]) : x[j])));
    }
    const int64_t now = row;
    row += gridDim.x;
    if (row < a.R) load(row);
    top = block_max_bits(top, buf[k]);
    const float s = row_scale(top);
    const float inv = reciprocal(s);
    if (threadIdx.x == 0) {
      a.scale[now] = s;
      if (a.hdr && top >= 0x7f800000u) atomicOr(a.hdr + 2, 1u);
    }
    uint32_t* q = reinterpret_cast<uint32_t*>(a.codes + now * a.pitch);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t v = threadIdx.x + (int64_t)i * blockDim.x;
      float x[N];
      uint32_t c[N / 4];
      Vec<T>::open(cur[i], x);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t b = code_of(FACTOR ? __fmul_rn(x[j], f[i * N + j]) : x[j], s, inv);
        c[j / 4] = j % 4 == 0 ? b : c[j / 4] | (b << (8 * (j % 4)));
      }
      if (v < nvec) {
        if (N == 8) reinterpret_cast<uint2*>(q)[v] = make_uint2(c[0], c[N / 4 - 1]);
        else q[v] = c[0];
      }
    }
  }
}

// Any other row: one CTA per row, read twice.
template <typename T>
__global__ void __launch_bounds__(kThreads) rows_any_kernel(const RowsArgs a) {
  __shared__ uint32_t buf[32];
  clear_part(a.clear, blockIdx.x, gridDim.x);
  const int64_t row = blockIdx.x;
  if (row >= a.R) return;
  const T* x = (const T*)a.P + row * a.K;
  uint32_t top = 0;
  for (int64_t k = threadIdx.x; k < a.K; k += kThreads) {
    const float v = a.f ? __fmul_rn(to_f32(x[k]), a.f[k]) : to_f32(x[k]);
    top = max(top, __float_as_uint(fabsf(v)));
  }
  top = block_max_bits(top, buf);
  const float s = row_scale(top);
  const float inv = reciprocal(s);
  if (threadIdx.x == 0) {
    a.scale[row] = s;
    if (a.hdr && top >= 0x7f800000u) atomicOr(a.hdr + 2, 1u);
  }
  int8_t* q = a.codes + row * a.pitch;
  for (int64_t k = threadIdx.x; k < a.pitch; k += kThreads) {
    uint32_t c = 0;
    if (k < a.K) c = code_of(a.f ? __fmul_rn(to_f32(x[k]), a.f[k]) : to_f32(x[k]), s, inv);
    q[k] = (int8_t)c;
  }
}

template <typename T, int NV>
void rows_go(const RowsArgs& a, unsigned ctas, int threads, cudaStream_t st) {
  if (a.f) rows_kernel<T, NV, true><<<ctas, threads, 0, st>>>(a);
  else rows_kernel<T, NV, false><<<ctas, threads, 0, st>>>(a);
}

// CTAs worth giving to clearing.
unsigned clear_ctas(const Clear& c) {
  const int64_t n = (c.n[0] + c.n[1] + 2047) / 2048;
  return (unsigned)(n < 592 ? n : 592);
}

// Vector rows: up to 512 threads and 8 vectors a thread (fp32 weights of
// 16384 columns, bf16 activations of 32768).  The CTAs are as many as the SMs
// hold at once, each over rows in turn; few rows get extra CTAs for clearing.
template <typename T>
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  const int64_t nvec = a.K / N;
  const unsigned clear = clear_ctas(a.clear);
  if (a.K % 16 == 0 && a.K > 0 && (uintptr_t)a.P % 16 == 0 && (uintptr_t)a.codes % 8 == 0 &&
      nvec <= 8 * 512) {
    int nv = 1;
    while (nv < 4 && nvec > (int64_t)nv * 256) nv *= 2;
    if (nvec > (int64_t)nv * 512) nv = 8;
    const int threads = (int)((nvec + nv - 1) / nv + 31) / 32 * 32;
    const int64_t most = (int64_t)148 * (1536 / threads);
    unsigned ctas = (unsigned)(a.R < most ? a.R : most);
    if (ctas < clear) ctas = clear;
    switch (nv) {
      case 1: rows_go<T, 1>(a, ctas, threads, st); break;
      case 2: rows_go<T, 2>(a, ctas, threads, st); break;
      case 4: rows_go<T, 4>(a, ctas, threads, st); break;
      default: rows_go<T, 8>(a, ctas, threads, st); break;
    }
  } else {
    rows_any_kernel<T><<<(unsigned)(a.R > clear ? a.R : clear), kThreads, 0, st>>>(a);
  }
  count_launch();
  return cudaGetLastError();
}

__global__ void __launch_bounds__(kThreads)
    dequantize_rows_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scale,
                           int64_t O, int64_t I, int64_t pitch, float* __restrict__ out) {
  const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (n >= O * I) return;
  const int64_t o = n / I;
  out[n] = __fmul_rn((float)codes[o * pitch + (n - o * I)], scale[o]);
}

// -------------------------------------------------------------- few tokens

// One dot-product job: out[t, j] = sum_k P[t, k] L(k, j), fp32; optionally
// the rows of P quantized on the way.
struct FewJob {
  const void* P;
  const float* L;   // [r x K], or [K x r] (kr)
  float* out;       // [R x r]
  int64_t K;
  int32_t kr, quantize;
};
struct FewArgs {
  FewJob job[2];    // the second one may be empty (P null)
  int32_t R, r, groups;
  RowsArgs rows;    // of the job that quantizes
};

// Four consecutive factor entries, zeros from `left` on.
__device__ __forceinline__ float4 load4(const float* p, int64_t left, bool wide) {
  if (wide && left >= 4) return __ldg(reinterpret_cast<const float4*>(p));
  float4 v;
  v.x = left > 0 ? __ldg(p) : 0.0f;
  v.y = left > 1 ? __ldg(p + 1) : 0.0f;
  v.z = left > 2 ? __ldg(p + 2) : 0.0f;
  v.w = left > 3 ? __ldg(p + 3) : 0.0f;
  return v;
}

// One CTA takes a token and eight columns of its factor; the one with the
// first eight also quantizes the token.  The rest of the grid clears.  What
// bounds it is latency: one pass over a row and eight factor rows (or eight
// columns), a block reduction, and a second pass for the codes.
template <typename T>
__global__ void __launch_bounds__(512) few_kernel(const FewArgs a) {
  constexpr int V = 4;  // consecutive elements a thread takes
  __shared__ float sums[16][8];
  __shared__ uint32_t buf[32];
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int per = a.R * a.groups, jobs = a.job[1].P ? 2 : 1;
  const int cta = (int)blockIdx.x;
  if (cta >= per * jobs) {
    clear_part(a.rows.clear, cta - per * jobs, (int64_t)gridDim.x - per * jobs);
    return;
  }
  const FewJob& job = a.job[cta / per];
  const int t = (cta % per) / a.groups, j0 = 8 * ((cta % per) % a.groups);
  const int64_t K = job.K;
  const T* x = (const T*)job.P + t * K;
  const bool quantize = job.quantize && j0 == 0;
  const bool xw = K % V == 0 && ((uintptr_t)job.P & (V * sizeof(T) - 1)) == 0;
  const bool lw = ((uintptr_t)job.L & 15) == 0 && (job.kr ? a.r % 4 == 0 : K % 4 == 0);
  const float* f = a.rows.f;
  const bool fw = f && ((uintptr_t)f & 15) == 0;
  const int cols = min(8, a.r - j0);

  auto load_x = [&](int64_t k, float (&v)[V]) {
    if (xw && sizeof(T) == 2) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(x + k));
      v[0] = __uint_as_float(w.x << 16);
      v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16);
      v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else if (xw) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(x + k));
      v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = k + i < K ? to_f32(x[k + i]) : 0.0f;
    }
  };
  auto scaled = [&](int64_t k, const float (&v)[V], float (&y)[V]) {
    if (!f) {
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = v[i];
      return;
    }
    const float4 w = load4(f + k, K - k, fw);
    y[0] = __fmul_rn(v[0], w.x);
    y[1] = __fmul_rn(v[1], w.y);
    y[2] = __fmul_rn(v[2], w.z);
    y[3] = __fmul_rn(v[3], w.w);
  };

  float acc[8] = {};
  uint32_t top = 0;
  for (int64_t k = (int64_t)threadIdx.x * V; k < K; k += 512 * V) {
    float v[V];
    load_x(k, v);
    if (job.kr) {
      float4 l[V][2];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float* p = job.L + (k + i) * a.r + j0;
        const int64_t left = k + i < K ? cols : 0;
        l[i][0] = load4(p, left, lw);
        l[i][1] = load4(p + 4, left - 4, lw);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float m[8] = {l[i][0].x, l[i][0].y, l[i][0].z, l[i][0].w,
                            l[i][1].x, l[i][1].y, l[i][1].z, l[i][1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(v[i], m[j], acc[j]);
      }
    } else {
      float4 l[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        l[j] = load4(job.L + (int64_t)(j0 + j) * K + k, j < cols ? K - k : 0, lw);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        acc[j] = fmaf(v[3], l[j].w, fmaf(v[2], l[j].z, fmaf(v[1], l[j].y, fmaf(v[0], l[j].x, acc[j]))));
    }
    if (quantize) {
      float y[V];
      scaled(k, v, y);
#pragma unroll
      for (int i = 0; i < V; ++i) top = max(top, __float_as_uint(fabsf(y[i])));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[warp][j] = acc[j];
  }
  top = block_max_bits(top, buf);
  if ((int)threadIdx.x < cols) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[w][threadIdx.x];
    job.out[(int64_t)t * a.r + j0 + threadIdx.x] = s;
  }
  if (!quantize) return;
  const float s = row_scale(top);
  const float inv = reciprocal(s);
  if (threadIdx.x == 0) a.rows.scale[t] = s;
  uint32_t* q = reinterpret_cast<uint32_t*>(a.rows.codes + t * a.rows.pitch);
  for (int64_t k = (int64_t)threadIdx.x * V; k < a.rows.pitch; k += 512 * V) {
    uint32_t c = 0;
    if (k < K) {
      float v[V], y[V];
      load_x(k, v);
      scaled(k, v, y);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (k + i < K) c |= code_of(y[i], s, inv) << (8 * i);
    }
    q[k / 4] = c;
  }
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

RowsArgs rows_args(const Int8Call& c, void* ws, Int8Clear header) {
  const int64_t K = c.dx ? c.O : c.I;
  const Layout l = layout(c.R, K);
  RowsArgs a = {};
  a.P = c.P;
  a.R = c.R;
  a.K = K;
  a.pitch = int8_pitch(K);
  a.f = c.dx ? c.wscale : nullptr;
  a.codes = (int8_t*)ws + l.codes;
  a.scale = (float*)((char*)ws + l.scale);
  a.clear.p[0] = (uint4*)header.p;
  a.clear.n[0] = (int64_t)(header.bytes / 16);
  a.clear.p[1] = (uint4*)((char*)ws + l.total);  // the product's sums and tickets
  a.clear.n[1] = (int64_t)(int8_tc_zeroed(c.dx, c.R, c.O, c.I) / 16);
  return a;
}

}  // namespace

cudaError_t launch_int8_quantize(const float* W, int64_t O, int64_t I, int8_t* codes, float* scale,
                                 void* ws, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(ws, 0, kWsHeader, st);
  if (e != cudaSuccess || O == 0) return e;
  RowsArgs a = {};
  a.P = W;
  a.R = O;
  a.K = I;
  a.pitch = int8_pitch(I);
  a.codes = codes;
  a.scale = scale;
  a.hdr = (uint32_t*)ws;
  return launch_rows<float>(a, st);
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

cudaError_t launch_int8_rows(const Int8Call& c, void* ws, Int8Clear header, cudaStream_t st) {
  const RowsArgs a = rows_args(c, ws, header);
  return c.bf16 ? launch_rows<__nv_bfloat16>(a, st) : launch_rows<float>(a, st);
}

cudaError_t launch_int8_product(const Int8Call& c, void* ws, uint32_t* hdr, cudaStream_t st) {
  const Layout l = layout(c.R, c.dx ? c.O : c.I);
  return launch_int8_tc(c, (const int8_t*)ws + l.codes, (const float*)((char*)ws + l.scale), nullptr,
                        (char*)ws + l.total, hdr, st);
}

cudaError_t launch_int8_few(const Int8Call& c, const Int8Few& f, void* ws, Int8Clear header, uint32_t* hdr,
                            cudaStream_t st) {
  FewArgs a = {};
  a.rows = rows_args(c, ws, header);
  a.R = (int32_t)c.R;
  a.r = c.r;
  a.groups = (c.r + 7) / 8;
  a.job[0] = {c.P, f.F, f.T, a.rows.K, c.dx ? 1 : 0, 1};
  if (f.U_new) a.job[1] = {f.X, f.A, f.U_new, c.I, 0, 0};
  const unsigned ctas = (unsigned)(a.R * a.groups * (f.U_new ? 2 : 1)) + clear_ctas(a.rows.clear);
  if (c.bf16) few_kernel<__nv_bfloat16><<<ctas, 512, 0, st>>>(a);
  else few_kernel<float><<<ctas, 512, 0, st>>>(a);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const Layout l = layout(c.R, a.rows.K);
  return launch_int8_tc(c, a.rows.codes, a.rows.scale, &f, (char*)ws + l.total, hdr, st);
}

}  // namespace qlora
