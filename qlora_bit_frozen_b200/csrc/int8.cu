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
#include "int8_dev.cuh"
#include "internal.h"

namespace qlora {
namespace {

using namespace int8;

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

// Code of x: rint(fl(x / s)), by division.
__device__ __forceinline__ uint32_t code_exact(float x, float s) {
  const float q = s > 0.0f ? fminf(fmaxf(__fdiv_rn(x, s), -127.0f), 127.0f) : 0.0f;
  return __float_as_uint(__fadd_rn(q, 12582912.0f));
}

// Reciprocal of the scale; NaN where it is not a normal number.
__device__ __forceinline__ float reciprocal(float s) {
  return s >= 1e-37f ? __fdiv_rn(1.0f, s) : __uint_as_float(0x7fc00000u);
}

// Two fp32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ float lo_of(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi_of(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// max(|a|, |b|, |c|); a NaN wins.
__device__ __forceinline__ float top3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Codes of N values (in pairs), packed.  With M = 1.5 2^23 the sum x inv + M,
// rounded once, is M plus the integer nearest to x inv (ties to even), and its
// low byte is that integer.  x inv is within 127 2^-24 of the quotient and the
// quotient's own rounding within half of that, so the definition's integer is
// another one only where x inv lies within 1.2e-5 of a half; there (3e-5), and
// for scales without a reciprocal, the division is done.  One test serves all
// N: a branch for each of them took 36 issue slots an element, this takes 4.
template <int N>
__device__ __forceinline__ void codes_of(const uint64_t (&x)[N / 2], float s, float inv, uint32_t (&c)[N / 4]) {
  const uint64_t inv2 = pack2(inv, inv), M = pack2(12582912.0f, 12582912.0f), minus = pack2(-1.0f, -1.0f);
  uint32_t t[N];
  float worst = 0.0f;
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    const uint64_t r = fma2(x[j], inv2, M);
    const uint64_t d = fma2(x[j], inv2, fma2(r, minus, M));  // x inv - nearest
    worst = top3(worst, lo_of(d), hi_of(d));
    t[2 * j] = (uint32_t)r;
    t[2 * j + 1] = (uint32_t)(r >> 32);
  }
  if (!(worst < 0.49997f)) {
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = code_exact(j & 1 ? hi_of(x[j / 2]) : lo_of(x[j / 2]), s);
  }
#pragma unroll
  for (int j = 0; j < N; j += 4)
    c[j / 4] = __byte_perm(__byte_perm(t[j], t[j + 1], 0x0040), __byte_perm(t[j + 2], t[j + 3], 0x0040), 0x5410);
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
  int8_t* codes;       // [R x pitch], zeros from K to the next multiple of 16
  float* scale;        // [R]
  uint32_t* bad;       // set where a row has a NaN or Inf, nullable
  Clear clear;
};

// 16 bytes of activations as pairs of floats (8 bf16 or 4 fp32).
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void open(uint4 v, uint64_t (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (uint64_t)(w[i] << 16) | ((uint64_t)(w[i] & 0xffff0000u) << 32);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void open(uint4 v, uint64_t (&x)[2]) {
    x[0] = (uint64_t)v.x | ((uint64_t)v.y << 32);
    x[1] = (uint64_t)v.z | ((uint64_t)v.w << 32);
  }
};

// Largest magnitude of a vector and of `top`; a NaN wins.
template <typename T>
__device__ __forceinline__ float top_of(uint4 v, float top) {
  if (Vec<T>::N == 8) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
    const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
    return top3(top, __uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
  }
  return top3(top3(top, __uint_as_float(v.x), __uint_as_float(v.y)), __uint_as_float(v.z), __uint_as_float(v.w));
}

// Rows that take 16-byte accesses (K a multiple of 16, P aligned): a thread
// keeps its NV vectors of the row in registers between the maximum and the
// codes, so the row is read once, and the next row is on its way while this one
// is reduced.  The column factors of those vectors stay in registers over all
// the rows that the CTA takes (from shared memory they cost more than a third
// of the row's time).  16384 x 5120 in bf16 47 us (252 MB, 5.4 TB/s); 8192 x
// 12288 with factors 74 us (302 MB, 4.1 TB/s): instruction issue, half of all
// slots, and a barrier a row hold it below HBM's rate there.
template <int NV, bool FACTOR>
constexpr int rows_threads() {  // most threads: 64, 85 or 102 registers each
  return !FACTOR || NV == 1 ? 1024 : NV == 2 ? 768 : 640;
}
template <typename T, int NV, bool FACTOR>
__global__ void __launch_bounds__(rows_threads<NV, FACTOR>()) rows_kernel(const RowsArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ uint32_t buf[2][32];
  const int nvec = (int)(a.K / N);
  uint64_t f[FACTOR ? NV * N / 2 : 1];
  if (FACTOR) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float* p = a.f + (int64_t)v * N + 2 * j;
        f[i * (N / 2) + j] = v < nvec ? pack2(__ldg(p), __ldg(p + 1)) : 0;
      }
    }
  }
  auto scaled = [&](uint4 w, int i, uint64_t (&x)[N / 2]) {  // vector i of the thread times its factors
    Vec<T>::open(w, x);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) x[j] = mul2(x[j], f[i * (N / 2) + j]);
  };
  uint4 next[NV];
  auto load = [&](int64_t row) {
    const uint4* x = reinterpret_cast<const uint4*>((const T*)a.P + row * a.K);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      next[i] = v < nvec ? __ldg(x + v) : make_uint4(0, 0, 0, 0);
    }
  };
  int64_t row = blockIdx.x;
  if (row < a.R) load(row);
  clear_part(a.clear, blockIdx.x, gridDim.x);
  for (int k = 0; row < a.R; k ^= 1) {
    uint4 cur[NV];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cur[i] = next[i];
      if (FACTOR) {
        uint64_t x[N / 2];
        scaled(cur[i], i, x);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) top = top3(top, lo_of(x[j]), hi_of(x[j]));
      } else {
        top = top_of<T>(cur[i], top);
      }
    }
    const int64_t now = row;
    row += gridDim.x;
    if (row < a.R) load(row);
    const uint32_t bits = block_max_bits(__float_as_uint(top), buf[k]);
    const float s = row_scale(bits);
    const float inv = reciprocal(s);
    if (threadIdx.x == 0) {
      a.scale[now] = s;
      if (a.bad && bits >= 0x7f800000u) *a.bad = 1;
    }
    uint32_t* q = reinterpret_cast<uint32_t*>(a.codes + now * a.pitch);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        uint32_t c[N / 4];
        uint64_t x[N / 2];
        if (FACTOR) scaled(cur[i], i, x);
        else Vec<T>::open(cur[i], x);
        codes_of<N>(x, s, inv, c);
        if (N == 8) reinterpret_cast<uint2*>(q)[v] = make_uint2(c[0], c[N / 4 - 1]);
        else q[v] = c[0];
      }
    }
  }
}

// Other rows of up to 512 columns: a warp takes a row, 16 values a lane in
// registers.  8747 x 171 in fp32 8 us, a CTA a row 16.  (For longer rows a CTA that
// keeps 16 values a thread took twice the time of reading the row again.)
constexpr int kAny = 16;
template <typename T>
__global__ void __launch_bounds__(kThreads) rows_short_kernel(const RowsArgs a) {
  clear_part(a.clear, blockIdx.x, gridDim.x);
  const int first = threadIdx.x & 31, step = 32;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.R) return;
  const T* p = (const T*)a.P + row * a.K;
  const int K = (int)a.K, end = (int)int8_pitch(a.K);
  uint64_t x[kAny / 2];
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kAny; i += 2) {
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = first + (i + h) * step;
      v[h] = k < K ? to_f32(p[k]) : 0.0f;
      if (a.f && k < K) v[h] = __fmul_rn(v[h], __ldg(a.f + k));
    }
    x[i / 2] = pack2(v[0], v[1]);
    top = top3(top, v[0], v[1]);
  }
  const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  const float s = row_scale(bits);
  if (first == 0) {
    a.scale[row] = s;
    if (a.bad && bits >= 0x7f800000u) *a.bad = 1;
  }
  uint32_t c[kAny / 4];
  codes_of<kAny>(x, s, reciprocal(s), c);
  int8_t* q = a.codes + row * a.pitch;
#pragma unroll
  for (int i = 0; i < kAny; ++i) {
    const int k = first + i * step;
    if (k < end) q[k] = (int8_t)(k < K ? c[i / 4] >> (8 * (i & 3)) : 0);
  }
}

// Longer ones: one CTA per row, read twice.
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
  if (threadIdx.x == 0) {
    a.scale[row] = s;
    if (a.bad && top >= 0x7f800000u) *a.bad = 1;
  }
  int8_t* q = a.codes + row * a.pitch;
  for (int64_t k = threadIdx.x; k < a.pitch; k += kThreads) {
    uint32_t c = 0;
    if (k < a.K) c = code_exact(a.f ? __fmul_rn(to_f32(x[k]), a.f[k]) : to_f32(x[k]), s);
    q[k] = (int8_t)c;
  }
}

// Grid: what the SMs hold at once of this kernel, each CTA over rows in turn
// (more would read the column factors again); few rows get extra CTAs for
// clearing.
template <typename T, int NV, bool FACTOR>
void rows_launch(const RowsArgs& a, unsigned clear, int threads, cudaStream_t st) {
  static const int regs = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, rows_kernel<T, NV, FACTOR>) == cudaSuccess ? (f.numRegs + 7) / 8 * 8 : 64;
  }();
  const int by_regs = 65536 / (regs * threads), by_threads = 2048 / threads;
  const int64_t most = (int64_t)sm_count() * (by_regs < 1 ? 1 : by_regs < by_threads ? by_regs : by_threads);
  unsigned ctas = (unsigned)(a.R < most ? a.R : most);
  if (ctas < clear) ctas = clear;
  rows_kernel<T, NV, FACTOR><<<ctas, threads, 0, st>>>(a);
}
template <typename T, int NV>
void rows_go(const RowsArgs& a, unsigned clear, int threads, cudaStream_t st) {
  if (a.f) rows_launch<T, NV, true>(a, clear, threads, st);
  else rows_launch<T, NV, false>(a, clear, threads, st);
}

// CTAs worth giving to clearing.
unsigned clear_ctas(const Clear& c) {
  const int64_t n = (c.n[0] + c.n[1] + 2047) / 2048;
  return (unsigned)(n < 592 ? n : 592);
}

// Vector rows: up to four vectors a thread (32768 bf16 or 16384 fp32 columns,
// 20480 or 10240 with factors).
template <typename T>
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) {
  const int64_t nvec = a.K / Vec<T>::N;
  const unsigned clear = clear_ctas(a.clear);
  const bool wide = a.K % 16 == 0 && a.K > 0 && (uintptr_t)a.P % 16 == 0 && (uintptr_t)a.codes % 8 == 0;
  if (wide && nvec <= 4 * (a.f ? rows_threads<4, true>() : 1024)) {
    // more vectors a thread, more warps to the SM: two with factors as long as
    // 768 threads reach, else four from 512 vectors on
    const int nv = nvec <= 256 ? 1 : nvec <= (a.f ? 2 * 768 : 512) ? 2 : 4;
    const int threads = (int)((nvec + nv - 1) / nv + 31) / 32 * 32;
    switch (nv) {
      case 1: rows_go<T, 1>(a, clear, threads, st); break;
      case 2: rows_go<T, 2>(a, clear, threads, st); break;
      default: rows_go<T, 4>(a, clear, threads, st); break;
    }
  } else if (a.K <= 32 * kAny) {
    const int64_t ctas = (a.R + kThreads / 32 - 1) / (kThreads / 32);
    rows_short_kernel<T><<<(unsigned)(ctas > clear ? ctas : clear), kThreads, 0, st>>>(a);
  } else {
    rows_any_kernel<T><<<(unsigned)(a.R > clear ? a.R : clear), kThreads, 0, st>>>(a);
  }
  count_launch();
  return cudaGetLastError();
}

// HBM-bound: N codes a thread at a time (four where the rows of the output take
// 16-byte stores), CTA after CTA over the whole matrix.  17408 x 5120: 92 us (one
// code a thread and a 64-bit division each: 266).
template <int N>
__global__ void __launch_bounds__(kThreads)
    dequantize_rows_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scale,
                           int64_t O, int64_t I, int64_t pitch, float* __restrict__ out) {
  const int64_t per = I / N, count = O * per;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < count; e += (int64_t)gridDim.x * kThreads) {
    const int64_t o = count <= UINT32_MAX ? (int64_t)((uint32_t)e / (uint32_t)per) : e / per, k = e - o * per;
    const float s = __ldg(scale + o);
    if (N == 4) {
      const char4 c = __ldcs(reinterpret_cast<const char4*>(codes + o * pitch) + k);
      __stcs(reinterpret_cast<float4*>(out) + e, make_float4(__fmul_rn((float)c.x, s), __fmul_rn((float)c.y, s),
                                                             __fmul_rn((float)c.z, s), __fmul_rn((float)c.w, s)));
    } else {
      out[e] = __fmul_rn((float)codes[o * pitch + k], s);
    }
  }
}

// -------------------------------------------------------------- few tokens

// One dot-product job: out[t, j] = sum_k P[t, k] L(k, j), fp32, for the rows t
// of P, which may be quantized on the way; and / or the values out (or, with P
// null, in) split into three bf16 parts, [3][NP][ld] with the tokens along a
// row, as the column products read them.
struct FewJob {
  const void* P;
  const float* L;   // [r x K], or [K x r] (kr)
  float* out;       // [R x r]
  const float* in;  // [R x r], split only
  uint16_t* parts;  // nullable
  int64_t K;
  int32_t kr, quantize, ctas;
};
struct FewArgs {
  FewJob job[2];
  int32_t R, r, groups, NP;
  int64_t ld;
  RowsArgs rows;    // of the job that quantizes
};

__device__ __forceinline__ void put_parts(const FewArgs& a, uint16_t* parts, int64_t t, int j, float v) {
  // the remainders are exact in fp32
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    parts[((int64_t)q * a.NP + j) * a.ld + t] = __bfloat16_as_ushort(b);
    v -= __bfloat162float(b);
  }
  if (t + 1 == a.R)  // zeros up to the row's end: they meet zero rows of P
    for (int q = 0; q < 3; ++q)
      for (int64_t e = a.R; e < a.ld; ++e) parts[((int64_t)q * a.NP + j) * a.ld + e] = 0;
}

// V elements of a row from k on (16-byte loads of aligned rows, else one by one).
template <typename T, bool WIDE>
__device__ __forceinline__ void few_row(const T* x, int64_t k, int64_t K, float (&v)[8]) {
  if (WIDE && sizeof(T) == 2) {
    if (k < K) {
      uint64_t w[4];
      Vec<__nv_bfloat16>::open(__ldg(reinterpret_cast<const uint4*>(x + k)), w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = lo_of(w[i]);
        v[2 * i + 1] = hi_of(w[i]);
      }
    }
  } else if (WIDE) {
    if (k < K) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(x + k));
      const float4 b = __ldg(reinterpret_cast<const float4*>(x + k) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) v[i] = to_f32(x[k + i]);
  }
}

// TOK tokens and eight columns of their factor per CTA; with one token the CTA
// of the first eight columns also quantizes it.  In a wide call K is a multiple
// of 8 (and, for factors [K x r], r of 4) and everything is 16-byte aligned.  A
// factor [r x K] is read eight elements a thread, a factor [K x r] one row a
// thread (eight rows in flight), so that either way neighbouring threads read
// neighbouring bytes.
template <typename T, bool KR, bool WIDE, int TOK>
__device__ __forceinline__ void few_tokens(const FewArgs& a, const FewJob& job, int t0, int j0,
                                           float (*sums)[8 * TOK], uint32_t* buf) {
  const int64_t K = job.K;
  const T* x = (const T*)job.P + t0 * K;
  const bool quantize = TOK == 1 && job.quantize && j0 == 0;
  const float* f = a.rows.f;
  const int cols = min(8, a.r - j0), toks = TOK == 1 ? 1 : min(TOK, a.R - t0), threads = (int)blockDim.x;
  float acc[TOK][8] = {};
  uint32_t top = 0;
  for (int64_t base = 0; base < K; base += threads * 8) {
    float v[TOK][8] = {};
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      if (t >= toks) continue;
      if (KR) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t k = base + threads * i + threadIdx.x;
          if (k < K) v[t][i] = to_f32(x[t * K + k]);
        }
      } else {
        few_row<T, WIDE>(x + t * K, base + (int64_t)threadIdx.x * 8, K, v[t]);
      }
    }
    // Row q of the factor's block: its row j0 + q of [r x K], or row k of [K x r].
    auto factor = [&](int q, float (&l)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) l[i] = 0.0f;
      if (KR) {
        const int64_t k = base + threads * q + threadIdx.x;
        if (k >= K) return;
        const float* p = job.L + k * a.r + j0;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          if (WIDE) {
            if (j < cols) {
              const float4 w = __ldg(reinterpret_cast<const float4*>(p + j));
              l[j] = w.x; l[j + 1] = w.y; l[j + 2] = w.z; l[j + 3] = w.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (j + i < cols) l[j + i] = __ldg(p + j + i);
          }
        }
      } else if (q < cols) {
        few_row<float, WIDE>(job.L + (int64_t)(j0 + q) * K, base + (int64_t)threadIdx.x * 8, K, l);
      }
    };
    if constexpr (TOK == 1) {
      // All of it on its way before the first product; this loop nest is what the
      // compiler keeps in that order (16 loads a thread in flight).
      float l[8][8];
#pragma unroll
      for (int q = 0; q < 8; ++q) factor(q, l[q]);
      if (KR) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[0][j] = fmaf(v[0][q], l[q][j], acc[0][j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[0][j] = fmaf(v[0][i], l[j][i], acc[0][j]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float l[8];
        factor(q, l);
#pragma unroll
        for (int t = 0; t < TOK; ++t)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (KR) acc[t][i] = fmaf(v[t][q], l[i], acc[t][i]);
            else acc[t][q] = fmaf(v[t][i], l[i], acc[t][q]);
          }
      }
    }
    if (quantize) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t k = KR ? base + threads * i + threadIdx.x : base + (int64_t)threadIdx.x * 8 + i;
        float y = v[0][i];
        if (f && k < K) y = __fmul_rn(y, __ldg(f + k));
        top = max(top, __float_as_uint(fabsf(y)));
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TOK; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[t][j] += __shfl_xor_sync(0xffffffffu, acc[t][j], o);
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int t = 0; t < TOK; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[threadIdx.x >> 5][8 * t + j] = acc[t][j];
  }
  top = block_max_bits(top, buf);
  if ((int)threadIdx.x < 8 * toks && (int)(threadIdx.x & 7) < cols) {
    float s = 0.0f;
    for (int w = 0; w < threads / 32; ++w) s += sums[w][threadIdx.x];
    const int64_t t = t0 + (threadIdx.x >> 3);
    const int j = j0 + (threadIdx.x & 7);
    job.out[t * a.r + j] = s;
    if (job.parts) put_parts(a, job.parts, t, j, s);
  }
  if (!quantize) return;
  const float s = row_scale(top);
  const float inv = reciprocal(s);
  if (threadIdx.x == 0) a.rows.scale[t0] = s;
  uint2* q = reinterpret_cast<uint2*>(a.rows.codes + t0 * a.rows.pitch);
  for (int64_t k = (int64_t)threadIdx.x * 8; k < a.rows.pitch; k += threads * 8) {
    float v[8] = {};
    uint32_t c[2];
    few_row<T, WIDE>(x, k, K, v);  // zeros past the row, whose code is 0
    if (f) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) v[i] = __fmul_rn(v[i], __ldg(f + k + i));
    }
    uint64_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = pack2(v[2 * i], v[2 * i + 1]);
    codes_of<8>(y, s, inv, c);
    q[k / 8] = make_uint2(c[0], c[1]);
  }
}

// One token a CTA: latency is what bounds it, a pass over a row beside eight
// factor rows (or columns), a block reduction, and a second pass for the codes.
// One token of 4096 columns, rank 8: 4.6 us.  Four tokens a CTA (fp32 or
// unaligned activations by themselves): a quarter of the factor's reads from L2,
// which are what bounds that (747 tokens of 13568 columns in fp32: 28 us).  The
// last CTAs of the grid clear.
template <typename T, bool WIDE, int TOK>
__global__ void __launch_bounds__(512) few_kernel(const FewArgs a) {
  __shared__ float sums[16][8 * TOK];
  __shared__ uint32_t buf[32];
  if (threadIdx.x == 0) griddep_launch_dependents();
  int cta = (int)blockIdx.x;
  for (int k = 0; k < 2; ++k) {
    const FewJob& job = a.job[k];
    if (cta >= job.ctas) {
      cta -= job.ctas;
      continue;
    }
    if (!job.P) {
      const int64_t n = (int64_t)a.R * a.r;
      for (int64_t e = (int64_t)cta * blockDim.x + threadIdx.x; e < n; e += (int64_t)job.ctas * blockDim.x)
        put_parts(a, job.parts, e / a.r, (int)(e % a.r), __ldg(job.in + e));
      return;
    }
    const int t0 = TOK * (cta / a.groups), j0 = 8 * (cta % a.groups);
    if (job.kr) few_tokens<T, true, WIDE, TOK>(a, job, t0, j0, sums, buf);
    else few_tokens<T, false, WIDE, TOK>(a, job, t0, j0, sums, buf);
    return;
  }
  const int used = a.job[0].ctas + a.job[1].ctas;
  clear_part(a.rows.clear, cta, (int64_t)gridDim.x - used);
}

// The jobs of `a` (R, r and the jobs' matrices filled in), `extra` CTAs for
// clearing.
template <int TOK>
cudaError_t few_go(FewArgs& a, bool bf16, unsigned extra, cudaStream_t st) {
  a.groups = (a.r + 7) / 8;
  bool wide = true;
  int64_t K = 0;
  for (FewJob& job : a.job) {
    if (!job.P) continue;
    if (a.r == 1) job.kr = 0;  // the same bytes
    job.ctas = (a.R + TOK - 1) / TOK * a.groups;
    if (job.K > K) K = job.K;
    if (job.K % 8 != 0 || (uintptr_t)job.P % 16 != 0 || (uintptr_t)job.L % 16 != 0 || (job.kr && a.r % 4 != 0))
      wide = false;
  }
  int threads = (int)((K + 255) / 256) * 32;
  threads = threads < 128 ? 128 : threads > 512 ? 512 : threads;
  const unsigned ctas = (unsigned)(a.job[0].ctas + a.job[1].ctas) + extra;
  if (ctas == 0) return cudaSuccess;
  if (bf16) {
    if (wide) few_kernel<__nv_bfloat16, true, TOK><<<ctas, threads, 0, st>>>(a);
    else few_kernel<__nv_bfloat16, false, TOK><<<ctas, threads, 0, st>>>(a);
  } else {
    if (wide) few_kernel<float, true, TOK><<<ctas, threads, 0, st>>>(a);
    else few_kernel<float, false, TOK><<<ctas, threads, 0, st>>>(a);
  }
  count_launch();
  return cudaGetLastError();
}

struct Layout {
  size_t scale, codes, total;
};
Layout layout(int64_t R, int64_t K) {
  Layout l;
  l.scale = 0;
  l.codes = align_up((size_t)R * 4, 256);
  l.total = l.codes + align_up((size_t)R * (size_t)int8_act_pitch(K), 256);
  return l;
}

RowsArgs rows_args(const Int8Call& c, void* ws, Int8Clear header) {
  const int64_t K = c.dx ? c.O : c.I;
  const Layout l = layout(c.R, K);
  RowsArgs a = {};
  a.P = c.P;
  a.R = c.R;
  a.K = K;
  a.pitch = int8_act_pitch(K);
  a.f = c.dx ? c.wscale : nullptr;
  a.codes = (int8_t*)ws + l.codes;
  a.scale = (float*)((char*)ws + l.scale);
  a.clear.p[0] = (uint4*)header.p;
  a.clear.n[0] = (int64_t)(header.bytes / 16);
  a.clear.p[1] = (uint4*)((char*)ws + l.total);  // the product's sums and tickets
  a.clear.n[1] = (int64_t)(int8_tc_zeroed(c.dx, c.R, c.O, c.I, c.r) / 16);
  return a;
}

}  // namespace

cudaError_t launch_int8_quantize(const float* W, int64_t O, int64_t I, int8_t* codes, float* scale,
                                 uint32_t* bad, cudaStream_t st) {
  if (O == 0) return cudaSuccess;
  RowsArgs a = {};
  a.P = W;
  a.R = O;
  a.K = I;
  a.pitch = int8_pitch(I);
  a.codes = codes;
  a.scale = scale;
  a.bad = bad;
  return launch_rows<float>(a, st);
}

cudaError_t launch_int8_dequantize(const int8_t* codes, const float* scale, int64_t O, int64_t I,
                                   float* out, cudaStream_t st) {
  if (O * I == 0) return cudaSuccess;
  const bool wide = I % 4 == 0 && (uintptr_t)out % 16 == 0 && (uintptr_t)codes % 4 == 0;
  const int64_t need = (O * I / (wide ? 4 : 1) + kThreads - 1) / kThreads, most = (int64_t)sm_count() * 32;
  const unsigned ctas = (unsigned)(need < most ? need : most);
  if (wide) dequantize_rows_kernel<4><<<ctas, kThreads, 0, st>>>(codes, scale, O, I, int8_pitch(I), out);
  else dequantize_rows_kernel<1><<<ctas, kThreads, 0, st>>>(codes, scale, O, I, int8_pitch(I), out);
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

cudaError_t launch_int8_product(const Int8Call& c, void* ws, uint32_t* hdr, const Int8Few* few,
                                cudaStream_t st) {
  const Layout l = layout(c.R, c.dx ? c.O : c.I);
  return launch_int8_tc(c, (const int8_t*)ws + l.codes, (const float*)((char*)ws + l.scale), few,
                        (char*)ws + l.total, hdr, st);
}

bool int8_few_applies(int64_t R, int64_t K, int32_t r) {
  // every CTA reads eight factor rows from L2: up to 48 MB, about what the
  // separate launches cost in latency
  return R <= kInt8Few || R * ((r + 7) / 8) * K <= (int64_t)48 * 1024 * 1024 / 32;
}

cudaError_t launch_int8_few(const Int8Call& c, const Int8Few& f, void* ws, Int8Clear header,
                            cudaStream_t st) {
  FewArgs a = {};
  a.rows = rows_args(c, ws, header);
  a.R = (int32_t)c.R;
  a.r = c.r;
  a.NP = f.NP;
  a.ld = f.ld;
  if (f.T) a.job[0] = {c.P, f.F, f.T, nullptr, f.T_parts, a.rows.K, c.dx ? 1 : 0, c.out ? 1 : 0, 0};
  if (f.U_new) a.job[1] = {f.X, f.A, f.U_new, nullptr, f.U_parts, c.I, 0, 0, 0};
  else if (f.U_parts)
    a.job[1] = {nullptr, nullptr, nullptr, f.U, f.U_parts, 0, 0, 0, (int32_t)((c.R * c.r + 4095) / 4096)};
  return few_go<1>(a, c.bf16, clear_ctas(a.rows.clear), st);
}

cudaError_t launch_int8_dots(const Int8Dot* d, int count, bool bf16, int64_t R, int32_t r, cudaStream_t st) {
  FewArgs a = {};
  a.R = (int32_t)R;
  a.r = r;
  for (int i = 0; i < count; ++i) a.job[i] = {d[i].P, d[i].L, d[i].out, nullptr, nullptr, d[i].K, d[i].kr ? 1 : 0, 0, 0};
  return few_go<4>(a, bf16, 0, st);
}

}  // namespace qlora
