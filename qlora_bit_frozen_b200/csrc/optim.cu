// optim.cu -- one training step's optimizer work over many tensors at once:
// the global gradient norm and AdamW with states in 32 or in 8 bits
// ("QLoRA Fine-Tuning", "Training lifecycle": only the LoRA factors are
// optimizer inputs; a model has two small factors for every adapted linear,
// so hundreds of tensors, each far too small to fill the GPU alone).
//
// The tensors' descriptors travel as kernel parameters (no device table, no
// copy, and a captured graph holds them).  The 256-value blocks of all
// tensors are dealt out to the CTAs in equal contiguous runs; a warp finds
// the tensor of its first block by bisection over the descriptors' first
// blocks and walks on from there.
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = QLORA_STATE_BLOCK;  // values per warp and per 8-bit scale

struct Desc {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  uint32_t first;  // first block of this tensor in the launch
  uint8_t pbf16, gbf16, vec, pad;
};

// Descriptors of one launch.  A kernel takes up to 32764 bytes of
// parameters; a launch of few tensors takes the smaller form, whose
// parameters cost less to copy.
template <int CAP>
struct Batch {
  int32_t count;
  uint32_t blocks;
  Desc d[CAP];
};
constexpr int kFew = 60;    // below 4 KB of parameters
constexpr int kSome = 125;  // 8 KB
constexpr int kMany = 500;
static_assert(sizeof(Batch<kMany>) + 128 <= 32764, "kernel parameter limit");

template <int CAP>
__device__ __forceinline__ int find(const Batch<CAP>& b, uint32_t blk) {
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.d[mid].first <= blk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The run of blocks of this CTA, which its warps take in turn.
struct Run {
  uint32_t lo, hi;
};
__device__ __forceinline__ Run my_run(uint32_t blocks) {
  return {(uint32_t)((uint64_t)blocks * blockIdx.x / gridDim.x),
          (uint32_t)((uint64_t)blocks * (blockIdx.x + 1) / gridDim.x)};
}

// A lane's eight values of a block: two runs of four where the arrays take
// vector accesses, else every 32nd value.
template <bool VEC>
__device__ __forceinline__ int place(int lane, int j) {
  return VEC ? (j >> 2) * 128 + 4 * lane + (j & 3) : lane + 32 * j;
}

template <bool VEC>
__device__ __forceinline__ void load_f32(const float* a, int lane, int left, float (&x)[8]) {
  if (VEC && left >= kBlock) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 t = __ldcs(reinterpret_cast<const float4*>(a) + 32 * h + lane);
      x[4 * h] = t.x; x[4 * h + 1] = t.y; x[4 * h + 2] = t.z; x[4 * h + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = place<VEC>(lane, j) < left ? a[place<VEC>(lane, j)] : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void load_bf16(const uint16_t* a, int lane, int left, float (&x)[8]) {
  if (VEC && left >= kBlock) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint2 t = __ldcs(reinterpret_cast<const uint2*>(a) + 32 * h + lane);
      x[4 * h] = __uint_as_float(t.x << 16);
      x[4 * h + 1] = __uint_as_float(t.x & 0xffff0000u);
      x[4 * h + 2] = __uint_as_float(t.y << 16);
      x[4 * h + 3] = __uint_as_float(t.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = place<VEC>(lane, j) < left ? bf16_bits_to_float(a[place<VEC>(lane, j)]) : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void load_any(const void* a, bool bf16, int64_t at, int lane, int left,
                                         float (&x)[8]) {
  if (bf16) load_bf16<VEC>((const uint16_t*)a + at, lane, left, x);
  else load_f32<VEC>((const float*)a + at, lane, left, x);
}

template <bool VEC>
__device__ __forceinline__ void store_f32(float* a, int lane, int left, const float (&x)[8]) {
  if (VEC && left >= kBlock) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      reinterpret_cast<float4*>(a)[32 * h + lane] =
          make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (place<VEC>(lane, j) < left) a[place<VEC>(lane, j)] = x[j];
  }
}

template <bool VEC>
__device__ __forceinline__ void store_any(void* a, bool bf16, int64_t at, int lane, int left,
                                          const float (&x)[8]) {
  if (!bf16) {
    store_f32<VEC>((float*)a + at, lane, left, x);
    return;
  }
  uint16_t* o = (uint16_t*)a + at;
  if (VEC && left >= kBlock) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      reinterpret_cast<uint2*>(o)[32 * h + lane] =
          make_uint2(pack_bf16x2(x[4 * h], x[4 * h + 1]), pack_bf16x2(x[4 * h + 2], x[4 * h + 3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (place<VEC>(lane, j) < left)
        o[place<VEC>(lane, j)] = (uint16_t)(pack_bf16x2(x[j], 0.0f) & 0xffffu);
  }
}

// Eight code bytes of a lane, byte j of the pair of words = code of value j.
template <bool VEC>
__device__ __forceinline__ void load_codes(const uint8_t* a, int lane, int left, uint32_t (&w)[2]) {
  if (VEC && left >= kBlock) {
    w[0] = __ldcs(reinterpret_cast<const uint32_t*>(a) + lane);
    w[1] = __ldcs(reinterpret_cast<const uint32_t*>(a) + 32 + lane);
  } else {
    w[0] = w[1] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (place<VEC>(lane, j) < left)
        w[j >> 2] |= (uint32_t)a[place<VEC>(lane, j)] << (8 * (j & 3));
  }
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* a, int lane, int left, const uint32_t (&w)[2]) {
  if (VEC && left >= kBlock) {
    reinterpret_cast<uint32_t*>(a)[lane] = w[0];
    reinterpret_cast<uint32_t*>(a)[32 + lane] = w[1];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (place<VEC>(lane, j) < left)
        a[place<VEC>(lane, j)] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
}

// ------------------------------------------------------------------ AdamW

struct AdamWArgs {
  float b1, b2, omb1, omb2, eps, decay;
  float step_size, inv_rbc2;  // lr / bc1, 1 / sqrt(bc2) (when control is null)
  double lr, b1d, b2d;
  const qlora_step_control* control;
  float z;           // -0
  int32_t follows;  // launched over the end of the call's launch before
};

// b^t by squaring: the same 64-bit products on the host and on the device.
__host__ __device__ inline double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

__host__ __device__ inline void bias_terms(double lr, double b1, double b2, int64_t t, float* step_size,
                                           float* inv_rbc2) {
  *step_size = (float)(lr / (1.0 - power(b1, t)));
  *inv_rbc2 = (float)(1.0 / sqrt(1.0 - power(b2, t)));
}

__device__ __forceinline__ float inverse_of(float scale) {
  return scale < 1.17549435e-38f ? 0.0f : __fdiv_rn(1.0f, scale);  // NaN stays NaN
}

// Largest of non-negative values by their bits, so that a NaN wins.
__device__ __forceinline__ float warp_max_bits(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// Two fp32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ uint64_t twice(float x) { return pair(x, x); }
__device__ __forceinline__ float lo_of(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi_of(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// A product that an addition follows, as a fused multiply-add of z = -0 (which
// leaves it and its sign as they are): a packed multiply and add were compiled
// to one rounding, also with a constant for z, so z is an argument of the kernel.
__device__ __forceinline__ uint64_t prod2(uint64_t a, float b, float z) { return fma2(a, twice(b), twice(z)); }
__device__ __forceinline__ uint64_t abs2(uint64_t a) { return a & 0x7fffffff7fffffffull; }
// max(|a|, |b|, |c|); a NaN wins.
__device__ __forceinline__ float top3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float root_approx(float u) {
  float a;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(u));
  return a;
}

// Bytes 2 h and 2 h + 1 of w as floats, exactly: a byte becomes the low
// mantissa bits of 2^23, which bias (2^23, and 128 more for signed bytes with
// their top bit flipped) takes off again.
__device__ __forceinline__ uint64_t bytes_f32(uint32_t w, int h, float bias) {
  return add2(pair(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | (uint32_t)(2 * h))),
                   __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | (uint32_t)(2 * h + 1)))),
              twice(-bias));
}

// rint(top x) for |x| <= 1 (a little above by rounding) in the low bytes of the
// sums with M = 1.5 2^23 (nearest, ties to even; two's complement), and how far
// top x is from that integer at most.
__device__ __forceinline__ uint64_t rounded(uint64_t x, float top, float& worst) {
  const uint64_t M = twice(12582912.0f), t2 = twice(top);
  const uint64_t r = fma2(x, t2, M);
  const uint64_t d = fma2(x, t2, fma2(r, twice(-1.0f), M));
  worst = top3(worst, lo_of(d), hi_of(d));
  return r;
}
// The same for one value by the definition: the root and the product each
// rounded to nearest.
__device__ __forceinline__ float rounded_exact(float u, float top) {
  return __fadd_rn(__fmul_rn(__fsqrt_rn(u), top), 12582912.0f);
}

// Four low bytes to a word.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// One block.  Bound by HBM with 32-bit states; with 8-bit ones (16 bytes a value)
// nothing is full, 68% of the issue slots and half of HBM's rate: a warp has one
// block on its way at a time, so arithmetic and memory take turns.  All but the
// division and the root work on pairs, and the codes' roots are the approximate ones: their
// products are within 255 (2^-22 + 2^-24) of the definition's, so they round to
// the same integer unless within 1e-4 of a half; only then (2e-4, one test for
// the lane's eight values) are the exact roots taken.  64 M values, fp32 parameters
// and gradients, 8-bit states: 224 us (1.03 GB, 4.6 TB/s); 1.1 M values with 32-bit
// states 6.8 us.
template <int BITS, bool VEC>
__device__ __forceinline__ void adamw_block(const Desc& d, int64_t blk, int lane, const AdamWArgs& a,
                                            float scale, float step_size, float inv_rbc2) {
  const int64_t at = blk * kBlock;
  const int left = d.n - at < kBlock ? (int)(d.n - at) : kBlock;
  float g[8], p[8], mf[8], vf[8];
  uint32_t mw[2], vw[2];
  float ms = 0.0f, vs = 0.0f;
  load_any<VEC>(d.g, d.gbf16, at, lane, left, g);
  load_any<VEC>(d.p, d.pbf16, at, lane, left, p);
  if constexpr (BITS == 32) {
    load_f32<VEC>((const float*)d.m + at, lane, left, mf);
    load_f32<VEC>((const float*)d.v + at, lane, left, vf);
  } else {
    load_codes<VEC>((const uint8_t*)d.m + at, lane, left, mw);
    load_codes<VEC>((const uint8_t*)d.v + at, lane, left, vw);
    ms = d.ms[blk];
    vs = d.vs[blk];
  }
  uint64_t m[4], r[4];
  float mtop = 0.0f, rtop = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint64_t v;
    if constexpr (BITS == 32) {
      m[j] = pair(mf[2 * j], mf[2 * j + 1]);
      v = pair(vf[2 * j], vf[2 * j + 1]);
    } else {
      const uint64_t km = mul2(bytes_f32(mw[j >> 1] ^ 0x80808080u, j & 1, 8388736.0f), twice(1.0f / 127.0f));
      const uint64_t kv = mul2(bytes_f32(vw[j >> 1], j & 1, 8388608.0f), twice(1.0f / 255.0f));
      m[j] = mul2(mul2(km, abs2(km)), twice(ms));
      const uint64_t root = mul2(mul2(kv, kv), twice(vs));
      v = mul2(root, root);
    }
    const uint64_t gs = mul2(pair(g[2 * j], g[2 * j + 1]), twice(scale));
    m[j] = add2(prod2(m[j], a.b1, a.z), prod2(gs, a.omb1, a.z));
    v = add2(prod2(v, a.b2, a.z), prod2(mul2(gs, gs), a.omb2, a.z));
    r[j] = pair(__fsqrt_rn(lo_of(v)), __fsqrt_rn(hi_of(v)));
    const uint64_t num = mul2(m[j], twice(step_size));
    const uint64_t den = add2(prod2(r[j], inv_rbc2, a.z), twice(a.eps));
    const uint64_t step = pair(__fdiv_rn(lo_of(num), lo_of(den)), __fdiv_rn(hi_of(num), hi_of(den)));
    const uint64_t pn = add2(prod2(pair(p[2 * j], p[2 * j + 1]), a.decay, a.z), step ^ 0x8000000080000000ull);
    p[2 * j] = lo_of(pn);
    p[2 * j + 1] = hi_of(pn);
    if constexpr (BITS == 32) {
      mf[2 * j] = lo_of(m[j]);
      mf[2 * j + 1] = hi_of(m[j]);
      vf[2 * j] = lo_of(v);
      vf[2 * j + 1] = hi_of(v);
    } else {
      mtop = top3(mtop, lo_of(m[j]), hi_of(m[j]));
      rtop = top3(rtop, lo_of(r[j]), hi_of(r[j]));
    }
  }
  store_any<VEC>(d.p, d.pbf16, at, lane, left, p);
  if constexpr (BITS == 32) {
    store_f32<VEC>((float*)d.m + at, lane, left, mf);
    store_f32<VEC>((float*)d.v + at, lane, left, vf);
  } else {
    mtop = warp_max_bits(mtop);
    rtop = warp_max_bits(rtop);
    const float im = inverse_of(mtop), iv = inverse_of(rtop);
    const float least = iv > 0.0f ? 1.0f / 255.0f : 0.0f;  // code 1
    uint64_t km[4], kv[4];
    float worst = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t um = mul2(abs2(m[j]), twice(im)), uv = mul2(r[j], twice(iv));
      km[j] = rounded(pair(copysignf(root_approx(lo_of(um)), lo_of(m[j])),
                           copysignf(root_approx(hi_of(um)), hi_of(m[j]))), 127.0f, worst);
      kv[j] = rounded(pair(fmaxf(root_approx(lo_of(uv)), lo_of(r[j]) > 0.0f ? least : 0.0f),
                           fmaxf(root_approx(hi_of(uv)), hi_of(r[j]) > 0.0f ? least : 0.0f)), 255.0f, worst);
    }
    uint32_t cm[8], cv[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cm[2 * j] = (uint32_t)km[j];
      cm[2 * j + 1] = (uint32_t)(km[j] >> 32);
      cv[2 * j] = (uint32_t)kv[j];
      cv[2 * j + 1] = (uint32_t)(kv[j] >> 32);
    }
    if (!(worst < 0.4998f)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float mj = j & 1 ? hi_of(m[j >> 1]) : lo_of(m[j >> 1]);
        const float rj = j & 1 ? hi_of(r[j >> 1]) : lo_of(r[j >> 1]);
        const uint32_t k = __float_as_uint(rounded_exact(__fmul_rn(fabsf(mj), im), 127.0f)) & 255u;
        const uint32_t u = __float_as_uint(rounded_exact(__fmul_rn(rj, iv), 255.0f)) & 255u;
        cm[j] = mj < 0.0f ? 0u - k : k;
        cv[j] = rj > 0.0f && iv > 0.0f ? max(u, 1u) : u;
      }
    }
    const uint32_t wm[2] = {pack4(cm[0], cm[1], cm[2], cm[3]), pack4(cm[4], cm[5], cm[6], cm[7])};
    const uint32_t wv[2] = {pack4(cv[0], cv[1], cv[2], cv[3]), pack4(cv[4], cv[5], cv[6], cv[7])};
    store_codes<VEC>((uint8_t*)d.m + at, lane, left, wm);
    store_codes<VEC>((uint8_t*)d.v + at, lane, left, wv);
    if (lane == 0) {
      d.ms[blk] = mtop;
      d.vs[blk] = rtop;
    }
  }
}

template <int BITS, int CAP>
__global__ void __launch_bounds__(kThreads, 4)
    adamw_kernel(const __grid_constant__ Batch<CAP> b, const AdamWArgs a) {
  __shared__ float terms[2];
  // The launches of one call share nothing: the next one may start as this one
  // runs out of work, and ends only after it.
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  float scale = 1.0f, step_size = a.step_size, inv_rbc2 = a.inv_rbc2;
  if (a.control) {
    if (a.control->skip || a.control->step < 1) {
      if (a.follows && threadIdx.x == 0) griddep_wait();
      return;
    }
    scale = a.control->scale;
    if (threadIdx.x == 0) bias_terms(a.lr, a.b1d, a.b2d, a.control->step, &terms[0], &terms[1]);
    __syncthreads();
    step_size = terms[0];
    inv_rbc2 = terms[1];
  }
  const Run run = my_run(b.blocks);
  uint32_t blk = run.lo + (threadIdx.x >> 5);
  int i = blk < run.hi ? find(b, blk) : 0;
  for (; blk < run.hi; blk += kThreads / 32) {
    while (i + 1 < b.count && b.d[i + 1].first <= blk) ++i;
    const Desc& d = b.d[i];
    if (d.vec) adamw_block<BITS, true>(d, blk - d.first, lane, a, scale, step_size, inv_rbc2);
    else adamw_block<BITS, false>(d, blk - d.first, lane, a, scale, step_size, inv_rbc2);
  }
  if (a.follows && threadIdx.x == 0) griddep_wait();
}

// ------------------------------------------------------------------- norm

// Each CTA adds the squares of its blocks in 64 bits and leaves one sum.  64 M
// fp32 values: 51 us with the launch after it (257 MB, 5.0 TB/s).
template <int CAP>
__global__ void __launch_bounds__(kThreads)
    sumsq_kernel(const __grid_constant__ Batch<CAP> b, double* __restrict__ part) {
  __shared__ double sums[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) griddep_launch_dependents();  // the norm kernel waits for this grid
  const Run run = my_run(b.blocks);
  uint32_t blk = run.lo + warp;
  int i = blk < run.hi ? find(b, blk) : 0;
  double acc = 0.0;
  // four blocks on their way at a time
  while (blk < run.hi) {
    float g[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[k][j] = 0.0f;
      if (blk < run.hi) {
        while (i + 1 < b.count && b.d[i + 1].first <= blk) ++i;
        const Desc& d = b.d[i];
        const int64_t at = (int64_t)(blk - d.first) * kBlock;
        const int left = d.n - at < kBlock ? (int)(d.n - at) : kBlock;
        if (d.vec) load_any<true>(d.g, d.gbf16, at, lane, left, g[k]);
        else load_any<false>(d.g, d.gbf16, at, lane, left, g[k]);
      }
      blk += kThreads / 32;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc = fma((double)g[k][j], (double)g[k][j], acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) sums[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += sums[w];
    part[blockIdx.x] = s;
  }
}

__global__ void __launch_bounds__(kThreads)
    norm_kernel(const double* __restrict__ part, int32_t n, float max_norm, qlora_step_control* c) {
  __shared__ double sums[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) sums[warp] = acc;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double s = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) s += sums[w];
  const float norm = (float)sqrt(s);
  const bool ok = isfinite(norm);
  c->norm = norm;
  c->scale = (ok && max_norm > 0.0f && norm > max_norm) ? __fdiv_rn(max_norm, norm) : 1.0f;
  c->skip = ok ? 0 : 1;
  c->step += ok ? 1 : 0;
}

// ------------------------------------------------------------------- host

bool on(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int sm_count() {
  static std::atomic<int> count[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    count[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

constexpr int kCtasPerSm = 4;  // one wave at up to 64 registers a thread

// Fills the batch with the tensors from `i` on that fit one launch; returns
// where the next one begins.
template <int CAP>
int32_t fill(Batch<CAP>& b, const qlora_tensor* t, int32_t count, int32_t i, int bits, bool grads_only) {
  b.count = 0;
  uint64_t blocks = 0;
  for (; i < count && b.count < CAP; ++i) {
    if (t[i].n == 0) continue;
    const uint64_t nb = (uint64_t)(t[i].n + kBlock - 1) / kBlock;
    if (b.count > 0 && blocks + nb > 0x7fffffffull) break;
    Desc& d = b.d[b.count++];
    d.p = t[i].param;
    d.g = t[i].grad;
    d.m = t[i].m;
    d.v = t[i].v;
    d.ms = t[i].m_scale;
    d.vs = t[i].v_scale;
    d.n = t[i].n;
    d.first = (uint32_t)blocks;
    d.pbf16 = t[i].param_type == QLORA_DTYPE_BF16;
    d.gbf16 = t[i].grad_type == QLORA_DTYPE_BF16;
    d.vec = on(d.g, d.gbf16 ? 8 : 16) &&
            (grads_only || (on(d.p, d.pbf16 ? 8 : 16) && on(d.m, bits == 8 ? 4 : 16) &&
                            on(d.v, bits == 8 ? 4 : 16)));
    d.pad = 0;
    blocks += nb;
  }
  b.blocks = (uint32_t)blocks;
  return i;
}

unsigned ctas_for(uint32_t blocks, int sms) {
  const uint32_t need = (blocks + kThreads / 32 - 1) / (kThreads / 32);
  const uint32_t most = (uint32_t)(sms * kCtasPerSm);
  return need < most ? need : most;
}

template <int CAP>
cudaError_t adamw_all(const qlora_tensor* t, int32_t count, int32_t bits, AdamWArgs a, cudaStream_t st) {
  const int sms = sm_count();
  a.follows = 0;
  for (int32_t i = 0; i < count;) {
    Batch<CAP> b;
    i = fill(b, t, count, i, bits, false);
    if (b.count == 0) break;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas_for(b.blocks, sms));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.follows ? 1 : 0;
    const cudaError_t e = bits == 8 ? cudaLaunchKernelEx(&cfg, adamw_kernel<8, CAP>, b, a)
                                    : cudaLaunchKernelEx(&cfg, adamw_kernel<32, CAP>, b, a);
    count_launch();
    if (e != cudaSuccess) return e;
    a.follows = 1;
  }
  return cudaGetLastError();
}

template <int CAP>
cudaError_t sumsq_all(const qlora_tensor* t, int32_t count, double* part, int32_t* n, cudaStream_t st) {
  const int sms = sm_count();
  *n = 0;
  for (int32_t i = 0; i < count;) {
    Batch<CAP> b;
    i = fill(b, t, count, i, 32, true);
    if (b.count == 0) break;
    const unsigned ctas = ctas_for(b.blocks, sms);
    sumsq_kernel<CAP><<<ctas, kThreads, 0, st>>>(b, part + *n);
    count_launch();
    *n += (int32_t)ctas;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_norm_ws(const qlora_tensor* t, int32_t count) {
  // one sum per CTA; a launch holds at least kMany tensors (or, past 2^31
  // blocks, one), so this bounds the launches of either form
  size_t launches = (size_t)count / kMany + 1;
  uint64_t blocks = 0;
  for (int32_t i = 0; i < count; ++i) blocks += (uint64_t)(t[i].n + kBlock - 1) / kBlock;
  launches += 2 * (size_t)(blocks / 0x7fffffffull);
  return align_up(launches * (size_t)sm_count() * kCtasPerSm * sizeof(double), 256);
}

cudaError_t launch_grad_norm(const qlora_tensor* t, int32_t count, float max_norm,
                             qlora_step_control* control, void* ws, cudaStream_t st) {
  double* part = (double*)ws;
  int32_t n = 0;
  cudaError_t e = count <= kFew    ? sumsq_all<kFew>(t, count, part, &n, st)
                  : count <= kSome ? sumsq_all<kSome>(t, count, part, &n, st)
                                   : sumsq_all<kMany>(t, count, part, &n, st);
  if (e != cudaSuccess) return e;
  // its launch overlaps the last sums; it waits for their grid itself
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n > 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, norm_kernel, (const double*)part, n, max_norm, control);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_adamw(const qlora_tensor* t, int32_t count, int32_t bits, int64_t step, float lr,
                         float beta1, float beta2, float eps, float weight_decay,
                         const qlora_step_control* control, cudaStream_t st) {
  AdamWArgs a = {};
  a.b1 = beta1;
  a.b2 = beta2;
  a.omb1 = (float)(1.0 - (double)beta1);
  a.omb2 = (float)(1.0 - (double)beta2);
  a.eps = eps;
  a.decay = (float)(1.0 - (double)lr * (double)weight_decay);
  a.lr = lr;
  a.b1d = beta1;
  a.b2d = beta2;
  a.control = control;
  a.z = -0.0f;
  if (!control) bias_terms(a.lr, a.b1d, a.b2d, step, &a.step_size, &a.inv_rbc2);
  return count <= kFew    ? adamw_all<kFew>(t, count, bits, a, st)
         : count <= kSome ? adamw_all<kSome>(t, count, bits, a, st)
                          : adamw_all<kMany>(t, count, bits, a, st);
}

}  // namespace qlora
